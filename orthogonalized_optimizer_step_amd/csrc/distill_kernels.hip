// Distillation loss on a teacher's top logits, and its gradient.
//
// Row by row, with student logits z (vocab values), teacher logits t_k at
// indices i_k and temperature T:
//   p = softmax of t / T over the present entries (index inside the
//   vocabulary, t_k > -inf);  q_j = exp((z_j - m) / T) / s with m = max z and
//   s = sum exp((z - m) / T)
//   loss = T^2 sum_k p_k (log p_k - log q_{i_k})   (terms with p_k = 0 are 0)
//   dz_j = gl T (q_j - sum over k with i_k = j of p_k)
// A row with no present entry has loss 0 and gradient 0, whatever z holds; a
// row whose loss has gradient gl = 0 has gradient 0.
//
// With c = log2(e) / T an exponential is 2^(z c - R), R = fl(m c): a fma and a
// v_exp_f32.  m need only be near the largest logit, and the rounding of R is
// the same in every term and cancels in q and in the loss.  Where |m c|
// reaches 2^20 (the largest of a row, or of what a thread has seen of it, is a
// mask's value) that rounding would not stay small: it would make infinite
// terms.  2^((z - m) c) is formed there instead.
#include <algorithm>

#include "train_device.h"
#include "train_internal.h"

namespace dion {

namespace {

constexpr float NEG = -__builtin_inff();
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Exponentials relative to the reference m: 2^((z - a) c - b), with a = 0 and
// b = R where R is small, a = m and b = 0 where it is not.  Sums relative to
// either kind meet exactly in of().
struct Ref {
  float m, c, a, b;
  bool wide, none;   // none: of nothing but -inf (a sum of 0)
  __device__ __forceinline__ Ref(float m_, float c_) : m(m_ == NEG ? 0.f : m_), c(c_), none(m_ == NEG) {
    const float R = m * c;
    wide = !(fabsf(R) < 0x1p20f);
    a = wide ? m : 0.f;
    b = wide ? 0.f : R;
  }
  __device__ __forceinline__ float exponent(float z) const { return fmaf(z - a, c, -b); }
  __device__ __forceinline__ float operator()(float z) const { return exp2_fast(exponent(z)); }
  __device__ __forceinline__ float near(float z) const { return exp2_fast(fmaf(z, c, -b)); }   // the same where !wide
  // log of the same
  __device__ __forceinline__ float log(float z) const { return exponent(z) * LN2; }
  // What a sum relative to `o` is worth here: by the rounded references, as its
  // terms were formed.  (One fused from the products, m c - R, would be off by
  // the rounding of R: 2^-5 where R is near 2^19, 2^-20 where it is near 20.)
  __device__ __forceinline__ float of(const Ref& o) const {
#pragma clang fp contract(off)
    return o.none ? 0.f : exp2_fast(fmaf(o.a - a, c, o.b - b));
  }
};

// Joins sums s relative to references m over a wave.
__device__ __forceinline__ void wave_join(float& m, float& s, float c) {
  const float mm = wave_max(m);
  s = wave_sum(s * Ref(mm, c).of(Ref(m, c)));
  m = mm;
}

// Joins the W values that the waves of a block left in LDS, the same in every lane.
template <int W> __device__ __forceinline__ float join_sum(const float* v) {
  const int lane = threadIdx.x & 63;
  return row_reduce<W>(lane < W ? v[lane] : 0.f, 0.f, Add());
}
template <int W> __device__ __forceinline__ float join_max(const float* v) {
  const int lane = threadIdx.x & 63;
  return row_reduce<W>(lane < W ? v[lane] : NEG, NEG, MaxNan());
}

// What the block knows of one row's teacher, in LDS.
template <int NT> struct Teacher {
  static constexpr int W = NT / 64, KPT = kDistillMaxK / NT;   // entries a thread holds
  __attribute__((aligned(16))) int idx[kDistillMaxK];   // -1 where absent; up to k rounded up to the wave
  __attribute__((aligned(16))) float e[kDistillMaxK];   // exp((t - top) / T), 0 where absent
  float fix[kDistillMaxK];   // the gradient at the entry
  float wm[W], ws[W], wt[W], wl[W], we[W];
  int live[W];
};

template <int NT> struct Entries {   // a thread's entries k = tid + i NT of a row
  static constexpr int KPT = kDistillMaxK / NT;
  float t[KPT];
  int idx[KPT];
  __device__ __forceinline__ void load(const DistillArgs& a, int64_t row) {
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      const int k = threadIdx.x + i * NT;
      t[i] = NEG;
      idx[i] = -1;
      if (i * NT < a.k && k < a.k) {
        const int64_t at = row * a.k + k;
        const int64_t j = a.idx64 ? ((const int64_t*)a.idx)[at] : (int64_t)((const int32_t*)a.idx)[at];
        const float v = load_fmt(a.t, at, a.t_fmt);
        if (j >= 0 && j < a.vocab && v != NEG) {
          t[i] = v;
          idx[i] = (int)j;
        }
      }
    }
  }
  __device__ __forceinline__ bool any() const {
    bool r = false;
#pragma unroll
    for (int i = 0; i < KPT; ++i) r |= idx[i] >= 0;
    return r;
  }
};

template <typename Z, int NT> struct Row {
  static constexpr int W = NT / 64, KPT = kDistillMaxK / NT;
  float m, s;        // the row's statistics
  // whether this wave holds any of the entries that its threads number i
  static __device__ __forceinline__ bool has(const DistillArgs& a, int i) {
    return i * NT + (int)(threadIdx.x & ~63u) < a.k;
  }
  float u[KPT];      // (t - top) / T of the thread's entries (NEG where absent)
  float zi[KPT];     // the student's logit there

  // Joins the threads' (m, s) (when FWD) and forms the teacher's distribution:
  // E.idx and .e of T are filled.  Two LDS barriers.
  template <bool FWD>
  __device__ __forceinline__ void join(const DistillArgs& a, const Entries<NT>& E, Teacher<NT>& T, float c) {
    const int tid = threadIdx.x, wave = tid >> 6;
    float top = NEG;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      if (has(a, i) && E.idx[i] >= 0) top = max_nan(top, E.t[i]);
    }
    top = wave_max(top);
    if (FWD) wave_join(m, s, c);
    if ((tid & 63) == 0) {
      T.wt[wave] = top;
      T.wm[wave] = m;
      T.ws[wave] = s;
    }
    lds_barrier();
    top = join_max<W>(T.wt);
    if (FWD) {
      m = join_max<W>(T.wm);
      const int lane = tid & 63;
      s = row_reduce<W>(lane < W ? T.ws[lane] * Ref(m, c).of(Ref(T.wm[lane], c)) : 0.f, 0.f, Add());
    }
    float es = 0.f;
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      if (has(a, i)) {
        u[i] = E.idx[i] >= 0 ? (E.t[i] - top) / a.temp : NEG;
        const float e = expf(u[i]);
        es += e;
        const int k = tid + i * NT;
        T.idx[k] = E.idx[i];
        T.e[k] = e;
      }
    }
    es = wave_sum(es);
    if ((tid & 63) == 0) T.we[wave] = es;
    lds_barrier();
    inv_es = 1.f / join_sum<W>(T.we);
  }
  float inv_es;

  // This thread's share of the loss over T^2.  With u the exponents of either
  // side it is sum p (u_t - u_z) + log(s / es): the logarithms of the two sums
  // enter once, as one, and not rounded into every entry's.
  __device__ __forceinline__ float loss(const DistillArgs& a, const Teacher<NT>& T, float c) const {
    const Ref r(m, c);
    float l = threadIdx.x == 0 ? logf(s * inv_es) : 0.f;
#pragma unroll
    for (int i = 0; i < KPT; ++i)
      if (has(a, i)) {
        const float p = T.e[threadIdx.x + i * NT] * inv_es;
        if (p != 0.f) l += p * (u[i] - r.log(zi[i]));
      }
    return l;
  }

  // the gradient at the thread's entries, into T.fix (entries in [lo, hi))
  __device__ __forceinline__ void fix(const DistillArgs& a, const Entries<NT>& E, Teacher<NT>& T, float c, float gt) const {
    const Ref r(m, c);
#pragma unroll
    for (int i = 0; i < KPT; ++i) {
      if (!has(a, i)) continue;
      float p = 0.f;   // every entry with this index
#pragma unroll 4
      for (int o = 0; o < a.k; o += 4) {
        const intx4 j = *(const intx4*)(T.idx + o);
        const floatx4 e = *(const floatx4*)(T.e + o);
#pragma unroll
        for (int q = 0; q < 4; ++q) p += j[q] == E.idx[i] ? e[q] : 0.f;
      }
      if (E.idx[i] < 0) continue;
      T.fix[threadIdx.x + i * NT] = gt * (r(zi[i]) / s - p * inv_es);
    }
  }

  // the student's logits at the entries in [lo, hi)
  __device__ __forceinline__ void gather(const DistillArgs& a, const Entries<NT>& E, const Z* z, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < KPT; ++i) zi[i] = has(a, i) && E.idx[i] >= lo && E.idx[i] < hi ? to_f(z[E.idx[i]]) : 0.f;
  }
};

// The entries whose element this wave wrote in its pass over the row: a wave's
// stores to one address keep their order, so no wait is needed between.
// Element j belongs to the wave of thread (j / N) % NT.
template <typename Z, int NT>
__device__ __forceinline__ void write_fixes(const DistillArgs& a, const Teacher<NT>& T, Z* dz, int lo, int hi) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int k = lane; k < a.k; k += 64) {
    const int j = T.idx[k];
    if (j >= lo && j < hi && (((j - lo) / Chunk<Z>::N) % NT) >> 6 == wave) dz[j] = from_f<Z>(T.fix[k]);
  }
}

// The running largest value and sum of elements [lo, hi) of a row, by the
// block's threads, AHEAD chunks at once.
template <typename Z, int NT, int AHEAD = 4>
__device__ __forceinline__ void stream_sum(const Z* z, int lo, int hi, float c, float& m, float& s) {
  typedef Chunk<Z> C;
  m = NEG;
  s = 0.f;
#pragma unroll AHEAD
  for (int j = lo + (int)threadIdx.x * C::N; j < hi; j += NT * C::N) {
    const uintx4 v = C::load(z, j, hi, NEG);
    float f[C::N];
    C::unpack(v, f);
    const float cm = C::largest(m, v);
    if (cm > m) {
      s *= Ref(cm, c).of(Ref(m, c));
      m = cm;
    }
    const Ref r(m, c);
#pragma unroll
    for (int i = 0; i < C::N; ++i) s += r(f[i]);
  }
}

// A few rows over a large vocabulary: one share of a row to a block, its
// statistics and the logits at the teacher's entries there into scratch, for
// k_distill_rows.
template <typename Z, int NT> __global__ __launch_bounds__(NT) void k_distill_part(DistillArgs a) {
  __shared__ float wm[NT / 64], ws[NT / 64];
  const float c = LOG2E / a.temp;
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t row = blockIdx.x;
  const int lo = (int)((int64_t)a.vocab * blockIdx.y / a.shares), hi = (int)((int64_t)a.vocab * (blockIdx.y + 1) / a.shares);
  const Z* z = (const Z*)a.z + row * a.ldz;
  for (int k = tid; k < a.k; k += NT) {
    const int64_t at = row * a.k + k;
    const int64_t j = a.idx64 ? ((const int64_t*)a.idx)[at] : (int64_t)((const int32_t*)a.idx)[at];
    if (j >= lo && j < hi) a.zi[at] = to_f(z[j]);
  }
  float m, s;
  stream_sum<Z, NT>(z, lo, hi, c, m, s);
  wave_join(m, s, c);
  if (lane == 0) {
    wm[tid >> 6] = m;
    ws[tid >> 6] = s;
  }
  __syncthreads();
  if (tid == 0) {
    m = NEG;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) m = fmaxf(m, wm[w]);
    s = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) s += ws[w] * Ref(m, c).of(Ref(wm[w], c));
    a.parts[row * a.shares + blockIdx.y] = make_float2(m, s);
  }
}

// Loss and statistics (FWD), gradient (BWD), or both with the row read a
// second time while it is still in the caches; without FWD the statistics are
// given, or (few rows) joined here from the shares' parts, and then the loss
// is formed too.  A block walks rows gridDim.x apart, fetching the teacher's
// entries and the logits at them a row ahead; few rows may be shared between
// gridDim.y blocks each (rows <= gridDim.x then).
template <typename Z, int NT, bool FWD, bool BWD>
__global__ __launch_bounds__(NT) void k_distill_rows(DistillArgs a) {
  typedef Chunk<Z> C;
  constexpr int W = NT / 64, KPT = kDistillMaxK / NT;
  __shared__ Teacher<NT> both[2];   // rows in turn, so that one may be written while the last is still read
  int turn = 0;
  const float c = LOG2E / a.temp;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  // this block's columns: whole chunks of all threads
  const int per = (int)(((int64_t)a.vocab + gridDim.y - 1) / gridDim.y + NT * C::N - 1) / (NT * C::N) * (NT * C::N);
  const int lo = min(a.vocab, (int)blockIdx.y * per), hi = min(a.vocab, lo + per);
  if (lo >= hi) return;
  const bool joins = FWD || a.parts;   // the loss is formed here
  auto gather = [&](Row<Z, NT>& R, const Entries<NT>& E, int64_t row) {
    if (a.parts) {
#pragma unroll
      for (int i = 0; i < KPT; ++i) R.zi[i] = E.idx[i] >= 0 ? a.zi[row * a.k + tid + i * NT] : 0.f;
    } else {
      R.gather(a, E, (const Z*)a.z + row * a.ldz, joins ? 0 : lo, joins ? a.vocab : hi);
    }
  };
  Entries<NT> E, En;
  Row<Z, NT> R, Rn;
  int64_t row = blockIdx.x;
  E.load(a, row);
  const bool mine = __any(E.any());
  if (lane == 0) both[1].live[wave] = mine;
  lds_barrier();
  bool live = __any(both[1].live[tid % W]);
  if (!FWD && live) gather(R, E, row);
  for (; row < a.rows; row += gridDim.x) {
    Teacher<NT>& T = both[turn];
    turn ^= 1;
    const Z* z = (const Z*)a.z + row * a.ldz;
    Z* dz = BWD ? (Z*)a.dz + row * a.ldd : nullptr;
    const int64_t next = row + gridDim.x;
    const bool more = next < a.rows;
    if (more) En.load(a, next);
    const float g = BWD && a.gl ? a.gl[row] : 1.f;
    const float gt = g * a.temp;
    const bool work = live && (joins || g != 0.f);   // beyond writing zeros
    if (work) {
      if (FWD) {
        stream_sum<Z, NT>(z, 0, a.vocab, c, R.m, R.s);
        gather(R, E, row);   // in the caches now
      } else if (a.parts) {
        const float2 p = lane < a.shares ? a.parts[row * a.shares + lane] : make_float2(NEG, 0.f);
        R.m = p.x;
        R.s = p.y;
        wave_join(R.m, R.s, c);
      } else {
        const float2 st = a.stats[row];
        R.m = st.x;
        R.s = st.y;
      }
      R.template join<FWD>(a, E, T, c);
      if (BWD) R.fix(a, E, T, c, gt);
      if (joins) {
        const float part = wave_sum(R.loss(a, T, c));
        if (lane == 0) T.wl[wave] = part;
      }
    }
    const bool some = __any(more && En.any());
    if (lane == 0) T.live[wave] = some;
    lds_barrier();
    const bool live_next = __any(T.live[tid % W]);
    if (joins && blockIdx.y == 0) {
      const float l = work ? join_sum<W>(T.wl) : 0.f;
      if (tid == 0) {
        if (a.loss) a.loss[row] = a.temp * a.temp * l;
        if (a.stats) a.stats[row] = work ? make_float2(R.m, R.s) : make_float2(0.f, 1.f);
      }
    }
    if (!FWD && live_next) gather(Rn, En, next);
    if (BWD) {
      if (!live || g == 0.f) {
        const float zero[C::N] = {};
        for (int j = lo + tid * C::N; j < hi; j += NT * C::N) C::store(dz, j, hi, zero);
      } else {
        const float k = gt / R.s;
        const Ref r(R.m, c);
#pragma unroll 4
        for (int j = lo + tid * C::N; j < hi; j += NT * C::N) {
          float f[C::N];
          C::unpack(C::load(z, j, hi, NEG), f);
#pragma unroll
          for (int i = 0; i < C::N; ++i) f[i] = r(f[i]) * k;
          C::store(dz, j, hi, f);
        }
        write_fixes<Z, NT>(a, T, dz, lo, hi);
      }
    }
    E = En;
    if (!FWD) {
#pragma unroll
      for (int i = 0; i < KPT; ++i) R.zi[i] = Rn.zi[i];
    }
    live = live_next;
  }
}

// Loss and gradient with the row held in registers: up to NC whole 16-byte
// chunks a thread (chunk i of thread t at element (i NT + t) N) and one more
// for the rest of the row, -inf past its end.  A block walks rows gridDim.x
// apart.  As it writes chunk i of one row's gradient it asks for chunk i of
// its next row, and takes the chunk that it asked for LAG steps before into
// that row's largest value and sum: a logit is read once (a block whose next
// row is not there or has no teacher loads its own again, for nothing), and the
// arithmetic of both passes runs while memory is busy.  The teacher's entries
// and the logits at them are fetched a row ahead too, for between two rows
// nothing else is under way.  8192 x 128256 bf16 takes 884 us (4.6 TB/s over
// the logits read and the gradients written); a plain pass that reads and
// writes rows in the same order takes 810, one in the order of addresses 670.
// Reading the row twice (k_distill_rows) takes 1218.
template <typename Z, int NT, int NC, int BLOCKS>
__global__ __launch_bounds__(NT, NT * BLOCKS / 256) void k_distill_step(DistillArgs a) {
  typedef Chunk<Z> C;
  constexpr int W = NT / 64, STEP = NT * C::N, LAG = 4;
  __shared__ Teacher<NT> both[2];   // rows in turn, so that one may be written while the last is still read
  int turn = 0;
  const float c = LOG2E / a.temp;
  const int tid = threadIdx.x, wave = tid >> 6, j0 = tid * C::N;
  const int whole = a.vocab / STEP, jt = whole * STEP + j0;   // chunks that every thread has; its place in the rest
  uintx4 data[NC], tail;
  auto values = [&](uintx4& d, float* v) {   // unpacked anew in each pass: held in 32 bits they would not fit
    asm volatile("" : "+v"(d));
    C::unpack(d, v);
  };
  auto fetch = [&](const Z* z, int i) {
    if (i < NC) data[i] = *(const uintx4u*)(z + i * STEP + j0);
    else tail = C::load(z, jt, a.vocab, NEG);
  };
  // The running largest value and the sum relative to it, from a floor on: a
  // thread whose first chunks are masked starts from the floor's reference, by
  // which they are 0, and not from one of the mask's size.  (8192 x 128256 bf16:
  // 887 us so, 901 with a Ref's way for such sizes in every term.)
  const auto floor = [&]() { return fmaxf(-(0x1p19f * LN2) * a.temp, -3.402823466e+38f); };
  float m = floor(), mR = m * c, s = 0.f;
  auto absorb = [&](uintx4& d) {
    float v[C::N];
    values(d, v);
    float cm = m;
#pragma unroll
    for (int e = 0; e < C::N; e += 2) cm = max3(cm, v[e], v[e + 1]);
    if (cm > m) {
#pragma clang fp contract(off)   // R is rounded first
      const float R = cm * c;
      s *= exp2_fast(mR - R);
      mR = R;
      m = cm;
    }
#pragma unroll
    for (int e = 0; e < C::N; ++e) s += exp2_fast(fmaf(v[e], c, -mR));
  };
  Entries<NT> E, En;
  int64_t row = blockIdx.x;
  E.load(a, row);
  if (__any(E.any()) && (tid & 63) == 0) both[1].live[wave] = 1;
  else if ((tid & 63) == 0) both[1].live[wave] = 0;
  lds_barrier();
  bool live = __any(both[1].live[tid % W]);
  Row<Z, NT> R, Rn;
  {
    const Z* z = (const Z*)a.z + row * a.ldz;
    R.gather(a, E, z, 0, a.vocab);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (i < whole) fetch(z, i);
    if (jt < a.vocab) fetch(z, NC);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (i < whole) absorb(data[i]);
    if (jt < a.vocab) absorb(tail);
  }
  for (; row < a.rows; row += gridDim.x) {
    const Z* z = (const Z*)a.z + row * a.ldz;
    Z* dz = (Z*)a.dz + row * a.ldd;
    const int64_t next = row + gridDim.x;
    const bool more = next < a.rows;
    if (more) En.load(a, next);
    const float g = a.gl ? a.gl[row] : 1.f;
    Teacher<NT>& T = both[turn];
    turn ^= 1;
    R.m = m;
    R.s = s;
    float k = 0.f;
    bool zero = true;
    if (live) {
      R.template join<true>(a, E, T, c);
      if (R.m == floor() || Ref(R.m, c).wide) {   // of masks' values alone, or as large: rare, so from memory again
        stream_sum<Z, NT, 1>(z, 0, a.vocab, c, R.m, R.s);
        R.template join<true>(a, E, T, c);
      }
      R.fix(a, E, T, c, g * a.temp);
      const float part = wave_sum(R.loss(a, T, c));
      if ((tid & 63) == 0) T.wl[wave] = part;
      k = g * a.temp / R.s;
      zero = g == 0.f;
    }
    const bool some = __any(more && En.any());
    if ((tid & 63) == 0) T.live[wave] = some;
    lds_barrier();
    const bool live_next = __any(T.live[tid % W]);
    const float l = live ? join_sum<W>(T.wl) : 0.f;
    if (tid == 0) a.loss[row] = a.temp * a.temp * l;
    const Z* zn = live_next ? (const Z*)a.z + next * a.ldz : z;   // without a next row the loads are for nothing
    const Ref r(R.m, c);
    const bool apart = zero || r.wide;
    if (apart) {   // rare: from memory
      for (int j = j0; j < a.vocab; j += STEP) {
        float v[C::N] = {};
        if (!zero) C::unpack(C::load(z, j, a.vocab, NEG), v);
#pragma unroll
        for (int e = 0; e < C::N; ++e) v[e] = zero ? 0.f : r(v[e]) * k;
        C::store(dz, j, a.vocab, v);
      }
    }
    if (live_next) Rn.gather(a, En, zn, 0, a.vocab);
    m = floor();
    mR = m * c;
    s = 0.f;
    auto write = [&](uintx4& d, int i) {
      float v[C::N];
      values(d, v);
#pragma unroll
      for (int e = 0; e < C::N; ++e) v[e] = r.near(v[e]) * k;
      if (!apart) {
        if (i < NC) __builtin_nontemporal_store(C::pack(v), (uintx4u*)(dz + i * STEP + j0));
        else C::store(dz, jt, a.vocab, v);
      }
      fetch(zn, i);
    };
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (i < whole) {
        write(data[i], i);
        if (i >= LAG) absorb(data[i - LAG]);
      }
    if (jt < a.vocab) write(tail, NC);
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (i < whole && i >= whole - LAG) absorb(data[i]);
    if (jt < a.vocab) absorb(tail);
    if (!zero) write_fixes<Z, NT>(a, T, dz, 0, a.vocab);
    E = En;
#pragma unroll
    for (int i = 0; i < Row<Z, NT>::KPT; ++i) R.zi[i] = Rn.zi[i];
    live = live_next;
  }
}

}  // namespace

// Shares of a row, where a few rows are split (0: they are not).  It costs a
// launch, and pays from 128 KB a row with the gradient (4 x 129000 fp16: 31 us
// on one CU a row, 18 split), from 320 KB without (5 x 50257 fp32: 10 on one
// CU, 15 split).  Shares of 8192 logits at least, two blocks to a CU at most.
static int distill_shares(int64_t rows, int vocab, int fmt, bool gradient) {
  const int64_t bytes = (int64_t)vocab * (fmt == 1 ? 4 : 2);
  if (rows > 128 || rows == 0 || bytes < (gradient ? 128 : 320) << 10) return 0;
  return (int)std::min<int64_t>(std::min<int64_t>(64, vocab / 8192), 512 / rows);
}

size_t distill_scratch(int64_t rows, int vocab, int k, int fmt, bool gradient) {
  const int shares = distill_shares(rows, vocab, fmt, gradient);
  return shares ? ((size_t)rows * shares * 8 + (size_t)rows * k * 4 + 255) / 256 * 256 : 0;
}

template <typename Z> constexpr int format_of() { return sizeof(Z) == 4 ? 1 : 0; }   // by size: all that shares go by

template <typename Z, bool FWD, bool BWD>
static void launch_rows(const DistillArgs& a, hipStream_t s) {
  // One row to a block: of 1024 threads where there are at most as many rows
  // as CUs (the gradient's are shared out to fill the CUs), of 256 for short
  // rows, eight of them to a CU, of 512 otherwise.  The gradient's blocks stay
  // and walk their rows; the loss' rows each get a block of their own.
  const int64_t most = BWD ? 1 : 1 << 10;
  if (a.rows <= 256) {
    const int64_t share = !FWD && BWD ? std::min<int64_t>(256 / a.rows, (a.vocab + 16383) / 16384) : 1;
    hipLaunchKernelGGL((k_distill_rows<Z, 1024, FWD, BWD>), dim3((unsigned)a.rows, (unsigned)share), dim3(1024), 0, s, a);
  } else if (a.vocab <= 256 * 8 * Chunk<Z>::N) {
    hipLaunchKernelGGL((k_distill_rows<Z, 256, FWD, BWD>), dim3((unsigned)std::min<int64_t>(a.rows, 2048 * most)),
                       dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_distill_rows<Z, 512, FWD, BWD>), dim3((unsigned)std::min<int64_t>(a.rows, 1024 * most)),
                       dim3(512), 0, s, a);
  }
}

// A few rows in shares: the parts, then the loss (and the gradient).
template <typename Z, bool BWD>
static bool launch_shared(DistillArgs a, hipStream_t s) {
  a.shares = distill_shares(a.rows, a.vocab, format_of<Z>(), BWD);
  if (!a.shares || !a.parts) return false;   // parts: checked scratch, wherever there are shares
  a.zi = (float*)(a.parts + a.rows * a.shares);
  const dim3 grid((unsigned)a.rows, (unsigned)a.shares);
  hipLaunchKernelGGL((k_distill_part<Z, 256>), grid, dim3(256), 0, s, a);
  hipLaunchKernelGGL((k_distill_rows<Z, 256, false, BWD>), BWD ? grid : dim3((unsigned)a.rows), dim3(256), 0, s, a);
  return true;
}

template <typename Z>
static void launch_forward(const DistillArgs& a, hipStream_t s) {
  if (launch_shared<Z, false>(a, s)) return;
  DistillArgs b = a;
  b.parts = nullptr;
  launch_rows<Z, true, false>(b, s);
}

template <typename Z, int NT, int NC, int BLOCKS>
static void launch_held(const DistillArgs& a, hipStream_t s) {
  const int64_t most = 256 * BLOCKS;   // as many blocks as the CUs hold at once
  hipLaunchKernelGGL((k_distill_step<Z, NT, NC, BLOCKS>), dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(NT), 0, s, a);
}

template <typename Z>
static void launch_step(const DistillArgs& a, hipStream_t s) {
  constexpr int N = Chunk<Z>::N;
  if (launch_shared<Z, true>(a, s)) return;
  DistillArgs b = a;
  b.parts = nullptr;
  if (a.vocab < 256 * 9 * N) launch_held<Z, 256, 8, 4>(b, s);
  else if (a.vocab < 512 * 9 * N) launch_held<Z, 512, 8, 2>(b, s);
  else if (a.vocab < 512 * 17 * N) launch_held<Z, 512, 16, 2>(b, s);
  else if (a.vocab < 1024 * 17 * N) launch_held<Z, 1024, 16, 1>(b, s);
  else launch_rows<Z, true, true>(b, s);
}

#define DION_DISTILL(F, fmt, a, s)            \
  do {                                        \
    if (fmt == 1) F<float>(a, s);             \
    else if (fmt == 0) F<bf16_t>(a, s);       \
    else F<fp16_t>(a, s);                     \
  } while (0)

template <typename Z> static void launch_gradient(const DistillArgs& a, hipStream_t s) { launch_rows<Z, false, true>(a, s); }

void launch_distill_forward(int fmt, const DistillArgs& a, hipStream_t s) { DION_DISTILL(launch_forward, fmt, a, s); }
void launch_distill_backward(int fmt, const DistillArgs& a, hipStream_t s) { DION_DISTILL(launch_gradient, fmt, a, s); }
void launch_distill_step(int fmt, const DistillArgs& a, hipStream_t s) { DION_DISTILL(launch_step, fmt, a, s); }

}  // namespace dion
