// Log probabilities of given tokens with the entropy and the top alternatives
// of each row, and their gradient.
//
// Row by row, with logits z (vocab values), a token t and temperature T:
//   u_j = (z_j - m) / T, m = max z      s = sum exp u_j      q_j = exp(u_j) / s
//   logprob = u_t - log s      entropy = -sum q_j log q_j = log s - sum exp(u_j) u_j / s
//   top alternatives: the k largest logits, equal ones by their index
//   dz_j = (gl ([j = t] - q_j) - ge q_j (log q_j + entropy)) / T
// Both terms of the entropy are at least 0 as they are computed too (s at least
// 1, its second sum at most 0), so nothing cancels between them, no entropy is
// negative and no log probability above 0.  s holds what lies beside the largest
// logit to half a unit of 1 for each addition that its 1 takes part in: a few
// 2^-24, absolute, is what log s and the entropy of a nearly certain row are off
// by.  Where a factor is u itself it is -200 (in powers of two) at least: below
// that exp(u) is 0 in fp32, and so is the product (u = -inf of a masked entry
// among them).  How many threads share a row depends on the number of rows and
// of alternatives, and with it the order of the sums: a row's last bits do too.
//
// Reading bounds long batches: 8192 x 128256 bf16 take 355 to 375 us without
// alternatives (5.6 to 5.9 TB/s; torch's sums and maxima of as long rows read at 5.8
// to 6.2), 382 to 396 with 64 of them; the gradient of 4096 x 50257 164 to 175 (4.7
// to 5.0 TB/s read and written).
#include <algorithm>

#include "model_internal.h"
#include "train_device.h"

namespace dion {

namespace {

constexpr float NEG = -__builtin_inff(), LOWEST = -3.402823466e+38f;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ __forceinline__ float factor(float v) { return fmaxf(v, -200.f); }

// While a row is read exponents are powers of two, v = z c - R with c = log2(e)
// / T and R = fl(m c), one fma each.  The rounding of R is the same in every
// term, as long as sums go from one reference to another by the rounded R's,
// and is taken out of the row's sums at their end.  References of a mask's
// size (|m c| from WIDE on), for which it would not stay small, are taken by
// differences instead: v = (z - m) c.
constexpr float WIDE = 0x1.fp18f, FLOOR = 0x1p19f;

// Sums over what was seen of a row, relative to its largest value m: s of 2^v
// and w of 2^v v.  FAR sums go by differences and start from the lowest finite
// value; the others from a floor (m c = -2^19), by which masked entries are 0:
// a row with nothing above it, or that is wide, is summed again by the former.
// A NaN or +inf makes s NaN.
template <bool FAR> struct Sums {
  float m, r, s, w;
  __device__ __forceinline__ static float start(float temp) { return FAR ? LOWEST : fmaxf(-(FLOOR * LN2) * temp, LOWEST); }
  __device__ __forceinline__ void clear(float temp, float c) { m = start(temp), r = m * c, s = w = 0.f; }
  __device__ __forceinline__ void to(float other, float c) {   // relative to another value, at least m
#pragma clang fp contract(off)   // R is rounded first
    const float o = other * c, d = FAR ? (m - other) * c : r - o, f = exp2_fast(d);
    w = f * (w + s * (FAR ? factor(d) : d));
    s *= f;
    m = other;
    r = o;
  }
  // N elements, summed by themselves before they join the others: a thread that
  // holds a likely token has an s near 1, and one exponential after another
  // would lose what it has below half a unit of that, always downwards.
  // CLAMP: for chunks with elements so far below m that v would be -inf
  template <bool CLAMP, int N> __device__ __forceinline__ void add(const float* z, float c) {
    float ps, pw;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = FAR ? (z[i] - m) * c : fmaf(z[i], c, -r), e = exp2_fast(v), ev = e * (FAR || CLAMP ? factor(v) : v);
      ps = i ? ps + e : e;
      pw = i ? pw + ev : ev;
    }
    s += ps;
    w += pw;
  }
  // all of it into other sums, which go on
  __device__ __forceinline__ void into(Sums& other, float c) {
    other.to(m, c);   // (m is the largest so far)
    other.s += s;
    other.w += w;
    s = w = 0.f;
  }
  // over the block, the same in every thread
  template <int NT> __device__ __forceinline__ void join(float c, float (*red)[NT / 64]) {
    constexpr int W = NT / 64;
    to(wave_max(m), c);
    s = wave_sum(s);
    w = wave_sum(w);
    const int lane = threadIdx.x & 63;
    if (lane == 0) red[0][threadIdx.x >> 6] = m, red[1][threadIdx.x >> 6] = s, red[2][threadIdx.x >> 6] = w;
    lds_barrier();
    m = red[0][lane % W];
    r = m * c;
    s = lane < W ? red[1][lane] : 0.f;
    w = lane < W ? red[2][lane] : 0.f;
    to(row_reduce<W>(lane < W ? m : LOWEST, LOWEST, MaxNan()), c);
    s = row_reduce<W>(s, 0.f, Add());
    w = row_reduce<W>(w, 0.f, Add());
    lds_barrier();   // red may be written again
    if (!FAR) {   // every v is larger by what R was rounded by, the largest one's 0 too
#pragma clang fp contract(off)   // off s rounds as the largest one's part of w did
      const float off = fmaf(m, c, -r), f = exp2_fast(off), inv = __builtin_amdgcn_rcpf(f);   // f is near 1
      w = (w - off * s) * inv;
      // s / f: f is a term of s and no term is negative, so 1 at least, exactly 1 of one logit alone
      const float q = s * inv;
      s = fmaf(fmaf(-q, f, s), inv, q);
    }
    w = w > 0.f ? 0.f : w;   // of terms that are 0 at most (NaN stays)
  }
  __device__ __forceinline__ bool wide(float c) const { return !(fabsf(m * c) < WIDE); }
};

// Logits as whole numbers in their order (-0 as 0).  What is no alternative,
// -inf, lies below ABSENT; NaN is taken as -inf.
constexpr uint32_t ABSENT = 0x00800000u;
__device__ __forceinline__ uint32_t key_of(float z) {
  const int u = __float_as_int(fmaxf(z, NEG) + 0.f);
  return (uint32_t)(u ^ (u >> 31 | (int)0x80000000));
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k ^ (k >> 31 ? 0x80000000u : ~0u)); }

// Additions to one sum: those of rows with more (LONG below) go on in another
// one, so that of 2^30 logits no sum has more than 1024 terms.  (Rows of 2^19
// logits, the longest with alternatives, have 128 at most.)
constexpr int RUN = 512;

constexpr int KEYS = 16, SUB = 8;   // keys a thread holds: of a row's groups, of a level below

template <int NT> struct TopShared {
  __attribute__((aligned(16))) int count[2][NT / 64];
  int total, listed[2];
  union {
    struct {   // of select()
      int entry[KEYS * (NT / 64)];
      int id[2][NT];    // the selected, ascending, of two levels in turn (k <= NT)
    };
    int near[2 * NT];   // groups that may hold one of the largest
  };
  __attribute__((aligned(16))) unsigned long long order[2 * NT];   // key above, the lower index first
  uint32_t group[KEYS * NT];   // the largest of each group (as they are, then as keys of a level)
};

// The sum of the waves' counts c, the same in every thread.
template <int NT> __device__ __forceinline__ int block_count(int c, TopShared<NT>& sh, int& turn) {
  constexpr int W = NT / 64;
  if ((threadIdx.x & 63) == 0) sh.count[turn][threadIdx.x >> 6] = c;
  lds_barrier();
  int total = 0;
#pragma unroll
  for (int w = 0; w < W; w += 4) {
    const intx4 v = *(const intx4*)(sh.count[turn] + w);
    total += v[0] + v[1] + v[2] + v[3];
  }
  turn ^= 1;
  return total;
}

// Places in a list in LDS for `mine` entries of each thread, in no order that
// matters: the first of the thread's.
__device__ __forceinline__ int places(int mine, int* listed) {
  int upto = mine;   // sums over the lanes so far, as in wave_reduce
  const auto add = [&](int other) { upto += other; };
  add(__builtin_amdgcn_update_dpp(0, upto, 0x111, 0xf, 0xf, false));
  add(__builtin_amdgcn_update_dpp(0, upto, 0x112, 0xf, 0xf, false));
  add(__builtin_amdgcn_update_dpp(0, upto, 0x114, 0xf, 0xf, false));
  add(__builtin_amdgcn_update_dpp(0, upto, 0x118, 0xf, 0xf, false));
  add(__builtin_amdgcn_update_dpp(0, upto, 0x142, 0xa, 0xf, false));
  add(__builtin_amdgcn_update_dpp(0, upto, 0x143, 0xc, 0xf, false));
  const int all = __builtin_amdgcn_readlane(upto, 63);
  if (all == 0) return 0;
  int at = 0;
  if ((threadIdx.x & 63) == 0) at = atomicAdd(listed, all);
  return __builtin_amdgcn_readfirstlane(at) + upto - mine;
}

// The k largest of the first `used` NT keys in sh.group, equal ones by their
// position: put(position, o) is called for each with its place o in the order
// of positions.  The k-th largest key is found bit by bit, by counting the
// keys that are at least as large.  For rare rows, so with little code and few
// registers.
template <int NT, typename Put>
__device__ __forceinline__ void select(int used, int k, TopShared<NT>& sh, Put put) {
  constexpr int W = NT / 64;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  uint32_t least = 0;
  int turn = 0;
#pragma unroll 1
  for (int b = 31; b >= 0; --b) {
    const uint32_t cand = least | 1u << b;
    int c = 0;
#pragma unroll 1
    for (int i = 0; i < used; ++i) c += (int)__popcll(__ballot(sh.group[i * NT + t] >= cand));
    const int total = block_count<NT>(c, sh, turn);
    if (total >= k) least = cand;
    if (total == k) break;
  }
  // what lies above it, and the first of those equal to it
#pragma unroll 1
  for (int i = 0; i < KEYS; ++i) {
    const uint32_t v = i < used ? sh.group[i * NT + t] : 0;
    const int e = (int)__popcll(__ballot(v > least)) | (int)__popcll(__ballot(i < used && v == least)) << 16;
    if (lane == 0) sh.entry[i * W + wave] = e;
  }
  lds_barrier();
  if (wave == 0) {   // exclusive sums in the order of positions
    constexpr int E = KEYS * W, PER = (E + 63) / 64;
    int v[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane * PER + i;
      v[i] = sum;
      sum += e < E ? sh.entry[e] : 0;
    }
    int before = sum;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
      const int up = __shfl_up(before, o);
      if (lane >= o) before += up;
    }
    if (lane == 63) sh.total = before;
    before -= sum;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (lane * PER + i < E) sh.entry[lane * PER + i] = before + v[i];
  }
  lds_barrier();
  const int need = k - (sh.total & 0xffff);
  const unsigned long long below = (1ull << lane) - 1;
#pragma unroll 1
  for (int i = 0; i < used; ++i) {
    const uint32_t v = sh.group[i * NT + t];
    const unsigned long long more = __ballot(v > least), same = __ballot(v == least);
    const int e = sh.entry[i * W + wave];
    const int gt = (e & 0xffff) + (int)__popcll(more & below), eq = (e >> 16) + (int)__popcll(same & below);
    if (v > least || (v == least && eq < need)) put(i * NT + t, gt + min(eq, need));
  }
  lds_barrier();
}

// A row's chunks one by one, for sums by differences.
template <typename Z, int NT>
__device__ __forceinline__ void far_sums(const Z* z, int vocab, float temp, float c, Sums<true>& S) {
  typedef Chunk<Z> C;
  S.clear(temp, c);
  Sums<true> part;
  part.clear(temp, c);
  int64_t j = threadIdx.x * C::N;
  while (j < vocab) {
    for (int i = 0; i < RUN && j < vocab; ++i, j += NT * C::N) {
      const uintx4 v = C::load(z, (int)j, vocab, NEG);
      const float top = C::largest(part.m, v);
      if (top > part.m) part.to(top, c);
      float f[C::N];
      C::unpack(v, f);
      part.template add<true, C::N>(f, c);
    }
    part.into(S, c);
  }
}

// The row's token and its logit; -1 where there is none inside the vocabulary.
template <typename Z> __device__ __forceinline__ int64_t token_of(const LogprobArgs& a, int64_t row, float& z) {
  if (!a.tok) return -1;
  const int64_t t = a.tok64 ? ((const int64_t*)a.tok)[row] : (int64_t)((const int32_t*)a.tok)[row];
  if (t < 0 || t >= a.vocab) return -1;
  z = to_f(((const Z*)a.z)[row * a.ldz + t]);
  return t;
}

// One row to a block, read once, chunk i NT + t of 16 bytes by thread t, AHEAD
// of them asked for before they are used.  With the alternatives (TOP), the
// largest of each group of 2^lg neighbouring chunks is kept in LDS: a bound
// that k or a few more groups reach is reached by k logits at least, and by
// none outside those groups, which are read again (from the caches) and their
// logits above it ranked against one another.  Where no such bound is found
// (many equal logits, or large ones side by side), the k groups with the
// largest maxima are taken, equal ones by their order: k other groups' maxima
// come before anything in the rest.  Then the same for parts of those groups,
// down to single logits.  A few rows are shared between gridDim.y blocks each,
// whose sums and alternatives k_logprobs_join puts together.
// Eight chunks ahead; six where 1024 threads look for alternatives, whose 128
// registers hold no more (bf16, six and eight with ten of them spilled, us: 256 x
// 50257 with 20 17.3 and 19.6, 64 x 128256 with 20 18.3 and 19.2, 600 x 50257 with
// 500 110 and 115; fp32 20.6 either way).
template <typename Z, int NT, bool TOP, bool LONG>
__global__ __launch_bounds__(NT, 4) void k_logprobs(LogprobArgs a, int lg) {
  typedef Chunk<Z> C;
  constexpr int N = C::N, AHEAD = NT == 1024 && TOP ? 6 : 8, STEP = NT * N;
  __shared__ float red[3][NT / 64];
  __shared__ TopShared<TOP ? NT : 64> sh;
  const float c = LOG2E / a.temp;
  const int t = threadIdx.x;
  const int first = a.parts ? (int)blockIdx.y * a.per : 0;   // this block's logits: a share of the row, or all
  const int vocab = a.parts ? min(a.per, a.vocab - first) : a.vocab;
  const int whole = vocab / STEP;   // steps in which every thread has a chunk
  uintx4 none4;
  {
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = NEG;
    none4 = C::pack(f);
  }
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const Z* z = (const Z*)a.z + row * a.ldz + first;
    float zt = 0.f;
    const int64_t token = a.parts ? -1 : token_of<Z>(a, row, zt);
    Sums<false> S;
    S.clear(a.temp, c);
    auto absorb = [&](const uintx4& v0, const uintx4& v1, int step) {   // two chunks at once
      float f[2][N], top = S.m, low = __builtin_inff();
      C::unpack(v0, f[0]);
      C::unpack(v1, f[1]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float most = NEG;
#pragma unroll
        for (int i = 0; i < N; i += 2) {
          most = max3(most, f[u][i], f[u][i + 1]);
          low = min3(low, f[u][i], f[u][i + 1]);
        }
        top = fmaxf(top, most);
        if (TOP) {
          if (lg >= 2) {
            most = fmaxf(most, lane_move<0xb1, 0xf>(most, most));   // lane xor 1
            most = fmaxf(most, lane_move<0x4e, 0xf>(most, most));   // lane xor 2
          }
          if (lg == 3) most = fmaxf(most, lane_move<0x141, 0xf>(most, most));   // the other half of 8
          if ((t & ((1 << lg) - 1)) == 0) sh.group[((step + u) * NT + t) >> lg] = __float_as_uint(most);
        }
      }
      if (top > S.m) S.to(top, c);
      if (!(fmaf(low, c, -S.r) > -200.f)) S.template add<true, 2 * N>(f[0], c);
      else S.template add<false, 2 * N>(f[0], c);
    };
    const int rest = vocab - whole * STEP;   // of the row, a chunk of some threads
    const uintx4 last = rest ? C::load(z + (int64_t)whole * STEP, min(t * N, rest), rest, NEG) : none4;
    const Z* p = z + t * N;
    auto fetch = [&](int i) {
      return i < whole ? *(const uintx4u*)(p + (int64_t)i * STEP) : i == whole ? (uintx4u)last : (uintx4u)none4;
    };
    const int steps = whole + (rest ? 1 : 0);
    uintx4 v[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) v[u] = fetch(u);
    Sums<false> R;
    if (LONG) R.clear(a.temp, c);
    for (int i = 0; i < steps; i += AHEAD) {
#pragma unroll
      for (int u = 0; u < AHEAD; u += 2) {
        if (i + u >= steps) break;
        absorb(v[u], v[u + 1], i + u);
        if (i + u + AHEAD < steps) {
          v[u] = fetch(i + u + AHEAD);
          v[u + 1] = fetch(i + u + 1 + AHEAD);
        }
      }
      if (LONG && (i & (2 * RUN - 1)) == 2 * RUN - AHEAD) S.into(R, c);
    }
    if (LONG) {
      S.into(R, c);
      S = R;
    }
    S.template join<NT>(c, red);
    float m = S.m, s = S.s, w = S.w;
    if (S.wide(c)) {   // rare: again, from the caches
      Sums<true> F;
      far_sums<Z, NT>(z, vocab, a.temp, c, F);
      F.template join<NT>(c, red);
      m = F.m, s = F.s, w = F.w;
    }
    // a row with nothing but -inf has no distribution: logprob -inf, entropy 0
    const bool none = s == 0.f;
    const float logs = logf(s), entropy = none ? 0.f : logs - w / s * LN2;
    auto logprob = [&](float v) { return none ? NEG : (v - m) / a.temp - logs; };
    if (t == 0) {
      if (a.parts) {
        a.parts[row * a.shares + blockIdx.y] = make_float4(m, s, w, 0.f);
      } else {
        if (a.tok) a.logprob[row] = token >= 0 ? logprob(zt) : 0.f;
        a.entropy[row] = entropy;
        if (a.stats) a.stats[row] = make_float4(m, s, entropy, logs);
      }
    }
    if constexpr (TOP) {
      int size = N << lg, n = (vocab + size - 1) / size, k = min(a.k, n);
      auto output = [&](int i, unsigned long long v) {   // place i
        const uint32_t best = (uint32_t)(v >> 32);
        if (a.parts) {
          a.list[(row * a.shares + blockIdx.y) * a.k + i] = best >= ABSENT ? v : 0;
        } else {
          a.top[row * a.k + i] = best >= ABSENT ? logprob(value_of(best)) : NEG;
          a.index[row * a.k + i] = best >= ABSENT ? (int64_t)(0xffffffffu - (uint32_t)v) : -1;
        }
      };
      auto pair = [&](uint32_t key, int id) {
        return (unsigned long long)key << 32 | (0xffffffffu - (uint32_t)(first + id));
      };
      bool done = false;
      {
        float held[KEYS];   // (written before the joins' barriers)
#pragma unroll
        for (int i = 0; i < KEYS; ++i) {
          const float v = __uint_as_float(sh.group[i * NT + t]);
          held[i] = i * NT + t < n ? v : NEG;
        }
        int turn = 0;
        auto reached = [&](uint32_t key) {
          const float bound = value_of(key);
          int c = 0;
#pragma unroll
          for (int i = 0; i < KEYS; ++i) c += (int)__popcll(__ballot(held[i] >= bound));
          return block_count<NT>(c, sh, turn);
        };
        // The bound: down from the largest in growing steps (half an exponent's
        // first), then between the last two.  Groups hold more than one logit above
        // it now and then: few enough that their lists hold those as well (k = 256
        // of 50257, 4096 rows: 165 us, 260 with as many groups as the lists have).
        const int few = min(NT + NT / 2, 2 * a.k + 64);
        const uint32_t top = max(key_of(m), ABSENT);
        uint32_t lo = top + 1, hi = top + 1, step = 1u << 22;
        int reach = 0;
        while (reach < a.k && lo > ABSENT) {
          hi = lo;
          lo = top - ABSENT > step ? top - step : ABSENT;
          step = step >> 31 ? ~0u : 2 * step;
          reach = reached(lo);
        }
        while (reach > few && hi - lo > 1) {
          const uint32_t mid = lo + (hi - lo) / 2;
          const int c = reached(mid);
          if (c >= a.k) lo = mid, reach = c;
          else hi = mid;
        }
        if (reach <= few) {
          const float bound = value_of(lo);
          if (t < 2) sh.listed[t] = 0;
          lds_barrier();
          uint32_t hits = 0;
#pragma unroll
          for (int i = 0; i < KEYS; ++i) hits |= held[i] >= bound ? 1u << i : 0;
          int at = places(__popc(hits), &sh.listed[0]);
          for (; hits; hits &= hits - 1) sh.near[at++] = (__ffs(hits) - 1) * NT + t;
          lds_barrier();
          for (int q0 = 0; q0 < reach << lg; q0 += NT) {
            const int q = q0 + t;
            float f[N];
            int j = vocab;
            if (q < reach << lg) j = ((sh.near[q >> lg] << lg) + (q & ((1 << lg) - 1))) * N;
            const uintx4 v = C::load(z, min(j, vocab), vocab, NEG);
            C::unpack(v, f);
#pragma unroll
            for (int e = 0; e < N; ++e) hits |= f[e] >= bound ? 1u << e : 0;
            at = places(__popc(hits), &sh.listed[1]);
            for (; hits; hits &= hits - 1) {
              const int e = __ffs(hits) - 1;
              float x = f[0];
#pragma unroll
              for (int o = 1; o < N; ++o) x = e == o ? f[o] : x;
              if (at < 2 * NT) sh.order[at] = pair(key_of(x), j + e);
              ++at;
            }
          }
          lds_barrier();
          const int found = sh.listed[1];
          if (found <= 2 * NT) {
            done = true;
            if (t == 0 && found < 2 * NT) sh.order[found] = 0;   // pairs are read
            lds_barrier();
            for (int i = t; i < found; i += NT) {
              const unsigned long long v = sh.order[i];
              int rank = 0;
#pragma unroll 4
              for (int o = 0; o < found; o += 2) {
                const ulonglong2 w = *(const ulonglong2*)(sh.order + o);
                rank += (w.x > v) + (w.y > v);
              }
              if (rank < a.k) output(rank, v);
            }
            for (int i = found + t; i < a.k; i += NT) output(i, 0);
          }
        }
      }
      if (!done) {
        int turn = 0;
        const int used = (n + NT - 1) / NT;
        lds_barrier();   // counts and lists may be written
#pragma unroll 1
        for (int i = 0; i < used; ++i) {
          const int g = i * NT + t;
          sh.group[g] = g < n ? key_of(__uint_as_float(sh.group[g])) : 0;
        }
        select<NT>(used, k, sh, [&](int g, int o) { sh.id[0][o] = g; });
#pragma unroll 1
        while (size > 1) {
          const int part = max(1, size / SUB), r = size / part;
          // the parts that lie in the row at all: only its last group may hold others, behind them
          const int parts = (vocab + part - 1) / part, last_id = sh.id[turn][k - 1], all = k * r;
          n = all - max(0, (last_id + 1) * r - parts);
          const int held = (all + NT - 1) / NT, from = turn;
#pragma unroll 1
          for (int i = 0; i < held; ++i) {
            const int q = i * NT + t;
            float top = NEG;
            if (q < all) {
              const int j = (sh.id[from][q / r] * r + q % r) * part;
              for (int e = 0; e < part; ++e)
                if (j + e < vocab) top = fmaxf(top, to_f(z[j + e]));
            }
            sh.group[q] = q < all ? key_of(top) : 0;
          }
          k = min(a.k, n);
          turn ^= 1;
          select<NT>(held, k, sh, [&](int q, int o) {
            sh.id[turn][o] = sh.id[from][q / r] * r + q % r;
            if (part == 1) sh.order[o] = pair(sh.group[q], sh.id[turn][o]);
          });
          size = part;
        }
        // in order: a bitonic sort of as many places as a power of two
        int places = 2;
        while (places < k) places *= 2;
        for (int i = t; i < places; i += NT)
          if (i >= k) sh.order[i] = 0;
        lds_barrier();
#pragma unroll 1
        for (int len = 2; len <= places; len *= 2)
#pragma unroll 1
          for (int d = len / 2; d > 0; d /= 2) {
            for (int q = t; q < places / 2; q += NT) {
              const int lo = q / d * 2 * d + q % d, hi = lo + d;
              const unsigned long long x = sh.order[lo], y = sh.order[hi];
              if ((x < y) == ((lo & len) == 0)) sh.order[lo] = y, sh.order[hi] = x;
            }
            lds_barrier();
          }
        for (int i = t; i < a.k; i += NT) output(i, i < k ? sh.order[i] : 0);
      }
      lds_barrier();   // the next row's groups may be written
    }
  }
}

// A few rows in shares: their sums relative to the row's largest logit, and the
// k first of the shares' alternatives.  Wave w walks list w, four at a time,
// until they are behind the k first: an alternative's place is the number of
// those before it in every list, one lane to a list.
constexpr int kShares = 16, kSharedTop = 32;
template <typename Z> __global__ __launch_bounds__(64 * kShares) void k_logprobs_join(LogprobArgs a) {
  __shared__ unsigned long long list[kShares * kSharedTop];
  const float c = LOG2E / a.temp;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, other = lane & 15;
  const int64_t row = blockIdx.x;
  const int n = a.shares * a.k;
  for (int i = t; i < n; i += 64 * kShares) list[i] = a.list[row * n + i];
  float zt = 0.f;
  const int64_t token = token_of<Z>(a, row, zt);
  const float4 p = lane < a.shares ? a.parts[row * a.shares + lane] : make_float4(LOWEST, 0.f, 0.f, 0.f);
  Sums<true> S;
  S.m = p.x, S.r = p.x * c, S.s = p.y, S.w = p.z;
  S.to(wave_max(S.m), c);
  const float m = S.m, s = wave_sum(S.s), w = wave_sum(S.w);
  const bool none = s == 0.f;
  const float logs = logf(s), entropy = none ? 0.f : logs - w / s * LN2;
  auto logprob = [&](float v) { return none ? NEG : (v - m) / a.temp - logs; };
  if (t == 0) {
    if (a.tok) a.logprob[row] = token >= 0 ? logprob(zt) : 0.f;
    a.entropy[row] = entropy;
    if (a.stats) a.stats[row] = make_float4(m, s, entropy, logs);
  }
  __syncthreads();
  // how many of list `other` are above v (the lists descend, absent ones are 0)
  auto above = [&](unsigned long long v) {
    int lo = 0, hi = other < a.shares ? a.k : 0;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (list[other * a.k + mid] > v) lo = mid + 1;
      else hi = mid;
    }
    return row16_reduce((float)lo, Add());
  };
  if (wave < a.shares)
    for (int i = lane >> 4;; i += 4) {
      const unsigned long long v = i < a.k ? list[wave * a.k + i] : 0;
      const int place = (int)above(v);
      const bool here = v != 0 && place < a.k;
      if (!__any(here)) break;
      if (here && other == 0) {
        a.top[row * a.k + place] = logprob(value_of((uint32_t)(v >> 32)));
        a.index[row * a.k + place] = (int64_t)(0xffffffffu - (uint32_t)v);
      }
    }
  if (a.k > 0 && wave == 0) {   // places without one
    for (int i = (int)above(0) + lane; i < a.k; i += 64) {
      a.top[row * a.k + i] = NEG;
      a.index[row * a.k + i] = -1;
    }
  }
}

// Gradient: a row to a block, or (few rows) its columns shared between
// gridDim.y blocks; U chunks of a thread asked for at once.
template <typename Z, int NT, int U>
__global__ __launch_bounds__(NT, 8) void k_logprobs_backward(LogprobArgs a) {
  typedef Chunk<Z> C;
  constexpr int N = C::N;
  const float c = LOG2E / a.temp, it = 1.f / a.temp;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const Z* z = (const Z*)a.z + row * a.ldz;
    Z* dz = (Z*)a.dz + row * a.ldd;
    int64_t token = a.tok ? (a.tok64 ? ((const int64_t*)a.tok)[row] : (int64_t)((const int32_t*)a.tok)[row]) : -1;
    if (token < 0 || token >= a.vocab) token = -1;
    const float gl = a.gl && token >= 0 ? a.gl[row] : 0.f, ge = a.ge ? a.ge[row] : 0.f;
    const float4 st = a.stats[row];   // m, s, entropy, log s
    const bool zero = (gl == 0.f && ge == 0.f) || st.y == 0.f;
    // q (gl + ge (log q + entropy)) = 2^v (slope + rise v) / s
    const float k = -it / st.y, rise = ge * LN2, slope = gl + ge * (st.z - st.w);
    const int64_t all = (int64_t)gridDim.y * NT * N;
    for (int64_t j0 = ((int64_t)blockIdx.y * NT + threadIdx.x) * N; j0 < a.vocab; j0 += U * all) {
      uintx4 in[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (!zero && j0 + u * all < a.vocab) in[u] = C::load(z, (int)(j0 + u * all), a.vocab, NEG);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = j0 + u * all;
        if (j >= a.vocab) break;
        float f[N] = {};
        if (!zero) {
          C::unpack(in[u], f);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float v = (f[i] - st.x) * c;
            f[i] = exp2_fast(v) * k * fmaf(rise, factor(v), slope);
          }
          if (token >= j && token < j + N) {
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (j + i == token) f[i] += gl * it;
          }
        }
        C::store(dz, (int)j, a.vocab, f);
      }
    }
  }
}

// Shares of a row, where a few rows are split (0: they are not), and the logits
// of one.  A row on one CU waits for its exponentials, and a second launch costs
// 2.5 to 5 (us, one CU a row and 16 shares: 1 x 128256 bf16 10.4 and 7.0, with 20
// alternatives 16.0 and 12.3, with 64 16.5 and 16.9; 1 x 32001 8.0 and 6.6, with
// 20 13.8 and 13.0; 64 x 128256 12.3 and 11.4, with 20 18.8 and 18.3).
int logprob_shares(int64_t rows, int vocab, int k, int& per) {
  if (rows == 0 || rows > 32 || k > kSharedTop || vocab < (k ? 49152 : 24576)) return 0;
  const int most = (int)std::min<int64_t>(kShares, 256 / rows);
  per = (int)(((int64_t)vocab + most - 1) / most + 4095) / 4096 * 4096;
  return (vocab + per - 1) / per;
}

template <typename Z, int NT, bool TOP>
void launch_rows(const LogprobArgs& a, int lg, hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>(a.rows, 1 << 20), (unsigned)(a.parts ? a.shares : 1));
  const bool runs = (a.parts ? a.per : a.vocab) > 2 * RUN * NT * Chunk<Z>::N;   // (TOP: never)
  if (!TOP && runs) hipLaunchKernelGGL((k_logprobs<Z, NT, false, true>), grid, dim3(NT), 0, s, a, lg);
  else hipLaunchKernelGGL((k_logprobs<Z, NT, TOP, false>), grid, dim3(NT), 0, s, a, lg);
}

// Threads of a row: 256, of which a CU holds four rows (104 to 128 registers; five
// of fp32 without alternatives, 88), or 1024 where there is a row to a CU at most
// and it is long, or the lists of 256 do not hold k (us,
// bf16, 256 and 1024 threads: 4096 x 50257 90 and 149, with 64 alternatives 116
// and 254; 300 x 128256 22 and 26, 33 and 38; 64 x 128256 16.5 and 12.0, 26.1 and
// 19.8; 64 x 65536 10.5 and 8.2, 18.4 and 15.6; 64 x 32001 7.1 and 7.1, 13.7 and
// 15.4; 64 x 8000 4.9 and 5.8, 11.4 and 14.1).
template <typename Z> void launch_forward(LogprobArgs a, hipStream_t s) {
  constexpr int N = Chunk<Z>::N;
  // groups of one, four or eight chunks, as many as the keys that the threads hold
  const auto groups = [&](int64_t nt, int64_t vocab) {
    return vocab <= nt * KEYS * N ? 0 : vocab <= nt * KEYS * N * 4 ? 2 : 3;
  };
  a.shares = logprob_shares(a.rows, a.vocab, a.k, a.per);
  if (a.shares && a.parts) {   // parts: checked scratch, wherever there are shares
    a.list = (uint64_t*)(a.parts + a.rows * a.shares);
    if (a.k) launch_rows<Z, 256, true>(a, groups(256, a.per), s);
    else launch_rows<Z, 256, false>(a, 0, s);
    hipLaunchKernelGGL((k_logprobs_join<Z>), dim3((unsigned)a.rows), dim3(64 * kShares), 0, s, a);
    return;
  }
  a.parts = nullptr;
  if (a.k == 0) {
    if (a.rows > 256 || a.vocab <= 256 * KEYS * N) launch_rows<Z, 256, false>(a, 0, s);
    else launch_rows<Z, 1024, false>(a, 0, s);
    return;
  }
  const bool small = a.k <= 256 && a.vocab <= 256 * KEYS * N * 8;
  if (small && (a.rows > 256 || a.vocab <= 256 * KEYS * N)) launch_rows<Z, 256, true>(a, groups(256, a.vocab), s);
  else launch_rows<Z, 1024, true>(a, groups(1024, a.vocab), s);
}

// 4096 x 50257 and 8192 x 128256 bf16 (us): 164 and 823 on 512 threads with two
// chunks and eight waves a SIMD, 165 and 828 on 256, 172 and 813 on 256 with
// four chunks and four waves, 183 and 909 with a piece of a row to a block in
// the order of addresses.
template <typename Z> void launch_gradient(const LogprobArgs& a, hipStream_t s) {
  constexpr int NT = 512, N = Chunk<Z>::N;
  const int64_t most = ((int64_t)a.vocab + NT * N - 1) / (NT * N);
  const int64_t share = std::max<int64_t>(1, std::min<int64_t>(most, 1024 / std::min<int64_t>(a.rows, 1024)));
  hipLaunchKernelGGL((k_logprobs_backward<Z, NT, 2>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20), (unsigned)share),
                     dim3(NT), 0, s, a);
}

}  // namespace

size_t logprob_scratch(int64_t rows, int vocab, int k, int) {
  int per = 0;
  const int shares = logprob_shares(rows, vocab, k, per);
  return (size_t)rows * shares * (16 + 8 * (size_t)k);
}

void launch_token_logprobs(int fmt, const LogprobArgs& a, hipStream_t s) {
  if (fmt == 1) launch_forward<float>(a, s);
  else if (fmt == 0) launch_forward<bf16_t>(a, s);
  else launch_forward<fp16_t>(a, s);
}

void launch_token_logprobs_backward(int fmt, const LogprobArgs& a, hipStream_t s) {
  if (fmt == 1) launch_gradient<float>(a, s);
  else if (fmt == 0) launch_gradient<bf16_t>(a, s);
  else launch_gradient<fp16_t>(a, s);
}

}  // namespace dion
