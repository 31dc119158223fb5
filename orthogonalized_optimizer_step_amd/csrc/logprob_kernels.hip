// Log probabilities of given tokens with the entropy and the top alternatives
// of each row, and their gradient.
//
// Row by row, with logits z (vocab values), a token t and temperature T:
//   u_j = (z_j - m) / T, m = max z      s = sum exp u_j      q_j = exp(u_j) / s
//   logprob = u_t - log s      entropy = -sum q_j log q_j = log s - sum exp(u_j) u_j / s
//   top alternatives: the k largest logits, equal ones by their index
//   dz_j = (gl ([j = t] - q_j) - ge q_j (log q_j + entropy)) / T
// Both terms of the entropy are at least 0, so nothing cancels however little
// of it there is.  Where a factor is u itself it is -200 (in powers of two) at
// least: below that exp(u) is 0 in fp32, and so is the product (u = -inf of a
// masked entry among them).
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
  // CLAMP: for chunks with elements so far below m that v would be -inf
  template <bool CLAMP, int N> __device__ __forceinline__ void add(const float* z, float c) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = FAR ? (z[i] - m) * c : fmaf(z[i], c, -r), e = exp2_fast(v);
      s += e;
      w += e * (FAR || CLAMP ? factor(v) : v);
    }
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
    if (!FAR) {   // every v is larger by what R was rounded by
      const float off = fmaf(m, c, -r), f = exp2_fast(-off);
      w = (w - off * s) * f;
      s *= f;
    }
  }
  __device__ __forceinline__ bool wide(float c) const { return !(fabsf(m * c) < WIDE); }
};

// Logits as whole numbers in their order, -inf and NaN as 0 (no alternative), -0 as 0.
template <typename Z> struct Key {
  static constexpr int BITS = 8 * sizeof(Z), MANTISSA = sizeof(Z) == 4 ? 23 : sizeof(Z) == 2 && (float)(Z)257.f == 257.f ? 10 : 7;
  static __device__ __forceinline__ uint32_t of(float z) {
    union { Z z; uint16_t h; uint32_t w; } c;
    c.w = 0;
    c.z = (Z)(z + 0.f);
    const uint32_t u = sizeof(Z) == 2 ? c.h : c.w, sign = 1u << (BITS - 1), all = sign | (sign - 1);
    return z > NEG ? (u & sign ? ~u & all : u | sign) : 0u;
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    const uint32_t sign = 1u << (BITS - 1), all = sign | (sign - 1), u = k & sign ? k ^ sign : ~k & all;
    union { Z z; uint16_t h; uint32_t w; } c;
    if (sizeof(Z) == 2) c.h = (uint16_t)u;
    else c.w = u;
    return (float)c.z;
  }
};

constexpr int KEYS = 16, SUB = 8;   // keys a thread holds: of a row's groups, of a level below

template <int NT> struct TopShared {
  __attribute__((aligned(16))) int count[2][NT / 64];
  int total, listed[2];
  union {
    struct {   // of select()
      int entry[KEYS * (NT / 64)];
      int id[2][NT];                                            // the selected, ascending, of two levels in turn (k <= NT)
      uint32_t key[NT];
    };
    int near[2 * NT];   // groups that may hold one of the largest
  };
  __attribute__((aligned(16))) unsigned long long order[2 * NT];   // key above, the lower index first
  uint32_t group[KEYS * NT];                                    // the largest of each group, as keys
};

// How many of the block's n keys are at least `least`, the same in every thread.
// (key(i): key i of the thread, the first `used` of K.)
template <int NT, int K, typename Key>
__device__ __forceinline__ int count_keys(Key key, int used, uint32_t least, TopShared<NT>& sh, int& turn) {
  constexpr int W = NT / 64;
  int c = 0;
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (i < used) c += __popcll(__ballot(key(i) >= least));
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

// Lanes with `yes` get places in a list in LDS, in no order that matters; the
// others a place behind any list's end.
__device__ __forceinline__ int place(bool yes, int* listed) {
  const unsigned long long all = __ballot(yes);
  if (!all) return 1 << 30;
  int at = 0;
  if ((threadIdx.x & 63) == 0) at = atomicAdd(listed, (int)__popcll(all));
  at = __builtin_amdgcn_readfirstlane(at);
  return yes ? at + (int)__popcll(all & ((1ull << (threadIdx.x & 63)) - 1)) : 1 << 30;
}

// The k largest of n <= K NT keys (key i of thread t has position i NT + t),
// equal ones by their position: put(i, o) is called for each with its place o
// in the order of positions.  The k-th largest key is found bit by bit, by
// counting the keys that are at least as large.
template <int NT, int K, int BITS, typename Key, typename Put>
__device__ __forceinline__ void select(Key key, int n, int k, TopShared<NT>& sh, Put put) {
  constexpr int W = NT / 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int used = (n + NT - 1) / NT;
  uint32_t least = 0;
  int turn = 0;
  for (int b = BITS - 1; b >= 0; --b) {
    const uint32_t cand = least | 1u << b;
    const int total = count_keys<NT, K>(key, used, cand, sh, turn);
    if (total >= k) least = cand;
    if (total == k) break;
  }
  // what lies above it, and the first of those equal to it
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const uint32_t v = key(i);
    const int e = __popcll(__ballot(v > least)) | __popcll(__ballot(v == least)) << 16;
    if (lane == 0) sh.entry[i * W + wave] = e;
  }
  lds_barrier();
  if (wave == 0) {   // exclusive sums in the order of positions
    constexpr int E = K * W, PER = (E + 63) / 64;
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
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const uint32_t v = key(i);
    const unsigned long long more = __ballot(v > least), same = __ballot(v == least);
    const int e = sh.entry[i * W + wave];
    const int gt = (e & 0xffff) + __popcll(more & below), eq = (e >> 16) + __popcll(same & below);
    if (v > least || (v == least && eq < need)) put(i, gt + min(eq, need));
  }
  lds_barrier();
}

// The rest of a row's chunks one by one, for sums by differences.
template <typename Z, int NT>
__device__ __forceinline__ void far_sums(const Z* z, int vocab, float temp, float c, Sums<true>& S) {
  typedef Chunk<Z> C;
  S.clear(temp, c);
  for (int64_t j = threadIdx.x * C::N; j < vocab; j += NT * C::N) {
    const uintx4 v = C::load(z, (int)j, vocab, NEG);
    const float top = C::largest(S.m, v);
    if (top > S.m) S.to(top, c);
    float f[C::N];
    C::unpack(v, f);
    S.template add<true, C::N>(f, c);
  }
}

// One row to a block, read once, chunk i NT + t of 16 bytes by thread t, U of
// them at once and the next U asked for before they are used.  With the
// alternatives (TOP), the largest of each group of 2^lg neighbouring chunks is
// kept in LDS, for the k largest logits lie in the k groups with the largest
// maxima (equal ones by their order): k other groups' maxima come before
// anything in the rest.  The same again for parts of those groups, which are
// in the caches, down to single logits.
template <typename Z, int NT, bool TOP>
__global__ __launch_bounds__(NT, 4) void k_logprobs(LogprobArgs a, int lg) {
  typedef Chunk<Z> C;
  constexpr int N = C::N, U = 4, STEP = NT * N;
  __shared__ float red[3][NT / 64];
  __shared__ TopShared<TOP ? NT : 64> sh;
  const float c = LOG2E / a.temp;
  const int t = threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const Z* z = (const Z*)a.z + row * a.ldz;
    int64_t token = -1;
    float zt = 0.f;
    if (a.tok) {
      token = a.tok64 ? ((const int64_t*)a.tok)[row] : (int64_t)((const int32_t*)a.tok)[row];
      if (token >= 0 && token < a.vocab) zt = to_f(z[token]);
      else token = -1;
    }
    Sums<false> S;
    S.clear(a.temp, c);
    auto absorb = [&](const uintx4 (&v)[U], int step) {
#pragma unroll
      for (int h = 0; h < U; h += 2) {   // two chunks: as many values as there are registers for
        float f[2][N], top = S.m, low = __builtin_inff();
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          C::unpack(v[h + u], f[u]);
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
            if ((t & ((1 << lg) - 1)) == 0) sh.group[((step + h + u) * NT + t) >> lg] = Key<Z>::of(most);
          }
        }
        if (top > S.m) S.to(top, c);
        if (!(fmaf(low, c, -S.r) > -200.f)) {
          S.template add<true, N>(f[0], c);
          S.template add<true, N>(f[1], c);
        } else {
          S.template add<false, N>(f[0], c);
          S.template add<false, N>(f[1], c);
        }
      }
    };
    const int whole = a.vocab / STEP / U * U;   // steps in batches of whole chunks
    if (whole > 0) {
      uintx4 v[U], next[U];
      const Z* p = z + t * N;
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = *(const uintx4u*)(p + (int64_t)u * STEP);
      for (int i = 0; i < whole; i += U) {
        if (i + U < whole) {
#pragma unroll
          for (int u = 0; u < U; ++u) next[u] = *(const uintx4u*)(p + (int64_t)(i + U + u) * STEP);
        }
        absorb(v, i);
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = next[u];
      }
    }
    if ((int64_t)whole * STEP < a.vocab) {   // fewer than U steps and a part of one
      uintx4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t j = (int64_t)(whole + u) * STEP + t * N;
        v[u] = C::load(z, (int)min(j, (int64_t)a.vocab), a.vocab, NEG);
      }
      absorb(v, whole);
    }
    S.template join<NT>(c, red);
    float m = S.m, s = S.s, w = S.w;
    if (S.wide(c)) {   // rare: again, from the caches
      Sums<true> F;
      far_sums<Z, NT>(z, a.vocab, a.temp, c, F);
      F.template join<NT>(c, red);
      m = F.m, s = F.s, w = F.w;
    }
    // a row with nothing but -inf has no distribution: logprob -inf, entropy 0
    const bool none = s == 0.f;
    const float logs = logf(s), entropy = none ? 0.f : logs - w / s * LN2;
    auto logprob = [&](float v) { return none ? NEG : (v - m) / a.temp - logs; };
    if (t == 0) {
      if (a.tok) a.logprob[row] = token >= 0 ? logprob(zt) : 0.f;
      a.entropy[row] = entropy;
      if (a.stats) a.stats[row] = make_float4(m, s, entropy, logs);
    }
    if constexpr (TOP) {
      int size = N << lg, n = (a.vocab + size - 1) / size, k = min(a.k, n), turn = 0;
      auto output = [&](int i, unsigned long long v) {   // place i
        const uint32_t best = (uint32_t)(v >> 32);
        a.top[row * a.k + i] = best ? logprob(Key<Z>::value(best)) : NEG;
        a.index[row * a.k + i] = best ? (int64_t)(0xffffffffu - (uint32_t)v) : -1;
      };
      auto pair = [&](uint32_t key, int id) { return (unsigned long long)key << 32 | (0xffffffffu - (uint32_t)id); };
      bool done = false;
      {
        const auto key = [&](int i) { return i * NT + t < n ? sh.group[i * NT + t] : 0u; };   // (written before the joins' barriers)
        // A bound that few groups reach, k or more of them where there are as
        // many: down from the largest in growing steps, then between the last two.
        const int used = (n + NT - 1) / NT, few = min(2 * NT, 2 * a.k + 64);
        const uint32_t top = Key<Z>::of(m);
        uint32_t lo = top + 1, hi = top + 1, step = 1u << (Key<Z>::MANTISSA - 1);
        int reach = 0;
        while (reach < a.k && lo > 1) {
          hi = lo;
          lo = top > step ? top - step + 1 : 1;
          step = step >> 31 ? ~0u : 2 * step;
          reach = count_keys<NT, KEYS>(key, used, lo, sh, turn);
        }
        while (reach > few && hi - lo > 1) {
          const uint32_t mid = lo + (hi - lo) / 2;
          const int c = count_keys<NT, KEYS>(key, used, mid, sh, turn);
          if (c >= a.k) lo = mid, reach = c;
          else hi = mid;
        }
        if (reach <= few) {
          // everything that reaches it lies in them; each is ranked against all others
          if (t < 2) sh.listed[t] = 0;
          lds_barrier();
#pragma unroll
          for (int i = 0; i < KEYS; ++i)
            if (i < used) {
              const int at = place(key(i) >= lo, &sh.listed[0]);
              if (at < few) sh.near[at] = i * NT + t;
            }
          lds_barrier();
          for (int q0 = 0; q0 < reach << lg; q0 += NT) {
            const int q = q0 + t;
            float f[N];
            int j = a.vocab;
            if (q < reach << lg) j = ((sh.near[q >> lg] << lg) + (q & ((1 << lg) - 1))) * N;
            C::unpack(C::load(z, min(j, a.vocab), a.vocab, NEG), f);
#pragma unroll
            for (int e = 0; e < N; ++e) {
              const uint32_t v = Key<Z>::of(f[e]);
              const int at = place(v >= lo, &sh.listed[1]);
              if (at < 2 * NT) sh.order[at] = pair(v, j + e);
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
              for (int o = 0; o < found; o += 2) {
                const ulonglong2 w = *(const ulonglong2*)(sh.order + o);
                rank += (w.x > v) + (w.y > v);
              }
              if (rank < a.k) output(rank, v);
            }
            for (int i = found + t; i < a.k; i += NT) output(i, 0);
          }
        }
        if (!done) {   // many equal ones, or large ones side by side: exactly the k groups
          lds_barrier();   // the counts may be written
          select<NT, KEYS, Key<Z>::BITS>(key, n, k, sh, [&](int i, int o) { sh.id[0][o] = i * NT + t; });
        }
        turn = 0;
      }
      while (!done && size > 1) {
        const int part = max(1, size / SUB), r = size / part;
        uint32_t sub[SUB];
        int id[SUB];
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
          const int q = i * NT + t;
          sub[i] = 0;
          id[i] = 0;
          if (q < k * r) {
            id[i] = sh.id[turn][q / r] * r + q % r;
            const int j = id[i] * part;
            float top = NEG;
            for (int e = 0; e < part; ++e)
              if (j + e < a.vocab) top = fmaxf(top, to_f(z[j + e]));
            sub[i] = Key<Z>::of(top);
          }
        }
        // the parts that lie in the row at all: only its last group may hold others, behind them
        const int parts = (a.vocab + part - 1) / part, last = sh.id[turn][k - 1];
        n = k * r - max(0, (last + 1) * r - parts);
        k = min(a.k, n);
        turn ^= 1;
        select<NT, SUB, Key<Z>::BITS>([&](int i) { return sub[i]; }, n, k, sh, [&](int i, int o) {
          sh.id[turn][o] = id[i];
          sh.key[o] = sub[i];
        });
        size = part;
      }
      if (!done) {   // in order: a bitonic sort of as many places as a power of two
        int places = 2;
        while (places < k) places *= 2;
        for (int i = t; i < places; i += NT) sh.order[i] = i < k ? pair(sh.key[i], sh.id[turn][i]) : 0;
        lds_barrier();
        for (int len = 2; len <= places; len *= 2)
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

// Gradient: columns shared between gridDim.y blocks.
template <typename Z, int NT>
__global__ __launch_bounds__(NT) void k_logprobs_backward(LogprobArgs a) {
  typedef Chunk<Z> C;
  constexpr int N = C::N, U = 4;
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

template <typename Z, int NT, bool TOP>
void launch_rows(const LogprobArgs& a, int lg, hipStream_t s) {
  hipLaunchKernelGGL((k_logprobs<Z, NT, TOP>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(NT), 0, s, a, lg);
}

template <typename Z> void launch_forward(const LogprobArgs& a, hipStream_t s) {
  constexpr int N = Chunk<Z>::N;
  if (a.k == 0) {
    if (a.rows > 256 || a.vocab <= 256 * 8 * N) launch_rows<Z, 256, false>(a, 0, s);
    else launch_rows<Z, 1024, false>(a, 0, s);
    return;
  }
  // groups of one, four or eight chunks, as many as the keys that the threads hold
  const auto groups = [&](int64_t nt) { return a.vocab <= nt * KEYS * N ? 0 : a.vocab <= nt * KEYS * N * 4 ? 2 : 3; };
  const bool small = a.k <= 256 && a.vocab <= 256 * KEYS * N * 8;
  if (small && (a.rows > 256 || a.vocab <= 256 * 8 * N)) launch_rows<Z, 256, true>(a, groups(256), s);
  else launch_rows<Z, 1024, true>(a, groups(1024), s);
}

template <typename Z> void launch_gradient(const LogprobArgs& a, hipStream_t s) {
  constexpr int N = Chunk<Z>::N;
  const int64_t most = ((int64_t)a.vocab + 256 * N - 1) / (256 * N);
  const int64_t share = std::max<int64_t>(1, std::min<int64_t>(most, 1024 / std::min<int64_t>(a.rows, 1024)));
  hipLaunchKernelGGL((k_logprobs_backward<Z, 256>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20), (unsigned)share),
                     dim3(256), 0, s, a);
}

}  // namespace

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
