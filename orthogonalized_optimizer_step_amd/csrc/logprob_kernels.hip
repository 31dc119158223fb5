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
__device__ __forceinline__ float factor(float v) { return fmaxf(v, -200.f); }

// Sums over what was seen of a row, relative to its largest value m (or the
// lowest finite one, so that m is always finite or +inf): s of 2^v and w of
// 2^v v, with v = (z - m) c, c = log2(e) / T.  A NaN or +inf makes s NaN.
struct Sums {
  float m, s, w;
  __device__ __forceinline__ void clear() { m = LOWEST, s = w = 0.f; }
  __device__ __forceinline__ void to(float other, float c) {   // relative to another value, at least m
    const float d = (m - other) * c, f = exp2_fast(d);
    w = f * (w + s * factor(d));
    s *= f;
    m = other;
  }
  template <int N> __device__ __forceinline__ void add(const float* z, float c) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float v = (z[i] - m) * c, e = exp2_fast(v);
      s += e;
      w += e * factor(v);
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
    m = lane < W ? red[0][lane] : LOWEST;
    s = lane < W ? red[1][lane] : 0.f;
    w = lane < W ? red[2][lane] : 0.f;
    to(row_reduce<W>(m, LOWEST, MaxNan()), c);
    s = row_reduce<W>(s, 0.f, Add());
    w = row_reduce<W>(w, 0.f, Add());
  }
};

// Logits as whole numbers in their order, -inf and NaN as 0 (no alternative), -0 as 0.
template <typename Z> struct Key {
  static constexpr int BITS = 8 * sizeof(Z);
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
  int entry[KEYS * (NT / 64)];
  int total;
  int id[2][kLogprobMaxTop];                 // the selected, ascending, of two levels in turn
  uint32_t key[kLogprobMaxTop];
  unsigned long long order[kLogprobMaxTop];   // key above, the lower index first
};

// The k largest of n = K NT keys (key i of thread t has position i NT + t),
// equal ones by their position: put(i, o) is called for each with its place o
// in the order of positions.  The k-th largest key is found bit by bit, by
// counting the keys that are at least as large.  k <= the keys that count.
template <int NT, int K, int BITS, typename Put>
__device__ __forceinline__ void select(const uint32_t (&key)[K], int k, TopShared<NT>& sh, Put put) {
  constexpr int W = NT / 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t least = 0;
  int turn = 0;
  for (int b = BITS - 1; b >= 0; --b) {
    const uint32_t cand = least | 1u << b;
    int c = 0;
#pragma unroll
    for (int i = 0; i < K; ++i) c += __popcll(__ballot(key[i] >= cand));
    if (lane == 0) sh.count[turn][wave] = c;
    lds_barrier();
    int total = 0;
#pragma unroll
    for (int w = 0; w < W; w += 4) {
      const intx4 v = *(const intx4*)(sh.count[turn] + w);
      total += v[0] + v[1] + v[2] + v[3];
    }
    turn ^= 1;
    if (total >= k) least = cand;
    if (total == k) break;
  }
  // what lies above it, and the first of those equal to it
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int e = __popcll(__ballot(key[i] > least)) | __popcll(__ballot(key[i] == least)) << 16;
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
    const unsigned long long more = __ballot(key[i] > least), same = __ballot(key[i] == least);
    const int e = sh.entry[i * W + wave];
    const int gt = (e & 0xffff) + __popcll(more & below), eq = (e >> 16) + __popcll(same & below);
    if (key[i] > least || (key[i] == least && eq < need)) put(i, gt + min(eq, need));
  }
  lds_barrier();
}

// One row to a block.  A thread's group i is the P chunks of 16 bytes from
// chunk (i NT + t) P on: groups are in the order of the row.  With the
// alternatives (TOP), the largest of each group is kept, for the k largest
// logits lie in the k groups with the largest maxima (equal ones by their
// order): k other groups' maxima come before anything in the rest.  The same
// again for parts of those groups, down to single logits.
template <typename Z, int NT, bool TOP>
__global__ __launch_bounds__(NT) void k_logprobs(LogprobArgs a, int P) {
  typedef Chunk<Z> C;
  constexpr int N = C::N, U = 4;
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
    Sums S;
    S.clear();
    uint32_t key[TOP ? KEYS : 1];
    // U groups at once, chunk p of each
    auto absorb = [&](const uintx4 (&v)[U], float (&most)[U]) {
      float top = S.m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        most[u] = C::largest(most[u], v[u]);
        top = fmaxf(top, most[u]);
      }
      if (top > S.m) S.to(top, c);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[N];
        C::unpack(v[u], f);
        S.template add<N>(f, c);
      }
    };
    auto groups = [&](int i, float (&most)[U]) {
      for (int p = 0; p < P; ++p) {
        uintx4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t j = (((int64_t)(i + u) * NT + t) * P + p) * N;
          v[u] = C::load(z, (int)min(j, (int64_t)a.vocab), a.vocab, NEG);
        }
        absorb(v, most);
      }
    };
    if constexpr (TOP) {
#pragma unroll
      for (int i = 0; i < KEYS; i += U) {
        float most[U] = {NEG, NEG, NEG, NEG};
        if ((int64_t)i * NT * P * N < a.vocab) groups(i, most);
#pragma unroll
        for (int u = 0; u < U; ++u) key[i + u] = Key<Z>::of(most[u]);
      }
    } else {
      for (int i = 0; (int64_t)i * NT * P * N < a.vocab; i += U) {
        float most[U] = {NEG, NEG, NEG, NEG};
        groups(i, most);
      }
    }
    S.template join<NT>(c, red);
    // a row with nothing but -inf has no distribution: logprob -inf, entropy 0
    const bool none = S.s == 0.f;
    const float logs = logf(S.s), entropy = none ? 0.f : logs - S.w / S.s * LN2;
    auto logprob = [&](float v) { return none ? NEG : (v - S.m) / a.temp - logs; };
    if (t == 0) {
      if (a.tok) a.logprob[row] = token >= 0 ? logprob(zt) : 0.f;
      a.entropy[row] = entropy;
      if (a.stats) a.stats[row] = make_float4(S.m, S.s, entropy, logs);
    }
    if constexpr (TOP) {
      int size = P * N, n = (a.vocab + size - 1) / size, k = min(a.k, n), turn = 0;
      select<NT, KEYS, Key<Z>::BITS>(key, k, sh, [&](int i, int o) {
        sh.id[0][o] = i * NT + t;
        sh.key[o] = key[i];
      });
      while (size > 1) {
        const int part = max(1, size / SUB), r = size / part;
        uint32_t sub[SUB];
        int id[SUB];
        n = 0;
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
          const int q = i * NT + t;
          sub[i] = 0;
          id[i] = 0;
          if (q < k * r) {
            id[i] = sh.id[turn][q / r] * r + q % r;
            const int j = id[i] * part;
            float m = NEG;
            for (int e = 0; e < part; ++e)
              if (j + e < a.vocab) m = fmaxf(m, to_f(z[j + e]));
            sub[i] = Key<Z>::of(m);
          }
        }
        // the parts that lie in the row at all: only its last group may hold others, behind them
        const int parts = (a.vocab + part - 1) / part, last = sh.id[turn][k - 1];
        n = k * r - max(0, (last + 1) * r - parts);
        k = min(a.k, n);
        turn ^= 1;
        select<NT, SUB, Key<Z>::BITS>(sub, k, sh, [&](int i, int o) {
          sh.id[turn][o] = id[i];
          sh.key[o] = sub[i];
        });
        size = part;
      }
      // in order: a bitonic sort of as many places as a power of two
      int places = 2;
      while (places < k) places *= 2;
      for (int i = t; i < places; i += NT)
        sh.order[i] = i < k ? (unsigned long long)sh.key[i] << 32 | (0xffffffffu - (uint32_t)sh.id[turn][i]) : 0;
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
      for (int i = t; i < a.k; i += NT) {
        const uint32_t best = i < k ? (uint32_t)(sh.order[i] >> 32) : 0;
        a.top[row * a.k + i] = best ? logprob(Key<Z>::value(best)) : NEG;
        a.index[row * a.k + i] = best ? (int64_t)(0xffffffffu - (uint32_t)sh.order[i]) : -1;
      }
    }
    lds_barrier();   // the next row's sums may be written
  }
}

// Gradient: columns shared between gridDim.y blocks.
template <typename Z, int NT>
__global__ __launch_bounds__(NT) void k_logprobs_backward(LogprobArgs a) {
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
    // q (gl + ge (log q + entropy)) = exp2(v) (slope + rise v) / s
    const float k = -it / st.y, rise = ge * LN2, slope = gl + ge * (st.z - st.w);
    for (int64_t j = ((int64_t)blockIdx.y * NT + threadIdx.x) * N; j < a.vocab; j += (int64_t)gridDim.y * NT * N) {
      float f[N] = {};
      if (!zero) {
        C::unpack(C::load(z, (int)j, a.vocab, NEG), f);
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

template <typename Z, int NT, bool TOP>
void launch_rows(const LogprobArgs& a, int P, hipStream_t s) {
  hipLaunchKernelGGL((k_logprobs<Z, NT, TOP>), dim3((unsigned)std::min<int64_t>(a.rows, 1 << 20)), dim3(NT), 0, s, a, P);
}

template <typename Z> void launch_forward(const LogprobArgs& a, hipStream_t s) {
  constexpr int N = Chunk<Z>::N;
  if (a.k == 0) {
    if (a.vocab <= 256 * 8 * N) launch_rows<Z, 256, false>(a, 1, s);
    else if (a.rows > 256) launch_rows<Z, 512, false>(a, 1, s);
    else launch_rows<Z, 1024, false>(a, 1, s);
  } else if (a.vocab <= 256 * KEYS * N && a.k <= 256) {
    launch_rows<Z, 256, true>(a, 1, s);
  } else {
    int P = 1;
    while ((int64_t)P * 1024 * KEYS * N < a.vocab) P *= 2;
    launch_rows<Z, 1024, true>(a, P, s);
  }
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
