// kg_gate.hip -- the router's choice on gfx950: C ABI kg_gate and kg_gate_bwd.
//
// For a token's logits x[0 .. G): scores s = softmax(x) or sigmoid(x); the k largest keys (x, or
// s + bias) in descending order, ties to the lower index; their weights; and over all tokens the
// slots per expert and the sums of the probabilities that the balance loss multiplies them with.
// A logit of -inf or NaN is never chosen.
//
// One pass over the logits, bound by their bytes for many tokens. 16 lanes hold a token's logits
// (64 lanes from 257 experts on), 4 to 16 each, so a wave works on four tokens at once and the
// steps of a reduction stay within a row of 16 lanes, which DPP reads without LDS.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "kg_host.h"
#include "kgwgrad.h"

namespace kg {

constexpr int kGateMaxK = 16;       // lane j of a token's lanes holds its j-th choice
constexpr int kGateThreads = 512;   // per workgroup
constexpr int kGateBlocks = 512;    // most workgroups of a launch, each with a line of sums
constexpr float kGateTiny = 1e-20f; // beside the sum of a token's chosen scores

struct GateParams {
  const void* X;
  const float* bias;
  int* idx;
  float* w;
  int* counts;
  float* psum;
  float* loss;
  int* part_counts;  // [blocks][G]
  float* part_psum;  // [blocks][G]
  double* part_loss;
  int* ticket;
  int64_t T, ldx;
  double coef;
  float scale;
  int G, k, flags, stats;
};

typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned short h4_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ float widen(unsigned short h) {
  return __builtin_bit_cast(float, (uint32_t)h << 16);
}
__device__ __forceinline__ unsigned short narrow(float f) {
  return __builtin_bit_cast(unsigned short, (__bf16)f);  // to nearest, ties to even
}
template <bool B16>
__device__ __forceinline__ float gate_at(const void* row, int i) {
  if constexpr (B16) return widen(((const unsigned short*)row)[i]);
  else return ((const float*)row)[i];
}

// Reductions over the LPR lanes of a token; every lane gets the result.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
template <int LPR, class F>
__device__ __forceinline__ uint32_t reduce(uint32_t x, F f) {
  x = f(x, dpp<0x128>(x));  // row_ror: 8, 4, 2, 1
  x = f(x, dpp<0x124>(x));
  x = f(x, dpp<0x122>(x));
  x = f(x, dpp<0x121>(x));
  if constexpr (LPR == 64) {
    auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = f(r[0], r[1]);
    r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = f(r[0], r[1]);
  }
  return x;
}
template <int LPR>
__device__ __forceinline__ uint32_t max_of(uint32_t x) {
  return reduce<LPR>(x, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LPR>
__device__ __forceinline__ uint32_t min_of(uint32_t x) {
  return reduce<LPR>(x, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
__device__ __forceinline__ float as_f(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ uint32_t as_u(float x) { return __builtin_bit_cast(uint32_t, x); }
template <int LPR>
__device__ __forceinline__ float max_of(float x) {
  return as_f(reduce<LPR>(as_u(x), [](uint32_t a, uint32_t b) { return as_u(fmaxf(as_f(a), as_f(b))); }));
}
template <int LPR>
__device__ __forceinline__ float sum_of(float x) {
  return as_f(reduce<LPR>(as_u(x), [](uint32_t a, uint32_t b) { return as_u(as_f(a) + as_f(b)); }));
}

// A float's place in the order of all floats, as an unsigned number (both zeros the same). What is
// never chosen, -inf and NaN, has the lowest place of all.
constexpr uint32_t kNever = 0x007FFFFFu;
__device__ __forceinline__ uint32_t place(float x) {
  const uint32_t u = as_u(fmaxf(x + 0.0f, -INFINITY));  // (the maximum passes over NaN)
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value(uint32_t p) {
  return as_f(p & 0x80000000u ? p ^ 0x80000000u : ~p);
}

// A token's lanes: lane l of LPR holds elements at(v), v = 0 .. V - 1, in runs of four.
template <int LPR, int C>
struct Lanes {
  static constexpr int V = 4 * C, ROWS = 64 / LPR;
  static __device__ __forceinline__ int at(int l, int v) { return ((v >> 2) * LPR + l) * 4 + (v & 3); }
};

template <bool B16, int LPR, int C>
__device__ __forceinline__ void gate_load(const void* row, int G, int l, float (&x)[4 * C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = (c * LPR + l) * 4;
    if ((c + 1) * LPR * 4 <= G || i + 4 <= G) {
      if constexpr (B16) {
        const h4_any h = *(const h4_any*)((const unsigned short*)row + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * c + e] = widen(h[e]);
      } else {
        const f4_any f = *(const f4_any*)((const float*)row + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * c + e] = f[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * c + e] = i + e < G ? gate_at<B16>(row, i + e) : -INFINITY;
    }
  }
}

// exp(x - m) by the exponential unit: two roundings of the exponent, 2^-24 of its size each, and one of
// the result. (As 2^(x log2(e) - m log2(e)), one instruction less, it would overflow for masks of the
// type's lowest value.)
constexpr float kLog2E = 1.44269504f;
__device__ __forceinline__ float exp_less(float x, float m) {
  return __builtin_amdgcn_exp2f((x - m) * kLog2E);
}
// (a sum from 1 to infinity: v_rcp_f32 is within 2^-23 there)
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2E * x));
}

// Scores of a token in place of its logits. *top: the largest logit (softmax; 0 where there is
// none), *inv: one over the sum (0 for a token without experts; finite for any sum).
template <int LPR, int V>
__device__ __forceinline__ void gate_scores(float (&x)[V], bool sig, float* top, float* inv) {
  float m = 0.0f, sum = 0.0f;
  if (sig) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = sigmoid(x[v]);
      sum += x[v];
    }
  } else {
    m = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) m = fmaxf(m, x[v]);
    m = max_of<LPR>(m);
    if (m == -INFINITY) m = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v] = exp_less(x[v], m);
      sum += x[v];
    }
  }
  sum = sum_of<LPR>(sum);
  *top = m;
  *inv = sum == 0.0f ? 0.0f : sum < 0x1p-126f ? 0x1p126f : 1.0f / sum;
}

// The first `n` in order of (place descending, index ascending): the j-th one's index to lane j (-1
// where there is none).
template <int LPR, int V>
__device__ __forceinline__ int choose_exact(uint32_t (&p)[V], int l, int n) {
  int index = -1;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) m = m > p[v] ? m : p[v];
    m = max_of<LPR>(m);
    uint32_t at = 0xFFFFFFFFu;
#pragma unroll
    for (int v = V - 1; v >= 0; --v)
      if (p[v] == m) at = (uint32_t)Lanes<LPR, V / 4>::at(l, v);
    at = min_of<LPR>(at);
    if (l == j) index = m > kNever ? (int)at : -1;
    const uint32_t rel = at - 4 * l;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (rel == (uint32_t)((v >> 2) * LPR * 4 + (v & 3))) p[v] = 0;
  }
  return index;
}

// Keys that hold a place's upper bits and, reversed, the index are distinct, so the next one is the
// largest below the last, found without taking any out: of key - last, unsigned, the keys below
// have the largest. The j-th largest of the tokens' keys to lane j, j < n (0 where there is none); the
// n-th, which may have no lane, is *end.
template <bool B16, int LPR>
constexpr uint32_t kIndexBits = B16 ? 0xFFFFu : LPR == 16 ? 0xFFu : 0x3FFu;
template <bool B16, int LPR, int V>
__device__ __forceinline__ uint32_t largest_keys(const uint32_t (&key)[V], int l, int n,
                                                 uint32_t* end = nullptr) {
  constexpr uint32_t MASK = kIndexBits<B16, LPR>;
  uint32_t last = 0, mine = 0;
  bool more = true;
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t t = key[v] - last;
      m = m > t ? m : t;
    }
    m = max_of<LPR>(m) + last;
    more = more && (m | MASK) > (kNever | MASK);  // (places and masks end in ones)
    if (l == j) mine = more ? m : 0u;
    last = m;
  }
  if (end) *end = more ? last : 0u;
  return mine;
}

// The k largest logits. bf16's 16 bits are a whole place; fp32 choices whose places differ in the
// cut bits alone are ambiguous, and a wave with one of those (or with equal logits) chooses again by
// whole places (16 of 256 experts, 65536 tokens: 38 us; 67 where every wave does).
template <bool B16, int LPR, int V>
__device__ __forceinline__ int choose_logits(const float (&x)[V], const uint32_t (&id)[V], int l,
                                             int k) {
  constexpr uint32_t MASK = kIndexBits<B16, LPR>;
  uint32_t key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) key[v] = (place(x[v]) & ~MASK) | id[v];
  uint32_t end;
  const uint32_t mine = largest_keys<B16, LPR, V>(key, l, k + (B16 ? 0 : 1), &end);
  int index = mine ? (int)(MASK - (mine & MASK)) : -1;
  if constexpr (!B16) {
    uint32_t next = (uint32_t)__shfl_down((int)mine, 1, LPR);
    if (l == k - 1) next = end;  // (16 choices of 16 lanes: the 17th key has no lane)
    if (__any(l < k && next != 0 && ((mine ^ next) & ~MASK) == 0)) {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = place(x[v]);
      index = choose_exact<LPR, V>(key, l, k);
    }
  }
  return index;
}

// One score in 64 bits; `top` and `z` are the softmax's largest logit and sum.
__device__ __forceinline__ double score64(float x, bool sig, float top, double z) {
  return sig ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / z;
}

template <bool B16, int LPR, int C>
__device__ double sum64(const void* row, int G, int l, float top) {
  double z = 0;
#pragma unroll 1
  for (int i = 4 * l; i < G; i += (i & 3) == 3 ? 4 * LPR - 3 : 1)
    z += exp((double)gate_at<B16>(row, i) - (double)top);
#pragma unroll 1
  for (int d = 1; d < LPR; d <<= 1) z += __shfl_xor(z, d, LPR);
  return z;
}

// The k largest of score + bias in 64 bits, each time the first in order behind the last one.
template <bool B16, int LPR, int C>
__device__ __attribute__((noinline)) int choose64(const void* row, const float* bias, int G, int l,
                                                  int k, bool sig, float top) {
  const double z = sig ? 1.0 : sum64<B16, LPR, C>(row, G, l, top);
  double last = INFINITY;
  int last_at = -1, index = -1;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    double best = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll 1
    for (int i = 4 * l; i < G; i += (i & 3) == 3 ? 4 * LPR - 3 : 1) {
      const float x = gate_at<B16>(row, i);
      const double key = score64(x, sig, top, z) + (double)bias[i];
      if (x > -INFINITY && (key < last || (key == last && i > last_at)) && key > best) {
        best = key;
        at = i;
      }
    }
#pragma unroll 1
    for (int d = 1; d < LPR; d <<= 1) {
      const double o = __shfl_xor(best, d, LPR);
      const int oa = __shfl_xor(at, d, LPR);
      if (o > best || (o == best && oa < at)) {
        best = o;
        at = oa;
      }
    }
    const bool none = best == -INFINITY;
    if (l == j) index = none ? -1 : at;
    last = none ? -INFINITY : best;
    last_at = none ? 0x7FFFFFFF : at;
  }
  return index;
}

// The k largest of score + bias. Cut 32-bit keys give k + 1 candidates and a bound for all others;
// the candidates are put in order by their whole 32-bit keys where those tell them apart, else by
// 64-bit ones; and where the k-th is not above the bound, everything is chosen in 64 bits. A 32-bit
// key is off by less than 2^-19 (a score is at most 1; its sum has at most 22 roundings in a row,
// the exponential and the quotient a few) and 2^-23 of the key itself.
template <bool B16, int LPR, int V>
__device__ __forceinline__ int choose_biased(const float (&x)[V], const float (&s)[V],
                                             const uint32_t (&id)[V], float inv, float top,
                                             const void* row, const float* bias, int G, int l, int k,
                                             bool sig) {
  constexpr uint32_t MASK = kIndexBits<false, LPR>;
  uint32_t key[V];
  const float factor = sig ? 1.0f : inv;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = Lanes<LPR, V / 4>::at(l, v);
    const float f = i < G ? fmaf(s[v], factor, bias[i]) : 0.0f;
    key[v] = ((i < G && x[v] > -INFINITY ? place(f) : kNever) & ~MASK) | id[v];
  }
  const uint32_t mine = largest_keys<false, LPR, V>(key, l, k + 2);  // (a token has that many lanes)
  const bool in = l <= k && mine != 0;
  const int index = in ? (int)(MASK - (mine & MASK)) : -1;
  float f = -INFINITY;
  if (in) {
    const float own = gate_at<B16>(row, index);
    f = (sig ? sigmoid(own) : exp_less(own, top) * inv) + bias[index];
  }
  // the most that any other can have
  const uint32_t beyond = (uint32_t)__shfl((int)mine, k + 1, LPR);
  const float bound = beyond ? value(beyond | MASK) : -INFINITY;
  int rank = 0;
  bool close = false, low = false;
#pragma unroll 1
  for (int j = 0; j <= k; ++j) {
    const float o = __shfl(f, j, LPR);
    const int oi = __shfl(index, j, LPR);
    rank += o > f || (o == f && oi >= 0 && oi < index);
    close |= in && oi >= 0 && j != l && !(fabsf(o - f) > 0x1p-18f + 0x1p-22f * fabsf(f));
  }
  if (in && rank < k && beyond) low = !(f - bound > 0x1p-18f + 0x1p-22f * fabsf(f));
  if (__any(low)) {
    const int all = choose64<B16, LPR, V / 4>(row, bias, G, l, k, sig, top);  // with every lane
    return l < k ? all : -1;
  }
  if (__any(close)) {
    const double z = sig ? 1.0 : sum64<B16, LPR, V / 4>(row, G, l, top);
    double d = -INFINITY;
    if (in) d = score64(gate_at<B16>(row, index), sig, top, z) + (double)bias[index];
    rank = 0;
#pragma unroll 1
    for (int j = 0; j <= k; ++j) {
      const double o = __shfl(d, j, LPR);
      const int oi = __shfl(index, j, LPR);
      rank += o > d || (o == d && oi >= 0 && oi < index);
    }
  }
  // to the lane of its rank; lanes without a candidate are behind those with one
  const int lane = threadIdx.x & 63, to = (lane & ~(LPR - 1)) + (in ? rank : l);
  const int out = __builtin_amdgcn_ds_permute(4 * to, index);
  return l < k ? out : -1;
}

// The sums over all workgroups' lines, in a fixed order; the last workgroup to finish adds up the
// loss, in one as well.
constexpr int kGateSumExperts = 8;
constexpr int kGateSumThreads = 1024;  // 128 lines at a time (65536 tokens, 256 experts: 5 us)
__global__ __launch_bounds__(kGateSumThreads) void kg_gate_sum_kernel(GateParams p, int blocks) {
  constexpr int E = kGateSumExperts, S = kGateSumThreads / E, WAVES = kGateSumThreads / 64;
  __shared__ double sums[WAVES][E];
  __shared__ int cnts[WAVES][E];
  const int e = threadIdx.x % E, part = threadIdx.x / E, g = blockIdx.x * E + e;
  double sum = 0;
  int cnt = 0;
  if (g < p.G) {
#pragma unroll 4
    for (int b = part; b < blocks; b += S) {
      sum += (double)p.part_psum[(int64_t)b * p.G + g];
      cnt += p.part_counts[(int64_t)b * p.G + g];
    }
  }
#pragma unroll
  for (int d = E; d < 64; d <<= 1) {
    sum += __shfl_xor(sum, d, 64);
    cnt += __shfl_xor(cnt, d, 64);
  }
  if ((threadIdx.x & 63) < E) {
    sums[threadIdx.x >> 6][e] = sum;
    cnts[threadIdx.x >> 6][e] = cnt;
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  const bool own = threadIdx.x < E;
  double term = 0;
  if (own) {
#pragma unroll
    for (int i = 1; i < WAVES; ++i) {
      sum += sums[i][e];
      cnt += cnts[i][e];
    }
    if (g < p.G) {
      if (p.counts) p.counts[g] = cnt;
      if (p.psum) p.psum[g] = (float)sum;
    }
    term = sum * (double)cnt;
  }
  if (!p.loss) return;
#pragma unroll
  for (int d = 1; d < E; d <<= 1) term += __shfl_xor(term, d, 64);
  int last = 0;
  if (threadIdx.x == 0) {
    __hip_atomic_store(&p.part_loss[blockIdx.x], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(p.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
           (int)gridDim.x - 1;
  }
  if (!__shfl(last, 0, 64)) return;
  double total = 0;
  for (unsigned b = threadIdx.x; b < gridDim.x; b += 64)
    total += __hip_atomic_load(&p.part_loss[b], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d, 64);
  if (threadIdx.x == 0) *p.loss = (float)(p.coef * total);
}

template <bool B16, int LPR, int C, bool BIAS>
__global__ __launch_bounds__(kGateThreads) void kg_gate_kernel(GateParams p) {
  using L = Lanes<LPR, C>;
  constexpr int V = L::V, WAVES = kGateThreads / 64, EXPERTS = LPR * V;
  __shared__ int counts[EXPERTS];
  __shared__ float lines[WAVES][EXPERTS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane % LPR, sub = lane / LPR;
  const bool sig = (p.flags & KG_GATE_SIGMOID) != 0, norm = (p.flags & KG_GATE_NORM) != 0;
  if (p.stats) {
    for (int i = threadIdx.x; i < EXPERTS; i += kGateThreads) counts[i] = 0;
    __syncthreads();
  }
  float sums[V];
  uint32_t id[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    sums[v] = 0.0f;
    id[v] = kIndexBits<B16 && !BIAS, LPR> - (uint32_t)L::at(l, v);
  }
  const int64_t step = (int64_t)gridDim.x * WAVES * L::ROWS;
  const int64_t begin = ((int64_t)blockIdx.x * WAVES + wave) * L::ROWS;
  float ahead[V];
  auto load = [&](int64_t t0) {
    const int64_t t = t0 + sub < p.T ? t0 + sub : p.T - 1;
    gate_load<B16, LPR, C>((const char*)p.X + t * p.ldx * (B16 ? 2 : 4), p.G, l, ahead);
  };
  if (begin < p.T) load(begin);
  for (int64_t t0 = begin; t0 < p.T; t0 += step) {
    const bool live = t0 + sub < p.T;
    const int64_t t = live ? t0 + sub : p.T - 1;
    const void* row = (const char*)p.X + t * p.ldx * (B16 ? 2 : 4);
    float x[V], s[V], top, inv;
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = x[v] = ahead[v];
    if (t0 + step < p.T) load(t0 + step);  // the next tokens' logits are on their way meanwhile
    gate_scores<LPR, V>(s, sig, &top, &inv);
    int index;
    if constexpr (BIAS) index = choose_biased<B16, LPR, V>(x, s, id, inv, top, row, p.bias, p.G, l, p.k, sig);
    else index = choose_logits<B16, LPR, V>(x, id, l, p.k);
    if (l >= p.k) index = -1;
    float w = 0.0f;
    if (index >= 0) {
      const float own = gate_at<B16>(row, index);
      w = sig ? sigmoid(own) : exp_less(own, top) * inv;
    }
    if (norm) w = w / (sum_of<LPR>(w) + kGateTiny);
    if (live && l < p.k) {
      p.idx[t * p.k + l] = index;
      p.w[t * p.k + l] = index >= 0 ? p.scale * w : 0.0f;  // (the sum of a row with NaN may be NaN)
    }
    if (p.stats && live) {
      if (index >= 0) atomicAdd(&counts[index], 1);
#pragma unroll
      for (int v = 0; v < V; ++v) sums[v] += s[v] * inv;
    }
  }
  if (!p.stats) return;
  // the wave's tokens side by side, then the waves, in a fixed order
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (LPR == 16) {
      auto r = __builtin_amdgcn_permlane16_swap(as_u(sums[v]), as_u(sums[v]), false, false);
      const float two = as_f(r[0]) + as_f(r[1]);
      r = __builtin_amdgcn_permlane32_swap(as_u(two), as_u(two), false, false);
      sums[v] = as_f(r[0]) + as_f(r[1]);
    }
    if (sub == 0) lines[wave][L::at(l, v)] = sums[v];
  }
  __syncthreads();
  for (int g = threadIdx.x; g < p.G; g += kGateThreads) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) sum += lines[i][g];
    p.part_psum[(int64_t)blockIdx.x * p.G + g] = sum;
    p.part_counts[(int64_t)blockIdx.x * p.G + g] = counts[g];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.ticket = 0;
}

// ------------------------------------------------------------------------------- gradient

struct GateBwdParams {
  const void* X;
  const int* idx;
  const float* dw;
  const int* counts;
  const float* dloss;
  void* dX;
  int64_t T, ldx, ldd;
  float coef, scale;
  int G, k, flags;
};

// What a wave's lanes wrote to LDS before is there for its other lanes (LDS serves a wave in order).
__device__ __forceinline__ void wave_meets() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// dx of a token. With c_g = dloss coef counts[g], and d_j the gradient of the j-th chosen score
// (through its quotient with NORM), softmax: dp = c + d, dx = p (dp - sum p dp); sigmoid:
// dx = s (1 - s) (d + (c - sum p c) / sum s). The d_j reach the lanes of their experts through LDS.
template <bool B16, int LPR, int C>
__global__ __launch_bounds__(kGateThreads) void kg_gate_bwd_kernel(GateBwdParams p) {
  using L = Lanes<LPR, C>;
  constexpr int V = L::V, WAVES = kGateThreads / 64, EXPERTS = LPR * V;
  __shared__ __attribute__((aligned(16))) float spread[WAVES][L::ROWS][EXPERTS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l = lane % LPR, sub = lane / LPR;
  const bool sig = (p.flags & KG_GATE_SIGMOID) != 0, norm = (p.flags & KG_GATE_NORM) != 0;
  float even[V];  // dloss coef counts
  const float dl = p.counts ? p.coef * (p.dloss ? *p.dloss : 1.0f) : 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = L::at(l, v);
    even[v] = p.counts && i < p.G ? dl * (float)p.counts[i] : 0.0f;
  }
  float* mine = spread[wave][sub];
  const int64_t step = (int64_t)gridDim.x * WAVES * L::ROWS;
  for (int64_t t0 = ((int64_t)blockIdx.x * WAVES + wave) * L::ROWS; t0 < p.T; t0 += step) {
    const bool live = t0 + sub < p.T;
    const int64_t t = live ? t0 + sub : p.T - 1;
    const void* row = (const char*)p.X + t * p.ldx * (B16 ? 2 : 4);
    int index = -1;
    float dw = 0.0f, own = 0.0f;
    if (p.dw && l < p.k) {
      index = p.idx[t * p.k + l];
      if (index < 0 || index >= p.G) index = -1;
      if (index >= 0) {
        dw = p.dw[t * p.k + l];
        own = gate_at<B16>(row, index);
      }
    }
    float s[V], x[V], top, inv;
    gate_load<B16, LPR, C>(row, p.G, l, x);
#pragma unroll
    for (int v = 0; v < V; ++v) s[v] = x[v];
    gate_scores<LPR, V>(s, sig, &top, &inv);
    float chosen = 0.0f, d = dw;
    if (index >= 0) chosen = sig ? sigmoid(own) : exp_less(own, top) * inv;
    if (norm) {
      const float sum = sum_of<LPR>(chosen) + kGateTiny, mean = sum_of<LPR>(dw * chosen) / sum;
      d = (dw - mean) / sum;
    }
    d *= p.scale;
#pragma unroll
    for (int c = 0; c < C; ++c) *(float4*)(mine + (c * LPR + l) * 4) = float4{0, 0, 0, 0};
    wave_meets();
    if (index >= 0) atomicAdd(mine + index, d);
    wave_meets();
    float dx[V], sum = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float4 f = *(const float4*)(mine + (c * LPR + l) * 4);
      dx[4 * c] = f.x, dx[4 * c + 1] = f.y, dx[4 * c + 2] = f.z, dx[4 * c + 3] = f.w;
    }
    wave_meets();
    if (sig) {
#pragma unroll
      for (int v = 0; v < V; ++v) sum += s[v] * inv * even[v];
      sum = sum_of<LPR>(sum);
#pragma unroll
      for (int v = 0; v < V; ++v)
        dx[v] = x[v] == -INFINITY ? 0.0f : s[v] * sigmoid(-x[v]) * (dx[v] + (even[v] - sum) * inv);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        s[v] *= inv;
        dx[v] += even[v];
        sum += s[v] * dx[v];
      }
      sum = sum_of<LPR>(sum);
#pragma unroll
      for (int v = 0; v < V; ++v) dx[v] = s[v] * (dx[v] - sum);
    }
    if (!live) continue;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = (c * LPR + l) * 4;
      if constexpr (B16) {
        unsigned short* o = (unsigned short*)p.dX + t * p.ldd + i;
        if ((c + 1) * LPR * 4 <= p.G || i + 4 <= p.G) {
          *(h4_any*)o = h4_any{narrow(dx[4 * c]), narrow(dx[4 * c + 1]), narrow(dx[4 * c + 2]),
                               narrow(dx[4 * c + 3])};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < p.G) o[e] = narrow(dx[4 * c + e]);
        }
      } else {
        float* o = (float*)p.dX + t * p.ldd + i;
        if ((c + 1) * LPR * 4 <= p.G || i + 4 <= p.G) {
          *(f4_any*)o = f4_any{dx[4 * c], dx[4 * c + 1], dx[4 * c + 2], dx[4 * c + 3]};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < p.G) o[e] = dx[4 * c + e];
        }
      }
    }
  }
}

// Whether a token has 16 lanes. Few tokens of more than 64 experts have 64, so that a lane has fewer
// of the logits that each step goes through.
constexpr int kGateFew = 1024;
static bool gate_row16(int64_t T, int G) { return G <= 64 || (G <= 256 && T > kGateFew); }
static int64_t gate_blocks(int64_t T, int G) {
  const int64_t rows = kGateThreads / 64 * (gate_row16(T, G) ? 4 : 1);
  const int64_t n = (T + rows - 1) / rows;
  return n < 1 ? 1 : n < kGateBlocks ? n : kGateBlocks;
}
static int64_t gate_sum_blocks(int G) { return (G + kGateSumExperts - 1) / kGateSumExperts; }
// Bytes of workspace that a call uses: a line of sums for each workgroup.
static int64_t gate_bytes(int64_t T, int G) {
  return 64 + gate_sum_blocks(G) * 8 + gate_blocks(T, G) * G * 8;
}

static bool gate_sizes_ok(int64_t T, int G, int k) { return T >= 0 && G >= 1 && k >= 1 && k <= G; }
static bool gate_sizes_taken(int64_t T, int G, int k, int64_t ld) {
  return G <= 1024 && k <= kGateMaxK && T <= INT32_MAX / k && ld <= (1 << 30);
}

}  // namespace kg

// The kernel of a launch: by type and by how many logits a lane holds.
#define KG_GATE_PICK(fn, b16, G, row16, ...)                                                          \
  ((b16) ? KG_GATE_SIZE(fn, true, G, row16, __VA_ARGS__) : KG_GATE_SIZE(fn, false, G, row16, __VA_ARGS__))
#define KG_GATE_SIZE(fn, b16, G, row16, ...)            \
  ((row16) ? ((G) <= 64    ? fn<b16, 16, 1 __VA_ARGS__> \
              : (G) <= 128 ? fn<b16, 16, 2 __VA_ARGS__> \
                           : fn<b16, 16, 4 __VA_ARGS__>) \
           : ((G) <= 256   ? fn<b16, 64, 1 __VA_ARGS__> \
              : (G) <= 512 ? fn<b16, 64, 2 __VA_ARGS__> \
                           : fn<b16, 64, 4 __VA_ARGS__>))
#define KG_GATE_COMMA_TRUE , true
#define KG_GATE_COMMA_FALSE , false

extern "C" int64_t kg_gate_workspace_bytes(int64_t T, int G) {
  using namespace kg;
  if (T < 0 || G < 1 || G > 1024 || T > INT32_MAX) return -1;
  // Enough for fewer tokens too: kGateFew of them may take more workgroups than a few more do. (More
  // experts never take fewer.)
  const int64_t few = gate_bytes(T < kGateFew ? T : kGateFew, G), own = gate_bytes(T, G);
  return few > own ? few : own;
}

extern "C" int kg_gate(const void* X, int64_t ldx, const float* bias, int64_t T, int G, int k,
                       int type, int flags, double scale, double coef, int32_t* idx, float* w,
                       int32_t* counts, float* psum, float* loss, void* workspace,
                       int64_t workspace_bytes, void* stream) {
  using namespace kg;
  if (type != KG_ROWS_BF16 && type != KG_ROWS_F32) return KG_ERR_DTYPE;
  if (flags & ~(KG_GATE_SIGMOID | KG_GATE_NORM)) return KG_ERR_DTYPE;
  if (!gate_sizes_ok(T, G, k) || ldx < G || workspace_bytes < 0) return KG_ERR_SHAPE;
  if (!gate_sizes_taken(T, G, k, ldx)) return KG_ERR_UNSUPPORTED;
  const bool stats = counts || psum || loss, b16 = type == KG_ROWS_BF16;
  if (T == 0 && !stats) return KG_OK;
  if (T > 0 && (!X || !idx || !w)) return KG_ERR_NULL;
  if (stats && !workspace) return KG_ERR_NULL;
  const size_t e = b16 ? 2 : 4;
  if (((uintptr_t)X & (e - 1)) || ((uintptr_t)bias & 3) || ((uintptr_t)idx & 3) ||
      ((uintptr_t)w & 3) || ((uintptr_t)counts & 3) || ((uintptr_t)psum & 3) ||
      ((uintptr_t)loss & 3) || (stats && ((uintptr_t)workspace & 15)))
    return KG_ERR_ALIGN;
  const int64_t need = stats ? gate_bytes(T, G) : 0;
  if (workspace_bytes < need) return KG_ERR_SHAPE;
  const void* outs[] = {idx, w, counts, psum, loss, stats ? workspace : nullptr};
  const size_t sizes[] = {(size_t)T * k * 4, (size_t)T * k * 4, (size_t)G * 4, (size_t)G * 4, 4,
                          (size_t)need};
  const size_t xbytes = T > 0 ? ((size_t)(T - 1) * ldx + G) * e : 0;
  for (int i = 0; i < 6; ++i) {
    if (ranges_overlap(outs[i], sizes[i], X, xbytes) ||
        ranges_overlap(outs[i], sizes[i], bias, (size_t)G * 4))
      return KG_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(outs[i], sizes[i], outs[j], sizes[j])) return KG_ERR_ALIAS;
  }
  const int64_t blocks = gate_blocks(T, G);
  GateParams p;
  p.X = X, p.bias = bias, p.idx = idx, p.w = w, p.counts = counts, p.psum = psum, p.loss = loss;
  p.T = T, p.ldx = ldx, p.coef = coef, p.scale = (float)scale;
  p.G = G, p.k = k, p.flags = flags, p.stats = stats;
  p.ticket = (int*)workspace;
  p.part_loss = stats ? (double*)((char*)workspace + 64) : nullptr;
  p.part_psum = stats ? (float*)(p.part_loss + gate_sum_blocks(G)) : nullptr;
  p.part_counts = stats ? (int*)(p.part_psum + blocks * G) : nullptr;
  // (the choice by biased scores holds two more than it makes)
  const bool row16 = gate_row16(T, G) && !(bias && k + 2 > 16);
  void (*fn)(GateParams) = bias ? KG_GATE_PICK(kg_gate_kernel, b16, G, row16, KG_GATE_COMMA_TRUE)
                                : KG_GATE_PICK(kg_gate_kernel, b16, G, row16, KG_GATE_COMMA_FALSE);
  const int rc = launch(fn, blocks, kGateThreads, 0, stream, p);
  if (rc != KG_OK || !stats) return rc;
  return launch(kg_gate_sum_kernel, gate_sum_blocks(G), kGateSumThreads, 0, stream, p, (int)blocks);
}

extern "C" int kg_gate_bwd(const void* X, int64_t ldx, const int32_t* idx, const float* dw,
                           const int32_t* counts, const float* dloss, int64_t T, int G, int k,
                           int type, int flags, double scale, double coef, void* dX, int64_t ldd,
                           void* stream) {
  using namespace kg;
  if (type != KG_ROWS_BF16 && type != KG_ROWS_F32) return KG_ERR_DTYPE;
  if (flags & ~(KG_GATE_SIGMOID | KG_GATE_NORM)) return KG_ERR_DTYPE;
  if (!gate_sizes_ok(T, G, k) || ldx < G || ldd < G) return KG_ERR_SHAPE;
  if (!gate_sizes_taken(T, G, k, ldx > ldd ? ldx : ldd)) return KG_ERR_UNSUPPORTED;
  if (T == 0) return KG_OK;
  if (!X || !dX || (dw && !idx)) return KG_ERR_NULL;
  const bool b16 = type == KG_ROWS_BF16;
  const size_t e = b16 ? 2 : 4;
  if (((uintptr_t)X & (e - 1)) || ((uintptr_t)dX & (e - 1)) || ((uintptr_t)idx & 3) ||
      ((uintptr_t)dw & 3) || ((uintptr_t)counts & 3) || ((uintptr_t)dloss & 3))
    return KG_ERR_ALIGN;
  const size_t dbytes = ((size_t)(T - 1) * ldd + G) * e;
  if (ranges_overlap(dX, dbytes, X, ((size_t)(T - 1) * ldx + G) * e) ||
      ranges_overlap(dX, dbytes, idx, (size_t)T * k * 4) ||
      ranges_overlap(dX, dbytes, dw, (size_t)T * k * 4) ||
      ranges_overlap(dX, dbytes, counts, (size_t)G * 4) || ranges_overlap(dX, dbytes, dloss, 4))
    return KG_ERR_ALIAS;
  GateBwdParams p;
  p.X = X, p.idx = idx, p.dw = dw, p.counts = counts, p.dloss = dloss, p.dX = dX;
  p.T = T, p.ldx = ldx, p.ldd = ldd, p.coef = (float)coef, p.scale = (float)scale;
  p.G = G, p.k = k, p.flags = flags;
  const bool row16 = gate_row16(T, G);
  const int64_t rows = kGateThreads / 64 * (row16 ? 4 : 1);
  int64_t blocks = (T + rows - 1) / rows;
  if (blocks > 2 * kGateBlocks) blocks = 2 * kGateBlocks;
  void (*fn)(GateBwdParams) = KG_GATE_PICK(kg_gate_bwd_kernel, b16, G, row16, );
  return launch(fn, blocks, kGateThreads, 0, stream, p);
}
