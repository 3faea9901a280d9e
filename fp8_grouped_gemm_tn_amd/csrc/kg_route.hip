// kg_route.hip -- tokens into expert order and back on gfx950, C ABI kg_route,
// kg_dispatch, kg_dispatch_fp8, kg_combine, kg_combine_bwd.
//
// The products of an expert layer (kg_fprop, kg_dgrad, kg_wgrad) read rows in expert
// order: expert g's rows are contiguous. With idx [T, k] the experts that a router chose
// for each token, slot s = t * k + j holds expert e(s) = idx[t][j] (G, "dropped", when it
// lies outside [0, G)), and
//   row(s)  = the rank of s in the order by (e(s), s): a stable counting sort;
//   ks[g]   = number of slots of expert g;
//   pos[s]  = row(s), or ~row(s) (negative) for a dropped slot;
//   src[r]  = s for row(s) = r, or ~s.
// Dropped slots take the rows behind the last expert's, so the rows are a permutation of
// the slots and every row is written exactly once (zeros for the dropped ones).
//   dispatch      Xp[row] = X[t]          its gradient is combine without weights
//   dispatch_fp8  the same as e4m3 codes with one scale per row and 128 channels
//   combine       out[t] = sum_j w[t][j] Y[pos[t][j]]
//   combine_bwd   dY[row] = w[t][j] dOut[t],  dw[t][j] = <dOut[t], Y[row]>
// All of it is bound by memory: each kernel reads and writes its rows once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kg_device.h"
#include "kg_host.h"
#include "kgwgrad.h"

namespace kg {

constexpr int kRouteMaxGroups = 1024;
constexpr int kRouteKeys = kRouteMaxGroups + 1;  // + the dropped slots

// ------------------------------------------------------------------------------ sort plan

// Waves of a sorting workgroup; each ranks a contiguous run of slots in order.
constexpr int kSortWaves = 8, kSortThreads = 64 * kSortWaves;
// The two-pass plan cuts the slots into at most kSortBlocks blocks of at least kSortBlock.
constexpr int kSortBlocks = 256, kSortBlock = 2048;
// Up to this many slots one workgroup of kSoloWaves waves does everything in one launch (256
// experts: 4096 slots 7.6 us, 8192 slots 11.5 us against 9.4 in two passes).
constexpr int kSoloWaves = 16;
constexpr int kSoloSlots = 4096;

__device__ __forceinline__ int slot_key(const int32_t* idx, int64_t s, int G) {
  const int e = idx[s];
  return (unsigned)e < (unsigned)G ? e : G;
}

// Adds the slots [s0, s1) of this wave to its histogram row.
__device__ __forceinline__ void wave_count(const int32_t* idx, int64_t s0, int64_t s1, int G,
                                           int* row) {
  const int lane = threadIdx.x & 63;
  for (int64_t s = s0 + lane; s < s1; s += 64) atomicAdd(row + slot_key(idx, s, G), 1);
}

// Ranks the slots [s0, s1) of this wave in order: next[e] is the row of the wave's next slot
// of expert e. Lanes of one expert find each other by one ballot per bit of the key; the
// lowest of them moves next[e] on by their number, so a slot's row does not depend on timing.
__device__ __forceinline__ void wave_rank(const int32_t* idx, int64_t s0, int64_t s1, int G,
                                          int bits, volatile int* next, int32_t* pos,
                                          int32_t* src) {
  const int lane = threadIdx.x & 63;
  for (int64_t base = s0; base < s1; base += 64) {
    const int64_t s = base + lane;
    const bool on = s < s1;
    const int e = on ? slot_key(idx, s, G) : 0;
    uint64_t peers = __ballot(on);
    for (int b = 0; b < bits; ++b) {
      const bool bit = (e >> b) & 1;
      const uint64_t m = __ballot(bit);
      peers &= bit ? m : ~m;
    }
    const int rank = __popcll(peers & ((1ull << lane) - 1));
    int row = 0;
    if (on) row = next[e] + rank;
    __builtin_amdgcn_wave_barrier();  // every lane has read next[e] before it moves on
    if (on && rank == 0) next[e] = row + __popcll(peers);
    __builtin_amdgcn_wave_barrier();
    if (on) {
      const bool kept = e < G;
      pos[s] = kept ? row : ~row;
      if (src != nullptr) src[row] = kept ? (int32_t)s : ~(int32_t)s;
    }
  }
}

// Exclusive scan over keys 0 .. G of total[], in place, by the whole workgroup (each
// thread owns PER consecutive keys). `part` holds one int per wave.
template <int THREADS>
__device__ __forceinline__ void scan_keys(int* total, int G, int* part) {
  constexpr int PER = (kRouteKeys + THREADS - 1) / THREADS;
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  int v[PER], own = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    v[i] = e <= G ? total[e] : 0;
    own += v[i];
  }
  int incl = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(incl, d, 64);
    if (lane >= d) incl += u;
  }
  if (lane == 63) part[w] = incl;
  __syncthreads();
  int run = incl - own;
  for (int i = 0; i < w; ++i) run += part[i];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = t * PER + i;
    if (e <= G) total[e] = run;
    run += v[i];
  }
  __syncthreads();
}

// Everything in one workgroup: the waves count their runs of slots, the counts are scanned
// over waves and experts, the waves rank their runs.
__global__ __launch_bounds__(64 * kSoloWaves) void kg_route_solo_kernel(
    const int32_t* idx, int n, int G, int bits, int32_t* ks, int32_t* pos, int32_t* src) {
  extern __shared__ int sm[];
  __shared__ int part[kSoloWaves];
  const int keys = G + 1, t = threadIdx.x, w = t >> 6;
  int* hist = sm;                       // [kSoloWaves][keys]
  int* total = sm + kSoloWaves * keys;  // [keys]
  for (int i = t; i < kSoloWaves * keys; i += 64 * kSoloWaves) hist[i] = 0;
  __syncthreads();
  const int run = ((n + kSoloWaves - 1) / kSoloWaves + 63) & ~63;
  const int s0 = min(n, w * run), s1 = min(n, s0 + run);
  wave_count(idx, s0, s1, G, hist + w * keys);
  __syncthreads();
  for (int e = t; e < keys; e += 64 * kSoloWaves) {
    int sum = 0;
    for (int i = 0; i < kSoloWaves; ++i) {
      const int c = hist[i * keys + e];
      hist[i * keys + e] = sum;
      sum += c;
    }
    total[e] = sum;
    if (e < G) ks[e] = sum;
  }
  __syncthreads();
  scan_keys<64 * kSoloWaves>(total, G, part);
  for (int e = t; e < keys; e += 64 * kSoloWaves)
    for (int i = 0; i < kSoloWaves; ++i) hist[i * keys + e] += total[e];
  __syncthreads();
  wave_rank(idx, s0, s1, G, bits, hist + w * keys, pos, src);
}

// Pass 1: counts of every block of slots, counts[block][key].
__global__ __launch_bounds__(kSortThreads) void kg_route_count_kernel(const int32_t* idx,
                                                                     int64_t n, int per, int G,
                                                                     int32_t* counts) {
  extern __shared__ int sm[];
  const int keys = G + 1;
  for (int i = threadIdx.x; i < keys; i += kSortThreads) sm[i] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * per;
  const int64_t s1 = s0 + per < n ? s0 + per : n;
  for (int64_t s = s0 + threadIdx.x; s < s1; s += kSortThreads)
    atomicAdd(sm + slot_key(idx, s, G), 1);
  __syncthreads();
  for (int i = threadIdx.x; i < keys; i += kSortThreads)
    counts[(int64_t)blockIdx.x * keys + i] = sm[i];
}

// Pass 2: every block adds up the counts (all of them for the experts' first rows, the earlier
// blocks' for its own place in each) and ranks its slots. Reading counts in every block is at
// most 256 x 256 x (G + 1) words from the L2, and saves a launch and its wait (131072 slots of
// 256 experts 30 -> 11 us, 2 M slots 265 -> 34 us).
__global__ __launch_bounds__(kSortThreads) void kg_route_rank_kernel(
    const int32_t* __restrict__ idx, int64_t n, int per, int G, int bits,
    const int32_t* __restrict__ counts, int blocks, int32_t* __restrict__ ks,
    int32_t* __restrict__ pos, int32_t* __restrict__ src) {
  extern __shared__ int sm[];
  __shared__ int part[kSortWaves];
  const int keys = G + 1, t = threadIdx.x, w = t >> 6, me = blockIdx.x;
  int* hist = sm;                       // [kSortWaves][keys]
  int* total = sm + kSortWaves * keys;  // [keys]
  for (int i = t; i < kSortWaves * keys; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  const int64_t b0 = (int64_t)me * per;
  const int64_t b1 = b0 + per < n ? b0 + per : n;
  const int run = per / kSortWaves;
  const int64_t s0 = b0 + w * run < b1 ? b0 + w * run : b1, s1 = s0 + run < b1 ? s0 + run : b1;
  wave_count(idx, s0, s1, G, hist + w * keys);
  constexpr int PER = (kRouteKeys + kSortThreads - 1) / kSortThreads;
  int before[PER];
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const int e = t + x * kSortThreads;
    before[x] = 0;
    if (e >= keys) continue;
    int sum = 0;
#pragma unroll 16
    for (int b = 0; b < blocks; ++b) {
      const int c = counts[(int64_t)b * keys + e];
      sum += c;
      before[x] += b < me ? c : 0;
    }
    total[e] = sum;
    if (me == 0 && e < G) ks[e] = sum;
  }
  __syncthreads();
  scan_keys<kSortThreads>(total, G, part);
#pragma unroll
  for (int x = 0; x < PER; ++x) {
    const int e = t + x * kSortThreads;
    if (e >= keys) continue;
    int sum = total[e] + before[x];
    for (int i = 0; i < kSortWaves; ++i) {
      const int c = hist[i * keys + e];
      hist[i * keys + e] = sum;
      sum += c;
    }
  }
  __syncthreads();
  wave_rank(idx, s0, s1, G, bits, hist + w * keys, pos, src);
}

// ---------------------------------------------------------------------------------- rows

// 16 bytes at any address that the element type allows (gfx950 takes unaligned accesses).
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(1)));
typedef int v2i_any __attribute__((ext_vector_type(2), aligned(1)));

struct RowShape {
  int64_t T;
  int64_t rows;  // T * k
  int k, H;
  int lanes;  // threads of a run: a power of two up to the workgroup's 256
  int runs;   // runs of `lanes` units per token (the kernels that take one unit per thread)
  int64_t groups;  // workgroups that have work
};

// A launch holds fewer than 2^32 threads in x: more workgroups go over y as well.
constexpr int64_t kGroupsX = 1 << 23;
__device__ __forceinline__ int64_t group_id() {
  return (int64_t)blockIdx.y * kGroupsX + blockIdx.x;
}

__device__ __forceinline__ float bf16_to_f32(uint32_t u) { return __uint_as_float(u << 16); }

// The nearest bf16, ties to even (a NaN stays a NaN).
__device__ __forceinline__ uint32_t f32_to_bf16(float x) {
  return __builtin_bit_cast(unsigned short, (__bf16)x);
}

// N values of a row: bf16 or fp32, 16 bytes.
template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4;
  static constexpr int ELEM = BF16 ? 2 : 4;
  static __device__ __forceinline__ void unpack(const v4i& x, float (&f)[N]) {
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_to_f32((uint32_t)x[i] & 0xFFFFu);
        f[2 * i + 1] = __uint_as_float((uint32_t)x[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __int_as_float(x[i]);
    }
  }
  static __device__ __forceinline__ v4i pack(const float (&f)[N]) {
    v4i x;
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = (int)(f32_to_bf16(f[2 * i]) | f32_to_bf16(f[2 * i + 1]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __float_as_int(f[i]);
    }
    return x;
  }
  static __device__ __forceinline__ float load1(const unsigned char* p) {
    return BF16 ? bf16_to_f32(*(const unsigned short*)p) : *(const float*)p;
  }
  static __device__ __forceinline__ void store1(unsigned char* p, float x) {
    if constexpr (BF16)
      *(unsigned short*)p = (unsigned short)f32_to_bf16(x);
    else
      *(float*)p = x;
  }
};

__device__ __forceinline__ v4i load16(const unsigned char* p) { return *(const v4i_any*)p; }
__device__ __forceinline__ void store16(unsigned char* p, const v4i& x) { *(v4i_any*)p = x; }
// ... past the caches, for what is read or written once. (16384 tokens of 8 slots, 7168
// channels, inputs not in the caches: bf16 rows 412 us, 5.1 TB/s, with a run of tokens per
// XCD, 435 without; fp8 rows 248 us, 4.9 TB/s; sums of k rows 369 us, 5.7 TB/s,
// 408 with outputs through the caches; gradients 782 us, 5.1 TB/s. Rows that start inside a
// line gain less: 2951 channels 160 us past the caches and 165 through them, 1122 channels
// 373 and 361.)
__device__ __forceinline__ v4i load16_once(const unsigned char* p) {
  return __builtin_nontemporal_load((const v4i_any*)p);
}
__device__ __forceinline__ void store16_once(unsigned char* p, const v4i& x) {
  __builtin_nontemporal_store(x, (v4i_any*)p);
}

// The row that slot value `at` (of pos) names, or -1 for one outside [0, rows): a bad value
// reads and writes nothing.
__device__ __forceinline__ int64_t named_row(int at, int64_t rows) {
  const int r = at < 0 ? ~at : at;
  return r < rows ? r : -1;
}

// Token and unit of a thread: `lane` of run `sub` in workgroup `id`, which holds `per` runs of
// s.lanes units; a token has s.runs runs. False where there is none. Where runs > 1 row_shape
// keeps T * runs below 2^32, so 32 bits hold the run's number q in every workgroup that has
// work, but not in those that fill up the launch's last line.
__host__ __device__ constexpr bool unit_of(const RowShape& s, int64_t id, int per, int sub,
                                           int lane, int64_t* t, int* c) {
  const int64_t q = id * per + sub;
  const int64_t tok = s.runs == 1 ? q : (uint32_t)q / (uint32_t)s.runs;
  *t = tok;
  *c = (int)(q - tok * s.runs) * s.lanes + lane;
  return id < s.groups && tok < s.T;
}

// This thread's token and unit of its row. Workgroups go to the 8 XCDs in turn; BY_XCD gives each
// XCD a run of tokens instead.
template <bool BY_XCD = false, int THREADS = 256>
__device__ __forceinline__ bool my_unit(const RowShape& s, int64_t* t, int* c) {
  const int64_t b = group_id(), per = s.groups / 8;
  const int64_t id = BY_XCD && b < per * 8 ? (b & 7) * per + b / 8 : b;
  return unit_of(s, id, THREADS / s.lanes, threadIdx.x / s.lanes, threadIdx.x & (s.lanes - 1), t, c);
}

// Byte offset of 16-byte unit c of a row of `bytes` >= 16: the last unit ends with the row, so
// where the row is no whole number of units it overlaps the one before and writes the same values
// there. (Rows of 1122 bf16 channels, 40482 tokens of 8 slots, copied and summed: 473 us with a
// last unit in elements, 374 with this one; rows of 318, 19888 tokens of 4 slots, gradients
// 106 / 52.)
__device__ __forceinline__ int64_t unit_at(int c, int64_t bytes) {
  const int64_t o = 16 * (int64_t)c;
  return o < bytes - 16 ? o : bytes - 16;
}

// Slots j0 .. j0 + 7 of token t (none past its k).
struct Slots {
  int at[8];
  __device__ __forceinline__ Slots(const int32_t* pos, const RowShape& s, int64_t t, int j0) {
    const int32_t* p = pos + t * s.k + j0;
#pragma unroll
    for (int i = 0; i < 8; ++i) at[i] = j0 + i < s.k ? p[i] : INT32_MAX;
  }
};

// Xp[pos] = X[token], or zeros for dropped slots. A thread reads 16 bytes of its token's row
// once and writes them to the k rows.
template <int ELEM>
__global__ __launch_bounds__(256) void kg_dispatch_kernel(const unsigned char* __restrict__ X,
                                                          int64_t ldx,
                                                          const int32_t* __restrict__ pos,
                                                          RowShape s,
                                                          unsigned char* __restrict__ Xp) {
  int64_t t;
  int c;
  if (!my_unit<true>(s, &t, &c)) return;
  const int64_t bytes = (int64_t)s.H * ELEM;
  if (16 * (int64_t)c >= bytes) return;
  const unsigned char* x = X + t * ldx * ELEM;
  if (bytes >= 16) {
    const int64_t o = unit_at(c, bytes);
    const v4i v = load16(x + o);
    for (int j0 = 0; j0 < s.k; j0 += 8) {
      const Slots p(pos, s, t, j0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t r = named_row(p.at[i], s.rows);
        if (r >= 0) store16_once(Xp + r * bytes + o, p.at[i] < 0 ? v4i{0, 0, 0, 0} : v);
      }
    }
  } else {
    for (int j = 0; j < s.k; ++j) {
      const int at = pos[t * s.k + j];
      const int64_t r = named_row(at, s.rows);
      if (r < 0) continue;
      for (int e = 0; e < s.H; ++e) {
        if constexpr (ELEM == 2)
          ((unsigned short*)Xp)[r * s.H + e] = at < 0 ? 0 : ((const unsigned short*)x)[e];
        else
          ((uint32_t*)Xp)[r * s.H + e] = at < 0 ? 0 : ((const uint32_t*)x)[e];
      }
    }
  }
}

// Scale blocks of a row, rounded up to whole 16-byte units.
__host__ __device__ constexpr int padded_blocks(int H) { return ((H + 127) / 128 + 3) & ~3; }

// Largest of 8 neighbouring lanes' values.
__device__ __forceinline__ float max8(float v) {
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

// Codes of four quotients x / s (binary32, rounded to nearest; e4m3: nearest, ties to the
// even code), NaN as 0x7F, as kg_requant rounds them. By the choice of s a finite |x / s| stays
// below 464, from where 448 would no longer be the nearest value (the scale of a block of
// subnormal numbers is rounded to 2^-149, which moves it by less than 1/256).
__device__ __forceinline__ int codes4(float a, float b, float c, float d, float s) {
  uint32_t q = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a / s, b / s, 0, false);
  q = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c / s, d / s, (int)q, true);
  // the conversion's NaN is 0xFF or 0x7F: clear the sign of bytes whose low bits are ones
  return (int)(q ^ (((q & 0x7F7F7F7Fu) + 0x01010101u) & q & 0x80808080u));
}

// e4m3 rows: 8 lanes hold one 128-channel block, 16 channels each; its scale is amax / 448 (1
// for a block of zeros). The codes (16 bytes per thread) go to the token's k rows. Here a unit
// is 16 channels.
// The scales belong to k rows of sa [blocks, rows], each a 4-byte store to a line of its own, and
// as many L2 requests as the codes' 128-byte ones. So many of them go to token_sa [T, padded
// blocks] once per token, each row's slot goes to slot_of, and kg_row_scales_kernel writes
// sa along its rows. Measured with 8 slots, 7168 channels, one step / two: 1024 tokens 14.8 /
// 16.7 us, 4096 tokens 47.8 / 48.6, 8192 tokens 138.5 / 124.7 (4.8 TB/s), 16384 tokens
// 278 / 248.
__global__ __launch_bounds__(256) void kg_dispatch_fp8_kernel(const unsigned char* __restrict__ X,
                                                              int64_t ldx,
                                                              const int32_t* __restrict__ pos,
                                                              RowShape s,
                                                              unsigned char* __restrict__ Q,
                                                              float* __restrict__ sa,
                                                              float* __restrict__ token_sa,
                                                              int32_t* __restrict__ slot_of) {
  int64_t t;
  int c;
  if (!my_unit(s, &t, &c)) return;  // whole groups of 16 lanes or more: shuffles stay inside
  const bool in = c < s.H >> 4;     // H is a multiple of 16
  const unsigned char* x = X + t * ldx * 2;
  float f[16] = {};
  if (in) {
    float a[8], b[8];
    Vec<true>::unpack(load16(x + 32 * (int64_t)c), a);
    Vec<true>::unpack(load16(x + 32 * (int64_t)c + 16), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = a[i], f[8 + i] = b[i];
  }
  float amax = 0.f;  // fmaxf passes over NaNs
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
  amax = max8(amax);
  if (!in) return;
  const float sc = amax == 0.f ? 1.0f : amax / 448.0f;
  v4i q;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = codes4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3], sc);
  for (int j0 = 0; j0 < s.k; j0 += 8) {
    const Slots p(pos, s, t, j0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = named_row(p.at[i], s.rows);
      if (r < 0) continue;
      store16_once(Q + r * s.H + 16 * (int64_t)c, p.at[i] < 0 ? v4i{0, 0, 0, 0} : q);
      if (token_sa == nullptr) {
        if ((c & 7) == 0) sa[(int64_t)(c >> 3) * s.rows + r] = p.at[i] < 0 ? 1.0f : sc;
      } else if (c == 0) {
        slot_of[r] = (int32_t)(t * s.k + j0 + i);
      }
    }
  }
  if (token_sa != nullptr && (c & 7) == 0) token_sa[t * padded_blocks(s.H) + (c >> 3)] = sc;
}

// sa[kb][r] for kRowBlocks blocks of 256 rows per workgroup, from the token that row r's slot
// belongs to. slot_of was not cleared: a row that no slot names is told by its slot's
// position, and left alone as in the direct form.
constexpr int kRowBlocks = 8;
__global__ __launch_bounds__(256) void kg_row_scales_kernel(const int32_t* __restrict__ pos,
                                                            const int32_t* __restrict__ slot_of,
                                                            const float* __restrict__ token_sa,
                                                            RowShape s, float* __restrict__ sa) {
  const int64_t r = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (r >= s.rows) return;
  const int slot = slot_of[r];
  if (slot < 0 || slot >= s.rows) return;
  const int at = pos[slot];
  if ((at < 0 ? ~at : at) != r) return;
  const int kb0 = blockIdx.y * kRowBlocks, blocks = (s.H + 127) / 128;
  const float* from = token_sa + (int64_t)(slot / s.k) * padded_blocks(s.H) + kb0;
#pragma unroll
  for (int h = 0; h < kRowBlocks; h += 4) {
    if (kb0 + h >= blocks) break;
    const v4f x = *(const v4f*)(from + h);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (kb0 + h + i < blocks) sa[(int64_t)(kb0 + h + i) * s.rows + r] = at < 0 ? 1.0f : x[i];
  }
}

// out[t] = sum_j w[t][j] Y[pos[t][j]] in fp32, j in order, rounded once. Dropped slots are
// left out, whatever their weight holds. Up to eight rows are read before the first is used.
template <bool BF16>
__global__ __launch_bounds__(256) void kg_combine_kernel(const unsigned char* __restrict__ Y,
                                                         const int32_t* __restrict__ pos,
                                                         const float* __restrict__ w, RowShape s,
                                                         unsigned char* __restrict__ out,
                                                         int64_t ldo) {
  using V = Vec<BF16>;
  int64_t t;
  int c;
  if (!my_unit(s, &t, &c)) return;
  const int64_t bytes = (int64_t)s.H * V::ELEM;
  if (16 * (int64_t)c >= bytes) return;
  const float* wt = w == nullptr ? nullptr : w + t * s.k;
  unsigned char* to = out + t * ldo * V::ELEM;
  if (bytes >= 16) {
    const int64_t o = unit_at(c, bytes);
    float acc[V::N] = {};
    for (int j0 = 0; j0 < s.k; j0 += 8) {
      const Slots p(pos, s, t, j0);
      v4i y[8];
      float wj[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        wj[i] = 1.0f;
        if (p.at[i] >= 0 && p.at[i] < s.rows) {
          y[i] = load16_once(Y + p.at[i] * bytes + o);
          if (wt != nullptr) wj[i] = wt[j0 + i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!(p.at[i] >= 0 && p.at[i] < s.rows)) continue;
        float f[V::N];
        V::unpack(y[i], f);
#pragma unroll
        for (int e = 0; e < V::N; ++e) acc[e] = fmaf(wj[i], f[e], acc[e]);
      }
    }
    store16_once(to + o, V::pack(acc));
  } else {
    for (int e = 0; e < s.H; ++e) {
      float acc = 0.f;
      for (int j = 0; j < s.k; ++j) {
        const int at = pos[t * s.k + j];
        if (at >= 0 && at < s.rows)
          acc = fmaf(wt == nullptr ? 1.0f : wt[j], V::load1(Y + at * bytes + e * V::ELEM), acc);
      }
      V::store1(to + e * V::ELEM, acc);
    }
  }
}

// Scalar loads, for addresses that are the same in a whole wave.
typedef __attribute__((address_space(4))) const int32_t ConstInt;
typedef __attribute__((address_space(4))) const float ConstFloat;

// dY[row] = w dOut[t] (zeros for dropped rows), dw = <dOut[t], Y[row]> (0 for dropped
// slots). S slots at a time: a thread keeps their partial dot products over its channels, then
// the token's threads add theirs in a fixed order. Without dw the units of a token may lie in
// several workgroups (s.runs > 1).
// S = 8 reads dOut once. S = 1 is for few slots: s then counts slots as tokens of one slot,
// `per_row` of them to a row of dOut, so that more compute units share the work (8 slots, 7168
// bf16 channels, S 8 / 1: 16 tokens 12.4 / 4.7 us, 64 tokens 12.7 / 8.0, 128 tokens 15.5 / 15.7,
// 256 tokens 18.6 / 29.0; 2048 channels 6.6 / 4.5, 6.9 / 4.6, 7.1 / 4.9, 7.9 / 8.7; 777 tokens of
// 2 slots, 1235 channels 8.9 / 8.2).
// WAVE: whole waves work on one token (s.lanes >= 64), so its positions and weights are scalars.
template <bool BF16, int S, int THREADS, bool WAVE>
__global__ __launch_bounds__(THREADS) void kg_combine_bwd_kernel(
    const unsigned char* __restrict__ dOut, int64_t ldo, const unsigned char* __restrict__ Y,
    const int32_t* __restrict__ pos, const float* __restrict__ w, RowShape s, int per_row,
    unsigned char* __restrict__ dY, float* __restrict__ dw) {
  using V = Vec<BF16>;
  __shared__ float part[THREADS / 64][S];
  const int lane = threadIdx.x & (s.lanes - 1);
  int64_t t;
  int first;
  const bool live = my_unit<false, THREADS>(s, &t, &first);
  if (!live) t = 0;  // (its threads take part in the sums of others)
  if constexpr (WAVE) t = uniform((int)t);
  const int64_t bytes = (int64_t)s.H * V::ELEM;
  const int units = (int)((bytes + 15) >> 4);
  const unsigned char* d = dOut + (S == 1 ? (uint32_t)t / (uint32_t)per_row : t) * ldo * V::ELEM;
  for (int j0 = 0; j0 < s.k; j0 += S) {
    float dot[S] = {}, wj[S];
    int at[S];
    int kept = 0;  // bit i: slot j0 + i has a row
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const bool on = j0 + i < s.k;
      const int64_t slot = t * s.k + j0 + i;
      if constexpr (WAVE) {
        at[i] = on ? ((const ConstInt*)pos)[slot] : INT32_MAX;
        wj[i] = on && w != nullptr ? ((const ConstFloat*)w)[slot] : 1.0f;
      } else {
        at[i] = on ? pos[slot] : INT32_MAX;
        wj[i] = on && w != nullptr ? w[slot] : 1.0f;
      }
      kept |= (at[i] >= 0 && at[i] < s.rows) << i;
    }
    if (live && bytes >= 16) {
      for (int c = first; c < units; c += s.lanes * s.runs) {
        const int64_t o = unit_at(c, bytes);
        // elements that the unit before has counted
        const int seen = (int)(16 * (int64_t)c - o) / V::ELEM;
        float g[V::N];
        V::unpack(load16(d + o), g);
        v4i y[S];
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (dw != nullptr && (kept >> i & 1))
            y[i] = load16_once(Y + at[i] * bytes + o);
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int64_t r = named_row(at[i], s.rows);
          if (r < 0) continue;
          float f[V::N];
          if (at[i] < 0) {
            store16(dY + r * bytes + o, v4i{0, 0, 0, 0});
            continue;
          }
#pragma unroll
          for (int e = 0; e < V::N; ++e) f[e] = wj[i] * g[e];
          store16_once(dY + r * bytes + o, V::pack(f));
          if (dw != nullptr) {
            V::unpack(y[i], f);
#pragma unroll
            for (int e = 0; e < V::N; ++e)
              if (e >= seen) dot[i] = fmaf(g[e], f[e], dot[i]);
          }
        }
      }
    } else if (live && lane == 0) {
      for (int e = 0; e < s.H; ++e) {
        const int64_t b = e * V::ELEM;
        const float g = V::load1(d + b);
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int64_t r = named_row(at[i], s.rows);
          if (r < 0) continue;
          V::store1(dY + r * bytes + b, at[i] < 0 ? 0.f : wj[i] * g);
          if (dw != nullptr && at[i] >= 0) dot[i] = fmaf(g, V::load1(Y + r * bytes + b), dot[i]);
        }
      }
    }
    if (dw == nullptr) continue;
    const int me = threadIdx.x & 63;
    int mine = 0;  // the sum that this lane ends with
    if constexpr (S == 8) {
      // In the first three steps a lane hands half of its sums over and keeps the other half,
      // so ten shuffles add eight sums over a wave; then lanes 8 m + (0 .. 7) hold sum
      // 4 * bit 0 + 2 * bit 1 + bit 2 of their number.
#pragma unroll
      for (int step = 0; step < 3; ++step) {
        const int half = 4 >> step;
        const bool up = (me >> step) & 1;
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const float keep = up ? dot[half + i] : dot[i], give = up ? dot[i] : dot[half + i];
          dot[i] = keep + __shfl_xor(give, 1 << step, 64);
        }
      }
      mine = 4 * (me & 1) + 2 * ((me >> 1) & 1) + ((me >> 2) & 1);
    }
    for (int o = S; o < s.lanes && o < 64; o <<= 1) dot[0] += __shfl_xor(dot[0], o, 64);
    if (s.lanes > 64) {  // a token's threads are s.lanes / 64 whole waves of the workgroup
      const int wave = threadIdx.x >> 6, begin = wave & ~(s.lanes / 64 - 1);
      __syncthreads();
      if (me < S) part[wave][mine] = dot[0];
      __syncthreads();
      dot[0] = 0.f;
      for (int v = 0; v < s.lanes / 64; ++v) dot[0] += part[begin + v][mine];
    }
    if (live && lane < S && j0 + mine < s.k)
      dw[t * s.k + j0 + mine] = (kept >> mine & 1) ? dot[0] : 0.f;
  }
}

// kg_combine_bwd takes slots one by one while the card holds all the workgroups at once: two of 1024
// threads on each of 256 compute units (on fewer of them it would be slower, not wrong).
constexpr int64_t kSingleGroups = 2 * 256;

// Scales (rows times blocks) from which kg_dispatch_fp8 writes them in a second step.
constexpr int64_t kTwoStepScales = 1 << 21;

static int key_bits(int G) {
  int b = 1;
  while ((1 << b) <= G) ++b;
  return b;
}

// Slots per block of the two-pass plan: whole runs of 64 for each wave.
static int64_t route_block(int64_t n) {
  int64_t per = (n + kSortBlocks - 1) / kSortBlocks;
  per = (per + kSortThreads - 1) / kSortThreads * kSortThreads;
  return per > kSortBlock ? per : kSortBlock;
}
static int64_t route_blocks(int64_t n) { return (n + route_block(n) - 1) / route_block(n); }

// Checks that the row kernels share, and their launch shape. A token's row is cut into units of
// `unit` bytes (the last one partial).
//  SPLIT: runs of `lanes` units (16 to 256, a power of two, the largest of those that leave the
//    fewest threads without a unit), one unit per thread.
//  LOOP: one run of threads loops over the token's units; as many threads as units, up to 256.
//  WIDE: ... up to the 1024 of its workgroups.
// (LOOP with fewer threads, so that fewer are idle in the last turn: kg_combine_bwd on 200 tokens
// of 8 slots, 7168 channels, 24 us with 128, 17 with 256; 4096 tokens 189 / 186.)
enum RowForm { SPLIT, LOOP, WIDE };
static int row_shape(int64_t T, int k, int H, int elem, int unit, RowForm form, RowShape* s) {
  if (T < 0 || k < 0 || H < 0) return KG_ERR_SHAPE;
  if (H > (1 << 24) || k > 4096 || (k > 0 && T > (int64_t)(INT32_MAX - 1) / k) || T > INT32_MAX - 1)
    return KG_ERR_UNSUPPORTED;
  s->T = T;
  s->rows = T * k;
  s->k = k;
  s->H = H;
  const int64_t units = ((int64_t)H * elem + unit - 1) / unit;
  const int most = form == WIDE ? 1024 : 256;
  s->lanes = most;
  int64_t least = INT64_MAX;
  for (int lanes = most; lanes >= 16; lanes /= 2) {
    const int64_t threads = (units + lanes - 1) / lanes * lanes;
    if (form == SPLIT ? threads < least && (lanes >= 64 || units < 64) : lanes >= units) {
      least = threads;
      s->lanes = lanes;
    }
  }
  s->runs = form == SPLIT && units > 0 ? (int)((units + s->lanes - 1) / s->lanes) : 1;
  const int per = most / s->lanes;
  s->groups = (T * s->runs + per - 1) / per;
  return s->groups <= kGroupsX * 65535 && (s->runs == 1 || T * s->runs < ((int64_t)1 << 32) - 256)
             ? KG_OK
             : KG_ERR_UNSUPPORTED;
}

// (without dw the positions come in vector loads: 4096 tokens of 2 slots, 1024 channels 8.7 us,
// with scalar ones 10.8)
template <bool BF16>
static auto combine_bwd_kernel(const RowShape& s, bool need_dw, bool single) {
  if (s.lanes < 64 || !need_dw)
    return single ? kg_combine_bwd_kernel<BF16, 1, 1024, false>
                  : kg_combine_bwd_kernel<BF16, 8, 256, false>;
  return single ? kg_combine_bwd_kernel<BF16, 1, 1024, true>
                : kg_combine_bwd_kernel<BF16, 8, 256, true>;
}

// A row kernel on s.groups workgroups (those past them in the last line have no token).
template <typename... P>
static int launch_rows(void (*fn)(P...), const RowShape& s, int threads, void* stream,
                       typename same<P>::type... args) {
  const int64_t x = s.groups < kGroupsX ? s.groups : kGroupsX;
  return launch2(fn, x, (int)((s.groups + x - 1) / x), threads, 0, stream, args...);
}

}  // namespace kg

using namespace kg;

extern "C" int64_t kg_route_workspace_bytes(int64_t T, int k, int G) {
  if (T < 0 || k < 0 || G < 0 || G > kRouteMaxGroups || k > 4096 || T > INT32_MAX - 1 ||
      (k > 0 && T > (int64_t)(INT32_MAX - 1) / k))
    return -1;
  const int64_t n = T * k;
  return n <= kSoloSlots ? 0 : route_blocks(n) * (G + 1) * 4;
}

extern "C" int kg_route(const int32_t* idx, int64_t T, int k, int G, int32_t* ks, int32_t* pos,
                        int32_t* src, void* workspace, int64_t workspace_bytes, void* stream) {
  if (T < 0 || k < 0 || G < 0 || workspace_bytes < 0) return KG_ERR_SHAPE;
  const int64_t need = kg_route_workspace_bytes(T, k, G);
  if (need < 0) return KG_ERR_UNSUPPORTED;
  const int64_t n = T * k;
  if (G == 0 && n == 0) return KG_OK;
  if ((G > 0 && ks == nullptr) || (n > 0 && (idx == nullptr || pos == nullptr)) ||
      (need > 0 && workspace == nullptr))
    return KG_ERR_NULL;
  if (workspace_bytes < need) return KG_ERR_SHAPE;
  if (((uintptr_t)idx | (uintptr_t)ks | (uintptr_t)pos | (uintptr_t)src |
       (need > 0 ? (uintptr_t)workspace : 0)) & 3)
    return KG_ERR_ALIGN;
  const struct { const void* p; size_t n; } r[5] = {{idx, (size_t)n * 4}, {ks, (size_t)G * 4},
      {pos, (size_t)n * 4}, {src, (size_t)n * 4}, {workspace, (size_t)need}};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (ranges_overlap(r[i].p, r[i].n, r[j].p, r[j].n)) return KG_ERR_ALIAS;
  const int bits = key_bits(G), keys = G + 1;
  if (n <= kSoloSlots) {
    const size_t lds = (size_t)(kSoloWaves + 1) * keys * 4;
    if (lds > 65536 &&
        hipFuncSetAttribute((const void*)kg_route_solo_kernel,
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
      return KG_ERR_HIP;
    return launch(kg_route_solo_kernel, 1, 64 * kSoloWaves, lds, stream, idx, (int)n, G, bits, ks,
                  pos, src);
  }
  const int64_t blocks = route_blocks(n);
  const int per = (int)route_block(n);
  int32_t* counts = (int32_t*)workspace;
  const int rc = launch(kg_route_count_kernel, blocks, kSortThreads, (size_t)keys * 4, stream, idx,
                        n, per, G, counts);
  if (rc != KG_OK) return rc;
  return launch(kg_route_rank_kernel, blocks, kSortThreads, (size_t)(kSortWaves + 1) * keys * 4,
                stream, idx, n, per, G, bits, counts, (int)blocks, ks, pos, src);
}

extern "C" int kg_dispatch(const void* X, int64_t ldx, const int32_t* pos, int64_t T, int k, int H,
                           int type, void* Xp, void* stream) {
  if (type != KG_ROWS_BF16 && type != KG_ROWS_F32) return KG_ERR_DTYPE;
  const int elem = type == KG_ROWS_BF16 ? 2 : 4;
  RowShape s;
  const int rc = row_shape(T, k, H, elem, 16, SPLIT, &s);
  if (rc != KG_OK) return rc;
  if (ldx < H) return KG_ERR_SHAPE;
  if (s.rows == 0 || H == 0) return KG_OK;
  if (X == nullptr || pos == nullptr || Xp == nullptr) return KG_ERR_NULL;
  if ((((uintptr_t)X | (uintptr_t)Xp) & (elem - 1)) || ((uintptr_t)pos & 3)) return KG_ERR_ALIGN;
  const size_t out = (size_t)s.rows * H * elem;
  if (ranges_overlap(X, ((size_t)(T - 1) * ldx + H) * elem, Xp, out) ||
      ranges_overlap(pos, (size_t)s.rows * 4, Xp, out))
    return KG_ERR_ALIAS;
  auto fn = elem == 2 ? kg_dispatch_kernel<2> : kg_dispatch_kernel<4>;
  return launch_rows(fn, s, 256, stream, (const unsigned char*)X, ldx, pos, s, (unsigned char*)Xp);
}

extern "C" int64_t kg_dispatch_fp8_workspace_bytes(int64_t T, int k, int H) {
  RowShape s;
  if (row_shape(T, k, H, 2, 32, SPLIT, &s) != KG_OK) return -1;
  if (s.rows * ((H + 127) / 128) < kTwoStepScales) return 0;
  return T * padded_blocks(H) * 4 + s.rows * 4;
}

extern "C" int kg_dispatch_fp8(const void* X, int64_t ldx, const int32_t* pos, int64_t T, int k,
                               int H, void* Q, float* sa, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  RowShape s;
  if (workspace_bytes < 0) return KG_ERR_SHAPE;
  const int rc = row_shape(T, k, H, 2, 32, SPLIT, &s);
  if (rc != KG_OK) return rc;
  if (ldx < H) return KG_ERR_SHAPE;
  if (H % 16 != 0) return KG_ERR_ALIGN;
  if (s.rows == 0 || H == 0) return KG_OK;
  if (X == nullptr || pos == nullptr || Q == nullptr || sa == nullptr) return KG_ERR_NULL;
  const int64_t need = kg_dispatch_fp8_workspace_bytes(T, k, H);
  const bool two = workspace != nullptr && need > 0 && workspace_bytes >= need;
  if (((uintptr_t)X & 1) || (((uintptr_t)pos | (uintptr_t)sa) & 3) ||
      (two && ((uintptr_t)workspace & 15)))
    return KG_ERR_ALIGN;
  const size_t np = (size_t)s.rows * 4;
  const struct { const void* p; size_t n; bool written; } r[5] = {
      {X, ((size_t)(T - 1) * ldx + H) * 2, false}, {pos, np, false}, {Q, (size_t)s.rows * H, true},
      {sa, (size_t)((H + 127) / 128) * s.rows * 4, true}, {two ? workspace : nullptr, (size_t)need, true}};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (r[j].written && ranges_overlap(r[i].p, r[i].n, r[j].p, r[j].n)) return KG_ERR_ALIAS;
  float* token_sa = two ? (float*)workspace : nullptr;
  int32_t* slot_of = two ? (int32_t*)(token_sa + T * padded_blocks(H)) : nullptr;
  const int e = launch_rows(kg_dispatch_fp8_kernel, s, 256, stream, (const unsigned char*)X, ldx,
                       pos, s, (unsigned char*)Q, sa, token_sa, slot_of);
  if (e != KG_OK || !two) return e;
  const int groups = ((H + 127) / 128 + kRowBlocks - 1) / kRowBlocks;
  return launch2(kg_row_scales_kernel, (s.rows + 255) / 256, groups, 256, 0, stream, pos, slot_of,
                 token_sa, s, sa);
}

extern "C" int kg_combine(const void* Y, const int32_t* pos, const float* w, void* out, int64_t ldo,
                          int64_t T, int k, int H, int type, void* stream) {
  if (type != KG_ROWS_BF16 && type != KG_ROWS_F32) return KG_ERR_DTYPE;
  const int elem = type == KG_ROWS_BF16 ? 2 : 4;
  RowShape s;
  const int rc = row_shape(T, k, H, elem, 16, SPLIT, &s);
  if (rc != KG_OK) return rc;
  if (ldo < H) return KG_ERR_SHAPE;
  if (T == 0 || H == 0) return KG_OK;
  if (out == nullptr || (s.rows > 0 && (Y == nullptr || pos == nullptr))) return KG_ERR_NULL;
  if ((((uintptr_t)Y | (uintptr_t)out) & (elem - 1)) || (((uintptr_t)pos | (uintptr_t)w) & 3))
    return KG_ERR_ALIGN;
  const size_t no = ((size_t)(T - 1) * ldo + H) * elem;
  if (ranges_overlap(Y, (size_t)s.rows * H * elem, out, no) ||
      ranges_overlap(pos, (size_t)s.rows * 4, out, no) ||
      ranges_overlap(w, (size_t)s.rows * 4, out, no))
    return KG_ERR_ALIAS;
  auto fn = elem == 2 ? kg_combine_kernel<true> : kg_combine_kernel<false>;
  return launch_rows(fn, s, 256, stream, (const unsigned char*)Y, pos, w, s,
                (unsigned char*)out, ldo);
}

extern "C" int kg_combine_bwd(const void* dOut, int64_t ldo, const void* Y, const int32_t* pos,
                              const float* w, void* dY, float* dw, int64_t T, int k, int H,
                              int type, void* stream) {
  if (type != KG_ROWS_BF16 && type != KG_ROWS_F32) return KG_ERR_DTYPE;
  const int elem = type == KG_ROWS_BF16 ? 2 : 4;
  RowShape s;
  const int rc = row_shape(T, k, H, elem, 16, dw == nullptr ? SPLIT : LOOP, &s);
  if (rc != KG_OK) return rc;
  RowShape one;
  const bool single = dw != nullptr && row_shape(s.rows, 1, H, elem, 16, WIDE, &one) == KG_OK &&
                      one.groups <= kSingleGroups;
  if (single) s = one;
  if (ldo < H) return KG_ERR_SHAPE;
  if (s.rows == 0) return KG_OK;
  if (pos == nullptr) return KG_ERR_NULL;
  if (H > 0 && (dOut == nullptr || dY == nullptr || (dw != nullptr && Y == nullptr)))
    return KG_ERR_NULL;
  if ((((uintptr_t)dOut | (uintptr_t)Y | (uintptr_t)dY) & (elem - 1)) ||
      (((uintptr_t)pos | (uintptr_t)w | (uintptr_t)dw) & 3))
    return KG_ERR_ALIGN;
  const size_t nd = ((size_t)(T - 1) * ldo + H) * elem, ny = (size_t)s.rows * H * elem;
  const size_t np = (size_t)s.rows * 4;
  const struct { const void* p; size_t n; } in[4] = {{dOut, nd}, {Y, ny}, {pos, np}, {w, np}};
  for (int i = 0; i < 4; ++i)
    if (ranges_overlap(in[i].p, in[i].n, dY, ny) || ranges_overlap(in[i].p, in[i].n, dw, np))
      return KG_ERR_ALIAS;
  if (ranges_overlap(dY, ny, dw, np)) return KG_ERR_ALIAS;
  auto fn = elem == 2 ? combine_bwd_kernel<true>(s, dw != nullptr, single)
                      : combine_bwd_kernel<false>(s, dw != nullptr, single);
  return launch_rows(fn, s, single ? 1024 : 256, stream, (const unsigned char*)dOut, ldo,
                     (const unsigned char*)Y, pos, w, s, k, (unsigned char*)dY, dw);
}
