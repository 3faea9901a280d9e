// kg_fprop_w4.hip -- the forward product of expert rows with 4-bit weights on gfx950, C ABI
// kg_fprop_w4.
//
// y = x w^T per expert as in kg_fprop, with x bf16 and two codes of w in a byte:
//
//   whole numbers  w = (q - z) s, q 0 .. 15, one scale s (and zero point z, or 8) per `group` channels
//   e2m1           w = e2m1(q) 2^(e - 127), one exponent byte e per 32 channels
//
// Products are exact on the bf16 MFMA and summed in fp32: e2m1 values times a power of two are bf16
// numbers, made by the conversion instruction that takes the scale along; whole numbers are bf16
// numbers before their scale, which multiplies the group's sum. The result is rounded once.
//
// Two kernels, as in kg_fprop. Streaming (few rows): W goes from memory into registers, the
// contraction axis is split over a workgroup's waves; W's bytes bound it. Tiled: a workgroup widens
// its outputs' codes once into LDS, beside its tokens.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "kg_device.h"
#include "kg_host.h"
#include "kg_rows.h"
#include "kg_sched.h"
#include "kg_w4_plan.h"
#include "kgwgrad.h"

namespace kg {

struct WParams {
  const unsigned char* A;   // [M_total, K] bf16, row stride lda elements
  const unsigned char* W;   // [G, N, K / 2]
  const unsigned char* sw;  // [G, N, K / group] bf16, fp32 or bytes
  const unsigned char* zp;  // the same shape, or null
  void* D;                  // [M_total, N] fp32 or bf16, row stride ldd
  const int32_t* ms;        // [G]
  int* status;
  int64_t M_total, lda, ldd;
  int G, N, K;
  int tiles_n;
  int lds_rows;      // token rows that the streaming kernel's LDS holds
  int lds_s, lds_z;  // where scales and zero points begin there
  int waves, split;  // waves of a workgroup, and of those that share an output
};

// Formats: whole numbers by channels per scale, and e2m1.
constexpr int kE2M1 = 0;
template <int GRP>
constexpr int kPerScale = GRP == kE2M1 ? 32 : GRP;  // channels
template <int GRP, bool SB>
constexpr int kScaleBytes = GRP == kE2M1 ? 1 : SB ? 2 : 4;

typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc rsrc_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)bytes, kRsrcWord3);
}
__device__ __forceinline__ v4i load16(Rsrc r, uint32_t off) {
  typedef unsigned int v4u __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(v4i, (v4u)__builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ uint32_t load4(Rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t load2(Rsrc r, uint32_t off) {
  return (unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t load1(Rsrc r, uint32_t off) {
  return (unsigned char)__builtin_amdgcn_raw_buffer_load_b8(r, (int)off, 0, 0);
}
__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }

// Eight e2m1 codes times 2^(e - 127), of which `scale` has the exponent bits.
__device__ __forceinline__ v8bf eight_e2m1(uint32_t x, float scale) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 0);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 1);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 2);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 3);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight whole numbers minus z, as bf16 (exact: at most 8 bits).
__device__ __forceinline__ v8bf eight_less(uint32_t x, float z) {
  const uint32_t even = x & 0x0F0F0F0Fu, odd = (x >> 4) & 0x0F0F0F0Fu;
  v4i r;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const float lo = (float)((even >> (8 * b)) & 0xFF) - z, hi = (float)((odd >> (8 * b)) & 0xFF) - z;
    r[b] = (int)__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi),
                                      __builtin_bit_cast(uint32_t, lo), 0x07060302);
  }
  return __builtin_bit_cast(v8bf, r);
}

// Stores N neighbouring outputs of one row, of which `left` exist, at element `at`.
template <bool OUTB, int N>
__device__ __forceinline__ void store_outputs(void* D, int64_t at, int left, const float (&x)[N]) {
  if constexpr (OUTB) {
    typedef unsigned short vec __attribute__((ext_vector_type(N), aligned(2)));
    unsigned short h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = __builtin_bit_cast(unsigned short, (__bf16)x[i]);
    unsigned short* d = (unsigned short*)D + at;
    if (left >= N) {
      vec v;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = h[i];
      *(vec*)d = v;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) d[i] = h[i];
    }
  } else {
    typedef float vec __attribute__((ext_vector_type(N < 4 ? N : 4), aligned(4)));
    constexpr int P = N < 4 ? N : 4;
    float* d = (float*)D + at;
#pragma unroll
    for (int o = 0; o < N; o += P) {
      if (left >= o + P) {
        vec v;
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = x[o + i];
        *(vec*)(d + o) = v;
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i)
          if (o + i < left) d[o + i] = x[o + i];
      }
    }
  }
}

// Waits for this wave's LDS operations, then for the workgroup's other waves; loads into
// registers stay under way.
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(63) & ~0xF00);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// ------------------------------------------------------------------------ streaming kernel

// A workgroup has one expert's rows in LDS, as many at a time as that holds (16 at most), and sets of
// waves with 16 NJ outputs each; the waves of a set take runs of blocks of 128 channels, each with D
// blocks of W under way, and add up in LDS in a fixed order.
//
// Tokens are the MFMA's rows, outputs its columns: a lane holds one output (of each tile), whose
// codes and scales it reads itself, so scales need no exchange between lanes. A workgroup's
// outputs are dealt to its tiles in turn, so a lane has neighbouring ones and stores them together.
//
// A whole-number code is put into the mantissa bits of the bf16 number 16 (two instructions for
// two codes, four channels apart; the tokens' channels are put into the same order). A group's sum of
// x (16 + q) then loses (16 + z) times the group's sum of x, which an MFMA with ones gives in the
// lanes that need it, before it is scaled.
constexpr int kMaxSplit = 8;  // waves that share the contraction axis of an output

// Scales that a lane holds per block of 128 channels (e2m1: of its own 32 channels).
template <int GRP>
constexpr int kScales = GRP == kE2M1 || GRP == 128 ? 1 : 128 / GRP;

// Codes c and c + 4 of eight, c = 0 .. 3, as the bf16 numbers 16 + q. The constants come in a scalar
// and a vector register: written as numbers they cost two instructions where v_and_or_b32 is one.
struct Plus {
  uint32_t mask, base;
  __device__ __forceinline__ Plus() {
    asm("s_mov_b32 %0, 0x00780078" : "=s"(mask));
    asm("v_mov_b32 %0, 0x41804180" : "=v"(base));
  }
};
__device__ __forceinline__ v8bf eight_plus(uint32_t x, const Plus& c) {
  const uint32_t mask = c.mask, base = c.base;
  return __builtin_bit_cast(v8bf, v4i{(int)(((x << 3) & mask) | base), (int)(((x >> 1) & mask) | base),
                                      (int)(((x >> 5) & mask) | base), (int)(((x >> 9) & mask) | base)});
}
// Eight tokens' channels in that order.
__device__ __forceinline__ v8bf by_fours(const v4i& x) {
  const uint32_t a = x.x, b = x.y, c = x.z, d = x.w;
  return __builtin_bit_cast(v8bf, v4i{(int)__builtin_amdgcn_perm(c, a, 0x05040100),
                                      (int)__builtin_amdgcn_perm(c, a, 0x07060302),
                                      (int)__builtin_amdgcn_perm(d, b, 0x05040100),
                                      (int)__builtin_amdgcn_perm(d, b, 0x07060302)});
}

// A lane's 32 channels of one block: lane quad q reads the bytes of channels 32 q .. 32 q + 31 of
// its output, and word j of them meets the tokens' channels 8 chunk<GRP>(q, j) .. + 7. With scales
// per 32 or 64 channels the quads exchange words (a 4 x 4 transposition), so that MFMA j covers
// channels 32 j .. 32 j + 31 alone.
template <int GRP>
__device__ __forceinline__ constexpr int chunk(int q, int j) {
  return GRP == kE2M1 || GRP == 128 ? 4 * q + j : 4 * j + q;
}
template <int GRP>
__device__ __forceinline__ void deal(v4i& x) {
  if constexpr (GRP == 32 || GRP == 64) {
    auto a = __builtin_amdgcn_permlane32_swap((unsigned)x.x, (unsigned)x.z, false, false);
    auto b = __builtin_amdgcn_permlane32_swap((unsigned)x.y, (unsigned)x.w, false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    x = v4i{(int)c[0], (int)c[1], (int)d[0], (int)d[1]};
  }
}

// LDS layout of the tokens: 256-byte blocks of 128 channels, row by row, with 16-byte chunk c of a
// block in slot c ^ key. A 16-byte read serves lanes 0-3, 12-15, 20-27 at a time, then the other 16
// of the lower half (the upper half alike): the 16 tokens once each, some with quad q's chunk and the
// rest with quad q + 1's. The slots are distinct if no two of those tokens' keys differ by the
// two chunks' difference: 1 where quads hold neighbouring chunks, 4 where they hold four each.
template <int GRP>
__device__ __forceinline__ constexpr int key_of(int r) {
  return chunk<GRP>(1, 0) == 1 ? r & 15 : (r & 10) | ((r & 1) << 2) | ((r >> 2) & 1);
}

// `bytes` bytes from memory (at any address) to LDS at smem + at, by all `waves` waves of the workgroup: whole
// 16-byte units straight there, the last few bytes through registers once those have landed
// (they would else be zeroed behind them). Up to the next KB is overwritten.
__device__ __forceinline__ void copy_units(unsigned char* smem, int at, const unsigned char* from,
                                           int bytes, int w, int waves, int lane) {
  const v4i r = make_rsrc(from, (uint32_t)bytes);
  for (int x = w; 1024 * x < bytes; x += waves) {
    const int o = 1024 * x + 16 * lane;
    load16_lds(r, lds_addr(smem) + at + 1024 * x, o + 16 <= bytes ? (uint32_t)o : kOobOffset);
  }
}
__device__ __forceinline__ void copy_rest(unsigned char* smem, int at, const unsigned char* from,
                                          int bytes, int t) {
  const int o = (bytes & ~15) + t;
  if (t < (bytes & 15)) smem[at + o] = from[o];
}

template <int GRP, bool SB, int NJ, bool OUTB>
__global__ __launch_bounds__(1024, 4) void kg_fprop_w4_stream_kernel(WParams p) {
  constexpr int N0 = 16 * NJ, NG = kScales<GRP>;
  constexpr int D = NJ == 2 ? 4 : 6, SBYTES = kScaleBytes<GRP, SB>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int per = p.tiles_n;  // workgroups per expert
  const int sets = p.waves / p.split;  // of waves, with outputs of their own
  const int nth = blockIdx.x / per, n0 = (blockIdx.x - nth * per) * N0 * sets;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, j = lane & 15;
  int64_t row0;
  int rows, g;
  if (!find_rows(p.ms, p.G, p.M_total, nth, &g, &row0, &rows)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = KG_ERR_KSUM;
    return;
  }
  // (known to be one value per wave: buffers are described by scalars)
  g = uniform(g), rows = uniform(rows);
  if (rows == 0) return;  // fewer experts have rows than could: no load is under way yet
  row0 = uniform((int)row0);  // below 2^31
  const int nk = (p.K + 127) / 128, pieces = w_pieces(nk);
  const int kbytes = p.K / 2, groups = p.K / kPerScale<GRP>;
  const int all = min(N0 * sets, p.N - n0);  // outputs of the workgroup
  const int64_t out0 = (int64_t)g * p.N + n0;
  const unsigned char* sbase = p.sw + out0 * groups * SBYTES;
  const unsigned char* zbase = p.zp + out0 * groups;
  // ... and of this wave, the part-th of those that share them
  const int side = w / p.split, part = w - side * p.split, m0 = side * N0;
  const int outs = w_set_outs(all, m0, N0);
  const unsigned char* wbase = p.W + (out0 + (outs ? m0 : 0)) * kbytes;
  const bool zeros = p.zp != nullptr;
  uint32_t woff[NJ];
  int soff[NJ];
#pragma unroll
  for (int i = 0; i < NJ; ++i) {
    woff[i] = (uint32_t)((NJ * j + i) * kbytes + 16 * q);  // past the last output: zeros
    soff[i] = min(m0 + NJ * j + i, all - 1) * groups;
  }
  // the outputs' scales and zero points, which lie side by side
  const int sbytes = all * groups * SBYTES, zbytes = zeros ? all * groups : 0;
  copy_units(smem, p.lds_s, sbase, sbytes, w, p.waves, lane);
  if (zeros) copy_units(smem, p.lds_z, zbase, zbytes, w, p.waves, lane);
  for (int r0 = 0; r0 < rows; r0 += p.lds_rows) {
    const int here = min(p.lds_rows, rows - r0);
    // the tokens, a row's 4 blocks of 256 bytes per load of a wave; channels past K are zeros
    {
      const int64_t lda2 = 2 * p.lda;
      const v4i ar = make_rsrc(p.A + (row0 + r0) * lda2, (uint32_t)((here - 1) * lda2 + 2 * p.K));
      const uint32_t lds = lds_addr(smem);
      int row = 0, piece = w;
      while (piece >= pieces) piece -= pieces, ++row;
      while (row < here) {
        const int ch = 8 * (j ^ key_of<GRP>(row & 15)) + 128 * (4 * piece + q);
        load16_lds(ar, lds + 1024 * (row * pieces + piece),
                   ch < p.K ? (uint32_t)(row * (int)lda2 + 2 * ch) : kOobOffset);
        piece += p.waves;
        while (piece >= pieces) piece -= pieces, ++row;
      }
    }
    v4i wx[D][NJ];
    // This wave's blocks, [from, to); what lies past them reads as zeros.
    const int from = part * nk / p.split, to = (part + 1) * nk / p.split;
    auto load = [&](int kb, int d) {
      const Rsrc wr = rsrc_of(wbase + kb * 64, w_codes_left(outs, kbytes, kb, to));
#pragma unroll
      for (int i = 0; i < NJ; ++i) wx[d][i] = load16(wr, woff[i]);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) load(from + d, d);
    wait_all_and_barrier();
    if (r0 == 0) {
      copy_rest(smem, p.lds_s, sbase, sbytes, threadIdx.x);
      copy_rest(smem, p.lds_z, zbase, zbytes, threadIdx.x);
    }
    if constexpr (GRP != kE2M1) {
      for (int c = threadIdx.x; c < here * pieces * 64; c += 64 * p.waves) {
        v4i* x = (v4i*)smem + c;
        *x = __builtin_bit_cast(v4i, by_fours(*x));
      }
    }
    __syncthreads();
    v4f acc[NJ];
#pragma unroll
    for (int i = 0; i < NJ; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
    // (lanes of rows that do not exist compute row 0 once more)
    const int jr = j < here ? j : 0, key = key_of<GRP>(jr);
    const unsigned char* tok[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
      tok[c] = smem + jr * pieces * 1024 + from * 256 + 16 * (chunk<GRP>(q, c) ^ key);
    auto block = [&](int kb, int d) {
      v4i tx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) tx[c] = *(const v4i*)(tok[c] + 256 * d);
      // (one word of each tile at a time: widened words of a whole block would not fit the registers)
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (GRP == kE2M1) {
        float s[NJ];
#pragma unroll
        for (int i = 0; i < NJ; ++i) {  // (past K: any scale that is a number)
          const int n = 4 * kb + q;
          s[i] = as_float((n < groups ? (uint32_t)smem[p.lds_s + soff[i] + n] : 127u) << 23);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const v8bf x = __builtin_bit_cast(v8bf, tx[c]);
#pragma unroll
          for (int i = 0; i < NJ; ++i)
            acc[i] = mfma_bf16(x, eight_e2m1((uint32_t)wx[d][i][c], s[i]), acc[i]);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        constexpr int one = 0x3F803F80;
        const v8bf ones = __builtin_bit_cast(v8bf, v4i{one, one, one, one});
        const Plus plus;
#pragma unroll
        for (int i = 0; i < NJ; ++i) deal<GRP>(wx[d][i]);
        float sc[NJ][NG], sz[NJ][NG];
#pragma unroll
        for (int i = 0; i < NJ; ++i)
#pragma unroll
          for (int n = 0; n < NG; ++n) {  // (past K: 0)
            const int g = NG * kb + n, at = soff[i] + g;
            const bool in = GRP == 128 || g < groups;
            const unsigned char* f = smem + p.lds_s + at * SBYTES;
            sc[i][n] = !in ? 0.f : SB ? as_float((uint32_t) * (const unsigned short*)f << 16) : *(const float*)f;
            sz[i][n] = 16.f + (zeros ? in ? (float)smem[p.lds_z + at] : 0.f : 8.f);
          }
        v4f sum, part[NJ];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const v8bf x = __builtin_bit_cast(v8bf, tx[c]);
          const bool first = c % (4 / NG) == 0, last = (c + 1) % (4 / NG) == 0;
          sum = mfma_bf16(x, ones, first ? v4f{0.f, 0.f, 0.f, 0.f} : sum);
#pragma unroll
          for (int i = 0; i < NJ; ++i)
            part[i] = mfma_bf16(x, eight_plus((uint32_t)wx[d][i][c], plus),
                                first ? v4f{0.f, 0.f, 0.f, 0.f} : part[i]);
          if (last) {
            const int n = c / (4 / NG);
#pragma unroll
            for (int i = 0; i < NJ; ++i) {
              const float s = sc[i][n], z = sz[i][n];
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[i][r] = fmaf(s, fmaf(-z, sum[r], part[i][r]), acc[i][r]);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    for (int k0 = from; k0 < to; k0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        if (k0 + d < to) block(k0 + d, d);
        load(k0 + d + D, d);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) tok[c] += 256 * D;
    }
    __syncthreads();  // every wave has read the tokens
    v4f* sums = (v4f*)smem;
#pragma unroll
    for (int i = 0; i < NJ; ++i) sums[(w * NJ + i) * 64 + lane] = acc[i];
    __syncthreads();
    if (part < 4) {  // wave r of those that share outputs joins and stores row r of each lane's four
      float x[NJ];
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        const float* f = (const float*)(sums + (side * p.split * NJ + i) * 64 + lane) + part;
        x[i] = f[0];
#pragma unroll
        for (int v = 1; v < kMaxSplit; ++v)
          if (v < p.split) x[i] += f[v * NJ * 64 * 4];
      }
      const int row = 4 * q + part;
      if (row < here)
        store_outputs<OUTB, NJ>(p.D, (row0 + r0 + row) * p.ldd + n0 + m0 + NJ * j, outs - NJ * j, x);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------- tiled kernel

// BT tokens x BN outputs per workgroup of 8 waves, two LDS stages of KS times 64 channels: widened
// weights, tokens, and whole-number codes' scales. Codes, scales and tokens come into registers D
// blocks ahead (the compiler counts those loads); during block kb the threads widen block kb + 1
// into the other stage, a word between MFMAs.
//
// With KS = 2 each half of the waves (WT of them along the tokens) multiplies one half of a block's
// channels, and the halves' sums are joined in LDS at the end. A block's time in a small tile is
// latency, so longer blocks are what makes few tiles fast.
//
// Outputs are the MFMA's rows, tokens its columns, as in kg_fprop: by the order in which
// the outputs are dealt to its rows a lane holds eight neighbouring outputs of one token.
template <int BT_, int BN_, int WT_, int KS_, int D_>
struct WCfg {
  static constexpr int BT = BT_, BN = BN_, WT = WT_, KS = KS_, WN = 8 / KS_ / WT_, D = D_;
  static constexpr int THREADS = 512, TK = 64 * KS;
  static constexpr int TT = BT / WT / 16;  // 16-token tiles of a wave
  static constexpr int NI = BN / WN / 16;  // 16-output tiles of a wave
  static constexpr int OPW = BN * 128, OPT = BT * 128, PART = OPW + OPT + 2 * BN * 4;
  static constexpr int STAGE = KS * PART;
  static constexpr int WORDS = BN * KS / 64;              // of eight codes, of a thread and block
  static constexpr int UNITS = (BT * 8 * KS + 511) / 512; // of 16 bytes of tokens
  static_assert(NI % 2 == 0 && WORDS == 4, "whole runs of outputs, one load of codes");
  static_assert((KS - 1) * BT * BN * 4 <= 2 * STAGE, "the halves' sums fit");
};
// Row m of MFMA row tile i holds output wrow(i, m) of the wave's.
__device__ __forceinline__ constexpr int wrow(int i, int m) {
  return 32 * (i >> 1) + 8 * (m >> 2) + 4 * (i & 1) + (m & 3);
}
// LDS slot of 16-byte chunk c of a row is c ^ key, the key m & 7 of the MFMA row (column) m.
__device__ __forceinline__ constexpr int key_t(int r) { return r & 7; }
__device__ __forceinline__ constexpr int key_w(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }

template <class C, int GRP, bool SB, bool OUTB>
__global__ __launch_bounds__(C::THREADS, 2) void kg_fprop_w4_kernel(WParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int TT = C::TT, NI = C::NI, D = C::D, BN = C::BN, BT = C::BT, KS = C::KS;
  constexpr bool INT = GRP != kE2M1;
  constexpr int NG = GRP == 32 ? 2 : 1;  // scales of an output and block (whole numbers)
  int* off = (int*)(smem + 2 * C::STAGE);  // [G + 1]
  int* boff = off + p.G + 1;
  if (!f_offsets<C::THREADS>(p.ms, p.G, BT, p.M_total, off, boff)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = KG_ERR_KSUM;
    return;
  }
  const int mt_total = boff[p.G], total = mt_total * p.tiles_n;
  const int grid = gridDim.x, b = blockIdx.x;
  // XCD-contiguous runs when the items take several rounds, as in kg_fprop
  const int slot = (grid % 8 == 0 && total > grid) ? (b % 8) * (grid / 8) + b / 8 : b;
  const int nk = (p.K + C::TK - 1) / C::TK, kbytes = p.K / 2, groups = p.K / kPerScale<GRP>;
  const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6);
  const int q = lane >> 4, j = lane & 15;
  const int hk = w / (8 / KS), wt = w % C::WT, wn = w % (8 / KS) / C::WT;
  const int c0 = 16 * (q ^ (j & 7)), c1 = 16 * ((q + 4) ^ (j & 7));
  const unsigned char* own = smem + hk * C::PART;
  const unsigned char* fragw = own + (wn * NI * 16 + wrow(0, j)) * 128;
  const unsigned char* fragt = own + C::OPW + (wt * TT * 16 + j) * 128;
  const unsigned char* scales = own + C::OPW + C::OPT + (wn * NI * 16 + 8 * q) * 4;
  // this thread's codes: words [first, first + WORDS) of eight codes of output `out`
  constexpr int PER_ROW = 512 / BN;
  const int out = t / PER_ROW, first = t % PER_ROW * C::WORDS;
  const int side = first / 8, quarter = first / 4;  // 64 channels, 32 channels of the block
  for (int base = 0; base < total; base += grid) {
    const int idx = base + slot;
    if (idx >= total) break;
    const int per_panel = kPanelM * p.tiles_n;
    const int panel = idx / per_panel, wi = idx - panel * per_panel;
    const int pm = min(kPanelM, mt_total - panel * kPanelM);
    const int mtg = panel * kPanelM + wi % pm, nt = uniform(wi / pm);
    int lo_g = 0, hi_g = p.G;  // expert of m-tile mtg: the last g with boff[g] <= mtg
    while (hi_g - lo_g > 1) {
      const int mid = (lo_g + hi_g) >> 1;
      if (boff[mid] <= mtg) lo_g = mid; else hi_g = mid;
    }
    const int g = uniform(lo_g);
    const int row0 = uniform(off[g] + (mtg - boff[g]) * BT);
    const int rows = uniform(min(BT, off[g + 1] - row0));
    const int n0 = nt * BN, outs = min(BN, p.N - n0);
    const int64_t out0 = (int64_t)g * p.N + n0;
    const unsigned char* wbase = p.W + out0 * kbytes;
    const unsigned char* sbase = p.sw + out0 * groups * kScaleBytes<GRP, SB>;
    const unsigned char* zbase = p.zp ? p.zp + out0 * groups : sbase;
    const unsigned char* abase = p.A + (int64_t)row0 * p.lda * 2;
    const int lda2 = (int)(2 * p.lda);
    const uint32_t woff = (uint32_t)(out * kbytes + 4 * first), soff = (uint32_t)(out * groups + (kPerScale<GRP> == 32 ? quarter : GRP == 64 ? side : 0));
    // Ring of the loads. Rows and outputs that do not exist and blocks past the last one read as
    // zeros; so do the tokens' channels past K.
    v4i ax[D][C::UNITS], wx[D];
    uint32_t sx[D], zx[D];
    auto load_tokens = [&](int kb, int d, int x) {
      const int left = min(2 * C::TK, 2 * p.K - 2 * C::TK * kb);
      const Rsrc ar = rsrc_of(abase + (int64_t)kb * 2 * C::TK,
                              kb < nk ? (uint32_t)((rows - 1) * lda2 + left) : 0u);
      const int u = 512 * x + t, c = u % (8 * KS);
      const bool ok = (BT * 8 * KS % 512 == 0 || u < BT * 8 * KS) && 16 * c < left;
      ax[d][x] = load16(ar, ok ? (uint32_t)(u / (8 * KS) * lda2 + 16 * c) : kOobOffset);
    };
    auto load_codes = [&](int kb, int d) {
      const bool in = kb < nk;
      const int n = kb * C::TK / kPerScale<GRP>;  // an output's first scale
      const Rsrc wr = rsrc_of(wbase + kb * (C::TK / 2),
                              in ? (uint32_t)max(0, outs * kbytes - kb * (C::TK / 2)) : 0u);
      const Rsrc sr = rsrc_of(sbase + n * kScaleBytes<GRP, SB>,
                              in ? (uint32_t)((outs * groups - n) * kScaleBytes<GRP, SB>) : 0u);
      wx[d] = load16(wr, woff);
      // (the last channels of K's last block may not exist)
      const bool exists = C::TK * kb + 32 * quarter < p.K;
      const uint32_t at = exists ? soff : kOobOffset / 4;
      if constexpr (!INT) {
        sx[d] = load1(sr, at);
      } else {
        sx[d] = SB ? load2(sr, 2 * at) : load4(sr, 4 * at);
        zx[d] = load1(rsrc_of(zbase + n, in ? (uint32_t)(outs * groups - n) : 0u), at);
      }
    };
    v4f acc[NI][TT];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[i][tt] = v4f{0.f, 0.f, 0.f, 0.f};
    // What this thread writes of block kb, held in slot d, into its stage
    auto put_tokens = [&](int kb, int d, int x) {
      const int u = 512 * x + t, r = u / (8 * KS), c = u % (8 * KS);
      if (BT * 8 * KS % 512 == 0 || u < BT * 8 * KS)
        *(v4i*)(smem + (kb & 1) * C::STAGE + c / 8 * C::PART + C::OPW + r * 128 +
                16 * ((c & 7) ^ key_t(r))) = ax[d][x];
    };
    auto put_word = [&](int kb, int d, int n) {
      v8bf v;
      if constexpr (INT) v = eight_less((uint32_t)wx[d][n], p.zp ? (float)zx[d] : 8.f);
      else v = eight_e2m1((uint32_t)wx[d][n], as_float(sx[d] << 23));
      *(v8bf*)(smem + (kb & 1) * C::STAGE + side * C::PART + out * 128 +
               16 * ((first % 8 + n) ^ key_w(out))) = v;
    };
    auto put_scale = [&](int kb, int d) {
      if constexpr (INT)
        if (first % (GRP == 32 ? 4 : 8) == 0)
          *(float*)(smem + (kb & 1) * C::STAGE + side * C::PART + C::OPW + C::OPT +
                    ((GRP == 32 ? quarter % 2 : 0) * BN + out) * 4) = as_float(SB ? sx[d] << 16 : sx[d]);
    };
    v8bf tf[TT][2], wf[2][2];
    v4f sc[3][NG];
    auto read_t = [&](int kb, int tt) {
      const unsigned char* r = fragt + (kb & 1) * C::STAGE + 16 * tt * 128;
      tf[tt][0] = *(const v8bf*)(r + c0);
      tf[tt][1] = *(const v8bf*)(r + c1);
    };
    auto read_w = [&](int kb, int i) {
      const unsigned char* r = fragw + (kb & 1) * C::STAGE + wrow(i, 0) * 128;
      wf[i & 1][0] = *(const v8bf*)(r + c0);
      wf[i & 1][1] = *(const v8bf*)(r + c1);
      if constexpr (INT) {
#pragma unroll
        for (int n = 0; n < NG; ++n)
          sc[i % 3][n] = *(const v4f*)(scales + (kb & 1) * C::STAGE + (n * BN + wrow(i, 0)) * 4);
      }
    };
    auto load = [&](int kb, int d) {
      load_codes(kb, d);
#pragma unroll
      for (int x = 0; x < C::UNITS; ++x) load_tokens(kb, d, x);
    };
    if (nk > 0) {
#pragma unroll
      for (int d = 0; d < D; ++d) load(d, d);
#pragma unroll
      for (int n = 0; n < C::WORDS; ++n) put_word(0, 0, n);
      put_scale(0, 0);
#pragma unroll
      for (int x = 0; x < C::UNITS; ++x) put_tokens(0, 0, x);
      load(D, 0);
      meet();
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) read_t(0, tt);
    }
    // Block kb; block kb + 1 is in slot d, and written to its stage in turn with the MFMAs before the
    // last tile of outputs. One meeting per block, there: behind it the next block's tokens are read,
    // and every wave has read this block's weights, whose stage the next block writes to.
    auto block = [&](int kb, int d) {
      constexpr int S = NI * 2 * TT, LAST = S - 2 * TT, WORK = C::WORDS + C::UNITS;
      v4f part[2][TT];
      auto add = [&](int i, int tt, int n) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][tt][r] = fmaf(sc[i % 3][n][r], part[i & 1][tt][r], acc[i][tt][r]);
        asm volatile("" : "+v"(acc[i][tt]));
      };
      read_w(kb, 0);
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const int i = u / (2 * TT), h = u / TT % 2, tt = u % TT;
        if (u == LAST) meet();
        if (h == 0 && tt == 0 && i + 1 < NI) read_w(kb, i + 1);
        if constexpr (INT) {
          const bool fresh = h == 0 || NG == 2;
          // sums are scaled and added half a tile after their last MFMA was issued
          if (h == 0 && i > 0) add(i - 1, tt, NG - 1);
          if (h == 1 && NG == 2) add(i, tt, 0);
          part[i & 1][tt] = mfma_bf16(wf[i & 1][h], tf[tt][h],
                                      fresh ? v4f{0.f, 0.f, 0.f, 0.f} : part[i & 1][tt]);
        } else {
          acc[i][tt] = mfma_bf16(wf[i & 1][h], tf[tt][h], acc[i][tt]);
        }
        if (i == NI - 1 && h == 1) read_t(kb + 1, tt);  // (past the last block: not used)
#pragma unroll
        for (int x = 0; x < WORK; ++x) {
          if (x * LAST / WORK != u) continue;
          if (x < C::WORDS) {
            put_word(kb + 1, d, x);
            if (x == C::WORDS - 1) {
              put_scale(kb + 1, d);
              load_codes(kb + 1 + D, d);
            }
          } else {
            put_tokens(kb + 1, d, x - C::WORDS);
            load_tokens(kb + 1 + D, d, x - C::WORDS);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (INT) {
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) add(NI - 1, tt, NG - 1);
      }
    };
    for (int k0 = 0; k0 < nk; k0 += D) {
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (k0 + d < nk) block(k0 + d, (d + 1) % D);
    }
    if constexpr (KS == 2) {
      v4f* sums = (v4f*)smem + (w % 4) * NI * TT * 64 + lane;
      __syncthreads();  // every wave has read the last stage
      if (hk == 1) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int tt = 0; tt < TT; ++tt) sums[(i * TT + tt) * 64] = acc[i][tt];
      }
      __syncthreads();
      if (hk == 0) {
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int tt = 0; tt < TT; ++tt) {
            const v4f y = sums[(i * TT + tt) * 64];
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[i][tt][r] += y[r];
          }
      }
      __syncthreads();  // the next tile's first stage may take their place
    }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int r = (wt * TT + tt) * 16 + j;
      if (r >= rows || hk != 0) continue;
      const int64_t at = (int64_t)(row0 + r) * p.ldd + n0;
#pragma unroll
      for (int i = 0; i < NI; i += 2) {
        const int n = wn * NI * 16 + 16 * i + 8 * q;
        const float x[8] = {acc[i][tt][0],     acc[i][tt][1],     acc[i][tt][2],     acc[i][tt][3],
                            acc[i + 1][tt][0], acc[i + 1][tt][1], acc[i + 1][tt][2], acc[i + 1][tt][3]};
        store_outputs<OUTB, 8>(p.D, at + n, outs - n, x);
      }
    }
  }
}

struct WLaunch {
  const void* fn;
  int bt, bn, lds;
};

// The kernel by type: format, scale type, result type.
template <template <int, bool, bool> class F>
static const void* w_pick(int kind, int group, bool outb) {
  if (kind == KG_W4_E2M1) return outb ? F<kE2M1, false, true>::fn() : F<kE2M1, false, false>::fn();
  const bool sb = kind == KG_W4_INT_BF16;
#define KG_W4_GROUP(g)                                                      \
  (sb ? (outb ? F<g, true, true>::fn() : F<g, true, false>::fn())           \
      : (outb ? F<g, false, true>::fn() : F<g, false, false>::fn()))
  return group == 32 ? KG_W4_GROUP(32) : group == 64 ? KG_W4_GROUP(64) : KG_W4_GROUP(128);
#undef KG_W4_GROUP
}
template <int NJ>
struct StreamOf {
  template <int GRP, bool SB, bool OUTB>
  struct F {
    static const void* fn() { return (const void*)kg_fprop_w4_stream_kernel<GRP, SB, NJ, OUTB>; }
  };
};
template <class C>
struct TiledOf {
  template <int GRP, bool SB, bool OUTB>
  struct F {
    static const void* fn() { return (const void*)kg_fprop_w4_kernel<C, GRP, SB, OUTB>; }
  };
};
template <class C>
static WLaunch w_tiled(int kind, int group, bool outb) {
  return WLaunch{w_pick<TiledOf<C>::template F>(kind, group, outb), C::BT, C::BN, 2 * C::STAGE};
}

// The tiled kernel of w_tile's choice.
static WLaunch w_tiled(const WTile& t, int kind, int group, bool outb) {
  // (256 x 256 for e2m1 only: with the sums of whole numbers' groups it does not fit the registers)
  using Large = WCfg<256, 256, 4, 1, 1>;
  return t.bt == 32    ? w_tiled<WCfg<32, 128, 1, 2, 2>>(kind, group, outb)
         : t.bt == 64  ? w_tiled<WCfg<64, 128, 2, 2, 2>>(kind, group, outb)
         : t.bn == 128 ? w_tiled<WCfg<128, 128, 2, 2, 1>>(kind, group, outb)
         : t.bt == 128 ? w_tiled<WCfg<128, 256, 2, 1, 2>>(kind, group, outb)
                       : WLaunch{outb ? (const void*)kg_fprop_w4_kernel<Large, kE2M1, false, true>
                                      : (const void*)kg_fprop_w4_kernel<Large, kE2M1, false, false>,
                                 Large::BT, Large::BN, 2 * Large::STAGE};
}

// Lets a kernel have all of a compute unit's LDS, once per kernel and device.
static bool w_lds_allowed(const void* fn, int dev) {
  static std::mutex mu;
  static const void* set[64][128];
  static int count[64];
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 0; i < count[dev]; ++i)
    if (set[dev][i] == fn) return true;
  if (hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)kWLds) != hipSuccess)
    return false;
  if (count[dev] < 128) set[dev][count[dev]++] = fn;
  return true;
}

}  // namespace kg

extern "C" int kg_fprop_w4(const void* A, int64_t lda, const void* W, const void* sw,
                           const void* zp, void* D, int64_t ldd, const int32_t* ms, int G, int N,
                           int K, int64_t M_total, int group, int kind, int flags, void* stream) {
  using namespace kg;
  if (kind < KG_W4_INT_BF16 || kind > KG_W4_E2M1 || (flags & ~KG_FLAG_D_BF16)) return KG_ERR_DTYPE;
  const bool outb = (flags & KG_FLAG_D_BF16) != 0, mx = kind == KG_W4_E2M1;
  if (G < 0 || N < 0 || K < 0 || M_total < 0 || lda < K || ldd < N) return KG_ERR_SHAPE;
  if (mx ? group != 32 : group != 32 && group != 64 && group != 128) return KG_ERR_GRAN;
  if (G > kMaxGroups || N > (1 << 24) || lda > (1 << 22) || M_total > INT32_MAX || ldd > (1 << 30))
    return KG_ERR_UNSUPPORTED;
  if (K % group != 0 || lda % 8 != 0) return KG_ERR_ALIGN;
  if (G == 0 || N == 0 || M_total == 0) return KG_OK;
  if (!D || !ms || (K > 0 && (!A || !W || !sw))) return KG_ERR_NULL;
  if (mx && zp) return KG_ERR_DTYPE;
  const int el = outb ? 2 : 4, sb = mx ? 1 : kind == KG_W4_INT_BF16 ? 2 : 4;
  if (((uintptr_t)A & 15) || ((uintptr_t)W & 15) || ((uintptr_t)sw & (sb - 1)) ||
      ((uintptr_t)D & (el - 1)) || ((uintptr_t)ms & 3))
    return KG_ERR_ALIGN;
  const size_t dbytes = ((size_t)(M_total - 1) * ldd + N) * el;
  const size_t scales = (size_t)G * N * (K / group);
  if (ranges_overlap(A, ((size_t)(M_total - 1) * lda + K) * 2, D, dbytes) ||
      ranges_overlap(W, (size_t)G * N * (K / 2), D, dbytes) ||
      ranges_overlap(sw, scales * sb, D, dbytes) || ranges_overlap(zp, scales, D, dbytes) ||
      ranges_overlap(ms, (size_t)G * 4, D, dbytes))
    return KG_ERR_ALIAS;
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return KG_ERR_HIP;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return KG_ERR_HIP;
  WParams p;
  p.A = (const unsigned char*)A;
  p.W = (const unsigned char*)W;
  p.sw = (const unsigned char*)sw;
  p.zp = (const unsigned char*)zp;
  p.D = D;
  p.ms = ms;
  p.status = status_word_address();
  if (p.status == nullptr) return KG_ERR_HIP;
  p.M_total = M_total;
  p.lda = lda;
  p.ldd = ldd;
  p.G = G;
  p.N = N;
  p.K = K;
  p.lds_rows = p.lds_s = p.lds_z = 0;
  p.waves = p.split = 8;
  WLaunch l;
  int64_t grid;
  int threads = 512;
  const WStream st = w_stream(M_total, G, N, K, cus, kind, group, zp != nullptr);
  const int64_t live = G < M_total ? G : M_total;
  const WTile tile = w_tile(M_total, G, N, K, cus, kind);
  if (w_streams(st, tile)) {
    const int bn = 16 * st.nj * st.waves / st.split;
    l.fn = st.nj == 1 ? w_pick<StreamOf<1>::F>(kind, group, outb) : w_pick<StreamOf<2>::F>(kind, group, outb);
    l.lds = (int)st.lds;
    p.lds_rows = (int)st.rows;
    p.waves = st.waves, p.split = st.split;
    threads = 64 * st.waves;
    p.lds_s = (int)st.tokens;
    p.lds_z = (int)(st.tokens + st.scales);
    p.tiles_n = (N + bn - 1) / bn;
    grid = live * p.tiles_n;
    if (grid > INT32_MAX / 1024) return KG_ERR_UNSUPPORTED;
  } else {
    l = w_tiled(tile, kind, group, outb);
    l.lds += 2 * (G + 1) * 4;
    p.tiles_n = (N + l.bn - 1) / l.bn;
    const int64_t max_items = (M_total / l.bt + G) * (int64_t)p.tiles_n;
    if (max_items > INT32_MAX - 4096) return KG_ERR_UNSUPPORTED;  // (indexes pass it by a grid)
    grid = max_items < cus ? max_items : cus;
  }
  if (!w_lds_allowed(l.fn, dev)) return KG_ERR_HIP;
  void* args[] = {&p};
  return hipLaunchKernel(l.fn, dim3((unsigned)grid), dim3((unsigned)threads), args, (size_t)l.lds,
                         (hipStream_t)stream) == hipSuccess
             ? KG_OK
             : KG_ERR_HIP;
}
