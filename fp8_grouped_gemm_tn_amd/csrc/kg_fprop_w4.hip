// kg_fprop_w4.hip -- the forward product of expert rows with 4-bit weights on gfx950, C ABI
// kg_fprop_w4.
//
// y = x w^T per expert as in kg_fprop, with x bf16 and two codes of w in a byte:
//
//   whole numbers  w = (q - z) s, q 0 .. 15, one scale s (and zero point z, or 8) per `group` channels
//   e2m1           w = e2m1(q) 2^(e - 127), one exponent byte e per 32 channels
//
// Products are exact on the bf16 MFMA: e2m1 values times a power of two are bf16 numbers, made by
// the conversion instruction that takes the scale along; whole-number codes become 16 + q by
// putting q into the mantissa bits of the bf16 number 16. A group's sum of x (16 + q) then loses
// (16 + z) times the group's sum of x, which an MFMA with ones gives in the lanes that need it, and
// is scaled and added in fp32. The result is rounded once.
//
// Tokens are the MFMA's rows, outputs its columns: a lane holds one output (of each tile), whose
// codes and scales it reads itself, so scales need no exchange between lanes. A wave's outputs are
// dealt to its tiles in turn, so a lane has neighbouring ones and stores them together.
//
// Two kernels, as in kg_fprop. Streaming (few rows): W goes from memory into registers, the
// contraction axis is split over a workgroup's waves; W's bytes bound it. Tiled: tokens go through
// LDS, each wave reads and widens its own outputs' codes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "kg_device.h"
#include "kg_host.h"
#include "kg_rows.h"
#include "kg_sched.h"
#include "kgwgrad.h"

namespace kg {

struct WParams {
  const unsigned char* A;   // [M_total, K] bf16, row stride lda elements
  const unsigned char* W;   // [G, N, K / 2]
  const void* sw;           // [G, N, K / group]
  const unsigned char* zp;  // the same shape, or null
  void* D;                  // [M_total, N] fp32 or bf16, row stride ldd
  const int32_t* ms;        // [G]
  int* status;
  int64_t M_total, lda, ldd;
  int G, N, K;
  int tiles_n;
};

// Formats: whole numbers by channels per scale, and e2m1.
constexpr int kE2M1 = 0;
// Scales that a lane holds per block of 128 channels (e2m1: of its own 32 channels).
template <int GRP>
constexpr int kScales = GRP == kE2M1 || GRP == 128 ? 1 : 128 / GRP;

// Two codes (a byte) become 16 + q: the byte goes into the upper half of both 16-bit lanes, from
// where the shifts bring either nibble to bits 3 .. 6.
typedef unsigned short v2us __attribute__((ext_vector_type(2)));
template <int B>
__device__ __forceinline__ int two_codes(uint32_t x) {
  v2us h = __builtin_bit_cast(v2us, __builtin_amdgcn_perm(x, x, 0x000C000Cu | B << 24 | B << 8));
  h = h >> v2us{5, 9};
  return (int)((__builtin_bit_cast(uint32_t, h) & 0x00780078u) | 0x41804180u);
}

// Eight codes as the MFMA reads them.
template <int GRP>
__device__ __forceinline__ v8bf eight_codes(uint32_t x, float scale) {
  if constexpr (GRP == kE2M1) {
    const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 0);
    const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 1);
    const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 2);
    const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 3);
    return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
  } else {
    return __builtin_bit_cast(
        v8bf, v4i{two_codes<0>(x), two_codes<1>(x), two_codes<2>(x), two_codes<3>(x)});
  }
}

// A lane's 32 channels of one block: lane quad q reads the bytes of channels 32 q .. 32 q + 31 of
// its output, and word j of them meets the tokens' channels chunk<GRP>(q, j) .. + 7. With scales
// per 32 or 64 channels the quads exchange words (a 4 x 4 transposition), so that MFMA j covers
// channels 32 j .. 32 j + 31 alone.
template <int GRP>
__device__ __forceinline__ constexpr int chunk(int q, int j) {  // of 8 channels
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

// A lane's scales of one block (and what is subtracted per unit of x: 16 + z).
template <int GRP>
struct Scales {
  float s[kScales<GRP>], z[kScales<GRP>];
};
typedef unsigned short us2_any __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned short us4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f2_any __attribute__((ext_vector_type(2), aligned(4)));
typedef float f4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned char uc2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef unsigned char uc4_any __attribute__((ext_vector_type(4), aligned(1)));
__device__ __forceinline__ float bf(unsigned short h) {
  return __builtin_bit_cast(float, (uint32_t)h << 16);
}

// Scales of block kb of the output whose scales begin at element `at`; `left` groups of this
// block exist (kScales unless TAIL).
template <int GRP, bool SB, bool TAIL>
__device__ __forceinline__ Scales<GRP> load_scales(const WParams& p, int64_t at, int kb, int q,
                                                   int left) {
  constexpr int NG = kScales<GRP>;
  Scales<GRP> r;
  if constexpr (GRP == kE2M1) {
    const unsigned char* e = (const unsigned char*)p.sw + at + 4 * kb;
    const int byte = !TAIL || q < left ? e[q] : 127;
    r.s[0] = __builtin_bit_cast(float, (uint32_t)byte << 23);
    r.z[0] = 0.f;
  } else {
    const int64_t o = at + (int64_t)NG * kb;
    // without zero points the bytes of the scales are read in their place, and not used
    const unsigned char* z = (p.zp ? p.zp : (const unsigned char*)p.sw) + o;
    int zi[NG];
    if constexpr (TAIL || NG == 1) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const bool in = !TAIL || i < left;
        if constexpr (SB) r.s[i] = in ? bf(((const unsigned short*)p.sw)[o + i]) : 0.f;
        else r.s[i] = in ? ((const float*)p.sw)[o + i] : 0.f;
        zi[i] = in ? z[i] : 0;
      }
    } else if constexpr (NG == 2) {
      if constexpr (SB) {
        const us2_any h = *(const us2_any*)((const unsigned short*)p.sw + o);
        r.s[0] = bf(h[0]), r.s[1] = bf(h[1]);
      } else {
        const f2_any f = *(const f2_any*)((const float*)p.sw + o);
        r.s[0] = f[0], r.s[1] = f[1];
      }
      const uc2_any b = *(const uc2_any*)z;
      zi[0] = b[0], zi[1] = b[1];
    } else {
      if constexpr (SB) {
        const us4_any h = *(const us4_any*)((const unsigned short*)p.sw + o);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.s[i] = bf(h[i]);
      } else {
        const f4_any f = *(const f4_any*)((const float*)p.sw + o);
#pragma unroll
        for (int i = 0; i < 4; ++i) r.s[i] = f[i];
      }
      const uc4_any b = *(const uc4_any*)z;
#pragma unroll
      for (int i = 0; i < 4; ++i) zi[i] = b[i];
    }
#pragma unroll
    for (int i = 0; i < NG; ++i) r.z[i] = 16.f + (p.zp ? (float)zi[i] : 8.f);
  }
  return r;
}

__device__ __forceinline__ v8bf ones() {
  constexpr int one = 0x3F803F80;
  return __builtin_bit_cast(v8bf, v4i{one, one, one, one});
}

// Adds one block: the widened codes w[i][j] (word j of output tile i) and a token tile's words t[j].
template <int GRP, int NI>
__device__ __forceinline__ void add_block(const v8bf (&w)[NI][4], const Scales<GRP> (&sc)[NI],
                                          const v8bf (&t)[4], v4f (&acc)[NI]) {
  if constexpr (GRP == kE2M1) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i] = mfma_bf16(t[j], w[i][j], acc[i]);
  } else {
    constexpr int NG = kScales<GRP>, PER = 4 / NG;  // MFMAs per group
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      v4f sum = {0.f, 0.f, 0.f, 0.f}, part[NI];
#pragma unroll
      for (int j = g * PER; j < (g + 1) * PER; ++j) {
        sum = mfma_bf16(t[j], ones(), sum);
#pragma unroll
        for (int i = 0; i < NI; ++i)
          part[i] = mfma_bf16(t[j], w[i][j], j == g * PER ? v4f{0.f, 0.f, 0.f, 0.f} : part[i]);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][r] = fmaf(sc[i].s[g], fmaf(-sc[i].z[g], sum[r], part[i][r]), acc[i][r]);
    }
  }
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
    typedef float vec __attribute__((ext_vector_type(N), aligned(4)));
    float* d = (float*)D + at;
    if (left >= N) {
      vec v;
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = x[i];
      *(vec*)d = v;
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) d[i] = x[i];
    }
  }
}

__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  typedef unsigned int v4u __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)bytes, kRsrcWord3);
}

// ------------------------------------------------------------------------ streaming kernel

// A workgroup computes 16 NJ outputs of one expert for all its rows, 16 TT at a time; its 8 waves
// take the blocks of 128 channels in turn, with the next block's operands on their way, and add
// up in LDS in a fixed order. Rows, outputs and channels that do not exist read as zeros.
constexpr int kW4Waves = 8;

template <int GRP, bool SB, int TT, int NJ, bool OUTB>
__global__ __launch_bounds__(64 * kW4Waves) void kg_fprop_w4_stream_kernel(WParams p) {
  constexpr int N0 = 16 * NJ;
  __shared__ v4f sums[kW4Waves][TT * NJ][64];
  const int per = p.tiles_n;  // workgroups per expert
  const int nth = blockIdx.x / per, n0 = (blockIdx.x - nth * per) * N0;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, j = lane & 15;
  int64_t row0;
  int rows, g;
  if (!find_rows(p.ms, p.G, p.M_total, nth, &g, &row0, &rows)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = KG_ERR_KSUM;
    return;
  }
  if (rows == 0) return;
  const int nk = (p.K + 127) / 128, nfull = p.K / 128, kbytes = p.K / 2;
  const int outs = min(N0, p.N - n0);
  const int64_t out0 = (int64_t)g * p.N + n0;
  const __amdgpu_buffer_rsrc_t wr = rsrc_of(p.W + out0 * kbytes, (uint32_t)(outs * kbytes));
  uint32_t woff[NJ];
  int64_t sat[NJ];
#pragma unroll
  for (int i = 0; i < NJ; ++i) {
    woff[i] = (uint32_t)((NJ * j + i) * kbytes + 16 * q);
    sat[i] = (out0 + min(NJ * j + i, outs - 1)) * (p.K / (GRP == kE2M1 ? 32 : GRP));
  }
  for (int r0 = 0; r0 < rows; r0 += 16 * TT) {
    const int here = min(16 * TT, rows - r0);
    const int64_t lda2 = 2 * p.lda;
    const __amdgpu_buffer_rsrc_t ar =
        rsrc_of(p.A + (row0 + r0) * lda2, (uint32_t)((here - 1) * lda2 + 2 * p.K));
    uint32_t aoff[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) aoff[tt] = (uint32_t)((16 * tt + j) * lda2);
    v4f acc[TT][NJ];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
      for (int i = 0; i < NJ; ++i) acc[tt][i] = v4f{0.f, 0.f, 0.f, 0.f};
    v4i wx[2][NJ], tx[2][TT][4];
    Scales<GRP> sc[2][NJ];
    auto load = [&](int kb, int h) {
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        wx[h][i] = load16(wr, woff[i] + (uint32_t)kb * 64);
        sc[h][i] = load_scales<GRP, SB, false>(p, sat[i], kb, q, 4);
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tx[h][tt][c] = load16(ar, aoff[tt] + (uint32_t)kb * 256 + 16 * chunk<GRP>(q, c));
    };
    auto block = [&](int h) {
      v8bf wf[NJ][4];
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        deal<GRP>(wx[h][i]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          wf[i][c] = eight_codes<GRP>((uint32_t)wx[h][i][c], sc[h][i].s[0]);
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        v8bf t[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) t[c] = __builtin_bit_cast(v8bf, tx[h][tt][c]);
        add_block<GRP, NJ>(wf, sc[h], t, acc[tt]);
      }
    };
    // This wave's blocks w, w + 8, ...; every load in the loop is unconditional, so the compiler
    // counts how many are under way.
    const int nb = nfull > w ? (nfull - w + kW4Waves - 1) / kW4Waves : 0;
    int n = 0, kb = w;
    if (nb > 0) load(kb, 0);
    for (; n + 2 < nb; n += 2, kb += 2 * kW4Waves) {
      load(kb + kW4Waves, 1);
      block(0);
      __builtin_amdgcn_sched_barrier(0);
      load(kb + 2 * kW4Waves, 0);
      block(1);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (n + 1 < nb) {
      load(kb + kW4Waves, 1);
      block(0);
      block(1);
    } else if (n < nb) {
      block(0);
    }
    if constexpr (GRP != 128) {
      if (nfull < nk && w == nfull % kW4Waves) {  // the last block's K % 128 channels
        const int left = p.K - nfull * 128;
#pragma unroll
        for (int i = 0; i < NJ; ++i) {
          wx[0][i] = load16(wr, woff[i] + (uint32_t)nfull * 64);
          sc[0][i] =
              load_scales<GRP, SB, true>(p, sat[i], nfull, q, left / (GRP == kE2M1 ? 32 : GRP));
        }
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int ch = 8 * chunk<GRP>(q, c);
            tx[0][tt][c] = load16(
                ar, ch < left ? aoff[tt] + (uint32_t)nfull * 256 + 2 * ch : kOobOffset);
          }
        block(0);
      }
    }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
      for (int i = 0; i < NJ; ++i) sums[w][tt * NJ + i][lane] = acc[tt][i];
    __syncthreads();
    // wave w joins and stores row r = w % 4 of each lane's four of token tile w / 4
    for (int u = w; u < 4 * TT; u += kW4Waves) {
      const int tt = u >> 2, r = u & 3;
      float x[NJ];
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        x[i] = sums[0][tt * NJ + i][lane][r];
#pragma unroll
        for (int v = 1; v < kW4Waves; ++v) x[i] += sums[v][tt * NJ + i][lane][r];
      }
      const int row = r0 + 16 * tt + 4 * q + r;
      if (row < rows)
        store_outputs<OUTB, NJ>(p.D, (row0 + row) * p.ldd + n0 + NJ * j, outs - NJ * j, x);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------- tiled kernel

// BT tokens x BN outputs per workgroup of 8 waves (WT along the tokens), two stages of one block of
// 128 channels of the tokens in LDS; codes and scales go into registers one block ahead.
template <int BT_, int BN_, int WT_>
struct WCfg {
  static constexpr int BT = BT_, BN = BN_, WT = WT_, WN = 8 / WT_, THREADS = 512;
  static constexpr int TT = BT / WT / 16;  // 16-token tiles of a wave
  static constexpr int NI = BN / WN / 16;  // 16-output tiles of a wave
  static constexpr int STAGE = BT * 256;
  static constexpr int LOADS = (BT + 31) / 32;  // a wave's 1 KB loads of a stage
  static_assert(BT % 16 == 0 && BT * 256 % 1024 == 0, "whole wave loads");
};

// LDS layout: a token's 256 bytes in order, but its 16-byte chunk c in slot c ^ key. A 16-byte read
// serves lanes 0-3, 12-15, 20-27 at a time, then the other 16 of the lower half (the upper half
// alike): the tokens of a tile once each, some with quad q's chunk and the rest with quad
// q + 1's. The slots are distinct if no two of those tokens' keys differ by the two chunks'
// difference: 1 where quads hold neighbouring chunks, 4 where they hold four each.
template <int GRP>
__device__ __forceinline__ constexpr int key_of(int r) {
  return chunk<GRP>(1, 0) == 1 ? r & 15 : (r & 10) | ((r & 1) << 2) | ((r >> 2) & 1);
}

template <class C, int GRP, bool SB, bool OUTB>
__global__ __launch_bounds__(C::THREADS, 2) void kg_fprop_w4_kernel(WParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int TT = C::TT, NI = C::NI;
  int* off = (int*)(smem + 2 * C::STAGE);  // [G + 1]
  int* boff = off + p.G + 1;
  if (!f_offsets<C::THREADS>(p.ms, p.G, C::BT, p.M_total, off, boff)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = KG_ERR_KSUM;
    return;
  }
  const int mt_total = boff[p.G], total = mt_total * p.tiles_n;
  const int grid = gridDim.x, b = blockIdx.x;
  // XCD-contiguous runs when the items take several rounds, as in kg_fprop
  const int slot = (grid % 8 == 0 && total > grid) ? (b % 8) * (grid / 8) + b / 8 : b;
  const int nk = (p.K + 127) / 128, kbytes = p.K / 2;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, j = lane & 15;
  const int wt = w % C::WT, wn = w / C::WT;
  const uint32_t lds = lds_addr(smem);
  for (int base = 0; base < total; base += grid) {
    const int idx = base + slot;
    if (idx >= total) break;
    const int per_panel = kPanelM * p.tiles_n;
    const int panel = idx / per_panel, wi = idx - panel * per_panel;
    const int pm = min(kPanelM, mt_total - panel * kPanelM);
    const int mtg = panel * kPanelM + wi % pm, nt = wi / pm;
    int lo_g = 0, hi_g = p.G;  // expert of m-tile mtg: the last g with boff[g] <= mtg
    while (hi_g - lo_g > 1) {
      const int mid = (lo_g + hi_g) >> 1;
      if (boff[mid] <= mtg) lo_g = mid; else hi_g = mid;
    }
    const int g = uniform(lo_g);
    const int row0 = uniform(off[g] + (mtg - boff[g]) * C::BT);
    const int rows = uniform(min(C::BT, off[g + 1] - row0));
    const int n0 = nt * C::BN + wn * NI * 16;  // this wave's outputs
    const int outs = uniform(max(0, min(NI * 16, p.N - n0)));
    const int64_t out0 = (int64_t)g * p.N + (outs ? n0 : 0);
    const __amdgpu_buffer_rsrc_t wr = rsrc_of(p.W + out0 * kbytes, (uint32_t)(outs * kbytes));
    uint32_t woff[NI];
    int64_t sat[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      woff[i] = (uint32_t)((NI * j + i) * kbytes + 16 * q);
      sat[i] = (out0 + min(NI * j + i, max(outs, 1) - 1)) * (p.K / (GRP == kE2M1 ? 32 : GRP));
    }
    // tokens: wave w's load x takes rows 4 (w + 8 x) .. + 3
    const unsigned char* A = p.A + (int64_t)row0 * p.lda * 2;
    const int lda2 = (int)(2 * p.lda);
    auto load_tokens = [&](int kb) {
      const int left = min(256, 2 * p.K - kb * 256);
      const v4i r = make_rsrc(A + (int64_t)kb * 256, (uint32_t)((rows - 1) * lda2 + left));
#pragma unroll
      for (int x = 0; x < C::LOADS; ++x) {
        if (C::BT % 32 != 0 && w + 8 * x >= C::BT / 4) continue;
        const int row = 4 * (w + 8 * x) + q, c = 16 * ((lane & 15) ^ key_of<GRP>(row & 15));
        load16_lds(r, lds + (kb & 1) * C::STAGE + 1024 * (w + 8 * x),
                   c < left ? (uint32_t)(row * lda2 + c) : kOobOffset);
      }
    };
    v4i wx[NI];
    Scales<GRP> sn[NI];
    auto load_codes = [&](int kb) {
      const int left = (p.K - kb * 128) / (GRP == kE2M1 ? 32 : GRP);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        wx[i] = load16(wr, woff[i] + (uint32_t)kb * 64);
        if (GRP == 128 || kb * 128 + 128 <= p.K) sn[i] = load_scales<GRP, SB, false>(p, sat[i], kb, q, 4);
        else sn[i] = load_scales<GRP, SB, true>(p, sat[i], kb, q, left);
      }
    };
    v4f acc[TT][NI];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[tt][i] = v4f{0.f, 0.f, 0.f, 0.f};
    const int key = key_of<GRP>(j);
    const unsigned char* frag = smem + (wt * TT * 16 + j) * 256;
    if (nk > 0) {
      load_tokens(0);
      load_codes(0);
    }
    for (int kb = 0; kb < nk; ++kb) {
      v8bf wf[NI][4];
      Scales<GRP> sc[NI];
      // this block's tokens are there, the last block's have been read by every wave
      wait_all_and_barrier();
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        sc[i] = sn[i];
        deal<GRP>(wx[i]);
#pragma unroll
        for (int c = 0; c < 4; ++c) wf[i][c] = eight_codes<GRP>((uint32_t)wx[i][c], sc[i].s[0]);
      }
      if (kb + 1 < nk) {
        load_tokens(kb + 1);
        load_codes(kb + 1);
      }
      const unsigned char* st = frag + (kb & 1) * C::STAGE;
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        v8bf t[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          t[c] = *(const v8bf*)(st + tt * 16 * 256 + 16 * (chunk<GRP>(q, c) ^ key));
        add_block<GRP, NI>(wf, sc, t, acc[tt]);
      }
    }
#pragma unroll
    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = (wt * TT + tt) * 16 + 4 * q + r;
        if (row >= rows) continue;
        float x[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) x[i] = acc[tt][i][r];
        store_outputs<OUTB, NI>(p.D, (int64_t)(row0 + row) * p.ldd + n0 + NI * j, outs - NI * j, x);
      }
    __syncthreads();  // every wave has read the last stage
  }
}

struct WLaunch {
  const void* fn;
  int bt, bn, lds, id;  // id < 0: streaming
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
template <int TT, int NJ>
struct StreamOf {
  template <int GRP, bool SB, bool OUTB>
  struct F {
    static const void* fn() { return (const void*)kg_fprop_w4_stream_kernel<GRP, SB, TT, NJ, OUTB>; }
  };
};
template <class C>
struct TiledOf {
  template <int GRP, bool SB, bool OUTB>
  struct F {
    static const void* fn() { return (const void*)kg_fprop_w4_kernel<C, GRP, SB, OUTB>; }
  };
};
template <int TT, int NJ>
static WLaunch w_stream(int kind, int group, bool outb) {
  return WLaunch{w_pick<StreamOf<TT, NJ>::template F>(kind, group, outb), 16 * TT, 16 * NJ, 0, -1};
}
template <class C>
static WLaunch w_tiled(int kind, int group, bool outb, int id) {
  return WLaunch{w_pick<TiledOf<C>::template F>(kind, group, outb), C::BT, C::BN, 2 * C::STAGE, id};
}

// Which kernel and tile, by M_total and G (the experts' sizes are known on the device only); every
// choice is right for every distribution of the rows.
static WLaunch w_choose(int64_t M, int G, int N, int cus, int kind, int group, bool outb) {
  const int64_t avg = (M + G - 1) / G, live = G < M ? G : M;
  if (avg <= 16) {
    if (live * ((N + 31) / 32) <= cus / 2) return w_stream<1, 1>(kind, group, outb);
    return w_stream<1, 2>(kind, group, outb);
  }
  if (avg <= 64) return w_tiled<WCfg<64, 256, 1>>(kind, group, outb, 0);
  return w_tiled<WCfg<128, 256, 2>>(kind, group, outb, 1);
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
  p.sw = sw;
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
  WLaunch l = w_choose(M_total, G, N, cus, kind, group, outb);
  p.tiles_n = (N + l.bn - 1) / l.bn;
  int64_t grid;
  if (l.id < 0) {
    grid = (int64_t)(G < M_total ? G : M_total) * p.tiles_n;
    if (grid > INT32_MAX / 512) return KG_ERR_UNSUPPORTED;
  } else {
    l.lds += 2 * (G + 1) * 4;
    static std::mutex mu;
    static const void* set[64][64];  // kernels that may have the largest LDS size
    static int count[64];
    {
      std::lock_guard<std::mutex> lk(mu);
      bool found = false;
      for (int i = 0; i < count[dev]; ++i) found |= set[dev][i] == l.fn;
      if (!found) {
        if (hipFuncSetAttribute(l.fn, hipFuncAttributeMaxDynamicSharedMemorySize,
                                l.lds - 2 * (G + 1) * 4 + 2 * (kMaxGroups + 1) * 4) != hipSuccess)
          return KG_ERR_HIP;
        if (count[dev] < 64) set[dev][count[dev]++] = l.fn;
      }
    }
    const int64_t max_items = (M_total / l.bt + G) * (int64_t)p.tiles_n;
    if (max_items > INT32_MAX - 4096) return KG_ERR_UNSUPPORTED;  // (indexes pass it by a grid)
    grid = max_items < cus ? max_items : cus;
  }
  void* args[] = {&p};
  return hipLaunchKernel(l.fn, dim3((unsigned)grid), dim3(512), args, (size_t)l.lds,
                         (hipStream_t)stream) == hipSuccess
             ? KG_OK
             : KG_ERR_HIP;
}
