// kg_fprop.hip -- the forward product of expert rows on gfx950, C ABI kg_fprop.
//
// y = x w^T per expert, the product whose two gradients kg_dgrad and kg_wgrad compute.
// Expert g owns the contiguous rows [off[g], off[g+1]) of A; for such a row t and output n
//
//   D[t][n] = sum over 128-channel blocks kb of sa[kb][t] * sw[g][n/128][kb] *
//             sum_{k in kb} A[t][k] * W[g][n][k]
//
// with A [M_total, K] e4m3 (row stride lda), sa [ceil(K/128), M_total] fp32, W [G, N, K]
// e4m3 (the tensor that kg_dgrad reads as [G, K, N]), sw [G, ceil(N/128), ceil(K/128)] fp32.
// A block's partial sum is formed exactly (bf16 MFMA on widened fp8 values, whose products
// are exact, summed in fp32) or by the fp8 MFMA (KG_FLAG_FP8_MFMA), multiplied by its two
// scales and added in fp32; the result is rounded once, to fp32 or bf16.
//
// Both operands have the contraction axis contiguous, so a lane's MFMA operand is two
// 16-byte runs of one row; which runs is free as long as both operands agree (the sum runs
// over all 128 channels of a block). W's rows are the MFMA's rows and tokens its columns:
// a lane then holds one token, whose scale it multiplies into the weight block's once per
// block, and by the order in which W's rows are dealt to the MFMA's rows it holds runs of
// eight neighbouring outputs of that token, so the results go from registers to memory in
// 16-byte stores without a trip through LDS.
//
// Two kernels. The tiled kernel (many rows per expert) stages both operands in LDS; the
// streaming kernel (few rows) reads W from memory straight into registers, split over
// the contraction axis among a workgroup's waves, since W is then read for so few rows
// that its bytes alone set the time.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "kg_device.h"
#include "kg_host.h"
#include "kg_sched.h"
#include "kgwgrad.h"

namespace kg {

struct FParams {
  const unsigned char* A;  // [M_total, K] e4m3fn, row stride lda
  const float* sa;         // [ceil(K/128), M_total]
  const unsigned char* W;  // [G, N, K] e4m3fn
  const float* sw;         // [G, ceil(N/128), ceil(K/128)]
  void* D;                 // [M_total, N] fp32 or bf16, row stride ldd
  const int32_t* ms;       // [G]
  int* status;
  int64_t M_total, lda, ldd;
  int G, N, K;
  int tiles_n;
  int vec;  // D's rows start at 16-byte boundaries
};

// Row m (0 .. 15) of MFMA row tile i holds output row frow(i, m) of the wave's: pairs of
// tiles cover 32 outputs such that result lanes (which hold rows 4q .. 4q+3 of both tiles)
// have outputs 8q .. 8q+7 of them.
__device__ __forceinline__ constexpr int frow(int i, int m) {
  return 32 * (i >> 1) + 8 * (m >> 2) + 4 * (i & 1) + (m & 3);
}

// 8 fp8 values as bf16 (exact).
__device__ __forceinline__ v8bf fwiden(int lo, int hi) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, 1.0f, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)lo, 1.0f, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, 1.0f, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)hi, 1.0f, true);
  return v8bf{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// A lane's 32 operand bytes of one block, as the MFMA of the mode reads them.
template <bool FAST>
struct Frag;
template <>
struct Frag<true> {
  v8i x;
  __device__ __forceinline__ void set(const v4i& lo, const v4i& hi) {
    x = v8i{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  }
};
template <>
struct Frag<false> {
  v8bf x[4];
  __device__ __forceinline__ void set(const v4i& lo, const v4i& hi) {
    x[0] = fwiden(lo.x, lo.y);
    x[1] = fwiden(lo.z, lo.w);
    x[2] = fwiden(hi.x, hi.y);
    x[3] = fwiden(hi.z, hi.w);
  }
};

// The partial sum of one block: 16 outputs x 16 tokens over 128 channels.
__device__ __forceinline__ v4f block_sum(const Frag<true>& w, const Frag<true>& t) {
  return mfma_fp8(w.x, t.x, v4f{0.f, 0.f, 0.f, 0.f});
}
__device__ __forceinline__ v4f block_sum(const Frag<false>& w, const Frag<false>& t) {
  v4f s = mfma_bf16(w.x[0], t.x[0], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
  for (int k = 1; k < 4; ++k) s = mfma_bf16(w.x[k], t.x[k], s);
  return s;
}

// Stores eight outputs [n, n + 8) of one token; `left` = N - n of them exist.
template <bool OUTB>
__device__ __forceinline__ void store_run(void* D, int64_t at, int left, bool vec, const v4f& a,
                                          const v4f& b) {
  if constexpr (OUTB) {
    unsigned short* d = (unsigned short*)D + at;
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    v8bf h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (__bf16)x[i];  // to nearest, ties to even
    if (vec && left >= 8) {
      *(v4i*)d = __builtin_bit_cast(v4i, h);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) d[i] = __builtin_bit_cast(unsigned short, (__bf16)x[i]);
    }
  } else {
    float* d = (float*)D + at;
    if (vec && left >= 8) {
      *(v4f*)d = a;
      *(v4f*)(d + 4) = b;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) d[i] = a[i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 + i < left) d[4 + i] = b[i];
    }
  }
}

// ---------------------------------------------------------------------------- tiled kernel

// BT tokens x BN outputs per workgroup of 8 waves (WT along the tokens); stages of one
// 128-channel block: BN rows of W, BT rows of A, the BT token scales.
template <int BT_, int BN_, int WT_>
struct FCfg {
  static constexpr int BT = BT_, BN = BN_, WT = WT_, WN = 8 / WT_, THREADS = 512, TK = 128;
  static constexpr int TT = BT / WT / 16;  // 16-token tiles of a wave
  static constexpr int NI = BN / WN / 16;  // 16-output tiles of a wave
  static constexpr int NS = 2;
  static constexpr int OPW = BN * TK, OPT = BT * TK;
  static constexpr int SA_OFF = OPW + OPT;
  static constexpr int SA_BYTES = (BT * 4 + 1023) / 1024 * 1024;
  static constexpr int STAGE = SA_OFF + SA_BYTES;
  static constexpr int LOADS_W = BN / 8, LOADS_T = BT / 8;  // 1 KB wave loads: 8 rows each
  static constexpr int LOADS = LOADS_W + LOADS_T + SA_BYTES / 1024;
  static constexpr int SLOTS = (LOADS + 7) / 8;
  static_assert(NI % 2 == 0 && BN / WN <= 128 && 128 % (BN / WN) == 0,
                "a wave's outputs lie in one weight-scale block");
};

// Row r's 16-byte chunk c lies in slot c ^ fkey(r) of the row's 128 bytes. The 16-byte LDS
// reads go 32 lanes at a time and are free of conflicts when their chunks are distinct
// modulo 512 bytes: the 16 rows that two lane groups name (16 neighbouring ones for
// tokens, frow's for W) share r mod 4 four at a time, and those four have distinct keys.
__device__ __forceinline__ constexpr int fkey(int r) {
  const int y = (r >> 2) & 7;
  return 2 * ((y & 3) ^ (y >> 2));
}

template <class C>
__device__ __forceinline__ void f_load_stage(const FParams& p, unsigned char* st, int64_t row0,
                                             int rows, int g, int n0, int kb) {
  const int w = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int k0 = kb * C::TK;
  const int kin = min(C::TK, p.K - k0);       // channels of this block that exist
  const int outs = min(C::BN, p.N - n0);      // outputs of this tile that exist
  const v4i rw = make_rsrc(p.W + ((int64_t)g * p.N + n0) * p.K + k0,
                           (uint32_t)((outs - 1) * p.K + kin));
  const v4i rt = make_rsrc(p.A + row0 * p.lda + k0, (uint32_t)((rows - 1) * (int)p.lda + kin));
  const v4i rs = make_rsrc(p.sa + (int64_t)kb * p.M_total + row0, (uint32_t)(rows * 4));
  const uint32_t base = lds_addr(st);
#pragma unroll
  for (int s = 0; s < C::SLOTS; ++s) {
    const int k = w + 8 * s;
    if (k >= C::LOADS) break;
    const uint32_t to = base + 1024 * k;
    if (k < C::LOADS_W + C::LOADS_T) {
      const bool is_w = k < C::LOADS_W;
      const int r = 8 * (is_w ? k : k - C::LOADS_W) + (lane >> 3);
      const int ch = (lane & 7) ^ fkey(r);
      const uint32_t off = 16 * ch < kin ? (uint32_t)(r * (is_w ? p.K : (int)p.lda) + 16 * ch)
                                         : kOobOffset;
      load16_lds(is_w ? rw : rt, to, off);
    } else {
      load16_lds(rs, to, 1024 * (k - C::LOADS_W - C::LOADS_T) + 16 * lane);
    }
  }
}

template <class C, bool FAST>
__device__ __forceinline__ void f_compute(const unsigned char* st, float swv,
                                          v4f (&acc)[C::NI][C::TT]) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int q = lane >> 4, j = lane & 15;
  const int wt = w % C::WT, wn = w / C::WT;
  const int t0 = wt * C::TT * 16, n0 = wn * C::NI * 16;
  const float* sS = (const float*)(st + C::SA_OFF);
  auto frag = [&](int off, int r) {
    const unsigned char* row = st + off + r * C::TK;
    const int key = fkey(r);
    Frag<FAST> f;
    f.set(*(const v4i*)(row + 16 * (q ^ key)), *(const v4i*)(row + 16 * ((q + 4) ^ key)));
    return f;
  };
  Frag<FAST> tf[C::TT];
  float s[C::TT];
#pragma unroll
  for (int tt = 0; tt < C::TT; ++tt) {
    tf[tt] = frag(C::OPW, t0 + 16 * tt + j);
    s[tt] = sS[t0 + 16 * tt + j] * swv;
  }
#pragma unroll
  for (int i = 0; i < C::NI; ++i) {
    const Frag<FAST> wf = frag(0, n0 + frow(i, j));
    v4f part[C::TT];
#pragma unroll
    for (int tt = 0; tt < C::TT; ++tt) part[tt] = block_sum(wf, tf[tt]);
#pragma unroll
    for (int tt = 0; tt < C::TT; ++tt)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][tt][r] = fmaf(s[tt], part[tt][r], acc[i][tt][r]);
  }
}

template <class C, bool FAST, bool OUTB>
__global__ __launch_bounds__(C::THREADS, 1) void kg_fprop_kernel(FParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ int64_t wsum_k[kMaxWaves];
  __shared__ int32_t wsum_b[kMaxWaves];
  Sched s = sched_carve(smem + C::NS * C::STAGE, p.G);
  if (sched_build<C::THREADS>(p.ms, p.G, C::BT, p.M_total, s, wsum_k, wsum_b) != KG_OK) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = KG_ERR_KSUM;
    return;
  }
  const int mt_total = s.boff[p.G], total = mt_total * p.tiles_n;
  const int grid = gridDim.x, b = blockIdx.x;
  const int slot = (grid % 8 == 0 && total > grid) ? (b % 8) * (grid / 8) + b / 8 : b;
  const int nk = (p.K + C::TK - 1) / C::TK, nsc = (p.N + 127) / 128;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int q = lane >> 4, j = lane & 15;
  const int wt = w % C::WT, wn = w / C::WT;
  for (int base = 0; base < total; base += grid) {
    const int idx = base + slot;
    if (idx >= total) break;
    // panels of kPanelM m-tiles, m-tiles fastest, as in kg_dgrad
    const int per_panel = kPanelM * p.tiles_n;
    const int panel = idx / per_panel, wi = idx - panel * per_panel;
    const int pm = min(kPanelM, mt_total - panel * kPanelM);
    const int mtg = panel * kPanelM + wi % pm, nt = wi / pm;
    int lo_g = 0, hi_g = p.G;  // expert of m-tile mtg: the last g with boff[g] <= mtg
    while (hi_g - lo_g > 1) {
      const int mid = (lo_g + hi_g) >> 1;
      if (s.boff[mid] <= mtg) lo_g = mid; else hi_g = mid;
    }
    const int g = uniform(lo_g);
    const int64_t row0 = s.off[g] + (int64_t)(mtg - s.boff[g]) * C::BT;
    const int rows = uniform((int)min((int64_t)C::BT, s.off[g + 1] - row0));
    const int n0 = nt * C::BN;
    const int nw = n0 + wn * C::NI * 16;  // this wave's outputs, one weight-scale block
    const float* swg = p.sw + ((int64_t)g * nsc + min(nw / 128, nsc - 1)) * nk;
    v4f acc[C::NI][C::TT];
#pragma unroll
    for (int i = 0; i < C::NI; ++i)
#pragma unroll
      for (int tt = 0; tt < C::TT; ++tt) acc[i][tt] = v4f{0.f, 0.f, 0.f, 0.f};
    __syncthreads();  // every wave is done with the previous item's stages
    if (nk > 0) f_load_stage<C>(p, smem, row0, rows, g, n0, 0);
    for (int kb = 0; kb < nk; ++kb) {
      // stage kb is in buffer kb % 2; stage kb + 1 loads into the other one meanwhile
      __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      __syncthreads();
      if (kb + 1 < nk)
        f_load_stage<C>(p, smem + ((kb + 1) & 1) * C::STAGE, row0, rows, g, n0, kb + 1);
      f_compute<C, FAST>(smem + (kb & 1) * C::STAGE, swg[kb], acc);
    }
#pragma unroll
    for (int tt = 0; tt < C::TT; ++tt) {
      const int r = (wt * C::TT + tt) * 16 + j;
      if (r >= rows) continue;
      const int64_t at = (row0 + r) * p.ldd;
#pragma unroll
      for (int i = 0; i < C::NI; i += 2) {
        const int n = nw + 16 * i + 8 * q;
        store_run<OUTB>(p.D, at + n, p.N - n, p.vec, acc[i][tt], acc[i + 1][tt]);
      }
    }
  }
}

// ------------------------------------------------------------------------ streaming kernel

// A workgroup computes 32 outputs of one expert for all its rows, 16 TT at a time. Its 8
// waves take the blocks of the contraction axis in turn, each adding up its blocks in
// registers; the waves' sums are added in LDS in a fixed order. Grid: G x ceil(N / 32).
constexpr int kStreamWaves = 8, kStreamN = 32;

// Offsets by a scan of ms in every wave. Returns false if ms is inconsistent.
__device__ __forceinline__ bool find_rows(const FParams& p, int g, int64_t* row0, int* rows) {
  const int lane = threadIdx.x & 63;
  int64_t sum = 0, before = 0;
  int mine = 0, neg = 0;
  for (int i = lane; i < p.G; i += 64) {
    const int v = p.ms[i];
    neg |= v < 0;
    sum += v;
    if (i < g) before += v;
    if (i == g) mine = v;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    sum += __shfl_xor(sum, d, 64);
    before += __shfl_xor(before, d, 64);
    mine += __shfl_xor(mine, d, 64);
    neg |= __shfl_xor(neg, d, 64);
  }
  *row0 = before;
  *rows = uniform(mine);
  return neg == 0 && sum == p.M_total;
}

// 16 bytes at p + off, zeros if they lie past `limit`.
__device__ __forceinline__ v4i load_in(const unsigned char* p, int off, int limit) {
  v4i x = {0, 0, 0, 0};
  if (off < limit) x = *(const v4i*)(p + off);
  return x;
}

template <int TT, bool FAST, bool OUTB>
__global__ __launch_bounds__(64 * kStreamWaves) void kg_fprop_stream_kernel(FParams p) {
  __shared__ v4f sums[kStreamWaves][2 * TT][64];
  const int per = p.tiles_n;  // workgroups per expert
  const int g = blockIdx.x / per, n0 = (blockIdx.x - g * per) * kStreamN;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int q = lane >> 4, j = lane & 15;
  int64_t row0;
  int rows;
  if (!find_rows(p, g, &row0, &rows)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = KG_ERR_KSUM;
    return;
  }
  const int nk = (p.K + 127) / 128, nsc = (p.N + 127) / 128;
  const float* swg = p.sw + ((int64_t)g * nsc + n0 / 128) * nk;
  const unsigned char* wrow[2];
  bool won[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int n = n0 + frow(i, j);
    won[i] = n < p.N;
    wrow[i] = p.W + ((int64_t)g * p.N + (won[i] ? n : 0)) * p.K;
  }
  for (int r0 = 0; r0 < rows; r0 += 16 * TT) {
    const unsigned char* arow[TT];
    bool aon[TT];
    const float* sa[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int r = r0 + 16 * tt + j;
      aon[tt] = r < rows;
      arow[tt] = p.A + (row0 + (aon[tt] ? r : 0)) * p.lda;
      sa[tt] = p.sa + row0 + (aon[tt] ? r : 0);
    }
    v4f acc[2][TT];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[i][tt] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int kb = w; kb < nk; kb += kStreamWaves) {
      const int k0 = kb * 128 + 32 * q;  // a lane's 32 channels are neighbours
      Frag<FAST> wf[2], tf[TT];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int lim = won[i] ? p.K : 0;
        wf[i].set(load_in(wrow[i], k0, lim), load_in(wrow[i], k0 + 16, lim));
      }
      const float swv = swg[kb];
      float s[TT];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        const int lim = aon[tt] ? p.K : 0;
        tf[tt].set(load_in(arow[tt], k0, lim), load_in(arow[tt], k0 + 16, lim));
        s[tt] = sa[tt][(int64_t)kb * p.M_total] * swv;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const v4f part = block_sum(wf[i], tf[tt]);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][tt][r] = fmaf(s[tt], part[r], acc[i][tt][r]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) sums[w][i * TT + tt][lane] = acc[i][tt];
    __syncthreads();
    if (w < TT) {  // wave w joins and stores token tile w
      v4f x[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x[i] = sums[0][i * TT + w][lane];
#pragma unroll
        for (int v = 1; v < kStreamWaves; ++v) {
          const v4f y = sums[v][i * TT + w][lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) x[i][r] += y[r];
        }
      }
      const int r = r0 + 16 * w + j, n = n0 + 8 * q;
      if (r < rows) store_run<OUTB>(p.D, (row0 + r) * p.ldd + n, p.N - n, p.vec, x[0], x[1]);
    }
    __syncthreads();
  }
}

struct FLaunch {
  const void* fn;
  int bt, bn, lds, id;
};

template <class C>
static FLaunch f_tiled(bool fast, bool outb, int id) {
  const void* fn = fast ? (outb ? (const void*)kg_fprop_kernel<C, true, true>
                                : (const void*)kg_fprop_kernel<C, true, false>)
                        : (outb ? (const void*)kg_fprop_kernel<C, false, true>
                                : (const void*)kg_fprop_kernel<C, false, false>);
  return FLaunch{fn, C::BT, C::BN, C::NS * C::STAGE, id};
}

template <int TT>
static FLaunch f_stream(bool fast, bool outb) {
  const void* fn = fast ? (outb ? (const void*)kg_fprop_stream_kernel<TT, true, true>
                                : (const void*)kg_fprop_stream_kernel<TT, true, false>)
                        : (outb ? (const void*)kg_fprop_stream_kernel<TT, false, true>
                                : (const void*)kg_fprop_stream_kernel<TT, false, false>);
  return FLaunch{fn, 16 * TT, kStreamN, 0, -1};
}

}  // namespace kg

extern "C" int kg_fprop(const void* A, int64_t lda, const float* sa, const void* W, const float* sw,
                        void* D, int64_t ldd, const int32_t* ms, int G, int N, int K,
                        int64_t M_total, int flags, void* stream) {
  using namespace kg;
  if (flags & ~(KG_FLAG_FP8_MFMA | KG_FLAG_D_BF16)) return KG_ERR_DTYPE;
  const bool fast = (flags & KG_FLAG_FP8_MFMA) != 0, outb = (flags & KG_FLAG_D_BF16) != 0;
  if (G < 0 || N < 0 || K < 0 || M_total < 0 || lda < K || ldd < N) return KG_ERR_SHAPE;
  if (G > kMaxGroups || N > (1 << 24) || K > (1 << 23) || M_total > INT32_MAX ||
      lda > (1 << 23) || ldd > (1 << 30))
    return KG_ERR_UNSUPPORTED;
  if (K % 16 != 0 || lda % 16 != 0) return KG_ERR_ALIGN;
  if (G == 0 || N == 0 || M_total == 0) return KG_OK;
  if (D == nullptr || ms == nullptr) return KG_ERR_NULL;
  if (K > 0 && (A == nullptr || sa == nullptr || W == nullptr || sw == nullptr))
    return KG_ERR_NULL;
  const int el = outb ? 2 : 4;
  if (((uintptr_t)A & 15) || ((uintptr_t)W & 15) || ((uintptr_t)sa & 3) || ((uintptr_t)sw & 3) ||
      ((uintptr_t)D & (el - 1)) || ((uintptr_t)ms & 3))
    return KG_ERR_ALIGN;
  const int64_t nk = (K + 127) / 128, nsc = (N + 127) / 128;
  const size_t dbytes = ((size_t)(M_total - 1) * ldd + N) * el;
  if (ranges_overlap(A, (size_t)(M_total - 1) * lda + K, D, dbytes) ||
      ranges_overlap(W, (size_t)G * N * K, D, dbytes) ||
      ranges_overlap(sa, (size_t)nk * M_total * 4, D, dbytes) ||
      ranges_overlap(sw, (size_t)G * nsc * nk * 4, D, dbytes) ||
      ranges_overlap(ms, (size_t)G * 4, D, dbytes))
    return KG_ERR_ALIAS;
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return KG_ERR_HIP;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return KG_ERR_HIP;
  FParams p;
  p.A = (const unsigned char*)A;
  p.sa = sa;
  p.W = (const unsigned char*)W;
  p.sw = sw;
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
  p.vec = ((uintptr_t)D & 15) == 0 && ldd * el % 16 == 0;
  const int64_t avg = (M_total + G - 1) / G;
  const bool stream_w = avg <= 64;
  FLaunch l;
  int64_t grid;
  if (stream_w) {
    l = avg <= 16 ? f_stream<1>(fast, outb) : avg <= 32 ? f_stream<2>(fast, outb)
                                                        : f_stream<4>(fast, outb);
    p.tiles_n = (N + l.bn - 1) / l.bn;
    grid = (int64_t)G * p.tiles_n;
    if (grid > INT32_MAX) return KG_ERR_UNSUPPORTED;
  } else {
    if (fast)
      l = f_tiled<FCfg<256, 256, 4>>(fast, outb, 0);
    else
      l = f_tiled<FCfg<256, 128, 4>>(fast, outb, 1);
    l.lds += sched_bytes(G);
    static std::mutex mu;
    static int set[64][2][2];  // the largest LDS size asked for so far
    std::lock_guard<std::mutex> lk(mu);
    if (set[dev][l.id][outb] < l.lds) {
      if (hipFuncSetAttribute(l.fn, hipFuncAttributeMaxDynamicSharedMemorySize, l.lds) !=
          hipSuccess)
        return KG_ERR_HIP;
      set[dev][l.id][outb] = l.lds;
    }
    p.tiles_n = (N + l.bn - 1) / l.bn;
    const int64_t max_items = (M_total / l.bt + G) * (int64_t)p.tiles_n;
    if (max_items > INT32_MAX) return KG_ERR_UNSUPPORTED;
    grid = max_items < cus ? max_items : cus;
  }
  void* args[] = {&p};
  return hipLaunchKernel(l.fn, dim3((unsigned)grid), dim3(512), args, (size_t)l.lds,
                         (hipStream_t)stream) == hipSuccess
             ? KG_OK
             : KG_ERR_HIP;
}
