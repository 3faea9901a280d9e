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

// Stores eight outputs [n, n + 8) of one token; `left` = N - n of them exist. Rows of D may start
// at any element: gfx950 takes 16-byte stores at any address.
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));
template <bool OUTB>
__device__ __forceinline__ void store_run(void* D, int64_t at, int left, const v4f& a,
                                          const v4f& b) {
  if constexpr (OUTB) {
    unsigned short* d = (unsigned short*)D + at;
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (left >= 8) {
      v8bf h;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (__bf16)x[i];  // to nearest, ties to even
      *(v4i_any*)d = __builtin_bit_cast(v4i, h);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) d[i] = __builtin_bit_cast(unsigned short, (__bf16)x[i]);
    }
  } else {
    float* d = (float*)D + at;
    if (left >= 8) {
      *(v4f_any*)d = a;
      *(v4f_any*)(d + 4) = b;
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

// ... and four.
template <bool OUTB>
__device__ __forceinline__ void store_four(void* D, int64_t at, int left, const v4f& a) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= left) continue;
    if constexpr (OUTB)
      ((unsigned short*)D)[at + i] = __builtin_bit_cast(unsigned short, (__bf16)(float)a[i]);
    else
      ((float*)D)[at + i] = a[i];
  }
}

// ---------------------------------------------------------------------------- tiled kernel

// BT tokens x BN outputs per workgroup of 8 waves (WT along the tokens, PER_CU such
// workgroups per compute unit), two stages of one
// 128-channel block in LDS: BN rows of W, BT rows of A, the BT token scales.
// With ROTATE each tile begins at a block of its own and goes round: tiles that run side by side
// would else all read the same channels of W's rows, and where the rows lie a multiple of 4096
// bytes apart those are in few of the memory channels. (32 experts, 8 rows each, N 4096, K 4096:
// 155 -> 93 us; 64 experts of 4 rows, N 1024, K 4096: 62 -> 46.) It is for such rows only: else
// nothing is gained (K 3584 and 7168 within 1%), and where latency counts the extra
// instructions cost (256 tokens of one expert, K 7168: 26.4 -> 28.9 us), and for few tokens:
// tiles of other outputs no longer read the tokens' blocks at the same time.
template <int BT_, int BN_, int WT_, int PER_CU_, bool ROTATE_ = false>
struct FCfg {
  static constexpr int PER_CU = PER_CU_;  // workgroups per compute unit
  static constexpr bool ROTATE = ROTATE_;
  static constexpr int BT = BT_, BN = BN_, WT = WT_, WN = 8 / WT_, THREADS = 512, TK = 128;
  static constexpr int TT = BT / WT / 16;  // 16-token tiles of a wave
  static constexpr int NI = BN / WN / 16;  // 16-output tiles of a wave
  // A block's partial sums of a wave, and how many MFMAs after its own each is scaled and added
  // (a whole block's where it has fewer than three).
  static constexpr int SUMS = NI * TT, LAG = SUMS < 3 ? SUMS : 3;
  static constexpr int NS = 2;
  static constexpr int OPW = BN * TK, OPT = BT * TK;
  static constexpr int SA_OFF = OPW + OPT;
  static constexpr int STAGE = SA_OFF + BT * 4;
  static constexpr int LW = BN / 64, LT = BT / 64;  // a wave's 1 KB loads of W and of A
  static constexpr int LOADS = LW + LT + 1;         // ... and one of token scales
  static_assert(NI % 2 == 0 && BN / WN <= 128 && 128 % (BN / WN) == 0,
                "a wave's outputs lie in one weight-scale block");
  static_assert(BT <= 512 && BT % 64 == 0 && BN % 64 == 0, "whole wave loads");
};

// LDS layout: a row's 128 channel bytes in order, but its 16-byte chunk c in slot c ^ key.
// A 16-byte LDS read serves 16 lanes at a time (lanes 0-3, 12-15, 20-27, then the other 16 of
// the lower half; the upper half alike), without conflicts if their chunks are distinct
// modulo 256 bytes. With key = m & 7 for the row that MFMA row (or column) m reads they are:
// tokens lie in that order, W's rows in frow's. (Measured: 0 conflict cycles, where keys
// chosen for 32 lanes and 512 bytes cost one per access.)
__device__ __forceinline__ constexpr int key_t(int r) { return r & 7; }
__device__ __forceinline__ constexpr int key_w(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }

// 4 bytes per lane global -> LDS at `lds` + 4 * lane (see load16_lds).
__device__ __forceinline__ void load4_lds(v4i r, uint32_t lds, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(r), "s"(__builtin_amdgcn_readfirstlane((int)lds))
               : "memory", "m0");
}

// This wave's loads of one tile. Load x of an operand takes its rows 8 (wave + 8 x) ..
// 8 (wave + 8 x) + 7. Rows that the tile lacks, channels past K, and stages past the last
// block read as zeros; every stage is LOADS loads of each wave, so waits can count them.
template <class C>
struct FLoads {
  const unsigned char *W, *A;
  const float* sa;
  int64_t M_total;
  int K, lda, nk, outs, rows, wave;
  int first;  // the block that the tile begins with
  uint32_t offw, offt, offs, lds;
  bool endw, endt;  // this lane's chunk lies past the last block's channels
  __device__ __forceinline__ void setup(const FParams& p, const unsigned char* smem, int64_t row0,
                                        int rows_, int g, int n0, int nk_, int first_) {
    wave = uniform(threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    W = p.W + ((int64_t)g * p.N + n0) * p.K;
    A = p.A + row0 * p.lda;
    sa = p.sa + row0;
    M_total = p.M_total;
    K = p.K, lda = (int)p.lda, nk = nk_, first = first_;
    outs = min(C::BN, p.N - n0), rows = rows_;
    const int r = 8 * wave + (lane >> 3);
    const int cw = (lane & 7) ^ key_w(r), ct = (lane & 7) ^ key_t(r);
    offw = (uint32_t)(r * K + 16 * cw);
    offt = (uint32_t)(r * lda + 16 * ct);
    const int last = K - (nk - 1) * C::TK;
    endw = 16 * cw >= last;
    endt = 16 * ct >= last;
    // the scales: 64 tokens per wave (with fewer than 512 tokens several waves load the same
    // ones to the same place)
    const int part = wave % (C::BT / 64);
    offs = 256 * part + 4 * lane;
    lds = lds_addr(smem);
  }
  __device__ __forceinline__ int channels(int kb) const { return min(C::TK, K - kb * C::TK); }
  // The block that the tile takes as its kb-th.
  __device__ __forceinline__ int block(int kb) const {
    if constexpr (!C::ROTATE) return kb;
    const int k = kb + first;
    return k >= nk ? k - nk : k;
  }
  __device__ __forceinline__ void load(int kw, int kt, int x) const {
    if (x < C::LW) {
      const int k = block(kw);
      const v4i r = make_rsrc(W + (int64_t)k * C::TK,
                              kw < nk ? (uint32_t)((outs - 1) * K + channels(k)) : 0u);
      load16_lds(r, lds + (kw & 1) * C::STAGE + 1024 * (wave + 8 * x),
                 (offw + (uint32_t)(64 * x * K)) | (k == nk - 1 && endw ? kOobOffset : 0u));
    } else if (x < C::LW + C::LT) {
      const int y = x - C::LW, k = block(kt);
      const v4i r = make_rsrc(A + (int64_t)k * C::TK,
                              kt < nk ? (uint32_t)((rows - 1) * lda + channels(k)) : 0u);
      load16_lds(r, lds + (kt & 1) * C::STAGE + C::OPW + 1024 * (wave + 8 * y),
                 (offt + (uint32_t)(64 * y * lda)) | (k == nk - 1 && endt ? kOobOffset : 0u));
    } else {
      const v4i r =
          make_rsrc(sa + (int64_t)block(kt) * M_total, kt < nk ? (uint32_t)(rows * 4) : 0u);
      load4_lds(r, lds + (kt & 1) * C::STAGE + C::SA_OFF + 256 * (wave % (C::BT / 64)), offs);
    }
  }
};

// Waits for all but N of this wave's vector-memory operations and for all its LDS reads, then
// for the workgroup's other waves.
template <int N>
__device__ __forceinline__ void f_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(N) & ~0xF00);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Weight scales through scalar loads: a vector load among the stages' would make the
// compiler wait for them.
typedef __attribute__((address_space(4))) const float ConstFloat;

// Exclusive scans over the experts, in LDS: off[g] rows and boff[g] tiles of `bt` rows before
// expert g, g = 0 .. G. Returns false if ms holds a negative count or does not add up to
// M_total. (kg_sched.h's scan also orders the experts by length, G^2 LDS reads, which a walk in
// expert order does not need.)
template <int THREADS>
__device__ __forceinline__ bool f_offsets(const int32_t* ms, int G, int bt, int64_t M_total,
                                          int* off, int* boff) {
  constexpr int E = kMaxGroups / THREADS, W = THREADS / 64;
  __shared__ int64_t rows_of[W];
  __shared__ int tiles_of[W];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  int kv[E], bv[E], neg = 0, own_b = 0;
  int64_t own = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int g = E * t + e;
    kv[e] = g < G ? ms[g] : 0;
    neg |= kv[e] < 0;
    bv[e] = kv[e] > 0 ? kv[e] / bt + (kv[e] % bt != 0) : 0;
    own += kv[e];
    own_b += bv[e];
  }
  const int64_t to = wave_incl_scan<int64_t>(own);
  const int to_b = wave_incl_scan<int>(own_b);
  if (lane == 63) {
    rows_of[w] = to;
    tiles_of[w] = to_b;
  }
  const int any_neg = __syncthreads_or(neg);
  int64_t total = 0, run = to - own;
  int run_b = to_b - own_b;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    total += rows_of[i];
    if (i < w) {
      run += rows_of[i];
      run_b += tiles_of[i];
    }
  }
  if (any_neg || total != M_total) return false;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int g = E * t + e;
    if (g <= G) {  // (G < kMaxGroups: else the last entry is the next line's)
      off[g] = (int)run;
      boff[g] = run_b;
    }
    run += kv[e];
    run_b += bv[e];
  }
  if (t == THREADS - 1 && G == kMaxGroups) {
    off[G] = (int)run;
    boff[G] = run_b;
  }
  __syncthreads();
  return true;
}

// The loop over the blocks. The token fragments are read one block ahead, each right after its
// last MFMA of the block before, so the buffer that block kb's tokens came from is free during
// block kb and their block kb + 2 loads into it. W's block kb has been read before the
// block's last tile of outputs, and its block kb + 2 loads into that buffer from there. So
// every load has a whole block's time or more to arrive. The waves meet twice per block: before
// the next tokens are read, and at the block's end. (With one meeting, all loads awaited:
// 33 -> 45 us on 256 tokens of one expert, nothing gained on large problems.)
//
// A partial sum is scaled and added LAG MFMAs after it was issued, four fmas between two
// MFMAs, so neither waits for the other; the empty asm keeps the compiler from moving the
// sums to the end of the block (which spilled), sched_barrier keeps the interleaving.
// The loads are spread over the block: issued in one burst they block the wave's own
// instruction stream until the memory pipeline takes them.
//
// On 32768 tokens of 8 experts, K 7168, N 4096 (fp8 MFMA, bf16 out, 256 x 256): 1480 us with
// a burst of loads, a vector load of the weight scale and no fragments ahead; 1110 with the
// scale through a scalar load and four waves loading; 870 with fragments ahead and counted
// waits, 847 without LDS conflicts and with spread loads (812 to 856 by card; the first launches
// behind an idle time take up to 1190, until the clock has settled). A counted launch takes 1.67 M
// cycles at 2.05 GHz, MFMA busy for 0.94 M of them. Tried without gain: the next tile's first
// loads before this one's stores (877), loads into the L2 two to four blocks ahead (912), 32 x 32
// MFMAs (924), raised wave priority (873), the last round's tiles in quarters (840).
template <class C, bool FAST, bool OUTB>
__global__ __launch_bounds__(C::THREADS, 2 * C::PER_CU) void kg_fprop_kernel(FParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int LAG = C::LAG, S = C::SUMS;
  int* off = (int*)(smem + C::NS * C::STAGE);  // [G + 1]
  int* boff = off + p.G + 1;
  if (!f_offsets<C::THREADS>(p.ms, p.G, C::BT, p.M_total, off, boff)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = KG_ERR_KSUM;
    return;
  }
  const int mt_total = boff[p.G], total = mt_total * p.tiles_n;
  const int grid = gridDim.x, b = blockIdx.x;
  // XCD-contiguous runs when the items take several rounds, as in kg_dgrad
  const int slot = (grid % 8 == 0 && total > grid) ? (b % 8) * (grid / 8) + b / 8 : b;
  const int nk = (p.K + C::TK - 1) / C::TK, nsc = (p.N + 127) / 128;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, j = lane & 15;
  const int wt = w % C::WT, wn = w / C::WT;
  const int c0 = 16 * (q ^ (j & 7)), c1 = 16 * ((q + 4) ^ (j & 7));
  const unsigned char* fragw = smem + (wn * C::NI * 16 + frow(0, j)) * C::TK;
  const unsigned char* fragt = smem + C::OPW + (wt * C::TT * 16 + j) * C::TK;
  const unsigned char* scale = smem + C::SA_OFF + 4 * (wt * C::TT * 16 + j);
  for (int base = 0; base < total; base += grid) {
    const int idx = base + slot;
    if (idx >= total) break;
    // panels of kPanelM m-tiles, m-tiles fastest, as in kg_dgrad (2 or 8: the same times)
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
    const int n0 = nt * C::BN;
    const int nw = n0 + wn * C::NI * 16;  // this wave's outputs, in one weight-scale block
    const ConstFloat* swg =
        (const ConstFloat*)p.sw + ((int64_t)g * nsc + min(nw / 128, nsc - 1)) * nk;
    v4f acc[C::NI][C::TT];
#pragma unroll
    for (int i = 0; i < C::NI; ++i)
#pragma unroll
      for (int tt = 0; tt < C::TT; ++tt) acc[i][tt] = v4f{0.f, 0.f, 0.f, 0.f};
    FLoads<C> L;
    L.setup(p, smem, row0, rows, g, n0, nk, C::ROTATE && nk > 0 ? (nt + 5 * g) % nk : 0);
    Frag<FAST> tf[C::TT], wf[2];
    float sc[C::TT];
    auto read_t = [&](int kb, int tt) {
      const unsigned char* r = fragt + (kb & 1) * C::STAGE + 16 * tt * C::TK;
      tf[tt].set(*(const v4i*)(r + c0), *(const v4i*)(r + c1));
      sc[tt] = *(const float*)(scale + (kb & 1) * C::STAGE + 64 * tt);
    };
    auto read_w = [&](int kb, int i) {
      const unsigned char* r = fragw + (kb & 1) * C::STAGE + frow(i, 0) * C::TK;
      wf[i & 1].set(*(const v4i*)(r + c0), *(const v4i*)(r + c1));
    };
    float swv = 0.f;
    if (nk > 0) {
      // (behind the previous tile's last meeting, so every wave is done with its stages; its
      // stores may be under way, and so may its last loads, which read nothing: a wave's
      // operations end in order, and a place in LDS is always loaded by the same wave)
      swv = swg[L.block(0)];
#pragma unroll
      for (int x = C::LW; x < C::LOADS; ++x) L.load(0, 0, x);
#pragma unroll
      for (int x = 0; x < C::LW; ++x) L.load(0, 0, x);
#pragma unroll
      for (int x = C::LW; x < C::LOADS; ++x) L.load(0, 1, x);
#pragma unroll
      for (int x = 0; x < C::LW; ++x) L.load(1, 0, x);
      f_meet<C::LOADS>();
#pragma unroll
      for (int tt = 0; tt < C::TT; ++tt) read_t(0, tt);
      f_meet<C::LOADS>();
    }
    for (int kb = 0; kb < nk; ++kb) {
      read_w(kb, 0);
      float sx[C::TT];
#pragma unroll
      for (int tt = 0; tt < C::TT; ++tt) sx[tt] = sc[tt] * swv;
      v4f part[LAG + 1];
      auto add = [&](int u) {
        const int i = u / C::TT, tt = u % C::TT;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][tt][r] = fmaf(sx[tt], part[u % (LAG + 1)][r], acc[i][tt][r]);
        asm volatile("" : "+v"(acc[i][tt]));
      };
#pragma unroll
      for (int u = 0; u < S; ++u) {
        const int i = u / C::TT, tt = u % C::TT;
        // the tokens' next block is there, W's block has been read (of the loads, W's next one
        // and the tokens' next but one may be under way)
        if (u == S - C::TT) f_meet<C::LOADS>();
        if (tt == 0 && i + 1 < C::NI) read_w(kb, i + 1);
        part[u % (LAG + 1)] = block_sum(wf[i & 1], tf[tt]);
        if (i == C::NI - 1) read_t(kb + 1, tt);  // (past the last block: not used)
        if (u >= LAG) add(u - LAG);
#pragma unroll
        for (int x = 0; x < C::LT + 1; ++x)
          if (x * (S - C::TT) / (C::LT + 1) == u) L.load(0, kb + 2, C::LW + x);
#pragma unroll
        for (int x = 0; x < C::LW; ++x)
          if (S - C::TT + x * C::TT / C::LW == u) L.load(kb + 2, 0, x);
        if (u == S / 2) swv = swg[L.block(min(kb + 1, nk - 1))];
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int u = S - LAG; u < S; ++u) add(u);
      // W's next block is there, and the tokens' has been read (the loads of the two after
      // them may be under way)
      f_meet<C::LOADS>();
    }
#pragma unroll
    for (int tt = 0; tt < C::TT; ++tt) {
      const int r = (wt * C::TT + tt) * 16 + j;
      if (r >= rows) continue;
      const int64_t at = (int64_t)(row0 + r) * p.ldd;
#pragma unroll
      for (int i = 0; i < C::NI; i += 2) {
        const int n = nw + 16 * i + 8 * q;
        store_run<OUTB>(p.D, at + n, p.N - n, acc[i][tt], acc[i + 1][tt]);
      }
    }
  }
  // no load into this workgroup's LDS outlives it
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
}

// ------------------------------------------------------------------------ streaming kernel

// A workgroup computes 16 NJ outputs of one expert for all its rows, 16 TT at a time: grid
// min(G, M_total) x ceil(N / (16 NJ)), the experts without rows left out. Its 8 waves take the
// blocks of the contraction axis in turn, each adding up its blocks in registers, with the next
// block's operands on their way (two or three more: slower, 140 -> 165 us); the waves' sums are
// added in LDS in a fixed order. A lane reads 32 neighbouring channels of a row, so a
// row's 128 bytes go to four lanes of one load.
//
// Bound by W's bytes: 64 rows dealt out over 32 experts of 4096 x 7168, 28 of which get some (0.82
// GB), take 124 to 136 us by card, 6.0 to 6.6 TB/s (with one block's loads at a time 138 us where
// this takes 127; with 64 outputs per workgroup 139).
constexpr int kStreamWaves = 8, kStreamN = 32;

// The expert with rows that `nth` others with rows come before, its first row and their number, by
// a scan of ms in every wave (a lane holds consecutive experts). rows = 0: there is none.
// Returns false if ms is inconsistent.
__device__ __forceinline__ bool find_rows(const FParams& p, int nth, int* g, int64_t* row0,
                                          int* rows) {
  const int lane = threadIdx.x & 63, per = (p.G + 63) / 64;
  const int e0 = lane * per, e1 = min(p.G, e0 + per);
  int64_t sum = 0;
  int live = 0, neg = 0;
  for (int e = e0; e < e1; ++e) {
    const int v = p.ms[e];
    neg |= v < 0;
    sum += v;
    live += v > 0;
  }
  int64_t to = sum;  // rows and experts up to this lane's last one
  int live_to = live;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t u = __shfl_up(to, d, 64);
    const int v = __shfl_up(live_to, d, 64);
    if (lane >= d) {
      to += u;
      live_to += v;
    }
  }
  const bool ok = __ballot(neg != 0) == 0 && __shfl(to, 63, 64) == p.M_total;
  const uint64_t has = __ballot(live_to > nth);  // the first such lane has the expert
  *rows = 0;
  *g = 0;
  *row0 = 0;
  if (!ok || has == 0) return ok;
  const int owner = __builtin_ctzll(has);
  int64_t at = to - sum;
  int mine = 0, mg = 0, left = nth - (live_to - live);
  for (int e = e0; e < e1 && lane == owner; ++e) {
    const int v = p.ms[e];
    if (v > 0 && left-- == 0) {
      mine = v;
      mg = e;
      break;
    }
    at += v;
  }
  *row0 = __shfl(at, owner, 64);
  *rows = uniform(__shfl(mine, owner, 64));
  *g = uniform(__shfl(mg, owner, 64));
  return true;
}

template <int TT, int NJ, bool FAST, bool OUTB>
__global__ __launch_bounds__(64 * kStreamWaves) void kg_fprop_stream_kernel(FParams p) {
  constexpr int N0 = 16 * NJ;  // outputs of a workgroup
  __shared__ v4f sums[kStreamWaves][NJ * TT][64];
  const int per = p.tiles_n;  // workgroups per expert
  const int nth = blockIdx.x / per, n0 = (blockIdx.x - nth * per) * N0;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, j = lane & 15;
  int64_t row0;
  int rows, g;
  if (!find_rows(p, nth, &g, &row0, &rows)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.status = KG_ERR_KSUM;
    return;
  }
  const int nk = (p.K + 127) / 128, nfull = p.K / 128, nsc = (p.N + 127) / 128;
  const ConstFloat* swg = (const ConstFloat*)p.sw + ((int64_t)g * nsc + n0 / 128) * nk;
  // rows past the end name the last one: what they give is not stored
  const unsigned char* wrow[NJ];
#pragma unroll
  for (int i = 0; i < NJ; ++i)
    wrow[i] =
        p.W + ((int64_t)g * p.N + min(n0 + (NJ == 1 ? j : frow(i, j)), p.N - 1)) * p.K + 32 * q;
  for (int r0 = 0; r0 < rows; r0 += 16 * TT) {
    const unsigned char* arow[TT];
    const float* sa[TT];
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int64_t r = row0 + min(r0 + 16 * tt + j, rows - 1);
      arow[tt] = p.A + r * p.lda + 32 * q;
      sa[tt] = p.sa + r;
    }
    v4f acc[NJ][TT];
#pragma unroll
    for (int i = 0; i < NJ; ++i)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[i][tt] = v4f{0.f, 0.f, 0.f, 0.f};
    auto block = [&](const v4i (&wx)[NJ][2], const v4i (&tx)[TT][2], const float (&s)[TT],
                     float swv) {
      Frag<FAST> tf[TT];
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) tf[tt].set(tx[tt][0], tx[tt][1]);
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        Frag<FAST> wf;
        wf.set(wx[i][0], wx[i][1]);
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) {
          const v4f part = block_sum(wf, tf[tt]);
          const float sx = s[tt] * swv;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][tt][r] = fmaf(sx, part[r], acc[i][tt][r]);
        }
      }
    };
    v4i wx[2][NJ][2], tx[2][TT][2];
    float s[2][TT], sv[2];
    auto load = [&](int kb, int h) {
      sv[h] = swg[kb];
#pragma unroll
      for (int i = 0; i < NJ; ++i) {
        wx[h][i][0] = *(const v4i*)(wrow[i] + kb * 128);
        wx[h][i][1] = *(const v4i*)(wrow[i] + kb * 128 + 16);
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) {
        tx[h][tt][0] = *(const v4i*)(arow[tt] + kb * 128);
        tx[h][tt][1] = *(const v4i*)(arow[tt] + kb * 128 + 16);
        s[h][tt] = sa[tt][(int64_t)kb * p.M_total];
      }
    };
    // This wave's blocks w, w + 8, ... In the loop every load is unconditional, so the compiler
    // knows how many are under way and waits for no more than it needs (loads under conditions:
    // the 64 rows above 136 us, not 128).
    const int nb = nfull > w ? (nfull - w + kStreamWaves - 1) / kStreamWaves : 0;
    int n = 0, kb = w;
    if (nb > 0) load(kb, 0);
    for (; n + 2 < nb; n += 2, kb += 2 * kStreamWaves) {
      load(kb + kStreamWaves, 1);
      block(wx[0], tx[0], s[0], sv[0]);
      __builtin_amdgcn_sched_barrier(0);
      load(kb + 2 * kStreamWaves, 0);
      block(wx[1], tx[1], s[1], sv[1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (n + 1 < nb) {
      load(kb + kStreamWaves, 1);
      block(wx[0], tx[0], s[0], sv[0]);
      block(wx[1], tx[1], s[1], sv[1]);
    } else if (n < nb) {
      block(wx[0], tx[0], s[0], sv[0]);
    }
    if (nfull < nk && w == nfull % kStreamWaves) {  // the last block's K % 128 channels
      const int left = p.K - nfull * 128 - 32 * q;
      const v4i zero = {0, 0, 0, 0};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < NJ; ++i)
          wx[0][i][h] = 16 * h < left ? *(const v4i*)(wrow[i] + nfull * 128 + 16 * h) : zero;
#pragma unroll
        for (int tt = 0; tt < TT; ++tt)
          tx[0][tt][h] = 16 * h < left ? *(const v4i*)(arow[tt] + nfull * 128 + 16 * h) : zero;
      }
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) s[0][tt] = sa[tt][(int64_t)nfull * p.M_total];
      block(wx[0], tx[0], s[0], swg[nfull]);
    }
#pragma unroll
    for (int i = 0; i < NJ; ++i)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) sums[w][i * TT + tt][lane] = acc[i][tt];
    __syncthreads();
    // wave w joins and stores one pair of output tiles (or the only one) of token tile w % TT
    constexpr int PAIR = NJ == 1 ? 1 : 2;
    if (w < TT * NJ / PAIR) {
      const int tt = w % TT, i0 = PAIR * (w / TT);
      v4f x[PAIR];
#pragma unroll
      for (int i = 0; i < PAIR; ++i) {
        x[i] = sums[0][(i0 + i) * TT + tt][lane];
#pragma unroll
        for (int v = 1; v < kStreamWaves; ++v) {
          const v4f y = sums[v][(i0 + i) * TT + tt][lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) x[i][r] += y[r];
        }
      }
      const int r = r0 + 16 * tt + j, n = n0 + 16 * i0 + 4 * PAIR * q;
      if (r < rows) {
        const int64_t at = (row0 + r) * p.ldd + n;
        if constexpr (PAIR == 2) store_run<OUTB>(p.D, at, p.N - n, x[0], x[1]);
        else store_four<OUTB>(p.D, at, p.N - n, x[0]);
      }
    }
    __syncthreads();
  }
}

struct FLaunch {
  const void* fn;
  int bt, bn, lds, per_cu, id;
};

template <class C, bool FAST>
static FLaunch f_tiled(bool outb, int id) {
  const void* fn = outb ? (const void*)kg_fprop_kernel<C, FAST, true>
                        : (const void*)kg_fprop_kernel<C, FAST, false>;
  return FLaunch{fn, C::BT, C::BN, C::NS * C::STAGE, C::PER_CU, id};
}

template <int TT, int NJ, bool FAST>
static FLaunch f_stream(bool outb) {
  const void* fn = outb ? (const void*)kg_fprop_stream_kernel<TT, NJ, FAST, true>
                        : (const void*)kg_fprop_stream_kernel<TT, NJ, FAST, false>;
  return FLaunch{fn, 16 * TT, 16 * NJ, 0, 1, -1};
}

// A tile and what one block of it takes on every compute unit, in tenths of a microsecond:
// `first` while there are no more tiles than compute units, else `round` for PER_CU of them.
struct FTile {
  FLaunch l;
  int first, round;
};

// Which kernel and tile. The experts' sizes are known on the device only, so this goes by
// M_total and G; every choice is right for every distribution of the rows.
//  * Streaming where it takes few workgroups and passes, 3 per compute unit (a tile's time is
//    then the latency of its blocks): streaming / 64 x 128 tiles with K 7168, N 4096: 1, 16, 64
//    rows of one expert 8 / 42, 10 / 25, 20 / 25 us; 4 experts of 2 and 16 rows 20 / 23 and
//    27 / 23; 4 of 4 rows, N 7168, K 2048 14 / 12. A workgroup has 16 outputs where 32
//    would leave half of the compute units idle (what one has under way bounds it: N 4096,
//    K 7168, 1 row 8.1 us with 16 outputs, 10.5 with 32; 16 rows, N 8192 16.2 and 13.0),
//    else 32. TT token tiles hold the rows of a pass: the average, or twice it where several
//    experts share M_total unevenly, up to 32, or 64 of one expert (N 4096, K 7168, 64 rows: 19.8
//    us, in passes of 32 22.4), not in exact products, whose widened fragments spill (23.6).
//  * Streaming as well for the fewest rows of long weight rows with the fp8 MFMA. Measured where the
//    rule above does not take it, with 32 to 128 experts, N 2048 to 8192: the time of the tile
//    chosen else over streaming's, rows in different experts (from G on as many for each) /
//    dealt out at random:
//                         M < G          M = G          M = 2 G        M = 3 G
//      fp8, K 2048                       0.86 / 0.91    0.86 / 0.92    0.84 / 0.86
//      K 3584, 4096       0.99 / 1.02    1.01 / 1.11    0.99 / 1.04    0.97 / 0.98
//      K 5120 to 7168     1.04 / 1.09    1.05 / 1.16    1.04 / 1.10    1.03 / 1.04
//      K 8192                            1.00 / 1.05    0.97 / 1.00    0.97 / 0.99
//      exact, K 3584, 4096  0.89 / 0.93  0.83 / 0.96    0.82 / 0.88
//      K 5120 to 7168     0.95 / 1.02    0.91 / 1.04    0.90 / 0.96
//    (32 experts, N 4096, K 7168, fp8, 1 row each / 32 dealt out: 156 and 164 us / 107 and 131;
//    exact 180 and 161 / 128 and 149.)
//  * Else the tile with the least estimated time, rounds over the compute units times a
//    block's time. The number of 16-byte operand reads per MFMA falls with the tile's size,
//    the latency of a block and the rows that an expert's last tile leaves empty rise.
//    fp8 MFMA, 64 x 64 / 64 x 128 / 128 x 128 / 256 x 256: 256 rows, N 4096, K 7168 25 / 27 /
//    34 / 75 us; 512 rows, K 4096 29 / 18 / 23 / 47; 1024 rows 41 / 29 / 25 / 47; 32 experts
//    of 32 and 97 rows, K 7168 195 / 187 / 173 / 196 and 328 / 259 / 240 / 212.
//    Exact products, 64 x 64 / 64 x 128 / 128 x 128 / 128 x 256: 256 rows 36 / 47 / 61 / 95 us;
//    1024 rows, K 4096 59 / 45 / 41 / 57; 32 experts of 16 and 64 rows, K 7168 214 / 171 /
//    247 / 207 and 312 / 246 / 268 / 226; 32768 rows of 8 experts, K 7168 1.61 to 1.71 ms by
//    card with 128 x 256 (256 x 256, whose widened fragments spill: the same). Two 128 x 128 workgroups
//    per compute unit spill too (61 -> 110 us on the 256 rows).
static FLaunch f_choose(int64_t M, int G, int N, int K, int cus, bool fast, bool outb) {
  const int64_t avg = (M + G - 1) / G, live = G < M ? G : M;
  const int64_t groups = live * ((N + kStreamN - 1) / kStreamN), rows = G == 1 ? avg : 2 * avg;
  if ((avg <= 64 && groups * ((rows + 15) / 16) <= 3 * cus) ||
      (fast && groups < (1 << 23) && M <= (K > 4096 ? 2 : 1) * (int64_t)G && K >= 3584)) {
    if (fast && G == 1 && rows > 32) return f_stream<4, 1, true>(outb);
    if (groups <= cus / 2) {
      if (rows <= 16) return fast ? f_stream<1, 1, true>(outb) : f_stream<1, 1, false>(outb);
      return fast ? f_stream<2, 1, true>(outb) : f_stream<2, 1, false>(outb);
    }
    if (rows <= 16) return fast ? f_stream<1, 2, true>(outb) : f_stream<1, 2, false>(outb);
    return fast ? f_stream<2, 2, true>(outb) : f_stream<2, 2, false>(outb);
  }
  using Tile64 = FCfg<64, 64, 4, 2>;
  using Tile64x128 = FCfg<64, 128, 2, 2>;
  using Tile64x128R = FCfg<64, 128, 2, 2, true>;
  // (more tiles than compute units: 8 experts of 16 rows, N 2048, without / with: fp8 15 / 18 us,
  // exact 21 / 27)
  const bool rotate = K % 4096 == 0 && avg <= 64 && live * ((N + 127) / 128) > cus;
  const FTile tiles[4] = {
      {fast ? f_tiled<FCfg<256, 256, 4, 1>, true>(outb, 0)
            : f_tiled<FCfg<128, 256, 2, 1>, false>(outb, 1), fast ? 15 : 18, fast ? 15 : 18},
      {fast ? f_tiled<FCfg<128, 128, 4, 2>, true>(outb, 2)
            : f_tiled<FCfg<128, 128, 4, 1>, false>(outb, 3), fast ? 7 : 12, 12},
      {rotate ? (fast ? f_tiled<Tile64x128R, true>(outb, 4) : f_tiled<Tile64x128R, false>(outb, 5))
              : (fast ? f_tiled<Tile64x128, true>(outb, 6) : f_tiled<Tile64x128, false>(outb, 7)),
       fast ? 5 : 8, fast ? 10 : 15},
      {fast ? f_tiled<Tile64, true>(outb, 8) : f_tiled<Tile64, false>(outb, 9), fast ? 4 : 6,
       fast ? 8 : 9}};
  int best = rotate ? 2 : 0;
  int64_t least = INT64_MAX;
  for (int i = 0; i < 4 && !rotate; ++i) {
    const FLaunch& l = tiles[i].l;
    // tiles along the rows, in tenths: one expert's are known; of several, each has a last
    // one that is half filled on average
    int64_t mt = live == 1 ? (M + l.bt - 1) / l.bt * 10 : 10 * M / l.bt + 5 * live;
    if (mt < 10 * live) mt = 10 * live;
    const int64_t n = (mt * ((N + l.bn - 1) / l.bn) + 9) / 10, at_once = (int64_t)cus * l.per_cu;
    const int64_t t = n <= cus ? tiles[i].first : (n + at_once - 1) / at_once * tiles[i].round;
    // ties go to the smaller tile, whose estimate errs less
    if (t <= least) {
      least = t;
      best = i;
    }
  }
  return tiles[best].l;
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
  FLaunch l = f_choose(M_total, G, N, K, cus, fast, outb);
  p.tiles_n = (N + l.bn - 1) / l.bn;
  int64_t grid;
  if (l.id < 0) {
    grid = (int64_t)(G < M_total ? G : M_total) * p.tiles_n;
  } else {
    l.lds += 2 * (G + 1) * 4;
    static std::mutex mu;
    static int set[64][10][2];  // the largest LDS size asked for so far
    {
      std::lock_guard<std::mutex> lk(mu);
      if (set[dev][l.id][outb] < l.lds) {
        if (hipFuncSetAttribute(l.fn, hipFuncAttributeMaxDynamicSharedMemorySize, l.lds) !=
            hipSuccess)
          return KG_ERR_HIP;
        set[dev][l.id][outb] = l.lds;
      }
    }
    const int64_t max_items = (M_total / l.bt + G) * (int64_t)p.tiles_n;
    if (max_items > INT32_MAX - 4096) return KG_ERR_UNSUPPORTED;  // (indexes pass it by a grid)
    const int64_t at_once = (int64_t)cus * l.per_cu;
    grid = max_items < at_once ? max_items : at_once;
  }
  void* args[] = {&p};
  return hipLaunchKernel(l.fn, dim3((unsigned)grid), dim3(512), args, (size_t)l.lds,
                         (hipStream_t)stream) == hipSuccess
             ? KG_OK
             : KG_ERR_HIP;
}
