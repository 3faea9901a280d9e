// kg_ortho.hip -- weight updates made nearly orthogonal on gfx950, C ABI kg_orthogonalize.
//
// Newton-Schulz: X = U / |U|_F, and `steps` times, on the side of the shorter axis n of n x m,
//   A = X X^T,  B = b A + c A A,  X = a X + B X,  (a, b, c) = (3.4445, -4.7750, 2.0315),
// which takes every singular value of X towards 1 (into 0.68 .. 1.27, not onto it).
//
// The work is the three products, on the fp16 MFMA (bf16's rate; every matrix here has entries
// bounded by its singular values, so fp16's range suffices, and its 11 bits are 8 times as exact).
// A and A A are symmetric: only tiles on one side of the diagonal are computed, and stored
// twice. All three products are of the form C[i][j] = sum_k P[i][k] Q[j][k] with contiguous k:
// A of rows of X, A A of rows of A, B X of rows of B and of X^T, so X is kept in both orders, and the
// kernel that makes X writes both.
//
// What fp16 costs, and what is done about it. Small singular values grow by a = 3.4445 a step and
// carry the rounding of a X with them, so the X that is multiplied by a is kept as two halves
// (22 bits) up to the last step but one. A and B are near multiples of the identity in the end, so
// the rounding of their diagonals, which acts as a common factor, is kept beside them in fp32. With
// both, results of five steps are 0.4e-3 to 1.5e-3 of their norm off 64-bit ones (gaussian,
// channel-scaled, low-rank and decaying spectra; 24 x 40 to 777 x 1000), against 1e-2 to 3e-1 with bf16
// operands. More steps add to it (8: 0.4e-3 to 2.8e-3), as the iteration does not settle.
//
// Powers of two bring the entries into fp16's range: X by about sqrt(m) (entries of an orthonormal
// row are 1 / sqrt(m)), A and B by 2^13 (|A| <= 1.7, |B| <= 2.9).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "kg_device.h"
#include "kg_host.h"
#include "kgwgrad.h"

namespace kg {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr float kNsA = 3.4445f, kNsB = -4.7750f, kNsC = 2.0315f;
constexpr float kScaleA = 0x1p13f, kScaleB = 0x1p13f, kLow = 0x1p11f;
constexpr int kNormChunks = 256;  // partial sums of squares per matrix, at most
constexpr int kOrthoMax = 1 << 16;

struct OParams {
  const void* U;
  unsigned short* O;
  double* parts;  // [G][kNormChunks]
  unsigned short *X, *XT, *XN, *LO, *A, *B;  // XN: the X^T that a step writes
  float *dA, *dB;
  int64_t sx, sxt, sa;  // elements of a matrix's X, XT and A
  float cx;             // scale of X
  int G, R, C, n, m, np, mp, ldn, ldm;
  int b16, wide, tiles_i, tiles_j, per;  // per: tiles of a matrix
  int low_in, low_out;
  int chunks;
  int first, count, quarter;  // tiles of this launch; whether each is a quarter of one twice as large
};

// Eight neighbours of U from element `at`, of which the first `n` count; the rest are zeros. Loaded as they lie
// (also what follows, up to U's end), so that several loads are under way before the first is used.
struct Eight {
  v4i a, b;
};
__device__ __forceinline__ Eight u_load(const OParams& p, int64_t at, int n) {
  typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));
  Eight x = {};
  if (n > 0) {
    if (at + 8 <= (int64_t)p.G * p.R * p.C) {
      const char* u = (const char*)p.U + at * (p.b16 ? 2 : 4);
      x.a = *(const v4i_any*)u;
      if (!p.b16) x.b = *(const v4i_any*)(u + 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= n) continue;
        if (p.b16) x.a[e >> 1] |= (int)((const unsigned short*)p.U)[at + e] << (16 * (e & 1));
        else (e < 4 ? x.a : x.b)[e & 3] = ((const int*)p.U)[at + e];
      }
    }
  }
  return x;
}
__device__ __forceinline__ void u_values(const OParams& p, const Eight& u, int n, float* x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int two = u.a[e >> 1], one = (e < 4 ? u.a : u.b)[e & 3];
    const int bits = !p.b16 ? one : e & 1 ? two & (int)0xFFFF0000 : two << 16;
    x[e] = e < n ? __builtin_bit_cast(float, bits) : 0.f;
  }
}

// x times inv, rounded to fp32. (Left alone, the compiler rounds 64 bits straight to fp16 behind it, in
// some 25 instructions: the card has no such conversion.)
__device__ __forceinline__ float scaled(float x, double inv) {
  float v = (float)((double)x * inv);
  asm("" : "+v"(v));
  return v;
}

// ---------------------------------------------------------------------------- norm, first X

// Sums of squares in 64 bits (fp32 squares of gradients may leave its range), in a fixed order.
// 8 x 4096 x 7168 bf16: 96 us, 4.9 TB/s.
constexpr int kNormStep = 8 * 256;
__host__ __device__ constexpr int64_t norm_chunk(int64_t size) {
  const int64_t even = (size + kNormChunks - 1) / kNormChunks;
  return (even + 2 * kNormStep - 1) / (2 * kNormStep) * (2 * kNormStep);
}
__global__ __launch_bounds__(256) void kg_ortho_norm_kernel(OParams p) {
  __shared__ double sums[4];
  const int64_t size = (int64_t)p.R * p.C, base = (int64_t)blockIdx.y * size, per = norm_chunk(size);
  const int64_t from = blockIdx.x * per, to = from + per < size ? from + per : size;
  double s = 0;
#pragma unroll 4
  for (int64_t i = from + 8 * threadIdx.x; i < to; i += kNormStep) {
    const int n = to - i < 8 ? (int)(to - i) : 8;
    float x[8];
    u_values(p, u_load(p, base + i, n), n, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fma((double)x[e], (double)x[e], s);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    p.parts[blockIdx.y * kNormChunks + blockIdx.x] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// X and X^T of U / |U|, scaled, with their low halves; zeros in the padding. One 64 x 64 tile
// per workgroup, turned in LDS (16-byte chunk c of a row in slot c ^ its key, as the reads that
// turn it take four neighbouring rows at once). Memory bounds it: 8 x 4096 x 7168 bf16 370 us, 5.1 TB/s.
__global__ __launch_bounds__(256) void kg_ortho_init_kernel(OParams p) {
  __shared__ __attribute__((aligned(16))) unsigned char lds[2][64 * 128];  // X, low halves
  __shared__ double inv_s;
  const int g = blockIdx.y, t = threadIdx.x;
  // rows and columns of U, and of the padded matrix
  const int cp = p.wide ? p.mp : p.np;
  const int across = cp / 64, r0 = blockIdx.x / across * 64, c0 = blockIdx.x % across * 64;
  const int64_t base = (int64_t)g * p.R * p.C;
  const int r = t >> 3, c = t & 7;
  Eight raw[2];
  int left[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = r0 + r + 32 * half, col = c0 + 8 * c;
    left[half] = row < p.R ? p.C - col : 0;
    raw[half] = u_load(p, base + (int64_t)row * p.C + col, left[half]);
  }
  if (t < 64) {
    double s = 0;
    for (int i = t; i < p.chunks; i += 64) s += p.parts[g * kNormChunks + i];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
    if (t == 0) inv_s = s > 0 ? (double)p.cx / sqrt(s) : s == 0 ? 0.0 : s;  // NaN stays
  }
  __syncthreads();
  const double inv = inv_s;
  // direct: the order of U's rows; turned: the other one
  unsigned short* direct = p.wide ? p.X + g * p.sx : p.XT + g * p.sxt;
  unsigned short* turned = p.wide ? p.XT + g * p.sxt : p.X + g * p.sx;
  unsigned short* low = p.LO + g * p.sxt;  // in the order of X^T
  const int ldd = p.wide ? p.ldm : p.ldn, ldt = p.wide ? p.ldn : p.ldm;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = r + 32 * half;
    float x[8];
    u_values(p, raw[half], left[half], x);
    v8h h, l;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = scaled(x[e], inv);
      h[e] = (_Float16)v;
      l[e] = (_Float16)((v - (float)h[e]) * kLow);
    }
    const int slot = row * 128 + 16 * (c ^ (row & 7));
    *(v8h*)(lds[0] + slot) = h;
    const int64_t at = (int64_t)(r0 + row) * ldd + c0 + 8 * c;
    *(v8h*)(direct + at) = h;
    if (p.wide) *(v8h*)(lds[1] + slot) = l;
    else *(v8h*)(low + at) = l;
  }
  __syncthreads();
  // wave w turns 16 columns: lane c of 16 gets column c of 4 rows per read
  const int w = t >> 6, lane = t & 63, jl = lane & 15, c4 = lane & 3;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which == 1 && !p.wide) break;
#pragma unroll
    for (int jb = 0; jb < 2; ++jb) {
      const int j = 32 * jb + 8 * (lane >> 4);
      v4bf half[2];
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int row = j + 4 * s + (jl >> 2);
        half[s] = tr16(lds[which] + row * 128 + 16 * ((2 * w + (c4 >> 1)) ^ (row & 7)) + 8 * (c4 & 1));
      }
      const v2i a = __builtin_bit_cast(v2i, half[0]), b = __builtin_bit_cast(v2i, half[1]);
      unsigned short* to = which == 0 ? turned : low;
      *(v4i*)(to + (int64_t)(c0 + 16 * w + jl) * ldt + r0 + j) = v4i{a.x, a.y, b.x, b.y};
    }
  }
}

// ------------------------------------------------------------------------------- products

// BS x BS results per workgroup, LDS stages of 64 k (128 bytes) of BS rows of P and of Q. Loads go
// straight to LDS, waits count them. With 8 waves (4 along j, 2 along i) and two stages the loop is
// kg_fprop's: Q's fragments are read a block ahead, loads are spread over the MFMAs. With 4 waves, for
// products of few tiles, what counts is how much is under way: three blocks, and what the end needs.
template <int BS_, int PER_CU_, int WAVES_ = 8, int STAGES_ = 2>
struct OCfg {
  static constexpr int BS = BS_, PER_CU = PER_CU_, WAVES = WAVES_, STAGES = STAGES_, TK = 64;
  static constexpr int THREADS = 64 * WAVES, WT = WAVES / 2, WN = 2;
  static constexpr int TT = BS / WT / 16, NI = BS / WN / 16;
  static constexpr int OPW = BS * 128, STAGE = 2 * OPW;
  static constexpr int LW = BS / (8 * WAVES), LOADS = 2 * LW;
  static_assert(NI % 2 == 0 && BS * BS * 2 <= STAGES * STAGE, "a wave's results fit in LDS");
};

// (as in kg_fprop: row m of MFMA row tile i holds result row orow(i, m) of the wave's, so a
// lane's four results of two tiles are eight neighbours)
__device__ __forceinline__ constexpr int orow(int i, int m) {
  return 32 * (i >> 1) + 8 * (m >> 2) + 4 * (i & 1) + (m & 3);
}
// LDS slot of chunk c of a row is c ^ key, with the key m & 7 of the MFMA row (column) m.
__device__ __forceinline__ constexpr int okey_q(int r) { return r & 7; }
__device__ __forceinline__ constexpr int okey_p(int r) { return (r & 3) | ((r >> 3) & 1) << 2; }

template <int N>
__device__ __forceinline__ void o_meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(N) & ~0xF00);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ v4f mfma_f16(const v8h& a, const v8h& b, const v4f& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

enum { kGram, kPoly, kStep, kLast };  // A; B; X; X as the result

// Tile idx of the triangle of T x T tiles: panels of 4 rows I, in each J upwards.
__device__ __forceinline__ void triangle(int idx, int T, int* I, int* J) {
  for (int r = 0;; r += 4) {
    const int rows = min(4, T - r), head = rows * (rows + 1) / 2;
    const int n = head + rows * (T - r - rows);
    if (idx < n) {
      if (idx >= head) {
        *J = r + rows + (idx - head) / rows;
        *I = r + (idx - head) % rows;
      } else {
        int j = 0;
        while (idx > j) idx -= ++j;
        *J = r + j;
        *I = r + idx;
      }
      return;
    }
    idx -= n;
  }
}

template <class C, int MODE>
__global__ __launch_bounds__(C::THREADS, C::WAVES / 4 * C::PER_CU) void kg_ortho_kernel(OParams p) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int TT = C::TT, NI = C::NI;
  constexpr bool SYM = MODE == kGram || MODE == kPoly;
  const int total = p.count, grid = gridDim.x, b = blockIdx.x;
  // neighbouring tiles on one XCD (workgroups go round the eight): its L2 holds what they share
  const int slot = grid % 8 == 0 ? (b % 8) * (grid / 8) + b / 8 : b;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, jl = lane & 15;
  const int wt = w % C::WT, wn = w / C::WT;
  const int c0 = 16 * (q ^ (jl & 7)), c1 = 16 * ((q + 4) ^ (jl & 7));
  const unsigned char* fragp = smem + (wn * NI * 16 + orow(0, jl)) * 128;
  const unsigned char* fragq = smem + C::OPW + (wt * TT * 16 + jl) * 128;
  const uint32_t lds = lds_addr(smem);
  const int ld = MODE == kGram ? p.ldm : p.ldn, nk = (MODE == kGram ? p.mp : p.np) / C::TK;
  const int rows_j = SYM ? p.np : p.mp;
  // this lane's row and chunk of a load of 8 rows, for P and Q
  const int lr = 8 * w + (lane >> 3);
  const uint32_t offp = (uint32_t)(lr * ld * 2 + 16 * ((lane & 7) ^ okey_p(lr)));
  const uint32_t offq = (uint32_t)(lr * ld * 2 + 16 * ((lane & 7) ^ okey_q(lr)));
  for (int base = 0; base < total; base += grid) {
    if (base + slot >= total) break;
    const int idx = p.first + (p.quarter ? (base + slot) >> 2 : base + slot);
    const int g = idx / p.per;
    int I, J;
    if constexpr (SYM) {
      triangle(idx - g * p.per, p.tiles_i, &I, &J);
    } else {
      const int r = idx - g * p.per, per_panel = 4 * p.tiles_j, panel = r / per_panel;
      const int wi = r - panel * per_panel, pm = min(4, p.tiles_i - 4 * panel);
      I = 4 * panel + wi % pm, J = wi / pm;
    }
    if (p.quarter) {
      I = 2 * I + ((base + slot) >> 1 & 1), J = 2 * J + ((base + slot) & 1);
      if ((SYM && I > J) || I * C::BS >= p.np || J * C::BS >= rows_j) continue;
    }
    const int i0 = uniform(I) * C::BS, j0 = uniform(J) * C::BS;
    const unsigned short* P = MODE == kGram   ? p.X + g * p.sx
                              : MODE == kPoly ? p.A + g * p.sa
                                              : p.B + g * p.sa;
    const unsigned short* Q = SYM ? P : p.XT + g * p.sxt;
    const unsigned char* Pb = (const unsigned char*)(P + (int64_t)i0 * ld);
    const unsigned char* Qb = (const unsigned char*)(Q + (int64_t)j0 * ld);
    const uint32_t pbytes = (uint32_t)((min(C::BS, p.np - i0) - 1) * ld * 2 + 128);
    const uint32_t qbytes = (uint32_t)((min(C::BS, rows_j - j0) - 1) * ld * 2 + 128);
    // rows that the matrix lacks and blocks past the last one read as zeros
    auto load_p = [&](int kb, int x) {
      load16_lds(make_rsrc(Pb + (int64_t)kb * 128, kb < nk ? pbytes : 0u),
                 lds + kb % C::STAGES * C::STAGE + 1024 * (w + C::WAVES * x),
                 offp + (uint32_t)(8 * C::WAVES * x * ld * 2));
    };
    auto load_q = [&](int kb, int x) {
      load16_lds(make_rsrc(Qb + (int64_t)kb * 128, kb < nk ? qbytes : 0u),
                 lds + kb % C::STAGES * C::STAGE + C::OPW + 1024 * (w + C::WAVES * x),
                 offq + (uint32_t)(8 * C::WAVES * x * ld * 2));
    };
    v4f acc[NI][TT];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) acc[i][tt] = v4f{0.f, 0.f, 0.f, 0.f};
    v8h qf[TT][2], pf[2][2];
    auto read_q = [&](int kb, int tt) {
      const unsigned char* r = fragq + kb % C::STAGES * C::STAGE + 16 * tt * 128;
      qf[tt][0] = *(const v8h*)(r + c0);
      qf[tt][1] = *(const v8h*)(r + c1);
    };
    auto read_p = [&](int kb, int i) {
      const unsigned char* r = fragp + kb % C::STAGES * C::STAGE + orow(i, 0) * 128;
      pf[i & 1][0] = *(const v8h*)(r + c0);
      pf[i & 1][1] = *(const v8h*)(r + c1);
    };
    // What the ends of results need: before the products where there are registers for it, else
    // each column tile's before the one before it is stored (a wait for loads is one for all
    // stores that went before them).
    const int iw = i0 + wn * NI * 16, jw = j0 + wt * TT * 16;
    constexpr bool EARLY = C::STAGES > 2;
    static_assert(!EARLY || TT == 2);
    v8h ea[2][NI / 2], el[2][NI / 2];  // A or X; low halves
    float dj[2];
    auto fetch = [&](int tt) {
      const int j = jw + 16 * tt + jl;
#pragma unroll
      for (int i2 = 0; i2 < NI / 2; ++i2) {
        const int i = iw + 32 * i2 + 8 * q;
        const bool in = j < rows_j && i < p.np;
        const int64_t at = (int64_t)j * p.ldn + i;
        ea[tt & 1][i2] = el[tt & 1][i2] = v8h{};
        if constexpr (MODE == kPoly) {
          if (in) ea[tt & 1][i2] = *(const v8h*)(p.A + g * p.sa + at);
        } else if constexpr (MODE != kGram) {
          if (in) ea[tt & 1][i2] = *(const v8h*)(p.XT + g * p.sxt + at);
          if (in && p.low_in) el[tt & 1][i2] = *(const v8h*)(p.LO + g * p.sxt + at);
        }
      }
      if constexpr (MODE == kPoly) dj[tt & 1] = j < p.np ? p.dA[g * p.np + j] : 0.f;
    };
    // the diagonals' roundings of the tile's rows i, to LDS behind the stages
    float* dis = (float*)(smem + C::STAGES * C::STAGE);
    float di_mine = 0.f;
    if (MODE != kGram && (int)threadIdx.x < C::BS && i0 + (int)threadIdx.x < p.np)
      di_mine = (MODE == kPoly ? p.dA : p.dB)[g * p.np + i0 + threadIdx.x];
    if constexpr (EARLY) {
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) fetch(tt);
#pragma unroll
      for (int kb = 0; kb < C::STAGES - 1; ++kb)
#pragma unroll
        for (int x = 0; x < C::LW; ++x) {
          load_q(kb, x);
          load_p(kb, x);
        }
      for (int kb = 0; kb < nk; ++kb) {
        // block kb is there, block kb - 1 has been read by every wave
        o_meet<(C::STAGES - 2) * C::LOADS>();
#pragma unroll
        for (int x = 0; x < C::LW; ++x) {
          load_q(kb + C::STAGES - 1, x);
          load_p(kb + C::STAGES - 1, x);
        }
#pragma unroll
        for (int tt = 0; tt < TT; ++tt) read_q(kb, tt);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          read_p(kb, i);
#pragma unroll
          for (int u = 0; u < 2 * TT; ++u)
            acc[i][u % TT] = mfma_f16(pf[i & 1][u / TT], qf[u % TT][u / TT], acc[i][u % TT]);
        }
      }
    } else {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int x = 0; x < C::LW; ++x) load_q(kb, x);
#pragma unroll
        for (int x = 0; x < C::LW; ++x) load_p(kb, x);
      }
      o_meet<C::LOADS>();
#pragma unroll
      for (int tt = 0; tt < TT; ++tt) read_q(0, tt);
      o_meet<C::LOADS>();
      for (int kb = 0; kb < nk; ++kb) {
        constexpr int S = NI * 2 * TT, LASTI = S - 2 * TT;  // MFMAs of a block, and before the last i
        read_p(kb, 0);
#pragma unroll
        for (int u = 0; u < S; ++u) {
          const int i = u / (2 * TT), h = u / TT % 2, tt = u % TT;
          // Q's next block is there, P's block has been read by every wave
          if (u == LASTI) o_meet<C::LOADS>();
          if (h == 0 && tt == 0 && i + 1 < NI) read_p(kb, i + 1);
          acc[i][tt] = mfma_f16(pf[i & 1][h], qf[tt][h], acc[i][tt]);
          if (i == NI - 1 && h == 1) read_q(kb + 1, tt);  // (past the last block: not used)
#pragma unroll
          for (int x = 0; x < C::LW; ++x) {
            if (x * LASTI / C::LW == u) load_q(kb + 2, x);
            if (LASTI + x * 2 * TT / C::LW == u) load_p(kb + 2, x);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        // P's next block is there, Q's has been read by every wave
        o_meet<C::LOADS>();
      }
    }
    if (MODE != kGram && threadIdx.x < C::BS) dis[threadIdx.x] = di_mine;
    // No load is under way into the LDS that turns the results.
    o_meet<0>();
    if constexpr (!EARLY) fetch(0);
    unsigned char* turn = smem + w * (TT * 16 * NI * 16 * 2);  // [j][i] of this wave
    const bool mirror = !SYM || I != J;
    unsigned short* out = MODE == kGram   ? p.A + g * p.sa
                          : MODE == kPoly ? p.B + g * p.sa
                                          : p.XN + g * p.sxt;
#pragma unroll
    for (int tt = 0; tt < TT; ++tt) {
      const int j = jw + 16 * tt + jl;
      if (!EARLY && tt + 1 < TT) fetch(tt + 1);
#pragma unroll
      for (int i2 = 0; i2 < NI / 2; ++i2) {
        const int i = iw + 32 * i2 + 8 * q;
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = acc[2 * i2 + (e >> 2)][tt][e & 3];
        const bool in = j < rows_j && i < p.np;
        const int64_t at = (int64_t)j * p.ldn + i;
        v8h o;
        if constexpr (MODE == kGram) {
          const float s = kScaleA / (p.cx * p.cx);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] *= s;
            o[e] = (_Float16)v[e];
          }
        } else if constexpr (MODE == kPoly) {
          const v8h a = ea[tt & 1][i2];
          const float* di = dis + (i - i0);
          constexpr float fb = kScaleB / kScaleA * kNsB, fc = kScaleB / (kScaleA * kScaleA) * kNsC;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = (float)a[e], d = dj[tt & 1];
            v[e] = fmaf(fc, fmaf(di[e] + d, x, v[e]), fb * (i + e == j ? x + d : x));
            o[e] = (_Float16)v[e];
          }
        } else {
          const v8h a = ea[tt & 1][i2], l = el[tt & 1][i2];
          const float* di = dis + (i - i0);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float st = fmaf((float)l[e], 1 / kLow, (float)a[e]);
            v[e] = fmaf(kNsA + di[e] / kScaleB, st, v[e] / kScaleB);
            if constexpr (MODE == kStep) o[e] = (_Float16)v[e];
            else o[e] = __builtin_bit_cast(_Float16, (__bf16)(v[e] / p.cx));
          }
        }
        if constexpr (SYM) {
          float* d = MODE == kGram ? p.dA : p.dB;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (i + e == j && in) d[g * p.np + j] = v[e] - (float)o[e];
        }
        if constexpr (MODE == kLast) {
          if (!p.wide && j < p.m && i < p.n) {  // O [m, n]
            unsigned short* d = p.O + ((int64_t)g * p.m + j) * p.n + i;
            if (i + 8 <= p.n) {
              typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));
              *(v4i_any*)d = __builtin_bit_cast(v4i, o);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const _Float16 one = o[e];  // (a bit cast of the element itself reads the first one)
                if (i + e < p.n) d[e] = __builtin_bit_cast(unsigned short, one);
              }
            }
          }
        } else if (in) {
          *(v8h*)(out + at) = o;
        }
        if constexpr (MODE == kStep) {
          if (p.low_out && in) {
            v8h l;
#pragma unroll
            for (int e = 0; e < 8; ++e) l[e] = (_Float16)((v[e] - (float)o[e]) * kLow);
            *(v8h*)(p.LO + g * p.sxt + at) = l;
          }
        }
        if (mirror && (MODE != kLast || p.wide)) {
          const int jr = 16 * tt + jl, c = 4 * i2 + q;
          *(v8h*)(turn + jr * (NI * 32) + 16 * (c ^ (jr & (2 * NI - 1)))) = o;
        }
      }
    }
    if (mirror && (MODE != kLast || p.wide)) {
      // the other order: lane c of 16 gets column i = c of 4 rows j per read
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int r4 = (lane & 15) >> 2, c4 = lane & 3;
      unsigned short* mir = MODE == kGram   ? p.A + g * p.sa
                            : MODE == kPoly ? p.B + g * p.sa
                                            : p.X + g * p.sx;
      const int ldo = SYM ? p.ldn : p.ldm;
#pragma unroll
      for (int ib = 0; ib < NI; ++ib)
#pragma unroll
        for (int jb = 0; jb < (TT + 1) / 2; ++jb) {
          const int jr = 32 * jb + 8 * q;
          const int c = 2 * ib + (c4 >> 1);
          v4bf half[2];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int row = jr + 4 * s + r4;
            half[s] = tr16(turn + row * (NI * 32) + 16 * (c ^ (row & (2 * NI - 1))) + 8 * (c4 & 1));
          }
          const v2i x = __builtin_bit_cast(v2i, half[0]), y = __builtin_bit_cast(v2i, half[1]);
          const v4i o = {x.x, x.y, y.x, y.y};
          const int i = iw + 16 * ib + jl, j = jw + jr;
          if constexpr (MODE == kLast) {
            if (i < p.n && j < p.m) {  // O [n, m]
              unsigned short* d = p.O + ((int64_t)g * p.n + i) * p.m + j;
              if (j + 8 <= p.m) {
                typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));
                *(v4i_any*)d = o;
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (j + e < p.m) d[e] = (unsigned short)((uint32_t)o[e >> 1] >> (16 * (e & 1)));
              }
            }
          } else if (i < p.np && j < rows_j) {
            *(v4i*)(mir + (int64_t)i * ldo + j) = o;
          }
        }
    }
    __syncthreads();  // the results have left the LDS that the next tile loads into
  }
}

// ---------------------------------------------------------------------- small matrices

// A matrix with a short axis of up to 128 whose X fits in LDS, from U to O in one workgroup: the 17
// launches of the other way take 3 to 5 us each however small their matrices are. X [NP][mp] lies in
// LDS as fp16, A and then B [NP][NP] beside it. A wave owns every eighth tile of 16 columns of X, whose
// state stays in its registers in fp32; X's other order is read by the transposing reads. A and
// A A: wave w % NI has the tiles (i, i + d), d = 0 .. NI / 2, round the end, so each pair of
// rows meets once (twice at d = NI / 2); with NI < 8 the waves share m and add up in LDS, in order.
// In us, here and by launches: 4 of 24 x 24 13 and 56, 8 of 64 x 256 25 and 63, 8 of 32 x 2048 54
// and 99, 8 of 128 x 384 65 and 72, 300 of 100 x 380 135 and 495. What bounds it: of 65, the norm takes 4,
// U's two ways into LDS 16, a step 8, half of it B X, which reads B anew for every column tile.

// Column tiles of a wave: 128 registers of state (n > 64, where the sums take twice as many, 96)
template <int NI>
constexpr int kSmallTiles = NI == 8 ? 3 : 32 / NI;
struct SmallLds {
  int a, da, db, parts, total;  // byte offsets
};
__host__ __device__ constexpr SmallLds small_lds(int ni, int mp) {
  SmallLds s{};
  const int np = 16 * ni, lda = np < 64 ? 64 : np;
  s.a = np * mp * 2;
  s.da = s.a + np * lda * 2;
  s.db = s.da + np * 4;
  s.parts = s.db + np * 4;
  s.total = s.parts + (ni < 8 ? (8 - ni) * (ni / 2 + 1) * 1024 : 64);  // (and the norm's sums before)
  return s;
}

template <int NI>
__global__ __launch_bounds__(512, 2) void kg_ortho_small_kernel(OParams p, int steps) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  constexpr int NP = 16 * NI, LDA = NP < 64 ? 64 : NP, TJ = kSmallTiles<NI>, D = NI / 2 + 1;
  constexpr int GROUPS = 8 / NI, PAIR = NI == 2 ? 2 : 1;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  const int q = lane >> 4, jl = lane & 15, mp = p.mp, g = blockIdx.x;
  const SmallLds at = small_lds(NI, mp);
  unsigned char *X = smem, *A = smem + at.a;
  float *dA = (float*)(smem + at.da), *dB = (float*)(smem + at.db);
  const int64_t base = (int64_t)g * p.R * p.C;
  // f(row, c, values) for U's units of eight elements 8 c .. of a row, four of them under way
  const int units_row = (p.C + 7) / 8, units = p.R * units_row;
  const int row0 = threadIdx.x / units_row, c0 = threadIdx.x - row0 * units_row;
  const int rows_on = 512 / units_row, on = 512 - rows_on * units_row;  // the next unit of a thread
  auto each = [&](auto f) {
    int row = row0, c = c0;
    for (int u = threadIdx.x; u < units; u += 4 * 512) {
      Eight raw[4];
      int rows[4], cs[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        rows[s] = row, cs[s] = c;
        raw[s] = u_load(p, base + (int64_t)row * p.C + 8 * c, row < p.R ? p.C - 8 * c : 0);
        row += rows_on, c += on;
        if (c >= units_row) c -= units_row, ++row;
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        float x[8];
        u_values(p, raw[s], p.C - 8 * cs[s], x);
        if (rows[s] < p.R) f(rows[s], cs[s], x);
      }
    }
  };
  double sum = 0;
  each([&](int, int, const float* x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fma((double)x[e], (double)x[e], sum);
  });
  for (int c = threadIdx.x; c < NP * mp / 8; c += 512) *(v4i*)(X + 16 * c) = v4i{0, 0, 0, 0};
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
  double* sums = (double*)(smem + at.parts);
  if (lane == 0) sums[w] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += sums[i];
  const double inv = sum > 0 ? (double)p.cx / sqrt(sum) : sum == 0 ? 0.0 : sum;  // NaN stays
  // X [16 it + jl][16 (w + 8 t) + 4 q + r] is st[t][it][r], its fp16 value in LDS: 16-byte chunk c of
  // a row in slot c ^ (row & 7)
  v4f st[TJ][NI];
  typedef unsigned short v4u16 __attribute__((ext_vector_type(4)));
  auto place = [&](int t, int it) {
    return (v4u16*)(X + (16 * it + jl) * mp * 2 +
                    16 * ((2 * (w + 8 * t) + (q >> 1)) ^ (jl & 7)) + 8 * (q & 1));
  };
  auto put = [&](int t) {
#pragma unroll
    for (int it = 0; it < NI; ++it) {
      v4u16 o;
#pragma unroll
      for (int r = 0; r < 4; ++r) o[r] = __builtin_bit_cast(unsigned short, (_Float16)st[t][it][r]);
      *place(t, it) = o;
    }
  };
  // U over its norm comes into the registers through X's place: first what its fp16 values lack, then
  // those, which stay there
  v4u16 low[TJ][NI];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    each([&](int row, int c, const float* x) {
      v8h h;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = scaled(x[e], inv);
        h[e] = (_Float16)v;
        if (half == 0) h[e] = (_Float16)((v - (float)h[e]) * kLow);
      }
      if (p.wide) {
        *(v8h*)(X + row * mp * 2 + 16 * (c ^ (row & 7))) = h;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)  // (NP is a multiple of 8)
          *(_Float16*)(X + (8 * c + e) * mp * 2 + 16 * ((row >> 3) ^ e) + 2 * (row & 7)) = h[e];
      }
    });
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TJ; ++t)
#pragma unroll
      for (int it = 0; it < NI; ++it) {
        v4u16 o = {};
        if (16 * (w + 8 * t) < mp) o = *place(t, it);
        if (half == 0) {
          low[t][it] = o;
          continue;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const unsigned short hi = o[r], lo = low[t][it][r];
          st[t][it][r] = fmaf((float)__builtin_bit_cast(_Float16, lo), 1 / kLow,
                              (float)__builtin_bit_cast(_Float16, hi));
        }
      }
    if (half == 0) __syncthreads();
  }
  auto x_row = [&](int i, int kb) {
    return *(const v8h*)(X + (16 * i + jl) * mp * 2 + 16 * ((4 * kb + q) ^ (jl & 7)));
  };
  auto a_row = [&](int i, int kb) {
    return *(const v8h*)(A + (16 * i + jl) * LDA * 2 + 16 * ((4 * kb + q) ^ (jl & 7)));
  };
  // a tile of A or B, [16 i + jl][16 j + 4 q + r], in both orders where no other wave has it
  const int i = w % NI, grp = w / NI;
  auto put_a = [&](int d, const v4f& v) {
    typedef _Float16 v4h __attribute__((ext_vector_type(4)));
    const int j = (i + d) % NI;
    v4h o;
#pragma unroll
    for (int r = 0; r < 4; ++r) o[r] = (_Float16)v[r];
    *(v4h*)(A + (16 * i + jl) * LDA * 2 + 16 * ((2 * j + (q >> 1)) ^ (jl & 7)) + 8 * (q & 1)) = o;
    if (d > 0 && d < NI / 2) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 4 * q + r;
        *(_Float16*)(A + (16 * j + row) * LDA * 2 + 16 * ((2 * i + (jl >> 3)) ^ (row & 7)) +
                     2 * (jl & 7)) = o[r];
      }
    }
  };
  for (int step = 0; step < steps; ++step) {
    __syncthreads();  // X is there, B has been read
    v4f acc[D], a[D];
#pragma unroll
    for (int d = 0; d < D; ++d) acc[d] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int kb = grp; kb < mp / 32; kb += GROUPS) {
      const v8h own = x_row(i, kb);
#pragma unroll
      for (int d = 0; d < D; ++d)
        acc[d] = mfma_f16(d == 0 ? own : x_row((i + d) % NI, kb), own, acc[d]);
    }
    if constexpr (GROUPS > 1) {
      v4f* parts = (v4f*)(smem + at.parts);
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (grp > 0) parts[((w - NI) * D + d) * 64 + lane] = acc[d];
      __syncthreads();
#pragma unroll
      for (int d = 0; d < D; ++d)
#pragma unroll
        for (int s = 0; s < GROUPS - 1; ++s)
          if (grp == 0) acc[d] += parts[((s * NI + i) * D + d) * 64 + lane];
    }
    const float sa = kScaleA / (p.cx * p.cx);
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        acc[d][r] *= sa;
        a[d][r] = (float)(_Float16)acc[d][r];
      }
    if (grp == 0) {
#pragma unroll
      for (int d = 0; d < D; ++d) put_a(d, acc[d]);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * q + r == jl) dA[16 * i + jl] = acc[0][r] - a[0][r];
    }
    __syncthreads();  // A is there
#pragma unroll
    for (int d = 0; d < D; ++d) acc[d] = v4f{0.f, 0.f, 0.f, 0.f};
    if (grp == 0) {
#pragma unroll
      for (int kb = 0; kb < NP / 32; ++kb) {
        const v8h own = a_row(i, kb);
#pragma unroll
        for (int d = 0; d < D; ++d)
          acc[d] = mfma_f16(d == 0 ? own : a_row((i + d) % NI, kb), own, acc[d]);
      }
    }
    __syncthreads();  // A has been read
    if (grp == 0) {
      constexpr float fb = kScaleB / kScaleA * kNsB, fc = kScaleB / (kScaleA * kScaleA) * kNsC;
      const float di = dA[16 * i + jl];
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const v4f dj = *(const v4f*)(dA + 16 * ((i + d) % NI) + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const bool diag = d == 0 && 4 * q + r == jl;
          acc[d][r] = fmaf(fc, fmaf(di + dj[r], a[d][r], acc[d][r]),
                           fb * (diag ? a[d][r] + di : a[d][r]));
          if (diag) dB[16 * i + jl] = acc[d][r] - (float)(_Float16)acc[d][r];
        }
        put_a(d, acc[d]);
      }
    }
    __syncthreads();  // B is there
    float own[NI];
#pragma unroll
    for (int it = 0; it < NI; ++it) own[it] = kNsA + dB[16 * it + jl] / kScaleB;
#pragma unroll
    for (int t = 0; t < TJ; t += PAIR) {
      __builtin_amdgcn_sched_barrier(0);
      if (16 * (w + 8 * t) >= mp) break;
      v4f y[PAIR][NI];
#pragma unroll
      for (int b = 0; b < PAIR; ++b)
#pragma unroll
        for (int it = 0; it < NI; ++it) y[b][it] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < NP / 32; ++kb) {
        v8h x[PAIR];
#pragma unroll
        for (int b = 0; b < PAIR; ++b) {
          // (a tile past the last one, which is not kept, reads the last one's columns)
          const int jt = min(w + 8 * (t + b), mp / 16 - 1), c = 2 * jt + ((lane & 3) >> 1);
          v4bf half[2];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int row = 32 * kb + 8 * q + 4 * s + (jl >> 2);
            half[s] = tr16(X + row * mp * 2 + 16 * (c ^ (row & 7)) + 8 * (lane & 1));
          }
          const v2i lo = __builtin_bit_cast(v2i, half[0]), hi = __builtin_bit_cast(v2i, half[1]);
          x[b] = __builtin_bit_cast(v8h, v4i{lo.x, lo.y, hi.x, hi.y});
        }
#pragma unroll
        for (int it = 0; it < NI; ++it) {
          const v8h bf = a_row(it, kb);
#pragma unroll
          for (int b = 0; b < PAIR; ++b) y[b][it] = mfma_f16(x[b], bf, y[b][it]);
        }
      }
#pragma unroll
      for (int b = 0; b < PAIR; ++b) {
#pragma unroll
        for (int it = 0; it < NI; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            st[t + b][it][r] = fmaf(own[it], st[t + b][it][r], y[b][it][r] / kScaleB);
        if (step + 1 < steps && 16 * (w + 8 * (t + b)) < mp) put(t + b);
      }
    }
  }
  // the results leave through X's place as well (which the wave alone read last)
  const float out = 1 / p.cx;  // a power of two
#pragma unroll
  for (int t = 0; t < TJ; ++t)
    if (16 * (w + 8 * t) < mp) {
#pragma unroll
      for (int it = 0; it < NI; ++it) {
        v4u16 o;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          o[r] = __builtin_bit_cast(unsigned short, (__bf16)(st[t][it][r] * out));
        *place(t, it) = o;
      }
    }
  __syncthreads();
  for (int row = row0, c = c0; row < p.R;) {
    const int n = p.C - 8 * c;
    typedef unsigned short h8 __attribute__((ext_vector_type(8), aligned(2)));
    h8 o;
    if (p.wide) {
      o = *(const h8*)(X + row * mp * 2 + 16 * (c ^ (row & 7)));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        o[e] = *(const unsigned short*)(X + (8 * c + e) * mp * 2 + 16 * ((row >> 3) ^ e) +
                                        2 * (row & 7));
    }
    unsigned short* d = p.O + base + (int64_t)row * p.C + 8 * c;
    if (n >= 8) {
      *(h8*)d = o;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) d[e] = o[e];
    }
    row += rows_on, c += on;
    if (c >= units_row) c -= units_row, ++row;
  }
}

struct OSizes {
  int n, m, np, mp, ldn, ldm;
  int64_t sx, sxt, sa;
  // byte offsets in the workspace
  int64_t x, xt[2], lo, a, b, da, db, total;
};

// Rows that lie a multiple of 4096 bytes apart would use few of the memory's channels.
static int o_ld(int x) { return x % 2048 == 0 ? x + 64 : x; }

static OSizes o_sizes(int G, int R, int C) {
  OSizes s;
  s.n = R < C ? R : C, s.m = R < C ? C : R;
  s.np = (s.n + 63) / 64 * 64, s.mp = (s.m + 63) / 64 * 64;
  s.ldn = o_ld(s.np), s.ldm = o_ld(s.mp);
  s.sx = (int64_t)s.np * s.ldm, s.sxt = (int64_t)s.mp * s.ldn, s.sa = (int64_t)s.np * s.ldn;
  int64_t at = (int64_t)G * kNormChunks * 8;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  s.x = take(2 * s.sx * G);
  s.xt[0] = take(2 * s.sxt * G);
  s.xt[1] = take(2 * s.sxt * G);
  s.lo = take(2 * s.sxt * G);
  s.a = take(2 * s.sa * G);
  s.b = take(2 * s.sa * G);
  s.da = take(4ll * s.np * G);
  s.db = take(4ll * s.np * G);
  s.total = at;
  return s;
}

static bool o_taken(int G, int R, int C) {
  return G <= kOrthoMax - 1 && R <= kOrthoMax && C <= kOrthoMax;
}

template <class C, int MODE>
static int o_launch(OParams& p, int cus, int dev, void* stream) {
  constexpr int LDS = C::STAGES * C::STAGE + C::BS * 4;
  static std::mutex mu;
  static bool set[64];
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!set[dev] &&
        hipFuncSetAttribute((const void*)kg_ortho_kernel<C, MODE>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, LDS) != hipSuccess)
      return KG_ERR_HIP;
    set[dev] = true;
  }
  return launch(kg_ortho_kernel<C, MODE>,
                std::min<int64_t>((p.count + 7) / 8 * 8, (int64_t)cus * C::PER_CU), C::THREADS, LDS,
                stream, p);
}

// A product's tiles, by the rounds that each size takes (256: one workgroup on a compute unit, 128:
// two, 64: three; 128's rounds in halves, as a workgroup alone on its compute unit is faster).
// Measured in us, 256 / 128 / 64, for n, m, matrices:
//   A    832, 1024, 3     28 / 12 / 10        B X   832, 1024, 3     45 / 17 / 16
//        2048, 2048, 1    47 / 19 / 24              256, 1024, 32    37 / 23 / 27
//        4096, 4096, 1    94 / 91 / 126             1536, 2048, 4    65 / 73 / 77
//        2048, 7168, 8   332 / 329 / -              2048, 7168, 8   624 / 748 / -
//        4096, 7168, 8   874 / 1060 / -             4096, 7168, 8  1884 / 2750 / -
// Where 256's last round is less than half full, its tiles are quartered instead: 4096, 7168, 8
// has 4 rounds and 64 tiles (A 884 -> 790 us, A A 578 -> 517).
template <int MODE>
static int o_product(OParams& p, int cus, int dev, void* stream) {
  constexpr bool SYM = MODE == kGram || MODE == kPoly;
  auto tiles = [&](int bs) {
    p.tiles_i = (p.np + bs - 1) / bs, p.tiles_j = SYM ? p.tiles_i : (p.mp + bs - 1) / bs;
    const int64_t per = SYM ? (int64_t)p.tiles_i * (p.tiles_i + 1) / 2 : (int64_t)p.tiles_i * p.tiles_j;
    p.per = (int)per, p.count = (int)(per * p.G);
    return per * p.G;
  };
  p.first = p.quarter = 0;
  const int64_t n64 = tiles(64), n128 = tiles(128);
  if (n128 > INT32_MAX / 4 - 4096) return KG_ERR_UNSUPPORTED;
  const int blocks = (MODE == kGram ? p.mp : p.np) / 64;
  if (n64 <= (blocks <= 16 ? 3 : 2) * cus) {
    tiles(64);
    return o_launch<OCfg<64, 3, 4, 3>, MODE>(p, cus, dev, stream);
  }
  const int64_t n256 = tiles(256), rest = n256 % cus, halves = (n128 + cus - 1) / cus;
  if (n256 >= cus && rest > 0 && rest <= cus / 2) {
    p.count = (int)(n256 - rest);
    const int rc = o_launch<OCfg<256, 1>, MODE>(p, cus, dev, stream);
    if (rc != KG_OK) return rc;
    p.first = p.count, p.count = (int)(4 * rest), p.quarter = 1;
    return o_launch<OCfg<128, 2>, MODE>(p, cus, dev, stream);
  }
  if (31 * ((n256 + cus - 1) / cus) <= 10 * halves)
    return o_launch<OCfg<256, 1>, MODE>(p, cus, dev, stream);
  tiles(128);
  return o_launch<OCfg<128, 2>, MODE>(p, cus, dev, stream);
}

// The small kernel's row tiles, 0 where it does not fit or is slower: by columns of U, n > 64, its LDS
// stores meet in the banks, so a few long ones of those are left to the launches (8 of 384 x 128:
// 85 us, 71 there; 8 of 128 x 384: 65 and 72; 300 of 100 x 380: 135 and 495).
static int small_rows(const OParams& p) {
  const int ni = p.n <= 32 ? 2 : p.n <= 64 ? 4 : 8, mp = p.mp;
  const int tiles = ni == 2 ? kSmallTiles<2> : ni == 4 ? kSmallTiles<4> : kSmallTiles<8>;
  if (p.n > 128 || mp > 128 * tiles || small_lds(ni, mp).total > 160 * 1024) return 0;
  return ni == 8 && !p.wide && mp > 256 && p.G <= 16 ? 0 : ni;
}
template <int NI>
static int small_launch(OParams& p, int steps, int dev, void* stream) {
  static std::mutex mu;
  static bool set[64];
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!set[dev] && hipFuncSetAttribute((const void*)kg_ortho_small_kernel<NI>,
                                         hipFuncAttributeMaxDynamicSharedMemorySize,
                                         160 * 1024) != hipSuccess)
      return KG_ERR_HIP;
    set[dev] = true;
  }
  return launch(kg_ortho_small_kernel<NI>, p.G, 512, small_lds(NI, p.mp).total, stream, p, steps);
}

}  // namespace kg

extern "C" int64_t kg_orthogonalize_workspace_bytes(int G, int R, int C) {
  using namespace kg;
  if (G < 0 || R < 0 || C < 0 || !o_taken(G, R, C)) return -1;
  return G == 0 || R == 0 || C == 0 ? 0 : o_sizes(G, R, C).total;
}

extern "C" int kg_orthogonalize(const void* U, void* O, int G, int R, int C, int type, int steps,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  using namespace kg;
  if (type != KG_ROWS_BF16 && type != KG_ROWS_F32) return KG_ERR_DTYPE;
  if (G < 0 || R < 0 || C < 0 || steps < 1 || workspace_bytes < 0) return KG_ERR_SHAPE;
  if (!o_taken(G, R, C) || steps > 64) return KG_ERR_UNSUPPORTED;
  if (G == 0 || R == 0 || C == 0) return KG_OK;
  if (!U || !O || !workspace) return KG_ERR_NULL;
  const size_t e = type == KG_ROWS_BF16 ? 2 : 4;
  if (((uintptr_t)U & (e - 1)) || ((uintptr_t)O & 1) || ((uintptr_t)workspace & 255))
    return KG_ERR_ALIGN;
  const OSizes s = o_sizes(G, R, C);
  if (workspace_bytes < s.total) return KG_ERR_SHAPE;
  const size_t count = (size_t)G * R * C;
  if (ranges_overlap(workspace, s.total, U, count * e) ||
      ranges_overlap(workspace, s.total, O, count * 2))
    return KG_ERR_ALIAS;
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return KG_ERR_HIP;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return KG_ERR_HIP;
  char* ws = (char*)workspace;
  OParams p;
  p.U = U, p.O = (unsigned short*)O, p.parts = (double*)ws;
  p.X = (unsigned short*)(ws + s.x);
  p.LO = (unsigned short*)(ws + s.lo);
  p.A = (unsigned short*)(ws + s.a);
  p.B = (unsigned short*)(ws + s.b);
  p.dA = (float*)(ws + s.da), p.dB = (float*)(ws + s.db);
  p.sx = s.sx, p.sxt = s.sxt, p.sa = s.sa;
  p.cx = (float)ldexp(1.0, (int)lrint(log2((double)s.m) / 2));
  p.G = G, p.R = R, p.C = C, p.n = s.n, p.m = s.m, p.np = s.np, p.mp = s.mp;
  p.ldn = s.ldn, p.ldm = s.ldm;
  p.b16 = type == KG_ROWS_BF16, p.wide = R <= C;
  p.XT = (unsigned short*)(ws + s.xt[0]), p.XN = (unsigned short*)(ws + s.xt[1]);
  // (a workgroup of the small kernel writes its matrix while others may still read theirs)
  const bool apart = G == 1 || (U == O && e == 2) || !ranges_overlap(U, count * e, O, count * 2);
  const int rows = apart ? small_rows(p) : 0;
  if (rows)
    return rows == 2   ? small_launch<2>(p, steps, dev, stream)
           : rows == 4 ? small_launch<4>(p, steps, dev, stream)
                       : small_launch<8>(p, steps, dev, stream);
  const int64_t chunk = norm_chunk((int64_t)R * C);
  p.chunks = (int)(((int64_t)R * C + chunk - 1) / chunk);
  int rc = launch2(kg_ortho_norm_kernel, p.chunks, G, 256, 0, stream, p);
  if (rc == KG_OK)
    rc = launch2(kg_ortho_init_kernel, (int64_t)(s.np / 64) * (s.mp / 64), G, 256, 0, stream, p);
  for (int t = 0; t < steps && rc == KG_OK; ++t) {
    p.low_in = t < steps - 1, p.low_out = t + 1 < steps - 1;
    rc = o_product<kGram>(p, cus, dev, stream);
    if (rc == KG_OK) rc = o_product<kPoly>(p, cus, dev, stream);
    if (rc == KG_OK)
      rc = t < steps - 1 ? o_product<kStep>(p, cus, dev, stream)
                         : o_product<kLast>(p, cus, dev, stream);
    unsigned short* x = p.XT;
    p.XT = p.XN, p.XN = x;
  }
  return rc;
}
