// kg_rows.h -- where each expert's rows are, for the kernels whose rows are grouped by expert.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kg_sched.h"

namespace kg {

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

// Inclusive scans over a wave by DPP: within rows of 16 lanes, then from row to row. (Shuffles through
// LDS take 1 us of a short kernel's time.)
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_0(int x) {
  return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ void scan_step(int64_t* sum, int* count) {
  const uint32_t lo = (uint32_t)dpp_or_0<CTRL, ROWS>((int)(uint32_t)*sum);
  const int hi = dpp_or_0<CTRL, ROWS>((int)(*sum >> 32));
  *sum += (int64_t)(((uint64_t)(uint32_t)hi << 32) | lo);
  *count += dpp_or_0<CTRL, ROWS>(*count);
}
__device__ __forceinline__ int64_t read_lane(int64_t x, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// The expert with rows that `nth` others with rows come before, its first row and their number, by
// a scan of ms in every wave (a lane holds consecutive experts). rows = 0: there is none.
// Returns false if ms is inconsistent.
__device__ __forceinline__ bool find_rows(const int32_t* ms, int G, int64_t M_total, int nth,
                                          int* g, int64_t* row0, int* rows) {
  const int lane = threadIdx.x & 63, per = (G + 63) / 64;
  const int e0 = lane * per, e1 = min(G, e0 + per);
  int64_t sum = 0;
  int live = 0, neg = 0;
  for (int e = e0; e < e1; ++e) {
    const int v = ms[e];
    neg |= v < 0;
    sum += v;
    live += v > 0;
  }
  int64_t to = sum;  // rows and experts up to this lane's last one
  int live_to = live;
  scan_step<0x111, 0xF>(&to, &live_to);  // row_shr: 1, 2, 4, 8
  scan_step<0x112, 0xF>(&to, &live_to);
  scan_step<0x114, 0xF>(&to, &live_to);
  scan_step<0x118, 0xF>(&to, &live_to);
  scan_step<0x142, 0xA>(&to, &live_to);  // row_bcast: 15, 31
  scan_step<0x143, 0xC>(&to, &live_to);
  const bool ok = __ballot(neg != 0) == 0 && read_lane(to, 63) == M_total;
  const uint64_t has = __ballot(live_to > nth);  // the first such lane has the expert
  *rows = 0;
  *g = 0;
  *row0 = 0;
  if (!ok || has == 0) return ok;
  const int owner = __builtin_ctzll(has);
  int64_t at = to - sum;
  int mine = (int)sum, mg = e0;
  if (per > 1) {
    int left = nth - (live_to - live);
    mine = 0;
    for (int e = e0; e < e1 && lane == owner; ++e) {
      const int v = ms[e];
      if (v > 0 && left-- == 0) {
        mine = v;
        mg = e;
        break;
      }
      at += v;
    }
  }
  *row0 = read_lane(at, owner);
  *rows = __builtin_amdgcn_readlane(mine, owner);
  *g = __builtin_amdgcn_readlane(mg, owner);
  return true;
}

}  // namespace kg
