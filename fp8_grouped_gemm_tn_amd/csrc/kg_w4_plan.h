// kg_w4_plan.h -- kg_fprop_w4's arithmetic that needs no GPU, which kernel a call takes among it: plain
// C++, so that it can be checked on the host by itself. (Constant expressions: device code calls
// them too.)
#pragma once
#include <stdint.h>

#include "kgwgrad.h"

namespace kg {

// Of a workgroup's `all` outputs, how many a set of waves has that takes `most` from output m0 on:
// none, if the workgroup's last set lies behind the expert's last output.
constexpr int w_set_outs(int all, int m0, int most) {
  return all <= m0 ? 0 : all - m0 < most ? all - m0 : most;
}

// Streaming: the bytes of W from block kb (64 bytes of codes) of a set's first output to the end of its
// last one, which is all that its waves may read; none behind a wave's last block, and none for
// a set without outputs.
constexpr uint32_t w_codes_left(int outs, int kbytes, int kb, int to) {
  return outs > 0 && kb < to ? (uint32_t)(outs * kbytes - 64 * kb) : 0u;
}

// Streaming: the KB of LDS of a row's tokens, four blocks of 128 channels each; one at least.
constexpr int w_pieces(int nk) { return nk > 4 ? (nk + 3) / 4 : 1; }

// Which kernel and tile, by M_total and G (the experts' sizes are known on the device only), from
// estimates of the time in ns whose figures are measured; every choice is right for every
// distribution of the rows. Measured in us, equal rows, streaming / 32 x 128 / 64 x 128 / 128 x 128 /
// 128 x 256 (/ 256 x 256):
//   e2m1  1 expert, N 4096, K 7168    16 rows 18 / 32 / 39 / 49 / 83, 64 rows 56 / 34 / 39 / 50 / 85
//         8 of N 2048, K 2048         16 rows each 10 / 13 / 15 / 19 / 28 / 43, 128 rows 49 / 24 / 18 / 21 / 30 / 45
//         32 of N 4096, K 7168        4 rows each 101 / 171 / 182 / 208 / 216 / 304,
//                                     256 rows - / 1127 / 695 / 504 / 517 / 397
//   whole numbers, 128 per scale, the last 32 experts
//                                     4 rows each 109 / 231 / 241 / 295 / 287, 256 rows - / 1588 / 940 / 672 / 663
// (The estimates take experts' rows to be uneven, so at equal rows the next larger tile may be taken.)

constexpr int64_t kWLds = 160 * 1024 - 512;  // that a workgroup may ask for

// Streaming: 16 waves on a compute unit, as two workgroups, or as one whose LDS then holds twice the
// rows (8 rows of 8 experts, N 4096, K 7168, e2m1: 42 us as two, 24 as one; 2 rows: 22 and 23). A set
// has 16 outputs where 32 would leave half of the compute units idle (1 row of 1 expert: 6.9 us with
// 16, 8.3 with 32; 2 rows of 8 experts: 34 and 27). 8 waves share them, or 4 where that still fills
// every compute unit (2 rows of 8 experts: 27 us with 8, 22 with 4; of 1 expert: 8.3 and 11).
struct WStream {
  int64_t rows, lds, tokens, scales, ns;  // rows 0: it cannot be used
  int nj, waves, split;
};
constexpr int64_t w_kbytes(int64_t n) { return (n + 1023) / 1024 * 1024; }
constexpr WStream w_stream(int64_t M, int G, int N, int K, int cus, int kind, int group, bool zp) {
  const int64_t live = G < M ? G : M, per_out = K / group, nk = (K + 127) / 128;
  const int sb = kind == KG_W4_E2M1 ? 1 : kind == KG_W4_INT_BF16 ? 2 : 4;
  const int64_t row_bytes = 1024ll * w_pieces((int)nk);
  const int64_t most = M < 16 ? M : 16, uneven = G == 1 ? M : (3 * ((M + G - 1) / G) + 1) / 2;
  const int64_t block_ns = kind == KG_W4_E2M1 ? 400 : group == 32 ? 850 : 600;
  WStream best{};
  best.ns = INT64_MAX;
  for (int waves = 8; waves <= 16; waves += 8) {
    WStream s{};
    s.waves = waves;
    s.nj = live * ((N + 31) / 32) <= cus / 2 ? 1 : 2;
    s.split = s.nj == 2 && live * ((N + 63) / 64) >= 2 * cus ? 4 : 8;
    const int bn = 16 * s.nj * waves / s.split;
    s.scales = w_kbytes(bn * per_out * sb);
    const int64_t rest = s.scales + (zp ? w_kbytes(bn * per_out) : 0);
    const int64_t room = (waves == 8 ? 79 : 159) * 1024 - rest;
    s.rows = room / row_bytes;
    if (s.rows > most) s.rows = most;
    if (s.rows < 1) continue;
    s.tokens = w_kbytes(s.rows * row_bytes);
    if (s.tokens < waves * s.nj * 1024) s.tokens = waves * s.nj * 1024;
    s.lds = s.tokens + rest;
    if (s.lds > kWLds) continue;  // (the waves' sums take the tokens' place in the end, and may be more)
    // a workgroup's start and end, and a wave's blocks
    const int64_t wgs = live * ((N + bn - 1) / bn), slots = (int64_t)cus * 16 / waves;
    const int64_t passes = (uneven + s.rows - 1) / s.rows, blocks = nk / s.split + 1;
    s.ns = 3000 + passes * ((wgs + slots - 1) / slots) *
                      (2600 + blocks * block_ns * (wgs * waves > 8 * cus ? 2 : 1));
    if (s.ns < best.ns) best = s;
  }
  return best;
}

// Tiles (bt rows, bn outputs): rounds over the compute units times the blocks' time. Of several experts
// each has a last tile that is half filled on average.
struct WTile {
  int bt, bn;
  int64_t ns;
};
constexpr WTile w_tile(int64_t M, int G, int N, int K, int cus, int kind) {
  const bool mx = kind == KG_W4_E2M1;
  const struct {
    int bt, bn, ns;  // of 128 channels
  } tiles[] = {{32, 128, mx ? 500 : 780},
               {64, 128, mx ? 630 : 940},
               {128, 128, mx ? 830 : 1270},
               {128, 256, mx ? 1500 : 2200},
               {256, 256, 2350}};
  const int64_t live = G < M ? G : M;
  WTile t{0, 0, INT64_MAX};
  for (int i = 0; i < (mx ? 5 : 4); ++i) {
    int64_t mt = live == 1 ? (M + tiles[i].bt - 1) / tiles[i].bt * 2 : 2 * M / tiles[i].bt + live;
    if (mt < 2 * live) mt = 2 * live;
    const int64_t n = (mt * ((N + tiles[i].bn - 1) / tiles[i].bn) + 1) / 2;
    const int64_t ns = 4500 + (n + cus - 1) / cus * ((K + 127) / 128 * tiles[i].ns + 1000);
    if (ns < t.ns) t = WTile{tiles[i].bt, tiles[i].bn, ns};
  }
  return t;
}
constexpr bool w_streams(const WStream& s, const WTile& t) { return s.rows > 0 && s.ns <= t.ns; }

}  // namespace kg
