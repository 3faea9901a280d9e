// kg_w4_plan.h -- kg_fprop_w4's arithmetic that needs no GPU: plain C++, so that it can be checked on
// the host by itself. (Constant expressions: device code calls them too.)
#pragma once
#include <stdint.h>

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

}  // namespace kg
