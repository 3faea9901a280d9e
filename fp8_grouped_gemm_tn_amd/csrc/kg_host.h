// kg_host.h -- host-side helpers shared by the library's translation units.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kgwgrad.h"

namespace kg {

// Device address of the current device's status word (see kg_status), or null if the
// HIP runtime reports an error. Defined in kglib.hip; looked up once per device.
__attribute__((visibility("hidden"))) int* status_word_address();

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

template <typename T>
struct same {
  using type = T;
};

// Enqueues fn(args...) on grid_x by grid_y workgroups and returns KG_OK, or KG_ERR_HIP if this
// launch was refused (an error that some earlier call left behind is not looked at and stays
// where it is).
template <typename... P>
inline int launch2(void (*fn)(P...), int64_t grid_x, int grid_y, int block, size_t lds,
                   void* stream, typename same<P>::type... args) {
  void* ptrs[] = {(void*)&args...};
  return hipLaunchKernel((const void*)fn, dim3((unsigned)grid_x, (unsigned)grid_y),
                         dim3((unsigned)block), ptrs, lds, (hipStream_t)stream) == hipSuccess
             ? KG_OK
             : KG_ERR_HIP;
}

template <typename... P>
inline int launch(void (*fn)(P...), int64_t grid, int block, size_t lds, void* stream,
                  typename same<P>::type... args) {
  return launch2(fn, grid, 1, block, lds, stream, args...);
}

}  // namespace kg
