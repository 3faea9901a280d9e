// kglib.hip -- the translation unit of the K-grouped kernels (and of the requantiser and
// dgrad, which kgwgrad.hip includes), plus what the library's other translation units
// need of it: the device address of the status word that kg_status reads.
#include "kgwgrad.hip"

#include "kg_host.h"

namespace kg {

int* status_word_address() {
  static std::mutex mu;
  static void* at[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lk(mu);
  if (at[dev] == nullptr &&
      hipGetSymbolAddress(&at[dev], HIP_SYMBOL(kgwgrad_status_word)) != hipSuccess)
    at[dev] = nullptr;
  return (int*)at[dev];
}

}  // namespace kg
