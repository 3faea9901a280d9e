// kg_adamw.hip -- one AdamW step over many tensors on gfx950, C ABI kg_adamw_items,
// kg_adamw_table_bytes, kg_adamw_pack, kg_adamw.
//
// Per element, in binary32, every operation rounded by itself (no fused multiply-adds, so
// that the states are the same bits wherever the formula is computed that way):
//   g' = g * gscale
//   m  = m * b1 + g' * (1 - b1)
//   v  = v * b2 + (g' * g') * (1 - b2)
//   p  = p * (1 - lr wd) - (m / (sqrt(v) * (1 - b2^t)^-1/2 + eps)) * (lr / (1 - b1^t))
//
// 8-bit states (KG_ADAMW_8BIT): each 128 consecutive elements of a tensor (the last block may
// be shorter) share two fp32 scales. With amax the block's largest |m|, m is held as e4m3
// codes of m * (448 * fl(1 / amax)) with scale amax * fl(1 / 448); r = sqrt(v) likewise, so
// that a block's v spans 2^36. A nonzero r never becomes zero (its code is at least the
// smallest one): a lost r would divide the next step's m by eps alone. A block whose amax is
// below 2^-118 (where 448 / amax would overflow) is held as zeros. p is updated with the new
// m and v before they are rounded.
//
// Bound by memory: 30 bytes per element with fp32 states (fp32 p and g, bf16 copy), 16.1
// with 8-bit ones (bf16 g). One launch for all tensors: the table holds a descriptor per
// tensor and, for every item of kItem elements, the tensor it belongs to, so a workgroup
// reaches its pointers in two dependent loads however many tensors there are.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

#include "kg_device.h"
#include "kg_host.h"
#include "kgwgrad.h"

namespace kg {

constexpr int kAdamThreads = 256;
constexpr int kAdamPer = 8;  // consecutive elements per thread: 16 threads hold one block
constexpr int kItem = kAdamThreads * kAdamPer;

// A launch holds fewer than 2^32 threads: 3.4e10 elements.
constexpr int64_t kMaxItems = ((int64_t)1 << 32) / kAdamThreads - 1;

struct AdamDesc {
  kg_adamw_tensor t;
  int64_t first_item;
};
static_assert(sizeof(AdamDesc) == 72, "descriptor layout");

template <bool PACKED>
struct DescFor {
  typedef const AdamDesc type;
};
template <>
struct DescFor<true> {
  typedef const AdamDesc& type;
};

struct AdamArgs {
  float b1, c1, b2, c2, eps, lr, wd, decay, rate, rbc2;
  const float* gscale;
  const float* dyn;
};

// Vectors at any address that the element type allows.
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(2)));
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(2)));
typedef int v2i_any __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ float widen(unsigned short x) {
  return __uint_as_float((uint32_t)x << 16);
}
__device__ __forceinline__ unsigned short narrow(float x) {
  return __builtin_bit_cast(unsigned short, (__bf16)x);
}

// Eight consecutive values of type float or bf16; `n` of them exist (8 in all but the last
// thread of a tensor), the others read as zero and are not written.
template <bool BF16>
__device__ __forceinline__ void load8(const void* base, int64_t at, int n, float (&x)[8]) {
  if (n == 8) {
    if constexpr (BF16) {
      const v4i w = *(const v4i_any*)((const unsigned short*)base + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float((uint32_t)w[i] << 16);
        x[2 * i + 1] = __uint_as_float((uint32_t)w[i] & 0xFFFF0000u);
      }
    } else {
      const v4f a = *(const v4f_any*)((const float*)base + at);
      const v4f b = *(const v4f_any*)((const float*)base + at + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = a[i];
        x[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = i >= n ? 0.f
             : BF16 ? widen(((const unsigned short*)base)[at + i])
                    : ((const float*)base)[at + i];
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, int64_t at, int n, const float (&x)[8]) {
  if (n == 8) {
    if constexpr (BF16) {
      v4i w;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (int)((uint32_t)narrow(x[2 * i]) | (uint32_t)narrow(x[2 * i + 1]) << 16);
      *(v4i_any*)((unsigned short*)base + at) = w;
    } else {
      *(v4f_any*)((float*)base + at) = v4f{x[0], x[1], x[2], x[3]};
      *(v4f_any*)((float*)base + at + 4) = v4f{x[4], x[5], x[6], x[7]};
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (BF16)
          ((unsigned short*)base)[at + i] = narrow(x[i]);
        else
          ((float*)base)[at + i] = x[i];
      }
  }
}

// Eight e4m3 codes as the values they stand for, times the block's scale.
__device__ __forceinline__ void load_codes(const void* base, int64_t at, int n, float s,
                                           float (&x)[8]) {
#pragma clang fp contract(off)
  v2i w = {0, 0};
  const unsigned char* p = (const unsigned char*)base + at;
  if (n == 8) {
    w = *(const v2i_any*)p;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) w[i >> 2] |= (int)p[i] << (8 * (i & 3));
  }
  typedef float v2f __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const v2f a = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], false);
    const v2f b = __builtin_amdgcn_cvt_pk_f32_fp8(w[h], true);
    x[4 * h] = a.x * s;
    x[4 * h + 1] = a.y * s;
    x[4 * h + 2] = b.x * s;
    x[4 * h + 3] = b.y * s;
  }
}

// Codes and scale of a block held by 16 neighbouring lanes, 8 values each; UP: what is above
// zero keeps a code above zero. A value that is not finite makes the scale so too (its bit
// pattern is the largest), and with it the whole block: it shows in the next step.
template <bool UP>
__device__ __forceinline__ void store_codes(void* base, float* scales, int64_t at, int n,
                                            const float (&x)[8]) {
#pragma clang fp contract(off)
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    if (i < n) top = b > top ? b : top;
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) {
    const uint32_t u = __shfl_xor(top, d, 64);
    top = u > top ? u : top;
  }
  const float amax = __uint_as_float(top);
  const bool kept = !(amax < 0x1p-118f);
  const float inv = kept ? 448.0f * (1.0f / amax) : 0.0f;
  if (n > 0 && (threadIdx.x & 15) == 0) scales[at >> 7] = kept ? amax * (1.0f / 448.0f) : 0.0f;
  v2i w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = x[4 * h + i] * inv;
      // 2^-9 is the smallest e4m3 value above zero
      if (UP && y[i] > 0.f) y[i] = fmaxf(y[i], 0x1p-9f);
    }
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    w[h] = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], q, true);
  }
  unsigned char* p = (unsigned char*)base + at;
  if (n == 8) {
    *(v2i_any*)p = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (unsigned char)((uint32_t)w[i >> 2] >> (8 * (i & 3)));
  }
}

template <bool PB, bool GB, bool PACKED>
__global__ __launch_bounds__(kAdamThreads) void kg_adamw_kernel(const AdamDesc* table,
                                                                const int32_t* owner, AdamArgs a) {
#pragma clang fp contract(off)
  // fp32 states: the descriptor is read as a whole ahead of the stores, not again after them (160
  // tensors of up to 40000 elements 6.6 -> 6.1 us; eight of 29.4 M elements 1306 us, 5.4 TB/s,
  // either way). 8-bit states lose by it (those eight 670 -> 701 us).
  typename DescFor<PACKED>::type d = table[owner[blockIdx.x]];
  const int64_t at =
      ((int64_t)blockIdx.x - d.first_item) * kItem + threadIdx.x * kAdamPer;
  const int64_t left = d.t.n - at;
  const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
  float lr = a.lr, decay = a.decay, rate = a.rate, rbc2 = a.rbc2;
  if (a.dyn != nullptr) {  // {lr, 1 - b1^t, 1 - b2^t} in device memory
    lr = a.dyn[0];
    decay = 1.0f - lr * a.wd;
    rate = lr / a.dyn[1];
    rbc2 = 1.0f / sqrtf(a.dyn[2]);
  }
  const float gs = a.gscale != nullptr ? *a.gscale : 1.0f;
  float p[8], g[8], m[8], v[8];
  load8<PB>(d.t.p, at, n, p);
  load8<GB>(d.t.g, at, n, g);
  if constexpr (PACKED) {
    const bool in = n > 0;
    load_codes(d.t.m, at, n, in ? d.t.m_scale[at >> 7] : 0.f, m);
    load_codes(d.t.v, at, n, in ? d.t.v_scale[at >> 7] : 0.f, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * v[i];
  } else {
    load8<false>(d.t.m, at, n, m);
    load8<false>(d.t.v, at, n, v);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = a.gscale != nullptr ? g[i] * gs : g[i];
    m[i] = m[i] * a.b1 + gi * a.c1;
    v[i] = v[i] * a.b2 + (gi * gi) * a.c2;
    const float r = sqrtf(v[i]);
    p[i] = p[i] * decay - (m[i] / (r * rbc2 + a.eps)) * rate;
    if constexpr (PACKED) v[i] = r;
  }
  store8<PB>(d.t.p, at, n, p);
  if (d.t.copy != nullptr) store8<true>(d.t.copy, at, n, p);
  if constexpr (PACKED) {
    store_codes<false>(d.t.m, d.t.m_scale, at, n, m);
    store_codes<true>(d.t.v, d.t.v_scale, at, n, v);
  } else {
    store8<false>(d.t.m, at, n, m);
    store8<false>(d.t.v, at, n, v);
  }
}

// A byte range that a step reads or writes.
struct Span {
  uintptr_t a, b;
  bool written;
};

static int by_start(const void* x, const void* y) {
  const uintptr_t a = ((const Span*)x)->a, b = ((const Span*)y)->a;
  return a < b ? -1 : a > b;
}

static int64_t items_of(int64_t n) { return n / kItem + (n % kItem != 0); }

}  // namespace kg

using namespace kg;

extern "C" int64_t kg_adamw_items(const kg_adamw_tensor* tensors, int count) {
  if (count < 0 || (count > 0 && tensors == nullptr)) return -1;
  int64_t items = 0;
  for (int i = 0; i < count; ++i) {
    if (tensors[i].n < 0) return -1;
    items += items_of(tensors[i].n);
    if (items > kMaxItems) return -1;
  }
  return items;
}

extern "C" int64_t kg_adamw_table_bytes(const kg_adamw_tensor* tensors, int count) {
  const int64_t items = kg_adamw_items(tensors, count);
  return items < 0 ? -1 : (int64_t)count * (int64_t)sizeof(AdamDesc) + items * 4;
}

extern "C" int kg_adamw_pack(const kg_adamw_tensor* tensors, int count, int kinds, void* image,
                             int64_t image_bytes) {
  if (kinds & ~(KG_ADAMW_P_BF16 | KG_ADAMW_G_BF16 | KG_ADAMW_8BIT)) return KG_ERR_DTYPE;
  if (count < 0) return KG_ERR_SHAPE;
  if (count == 0) return KG_OK;
  if (tensors == nullptr || image == nullptr) return KG_ERR_NULL;
  const int64_t bytes = kg_adamw_table_bytes(tensors, count);
  if (bytes < 0) {
    for (int i = 0; i < count; ++i)
      if (tensors[i].n < 0) return KG_ERR_SHAPE;
    return KG_ERR_UNSUPPORTED;
  }
  if (image_bytes < bytes) return KG_ERR_SHAPE;
  const int ep = kinds & KG_ADAMW_P_BF16 ? 2 : 4, eg = kinds & KG_ADAMW_G_BF16 ? 2 : 4;
  const bool packed = (kinds & KG_ADAMW_8BIT) != 0;
  const int es = packed ? 1 : 4;
  Span* spans = (Span*)malloc((size_t)count * 7 * sizeof(Span));
  if (spans == nullptr) return KG_ERR_UNSUPPORTED;
  int rc = KG_OK;
  size_t ns = 0;
  AdamDesc* desc = (AdamDesc*)image;
  int32_t* owner = (int32_t*)(desc + count);
  int64_t item = 0;
  for (int i = 0; i < count && rc == KG_OK; ++i) {
    const kg_adamw_tensor& t = tensors[i];
    desc[i].t = t;
    desc[i].first_item = item;
    const int64_t k = items_of(t.n);
    for (int64_t j = 0; j < k; ++j) owner[item + j] = i;
    item += k;
    if (t.n == 0) continue;
    const int64_t nb = t.n / 128 + (t.n % 128 != 0);
    if (t.p == nullptr || t.g == nullptr || t.m == nullptr || t.v == nullptr ||
        (packed && (t.m_scale == nullptr || t.v_scale == nullptr)))
      rc = KG_ERR_NULL;
    else if (((uintptr_t)t.p & (ep - 1)) || ((uintptr_t)t.g & (eg - 1)) ||
             (((uintptr_t)t.m | (uintptr_t)t.v) & (es - 1)) || ((uintptr_t)t.copy & 1) ||
             (packed && (((uintptr_t)t.m_scale | (uintptr_t)t.v_scale) & 3)))
      rc = KG_ERR_ALIGN;
    auto add = [&](const void* p, int64_t n, bool written) {
      if (p != nullptr) spans[ns++] = Span{(uintptr_t)p, (uintptr_t)p + (uintptr_t)n, written};
    };
    add(t.p, t.n * ep, true);
    add(t.g, t.n * eg, false);
    add(t.m, t.n * es, true);
    add(t.v, t.n * es, true);
    add(t.copy, t.n * 2, true);
    if (packed) {
      add(t.m_scale, nb * 4, true);
      add(t.v_scale, nb * 4, true);
    }
  }
  // what a step writes may share no byte with anything else (gradients may with each other)
  if (rc == KG_OK) {
    qsort(spans, ns, sizeof(Span), by_start);
    uintptr_t written = 0, any = 0;  // ends of the ranges so far
    for (size_t i = 0; i < ns; ++i) {
      if (spans[i].a < written || (spans[i].written && spans[i].a < any)) rc = KG_ERR_ALIAS;
      if (spans[i].b > any) any = spans[i].b;
      if (spans[i].written && spans[i].b > written) written = spans[i].b;
    }
  }
  free(spans);
  return rc;
}

extern "C" int kg_adamw(const void* table, int count, int64_t items, int kinds, double lr,
                        double beta1, double beta2, double eps, double weight_decay, int64_t step,
                        const float* gscale, const float* dyn, void* stream) {
  if (kinds & ~(KG_ADAMW_P_BF16 | KG_ADAMW_G_BF16 | KG_ADAMW_8BIT)) return KG_ERR_DTYPE;
  if (count < 0 || items < 0 || (dyn == nullptr && step < 1)) return KG_ERR_SHAPE;
  if (!(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1 && eps >= 0 && lr >= 0 &&
        weight_decay >= 0))
    return KG_ERR_SHAPE;
  if (items > kMaxItems) return KG_ERR_UNSUPPORTED;
  if (count == 0 || items == 0) return KG_OK;
  if (table == nullptr) return KG_ERR_NULL;
  if (((uintptr_t)table & 7) || (((uintptr_t)gscale | (uintptr_t)dyn) & 3)) return KG_ERR_ALIGN;
  AdamArgs a;
  a.b1 = (float)beta1;
  a.c1 = (float)(1 - beta1);
  a.b2 = (float)beta2;
  a.c2 = (float)(1 - beta2);
  a.eps = (float)eps;
  a.lr = (float)lr;
  a.wd = (float)weight_decay;
  a.decay = (float)(1 - lr * weight_decay);
  const double t = (double)step;
  a.rate = dyn != nullptr ? 0.f : (float)(lr / (1 - pow(beta1, t)));
  a.rbc2 = dyn != nullptr ? 0.f : (float)(1 / sqrt(1 - pow(beta2, t)));
  a.gscale = gscale;
  a.dyn = dyn;
  const AdamDesc* desc = (const AdamDesc*)table;
  const int32_t* owner = (const int32_t*)(desc + count);
  using Fn = void (*)(const AdamDesc*, const int32_t*, AdamArgs);
  static const Fn fns[8] = {
      kg_adamw_kernel<false, false, false>, kg_adamw_kernel<true, false, false>,
      kg_adamw_kernel<false, true, false>,  kg_adamw_kernel<true, true, false>,
      kg_adamw_kernel<false, false, true>,  kg_adamw_kernel<true, false, true>,
      kg_adamw_kernel<false, true, true>,   kg_adamw_kernel<true, true, true>};
  return launch(fns[kinds], items, kAdamThreads, 0, stream, desc, owner, a);
}
