// cache_device.cuh -- device building blocks of the paged 8-bit cache.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "cache_internal.h"

namespace alhr {

// First code row of (block, head); rows are below 2^31 (checked on the host), bytes are not.
__device__ __forceinline__ long long block_row(const CacheView& c, int block, int head) {
  return (static_cast<long long>(block) * c.heads + head) << c.bs_log;
}

__device__ __forceinline__ void cache_flag(uint32_t* dev_err, uint32_t bit) {
  if (dev_err) atomicOr(dev_err, bit);
}

// Eight consecutive numbers of type T (an alhr_type) as fp32.
template <int T>
__device__ __forceinline__ void unpack8(const uint4& a, const uint4& b, float (&x)[8]) {
  if constexpr (T == ALHR_TYPE_FP32) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (T == ALHR_TYPE_BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace alhr
