// elem.cuh -- 16-byte vectors of the element types the row operators take
// (bf16, fp16, fp32), widened to fp32 and rounded back to nearest even.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/moe.h"

namespace moe {

template <int kDtype>
struct Elem {
  static constexpr int kBytes = kDtype == MOE_T_FP32 ? 4 : 2;
  static constexpr int kPerVec = 16 / kBytes;   // elements of a 16-byte vector

  __device__ static __forceinline__ void unpack(const uint4& v, float (&f)[kPerVec]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (kDtype == MOE_T_FP32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = __uint_as_float(w[q]);
    } else if constexpr (kDtype == MOE_T_BF16) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[2 * q] = __uint_as_float(w[q] << 16);
        f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[q]));
        f[2 * q] = p.x;
        f[2 * q + 1] = p.y;
      }
    }
  }

  __device__ static __forceinline__ uint4 pack(const float (&f)[kPerVec]) {
    uint32_t w[4];
    if constexpr (kDtype == MOE_T_FP32) {
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = __float_as_uint(f[q]);
    } else if constexpr (kDtype == MOE_T_BF16) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
        w[q] = *reinterpret_cast<uint32_t*>(&b);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        __half2 b = __floats2half2_rn(f[2 * q], f[2 * q + 1]);
        w[q] = *reinterpret_cast<uint32_t*>(&b);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

}  // namespace moe
