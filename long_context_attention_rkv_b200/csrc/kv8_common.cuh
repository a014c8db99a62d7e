// Code conversions of the 8-bit block cache, shared by its store and decode kernels.
#pragma once

#include <cuda_fp8.h>

#include "device_common.cuh"

namespace rkv {
namespace kv8 {

template <bool kE4M3>
__device__ __forceinline__ constexpr float qmax()
{
    return kE4M3 ? 448.0f : 127.0f;
}

// The smallest scale of a nonzero block: keeps 1 / scale and products with it well inside fp32.
constexpr float kMinScale = 0x1p-64f;

// Code of a value already divided by the scale: nearest, ties to even, at most qmax in magnitude.
template <bool kE4M3>
__device__ __forceinline__ uint32_t encode(float t)
{
    if constexpr (kE4M3)
        return __nv_cvt_float_to_fp8(t, __NV_SATFINITE, __NV_E4M3);
    else
        return static_cast<uint32_t>(max(-127, min(127, __float2int_rn(t)))) & 0xffu;
}

template <bool kE4M3>
__device__ __forceinline__ float decode(uint32_t c)
{
    if constexpr (kE4M3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c), __NV_E4M3);
        return __half2float(__half(h));
    } else {
        return static_cast<float>(static_cast<int8_t>(c));
    }
}

}  // namespace kv8
}  // namespace rkv
