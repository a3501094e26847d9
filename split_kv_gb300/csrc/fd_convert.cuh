// fd_convert.cuh -- 16-bit and E4M3 values to and from 32 bits, shared by the
// kernels that write into caches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>
#include <string.h>

namespace fdk {

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return __half22float2(h);
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// two values to the 16-bit type, nearest even
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}

__device__ __forceinline__ float nan_for_inf(float x) {
    return fabsf(x) <= 3.402823466e38f ? x : __uint_as_float(0x7fc00000u);
}

// two values to E4M3, nearest even; NaN stays NaN, and with SPECIAL infinities
// become NaN (the conversion would make them 448)
template <bool SPECIAL>
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    if constexpr (SPECIAL) {
        a = nan_for_inf(a);
        b = nan_for_inf(b);
    }
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace fdk
