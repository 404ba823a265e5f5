// sel_dtype.cuh -- element types of the operators around selection: their
// sizes, conversions, and the checks that the 4-bit entry points share.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "sel.h"

namespace sel {

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// The value of a 16-bit pattern of T.
template <typename T>
__device__ __forceinline__ float bits_f32(uint16_t b);
template <>
__device__ __forceinline__ float bits_f32<__half>(uint16_t b) { return __half2float(__ushort_as_half(b)); }
template <>
__device__ __forceinline__ float bits_f32<__nv_bfloat16>(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// One rounding to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Element i of an array of a type that is known at run time only.
__device__ __forceinline__ void store_as(void* p, int dtype, uint64_t i, float x) {
    if (dtype == SEL_F32) static_cast<float*>(p)[i] = x;
    else if (dtype == SEL_F16) static_cast<__half*>(p)[i] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
}

__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
    return v;
}

// Bytes of an element, 0 for an unknown type.
inline uint32_t dtype_bytes(int dtype) {
    return dtype == SEL_F32 ? 4u : dtype == SEL_F16 || dtype == SEL_BF16 ? 2u : 0u;
}

inline bool misaligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

// Shape and types of a 4-bit matrix.
inline sel_status check_w4(int dtype, uint32_t V, uint32_t H, uint32_t group) {
    if (dtype != SEL_F16 && dtype != SEL_BF16) return SEL_EINVAL;
    if (V == 0 || V > SEL_MAX_V || H == 0 || H > SEL_MAX_H) return SEL_EINVAL;
    if (group != 32 && group != 64 && group != 128) return SEL_EUNSUPPORTED;
    return H % group == 0 ? SEL_OK : SEL_EINVAL;
}

}  // namespace sel
