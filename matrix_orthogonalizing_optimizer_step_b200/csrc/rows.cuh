// Row access shared by the embedding and LayerNorm kernels: 8 consecutive
// elements per thread (16 bytes of bf16, two 16-byte accesses of fp32) where
// the pointers, strides and widths allow it, single elements otherwise.
#pragma once
#include <cuda_bf16.h>

#include "muon_internal.h"

namespace muon {

template <typename T>
struct Raw8;  // 8 elements as loaded
template <>
struct Raw8<float> {
    float4 a, b;
};
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
};

__device__ __forceinline__ Raw8<float> ld8(const float* p) {
    return {*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4)};
}
__device__ __forceinline__ Raw8<__nv_bfloat16> ld8(const __nv_bfloat16* p) {
    return {*reinterpret_cast<const uint4*>(p)};
}

__device__ __forceinline__ void to_float8(const Raw8<float>& r, float* v) {
    v[0] = r.a.x, v[1] = r.a.y, v[2] = r.a.z, v[3] = r.a.w;
    v[4] = r.b.x, v[5] = r.b.y, v[6] = r.b.z, v[7] = r.b.w;
}
__device__ __forceinline__ void to_float8(const Raw8<__nv_bfloat16>& r, float* v) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of its fp32
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ void st8(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 16-byte aligned base and rows: every row starts on a 16-byte boundary
inline bool rows_vec_ok(const void* p, long long ld, int dt) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * dtype_size(dt)) % 16 == 0;
}

}  // namespace muon
