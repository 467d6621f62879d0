// Device helpers of the operators around the scan (convolution, norms): vector loads that
// keep their 16 bytes packed until they are used, the SiLU and its derivative, sums over a
// team of warps, and the reduction of per-block partial sums.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssd_device.cuh"

namespace ssd {
namespace layer {

// VEC consecutive elements as loaded: 16 bytes or less per load instruction.
template <typename T, int VEC>
struct Pack;

template <>
struct Pack<float, 1> {
    float v;
    __device__ __forceinline__ void load(const float* p) { v = *p; }
    __device__ __forceinline__ void zero() { v = 0.f; }
    __device__ __forceinline__ void get(float* f) const { f[0] = v; }
};
template <>
struct Pack<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
};
template <>
struct Pack<float, 8> {
    Pack<float, 4> a, b;
    __device__ __forceinline__ void load(const float* p) { a.load(p), b.load(p + 4); }
    __device__ __forceinline__ void zero() { a.zero(), b.zero(); }
    __device__ __forceinline__ void get(float* f) const { a.get(f), b.get(f + 4); }
};
__device__ __forceinline__ void unpack2(uint32_t w, float* f) {
    f[0] = __uint_as_float(w << 16);
    f[1] = __uint_as_float(w & 0xffff0000u);
}
template <>
struct Pack<__nv_bfloat16, 1> {
    __nv_bfloat16 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *p; }
    __device__ __forceinline__ void zero() { v = __float2bfloat16_rn(0.f); }
    __device__ __forceinline__ void get(float* f) const { f[0] = __bfloat162float(v); }
};
template <>
struct Pack<__nv_bfloat16, 4> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v = *reinterpret_cast<const uint2*>(p);
    }
    __device__ __forceinline__ void zero() { v = make_uint2(0u, 0u); }
    __device__ __forceinline__ void get(float* f) const { unpack2(v.x, f), unpack2(v.y, f + 2); }
};
template <>
struct Pack<__nv_bfloat16, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v = *reinterpret_cast<const uint4*>(p);
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void get(float* f) const {
        unpack2(v.x, f), unpack2(v.y, f + 2), unpack2(v.z, f + 4), unpack2(v.w, f + 6);
    }
};

template <int VEC>
__device__ __forceinline__ void store_vec(float* p, const float* f) {
    if constexpr (VEC == 1) {
        *p = f[0];
    } else {
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&r);
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float* f) {
    if constexpr (VEC == 1) {
        *p = __float2bfloat16_rn(f[0]);
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]),
                                                  pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
}

// Parameters (weight, bias) are float32 or bfloat16, whatever the activations' type.
__device__ __forceinline__ float param(const void* p, long long i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                : static_cast<const float*>(p)[i];
}
__device__ __forceinline__ void set_param(void* p, long long i, float v, int bf16) {
    if (bf16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(p)[i] = v;
}

// sigmoid(v).  float32 tensors take expf and a correctly rounded quotient.  bfloat16
// tensors take the hardware's approximations: their relative error (about 1e-6 at
// |v| = 10) is far below the 2^-9 of the result's rounding, and the two MUFU operations
// an element then costs fit under the memory time.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float v) {
    if constexpr (sizeof(T) == 4)
        return 1.f / (1.f + expf(-v));
    else
        return __fdividef(1.f, 1.f + __expf(-v));
}

}  // namespace layer
}  // namespace ssd
