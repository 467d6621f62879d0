// Device helpers of the operators around the scan (convolution, norms): vector loads that
// keep their 16 bytes packed until they are used, bounded waits, parameters of either type, the
// sigmoid, and pairs of channels in one register pair.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "layer_ring.cuh"
#include "ssd_device.cuh"
#include "tc_ptx.cuh"

namespace ssd {
namespace layer {

// VEC consecutive elements as loaded: 16 bytes or less per load instruction.  stream(): from
// global memory that will not be read again.
template <typename T, int VEC>
struct Pack;

template <>
struct Pack<float, 1> {
    float v;
    __device__ __forceinline__ void load(const float* p) { v = *p; }
    __device__ __forceinline__ void stream(const float* p) { v = __ldcs(p); }
    __device__ __forceinline__ void zero() { v = 0.f; }
    __device__ __forceinline__ void get(float* f) const { f[0] = v; }
};
template <>
struct Pack<float, 4> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void stream(const float* p) {
        v = __ldcs(reinterpret_cast<const float4*>(p));
    }
    __device__ __forceinline__ void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    }
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
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
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
    } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint32_t*>(p) = pack2(f[0], f[1]);
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]),
                                                  pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
}

template <>
struct Pack<float, 2> {
    float2 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float2*>(p); }
    __device__ __forceinline__ void stream(const float* p) {
        v = __ldcs(reinterpret_cast<const float2*>(p));
    }
    __device__ __forceinline__ void zero() { v = make_float2(0.f, 0.f); }
    __device__ __forceinline__ void get(float* f) const { f[0] = v.x, f[1] = v.y; }
};
template <>
struct Pack<__nv_bfloat16, 2> {
    uint32_t v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        v = *reinterpret_cast<const uint32_t*>(p);
    }
    __device__ __forceinline__ void zero() { v = 0u; }
    __device__ __forceinline__ void get(float* f) const { unpack2(v, f); }
};

// Waits for phase `parity` of a copy's barrier.  The wait is bounded (2 s); one that runs out
// records SSD_ERR_TIMEOUT and lets every later wait of the thread pass at once, so that a lost
// copy ends in a status and wrong values, not in a hang.  The thread that issues the copies then
// issues no more, and before it leaves waits once more, bounded again, for those on their way:
// they may be late, and must not land in shared memory that by then is another block's.
static __device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, int* status) {
    if (tc::mbar_wait(bar, parity)) return false;
    atomicCAS(status, 0, (int)SSD_ERR_TIMEOUT);
    return true;
}
// `left`: the copies that the thread has still to issue, 0 or more; where a wait has run out, minus
// one and those (so that the one register says both).
__device__ __forceinline__ void wait_copy(uint64_t* bar, uint32_t parity, int* status, int& left) {
    if (!tc::mbar_try_wait(bar, parity) && left >= 0 && wait_long(bar, parity, status)) left = ~left;
}
// After the last use of a ring, in the thread that issues its copies: nothing is on its way any more
// unless a wait ran out.  idle: places gone over without a copy for them, at the end.
__device__ __forceinline__ void drain_ring(uint64_t* full, int places, int stage, uint32_t parity,
                                           int left, int idle = 0) {
    if (left < 0)
        for (int s = 0; s < places; ++s)
            tc::mbar_wait(&full[s], landed_parity(s, places, stage, parity, ~left + idle));
}

// Parameters (weight, bias) are float32 or bfloat16, whatever the activations' type.
__device__ __forceinline__ float param(const void* p, long long i, int bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                : static_cast<const float*>(p)[i];
}
// Parameters i .. i + VEC; p + i need not be aligned for a vector, which is looked at here.
template <int VEC>
__device__ __forceinline__ void params(const void* p, long long i, int bf16, float* f) {
    if constexpr (VEC >= 4) {
        if (!bf16 && ((reinterpret_cast<uintptr_t>(p) + 4 * i) & 15) == 0) {
#pragma unroll
            for (int e = 0; e < VEC; e += 4) {
                Pack<float, 4> v;
                v.load(static_cast<const float*>(p) + i + e);
                v.get(f + e);
            }
            return;
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = param(p, i + e, bf16);
}
__device__ __forceinline__ void set_param(void* p, long long i, float v, int bf16) {
    if (bf16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<float*>(p)[i] = v;
}

// 1 / (1 + 2^(-v log2 e)).  float32 tensors take expf and a correctly rounded quotient.
// bfloat16 tensors take the hardware's base-2 exponential and reciprocal, denormals flushed
// (the sum with 1 drops them in any case): their relative error (about 1e-6 at |v| = 10, 2e-7 up
// to 4) is far below the 2^-9 of the bf16 results' rounding.  What such a call keeps in float32 (the
// step's state, the gated norm's 1 / deviation, the weights' gradients) has it too, from inputs
// that were rounded to 2^-9.  An element then costs two operations of the special function unit and
// three of the others.  Both ends come out right: 2^inf = inf,
// 1 / inf = 0.
template <typename T>
__device__ __forceinline__ float sigmoid_of(float v) {
    if constexpr (sizeof(T) == 4) {
        return 1.f / (1.f + expf(-v));
    } else {
        float e, r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.44269504f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
        return r;
    }
}

// Two channels in one 64-bit register pair: one instruction does both, which halves the issue
// slots of the multiply-adds.  A single channel is a plain float.
struct F2 {
    unsigned long long v;
};
template <int VEC>
struct Lanes {
    using V = F2;
    static constexpr int N = VEC / 2;
};
template <>
struct Lanes<1> {
    using V = float;
    static constexpr int N = 1;
};
__device__ __forceinline__ F2 join(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(F2 x, float* f) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f[0]), "=f"(f[1]) : "l"(x.v));
}
__device__ __forceinline__ F2 fma_(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul_(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add_(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 sub_(F2 a, F2 b) {
    F2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ float sub_(float a, float b) { return a - b; }
__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float mul_(float a, float b) { return a * b; }
__device__ __forceinline__ float add_(float a, float b) { return a + b; }
template <typename V>
__device__ __forceinline__ V both(float x);
template <>
__device__ __forceinline__ F2 both<F2>(float x) { return join(x, x); }
template <>
__device__ __forceinline__ float both<float>(float x) { return x; }
template <int VEC>
__device__ __forceinline__ void to_lanes(const float* f, typename Lanes<VEC>::V* v) {
    if constexpr (VEC == 1)
        v[0] = f[0];
    else
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) v[i] = join(f[2 * i], f[2 * i + 1]);
}
template <int VEC>
__device__ __forceinline__ void from_lanes(const typename Lanes<VEC>::V* v, float* f) {
    if constexpr (VEC == 1)
        f[0] = v[0];
    else
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) split(v[i], f + 2 * i);
}
template <typename T>
__device__ __forceinline__ F2 sigmoid_lanes(F2 v) {
    float f[2];
    split(v, f);
    return join(sigmoid_of<T>(f[0]), sigmoid_of<T>(f[1]));
}
template <typename T>
__device__ __forceinline__ float sigmoid_lanes(float v) {
    return sigmoid_of<T>(v);
}
// The derivative of v s, s = sigmoid(v), from s and p = v s: s + p (1 - s).  1 - s is exact from
// s = 1/2 on and 0 where s = 1, so that nothing cancels at large v, where s + p or p - p s would
// lose s beside p.
template <typename V>
__device__ __forceinline__ V silu_slope(V s, V p) {
    return fma_(p, sub_(both<V>(1.f), s), s);
}

}  // namespace layer
}  // namespace ssd
