// One token for every row of a serving batch: the short convolution's window advanced, the
// convolution, its SiLU and the scan's recurrence, in one launch.
//
//   v      = silu(b + sum_{j < K} w[K-1-j] u[pos-j])    over the channels of x, B and C
//   delta  = softplus(raw_dt + delta_init)
//   H      <- exp(-delta) H + delta x B^T,   y = H C     (H is P x N, fp32, in place)
//
// The window is the convolution's state: K rows of channels per cache slot, row p mod K
// holding the token at position p.  Every block of a row reads the rows of positions
// pos-1 .. pos-K+1 and the new token; one of them writes row pos mod K, which none reads, so
// the blocks need not wait for one another.
//
// Bound by the state's bytes (2 P N 4 per row and head).  One CTA takes PR rows of one
// head's state; it has its first pieces of the state in flight while it works out the
// PR + 2 N channels it needs (B and C again in every CTA of a group: 2 N K elements out of
// L2 against 8 PR N bytes of state).  With few rows in the batch a head's state is split
// over several CTAs, so that the whole GPU's loads are in flight.
#include <limits.h>
#include <math.h>

#include "layer_device.cuh"
#include "layer_host.cuh"

namespace ssd {
namespace layer {

namespace {

constexpr int kStepThreads = 256;
constexpr int kPieces = 8;  // float4 pieces of the state a thread has in flight

struct StepArgs {
    float* state;
    void* window;
    const void* u;
    const float* raw;
    const void* w;
    const void* b;
    const int* pos;
    const int* slots;
    void* y;
    long long us, C;
    int H, P, N, G, nslots, split, wbf16;
    float delta_init;
};

// The taps of channel c.
template <int K>
__device__ __forceinline__ void taps(const StepArgs& a, long long c, float* w) {
    if constexpr (K == 4) {
        if (!a.wbf16 && (reinterpret_cast<uintptr_t>(a.w) & 15) == 0) {
            Pack<float, 4> v;
            v.load(static_cast<const float*>(a.w) + c * K);
            v.get(w);
            return;
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = param(a.w, c * K + k, a.wbf16);
}

template <typename T, int K>
__global__ void __launch_bounds__(kStepThreads, 4) conv_step_kernel(const StepArgs a) {
    __shared__ float xs[128], bs[128], cs[128];
    const int row = blockIdx.y;
    const int h = blockIdx.x / a.split, part = blockIdx.x - h * a.split;
    const int PR = a.P / a.split, p0 = part * PR;
    const int slot = a.slots ? a.slots[row] : row;
    T* y = static_cast<T*>(a.y) + ((long long)row * a.H + h) * a.P + p0;
    if (slot < 0 || slot >= a.nslots) {  // a padding row of the batch
        for (int i = threadIdx.x; i < PR; i += kStepThreads) st_out(y, i, 0.f);
        return;
    }
    const int n4 = a.N >> 2, total = PR * n4;  // float4 pieces of this CTA
    float4* s4 = reinterpret_cast<float4*>(
        a.state + (((long long)slot * a.H + h) * a.P + p0) * a.N);
    float4 piece[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int e = i * kStepThreads + threadIdx.x;
        if (e < total) piece[i] = s4[e];
    }

    const int Hg = a.H / a.G, g = h / Hg;
    const int pos = a.pos[row];
    const float delta = softplus_f(a.raw[(long long)row * a.H + h] + a.delta_init);
    const float decay = expf(-delta);
    int at[K];  // at[j]: the window's row of position pos - j
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int r = (int)(((long long)pos - j) % K);
        at[j] = r < 0 ? r + K : r;
    }
    T* win = static_cast<T*>(a.window) + (long long)slot * K * a.C;
    const T* u = static_cast<const T*>(a.u) + row * a.us;
    const bool owns_bc = part == 0 && h == g * Hg;
    for (int i = threadIdx.x; i < PR + 2 * a.N; i += kStepThreads) {
        const int j = i - PR;  // B and C channels follow the x channels
        const long long c = j < 0        ? (long long)h * a.P + p0 + i
                            : j < a.N    ? (long long)a.H * a.P + g * a.N + j
                                         : (long long)a.H * a.P + (a.G + g) * a.N + (j - a.N);
        const T tok = u[c];
        float w[K];
        taps<K>(a, c, w);
        float v = w[K - 1] * static_cast<float>(tok);
        if (a.b) v += param(a.b, c, a.wbf16);
#pragma unroll
        for (int k = 1; k < K; ++k)
            v = fmaf(w[K - 1 - k], static_cast<float>(win[at[k] * a.C + c]), v);
        if (j < 0 || owns_bc) win[at[0] * a.C + c] = tok;
        v *= sigmoid_of<float>(v);
        if (j < 0)
            xs[i] = delta * v;
        else if (j < a.N)
            bs[j] = v;
        else
            cs[j - a.N] = v;
    }
    __syncthreads();

    for (int base = 0; base < total; base += kPieces * kStepThreads) {
        if (base > 0)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int e = base + i * kStepThreads + threadIdx.x;
                if (e < total) piece[i] = s4[e];
            }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int e = base + i * kStepThreads + threadIdx.x;
            if (base + i * kStepThreads >= total) break;  // the same for the whole block
            const bool in = e < total;
            const int p = e / n4, n = (e - p * n4) * 4;
            float sum = 0.f;
            if (in) {
                const float xv = xs[p];
                float4 s;
                s.x = fmaf(decay, piece[i].x, xv * bs[n]);
                s.y = fmaf(decay, piece[i].y, xv * bs[n + 1]);
                s.z = fmaf(decay, piece[i].z, xv * bs[n + 2]);
                s.w = fmaf(decay, piece[i].w, xv * bs[n + 3]);
                s4[e] = s;
                sum = s.x * cs[n] + s.y * cs[n + 1] + s.z * cs[n + 2] + s.w * cs[n + 3];
            }
            // the n4 consecutive lanes of one row (n4 divides 32)
            for (int o = n4 >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o, n4);
            if (in && n == 0) st_out(y, p, sum);
        }
    }
}

bool pow2_8_128(int v) { return v >= 8 && v <= 128 && (v & (v - 1)) == 0; }

}  // namespace
}  // namespace layer
}  // namespace ssd

using namespace ssd;
using namespace ssd::layer;

extern "C" {

ssd_status_t ssd_conv_decode_step(const ssd_problem_t* prob, int32_t width, int32_t wdtype,
                                  int32_t nslots, int64_t u_stride, float* state,
                                  void* conv_state, const void* u, const float* raw_dt,
                                  const void* weight, const void* bias, const int32_t* positions,
                                  const int32_t* slots, void* y, void* stream) {
    set_last_launches(0);
    if (!prob) return SSD_ERR_INVALID_ARG;
    const ssd_problem_t& p = *prob;
    if (p.batch < 1 || p.seqlen != 1 || p.nseq != 0 || p.nheads < 1 || p.ngroups < 1 ||
        p.headdim < 1 || p.dstate < 1 || p.nheads % p.ngroups != 0 || !isfinite(p.delta_init) ||
        !dtype_ok(p.dtype) || !dtype_ok(wdtype) || width < 1 || nslots < 1)
        return SSD_ERR_INVALID_ARG;
    if (!pow2_8_128(p.headdim) || !pow2_8_128(p.dstate) || width < 2 || width > 4 ||
        p.batch > 65535 || (long long)p.nheads * p.headdim > (1 << 24) ||
        (long long)p.ngroups * p.dstate > (1 << 22))
        return SSD_ERR_UNSUPPORTED;
    const long long C = (long long)p.nheads * p.headdim + 2LL * p.ngroups * p.dstate;
    if (u_stride < C || (!slots && nslots < p.batch)) return SSD_ERR_INVALID_ARG;
    if (!state || !conv_state || !u || !raw_dt || !weight || !positions || !y)
        return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(p.dtype);
    const size_t we = dtype_size(wdtype);
    if (!aligned_to(state, 16) || !aligned_to(conv_state, e) || !aligned_to(u, e) ||
        !aligned_to(y, e) || !aligned_to(raw_dt, 4) || !aligned_to(weight, we) ||
        !aligned_to(bias, we) || !aligned_to(positions, 4) || !aligned_to(slots, 4))
        return SSD_ERR_ALIGNMENT;
    const Span ss(state, nslots, (long long)p.nheads * p.headdim * p.dstate,
                  (long long)p.nheads * p.headdim * p.dstate, 4);
    const Span sw(conv_state, nslots, width * C, width * C, e);
    const Span su(u, p.batch, u_stride, C, e);
    const Span sy(y, p.batch, p.nheads * p.headdim, p.nheads * p.headdim, e);
    if (ss.overlaps(sw) || ss.overlaps(su) || ss.overlaps(sy) || sw.overlaps(su) ||
        sw.overlaps(sy) || sy.overlaps(su))
        return SSD_ERR_INVALID_ARG;
    StepArgs a = {};
    a.state = state, a.window = conv_state, a.u = u, a.raw = raw_dt, a.w = weight, a.b = bias;
    a.pos = positions, a.slots = slots, a.y = y, a.us = u_stride, a.C = C;
    a.H = p.nheads, a.P = p.headdim, a.N = p.dstate, a.G = p.ngroups;
    a.nslots = nslots, a.wbf16 = wdtype == SSD_DTYPE_BF16, a.delta_init = p.delta_init;
    // CTAs per head: split while the batch leaves SMs with fewer than two CTAs and every
    // thread keeps a piece of the state
    a.split = 1;
    const long long units = p.batch * p.nheads, want = 2LL * sm_count();
    while (units * a.split < want && p.headdim / (2 * a.split) * (p.dstate / 4) >= kStepThreads)
        a.split *= 2;
    const dim3 grid((unsigned)(p.nheads * a.split), (unsigned)p.batch);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("conv_decode_step");
    if (p.dtype == SSD_DTYPE_BF16) {
        if (width == 2)
            conv_step_kernel<__nv_bfloat16, 2><<<grid, kStepThreads, 0, L.stream>>>(a);
        else if (width == 3)
            conv_step_kernel<__nv_bfloat16, 3><<<grid, kStepThreads, 0, L.stream>>>(a);
        else
            conv_step_kernel<__nv_bfloat16, 4><<<grid, kStepThreads, 0, L.stream>>>(a);
    } else {
        if (width == 2)
            conv_step_kernel<float, 2><<<grid, kStepThreads, 0, L.stream>>>(a);
        else if (width == 3)
            conv_step_kernel<float, 3><<<grid, kStepThreads, 0, L.stream>>>(a);
        else
            conv_step_kernel<float, 4><<<grid, kStepThreads, 0, L.stream>>>(a);
    }
    const cudaError_t err = L.end();
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
