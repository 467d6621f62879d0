// One token of linear attention for every row of a serving batch, over cache slots:
//     S <- a S + v k^T,   o = scale S q       (S is P x N, fp32, in place)
//
// Bound by the state's bytes, 2 P N 4 a row and head.  A block takes a run of rows p of one head's
// state, which lie next to one another in memory, and every thread has all its pieces of them in
// flight before it waits for the first; the lanes of a row add up its product with q.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "layer_device.cuh"
#include "layer_host.cuh"

namespace ssd {
namespace layer {

namespace {

constexpr int kThreads = 128;
constexpr int kPieces = 8;  // of a thread in flight

struct StepArgs {
    float* state;
    const void *q, *k, *v;
    void* o;
    const float* ld;
    const int* slots;
    long long qs, ks, vs, os;
    int H, r, P, N, nslots;
    int lanes;   // of a row: a power of two
    int rows;    // of the state a block takes
    float scale;
};

// VEC: elements of a piece; N is a multiple of it.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 6) attn_step_kernel(const StepArgs a) {
    const int row = blockIdx.z, h = blockIdx.y;
    const int slot = a.slots ? a.slots[row] : row;
    const int p0 = blockIdx.x * a.rows, np = min(a.rows, a.P - p0);
    T* o = static_cast<T*>(a.o) + row * a.os + (long long)h * a.P + p0;
    if (slot < 0 || slot >= a.nslots) {  // a padding row of the batch
        for (int i = threadIdx.x; i < np; i += kThreads) st_out(o, i, 0.f);
        return;
    }
    const int lane = threadIdx.x & (a.lanes - 1), first = threadIdx.x / a.lanes;
    const int step = kThreads / a.lanes, units = a.N / VEC;
    float* s = a.state + (((long long)slot * a.H + h) * a.P + p0) * a.N;
    const T* q = static_cast<const T*>(a.q) + row * a.qs + (long long)h * a.N;
    const T* k = static_cast<const T*>(a.k) + row * a.ks + (long long)(h / a.r) * a.N;
    const T* v = static_cast<const T*>(a.v) + row * a.vs + (long long)(h / a.r) * a.P + p0;
    const float decay = expf(a.ld[h]);
    if constexpr (VEC == 4) {  // a row fits its lanes
        const bool in = lane < units;
        for (int b = 0; b < np; b += kPieces * step) {
            float4 piece[kPieces];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = b + i * step + first;
                if (in && p < np) piece[i] = *reinterpret_cast<const float4*>(s + (long long)p * a.N + 4 * lane);
            }
            float qq[4] = {}, kk[4] = {};
            if (in)
#pragma unroll
                for (int c = 0; c < 4; ++c) qq[c] = static_cast<float>(q[4 * lane + c]), kk[c] = static_cast<float>(k[4 * lane + c]);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int p = b + i * step + first;
                float sum = 0.f;
                if (in && p < np) {
                    const float vv = static_cast<float>(v[p]);
                    float4 w;
                    w.x = fmaf(decay, piece[i].x, vv * kk[0]);
                    w.y = fmaf(decay, piece[i].y, vv * kk[1]);
                    w.z = fmaf(decay, piece[i].z, vv * kk[2]);
                    w.w = fmaf(decay, piece[i].w, vv * kk[3]);
                    *reinterpret_cast<float4*>(s + (long long)p * a.N + 4 * lane) = w;
                    sum = (w.x * qq[0] + w.y * qq[1]) + (w.z * qq[2] + w.w * qq[3]);
                }
                for (int m = a.lanes >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
                if (lane == 0 && p < np) st_out(o, p, sum * a.scale);
            }
        }
    } else {
        for (int b = 0; b < np; b += step) {  // all lanes of a warp go round as often
            const int p = b + first;
            float sum = 0.f;
            if (p < np) {
                const float vv = static_cast<float>(v[p]);
                for (int n = lane; n < a.N; n += a.lanes) {
                    const float w = fmaf(decay, s[(long long)p * a.N + n], vv * static_cast<float>(k[n]));
                    s[(long long)p * a.N + n] = w;
                    sum = fmaf(w, static_cast<float>(q[n]), sum);
                }
            }
            for (int m = a.lanes >> 1; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
            if (lane == 0 && p < np) st_out(o, p, sum * a.scale);
        }
    }
}

}  // namespace
}  // namespace layer
}  // namespace ssd

using namespace ssd;
using namespace ssd::layer;

extern "C" ssd_status_t ssd_linear_attention_step(const ssd_linattn_t* prob, int32_t nslots, float* state,
                                                  const void* q, const void* k, const void* v,
                                                  const float* log_decay, const int32_t* slots, void* o,
                                                  void* stream) {
    set_last_launches(0);
    if (!prob) return SSD_ERR_INVALID_ARG;
    const ssd_linattn_t& p = *prob;
    if (p.batch < 1 || p.seqlen != 1 || p.nseq != 0 || p.nheads < 1 || p.ngroups < 1 || p.headdim < 1 ||
        p.dstate < 1 || p.nheads % p.ngroups != 0 || !isfinite(p.scale) || !dtype_ok(p.dtype) || nslots < 1)
        return SSD_ERR_INVALID_ARG;
    if (p.headdim > 128 || p.dstate > 128 || p.batch > 65535 || p.nheads > 65535) return SSD_ERR_UNSUPPORTED;
    const long long B = p.batch, H = p.nheads, G = p.ngroups, P = p.headdim, N = p.dstate;
    if (p.q_stride < H * N || p.k_stride < G * N || p.v_stride < G * P || p.o_stride < H * P ||
        (!slots && nslots < B))
        return SSD_ERR_INVALID_ARG;
    if (!state || !q || !k || !v || !log_decay || !o) return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(p.dtype);
    if (!aligned_to(state, 16) || !aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) ||
        !aligned_to(o, e) || !aligned_to(log_decay, 4) || !aligned_to(slots, 4))
        return SSD_ERR_ALIGNMENT;
    if (clash({Span(state, nslots * H * P * N, 4), Span(o, B, p.o_stride, H * P, e)},
              {Span(q, B, p.q_stride, H * N, e), Span(k, B, p.k_stride, G * N, e),
               Span(v, B, p.v_stride, G * P, e), Span(log_decay, H, 4), Span(slots, slots ? B : 0, 4)}))
        return SSD_ERR_INVALID_ARG;
    StepArgs a = {};
    a.state = state, a.q = q, a.k = k, a.v = v, a.o = o, a.ld = log_decay, a.slots = slots;
    a.qs = p.q_stride, a.ks = p.k_stride, a.vs = p.v_stride, a.os = p.o_stride;
    a.H = p.nheads, a.r = (int)(H / G), a.P = p.headdim, a.N = p.dstate, a.nslots = nslots;
    a.scale = p.scale;
    const int vec = N % 4 == 0 ? 4 : 1;
    a.lanes = 1;
    while (a.lanes < 32 && a.lanes * vec < N) a.lanes *= 2;
    // rows of the state a block takes: as many as its threads have in flight at once, halved while the
    // batch leaves SMs with fewer than two blocks and each thread keeps a piece
    a.rows = std::min((int)P, std::max(1, kPieces * kThreads / a.lanes));
    while (B * H * ((P + a.rows - 1) / a.rows) < 2LL * sm_count() && a.rows * a.lanes >= 2 * kThreads)
        a.rows = (a.rows + 1) / 2;
    const dim3 grid((unsigned)((P + a.rows - 1) / a.rows), (unsigned)H, (unsigned)B);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("linattn_step");
    if (p.dtype == SSD_DTYPE_BF16) {
        if (vec == 4)
            attn_step_kernel<__nv_bfloat16, 4><<<grid, kThreads, 0, L.stream>>>(a);
        else
            attn_step_kernel<__nv_bfloat16, 1><<<grid, kThreads, 0, L.stream>>>(a);
    } else {
        if (vec == 4)
            attn_step_kernel<float, 4><<<grid, kThreads, 0, L.stream>>>(a);
        else
            attn_step_kernel<float, 1><<<grid, kThreads, 0, L.stream>>>(a);
    }
    const cudaError_t err = L.end();
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}
