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
// Bound by the state's bytes (2 P N 4 per row and head).  With a large batch a CTA takes several
// heads of one group, one after the other: the B and C channels (2 N of them, against P of x a
// head) are then worked out once for all.  With few rows in the batch a head's state is split
// over several CTAs, so that the whole GPU's loads are in flight.  A CTA has its first pieces
// of the state on their way while it works out its channels.
//
// GB300, 80 heads x 64 x 128, bf16, K = 4: 128 rows (4 of them padding) 112 us (86 % of the
// measured copy rate on the state's bytes of the 124 rows), one row 6.2 us, the host's time to
// launch it (4.3 us a launch in a replayed CUDA graph).
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
    int H, P, N, G, nslots, wbf16;
    int split, heads;  // CTAs a head, heads a CTA (one of the two is 1)
    int log_n4;        // log2 of the float4 pieces in a row of the state
    float delta_init;
};
constexpr int kMostHeads = 8;

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

// The sums over the 2^LOG lanes of a row of kPieces values a lane, in LOG steps that halve the
// values as long as there are several: lane bits from the top choose which value a lane goes on
// with.  Returns this lane's sum, of the value `*which`; the lanes whose low bits (below those
// used for the choice) are zero between them have one each.
template <int LOG>
__device__ __forceinline__ float halving_sum(float (&v)[kPieces], int lane, int* which) {
    int n = kPieces, id = 0;
#pragma unroll
    for (int step = 0; step < LOG; ++step) {
        const int o = 1 << (LOG - 1 - step);
        if (n > 1) {
            n >>= 1;
            const bool up = lane & o;
            id = id * 2 + up;
#pragma unroll
            for (int i = 0; i < kPieces / 2; ++i)
                if (i < n) {
                    const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    *which = id;
    return v[0];
}

// One head's rows p0 .. p0 + PR of the state: H <- decay H + xs B^T in place, y = H C.
// LOG: log2 of the pieces in a row, 3 or more (0: fewer, known at run time).
template <typename T, int LOG>
__device__ __forceinline__ void step_rows(float4* s4, float4 (&piece)[kPieces], int total, int log_n4,
                                          float decay, const float* xs, const float* bs,
                                          const float* cs, T* y) {
    const int ln4 = LOG ? LOG : log_n4, n4 = 1 << ln4;
    for (int base = 0; base < total; base += kPieces * kStepThreads) {
        if (base > 0)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int e = base + i * kStepThreads + threadIdx.x;
                if (e < total) piece[i] = s4[e];
            }
        // a thread's pieces lie in the same columns (n4 divides the block's threads)
        const int n = (threadIdx.x & (n4 - 1)) * 4;
        const float4 bv = *reinterpret_cast<const float4*>(bs + n);
        const float4 cv = *reinterpret_cast<const float4*>(cs + n);
        float sum[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int e = base + i * kStepThreads + threadIdx.x;
            sum[i] = 0.f;
            if (e < total) {
                const float xv = xs[e >> ln4];
                float4 s;
                s.x = fmaf(decay, piece[i].x, xv * bv.x);
                s.y = fmaf(decay, piece[i].y, xv * bv.y);
                s.z = fmaf(decay, piece[i].z, xv * bv.z);
                s.w = fmaf(decay, piece[i].w, xv * bv.w);
                s4[e] = s;
                sum[i] = (s.x * cv.x + s.y * cv.y) + (s.z * cv.z + s.w * cv.w);
            }
        }
        if constexpr (LOG >= 3) {
            int which;
            const float t = halving_sum<LOG>(sum, threadIdx.x & (n4 - 1), &which);
            const int e = base + which * kStepThreads + threadIdx.x;
            if ((threadIdx.x & ((n4 >> 3) - 1)) == 0 && e < total) st_out(y, e >> ln4, t);
        } else {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                for (int o = n4 >> 1; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o, n4);
                const int e = base + i * kStepThreads + threadIdx.x;
                if (n == 0 && e < total) st_out(y, e >> ln4, sum[i]);
            }
        }
    }
}

template <typename T, int K>
__global__ void __launch_bounds__(kStepThreads, 3) conv_step_kernel(const StepArgs a) {
    __shared__ __align__(16) float xs[kMostHeads][128], bs[128], cs[128];
    __shared__ float decays[kMostHeads];
    const int row = blockIdx.y;
    const int unit = blockIdx.x / a.split, part = blockIdx.x - unit * a.split;
    const int h0 = unit * a.heads;
    const int PR = a.P / a.split, p0 = part * PR;
    const int slot = a.slots ? a.slots[row] : row;
    T* y = static_cast<T*>(a.y) + ((long long)row * a.H + h0) * a.P + p0;
    if (slot < 0 || slot >= a.nslots) {  // a padding row of the batch
        for (int i = threadIdx.x; i < PR * a.heads; i += kStepThreads) st_out(y, i, 0.f);
        return;
    }
    const int total = PR << a.log_n4;  // float4 pieces of a head here
    float4* s4 =
        reinterpret_cast<float4*>(a.state + (((long long)slot * a.H + h0) * a.P + p0) * a.N);
    float4 piece[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int e = i * kStepThreads + threadIdx.x;
        if (e < total) piece[i] = s4[e];
    }

    const int g = h0 / (a.H / a.G);
    const int pos = a.pos[row];
    const float* raw = a.raw + (long long)row * a.H + h0;
    if (threadIdx.x >= kStepThreads - a.heads) {  // the threads with the fewest channels
        const int h = kStepThreads - 1 - threadIdx.x;
        decays[h] = expf(-softplus_f(raw[h] + a.delta_init));
    }
    int at[K];  // at[j]: the window's row of position pos - j
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const int r = (int)(((long long)pos - j) % K);
        at[j] = r < 0 ? r + K : r;
    }
    T* win = static_cast<T*>(a.window) + (long long)slot * K * a.C;
    const T* u = static_cast<const T*>(a.u) + row * a.us;
    const bool owns_bc = part == 0 && h0 == g * (a.H / a.G);
    const int nx = PR * a.heads;  // x channels (several heads: whole ones, next to one another)
    for (int i = threadIdx.x; i < nx + 2 * a.N; i += kStepThreads) {
        const int j = i - nx;  // B and C channels follow the x channels
        const long long c = j < 0     ? (long long)h0 * a.P + p0 + i
                            : j < a.N ? (long long)a.H * a.P + g * a.N + j
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
        v *= sigmoid_of<T>(v);
        if (j < 0)
            xs[0][i] = v * softplus_f(raw[i / PR] + a.delta_init);  // PR channels a head
        else if (j < a.N)
            bs[j] = v;
        else
            cs[j - a.N] = v;
    }
    __syncthreads();
    for (int h = 0; h < a.heads; ++h) {
        if (h > 0)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int e = i * kStepThreads + threadIdx.x;
                if (e < total) piece[i] = s4[e];
            }
        const float* x = &xs[0][0] + h * PR;
        if (a.log_n4 == 5)
            step_rows<T, 5>(s4, piece, total, 5, decays[h], x, bs, cs, y);
        else if (a.log_n4 == 4)
            step_rows<T, 4>(s4, piece, total, 4, decays[h], x, bs, cs, y);
        else
            step_rows<T, 0>(s4, piece, total, a.log_n4, decays[h], x, bs, cs, y);
        s4 += (long long)a.P << a.log_n4;
        y += a.P;
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
    const long long hp = (long long)p.nheads * p.headdim;
    if (clash({Span(state, nslots * hp * p.dstate, 4), Span(conv_state, nslots * width * C, e),
               Span(y, p.batch * hp, e)},
              {Span(u, p.batch, u_stride, C, e), Span(raw_dt, p.batch * (long long)p.nheads, 4),
               Span(weight, C * width, we), Span(bias, C, we), Span(positions, p.batch, 4),
               Span(slots, p.batch, 4)}))
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
    // Heads a CTA: while that leaves five rounds of the three CTAs an SM holds, so that the last,
    // partly filled one weighs little (128 rows of 80 heads: 4 heads 111 us, 8 122, 1 139).
    a.heads = 1;
    const int per_group = p.nheads / p.ngroups;
    while (a.split == 1 && a.heads < kMostHeads && per_group % (2 * a.heads) == 0 &&
           units / (2 * a.heads) >= 15LL * sm_count())
        a.heads *= 2;
    for (int n = p.dstate / 4; n > 1; n >>= 1) ++a.log_n4;
    const dim3 grid((unsigned)(p.nheads / a.heads * a.split), (unsigned)p.batch);
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
