// One token of linear attention for every row of a serving batch, over cache slots:
//     S <- a S + v k^T,   o = scale S q       (S is P x N, fp32, in place)
//
// Bound by the state's bytes, 2 P N 4 a row and head.  A block takes a run of rows p of one head's
// state, which lie next to one another in memory, and every thread has all its pieces of them in
// flight before it waits for the first; the lanes of a row add up its product with q.
//
// GB300, 80 heads x 64 x 128, bf16: 128 rows (4 of them padding) 110 us, 88 % of the copy rate on the
// live rows' bytes (119 with blocks of 256 threads and 32 KB); one row 6.1 us, the host's time for the
// call (3.5 in a replayed graph).
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "layer_device.cuh"
#include "linattn.cuh"

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

// `width` elements of each of `n` tokens, `stride` apart, as rows of 128 floats: a warp takes every
// fourth token, and has its elements on their way before the first is put down.
template <typename T>
struct Rows4 {
    T x[linattn::kFewTokens / (kThreads / 32)][4];
    __device__ __forceinline__ void load(const T* from, long long stride, int width, int n) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int u = 0; u < linattn::kFewTokens / (kThreads / 32); ++u) {
            const int t = (threadIdx.x >> 5) + u * (kThreads / 32);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (t < n && lane + 32 * c < width) x[u][c] = from[t * stride + lane + 32 * c];
        }
    }
    __device__ __forceinline__ void store(float* to, int width, int n) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int u = 0; u < linattn::kFewTokens / (kThreads / 32); ++u) {
            const int t = (threadIdx.x >> 5) + u * (kThreads / 32);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (t < n && lane + 32 * c < width) to[t * 128 + lane + 32 * c] = static_cast<float>(x[u][c]);
        }
    }
};

// A few tokens of every sequence in the same way: the state stays in registers over them, their q, k
// and v in shared memory.  A chunked walk's fixed steps take longer than sixteen tokens here: seven
// tokens of 80 heads of 64 x 128, 10.2 us a call against the walk's 12.3 (8.0 in a replayed graph).
// Bound by latency: each token's sums wait for the update before.
template <typename T, int PIECES>
__global__ void __launch_bounds__(kThreads, 4) attn_few_kernel(const __grid_constant__ linattn::WalkArgs a, int lanes, int rows) {
    constexpr int kTokens = linattn::kFewTokens;
    __shared__ __align__(16) float qs[kTokens][128], ks[kTokens][128];
    __shared__ float vs[kTokens][128];
    const linattn::Pass& p = a.pass[0];
    const int h = blockIdx.y, N = p.kd, p0 = blockIdx.x * rows, np = min(rows, p.vd - p0);
    T* out = static_cast<T*>(p.out) + (long long)h * p.vd + p0;
    if (a.cu && blockIdx.z == 0) {
        const linattn::Outside none(a);
        for (long long t = 0; t < none.n; ++t)
            for (int i = threadIdx.x; i < np; i += kThreads) st_out(out, none.token(t) * p.os + i, 0.f);
    }
    for (int s = blockIdx.z; s < a.nseq; s += gridDim.z) {
        const linattn::Seg g = linattn::sequence(a, s);
        const int lane = threadIdx.x & (lanes - 1), first = threadIdx.x / lanes, step = kThreads / lanes;
        const bool in = 4 * lane < N;
        const long long at = (((long long)s * a.H + h) * p.vd + p0) * N + 4 * lane;
        float4 S[PIECES];
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
            const int r = i * step + first;
            S[i] = p.s_in && in && r < np ? *reinterpret_cast<const float4*>(p.s_in + at + (long long)r * N)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        __syncthreads();
        const T* q = static_cast<const T*>(p.q) + g.start * p.qs + (long long)h * N;
        const T* k = static_cast<const T*>(p.k) + g.start * p.ks + (long long)(h / p.kr) * N;
        const T* v = static_cast<const T*>(p.v) + g.start * p.vs + (long long)(h / p.vr) * p.vd + p0;
        {
            Rows4<T> qr, kr, vr;
            qr.load(q, p.qs, N, g.len);
            kr.load(k, p.ks, N, g.len);
            vr.load(v, p.vs, np, g.len);
            qr.store(&qs[0][0], N, g.len);
            kr.store(&ks[0][0], N, g.len);
            vr.store(&vs[0][0], np, g.len);
        }
        __syncthreads();
        const float decay = expf(a.ld[h]);
        for (int t = 0; t < g.len; ++t) {
            float4 qq = make_float4(0.f, 0.f, 0.f, 0.f), kk = qq;
            if (in) qq = *reinterpret_cast<const float4*>(&qs[t][4 * lane]), kk = *reinterpret_cast<const float4*>(&ks[t][4 * lane]);
            float sum[PIECES];
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int r = i * step + first;
                const float vv = r < np ? vs[t][r] : 0.f;
                float4& w = S[i];
                w.x = fmaf(decay, w.x, vv * kk.x);
                w.y = fmaf(decay, w.y, vv * kk.y);
                w.z = fmaf(decay, w.z, vv * kk.z);
                w.w = fmaf(decay, w.w, vv * kk.w);
                sum[i] = (w.x * qq.x + w.y * qq.y) + (w.z * qq.z + w.w * qq.w);
            }
            for (int m = lanes >> 1; m > 0; m >>= 1)
#pragma unroll
                for (int i = 0; i < PIECES; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], m);
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < PIECES; ++i) {
                    const int r = i * step + first;
                    if (r < np) st_out(out, (g.start + t) * p.os + r, sum[i] * p.sx);
                }
        }
        if (p.s_out && in)
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int r = i * step + first;
                if (r < np) *reinterpret_cast<float4*>(p.s_out + at + (long long)r * N) = S[i];
            }
    }
}

// Lanes of a row of N elements in pieces of `vec`, and the rows of P that a block takes: as many as
// its threads have in flight at once, halved while there are fewer than two blocks for each SM and
// each thread keeps a piece.
void step_shape(int P, int N, int vec, long long heads, int* lanes, int* rows) {
    *lanes = 1;
    while (*lanes < 32 && *lanes * vec < N) *lanes *= 2;
    *rows = std::min(P, std::max(1, kPieces * kThreads / *lanes));
    while (heads * ((P + *rows - 1) / *rows) < 2LL * sm_count() && *rows * *lanes >= 2 * kThreads)
        *rows = (*rows + 1) / 2;
}

}  // namespace
}  // namespace layer

bool linattn::few_fits(const WalkArgs& a) {
    const Pass& p = a.pass[0];
    return (a.cu ? a.T : a.rowlen) <= kFewTokens && p.kd % 4 == 0 && layer::aligned_to(p.s_in, 16) &&
           layer::aligned_to(p.s_out, 16);
}

cudaError_t linattn::few_tokens(const WalkArgs& a, int dtype, Launch& L) {
    const Pass& p = a.pass[0];
    int lanes = 1;
    while (lanes < 32 && lanes * 4 < p.kd) lanes *= 2;
    // as few pieces of the state a thread as leave the blocks one round of the four an SM holds: the
    // tokens' steps wait for one another, so that only blocks side by side hide them
    const auto rows_of = [&](int pieces) { return std::min(p.vd, pieces * layer::kThreads / lanes); };
    int pieces = 2;
    while (pieces < 8 && (long long)a.nseq * a.H * ((p.vd + rows_of(pieces) - 1) / rows_of(pieces)) > 4LL * sm_count())
        pieces *= 2;
    const int rows = rows_of(pieces);
    const dim3 grid((unsigned)((p.vd + rows - 1) / rows), (unsigned)a.H, (unsigned)std::min(a.nseq, 65535));
    const auto run = [&](auto t) {
        using T = decltype(t);
        if (pieces == 2)
            layer::attn_few_kernel<T, 2><<<grid, layer::kThreads, 0, L.stream>>>(a, lanes, rows);
        else if (pieces == 4)
            layer::attn_few_kernel<T, 4><<<grid, layer::kThreads, 0, L.stream>>>(a, lanes, rows);
        else
            layer::attn_few_kernel<T, 8><<<grid, layer::kThreads, 0, L.stream>>>(a, lanes, rows);
    };
    L.begin("linattn_few");
    if (dtype == SSD_DTYPE_BF16)
        run(__nv_bfloat16());
    else
        run(float());
    return L.end();
}

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
    const int vec = N % 4 == 0 ? 4 : 1;  // elements of the state in a piece
    if (!aligned_to(state, 4 * vec) || !aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) ||
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
    step_shape(p.headdim, p.dstate, vec, B * H, &a.lanes, &a.rows);
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
