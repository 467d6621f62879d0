// Layer norm and its mean-free form (root mean square), with the residual add in front
// fused in, and the backward pass with the sums for the weight's and bias's gradients.
// Row by row, D columns:
//
//   v = x + r;  mu = mean(v) (0 for rms);  rstd = (mean((v - mu)^2) + eps)^-1/2
//   y = (v - mu) rstd w + b;  h = v in the residual's type
//
//   xh = (h - mu) rstd;  a = w dy
//   dv = rstd (a - mean(a) - xh mean(a xh)) + dh  (rms: without mean(a))
//   dw = sum over rows of dy xh;  db = sum over rows of dy
//
// Both are bound by HBM.  A team of warps holds the whole row in registers, so v is read
// once, the variance is the two-pass one (sums of squares of v - mu), and in the backward a
// block keeps its columns' dw and db in registers over all the rows it takes; a second
// kernel adds the blocks' partial sums in a fixed order.
//
// What costs time beside HBM is a row's fixed part: its sums, barriers and addresses.  So a
// thread's columns beyond the row count as zeros instead of taking branches, and a thread holds as
// many elements as its registers allow.
//
// GB300, 32768 x 2560, bf16 with a float32 residual: forward 156 us (95 % of the measured copy
// rate), backward 221 us (90 %, its partial sums included); without a residual 65 and 103 us
// (76 and 72 %); float32 with a residual 203 and 236 us (97 and 84 %), without 133 and 183 us
// (74 and 81 %).  Backward of bf16 rows with a float32 h and no gradient of it, the last norm of
// a network, 189 us (78 %; at 5120 columns 95 %).  Rows of more than 8192 columns: 8192 x 16384 with
// a float32 residual 299 us forward (80 %), 691 backward (46 %: spills).
#include <limits.h>

#include <type_traits>

#include "layer_device.cuh"
#include "layer_host.cuh"
#include "layer_team.cuh"

namespace ssd {
namespace layer {

namespace {

struct NormArgs {
    const void* x;
    const void* res;
    const void* w;
    const void* b;
    void* y;
    void* h;
    float2* stats;
    // backward
    const void* dy;
    const void* hin;
    const void* dh;
    const float2* stats_in;
    void* dx;
    void* dres;
    float* partial;
    long long rows, xs, rs, hs, ys;
    int D, nw, width, teams;
    int layer;     // 0: rms
    int wbf16;
    int nk;        // partial rows: d_weight (and d_bias)
    int stages;
    int* status;
    float eps, inv;  // inv: 1 / D
};

// This thread's parameters of its columns (zero beyond the row).
template <int VEC, int NV>
__device__ __forceinline__ void columns_of(const void* p, const Team& t, int cols, int bf16,
                                           typename Lanes<VEC>::V (*v)[Lanes<VEC>::N]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = ((t.warp * NV + i) * 32 + t.lane) * VEC;
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = 0.f;
        if (p && c < cols) params<VEC>(p, c, bf16, f);
        to_lanes<VEC>(f, v[i]);
    }
}

// RES: with a residual.
template <typename T, typename TR, bool RES, int VEC, int NV>
__global__ void __maxnreg__(fwd_regs(VEC, NV)) norm_fwd_kernel(const NormArgs a) {
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    __shared__ TeamBuf<1> buf;
    const Team t = team_of(a.nw, a.width);
    const RowRange rows((long long)blockIdx.x * a.teams + t.id, (long long)gridDim.x * a.teams, a.rows);
    // Short rows without a residual: two on their way, 52 us instead of 55 at 131072 x 512 and 58
    // instead of 62 at 262144 x 256; wider ones have no registers for it or gain nothing.
    constexpr int DEPTH = !RES && VEC * NV <= 16 ? 2 : 1;
    // A float32 residual beside bf16 rows is read as a stream (h replaces it): 156 us instead of
    // 161 at 32768 x 2560, 129 instead of 134 at 65536 x 1024; of the rows' own type 108 instead
    // of 107.
    constexpr bool STREAM = RES && sizeof(TR) > sizeof(T);
    using In = Rows<T, TR, 1, RES ? 1 : 0, VEC, NV, false, DEPTH, STREAM>;
    In in;
    auto from_a = [&](int, int row) { return row_at<T>(a.x, row, a.xs); };
    auto from_b = [&](int, int row) { return row_at<TR>(a.res, row, a.rs); };
    in.begin(t, rows, a.D, 0, nullptr, nullptr, nullptr);
    buf.clear();  // and its barrier
    in.start(t, from_a, from_b);
    V w[NV][N], b[NV][N];
    columns_of<VEC, NV>(a.w, t, a.D, a.wbf16, w);
    columns_of<VEC, NV>(a.b, t, a.D, a.wbf16, b);
    const bool layer = a.layer;
    const float inv = a.inv, eps = a.eps;
    int flip = 0;
    // every team of the block takes the rounds of its first team, the last perhaps without a row
    int row = rows.first, first = blockIdx.x * a.teams;
    auto one = [&](auto slot) {
        constexpr int S = decltype(slot)::value;
        const bool on = row < rows.rows;
        V v[NV][N];
        V s = both<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            in.template get_a<S>(t, i, 0, v[i]);
            if constexpr (RES) {
                V r[N];
                in.template get_b<S>(t, i, 0, r);
#pragma unroll
                for (int e = 0; e < N; ++e) v[i][e] = add_(v[i][e], r[e]);
                if (on && in.in[i])
                    store_lanes<VEC>(static_cast<TR*>(a.h) + row * a.hs + In::column(t, i), v[i]);
            }
#pragma unroll
            for (int e = 0; e < N; ++e) s = add_(s, v[i][e]);
        }
        in.template done<S>(t, from_a, from_b);
        float mean = 0.f;
        if (layer) {
            float m = lane_sum(s);
            team_sum<1>(t, &m, buf, flip);
            flip ^= 1;
            mean = m * inv;
        }
        V q = both<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const V minus = both<V>(in.in[i] ? -mean : 0.f);  // nothing beyond the row
#pragma unroll
            for (int e = 0; e < N; ++e) {
                v[i][e] = add_(v[i][e], minus);
                q = fma_(v[i][e], v[i][e], q);
            }
        }
        float var = lane_sum(q);
        team_sum<1>(t, &var, buf, flip);
        flip ^= 1;
        const float rstd = __frsqrt_rn(fmaf(var, inv, eps));
        if (on && t.rank == 0 && a.stats) a.stats[row] = make_float2(mean, rstd);
        T* y = static_cast<T*>(a.y) + row * a.ys + In::column(t, 0);
        const V r = both<V>(rstd);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = fma_(mul_(v[i][e], r), w[i][e], b[i][e]);
            if (on && in.in[i]) store_lanes<VEC>(y + i * 32 * VEC, o);
        }
        first += rows.by, row += rows.by;
    };
    while (first < rows.rows) {
        one(std::integral_constant<int, 0>());
        if constexpr (DEPTH > 1)
            if (first < rows.rows) one(std::integral_constant<int, 1>());
    }
}

// DH: with the residual stream's gradient.
template <typename T, typename TR, bool DH, int VEC, int NV, bool BULK>
__global__ void __maxnreg__(bwd_regs(VEC, NV, BULK)) norm_bwd_kernel(const NormArgs a) {
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    __shared__ TeamBuf<2> buf;
    extern __shared__ __align__(128) char ring[];
    const Team t = team_of(a.nw, a.width);
    const RowRange rows((long long)blockIdx.x * a.teams + t.id, (long long)gridDim.x * a.teams, a.rows);
    using In = Rows<T, TR, 1, DH ? 2 : 1, VEC, NV, BULK>;
    In in;
    __shared__ RowBars bars;
    auto from_a = [&](int, int row) { return row_at<T>(a.dy, row, a.ys); };
    auto from_b = [&](int k, int row) {
        return DH && k == 1 ? row_at<TR>(a.dh, row, a.rs) : row_at<TR>(a.hin, row, a.hs);
    };
    in.begin(t, rows, a.D, a.stages, ring, &bars, a.status);
    buf.clear();  // and its barrier
    in.start(t, from_a, from_b);
    V w[NV][N], dw[NV][N], db[NV][N];
    columns_of<VEC, NV>(a.w, t, a.D, a.wbf16, w);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = db[i][e] = both<V>(0.f);
    const bool both_out = a.dres != nullptr;
    const float inv = a.inv, inv1 = a.layer ? a.inv : 0.f;
    float2 next = rows.first < rows.rows ? a.stats_in[rows.first] : make_float2(0.f, 0.f);
    int flip = 0;
    // every team of the block takes the rounds of its first team, the last perhaps without a row
    int row = rows.first;
    for (int first = blockIdx.x * a.teams; first < rows.rows; first += rows.by, row += rows.by) {
        const float2 st = next;
        if (row + rows.by < rows.rows) next = a.stats_in[row + rows.by];
        const bool on = row < rows.rows;
        V xh[NV][N], d[NV][N], g[NV][N];
        V s0 = both<V>(0.f), s1 = both<V>(0.f);
        const V r = both<V>(st.y);
        if (on) {
            in.arrived();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const V minus = both<V>(in.in[i] ? -st.x : 0.f);  // nothing beyond the row
                in.get_a(t, i, 0, d[i]);
                in.get_b(t, i, 0, xh[i]);
                if constexpr (DH) in.get_b(t, i, 1, g[i]);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    xh[i][e] = mul_(add_(xh[i][e], minus), r);
                    dw[i][e] = fma_(d[i][e], xh[i][e], dw[i][e]);
                    db[i][e] = add_(db[i][e], d[i][e]);
                    d[i][e] = mul_(d[i][e], w[i][e]);
                    s0 = add_(s0, d[i][e]);
                    s1 = fma_(d[i][e], xh[i][e], s1);
                }
            }
        }
        in.done(t, from_a, from_b);
        float sum[2] = {lane_sum(s0), lane_sum(s1)};
        team_sum<2>(t, sum, buf, flip);
        flip ^= 1;
        in.reuse(t, from_a, from_b);
        if (on) {
            const V c1 = both<V>(-sum[0] * inv1), c2 = both<V>(-sum[1] * inv);
            T* dx = static_cast<T*>(a.dx) + row * a.xs + In::column(t, 0);
            TR* dres = static_cast<TR*>(a.dres) + (long long)row * a.D + In::column(t, 0);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                V o[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const V k = fma_(xh[i][e], c2, add_(d[i][e], c1));
                    if constexpr (DH)
                        o[e] = fma_(k, r, g[i][e]);
                    else
                        o[e] = mul_(k, r);
                }
                if (in.in[i]) store_lanes<VEC>(dx + i * 32 * VEC, o);
                if (both_out && in.in[i]) store_lanes<VEC>(dres + i * 32 * VEC, o);
            }
        }
    }
    float* part = a.partial + (long long)blockIdx.x * a.nk * a.D;
    if (a.teams > 1) {  // the teams' sums are joined in order, in the ring's place
        in.drain(t, row - rows.by >= rows.rows);
        float* acc = reinterpret_cast<float*>(ring);
        __syncthreads();
        for (int k = 0; k < a.teams; ++k) {
            if (t.id == k)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = In::column(t, i);
                    if (c >= a.D) continue;
                    float f[VEC], g[VEC];
                    from_lanes<VEC>(dw[i], f);
                    from_lanes<VEC>(db[i], g);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        acc[c + e] = k == 0 ? f[e] : acc[c + e] + f[e];
                        acc[a.D + c + e] = k == 0 ? g[e] : acc[a.D + c + e] + g[e];
                    }
                }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < a.nk * a.D; i += blockDim.x) part[i] = acc[i];
        return;
    }
    in.drain(t, row - rows.by >= rows.rows);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = In::column(t, i);
        if (c >= a.D) continue;
        store_lanes<VEC>(part + c, dw[i]);
        if (a.nk > 1) store_lanes<VEC>(part + a.D + c, db[i]);
    }
}

// ------------------------------------------------------------------ host
ssd_status_t check_norm(const ssd_norm_t* p) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->rows < 0 || p->dim < 1) return SSD_ERR_INVALID_ARG;
    if (!dtype_ok(p->dtype) || !dtype_ok(p->rdtype) || !dtype_ok(p->wdtype))
        return SSD_ERR_INVALID_ARG;
    if (p->kind != SSD_NORM_LAYER && p->kind != SSD_NORM_RMS) return SSD_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || p->eps > 1e30f) return SSD_ERR_INVALID_ARG;
    if (p->x_stride < p->dim || p->r_stride < p->dim || p->h_stride < p->dim ||
        p->y_stride < p->dim)
        return SSD_ERR_INVALID_ARG;
    // the residual stream is kept in the activations' type or in float32
    if (p->dtype == SSD_DTYPE_F32 && p->rdtype != SSD_DTYPE_F32) return SSD_ERR_UNSUPPORTED;
    if (p->rows > INT_MAX - (1 << 20)) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Elements of a vector at most: 16 bytes of the widest tensor.  (bf16 rows beside a float32
// residual in vectors of eight would touch every 32-byte sector of the float32 rows twice, in
// halves: 298 us instead of 216 for the backward at 32768 x 2560.)
int most_vec(const ssd_norm_t* p, bool residual) {
    return p->dtype == SSD_DTYPE_F32 || (residual && p->rdtype == SSD_DTYPE_F32) ? 4 : 8;
}
RowCost fwd_cost(const ssd_norm_t* p, bool residual) {
    return {false, 1, (int)dtype_size(p->dtype), residual ? 1 : 0, (int)dtype_size(p->rdtype)};
}
RowCost bwd_cost(const ssd_norm_t* p, bool dh) {
    return {true, 1, (int)dtype_size(p->dtype), dh ? 2 : 1, (int)dtype_size(p->rdtype)};
}
// Shared memory of a backward's block: the ring, or the sums of several teams at the end.
size_t bwd_smem(const RowPlan& p, int dim) {
    const size_t sums = p.teams > 1 ? sizeof(float) * 2 * dim : 0;
    return p.ring > sums ? p.ring : sums;
}

template <bool BWD, typename T, typename TR, bool OPT, int VEC, int NV, bool BULK>
cudaError_t launch_mode(const RowPlan& p, unsigned grid, const NormArgs& a, cudaStream_t s) {
    constexpr auto kernel = [] {
        if constexpr (BWD)
            return &norm_bwd_kernel<T, TR, OPT, VEC, NV, BULK>;
        else
            return &norm_fwd_kernel<T, TR, OPT, VEC, NV>;
    }();
    const size_t smem = BWD ? bwd_smem(p, a.D) : 0;
    const cudaError_t e = allow_smem<kernel>(smem);
    if (e == cudaSuccess) kernel<<<grid, p.threads(), smem, s>>>(a);
    return e;
}
// The backward's wide rows come by bulk copies unless a warp has lanes to spare.
template <bool BWD, typename T, typename TR, bool OPT, int VEC, int NV>
cudaError_t launch_nv(const RowPlan& p, unsigned grid, const NormArgs& a, cudaStream_t s) {
    if constexpr (BWD && VEC >= 4) {
        if (p.bulk) return launch_mode<BWD, T, TR, OPT, VEC, NV, true>(p, grid, a, s);
        if constexpr (NV == 1) return launch_mode<BWD, T, TR, OPT, VEC, NV, false>(p, grid, a, s);
        return cudaErrorInvalidValue;
    } else {
        return launch_mode<BWD, T, TR, OPT, VEC, NV, false>(p, grid, a, s);
    }
}
template <bool BWD, typename T, typename TR, bool OPT, int VEC>
cudaError_t launch_vec(const RowPlan& p, unsigned grid, const NormArgs& a, cudaStream_t s) {
    switch (p.nv) {
        case 1: return launch_nv<BWD, T, TR, OPT, VEC, 1>(p, grid, a, s);
        case 2: return launch_nv<BWD, T, TR, OPT, VEC, 2>(p, grid, a, s);
        case 3: return launch_nv<BWD, T, TR, OPT, VEC, 3>(p, grid, a, s);
        case 4: return launch_nv<BWD, T, TR, OPT, VEC, 4>(p, grid, a, s);
        case 6:
            if constexpr (most_vectors(VEC) >= 8) return launch_nv<BWD, T, TR, OPT, VEC, 6>(p, grid, a, s);
            break;
        case 8:
            if constexpr (most_vectors(VEC) >= 8) return launch_nv<BWD, T, TR, OPT, VEC, 8>(p, grid, a, s);
            break;
        case 16:
            if constexpr (most_vectors(VEC) >= 16) return launch_nv<BWD, T, TR, OPT, VEC, 16>(p, grid, a, s);
            break;
    }
    return cudaErrorInvalidValue;
}
template <bool BWD, typename T, typename TR, bool OPT>
cudaError_t launch_types(const RowPlan& p, unsigned grid, const NormArgs& a, cudaStream_t s) {
    constexpr int wide = sizeof(T) == 2 && sizeof(TR) == 2 ? 8 : 4;
    if (p.vec == wide) return launch_vec<BWD, T, TR, OPT, wide>(p, grid, a, s);
    if (p.vec == 2) return launch_vec<BWD, T, TR, OPT, 2>(p, grid, a, s);
    return launch_vec<BWD, T, TR, OPT, 1>(p, grid, a, s);
}
// `opt`: with a residual (forward) or with its gradient (backward).
template <bool BWD>
cudaError_t launch_norm(const ssd_norm_t* n, bool opt, const RowPlan& p, unsigned grid,
                        const NormArgs& a, cudaStream_t s) {
    using B16 = __nv_bfloat16;
    const bool mixed = n->dtype == SSD_DTYPE_BF16 && n->rdtype == SSD_DTYPE_F32;
    if (mixed && opt) return launch_types<BWD, B16, float, true>(p, grid, a, s);
    if constexpr (BWD)
        if (mixed) return launch_types<BWD, B16, float, false>(p, grid, a, s);
    if (n->dtype == SSD_DTYPE_BF16)
        return opt ? launch_types<BWD, B16, B16, true>(p, grid, a, s)
                   : launch_types<BWD, B16, B16, false>(p, grid, a, s);
    return opt ? launch_types<BWD, float, float, true>(p, grid, a, s)
               : launch_types<BWD, float, float, false>(p, grid, a, s);
}

}  // namespace
}  // namespace layer
}  // namespace ssd

using namespace ssd;
using namespace ssd::layer;

extern "C" {

ssd_status_t ssd_norm_forward(const ssd_norm_t* norm, const void* x, const void* residual,
                              const void* weight, const void* bias, void* y, void* h,
                              float* stats, void* stream) {
    set_last_launches(0);
    ssd_status_t st = check_norm(norm);
    if (st != SSD_OK) return st;
    if (!weight || (residual != nullptr) != (h != nullptr)) return SSD_ERR_INVALID_ARG;
    if (norm->rows > 0 && (!x || !y)) return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(norm->dtype), re = dtype_size(norm->rdtype);
    const size_t we = dtype_size(norm->wdtype);
    if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(residual, re) || !aligned_to(h, re) ||
        !aligned_to(weight, we) || !aligned_to(bias, we) || !aligned_to(stats, 8))
        return SSD_ERR_ALIGNMENT;
    if (norm->rows == 0) return SSD_OK;
    // h may replace the residual and y may replace x; any other overlap is refused
    const long long n = norm->rows;
    const int D = norm->dim;
    const Span sx(x, n, norm->x_stride, D, e), sr(residual, n, norm->r_stride, D, re);
    const Span sy(y, n, norm->y_stride, D, e), sh(h, n, norm->h_stride, D, re);
    const bool same_y = x == y && norm->x_stride == norm->y_stride;
    const bool same_h = residual == h && norm->r_stride == norm->h_stride;
    if (clash({sy, sh, Span(stats, 2 * n, 4)},
              {same_y ? Span() : sx, same_h ? Span() : sr, Span(weight, D, we), Span(bias, D, we)}))
        return SSD_ERR_INVALID_ARG;
    const void* ptrs[4] = {x, y, residual, h};
    const size_t sizes[4] = {e, e, re, re};
    RowPlan p;
    const long long strides[5] = {D, norm->x_stride, norm->r_stride, norm->h_stride, norm->y_stride};
    const bool opt = residual != nullptr;
    if (!plan_row(D, common_vec(most_vec(norm, opt), strides, 5, ptrs, sizes, 4), fwd_cost(norm, opt), &p))
        return SSD_ERR_UNSUPPORTED;
    NormArgs a = {};
    a.x = x, a.res = residual, a.w = weight, a.b = bias, a.y = y, a.h = h;
    a.stats = reinterpret_cast<float2*>(stats);
    a.rows = n, a.xs = norm->x_stride, a.rs = norm->r_stride, a.hs = norm->h_stride,
    a.ys = norm->y_stride;
    a.D = D, a.nw = p.nw, a.width = p.width, a.teams = p.teams, a.stages = p.stages;
    a.status = status_word();
    if (!a.status) return SSD_ERR_CUDA;
    a.layer = norm->kind == SSD_NORM_LAYER, a.wbf16 = norm->wdtype == SSD_DTYPE_BF16;
    a.eps = norm->eps, a.inv = (float)(1.0 / D);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("norm_fwd");
    cudaError_t err = launch_norm<false>(norm, opt, p, (unsigned)team_blocks(n, p), a, L.stream);
    const cudaError_t last = L.end();
    if (err == cudaSuccess) err = last;
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_norm_workspace_size(const ssd_norm_t* norm, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    ssd_status_t st = check_norm(norm);
    if (st != SSD_OK) return st;
    size_t most = 256;
    bool any = false;
    for (int i = 0; i < 6; ++i) {  // any may run, by the pointers' alignment and with dh or without
        const int vec = i < 2 ? most_vec(norm, true) : i < 4 ? 2 : 1;
        RowPlan p;
        if (norm->dim % vec || !plan_row(norm->dim, vec, bwd_cost(norm, i & 1), &p)) continue;
        any = true;
        const size_t n = sizeof(float) * (size_t)team_blocks(norm->rows, p) * 2 * norm->dim;
        if (n > most) most = n;
    }
    if (!any) return SSD_ERR_UNSUPPORTED;
    *bytes = (most + 255) / 256 * 256;
    return SSD_OK;
}

ssd_status_t ssd_norm_backward(const ssd_norm_t* norm, const void* dy, const void* h,
                               const void* dh, const void* weight, const float* stats, void* dx,
                               void* d_residual, void* d_weight, void* d_bias, void* workspace,
                               size_t workspace_bytes, void* stream) {
    set_last_launches(0);
    ssd_status_t st = check_norm(norm);
    if (st != SSD_OK) return st;
    if (!weight || !d_weight) return SSD_ERR_INVALID_ARG;
    const long long n = norm->rows;
    const int D = norm->dim;
    if (n > 0 && (!dy || !h || !stats || !dx)) return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(norm->dtype), re = dtype_size(norm->rdtype);
    const size_t we = dtype_size(norm->wdtype);
    if (!aligned_to(dy, e) || !aligned_to(dx, e) || !aligned_to(h, re) || !aligned_to(dh, re) ||
        !aligned_to(d_residual, re) || !aligned_to(weight, we) || !aligned_to(d_weight, we) ||
        !aligned_to(d_bias, we) || !aligned_to(stats, 8))
        return SSD_ERR_ALIGNMENT;
    // a gradient may replace the gradient it is computed from, element by element
    const Span sdy(dy, n, norm->y_stride, D, e), sdx(dx, n, norm->x_stride, D, e);
    const Span sh(h, n, norm->h_stride, D, re), sdh(dh, n, norm->r_stride, D, re);
    const Span sdr(d_residual, n, D, D, re);
    const bool dx_dy = dx == dy && norm->x_stride == norm->y_stride;
    const bool dx_dh = dx == dh && norm->x_stride == norm->r_stride && e == re;
    const bool dr_dh = d_residual == dh && norm->r_stride == D;
    size_t need = 0;
    st = ssd_norm_workspace_size(norm, &need);
    if (st != SSD_OK) return st;
    if (clash({sdx, sdr, Span(d_weight, D, we), Span(d_bias, D, we), Span(workspace, need, 1)},
              {dx_dy ? Span() : sdy, dx_dh || dr_dh ? Span() : sdh, sh, Span(weight, D, we),
               Span(stats, 2 * n, 4)}))
        return SSD_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return SSD_ERR_ALIGNMENT;
    const void* ptrs[5] = {dy, dx, h, dh, d_residual};
    const size_t sizes[5] = {e, e, re, re, re};
    RowPlan p;
    const long long strides[5] = {D, norm->x_stride, norm->r_stride, norm->h_stride, norm->y_stride};
    if (!plan_row(D, common_vec(most_vec(norm, true), strides, 5, ptrs, sizes, 5), bwd_cost(norm, dh), &p))
        return SSD_ERR_UNSUPPORTED;
    NormArgs a = {};
    a.dy = dy, a.hin = h, a.dh = dh, a.w = weight, a.dx = dx, a.dres = d_residual;
    a.stats_in = reinterpret_cast<const float2*>(stats);
    a.partial = static_cast<float*>(workspace);
    a.rows = n, a.xs = norm->x_stride, a.rs = norm->r_stride, a.hs = norm->h_stride,
    a.ys = norm->y_stride;
    a.D = D, a.nw = p.nw, a.width = p.width, a.teams = p.teams, a.stages = p.stages;
    a.status = status_word();
    if (!a.status) return SSD_ERR_CUDA;
    a.layer = norm->kind == SSD_NORM_LAYER, a.wbf16 = norm->wdtype == SSD_DTYPE_BF16;
    a.nk = d_bias ? 2 : 1;
    a.inv = (float)(1.0 / D);
    const int blocks = team_blocks(n, p);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (blocks > 0) {
        L.begin("norm_bwd");
        err = launch_norm<true>(norm, dh != nullptr, p, (unsigned)blocks, a, L.stream);
        const cudaError_t last = L.end();
        if (err == cudaSuccess) err = last;
    }
    if (err == cudaSuccess) {
        ReduceDst d = {};
        d.dst[0] = d_weight, d.step[0] = 1;
        d.dst[1] = d_bias, d.step[1] = 1;
        err = launch_partial_sum(a.partial, blocks, a.nk, D, d, norm->wdtype, L);
    }
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
