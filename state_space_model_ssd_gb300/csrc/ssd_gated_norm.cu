// The scan's output times the SiLU of its gate, normed by its root mean square within each
// of G groups of the columns, and the backward pass:
//
//   v = y silu(z);  rstd = (mean over the group of v^2 + eps)^-1/2;  out = v rstd w
//
//   xh = v rstd;  a = w dout
//   dv = rstd (a - xh mean(a xh));  dy = dv silu(z);  dz = dv y s (1 + z (1 - s)), s = sigmoid(z)
//   dw = sum over rows of dout xh
//
// Bound by HBM (three tensors forward, five backward).  A (row, group) is one row of a team;
// blocks stay with one group, so that the backward's dw stays in registers.
//
// GB300, 32768 x 5120, bf16: forward 155 us (95 % of the measured copy rate); backward 276 us in
// one group (90 %), 327 in eight (76 %: three warps a row of 640 columns leave a sixth of their
// lanes idle and share out the sums' fixed cost less well).  Float32, 16384 x 5120: forward 216 us
// (69 %: its 32 elements a thread spill), backward 305 us (81 %).  bf16, 8192 x 16384: forward
// 126 us (94 %), backward 483 us (41 %: spills).
#include <limits.h>

#include "layer_device.cuh"
#include "layer_host.cuh"
#include "layer_team.cuh"

namespace ssd {
namespace layer {

namespace {

struct GatedArgs {
    const void* y;
    const void* z;
    const void* w;
    void* out;
    float* rstd;
    const void* dout;
    const float* rstd_in;
    void* dy;
    void* dz;
    float* partial;
    long long rows, ys, zs, os, dys, dzs;
    int D, G, n;   // columns, groups, columns of a group
    int nw, width, teams;
    int nrb;       // blocks of a group
    int wbf16;
    int stages;
    int* status;
    float eps, inv;  // inv: 1 / n
};

template <int VEC, int NV>
__device__ __forceinline__ void weights_of(const GatedArgs& a, const Team& t, int g0,
                                           typename Lanes<VEC>::V (*v)[Lanes<VEC>::N]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = ((t.warp * NV + i) * 32 + t.lane) * VEC;
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = 0.f;
        if (c < a.n) params<VEC>(a.w, g0 + c, a.wbf16, f);
        to_lanes<VEC>(f, v[i]);
    }
}

template <typename T, int VEC, int NV>
__global__ void __maxnreg__(fwd_regs(VEC, NV)) gated_fwd_kernel(const GatedArgs a) {
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    __shared__ TeamBuf<1> buf;
    const Team t = team_of(a.nw, a.width);
    const int g = blockIdx.x % a.G, rb = blockIdx.x / a.G;
    const int g0 = g * a.n;
    const RowRange rows((long long)rb * a.teams + t.id, (long long)a.nrb * a.teams, a.rows);
    using In = Rows<T, T, 2, 0, VEC, NV, false>;
    In in;
    auto from_a = [&](int k, int row) {
        return (k == 0 ? row_at<T>(a.y, row, a.ys) : row_at<T>(a.z, row, a.zs)) + g0;
    };
    auto from_b = [&](int, int) { return static_cast<const T*>(nullptr); };
    in.begin(t, rows, a.n, 0, nullptr, nullptr, nullptr);
    buf.clear();  // and its barrier
    in.start(t, from_a, from_b);
    V w[NV][N];
    weights_of<VEC, NV>(a, t, g0, w);
    const float inv = a.inv, eps = a.eps;
    int flip = 0;
    // every team of the block takes the rounds of its first team, the last perhaps without a row
    int row = rows.first;
    for (int first = rb * a.teams; first < rows.rows; first += rows.by, row += rows.by) {
        const bool on = row < rows.rows;
        V v[NV][N];
        V q = both<V>(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V z[N];
            in.get_a(t, i, 0, v[i]);
            in.get_a(t, i, 1, z);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                v[i][e] = mul_(v[i][e], mul_(z[e], sigmoid_lanes<T>(z[e])));
                q = fma_(v[i][e], v[i][e], q);
            }
        }
        in.done(t, from_a, from_b);
        float sum = lane_sum(q);
        team_sum<1>(t, &sum, buf, flip);
        flip ^= 1;
        const float rstd = __frsqrt_rn(fmaf(sum, inv, eps));
        if (on && t.rank == 0 && a.rstd) a.rstd[(long long)row * a.G + g] = rstd;
        T* out = static_cast<T*>(a.out) + row * a.os + g0 + In::column(t, 0);
        const V r = both<V>(rstd);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            V o[N];
#pragma unroll
            for (int e = 0; e < N; ++e) o[e] = mul_(mul_(v[i][e], r), w[i][e]);
            if (on && in.in[i]) store_lanes<VEC>(out + i * 32 * VEC, o);
        }
    }
}

template <typename T, int VEC, int NV, bool BULK>
__global__ void __maxnreg__(bwd_regs(VEC, NV, BULK)) gated_bwd_kernel(const GatedArgs a) {
    using V = typename Lanes<VEC>::V;
    constexpr int N = Lanes<VEC>::N;
    __shared__ TeamBuf<1> buf;
    extern __shared__ __align__(128) char ring[];
    const Team t = team_of(a.nw, a.width);
    const int g = blockIdx.x % a.G, rb = blockIdx.x / a.G;
    const int g0 = g * a.n;
    const RowRange rows((long long)rb * a.teams + t.id, (long long)a.nrb * a.teams, a.rows);
    using In = Rows<T, T, 3, 0, VEC, NV, BULK>;
    In in;
    __shared__ RowBars bars;
    auto from_a = [&](int k, int row) {
        return (k == 0   ? row_at<T>(a.dout, row, a.os)
                : k == 1 ? row_at<T>(a.y, row, a.ys)
                         : row_at<T>(a.z, row, a.zs)) +
               g0;
    };
    auto from_b = [&](int, int) { return static_cast<const T*>(nullptr); };
    in.begin(t, rows, a.n, a.stages, ring, &bars, a.status);
    buf.clear();  // and its barrier
    in.start(t, from_a, from_b);
    V w[NV][N], dw[NV][N];
    weights_of<VEC, NV>(a, t, g0, w);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = both<V>(0.f);
    const float inv = a.inv;
    float next = rows.first < rows.rows ? a.rstd_in[(long long)rows.first * a.G + g] : 0.f;
    int flip = 0;
    // every team of the block takes the rounds of its first team, the last perhaps without a row
    int row = rows.first;
    for (int first = rb * a.teams; first < rows.rows; first += rows.by, row += rows.by) {
        const V r = both<V>(next);
        if (row + rows.by < rows.rows) next = a.rstd_in[(long long)(row + rows.by) * a.G + g];
        const bool on = row < rows.rows;
        // d = w dout, gate = silu(z), gy = y silu'(z)
        V d[NV][N], xh[NV][N], gate[NV][N], gy[NV][N];
        V s = both<V>(0.f);
        if (on) {
            in.arrived();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                V y[N], z[N];
                in.get_a(t, i, 0, d[i]);
                in.get_a(t, i, 1, y);
                in.get_a(t, i, 2, z);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const V sg = sigmoid_lanes<T>(z[e]);
                    gate[i][e] = mul_(z[e], sg);
                    gy[i][e] = mul_(y[e], silu_slope(sg, gate[i][e]));
                    xh[i][e] = mul_(mul_(y[e], gate[i][e]), r);
                    dw[i][e] = fma_(d[i][e], xh[i][e], dw[i][e]);
                    d[i][e] = mul_(d[i][e], w[i][e]);
                    s = fma_(d[i][e], xh[i][e], s);
                }
            }
        }
        in.done(t, from_a, from_b);
        float sum = lane_sum(s);
        team_sum<1>(t, &sum, buf, flip);
        flip ^= 1;
        in.reuse(t, from_a, from_b);
        if (on) {
            const V c2 = both<V>(-sum * inv);
            T* dy = static_cast<T*>(a.dy) + row * a.dys + g0 + In::column(t, 0);
            T* dz = static_cast<T*>(a.dz) + row * a.dzs + g0 + In::column(t, 0);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                V oy[N], oz[N];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const V dv = mul_(fma_(xh[i][e], c2, d[i][e]), r);
                    oy[e] = mul_(dv, gate[i][e]);
                    oz[e] = mul_(dv, gy[i][e]);
                }
                if (in.in[i]) store_lanes<VEC>(dy + i * 32 * VEC, oy);
                if (in.in[i]) store_lanes<VEC>(dz + i * 32 * VEC, oz);
            }
        }
    }
    float* part = a.partial + (long long)rb * a.D + g0;
    if (a.teams > 1) {  // the teams' sums are joined in order, in the ring's place
        in.drain(t, row - rows.by >= rows.rows);
        float* acc = reinterpret_cast<float*>(ring);
        __syncthreads();
        for (int k = 0; k < a.teams; ++k) {
            if (t.id == k)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = In::column(t, i);
                    if (c >= a.n) continue;
                    float f[VEC];
                    from_lanes<VEC>(dw[i], f);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) acc[c + e] = k == 0 ? f[e] : acc[c + e] + f[e];
                }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < a.n; i += blockDim.x) part[i] = acc[i];
        return;
    }
    in.drain(t, row - rows.by >= rows.rows);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = In::column(t, i);
        if (c < a.n) store_lanes<VEC>(part + c, dw[i]);
    }
}

// ------------------------------------------------------------------ host
ssd_status_t check_gated(const ssd_gated_norm_t* p) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->rows < 0 || p->dim < 1 || p->groups < 1 || p->dim % p->groups) return SSD_ERR_INVALID_ARG;
    if (!dtype_ok(p->dtype) || !dtype_ok(p->wdtype)) return SSD_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || p->eps > 1e30f) return SSD_ERR_INVALID_ARG;
    if (p->y_stride < p->dim || p->z_stride < p->dim || p->out_stride < p->dim ||
        p->dy_stride < p->dim || p->dz_stride < p->dim)
        return SSD_ERR_INVALID_ARG;
    if (p->rows > INT_MAX - (1 << 20) || p->rows * p->groups > INT_MAX) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

RowCost fwd_cost(const ssd_gated_norm_t* p) { return {false, 2, (int)dtype_size(p->dtype), 0, 0}; }
RowCost bwd_cost(const ssd_gated_norm_t* p) { return {true, 3, (int)dtype_size(p->dtype), 0, 0}; }
int most_vec(const ssd_gated_norm_t* p) { return p->dtype == SSD_DTYPE_BF16 ? 8 : 4; }

// Blocks of one group.
int gated_blocks(long long rows, int groups, const RowPlan& p) {
    const long long most = ((long long)sm_count() * p.per_sm + groups - 1) / groups;
    const long long want = (rows + p.teams - 1) / p.teams;
    return (int)(want < most ? want : most);
}

// Shared memory of a backward's block: the ring, or the sums of several teams at the end.
size_t bwd_smem(const RowPlan& p, int n) {
    const size_t sums = p.teams > 1 ? sizeof(float) * n : 0;
    return p.ring > sums ? p.ring : sums;
}

template <bool BWD, typename T, int VEC, int NV, bool BULK>
cudaError_t launch_mode(const RowPlan& p, unsigned grid, const GatedArgs& a, cudaStream_t s) {
    constexpr auto kernel = [] {
        if constexpr (BWD)
            return &gated_bwd_kernel<T, VEC, NV, BULK>;
        else
            return &gated_fwd_kernel<T, VEC, NV>;
    }();
    const size_t smem = BWD ? bwd_smem(p, a.n) : 0;
    const cudaError_t e = allow_smem<kernel>(smem);
    if (e == cudaSuccess) kernel<<<grid, p.threads(), smem, s>>>(a);
    return e;
}
// The backward's wide rows come by bulk copies unless a warp has lanes to spare.
template <bool BWD, typename T, int VEC, int NV>
cudaError_t launch_nv(const RowPlan& p, unsigned grid, const GatedArgs& a, cudaStream_t s) {
    if constexpr (BWD && VEC >= 4) {
        if (p.bulk) return launch_mode<BWD, T, VEC, NV, true>(p, grid, a, s);
        if constexpr (NV == 1) return launch_mode<BWD, T, VEC, NV, false>(p, grid, a, s);
        return cudaErrorInvalidValue;
    } else {
        return launch_mode<BWD, T, VEC, NV, false>(p, grid, a, s);
    }
}
template <bool BWD, typename T, int VEC>
cudaError_t launch_vec(const RowPlan& p, unsigned grid, const GatedArgs& a, cudaStream_t s) {
    switch (p.nv) {
        case 1: return launch_nv<BWD, T, VEC, 1>(p, grid, a, s);
        case 2: return launch_nv<BWD, T, VEC, 2>(p, grid, a, s);
        case 3: return launch_nv<BWD, T, VEC, 3>(p, grid, a, s);
        case 4: return launch_nv<BWD, T, VEC, 4>(p, grid, a, s);
        case 6:
            if constexpr (most_vectors(VEC) >= 8) return launch_nv<BWD, T, VEC, 6>(p, grid, a, s);
            break;
        case 8:
            if constexpr (most_vectors(VEC) >= 8) return launch_nv<BWD, T, VEC, 8>(p, grid, a, s);
            break;
        case 16:
            if constexpr (most_vectors(VEC) >= 16) return launch_nv<BWD, T, VEC, 16>(p, grid, a, s);
            break;
    }
    return cudaErrorInvalidValue;
}
template <bool BWD, typename T>
cudaError_t launch_type(const RowPlan& p, unsigned grid, const GatedArgs& a, cudaStream_t s) {
    constexpr int wide = sizeof(T) == 2 ? 8 : 4;
    if (p.vec == wide) return launch_vec<BWD, T, wide>(p, grid, a, s);
    if (p.vec == 2) return launch_vec<BWD, T, 2>(p, grid, a, s);
    return launch_vec<BWD, T, 1>(p, grid, a, s);
}
template <bool BWD>
cudaError_t launch_gated(const ssd_gated_norm_t* n, const RowPlan& p, unsigned grid,
                         const GatedArgs& a, cudaStream_t s) {
    return n->dtype == SSD_DTYPE_F32 ? launch_type<BWD, float>(p, grid, a, s)
                                     : launch_type<BWD, __nv_bfloat16>(p, grid, a, s);
}

void fill_args(const ssd_gated_norm_t* g, const RowPlan& p, GatedArgs* a) {
    a->rows = g->rows;
    a->ys = g->y_stride, a->zs = g->z_stride, a->os = g->out_stride;
    a->dys = g->dy_stride, a->dzs = g->dz_stride;
    a->D = g->dim, a->G = g->groups, a->n = g->dim / g->groups;
    a->nw = p.nw, a->width = p.width, a->teams = p.teams, a->stages = p.stages;
    a->status = status_word();
    a->wbf16 = g->wdtype == SSD_DTYPE_BF16;
    a->eps = g->eps, a->inv = (float)(1.0 / a->n);
}

}  // namespace
}  // namespace layer
}  // namespace ssd

using namespace ssd;
using namespace ssd::layer;

extern "C" {

ssd_status_t ssd_gated_norm_forward(const ssd_gated_norm_t* norm, const void* y, const void* z,
                                    const void* weight, void* out, float* rstd, void* stream) {
    set_last_launches(0);
    ssd_status_t st = check_gated(norm);
    if (st != SSD_OK) return st;
    if (!weight) return SSD_ERR_INVALID_ARG;
    const long long n = norm->rows;
    if (n > 0 && (!y || !z || !out)) return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(norm->dtype);
    if (!aligned_to(y, e) || !aligned_to(z, e) || !aligned_to(out, e) || !aligned_to(rstd, 4) ||
        !aligned_to(weight, dtype_size(norm->wdtype)))
        return SSD_ERR_ALIGNMENT;
    if (n == 0) return SSD_OK;
    // out may replace y or z, element by element
    const Span sy(y, n, norm->y_stride, norm->dim, e), sz(z, n, norm->z_stride, norm->dim, e);
    const Span so(out, n, norm->out_stride, norm->dim, e);
    const bool out_y = out == y && norm->out_stride == norm->y_stride;
    const bool out_z = out == z && norm->out_stride == norm->z_stride;
    if (clash({so, Span(rstd, n * norm->groups, 4)},
              {out_y ? Span() : sy, out_z ? Span() : sz,
               Span(weight, norm->dim, dtype_size(norm->wdtype))}))
        return SSD_ERR_INVALID_ARG;
    const void* ptrs[3] = {y, z, out};
    const size_t sizes[3] = {e, e, e};
    const long long strides[4] = {norm->dim / norm->groups, norm->y_stride, norm->z_stride,
                                  norm->out_stride};
    RowPlan p;
    if (!plan_row(norm->dim / norm->groups, common_vec(most_vec(norm), strides, 4, ptrs, sizes, 3),
                  fwd_cost(norm), &p))
        return SSD_ERR_UNSUPPORTED;
    GatedArgs a = {};
    fill_args(norm, p, &a);
    if (!a.status) return SSD_ERR_CUDA;
    a.y = y, a.z = z, a.w = weight, a.out = out, a.rstd = rstd;
    a.nrb = gated_blocks(n, norm->groups, p);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("gated_norm_fwd");
    cudaError_t err = launch_gated<false>(norm, p, (unsigned)a.nrb * norm->groups, a, L.stream);
    const cudaError_t last = L.end();
    if (err == cudaSuccess) err = last;
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_gated_norm_workspace_size(const ssd_gated_norm_t* norm, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    ssd_status_t st = check_gated(norm);
    if (st != SSD_OK) return st;
    const int n = norm->dim / norm->groups;
    size_t most = 256;
    bool any = false;
    for (int vec = most_vec(norm); vec >= 1; vec = vec > 2 ? 2 : vec - 1) {  // any may run, by the pointers' alignment
        RowPlan p;
        if (n % vec || !plan_row(n, vec, bwd_cost(norm), &p)) continue;
        any = true;
        const size_t b = sizeof(float) * (size_t)gated_blocks(norm->rows, norm->groups, p) * norm->dim;
        if (b > most) most = b;
    }
    if (!any) return SSD_ERR_UNSUPPORTED;
    *bytes = (most + 255) / 256 * 256;
    return SSD_OK;
}

ssd_status_t ssd_gated_norm_backward(const ssd_gated_norm_t* norm, const void* dout, const void* y,
                                     const void* z, const void* weight, const float* rstd,
                                     void* dy, void* dz, void* d_weight, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    set_last_launches(0);
    ssd_status_t st = check_gated(norm);
    if (st != SSD_OK) return st;
    if (!weight || !d_weight) return SSD_ERR_INVALID_ARG;
    const long long n = norm->rows;
    if (n > 0 && (!dout || !y || !z || !rstd || !dy || !dz)) return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(norm->dtype);
    const size_t we = dtype_size(norm->wdtype);
    if (!aligned_to(dout, e) || !aligned_to(y, e) || !aligned_to(z, e) || !aligned_to(dy, e) ||
        !aligned_to(dz, e) || !aligned_to(rstd, 4) || !aligned_to(weight, we) ||
        !aligned_to(d_weight, we))
        return SSD_ERR_ALIGNMENT;
    size_t need = 0;
    st = ssd_gated_norm_workspace_size(norm, &need);
    if (st != SSD_OK) return st;
    // outputs may replace inputs element by element; any other overlap is refused
    const int D = norm->dim;
    auto in = [&](const void* p, long long stride) {
        const bool replaced = (p == dy && stride == norm->dy_stride) || (p == dz && stride == norm->dz_stride);
        return replaced ? Span() : Span(p, n, stride, D, e);
    };
    if (clash({Span(dy, n, norm->dy_stride, D, e), Span(dz, n, norm->dz_stride, D, e),
               Span(d_weight, D, we), Span(workspace, need, 1)},
              {in(dout, norm->out_stride), in(y, norm->y_stride), in(z, norm->z_stride),
               Span(weight, D, we), Span(rstd, n * norm->groups, 4)}))
        return SSD_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return SSD_ERR_ALIGNMENT;
    const void* ptrs[5] = {dout, y, z, dy, dz};
    const size_t sizes[5] = {e, e, e, e, e};
    const long long strides[6] = {norm->dim / norm->groups, norm->y_stride, norm->z_stride,
                                  norm->out_stride, norm->dy_stride, norm->dz_stride};
    RowPlan p;
    if (!plan_row(norm->dim / norm->groups, common_vec(most_vec(norm), strides, 6, ptrs, sizes, 5),
                  bwd_cost(norm), &p))
        return SSD_ERR_UNSUPPORTED;
    GatedArgs a = {};
    fill_args(norm, p, &a);
    if (!a.status) return SSD_ERR_CUDA;
    a.dout = dout, a.y = y, a.z = z, a.w = weight, a.rstd_in = rstd, a.dy = dy, a.dz = dz;
    a.partial = static_cast<float*>(workspace);
    a.nrb = gated_blocks(n, norm->groups, p);
    const unsigned grid = (unsigned)a.nrb * norm->groups;
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (grid > 0) {
        L.begin("gated_norm_bwd");
        err = launch_gated<true>(norm, p, grid, a, L.stream);
        const cudaError_t last = L.end();
        if (err == cudaSuccess) err = last;
    }
    if (err == cudaSuccess) {
        ReduceDst d = {};
        d.dst[0] = d_weight, d.step[0] = 1;
        err = launch_partial_sum(a.partial, a.nrb, 1, norm->dim, d, norm->wdtype, L);
    }
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
