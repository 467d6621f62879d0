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
#include <limits.h>

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
    int D, nw, teams;
    int layer;     // 0: rms
    int wbf16;
    int nk;        // partial rows: d_weight (and d_bias)
    float eps;
};

template <typename T, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(team_threads(VEC)) norm_fwd_kernel(const NormArgs a) {
    __shared__ float buf[2][32];
    const Team t = team_of(a.nw);
    const long long row = (long long)blockIdx.x * a.teams + t.id;
    const bool in = row < a.rows;
    float v[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (in && c < a.D) {
            Pack<T, VEC> px;
            px.load(static_cast<const T*>(a.x) + row * a.xs + c);
            if (a.res) {
                Pack<TR, VEC> pr;
                pr.load(static_cast<const TR*>(a.res) + row * a.rs + c);
                float r[VEC];
                pr.get(r);
                px.get(v[i]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] += r[e];
                store_vec<VEC>(static_cast<TR*>(a.h) + row * a.hs + c, v[i]);
            } else {
                px.get(v[i]);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) s += v[i][e];
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
        }
    }
    float mean = 0.f;
    if (a.layer) {
        team_sum<1>(t, &s, buf[0]);
        mean = s / a.D;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c < a.D)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = v[i][e] - mean;
                q = fmaf(d, d, q);
            }
    }
    team_sum<1>(t, &q, buf[1]);
    const float rstd = 1.f / sqrtf(q / a.D + a.eps);
    if (!in) return;
    if (t.thread == 0 && a.stats) a.stats[row] = make_float2(mean, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c >= a.D) continue;
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            o[e] = (v[i][e] - mean) * rstd * param(a.w, c + e, a.wbf16);
            if (a.b) o[e] += param(a.b, c + e, a.wbf16);
        }
        store_vec<VEC>(static_cast<T*>(a.y) + row * a.ys + c, o);
    }
}

// One row's inputs as loaded, so that the next row's loads run under this row's sums.
template <typename T, typename TR, int VEC, int NV>
struct NormRow {
    Pack<T, VEC> dy[NV];
    Pack<TR, VEC> h[NV], dh[NV];
    float2 st;
    __device__ __forceinline__ void load(const NormArgs& a, const Team& t, long long row) {
        st = make_float2(0.f, 0.f);
        if (row < a.rows) st = a.stats_in[row];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (row < a.rows && c < a.D) {
                dy[i].load(static_cast<const T*>(a.dy) + row * a.ys + c);
                h[i].load(static_cast<const TR*>(a.hin) + row * a.hs + c);
                if (a.dh) dh[i].load(static_cast<const TR*>(a.dh) + row * a.rs + c);
            } else {
                dy[i].zero(), h[i].zero();
            }
        }
    }
};

template <typename T, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(team_threads(VEC)) norm_bwd_kernel(const NormArgs a) {
    __shared__ float buf[2][64];
    extern __shared__ float acc[];  // several teams: their sums, joined at the end
    const Team t = team_of(a.nw);
    float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[i][e] = c < a.D ? param(a.w, c + e, a.wbf16) : 0.f;
            dw[i][e] = db[i][e] = 0.f;
        }
    }
    const long long step = (long long)gridDim.x * a.teams;
    NormRow<T, TR, VEC, NV> cur, next;
    long long row = (long long)blockIdx.x * a.teams + t.id;
    next.load(a, t, row);
    int flip = 0;
    // every team of the block takes the same number of rows (some of them beyond the last)
    for (long long first = (long long)blockIdx.x * a.teams; first < a.rows; first += step) {
        cur = next;
        next.load(a, t, row + step);
        float xh[NV][VEC], d[NV][VEC];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            cur.h[i].get(xh[i]);
            cur.dy[i].get(d[i]);
            const int c = (t.thread + i * a.nw * 32) * VEC;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                xh[i][e] = c < a.D ? (xh[i][e] - cur.st.x) * cur.st.y : 0.f;
                dw[i][e] = fmaf(d[i][e], xh[i][e], dw[i][e]);
                db[i][e] += d[i][e];
                d[i][e] *= w[i][e];
                sum[0] += d[i][e];
                sum[1] = fmaf(d[i][e], xh[i][e], sum[1]);
            }
        }
        team_sum<2>(t, sum, buf[flip]);
        flip ^= 1;
        const float c1 = a.layer ? sum[0] / a.D : 0.f, c2 = sum[1] / a.D;
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t.thread + i * a.nw * 32) * VEC;
                if (c >= a.D) continue;
                float o[VEC], g[VEC];
                if (a.dh) cur.dh[i].get(g);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    o[e] = (d[i][e] - c1 - xh[i][e] * c2) * cur.st.y;
                    if (a.dh) o[e] += g[e];
                }
                store_vec<VEC>(static_cast<T*>(a.dx) + row * a.xs + c, o);
                if (a.dres) store_vec<VEC>(static_cast<TR*>(a.dres) + row * a.D + c, o);
            }
        }
        row += step;
    }
    if (a.teams > 1) {
        for (int k = 0; k < a.teams; ++k) {
            if (t.id == k)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (t.thread + i * a.nw * 32) * VEC;
                    if (c >= a.D) continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        acc[c + e] = k == 0 ? dw[i][e] : acc[c + e] + dw[i][e];
                        acc[a.D + c + e] = k == 0 ? db[i][e] : acc[a.D + c + e] + db[i][e];
                    }
                }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < a.nk * a.D; i += blockDim.x)
            a.partial[(long long)blockIdx.x * a.nk * a.D + i] = acc[i];
        return;
    }
    float* part = a.partial + (long long)blockIdx.x * a.nk * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c >= a.D) continue;
        store_vec<VEC>(part + c, dw[i]);
        if (a.nk > 1) store_vec<VEC>(part + a.D + c, db[i]);
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
    if (p->rows > INT_MAX) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

// Vector length of the rows: 16 bytes of the activations, or single elements.
int row_vec(const ssd_norm_t* p, const void* const* ptrs, int np) {
    const int vec = p->dtype == SSD_DTYPE_BF16 ? 8 : 4;
    if (p->dim % vec || p->x_stride % vec || p->r_stride % vec || p->h_stride % vec ||
        p->y_stride % vec)
        return 1;
    for (int i = 0; i < np; ++i)
        if (!aligned_to(ptrs[i], 16)) return 1;
    return vec;
}

// Blocks of the backward, each with a share of the rows and one partial sum per column.
int bwd_blocks(long long rows, const RowPlan& p) {
    const int per_sm = 1024 / (p.nw * p.teams * 32);
    const long long most = (long long)sm_count() * (per_sm < 1 ? 1 : per_sm);
    const long long want = (rows + p.teams - 1) / p.teams;
    return (int)(want < most ? want : most);
}

template <typename T, typename TR, int VEC>
void launch_fwd(const RowPlan& p, unsigned grid, const NormArgs& a, cudaStream_t s) {
    const int threads = p.nw * p.teams * 32;
    if (p.nv == 1)
        norm_fwd_kernel<T, TR, VEC, 1><<<grid, threads, 0, s>>>(a);
    else if (p.nv == 2)
        norm_fwd_kernel<T, TR, VEC, 2><<<grid, threads, 0, s>>>(a);
    else if (p.nv == 4)
        norm_fwd_kernel<T, TR, VEC, 4><<<grid, threads, 0, s>>>(a);
    else if constexpr (VEC < 8)
        norm_fwd_kernel<T, TR, VEC, 8><<<grid, threads, 0, s>>>(a);
}
template <typename T, typename TR, int VEC>
void launch_bwd(const RowPlan& p, unsigned grid, const NormArgs& a, cudaStream_t s) {
    const int threads = p.nw * p.teams * 32;
    const size_t smem = p.teams > 1 ? sizeof(float) * 2 * a.D : 0;
    if (p.nv == 1)
        norm_bwd_kernel<T, TR, VEC, 1><<<grid, threads, smem, s>>>(a);
    else if (p.nv == 2)
        norm_bwd_kernel<T, TR, VEC, 2><<<grid, threads, smem, s>>>(a);
    else if (p.nv == 4)
        norm_bwd_kernel<T, TR, VEC, 4><<<grid, threads, smem, s>>>(a);
    else if constexpr (VEC < 8)
        norm_bwd_kernel<T, TR, VEC, 8><<<grid, threads, smem, s>>>(a);
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
    if ((sy.overlaps(sx) && !same_y) || (sh.overlaps(sr) && !same_h) || sy.overlaps(sr) ||
        sh.overlaps(sx) || sy.overlaps(sh))
        return SSD_ERR_INVALID_ARG;
    const void* ptrs[4] = {x, residual, y, h};
    RowPlan p;
    if (!plan_row(D, row_vec(norm, ptrs, 4), &p)) return SSD_ERR_UNSUPPORTED;
    NormArgs a = {};
    a.x = x, a.res = residual, a.w = weight, a.b = bias, a.y = y, a.h = h;
    a.stats = reinterpret_cast<float2*>(stats);
    a.rows = n, a.xs = norm->x_stride, a.rs = norm->r_stride, a.hs = norm->h_stride,
    a.ys = norm->y_stride;
    a.D = D, a.nw = p.nw, a.teams = p.teams;
    a.layer = norm->kind == SSD_NORM_LAYER, a.wbf16 = norm->wdtype == SSD_DTYPE_BF16;
    a.eps = norm->eps;
    const unsigned grid = (unsigned)((n + p.teams - 1) / p.teams);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("norm_fwd");
    using B16 = __nv_bfloat16;
    const bool rf32 = norm->rdtype == SSD_DTYPE_F32;
    if (norm->dtype == SSD_DTYPE_F32)
        p.vec > 1 ? launch_fwd<float, float, 4>(p, grid, a, L.stream)
                  : launch_fwd<float, float, 1>(p, grid, a, L.stream);
    else if (rf32)
        p.vec > 1 ? launch_fwd<B16, float, 8>(p, grid, a, L.stream)
                  : launch_fwd<B16, float, 1>(p, grid, a, L.stream);
    else
        p.vec > 1 ? launch_fwd<B16, B16, 8>(p, grid, a, L.stream)
                  : launch_fwd<B16, B16, 1>(p, grid, a, L.stream);
    const cudaError_t err = L.end();
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_norm_workspace_size(const ssd_norm_t* norm, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    ssd_status_t st = check_norm(norm);
    if (st != SSD_OK) return st;
    size_t most = 256;
    const int wide = norm->dtype == SSD_DTYPE_BF16 ? 8 : 4;
    const int vecs[2] = {wide, 1};  // either may run, by the pointers' alignment
    bool any = false;
    for (int vec : vecs) {
        RowPlan p;
        if ((vec > 1 && norm->dim % vec) || !plan_row(norm->dim, vec, &p)) continue;
        any = true;
        const size_t n = sizeof(float) * (size_t)bwd_blocks(norm->rows, p) * 2 * norm->dim;
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
    if ((sdx.overlaps(sdy) && !dx_dy) || (sdx.overlaps(sdh) && !dx_dh) || sdx.overlaps(sh) ||
        sdx.overlaps(sdr) || sdr.overlaps(sdy) || sdr.overlaps(sh) || (sdr.overlaps(sdh) && !dr_dh))
        return SSD_ERR_INVALID_ARG;
    size_t need = 0;
    st = ssd_norm_workspace_size(norm, &need);
    if (st != SSD_OK) return st;
    if (!workspace || workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return SSD_ERR_ALIGNMENT;
    const void* ptrs[5] = {dy, h, dh, dx, d_residual};
    RowPlan p;
    if (!plan_row(D, row_vec(norm, ptrs, 5), &p)) return SSD_ERR_UNSUPPORTED;
    NormArgs a = {};
    a.dy = dy, a.hin = h, a.dh = dh, a.w = weight, a.dx = dx, a.dres = d_residual;
    a.stats_in = reinterpret_cast<const float2*>(stats);
    a.partial = static_cast<float*>(workspace);
    a.rows = n, a.xs = norm->x_stride, a.rs = norm->r_stride, a.hs = norm->h_stride,
    a.ys = norm->y_stride;
    a.D = D, a.nw = p.nw, a.teams = p.teams;
    a.layer = norm->kind == SSD_NORM_LAYER, a.wbf16 = norm->wdtype == SSD_DTYPE_BF16;
    a.nk = d_bias ? 2 : 1;
    const int blocks = bwd_blocks(n, p);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (blocks > 0) {
        L.begin("norm_bwd");
        using B16 = __nv_bfloat16;
        if (norm->dtype == SSD_DTYPE_F32)
            p.vec > 1 ? launch_bwd<float, float, 4>(p, blocks, a, L.stream)
                      : launch_bwd<float, float, 1>(p, blocks, a, L.stream);
        else if (norm->rdtype == SSD_DTYPE_F32)
            p.vec > 1 ? launch_bwd<B16, float, 8>(p, blocks, a, L.stream)
                      : launch_bwd<B16, float, 1>(p, blocks, a, L.stream);
        else
            p.vec > 1 ? launch_bwd<B16, B16, 8>(p, blocks, a, L.stream)
                      : launch_bwd<B16, B16, 1>(p, blocks, a, L.stream);
        err = L.end();
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
