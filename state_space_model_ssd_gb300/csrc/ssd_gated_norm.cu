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
    int nw, teams;
    int nrb;       // blocks of a group
    int wbf16;
    float eps;
};

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(team_threads(VEC)) gated_fwd_kernel(const GatedArgs a) {
    __shared__ float buf[32];
    const Team t = team_of(a.nw);
    const int g = blockIdx.x % a.G;
    const long long row = (long long)(blockIdx.x / a.G) * a.teams + t.id;
    const bool in = row < a.rows;
    const int g0 = g * a.n;
    float v[NV][VEC];
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
        if (in && c < a.n) {
            Pack<T, VEC> py, pz;
            py.load(static_cast<const T*>(a.y) + row * a.ys + g0 + c);
            pz.load(static_cast<const T*>(a.z) + row * a.zs + g0 + c);
            float z[VEC];
            py.get(v[i]);
            pz.get(z);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[i][e] *= z[e] * sigmoid_of<T>(z[e]);
                q = fmaf(v[i][e], v[i][e], q);
            }
        }
    }
    team_sum<1>(t, &q, buf);
    const float rstd = 1.f / sqrtf(q / a.n + a.eps);
    if (!in) return;
    if (t.thread == 0 && a.rstd) a.rstd[row * a.G + g] = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c >= a.n) continue;
        float o[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = v[i][e] * rstd * param(a.w, g0 + c + e, a.wbf16);
        store_vec<VEC>(static_cast<T*>(a.out) + row * a.os + g0 + c, o);
    }
}

template <typename T, int VEC, int NV>
struct GatedRow {
    Pack<T, VEC> d[NV], y[NV], z[NV];
    float rstd;
    __device__ __forceinline__ void load(const GatedArgs& a, const Team& t, int g, long long row) {
        rstd = row < a.rows ? a.rstd_in[row * a.G + g] : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (row < a.rows && c < a.n) {
                d[i].load(static_cast<const T*>(a.dout) + row * a.os + g * a.n + c);
                y[i].load(static_cast<const T*>(a.y) + row * a.ys + g * a.n + c);
                z[i].load(static_cast<const T*>(a.z) + row * a.zs + g * a.n + c);
            } else {
                d[i].zero(), y[i].zero(), z[i].zero();
            }
        }
    }
};

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(team_threads(VEC)) gated_bwd_kernel(const GatedArgs a) {
    __shared__ float buf[2][32];
    extern __shared__ float acc[];  // several teams: their sums, joined at the end
    const Team t = team_of(a.nw);
    const int g = blockIdx.x % a.G, rb = blockIdx.x / a.G;
    const int g0 = g * a.n;
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[i][e] = c < a.n ? param(a.w, g0 + c + e, a.wbf16) : 0.f;
            dw[i][e] = 0.f;
        }
    }
    const long long step = (long long)a.nrb * a.teams;
    GatedRow<T, VEC, NV> cur, next;
    long long row = (long long)rb * a.teams + t.id;
    next.load(a, t, g, row);
    int flip = 0;
    for (long long first = (long long)rb * a.teams; first < a.rows; first += step) {
        cur = next;
        next.load(a, t, g, row + step);
        float d[NV][VEC], xh[NV][VEC];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float y[VEC], z[VEC];
            cur.d[i].get(d[i]);
            cur.y[i].get(y);
            cur.z[i].get(z);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                xh[i][e] = y[e] * (z[e] * sigmoid_of<T>(z[e])) * cur.rstd;
                dw[i][e] = fmaf(d[i][e], xh[i][e], dw[i][e]);
                d[i][e] *= w[i][e];
                sum = fmaf(d[i][e], xh[i][e], sum);
            }
        }
        team_sum<1>(t, &sum, buf[flip]);
        flip ^= 1;
        const float c2 = sum / a.n;
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t.thread + i * a.nw * 32) * VEC;
                if (c >= a.n) continue;
                float y[VEC], z[VEC], oy[VEC], oz[VEC];
                cur.y[i].get(y);
                cur.z[i].get(z);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float s = sigmoid_of<T>(z[e]);
                    const float dv = (d[i][e] - xh[i][e] * c2) * cur.rstd;
                    oy[e] = dv * (z[e] * s);
                    oz[e] = dv * y[e] * (s * fmaf(z[e], 1.f - s, 1.f));
                }
                store_vec<VEC>(static_cast<T*>(a.dy) + row * a.dys + g0 + c, oy);
                store_vec<VEC>(static_cast<T*>(a.dz) + row * a.dzs + g0 + c, oz);
            }
        }
        row += step;
    }
    float* part = a.partial + (long long)rb * a.D + g0;
    if (a.teams > 1) {
        for (int k = 0; k < a.teams; ++k) {
            if (t.id == k)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = (t.thread + i * a.nw * 32) * VEC;
                    if (c >= a.n) continue;
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        acc[c + e] = k == 0 ? dw[i][e] : acc[c + e] + dw[i][e];
                }
            __syncthreads();
        }
        for (int i = threadIdx.x; i < a.n; i += blockDim.x) part[i] = acc[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c < a.n) store_vec<VEC>(part + c, dw[i]);
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
    if (p->rows > INT_MAX || p->rows * p->groups > INT_MAX) return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}

int gated_vec(const ssd_gated_norm_t* p, const void* const* ptrs, int np) {
    const int vec = p->dtype == SSD_DTYPE_BF16 ? 8 : 4;
    if ((p->dim / p->groups) % vec || p->y_stride % vec || p->z_stride % vec ||
        p->out_stride % vec || p->dy_stride % vec || p->dz_stride % vec)
        return 1;
    for (int i = 0; i < np; ++i)
        if (!aligned_to(ptrs[i], 16)) return 1;
    return vec;
}

// Blocks of one group in the backward.
int gated_blocks(long long rows, int groups, const RowPlan& p) {
    const int per_sm = 1024 / (p.nw * p.teams * 32);
    long long most = ((long long)sm_count() * (per_sm < 1 ? 1 : per_sm) + groups - 1) / groups;
    const long long want = (rows + p.teams - 1) / p.teams;
    return (int)(want < most ? want : most);
}

template <typename T, int VEC>
void launch_fwd(const RowPlan& p, unsigned grid, const GatedArgs& a, cudaStream_t s) {
    const int threads = p.nw * p.teams * 32;
    if (p.nv == 1)
        gated_fwd_kernel<T, VEC, 1><<<grid, threads, 0, s>>>(a);
    else if (p.nv == 2)
        gated_fwd_kernel<T, VEC, 2><<<grid, threads, 0, s>>>(a);
    else if (p.nv == 4)
        gated_fwd_kernel<T, VEC, 4><<<grid, threads, 0, s>>>(a);
    else if constexpr (VEC < 8)
        gated_fwd_kernel<T, VEC, 8><<<grid, threads, 0, s>>>(a);
}
template <typename T, int VEC>
void launch_bwd(const RowPlan& p, unsigned grid, const GatedArgs& a, cudaStream_t s) {
    const int threads = p.nw * p.teams * 32;
    const size_t smem = p.teams > 1 ? sizeof(float) * a.n : 0;
    if (p.nv == 1)
        gated_bwd_kernel<T, VEC, 1><<<grid, threads, smem, s>>>(a);
    else if (p.nv == 2)
        gated_bwd_kernel<T, VEC, 2><<<grid, threads, smem, s>>>(a);
    else if (p.nv == 4)
        gated_bwd_kernel<T, VEC, 4><<<grid, threads, smem, s>>>(a);
    else if constexpr (VEC < 8)
        gated_bwd_kernel<T, VEC, 8><<<grid, threads, smem, s>>>(a);
}

void fill_args(const ssd_gated_norm_t* g, const RowPlan& p, GatedArgs* a) {
    a->rows = g->rows;
    a->ys = g->y_stride, a->zs = g->z_stride, a->os = g->out_stride;
    a->dys = g->dy_stride, a->dzs = g->dz_stride;
    a->D = g->dim, a->G = g->groups, a->n = g->dim / g->groups;
    a->nw = p.nw, a->teams = p.teams;
    a->wbf16 = g->wdtype == SSD_DTYPE_BF16;
    a->eps = g->eps;
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
    if ((so.overlaps(sy) && !(out == y && norm->out_stride == norm->y_stride)) ||
        (so.overlaps(sz) && !(out == z && norm->out_stride == norm->z_stride)))
        return SSD_ERR_INVALID_ARG;
    const void* ptrs[3] = {y, z, out};
    RowPlan p;
    if (!plan_row(norm->dim / norm->groups, gated_vec(norm, ptrs, 3), &p))
        return SSD_ERR_UNSUPPORTED;
    GatedArgs a = {};
    fill_args(norm, p, &a);
    a.y = y, a.z = z, a.w = weight, a.out = out, a.rstd = rstd;
    const unsigned grid = (unsigned)((n + p.teams - 1) / p.teams * norm->groups);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("gated_norm_fwd");
    if (norm->dtype == SSD_DTYPE_F32)
        p.vec > 1 ? launch_fwd<float, 4>(p, grid, a, L.stream)
                  : launch_fwd<float, 1>(p, grid, a, L.stream);
    else
        p.vec > 1 ? launch_fwd<__nv_bfloat16, 8>(p, grid, a, L.stream)
                  : launch_fwd<__nv_bfloat16, 1>(p, grid, a, L.stream);
    const cudaError_t err = L.end();
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_gated_norm_workspace_size(const ssd_gated_norm_t* norm, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    ssd_status_t st = check_gated(norm);
    if (st != SSD_OK) return st;
    const int n = norm->dim / norm->groups;
    size_t most = 256;
    const int vecs[2] = {norm->dtype == SSD_DTYPE_BF16 ? 8 : 4, 1};
    bool any = false;
    for (int vec : vecs) {
        RowPlan p;
        if ((vec > 1 && n % vec) || !plan_row(n, vec, &p)) continue;
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
    // outputs may replace inputs element by element; any other overlap is refused
    struct Side {
        const void* p;
        long long stride;
    };
    const Side ins[3] = {{dout, norm->out_stride}, {y, norm->y_stride}, {z, norm->z_stride}};
    const Side os[2] = {{dy, norm->dy_stride}, {dz, norm->dz_stride}};
    for (const Side& o : os) {
        const Span so(o.p, n, o.stride, norm->dim, e);
        for (const Side& i : ins)
            if (so.overlaps(Span(i.p, n, i.stride, norm->dim, e)) &&
                !(o.p == i.p && o.stride == i.stride))
                return SSD_ERR_INVALID_ARG;
    }
    if (Span(dy, n, norm->dy_stride, norm->dim, e).overlaps(Span(dz, n, norm->dz_stride, norm->dim, e)))
        return SSD_ERR_INVALID_ARG;
    size_t need = 0;
    st = ssd_gated_norm_workspace_size(norm, &need);
    if (st != SSD_OK) return st;
    if (!workspace || workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return SSD_ERR_ALIGNMENT;
    const void* ptrs[5] = {dout, y, z, dy, dz};
    RowPlan p;
    if (!plan_row(norm->dim / norm->groups, gated_vec(norm, ptrs, 5), &p))
        return SSD_ERR_UNSUPPORTED;
    GatedArgs a = {};
    fill_args(norm, p, &a);
    a.dout = dout, a.y = y, a.z = z, a.w = weight, a.rstd_in = rstd, a.dy = dy, a.dz = dz;
    a.partial = static_cast<float*>(workspace);
    a.nrb = gated_blocks(n, norm->groups, p);
    const unsigned grid = (unsigned)a.nrb * norm->groups;
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (grid > 0) {
        L.begin("gated_norm_bwd");
        if (norm->dtype == SSD_DTYPE_F32)
            p.vec > 1 ? launch_bwd<float, 4>(p, grid, a, L.stream)
                      : launch_bwd<float, 1>(p, grid, a, L.stream);
        else
            p.vec > 1 ? launch_bwd<__nv_bfloat16, 8>(p, grid, a, L.stream)
                      : launch_bwd<__nv_bfloat16, 1>(p, grid, a, L.stream);
        err = L.end();
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
