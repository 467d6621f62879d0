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

// The N tensors of one row, thread by thread, on their way: through the ring (S stages) or, in
// single elements (S = 0), through registers one row ahead.
template <typename T, int VEC, int NV, int S, int N>
struct Rows {
    Pack<T, VEC> next[S ? 1 : NV][N];
    const T* src[N];         // this thread's first element of row 0
    long long stride[N];
    char* ring;
    int thr, nthr;
    static constexpr int bytes = VEC * (int)sizeof(T);
    __device__ __forceinline__ char* at(int stage, int i, int k) const {
        return ring + ((size_t)(stage * NV + i) * N + k) * nthr * bytes;
    }
    __device__ __forceinline__ void load(const GatedArgs& a, const Team& t, long long row, int stage) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (row < a.rows && c < a.n)
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    const T* p = src[k] + row * stride[k] + c;
                    if constexpr (S > 0)
                        Slot<T, VEC>::copy(at(stage, i, k), thr, nthr, p);
                    else
                        next[i][k].load(p);
                }
        }
        if constexpr (S > 0) cp_async_commit();
    }
    __device__ __forceinline__ void get(int stage, int i, int k, float* f) const {
        if constexpr (S > 0)
            Slot<T, VEC>::read(at(stage, i, k), thr, nthr, f);
        else
            next[i][k].get(f);
    }
};

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(team_threads(VEC)) gated_fwd_kernel(const GatedArgs a) {
    constexpr int S = ring_stages(VEC, NV);
    __shared__ float buf[2][32];
    extern __shared__ __align__(16) char ring[];
    const Team t = team_of(a.nw);
    const int g = blockIdx.x % a.G, rb = blockIdx.x / a.G;
    const int g0 = g * a.n;
    float w[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c < a.n) params<VEC>(a.w, g0 + c, a.wbf16, w[i]);
    }
    const long long step = (long long)a.nrb * a.teams;
    long long row = (long long)rb * a.teams + t.id;
    Rows<T, VEC, NV, S, 2> in;
    in.ring = ring, in.thr = threadIdx.x, in.nthr = blockDim.x;
    in.src[0] = static_cast<const T*>(a.y) + g0, in.stride[0] = a.ys;
    in.src[1] = static_cast<const T*>(a.z) + g0, in.stride[1] = a.zs;
#pragma unroll
    for (int s = 0; s < (S ? S : 1); ++s) in.load(a, t, row + s * step, s);
    int stage = 0, flip = 0;
    // every team of the block takes the same number of rows (some of them beyond the last)
    for (long long first = (long long)rb * a.teams; first < a.rows; first += step) {
        if constexpr (S > 0) cp_async_wait<(S ? S - 1 : 0)>();
        const bool on = row < a.rows;
        float v[NV][VEC];
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (on && c < a.n) {
                float z[VEC];
                in.get(stage, i, 0, v[i]);
                in.get(stage, i, 1, z);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    v[i][e] *= z[e] * sigmoid_of<T>(z[e]);
                    q = fmaf(v[i][e], v[i][e], q);
                }
            }
        }
        // this thread's places of the stage are read: the row S rounds on takes them
        in.load(a, t, row + (S ? S : 1) * step, stage);
        team_sum<1>(t, &q, buf[flip]);
        flip ^= 1;
        const float rstd = 1.f / sqrtf(q / a.n + a.eps);
        if (on) {
            if (t.thread == 0 && a.rstd) a.rstd[row * a.G + g] = rstd;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t.thread + i * a.nw * 32) * VEC;
                if (c >= a.n) continue;
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) o[e] = v[i][e] * rstd * w[i][e];
                store_vec<VEC>(static_cast<T*>(a.out) + row * a.os + g0 + c, o);
            }
        }
        row += step;
        if (S > 1) stage = stage + 1 == S ? 0 : stage + 1;
    }
}

template <typename T, int VEC, int NV>
__global__ void __launch_bounds__(team_threads(VEC)) gated_bwd_kernel(const GatedArgs a) {
    constexpr int S = ring_stages(VEC, NV);
    __shared__ float buf[2][32];
    extern __shared__ __align__(16) char ring[];
    const Team t = team_of(a.nw);
    const int g = blockIdx.x % a.G, rb = blockIdx.x / a.G;
    const int g0 = g * a.n;
    float w[NV][VEC], dw[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c < a.n) params<VEC>(a.w, g0 + c, a.wbf16, w[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = 0.f;
    }
    const long long step = (long long)a.nrb * a.teams;
    long long row = (long long)rb * a.teams + t.id;
    Rows<T, VEC, NV, S, 3> in;
    in.ring = ring, in.thr = threadIdx.x, in.nthr = blockDim.x;
    in.src[0] = static_cast<const T*>(a.dout) + g0, in.stride[0] = a.os;
    in.src[1] = static_cast<const T*>(a.y) + g0, in.stride[1] = a.ys;
    in.src[2] = static_cast<const T*>(a.z) + g0, in.stride[2] = a.zs;
#pragma unroll
    for (int s = 0; s < (S ? S : 1); ++s) in.load(a, t, row + s * step, s);
    float next = row < a.rows ? a.rstd_in[row * a.G + g] : 0.f;
    int stage = 0, flip = 0;
    // every team of the block takes the same number of rows (some of them beyond the last)
    for (long long first = (long long)rb * a.teams; first < a.rows; first += step) {
        const float rstd = next;
        next = row + step < a.rows ? a.rstd_in[(row + step) * a.G + g] : 0.f;
        if constexpr (S > 0) cp_async_wait<(S ? S - 1 : 0)>();
        const bool on = row < a.rows;
        // d = w dout, gate = silu(z), gy = y silu'(z)
        float d[NV][VEC], xh[NV][VEC], gate[NV][VEC], gy[NV][VEC];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (on && c < a.n) {
                float y[VEC], z[VEC];
                in.get(stage, i, 0, d[i]);
                in.get(stage, i, 1, y);
                in.get(stage, i, 2, z);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float s = sigmoid_of<T>(z[e]);
                    gate[i][e] = z[e] * s;
                    gy[i][e] = y[e] * fmaf(gate[i][e], 1.f - s, s);
                    xh[i][e] = y[e] * gate[i][e] * rstd;
                    dw[i][e] = fmaf(d[i][e], xh[i][e], dw[i][e]);
                    d[i][e] *= w[i][e];
                    sum = fmaf(d[i][e], xh[i][e], sum);
                }
            }
        }
        // this thread's places of the stage are read: the row S rounds on takes them
        in.load(a, t, row + (S ? S : 1) * step, stage);
        team_sum<1>(t, &sum, buf[flip]);
        flip ^= 1;
        const float c2 = sum / a.n;
        if (on) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t.thread + i * a.nw * 32) * VEC;
                if (c >= a.n) continue;
                float oy[VEC], oz[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float dv = (d[i][e] - xh[i][e] * c2) * rstd;
                    oy[e] = dv * gate[i][e];
                    oz[e] = dv * gy[i][e];
                }
                store_vec<VEC>(static_cast<T*>(a.dy) + row * a.dys + g0 + c, oy);
                store_vec<VEC>(static_cast<T*>(a.dz) + row * a.dzs + g0 + c, oz);
            }
        }
        row += step;
        if (S > 1) stage = stage + 1 == S ? 0 : stage + 1;
    }
    float* part = a.partial + (long long)rb * a.D + g0;
    if (a.teams > 1) {  // the teams' sums are joined in order, in the ring's place
        if constexpr (S > 0) cp_async_wait<0>();
        float* acc = reinterpret_cast<float*>(ring);
        __syncthreads();
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

constexpr int kFwdRegs[2] = {32, 4}, kBwdRegs[2] = {40, 7};
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

template <typename T, int VEC, int NV>
cudaError_t launch_nv(bool bwd, const RowPlan& p, unsigned grid, const GatedArgs& a,
                      cudaStream_t s) {
    const size_t smem = bwd ? bwd_smem(p, a.n) : p.ring;
    const cudaError_t e = bwd ? allow_smem<&gated_bwd_kernel<T, VEC, NV>>(smem)
                              : allow_smem<&gated_fwd_kernel<T, VEC, NV>>(smem);
    if (e != cudaSuccess) return e;
    if (bwd)
        gated_bwd_kernel<T, VEC, NV><<<grid, p.threads(), smem, s>>>(a);
    else
        gated_fwd_kernel<T, VEC, NV><<<grid, p.threads(), smem, s>>>(a);
    return cudaSuccess;
}
template <typename T, int VEC>
cudaError_t launch_vec(bool bwd, const RowPlan& p, unsigned grid, const GatedArgs& a,
                       cudaStream_t s) {
    if (p.nv == 1) return launch_nv<T, VEC, 1>(bwd, p, grid, a, s);
    if (p.nv == 2) return launch_nv<T, VEC, 2>(bwd, p, grid, a, s);
    if (p.nv == 4) return launch_nv<T, VEC, 4>(bwd, p, grid, a, s);
    if constexpr (most_vectors(VEC, sizeof(T)) == 8) return launch_nv<T, VEC, 8>(bwd, p, grid, a, s);
    return cudaErrorInvalidValue;
}
template <typename T>
cudaError_t launch_type(bool bwd, const RowPlan& p, unsigned grid, const GatedArgs& a,
                        cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (p.vec == 8) return launch_vec<T, 8>(bwd, p, grid, a, s);
    if (p.vec == 4) return launch_vec<T, 4>(bwd, p, grid, a, s);
    if (p.vec == 2) return launch_vec<T, 2>(bwd, p, grid, a, s);
    return launch_vec<T, 1>(bwd, p, grid, a, s);
}
cudaError_t launch_gated(const ssd_gated_norm_t* n, bool bwd, const RowPlan& p, unsigned grid,
                         const GatedArgs& a, cudaStream_t s) {
    return n->dtype == SSD_DTYPE_F32 ? launch_type<float>(bwd, p, grid, a, s)
                                     : launch_type<__nv_bfloat16>(bwd, p, grid, a, s);
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
    const size_t sizes[3] = {e, e, e};
    const long long strides[4] = {norm->dim / norm->groups, norm->y_stride, norm->z_stride,
                                  norm->out_stride};
    RowPlan p;
    if (!plan_row(norm->dim / norm->groups, common_vec(most_vec(norm), strides, 4, ptrs, sizes, 3),
                  most_vec(norm), 2 * (int)e, kFwdRegs, &p))
        return SSD_ERR_UNSUPPORTED;
    GatedArgs a = {};
    fill_args(norm, p, &a);
    a.y = y, a.z = z, a.w = weight, a.out = out, a.rstd = rstd;
    a.nrb = gated_blocks(n, norm->groups, p);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("gated_norm_fwd");
    cudaError_t err = launch_gated(norm, false, p, (unsigned)a.nrb * norm->groups, a, L.stream);
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
    for (int vec = most_vec(norm); vec >= 1; vec >>= 1) {  // any may run, by the pointers' alignment
        RowPlan p;
        if (n % vec || !plan_row(n, vec, most_vec(norm), 3 * (int)dtype_size(norm->dtype), kBwdRegs, &p))
            continue;
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
    const size_t sizes[5] = {e, e, e, e, e};
    const long long strides[6] = {norm->dim / norm->groups, norm->y_stride, norm->z_stride,
                                  norm->out_stride, norm->dy_stride, norm->dz_stride};
    RowPlan p;
    if (!plan_row(norm->dim / norm->groups, common_vec(most_vec(norm), strides, 6, ptrs, sizes, 5),
                  most_vec(norm), 3 * (int)e, kBwdRegs, &p))
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
        err = launch_gated(norm, true, p, grid, a, L.stream);
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
