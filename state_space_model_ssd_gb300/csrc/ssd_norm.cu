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

// The inputs of one row, thread by thread, on their way: through the ring (S stages) or, in
// single elements (S = 0), through registers one row ahead.
template <typename T, typename TR, int VEC, int NV, int S>
struct FwdRow {
    Pack<T, VEC> nx[S ? 1 : NV];
    Pack<TR, VEC> nr[S ? 1 : NV];
    char* ring;
    int thr, nthr;
    static constexpr int xb = VEC * (int)sizeof(T), rb = VEC * (int)sizeof(TR);
    __device__ __forceinline__ char* at(int stage, int i) const {
        return ring + (size_t)(stage * NV + i) * nthr * (xb + rb);
    }
    __device__ __forceinline__ void load(const NormArgs& a, const Team& t, long long row, int stage) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (row < a.rows && c < a.D) {
                const T* x = static_cast<const T*>(a.x) + row * a.xs + c;
                const TR* r = static_cast<const TR*>(a.res) + row * a.rs + c;
                if constexpr (S > 0) {
                    char* p = at(stage, i);
                    Slot<T, VEC>::copy(p, thr, nthr, x);
                    if (a.res) Slot<TR, VEC>::copy(p + nthr * xb, thr, nthr, r);
                } else {
                    nx[i].load(x);
                    if (a.res) nr[i].load(r);
                }
            }
        }
        if constexpr (S > 0) cp_async_commit();
    }
    // vector i of x and (res) of the residual
    __device__ __forceinline__ void get(int stage, int i, bool res, float* x, float* r) const {
        if constexpr (S > 0) {
            const char* p = at(stage, i);
            Slot<T, VEC>::read(p, thr, nthr, x);
            if (res) Slot<TR, VEC>::read(p + nthr * xb, thr, nthr, r);
        } else {
            nx[i].get(x);
            if (res) nr[i].get(r);
        }
    }
};

template <typename T, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(team_threads(VEC)) norm_fwd_kernel(const NormArgs a) {
    constexpr int S = ring_stages(VEC, NV);
    __shared__ float buf[2][32];
    extern __shared__ __align__(16) char ring[];
    const Team t = team_of(a.nw);
    float w[NV][VEC], b[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c < a.D) {
            params<VEC>(a.w, c, a.wbf16, w[i]);
            if (a.b) params<VEC>(a.b, c, a.wbf16, b[i]);
        }
        if (c >= a.D || !a.b)
#pragma unroll
            for (int e = 0; e < VEC; ++e) b[i][e] = 0.f;
    }
    const long long step = (long long)gridDim.x * a.teams;
    long long row = (long long)blockIdx.x * a.teams + t.id;
    FwdRow<T, TR, VEC, NV, S> in;
    in.ring = ring, in.thr = threadIdx.x, in.nthr = blockDim.x;
#pragma unroll
    for (int s = 0; s < (S ? S : 1); ++s) in.load(a, t, row + s * step, s);
    int stage = 0, flip = 0;
    // every team of the block takes the same number of rows (some of them beyond the last)
    for (long long first = (long long)blockIdx.x * a.teams; first < a.rows; first += step) {
        if constexpr (S > 0) cp_async_wait<(S ? S - 1 : 0)>();
        const bool on = row < a.rows;
        float v[NV][VEC];
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (on && c < a.D) {
                float r[VEC];
                in.get(stage, i, a.res != nullptr, v[i], r);
                if (a.res) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[i][e] += r[e];
                    store_vec<VEC>(static_cast<TR*>(a.h) + row * a.hs + c, v[i]);
                }
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += v[i][e];
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
            }
        }
        // this thread's places of the stage are read: the row S rounds on takes them
        in.load(a, t, row + (S ? S : 1) * step, stage);
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
        // rms rows take the two buffers in turn
        team_sum<1>(t, &q, buf[a.layer ? 1 : flip]);
        const float rstd = 1.f / sqrtf(q / a.D + a.eps);
        if (on) {
            if (t.thread == 0 && a.stats) a.stats[row] = make_float2(mean, rstd);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t.thread + i * a.nw * 32) * VEC;
                if (c >= a.D) continue;
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    o[e] = fmaf((v[i][e] - mean) * rstd, w[i][e], b[i][e]);
                store_vec<VEC>(static_cast<T*>(a.y) + row * a.ys + c, o);
            }
        }
        flip ^= 1;
        row += step;
        if (S > 1) stage = stage + 1 == S ? 0 : stage + 1;
    }
}

// The same for the backward: dy, h and (dh) the residual stream's gradient.
template <typename T, typename TR, int VEC, int NV, int S>
struct BwdRow {
    Pack<T, VEC> ndy[S ? 1 : NV];
    Pack<TR, VEC> nh[S ? 1 : NV], ndh[S ? 1 : NV];
    char* ring;
    int thr, nthr;
    static constexpr int db = VEC * (int)sizeof(T), hb = VEC * (int)sizeof(TR);
    __device__ __forceinline__ char* at(int stage, int i) const {
        return ring + (size_t)(stage * NV + i) * nthr * (db + 2 * hb);
    }
    __device__ __forceinline__ void load(const NormArgs& a, const Team& t, long long row, int stage) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (row < a.rows && c < a.D) {
                const T* dy = static_cast<const T*>(a.dy) + row * a.ys + c;
                const TR* h = static_cast<const TR*>(a.hin) + row * a.hs + c;
                const TR* dh = static_cast<const TR*>(a.dh) + row * a.rs + c;
                if constexpr (S > 0) {
                    char* p = at(stage, i);
                    Slot<T, VEC>::copy(p, thr, nthr, dy);
                    Slot<TR, VEC>::copy(p + nthr * db, thr, nthr, h);
                    if (a.dh) Slot<TR, VEC>::copy(p + nthr * (db + hb), thr, nthr, dh);
                } else {
                    ndy[i].load(dy);
                    nh[i].load(h);
                    if (a.dh) ndh[i].load(dh);
                }
            }
        }
        if constexpr (S > 0) cp_async_commit();
    }
    __device__ __forceinline__ void get(int stage, int i, float* dy, float* h) const {
        if constexpr (S > 0) {
            Slot<T, VEC>::read(at(stage, i), thr, nthr, dy);
            Slot<TR, VEC>::read(at(stage, i) + nthr * db, thr, nthr, h);
        } else {
            ndy[i].get(dy);
            nh[i].get(h);
        }
    }
    __device__ __forceinline__ void get_dh(int stage, int i, float* dh) const {
        if constexpr (S > 0)
            Slot<TR, VEC>::read(at(stage, i) + nthr * (db + hb), thr, nthr, dh);
        else
            ndh[i].get(dh);
    }
};

template <typename T, typename TR, int VEC, int NV>
__global__ void __launch_bounds__(team_threads(VEC)) norm_bwd_kernel(const NormArgs a) {
    constexpr int S = ring_stages(VEC, NV);
    __shared__ float buf[2][64];
    extern __shared__ __align__(16) char ring[];
    const Team t = team_of(a.nw);
    float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t.thread + i * a.nw * 32) * VEC;
        if (c < a.D) params<VEC>(a.w, c, a.wbf16, w[i]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) dw[i][e] = db[i][e] = 0.f;
    }
    const long long step = (long long)gridDim.x * a.teams;
    long long row = (long long)blockIdx.x * a.teams + t.id;
    BwdRow<T, TR, VEC, NV, S> in;
    in.ring = ring, in.thr = threadIdx.x, in.nthr = blockDim.x;
#pragma unroll
    for (int s = 0; s < (S ? S : 1); ++s) in.load(a, t, row + s * step, s);
    float2 next = row < a.rows ? a.stats_in[row] : make_float2(0.f, 0.f);
    int stage = 0, flip = 0;
    // every team of the block takes the same number of rows (some of them beyond the last)
    for (long long first = (long long)blockIdx.x * a.teams; first < a.rows; first += step) {
        const float2 st = next;
        next = row + step < a.rows ? a.stats_in[row + step] : make_float2(0.f, 0.f);
        if constexpr (S > 0) cp_async_wait<(S ? S - 1 : 0)>();
        const bool on = row < a.rows;
        float xh[NV][VEC], d[NV][VEC], g[NV][VEC];
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t.thread + i * a.nw * 32) * VEC;
            if (on && c < a.D) {
                in.get(stage, i, d[i], xh[i]);
                if (a.dh) in.get_dh(stage, i, g[i]);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    xh[i][e] = (xh[i][e] - st.x) * st.y;
                    dw[i][e] = fmaf(d[i][e], xh[i][e], dw[i][e]);
                    db[i][e] += d[i][e];
                    d[i][e] *= w[i][e];
                    sum[0] += d[i][e];
                    sum[1] = fmaf(d[i][e], xh[i][e], sum[1]);
                }
            }
        }
        // this thread's places of the stage are read: the row S rounds on takes them
        in.load(a, t, row + (S ? S : 1) * step, stage);
        team_sum<2>(t, sum, buf[flip]);
        flip ^= 1;
        const float c1 = a.layer ? sum[0] / a.D : 0.f, c2 = sum[1] / a.D;
        if (on) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t.thread + i * a.nw * 32) * VEC;
                if (c >= a.D) continue;
                float o[VEC];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    o[e] = (d[i][e] - c1 - xh[i][e] * c2) * st.y;
                    if (a.dh) o[e] += g[i][e];
                }
                store_vec<VEC>(static_cast<T*>(a.dx) + row * a.xs + c, o);
                if (a.dres) store_vec<VEC>(static_cast<TR*>(a.dres) + row * a.D + c, o);
            }
        }
        row += step;
        if (S > 1) stage = stage + 1 == S ? 0 : stage + 1;
    }
    float* part = a.partial + (long long)blockIdx.x * a.nk * a.D;
    if (a.teams > 1) {  // the teams' sums are joined in order, in the ring's place
        if constexpr (S > 0) cp_async_wait<0>();
        float* acc = reinterpret_cast<float*>(ring);
        __syncthreads();
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
        for (int i = threadIdx.x; i < a.nk * a.D; i += blockDim.x) part[i] = acc[i];
        return;
    }
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

// Bytes of a column that a forward (x, residual) and a backward (dy, h, dh) read.
int fwd_col(const ssd_norm_t* p) { return (int)(dtype_size(p->dtype) + dtype_size(p->rdtype)); }
int bwd_col(const ssd_norm_t* p) { return (int)(dtype_size(p->dtype) + 2 * dtype_size(p->rdtype)); }
constexpr int kFwdRegs[2] = {28, 4}, kBwdRegs[2] = {40, 6};
int most_vec(const ssd_norm_t* p) { return p->dtype == SSD_DTYPE_BF16 ? 8 : 4; }

int row_vec(const ssd_norm_t* p, const void* const* ptrs, const size_t* sizes, int np) {
    const long long strides[5] = {p->dim, p->x_stride, p->r_stride, p->h_stride, p->y_stride};
    return common_vec(most_vec(p), strides, 5, ptrs, sizes, np);
}

// Shared memory of a block: the ring, or the sums of several teams at the end.
size_t fwd_smem(const RowPlan& p) { return p.ring; }
size_t bwd_smem(const RowPlan& p, int dim) {
    const size_t sums = p.teams > 1 ? sizeof(float) * 2 * dim : 0;
    return p.ring > sums ? p.ring : sums;
}

template <typename T, typename TR, int VEC, int NV>
cudaError_t launch_fwd_nv(const RowPlan& p, unsigned grid, const NormArgs& a, cudaStream_t s) {
    const cudaError_t e = allow_smem<&norm_fwd_kernel<T, TR, VEC, NV>>(fwd_smem(p));
    if (e == cudaSuccess)
        norm_fwd_kernel<T, TR, VEC, NV><<<grid, p.threads(), fwd_smem(p), s>>>(a);
    return e;
}
template <typename T, typename TR, int VEC, int NV>
cudaError_t launch_bwd_nv(const RowPlan& p, unsigned grid, const NormArgs& a, cudaStream_t s) {
    const cudaError_t e = allow_smem<&norm_bwd_kernel<T, TR, VEC, NV>>(bwd_smem(p, a.D));
    if (e == cudaSuccess)
        norm_bwd_kernel<T, TR, VEC, NV><<<grid, p.threads(), bwd_smem(p, a.D), s>>>(a);
    return e;
}
template <typename T, typename TR, int VEC>
cudaError_t launch_vec(bool bwd, const RowPlan& p, unsigned grid, const NormArgs& a,
                       cudaStream_t s) {
    if (p.nv == 1)
        return bwd ? launch_bwd_nv<T, TR, VEC, 1>(p, grid, a, s)
                   : launch_fwd_nv<T, TR, VEC, 1>(p, grid, a, s);
    if (p.nv == 2)
        return bwd ? launch_bwd_nv<T, TR, VEC, 2>(p, grid, a, s)
                   : launch_fwd_nv<T, TR, VEC, 2>(p, grid, a, s);
    if (p.nv == 4)
        return bwd ? launch_bwd_nv<T, TR, VEC, 4>(p, grid, a, s)
                   : launch_fwd_nv<T, TR, VEC, 4>(p, grid, a, s);
    if constexpr (most_vectors(VEC, sizeof(T)) == 8)
        return bwd ? launch_bwd_nv<T, TR, VEC, 8>(p, grid, a, s)
                   : launch_fwd_nv<T, TR, VEC, 8>(p, grid, a, s);
    return cudaErrorInvalidValue;
}
template <typename T, typename TR>
cudaError_t launch_types(bool bwd, const RowPlan& p, unsigned grid, const NormArgs& a,
                         cudaStream_t s) {
    if constexpr (sizeof(T) == 2)
        if (p.vec == 8) return launch_vec<T, TR, 8>(bwd, p, grid, a, s);
    if (p.vec == 4) return launch_vec<T, TR, 4>(bwd, p, grid, a, s);
    if (p.vec == 2) return launch_vec<T, TR, 2>(bwd, p, grid, a, s);
    return launch_vec<T, TR, 1>(bwd, p, grid, a, s);
}
cudaError_t launch_norm(const ssd_norm_t* n, bool bwd, const RowPlan& p, unsigned grid,
                        const NormArgs& a, cudaStream_t s) {
    if (n->dtype == SSD_DTYPE_F32) return launch_types<float, float>(bwd, p, grid, a, s);
    if (n->rdtype == SSD_DTYPE_F32) return launch_types<__nv_bfloat16, float>(bwd, p, grid, a, s);
    return launch_types<__nv_bfloat16, __nv_bfloat16>(bwd, p, grid, a, s);
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
    const void* ptrs[4] = {x, y, residual, h};
    const size_t sizes[4] = {e, e, re, re};
    RowPlan p;
    if (!plan_row(D, row_vec(norm, ptrs, sizes, 4), most_vec(norm), fwd_col(norm), kFwdRegs, &p))
        return SSD_ERR_UNSUPPORTED;
    NormArgs a = {};
    a.x = x, a.res = residual, a.w = weight, a.b = bias, a.y = y, a.h = h;
    a.stats = reinterpret_cast<float2*>(stats);
    a.rows = n, a.xs = norm->x_stride, a.rs = norm->r_stride, a.hs = norm->h_stride,
    a.ys = norm->y_stride;
    a.D = D, a.nw = p.nw, a.teams = p.teams;
    a.layer = norm->kind == SSD_NORM_LAYER, a.wbf16 = norm->wdtype == SSD_DTYPE_BF16;
    a.eps = norm->eps;
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("norm_fwd");
    cudaError_t err = launch_norm(norm, false, p, (unsigned)team_blocks(n, p), a, L.stream);
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
    for (int vec = most_vec(norm); vec >= 1; vec >>= 1) {  // any may run, by the pointers' alignment
        RowPlan p;
        if (norm->dim % vec || !plan_row(norm->dim, vec, most_vec(norm), bwd_col(norm), kBwdRegs, &p)) continue;
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
    if ((sdx.overlaps(sdy) && !dx_dy) || (sdx.overlaps(sdh) && !dx_dh) || sdx.overlaps(sh) ||
        sdx.overlaps(sdr) || sdr.overlaps(sdy) || sdr.overlaps(sh) || (sdr.overlaps(sdh) && !dr_dh))
        return SSD_ERR_INVALID_ARG;
    size_t need = 0;
    st = ssd_norm_workspace_size(norm, &need);
    if (st != SSD_OK) return st;
    if (!workspace || workspace_bytes < need) return SSD_ERR_WORKSPACE;
    if (!aligned_to(workspace, 256)) return SSD_ERR_ALIGNMENT;
    const void* ptrs[5] = {dy, dx, h, dh, d_residual};
    const size_t sizes[5] = {e, e, re, re, re};
    RowPlan p;
    if (!plan_row(D, row_vec(norm, ptrs, sizes, 5), most_vec(norm), bwd_col(norm), kBwdRegs, &p))
        return SSD_ERR_UNSUPPORTED;
    NormArgs a = {};
    a.dy = dy, a.hin = h, a.dh = dh, a.w = weight, a.dx = dx, a.dres = d_residual;
    a.stats_in = reinterpret_cast<const float2*>(stats);
    a.partial = static_cast<float*>(workspace);
    a.rows = n, a.xs = norm->x_stride, a.rs = norm->r_stride, a.hs = norm->h_stride,
    a.ys = norm->y_stride;
    a.D = D, a.nw = p.nw, a.teams = p.teams;
    a.layer = norm->kind == SSD_NORM_LAYER, a.wbf16 = norm->wdtype == SSD_DTYPE_BF16;
    a.nk = d_bias ? 2 : 1;
    const int blocks = team_blocks(n, p);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (blocks > 0) {
        L.begin("norm_bwd");
        err = launch_norm(norm, true, p, (unsigned)blocks, a, L.stream);
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
