// Linear attention with a decay for each head: the C entry points, the walk on the plain cores
// (any type and size), the scan over segments, and the sum of shared heads' gradients.  The
// mathematics is in linattn.cuh.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "layer_device.cuh"
#include "linattn.cuh"

namespace ssd {
namespace linattn {

namespace {

using namespace layer;

constexpr int kThreads = 256;
constexpr int kQ = 32;           // tokens of a chunk
constexpr int kVT = kSimtTile;
constexpr int kVS = kVT + 1;     // rows of shared memory one word apart from a multiple of 32

__host__ __device__ constexpr size_t simt_smem(int kd) {
    return sizeof(float) * (2 * (size_t)kQ * (kd + 1) + 2 * (size_t)kQ * kVS + (size_t)kd * kVS + kQ + 2);
}

// One segment, head and tile of v's columns: 32 tokens at a time, everything in float32 in
// shared memory, each thread a 2 x 2 piece of the 32 x 32 products and up to 4 x 4 of the state.
// Bound by shared memory: the four products read two words for two multiply-adds.  It serves
// float32 and the sizes that the tensor cores do not take.  OUT: false where only the state after
// the segment is wanted.
template <typename T, bool OUT>
__global__ void __launch_bounds__(kThreads) simt_walk_kernel(const __grid_constant__ WalkArgs a) {
    extern __shared__ float sm[];
    const long long item = blockIdx.x;
    const long long id = item / ((long long)a.tiles * a.H);
    const int rest = (int)(item - id * a.tiles * a.H);
    const int h = rest / a.tiles;
    int tile = rest - h * a.tiles;
    const Pass& p = pass_of(a, tile);
    const int v0 = tile * kVT, vw = min(kVT, p.vd - v0);
    const int tid = threadIdx.x, kd = p.kd, ks1 = kd + 1;
    float* qs = sm;
    float* ks = qs + kQ * ks1;
    float* vs = ks + kQ * ks1;
    float* sc = vs + kQ * kVS;
    float* S = sc + kQ * kVS;
    float* pw = S + kd * kVS;  // a^0 .. a^(kQ + 1)

    const T* v = static_cast<const T*>(p.v) + (long long)(h / p.vr) * p.vd + v0;
    if (OUT && a.cu) {  // tokens behind the last sequence
        for (long long t = border(a, a.nseq) + id; t < a.T; t += a.ids)
            for (int c = tid; c < vw; c += kThreads) {
                const long long o = t * p.os + (long long)(h / p.outr) * p.vd + v0 + c;
                if (p.out_f32)
                    st_out(static_cast<float*>(p.out), o, 0.f);
                else
                    st_out(static_cast<T*>(p.out), o, 0.f);
            }
    }
    const Seg g = segment(a, id);
    if (!g.there) return;
    // the summing launch: nothing comes after the walk's last segment
    if (!OUT && g.k == (p.reverse ? 0 : g.cnt - 1)) return;

    const float ld = a.ld[h], ld2 = ld * 1.44269504f;
    for (int d = tid; d < kQ + 2; d += kThreads) pw[d] = power(ld2, d);
    const long long seq_state = ((long long)g.seq * a.H + h) * p.kd * p.vd;
    const long long seg_state = (id * a.H + h) * p.kd * p.vd;
    const float* in = !OUT ? nullptr : p.s_seg ? p.s_seg + seg_state : p.s_in ? p.s_in + seq_state : nullptr;
    for (int e = tid; e < kd * kVT; e += kThreads) {
        // neighbouring threads take neighbouring elements of the state in memory
        const int n = p.sn == 1 ? e % kd : e / kVT, c = p.sn == 1 ? e / kd : e % kVT;
        S[n * kVS + c] = in && c < vw ? in[n * p.sn + (v0 + c) * p.sp] : 0.f;
    }
    const T* q = static_cast<const T*>(p.q) + (long long)(h / p.qr) * kd;
    const T* k = static_cast<const T*>(p.k) + (long long)(h / p.kr) * kd;
    const int i0 = (tid / 16) * 2, j0 = (tid % 16) * 2;

    for (int c0 = 0; c0 < g.len; c0 += kQ) {
        const int n = min(kQ, g.len - c0);
        __syncthreads();
#pragma unroll 4
        for (int e = tid; e < kQ * kd; e += kThreads) {
            const int r = e / kd, c = e - r * kd;
            const long long t = g.start + (p.reverse ? g.len - 1 - (c0 + r) : c0 + r);
            if (OUT) qs[r * ks1 + c] = r < n ? static_cast<float>(q[t * p.qs + c]) : 0.f;
            ks[r * ks1 + c] = r < n ? static_cast<float>(k[t * p.ks + c]) : 0.f;
        }
#pragma unroll
        for (int e = tid; e < kQ * kVT; e += kThreads) {
            const int r = e / kVT, c = e - r * kVT;
            const long long t = g.start + (p.reverse ? g.len - 1 - (c0 + r) : c0 + r);
            vs[r * kVS + c] = r < n && c < vw ? static_cast<float>(v[t * p.vs + c]) : 0.f;
        }
        __syncthreads();
        if (OUT) {
            if (j0 <= i0 + 1 && i0 < n) {
                float d[2][2] = {};
#pragma unroll 8
                for (int c = 0; c < kd; ++c) {
                    const float q0 = qs[i0 * ks1 + c], q1 = qs[(i0 + 1) * ks1 + c];
                    const float k0 = ks[j0 * ks1 + c], k1 = ks[(j0 + 1) * ks1 + c];
                    d[0][0] = fmaf(q0, k0, d[0][0]), d[0][1] = fmaf(q0, k1, d[0][1]);
                    d[1][0] = fmaf(q1, k0, d[1][0]), d[1][1] = fmaf(q1, k1, d[1][1]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        if (j0 + y <= i0 + x)
                            sc[(i0 + x) * kVS + j0 + y] = d[x][y] * pw[i0 + x - j0 - y] * p.si;
            }
            __syncthreads();
            if (i0 < n) {
                float o[2][2] = {}, w[2][2] = {};
#pragma unroll 4
                for (int j = 0; j <= i0 + 1; ++j) {  // the entry above the diagonal is not read
                    const float a0 = j <= i0 ? sc[i0 * kVS + j] : 0.f, a1 = sc[(i0 + 1) * kVS + j];
                    const float b0 = vs[j * kVS + j0], b1 = vs[j * kVS + j0 + 1];
                    if (j <= i0) o[0][0] = fmaf(a0, b0, o[0][0]), o[0][1] = fmaf(a0, b1, o[0][1]);
                    o[1][0] = fmaf(a1, b0, o[1][0]), o[1][1] = fmaf(a1, b1, o[1][1]);
                }
#pragma unroll 8
                for (int c = 0; c < kd; ++c) {
                    const float a0 = qs[i0 * ks1 + c], a1 = qs[(i0 + 1) * ks1 + c];
                    const float b0 = S[c * kVS + j0], b1 = S[c * kVS + j0 + 1];
                    w[0][0] = fmaf(a0, b0, w[0][0]), w[0][1] = fmaf(a0, b1, w[0][1]);
                    w[1][0] = fmaf(a1, b0, w[1][0]), w[1][1] = fmaf(a1, b1, w[1][1]);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    if (i0 + x < n) {
                        const int r = c0 + i0 + x;
                        const long long t = g.start + (p.reverse ? g.len - 1 - r : r);
                        const float f = pw[i0 + x + 1 - p.reverse] * p.sx;
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            if (j0 + y < vw) {
                                const float val = fmaf(f, w[x][y], o[x][y]);
                                const long long at = t * p.os + (long long)(h / p.outr) * p.vd + v0 + j0 + y;
                                if (p.out_f32)
                                    st_out(static_cast<float*>(p.out), at, val);
                                else
                                    st_out(static_cast<T*>(p.out), at, val);
                            }
                    }
            }
            __syncthreads();
        }
        // the state: v's rows take their weights first
        for (int e = tid; e < kQ * kVT; e += kThreads) {
            const int r = e / kVT, c = e - r * kVT;
            if (r < n) vs[r * kVS + c] *= pw[n - 1 - r + p.reverse] * p.su;
        }
        __syncthreads();
        const Decay decay(ld, n);
        for (int u = tid; u < (kd + 3) / 4 * (kVT / 4); u += kThreads) {
            const int n0 = u / (kVT / 4) * 4, p0 = u % (kVT / 4) * 4;
            float d[4][4] = {};
#pragma unroll 4
            for (int r = 0; r < n; ++r) {
                float kk[4], vv[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    kk[x] = n0 + x < kd ? ks[r * ks1 + n0 + x] : 0.f;
                    vv[x] = vs[r * kVS + p0 + x];
                }
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) d[x][y] = fmaf(kk[x], vv[y], d[x][y]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (n0 + x < kd) {
                        float* s = &S[(n0 + x) * kVS + p0 + y];
                        *s = decay(*s) + d[x][y];
                    }
        }
    }
    __syncthreads();
    float* out = !OUT ? p.s_sum + seg_state
                 : p.s_out && g.k == (p.reverse ? 0 : g.cnt - 1) ? p.s_out + seq_state : nullptr;
    if (!out) return;
    for (int e = tid; e < kd * kVT; e += kThreads) {
        const int n = p.sn == 1 ? e % kd : e / kVT, c = p.sn == 1 ? e / kd : e % kVT;
        if (c < vw) out[n * p.sn + (v0 + c) * p.sp] = S[n * kVS + c];
    }
}

template <typename T, bool OUT>
cudaError_t simt_launch(const WalkArgs& a, cudaStream_t stream) {
    int kd = 0;
    for (int i = 0; i < a.npass; ++i) kd = std::max(kd, a.pass[i].kd);
    const size_t smem = simt_smem(kd);
    cudaError_t e = cudaFuncSetAttribute(simt_walk_kernel<T, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)simt_smem(128));
    if (e != cudaSuccess) return e;
    simt_walk_kernel<T, OUT><<<(unsigned)(a.ids * a.H * a.tiles), kThreads, smem, stream>>>(a);
    return cudaSuccess;
}

// The states that enter each segment, in the walk's direction, over what each segment adds:
// S <- a^len S + sum.  A thread goes through one sequence with VEC elements of a head's state; eight
// segments' loads are on their way ahead of their stores.  Bound by the states' bytes, read and
// written once.
template <int VEC>
__global__ void __launch_bounds__(kThreads) segment_scan_kernel(const __grid_constant__ WalkArgs a) {
    const Pass& p = a.pass[blockIdx.z];
    const int size = p.kd * p.vd, row = a.H * size;  // less than 2^31: check_sizes
    const int e = ((int)blockIdx.x * kThreads + threadIdx.x) * VEC;
    if (e >= row) return;
    const float ld = a.ld[e / size];
    const Decay whole(ld, a.Ls);
    for (int s = blockIdx.y; s < a.nseq; s += gridDim.y) {
        const Seg g = sequence(a, s);
        Pack<float, VEC> v;
        float S[VEC];
        v.zero();
        if (p.s_in) v.load(p.s_in + (long long)s * row + e);
        v.get(S);
        // from the walk's first segment on
        const long long step = p.reverse ? -(long long)row : row;
        float* at = p.s_sum + (first_segment(a, s) + (p.reverse ? g.cnt - 1 : 0)) * row + e;
        // the short segment is the sequence's last: from the end the first
        const Decay last(ld, g.len - (g.cnt - 1) * a.Ls);
        const int short_one = p.reverse ? 0 : g.cnt - 1, summed = p.s_out ? g.cnt : g.cnt - 1;
        for (int k0 = 0; k0 < g.cnt; k0 += 8) {
            Pack<float, VEC> add[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                add[i].zero();
                if (k0 + i < summed) add[i].load(at + (k0 + i) * step);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (k0 + i < g.cnt) {
                    store_vec<VEC>(at + (k0 + i) * step, S);
                    float f[VEC];
                    add[i].get(f);
#pragma unroll
                    for (int u = 0; u < VEC; ++u) S[u] = (k0 + i == short_one ? last(S[u]) : whole(S[u])) + f[u];
                }
        }
        if (p.s_out) store_vec<VEC>(p.s_out + (long long)s * row + e, S);
    }
}

// Final states of sequences that are not cut: what the sums left there, and the decayed initial ones.
__global__ void __launch_bounds__(kThreads) final_state_kernel(const __grid_constant__ WalkArgs a) {
    const Pass& p = a.pass[0];
    const int size = p.kd * p.vd, row = a.H * size;
    const int e = (int)blockIdx.x * kThreads + threadIdx.x;
    if (e >= row) return;
    const float ld = a.ld[e / size];
    for (int s = blockIdx.y; s < a.nseq; s += gridDim.y) {
        const long long at = (long long)s * row + e;
        p.s_out[at] += Decay(ld, sequence(a, s).len)(p.s_in[at]);
    }
}

// The gradients of shared heads: out[t][g][c] = sum of part[t][g r + i][c], i < r, in order; VEC
// columns a thread.  Bound by the parts' bytes.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) shared_sum_kernel(const float* part, T* out, long long T_,
                                                              int G, int r, int D, long long stride) {
    const int row = G * D / VEC;  // vectors of a token
    for (long long t = blockIdx.y; t < T_; t += gridDim.y)
        for (int e = blockIdx.x * kThreads + threadIdx.x; e < row; e += gridDim.x * kThreads) {
            const int g = e * VEC / D, c = e * VEC - g * D;
            const float* src = part + ((t * G + g) * r) * D + c;
            float s[VEC] = {};
            for (int i0 = 0; i0 < r; i0 += 4) {
                Pack<float, VEC> v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[i].zero();
                    if (i0 + i < r) v[i].load(src + (long long)(i0 + i) * D);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f[VEC];
                    v[i].get(f);
                    if (i0 + i < r)
#pragma unroll
                        for (int u = 0; u < VEC; ++u) s[u] += f[u];
                }
            }
            store_vec<VEC>(out + t * stride + (long long)g * D + c, s);
        }
}

// ---------------------------------------------------------------- host
struct Plan {
    long long T;
    int n;                       // sequences
    int Ls, per;
    long long ids;
    size_t s_seg, r_seg, dk_part, dv_part, total;
    bool fits;                   // its items are fewer than 2^31
};

ssd_status_t check_sizes(const ssd_linattn_t* p, bool bwd) {
    if (!p) return SSD_ERR_INVALID_ARG;
    if (p->batch < 1 || p->seqlen < 0 || p->nheads < 1 || p->ngroups < 1 || p->headdim < 1 ||
        p->dstate < 1 || p->nseq < 0 || p->nheads % p->ngroups != 0 || !dtype_ok(p->dtype) ||
        !isfinite(p->scale) || (p->nseq > 0 && p->batch != 1))
        return SSD_ERR_INVALID_ARG;
    const long long H = p->nheads, G = p->ngroups, P = p->headdim, N = p->dstate;
    // a head's state has up to 2^14 elements, all heads' together fewer than 2^31
    if (p->headdim > 128 || p->dstate > 128 || p->nheads > 65535 || p->batch > INT_MAX ||
        p->seqlen > INT_MAX || p->batch * p->seqlen > INT_MAX)
        return SSD_ERR_UNSUPPORTED;
    if (p->q_stride < H * N || p->k_stride < G * N || p->v_stride < G * P || p->o_stride < H * P)
        return SSD_ERR_INVALID_ARG;
    if (bwd && (p->dq_stride < H * N || p->dk_stride < G * N || p->dv_stride < G * P))
        return SSD_ERR_INVALID_ARG;
    return SSD_OK;
}

// A tensor of tokens as the bytes it has: those of one projection's rows may lie between one
// another, which the address ranges alone would refuse.
struct Rows : Span {
    size_t stride, width;
    Rows(const void* p, long long rows, long long stride_, long long width_, size_t e)
        : Span(p, rows, stride_, width_, e), stride((size_t)stride_ * e), width((size_t)width_ * e) {}
    Rows(const void* p, long long n, size_t e) : Rows(p, 1, n, n, e) {}
    bool shares(const Rows& o) const {
        if (!overlaps(o)) return false;
        if (stride != o.stride || stride == 0) return true;
        const size_t d = o.lo >= lo ? (o.lo - lo) % stride : (stride - (lo - o.lo) % stride) % stride;
        return d < width || d + o.width > stride;
    }
};
bool rows_clash(std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
    for (const Rows* o = outs.begin(); o != outs.end(); ++o) {
        for (const Rows* q = o + 1; q != outs.end(); ++q)
            if (o->shares(*q)) return true;
        for (const Rows& i : ins)
            if (o->shares(i)) return true;
    }
    return false;
}

size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

// How the sequences are cut, by sizes alone.  Not at all while the longest one may be short, or a dense
// batch has items for twice the SMs; otherwise into segments that leave several items for each SM, up to
// 4096 tokens.  On the tensor cores a segment has at least 512 tokens: shorter ones would move more of
// states (P N float32 four times each) than of tokens.  The plain walk takes 5 us for 32 tokens, one
// after the other, so that 64 are worth the two launches more (2 x 333 tokens of 5 heads in float32,
// backward: 57 us uncut, 31).
Plan make_plan(const ssd_linattn_t& p, bool bwd) {
    Plan l = {};
    l.T = p.batch * p.seqlen;
    l.n = p.nseq ? p.nseq : (int)p.batch;
    const auto tensor = [](int n) { return n == 64 || n == 128; };
    const bool tc = p.dtype == SSD_DTYPE_BF16 && tensor(p.headdim) && tensor(p.dstate);
    const int tile = tc ? kTcTile : kSimtTile, least = tc ? 512 : 64, step = tc ? kTcChunk : kQ;
    const auto tiles = [&](int n) { return (n + tile - 1) / tile; };
    // items for each run of tokens
    const long long per_cut = (long long)p.nheads * ((bwd ? 2 * tiles(p.dstate) : 0) + tiles(p.headdim));
    const long long sms = sm_count();
    const bool dense_full = !p.nseq && l.n * per_cut >= 2 * sms;
    if (p.seqlen > least && !dense_full) {
        const long long want = (8 * sms + per_cut - 1) / per_cut;  // cuts of all tokens
        long long Ls = (l.T / want + step - 1) / step * step;
        Ls = std::min<long long>(std::max<long long>(Ls, least), 4096);
        if (Ls < p.seqlen) l.Ls = (int)Ls;
    }
    l.per = l.Ls ? (int)((p.seqlen + l.Ls - 1) / l.Ls) : 1;
    l.ids = !l.Ls ? l.n : p.nseq ? l.T / l.Ls + l.n : (long long)l.n * l.per;
    l.fits = 2 * l.ids * per_cut <= INT_MAX;  // twice: rows off 16 bytes take the plain walk, in tiles of 32
    const size_t state = (size_t)p.headdim * p.dstate * sizeof(float);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t r = at;
        at += up(n);
        return r;
    };
    if (l.Ls) {
        l.s_seg = take((size_t)l.ids * p.nheads * state);
        if (bwd) l.r_seg = take((size_t)l.ids * p.nheads * state);
    }
    if (bwd && p.nheads != p.ngroups) {
        l.dk_part = take((size_t)l.T * p.nheads * p.dstate * sizeof(float));
        l.dv_part = take((size_t)l.T * p.nheads * p.headdim * sizeof(float));
    }
    l.total = at;
    return l;
}

WalkArgs common(const ssd_linattn_t& p, const Plan& l, const float* ld, const int32_t* cu) {
    WalkArgs a = {};
    a.ld = ld, a.cu = cu, a.T = l.T, a.rowlen = p.seqlen, a.nseq = l.n, a.H = p.nheads;
    a.Ls = l.Ls, a.per = l.per, a.ids = l.ids;
    return a;
}

void set_tiles(WalkArgs& a, int tile) {
    a.tiles = 0;
    for (int i = 0; i < a.npass; ++i) {
        a.pass[i].tiles = (a.pass[i].vd + tile - 1) / tile;
        a.tiles += a.pass[i].tiles;
    }
}

cudaError_t launch_walk(WalkArgs a, bool tc, bool sums, int dtype, Launch& L) {
    set_tiles(a, tc ? kTcTile : kSimtTile);
    if (tc) return sums ? tc_sums(a, L) : tc_walk(a, L);
    L.begin(sums ? "linattn_sums" : "linattn_walk");
    const bool b = dtype == SSD_DTYPE_BF16;
    cudaError_t e = sums ? (b ? simt_launch<__nv_bfloat16, false>(a, L.stream)
                              : simt_launch<float, false>(a, L.stream))
                         : (b ? simt_launch<__nv_bfloat16, true>(a, L.stream)
                              : simt_launch<float, true>(a, L.stream));
    const cudaError_t last = L.end();
    return e != cudaSuccess ? e : last;
}

cudaError_t launch_scan(const WalkArgs& a, Launch& L) {
    const int state = a.pass[0].kd * a.pass[0].vd;
    bool four = state % 4 == 0;
    for (int i = 0; i < a.npass; ++i) four = four && aligned_to(a.pass[i].s_in, 16) && aligned_to(a.pass[i].s_out, 16);
    const long long n = (long long)a.H * state / (four ? 4 : 1);
    const dim3 grid((unsigned)((n + kThreads - 1) / kThreads), (unsigned)std::min(a.nseq, 65535), (unsigned)a.npass);
    L.begin("linattn_scan");
    if (four)
        segment_scan_kernel<4><<<grid, kThreads, 0, L.stream>>>(a);
    else
        segment_scan_kernel<1><<<grid, kThreads, 0, L.stream>>>(a);
    return L.end();
}

// On the tensor cores the final states of a pass come from the sums (linattn_tc_sums), so that the walk
// does without exact ones: of sequences that are cut by the scan over them, of long ones with states of 128
// channels by a pass of their own, into the final states themselves.
bool sums_pay(const WalkArgs& a, const Pass& p) {
    return p.s_out && (a.Ls || ((p.kd == 128 || p.vd == 128) && !a.cu && a.rowlen >= 1024));
}
cudaError_t final_states(const WalkArgs& a, const Pass& p, int dtype, Launch& L) {
    WalkArgs f = a;
    f.pass[0] = p;
    f.npass = 1;
    f.pass[0].s_sum = p.s_out;
    cudaError_t e = launch_walk(f, true, true, dtype, L);
    if (e != cudaSuccess || !p.s_in) return e;
    const long long n = (long long)a.H * p.kd * p.vd;
    L.begin("linattn_final");
    final_state_kernel<<<dim3((unsigned)((n + kThreads - 1) / kThreads), (unsigned)std::min(a.nseq, 65535)),
                         kThreads, 0, L.stream>>>(f);
    return L.end();
}

cudaError_t launch_shared_sum(const float* part, void* out, const ssd_linattn_t& p, long long T, int D,
                              long long stride, Launch& L) {
    const int r = p.nheads / p.ngroups;
    if (T == 0) return cudaSuccess;
    // four columns where they and out's rows allow it
    const bool four = D % 4 == 0 && stride % 4 == 0 && aligned_to(out, p.dtype == SSD_DTYPE_BF16 ? 8 : 16);
    const int row = p.ngroups * D / (four ? 4 : 1);
    const dim3 grid((unsigned)((row + kThreads - 1) / kThreads), (unsigned)std::min<long long>(T, 65535));
    L.begin("linattn_shared_sum");
    if (p.dtype == SSD_DTYPE_BF16) {
        auto* o = static_cast<__nv_bfloat16*>(out);
        if (four)
            shared_sum_kernel<__nv_bfloat16, 4><<<grid, kThreads, 0, L.stream>>>(part, o, T, p.ngroups, r, D, stride);
        else
            shared_sum_kernel<__nv_bfloat16, 1><<<grid, kThreads, 0, L.stream>>>(part, o, T, p.ngroups, r, D, stride);
    } else {
        auto* o = static_cast<float*>(out);
        if (four)
            shared_sum_kernel<float, 4><<<grid, kThreads, 0, L.stream>>>(part, o, T, p.ngroups, r, D, stride);
        else
            shared_sum_kernel<float, 1><<<grid, kThreads, 0, L.stream>>>(part, o, T, p.ngroups, r, D, stride);
    }
    return L.end();
}

}  // namespace
}  // namespace linattn
}  // namespace ssd

using namespace ssd;
using namespace ssd::layer;
using namespace ssd::linattn;

extern "C" {

ssd_status_t ssd_linear_attention_workspace_size(const ssd_linattn_t* prob, int for_backward,
                                                 size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    const ssd_status_t st = check_sizes(prob, for_backward != 0);
    if (st != SSD_OK) return st;
    const Plan l = make_plan(*prob, for_backward != 0);
    if (!l.fits) return SSD_ERR_UNSUPPORTED;
    *bytes = l.total;
    return SSD_OK;
}

ssd_status_t ssd_linear_attention_forward(const ssd_linattn_t* prob, const void* q, const void* k,
                                          const void* v, const float* log_decay,
                                          const int32_t* cu_seqlens, const float* initial_state,
                                          void* o, float* final_state, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    set_last_launches(0);
    const ssd_status_t st = check_sizes(prob, false);
    if (st != SSD_OK) return st;
    const ssd_linattn_t& p = *prob;
    if ((p.nseq > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    const long long T = p.batch * p.seqlen, H = p.nheads, G = p.ngroups, P = p.headdim, N = p.dstate;
    if ((T > 0 && (!q || !k || !v || !o)) || !log_decay) return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(p.dtype);
    if (!aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) || !aligned_to(o, e) ||
        !aligned_to(log_decay, 4) || !aligned_to(cu_seqlens, 4) || !aligned_to(initial_state, 4) ||
        !aligned_to(final_state, 4) || !aligned_to(workspace, 256))
        return SSD_ERR_ALIGNMENT;
    const Plan l = make_plan(p, false);
    if (!l.fits) return SSD_ERR_UNSUPPORTED;
    if (l.total > 0 && (!workspace || workspace_bytes < l.total)) return SSD_ERR_WORKSPACE;
    const long long states = (long long)l.n * H * P * N;
    if (rows_clash({Rows(o, T, p.o_stride, H * P, e), Rows(final_state, states, 4), Rows(workspace, l.total, 1)},
              {Rows(q, T, p.q_stride, H * N, e), Rows(k, T, p.k_stride, G * N, e),
               Rows(v, T, p.v_stride, G * P, e), Rows(log_decay, H, 4),
               Rows(cu_seqlens, p.nseq ? p.nseq + 1 : 0, 4), Rows(initial_state, states, 4)}))
        return SSD_ERR_INVALID_ARG;
    WalkArgs a = common(p, l, log_decay, cu_seqlens);
    if (!(a.status = status_word())) return SSD_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    const int r = (int)(H / G);
    Pass& f = a.pass[0];
    f.q = q, f.k = k, f.v = v, f.out = o;
    f.qs = p.q_stride, f.ks = p.k_stride, f.vs = p.v_stride, f.os = p.o_stride;
    f.kd = p.dstate, f.vd = p.headdim, f.qr = 1, f.kr = r, f.vr = r, f.outr = 1;
    f.si = f.sx = p.scale, f.su = 1.f;
    f.s_in = initial_state, f.s_out = final_state;
    f.sn = 1, f.sp = N;
    f.out_f32 = p.dtype == SSD_DTYPE_F32;
    a.npass = 1;
    const bool tc = p.dtype == SSD_DTYPE_BF16 && T > 0 && tc_fits(f);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    if (few_fits(a)) {
        err = few_tokens(a, p.dtype, L);
        set_last_launches(L.count);
        return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
    }
    const bool by_sums = tc && sums_pay(a, f);
    if (l.Ls) {
        if (!by_sums) f.s_out = nullptr;  // the walk's
        f.s_sum = reinterpret_cast<float*>(ws + l.s_seg);
        err = launch_walk(a, tc, true, p.dtype, L);
        if (err == cudaSuccess) err = launch_scan(a, L);
        f.s_seg = f.s_sum;
    } else if (by_sums) {
        err = final_states(a, f, p.dtype, L);
    }
    f.s_out = by_sums ? nullptr : final_state;
    if (err == cudaSuccess) err = launch_walk(a, tc, false, p.dtype, L);
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_linear_attention_backward(const ssd_linattn_t* prob, const void* q, const void* k,
                                           const void* v, const float* log_decay,
                                           const int32_t* cu_seqlens, const float* initial_state,
                                           const void* dout, const float* d_final_state, void* dq,
                                           void* dk, void* dv, float* d_initial_state,
                                           void* workspace, size_t workspace_bytes, void* stream) {
    set_last_launches(0);
    const ssd_status_t st = check_sizes(prob, true);
    if (st != SSD_OK) return st;
    const ssd_linattn_t& p = *prob;
    if ((p.nseq > 0) != (cu_seqlens != nullptr)) return SSD_ERR_INVALID_ARG;
    const long long T = p.batch * p.seqlen, H = p.nheads, G = p.ngroups, P = p.headdim, N = p.dstate;
    if ((T > 0 && (!q || !k || !v || !dout || !dq || !dk || !dv)) || !log_decay) return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(p.dtype);
    if (!aligned_to(q, e) || !aligned_to(k, e) || !aligned_to(v, e) || !aligned_to(dout, e) ||
        !aligned_to(dq, e) || !aligned_to(dk, e) || !aligned_to(dv, e) || !aligned_to(log_decay, 4) ||
        !aligned_to(cu_seqlens, 4) || !aligned_to(initial_state, 4) || !aligned_to(d_final_state, 4) ||
        !aligned_to(d_initial_state, 4) || !aligned_to(workspace, 256))
        return SSD_ERR_ALIGNMENT;
    const Plan l = make_plan(p, true);
    if (!l.fits) return SSD_ERR_UNSUPPORTED;
    if (l.total > 0 && (!workspace || workspace_bytes < l.total)) return SSD_ERR_WORKSPACE;
    const long long states = (long long)l.n * H * P * N;
    if (rows_clash({Rows(dq, T, p.dq_stride, H * N, e), Rows(dk, T, p.dk_stride, G * N, e),
               Rows(dv, T, p.dv_stride, G * P, e), Rows(d_initial_state, states, 4),
               Rows(workspace, l.total, 1)},
              {Rows(q, T, p.q_stride, H * N, e), Rows(k, T, p.k_stride, G * N, e),
               Rows(v, T, p.v_stride, G * P, e), Rows(dout, T, p.o_stride, H * P, e),
               Rows(log_decay, H, 4), Rows(cu_seqlens, p.nseq ? p.nseq + 1 : 0, 4),
               Rows(initial_state, states, 4), Rows(d_final_state, states, 4)}))
        return SSD_ERR_INVALID_ARG;
    WalkArgs a = common(p, l, log_decay, cu_seqlens);
    if (!(a.status = status_word())) return SSD_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    const int r = (int)(H / G);
    const int f32 = p.dtype == SSD_DTYPE_F32;
    // dq from (do, v, k); dk from (v, do, q); dv from (k, q, do): linattn.cuh
    Pass& f = a.pass[0];
    f.q = dout, f.k = v, f.v = k, f.out = dq;
    f.qs = p.o_stride, f.ks = p.v_stride, f.vs = p.k_stride, f.os = p.dq_stride;
    f.kd = p.headdim, f.vd = p.dstate, f.qr = 1, f.kr = r, f.vr = r, f.outr = 1;
    f.si = f.sx = p.scale, f.su = 1.f;
    f.s_in = initial_state, f.sn = N, f.sp = 1, f.out_f32 = f32;
    Pass& g = a.pass[1];
    g.q = v, g.k = dout, g.v = q, g.out = dk;
    g.qs = p.v_stride, g.ks = p.o_stride, g.vs = p.q_stride, g.os = p.dk_stride;
    g.kd = p.headdim, g.vd = p.dstate, g.qr = r, g.kr = 1, g.vr = 1, g.outr = 1;
    g.reverse = 1, g.si = g.su = p.scale, g.sx = 1.f;
    g.s_in = d_final_state, g.sn = N, g.sp = 1, g.out_f32 = f32;
    Pass& d = a.pass[2];
    d.q = k, d.k = q, d.v = dout, d.out = dv;
    d.qs = p.k_stride, d.ks = p.q_stride, d.vs = p.o_stride, d.os = p.dv_stride;
    d.kd = p.dstate, d.vd = p.headdim, d.qr = r, d.kr = 1, d.vr = 1, d.outr = 1;
    d.reverse = 1, d.si = d.su = p.scale, d.sx = 1.f;
    d.s_in = d_final_state, d.s_out = d_initial_state, d.sn = 1, d.sp = N, d.out_f32 = f32;
    a.npass = 3;
    const bool tc = p.dtype == SSD_DTYPE_BF16 && T > 0 && tc_fits(f) && tc_fits(g) && tc_fits(d);
    if (r > 1) {  // each head's own part, summed after the walk
        g.out = ws + l.dk_part, g.os = H * N, g.out_f32 = 1;
        d.out = ws + l.dv_part, d.os = H * P, d.out_f32 = 1;
    }
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    const bool by_sums = tc && sums_pay(a, d);
    if (l.Ls) {
        // the states by segments from k and v, their adjoints from q and do
        WalkArgs s = a;
        s.npass = 2;
        s.pass[0].s_sum = reinterpret_cast<float*>(ws + l.s_seg);
        s.pass[1] = d;
        s.pass[1].s_sum = reinterpret_cast<float*>(ws + l.r_seg);
        if (!by_sums) s.pass[1].s_out = nullptr;
        err = launch_walk(s, tc, true, p.dtype, L);
        if (err == cudaSuccess) err = launch_scan(s, L);
        f.s_seg = s.pass[0].s_sum;
        g.s_seg = d.s_seg = s.pass[1].s_sum;
    } else if (by_sums) {
        err = final_states(a, d, p.dtype, L);
    }
    if (by_sums) d.s_out = nullptr;
    if (err == cudaSuccess) err = launch_walk(a, tc, false, p.dtype, L);
    if (r > 1 && err == cudaSuccess)
        err = launch_shared_sum(static_cast<const float*>(g.out), dk, p, T, (int)N, p.dk_stride, L);
    if (r > 1 && err == cudaSuccess)
        err = launch_shared_sum(static_cast<const float*>(d.out), dv, p, T, (int)P, p.dv_stride, L);
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
