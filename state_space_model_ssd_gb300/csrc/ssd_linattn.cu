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
constexpr int kRows = kQ / 8;    // of them, what a warp loads

// Rows of q and k in shared memory are an odd number of 16 bytes long: eight threads read four channels
// of eight rows in one go (20720 tokens of 7 heads, 90 x 90, at an even one: 840 us, so 524).
__host__ __device__ constexpr int whole4(int kd) { return (kd + 3) / 4 * 4; }
__host__ __device__ constexpr int row_words(int kd) { return (whole4(kd) / 4 | 1) * 4; }
__host__ __device__ constexpr size_t simt_smem(int kd, int vt) {
    return sizeof(float) * (2 * (size_t)kQ * row_words(kd) + 2 * (size_t)kQ * vt + (size_t)kQ * (kQ + 1) +
                            (size_t)whole4(kd) * (vt + 4) + kQ + 2);
}

__device__ __forceinline__ float4 four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}
// o += a b for VPT neighbouring columns
template <int VPT>
__device__ __forceinline__ void add_row(float* o, float a, const float* b) {
    if constexpr (VPT == 4) {
        const float4 f = four(b);
        o[0] = fmaf(a, f.x, o[0]), o[1] = fmaf(a, f.y, o[1]), o[2] = fmaf(a, f.z, o[2]), o[3] = fmaf(a, f.w, o[3]);
    } else {
        const float2 f = *reinterpret_cast<const float2*>(b);
        o[0] = fmaf(a, f.x, o[0]), o[1] = fmaf(a, f.y, o[1]);
    }
}
template <int VPT, typename O>
__device__ __forceinline__ void put_row(O* p, const float* f, int n, bool vec) {
    if (vec && n >= VPT) {
        store_vec<VPT>(p, f);
        return;
    }
#pragma unroll
    for (int y = 0; y < VPT; ++y)
        if (y < n) st_out(p, y, f[y]);
}

// One segment, head and tile of VT columns of v: 32 tokens at a time, everything in float32 in
// shared memory.  A thread has the rows i and i + 16 of the products, one or two columns of the scores
// and VT / 16 of the outputs, and pieces of 4 x 4 of the state; the next chunk's rows come into registers
// meanwhile.  Operands are read four at a time, so that multiply-adds and shared memory take about as
// long.  Bound by the issue of instructions, 65 % of which are multiply-adds at 128 channels (32768 tokens of
// 16 heads in float32, 64 x 128: 947 us for the walk, 367 for the sums; with 2 x 2 pieces read word by word
// 1516 and 654).  It serves float32 and the sizes that the tensor cores do not take.  OUT: false where only the
// state after the segment is wanted.
template <typename T, bool OUT, int VT>
__global__ void __launch_bounds__(kThreads, 2) simt_walk_kernel(const __grid_constant__ WalkArgs a) {
    extern __shared__ __align__(16) float sm[];
    constexpr int VPT = VT / 16, kS = VT + 4;
    const long long item = blockIdx.x;
    const long long id = item / ((long long)a.tiles * a.H);
    const int rest = (int)(item - id * a.tiles * a.H);
    const int h = rest / a.tiles;
    int tile = rest - h * a.tiles;
    const Pass& p = pass_of(a, tile);
    const int v0 = tile * VT, vw = min(VT, p.vd - v0);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int kd = p.kd, kd4 = whole4(kd), ks1 = row_words(kd);
    float* qs = sm;
    float* ks = qs + kQ * ks1;
    float* vs = ks + kQ * ks1;   // v, and v with the weights of the state
    float* ws = vs + kQ * VT;
    float* S = ws + kQ * VT;
    float* sc = S + kd4 * kS;    // rows of kQ + 1
    float* pw = sc + kQ * (kQ + 1);  // a^0 .. a^(kQ + 1)

    const T* v = static_cast<const T*>(p.v) + (long long)(h / p.vr) * p.vd + v0;
    const long long o_at = (long long)(h / p.outr) * p.vd + v0;
    if (OUT && a.cu) {
        const Outside none(a);
        for (long long r = id; r < none.n; r += a.ids) {
            const long long t = none.token(r);
            for (int c = tid; c < vw; c += kThreads) {
                if (p.out_f32)
                    st_out(static_cast<float*>(p.out), t * p.os + o_at + c, 0.f);
                else
                    st_out(static_cast<T*>(p.out), t * p.os + o_at + c, 0.f);
            }
        }
    }
    const Seg g = segment(a, id);
    if (!g.there) return;
    // the summing launch: nothing comes after the walk's last segment
    if (!OUT && g.k == (p.reverse ? 0 : g.cnt - 1)) return;

    const float ld = a.ld[h], ld2 = ld * 1.44269504f;
    for (int d = tid; d < kQ + 2; d += kThreads) pw[d] = power(ld2, d);
    const long long seq_state = ((long long)g.seq * a.H + h) * kd * p.vd;
    const long long seg_state = (id * a.H + h) * kd * p.vd;
    const float* in = !OUT ? nullptr : p.s_seg ? p.s_seg + seg_state : p.s_in ? p.s_in + seq_state : nullptr;
    // a warp takes neighbouring elements of the state in memory, 8 x 4 of them where they follow one
    // another along n: rows of shared memory are 16 bytes apart in the banks
    const int nb = (kd4 + 7) / 8, elems = nb * 8 * VT;
    const auto place = [&](int e, int& n, int& c) {
        const int w = e >> 5;
        if (p.sn == 1)
            n = (e & 7) + 8 * (w % nb), c = (e >> 3 & 3) + 4 * (w / nb);
        else
            n = e / VT, c = e % VT;
    };
#pragma unroll 1
    for (int e = tid; e < elems; e += kThreads) {
        int n, c;
        place(e, n, c);
        if (n < kd4) S[n * kS + c] = in && n < kd && c < vw ? in[n * p.sn + (v0 + c) * p.sp] : 0.f;
    }
    const T* q = static_cast<const T*>(p.q) + (long long)(h / p.qr) * kd;
    const T* k = static_cast<const T*>(p.k) + (long long)(h / p.kr) * kd;
    const int i = tid / 16, j = tid % 16, j0 = j * VPT;
    const int bytes = p.out_f32 ? 4 : (int)sizeof(T);
    const bool vec = OUT && ((p.os | o_at) & (VPT - 1)) == 0 &&
                     (reinterpret_cast<uintptr_t>(p.out) & (VPT * bytes - 1)) == 0;

    float rq[kRows][4], rk[kRows][4], rv[kRows][VT / 32];  // the rows warp + 8 x of the next chunk
    const auto fetch = [&](int c0) {
#pragma unroll
        for (int x = 0; x < kRows; ++x) {
            const int r = c0 + warp + 8 * x;
            const bool in_seg = r < g.len;
            const long long t = g.start + (p.reverse ? g.len - 1 - r : r);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int c = lane + 32 * y;
                const bool there = in_seg && c < kd;
                if (OUT) rq[x][y] = there ? static_cast<float>(q[t * p.qs + c]) : 0.f;
                rk[x][y] = there ? static_cast<float>(k[t * p.ks + c]) : 0.f;
            }
#pragma unroll
            for (int y = 0; y < VT / 32; ++y) {
                const int c = lane + 32 * y;
                rv[x][y] = in_seg && c < vw ? static_cast<float>(v[t * p.vs + c]) : 0.f;
            }
        }
    };
#pragma unroll 1
    for (int c0 = -kQ; c0 < g.len; c0 += kQ) {
        const int n = min(kQ, g.len - c0);
        __syncthreads();
#pragma unroll
        for (int x = 0; x < kRows; ++x) {
            if (c0 < 0) break;
            const int r = warp + 8 * x;
            const float w = r < n ? pw[n - 1 - r + p.reverse] * p.su : 0.f;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int c = lane + 32 * y;
                if (c < kd4) {
                    if (OUT) qs[r * ks1 + c] = rq[x][y];
                    ks[r * ks1 + c] = rk[x][y];
                }
            }
#pragma unroll
            for (int y = 0; y < VT / 32; ++y) {
                const int c = lane + 32 * y;
                if (OUT) vs[r * VT + c] = rv[x][y];
                ws[r * VT + c] = rv[x][y] * w;
            }
        }
        __syncthreads();
        if (c0 + kQ < g.len) fetch(c0 + kQ);
        if (c0 < 0) continue;
        if (OUT) {
            if (i < n) {  // the scores (i, j), (i + 16, j), (i + 16, j + 16)
                float d00 = 0.f, d10 = 0.f, d11 = 0.f;
                const float* q0 = qs + i * ks1;
                const float* k0 = ks + j * ks1;
#pragma unroll 4
                for (int c = 0; c < kd4; c += 4) {
                    const float4 ka = four(k0 + c), qb = four(q0 + 16 * ks1 + c);
                    d00 = dot4(four(q0 + c), ka, d00);
                    d10 = dot4(qb, ka, d10);
                    d11 = dot4(qb, four(k0 + 16 * ks1 + c), d11);
                }
                float* s0 = sc + i * (kQ + 1) + j;
                float* s1 = s0 + 16 * (kQ + 1);
                if (j <= i) s0[0] = d00 * pw[i - j] * p.si, s1[16] = d11 * pw[i - j] * p.si;
                s1[0] = d10 * pw[i + 16 - j] * p.si;
            }
            __syncthreads();
            if (i < n) {
                float o[2][VPT] = {}, w[2][VPT] = {};
                const float* s0 = sc + i * (kQ + 1);
                const float* s1 = s0 + 16 * (kQ + 1);
#pragma unroll 4
                for (int c = 0; c <= i; ++c) {  // entries above the diagonal are not read
                    add_row<VPT>(o[0], s0[c], vs + c * VT + j0);
                    add_row<VPT>(o[1], s1[c], vs + c * VT + j0);
                }
                if (i + 16 < n)
#pragma unroll 4
                    for (int c = i + 1; c <= i + 16; ++c) add_row<VPT>(o[1], s1[c], vs + c * VT + j0);
                const float* q0 = qs + i * ks1;
                const float* q1 = q0 + 16 * ks1;
#pragma unroll 2
                for (int c = 0; c < kd4; c += 4) {
                    const float4 a0 = four(q0 + c), a1 = four(q1 + c);
                    const float* b = S + c * kS + j0;
                    add_row<VPT>(w[0], a0.x, b), add_row<VPT>(w[1], a1.x, b);
                    add_row<VPT>(w[0], a0.y, b + kS), add_row<VPT>(w[1], a1.y, b + kS);
                    add_row<VPT>(w[0], a0.z, b + 2 * kS), add_row<VPT>(w[1], a1.z, b + 2 * kS);
                    add_row<VPT>(w[0], a0.w, b + 3 * kS), add_row<VPT>(w[1], a1.w, b + 3 * kS);
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = i + 16 * x;
                    if (r >= n || j0 >= vw) continue;
                    const long long t = g.start + (p.reverse ? g.len - 1 - c0 - r : c0 + r);
                    const float f = pw[r + 1 - p.reverse] * p.sx;
                    float val[VPT];
#pragma unroll
                    for (int y = 0; y < VPT; ++y) val[y] = fmaf(f, w[x][y], o[x][y]);
                    const long long at = t * p.os + o_at + j0;
                    if (p.out_f32)
                        put_row<VPT>(static_cast<float*>(p.out) + at, val, vw - j0, vec);
                    else
                        put_row<VPT>(static_cast<T*>(p.out) + at, val, vw - j0, vec);
                }
            }
            __syncthreads();
        }
        const Decay decay(ld, n);
#pragma unroll 1
        for (int u = tid; u < kd4 / 4 * (VT / 4); u += kThreads) {
            const int n0 = u / (VT / 4) * 4, p0 = u % (VT / 4) * 4;
            float d[4][4] = {};
#pragma unroll 4
            for (int r = 0; r < n; ++r) {
                const float4 kk = four(ks + r * ks1 + n0);
                const float* b = ws + r * VT + p0;
                add_row<4>(d[0], kk.x, b), add_row<4>(d[1], kk.y, b);
                add_row<4>(d[2], kk.z, b), add_row<4>(d[3], kk.w, b);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (n0 + x >= kd) break;  // stays 0 for any v
                float4* s = reinterpret_cast<float4*>(S + (n0 + x) * kS + p0);
                const float4 f = *s;
                *s = make_float4(decay(f.x) + d[x][0], decay(f.y) + d[x][1], decay(f.z) + d[x][2],
                                 decay(f.w) + d[x][3]);
            }
        }
    }
    __syncthreads();
    float* out = !OUT ? p.s_sum + seg_state
                 : p.s_out && g.k == (p.reverse ? 0 : g.cnt - 1) ? p.s_out + seq_state : nullptr;
    if (!out) return;
#pragma unroll 1
    for (int e = tid; e < elems; e += kThreads) {
        int n, c;
        place(e, n, c);
        if (n < kd && c < vw) out[n * p.sn + (v0 + c) * p.sp] = S[n * kS + c];
    }
}

template <typename T, bool OUT, int VT>
cudaError_t simt_launch(const WalkArgs& a, cudaStream_t stream) {
    int kd = 0;
    for (int i = 0; i < a.npass; ++i) kd = std::max(kd, a.pass[i].kd);
    cudaError_t e = cudaFuncSetAttribute(simt_walk_kernel<T, OUT, VT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)simt_smem(128, VT));
    if (e != cudaSuccess) return e;
    simt_walk_kernel<T, OUT, VT><<<(unsigned)(a.ids * a.H * a.tiles), kThreads, simt_smem(kd, VT), stream>>>(a);
    return cudaSuccess;
}
template <typename T>
cudaError_t simt_launch(const WalkArgs& a, bool sums, int tile, cudaStream_t stream) {
    if (tile == 32) return sums ? simt_launch<T, false, 32>(a, stream) : simt_launch<T, true, 32>(a, stream);
    return sums ? simt_launch<T, false, 64>(a, stream) : simt_launch<T, true, 64>(a, stream);
}

// The states that enter each segment, in the walk's direction, over what each segment adds:
// S <- a^len S + sum.  A thread goes through one sequence with VEC elements of a head's state; eight
// segments' loads are on their way ahead of their stores.  Bound by the states' bytes, read and
// written once.
template <int VEC>
__global__ void __launch_bounds__(kThreads, 4) segment_scan_kernel(const __grid_constant__ WalkArgs a) {
    const Pass& p = a.pass[blockIdx.z];
    const int size = p.kd * p.vd, row = a.H * size;  // less than 2^31: check_sizes
    const int e = ((int)blockIdx.x * kThreads + threadIdx.x) * VEC;
    if (e >= row) return;
    const float ld = a.ld[e / size];
    const Decay whole(ld, a.Ls);
    for (int s = blockIdx.y; s < a.nseq; s += gridDim.y) {
        Pack<float, VEC> v;  // on its way before the sequence is looked up
        v.zero();
        if (p.s_in) v.load(p.s_in + (long long)s * row + e);
        const Seg g = sequence(a, s);
        float S[VEC];
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
                if (k0 + i >= g.cnt) break;
                add[i].zero();
                if (k0 + i < summed) add[i].load(at + (k0 + i) * step);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (k0 + i >= g.cnt) break;
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

// Tensors laid out anew: element (t, h, c) of to is that of from, or 0 outside of from's h and c.
struct Copy {
    const void* from;
    void* to;
    long long n, fs, ts;  // t < n, and elements from one to the next
    int h, c, fh, fc;     // of to, and of from
    int fw, tw;           // elements from one h to the next
    int f32;
};
struct Copies {
    Copy c[6];
    int n;
};
// A lane has four elements of a row and 16 or all lanes a row (c up to 64, or 128); four rows are on
// their way at a time.  Bound by the bytes where rows start on four elements, else by single loads and
// stores.
template <typename T>
__device__ __forceinline__ void copy_rows(const Copy& j) {
    const int lane = threadIdx.x & 31, lanes = j.c <= 64 ? 16 : 32, at_once = 32 / lanes;
    const int c = lane % lanes * 4, sub = lane / lanes;
    const unsigned groups = (unsigned)(j.h + 4 * at_once - 1) / (4 * at_once);
    const long long items = j.n * groups;
    const T* from = static_cast<const T*>(j.from) + c;
    T* to = static_cast<T*>(j.to) + c;
    const auto fours = [](const void* p, long long a, int b) {
        return ((a | b) & 3) == 0 && (reinterpret_cast<uintptr_t>(p) & (4 * sizeof(T) - 1)) == 0;
    };
    const int in = j.fc - c, out = j.c - c;  // elements from c on
    const bool load4 = in >= 4 && fours(j.from, j.fs, j.fw), store4 = out >= 4 && fours(j.to, j.ts, j.tw);
    for (long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < items;
         i += (long long)gridDim.x * (kThreads / 32)) {
        const long long t = items <= UINT_MAX ? (unsigned)i / groups : i / groups;
        const int h0 = (int)(i - t * groups) * 4 * at_once + sub;
        float v[4][4] = {};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int h = h0 + x * at_once;
            const T* p = from + t * j.fs + (long long)h * j.fw;
            if (h >= j.fh) continue;
            if (load4) {
                Pack<T, 4> q;
                q.load(p);
                q.get(v[x]);
            } else {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (y < in) v[x][y] = static_cast<float>(p[y]);
            }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int h = h0 + x * at_once;
            if (h < j.h) put_row<4>(to + t * j.ts + (long long)h * j.tw, v[x], out, store4);
        }
    }
}
__global__ void __launch_bounds__(kThreads) copies_kernel(const __grid_constant__ Copies a) {
    const Copy& j = a.c[blockIdx.y];
    if (j.f32)
        copy_rows<float>(j);
    else
        copy_rows<__nv_bfloat16>(j);
}

// ---------------------------------------------------------------- host
// Rows of one head and token from which the tensors are laid out anew: see pads.
constexpr long long kPadRows = 16384;

struct Plan {
    long long T;
    int n;                       // sequences
    int Ls, per;
    long long ids;
    size_t s_seg, r_seg, dk_part, dv_part, total;
    bool fits;                   // its items are fewer than 2^31
    bool tc;                     // it runs on the tensor cores
    // bf16 of other channels than 64 and 128 or with rows off 16 bytes, laid out in the workspace for the
    // tensor cores: the problem as it is there (pads) and its tensors: q, k, v, o or do, the gradients, the
    // states
    bool pads;
    ssd_linattn_t p;
    size_t q, k, v, o, dq, dk, dv, s_in, s_out, r_in;
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
bool tensor(int n) { return n == 64 || n == 128; }
// Whether rows are worth laying out anew, with zeros up to 64 or 128 channels: two passes over the
// tensors, which are at most four times as wide, and two launches, so that few tokens are not.  32768
// tokens of 24 heads, 80 x 96: forward 776 us of which 405 are the copies, backward 1487 (669), on the
// plain cores 4085 and 9442; 64 x 128 with three more elements a token 527 and 1054, on the plain cores 2740
// and 7724; 16384 rows of 33 x 33 channels 56 and 63, for 52 and 103.
bool pads(const ssd_linattn_t& p, bool rows16) {
    const int P = p.headdim <= 64 ? 64 : 128, N = p.dstate <= 64 ? 64 : 128;
    return p.dtype == SSD_DTYPE_BF16 && !(rows16 && tensor(p.headdim) && tensor(p.dstate)) && p.seqlen > kFewTokens &&
           p.batch * p.seqlen * p.nheads >= kPadRows && P + N <= 4 * (p.headdim + p.dstate);
}
// Whether tokens of bf16 tensors that start on 16 bytes do so too.  Gradients of shared heads are
// written by a kernel of their own.
bool tokens16(const ssd_linattn_t& p, bool bwd) {
    int64_t s = p.q_stride | p.k_stride | p.v_stride | p.o_stride;
    if (bwd) s |= p.dq_stride;
    if (bwd && p.nheads == p.ngroups) s |= p.dk_stride | p.dv_stride;
    return s % 8 == 0;
}
// rows16: every token starts on 16 bytes.
Plan make_plan(const ssd_linattn_t& given, bool bwd, bool rows16, bool copies = true) {
    Plan l = {};
    ssd_linattn_t& p = l.p;
    p = given;
    l.pads = copies && pads(p, rows16);
    if (l.pads) {
        p.headdim = p.headdim <= 64 ? 64 : 128, p.dstate = p.dstate <= 64 ? 64 : 128;
        const int64_t H = p.nheads, G = p.ngroups;
        p.q_stride = p.dq_stride = H * p.dstate, p.k_stride = p.dk_stride = G * p.dstate;
        p.o_stride = H * p.headdim, p.v_stride = p.dv_stride = G * p.headdim;
    }
    l.T = p.batch * p.seqlen;
    l.n = p.nseq ? p.nseq : (int)p.batch;
    const bool tc = p.dtype == SSD_DTYPE_BF16 && tensor(p.headdim) && tensor(p.dstate) && (rows16 || l.pads);
    l.tc = tc;
    const int tile = tc ? kTcTile : simt_tile(bwd ? std::max(p.headdim, p.dstate) : p.headdim);
    const int least = tc ? 512 : 64, step = tc ? kTcChunk : kQ;
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
    l.fits = 2 * l.ids * per_cut <= INT_MAX;  // twice: a pass of few columns may go by itself in tiles of 32
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
    if (l.pads) {
        const size_t states = (size_t)l.n * p.nheads * state, T = 2 * (size_t)l.T;
        const size_t q = T * p.q_stride, k = T * p.k_stride, v = T * p.v_stride;
        l.q = take(q), l.k = take(k), l.v = take(v), l.o = take(T * p.o_stride);
        l.s_in = take(states), l.s_out = take(states);
        if (bwd) l.dq = take(q), l.dk = take(k), l.dv = take(v), l.r_in = take(states);
    }
    l.total = at;
    return l;
}
// The plan of a call whose tensors start on 16 bytes, or do not: then the strides, by which the workspace
// was asked for, say nothing, and there are copies if it holds them.
Plan call_plan(const ssd_linattn_t& p, bool bwd, std::initializer_list<const void*> tensors, size_t workspace_bytes) {
    const Plan l = make_plan(p, bwd, tokens16(p, bwd));
    uintptr_t at = 0;
    for (const void* t : tensors) at |= (uintptr_t)t;
    if (!l.tc || l.pads || at % 16 == 0) return l;
    const Plan c = make_plan(p, bwd, false);
    return c.pads && workspace_bytes >= c.total ? c : make_plan(p, bwd, false, false);
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
    int vd = 0;
    for (int i = 0; i < a.npass; ++i) vd = std::max(vd, a.pass[i].vd);
    const int tile = tc ? kTcTile : simt_tile(vd);
    set_tiles(a, tile);
    if (tc) return sums ? tc_sums(a, L) : tc_walk(a, L);
    L.begin(sums ? "linattn_sums" : "linattn_walk");
    const cudaError_t e = dtype == SSD_DTYPE_BF16 ? simt_launch<__nv_bfloat16>(a, sums, tile, L.stream)
                                                  : simt_launch<float>(a, sums, tile, L.stream);
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

// The launches of a problem whose arguments have been checked.
cudaError_t run_forward(const ssd_linattn_t& p, const Plan& l, const void* q, const void* k, const void* v,
                        const float* ld, const int32_t* cu, const float* initial_state, void* o,
                        float* final_state, char* ws, Launch& L) {
    const long long T = l.T, H = p.nheads, G = p.ngroups, N = p.dstate;
    WalkArgs a = common(p, l, ld, cu);
    if (!(a.status = status_word())) return cudaErrorUnknown;
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
    cudaError_t err = cudaSuccess;
    if (few_fits(a)) {
        return few_tokens(a, p.dtype, L);
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
    return err;
}
cudaError_t run_backward(const ssd_linattn_t& p, const Plan& l, const void* q, const void* k, const void* v,
                     const float* ld, const int32_t* cu, const float* initial_state, const void* dout,
                     const float* d_final_state, void* dq, void* dk, void* dv, float* d_initial_state, char* ws,
                     Launch& L) {
    const long long T = l.T, H = p.nheads, G = p.ngroups, P = p.headdim, N = p.dstate;
    WalkArgs a = common(p, l, ld, cu);
    if (!(a.status = status_word())) return cudaErrorUnknown;
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
    return err;
}

// The copies between a call's tensors and those in the workspace.
struct Padding {
    const ssd_linattn_t &u, &p;  // as the user has it, and as it is in the workspace
    const Plan& l;
    char* ws;
    Copies a = {};
    void add(const void* from, void* to, long long n, long long fs, long long ts, int h, int c, int fh, int fc,
             int fw, int tw, int f32) {
        a.c[a.n++] = {from, to, n, fs, ts, h, c, fh, fc, fw, tw, f32};
    }
    void* in(const void* x, size_t at, long long stride, int heads, int width, int wide) {
        add(x, ws + at, l.T, stride, (long long)heads * wide, heads, wide, heads, width, width, wide, 0);
        return ws + at;
    }
    void out(size_t at, void* x, long long stride, int heads, int width, int wide) {
        add(ws + at, x, l.T, (long long)heads * wide, stride, heads, width, heads, width, wide, width, 0);
    }
    // states [n, H, P, N]; NULL where the call has none
    float* state_in(const float* x, size_t at) {
        if (!x) return nullptr;
        add(x, ws + at, (long long)l.n * u.nheads, (long long)u.headdim * u.dstate, (long long)p.headdim * p.dstate,
            p.headdim, p.dstate, u.headdim, u.dstate, u.dstate, p.dstate, 1);
        return reinterpret_cast<float*>(ws + at);
    }
    void state_out(size_t at, float* x) {
        if (x)
            add(ws + at, x, (long long)l.n * u.nheads, (long long)p.headdim * p.dstate,
                (long long)u.headdim * u.dstate, u.headdim, u.dstate, u.headdim, u.dstate, p.dstate, u.dstate, 1);
    }
    cudaError_t launch(const char* name, Launch& L) {
        long long items = 0;  // at most: four rows each
        for (int i = 0; i < a.n; ++i) items = std::max(items, a.c[i].n * ((a.c[i].h + 3) / 4));
        const long long blocks = std::min<long long>((items + kThreads / 32 - 1) / (kThreads / 32), 8ll * sm_count());
        L.begin(name);
        copies_kernel<<<dim3((unsigned)blocks, (unsigned)a.n), kThreads, 0, L.stream>>>(a);
        a.n = 0;
        return L.end();
    }
};

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
    const bool bwd = for_backward != 0;
    const Plan l = make_plan(*prob, bwd, tokens16(*prob, bwd));
    if (!l.fits) return SSD_ERR_UNSUPPORTED;
    // enough for the plain cores too, where a call's tensors may not start on 16 bytes
    *bytes = l.tc && !l.pads ? std::max(l.total, make_plan(*prob, bwd, false, false).total) : l.total;
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
    const Plan l = call_plan(p, false, {q, k, v, o}, workspace_bytes);
    if (!l.fits) return SSD_ERR_UNSUPPORTED;
    if (l.total > 0 && (!workspace || workspace_bytes < l.total)) return SSD_ERR_WORKSPACE;
    const long long states = (long long)l.n * H * P * N;
    if (rows_clash({Rows(o, T, p.o_stride, H * P, e), Rows(final_state, states, 4), Rows(workspace, l.total, 1)},
              {Rows(q, T, p.q_stride, H * N, e), Rows(k, T, p.k_stride, G * N, e),
               Rows(v, T, p.v_stride, G * P, e), Rows(log_decay, H, 4),
               Rows(cu_seqlens, p.nseq ? p.nseq + 1 : 0, 4), Rows(initial_state, states, 4)}))
        return SSD_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (l.pads) {
        const ssd_linattn_t& w = l.p;
        Padding c{p, w, l, ws};
        const void* wq = c.in(q, l.q, p.q_stride, p.nheads, p.dstate, w.dstate);
        const void* wk = c.in(k, l.k, p.k_stride, p.ngroups, p.dstate, w.dstate);
        const void* wv = c.in(v, l.v, p.v_stride, p.ngroups, p.headdim, w.headdim);
        const float* in = c.state_in(initial_state, l.s_in);
        err = c.launch("linattn_pad", L);
        if (err == cudaSuccess)
            err = run_forward(w, l, wq, wk, wv, log_decay, cu_seqlens, in, ws + l.o,
                          final_state ? reinterpret_cast<float*>(ws + l.s_out) : nullptr, ws, L);
        c.out(l.o, o, p.o_stride, p.nheads, p.headdim, w.headdim);
        c.state_out(l.s_out, final_state);
        if (err == cudaSuccess) err = c.launch("linattn_unpad", L);
    } else {
        err = run_forward(p, l, q, k, v, log_decay, cu_seqlens, initial_state, o, final_state, ws, L);
    }
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
    const bool own = p.nheads == p.ngroups;
    const Plan l = call_plan(p, true, {q, k, v, dout, dq, own ? dk : nullptr, own ? dv : nullptr}, workspace_bytes);
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
    char* ws = static_cast<char*>(workspace);
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err;
    if (l.pads) {
        const ssd_linattn_t& w = l.p;
        Padding c{p, w, l, ws};
        const void* wq = c.in(q, l.q, p.q_stride, p.nheads, p.dstate, w.dstate);
        const void* wk = c.in(k, l.k, p.k_stride, p.ngroups, p.dstate, w.dstate);
        const void* wv = c.in(v, l.v, p.v_stride, p.ngroups, p.headdim, w.headdim);
        const void* wo = c.in(dout, l.o, p.o_stride, p.nheads, p.headdim, w.headdim);
        const float* in = c.state_in(initial_state, l.s_in);
        const float* rin = c.state_in(d_final_state, l.r_in);
        err = c.launch("linattn_pad", L);
        if (err == cudaSuccess)
            err = run_backward(w, l, wq, wk, wv, log_decay, cu_seqlens, in, wo, rin, ws + l.dq, ws + l.dk, ws + l.dv,
                           d_initial_state ? reinterpret_cast<float*>(ws + l.s_out) : nullptr, ws, L);
        c.out(l.dq, dq, p.dq_stride, p.nheads, p.dstate, w.dstate);
        c.out(l.dk, dk, p.dk_stride, p.ngroups, p.dstate, w.dstate);
        c.out(l.dv, dv, p.dv_stride, p.ngroups, p.headdim, w.headdim);
        c.state_out(l.s_out, d_initial_state);
        if (err == cudaSuccess) err = c.launch("linattn_unpad", L);
    } else {
        err = run_backward(p, l, q, k, v, log_decay, cu_seqlens, initial_state, dout, d_final_state, dq, dk, dv,
                       d_initial_state, ws, L);
    }
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
