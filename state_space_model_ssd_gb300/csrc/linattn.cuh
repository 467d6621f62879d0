// Linear attention with a decay for each head: what its kernels share.
//
// Forward and backward are the same walk over the tokens with other tensors in its three places.
// With q, k of kd channels, v of vd, and S of kd x vd, a walk computes in each chunk of n tokens
//     out_i = si sum_{j <= i} a^(i-j) (q_i . k_j) v_j + sx a^(i+1-e) S^T q_i,
//     S     = a^n S + su sum_j a^(n-1-j+e) k_j v_j^T,
// where i and j count in the walk's direction and e is 1 in a walk from the end:
//     o   from (q, k, v)    forwards,   si = sx = scale, su = 1
//     dq  from (do, v, k)   forwards,   si = sx = scale, su = 1       (the same states, transposed)
//     dv  from (k, q, do)   from the end, si = su = scale, sx = 1     (the states' adjoints)
//     dk  from (v, do, q)   from the end, si = su = scale, sx = 1     (the same, transposed)
// A long sequence is cut into segments of Ls tokens: one launch sums what each segment adds to
// the state, a scan over the segments leaves the state that enters each, and the walks start from
// those.
#pragma once

#include "layer_host.cuh"
#include "ssd_device.cuh"

namespace ssd {
namespace linattn {

struct Pass {
    const void *q, *k, *v;
    void* out;
    long long qs, ks, vs, os;  // elements from one token to the next
    int kd, vd;
    int qr, kr, vr, outr;      // heads that share one of the tensor's
    int out_f32;               // out is float32 whatever the inputs are
    int reverse;
    float si, sx, su;
    // states: element (n, p) of sequence s, head h at (s H + h) kd vd + n sn + p sp
    const float* s_in;         // before the walk's first token, per sequence (NULL: zero)
    float* s_out;              // after its last one, per sequence (NULL: not wanted)
    const float* s_seg;        // before each segment (NULL: the sequences are not cut)
    float* s_sum;              // what each segment adds (the summing launch)
    long long sn, sp;
    int tiles;                 // tiles of vd
};

struct WalkArgs {
    Pass pass[3];
    int npass, tiles;          // tiles of all passes
    const float* ld;
    const int* cu;
    long long T, rowlen;       // rowlen: tokens of a dense row
    int nseq, H;
    int Ls;                    // tokens a segment; 0: the sequences are not cut
    int per;                   // segments of a dense row
    long long ids;             // segments, with holes where the sequences are packed
    int* status;
};

// Segment `id`: `k` counts those of its sequence.
struct Seg {
    long long start;
    int len, seq, k, cnt;
    bool there;
};

__device__ __forceinline__ long long border(const WalkArgs& a, int s) {
    const long long v = a.cu[s];
    return v < 0 ? 0 : v > a.T ? a.T : v;
}
// The tokens of no sequence, before the first border and from the last one on: their outputs are zero.
struct Outside {
    long long first, last, n;
    __device__ __forceinline__ explicit Outside(const WalkArgs& a)
        : first(border(a, 0)), last(border(a, a.nseq)), n(first + a.T - last) {}
    __device__ __forceinline__ long long token(long long i) const { return i < first ? i : last + (i - first); }
};
// The first segment of sequence s; packed sequences have cu[s] / Ls + s of them before it, some
// of which may be holes: ceil(len / Ls) is at most floor((cu + len) / Ls) - floor(cu / Ls) + 1.
__device__ __forceinline__ long long first_segment(const WalkArgs& a, int s) {
    if (!a.Ls) return s;
    return a.cu ? (long long)((unsigned)border(a, s) / (unsigned)a.Ls) + s : (long long)s * a.per;
}
__device__ __forceinline__ Seg sequence(const WalkArgs& a, int s) {
    Seg g;
    g.seq = s;
    if (a.cu) {
        g.start = border(a, s);
        const long long len = border(a, s + 1) - g.start;
        g.len = len < 0 ? 0 : (int)len;
    } else {
        g.start = s * a.rowlen;
        g.len = (int)a.rowlen;
    }
    g.cnt = a.Ls ? (g.len + a.Ls - 1) / a.Ls : 1;
    if (g.cnt < 1) g.cnt = 1;
    g.k = 0;
    g.there = true;
    return g;
}
__device__ __forceinline__ Seg segment(const WalkArgs& a, long long id) {
    int s = (int)id;
    if (a.Ls && !a.cu) {
        s = (int)(id / a.per);
    } else if (a.Ls) {
        int lo = 0, hi = a.nseq - 1;  // the last sequence whose first segment is not behind id
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first_segment(a, mid) <= id)
                lo = mid;
            else
                hi = mid - 1;
        }
        s = lo;
    }
    Seg g = sequence(a, s);
    if (!a.Ls) return g;
    const long long k = id - first_segment(a, s);
    g.there = k >= 0 && k < g.cnt;
    if (!g.there) return g;
    g.k = (int)k;
    g.start += k * a.Ls;
    const int left = g.len - g.k * a.Ls;
    g.len = left < a.Ls ? left : a.Ls;
    return g;
}

// a^d from log2 a; a = 0 too.
__device__ __forceinline__ float power(float ld2, int d) { return d == 0 ? 1.f : exp2f(ld2 * d); }
// A state decayed over d tokens, a^d S.  Near 1 the factor is applied as S + (a^d - 1) S, so that
// a state decayed over many chunks does not carry the rounding of a^d as often as it is decayed;
// below 1/2 that sum would cancel, and few factors matter.
struct Decay {
    float m, keep;  // keep: 1 or 0
    Decay() = default;
    __device__ __forceinline__ Decay(float ld, int d) {
        const float m1 = d == 0 ? 0.f : expm1f(ld * d);
        keep = m1 > -0.5f ? 1.f : 0.f;
        m = keep != 0.f ? m1 : expf(ld * d);
    }
    __device__ __forceinline__ float operator()(float S) const { return fmaf(m, S, keep * S); }
};

// The tile of item `t` among the passes' tiles.
__device__ __forceinline__ const Pass& pass_of(const WalkArgs& a, int& t) {
    int p = 0;
    while (p + 1 < a.npass && t >= a.pass[p].tiles) t -= a.pass[p++].tiles;
    return a.pass[p];
}

// A forward of at most so many tokens a sequence is stepped through them (ssd_linattn_step.cu).
constexpr int kFewTokens = 16;
bool few_fits(const WalkArgs& a);
cudaError_t few_tokens(const WalkArgs& a, int dtype, Launch& L);

// Columns of v a block of the plain walk takes: 64, for which it computes the scores half as often as with 32
// (32768 tokens of 16 heads in float32, 64 x 128, forward 1354 us, with 32 1646; 90 columns 760 and 1260),
// but for passes that have no more than 32.
inline int simt_tile(int vd) { return vd <= 32 ? 32 : 64; }

// The tensor-core walk (ssd_linattn_tc.cu): whether it takes these tensors, and the launches.
constexpr int kTcTile = 64;
constexpr int kTcChunk = 128;
bool tc_fits(const Pass& p);
cudaError_t tc_sums(const WalkArgs& a, Launch& L);
cudaError_t tc_walk(const WalkArgs& a, Launch& L);

}  // namespace linattn
}  // namespace ssd
