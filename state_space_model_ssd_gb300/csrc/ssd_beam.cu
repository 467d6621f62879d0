// Beam search: the selection of the best candidates over beams and vocabulary, and the move of
// cached states to the beams that go on from them.
//
// Selection.  A candidate's score is scores_i + x_t - log sum exp x.  Two launches, the second of which
// starts while the first ends:
//  * A block takes a slice of one beam's logits, which its threads hold in registers: read once,
//    bound by those bytes.  It leaves the slice's maximum, the sum of exp(x - maximum), and its
//    `keep` best logits.  To find them each of the eight warps takes the r-th best of its threads' own
//    maxima, r = keep / 8 rounded up: at least `keep` elements of the slice reach the lowest of the
//    eight, and few more do (about 60 of 8192 for 16).  Those are gathered and ranked.
//  * A block for each batch row adds up the slices' sums in float64, turns the slices' best into
//    scores in float64, and takes the best in the same way.  Between beams, whose scores differ by
//    their logarithms' rounding, float64 decides; within a beam the logits do.
// Ranks are counted (how many others come before), so that nothing depends on an order of arrival.
// GB300: 64 x 8 x 50277 float32 logits, 16 kept: MEASURE_A us; 1 x 4 x 50277 bf16, 8 kept: MEASURE_B us.
//
// Reordering.  The copies follow from slots and parents alone, up to 64 of each a batch row: every
// block works them out for its row again and copies its share of each state.
#include <limits.h>
#include <math.h>

#include <algorithm>

#include "layer_device.cuh"
#include "layer_host.cuh"

namespace ssd {
namespace layer {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMostKeep = 64, kMostBeams = 64;

// A number that is larger for larger floats; -0 counts as 0.  NaN is dealt with before.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long ordered(double x) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

struct SelectArgs {
    const void* logits;
    const float* scores;
    const uint8_t* finished;
    float* out_scores;
    int *parents, *tokens;
    // of slice s of beam row r: best[(r slices + s) keep + i], the logit and its token (-1: none)
    float* best;
    int* best_token;
    float2* sums;  // the slice's maximum, the sum of exp(x - maximum)
    long long stride;
    int beams, vocab, keep, slices, pad;
};

// The first `keep` of `m` pairs (key, index), largest key first, equal keys by index, to ranks
// 0 .. min(m, keep) - 1: sink(rank, i) for the i-th pair.
template <typename Key, typename Sink>
__device__ __forceinline__ void rank_all(const Key* key, const int* idx, int m, int keep, Sink sink) {
    for (int i = threadIdx.x; i < m; i += kThreads) {
        const Key x = key[i];
        const int at = idx[i];
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < m; ++j) before += key[j] > x || (key[j] == x && idx[j] < at);
        if (before < keep) sink(before, i);
    }
}
// The largest key of a warp.
__device__ __forceinline__ uint32_t warp_max(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
__device__ __forceinline__ unsigned long long warp_max(unsigned long long x) {
    const uint32_t hi = (uint32_t)(x >> 32), top = warp_max(hi);
    return (unsigned long long)top << 32 | warp_max(hi == top ? (uint32_t)x : 0u);
}
// The r-th largest of a warp's keys (0 where there are fewer).
template <typename Key>
__device__ __forceinline__ Key warp_nth(Key x, int r, int lane) {
    Key best = warp_max(x);
    for (int k = 1; k < r; ++k) {  // the first lane that has it gives it up
        const unsigned mine = __ballot_sync(0xffffffffu, x == best);
        if (lane == __ffs(mine) - 1) x = 0;
        best = warp_max(x);
    }
    return best;
}

template <typename T, int E>
__global__ void __launch_bounds__(kThreads, 4) beam_slice_kernel(const SelectArgs a) {
    constexpr int kList = 2048;  // more candidates than this (equal ones) take the long way
    __shared__ uint32_t lkey[kList];
    __shared__ int lidx[kList];
    __shared__ uint32_t top_key[kWarps], nth_key[kWarps];
    __shared__ float part[kWarps];
    __shared__ int count;
    const int row = blockIdx.y, slice = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (a.finished && a.finished[row]) return;
    const T* x = static_cast<const T*>(a.logits) + (long long)row * a.stride;
    const int base = slice * kThreads * E, n = min(kThreads * E, a.vocab - base);
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = e * kThreads + tid;
        f[e] = i < n ? static_cast<float>(x[base + i]) : -INFINITY;
    }
    float top = f[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(f[e], top);  // the other one of a NaN and a number
    const uint32_t mine = tid < n ? ordered(top) : 0u;
    const uint32_t best = warp_max(mine), nth = warp_nth(mine, (a.keep + kWarps - 1) / kWarps, lane);
    if (tid == 0) count = 0;
    if (lane == 0) top_key[warp] = best, nth_key[warp] = nth;
    __syncthreads();
    uint32_t mk = top_key[0], bound = nth_key[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mk = max(mk, top_key[w]), bound = min(bound, nth_key[w]);
    // a warp without that many threads with elements bounds nothing
    const float low = bound ? __uint_as_float(bound & 0x80000000u ? bound ^ 0x80000000u : ~bound) : -INFINITY;
    const float m = __uint_as_float(mk & 0x80000000u ? mk ^ 0x80000000u : ~mk);
    const float shift = m == -INFINITY ? 0.f : m;  // nothing but -inf: a sum of 0, or of a NaN
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) sum += __expf(f[e] - shift);
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = e * kThreads + tid;
        if (f[e] >= low && i < n) {  // no NaN is: its beam has no candidates
            const int to = atomicAdd(&count, 1);
            if (to < kList) lkey[to] = ordered(f[e]), lidx[to] = i;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        float s = part[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s += part[w];
        a.sums[(long long)row * a.slices + slice] = make_float2(m, s);
    }
    const long long out = ((long long)row * a.slices + slice) * a.keep;
    int found = count;
    if (found <= kList) {
        rank_all(lkey, lidx, found, a.keep, [&](int rank, int i) {
            const uint32_t u = lkey[i];
            a.best[out + rank] = __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
            a.best_token[out + rank] = base + lidx[i];
        });
    } else {
        // one after the other: the best that comes behind the last one taken
        uint32_t last = 0xffffffffu;
        int last_i = -1;
        for (int r = 0; r < a.keep; ++r) {
            uint32_t key = 0u;
            int at = INT_MAX;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int i = e * kThreads + tid;
                const uint32_t k = ordered(f[e]);
                if (i < n && f[e] == f[e] && (k < last || (k == last && i > last_i)) && k > key) key = k, at = i;
            }
            const uint32_t wk = warp_max(key);
            const int wi = (int)__reduce_min_sync(0xffffffffu, (unsigned)(key == wk ? at : INT_MAX));
            __syncthreads();
            if (lane == 0) top_key[warp] = wk, nth_key[warp] = (uint32_t)wi;
            __syncthreads();
            last = top_key[0], last_i = (int)nth_key[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
                if (top_key[w] > last || (top_key[w] == last && (int)nth_key[w] < last_i))
                    last = top_key[w], last_i = (int)nth_key[w];
            if (tid == 0) {
                a.best[out + r] = __uint_as_float(last & 0x80000000u ? last ^ 0x80000000u : ~last);
                a.best_token[out + r] = base + last_i;
            }
        }
        found = a.keep;
    }
    for (int i = found + tid; i < a.keep; i += kThreads) a.best_token[out + i] = -1;
}

// Candidates of a thread and round of the merge.
constexpr int kRound = 4;

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const SelectArgs a) {
    constexpr int kList = kMostKeep + kRound * kThreads;
    __shared__ double base[kMostBeams];  // scores_i - log sum exp, NaN: nothing to choose from
    __shared__ unsigned long long lkey[kList], nth_key[kWarps];
    __shared__ int lidx[kList], count;
    // the best so far, in order
    __shared__ unsigned long long rkey[kMostKeep];
    __shared__ int ridx[kMostKeep];
    const long long b = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = warp; i < a.beams; i += kWarps) {
        const long long row = b * a.beams + i;
        const float score = a.scores[row];
        double v = isfinite(score) ? (double)score : (double)NAN;
        if (!(a.finished && a.finished[row])) {
            float m = -INFINITY;
            const float2* s = a.sums + row * a.slices;
            for (int k = lane; k < a.slices; k += 32) m = fmaxf(m, s[k].x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            double t = 0.0;  // a slice of nothing but -inf has a sum of 0 or NaN
            for (int k = lane; k < a.slices; k += 32)
                t += s[k].x == -INFINITY ? (double)s[k].y : (double)s[k].y * exp((double)s[k].x - (double)m);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            v = isfinite(m) ? v - ((double)m + log(t)) : (double)NAN;
        }
        if (lane == 0) base[i] = v;
    }
    int have = 0;  // of the best so far
    const int per = a.slices * a.keep;
    const long long all = (long long)a.beams * per;
    __syncthreads();
    for (long long c0 = 0; c0 < all; c0 += kRound * kThreads) {
        unsigned long long ck[kRound], best = 0;
        int ci[kRound];
        // what a full list's last entry comes before is out
        const unsigned long long floor_key = have == a.keep ? rkey[a.keep - 1] : 0ull;
        const int floor_idx = have == a.keep ? ridx[a.keep - 1] : INT_MAX;
        bool any = false;
#pragma unroll
        for (int u = 0; u < kRound; ++u) {
            const long long c = c0 + u * kThreads + tid;
            ck[u] = 0ull, ci[u] = INT_MAX;
            if (c < all) {
                const int i = (int)(c / per), k = (int)(c - (long long)i * per);
                const long long row = b * a.beams + i;
                const bool ended = a.finished && a.finished[row];
                const double from = base[i];
                double v = -(double)INFINITY;
                int t = -1;
                if (ended || !isfinite(from)) {
                    // the first tokens, at -inf; an ended beam's padding token at its score
                    if (k < a.keep && k < a.vocab) t = k;
                    if (ended && isfinite(from)) {
                        if (k == a.keep - 1 && a.pad >= a.keep) t = a.pad;
                        if (t == a.pad) v = from;
                    }
                } else {
                    t = a.best_token[row * per + k];
                    if (t >= 0) v = from + (double)a.best[row * per + k];
                }
                if (t >= 0) {
                    const unsigned long long key = ordered(v);
                    const int at = i * a.vocab + t;
                    if (key > floor_key || (key == floor_key && at < floor_idx)) {
                        ck[u] = key, ci[u] = at, any = true;
                        best = max(best, key);
                    }
                }
            }
        }
        const unsigned long long nth = warp_nth(best, (a.keep + kWarps - 1) / kWarps, lane);
        if (lane == 0) nth_key[warp] = nth;
        if (tid == 0) count = have;
        if (tid < have) lkey[tid] = rkey[tid], lidx[tid] = ridx[tid];
        if (!__syncthreads_or(any)) continue;
        unsigned long long bound = nth_key[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) bound = min(bound, nth_key[w]);
#pragma unroll
        for (int u = 0; u < kRound; ++u)
            if (ci[u] != INT_MAX && ck[u] >= bound) {
                const int to = atomicAdd(&count, 1);
                lkey[to] = ck[u], lidx[to] = ci[u];
            }
        __syncthreads();
        rank_all(lkey, lidx, count, a.keep, [&](int rank, int i) { rkey[rank] = lkey[i], ridx[rank] = lidx[i]; });
        have = min(count, a.keep);
        __syncthreads();
    }
    if (tid < have) {
        const unsigned long long u = rkey[tid];
        const long long out = b * a.keep + tid;
        a.out_scores[out] = (float)__longlong_as_double((long long)(u >> 63 ? u ^ 0x8000000000000000ull : ~u));
        a.parents[out] = ridx[tid] / a.vocab;
        a.tokens[out] = ridx[tid] % a.vocab;
    }
}

// ---------------------------------------------------------------- reordering
constexpr int kMostCaches = 96;  // of one launch
struct ReorderArgs {
    const int *slots, *parents;
    int* new_slots;
    char* cache[kMostCaches];
    long long bytes[kMostCaches], stride[kMostCaches];
    int first[kMostCaches + 1];  // pieces of a slot before each cache's
    int ncaches, beams, nslots;
};
constexpr int kPiece = 4 * 16 * kThreads;  // bytes that a block has on their way at a time

// One piece of a copy in words of V.
template <typename V>
__device__ __forceinline__ void copy_piece(char* dst, const char* src, int bytes) {
    V* d = reinterpret_cast<V*>(dst);
    const V* s = reinterpret_cast<const V*>(src);
    const int n = bytes / (int)sizeof(V);
    for (int i0 = 0; i0 < n; i0 += 4 * kThreads) {
        V v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kThreads + threadIdx.x;
            if (i < n) v[u] = s[i];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kThreads + threadIdx.x;
            if (i < n) d[i] = v[u];
        }
    }
}

__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const __grid_constant__ ReorderArgs a) {
    __shared__ int par[kMostBeams], slot[kMostBeams], src[kMostBeams], dst[kMostBeams];
    __shared__ unsigned used[2], repeats[2], moves[2];  // beams, a bit each
    const int b = blockIdx.y, K = a.beams, tid = threadIdx.x, lane = tid & 31;
    if (tid < K) {
        par[tid] = a.parents[(long long)b * K + tid];
        slot[tid] = a.slots[(long long)b * K + tid];
    }
    if (tid < 2) used[tid] = 0u;
    __syncthreads();
    const unsigned below = (1u << lane) - 1;
    const int p = tid < K ? par[tid] : -1;
    const bool there = p >= 0 && p < K;
    bool again = false;  // whether a beam before this one has its parent
    if (there) {
        for (int j = 0; j < tid; ++j) again |= par[j] == p;
        atomicOr(&used[p >> 5], 1u << (p & 31));
    }
    if (tid < 64) {
        const unsigned r = __ballot_sync(0xffffffffu, again);
        if (lane == 0) repeats[tid >> 5] = r;
    }
    __syncthreads();
    int from = -1, to = -1;
    if (there) {
        from = to = slot[p];
        if (again) {  // as many beams that nobody goes on from are taken as repeat a parent before it
            int rank = __popc(repeats[tid >> 5] & below) + (tid >= 32 ? __popc(repeats[0]) : 0);
            const unsigned free0 = ~used[0], free1 = ~used[1];
            const int in0 = __popc(free0);
            to = slot[rank < in0 ? __fns(free0, 0, rank + 1) : 32 + __fns(free1, 0, rank - in0 + 1)];
        }
    }
    if (tid < K && blockIdx.x == 0) a.new_slots[(long long)b * K + tid] = to;
    const bool move = from != to && from >= 0 && to >= 0 && from < a.nslots && to < a.nslots;
    if (tid < 64) {
        const unsigned m = __ballot_sync(0xffffffffu, move);
        if (lane == 0) moves[tid >> 5] = m;
    }
    __syncthreads();
    if (move) {
        const int at = __popc(moves[tid >> 5] & below) + (tid >= 32 ? __popc(moves[0]) : 0);
        src[at] = from, dst[at] = to;
    }
    const int copies = __popc(moves[0]) + __popc(moves[1]);
    __syncthreads();
    const int per = a.first[a.ncaches];
    const long long tasks = (long long)copies * per;
    for (long long t = blockIdx.x; t < tasks; t += gridDim.x) {
        const int j = (int)(t / per), r = (int)(t - (long long)j * per);
        int c = 0, hi = a.ncaches - 1;
        while (c < hi) {  // the cache that piece r is of
            const int mid = (c + hi + 1) >> 1;
            if (a.first[mid] <= r)
                c = mid;
            else
                hi = mid - 1;
        }
        const long long at = (long long)(r - a.first[c]) * kPiece;
        const int bytes = (int)min((long long)kPiece, a.bytes[c] - at);
        char* to_ = a.cache[c] + dst[j] * a.stride[c] + at;
        const char* from_ = a.cache[c] + src[j] * a.stride[c] + at;
        const uintptr_t off = (uintptr_t)a.cache[c] | (uintptr_t)a.stride[c] | (uintptr_t)a.bytes[c];
        if ((off & 15) == 0)
            copy_piece<uint4>(to_, from_, bytes);
        else if ((off & 3) == 0)
            copy_piece<uint32_t>(to_, from_, bytes);
        else
            copy_piece<char>(to_, from_, bytes);
    }
}

// ---------------------------------------------------------------- host
ssd_status_t check_beam(const ssd_beam_t* p) {
    if (!p || p->batch < 1 || p->beams < 1 || p->vocab < 1 || p->keep < 1 || !dtype_ok(p->dtype) ||
        p->stride < p->vocab || p->pad_token < 0 || p->pad_token >= p->vocab ||
        p->keep > (long long)p->beams * p->vocab)
        return SSD_ERR_INVALID_ARG;
    if (p->beams > kMostBeams || p->keep > kMostKeep || p->vocab > (1 << 24) ||
        p->batch * p->beams > 65535)
        return SSD_ERR_UNSUPPORTED;
    return SSD_OK;
}
constexpr int kWide = 32, kNarrow = 8;  // elements a thread
struct SelectPlan {
    int e, slices;
    size_t best, token, sums, total;
};
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
// Eight elements a thread while slices of 32 leave fewer than two blocks for each SM: then a slice's
// latency is all there is.
SelectPlan select_plan(const ssd_beam_t& p) {
    SelectPlan l;
    auto slices = [&](int e) { return (p.vocab + kThreads * e - 1) / (kThreads * e); };
    l.e = p.batch * p.beams * slices(kWide) >= 2LL * sm_count() ? kWide : kNarrow;
    l.slices = slices(l.e);
    const size_t n = (size_t)p.batch * p.beams * l.slices;
    l.best = 0;
    l.token = up(n * p.keep * 4);
    l.sums = l.token + up(n * p.keep * 4);
    l.total = l.sums + up(n * 8);
    return l;
}

template <typename T>
void launch_slices(const SelectArgs& a, const SelectPlan& l, dim3 grid, cudaStream_t s) {
    if (l.e == kWide)
        beam_slice_kernel<T, kWide><<<grid, kThreads, 0, s>>>(a);
    else
        beam_slice_kernel<T, kNarrow><<<grid, kThreads, 0, s>>>(a);
}

}  // namespace
}  // namespace layer
}  // namespace ssd

using namespace ssd;
using namespace ssd::layer;

extern "C" {

ssd_status_t ssd_beam_select_workspace_size(const ssd_beam_t* beam, size_t* bytes) {
    if (!bytes) return SSD_ERR_INVALID_ARG;
    const ssd_status_t st = check_beam(beam);
    if (st != SSD_OK) return st;
    *bytes = select_plan(*beam).total;
    return SSD_OK;
}

ssd_status_t ssd_beam_select(const ssd_beam_t* beam, const void* logits, const float* scores,
                             const uint8_t* finished, float* out_scores, int32_t* parents,
                             int32_t* tokens, void* workspace, size_t workspace_bytes,
                             void* stream) {
    set_last_launches(0);
    const ssd_status_t st = check_beam(beam);
    if (st != SSD_OK) return st;
    const ssd_beam_t& p = *beam;
    if (!logits || !scores || !out_scores || !parents || !tokens) return SSD_ERR_INVALID_ARG;
    const size_t e = dtype_size(p.dtype);
    if (!aligned_to(logits, e) || !aligned_to(scores, 4) || !aligned_to(out_scores, 4) ||
        !aligned_to(parents, 4) || !aligned_to(tokens, 4) || !aligned_to(workspace, 256))
        return SSD_ERR_ALIGNMENT;
    const SelectPlan l = select_plan(p);
    if (!workspace || workspace_bytes < l.total) return SSD_ERR_WORKSPACE;
    const long long rows = p.batch * p.beams, outs = p.batch * p.keep;
    if (clash({Span(out_scores, outs, 4), Span(parents, outs, 4), Span(tokens, outs, 4),
               Span(workspace, l.total, 1)},
              {Span(logits, rows, p.stride, p.vocab, e), Span(scores, rows, 4),
               Span(finished, finished ? rows : 0, 1)}))
        return SSD_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    SelectArgs a = {};
    a.logits = logits, a.scores = scores, a.finished = finished;
    a.out_scores = out_scores, a.parents = parents, a.tokens = tokens;
    a.best = reinterpret_cast<float*>(ws + l.best);
    a.best_token = reinterpret_cast<int*>(ws + l.token);
    a.sums = reinterpret_cast<float2*>(ws + l.sums);
    a.stride = p.stride, a.beams = p.beams, a.vocab = p.vocab, a.keep = p.keep, a.slices = l.slices;
    a.pad = p.pad_token;
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    L.begin("beam_slices");
    const dim3 grid((unsigned)l.slices, (unsigned)rows);
    if (p.dtype == SSD_DTYPE_BF16)
        launch_slices<__nv_bfloat16>(a, l, grid, L.stream);
    else
        launch_slices<float>(a, l, grid, L.stream);
    cudaError_t err = L.end();
    if (err == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)p.batch);
        cfg.blockDim = dim3(kThreads);
        cfg.stream = L.stream;
        cudaLaunchAttribute at = {};
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        L.begin("beam_merge");
        err = cudaLaunchKernelEx(&cfg, beam_merge_kernel, a);
        const cudaError_t last = L.end();
        if (err == cudaSuccess) err = last;
    }
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

ssd_status_t ssd_beam_reorder(int64_t batch, int32_t beams, const int32_t* slots,
                              const int32_t* parents, int32_t* new_slots, int32_t ncaches,
                              void* const* caches, const int64_t* slot_bytes,
                              const int64_t* slot_strides, int32_t nslots, void* stream) {
    set_last_launches(0);
    if (batch < 1 || beams < 1 || ncaches < 0 || nslots < 1 || !slots || !parents || !new_slots ||
        (ncaches > 0 && (!caches || !slot_bytes || !slot_strides)))
        return SSD_ERR_INVALID_ARG;
    if (beams > kMostBeams || batch > 65535 || ncaches > (1 << 16)) return SSD_ERR_UNSUPPORTED;
    if (!aligned_to(slots, 4) || !aligned_to(parents, 4) || !aligned_to(new_slots, 4)) return SSD_ERR_ALIGNMENT;
    const Span out(new_slots, batch * beams, 4), si(slots, batch * beams, 4), pi(parents, batch * beams, 4);
    if (clash({out}, {si, pi})) return SSD_ERR_INVALID_ARG;
    for (int i = 0; i < ncaches; ++i) {
        if (!caches[i] || slot_bytes[i] < 0 || slot_strides[i] < slot_bytes[i]) return SSD_ERR_INVALID_ARG;
        const Span c(caches[i], nslots, slot_strides[i], slot_bytes[i], 1);
        if (clash({c}, {out, si, pi})) return SSD_ERR_INVALID_ARG;
        if (slot_bytes[i] > (1LL << 31)) return SSD_ERR_UNSUPPORTED;
    }
    Launch L;
    L.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaSuccess;
    int done = 0;
    do {  // as many caches a launch as its arguments hold
        ReorderArgs a = {};
        a.slots = slots, a.parents = parents, a.new_slots = new_slots;
        a.beams = beams, a.nslots = nslots;
        a.ncaches = std::min(ncaches - done, kMostCaches);
        for (int i = 0; i < a.ncaches; ++i) {
            a.cache[i] = static_cast<char*>(caches[done + i]);
            a.bytes[i] = slot_bytes[done + i], a.stride[i] = slot_strides[done + i];
            a.first[i + 1] = a.first[i] + (int)((a.bytes[i] + kPiece - 1) / kPiece);
        }
        // eight blocks an SM over the batch rows, no more than a row can have pieces
        const long long pieces = (long long)a.first[a.ncaches] * std::max(1, beams - 1);
        const long long blocks = std::min<long long>(pieces, (8LL * sm_count() + batch - 1) / batch);
        L.begin("beam_reorder");
        beam_reorder_kernel<<<dim3((unsigned)std::max<long long>(blocks, 1), (unsigned)batch), kThreads, 0,
                              L.stream>>>(a);
        err = L.end();
        done += a.ncaches;
    } while (err == cudaSuccess && done < ncaches);
    set_last_launches(L.count);
    return err == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
