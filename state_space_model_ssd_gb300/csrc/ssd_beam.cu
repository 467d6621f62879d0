// Beam search: the selection of the best candidates over beams and vocabulary, and the move of
// cached states to the beams that go on from them.
//
// Selection.  A candidate's score is scores_i + x_t - log sum exp x.  Two launches, the second of which
// starts while the first ends:
//  * A block takes a slice of one beam's logits, which its threads hold in registers: read once,
//    bound by those bytes.  It leaves the slice's maximum rounded up, the sum of exp(x - that), and
//    its `keep` best logits.  To find them each of the eight warps takes the r-th best of its threads' own
//    maxima, r = keep / 8 rounded up: at least `keep` elements of the slice reach the lowest of the
//    eight, and few more do (about 35 of 4096 for 16).  Those are gathered and ranked.  Elements at -inf are
//    neither: a masked vocabulary costs no more than an open one (one token in a hundred open 51 us, where
//    ranking the others took 524).
//  * A block for each batch row adds up the slices' sums as pairs of floats, turns the slices' best into
//    scores in float64, and takes the best in the same way.  Equal scores of one beam are ordered by
//    their logits.
// Ranks are counted (how many others come before), so that nothing depends on an order of arrival.
// GB300: 64 x 8 x 50277 float32 logits, 16 kept: 53 us, of which the slices 36 (42 % of the copy rate:
// 400 instructions a warp for sixteen elements a thread keep the SMs busier than memory) and the
// merge, a chain of latencies, 16.  1 x 4 x 50277 bf16, 8 kept: 13 us a call, 9.9 in a replayed graph.
//
// Reordering.  The copies follow from slots and parents alone, up to 64 of each a batch row: every
// block works them out for its row again, in masks of bits, and copies pieces of 16 KB in turn over all
// copies and caches.  Bound by the bytes of the states that move: 16 x 4 beams, half of them doubled,
// 24 layers of states of 24 heads x 64 x 128 and windows: 196 us (92 % of the copy rate; each cache
// shared out by itself 221).
#include <float.h>
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
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ unsigned long long ordered(double x) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ double unordered(unsigned long long u) {
    return __longlong_as_double((long long)(u >> 63 ? u ^ 1ull << 63 : ~u));
}
// A number as the sum of two floats, the second at most half a step of the first: 48 bits without the
// float64 units, of which this GPU has few.  The sums are Knuth's and Dekker's.
struct Pair {
    float hi, lo;
    __device__ __forceinline__ Pair plus(float x) const {
        const float s = hi + x, b = s - hi;
        const float rest = (hi - (s - b)) + (x - b) + lo;  // exact but for the last sum
        const float t = s + rest;
        return Pair{t, (s - t) + rest};
    }
    __device__ __forceinline__ Pair plus(Pair x) const {
        const Pair r = plus(x.hi);
        const float t = r.hi + (r.lo + x.lo);
        return Pair{t, (r.hi - t) + (r.lo + x.lo)};
    }
    __device__ __forceinline__ Pair times(Pair x) const {
        const float p = hi * x.hi, rest = fmaf(hi, x.hi, -p) + (hi * x.lo + lo * x.hi);
        const float t = p + rest;
        return Pair{t, (p - t) + rest};
    }
};
// e^-n for a whole n >= 0, by the powers of two in n.
__device__ __forceinline__ Pair exp_minus(float n) {
    const Pair e[7] = {{0.3678794503211975f, -9.149755619830557e-09f}, {0.1353352814912796f, 1.7453331002670325e-09f}, {0.018315639346837997f, -4.581038048900865e-10f}, {0.000335462624207139f, 3.695373000656144e-12f}, {1.1253517584464134e-07f, -1.1253822674030483e-15f}, {1.2664165777252073e-14f, -2.2815788510487642e-22f}, {1.6038109389511792e-28f, -4.840254038107756e-36f}};
    if (n > 103.f) return Pair{0.f, 0.f};
    Pair r{1.f, 0.f};
    const int k = (int)n;
#pragma unroll
    for (int b = 0; b < 7; ++b)
        if (k >> b & 1) r = r.times(e[b]);
    return r;
}
// log x for x > 0: with x = 2^e f, f within sqrt(2) of 1, and s = (f - 1) / (f + 1),
// log f = 2 s + 2 s^3 / 3 + 2 s^5 / 5 + ..., the first term as a pair.  Off by a few 1e-10, so that what the
// slices' float32 sums are off by is what counts (some 1e-8 of 50277 normal logits).
__device__ __forceinline__ Pair log_of(Pair x) {
    int e = (int)(__float_as_uint(x.hi) >> 23) - 127;
    float f = __uint_as_float((__float_as_uint(x.hi) & 0x7fffffu) | 0x3f800000u);
    if (f > 1.41421356f) f *= 0.5f, ++e;
    const float lo = ldexpf(x.lo, -e);
    const Pair n = Pair{f - 1.f, 0.f}.plus(lo), d = Pair{f, lo}.plus(1.f);
    const float s = n.hi / d.hi;
    const float rest = (fmaf(-s, d.hi, n.hi) + (n.lo - s * d.lo)) / d.hi;
    const float z = s * s;
    float p = 2.f / 13.f;
    p = fmaf(p, z, 2.f / 11.f), p = fmaf(p, z, 2.f / 9.f), p = fmaf(p, z, 2.f / 7.f);
    p = fmaf(p, z, 2.f / 5.f), p = fmaf(p, z, 2.f / 3.f);
    // log 2 in a part whose multiples are exact, and the rest
    return Pair{e * 0.693145751953125f, 0.f}.plus(Pair{2.f * s, 2.f * rest + s * (z * p)}).plus(e * 1.428606765330187e-06f);
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
    float2* sums;  // the slice's maximum rounded up, the sum of exp(x - that)
    long long stride;
    int beams, vocab, keep, slices, pad;
};

// The first `keep` of `m` pairs (key, index), largest key first, equal keys by index, to ranks
// 0 .. min(m, keep) - 1: sink(rank, i) for the i-th pair.
template <typename Key, typename Index, typename Sink>
__device__ __forceinline__ void rank_all(const Key* key, const Index* idx, int m, int keep, Sink sink) {
    for (int i = threadIdx.x; i < m; i += kThreads) {
        const Key x = key[i];
        const Index at = idx[i];
        int before = 0;
#pragma unroll 4
        for (int j = 0; j < m; ++j) before += key[j] > x || (key[j] == x && idx[j] < at);
        if (before < keep) sink(before, i);
    }
}
// The largest key of a warp.
__device__ __forceinline__ uint32_t warp_max(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
// The r-th largest of a warp's keys (0 where there are fewer).
__device__ __forceinline__ uint32_t warp_nth(uint32_t x, int r, int lane) {
    uint32_t best = warp_max(x);
    for (int k = 1; k < r; ++k) {  // the first lane that has it gives it up
        const unsigned mine = __ballot_sync(0xffffffffu, x == best);
        if (lane == __ffs(mine) - 1) x = 0;
        best = warp_max(x);
    }
    return best;
}

template <typename T, int E>
__global__ void __launch_bounds__(kThreads, 6) beam_slice_kernel(const SelectArgs a) {
    // more candidates than are ranked: with less shared memory for a block the merge's do not fit in beside
    // them before the SM is empty (64 x 8 x 50277 float32: 54.5 us, so 53.0)
    constexpr int kList = 2048;
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
    x += base + tid;
    if (n == kThreads * E) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = static_cast<float>(x[e * kThreads]);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = e * kThreads + tid < n ? static_cast<float>(x[e * kThreads]) : -INFINITY;
    }
    float top = f[0];
#pragma unroll
    for (int e = 1; e < E; ++e) top = fmaxf(f[e], top);  // the other one of a NaN and a number
    const uint32_t mine = top > -INFINITY ? ordered(top) : 0u;  // 0: nothing to choose from
    const uint32_t best = warp_max(mine), nth = warp_nth(mine, (a.keep + kWarps - 1) / kWarps, lane);
    if (tid == 0) count = 0;
    if (lane == 0) top_key[warp] = best, nth_key[warp] = nth;
    __syncthreads();
    const uint32_t mk = warp_max(lane < kWarps ? top_key[lane] : 0u);
    const uint32_t bound = ~warp_max(lane < kWarps ? ~nth_key[lane] : 0u);
    float low = -FLT_MAX;
    if (bound) {
        low = unordered(bound);
    } else if (__syncthreads_count(mine != 0u) >= a.keep) {
        // masks leave a warp without that many threads with elements above -inf, which bounds nothing: the
        // keep-th best of all threads' own maxima, bit by bit
        uint32_t t = 0u;
        for (int bit = 31; bit >= 0; --bit) {
            const int reached = __syncthreads_count(mine >= (t | 1u << bit));
            if (reached >= a.keep) t |= 1u << bit;
            if (reached == a.keep) break;
        }
        low = unordered(t);
    }
    const float m = mk ? unordered(mk) : -INFINITY;
    // a whole number, so that sums of other slices come to it by whole powers of e; nothing but -inf: a
    // sum of 0, or of a NaN
    const float shift = m == -INFINITY ? 0.f : ceilf(m);
    F2 sums = both<F2>(0.f);
    unsigned reach = 0u;  // the elements that reach the bound, a bit each
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        float d[2];
        split(mul_(add_(join(f[e], f[e + 1]), both<F2>(-shift)), both<F2>(1.44269504f)), d);
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(d[0]));
        asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(d[1]));
        sums = add_(sums, join(d[0], d[1]));
        // no NaN reaches it: its beam has no candidates
        reach |= (f[e] >= low ? 1u << e : 0u) | (f[e + 1] >= low ? 2u << e : 0u);
    }
    float halves[2];
    split(sums, halves);
    float sum = halves[0] + halves[1];
    for (; reach; reach &= reach - 1) {
        const int i = (__ffs(reach) - 1) * kThreads + tid;
        if (i >= n) break;
        const int to = atomicAdd(&count, 1);
        if (to < kList) lkey[to] = ordered(static_cast<float>(x[i - tid])), lidx[to] = i;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        float s = part[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s += part[w];
        a.sums[(long long)row * a.slices + slice] = make_float2(m == -INFINITY ? m : shift, s);
    }
    const long long out = ((long long)row * a.slices + slice) * a.keep;
    int found = count;
    // Ranks take a step for each pair, of which a thread has that many; the long way takes some hundred
    // instructions and two barriers for each candidate kept.  Ties decide which is less: logits of one value,
    // 64 x 8 x 50277 float32, 16 kept, 247 us, ranked 769.  A limit of 22 sends open vocabularies the long way
    // (1 kept: 41.0 us, so 39.1), one of 200 leaves ties to the ranks (32 kept, one value: 513 and 909).
    if (found <= kList && found * ((found + kThreads - 1) / kThreads) <= 64 * a.keep) {
        rank_all(lkey, lidx, found, a.keep, [&](int rank, int i) {
            const uint32_t u = lkey[i];
            a.best[out + rank] = unordered(u);
            a.best_token[out + rank] = base + lidx[i];
        });
    } else {
        // one after the other: the best that comes behind the last one taken
        uint32_t last = 0xffffffffu, key = 0u;
        int last_i = INT_MAX, at = INT_MAX;
        for (int r = 0; r < a.keep; ++r) {
            if (at == last_i) {  // at first, and where the last one was this thread's
                key = 0u, at = INT_MAX;
#pragma unroll 4
                for (int i = tid; i < n; i += kThreads) {
                    const float logit = static_cast<float>(x[i - tid]);
                    const uint32_t k = ordered(logit);
                    if (logit >= low && (k < last || (k == last && i > last_i)) && k > key) key = k, at = i;
                }
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
                a.best[out + r] = unordered(last);
                a.best_token[out + r] = base + last_i;
            }
        }
        found = a.keep;
    }
    // where fewer are above -inf, the slice's first tokens at -inf
#pragma unroll 1
    for (int e = 0; e < n && found < a.keep; e += kThreads) {
        const int i = e + tid;
        const bool masked = i < n && static_cast<float>(x[e]) == -INFINITY;
        const unsigned those = __ballot_sync(0xffffffffu, masked);
        __syncthreads();
        if (lane == 0) top_key[warp] = __popc(those);
        __syncthreads();
        int to = found + __popc(those & ((1u << lane) - 1));
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            to += w < warp ? top_key[w] : 0;
            found += top_key[w];
        }
        if (masked && to < a.keep) a.best[out + to] = -INFINITY, a.best_token[out + to] = base + i;
    }
    for (int i = found + tid; i < a.keep; i += kThreads) a.best_token[out + i] = -1;
}

// Candidates of a thread and round of the merge.
constexpr int kRound = 4;

// Where candidates of equal scores come: by beam, logit (largest first) and token.  A beam's scores
// are one float64 sum each, which never falls where the logit rises, so that its candidates come in the
// order of their logits however coarse the sums are.
__device__ __forceinline__ unsigned long long place(int beam, uint32_t logit, int token) {
    return (unsigned long long)beam << 56 | (unsigned long long)~logit << 24 | (unsigned)token;
}

__global__ void __launch_bounds__(kThreads) beam_merge_kernel(const SelectArgs a) {
    constexpr int kList = kMostKeep + kRound * kThreads;
    __shared__ double base[kMostBeams];  // scores_i - log sum exp, NaN: nothing to choose from
    __shared__ float near[kMostBeams];   // the same rounded
    __shared__ bool over[kMostBeams];
    __shared__ unsigned long long lkey[kList], lat[kList];
    __shared__ int count, masked[kRound][kWarps];
    // the best so far, in order
    __shared__ unsigned long long rkey[kMostKeep], rat[kMostKeep];
    const long long b = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = warp; i < a.beams; i += kWarps) {
        const long long row = b * a.beams + i;
        const float score = a.scores[row];
        double v = isfinite(score) ? score : NAN;
        if (!(a.finished && a.finished[row])) {
            float m = -INFINITY;
            const float2* s = a.sums + row * a.slices;
            for (int k = lane; k < a.slices; k += 32) m = fmaxf(m, s[k].x);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            Pair t{0.f, 0.f};
            for (int k = lane; k < a.slices; k += 32) {
                const float2 at = s[k];
                // a slice of nothing but -inf has a sum of 0 or NaN
                t = t.plus(at.x == -INFINITY ? Pair{at.y, 0.f} : exp_minus(m - at.x).times(Pair{at.y, 0.f}));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                t = t.plus(Pair{__shfl_xor_sync(0xffffffffu, t.hi, o), __shfl_xor_sync(0xffffffffu, t.lo, o)});
            const Pair l = log_of(t).plus(m);
            v = isfinite(m) && isfinite(t.hi) ? v - ((double)l.hi + l.lo) : NAN;
        }
        if (lane == 0) {
            base[i] = v;
            near[i] = (float)v;
            over[i] = a.finished && a.finished[row];
        }
    }
    int have = 0;  // of the best so far
    const int per = a.slices * a.keep, all = a.beams * per;
    const int* tokens = a.best_token + b * all;
    const float* logits = a.best + b * all;
    __syncthreads();
    // the largest of the beams' sums
    float most = 0.f;
    for (int i = lane; i < a.beams; i += 32) most = fmaxf(most, fabsf(near[i]));
    most = __uint_as_float(warp_max(__float_as_uint(most)));
    // what a candidate's float32 score must reach so that its score proper can reach one whose float32 score
    // is `bound`: both are off by 2^-24 of themselves and of the beam's sum at most (FLT_MAX stands for +inf)
    const auto reach = [&](float bound) {
        const float t = fminf(bound, FLT_MAX);
        return t - (fabsf(t) * 0x1p-22f + most * 0x1p-22f + FLT_MIN);
    };
    for (int c0 = 0; c0 < all; c0 += kRound * kThreads) {
        int ct[kRound];
        float x[kRound], score[kRound];
#pragma unroll
        for (int u = 0; u < kRound; ++u) {
            const int c = c0 + u * kThreads + tid;
            ct[u] = c < all ? tokens[c] : -1;
            x[u] = c < all ? logits[c] : 0.f;
        }
        // with a full list, what cannot come before its last entry is out, and so is all at -inf: it comes
        // in the order of its places
        const float floor = have == a.keep ? reach((float)unordered(rkey[a.keep - 1])) : -INFINITY;
        uint32_t best = 0u;  // of what is above -inf
        bool any = false;
#pragma unroll
        for (int u = 0; u < kRound; ++u) {
            const int c = c0 + u * kThreads + tid;
            score[u] = -INFINITY;
            if (c < all) {
                const int i = c / per, k = c - i * per;
                const float from = near[i];
                const bool choice = from == from;
                if (over[i] || !choice) {
                    // the first tokens, at -inf; an ended beam's padding token at its score
                    ct[u] = k < a.keep && k < a.vocab ? k : -1;
                    x[u] = -INFINITY;
                    if (over[i] && choice) {
                        if (k == a.keep - 1 && a.pad >= a.keep) ct[u] = a.pad;
                        if (ct[u] == a.pad) x[u] = 0.f;
                    }
                }
                if (x[u] != -INFINITY) score[u] = from + x[u];
                if (have == a.keep && (x[u] == -INFINITY || score[u] < floor)) ct[u] = -1;
                if (ct[u] >= 0) any = true;
                if (ct[u] >= 0 && x[u] != -INFINITY) best = max(best, ordered(score[u]));
            }
        }
        if (tid == 0) count = have;
        if (tid < have) lkey[tid] = rkey[tid], lat[tid] = rat[tid];
        if (!__syncthreads_or(any)) continue;
        // the keep-th best of the threads' own best, bit by bit: at least `keep` candidates reach it (beams
        // differ too much for a bound by warps)
        uint32_t bound = 0u;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t t = bound | 1u << bit;
            const int n = __syncthreads_count(best >= t);
            if (n >= a.keep) bound = t;
            if (n == a.keep) break;
        }
        const float low = bound ? reach(unordered(bound)) : -INFINITY;
#pragma unroll
        for (int u = 0; u < kRound; ++u)
            if (ct[u] >= 0 && x[u] != -INFINITY && score[u] >= low) {
                const int i = (c0 + u * kThreads + tid) / per, to = atomicAdd(&count, 1);
                lkey[to] = ordered(base[i] + x[u]);
                lat[to] = place(i, ordered(x[u]), ct[u]);
            }
        if (!bound && have < a.keep) {  // maybe fewer than are kept: the first at -inf too
            unsigned those[kRound];
#pragma unroll
            for (int u = 0; u < kRound; ++u) {
                those[u] = __ballot_sync(0xffffffffu, ct[u] >= 0 && x[u] == -INFINITY);
                if (lane == 0) masked[u][warp] = __popc(those[u]);
            }
            __syncthreads();
            int before = 0;
#pragma unroll
            for (int u = 0; u < kRound; ++u) {
                int r = before + __popc(those[u] & ((1u << lane) - 1));
                for (int w = 0; w < kWarps; ++w) {
                    r += w < warp ? masked[u][w] : 0;
                    before += masked[u][w];
                }
                if (those[u] >> lane & 1 && r < a.keep) {
                    const int to = atomicAdd(&count, 1);
                    lkey[to] = ordered((double)-INFINITY);
                    lat[to] = place((c0 + u * kThreads + tid) / per, 0u, ct[u]);
                }
            }
        }
        __syncthreads();
        rank_all(lkey, lat, count, a.keep, [&](int rank, int i) { rkey[rank] = lkey[i], rat[rank] = lat[i]; });
        have = min(count, a.keep);
        __syncthreads();
    }
    if (tid < have) {
        const unsigned long long at = rat[tid];
        const long long out = b * a.keep + tid;
        a.out_scores[out] = (float)unordered(rkey[tid]);
        a.parents[out] = (int)(at >> 56);
        a.tokens[out] = (int)(at & 0xffffffu);
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
        else if ((off & 1) == 0)
            copy_piece<uint16_t>(to_, from_, bytes);
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
constexpr int kWide = 16, kNarrow = 8;  // elements a thread
struct SelectPlan {
    int e, slices;
    size_t best, token, sums, total;
};
size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
// Eight elements a thread while slices of 16 leave fewer than two blocks for each SM: then a slice's
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
