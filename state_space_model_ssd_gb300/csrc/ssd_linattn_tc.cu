// Linear attention on the tensor cores: the walk of linattn.cuh in chunks of 128 tokens, one tile of
// 64 columns of v at a time, and the sums over segments.
//
// A chunk takes four products, all with float32 accumulators in TMEM:
//     A   = q k^T                     128 x 128, over the kd channels
//     O1  = (A masked by a^(i-j)) v   128 x 64: the mask's product is rounded to bf16 and is the
//                                     operand that stays in TMEM
//     O2  = q S                       128 x 64, S rounded to bf16 in shared memory
//     U   = k^T W                     kd x 64, W the rows of v times a^(n-1-j)
//     out = si O1 + sx a^(i+1) O2,    S <- a^n S + U
// The state goes from chunk to chunk in registers, in float32.  W must not be rounded to bf16: the
// states are float32 outputs.  So W is split into three bf16 terms, W = W1 + W2 + W3 to 2^-25 (two,
// to 2^-18, in calls that return no state, whose outputs are all rounded to 2^-9), which stand
// side by side as one operand of 192 columns: the products k W1, k W2, k W3 come out beside one
// another and are added in float32.  A power a^(i-j) is never split into a^i a^-j over more than 16
// tokens below the diagonal, so that nothing overflows.
//
// One block an SM with warps for each task: scores (A to the masked operand, and the outputs), state
// (U into S), weights (v to W), one for the copies in (TMA, two or three chunks ahead), one for the
// products.  Blocks stay and take items in turn; the tiles of all passes of one segment and head are
// next to one another, so that what they all read comes from L2 after the first.
#include <algorithm>

#include "linattn.cuh"
#include "tc_common.cuh"

namespace ssd {
namespace linattn {

namespace {

using namespace tc;
using tcc::pack_bf16;

constexpr int kQ = kTcChunk;                 // 128 tokens
constexpr int kV = kTcTile;                  // 64 columns
constexpr int kSub = kQ * 128;               // bytes of a tile of 64 channels: rows of 128 bytes
constexpr int kWalkThreads = 14 * 32;
constexpr int kSumThreads = 6 * 32;
constexpr int kMostStages = 4;
constexpr uint64_t kLimitNs = 2000000000ull;

struct Maps {
    CUtensorMap m[3][3];  // of each pass: q, k, v
};
struct Geometry {
    int stages, kblocks;    // chunks in shared memory at a time; most blocks of 64 channels of q and k
    int stage_bytes, w_at, s_at, aux_at;
    int items;
};

// Barriers and what else is small, behind the tiles.
struct Aux {
    uint64_t full[kMostStages], empty[kMostStages], made[2];
    uint64_t scores, masked, weights, weights_free, state, outs, outs_free, sums, sums_free;
    uint32_t tmem;
    int stop;
    float pw[4][kQ];  // a^0 .. a^127, a copy for each of the scores' warps
};

// Waits for a phase, at most kLimitNs: one that runs out records SSD_ERR_TIMEOUT and ends every wait
// of the block, so that a lost arrival is a status and wrong values, not a hang.  What is seldom gone
// through stays out of line here and below: the tasks' loops have to fit the instruction cache
// together (with everything inlined, 145 KB of code, a chunk took 1.7 times as long).
__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t parity, volatile int* stop, int* status) {
    const uint64_t t0 = globaltimer_ns();
    while (!*stop) {
        if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
        if (globaltimer_ns() - t0 > kLimitNs) {
            *stop = 1;
            atomicCAS(status, 0, (int)SSD_ERR_TIMEOUT);
        }
    }
    return false;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* stop, int* status) {
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, stop, status);
}
// After a wait that ran out: what is on its way must end before the block does.
__device__ __noinline__ void drain(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 20000) && globaltimer_ns() - t0 < kLimitNs) {
    }
}
// wait() for a whole warp, whose lanes go on or stop together.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* stop, int* status) {
    return __all_sync(0xffffffffu, wait(bar, parity, stop, status));
}

// D[tmem] (+)= A[tmem] B[smem]: A's rows in the lanes, two bf16 of a row in each column.
__device__ __forceinline__ void mma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Row `row` of a 128 x 64 tile of v times w into NT tiles kSub apart: each term is what the ones before
// it left, rounded to bf16.  A weight of a token behind the sequence's end is a zero row.
template <int NT>
__device__ __forceinline__ void split_row(const unsigned char* v, unsigned char* w_out, int row, float w, bool in) {
    const uint32_t base = row * 128, x = row & 7;
#pragma unroll 1
    for (int c = 0; c < 8; ++c) {
        const uint32_t at = base + ((c ^ x) << 4);
        const uint4 raw = *reinterpret_cast<const uint4*>(v + at);
        const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
        uint32_t t[NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo = in ? bf_lo(words[i]) * w : 0.f, hi = in ? bf_hi(words[i]) * w : 0.f;
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                t[k][i] = pack_bf16(lo, hi);
                if (k + 1 < NT) lo -= bf_lo(t[k][i]), hi -= bf_hi(t[k][i]);
            }
        }
#pragma unroll
        for (int k = 0; k < NT; ++k)
            *reinterpret_cast<uint4*>(w_out + k * kSub + at) = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
    }
}
__device__ __forceinline__ void zero_row(unsigned char* tile, int row) {
#pragma unroll
    for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(tile + row * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
}

// Adds the NT terms of columns [col, col + 16) of U, kV columns apart, of this thread's lane.
template <int NT>
__device__ __forceinline__ void load_sum16(uint32_t taddr, float* f) {
    uint32_t r[NT][16];
#pragma unroll
    for (int k = 0; k < NT; ++k) tmem_ld16(taddr + k * kV, r[k]);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < NT; ++k) reg_dep16(r[k]);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float s = __uint_as_float(r[NT - 1][i]);  // the small terms first
#pragma unroll
        for (int k = NT - 2; k >= 0; --k) s += __uint_as_float(r[k][i]);
        f[i] = s;
    }
}

// Steps of 16 of a product move both operands' descriptors by a constant.
__device__ __forceinline__ uint64_t moved(uint64_t desc, int bytes) { return desc + (uint64_t)(bytes >> 4); }

// k^T W over the chunk's 128 tokens: `k` and `w` shared-memory addresses.  64 channels of k fill the
// 128 lanes twice.
template <int NT>
__device__ __forceinline__ void mma_sums(uint32_t d, uint32_t k, uint32_t w, int kblocks, uint32_t acc) {
    const uint32_t id = idesc_bf16(128, NT * kV, 1, 1);
    const uint64_t kd = sw128_desc(k, kblocks == 2 ? kSub : 0, 1024), wd = sw128_desc(w, kSub, 1024);
#pragma unroll
    for (int i = 0; i < kQ / 16; ++i) mma_bf16(d, moved(kd, i * 2048), moved(wd, i * 2048), id, acc | (i > 0));
}

struct Item {
    Seg g;
    const Pass* p;
    long long id;
    int pass, h, v0, chunks;
    float ld;
};
__device__ __noinline__ void take(const WalkArgs& a, int item, Item* t) {
    const int row = a.H * a.tiles;
    const int id = item / row, rest = item - id * row;
    t->id = id;
    t->h = rest / a.tiles;
    int tile = rest - t->h * a.tiles;
    t->pass = 0;
    while (t->pass + 1 < a.npass && tile >= a.pass[t->pass].tiles) tile -= a.pass[t->pass++].tiles;
    t->p = &a.pass[t->pass];
    t->v0 = tile * kV;
    t->g = segment(a, t->id);
    t->chunks = t->g.there ? (t->g.len + kQ - 1) / kQ : 0;
    t->ld = a.ld[t->h];
}
__device__ __noinline__ Decay decay_of(float ld, int n) { return Decay(ld, n); }
// First token and tokens of the walk's c-th chunk: chunks lie from the segment's start on, so that a walk
// from the end begins with the short one.
__device__ __forceinline__ long long chunk_start(const Item& t, int c, int* n) {
    const int at = (t.p->reverse ? t.chunks - 1 - c : c) * kQ;
    *n = min(kQ, t.g.len - at);
    return t.g.start + at;
}

// One chunk's tiles; a thread that issues copies keeps an item's maps and heads at hand.
struct Tiles {
    const CUtensorMap *q, *k, *v;
    int hq, hk, hv, v0, kb;
    __device__ __forceinline__ Tiles(const Maps& maps, const Item& t)
        : q(&maps.m[t.pass][0]), k(&maps.m[t.pass][1]), v(&maps.m[t.pass][2]), hq(t.h / t.p->qr),
          hk(t.h / t.p->kr), hv(t.h / t.p->vr), v0(t.v0), kb(t.p->kd / 64) {}
    template <bool WITH_Q>
    __device__ __forceinline__ void load(int t0, unsigned char* st, int kbytes, uint64_t* bar) const {
        mbar_expect_tx(bar, (uint32_t)(((WITH_Q ? 2 : 1) * kb + 1) * kSub));
        tma_load_3d(st + (WITH_Q ? 2 : 1) * kbytes, v, bar, v0, hv, t0);
#pragma unroll 1
        for (int b = 0; b < kb; ++b, st += kSub) {
            tma_load_3d(st + (WITH_Q ? kbytes : 0), k, bar, b * 64, hk, t0);
            if (WITH_Q) tma_load_3d(st, q, bar, b * 64, hq, t0);
        }
    }
};

// `words` (32 or 64) of a row in stores of 32 bytes, which fill whole sectors, or of 16.
__device__ __forceinline__ void store_row(char* row, const uint32_t* w, int words, bool wide) {
#pragma unroll
    for (int i = 0; i < 64; i += 8)
        if (i < words) {
            if (wide) {
                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + 4 * i), "r"(w[i]),
                             "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                             "r"(w[i + 7])
                             : "memory");
            } else {
                reinterpret_cast<uint4*>(row)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
                reinterpret_cast<uint4*>(row)[i / 4 + 1] = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
            }
        }
}

// ---------------------------------------------------------------- the walk
constexpr uint32_t kColScores = 0, kColMasked = 128, kColO1 = 192, kColO2 = 256, kColU = 320;  // 512 columns

// The state's task for one item: row n of S, all of the tile's columns, a thread (64 channels leave
// the upper two warps with nothing but their arrivals).
template <int NT>
__device__ __forceinline__ bool state_item(const WalkArgs& a, const Item& t, Aux* x, unsigned char* s_tile,
                                           uint32_t u_cols, int n, int& g, int* status) {
    const Pass& p = *t.p;
    const bool mine = n < p.kd;  // the same for a whole warp
    const long long size = (long long)p.kd * p.vd, from = (long long)t.v0 * p.sp + n * p.sn;
    const long long seq = ((long long)t.g.seq * a.H + t.h) * size;
    float S[kV];
    {
        const float* in = p.s_seg ? p.s_seg + (t.id * a.H + t.h) * size : p.s_in ? p.s_in + seq : nullptr;
        const bool some = in && mine;
        in += from;
#pragma unroll
        for (int i = 0; i < kV; ++i) S[i] = some ? in[i * p.sp] : 0.f;
    }
    const Decay whole = decay_of(t.ld, kQ), part = decay_of(t.ld, (t.g.len - 1) % kQ + 1);
    const int short_one = p.reverse ? 0 : t.chunks - 1;
#pragma unroll 1
    for (int c = 0; c < t.chunks; ++c, ++g) {
        // the last chunk's q S has read the tile
        if (g > 0 && !wait_warp(&x->outs, (g - 1) & 1, &x->stop, status)) return false;
        if (mine)
#pragma unroll
            for (int i = 0; i < kV; i += 8)
                *reinterpret_cast<uint4*>(s_tile + n * 128 + (((i >> 3) ^ (n & 7)) << 4)) =
                    make_uint4(pack_bf16(S[i], S[i + 1]), pack_bf16(S[i + 2], S[i + 3]),
                               pack_bf16(S[i + 4], S[i + 5]), pack_bf16(S[i + 6], S[i + 7]));
        fence_proxy_async();
        mbar_arrive(&x->state);
        const float m = c == short_one ? part.m : whole.m, keep = c == short_one ? part.keep : whole.keep;
        if (!wait_warp(&x->sums, g & 1, &x->stop, status)) return false;
        tc_fence_after();
        if (mine)
#pragma unroll
            for (int i = 0; i < kV; i += 16) {
                float u[16];
                load_sum16<NT>(u_cols + i, u);
#pragma unroll
                for (int e = 0; e < 16; ++e) S[i + e] = fmaf(m, S[i + e], keep * S[i + e]) + u[e];
            }
        tc_fence_before();
        mbar_arrive(&x->sums_free);
    }
    if (mine && p.s_out && t.g.k == (p.reverse ? 0 : t.g.cnt - 1)) {
        float* out = p.s_out + seq + from;
#pragma unroll
        for (int i = 0; i < kV; ++i) out[i * p.sp] = S[i];
    }
    return true;
}

template <int NT>
__global__ void __launch_bounds__(kWalkThreads, 1)
    tc_walk_kernel(const __grid_constant__ WalkArgs a, const __grid_constant__ Maps maps, const Geometry geo) {
    extern __shared__ __align__(1024) unsigned char sm[];
    Aux* x = reinterpret_cast<Aux*>(sm + geo.aux_at);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tid = threadIdx.x & 127;                            // within a task's four warps
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;  // the warp's lanes of TMEM
    const int kbytes = geo.kblocks * kSub;
    int* status = a.status;
    if (threadIdx.x == 0) {
        for (int s = 0; s < geo.stages; ++s) mbar_init(&x->full[s], 1), mbar_init(&x->empty[s], 1);
        mbar_init(&x->scores, 1), mbar_init(&x->outs, 1), mbar_init(&x->sums, 1);
        mbar_init(&x->weights_free, 1);
        mbar_init(&x->masked, 128), mbar_init(&x->weights, 128), mbar_init(&x->state, 128);
        mbar_init(&x->outs_free, 128), mbar_init(&x->sums_free, 128);
        x->stop = 0;
        fence_mbar_init();
    }
    if (warp == 13) tmem_alloc(&x->tmem, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x->tmem;
    int g = 0;  // chunks of this block so far

    if (warp < 4) {
        // ------------------------------------------------ scores: the masked operand, and the outputs
        const uint32_t mine = tmem + lane_base;
        const int i = tid, w0 = 32 * warp;
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, item, &t);
            const Pass& p = *t.p;
            const bool rev = p.reverse;
            char* out = static_cast<char*>(p.out);
            const int oe = p.out_f32 ? 4 : 2;
            const long long col = (long long)(t.h / p.outr) * p.vd + t.v0;
            if (a.cu) {  // tokens behind the last sequence
                for (long long r = border(a, a.nseq) + t.id; r < a.T; r += a.ids)
                    if (i < kV * oe / 16)
                        *reinterpret_cast<uint4*>(out + (r * p.os + col) * oe + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            if (t.chunks == 0) continue;
            const float ld2 = t.ld * 1.44269504f;
            float* pw = x->pw[warp];
            __syncwarp();  // the last item's are no longer read
            for (int d = lane; d < kQ; d += 32) pw[d] = power(ld2, d);
            __syncwarp();
            float far[16];  // a block's factors by column, beside the row's
#pragma unroll
            for (int e = 0; e < 16; ++e) far[e] = pw[rev ? e : 15 - e];
            const float fi = p.si, fx_whole = power(ld2, rev ? kQ - 1 - i : i + 1) * p.sx;
            const bool wide = ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(p.os * oe)) & 31) == 0;
            for (int c = 0; c < t.chunks; ++c, ++g) {
                int n;
                const long long t0 = chunk_start(t, c, &n);
                if (!wait_warp(&x->scores, g & 1, &x->stop, status)) goto done;
                tc_fence_after();
                // the operand's last reader, the product before, has finished: its outputs were read
#pragma unroll 1
                for (int b = 0; b < kQ / 16; ++b) {
                    const int j0 = 16 * b;
                    uint32_t o[8];
                    if (rev ? j0 + 15 < w0 : j0 > w0 + 31) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = 0u;
                    } else {
                        uint32_t s[16];
                        tmem_ld16(mine + kColScores + j0, s);
                        tmem_wait_ld_regs<16>(s);
                        if (n == kQ && (rev ? j0 >= w0 + 31 : j0 + 15 <= w0)) {
                            const float r = pw[rev ? j0 - i : i - j0 - 15];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = pack_bf16(__uint_as_float(s[2 * e]) * (r * far[2 * e]),
                                                 __uint_as_float(s[2 * e + 1]) * (r * far[2 * e + 1]));
                        } else {
                            // what is masked may be an infinity or a NaN, and is left out, not multiplied
                            float f[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const int d = rev ? j0 + e - i : i - j0 - e;
                                f[e] = d >= 0 && j0 + e < n ? __uint_as_float(s[e]) * pw[d & (kQ - 1)] : 0.f;
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
                        }
                    }
                    tmem_st8(mine + kColMasked + 8 * b, o);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&x->masked);
                if (!wait_warp(&x->outs, g & 1, &x->stop, status)) goto done;
                tc_fence_after();
                const float fx = n == kQ || !rev ? fx_whole : pw[max(n - 1 - i, 0)] * p.sx;
                char* row = out + ((t0 + i) * p.os + col) * oe;
                // both halves are read before the columns are given back, added and stored after
                uint32_t o1[kV], o2[kV];
#pragma unroll
                for (int e = 0; e < kV; e += 16) {
                    tmem_ld16(mine + kColO1 + e, *reinterpret_cast<uint32_t(*)[16]>(o1 + e));
                    tmem_ld16(mine + kColO2 + e, *reinterpret_cast<uint32_t(*)[16]>(o2 + e));
                }
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < kV; e += 16) reg_dep16(o1 + e), reg_dep16(o2 + e);
                tc_fence_before();
                mbar_arrive(&x->outs_free);
#pragma unroll
                for (int e = 0; e < kV; ++e)
                    o1[e] = __float_as_uint(fmaf(fx, __uint_as_float(o2[e]), fi * __uint_as_float(o1[e])));
                if (i < n) {
                    if (!p.out_f32) {
#pragma unroll
                        for (int e = 0; e < kV / 2; ++e)
                            o1[e] = pack_bf16(__uint_as_float(o1[2 * e]), __uint_as_float(o1[2 * e + 1]));
                    }
                    store_row(row, o1, p.out_f32 ? kV : kV / 2, wide);
                }
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------ state
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, item, &t);
            if (!t.g.there) continue;
            if (!state_item<NT>(a, t, x, sm + geo.s_at, tmem + lane_base + kColU, tid, g, status)) goto done;
        }
    } else if (warp < 12) {
        // ------------------------------------------------ weights
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, item, &t);
            const Pass& p = *t.p;
            const float ld2 = t.ld * 1.44269504f;
            const float whole = power(ld2, p.reverse ? tid + 1 : kQ - 1 - tid) * p.su;
            for (int c = 0; c < t.chunks; ++c, ++g) {
                int n;
                chunk_start(t, c, &n);
                const int s = g % geo.stages;
                unsigned char* st = sm + s * geo.stage_bytes;
                if (!wait_warp(&x->full[s], (g / geo.stages) & 1, &x->stop, status)) goto done;
                // the product before has read the last weights
                if (g > 0 && !wait_warp(&x->weights_free, (g - 1) & 1, &x->stop, status)) goto done;
                const bool in = tid < n;
                const float w = n == kQ || p.reverse ? whole : in ? power(ld2, n - 1 - tid) * p.su : 0.f;
                split_row<NT>(st + 2 * kbytes, sm + geo.w_at, tid, w, in);
                if (!in) {  // rows of other sequences meet zeros, which an infinity or a NaN would outlive
                    zero_row(st + 2 * kbytes, tid);
                    for (int b = 0; b < p.kd / 64; ++b) zero_row(st + kbytes + b * kSub, tid);
                }
                fence_proxy_async();
                mbar_arrive(&x->weights);
            }
        }
    } else if (warp == 12) {
        // ------------------------------------------------ copies in
        if (lane == 0) {
            for (int item = blockIdx.x; item < geo.items && !x->stop; item += gridDim.x) {
                Item t;
                take(a, item, &t);
                const Tiles tiles(maps, t);
                for (int c = 0; c < t.chunks; ++c, ++g) {
                    int n;
                    const long long t0 = chunk_start(t, c, &n);
                    const int s = g % geo.stages;
                    if (g >= geo.stages && !wait(&x->empty[s], (g / geo.stages - 1) & 1, &x->stop, status)) break;
                    tiles.load<true>((int)t0, sm + s * geo.stage_bytes, kbytes, &x->full[s]);
                }
            }
            // after a wait that ran out: copies on their way must not land in the next block's memory
            if (*(volatile int*)&x->stop)
                for (int k = max(0, g - geo.stages); k < g; ++k)
                    drain(&x->full[k % geo.stages], (k / geo.stages) & 1);
        }
        __syncwarp();
    } else if (warp == 13) {
        // ------------------------------------------------ products
        if (lane == 0) {
            const uint32_t id_a = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, kV, 0, 1);
            const uint32_t w_tile = smem_u32(sm + geo.w_at);
            const uint64_t s_desc = sw128_desc(smem_u32(sm + geo.s_at), 16, 1024);
            bool stop = false;
            for (int item = blockIdx.x; item < geo.items && !stop; item += gridDim.x) {
                Item t;
                take(a, item, &t);
                const int kb = t.p->kd / 64;
                for (int c = 0; c < t.chunks; ++c, ++g) {
                    const int s = g % geo.stages;
                    const uint32_t q = smem_u32(sm + s * geo.stage_bytes), k = q + kbytes, v = k + kbytes;
                    stop = !wait(&x->full[s], (g / geo.stages) & 1, &x->stop, status);
                    if (stop) break;
                    // the scores before were read before their product, which is behind this one
                    const uint64_t qd = sw128_desc(q, 16, 1024), kd = sw128_desc(k, 16, 1024);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < 4 * kb)
                            mma_bf16(tmem + kColScores, moved(qd, (i >> 2) * kSub + (i & 3) * 32),
                                     moved(kd, (i >> 2) * kSub + (i & 3) * 32), id_a, i > 0);
                    mma_commit(&x->scores);
                    stop = !wait(&x->weights, g & 1, &x->stop, status) ||
                           (g > 0 && !wait(&x->sums_free, (g - 1) & 1, &x->stop, status));
                    if (stop) break;
                    tc_fence_after();
                    mma_sums<NT>(tmem + kColU, k, w_tile, kb, 0u);
                    mma_commit(&x->sums);
                    mma_commit(&x->weights_free);
                    stop = !wait(&x->state, g & 1, &x->stop, status) ||
                           (g > 0 && !wait(&x->outs_free, (g - 1) & 1, &x->stop, status));
                    if (stop) break;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < 4 * kb)
                            mma_bf16(tmem + kColO2, moved(qd, (i >> 2) * kSub + (i & 3) * 32),
                                     moved(s_desc, i * 2048), id_o, i > 0);
                    stop = !wait(&x->masked, g & 1, &x->stop, status);
                    if (stop) break;
                    tc_fence_after();
                    const uint64_t vd = sw128_desc(v, 16, 1024);
#pragma unroll
                    for (int i = 0; i < kQ / 16; ++i)
                        mma_bf16_ta(tmem + kColO1, tmem + kColMasked + 8 * i, moved(vd, i * 2048), id_o, i > 0);
                    mma_commit(&x->outs);
                    mma_commit(&x->empty[s]);
                }
            }
            if (stop) {  // what was issued must end before the columns are given back
                uint64_t* bar = &x->weights_free;
                mma_commit(bar);
                for (int k = 0; k < 2; ++k) drain(bar, k);
            }
        }
        __syncwarp();
    }
done:
    __syncthreads();
    if (warp == 13) {
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- sums over segments
// U = k^T W over a whole segment, each token weighted by its power to the segment's end (or, in a
// walk from the end, its start), in one accumulation: the state after the segment from none before.
// Bound by the bytes of k and v.
template <int NT>
__global__ void __launch_bounds__(kSumThreads, 1)
    tc_sums_kernel(const __grid_constant__ WalkArgs a, const __grid_constant__ Maps maps, const Geometry geo) {
    extern __shared__ __align__(1024) unsigned char sm[];
    Aux* x = reinterpret_cast<Aux*>(sm + geo.aux_at);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const int kbytes = geo.kblocks * kSub;
    int* status = a.status;
    if (threadIdx.x == 0) {
        for (int s = 0; s < geo.stages; ++s) mbar_init(&x->full[s], 1), mbar_init(&x->empty[s], 1);
        for (int s = 0; s < 2; ++s) mbar_init(&x->made[s], 128);
        mbar_init(&x->sums, 1), mbar_init(&x->sums_free, 128);
        x->stop = 0;
        fence_mbar_init();
    }
    if (warp == 5) tmem_alloc(&x->tmem, 256);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x->tmem;
    int g = 0, m = 0;  // chunks and items of this block so far
    const auto wanted = [&](const Item& t) {  // nothing comes after a walk's last segment
        return t.g.there && t.g.k != (t.p->reverse ? 0 : t.g.cnt - 1);
    };
    // two sets of weights: one chunk's are made while the other's are read
    if (warp < 4) {
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, item, &t);
            if (!wanted(t)) continue;
            const Pass& p = *t.p;
            const float ld2 = t.ld * 1.44269504f;
            for (int c = 0; c < t.chunks; ++c, ++g) {
                const int s = g % geo.stages, at = c * kQ + tid;
                unsigned char* st = sm + s * geo.stage_bytes;
                if (!wait_warp(&x->full[s], (g / geo.stages) & 1, &x->stop, status)) goto done;
                // the set's last reader has finished: its stage was given back before
                if (g >= 2 && !wait_warp(&x->empty[(g - 2) % geo.stages], ((g - 2) / geo.stages) & 1, &x->stop, status))
                    goto done;
                const bool in = at < t.g.len;
                const float w = in ? power(ld2, p.reverse ? at + 1 : t.g.len - 1 - at) * p.su : 0.f;
                split_row<NT>(st + kbytes, sm + geo.w_at + (g & 1) * NT * kSub, tid, w, in);
                if (!in)
                    for (int b = 0; b < p.kd / 64; ++b) zero_row(st + b * kSub, tid);
                fence_proxy_async();
                mbar_arrive(&x->made[g & 1]);
            }
            if (!wait_warp(&x->sums, m & 1, &x->stop, status)) goto done;
            tc_fence_after();
            if (tid < p.kd) {
                float* out = p.s_sum + (t.id * a.H + t.h) * (long long)p.kd * p.vd + tid * p.sn + t.v0 * p.sp;
#pragma unroll 1
                for (int i = 0; i < kV; i += 16) {
                    float u[16];
                    load_sum16<NT>(tmem + lane_base + i, u);
#pragma unroll
                    for (int e = 0; e < 16; ++e) out[(i + e) * p.sp] = u[e];
                }
            }
            tc_fence_before();
            mbar_arrive(&x->sums_free);
            ++m;
        }
    } else if (warp == 4) {
        if (lane == 0) {
            for (int item = blockIdx.x; item < geo.items && !x->stop; item += gridDim.x) {
                Item t;
                take(a, item, &t);
                if (!wanted(t)) continue;
                const Tiles tiles(maps, t);
                for (int c = 0; c < t.chunks; ++c, ++g) {
                    const int s = g % geo.stages;
                    if (g >= geo.stages && !wait(&x->empty[s], (g / geo.stages - 1) & 1, &x->stop, status)) break;
                    tiles.load<false>((int)t.g.start + c * kQ, sm + s * geo.stage_bytes, kbytes, &x->full[s]);
                }
            }
            if (*(volatile int*)&x->stop)
                for (int k = max(0, g - geo.stages); k < g; ++k)
                    drain(&x->full[k % geo.stages], (k / geo.stages) & 1);
        }
        __syncwarp();
    } else {
        if (lane == 0) {
            bool stop = false;
            for (int item = blockIdx.x; item < geo.items && !stop; item += gridDim.x) {
                Item t;
                take(a, item, &t);
                if (!wanted(t)) continue;
                if (m > 0 && !wait(&x->sums_free, (m - 1) & 1, &x->stop, status)) break;
                tc_fence_after();
                for (int c = 0; c < t.chunks; ++c, ++g) {
                    const int s = g % geo.stages;
                    stop = !wait(&x->made[g & 1], (g >> 1) & 1, &x->stop, status);
                    if (stop) break;
                    tc_fence_after();
                    mma_sums<NT>(tmem, smem_u32(sm + s * geo.stage_bytes),
                                 smem_u32(sm + geo.w_at + (g & 1) * NT * kSub), t.p->kd / 64, c > 0);
                    mma_commit(&x->empty[s]);
                }
                if (stop) break;
                mma_commit(&x->sums);
                ++m;
            }
            if (*(volatile int*)&x->stop) {
                mma_commit(&x->sums);
                for (int k = 0; k < 2; ++k) drain(&x->sums, k);
            }
        }
        __syncwarp();
    }
done:
    __syncthreads();
    if (warp == 5) {
        tmem_relinquish();
        tmem_dealloc(tmem, 256);
    }
}

// ---------------------------------------------------------------- host
// [T][heads][D] bf16 with tokens `stride` elements apart, tiles of 128 tokens x 64 channels of a head.
bool make_map(CUtensorMap* m, const void* base, long long T, int heads, int D, long long stride) {
    tcc::EncodeTiledFn enc = tcc::encode_fn();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)T};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)kQ};
    cuuint32_t es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_maps(const WalkArgs& a, Maps* m) {
    for (int i = 0; i < a.npass; ++i) {
        const Pass& p = a.pass[i];
        if (!make_map(&m->m[i][0], p.q, a.T, a.H / p.qr, p.kd, p.qs) ||
            !make_map(&m->m[i][1], p.k, a.T, a.H / p.kr, p.kd, p.ks) ||
            !make_map(&m->m[i][2], p.v, a.T, a.H / p.vr, p.vd, p.vs))
            return false;
    }
    return true;
}

constexpr int kMostSmem = 227 * 1024;

template <typename K>
cudaError_t launch(K kernel, const WalkArgs& a, const Maps& m, const Geometry& geo, int threads, size_t smem,
                   cudaStream_t stream) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)std::min<long long>(geo.items, sm_count());
    kernel<<<grid, threads, smem, stream>>>(a, m, geo);
    return cudaSuccess;
}

int kblocks_of(const WalkArgs& a) {
    int kd = 0;
    for (int i = 0; i < a.npass; ++i) kd = std::max(kd, a.pass[i].kd);
    return kd / 64;
}
// Two terms where every output is bf16.
bool exact_states(const WalkArgs& a) {
    for (int i = 0; i < a.npass; ++i)
        if (a.pass[i].s_out) return true;
    return false;
}

}  // namespace

bool tc_fits(const Pass& p) {
    const auto ok = [](const void* q, long long stride, int e) {
        return ((uintptr_t)q & 15) == 0 && stride * e % 16 == 0;
    };
    return (p.kd == 64 || p.kd == 128) && (p.vd == 64 || p.vd == 128) && ok(p.q, p.qs, 2) && ok(p.k, p.ks, 2) &&
           ok(p.v, p.vs, 2) && ok(p.out, p.os, p.out_f32 ? 4 : 2);
}

cudaError_t tc_walk(const WalkArgs& a, Launch& L) {
    Maps m;
    if (!make_maps(a, &m)) return cudaErrorInvalidValue;
    const bool three = exact_states(a);
    Geometry geo;
    geo.kblocks = kblocks_of(a);
    geo.items = (int)(a.ids * a.H * a.tiles);  // the caller has seen to it that these fit
    geo.stage_bytes = (2 * geo.kblocks + 1) * kSub;
    const int rest = (three ? 3 : 2) * kSub + geo.kblocks * 64 * 128 + (int)sizeof(Aux);
    geo.stages = std::min(3, (kMostSmem - rest) / geo.stage_bytes);
    geo.w_at = geo.stages * geo.stage_bytes;
    geo.s_at = geo.w_at + (three ? 3 : 2) * kSub;
    geo.aux_at = geo.s_at + geo.kblocks * 64 * 128;
    const size_t smem = (size_t)geo.aux_at + sizeof(Aux);
    L.begin("linattn_tc_walk");
    const cudaError_t e = three ? launch(tc_walk_kernel<3>, a, m, geo, kWalkThreads, smem, L.stream)
                                : launch(tc_walk_kernel<2>, a, m, geo, kWalkThreads, smem, L.stream);
    const cudaError_t last = L.end();
    return e != cudaSuccess ? e : last;
}

cudaError_t tc_sums(const WalkArgs& a, Launch& L) {
    Maps m;
    if (!make_maps(a, &m)) return cudaErrorInvalidValue;
    const bool three = exact_states(a);
    Geometry geo;
    geo.kblocks = kblocks_of(a);
    geo.items = (int)(a.ids * a.H * a.tiles);  // the caller has seen to it that these fit
    geo.stage_bytes = (geo.kblocks + 1) * kSub;
    const int w = 2 * (three ? 3 : 2) * kSub;
    geo.stages = std::min(kMostStages, (kMostSmem - w - (int)sizeof(Aux)) / geo.stage_bytes);
    geo.w_at = geo.stages * geo.stage_bytes;
    geo.s_at = geo.aux_at = geo.w_at + w;
    const size_t smem = (size_t)geo.aux_at + sizeof(Aux);
    L.begin("linattn_tc_sums");
    const cudaError_t e = three ? launch(tc_sums_kernel<3>, a, m, geo, kSumThreads, smem, L.stream)
                                : launch(tc_sums_kernel<2>, a, m, geo, kSumThreads, smem, L.stream);
    const cudaError_t last = L.end();
    return e != cudaSuccess ? e : last;
}

}  // namespace linattn
}  // namespace ssd
