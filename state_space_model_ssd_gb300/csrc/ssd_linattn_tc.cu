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
// One block an SM, four warps for each of four tasks: mask (A to the masked operand), outputs,
// state (U into S) and weights (v to W); one warp for the copies in (TMA, two or three chunks ahead);
// two that issue products, A and O1 in one, U and O2 in the other, so that the chunk's two chains
// (scores, mask, outputs; weights, sums, state) wait for each other only at the outputs.  Blocks
// stay and take items in turn, or, where items are long and of unequal cost, there is a block for
// each item, the dearest first.  The tiles of all passes of one segment and head are next to one
// another, so that what they all read comes from L2 after the first.
#include <algorithm>

#include "layer_device.cuh"
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
constexpr int kWalkThreads = 19 * 32;
constexpr int kSumThreads = 6 * 32;
constexpr int kMostStages = 4;
constexpr uint64_t kLimitNs = 2000000000ull;

struct Maps {
    CUtensorMap m[3][3];  // of each pass: q, k, v
};
struct Geometry {
    int stages, v_stages;   // chunks of q and k, and of v, in shared memory at a time
    int kblocks;            // most blocks of 64 channels of q and k
    int stage_bytes, v_at, w_at, s_at, aux_at;
    int items, by_pass;
};

// Barriers and what else is small, behind the tiles.
struct Aux {
    uint64_t full[kMostStages], empty[kMostStages], full_v[kMostStages], empty_v[kMostStages], weights[kMostStages];
    uint64_t made[2];
    uint64_t scores[2], masked[2], masked_free, state, state_free, outs, outs_free, sums, sums_free;
    uint32_t tmem;
    int stop;
    float diag[4][64];  // for each of the mask's warps: a^0 .. a^31 in the columns' order, zeros before or after
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

// One thread of a warp that is together.  The products' warps go through their loops as warps, on
// values that are the same in all lanes, so that descriptors stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
template <typename T>
__device__ __forceinline__ T same(T v) {
    return __shfl_sync(0xffffffffu, v, 0);
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
// 32 lanes x 8 columns: tmem_ld16 of half the width.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void reg_dep8(uint32_t* r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                 :
                 : "memory");
}
using layer::F2;
__device__ __forceinline__ F2 pair(uint32_t a, uint32_t b) { return layer::join(__uint_as_float(a), __uint_as_float(b)); }
__device__ __forceinline__ uint32_t pack(F2 v) {
    float f[2];
    layer::split(v, f);
    return pack_bf16(f[0], f[1]);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Row `row` of a 128 x 64 tile of v times w into NT tiles kSub apart: each term is what the ones before
// it left, rounded to bf16.  A weight of a token behind the sequence's end is a zero row.
template <int NT>
__device__ __forceinline__ void split_row(const unsigned char* v, unsigned char* w_out, int row, float w, bool in) {
    const uint32_t base = row * 128, x = row & 7;
    const F2 ww = layer::both<F2>(w);
#pragma unroll 2
    for (int c = 0; c < 8; ++c) {
        const uint32_t at = base + ((c ^ x) << 4);
        uint4 raw = *reinterpret_cast<const uint4*>(v + at);
        if (!in) raw = make_uint4(0u, 0u, 0u, 0u);
        const uint32_t words[4] = {raw.x, raw.y, raw.z, raw.w};
        uint32_t t[NT][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            F2 f = layer::mul_(layer::join(bf_lo(words[i]), bf_hi(words[i])), ww);
#pragma unroll
            for (int k = 0; k < NT; ++k) {
                t[k][i] = pack(f);
                if (k + 1 < NT) f = layer::sub_(f, layer::join(bf_lo(t[k][i]), bf_hi(t[k][i])));
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

// Adds the NT terms of columns [col, col + 8) of U, kV columns apart, of this thread's lane.
template <int NT>
__device__ __forceinline__ void load_sum8(uint32_t taddr, F2* f) {
    uint32_t r[NT][8];
#pragma unroll
    for (int k = 0; k < NT; ++k) tmem_ld8(taddr + k * kV, r[k]);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < NT; ++k) reg_dep8(r[k]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[i] = pair(r[NT - 1][2 * i], r[NT - 1][2 * i + 1]);  // the small terms first
#pragma unroll
        for (int k = NT - 2; k >= 0; --k) f[i] = layer::add_(f[i], pair(r[k][2 * i], r[k][2 * i + 1]));
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
__device__ __noinline__ void take(const WalkArgs& a, int by_pass, int item, Item* t) {
    int id, tile, pass = 0;
    if (by_pass) {  // pass by pass, the tiles of one segment and head next to one another
        const int pairs = (int)a.ids * a.H;
        while (pass + 1 < a.npass && item >= pairs * a.pass[pass].tiles) item -= pairs * a.pass[pass++].tiles;
        const int w = a.pass[pass].tiles, pair = item / w;
        tile = item - pair * w;
        id = pair / a.H;
        t->h = pair - id * a.H;
    } else {  // the tiles of all passes of one
        const int row = a.H * a.tiles;
        id = item / row;
        const int rest = item - id * row;
        t->h = rest / a.tiles;
        tile = rest - t->h * a.tiles;
        while (pass + 1 < a.npass && tile >= a.pass[pass].tiles) tile -= a.pass[pass++].tiles;
    }
    t->id = id;
    t->pass = pass;
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
    __device__ __forceinline__ void load_qk(int t0, unsigned char* st, int kbytes, uint64_t* bar) const {
        mbar_expect_tx(bar, (uint32_t)((WITH_Q ? 2 : 1) * kb * kSub));
#pragma unroll 1
        for (int b = 0; b < kb; ++b, st += kSub) {
            tma_load_3d(st + (WITH_Q ? kbytes : 0), k, bar, b * 64, hk, t0);
            if (WITH_Q) tma_load_3d(st, q, bar, b * 64, hq, t0);
        }
    }
    __device__ __forceinline__ void load_v(int t0, unsigned char* at, uint64_t* bar) const {
        mbar_expect_tx(bar, kSub);
        tma_load_3d(at, v, bar, v0, hv, t0);
    }
};

// 8 words of a row in a store of 32 bytes, which fills a whole sector, or in two of 16.
__device__ __forceinline__ void store8(char* at, const uint32_t* w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// ---------------------------------------------------------------- the walk
// TMEM, 512 columns.  With two terms the scores have two places, and the masked operand goes over the
// scores it came from; with three the scores have one, and the operand its own.
template <int NT>
struct Cols {
    static constexpr int kPlaces = NT == 2 ? 2 : 1;
    static constexpr uint32_t scores(int g) { return NT == 2 ? (g & 1) * 128 : 0; }
    static constexpr uint32_t masked(int g) { return NT == 2 ? (g & 1) * 128 : 128; }
    static constexpr uint32_t o1 = NT == 2 ? 256 : 192, o2 = o1 + kV, u = o2 + kV;
    static_assert(u + NT * kV <= 512, "TMEM");
    // the place and parity of chunk g's scores and masks
    static constexpr int at(int g) { return kPlaces == 2 ? g & 1 : 0; }
    static constexpr int parity(int g) { return kPlaces == 2 ? (g >> 1) & 1 : g & 1; }
};

// The mask's task for one chunk: 32 scores of a row at a time.  Those far from the diagonal take the
// row's power at the group's nearer end times the column's from there, so that no power is of a
// negative distance; those at it a table of the powers with zeros beyond it.
template <int NT>
__device__ __forceinline__ void mask_chunk(uint32_t lanes, int g, int n, bool rev, int warp, int lane, float ld2,
                                           const float* diag, const F2* far) {
    const int i = 32 * warp + lane;
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
        const int j0 = 32 * q;
        uint32_t o[16];
        if (rev ? q < warp : q > warp) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0u;
        } else {
            uint32_t s[32];
            tmem_ld16(lanes + Cols<NT>::scores(g) + j0, *reinterpret_cast<uint32_t(*)[16]>(s));
            tmem_ld16(lanes + Cols<NT>::scores(g) + j0 + 16, *reinterpret_cast<uint32_t(*)[16]>(s + 16));
            tmem_wait_ld_regs<32>(s);
            if (j0 + 32 > n) {  // tokens of other sequences, an infinity or a NaN maybe
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (j0 + e >= n) s[e] = 0u;
            }
            if (q == warp) {
                const float* f = diag + 31 - lane;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = pack(layer::mul_(pair(s[2 * e], s[2 * e + 1]), layer::join(f[2 * e], f[2 * e + 1])));
            } else {
                // forwards the power to the half's last column, from the end to its first
                const int d = rev ? j0 - i : i - j0 - 15, step = rev ? 16 : -16;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const F2 r = layer::both<F2>(power(ld2, d + h * step));
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o[8 * h + e] =
                            pack(layer::mul_(pair(s[16 * h + 2 * e], s[16 * h + 2 * e + 1]), layer::mul_(r, far[e])));
                }
            }
        }
        tmem_st8(lanes + Cols<NT>::masked(g) + j0 / 2, o);
        tmem_st8(lanes + Cols<NT>::masked(g) + j0 / 2 + 8, o + 8);
    }
    tmem_wait_st();
}

// The state's task for one item: row n of S, all of the tile's columns, a thread (64 channels leave
// the upper two warps with nothing but their arrivals).
template <int NT>
__device__ __forceinline__ bool state_item(const WalkArgs& a, const Item& t, Aux* x, unsigned char* s_tile,
                                           uint32_t u_cols, int n, int& g, int* status) {
    const Pass& p = *t.p;
    const bool mine = n < p.kd;  // the same for a whole warp
    const long long size = (long long)p.kd * p.vd, from = (long long)t.v0 * p.sp + n * p.sn;
    const long long seq = ((long long)t.g.seq * a.H + t.h) * size;
    F2 S[kV / 2];
    {
        const float* in = p.s_seg ? p.s_seg + (t.id * a.H + t.h) * size : p.s_in ? p.s_in + seq : nullptr;
        const bool some = in && mine;
        in += from;
#pragma unroll
        for (int i = 0; i < kV / 2; ++i)
            S[i] = some ? layer::join(in[2 * i * p.sp], in[(2 * i + 1) * p.sp]) : layer::join(0.f, 0.f);
    }
    const Decay whole = decay_of(t.ld, kQ), part = decay_of(t.ld, (t.g.len - 1) % kQ + 1);
    const int short_one = p.reverse ? 0 : t.chunks - 1;
#pragma unroll 1
    for (int c = 0; c < t.chunks; ++c, ++g) {
        // the last chunk's q S has read the tile
        if (g > 0 && !wait_warp(&x->state_free, (g - 1) & 1, &x->stop, status)) return false;
        if (mine)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                *reinterpret_cast<uint4*>(s_tile + n * 128 + ((i ^ (n & 7)) << 4)) =
                    make_uint4(pack(S[4 * i]), pack(S[4 * i + 1]), pack(S[4 * i + 2]), pack(S[4 * i + 3]));
        fence_proxy_async();
        mbar_arrive(&x->state);
        const Decay d = c == short_one ? part : whole;
        const F2 m = layer::both<F2>(d.m);
        if (!wait_warp(&x->sums, g & 1, &x->stop, status)) return false;
        tc_fence_after();
        if (mine)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                F2 u[4];
                load_sum8<NT>(u_cols + 8 * i, u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (d.keep != 0.f) u[e] = layer::add_(u[e], S[4 * i + e]);
                    S[4 * i + e] = layer::fma_(m, S[4 * i + e], u[e]);
                }
            }
        tc_fence_before();
        mbar_arrive(&x->sums_free);
    }
    if (mine && p.s_out && t.g.k == (p.reverse ? 0 : t.g.cnt - 1)) {
        float* out = p.s_out + seq + from;
#pragma unroll
        for (int i = 0; i < kV / 2; ++i) {
            float f[2];
            layer::split(S[i], f);
            out[2 * i * p.sp] = f[0], out[(2 * i + 1) * p.sp] = f[1];
        }
    }
    return true;
}

template <int NT>
__global__ void __launch_bounds__(kWalkThreads, 1)
    tc_walk_kernel(const __grid_constant__ WalkArgs a, const __grid_constant__ Maps maps, const Geometry geo) {
    using C = Cols<NT>;
    extern __shared__ __align__(1024) unsigned char sm[];
    Aux* x = reinterpret_cast<Aux*>(sm + geo.aux_at);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tid = threadIdx.x & 127;                            // within a task's four warps
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;  // the warp's lanes of TMEM
    const int kbytes = geo.kblocks * kSub;
    int* status = a.status;
    if (threadIdx.x == 0) {
        for (int s = 0; s < geo.stages; ++s) {
            mbar_init(&x->full[s], 1), mbar_init(&x->empty[s], 2);
        }
        for (int s = 0; s < geo.v_stages; ++s) {
            mbar_init(&x->full_v[s], 1), mbar_init(&x->empty_v[s], 2), mbar_init(&x->weights[s], 128);
        }
        for (int s = 0; s < 2; ++s) mbar_init(&x->scores[s], 1), mbar_init(&x->masked[s], 128);
        mbar_init(&x->masked_free, 1), mbar_init(&x->state_free, 1), mbar_init(&x->sums, 1);
        mbar_init(&x->outs, 2);
        mbar_init(&x->state, 128), mbar_init(&x->outs_free, 128);
        mbar_init(&x->sums_free, 128);
        x->stop = 0;
        fence_mbar_init();
    }
    if (warp == 16) tmem_alloc(&x->tmem, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x->tmem;
    int g = 0;  // chunks of this block so far

    if (warp < 4) {
        // ------------------------------------------------ mask
        float* diag = x->diag[warp];
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, geo.by_pass, item, &t);
            const bool rev = t.p->reverse;
            const float ld2 = t.ld * 1.44269504f;
            __syncwarp();  // the last item's are no longer read
            // column e of row `lane` is at 31 - lane + e: from the end a^(e - lane), else a^(lane - e)
            diag[rev ? lane : lane + 31] = 0.f;
            __syncwarp();
            diag[rev ? lane + 31 : 31 - lane] = power(ld2, lane);
            __syncwarp();
            F2 far[8];
            const float* first = rev ? diag + 31 : diag + 16;  // a^0 .. a^15, or a^15 .. a^0
#pragma unroll
            for (int e = 0; e < 8; ++e) far[e] = layer::join(first[2 * e], first[2 * e + 1]);
#pragma unroll 1
            for (int c = 0; c < t.chunks; ++c, ++g) {
                int n;
                chunk_start(t, c, &n);
                if (!wait_warp(&x->scores[C::at(g)], C::parity(g), &x->stop, status)) goto done;
                // where the operand has one place: its last reader
                if (C::kPlaces == 1 && g > 0 && !wait_warp(&x->masked_free, (g - 1) & 1, &x->stop, status)) goto done;
                tc_fence_after();
                mask_chunk<NT>(tmem + lane_base, g, n, rev, warp, lane, ld2, diag, far);
                tc_fence_before();
                mbar_arrive(&x->masked[C::at(g)]);
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------ outputs
        const uint32_t mine = tmem + lane_base;
        const int i = tid;
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, geo.by_pass, item, &t);
            const Pass& p = *t.p;
            const bool rev = p.reverse, f32 = p.out_f32;
            char* out = static_cast<char*>(p.out);
            const int oe = f32 ? 4 : 2;
            const long long col = (long long)(t.h / p.outr) * p.vd + t.v0;
            if (a.cu) {  // tokens behind the last sequence
                for (long long r = border(a, a.nseq) + t.id; r < a.T; r += a.ids)
                    if (i < kV * oe / 16)
                        *reinterpret_cast<uint4*>(out + (r * p.os + col) * oe + i * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            if (t.chunks == 0) continue;
            const float ld2 = t.ld * 1.44269504f;
            const F2 fi = layer::both<F2>(p.si);
            const float fx_whole = power(ld2, rev ? kQ - 1 - i : i + 1) * p.sx;
            const bool wide = ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(p.os * oe)) & 31) == 0;
#pragma unroll 1
            for (int c = 0; c < t.chunks; ++c, ++g) {
                int n;
                const long long t0 = chunk_start(t, c, &n);
                const F2 fx = layer::both<F2>(n == kQ || !rev ? fx_whole : power(ld2, max(n - 1 - i, 0)) * p.sx);
                char* row = out + ((t0 + i) * p.os + col) * oe;
                if (!wait_warp(&x->outs, g & 1, &x->stop, status)) goto done;
                tc_fence_after();
#pragma unroll 1
                for (int h = 0; h < 2; ++h, row += 32 * oe) {
                    uint32_t o1[32], o2[32];
#pragma unroll
                    for (int e = 0; e < 32; e += 16) {
                        tmem_ld16(mine + C::o1 + 32 * h + e, *reinterpret_cast<uint32_t(*)[16]>(o1 + e));
                        tmem_ld16(mine + C::o2 + 32 * h + e, *reinterpret_cast<uint32_t(*)[16]>(o2 + e));
                    }
                    tmem_wait_ld_regs<32>(o1);
                    tmem_wait_ld_regs<32>(o2);
                    if (h == 1) {
                        tc_fence_before();
                        mbar_arrive(&x->outs_free);
                    }
                    F2 v[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] = layer::fma_(fx, pair(o2[2 * e], o2[2 * e + 1]), layer::mul_(fi, pair(o1[2 * e], o1[2 * e + 1])));
                    if (i < n) {
                        if (f32) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float f[2];
                                layer::split(v[e], f);
                                o1[2 * e] = __float_as_uint(f[0]), o1[2 * e + 1] = __float_as_uint(f[1]);
                            }
                            store8(row + 64, o1 + 16, wide);
                            store8(row + 96, o1 + 24, wide);
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e) o1[e] = pack(v[e]);
                        }
                        store8(row, o1, wide);
                        store8(row + 32, o1 + 8, wide);
                    }
                }
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------ state
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, geo.by_pass, item, &t);
            if (!t.g.there) continue;
            if (!state_item<NT>(a, t, x, sm + geo.s_at, tmem + lane_base + C::u, tid, g, status)) goto done;
        }
    } else if (warp < 16) {
        // ------------------------------------------------ weights
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, geo.by_pass, item, &t);
            const Pass& p = *t.p;
            const float ld2 = t.ld * 1.44269504f;
            const float whole = power(ld2, p.reverse ? tid + 1 : kQ - 1 - tid) * p.su;
#pragma unroll 1
            for (int c = 0; c < t.chunks; ++c, ++g) {
                int n;
                chunk_start(t, c, &n);
                const int s = g % geo.v_stages;
                unsigned char* v = sm + geo.v_at + s * kSub;
                if (!wait_warp(&x->full_v[s], (g / geo.v_stages) & 1, &x->stop, status)) goto done;
                // the product before has read the last weights
                if (g > 0 && !wait_warp(&x->sums, (g - 1) & 1, &x->stop, status)) goto done;
                const bool in = tid < n;
                const float w = n == kQ || p.reverse ? whole : power(ld2, max(n - 1 - tid, 0)) * p.su;
                split_row<NT>(v, sm + geo.w_at, tid, w, in);
                if (n < kQ) {  // rows of other sequences meet zeros, which an infinity or a NaN would outlive
                    const int k = g % geo.stages;
                    if (!wait_warp(&x->full[k], (g / geo.stages) & 1, &x->stop, status)) goto done;
                    if (!in) {
                        zero_row(v, tid);
                        for (int b = 0; b < p.kd / 64; ++b)
                            zero_row(sm + k * geo.stage_bytes + kbytes + b * kSub, tid);
                    }
                }
                fence_proxy_async();
                mbar_arrive(&x->weights[s]);
            }
        }
    } else if (warp == 16) {
        // ------------------------------------------------ copies in
        if (lane == 0) {
            int issued = 0;
            for (int item = blockIdx.x; item < geo.items && !x->stop; item += gridDim.x) {
                Item t;
                take(a, geo.by_pass, item, &t);
                const Tiles tiles(maps, t);
                for (int c = 0; c < t.chunks; ++c, ++g) {
                    int n;
                    const int t0 = (int)chunk_start(t, c, &n), s = g % geo.stages, vs = g % geo.v_stages;
                    if (g >= geo.stages && !wait(&x->empty[s], (g / geo.stages - 1) & 1, &x->stop, status)) break;
                    tiles.load_qk<true>(t0, sm + s * geo.stage_bytes, kbytes, &x->full[s]);
                    ++issued;
                    if (g >= geo.v_stages && !wait(&x->empty_v[vs], (g / geo.v_stages - 1) & 1, &x->stop, status)) break;
                    tiles.load_v(t0, sm + geo.v_at + vs * kSub, &x->full_v[vs]);
                }
            }
            // after a wait that ran out: copies on their way must not land in the next block's memory
            if (*(volatile int*)&x->stop) {
                for (int k = max(0, issued - geo.stages); k < issued; ++k)
                    drain(&x->full[k % geo.stages], (k / geo.stages) & 1);
                for (int k = max(0, g - geo.v_stages); k < g; ++k)
                    drain(&x->full_v[k % geo.v_stages], (k / geo.v_stages) & 1);
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------ products: scores, and the masked ones with v
        const uint32_t id_a = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, kV, 0, 1);
        const uint32_t base = same(smem_u32(sm)), tm = same(tmem);
        int item = blockIdx.x - gridDim.x, left = 0, kb = 0;
        for (bool more = true; more; ++g) {
            while (left == 0 && more) {
                item += gridDim.x;
                more = item < geo.items;
                if (more) {
                    Item t;
                    take(a, geo.by_pass, item, &t);
                    left = same(t.chunks), kb = same(t.p->kd / 64);
                }
            }
            if (more) {
                const int s = g % geo.stages;
                // with one place for the scores, those before have been read
                if (!wait_warp(&x->full[s], (g / geo.stages) & 1, &x->stop, status) ||
                    (C::kPlaces == 1 && g > 0 && !wait_warp(&x->masked[0], (g - 1) & 1, &x->stop, status)))
                    break;
                tc_fence_after();
                if (elect_one()) {
                    uint64_t qd = sw128_desc(base + s * geo.stage_bytes, 16, 1024), kd = moved(qd, kbytes);
#pragma unroll 1
                    for (int b = 0; b < kb; ++b, qd = moved(qd, kSub), kd = moved(kd, kSub))
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(tm + C::scores(g), moved(qd, i * 32), moved(kd, i * 32), id_a, b + i > 0);
                    mma_commit(&x->scores[C::at(g)]);
                    mma_commit(&x->empty[s]);
                }
                --left;
            }
            if (g > 0) {  // the masked product of the chunk before, whose mask this one's scores went ahead of
                const int k = g - 1, s = k % geo.v_stages;
                // with the weights v's rows behind the sequence's end are zero
                if (!wait_warp(&x->masked[C::at(k)], C::parity(k), &x->stop, status) ||
                    !wait_warp(&x->weights[s], (k / geo.v_stages) & 1, &x->stop, status) ||
                    (k > 0 && !wait_warp(&x->outs_free, (k - 1) & 1, &x->stop, status)))
                    break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t vd = sw128_desc(base + geo.v_at + s * kSub, 16, 1024);
#pragma unroll
                    for (int i = 0; i < kQ / 16; ++i)
                        mma_bf16_ta(tm + C::o1, tm + C::masked(k) + 8 * i, moved(vd, i * 2048), id_o, i > 0);
                    mma_commit(&x->outs);
                    if (C::kPlaces == 1) mma_commit(&x->masked_free);
                    mma_commit(&x->empty_v[s]);
                }
            }
        }
        if (*(volatile int*)&x->stop) {  // what was issued must end before the columns are given back
            if (elect_one()) mma_commit(&x->scores[0]);
            for (int k = 0; k < 2; ++k) drain(&x->scores[0], k);
        }
    } else {
        // ------------------------------------------------ products: the sums, and q with the state
        const uint32_t id_o = idesc_bf16(128, kV, 0, 1);
        const uint32_t base = same(smem_u32(sm)), tm = same(tmem);
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            Item t;
            take(a, geo.by_pass, item, &t);
            const int kb = same(t.p->kd / 64), chunks = same(t.chunks);
            for (int c = 0; c < chunks; ++c, ++g) {
                const int s = g % geo.stages, vs = g % geo.v_stages;
                if (!wait_warp(&x->full[s], (g / geo.stages) & 1, &x->stop, status) ||
                    !wait_warp(&x->weights[vs], (g / geo.v_stages) & 1, &x->stop, status) ||
                    (g > 0 && !wait_warp(&x->sums_free, (g - 1) & 1, &x->stop, status)))
                    goto stopped;
                tc_fence_after();
                if (elect_one()) {
                    mma_sums<NT>(tm + C::u, base + s * geo.stage_bytes + kbytes, base + geo.w_at, kb, 0u);
                    mma_commit(&x->sums);
                    mma_commit(&x->empty_v[vs]);
                }
                if (!wait_warp(&x->state, g & 1, &x->stop, status) ||
                    (g > 0 && !wait_warp(&x->outs_free, (g - 1) & 1, &x->stop, status)))
                    goto stopped;
                tc_fence_after();
                if (elect_one()) {
                    uint64_t qd = sw128_desc(base + s * geo.stage_bytes, 16, 1024);
                    uint64_t sd = sw128_desc(base + geo.s_at, 16, 1024);
#pragma unroll 1
                    for (int b = 0; b < kb; ++b, qd = moved(qd, kSub), sd = moved(sd, 8192))
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(tm + C::o2, moved(qd, i * 32), moved(sd, i * 2048), id_o, b + i > 0);
                    mma_commit(&x->state_free);
                    mma_commit(&x->outs);
                    mma_commit(&x->empty[s]);
                }
            }
        }
    stopped:
        if (*(volatile int*)&x->stop) {
            if (elect_one()) mma_commit(&x->sums);
            for (int k = 0; k < 2; ++k) drain(&x->sums, k);
        }
    }
done:
    __syncthreads();
    if (warp == 16) {
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
        // a chunk's copies are announced in two steps
        for (int s = 0; s < geo.stages; ++s) mbar_init(&x->full[s], 2), mbar_init(&x->empty[s], 1);
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
            take(a, geo.by_pass, item, &t);
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
                for (int i = 0; i < kV; i += 8) {
                    F2 u[4];
                    load_sum8<NT>(tmem + lane_base + i, u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float f[2];
                        layer::split(u[e], f);
                        out[(i + 2 * e) * p.sp] = f[0], out[(i + 2 * e + 1) * p.sp] = f[1];
                    }
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
                take(a, geo.by_pass, item, &t);
                if (!wanted(t)) continue;
                const Tiles tiles(maps, t);
                for (int c = 0; c < t.chunks; ++c, ++g) {
                    const int s = g % geo.stages;
                    if (g >= geo.stages && !wait(&x->empty[s], (g / geo.stages - 1) & 1, &x->stop, status)) break;
                    unsigned char* st = sm + s * geo.stage_bytes;
                    tiles.load_qk<false>((int)t.g.start + c * kQ, st, kbytes, &x->full[s]);
                    tiles.load_v((int)t.g.start + c * kQ, st + kbytes, &x->full[s]);
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
                take(a, geo.by_pass, item, &t);
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
    const unsigned grid = (unsigned)(geo.by_pass ? geo.items : std::min(geo.items, sm_count()));
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

cudaError_t tc_walk(const WalkArgs& given, Launch& L) {
    WalkArgs a = given;
    // whole sequences: a block for each item, those with the larger states first
    const bool by_pass = !a.Ls && !a.cu && a.rowlen >= 16 * kQ;
    if (by_pass)
        std::stable_sort(a.pass, a.pass + a.npass, [](const Pass& x, const Pass& y) { return x.kd > y.kd; });
    Maps m;
    if (!make_maps(a, &m)) return cudaErrorInvalidValue;
    const bool three = exact_states(a);
    Geometry geo;
    geo.by_pass = by_pass;
    geo.kblocks = kblocks_of(a);
    geo.items = (int)(a.ids * a.H * a.tiles);  // the caller has seen to it that these fit
    geo.stage_bytes = 2 * geo.kblocks * kSub;
    const int w = (three ? 3 : 2) * kSub, state = geo.kblocks * 64 * 128;
    const auto total = [&](int stages, int v_stages) {
        return stages * geo.stage_bytes + v_stages * kSub + w + state + (int)sizeof(Aux);
    };
    geo.stages = geo.v_stages = 2;
    // v is given back last, and gets its place first
    while (geo.v_stages < kMostStages && total(geo.stages, geo.v_stages + 1) <= kMostSmem) {
        ++geo.v_stages;
        if (geo.stages < geo.v_stages && total(geo.stages + 1, geo.v_stages) <= kMostSmem) ++geo.stages;
    }
    geo.v_at = geo.stages * geo.stage_bytes;
    geo.w_at = geo.v_at + geo.v_stages * kSub;
    geo.s_at = geo.w_at + w;
    geo.aux_at = geo.s_at + state;
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
    geo.by_pass = 0;
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
