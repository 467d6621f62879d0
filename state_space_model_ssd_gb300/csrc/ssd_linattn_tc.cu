// Linear attention on the tensor cores: the walk of linattn.cuh in chunks of 128 tokens, one tile of
// 64 columns of v at a time, and the sums over segments.
//
// A chunk takes four products, all with float32 accumulators in TMEM:
//     A   = q k^T                     128 x 128, over the kd channels
//     O1  = (A masked by a^(i-j)) v   128 x 64: the mask's product is rounded to bf16, or split into
//                                     two bf16 terms, and is the operand that stays in TMEM
//     O2  = q S                       128 x 64, S rounded to bf16 in shared memory
//     U   = k^T W                     kd x 64, W the rows of v times a^(n-1-j)
//     out = si O1 + sx a^(i+1) O2,    S <- a^n S + U
// The state goes from chunk to chunk in registers, in float32.  W must not be rounded to bf16: the
// states are float32 outputs.  So W is split into three bf16 terms, W = W1 + W2 + W3 to 2^-25 (two,
// to 2^-18, in calls that return no state, whose outputs are all rounded to 2^-9), which stand
// side by side as one operand: the products k W1 and k W2 come out beside one another (k W3 is added
// to the second) and are added in float32.  A power a^(i-j) is never split into a^i a^-j over more than 16
// tokens below the diagonal, so that nothing overflows.
//
// One block an SM: sixteen warps that all go through the same steps of a chunk (mask, state, the next
// chunk's weights, outputs), each on its 32 rows and a quarter of the columns; a warp for the items and the
// copies in (TMA, two to four chunks ahead), one for the copies out, and two that issue products: A and
// O1 in one, O2 and U in the other.  While the sixteen are at one step, the products of the steps before
// run.  Two things decide the pace.  Instructions: with a task for each four warps (mask, outputs, state,
// weights side by side) every stream goes straight through some hundred instructions a chunk and the
// caches hold 79 % of them, against 95 % where sixteen warps follow one another (32768 tokens of 80
// heads forward 400 us, so 345).  And the stack: beside the tiles nothing is left of L1 for it, see Item.
// Blocks stay and take items in turn, or, where items are long and of unequal cost, there is a block
// for each item, the dearest first.  The tiles of all passes of one segment and head are next to one
// another, so that what they all read comes from L2 after the first.
//
// GB300, 32768 tokens of 80 heads, 64 x 128 states: forward 338 us for the walk (88 % of the copy rate on its
// bytes), 167 for the sums, 17 for the scan; backward, five tiles for each head's chunk, 1337 us:
// 3700 cycles for a tile's chunk with 55 % of the issue slots and a third of the tensor pipe in use, no
// step of it more than 9 % by itself.
#include <algorithm>
#include <utility>

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
constexpr int kWalkThreads = 20 * 32;
constexpr int kSumThreads = 18 * 32;
constexpr int kTeam = 16;                    // warps that work on the numbers
constexpr int kMostStages = 4;
constexpr uint64_t kLimitNs = 2000000000ull;

struct Maps {
    CUtensorMap m[3][4];  // of each pass: q, k, v, and out where it is bf16
};
struct Geometry {
    int stages, v_stages;   // chunks of q and k, and of v, in shared memory at a time
    int kblocks;            // most blocks of 64 channels of q and k
    int stage_bytes, v_at, w_at, s_at, aux_at;
    int items, by_pass;
};

// What a block works on at a time: one segment, head and tile.  It is kept in shared memory, as nothing
// that is read often may be on the stack: beside 227 KB of shared memory there is no L1 to hold it (a
// few spilled registers, at 9 % hits, cost a third of the walk's time).
struct Item {
    Seg g;
    const Pass* p;
    long long id;
    int pass, h, v0, chunks, kb, rev, f32, short_one;  // short_one: the chunk that may be short
    float ld, ld2, si, sx, su;
    Decay whole, last;  // over a whole chunk, and over the short one
    char* out;          // the tile's columns of the segment's first token
    long long os;       // bytes from one token of out to the next
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
    const Pass& p = *t->p;
    const float ld = a.ld[t->h];
    t->ld = ld, t->ld2 = ld * 1.44269504f;
    t->kb = p.kd / 64, t->rev = p.reverse, t->f32 = p.out_f32, t->si = p.si, t->sx = p.sx, t->su = p.su;
    t->short_one = p.reverse ? 0 : t->chunks - 1;
    t->whole = Decay(ld, kQ), t->last = Decay(ld, (t->g.len - 1) % kQ + 1);
    t->os = p.os * (p.out_f32 ? 4 : 2);
    t->out = static_cast<char*>(p.out) + t->g.start * t->os +
             ((long long)(t->h / p.outr) * p.vd + t->v0) * (p.out_f32 ? 4 : 2);
}
// Barriers and what else is small, behind the tiles.
constexpr int kBelow = 32;  // zeros before a^0
struct Aux {
    uint64_t full[kMostStages], empty[kMostStages], full_v[kMostStages], empty_v[kMostStages], weights[kMostStages],
        outputs[kMostStages];
    uint64_t scores, masked, outs, outs_free, sums, item_full[2], item_empty[2];
    uint32_t tmem;
    int stop;
    // the item the block works on and the next, and the powers of their heads by column minus row, in
    // the order of the columns: a^127 .. a^0 and kBelow zeros, or, in a walk from the end, the zeros and
    // a^0 .. a^127; made by the warp that copies in
    Item items[2];
    alignas(16) float powers[2][kBelow + kQ];
};
struct SumsAux {
    uint64_t full[kMostStages], empty[kMostStages], made[2], used[2], sums[2], sums_free[2];
    uint32_t tmem;
    int stop;
    Item items[kSumThreads / 32];  // of each warp
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

// A look at a barrier ahead of its wait: the answer comes while other work goes on.
__device__ __forceinline__ bool peek(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool wait_peeked(bool seen, uint64_t* bar, uint32_t parity, volatile int* stop, int* status) {
    return __all_sync(0xffffffffu, seen) || __all_sync(0xffffffffu, wait_long(bar, parity, stop, status));
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

// Pieces first .. first + pieces of 8 columns of row `row` of a 128 x 64 tile of v, times w, into NT
// tiles kSub apart: each term is what the ones before it left, rounded to bf16.  A token behind the
// sequence's end is a zero row.
template <int NT>
__device__ __forceinline__ void split_row(const unsigned char* v, unsigned char* w_out, int row, int first, int pieces,
                                          float w, bool in) {
    const uint32_t base = row * 128, x = row & 7;
    const F2 ww = layer::both<F2>(w);
#pragma unroll 2
    for (int c = first; c < first + pieces; ++c) {
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

// Columns [col, col + 8) of U: the large term and, kV columns on, the small ones, added.
__device__ __forceinline__ void load_sum8(uint32_t taddr, F2* f) {
    uint32_t r[2][8];
    tmem_ld8(taddr, r[0]);
    tmem_ld8(taddr + kV, r[1]);
    tmem_wait_ld();
    reg_dep8(r[0]), reg_dep8(r[1]);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = layer::add_(pair(r[1][2 * i], r[1][2 * i + 1]), pair(r[0][2 * i], r[0][2 * i + 1]));
}

// Steps of 16 of a product move both operands' descriptors by a constant.
__device__ __forceinline__ uint64_t moved(uint64_t desc, int bytes) { return desc + (uint64_t)(bytes >> 4); }

// k^T W over the chunk's 128 tokens: `k` and `w` shared-memory addresses.  64 channels of k fill the
// 128 lanes twice.  The first two terms go side by side, the third onto the second.
template <int NT>
__device__ __forceinline__ void mma_sums(uint32_t d, uint32_t k, uint32_t w, int kblocks, uint32_t acc) {
    const uint64_t kd = sw128_desc(k, kblocks == 2 ? kSub : 0, 1024), wd = sw128_desc(w, kSub, 1024);
#pragma unroll
    for (int i = 0; i < kQ / 16; ++i)
        mma_bf16(d, moved(kd, i * 2048), moved(wd, i * 2048), idesc_bf16(128, 2 * kV, 1, 1), acc | (i > 0));
    if constexpr (NT == 3) {
#pragma unroll
        for (int i = 0; i < kQ / 16; ++i)
            mma_bf16(d + kV, moved(kd, i * 2048), moved(wd, 2 * kSub + i * 2048), idesc_bf16(128, kV, 1, 1), 1u);
    }
}

// An item's chunks, from registers (what `take` filled in is in memory, and read again after every
// barrier).  They lie from the segment's start on, so that a walk from the end begins with the short
// one.
struct Chunks {
    long long start;
    int len, chunks;
    bool rev;
    __device__ __forceinline__ explicit Chunks(const Item& t)
        : start(t.g.start), len(t.g.len), chunks(t.chunks), rev(t.p->reverse) {}
    // the first token of the walk's c-th chunk, in the segment
    __device__ __forceinline__ int first(int c) const { return (rev ? chunks - 1 - c : c) * kQ; }
};

// A place in a ring of barriers and the parity of its phase.
struct Place {
    int s = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int places) {
        if (++s == places) s = 0, phase ^= 1u;
    }
};

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
// Columns of TMEM: the scores, the masked operand, the two parts of the outputs (that from the state
// in two places, so that chunk k's need not wait for the last outputs to be read), the sums.  A masked
// operand of two terms lies over the scores: in place of 16 of them eight columns of each.
struct C {
    static constexpr uint32_t scores = 0, masked = 128, o1 = 192, u = 384;
    static constexpr uint32_t o2(int k) { return 256 + (k & 1) * kV; }
};

// NT, MT: terms of the weighted rows of v and of the masked scores.
template <int NT, int MT>
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
        for (int s = 0; s < geo.stages; ++s) {
            mbar_init(&x->full[s], 1), mbar_init(&x->empty[s], 2);
        }
        for (int s = 0; s < geo.v_stages; ++s) {
            mbar_init(&x->full_v[s], 1), mbar_init(&x->empty_v[s], 1);
            mbar_init(&x->weights[s], kTeam), mbar_init(&x->outputs[s], kTeam);
        }
        mbar_init(&x->scores, 1), mbar_init(&x->sums, 1), mbar_init(&x->outs, 1);
        for (int s = 0; s < 2; ++s) mbar_init(&x->item_full[s], 1), mbar_init(&x->item_empty[s], kTeam + 3);
        mbar_init(&x->masked, kTeam), mbar_init(&x->outs_free, kTeam);
        x->stop = 0;
        fence_mbar_init();
    }
    if (warp == 16) tmem_alloc(&x->tmem, 512);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x->tmem;
    int g = 0;         // chunks of this block so far
    Place qk, vv, it;  // where the chunk's q and k, its v, and the item are
    Place done_v;      // where the v of the chunk is whose outputs are next
    const auto give_back = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(&x->item_empty[it.s]);
        it.next(2);
    };

    if (warp < kTeam) {
        // ------------------------------------------------ the team: row i, a quarter of the columns
        const uint32_t mine = tmem + lane_base;
        const int i = tid, quad = warp & 3, part = warp >> 2;
        const uint32_t cols = mine + 16 * part;   // a quarter of 64 columns
        unsigned char* w_tile = sm + geo.w_at;
        unsigned char* s_tile = sm + geo.s_at;
        // the scores' groups of 16 columns that are this warp's: one from either end, so that none has
        // two below the diagonal while another has none
        const int j0 = 16 * part, j1 = 16 * (7 - part);
        const auto arrive = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x, give_back()) {
            if (!wait_warp(&x->item_full[it.s], it.phase, &x->stop, status)) break;
            const Item& t = x->items[it.s];
            if (a.cu) {
                const int oe = t.f32 ? 4 : 2;
                const Outside none(a);
                for (long long r = t.id; r < none.n; r += a.ids)
                    if (i < oe)
                        *reinterpret_cast<uint4*>(t.out + (none.token(r) - t.g.start) * t.os + 16 * part * oe + i * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
            }
            if (!t.g.there) continue;
            const bool state_row = i < t.p->kd;  // 64 channels leave half of the lanes out; whole warps
            // this thread's part of the state of sequence or segment `row`, columns t.p->sp apart
            const auto state_at = [&](long long row) {
                return ((row * a.H + t.h) * t.p->kd) * t.p->vd + (t.v0 + 16 * part) * t.p->sp + i * t.p->sn;
            };
            F2 S[8];
            {
                const float* in = t.p->s_seg  ? t.p->s_seg + state_at(t.id)
                                  : t.p->s_in ? t.p->s_in + state_at(t.g.seq)
                                              : nullptr;
                const long long sp = t.p->sp;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    S[e] = in && state_row ? layer::join(in[2 * e * sp], in[(2 * e + 1) * sp]) : layer::join(0.f, 0.f);
            }
            const int rev = t.rev, chunks = t.chunks;
            const bool some0 = rev ? j0 + 15 >= 32 * quad : j0 <= 32 * quad + 31;
            const bool some1 = rev ? j1 + 15 >= 32 * quad : j1 <= 32 * quad + 31;
            // of a group off the diagonal: the row's power to its nearer column
            const float r0 = power(t.ld2, max(rev ? j0 - i : i - j0 - 15, 0));
            const float r1 = power(t.ld2, max(rev ? j1 - i : i - j1 - 15, 0));
            const float fx_whole = power(t.ld2, rev ? kQ - 1 - i : i + 1) * t.sx;
            const float w_whole = power(t.ld2, rev ? i + 1 : kQ - 1 - i) * t.su;

            const int short_one = t.short_one, short_n = t.g.len - (chunks - 1) * kQ;
            bool seen = false;  // what the last look at the barrier of the next wait said
#pragma unroll 1
            for (int c = -1; c < chunks; ++c) {
                const int k = g + c;  // of all the block's chunks
                const int n = c == short_one ? short_n : kQ;
                if (c >= 0) {
                    // ---- mask
                    if (!wait_peeked(seen, &x->scores, k & 1, &x->stop, status)) goto done;
                    tc_fence_after();
                    // times a^distance, or 0 on the other side of the diagonal
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int j = u ? j1 : j0;
                        uint32_t s[16], low[8];
                        const auto put = [&](int e, F2 f) {
                            s[e] = pack(f);
                            if constexpr (MT == 2) low[e] = pack(layer::sub_(f, layer::join(bf_lo(s[e]), bf_hi(s[e]))));
                        };
                        if (u ? some1 : some0) {
                            tmem_ld16(mine + C::scores + j, s);
                            tmem_wait_ld_regs<16>(s);
                            if (n < kQ) {  // tokens of other sequences, an infinity or a NaN maybe
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if (j + e >= n) s[e] = 0u;
                            }
                            if (j >> 5 == quad) {  // at the diagonal: the table from the row's place on
                                const float* at = x->powers[it.s] + (rev ? kBelow : kQ - 1) - i + j;
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    put(e, layer::mul_(pair(s[2 * e], s[2 * e + 1]), layer::join(at[2 * e], at[2 * e + 1])));
                            } else {  // a^15 .. a^0, or from the end a^0 .. a^15, the same for all rows
                                const float4* at = reinterpret_cast<const float4*>(x->powers[it.s] + (rev ? kBelow : kQ - 16));
                                const F2 r = layer::both<F2>(u ? r1 : r0);
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float4 f = at[e];
                                    put(2 * e, layer::mul_(pair(s[4 * e], s[4 * e + 1]), layer::mul_(r, layer::join(f.x, f.y))));
                                    put(2 * e + 1, layer::mul_(pair(s[4 * e + 2], s[4 * e + 3]), layer::mul_(r, layer::join(f.z, f.w))));
                                }
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e) s[e] = low[e] = 0u;
                        }
                        if constexpr (MT == 2) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) s[8 + e] = low[e];
                            tmem_st16(mine + C::scores + j, s);
                        } else {
                            tmem_st8(mine + C::masked + j / 2, s);
                        }
                    }
                    seen = peek(&x->sums, k & 1);
                    tmem_wait_st();
                    tc_fence_before();
                    arrive(&x->masked);
                    // ---- state
                    if (!wait_peeked(seen, &x->sums, k & 1, &x->stop, status)) goto done;
                    tc_fence_after();
                    seen = peek(&x->full_v[vv.s], vv.phase);
                    {
                        const Decay& d = c == short_one ? t.last : t.whole;
                        const F2 m = layer::both<F2>(d.m), keep = layer::both<F2>(d.keep);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            F2 add[4];
                            load_sum8(cols + C::u + 8 * h, add);
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                S[4 * h + e] = layer::fma_(m, S[4 * h + e], layer::fma_(keep, S[4 * h + e], add[e]));
                        }
                    }
                    tc_fence_before();
                }
                if (c + 1 < chunks) {
                    // ---- for the next chunk: the weights and S as bf16 (at an item's start its loads arrive
                    // meanwhile); q S and the sums before, which came with one another, have read the last ones
                    const int m = c + 1 == short_one ? short_n : kQ;
                    unsigned char* v = sm + geo.v_at + vv.s * kSub;
                    if (!wait_peeked(c >= 0 && seen, &x->full_v[vv.s], vv.phase, &x->stop, status)) goto done;
                    const bool in = i < m;
                    const float w = m == kQ || rev ? w_whole : power(t.ld2, max(m - 1 - i, 0)) * t.su;
                    split_row<NT>(v, w_tile, i, 2 * part, 2, w, in);
                    if (state_row) {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<uint4*>(s_tile + i * 128 + (((2 * part + e) ^ (i & 7)) << 4)) =
                                make_uint4(pack(S[4 * e]), pack(S[4 * e + 1]), pack(S[4 * e + 2]), pack(S[4 * e + 3]));
                    }
                    seen = c >= 0 && peek(&x->outs, k & 1);
                    if (m < kQ) {  // rows of other sequences meet zeros, which an infinity or a NaN would outlive
                        if (!wait_warp(&x->full[qk.s], qk.phase, &x->stop, status)) goto done;
                        if (!in && part <= t.kb) zero_row(part ? sm + qk.s * geo.stage_bytes + kbytes + (part - 1) * kSub : v, i);
                    }
                    fence_proxy_async();
                    arrive(&x->weights[vv.s]);
                    qk.next(geo.stages), vv.next(geo.v_stages);
                }
                if (c >= 0) {
                    // ---- outputs
                    const F2 fx = layer::both<F2>(n == kQ || !rev ? fx_whole : power(t.ld2, max(n - 1 - i, 0)) * t.sx);
                    if (!wait_peeked(c + 1 < chunks && seen, &x->outs, k & 1, &x->stop, status)) goto done;
                    tc_fence_after();
                    uint32_t o1[16], o2[16];
                    tmem_ld16(cols + C::o1, o1);
                    tmem_ld16(cols + C::o2(k), o2);
                    tmem_wait_ld_regs<16>(o1);
                    reg_dep16(o2);
                    tc_fence_before();
                    arrive(&x->outs_free);
                    seen = peek(&x->scores, (k + 1) & 1);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const F2 v = layer::fma_(fx, pair(o2[2 * e], o2[2 * e + 1]),
                                                 layer::mul_(layer::both<F2>(t.si), pair(o1[2 * e], o1[2 * e + 1])));
                        float f[2];
                        layer::split(v, f);
                        o1[2 * e] = __float_as_uint(f[0]), o1[2 * e + 1] = __float_as_uint(f[1]);
                        o2[e] = pack(v);
                    }
                    if (n == kQ && !t.f32) {
                        // over the chunk's v, which all its products have read
                        unsigned char* tile = sm + geo.v_at + done_v.s * kSub + i * 128;
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<uint4*>(tile + (((2 * part + e) ^ (i & 7)) << 4)) =
                                make_uint4(o2[4 * e], o2[4 * e + 1], o2[4 * e + 2], o2[4 * e + 3]);
                        fence_proxy_async();
                    } else if (i < n) {
                        const int oe = t.f32 ? 4 : 2;
                        char* row = t.out + (long long)((rev ? chunks - 1 - c : c) * kQ + i) * t.os + 16 * part * oe;
                        const bool wide = ((reinterpret_cast<uintptr_t>(t.out) | (uintptr_t)t.os) & 31) == 0;
                        if (t.f32) {
                            store8(row, o1, wide);
                            store8(row + 32, o1 + 8, wide);
                        } else {
                            store8(row, o2, wide);
                        }
                    }
                    arrive(&x->outputs[done_v.s]);
                    done_v.next(geo.v_stages);
                }
            }
            g += chunks;
            if (t.p->s_out && t.g.k == (rev ? 0 : t.g.cnt - 1) && state_row) {
                float* final = t.p->s_out + state_at(t.g.seq);
                const long long sp = t.p->sp;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f[2];
                    layer::split(S[e], f);
                    final[2 * e * sp] = f[0], final[(2 * e + 1) * sp] = f[1];
                }
            }
        }
    } else if (warp == 16) {
        // ------------------------------------------------ items, their powers, and copies in
        int issued = 0;
        for (int item = blockIdx.x, m = 0; item < geo.items; item += gridDim.x, ++m, it.next(2)) {
            if (m >= 2 && !wait_warp(&x->item_empty[it.s], it.phase ^ 1u, &x->stop, status)) break;
            Item& t = x->items[it.s];
            if (lane == 0) take(a, geo.by_pass, item, &t);
            __syncwarp();
            for (int e = lane; e < kBelow + kQ; e += 32) {
                const int d = t.rev ? e - kBelow : kQ - 1 - e;
                x->powers[it.s][e] = d < 0 ? 0.f : power(t.ld2, d);
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&x->item_full[it.s]);
                const Tiles tiles(maps, t);
                const Chunks ch(t);
                for (int c = 0; c < ch.chunks; ++c, ++g, qk.next(geo.stages), vv.next(geo.v_stages)) {
                    const int t0 = (int)ch.start + ch.first(c);
                    // a place's phase of being given back is one behind that of being filled
                    if (g >= geo.stages && !wait(&x->empty[qk.s], qk.phase ^ 1u, &x->stop, status)) break;
                    tiles.load_qk<true>(t0, sm + qk.s * geo.stage_bytes, kbytes, &x->full[qk.s]);
                    ++issued;
                    if (g >= geo.v_stages && !wait(&x->empty_v[vv.s], vv.phase ^ 1u, &x->stop, status)) break;
                    tiles.load_v(t0, sm + geo.v_at + vv.s * kSub, &x->full_v[vv.s]);
                }
            }
            if (__any_sync(0xffffffffu, *(volatile int*)&x->stop)) break;
        }
        // after a wait that ran out: copies on their way must not land in the next block's memory
        if (lane == 0 && *(volatile int*)&x->stop) {
            for (int k = max(0, issued - geo.stages); k < issued; ++k)
                drain(&x->full[k % geo.stages], (k / geo.stages) & 1);
            for (int k = max(0, g - geo.v_stages); k < g; ++k)
                drain(&x->full_v[k % geo.v_stages], (k / geo.v_stages) & 1);
        }
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------ products: scores, and the masked ones with v
        const uint32_t id_a = idesc_bf16(128, 128, 0, 0), id_o = idesc_bf16(128, kV, 0, 1);
        const uint32_t base = same(smem_u32(sm)), tm = same(tmem);
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x, give_back()) {
            if (!wait_warp(&x->item_full[it.s], it.phase, &x->stop, status)) break;
            const Item& t = x->items[it.s];
            const int kb = same(t.kb), chunks = same(t.chunks);
            for (int c = 0; c < chunks; ++c, ++g, qk.next(geo.stages), vv.next(geo.v_stages)) {
                // the scores before have been read: their mask was waited for.  So has the operand over them
                // when its product is done
                if (!wait_warp(&x->full[qk.s], qk.phase, &x->stop, status) ||
                    (MT == 2 && g > 0 && !wait_warp(&x->outs, (g - 1) & 1, &x->stop, status)))
                    goto stopped_a;
                tc_fence_after();
                if (elect_one()) {
                    uint64_t qd = sw128_desc(base + qk.s * geo.stage_bytes, 16, 1024), kd = moved(qd, kbytes);
#pragma unroll 1
                    for (int b = 0; b < kb; ++b, qd = moved(qd, kSub), kd = moved(kd, kSub))
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(tm + C::scores, moved(qd, i * 32), moved(kd, i * 32), id_a, b + i > 0);
                    mma_commit(&x->scores);
                    mma_commit(&x->empty[qk.s]);
                }
                // with the weights v's rows behind the sequence's end are zero
                if (!wait_warp(&x->masked, g & 1, &x->stop, status) ||
                    !wait_warp(&x->weights[vv.s], vv.phase, &x->stop, status) ||
                    (g > 0 && !wait_warp(&x->outs_free, (g - 1) & 1, &x->stop, status)))
                    goto stopped_a;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t vd = sw128_desc(base + geo.v_at + vv.s * kSub, 16, 1024);
#pragma unroll
                    for (int i = 0; i < kQ / 16 * MT; ++i)  // 16 tokens, of two terms the larger ones first
                        mma_bf16_ta(tm + C::o1, tm + (MT == 2 ? C::scores : C::masked) + 8 * i,
                                    moved(vd, i / MT * 2048), id_o, i > 0);
                    mma_commit(&x->outs);
                }
            }
        }
    stopped_a:
        if (*(volatile int*)&x->stop) {  // what was issued must end before the columns are given back
            if (elect_one()) mma_commit(&x->scores);
            for (int k = 0; k < 2; ++k) drain(&x->scores, k);
        }
    } else if (warp == 18) {
        // ------------------------------------------------ products: the sums, and q with the state
        const uint32_t id_o = idesc_bf16(128, kV, 0, 1);
        const uint32_t base = same(smem_u32(sm)), tm = same(tmem);
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x, give_back()) {
            if (!wait_warp(&x->item_full[it.s], it.phase, &x->stop, status)) break;
            const Item& t = x->items[it.s];
            const int kb = same(t.kb), chunks = same(t.chunks);
            for (int c = 0; c < chunks; ++c, ++g, qk.next(geo.stages), vv.next(geo.v_stages)) {
                const int s = qk.s, vs = vv.s;
                // weights come with the state, after the last sums have been read
                if (!wait_warp(&x->full[s], qk.phase, &x->stop, status) ||
                    !wait_warp(&x->weights[vs], vv.phase, &x->stop, status))
                    goto stopped;
                tc_fence_after();
                if (elect_one()) {
                    uint64_t qd = sw128_desc(base + s * geo.stage_bytes, 16, 1024);
                    uint64_t sd = sw128_desc(base + geo.s_at, 16, 1024);
#pragma unroll 1
                    for (int b = 0; b < kb; ++b, qd = moved(qd, kSub), sd = moved(sd, 8192))
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(tm + C::o2(g), moved(qd, i * 32), moved(sd, i * 2048), id_o, b + i > 0);
                    mma_sums<NT>(tm + C::u, base + s * geo.stage_bytes + kbytes, base + geo.w_at, kb, 0u);
                    mma_commit(&x->sums);
                    mma_commit(&x->empty[s]);
                }
            }
        }
    stopped:
        if (*(volatile int*)&x->stop) {
            if (elect_one()) mma_commit(&x->sums);
            for (int k = 0; k < 2; ++k) drain(&x->sums, k);
        }
    } else {
        // ------------------------------------------------ copies out, and v given back
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x, give_back()) {
            if (!wait_warp(&x->item_full[it.s], it.phase, &x->stop, status)) break;
            const Item& t = x->items[it.s];
            const Chunks ch(t);
            const CUtensorMap* map = &maps.m[t.pass][3];
            const int head = t.h / t.p->outr, v0 = t.v0, short_one = t.g.len == kQ * ch.chunks ? -1 : t.short_one;
            const bool bulk = !t.f32;
            for (int c = 0; c < ch.chunks; ++c, vv.next(geo.v_stages)) {
                if (!wait_warp(&x->outputs[vv.s], vv.phase, &x->stop, status)) goto done;
                if (lane == 0) {
                    if (bulk && c != short_one) {
                        tma_store_3d(map, sm + geo.v_at + vv.s * kSub, v0, head, (int)ch.start + ch.first(c));
                        tma_store_commit();
                        tma_store_wait_read<0>();
                    }
                    mbar_arrive(&x->empty_v[vv.s]);
                }
                __syncwarp();
            }
        }
        if (lane == 0) tma_store_wait_all<0>();
        __syncwarp();
    }
done:
    __syncthreads();
    if (warp == 16) {
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- sums over segments
constexpr int kRun = 4;

// U = k^T W over a whole segment, each token weighted by its power to the segment's end (or, in a
// walk from the end, its start): the state after the segment from none before.  The tensor cores
// accumulate kRun chunks, whose sums are added up in registers: over 4096 tokens in one accumulation,
// which does not round to nearest, a slowly decaying state was off by 3e-6.
// Bound by the bytes of k and v.  Where the final states are wanted it takes the last segments too, with
// three terms, and the walk does with two: in shared memory the third leaves a walk over 128 channels
// two places for v, where three keep it going (32768 tokens of 80 heads, 64 x 128: 509 against 338 us).
template <int NT>
__global__ void __launch_bounds__(kSumThreads, 1)
    tc_sums_kernel(const __grid_constant__ WalkArgs a, const __grid_constant__ Maps maps, const Geometry geo) {
    extern __shared__ __align__(1024) unsigned char sm[];
    SumsAux* x = reinterpret_cast<SumsAux*>(sm + geo.aux_at);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = threadIdx.x & 127, part = warp >> 2;
    const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
    const int kbytes = geo.kblocks * kSub;
    int* status = a.status;
    if (threadIdx.x == 0) {
        // a chunk's copies are announced in two steps
        for (int s = 0; s < geo.stages; ++s) mbar_init(&x->full[s], 2), mbar_init(&x->empty[s], 1);
        for (int s = 0; s < 2; ++s) mbar_init(&x->made[s], kTeam), mbar_init(&x->used[s], 1);
        for (int s = 0; s < 2; ++s) mbar_init(&x->sums[s], 1), mbar_init(&x->sums_free[s], kTeam);
        x->stop = 0;
        fence_mbar_init();
    }
    if (warp == 17) tmem_alloc(&x->tmem, 256);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = x->tmem;
    Item& t = x->items[warp];
    int g = 0, m = 0;  // chunks and runs of this block so far
    Place st, w_set;   // of two sets of weights one chunk's are made while the other's are read
    const auto wanted = [](const Item& t) {  // nothing but the final state comes after a walk's last segment
        return t.g.there && (t.p->s_out || t.g.k != (t.rev ? 0 : t.g.cnt - 1));
    };
    const auto next_item = [&](int item) {
        __syncwarp();
        if (lane == 0) take(a, geo.by_pass, item, &t);
        __syncwarp();
        return wanted(t);
    };
    const auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    if (warp < kTeam) {
        // ------------------------------------------------ weights: a row, a quarter of the columns a thread
        // what the run before has left is read one run later, when its products are done; the item that its
        // last run ends has `out` for the whole
        F2 acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = layer::both<F2>(0.f);
        float* out = nullptr;
        int sp = 0;
        bool ends = false, row = false;
        const auto read_run = [&] {
            if (!wait_warp(&x->sums[(m - 1) & 1], ((m - 1) >> 1) & 1, &x->stop, status)) return false;
            tc_fence_after();
            const uint32_t from = tmem + lane_base + ((m - 1) & 1) * 2 * kV + 16 * part;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                F2 u[4];
                load_sum8(from + 8 * h, u);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[4 * h + e] = layer::add_(acc[4 * h + e], u[e]);
            }
            tc_fence_before();
            arrive(&x->sums_free[(m - 1) & 1]);
            if (ends) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f[2];
                    layer::split(acc[e], f);
                    if (row) out[2 * e * sp] = f[0], out[(2 * e + 1) * sp] = f[1];
                    acc[e] = layer::both<F2>(0.f);
                }
                __syncwarp();
            }
            return true;
        };
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            if (!next_item(item)) continue;
            const int chunks = t.chunks;
            if (chunks == 0) {  // an empty sequence; the products' warp passes it over
                float* zero = t.p->s_sum + (t.id * a.H + t.h) * (long long)t.p->kd * t.p->vd + i * t.p->sn +
                              (t.v0 + 16 * part) * t.p->sp;
                if (i < t.p->kd)
#pragma unroll
                    for (int e = 0; e < 16; ++e) zero[e * t.p->sp] = 0.f;
                continue;
            }
#pragma unroll 1
            for (int c = 0; c < chunks; ++c, ++g, st.next(geo.stages), w_set.next(2)) {
                const int at = c * kQ + i;
                unsigned char* v = sm + st.s * geo.stage_bytes + kbytes;
                const bool in = at < t.g.len;
                const float w = in ? power(t.ld2, t.rev ? at + 1 : t.g.len - 1 - at) * t.su : 0.f;
                if (!wait_warp(&x->full[st.s], st.phase, &x->stop, status)) goto done;
                if (g >= 2 && !wait_warp(&x->used[w_set.s], w_set.phase ^ 1u, &x->stop, status)) goto done;
                split_row<NT>(v, sm + geo.w_at + w_set.s * NT * kSub, i, 2 * part, 2, w, in);
                if (!in && part < t.kb) zero_row(v - kbytes + part * kSub, i);
                fence_proxy_async();
                arrive(&x->made[w_set.s]);
                if (c % kRun == 0) {
                    if (m > 0 && !read_run()) goto done;
                    ++m;
                    ends = c + kRun >= chunks;
                    sp = (int)t.p->sp, row = i < t.p->kd;
                    out = t.p->s_sum + (t.id * a.H + t.h) * (long long)t.p->kd * t.p->vd + i * t.p->sn +
                          (t.v0 + 16 * part) * t.p->sp;
                }
            }
        }
        if (m > 0 && !read_run()) goto done;
    } else if (warp == 16) {
        // ------------------------------------------------ copies in
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            if (!next_item(item)) continue;
            if (lane == 0) {
                const Tiles tiles(maps, t);
                const int chunks = t.chunks, t0 = (int)t.g.start;
                for (int c = 0; c < chunks; ++c, ++g, st.next(geo.stages)) {
                    if (g >= geo.stages && !wait(&x->empty[st.s], st.phase ^ 1u, &x->stop, status)) break;
                    unsigned char* to = sm + st.s * geo.stage_bytes;
                    tiles.load_qk<false>(t0 + c * kQ, to, kbytes, &x->full[st.s]);
                    tiles.load_v(t0 + c * kQ, to + kbytes, &x->full[st.s]);
                }
            }
            if (__any_sync(0xffffffffu, *(volatile int*)&x->stop)) break;
        }
        if (lane == 0 && *(volatile int*)&x->stop)
            for (int k = max(0, g - geo.stages); k < g; ++k)
                drain(&x->full[k % geo.stages], (k / geo.stages) & 1);
        __syncwarp();
    } else {
        // ------------------------------------------------ products
        const uint32_t base = same(smem_u32(sm)), tm = same(tmem);
        for (int item = blockIdx.x; item < geo.items; item += gridDim.x) {
            if (!next_item(item)) continue;
            const int kb = same(t.kb), chunks = same(t.chunks);
            for (int c = 0; c < chunks; ++c, st.next(geo.stages), w_set.next(2)) {
                if (c % kRun == 0 && m > 1 && !wait_warp(&x->sums_free[m & 1], ((m >> 1) - 1) & 1, &x->stop, status))
                    goto stopped;
                if (!wait_warp(&x->made[w_set.s], w_set.phase, &x->stop, status)) goto stopped;
                tc_fence_after();
                if (elect_one()) {
                    mma_sums<NT>(tm + (m & 1) * 2 * kV, base + st.s * geo.stage_bytes,
                                 base + geo.w_at + w_set.s * NT * kSub, kb, c % kRun > 0);
                    mma_commit(&x->empty[st.s]);
                    mma_commit(&x->used[w_set.s]);
                    if (c % kRun == kRun - 1 || c + 1 == chunks) mma_commit(&x->sums[m & 1]);
                }
                m += c % kRun == kRun - 1 || c + 1 == chunks;
            }
        }
    stopped:
        if (*(volatile int*)&x->stop) {
            if (elect_one()) mma_commit(&x->sums[0]);
            for (int k = 0; k < 2; ++k) drain(&x->sums[0], k);
        }
    }
done:
    __syncthreads();
    if (warp == 17) {
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
            !make_map(&m->m[i][2], p.v, a.T, a.H / p.vr, p.vd, p.vs) ||
            (!p.out_f32 && !make_map(&m->m[i][3], p.out, a.T, a.H / p.outr, p.vd, p.os)))
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
    for (int i = 1; by_pass && i < a.npass; ++i)
        for (int j = i; j > 0 && a.pass[j].kd > a.pass[j - 1].kd; --j) std::swap(a.pass[j], a.pass[j - 1]);
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
    // Scores of one term are off by a rounding of bf16, which adds to that of the output: 1.4 times its error, as
    // does a state that meets q.  Where no state has come in, or tokens are so few that roundings do not
    // average (14 tokens of 2 heads: 1.5 times), they are two terms: sequences within a chunk, and launches of
    // one block an SM at most, whose time is latencies.  64 x 128 tokens of 32 heads, 64 x 64 states, forward
    // 57.8 us, so 65.8; 2048 tokens of 16 heads 27.2, so 28.9.  Everywhere it would cost 32768 tokens of 80 heads
    // 542 us for 518 forward and 1635 for 1343 backward, and leave 1.4 times, for the states.
    const bool two = (a.cu ? a.T : a.rowlen) <= kQ || geo.items <= sm_count();
    const auto kernel = three ? two ? tc_walk_kernel<3, 2> : tc_walk_kernel<3, 1>
                              : two ? tc_walk_kernel<2, 2> : tc_walk_kernel<2, 1>;
    const cudaError_t e = launch(kernel, a, m, geo, kWalkThreads, smem, L.stream);
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
    geo.stages = std::min(kMostStages, (kMostSmem - w - (int)sizeof(SumsAux)) / geo.stage_bytes);
    geo.w_at = geo.stages * geo.stage_bytes;
    geo.s_at = geo.aux_at = geo.w_at + w;
    const size_t smem = (size_t)geo.aux_at + sizeof(SumsAux);
    L.begin("linattn_tc_sums");
    const cudaError_t e = three ? launch(tc_sums_kernel<3>, a, m, geo, kSumThreads, smem, L.stream)
                                : launch(tc_sums_kernel<2>, a, m, geo, kSumThreads, smem, L.stream);
    const cudaError_t last = L.end();
    return e != cudaSuccess ? e : last;
}

}  // namespace linattn
}  // namespace ssd
