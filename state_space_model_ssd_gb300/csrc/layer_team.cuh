// Rows of a norm are worked on by teams: `nw` warps that hold one row in registers.  A warp
// owns NV * 32 * VEC neighbouring columns, a lane VEC of them NV times over, 32 * VEC apart, so
// that all of a thread's places in a row are offsets known when compiling.  A block holds one
// team, or several teams of a warp or less (8 or 16 lanes, for rows of so few vectors).
#pragma once

#include <atomic>

#include "layer_device.cuh"
#include "layer_host.cuh"

namespace ssd {
namespace layer {

struct Team {
    int nw;      // warps in the team
    int width;   // lanes of a warp in the team
    int warp;    // this warp in its team
    int lane;    // this lane of them
    int rank;    // this thread in its team
    int id;      // the team in its block
};
__device__ __forceinline__ Team team_of(int nw, int width) {
    Team t;
    const int w = threadIdx.x >> 5;
    t.nw = nw;
    t.width = width;
    t.lane = threadIdx.x & (width - 1);
    t.id = width == 32 ? w / nw : threadIdx.x / width;
    t.warp = width == 32 ? w - t.id * nw : 0;
    t.rank = t.warp * 32 + t.lane;
    return t;
}

// Where the warps of a team meet: N floats per warp.  Zeroed once, so that the places of
// warps a team does not have add nothing.
template <int N>
struct TeamBuf {
    float4 v[2][N][8];
    __device__ __forceinline__ void clear() {
        float* f = reinterpret_cast<float*>(v);
        for (int i = threadIdx.x; i < 2 * N * 32; i += blockDim.x) f[i] = 0.f;
        __syncthreads();
    }
    __device__ __forceinline__ float sum4(int flip, int i, int k) const {
        const float4 w = v[flip][i][k];
        return (w.x + w.y) + (w.z + w.w);
    }
};
// Sums N values over the team, the same bits in every thread.  Every thread of the block
// calls it (one-warp teams need no barrier).  Two calls in a row take different halves of the
// buffer (`flip`); a third comes after the barrier of the second, when every thread has read
// the first.
template <int N>
__device__ __forceinline__ void team_sum(const Team& t, float* x, TeamBuf<N>& buf, int flip) {
    if (t.width == 32) {  // the same for the block
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    } else {
        for (int o = t.width >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
    }
    if (t.nw == 1) return;
    if (t.lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<float*>(buf.v[flip][i])[t.warp] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = buf.sum4(flip, i, 0) + buf.sum4(flip, i, 1);
    if (t.nw <= 8) return;  // the same for the block
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] += buf.sum4(flip, i, 2) + buf.sum4(flip, i, 3);
    if (t.nw <= 16) return;
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] += (buf.sum4(flip, i, 4) + buf.sum4(flip, i, 5)) + (buf.sum4(flip, i, 6) + buf.sum4(flip, i, 7));
}

// A row's vectors: `most` elements (16 bytes of the widest tensor) where every row of every
// tensor starts on 16 bytes, else two elements or one, whichever divides the row's length, the
// strides and the addresses.
inline int common_vec(int most, const long long* strides, int ns, const void* const* ptrs,
                      const size_t* sizes, int np) {
    bool wide = true, pairs = true;
    for (int i = 0; i < ns; ++i) pairs = pairs && strides[i] % 2 == 0;
    for (int i = 0; i < np; ++i) {
        const long long n = 16 / (long long)sizes[i];
        for (int k = 0; k < ns; ++k) wide = wide && strides[k] % n == 0;
        wide = wide && aligned_to(ptrs[i], 16);
        pairs = pairs && aligned_to(ptrs[i], 2 * sizes[i]);
    }
    return wide ? most : pairs ? 2 : 1;
}

// How a row of `dim` columns is laid over threads.
struct RowPlan {
    int vec;     // elements of a vector
    int nv;      // vectors a thread holds: 1, 2, 3, 4, 6, 8 or 16
    int nw;      // warps in a team
    int width;   // lanes of a warp in a team
    int teams;   // teams in a block
    int regs;    // registers of a thread
    int per_sm;  // blocks an SM holds at once
    bool bulk;   // rows arrive by bulk copies (or through registers)
    int stages;  // rows in flight then
    size_t ring; // bytes of shared memory they take
    int threads() const { return nw * teams * width; }
};
// Longest rows.
constexpr int most_columns(int vec) { return vec >= 4 ? 16384 : 8192; }
constexpr int most_vectors(int vec) { return vec == 8 ? 4 : vec == 1 ? 16 : 8; }
// Registers of a thread that holds e elements of a row: few, since they decide how many rows an SM
// works on.  They do not hold everything.  A thread stores to local memory (-Xptxas -v) 4 to 64
// bytes in some backwards of up to 16 elements in wide vectors; 48 to 240 in the forwards without a
// residual and the float32 gated one at 32 elements, which rows of 832 columns on may take; 16 to 384
// in backwards of 12 and 16 elements in pairs or single elements (more than 4096 columns); and beyond
// 8192 columns 300 to 1360 in the backwards, 108 to 768 in forwards with a residual.
constexpr int fwd_regs(int vec, int nv) {
    const int e = vec * nv;
    return e <= 2 ? 40 : e <= 4 ? 56 : e <= 8 ? 80 : 128;
}
constexpr int bwd_regs(int vec, int nv, bool bulk) {
    const int e = vec * nv;
    return e <= 2 ? 56 : e <= 4 ? (bulk ? 64 : 80) : e <= 8 ? (bulk ? 96 : 112) : 128;
}
// What a row's plan goes by: the tensors read, na of `ab` bytes an element and nb of `bb`.
struct RowCost {
    bool bwd;
    int na, ab, nb, bb;
};
// Warps of so many registers a thread that an SM holds: each quarter has 16384 registers.
inline int resident_warps(int regs) { return 4 * (16384 / (32 * regs)); }
inline bool plan_row(int dim, int vec, const RowCost& cost, RowPlan* p) {
    if (dim > most_columns(vec)) return false;
    p->vec = vec;
    const int nvec = (dim + vec - 1) / vec;
    // Elements a thread holds, where more threads do as well, in bf16 rows but for the residuals and
    // gradients named.  At 32768 x 2560 (us): a forward
    // without a residual 72 with 16, 65 with 32 (at 32768 x 5120 221 and 114; single elements
    // 130 with 8, 107 with 16); with a bf16 residual 113, 107, 133 with 16, 24, 32; with a float32
    // residual 168, 160, 184 with 12, 16, 24 (single elements 202, 212 with 8, 16); a backward
    // with the residual's gradient 222, 267 with 8, 16 (single elements 309, 273 with 4, 8),
    // without it 134, 109.  Float32 rows take the same counts: a forward without a residual 133
    // (74 % of the copy rate), its row ahead alone 32 registers; fewer were not tried there.
    const int hold = cost.bwd ? (vec <= 2 || cost.nb > 1 ? 8 : 16)
                              : cost.nb == 0 ? (vec == 1 ? 16 : 32) : vec == 1 ? 8 : vec == 8 ? 24 : 16;
    // The constants here and below come from the widths that their figures name; between those they
    // are steps (512 threads leave ten warps an SM at 2560 columns, sixteen at 2048 and 4096).
    // A warp spends about as long on a row's sums and addresses as on fourteen elements a lane,
    // and up to sixteen warps on an SM each add their share of its rate: the plan with the least
    // of that time per row wins.
    double best = -1;
    const int sizes[7] = {1, 2, 3, 4, 6, 8, 16};
    for (int nv : sizes) {
        if (nv > most_vectors(vec) || (nv * vec > hold && best >= 0)) break;
        const int nw = ((nvec + nv - 1) / nv + 31) / 32, teams = nw == 1 ? 4 : 1;
        // A backward's rows come by bulk copies from a full warp on: at 32768 x 5120 312 us
        // against 529 through registers, which its sums need.  A forward has registers to spare
        // (158 against 175 us at 32768 x 2560).
        const bool bulk = cost.bwd && vec >= 4 && nvec > 32;
        const int regs = cost.bwd ? bwd_regs(vec, nv, bulk) : fwd_regs(vec, nv);
        int warps = resident_warps(regs) / (nw * teams) * (nw * teams);
        if (nw > 32 || warps == 0) continue;
        if (warps > 16) warps = 16;
        double c = nw * (14.0 + nv * vec) / warps;
        if (cost.bwd && nv * vec > 8) c *= 1.25;  // as measured: 392 us against 332 in 8 groups of 640
        if (best >= 0 && c >= best) continue;
        best = c;
        p->nv = nv;
        p->nw = nw;
        p->bulk = bulk;
        p->regs = regs;
    }
    if (best < 0) return false;
    p->width = nvec <= 8 ? 8 : nvec <= 16 ? 16 : 32;
    p->teams = p->nw == 1 ? 128 / p->width : 1;
    p->per_sm = resident_warps(p->regs) / (p->threads() / 32);
    if (p->per_sm > 16) p->per_sm = 16;
    // Where a row's arithmetic is little, sixteen warps are enough, and fewer blocks with more
    // rows each on their way do better: 222 us against 242 at 32768 x 2560 with one block of ten
    // warps an SM instead of two.  Not so the gated rows (332 us against 365 in 8 groups of 640).
    if (p->bulk && cost.nb > 0 && p->per_sm * p->threads() > 512) p->per_sm = 512 / p->threads() > 1 ? 512 / p->threads() : 1;
    const size_t bytes = (size_t)dim * (cost.na * cost.ab + cost.nb * cost.bb) * p->teams;
    // More than 48 KB of rows with their residual on their way to an SM get into each other's
    // way: 204 us against 220 at 32768 x 2560 in float32 with two blocks an SM instead of three.
    // Not so the gated rows (182 us against 155 at 32768 x 5120).
    if (!cost.bwd && cost.nb > 0)
        while (p->per_sm > 1 && p->per_sm * bytes > 48 << 10) --p->per_sm;
    p->stages = 0;
    p->ring = 0;
    if (p->bulk) {
        // two to eight rows in flight a team, within what the blocks of an SM can share
        const size_t all = 210 << 10;
        while (p->per_sm > 1 && 2 * bytes + 4096 > all / p->per_sm) --p->per_sm;
        size_t s = (all / p->per_sm - 4096) / bytes;
        p->stages = s > 8 ? 8 : s < 1 ? 1 : (int)s;
        p->ring = p->stages * bytes;
    }
    return true;
}
// The tensors of a team's rows on their way to its threads: by bulk copies into a ring of
// `stages` rows in shared memory, which one thread of the team issues (backwards of a warp and
// more in vectors of 16 bytes), or through registers, DEPTH rows ahead.  The first NA tensors
// have elements of type A, the NB others of type B, read as a stream with STREAM.
constexpr int kMostStages = 8;
struct RowBars {
    uint64_t full[4][kMostStages];  // by team of the block
};
// The rows of a team: first, first + by, ... below `rows` (all below 2^31).
struct RowRange {
    int first, by, rows;
    __device__ __forceinline__ RowRange(long long f, long long b, long long n)
        : first((int)(f < n ? f : n)), by((int)b), rows((int)n) {}
    __device__ __forceinline__ int count() const {
        return first < rows ? (int)(((unsigned)(rows - first) - 1) / (unsigned)by) + 1 : 0;
    }
};
// Where a kernel's rows come from: pointers and strides in the kernel's parameters, so that an
// address costs no register between its uses.
template <typename T>
__device__ __forceinline__ const T* row_at(const void* p, int row, long long stride) {
    return static_cast<const T*>(p) + row * stride;
}
// From(): k -> the start of a row of tensor k.
template <typename A, typename B, int NA, int NB, int VEC, int NV, bool BULK, int DEPTH = 1,
          bool STREAM = false>
struct Rows {
    Pack<A, VEC> ra[DEPTH][BULK ? 1 : NV][NA];
    Pack<B, VEC> rb[DEPTH][BULK ? 1 : NV][NB ? NB : 1];
    int next, by;              // the next row to load
    int left;                  // rows still to load (as wait_copy has it)
    bool in[NV];               // whether vector i lies in the row
    char* ring;                // this team's
    uint64_t* full;
    int cols, stages, fill, stage;
    uint32_t parity;
    int* status;

    static __device__ __forceinline__ int column(const Team& t, int i) {
        return ((t.warp * NV + i) * 32 + t.lane) * VEC;
    }
    // The rows of `r`, of `n` columns.  A barrier of the block has to come between this and
    // start().
    __device__ __forceinline__ void begin(const Team& t, const RowRange& r, int n, int nstages, char* all,
                                          RowBars* bars, int* status_word) {
        next = r.first;
        by = r.by;
        left = BULK && t.rank != 0 ? 0 : r.count();  // one thread issues the copies
        cols = n;
#pragma unroll
        for (int i = 0; i < NV; ++i) in[i] = column(t, i) < n;
        if constexpr (BULK) {
            stages = nstages;
            fill = stage = 0;
            parity = 0;
            status = status_word;
            full = bars->full[t.id];
            ring = all + t.id * stages * row_bytes();
            if (t.rank == 0) {
                for (int s = 0; s < stages; ++s) tc::mbar_init(&full[s], 1);
                tc::fence_mbar_init();
            }
        } else {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
#pragma unroll
                    for (int k = 0; k < NA; ++k) ra[d][i][k].zero();
#pragma unroll
                    for (int k = 0; k < NB; ++k) rb[d][i][k].zero();
                }
        }
    }
    __device__ __forceinline__ uint32_t row_bytes() const {
        return (uint32_t)cols * (NA * (int)sizeof(A) + NB * (int)sizeof(B));
    }
    template <typename FA, typename FB>
    __device__ __forceinline__ void start(const Team& t, const FA& from_a, const FB& from_b) {
        if constexpr (BULK) {
            for (int s = 0; s < stages; ++s) issue(from_a, from_b);
        } else {
            fetch<0>(t, from_a, from_b);
            if constexpr (DEPTH > 1) fetch<1>(t, from_a, from_b);
        }
    }
    template <typename FA, typename FB>
    __device__ __forceinline__ void issue(const FA& from_a, const FB& from_b) {
        if (left > 0) {
            uint64_t* bar = &full[fill];
            char* at = ring + fill * row_bytes();
            tc::mbar_expect_tx(bar, row_bytes());
#pragma unroll
            for (int k = 0; k < NA; ++k)
                tc::bulk_load(at + k * cols * (int)sizeof(A), from_a(k, next), cols * (int)sizeof(A), bar);
            at += NA * cols * (int)sizeof(A);
#pragma unroll
            for (int k = 0; k < NB; ++k)
                tc::bulk_load(at + k * cols * (int)sizeof(B), from_b(k, next), cols * (int)sizeof(B), bar);
            next += by;
            --left;
            fill = fill + 1 == stages ? 0 : fill + 1;
        }
    }
    // S: which of the DEPTH.
    template <int S, typename FA, typename FB>
    __device__ __forceinline__ void fetch(const Team& t, const FA& from_a, const FB& from_b) {
        const bool more = left > 0;
#pragma unroll
        for (int k = 0; k < NA; ++k) {
            const A* p = from_a(k, next) + column(t, 0);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (more && in[i]) ra[S][i][k].load(p + i * 32 * VEC);
        }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            const B* p = from_b(k, next) + column(t, 0);
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (more && in[i]) {
                    if constexpr (STREAM)
                        rb[S][i][k].stream(p + i * 32 * VEC);
                    else
                        rb[S][i][k].load(p + i * 32 * VEC);
                }
        }
        next += by;
        --left;
    }
    // Before the first get of a row that this team has.
    __device__ __forceinline__ void arrived() {
        if constexpr (BULK) wait_copy(&full[stage], parity, status, left);
    }
    // After the last get of a row: registers take the next row.
    template <int S = 0, typename FA, typename FB>
    __device__ __forceinline__ void done(const Team& t, const FA& from_a, const FB& from_b) {
        if constexpr (!BULK) fetch<S>(t, from_a, from_b);
    }
    // Once the whole team has done its gets (a team of one warp waits for itself here): the
    // row's place takes another.
    template <typename FA, typename FB>
    __device__ __forceinline__ void reuse(const Team& t, const FA& from_a, const FB& from_b) {
        if constexpr (BULK) {
            if (t.nw == 1) __syncwarp();
            issue(from_a, from_b);
            if (++stage == stages) stage = 0, parity ^= 1;
        }
    }
    // After the last row, before the block ends or its ring is used for something else.  idle: the
    // team went through the last round without a row (and over a place more than its rows took).
    __device__ __forceinline__ void drain(const Team& t, bool idle) const {
        if constexpr (BULK)
            if (t.rank == 0) drain_ring(full, stages, stage, parity, left, idle);
    }
    // A vector of this thread; zeros where it lies beyond the row, so that sums need no branch.
    template <int S = 0>
    __device__ __forceinline__ void get_a(const Team& t, int i, int k, typename Lanes<VEC>::V* v) const {
        float f[VEC];
        if constexpr (BULK) {
            Pack<A, VEC> p;
            p.zero();
            if (in[i]) p.load(reinterpret_cast<const A*>(ring + stage * row_bytes()) + k * cols + column(t, i));
            p.get(f);
        } else {
            ra[S][i][k].get(f);
        }
        to_lanes<VEC>(f, v);
    }
    template <int S = 0>
    __device__ __forceinline__ void get_b(const Team& t, int i, int k, typename Lanes<VEC>::V* v) const {
        float f[VEC];
        if constexpr (BULK) {
            Pack<B, VEC> p;
            p.zero();
            if (in[i]) p.load(reinterpret_cast<const B*>(ring + stage * row_bytes() + NA * cols * (int)sizeof(A)) +
                   k * cols + column(t, i));
            p.get(f);
        } else {
            rb[S][i][k].get(f);
        }
        to_lanes<VEC>(f, v);
    }
};
__device__ __forceinline__ float lane_sum(F2 v) {
    float f[2];
    split(v, f);
    return f[0] + f[1];
}
__device__ __forceinline__ float lane_sum(float v) { return v; }
template <int VEC, typename T>
__device__ __forceinline__ void store_lanes(T* p, const typename Lanes<VEC>::V* v) {
    float f[VEC];
    from_lanes<VEC>(v, f);
    store_vec<VEC>(p, f);
}

// Blocks that share `rows` rows: as many as the GPU holds at once.
inline int team_blocks(long long rows, const RowPlan& p) {
    const long long most = (long long)sm_count() * p.per_sm;
    const long long want = (rows + p.teams - 1) / p.teams;
    return (int)(want < most ? want : most);
}
// Lets a kernel take more than 48 KB of shared memory (once per kernel and device); a kernel's
// static arrays, up to 8 KB here, count too.
template <auto Kernel>
cudaError_t allow_smem(size_t bytes) {
    if (bytes <= (40 << 10)) return cudaSuccess;
    static std::atomic<unsigned long long> done{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 216 << 10);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}

}  // namespace layer
}  // namespace ssd
