// Rows of a norm are worked on by teams: `nw` warps that hold one row in registers, thread
// by thread VEC neighbouring columns NV times over.  A block holds one team, or several
// one-warp teams.
#pragma once

#include <atomic>

#include "layer_device.cuh"
#include "layer_host.cuh"

namespace ssd {
namespace layer {

struct Team {
    int nw;      // warps in the team
    int warp;    // this warp in its team
    int lane;
    int thread;  // this thread in its team
    int id;      // the team in its block
};
__device__ __forceinline__ Team team_of(int nw) {
    Team t;
    const int w = threadIdx.x >> 5;
    t.nw = nw;
    t.id = w / nw;
    t.warp = w - t.id * nw;
    t.lane = threadIdx.x & 31;
    t.thread = t.warp * 32 + t.lane;
    return t;
}

// Sums N values over the team, the same bits in every thread.  Every thread of the block
// calls it (one-warp teams need no barrier).  `buf` holds 32 N floats per call in flight;
// two calls in a row take different buffers, and a third comes after the barrier of the
// second, when every thread has read the first.
template <int N>
__device__ __forceinline__ void team_sum(const Team& t, float* v, float* buf) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (t.nw == 1) return;
    if (t.lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) buf[i * 32 + t.warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] = t.lane < t.nw ? buf[i * 32 + t.lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
}

// A row's vectors: 16 bytes of the activations where every row starts on 16 bytes, else 8,
// 4 or one element, whichever divides the row's length, the strides and the addresses.
inline int common_vec(int most, const long long* strides, int ns, const void* const* ptrs,
                      const size_t* sizes, int np) {
    for (int vec = most; vec > 1; vec >>= 1) {
        bool ok = true;
        for (int i = 0; i < ns; ++i) ok = ok && strides[i] % vec == 0;
        for (int i = 0; i < np; ++i)
            ok = ok && aligned_to(ptrs[i], vec * sizes[i] < 16 ? vec * sizes[i] : 16);
        if (ok) return vec;
    }
    return 1;
}

// How a row of `dim` columns is laid over threads.
struct RowPlan {
    int vec;     // elements of a vector
    int nv;      // vectors a thread holds
    int nw;      // warps in a team
    int teams;   // teams in a block
    int per_sm;  // blocks an SM holds at once
    size_t ring; // bytes of the rows in flight
    int threads() const { return nw * teams * 32; }
};
constexpr int team_threads(int vec) { return vec == 1 ? 1024 : 512; }
// (rows of up to 16384 columns in vectors of 16 bytes, 8192 otherwise)
constexpr int most_vectors(int vec, int esize) { return esize == 2 && vec >= 4 ? 4 : 8; }
// Rows in flight.  Four cover the latency of HBM where a thread holds one vector; wider rows
// have enough bytes in flight with two, and the widest do not fit twice.  Rows in single
// elements are loaded to registers one row ahead (0): a copy moves 4 bytes at least.
constexpr int ring_stages(int vec, int nv) {
    return vec == 1 ? 0 : nv == 1 ? 4 : nv * vec <= 16 ? 2 : 1;
}
// `col_bytes`: bytes of a column in all tensors that are read; `regs`: registers of a thread
// that holds e elements of a row are about regs[0] + regs[1] e, 128 at most.  Longest rows:
// 16384 columns in vectors of 16 bytes, 8192 otherwise.
inline bool plan_row(int dim, int vec, int most, int col_bytes, const int (&regs)[2], RowPlan* p) {
    if (dim > (vec == most ? 16384 : 8192)) return false;
    p->vec = vec;
    const int nvec = (dim + vec - 1) / vec;
    if (vec == 1)  // single elements: up to four a thread for loads in flight, then more threads
        p->nv = nvec <= 256 ? 1 : nvec <= 512 ? 2 : nvec <= 4096 ? 4 : 8;
    else
        for (p->nv = 1; (nvec + p->nv - 1) / p->nv > 512;) p->nv <<= 1;
    p->nw = ((nvec + p->nv - 1) / p->nv + 31) / 32;
    if (p->nv > most_vectors(vec, most == 8 ? 2 : 4) || p->nw * 32 > team_threads(vec)) return false;
    p->teams = p->nw == 1 ? 4 : 1;
    p->ring = (size_t)ring_stages(vec, p->nv) * p->threads() * p->nv * vec * col_bytes;
    int r = regs[0] + regs[1] * p->nv * vec;
    if (r > (vec == 1 ? 64 : 128)) r = vec == 1 ? 64 : 128;
    p->per_sm = 65536 / ((r + 7) / 8 * 8) / p->threads();
    const int fit = (int)((size_t)(220 << 10) / (p->ring + 2048));
    if (fit < p->per_sm) p->per_sm = fit;
    if (p->per_sm > 16) p->per_sm = 16;
    if (p->per_sm < 1) p->per_sm = 1;
    return true;
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
