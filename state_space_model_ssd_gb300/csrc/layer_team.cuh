// Rows of a norm are worked on by teams: `nw` warps that hold one row in registers, thread
// by thread VEC neighbouring columns NV times over.  A block holds one team, or several
// one-warp teams.
#pragma once

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

// Threads of a block at most: rows in single elements take up to 1024, rows in vectors 512,
// which leaves a thread the registers that its vectors need.
constexpr int team_threads(int vec) { return vec == 1 ? 1024 : 512; }

// How a row of `dim` columns is laid over threads.
struct RowPlan {
    int vec;    // elements of a vector (1: rows or pointers not aligned for more)
    int nv;     // vectors a thread holds: at most 8, and at most 32 elements
    int nw;     // warps in a team
    int teams;  // teams in a block
};
// Longest rows: 16384 columns in vectors, 8192 in single elements.
inline bool plan_row(int dim, int vec, RowPlan* p) {
    p->vec = vec;
    const int nvec = (dim + vec - 1) / vec;
    const int most = vec == 8 ? 4 : 8;
    // single elements: several per thread before the team grows, for loads in flight
    const int first = vec == 1 ? 256 : 512;
    p->nv = 1;
    while (p->nv < most && (nvec + p->nv - 1) / p->nv > first) p->nv <<= 1;
    const int threads = ((nvec + p->nv - 1) / p->nv + 31) / 32 * 32;
    if (threads > team_threads(vec)) return false;
    p->nw = threads / 32;
    p->teams = p->nw == 1 ? 4 : 1;
    return true;
}

}  // namespace layer
}  // namespace ssd
