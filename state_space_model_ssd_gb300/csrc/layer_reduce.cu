// The second pass of the weight gradients: the blocks of a backward kernel each leave one
// float32 partial sum per weight, and this kernel adds them in a fixed order, so the
// gradients are bit-identical from run to run (no atomics).
//
// A block owns 32 columns; its 32 warps take the partials in turn, then one warp adds the
// 32 warp sums.  Bound by the latency of the loads (each warp nb / 32 of them, four in
// flight); the bytes (nb * nk * C * 4) come from L2, where the kernel before left them.
#include "layer_device.cuh"
#include "layer_host.cuh"

namespace ssd {
namespace layer {

namespace {

constexpr int kSumWarps = 32;

__global__ void __launch_bounds__(32 * kSumWarps)
    partial_sum_kernel(const float* __restrict__ partial, int nb, int nk, long long C, ReduceDst d,
                       int bf16) {
    __shared__ float part[kSumWarps][33];
    const long long M = C * nk;
    const long long m = (long long)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (m < M) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
        int y = threadIdx.y;
        for (; y + 3 * kSumWarps < nb; y += 4 * kSumWarps)
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] += partial[(y + i * kSumWarps) * M + m];
        for (; y < nb; y += kSumWarps) t[0] += partial[y * M + m];
        s = (t[0] + t[1]) + (t[2] + t[3]);
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || m >= M) return;
    for (int i = 1; i < kSumWarps; ++i) s += part[i][threadIdx.x];
    const int k = (int)(m / C);
    if (d.dst[k]) set_param(d.dst[k], (m - k * C) * d.step[k], s, bf16);
}

}  // namespace

cudaError_t launch_partial_sum(const float* partial, int nb, int nk, long long C,
                               const ReduceDst& d, int wdtype, Launch& L) {
    L.begin("partial_sum");
    partial_sum_kernel<<<(unsigned)((C * nk + 31) / 32), dim3(32, kSumWarps), 0, L.stream>>>(
        partial, nb, nk, C, d, wdtype == SSD_DTYPE_BF16);
    return L.end();
}

}  // namespace layer
}  // namespace ssd
