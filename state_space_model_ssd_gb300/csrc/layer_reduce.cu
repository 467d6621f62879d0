// The status word of the operators around the scan, and the second pass of the weight
// gradients: the blocks of a backward kernel each leave one
// float32 partial sum per weight, and this kernel adds them in a fixed order, so the
// gradients are bit-identical from run to run (no atomics).
//
// A block owns 32 columns; its warps take the partials in turn, eight loads in flight each,
// then the warp sums are added.  Bound by the latency of the loads; the bytes (nb * nk * C *
// 4) come from L2, where the kernel before left them.  The launch itself overlaps the end of
// that kernel; griddepcontrol.wait holds the loads back until it has finished.
#include <atomic>

#include "layer_device.cuh"
#include "layer_host.cuh"

namespace ssd {
namespace layer {

namespace {

template <int W>
__global__ void __launch_bounds__(32 * W)
    partial_sum_kernel(const float* partial, int nb, int nk, long long C, ReduceDst d, int bf16) {
    __shared__ float part[W][32];
    const long long M = C * nk;
    const long long m = (long long)blockIdx.x * 32 + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s = 0.f;
    if (m < M) {
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int y = threadIdx.y; y < nb; y += 8 * W)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (y + i * W < nb) t[i] += partial[(y + i * W) * M + m];
        s = ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
    }
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y != 0 || m >= M) return;
#pragma unroll
    for (int i = 1; i < W; ++i) s += part[i][threadIdx.x];
    int k = 0;
    long long c = m;
    while (c >= C) c -= C, ++k;
    if (d.dst[k]) set_param(d.dst[k], c * d.step[k], s, bf16);
}

template <int W>
cudaError_t launch(const float* partial, int nb, int nk, long long C, const ReduceDst& d, int bf16,
                   cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((C * nk + 31) / 32));
    cfg.blockDim = dim3(32, W);
    cfg.stream = stream;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, partial_sum_kernel<W>, partial, nb, nk, C, d, bf16);
}

__device__ int g_status;

}  // namespace

int* status_word() {
    static std::atomic<int*> word[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    int* p = word[dev].load();
    if (!p) {
        void* q = nullptr;
        if (cudaGetSymbolAddress(&q, g_status) != cudaSuccess) return nullptr;
        p = static_cast<int*>(q);
        word[dev].store(p);
    }
    return p;
}

cudaError_t launch_partial_sum(const float* partial, int nb, int nk, long long C,
                               const ReduceDst& d, int wdtype, Launch& L) {
    const int bf16 = wdtype == SSD_DTYPE_BF16;
    L.begin("partial_sum");
    // few partials take few warps, so that a thread has its eight loads to make
    cudaError_t e = nb <= 64    ? launch<8>(partial, nb, nk, C, d, bf16, L.stream)
                    : nb <= 256 ? launch<16>(partial, nb, nk, C, d, bf16, L.stream)
                                : launch<32>(partial, nb, nk, C, d, bf16, L.stream);
    const cudaError_t last = L.end();
    return e != cudaSuccess ? e : last;
}

}  // namespace layer
}  // namespace ssd

using namespace ssd;

extern "C" ssd_status_t ssd_layer_status(void* stream, int32_t* device_status) {
    if (!device_status) return SSD_ERR_INVALID_ARG;
    int* word = layer::status_word();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int v = 0;
    if (!word || cudaMemcpyAsync(&v, word, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaMemsetAsync(word, 0, sizeof(int), s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return SSD_ERR_CUDA;
    *device_status = v;
    return SSD_OK;
}
