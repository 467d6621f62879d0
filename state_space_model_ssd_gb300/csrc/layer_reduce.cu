// The status word of the operators around the scan, and the second pass of the weight
// gradients: the blocks of a backward kernel each leave one
// float32 partial sum per weight, and this kernel adds them in a fixed order, so the
// gradients are bit-identical from run to run (no atomics).
//
// A block owns 32 vectors of columns (four columns, or one where a row of partials does not
// start on 16 bytes); its warps take the partials in turn, eight loads in flight each, then
// the warp sums are added.  Bound by the latency of the loads; the bytes (nb * nk * C * 4) come
// from L2, where the kernel before left them.  The launch itself overlaps the end of that
// kernel; griddepcontrol.wait holds the loads back until it has finished.
#include <atomic>

#include "layer_device.cuh"
#include "layer_host.cuh"

namespace ssd {
namespace layer {

namespace {

template <int W, int VEC>
__global__ void __launch_bounds__(32 * W)
    partial_sum_kernel(const float* partial, int nb, int nk, long long C, ReduceDst d, int bf16) {
    __shared__ float part[W][VEC][32];
    const long long M = C * nk;
    const long long m = ((long long)blockIdx.x * 32 + threadIdx.x) * VEC;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float s[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = 0.f;
    if (m < M) {
        const float* p = partial + m;
        for (int y = threadIdx.y; y < nb; y += 8 * W) {
            Pack<float, VEC> v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (y + i * W < nb)
                    v[i].load(p + (long long)(y + i * W) * M);
                else
                    v[i].zero();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float f[VEC];
                v[i].get(f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[e] += f[e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[threadIdx.y][e][threadIdx.x] = s[e];
    __syncthreads();
    // warp e adds column e of the vectors
    const int e = threadIdx.y;
    if (e >= VEC || m >= M) return;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) sum += part[i][e][threadIdx.x];
    int k = 0;
    long long c = m + e;
    while (c >= C) c -= C, ++k;
    if (d.dst[k]) set_param(d.dst[k], c * d.step[k], sum, bf16);
}

template <int W, int VEC>
cudaError_t launch(const float* partial, int nb, int nk, long long C, const ReduceDst& d, int bf16,
                   cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((C * nk + 32 * VEC - 1) / (32 * VEC)));
    cfg.blockDim = dim3(32, W);
    cfg.stream = stream;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, partial_sum_kernel<W, VEC>, partial, nb, nk, C, d, bf16);
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
    // few partials take few warps, so that a thread has its eight loads to make; vectors of four
    // once there are columns enough to fill the GPU with them
    const bool wide = C * nk % 4 == 0 && C * nk >= 8192;
    cudaError_t e;
    if (nb <= 64)
        e = wide ? launch<8, 4>(partial, nb, nk, C, d, bf16, L.stream)
                 : launch<8, 1>(partial, nb, nk, C, d, bf16, L.stream);
    else
        e = wide ? launch<16, 4>(partial, nb, nk, C, d, bf16, L.stream)
                 : launch<32, 1>(partial, nb, nk, C, d, bf16, L.stream);
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
