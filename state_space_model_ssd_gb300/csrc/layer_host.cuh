// Host-side helpers of the operators around the scan: argument checks and launch counting.
#pragma once

#include <stdint.h>

#include "ssd_internal.cuh"

namespace ssd {

// The count ssd_last_launch_count() reports for this host thread.
void set_last_launches(int n);

namespace layer {

inline bool dtype_ok(int d) { return d == SSD_DTYPE_F32 || d == SSD_DTYPE_BF16; }
inline size_t dtype_size(int d) { return d == SSD_DTYPE_BF16 ? 2 : 4; }
inline bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Where the kernels of the operators around the scan record a wait that ran out, on the current
// device (nullptr: no such device).
int* status_word();

// A tensor as the address range it spans: `rows` rows of `width` elements, `stride`
// elements apart.
struct Span {
    uintptr_t lo, hi;
    Span(const void* p, long long rows, long long stride, long long width, size_t e)
        : lo((uintptr_t)p),
          hi(p && rows > 0 ? lo + (size_t)((rows - 1) * stride + width) * e : lo) {}
    bool overlaps(const Span& o) const { return lo < o.hi && o.lo < hi; }
};

// Sums per-block partials on `stream`: out value (k, c) = sum over y < nb of
// partial[y][k][c], for nk <= 9 rows k of C columns; row k goes to dst[k], element
// c * step[k] (NULL: dropped), in float32 or bfloat16.
struct ReduceDst {
    void* dst[9];
    int step[9];
};
cudaError_t launch_partial_sum(const float* partial, int nb, int nk, long long C,
                               const ReduceDst& d, int wdtype, Launch& L);

}  // namespace layer
}  // namespace ssd
