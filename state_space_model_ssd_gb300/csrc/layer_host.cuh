// Host-side helpers of the operators around the scan: argument checks and launch counting.
#pragma once

#include <stdint.h>

#include <initializer_list>

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
    uintptr_t lo = 0, hi = 0;
    Span() {}
    Span(const void* p, long long rows, long long stride, long long width, size_t e)
        : lo((uintptr_t)p),
          hi(p && rows > 0 ? lo + (size_t)((rows - 1) * stride + width) * e : lo) {}
    Span(const void* p, long long n, size_t e) : Span(p, 1, n, n, e) {}  // n elements
    bool overlaps(const Span& o) const { return lo < hi && o.lo < o.hi && lo < o.hi && o.lo < hi; }
};
// Whether an output lies over another output or over an input.  An input that one of the
// outputs may replace is left out by the caller where that output has taken its very place:
// the comparisons of that output with the others then stand for its own.
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (o->overlaps(*q)) return true;
        for (const Span& i : ins)
            if (o->overlaps(i)) return true;
    }
    return false;
}

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
