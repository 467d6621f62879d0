// Which phase of its barrier to wait for before a ring of places in shared memory is left.  Copies go
// into the places in turn and are used in turn; `stage` is the place after the last one used and
// `parity` that of the phase its next copy completes (it changes with every pass over the ring).
// Plain C++, so that it can be checked without a GPU.
#pragma once

#include <stdint.h>

namespace ssd {
namespace layer {

// The parity of the phase that the last copy into `place` completes, where the last `unissued` of
// the copies that would have been used were never issued.  A place that took no copy gets the parity
// of the phase before its first, which counts as complete.
constexpr uint32_t landed_parity(int place, int places, int stage, uint32_t parity, int unissued) {
    int fill = stage - unissued;  // the place after the last copy
    while (fill < 0) {
        fill += places;
        parity ^= 1u;
    }
    return place < fill ? parity : parity ^ 1u;
}

}  // namespace layer
}  // namespace ssd
