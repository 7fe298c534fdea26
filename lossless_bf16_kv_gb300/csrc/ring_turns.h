// ring_turns.h -- what a ring of tiles that several warps fill in turn still has in
// flight (host and device; plain C++, so that the host can check it).
#pragma once

#include "wait_time.h"

namespace splitzip {

// The last tile put into each stage; tile n goes into stage n % kStages.  Warps may
// put neighbouring tiles, which are stages apart, in either order, so one number for the
// ring would be the smaller of two.  A stage's own tiles come in order: the next one
// waits until every warp is done with the one before.
template <int kStages>
struct RingTurns {
    uint32_t last[kStages];  // 1 more than the tile; 0: none yet
    SPLITZIP_HOST_DEVICE void clear() {
        for (int i = 0; i < kStages; i++) last[i] = 0;
    }
    SPLITZIP_HOST_DEVICE void put(uint32_t n) { last[n % kStages] = n + 1; }
    SPLITZIP_HOST_DEVICE bool used(uint32_t stage) const { return last[stage] != 0; }
    // Of the phase that the stage's last tile completes.
    SPLITZIP_HOST_DEVICE uint32_t parity(uint32_t stage) const { return (last[stage] - 1) / kStages & 1; }
};

}  // namespace splitzip
