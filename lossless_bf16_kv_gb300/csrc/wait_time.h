// wait_time.h -- how long a bounded wait has lasted (host and device; plain C++, so
// that the host can check it).
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SPLITZIP_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SPLITZIP_HOST_DEVICE inline
#endif

namespace splitzip {

// A wait looks at the clock between rounds of polls, which take microseconds.  The
// clock goes on while another program has the GPU, and then a round seems to take
// as long as that was: no round counts for more than this (2^24 ns).
constexpr uint32_t kMostRound = 1u << 14;

// What a wait may last: two seconds, and for each tile of work that the longest wait
// of a launch has to sit out 16 us, many times what one takes.  In units of 2^10 ns.
SPLITZIP_HOST_DEVICE constexpr uint32_t wait_limit(uint32_t tiles) { return (2000000000u >> 10) + 16u * tiles; }

// Counts in units of 2^10 ns, from the lower 32 bits of a clock in ns.
struct WaitTime {
    uint32_t last, waited;
    SPLITZIP_HOST_DEVICE explicit WaitTime(uint32_t now) : last(now), waited(0) {}
    SPLITZIP_HOST_DEVICE void round(uint32_t now) {
        const uint32_t units = (now - last) >> 10;
        waited += units < kMostRound ? units : kMostRound;
        last += units << 10;  // what is left counts with the next round
    }
};

}  // namespace splitzip
