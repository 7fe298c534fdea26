// api_checks.h -- argument checks that the serving entry points share (host side).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/splitzip_serving_testing.h"
#include "serving.h"

namespace splitzip {

inline splitzip_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SPLITZIP_OK : SPLITZIP_ERR_CUDA; }

inline bool dim_ok(uint32_t d) { return d == 64 || d == 128; }
inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// A view of nb x nt x nh rows.  Strides of dimensions of length 1 are not
// looked at; only an input's batch stride may be 0 (one sequence shared by the
// batch: as an output, all of it would be written to the same rows).
inline bool view_ok(const splitzip_view& v, uint32_t elem, uint32_t nb, uint32_t nt, uint32_t nh, bool output = false) {
    const int64_t unit = 16 / elem, most = 1ll << 38;
    const auto ok = [=](uint32_t n, int64_t s, int64_t least) { return n <= 1 || (s >= least && s < most && s % unit == 0); };
    return v.data && aligned(v.data, 16) && ok(nb, v.stride_b, output ? 1 : 0) && ok(nt, v.stride_t, 1) && ok(nh, v.stride_h, 1);
}

constexpr uint64_t kMax31 = 0x7FFFFFFFull;
// Slots and query rows of the attention calls: their kernels look up to two tiles
// of 128 past the last one in signed 32-bit numbers.
constexpr uint64_t kMostTokens = (1ull << 31) - 256;

// What a test leaves out, and how long waits last in it.
inline bool wait_test(const splitzip_wait_test_opts* opts, WaitTest& test) {
    if (!opts || opts->wait_ms > 2000) return false;
    test.limit = opts->wait_ms * 1000000u >> 10;
    test.cta = opts->cta;
    test.tile = opts->tile;
    return true;
}

}  // namespace splitzip
