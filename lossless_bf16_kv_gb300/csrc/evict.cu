// evict.cu -- thinning a cache to its first, last and most attended slots
// (sm_103a): a selection per (sequence, key/value head), then a gather.
//
// Selection: weights are compared as 32-bit keys in which unsigned order is
// the order of the values (NaN lowest, -0 equal to 0).  The smallest key that
// is kept is found by radix selection, 11, 11 and 10 bits from the top: a
// histogram of the digit among the keys that still match, then the digit in
// which the count from the top passes the number wanted.  A last pass in slot
// order writes the kept slots; of the slots at the smallest kept key only the
// first ones needed are kept.  One CTA per row, no communication between CTAs.
// The keys are read once and stay in shared memory where they fit (rows of up
// to 51200 slots): 512 rows of 16384 took 91 us reading the weights again from
// L2 in each of four passes of eight bits, with a CTA barrier every 1024 slots
// of the last pass; they take 49 us now that every thread ranks a short run of
// its own (0.7 TB/s: two CTAs to an SM, which wait for loads and barriers in turn).
//
// Gather: kept rows are copied in order.  HBM bounds it: at 64 x 8 rows, 2048
// of 16384 slots of 128 BF16 values kept, 1.07 GB in 154 us (6.6 TB/s, 97% of a
// copy's rate).
#include <cstdint>

#include "common.cuh"
#include "serving.h"

namespace splitzip {
namespace {

constexpr int kSelectThreads = 1024;

__device__ __forceinline__ uint32_t weight_key(float w) {
    if (w != w) return 0u;
    const uint32_t b = __float_as_uint(w + 0.0f);  // -0 + 0 = +0
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr int kBins = 2048;
constexpr uint32_t kMostKeys = 51200;  // slots whose keys fit in shared memory, 200 KB

struct SelectShared {
    uint32_t hist[kBins];
    uint32_t warp[2][kSelectThreads / 32];
    uint32_t digit, want;
};

// Exclusive sums over the warps of each warp's value.
__device__ __forceinline__ uint32_t before_warp(uint32_t v, uint32_t warp, uint32_t* all) {
    const uint32_t lane = threadIdx.x & 31;
    if (lane == 0) all[warp] = v;
    __syncthreads();
    const uint32_t own = all[lane];
    uint32_t x = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d) x += y;
    }
    return __shfl_sync(0xFFFFFFFFu, x - own, warp);
}

// Exclusive sums over the threads of each thread's value.
__device__ __forceinline__ uint32_t before_thread(uint32_t v, uint32_t lane, uint32_t warp, uint32_t* all) {
    uint32_t incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += y;
    }
    return before_warp(__shfl_sync(0xFFFFFFFFu, incl, 31), warp, all) + incl - v;
}

template <bool kInShared>
__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ splitzip_evict_args a) {
    __shared__ SelectShared sh;
    extern __shared__ uint32_t keys[];
    const uint32_t row = blockIdx.x, b = row / a.kv_heads;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int32_t len = a.lens ? a.lens[b] : (int32_t)a.kv_tokens;
    const uint32_t n = len < 0 ? 0u : min((uint32_t)len, a.kv_tokens);
    const float* w = a.weights + (uint64_t)row * a.kv_tokens;
    int32_t* index = a.index + (uint64_t)row * a.budget;
    float* w_out = a.weights_out ? a.weights_out + (uint64_t)row * a.budget : nullptr;
    const uint32_t kept = min(n, a.budget);
    if (a.lens_out && row % a.kv_heads == 0 && tid == 0) a.lens_out[b] = (int32_t)kept;
    for (uint32_t j = kept + tid; j < a.budget; j += kSelectThreads) {
        index[j] = -1;
        if (w_out) w_out[j] = 0.0f;
    }
    if (n <= a.budget) {
        for (uint32_t j = tid; j < n; j += kSelectThreads) {
            index[j] = (int32_t)j;
            if (w_out) w_out[j] = w[j];
        }
        return;
    }
    const uint32_t lo = a.keep_first, hi = n - a.keep_last;  // the slots to choose from
    uint32_t want = a.budget - a.keep_first - a.keep_last;   // how many of them, < hi - lo
    uint32_t least = 0;                                      // the smallest key kept
    auto key = [&](uint32_t i) { return kInShared ? keys[i] : weight_key(w[i]); };
    if (kInShared && !want) {
        for (uint32_t i = tid; i < n; i += kSelectThreads) keys[i] = weight_key(w[i]);
    }
    if (want) {
        uint32_t prefix = 0;
#pragma unroll
        for (int pass = 0; pass < 3; pass++) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            for (uint32_t i = tid; i < kBins; i += kSelectThreads) sh.hist[i] = 0;
            __syncthreads();
            if (pass == 0) {
                // The weight 0 is common (slots never attended) and counted apart.
                constexpr uint32_t kZero = 0x80000000u;
                uint32_t zeros = 0;
#pragma unroll 8
                for (uint32_t i = tid; i < n; i += kSelectThreads) {
                    const uint32_t k = weight_key(w[i]);
                    if (kInShared) keys[i] = k;
                    if (i < lo || i >= hi) continue;
                    if (k == kZero) zeros++;
                    else atomicAdd(&sh.hist[k >> shift], 1u);
                }
                zeros = __reduce_add_sync(0xFFFFFFFFu, zeros);
                if (lane == 0 && zeros) atomicAdd(&sh.hist[kZero >> shift], zeros);
            } else {
#pragma unroll 4
                for (uint32_t i = lo + tid; i < hi; i += kSelectThreads) {
                    const uint32_t k = key(i);
                    if (k >> (shift + bits) == prefix) atomicAdd(&sh.hist[(k >> shift) & ((1u << bits) - 1u)], 1u);
                }
            }
            __syncthreads();
            // Thread t holds digits kBins - 1 - 2 t and the one below.
            const uint32_t d0 = kBins - 1 - 2 * tid, c0 = sh.hist[d0], c1 = sh.hist[d0 - 1];
            const uint32_t before = before_thread(c0 + c1, lane, warp, sh.warp[0]);
            if (before < want && want <= before + c0 + c1) {
                const bool upper = want <= before + c0;
                sh.digit = upper ? d0 : d0 - 1;
                sh.want = want - before - (upper ? 0 : c0);
            }
            __syncthreads();
            prefix = prefix << bits | sh.digit;
            want = sh.want;
        }
        least = prefix;
    }
    // Each thread ranks a short run of slots: how many before it are kept for good,
    // and how many have the smallest kept key (the first `want` of those are kept, so
    // a slot's place depends on how many came before).  Slots that are always kept
    // get a key above every weight's.  Runs of odd length: no bank conflicts.
    constexpr uint32_t kAlways = 0xFFFFFFFFu;
    __syncthreads();
    if (kInShared) {
        for (uint32_t i = tid; i < lo; i += kSelectThreads) keys[i] = kAlways;
        for (uint32_t i = hi + tid; i < n; i += kSelectThreads) keys[i] = kAlways;
        __syncthreads();
    }
    // The keys kept for good are those from `sure_key` on.
    const uint32_t sure_key = a.budget == a.keep_first + a.keep_last ? kAlways : least + 1;
    auto rank_key = [&](uint32_t i) { return kInShared ? keys[i] : i < lo || i >= hi ? kAlways : weight_key(w[i]); };
    const uint32_t run = ((n + kSelectThreads - 1) / kSelectThreads) | 1u, from = min(tid * run, n), to = min(from + run, n);
    uint32_t sure = 0, equal = 0;
    for (uint32_t i = from; i < to; i++) {
        const uint32_t k = rank_key(i);
        sure += k >= sure_key;
        equal += k == least;
    }
    if (want == 0) equal = 0;
    sure = before_thread(sure, lane, warp, sh.warp[0]);
    equal = before_thread(equal, lane, warp, sh.warp[1]);
    for (uint32_t i = from; i < to; i++) {
        const uint32_t k = rank_key(i);
        const bool eq = k == least;
        if (k >= sure_key || (eq && equal < want)) {
            const uint32_t at = sure + min(equal, want);
            index[at] = (int32_t)i;
            if (w_out) w_out[at] = w[i];
        }
        sure += k >= sure_key;
        equal += eq;
    }
}

constexpr int kGatherRows = 4;  // rows of K and V a group of lanes has in flight

template <int kRowBytes>
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ splitzip_evict_args a) {
    constexpr int kLanes = kRowBytes / 16;
    const uint32_t e = a.cache_format == SPLITZIP_FORMAT_E5M2 ? 1 : 2;
    const uint32_t lane = threadIdx.x % kLanes;
    const uint32_t groups = 256 / kLanes;
    const uint32_t b = blockIdx.y;
    const uint64_t rows = (uint64_t)a.budget * a.kv_heads;
    const uint64_t first = (uint64_t)blockIdx.x * groups * kGatherRows + threadIdx.x / kLanes;
    const uint8_t* src[2] = {static_cast<const uint8_t*>(a.k.data) + (int64_t)b * a.k.stride_b * e,
                             static_cast<const uint8_t*>(a.v.data) + (int64_t)b * a.v.stride_b * e};
    uint8_t* dst[2] = {static_cast<uint8_t*>(a.k_out.data) + (int64_t)b * a.k_out.stride_b * e,
                       static_cast<uint8_t*>(a.v_out.data) + (int64_t)b * a.v_out.stride_b * e};
    int32_t from[kGatherRows];
    uint32_t j[kGatherRows], h[kGatherRows];
    uint4 x[kGatherRows][2];
#pragma unroll
    for (int r = 0; r < kGatherRows; r++) {
        const uint64_t i = first + (uint64_t)r * groups;
        from[r] = -2;  // past the end
        if (i < rows) {
            j[r] = (uint32_t)(i / a.kv_heads);
            h[r] = (uint32_t)(i - (uint64_t)j[r] * a.kv_heads);
            from[r] = a.index[((uint64_t)b * a.kv_heads + h[r]) * a.budget + j[r]];
        }
    }
#pragma unroll
    for (int r = 0; r < kGatherRows; r++) {
        x[r][0] = x[r][1] = make_uint4(0, 0, 0, 0);
        if (from[r] >= 0) {
            x[r][0] = ld_stream16(src[0] + (from[r] * a.k.stride_t + h[r] * a.k.stride_h) * e + 16 * lane);
            x[r][1] = ld_stream16(src[1] + (from[r] * a.v.stride_t + h[r] * a.v.stride_h) * e + 16 * lane);
        }
    }
#pragma unroll
    for (int r = 0; r < kGatherRows; r++) {
        if (from[r] == -2) continue;
        st_stream16(dst[0] + (j[r] * a.k_out.stride_t + h[r] * a.k_out.stride_h) * e + 16 * lane, x[r][0]);
        st_stream16(dst[1] + (j[r] * a.v_out.stride_t + h[r] * a.v_out.stride_h) * e + 16 * lane, x[r][1]);
    }
}

template <int kRowBytes>
cudaError_t launch_gather(const splitzip_evict_args& a, cudaStream_t s) {
    const uint64_t per_cta = (uint64_t)(256 / (kRowBytes / 16)) * kGatherRows;
    const uint64_t rows = (uint64_t)a.budget * a.kv_heads;
    gather_kernel<kRowBytes><<<dim3((unsigned)((rows + per_cta - 1) / per_cta), a.batch), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const splitzip_evict_args& a, cudaStream_t s) {
    cudaError_t e;
    if (a.kv_tokens <= kMostKeys) {
        Wave w;
        e = launch_wave<select_kernel<true>>(kSelectThreads, 4 * kMostKeys, w);
        if (e != cudaSuccess) return e;
        select_kernel<true><<<a.batch * a.kv_heads, kSelectThreads, 4 * a.kv_tokens, s>>>(a);
    } else {
        select_kernel<false><<<a.batch * a.kv_heads, kSelectThreads, 0, s>>>(a);
    }
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const uint32_t row_bytes = a.head_dim * (a.cache_format == SPLITZIP_FORMAT_E5M2 ? 1 : 2);
    if (row_bytes == 64) return launch_gather<64>(a, s);
    if (row_bytes == 128) return launch_gather<128>(a, s);
    return launch_gather<256>(a, s);
}

}  // namespace splitzip
