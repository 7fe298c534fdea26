// evict.cu -- thinning a cache to its first, last and most attended slots
// (sm_103a): a selection per (sequence, key/value head), then a gather.
//
// Selection: weights are compared as 32-bit keys in which unsigned order is
// the order of the values (NaN lowest, -0 equal to 0).  The smallest key that
// is kept is found by radix selection, eight bits at a time from the top: a
// histogram of the digit among the keys that still match, then the digit in
// which the count from the top passes the number wanted.  A last pass in slot
// order writes the kept slots; of the slots at the smallest kept key only the
// first ones needed are kept.  One CTA per row, no communication between CTAs.
//
// Gather: kept rows are copied in order.  HBM bounds it: at 64 x 8 rows, 2048
// of 16384 slots of 128 BF16 values kept, 1.07 GB.
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

// Exclusive rank of each thread's flags a, b over the CTA, and their totals.
__device__ __forceinline__ void block_rank(bool a, bool b, uint32_t& ra, uint32_t& rb, uint32_t& ta,
                                           uint32_t& tb, uint32_t (*sums)[kSelectThreads / 32]) {
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ba = __ballot_sync(0xFFFFFFFFu, a), bb = __ballot_sync(0xFFFFFFFFu, b);
    const uint32_t below = (1u << lane) - 1u;
    if (lane == 0) {
        sums[0][warp] = __popc(ba);
        sums[1][warp] = __popc(bb);
    }
    __syncthreads();
    uint32_t xa = sums[0][lane], xb = sums[1][lane];
    const uint32_t oa = xa, ob = xb;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t ya = __shfl_up_sync(0xFFFFFFFFu, xa, d), yb = __shfl_up_sync(0xFFFFFFFFu, xb, d);
        if (lane >= d) xa += ya, xb += yb;
    }
    ta = __shfl_sync(0xFFFFFFFFu, xa, 31);
    tb = __shfl_sync(0xFFFFFFFFu, xb, 31);
    ra = __shfl_sync(0xFFFFFFFFu, xa - oa, warp) + __popc(ba & below);
    rb = __shfl_sync(0xFFFFFFFFu, xb - ob, warp) + __popc(bb & below);
    __syncthreads();
}

__global__ void __launch_bounds__(kSelectThreads) select_kernel(const __grid_constant__ splitzip_evict_args a) {
    __shared__ uint32_t hist[256];
    __shared__ uint32_t sums[2][kSelectThreads / 32];
    __shared__ uint32_t s_digit, s_want;
    const uint32_t row = blockIdx.x, b = row / a.kv_heads;
    const uint32_t tid = threadIdx.x;
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
    uint32_t least = 0xFFFFFFFFu;                            // smallest key kept; none yet
    if (want) {
        uint32_t prefix = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (uint32_t i = lo + tid; i < hi; i += kSelectThreads) {
                const uint32_t k = weight_key(w[i]);
                if (shift == 24 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
            }
            __syncthreads();
            if (tid < 32) {  // lane l holds digits 255 - 8 l down to 248 - 8 l
                uint32_t c[8], sum = 0;
#pragma unroll
                for (int i = 0; i < 8; i++) sum += c[i] = hist[255 - 8 * tid - i];
                uint32_t incl = sum;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, d);
                    if (tid >= d) incl += y;
                }
                uint32_t before = incl - sum;
                if (before < want && want <= incl) {
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        if (before < want && want <= before + c[i]) {
                            s_digit = 255 - 8 * tid - i;
                            s_want = want - before;
                        }
                        before += c[i];
                    }
                }
            }
            __syncthreads();
            prefix = prefix << 8 | s_digit;
            want = s_want;
            __syncthreads();
        }
        least = prefix;
    }
    uint32_t out = 0, equal_before = 0;
    for (uint32_t base = 0; base < n; base += kSelectThreads) {
        const uint32_t i = base + tid;
        const float v = i < n ? w[i] : 0.0f;
        const bool always = i < n && (i < lo || i >= hi), choice = i >= lo && i < hi;
        const uint32_t k = weight_key(v);
        const bool equal = choice && k == least;
        uint32_t re, rk, te, tk;
        // Equal keys are kept while fewer than `want` came before: two ranks,
        // since a slot's place depends on which equal ones before it are kept.
        block_rank(equal, always || (choice && k > least), re, rk, te, tk, sums);
        const uint32_t eq_at = equal_before + re;
        const bool keep = always || (choice && k > least) || (equal && eq_at < want);
        const uint32_t at = out + rk + (min(eq_at, want) - min(equal_before, want));
        if (keep) {
            index[at] = (int32_t)i;
            if (w_out) w_out[at] = v;
        }
        out += tk + (min(equal_before + te, want) - min(equal_before, want));
        equal_before += te;
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
    select_kernel<<<a.batch * a.kv_heads, kSelectThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const uint32_t row_bytes = a.head_dim * (a.cache_format == SPLITZIP_FORMAT_E5M2 ? 1 : 2);
    if (row_bytes == 64) return launch_gather<64>(a, s);
    if (row_bytes == 128) return launch_gather<128>(a, s);
    return launch_gather<256>(a, s);
}

}  // namespace splitzip
