// pages.cu -- rows into and out of the pages of a cache (sm_103a): the store that
// quantises new keys and values, and the load that widens them back.
//
// A block of head_dim / 4 values x becomes codes c = rne(x 2^-k) with k the smallest
// power for which the largest |x| 2^-k does not round past the largest code.  That
// largest |x| is an 8-bit significand 1.f times 2^E, so k = E - 6 for INT8, or E - 5
// where 1.f is 255/128 (127.5 rounds to 128); and k = E - 2 for E2M1, or E - 1 from
// 1.75 on (7 rounds past 6).  x 2^-k is exact in 32 bits: one rounding in all, and
// no division.
//
// Both move each byte once, so HBM bounds them.  A row is shared by head_dim / 8
// lanes of eight values (16 bytes of BF16); a group of lanes takes kRows tokens of one
// head, and the groups of a CTA neighbouring tokens, whose rows are neighbours in
// a page that lies head by head (E2M1 rows of head_dim 64 are 32 bytes).  A group of
// the load takes tokens that lie side by side in one page, so the page, the address
// and (where they are contiguous) the exponent bytes are found once for them.
//
// 16 sequences of 16k tokens, 8 heads of 128, read back: BF16 309 us (6.9 TB/s read and
// written), E5M2 235, 8 bits 240, 4 bits 202, all within 2% of a copy's rate.  One layer
// of a 16k prompt stored and read back: 35, 29, 33 and 31 us, where the store of quantised
// rows is bound by its instructions as much (in 8 bits 1.4 us of it were addresses in 64
// bits of what fits 32).
#include <cstdint>

#include <cuda_bf16.h>

#include "common.cuh"
#include "pages.cuh"
#include "tcgen.cuh"

namespace splitzip {
namespace {

constexpr int kThreadsPages = 256, kRows = 4;
// Tokens of a CTA.
template <int D>
constexpr uint32_t kTokens = kThreadsPages / (D / 8) * kRows;

// What both kernels' CTAs take: one of keys and values, a sequence (0 for the
// store), a head, and kTokens tokens from `first` on.
struct Part {
    uint32_t b, h, first;
    bool v;
};
template <int D>
__device__ __forceinline__ Part part_of(uint32_t block, uint32_t heads, uint32_t token_ctas) {
    const uint32_t x = block / token_ctas, y = x / heads;
    return {y >> 1, x - y * heads, (block - x * token_ctas) * kTokens<D>, (y & 1) != 0};
}

// The largest magnitude's BF16 bits over the lanes of a block (`lanes` neighbours), of
// pairs of them.
template <int kLanes>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
#pragma unroll
    for (int i = 1; i < kLanes; i *= 2) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, i));
    return max(m & 0xFFFFu, m >> 16);
}

// The block's power from its largest magnitude's BF16 bits, and its exponent byte.
template <int kFmt>
__device__ __forceinline__ int block_power(uint32_t top, uint32_t& e) {
    constexpr int kAway = kFmt == kInt8 ? 6 : 2, kLow = kFmt == kInt8 ? -24 : -23, kHigh = kFmt == kInt8 ? 9 : 13;
    constexpr uint32_t kNext = kFmt == kInt8 ? 127 : 96;  // fraction bits from where the next power is taken
    const int k = min(max((int)((top + (128 - kNext)) >> 7) - 127 - kAway, kLow), kHigh);
    e = top >= 0x7F80u ? 255u : top == 0u ? 0u : (uint32_t)(k + 127);
    return k;
}
// Four codes of values x times the power's inverse: added to 1.5 2^23, whose step is 1,
// they are rounded to nearest even into the sum's lower byte.
__device__ __forceinline__ uint32_t to_int8x4(const float* x, float inv) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = __float_as_uint(fmaf(x[i], inv, 12582912.0f));
    return prmt(prmt(r[0], r[1], 0x0040), prmt(r[2], r[3], 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t to_e2m1x8(const float* x, float inv) {
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; i++) z[i] = x[i] * inv;
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
    return r;
}

struct StoreParams {
    splitzip_pages_store_args a;
    uint32_t token_ctas, page_shift;
};

template <int D, int kFmt>
__global__ void __launch_bounds__(kThreadsPages) store_kernel(const __grid_constant__ StoreParams p) {
    constexpr uint32_t kLanes = D / 8, kGroups = kThreadsPages / kLanes;
    const splitzip_pages_store_args& a = p.a;
    const Part part = part_of<D>(blockIdx.x, a.pool.kv_heads, p.token_ctas);
    const uint32_t lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    const splitzip_view& in = part.v ? a.v : a.k;
    const splitzip_page_rows& out = part.v ? a.pool.v : a.pool.k;
    const uint64_t slots = (uint64_t)a.pool.pages << p.page_shift;
    const uint8_t* src = static_cast<const uint8_t*>(in.data) + 2 * (part.h * in.stride_h) + 16 * lane;
    constexpr uint32_t kElem = kFmt == kBf16 ? 2 : 1, kPiece = kRowBytes<D, kFmt> / kLanes;
    uint8_t* to = static_cast<uint8_t*>(out.data) + kElem * (part.h * out.stride_h) + kPiece * lane;
    uint8_t* to_exp = kQuantised<kFmt> ? out.exponents + part.h * out.exp_stride_h : nullptr;
    uint4 x[kRows];
    int64_t slot[kRows];
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        const uint32_t t = part.first + r * kGroups + group;
        x[r] = make_uint4(0, 0, 0, 0);
        slot[r] = -1;
        if (t < a.n) {
            x[r] = ld_stream16(src + 2 * ((int64_t)t * in.stride_t));
            slot[r] = a.slots[t];
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        const bool there = slot[r] >= 0 && (uint64_t)slot[r] < slots;
        const uint32_t page = (uint32_t)(slot[r] >> p.page_shift), at = (uint32_t)slot[r] & (a.pool.page_tokens - 1);
        uint8_t* row = to + kElem * ((int64_t)page * out.stride_p + (int64_t)at * out.stride_t);
        const uint32_t w[4] = {x[r].x, x[r].y, x[r].z, x[r].w};
        if constexpr (kFmt == kBf16) {
            if (there) *reinterpret_cast<uint4*>(row) = x[r];
        } else {
            float f[8];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
            if constexpr (kFmt == kE5m2) {
                if (there) *reinterpret_cast<uint2*>(row) = make_uint2(pack4_e5m2(f), pack4_e5m2(f + 4));
            } else {
                uint32_t e;
                const uint32_t top = block_max<kLanes / 4>(__vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                                                                    __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu)));
                const int k = block_power<kFmt>(top, e);
                // 0 for a block that holds an infinity or a NaN: its codes are 0 below.
                const float inv = __uint_as_float((uint32_t)(127 - k) << 23);
                if (kFmt == kInt8 && top >= 0x477Fu) {  // from 65280 on, 127.5 times the largest power
#pragma unroll
                    for (int i = 0; i < 8; i++) f[i] = fminf(fmaxf(f[i], -65024.0f), 65024.0f);
                }
                const bool odd = top >= 0x7F80u;
                // The four exponent bytes, gathered over the row's lanes.
                e <<= 8 * (lane / (kLanes / 4));
#pragma unroll
                for (uint32_t i = kLanes / 4; i < kLanes; i *= 2) e |= __shfl_xor_sync(0xFFFFFFFFu, e, i);
                if (there) {
                    if constexpr (kFmt == kInt8) *reinterpret_cast<uint2*>(row) = odd ? make_uint2(0, 0) : make_uint2(to_int8x4(f, inv), to_int8x4(f + 4, inv));
                    else *reinterpret_cast<uint32_t*>(row) = odd ? 0u : to_e2m1x8(f, inv);
                    if (lane == 0)
                        *reinterpret_cast<uint32_t*>(to_exp + (int64_t)page * out.exp_stride_p + (int64_t)at * out.exp_stride_t) = e;
                }
            }
        }
    }
}

// Eight values of a row, as they lie in a page, in BF16; bytes: the row's exponents.
template <int D, int kFmt>
__device__ __forceinline__ uint4 to_bf16(uint4 x, uint32_t bytes, uint32_t lane) {
    if constexpr (kFmt == kBf16) return x;
    uint32_t h[4];
    if constexpr (kFmt == kE5m2) {
        const uint32_t w[4] = {e5m2_01(x.x), e5m2_23(x.x), e5m2_01(x.y), e5m2_23(x.y)};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 f = unpack2<true>(w[i]);
            h[i] = pack2<false>(f.x, f.y);
        }
    } else {
        const float f = block_scale(bytes >> 8 * (lane / (D / 32)) & 255u);
        const uint64_t scale = pair(f, f);
        if constexpr (kFmt == kInt8) {
            // A byte b as 2^23 + (b + 128), less what is too much: exact in 32 bits.
            const uint64_t less = pair(-8388736.0f, -8388736.0f);
            const uint32_t w[2] = {int8_bias(x.x), int8_bias(x.y)};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const uint32_t s = 0x7440u + 2 * (i & 1);
                float a, b;
                unpair(mul2(add2(pair(__uint_as_float(prmt(w[i >> 1], 0x4B000000u, s)), __uint_as_float(prmt(w[i >> 1], 0x4B000000u, s + 1))), less), scale), a, b);
                h[i] = pack2<false>(a, b);
            }
        } else {
            uint32_t w[4];
            e2m1_pairs(w, x.x);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 g = unpack2<true>(w[i]);
                float a, b;
                unpair(mul2(pair(g.x, g.y), scale), a, b);
                h[i] = pack2<false>(a, b);
            }
        }
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// The same in FP16, which holds every value that the store leaves (infinities and NaN too).
template <int D, int kFmt>
__device__ __forceinline__ uint4 to_f16(uint4 x, uint32_t bytes, uint32_t lane) {
    if constexpr (kFmt == kE5m2) return make_uint4(e5m2_01(x.x), e5m2_23(x.x), e5m2_01(x.y), e5m2_23(x.y));
    const float f = block_scale(bytes >> 8 * (lane / (D / 32)) & 255u);
    const uint32_t s = pack2<true>(f, f);
    uint32_t h[4];
    if constexpr (kFmt == kInt8) {
        const uint32_t lo = int8_bias(x.x), hi = int8_bias(x.y);
        h[0] = int8_pair<kInt8_01>(lo), h[1] = int8_pair<kInt8_23>(lo), h[2] = int8_pair<kInt8_01>(hi), h[3] = int8_pair<kInt8_23>(hi);
    } else {
        e2m1_pairs(h, x.x);
    }
    return make_uint4(mul_half2(h[0], s), mul_half2(h[1], s), mul_half2(h[2], s), mul_half2(h[3], s));
}

// A group's kRows tokens from t on (all of one page), of one head of keys or values, up
// to token n: put(row, x) takes eight values in kOut: BF16, FP16, or E5M2 rows as they are.
template <int D, int kFmt, int kOut, class Put>
__device__ __forceinline__ void load_rows(const splitzip_pool& pool, const splitzip_page_rows& in, uint32_t page, uint32_t h, uint32_t t, uint32_t n,
                                          bool bulk_exps, uint32_t lane, const Put& put) {
    const bool bad = page >= pool.pages;
    const int64_t at = t & (pool.page_tokens - 1), from = bad ? 0 : page;
    const uint8_t* src = static_cast<const uint8_t*>(in.data) + (kFmt == kBf16 ? 2 : 1) * (from * in.stride_p + at * in.stride_t + h * in.stride_h) +
                         kRowBytes<D, kFmt> / (D / 8) * lane;
    const int64_t step = (kFmt == kBf16 ? 2 : 1) * in.stride_t;
    uint4 x[kRows];
    uint32_t e[kRows] = {};
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        x[r] = make_uint4(0, 0, 0, 0);
        if constexpr (kFmt == kBf16) {
            x[r] = ld_stream16(src + r * step);
        } else if constexpr (kFmt == kE2m1) {
            x[r].x = ld_stream4(src + r * step);
        } else {
            const uint2 y = ld_stream8(src + r * step);
            x[r].x = y.x, x[r].y = y.y;
        }
    }
    if constexpr (kQuantised<kFmt>) {
        const uint8_t* bytes = in.exponents + from * in.exp_stride_p + at * in.exp_stride_t + h * in.exp_stride_h;
        if (bulk_exps) {
            const uint4 y = *reinterpret_cast<const uint4*>(bytes);
            e[0] = y.x, e[1] = y.y, e[2] = y.z, e[3] = y.w;
        } else {
#pragma unroll
            for (int r = 0; r < kRows; r++) e[r] = *reinterpret_cast<const uint32_t*>(bytes + r * in.exp_stride_t);
        }
    }
    static_assert(kRows == 4, "four rows' exponents in 16 bytes");
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        if (t + r >= n) break;
        if constexpr (kOut == kE5m2) put(t + r, bad ? make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0, 0) : x[r]);
        else if constexpr (kOut == kF16) put(t + r, bad ? make_uint4(0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u) : to_f16<D, kFmt>(x[r], e[r], lane));
        else put(t + r, bad ? make_uint4(0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u) : to_bf16<D, kFmt>(x[r], e[r], lane));
    }
}

struct LoadParams {
    splitzip_pages_load_args a;
    uint32_t token_ctas, page_shift, bulk_exps;
};

template <int D, int kFmt, int kOut>
__global__ void __launch_bounds__(kThreadsPages) load_kernel(const __grid_constant__ LoadParams p) {
    constexpr uint32_t kLanes = D / 8;
    const splitzip_pages_load_args& a = p.a;
    const Part part = part_of<D>(blockIdx.x, a.pool.kv_heads, p.token_ctas);
    const int32_t len = a.lens ? a.lens[part.b] : (int32_t)a.tokens;
    const uint32_t n = len < 0 ? 0u : min((uint32_t)len, a.tokens);
    const uint32_t lane = threadIdx.x % kLanes, t = part.first + threadIdx.x / kLanes * kRows;
    if (t >= n) return;
    const splitzip_view& out = part.v ? a.v_out : a.k_out;
    constexpr int kElem = kOut == kE5m2 ? 1 : 2;
    uint8_t* to = static_cast<uint8_t*>(out.data) + kElem * (part.b * out.stride_b + part.h * out.stride_h + 8 * lane);
    const uint32_t page = (uint32_t)a.table[(uint64_t)part.b * a.table_width + (t >> p.page_shift)];
    load_rows<D, kFmt, kOut>(a.pool, part.v ? a.pool.v : a.pool.k, page, part.h, t, n, p.bulk_exps, lane, [&](uint32_t row, uint4 x) {
        uint8_t* at = to + kElem * ((int64_t)row * out.stride_t);
        if constexpr (kOut == kE5m2) st_stream8(at, make_uint2(x.x, x.y));
        else st_stream16(at, x);
    });
}

// The caches of long sequences, widened to FP16 for launch_paged_tiles: the load's work, to
// contiguous rows, which the products then find in L2 where they fit (8k tokens of 8 heads
// of 128 in 8 bits: 11 us).  FP16 and not BF16, as the softmax weights take their values'
// type: 11 bits of each, as where tiles are widened one by one, and not 8.
struct WidenParams {
    splitzip_paged_attention_args a;
    uint32_t token_ctas, page_shift, bulk_exps;
    uint32_t group, rows_from, sequences, tokens;  // tokens of a widened cache
    uint8_t* to;
};

template <int D, int kFmt>
__global__ void __launch_bounds__(kThreadsPages) widen_kernel(const __grid_constant__ WidenParams p) {
    constexpr uint32_t kLanes = D / 8;
    const splitzip_paged_attention_args& a = p.a;
    __shared__ int32_t found, from, count, len;
    const Part part = part_of<D>(blockIdx.x, a.pool.kv_heads, p.token_ctas);
    if (threadIdx.x < 32) {  // the part.b-th long sequence
        const uint32_t b = nth_long(a, part.b, p.group, p.rows_from, threadIdx.x);
        if (threadIdx.x == 0) {
            found = (int32_t)b;
            if (b < a.batch) {
                const Sequence s(a, b);
                from = s.row, count = s.count, len = s.n;
            }
        }
    }
    __syncthreads();
    if (found >= (int32_t)a.batch) return;
    const uint32_t lane = threadIdx.x % kLanes, t = part.first + threadIdx.x / kLanes * kRows, n = (uint32_t)len;
    // What no query sees need not be there, and its page may have been given away.
    const Mask mask(len, count, a.window, a.sinks);
    const auto seen = [&](uint32_t s, uint32_t run) {
        return s < n && ((int64_t)s + run > (int64_t)mask.first - (int64_t)mask.window + 1 || s < (uint32_t)mask.sinks);
    };
    if (!seen(t & ~127u, 128)) return;  // a tile of the products
    uint8_t* to = p.to + 2 * ((((uint64_t)part.b * 2 + part.v) * a.pool.kv_heads + part.h) * p.tokens * D + 8 * lane);
    const auto put = [&](uint32_t row, uint4 x) { *reinterpret_cast<uint4*>(to + 2 * (uint64_t)row * D) = x; };
    const bool here = seen(t, kRows);
    if (here) {
        const uint32_t page = (uint32_t)a.table[(uint64_t)found * a.table_width + (t >> p.page_shift)];
        load_rows<D, kFmt, kF16>(a.pool, part.v ? a.pool.v : a.pool.k, page, part.h, t, n, p.bulk_exps, lane, put);
    }
    // The rest of a tile is zeros and not what the workspace held: infinities and NaN among
    // that would be kept out of the products one by one.
#pragma unroll
    for (uint32_t r = 0; r < kRows; r++)
        if (!here || t + r >= n) put(t + r, make_uint4(0, 0, 0, 0));
}

inline uint32_t log2_of(uint32_t x) {
    uint32_t n = 0;
    while (x >>= 1) n++;
    return n;
}

template <int D>
cudaError_t store(const splitzip_pages_store_args& a, cudaStream_t s) {
    const uint32_t token_ctas = (uint32_t)(((uint64_t)a.n + kTokens<D> - 1) / kTokens<D>);
    const StoreParams p{a, token_ctas, log2_of(a.pool.page_tokens)};
    const uint32_t ctas = token_ctas * a.pool.kv_heads * 2;
    switch (a.pool.format) {
        case kBf16: store_kernel<D, kBf16><<<ctas, kThreadsPages, 0, s>>>(p); break;
        case kE5m2: store_kernel<D, kE5m2><<<ctas, kThreadsPages, 0, s>>>(p); break;
        case kInt8: store_kernel<D, kInt8><<<ctas, kThreadsPages, 0, s>>>(p); break;
        default: store_kernel<D, kE2m1><<<ctas, kThreadsPages, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}

template <int D>
cudaError_t load(const splitzip_pages_load_args& a, cudaStream_t s) {
    const uint32_t token_ctas = (a.tokens + kTokens<D> - 1) / kTokens<D>;
    const LoadParams p{a, token_ctas, log2_of(a.pool.page_tokens), bulk_exponents(a.pool)};
    const uint32_t ctas = token_ctas * a.pool.kv_heads * 2 * a.batch;
    switch (a.pool.format) {
        case kBf16: load_kernel<D, kBf16, kBf16><<<ctas, kThreadsPages, 0, s>>>(p); break;
        case kE5m2:
            if (a.out_format == kE5m2) load_kernel<D, kE5m2, kE5m2><<<ctas, kThreadsPages, 0, s>>>(p);
            else load_kernel<D, kE5m2, kBf16><<<ctas, kThreadsPages, 0, s>>>(p);
            break;
        case kInt8: load_kernel<D, kInt8, kBf16><<<ctas, kThreadsPages, 0, s>>>(p); break;
        default: load_kernel<D, kE2m1, kBf16><<<ctas, kThreadsPages, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

template <int D>
static cudaError_t widen(const WidenParams& p, cudaStream_t s) {
    const uint32_t ctas = p.token_ctas * p.a.pool.kv_heads * 2 * p.sequences;
    switch (p.a.pool.format) {
        case kE5m2: widen_kernel<D, kE5m2><<<ctas, kThreadsPages, 0, s>>>(p); break;
        case kInt8: widen_kernel<D, kInt8><<<ctas, kThreadsPages, 0, s>>>(p); break;
        default: widen_kernel<D, kE2m1><<<ctas, kThreadsPages, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}
cudaError_t launch_paged_widen(const splitzip_paged_attention_args& a, uint32_t rows_from, void* widened, cudaStream_t s) {
    const uint32_t tokens = a.pool.head_dim == 64 ? kTokens<64> : kTokens<128>;
    WidenParams p{a};
    p.page_shift = log2_of(a.pool.page_tokens);
    p.bulk_exps = bulk_exponents(a.pool);
    p.group = a.q_heads / a.pool.kv_heads;
    p.rows_from = rows_from;
    p.sequences = (uint32_t)widened_sequences(a, rows_from);
    p.tokens = (uint32_t)widened_tokens(a);
    p.token_ctas = p.tokens / tokens;  // which divides 128
    p.to = static_cast<uint8_t*>(widened);
    return a.pool.head_dim == 64 ? widen<64>(p, s) : widen<128>(p, s);
}
cudaError_t launch_pages_store(const splitzip_pages_store_args& a, cudaStream_t s) {
    return a.pool.head_dim == 64 ? store<64>(a, s) : store<128>(a, s);
}
cudaError_t launch_pages_load(const splitzip_pages_load_args& a, cudaStream_t s) {
    return a.pool.head_dim == 64 ? load<64>(a, s) : load<128>(a, s);
}

}  // namespace splitzip
