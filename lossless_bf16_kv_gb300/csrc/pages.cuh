// pages.cuh -- rows of a paged cache (sm_103a): their formats, where they lie, and
// the widening of quantised codes to FP16.
#pragma once

#include <cstdint>

#include "attention.cuh"
#include "pages.h"

namespace splitzip {

enum Format : int {
    kBf16 = SPLITZIP_FORMAT_BF16, kE5m2 = SPLITZIP_FORMAT_E5M2, kInt8 = SPLITZIP_FORMAT_INT8, kE2m1 = SPLITZIP_FORMAT_E2M1,
    kF16  // no pool's: caches widened ahead of the products
};

template <int kFmt>
constexpr bool kWide = kFmt != kBf16;  // operands are FP16 ..
template <int kFmt>
constexpr bool kWidens = kWide<kFmt> && kFmt != kF16;  // .. and widened from the cache's bytes by the attention kernel
template <int kFmt>
constexpr bool kQuantised = kFmt == kInt8 || kFmt == kE2m1;
// Bytes of a row's codes.
template <int D, int kFmt>
constexpr int kRowBytes = !kWidens<kFmt> ? 2 * D : kFmt == kE2m1 ? D / 2 : D;

// New tokens of a sequence whose rows are from .. to - 1; 0 where that is no range to be taken.
__device__ __forceinline__ int32_t sequence_count(const splitzip_paged_attention_args& a, int32_t from, int32_t to) {
    return from >= 0 && to >= from && (uint32_t)to <= a.tokens && (uint32_t)(to - from) <= a.max_q_tokens ? to - from : 0;
}

// One sequence of a batch: its new tokens' first row, their number (0: left out),
// its length.
struct Sequence {
    int32_t row, count, n;
    __device__ __forceinline__ Sequence(const splitzip_paged_attention_args& a, uint32_t b) {
        const int32_t from = a.q_start[b], to = a.q_start[b + 1], len = a.lens[b];
        row = from;
        count = sequence_count(a, from, to);
        n = len < 0 ? 0 : min(len, (int32_t)a.kv_tokens);
    }
};

// The n-th (from 0) sequence with more than rows_from query rows; a.batch where there is
// none.  A whole warp.
__device__ __forceinline__ uint32_t nth_long(const splitzip_paged_attention_args& a, uint32_t n, uint32_t group, uint32_t rows_from, uint32_t lane) {
    for (uint32_t b = 0; b < a.batch; b += 32) {
        const bool is = b + lane < a.batch && (uint32_t)sequence_count(a, a.q_start[b + lane], a.q_start[b + lane + 1]) * group > rows_from;
        const uint32_t found = __ballot_sync(0xFFFFFFFFu, is), before = __popc(found & ((1u << lane) - 1u));
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, is && before == n);
        if (hit) return b + (uint32_t)__ffs(hit) - 1;
        n -= __popc(found);
    }
    return a.batch;
}

// 2^(e - 127) for an exponent byte: 0 for 0, NaN for 255.
__device__ __forceinline__ float block_scale(uint32_t e) {
    const uint32_t bits = e << 23;
    return __uint_as_float(e == 255u ? bits | 0x400000u : bits);
}

// FP16 pairs of codes, exact.  INT8: two bytes of r, as 1024 + (b + 128) less 1152
// (1024 to 2047 have a step of 1 in FP16, so the byte is the lower half of the value).
template <int kSelect>
__device__ __forceinline__ uint32_t int8_pair(uint32_t biased) {
    const uint32_t w = prmt(biased, 0x64646464u, kSelect);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&w), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&v);
}
// The same times a pair of powers of up to 2^5 (exponent byte kInt8OneStep), in one step: 1152 times those is still
// an FP16 number, and the sum of the exact products is rounded once, to what it is.
constexpr uint32_t kInt8OneStep = 127 + 5;
template <int kSelect>
__device__ __forceinline__ uint32_t int8_scaled(uint32_t biased, uint32_t powers) {
    const uint32_t w = prmt(biased, 0x64646464u, kSelect);
    const __half2 f = *reinterpret_cast<const __half2*>(&powers);
    const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&w), f, __hmul2(f, __half2half2(__ushort_as_half(0xE480))));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t int8_bias(uint32_t r) { return r ^ 0x80808080u; }
constexpr int kInt8_01 = 0x4140, kInt8_23 = 0x4342, kInt8_02 = 0x4240, kInt8_13 = 0x4341;
// E2M1: the two halves of each byte of r (the lower half first).
__device__ __forceinline__ void e2m1_pairs(uint32_t (&h)[4], uint32_t r) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(r));
}
// Whether one of four exponent bytes stands for more than 2^5.
__device__ __forceinline__ bool above_5(uint32_t x) { return (((x & 0x7F7F7F7Fu) + 0x7B7B7B7Bu) & x & 0x80808080u) != 0; }
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// One value of a row as the products have it, for the rare ones that are not finite.
template <int D, int kFmt>
__device__ __forceinline__ float page_value(const uint8_t* row, const uint8_t* exps, uint32_t d) {
    if (kFmt == kBf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[d]);
    if (kFmt == kF16) return __half2float(reinterpret_cast<const __half*>(row)[d]);
    if (kFmt == kE5m2) return __half2float(__ushort_as_half((unsigned short)(row[d] << 8)));
    uint32_t w[4];
    if (kFmt == kInt8) w[0] = int8_pair<kInt8_01>(int8_bias(row[d]));
    else e2m1_pairs(w, row[d / 2]);
    const uint32_t f = pack2<true>(block_scale(exps[d / (D / 4)]), 0.0f);
    const float2 v = unpack2<true>(mul_half2(kFmt == kE2m1 && (d & 1) ? w[0] >> 16 : w[0], f));
    return v.x;
}

}  // namespace splitzip
