// attention.cuh -- what the attention kernels share (sm_103a): which slots a
// row of queries sees, warp-level matrix instructions and the E5M2 forms.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "serving.h"

namespace splitzip {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kSms = 152;  // of a GB300

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The visible slots of one sequence's queries.
struct Mask {
    int32_t n;         // slots in use
    int32_t first;     // position of query token 0 (may be negative)
    uint32_t window;   // at most 2^31: unlimited
    int32_t sinks;
    __device__ __forceinline__ Mask(const splitzip_attention_args& a, uint32_t b) {
        const int32_t len = a.lens ? a.lens[b] : (int32_t)a.kv_tokens;
        n = len < 0 ? 0 : min(len, (int32_t)a.kv_tokens);
        first = n - (int32_t)a.q_tokens;
        window = a.window ? min(a.window, 0x80000000u) : 0x80000000u;
        sinks = (int32_t)min(a.sinks, 0x7FFFFFFFu);
    }
    // Position of query token t; every negative one as -1.
    __device__ __forceinline__ int32_t pos(uint32_t t) const { return max(-1, first + (int32_t)t); }
    // p - s is taken modulo 2^32: for s > p it is at least 2^31.
    __device__ __forceinline__ bool sees(int32_t p, int32_t s) const {
        return (uint32_t)(p - s) < window || (s < sinks && s <= p);
    }
    // Whether every position in [p0, p1] (p0 >= 0) sees every slot in [s0, s1].
    __device__ __forceinline__ bool all(int32_t p0, int32_t p1, int32_t s0, int32_t s1) const {
        return s1 <= p0 && ((uint32_t)(p1 - s0) < window || s1 < sinks);
    }
};

// The tiles of `unit` slots that some position in [p0, p1] sees, numbered from
// 0: first those that hold sinks before the window, then those of the window.
struct SlotTiles {
    uint32_t head, from, count;
    __device__ __forceinline__ SlotTiles(const Mask& m, int32_t p0, int32_t p1, uint32_t unit) {
        head = from = count = 0;
        if (p1 < 0) return;  // else p1 < n
        const int64_t back = (int64_t)max(p0, 0) - (int64_t)m.window + 1;
        const uint32_t lo = back > 0 ? (uint32_t)back : 0u;
        from = lo / unit;
        const uint32_t sinks = (uint32_t)min(m.sinks, p1 + 1);
        head = min((sinks + unit - 1) / unit, from);
        count = head + (uint32_t)p1 / unit + 1 - from;
    }
    __device__ __forceinline__ uint32_t tile(uint32_t j) const { return j < head ? j : j - head + from; }
};

// ----------------------------------------------------- thread-block cluster

// All threads of the cluster; shared-memory writes before it are seen after it.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A 32-bit (4 x 32-bit) value at this CTA's shared address, of the cluster's CTA `rank`.
__device__ __forceinline__ float cluster_ld(uint32_t addr, uint32_t rank) {
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr, uint32_t rank) {
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(addr), "r"(rank)
        : "memory");
    return v;
}

// ------------------------------------------------- warp matrix products

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d += a (16 x 16) b (16 x 8), BF16 or FP16 operands, 32-bit sums.
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (kHalf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (kHalf) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool kHalf>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// --------------------------------------------------------- E5M2 operands
//
// An E5M2 value is the upper byte of the FP16 value it stands for, so E5M2
// keys and values enter FP16 matrix products exactly, by a byte permute.
// Queries are BF16: each row is scaled by a power of two that brings its
// largest magnitude into [1, 2), which FP16 then holds with all 8 significant
// bits down to 2^-17 of the largest; smaller ones are off by up to 2^-25 of it.  A
// score is then off by up to 2^-25 max|q| sum|k|.  Where the keys' channels are
// alike that is below the rounding of a 32-bit sum over the row; it is not where
// the row's small queries meet keys far larger than the others (E5M2 keys may:
// a query of 2^-20 of the largest enters with 5 bits).  The power goes back into
// the score's scale.

// Position in a 16-value run of the matrix product's contraction index of the
// run's value d, such that a lane's four consecutive bytes (4 q .. 4 q + 3)
// are the indices 2q, 2q+1, 2q+8, 2q+9 that the fragment layout gives it.
__device__ __forceinline__ uint32_t e5m2_place(uint32_t d) {
    return ((d & 12u) >> 1) + (d & 1u) + ((d & 2u) << 2);
}
__device__ __forceinline__ uint32_t e5m2_01(uint32_t r) { return prmt(r, 0u, 0x1404u); }  // bytes 0, 1
__device__ __forceinline__ uint32_t e5m2_23(uint32_t r) { return prmt(r, 0u, 0x3424u); }
__device__ __forceinline__ uint32_t e5m2_02(uint32_t r) { return prmt(r, 0u, 0x2404u); }
__device__ __forceinline__ uint32_t e5m2_13(uint32_t r) { return prmt(r, 0u, 0x3414u); }

// 2^-e for the largest magnitude's bits of a row of BF16 values (e its
// exponent; 2^-127 for a row with infinities or NaN); 1 for a row of zeros and
// values below 2^-126, whose scores with E5M2 keys are below 2^-100.
__device__ __forceinline__ float row_power(uint32_t max_bf16_bits) {
    const uint32_t e = max_bf16_bits >> 7;  // biased exponent
    if (e == 0u) return 1.0f;
    return e >= 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - e) << 23);
}

// Whether a packed pair of values holds an infinity or a NaN, and the pair
// with those replaced by zeros.
template <bool kHalf>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t v) {
    constexpr uint32_t kExp = kHalf ? 0x7C00u : 0x7F80u;
    if ((v & kExp) == kExp) v &= 0xFFFF0000u;
    if ((v >> 16 & kExp) == kExp) v &= 0x0000FFFFu;
    return v;
}

}  // namespace splitzip
