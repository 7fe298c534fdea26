// norm_rope.cu -- per-head RMS norm of queries and keys, the position rotation
// and the store into the cache, in one pass (sm_103a).
//
// For a row x of head_dim values: y = x * rsqrt(sum(x^2) / head_dim + eps) * w,
// then pairs (a, b) of its first rot_dim values become (a c - b s, b c + a s).
// Every input is read once and every output written once, so HBM bounds it: at
// 16384 tokens of 32 + 8 + 8 heads of 128, 411 MB.
//
// A row is shared by a few lanes, each holding two runs of kRun values (one load
// and one store each, adjacent lanes adjacent runs).  Which two runs is chosen
// so that the rotation needs no other lane: for pairs (i, i + R/2) run u goes
// with run u + R / (2 kRun), and interleaved pairs lie inside a run.  The sum of
// squares is the only exchange between lanes.  A group of lanes takes kRows
// heads of one kind (queries, keys or values) of one token, so addresses,
// weights and the token's table row are found once for them.  Runs of eight
// (16-byte loads) leave half as many instructions, which limited runs of four:
// 16384 tokens of 48 heads of 128 take 74-75 us (5.5 TB/s, 81% of a copy's rate)
// against 88, and 76 into an E5M2 cache; runs of four remain for a rot_dim that is
// not a multiple of sixteen.  With two and four rows into BF16 caches the compiler
// spills 20 and 44 bytes a thread; one CTA less to an SM spills nothing and is slower
// (the 16384 tokens 75 us where this takes 69, with their cache in one piece).
#include <cstdint>

#include <cuda_bf16.h>

#include "attention.cuh"
#include "common.cuh"
#include "lane_groups.h"
#include "serving.h"

namespace splitzip {
namespace {

// A run of values as it lies in memory (8 or 16 bytes of BF16).
template <int kRun>
struct Run {
    uint32_t w[kRun / 2];
};
template <int kRun>
__device__ __forceinline__ Run<kRun> load_run(const void* p) {
    Run<kRun> r;
    if constexpr (kRun == 8) {
        const uint4 v = ld_stream16(p);
        r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
    } else {
        const uint2 v = ld_stream8(p);
        r.w[0] = v.x, r.w[1] = v.y;
    }
    return r;
}
template <int kRun>
__device__ __forceinline__ void store_run(void* p, const Run<kRun>& r) {
    if constexpr (kRun == 8) st_stream16(p, make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]));
    else st_stream8(p, make_uint2(r.w[0], r.w[1]));
}
template <int kRun>
__device__ __forceinline__ void unpack(const Run<kRun>& r, float (&f)[kRun]) {
#pragma unroll
    for (int i = 0; i < kRun / 2; i++) {
        f[2 * i] = __uint_as_float(r.w[i] << 16);
        f[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
}
template <int kRun>
__device__ __forceinline__ Run<kRun> pack_bf16(const float (&f)[kRun]) {
    Run<kRun> r;
#pragma unroll
    for (int i = 0; i < kRun / 2; i++) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        r.w[i] = *reinterpret_cast<const uint32_t*>(&a);
    }
    return r;
}
// Four E5M2 bytes, to nearest even.  The conversion instruction saturates; a
// value of at least 61440, half way from the largest finite value (57344) to
// the next step (65536), rounds to infinity instead.  NaN stays NaN.
__device__ __forceinline__ uint32_t pack4_e5m2(const float* f) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
    uint32_t w = (uint32_t)lo | ((uint32_t)hi << 16);
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (fabsf(f[i]) >= 61440.0f) w = (w & ~(0x7Fu << (8 * i))) | (0x7Cu << (8 * i));
    return w;
}
template <int kRun>
__device__ __forceinline__ void store_e5m2(uint8_t* p, const float (&f)[kRun]) {
    if constexpr (kRun == 8) st_stream8(p, make_uint2(pack4_e5m2(f), pack4_e5m2(f + 4)));
    else st_stream4(p, pack4_e5m2(f));
}

constexpr int kThreadsRope = 128;

struct NormRopeParams {
    splitzip_norm_rope_args a;
    uint32_t q_parts, kv_parts, parts;  // groups of kRows heads: of the queries, of keys or values, of a token
    uint32_t items;                     // n * parts
};

template <int D, int kRun, int kRows, bool kF8>
__global__ void __launch_bounds__(kThreadsRope, kRun == 8 && kRows == 4 ? 5 : 6) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr uint32_t kLanes = D / (2 * kRun);
    const splitzip_norm_rope_args& a = p.a;
    const uint32_t lane = threadIdx.x % kLanes;
    const uint32_t item = lane_group(blockIdx.x, threadIdx.x, kThreadsRope, kLanes);
    if (__all_sync(0xFFFFFFFFu, item >= p.items)) return;
    const bool active = item < p.items;
    const uint32_t tok = active ? item / p.parts : 0, part = active ? item - tok * p.parts : 0;
    const bool q = part < p.q_parts, k = !q && part < p.q_parts + p.kv_parts;
    const splitzip_view& in = q ? a.q : k ? a.k : a.v;
    const uint32_t h0 = (q ? part : k ? part - p.q_parts : part - p.q_parts - p.kv_parts) * kRows;
    const uint32_t rows = active ? min((uint32_t)kRows, (q ? a.q_heads : a.kv_heads) - h0) : 0;

    // This lane's two runs.
    const uint32_t turned = a.rot_dim / (2 * kRun);  // lanes whose runs are rotated
    const bool turns = lane < turned && (q || k);
    const uint32_t u0 = kRun * (lane < turned ? lane : a.rot_dim / kRun + (lane - turned));
    const uint32_t u1 = lane < turned ? u0 + a.rot_dim / 2 : u0 + (D - a.rot_dim) / 2;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(in.data) + (int64_t)tok * in.stride_t + h0 * in.stride_h;
    Run<kRun> x[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        if (r < (int)rows) {
            x[r][0] = load_run<kRun>(src + r * in.stride_h + u0);
            x[r][1] = load_run<kRun>(src + r * in.stride_h + u1);
        } else {
#pragma unroll
            for (int i = 0; i < kRun / 2; i++) x[r][0].w[i] = x[r][1].w[i] = 0;
        }
    }
    int64_t slot = -1;
    if (active && !q) slot = a.slots[tok];
    // The factors of kRun pairs: of the first run's values with the second's, or,
    // interleaved, half of them in each run.
    alignas(16) float c[kRun], s[kRun];
    if (turns && active) {
        const int32_t pos = a.positions[tok];
        if (pos >= 0 && (uint64_t)pos < a.table_rows) {
            const float* t = a.table + (uint64_t)pos * a.rot_dim;
            const uint32_t f0 = a.interleaved ? u0 / 2 : u0, f1 = a.interleaved ? u1 / 2 : u0 + kRun / 2;
            const float* at[4] = {t + f0, t + f1, t + a.rot_dim / 2 + f0, t + a.rot_dim / 2 + f1};
#pragma unroll
            for (int x = 0; x < 4; x++) {
                float* to = (x < 2 ? c : s) + (x & 1) * (kRun / 2);
                if constexpr (kRun == 8) *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(at[x]);
                else *reinterpret_cast<float2*>(to) = *reinterpret_cast<const float2*>(at[x]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kRun; i++) c[i] = s[i] = __int_as_float(0x7FC00000);
        }
    }
    const void* weight = q ? a.q_weight : k ? a.k_weight : nullptr;
    Run<kRun> w0, w1;
    if (weight) {
        w0 = load_run<kRun>(static_cast<const __nv_bfloat16*>(weight) + u0);
        w1 = load_run<kRun>(static_cast<const __nv_bfloat16*>(weight) + u1);
    }
    const splitzip_view& cache = k ? a.k_cache : a.v_cache;
    // A row between two sequences of the cache is someone else's memory.
    const bool store = !q && slot >= 0 && (uint64_t)slot < a.cache_rows &&
                       (!a.cache_step || (uint32_t)slot % a.cache_step < a.cache_tokens);
    const int64_t at = q ? (int64_t)tok * a.q_out.stride_t + h0 * a.q_out.stride_h : slot * cache.stride_t + h0 * cache.stride_h;
    const int64_t step = q ? a.q_out.stride_h : cache.stride_h;
    uint8_t* dst = static_cast<uint8_t*>(q ? a.q_out.data : cache.data) + at * (q || !kF8 ? 2 : 1);
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        float y[2][kRun];
        unpack<kRun>(x[r][0], y[0]);
        unpack<kRun>(x[r][1], y[1]);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kRun; i++) sum = fmaf(y[0][i], y[0][i], fmaf(y[1][i], y[1][i], sum));
#pragma unroll
        for (uint32_t d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (q || k) {
            const float norm = rsqrtf(sum * (1.0f / D) + a.eps);
            if (weight) {
                float f[2][kRun];
                unpack<kRun>(w0, f[0]);
                unpack<kRun>(w1, f[1]);
#pragma unroll
                for (int i = 0; i < kRun; i++) y[0][i] *= norm * f[0][i], y[1][i] *= norm * f[1][i];
            } else {
#pragma unroll
                for (int i = 0; i < kRun; i++) y[0][i] *= norm, y[1][i] *= norm;
            }
            if (turns && a.interleaved) {
#pragma unroll
                for (int i = 0; i < kRun; i++) {
                    float &u = y[2 * i / kRun][2 * i % kRun], &v = y[2 * i / kRun][2 * i % kRun + 1];
                    const float uu = u * c[i] - v * s[i];
                    v = v * c[i] + u * s[i];
                    u = uu;
                }
            } else if (turns) {
#pragma unroll
                for (int i = 0; i < kRun; i++) {
                    const float u = y[0][i], v = y[1][i];
                    y[0][i] = u * c[i] - v * s[i];
                    y[1][i] = v * c[i] + u * s[i];
                }
            }
        }
        if (r >= (int)rows || !(q || store)) continue;
        if (q || !kF8) {
            __nv_bfloat16* row = reinterpret_cast<__nv_bfloat16*>(dst) + r * step;
            store_run<kRun>(row + u0, q || k ? pack_bf16<kRun>(y[0]) : x[r][0]);
            store_run<kRun>(row + u1, q || k ? pack_bf16<kRun>(y[1]) : x[r][1]);
        } else {
            store_e5m2<kRun>(dst + r * step + u0, y[0]);
            store_e5m2<kRun>(dst + r * step + u1, y[1]);
        }
    }
}

template <int D, int kRun, int kRows, bool kF8>
cudaError_t launch(NormRopeParams& p, cudaStream_t s) {
    p.q_parts = (p.a.q_heads + kRows - 1) / kRows;
    p.kv_parts = (p.a.kv_heads + kRows - 1) / kRows;
    p.parts = p.q_parts + 2 * p.kv_parts;
    p.items = p.a.n * p.parts;
    const uint64_t threads = (uint64_t)p.items * (D / (2 * kRun));
    norm_rope_kernel<D, kRun, kRows, kF8><<<(unsigned)((threads + kThreadsRope - 1) / kThreadsRope), kThreadsRope, 0, s>>>(p);
    return cudaGetLastError();
}

template <int D, bool kF8>
cudaError_t launch_dim(NormRopeParams& p, cudaStream_t s) {
    // Runs of eight where the rotated values are whole pairs of them.
    const bool eight = p.a.rot_dim % 16 == 0;
    // One row per group of lanes where the rows do not fill the GPU anyway (fewer than 8
    // warps' worth per SM), two (or four of half the lanes' size) where they do, and four
    // where they fill it many times: 48 heads of 128 of 16384 tokens take 70 us with four
    // and 74 with two, of 1024 tokens 7.3 and 6.4.
    const uint64_t rows = (uint64_t)p.a.n * (p.a.q_heads + 2 * p.a.kv_heads), lanes = rows * (D / 16);
    const bool few = lanes < kSms * 256, many = lanes >= kSms * 256 * 16;
    if (eight) return few ? launch<D, 8, 1, kF8>(p, s) : many ? launch<D, 8, 4, kF8>(p, s) : launch<D, 8, 2, kF8>(p, s);
    return few ? launch<D, 4, 1, kF8>(p, s) : launch<D, 4, 4, kF8>(p, s);
}

}  // namespace

cudaError_t launch_norm_rope(const splitzip_norm_rope_args& a, cudaStream_t s) {
    NormRopeParams p;
    p.a = a;
    const bool f8 = a.cache_format == SPLITZIP_FORMAT_E5M2;
    if (a.head_dim == 64) return f8 ? launch_dim<64, true>(p, s) : launch_dim<64, false>(p, s);
    return f8 ? launch_dim<128, true>(p, s) : launch_dim<128, false>(p, s);
}

}  // namespace splitzip
