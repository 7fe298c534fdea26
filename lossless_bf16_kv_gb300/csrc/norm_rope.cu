// norm_rope.cu -- per-head RMS norm of queries and keys, the position rotation
// and the store into the cache, in one pass (sm_103a).
//
// For a row x of head_dim values: y = x * rsqrt(sum(x^2) / head_dim + eps) * w,
// then pairs (a, b) of its first rot_dim values become (a c - b s, b c + a s).
// Every input is read once and every output written once, so HBM bounds it: at
// 16384 tokens of 32 + 8 + 8 heads of 128, 411 MB.
//
// A row is shared by head_dim / 8 lanes, each holding two runs of four values
// (8-byte loads and stores, adjacent lanes adjacent runs).  Which two runs is
// chosen so that the rotation needs no other lane: for pairs (i, i + R/2) run
// u goes with run u + R/8, and interleaved pairs lie inside a run.  The sum of
// squares is the only exchange between lanes.  A group of lanes takes kRows
// heads of one token, loaded before the first is used, so the token's table
// row is read once for them and enough bytes are in flight.
#include <cstdint>

#include <cuda_bf16.h>

#include "common.cuh"
#include "serving.h"

namespace splitzip {
namespace {

__device__ __forceinline__ void unpack4(uint2 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xFFFF0000u);
}
__device__ __forceinline__ uint2 pack4_bf16(const float (&f)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
// Four E5M2 bytes, to nearest even.  The conversion instruction saturates; a
// value of at least 61440, half way from the largest finite value (57344) to
// the next step (65536), rounds to infinity instead.  NaN stays NaN.
__device__ __forceinline__ uint32_t pack4_e5m2(const float (&f)[4]) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
    uint32_t w = (uint32_t)lo | ((uint32_t)hi << 16);
#pragma unroll
    for (int i = 0; i < 4; i++)
        if (fabsf(f[i]) >= 61440.0f) w = (w & ~(0x7Fu << (8 * i))) | (0x7Cu << (8 * i));
    return w;
}

struct NormRopeParams {
    splitzip_norm_rope_args a;
    uint32_t heads;       // q_heads + 2 kv_heads
    uint32_t head_parts;  // ceil(heads / rows a group takes)
    uint32_t items;       // n * head_parts
};

template <int D, int kRows, bool kF8>
__global__ void __launch_bounds__(256) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int kLanes = D / 8;
    const splitzip_norm_rope_args& a = p.a;
    const uint32_t lane = threadIdx.x % kLanes;
    const uint32_t item = (blockIdx.x * blockDim.x + threadIdx.x) / kLanes;
    const bool active = item < p.items;
    const uint32_t tok = active ? item / p.head_parts : 0;
    const uint32_t h0 = active ? (item - tok * p.head_parts) * kRows : p.heads;

    // This lane's two runs of four values.
    const uint32_t turned = a.rot_dim / 8;  // lanes whose runs are rotated
    uint32_t u0, u1;
    if (lane < turned) {
        u0 = lane;
        u1 = lane + turned;
    } else {
        u0 = a.rot_dim / 4 + (lane - turned);
        u1 = u0 + (D - a.rot_dim) / 8;
    }
    uint2 x[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        const uint32_t h = h0 + r;
        if (h < p.heads) {
            const bool q = h < a.q_heads, k = h < a.q_heads + a.kv_heads;
            const splitzip_view& v = q ? a.q : k ? a.k : a.v;
            const uint32_t hh = q ? h : k ? h - a.q_heads : h - a.q_heads - a.kv_heads;
            const uint2* row = reinterpret_cast<const uint2*>(
                static_cast<const __nv_bfloat16*>(v.data) + (int64_t)tok * v.stride_t + hh * v.stride_h);
            x[r][0] = row[u0];
            x[r][1] = row[u1];
        } else {
            x[r][0] = x[r][1] = make_uint2(0, 0);
        }
    }
    float c[2][4], s[2][4];  // per run and value: its own factor, its partner's (sign included)
#pragma unroll
    for (int i = 0; i < 4; i++) c[0][i] = c[1][i] = 1.0f, s[0][i] = s[1][i] = 0.0f;
    int64_t slot = -1;
    if (active) {
        slot = a.slots[tok];
        if (lane < turned) {
            const int32_t pos = a.positions[tok];
            if (pos >= 0 && (uint64_t)pos < a.table_rows) {
                const float* t = a.table + (uint64_t)pos * a.rot_dim;
                if (a.interleaved) {
                    const float2 c0 = *reinterpret_cast<const float2*>(t + 2 * u0);
                    const float2 c1 = *reinterpret_cast<const float2*>(t + 2 * u1);
                    const float2 s0 = *reinterpret_cast<const float2*>(t + a.rot_dim / 2 + 2 * u0);
                    const float2 s1 = *reinterpret_cast<const float2*>(t + a.rot_dim / 2 + 2 * u1);
                    c[0][0] = c[0][1] = c0.x, c[0][2] = c[0][3] = c0.y;
                    c[1][0] = c[1][1] = c1.x, c[1][2] = c[1][3] = c1.y;
                    s[0][0] = -s0.x, s[0][1] = s0.x, s[0][2] = -s0.y, s[0][3] = s0.y;
                    s[1][0] = -s1.x, s[1][1] = s1.x, s[1][2] = -s1.y, s[1][3] = s1.y;
                } else {
                    const float4 cc = *reinterpret_cast<const float4*>(t + 4 * u0);
                    const float4 ss = *reinterpret_cast<const float4*>(t + a.rot_dim / 2 + 4 * u0);
                    c[0][0] = c[1][0] = cc.x, c[0][1] = c[1][1] = cc.y;
                    c[0][2] = c[1][2] = cc.z, c[0][3] = c[1][3] = cc.w;
                    s[0][0] = -ss.x, s[0][1] = -ss.y, s[0][2] = -ss.z, s[0][3] = -ss.w;
                    s[1][0] = ss.x, s[1][1] = ss.y, s[1][2] = ss.z, s[1][3] = ss.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) c[0][i] = c[1][i] = __int_as_float(0x7FC00000);
            }
        }
    }
    const bool store = slot >= 0 && (uint64_t)slot < a.cache_rows;
#pragma unroll
    for (int r = 0; r < kRows; r++) {
        const uint32_t h = h0 + r;
        float y[2][4];
        unpack4(x[r][0], y[0]);
        unpack4(x[r][1], y[1]);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; i++) sum = fmaf(y[0][i], y[0][i], fmaf(y[1][i], y[1][i], sum));
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        if (h >= p.heads) continue;
        const bool q = h < a.q_heads, k = h < a.q_heads + a.kv_heads;
        if (k) {  // a query or a key
            const float norm = rsqrtf(sum * (1.0f / D) + a.eps);
            const void* weight = q ? a.q_weight : a.k_weight;
            float w[2][4];
            if (weight) {
                unpack4(static_cast<const uint2*>(weight)[u0], w[0]);
                unpack4(static_cast<const uint2*>(weight)[u1], w[1]);
            }
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int i = 0; i < 4; i++) y[j][i] *= weight ? norm * w[j][i] : norm;
            if (lane < turned) {
                float z[2][4];
#pragma unroll
                for (int j = 0; j < 2; j++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        z[j][i] = y[j][i] * c[j][i] + (a.interleaved ? y[j][i ^ 1] : y[j ^ 1][i]) * s[j][i];
#pragma unroll
                for (int j = 0; j < 2; j++)
#pragma unroll
                    for (int i = 0; i < 4; i++) y[j][i] = z[j][i];
            }
        }
        if (q) {
            uint2* row = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.q_out.data) +
                                                  (int64_t)tok * a.q_out.stride_t + h * a.q_out.stride_h);
            row[u0] = pack4_bf16(y[0]);
            row[u1] = pack4_bf16(y[1]);
        } else if (store) {
            const splitzip_view& v = k ? a.k_cache : a.v_cache;
            const uint32_t hh = k ? h - a.q_heads : h - a.q_heads - a.kv_heads;
            const int64_t at = slot * v.stride_t + hh * v.stride_h;
            if (kF8) {
                uint32_t* row = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(v.data) + at);
                row[u0] = pack4_e5m2(y[0]);
                row[u1] = pack4_e5m2(y[1]);
            } else {
                uint2* row = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(v.data) + at);
                row[u0] = k ? pack4_bf16(y[0]) : x[r][0];
                row[u1] = k ? pack4_bf16(y[1]) : x[r][1];
            }
        }
    }
}

template <int D, int kRows, bool kF8>
cudaError_t launch(NormRopeParams& p, cudaStream_t s) {
    p.head_parts = (p.heads + kRows - 1) / kRows;
    p.items = p.a.n * p.head_parts;
    const uint64_t threads = (uint64_t)p.items * (D / 8);
    norm_rope_kernel<D, kRows, kF8><<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(p);
    return cudaGetLastError();
}

template <int D, bool kF8>
cudaError_t launch_dim(NormRopeParams& p, cudaStream_t s) {
    // One row per group of lanes where the rows do not fill the GPU anyway
    // (fewer than 8 warps' worth per SM), four where they do.
    const uint64_t rows = (uint64_t)p.a.n * p.heads;
    return rows * (D / 8) < 152ull * 256 ? launch<D, 1, kF8>(p, s) : launch<D, 4, kF8>(p, s);
}

}  // namespace

cudaError_t launch_norm_rope(const splitzip_norm_rope_args& a, cudaStream_t s) {
    NormRopeParams p;
    p.a = a;
    p.heads = a.q_heads + 2 * a.kv_heads;
    const bool f8 = a.cache_format == SPLITZIP_FORMAT_E5M2;
    if (a.head_dim == 64) return f8 ? launch_dim<64, true>(p, s) : launch_dim<64, false>(p, s);
    return f8 ? launch_dim<128, true>(p, s) : launch_dim<128, false>(p, s);
}

}  // namespace splitzip
