// attention_rows.cuh -- what the attention kernels of few query rows share (sm_103a):
// tiles of slots in shared memory, and the joining of warps, of a cluster's
// splits, and of clusters.
#pragma once

#include <cstdint>

#include "attention.cuh"

namespace splitzip {

constexpr int kWarpsRows = 4;
constexpr int kStagesRows = 2;
constexpr uint32_t kCtasPerSm = 3;  // of 16-row tiles, by registers and shared memory
constexpr int kTileBytes = 4096;  // of keys, and of values, per warp and stage
// log2 of p at a row's maximum: m is that much less than the maximum.  FP16 holds p in
// full from 2^-14 to 2^16, so with 2^15 on top terms down to 2^-29 of a row's largest
// keep all bits and those below 2^-40 vanish.  With 1 on top those below 2^-25 do,
// and 2^17 slots of them are 2^-8 of the sum.
template <bool kF8>
constexpr float kLift = kF8 ? 15.0f : 0.0f;

__device__ __forceinline__ void add_scaled(float4& v, float f, float4 x) {
    v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
}

// The warps' maxima and sums of a CTA's rows, and those of all its warps.
template <int kTileRows>
struct RowsShared {
    float m[kWarpsRows][kTileRows], l[kWarpsRows][kTileRows], mm[kTileRows], ll[kTileRows];
    uint32_t last;
};

// Floats of a partial result in memory: rows of o, m and l.
template <int D, int kTileRows>
constexpr uint32_t kPartFloats = kTileRows * (D + 4);

// Joins the partial results of one row tile: of this CTA's warps (rows of D values
// in `os`, warp by warp, with their m and l in sh), then of the splits of its
// cluster, then, where there are more clusters (splits / cluster), through the row
// tile's `partials`: is_last() counts this CTA (one thread calls it) and says whether
// it is the last one.  store(r, c, o, m, l) takes four columns of a row of the tile
// once they are complete.  All threads of the CTA, and of the cluster, call it.
template <int D, int kTileRows, class Last, class Store>
__device__ __forceinline__ void join_rows(float* os, RowsShared<kTileRows>& sh, uint32_t split, uint32_t splits, uint32_t cluster,
                                          uint32_t nrows, float* all, const Last& is_last, const Store& store) {
    const uint32_t tid = threadIdx.x;
    for (uint32_t at = tid; at < nrows * (D / 4); at += 32 * kWarpsRows) {
        const uint32_t r = at / (D / 4), c = 4 * (at % (D / 4));
        float mm = sh.m[0][r];
#pragma unroll
        for (int w = 1; w < kWarpsRows; w++) mm = fmaxf(mm, sh.m[w][r]);
        const float use = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarpsRows; w++) {
            const float f = exp2_approx(sh.m[w][r] - use);
            ll = fmaf(f, sh.l[w][r], ll);
            add_scaled(v, f, *reinterpret_cast<const float4*>(os + (w * kTileRows + r) * D + c));
        }
        *reinterpret_cast<float4*>(os + r * D + c) = v;  // over the first warp's, which only this thread reads
        if (c == 0) {
            sh.mm[r] = mm;
            sh.ll[r] = ll;
        }
    }

    // Join the cluster: each of its CTAs a share of the outputs.
    const uint32_t rank = split % cluster, groups = splits / cluster;
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    constexpr uint32_t kPart = kPartFloats<D, kTileRows>;
    const uint32_t group = split / cluster;
    for (uint32_t at = rank * 32 * kWarpsRows + tid; at < nrows * (D / 4); at += cluster * 32 * kWarpsRows) {
        const uint32_t r = at / (D / 4), c = 4 * (at % (D / 4));
        float m8[8], l8[8];
        float4 v8[8];
#pragma unroll
        for (int i = 0; i < 8; i++) {
            m8[i] = -INFINITY;
            l8[i] = 0.0f;
            v8[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < (int)cluster) {
                m8[i] = cluster_ld(smem_addr(&sh.mm[r]), i);
                l8[i] = cluster_ld(smem_addr(&sh.ll[r]), i);
                v8[i] = cluster_ld4(smem_addr(os + r * D + c), i);
            }
        }
        float mm = m8[0];
#pragma unroll
        for (int i = 1; i < 8; i++) mm = fmaxf(mm, m8[i]);
        const float use = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float f = exp2_approx(m8[i] - use);
            ll = fmaf(f, l8[i], ll);
            add_scaled(v, f, v8[i]);
        }
        if (groups == 1) {
            store(r, c, v, mm, ll);
        } else {
            float* q = all + group * kPart + r * (D + 4);
            __stcg(reinterpret_cast<float4*>(q + c), v);
            if (c == 0) __stcg(reinterpret_cast<float2*>(q + D), make_float2(mm, ll));
        }
    }
    if (cluster > 1) cluster_sync();  // this CTA's shared memory has been read
    if (groups == 1) return;
    __threadfence();
    __syncthreads();
    if (tid == 0) sh.last = is_last();
    __syncthreads();
    if (!sh.last) return;
    __threadfence();
    for (uint32_t at = tid; at < nrows * (D / 4); at += 32 * kWarpsRows) {
        const uint32_t r = at / (D / 4), c = 4 * (at % (D / 4));
        const float* q = all + r * (D + 4);
        float mm = -INFINITY, ll = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (uint32_t i = 0; i < groups; i++) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(q + i * kPart + D));
            const float4 x = __ldcg(reinterpret_cast<const float4*>(q + i * kPart + c));
            const float top = fmaxf(mm, ml.x), use = top == -INFINITY ? 0.0f : top;
            const float f = exp2_approx(mm - use), g = exp2_approx(ml.x - use);
            ll = fmaf(f, ll, g * ml.y);
            v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
            add_scaled(v, g, x);
            mm = top;
        }
        store(r, c, v, mm, ll);
    }
}

// Splits of each row tile, of `units` row tiles that see up to `most` slots each; `ctas`
// of the kernel's fit an SM.
uint32_t attention_rows_splits(uint64_t units, uint64_t most, uint32_t slots, uint32_t tile_rows, uint32_t head_dim, uint32_t ctas = kCtasPerSm);
// Bytes of workspace that they need.
size_t attention_rows_bytes(uint64_t units, uint32_t splits, uint32_t tile_rows, uint32_t head_dim);

}  // namespace splitzip
