// attention_rows.cu -- attention of few query rows over a long cache (sm_103a).
//
// The query rows of one key/value head (query tokens times its group of query
// heads) are cut into tiles of 16 or 32 rows; a tile's slots are cut into
// splits, one CTA each, so that a single token still uses the whole GPU.  Each
// of a CTA's four warps walks its own slot tiles with its own running maximum
// m, sum l and output o:
//     s = q k^T, m' = max(m, s), p = exp(s - m'), l = l exp(m - m') + sum p,
//     o = o exp(m - m') + p v,
// and the partial (m, l, o) are joined by the same rule: over the warps in
// shared memory, over up to eight splits through the shared memory of their
// thread-block cluster, over more than that by the CTA that finishes last,
// always in the same order.  Every key and value is read once: HBM bounds it.
// A warp keeps a private ring of slot tiles filled by cp.async, so nothing in
// the loop waits for another warp.
//
// The products are mma.sync: with one token of a group of four to eight heads
// most rows of a 128-row tensor-memory tile would be padding, and at 16 rows the
// tensor units are 16% busy here.  16 sequences of 16384 tokens, 8 heads of 128
// for 32 query heads: 153 us in BF16 (7.0 TB/s, above a copy's 6.8: nothing is
// written), 87 us in E5M2 (6.2 TB/s, next to the widening).  One sequence: 16.8
// and 13.8 us, of which 5.6 are what a call of 128 slots takes, its chain of
// loads, products and joins.
#include <algorithm>
#include <cstdint>

#include "attention.cuh"

namespace splitzip {
namespace {

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

struct RowsParams {
    splitzip_attention_args a;
    uint32_t group, rows, row_tiles, splits, cluster;  // splits: a multiple of the cluster size
    uint32_t* counters;
    float* partials;
};

template <int D, bool kF8, int MT>
struct RowsShape {
    static constexpr int kElem = kF8 ? 1 : 2;
    static constexpr int kRow = D * kElem;             // bytes of a key
    static constexpr int kSlots = kTileBytes / kRow;   // slots per warp tile
    static constexpr int kTileRows = 16 * MT;
    static constexpr int kRing = kWarpsRows * kStagesRows * 2 * kTileBytes;
    static constexpr int kQ = kTileRows * D * 2;
    static constexpr int kSmem = kRing + kQ;
};

// Byte offset of 16-byte chunk c of row r in a tile of rows of kRow bytes; the
// chunks of eight consecutive rows at one c fall into eight different banks
// groups, as ldmatrix reads them.
template <int kRow>
__device__ __forceinline__ uint32_t chunk_at(uint32_t r, uint32_t c) {
    if (kRow >= 128) return r * kRow + ((c ^ (r & 7u)) << 4);
    return r * kRow + ((c ^ ((r >> 1) & 3u)) << 4);  // two rows to 128 bytes
}

__device__ __forceinline__ void add_scaled(float4& v, float f, float4 x) {
    v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
}

template <int D, bool kF8, int MT>
__global__ void __launch_bounds__(32 * kWarpsRows, MT == 1 ? kCtasPerSm : 1) rows_kernel(const __grid_constant__ RowsParams p) {
    using S = RowsShape<D, kF8, MT>;
    constexpr int NT = S::kSlots / 8;    // n-tiles of the scores
    constexpr int KS = D / 16;           // k-steps of the scores
    constexpr int PS = S::kSlots / 16;   // k-steps of the output
    constexpr int OT = D / 8;            // n-tiles of the output
    constexpr int kChunks = S::kRow / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_scale[S::kTileRows];
    __shared__ float s_m[kWarpsRows][S::kTileRows], s_l[kWarpsRows][S::kTileRows], s_mm[S::kTileRows], s_ll[S::kTileRows];
    __shared__ uint32_t s_last;
    const splitzip_attention_args& a = p.a;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t unit = blockIdx.x / p.splits;
    const uint32_t split = blockIdx.x - unit * p.splits;
    const uint32_t bh = unit / p.row_tiles, rt = unit - bh * p.row_tiles;
    const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
    const Mask mask(a, b);
    const uint32_t r0 = rt * S::kTileRows, r1 = min(r0 + S::kTileRows, p.rows);
    const int32_t p0 = mask.first + (int32_t)(r0 / p.group), p1 = mask.first + (int32_t)((r1 - 1) / p.group);
    const SlotTiles tiles(mask, p0, p1, S::kSlots);
    const uint32_t j0 = (uint32_t)((uint64_t)tiles.count * split / p.splits);
    const uint32_t j1 = (uint32_t)((uint64_t)tiles.count * (split + 1) / p.splits);

    uint8_t* ring = smem + warp * (kStagesRows * 2 * kTileBytes);
    uint8_t* qs = smem + S::kRing;
    const uint8_t* kbase = static_cast<const uint8_t*>(a.k.data) + (b * a.k.stride_b + h * a.k.stride_h) * S::kElem;
    const uint8_t* vbase = static_cast<const uint8_t*>(a.v.data) + (b * a.v.stride_b + h * a.v.stride_h) * S::kElem;
    // A lane copies one 16-byte chunk of every kStep-th row of a tile.  Slots past
    // the last one in use are loaded as copies of it and masked.
    constexpr int kStep = 32 / kChunks, kCopies = S::kSlots / kStep;
    const uint32_t lr = lane / kChunks, lc = lane % kChunks;
    const int64_t kstride = a.k.stride_t * S::kElem, vstride = a.v.stride_t * S::kElem;
    const uint8_t *klane = kbase + 16 * lc, *vlane = vbase + 16 * lc;
    auto load = [&](uint32_t j, uint32_t stage) {
        if (j < j1) {
            const int32_t s0 = (int32_t)(tiles.tile(j) * S::kSlots);
            uint8_t* dk = ring + stage * (2 * kTileBytes);
            if (s0 + S::kSlots <= mask.n) {
                const uint8_t *k = klane + (s0 + (int64_t)lr) * kstride, *v = vlane + (s0 + (int64_t)lr) * vstride;
#pragma unroll
                for (int i = 0; i < kCopies; i++) {
                    cp_async16(dk + chunk_at<S::kRow>(i * kStep + lr, lc), k);
                    cp_async16(dk + kTileBytes + chunk_at<S::kRow>(i * kStep + lr, lc), v);
                    k += kStep * kstride;
                    v += kStep * vstride;
                }
            } else {
                for (int i = 0; i < kCopies; i++) {
                    const uint32_t r = i * kStep + lr;
                    const int64_t slot = min(s0 + (int32_t)r, mask.n - 1);
                    cp_async16(dk + chunk_at<S::kRow>(r, lc), klane + slot * kstride);
                    cp_async16(dk + kTileBytes + chunk_at<S::kRow>(r, lc), vlane + slot * vstride);
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStagesRows - 1; i++) load(j0 + warp + i * kWarpsRows, i);

    // Queries: one warp per row, as FP16 of the scaled row for E5M2.
    for (uint32_t r = warp; r < S::kTileRows; r += kWarpsRows) {
        const uint32_t row = r0 + r, t = row / p.group, g = row - t * p.group;
        constexpr int V = D / 32;  // values per lane: 2 or 4
        uint32_t v[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; i++) v[i] = 0;
        if (row < r1) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                static_cast<const __nv_bfloat16*>(a.q.data) + b * a.q.stride_b + (int64_t)t * a.q.stride_t +
                (h * p.group + g) * a.q.stride_h);
#pragma unroll
            for (int i = 0; i < V / 2; i++) v[i] = src[lane * (V / 2) + i];
        }
        float power = 1.0f;
        if (kF8) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < V / 2; i++) top = max(top, max(v[i] & 0x7FFFu, v[i] >> 16 & 0x7FFFu));
            power = row_power(__reduce_max_sync(0xFFFFFFFFu, top));
        }
#pragma unroll
        for (int i = 0; i < V / 2; i++) {
            uint32_t d = lane * V + 2 * i, w = v[i];
            if (kF8) {
                w = pack2<true>(__uint_as_float(v[i] << 16) * power, __uint_as_float(v[i] & 0xFFFF0000u) * power);
                d = (d & ~15u) + e5m2_place(d & 15u);
            }
            *reinterpret_cast<uint32_t*>(qs + chunk_at<2 * D>(r, d / 8) + 2 * (d % 8)) = w;
        }
        if (lane == 0) s_scale[r] = a.scale * kLog2e / power;
    }
    __syncthreads();

    // This thread's rows: 16 i + lane / 4 and that + 8.
    int32_t pos[MT][2];
    float scale[MT][2], m[MT][2], l[MT][2], o[MT][OT][4];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const uint32_t r = 16 * i + 8 * x + lane / 4;
            pos[i][x] = r0 + r < r1 ? mask.pos((r0 + r) / p.group) : -1;
            scale[i][x] = s_scale[r];
            m[i][x] = -INFINITY;
            l[i][x] = 0.0f;
        }
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < OT; j++)
#pragma unroll
            for (int x = 0; x < 4; x++) o[i][j][x] = 0.0f;

    const uint32_t qaddr = smem_addr(qs);
    uint32_t qf[KS][4];  // one row tile: its query fragments stay in registers
    if (MT == 1)
#pragma unroll
        for (int k = 0; k < KS; k++) ldmatrix4(qf[k], qaddr + chunk_at<2 * D>(lane & 15, 2 * k + (lane >> 4)));
    bool odd = false;  // a value of a partly visible tile was infinite or NaN
    uint32_t stage = 0;
    for (uint32_t j = j0 + warp; j < j1; j += kWarpsRows) {
        cp_async_wait<kStagesRows - 2>();
        __syncwarp();
        load(j + (kStagesRows - 1) * kWarpsRows, stage == 0 ? kStagesRows - 1 : stage - 1);
        const uint32_t ks = smem_addr(ring + stage * (2 * kTileBytes)), vs = ks + kTileBytes;
        stage = stage == kStagesRows - 1 ? 0 : stage + 1;
        const int32_t s0 = (int32_t)(tiles.tile(j) * S::kSlots);
        const bool whole = p0 >= 0 && mask.all(p0, p1, s0, s0 + S::kSlots - 1);

        float sc[MT][NT][4];
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int x = 0; x < 4; x++) sc[i][n][x] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; k++) {
            uint32_t q[MT][4];
#pragma unroll
            for (int i = 0; i < MT; i++) {
                if (MT == 1)
#pragma unroll
                    for (int x = 0; x < 4; x++) q[i][x] = qf[k][x];
                else
                    ldmatrix4(q[i], qaddr + chunk_at<2 * D>(16 * i + (lane & 15), 2 * k + (lane >> 4)));
            }
            if (kF8) {
#pragma unroll
                for (int n = 0; n < NT; n += 4) {
                    uint32_t r[4];
                    ldmatrix4(r, ks + chunk_at<S::kRow>(8 * n + lane, k));
#pragma unroll
                    for (int x = 0; x < 4; x++)
#pragma unroll
                        for (int i = 0; i < MT; i++) mma16816<true>(sc[i][n + x], q[i], e5m2_01(r[x]), e5m2_23(r[x]));
                }
            } else {
#pragma unroll
                for (int n = 0; n < NT; n += 2) {
                    uint32_t r[4];
                    ldmatrix4(r, ks + chunk_at<S::kRow>(8 * n + 8 * (lane >> 4) + (lane & 7), 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                    for (int i = 0; i < MT; i++) {
                        mma16816<false>(sc[i][n], q[i], r[0], r[1]);
                        mma16816<false>(sc[i][n + 1], q[i], r[2], r[3]);
                    }
                }
            }
        }
        uint32_t pr[MT][PS][4];
#pragma unroll
        for (int i = 0; i < MT; i++) {
            float top[2] = {m[i][0] + kLift<kF8>, m[i][1] + kLift<kF8>};
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    float v = sc[i][n][x] * scale[i][x >> 1];
                    if (!whole && !mask.sees(pos[i][x >> 1], s0 + 8 * n + 2 * (int32_t)(lane & 3) + (x & 1))) v = -INFINITY;
                    sc[i][n][x] = v;
                    top[x >> 1] = fmaxf(top[x >> 1], v);
                }
#pragma unroll
            for (int x = 0; x < 2; x++) {
                top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], 1));
                top[x] = fmaxf(top[x], __shfl_xor_sync(0xFFFFFFFFu, top[x], 2));
            }
            top[0] -= kLift<kF8>, top[1] -= kLift<kF8>;
            const bool same = top[0] == m[i][0] && top[1] == m[i][1];
            const float use[2] = {top[0] == -INFINITY ? 0.0f : top[0], top[1] == -INFINITY ? 0.0f : top[1]};
            if (!__all_sync(0xFFFFFFFFu, same)) {
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const float f = exp2_approx(m[i][x] - use[x]);
                    l[i][x] *= f;
#pragma unroll
                    for (int n = 0; n < OT; n++) {
                        o[i][n][2 * x] *= f;
                        o[i][n][2 * x + 1] *= f;
                    }
                    m[i][x] = top[x];
                }
            }
#pragma unroll
            for (int n = 0; n < NT; n++) {
                float e[4];
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    e[x] = exp2_approx(sc[i][n][x] - use[x >> 1]);
                    l[i][x >> 1] += e[x];
                }
                // p in 16 bits for the product: a relative error of up to 2^-8 (BF16) or
                // 2^-11 (FP16, down to 2^-29 of the row's largest) of each term,
                // independent from term to term.
                pr[i][n >> 1][2 * (n & 1)] = pack2<kF8>(e[0], e[1]);
                pr[i][n >> 1][2 * (n & 1) + 1] = pack2<kF8>(e[2], e[3]);
            }
        }
#pragma unroll
        for (int k = 0; k < PS; k++) {
#pragma unroll
            for (int n = 0; n < OT; n += kF8 ? 4 : 2) {
                uint32_t r[4];
                ldmatrix4_trans(r, vs + chunk_at<S::kRow>(16 * k + 8 * ((lane >> 3) & 1) + (lane & 7),
                                                          n / 2 * S::kElem + (lane >> 4)));
                uint32_t v[kF8 ? 8 : 4];
                if (kF8) {
#pragma unroll
                    for (int x = 0; x < 4; x += 2) {
                        v[2 * x] = e5m2_02(r[x]);
                        v[2 * x + 1] = e5m2_02(r[x + 1]);
                        v[2 * x + 2] = e5m2_13(r[x]);
                        v[2 * x + 3] = e5m2_13(r[x + 1]);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 4; x++) v[x] = r[x];
                }
                if (!whole) {  // 0 x infinity is not 0: keep such values out of the product
#pragma unroll
                    for (int x = 0; x < (kF8 ? 8 : 4); x++) {
                        const uint32_t f = finite_or_zero<kF8>(v[x]);
                        odd |= f != v[x];
                        v[x] = f;
                    }
                }
#pragma unroll
                for (int x = 0; x < (kF8 ? 4 : 2); x++)
#pragma unroll
                    for (int i = 0; i < MT; i++) mma16816<kF8>(o[i][n + x], pr[i][k], v[2 * x], v[2 * x + 1]);
            }
        }
    }
    cp_async_wait<0>();
    // Column of o[..][n][x] in the head.
    auto column = [&](int n, int x) {
        return kF8 ? 16 * (n / 2) + 4 * (int)(lane & 3) + 2 * (x & 1) + (n & 1) : 8 * n + 2 * (int)(lane & 3) + (x & 1);
    };
    if (__any_sync(0xFFFFFFFFu, odd)) {
        // The infinite and NaN values of partly visible tiles go to the rows that
        // see them: whatever their (positive) weight, the sum takes their value.
        for (uint32_t j = j0 + warp; j < j1; j += kWarpsRows) {
            const int32_t s0 = (int32_t)(tiles.tile(j) * S::kSlots);
            if (p0 >= 0 && mask.all(p0, p1, s0, s0 + S::kSlots - 1)) continue;
            for (int32_t s = s0; s < min(s0 + S::kSlots, mask.n); s++)
#pragma unroll
                for (int n = 0; n < OT; n++)
#pragma unroll
                    for (int x = 0; x < 2; x++) {
                        const uint8_t* at = vbase + s * a.v.stride_t * S::kElem + column(n, x) * S::kElem;
                        const float v = kF8 ? __half2float(__ushort_as_half((unsigned short)(*at << 8)))
                                            : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(at));
                        if (isfinite(v)) continue;
#pragma unroll
                        for (int i = 0; i < MT; i++)
#pragma unroll
                            for (int y = 0; y < 2; y++)
                                if (mask.sees(pos[i][y], s)) o[i][n][2 * y + x] += v;
                    }
        }
    }

    // Join the warps: everything into shared memory (over the ring), then each
    // thread a share of the columns.
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int x = 0; x < 2; x++) {
            l[i][x] += __shfl_xor_sync(0xFFFFFFFFu, l[i][x], 1);
            l[i][x] += __shfl_xor_sync(0xFFFFFFFFu, l[i][x], 2);
            if ((lane & 3) == 0) {
                s_m[warp][16 * i + 8 * x + lane / 4] = m[i][x];
                s_l[warp][16 * i + 8 * x + lane / 4] = l[i][x];
            }
        }
    __syncthreads();  // every warp is done with its ring
    float* os = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int n = 0; n < OT; n++)
#pragma unroll
            for (int x = 0; x < 4; x++)
                os[(warp * S::kTileRows + 16 * i + 8 * (x >> 1) + lane / 4) * D + column(n, x)] = o[i][n][x];
    __syncthreads();

    const uint32_t nrows = r1 - r0;
    for (uint32_t at = tid; at < nrows * (D / 4); at += 32 * kWarpsRows) {
        const uint32_t r = at / (D / 4), c = 4 * (at % (D / 4));
        float mm = s_m[0][r];
#pragma unroll
        for (int w = 1; w < kWarpsRows; w++) mm = fmaxf(mm, s_m[w][r]);
        const float use = mm == -INFINITY ? 0.0f : mm;
        float ll = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarpsRows; w++) {
            const float f = exp2_approx(s_m[w][r] - use);
            ll = fmaf(f, s_l[w][r], ll);
            add_scaled(v, f, *reinterpret_cast<const float4*>(os + (w * S::kTileRows + r) * D + c));
        }
        *reinterpret_cast<float4*>(os + r * D + c) = v;  // over the first warp's, which only this thread reads
        if (c == 0) {
            s_mm[r] = mm;
            s_ll[r] = ll;
        }
    }

    // Join the cluster: each of its CTAs a share of the outputs.
    const uint32_t cluster = p.cluster, rank = split % cluster, groups = p.splits / cluster;
    if (cluster > 1) cluster_sync();
    else __syncthreads();
    auto store = [&](uint32_t r, uint32_t c, float4 v, float mm, float ll) {
        const uint32_t row = r0 + r, t = row / p.group, g = row - t * p.group;
        const uint32_t hq = h * p.group + g;
        const bool none = ll == 0.0f;  // nothing seen, or scores of -infinity alone
        const float inv = 1.0f / ll;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + b * a.out.stride_b + (int64_t)t * a.out.stride_t +
                             hq * a.out.stride_h;
        *reinterpret_cast<uint2*>(out + c) =
            none ? make_uint2(0, 0) : make_uint2(pack2<false>(v.x * inv, v.y * inv), pack2<false>(v.z * inv, v.w * inv));
        if (c == 0 && a.lse)
            a.lse[((uint64_t)b * a.q_heads + hq) * a.q_tokens + t] = none ? -INFINITY : (mm + log2f(ll)) * kLn2;
    };
    constexpr uint32_t kPart = S::kTileRows * (D + 4);  // floats of a partial result: rows of o, m, l
    const uint32_t group = split / cluster;
    float* all = p.partials + (uint64_t)unit * groups * kPart;
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
                m8[i] = cluster_ld(smem_addr(&s_mm[r]), i);
                l8[i] = cluster_ld(smem_addr(&s_ll[r]), i);
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
    if (tid == 0) {
        s_last = atomicAdd(p.counters + unit, 1u) == p.splits - 1;
        if (s_last) p.counters[unit] = 0;  // ready for the next call
    }
    __syncthreads();
    if (!s_last) return;
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

template <int D, bool kF8, int MT>
cudaError_t launch(const RowsParams& p, uint32_t ctas, cudaStream_t s) {
    using S = RowsShape<D, kF8, MT>;
    Wave w;
    const cudaError_t e = launch_wave<rows_kernel<D, kF8, MT>>(32 * kWarpsRows, S::kSmem, w);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * kWarpsRows);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rows_kernel<D, kF8, MT>, p);
}

template <int D, bool kF8>
cudaError_t launch_tile(const RowsParams& p, uint32_t tile_rows, uint32_t ctas, cudaStream_t s) {
    return tile_rows == 16 ? launch<D, kF8, 1>(p, ctas, s) : launch<D, kF8, 2>(p, ctas, s);
}

}  // namespace

bool attention_rows_plan(const splitzip_attention_args& a, AttentionPlan& p) {
    const uint32_t group = a.q_heads / a.kv_heads;
    p.rows = a.q_tokens * group;
    p.tile_rows = p.rows <= 16 ? 16 : 32;
    p.row_tiles = (p.rows + p.tile_rows - 1) / p.tile_rows;
    const uint64_t units = (uint64_t)a.batch * a.kv_heads * p.row_tiles;
    const uint32_t slots = kTileBytes / (a.head_dim * (a.cache_format == SPLITZIP_FORMAT_E5M2 ? 1 : 2));
    // The slots a row tile can see at most.
    uint64_t most = a.kv_tokens;
    if (a.window) most = std::min(most, (uint64_t)a.window + a.sinks + (p.tile_rows + group - 1) / group + 2 * slots);
    // As many splits as run at once, of which each warp has a tile of slots (512 slots of
    // 8 units: 5.8 us with 8 splits, 6.6 with 4).  Three 16-row CTAs fit an SM, but a
    // cluster lies within one of the GPU's groups of SMs, and fewer of the large ones run
    // at once (as cudaOccupancyMaxActiveClusters has it): 64 units of 8192 slots take 44 us
    // in 6 splits, 59 in 7, 50 in 3; 128 units of 16384 slots 154 in 3, 191 in 4, 158 in 6.
    // Of 32-row CTAs two fit, and 256 are few enough for all sizes: 128 units of 16384
    // slots take 175 us in 2 splits and 243 in 3.
    static constexpr uint64_t kAtOnce[9] = {0, 3 * kSms, 228, 148, 110, 87, 74, 59, 51};
    const uint64_t tiles = (most + kWarpsRows * slots - 1) / (kWarpsRows * slots);
    uint64_t splits = 8;
    while (splits > 1 && (splits > tiles || units > (p.tile_rows == 16 ? kAtOnce[splits] : 256 / splits))) splits--;
    // Up to eight splits are one cluster.  More are clusters of eight, of which the last
    // one joins all: that costs as much as a few tiles, more with more to join.  8 units,
    // 16-row tiles: 4096 slots of 64 take 7.5 us with 8 splits and 8.6 with 32, 8192 of
    // 128 16.6 and 12.2 (13.0 with 40); 32-row tiles: 4096 of 128 18.2 and 22.3, 12000
    // 33.9 and 27.7; 131072 slots of 128 take 88 us with 32 splits, 115 with 56.
    const uint64_t more = std::min(256 / units, tiles) / 8 * 8, join = p.tile_rows * a.head_dim > 2048 ? 10 : 4;
    if (more > 8 && tiles / more + join < tiles / 8) splits = more;
    p.splits = (uint32_t)splits;
    if (units * p.splits > 0x7FFFFFFFull) return false;
    static_assert(4 * kSms <= kAttentionStatus, "splits in several clusters are counted by row tile");
    p.bytes = kAttentionHeader + (p.splits > 8 ? units * (p.splits / 8) * p.tile_rows * (a.head_dim + 4) * 4 : 0);
    return true;
}

cudaError_t launch_attention_rows(const splitzip_attention_args& a, const AttentionPlan& plan, void* workspace,
                             cudaStream_t s) {
    RowsParams p;
    p.a = a;
    p.group = a.q_heads / a.kv_heads;
    p.rows = plan.rows;
    p.row_tiles = plan.row_tiles;
    p.splits = plan.splits;
    p.cluster = std::min(plan.splits, 8u);
    p.counters = reinterpret_cast<uint32_t*>(workspace);
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kAttentionHeader);
    const uint32_t ctas = a.batch * a.kv_heads * plan.row_tiles * plan.splits;
    const bool f8 = a.cache_format == SPLITZIP_FORMAT_E5M2;
    if (a.head_dim == 64)
        return f8 ? launch_tile<64, true>(p, plan.tile_rows, ctas, s) : launch_tile<64, false>(p, plan.tile_rows, ctas, s);
    return f8 ? launch_tile<128, true>(p, plan.tile_rows, ctas, s) : launch_tile<128, false>(p, plan.tile_rows, ctas, s);
}

}  // namespace splitzip
