// attention_tiles.cu -- attention of many query rows on the tensor cores
// (sm_103a).
//
// A CTA takes two tiles of 128 query rows of one key/value head (128 / group
// tokens each, all heads of the group side by side, so a tile spans few
// positions and masks waste little) and walks the 128-slot tiles they see:
//     S = Q K^T, P = exp(S - m), O = O exp(m_old - m) + P V, l likewise.
// Both products are tcgen05.mma with accumulators in tensor memory: S of the
// two query tiles in columns 0..255, O in 256..511, P over S's columns, from
// where the second product takes it as its first operand.  The two tiles
// alternate: while one tile's warps do its softmax, the tensor cores run the
// other's O += P V and next S = Q K^T.  Per tile and step the two products take
// 2 x 512 cycles at head_dim 128, the 128 x 128 exponentials 512.
//
// Roles: warps 0-3 and 4-7 softmax (one thread per row, so row statistics need
// no exchange), 8 issues the products, 9 the TMA loads of a ring of key and
// value tiles, 10 and 11 keep infinities and NaN of partly visible tiles out of
// the second product (0 x infinity is not 0).
//
// The running maximum is only raised when a row's maximum grows by more than
// 2^8 (in which case O and l are rescaled by the softmax warps, after the
// product that wrote O): P stays below 2^8, and the quotient O / l is the same.
#include <algorithm>
#include <cstdint>

#include "attention.cuh"
#include "tcgen.cuh"
#include "tensor_map.h"

namespace splitzip {
namespace {

constexpr int kBN = 128;       // slots per step
constexpr int kTileM = 128;    // query rows per tile
constexpr int kThreadsTiles = 384;
constexpr float kLazy = 8.0f;  // log2 of how far P may exceed 1

template <int D>
struct TilesShape {
    static constexpr int kKV = kBN * D * 2;      // bytes of a key or value tile
    static constexpr int kQ = kTileM * D * 2;    // bytes of a query tile
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int kSmem = 2 * kQ + kStages * kKV + 1024;
};

struct TilesParams {
    splitzip_attention_args a;
    CUtensorMap qmap, kmap, vmap;
    uint32_t group, tokens;   // query tokens per tile: 128 / group
    uint32_t row_ctas, splits;
    uint32_t one_q, one_k, one_v;  // the batch is one sequence: coordinate 0
    uint32_t* counters;
    uint32_t* status;
    float* partials;
};

struct TilesBars {
    uint64_t full[8], empty[8], ok[8];  // ring stage: loaded, free again, values fit for the product
    uint64_t q_full;
    uint64_t s_full[2], p_full[2], o_full[2], drained;
    uint32_t tmem, err, odd, last;
};

// Bits of the slots s0 .. s0 + 31 that a query at `pos` sees.
__device__ __forceinline__ uint32_t seen_bits(const Mask& m, int32_t pos, int32_t s0) {
    const int32_t hi = min(pos - s0, 31);  // slots s0 + j with j <= hi, and
    if (hi < 0) return 0u;                 // j >= lo (window) or j <= sk (sinks)
    const uint32_t upto = 0xFFFFFFFFu >> (31 - hi);
    const int64_t lo = (int64_t)pos - (int64_t)m.window + 1 - s0;
    const uint32_t in_window = lo <= 0 ? 0xFFFFFFFFu : lo > 31 ? 0u : 0xFFFFFFFFu << (uint32_t)lo;
    const int32_t sk = min(m.sinks - 1 - s0, 31);
    const uint32_t sink = sk < 0 ? 0u : 0xFFFFFFFFu >> (31 - sk);
    return upto & (in_window | sink);
}

template <int D, bool kHalf>
__global__ void __launch_bounds__(kThreadsTiles, 1) tiles_kernel(const __grid_constant__ TilesParams p) {
    using S = TilesShape<D>;
    constexpr uint32_t kShapeS = mma_shape(kHalf, kBN, false), kShapeO = mma_shape(kHalf, D, true);
    constexpr uint32_t kColO = 256;
    extern __shared__ uint8_t smem_raw[];
    __shared__ TilesBars bars;
    uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* qs = smem;                 // two tiles, each D / 64 blocks of 128 rows of 128 bytes
    uint8_t* ring = smem + 2 * S::kQ;   // kStages tiles, each D / 64 blocks of 128 slots of 128 bytes
    const splitzip_attention_args& a = p.a;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // The last row tiles see the most slots: they go first.
    uint32_t unit = blockIdx.x / p.splits;
    const uint32_t split = blockIdx.x - unit * p.splits;
    const uint32_t rc = p.row_ctas - 1 - unit % p.row_ctas, bh = unit / p.row_ctas;
    const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
    const Mask mask(a, b);
    const uint32_t t0 = rc * 2 * p.tokens, t1 = min(t0 + 2 * p.tokens, a.q_tokens);
    const int32_t p0 = mask.first + (int32_t)t0, p1 = mask.first + (int32_t)t1 - 1;
    const SlotTiles tiles(mask, p0, p1, kBN);
    const uint32_t j0 = (uint32_t)((uint64_t)tiles.count * split / p.splits);
    const uint32_t steps = (uint32_t)((uint64_t)tiles.count * (split + 1) / p.splits) - j0;
    auto slot0 = [&](uint32_t i) { return (int32_t)(tiles.tile(j0 + i) * kBN); };
    auto whole_cta = [&](int32_t s0) { return p0 >= 0 && mask.all(p0, p1, s0, s0 + kBN - 1); };
    volatile uint32_t* err = &bars.err;

    if (warp == 8) tmem_alloc<512>(&bars.tmem);
    if (tid == 0) {
        for (int i = 0; i < S::kStages; i++) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        for (int i = 0; i < 8; i++) mbar_init(&bars.ok[i], 2);  // of step i mod 8: fewer are in the ring
        mbar_init(&bars.q_full, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 4);
            mbar_init(&bars.o_full[i], 1);
        }
        mbar_init(&bars.drained, 1);
        bars.err = bars.odd = 0;
        fence_mbar_init();
    }
    // Rows of a tile that hold no query (128 is not a multiple of every group).
    if (tid < 256) {
        const uint32_t r = tid & 127;
        if (r >= p.tokens * p.group)
#pragma unroll
            for (int i = 0; i < D / 64; i++)
#pragma unroll
                for (int c = 0; c < 8; c++)
                    *reinterpret_cast<uint4*>(qs + (tid >> 7) * S::kQ + i * (kTileM * 128) + r * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
        fence_async_proxy();
    }
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    const uint32_t tmem = bars.tmem;

    if (warp >= 8) {
        regs_dec<72>();
        if (warp == 9 && lane == 0 && steps) {  // TMA
            const uint32_t rows = p.tokens * p.group;
            mbar_arrive_expect_tx(&bars.q_full, 2 * rows * D * 2);
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int i = 0; i < D / 64; i++)
                    tma_load4(qs + t * S::kQ + i * (kTileM * 128), &p.qmap, 64 * i, (int32_t)(h * p.group),
                              (int32_t)(t0 + t * p.tokens), p.one_q ? 0 : (int32_t)b, &bars.q_full);
            uint32_t i = 0;
            for (uint32_t st = 0, ph = 0; i < 2 * steps; i++) {
                if (i >= S::kStages && !mbar_wait_bounded(&bars.empty[st], ph ^ 1, err)) break;
                const bool v = i & 1;
                mbar_arrive_expect_tx(&bars.full[st], S::kKV);
#pragma unroll
                for (int x = 0; x < D / 64; x++)
                    tma_load4(ring + st * S::kKV + x * (kBN * 128), v ? &p.vmap : &p.kmap, 64 * x, slot0(i >> 1),
                              (int32_t)h, (v ? p.one_v : p.one_k) ? 0 : (int32_t)b, &bars.full[st]);
                if (++st == S::kStages) st = 0, ph ^= 1;
            }
            // Every load has landed before this CTA may end, also where a wait gave up.
            uint32_t late = 0;
            mbar_wait_bounded(&bars.q_full, 0, &late);
            for (uint32_t x = i > S::kStages ? i - S::kStages : 0; x < i; x++)
                mbar_wait_bounded(&bars.full[x % S::kStages], (x / S::kStages) & 1, &late);
        } else if (warp == 8 && lane == 0 && steps) {  // matrix products
            const uint32_t qa = smem_addr(qs), ra = smem_addr(ring);
            auto issue_s = [&](uint32_t t, uint32_t st) {
#pragma unroll
                for (int k = 0; k < D / 16; k++) {
                    const uint32_t at = (k >> 2) * (kBN * 128) + (k & 3) * 32;
                    mma_ss(tmem + t * kBN, desc_rows(qa + t * S::kQ + at), desc_rows(ra + st * S::kKV + at), kShapeS, k > 0);
                }
                mma_commit(&bars.s_full[t]);
            };
            uint32_t st = 0, ph = 0;
            auto next = [&]() {
                if (++st == S::kStages) st = 0, ph ^= 1;
            };
            bool go = mbar_wait_bounded(&bars.q_full, 0, err) && mbar_wait_bounded(&bars.full[0], 0, err);
            if (go) {
                tcgen_fence_after();
                issue_s(0, 0);
                issue_s(1, 0);
                mma_commit(&bars.empty[0]);
                next();
            }
            for (uint32_t i = 0; go && i < steps; i++) {
                const uint32_t vst = st;
                if (!mbar_wait_bounded(&bars.ok[i & 7], (i >> 3) & 1, err) || !mbar_wait_bounded(&bars.full[st], ph, err)) break;
                next();
                const bool more = i + 1 < steps;
                for (uint32_t t = 0; t < 2; t++) {
                    if (!mbar_wait_bounded(&bars.p_full[t], i & 1, err)) {
                        go = false;
                        break;
                    }
                    tcgen_fence_after();
#pragma unroll
                    for (int k = 0; k < kBN / 16; k++)
                        mma_ts(tmem + kColO + t * D, tmem + t * kBN + 8 * k,
                               desc_columns(ra + vst * S::kKV + k * 2048, kBN * 128), kShapeO, i > 0 || k > 0);
                    if (!more) {
                        mma_commit(&bars.o_full[t]);
                    } else {
                        if (t == 0 && !mbar_wait_bounded(&bars.full[st], ph, err)) {
                            go = false;
                            break;
                        }
                        issue_s(t, st);
                    }
                }
                if (!go) break;
                mma_commit(&bars.empty[vst]);
                if (more) {
                    mma_commit(&bars.empty[st]);
                    next();
                }
            }
            uint32_t late = 0;
            mma_commit(&bars.drained);
            mbar_wait_bounded(&bars.drained, 0, &late);
        } else if (warp >= 10) {
            // Values of partly visible tiles: infinities and NaN become 0 here and are
            // added to the rows that see them at the end.
            for (uint32_t i = 0; i < steps; i++) {
                const uint32_t n = 2 * i + 1, st = n % S::kStages, ph = (n / S::kStages) & 1;
                if (!mbar_wait_bounded(&bars.full[st], ph, err)) break;
                if (!whole_cta(slot0(i))) {
                    bool found = false;
                    uint4* tile = reinterpret_cast<uint4*>(ring + st * S::kKV);
                    for (uint32_t x = tid - 320; x < S::kKV / 16; x += 64) {
                        uint4 v = tile[x];
                        const uint4 f = make_uint4(finite_or_zero<kHalf>(v.x), finite_or_zero<kHalf>(v.y), finite_or_zero<kHalf>(v.z),
                                                   finite_or_zero<kHalf>(v.w));
                        if (f.x != v.x || f.y != v.y || f.z != v.z || f.w != v.w) {
                            tile[x] = f;
                            found = true;
                        }
                    }
                    if (found) {
                        bars.odd = 1;
                        fence_async_proxy();
                    }
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&bars.ok[i & 7]);
            }
        }
    } else {
        regs_inc<216>();
        const uint32_t t = warp >> 2, r = tid & 127;
        const uint32_t tok = t0 + t * p.tokens + r / p.group, g = r % p.group;
        const bool valid = r < p.tokens * p.group && tok < a.q_tokens;
        const int32_t pos = valid ? mask.pos(tok) : -1;
        // Positions of this tile, for whole tiles of slots.
        const uint32_t ta = t0 + t * p.tokens, tb = min(ta + p.tokens, a.q_tokens);
        const int32_t q0 = mask.first + (int32_t)ta, q1 = mask.first + (int32_t)tb - 1;
        const float scale = a.scale * kLog2e;
        const uint32_t lanes = ((warp & 3) * 32) << 16;
        const uint32_t sa = tmem + lanes + t * kBN, oa = tmem + lanes + kColO + t * D;
        float m = -INFINITY, l = 0.0f;
        bool go = true;
        for (uint32_t i = 0; i < steps; i++) {
            if (!mbar_wait_bounded(&bars.s_full[t], i & 1, err)) {
                go = false;
                break;
            }
            tcgen_fence_after();
            uint32_t s[4][32];
#pragma unroll
            for (int c = 0; c < 4; c++) tmem_ld32(s[c], sa + 32 * c);
            tmem_wait_ld();
            const int32_t s0 = slot0(i);
            if (!(ta < a.q_tokens && q0 >= 0 && mask.all(q0, q1, s0, s0 + kBN - 1))) {
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const uint32_t seen = seen_bits(mask, pos, s0 + 32 * c);
#pragma unroll
                    for (int x = 0; x < 32; x++)
                        if (!(seen >> x & 1u)) s[c][x] = 0xFF800000u;
                }
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 4; c++)
#pragma unroll
                for (int x = 0; x < 32; x += 2)
                    top[(x >> 1) & 3] = fmaxf(fmaxf(top[(x >> 1) & 3], __uint_as_float(s[c][x])), __uint_as_float(s[c][x + 1]));
            const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
            const bool raise = now > m + kLazy;  // from -inf too
            if (__any_sync(0xFFFFFFFFu, raise)) {
                const float f = raise ? exp2_approx(m - now) : 1.0f;
                if (raise) m = now;
                l *= f;
                if (i) {
                    const uint64_t ff = pair(f, f);
#pragma unroll
                    for (int c = 0; c < D / 32; c++) {
                        uint32_t o[32];
                        tmem_ld32(o, oa + 32 * c);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; x += 2) {
                            float u, v;
                            unpair(mul2(pair(__uint_as_float(o[x]), __uint_as_float(o[x + 1])), ff), u, v);
                            o[x] = __float_as_uint(u);
                            o[x + 1] = __float_as_uint(v);
                        }
                        tmem_st32(oa + 32 * c, o);
                    }
                }
            }
            const float use = m == -INFINITY ? 0.0f : m;
            const uint64_t sc = pair(scale, scale), neg = pair(-use, -use);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 4; c += 2) {
                uint32_t w[32];
#pragma unroll
                for (int x = 0; x < 64; x += 2) {
                    const uint32_t(&sx)[32] = s[c + (x >> 5)];
                    float u, v;
                    unpair(fma2(pair(__uint_as_float(sx[x & 31]), __uint_as_float(sx[(x & 31) + 1])), sc, neg), u, v);
                    u = exp2_approx(u);
                    v = exp2_approx(v);
                    sum[(x >> 1) & 1] = add2(sum[(x >> 1) & 1], pair(u, v));
                    // P in 16 bits: an error of up to 2^-8 (BF16) or 2^-11 (FP16) of each term.
                    w[x >> 1] = pack2<kHalf>(u, v);
                }
                tmem_st32(sa + 16 * c, w);
            }
            float u, v, u2, v2;
            unpair(sum[0], u, v);
            unpair(sum[1], u2, v2);
            l += (u + v) + (u2 + v2);
            tmem_wait_st();
            tcgen_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.p_full[t]);
        }
        if (steps && go) go = mbar_wait_bounded(&bars.o_full[t], 0, err);
        tcgen_fence_after();
        __syncwarp();
        const bool sees = pos >= 0;
        const uint32_t hq = h * p.group + g;
        const bool alone = p.splits == 1;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + b * a.out.stride_b + (int64_t)tok * a.out.stride_t +
                             hq * a.out.stride_h;
        float* part = p.partials + ((uint64_t)blockIdx.x * 256 + t * 128 + r) * (D + 4);
        const bool odd = *reinterpret_cast<volatile uint32_t*>(&bars.odd);
        const uint8_t* vbase = static_cast<const uint8_t*>(a.v.data) + (b * a.v.stride_b + h * a.v.stride_h) * 2;
        const float inv = !go ? __int_as_float(0x7FC00000) : 1.0f / l;  // a wait that gave up: NaN
#pragma unroll 1
        for (int c = 0; c < D / 32; c++) {
            uint32_t o[32];
            __syncwarp();
            if (steps) {
                tmem_ld32(o, oa + 32 * c);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int x = 0; x < 32; x++) o[x] = 0;
            }
            if (odd) {
                for (uint32_t i = 0; i < steps; i++) {
                    const int32_t s0 = slot0(i);
                    if (whole_cta(s0)) continue;
                    for (int32_t s = s0; s < min(s0 + kBN, mask.n); s++) {
                        if (!mask.sees(pos, s)) continue;
                        const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(vbase + s * a.v.stride_t * 2) + 32 * c;
#pragma unroll
                        for (int x = 0; x < 32; x++) {
                            const float v = __bfloat162float(row[x]);
                            if (!isfinite(v)) o[x] = __float_as_uint(__uint_as_float(o[x]) + v);
                        }
                    }
                }
            }
            if (valid && alone) {
#pragma unroll
                for (int x = 0; x < 32; x += 8) {
                    uint4 w;
                    uint32_t* ww = &w.x;
#pragma unroll
                    for (int y = 0; y < 4; y++)
                        ww[y] = sees ? pack2<false>(__uint_as_float(o[x + 2 * y]) * inv, __uint_as_float(o[x + 2 * y + 1]) * inv) : 0u;
                    *reinterpret_cast<uint4*>(out + 32 * c + x) = w;
                }
            } else if (valid) {
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                    __stcg(reinterpret_cast<float4*>(part + 32 * c + x),
                           make_float4(__uint_as_float(o[x]), __uint_as_float(o[x + 1]), __uint_as_float(o[x + 2]),
                                       __uint_as_float(o[x + 3])));
            }
        }
        if (valid) {
            if (!go) l = __int_as_float(0x7FC00000);
            if (!alone)
                __stcg(reinterpret_cast<float4*>(part + D), make_float4(m, l, 0.0f, 0.0f));
            else if (a.lse)
                a.lse[((uint64_t)b * a.q_heads + hq) * a.q_tokens + tok] = sees ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
        tcgen_fence_before();
        if (tid == 0 && !go) atomicOr(p.status, kStatusTimeout);
        if (p.splits > 1) {
            // Join the splits: the CTA that comes last, in the order of the splits.
            __threadfence();
            named_sync(1, 256);
            if (tid == 0) {
                bars.last = atomicAdd(p.counters + unit, 1u) == p.splits - 1;
                if (bars.last) p.counters[unit] = 0;  // ready for the next call
            }
            named_sync(1, 256);
            if (bars.last) {
                __threadfence();
            constexpr uint32_t kLanes = D / 4;  // threads to a row
            const float* all = p.partials + (uint64_t)unit * p.splits * 256 * (D + 4);
            for (uint32_t r = tid / kLanes; r < 256; r += 256 / kLanes) {
                const uint32_t rr = r & 127, rtok = t0 + (r >> 7) * p.tokens + rr / p.group, rg = rr % p.group;
                if (rr >= p.tokens * p.group || rtok >= a.q_tokens) continue;
                const uint32_t c = 4 * (tid % kLanes);
                float mm = -INFINITY;
                for (uint32_t i = 0; i < p.splits; i++) mm = fmaxf(mm, __ldcg(all + ((uint64_t)i * 256 + r) * (D + 4) + D));
                const float base = mm == -INFINITY ? 0.0f : mm;
                float ll = 0.0f;
                float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                for (uint32_t i = 0; i < p.splits; i++) {
                    const float* q = all + ((uint64_t)i * 256 + r) * (D + 4);
                    const float2 ml = __ldcg(reinterpret_cast<const float2*>(q + D));
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(q + c));
                    const float f = exp2_approx(ml.x - base);
                    ll = fmaf(f, ml.y, ll);
                    o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
                }
                const bool seen = mask.pos(rtok) >= 0;
                const float rl = 1.0f / ll;
                const uint32_t rh = h * p.group + rg;
                __nv_bfloat16* row = static_cast<__nv_bfloat16*>(a.out.data) + b * a.out.stride_b + (int64_t)rtok * a.out.stride_t +
                                     rh * a.out.stride_h;
                const uint2 w = make_uint2(pack2<false>(o.x * rl, o.y * rl), pack2<false>(o.z * rl, o.w * rl));
                *reinterpret_cast<uint2*>(row + c) = seen ? w : make_uint2(0, 0);
                if (c == 0 && a.lse) a.lse[((uint64_t)b * a.q_heads + rh) * a.q_tokens + rtok] = seen ? (mm + log2f(ll)) * kLn2 : -INFINITY;
            }
            }
        }
    }
    __syncthreads();
    tcgen_fence_after();
    if (warp == 8) tmem_free<512>(tmem);
}

template <int D>
cudaError_t launch(const TilesParams& p, uint32_t ctas, cudaStream_t s) {
    Wave w;
    const cudaError_t e = launch_wave<tiles_kernel<D, false>>(kThreadsTiles, TilesShape<D>::kSmem, w);
    if (e != cudaSuccess) return e;
    tiles_kernel<D, false><<<ctas, kThreadsTiles, TilesShape<D>::kSmem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

bool attention_tiles_plan(const splitzip_attention_args& a, AttentionPlan& p) {
    const uint32_t group = a.q_heads / a.kv_heads, tokens = kTileM / group;
    p.rows = a.q_tokens * group;
    p.tile_rows = 2 * tokens * group;
    p.row_tiles = (a.q_tokens + 2 * tokens - 1) / (2 * tokens);
    const uint64_t units = (uint64_t)a.batch * a.kv_heads * p.row_tiles;
    // The tiles of slots a CTA's rows can see at most.
    uint64_t most = (a.kv_tokens + kBN - 1) / kBN;
    if (a.window)
        most = std::min(most, ((uint64_t)a.window + 2 * tokens + kBN - 1) / kBN + 1 + ((uint64_t)a.sinks + kBN - 1) / kBN);
    // Fill the GPU with one CTA per SM if each split still has four steps.
    const uint64_t splits = std::min((uint64_t)kSms / units, most / 4);
    p.splits = (uint32_t)(splits < 1 ? 1 : splits);
    if (units * p.splits > 0x7FFFFFFFull) return false;
    p.bytes = kAttentionHeader + (p.splits > 1 ? units * p.splits * 256 * (a.head_dim + 4) * 4 : 0);
    return true;
}

bool attention_tiles_usable(const splitzip_attention_args& a) {
    return a.scale > 0.0f && a.cache_format == SPLITZIP_FORMAT_BF16;  // maxima are taken before scaling
}

cudaError_t launch_attention_tiles(const splitzip_attention_args& a, const AttentionPlan& plan, void* workspace,
                                   cudaStream_t s) {
    TilesParams p;
    p.a = a;
    p.group = a.q_heads / a.kv_heads;
    p.tokens = kTileM / p.group;
    p.row_ctas = plan.row_tiles;
    p.splits = plan.splits;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.counters = reinterpret_cast<uint32_t*>(ws);
    p.status = reinterpret_cast<uint32_t*>(ws + kAttentionStatus);
    p.partials = reinterpret_cast<float*>(ws + kAttentionHeader);
    if (!make_map(p.qmap, a.q, a.head_dim, a.q_heads, a.q_tokens, a.batch, p.group, p.tokens, true, &p.one_q) ||
        !make_map(p.kmap, a.k, a.head_dim, a.kv_heads, a.kv_tokens, a.batch, 1, kBN, false, &p.one_k) ||
        !make_map(p.vmap, a.v, a.head_dim, a.kv_heads, a.kv_tokens, a.batch, 1, kBN, false, &p.one_v))
        return cudaErrorInvalidValue;
    const uint32_t ctas = a.batch * a.kv_heads * plan.row_tiles * plan.splits;
    return a.head_dim == 64 ? launch<64>(p, ctas, s) : launch<128>(p, ctas, s);
}

}  // namespace splitzip
