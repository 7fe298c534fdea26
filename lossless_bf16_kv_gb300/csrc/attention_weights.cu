// attention_weights.cu -- the attention weight that cached slots get (sm_103a).
//
// w[t] = sum over query rows r that see slot t of exp(scale q_r.k_t - lse_r).
// The scores are computed transposed on the tensor cores, S = K Q^T with slots
// as the 128 rows of the accumulator: a thread holds one slot's row, so its sum
// needs no exchange and no atomics, and its order is fixed.
//
// A CTA owns 128 slots of one key/value head, keeps their keys in shared memory
// and walks the tiles of 128 query rows (128 / group tokens, the group's heads
// side by side) that can see any of them.  The columns a slot's row takes part
// in are one range: tokens from the slot's own to the last that has it in its
// window.  Two accumulators of 128 columns in tensor memory take turns, so the
// products run ahead of the exponentials, and two CTAs share an SM.  128 x 128
// scores of head_dim 128 take 512 cycles of the tensor cores and 512 of the
// exponential units.
//
// Roles: warps 0-3 and 4-7 sum the lower and the upper 64 columns, 8 issues the
// products, 9 the TMA loads, 10 and 11 bring each query tile's lse to shared
// memory.  E5M2 keys are widened to BF16 (exact) while they are brought in.
#include <cstdint>

#include "attention.cuh"
#include "tcgen.cuh"
#include "tensor_map.h"

namespace splitzip {
namespace {

constexpr int kThreadsWeights = 384;
constexpr int kSlotTile = 128, kRowTile = 128;
constexpr int kQStages = 2, kMetas = 4;

struct WeightsParams {
    splitzip_attention_args a;
    CUtensorMap qmap, kmap;
    const float* in;
    float* out;
    uint32_t group, tokens;  // tokens of a query tile: 128 / group
    uint32_t slot_ctas;
    uint32_t one_q, one_k;  // the batch is one sequence: coordinate 0
};

template <int D>
struct WeightsShape {
    static constexpr int kTile = 128 * D * 2;
    static constexpr int kSmem = (1 + kQStages) * kTile + 1024;
};

struct WeightsShared {
    uint64_t k_full, q_full[kQStages], q_empty[kQStages];
    uint64_t s_full[2], s_free[2];
    uint64_t meta_full[kMetas], meta_free[kMetas];
    uint64_t drained;
    uint32_t tmem, err;
    alignas(16) float lse[kMetas][kRowTile];  // times -log2(e)
    float upper[kSlotTile];                   // sums of the upper columns
};

// Two E5M2 values (the bytes `which` and `which` + 1 of r) as BF16.
__device__ __forceinline__ uint32_t e5m2_to_bf16(uint32_t r, uint32_t select) {
    const uint32_t h = prmt(r, 0u, select);  // FP16, exact
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack2<false>(f.x, f.y);
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kThreadsWeights, 2) weights_kernel(const __grid_constant__ WeightsParams p) {
    using S = WeightsShape<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ WeightsShared sh;
    uint8_t* ks = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* ring = ks + S::kTile;
    const splitzip_attention_args& a = p.a;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // The first slots are seen by the most queries: they go first, of all heads.
    const uint32_t heads = a.batch * a.kv_heads, sc = blockIdx.x / heads, bh = blockIdx.x - sc * heads;
    const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
    const Mask mask(a, b);
    const int32_t s_lo = (int32_t)(sc * kSlotTile), s_hi = (int32_t)min((int64_t)s_lo + kSlotTile, (int64_t)a.kv_tokens) - 1;

    // Query tokens that can see one of these slots: positions from s_lo on, and
    // up to the window's end behind s_hi unless s_lo is a sink.
    int64_t t_lo = max((int64_t)0, (int64_t)s_lo - mask.first);
    int64_t t_hi = s_lo < mask.n ? (int64_t)a.q_tokens : 0;
    if (s_lo >= mask.sinks) t_hi = min(t_hi, (int64_t)s_hi + mask.window - mask.first);
    const uint32_t i0 = t_hi > t_lo ? (uint32_t)(t_lo / p.tokens) : 0;
    const uint32_t steps = t_hi > t_lo ? (uint32_t)((t_hi + p.tokens - 1) / p.tokens) - i0 : 0;
    auto rows_of = [&](uint32_t i) { return min(p.tokens, a.q_tokens - (i0 + i) * p.tokens) * p.group; };
    volatile uint32_t* err = &sh.err;

    if (warp == 8) tmem_alloc<256>(&sh.tmem);
    if (tid == 0) {
        mbar_init(&sh.k_full, 1);
        for (int i = 0; i < kQStages; i++) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 8);
        }
        for (int i = 0; i < kMetas; i++) {
            mbar_init(&sh.meta_full[i], 2);
            mbar_init(&sh.meta_free[i], 8);
        }
        mbar_init(&sh.drained, 1);
        sh.err = 0;
        fence_mbar_init();
    }
    if (kF8 && steps) {
        // 16 keys' bytes at a time, into the swizzled rows that the TMA writes for BF16.
        const uint8_t* kbase = static_cast<const uint8_t*>(a.k.data) + b * a.k.stride_b + h * a.k.stride_h;
        for (uint32_t x = tid; x < kSlotTile * (D / 16); x += kThreadsWeights) {
            const uint32_t r = x / (D / 16), c = x % (D / 16);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (s_lo + (int32_t)r <= s_hi) v = *reinterpret_cast<const uint4*>(kbase + (int64_t)(s_lo + r) * a.k.stride_t + 16 * c);
            uint8_t* row = ks + (c >> 2) * (kSlotTile * 128) + r * 128;
            const uint32_t c0 = 2 * (c & 3);
            *reinterpret_cast<uint4*>(row + ((c0 ^ (r & 7)) << 4)) = make_uint4(
                e5m2_to_bf16(v.x, 0x1404), e5m2_to_bf16(v.x, 0x3424), e5m2_to_bf16(v.y, 0x1404), e5m2_to_bf16(v.y, 0x3424));
            *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(
                e5m2_to_bf16(v.z, 0x1404), e5m2_to_bf16(v.z, 0x3424), e5m2_to_bf16(v.w, 0x1404), e5m2_to_bf16(v.w, 0x3424));
        }
        fence_async_proxy();
    }
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp == 9) {
        if (lane == 0 && steps) {  // TMA
            if (!kF8) {
                mbar_arrive_expect_tx(&sh.k_full, S::kTile);
#pragma unroll
                for (int x = 0; x < D / 64; x++)
                    tma_load4(ks + x * (kSlotTile * 128), &p.kmap, 64 * x, s_lo, (int32_t)h, p.one_k ? 0 : (int32_t)b, &sh.k_full);
            }
            uint32_t i = 0;
            for (; i < steps; i++) {
                const uint32_t st = i % kQStages, use = i / kQStages;
                if (use && !mbar_wait_bounded(&sh.q_empty[st], (use - 1) & 1, err)) break;
                mbar_arrive_expect_tx(&sh.q_full[st], p.tokens * p.group * D * 2);
#pragma unroll
                for (int x = 0; x < D / 64; x++)
                    tma_load4(ring + st * S::kTile + x * (kRowTile * 128), &p.qmap, 64 * x, (int32_t)(h * p.group),
                              (int32_t)((i0 + i) * p.tokens), p.one_q ? 0 : (int32_t)b, &sh.q_full[st]);
            }
            // Every load has landed before this CTA may end, also where a wait gave up.
            uint32_t late = 0;
            if (!kF8) mbar_wait_bounded(&sh.k_full, 0, &late);
            for (uint32_t x = i > kQStages ? i - kQStages : 0; x < i; x++)
                mbar_wait_bounded(&sh.q_full[x % kQStages], (x / kQStages) & 1, &late);
        }
    } else if (warp == 8) {
        if (steps) {  // matrix products: the whole warp waits, one lane issues
            const bool leader = elect_one();
            const uint32_t ka = desc_rows(smem_addr(ks)), qa = desc_rows(smem_addr(ring));
            bool go = kF8 || mbar_wait_bounded(&sh.k_full, 0, err);
            for (uint32_t i = 0; go && i < steps; i++) {
                const uint32_t st = i % kQStages, x = i & 1;
                go = mbar_wait_bounded(&sh.q_full[st], (i / kQStages) & 1, err) &&
                     (i < 2 || mbar_wait_bounded(&sh.s_free[x], ((i >> 1) - 1) & 1, err));
                if (!go) break;
                // As many columns as the tile has rows, in steps of 16.
                const uint32_t shape = mma_shape(false, (rows_of(i) + 15) & ~15u, false);
                tcgen_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < D / 16; k++) {
                        const uint32_t at = (k >> 2) * (kSlotTile * 128) + (k & 3) * 32;
                        mma_ss(tmem + x * kRowTile, desc(ka, at), desc(qa + st * (S::kTile >> 4), at), shape, k > 0);
                    }
                    mma_commit(&sh.s_full[x]);
                    mma_commit(&sh.q_empty[st]);
                }
                __syncwarp();  // no lane falls a phase behind
            }
            uint32_t late = 0;
            __syncwarp();
            if (leader) mma_commit(&sh.drained);
            mbar_wait_bounded(&sh.drained, 0, &late);
        }
    } else if (warp >= 10) {
        const uint32_t ra = tid - 320, rb = ra + 64;
        const float* la = a.lse + ((uint64_t)b * a.q_heads + h * p.group + ra % p.group) * a.q_tokens + i0 * p.tokens + ra / p.group;
        const float* lb = a.lse + ((uint64_t)b * a.q_heads + h * p.group + rb % p.group) * a.q_tokens + i0 * p.tokens + rb / p.group;
        for (uint32_t i = 0; i < steps; i++, la += p.tokens, lb += p.tokens) {
            const uint32_t x = i % kMetas, use = i / kMetas;
            if (use && !mbar_wait_bounded(&sh.meta_free[x], (use - 1) & 1, err)) break;
            const uint32_t rows = rows_of(i);
            sh.lse[x][ra] = ra < rows ? *la * -kLog2e : 0.0f;
            sh.lse[x][rb] = rb < rows ? *lb * -kLog2e : 0.0f;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.meta_full[x]);
        }
    } else {
        const uint32_t half = warp >> 2, c0 = half * 64;
        const int32_t slot = s_lo + (int32_t)(tid & 127);
        const float scale = a.scale * kLog2e;
        const uint64_t scale2 = pair(scale, scale);
        const uint32_t sa = tmem + (((warp & 3) * 32) << 16) + c0;
        // Query tokens that see this slot, [see_lo, see_hi) from the first tile on, and
        // the tiles all of whose tokens see all of this warp's slots.
        const int64_t behind = (int64_t)slot - mask.first - (int64_t)i0 * p.tokens, last = (int64_t)a.q_tokens - (int64_t)i0 * p.tokens;
        const int32_t see_lo = (int32_t)min(max(behind, (int64_t)0), last);
        const int32_t see_hi = slot < mask.sinks ? (int32_t)last : (int32_t)max(min(behind + mask.window, last), (int64_t)0);
        const uint32_t whole_lo = __reduce_max_sync(0xFFFFFFFFu, ((uint32_t)see_lo + p.tokens - 1) / p.tokens);
        const uint32_t whole_hi = __reduce_min_sync(0xFFFFFFFFu, (uint32_t)see_hi / p.tokens);
        const int32_t group = (int32_t)p.group, tokens = (int32_t)p.tokens;
        const bool full = p.tokens * p.group >= c0 + 64;  // all of this half's columns are in use
        float sum = 0.0f;
        for (uint32_t i = 0; i < steps; i++) {
            const uint32_t x = i & 1, mx = i % kMetas;
            if (!mbar_wait_bounded(&sh.meta_full[mx], (i / kMetas) & 1, err) ||
                !mbar_wait_bounded(&sh.s_full[x], (i >> 1) & 1, err)) {
                sum = __int_as_float(0x7FC00000);  // a wait that gave up: NaN
                break;
            }
            tcgen_fence_after();
            uint32_t s[2][32];
            tmem_ld32(s[0], sa + x * kRowTile);
            tmem_ld32(s[1], sa + x * kRowTile + 32);
            const bool whole = i >= whole_lo && i < whole_hi;
            tmem_wait_ld();
            tmem_loaded(s[0]);
            tmem_loaded(s[1]);
            uint64_t part[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < 2; c++) {
                if (!whole || (!full && p.tokens * p.group < c0 + 32 * c + 32)) {
                    // This tile's columns that the slot takes part in.
                    const int32_t t0 = (int32_t)i * tokens, at = (int32_t)c0 + 32 * c;
                    const int32_t l = max(0, min(tokens, see_lo - t0)) * group - at, u = max(0, min(tokens, see_hi - t0)) * group - at;
                    const uint32_t from = l <= 0 ? 0xFFFFFFFFu : l > 31 ? 0u : 0xFFFFFFFFu << l;
                    const uint32_t below = u <= 0 ? 0u : u > 31 ? 0xFFFFFFFFu : ~(0xFFFFFFFFu << u);
                    const uint32_t in = from & below;
#pragma unroll
                    for (int y = 0; y < 32; y++) {
                        const float e = exp2_approx(fmaf(__uint_as_float(s[c][y]), scale, sh.lse[mx][c0 + 32 * c + y]));
                        part[y & 1] = add2(part[y & 1], pair(in >> y & 1u ? e : 0.0f, 0.0f));
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < 32; y += 4) {
                        const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(&sh.lse[mx][c0 + 32 * c + y]);
#pragma unroll
                        for (int z = 0; z < 4; z += 2) {
                            float u, v;
                            unpair(fma2(pair(__uint_as_float(s[c][y + z]), __uint_as_float(s[c][y + z + 1])), scale2, z ? l.y : l.x), u, v);
                            part[z >> 1] = add2(part[z >> 1], pair(exp2_approx(u), exp2_approx(v)));
                        }
                    }
                }
            }
            float u, v, u2, v2;
            unpair(part[0], u, v);
            unpair(part[1], u2, v2);
            sum += (u + v) + (u2 + v2);
            tcgen_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.s_free[x]);
                mbar_arrive(&sh.meta_free[mx]);
            }
        }
        if (half) sh.upper[tid & 127] = sum;
        named_sync(1, 256);
        if (!half && slot <= s_hi) {
            const uint64_t at = (uint64_t)bh * a.kv_tokens + (uint32_t)slot;
            p.out[at] = (p.in ? p.in[at] : 0.0f) + (sum + sh.upper[tid & 127]);
        }
        tcgen_fence_before();
    }
    __syncthreads();
    tcgen_fence_after();
    if (warp == 8) tmem_free<256>(tmem);
}

template <int D, bool kF8>
cudaError_t launch(const WeightsParams& p, uint32_t ctas, cudaStream_t s) {
    Wave w;
    const cudaError_t e = launch_wave<weights_kernel<D, kF8>>(kThreadsWeights, WeightsShape<D>::kSmem, w);
    if (e != cudaSuccess) return e;
    weights_kernel<D, kF8><<<ctas, kThreadsWeights, WeightsShape<D>::kSmem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_weights(const splitzip_attention_args& a, const float* weights_in, float* weights_out,
                                     cudaStream_t s) {
    WeightsParams p;
    p.a = a;
    p.in = weights_in;
    p.out = weights_out;
    p.group = a.q_heads / a.kv_heads;
    p.tokens = kRowTile / p.group;
    p.slot_ctas = (a.kv_tokens + kSlotTile - 1) / kSlotTile;
    const bool f8 = a.cache_format == SPLITZIP_FORMAT_E5M2;
    if (!make_map(p.qmap, a.q, 2, a.head_dim, a.q_heads, a.q_tokens, a.batch, p.group, p.tokens, true, &p.one_q))
        return cudaErrorInvalidValue;
    if (!f8 && !make_map(p.kmap, a.k, 2, a.head_dim, a.kv_heads, a.kv_tokens, a.batch, 1, kSlotTile, false, &p.one_k))
        return cudaErrorInvalidValue;
    const uint32_t ctas = a.batch * a.kv_heads * p.slot_ctas;
    if (a.head_dim == 64) return f8 ? launch<64, true>(p, ctas, s) : launch<64, false>(p, ctas, s);
    return f8 ? launch<128, true>(p, ctas, s) : launch<128, false>(p, ctas, s);
}

}  // namespace splitzip
