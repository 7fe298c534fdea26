// attention_weights.cu -- the attention weight that cached slots get (sm_103a).
//
// w[t] = sum over query rows r that see slot t of exp(scale q_r.k_t - lse_r).
// The scores are computed transposed on the tensor cores, S = K Q^T with slots
// as the 128 rows of the accumulator: a thread holds one slot's row, so its sum
// needs no exchange and no atomics, and its order is fixed.
//
// A CTA owns two tiles of 128 slots of one key/value head, keeps their keys in
// shared memory and walks the tiles of query rows (128 / group tokens, the
// group's heads side by side) that can see any of them; each query tile is read
// once for both.  Per slot tile two accumulators of 128 columns in tensor
// memory take turns, so the products run ahead of the exponentials.  128 x 128
// scores of head_dim 128 take 512 cycles of the tensor cores and 512 of the
// exponential units.
//
// Roles: warps 0-3 and 4-7 sum the slots of one tile each, 8 issues the
// products, 9 the TMA loads, 10 and 11 bring each query tile's lse and
// positions to shared memory.  E5M2 keys are widened to BF16 (exact) while they
// are brought in.
#include <algorithm>
#include <cstdint>

#include "attention.cuh"
#include "tcgen.cuh"
#include "tensor_map.h"

namespace splitzip {
namespace {

constexpr int kThreadsWeights = 384;
constexpr int kSlotTile = 128, kRowTile = 128;
constexpr int kQStages = 3, kMetas = 4;

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
    static constexpr int kSmem = (2 + kQStages) * kTile + 1024;
};

struct WeightsShared {
    uint64_t k_full, q_full[kQStages], q_empty[kQStages];
    uint64_t s_full[2][2], s_free[2][2];
    uint64_t meta_full[kMetas], meta_free[kMetas];
    uint64_t drained;
    uint32_t tmem, err;
    alignas(16) float lse[kMetas][kRowTile];    // times -log2(e)
    alignas(16) int32_t pos[kMetas][kRowTile];  // -1: no query in this row
};

// Two E5M2 values (the bytes `which` and `which` + 1 of r) as BF16.
__device__ __forceinline__ uint32_t e5m2_to_bf16(uint32_t r, uint32_t select) {
    const uint32_t h = prmt(r, 0u, select);  // FP16, exact
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack2<false>(f.x, f.y);
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kThreadsWeights, 1) weights_kernel(const __grid_constant__ WeightsParams p) {
    using S = WeightsShape<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ WeightsShared sh;
    uint8_t* ks = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* ring = ks + 2 * S::kTile;
    const splitzip_attention_args& a = p.a;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bh = blockIdx.x / p.slot_ctas, sc = blockIdx.x - bh * p.slot_ctas;
    const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
    const Mask mask(a, b);
    const int32_t s_lo = (int32_t)(sc * 2 * kSlotTile), s_hi = (int32_t)min((int64_t)s_lo + 2 * kSlotTile, (int64_t)a.kv_tokens) - 1;

    // Query tokens that can see one of these slots: positions from s_lo on, and
    // up to the window's end behind s_hi unless s_lo is a sink.
    int64_t t_lo = max((int64_t)0, (int64_t)s_lo - mask.first);
    int64_t t_hi = s_lo < mask.n ? (int64_t)a.q_tokens : 0;
    if (s_lo >= mask.sinks) t_hi = min(t_hi, (int64_t)s_hi + mask.window - mask.first);
    const uint32_t i0 = t_hi > t_lo ? (uint32_t)(t_lo / p.tokens) : 0;
    const uint32_t steps = t_hi > t_lo ? (uint32_t)((t_hi + p.tokens - 1) / p.tokens) - i0 : 0;
    auto rows_of = [&](uint32_t i) { return min(p.tokens, a.q_tokens - (i0 + i) * p.tokens) * p.group; };
    volatile uint32_t* err = &sh.err;

    if (warp == 8) tmem_alloc512(&sh.tmem);
    if (tid == 0) {
        mbar_init(&sh.k_full, 1);
        for (int i = 0; i < kQStages; i++) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&sh.s_full[i >> 1][i & 1], 1);
            mbar_init(&sh.s_free[i >> 1][i & 1], 4);
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
        for (uint32_t x = tid; x < 2 * kSlotTile * (D / 16); x += kThreadsWeights) {
            const uint32_t r = x / (D / 16), c = x % (D / 16);
            uint4 v = make_uint4(0, 0, 0, 0);
            if (s_lo + (int32_t)r <= s_hi) v = *reinterpret_cast<const uint4*>(kbase + (int64_t)(s_lo + r) * a.k.stride_t + 16 * c);
            uint8_t* row = ks + (r >> 7) * S::kTile + (c >> 2) * (kSlotTile * 128) + (r & 127) * 128;
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
                mbar_arrive_expect_tx(&sh.k_full, 2 * S::kTile);
#pragma unroll
                for (int t = 0; t < 2; t++)
#pragma unroll
                    for (int x = 0; x < D / 64; x++)
                        tma_load4(ks + t * S::kTile + x * (kSlotTile * 128), &p.kmap, 64 * x, s_lo + t * kSlotTile,
                                  (int32_t)h, p.one_k ? 0 : (int32_t)b, &sh.k_full);
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
        if (lane == 0 && steps) {  // matrix products
            const uint32_t ka = smem_addr(ks), qa = smem_addr(ring);
            bool go = kF8 || mbar_wait_bounded(&sh.k_full, 0, err);
            for (uint32_t i = 0; go && i < steps; i++) {
                const uint32_t st = i % kQStages, x = i & 1;
                go = mbar_wait_bounded(&sh.q_full[st], (i / kQStages) & 1, err);
                // As many columns as the tile has rows, in steps of 16.
                const uint32_t shape = mma_shape(false, (rows_of(i) + 15) & ~15u, false);
                for (uint32_t t = 0; go && t < 2; t++) {
                    if (i >= 2) go = mbar_wait_bounded(&sh.s_free[t][x], ((i >> 1) - 1) & 1, err);
                    if (!go) break;
                    tcgen_fence_after();
#pragma unroll
                    for (int k = 0; k < D / 16; k++) {
                        const uint32_t at = (k >> 2) * (kSlotTile * 128) + (k & 3) * 32;
                        mma_ss(tmem + (2 * t + x) * kRowTile, desc_rows(ka + t * S::kTile + at), desc_rows(qa + st * S::kTile + at),
                               shape, k > 0);
                    }
                    mma_commit(&sh.s_full[t][x]);
                }
                if (go) mma_commit(&sh.q_empty[st]);
            }
            uint32_t late = 0;
            mma_commit(&sh.drained);
            mbar_wait_bounded(&sh.drained, 0, &late);
        }
    } else if (warp >= 10) {
        for (uint32_t i = 0; i < steps; i++) {
            const uint32_t x = i % kMetas, use = i / kMetas;
            if (use && !mbar_wait_bounded(&sh.meta_free[x], (use - 1) & 1, err)) break;
            const uint32_t rows = rows_of(i);
            for (uint32_t r = tid - 320; r < kRowTile; r += 64) {
                const uint32_t t = (i0 + i) * p.tokens + r / p.group, g = r % p.group;
                const bool valid = r < rows;
                sh.pos[x][r] = valid ? mask.pos(t) : -1;
                sh.lse[x][r] = valid ? a.lse[((uint64_t)b * a.q_heads + h * p.group + g) * a.q_tokens + t] * -kLog2e : 0.0f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.meta_full[x]);
        }
    } else {
        const uint32_t t = warp >> 2;
        const int32_t s0 = s_lo + (int32_t)(t * kSlotTile), slot = s0 + (int32_t)(tid & 127);
        const float scale = a.scale * kLog2e;
        const uint64_t scale2 = pair(scale, scale);
        const uint32_t lanes = ((warp & 3) * 32) << 16;
        float sum = 0.0f;
        for (uint32_t i = 0; i < steps; i++) {
            const uint32_t x = i & 1, mx = i % kMetas;
            if (!mbar_wait_bounded(&sh.meta_full[mx], (i / kMetas) & 1, err) ||
                !mbar_wait_bounded(&sh.s_full[t][x], (i >> 1) & 1, err)) {
                sum = __int_as_float(0x7FC00000);  // a wait that gave up: NaN
                break;
            }
            tcgen_fence_after();
            const uint32_t ta = (i0 + i) * p.tokens, rows = rows_of(i);
            const int32_t q0 = mask.first + (int32_t)ta, q1 = q0 + (int32_t)(rows / p.group) - 1;
            const bool whole = q0 >= 0 && mask.all(q0, q1, s0, s0 + kSlotTile - 1);
            uint64_t part[2] = {0, 0};
#pragma unroll 1
            for (uint32_t c = 0; c < rows; c += 32) {
                uint32_t s[32];
                __syncwarp();
                tmem_ld32(s, tmem + lanes + (2 * t + x) * kRowTile + c);
                tmem_wait_ld();
                if (whole && c + 32 <= rows) {
#pragma unroll
                    for (int y = 0; y < 32; y += 4) {
                        const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(&sh.lse[mx][c + y]);
#pragma unroll
                        for (int z = 0; z < 4; z += 2) {
                            float u, v;
                            unpair(fma2(pair(__uint_as_float(s[y + z]), __uint_as_float(s[y + z + 1])), scale2, z ? l.y : l.x), u, v);
                            part[z >> 1] = add2(part[z >> 1], pair(exp2_approx(u), exp2_approx(v)));
                        }
                    }
                } else {
                    float u = 0.0f;
#pragma unroll
                    for (int y = 0; y < 32; y++) {
                        const float e = exp2_approx(fmaf(__uint_as_float(s[y]), scale, sh.lse[mx][c + y]));
                        if (mask.sees(sh.pos[mx][c + y], slot)) u += e;
                    }
                    part[0] = add2(part[0], pair(u, 0.0f));
                }
            }
            float u, v, u2, v2;
            unpair(part[0], u, v);
            unpair(part[1], u2, v2);
            sum += (u + v) + (u2 + v2);
            tcgen_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.s_free[t][x]);
                mbar_arrive(&sh.meta_free[mx]);
            }
        }
        if (slot <= s_hi) {
            const uint64_t at = (uint64_t)bh * a.kv_tokens + (uint32_t)slot;
            p.out[at] = (p.in ? p.in[at] : 0.0f) + sum;
        }
        tcgen_fence_before();
    }
    __syncthreads();
    tcgen_fence_after();
    if (warp == 8) tmem_free512(tmem);
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
    p.slot_ctas = (a.kv_tokens + 2 * kSlotTile - 1) / (2 * kSlotTile);
    const bool f8 = a.cache_format == SPLITZIP_FORMAT_E5M2;
    if (!make_map(p.qmap, a.q, a.head_dim, a.q_heads, a.q_tokens, a.batch, p.group, p.tokens, true, &p.one_q))
        return cudaErrorInvalidValue;
    if (!f8 && !make_map(p.kmap, a.k, a.head_dim, a.kv_heads, a.kv_tokens, a.batch, 1, kSlotTile, false, &p.one_k))
        return cudaErrorInvalidValue;
    const uint32_t ctas = a.batch * a.kv_heads * p.slot_ctas;
    if (a.head_dim == 64) return f8 ? launch<64, true>(p, ctas, s) : launch<64, false>(p, ctas, s);
    return f8 ? launch<128, true>(p, ctas, s) : launch<128, false>(p, ctas, s);
}

}  // namespace splitzip
