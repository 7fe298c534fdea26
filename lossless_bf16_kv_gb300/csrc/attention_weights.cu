// attention_weights.cu -- the attention weight that cached slots get (sm_103a).
//
// w[t] = sum over query rows r that see slot t of exp(scale q_r.k_t - lse_r).
// The scores are computed transposed, k q^T, with slots as the rows of the
// product: a slot's sum then stays with the lanes that hold its row, needs no
// atomics and has a fixed order.  A CTA owns 128 slots of one key/value head,
// holds their keys as matrix fragments in registers and walks the query rows
// that can see any of them, 64 at a time through shared memory.
#include <cstdint>

#include "attention.cuh"

namespace splitzip {
namespace {

constexpr int kWeightThreads = 128;
constexpr int kWeightSlots = 128;  // 32 per warp
constexpr int kWeightRows = 64;    // query rows per step

struct WeightsParams {
    splitzip_attention_args a;
    const float* in;
    float* out;
    uint32_t group, rows, slot_tiles;
};

template <int D, bool kF8>
__global__ void __launch_bounds__(kWeightThreads) weights_kernel(const __grid_constant__ WeightsParams p) {
    constexpr int KS = D / 16;
    __shared__ __align__(128) uint8_t qs[kWeightRows * D * 2];
    __shared__ float s_scale[kWeightRows], s_lse[kWeightRows];
    __shared__ int32_t s_pos[kWeightRows];
    const splitzip_attention_args& a = p.a;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t bh = blockIdx.x / p.slot_tiles, st = blockIdx.x - bh * p.slot_tiles;
    const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
    const Mask mask(a, b);
    const int32_t s0 = (int32_t)(st * kWeightSlots), s1 = s0 + kWeightSlots - 1;

    // Query tokens that can see a slot of this tile: positions from s0 on (and
    // not negative), below the window's end behind s1 unless s0 is a sink.
    const int64_t t_lo = max((int64_t)0, (int64_t)max(s0, 0) - mask.first);
    int64_t t_hi = s0 < mask.n ? (int64_t)a.q_tokens : 0;
    if (s0 >= mask.sinks) t_hi = min(t_hi, (int64_t)s1 + mask.window - mask.first);
    const uint32_t r_lo = (uint32_t)(min(t_lo, (int64_t)a.q_tokens) * p.group);
    const uint32_t r_hi = t_hi > t_lo ? (uint32_t)(t_hi * p.group) : r_lo;

    uint32_t kf[2][KS][4];
    {
        const uint32_t elem = kF8 ? 1 : 2;
        const uint8_t* kbase = static_cast<const uint8_t*>(a.k.data) + (b * a.k.stride_b + h * a.k.stride_h) * elem;
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int k = 0; k < KS; k++)
#pragma unroll
                for (int y = 0; y < 2; y++) {
                    const int32_t slot = max(0, min(s0 + (int32_t)(32 * warp + 16 * i + 8 * y + lane / 4), mask.n - 1));
                    const uint8_t* row = kbase + slot * a.k.stride_t * elem;
                    if (kF8) {
                        const uint32_t v = *reinterpret_cast<const uint32_t*>(row + 16 * k + 4 * (lane & 3));
                        kf[i][k][y] = e5m2_01(v);
                        kf[i][k][2 + y] = e5m2_23(v);
                    } else {
                        const uint32_t* v = reinterpret_cast<const uint32_t*>(row + 32 * k + 4 * (lane & 3));
                        kf[i][k][y] = v[0];
                        kf[i][k][2 + y] = v[4];
                    }
                }
    }
    float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    for (uint32_t base = r_lo; base < r_hi; base += kWeightRows) {
        __syncthreads();
        for (uint32_t r = warp; r < kWeightRows; r += kWeightThreads / 32) {
            const uint32_t row = base + r, t = row / p.group, g = row - t * p.group;
            constexpr int V = D / 32;
            uint32_t v[V / 2];
#pragma unroll
            for (int i = 0; i < V / 2; i++) v[i] = 0;
            if (row < r_hi) {
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
                *reinterpret_cast<uint32_t*>(qs + r * (2 * D) + (((d / 8) ^ (r & 7u)) << 4) + 2 * (d % 8)) = w;
            }
            if (lane == 0) {
                s_scale[r] = a.scale * kLog2e / power;
                s_pos[r] = row < r_hi ? mask.pos(t) : -1;
                s_lse[r] = row < r_hi ? a.lse[((uint64_t)b * a.q_heads + h * p.group + g) * a.q_tokens + t] * kLog2e : 0.0f;
            }
        }
        __syncthreads();
#pragma unroll 2
        for (uint32_t n = 0; n < kWeightRows / 8; n++) {
            float sc[2][4] = {};
#pragma unroll
            for (int k = 0; k < KS; k += 2) {
                uint32_t q[4];
                ldmatrix4(q, smem_addr(qs) + (8 * n + (lane & 7)) * (2 * D) + (((2 * k + (lane >> 3)) ^ (lane & 7u)) << 4));
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    mma16816<kF8>(sc[i], kf[i][k], q[0], q[1]);
                    mma16816<kF8>(sc[i], kf[i][k + 1], q[2], q[3]);
                }
            }
#pragma unroll
            for (int x = 0; x < 2; x++) {
                const uint32_t r = 8 * n + 2 * (lane & 3) + x;
                const float scale = s_scale[r], lse = s_lse[r];
                const int32_t pos = s_pos[r];
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int y = 0; y < 2; y++) {
                        const int32_t slot = s0 + (int32_t)(32 * warp + 16 * i + 8 * y + lane / 4);
                        if (mask.sees(pos, slot)) sum[i][y] += exp2_approx(fmaf(sc[i][2 * y + x], scale, -lse));
                    }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int y = 0; y < 2; y++) {
            sum[i][y] += __shfl_xor_sync(0xFFFFFFFFu, sum[i][y], 1);
            sum[i][y] += __shfl_xor_sync(0xFFFFFFFFu, sum[i][y], 2);
            const uint32_t slot = (uint32_t)s0 + 32 * warp + 16 * i + 8 * y + lane / 4;
            if ((lane & 3) == 0 && slot < a.kv_tokens) {
                const uint64_t at = (uint64_t)bh * a.kv_tokens + slot;
                p.out[at] = (p.in ? p.in[at] : 0.0f) + sum[i][y];
            }
        }
}

}  // namespace

cudaError_t launch_attention_weights(const splitzip_attention_args& a, const float* weights_in, float* weights_out,
                                     cudaStream_t s) {
    WeightsParams p;
    p.a = a;
    p.in = weights_in;
    p.out = weights_out;
    p.group = a.q_heads / a.kv_heads;
    p.rows = a.q_tokens * p.group;
    p.slot_tiles = (a.kv_tokens + kWeightSlots - 1) / kWeightSlots;
    const uint32_t ctas = a.batch * a.kv_heads * p.slot_tiles;
    const bool f8 = a.cache_format == SPLITZIP_FORMAT_E5M2;
    if (a.head_dim == 64) {
        if (f8) weights_kernel<64, true><<<ctas, kWeightThreads, 0, s>>>(p);
        else weights_kernel<64, false><<<ctas, kWeightThreads, 0, s>>>(p);
    } else {
        if (f8) weights_kernel<128, true><<<ctas, kWeightThreads, 0, s>>>(p);
        else weights_kernel<128, false><<<ctas, kWeightThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

}  // namespace splitzip
