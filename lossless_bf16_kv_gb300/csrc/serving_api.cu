// serving_api.cu -- the extern "C" entry points of include/splitzip_serving.h:
// host-side argument checks and status mapping.
#include <cmath>
#include <cstdint>

#include "api_checks.h"
#include "serving.h"
#include "trace.h"

using namespace splitzip;

namespace {

inline uint32_t elem_bytes(uint32_t format) { return format == SPLITZIP_FORMAT_E5M2 ? 1 : 2; }
inline bool format_ok(uint32_t format) { return format == SPLITZIP_FORMAT_BF16 || format == SPLITZIP_FORMAT_E5M2; }

bool sizes_ok(const splitzip_attention_args& a) {
    if (!dim_ok(a.head_dim) || !format_ok(a.cache_format)) return false;
    if (!a.batch || !a.q_tokens || !a.kv_tokens || !a.kv_heads || !a.q_heads) return false;
    if (a.q_heads % a.kv_heads || a.q_heads / a.kv_heads > SPLITZIP_MAX_GROUP) return false;
    return (uint64_t)a.q_tokens * (a.q_heads / a.kv_heads) <= kMostTokens && a.kv_tokens <= kMostTokens &&
           (uint64_t)a.batch * a.kv_heads <= kMax31;
}

// Tiles of 128 query rows on the tensor cores from 17 rows of a key/value head on
// (the other kernel's smaller tile), and only for scales that kernel takes.  E5M2
// caches, which the other kernel widens at less cost, from 65 rows on, and from 33 on
// at head_dim 128 with enough units (sequences times key/value heads) to fill the GPU:
// there the other kernel walks each cache twice.  In us, this kernel and the other:
//   BF16, head_dim 128, 128 units of 16384 slots: 16 rows 159 and 157, 24 161 and 172,
//     64 163 and 320; 16 units of 2048: 16 rows 11.7 and 11.2, 24 13.0 and 15.5; 512
//     units of 1024: 24 rows 76 and 70, 40 79 and 123.
//   E5M2, head_dim 128, 40 rows: 128 units of 16384 265 and 278, 512 of 1024 103 and
//     110, 24 of 8192 33 and 40; 16 of 8192 30 and 29, 16 of 2048 17.4 and 15.5.
//   E5M2, head_dim 64, 64 rows: 128 units of 16384 194 and 170, 32 of 16384 45 and 53,
//     16 of 2048 13.4 and 12.7; 128 rows: 196 and 331, 48 and 92, 15.3 and 15.3.
// Neither side holds for one or two units and a long cache, of which a cluster of
// eight is all that this kernel makes: 2 units of 60000 slots, head_dim 128, 64 rows,
// BF16 56 and 43.
bool on_tiles(const splitzip_attention_args& a, const AttentionPlan& rows) {
    uint32_t most = 16;  // rows of the other kernel
    if (a.cache_format == SPLITZIP_FORMAT_E5M2) most = a.head_dim == 128 && (uint64_t)a.batch * a.kv_heads > 16 ? 32 : 64;
    return rows.rows > most && attention_tiles_usable(a);
}
bool plans(const splitzip_attention_args& a, AttentionPlan& rows, AttentionPlan& tiles) {
    return attention_rows_plan(a, rows) && attention_tiles_plan(a, tiles);
}
size_t bytes_of(const AttentionPlan& rows, const AttentionPlan& tiles) {
    return rows.bytes > tiles.bytes ? rows.bytes : tiles.bytes;
}

// Both calls, as users make them and (test) with a copy left out.
splitzip_status attention(const splitzip_attention_args* a, void* workspace, size_t workspace_bytes,
                          splitzip_stream_t s, const WaitTest* test) {
    AttentionPlan rows, tiles;
    if (!a || !sizes_ok(*a) || !plans(*a, rows, tiles)) return SPLITZIP_ERR_INVALID_ARG;
    const uint32_t e = elem_bytes(a->cache_format);
    if (!view_ok(a->q, 2, a->batch, a->q_tokens, a->q_heads) || !view_ok(a->out, 2, a->batch, a->q_tokens, a->q_heads, true) ||
        !view_ok(a->k, e, a->batch, a->kv_tokens, a->kv_heads) || !view_ok(a->v, e, a->batch, a->kv_tokens, a->kv_heads))
        return SPLITZIP_ERR_INVALID_ARG;
    if (!aligned(a->lse, 4) || !aligned(a->lens, 4) || !std::isfinite(a->scale)) return SPLITZIP_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < bytes_of(rows, tiles))
        return SPLITZIP_ERR_INVALID_ARG;
    if (on_tiles(*a, rows))
        return from_cuda(launch_attention_tiles(*a, tiles, workspace, test ? *test : WaitTest(), (cudaStream_t)s));
    if (test) return SPLITZIP_ERR_INVALID_ARG;
    return from_cuda(launch_attention_rows(*a, rows, workspace, (cudaStream_t)s));
}

splitzip_status attention_weights(const splitzip_attention_args* a, const float* weights_in, float* weights_out,
                                  splitzip_stream_t s, const WaitTest& test) {
    if (!a || !sizes_ok(*a) || !weights_out || !a->lse) return SPLITZIP_ERR_INVALID_ARG;
    if ((uint64_t)a->batch * a->kv_heads * ((a->kv_tokens + 127ull) / 128) > kMax31) return SPLITZIP_ERR_INVALID_ARG;
    if (!view_ok(a->q, 2, a->batch, a->q_tokens, a->q_heads) ||
        !view_ok(a->k, elem_bytes(a->cache_format), a->batch, a->kv_tokens, a->kv_heads))
        return SPLITZIP_ERR_INVALID_ARG;
    if (!aligned(a->lse, 4) || !aligned(a->lens, 4) || !aligned(weights_in, 4) || !aligned(weights_out, 4) ||
        !std::isfinite(a->scale))
        return SPLITZIP_ERR_INVALID_ARG;
    return from_cuda(launch_attention_weights(*a, weights_in, weights_out, test, (cudaStream_t)s));
}

}  // namespace

extern "C" {

splitzip_status splitzip_qk_norm_rope(const splitzip_norm_rope_args* a, splitzip_stream_t s) {
    TraceRange trace("splitzip_qk_norm_rope");
    if (!a || !dim_ok(a->head_dim) || !format_ok(a->cache_format) || !a->q_heads || !a->kv_heads)
        return SPLITZIP_ERR_INVALID_ARG;
    if (a->rot_dim % 8 || a->rot_dim > a->head_dim || !(a->eps >= 0.0f)) return SPLITZIP_ERR_INVALID_ARG;
    if ((uint64_t)a->q_heads + 2ull * a->kv_heads > kMax31 ||
        (uint64_t)a->n * ((uint64_t)a->q_heads + 2ull * a->kv_heads) > kMax31)
        return SPLITZIP_ERR_INVALID_ARG;
    if (a->cache_step && (a->cache_tokens > a->cache_step || a->cache_rows > 1ull << 32)) return SPLITZIP_ERR_INVALID_ARG;
    if (!a->n) return SPLITZIP_OK;
    if (a->rot_dim && (!a->positions || !a->table)) return SPLITZIP_ERR_INVALID_ARG;
    if (!a->slots || !aligned(a->slots, 8) || !aligned(a->positions, 4) || !aligned(a->table, 16) ||
        !aligned(a->q_weight, 16) || !aligned(a->k_weight, 16))
        return SPLITZIP_ERR_INVALID_ARG;
    const uint32_t e = elem_bytes(a->cache_format);
    const uint32_t rows = a->cache_rows > kMax31 ? (uint32_t)kMax31 : (uint32_t)a->cache_rows;
    if (!view_ok(a->q, 2, 1, a->n, a->q_heads) || !view_ok(a->k, 2, 1, a->n, a->kv_heads) ||
        !view_ok(a->v, 2, 1, a->n, a->kv_heads) || !view_ok(a->q_out, 2, 1, a->n, a->q_heads) ||
        !view_ok(a->k_cache, e, 1, rows, a->kv_heads) || !view_ok(a->v_cache, e, 1, rows, a->kv_heads))
        return SPLITZIP_ERR_INVALID_ARG;
    return from_cuda(launch_norm_rope(*a, (cudaStream_t)s));
}

size_t splitzip_attention_workspace_bytes(const splitzip_attention_args* a) {
    AttentionPlan rows, tiles;
    return a && sizes_ok(*a) && plans(*a, rows, tiles) ? bytes_of(rows, tiles) : 0;
}

splitzip_status splitzip_attention(const splitzip_attention_args* a, void* workspace, size_t workspace_bytes,
                                   splitzip_stream_t s) {
    TraceRange trace("splitzip_attention");
    return attention(a, workspace, workspace_bytes, s, nullptr);
}

splitzip_status splitzip_attention_test(const splitzip_attention_args* a, void* workspace, size_t workspace_bytes,
                                        splitzip_stream_t s, const splitzip_wait_test_opts* opts) {
    WaitTest test;
    return wait_test(opts, test) ? attention(a, workspace, workspace_bytes, s, &test) : SPLITZIP_ERR_INVALID_ARG;
}

splitzip_status splitzip_attention_status(void* workspace, splitzip_stream_t s) {
    TraceRange trace("splitzip_attention_status");
    if (!workspace || !aligned(workspace, 16)) return SPLITZIP_ERR_INVALID_ARG;
    uint32_t* status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kAttentionStatus);
    uint32_t bits = 0;
    cudaError_t e = cudaMemcpyAsync(&bits, status, sizeof(bits), cudaMemcpyDeviceToHost, (cudaStream_t)s);
    if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)s);
    if (e == cudaSuccess && bits) e = cudaMemsetAsync(status, 0, sizeof(bits), (cudaStream_t)s);
    if (e != cudaSuccess) return SPLITZIP_ERR_CUDA;
    return bits ? SPLITZIP_ERR_TIMEOUT : SPLITZIP_OK;
}

splitzip_status splitzip_attention_weights(const splitzip_attention_args* a, const float* weights_in,
                                           float* weights_out, splitzip_stream_t s) {
    TraceRange trace("splitzip_attention_weights");
    return attention_weights(a, weights_in, weights_out, s, WaitTest());
}

splitzip_status splitzip_attention_weights_test(const splitzip_attention_args* a, const float* weights_in,
                                                float* weights_out, splitzip_stream_t s,
                                                const splitzip_wait_test_opts* opts) {
    WaitTest test;
    return wait_test(opts, test) ? attention_weights(a, weights_in, weights_out, s, test) : SPLITZIP_ERR_INVALID_ARG;
}

splitzip_status splitzip_evict(const splitzip_evict_args* a, splitzip_stream_t s) {
    TraceRange trace("splitzip_evict");
    if (!a || !dim_ok(a->head_dim) || !format_ok(a->cache_format)) return SPLITZIP_ERR_INVALID_ARG;
    if (!a->batch || a->batch > 65535 || !a->kv_tokens || !a->kv_heads || !a->budget) return SPLITZIP_ERR_INVALID_ARG;
    if (a->kv_tokens > kMax31 || a->budget > kMax31 || (uint64_t)a->batch * a->kv_heads > kMax31 ||
        (uint64_t)a->budget * a->kv_heads > kMax31 * 16)
        return SPLITZIP_ERR_INVALID_ARG;
    if ((uint64_t)a->keep_first + a->keep_last > a->budget) return SPLITZIP_ERR_INVALID_ARG;
    const uint32_t e = elem_bytes(a->cache_format);
    if (!view_ok(a->k, e, a->batch, a->kv_tokens, a->kv_heads) || !view_ok(a->v, e, a->batch, a->kv_tokens, a->kv_heads) ||
        !view_ok(a->k_out, e, a->batch, a->budget, a->kv_heads, true) ||
        !view_ok(a->v_out, e, a->batch, a->budget, a->kv_heads, true))
        return SPLITZIP_ERR_INVALID_ARG;
    if (!a->weights || !a->index || !aligned(a->weights, 4) || !aligned(a->index, 4) || !aligned(a->weights_out, 4) ||
        !aligned(a->lens, 4) || !aligned(a->lens_out, 4))
        return SPLITZIP_ERR_INVALID_ARG;
    return from_cuda(launch_evict(*a, (cudaStream_t)s));
}

}  // extern "C"
