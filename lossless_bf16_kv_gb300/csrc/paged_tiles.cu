// paged_tiles.cu -- plan and launch of paged_tiles.cuh (host).
#include <algorithm>
#include <cstdint>

#include "paged_tiles.cuh"

namespace splitzip {

namespace {

// All new tokens of a sequence in one tile, and slots for two (as attention_tiles.cu).
inline bool is_twin(const splitzip_paged_attention_args& a) {
    return a.max_q_tokens <= kTileM / (a.q_heads / a.pool.kv_heads) && a.kv_tokens > kBN;
}

}  // namespace

bool paged_tiles_plan(const splitzip_paged_attention_args& a, uint32_t rows_from, PagedPlan& p) {
    const uint32_t group = a.q_heads / a.pool.kv_heads, tokens = kTileM / group;
    const uint64_t per = is_twin(a) ? tokens : 2 * tokens, most_ctas = (a.max_q_tokens + per - 1) / per;
    // The row tiles that a batch of these sizes may have: of its sequences of more than
    // rows_from rows, each with one that is not full.
    const uint64_t sequences = std::min<uint64_t>(a.batch, (uint64_t)a.tokens * group / (rows_from + 1));
    p.row_tiles = (uint32_t)std::max<uint64_t>(1, std::min(sequences * most_ctas, (a.tokens + sequences * (per - 1)) / per));
    // The splits are for as many as there are if sequences are as long as they may be.
    const uint64_t likely = a.tokens / a.max_q_tokens * most_ctas + (a.tokens % a.max_q_tokens + per - 1) / per;
    const uint64_t units = std::min<uint64_t>(p.row_tiles, likely) * a.pool.kv_heads;
    uint64_t most = ((uint64_t)a.kv_tokens + kBN - 1) / kBN;
    if (a.window)
        most = std::min(most, ((uint64_t)a.window + 2 * tokens + kBN - 1) / kBN + 1 + ((uint64_t)a.sinks + kBN - 1) / kBN);
    p.splits = attention_tiles_splits(units, most, is_twin(a) ? 2 : 1);
    p.bytes = kAttentionHeader;
    return (uint64_t)p.row_tiles * a.pool.kv_heads * p.splits <= 0x7FFFFFFFull;
}

cudaError_t launch_paged_tiles(const splitzip_paged_attention_args& a, uint32_t rows_from, const PagedPlan& plan, void* workspace,
                               cudaStream_t s) {
    PagedTilesParams p;
    p.a = a;
    p.group = a.q_heads / a.pool.kv_heads;
    p.tokens = kTileM / p.group;
    p.splits = plan.splits;
    p.box = std::min<uint32_t>(a.pool.page_tokens, tile_part(a.pool));
    p.boxes = kBN / p.box;
    p.page_shift = 0;
    while ((1u << p.page_shift) < a.pool.page_tokens) p.page_shift++;
    p.bulk_exps = bulk_exponents(a.pool);
    p.rows_from = rows_from;
    p.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kAttentionStatus);
    p.wait_limit = wait_limit(0);  // a wait lasts a few steps at most
    const splitzip_pool& pool = a.pool;
    const bool wide = pool.format != kBf16;
    uint32_t one;
    if ((!wide && !make_map(p.qmap, a.q, 2, pool.head_dim, a.q_heads, a.tokens, 1, p.group, p.tokens, true, &one)) ||
        !page_map(p.kmap, pool, pool.k, p.box) || !page_map(p.vmap, pool, pool.v, p.box))
        return cudaErrorInvalidValue;
    const uint32_t ctas = plan.row_tiles * pool.kv_heads * plan.splits;
    if (pool.head_dim == 64) return is_twin(a) ? launch_paged_64_twin(p, ctas, s) : launch_paged_64(p, ctas, s);
    return is_twin(a) ? launch_paged_128_twin(p, ctas, s) : launch_paged_128(p, ctas, s);
}

}  // namespace splitzip
