// paged_tiles.cu -- plan and launch of paged_tiles.cuh (host).
#include <algorithm>
#include <cstdint>

#include "paged_tiles.cuh"

namespace splitzip {

namespace {

// The most new tokens of a sequence that the launch takes.
inline uint32_t most_tokens(const splitzip_paged_attention_args& a, uint32_t rows_upto) {
    return std::min(a.max_q_tokens, rows_upto / (a.q_heads / a.pool.kv_heads));
}
// All of them in one tile, and slots for two (as attention_tiles.cu).
inline bool is_twin(const splitzip_paged_attention_args& a, uint32_t rows_upto) {
    return most_tokens(a, rows_upto) <= kTileM / (a.q_heads / a.pool.kv_heads) && a.kv_tokens > kBN;
}

}  // namespace

bool paged_tiles_plan(const splitzip_paged_attention_args& a, uint32_t rows_from, uint32_t rows_upto, PagedPlan& p) {
    const uint32_t group = a.q_heads / a.pool.kv_heads, tokens = kTileM / group, most_new = most_tokens(a, rows_upto);
    const bool twin = is_twin(a, rows_upto);
    const uint64_t per = twin ? tokens : 2 * tokens, most_ctas = (most_new + per - 1) / per;
    // The row tiles that a batch of these sizes may have: of its sequences of more than
    // rows_from rows, each with one that is not full.
    const uint64_t sequences = std::min<uint64_t>(a.batch, (uint64_t)a.tokens * group / (rows_from + 1));
    p.row_tiles = (uint32_t)std::max<uint64_t>(1, std::min(sequences * most_ctas, (a.tokens + sequences * (per - 1)) / per));
    // The splits are for as many as there are if sequences are as long as they may be.
    const uint64_t likely = a.tokens / most_new * most_ctas + (a.tokens % most_new + per - 1) / per;
    const uint64_t units = std::min<uint64_t>(p.row_tiles, likely) * a.pool.kv_heads;
    uint64_t most = ((uint64_t)a.kv_tokens + kBN - 1) / kBN;
    if (a.window)
        most = std::min(most, ((uint64_t)a.window + 2 * tokens + kBN - 1) / kBN + 1 + ((uint64_t)a.sinks + kBN - 1) / kBN);
    uint64_t steps;
    p.splits = attention_tiles_splits(units, most, twin ? 2 : 1, &steps);
    // Or no splits, and the row tiles behind the last whole wave cut (as many as there are on
    // the device) into pieces, as PagedTilesParams::part_of has it: where that takes fewer
    // steps.  Joining through memory costs 4 and another for each piece.
    const uint64_t waves = units / kSms, rest = units % kSms;
    bool cut = !twin && rest && rest <= kSms * 2 / 3 && most >= PagedTilesParams::kLeastCut;
    if (cut) {
        uint64_t n = std::min<uint64_t>(kSms / rest, PagedTilesParams::kMostPieces);
        while (n > 1 && n * n > most) n--;
        const uint64_t longest = rest <= kSms / 2 ? (most + n - 1) / n : most - most / 3;
        cut = waves * (most + kSplitCost) + longest + kSplitCost + 4 + std::max<uint64_t>(n, 2) < steps;
    }
    if (cut) p.splits = 1;
    p.ctas = (uint64_t)p.row_tiles * a.pool.kv_heads * p.splits;
    p.bytes = 0;
    if (cut) {
        p.ctas += kSms;
        // Whatever the ranges on the device are: thirds make the most pieces.
        p.bytes = 2 * (kSms * 2 / 3) * sizeof(float4) * (a.pool.head_dim == 64 ? kPieceFloat4s<64> : kPieceFloat4s<128>);
        static_assert(2 * (kSms * 2 / 3) >= kSms, "equal pieces are kSms at most");
    }
    return p.ctas <= 0x7FFFFFFFull;
}

cudaError_t launch_paged_tiles(const splitzip_paged_attention_args& a, uint32_t rows_from, uint32_t rows_upto, const PagedPlan& plan, void* workspace,
                               size_t at_partials, const void* widened, bool beside, const WaitTest& test, cudaStream_t s) {
    PagedTilesParams p;
    p.a = a;
    p.group = a.q_heads / a.pool.kv_heads;
    p.tokens = kTileM / p.group;
    p.splits = plan.splits;
    uint8_t* space = static_cast<uint8_t*>(workspace);
    p.partials = plan.bytes ? reinterpret_cast<float4*>(space + at_partials) : nullptr;
    p.counters = reinterpret_cast<uint32_t*>(space + kTilesCounters + (widened ? kSms : 0));
    static_assert(kTilesCounters + 2 * kSms <= kAttentionStatus && kSms % 4 == 0, "a byte for each row tile that is cut");
    p.rows_from = rows_from;
    p.rows_upto = rows_upto;
    p.widened = widened != nullptr;
    splitzip_pool& pool = p.a.pool;
    if (widened) {
        const int64_t t = (int64_t)widened_tokens(a), d = pool.head_dim;
        pool.format = kF16;
        pool.pages = (uint32_t)widened_sequences(a, rows_from);
        pool.page_tokens = (uint32_t)t;
        pool.k = {const_cast<void*>(widened), 2 * t * d * pool.kv_heads, d, t * d, nullptr, 0, 0, 0};
        pool.v = pool.k;
        pool.v.data = static_cast<uint8_t*>(pool.k.data) + 2 * t * d * pool.kv_heads;
        p.slot_mask = 0x7FFFFFFFu;
    } else {
        p.slot_mask = pool.page_tokens - 1;
    }
    p.box = std::min<uint32_t>(pool.page_tokens, tile_part(pool));
    p.boxes = kBN / p.box;
    p.page_shift = 0;
    while ((1u << p.page_shift) < a.pool.page_tokens) p.page_shift++;
    p.bulk_exps = bulk_exponents(pool);
    p.status = reinterpret_cast<uint32_t*>(space + kAttentionStatus);
    p.wait_limit = test.limit ? test.limit : wait_limit(0);  // a wait lasts a few steps at most
    p.test_cta = test.cta;
    p.test_tile = test.tile;
    const bool wide = pool.format != kBf16;
    uint32_t one;
    if ((!wide && !make_map(p.qmap, a.q, 2, pool.head_dim, a.q_heads, a.tokens, 1, p.group, p.tokens, true, &one)) ||
        !page_map(p.kmap, pool, pool.k, p.box) || !page_map(p.vmap, pool, pool.v, p.box))
        return cudaErrorInvalidValue;
    const uint32_t ctas = (uint32_t)plan.ctas;
    const bool twin = is_twin(a, rows_upto);
    if (pool.head_dim == 64) return twin ? launch_paged_64_twin(p, ctas, beside, s) : launch_paged_64(p, ctas, beside, s);
    return twin ? launch_paged_128_twin(p, ctas, beside, s) : launch_paged_128(p, ctas, beside, s);
}

}  // namespace splitzip
