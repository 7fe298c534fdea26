// pages_api.cu -- the extern "C" entry points of include/splitzip_pages.h:
// host-side argument checks and status mapping.
#include <cmath>
#include <cstdint>

#include "../../include/splitzip_pages_testing.h"
#include "api_checks.h"
#include "pages.h"
#include "trace.h"

using namespace splitzip;

namespace {

bool quantised(uint32_t format) { return format == SPLITZIP_FORMAT_INT8 || format == SPLITZIP_FORMAT_E2M1; }

bool pool_sizes_ok(const splitzip_pool& p) {
    return dim_ok(p.head_dim) && p.format <= SPLITZIP_FORMAT_E2M1 && p.pages && p.pages <= kMax31 && p.kv_heads &&
           p.page_tokens >= 16 && p.page_tokens <= 65536 && (p.page_tokens & (p.page_tokens - 1)) == 0;
}
// Strides of dimensions of length 1 are not looked at.
bool rows_ok(const splitzip_page_rows& r, const splitzip_pool& p) {
    const int64_t unit = p.format == SPLITZIP_FORMAT_BF16 ? 8 : 16, most = 1ll << 38;
    const auto ok = [=](uint32_t n, int64_t s, int64_t of) { return n <= 1 || (s > 0 && s < most && s % of == 0); };
    if (!r.data || !aligned(r.data, 16) || !ok(p.pages, r.stride_p, unit) || !ok(p.page_tokens, r.stride_t, unit) ||
        !ok(p.kv_heads, r.stride_h, unit))
        return false;
    return !quantised(p.format) || (r.exponents && aligned(r.exponents, 4) && ok(p.pages, r.exp_stride_p, 4) &&
                                    ok(p.page_tokens, r.exp_stride_t, 4) && ok(p.kv_heads, r.exp_stride_h, 4));
}
bool pool_ok(const splitzip_pool& p) { return pool_sizes_ok(p) && rows_ok(p.k, p) && rows_ok(p.v, p); }

bool sizes_ok(const splitzip_paged_attention_args& a) {
    if (!pool_sizes_ok(a.pool) || !a.batch || !a.tokens || !a.max_q_tokens || !a.kv_tokens || !a.q_heads) return false;
    const uint32_t hk = a.pool.kv_heads;
    if (a.q_heads % hk || a.q_heads / hk > SPLITZIP_MAX_GROUP || a.max_q_tokens > a.tokens) return false;
    return (uint64_t)a.tokens * (a.q_heads / hk) <= kMostTokens && a.kv_tokens <= kMostTokens &&
           a.kv_tokens <= (uint64_t)a.table_width * a.pool.page_tokens && (uint64_t)a.batch * hk <= kMax31 &&
           (uint64_t)a.batch * hk * a.tokens <= kMax31;
}

// Which kernels take a call's sequences, by their query rows (new tokens times the heads
// of a group).
struct Plans {
    bool few, some, many;   // which of them may have sequences
    uint32_t upto, from;    // the most rows of the few-row kernel; more than that many: over caches widened first
    PagedPlan rows, tiles, wide;
    // Of the workspace: where partial results and the widened caches lie, and in all.
    size_t at_tiles, at_wide, at_widened, bytes;
};
bool plan(const splitzip_paged_attention_args& a, Plans& p) {
    constexpr uint32_t kFewRows = 16;
    constexpr uint64_t kMostWidened = 4ull << 30;
    const uint32_t many_rows = a.pool.format == SPLITZIP_FORMAT_E5M2 && a.pool.head_dim == 128 ? 2048 : 1024;
    const uint32_t group = a.q_heads / a.pool.kv_heads;
    const uint64_t most = (uint64_t)a.max_q_tokens * group;
    // Tiles of 128 query rows on the tensor cores from 17 rows on: where the other kernel
    // would read each key a third time (8 heads of 128, 20 rows of each of 16 sequences of
    // 16k: BF16 159 us, 248 there, E5M2 172 and 190, INT8 202 and 300, E2M1 190 and 273; of
    // 2 of 8k 25 to 30 in both).  One sequence that may have as many goes to them whatever
    // it has, and so does a batch whose single tokens have as many.
    p.few = most <= kFewRows || (a.batch > 1 && group <= kFewRows);
    p.upto = p.few ? kFewRows : 0;
    // Each pair of such tiles widens the slots that it reads.  With more than four pairs to
    // a sequence and head, widening its cache to FP16 ahead of them costs less; E5M2's bytes
    // are widened by a permute alone, in half the time, and at head_dim 128 the products
    // cover that up to eight pairs.  8 heads, 2 sequences of 16k, widened ahead and not, us:
    //   rows           512         1024        1536        2048        4096
    //   INT8  128    98   77    141  130    185  179    219  230
    //   INT8   64    69   59    102  101    131  139    163  182    293  350
    //   E2M1  128    94   75    136  129    181  181    215  231
    //   E5M2   64    68   55    101   94    131  129    162  168    292  323
    //   E5M2  128    97   71    139  119    184  167    219  210    392  405
    p.from = a.batch > 1 ? many_rows : 0;
    p.many = a.pool.format != SPLITZIP_FORMAT_BF16 && most > many_rows && widened_bytes(a, p.from) <= kMostWidened;
    p.some = most > kFewRows && !(p.many && a.batch == 1);
    if (!p.many) p.from = 0xFFFFFFFFu;
    if (p.few && !paged_rows_plan(a, p.upto, p.rows)) return false;
    if (p.some && !paged_tiles_plan(a, p.upto, p.from, p.tiles)) return false;
    if (p.many && !paged_tiles_plan(a, p.from, 0xFFFFFFFFu, p.wide)) return false;
    const auto after = [](size_t at, size_t bytes) { return (at + bytes + 127) / 128 * 128; };
    p.at_tiles = after(p.few ? p.rows.bytes : kAttentionHeader, 0);
    p.at_wide = after(p.at_tiles, p.some ? p.tiles.bytes : 0);
    p.at_widened = after(p.at_wide, p.many ? p.wide.bytes : 0);
    p.bytes = p.at_widened + (p.many ? widened_bytes(a, p.from) : 0);
    return true;
}

// The call as users make it and (test) with a copy left out.
splitzip_status attention(const splitzip_paged_attention_args* a, void* workspace, size_t workspace_bytes, splitzip_stream_t s, const WaitTest& test) {
    Plans p;
    if (!a || !sizes_ok(*a) || !plan(*a, p) || !pool_ok(a->pool)) return SPLITZIP_ERR_INVALID_ARG;
    if (!view_ok(a->q, 2, 1, a->tokens, a->q_heads) || !view_ok(a->out, 2, 1, a->tokens, a->q_heads, true)) return SPLITZIP_ERR_INVALID_ARG;
    if (!a->table || !a->q_start || !a->lens || !aligned(a->table, 4) || !aligned(a->q_start, 4) || !aligned(a->lens, 4) ||
        !aligned(a->lse, 4) || !std::isfinite(a->scale) || !(a->scale > 0.0f))
        return SPLITZIP_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < p.bytes) return SPLITZIP_ERR_INVALID_ARG;
    const cudaStream_t stream = (cudaStream_t)s;
    cudaError_t e = cudaSuccess;
    if (p.many) {
        void* wide = static_cast<uint8_t*>(workspace) + p.at_widened;
        e = launch_paged_widen(*a, p.from, wide, stream);
        if (e == cudaSuccess) e = launch_paged_tiles(*a, p.from, 0xFFFFFFFFu, p.wide, workspace, p.at_wide, wide, false, test, stream);
    }
    if (e == cudaSuccess && p.some) e = launch_paged_tiles(*a, p.upto, p.from, p.tiles, workspace, p.at_tiles, nullptr, p.many, test, stream);
    if (e == cudaSuccess && p.few) e = launch_paged_rows(*a, p.upto, p.rows, workspace, p.many || p.some, test, stream);
    return from_cuda(e);
}

}  // namespace

extern "C" {

splitzip_status splitzip_pages_store(const splitzip_pages_store_args* a, splitzip_stream_t s) {
    TraceRange trace("splitzip_pages_store");
    if (!a || !pool_sizes_ok(a->pool) || (uint64_t)a->n * a->pool.kv_heads > kMax31) return SPLITZIP_ERR_INVALID_ARG;
    if (!a->n) return SPLITZIP_OK;
    if (!pool_ok(a->pool) || !view_ok(a->k, 2, 1, a->n, a->pool.kv_heads) || !view_ok(a->v, 2, 1, a->n, a->pool.kv_heads) ||
        !a->slots || !aligned(a->slots, 8))
        return SPLITZIP_ERR_INVALID_ARG;
    return from_cuda(launch_pages_store(*a, (cudaStream_t)s));
}

splitzip_status splitzip_pages_load(const splitzip_pages_load_args* a, splitzip_stream_t s) {
    TraceRange trace("splitzip_pages_load");
    if (!a || !pool_ok(a->pool) || !a->batch || !a->tokens || a->tokens > kMostTokens) return SPLITZIP_ERR_INVALID_ARG;
    const uint32_t e = a->out_format == SPLITZIP_FORMAT_E5M2 ? 1 : 2;
    if (a->out_format != SPLITZIP_FORMAT_BF16 && (e == 2 || a->pool.format != SPLITZIP_FORMAT_E5M2)) return SPLITZIP_ERR_INVALID_ARG;
    if (a->tokens > (uint64_t)a->table_width * a->pool.page_tokens || (uint64_t)a->batch * a->pool.kv_heads > kMax31 ||
        2ull * a->batch * a->pool.kv_heads > kMax31 / ((a->tokens + 31) / 32))
        return SPLITZIP_ERR_INVALID_ARG;
    if (!a->table || !aligned(a->table, 4) || !aligned(a->lens, 4) ||
        !view_ok(a->k_out, e, a->batch, a->tokens, a->pool.kv_heads, true) ||
        !view_ok(a->v_out, e, a->batch, a->tokens, a->pool.kv_heads, true))
        return SPLITZIP_ERR_INVALID_ARG;
    return from_cuda(launch_pages_load(*a, (cudaStream_t)s));
}

size_t splitzip_paged_attention_workspace_bytes(const splitzip_paged_attention_args* a) {
    Plans p;
    return a && sizes_ok(*a) && plan(*a, p) ? p.bytes : 0;
}

splitzip_status splitzip_paged_attention(const splitzip_paged_attention_args* a, void* workspace, size_t workspace_bytes,
                                         splitzip_stream_t s) {
    TraceRange trace("splitzip_paged_attention");
    return attention(a, workspace, workspace_bytes, s, WaitTest());
}

splitzip_status splitzip_paged_attention_test(const splitzip_paged_attention_args* a, void* workspace, size_t workspace_bytes,
                                              splitzip_stream_t s, const splitzip_wait_test_opts* opts) {
    WaitTest test;
    return wait_test(opts, test) ? attention(a, workspace, workspace_bytes, s, test) : SPLITZIP_ERR_INVALID_ARG;
}

}  // extern "C"
