// attention_tiles.cu -- attention of many query rows over strided caches (sm_103a):
// where its work and its rows lie, and its plan.  The kernel is attention_tiles.cuh.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "attention_tiles.cuh"

namespace splitzip {
namespace {

struct TilesParams {
    splitzip_attention_args a;
    CUtensorMap qmap, kmap, vmap;
    uint32_t group, tokens;   // query tokens per tile: 128 / group
    uint32_t row_ctas, splits;
    uint32_t one_q, one_k, one_v;  // the batch is one sequence: coordinate 0
    uint32_t* status;
    uint32_t wait_limit;
    uint32_t test_cta, test_tile;  // a copy that a test has left out

    static constexpr bool kPaged = false;
    __device__ __forceinline__ uint32_t raw_arrivals() const { return 1; }
    // This CTA's part of the work: one thread.  The last row tiles see the most slots: they go first.
    template <bool kTwin>
    __device__ __forceinline__ void place(TilesShared& sh) const {
        const uint32_t unit = blockIdx.x / splits, split = blockIdx.x - unit * splits;
        const uint32_t heads = a.batch * a.kv_heads, rc = row_ctas - 1 - unit / heads, bh = unit % heads;
        sh.b = bh / a.kv_heads;
        sh.h = bh - sh.b * a.kv_heads;
        set_work<kTwin>(sh, Mask(a, sh.b), rc * 2 * tokens, a.q_tokens, tokens, [&](uint32_t n, uint32_t& j0, uint32_t& j1) {
            j0 = (uint32_t)((uint64_t)n * split / splits);
            j1 = (uint32_t)((uint64_t)n * (split + 1) / splits);
        });
    }
    // Where query token tok and query head hq of this CTA's sequence lie.
    __device__ __forceinline__ uint32_t queries(const TilesShared&) const { return a.q_tokens; }
    __device__ __forceinline__ const __nv_bfloat16* query(const TilesShared& sh, uint32_t tok, uint32_t hq) const {
        return static_cast<const __nv_bfloat16*>(a.q.data) + (int64_t)sh.b * a.q.stride_b + (int64_t)tok * a.q.stride_t + (int64_t)hq * a.q.stride_h;
    }
    __device__ __forceinline__ __nv_bfloat16* out(const TilesShared& sh, uint32_t tok, uint32_t hq) const {
        return static_cast<__nv_bfloat16*>(a.out.data) + (int64_t)sh.b * a.out.stride_b + (int64_t)tok * a.out.stride_t +
               (int64_t)hq * a.out.stride_h;
    }
    __device__ __forceinline__ float* lse(const TilesShared& sh, uint32_t tok, uint32_t hq) const {
        return a.lse + ((uint64_t)sh.b * a.q_heads + hq) * a.q_tokens + tok;
    }
    // The rows of this CTA's values by slot.
    struct Row {
        const uint8_t *data, *exponents;
    };
    template <int kElem>
    __device__ __forceinline__ auto values(const TilesShared& sh) const {
        const uint8_t* base = static_cast<const uint8_t*>(a.v.data) + ((int64_t)sh.b * a.v.stride_b + (int64_t)sh.h * a.v.stride_h) * kElem;
        return [base, this](int32_t s) { return Row{base + s * a.v.stride_t * kElem, nullptr}; };
    }
};

}  // namespace

// All rows in one tile, and slots for two: both tiles of a CTA hold the rows and take every other slot tile.
inline bool is_twin(const splitzip_attention_args& a) {
    return a.q_tokens <= kTileM / (a.q_heads / a.kv_heads) && a.kv_tokens > kBN;
}

uint32_t attention_tiles_splits(uint64_t units, uint64_t most, uint64_t at_once, uint64_t* steps) {
    // The splits (one cluster) with the least time, as waves of clusters times the steps
    // of a split plus kSplitCost steps for a CTA's start, join and end.  A cluster lies
    // within one of the GPU's groups of SMs, so fewer of the large ones run at once (as
    // cudaOccupancyMaxActiveClusters has it): 16 units of 2048 slots of 64 take 20.6 us
    // in 8 splits, two waves, and 11.7 in 6.
    constexpr uint64_t kAtOnce[9] = {0, kSms, 76, 46, 36, 28, 23, 15, 15};
    uint64_t best = ~0ull;
    uint32_t splits = 1;
    for (uint64_t n = 1; n <= 8 && (n == 1 || 2 * n <= most); n++) {
        const uint64_t time = (units + kAtOnce[n] - 1) / kAtOnce[n] * (((most + n - 1) / n + at_once - 1) / at_once + kSplitCost);
        if (time < best) {
            best = time;
            splits = (uint32_t)n;
        }
    }
    if (steps) *steps = best;
    return splits;
}

bool attention_tiles_plan(const splitzip_attention_args& a, AttentionPlan& p) {
    const uint32_t group = a.q_heads / a.kv_heads, tokens = kTileM / group;
    p.rows = a.q_tokens * group;
    p.tile_rows = 2 * tokens * group;
    p.row_tiles = (a.q_tokens + 2 * tokens - 1) / (2 * tokens);
    const uint64_t units = (uint64_t)a.batch * a.kv_heads * p.row_tiles, at_once = is_twin(a) ? 2 : 1;
    // The tiles of slots a CTA's rows can see at most.
    uint64_t most = (a.kv_tokens + kBN - 1) / kBN;
    if (a.window)
        most = std::min(most, ((uint64_t)a.window + 2 * tokens + kBN - 1) / kBN + 1 + ((uint64_t)a.sinks + kBN - 1) / kBN);
    p.splits = attention_tiles_splits(units, most, at_once);
    p.bytes = kAttentionHeader;
    return units * p.splits <= 0x7FFFFFFFull;
}

bool attention_tiles_usable(const splitzip_attention_args& a) {
    return a.scale > 0.0f;  // maxima are taken before scaling
}

cudaError_t launch_attention_tiles(const splitzip_attention_args& a, const AttentionPlan& plan, void* workspace,
                                   const WaitTest& test, cudaStream_t s) {
    TilesParams p;
    p.a = a;
    p.group = a.q_heads / a.kv_heads;
    p.tokens = kTileM / p.group;
    p.row_ctas = plan.row_tiles;
    p.splits = plan.splits;
    p.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kAttentionStatus);
    p.wait_limit = test.limit ? test.limit : wait_limit(0);  // a wait lasts a few steps at most
    p.test_cta = test.cta;
    p.test_tile = test.tile;
    const bool f8 = a.cache_format == SPLITZIP_FORMAT_E5M2;
    p.one_q = 1;
    if ((!f8 && !make_map(p.qmap, a.q, 2, a.head_dim, a.q_heads, a.q_tokens, a.batch, p.group, p.tokens, true, &p.one_q)) ||
        !make_map(p.kmap, a.k, f8 ? 1 : 2, a.head_dim, a.kv_heads, a.kv_tokens, a.batch, 1, kBN, false, &p.one_k) ||
        !make_map(p.vmap, a.v, f8 ? 1 : 2, a.head_dim, a.kv_heads, a.kv_tokens, a.batch, 1, kBN, false, &p.one_v))
        return cudaErrorInvalidValue;
    const uint32_t ctas = a.batch * a.kv_heads * plan.row_tiles * plan.splits;
    const auto go = [&](auto twin) {
        constexpr bool kTwin = decltype(twin)::value;
        if (a.head_dim == 64) return f8 ? launch_tiles<64, kE5m2, kTwin>(p, ctas, s) : launch_tiles<64, kBf16, kTwin>(p, ctas, s);
        return f8 ? launch_tiles<128, kE5m2, kTwin>(p, ctas, s) : launch_tiles<128, kBf16, kTwin>(p, ctas, s);
    };
    return is_twin(a) ? go(std::true_type()) : go(std::false_type());
}

}  // namespace splitzip
