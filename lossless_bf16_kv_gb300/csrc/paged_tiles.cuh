// paged_tiles.cuh -- attention of many query rows over pages (sm_103a): where the
// work and the rows of attention_tiles.cuh lie when the queries are packed and the
// cache is in pages.
//
// A CTA's row tiles belong to one sequence.  How many a batch has is on the device,
// so the grid is as large as it can be, each CTA counts the sequences' row tiles up
// to its own, and those past the last one leave.  Row tiles that do not fill a last wave
// of CTAs are cut into pieces.
//
// A tile of 128 slots is loaded page by page, one TMA box of up to 128 rows each, by as
// many lanes of a loading warp, one for the keys and one for the values; where tiles of
// head_dim 128 are widened they come in two parts, so that four of these fit beside the
// widened ones.  Quantised codes are widened to FP16 in shared memory as E5M2 ones are, by
// eight warps; their exponent bytes come with their tile, on the same barrier: one bulk
// copy a page where they are contiguous, else 4 bytes a lane.
//
// BF16 caches run as strided ones do (a chunk of 4096 after 12k tokens, 32 heads over 8 of
// 128: 632 us, 1.5 PFLOP/s, with pages of 16 and of 128 slots alike).  The widening warps
// bound the others: a chunk of 2048 in 8k tokens of 8 bits takes 215 us, where one over a
// BF16 cache takes 177, and 188 with the cache widened to FP16 ahead of the products.
#pragma once

#include "attention_tiles.cuh"

namespace splitzip {

struct PagedTilesParams {
    splitzip_paged_attention_args a;
    CUtensorMap qmap, kmap, vmap;
    uint32_t group, tokens;    // query tokens per tile: 128 / group
    uint32_t splits;           // a cluster's
    float4* partials;          // of pieces of work, or NULL: no CTA's is cut
    uint32_t* counters;        // a byte for each row tile that is cut
    uint32_t box, boxes;       // slots to a TMA box, and boxes to a tile
    uint32_t page_shift;
    uint32_t bulk_exps;        // a page's exponent bytes of a head are contiguous, in multiples of 16 bytes
    uint32_t slot_mask;        // of a slot within its page
    uint32_t rows_from, rows_upto;  // only sequences with more query rows than the one, up to the other
    uint32_t widened;          // the pool holds one page for each of these sequences, in their order
    uint32_t* status;
    uint32_t wait_limit;
    uint32_t test_cta, test_tile;  // a copy that a test has left out

    static constexpr bool kPaged = true;
    // The most pieces of a row tile, and the least slot tiles of one that is cut.
    static constexpr uint32_t kMostPieces = 16, kLeastCut = 24;
    // On a raw tile's barrier: its copies', and the lanes' whose own copies bring the exponents.
    __device__ __forceinline__ uint32_t raw_arrivals() const { return (a.pool.format == kInt8 || a.pool.format == kE2m1) && !bulk_exps ? 33 : 1; }
    // Row-tile CTAs of a sequence.
    template <bool kTwin>
    __device__ __forceinline__ uint32_t ctas_of(uint32_t b) const {
        if (b >= a.batch) return 0;
        const uint32_t count = (uint32_t)sequence_count(a, a.q_start[b], a.q_start[b + 1]), per = kTwin ? tokens : 2 * tokens;
        return count * group > rows_from && count * group <= rows_upto ? (count + per - 1) / per : 0;
    }
    // Which of `units` row tiles a CTA takes, and which piece of it.
    struct Part {
        uint32_t unit, piece, pieces, first_piece, counter;
        bool thirds;  // two pieces, the first of two thirds
    };
    // A CTA fills an SM, so `units` of about the same work take whole waves of kSms and one
    // that is not full, whose row tiles are cut: into equal pieces where there are two or more
    // SMs to each, else, up to two thirds of a wave, into a piece of two thirds and one of the
    // rest, two of which an SM without a large one takes in turn.  Pieces are joined through
    // memory, which costs 10 us (a cluster's splits half of that, but few clusters run at
    // once): worth it from 24 slot tiles on, 48 where it saves a third, in at most as many
    // pieces as those have steps.  A chunk in 16k of BF16, 32 heads over 8 of 128, cut and not:
    // 80 row tiles 149 us and 187, 160 237 and 291, 192 269 and 300, 232 338 and 356; 256, as
    // pieces of three and one quarter, 371 and 362, so those are not.
    __device__ __forceinline__ Part part_of(uint32_t units) const {
        // Where ranges that overlap make more of them than the grid is for, none is cut: a piece
        // that no CTA takes would leave its counter behind.
        const bool cut = partials && units + kSms <= gridDim.x;
        const uint32_t i = blockIdx.x, whole = cut ? units - units % kSms : units, rest = units - whole;
        if (i < whole || !rest || rest > kSms * 2 / 3) return {i, 0, 1, 0, 0, false};
        const uint32_t j = i - whole;
        if (rest <= kSms / 2) {
            const uint32_t n = min(kSms / rest, kMostPieces), r = j / n;
            return {r < rest ? whole + r : units, j - r * n, n, r * n, r, false};
        }
        const uint32_t r = j < rest ? j : j - rest;
        return {r < rest ? whole + r : units, j < rest ? 0u : 1u, 2, 2 * r, r, true};
    }
    // This CTA's part of the work: one warp.  count stays 0 where there is none.  The last
    // sequence's last tiles, which see the most of its slots, go first.
    template <bool kTwin>
    __device__ __forceinline__ void place(TilesShared& sh, uint32_t lane) const {
        uint32_t total = 0;
        for (uint32_t b = 0; b < a.batch; b += 32) total += __reduce_add_sync(0xFFFFFFFFu, ctas_of<kTwin>(b + lane));
        Part part;
        if (kTwin || splits > 1) part = {blockIdx.x / splits, blockIdx.x % splits, splits, 0, 0, false};
        else part = part_of(total * a.pool.kv_heads);
        const uint32_t h = part.unit % a.pool.kv_heads, at = part.unit / a.pool.kv_heads;
        if (lane == 0) sh.count = 0;
        if (at >= total) return;
        uint32_t left = total - 1 - at, before = 0;  // row tiles, and sequences, before this one
        for (uint32_t b = 0; b < a.batch; b += 32) {
            const uint32_t mine = ctas_of<kTwin>(b + lane), some = __ballot_sync(0xFFFFFFFFu, mine != 0);
            uint32_t upto = mine;
#pragma unroll
            for (int i = 1; i < 32; i *= 2) {
                const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, upto, i);
                if (lane >= (uint32_t)i) upto += x;
            }
            const uint32_t found = __ballot_sync(0xFFFFFFFFu, left < upto);
            if (!found) {
                left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
                before += __popc(some);
                continue;
            }
            if (lane == (uint32_t)__ffs(found) - 1) {
                const Sequence seq(a, b + lane);
                sh.b = b + lane;
                sh.h = h;
                sh.first_row = seq.row;
                sh.count = seq.count;
                sh.rank = before + __popc(some & ((1u << lane) - 1u));
                set_work<kTwin>(sh, Mask(seq.n, seq.count, a.window, a.sinks), (left - (upto - mine)) * (kTwin ? tokens : 2 * tokens),
                                (uint32_t)seq.count, tokens, [&](uint32_t n, uint32_t& j0, uint32_t& j1) {
                    uint32_t pieces = part.pieces;
                    if (!kTwin && splits == 1) {
                        if (n < (part.thirds ? 2 : 1) * kLeastCut) pieces = 1;
                        while (pieces * pieces > n && pieces > 1) pieces--;
                        sh.piece = part.piece, sh.pieces = pieces, sh.first_piece = part.first_piece, sh.counter = part.counter;
                        if (part.piece >= pieces) sh.count = 0;  // another one has it all
                    }
                    const auto upto = [&](uint32_t x) {
                        return part.thirds && pieces > 1 ? x == 1 ? n - n / 3 : x * n / 2 : (uint32_t)((uint64_t)n * x / pieces);
                    };
                    j0 = upto(part.piece), j1 = upto(part.piece + 1);
                });
            }
            return;
        }
    }
    // Where query token tok and query head hq of this CTA's sequence lie.
    __device__ __forceinline__ uint32_t queries(const TilesShared& sh) const { return (uint32_t)sh.count; }
    __device__ __forceinline__ const __nv_bfloat16* query(const TilesShared& sh, uint32_t tok, uint32_t hq) const {
        return static_cast<const __nv_bfloat16*>(a.q.data) + (int64_t)(sh.first_row + tok) * a.q.stride_t + (int64_t)hq * a.q.stride_h;
    }
    __device__ __forceinline__ __nv_bfloat16* out(const TilesShared& sh, uint32_t tok, uint32_t hq) const {
        return static_cast<__nv_bfloat16*>(a.out.data) + (int64_t)(sh.first_row + tok) * a.out.stride_t + (int64_t)hq * a.out.stride_h;
    }
    __device__ __forceinline__ float* lse(const TilesShared& sh, uint32_t tok, uint32_t hq) const {
        return a.lse + (uint64_t)hq * a.tokens + sh.first_row + tok;
    }
    // Whether a query of this CTA may see one of the slots s .. s + run - 1.
    __device__ __forceinline__ bool run_seen(const volatile TilesShared& sh, int32_t s, uint32_t run) const {
        return s <= sh.p1 && ((int64_t)s + run > (int64_t)sh.p0 - (int64_t)sh.window + 1 || s < sh.sinks);
    }
    __device__ __forceinline__ uint32_t page(const volatile TilesShared& sh, int32_t s) const {
        return widened ? sh.rank : (uint32_t)a.table[(uint64_t)sh.b * a.table_width + ((uint32_t)s >> page_shift)];
    }
    // The rows of this CTA's values by slot; none where the page is outside the pool.
    struct Row {
        const uint8_t *data, *exponents;
    };
    template <int kElem>
    __device__ __forceinline__ auto values(const TilesShared& sh) const {
        return [&sh, this](int32_t s) {
            const splitzip_page_rows& v = a.pool.v;
            const uint32_t x = page(sh, s);
            if (x >= a.pool.pages) return Row{nullptr, nullptr};
            const int64_t at = (uint32_t)s & slot_mask;
            return Row{static_cast<const uint8_t*>(v.data) + (x * v.stride_p + at * v.stride_t + (int64_t)sh.h * v.stride_h) * kElem,
                       v.exponents + x * v.exp_stride_p + at * v.exp_stride_t + (int64_t)sh.h * v.exp_stride_h};
        };
    }
};

// Slots of a part that a tile is loaded in.
template <int D>
uint32_t tile_part_of(uint32_t format) {
    return format == kBf16 || format == kF16 ? TilesShape<D, kBf16, true>::kPartSlots
           : format == kE5m2 ? TilesShape<D, kE5m2, true>::kPartSlots
           : format == kInt8 ? TilesShape<D, kInt8, true>::kPartSlots
                             : TilesShape<D, kE2m1, true>::kPartSlots;
}
inline uint32_t tile_part(const splitzip_pool& p) { return p.head_dim == 64 ? tile_part_of<64>(p.format) : tile_part_of<128>(p.format); }

template <int D, bool kTwin>
cudaError_t launch_paged_format(const PagedTilesParams& p, uint32_t ctas, bool beside, cudaStream_t s) {
    switch (p.a.pool.format) {
        case kBf16: return launch_tiles<D, kBf16, kTwin>(p, ctas, s, beside);
        case kE5m2: return launch_tiles<D, kE5m2, kTwin>(p, ctas, s, beside);
        case kInt8: return launch_tiles<D, kInt8, kTwin>(p, ctas, s, beside);
        case kF16:  // of many rows, never twins
            if constexpr (kTwin) return cudaErrorInvalidValue;
            else return launch_tiles<D, kF16, kTwin>(p, ctas, s, beside);
        default: return launch_tiles<D, kE2m1, kTwin>(p, ctas, s, beside);
    }
}
// One for each head_dim and kind of tile, compiled side by side.
cudaError_t launch_paged_64(const PagedTilesParams& p, uint32_t ctas, bool beside, cudaStream_t s);
cudaError_t launch_paged_64_twin(const PagedTilesParams& p, uint32_t ctas, bool beside, cudaStream_t s);
cudaError_t launch_paged_128(const PagedTilesParams& p, uint32_t ctas, bool beside, cudaStream_t s);
cudaError_t launch_paged_128_twin(const PagedTilesParams& p, uint32_t ctas, bool beside, cudaStream_t s);

}  // namespace splitzip
