// attention_tiles.cuh -- attention of many query rows on the tensor cores
// (sm_103a), over strided caches (attention_tiles.cu) and pages (paged_tiles.cu).
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
// 2 x 512 cycles at head_dim 128, the 128 x 128 exponentials 512; a tile's next
// S has to wait for its P (which lies over S), so the softmax's latency should
// stay near the 1024 cycles of the other tile's products.  Hence two threads to
// a row, 64 slots each.  The latency is what bounds it: of a step's 2900 cycles
// the softmax takes 1550 (scores into registers 280, their maximum 260,
// exponentials 850, settling 150), handing over 250, the products 1120.
//
// At head_dim 64 there is room for P beside S and O: S of the next step is made
// as soon as the softmax warps have this step's in registers, and their chain of
// about 2500 cycles a step does not wait for it.
//
// 8192 causal tokens, 32 heads over 8: head_dim 128 368 us (1.49 PFLOP/s visible)
// in BF16, 500 in E5M2; head_dim 64 271 (1.0) and 329.  16384 tokens in a window
// of 4096 with sinks, head_dim 128: 733-740 us (1.31), 940 in E5M2.
//
// Where one tile holds all rows, both tiles of a CTA are that one (twins): each
// takes every other tile of slots, and they are joined like splits.  64 rows over
// 128 caches of 16384 slots: head_dim 128 161 us, 6.7 TB/s (217 with the second
// tile empty), head_dim 64 92 (172).
//
// Roles: warps 0-15 softmax (four per tile and half of the slots), 16 issues
// the products of both tiles (from two warps they interleave and both tiles wait
// for both: 734 against 879 us at 16k), 17 the TMA loads; the rest keep
// infinities and NaN of partly visible tiles out of the second product (0 x
// infinity is not 0) and, for an E5M2 cache, widen its tiles to FP16 (exact: an
// E5M2 value is the upper byte of the FP16 value it stands for), half of these
// warps the keys, half the values, and in shared memory, as the products read
// it.  The queries are then FP16 too, each row scaled by a power of two.  Over pages
// warp 17 loads the keys alone, the values are another warp's, and eight warps widen
// (E5M2, and quantised codes times their powers, each value exact in FP16).
//
// What the roles share sits in shared memory and is read from there: a softmax
// thread's 104 registers (96 for E5M2) hold 64 scores and little else, and a value
// spilled in its loop costs hundreds of cycles in every step.  The compiler still
// spills 20 to 24 bytes a thread in the E5M2 kernels of head_dim 128, and 8 in the
// BF16 one of shared rows at 64.
//
// The running maximum is only raised when a row's maximum grows by more than
// 2^8 (in which case O and l are rescaled by the softmax warps, after the
// product that wrote O): P stays below 2^8, and the quotient O / l is the same.
// For an E5M2 cache P is FP16, which has fewer exponents: there it is up to 2^9 at
// a maximum just taken and 2^15.9 before the next, so that terms down to 2^-22 of a
// row's largest keep all bits and those below 2^-33 vanish (with 1 and 2^8 those
// below 2^-25 did, and 2^17 slots of them are 2^-8 of the sum).  Giving the growth
// less room costs steps that settle: 2^11 and 2^4 made 16384 tokens in a window
// behind sinks 1016 us, where 2^9 and 2^6.9 take 938, as 1 and 2^8 did.
// Each half of a row starts with the maximum that it would choose by itself, and
// the two settle after their exponentials: an exchange before them in every step
// cost 285 us where this takes 273.
#pragma once

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "attention.cuh"
#include "pages.cuh"
#include "tcgen.cuh"
#include "tensor_map.h"

namespace splitzip {

// Splits of `units` row tiles that see up to `most` tiles of slots and take `at_once` of them a
// step, and the steps that this takes in all.
constexpr uint64_t kSplitCost = 4;  // of a CTA, in steps
uint32_t attention_tiles_splits(uint64_t units, uint64_t most, uint64_t at_once, uint64_t* steps = nullptr);

constexpr int kBN = 128;       // slots per step
constexpr int kTileM = 128;    // query rows per tile
constexpr int kSoftmax = 512;  // threads
constexpr int kScoresOf = 16;  // scores turned into P at a time: eight words
// log2 of P at a maximum just taken, and of how far a P may exceed that.
template <bool kF8>
constexpr float kTilesLift = kF8 ? 9.0f : 0.0f;
template <bool kF8>
constexpr float kTilesLazy = kF8 ? 6.9f : 8.0f;

template <int D, int kFmt, bool kPaged>
struct TilesShape {
    static constexpr int kKV = kBN * D * 2;      // bytes of a key or value tile in 16 bits
    // Where it is widened, a tile comes as it lies in the cache, in one part or two, of kRaw bytes and kExps of exponents.
    static constexpr int kParts = kPaged && kWidens<kFmt> && D == 128 ? 2 : 1, kPartSlots = kBN / kParts;
    static constexpr int kRaw = kPartSlots * kRowBytes<D, kFmt>;
    static constexpr int kQ = kTileM * D * 2;    // bytes of a query tile
    static constexpr int kStages = D == 128 ? (kWidens<kFmt> || kPaged ? 4 : 5) : (kWidens<kFmt> ? 6 : 8);
    static constexpr int kRaws = !kWidens<kFmt> ? 0 : kPaged ? 4 : 2;
    static constexpr int kExps = kQuantised<kFmt> ? kPartSlots * 4 : 0;
    // Threads: softmax, a warp for the products, one for the loads, and those that
    // tend the values; registers of a softmax thread and of another.
    static constexpr bool kManyTend = kWidens<kFmt> && kPaged;
    static constexpr int kTend = kManyTend ? 10 : kWidens<kFmt> ? 6 : 2, kThreads = kSoftmax + 32 * (2 + kTend);
    static constexpr int kRegs = kWidens<kFmt> ? 96 : 104, kOtherRegs = kManyTend ? 40 : kWidens<kFmt> ? 48 : 64;
    // Warps that widen a tile, and those that say that its values are fit.
    static constexpr int kTenders = kManyTend ? 8 : kPaged ? 1 : kTend;  // the next one loads the values' pages
    static constexpr int kWiden = kTenders > 1 ? kTenders / 2 : 1, kFit = kWidens<kFmt> ? kWiden : kTenders;
    static_assert(kThreads % 128 == 0 && kSoftmax * kRegs + (kThreads - kSoftmax) * kOtherRegs <= kThreads * (65536 / kThreads / 8 * 8),
                  "register shares add up to what the CTA is launched with");
    static constexpr int kRowFloats = D + 4;     // of a row's partial result: o, m, l
    // Tensor memory: S of the query tiles from column 0, O, and P over S or apart.
    static constexpr bool kApart = D == 64;
    static constexpr uint32_t kColO = 2 * kBN, kColP = kApart ? kColO + 2 * D : 0, kStepP = kApart ? kBN / 2 : kBN;
    static constexpr uint32_t kHalfP = kApart ? kBN / 4 : kBN / 2;  // over S, each half of P over its own scores
    static constexpr int kUsed = 2 * kQ + kStages * kKV + kRaws * (kRaw + kExps);
    // Where exponents take the room, the two threads of a row exchange through one place.
    static constexpr bool kOneRow = kQuantised<kFmt>;
    static_assert(kUsed >= 2 * kTileM * kRowFloats * 4, "partial results take the place of the tiles");
};

struct TilesShared {
    uint64_t full[8], empty[8];  // ring stage: tile there in 16 bits, free again
    uint64_t ok[8];              // step i mod 8: its values are fit for the product
    uint64_t raw_full[4], raw_empty[4];  // tiles as they lie in the cache
    uint64_t q_full;
    uint64_t s_full[2], p_full[2], o_full[2], drained;  // of the query tiles
    uint64_t s_free[2], o_done[2];  // P apart: S is in registers, a step's O is there
    WaitLimit wait;
    uint32_t tmem, odd, lost;  // lost: a page that a query sees is outside the pool
    // This CTA's work: sequence, head, first query token; the first slot of step
    // 0, the step that jumps from the sinks to the window and to where.
    uint32_t b, h, t0, steps;
    int32_t first_row, count;  // a packed sequence's first query token, and their number
    uint32_t rank;             // its number among those of the launch
    // Pieces of this CTA's work, joined through memory: which one, of how many; the first
    // one's place there, and the counter.
    uint32_t piece, pieces, first_piece, counter, last;
    int32_t s0, jump_at, jump_to;
    int32_t n, first, sinks, p0, p1;
    uint32_t window;
    int32_t upto[2], after[2], whole_sinks;  // WholeTiles of the query tiles
    float row[2][2][kTileM];  // [half][tile]: exchanged by the two threads of a row, the second half where there is room
};

// The first slot of each step in turn.
struct StepSlots {
    int32_t s0, at, to, i;
    __device__ __forceinline__ explicit StepSlots(const volatile TilesShared& sh)
        : s0(sh.s0), at(sh.jump_at), to(sh.jump_to), i(0) {}
    __device__ __forceinline__ void next() { s0 = ++i == at ? to : s0 + kBN; }
};
// The first slot of step j.
__device__ __forceinline__ int32_t step_slot(const volatile TilesShared& sh, int32_t j) {
    const int32_t at = sh.jump_at;
    return at < 0 || j < at ? sh.s0 + j * kBN : sh.jump_to + (j - at) * kBN;
}
// The tiles of slots that every query of [p0, p1] sees, from the tile's first slot.
struct WholeTiles {
    int32_t upto, after, sinks;
    __device__ __forceinline__ WholeTiles(const volatile TilesShared& sh, int32_t p0, int32_t p1) {
        upto = p0 - (kBN - 1);
        const int64_t back = (int64_t)p1 - (int64_t)sh.window;
        after = back < -1 ? -1 : (int32_t)back;
        sinks = sh.sinks - kBN;
    }
    __device__ __forceinline__ bool operator()(int32_t s0) const { return s0 <= upto && (s0 > after || s0 <= sinks); }
};

// The other thread's value of the two of a row, both of which call it; `there`: this
// thread's has been left already (where it leaves it first), and a barrier passed.
template <bool kOneRow>
__device__ __forceinline__ float exchange(TilesShared& sh, uint32_t t, uint32_t half, uint32_t r, uint32_t bar, float v, bool there = false) {
    if (!there) {
        if (!kOneRow || !half) sh.row[half][t][r] = v;
        named_sync(bar, 64);
    }
    if (!kOneRow) return sh.row[half ^ 1][t][r];
    float other = 0.0f;
    if (half) {
        other = sh.row[0][t][r];
        sh.row[0][t][r] = v;
    }
    named_sync(bar, 64);
    if (!half) other = sh.row[0][t][r];
    return other;
}

// What a CTA's query tokens from t0 on, of `count`, walk: of the slot tiles that they see
// those from j0 to j1 - 1, as cut(their number, j0, j1) has it.
template <bool kTwin, class Cut>
__device__ __forceinline__ void set_work(TilesShared& sh, const Mask& mask, uint32_t t0, uint32_t count, uint32_t tokens, const Cut& cut) {
    const uint32_t t1 = min(t0 + 2 * tokens, count);
    sh.p0 = mask.first + (int32_t)t0;
    sh.p1 = mask.first + (int32_t)t1 - 1;
    const SlotTiles tiles(mask, sh.p0, sh.p1, kBN);
    uint32_t j0, j1;
    cut(tiles.count, j0, j1);
    sh.t0 = t0;
    sh.steps = j1 - j0;
    sh.s0 = (int32_t)(tiles.tile(j0) * kBN);
    sh.jump_at = j0 < tiles.head ? (int32_t)(tiles.head - j0) : -1;
    sh.jump_to = (int32_t)(tiles.from * kBN);
    sh.n = mask.n;
    sh.first = mask.first;
    sh.sinks = mask.sinks;
    sh.window = mask.window;
    for (int t = 0; t < 2; t++) {
        // All tiles of slots are whole for a tile without queries: its rows go nowhere, and
        // masking every step would make it the CTA's slower one.
        const uint32_t ta = t0 + (kTwin ? 0 : t * tokens), tb = min(ta + tokens, count);
        const WholeTiles whole(sh, mask.first + (int32_t)ta, mask.first + (int32_t)tb - 1);
        sh.upto[t] = ta < count ? whole.upto : 0x7FFFFFFF;
        sh.after[t] = ta < count ? whole.after : -1;
        sh.whole_sinks = whole.sinks;
    }
}

// Bits of the slots s0 .. s0 + 31 that a query sees: those from `lo` (the start
// of its window) to `pos`, and the first `sinks`.
__device__ __forceinline__ uint32_t seen_bits(int32_t pos, int32_t lo, int32_t sinks, int32_t s0) {
    const int32_t hi = pos - s0, l = lo - s0, k = sinks - s0;
    const uint32_t upto = hi < 0 ? 0u : hi >= 31 ? 0xFFFFFFFFu : ~(0xFFFFFFFEu << hi);
    const uint32_t from = l <= 0 ? 0xFFFFFFFFu : l > 31 ? 0u : 0xFFFFFFFFu << l;
    const uint32_t sink = k <= 0 ? 0u : k > 31 ? 0xFFFFFFFFu : ~(0xFFFFFFFFu << k);
    return upto & (from | sink);
}

// ------------------------------------------------------------------ roles

// The query tiles, from token `first` of the tensor on.
template <int D, int kFmt, bool kTwin, class Params>
__device__ __forceinline__ void load_queries(const Params& p, TilesShared& sh, uint8_t* qs, uint32_t first, int32_t b) {
    using S = TilesShape<D, kFmt, Params::kPaged>;
    mbar_arrive_expect_tx(&sh.q_full, 2 * p.tokens * p.group * D * 2);
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int i = 0; i < D / 64; i++)
            tma_load4(qs + t * S::kQ + i * (kTileM * 128), &p.qmap, 64 * i, (int32_t)sh.h * (int32_t)p.group,
                      (int32_t)(first + (kTwin ? 0 : t * p.tokens)), b, &sh.q_full);
}

template <int D, int kFmt, bool kTwin, class Params>
__device__ __forceinline__ void load_tiles(const Params& p, TilesShared& sh, uint8_t* qs, uint8_t* ring, uint8_t* raw) {
    using S = TilesShape<D, kFmt, Params::kPaged>;
    volatile WaitLimit* wait = &sh.wait;
    const int32_t b = (int32_t)sh.b, h = (int32_t)sh.h;
    const uint32_t steps = sh.steps;
    if (!kWide<kFmt>) load_queries<D, kFmt, kTwin>(p, sh, qs, sh.t0, p.one_q ? 0 : b);
    constexpr int kN = kWide<kFmt> ? S::kRaws : S::kStages;
    uint64_t* full = kWide<kFmt> ? sh.raw_full : sh.full;
    uint64_t* empty = kWide<kFmt> ? sh.raw_empty : sh.empty;
    StepSlots slots(sh);
    const uint32_t left_out = blockIdx.x == p.test_cta ? p.test_tile : 0xFFFFFFFFu;
    uint32_t i = 0;
    for (uint32_t st = 0, ph = 0; i < 2 * steps; i++) {
        if (i >= kN && !mbar_wait_bounded(&empty[st], ph ^ 1, wait)) break;
        const bool v = i & 1;
        const int32_t bb = (v ? p.one_v : p.one_k) ? 0 : b;
        mbar_arrive_expect_tx(&full[st], kWide<kFmt> ? S::kRaw : S::kKV);
        if (i == left_out) {
        } else if (kWide<kFmt>) {
            tma_load4(raw + st * S::kRaw, v ? &p.vmap : &p.kmap, 0, slots.s0, h, bb, &full[st]);
        } else {
#pragma unroll
            for (int x = 0; x < D / 64; x++)
                tma_load4(ring + st * S::kKV + x * (kBN * 128), v ? &p.vmap : &p.kmap, 64 * x, slots.s0, h, bb, &full[st]);
        }
        if (v) slots.next();
        if (++st == kN) st = 0, ph ^= 1;
    }
    // Every load has landed before this CTA may end, also where a wait gave up.
    if (!kWide<kFmt>) mbar_wait_bounded<true>(&sh.q_full, 0, wait);
    for (uint32_t x = i > kN ? i - kN : 0; x < i; x++) mbar_wait_bounded<true>(&full[x % kN], (x / kN) & 1, wait);
}

// The keys' tiles, or the values', from pages, a tile being one or more boxes of
// slots of one page each: lane i of the warp looks up and loads box i, the page from one
// step ahead.  What no query sees, or lies outside the pool, is loaded from behind its
// last page: as zeros.  The keys have one warp and the values another, as a tile of pages
// of 16 slots is 16 copies of each (a chunk of 4096 over 16k, not cut: 684 us, with one 837).
template <int D, int kFmt, bool kTwin, class Params>
__device__ __forceinline__ void load_page_tiles(const Params& p, TilesShared& sh, uint8_t* qs, uint8_t* ring, uint8_t* raw, bool values, uint32_t lane) {
    using S = TilesShape<D, kFmt, Params::kPaged>;
    constexpr int kRow = kWidens<kFmt> ? kRowBytes<D, kFmt> : 128;  // bytes of a row of a box
    volatile WaitLimit* wait = &sh.wait;
    const uint32_t steps = sh.steps;
    if (!kWide<kFmt> && !values && lane == 0) load_queries<D, kFmt, kTwin>(p, sh, qs, (uint32_t)sh.first_row + sh.t0, 0);
    const auto look_up = [&](uint32_t j) {
        if (lane >= p.boxes || j >= steps) return p.a.pool.pages;
        const int32_t s = step_slot(sh, (int32_t)j) + (int32_t)(lane * p.box);
        if (!p.run_seen(sh, s, p.box)) return p.a.pool.pages;
        const uint32_t page = p.page(sh, s);
        if (page >= p.a.pool.pages) *const_cast<volatile uint32_t*>(&sh.lost) = 1;
        return min(page, p.a.pool.pages);
    };
    constexpr uint32_t kN = kWidens<kFmt> ? S::kRaws : S::kStages, kParts = S::kParts;
    uint64_t* full = kWidens<kFmt> ? sh.raw_full : sh.full;
    uint64_t* empty = kWidens<kFmt> ? sh.raw_empty : sh.empty;
    uint8_t* exps = raw + S::kRaws * S::kRaw;  // of each raw stage, by slot
    const bool bulk = kQuantised<kFmt> && p.bulk_exps;
    const CUtensorMap* map = values ? &p.vmap : &p.kmap;
    const splitzip_page_rows& rows = values ? p.a.pool.v : p.a.pool.k;
    const uint32_t part_boxes = p.boxes / kParts, slots_mask = p.slot_mask;
    uint32_t now = look_up(0), ahead = look_up(1);
    // Parts of the keys', values', next keys' .. tiles are numbered in turn.
    const uint32_t first = values ? kParts : 0;
    uint32_t i = 0;  // parts issued
    uint32_t st = first % kN, ph = 0;
    // No stage takes both keys and values: each warp then waits for every turn of its stages,
    // and no turn of another's passes unseen, after which a parity would say the opposite.
    static_assert(kN % (2 * kParts) == 0, "stages of keys and of values are apart");
    uint32_t m = first;
    for (; i < kParts * steps; i++) {
        const uint32_t step = i / kParts, part = i % kParts;
        if (m >= kN && !mbar_wait_bounded(&empty[st], ph ^ 1, wait)) break;
        const uint32_t s0 = (uint32_t)step_slot(sh, (int32_t)step) + part * S::kPartSlots;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], kWidens<kFmt> ? S::kRaw + (bulk ? S::kExps : 0) : S::kKV);
        __syncwarp();
        const uint32_t mine = lane - part * part_boxes;  // this lane's box of the part
        if (mine < part_boxes && !(blockIdx.x == p.test_cta && m == p.test_tile)) {
            const int32_t at = (int32_t)((s0 + mine * p.box) & slots_mask);
            if (kWidens<kFmt>) {
                tma_load4(raw + st * S::kRaw + mine * p.box * kRow, map, 0, at, (int32_t)sh.h, (int32_t)now, &full[st]);
            } else {
#pragma unroll
                for (int x = 0; x < D / 64; x++)
                    tma_load4(ring + st * S::kKV + x * (kBN * 128) + mine * p.box * kRow, map, 64 * x, at, (int32_t)sh.h, (int32_t)now, &full[st]);
            }
        }
        if (kQuantised<kFmt>) {  // where no query sees them, any page's: they multiply zeros
            const uint8_t* from = rows.exponents + (int64_t)sh.h * rows.exp_stride_h;
            uint8_t* to = exps + st * S::kExps;
            const uint32_t some = now < p.a.pool.pages ? now : 0;
            if (bulk) {
                if (mine < part_boxes)
                    bulk_load(to + 4 * mine * p.box, from + some * rows.exp_stride_p + 4 * ((s0 + mine * p.box) & slots_mask), 4 * p.box, &full[st]);
            } else {
#pragma unroll
                for (uint32_t r = lane; r < S::kPartSlots; r += 32) {
                    const int64_t page = __shfl_sync(0xFFFFFFFFu, some, part * part_boxes + r / p.box);
                    cp_async4(to + 4 * r, from + page * rows.exp_stride_p + ((s0 + r) & slots_mask) * rows.exp_stride_t);
                }
                cp_async_arrive(&full[st]);
            }
        }
        uint32_t on = 1;
        if (part == kParts - 1) {
            now = ahead;
            ahead = look_up(step + 2);
            on += kParts;
        }
        m += on;
        st += on;
        if (st >= kN) st -= kN, ph ^= 1;
    }
    // Every load has landed before this CTA may end, also where a wait gave up.
    if (!kWide<kFmt> && !values) mbar_wait_bounded<true>(&sh.q_full, 0, wait);
    // Of a stage the last turn: those of the last kN parts of both warps, where all have been
    // issued, else of this one's (a turn that is past already costs the failing CTA the limit).
    const uint32_t end = i == kParts * steps ? 2 * i : m;
    while (i--) {
        const uint32_t x = 2 * kParts * (i / kParts) + first + i % kParts;
        if (x + kN < end) break;
        mbar_wait_bounded<true>(&full[x % kN], (x / kN) & 1, wait);
    }
}

template <int D, int kFmt, bool kTwin, class Params>
__device__ __forceinline__ void issue_products(TilesShared& sh, uint32_t tmem, const uint8_t* qs, const uint8_t* ring) {
    using S = TilesShape<D, kFmt, Params::kPaged>;
    constexpr uint32_t kShapeS = mma_shape(kWide<kFmt>, kBN, false), kShapeO = mma_shape(kWide<kFmt>, D, true);
    volatile WaitLimit* wait = &sh.wait;
    const bool leader = elect_one();
    const uint32_t steps = sh.steps;
    const uint32_t qd = desc_rows(smem_addr(qs)), kd = desc_rows(smem_addr(ring)), vd = desc_columns(smem_addr(ring), kBN * 128);
    // One lane issues, in straight runs: S of query tile t from the keys in stage
    // st, and O += P V with the values in stage st.
    auto issue_s = [&](uint32_t t, uint32_t st) {
        const uint32_t qa = qd + t * (S::kQ >> 4), ka = kd + st * (S::kKV >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
            const uint32_t at = (k >> 2) * (kBN * 128) + (k & 3) * 32;
            mma_ss(tmem + t * kBN, desc(qa, at), desc(ka, at), kShapeS, k > 0);
        }
        mma_commit(&sh.s_full[t]);
    };
    auto issue_o = [&](uint32_t t, uint32_t st, bool add) {
        const uint32_t va = vd + st * (S::kKV >> 4);
        const uint32_t o = tmem + S::kColO + t * D, pa = tmem + S::kColP + t * S::kStepP;
        mma_ts(o, pa, desc(va, 0), kShapeO, add);
#pragma unroll
        for (int k = 1; k < kBN / 16; k++) mma_ts(o, pa + (k >> 2) * S::kHalfP + (k & 3) * 8, desc(va, k * 2048), kShapeO, true);
    };
    // Twins: slot tile j is tile j & 1's.  Its next keys are four stages on at most.
    static_assert(S::kStages >= 4, "the ring reaches from a slot tile's values to the next but one's keys");
    const auto run_twins = [&]() {
        const auto at = [](uint32_t n) { return n % S::kStages; };
        const auto loaded = [&](uint32_t n) { return mbar_wait_bounded(&sh.full[at(n)], (n / S::kStages) & 1, wait); };
        if (!mbar_wait_bounded(&sh.q_full, 0, wait)) return;
        for (uint32_t j = 0; j < min(steps, 2u); j++) {
            if (!loaded(2 * j)) return;
            tcgen_fence_after();
            if (leader) {
                issue_s(j, at(2 * j));
                mma_commit(&sh.empty[at(2 * j)]);
            }
            __syncwarp();
        }
        for (uint32_t j = 0; j < steps; j++) {
            const uint32_t t = j & 1, vst = at(2 * j + 1), kst = at(2 * j + 4), turn = (j >> 1) & 1;
            const bool more = j + 2 < steps;
            const auto next_s = [&]() {
                if (!loaded(2 * j + 4)) return false;
                tcgen_fence_after();
                if (leader) {
                    issue_s(t, kst);
                    mma_commit(&sh.empty[kst]);
                }
                __syncwarp();
                return true;
            };
            if (!mbar_wait_bounded(&sh.ok[j & 7], (j >> 3) & 1, wait) || !loaded(2 * j + 1)) return;
            if (S::kApart && more && !(mbar_wait_bounded(&sh.s_free[t], turn, wait) && next_s())) return;
            if (!mbar_wait_bounded(&sh.p_full[t], turn, wait)) return;
            tcgen_fence_after();
            if (leader) {
                issue_o(t, vst, j > 1);
                mma_commit(&sh.empty[vst]);
                if (S::kApart && more) mma_commit(&sh.o_done[t]);
                if (!more) mma_commit(&sh.o_full[t]);
                if (steps == 1) mma_commit(&sh.o_full[1]);
            }
            __syncwarp();
            if (!S::kApart && more && !next_s()) return;
        }
    };
    uint32_t st = 0, ph = 0;
    auto next = [&]() {
        if (++st == S::kStages) st = 0, ph ^= 1;
    };
    const auto run = [&]() {
        if (!mbar_wait_bounded(&sh.q_full, 0, wait) || !mbar_wait_bounded(&sh.full[0], 0, wait)) return;
        tcgen_fence_after();
        if (leader) {
            issue_s(0, 0);
            issue_s(1, 0);
            mma_commit(&sh.empty[0]);
        }
        __syncwarp();
        next();
        for (uint32_t i = 0; i + 1 < steps; i++) {
            const uint32_t vst = st, vph = ph;
            next();
            if (!mbar_wait_bounded(&sh.full[st], ph, wait)) return;
            if (!mbar_wait_bounded(&sh.ok[i & 7], (i >> 3) & 1, wait) || !mbar_wait_bounded(&sh.full[vst], vph, wait)) return;
#pragma unroll
            for (uint32_t t = 0; t < 2; t++) {
                if constexpr (S::kApart) {
                    if (!mbar_wait_bounded(&sh.s_free[t], i & 1, wait)) return;
                    tcgen_fence_after();
                    if (leader) {
                        issue_s(t, st);
                        if (t) mma_commit(&sh.empty[st]);
                    }
                    __syncwarp();
                }
                if (!mbar_wait_bounded(&sh.p_full[t], i & 1, wait)) return;
                tcgen_fence_after();
                if (leader) {
                    issue_o(t, vst, i > 0);
                    if constexpr (S::kApart) {
                        mma_commit(&sh.o_done[t]);
                        if (t) mma_commit(&sh.empty[vst]);
                    } else {
                        issue_s(t, st);
                        if (t) {
                            mma_commit(&sh.empty[vst]);
                            mma_commit(&sh.empty[st]);
                        }
                    }
                }
                __syncwarp();
            }
            next();
        }
        const uint32_t i = steps - 1;
        if (!mbar_wait_bounded(&sh.ok[i & 7], (i >> 3) & 1, wait) || !mbar_wait_bounded(&sh.full[st], ph, wait)) return;
#pragma unroll
        for (uint32_t t = 0; t < 2; t++) {
            if (!mbar_wait_bounded(&sh.p_full[t], i & 1, wait)) return;
            tcgen_fence_after();
            if (leader) {
                issue_o(t, st, i > 0);
                mma_commit(&sh.o_full[t]);
            }
            __syncwarp();
        }
    };
    if constexpr (kTwin) run_twins();
    else run();
    __syncwarp();
    if (leader) mma_commit(&sh.drained);
    mbar_wait_bounded<true>(&sh.drained, 0, wait);
}

// Values of partly visible tiles: infinities and NaN become 0 here and are added
// to the rows that see them at the end.  E5M2 tiles are widened on the way.
template <int D, int kFmt, class Params>
__device__ __forceinline__ void tend_values(const Params& p, TilesShared& sh, uint8_t* ring, const uint8_t* raw, uint32_t thread) {
    using S = TilesShape<D, kFmt, Params::kPaged>;
    volatile WaitLimit* wait = &sh.wait;
    const uint32_t lane = thread & 31, steps = sh.steps;
    StepSlots slots(sh);
    const WholeTiles whole(sh, sh.p0, sh.p1);
    if constexpr (kWidens<kFmt> && Params::kPaged) {
        // Half of the warps widen the keys, half the values, 16 bytes of the cache a lane:
        // the lanes of a quarter warp take rows of their own, which the swizzles of both
        // tiles spread over the banks, so a lane's places in them stay.
        constexpr uint32_t kWarps = S::kWiden, kCh = kRowBytes<D, kFmt> / 16;
        constexpr uint32_t kRows = kCh == 2 ? 16 : 8, kEach = kCh == 8 ? 2 : 1;  // rows of a warp at once, chunks of a lane
        constexpr uint32_t kOut = 2 * D / kRowBytes<D, kFmt>;                    // 16-byte chunks of FP16 out of one
        const uint32_t mine = thread / (32 * kWarps), warp = (thread >> 5) % kWarps;
        const uint32_t r0 = warp * kRows + (lane & 7) + (kCh == 2 ? lane >> 4 << 3 : 0);  // its first row, the others a multiple of 8 on
        const uint32_t c0 = kCh == 2 ? lane >> 3 & 1 : kEach * (lane >> 3);               // its first chunk, in a row and ..
        const uint32_t shift = kCh == 2 ? lane << 1 & 16 : lane & 24;                     // .. of its block's exponent byte
        const uint8_t* exps = raw + S::kRaws * S::kRaw;
        uint32_t from[kEach], to[kEach * kOut];  // where its chunks lie
#pragma unroll
        for (uint32_t x = 0; x < kEach; x++) from[x] = chunk_at<kRowBytes<D, kFmt>>(r0, c0 + x);
#pragma unroll
        for (uint32_t y = 0; y < kEach * kOut; y++) {
            const uint32_t chunk = kOut * c0 + y;
            to[y] = (chunk >> 3) * (kBN * 128) + r0 * 128 + (((chunk ^ r0) & 7) << 4);
        }
        bool found = false;
        // One part of a tile; kPart: it may hold infinities and NaN that some query does not see.
        const auto widen = [&](auto is_part, const uint8_t* src, const uint8_t* e, uint8_t* dst) {
            constexpr bool kPart = decltype(is_part)::value;
#pragma unroll 2
            for (uint32_t r = 0; r < S::kPartSlots; r += kWarps * kRows) {
                uint4 v[kEach];
#pragma unroll
                for (uint32_t x = 0; x < kEach; x++) v[x] = *reinterpret_cast<const uint4*>(src + r * kRowBytes<D, kFmt> + from[x]);
                uint32_t bytes = 0;
                if constexpr (kQuantised<kFmt>) bytes = *reinterpret_cast<const uint32_t*>(e + 4 * (r + r0));
                const auto put = [&](uint32_t y, uint32_t h0, uint32_t h1, uint32_t h2, uint32_t h3) {
                    if constexpr (kPart) {
                        const uint32_t z0 = finite_or_zero<true>(h0), z1 = finite_or_zero<true>(h1), z2 = finite_or_zero<true>(h2),
                                       z3 = finite_or_zero<true>(h3);
                        found |= z0 != h0 || z1 != h1 || z2 != h2 || z3 != h3;
                        h0 = z0, h1 = z1, h2 = z2, h3 = z3;
                    }
                    *reinterpret_cast<uint4*>(dst + r * 128 + to[y]) = make_uint4(h0, h1, h2, h3);
                };
                // This lane's power, twice.
                const auto power = [&](uint32_t by) {
                    const float f = block_scale(bytes >> by & 255u);
                    return pack2<true>(f, f);
                };
                if constexpr (kFmt == kE5m2) {
#pragma unroll
                    for (uint32_t x = 0; x < kEach; x++) {
                        put(2 * x, e5m2_01(v[x].x), e5m2_23(v[x].x), e5m2_01(v[x].y), e5m2_23(v[x].y));
                        put(2 * x + 1, e5m2_01(v[x].z), e5m2_23(v[x].z), e5m2_01(v[x].w), e5m2_23(v[x].w));
                    }
                } else if constexpr (kFmt == kInt8) {
                    const uint32_t s = power(shift);
                    const auto all = [&](auto one_step) {
#pragma unroll
                        for (uint32_t x = 0; x < 2 * kEach; x++) {
                            const uint32_t lo = int8_bias(x & 1 ? v[x >> 1].z : v[x >> 1].x), hi = int8_bias(x & 1 ? v[x >> 1].w : v[x >> 1].y);
                            if constexpr (decltype(one_step)::value)
                                put(x, int8_scaled<kInt8_01>(lo, s), int8_scaled<kInt8_23>(lo, s), int8_scaled<kInt8_01>(hi, s),
                                    int8_scaled<kInt8_23>(hi, s));
                            else
                                put(x, mul_half2(int8_pair<kInt8_01>(lo), s), mul_half2(int8_pair<kInt8_23>(lo), s),
                                    mul_half2(int8_pair<kInt8_01>(hi), s), mul_half2(int8_pair<kInt8_23>(hi), s));
                        }
                    };
                    if (__any_sync(0xFFFFFFFFu, above_5(bytes))) all(std::false_type());
                    else all(std::true_type());
                } else {
                    const uint32_t s0 = power(shift), s1 = D == 128 ? s0 : power(shift + 8);
                    const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                    for (int y = 0; y < 4; y++) {
                        const uint32_t s = y < 2 ? s0 : s1;
                        uint32_t z[4];
                        e2m1_pairs(z, w[y]);
                        put(y, mul_half2(z[0], s), mul_half2(z[1], s), mul_half2(z[2], s), mul_half2(z[3], s));
                    }
                }
            }
        };
        for (uint32_t n = mine; n < 2 * steps; n += 2, slots.next()) {
            const uint32_t st = n % S::kStages;
            if (n >= S::kStages && !mbar_wait_bounded(&sh.empty[st], (n / S::kStages - 1) & 1, wait)) break;
            const bool part = mine && (sh.p0 < 0 || !whole(slots.s0));
            bool there = true;
#pragma unroll 1
            for (uint32_t u = 0; u < S::kParts; u++) {
                const uint32_t m = n * S::kParts + u, rs = m % S::kRaws;
                there = mbar_wait_bounded(&sh.raw_full[rs], (m / S::kRaws) & 1, wait);
                if (!there) break;
                const uint8_t *src = raw + rs * S::kRaw, *e = exps + rs * S::kExps;
                uint8_t* dst = ring + st * S::kKV + u * (S::kPartSlots * 128);
                if (part) widen(std::true_type(), src, e, dst);
                else widen(std::false_type(), src, e, dst);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.raw_empty[rs]);
            }
            if (!there) break;
            if (found) sh.odd = 1;
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.full[st]);
                if (mine) mbar_arrive(&sh.ok[(n >> 1) & 7]);
            }
        }
    } else if constexpr (kWidens<kFmt>) {
        // Half of the warps widen the keys, half the values.
        const uint32_t mine = thread >= 16 * S::kTend, in_half = thread - mine * 16 * S::kTend;
        for (uint32_t n = mine; n < 2 * steps; n += 2, slots.next()) {
            const uint32_t rs = n % S::kRaws, st = n % S::kStages;
            if (!mbar_wait_bounded(&sh.raw_full[rs], (n / S::kRaws) & 1, wait)) break;
            if (n >= S::kStages && !mbar_wait_bounded(&sh.empty[st], (n / S::kStages - 1) & 1, wait)) break;
            const bool part = mine && (sh.p0 < 0 || !whole(slots.s0));
            bool found = false;
            // 16 bytes of a row become two adjacent 16-byte chunks of the swizzled row.
#pragma unroll 4
            for (uint32_t x = in_half; x < S::kRaw / 16; x += 16 * S::kTend) {
                const uint32_t r = x / (D / 16), c = x % (D / 16);
                const uint4 v = *reinterpret_cast<const uint4*>(raw + rs * S::kRaw + 16 * x);
                uint4 lo = make_uint4(e5m2_01(v.x), e5m2_23(v.x), e5m2_01(v.y), e5m2_23(v.y));
                uint4 hi = make_uint4(e5m2_01(v.z), e5m2_23(v.z), e5m2_01(v.w), e5m2_23(v.w));
                if (part) {
                    const uint4 l = lo, u = hi;
                    lo = make_uint4(finite_or_zero<true>(l.x), finite_or_zero<true>(l.y), finite_or_zero<true>(l.z), finite_or_zero<true>(l.w));
                    hi = make_uint4(finite_or_zero<true>(u.x), finite_or_zero<true>(u.y), finite_or_zero<true>(u.z), finite_or_zero<true>(u.w));
                    found |= l.x != lo.x || l.y != lo.y || l.z != lo.z || l.w != lo.w || u.x != hi.x || u.y != hi.y || u.z != hi.z || u.w != hi.w;
                }
                // Rows of the second block of 64 values store their upper half first, so that
                // the eight lanes of a row hit different banks.
                uint8_t* row = ring + st * S::kKV + (c >> 2) * (kBN * 128) + r * 128;
                const uint32_t c0 = 2 * (c & 3), second = c >> 2;
                *reinterpret_cast<uint4*>(row + (((c0 + second) ^ (r & 7)) << 4)) = second ? hi : lo;
                *reinterpret_cast<uint4*>(row + (((c0 + 1 - second) ^ (r & 7)) << 4)) = second ? lo : hi;
            }
            if (found) sh.odd = 1;
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sh.raw_empty[rs]);
                mbar_arrive(&sh.full[st]);
                if (mine) mbar_arrive(&sh.ok[(n >> 1) & 7]);
            }
        }
    } else {
        for (uint32_t i = 0; i < steps; i++, slots.next()) {
            const uint32_t n = 2 * i + 1, st = n % S::kStages, ph = (n / S::kStages) & 1;
            // Stages that keys and values share (an odd number): every turn is waited for, as a
            // parity says the opposite while a turn before it has not come.
            if (S::kStages % 2 && !mbar_wait_bounded(&sh.full[(n - 1) % S::kStages], ((n - 1) / S::kStages) & 1, wait)) break;
            if (!mbar_wait_bounded(&sh.full[st], ph, wait)) break;
            if (sh.p0 < 0 || !whole(slots.s0)) {
                bool found = false;
                uint4* tile = reinterpret_cast<uint4*>(ring + st * S::kKV);
#pragma unroll 4
                for (uint32_t x = thread; x < S::kKV / 16; x += 32 * S::kTenders) {
                    const uint4 v = tile[x];
                    const uint4 f = make_uint4(finite_or_zero<kWide<kFmt>>(v.x), finite_or_zero<kWide<kFmt>>(v.y), finite_or_zero<kWide<kFmt>>(v.z),
                                               finite_or_zero<kWide<kFmt>>(v.w));
                    if (f.x != v.x || f.y != v.y || f.z != v.z || f.w != v.w) {
                        tile[x] = f;
                        found = true;
                    }
                }
                if (found) {
                    sh.odd = 1;
                    fence_async_proxy();
                }
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&sh.ok[i & 7]);
        }
    }
}

// The rows' softmax, slots 64 half .. 64 half + 63 of each step.  l is this
// half's sum.  Returns false where a wait gave up.
template <int D, int kFmt, bool kTwin, class Params>
__device__ __forceinline__ bool softmax_rows(const Params& p, TilesShared& sh, uint32_t tmem, uint32_t t, uint32_t half,
                                             uint32_t r, uint32_t pair_bar, int32_t pos, float scale, float& m, float& l) {
    volatile WaitLimit* wait = &sh.wait;
    using S = TilesShape<D, kFmt, Params::kPaged>;
    const uint32_t sa = tmem + t * kBN, oa = tmem + S::kColO + t * D + half * (D / 2), pa = tmem + S::kColP + t * S::kStepP + half * S::kHalfP;
    // What a step needs only a moment is read again from shared memory, as volatile.
    const volatile TilesShared& now_sh = sh;
    constexpr uint32_t kStride = kTwin ? 2 : 1;  // from this tile's slot tile to its next
    uint32_t j = 0;
    int32_t s0 = sh.s0;
    const auto advance = [&](int32_t at, int32_t to) { s0 = (int32_t)++j == at ? to : s0 + kBN; };
    if (kTwin && t) advance(sh.jump_at, sh.jump_to);
    m = -INFINITY;
    l = 0.0f;
    bool ready = true, more = j < now_sh.steps;
    for (uint32_t i = 0; more; i++) {
        ready = mbar_wait_bounded(&sh.s_full[t], i & 1, wait) && ready;
        tcgen_fence_after();
        uint32_t s[2][32];
        tmem_ld32(s[0], sa + 64 * half);
        tmem_ld32(s[1], sa + 64 * half + 32);
        const int32_t upto = now_sh.upto[t], after = now_sh.after[t], whole_sinks = now_sh.whole_sinks;
        const int32_t jump_at = now_sh.jump_at, jump_to = now_sh.jump_to;
        const bool part = !((s0 <= upto) & ((s0 > after) | (s0 <= whole_sinks)));
        more = j + kStride < now_sh.steps;
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        tmem_wait_ld();
        tmem_loaded(s[0]);
        tmem_loaded(s[1]);
        if constexpr (S::kApart) {
            tcgen_fence_before();
            __syncwarp();
            if ((r & 31) == 0) mbar_arrive(&sh.s_free[t]);
        }
#pragma unroll
        for (int c = 0; c < 2; c++) {
            if (part) {
                const int64_t back = (int64_t)pos - (int64_t)now_sh.window + 1;
                const uint32_t seen = seen_bits(pos, back < 0 ? 0 : (int32_t)back, now_sh.sinks, s0 + 64 * (int32_t)half + 32 * c);
#pragma unroll
                for (int x = 0; x < 32; x++)
                    if (!(seen >> x & 1u)) s[c][x] = 0xFF800000u;
            }
#pragma unroll
            for (int x = 0; x < 32; x += 2)
                top[(x >> 1) & 3] = max3(top[(x >> 1) & 3], __uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1]));
        }
        advance(jump_at, jump_to);
        if (kTwin) advance(jump_at, jump_to);
        const float own = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
        if constexpr (S::kApart) {  // the last step's product is done with P
            if (i) ready = mbar_wait_bounded(&sh.o_done[t], (i - 1) & 1, wait) && ready;
            tcgen_fence_after();
            __syncwarp();
        }
        // P of this half by the maximum that it would choose; an integer, so that P can
        // be brought to another one without a second rounding.
        const float mine = own > m + (kTilesLift<kWide<kFmt>> + kTilesLazy<kWide<kFmt>>) ? ceilf(own) - kTilesLift<kWide<kFmt>> : m;  // from -inf too
        const float use = mine == -INFINITY ? 0.0f : mine;
        const uint64_t sc = pair(scale, scale), neg = pair(-use, -use);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 64 / kScoresOf; c++) {
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < kScoresOf; x += 2) {
                const int y = kScoresOf * c + x;
                float u, v;
                unpair(fma2(pair(__uint_as_float(s[y >> 5][y & 31]), __uint_as_float(s[y >> 5][(y & 31) + 1])), sc, neg), u, v);
                u = exp2_approx(u);
                v = exp2_approx(v);
                sum[(x >> 1) & 1] = add2(sum[(x >> 1) & 1], pair(u, v));
                // P in 16 bits: an error of up to 2^-8 (BF16) or 2^-11 (FP16, down to 2^-22 of
                // the row's largest) of each term.
                w[x >> 1] = pack2<kWide<kFmt>>(u, v);
            }
            tmem_st8(pa + 8 * c, w);
        }
        float u, v, u2, v2;
        unpair(sum[0], u, v);
        unpair(sum[1], u2, v2);
        float add = (u + v) + (u2 + v2);
        tmem_wait_st();
        // In the first step and rarely after it one of the rows of these two warps has a
        // new maximum, and they settle on one.  Where one's wait gave up, both return.
        if (named_any(pair_bar, 64, mine != m || !ready)) {
            if (!S::kOneRow || !half) sh.row[half][t][r] = mine;
            if (named_any(pair_bar, 64, !ready)) return false;
            const float now = fmaxf(mine, exchange<S::kOneRow>(sh, t, half, r, pair_bar, mine, true));
            const float f = m == now ? 1.0f : exp2_approx(m - now), g = mine == now ? 1.0f : exp2_approx(mine - now);
            m = now;
            l *= f;
            add *= g;
            if (i) {  // this half's columns of O
                const uint64_t ff = pair(f, f);
#pragma unroll
                for (int c = 0; c < D / 16; c++) {
                    uint32_t o[8];
                    tmem_ld8(o, oa + 8 * c);
                    tmem_wait_ld();
                    tmem_loaded(o);
#pragma unroll
                    for (int x = 0; x < 8; x += 2) {
                        float u, v;
                        unpair(mul2(pair(__uint_as_float(o[x]), __uint_as_float(o[x + 1])), ff), u, v);
                        o[x] = __float_as_uint(u);
                        o[x + 1] = __float_as_uint(v);
                    }
                    tmem_st8(oa + 8 * c, o);
                }
            }
            if (__any_sync(0xFFFFFFFFu, mine != now)) {
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    uint32_t w[8];
                    tmem_ld8(w, pa + 8 * c);
                    tmem_wait_ld();
                    tmem_loaded(w);
#pragma unroll
                    for (int x = 0; x < 8; x++) {
                        const float2 y = unpack2<kWide<kFmt>>(w[x]);
                        w[x] = pack2<kWide<kFmt>>(y.x * g, y.y * g);
                    }
                    tmem_st8(pa + 8 * c, w);
                }
            }
            tmem_wait_st();
        }
        l += add;
        tcgen_fence_before();
        __syncwarp();
        if ((r & 31) == 0) mbar_arrive(&sh.p_full[t]);
    }
    // Both tiles' products are done: a CTA's partial results take the tiles' place.
    const bool go = sh.steps == 0 || (ready && mbar_wait_bounded(&sh.o_full[0], 0, wait) && mbar_wait_bounded(&sh.o_full[1], 0, wait));
    tcgen_fence_after();
    return go;
}

// Columns 32 c .. 32 c + 31 of this row of O.
template <int D, int kFmt, bool kTwin, class Params>
__device__ __forceinline__ void read_output(const Params& p, const TilesShared& sh, uint32_t oa, uint32_t t, int32_t pos, int c,
                                            float (&o)[32]) {
    constexpr int kElem = kWidens<kFmt> ? 1 : 2;
    const uint32_t steps = sh.steps;
    const bool any = kTwin ? steps > t : steps != 0;
    uint32_t w[32];
    __syncwarp();
    if (any) {
        tmem_ld32(w, oa + 32 * c);
        tmem_wait_ld();
        tmem_loaded(w);
    }
#pragma unroll
    for (int x = 0; x < 32; x++) o[x] = any ? __uint_as_float(w[x]) : 0.0f;
    if (*reinterpret_cast<const volatile uint32_t*>(&sh.odd)) {
        // The infinite and NaN values of partly visible tiles go to the rows that
        // see them: whatever their (positive) weight, the sum takes their value.
        const WholeTiles whole(sh, sh.p0, sh.p1);
        const int32_t n = sh.n, sinks = sh.sinks;
        const uint32_t window = sh.window;
        const auto values = p.template values<kElem>(sh);
        StepSlots slots(sh);
        for (uint32_t i = 0; i < steps; i++, slots.next()) {
            if ((kTwin && (i & 1) != t) || (sh.p0 >= 0 && whole(slots.s0))) continue;
            for (int32_t s = slots.s0; s < min(slots.s0 + kBN, n); s++) {
                if (!((uint32_t)(pos - s) < window || (s < sinks && s <= pos))) continue;
                const auto row = values(s);
                if (!row.data) continue;
#pragma unroll
                for (int x = 0; x < 32; x++) {
                    const float v = page_value<D, kFmt>(row.data, row.exponents, 32 * c + x);
                    if (!isfinite(v)) o[x] += v;
                }
            }
        }
    }
}

// Rows [columns in fours, then m and l][row] of a piece's partial result.
template <int D>
constexpr uint32_t kPieceFloat4s = (D / 4 + 1) * 2 * kTileM;

// Leaves this piece's rows in memory, and joins all pieces', in their order, in the CTA that
// comes last.  Lanes hold neighbouring rows, so both ways run in whole lines.  All softmax
// threads.
template <int D, int kFmt, class Params>
__device__ __forceinline__ void join_pieces(const Params& p, TilesShared& sh, uint32_t oa, uint32_t t, uint32_t half, uint32_t r, bool valid,
                                            int32_t pos, float m, float l, __nv_bfloat16* out, float* lse) {
    constexpr uint32_t kBar = 9, kStep = 2 * kTileM;  // a barrier that no pair of warps has
    const uint32_t row = t * kTileM + r, pieces = sh.pieces;
    float4* all = p.partials + (uint64_t)sh.first_piece * kPieceFloat4s<D> + row;
    float4* mine = all + sh.piece * kPieceFloat4s<D>;
#pragma unroll 1
    for (int c = half * (D / 64); c < (int)(half + 1) * (D / 64); c++) {  // this half's columns
        float o[32];
        read_output<D, kFmt, false>(p, sh, oa, t, pos, c, o);
#pragma unroll
        for (int x = 0; x < 32; x += 4) __stcg(mine + (8 * c + x / 4) * kStep, make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]));
    }
    if (half == 0) __stcg(mine + D / 4 * kStep, make_float4(m, l, 0.0f, 0.0f));
    __threadfence();
    named_sync(kBar, kSoftmax);
    if (threadIdx.x == 0) {  // a byte counts, and is 0 again for the next call when the last one has counted
        const uint32_t by = 8 * (sh.counter & 3);
        sh.last = (atomicAdd(p.counters + sh.counter / 4, 1u << by) >> by & 255u) == pieces - 1;
        if (sh.last) atomicSub(p.counters + sh.counter / 4, pieces << by);
        __threadfence();
    }
    named_sync(kBar, kSoftmax);
    if (!*reinterpret_cast<const volatile uint32_t*>(&sh.last)) return;
    float top = -INFINITY, sum = 0.0f;
    for (uint32_t i = 0; i < pieces; i++) top = fmaxf(top, __ldcg(all + i * kPieceFloat4s<D> + D / 4 * kStep).x);
    const float base = top == -INFINITY ? 0.0f : top;
    for (uint32_t i = 0; i < pieces; i++) {
        const float4 ml = __ldcg(all + i * kPieceFloat4s<D> + D / 4 * kStep);
        sum = fmaf(ml.y, exp2_approx(ml.x - base), sum);
    }
    const bool none = sum == 0.0f;  // nothing seen, or scores of -infinity alone
    const float inv = 1.0f / sum;
#pragma unroll 1
    for (int c = half * (D / 32); c < (int)(half + 1) * (D / 32); c++) {
        float4 v[4];
#pragma unroll
        for (int x = 0; x < 4; x++) v[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
        for (uint32_t i = 0; i < pieces; i++) {
            const float4* from = all + i * kPieceFloat4s<D>;
            const float f = exp2_approx(__ldcg(from + D / 4 * kStep).x - base);
#pragma unroll
            for (int x = 0; x < 4; x++) {
                const float4 y = __ldcg(from + (4 * c + x) * kStep);
                v[x] = make_float4(fmaf(y.x, f, v[x].x), fmaf(y.y, f, v[x].y), fmaf(y.z, f, v[x].z), fmaf(y.w, f, v[x].w));
            }
        }
        if (valid) {
#pragma unroll
            for (int x = 0; x < 4; x += 2)
                *reinterpret_cast<uint4*>(out + 16 * c + 4 * x) =
                    none ? make_uint4(0, 0, 0, 0)
                         : make_uint4(pack2<false>(v[x].x * inv, v[x].y * inv), pack2<false>(v[x].z * inv, v[x].w * inv),
                                      pack2<false>(v[x + 1].x * inv, v[x + 1].y * inv), pack2<false>(v[x + 1].z * inv, v[x + 1].w * inv));
        }
    }
    if (valid && lse && half == 0) *lse = none ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int D, int kFmt, bool kTwin, class Params>
__global__ void __launch_bounds__(TilesShape<D, kFmt, Params::kPaged>::kThreads, 1) tiles_kernel(const __grid_constant__ Params p) {
    using S = TilesShape<D, kFmt, Params::kPaged>;
    extern __shared__ __align__(1024) uint8_t qs[];
    TilesShared& sh = *reinterpret_cast<TilesShared*>(qs + S::kUsed);
    uint8_t* ring = qs + 2 * S::kQ;             // tiles of D / 64 blocks of 128 rows of 128 bytes, as qs
    uint8_t* raw = ring + S::kStages * S::kKV;  // E5M2 tiles as they are
    const uint32_t warp = threadIdx.x >> 5;

    if constexpr (Params::kPaged) {  // more CTAs than the sequences' row tiles need: the others leave, with their clusters
        if (warp == 0) p.template place<kTwin>(sh, threadIdx.x);
        __syncthreads();
        launch_dependents();  // another launch of the same call, which touches nothing of this one's
        if (!sh.count) {
            if (blockIdx.x == gridDim.x - 1) wait_prerequisite_grid();
            return;
        }
    }
    if (warp == 16) tmem_alloc<512>(&sh.tmem);
    if (threadIdx.x == 0) {
        if constexpr (!Params::kPaged) p.template place<kTwin>(sh);
        for (int i = 0; i < 8; i++) {
            mbar_init(&sh.full[i], kWidens<kFmt> ? S::kWiden : 1);
            mbar_init(&sh.empty[i], 1);
            mbar_init(&sh.ok[i], S::kFit);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&sh.raw_full[i], p.raw_arrivals());
            mbar_init(&sh.raw_empty[i], S::kWiden);
        }
        mbar_init(&sh.q_full, kWide<kFmt> ? kSoftmax : 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 8);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.s_free[i], 8);
            mbar_init(&sh.o_done[i], 1);
        }
        mbar_init(&sh.drained, 1);
        sh.wait.given_up = sh.odd = sh.lost = 0;
        sh.wait.limit = p.wait_limit;
        fence_mbar_init();
    }
    if (!kWide<kFmt> && threadIdx.x < 256) {
        // Rows of a tile that hold no query (128 is not a multiple of every group).
        const uint32_t r = threadIdx.x & 127;
        if (r >= p.tokens * p.group) {
#pragma unroll
            for (int i = 0; i < D / 8; i++)
                *reinterpret_cast<uint4*>(qs + (threadIdx.x >> 7) * S::kQ + (i >> 3) * (kTileM * 128) + r * 128 + 16 * (i & 7)) =
                    make_uint4(0, 0, 0, 0);
            fence_async_proxy();
        }
    }
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp >= 16) {
        regs_dec<S::kOtherRegs>();
        if (sh.steps) {
            if (warp == 16) issue_products<D, kFmt, kTwin, Params>(sh, tmem, qs, ring);
            else if (warp > 17 && warp < 18 + S::kTenders) tend_values<D, kFmt>(p, sh, ring, raw, threadIdx.x - (kSoftmax + 64));
            else if constexpr (Params::kPaged) {
                if (warp == 17 || warp == 18 + S::kTenders) load_page_tiles<D, kFmt, kTwin>(p, sh, qs, ring, raw, warp != 17, threadIdx.x & 31);
            } else if ((threadIdx.x & 31) == 0) load_tiles<D, kFmt, kTwin>(p, sh, qs, ring, raw);
        }
        __syncwarp();
        if (kTwin || p.splits > 1) {  // with the softmax warps below
            cluster_sync();
            cluster_sync();
        }
    } else {
        regs_inc<S::kRegs>();
        const uint32_t t = (warp >> 2) & 1, half = warp >> 3, r = threadIdx.x & 127;
        const uint32_t pair_bar = 1 + (warp & 7);  // of the two warps of the same rows
        float m, l;
        bool go;
        {
            const uint32_t tok = sh.t0 + (kTwin ? 0 : t * p.tokens) + r / p.group, g = r % p.group;
            const bool valid = r < p.tokens * p.group && tok < p.queries(sh);
            const int32_t pos = valid ? max(-1, sh.first + (int32_t)tok) : -1;
            float scale = p.a.scale * kLog2e;
            // Only where there are steps: the products, which wait for all queries, keep this
            // apart from the partial results that take the queries' place.
            if (kWide<kFmt> && sh.steps) {
                // This thread's half of its query row: FP16 of the row scaled by a power of two.
                const uint4* src = reinterpret_cast<const uint4*>(p.query(sh, tok, sh.h * p.group + g)) + half * (D / 16);
                uint4 v[D / 16];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < D / 16; i++) {
                    v[i] = valid ? src[i] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int x = 0; x < 4; x++) top = max(top, max(w[x] & 0x7FFFu, w[x] >> 16 & 0x7FFFu));
                }
                const float power = row_power(max(top, __float_as_uint(exchange<S::kOneRow>(sh, t, half, r, pair_bar, __uint_as_float(top)))));
                scale = fmaxf(scale / power, 0x1p-126f);  // never 0, which -infinity is multiplied by
#pragma unroll
                for (int i = 0; i < D / 16; i++) {
                    uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int x = 0; x < 4; x++)
                        w[x] = pack2<true>(__uint_as_float(w[x] << 16) * power, __uint_as_float(w[x] & 0xFFFF0000u) * power);
                    const uint32_t c = half * (D / 16) + i;  // 16-byte chunk of the row
                    *reinterpret_cast<uint4*>(qs + t * S::kQ + (c >> 3) * (kTileM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_async_proxy();
                mbar_arrive(&sh.q_full);
            }
            go = softmax_rows<D, kFmt, kTwin>(p, sh, tmem + (((warp & 3) * 32) << 16), t, half, r, pair_bar, pos, scale, m, l);
        }
        // The row's sum, of both halves in the same order.
        __syncwarp();
        const float other = exchange<S::kOneRow>(sh, t, half, r, pair_bar, l);
        l = half ? other + l : l + other;
        if ((threadIdx.x & 31) == 0 && !go) atomicOr(p.status, kStatusTimeout);
        if (!go || *reinterpret_cast<const volatile uint32_t*>(&sh.lost)) l = __int_as_float(0x7FC00000);  // a wait that gave up, a lost page: NaN

        // Derived again rather than kept through the loop.
        const uint32_t rr = opaque(threadIdx.x) & 127;
        const uint32_t tok = sh.t0 + (kTwin ? 0 : t * p.tokens) + rr / p.group, g = rr % p.group, hq = sh.h * p.group + g;
        const bool valid = rr < p.tokens * p.group && tok < p.queries(sh);
        const int32_t pos = valid ? max(-1, sh.first + (int32_t)tok) : -1;
        const uint32_t oa = tmem + (((warp & 3) * 32) << 16) + S::kColO + t * D;
        __nv_bfloat16* out = p.out(sh, tok, hq);
        float* lse = p.a.lse ? p.lse(sh, tok, hq) : nullptr;
        bool done = false;
        if constexpr (Params::kPaged && !kTwin) {
            done = p.splits == 1 && sh.pieces > 1;
            if (done) join_pieces<D, kFmt>(p, sh, oa, t, half, rr, valid, pos, m, l, out, lse);
        }
        if (done) {
        } else if (!kTwin && p.splits == 1) {
            const float inv = 1.0f / l;
            const bool none = l == 0.0f;  // nothing seen, or scores of -infinity alone
#pragma unroll 1
            for (int c = half * (D / 64); c < (int)(half + 1) * (D / 64); c++) {  // this half's columns
                float o[32];
                read_output<D, kFmt, kTwin>(p, sh, oa, t, pos, c, o);
                if (valid) {
#pragma unroll
                    for (int x = 0; x < 32; x += 8)
                        *reinterpret_cast<uint4*>(out + 32 * c + x) =
                            none ? make_uint4(0, 0, 0, 0)
                                 : make_uint4(pack2<false>(o[x] * inv, o[x + 1] * inv), pack2<false>(o[x + 2] * inv, o[x + 3] * inv),
                                              pack2<false>(o[x + 4] * inv, o[x + 5] * inv), pack2<false>(o[x + 6] * inv, o[x + 7] * inv));
                }
            }
            if (valid && lse && half == 0) *lse = none ? -INFINITY : (m + log2f(l)) * kLn2;
        } else {
            // Join the cluster's splits: every CTA leaves its rows in shared memory and
            // joins a share of them, in the order of the splits.
            float* rows = reinterpret_cast<float*>(qs);
#pragma unroll 1
            for (int c = half * (D / 64); c < (int)(half + 1) * (D / 64); c++) {  // this half's columns
                float o[32];
                read_output<D, kFmt, kTwin>(p, sh, oa, t, pos, c, o);
                float4* to = reinterpret_cast<float4*>(rows + (t * kTileM + rr) * S::kRowFloats + 32 * c);
#pragma unroll
                for (int x = 0; x < 32; x += 4) to[x >> 2] = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
            }
            if (half == 0) {
                rows[(t * kTileM + rr) * S::kRowFloats + D] = m;
                rows[(t * kTileM + rr) * S::kRowFloats + D + 1] = l;
            }
            __syncwarp();
            cluster_sync();
            constexpr uint32_t kLanes = D / 4;  // threads to a row
            const uint32_t rank = blockIdx.x % p.splits, c = 4 * (threadIdx.x % kLanes);
            for (uint32_t x = threadIdx.x / kLanes * p.splits + rank; x < (kTwin ? 1 : 2) * kTileM; x += kSoftmax / kLanes * p.splits) {
                const uint32_t xr = x & 127, xt = sh.t0 + (x >> 7) * p.tokens + xr / p.group, xh = sh.h * p.group + xr % p.group;
                if (xr >= p.tokens * p.group || xt >= p.queries(sh)) continue;
                const uint32_t at = smem_addr(rows + x * S::kRowFloats);
                float mm = -INFINITY, ll = 0.0f;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                for (uint32_t i = 0; i < p.splits * (kTwin ? 2 : 1); i++) {
                    const uint32_t from = kTwin ? i >> 1 : i, row = kTwin ? at + (i & 1) * (kTileM * S::kRowFloats * 4) : at;
                    const float mi = cluster_ld(row + 4 * D, from), li = cluster_ld(row + 4 * D + 4, from);
                    const float4 y = cluster_ld4(row + 4 * c, from);
                    const float top = fmaxf(mm, mi), base = top == -INFINITY ? 0.0f : top;
                    const float f = exp2_approx(mm - base), gi = exp2_approx(mi - base);
                    ll = fmaf(ll, f, li * gi);
                    v = make_float4(fmaf(v.x, f, y.x * gi), fmaf(v.y, f, y.y * gi), fmaf(v.z, f, y.z * gi), fmaf(v.w, f, y.w * gi));
                    mm = top;
                }
                const bool none = ll == 0.0f;
                const float inv = 1.0f / ll;
                __nv_bfloat16* to = p.out(sh, xt, xh);
                *reinterpret_cast<uint2*>(to + c) =
                    none ? make_uint2(0, 0) : make_uint2(pack2<false>(v.x * inv, v.y * inv), pack2<false>(v.z * inv, v.w * inv));
                if (c == 0 && p.a.lse) *p.lse(sh, xt, xh) = none ? -INFINITY : (mm + log2f(ll)) * kLn2;
            }
            __syncwarp();
            cluster_sync();  // this CTA's rows have been read
        }
        tcgen_fence_before();
    }
    __syncthreads();
    tcgen_fence_after();
    if (warp == 16) tmem_free<512>(tmem);
    // As such another launch, this one ends after the one ahead of it.
    if (Params::kPaged && blockIdx.x == gridDim.x - 1) wait_prerequisite_grid();
}

template <int D, int kFmt, bool kTwin, class Params>
cudaError_t launch_tiles(const Params& p, uint32_t ctas, cudaStream_t s, bool beside = false) {
    using S = TilesShape<D, kFmt, Params::kPaged>;
    constexpr int kSmem = S::kUsed + (int)sizeof(TilesShared) - (S::kOneRow ? (int)sizeof(TilesShared::row) / 2 : 0);
    static_assert(kSmem <= 232448, "shared memory of a CTA");
    Wave w;
    const cudaError_t e = launch_wave<tiles_kernel<D, kFmt, kTwin, Params>>(TilesShape<D, kFmt, Params::kPaged>::kThreads, kSmem, w);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.splits;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(TilesShape<D, kFmt, Params::kPaged>::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, tiles_kernel<D, kFmt, kTwin, Params>, p);
}

}  // namespace splitzip
