// attention_weights.cu -- the attention weight that cached slots get (sm_103a).
//
// w[t] = sum over query rows r that see slot t of exp(scale q_r.k_t - lse_r).
// The scores are computed transposed on the tensor cores, S = K Q^T with slots
// as the 128 rows of the accumulator: a thread holds one slot's row, so its sum
// needs no atomics, and its order is fixed.
//
// One CTA per SM walks over items: 128 slots of one key/value head, whose keys
// stay in shared memory while the tiles of 128 query rows (128 / group tokens,
// the group's heads side by side) that can see any of them pass by.  The items
// that most queries see come first and each CTA takes them in turn, every
// second round from the other end, which evens out the causal triangle.  The
// next item's keys and queries are on their way while one is worked on.
//
// Four accumulators of 128 columns fill tensor memory: the products run ahead of
// the exponentials, of which 128 x 128 scores take 512 cycles of the units, as
// the products of head_dim 128 do of the tensor cores.  The columns that a slot
// takes part in are one range: tokens from the slot's own to the last that has
// it in its window.
//
// What bounds it is the latency of its roles: a group of warps takes about 1900
// cycles for a query tile, which with two groups is 950 each, and the warp that
// issues the products not much less to issue and commit them in turn, where the
// products and the exponentials take 512 each.  Two prompts of 3000 tokens, 32
// heads of 128 over 8: 72.5 us (0.78 PFLOP/s over the visible pairs); the last 64
// tokens over 16384: 14.6-15.3 us (keys at 2.3 TB/s).  Keys in tensor memory
// as the first operand gave 71 and 16 us, with a third fewer accumulators.
//
// Roles: warps 0-15 sum (0-7 the even, 8-15 the odd query tiles, four warps to
// 64 columns), 16 issues the products, 17 the TMA loads, 18 brings each query
// tile's lse, 19 works out the items for all (done by every warp for itself it
// cost half of an item of two query tiles); for an E5M2 cache 20-23 widen the
// keys to BF16 (exact).
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "attention.cuh"
#include "tcgen.cuh"
#include "tensor_map.h"

namespace splitzip {
namespace {

constexpr int kSum = 512;  // threads
constexpr int kSlotTile = 128, kRowTile = 128;
constexpr int kKStages = 2, kQStages = 3, kRaws = 2, kMetas = 8, kItems = 4;

struct WeightsParams {
    splitzip_attention_args a;
    CUtensorMap qmap, kmap;
    const float* in;
    float* out;
    uint32_t group, tokens;  // tokens of a query tile: 128 / group
    uint32_t items;          // (slot tile, sequence and head), slot tiles outermost
    ChunkDiv by_heads, by_kv_heads, by_tokens;  // divisions by batch * kv_heads, kv_heads, tokens
    uint32_t window;         // at most 2^31: unlimited
    uint32_t one_q, one_k;   // the batch is one sequence: coordinate 0
    uint32_t wait_limit;
    uint32_t test_cta, test_tile;  // a copy that a test has left out
};

template <int D, bool kF8>
struct WeightsShape {
    static constexpr int kTile = 128 * D * 2, kRaw = 128 * D;
    static constexpr int kThreads = kSum + 32 * (kF8 ? 8 : 4);
    static constexpr int kRegs = kF8 ? 96 : 104, kOtherRegs = kF8 ? 48 : 64;
    static_assert(kSum * kRegs + (kThreads - kSum) * kOtherRegs <= kThreads * (65536 / kThreads / 8 * 8),
                  "register shares add up to what the CTA is launched with");
    static constexpr int kUsed = (kKStages + kQStages) * kTile + (kF8 ? kRaws * kRaw : 0);
};

// One item: its slots s_lo .. s_hi of key/value head h of sequence b (bh counts
// both), the query tiles i0 .. i0 + steps - 1 that can see them; from the first of
// these tiles on, how many query tokens there are (last) and which of them is at
// the position of s_lo (behind, may be negative); the tiles all of whose tokens
// see all of the slots, whole_lo .. whole_hi - 1.
constexpr uint32_t kNoItem = 0xFFFFFFFFu;  // bh of the end of the list
struct Item {
    uint32_t b, h, bh, i0, steps;
    int32_t s_lo, s_hi, last, behind, sinks;
    uint32_t whole_lo, whole_hi;
    // The query tokens that see slot s_lo + r, from the first tile on: [see_from, see_end).
    __device__ __forceinline__ int32_t see_from(uint32_t r) const { return min(max(behind + (int32_t)r, 0), last); }
    __device__ __forceinline__ int32_t see_end(const WeightsParams& p, uint32_t r) const {
        const int64_t end = (int64_t)behind + (int32_t)r + p.window;
        return s_lo + (int32_t)r < sinks || end >= last ? last : max((int32_t)end, 0);
    }
};

struct WeightsShared {
    uint64_t item_full[kItems], item_free[kItems];
    Item item[kItems];
    uint64_t k_full[kKStages], k_empty[kKStages], q_full[kQStages], q_empty[kQStages];
    uint64_t raw_full[kRaws], raw_empty[kRaws];
    uint64_t s_full[4], s_free[4];
    uint64_t meta_full[kMetas], meta_free[kMetas];
    uint64_t drained;
    WaitLimit wait;
    uint32_t tmem;
    alignas(16) float lse[kMetas][kRowTile];  // times -log2(e)
    float part[2][4][kSlotTile];              // sums of the four groups of warps, by item
};

// The items in turn, as warp 19 left them.  Whole warps call this.
struct Items {
    WeightsShared& sh;
    uint32_t at;
    Item w;
    __device__ __forceinline__ explicit Items(WeightsShared& s) : sh(s), at(0) {}
    __device__ __forceinline__ bool ready() { return mbar_try_wait(&sh.item_full[at % kItems], (at / kItems) & 1); }
    // The next item with steps, or any with kAll; false at the end, or where the wait gave up.
    template <bool kAll = false>
    __device__ __forceinline__ bool next() {
        while (true) {
            const uint32_t x = at % kItems;
            if (!mbar_wait_bounded(&sh.item_full[x], (at / kItems) & 1, &sh.wait)) return false;
            w = sh.item[x];
            __syncwarp();
            if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.item_free[x]);
            at++;
            if (w.bh == kNoItem) return false;
            if (kAll || w.steps) return true;
        }
    }
};
__device__ __forceinline__ uint32_t tile_rows(const WeightsParams& p, const Item& w, uint32_t i) {
    return min(p.tokens, (uint32_t)w.last - i * p.tokens) * p.group;
}

// x / d, where d may be 1 too.
__device__ __forceinline__ uint32_t quotient(const ChunkDiv& c, uint32_t x) { return c.d == 1 ? x : chunk_quot32(c, x); }

// Items are taken in rounds over the CTAs, every second one from the other end.
__device__ __forceinline__ void plan_items(const WeightsParams& p, WeightsShared& sh) {
    const splitzip_attention_args& a = p.a;
    const uint32_t heads = a.batch * a.kv_heads;
    for (uint32_t round = 0;; round++) {
        const uint32_t x = round % kItems, use = round / kItems;
        const uint64_t first_of = (uint64_t)round * gridDim.x;
        const uint64_t at = first_of + (round & 1u ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        Item w;
        w.bh = kNoItem;
        if (first_of < p.items) {
            w.steps = 0;
            w.bh = 0;
            w.s_lo = 0;
            w.s_hi = -1;  // no slots, where a last round does not reach this CTA
            if (at < p.items) {
                const uint32_t sc = quotient(p.by_heads, (uint32_t)at);
                w.bh = (uint32_t)at - sc * heads;
                w.b = quotient(p.by_kv_heads, w.bh);
                w.h = w.bh - w.b * a.kv_heads;
                const Mask mask(a, w.b);
                w.s_lo = (int32_t)(sc * kSlotTile);
                w.s_hi = (int32_t)min((int64_t)w.s_lo + kSlotTile, (int64_t)a.kv_tokens) - 1;
                w.sinks = mask.sinks;
                // Positions from s_lo on, and up to the window's end behind s_hi unless s_lo is a sink.
                const int64_t t_lo = max((int64_t)0, (int64_t)w.s_lo - mask.first);
                int64_t t_hi = w.s_lo < mask.n ? (int64_t)a.q_tokens : 0;
                if (w.s_lo >= w.sinks) t_hi = min(t_hi, (int64_t)w.s_hi + mask.window - mask.first);
                if (t_hi > t_lo) {
                    w.i0 = quotient(p.by_tokens, (uint32_t)t_lo);
                    w.steps = quotient(p.by_tokens, (uint32_t)t_hi + p.tokens - 1) - w.i0;
                    w.last = (int32_t)(a.q_tokens - w.i0 * p.tokens);
                    w.behind = (int32_t)((int64_t)w.s_lo - mask.first - (int64_t)w.i0 * p.tokens);
                    w.whole_lo = quotient(p.by_tokens, (uint32_t)max(w.behind + kSlotTile - 1, 0) + p.tokens - 1);
                    // The first slot that is no sink is the first to leave the window.
                    const uint32_t r = (uint32_t)min(max(w.sinks - w.s_lo, 0), kSlotTile - 1);
                    w.whole_hi = quotient(p.by_tokens, (uint32_t)w.see_end(p, r));
                }
            }
        }
        if (use && !mbar_wait_bounded(&sh.item_free[x], (use - 1) & 1, &sh.wait)) return;
        sh.item[x] = w;
        mbar_arrive(&sh.item_full[x]);
        if (w.bh == kNoItem) return;
    }
}

// Two E5M2 values (selected bytes of r, as the upper bytes of FP16) as BF16.
__device__ __forceinline__ uint32_t e5m2_to_bf16(uint32_t r, uint32_t select) {
    const uint32_t h = prmt(r, 0u, select);  // FP16, exact
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack2<false>(f.x, f.y);
}

template <int D, bool kF8>
__device__ __forceinline__ void load_items(const WeightsParams& p, WeightsShared& sh, uint8_t* ks, uint8_t* ring, uint8_t* raw) {
    using S = WeightsShape<D, kF8>;
    constexpr uint32_t kN = kF8 ? kRaws : kKStages;
    volatile WaitLimit* wait = &sh.wait;
    uint64_t* k_full = kF8 ? sh.raw_full : sh.k_full;
    uint64_t* k_empty = kF8 ? sh.raw_empty : sh.k_empty;
    uint32_t it = 0, n = 0;
    bool go = true;
    const bool leader = elect_one();
    const uint32_t left_out = blockIdx.x == p.test_cta ? p.test_tile : 0xFFFFFFFFu;
    Items list(sh);
    while (go && list.next()) {
        const Item& w = list.w;
        const uint32_t ks_at = it % kN, use = it / kN;
        if (use && !mbar_wait_bounded(&k_empty[ks_at], (use - 1) & 1, wait)) break;
        if (leader) mbar_arrive_expect_tx(&k_full[ks_at], kF8 ? S::kRaw : S::kTile);
        if (it + n == left_out) {
        } else if (kF8) {
            if (leader) tma_load4(raw + ks_at * S::kRaw, &p.kmap, 0, w.s_lo, (int32_t)w.h, p.one_k ? 0 : (int32_t)w.b, &k_full[ks_at]);
        } else if (leader) {
#pragma unroll
            for (int x = 0; x < D / 64; x++)
                tma_load4(ks + ks_at * S::kTile + x * (kSlotTile * 128), &p.kmap, 64 * x, w.s_lo, (int32_t)w.h,
                          p.one_k ? 0 : (int32_t)w.b, &k_full[ks_at]);
        }
        it++;
        for (uint32_t i = 0; i < w.steps; i++, n++) {
            const uint32_t st = n % kQStages, quse = n / kQStages;
            if (quse && !(go = mbar_wait_bounded(&sh.q_empty[st], (quse - 1) & 1, wait))) break;
            if (leader) {
                mbar_arrive_expect_tx(&sh.q_full[st], p.tokens * p.group * D * 2);
#pragma unroll
                for (int x = 0; x < D / 64 && it + n != left_out; x++)
                    tma_load4(ring + st * S::kTile + x * (kRowTile * 128), &p.qmap, 64 * x, (int32_t)(w.h * p.group),
                              (int32_t)((w.i0 + i) * p.tokens), p.one_q ? 0 : (int32_t)w.b, &sh.q_full[st]);
            }
            __syncwarp();  // no lane falls a phase behind
        }
    }
    // Every load has landed before this CTA may end, also where a wait gave up.
    for (uint32_t x = it > kN ? it - kN : 0; x < it; x++) mbar_wait_bounded<true>(&k_full[x % kN], (x / kN) & 1, wait);
    for (uint32_t x = n > kQStages ? n - kQStages : 0; x < n; x++)
        mbar_wait_bounded<true>(&sh.q_full[x % kQStages], (x / kQStages) & 1, wait);
}

// The whole warp takes the items, one lane issues.
template <int D, bool kF8>
__device__ __forceinline__ void issue_items(const WeightsParams& p, WeightsShared& sh, uint32_t tmem, const uint8_t* ks, const uint8_t* ring) {
    using S = WeightsShape<D, kF8>;
    volatile WaitLimit* wait = &sh.wait;
    const bool leader = elect_one();
    const uint32_t kd = desc_rows(smem_addr(ks)), qd = desc_rows(smem_addr(ring));
    const uint32_t leader_lane = __ffs(__ballot_sync(0xFFFFFFFFu, leader)) - 1;
    // As many columns as a tile has rows, in steps of 16; here, of all but an item's last.
    const uint32_t most = mma_shape(false, (p.tokens * p.group + 15) & ~15u, false);
    uint32_t it = 0, n = 0, st = 0, turn = 0;  // item, tile, query stage and its phase
    bool go = true, ready = false;             // ready: the next tile's queries and accumulator are
    Items list(sh);
    while (go && list.next()) {
        const Item& w = list.w;
        const uint32_t kst = it % kKStages;
        go = mbar_wait_bounded(&sh.k_full[kst], (it / kKStages) & 1, wait);
        tcgen_fence_after();
        if (leader) {
            const uint32_t ka = kd + kst * (S::kTile >> 4);
            for (uint32_t i = 0; go && i < w.steps; i++, n++) {
                const uint32_t x = n & 3;
                go = ready || (mbar_wait_bounded(&sh.q_full[st], turn, wait) &&
                               (n < 4 || mbar_wait_bounded(&sh.s_free[x], ((n >> 2) - 1) & 1, wait)));
                if (!go) break;
                const uint32_t shape = i + 1 < w.steps ? most : mma_shape(false, (tile_rows(p, w, i) + 15) & ~15u, false);
                const uint32_t qa = qd + st * (S::kTile >> 4);
                tcgen_fence_after();
#pragma unroll
                for (int k = 0; k < D / 16; k++) {
                    const uint32_t off = (k >> 2) * (kSlotTile * 128) + (k & 3) * 32;
                    mma_ss(tmem + x * kRowTile, desc(ka, off), desc(qa, off), shape, k > 0);
                    if (k == D / 32 - 1) {  // a look ahead while these run: 72.5 us at 2 x 3000, 74.2 without
                        const uint32_t m = n + 1;
                        const bool wraps = st + 1 == kQStages;
                        const bool q = mbar_test(&sh.q_full[wraps ? 0 : st + 1], wraps ? turn ^ 1 : turn);
                        const bool f = m < 4 || mbar_test(&sh.s_free[m & 3], ((m >> 2) - 1) & 1);
                        ready = q & f;
                    }
                }
                mma_commit(&sh.s_full[x]);
                mma_commit(&sh.q_empty[st]);
                if (i + 1 == w.steps) mma_commit(&sh.k_empty[kst]);
                if (++st == kQStages) st = 0, turn ^= 1;
            }
        }
        go = __shfl_sync(0xFFFFFFFFu, (int)go, leader_lane) != 0;
        it++;
    }
    __syncwarp();
    if (leader) mma_commit(&sh.drained);
    mbar_wait_bounded<true>(&sh.drained, 0, wait);
}

// One warp; two tiles' values are on their way while an earlier one's are handed over.
__device__ __forceinline__ void bring_lse(const WeightsParams& p, WeightsShared& sh) {
    volatile WaitLimit* wait = &sh.wait;
    const uint32_t lane = threadIdx.x & 31;
    uint32_t place[4];  // of this lane's four rows: token in the tile
    uint64_t head[4];   // and the start of the query head's values
#pragma unroll
    for (int y = 0; y < 4; y++) {
        const uint32_t r = 32 * y + lane;
        place[y] = r / p.group;
        head[y] = (uint64_t)(r - place[y] * p.group) * p.a.q_tokens;
    }
    float value[2][4] = {};
    uint32_t n = 0, held = 0;  // value[2 - held ..] are the tiles n - held ..
    auto hand_over = [&]() {   // the oldest tile held
        const uint32_t of = n - held, x = of % kMetas, use = of / kMetas;
        if (use && !mbar_wait_bounded(&sh.meta_free[x], (use - 1) & 1, wait)) return false;
#pragma unroll
        for (int y = 0; y < 4; y++) {
            // -infinity: the query has no score above it, and gives no weight.
            const float v = held == 2 ? value[0][y] : value[1][y];
            sh.lse[x][32 * y + lane] = v == -INFINITY ? 0.0f : v * -kLog2e;
        }
        held--;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.meta_full[x]);
        return true;
    };
    Items list(sh);
    while (true) {
        // Nothing is held while waiting for an item: the others may need it to go on.
        if (!__all_sync(0xFFFFFFFFu, list.ready()))
            while (held)
                if (!hand_over()) return;
        if (!list.next<true>()) break;
        const Item& w = list.w;
        const float* lse = p.a.lse + ((uint64_t)w.b * p.a.q_heads + w.h * p.group) * p.a.q_tokens + w.i0 * p.tokens;
        for (uint32_t i = 0; i < w.steps; i++) {
            const uint32_t rows = tile_rows(p, w, i);
            float next[4];
#pragma unroll
            for (int y = 0; y < 4; y++) next[y] = 32 * y + lane < rows ? __ldg(lse + head[y] + i * p.tokens + place[y]) : 0.0f;
            if (held == 2 && !hand_over()) return;
#pragma unroll
            for (int y = 0; y < 4; y++) value[0][y] = value[1][y], value[1][y] = next[y];
            n++;
            held++;
        }
    }
    while (held)
        if (!hand_over()) return;
}

template <int D>
__device__ __forceinline__ void widen_keys(const WeightsParams& p, WeightsShared& sh, uint8_t* ks, const uint8_t* raw, uint32_t thread) {
    using S = WeightsShape<D, true>;
    volatile WaitLimit* wait = &sh.wait;
    uint32_t it = 0;
    Items list(sh);
    while (list.next()) {
        const uint32_t rs = it % kRaws, st = it % kKStages;
        if (!mbar_wait_bounded(&sh.raw_full[rs], (it / kRaws) & 1, wait)) return;
        if (it >= kKStages && !mbar_wait_bounded(&sh.k_empty[st], (it / kKStages - 1) & 1, wait)) return;
        // 16 bytes of a row become two adjacent 16-byte chunks of the swizzled row.
#pragma unroll 2
        for (uint32_t x = thread; x < kSlotTile * (D / 16); x += 128) {
            const uint32_t r = x / (D / 16), c = x % (D / 16), c0 = 2 * (c & 3);
            const uint4 v = *reinterpret_cast<const uint4*>(raw + rs * S::kRaw + 16 * x);
            uint8_t* row = ks + st * S::kTile + (c >> 2) * (kSlotTile * 128) + r * 128;
            *reinterpret_cast<uint4*>(row + ((c0 ^ (r & 7)) << 4)) = make_uint4(
                e5m2_to_bf16(v.x, 0x1404), e5m2_to_bf16(v.x, 0x3424), e5m2_to_bf16(v.y, 0x1404), e5m2_to_bf16(v.y, 0x3424));
            *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (r & 7)) << 4)) = make_uint4(
                e5m2_to_bf16(v.z, 0x1404), e5m2_to_bf16(v.z, 0x3424), e5m2_to_bf16(v.w, 0x1404), e5m2_to_bf16(v.w, 0x3424));
        }
        fence_async_proxy();
        __syncwarp();
        if ((thread & 31) == 0) {
            mbar_arrive(&sh.raw_empty[rs]);
            mbar_arrive(&sh.k_full[st]);
        }
        it++;
    }
}

// NaN for the items from this CTA's round on.
__device__ __forceinline__ void give_up(const WeightsParams& p, uint32_t round, uint32_t g, uint32_t r) {
    const uint32_t heads = p.a.batch * p.a.kv_heads;
    for (; g == 0 && (uint64_t)round * gridDim.x < p.items; round++) {
        const uint64_t at = (uint64_t)round * gridDim.x + (round & 1u ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        const uint64_t sc = at / heads, slot = sc * kSlotTile + r;
        if (at < p.items && slot < p.a.kv_tokens) p.out[(at - sc * heads) * p.a.kv_tokens + slot] = __int_as_float(0x7FC00000);
    }
}

// Group of warps g: columns 64 (g & 1) .. of the query tiles n with (n & 1) = g >> 1.
__device__ __forceinline__ void sum_items(const WeightsParams& p, WeightsShared& sh, uint32_t tmem, uint32_t g, uint32_t r) {
    volatile WaitLimit* wait = &sh.wait;
    const uint32_t c0 = (g & 1) * 64;
    const float scale = p.a.scale * kLog2e;
    const uint64_t scale2 = pair(scale, scale);
    const int32_t group = (int32_t)p.group, tokens = (int32_t)p.tokens;
    const bool full = p.tokens * p.group >= c0 + 64;  // all of these columns are in use
    uint32_t n = 0, at = 0;
    for (;; at++) {
        // The item's record is read where it lies, and given back at the item's end.
        // Where a wait for one gave up, all return at the barrier below.
        const uint32_t rec = at % kItems;
        const bool ok = mbar_wait_bounded(&sh.item_full[rec], (at / kItems) & 1, wait);
        const Item& w = sh.item[rec];
        if (!ok || w.bh == kNoItem) {
            if (named_any(1, kSum, !ok)) give_up(p, at, g, r);
            return;
        }
        const uint32_t steps = w.steps, whole_lo = w.whole_lo, whole_hi = w.whole_hi, parity = at & 1;
        const bool mine = g == 0 && w.s_lo + (int32_t)r <= w.s_hi;
        const uint64_t to = (uint64_t)w.bh * p.a.kv_tokens + (uint32_t)w.s_lo + r;
        const float before = mine && p.in ? p.in[to] : 0.0f;
        float sum = 0.0f;
        bool gave_up = false;
        uint32_t i = (n ^ (g >> 1)) & 1;  // the first of this group's tiles
        n += i;
        for (; i < steps; i += 2, n += 2) {
            const uint32_t x = n & 3, mx = n % kMetas;
            const uint32_t m_at = (n / kMetas) & 1, s_at = (n >> 2) & 1;
            const bool m_there = mbar_try_wait(&sh.meta_full[mx], m_at), s_there = mbar_try_wait(&sh.s_full[x], s_at);  // mostly both
            const bool there = (m_there & s_there) || (mbar_wait_bounded(&sh.meta_full[mx], m_at, wait) && mbar_wait_bounded(&sh.s_full[x], s_at, wait));
            if (!__all_sync(0xFFFFFFFFu, there)) {
                gave_up = true;
                break;
            }
            tcgen_fence_after();
            const uint32_t sa = tmem + x * kRowTile + c0;
            uint32_t s[2][32];
            tmem_ld32(s[0], sa);
            tmem_ld32(s[1], sa + 32);
            const bool whole = i >= whole_lo && i < whole_hi;
            uint64_t part[2] = {0, 0};
            tmem_wait_ld();
            tmem_loaded(s[0]);
            tmem_loaded(s[1]);
            tcgen_fence_before();
            __syncwarp();
            if ((r & 31) == 0) mbar_arrive(&sh.s_free[x]);
#pragma unroll
            for (int c = 0; c < 2; c++) {
                uint32_t(&v)[32] = s[c];
                const auto add = [&](auto masked, uint32_t in) {
#pragma unroll
                    for (int y = 0; y < 32; y += 4) {
                        const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(&sh.lse[mx][c0 + 32 * c + y]);
#pragma unroll
                        for (int z = 0; z < 4; z += 2) {
                            float e, f;
                            unpair(fma2(pair(__uint_as_float(v[y + z]), __uint_as_float(v[y + z + 1])), scale2, z ? l.y : l.x), e, f);
                            e = exp2_approx(e);
                            f = exp2_approx(f);
                            if (masked) {
                                e = in >> (y + z) & 1u ? e : 0.0f;
                                f = in >> (y + z + 1) & 1u ? f : 0.0f;
                            }
                            part[z >> 1] = add2(part[z >> 1], pair(e, f));
                        }
                    }
                };
                if (whole && (full || p.tokens * p.group >= c0 + 32 * c + 32)) {
                    add(std::false_type(), 0u);
                } else {
                    // This tile's columns that the slot takes part in.
                    const int32_t t0 = (int32_t)i * tokens, col = (int32_t)c0 + 32 * c;
                    const int32_t l = max(0, min(tokens, w.see_from(r) - t0)) * group - col;
                    const int32_t u = max(0, min(tokens, w.see_end(p, r) - t0)) * group - col;
                    const uint32_t from = l <= 0 ? 0xFFFFFFFFu : l > 31 ? 0u : 0xFFFFFFFFu << l;
                    const uint32_t below = u <= 0 ? 0u : u > 31 ? 0xFFFFFFFFu : ~(0xFFFFFFFFu << u);
                    if (__any_sync(0xFFFFFFFFu, from & below)) add(std::true_type(), from & below);
                }
            }
            float u, v, u2, v2;
            unpair(part[0], u, v);
            unpair(part[1], u2, v2);
            sum += (u + v) + (u2 + v2);
            __syncwarp();
            if ((r & 31) == 0) mbar_arrive(&sh.meta_free[mx]);
        }
        n += steps - i;  // to the next item's first tile
        sh.part[parity][g][r] = sum;
        __syncwarp();
        if ((r & 31) == 0) mbar_arrive(&sh.item_free[rec]);
        // After a wait that gave up the barriers' phases say nothing any more: this item and
        // those after it are NaN.
        if (named_any(1, kSum, gave_up)) {
            give_up(p, at, g, r);
            return;
        }
        if (mine) p.out[to] = before + ((sum + sh.part[parity][1][r]) + (sh.part[parity][2][r] + sh.part[parity][3][r]));
    }
}

template <int D, bool kF8>
__global__ void __launch_bounds__(WeightsShape<D, kF8>::kThreads, 1) weights_kernel(const __grid_constant__ WeightsParams p) {
    using S = WeightsShape<D, kF8>;
    extern __shared__ __align__(1024) uint8_t ks[];
    uint8_t* ring = ks + kKStages * S::kTile;   // query tiles
    uint8_t* raw = ring + kQStages * S::kTile;  // E5M2 keys as they are
    WeightsShared& sh = *reinterpret_cast<WeightsShared*>(ks + S::kUsed);
    const uint32_t tid = threadIdx.x, warp = tid >> 5;

    if (warp == 16) tmem_alloc<512>(&sh.tmem);
    if (tid == 0) {
        for (int i = 0; i < kKStages; i++) {
            mbar_init(&sh.k_full[i], kF8 ? 4 : 1);
            mbar_init(&sh.k_empty[i], 1);
        }
        for (int i = 0; i < kQStages; i++) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
        }
        for (int i = 0; i < kRaws; i++) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], 4);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.s_free[i], 8);
        }
        for (int i = 0; i < kMetas; i++) {
            mbar_init(&sh.meta_full[i], 1);
            mbar_init(&sh.meta_free[i], 8);
        }
        for (int i = 0; i < kItems; i++) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_free[i], S::kThreads / 32 - 1);  // every warp but the one that plans
        }
        mbar_init(&sh.drained, 1);
        sh.wait.given_up = 0;
        sh.wait.limit = p.wait_limit;
        fence_mbar_init();
    }
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    const uint32_t tmem = sh.tmem;

    if (warp < 16) {
        regs_inc<S::kRegs>();
        sum_items(p, sh, tmem + (((warp & 3) * 32) << 16), warp >> 2, tid & 127);
        tcgen_fence_before();
    } else {
        regs_dec<S::kOtherRegs>();
        if (warp == 16) issue_items<D, kF8>(p, sh, tmem, ks, ring);
        else if (warp == 17) load_items<D, kF8>(p, sh, ks, ring, raw);
        else if (warp == 18) bring_lse(p, sh);
        else if (warp == 19 && (tid & 31) == 0) plan_items(p, sh);
        else if (warp > 19) widen_keys<D>(p, sh, ks, raw, tid - (kSum + 128));
    }
    __syncthreads();
    tcgen_fence_after();
    if (warp == 16) tmem_free<512>(tmem);
}

template <int D, bool kF8>
cudaError_t launch(const WeightsParams& p, cudaStream_t s) {
    using S = WeightsShape<D, kF8>;
    constexpr int kSmem = S::kUsed + (int)sizeof(WeightsShared);
    static_assert(kSmem <= 232448, "shared memory of a CTA");
    Wave w;
    const cudaError_t e = launch_wave<weights_kernel<D, kF8>>(S::kThreads, kSmem, w);
    if (e != cudaSuccess) return e;
    weights_kernel<D, kF8><<<(unsigned)std::min((uint64_t)p.items, w.ctas()), S::kThreads, kSmem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attention_weights(const splitzip_attention_args& a, const float* weights_in, float* weights_out,
                                     const WaitTest& test, cudaStream_t s) {
    WeightsParams p;
    p.a = a;
    p.in = weights_in;
    p.out = weights_out;
    p.group = a.q_heads / a.kv_heads;
    p.tokens = kRowTile / p.group;
    p.items = a.batch * a.kv_heads * ((a.kv_tokens + kSlotTile - 1) / kSlotTile);
    p.by_heads = make_chunk_div(a.batch * a.kv_heads);
    p.by_kv_heads = make_chunk_div(a.kv_heads);
    p.by_tokens = make_chunk_div(p.tokens);
    p.window = a.window ? std::min(a.window, 0x80000000u) : 0x80000000u;
    p.wait_limit = test.limit ? test.limit : wait_limit((a.q_tokens + p.tokens - 1) / p.tokens);  // a wait lasts an item at most
    p.test_cta = test.cta;
    p.test_tile = test.tile;
    const bool f8 = a.cache_format == SPLITZIP_FORMAT_E5M2;
    if (!make_map(p.qmap, a.q, 2, a.head_dim, a.q_heads, a.q_tokens, a.batch, p.group, p.tokens, true, &p.one_q) ||
        !make_map(p.kmap, a.k, f8 ? 1 : 2, a.head_dim, a.kv_heads, a.kv_tokens, a.batch, 1, kSlotTile, false, &p.one_k))
        return cudaErrorInvalidValue;
    if (a.head_dim == 64) return f8 ? launch<64, true>(p, s) : launch<64, false>(p, s);
    return f8 ? launch<128, true>(p, s) : launch<128, false>(p, s);
}

}  // namespace splitzip
