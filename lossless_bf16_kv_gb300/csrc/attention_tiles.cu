// attention_tiles.cu -- attention of many query rows on the tensor cores
// (sm_103a).
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
// it.  The queries are then FP16 too, each row scaled by a power of two.
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
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "attention.cuh"
#include "tcgen.cuh"
#include "tensor_map.h"

namespace splitzip {
namespace {

constexpr int kBN = 128;       // slots per step
constexpr int kTileM = 128;    // query rows per tile
constexpr int kSoftmax = 512;  // threads
constexpr int kPart = 16;      // scores turned into P at a time: eight words
// log2 of P at a maximum just taken, and of how far a P may exceed that.
template <bool kF8>
constexpr float kLift = kF8 ? 9.0f : 0.0f;
template <bool kF8>
constexpr float kLazy = kF8 ? 6.9f : 8.0f;

template <int D, bool kF8>
struct TilesShape {
    static constexpr int kKV = kBN * D * 2;      // bytes of a key or value tile in 16 bits
    static constexpr int kRaw = kBN * D;         // bytes of one in E5M2
    static constexpr int kQ = kTileM * D * 2;    // bytes of a query tile
    static constexpr int kStages = D == 128 ? (kF8 ? 4 : 5) : (kF8 ? 6 : 8);
    static constexpr int kRaws = kF8 ? 2 : 0;
    // Threads: softmax, a warp for the products, one for the loads, and those that
    // tend the values; registers of a softmax thread and of another.
    static constexpr int kTend = kF8 ? 6 : 2, kThreads = kSoftmax + 32 * (2 + kTend);
    static constexpr int kRegs = kF8 ? 96 : 104, kOtherRegs = kF8 ? 48 : 64;
    static_assert(kThreads % 128 == 0 && kSoftmax * kRegs + (kThreads - kSoftmax) * kOtherRegs <= kThreads * (65536 / kThreads / 8 * 8),
                  "register shares add up to what the CTA is launched with");
    static constexpr int kRowFloats = D + 4;     // of a row's partial result: o, m, l
    // Tensor memory: S of the query tiles from column 0, O, and P over S or apart.
    static constexpr bool kApart = D == 64;
    static constexpr uint32_t kColO = 2 * kBN, kColP = kApart ? kColO + 2 * D : 0, kStepP = kApart ? kBN / 2 : kBN;
    static constexpr uint32_t kHalfP = kApart ? kBN / 4 : kBN / 2;  // over S, each half of P over its own scores
    static constexpr int kUsed = 2 * kQ + kStages * kKV + kRaws * kRaw;
    static_assert(kUsed >= 2 * kTileM * kRowFloats * 4, "partial results take the place of the tiles");
};

struct TilesParams {
    splitzip_attention_args a;
    CUtensorMap qmap, kmap, vmap;
    uint32_t group, tokens;   // query tokens per tile: 128 / group
    uint32_t row_ctas, splits;
    uint32_t one_q, one_k, one_v;  // the batch is one sequence: coordinate 0
    uint32_t* status;
    uint32_t wait_limit;
    uint32_t test_cta, test_tile;  // a copy that a test has left out
};

struct TilesShared {
    uint64_t full[8], empty[8];  // ring stage: tile there in 16 bits, free again
    uint64_t ok[8];              // step i mod 8: its values are fit for the product
    uint64_t raw_full[3], raw_empty[3];  // E5M2 tiles
    uint64_t q_full;
    uint64_t s_full[2], p_full[2], o_full[2], drained;  // of the query tiles
    uint64_t s_free[2], o_done[2];  // P apart: S is in registers, a step's O is there
    WaitLimit wait;
    uint32_t tmem, odd;
    // This CTA's work: sequence, head, first query token; the first slot of step
    // 0, the step that jumps from the sinks to the window and to where.
    uint32_t b, h, t0, steps;
    int32_t s0, jump_at, jump_to;
    int32_t n, first, sinks, p0, p1;
    uint32_t window;
    int32_t upto[2], after[2], whole_sinks;  // WholeTiles of the query tiles
    float row[2][2][kTileM];  // exchanged by the two threads of a row
};

// The first slot of each step in turn.
struct StepSlots {
    int32_t s0, at, to, i;
    __device__ __forceinline__ explicit StepSlots(const volatile TilesShared& sh)
        : s0(sh.s0), at(sh.jump_at), to(sh.jump_to), i(0) {}
    __device__ __forceinline__ void next() { s0 = ++i == at ? to : s0 + kBN; }
};
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

template <int D, bool kF8, bool kTwin>
__device__ __forceinline__ void load_tiles(const TilesParams& p, TilesShared& sh, uint8_t* qs, uint8_t* ring, uint8_t* raw) {
    using S = TilesShape<D, kF8>;
    volatile WaitLimit* wait = &sh.wait;
    const int32_t b = (int32_t)sh.b, h = (int32_t)sh.h;
    const uint32_t steps = sh.steps;
    if (!kF8) {
        mbar_arrive_expect_tx(&sh.q_full, 2 * p.tokens * p.group * D * 2);
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int i = 0; i < D / 64; i++)
                tma_load4(qs + t * S::kQ + i * (kTileM * 128), &p.qmap, 64 * i, h * (int32_t)p.group,
                          (int32_t)(sh.t0 + (kTwin ? 0 : t * p.tokens)), p.one_q ? 0 : b, &sh.q_full);
    }
    constexpr int kN = kF8 ? S::kRaws : S::kStages;
    uint64_t* full = kF8 ? sh.raw_full : sh.full;
    uint64_t* empty = kF8 ? sh.raw_empty : sh.empty;
    StepSlots slots(sh);
    const uint32_t left_out = blockIdx.x == p.test_cta ? p.test_tile : 0xFFFFFFFFu;
    uint32_t i = 0;
    for (uint32_t st = 0, ph = 0; i < 2 * steps; i++) {
        if (i >= kN && !mbar_wait_bounded(&empty[st], ph ^ 1, wait)) break;
        const bool v = i & 1;
        const int32_t bb = (v ? p.one_v : p.one_k) ? 0 : b;
        mbar_arrive_expect_tx(&full[st], kF8 ? S::kRaw : S::kKV);
        if (i == left_out) {
        } else if (kF8) {
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
    if (!kF8) mbar_wait_bounded<true>(&sh.q_full, 0, wait);
    for (uint32_t x = i > kN ? i - kN : 0; x < i; x++) mbar_wait_bounded<true>(&full[x % kN], (x / kN) & 1, wait);
}

template <int D, bool kF8, bool kTwin>
__device__ __forceinline__ void issue_products(TilesShared& sh, uint32_t tmem, const uint8_t* qs, const uint8_t* ring) {
    using S = TilesShape<D, kF8>;
    constexpr uint32_t kShapeS = mma_shape(kF8, kBN, false), kShapeO = mma_shape(kF8, D, true);
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
template <int D, bool kF8>
__device__ __forceinline__ void tend_values(TilesShared& sh, uint8_t* ring, const uint8_t* raw, uint32_t thread) {
    using S = TilesShape<D, kF8>;
    volatile WaitLimit* wait = &sh.wait;
    const uint32_t lane = thread & 31, steps = sh.steps;
    StepSlots slots(sh);
    const WholeTiles whole(sh, sh.p0, sh.p1);
    if constexpr (kF8) {
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
            if (!mbar_wait_bounded(&sh.full[st], ph, wait)) break;
            if (sh.p0 < 0 || !whole(slots.s0)) {
                bool found = false;
                uint4* tile = reinterpret_cast<uint4*>(ring + st * S::kKV);
#pragma unroll 4
                for (uint32_t x = thread; x < S::kKV / 16; x += 32 * S::kTend) {
                    const uint4 v = tile[x];
                    const uint4 f = make_uint4(finite_or_zero<false>(v.x), finite_or_zero<false>(v.y), finite_or_zero<false>(v.z),
                                               finite_or_zero<false>(v.w));
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
template <int D, bool kF8, bool kTwin>
__device__ __forceinline__ bool softmax_rows(const TilesParams& p, TilesShared& sh, uint32_t tmem, uint32_t t, uint32_t half,
                                             uint32_t r, uint32_t pair_bar, int32_t pos, float scale, float& m, float& l) {
    volatile WaitLimit* wait = &sh.wait;
    using S = TilesShape<D, kF8>;
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
        const float mine = own > m + (kLift<kF8> + kLazy<kF8>) ? ceilf(own) - kLift<kF8> : m;  // from -inf too
        const float use = mine == -INFINITY ? 0.0f : mine;
        const uint64_t sc = pair(scale, scale), neg = pair(-use, -use);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 64 / kPart; c++) {
            uint32_t w[8];
#pragma unroll
            for (int x = 0; x < kPart; x += 2) {
                const int y = kPart * c + x;
                float u, v;
                unpair(fma2(pair(__uint_as_float(s[y >> 5][y & 31]), __uint_as_float(s[y >> 5][(y & 31) + 1])), sc, neg), u, v);
                u = exp2_approx(u);
                v = exp2_approx(v);
                sum[(x >> 1) & 1] = add2(sum[(x >> 1) & 1], pair(u, v));
                // P in 16 bits: an error of up to 2^-8 (BF16) or 2^-11 (FP16, down to 2^-22 of
                // the row's largest) of each term.
                w[x >> 1] = pack2<kF8>(u, v);
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
            sh.row[t][half][r] = mine;
            if (named_any(pair_bar, 64, !ready)) return false;
            const float now = fmaxf(mine, sh.row[t][half ^ 1][r]);
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
                        const float2 y = unpack2<kF8>(w[x]);
                        w[x] = pack2<kF8>(y.x * g, y.y * g);
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
template <int D, bool kF8, bool kTwin>
__device__ __forceinline__ void read_output(const TilesParams& p, const TilesShared& sh, uint32_t oa, uint32_t t, int32_t pos, int c,
                                            float (&o)[32]) {
    constexpr int kElem = kF8 ? 1 : 2;
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
        const uint8_t* vbase = static_cast<const uint8_t*>(p.a.v.data) + ((int64_t)sh.b * p.a.v.stride_b + (int64_t)sh.h * p.a.v.stride_h + 32 * c) * kElem;
        StepSlots slots(sh);
        for (uint32_t i = 0; i < steps; i++, slots.next()) {
            if ((kTwin && (i & 1) != t) || (sh.p0 >= 0 && whole(slots.s0))) continue;
            for (int32_t s = slots.s0; s < min(slots.s0 + kBN, n); s++) {
                if (!((uint32_t)(pos - s) < window || (s < sinks && s <= pos))) continue;
                const uint8_t* row = vbase + s * p.a.v.stride_t * kElem;
#pragma unroll
                for (int x = 0; x < 32; x++) {
                    const float v = kF8 ? __half2float(__ushort_as_half((unsigned short)(row[x] << 8)))
                                        : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[x]);
                    if (!isfinite(v)) o[x] += v;
                }
            }
        }
    }
}

template <int D, bool kF8, bool kTwin>
__global__ void __launch_bounds__(TilesShape<D, kF8>::kThreads, 1) tiles_kernel(const __grid_constant__ TilesParams p) {
    using S = TilesShape<D, kF8>;
    extern __shared__ __align__(1024) uint8_t qs[];
    TilesShared& sh = *reinterpret_cast<TilesShared*>(qs + S::kUsed);
    uint8_t* ring = qs + 2 * S::kQ;             // tiles of D / 64 blocks of 128 rows of 128 bytes, as qs
    uint8_t* raw = ring + S::kStages * S::kKV;  // E5M2 tiles as they are
    const uint32_t warp = threadIdx.x >> 5;

    if (warp == 16) tmem_alloc<512>(&sh.tmem);
    if (threadIdx.x == 0) {
        const splitzip_attention_args& a = p.a;
        // The last row tiles see the most slots: they go first.
        const uint32_t unit = blockIdx.x / p.splits, split = blockIdx.x - unit * p.splits;
        const uint32_t heads = a.batch * a.kv_heads, rc = p.row_ctas - 1 - unit / heads, bh = unit % heads;
        const uint32_t b = bh / a.kv_heads, h = bh - b * a.kv_heads;
        const Mask mask(a, b);
        const uint32_t t0 = rc * 2 * p.tokens, t1 = min(t0 + 2 * p.tokens, a.q_tokens);
        sh.p0 = mask.first + (int32_t)t0;
        sh.p1 = mask.first + (int32_t)t1 - 1;
        const SlotTiles tiles(mask, sh.p0, sh.p1, kBN);
        const uint32_t j0 = (uint32_t)((uint64_t)tiles.count * split / p.splits);
        sh.b = b;
        sh.h = h;
        sh.t0 = t0;
        sh.steps = (uint32_t)((uint64_t)tiles.count * (split + 1) / p.splits) - j0;
        sh.s0 = (int32_t)(tiles.tile(j0) * kBN);
        sh.jump_at = j0 < tiles.head ? (int32_t)(tiles.head - j0) : -1;
        sh.jump_to = (int32_t)(tiles.from * kBN);
        sh.n = mask.n;
        sh.first = mask.first;
        sh.sinks = mask.sinks;
        sh.window = mask.window;
        for (int t = 0; t < 2; t++) {
            // No tile of slots is whole for a tile without queries.
            const uint32_t ta = t0 + (kTwin ? 0 : t * p.tokens), tb = min(ta + p.tokens, a.q_tokens);
            const WholeTiles whole(sh, mask.first + (int32_t)ta, mask.first + (int32_t)tb - 1);
            sh.upto[t] = ta < a.q_tokens ? whole.upto : -1;
            sh.after[t] = whole.after;
            sh.whole_sinks = whole.sinks;
        }
        for (int i = 0; i < 8; i++) {
            mbar_init(&sh.full[i], kF8 ? S::kTend / 2 : 1);
            mbar_init(&sh.empty[i], 1);
            mbar_init(&sh.ok[i], kF8 ? S::kTend / 2 : S::kTend);
        }
        for (int i = 0; i < 3; i++) {
            mbar_init(&sh.raw_full[i], 1);
            mbar_init(&sh.raw_empty[i], S::kTend / 2);
        }
        mbar_init(&sh.q_full, kF8 ? kSoftmax : 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i], 8);
            mbar_init(&sh.o_full[i], 1);
            mbar_init(&sh.s_free[i], 8);
            mbar_init(&sh.o_done[i], 1);
        }
        mbar_init(&sh.drained, 1);
        sh.wait.given_up = sh.odd = 0;
        sh.wait.limit = p.wait_limit;
        fence_mbar_init();
    }
    if (!kF8 && threadIdx.x < 256) {
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
            if (warp == 16) issue_products<D, kF8, kTwin>(sh, tmem, qs, ring);
            else if (warp > 17) tend_values<D, kF8>(sh, ring, raw, threadIdx.x - (kSoftmax + 64));
            else if ((threadIdx.x & 31) == 0) load_tiles<D, kF8, kTwin>(p, sh, qs, ring, raw);
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
            const bool valid = r < p.tokens * p.group && tok < p.a.q_tokens;
            const int32_t pos = valid ? max(-1, sh.first + (int32_t)tok) : -1;
            float scale = p.a.scale * kLog2e;
            // Only where there are steps: the products, which wait for all queries, keep this
            // apart from the partial results that take the queries' place.
            if (kF8 && sh.steps) {
                // This thread's half of its query row: FP16 of the row scaled by a power of two.
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const __nv_bfloat16*>(p.a.q.data) + (int64_t)sh.b * p.a.q.stride_b + (int64_t)tok * p.a.q.stride_t +
                    (int64_t)(sh.h * p.group + g) * p.a.q.stride_h) + half * (D / 16);
                uint4 v[D / 16];
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < D / 16; i++) {
                    v[i] = valid ? src[i] : make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int x = 0; x < 4; x++) top = max(top, max(w[x] & 0x7FFFu, w[x] >> 16 & 0x7FFFu));
                }
                sh.row[t][half][r] = __uint_as_float(top);
                named_sync(pair_bar, 64);
                const float power = row_power(max(top, __float_as_uint(sh.row[t][half ^ 1][r])));
                scale /= power;
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
            go = softmax_rows<D, kF8, kTwin>(p, sh, tmem + (((warp & 3) * 32) << 16), t, half, r, pair_bar, pos, scale, m, l);
        }
        // The row's sum, of both halves in the same order.
        __syncwarp();
        sh.row[t][half][r] = l;
        named_sync(pair_bar, 64);
        l = sh.row[t][0][r] + sh.row[t][1][r];
        if ((threadIdx.x & 31) == 0 && !go) atomicOr(p.status, kStatusTimeout);
        if (!go) l = __int_as_float(0x7FC00000);  // a wait that gave up: NaN

        // Derived again rather than kept through the loop.
        const uint32_t rr = opaque(threadIdx.x) & 127;
        const uint32_t tok = sh.t0 + (kTwin ? 0 : t * p.tokens) + rr / p.group, g = rr % p.group, hq = sh.h * p.group + g;
        const bool valid = rr < p.tokens * p.group && tok < p.a.q_tokens;
        const int32_t pos = valid ? max(-1, sh.first + (int32_t)tok) : -1;
        const uint32_t oa = tmem + (((warp & 3) * 32) << 16) + S::kColO + t * D;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out.data) + (int64_t)sh.b * p.a.out.stride_b +
                             (int64_t)tok * p.a.out.stride_t + (int64_t)hq * p.a.out.stride_h;
        float* lse = p.a.lse ? p.a.lse + ((uint64_t)sh.b * p.a.q_heads + hq) * p.a.q_tokens + tok : nullptr;
        if (!kTwin && p.splits == 1) {
            const float inv = 1.0f / l;
            const bool none = l == 0.0f;  // nothing seen, or scores of -infinity alone
#pragma unroll 1
            for (int c = half * (D / 64); c < (int)(half + 1) * (D / 64); c++) {  // this half's columns
                float o[32];
                read_output<D, kF8, kTwin>(p, sh, oa, t, pos, c, o);
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
                read_output<D, kF8, kTwin>(p, sh, oa, t, pos, c, o);
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
                if (xr >= p.tokens * p.group || xt >= p.a.q_tokens) continue;
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
                __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.a.out.data) + (int64_t)sh.b * p.a.out.stride_b +
                                    (int64_t)xt * p.a.out.stride_t + (int64_t)xh * p.a.out.stride_h;
                *reinterpret_cast<uint2*>(to + c) =
                    none ? make_uint2(0, 0) : make_uint2(pack2<false>(v.x * inv, v.y * inv), pack2<false>(v.z * inv, v.w * inv));
                if (c == 0 && p.a.lse)
                    p.a.lse[((uint64_t)sh.b * p.a.q_heads + xh) * p.a.q_tokens + xt] = none ? -INFINITY : (mm + log2f(ll)) * kLn2;
            }
            __syncwarp();
            cluster_sync();  // this CTA's rows have been read
        }
        tcgen_fence_before();
    }
    __syncthreads();
    tcgen_fence_after();
    if (warp == 16) tmem_free<512>(tmem);
}

template <int D, bool kF8, bool kTwin>
cudaError_t launch(const TilesParams& p, uint32_t ctas, cudaStream_t s) {
    constexpr int kSmem = TilesShape<D, kF8>::kUsed + (int)sizeof(TilesShared);
    static_assert(kSmem <= 232448, "shared memory of a CTA");
    Wave w;
    const cudaError_t e = launch_wave<tiles_kernel<D, kF8, kTwin>>(TilesShape<D, kF8>::kThreads, kSmem, w);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(TilesShape<D, kF8>::kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tiles_kernel<D, kF8, kTwin>, p);
}

}  // namespace

// All rows in one tile, and slots for two: both tiles of a CTA hold the rows and take every other slot tile.
inline bool is_twin(const splitzip_attention_args& a) {
    return a.q_tokens <= kTileM / (a.q_heads / a.kv_heads) && a.kv_tokens > kBN;
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
    // The splits (one cluster) with the least time, as waves of clusters times the steps
    // of a split plus kSplitCost steps for a CTA's start, join and end.  A cluster lies
    // within one of the GPU's groups of SMs, so fewer of the large ones run at once (as
    // cudaOccupancyMaxActiveClusters has it): 16 units of 2048 slots of 64 take 20.6 us
    // in 8 splits, two waves, and 11.7 in 6.
    constexpr uint64_t kSplitCost = 4, kAtOnce[9] = {0, kSms, 76, 46, 36, 28, 23, 15, 15};
    uint64_t best = ~0ull;
    p.splits = 1;
    for (uint64_t n = 1; n <= 8 && (n == 1 || 2 * n <= most); n++) {
        const uint64_t time = (units + kAtOnce[n] - 1) / kAtOnce[n] * (((most + n - 1) / n + at_once - 1) / at_once + kSplitCost);
        if (time < best) {
            best = time;
            p.splits = (uint32_t)n;
        }
    }
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
        if (a.head_dim == 64) return f8 ? launch<64, true, kTwin>(p, ctas, s) : launch<64, false, kTwin>(p, ctas, s);
        return f8 ? launch<128, true, kTwin>(p, ctas, s) : launch<128, false, kTwin>(p, ctas, s);
    };
    return is_twin(a) ? go(std::true_type()) : go(std::false_type());
}

}  // namespace splitzip
