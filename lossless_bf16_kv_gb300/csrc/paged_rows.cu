// paged_rows.cu -- attention of few query rows over pages (sm_103a).
//
// The query rows of one sequence and key/value head (its new tokens times the group's
// query heads) in tiles of 8 or 16, a tile's slots in splits, one CTA each, each of
// its four warps with its own slot tiles, running maximum, sum and output as in
// attention_rows.cu, joined at the end in a fixed order.  Every key and value is
// read once: HBM bounds BF16 (16 single tokens over 16k caches of 8 heads of 128, 32 query
// heads: 150 us, 7.1 TB/s) and E5M2 (80, 6.7); of quantised codes the instructions that
// widen them and their latencies (99 us in 8 bits, 76 in 4; 5.6 and 3.7 TB/s, issue slots
// half used).
//
// The products are transposed: S^T = K Q^T and O^T += V^T P^T, with slots, then a
// head's values as the 16 rows of an m16n8k16 product and the query rows as its 8
// columns.  One token of a group of up to eight heads fills those: half the products,
// exponentials and registers that 16 rows take.  P^T comes out of S^T by a
// transposition of 8 x 8 blocks between registers (movmatrix).
//
// A CTA's warps share a ring of slot tiles (64 or 128 slots, a quarter of them each
// warp's), which TMA fills page by page, swizzled as ldmatrix reads them.
// The warps take turns at loading the next tile, so the cost of that is shared, and
// each has the page numbers of its next turn four tiles ahead.  What no query sees is
// not looked up (its page may have been given away): it is loaded from behind the
// pool's last page, as zeros.
//
// Quantised codes become FP16 in registers on their way from shared memory to the
// products, exactly: codes by a byte permute and a subtraction (INT8) or a conversion
// (E2M1).  The keys' powers multiply the scores' sums over a block, in 32 bits.  The
// values' multiply the codes, as their slots are what is summed over: they are made
// FP16 once per tile and slot by one lane, those of neighbouring slots side by side.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "attention_rows.cuh"
#include "pages.cuh"
#include "ring_turns.h"
#include "tcgen.cuh"
#include "tensor_map.h"

namespace splitzip {
namespace {

struct PagedRowsParams {
    splitzip_paged_attention_args a;
    CUtensorMap kmap, vmap;
    uint32_t group, page_shift, row_tiles;
    uint32_t splits, cluster;  // of each row tile; splits 0: shared out by the sequences' lengths
    uint32_t rows_upto;   // only sequences with no more query rows than this
    uint32_t box, boxes;  // slots to a copy, and copies to a tile
    uint32_t bulk_exps;   // a page's exponent bytes of a head are contiguous, in multiples of 16 bytes
    uint32_t* counters;
    float* partials;
    uint32_t* status;
    uint32_t wait_limit;
    uint32_t test_cta, test_tile;  // a copy that a test has left out
};

// Slots of a tile that a warp takes.  32 give it two independent blocks of work, and half
// the waits of 16: 16 single tokens over 16k caches of 8 heads of 128, 4 query heads to
// each, E2M1 76 us (91 with 16), of 16 query heads 114 (140), E5M2 100 (108), INT8 126
// (146).  They do not fit in BF16, and in 8 bits only three CTAs of them fit an SM: in
// E5M2 that costs nothing (88 us in both), but INT8's widening wants the fourth one in
// tiles of 8 rows (24 windows of 4096 42 us, with 32 slots 46).
constexpr uint32_t warp_slots(uint32_t format, uint32_t d, uint32_t tile_rows) {
    return format == kBf16 || (format == kInt8 && tile_rows == 8) ? 2048 / d : 32;
}
// CTAs to an SM, by registers and shared memory.
constexpr uint32_t ctas_per_sm(uint32_t format, uint32_t d, uint32_t tile_rows) {
    return format != kBf16 && tile_rows == 8 && (d == 64 || format != kE5m2) ? 4 : 3;
}

template <int D, int kFmt, int kTileRows>
struct PagedShape {
    static constexpr int kRow = kRowBytes<D, kFmt>;
    static constexpr int kPart = warp_slots(kFmt, D, kTileRows);
    static constexpr int kSlots = kWarpsRows * kPart;        // slots per tile
    static constexpr int kTile = kSlots * kRow;              // bytes of its keys, and of its values
    static constexpr int kStages = kTile >= 16384 ? 2 : kTile >= 8192 ? 3 : 4;
    static constexpr int kExps = kQuantised<kFmt> ? 4 * kSlots : 0;  // bytes of its keys' exponents, and of its values'
    // Shared memory: the rings of tiles and of exponents, the values' powers, queries.
    static constexpr int kAtExps = kStages * 2 * kTile, kAtPowers = kAtExps + kStages * 2 * kExps;
    static constexpr int kAtQueries = kAtPowers + 2 * kExps;
    static_assert(kTile % 1024 == 0, "swizzled tiles");
};
// A CTA's part of the work: row tile rt of sequence b and head h, and which of its
// splits; the CTA with the first of those.
struct PagedPart {
    uint32_t b, h, rt, split, splits, first;
};

// Sequences whose work is shared out in one launch, by tables of their slot tiles.
constexpr uint32_t kMostShared = 1024;
// The least slot tiles of a split where work is shared out.
constexpr uint32_t kLeastTiles = 4;

// Shares the work out by the sequences' lengths: splits of at most T slot tiles, with the
// smallest T for which they are no more than the grid's CTAs.  `part` comes back with
// splits = 0 where this CTA has none.  All threads; `table` holds a word for each
// sequence.  T is found by bisection, by one warp: about a microsecond in all, with
// the loads of the sequences' ranges.
template <int kTileRows, int kSlots, class Params>
__device__ __forceinline__ void share_out(const Params& p, uint32_t* table, PagedPart& part) {
    const splitzip_paged_attention_args& a = p.a;
    constexpr uint32_t kTiles = 0x3FFFFFFFu;  // of a word; above, how many row tiles the sequence has
    for (uint32_t b = threadIdx.x; b < a.batch; b += 32 * kWarpsRows) {
        const Sequence seq(a, b);
        const uint32_t rows = (uint32_t)seq.count * p.group;
        uint32_t word = 0;
        if (rows && rows <= p.rows_upto) {
            const Mask mask(seq.n, seq.count, a.window, a.sinks);
            word = SlotTiles(mask, mask.first, seq.n - 1, kSlots).count | (rows + kTileRows - 1) / kTileRows << 30;
        }
        table[b] = word;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const uint32_t lane = threadIdx.x, heads = a.pool.kv_heads;
        uint32_t most = 1;
        for (uint32_t b = lane; b < a.batch; b += 32) most = max(most, table[b] & kTiles);
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        const auto ctas_of = [&](uint32_t word, uint32_t t) { return (word >> 30) * heads * max(1u, ((word & kTiles) + t - 1) / t); };
        uint32_t lo = max(kLeastTiles, (most + 254) / 255), hi = max(lo, most);  // a counter of 8 bits counts up to 255
        while (lo < hi) {
            const uint32_t t = (lo + hi) / 2;
            uint32_t sum = 0;
            for (uint32_t b = lane; b < a.batch; b += 32) sum += ctas_of(table[b], t);
            if (__reduce_add_sync(0xFFFFFFFFu, sum) <= gridDim.x) hi = t;
            else lo = t + 1;
        }
        uint32_t left = blockIdx.x;
        if (lane == 0) part.splits = 0;
        for (uint32_t b = 0; b < a.batch; b += 32) {
            const uint32_t word = b + lane < a.batch ? table[b + lane] : 0, here = ctas_of(word, lo);
            uint32_t upto = here;
#pragma unroll
            for (int i = 1; i < 32; i *= 2) {
                const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, upto, i);
                if (lane >= (uint32_t)i) upto += x;
            }
            const uint32_t found = __ballot_sync(0xFFFFFFFFu, left < upto);
            if (found) {
                if (lane == (uint32_t)__ffs(found) - 1) {
                    const uint32_t at = left - (upto - here), splits = max(1u, ((word & kTiles) + lo - 1) / lo);
                    const uint32_t unit = at / splits;
                    part.b = b + lane;
                    part.h = unit % heads;
                    part.rt = unit / heads;
                    part.split = at - unit * splits;
                    part.first = blockIdx.x - part.split;
                    part.splits = splits;
                }
                break;
            }
            left -= __shfl_sync(0xFFFFFFFFu, upto, 31);
        }
    }
    __syncthreads();
    fence_async_proxy();  // the tables' place is the tiles', which TMA writes
}

template <int kStages, int kTileRows>
struct PagedRowsShared {
    PagedPart part;
    uint64_t full[kStages], empty[kStages];
    WaitLimit wait;
    RingTurns<kStages> turns;  // tiles whose copies have been issued
    float scale[kTileRows];
    RowsShared<kTileRows> join;
};

// Byte offset of 16-byte chunk c of row r in a tile as TMA writes it: rows of 256
// bytes as two blocks of 128.
template <int kRow, int kSlots>
__device__ __forceinline__ uint32_t tile_at(uint32_t r, uint32_t c) {
    if (kRow == 256) return (c >> 3) * (kSlots * 128) + chunk_at<128>(r, c & 7u);
    return chunk_at<kRow>(r, c);
}

// Position of a head's value d in the products' contraction index, such that the four
// consecutive bytes of a fragment's row that a lane holds are the indices that the
// fragment layout gives it: four values, or eight of E2M1, the first four of them
// in one step and the others in the next.
template <int kFmt>
__device__ __forceinline__ uint32_t place(uint32_t d) {
    if (kFmt == kBf16) return d;
    if (kFmt == kE2m1) return (d & ~31u) + ((d & 4u) << 2) + ((d & 24u) >> 2) + (d & 1u) + ((d & 2u) << 2);
    return (d & ~15u) + e5m2_place(d & 15u);
}

// 2^(e - 127) for exponent byte kByte of four; infinity for 255.
template <int kByte>
__device__ __forceinline__ float power_of(uint32_t x) {
    return __uint_as_float((kByte < 3 ? x << (23 - 8 * kByte) : x >> 1) & 0x7F800000u);
}
// Whether one of four exponent bytes is 255.
__device__ __forceinline__ bool has_nan(uint32_t x) { return (((x & 0x7F7F7F7Fu) + 0x01010101u) & x & 0x80808080u) != 0; }

// The transpose of an 8 x 8 matrix of 16-bit values, a row to four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// NB: blocks of 8 query rows.
template <int D, int kFmt, int NB>
__global__ void __launch_bounds__(32 * kWarpsRows, ctas_per_sm(kFmt, D, 8 * NB)) paged_rows_kernel(const __grid_constant__ PagedRowsParams p) {
    using S = PagedShape<D, kFmt, 8 * NB>;
    constexpr bool kHalf = kWide<kFmt>;  // operands FP16, else BF16
    constexpr int kTileRows = 8 * NB;
    constexpr bool kBlockSums = kQuantised<kFmt> && !(kFmt == kE2m1 && D == 64);  // a step's 16 values are of one block
    constexpr int KS = D / 16;           // steps of the scores, and 16-value blocks of the output
    constexpr int PS = S::kPart / 16;    // 16-slot blocks of a warp's scores, steps of its output
    constexpr int kChunks = S::kRow / 16;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* qs = smem + S::kAtQueries;
    auto& sh = *reinterpret_cast<PagedRowsShared<S::kStages, kTileRows>*>(qs + kTileRows * D * 2);
    const splitzip_paged_attention_args& a = p.a;
    const splitzip_pool& pool = a.pool;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool shared = p.splits == 0;
    if (shared) share_out<kTileRows, S::kSlots>(p, reinterpret_cast<uint32_t*>(smem), sh.part);
    // A grid that was let start before the one ahead of it has ended ends after that: the
    // last CTA waits for it, and the others leave their SMs to those that are to come.
    struct AtEnd {
        __device__ ~AtEnd() {
            if (blockIdx.x == gridDim.x - 1) wait_prerequisite_grid();
        }
    } at_end;
    uint32_t b, h, rt, split, splits, first_cta;
    if (shared) {
        const PagedPart& part = sh.part;
        if (!part.splits) return;
        b = part.b, h = part.h, rt = part.rt, split = part.split, splits = part.splits, first_cta = part.first;
    } else {
        splits = p.splits;
        const uint32_t unit = blockIdx.x / splits, bh = unit / p.row_tiles;
        split = blockIdx.x - unit * splits, rt = unit - bh * p.row_tiles, b = bh / pool.kv_heads, h = bh - b * pool.kv_heads;
        first_cta = blockIdx.x - split;
    }
    const Sequence seq(a, b);
    const uint32_t rows = (uint32_t)seq.count * p.group;
    const uint32_t r0 = rt * kTileRows, r1 = min(r0 + kTileRows, rows);
    if (r0 >= rows || rows > p.rows_upto) return;  // with all of its cluster
    const Mask mask(seq.n, seq.count, a.window, a.sinks);
    const int32_t p0 = mask.first + (int32_t)(r0 / p.group), p1 = mask.first + (int32_t)((r1 - 1) / p.group);
    const SlotTiles tiles(mask, p0, p1, S::kSlots);
    const uint32_t j0 = (uint32_t)((uint64_t)tiles.count * split / splits);
    const uint32_t j1 = (uint32_t)((uint64_t)tiles.count * (split + 1) / splits);

    uint8_t* powers = smem + S::kAtPowers + warp * (8 * S::kPart);  // of this warp's values, [block][slot]
    volatile WaitLimit* wait = &sh.wait;
    const int32_t* table = a.table + (uint64_t)b * a.table_width;
    const uint32_t in_page = pool.page_tokens - 1, count = j1 - j0;

    // Lane i < boxes: the page of copy i of the CTA's n-th tile; `pages` where no query sees it.
    bool lost = false;  // a page that a query sees is outside the pool
    auto look_up = [&](uint32_t n) -> uint32_t {
        if (lane >= p.boxes || n >= count) return pool.pages;
        const int32_t s = (int32_t)(tiles.tile(j0 + n) * S::kSlots + p.box * lane);
        // The last slot is behind the start of the first query's window, or a sink.
        if (s > p1 || !((int64_t)s + p.box > (int64_t)p0 - (int64_t)mask.window + 1 || s < mask.sinks)) return pool.pages;
        const uint32_t page = (uint32_t)table[s >> p.page_shift];
        if (page < pool.pages) return page;
        lost = true;
        return pool.pages;
    };
    // The whole warp: the n-th tile into its stage, which is free.
    auto load = [&](uint32_t n, uint32_t page) {
        const uint32_t stage = n % S::kStages, s0 = tiles.tile(j0 + n) * S::kSlots;
        const bool bulk = kQuantised<kFmt> && p.bulk_exps;
        uint64_t* full = &sh.full[stage];
        uint8_t* dk = smem + stage * (2 * S::kTile);
        uint8_t* de = smem + S::kAtExps + stage * (2 * S::kExps);
        const uint8_t* kexps = pool.k.exponents + h * pool.k.exp_stride_h;
        const uint8_t* vexps = pool.v.exponents + h * pool.v.exp_stride_h;
        if (lane == 0) {
            sh.turns.put(n);
            mbar_arrive_expect_tx(full, 2 * S::kTile + (bulk ? 2 * S::kExps : 0));
        }
        __syncwarp();
        if (lane < p.boxes && !(blockIdx.x == p.test_cta && n == p.test_tile)) {
            const uint32_t first = p.box * lane;
            const int32_t at = (int32_t)((s0 + first) & in_page);
            constexpr int kBlocks = S::kRow == 256 ? 2 : 1, kBlockRow = S::kRow / kBlocks;
#pragma unroll
            for (int x = 0; x < kBlocks; x++) {
                tma_load4(dk + x * (S::kTile / 2) + first * kBlockRow, &p.kmap, 64 * x, at, (int32_t)h, (int32_t)page, full);
                tma_load4(dk + S::kTile + x * (S::kTile / 2) + first * kBlockRow, &p.vmap, 64 * x, at, (int32_t)h, (int32_t)page, full);
            }
            if (bulk) {  // where no query sees them, any page's: they multiply zeros
                const int64_t from = page < pool.pages ? page : 0;
                bulk_load(de + 4 * first, kexps + from * pool.k.exp_stride_p + 4 * at, 4 * p.box, full);
                bulk_load(de + S::kExps + 4 * first, vexps + from * pool.v.exp_stride_p + 4 * at, 4 * p.box, full);
            }
        }
        if (kQuantised<kFmt> && !bulk) {  // part of the phase, as the copies' bytes are
#pragma unroll 1
            for (uint32_t r = lane; r < S::kSlots; r += 32) {
                const uint32_t at = (s0 + r) & in_page, from = __shfl_sync(0xFFFFFFFFu, page, r / p.box);
                const int64_t some = from < pool.pages ? from : 0;
                cp_async4(de + 4 * r, kexps + some * pool.k.exp_stride_p + at * pool.k.exp_stride_t);
                cp_async4(de + S::kExps + 4 * r, vexps + some * pool.v.exp_stride_p + at * pool.v.exp_stride_t);
            }
            cp_async_arrive(full);
        }
    };
    uint32_t mine = S::kStages - 1 + warp;  // the next tile that this warp loads, and its pages
    uint32_t pages = look_up(mine);
    if (warp == 0) {
        if (lane == 0) {
            const uint32_t arrivals = kQuantised<kFmt> && !p.bulk_exps ? 33 : 1;
#pragma unroll
            for (int i = 0; i < S::kStages; i++) {
                mbar_init(&sh.full[i], arrivals);
                mbar_init(&sh.empty[i], kWarpsRows);
            }
            sh.wait.given_up = 0;
            sh.turns.clear();
            sh.wait.limit = p.wait_limit;
            fence_mbar_init();
            fence_async_proxy();
        }
        __syncwarp();
        for (uint32_t n = 0; n < min(count, (uint32_t)S::kStages - 1); n++) load(n, look_up(n));
    }

    // Queries: one warp per row, as FP16 of the scaled row where the cache is not BF16.
    for (uint32_t r = warp; r < kTileRows; r += kWarpsRows) {
        const uint32_t row = r0 + r, t = row / p.group, g = row - t * p.group;
        constexpr int V = D / 32;  // values per lane: 2 or 4
        uint32_t v[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; i++) v[i] = 0;
        if (row < r1) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(
                static_cast<const __nv_bfloat16*>(a.q.data) + (int64_t)(seq.row + t) * a.q.stride_t + (h * p.group + g) * a.q.stride_h);
#pragma unroll
            for (int i = 0; i < V / 2; i++) v[i] = src[lane * (V / 2) + i];
        }
        float power = 1.0f;
        if (kHalf) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < V / 2; i++) top = max(top, max(v[i] & 0x7FFFu, v[i] >> 16 & 0x7FFFu));
            power = row_power(__reduce_max_sync(0xFFFFFFFFu, top));
        }
#pragma unroll
        for (int i = 0; i < V / 2; i++) {
            const uint32_t d = place<kFmt>(lane * V + 2 * i);
            uint32_t w = v[i];
            if (kHalf) w = pack2<true>(__uint_as_float(v[i] << 16) * power, __uint_as_float(v[i] & 0xFFFF0000u) * power);
            *reinterpret_cast<uint32_t*>(qs + chunk_at<2 * D>(r, d / 8) + 2 * (d % 8)) = w;
        }
        // Never 0, which -infinity is multiplied by: such queries' scores are all 0 (the products
        // are below 2^25).
        if (lane == 0) sh.scale[r] = kHalf ? fmaxf(a.scale * kLog2e / power, 0x1p-126f) : a.scale * kLog2e;
    }
    __syncthreads();

    // This thread's query rows: 8 y + 2 (lane & 3) and the next.  m is the same for all
    // lanes that share a row, l each lane's own part.
    int32_t pos[NB][2];
    float scale[NB][2], m[NB][2], l[NB][2], o[KS][NB][4];
#pragma unroll
    for (int y = 0; y < NB; y++)
#pragma unroll
        for (int x = 0; x < 2; x++) {
            const uint32_t r = 8 * y + 2 * (lane & 3) + x;
            pos[y][x] = r0 + r < r1 ? mask.pos((r0 + r) / p.group) : -1;
            scale[y][x] = sh.scale[r];
            m[y][x] = -INFINITY;
            l[y][x] = 0.0f;
        }
#pragma unroll
    for (int k = 0; k < KS; k++)
#pragma unroll
        for (int y = 0; y < NB; y++)
#pragma unroll
            for (int x = 0; x < 4; x++) o[k][y][x] = 0.0f;

    uint32_t qf[KS][NB][2];  // the queries' fragments stay in registers
#pragma unroll
    for (int k = 0; k < KS; k += 2)
#pragma unroll
        for (int y = 0; y < NB; y++) {
            uint32_t r[4];
            ldmatrix4(r, smem_addr(qs) + chunk_at<2 * D>(8 * y + (lane & 7), 2 * k + (lane >> 3)));
            qf[k][y][0] = r[0], qf[k][y][1] = r[1], qf[k + 1][y][0] = r[2], qf[k + 1][y][1] = r[3];
        }
    bool odd = false;  // a value of a partly visible tile was infinite or NaN
    // A warp's part of a tile: keys at ks, values at vs, exponent bytes at e, the part's first row and slot.
    // kWhole: every query sees all of it.
    const auto walk = [&](auto is_whole, uint32_t ks, uint32_t vs, const uint32_t* e, uint32_t part, int32_t s0) {
        constexpr bool kWhole = decltype(is_whole)::value;
        bool rare = false;  // a block is NaN, or (INT8) its power above 2^5
        if constexpr (kQuantised<kFmt>) {
#pragma unroll
            for (uint32_t r = lane; r < 2 * S::kPart; r += 32) {  // the keys', then the values'
                const uint32_t s = r & (S::kPart - 1), x = e[r < S::kPart ? s : S::kSlots + s];
                rare |= kFmt == kInt8 ? above_5(x) : has_nan(x);
                const uint32_t lo = pack2<true>(power_of<0>(x), power_of<1>(x)), hi = pack2<true>(power_of<2>(x), power_of<3>(x));
                if (r >= S::kPart) {
                    uint16_t* to = reinterpret_cast<uint16_t*>(powers) + s;
                    to[0] = (uint16_t)lo, to[S::kPart] = (uint16_t)(lo >> 16);
                    to[2 * S::kPart] = (uint16_t)hi, to[3 * S::kPart] = (uint16_t)(hi >> 16);
                }
            }
            rare = __any_sync(0xFFFFFFFFu, rare);
            __syncwarp();
            if (rare) {  // infinity times 0 is NaN already, as the store leaves such blocks
                for (uint32_t r = lane; r < 4 * S::kPart; r += 32) {
                    uint16_t* at = reinterpret_cast<uint16_t*>(powers) + r;
                    if (*at == 0x7C00u) *at = 0x7E00u;
                }
                __syncwarp();
            }
        }
        // Scores of slots 16 i + lane / 4 and that + 8 (x >> 1) for this thread's rows (x & 1).
        float sc[PS][NB][4];
#pragma unroll
        for (int i = 0; i < PS; i++) {
#pragma unroll
            for (int y = 0; y < NB; y++)
#pragma unroll
                for (int x = 0; x < 4; x++) sc[i][y][x] = 0.0f;
            if constexpr (kFmt == kBf16) {
#pragma unroll
                for (int k = 0; k < KS; k++) {
                    uint32_t r[4];
                    ldmatrix4(r, ks + tile_at<S::kRow, S::kSlots>(part + 16 * i + (lane & 15), 2 * k + (lane >> 4)));
#pragma unroll
                    for (int y = 0; y < NB; y++) mma16816<kHalf>(sc[i][y], r, qf[k][y][0], qf[k][y][1]);
                }
            } else {
                uint32_t power[2] = {0, 0};  // the two slots' exponent bytes
                if constexpr (kQuantised<kFmt>) power[0] = e[16 * i + lane / 4], power[1] = e[16 * i + 8 + lane / 4];
                float sum[NB][4];  // over a block
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) {
                    uint32_t r[4];  // chunks c and c + 1 (x >> 1) of slots 0-7 and 8-15 (x & 1) of the block of slots
                    ldmatrix4(r, ks + chunk_at<S::kRow>(part + 16 * i + (lane & 15), c + (lane >> 4)));
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        const int block = kBlockSums ? (c + u) * (D / kChunks) / (D / 4) : 0;
                        const bool first = kBlockSums && (c + u) * (D / kChunks) % (D / 4) == 0;
                        const bool last = kBlockSums && (c + u + 1) * (D / kChunks) % (D / 4) == 0;
                        uint32_t w[2][4];
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            const uint32_t v = r[2 * u + x];
                            if constexpr (kFmt == kE5m2) {
                                w[x][0] = e5m2_01(v), w[x][1] = e5m2_23(v);
                            } else if constexpr (kFmt == kInt8) {
                                const uint32_t z = int8_bias(v);
                                w[x][0] = int8_pair<kInt8_01>(z), w[x][1] = int8_pair<kInt8_23>(z);
                            } else {
                                e2m1_pairs(w[x], v);
                                if constexpr (!kBlockSums) {
                                    // The 16 values of a step are of two blocks, a lane's eight of one.
                                    const float f = block_scale(power[x] >> (16 * u + ((lane & 2) << 2)) & 255u);
#pragma unroll
                                    for (int n = 0; n < 4; n++) w[x][n] = mul_half2(w[x][n], pack2<true>(f, f));
                                }
                            }
                        }
#pragma unroll
                        for (int n = 0; n < (kFmt == kE2m1 ? 2 : 1); n++) {
                            const int k = kFmt == kE2m1 ? 2 * (c + u) + n : c + u;
                            const uint32_t f[4] = {w[0][2 * n], w[1][2 * n], w[0][2 * n + 1], w[1][2 * n + 1]};
#pragma unroll
                            for (int y = 0; y < NB; y++) {
                                if (!kBlockSums) mma16816<true>(sc[i][y], f, qf[k][y][0], qf[k][y][1]);
                                else if (first && n == 0) mma16816_zero(sum[y], f, qf[k][y][0], qf[k][y][1]);
                                else mma16816<true>(sum[y], f, qf[k][y][0], qf[k][y][1]);
                            }
                        }
                        if (last) {
                            float s[2];
#pragma unroll
                            for (int x = 0; x < 2; x++)
                                s[x] = block == 0 ? power_of<0>(power[x]) : block == 1 ? power_of<1>(power[x]) : block == 2 ? power_of<2>(power[x]) : power_of<3>(power[x]);
#pragma unroll
                            for (int y = 0; y < NB; y++)
#pragma unroll
                                for (int x = 0; x < 4; x++) sc[i][y][x] = block ? fmaf(s[x >> 1], sum[y][x], sc[i][y][x]) : s[x >> 1] * sum[y][x];
                        }
                    }
                }
                if (kQuantised<kFmt> && rare) {  // a block of NaN makes its key's scores NaN
#pragma unroll
                    for (int y = 0; y < NB; y++)
#pragma unroll
                        for (int x = 0; x < 4; x++)
                            if (has_nan(power[x >> 1])) sc[i][y][x] = __int_as_float(0x7FC00000);
                }
            }
        }
        bool more = false;  // a row's maximum grows
        float top[NB][2];
#pragma unroll
        for (int y = 0; y < NB; y++)
#pragma unroll
            for (int x = 0; x < 2; x++) {
                float now = -INFINITY;
#pragma unroll
                for (int i = 0; i < PS; i++)
#pragma unroll
                    for (int z = 0; z < 4; z += 2) {
                        float& v = sc[i][y][x + z];
                        if (!kWhole && !mask.sees(pos[y][x], s0 + 16 * i + 4 * z + (int32_t)(lane / 4))) v = -INFINITY;
                        now = fmaxf(now, v);
                    }
                top[y][x] = fmaxf(now * scale[y][x] - kLift<kHalf>, m[y][x]);
                more |= top[y][x] != m[y][x];
            }
        if (__any_sync(0xFFFFFFFFu, more)) {  // more and more rarely
#pragma unroll
            for (int y = 0; y < NB; y++)
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    float now = top[y][x];
#pragma unroll
                    for (int i = 4; i < 32; i *= 2) now = fmaxf(now, __shfl_xor_sync(0xFFFFFFFFu, now, i));
                    const float f = exp2_approx(m[y][x] - (now == -INFINITY ? 0.0f : now));
                    l[y][x] *= f;
#pragma unroll
                    for (int k = 0; k < KS; k++) {
                        o[k][y][x] *= f;
                        o[k][y][2 + x] *= f;
                    }
                    m[y][x] = now;
                }
        }
        uint32_t pr[PS][NB][2];  // P^T's fragments
#pragma unroll
        for (int y = 0; y < NB; y++) {
            const float use[2] = {m[y][0] == -INFINITY ? 0.0f : m[y][0], m[y][1] == -INFINITY ? 0.0f : m[y][1]};
#pragma unroll
            for (int i = 0; i < PS; i++) {
                float e[4];
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    e[x] = exp2_approx(fmaf(sc[i][y][x], scale[y][x & 1], -use[x & 1]));
                    l[y][x & 1] += e[x];
                }
                // p in 16 bits for the product: a relative error of up to 2^-8 (BF16) or
                // 2^-11 (FP16, down to 2^-29 of the row's largest) of each term,
                // independent from term to term.
                pr[i][y][0] = transpose8(pack2<kHalf>(e[0], e[1]));
                pr[i][y][1] = transpose8(pack2<kHalf>(e[2], e[3]));
            }
        }
        const auto values = [&](auto is_rare) {
#pragma unroll
            for (int i = 0; i < PS; i++) {
                // Values of slots 2 (lane & 3) and the next, and of those + 8, as rows of V^T.
                const auto product = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                    uint32_t f[4] = {a0, a1, a2, a3};
                    if constexpr (!kWhole) {  // 0 x infinity is not 0: keep such values out of the product
#pragma unroll
                        for (int x = 0; x < 4; x++) {
                            const uint32_t v = finite_or_zero<kHalf>(f[x]);
                            odd |= v != f[x];
                            f[x] = v;
                        }
                    }
#pragma unroll
                    for (int y = 0; y < NB; y++) mma16816<kHalf>(o[k][y], f, pr[i][y][0], pr[i][y][1]);
                };
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) {
                    uint32_t r[4];  // chunks c and c + 1 (x >> 1) of slots 0-7 and 8-15 (x & 1) of the block, transposed
                    ldmatrix4_trans(r, vs + tile_at<S::kRow, S::kSlots>(part + 16 * i + (lane & 15), c + (lane >> 4)));
                    if constexpr (kFmt == kBf16) {
                        product(c / 2, r[0], r[2], r[1], r[3]);
                    } else {
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            uint32_t w[2][4];
#pragma unroll
                            for (int x = 0; x < 2; x++) {
                                const uint32_t v = r[2 * u + x];
                                [[maybe_unused]] uint32_t f = 0;
                                if constexpr (kQuantised<kFmt>) {
                                    const uint32_t block = kFmt == kInt8 ? (c + u) * 16 / (D / 4) : D == 128 ? c + u : 2 * (c + u) + (lane >> 4);
                                    f = *reinterpret_cast<const uint32_t*>(powers + 2 * (block * S::kPart + 16 * i + 8 * x + 2 * (lane & 3)));
                                }
                                if constexpr (kFmt == kE5m2) {
                                    w[x][0] = e5m2_02(v), w[x][1] = e5m2_13(v);
                                } else if constexpr (kFmt == kInt8) {
                                    const uint32_t z = int8_bias(v);
                                    if constexpr (decltype(is_rare)::value) {
                                        w[x][0] = mul_half2(int8_pair<kInt8_02>(z), f), w[x][1] = mul_half2(int8_pair<kInt8_13>(z), f);
                                    } else {
                                        w[x][0] = int8_scaled<kInt8_02>(z, f), w[x][1] = int8_scaled<kInt8_13>(z, f);
                                    }
                                } else {
                                    // Values 0 and 1, then 2 and 3 of the one slot and of the other, to each value
                                    // of both slots: 0 and 2, then 1 and 3.
                                    uint32_t z[4];
                                    e2m1_pairs(z, v);
                                    w[x][0] = prmt(z[0], z[2], 0x5410), w[x][1] = prmt(z[1], z[3], 0x5410);
                                    w[x][2] = prmt(z[0], z[2], 0x7632), w[x][3] = prmt(z[1], z[3], 0x7632);
#pragma unroll
                                    for (int n = 0; n < 4; n++) w[x][n] = mul_half2(w[x][n], f);
                                }
                            }
                            if constexpr (kFmt == kE2m1) {
                                product(2 * (c + u), w[0][0], w[0][2], w[1][0], w[1][2]);
                                product(2 * (c + u) + 1, w[0][1], w[0][3], w[1][1], w[1][3]);
                            } else {
                                product(c + u, w[0][0], w[0][1], w[1][0], w[1][1]);
                            }
                        }
                    }
                }
            }
        };
        if (kFmt == kInt8 && !rare) values(std::false_type());
        else values(std::true_type());
    };
    bool ready = true;
    uint32_t stage = 0, turn = 0;
    // The tile that takes the place of the one before the n-th; false where a wait gave up.
    const auto refill = [&](uint32_t n) {
        const uint32_t next = n + S::kStages - 1;
        if (next != mine) return true;
        if (next < count) {
            if (n) ready = mbar_wait_bounded(&sh.empty[next % S::kStages], (next / S::kStages - 1) & 1, wait);
            if (!ready) return false;
            load(next, pages);
        }
        mine += kWarpsRows;
        pages = look_up(mine);
        return true;
    };
    for (uint32_t n = 0; n < count; n++) {
        // With two stages the next tile is asked for before this one's work, to be on its way
        // meanwhile.  With more there are others on their way, and after it no warp waits
        // for the slowest (16k caches: BF16 162 us after, 153 before; INT8 97 and 102).
        if (S::kStages == 2 && !refill(n)) break;
        ready = mbar_wait_bounded(&sh.full[stage], turn, wait);
        if (!ready) break;
        const uint32_t ks = smem_addr(smem + stage * (2 * S::kTile)), vs = ks + S::kTile;
        // This warp's part of the tile: from its row `part` on.
        const uint32_t part = warp * S::kPart;
        const int32_t s0 = (int32_t)(tiles.tile(j0 + n) * S::kSlots + part);
        const uint32_t* e = reinterpret_cast<const uint32_t*>(smem + S::kAtExps + stage * (2 * S::kExps)) + part;
        // Nothing to do for slots behind the last query, or between sinks and windows.
        const bool seen = s0 <= p1 && ((int64_t)s0 + S::kPart > (int64_t)p0 - (int64_t)mask.window + 1 || s0 < mask.sinks);
        if (p0 >= 0 && mask.all(p0, p1, s0, s0 + S::kPart - 1)) walk(std::true_type(), ks, vs, e, part, s0);
        else if (seen) walk(std::false_type(), ks, vs, e, part, s0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[stage]);
        if (++stage == S::kStages) stage = 0, turn ^= 1;
        if (S::kStages > 2 && !refill(n)) break;
    }
    // The head's value of o[k][..][x].
    auto column = [&](int k, int x) {
        const int i = (int)(lane / 4), u = x >> 1;
        return kFmt == kBf16 ? 16 * k + 8 * u + i : kFmt == kE2m1 ? 32 * (k / 2) + 4 * i + 2 * (k & 1) + u : 16 * k + 2 * i + u;
    };
    if (__any_sync(0xFFFFFFFFu, odd)) {
        // The infinite and NaN values of partly visible tiles go to the rows that
        // see them: whatever their (positive) weight, the sum takes their value.
        for (uint32_t n = 0; n < count; n++) {
            const int32_t s0 = (int32_t)(tiles.tile(j0 + n) * S::kSlots + warp * S::kPart);
            if (p0 >= 0 && mask.all(p0, p1, s0, s0 + S::kPart - 1)) continue;
            for (int32_t s = s0; s < min(s0 + S::kPart, mask.n); s++) {
                if (s > p1) break;
                const bool sinks = s < mask.sinks;
                if (!sinks && (int64_t)s <= (int64_t)p0 - (int64_t)mask.window) continue;
                const uint32_t page = (uint32_t)table[s >> p.page_shift];
                if (page >= pool.pages) continue;
                const int64_t at = (uint32_t)s & in_page;
                constexpr int kElem = kFmt == kBf16 ? 2 : 1;
                const uint8_t* row = static_cast<const uint8_t*>(pool.v.data) +
                                     (h * pool.v.stride_h + page * pool.v.stride_p + at * pool.v.stride_t) * kElem;
                const uint8_t* bytes = pool.v.exponents + h * pool.v.exp_stride_h + page * pool.v.exp_stride_p + at * pool.v.exp_stride_t;
#pragma unroll
                for (int k = 0; k < KS; k++)
#pragma unroll
                    for (int x = 0; x < 4; x += 2) {
                        const float v = page_value<D, kFmt>(row, bytes, column(k, x));
                        if (isfinite(v)) continue;
#pragma unroll
                        for (int y = 0; y < NB; y++) {
                            if (mask.sees(pos[y][0], s)) o[k][y][x] += v;
                            if (mask.sees(pos[y][1], s)) o[k][y][x + 1] += v;
                        }
                    }
            }
        }
    }
    if (!ready && lane == 0) atomicOr(p.status, kStatusTimeout);
    lost = __any_sync(0xFFFFFFFFu, lost) || !ready;

    // Join the warps: everything into shared memory (over the ring).
#pragma unroll
    for (int y = 0; y < NB; y++)
#pragma unroll
        for (int x = 0; x < 2; x++) {
#pragma unroll
            for (int i = 4; i < 32; i *= 2) l[y][x] += __shfl_xor_sync(0xFFFFFFFFu, l[y][x], i);
            if (lane < 4) {
                sh.join.m[warp][8 * y + 2 * lane + x] = m[y][x];
                sh.join.l[warp][8 * y + 2 * lane + x] = lost ? __int_as_float(0x7FC00000) : l[y][x];
            }
        }
    __syncthreads();  // every warp is done with the ring
    if (*const_cast<volatile uint32_t*>(&sh.wait.given_up)) {  // nothing may land after this
        for (uint32_t i = 0; i < S::kStages; i++)
            if (sh.turns.used(i)) mbar_wait_bounded<true>(&sh.full[i], sh.turns.parity(i), wait);
        __syncthreads();
    }
    float* os = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int k = 0; k < KS; k++)
#pragma unroll
        for (int y = 0; y < NB; y++)
#pragma unroll
            for (int x = 0; x < 4; x++) os[(warp * kTileRows + 8 * y + 2 * (lane & 3) + (x & 1)) * D + column(k, x)] = o[k][y][x];
    __syncthreads();

    auto store = [&](uint32_t r, uint32_t c, float4 v, float mm, float ll) {
        const uint32_t row = r0 + r, t = row / p.group, hq = h * p.group + (row - t * p.group);
        const bool none = ll == 0.0f;  // nothing seen, or scores of -infinity alone
        const float inv = 1.0f / ll;
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out.data) + (int64_t)(seq.row + t) * a.out.stride_t + hq * a.out.stride_h;
        *reinterpret_cast<uint2*>(out + c) =
            none ? make_uint2(0, 0) : make_uint2(pack2<false>(v.x * inv, v.y * inv), pack2<false>(v.z * inv, v.w * inv));
        if (c == 0 && a.lse) a.lse[(uint64_t)hq * a.tokens + seq.row + t] = none ? -INFINITY : (mm + log2f(ll)) * kLn2;
    };
    const uint32_t cluster = shared ? 1 : p.cluster, unit = (b * pool.kv_heads + h) * p.row_tiles + rt;
    // Counters are ready for the next call when the last one has counted: words, or where
    // there may be many row tiles bytes of them.
    const auto is_last = [&] {
        if (!shared) {
            const bool last = atomicAdd(p.counters + unit, 1u) == splits - 1;
            if (last) p.counters[unit] = 0;
            return last;
        }
        const uint32_t by = 8 * (unit & 3);
        const bool last = (atomicAdd(p.counters + unit / 4, 1u << by) >> by & 255u) == splits - 1;
        if (last) atomicSub(p.counters + unit / 4, splits << by);
        return last;
    };
    float* all = p.partials + (uint64_t)(first_cta / cluster) * kPartFloats<D, kTileRows>;
    join_rows<D, kTileRows>(os, sh.join, split, splits, cluster, r1 - r0, all, is_last, store);
}

template <int D, int kFmt, int NB>
cudaError_t launch(const PagedRowsParams& p, uint32_t ctas, bool after_tiles, cudaStream_t s) {
    using S = PagedShape<D, kFmt, 8 * NB>;
    static_assert(S::kAtExps >= kWarpsRows * 8 * NB * D * 4, "partial results take the place of the ring");
    constexpr int kSmem = S::kAtQueries + 8 * NB * D * 2 + (int)sizeof(PagedRowsShared<S::kStages, 8 * NB>);
    Wave w;
    const cudaError_t e = launch_wave<paged_rows_kernel<D, kFmt, NB>>(32 * kWarpsRows, kSmem, w);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * kWarpsRows);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = after_tiles ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, paged_rows_kernel<D, kFmt, NB>, p);
}

template <int D, int kFmt>
cudaError_t launch_rows(const PagedRowsParams& p, uint32_t tile_rows, uint32_t ctas, bool after_tiles, cudaStream_t s) {
    return tile_rows == 8 ? launch<D, kFmt, 1>(p, ctas, after_tiles, s) : launch<D, kFmt, 2>(p, ctas, after_tiles, s);
}

template <int D>
cudaError_t launch_format(const PagedRowsParams& p, uint32_t tile_rows, uint32_t ctas, bool after_tiles, cudaStream_t s) {
    switch (p.a.pool.format) {
        case kBf16: return launch_rows<D, kBf16>(p, tile_rows, ctas, after_tiles, s);
        case kE5m2: return launch_rows<D, kE5m2>(p, tile_rows, ctas, after_tiles, s);
        case kInt8: return launch_rows<D, kInt8>(p, tile_rows, ctas, after_tiles, s);
        default: return launch_rows<D, kE2m1>(p, tile_rows, ctas, after_tiles, s);
    }
}

}  // namespace

// Rows of a tile: 8 where a sequence has no more, and in a batch with longer chunks,
// whose other sequences are taken to bring a token each, where those have no more
// (24 of them and a chunk of 1024 over 8k caches in 8 bits: the tokens take 62 us in
// tiles of 8 rows and 96 in tiles of 16).
inline uint32_t tile_rows(const splitzip_paged_attention_args& a, uint32_t rows_upto) {
    const uint64_t group = a.q_heads / a.pool.kv_heads, most = a.max_q_tokens * group;
    return std::min<uint64_t>(most, rows_upto) <= 8 || (most > rows_upto && group <= 8) ? 8 : 16;
}

bool paged_rows_plan(const splitzip_paged_attention_args& a, uint32_t rows_upto, PagedPlan& p) {
    const uint32_t group = a.q_heads / a.pool.kv_heads, d = a.pool.head_dim, tile = tile_rows(a, rows_upto);
    const uint64_t most_rows = (uint64_t)a.max_q_tokens * group;
    p.row_tiles = (uint32_t)((std::min<uint64_t>(most_rows, rows_upto) + tile - 1) / tile);
    const uint64_t units = (uint64_t)a.batch * a.pool.kv_heads * p.row_tiles;
    const uint32_t slots = warp_slots(a.pool.format, d, tile), ctas = ctas_per_sm(a.pool.format, d, tile);
    uint64_t most = a.kv_tokens;
    if (a.window) most = std::min(most, (uint64_t)a.window + a.sinks + (tile + group - 1) / group + 2 * slots);
    // In a batch with longer chunks one of the sequences is such a one, and of the others'
    // row tiles the first has the rows.
    const uint64_t likely = most_rows > rows_upto ? (uint64_t)std::max(1u, a.batch - 1) * a.pool.kv_heads : units;
    p.splits = attention_rows_splits(likely, most, slots, 16, d, ctas);
    // Splits in several clusters are counted by row tile, in a header of limited size.
    if (p.splits > 8 && units > kSms) p.splits = 8;
    p.ctas = units * p.splits;
    p.bytes = attention_rows_bytes(units, p.splits, tile, d);
    // Sequences of a batch differ in length, and a number of splits that is the same for all
    // does not fill the GPU evenly, or (eight to a cluster) not at all.  Sharing the work out
    // by length costs 5 us (the tables, and joining through memory), so it is for splits of
    // 3000 slots and more, and quantised caches, whose widening keeps the GPU busy for long
    // enough.  8 heads of 128, 32 query heads, splits alike and shared out, us:
    //   sequences of    half to full length      one length
    //   INT8   3 x 30k        57    42             59    46
    //         16 x 16k        86    76             94   100
    //         24 x 16k       111   109            128   135
    //         40 x  4k        70    59             76    78
    //   E2M1  16 x 16k        67    58             72    76
    // and not taken: INT8 4 x 16k 35 33, 36 38; 16 x 8k 46 45, 52 57; 75 x 4k (600 units for
    // 608 CTAs) 90 92, 101 104; E5M2 16 x 16k 67 70, 81 86; BF16 124 126.
    const uint64_t at_once = (uint64_t)kSms * ctas;
    static_assert(3 * kSms <= kAttentionStatus, "a byte of the workspace's header counts the splits of a row tile");
    if ((a.pool.format == kInt8 || a.pool.format == kE2m1) && a.batch > 1 && a.batch <= kMostShared &&
        units <= at_once * 3 / 4 && most / p.splits >= 3000) {
        p.splits = 0;
        p.ctas = at_once;
        p.bytes = kAttentionHeader + at_once * tile * (d + 4) * 4;
    }
    return p.ctas <= 0x7FFFFFFFull;
}

cudaError_t launch_paged_rows(const splitzip_paged_attention_args& a, uint32_t rows_upto, const PagedPlan& plan, void* workspace,
                              bool after_tiles, const WaitTest& test, cudaStream_t s) {
    PagedRowsParams p;
    p.a = a;
    p.group = a.q_heads / a.pool.kv_heads;
    p.page_shift = 0;
    while ((1u << p.page_shift) < a.pool.page_tokens) p.page_shift++;
    p.rows_upto = rows_upto;
    p.row_tiles = plan.row_tiles;
    p.splits = plan.splits;
    p.cluster = plan.splits ? std::min(plan.splits, 8u) : 1;
    const splitzip_pool& pool = a.pool;
    const uint32_t slots = kWarpsRows * warp_slots(pool.format, pool.head_dim, tile_rows(a, rows_upto));  // of a tile
    p.box = std::min(pool.page_tokens, slots);
    p.boxes = slots / p.box;
    p.bulk_exps = bulk_exponents(pool);
    if (!page_map(p.kmap, pool, pool.k, p.box) || !page_map(p.vmap, pool, pool.v, p.box)) return cudaErrorInvalidValue;
    p.status = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + kAttentionStatus);
    p.wait_limit = test.limit ? test.limit : wait_limit(0);  // a wait lasts a copy's time
    p.test_cta = test.cta;
    p.test_tile = test.tile;
    p.counters = reinterpret_cast<uint32_t*>(workspace);
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kAttentionHeader);
    const uint32_t ctas = (uint32_t)plan.ctas;
    return a.pool.head_dim == 64 ? launch_format<64>(p, tile_rows(a, rows_upto), ctas, after_tiles, s)
                                    : launch_format<128>(p, tile_rows(a, rows_upto), ctas, after_tiles, s);
}

}  // namespace splitzip
