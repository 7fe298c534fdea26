// paged_rows.cu -- attention of few query rows over pages (sm_103a).
//
// The query rows of one sequence and key/value head (its new tokens times the group's
// query heads) in tiles of 8 or 16, a tile's slots in splits, one CTA each, each of
// its four warps with its own slot tiles, running maximum, sum and output as in
// attention_rows.cu, joined at the end in a fixed order.  Every key and value is
// read once: HBM bounds it, next to the widening of quantised codes.
//
// The products are transposed: S^T = K Q^T and O^T += V^T P^T, with slots, then a
// head's values as the 16 rows of an m16n8k16 product and the query rows as its 8
// columns.  One token of a group of up to eight heads fills those: half the products,
// exponentials and registers that 16 rows take.  P^T comes out of S^T by a
// transposition of 8 x 8 blocks between registers (movmatrix).
//
// Pages hold at least 16 slots, and a warp's tiles 32 or 64 (16 of BF16 at head_dim
// 128), so a tile is a few runs of 16 slots of one page each.  The lanes hold the
// page numbers of a tile's runs from one tile ahead, so that no copy waits for the
// table.  A run that no query sees is not looked up (its page may have been given
// away) and is copied from the pool's first page, masked.
//
// Quantised codes become FP16 in registers on their way from shared memory to the
// products: codes by a byte permute and a subtraction (INT8) or a conversion
// (E2M1), then a multiplication by the block's power of two, all exact.  The powers
// are made FP16 once per tile and slot by one lane, and laid out as the fragments
// need them: a key's four side by side, the values' of neighbouring slots side by
// side.
#include <algorithm>
#include <cstdint>

#include "attention_rows.cuh"
#include "pages.cuh"

namespace splitzip {
namespace {

struct PagedRowsParams {
    splitzip_paged_attention_args a;
    uint32_t group, page_shift, row_tiles, splits, cluster;
    uint32_t rows_upto;  // only sequences with no more query rows than this
    uint32_t* counters;
    float* partials;
};

template <int D, int kFmt>
struct PagedShape {
    static constexpr int kRow = kRowBytes<D, kFmt>;
    static constexpr int kSlots = kFmt == kBf16 ? 2048 / D : 4096 / D;  // slots per warp tile
    static constexpr int kTile = kSlots * kRow;                         // bytes of its keys, and of its values
    static constexpr int kStages = kFmt == kE2m1 ? 4 : 2;
    static constexpr int kExps = kQuantised<kFmt> ? 4 * kSlots : 0;     // bytes of its keys' exponents, and of its values'
    static constexpr int kStage = 2 * (kTile + kExps);
    static constexpr int kScales = kQuantised<kFmt> ? 16 * kSlots : 0;  // of the powers as FP16, keys' and values'
    static constexpr int kRing = kWarpsRows * (kStages * kStage + kScales);
    static_assert(kRing >= kWarpsRows * 16 * D * 4, "partial results take the place of the ring");
};

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

// The transpose of an 8 x 8 matrix of 16-bit values, a row to four lanes.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// NB: blocks of 8 query rows.
template <int D, int kFmt, int NB>
__global__ void __launch_bounds__(32 * kWarpsRows, kCtasPerSm) paged_rows_kernel(const __grid_constant__ PagedRowsParams p) {
    using S = PagedShape<D, kFmt>;
    constexpr bool kHalf = kWide<kFmt>;  // operands FP16, else BF16
    constexpr int kTileRows = 8 * NB;
    constexpr int KS = D / 16;           // steps of the scores, and 16-value blocks of the output
    constexpr int PS = S::kSlots / 16;   // 16-slot blocks of the scores, steps of the output, runs of one page each
    constexpr int kChunks = S::kRow / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float s_scale[kTileRows];
    __shared__ RowsShared<kTileRows> sh;
    const splitzip_paged_attention_args& a = p.a;
    const splitzip_pool& pool = a.pool;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t unit = blockIdx.x / p.splits, split = blockIdx.x - unit * p.splits;
    const uint32_t bh = unit / p.row_tiles, rt = unit - bh * p.row_tiles;
    const uint32_t b = bh / pool.kv_heads, h = bh - b * pool.kv_heads;
    const Sequence seq(a, b);
    const uint32_t rows = (uint32_t)seq.count * p.group;
    const uint32_t r0 = rt * kTileRows, r1 = min(r0 + kTileRows, rows);
    if (r0 >= rows || rows > p.rows_upto) return;  // with all of its cluster
    const Mask mask(seq.n, seq.count, a.window, a.sinks);
    const int32_t p0 = mask.first + (int32_t)(r0 / p.group), p1 = mask.first + (int32_t)((r1 - 1) / p.group);
    const SlotTiles tiles(mask, p0, p1, S::kSlots);
    const uint32_t j0 = (uint32_t)((uint64_t)tiles.count * split / p.splits);
    const uint32_t j1 = (uint32_t)((uint64_t)tiles.count * (split + 1) / p.splits);

    uint8_t* ring = smem + warp * (S::kStages * S::kStage + S::kScales);
    uint8_t* scales = ring + S::kStages * S::kStage;  // keys' [slot][block], then values' [block][slot]
    uint8_t* qs = smem + S::kRing;
    constexpr int kElem = kFmt == kBf16 ? 2 : 1;
    const uint8_t* kbase = static_cast<const uint8_t*>(pool.k.data) + h * pool.k.stride_h * kElem;
    const uint8_t* vbase = static_cast<const uint8_t*>(pool.v.data) + h * pool.v.stride_h * kElem;
    const uint8_t* kexps = pool.k.exponents + h * pool.k.exp_stride_h;
    const uint8_t* vexps = pool.v.exponents + h * pool.v.exp_stride_h;
    const int32_t* table = a.table + (uint64_t)b * a.table_width;
    const uint32_t in_page = pool.page_tokens - 1;

    // Lane i < PS: the page of the tile's run i.  Slots past the last one in use are
    // taken as copies of it.
    bool lost = false;  // a page that a query sees is outside the pool
    auto look_up = [&](uint32_t j) -> uint32_t {
        if (lane >= PS || j >= j1) return 0;
        const int32_t s = (int32_t)(tiles.tile(j) * S::kSlots + 16 * lane);
        // The run's last slot is behind the start of the first query's window, or a sink.
        if (s > p1 || !((int64_t)s + 15 > (int64_t)p0 - (int64_t)mask.window || s < mask.sinks)) return 0;
        const uint32_t page = (uint32_t)table[s >> p.page_shift];
        if (page < pool.pages) return page;
        lost = true;
        return 0;
    };
    // A lane copies one 16-byte chunk of every kStep-th row of a tile.
    constexpr int kStep = 32 / kChunks;
    const uint32_t lr = lane / kChunks, lc = lane % kChunks;
    const int64_t kst = pool.k.stride_t * kElem, vst = pool.v.stride_t * kElem;
    auto load = [&](uint32_t j, uint32_t stage, uint32_t pages) {
        if (j < j1) {
            const int32_t s0 = (int32_t)(tiles.tile(j) * S::kSlots);
            uint8_t* dk = ring + stage * S::kStage;
            const bool full = s0 + S::kSlots <= mask.n;
#pragma unroll
            for (int i = 0; i < PS; i++) {
                const int64_t page = __shfl_sync(0xFFFFFFFFu, pages, i);
                const uint8_t* k = kbase + page * pool.k.stride_p * kElem + 16 * lc;
                const uint8_t* v = vbase + page * pool.v.stride_p * kElem + 16 * lc;
                const int32_t first = s0 + 16 * i;
                if (full) {
                    const uint32_t at = ((uint32_t)first & in_page) + lr;
                    k += at * kst;
                    v += at * vst;
#pragma unroll
                    for (int x = 0; x < 16 / kStep; x++) {
                        cp_async16(dk + chunk_at<S::kRow>(16 * i + x * kStep + lr, lc), k);
                        cp_async16(dk + S::kTile + chunk_at<S::kRow>(16 * i + x * kStep + lr, lc), v);
                        k += kStep * kst;
                        v += kStep * vst;
                    }
                } else {
#pragma unroll 1
                    for (int x = 0; x < 16 / kStep; x++) {
                        const uint32_t at = (uint32_t)min(first + x * kStep + (int32_t)lr, mask.n - 1) & in_page;
                        cp_async16(dk + chunk_at<S::kRow>(16 * i + x * kStep + lr, lc), k + at * kst);
                        cp_async16(dk + S::kTile + chunk_at<S::kRow>(16 * i + x * kStep + lr, lc), v + at * vst);
                    }
                }
            }
            if constexpr (kQuantised<kFmt>) {
                uint8_t* de = dk + 2 * S::kTile;
#pragma unroll
                for (int i = 0; i < S::kSlots / 32; i++) {
                    const int32_t s = s0 + 32 * i + (int32_t)lane;
                    const int64_t page = __shfl_sync(0xFFFFFFFFu, pages, 2 * i + (lane >> 4));
                    const uint32_t at = (uint32_t)(full ? s : min(s, mask.n - 1)) & in_page;
                    cp_async4(de + 4 * (32 * i + lane), kexps + page * pool.k.exp_stride_p + at * pool.k.exp_stride_t);
                    cp_async4(de + S::kExps + 4 * (32 * i + lane), vexps + page * pool.v.exp_stride_p + at * pool.v.exp_stride_t);
                }
            }
        }
        cp_async_commit();
    };
    uint32_t ahead = j0 + warp;  // the next tile to be copied, and its pages
    uint32_t pages = look_up(ahead);
    auto advance = [&](uint32_t stage) {
        const uint32_t now = pages, j = ahead;
        ahead += kWarpsRows;
        pages = look_up(ahead);
        load(j, stage, now);
    };
#pragma unroll
    for (int i = 0; i < S::kStages - 1; i++) advance(i);

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
        if (lane == 0) s_scale[r] = a.scale * kLog2e / power;
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
            scale[y][x] = s_scale[r];
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
    uint32_t stage = 0;
    for (uint32_t j = j0 + warp; j < j1; j += kWarpsRows) {
        cp_async_wait<S::kStages - 2>();
        __syncwarp();
        advance(stage == 0 ? S::kStages - 1 : stage - 1);
        const uint8_t* tile = ring + stage * S::kStage;
        const uint32_t ks = smem_addr(tile), vs = ks + S::kTile;
        stage = stage == S::kStages - 1 ? 0 : stage + 1;
        const int32_t s0 = (int32_t)(tiles.tile(j) * S::kSlots);
        const bool whole = p0 >= 0 && mask.all(p0, p1, s0, s0 + S::kSlots - 1);

        if constexpr (kQuantised<kFmt>) {
            const uint32_t* e = reinterpret_cast<const uint32_t*>(tile + 2 * S::kTile);
#pragma unroll
            for (int i = 0; i < S::kSlots / 32; i++) {
                const uint32_t s = 32 * i + lane;
                uint32_t w[2][2];
#pragma unroll
                for (int x = 0; x < 2; x++) {
                    const uint32_t v = e[x * S::kSlots + s];
                    w[x][0] = pack2<true>(block_scale(v & 255u), block_scale(v >> 8 & 255u));
                    w[x][1] = pack2<true>(block_scale(v >> 16 & 255u), block_scale(v >> 24));
                }
                *reinterpret_cast<uint2*>(scales + 8 * s) = make_uint2(w[0][0], w[0][1]);
                uint16_t* to = reinterpret_cast<uint16_t*>(scales + 8 * S::kSlots) + s;
                to[0] = (uint16_t)w[1][0], to[S::kSlots] = (uint16_t)(w[1][0] >> 16);
                to[2 * S::kSlots] = (uint16_t)w[1][1], to[3 * S::kSlots] = (uint16_t)(w[1][1] >> 16);
            }
            __syncwarp();
        }
        // Scores of slots 16 i + lane / 4 and that + 8 (x >> 1) for this thread's rows (x & 1).
        float sc[PS][NB][4];
#pragma unroll
        for (int i = 0; i < PS; i++) {
#pragma unroll
            for (int y = 0; y < NB; y++)
#pragma unroll
                for (int x = 0; x < 4; x++) sc[i][y][x] = 0.0f;
            const auto product = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                const uint32_t f[4] = {a0, a1, a2, a3};
#pragma unroll
                for (int y = 0; y < NB; y++) mma16816<kHalf>(sc[i][y], f, qf[k][y][0], qf[k][y][1]);
            };
            if constexpr (kFmt == kBf16) {
#pragma unroll
                for (int k = 0; k < KS; k++) {
                    uint32_t r[4];
                    ldmatrix4(r, ks + chunk_at<S::kRow>(16 * i + (lane & 15), 2 * k + (lane >> 4)));
                    product(k, r[0], r[1], r[2], r[3]);
                }
            } else {
                uint2 power[2];  // of the two slots
                if constexpr (kQuantised<kFmt>)
#pragma unroll
                    for (int x = 0; x < 2; x++) power[x] = *reinterpret_cast<const uint2*>(scales + 8 * (16 * i + 8 * x + lane / 4));
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) {
                    uint32_t r[4];  // chunks c and c + 1 (x >> 1) of slots 0-7 and 8-15 (x & 1) of the block
                    ldmatrix4(r, ks + chunk_at<S::kRow>(16 * i + (lane & 15), c + (lane >> 4)));
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        uint32_t w[2][4];
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            const uint32_t v = r[2 * u + x];
                            if constexpr (kFmt == kE5m2) {
                                w[x][0] = e5m2_01(v), w[x][1] = e5m2_23(v);
                            } else if constexpr (kFmt == kInt8) {
                                const uint32_t f = twice(power[x], (c + u) * 16 / (D / 4)), z = int8_bias(v);
                                w[x][0] = mul_half2(int8_pair<kInt8_01>(z), f), w[x][1] = mul_half2(int8_pair<kInt8_23>(z), f);
                            } else {
                                // A lane's eight values are one block's: its half of the 32, or all of them.
                                const uint32_t f = D == 128 ? twice(power[x], c + u)
                                                            : prmt(u ? power[x].y : power[x].x, 0u, lane & 2 ? 0x3232u : 0x1010u);
                                e2m1_pairs(w[x], v);
#pragma unroll
                                for (int n = 0; n < 4; n++) w[x][n] = mul_half2(w[x][n], f);
                            }
                        }
                        if constexpr (kFmt == kE2m1) {
                            product(2 * (c + u), w[0][0], w[1][0], w[0][1], w[1][1]);
                            product(2 * (c + u) + 1, w[0][2], w[1][2], w[0][3], w[1][3]);
                        } else {
                            product(c + u, w[0][0], w[1][0], w[0][1], w[1][1]);
                        }
                    }
                }
            }
        }
        bool more = false;  // a row's maximum grows
        float top[NB][2];
#pragma unroll
        for (int y = 0; y < NB; y++)
#pragma unroll
            for (int x = 0; x < 2; x++) top[y][x] = m[y][x] + kLift<kHalf>;
#pragma unroll
        for (int y = 0; y < NB; y++) {
#pragma unroll
            for (int i = 0; i < PS; i++)
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    float v = sc[i][y][x] * scale[y][x & 1];
                    if (!whole && !mask.sees(pos[y][x & 1], s0 + 16 * i + 8 * (x >> 1) + (int32_t)(lane / 4))) v = -INFINITY;
                    sc[i][y][x] = v;
                    top[y][x & 1] = fmaxf(top[y][x & 1], v);
                }
#pragma unroll
            for (int x = 0; x < 2; x++) {
                top[y][x] -= kLift<kHalf>;
                more |= top[y][x] != m[y][x];
            }
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
                    e[x] = exp2_approx(sc[i][y][x] - use[x & 1]);
                    l[y][x & 1] += e[x];
                }
                // p in 16 bits for the product: a relative error of up to 2^-8 (BF16) or
                // 2^-11 (FP16, down to 2^-29 of the row's largest) of each term,
                // independent from term to term.
                pr[i][y][0] = transpose8(pack2<kHalf>(e[0], e[1]));
                pr[i][y][1] = transpose8(pack2<kHalf>(e[2], e[3]));
            }
        }
#pragma unroll
        for (int i = 0; i < PS; i++) {
            // Values of slots 2 (lane & 3) and the next, and of those + 8, as rows of V^T.
            const auto product = [&](int k, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                uint32_t f[4] = {a0, a1, a2, a3};
                if (!whole) {  // 0 x infinity is not 0: keep such values out of the product
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
                ldmatrix4_trans(r, vs + chunk_at<S::kRow>(16 * i + (lane & 15), c + (lane >> 4)));
                if constexpr (kFmt == kBf16) {
                    product(c / 2, r[0], r[2], r[1], r[3]);
                } else {
#pragma unroll
                    for (int u = 0; u < 2; u++) {
                        uint32_t w[2][4];
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            const uint32_t v = r[2 * u + x];
                            uint32_t f = 0;
                            if constexpr (kQuantised<kFmt>) {
                                const uint32_t block = kFmt == kInt8 ? (c + u) * 16 / (D / 4) : D == 128 ? c + u : 2 * (c + u) + (lane >> 4);
                                f = *reinterpret_cast<const uint32_t*>(scales + 8 * S::kSlots + 2 * (block * S::kSlots + 16 * i + 8 * x + 2 * (lane & 3)));
                            }
                            if constexpr (kFmt == kE5m2) {
                                w[x][0] = e5m2_02(v), w[x][1] = e5m2_13(v);
                            } else if constexpr (kFmt == kInt8) {
                                const uint32_t z = int8_bias(v);
                                w[x][0] = mul_half2(int8_pair<kInt8_02>(z), f), w[x][1] = mul_half2(int8_pair<kInt8_13>(z), f);
                            } else {
                                // Bytes of the same value of both slots: values 0 and 2, then 1 and 3.
                                uint32_t z = (v & 0x0F0Fu) | (v >> 12 & 0xF0F0u);
                                z |= ((v >> 4 & 0x0F0Fu) | (v >> 16 & 0xF0F0u)) << 16;
                                e2m1_pairs(w[x], z);
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
        if constexpr (kQuantised<kFmt>) __syncwarp();  // the powers have been read
    }
    cp_async_wait<0>();
    // The head's value of o[k][..][x].
    auto column = [&](int k, int x) {
        const int i = (int)(lane / 4), u = x >> 1;
        return kFmt == kBf16 ? 16 * k + 8 * u + i : kFmt == kE2m1 ? 32 * (k / 2) + 4 * i + 2 * (k & 1) + u : 16 * k + 2 * i + u;
    };
    if (__any_sync(0xFFFFFFFFu, odd)) {
        // The infinite and NaN values of partly visible tiles go to the rows that
        // see them: whatever their (positive) weight, the sum takes their value.
        for (uint32_t j = j0 + warp; j < j1; j += kWarpsRows) {
            const int32_t s0 = (int32_t)(tiles.tile(j) * S::kSlots);
            if (p0 >= 0 && mask.all(p0, p1, s0, s0 + S::kSlots - 1)) continue;
            for (int32_t s = s0; s < min(s0 + S::kSlots, mask.n); s++) {
                if (s > p1) break;
                const bool sinks = s < mask.sinks;
                if (!sinks && (int64_t)s <= (int64_t)p0 - (int64_t)mask.window) continue;
                const uint32_t page = (uint32_t)table[s >> p.page_shift];
                if (page >= pool.pages) continue;
                const int64_t at = (uint32_t)s & in_page;
                const uint8_t* row = vbase + page * pool.v.stride_p * kElem + at * vst;
                const uint8_t* exps = vexps + page * pool.v.exp_stride_p + at * pool.v.exp_stride_t;
#pragma unroll
                for (int k = 0; k < KS; k++)
#pragma unroll
                    for (int x = 0; x < 4; x += 2) {
                        const float v = page_value<D, kFmt>(row, exps, column(k, x));
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
    lost = __any_sync(0xFFFFFFFFu, lost);

    // Join the warps: everything into shared memory (over the ring).
#pragma unroll
    for (int y = 0; y < NB; y++)
#pragma unroll
        for (int x = 0; x < 2; x++) {
#pragma unroll
            for (int i = 4; i < 32; i *= 2) l[y][x] += __shfl_xor_sync(0xFFFFFFFFu, l[y][x], i);
            if (lane < 4) {
                sh.m[warp][8 * y + 2 * lane + x] = m[y][x];
                sh.l[warp][8 * y + 2 * lane + x] = lost ? __int_as_float(0x7FC00000) : l[y][x];
            }
        }
    __syncthreads();  // every warp is done with its ring
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
    join_rows<D, kTileRows>(os, sh, unit, split, p.splits, p.cluster, r1 - r0, p.counters, p.partials, store);
}

template <int D, int kFmt, int NB>
cudaError_t launch(const PagedRowsParams& p, uint32_t ctas, cudaStream_t s) {
    constexpr int kSmem = PagedShape<D, kFmt>::kRing + 8 * NB * D * 2;
    Wave w;
    const cudaError_t e = launch_wave<paged_rows_kernel<D, kFmt, NB>>(32 * kWarpsRows, kSmem, w);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32 * kWarpsRows);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_rows_kernel<D, kFmt, NB>, p);
}

template <int D, int kFmt>
cudaError_t launch_rows(const PagedRowsParams& p, uint32_t tile_rows, uint32_t ctas, cudaStream_t s) {
    return tile_rows == 8 ? launch<D, kFmt, 1>(p, ctas, s) : launch<D, kFmt, 2>(p, ctas, s);
}

template <int D>
cudaError_t launch_format(const PagedRowsParams& p, uint32_t tile_rows, uint32_t ctas, cudaStream_t s) {
    switch (p.a.pool.format) {
        case kBf16: return launch_rows<D, kBf16>(p, tile_rows, ctas, s);
        case kE5m2: return launch_rows<D, kE5m2>(p, tile_rows, ctas, s);
        case kInt8: return launch_rows<D, kInt8>(p, tile_rows, ctas, s);
        default: return launch_rows<D, kE2m1>(p, tile_rows, ctas, s);
    }
}

}  // namespace

// Rows of a tile: 8 where a sequence has no more.
inline uint32_t tile_rows(const splitzip_paged_attention_args& a, uint32_t rows_upto) {
    return std::min<uint64_t>((uint64_t)a.max_q_tokens * (a.q_heads / a.pool.kv_heads), rows_upto) <= 8 ? 8 : 16;
}

bool paged_rows_plan(const splitzip_paged_attention_args& a, uint32_t rows_upto, PagedPlan& p) {
    const uint32_t group = a.q_heads / a.pool.kv_heads, d = a.pool.head_dim, tile = tile_rows(a, rows_upto);
    p.row_tiles = (uint32_t)((std::min<uint64_t>((uint64_t)a.max_q_tokens * group, rows_upto) + tile - 1) / tile);
    const uint64_t units = (uint64_t)a.batch * a.pool.kv_heads * p.row_tiles;
    const uint32_t slots = (a.pool.format == kBf16 ? 2048 : 4096) / d;
    uint64_t most = a.kv_tokens;
    if (a.window) most = std::min(most, (uint64_t)a.window + a.sinks + (tile + group - 1) / group + 2 * slots);
    p.splits = attention_rows_splits(units, most, slots, 16, d);
    p.bytes = attention_rows_bytes(units, p.splits, tile, d);
    return units * p.splits <= 0x7FFFFFFFull;
}

cudaError_t launch_paged_rows(const splitzip_paged_attention_args& a, uint32_t rows_upto, const PagedPlan& plan, void* workspace,
                              cudaStream_t s) {
    PagedRowsParams p;
    p.a = a;
    p.group = a.q_heads / a.pool.kv_heads;
    p.page_shift = 0;
    while ((1u << p.page_shift) < a.pool.page_tokens) p.page_shift++;
    p.rows_upto = rows_upto;
    p.row_tiles = plan.row_tiles;
    p.splits = plan.splits;
    p.cluster = std::min(plan.splits, 8u);
    p.counters = reinterpret_cast<uint32_t*>(workspace);
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kAttentionHeader);
    const uint32_t ctas = a.batch * a.pool.kv_heads * plan.row_tiles * plan.splits;
    return a.pool.head_dim == 64 ? launch_format<64>(p, tile_rows(a, rows_upto), ctas, s)
                                    : launch_format<128>(p, tile_rows(a, rows_upto), ctas, s);
}

}  // namespace splitzip
