// fp4_attention_rows.cu -- attention over a paged cache held in 4 bits, for
// many query rows to a KV head (sm_100a): prompts in pieces, drafted tokens.
//
// The same results as fp4_attention.cu.  Where that kernel expands every code
// again for each 8 or 16 rows, here 128 rows share an expanded tile: 128
// tokens of K and of V are turned into fp16 in shared memory and multiplied by
// tcgen05.mma, S = Q K^T (both operands K-major) and O += P V (P from tensor
// memory, V with its dimensions as the contiguous axis), sums in tensor memory.
//
// Warps of a block: eight on the query rows, two threads a row and 64 of a
// tile's columns each (query rows to fp16, softmax, output), four that own a
// cached token a thread (pages, codes to fp16), one that issues the products
// and one that walks the block's items.  Nothing is
// double-buffered: K of the next tile is expanded while this one's softmax
// runs, V after this one's second product, and two blocks of an SM fill each
// other's gaps (one with 256 dimensions).  The next scores are formed before
// this tile's weights are used, where tensor memory holds both.
//
// Bound by the latency of a tile's chain (scores, softmax, weights, product),
// about 3700 cycles for a tile in each of the two blocks, and the exponentials
// in it: one warp of a scheduler takes 12 cycles for a score, four of them 4.8
// each, which is why a row has two threads.
//
// Measured, 4 pieces of 200-500 tokens x 48 heads of 64 on 2000-4001 cached
// tokens with a window of 1024 (14.4 GFLOP): 60 us, 240 TFLOP/s; 105 us with
// the kernel for few rows.
//
// Operands are exact as there: code * block scale in fp16, and a query row
// scaled by a power of two.  The scores are taken against a reference that
// follows the running maximum only when that has grown by more than 2^4, since
// moving it means rescaling the sums in tensor memory; a weight is held as
// p * 2^11 in fp16, 2^-11 of its value or 2^-36 of the largest weight.
#include <cuda_runtime.h>

#include "fp4_async.cuh"
#include "fp4_plan.cuh"

namespace fp8q {

namespace {

using namespace fp4_plan;

__device__ uint32_t g_fp4_rows_error;

constexpr int kRows = 128;             // query rows of a tile
constexpr int kTokens = 128;           // cached tokens of a tile, a unit of the plan
constexpr int kThreads = 512;       // eight warps on rows, four on tokens, four others
constexpr int kTokenThread = 256;   // the first that owns a cached token
constexpr int kIssueThread = 384;   // the first of the warp that issues the products
constexpr float kShift = 11.0f;        // a weight is held as p * 2^11
// Tiles an item costs beside its own: 4 pieces of prompts take 62 us with none,
// 59 with one, 61 with two.
constexpr int kItemCost = 1;
constexpr float kSlack = 4.0f;         // growth of the maximum that is let pass

// ---------------------------------------------------------------------------
// tensor cores and tensor memory

__device__ __forceinline__ void tmem_load(uint32_t addr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
          "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(addr) : "memory");
}

__device__ __forceinline__ void tmem_store(uint32_t addr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        :: "r"(addr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
          "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}

__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 :: "r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]),
                    "r"(v[7]) : "memory");
}

__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// A shared-memory operand in 128-byte rows with the 128-byte swizzle, eight
// rows 1024 bytes apart; `panel` bytes between 64-element panels of a V row.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t panel) {
    return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | static_cast<uint64_t>(panel >> 4) << 16 |
           uint64_t{1024 >> 4} << 32 | uint64_t{1} << 46 | uint64_t{2} << 61;
}

// fp16 operands, fp32 sums, 128 x n; `rows_of_k`: the right operand's n axis is
// the contiguous one.
constexpr uint32_t instruction(int n, bool rows_of_k) {
    return 1u << 4 | (rows_of_k ? 1u : 0u) << 16 | static_cast<uint32_t>(n / 8) << 17 | (128u / 16) << 24;
}

__device__ __forceinline__ void mma_shared(uint32_t d, uint64_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d), "l"(a), "l"(b), "r"(kind), "r"(static_cast<uint32_t>(add)) : "memory");
}

__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, bool add) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(kind), "r"(static_cast<uint32_t>(add)) : "memory");
}

// Arrives at a barrier when the products issued so far are done.
__device__ __forceinline__ void mma_arrive(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(bar) : "memory");
}

// Byte offset of 16-byte piece `piece` of row `row` of an operand: 64 elements
// a panel of 128 rows, swizzled.
__device__ __forceinline__ uint32_t piece_at(int32_t row, int32_t piece) {
    return (piece / 8) * (128 * 128) + row * 128 + ((piece % 8) ^ (row & 7)) * 16;
}

// ---------------------------------------------------------------------------
// layout of a block

// What the walking warp tells the others about an item.
struct Item {
    int32_t tiles;              // of 128 cached tokens, in this block's part; -1: no more items
    int32_t begin, end, first;  // its cached tokens, and the first one any row sees
    int32_t ahead;              // query i sees tokens up to ahead + i
    int32_t token0, row0, rows;
    int32_t head, seq;
    int32_t part;               // -1: the whole item, else which of the block's parts
};

template <int D>
struct Layout {
    static constexpr int kBlocks = D == 256 ? 1 : 2;         // an SM holds
    static constexpr int kOperand = 128 * D * 2;             // bytes of Q, of K, of V
    // Columns of tensor memory: scores, sums, weights (two to a column), the
    // weights in place of the scores where all three do not fit half of it;
    // then each half of a row replaces its own scores.
    static constexpr bool kApart = D != 128;
    static constexpr int kSumsAt = 128;
    static constexpr int kWeightsAt = kApart ? 128 + D : 0;
    static constexpr int kWeightsHalf = kApart ? 32 : 64;    // columns from one half's weights to the other's
    static constexpr int kColumns = D == 256 ? 512 : 256;
    static constexpr int64_t kPartFloats = part_floats(kRows, D);
};

struct Control {
    uint64_t item_full[2], item_empty[2];
    uint64_t q_full, k_full, v_full;     // operands are in shared memory
    uint64_t scores, weights, summed;    // S is there; P is there; P V is done
    float halves[2][kRows];              // what the two threads of a row tell each other
    Item item[2];
    uint32_t gave_up, tmem;
    PlanShared<kThreads / 32> plan;
};

template <int D>
struct Shared {
    alignas(1024) uint8_t q[Layout<D>::kOperand];
    uint8_t k[Layout<D>::kOperand];
    uint8_t v[Layout<D>::kOperand];
    Control c;
};

struct Waits {
    Control &c;
    __device__ __forceinline__ void operator()(uint64_t &bar, uint32_t parity) const {
        barrier_wait(smem_addr(&bar), parity & 1, &c.gave_up, &g_fp4_rows_error);
    }
};

// One arrival for the warp, behind all its lanes' writes.
__device__ __forceinline__ void warp_arrive(uint64_t &bar) {
    __syncwarp();
    if (threadIdx.x % 32 == 0) barrier_arrive(smem_addr(&bar));
}

__device__ __forceinline__ void operands_written() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---------------------------------------------------------------------------
// the walking warp

__device__ __forceinline__ void walk_items(const Fp4Attention &a, Control &c, const Waits &wait, const Run &run,
                                           const Division &d, Split *record) {
    const int32_t lane = threadIdx.x % 32;
    uint32_t items = 0;
    Walk walk;
    walk.begin(d, run);
    for (;;) {
        const Tile x = tile_of(walk.s, d, walk.rt);
        const int64_t unit0 = walk.start + kItemCost;
        if (walk.start >= run.end) break;
        int32_t r0 = static_cast<int32_t>(max(int64_t{0}, run.at - unit0));
        int32_t r1 = static_cast<int32_t>(max(int64_t{0}, min(static_cast<int64_t>(x.units), run.end - unit0)));
        if (d.whole == 1 || (d.whole == 2 && x.units + kItemCost <= run.per_block)) {
            // the block that has an item's middle takes all of it
            const int64_t middle = walk.start + (x.units + d.item_cost) / 2;
            r0 = 0;
            r1 = middle >= run.at && middle < run.end ? x.units : 0;
        }
        if (r1 > r0) {
            const uint32_t slot = items % 2;
            if (items >= 2) wait(c.item_empty[slot], items / 2 - 1);
            if (!told(&c.gave_up)) return;
            if (lane == 0) {
                Item &it = c.item[slot];
                it.begin = x.begin + r0 * kTokens;
                it.end = min(x.end, x.begin + r1 * kTokens);
                it.first = x.first;
                it.tiles = it.end > it.begin ? (it.end - it.begin + kTokens - 1) / kTokens : 0;
                it.ahead = walk.s.length - walk.s.news;
                it.token0 = walk.s.token0;
                it.row0 = x.row0;
                it.rows = x.rows;
                it.head = walk.set;
                it.seq = walk.seq;
                it.part = r0 == 0 && r1 == x.units ? -1 : r0 == 0 ? 1 : 0;
                if (it.part == 1) {
                    record->token0 = it.token0;
                    record->row0 = it.row0;
                    record->rows = it.rows;
                    record->set = it.head;
                    record->blocks = static_cast<int32_t>(quotient(unit0 + x.units - 1, run.per_block)) - blockIdx.x + 1;
                }
                barrier_arrive(smem_addr(&c.item_full[slot]));
            }
            ++items;
        }
        if (!walk.next(a, d, x.units + kItemCost)) break;
    }
    const uint32_t slot = items % 2;
    if (items >= 2) wait(c.item_empty[slot], items / 2 - 1);
    if (!told(&c.gave_up)) return;
    if (lane == 0) {
        c.item[slot].tiles = -1;
        barrier_arrive(smem_addr(&c.item_full[slot]));
    }
}

// ---------------------------------------------------------------------------
// the warps that own a cached token a thread

template <int D>
__device__ __forceinline__ void expand_items(const Fp4Attention &a, Shared<D> &sm, const Waits &wait) {
    constexpr int kBlocks16 = D / 16;          // blocks of 16 dimensions
    const int32_t row = threadIdx.x - kTokenThread;
    const uint32_t at_row = row * 128 + (row & 7) * 16;     // piece c: this ^ 16 c, in its panel
    const int32_t tiles = a.pools.tiles;
    const int32_t shift = (tiles & (tiles - 1)) == 0 ? __ffs(tiles) - 1 : -1;
    uint32_t n = 0;                            // tiles so far
    for (uint32_t items = 0;; ++items) {
        wait(sm.c.item_full[items % 2], items / 2);
        const Item &shared = sm.c.item[items % 2];
        const int32_t count = told(&sm.c.gave_up) ? shared.tiles : -1, begin = shared.begin, first = shared.first, end = shared.end;
        const int32_t *table = a.block_table + static_cast<int64_t>(shared.seq) * a.table_stride;
        const int64_t head = static_cast<int64_t>(shared.head) * tiles;
        warp_arrive(sm.c.item_empty[items % 2]);
        if (count < 0) return;
        for (int32_t j = 0; j < count; ++j, ++n) {
            // Tokens no row sees count as zeros: a seen one's codes, no scale.
            const int32_t mine = begin + j * kTokens + row;
            const int32_t tok = max(first, min(mine, end - 1));
            const int32_t at16 = tok / 16, slot = tok % 16;
            const int32_t page_at = shift >= 0 ? at16 >> shift : at16 / tiles;
            int64_t page = table[page_at];
            if (page < 0 || page >= a.pools.num_blocks) {
                atomicOr(&g_fp4_rows_error, kFp4ErrSlot);
                page = 0;
            }
            const int64_t tile = page * a.pools.block_stride + (head + (at16 - page_at * tiles)) * (9 * D);
            // K, then V: one code for both, that it stays in the instruction caches.
#pragma unroll 1
            for (int32_t of_v = 0; of_v < 2; ++of_v) {
                const uint8_t *pool = of_v ? a.pools.v + tile : a.pools.k + tile;
                const uint8_t *code = pool + slot * (of_v ? 8 : D / 2);
                const uint8_t *scale = pool + 8 * D + slot * (of_v ? 1 : kBlocks16);
                const int32_t code_step = of_v ? 128 : 8, scale_step = of_v ? 16 : 1;
                uint2 codes[kBlocks16];
                uint32_t scales[kBlocks16];
#pragma unroll
                for (int b = 0; b < kBlocks16; ++b) {
                    codes[b] = *reinterpret_cast<const uint2 *>(code + b * code_step);
                    scales[b] = scale[b * scale_step];
                }
                // the last product with this operand is done
                if (n > 0) wait(of_v ? sm.c.summed : sm.c.scores, n - 1);
                uint8_t *dst = of_v ? sm.v : sm.k;
#pragma unroll
                for (int b = 0; b < kBlocks16; ++b) {
                    const uint32_t s = f16x2_of_e4m3x2(mine == tok ? scales[b] * 0x101u : 0);
                    uint32_t x[4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f16x2_of_e2m1x8(h ? codes[b].y : codes[b].x, x);
                        const int c = 2 * b + h;
                        *reinterpret_cast<uint4 *>(dst + c / 8 * (128 * 128) + (at_row ^ (c % 8 * 16))) =
                            make_uint4(mul_f16x2(x[0], s), mul_f16x2(x[1], s), mul_f16x2(x[2], s), mul_f16x2(x[3], s));
                    }
                }
                operands_written();
                warp_arrive(of_v ? sm.c.v_full : sm.c.k_full);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// the warp that issues the products

// True for one lane of a converged warp.
__device__ __forceinline__ bool one_lane() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

// All lanes run the same loops, so that operands are in uniform registers when
// one of them issues: a single thread's took 100 to 200 cycles a product.
template <int D>
__device__ __forceinline__ void issue_items(Shared<D> &sm, const Waits &wait, uint32_t tmem) {
    using L = Layout<D>;
    const uint64_t q = operand(smem_addr(sm.q), 16), k = operand(smem_addr(sm.k), 16),
                   v = operand(smem_addr(sm.v), 128 * 128);
    uint32_t n = 0, full = 0;                  // tiles, and items with any
    for (uint32_t items = 0;; ++items) {
        wait(sm.c.item_full[items % 2], items / 2);
        const int32_t tiles = told(&sm.c.gave_up) ? __shfl_sync(0xFFFFFFFFu, sm.c.item[items % 2].tiles, 0) : -1;
        warp_arrive(sm.c.item_empty[items % 2]);
        if (tiles < 0) return;
        if (tiles == 0) continue;
        wait(sm.c.q_full, full++);
        auto scores = [&]() {                  // S of a tile
            __syncwarp();
            tmem_after();
            if (one_lane()) {
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const int off = ((s / 4) * (128 * 128) + (s % 4) * 32) >> 4;
                    mma_shared(tmem, q + off, k + off, instruction(kTokens, false), s > 0);
                }
                mma_arrive(smem_addr(&sm.c.scores));
            }
            __syncwarp();
        };
        wait(sm.c.k_full, n);
        if (!L::kApart && n > 0) wait(sm.c.summed, n - 1);   // the last weights lie where the scores go
        scores();
        for (int32_t j = 0; j < tiles; ++j, ++n) {
            // The weights come last; nothing else is waited for behind them.
            if (j + 1 < tiles) wait(sm.c.k_full, n + 1);
            wait(sm.c.v_full, n);
            wait(sm.c.weights, n);             // the scores have been read, too
            if (L::kApart && j + 1 < tiles) scores();
            __syncwarp();
            tmem_after();
            if (one_lane()) {
#pragma unroll
                for (int s = 0; s < kTokens / 16; ++s)
                    mma_tmem(tmem + L::kSumsAt, tmem + L::kWeightsAt + s / 4 * L::kWeightsHalf + s % 4 * 8,
                             v + ((s * 16 * 128) >> 4), instruction(D, true), j > 0 || s > 0);
                mma_arrive(smem_addr(&sm.c.summed));
            }
            __syncwarp();
            if (!L::kApart && j + 1 < tiles) { // the weights lie where the scores go
                wait(sm.c.summed, n);
                scores();
            }
        }
    }
}

// ---------------------------------------------------------------------------
// the warps that own a query row a thread

constexpr int kColumns = kTokens / 2;  // of a tile, for each thread of a row

struct Pair {
    float x, y;
};
__device__ __forceinline__ uint64_t bits_of(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ Pair pair_of(uint64_t d) {
    Pair p;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(p.x), "=f"(p.y) : "l"(d));
    return p;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Columns outside [from, to) of 16 from column `at` count as unseen.
__device__ __forceinline__ void hide(float (&x)[16], int32_t at, int32_t from, int32_t to) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (static_cast<uint32_t>(at + i - from) >= static_cast<uint32_t>(to - from)) x[i] = -INFINITY;
}

// The largest of a thread's 64 scores of a row.
template <bool kEdge>
__device__ __forceinline__ float row_max(uint32_t t_scores, int32_t from, int32_t to) {
    float x[2][16], most[2] = {-INFINITY, -INFINITY};
    tmem_load(t_scores, x[0]);
#pragma unroll
    for (int q = 0; q < kColumns / 16; ++q) {
        tmem_wait_load();
        if (q + 1 < kColumns / 16) tmem_load(t_scores + 16 * (q + 1), x[(q + 1) % 2]);
        if (kEdge) hide(x[q % 2], 16 * q, from, to);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            most[0] = max3(most[0], x[q % 2][i], x[q % 2][i + 1]);
            most[1] = max3(most[1], x[q % 2][i + 2], x[q % 2][i + 3]);
        }
    }
    return fmaxf(most[0], most[1]);
}

// Their weights 2^(c s - ref + kShift), written as fp16 pairs; returns the sum.
// kSteps: unless this is false for a row, it is formed in steps, as single
// values: the product and sum of pairs come out fused.
template <int D, bool kEdge, bool kSteps>
__device__ __forceinline__ float row_weights(uint32_t t_scores, uint32_t t_weights, int32_t from, int32_t to,
                                             float c, float ref) {
    float x[2][16];
    const float against = kShift - ref;
    const uint64_t c2 = bits_of(c, c), against2 = bits_of(against, against);
    uint64_t sum[2] = {0, 0};
    tmem_load(t_scores, x[0]);
#pragma unroll
    for (int q = 0; q < kColumns / 16; ++q) {
        tmem_wait_load();
        if (q + 1 < kColumns / 16) tmem_load(t_scores + 16 * (q + 1), x[(q + 1) % 2]);
        if (kEdge) hide(x[q % 2], 16 * q, from, to);
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Pair s = {x[q % 2][2 * i], x[q % 2][2 * i + 1]};
            const Pair p = kSteps && in_steps<D>(c)
                               ? Pair{below_most(s.x, c, ref) + kShift, below_most(s.y, c, ref) + kShift}
                               : pair_of(fma_pair(bits_of(s.x, s.y), c2, against2));
            const float a = exp2_fast(p.x), b = exp2_fast(p.y);
            sum[i % 2] = add_pair(sum[i % 2], bits_of(a, b));
            w[i] = f16x2_of(a, b);
        }
        tmem_store8(t_weights + 8 * q, w);
    }
    const Pair p = pair_of(add_pair(sum[0], sum[1]));
    return p.x + p.y;
}

// The two warps of 32 rows meet.
__device__ __forceinline__ void pair_meet(int32_t quarter) {
    asm volatile("bar.sync %0, 64;" :: "r"(quarter + 1) : "memory");
}

// What the other thread of this row has found.
__device__ __forceinline__ float other_half(Control &c, int32_t half, int32_t row, float mine) {
    c.halves[half][row] = mine;
    pair_meet(row / 32);
    const float v = c.halves[half ^ 1][row];
    pair_meet(row / 32);                       // both have read
    return v;
}

// A thread's row of an item.
struct Mine {
    int32_t tiles;              // as in Item
    int32_t begin, part;
    bool busy, live;            // the warp has rows; the row is one of them
    RowPlace place;
    float c;                    // factor of raw scores: log2 of a weight
    int32_t hi, lo;             // tokens the row sees: [lo, hi)
    int32_t all_hi, all_lo;     // ... and all rows of the warp
};

// The next item: its query rows go to shared memory once the last product with
// the present ones is done, which the caller knows.  None if a wait was given up.
template <int D>
__device__ __forceinline__ Mine take_item(const Fp4Attention &a, Shared<D> &sm, const Waits &wait, uint32_t items,
                                          int32_t group, float k_scale) {
    constexpr int kPieces = D / 16;                    // 16-byte pieces of half a query row
    const int32_t half = threadIdx.x / 128, row = threadIdx.x % 128;
    wait(sm.c.item_full[items % 2], items / 2);
    Item it = sm.c.item[items % 2];
    if (!agree(row / 32 + 1, 64, told(&sm.c.gave_up))) it.tiles = -1;
    warp_arrive(sm.c.item_empty[items % 2]);
    Mine m;
    m.tiles = it.tiles;
    m.begin = it.begin;
    m.part = it.part;
    m.busy = row / 32 * 32 < it.rows && it.tiles >= 0;
    m.live = row < it.rows;
    m.c = 0.0f;
    if (it.tiles < 0) return m;
    const int32_t my_row = it.row0 + min(row, it.rows - 1);
    m.place = row_place(it.token0, my_row, it.head, group);
    const int32_t p = it.ahead + (m.place.token - it.token0) + 1;
    m.hi = min(it.end, p);
    m.lo = a.window > 0 ? max(0, p - a.window) : 0;
    m.all_hi = __reduce_min_sync(0xFFFFFFFFu, m.hi);
    m.all_lo = __reduce_max_sync(0xFFFFFFFFu, m.lo);
    if (it.tiles == 0) return m;
    if (m.busy) {
        uint4 x[kPieces];                              // this half of the query row
        const uint4 *src = reinterpret_cast<const uint4 *>(
            a.q + m.place.token * a.q_stride + static_cast<int64_t>(m.place.q_head) * D) + half * kPieces;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) x[i] = src[i];
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) most = max(most, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
        }
        most = max(most, __float_as_uint(other_half(sm.c, half, row, __uint_as_float(most))));
        const int32_t up = min(8 - (static_cast<int32_t>(most >> 7) - 127), 120);
        const float scale = m.live ? __int_as_float((127 + up) << 23) : 0.0f;
        m.c = fmaxf(a.softmax_scale * kLog2e * k_scale * __int_as_float((127 - up) << 23), 0x1p-100f);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            *reinterpret_cast<uint4 *>(sm.q + piece_at(row, half * kPieces + i)) =
                make_uint4(f16x2_of(bf16_low(x[i].x) * scale, bf16_high(x[i].x) * scale),
                           f16x2_of(bf16_low(x[i].y) * scale, bf16_high(x[i].y) * scale),
                           f16x2_of(bf16_low(x[i].z) * scale, bf16_high(x[i].z) * scale),
                           f16x2_of(bf16_low(x[i].w) * scale, bf16_high(x[i].w) * scale));
    }
    operands_written();
    warp_arrive(sm.c.q_full);
    return m;
}

// The output of a row, or its part.
template <int D>
__device__ __forceinline__ void put_out(const Fp4Attention &a, const Mine &m, float ref, float sum, uint32_t t_sums,
                                        int32_t half, int32_t row, float v_scale) {
    using L = Layout<D>;
    float *part = part_at(a.workspace, 2 * static_cast<int64_t>(blockIdx.x) + max(m.part, 0), L::kPartFloats);
    const float inv = row_factor(sum, v_scale);
    uint4 *out = reinterpret_cast<uint4 *>(a.out + m.place.token * a.out_stride +
                                           static_cast<int64_t>(m.place.q_head) * D);
#pragma unroll 2
    for (int q = half * (D / 32); q < (half + 1) * (D / 32); ++q) {
        float o[16];
        if (m.tiles > 0) {
            tmem_load(t_sums + 16 * q, o);
            tmem_wait_load();
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = 0.0f;
        }
        if (m.part >= 0) {                             // [dimensions / 4][rows]
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<float4 *>(part)[(4 * q + i) * kRows + row] =
                    make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else if (m.live) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                out[2 * q + i] = make_uint4(bf16x2_of(o[8 * i] * inv, o[8 * i + 1] * inv),
                                            bf16x2_of(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                            bf16x2_of(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                            bf16x2_of(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
        }
    }
    if (half == 0) {
        if (m.part >= 0) {
            part[kRows * D + row] = ref;
            part[kRows * D + kRows + row] = sum;
        } else if (m.live && a.lse != nullptr) {
            a.lse[static_cast<int64_t>(m.place.token) * a.q_heads + m.place.q_head] = row_lse(ref, sum, kShift);
        }
    }
    tmem_before();                                     // the sums have been read
}

// Where a row's scores, weights and sums lie in tensor memory.
struct RowPlaces {
    uint32_t scores, weights, sums;
};

// The tiles of an item.  kSteps: some row's weights are formed in steps.
template <int D, bool kSteps>
__device__ __forceinline__ void softmax_tiles(Shared<D> &sm, const Waits &wait, const Mine &m, const RowPlaces &t,
                                              uint32_t &n, float &ref, float &sum) {
    const int32_t half = threadIdx.x / 128, row = threadIdx.x % 128;
    const uint32_t t_scores = t.scores, t_weights = t.weights, t_sums = t.sums;
    for (int32_t j = 0; j < m.tiles; ++j, ++n) {
        wait(sm.c.scores, n);
        __syncwarp();
        tmem_after();
        // the last product is done: sums may be rescaled, weights replaced
        bool waited = n == 0;
        auto summed = [&]() {
            if (!waited) wait(sm.c.summed, n - 1);
            waited = true;
            __syncwarp();
            tmem_after();
        };
        if (!m.busy) summed();
        if (m.busy) {
            const int32_t base = m.begin + j * kTokens;
            const bool edge = base + kTokens > m.all_hi || base < m.all_lo;
            // columns this row sees, of this thread's
            const int32_t from = m.lo - base - kColumns * half, to = max(from, m.hi - base - kColumns * half);
            float top = edge ? row_max<true>(t_scores, from, to) : row_max<false>(t_scores, from, to);
            top = __fmul_rn(fmaxf(top, other_half(sm.c, half, row, top)), m.c);
            // The reference moves where a row of the warps has outgrown it.
            if (__any_sync(0xFFFFFFFFu, kSteps ? top - ref > kSlack : top > ref + kSlack)) {
                const float now = fmaxf(ref, top);
                const float f = exp2_fast(ref - (now == -INFINITY ? 0.0f : now));
                ref = now;
                sum *= f;
                if (j > 0) {
                    summed();
#pragma unroll 1
                    for (int q = half * (D / 32); q < (half + 1) * (D / 32); ++q) {
                        float o[16];
                        tmem_load(t_sums + 16 * q, o);
                        tmem_wait_load();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= f;
                        tmem_store(t_sums + 16 * q, o);
                    }
                }
            }
            const float from_ref = ref == -INFINITY ? 0.0f : ref;
            summed();
            sum += kSteps || edge ? row_weights<D, true, kSteps>(t_scores, t_weights, from, to, m.c, from_ref)
                                  : row_weights<D, false, false>(t_scores, t_weights, from, to, m.c, from_ref);
            tmem_wait_store();
        }
        tmem_before();
        warp_arrive(sm.c.weights);
    }
}

// The same out of line, where it costs the usual rows nothing.
template <int D>
__device__ __noinline__ void softmax_tiles_apart(Shared<D> &sm, Waits wait, Mine m, RowPlaces t, uint32_t *n,
                                                 float *ref, float *sum) {
    uint32_t my_n = *n;
    float my_ref = -INFINITY, my_sum = 0.0f;
    softmax_tiles<D, true>(sm, wait, m, t, my_n, my_ref, my_sum);
    *n = my_n, *ref = my_ref, *sum = my_sum;
}

template <int D>
__device__ __forceinline__ void softmax_items(const Fp4Attention &a, Shared<D> &sm, const Waits &wait,
                                              uint32_t tmem, int32_t group, float k_scale, float v_scale) {
    using L = Layout<D>;
    const int32_t half = threadIdx.x / 128, row = threadIdx.x % 128, quarter = row / 32;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const RowPlaces t = {tmem + lanes + kColumns * half, tmem + lanes + L::kWeightsAt + L::kWeightsHalf * half,
                         tmem + lanes + L::kSumsAt};
    uint32_t n = 0, items = 0;
    Mine m = take_item<D>(a, sm, wait, items, group, k_scale);
    while (m.tiles >= 0) {
        float ref = -INFINITY, sum = 0.0f;
        if (__any_sync(0xFFFFFFFFu, in_steps<D>(m.c)))
            softmax_tiles_apart<D>(sm, wait, m, t, &n, &ref, &sum);
        else
            softmax_tiles<D, false>(sm, wait, m, t, n, ref, sum);
        // The next item's rows are put in place while this one's last product
        // runs, and its first scores are formed while these sums are put out.
        const Mine next = take_item<D>(a, sm, wait, ++items, group, k_scale);
        if (m.tiles > 0) {
            wait(sm.c.summed, n - 1);
            __syncwarp();
            tmem_after();
        }
        if (m.busy) {
            sum += other_half(sm.c, half, row, sum);
            put_out<D>(a, m, ref, sum, t.sums, half, row, v_scale);
        }
        m = next;
    }
}

// ---------------------------------------------------------------------------
// the kernel

// Moves registers between the warp groups of a block: with two blocks on an SM
// a thread starts with 64, and 72 + 72 + 56 + 56 are four times that.
template <bool kMove, int kCount, bool kMore>
__device__ __forceinline__ void registers() {
    if constexpr (kMove && kMore) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kCount));
    if constexpr (kMove && !kMore) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kCount));
}

template <int D>
__global__ void __launch_bounds__(kThreads, Layout<D>::kBlocks) fp4_attention_rows_kernel(const Fp4Attention a,
                                                                                          int32_t whole) {
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    Shared<D> &sm = *reinterpret_cast<Shared<D> *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) / 1024 * 1024);   // the swizzle goes by the address
    Control &c = sm.c;
    const int32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0);
    const Division d = {a.q_heads / a.pools.heads, kRows, a.pools.heads, kTokens, kItemCost, a.window, whole};
    if (warp == kIssueThread / 32)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                     "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;"
                     :: "r"(smem_addr(&c.tmem)), "n"(L::kColumns) : "memory");
    if (threadIdx.x == 0) {
        c.gave_up = 0;
        for (int i = 0; i < 2; ++i) {
            barrier_init(smem_addr(&c.item_full[i]), 1);
            barrier_init(smem_addr(&c.item_empty[i]), 13);   // twelve warps and the issuing one
        }
        barrier_init(smem_addr(&c.q_full), 8);
        barrier_init(smem_addr(&c.k_full), 4);
        barrier_init(smem_addr(&c.v_full), 4);
        barrier_init(smem_addr(&c.scores), 1);
        barrier_init(smem_addr(&c.weights), 8);
        barrier_init(smem_addr(&c.summed), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();                                // nothing to wait for: not launched early
    pdl_allow_next();

    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    Split *record = static_cast<Split *>(a.workspace) + blockIdx.x;
    if (threadIdx.x == kThreads - 1) record->blocks = 0;
    tmem_before();
    const Run run = block_run<kThreads / 32>(a, d, &g_fp4_rows_error, c.plan);   // a block barrier at least
    tmem_after();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, c.tmem, 0);
    const bool scales_ok = fp4_scale_ok(k_scale) && fp4_scale_ok(v_scale);
    if (!scales_ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_fp4_rows_error, kFp4ErrScale);
    if (scales_ok && run.at < run.end) {
        const Waits wait{c};
        if (threadIdx.x < kTokenThread) {
            registers<L::kBlocks == 2, 72, true>();
            softmax_items<D>(a, sm, wait, tmem, d.group, k_scale, v_scale);
        } else if (threadIdx.x < kIssueThread) {
            registers<L::kBlocks == 2, 56, false>();
            expand_items<D>(a, sm, wait);
        } else {
            registers<L::kBlocks == 2, 56, false>();
            if (warp == kIssueThread / 32)
                issue_items<D>(sm, wait, tmem);
            else if (warp == kIssueThread / 32 + 1)
                walk_items(a, c, wait, run, d, record);
        }
    }
    __syncwarp();
    tmem_before();
    __syncthreads();
    let_land(&c.gave_up);
    if (warp == kIssueThread / 32) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(L::kColumns));
    }
}

constexpr int kJoinDims = 16;          // of a thread

// Block (c, y) merges 16 dimensions of the item that began in block c, a row a
// thread.
template <int D>
__global__ void __launch_bounds__(kRows) fp4_attention_rows_join_kernel(const Fp4Attention a) {
    using L = Layout<D>;
    constexpr int kBatch = 2, kQuads = kJoinDims / 4;
    pdl_wait();
    pdl_allow_next();
    const int32_t c = blockIdx.x, row = threadIdx.x;
    const Split s = static_cast<const Split *>(a.workspace)[c];
    if (s.blocks == 0 || row >= s.rows) return;
    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    float top = -INFINITY, l = 0.0f, x[kJoinDims];
#pragma unroll
    for (int j = 0; j < kJoinDims; ++j) x[j] = 0.0f;
    for (int32_t i0 = 0; i0 < s.blocks; i0 += kBatch) {
        float t[kBatch], m[kBatch];
        float4 v[kBatch][kQuads];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t i = i0 + k;
            t[k] = -INFINITY, m[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < kQuads; ++j) v[k][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < s.blocks) {
                // part 1 of block c, then part 0 of the blocks behind it
                const float *p = part_at(a.workspace, 2 * static_cast<int64_t>(c + i) + (i == 0 ? 1 : 0), L::kPartFloats);
                t[k] = p[kRows * D + row];
                m[k] = p[kRows * D + kRows + row];
#pragma unroll
                for (int j = 0; j < kQuads; ++j)
                    v[k][j] = reinterpret_cast<const float4 *>(p)[(kQuads * blockIdx.y + j) * kRows + row];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float now = fmaxf(top, t[k]);
            const float base = now == -INFINITY ? 0.0f : now;
            const float f = exp2_fast(top - base), e = exp2_fast(t[k] - base);
            top = now;
            l = l * f + m[k] * e;
#pragma unroll
            for (int j = 0; j < kQuads; ++j) {
                x[4 * j] = x[4 * j] * f + v[k][j].x * e;
                x[4 * j + 1] = x[4 * j + 1] * f + v[k][j].y * e;
                x[4 * j + 2] = x[4 * j + 2] * f + v[k][j].z * e;
                x[4 * j + 3] = x[4 * j + 3] * f + v[k][j].w * e;
            }
        }
    }
    const RowPlace place = row_place(s.token0, s.row0 + row, s.set, a.q_heads / a.pools.heads);
    const float inv = row_factor(l, v_scale);
    uint4 *out = reinterpret_cast<uint4 *>(a.out + place.token * a.out_stride +
                                           static_cast<int64_t>(place.q_head) * D + kJoinDims * blockIdx.y);
#pragma unroll
    for (int j = 0; j < kJoinDims; j += 8)
        out[j / 8] = make_uint4(bf16x2_of(x[j] * inv, x[j + 1] * inv), bf16x2_of(x[j + 2] * inv, x[j + 3] * inv),
                                bf16x2_of(x[j + 4] * inv, x[j + 5] * inv), bf16x2_of(x[j + 6] * inv, x[j + 7] * inv));
    if (a.lse != nullptr && blockIdx.y == 0)
        a.lse[static_cast<int64_t>(place.token) * a.q_heads + place.q_head] = row_lse(top, l, kShift);
}

// Enough items to fill the blocks: they are not split, and the parts (64 KB each
// with 128 dimensions) are saved; but where there is room for parts, items that
// cost more than a block's share are, or one long sequence among short ones
// would be left to a few blocks.
bool items_whole(int64_t num_tokens, int32_t group, int32_t kv_heads, int32_t dim) {
    const int64_t tiles = (num_tokens * group + kRows - 1) / kRows;
    return 2 * tiles * kv_heads >= 3 * (kMaxBlocks / 3) * (dim == 256 ? 1 : 2);
}

template <int D>
cudaError_t launch_dim(const Fp4Attention &a, cudaStream_t stream) {
    using L = Layout<D>;
    constexpr size_t kSmem = sizeof(Shared<D>) + 1024;
    static_assert(L::kBlocks * (kSmem + 1024) <= 228 * 1024, "the blocks of an SM fit its shared memory");
    auto kernel = fp4_attention_rows_kernel<D>;
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    int64_t grid = static_cast<int64_t>(sms) * L::kBlocks;
    if (grid > kMaxBlocks / 3 * L::kBlocks) grid = kMaxBlocks / 3 * L::kBlocks;
    // No more blocks than there can be points on the axis.
    const int32_t group = a.q_heads / a.pools.heads;
    const int64_t tiles = (static_cast<int64_t>(a.num_tokens) * group + kRows - 1) / kRows;
    const int64_t items = (tiles + a.batch) * a.pools.heads;
    const int64_t longest = a.table_width * a.pools.tiles * 16 / kTokens + 2 + kItemCost;
    if (items < grid && items * longest < grid) grid = items * longest;
    int32_t whole = 0;
    if (items_whole(a.num_tokens, group, a.pools.heads, D))
        whole = a.workspace_bytes >= fp4_attention_rows_workspace(a.num_tokens, group, a.pools.heads, D, true) ? 2 : 1;
    // Started on a free GPU, like the kernel for few rows.
    kernel<<<static_cast<unsigned>(grid), kThreads, kSmem, stream>>>(a, whole);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    g_launch_count.fetch_add(1, std::memory_order_relaxed);
    if (whole == 1) return cudaSuccess;
    return launch_pdl(fp4_attention_rows_join_kernel<D>, dim3(static_cast<unsigned>(grid), D / kJoinDims), kRows, 0, stream, a);
}

}  // namespace

int64_t fp4_attention_rows_workspace(int64_t num_tokens, int32_t group, int32_t kv_heads, int32_t dim,
                                     bool uneven) {
    if (items_whole(num_tokens, group, kv_heads, dim) && !uneven) return kRecordBytes;
    // a block begins one item that goes on, and ends one
    const int64_t blocks = kMaxBlocks / 3 * (dim == 256 ? 1 : 2);
    return kRecordBytes + blocks * 2 * 4 * part_floats(kRows, dim);
}

cudaError_t launch_fp4_attention_rows(const Fp4Attention &a, cudaStream_t stream) {
    return a.pools.dim == 64    ? launch_dim<64>(a, stream)
           : a.pools.dim == 128 ? launch_dim<128>(a, stream)
                                : launch_dim<256>(a, stream);
}

cudaError_t read_fp4_rows_error(uint32_t *bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_fp4_rows_error, sizeof(uint32_t));
    if (e == cudaSuccess && clear) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_fp4_rows_error, &zero, sizeof(uint32_t));
    }
    return e;
}

}  // namespace fp8q
