// fp4_attention_rows.cu -- attention over a paged cache held in 4 bits, for
// many query rows to a KV head (sm_100a): prompts in pieces, drafted tokens.
//
// The same results as fp4_attention.cu.  Where that kernel expands every code
// again for each 8 or 16 rows, here 128 rows share an expanded tile: 128
// tokens of K and of V are turned into fp16 in shared memory and multiplied by
// tcgen05.mma, S = Q K^T (both operands K-major) and O += P V (P from tensor
// memory, V with its dimensions as the contiguous axis), sums in tensor memory.
//
// Warps of a block: four that own a query row a thread (query rows to fp16,
// softmax, output), four that own a cached token a thread (pages, codes to
// fp16), and four of which one thread issues the products and one warp walks
// the block's items.  Nothing is double-buffered: K of the next tile is expanded
// while this one's softmax runs, V after this one's second product, and two
// blocks of an SM fill each other's gaps (one with 256 dimensions).
//
// Bound by the exponentials: 16 a cycle and SM, 1024 cycles for a tile, where
// the two products take 256 for each 64 dimensions.
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
constexpr int kThreads = 384;
constexpr float kShift = 11.0f;        // a weight is held as p * 2^11
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

__device__ __forceinline__ void tmem_store16(uint32_t addr, const float (&v)[16]) {
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
    // weights in place of the scores where all three do not fit half of it.
    static constexpr bool kApart = D != 128;
    static constexpr int kSumsAt = 128;
    static constexpr int kWeightsAt = kApart ? 128 + D : 0;
    static constexpr int kColumns = D == 256 ? 512 : 256;
    static constexpr int64_t kPartFloats = part_floats(kRows, D);
};

struct Control {
    uint64_t item_full[2], item_empty[2];
    uint64_t q_full, k_full, v_full;     // operands are in shared memory
    uint64_t scores, weights, summed;    // S is there; P is there; P V is done
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
        if (d.whole) {                   // the block that has an item's middle takes all of it
            const int64_t middle = walk.start + (x.units + kItemCost) / 2;
            r0 = 0;
            r1 = middle >= run.at && middle < run.end ? x.units : 0;
        }
        if (r1 > r0) {
            const uint32_t slot = items % 2;
            if (items >= 2) wait(c.item_empty[slot], items / 2 - 1);
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
    const int32_t row = threadIdx.x % 128;
    const int32_t tiles = a.pools.tiles;
    const int32_t shift = (tiles & (tiles - 1)) == 0 ? __ffs(tiles) - 1 : -1;
    uint32_t n = 0;                            // tiles so far
    for (uint32_t items = 0;; ++items) {
        wait(sm.c.item_full[items % 2], items / 2);
        const Item it = sm.c.item[items % 2];
        warp_arrive(sm.c.item_empty[items % 2]);
        if (it.tiles < 0) return;
        const int32_t *table = a.block_table + static_cast<int64_t>(it.seq) * a.table_stride;
        for (int32_t j = 0; j < it.tiles; ++j, ++n) {
            const int32_t tok = it.begin + j * kTokens + row;
            const bool live = tok >= it.first && tok < it.end;   // others count as zeros
            uint2 kc[kBlocks16], vc[kBlocks16];
            uint32_t kz[(kBlocks16 + 3) / 4], vz[kBlocks16];
#pragma unroll
            for (int b = 0; b < kBlocks16; ++b) kc[b] = vc[b] = make_uint2(0, 0), vz[b] = 0;
#pragma unroll
            for (int b = 0; b < kBlocks16 / 4; ++b) kz[b] = 0;
            if (live) {
                const int32_t at16 = tok / 16, slot = tok % 16;
                const int32_t page_at = shift >= 0 ? at16 >> shift : at16 / tiles;
                int64_t page = table[page_at];
                if (page < 0 || page >= a.pools.num_blocks) {
                    atomicOr(&g_fp4_rows_error, kFp4ErrSlot);
                    page = 0;
                }
                const int64_t tile = page * a.pools.block_stride +
                    (static_cast<int64_t>(it.head) * tiles + (at16 - page_at * tiles)) * (9 * D);
                const uint8_t *kt = a.pools.k + tile, *vt = a.pools.v + tile;
#pragma unroll
                for (int b = 0; b < kBlocks16; b += 2) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(kt + slot * (D / 2) + 8 * b);
                    kc[b] = make_uint2(x.x, x.y), kc[b + 1] = make_uint2(x.z, x.w);
                }
#pragma unroll
                for (int b = 0; b < kBlocks16 / 4; ++b)
                    kz[b] = *reinterpret_cast<const uint32_t *>(kt + 8 * D + slot * kBlocks16 + 4 * b);
#pragma unroll
                for (int b = 0; b < kBlocks16; ++b) {
                    vc[b] = *reinterpret_cast<const uint2 *>(vt + b * 128 + slot * 8);
                    vz[b] = vt[8 * D + b * 16 + slot];
                }
            }
            auto write = [&](uint8_t *dst, int32_t b, uint2 codes, uint32_t scale) {
                const uint32_t s = f16x2_of_e4m3x2(scale * 0x101u);
                uint32_t x[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f16x2_of_e2m1x8(h ? codes.y : codes.x, x);
                    *reinterpret_cast<uint4 *>(dst + piece_at(row, 2 * b + h)) =
                        make_uint4(mul_f16x2(x[0], s), mul_f16x2(x[1], s), mul_f16x2(x[2], s), mul_f16x2(x[3], s));
                }
            };
            if (n > 0) wait(sm.c.scores, n - 1);       // the last product with K is done
#pragma unroll
            for (int b = 0; b < kBlocks16; ++b) write(sm.k, b, kc[b], (kz[b / 4] >> (8 * (b % 4))) & 0xFFu);
            operands_written();
            warp_arrive(sm.c.k_full);
            if (n > 0) wait(sm.c.summed, n - 1);       // ... and with V
#pragma unroll
            for (int b = 0; b < kBlocks16; ++b) write(sm.v, b, vc[b], vz[b]);
            operands_written();
            warp_arrive(sm.c.v_full);
        }
    }
}

// ---------------------------------------------------------------------------
// the thread that issues the products

template <int D>
__device__ __forceinline__ void issue_items(Shared<D> &sm, const Waits &wait, uint32_t tmem) {
    using L = Layout<D>;
    const uint32_t q = smem_addr(sm.q), k = smem_addr(sm.k), v = smem_addr(sm.v);
    uint32_t n = 0, full = 0;                  // tiles, and items with any
    for (uint32_t items = 0;; ++items) {
        wait(sm.c.item_full[items % 2], items / 2);
        const int32_t tiles = sm.c.item[items % 2].tiles;
        barrier_arrive(smem_addr(&sm.c.item_empty[items % 2]));
        if (tiles < 0) return;
        if (tiles > 0) wait(sm.c.q_full, full++);
        for (int32_t j = 0; j < tiles; ++j, ++n) {
            wait(sm.c.k_full, n);
            if (!L::kApart && n > 0) wait(sm.c.summed, n - 1);   // the weights lie where the scores go
            tmem_after();
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint32_t at = (s / 4) * (128 * 128) + (s % 4) * 32;
                mma_shared(tmem, operand(q + at, 16), operand(k + at, 16), instruction(kTokens, false), s > 0);
            }
            mma_arrive(smem_addr(&sm.c.scores));
            wait(sm.c.weights, n);
            wait(sm.c.v_full, n);
            tmem_after();
#pragma unroll
            for (int s = 0; s < kTokens / 16; ++s)
                mma_tmem(tmem + L::kSumsAt, tmem + L::kWeightsAt + 8 * s, operand(v + s * 16 * 128, 128 * 128),
                         instruction(D, true), j > 0 || s > 0);
            mma_arrive(smem_addr(&sm.c.summed));
        }
    }
}

// ---------------------------------------------------------------------------
// the warps that own a query row a thread

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

// What a pass over a row's scores finds.
struct Found {
    float most;          // the largest raw score
    uint64_t sum;        // two sums of weights
};

// 16 columns of this row: their maximum, and with kWeights the weights
// 2^(c s + against), written as fp16 pairs, and their sum.  Columns outside
// [from, to) count as unseen.
template <bool kEdge, bool kWeights>
__device__ __forceinline__ void row_piece(float (&x)[16], int32_t q, uint32_t t_weights, int32_t from, int32_t to,
                                          uint64_t c2, uint64_t against2, Found &f) {
    if (kEdge) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (static_cast<uint32_t>(16 * q + i - from) >= static_cast<uint32_t>(to - from)) x[i] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 16; i += 2) f.most = max3(f.most, x[i], x[i + 1]);
    if (kWeights) {
        uint32_t w[8];
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Pair p = pair_of(fma_pair(bits_of(x[2 * i], x[2 * i + 1]), c2, against2));
            const float a = exp2_fast(p.x), b = exp2_fast(p.y);
            sum = add_pair(sum, bits_of(a, b));
            w[i] = f16x2_of(a, b);
        }
        f.sum = add_pair(f.sum, sum);
        tmem_store8(t_weights + 8 * q, w);
    }
}

// One pass over the 128 scores of a row, 16 fetched while 16 are used.  A loop:
// written out, its code did not stay in the instruction caches beside that of
// the other warps (no instruction to issue for 2.6 cycles of each that was).
template <bool kEdge, bool kWeights>
__device__ __forceinline__ Found row_pass(uint32_t t_scores, uint32_t t_weights, int32_t from, int32_t to,
                                          float c, float against) {
    float x[16], y[16];
    Found f = {-INFINITY, 0};
    const uint64_t c2 = bits_of(c, c), against2 = bits_of(against, against);
    tmem_load(t_scores, x);
#pragma unroll 1
    for (int32_t q = 0; q < kTokens / 16; q += 2) {
        tmem_wait_load();
        tmem_load(t_scores + 16 * q + 16, y);
        row_piece<kEdge, kWeights>(x, q, t_weights, from, to, c2, against2, f);
        tmem_wait_load();
        if (q + 2 < kTokens / 16) tmem_load(t_scores + 16 * q + 32, x);
        row_piece<kEdge, kWeights>(y, q + 1, t_weights, from, to, c2, against2, f);
    }
    return f;
}

template <int D>
__device__ __forceinline__ void softmax_items(const Fp4Attention &a, Shared<D> &sm, const Waits &wait,
                                              uint32_t tmem, int32_t group, float k_scale, float v_scale) {
    using L = Layout<D>;
    const int32_t warp = threadIdx.x / 32, row = threadIdx.x;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t t_scores = tmem + lanes, t_sums = t_scores + L::kSumsAt, t_weights = t_scores + L::kWeightsAt;
    uint32_t n = 0;
    for (uint32_t items = 0;; ++items) {
        wait(sm.c.item_full[items % 2], items / 2);
        const Item it = sm.c.item[items % 2];
        warp_arrive(sm.c.item_empty[items % 2]);
        if (it.tiles < 0) return;
        const bool busy = warp * 32 < it.rows;         // the warp has rows
        const bool live = row < it.rows;
        const int32_t my_row = it.row0 + min(row, it.rows - 1);
        const RowPlace place = row_place(it.token0, my_row, it.head, group);
        float c = 1.0f;                                // factor of raw scores: log2 of a weight
        if (busy && it.tiles > 0) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                a.q + place.token * a.q_stride + static_cast<int64_t>(place.q_head) * D);
            uint32_t most = 0;
#pragma unroll 8
            for (int i = 0; i < D / 8; ++i) {
                const uint4 x = src[i];
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) most = max(most, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
            }
            const int32_t up = min(8 - (static_cast<int32_t>(most >> 7) - 127), 120);
            const float scale = live ? __int_as_float((127 + up) << 23) : 0.0f;
            c = fmaxf(a.softmax_scale * kLog2e * k_scale * __int_as_float((127 - up) << 23), 0x1p-100f);
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
                const uint4 x = src[i];
                *reinterpret_cast<uint4 *>(sm.q + piece_at(row, i)) =
                    make_uint4(f16x2_of(bf16_low(x.x) * scale, bf16_high(x.x) * scale),
                               f16x2_of(bf16_low(x.y) * scale, bf16_high(x.y) * scale),
                               f16x2_of(bf16_low(x.z) * scale, bf16_high(x.z) * scale),
                               f16x2_of(bf16_low(x.w) * scale, bf16_high(x.w) * scale));
            }
        }
        if (it.tiles > 0) {
            operands_written();
            warp_arrive(sm.c.q_full);
        }
        // tokens this row sees, and those all rows of the warp see
        const int32_t p = it.ahead + my_row / group + 1;
        const int32_t hi = min(it.end, p), lo = a.window > 0 ? max(0, p - a.window) : 0;
        const int32_t all_hi = __reduce_min_sync(0xFFFFFFFFu, hi), all_lo = __reduce_max_sync(0xFFFFFFFFu, lo);
        float ref = -INFINITY, sum = 0.0f;
        for (int32_t j = 0; j < it.tiles; ++j, ++n) {
            if (n > 0) wait(sm.c.summed, n - 1);
            wait(sm.c.scores, n);
            __syncwarp();
            tmem_after();
            if (busy) {
                const int32_t base = it.begin + j * kTokens;
                const bool edge = base + kTokens > all_hi || base < all_lo;
                const int32_t from = lo - base, to = max(from, hi - base);   // columns this row sees
                // Moves the reference where a row of the warp has outgrown it.
                auto follow = [&](float top) -> bool {
                    if (!__any_sync(0xFFFFFFFFu, top > ref + kSlack)) return false;
                    const float now = fmaxf(ref, top);
                    const float f = exp2_fast(ref - (now == -INFINITY ? 0.0f : now));
                    ref = now;
                    sum *= f;
                    if (j > 0) {
#pragma unroll 1
                        for (int q = 0; q < D / 16; ++q) {
                            float o[16];
                            tmem_load(t_sums + 16 * q, o);
                            tmem_wait_load();
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= f;
                            tmem_store16(t_sums + 16 * q, o);
                        }
                    }
                    return true;
                };
                // Behind the first tile the maximum is found together with the
                // weights, and these are made again where it had grown; where
                // they replace the scores it has to come first.
                const bool max_first = !L::kApart || j == 0;
                if (max_first) {
                    const Found f = edge ? row_pass<true, false>(t_scores, 0, from, to, c, 0.0f)
                                         : row_pass<false, false>(t_scores, 0, from, to, c, 0.0f);
                    follow(f.most * c);
                }
                Found f;
                do {
                    const float against = kShift - (ref == -INFINITY ? 0.0f : ref);
                    f = edge ? row_pass<true, true>(t_scores, t_weights, from, to, c, against)
                             : row_pass<false, true>(t_scores, t_weights, from, to, c, against);
                } while (!max_first && follow(f.most * c));
                const Pair add = pair_of(f.sum);
                sum += add.x + add.y;
                tmem_wait_store();
            }
            tmem_before();
            warp_arrive(sm.c.weights);
        }

        // ---- output ----------------------------------------------------------
        if (it.tiles > 0) {
            wait(sm.c.summed, n - 1);
            __syncwarp();
            tmem_after();
        }
        if (!busy) continue;
        float *part = part_at(a.workspace, 2 * static_cast<int64_t>(blockIdx.x) + max(it.part, 0), L::kPartFloats);
        const float inv = row_factor(sum, v_scale);
        uint4 *out = reinterpret_cast<uint4 *>(a.out + place.token * a.out_stride +
                                               static_cast<int64_t>(place.q_head) * D);
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
            float o[16];
            if (it.tiles > 0) {
                tmem_load(t_sums + 16 * q, o);
                tmem_wait_load();
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = 0.0f;
            }
            if (it.part >= 0) {                        // [dimensions / 4][rows]
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    reinterpret_cast<float4 *>(part)[(4 * q + i) * kRows + row] =
                        make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            } else if (live) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    out[2 * q + i] = make_uint4(bf16x2_of(o[8 * i] * inv, o[8 * i + 1] * inv),
                                                bf16x2_of(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                                bf16x2_of(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                                                bf16x2_of(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
            }
        }
        if (it.part >= 0) {
            part[kRows * D + row] = ref;
            part[kRows * D + kRows + row] = sum;
        } else if (live && a.lse != nullptr) {
            a.lse[static_cast<int64_t>(place.token) * a.q_heads + place.q_head] = row_lse(ref, sum, kShift);
        }
        tmem_before();                                 // the sums have been read
    }
}

// ---------------------------------------------------------------------------
// the kernel

// Moves registers between the warp groups of a block: with two blocks on an SM
// a thread starts with 80, and 112 + 72 + 56 are three times that.
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
    const int32_t warp = threadIdx.x / 32;
    const Division d = {a.q_heads / a.pools.heads, kRows, a.pools.heads, kTokens, a.window, whole};
    if (warp == 8)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n\t"
                     "tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;"
                     :: "r"(smem_addr(&c.tmem)), "n"(L::kColumns) : "memory");
    if (threadIdx.x == 0) {
        c.gave_up = 0;
        for (int i = 0; i < 2; ++i) {
            barrier_init(smem_addr(&c.item_full[i]), 1);
            barrier_init(smem_addr(&c.item_empty[i]), 9);    // eight warps and the issuing thread
        }
        barrier_init(smem_addr(&c.q_full), 4);
        barrier_init(smem_addr(&c.k_full), 4);
        barrier_init(smem_addr(&c.v_full), 4);
        barrier_init(smem_addr(&c.scores), 1);
        barrier_init(smem_addr(&c.weights), 4);
        barrier_init(smem_addr(&c.summed), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    pdl_allow_next();

    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    Split *record = static_cast<Split *>(a.workspace) + blockIdx.x;
    if (threadIdx.x == kThreads - 1) record->blocks = 0;
    tmem_before();
    const Run run = block_run<kThreads / 32>(a, d, &g_fp4_rows_error, c.plan);   // a block barrier at least
    tmem_after();
    const uint32_t tmem = c.tmem;
    const bool scales_ok = fp4_scale_ok(k_scale) && fp4_scale_ok(v_scale);
    if (!scales_ok && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_fp4_rows_error, kFp4ErrScale);
    if (scales_ok && run.at < run.end) {
        const Waits wait{c};
        if (warp < 4) {
            registers<L::kBlocks == 2, 112, true>();
            softmax_items<D>(a, sm, wait, tmem, d.group, k_scale, v_scale);
        } else if (warp < 8) {
            registers<L::kBlocks == 2, 72, false>();
            expand_items<D>(a, sm, wait);
        } else {
            registers<L::kBlocks == 2, 56, false>();
            if (threadIdx.x == 256)
                issue_items<D>(sm, wait, tmem);
            else if (warp == 9)
                walk_items(a, c, wait, run, d, record);
        }
    }
    __syncwarp();
    tmem_before();
    __syncthreads();
    if (*static_cast<volatile uint32_t *>(&c.gave_up)) __nanosleep(1000000);   // products under way end
    if (warp == 8) {
        tmem_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(L::kColumns));
    }
}

// Block (c, y) merges 8 dimensions of the item that began in block c, a row a
// thread.
template <int D>
__global__ void __launch_bounds__(kRows) fp4_attention_rows_join_kernel(const Fp4Attention a) {
    using L = Layout<D>;
    constexpr int kBatch = 4;
    pdl_wait();
    pdl_allow_next();
    const int32_t c = blockIdx.x, row = threadIdx.x;
    const Split s = static_cast<const Split *>(a.workspace)[c];
    if (row / 32 * 32 >= s.rows || s.blocks == 0) return;
    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    float top = -INFINITY, l = 0.0f, x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    for (int32_t i0 = 0; i0 < s.blocks; i0 += kBatch) {
        float t[kBatch], m[kBatch];
        float4 v[kBatch][2];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t i = i0 + k;
            t[k] = -INFINITY, m[k] = 0.0f;
            v[k][0] = v[k][1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < s.blocks) {
                // part 1 of block c, then part 0 of the blocks behind it
                const float *p = part_at(a.workspace, 2 * static_cast<int64_t>(c + i) + (i == 0 ? 1 : 0), L::kPartFloats);
                t[k] = p[kRows * D + row];
                m[k] = p[kRows * D + kRows + row];
                v[k][0] = reinterpret_cast<const float4 *>(p)[(2 * blockIdx.y) * kRows + row];
                v[k][1] = reinterpret_cast<const float4 *>(p)[(2 * blockIdx.y + 1) * kRows + row];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const float now = fmaxf(top, t[k]);
            const float base = now == -INFINITY ? 0.0f : now;
            const float f = exp2_fast(top - base), e = exp2_fast(t[k] - base);
            top = now;
            l = l * f + m[k] * e;
            const float w[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w,
                                v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * f + w[j] * e;
        }
    }
    if (row >= s.rows) return;
    const RowPlace place = row_place(s.token0, s.row0 + row, s.set, a.q_heads / a.pools.heads);
    const float inv = row_factor(l, v_scale);
    *reinterpret_cast<uint4 *>(a.out + place.token * a.out_stride + static_cast<int64_t>(place.q_head) * D +
                               8 * blockIdx.y) =
        make_uint4(bf16x2_of(x[0] * inv, x[1] * inv), bf16x2_of(x[2] * inv, x[3] * inv),
                   bf16x2_of(x[4] * inv, x[5] * inv), bf16x2_of(x[6] * inv, x[7] * inv));
    if (a.lse != nullptr && blockIdx.y == 0)
        a.lse[static_cast<int64_t>(place.token) * a.q_heads + place.q_head] = row_lse(top, l, kShift);
}

template <int D>
cudaError_t launch_dim(const Fp4Attention &a, cudaStream_t stream) {
    using L = Layout<D>;
    constexpr size_t kSmem = sizeof(Shared<D>) + 1024;
    static_assert(L::kBlocks * (kSmem + 1024) <= 228 * 1024, "the blocks of an SM fit its shared memory");
    auto kernel = fp4_attention_rows_kernel<D>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
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
    // Enough items to fill the blocks: none is split, and the parts (64 KB each
    // with 128 dimensions) and their join are saved.
    const bool whole = tiles * a.pools.heads >= grid + grid / 2;
    // Started on a free GPU, like the kernel for few rows.
    kernel<<<static_cast<unsigned>(grid), kThreads, kSmem, stream>>>(a, whole);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    g_launch_count.fetch_add(1, std::memory_order_relaxed);
    if (whole) return cudaSuccess;
    return launch_pdl(fp4_attention_rows_join_kernel<D>, dim3(static_cast<unsigned>(grid), D / 8), kRows, 0, stream, a);
}

}  // namespace

int64_t fp4_attention_rows_workspace(int32_t dim) {
    return kRecordBytes + static_cast<int64_t>(kMaxBlocks / 3) * (dim == 256 ? 1 : 2) * 2 * 4 * part_floats(kRows, dim);
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
