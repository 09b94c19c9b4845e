// fp4_attention.cu -- attention over a paged cache held in 4 bits, for few
// query rows to a KV head (sm_100a).
//
// For each new token and query head, over the cached tokens j it sees:
//     a_j = c q.k_j,  p_j = exp(a_j - max a),  out = sum p_j v_j / sum p_j
// in one pass with a running maximum and sum, in fp32.
//
// Bound by memory traffic for single tokens: 9/8 byte of cache a dimension of
// K and V, and 4 * group flops.  The 4-bit codes are expanded in registers
// and go straight into warp matrix instructions: through shared memory (which
// is where the 5th generation tensor cores take their operands from) each
// expanded fp16 tile would cost four times the bytes of the codes, written
// and read again, for eight rows of a 128-row tile.  Many rows to a KV head
// share the expanded tile: fp4_attention_rows.cu.
//
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T, so the cache
// fills the 16-row side of m16n8k16 and the few query rows its 8-column side.
// The sum index of a matrix product may be permuted freely when both operands
// agree, so each lane takes neighbouring codes: for K, dimensions
// [t D/4, (t+1) D/4) of two tokens; for V, the D/8 dimensions of one g and
// four neighbouring tokens (g = lane / 4, t = lane % 4).
//
// Operands are exact.  code * block scale has at most six significant bits in
// [2^-10, 2688]: exact in fp16.  A query row is scaled by a power of two so
// that its largest element lies in [2^8, 2^9): its bf16 elements are exact in
// fp16 down to 2^-22 of the largest, and the rest is off by 2^-33 of it.
// p is scaled by 2^15 and rounded to fp16 (off by at most 2^-11 of its value for
// p > 2^-29).
// The tensor scales enter in fp32, K's with the softmax scale and V's at the
// end.
//
// What a step of 32 tokens cannot do without is one conversion and one
// product for each pair of codes; the rest is kept off the four warps that do
// it.  A fifth warp looks up pages and copies tiles ahead of them, across the
// items of the block too, so that the next sequence's tokens are under way
// while this one's sums are finished.  Its copies have to be few: a lane's
// copies are issued one after the other.  So a block takes four, two or one
// heads at once, with one, two or four of its warps on each: the heads of a
// page lie side by side, and one copy takes all of them when a page is 16
// tokens, or 32 tokens of one when it is longer.  The running maximum is joined
// over lanes only when some lane sees a larger score.
//
// Measured, 256 sequences of 3001-6000 tokens x 4 heads of 128 (664 MB):
// 137 us with the join in a graph, 4.8 TB/s, and 155 in separate calls; of the
// kernel alone its copies would take 109 and its arithmetic 107 (158 us with a
// copy for each head).  One sequence of 200003 tokens 40 us, of which 9000 cycles
// pass before the first product and 6 us in the join.  The checks of large scores
// and of waits that gave up are 0.4 to 1.9 us of these and of the times below.
#include <cuda_runtime.h>

#include <cmath>

#include "fp4_async.cuh"
#include "fp4_plan.cuh"

namespace fp8q {

namespace {

__device__ uint32_t g_fp4_attention_error;

constexpr float kShift = 15.0f;        // p is held as p * 2^15
// Steps an item costs beside its own.  64 sequences of 1-8192 tokens and 32
// drafts: 35.0 and 39.0 us with none, 27.1 and 37.0 with one, 25.1 and 35.1 with four.
constexpr int kItemCost = 4;

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

using namespace fp4_plan;

constexpr int kWarps = 4;              // warps that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStep = 32;              // cached tokens of a warp's step

// The four computing warps meet.
__device__ __forceinline__ void meet() {
    asm volatile("bar.sync 1, %0;" :: "n"(32 * kWarps) : "memory");
}

__device__ __forceinline__ uint32_t low_twice(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t high_twice(uint32_t w) {
    uint32_t d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(d) : "r"(w));
    return d;
}

// What the copying warp tells the others about an item.
struct Item {
    int32_t rounds;             // steps of every warp in this block's part; -1: no more items
    int32_t begin, end, first;  // its cached tokens, and the first one any row sees
    int32_t ahead;              // query i sees tokens up to ahead + i
    int32_t token0, row0, rows;
    int32_t set;                // its heads: kHeads * set and on
    int32_t part;               // -1: the whole item, else which of the block's parts
};

// T warps share a head and take steps in turn; a block has 4 / T heads.
template <int D, int NT, int T>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kHeads = kWarps / T;
    static constexpr int kTile = 9 * D;                  // bytes of 16 tokens of a head
    static constexpr int kMTiles = D / 16;               // of O^T
    static constexpr int kOwn = kMTiles / T;             // ... that each warp finishes
    static constexpr int kUnit = kStep * T;              // cached tokens of a round
    static constexpr int kBlocks = NT * D <= 128 ? 3 : 2;   // an SM holds: by registers
    static constexpr int kStages = D == 64 ? 5 : D == 256 ? 2 : NT == 1 ? 3 : 4;
    static constexpr int kQBytes = kRows * 2 * D;        // query rows of a head
    static constexpr int kHeadFloats = static_cast<int>(part_floats(kRows, D));
    static constexpr int64_t kPartFloats = static_cast<int64_t>(kHeads) * kHeadFloats;
};

template <int D, int NT, int T>
struct Shared {
    using S = Shape<D, NT, T>;
    alignas(128) uint8_t ring[S::kStages][4 * kWarps * S::kTile];
    // the query rows as they are, then in place as matrix operands
    alignas(16) uint8_t q[2][S::kHeads][S::kQBytes];
    // what the other warps of a head leave for the one that finishes it
    alignas(16) float4 sums[T > 1 ? kWarps : 1][T > 1 ? T - 1 : 1][T > 1 ? S::kOwn * NT : 1][T > 1 ? 32 : 1];
    alignas(8) uint64_t full[S::kStages];
    uint64_t empty[S::kStages];
    uint64_t item_full[2];
    uint64_t item_empty[2];
    Item item[2];
    uint32_t gave_up;
    float top[kWarps][S::kRows];
    float sum[kWarps][S::kRows];
    PlanShared<kWarps + 1> plan;
};

// Where tile m (0, 1: K; 2, 3: V) of a head's step lies in a stage: heads side
// by side when a page is one tile, else the two tiles of a head.
template <int D, int NT, int T>
__device__ __forceinline__ int32_t stage_at(bool by_tile, int32_t step, int32_t m, int32_t head) {
    using S = Shape<D, NT, T>;
    const int32_t at = by_tile ? (4 * step + m) * S::kHeads + head
                               : ((2 * step + m / 2) * S::kHeads + head) * 2 + m % 2;
    return at * S::kTile;
}

// ---------------------------------------------------------------------------
// the copying warp

template <int D, int NT, int T>
__device__ __forceinline__ void copy_items(const Fp4Attention &a, Shared<D, NT, T> &sm, const Run &run,
                                           const Division &d, Split *record) {
    using S = Shape<D, NT, T>;
    constexpr int kHeads = S::kHeads;
    const int32_t lane = threadIdx.x % 32;
    uint32_t stage = 0, lap = 0, items = 0;

    // This lane's copy of a round: some tiles of a step of K or of V.
    const int32_t tiles = a.pools.tiles;
    const int32_t shift = (tiles & (tiles - 1)) == 0 ? __ffs(tiles) - 1 : -1;
    const bool by_tile = tiles == 1, by_pair = tiles % 2 == 0;
    int32_t step, m, head, copies;       // m: its first tile, as in stage_at
    if (by_tile) {                       // one tile of all heads
        copies = 4 * T;
        step = lane / 4, m = lane % 4, head = 0;
    } else if (by_pair) {                // two tiles of one head
        copies = 2 * kWarps;
        step = lane / (2 * kHeads), m = 2 * (lane / kHeads % 2), head = lane % kHeads;
    } else {                             // one tile of one head
        copies = 4 * kWarps;
        step = lane / (4 * kHeads), m = lane / kHeads % 4, head = lane % kHeads;
    }
    const uint8_t *pool = m < 2 ? a.pools.k : a.pools.v;

    Walk walk;
    walk.begin(d, run);
    for (;;) {
        const Tile x = tile_of(walk.s, d, walk.rt);
        const int64_t unit0 = walk.start + kItemCost;
        if (unit0 >= run.end) break;
        const int32_t r0 = static_cast<int32_t>(max(int64_t{0}, run.at - unit0));
        const int32_t r1 = static_cast<int32_t>(min(static_cast<int64_t>(x.units), run.end - unit0));
        if (r1 > r0) {
            Item it;
            it.begin = x.begin + r0 * S::kUnit;
            it.end = min(x.end, x.begin + r1 * S::kUnit);
            it.first = x.first;
            it.rounds = it.end > it.begin ? (it.end - it.begin + S::kUnit - 1) / S::kUnit : 0;
            it.ahead = walk.s.length - walk.s.news;
            it.token0 = walk.s.token0;
            it.row0 = x.row0;
            it.rows = x.rows;
            it.set = walk.set;
            it.part = r0 == 0 && r1 == x.units ? -1 : r0 == 0 ? 1 : 0;

            const int32_t *table = a.block_table + static_cast<int64_t>(walk.seq) * a.table_stride;
            // The first of this lane's tiles that holds a seen token, its page
            // and its place in the page; no page: nothing to copy.
            struct Place { int32_t tile, count; int64_t page; };
            auto look_up = [&](int32_t at) {
                Place p;
                const int32_t lo = max(at + 32 * step + 16 * (m % 2), it.first & ~15);
                const int32_t hi = min(it.end, at + 32 * step + 16 * (by_pair ? 2 : m % 2 + 1));
                p.count = lane < copies && lo < hi ? (hi - lo + 15) / 16 : 0;
                p.tile = 0;
                p.page = 0;
                if (p.count > 0) {
                    const int32_t at16 = lo / 16;
                    const int32_t page_at = shift >= 0 ? at16 >> shift : at16 / tiles;
                    p.tile = at16 - page_at * tiles;
                    p.page = table[page_at];
                }
                return p;
            };
            Place now = look_up(it.begin);

            const uint32_t slot = items % 2;
            if (items >= 2) barrier_wait(smem_addr(&sm.item_empty[slot]), (items / 2 - 1) & 1, &sm.gave_up, &g_fp4_attention_error);
            if (!told(&sm.gave_up)) return;
            if (lane == 0) {
                sm.item[slot] = it;
                if (it.part == 1) {
                    record->token0 = it.token0;
                    record->row0 = it.row0;
                    record->rows = it.rows;
                    record->set = it.set;
                    record->blocks = static_cast<int32_t>(quotient(unit0 + x.units - 1, run.per_block)) - blockIdx.x + 1;
                }
            }
            // The query rows, behind the first tiles: those take longer.  The
            // rows of one token and head lie side by side.
            auto copy_rows = [&]() {
                const uint32_t bar = smem_addr(&sm.item_full[slot]);
                if (lane == 0) barrier_expect(bar, kHeads * x.rows * 2 * D);
                __syncwarp();
                const int32_t q_lo = walk.s.news > 1 ? x.row0 / d.group : 0;
                for (int32_t i = lane / kHeads;; i += 32 / kHeads) {
                    const int32_t qi = q_lo + i, h = lane % kHeads;
                    const int32_t lo = max(x.row0, qi * d.group), hi = min(x.row0 + x.rows, (qi + 1) * d.group);
                    if (lo >= hi) break;
                    const uint16_t *src = a.q + (it.token0 + qi) * a.q_stride +
                        ((static_cast<int64_t>(it.set) * kHeads + h) * d.group + (lo - qi * d.group)) * D;
                    copy_async(smem_addr(sm.q[slot][h]) + (lo - x.row0) * 2 * D, src, (hi - lo) * 2 * D, bar);
                }
            };
            ++items;

            int32_t at = it.begin;
            for (int32_t r = 0; r < it.rounds; ++r, at += S::kUnit) {
                const Place next = look_up(at + S::kUnit);
                const uint32_t full = smem_addr(&sm.full[stage]);
                if (lap > 0) barrier_wait(smem_addr(&sm.empty[stage]), (lap - 1) & 1, &sm.gave_up, &g_fp4_attention_error);
                if (lane == 0) {
                    const int32_t lo = max(at, it.first & ~15), hi = min(it.end, at + S::kUnit);
                    barrier_expect(full, (hi > lo ? (hi - lo + 15) / 16 : 0) * 2 * kHeads * S::kTile);
                }
                __syncwarp();
                if (now.count > 0) {
                    if (now.page < 0 || now.page >= a.pools.num_blocks) {
                        atomicOr(&g_fp4_attention_error, kFp4ErrSlot);
                        now.page = 0;
                    }
                    const uint8_t *src = pool + now.page * a.pools.block_stride +
                        ((static_cast<int64_t>(it.set) * kHeads + head) * tiles + now.tile) * S::kTile;
                    // a pair that starts with its second tile
                    const int32_t skip = by_pair ? now.tile % 2 : 0;
                    const uint32_t dst = smem_addr(sm.ring[stage]) +
                        stage_at<D, NT, T>(by_tile, step, m, head) + skip * S::kTile;
                    copy_async(dst, src, now.count * (by_tile ? kHeads : 1) * S::kTile, full);
                }
                if (++stage == S::kStages) {
                    stage = 0, ++lap;
                    if (!told(&sm.gave_up)) return;
                }
                now = next;
                if (r == 0) copy_rows();
            }
            if (it.rounds == 0) copy_rows();
        }
        if (!walk.next(a, d, x.units + kItemCost)) break;
    }
    const uint32_t slot = items % 2;
    if (items >= 2) barrier_wait(smem_addr(&sm.item_empty[slot]), (items / 2 - 1) & 1, &sm.gave_up, &g_fp4_attention_error);
            if (!told(&sm.gave_up)) return;
    if (lane == 0) {
        sm.item[slot].rounds = -1;
        barrier_arrive(smem_addr(&sm.item_full[slot]));
    }
}

// ---------------------------------------------------------------------------
// the computing warps

// Turns a head's query rows into the right operand of S^T, in place, each of
// its T warps a share, and finds the factors that turn raw scores of this
// lane's columns into the log2 of a weight.
template <int D, int NT, int T>
__device__ __forceinline__ void prepare_rows(const Fp4Attention &a, int32_t rows, uint8_t *q, float k_scale,
                                             float (&c)[NT][2]) {
    using S = Shape<D, NT, T>;
    const int32_t share = threadIdx.x / 32 % T, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    static_assert(NT * (D / 32) * 512 == S::kQBytes, "the operands take the place of the rows");
    uint4 x[NT][D / 32];                   // dimensions [t D/4, (t + 1) D/4) of row g
    float scale[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const bool live = n * 8 + g < rows;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x[n][i] = make_uint4(0, 0, 0, 0);
            if (live)
                x[n][i] = *reinterpret_cast<const uint4 *>(q + (n * 8 + g) * 2 * D + t * (D / 2) + 16 * i);
        }
        uint32_t most = 0;                 // largest magnitude pattern
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const uint32_t w[4] = {x[n][i].x, x[n][i].y, x[n][i].z, x[n][i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                most = max(most, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
        }
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        const int32_t up = min(8 - (static_cast<int32_t>(most >> 7) - 127), 120);
        scale[n] = __int_as_float((127 + up) << 23);
        const float back = __int_as_float((127 - up) << 23);
        // A factor above zero keeps masked scores at -infinity; raw scores are
        // below 2^30, so one this small stands for zero.
        const float mine = fmaxf(a.softmax_scale * kLog2e * k_scale * back, 0x1p-100f);
#pragma unroll
        for (int j = 0; j < 2; ++j) c[n][j] = __shfl_sync(0xFFFFFFFFu, mine, 4 * (2 * t + j));
    }
    if (T > 1) meet();                     // every warp has read the rows
    else __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            if (i % T == share)
                reinterpret_cast<uint4 *>(q)[(i * NT + n) * 32 + lane] = make_uint4(
                    f16x2_of(bf16_low(x[n][i].x) * scale[n], bf16_high(x[n][i].x) * scale[n]),
                    f16x2_of(bf16_low(x[n][i].y) * scale[n], bf16_high(x[n][i].y) * scale[n]),
                    f16x2_of(bf16_low(x[n][i].z) * scale[n], bf16_high(x[n][i].z) * scale[n]),
                    f16x2_of(bf16_low(x[n][i].w) * scale[n], bf16_high(x[n][i].w) * scale[n]));
    if (T > 1) meet();
    else __syncwarp();
}

// Raw scores of 32 tokens: S^T = K Q^T.
template <int D, int NT>
__device__ __forceinline__ void score_step(const uint8_t *tile0, const uint8_t *tile1, const uint4 *rows,
                                           float (&sc)[2][NT][4]) {
    const int32_t lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int32_t tok = 4 * (g / 2) + (g % 2);     // this lane's rows of a tile: tok, tok + 2
    constexpr int kWords = D / 32;                 // code words of a lane's part of a row
    constexpr int kPairs = (D + 127) / 128;        // pairs of block scales
    uint32_t ca[2][kWords], cb[2][kWords], za[2][kPairs], zb[2][kPairs];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const uint8_t *kt = m ? tile1 : tile0;
        const uint8_t *ra = kt + tok * (D / 2) + t * (D / 8);
        const uint8_t *rb = ra + D;
        const uint8_t *sa = kt + 8 * D + tok * (D / 16) + t * (D / 64);
        const uint8_t *sb = sa + D / 8;
        if constexpr (D == 64) {
            const uint2 x = *reinterpret_cast<const uint2 *>(ra);
            const uint2 y = *reinterpret_cast<const uint2 *>(rb);
            ca[m][0] = x.x, ca[m][1] = x.y, cb[m][0] = y.x, cb[m][1] = y.y;
            za[m][0] = *sa, zb[m][0] = *sb;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 x = reinterpret_cast<const uint4 *>(ra)[i];
                const uint4 y = reinterpret_cast<const uint4 *>(rb)[i];
                ca[m][4 * i] = x.x, ca[m][4 * i + 1] = x.y, ca[m][4 * i + 2] = x.z, ca[m][4 * i + 3] = x.w;
                cb[m][4 * i] = y.x, cb[m][4 * i + 1] = y.y, cb[m][4 * i + 2] = y.z, cb[m][4 * i + 3] = y.w;
            }
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                za[m][i] = reinterpret_cast<const uint16_t *>(sa)[i];
                zb[m][i] = reinterpret_cast<const uint16_t *>(sb)[i];
            }
        }
#pragma unroll
        for (int i = 0; i < kPairs; ++i)
            za[m][i] = f16x2_of_e4m3x2(za[m][i]), zb[m][i] = f16x2_of_e4m3x2(zb[m][i]);
    }
#pragma unroll
    for (int w = 0; w < kWords; ++w) {             // eight dimensions of each lane, two k-steps
        uint4 q[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) q[n] = rows[(w * NT + n) * 32 + lane];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint32_t s_a = w / 2 % 2 ? high_twice(za[m][w / 4]) : low_twice(za[m][w / 4]);
            const uint32_t s_b = w / 2 % 2 ? high_twice(zb[m][w / 4]) : low_twice(zb[m][w / 4]);
            uint32_t xa[4], xb[4];
            f16x2_of_e2m1x8(ca[m][w], xa);
            f16x2_of_e2m1x8(cb[m][w], xb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xa[i] = mul_f16x2(xa[i], s_a);
                xb[i] = mul_f16x2(xb[i], s_b);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                if (w == 0)
                    mma_first(sc[m][n], xa[0], xb[0], xa[1], xb[1], q[n].x, q[n].y);
                else
                    mma(sc[m][n], xa[0], xb[0], xa[1], xb[1], q[n].x, q[n].y);
                mma(sc[m][n], xa[2], xb[2], xa[3], xb[3], q[n].z, q[n].w);
            }
        }
    }
}

// O^T += V^T P^T of 16 tokens; tokens outside [lo, hi) of the tile may hold
// any scale byte and count as zero.
template <int D, int NT, bool kEdge>
__device__ __forceinline__ void add_tile(const uint8_t *vt, int32_t lo, int32_t hi,
                                         const uint32_t (&pf)[NT][2], float (&o)[D / 16][NT][4]) {
    const int32_t lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    constexpr int kBlocksOfLane = D / 128 > 0 ? D / 128 : 1;   // with D = 64 two g share one
    constexpr int kWords = D == 64 ? 1 : 2;
#pragma unroll
    for (int blk = 0; blk < kBlocksOfLane; ++blk) {
        const int32_t block = D == 64 ? g / 2 : g * kBlocksOfLane + blk;
        uint32_t x[4][kWords];
        const uint8_t *p = vt + block * 128 + t * 32;
        if constexpr (kWords == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i][0] = *reinterpret_cast<const uint32_t *>(p + 8 * i + 4 * (g % 2));
        } else {
            const uint4 a = reinterpret_cast<const uint4 *>(p)[0];
            const uint4 b = reinterpret_cast<const uint4 *>(p)[1];
            x[0][0] = a.x, x[0][1] = a.y, x[1][0] = a.z, x[1][1] = a.w;
            x[2][0] = b.x, x[2][1] = b.y, x[3][0] = b.z, x[3][1] = b.w;
        }
        uint32_t z = *reinterpret_cast<const uint32_t *>(vt + 8 * D + block * 16 + 4 * t);
        if (kEdge) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * t + i < lo || 4 * t + i >= hi) z &= ~(0xFFu << (8 * i));
        }
        const uint32_t s01 = f16x2_of_e4m3x2(z & 0xFFFFu), s23 = f16x2_of_e4m3x2(z >> 16);
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            // pair the codes of neighbouring tokens, then expand
            uint32_t e01[4], o01[4], e23[4], o23[4];
            constexpr uint32_t kLow = 0x0F0F0F0Fu;
            f16x2_of_e2m1x8((x[0][w] & kLow) | ((x[1][w] << 4) & ~kLow), e01);
            f16x2_of_e2m1x8(((x[0][w] >> 4) & kLow) | (x[1][w] & ~kLow), o01);
            f16x2_of_e2m1x8((x[2][w] & kLow) | ((x[3][w] << 4) & ~kLow), e23);
            f16x2_of_e2m1x8(((x[2][w] >> 4) & kLow) | (x[3][w] & ~kLow), o23);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t a0 = mul_f16x2(e01[i], s01), a1 = mul_f16x2(o01[i], s01);
                const uint32_t a2 = mul_f16x2(e23[i], s23), a3 = mul_f16x2(o23[i], s23);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma(o[(blk * kWords + w) * 4 + i][n], a0, a1, a2, a3, pf[n][0], pf[n][1]);
            }
        }
    }
}

template <int D, int NT, int T>
__device__ __forceinline__ void compute_items(const Fp4Attention &a, Shared<D, NT, T> &sm, const Division &d,
                                              float k_scale, float v_scale) {
    using S = Shape<D, NT, T>;
    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t hh = warp / T, step = warp % T;  // this warp's head, and its steps of a round
    const int32_t g = lane / 4, t = lane % 4;
    const int32_t tok_a = 4 * (g / 2) + (g % 2);   // this lane's score rows: tok_a, tok_a + 2
    const bool by_tile = a.pools.tiles == 1;
    int32_t place[4];                              // of its tiles in a stage
#pragma unroll
    for (int m = 0; m < 4; ++m) place[m] = stage_at<D, NT, T>(by_tile, step, m, hh);
    uint32_t stage = 0, phase = 0;
    for (uint32_t items = 0;; ++items) {
        const uint32_t slot = items % 2;
        barrier_wait(smem_addr(&sm.item_full[slot]), (items / 2) & 1, &sm.gave_up, &g_fp4_attention_error);
        const Item &it = sm.item[slot];
        if (!(T > 1 ? agree(1, 32 * kWarps, told(&sm.gave_up)) : told(&sm.gave_up)) || it.rounds < 0) return;

        float c[NT][2];
        prepare_rows<D, NT, T>(a, it.rows, sm.q[slot][hh], k_scale, c);
        bool steps = false;                        // some row's weights are formed in steps
#pragma unroll
        for (int n = 0; n < NT; ++n) steps |= in_steps<D>(c[n][0]) || in_steps<D>(c[n][1]);
        steps = __any_sync(0xFFFFFFFFu, steps);
        const uint4 *rows = reinterpret_cast<const uint4 *>(sm.q[slot][hh]);
        float top[NT][2], ref[NT][2], sum[NT][2];  // ref: what scores are taken against
        float o[S::kMTiles][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 2; ++j) top[n][j] = -INFINITY, ref[n][j] = -kShift, sum[n][j] = 0.0f;
#pragma unroll
            for (int i = 0; i < S::kMTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][n][j] = 0.0f;
        }
        // every row sees the tokens in [all_lo, all_hi)
        const int32_t all_hi = min(it.end, it.ahead + it.row0 / d.group + 1);
        const int32_t all_lo =
            a.window > 0 ? max(0, it.ahead + (it.row0 + it.rows - 1) / d.group + 1 - a.window) : 0;
        int32_t at = it.begin + step * kStep;
        const int32_t rounds = it.rounds;

        for (int32_t r = 0; r < rounds; ++r, at += S::kUnit) {
            barrier_wait(smem_addr(&sm.full[stage]), phase, &sm.gave_up, &g_fp4_attention_error);
            const uint8_t *ring = sm.ring[stage];
            const bool edge = at + kStep > all_hi || at < all_lo;
            if (T == 1 || at < it.end) {

            float sc[2][NT][4];
            score_step<D, NT>(ring + place[0], ring + place[1], rows, sc);
            if (edge) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int32_t ci = it.ahead + (it.row0 + min(n * 8 + 2 * t + j, it.rows - 1)) / d.group + 1;
                        const int32_t hi = min(it.end, ci), lo = a.window > 0 ? ci - a.window : 0;
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const int32_t tok = at + 16 * m + tok_a + 2 * h;
                                if (tok >= hi || tok < lo) sc[m][n][2 * h + j] = -INFINITY;
                            }
                    }
            }

            // ---- running maximum and sum -------------------------------------
            float mx[NT][2];
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[n][j] = c[n][j] * fmaxf(fmaxf(sc[0][n][j], sc[0][n][2 + j]),
                                                 fmaxf(sc[1][n][j], sc[1][n][2 + j]));
                    grew |= mx[n][j] > top[n][j];
                }
            if (__any_sync(0xFFFFFFFFu, grew) || steps) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float shrink[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float m = mx[n][j];
#pragma unroll
                        for (int off = 4; off < 32; off *= 2)
                            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
                        const float now = fmaxf(top[n][j], m);
                        // a column that has seen nothing yet keeps exp2(-inf) = 0
                        const float base = now == -INFINITY ? 0.0f : now;
                        shrink[j] = exp2_fast(top[n][j] - base);
                        top[n][j] = now;
                        ref[n][j] = base - kShift;
                        sum[n][j] *= shrink[j];
                    }
#pragma unroll
                    for (int i = 0; i < S::kMTiles; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[i][n][j] *= shrink[j & 1];
                }
                if (steps) {
                    // Raw scores below the maximum's: what follows is the same for all
                    // rows.  1 / c times c is off by 2^-23, of a difference.
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            if (!in_steps<D>(c[n][j])) continue;
                            const float most = top[n][j] == -INFINITY ? 0.0f : top[n][j];
                            ref[n][j] = -kShift;
#pragma unroll
                            for (int m = 0; m < 2; ++m)
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    float &x = sc[m][n][2 * h + j];
                                    x = below_most(x, c[n][j], most) * __frcp_rn(c[n][j]);
                                }
                        }
                }
            }
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float &x = sc[m][n][j];
                        x = exp2_fast(fmaf(x, c[n][j % 2], -ref[n][j % 2]));
                        sum[n][j % 2] += x;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        pf[m][n][h] = transpose8x8(f16x2_of(sc[m][n][2 * h], sc[m][n][2 * h + 1]));
                }

            // ---- O^T += V^T P^T ----------------------------------------------
            if (edge) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    add_tile<D, NT, true>(ring + place[2 + m], it.first - (at + 16 * m),
                                          it.end - (at + 16 * m), pf[m], o);
            } else {
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    add_tile<D, NT, false>(ring + place[2 + m], 0, 16, pf[m], o);
            }
            }
            __syncwarp();                      // every lane has read the stage
            if (lane == 0) barrier_arrive(smem_addr(&sm.empty[stage]));
            if (++stage == S::kStages) stage = 0, phase ^= 1;
        }

        // ---- join the warps of a head -------------------------------------------
        const int32_t busy = min(T, max(1, (it.end - it.begin + kStep - 1) / kStep));   // that had a step
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int off = 4; off < 32; off *= 2)
                    sum[n][j] += __shfl_xor_sync(0xFFFFFFFFu, sum[n][j], off);
        if (T > 1) {
            if (step < busy) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    if (g == 0) {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            sm.top[warp][n * 8 + 2 * t + j] = top[n][j];
                            sm.sum[warp][n * 8 + 2 * t + j] = sum[n][j];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < S::kMTiles; ++i) {
                        const int owner = i / S::kOwn;
                        if (owner != step)
                            sm.sums[hh * T + owner][step - (step > owner)][i % S::kOwn * NT + n][lane] =
                                make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
                    }
                }
            }
            meet();
        }
        // Each of its warps finishes a share of the dimensions.
        const int32_t head = it.set * S::kHeads + hh;
        float *part = part_at(a.workspace, 2 * static_cast<int64_t>(blockIdx.x) + max(it.part, 0), S::kPartFloats) +
                      hh * S::kHeadFloats;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[T][2], most[2], l[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                most[j] = top[n][j], l[j] = sum[n][j], f[0][j] = 1.0f;
                if (T > 1) {
                    const int32_t col = n * 8 + 2 * t + j;
                    most[j] = -INFINITY;
                    for (int w = 0; w < busy; ++w) most[j] = fmaxf(most[j], sm.top[hh * T + w][col]);
                    const float base = most[j] == -INFINITY ? 0.0f : most[j];
                    l[j] = 0.0f;
#pragma unroll
                    for (int w = 0; w < T; ++w) {
                        f[w][j] = w < busy ? exp2_fast(sm.top[hh * T + w][col] - base) : 0.0f;
                        if (w < busy) l[j] += f[w][j] * sm.sum[hh * T + w][col];
                    }
                }
            }
            const float inv[2] = {row_factor(l[0], v_scale), row_factor(l[1], v_scale)};
            uint32_t packed[2][S::kOwn];       // rounded pairs of dimensions, by row
#pragma unroll
            for (int ii = 0; ii < S::kOwn; ++ii) {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = o[ii][n][j];
#pragma unroll
                    for (int w = 1; w < T; ++w) x[j] = step == w ? o[w * S::kOwn + ii][n][j] : x[j];
                }
                if (T > 1) {
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int w = 0; w < T; ++w)
                        if (w < busy) {
                            const float4 v = w == step ? make_float4(x[0], x[1], x[2], x[3])
                                                       : sm.sums[warp][w - (w > step)][ii * NT + n][lane];
                            y[0] += f[w][0] * v.x, y[1] += f[w][1] * v.y;
                            y[2] += f[w][0] * v.z, y[3] += f[w][1] * v.w;
                        }
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[j] = y[j];
                }
                if (it.part >= 0)
                    reinterpret_cast<float4 *>(part)[((step * S::kOwn + ii) * NT + n) * 32 + lane] =
                        make_float4(x[0], x[1], x[2], x[3]);
                packed[0][ii] = bf16x2_of(x[0] * inv[0], x[2] * inv[0]);
                packed[1][ii] = bf16x2_of(x[1] * inv[1], x[3] * inv[1]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int32_t row = n * 8 + 2 * t + j;
                if (it.part >= 0) {
                    if (step == 0 && g == 0) {
                        part[S::kRows * D + row] = most[j];
                        part[S::kRows * D + S::kRows + row] = l[j];
                    }
                } else if (row < it.rows) {
                    const RowPlace p = row_place(it.token0, it.row0 + row, head, d.group);
                    uint16_t *out = a.out + p.token * a.out_stride + static_cast<int64_t>(p.q_head) * D +
                                    g * (D / 8) + step * S::kOwn * 2;
                    if constexpr (S::kOwn % 4 == 0) {
#pragma unroll
                        for (int i = 0; i < S::kOwn; i += 4)
                            *reinterpret_cast<uint4 *>(out + 2 * i) = make_uint4(
                                packed[j][i], packed[j][i + 1], packed[j][i + 2], packed[j][i + 3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < S::kOwn; ++i) *reinterpret_cast<uint32_t *>(out + 2 * i) = packed[j][i];
                    }
                    if (a.lse != nullptr && step == 0 && g == 0)
                        a.lse[static_cast<int64_t>(p.token) * a.q_heads + p.q_head] = row_lse(most[j], l[j], kShift);
                }
            }
        }
        // the operands were plain writes, and copies take their place
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (T > 1) meet();                     // the sums may be written again
        else __syncwarp();
        if (lane == 0) barrier_arrive(smem_addr(&sm.item_empty[slot]));
    }
}

template <int D, int NT, int T>
__device__ __forceinline__ Division division(const Fp4Attention &a) {
    using S = Shape<D, NT, T>;
    return {a.q_heads / a.pools.heads, S::kRows, a.pools.heads / S::kHeads, S::kUnit, kItemCost, a.window, 0};
}

template <int D, int NT, int T>
__global__ void __launch_bounds__(kThreads, (Shape<D, NT, T>::kBlocks)) fp4_attention_kernel(const Fp4Attention a) {
    using S = Shape<D, NT, T>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Shared<D, NT, T> &sm = *reinterpret_cast<Shared<D, NT, T> *>(smem_raw);
    const Division d = division<D, NT, T>(a);

    if (threadIdx.x < S::kStages) {
        barrier_init(smem_addr(&sm.full[threadIdx.x]), 1);
        barrier_init(smem_addr(&sm.empty[threadIdx.x]), kWarps);
    }
    if (threadIdx.x == 0) sm.gave_up = 0;
    if (threadIdx.x < 2) {
        barrier_init(smem_addr(&sm.item_full[threadIdx.x]), 1);
        barrier_init(smem_addr(&sm.item_empty[threadIdx.x]), kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();                                // nothing to wait for: not launched early
    pdl_allow_next();

    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    Split *record = static_cast<Split *>(a.workspace) + blockIdx.x;
    if (threadIdx.x == 32 * kWarps) record->blocks = 0;
    const Run run = block_run<kWarps + 1>(a, d, &g_fp4_attention_error, sm.plan);
    if (!fp4_scale_ok(k_scale) || !fp4_scale_ok(v_scale)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_fp4_attention_error, kFp4ErrScale);
        return;
    }
    if (run.at >= run.end) return;             // the whole block
    if (threadIdx.x >= 32 * kWarps)
        copy_items<D, NT, T>(a, sm, run, d, record);
    else
        compute_items<D, NT, T>(a, sm, d, k_scale, v_scale);
    let_land(&sm.gave_up);
}

// ---------------------------------------------------------------------------
// the join

// Two columns of a fragment, divided by their sums and stored.
template <int D>
__device__ __forceinline__ void store_joined(const Fp4Attention &a, const Split &s, int32_t head, int32_t i,
                                             int32_t col, const float (&x)[4], const float (&top)[2],
                                             const float (&l)[2], float v_scale) {
    const int32_t lane = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int32_t row = col + j;
        if (row >= s.rows) continue;
        const RowPlace p = row_place(s.token0, s.row0 + row, head, a.q_heads / a.pools.heads);
        const float inv = row_factor(l[j], v_scale);
        *reinterpret_cast<uint32_t *>(a.out + p.token * a.out_stride + static_cast<int64_t>(p.q_head) * D +
                                      (lane / 4) * (D / 8) + 2 * i) = bf16x2_of(x[j] * inv, x[2 + j] * inv);
        if (a.lse != nullptr && i == 0 && lane < 4)
            a.lse[static_cast<int64_t>(p.token) * a.q_heads + p.q_head] = row_lse(top[j], l[j], kShift);
    }
}

// Part i of the item that began in block c: part 1 of that block, then part 0
// of the blocks behind it.
template <int D, int NT, int T>
__device__ __forceinline__ const float *joined_part(const Fp4Attention &a, int32_t c, int32_t i, int32_t hh) {
    using S = Shape<D, NT, T>;
    return part_at(a.workspace, 2 * static_cast<int64_t>(c + i) + (i == 0 ? 1 : 0), S::kPartFloats) +
           hh * S::kHeadFloats;
}

constexpr int kJoinThreads = 256;
constexpr int kJoinSlots = 12;
constexpr int kJoinRefill = 4;          // slots filled again at once

// Block (c, hh) merges head hh of the item that began in block c, its parts met
// once with a running maximum like the tokens were.  An item has two or three
// of them as a rule and dozens where one sequence is much longer than the rest;
// fetching them costs one latency for twelve, without holding registers that
// would keep other blocks away.
template <int D, int NT, int T>
__global__ void __launch_bounds__(kJoinThreads) fp4_attention_join_kernel(const Fp4Attention a) {
    using S = Shape<D, NT, T>;
    constexpr int kRows = S::kRows, kUnits = S::kMTiles * NT, kWarpsHere = kJoinThreads / 32;
    constexpr int kMine = (kUnits + kWarpsHere - 1) / kWarpsHere;   // fragments of a warp
    extern __shared__ __align__(128) uint8_t smem_raw[];
    float (&slots)[kJoinSlots][S::kHeadFloats] = *reinterpret_cast<float (*)[kJoinSlots][S::kHeadFloats]>(smem_raw);
    __shared__ alignas(8) uint64_t full[kJoinSlots];
    __shared__ uint32_t gave_up;
    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x < kJoinSlots) barrier_init(smem_addr(&full[threadIdx.x]), 1);
    if (threadIdx.x == 0) gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    pdl_wait();
    pdl_allow_next();
    const int32_t c = blockIdx.x, hh = blockIdx.y;
    const Split s = static_cast<const Split *>(a.workspace)[c];
    if (s.blocks == 0) return;
    auto fetch = [&](int32_t i) {
        const uint32_t bar = smem_addr(&full[i % kJoinSlots]);
        barrier_expect(bar, S::kHeadFloats * 4);
        copy_async(smem_addr(slots[i % kJoinSlots]), joined_part<D, NT, T>(a, c, i, hh), S::kHeadFloats * 4, bar);
    };
    if (threadIdx.x == 0)
        for (int32_t i = 0; i < kJoinSlots && i < s.blocks; ++i) fetch(i);
    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    float top[kMine][2], l[kMine][2], x[kMine][4];
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
#pragma unroll
        for (int j = 0; j < 2; ++j) top[m][j] = -INFINITY, l[m][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) x[m][j] = 0.0f;
    }
    for (int32_t i = 0; i < s.blocks; ++i) {
        barrier_wait(smem_addr(&full[i % kJoinSlots]), (i / kJoinSlots) & 1, &gave_up, &g_fp4_attention_error);
        const float *p = slots[i % kJoinSlots];
#pragma unroll
        for (int m = 0; m < kMine; ++m) {
            const int32_t unit = warp + m * kWarpsHere;    // i * NT + n
            if (unit >= kUnits) continue;
            const int32_t col = (unit % NT) * 8 + 2 * (lane % 4);
            const float2 t = *reinterpret_cast<const float2 *>(p + kRows * D + col);
            const float2 n = *reinterpret_cast<const float2 *>(p + kRows * D + kRows + col);
            const float4 v = reinterpret_cast<const float4 *>(p)[unit * 32 + lane];
            const float tt[2] = {t.x, t.y}, nn[2] = {n.x, n.y}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float now = fmaxf(top[m][j], tt[j]);
                const float base = now == -INFINITY ? 0.0f : now;
                const float f = exp2_fast(top[m][j] - base), e = exp2_fast(tt[j] - base);
                top[m][j] = now;
                l[m][j] = l[m][j] * f + nn[j] * e;
                x[m][j] = x[m][j] * f + vv[j] * e;
                x[m][2 + j] = x[m][2 + j] * f + vv[2 + j] * e;
            }
        }
        if (i % kJoinRefill == kJoinRefill - 1 && i + 1 + kJoinSlots - kJoinRefill < s.blocks) {
            __syncthreads();                   // everybody has read the slots
            if (threadIdx.x == 0 && *static_cast<volatile uint32_t *>(&gave_up) == 0)
                for (int32_t k = i + 1 + kJoinSlots - kJoinRefill; k <= i + kJoinSlots && k < s.blocks; ++k) fetch(k);
        }
    }
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
        const int32_t unit = warp + m * kWarpsHere;
        if (unit < kUnits)
            store_joined<D>(a, s, s.set * S::kHeads + hh, unit / NT, (unit % NT) * 8 + 2 * (lane % 4), x[m],
                            top[m], l[m], v_scale);
    }
    let_land(&gave_up);
}

constexpr int kFewWarps = 16;

// With few items each has many parts: block (c, y) merges fragment y of the
// c-th item that is split, every warp some of the parts.  The maxima come first,
// all at once, so that the sums wait for nothing but their own loads.
template <int D, int NT, int T>
__global__ void __launch_bounds__(32 * kFewWarps) fp4_attention_join_few_kernel(const Fp4Attention a,
                                                                                int32_t blocks) {
    using S = Shape<D, NT, T>;
    constexpr int kRows = S::kRows, kUnits = S::kMTiles * NT;
    constexpr int kTop = (kMaxBlocks * 8 + 32 * kFewWarps - 1) / (32 * kFewWarps);   // maxima a thread loads
    constexpr int kBatch = 14;                 // sums under way
    __shared__ float weight[kMaxBlocks][8];    // 2^(top of the part - top)
    __shared__ float over_warps[kFewWarps][8];
    __shared__ float4 share[kFewWarps][32];
    __shared__ int32_t found;
    pdl_wait();
    pdl_allow_next();
    const Split *records = static_cast<const Split *>(a.workspace);
    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (warp == 0) {
        constexpr int kTurns = (kMaxBlocks + 31) / 32;
        int32_t mine = -1, before = 0;
        uint32_t those[kTurns];
#pragma unroll
        for (int k = 0; k < kTurns; ++k)
            those[k] = 32 * k + lane < blocks ? records[32 * k + lane].blocks : 0;
#pragma unroll
        for (int k = 0; k < kTurns; ++k) {
            those[k] = __ballot_sync(0xFFFFFFFFu, those[k] != 0);
            const int32_t n = __popc(those[k]), c = blockIdx.x;
            if (c >= before && c < before + n) mine = 32 * k + __fns(those[k], 0, c - before + 1);
            before += n;
        }
        if (lane == 0) found = mine;
    }
    __syncthreads();
    if (found < 0) return;
    const int32_t c = found;
    const Split s = records[c];
    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    const int32_t hh = blockIdx.y / kUnits, unit = blockIdx.y % kUnits;   // unit: i * NT + n
    const int32_t n8 = unit % NT * 8;          // its rows

    // Thread: row threadIdx.x % 8 of every 64th part.
    const int32_t row = n8 + threadIdx.x % 8;
    float t[kTop], n[kTop];
#pragma unroll
    for (int k = 0; k < kTop; ++k) {
        const int32_t i = threadIdx.x / 8 + k * (4 * kFewWarps);
        t[k] = -INFINITY, n[k] = 0.0f;
        if (i < s.blocks) {
            const float *p = joined_part<D, NT, T>(a, c, i, hh);
            t[k] = p[kRows * D + row];
            n[k] = p[kRows * D + kRows + row];
        }
    }
    auto over_rows = [&](float v, bool is_max) {
        for (int o = 8; o < 32; o *= 2) {
            const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
            v = is_max ? fmaxf(v, w) : v + w;
        }
        __syncthreads();
        if (lane < 8) over_warps[warp][lane] = v;
        __syncthreads();
        v = over_warps[0][threadIdx.x % 8];
        for (int w = 1; w < kFewWarps; ++w)
            v = is_max ? fmaxf(v, over_warps[w][threadIdx.x % 8]) : v + over_warps[w][threadIdx.x % 8];
        return v;
    };
    float most = -INFINITY, l = 0.0f;
#pragma unroll
    for (int k = 0; k < kTop; ++k) most = fmaxf(most, t[k]);
    most = over_rows(most, true);
    const float base = most == -INFINITY ? 0.0f : most;
#pragma unroll
    for (int k = 0; k < kTop; ++k) {
        const int32_t i = threadIdx.x / 8 + k * (4 * kFewWarps);
        const float f = exp2_fast(t[k] - base);
        if (i < s.blocks) weight[i][threadIdx.x % 8] = f;
        l += f * n[k];
    }
    l = over_rows(l, false);

    const int32_t col = 2 * (lane % 4);
    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int32_t i0 = warp; i0 < s.blocks; i0 += kFewWarps * kBatch) {
        float4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t i = i0 + k * kFewWarps;
            v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (i < s.blocks) v[k] = reinterpret_cast<const float4 *>(joined_part<D, NT, T>(a, c, i, hh))[unit * 32 + lane];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t i = i0 + k * kFewWarps;
            if (i < s.blocks) {
                const float f0 = weight[i][col], f1 = weight[i][col + 1];
                x[0] += f0 * v[k].x, x[1] += f1 * v[k].y, x[2] += f0 * v[k].z, x[3] += f1 * v[k].w;
            }
        }
    }
    share[warp][lane] = make_float4(x[0], x[1], x[2], x[3]);
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < kFewWarps; ++w) {
        const float4 v = share[w][lane];
        x[0] += v.x, x[1] += v.y, x[2] += v.z, x[3] += v.w;
    }
    // lane j of the warp holds row j % 8
    const float tops[2] = {__shfl_sync(0xFFFFFFFFu, most, col), __shfl_sync(0xFFFFFFFFu, most, col + 1)};
    const float sums[2] = {__shfl_sync(0xFFFFFFFFu, l, col), __shfl_sync(0xFFFFFFFFu, l, col + 1)};
    store_joined<D>(a, s, s.set * S::kHeads + hh, unit / NT, n8 + col, x, tops, sums, v_scale);
}

// ---------------------------------------------------------------------------
// launch

// Rows of a tile (8 * NT) for an average of `rows` rows a sequence: the
// smallest tile that holds them, up to what the accumulators leave room for
// in registers (NT * D <= 256; 24 rows of 128 spilled, and took 60 us for 32
// drafts of 5 to 40 rows where 16 rows at a time take 36).
int tiles_of(int64_t batch, int64_t num_tokens, int32_t group, int32_t dim) {
    const int64_t rows = (num_tokens + batch - 1) / batch * group;
    return rows <= 8 || dim == 256 ? 1 : 2;
}

// Sets of four heads with their row tiles, at least: below 32 no block takes
// four heads at once, whatever the lengths.
int64_t fours_of(int64_t batch, int64_t num_tokens, int32_t group, int32_t kv_heads, int32_t rows) {
    if (kv_heads % 4 != 0) return 0;
    const int64_t tiles = (num_tokens * group + rows - 1) / rows;
    return (tiles > batch ? tiles : batch) * (kv_heads / 4);
}
constexpr int64_t kFewFours = 32;

// Warps of a head: a block takes as many of two heads as divide their number,
// and four where the blocks' runs can be long.  Four heads in one copy read
// faster, and leave twice the parts to join.  The lengths are on the device, so
// the table's width stands for them: steps of a block are counted as if every
// sequence filled its table, and a table padded to the longest context takes four
// heads from 32 sequences on.  Measured with 4 heads of 128, four heads against
// two: 48 sequences of 3000-6000 tokens (20 steps of a block) 41.2 and 40.4 us, 64
// (27) 47.9 and 49.4, 96 (41) 60.6 and 63.9, 160 (68) 88.7 and 95.1; spread over
// 1-8192 tokens, where the parts count for more, 64 (35) 30.8 and 26.7, 96 (53)
// 31.8 and 30.0, 128 (71) 31.2 and 29.4; with rows for two tiles, 8 heads and
// 100-4000 tokens, 16 drafts (19) 39.4 and 39.4, 32 (38) 52.5 and 55.5.
int warps_of_head(const Fp4Attention &a, int32_t rows) {
    const int32_t heads = a.pools.heads;
    const int64_t fours = fours_of(a.batch, a.num_tokens, a.q_heads / heads, heads, rows);
    const int64_t blocks = kMaxBlocks / 3 * (rows * a.pools.dim <= 1024 ? 3 : 2);
    const int64_t steps = a.table_width * a.pools.tiles / 2;
    if (fours >= kFewFours && fours * steps >= (rows == 8 ? 40 : 32) * blocks) return 1;
    return heads % 2 == 0 ? 2 : 4;
}

template <int D, int NT, int T>
cudaError_t launch_tiles(const Fp4Attention &a, cudaStream_t stream) {
    using S = Shape<D, NT, T>;
    constexpr size_t kSmem = sizeof(Shared<D, NT, T>);
    static_assert(S::kBlocks * (kSmem + 1024) <= 228 * 1024, "the blocks of an SM fit its shared memory");
    auto kernel = fp4_attention_kernel<D, NT, T>;
    int sms = 0;
    cudaError_t e = device_sms(&sms);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    // No more blocks than there can be points on the axis.
    const int32_t group = a.q_heads / a.pools.heads;
    const int64_t items = ((static_cast<int64_t>(a.num_tokens) * group + S::kRows - 1) / S::kRows + a.batch) *
                          (a.pools.heads / S::kHeads);
    const int64_t longest = a.table_width * a.pools.tiles * 16 / S::kUnit + 2 + kItemCost;
    int64_t grid = static_cast<int64_t>(sms) * S::kBlocks;
    if (grid > kMaxBlocks / 3 * S::kBlocks) grid = kMaxBlocks / 3 * S::kBlocks;
    if (items < grid && items * longest < grid) grid = items * longest;
    // Started only when the GPU is free: blocks placed beside those of another
    // kernel found SMs set up for less shared memory, and the last third of them
    // ran behind the others (256 sequences of 3001-6000 tokens: 171 us, not 131).
    kernel<<<static_cast<unsigned>(grid), kThreads, kSmem, stream>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    g_launch_count.fetch_add(1, std::memory_order_relaxed);
    if (items * 8 <= sms && items < grid) {    // few items, and with them many parts of each
        fp4_attention_join_few_kernel<D, NT, T>
            <<<dim3(static_cast<unsigned>(items), S::kHeads * S::kMTiles * NT), 32 * kFewWarps, 0, stream>>>(
                a, static_cast<int32_t>(grid));
        e = cudaGetLastError();
        if (e == cudaSuccess) g_launch_count.fetch_add(1, std::memory_order_relaxed);
        return e;
    }
    constexpr size_t kJoinSmem = kJoinSlots * S::kHeadFloats * 4;
    if constexpr (kJoinSmem > 48 * 1024) {
        e = cudaFuncSetAttribute(fp4_attention_join_kernel<D, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kJoinSmem));
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(fp4_attention_join_kernel<D, NT, T>, dim3(static_cast<unsigned>(grid), S::kHeads),
                      kJoinThreads, kJoinSmem, stream, a);
}

template <int D, int NT>
cudaError_t launch_heads(const Fp4Attention &a, cudaStream_t stream) {
    const int t = warps_of_head(a, 8 * NT);
    return t == 1 ? launch_tiles<D, NT, 1>(a, stream)
           : t == 2 ? launch_tiles<D, NT, 2>(a, stream) : launch_tiles<D, NT, 4>(a, stream);
}

}  // namespace

// More than 32 rows a sequence on average: their tiles are shared.  Measured
// with 32 sequences of 1000-3000 tokens and 8 heads of 64 and 128, this kernel
// against the one by rows: 30 rows 42 and 61 us against 53 and 72; 35 rows
// (three tiles) 55 and 83 against 56 and 77; 60 rows 62 and 100 against 54 and
// 75.  With 256, 30 rows 201 and 330 against 329 and 462, 40 rows 300 and 489
// against 365 and 500.  The average is all that sizes tell: in a call of pieces of
// prompts and single tokens each is in the other's kernel.  64 single tokens on
// 3000-6000 and a piece of 512 on 4096 (4 heads of 128, 8 rows a token) take 182 us
// together, 47 and 75 in calls of their own.
bool fp4_attention_by_rows(int64_t batch, int64_t num_tokens, int32_t group) {
    return num_tokens * group > 32 * batch;
}

int64_t fp4_attention_workspace(int64_t batch, int64_t num_tokens, int32_t q_heads,
                                int32_t kv_heads, int32_t dim, bool uneven) {
    if (batch == 0) return 0;
    if (fp4_attention_by_rows(batch, num_tokens, q_heads / kv_heads)) return fp4_attention_rows_workspace(num_tokens, q_heads / kv_heads, kv_heads, dim, uneven);
    const int rows = 8 * tiles_of(batch, num_tokens, q_heads / kv_heads, dim);
    const int64_t blocks = rows * dim <= 1024 ? kMaxBlocks : kMaxBlocks / 3 * 2;   // as Shape::kBlocks
    const int heads = fours_of(batch, num_tokens, q_heads / kv_heads, kv_heads, rows) >= kFewFours ? 4
                      : kv_heads % 2 == 0 ? 2 : 1;     // of a block, at most
    return kRecordBytes + blocks * 2 * 4 * heads * part_floats(rows, dim);
}

cudaError_t launch_fp4_attention(const Fp4Attention &a, cudaStream_t stream) {
    if (fp4_attention_by_rows(a.batch, a.num_tokens, a.q_heads / a.pools.heads))
        return launch_fp4_attention_rows(a, stream);
    const int nt = tiles_of(a.batch, a.num_tokens, a.q_heads / a.pools.heads, a.pools.dim);
    switch (a.pools.dim) {
    case 64: return nt == 1 ? launch_heads<64, 1>(a, stream) : launch_heads<64, 2>(a, stream);
    case 128: return nt == 1 ? launch_heads<128, 1>(a, stream) : launch_heads<128, 2>(a, stream);
    default: return launch_heads<256, 1>(a, stream);
    }
}

cudaError_t read_fp4_attention_error(uint32_t *bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_fp4_attention_error, sizeof(uint32_t));
    if (e == cudaSuccess && clear) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_fp4_attention_error, &zero, sizeof(uint32_t));
    }
    return e;
}

}  // namespace fp8q
