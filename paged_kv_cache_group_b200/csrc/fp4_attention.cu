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
// p is scaled by 2^15 and rounded to fp16 (2^-12 of its value for p > 2^-29).
// The tensor scales enter in fp32, K's with the softmax scale and V's at the
// end.
//
// What a step of 32 tokens cannot do without is one conversion and one
// product for each pair of codes; the rest is kept off the four warps that do
// it.  A fifth warp looks up pages and copies tiles ahead of them, across the
// items of the block too, so that the next sequence's tokens are under way
// while this one's sums are finished.  The running maximum is joined over
// lanes only when some lane sees a larger score.
#include <cuda_runtime.h>

#include <cmath>

#include "fp4_device.cuh"
#include "fp4_plan.cuh"

namespace fp8q {

namespace {

__device__ uint32_t g_fp4_attention_error;

constexpr int kWaitTries = 1 << 20;    // polls of a barrier before giving up
constexpr float kShift = 15.0f;        // p is held as p * 2^15
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void barrier_init(uint32_t bar, uint32_t arrivals) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(arrivals) : "memory");
}

__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;"
                 :: "r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool barrier_done(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

__device__ __forceinline__ void copy_async(uint32_t dst, const void *src, uint32_t bytes,
                                           uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1], %2, [%3];" :: "r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

using namespace fp4_plan;

constexpr int kWarps = 4;              // warps that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kStep = 32;              // cached tokens of a warp's step
static_assert(kStep * kWarps == kUnit, "a unit is one step of every warp");

__device__ __forceinline__ void barrier_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
}

// Waits for a phase of a barrier.  Gives up after a bounded number of polls,
// and once a block has done so, after a few: its output is not valid then.
__device__ __forceinline__ void barrier_wait(uint32_t bar, uint32_t parity, volatile uint32_t *gave_up) {
    for (int32_t tries = 0; !barrier_done(bar, parity); ++tries)
        if (tries > kWaitTries || (tries > 1000 && *gave_up)) {
            *gave_up = 1;
            atomicOr(&g_fp4_attention_error, kFp4ErrWait);
            break;
        }
}

// The four computing warps meet.
__device__ __forceinline__ void meet() {
    asm volatile("bar.sync 1, %0;" :: "n"(32 * kWarps) : "memory");
}

__device__ __forceinline__ void load_scales(const Fp4Attention &a, float *ks, float *vs) {
    *ks = a.pools.scale_dev ? a.pools.scale_dev[0] : a.pools.k_scale;
    *vs = a.pools.scale_dev ? a.pools.scale_dev[1] : a.pools.v_scale;
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
    int32_t steps;              // 32-token steps of this block's part; -1: no more items
    int32_t begin, end, first;  // its cached tokens, and the first one any row sees
    int32_t ahead;              // query i sees tokens up to ahead + i
    int32_t token0, row0, rows, head;
    int32_t part;               // -1: the whole item, else which of the block's parts
};

template <int D, int NT>
struct Shape {
    static constexpr int kRows = 8 * NT;
    static constexpr int kTile = 9 * D;                  // bytes of 16 tokens of a head
    static constexpr int kMTiles = D / 16;               // of O^T
    static constexpr int kBlocks = NT * D <= 128 ? 3 : 2;   // an SM holds: by registers
    static constexpr int kStages = D == 64 ? 5 : D == 128 ? 3 : 2;
    static constexpr int kQPitch = 2 * D + 16;           // bytes: rows start in other banks
};

template <int D, int NT>
struct Shared {
    using S = Shape<D, NT>;
    alignas(128) uint8_t ring[kWarps][S::kStages][4 * S::kTile];   // K, K, V, V
    alignas(16) float4 sums[kWarps][S::kMTiles * NT][32];
    alignas(16) uint8_t q[2][S::kRows][S::kQPitch];
    alignas(8) uint64_t full[kWarps][S::kStages];
    uint64_t empty[kWarps][S::kStages];
    uint64_t item_full[2];
    uint64_t item_empty[2];
    Item item[2];
    uint32_t gave_up;
    float top[kWarps][S::kRows];
    float sum[kWarps][S::kRows];
    PlanShared<kWarps + 1> plan;
};

// ---------------------------------------------------------------------------
// the copying warp

template <int D, int NT>
__device__ __forceinline__ void copy_items(const Fp4Attention &a, Shared<D, NT> &sm, const Run &run,
                                           int32_t group, Split *record) {
    using S = Shape<D, NT>;
    const int32_t lane = threadIdx.x % 32;
    // A round of steps is 16 copies: lane = 4 * warp + (K, K, V, V).
    const int32_t to_warp = lane / 4, which = lane % 4;
    uint32_t fill = 0;                         // steps issued to this lane's warp
    uint32_t items = 0;
    Walk walk;
    walk.begin(a, run, group, S::kRows);
    for (;;) {
        const Tile x = tile_of(walk.s, walk.rt, group, S::kRows, a.window);
        const int64_t unit0 = walk.start + kItemCost;
        if (unit0 >= run.end) break;
        const int32_t r0 = static_cast<int32_t>(max(int64_t{0}, run.at - unit0));
        const int32_t r1 = static_cast<int32_t>(min(static_cast<int64_t>(x.units), run.end - unit0));
        if (r1 > r0) {
            Item it;
            it.begin = x.begin + r0 * kUnit;
            it.end = min(x.end, x.begin + r1 * kUnit);
            it.first = x.first;
            it.steps = it.end > it.begin ? (it.end - it.begin + kStep - 1) / kStep : 0;
            it.ahead = walk.s.length - walk.s.news;
            it.token0 = walk.s.token0;
            it.row0 = x.row0;
            it.rows = x.rows;
            it.head = walk.head;
            it.part = r0 == 0 && r1 == x.units ? -1 : r0 == 0 ? 1 : 0;

            const uint32_t slot = items % 2;
            if (items >= 2) barrier_wait(smem_addr(&sm.item_empty[slot]), (items / 2 - 1) & 1, &sm.gave_up);
            const uint32_t bar = smem_addr(&sm.item_full[slot]);
            if (lane == 0) {
                sm.item[slot] = it;
                barrier_expect(bar, x.rows * 2 * D);
                if (it.part == 1) {
                    record->token0 = it.token0;
                    record->row0 = it.row0;
                    record->rows = it.rows;
                    record->head = it.head;
                    record->blocks = static_cast<int32_t>((unit0 + x.units - 1) / run.per_block) - blockIdx.x + 1;
                }
            }
            __syncwarp();
            if (lane < x.rows) {
                const int32_t row = x.row0 + lane, qi = row / group;
                const uint16_t *src = a.q + (it.token0 + qi) * a.q_stride +
                    (static_cast<int64_t>(it.head) * group + (row - qi * group)) * D;
                copy_async(smem_addr(sm.q[slot][lane]), src, 2 * D, bar);
            }
            ++items;

            const int32_t *table = a.block_table + static_cast<int64_t>(walk.seq) * a.table_stride;
            const int32_t rounds = (it.steps + kWarps - 1) / kWarps;
            int32_t at = it.begin + to_warp * kStep;           // this lane's step
            auto look_up = [&](int32_t tok, int32_t *tile) -> int64_t {
                if (lane >= 4 * kWarps || tok >= it.end) return 0;
                *tile = tok / 16;
                const int32_t page_at = *tile / a.pools.tiles;
                *tile -= page_at * a.pools.tiles;
                return table[page_at];
            };
            int32_t tile = 0;
            int64_t page = look_up(at + 16 * (which & 1), &tile);
            for (int32_t r = 0; r < rounds; ++r) {
                int32_t tile_next = 0;
                const int64_t page_next = look_up(at + kUnit + 16 * (which & 1), &tile_next);
                if (lane < 4 * kWarps && at < it.end) {
                    const uint32_t stage = fill % S::kStages;
                    const uint32_t full = smem_addr(&sm.full[to_warp][stage]);
                    if (fill >= S::kStages)
                        barrier_wait(smem_addr(&sm.empty[to_warp][stage]), (fill / S::kStages - 1) & 1, &sm.gave_up);
                    if (which == 0) barrier_expect(full, (it.end - at > 16 ? 4 : 2) * S::kTile);
                    if (at + 16 * (which & 1) < it.end) {
                        if (page < 0 || page >= a.pools.num_blocks) {
                            atomicOr(&g_fp4_attention_error, kFp4ErrSlot);
                            page = 0;
                        }
                        const uint8_t *src = (which < 2 ? a.pools.k : a.pools.v) + page * a.pools.block_stride +
                            (static_cast<int64_t>(it.head) * a.pools.tiles + tile) * S::kTile;
                        copy_async(smem_addr(sm.ring[to_warp][stage]) + which * S::kTile, src, S::kTile, full);
                    }
                    ++fill;
                }
                __syncwarp();
                at += kUnit;
                page = page_next;
                tile = tile_next;
            }
        }
        if (!walk.next(a, x.units + kItemCost, group, S::kRows)) break;
    }
    const uint32_t slot = items % 2;
    if (items >= 2) barrier_wait(smem_addr(&sm.item_empty[slot]), (items / 2 - 1) & 1, &sm.gave_up);
    if (lane == 0) {
        sm.item[slot].steps = -1;
        barrier_arrive(smem_addr(&sm.item_full[slot]));
    }
}

// ---------------------------------------------------------------------------
// the computing warps

// The query rows as the right operand of S^T, and what each column needs.
template <int D, int NT>
struct Rows {
    uint32_t q[NT][D / 16][2];
    float c[NT][2];                        // factor of raw scores: log2 of a weight
    int32_t see_hi[NT][2], see_lo[NT][2];  // tokens the column sees
};

template <int D, int NT>
__device__ __forceinline__ void load_rows(const Fp4Attention &a, const Item &it,
                                          const uint8_t (&q)[8 * NT][Shape<D, NT>::kQPitch],
                                          int32_t group, float k_scale, Rows<D, NT> &r) {
    const int32_t lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const bool live = n * 8 + g < it.rows;
        uint32_t w[D / 8];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live) x = *reinterpret_cast<const uint4 *>(q[n * 8 + g] + t * (D / 2) + 16 * i);
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
        }
        uint32_t most = 0;                 // largest magnitude pattern
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            most = max(most, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        const int32_t up = min(8 - (static_cast<int32_t>(most >> 7) - 127), 120);
        const float scale = __int_as_float((127 + up) << 23);
        const float back = __int_as_float((127 - up) << 23);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            r.q[n][i][0] = f16x2_of(bf16_low(w[2 * i]) * scale, bf16_high(w[2 * i]) * scale);
            r.q[n][i][1] = f16x2_of(bf16_low(w[2 * i + 1]) * scale, bf16_high(w[2 * i + 1]) * scale);
        }
        // A factor above zero keeps masked scores at -infinity; raw scores are
        // below 2^30, so one this small stands for zero.
        const float mine_c = fmaxf(a.softmax_scale * kLog2e * k_scale * back, 0x1p-100f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            r.c[n][j] = __shfl_sync(0xFFFFFFFFu, mine_c, 4 * (2 * t + j));
            const int32_t col = n * 8 + 2 * t + j;
            const int32_t ci = (it.row0 + min(col, it.rows - 1)) / group;
            r.see_hi[n][j] = min(it.end, it.ahead + ci + 1);
            r.see_lo[n][j] = a.window > 0 ? max(0, it.ahead + ci + 1 - a.window) : 0;
        }
    }
}

// Raw scores of 16 tokens: S^T = K Q^T.
template <int D, int NT>
__device__ __forceinline__ void score_tile(const uint8_t *kt, const Rows<D, NT> &r, float (&sc)[NT][4]) {
    const int32_t lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int32_t tok = 4 * (g / 2) + (g % 2);     // this lane's rows: tok, tok + 2
    constexpr int kWords = D / 32;                 // code words of a lane's part of a row
    uint32_t ca[kWords], cb[kWords], za[(D + 127) / 128], zb[(D + 127) / 128];
    const uint8_t *ra = kt + tok * (D / 2) + t * (D / 8);
    const uint8_t *rb = ra + D;
    const uint8_t *sa = kt + 8 * D + tok * (D / 16) + t * (D / 64);
    const uint8_t *sb = sa + D / 8;
    if constexpr (D == 64) {
        const uint2 x = *reinterpret_cast<const uint2 *>(ra);
        const uint2 y = *reinterpret_cast<const uint2 *>(rb);
        ca[0] = x.x, ca[1] = x.y, cb[0] = y.x, cb[1] = y.y;
        za[0] = *sa, zb[0] = *sb;
    } else {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 x = reinterpret_cast<const uint4 *>(ra)[i];
            const uint4 y = reinterpret_cast<const uint4 *>(rb)[i];
            ca[4 * i] = x.x, ca[4 * i + 1] = x.y, ca[4 * i + 2] = x.z, ca[4 * i + 3] = x.w;
            cb[4 * i] = y.x, cb[4 * i + 1] = y.y, cb[4 * i + 2] = y.z, cb[4 * i + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < D / 128; ++i) {
            za[i] = reinterpret_cast<const uint16_t *>(sa)[i];
            zb[i] = reinterpret_cast<const uint16_t *>(sb)[i];
        }
    }
#pragma unroll
    for (int i = 0; i < (D + 127) / 128; ++i) za[i] = f16x2_of_e4m3x2(za[i]), zb[i] = f16x2_of_e4m3x2(zb[i]);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[n][j] = 0.0f;
#pragma unroll
    for (int blk = 0; blk < D / 64; ++blk) {       // 16 dimensions, four k-steps
        const uint32_t s_a = blk % 2 ? high_twice(za[blk / 2]) : low_twice(za[blk / 2]);
        const uint32_t s_b = blk % 2 ? high_twice(zb[blk / 2]) : low_twice(zb[blk / 2]);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint32_t xa[4], xb[4];
            f16x2_of_e2m1x8(ca[2 * blk + w], xa);
            f16x2_of_e2m1x8(cb[2 * blk + w], xb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                xa[i] = mul_f16x2(xa[i], s_a);
                xb[i] = mul_f16x2(xb[i], s_b);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int ks = 4 * blk + 2 * w + i;
                    mma(sc[n], xa[2 * i], xb[2 * i], xa[2 * i + 1], xb[2 * i + 1], r.q[n][ks][0],
                        r.q[n][ks][1]);
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

// The fp32 output of a row from its joined sums: nothing seen gives 0, a NaN
// among the scores stays one.
__device__ __forceinline__ float row_factor(float l, float v_scale) { return l == 0.0f ? 0.0f : v_scale / l; }
__device__ __forceinline__ float row_lse(float most, float l) {
    return l == 0.0f ? -INFINITY : kLn2 * (most + (log2f(l) - kShift));
}

// A pair of dimensions of one row, rounded and stored.
__device__ __forceinline__ void store_pair(const Fp4Attention &a, int32_t token, int32_t q_head,
                                           int32_t dim, int32_t at, float x, float y) {
    *reinterpret_cast<uint32_t *>(a.out + token * a.out_stride + static_cast<int64_t>(q_head) * dim + at) =
        bf16x2_of(x, y);
}

template <int D, int NT>
__device__ __forceinline__ void compute_items(const Fp4Attention &a, Shared<D, NT> &sm, int32_t group,
                                              float k_scale, float v_scale) {
    using S = Shape<D, NT>;
    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t g = lane / 4, t = lane % 4;
    const int32_t tok_a = 4 * (g / 2) + (g % 2);   // this lane's score rows: tok_a, tok_a + 2
    uint32_t drain = 0;                            // steps this warp has used
    for (uint32_t items = 0;; ++items) {
        const uint32_t slot = items % 2;
        barrier_wait(smem_addr(&sm.item_full[slot]), (items / 2) & 1, &sm.gave_up);
        const Item it = sm.item[slot];
        if (it.steps < 0) return;
        const int32_t steps = it.steps > warp ? (it.steps - warp + kWarps - 1) / kWarps : 0;

        Rows<D, NT> r;
        load_rows<D, NT>(a, it, sm.q[slot], group, k_scale, r);
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
        const int32_t all_hi = min(it.end, it.ahead + it.row0 / group + 1);   // every row sees below
        const int32_t all_lo =
            a.window > 0 ? max(0, it.ahead + (it.row0 + it.rows - 1) / group + 1 - a.window) : 0;

        for (int32_t k = 0; k < steps; ++k) {
            const int32_t at = it.begin + (warp + k * kWarps) * kStep;
            const uint32_t stage = drain % S::kStages;
            barrier_wait(smem_addr(&sm.full[warp][stage]), (drain / S::kStages) & 1, &sm.gave_up);
            const uint8_t *ring = sm.ring[warp][stage];
            const bool edge = at + kStep > all_hi || at < all_lo;

            float sc[2][NT][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) score_tile<D, NT>(ring + m * S::kTile, r, sc[m]);
            if (edge) {
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int32_t tok = at + 16 * m + tok_a + 2 * (j / 2);
                            if (tok >= r.see_hi[n][j % 2] || tok < r.see_lo[n][j % 2]) sc[m][n][j] = -INFINITY;
                        }
            }

            // ---- running maximum and sum -------------------------------------
            float mx[NT][2];
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    mx[n][j] = r.c[n][j] * fmaxf(fmaxf(sc[0][n][j], sc[0][n][2 + j]),
                                                 fmaxf(sc[1][n][j], sc[1][n][2 + j]));
                    grew |= mx[n][j] > top[n][j];
                }
            if (__any_sync(0xFFFFFFFFu, grew)) {
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
            }
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float &x = sc[m][n][j];
                        x = exp2_fast(fmaf(x, r.c[n][j % 2], -ref[n][j % 2]));
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
                    add_tile<D, NT, true>(ring + (2 + m) * S::kTile, it.first - (at + 16 * m),
                                          it.end - (at + 16 * m), pf[m], o);
            } else {
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    add_tile<D, NT, false>(ring + (2 + m) * S::kTile, 0, 16, pf[m], o);
            }
            ++drain;
            __syncwarp();                      // every lane has read the stage
            if (lane == 0) barrier_arrive(smem_addr(&sm.empty[warp][stage]));
        }

        // ---- join the warps ---------------------------------------------------
        const int32_t busy = min(kWarps, max(1, it.steps));    // warps that had a step
        if (warp < busy) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float l = sum[n][j];
#pragma unroll
                    for (int off = 4; off < 32; off *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
                    if (g == 0) {
                        sm.top[warp][n * 8 + 2 * t + j] = top[n][j];
                        sm.sum[warp][n * 8 + 2 * t + j] = l;
                    }
                }
#pragma unroll
                for (int i = 0; i < S::kMTiles; ++i)
                    sm.sums[warp][i * NT + n][lane] =
                        make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
            }
        }
        meet();
        // Each warp finishes a quarter of the dimensions.
        float *part = part_at(a.workspace, 2 * static_cast<int64_t>(blockIdx.x) + max(it.part, 0), S::kRows, D);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[kWarps][2], most[2], l[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int32_t col = n * 8 + 2 * t + j;
                most[j] = -INFINITY;
                for (int w = 0; w < busy; ++w) most[j] = fmaxf(most[j], sm.top[w][col]);
                const float base = most[j] == -INFINITY ? 0.0f : most[j];
                l[j] = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    f[w][j] = w < busy ? exp2_fast(sm.top[w][col] - base) : 0.0f;
                    if (w < busy) l[j] += f[w][j] * sm.sum[w][col];
                }
            }
#pragma unroll
            for (int ii = 0; ii < S::kMTiles / kWarps; ++ii) {
                const int i = warp * (S::kMTiles / kWarps) + ii;
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    if (w < busy) {
                        const float4 v = sm.sums[w][i * NT + n][lane];
                        x.x += f[w][0] * v.x, x.y += f[w][1] * v.y;
                        x.z += f[w][0] * v.z, x.w += f[w][1] * v.w;
                    }
                if (it.part >= 0) {
                    reinterpret_cast<float4 *>(part)[(i * NT + n) * 32 + lane] = x;
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int32_t row = n * 8 + 2 * t + j;
                        if (row >= it.rows) continue;
                        const int32_t qi = (it.row0 + row) / group;
                        const float inv = row_factor(l[j], v_scale);
                        store_pair(a, it.token0 + qi, it.head * group + (it.row0 + row - qi * group), D,
                                   g * (D / 8) + 2 * i, (j ? x.y : x.x) * inv, (j ? x.w : x.z) * inv);
                    }
                }
            }
            if (warp == 0 && g == 0) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int32_t row = n * 8 + 2 * t + j;
                    if (it.part >= 0) {
                        part[S::kRows * D + row] = most[j];
                        part[S::kRows * D + S::kRows + row] = l[j];
                    } else if (a.lse != nullptr && row < it.rows) {
                        const int32_t qi = (it.row0 + row) / group;
                        a.lse[static_cast<int64_t>(it.token0 + qi) * a.q_heads + it.head * group +
                              (it.row0 + row - qi * group)] = row_lse(most[j], l[j]);
                    }
                }
            }
        }
        meet();                                // the sums may be written again
        if (lane == 0) barrier_arrive(smem_addr(&sm.item_empty[slot]));
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kBlocks) fp4_attention_kernel(const Fp4Attention a) {
    using S = Shape<D, NT>;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Shared<D, NT> &sm = *reinterpret_cast<Shared<D, NT> *>(smem_raw);
    const int32_t group = a.q_heads / a.pools.heads;

    if (threadIdx.x < kWarps * S::kStages) {
        barrier_init(smem_addr(&sm.full[0][0] + threadIdx.x), 1);
        barrier_init(smem_addr(&sm.empty[0][0] + threadIdx.x), 1);
    }
    if (threadIdx.x == 0) sm.gave_up = 0;
    if (threadIdx.x < 2) {
        barrier_init(smem_addr(&sm.item_full[threadIdx.x]), 1);
        barrier_init(smem_addr(&sm.item_empty[threadIdx.x]), kWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    pdl_allow_next();

    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    Split *record = static_cast<Split *>(a.workspace) + blockIdx.x;
    if (threadIdx.x == 32 * kWarps) record->blocks = 0;
    if (!fp4_scale_ok(k_scale) || !fp4_scale_ok(v_scale)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_fp4_attention_error, kFp4ErrScale);
        return;
    }
    const Run run = block_run<kWarps + 1>(a, group, S::kRows, &g_fp4_attention_error, sm.plan);
    if (run.at >= run.end) return;             // the whole block
    if (threadIdx.x >= 32 * kWarps)
        copy_items<D, NT>(a, sm, run, group, record);
    else
        compute_items<D, NT>(a, sm, group, k_scale, v_scale);
    if (*static_cast<volatile uint32_t *>(&sm.gave_up)) __nanosleep(1000000);   // copies under way land
}

// ---------------------------------------------------------------------------
// the join

constexpr int kJoinWarps = 8;

// Block (c, y) merges some dimensions of the item that began in block c:
// `units` of the 32-lane, 4-value fragments its parts are stored in, eight or
// fewer, its warps shared out over the parts where there are fewer.
template <int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) fp4_attention_join_kernel(const Fp4Attention a,
                                                                             int32_t units) {
    using S = Shape<D, NT>;
    constexpr int kRows = S::kRows;
    __shared__ float weight[kMaxBlocks][kRows];    // 2^(top of the part - top)
    __shared__ float most_of[kRows], sum_of[kRows];
    __shared__ float4 share[kJoinWarps][32];
    pdl_wait();
    pdl_allow_next();
    const int32_t c = blockIdx.x;
    const Split s = static_cast<const Split *>(a.workspace)[c];
    if (s.blocks == 0) return;
    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    // part 1 of block c, then part 0 of the blocks behind it
    auto part = [&](int32_t i) -> const float * {
        return part_at(a.workspace, 2 * static_cast<int64_t>(c + i) + (i == 0 ? 1 : 0), kRows, D);
    };
    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    for (int32_t row = warp; row < kRows; row += kJoinWarps) {
        float most = -INFINITY;
        for (int32_t i = lane; i < s.blocks; i += 32) {
            weight[i][row] = part(i)[kRows * D + row];
            most = fmaxf(most, weight[i][row]);
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
        const float base = most == -INFINITY ? 0.0f : most;
        float l = 0.0f;
        for (int32_t i = lane; i < s.blocks; i += 32) {
            const float f = exp2_fast(weight[i][row] - base);
            weight[i][row] = f;
            l += f * part(i)[kRows * D + kRows + row];
        }
#pragma unroll
        for (int o = 16; o > 0; o /= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        if (lane == 0) most_of[row] = most, sum_of[row] = l;
    }
    __syncthreads();
    const int32_t groups = kJoinWarps / units, which = warp / units;
    const int32_t unit = blockIdx.y * units + warp % units;        // i * NT + n
    const int32_t col = (unit % NT) * 8 + 2 * (lane % 4);
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int32_t i = which; i < s.blocks; i += groups) {
        const float4 v = reinterpret_cast<const float4 *>(part(i))[unit * 32 + lane];
        const float f0 = weight[i][col], f1 = weight[i][col + 1];
        x.x += f0 * v.x, x.y += f1 * v.y, x.z += f0 * v.z, x.w += f1 * v.w;
    }
    share[warp][lane] = x;
    __syncthreads();
    if (which > 0) return;
    for (int32_t w = 1; w < groups; ++w) {
        const float4 v = share[w * units + warp][lane];
        x.x += v.x, x.y += v.y, x.z += v.z, x.w += v.w;
    }
    const int32_t group = a.q_heads / a.pools.heads;
    const int32_t i = unit / NT;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int32_t row = col + j;
        if (row >= s.rows) continue;
        const int32_t qi = (s.row0 + row) / group;
        const int32_t q_head = s.head * group + (s.row0 + row - qi * group);
        const float inv = row_factor(sum_of[row], v_scale);
        store_pair(a, s.token0 + qi, q_head, D, (lane / 4) * (D / 8) + 2 * i, (j ? x.y : x.x) * inv,
                   (j ? x.w : x.z) * inv);
        if (a.lse != nullptr && i == 0 && lane < 4)
            a.lse[static_cast<int64_t>(s.token0 + qi) * a.q_heads + q_head] = row_lse(most_of[row], sum_of[row]);
    }
}

// ---------------------------------------------------------------------------
// launch

// Rows of a tile (8 * NT) for an average of `rows` rows a sequence: the
// smallest tile that holds them, up to what the accumulators leave room for
// in registers (NT * D <= 256).
int tiles_of(int64_t batch, int64_t num_tokens, int32_t group, int32_t dim) {
    const int64_t rows = (num_tokens + batch - 1) / batch * group;
    return rows <= 8 || dim == 256 ? 1 : 2;
}

template <int D, int NT>
cudaError_t launch_tiles(const Fp4Attention &a, cudaStream_t stream) {
    using S = Shape<D, NT>;
    constexpr size_t kSmem = sizeof(Shared<D, NT>);
    static_assert(S::kBlocks * (kSmem + 1024) <= 228 * 1024, "the blocks of an SM fit its shared memory");
    auto kernel = fp4_attention_kernel<D, NT>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    // No more blocks than there can be points on the axis.
    const int32_t group = a.q_heads / a.pools.heads;
    const int64_t items = ((static_cast<int64_t>(a.num_tokens) * group + S::kRows - 1) / S::kRows + a.batch) *
                          a.pools.heads;
    const int64_t longest = (a.table_width * a.pools.tiles * 16 + kUnit - 1) / kUnit + 1 + kItemCost;
    int64_t grid = static_cast<int64_t>(sms) * S::kBlocks;
    if (grid > kMaxBlocks) grid = kMaxBlocks;
    if (items < grid && items * longest < grid) grid = items * longest;
    e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kThreads, kSmem, stream, a);
    if (e != cudaSuccess) return e;
    // Few items have many parts each: their dimensions go to several blocks.
    constexpr int32_t kUnits = S::kMTiles * NT;
    const int32_t units = items * 8 <= sms ? 1 : kUnits < kJoinWarps ? kUnits : kJoinWarps;
    return launch_pdl(fp4_attention_join_kernel<D, NT>,
                      dim3(static_cast<unsigned>(grid), static_cast<unsigned>(kUnits / units)),
                      32 * kJoinWarps, 0, stream, a, units);
}

}  // namespace

int64_t fp4_attention_workspace(int64_t batch, int64_t num_tokens, int32_t q_heads,
                                int32_t kv_heads, int32_t dim) {
    if (batch == 0) return 0;
    const int nt = tiles_of(batch, num_tokens, q_heads / kv_heads, dim);
    return kRecordBytes + kMaxBlocks * 2 * 4 * part_floats(8 * nt, dim);
}

cudaError_t launch_fp4_attention(const Fp4Attention &a, cudaStream_t stream) {
    const int nt = tiles_of(a.batch, a.num_tokens, a.q_heads / a.pools.heads, a.pools.dim);
    switch (a.pools.dim) {
    case 64: return nt == 1 ? launch_tiles<64, 1>(a, stream) : launch_tiles<64, 2>(a, stream);
    case 128: return nt == 1 ? launch_tiles<128, 1>(a, stream) : launch_tiles<128, 2>(a, stream);
    default: return launch_tiles<256, 1>(a, stream);
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
