// fp4_attention.cu -- attention over a paged cache held in 4 bits (sm_100a).
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
// and read again, for eight rows of a 128-row tile.
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
// Work is split over the whole cache, not over sequences.  A unit is 128
// cached tokens of one (sequence, KV head, row tile); every block takes an
// equal run of units, computed on the device from the lengths, so a launch
// depends on sizes only and may be captured.  An item whose units lie in
// several blocks leaves one partial result per block, which a second kernel
// joins in a fixed order.
#include <cuda_runtime.h>

#include <cmath>

#include "fp4_device.cuh"

namespace fp8q {

namespace {

__device__ uint32_t g_fp4_attention_error;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;             // 32-token steps in flight for each warp
constexpr int kStep = 32;              // cached tokens of a warp's step
constexpr int kUnit = kStep * kWarps;  // cached tokens of a unit
constexpr int kMaxBlocks = 592;        // blocks a workspace has room for
constexpr int kWaitTries = 1 << 22;    // polls of a copy before giving up
constexpr float kShift = 15.0f;        // p is held as p * 2^15
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void barrier_init(uint32_t bar) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" :: "r"(bar) : "memory");
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

// ---------------------------------------------------------------------------
// the plan

// One sequence as the kernel sees it: bad lengths and ranges are cut to what
// the buffers hold and reported.
struct Sequence {
    int32_t token0;     // first new token
    int32_t news;       // new tokens
    int32_t length;     // cached tokens, the new ones included
    int32_t first;      // first cached token any of them sees, rounded down to a tile
    int32_t row_tiles;
    int32_t units;      // units of each (head, row tile); at least one
};

__device__ __forceinline__ Sequence sequence(const Fp4Attention &a, int32_t b, int32_t group,
                                             int32_t rows_per_tile, bool *bad) {
    Sequence s;
    int64_t t0 = b, t1 = b + 1;
    if (a.q_start != nullptr) {
        t0 = a.q_start[b];
        t1 = a.q_start[b + 1];
    }
    if (t0 < 0 || t1 < t0 || t1 > a.num_tokens) {
        *bad = true;
        t0 = t0 < 0 ? 0 : t0;
        t1 = t1 > a.num_tokens ? a.num_tokens : t1;
        if (t1 < t0) t0 = t1 = 0;
    }
    const int64_t room = a.pools.num_blocks > 0 ? a.table_width * (a.pools.tiles * 16) : 0;
    int64_t length = a.seq_lens[b];
    if (length < 0 || length > room) {
        *bad = true;
        length = length < 0 ? 0 : room;
    }
    s.token0 = static_cast<int32_t>(t0);
    s.news = static_cast<int32_t>(t1 - t0);
    s.length = static_cast<int32_t>(length);
    int64_t first = 0;
    if (a.window > 0) {
        first = length - s.news + 1 - a.window;
        first = first < 0 ? 0 : first & ~int64_t{15};
    }
    s.first = static_cast<int32_t>(first);
    s.row_tiles = static_cast<int32_t>((static_cast<int64_t>(s.news) * group + rows_per_tile - 1) /
                                       rows_per_tile);
    const int32_t units = static_cast<int32_t>((length - first + kUnit - 1) / kUnit);
    s.units = units < 1 ? 1 : units;
    return s;
}

// A block's record of the item that begins in it and goes on in the blocks
// behind it: the join reads it.
struct Split {
    int32_t blocks;     // blocks that hold a part of the item; 0: no such item
    int32_t token0, row0, rows, head;
};

// Workspace: Split [kMaxBlocks], then for each block two parts (0: an item
// begun in an earlier block, 1: an item that goes on in the next one) of
// rows x dim sums, rows maxima and rows sums.
__host__ __device__ constexpr int64_t part_floats(int rows, int dim) {
    return static_cast<int64_t>(rows) * (dim + 2);
}

__device__ __forceinline__ float *part_at(void *workspace, int64_t index, int rows, int dim) {
    float *base = reinterpret_cast<float *>(static_cast<Split *>(workspace) + kMaxBlocks);
    return base + index * part_floats(rows, dim);
}

__device__ __forceinline__ void store_row2(const Fp4Attention &a, int32_t token, int32_t q_head,
                                           int32_t dim_at, int32_t dim, float x, float y) {
    *reinterpret_cast<uint32_t *>(a.out + token * a.out_stride + q_head * dim + dim_at) =
        bf16x2_of(x, y);
}

__device__ __forceinline__ void load_scales(const Fp4Attention &a, float *ks, float *vs) {
    *ks = a.pools.scale_dev ? a.pools.scale_dev[0] : a.pools.k_scale;
    *vs = a.pools.scale_dev ? a.pools.scale_dev[1] : a.pools.v_scale;
}

// ---------------------------------------------------------------------------
// the kernel

template <int D>
struct Stage {
    static constexpr int kTile = 9 * D;            // bytes of 16 tokens
    static constexpr int kBytes = 4 * kTile;       // K, K, V, V
};

template <int D, int NT>
struct Shared {
    alignas(128) uint8_t ring[kWarps][kStages][Stage<D>::kBytes];
    alignas(8) uint64_t full[kWarps][kStages];
    float top[kWarps][8 * NT];
    float sum[kWarps][8 * NT];
    int64_t scan[kWarps];
    int64_t total;
    int64_t base;
    int32_t seq;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) fp4_attention_kernel(const Fp4Attention a) {
    constexpr int kRows = 8 * NT;
    constexpr int kTile = Stage<D>::kTile;
    constexpr int kKSteps = D / 16;            // of S^T
    constexpr int kMTiles = D / 16;            // of O^T
    constexpr int kKWords = D / 32;            // code words of a lane's part of a K row
    constexpr int kVWords = D / 64;            // code words of a lane's part of a V row
    static_assert(kRows * D * 4 <= kStages * Stage<D>::kBytes, "a warp's sums fit its ring");
    extern __shared__ __align__(128) uint8_t smem_raw[];
    Shared<D, NT> &sm = *reinterpret_cast<Shared<D, NT> *>(smem_raw);

    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t g = lane / 4, t = lane % 4;
    const int32_t group = a.q_heads / a.pools.heads;
    const int32_t heads = a.pools.heads;

    if (lane < kStages) barrier_init(smem_addr(&sm.full[warp][lane]));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pdl_wait();
    pdl_allow_next();

    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    if (!fp4_scale_ok(k_scale) || !fp4_scale_ok(v_scale)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_fp4_attention_error, kFp4ErrScale);
        return;                                // the join finds the same and returns too
    }

    // ---- this block's units: a scan over the sequences --------------------
    bool bad = false;
    const int32_t per_thread = (a.batch + kThreads - 1) / kThreads;
    const int32_t b_begin = min(a.batch, static_cast<int32_t>(threadIdx.x) * per_thread);
    const int32_t b_end = min(a.batch, b_begin + per_thread);
    int64_t mine = 0;
    for (int32_t b = b_begin; b < b_end; ++b) {
        const Sequence s = sequence(a, b, group, kRows, &bad);
        mine += static_cast<int64_t>(s.units) * s.row_tiles * heads;
    }
    if (bad) atomicOr(&g_fp4_attention_error, kFp4ErrSequence);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) sm.scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sm.scan[w];
        total += sm.scan[w];
    }
    const int64_t per_block = (total + gridDim.x - 1) / gridDim.x;
    int64_t u = per_block * blockIdx.x;
    const int64_t u_end = min(total, u + per_block);
    Split *record = static_cast<Split *>(a.workspace) + blockIdx.x;
    if (threadIdx.x == 0) record->blocks = 0;
    if (u >= u_end) return;                    // the whole block
    if (mine > 0 && before <= u && u < before + mine) {
        for (int32_t b = b_begin; b < b_end; ++b) {
            const Sequence s = sequence(a, b, group, kRows, &bad);
            const int64_t n = static_cast<int64_t>(s.units) * s.row_tiles * heads;
            if (u < before + n) {
                sm.seq = b;
                sm.base = before;
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    int32_t b = sm.seq;
    int64_t base = sm.base;
    uint32_t fill = 0;                         // steps this warp has issued so far
    uint32_t drain = 0;                        // steps it has used

    // ---- items -------------------------------------------------------------
    while (u < u_end) {
        const Sequence s = sequence(a, b, group, kRows, &bad);
        const int64_t seq_units = static_cast<int64_t>(s.units) * s.row_tiles * heads;
        if (u >= base + seq_units) {           // on to the next sequence
            base += seq_units;
            ++b;
            continue;
        }
        const int32_t item = static_cast<int32_t>((u - base) / s.units);
        const int64_t item_base = base + static_cast<int64_t>(item) * s.units;
        const int32_t r0 = static_cast<int32_t>(u - item_base);
        const int32_t r1 = static_cast<int32_t>(min(static_cast<int64_t>(s.units), r0 + (u_end - u)));
        const int32_t head = item / s.row_tiles;
        const int32_t row0 = (item - head * s.row_tiles) * kRows;
        const int32_t rows = min(kRows, s.news * group - row0);
        const int32_t ahead = s.length - s.news;   // query i sees tokens up to ahead + i

        // the part of this block's tokens that some row of the tile sees
        const int32_t q_lo = row0 / group, q_hi = (row0 + rows - 1) / group;
        int32_t begin = s.first + r0 * kUnit;
        int32_t end = min(s.length, s.first + r1 * kUnit);
        end = min(end, ahead + q_hi + 1);
        const int32_t seen_lo = a.window > 0 ? max(0, ahead + q_lo + 1 - a.window) : 0;
        begin = max(begin, seen_lo & ~15);
        const int32_t all_hi = ahead + q_lo + 1;   // every row sees tokens below this
        const int32_t all_lo = a.window > 0 ? max(0, ahead + q_hi + 1 - a.window) : 0;
        const int32_t steps_all = end > begin ? (end - begin + kStep - 1) / kStep : 0;
        const int32_t steps = steps_all > warp ? (steps_all - warp + kWarps - 1) / kWarps : 0;

        // ---- copies ---------------------------------------------------------
        // Lanes 0..3 copy the step's K tiles and V tiles; tiles behind `end`
        // are left out.
        const int32_t *table = a.block_table + static_cast<int64_t>(b) * a.table_stride;
        auto issue = [&](int32_t k) {
            const int32_t at = begin + (warp + k * kWarps) * kStep;
            const uint32_t slot = fill % kStages;
            const uint32_t bar = smem_addr(&sm.full[warp][slot]);
            const int32_t tile_at = at + 16 * (lane & 1);
            const int32_t tiles = end - at > 16 ? 2 : 1;
            if (lane == 0) barrier_expect(bar, 2 * tiles * kTile);
            __syncwarp();
            if (lane < 4 && tile_at < end) {
                const int32_t tile = tile_at / 16;
                const int32_t page_at = tile / a.pools.tiles;
                int64_t page = table[page_at];
                if (page < 0 || page >= a.pools.num_blocks) {
                    atomicOr(&g_fp4_attention_error, kFp4ErrSlot);
                    page = 0;
                }
                const uint8_t *pool = lane < 2 ? a.pools.k : a.pools.v;
                const uint8_t *src = pool + page * a.pools.block_stride +
                    (static_cast<int64_t>(head) * a.pools.tiles + (tile - page_at * a.pools.tiles)) * kTile;
                copy_async(smem_addr(sm.ring[warp][slot]) + lane * kTile, src, kTile, bar);
            }
            ++fill;
        };
        for (int32_t k = 0; k < kStages && k < steps; ++k) issue(k);

        // ---- the query rows -------------------------------------------------
        uint32_t qf[NT][kKSteps][2];
        float c[NT][2];                        // factor of raw scores, by column
        int32_t see_hi[NT][2], see_lo[NT][2];  // tokens each column sees
        float top[NT][2], sum[NT][2];
        float o[kMTiles][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int32_t row = row0 + n * 8 + g;
            const bool live = n * 8 + g < rows;
            const int32_t qi = live ? row / group : 0;
            uint32_t w[D / 8];
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (live)
                    x = *reinterpret_cast<const uint4 *>(
                        a.q + (s.token0 + qi) * a.q_stride +
                        (static_cast<int64_t>(head) * group + (row - qi * group)) * D + t * (D / 4) + 8 * i);
                w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
            }
            uint32_t most = 0;                 // largest magnitude pattern
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                most = max(most, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
            int32_t up = 8 - (static_cast<int32_t>(most >> 7) - 127);
            up = min(up, 120);
            const float scale = __int_as_float((127 + up) << 23);
            const float back = __int_as_float((127 - up) << 23);
#pragma unroll
            for (int i = 0; i < kKSteps; ++i) {
                qf[n][i][0] = f16x2_of(bf16_low(w[2 * i]) * scale, bf16_high(w[2 * i]) * scale);
                qf[n][i][1] = f16x2_of(bf16_low(w[2 * i + 1]) * scale, bf16_high(w[2 * i + 1]) * scale);
            }
            const float mine_c = a.softmax_scale * kLog2e * k_scale * back;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                c[n][j] = __shfl_sync(0xFFFFFFFFu, mine_c, 4 * (2 * t + j));
                const int32_t col = n * 8 + 2 * t + j;
                const int32_t ci = (row0 + min(col, rows - 1)) / group;
                see_hi[n][j] = min(end, ahead + ci + 1);
                see_lo[n][j] = a.window > 0 ? max(0, ahead + ci + 1 - a.window) : 0;
                top[n][j] = -INFINITY;
                sum[n][j] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < kMTiles; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][n][j] = 0.0f;
        }

        const int32_t tok_a = 4 * (g / 2) + (g % 2);   // K rows of this lane: tok_a, tok_a + 2

        for (int32_t k = 0; k < steps; ++k) {
            const int32_t at = begin + (warp + k * kWarps) * kStep;
            const uint32_t slot = drain % kStages;
            {
                const uint32_t bar = smem_addr(&sm.full[warp][slot]);
                const uint32_t parity = (drain / kStages) & 1;
                int32_t tries = 0;
                while (!barrier_done(bar, parity)) {
                    if (++tries > kWaitTries) {
                        atomicOr(&g_fp4_attention_error, kFp4ErrWait);
                        break;
                    }
                }
                __syncwarp();
            }
            const uint8_t *ring = sm.ring[warp][slot];
            const bool edge = at + kStep > min(end, all_hi) || at < all_lo;

            // ---- S^T = K Q^T -------------------------------------------------
            float sc[2][NT][4];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint8_t *kt = ring + m * kTile;
                uint32_t ca[kKWords], cb[kKWords], za, zb;
                const uint8_t *ra = kt + tok_a * (D / 2) + t * (D / 8);
                const uint8_t *rb = ra + D;
                const uint8_t *sa = kt + 8 * D + tok_a * (D / 16) + t * (D / 64);
                const uint8_t *sb = sa + D / 8;
                if constexpr (D == 64) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(ra);
                    const uint2 y = *reinterpret_cast<const uint2 *>(rb);
                    ca[0] = x.x, ca[1] = x.y, cb[0] = y.x, cb[1] = y.y;
                    za = *sa, zb = *sb;
                } else {
#pragma unroll
                    for (int i = 0; i < kKWords / 4; ++i) {
                        const uint4 x = reinterpret_cast<const uint4 *>(ra)[i];
                        const uint4 y = reinterpret_cast<const uint4 *>(rb)[i];
                        ca[4 * i] = x.x, ca[4 * i + 1] = x.y, ca[4 * i + 2] = x.z, ca[4 * i + 3] = x.w;
                        cb[4 * i] = y.x, cb[4 * i + 1] = y.y, cb[4 * i + 2] = y.z, cb[4 * i + 3] = y.w;
                    }
                    if constexpr (D == 128) {
                        za = *reinterpret_cast<const uint16_t *>(sa);
                        zb = *reinterpret_cast<const uint16_t *>(sb);
                    } else {
                        za = *reinterpret_cast<const uint32_t *>(sa);
                        zb = *reinterpret_cast<const uint32_t *>(sb);
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[m][n][j] = 0.0f;
#pragma unroll
                for (int blk = 0; blk < D / 64; ++blk) {   // 16 dimensions, four k-steps
                    const uint32_t s_a = f16x2_of_e4m3x2(((za >> (8 * blk)) & 0xFFu) * 0x101u);
                    const uint32_t s_b = f16x2_of_e4m3x2(((zb >> (8 * blk)) & 0xFFu) * 0x101u);
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
                                mma(sc[m][n], xa[2 * i], xb[2 * i], xa[2 * i + 1], xb[2 * i + 1],
                                    qf[n][ks][0], qf[n][ks][1]);
                            }
                    }
                }
            }

            // ---- running maximum and sum -------------------------------------
            uint32_t pf[2][NT][2];
            bool grew = false;
            float shrink[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float &x = sc[m][n][2 * h + j];
                            x *= c[n][j];
                            if (edge) {
                                const int32_t tok = at + 16 * m + tok_a + 2 * h;
                                if (tok >= see_hi[n][j] || tok < see_lo[n][j]) x = -INFINITY;
                            }
                            mx = fmaxf(mx, x);
                        }
#pragma unroll
                    for (int off = 4; off < 32; off *= 2)
                        mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, off));
                    const float now = fmaxf(top[n][j], mx);
                    // a column that has seen nothing yet keeps exp2(-inf) = 0
                    const float ref = now == -INFINITY ? 0.0f : now;
                    shrink[n][j] = exp2_fast(top[n][j] - ref);
                    grew |= now != top[n][j];
                    top[n][j] = now;
                    float add = 0.0f;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float &x = sc[m][n][2 * h + j];
                            x = exp2_fast(x - (ref - kShift));
                            add += x;
                        }
                    sum[n][j] = sum[n][j] * shrink[n][j] + add;
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        pf[m][n][h] = transpose8x8(f16x2_of(sc[m][n][2 * h], sc[m][n][2 * h + 1]));
            }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int i = 0; i < kMTiles; ++i)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[i][n][j] *= shrink[n][j & 1];
            }

            // ---- O^T += V^T P^T ----------------------------------------------
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const uint8_t *vt = ring + (2 + m) * kTile;
                // blocks of 16 dimensions: with D = 64 two g share one
                constexpr int kBlocksOfLane = D / 128 > 0 ? D / 128 : 1;
#pragma unroll
                for (int blk = 0; blk < kBlocksOfLane; ++blk) {
                    constexpr int kWords = kVWords < 2 ? kVWords : 2;
                    const int32_t block = D == 64 ? g / 2 : g * kBlocksOfLane + blk;
                    uint32_t x[4][kWords];
                    const uint8_t *p = vt + block * 128 + t * 32;
                    if constexpr (kWords == 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i][0] = *reinterpret_cast<const uint32_t *>(p + 8 * i + 4 * (g % 2));
                    } else {
                        const uint4 lo = reinterpret_cast<const uint4 *>(p)[0];
                        const uint4 hi = reinterpret_cast<const uint4 *>(p)[1];
                        x[0][0] = lo.x, x[0][1] = lo.y, x[1][0] = lo.z, x[1][1] = lo.w;
                        x[2][0] = hi.x, x[2][1] = hi.y, x[3][0] = hi.z, x[3][1] = hi.w;
                    }
                    uint32_t z = *reinterpret_cast<const uint32_t *>(vt + 8 * D + block * 16 + 4 * t);
                    if (edge) {                // unwritten tokens may hold any scale byte
                        const int32_t tok = at + 16 * m + 4 * t;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (tok + i >= end) z &= ~(0xFFu << (8 * i));
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
                            const int mt = (blk * kWords + w) * 4 + i;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma(o[mt][n], a0, a1, a2, a3, pf[m][n][0], pf[m][n][1]);
                        }
                    }
                }
            }
            ++drain;
            __syncwarp();                      // every lane has read the stage
            if (k + kStages < steps) issue(k + kStages);
        }

        // ---- join the warps ---------------------------------------------------
        // A warp's copies have all arrived, so its ring is free for its sums:
        // [rows][D], row-major.
        float *mine_o = reinterpret_cast<float *>(sm.ring[warp][0]);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int32_t col = n * 8 + 2 * t + j;
                float l = sum[n][j];
#pragma unroll
                for (int off = 4; off < 32; off *= 2) l += __shfl_xor_sync(0xFFFFFFFFu, l, off);
                if (g == 0) {
                    sm.top[warp][col] = top[n][j];
                    sm.sum[warp][col] = l;
                }
#pragma unroll
                for (int i = 0; i < kMTiles; ++i) {
                    // dimensions of lane g: [g D/8, (g + 1) D/8)
                    *reinterpret_cast<float2 *>(mine_o + col * D + g * (D / 8) + 2 * i) =
                        make_float2(o[i][n][j], o[i][n][2 + j]);
                }
            }
        __syncthreads();
        const bool whole = r0 == 0 && r1 == s.units;
        const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (r0 == 0 ? 1 : 0);
        float *dst = part_at(a.workspace, part, kRows, D);
        if (!whole && r0 == 0 && threadIdx.x == 0) {
            const int64_t last = item_base + s.units - 1;
            record->token0 = s.token0;
            record->row0 = row0;
            record->rows = rows;
            record->head = head;
            record->blocks = static_cast<int32_t>(last / per_block) - blockIdx.x + 1;
        }
        for (int32_t i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
            const int32_t row = i / (D / 2), d = 2 * (i - row * (D / 2));
            float most = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) most = fmaxf(most, sm.top[w][row]);
            const float ref = most == -INFINITY ? 0.0f : most;
            float x = 0.0f, y = 0.0f, l = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = exp2_fast(sm.top[w][row] - ref);
                const float2 v = *reinterpret_cast<const float2 *>(
                    reinterpret_cast<const float *>(sm.ring[w][0]) + row * D + d);
                x += f * v.x;
                y += f * v.y;
                l += f * sm.sum[w][row];
            }
            if (whole) {
                const float inv = l > 0.0f ? v_scale / l : 0.0f;
                const int32_t qi = (row0 + row) / group;
                const int32_t q_head = head * group + (row0 + row - qi * group);
                store_row2(a, s.token0 + qi, q_head, d, D, x * inv, y * inv);
                if (a.lse != nullptr && d == 0)
                    a.lse[static_cast<int64_t>(s.token0 + qi) * a.q_heads + q_head] =
                        l > 0.0f ? kLn2 * (most + (log2f(l) - kShift)) : -INFINITY;
            } else {
                *reinterpret_cast<float2 *>(dst + row * D + d) = make_float2(x, y);
                if (d == 0) {
                    dst[kRows * D + row] = most;
                    dst[kRows * D + kRows + row] = l;
                }
            }
        }
        // the sums are plain reads and writes of memory the next copies fill
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        u += r1 - r0;
    }
}

// ---------------------------------------------------------------------------
// the join: block (c, row) merges row `row` of the item that began in block c

template <int D, int NT>
__global__ void __launch_bounds__(D) fp4_attention_join_kernel(const Fp4Attention a) {
    constexpr int kRows = 8 * NT;
    constexpr int kGroups = 2;                 // threads of a dimension pair
    __shared__ float2 half[D / 2];
    __shared__ float half_sum[2];
    pdl_wait();
    pdl_allow_next();
    float k_scale, v_scale;
    load_scales(a, &k_scale, &v_scale);
    if (!fp4_scale_ok(k_scale) || !fp4_scale_ok(v_scale)) return;
    const int32_t c = blockIdx.x, row = blockIdx.y;
    const Split s = static_cast<const Split *>(a.workspace)[c];
    if (s.blocks == 0 || row >= s.rows) return;
    const int32_t d = 2 * (threadIdx.x % (D / 2)), which = threadIdx.x / (D / 2);
    // part 1 of block c, then part 0 of the blocks behind it
    auto part = [&](int32_t i) {
        return part_at(a.workspace, 2 * static_cast<int64_t>(c + i) + (i == 0 ? 1 : 0), kRows, D);
    };
    float most = -INFINITY;
    for (int32_t i = 0; i < s.blocks; ++i) most = fmaxf(most, part(i)[kRows * D + row]);
    const float ref = most == -INFINITY ? 0.0f : most;
    float x = 0.0f, y = 0.0f, l = 0.0f;
#pragma unroll 4
    for (int32_t i = which; i < s.blocks; i += kGroups) {
        const float *p = part(i);
        const float f = exp2_fast(p[kRows * D + row] - ref);
        const float2 v = *reinterpret_cast<const float2 *>(p + row * D + d);
        x += f * v.x;
        y += f * v.y;
        l += f * p[kRows * D + kRows + row];
    }
    if (which == 1) {
        half[d / 2] = make_float2(x, y);
        if (d == 0) half_sum[0] = l;
    }
    __syncthreads();
    if (which == 1) return;
    x += half[d / 2].x;
    y += half[d / 2].y;
    l += half_sum[0];
    const int32_t group = a.q_heads / a.pools.heads;
    const int32_t qi = (s.row0 + row) / group;
    const int32_t q_head = s.head * group + (s.row0 + row - qi * group);
    const float inv = l > 0.0f ? v_scale / l : 0.0f;
    store_row2(a, s.token0 + qi, q_head, d, D, x * inv, y * inv);
    if (a.lse != nullptr && d == 0)
        a.lse[static_cast<int64_t>(s.token0 + qi) * a.q_heads + q_head] =
            l > 0.0f ? kLn2 * (most + (log2f(l) - kShift)) : -INFINITY;
}

// ---------------------------------------------------------------------------
// launch

// Rows of a tile (8 * NT) for an average of `rows` rows a sequence: the
// smallest tile that holds them, up to what the accumulators leave room for
// in registers (NT * D <= 256).
int tiles_of(int64_t batch, int64_t num_tokens, int32_t group, int32_t dim) {
    const int64_t rows = (num_tokens + batch - 1) / batch * group;
    int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
    while (nt * dim > 256) nt /= 2;
    return nt;
}

template <int D, int NT>
cudaError_t launch_tiles(const Fp4Attention &a, cudaStream_t stream) {
    constexpr size_t kSmem = sizeof(Shared<D, NT>);
    // Blocks an SM holds: by shared memory, and registers for at most 12 warps.
    constexpr int kResident = 3 * (kSmem + 1024) <= 228 * 1024 ? 3
                              : 2 * (kSmem + 1024) <= 228 * 1024 ? 2 : 1;
    auto kernel = fp4_attention_kernel<D, NT>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmem));
    if (e != cudaSuccess) return e;
    // No more blocks than there can be units.
    const int32_t group = a.q_heads / a.pools.heads;
    const int64_t row_tiles = (static_cast<int64_t>(a.num_tokens) * group + 8 * NT - 1) / (8 * NT) +
                              a.batch;
    const int64_t longest = (a.table_width * a.pools.tiles * 16 + kUnit - 1) / kUnit + 1;
    int64_t grid = static_cast<int64_t>(sms) * kResident;
    if (grid > kMaxBlocks) grid = kMaxBlocks;
    if (row_tiles * a.pools.heads < grid && row_tiles * a.pools.heads * longest < grid)
        grid = row_tiles * a.pools.heads * longest;
    e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), kThreads, kSmem, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(fp4_attention_join_kernel<D, NT>, dim3(static_cast<unsigned>(grid), 8 * NT), D,
                      0, stream, a);
}

}  // namespace

int64_t fp4_attention_workspace(int64_t batch, int64_t num_tokens, int32_t q_heads,
                                int32_t kv_heads, int32_t dim) {
    if (batch == 0) return 0;
    const int nt = tiles_of(batch, num_tokens, q_heads / kv_heads, dim);
    return kMaxBlocks * (static_cast<int64_t>(sizeof(Split)) + 2 * 4 * part_floats(8 * nt, dim));
}

cudaError_t launch_fp4_attention(const Fp4Attention &a, cudaStream_t stream) {
    const int nt = tiles_of(a.batch, a.num_tokens, a.q_heads / a.pools.heads, a.pools.dim);
    switch (a.pools.dim) {
    case 64:
        return nt == 1 ? launch_tiles<64, 1>(a, stream)
               : nt == 2 ? launch_tiles<64, 2>(a, stream) : launch_tiles<64, 4>(a, stream);
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
