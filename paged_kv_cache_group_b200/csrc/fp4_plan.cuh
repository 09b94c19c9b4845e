// How attention over the 4-bit cache is divided among the blocks of a launch.
//
// An item is one (sequence, set of KV heads, tile of query rows).  It is made
// of units of some cached tokens, counted from the first token its own rows
// see, and costs its units plus what loading its rows and finishing its sums take,
// in units.  Items are laid side by side on one axis, every block takes an equal
// run of it, and unit j of an item lies at the point item start + that cost + j.  A block finds its run from the lengths on the
// device, so a launch depends on sizes alone and may be captured.
//
// An item whose units lie in several blocks leaves one part in each: blocks
// behind the first leave part 0, the first one part 1 and a record of the item,
// from which the join merges the parts in a fixed order.
#pragma once

#include "fp4_device.cuh"

namespace fp8q {
namespace fp4_plan {

constexpr int kMaxBlocks = 444;        // blocks a workspace has room for

// How a kernel divides its work.
struct Division {
    int32_t group;       // query heads of a KV head
    int32_t tile_rows;   // rows of a tile
    int32_t sets;        // sets of KV heads
    int32_t unit;        // cached tokens of a unit
    int32_t item_cost;   // units an item costs beside its own
    int32_t window;
    int32_t whole;       // 0: items are split where runs end; 1: they are not;
                         // 2: only those that cost more than a run
};

// One sequence as the kernels see it: bad lengths and ranges are cut to what
// the buffers hold and reported.
struct Sequence {
    int32_t token0;     // first new token
    int32_t news;       // new tokens
    int32_t length;     // cached tokens, the new ones included
    int32_t row_tiles;
};

__device__ __forceinline__ Sequence sequence(const Fp4Attention &a, const Division &d, int32_t b,
                                             bool *bad) {
    Sequence s;
    int64_t t0 = b, t1 = b + 1;
    if (a.q_start != nullptr) {
        t0 = a.q_start[b];
        t1 = a.q_start[b + 1];
    }
    int64_t length = a.seq_lens[b];
    if (t0 < 0 || t1 < t0 || t1 > a.num_tokens) {
        *bad = true;
        t0 = t0 < 0 ? 0 : t0;
        t1 = t1 > a.num_tokens ? a.num_tokens : t1;
        if (t1 < t0) t0 = t1 = 0;
    }
    const int64_t room = a.pools.num_blocks > 0 ? a.table_width * (a.pools.tiles * 16) : 0;
    if (length < 0 || length > room) {
        *bad = true;
        length = length < 0 ? 0 : room;
    }
    s.token0 = static_cast<int32_t>(t0);
    s.news = static_cast<int32_t>(t1 - t0);
    s.length = static_cast<int32_t>(length);
    // rows of a call stay within 2^30
    s.row_tiles = (s.news * d.group + d.tile_rows - 1) / d.tile_rows;
    return s;
}

// a / b for a >= 0, b > 0: places on the axis hardly ever need 64 bits.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The rows of one tile of a sequence and the cached tokens they see.
struct Tile {
    int32_t row0, rows;
    int32_t first;      // the first token any row sees
    int32_t begin;      // ... rounded down to 32 slots: where units count from
    int32_t end;        // behind the last token any row sees; >= begin
    int32_t units;      // at least one
};

__device__ __forceinline__ Tile tile_of(const Sequence &s, const Division &d, int32_t rt) {
    Tile x;
    x.row0 = rt * d.tile_rows;
    x.rows = min(d.tile_rows, s.news * d.group - x.row0);
    const int32_t ahead = s.length - s.news;   // query i sees tokens up to ahead + i
    const int32_t q_lo = s.news > 1 ? x.row0 / d.group : 0;
    const int32_t q_hi = s.news > 1 ? (x.row0 + x.rows - 1) / d.group : 0;
    x.first = d.window > 0 ? max(0, ahead + q_lo + 1 - d.window) : 0;
    x.begin = x.first & ~31;
    x.end = max(x.begin, min(s.length, ahead + q_hi + 1));
    x.units = max(1, (x.end - x.begin + d.unit - 1) / d.unit);
    return x;
}

// Cost of all row tiles of one set of heads, of a whole warp's sequences at once: few
// tiles are summed by the lane that has the sequence, many by all lanes.
__device__ __forceinline__ int64_t set_cost(const Sequence &mine, const Division &d) {
    constexpr int32_t kFew = 4;
    const int32_t lane = threadIdx.x % 32;
    int64_t cost = 0;
    if (mine.row_tiles <= kFew)
        for (int32_t rt = 0; rt < mine.row_tiles; ++rt)
            cost += tile_of(mine, d, rt).units + d.item_cost;
    for (uint32_t many = __ballot_sync(0xFFFFFFFFu, mine.row_tiles > kFew); many; many &= many - 1) {
        const int32_t from = __ffs(many) - 1;
        Sequence s;
        s.token0 = 0;
        s.news = __shfl_sync(0xFFFFFFFFu, mine.news, from);
        s.length = __shfl_sync(0xFFFFFFFFu, mine.length, from);
        s.row_tiles = __shfl_sync(0xFFFFFFFFu, mine.row_tiles, from);
        int64_t sum = 0;
        for (int32_t rt = lane; rt < s.row_tiles; rt += 32)
            sum += tile_of(s, d, rt).units + d.item_cost;
#pragma unroll
        for (int o = 16; o > 0; o /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane == from) cost = sum;
    }
    return cost;
}

template <int kWarps>
struct PlanShared {
    int64_t scan[kWarps];
    int64_t base, cost;
    Sequence s;
    int32_t seq;
};

// A block's run of the axis and where it starts.
struct Run {
    int64_t at, end;     // [at, end); empty: no work
    int64_t per_block;
    int64_t base;        // start of sequence `seq` on the axis
    int64_t cost;        // of one of its sets of heads
    Sequence s;
    int32_t seq;
};

// Called by all kWarps warps of the block; holds two block barriers (one when
// the run is empty).
template <int kWarps>
__device__ __forceinline__ Run block_run(const Fp4Attention &a, const Division &d, uint32_t *error,
                                         PlanShared<kWarps> &sm) {
    constexpr int32_t kThreads = 32 * kWarps;
    const int32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int32_t per_thread = (a.batch + kThreads - 1) / kThreads;
    const int64_t b0 = static_cast<int64_t>(threadIdx.x) * per_thread;
    bool bad = false;
    auto look = [&](int32_t i) {
        Sequence s;
        s.token0 = s.news = s.length = s.row_tiles = 0;
        if (b0 + i < a.batch) s = sequence(a, d, static_cast<int32_t>(b0 + i), &bad);
        return s;
    };
    Sequence s = look(0);                      // most often the only one
    int64_t cost = set_cost(s, d), mine = cost * d.sets;
    for (int32_t i = 1; i < per_thread; ++i) mine += set_cost(look(i), d) * d.sets;
    if (bad) atomicOr(error, kFp4ErrSequence);
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
    Run r;
    r.per_block = quotient(total + gridDim.x - 1, gridDim.x);
    r.at = r.per_block * blockIdx.x;
    r.end = min(total, r.at + r.per_block);
    r.seq = 0;
    r.base = r.cost = 0;
    if (r.at >= r.end) return r;
    const bool here = mine > 0 && before <= r.at && r.at < before + mine;
    if (__any_sync(0xFFFFFFFFu, here)) {
        for (int32_t i = 0;; ++i) {
            if (here && before <= r.at && r.at < before + cost * d.sets) {
                sm.seq = static_cast<int32_t>(b0 + i);
                sm.base = before;
                sm.cost = cost;
                sm.s = s;
            }
            if (i + 1 >= per_thread) break;
            before += cost * d.sets;
            s = look(i + 1);
            cost = set_cost(s, d);
        }
    }
    __syncthreads();
    r.seq = sm.seq;
    r.base = sm.base;
    r.cost = sm.cost;
    r.s = sm.s;
    return r;
}

// Walks the items of a run, one warp; every lane holds the same state.
struct Walk {
    Sequence s;
    int32_t seq, set, rt;
    int64_t start;      // of the item on the axis

    __device__ __forceinline__ void begin(const Division &d, const Run &r) {
        const int32_t lane = threadIdx.x % 32;
        seq = r.seq;
        s = r.s;
        set = static_cast<int32_t>(quotient(r.at - r.base, r.cost));
        start = r.base + set * r.cost;
        rt = 0;
        for (int32_t first = 0; s.row_tiles > 1; first += 32) {   // the tile that holds r.at
            int32_t n = 0;
            if (first + lane < s.row_tiles)
                n = tile_of(s, d, first + lane).units + d.item_cost;
            int64_t incl = n;
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int64_t up = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += up;
            }
            const uint32_t beyond = __ballot_sync(0xFFFFFFFFu, n > 0 && start + incl > r.at);
            if (beyond) {
                const int32_t at = __ffs(beyond) - 1;
                rt = first + at;
                start += __shfl_sync(0xFFFFFFFFu, incl - n, at);
                return;
            }
            start += __shfl_sync(0xFFFFFFFFu, incl, 31);
            if (first + 32 >= s.row_tiles) return;    // not reached: the run starts in this set
        }
    }

    // To the next item; `cost` is the present one's.  False behind the last.
    __device__ __forceinline__ bool next(const Fp4Attention &a, const Division &d, int64_t cost) {
        start += cost;
        if (++rt < s.row_tiles) return true;
        rt = 0;
        if (++set < d.sets) return true;
        set = 0;
        bool bad = false;
        do {
            if (++seq >= a.batch) return false;
            s = sequence(a, d, seq, &bad);
        } while (s.row_tiles == 0);
        return true;
    }
};

// A block's record of the item that begins in it and goes on in the blocks
// behind it.
struct Split {
    int32_t blocks;     // blocks that hold a part of the item; 0: no such item
    int32_t token0, row0, rows, set;
};

// Workspace: Split [kMaxBlocks], then two parts for each block: for each head
// of the set rows x dim sums, rows maxima and rows sums of weights.
__host__ __device__ constexpr int64_t part_floats(int rows, int dim) {
    return static_cast<int64_t>(rows) * (dim + 2);
}
constexpr int64_t kRecordBytes = (kMaxBlocks * sizeof(Split) + 15) / 16 * 16;

__device__ __forceinline__ float *part_at(void *workspace, int64_t index, int64_t floats) {
    return reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + kRecordBytes) +
           index * floats;
}

}  // namespace fp4_plan
}  // namespace fp8q
