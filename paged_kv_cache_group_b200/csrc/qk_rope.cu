// qk_rope.cu -- norms of queries and keys for each head with the position
// rotation in the same pass (sm_100a).
//
// For each token and head, in fp32, rounded once at the end:
//     y = x * rsqrt(mean(x^2) + eps) * w          (y = x without a weight)
//     (a, b) -> (a cos - b sin, b cos + a sin)    for the rotary pairs of y
// with (a, b) = (y[i], y[i + rotary/2]) in the half layout and
// (y[2i], y[2i + 1]) interleaved, and the angle position * inv_freq[i].  At
// positions of a million an fp32 angle is off by up to 0.06 rad, so the turn
// count position * inv_freq / 2pi is formed and reduced in fp64; cosine and
// sine of the remaining half turn are fp32.
//
// Bound by memory traffic: 2 bytes in and 2 out an element.  There is no
// cosine table to read: a block computes the pairs of its few tokens once
// into shared memory and all heads of those tokens use them.
#include <cuda_runtime.h>

#include "fp4_device.cuh"

namespace fp8q {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 4;      // tokens of a block

// A lane's eight elements of a head as two runs of four: `first` and
// `second` start elements, and the first rotary pair they belong to (-1:
// passed through).
struct LanePlace {
    int32_t first, second, pair;
};

template <bool kInterleaved>
__device__ __forceinline__ LanePlace lane_place(int32_t lane, int32_t rotary) {
    const bool turned = lane * 8 < rotary;
    if (kInterleaved || !turned) return {8 * lane, 8 * lane + 4, turned ? 4 * lane : -1};
    return {4 * lane, rotary / 2 + 4 * lane, 4 * lane};
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const QkNormRope p,
                                                                int32_t tokens_per_block,
                                                                int32_t parts) {
    constexpr int kLanes = D / 8;               // lanes of one head
    constexpr int kGroups = kThreads / kLanes;  // heads in flight in the block
    __shared__ float2 turns[kMaxTokens][D / 2];
    pdl_wait();
    pdl_allow_next();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / parts) * tokens_per_block;
    const int32_t part = blockIdx.x % parts;
    const int32_t tokens = static_cast<int32_t>(
        p.num_tokens - t0 < tokens_per_block ? p.num_tokens - t0 : tokens_per_block);
    const int32_t half = p.rotary / 2;
    for (int32_t i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int32_t t = i / half, j = i - t * half;
        double u = static_cast<double>(p.positions[t0 + t]) * p.inv_freq[j] *
                   0.15915494309189533577;   // turns: angle / 2pi
        u -= rint(u);
        float sn, cs;
        sincospif(2.0f * static_cast<float>(u), &sn, &cs);
        turns[t][j] = make_float2(cs * p.rope_scale, sn * p.rope_scale);
    }
    __syncthreads();

    const int32_t lane = threadIdx.x % kLanes;
    const LanePlace at = lane_place<kInterleaved>(lane, p.rotary);
    const int32_t heads = p.q_heads + p.k_heads;
    const int32_t items = tokens * heads;
    // Every thread of a warp runs the same number of passes, for the shuffles;
    // a pass is kUnroll heads, all fetched before the first is used.
    constexpr int kUnroll = 4;
    const int32_t step = kGroups * parts;
    for (int32_t base = part * kGroups; base < items; base += kUnroll * step) {
        uint2 first[kUnroll], second[kUnroll];
        uint16_t *dst[kUnroll];
        int32_t token[kUnroll];                 // in the block; -1: no item
        bool is_q[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t item = base + u * step + threadIdx.x / kLanes;
            first[u] = second[u] = make_uint2(0, 0);
            token[u] = -1;
            if (item < items) {
                const int32_t t = tokens == 1 ? 0 : item / heads, h = item - t * heads;
                is_q[u] = h < p.q_heads;
                const int64_t row = t0 + t;
                const int32_t head = is_q[u] ? h : h - p.q_heads;
                const uint16_t *src =
                    (is_q[u] ? p.q + row * p.q_stride : p.k + row * p.k_stride) + head * D;
                dst[u] = (is_q[u] ? p.q_out + row * p.q_out_stride : p.k_out + row * p.k_out_stride) + head * D;
                token[u] = t;
                first[u] = *reinterpret_cast<const uint2 *>(src + at.first);
                second[u] = *reinterpret_cast<const uint2 *>(src + at.second);
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const uint2 a = first[u], b = second[u];
            float x[8] = {bf16_low(a.x), bf16_high(a.x), bf16_low(a.y), bf16_high(a.y),
                          bf16_low(b.x), bf16_high(b.x), bf16_low(b.y), bf16_high(b.y)};
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
            for (int o = kLanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (token[u] < 0) continue;
            const uint16_t *weight = is_q[u] ? p.q_weight : p.k_weight;
            if (weight != nullptr) {
                const float n = rsqrtf(sum * (1.0f / D) + p.eps);
                const uint2 wa = *reinterpret_cast<const uint2 *>(weight + at.first);
                const uint2 wb = *reinterpret_cast<const uint2 *>(weight + at.second);
                const float w[8] = {bf16_low(wa.x), bf16_high(wa.x), bf16_low(wa.y), bf16_high(wa.y),
                                    bf16_low(wb.x), bf16_high(wb.x), bf16_low(wb.y), bf16_high(wb.y)};
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * n * w[i];
            }
            if (at.pair >= 0) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 cs = turns[token[u]][at.pair + i];
                    const int s = kInterleaved ? 2 * i : i, v = kInterleaved ? 2 * i + 1 : i + 4;
                    const float c = x[s], e = x[v];
                    x[s] = c * cs.x - e * cs.y;
                    x[v] = e * cs.x + c * cs.y;
                }
            }
            *reinterpret_cast<uint2 *>(dst[u] + at.first) =
                make_uint2(bf16x2_of(x[0], x[1]), bf16x2_of(x[2], x[3]));
            *reinterpret_cast<uint2 *>(dst[u] + at.second) =
                make_uint2(bf16x2_of(x[4], x[5]), bf16x2_of(x[6], x[7]));
        }
    }
}

template <int D>
cudaError_t launch_dim(const QkNormRope &r, cudaStream_t stream) {
    constexpr int kGroups = kThreads / (D / 8);
    auto kernel = r.interleaved ? qk_norm_rope_kernel<D, true> : qk_norm_rope_kernel<D, false>;
    const int64_t heads = static_cast<int64_t>(r.q_heads) + r.k_heads;
    // Enough blocks to fill the GPU: fewer tokens a block first, then the
    // heads of a token split over several blocks.
    constexpr int64_t kFull = 148 * 8;
    int64_t per_block = r.num_tokens / kFull;
    per_block = per_block < 1 ? 1 : per_block > kMaxTokens ? kMaxTokens : per_block;
    const int64_t groups = (r.num_tokens + per_block - 1) / per_block;
    int64_t parts = kFull / groups;
    const int64_t most = (per_block * heads + kGroups - 1) / kGroups;
    parts = parts < 1 ? 1 : parts > most ? most : parts;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(groups * parts)), kThreads, 0, stream, r,
                      static_cast<int32_t>(per_block), static_cast<int32_t>(parts));
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRope &r, cudaStream_t stream) {
    return r.dim == 64    ? launch_dim<64>(r, stream)
           : r.dim == 128 ? launch_dim<128>(r, stream)
                          : launch_dim<256>(r, stream);
}

}  // namespace fp8q
