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
// Bound by memory traffic, 2 bytes in and 2 out an element, and nearly by
// instructions: about 56 for a lane's eight elements.  A warp keeps one token,
// so that its lanes' cosines and sines stay in registers for all heads of q and
// k (there is no table to read), as do the weights; pairs of values are
// multiplied and added at once.  Several warps share a token where there are
// few of them.
//
// Measured: 4593 tokens x 36 heads of 128 in 19.0 us (4.4 TB/s; 25.9 with the
// turns in shared memory and four tokens a block), 16 tokens in 2.9 us.
#include <cuda_runtime.h>

#include "fp4_device.cuh"

namespace fp8q {

namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 2;         // heads of a lane under way

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

// Two fp32 values in one 64-bit register.
struct Two {
    uint64_t v;
    __device__ __forceinline__ Two() {}
    __device__ __forceinline__ Two(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ float x() const { return __uint_as_float(static_cast<uint32_t>(v)); }
    __device__ __forceinline__ float y() const { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
};
__device__ __forceinline__ Two mul2(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ Two two_of(uint32_t bf16_pair) { return Two(bf16_low(bf16_pair), bf16_high(bf16_pair)); }
__device__ __forceinline__ uint32_t bf16_of(Two a) { return bf16x2_of(a.x(), a.y()); }

// What turns a lane's eight elements: for the half layout cosines, minus sines
// and sines of pairs 0, 1 and 2, 3; interleaved the same of one pair each.
template <bool kInterleaved>
struct Turn {
    Two c[kInterleaved ? 4 : 2], s[kInterleaved ? 4 : 2], minus_s[kInterleaved ? 1 : 2];
};

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 8) qk_norm_rope_kernel(const QkNormRope p, int32_t parts) {
    constexpr int kLanes = D / 8;               // lanes of one head
    constexpr int kCopies = 32 / kLanes;        // heads of a warp's pass
    pdl_wait();
    pdl_allow_next();
    const uint32_t warp = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    const int32_t lane = threadIdx.x % 32, copy = lane / kLanes;
    const uint32_t part = warp % static_cast<uint32_t>(parts);
    const int64_t token = warp / static_cast<uint32_t>(parts);
    if (token >= p.num_tokens) return;          // the whole warp
    const LanePlace at = lane_place<kInterleaved>(lane % kLanes, p.rotary);

    // A batch of heads, `step` apart; the first of q is under way while the
    // angles are made.
    const int32_t step = parts * kCopies, mine = static_cast<int32_t>(part) * kCopies + copy;
    uint2 lo[kUnroll], hi[kUnroll];
    auto fetch = [&](const uint16_t *src, int32_t first, int32_t heads) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int32_t h = first + u * step;
            lo[u] = hi[u] = make_uint2(0, 0);
            if (h < heads) {
                lo[u] = *reinterpret_cast<const uint2 *>(src + h * D + at.first);
                hi[u] = *reinterpret_cast<const uint2 *>(src + h * D + at.second);
            }
        }
    };
    const uint16_t *q = p.q + token * p.q_stride, *k = p.k + token * p.k_stride;
    const double position = static_cast<double>(p.positions[token]);
    fetch(q, mine, p.q_heads);

    // Cosines and sines of the token's pairs, shared out over the lanes.
    Turn<kInterleaved> turn;
    {
        __shared__ alignas(16) float2 turns[kThreads / 32][D / 2];
        float2 (&mine_turns)[D / 2] = turns[threadIdx.x / 32];
        for (int32_t j = lane; j < p.rotary / 2; j += 32) {
            double u = position * p.inv_freq[j] * 0.15915494309189533577;   // turns: angle / 2pi
            u -= rint(u);
            float sn, cs;
            sincospif(2.0f * static_cast<float>(u), &sn, &cs);
            mine_turns[j] = make_float2(cs * p.rope_scale, sn * p.rope_scale);
        }
        __syncwarp();
        float cs[4], sn[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = sn[i] = 0.0f;
        if (at.pair >= 0) {
            const float4 a = reinterpret_cast<const float4 *>(mine_turns)[at.pair / 2];
            const float4 b = reinterpret_cast<const float4 *>(mine_turns)[at.pair / 2 + 1];
            cs[0] = a.x, sn[0] = a.y, cs[1] = a.z, sn[1] = a.w;
            cs[2] = b.x, sn[2] = b.y, cs[3] = b.z, sn[3] = b.w;
        }
#pragma unroll
        for (int i = 0; i < (kInterleaved ? 4 : 2); ++i) {
            if (kInterleaved) {
                turn.c[i] = Two(cs[i], cs[i]);
                turn.s[i] = Two(-sn[i], sn[i]);
            } else {
                turn.c[i] = Two(cs[2 * i], cs[2 * i + 1]);
                turn.s[i] = Two(sn[2 * i], sn[2 * i + 1]);
                turn.minus_s[i] = Two(-sn[2 * i], -sn[2 * i + 1]);
            }
        }
    }

    auto heads_of = [&](const uint16_t *src, uint16_t *dst, int32_t heads, const uint16_t *weight) {
        Two w[4];
        if (weight != nullptr) {
            const uint2 a = *reinterpret_cast<const uint2 *>(weight + at.first);
            const uint2 b = *reinterpret_cast<const uint2 *>(weight + at.second);
            w[0] = two_of(a.x), w[1] = two_of(a.y), w[2] = two_of(b.x), w[3] = two_of(b.y);
        }
        // Every lane runs the same passes, for the shuffles.
        for (int32_t first = mine; first - copy < heads;) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int32_t h = first + u * step;
                Two x[4] = {two_of(lo[u].x), two_of(lo[u].y), two_of(hi[u].x), two_of(hi[u].y)};
                if (weight != nullptr) {
                    Two sums = mul2(x[0], x[0]);
#pragma unroll
                    for (int i = 1; i < 4; ++i) sums = fma2(x[i], x[i], sums);
                    float sum = sums.x() + sums.y();
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                    const float n = rsqrtf(sum * (1.0f / D) + p.eps);
                    const Two nn(n, n);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = mul2(mul2(x[i], nn), w[i]);
                }
                if (at.pair >= 0) {
                    if (kInterleaved) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[i] = fma2(Two(x[i].y(), x[i].x()), turn.s[i], mul2(x[i], turn.c[i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const Two a = x[i], b = x[2 + i];
                            x[i] = fma2(b, turn.minus_s[i], mul2(a, turn.c[i]));
                            x[2 + i] = fma2(a, turn.s[i], mul2(b, turn.c[i]));
                        }
                    }
                }
                if (h < heads) {
                    *reinterpret_cast<uint2 *>(dst + h * D + at.first) = make_uint2(bf16_of(x[0]), bf16_of(x[1]));
                    *reinterpret_cast<uint2 *>(dst + h * D + at.second) = make_uint2(bf16_of(x[2]), bf16_of(x[3]));
                }
            }
            first += kUnroll * step;
            if (first - copy < heads) fetch(src, first, heads);
        }
    };
    heads_of(q, p.q_out + token * p.q_out_stride, p.q_heads, p.q_weight);
    fetch(k, mine, p.k_heads);
    heads_of(k, p.k_out + token * p.k_out_stride, p.k_heads, p.k_weight);
}

template <int D>
cudaError_t launch_dim(QkNormRope r, cudaStream_t stream) {
    constexpr int kCopies = 256 / D;
    auto kernel = r.interleaved ? qk_norm_rope_kernel<D, true> : qk_norm_rope_kernel<D, false>;
    // Warps of a token: as many as fill the GPU, up to one pass of a head each.
    constexpr int64_t kFull = 148 * 32;
    const int64_t most = ((r.q_heads > r.k_heads ? r.q_heads : r.k_heads) + kCopies - 1) / kCopies;
    int64_t parts = kFull / r.num_tokens;
    parts = parts < 1 ? 1 : parts > most ? most : parts;
    // Warp indexes are 32 bits inside a launch.
    const int64_t chunk = (int64_t{1} << 30) / parts;
    for (int64_t left = r.num_tokens; left > 0; left -= chunk) {
        r.num_tokens = left < chunk ? left : chunk;
        const int64_t blocks = (r.num_tokens * parts + kThreads / 32 - 1) / (kThreads / 32);
        const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), kThreads, 0, stream, r,
                                         static_cast<int32_t>(parts));
        if (e != cudaSuccess) return e;
        r.positions += chunk;
        r.q += chunk * r.q_stride;
        r.k += chunk * r.k_stride;
        r.q_out += chunk * r.q_out_stride;
        r.k_out += chunk * r.k_out_stride;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const QkNormRope &r, cudaStream_t stream) {
    return r.dim == 64    ? launch_dim<64>(r, stream)
           : r.dim == 128 ? launch_dim<128>(r, stream)
                          : launch_dim<256>(r, stream);
}

}  // namespace fp8q
