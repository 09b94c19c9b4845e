// fp4_kv.cu -- K and V quantised to 4 bits as they are scattered into a paged
// cache, and gathered back as bf16 (sm_100a).
//
// A block of 16 neighbouring dimensions of one token's head shares an E4M3
// scale b under the tensor's fp32 scale s; with amax the block's largest |x|:
//     b = E4M3(RN(RN(amax / 6) / s)),  d = RN(b * s),  r = RN(1 / d)  (0 if d = 0)
//     code = E2M1(RN(x * r));          value = RN(code * b * s) -> bf16
// code * b has at most six significant bits and lies in [2^-10, 2688], so it
// is exact in fp16; only the product with s and the bf16 result round.
//
// Both kernels are bound by memory traffic: 2 bytes of bf16 on one side and
// 9/16 byte of cache on the other, with about two instructions an element.
// One thread owns one 16-element block of K and the same block of V: four
// 16-byte accesses in flight on the bf16 side, an 8-byte code word and a
// scale byte on the cache side, and no exchange between threads.  A warp takes
// one head of four neighbouring tokens (eight with 64 dimensions), so that V's
// code words, which lie by block and then by token, fill whole sectors: one
// token a warp asked for four times the sectors.
//
// Measured: 60001 tokens x 8 heads of 64 read in 30.7 us (5.1 TB/s, 40.5 with
// one token a warp); 4593 tokens x 4 heads of 128 written and read back in 9.4
// to 10.4 us, by GPU, for 24 MB: two launches that are mostly latency.
#include <cuda_runtime.h>

#include "fp4_device.cuh"

namespace fp8q {

namespace {

__device__ uint32_t g_fp4_kv_error;

constexpr int kThreads = 256;

// Where a block's code word and scale byte lie in a pool's tile of 16 tokens:
// K token-major, V block-major (the layouts attention reads fragments from).
struct BlockPlace {
    int64_t tile;        // byte offset of the tile in the pool
    uint32_t k_code, k_scale, v_code, v_scale;
};

template <int D>
__device__ __forceinline__ BlockPlace block_place(const Fp4Pools &p, int64_t slot, int32_t head,
                                                  int32_t block) {
    const int32_t block_size = p.tiles * 16;
    int64_t page;
    if ((block_size & (block_size - 1)) == 0)
        page = slot >> (__ffs(block_size) - 1);
    else if (slot >> 32 == 0)
        page = static_cast<uint32_t>(slot) / static_cast<uint32_t>(block_size);
    else
        page = slot / block_size;
    const int32_t off = static_cast<int32_t>(slot - page * block_size);
    const uint32_t tok = off & 15;
    BlockPlace b;
    b.tile = page * p.block_stride + (static_cast<int64_t>(head) * p.tiles + (off >> 4)) * (9 * D);
    b.k_code = tok * (D / 2) + block * 8;
    b.k_scale = 8 * D + tok * (D / 16) + block;
    b.v_code = block * 128 + tok * 8;
    b.v_scale = 8 * D + block * 16 + tok;
    return b;
}

// The work of a thread: a warp is kTokens tokens x kAcross blocks of one head.
template <int D>
struct Share {
    static constexpr int kBlocks = D / 16;
    static constexpr int kAcross = kBlocks < 8 ? kBlocks : 8;
    static constexpr int kTokens = 32 / kAcross;
    static constexpr int kParts = kBlocks / kAcross;    // warps of a head's tokens
    uint32_t token;
    int32_t head, block;

    __device__ __forceinline__ explicit Share(int32_t heads) {
        const uint32_t warp = blockIdx.x * (kThreads / 32) + threadIdx.x / 32, lane = threadIdx.x % 32;
        const uint32_t row = warp / kParts;             // (token group, head)
        const uint32_t group = row / static_cast<uint32_t>(heads);
        token = group * kTokens + lane / kAcross;
        head = static_cast<int32_t>(row - group * static_cast<uint32_t>(heads));
        block = static_cast<int32_t>(warp % kParts * kAcross + lane % kAcross);
    }
    static int64_t warps(int64_t tokens, int64_t heads) {
        return (tokens + kTokens - 1) / kTokens * heads * kParts;
    }
};

__device__ __forceinline__ void load_scales(const Fp4Pools &p, float *ks, float *vs) {
    *ks = p.scale_dev ? p.scale_dev[0] : p.k_scale;
    *vs = p.scale_dev ? p.scale_dev[1] : p.v_scale;
}

// 16 bf16 values (two 16-byte words) to a code word and a scale byte.
__device__ __forceinline__ uint2 quantise16(const uint4 &a, const uint4 &b, float scale,
                                            uint32_t *scale_code) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float x[16];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16_low(w[i]);
        x[2 * i + 1] = bf16_high(w[i]);
        amax = fmaxf(amax, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
    }
    const float t = __fdiv_rn(__fdiv_rn(amax, 6.0f), scale);
    unsigned short code;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(code) : "f"(0.0f), "f"(t));
    *scale_code = code & 0xFFu;
    float block_scale;
    {
        const uint32_t h = f16x2_of_e4m3x2(code) & 0xFFFFu;
        asm("cvt.f32.f16 %0, %1;" : "=f"(block_scale) : "h"(static_cast<unsigned short>(h)));
    }
    const float d = __fmul_rn(block_scale, scale);
    const float r = d > 0.0f ? __frcp_rn(d) : 0.0f;
    float lo[8], hi[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo[i] = __fmul_rn(x[i], r);
        hi[i] = __fmul_rn(x[8 + i], r);
    }
    return make_uint2(e2m1x8_of(lo), e2m1x8_of(hi));
}

template <int D>
__global__ void __launch_bounds__(kThreads) fp4_write_kernel(const Fp4Rows r, const Fp4Pools p) {
    pdl_wait();
    pdl_allow_next();
    const Share<D> me(p.heads);
    if (me.token >= r.num_tokens) return;
    // the rows do not wait for the slot
    const int64_t slot = r.slots[me.token];
    const int32_t e = me.head * D + me.block * 16;
    const uint4 *k = reinterpret_cast<const uint4 *>(r.k + me.token * r.key_stride + e);
    const uint4 *v = reinterpret_cast<const uint4 *>(r.v + me.token * r.value_stride + e);
    const uint4 k0 = __ldcs(k), k1 = __ldcs(k + 1), v0 = __ldcs(v), v1 = __ldcs(v + 1);
    float ks, vs;
    load_scales(p, &ks, &vs);
    if (slot < 0) return;
    if (slot >= p.num_blocks * (p.tiles * 16)) {
        atomicOr(&g_fp4_kv_error, kFp4ErrSlot);
        return;
    }
    const BlockPlace at = block_place<D>(p, slot, me.head, me.block);
    const bool k_ok = fp4_scale_ok(ks), v_ok = fp4_scale_ok(vs);
    if (!k_ok || !v_ok) atomicOr(&g_fp4_kv_error, kFp4ErrScale);
    uint32_t sc;
    if (k_ok) {
        const uint2 c = quantise16(k0, k1, ks, &sc);
        *reinterpret_cast<uint2 *>(p.k + at.tile + at.k_code) = c;
        p.k[at.tile + at.k_scale] = static_cast<uint8_t>(sc);
    }
    if (v_ok) {
        const uint2 c = quantise16(v0, v1, vs, &sc);
        *reinterpret_cast<uint2 *>(p.v + at.tile + at.v_code) = c;
        p.v[at.tile + at.v_scale] = static_cast<uint8_t>(sc);
    }
}

__device__ __forceinline__ void dequantise16(uint2 codes, uint32_t scale_code, float scale,
                                             uint4 *a, uint4 *b) {
    const uint32_t s2 = f16x2_of_e4m3x2(scale_code | scale_code << 8);
    uint32_t w[8];
    uint32_t h[4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        f16x2_of_e2m1x8(half ? codes.y : codes.x, h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t m = mul_f16x2(h[i], s2);
            float lo, hi;
            asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
                "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(lo), "=f"(hi) : "r"(m));
            w[4 * half + i] = bf16x2_of(__fmul_rn(lo, scale), __fmul_rn(hi, scale));
        }
    }
    *a = make_uint4(w[0], w[1], w[2], w[3]);
    *b = make_uint4(w[4], w[5], w[6], w[7]);
}

template <int D>
__global__ void __launch_bounds__(kThreads) fp4_read_kernel(const Fp4Rows r, const Fp4Pools p) {
    pdl_wait();
    pdl_allow_next();
    const Share<D> me(p.heads);
    if (me.token >= r.num_tokens) return;
    const int64_t slot = r.slots[me.token];
    if (slot < 0) return;
    if (slot >= p.num_blocks * (p.tiles * 16)) {
        atomicOr(&g_fp4_kv_error, kFp4ErrSlot);
        return;
    }
    const BlockPlace at = block_place<D>(p, slot, me.head, me.block);
    const uint2 kc = *reinterpret_cast<const uint2 *>(p.k + at.tile + at.k_code);
    const uint2 vc = *reinterpret_cast<const uint2 *>(p.v + at.tile + at.v_code);
    const uint32_t kb = p.k[at.tile + at.k_scale], vb = p.v[at.tile + at.v_scale];
    float ks, vs;
    load_scales(p, &ks, &vs);
    const bool k_ok = fp4_scale_ok(ks), v_ok = fp4_scale_ok(vs);
    if (!k_ok || !v_ok) atomicOr(&g_fp4_kv_error, kFp4ErrScale);
    const int32_t e = me.head * D + me.block * 16;
    uint4 a, b;
    if (k_ok) {
        dequantise16(kc, kb, ks, &a, &b);
        uint4 *k = reinterpret_cast<uint4 *>(r.k + me.token * r.key_stride + e);
        k[0] = a;
        k[1] = b;
    }
    if (v_ok) {
        dequantise16(vc, vb, vs, &a, &b);
        uint4 *v = reinterpret_cast<uint4 *>(r.v + me.token * r.value_stride + e);
        v[0] = a;
        v[1] = b;
    }
}

// Thread indexes are 32 bits inside a launch; more tokens than that take
// several launches.
template <int D, typename Kernel>
cudaError_t launch_rows(Kernel kernel, Fp4Rows r, const Fp4Pools &p, cudaStream_t stream) {
    const int64_t most = (int64_t{1} << 25) / (static_cast<int64_t>(p.heads) * Share<D>::kParts) *
                         Share<D>::kTokens;            // a multiple of a warp's tokens
    const int64_t all = r.num_tokens;
    for (int64_t done = 0; done < all; done += most) {
        Fp4Rows part = r;
        part.num_tokens = all - done < most ? all - done : most;
        part.k += done * r.key_stride;
        part.v += done * r.value_stride;
        part.slots += done;
        const int64_t warps = Share<D>::warps(part.num_tokens, p.heads);
        const unsigned blocks = static_cast<unsigned>((warps * 32 + kThreads - 1) / kThreads);
        // Scheduled early only if the blocks are few: several an SM are spread
        // unevenly beside those of the kernel before (4593 tokens written and
        // read back 11.5 us, else 9.4; 16 tokens 3.6 us, else 4.2).
        const cudaError_t e = launch_when(blocks <= 148, kernel, dim3(blocks), kThreads, 0, stream, part, p);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_fp4_write(const Fp4Rows &r, const Fp4Pools &p, cudaStream_t stream) {
    return p.dim == 64    ? launch_rows<64>(fp4_write_kernel<64>, r, p, stream)
           : p.dim == 128 ? launch_rows<128>(fp4_write_kernel<128>, r, p, stream)
                          : launch_rows<256>(fp4_write_kernel<256>, r, p, stream);
}

cudaError_t launch_fp4_read(const Fp4Rows &r, const Fp4Pools &p, cudaStream_t stream) {
    return p.dim == 64    ? launch_rows<64>(fp4_read_kernel<64>, r, p, stream)
           : p.dim == 128 ? launch_rows<128>(fp4_read_kernel<128>, r, p, stream)
                          : launch_rows<256>(fp4_read_kernel<256>, r, p, stream);
}

cudaError_t read_fp4_kv_error(uint32_t *bits, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_fp4_kv_error, sizeof(uint32_t));
    if (e == cudaSuccess && clear) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_fp4_kv_error, &zero, sizeof(uint32_t));
    }
    return e;
}

}  // namespace fp8q
