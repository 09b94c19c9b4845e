// Device and launch helpers shared by the kernels of the 4-bit KV cache and
// of the query/key norm with rotation.
#pragma once

#include <atomic>
#include <cstdint>
#include <utility>

#include <cuda_runtime.h>

#include "fp4_internal.h"

namespace fp8q {

extern std::atomic<int64_t> g_launch_count;   // kernels launched by the library

// Bits of the sticky error word, as in include/fp8q.h.
constexpr uint32_t kFp4ErrSlot = 0x1u;
constexpr uint32_t kFp4ErrScale = 0x2u;
constexpr uint32_t kFp4ErrSequence = 0x4u;
constexpr uint32_t kFp4ErrWait = 0x8u;

// Launch; if `early` with programmatic stream serialization: the kernel may be
// scheduled while the one before it on the stream runs, and waits for it itself.
template <typename... Params, typename... Args>
cudaError_t launch_when(bool early, void (*kernel)(Params...), dim3 grid, int block, size_t smem,
                        cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e == cudaSuccess) g_launch_count.fetch_add(1, std::memory_order_relaxed);
    return e;
}

template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, int block, size_t smem,
                       cudaStream_t stream, Args &&...args) {
    return launch_when(true, kernel, grid, block, smem, stream, std::forward<Args>(args)...);
}

// Multiprocessors of the current device.
inline cudaError_t device_sms(int *sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*sms > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
    return e;
}

// Every kernel passes its dependency wait before it lets its dependents
// start, so everything enqueued before it has completed when they start.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_allow_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 values rounded to a bf16 pair, `lo` in the low half.
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two fp32 values rounded to an fp16 pair, `lo` in the low half.
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Two E4M3 codes (bytes 0 and 1) as an fp16 pair: exact.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t codes) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<unsigned short>(codes)));
    return d;
}

// The eight E2M1 codes of a word as four fp16 pairs, low nibble first: exact.
__device__ __forceinline__ void f16x2_of_e2m1x8(uint32_t codes, uint32_t (&d)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3]) : "r"(codes));
}

// Eight fp32 values to E2M1 codes, v[0] in the lowest nibble: nearest-even,
// saturating to +-6, the sign of zero kept, NaN to +6.
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&v)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

__device__ __forceinline__ bool fp4_scale_ok(float s) {
    return s >= kFp4MinScale && s <= kFp4MaxScale;   // false for NaN
}

}  // namespace fp8q
