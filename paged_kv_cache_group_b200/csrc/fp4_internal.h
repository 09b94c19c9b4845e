// Internal interface between the C ABI of the 4-bit KV cache and of the
// query/key norm with rotation (fp4_api.cpp) and their kernels (fp4_kv.cu,
// fp4_attention.cu, qk_rope.cu).  The public surface is include/fp8q.h.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace fp8q {

// Tensor scales of a cache the 4-bit kernels accept: every block scale times
// such a scale, and its reciprocal, is a normal fp32 number.
constexpr float kFp4MinScale = 0x1p-96f;
constexpr float kFp4MaxScale = 0x1p96f;

// A pair of 4-bit pools: [num_blocks][heads][tiles][9 * dim] bytes, blocks
// block_stride bytes apart.
struct Fp4Pools {
    uint8_t *k = nullptr;
    uint8_t *v = nullptr;
    int64_t block_stride = 0;
    int64_t num_blocks = 0;
    int32_t tiles = 0;       // block_size / 16
    int32_t heads = 0;       // KV heads
    int32_t dim = 0;         // 64, 128 or 256
    float k_scale = 1.0f;    // used when scale_dev is null
    float v_scale = 1.0f;
    const float *scale_dev = nullptr;
};

// Rows of K and V moved between bf16 tensors and the pools.
struct Fp4Rows {
    uint16_t *k = nullptr;   // read by the write, written by the read
    uint16_t *v = nullptr;
    int64_t key_stride = 0;
    int64_t value_stride = 0;
    const int64_t *slots = nullptr;
    int64_t num_tokens = 0;
};

cudaError_t launch_fp4_write(const Fp4Rows &r, const Fp4Pools &p, cudaStream_t stream);
cudaError_t launch_fp4_read(const Fp4Rows &r, const Fp4Pools &p, cudaStream_t stream);

struct Fp4Attention {
    Fp4Pools pools;
    const uint16_t *q = nullptr;
    int64_t q_stride = 0;
    uint16_t *out = nullptr;
    int64_t out_stride = 0;
    float *lse = nullptr;               // [num_tokens, q_heads] or null
    const int32_t *block_table = nullptr;
    int64_t table_stride = 0;
    int64_t table_width = 0;
    const int32_t *seq_lens = nullptr;
    const int32_t *q_start = nullptr;   // null: sequence b has the one token b
    int32_t batch = 0;
    int32_t num_tokens = 0;
    int32_t q_heads = 0;
    int32_t window = 0;                 // 0: no window
    float softmax_scale = 1.0f;
    void *workspace = nullptr;
    int64_t workspace_bytes = 0;
};

// Bytes of workspace launch_fp4_attention needs for these sizes; with `uneven`
// what it can use where some sequences are much longer than others.
int64_t fp4_attention_workspace(int64_t batch, int64_t num_tokens, int32_t q_heads,
                                int32_t kv_heads, int32_t dim, bool uneven);
cudaError_t launch_fp4_attention(const Fp4Attention &a, cudaStream_t stream);

// Its kernel for many rows to a KV head (fp4_attention_rows.cu).
bool fp4_attention_by_rows(int64_t batch, int64_t num_tokens, int32_t group);
int64_t fp4_attention_rows_workspace(int64_t num_tokens, int32_t group, int32_t kv_heads, int32_t dim,
                                     bool uneven);
cudaError_t launch_fp4_attention_rows(const Fp4Attention &a, cudaStream_t stream);

struct QkNormRope {
    const uint16_t *q = nullptr;
    const uint16_t *k = nullptr;
    int64_t q_stride = 0;
    int64_t k_stride = 0;
    uint16_t *q_out = nullptr;
    uint16_t *k_out = nullptr;
    int64_t q_out_stride = 0;
    int64_t k_out_stride = 0;
    const int64_t *positions = nullptr;
    const double *inv_freq = nullptr;   // [rotary / 2]
    const uint16_t *q_weight = nullptr; // bf16 [dim] or null: no norm
    const uint16_t *k_weight = nullptr;
    int64_t num_tokens = 0;
    int32_t q_heads = 0;
    int32_t k_heads = 0;
    int32_t dim = 0;
    int32_t rotary = 0;
    float eps = 0.0f;
    float rope_scale = 1.0f;
    bool interleaved = false;
};

cudaError_t launch_qk_norm_rope(const QkNormRope &r, cudaStream_t stream);

// Reads (and with clear resets) the sticky error words of these kernels on
// the current device; the device must be idle.
cudaError_t read_fp4_kv_error(uint32_t *bits, bool clear);
cudaError_t read_fp4_attention_error(uint32_t *bits, bool clear);
cudaError_t read_fp4_rows_error(uint32_t *bits, bool clear);

}  // namespace fp8q
