// fp4_api.cpp -- the C ABI of the 4-bit KV cache and of the query/key norm
// with rotation (include/fp8q.h, sections 4 and 5): argument checks and
// dispatch to the kernels.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "fp4_internal.h"
#include "fp8q.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

fp8q_status from_cuda(cudaError_t e) { return e == cudaSuccess ? FP8Q_OK : FP8Q_ECUDA; }

bool valid_scale(float s) { return s >= fp8q::kFp4MinScale && s <= fp8q::kFp4MaxScale; }

// Row stride of a [rows, width] bf16 tensor.
bool valid_stride(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0; }

// Whether two [rows, width] bf16 tensors share memory; strides are valid_stride's.
bool rows_overlap(const void *a, int64_t a_stride, int64_t a_width, const void *b, int64_t b_stride,
                  int64_t b_width, int64_t rows) {
    const int64_t a0 = reinterpret_cast<intptr_t>(a) / 2, b0 = reinterpret_cast<intptr_t>(b) / 2;
    if (a0 + (rows - 1) * a_stride + a_width <= b0 || b0 + (rows - 1) * b_stride + b_width <= a0)
        return false;
    if (a_stride == b_stride) {
        // Row i + k of b begins at d + k * stride of row i of a.  Only the first of
        // them at or behind its beginning and the one before can reach into it.
        const int64_t d = b0 - a0, behind = (d % a_stride + a_stride) % a_stride;
        const int64_t k = (behind - d) / a_stride;
        return (behind < a_width && k > -rows && k < rows) ||
               (behind - a_stride + b_width > 0 && k - 1 > -rows && k - 1 < rows);
    }
    for (int64_t i = 0, j = 0; i < rows && j < rows;) {
        const int64_t x = a0 + i * a_stride, y = b0 + j * b_stride;
        if (x < y + b_width && y < x + a_width) return true;
        if (x < y) ++i;
        else ++j;
    }
    return false;
}

bool valid_dim(int32_t head_dim) { return head_dim == 64 || head_dim == 128 || head_dim == 256; }

bool make_pools(void *k_pool, void *v_pool, int32_t num_kv_heads, int32_t head_dim,
                int32_t block_size, int64_t block_stride, int64_t num_blocks, float k_scale,
                float v_scale, const float *scale_dev, fp8q::Fp4Pools *p) {
    if (num_kv_heads <= 0 || num_kv_heads > 65536 || !valid_dim(head_dim)) return false;
    if (block_size <= 0 || block_size % 16 != 0 || block_size > (1 << 24)) return false;
    const int64_t block_bytes = int64_t{9} * num_kv_heads * (block_size / 16) * head_dim;
    if (block_stride < block_bytes || block_stride % 16 != 0) return false;
    if (num_blocks < 0 || num_blocks > INT64_MAX / block_stride) return false;
    if (num_blocks > 0 && (k_pool == nullptr || v_pool == nullptr)) return false;
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16)) return false;
    if (scale_dev == nullptr ? !(valid_scale(k_scale) && valid_scale(v_scale))
                             : !aligned(scale_dev, 8))
        return false;
    p->k = static_cast<uint8_t *>(k_pool);
    p->v = static_cast<uint8_t *>(v_pool);
    p->block_stride = block_stride;
    p->num_blocks = num_blocks;
    p->tiles = block_size / 16;
    p->heads = num_kv_heads;
    p->dim = head_dim;
    p->k_scale = k_scale;
    p->v_scale = v_scale;
    p->scale_dev = scale_dev;
    return true;
}

bool make_rows(void *k, void *v, int64_t key_stride, int64_t value_stride,
               const int64_t *slot_mapping, int64_t num_tokens, const fp8q::Fp4Pools &p,
               fp8q::Fp4Rows *r) {
    const int64_t width = static_cast<int64_t>(p.heads) * p.dim;
    if (num_tokens < 0 || !valid_stride(key_stride, width) || !valid_stride(value_stride, width))
        return false;
    if (num_tokens > 0) {
        if (k == nullptr || v == nullptr || !aligned(k, 16) || !aligned(v, 16)) return false;
        if (slot_mapping == nullptr || !aligned(slot_mapping, 8)) return false;
        if (num_tokens > INT64_MAX / 2 / key_stride || num_tokens > INT64_MAX / 2 / value_stride)
            return false;
    }
    r->k = static_cast<uint16_t *>(k);
    r->v = static_cast<uint16_t *>(v);
    r->key_stride = key_stride;
    r->value_stride = value_stride;
    r->slots = slot_mapping;
    r->num_tokens = num_tokens;
    return true;
}

// The largest count of (token, query head) rows one call takes: row and tile
// indexes stay within 32 bits.
constexpr int64_t kMaxRows = int64_t{1} << 30;

bool valid_attention_sizes(int64_t batch, int64_t num_tokens, int32_t num_q_heads,
                           int32_t num_kv_heads, int32_t head_dim) {
    if (batch < 0 || batch > kMaxRows || num_tokens < 0) return false;
    if (num_kv_heads <= 0 || num_kv_heads > 65536 || !valid_dim(head_dim)) return false;
    if (num_q_heads <= 0 || num_q_heads % num_kv_heads != 0) return false;
    return num_tokens <= kMaxRows / num_q_heads;
}

}  // namespace

extern "C" {

FP8Q_API fp8q_status fp4_kv_write(const void *k, const void *v, int64_t key_stride,
                                  int64_t value_stride, const int64_t *slot_mapping,
                                  int64_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                                  void *k_pool, void *v_pool, int32_t block_size,
                                  int64_t block_stride, int64_t num_blocks, float k_scale,
                                  float v_scale, const float *scale_dev, void *stream) {
    fp8q::Fp4Pools p;
    fp8q::Fp4Rows r;
    if (!make_pools(k_pool, v_pool, num_kv_heads, head_dim, block_size, block_stride, num_blocks,
                    k_scale, v_scale, scale_dev, &p))
        return FP8Q_EINVAL;
    if (!make_rows(const_cast<void *>(k), const_cast<void *>(v), key_stride, value_stride,
                   slot_mapping, num_tokens, p, &r))
        return FP8Q_EINVAL;
    if (num_tokens == 0) return FP8Q_OK;
    return from_cuda(fp8q::launch_fp4_write(r, p, static_cast<cudaStream_t>(stream)));
}

FP8Q_API fp8q_status fp4_kv_read(void *k, void *v, int64_t key_stride, int64_t value_stride,
                                 const int64_t *slot_mapping, int64_t num_tokens,
                                 int32_t num_kv_heads, int32_t head_dim, const void *k_pool,
                                 const void *v_pool, int32_t block_size, int64_t block_stride,
                                 int64_t num_blocks, float k_scale, float v_scale,
                                 const float *scale_dev, void *stream) {
    fp8q::Fp4Pools p;
    fp8q::Fp4Rows r;
    if (!make_pools(const_cast<void *>(k_pool), const_cast<void *>(v_pool), num_kv_heads, head_dim,
                    block_size, block_stride, num_blocks, k_scale, v_scale, scale_dev, &p))
        return FP8Q_EINVAL;
    if (!make_rows(k, v, key_stride, value_stride, slot_mapping, num_tokens, p, &r))
        return FP8Q_EINVAL;
    if (num_tokens == 0) return FP8Q_OK;
    const int64_t width = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (rows_overlap(k, key_stride, width, v, value_stride, width, num_tokens)) return FP8Q_EINVAL;
    return from_cuda(fp8q::launch_fp4_read(r, p, static_cast<cudaStream_t>(stream)));
}

FP8Q_API int64_t fp4_kv_attention_workspace(int64_t batch, int64_t num_tokens,
                                            int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim) {
    if (!valid_attention_sizes(batch, num_tokens, num_q_heads, num_kv_heads, head_dim)) return -1;
    return fp8q::fp4_attention_workspace(batch, num_tokens, num_q_heads, num_kv_heads, head_dim, false);
}

FP8Q_API int64_t fp4_kv_attention_workspace_uneven(int64_t batch, int64_t num_tokens,
                                                   int32_t num_q_heads, int32_t num_kv_heads,
                                                   int32_t head_dim) {
    if (!valid_attention_sizes(batch, num_tokens, num_q_heads, num_kv_heads, head_dim)) return -1;
    return fp8q::fp4_attention_workspace(batch, num_tokens, num_q_heads, num_kv_heads, head_dim, true);
}

FP8Q_API fp8q_status fp4_kv_attention(const void *q, int64_t q_stride, const void *k_pool,
                                      const void *v_pool, int32_t block_size,
                                      int64_t block_stride, int64_t num_blocks,
                                      int32_t num_kv_heads, int32_t head_dim,
                                      const int32_t *block_table, int64_t table_stride,
                                      int64_t table_width, const int32_t *seq_lens,
                                      const int32_t *q_start, int64_t batch, int64_t num_tokens,
                                      int32_t num_q_heads, float softmax_scale, int64_t window,
                                      float k_scale, float v_scale, const float *scale_dev,
                                      void *out, int64_t out_stride, float *lse, void *workspace,
                                      int64_t workspace_bytes, void *stream) {
    fp8q::Fp4Attention a;
    if (!make_pools(const_cast<void *>(k_pool), const_cast<void *>(v_pool), num_kv_heads, head_dim,
                    block_size, block_stride, num_blocks, k_scale, v_scale, scale_dev, &a.pools))
        return FP8Q_EINVAL;
    if (!valid_attention_sizes(batch, num_tokens, num_q_heads, num_kv_heads, head_dim))
        return FP8Q_EINVAL;
    const int64_t width = static_cast<int64_t>(num_q_heads) * head_dim;
    if (!valid_stride(q_stride, width) || !valid_stride(out_stride, width)) return FP8Q_EINVAL;
    if (table_width < 0 || table_stride < table_width || window < 0) return FP8Q_EINVAL;
    if (table_width > kMaxRows / block_size) return FP8Q_EINVAL;
    if (batch > 0 && table_stride > INT64_MAX / 8 / batch) return FP8Q_EINVAL;
    if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.0f)) return FP8Q_EINVAL;
    if (q_start == nullptr && num_tokens != batch) return FP8Q_EINVAL;
    if (batch == 0 || num_tokens == 0) return FP8Q_OK;
    if (num_tokens > INT64_MAX / 2 / q_stride || num_tokens > INT64_MAX / 2 / out_stride)
        return FP8Q_EINVAL;
    if (q == nullptr || out == nullptr || !aligned(q, 16) || !aligned(out, 16)) return FP8Q_EINVAL;
    if (rows_overlap(q, q_stride, width, out, out_stride, width, num_tokens)) return FP8Q_EINVAL;
    if (seq_lens == nullptr || !aligned(seq_lens, 4) || !aligned(q_start, 4) || !aligned(lse, 4))
        return FP8Q_EINVAL;
    if ((table_width > 0 && block_table == nullptr) || !aligned(block_table, 4)) return FP8Q_EINVAL;
    if (workspace == nullptr || !aligned(workspace, 16) ||
        workspace_bytes < fp8q::fp4_attention_workspace(batch, num_tokens, num_q_heads,
                                                        num_kv_heads, head_dim, false))
        return FP8Q_EINVAL;
    a.q = static_cast<const uint16_t *>(q);
    a.q_stride = q_stride;
    a.out = static_cast<uint16_t *>(out);
    a.out_stride = out_stride;
    a.lse = lse;
    a.block_table = block_table;
    a.table_stride = table_stride;
    a.table_width = table_width;
    a.seq_lens = seq_lens;
    a.q_start = q_start;
    a.batch = static_cast<int32_t>(batch);
    a.num_tokens = static_cast<int32_t>(num_tokens);
    a.q_heads = num_q_heads;
    a.window = window > kMaxRows ? 0 : static_cast<int32_t>(window);   // wider than any table
    a.softmax_scale = softmax_scale;
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    return from_cuda(fp8q::launch_fp4_attention(a, static_cast<cudaStream_t>(stream)));
}

FP8Q_API fp8q_status qk_norm_rope(const void *q, const void *k, int64_t q_stride,
                                  int64_t k_stride, void *q_out, void *k_out,
                                  int64_t q_out_stride, int64_t k_out_stride,
                                  const int64_t *positions, const double *inv_freq,
                                  const void *q_weight, const void *k_weight, int64_t num_tokens,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t rotary_dim, int32_t interleaved, float eps,
                                  float rope_scale, void *stream) {
    if (num_tokens < 0 || num_tokens > INT32_MAX || !valid_dim(head_dim)) return FP8Q_EINVAL;
    if (num_q_heads < 0 || num_kv_heads < 0 || num_q_heads > 65536 || num_kv_heads > 65536)
        return FP8Q_EINVAL;
    if (num_q_heads + num_kv_heads == 0 || num_q_heads + num_kv_heads > 65536) return FP8Q_EINVAL;
    if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 8 != 0) return FP8Q_EINVAL;
    if (!std::isfinite(eps) || eps < 0.0f || !std::isfinite(rope_scale)) return FP8Q_EINVAL;
    if (num_tokens == 0) return FP8Q_OK;
    const void *in[2] = {q, k}, *out[2] = {q_out, k_out}, *weight[2] = {q_weight, k_weight};
    const int64_t stride[2] = {q_stride, k_stride}, out_stride[2] = {q_out_stride, k_out_stride};
    const int32_t heads[2] = {num_q_heads, num_kv_heads};
    for (int i = 0; i < 2; ++i) {
        if (!aligned(weight[i], 16)) return FP8Q_EINVAL;
        if (heads[i] == 0) {
            weight[i] = nullptr;               // the kernel loads it before it counts heads
            continue;
        }
        const int64_t width = static_cast<int64_t>(heads[i]) * head_dim;
        if (in[i] == nullptr || out[i] == nullptr) return FP8Q_EINVAL;
        if (!aligned(in[i], 16) || !aligned(out[i], 16)) return FP8Q_EINVAL;
        if (!valid_stride(stride[i], width) || !valid_stride(out_stride[i], width))
            return FP8Q_EINVAL;
        if (stride[i] > INT64_MAX / 4 / num_tokens || out_stride[i] > INT64_MAX / 4 / num_tokens)
            return FP8Q_EINVAL;
    }
    for (int i = 0; i < 2; ++i) {              // an output with the inputs and the other one
        const int64_t width = static_cast<int64_t>(heads[i]) * head_dim;
        for (int j = 0; j < 2 && heads[i] > 0; ++j) {
            const int64_t other = static_cast<int64_t>(heads[j]) * head_dim;
            if (heads[j] == 0) continue;
            if (!(i == j && in[i] == out[i] && stride[i] == out_stride[i]) &&
                rows_overlap(out[i], out_stride[i], width, in[j], stride[j], other, num_tokens))
                return FP8Q_EINVAL;
            if (i < j && rows_overlap(out[i], out_stride[i], width, out[j], out_stride[j], other, num_tokens))
                return FP8Q_EINVAL;
        }
    }
    if (positions == nullptr || !aligned(positions, 8)) return FP8Q_EINVAL;
    if ((rotary_dim > 0 && inv_freq == nullptr) || !aligned(inv_freq, 8)) return FP8Q_EINVAL;
    fp8q::QkNormRope r;
    r.q = static_cast<const uint16_t *>(q);
    r.k = static_cast<const uint16_t *>(k);
    r.q_stride = q_stride;
    r.k_stride = k_stride;
    r.q_out = static_cast<uint16_t *>(q_out);
    r.k_out = static_cast<uint16_t *>(k_out);
    r.q_out_stride = q_out_stride;
    r.k_out_stride = k_out_stride;
    r.positions = positions;
    r.inv_freq = inv_freq;
    r.q_weight = static_cast<const uint16_t *>(weight[0]);
    r.k_weight = static_cast<const uint16_t *>(weight[1]);
    r.num_tokens = num_tokens;
    r.q_heads = num_q_heads;
    r.k_heads = num_kv_heads;
    r.dim = head_dim;
    r.rotary = rotary_dim;
    r.eps = eps;
    r.rope_scale = rope_scale;
    r.interleaved = interleaved != 0;
    return from_cuda(fp8q::launch_qk_norm_rope(r, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
