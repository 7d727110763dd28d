// cache8_api.cpp -- the C ABI of the normed rotary writes and of the 8-bit cache
// (declared in include/pkv.h): host-side checks and dispatch. As in api.cpp,
// every check runs before the first launch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/pkv.h"
#include "launch.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether the byte ranges [a, a + na) and [b, b + nb) meet.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

pkv_status launched(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

// The checks that both forms of the normed write share: sizes, the vectors'
// alignment, what q_out may overlap. `value_bytes`: of a cached value.
pkv_status check_rows(const pkv::NormRopeParams& p, int64_t value_bytes) {
  if (p.head_dim % 8 != 0 || p.head_dim > 512) return PKV_ERR_UNSUPPORTED;
  if (p.num_tokens > INT32_MAX - (1 << 16)) return PKV_ERR_UNSUPPORTED;  // the grid counts past it
  const int64_t qrow = (int64_t)p.num_heads * p.head_dim, krow = (int64_t)p.num_kv_heads * p.head_dim;
  if (qrow + 2 * krow > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (!aligned(p.pool, 16) || !aligned(p.k, 16) || !aligned(p.v, 16)) return PKV_ERR_INVALID_ARG;
  if (p.k_stride < krow || p.v_stride < krow || p.k_stride % 8 != 0 || p.v_stride % 8 != 0)
    return PKV_ERR_INVALID_ARG;
  if (!p.q) return PKV_OK;
  if (!aligned(p.q, 16) || !aligned(p.q_out, 16) || !aligned(p.inv_freq, 8))
    return PKV_ERR_INVALID_ARG;
  const uintptr_t w = p.weight_f32 ? 4 : 2;
  if (!aligned(p.q_weight, w) || !aligned(p.k_weight, w)) return PKV_ERR_INVALID_ARG;
  if (p.q_stride < qrow || p.q_stride % 8 != 0) return PKV_ERR_INVALID_ARG;
  const int64_t n = p.num_tokens - 1, out = p.num_tokens * qrow * 2;
  if (overlap(p.q_out, out, p.pool, 2 * p.num_slots * krow * value_bytes) ||
      overlap(p.q_out, out, p.k, (n * p.k_stride + krow) * 2) ||
      overlap(p.q_out, out, p.v, (n * p.v_stride + krow) * 2) ||
      (overlap(p.q_out, out, p.q, (n * p.q_stride + qrow) * 2) &&
       (p.q_out != p.q || (p.q_stride != qrow && n > 0))))
    return PKV_ERR_INVALID_ARG;
  return PKV_OK;
}

bool bad_norm(int32_t rotary_dim, int32_t head_dim, float offset, float eps, float factor) {
  return rotary_dim < 0 || rotary_dim % 2 != 0 || rotary_dim > head_dim || !isfinite(factor) ||
         !isfinite(offset) || !isfinite(eps) || eps < 0.f;
}

// The arguments of an append and its checks; the rest of `p` is filled in.
pkv_status append(pkv::NormRopeParams& p, void* stream) {
  if (p.num_seqs == 0) return PKV_ERR_INVALID_ARG;
  if (!p.pool || !p.scales || !p.k || !p.v || !p.block_table || !p.cu_seqlens || !p.seq_lens)
    return PKV_ERR_INVALID_ARG;
  if (p.max_query_len < 1 || p.max_blocks <= 0 || !aligned(p.scales, 4)) return PKV_ERR_INVALID_ARG;
  if (p.head_dim != 64 && p.head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (p.block_size % 16 != 0 || p.block_size > 256) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)p.max_blocks * p.block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (2 * p.num_slots > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  // grid items of every share of the heads, counted in 32 bits
  const int64_t items = (int64_t)p.num_tokens / p.block_size + 2 * (int64_t)p.num_seqs;
  const int64_t shares = (2 * (int64_t)p.num_kv_heads + p.num_heads) / 2 + 1;
  if (items * (shares < 152 * 4 ? shares : 152 * 4) > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (pkv_status s = check_rows(p, 1); s != PKV_OK) return s;
  const int64_t scale_bytes = (int64_t)2 * p.num_blocks * p.num_kv_heads * 4;
  const int64_t pool_bytes = 2 * p.num_slots * p.num_kv_heads * p.head_dim;
  if (overlap(p.scales, scale_bytes, p.pool, pool_bytes) ||
      (p.q && overlap(p.q_out, (int64_t)p.num_tokens * p.num_heads * p.head_dim * 2, p.scales,
                      scale_bytes)))
    return PKV_ERR_INVALID_ARG;
  return launched(pkv::launch_append_fp8(p, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

pkv_status pkv_qk_norm_rope_kv_cache_write(
    void* q_out, void* kv_pool, const void* q, const void* k_new, const void* v_new,
    int64_t q_stride, int64_t k_stride, int64_t v_stride, const int32_t* positions,
    const int32_t* slot_mapping, const double* inv_freq, const void* q_weight,
    const void* k_weight, int32_t weights_f32, float weight_offset, float eps, float factor,
    int32_t interleaved, int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t rotary_dim, int32_t num_blocks, int32_t block_size,
    int32_t* dev_status, void* stream) {
  if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 ||
      block_size <= 0 || bad_norm(rotary_dim, head_dim, weight_offset, eps, factor))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !kv_pool || !q || !k_new || !v_new || !positions || !slot_mapping ||
      (!inv_freq && rotary_dim > 0))
    return PKV_ERR_INVALID_ARG;
  pkv::NormRopeParams p{};
  p.q_out = static_cast<uint16_t*>(q_out);
  p.pool = kv_pool;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k_new);
  p.v = static_cast<const uint16_t*>(v_new);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.slots = slot_mapping;
  p.inv_freq = inv_freq;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.weight_f32 = weights_f32 != 0;
  p.weight_offset = weight_offset;
  p.eps = eps;
  p.factor = factor;
  p.interleaved = interleaved != 0;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.rotary_dim = rotary_dim;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.status = dev_status;
  if (pkv_status s = check_rows(p, 2); s != PKV_OK) return s;
  return launched(pkv::launch_norm_rope(p, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_kv_cache_append_fp8(void* kv_pool, float* kv_scales, const void* k_new,
                                   const void* v_new, int64_t k_stride, int64_t v_stride,
                                   const int32_t* block_table, int32_t max_blocks_per_seq,
                                   const int32_t* cu_seqlens_q, const int32_t* seq_lens,
                                   int32_t num_seqs, int32_t num_tokens, int32_t max_query_len,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks,
                                   int32_t block_size, int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 ||
      block_size <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  pkv::NormRopeParams p{};
  p.pool = kv_pool;
  p.scales = kv_scales;
  p.k = static_cast<const uint16_t*>(k_new);
  p.v = static_cast<const uint16_t*>(v_new);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.factor = 1.f;
  p.num_tokens = num_tokens;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.block_table = block_table;
  p.cu_seqlens = cu_seqlens_q;
  p.seq_lens = seq_lens;
  p.max_blocks = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.max_query_len = max_query_len;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.status = dev_status;
  return append(p, stream);
}

pkv_status pkv_qk_norm_rope_kv_cache_append_fp8(
    void* q_out, void* kv_pool, float* kv_scales, const void* q, const void* k_new,
    const void* v_new, int64_t q_stride, int64_t k_stride, int64_t v_stride,
    const int32_t* positions, const int32_t* block_table, int32_t max_blocks_per_seq,
    const int32_t* cu_seqlens_q, const int32_t* seq_lens, const double* inv_freq,
    const void* q_weight, const void* k_weight, int32_t weights_f32, float weight_offset, float eps,
    float factor, int32_t interleaved, int32_t num_seqs, int32_t num_tokens, int32_t max_query_len,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t rotary_dim,
    int32_t num_blocks, int32_t block_size, int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      num_blocks <= 0 || block_size <= 0 ||
      bad_norm(rotary_dim, head_dim, weight_offset, eps, factor))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !q || !positions || (!inv_freq && rotary_dim > 0)) return PKV_ERR_INVALID_ARG;
  pkv::NormRopeParams p{};
  p.q_out = static_cast<uint16_t*>(q_out);
  p.pool = kv_pool;
  p.scales = kv_scales;
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k_new);
  p.v = static_cast<const uint16_t*>(v_new);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.weight_f32 = weights_f32 != 0;
  p.weight_offset = weight_offset;
  p.eps = eps;
  p.factor = factor;
  p.interleaved = interleaved != 0;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.rotary_dim = rotary_dim;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.block_table = block_table;
  p.cu_seqlens = cu_seqlens_q;
  p.seq_lens = seq_lens;
  p.max_blocks = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.max_query_len = max_query_len;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.status = dev_status;
  return append(p, stream);
}

pkv_status pkv_copy_blocks_fp8(void* kv_pool, float* kv_scales, const int32_t* copy_src,
                               const int32_t* copy_dst, int32_t num_copies, int32_t num_blocks,
                               int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                               int32_t* dev_status, void* stream) {
  if (num_copies < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_copies == 0) return PKV_OK;
  if (!kv_pool || !kv_scales || !copy_src || !copy_dst || !aligned(kv_pool, 16) ||
      !aligned(kv_scales, 4))
    return PKV_ERR_INVALID_ARG;
  const int64_t block_bytes = (int64_t)block_size * num_kv_heads * head_dim;
  if (block_bytes % 16 != 0) return PKV_ERR_UNSUPPORTED;
  if (num_copies > 65535 || block_bytes / 16 / 1024 > 65535) return PKV_ERR_UNSUPPORTED;
  return launched(pkv::launch_copy_blocks(kv_pool, copy_src, copy_dst, num_copies, num_blocks,
                                          block_bytes / 16, kv_scales, num_kv_heads, dev_status,
                                          static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
