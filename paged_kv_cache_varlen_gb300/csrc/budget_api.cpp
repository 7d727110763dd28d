// budget_api.cpp -- the C ABI of the rotary cache write and of the cache-
// budget calls (declared in include/pkv.h): host-side checks and dispatch.
// As in api.cpp, every check runs before the first launch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/pkv.h"
#include "launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether the byte ranges [a, a + na) and [b, b + nb) meet.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

pkv_status launched(cudaError_t e) { return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA; }

// Grid y dimension: one slice per request, and one more.
constexpr int32_t kMaxSeqs = 65534;

}  // namespace

extern "C" {

pkv_status pkv_rope_frequencies(double* inv_freq, float* factor, int32_t rotary_dim, double base,
                                int32_t kind, double stretch, double original_len, double low,
                                double high) {
  const double kTwoPi = 6.283185307179586476925;
  if (!inv_freq || !factor || rotary_dim <= 0 || rotary_dim % 2 != 0) return PKV_ERR_INVALID_ARG;
  if (!(base > 1.0) || !isfinite(base)) return PKV_ERR_INVALID_ARG;
  if (kind < PKV_ROPE_PLAIN || kind > PKV_ROPE_RAMP) return PKV_ERR_INVALID_ARG;
  if (kind != PKV_ROPE_PLAIN && (!(stretch >= 1.0) || !isfinite(stretch)))
    return PKV_ERR_INVALID_ARG;
  const bool by_turns = kind == PKV_ROPE_BANDS || kind == PKV_ROPE_RAMP;
  if (by_turns && (!(original_len > 0.0) || !isfinite(original_len) || !(low > 0.0) ||
                   !(high > low) || !isfinite(high)))
    return PKV_ERR_INVALID_ARG;
  const double r = rotary_dim;
  if (kind == PKV_ROPE_BASE) {
    if (rotary_dim <= 2) return PKV_ERR_INVALID_ARG;
    base *= pow(stretch, r / (r - 2.0));
  }
  double a = 0.0, b = 0.0;
  if (kind == PKV_ROPE_RAMP) {
    const double per = r / (2.0 * log(base));
    a = fmax(0.0, floor(per * log(original_len / (kTwoPi * high))));
    b = fmin(r - 1.0, ceil(per * log(original_len / (kTwoPi * low))));
  }
  for (int32_t p = 0; p < rotary_dim / 2; ++p) {
    const double f = pow(base, -2.0 * p / r);
    double keep = 1.0;  // share of the frequency that is not stretched
    if (kind == PKV_ROPE_LINEAR) keep = 0.0;
    if (kind == PKV_ROPE_BANDS)
      keep = fmin(1.0, fmax(0.0, (original_len * f / kTwoPi - low) / (high - low)));
    if (kind == PKV_ROPE_RAMP) keep = 1.0 - fmin(1.0, fmax(0.0, (p - a) / fmax(b - a, 0.001)));
    inv_freq[p] = keep == 1.0 ? f : f * (keep + (1.0 - keep) / stretch);
  }
  *factor = kind == PKV_ROPE_RAMP ? (float)(0.1 * log(stretch) + 1.0) : 1.0f;
  return PKV_OK;
}

pkv_status pkv_rope_kv_cache_write(void* q_out, void* kv_pool, const void* q, const void* k_new,
                                   const void* v_new, int64_t q_stride, int64_t k_stride,
                                   int64_t v_stride, const int32_t* positions,
                                   const int32_t* slot_mapping, const double* inv_freq,
                                   float factor, int32_t interleaved, int32_t num_tokens,
                                   int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                   int32_t rotary_dim, int32_t num_blocks, int32_t block_size,
                                   int32_t* dev_status, void* stream) {
  if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 ||
      block_size <= 0)
    return PKV_ERR_INVALID_ARG;
  if (rotary_dim <= 0 || rotary_dim % 2 != 0 || rotary_dim > head_dim || !isfinite(factor))
    return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !kv_pool || !q || !k_new || !v_new || !positions || !slot_mapping || !inv_freq)
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q_out) || !aligned16(kv_pool) || !aligned16(q) || !aligned16(k_new) ||
      !aligned16(v_new) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0)
    return PKV_ERR_INVALID_ARG;
  if (head_dim % 8 != 0 || head_dim > 512) return PKV_ERR_UNSUPPORTED;
  if (num_tokens > INT32_MAX - (1 << 16)) return PKV_ERR_UNSUPPORTED;  // the grid counts past it
  const int64_t qrow = (int64_t)num_heads * head_dim, krow = (int64_t)num_kv_heads * head_dim;
  if (qrow + krow > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (q_stride < qrow || k_stride < krow || v_stride < krow || q_stride % 8 != 0 ||
      k_stride % 8 != 0 || v_stride % 8 != 0)
    return PKV_ERR_INVALID_ARG;
  // halves whose length is no multiple of a vector stage the token's heads
  if (!interleaved && (rotary_dim / 2) % 8 != 0 && (qrow + krow) * 2 > 196 * 1024)
    return PKV_ERR_UNSUPPORTED;
  const int64_t n = num_tokens - 1;
  const int64_t out_bytes = num_tokens * qrow * 2;
  if (overlap(q_out, out_bytes, kv_pool, (int64_t)2 * num_blocks * block_size * krow * 2))
    return PKV_ERR_INVALID_ARG;
  if (overlap(q_out, out_bytes, k_new, (n * k_stride + krow) * 2) ||
      overlap(q_out, out_bytes, v_new, (n * v_stride + krow) * 2) ||
      (overlap(q_out, out_bytes, q, (n * q_stride + qrow) * 2) &&
       (q_out != q || (q_stride != qrow && n > 0))))
    return PKV_ERR_INVALID_ARG;
  pkv::RopeWriteParams p;
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
  p.factor = factor;
  p.interleaved = interleaved != 0;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.rotary_dim = rotary_dim;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.status = dev_status;
  return launched(pkv::launch_rope_write(p, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_attention_key_weights(float* weights_out, const float* weights_in, const void* q,
                                     const void* kv_pool, const float* lse,
                                     const int32_t* block_table, int32_t max_blocks_per_seq,
                                     const int32_t* cu_seqlens_q, const int32_t* seq_lens,
                                     const int32_t* prior_lens, const int32_t* weight_rows,
                                     int32_t num_rows, int32_t row_len, int32_t num_seqs,
                                     int32_t num_tokens, int32_t max_query_len,
                                     int32_t max_seq_len, int32_t num_heads,
                                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                     int32_t num_blocks, float scale, float decay,
                                     int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || num_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (num_seqs == 0) return PKV_ERR_INVALID_ARG;
  if (num_seqs > kMaxSeqs) return PKV_ERR_UNSUPPORTED;
  if (!weights_out || !weights_in || !q || !kv_pool || !lse || !block_table || !cu_seqlens_q ||
      !seq_lens)
    return PKV_ERR_INVALID_ARG;
  if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0)
    return PKV_ERR_INVALID_ARG;
  if (block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || head_dim <= 0 ||
      num_rows <= 0)
    return PKV_ERR_INVALID_ARG;
  if (max_query_len < 1 || max_seq_len < max_query_len || row_len < max_seq_len)
    return PKV_ERR_INVALID_ARG;
  if (!weight_rows && num_rows < num_seqs) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale) || !(decay >= 0.f) || !isfinite(decay))
    return PKV_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(kv_pool) || !aligned4(weights_out) || !aligned4(weights_in))
    return PKV_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)num_rows * num_kv_heads * row_len * 4;
  if (weights_in != weights_out && overlap(weights_out, bytes, weights_in, bytes))
    return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (block_size % 16 != 0 || block_size > 256) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)2 * num_blocks * block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const int32_t group = num_heads / num_kv_heads;
  if ((int64_t)max_query_len * group > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;
  if (max_seq_len > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;  // indexes past the last tile
  // the grid's units, (16-key tiles, KV heads), are counted in 32 bits
  if (((int64_t)max_seq_len / 16 + 1) * num_kv_heads > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;
  pkv::KeyWeightsParams p;
  p.out = weights_out;
  p.in = weights_in;
  p.q = static_cast<const uint16_t*>(q);
  p.pool = static_cast<const uint16_t*>(kv_pool);
  p.lse = lse;
  p.block_table = block_table;
  p.cu_seqlens = cu_seqlens_q;
  p.seq_lens = seq_lens;
  p.prior_lens = prior_lens;
  p.rows = weight_rows;
  p.num_rows = num_rows;
  p.row_len = row_len;
  p.max_blocks = max_blocks_per_seq;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.max_query_len = max_query_len;
  p.max_seq_len = max_seq_len;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.head_dim = head_dim;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.decay = decay;
  p.short_max_q = 0;
  p.no_short = 0;
  p.after_tc = 0;
  p.status = dev_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // Requests of up to 32 (query, head) columns keep their queries in a
  // warp's registers and are bound by reading K (mma.sync grid); longer ones
  // are bound by their products (tcgen05 grid, up to 128 heads a group).
  const int32_t short_q = 32 / group;
  if (max_query_len <= short_q || group > 128) return launched(pkv::launch_key_weights(p, st));
  p.short_max_q = short_q;
  // whether some request can be short: with num_tokens in all, and none
  // longer than max_query_len
  const bool any_short = short_q > 0 && (int64_t)num_seqs * max_query_len - num_tokens >=
                                            (int64_t)max_query_len - short_q;
  p.no_short = !any_short;
  CUtensorMap q_map{}, k_map{};
  if (!pkv::encode_q_tiles(&q_map, q, num_tokens, num_heads, num_kv_heads, head_dim) ||
      !pkv::encode_kv_view(&k_map, kv_pool, num_blocks, block_size, num_kv_heads, head_dim, 1))
    return PKV_ERR_CUDA;
  if (pkv::launch_key_weights_tc(p, q_map, k_map, st) != cudaSuccess) return PKV_ERR_CUDA;
  if (!any_short) return PKV_OK;
  p.after_tc = 1;
  return launched(pkv::launch_key_weights(p, st));
}

pkv_status pkv_evict_select(int32_t* kept, float* weights_out, const float* weights,
                            const int32_t* seq_lens, const int32_t* keep_lens,
                            const int32_t* weight_rows, int32_t num_rows, int32_t row_len,
                            int32_t num_seqs, int32_t num_kv_heads, int32_t max_seq_len,
                            int32_t max_keep_len, int32_t num_sink, int32_t num_recent,
                            int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || num_rows < 0 || max_seq_len < 0 || max_keep_len < 0 ||
      num_sink < 0 || num_recent < 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_keep_len == 0) return PKV_OK;
  if (num_seqs > kMaxSeqs || num_kv_heads > INT32_MAX / 8) return PKV_ERR_UNSUPPORTED;
  if (max_seq_len > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;  // indexes of a padded row
  if (!kept || !weights || !seq_lens || !keep_lens) return PKV_ERR_INVALID_ARG;
  if (row_len < max_seq_len || (weights_out && row_len < max_keep_len)) return PKV_ERR_INVALID_ARG;
  if (!weight_rows && num_rows < num_seqs) return PKV_ERR_INVALID_ARG;
  if (!aligned4(weights) || !aligned4(weights_out) || !aligned4(kept)) return PKV_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)num_rows * num_kv_heads * row_len * 4;
  if (weights_out && overlap(weights_out, bytes, weights, bytes)) return PKV_ERR_INVALID_ARG;
  pkv::EvictSelectParams p;
  p.kept = kept;
  p.out = weights_out;
  p.weights = weights;
  p.seq_lens = seq_lens;
  p.keep_lens = keep_lens;
  p.rows = weight_rows;
  p.num_rows = num_rows;
  p.row_len = row_len;
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.max_seq_len = max_seq_len;
  p.max_keep = max_keep_len;
  p.num_sink = num_sink;
  p.num_recent = num_recent;
  p.status = dev_status;
  return launched(pkv::launch_evict_select(p, static_cast<cudaStream_t>(stream)));
}

pkv_status pkv_evict_compact(void* kv_pool, const int32_t* src_table, int32_t max_src_blocks,
                             const int32_t* dst_table, int32_t max_dst_blocks,
                             const int32_t* kept, int32_t max_keep_len, const int32_t* keep_lens,
                             int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim,
                             int32_t block_size, int32_t num_blocks, int32_t* dev_status,
                             void* stream) {
  if (num_seqs < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
      max_src_blocks < 0 || max_dst_blocks < 0 || max_keep_len < 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_keep_len == 0) return PKV_OK;
  if (num_seqs > kMaxSeqs) return PKV_ERR_UNSUPPORTED;
  if (!kv_pool || !src_table || !dst_table || !kept || !keep_lens || !aligned16(kv_pool))
    return PKV_ERR_INVALID_ARG;
  if (head_dim % 8 != 0 || head_dim > 512) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_src_blocks * block_size > INT32_MAX ||
      (int64_t)max_dst_blocks * block_size > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  // rows of a request are counted in 32 bits
  if ((int64_t)max_keep_len * num_kv_heads > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;
  pkv::EvictCompactParams p;
  p.pool = static_cast<uint4*>(kv_pool);
  p.src_table = src_table;
  p.dst_table = dst_table;
  p.kept = kept;
  p.keep_lens = keep_lens;
  p.max_src = max_src_blocks;
  p.max_dst = max_dst_blocks;
  p.max_keep = max_keep_len;
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.head_vecs = head_dim / 8;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.status = dev_status;
  return launched(pkv::launch_evict_compact(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
