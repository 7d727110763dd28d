// window_api.cpp -- the C ABI of attention through a window and over an 8-bit
// cache (declared in include/pkv.h): host-side checks, partitions, dispatch. As in
// api.cpp, every check and encoding runs before the first launch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/pkv.h"
#include "launch.h"

namespace {

using pkv::AttnParams;

constexpr int32_t kMaxParts = 65535;  // the decode grid's y dimension
constexpr size_t kSchedBytes = 256;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// How a call's short requests are split: at most `parts` partitions of `size`
// keys that some query of the request sees.
struct Split {
  int32_t max_q;  // queries of the requests that the decode grids take
  int32_t ws_q;   // of which this call has at most so many
  int32_t size, parts;
  size_t lse_off, sched_off, total;
};

bool plan_split(Split* s, int32_t num_seqs, int32_t max_query_len, int32_t num_heads,
                int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len, int32_t window,
                int32_t num_sink, int32_t partition_size, bool eight) {
  if (partition_size < -1 || (partition_size > 0 && partition_size % 16 != 0)) return false;
  const int32_t group = num_heads / num_kv_heads;
  s->max_q = 32 / group > 1 ? 32 / group : 1;
  s->ws_q = max_query_len < s->max_q ? max_query_len : s->max_q;
  int64_t seen = ((int64_t)max_seq_len + 15) / 16 * 16;
  if (window > 0) {
    // chunks of 16 keys: the sinks', and the window's of the request's queries
    const int64_t most = (((int64_t)num_sink + 15) / 16 +
                          ((int64_t)window + s->ws_q - 1 + 15) / 16 + 1) * 16;
    if (most < seen) seen = most;
  }
  int64_t size = partition_size;
  if (partition_size == 0) size = seen;
  if (partition_size < 0) {
    // as many CTAs as keep every SM's slots filled about twice, in partitions of
    // at least 256 keys
    const int64_t rows = (int64_t)s->ws_q * group;
    const int64_t columns = eight && rows <= 8 ? 8 : 16;
    const int64_t base = (int64_t)num_seqs * num_kv_heads * ((rows + columns - 1) / columns);
    const int64_t want = (152 * 8 + base - 1) / base;
    size = ((seen + want - 1) / want + 63) / 64 * 64;
    if (size < 256) size = 256;
  }
  if (size > seen) size = seen;
  s->size = (int32_t)size;
  const int64_t parts = (seen + size - 1) / size;
  if (parts > kMaxParts) return false;
  s->parts = (int32_t)parts;
  s->lse_off = s->sched_off = 0;
  if (parts > 1) {
    const size_t rows = (size_t)num_seqs * s->ws_q * num_heads * parts;
    s->lse_off = round_up(rows * head_dim * sizeof(float), 256);
    s->sched_off = s->lse_off + round_up(rows * sizeof(float), 256);
  }
  s->total = s->sched_off + kSchedBytes;
  return true;
}

// Common to both calls; `scales` non-null: an 8-bit pool.
pkv_status attention(void* out, int32_t out_f32, float* out_lse, const void* q, const void* kv_pool,
                     const float* scales, bool eight, const int32_t* block_table,
                     int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
                     const int32_t* seq_lens, int32_t num_seqs, int32_t num_tokens,
                     int32_t max_query_len, int32_t max_seq_len, int32_t num_heads,
                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     int32_t num_blocks, int32_t window, int32_t num_sink, float scale,
                     int32_t partition_size, void* workspace, size_t workspace_bytes,
                     int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || num_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (num_seqs == 0) return PKV_ERR_INVALID_ARG;
  if (num_seqs > 65534) return PKV_ERR_UNSUPPORTED;  // grid z: requests + one
  if (!out || !q || !kv_pool || (eight && !scales) || !block_table || !cu_seqlens_q || !seq_lens)
    return PKV_ERR_INVALID_ARG;
  if (num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0)
    return PKV_ERR_INVALID_ARG;
  if (block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || head_dim <= 0)
    return PKV_ERR_INVALID_ARG;
  if (max_query_len < 1 || max_seq_len < max_query_len) return PKV_ERR_INVALID_ARG;
  if (window < 0 || num_sink < 0) return PKV_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return PKV_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_pool, 16) || !aligned(out, 16) || !aligned(scales, 4) ||
      !aligned(out_lse, 4))
    return PKV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (block_size % 16 != 0 || block_size > 256) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)2 * num_blocks * block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if ((int64_t)max_blocks_per_seq * block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  // (key indexes are formed up to a tile past the context)
  if (max_seq_len > INT32_MAX / 2) return PKV_ERR_UNSUPPORTED;
  if (num_heads > INT32_MAX / 65536) return PKV_ERR_UNSUPPORTED;
  const int32_t group = num_heads / num_kv_heads;
  Split sp{};
  if (partition_size < -1 || (partition_size > 0 && partition_size % 16 != 0))
    return PKV_ERR_INVALID_ARG;
  if (!plan_split(&sp, num_seqs, max_query_len, num_heads, num_kv_heads, head_dim, max_seq_len,
                  window, num_sink, partition_size, eight))
    return PKV_ERR_UNSUPPORTED;
  if ((int64_t)num_seqs * sp.ws_q * num_heads > INT32_MAX) return PKV_ERR_UNSUPPORTED;  // merge rows
  const bool prefill = max_query_len > sp.max_q;
  if (prefill && (group > 128 || !pkv::prefill_fits(num_seqs, head_dim, eight)))
    return PKV_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < sp.total || !aligned(workspace, 256))
    return PKV_ERR_WORKSPACE;

  AttnParams p{};
  p.out = static_cast<float*>(out);
  p.out_bf16 = !out_f32;
  p.out_lse = out_lse;
  p.q = static_cast<const uint16_t*>(q);
  p.kv_pool = kv_pool;
  p.scales = scales;
  p.block_table = block_table;
  p.cu_seqlens = cu_seqlens_q;
  p.seq_lens = seq_lens;
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
  // without a window every key lies in it
  p.window = window > 0 ? window : INT32_MAX;
  p.num_sink = num_sink;
  p.part_size = sp.size;
  p.num_parts = sp.parts;
  p.ws_q = sp.ws_q;
  char* ws = static_cast<char*>(workspace);
  if (sp.parts > 1) {
    p.ws_out = reinterpret_cast<float*>(ws);
    p.ws_lse = reinterpret_cast<float*>(ws + sp.lse_off);
  }
  p.sched = reinterpret_cast<int32_t*>(ws + sp.sched_off);
  p.status = dev_status;
  p.decode_max_q = sp.max_q;
  p.decode_max_rows = sp.ws_q * group;
  p.kv_splits = 1;

  // the 8-bit pool's one view serves both kernels
  CUtensorMap rows{}, q_map{}, boxes{};
  const bool ok =
      eight ? pkv::encode_kv8_view(&rows, kv_pool, num_blocks, block_size, num_kv_heads, head_dim)
            : pkv::encode_kv_view(&rows, kv_pool, num_blocks, block_size, num_kv_heads, head_dim,
                                  (uint32_t)(head_dim / 64));
  if (!ok) return PKV_ERR_CUDA;
  if (prefill &&
      (!pkv::encode_q_tiles(&q_map, q, num_tokens, num_heads, num_kv_heads, head_dim) ||
       (!eight &&
        !pkv::encode_kv_view(&boxes, kv_pool, num_blocks, block_size, num_kv_heads, head_dim, 1))))
    return PKV_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto decode = [&](const AttnParams& d) {
    return (eight ? pkv::launch_decode_fp8(d, rows, st) : pkv::launch_decode_mma(d, rows, st)) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
  };
  if (!prefill) return decode(p);
  // the prefill grid, then (unless no request can be short) the decode grid on
  // the SMs that it leaves, as in api.cpp; the work tickets start at zero
  if (cudaMemsetAsync(p.sched, 0, kSchedBytes, st) != cudaSuccess) return PKV_ERR_CUDA;
  const bool any_short = (int64_t)num_seqs * max_query_len - num_tokens >=
                         (int64_t)max_query_len - sp.max_q;
  AttnParams pp = p;
  if (any_short) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return PKV_ERR_CUDA;
    pp.shared_sms = sms;
  } else {
    pp.no_decode = 1;
  }
  if (pkv::launch_prefill(pp, q_map, eight ? rows : boxes, st) != cudaSuccess) return PKV_ERR_CUDA;
  if (!any_short) return PKV_OK;
  p.after_prefill = 1;
  return decode(p);
}

}  // namespace

extern "C" {

size_t pkv_window_attention_workspace_size(int32_t num_seqs, int32_t max_query_len,
                                           int32_t num_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t max_seq_len, int32_t window,
                                           int32_t num_sink, int32_t partition_size,
                                           int32_t eight_bit) {
  Split s{};
  if (num_seqs <= 0 || max_query_len < 1 || num_heads <= 0 || num_kv_heads <= 0 ||
      num_heads % num_kv_heads != 0 || head_dim <= 0 || max_seq_len < 1 || window < 0 ||
      num_sink < 0)
    return 0;
  if (!plan_split(&s, num_seqs, max_query_len, num_heads, num_kv_heads, head_dim, max_seq_len,
                  window, num_sink, partition_size, eight_bit != 0))
    return 0;
  return s.total;
}

pkv_status pkv_paged_attention_varlen_window(
    void* out, int32_t out_f32, float* out_lse, const void* q, const void* kv_pool,
    const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
    const int32_t* seq_lens, int32_t num_seqs, int32_t num_tokens, int32_t max_query_len,
    int32_t max_seq_len, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int32_t num_blocks, int32_t window, int32_t num_sink, float scale,
    int32_t partition_size, void* workspace, size_t workspace_bytes, int32_t* dev_status,
    void* stream) {
  return attention(out, out_f32, out_lse, q, kv_pool, nullptr, false, block_table,
                   max_blocks_per_seq, cu_seqlens_q, seq_lens, num_seqs, num_tokens, max_query_len,
                   max_seq_len, num_heads, num_kv_heads, head_dim, block_size, num_blocks, window,
                   num_sink, scale, partition_size, workspace, workspace_bytes, dev_status, stream);
}

pkv_status pkv_paged_attention_varlen_fp8(
    void* out, int32_t out_f32, float* out_lse, const void* q, const void* kv_pool,
    const float* kv_scales, const int32_t* block_table, int32_t max_blocks_per_seq,
    const int32_t* cu_seqlens_q, const int32_t* seq_lens, int32_t num_seqs, int32_t num_tokens,
    int32_t max_query_len, int32_t max_seq_len, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t window, int32_t num_sink,
    float scale, int32_t partition_size, void* workspace, size_t workspace_bytes,
    int32_t* dev_status, void* stream) {
  return attention(out, out_f32, out_lse, q, kv_pool, kv_scales, true, block_table,
                   max_blocks_per_seq, cu_seqlens_q, seq_lens, num_seqs, num_tokens, max_query_len,
                   max_seq_len, num_heads, num_kv_heads, head_dim, block_size, num_blocks, window,
                   num_sink, scale, partition_size, workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"
