// window_api.cpp -- the C ABI of attention through a window and over an 8-bit
// cache (declared in include/pkv.h): host-side checks and dispatch. As in
// api.cpp, every check and encoding runs before the first launch.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/pkv.h"
#include "launch.h"

namespace {

using pkv::AttnParams;

// Contexts of up to this many 16-key chunks are not divided: the grid that joins the
// pieces would cost more (64 single tokens, 200 of their keys seen: 19.1 us, 20.2 in
// shares; 8 tokens, 220 keys: 9.6 and 10.5. At twice as many keys 28.9 and 28.9; 8
// tokens 11.9 and 10.8).
constexpr int32_t kWholeChunks = 16;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether the byte ranges [a, a + na) and [b, b + nb) meet.
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (na == 0 || nb == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// How a call's short requests (up to 32 / G queries) run.
struct Plan {
  int32_t max_q;  // queries of the requests that the decode grid takes
  int32_t rows;   // (query, head) rows of one KV head that they have at most
  bool whole;     // no context is divided
  size_t cuts_off, sched_off, parts_off, total;
};

Plan plan_calls(int32_t max_query_len, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                int32_t max_seq_len, int32_t window, int32_t num_sink, bool eight) {
  Plan s{};
  const int32_t group = num_heads / num_kv_heads;
  s.max_q = 32 / group > 1 ? 32 / group : 1;
  const int32_t q = max_query_len < s.max_q ? max_query_len : s.max_q;
  s.rows = q * group;
  // keys that some query of a request sees, in 16-key chunks
  int64_t seen = ((int64_t)max_seq_len + 15) / 16;
  if (window > 0) {
    const int64_t most = ((int64_t)num_sink + 15) / 16 + ((int64_t)window + q + 14) / 16 + 1;
    if (most < seen) seen = most;
  }
  s.whole = seen <= kWholeChunks;
  if (!s.whole) {
    const size_t n = pkv::decode_rows_workspace(num_kv_heads, s.rows, head_dim, eight, &s.cuts_off);
    s.sched_off = round_up(n, 256);
  }
  s.parts_off = s.total = s.sched_off;
  if (max_query_len > s.max_q) {
    s.parts_off += round_up(pkv::prefill_rows_sched(), 256);
    s.total = s.parts_off + pkv::prefill_rows_workspace(head_dim);
  }
  if (s.total == 0) s.total = 256;  // (never none, so that a caller's pointer is not null)
  return s;
}

// Common to both calls; `scales` non-null: an 8-bit pool.
pkv_status attention(void* out, int32_t out_f32, float* out_lse, const void* q, const void* kv_pool,
                     const float* scales, bool eight, const int32_t* block_table,
                     int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
                     const int32_t* seq_lens, int32_t num_seqs, int32_t num_tokens,
                     int32_t max_query_len, int32_t max_seq_len, int32_t num_heads,
                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                     int32_t num_blocks, int32_t window, int32_t num_sink, float scale,
                     void* workspace, size_t workspace_bytes,
                     int32_t* dev_status, void* stream) {
  if (num_seqs < 0 || num_tokens < 0) return PKV_ERR_INVALID_ARG;
  if (num_tokens == 0) return PKV_OK;
  if (num_seqs == 0) return PKV_ERR_INVALID_ARG;
  if (num_seqs > 65534) return PKV_ERR_UNSUPPORTED;  // (as pkv_paged_attention_varlen)
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
  const Plan sp = plan_calls(max_query_len, num_heads, num_kv_heads, head_dim, max_seq_len, window,
                             num_sink, eight);
  const bool prefill = max_query_len > sp.max_q;
  if (prefill && (group > 128 || !pkv::prefill_rows_fits(num_seqs, head_dim)))
    return PKV_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < sp.total || !aligned(workspace, 256))
    return PKV_ERR_WORKSPACE;
  // what is written meets nothing that is read
  const int64_t out_rows = (int64_t)num_tokens * num_heads;
  const int64_t pool_values = (int64_t)2 * num_blocks * block_size * num_kv_heads * head_dim;
  struct Range {
    const void* at;
    int64_t bytes;
  };
  const Range written[] = {{out, out_rows * head_dim * (out_f32 ? 4 : 2)},
                           {out_lse, out_lse ? out_rows * 4 : 0},
                           {workspace, (int64_t)sp.total}};
  const Range read[] = {{q, out_rows * head_dim * 2},
                        {kv_pool, pool_values * (eight ? 1 : 2)},
                        {scales, eight ? (int64_t)2 * num_blocks * num_kv_heads * 4 : 0}};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlap(written[i].at, written[i].bytes, read[j].at, read[j].bytes))
        return PKV_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(written[i].at, written[i].bytes, written[j].at, written[j].bytes))
        return PKV_ERR_INVALID_ARG;
  }

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
  // without a window, or with one past every context, every key lies in it (2^30:
  // positions minus it stay in 32 bits)
  p.window = window > 0 && window < (1 << 30) ? window : 1 << 30;
  p.num_sink = num_sink;
  char* ws = static_cast<char*>(workspace);
  p.whole_segments = sp.whole;
  p.ws_out = reinterpret_cast<float*>(ws);
  p.ws_lse = reinterpret_cast<float*>(ws + sp.cuts_off);
  p.sched = reinterpret_cast<int32_t*>(ws + sp.sched_off);
  p.prefill_parts = reinterpret_cast<float*>(ws + sp.parts_off);
  p.status = dev_status;
  p.decode_max_q = sp.max_q;
  p.decode_max_rows = sp.rows;
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
    return pkv::launch_decode_rows(d, rows, st) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  };
  if (!prefill) return decode(p);
  // the prefill grid, then (unless no request can be short) the decode grid on
  // the SMs that it leaves, as in api.cpp; the work tickets start at zero
  if (cudaMemsetAsync(p.sched, 0, pkv::prefill_rows_sched(), st) != cudaSuccess) return PKV_ERR_CUDA;
  const bool any_short = (int64_t)num_seqs * max_query_len - num_tokens >=
                         (int64_t)max_query_len - sp.max_q;
  p.prefill_join = pkv::prefill_rows_join(p);
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
  if (pkv::launch_prefill_rows(pp, q_map, eight ? rows : boxes, st) != cudaSuccess) return PKV_ERR_CUDA;
  if (any_short) {
    p.after_prefill = 1;
    if (pkv_status e = decode(p); e != PKV_OK) return e;
  }
  if (!p.prefill_join) return PKV_OK;
  return pkv::launch_prefill_rows_join(p, st) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace

extern "C" {

size_t pkv_window_attention_workspace_size(int32_t max_query_len, int32_t num_heads,
                                           int32_t num_kv_heads, int32_t head_dim,
                                           int32_t max_seq_len, int32_t window, int32_t num_sink,
                                           int32_t eight_bit) {
  if (max_query_len < 1 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128) || max_seq_len < 1 || window < 0 || num_sink < 0)
    return 0;
  return plan_calls(max_query_len, num_heads, num_kv_heads, head_dim, max_seq_len, window, num_sink,
                    eight_bit != 0)
      .total;
}

pkv_status pkv_paged_attention_varlen_window(
    void* out, int32_t out_f32, float* out_lse, const void* q, const void* kv_pool,
    const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* cu_seqlens_q,
    const int32_t* seq_lens, int32_t num_seqs, int32_t num_tokens, int32_t max_query_len,
    int32_t max_seq_len, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int32_t num_blocks, int32_t window, int32_t num_sink, float scale,
    void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return attention(out, out_f32, out_lse, q, kv_pool, nullptr, false, block_table,
                   max_blocks_per_seq, cu_seqlens_q, seq_lens, num_seqs, num_tokens, max_query_len,
                   max_seq_len, num_heads, num_kv_heads, head_dim, block_size, num_blocks, window,
                   num_sink, scale, workspace, workspace_bytes, dev_status, stream);
}

pkv_status pkv_paged_attention_varlen_fp8(
    void* out, int32_t out_f32, float* out_lse, const void* q, const void* kv_pool,
    const float* kv_scales, const int32_t* block_table, int32_t max_blocks_per_seq,
    const int32_t* cu_seqlens_q, const int32_t* seq_lens, int32_t num_seqs, int32_t num_tokens,
    int32_t max_query_len, int32_t max_seq_len, int32_t num_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int32_t num_blocks, int32_t window, int32_t num_sink,
    float scale, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
  return attention(out, out_f32, out_lse, q, kv_pool, kv_scales, true, block_table,
                   max_blocks_per_seq, cu_seqlens_q, seq_lens, num_seqs, num_tokens, max_query_len,
                   max_seq_len, num_heads, num_kv_heads, head_dim, block_size, num_blocks, window,
                   num_sink, scale, workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"
