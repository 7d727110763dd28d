// launch.h -- internal launch interface between the C-ABI layer (api.cpp)
// and the kernels. Not part of the public ABI.
#pragma once

#include <cuda.h>  // CUtensorMap (type only; no driver-API linkage)
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

namespace pkv {

// A kernel's dynamic shared-memory limit is a per-device attribute: raise it
// once on every device the process launches the kernel on (thread-safe; a
// process may drive several GPUs from several host threads).
class SmemLimit {
 public:
  // carveout >= 0: the preferred share of an SM's memory that is shared memory, in %.
  cudaError_t ensure(const void* func, int bytes, int carveout = -1) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
    std::lock_guard<std::mutex> lock(mu_);
    if (done_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && carveout >= 0)
      e = cudaFuncSetAttribute(func, cudaFuncAttributePreferredSharedMemoryCarveout, carveout);
    if (e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
    return e;
  }

 private:
  static constexpr int kMaxDevices = 64;
  std::mutex mu_;
  std::atomic<bool> done_[kMaxDevices] = {};
};

struct KvWriteParams {
  void* pool;                 // [2][NB][BS][Hkv][D] bf16
  const void* k_new;          // [T][Hkv][D] bf16
  const void* v_new;          // [T][Hkv][D] bf16
  const int32_t* slot_mapping;  // [T]
  int32_t num_tokens;
  int64_t num_slots;          // NB * BS
  int32_t row_vecs;           // 16-byte vectors per token row = Hkv * D / 8
  int32_t* status;
};

// Attention problem shared by the decode, merge and prefill kernels.
// Key segments of a shared prefix of L tokens in the cascade's prefix pass:
// its 128-key tiles cut into segments of prefix_tiles_per_segment tiles, of
// which prefix_segment_count are non-empty (at most `splits`).
__host__ __device__ inline int prefix_tiles_per_segment(int L, int splits) {
  const int t = (L + 127) / 128;
  return (t + splits - 1) / splits;
}
__host__ __device__ inline int prefix_segment_count(int L, int splits) {
  const int t = (L + 127) / 128;
  const int tps = prefix_tiles_per_segment(L, splits);
  return tps > 0 ? (t + tps - 1) / tps : 0;
}

struct AttnParams {
  float* out;                 // [T][H][D] fp32
  float* out_lse;             // [T][H] fp32 or null
  const uint16_t* q;          // [T][H][D] bf16
  const void* kv_pool;        // [2][NB][BS][Hkv][D] bf16
  const int32_t* block_table; // [B][max_blocks]
  const int32_t* cu_seqlens;  // [B+1]; null: one query per request (request i is query i)
  const int32_t* seq_lens;    // [B]
  int32_t max_blocks;
  int32_t num_seqs, num_tokens, max_query_len, max_seq_len;
  int32_t num_heads, num_kv_heads, head_dim, block_size, num_blocks;
  float scale_log2;           // scale * log2(e)
  // split-KV for query_len == 1 requests (merged by the decode merge grid)
  int32_t part_size;          // tokens per partition (multiple of 16)
  int32_t num_parts;          // partitions per request covering max_seq_len
  float* ws_out;              // [B][num_parts][H][D] (null when num_parts == 1)
  float* ws_lse;              // [B][num_parts][H]
  int32_t* sched;             // prefill work tickets: [0] next item, [1] CTAs done;
                              // zero between calls
  int32_t* status;
  // key-range mode (both null otherwise): the keys of request i in its block
  // table sit at absolute positions key_start[i] + p, its queries at
  // query_start[i] + j; query j sees key p iff key_start + p <= query_start + j
  const int32_t* key_start;
  const int32_t* query_start;
  // requests of 1 .. decode_max_q queries run on the decode kernel (its MMA
  // rows are (query, head) pairs, at most decode_max_rows per request in the
  // launch); longer ones on the prefill kernel
  int32_t decode_max_q, decode_max_rows;
  // shared-prefix (cascade) pass of the prefill kernel (prefix_mode 1):
  // every query of a "request" (a prefix group) sees all seq_len keys, no
  // causal mask; the keys are cut into at most kv_splits segments, segment s
  // writing its normalised partial to out + s * split_out_stride and its lse
  // to out_lse + s * split_lse_stride
  int32_t prefix_mode;        // 0: ordinary causal prefill
  int32_t kv_splits;
  int64_t split_out_stride, split_lse_stride;
  // A call with both kinds of request launches the prefill grid, then the
  // decode grid right behind it on the same stream (programmatic dependent
  // launch), the two sharing the SMs:
  //   prefill grid, shared_sms > 0: it keeps about as many of the SMs as
  //     its share of the estimated work (prefill tiles against decode
  //     bytes, out of shared_sms), its other CTAs leave at once, so that
  //     the decode grid -- launched when every prefill CTA has started or
  //     left -- has the rest;
  //   decode grid, after_prefill: its CTAs do not wait for the prefill grid;
  //     one extra CTA (z = num_seqs) waits for it and exits, so that the
  //     decode grid completes only after the prefill grid has.
  //   no_decode: the host has shown that no request is short enough for the
  //     decode kernel (no decode grid is launched); the prefill kernel flags
  //     one that is as PKV_DEV_BAD_LENGTHS (in the calls with a window or an
  //     8-bit pool, whose batches may be padded, it computes that one too).
  int32_t shared_sms;
  int32_t after_prefill;
  int32_t no_decode;
  // decode grid only: request of grid slice z is order[z] (null: z), written
  // by a one-CTA kernel launched before the decode grid (longest context
  // first)
  int32_t* order;
  // decode grid only: the kernel enqueued right before it is this call's own
  // KV write (pkv_paged_attention_varlen_append), which writes only the slots
  // of the requests' query positions: CTAs of a plain decode batch read the
  // keys before the first query's position without waiting for it
  int32_t early_pool;
  // The calls with a window or an 8-bit pool: query position p sees key j iff
  // j <= p and (window == 0 or p - j < window or j < num_sink). out_bf16: `out`
  // holds bf16. scales: [2][NB][Hkv] of an e4m3 pool, else null.
  int32_t window, num_sink;
  int32_t out_bf16;
  const float* scales;
  // their decode grid (decode_rows.cu): the shares that the contexts are cut into;
  // with whole_segments no context is divided. ws_out: the pieces of divided
  // contexts, ws_lse: where the shares begin
  int32_t num_shares, whole_segments;
  float* prefill_parts;       // their prefill grid's pieces of divided items
  int32_t prefill_join;       // a grid of its own joins these
};

// The keys that the queries of one request see, in units of `tile` keys: the
// first `sink` units and those from unit `low` on, `count` in all up to the end
// of the context. (Without a window all of them.) Unit v of these is unit
// v < sink ? v : v - sink + low of the context.
struct Visible {
  int sink, low, count;
  __host__ __device__ int unit(int v) const { return v < sink ? v : v - sink + low; }
};
// qpos0: position of the first query; kv_end: one past the last key needed.
__host__ __device__ inline Visible visible_units(int window, int num_sink, int qpos0, int kv_end,
                                                 int tile) {
  Visible v;
  const int first = window > 0 && qpos0 >= window ? qpos0 - window + 1 : 0;
  v.low = first / tile;
  // (in 64 bits: num_sink may be any int)
  const int64_t s = ((int64_t)num_sink + tile - 1) / tile;
  v.sink = window > 0 ? (int)(s < v.low ? s : v.low) : 0;
  v.count = v.sink + (kv_end + tile - 1) / tile - v.low;
  return v;
}

cudaError_t launch_kv_write(const KvWriteParams& p, cudaStream_t stream);

// pkv_paged_attention_varlen with its workspace in caller-independent scratch
// of `scratch_bytes` bytes whose device address `scratch` returns (for the
// current device). Every host-side check runs first; a call whose workspace
// would exceed the scratch returns PKV_ERR_WORKSPACE; nothing is enqueued on
// an error. The work tickets are cleared on the stream before the launches.
int32_t attention_with_scratch(float* out, float* out_lse, const void* q, const void* kv_pool,
                               const int32_t* block_table, int32_t max_blocks_per_seq,
                               const int32_t* cu_seqlens_q, const int32_t* seq_lens,
                               int32_t num_seqs, int32_t num_tokens, int32_t max_query_len,
                               int32_t max_seq_len, int32_t num_heads, int32_t num_kv_heads,
                               int32_t head_dim, int32_t block_size, int32_t num_blocks,
                               float scale, int32_t partition_size, int32_t* dev_status,
                               void* stream, size_t scratch_bytes,
                               cudaError_t (*scratch)(void**));

// Decode kernel (query_len == 1 requests): TMA-staged pages, QK^T and PV on
// the warp-level tensor cores (mma.sync); split-KV partitions merged by a
// second, small grid launched behind it. `kv_map` views the pool as
// [D/64][Hkv][2*NB*BS rows][64] (strides 128 B, D*2, Hkv*D*2) with a box of
// {64, 16, 1, D/64} and 128-byte swizzle. Up to 16 query heads per CTA.
cudaError_t launch_decode_mma(const AttnParams& p, const CUtensorMap& kv_map,
                              cudaStream_t stream);

// The decode kernel of the calls with a window or an 8-bit pool (requests of up to
// decode_max_q queries). `kv_map`: of a bf16 pool as for launch_decode_mma, of an
// 8-bit one encode_kv8_view. Divided contexts are joined by a second grid, unless
// p.whole_segments.
cudaError_t launch_decode_rows(const AttnParams& p, const CUtensorMap& kv_map, cudaStream_t stream);
// Bytes of its pieces and cuts (which start at *cuts) for requests of up to
// max_rows (query, head) rows.
size_t decode_rows_workspace(int32_t num_kv_heads, int32_t max_rows, int32_t head_dim, bool eight,
                             size_t* cuts);

// Chunked-prefill kernel (query_len > 1 requests), tcgen05 tensor cores.
// `q_map`: q as [T][H][D] with a box of {64, G, 128/G}, 128-byte swizzle.
// `kv_map`: the pool viewed as for the decode kernel but with a box of
// {64, 16, 1, 1} (one 64-column chunk of 16 keys), 128-byte swizzle.
// Launched with programmatic dependent launch: its CTAs start work after the
// preceding grid has completed, and let the next grid launch as soon as
// each has started.
cudaError_t launch_prefill(const AttnParams& p, const CUtensorMap& q_map,
                           const CUtensorMap& kv_map, cudaStream_t stream);

// Whether the prefill kernel's shared memory (its K/V/Q stages plus the work
// list of num_seqs requests) fits the 227 KB a CTA may have: up to 8575
// requests at head_dim 128, 33151 at 64. False for other head dims.
bool prefill_fits(int32_t num_seqs, int32_t head_dim);

// The same of the calls with a window or an 8-bit pool: requests of more than
// decode_max_q queries. `kv_map`: of a bf16 pool as for launch_prefill, of an 8-bit
// one encode_kv8_view. prefill_rows_sched() bytes of p.sched are zero before the
// launch; p.prefill_parts has prefill_rows_workspace() bytes.
size_t prefill_rows_sched();
size_t prefill_rows_workspace(int32_t head_dim);
cudaError_t launch_prefill_rows(const AttnParams& p, const CUtensorMap& q_map,
                                const CUtensorMap& kv_map, cudaStream_t stream);
bool prefill_rows_fits(int32_t num_seqs, int32_t head_dim);
// Behind that grid (and the decode grid's), where p.prefill_join is set: joins the items
// that were cut. That is faster where each is cut into many pieces, in calls of few
// items (64 queries of 32 heads over 65536 keys, 8 items, 8 bits: 102 us; 109 when the
// CTA that comes last joins its item's pieces); the launch costs more than it saves
// where there are two of each (a mixed batch in a graph: 42.7 us, 38.2).
bool prefill_rows_join(const AttnParams& p);
cudaError_t launch_prefill_rows_join(const AttnParams& p, cudaStream_t stream);

// Shared-prefix (cascade) merge: row r of out (num_rows = B * H rows of
// head_dim) from the tail partial (slot 0) and the prefix segments (slots
// 1 .. segments of its request's group, prefix_segment_count of the group's
// prefix length; none for a request outside every group), each slot
// [num_rows][head_dim] fp32 with lse [num_rows]. Launched with programmatic
// dependent launch (waits for the grid before it).
cudaError_t launch_cascade_merge(float* out, float* out_lse, const float* part_out,
                                 const float* part_lse, int64_t num_rows, int32_t num_heads,
                                 int32_t head_dim, const int32_t* group_starts,
                                 const int32_t* prefix_lens, int32_t num_groups, int32_t splits,
                                 cudaStream_t stream);

// Whole-block copies in the pool; block_vecs = 16-byte vectors in one
// block of one half (K or V); scales: of an 8-bit pool, else null.
cudaError_t launch_copy_blocks(void* pool, const int32_t* src, const int32_t* dst,
                               int32_t num_copies, int32_t num_blocks, int64_t block_vecs,
                               float* scales, int32_t num_kv_heads, int32_t* status,
                               cudaStream_t stream);

// Public dense merge: part_out [P][T*H][D], part_lse [P][T*H].
cudaError_t launch_lse_merge(float* out, float* out_lse, const float* part_out,
                             const float* part_lse, int32_t num_parts, int64_t num_rows,
                             int32_t head_dim, cudaStream_t stream);

// The encoded TMA views that several calls use (api.cpp); false when the
// driver's encoder is missing or refuses.
// Pool as [D/64][Hkv][2*NB*BS rows][64], boxes of 16 rows of one KV head and
// `chunks` 64-column chunks.
bool encode_kv_view(CUtensorMap* map, const void* kv_pool, int32_t num_blocks, int32_t block_size,
                    int32_t num_kv_heads, int32_t head_dim, uint32_t chunks);
// The 8-bit pool as [Hkv][2*NB*BS rows][D] bytes, boxes of 16 rows of one KV
// head, 128-byte swizzle for 128-byte rows, 64-byte for 64.
bool encode_kv8_view(CUtensorMap* map, const void* kv_pool, int32_t num_blocks, int32_t block_size,
                     int32_t num_kv_heads, int32_t head_dim);
// q [T][H][D] in boxes of {64 columns, G heads, 128/G tokens}.
bool encode_q_tiles(CUtensorMap* map, const void* q, int32_t num_tokens, int32_t num_heads,
                    int32_t num_kv_heads, int32_t head_dim);

struct RopeWriteParams {
  uint16_t* q_out;            // [T][H][D] bf16
  void* pool;                 // [2][NB][BS][Hkv][D] bf16
  const uint16_t* q;          // rows of [H][D], q_stride elements apart
  const uint16_t* k;          // rows of [Hkv][D]
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* positions;   // [T]
  const int32_t* slots;       // [T]
  const double* inv_freq;     // [rotary_dim / 2] radians per position
  float factor;
  int32_t interleaved;
  int32_t num_tokens, num_heads, num_kv_heads, head_dim, rotary_dim;
  int64_t num_slots;          // NB * BS
  int32_t* status;
};
cudaError_t launch_rope_write(const RopeWriteParams& p, cudaStream_t stream);

// Norms of the query and key heads, rotation and cache write. Into a bf16 pool
// through `slots`, or (append) into an 8-bit pool through the requests' tables.
struct NormRopeParams {
  uint16_t* q_out;            // [T][H][D] bf16
  void* pool;                 // [2][NB][BS][Hkv][D] bf16, or e4m3
  float* scales;              // append: [2][NB][Hkv]
  const uint16_t* q;          // rows of [H][D], q_stride elements apart (append: may be null)
  const uint16_t* k;          // rows of [Hkv][D]
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* positions;   // [T]; null: nothing is rotated
  const int32_t* slots;       // [T] (bf16 pool)
  const double* inv_freq;     // [rotary_dim / 2] radians per position
  const void* q_weight;       // [D] bf16 or fp32; null: not normed
  const void* k_weight;
  int32_t weight_f32;
  float weight_offset, eps, factor;
  int32_t interleaved;
  int32_t num_tokens, num_heads, num_kv_heads, head_dim, rotary_dim;
  int64_t num_slots;          // NB * BS
  const int32_t* block_table; // append: [B][max_blocks]
  const int32_t* cu_seqlens;  // [B+1]
  const int32_t* seq_lens;    // [B]
  int32_t max_blocks, num_seqs, max_query_len, block_size, num_blocks;
  int32_t* status;
};
cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream);
cudaError_t launch_append_fp8(const NormRopeParams& p, cudaStream_t stream);

struct KeyWeightsParams {
  float* out;                 // [rows][Hkv][row_len]
  const float* in;            // the same shape; may be out
  const uint16_t* q;          // [T][H][D] bf16
  const uint16_t* pool;       // [2][NB][BS][Hkv][D] bf16
  const float* lse;           // [T][H]
  const int32_t* block_table; // [B][max_blocks]
  const int32_t* cu_seqlens;  // [B+1]
  const int32_t* seq_lens;    // [B]
  const int32_t* prior_lens;  // [B] or null: seq_len - query_len
  const int32_t* rows;        // [B] or null: row i
  int32_t num_rows, row_len, max_blocks;
  int32_t num_seqs, num_tokens, max_query_len, max_seq_len;
  int32_t num_heads, num_kv_heads, head_dim, block_size, num_blocks;
  float scale_log2;           // scale * log2(e)
  float decay;
  // requests of up to short_max_q queries run on the mma.sync grid, longer
  // ones on the tcgen05 grid; 0: all on the former. no_short: the former is
  // not launched, the latter flags a short request as PKV_DEV_BAD_LENGTHS
  int32_t short_max_q;
  int32_t no_short;
  int32_t after_tc;           // mma.sync grid: launched right behind the tcgen05 grid
  int32_t* status;
};
cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream);
// Requests longer than short_max_q; `q_map` as for the prefill kernel (boxes
// of 128 / G queries), `k_map` the pool in boxes of 16 keys and one 64-column
// chunk.
cudaError_t launch_key_weights_tc(const KeyWeightsParams& p, const CUtensorMap& q_map,
                                  const CUtensorMap& k_map, cudaStream_t stream);

struct EvictSelectParams {
  int32_t* kept;              // [B][Hkv][max_keep]
  float* out;                 // [rows][Hkv][row_len] or null
  const float* weights;       // [rows][Hkv][row_len]
  const int32_t* seq_lens;    // [B]
  const int32_t* keep_lens;   // [B]
  const int32_t* rows;        // [B] or null
  int32_t num_rows, row_len, num_seqs, num_kv_heads, max_seq_len, max_keep;
  int32_t num_sink, num_recent;
  int32_t* status;
};
cudaError_t launch_evict_select(const EvictSelectParams& p, cudaStream_t stream);

struct EvictCompactParams {
  uint4* pool;                // [2][NB][BS][Hkv][D] bf16
  const int32_t* src_table;   // [B][max_src]
  const int32_t* dst_table;   // [B][max_dst]
  const int32_t* kept;        // [B][Hkv][max_keep]
  const int32_t* keep_lens;   // [B]
  int32_t max_src, max_dst, max_keep, num_seqs, num_kv_heads, head_vecs, block_size, num_blocks;
  int32_t* status;
};
cudaError_t launch_evict_compact(const EvictCompactParams& p, cudaStream_t stream);

}  // namespace pkv
