// evict.cu -- cutting a request's cached context back to the keys that carry
// the most accumulated attention weight: the selection (per request and KV
// head) and the move of the kept rows to fresh blocks.
#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr uint32_t kFull = 0xffffffffu;

// ---------------------------------------------------------------------------
// Selection: the n heaviest of a row's keys by a radix search for the n-th
// largest value (three digits of 11, 11 and 10 bits, a histogram each), then
// one pass that writes the keys above it and the first of those equal to it,
// in index order.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// Order-preserving key of a weight: larger weights have larger keys, -0 and
// +0 the same one, a NaN the largest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictSelectParams p) {
  __shared__ int hist[kBins];
  __shared__ int warp_sum[kSelWarps];
  __shared__ int found_bin, found_rest;
  __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.x, i = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int L = __ldg(p.seq_lens + i), keep = __ldg(p.keep_lens + i);
  const int row = p.rows ? __ldg(p.rows + i) : i;
  if (L < 0 || L > p.max_seq_len || keep < 0 || keep > L || keep > p.max_keep) {
    if (threadIdx.x == 0 && h == 0) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  if (row < 0 || row >= p.num_rows) {
    if (threadIdx.x == 0 && h == 0) set_status(p.status, PKV_DEV_BAD_ROW);
    return;
  }
  if (keep == 0) return;
  const int64_t at = ((int64_t)row * p.num_kv_heads + h) * p.row_len;
  const float* w = p.weights + at;
  const int recent = min(p.num_recent, keep);
  const int sink = min(p.num_sink, keep - recent);
  const int lo = sink, hi = L - recent;  // keys [lo, hi) compete for `rest` places
  int rest = keep - sink - recent;

  // the rest-th largest key among [lo, hi): its digits from the top
  uint32_t prefix = 0;
  for (int digit = 0; digit < 3 && rest > 0; ++digit) {
    const int shift = digit == 0 ? 21 : (digit == 1 ? 10 : 0);
    const uint32_t mask = digit == 2 ? 1023u : 2047u;
    const uint32_t above = digit == 0 ? 0u : 0xffffffffu << (digit == 1 ? 21 : 10);
    for (int b = threadIdx.x; b < kBins; b += kSelThreads) hist[b] = 0;
    __syncthreads();
    for (int k = lo + threadIdx.x; k < hi; k += kSelThreads) {
      const uint32_t key = weight_key(w[k]);
      if ((key & above) == prefix) atomicAdd(&hist[(key >> shift) & mask], 1);
    }
    __syncthreads();
    // each thread sums 4 bins, counted from the largest; a scan over threads
    constexpr int kPer = kBins / kSelThreads;
    const int top = kBins - 1 - threadIdx.x * kPer;
    int mine = 0;
#pragma unroll
    for (int b = 0; b < kPer; ++b) mine += hist[top - b];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - mine;
    for (int x = 0; x < warp; ++x) before += warp_sum[x];
    if (before < rest && before + mine >= rest) {  // exactly one thread
      int left = rest - before;
      int b = top;
      while (left > hist[b]) left -= hist[b--];
      found_bin = b;
      found_rest = left;
    }
    __syncthreads();
    prefix |= (uint32_t)found_bin << shift;
    rest = found_rest;
  }
  // now: every key above `prefix` is kept, and the first `rest` equal to it
  const bool any = keep > sink + recent;

  // each warp takes a contiguous share of [0, L)
  const int share = ((L + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int b0 = min(L, warp * share), b1 = min(L, b0 + share);
  int gt = 0, eq = 0;
  for (int k = b0 + lane; k < b1; k += 32) {
    if (k < lo || k >= hi)
      ++gt;
    else if (any) {
      const uint32_t key = weight_key(w[k]);
      gt += key > prefix;
      eq += key == prefix;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(kFull, gt, o);
    eq += __shfl_xor_sync(kFull, eq, o);
  }
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  int ngt = 0, neq = 0;  // kept outright / equal, before this warp's share
  for (int x = 0; x < warp; ++x) {
    ngt += warp_gt[x];
    neq += warp_eq[x];
  }
  int32_t* kept = p.kept + ((int64_t)i * p.num_kv_heads + h) * p.max_keep;
  float* out = p.out ? p.out + at : nullptr;
  const uint32_t below = (1u << lane) - 1;
  for (int k0 = b0; k0 < b1; k0 += 32) {
    const int k = k0 + lane;
    bool take = false, tie = false;
    float v = 0.f;
    if (k < b1) {
      v = w[k];
      if (k < lo || k >= hi)
        take = true;
      else if (any) {
        const uint32_t key = weight_key(v);
        take = key > prefix;
        tie = key == prefix;
      }
    }
    const uint32_t mt = __ballot_sync(kFull, take), me = __ballot_sync(kFull, tie);
    const int eq_before = neq + __popc(me & below);
    if (take || (tie && eq_before < rest)) {
      const int o = ngt + __popc(mt & below) + min(eq_before, rest);
      kept[o] = k;
      if (out) out[o] = v;
    }
    ngt += __popc(mt);
    neq += __popc(me);
  }
}

// ---------------------------------------------------------------------------
// Move: row (j, h) of a request is head_dim bf16 values of K and of V; a
// group of head_vecs lanes moves both with 16-byte vectors. Consecutive
// groups take the KV heads of one destination token, so the destinations of
// a CTA are contiguous; the sources are runs of head_dim * 2 bytes.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const EvictCompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.y;
  const int keep = __ldg(p.keep_lens + i);
  if (keep < 0 || keep > p.max_keep || (int64_t)keep > (int64_t)p.max_dst * p.block_size) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int64_t half = (int64_t)p.num_blocks * p.block_size * p.num_kv_heads * p.head_vecs;
  const int64_t total = (int64_t)keep * p.num_kv_heads * p.head_vecs;
  for (int64_t v = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; v < total;
       v += (int64_t)gridDim.x * kMoveThreads) {
    const int64_t rr = v / p.head_vecs;
    const int c = (int)(v - rr * p.head_vecs);
    const int j = (int)(rr / p.num_kv_heads), h = (int)(rr - (int64_t)j * p.num_kv_heads);
    const int s = __ldg(p.kept + ((int64_t)i * p.num_kv_heads + h) * p.max_keep + j);
    if (s < 0 || s >= (int64_t)p.max_src * p.block_size) {
      set_status(p.status, PKV_DEV_BAD_KEPT);
      continue;
    }
    const int sb = __ldg(p.src_table + (int64_t)i * p.max_src + s / p.block_size);
    const int db = __ldg(p.dst_table + (int64_t)i * p.max_dst + j / p.block_size);
    if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
      set_status(p.status, PKV_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t from = (((int64_t)sb * p.block_size + s % p.block_size) * p.num_kv_heads + h) *
                             p.head_vecs + c;
    const int64_t to = (((int64_t)db * p.block_size + j % p.block_size) * p.num_kv_heads + h) *
                           p.head_vecs + c;
    const uint4 a = p.pool[from], b = p.pool[from + half];
    p.pool[to] = a;
    p.pool[to + half] = b;
  }
}

cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(dim3((unsigned)p.num_kv_heads, (unsigned)p.num_seqs),
                                        kSelThreads, stream, attr);
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
}

cudaError_t launch_evict_compact(const EvictCompactParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const int64_t vecs = (int64_t)p.max_keep * p.num_kv_heads * p.head_vecs;
  const int64_t ctas = (vecs + kMoveThreads - 1) / kMoveThreads;
  const cudaLaunchConfig_t cfg = config(
      dim3((unsigned)(ctas < (1 << 20) ? ctas : (1 << 20)), (unsigned)p.num_seqs), kMoveThreads,
      stream, attr);
  return cudaLaunchKernelEx(&cfg, evict_compact_kernel, p);
}

}  // namespace pkv
