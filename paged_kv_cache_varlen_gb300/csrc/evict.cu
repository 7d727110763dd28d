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
// largest value (digits of 11, 11 and 10 bits, a histogram each; it ends early
// when a digit's bin is taken whole), then one pass that writes the keys above
// it and the first of those equal to it, in index order.
//
// A row (request, KV head) is read once: its keys stay in the registers of the
// 512 threads of one CTA, or of a cluster of 2, 4 or 8 when it is long or the
// rows are few; the CTAs' histograms are added up over distributed shared
// memory. Rows past 131072 keys are read again for each digit (from L2). The
// row's 4 bytes a key are little: the passes' barriers and the histograms'
// atomics bound it.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

// Order-preserving key of a weight: larger weights have larger keys, -0 and
// +0 the same one, a NaN the largest.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0xffffffffu;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The int at the same shared-memory offset of cluster CTA `rank`.
__device__ __forceinline__ int ld_cluster(const int* p, int rank) {
  uint32_t remote;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// K: 32-key steps of a warp's share held in registers; 0: the row is read
// from memory in every pass.
template <int K>
__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const EvictSelectParams p, const int clusters) {
  __shared__ int hist[kBins];
  __shared__ int warp_sum[kSelWarps];
  __shared__ int found_bin, found_left, found_whole;
  __shared__ int warp_gt[kSelWarps], warp_eq[kSelWarps];
  __shared__ int cta_count[2];
  griddep_wait();
  griddep_launch_dependents();
  const int rank = blockIdx.x % clusters, h = blockIdx.x / clusters, i = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int L = __ldg(p.seq_lens + i), keep = __ldg(p.keep_lens + i);
  const int row = p.rows ? __ldg(p.rows + i) : i;
  // the CTAs of a cluster share the row: these exits are uniform
  if (L < 0 || L > p.max_seq_len || keep < 0 || keep > L || keep > p.max_keep) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  if (row < 0 || row >= p.num_rows) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, PKV_DEV_BAD_ROW);
    return;
  }
  if (keep == 0) return;
  const int64_t at = ((int64_t)row * p.num_kv_heads + h) * p.row_len;
  const float* w = p.weights + at;
  const int recent = min(p.num_recent, keep);
  const int sink = min(p.num_sink, keep - recent);
  const int lo = sink, hi = L - recent;  // keys [lo, hi) compete for `left` places
  int left = keep - sink - recent;
  const bool any = left > 0;

  // the warp's share of the row: `steps` times 32 keys, in index order
  const int per_step = clusters * kSelThreads;
  const int steps = (int)(((int64_t)L + per_step - 1) / per_step);
  const int64_t first = (int64_t)(rank * kSelWarps + warp) * steps * 32;
  const int base = (int)min((int64_t)L, first) + lane;
  const int end = (int)min((int64_t)L, first + (int64_t)steps * 32);
  float v[K > 0 ? K : 1];
  if (K > 0) {
#pragma unroll
    for (int j = 0; j < K; ++j) v[j] = base + j * 32 < end ? __ldg(w + base + j * 32) : 0.f;
  }
  // f(index, weight) of the lane's keys, in step with the whole warp
  auto for_keys = [&](auto f) {
    if (K > 0) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (j < steps) f(base + j * 32, v[j]);
    } else {
      for (int j = 0; j < steps; ++j)
        f(base + j * 32, base + j * 32 < end ? __ldg(w + base + j * 32) : 0.f);
    }
  };
  auto sync_cluster = [&] {
    __syncwarp();
    if (clusters > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };

  // the left-th largest key among [lo, hi): its digits from the top
  uint32_t prefix = 0, known = 0;  // the digits found, and their bits
  for (int digit = 0; digit < 3 && any; ++digit) {
    const int shift = digit == 0 ? 21 : (digit == 1 ? 10 : 0);
    const uint32_t mask = digit == 2 ? 1023u : 2047u;
    for (int b = threadIdx.x; b < kBins; b += kSelThreads) hist[b] = 0;
    __syncthreads();
    for_keys([&](int k, float x) {
      const uint32_t key = weight_key(x);
      if (k >= lo && k < hi && k < end && (key & known) == prefix)
        atomicAdd(&hist[(key >> shift) & mask], 1);
    });
    sync_cluster();
    // a thread has 4 bins, counted from the largest; a scan over the threads
    constexpr int kPer = kBins / kSelThreads;
    const int top = kBins - 1 - threadIdx.x * kPer;
    int n[kPer], mine = 0;
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      n[b] = hist[top - b];
      if (clusters > 1) {
        n[b] = 0;
        for (int c = 0; c < clusters; ++c) n[b] += ld_cluster(hist + top - b, c);
      }
      mine += n[b];
    }
    __syncwarp();
    if (clusters > 1) cluster_arrive();  // done with the others' histograms
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = incl - mine;
    for (int x = 0; x < warp; ++x) before += warp_sum[x];
    if (before < left && before + mine >= left) {  // exactly one thread
      int places = left - before, b = 0;
#pragma unroll
      for (int c = 0; c < kPer - 1; ++c)
        if (b == c && places > n[c]) {
          places -= n[c];
          b = c + 1;
        }
      found_bin = top - b;
      found_left = places;
      int size = n[0];
#pragma unroll
      for (int c = 1; c < kPer; ++c)
        if (b == c) size = n[c];
      found_whole = size == places;
    }
    __syncwarp();
    if (clusters > 1) cluster_wait();
    __syncthreads();
    prefix |= (uint32_t)found_bin << shift;
    known |= mask << shift;
    left = found_left;
    if (found_whole) break;  // every key with this prefix is kept
  }

  // kept: the protected keys, the keys above the prefix, and the first `left`
  // of those that match it
  auto classify = [&](int k, float x, bool* take, bool* tie) {
    const uint32_t key = weight_key(x) & known;
    const bool inside = k >= lo && k < hi;
    *take = k < end && (!inside || (any && key > prefix));
    *tie = k < end && inside && any && key == prefix;
  };
  int gt = 0, eq = 0;
  for_keys([&](int k, float x) {
    bool take, tie;
    classify(k, x, &take, &tie);
    gt += take;
    eq += tie;
  });
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
  int ngt = 0, neq = 0;  // kept outright / matching, before this warp's share
  if (clusters > 1) {
    if (threadIdx.x == 0) {
      int a = 0, b = 0;
      for (int x = 0; x < kSelWarps; ++x) {
        a += warp_gt[x];
        b += warp_eq[x];
      }
      cta_count[0] = a;
      cta_count[1] = b;
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    for (int c = 0; c < rank; ++c) {
      ngt += ld_cluster(&cta_count[0], c);
      neq += ld_cluster(&cta_count[1], c);
    }
    cluster_arrive();  // waited for before the CTA exits
  }
  for (int x = 0; x < warp; ++x) {
    ngt += warp_gt[x];
    neq += warp_eq[x];
  }
  int32_t* kept = p.kept + ((int64_t)i * p.num_kv_heads + h) * p.max_keep;
  float* out = p.out ? p.out + at : nullptr;
  const uint32_t below = (1u << lane) - 1;
  for_keys([&](int k, float x) {
    bool take, tie;
    classify(k, x, &take, &tie);
    const uint32_t mt = __ballot_sync(kFull, take), me = __ballot_sync(kFull, tie);
    const int eq_before = neq + __popc(me & below);
    if (take || (tie && eq_before < left)) {
      const int o = ngt + __popc(mt & below) + min(eq_before, left);
      kept[o] = k;
      if (out) out[o] = x;
    }
    ngt += __popc(mt);
    neq += __popc(me);
  });
  if (clusters > 1) {
    __syncwarp();
    cluster_wait();
  }
}

// ---------------------------------------------------------------------------
// Move: row (j, h) of a request is head_dim bf16 values of K and of V; a
// group of head_vecs lanes moves both with 16-byte vectors. Consecutive
// groups take the KV heads of one destination token, so a CTA's destinations
// are contiguous; the sources are runs of head_dim * 2 bytes. Every byte moves
// once: HBM-bound, and a thread has its four rows' loads in flight together.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 4;  // rows of a thread

__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(const EvictCompactParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int i = blockIdx.y;
  const int keep = __ldg(p.keep_lens + i);
  if (keep < 0 || keep > p.max_keep || (int64_t)keep > (int64_t)p.max_dst * p.block_size) {
    if (threadIdx.x == 0 && blockIdx.x == 0) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int groups = kMoveThreads / p.head_vecs;  // rows that the CTA moves at a time
  const int g = threadIdx.x / p.head_vecs, c = threadIdx.x - g * p.head_vecs;
  const int total = keep * p.num_kv_heads;  // (below 2^31: checked by the host)
  const int row0 = blockIdx.x * groups * kMoveRows + g;
  if (g >= groups || row0 >= total) return;
  const int64_t half = (int64_t)p.num_blocks * p.block_size * p.num_kv_heads * p.head_vecs;
  const int32_t* kept = p.kept + (int64_t)i * p.num_kv_heads * p.max_keep;
  const int32_t* src = p.src_table + (int64_t)i * p.max_src;
  const int32_t* dst = p.dst_table + (int64_t)i * p.max_dst;
  int j[kMoveRows], h[kMoveRows], s[kMoveRows], sb[kMoveRows], db[kMoveRows];
#pragma unroll
  for (int u = 0; u < kMoveRows; ++u) {
    const int r = row0 + u * groups;
    j[u] = r / p.num_kv_heads;
    h[u] = r - j[u] * p.num_kv_heads;
    s[u] = r < total ? __ldg(kept + (int64_t)h[u] * p.max_keep + j[u]) : -1;
  }
#pragma unroll
  for (int u = 0; u < kMoveRows; ++u) {
    const bool there = row0 + u * groups < total;
    const int b = s[u] / p.block_size;
    const bool good = s[u] >= 0 && b < p.max_src;
    if (there && !good) set_status(p.status, PKV_DEV_BAD_KEPT);
    sb[u] = good ? __ldg(src + b) : -1;
    db[u] = good ? __ldg(dst + j[u] / p.block_size) : -1;
    if (good && (sb[u] < 0 || sb[u] >= p.num_blocks || db[u] < 0 || db[u] >= p.num_blocks)) {
      set_status(p.status, PKV_DEV_BAD_BLOCK);
      sb[u] = -1;
    }
  }
  uint4 k[kMoveRows], v[kMoveRows];
#pragma unroll
  for (int u = 0; u < kMoveRows; ++u)
    if (sb[u] >= 0) {
      const uint4* from = p.pool + (((int64_t)sb[u] * p.block_size + s[u] % p.block_size) *
                                        p.num_kv_heads + h[u]) * p.head_vecs + c;
      k[u] = from[0];
      v[u] = from[half];
    }
#pragma unroll
  for (int u = 0; u < kMoveRows; ++u)
    if (sb[u] >= 0) {
      uint4* to = p.pool + (((int64_t)db[u] * p.block_size + j[u] % p.block_size) *
                                p.num_kv_heads + h[u]) * p.head_vecs + c;
      to[0] = k[u];
      to[half] = v[u];
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

namespace {

template <int K>
cudaError_t launch_select(const EvictSelectParams& p, int clusters, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg =
      config(dim3((unsigned)(p.num_kv_heads * clusters), (unsigned)p.num_seqs), kSelThreads,
             stream, attr);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)clusters;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<K>, p, clusters);
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads;
  // 16 keys a thread at most, in as few CTAs as hold the row; more CTAs while
  // the rows leave SMs without one and a thread has more than 4 keys
  const int64_t L = p.max_seq_len;
  int clusters = 1;
  while (clusters < kMaxCluster && L > (int64_t)clusters * kSelThreads * 16) clusters *= 2;
  while (clusters < kMaxCluster && rows * clusters * 2 <= 152 &&
         L > (int64_t)clusters * kSelThreads * 4)
    clusters *= 2;
  const int64_t steps = (L + clusters * kSelThreads - 1) / (clusters * kSelThreads);
  if (steps <= 4) return launch_select<4>(p, clusters, stream);
  if (steps <= 8) return launch_select<8>(p, clusters, stream);
  if (steps <= 16) return launch_select<16>(p, clusters, stream);
  if (steps <= 32) return launch_select<32>(p, clusters, stream);
  return launch_select<0>(p, clusters, stream);
}

cudaError_t launch_evict_compact(const EvictCompactParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const int64_t per_cta = (int64_t)(kMoveThreads / p.head_vecs) * kMoveRows;
  const int64_t ctas = ((int64_t)p.max_keep * p.num_kv_heads + per_cta - 1) / per_cta;
  const cudaLaunchConfig_t cfg =
      config(dim3((unsigned)ctas, (unsigned)p.num_seqs), kMoveThreads, stream, attr);
  return cudaLaunchKernelEx(&cfg, evict_compact_kernel, p);
}

}  // namespace pkv
