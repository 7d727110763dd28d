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
// largest value (digits of 11, 11 and 10 bits, a histogram each), then one pass
// that writes the keys above it and the first of those equal to it, in index
// order. The search ends early when a digit's bin is taken whole, or when it
// is so small that its keys can be ranked against one another (the usual case
// after one digit of some thousand keys).
//
// A row (request, KV head) is read once into the shared memory of one CTA, or
// of a cluster of 2, 4 or 8 when it is long or the rows are few; the CTAs'
// histograms are added up in the first one's. Rows of more than kStaged keys a
// CTA are read again in each pass (from L2). The row's 4 bytes a key are
// little: the instructions of the passes bound it (73 % of the issue slots),
// or their barriers when the rows are few. Measured: 64 x 8 rows of 1500 to
// 8192 keys, 1024 kept: 21.4 us; 2 x 8 rows of 128K, 8192 kept: 24 us.
// ---------------------------------------------------------------------------
constexpr int kBins = 2048;
constexpr int kScanThreads = 512;  // four bins each
constexpr int kMaxCluster = 8;
constexpr int kStaged = 40960;     // keys of a CTA's share that shared memory holds
// Copies of the histogram, one for each lane modulo kCopies: attention weights
// crowd into a few dozen bins of the first digit. Each starts 8 banks on, so
// that a bin's copies lie in different banks.
constexpr int kCopies = 2;
constexpr int kCopyStride = kBins + 8;
constexpr int kRanked = 384;  // keys at most that are ranked against one another

// Order-preserving key of a weight: larger weights have larger keys, -0 and
// +0 the same one, a NaN the largest but kProtected, which stands for the keys
// that are kept whatever their weight (and so need no care of their own: the
// selection is the `keep` largest keys of the row).
constexpr uint32_t kProtected = 0xffffffffu;
__device__ __forceinline__ uint32_t weight_key(float w) {
  const int32_t b = __float_as_int(w + 0.f);
  return w != w ? 0xfffffffeu : (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}

// The weight of a key, where it tells it; not finite for kProtected and NaN.
__device__ __forceinline__ float key_weight(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_addr(p)), "r"(rank));
  return remote;
}
// To the same shared-memory offset of cluster CTA `rank`.
__device__ __forceinline__ void st_cluster(const int* p, int rank, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ int take_cluster(const int* p, int rank, int add) {  // fetch and add
  int v;
  asm volatile("atom.shared::cluster.add.s32 %0, [%1], %2;"
               : "=r"(v)
               : "r"(cluster_addr(p, rank)), "r"(add)
               : "memory");
  return v;
}
__device__ __forceinline__ void add_cluster(const int* p, int rank, int v) {
  asm volatile("red.shared::cluster.add.s32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v)
               : "memory");
}

// Staged: the CTA's share of the row is kept in shared memory.
template <bool Staged>
__global__ void __launch_bounds__(1024, 2)
    evict_select_kernel(const EvictSelectParams p, const int clusters) {
  extern __shared__ __align__(16) uint32_t smem[];
  int* acc = reinterpret_cast<int*>(smem);  // [kBins] of the cluster, in rank 0 (none without)
  uint32_t* staged = smem + (clusters > 1 ? kBins : 0);
  __shared__ __align__(16) int hist[kCopies * kCopyStride];
  __shared__ int warp_sum[kScanThreads / 32];
  __shared__ int found[3];  // bin (or key), places left in it, its size
  __shared__ __align__(16) int list[kRanked];  // of the cluster, in rank 0
  __shared__ int list_n;
  __shared__ int warp_gt[32], warp_eq[32];
  __shared__ int cta_gt[kMaxCluster], cta_eq[kMaxCluster];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  const int rank = blockIdx.x % clusters, h = blockIdx.x / clusters, i = blockIdx.y;
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
  int left = keep;  // places for the keys that match the digits found so far

  // the warp's share of the row: `groups` times 4 steps of 32 keys, in index
  // order; key 32 j + lane of group g is component j of the lane's vector g
  const int per_group = clusters * (int)blockDim.x * 4;
  const int groups = (int)(((int64_t)L + per_group - 1) / per_group);
  const int64_t first = (int64_t)(rank * warps + warp) * groups * 128;
  const int base = (int)min((int64_t)L, first) + lane;
  const int end = (int)min((int64_t)L, first + (int64_t)groups * 128);
  // (no weight has key 0: it stands behind the share's end)
  auto key_of = [&](int k, float x) {
    return k >= end ? 0u : k < sink || k >= L - recent ? kProtected : weight_key(x);
  };
  auto count = [&](uint32_t bin) {
    atomicAdd(&hist[(lane % kCopies) * kCopyStride + bin], 1);
  };
  // (the protected keys are hundreds in one bin: added as a number, below)
  auto count_first = [&](uint32_t key) {
    if (key != kProtected && key != 0) count(key >> 21);
  };
  auto clear = [&] {
    for (int b = threadIdx.x; b < kCopies * kCopyStride / 4; b += blockDim.x)
      reinterpret_cast<int4*>(hist)[b] = make_int4(0, 0, 0, 0);
  };
  clear();
  if (threadIdx.x == 0) list_n = 0;
  for (int b = threadIdx.x; b < kRanked; b += blockDim.x) list[b] = 0;
  if (clusters > 1)
    for (int b = threadIdx.x; b < kBins; b += blockDim.x) acc[b] = 0;
  __syncthreads();
  uint4* mine = reinterpret_cast<uint4*>(staged) + warp * groups * 32 + lane;
  // groups whose keys are all there and compete: nothing to check key by key
  const int plain_lo = sink + lane, plain_hi = min(end, L - recent) - 128 + lane;
  auto load_keys = [&](int k) {
    const float* at_k = w + k;
    if (k >= plain_lo && k <= plain_hi)  // (the same for the whole warp)
      return make_uint4(weight_key(__ldg(at_k)), weight_key(__ldg(at_k + 32)),
                        weight_key(__ldg(at_k + 64)), weight_key(__ldg(at_k + 96)));
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = k + j * 32 < end ? __ldg(at_k + j * 32) : 0.f;
    return make_uint4(key_of(k, x[0]), key_of(k + 32, x[1]), key_of(k + 64, x[2]),
                      key_of(k + 96, x[3]));
  };
  // the keys, and the histogram of their first digit, in one pass
#pragma unroll 2
  for (int g = 0; g < groups; ++g) {
    const uint4 key = load_keys(base + g * 128);
    if (Staged) mine[g * 32] = key;
    count_first(key.x);
    count_first(key.y);
    count_first(key.z);
    count_first(key.w);
  }
  if (clusters > 1) cluster_sync();  // every CTA's acc is clear
  // f(key) of the lane's keys (each lane reads what it wrote)
  auto for_keys = [&](auto f) {
#pragma unroll 2
    for (int g = 0; g < groups; ++g) {
      const uint4 key = Staged ? mine[g * 32] : load_keys(base + g * 128);
      f(key.x);
      f(key.y);
      f(key.z);
      f(key.w);
    }
  };

  // the keep-th largest key: its digits from the top
  uint32_t prefix = 0, known = 0;  // the digits found, and their bits
  bool whole = false;              // whether every key that matches them is kept
  int gt = -1, eq = 0;  // the lane's keys above the prefix and matching it, once counted
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : (digit == 1 ? 10 : 0);
    const uint32_t mask = digit == 2 ? 1023u : 2047u;
    if (digit > 0) {
      clear();
      __syncthreads();
      for_keys([&](uint32_t key) {
        if ((key & known) == prefix) count((key >> shift) & mask);
      });
    }
    __syncthreads();
    // a thread has 4 bins, counted from the largest
    const int top = kBins - 1 - threadIdx.x * 4;
    int n[4] = {0, 0, 0, 0};
    if (threadIdx.x < kScanThreads) {
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        const int4 x = *reinterpret_cast<const int4*>(hist + c * kCopyStride + top - 3);
        n[0] += x.w;
        n[1] += x.z;
        n[2] += x.y;
        n[3] += x.x;
      }
      if (digit == 0 && threadIdx.x == 0 && rank == 0) n[0] += sink + recent;
    }
    if (clusters > 1) {
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (n[b] != 0) add_cluster(acc + top - b, 0, n[b]);
      cluster_sync();
      if (rank == 0 && threadIdx.x < kScanThreads) {
        int4* own = reinterpret_cast<int4*>(acc + top - 3);
        const int4 x = *own;
        n[0] = x.w;
        n[1] = x.z;
        n[2] = x.y;
        n[3] = x.x;
        *own = make_int4(0, 0, 0, 0);  // for the next digit
      }
    }
    if (rank == 0) {
      // the bin of the left-th key: a scan over the threads
      const int sum = n[0] + n[1] + n[2] + n[3];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31 && warp < kScanThreads / 32) warp_sum[warp] = incl;
      __syncthreads();
      const int before =
          incl - sum + __reduce_add_sync(kFull, lane < min(warp, kScanThreads / 32) ? warp_sum[lane] : 0);
      if (sum > 0 && before < left && before + sum >= left) {  // exactly one thread
        int places = left - before, b = 0, size = n[0];
#pragma unroll
        for (int c = 0; c < 3; ++c)
          if (b == c && places > n[c]) {
            places -= n[c];
            b = c + 1;
            size = n[c + 1];
          }
        for (int c = 0; c < clusters; ++c) {
          if (clusters > 1) {
            st_cluster(found + 0, c, top - b);
            st_cluster(found + 1, c, places);
            st_cluster(found + 2, c, size);
          } else {
            found[0] = top - b;
            found[1] = places;
            found[2] = size;
          }
        }
      }
    }
    if (clusters > 1)
      cluster_sync();
    else
      __syncthreads();
    prefix |= (uint32_t)found[0] << shift;
    known |= mask << shift;
    left = found[1];
    const int size = found[2];
    whole = size == left;  // every key with this prefix is kept
    if (whole || known == 0xffffffffu) break;
    if (size > kRanked) continue;  // (`found` is written again only behind the next barriers)
    // the bin's keys, in any order, to rank 0: the lane's one or none from a
    // register, several by another pass
    int matches = 0;
    uint32_t match = 0;
    gt = 0;
    for_keys([&](uint32_t key) {
      gt += (key & known) > prefix;
      if ((key & known) == prefix) {
        ++matches;
        match = key;
      }
    });
    int place = matches;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, place, o);
      if (lane >= o) place += x;
    }
    int start = 0;
    if (lane == 31 && place > 0)
      start = clusters > 1 ? take_cluster(&list_n, 0, place) : atomicAdd(&list_n, place);
    place += __shfl_sync(kFull, start, 31) - matches;
    auto put = [&](uint32_t key) {
      if (clusters > 1)
        st_cluster(list + place++, 0, (int)key);
      else
        list[place++] = (int)key;
    };
    if (matches == 1) put(match);
    if (matches > 1)
      for_keys([&](uint32_t key) {
        if ((key & known) == prefix) put(key);
      });
    if (clusters > 1)
      cluster_sync();
    else
      __syncthreads();
    if (rank == 0 && threadIdx.x < size) {
      const uint32_t own = (uint32_t)list[threadIdx.x];
      int above = 0, same = 0;  // (the list's last vector is padded with 0)
      auto meet = [&](int key) {
        above += (uint32_t)key > own;
        same += (uint32_t)key == own;
      };
#pragma unroll 4
      for (int j = 0; j < size; j += 4) {
        const int4 four = *reinterpret_cast<const int4*>(list + j);
        meet(four.x);
        meet(four.y);
        meet(four.z);
        meet(four.w);
      }
      if (above < left && left <= above + same)  // (equal keys write the same)
        for (int c = 0; c < clusters; ++c) {
          if (clusters > 1) {
            st_cluster(found + 0, c, (int)own);
            st_cluster(found + 1, c, left - above);
            st_cluster(found + 2, c, same);
          } else {
            found[0] = (int)own;
            found[1] = left - above;
            found[2] = same;
          }
        }
    }
    if (clusters > 1)
      cluster_sync();
    else
      __syncthreads();
    const uint32_t key_found = (uint32_t)found[0];
    if (matches == 1) {
      gt += match > key_found;
      eq = match == key_found;
    } else if (matches > 1) {
      for_keys([&](uint32_t key) {
        if ((key & known) != prefix) return;
        gt += key > key_found;
        eq += key == key_found;
      });
    }
    prefix = key_found;
    known = 0xffffffffu;
    left = found[1];
    whole = found[2] == left;
    break;
  }

  // kept: the keys above the prefix, and the first `left` of those that match it
  if (gt < 0) {
    gt = 0;
    for_keys([&](uint32_t key) {
      gt += (key & known) > prefix;
      eq += (key & known) == prefix;
    });
  }
  gt = __reduce_add_sync(kFull, gt);
  eq = __reduce_add_sync(kFull, eq);
  if (lane == 0) {
    warp_gt[warp] = gt;
    warp_eq[warp] = eq;
  }
  __syncthreads();
  // kept outright / matching, before this warp's share
  int ngt = __reduce_add_sync(kFull, lane < warp ? warp_gt[lane] : 0);
  int neq = __reduce_add_sync(kFull, lane < warp ? warp_eq[lane] : 0);
  if (clusters > 1) {
    if (warp == warps - 1 && lane < clusters) {
      st_cluster(cta_gt + rank, lane, ngt + gt);
      st_cluster(cta_eq + rank, lane, neq + eq);
    }
    cluster_sync();
    for (int c = 0; c < rank; ++c) {
      ngt += cta_gt[c];
      neq += cta_eq[c];
    }
  }
  int32_t* kept = p.kept + ((int64_t)i * p.num_kv_heads + h) * p.max_keep;
  float* out = p.out ? p.out + at : nullptr;
  const uint32_t below = (1u << lane) - 1;
  ngt += whole ? neq : min(neq, left);  // the keys kept before this warp's share
  for (int g = 0; g < groups; ++g) {
    const uint4 four = Staged ? mine[g * 32] : load_keys(base + g * 128);
    const uint32_t key[4] = {four.x, four.y, four.z, four.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // in step with the whole warp
      const uint32_t digits = key[j] & known;
      bool keep_it = digits >= prefix;
      if (!whole) {
        const uint32_t me = __ballot_sync(kFull, digits == prefix);
        if (digits == prefix && neq + __popc(me & below) >= left) keep_it = false;
        neq += __popc(me);
      }
      const uint32_t m = __ballot_sync(kFull, keep_it);
      if (keep_it) {
        const int o = ngt + __popc(m & below), k = base + g * 128 + j * 32;
        kept[o] = k;
        if (out) {
          // (a key does not tell a zero's sign, a NaN's bits, a protected weight)
          const float x = key_weight(key[j]);
          out[o] = isfinite(x) && x != 0.f ? x : __ldg(w + k);
        }
      }
      ngt += __popc(m);
    }
  }
}

// ---------------------------------------------------------------------------
// Move: row (j, h) of a request is head_dim bf16 values of K and of V; a
// group of head_vecs lanes moves both with 16-byte vectors. Consecutive
// groups take the KV heads of one destination token, so a CTA's destinations
// are contiguous; the sources are runs of head_dim * 2 bytes. Every byte moves
// once: HBM-bound, and a thread has its four rows' loads in flight together.
// Measured: 64 requests, 1024 tokens of 8 heads of 128 each: 88.5 us, 6.1 TB/s
// (90 % of the measured copy rate); with 2 or 8 rows a thread 94.7 and 106 us,
// with 256 or 512 threads 91.7 and 96.8 us.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 128;
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

template <bool Staged>
cudaError_t launch_select(const EvictSelectParams& p, int clusters, int threads, int staged,
                          cudaStream_t stream) {
  auto kernel = evict_select_kernel<Staged>;
  static SmemLimit limit;
  if (Staged) {
    cudaError_t e =
        limit.ensure(reinterpret_cast<const void*>(kernel), (kStaged + kBins) * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg =
      config(dim3((unsigned)(p.num_kv_heads * clusters), (unsigned)p.num_seqs), threads, stream,
             attr);
  cfg.dynamicSmemBytes = ((size_t)staged + (clusters > 1 ? kBins : 0)) * 4;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)clusters;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, clusters);
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads, L = p.max_seq_len;
  // as few CTAs as keep a share at 8192 keys (four CTAs an SM), twice as many
  // while the rows leave SMs without one and a share has over 2048 keys
  int clusters = 1;
  while (clusters < kMaxCluster && L > (int64_t)clusters * 8192) clusters *= 2;
  while (clusters < kMaxCluster && rows * clusters * 2 <= 152 && L > (int64_t)clusters * 2048)
    clusters *= 2;
  const int threads = L > (int64_t)clusters * 8192 ? 1024 : 512;
  const int64_t per_group = (int64_t)clusters * threads * 4;
  const int64_t share = (L + per_group - 1) / per_group * threads * 4;
  if (share <= kStaged) return launch_select<true>(p, clusters, threads, (int)share, stream);
  return launch_select<false>(p, clusters, threads, 0, stream);
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
