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
// largest value, then one pass that writes the keys above it and the first of
// those equal to it, in index order. The search counts the keys in 2048 bins,
// finds the n-th one's bin, counts that bin's keys by their next 11 bits, and so
// on; it ends when a bin is taken whole, or is so small that its keys can be
// ranked against one another. The first bins are 1/32 of an octave each, so the
// latter is the usual case after one pass of 100K keys.
//
// A row (request, KV head) is read once into the shared memory of one CTA, or,
// when the rows are few, of a cluster, as long as each of its CTAs has an SM
// (launch_evict_select). The CTAs add up one another's bins by groups of 32,
// then the 32 of one group, so that each finds the same bin for itself with one
// barrier a pass. Rows of more than kStaged keys a CTA are read again in each
// pass (from L2). The row's 4 bytes a key are little: the instructions bound it
// (70 % of the issue slots of the SMs at work; the SMs that get a fourth row
// end last), or barriers and latency when the rows are few. Measured: 64 x 8
// rows of 1500 to 8192 keys, 1024 kept: 14.1 us; 2 x 8 rows of 128K, 8192 kept:
// 18.3 us.
// ---------------------------------------------------------------------------
constexpr int kBins = 2048;
constexpr int kGroups = kBins / 32;  // sums of 32 bins, one bin a lane
constexpr int kMaxCluster = 8;
constexpr int kStaged = 40960;     // keys of a CTA's share that shared memory holds
constexpr int kRanked = 384;       // keys at most that are ranked against one another

// Order-preserving key of a weight: larger weights have larger keys, -0 and
// +0 the same one, a NaN the largest but kProtected, which stands for the keys
// that are kept whatever their weight (and so need no care of their own: the
// selection is the `keep` largest keys of the row).
constexpr uint32_t kProtected = 0xffffffffu;
__device__ __forceinline__ uint32_t weight_key(float w) {
  const int32_t b = __float_as_int(w + 0.f);
  return w != w ? 0xfffffffeu : (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}

// The bins of the first pass: 32 an octave from 2^-40 to 2^24, where a weight
// that decides anything lies; the first and the last bin take what is below and
// above. (It is monotonic, so any row may be counted so; a row whose keep-th
// key lies in one of the two end bins is counted again by the key's bits.)
constexpr int kFineShift = 23 - 5;
constexpr int kFineLow = (int)(0x80000000u >> kFineShift) + (127 - 40) * 32;
__device__ __forceinline__ uint32_t fine_bin(uint32_t key) {
  return (uint32_t)min(max((int)(key >> kFineShift) - kFineLow, 0), kBins - 1);
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
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(remote)
               : "r"(smem_addr(p)), "r"(rank));
  return remote;
}
// To the same shared-memory offset of cluster CTA `rank`.
__device__ __forceinline__ void st_cluster(const int* p, int rank, int v) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ int ld_cluster(const int* p, int rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];"
               : "=r"(v)
               : "r"(cluster_addr(p, rank))
               : "memory");
  return v;
}
// The sum of *p over the cluster's CTAs.
__device__ __forceinline__ int sum_cluster(const int* p, int clusters) {
  if (clusters == 1) return *p;
  int x[kMaxCluster], sum = 0;
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) x[c] = c < clusters ? ld_cluster(p, c) : 0;
#pragma unroll
  for (int c = 0; c < kMaxCluster; ++c) sum += x[c];
  return sum;
}
__device__ __forceinline__ int inclusive_sum(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Staged: the CTA's share of the row is kept in shared memory.
template <bool Staged>
__global__ void __launch_bounds__(1024, 2)
    evict_select_kernel(const EvictSelectParams p, const int clusters) {
  extern __shared__ __align__(16) uint32_t staged[];
  // (two of each in turn: the other CTAs read them, and one is written again
  // only behind the barrier that follows every read of it)
  __shared__ __align__(16) int hist[2][kBins];
  __shared__ int group_sum[2][kGroups];  // of 32 bins, from the largest
  __shared__ int found[3];  // bin (or key), places left in it, its size
  __shared__ __align__(16) int list[kRanked];  // the CTA's keys, then
  __shared__ __align__(16) int all[kRanked];   // the cluster's
  __shared__ int list_n;
  __shared__ int warp_gt[32], warp_eq[32];
  __shared__ int cta_gt[kMaxCluster], cta_eq[kMaxCluster];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  griddep_wait();
  griddep_launch_dependents();
  uint32_t h, rank;  // a cluster, or a CTA on its own, has a row
  asm("mov.u32 %0, %%clusterid.x;" : "=r"(h));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int i = blockIdx.y;
  const int L = __ldg(p.seq_lens + i), keep = __ldg(p.keep_lens + i);
  const int row = p.rows ? __ldg(p.rows + i) : i;
  // the CTAs of a cluster share the row: these exits are uniform
  if (L < 0 || L > p.max_seq_len || keep < 0 || keep > L || keep > p.max_keep) {
    if (threadIdx.x == 0 && rank == 0 && h == 0) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  if (row < 0 || row >= p.num_rows) {
    if (threadIdx.x == 0 && rank == 0 && h == 0) set_status(p.status, PKV_DEV_BAD_ROW);
    return;
  }
  if (keep == 0) return;
  const int64_t at = ((int64_t)row * p.num_kv_heads + h) * p.row_len;
  const float* w = p.weights + at;
  const int recent = min(p.num_recent, keep);
  const int sink = min(p.num_sink, keep - recent);
  int left = keep;  // places for the keys that match the digits found so far

  // the warp's share of the row: `groups` times 128 keys; a lane's vector of a
  // group is its keys 4 lane to 4 lane + 3
  const int per_group = clusters * (int)blockDim.x * 4;
  const int groups = (int)(((uint32_t)L + (uint32_t)per_group - 1) / (uint32_t)per_group);
  // (at most L + per_group: below 2^32)
  const uint32_t first = (rank * warps + warp) * (uint32_t)groups * 128;
  const int base = (int)min((uint32_t)L, first);
  const int end = (int)min((uint32_t)L, first + (uint32_t)groups * 128);
  // (no weight has key 0: it stands behind the share's end)
  auto key_of = [&](int k, float x) {
    return k >= end ? 0u : k < sink || k >= L - recent ? kProtected : weight_key(x);
  };
  auto clear = [&](int b, int last) {
#pragma unroll 1
    for (int v = threadIdx.x; v < kBins / 4; v += blockDim.x)
      reinterpret_cast<int4*>(hist[b])[v] = make_int4(0, 0, 0, v == kBins / 4 - 1 ? last : 0);
  };
  // (the protected keys would be hundreds in one bin: added as a number)
  clear(0, rank == 0 ? sink + recent : 0);
  if (threadIdx.x == 0) list_n = 0;
#pragma unroll 1
  for (int b = threadIdx.x; b < kRanked; b += blockDim.x) list[b] = 0;
  __syncthreads();
  uint4* mine = reinterpret_cast<uint4*>(staged) + warp * groups * 32 + lane;
  // the weights of the lane's vectors of groups g and g + 1 (a row may be read
  // to the end of its storage), and their keys
  const bool vectors = ((p.row_len & 3) | (reinterpret_cast<uintptr_t>(p.weights) & 15)) == 0;
  auto load_two = [&](int g, float4* x) {
    const int k = base + g * 128 + lane * 4;
    if (vectors) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k + u * 128 < end) x[u] = __ldg(reinterpret_cast<const float4*>(w + k + u * 128));
      }
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at_k = k + u * 128;
        x[u].x = at_k < end ? __ldg(w + at_k) : 0.f;
        x[u].y = at_k + 1 < end ? __ldg(w + at_k + 1) : 0.f;
        x[u].z = at_k + 2 < end ? __ldg(w + at_k + 2) : 0.f;
        x[u].w = at_k + 3 < end ? __ldg(w + at_k + 3) : 0.f;
      }
    }
  };
  // groups whose keys are all there and compete: nothing to check key by key
  const int plain_hi = min(end, L - recent) - 128;
  auto plain = [&](int g) { return base + g * 128 >= sink && base + g * 128 <= plain_hi; };
  auto keys_of = [&](int g, const float4& x) {
    const int k = base + g * 128 + lane * 4;
    if (plain(g))
      return make_uint4(weight_key(x.x), weight_key(x.y), weight_key(x.z), weight_key(x.w));
    return make_uint4(key_of(k, x.x), key_of(k + 1, x.y), key_of(k + 2, x.z), key_of(k + 3, x.w));
  };
  auto count_first = [&](uint32_t key) { atomicAdd(&hist[0][fine_bin(key)], 1); };
  auto count_if = [&](uint32_t key) {
    if (key != kProtected && key != 0) count_first(key);
  };
  // the keys, and the histogram of their first digit, in one pass
  for (int g = 0; g < groups; g += 2) {
    float4 x[2];
    load_two(g, x);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (g + u == groups) break;
      const uint4 key = keys_of(g + u, x[u]);
      if (Staged) mine[(g + u) * 32] = key;
      if (plain(g + u)) {
        count_first(key.x);
        count_first(key.y);
        count_first(key.z);
        count_first(key.w);
      } else {
        count_if(key.x);
        count_if(key.y);
        count_if(key.z);
        count_if(key.w);
      }
    }
  }
  // f(key) of the lane's keys (each lane reads what it wrote)
  auto for_keys = [&](auto f) {
#pragma unroll 2
    for (int g = 0; g < groups; ++g) {
      uint4 key;
      if (Staged) {
        key = mine[g * 32];
      } else {
        float4 x[2];
        load_two(g, x);
        key = keys_of(g, x[0]);
      }
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
  int shift = kFineShift;
  uint32_t mask = kBins - 1;
  for (int pass = 0;; ++pass) {
    const int* bins = hist[pass & 1];
    if (pass > 0) {
      clear(pass & 1, 0);
      __syncthreads();
      for_keys([&](uint32_t key) {
        if ((key & known) == prefix) atomicAdd(&hist[pass & 1][(key >> shift) & mask], 1);
      });
    }
    __syncthreads();
#pragma unroll 1
    for (int v = threadIdx.x; v < kBins / 4; v += blockDim.x) {
      const int4 x = reinterpret_cast<const int4*>(bins)[kBins / 4 - 1 - v];
      int sum = x.x + x.y + x.z + x.w;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if ((lane & 7) == 0) group_sum[pass & 1][v / 8] = sum;
    }
    if (clusters > 1)
      cluster_sync();
    else
      __syncthreads();
    if (warp == 0) {
      // the group of bins of the left-th key, then its bin
      const int* sums = group_sum[pass & 1] + 2 * lane;
      const int n0 = sum_cluster(sums, clusters), n1 = sum_cluster(sums + 1, clusters);
      const int upto = inclusive_sum(n0 + n1, lane), upto0 = upto - n1;
      const uint32_t at = __ballot_sync(kFull, upto >= left);  // the first of these
      const int owner = at ? __ffs(at) - 1 : 31;
      const bool second = upto0 < left;
      const int group = __shfl_sync(kFull, 2 * lane + second, owner);
      const int before = __shfl_sync(kFull, second ? upto0 : upto0 - n0, owner);
      const int bin = kBins - 1 - (group * 32 + lane);
      const int n = sum_cluster(bins + bin, clusters);
      const int incl = before + inclusive_sum(n, lane);
      if (incl - n < left && incl >= left) {  // exactly one lane
        found[0] = bin;
        found[1] = left - (incl - n);
        found[2] = n;
      }
    }
    __syncthreads();
    // (`found` is written again only behind the next barriers)
    if (pass > 0) {
      prefix |= (uint32_t)found[0] << shift;
      known |= mask << shift;
    } else if (found[0] > 0 && found[0] < kBins - 1) {
      prefix = (uint32_t)(found[0] + kFineLow) << shift;
      known = ~0u << shift;
    } else {
      shift = 32 - 11;
      continue;
    }
    left = found[1];
    const int size = found[2];
    whole = size == left;  // every key with this prefix is kept
    if (whole || known == 0xffffffffu) break;
    if (size > kRanked) {
      const int next = max(shift - 11, 0);
      mask = (1u << (shift - next)) - 1;
      shift = next;
      continue;
    }
    // the bin's keys, in any order, to a list: the lane's one or none from a
    // register, several by another pass
    int matches = 0;
    uint32_t match = 0;
    gt = 0;
    for_keys([&](uint32_t key) {
      gt += key > (prefix | ~known);
      if (key - prefix <= ~known) {
        ++matches;
        match = key;
      }
    });
    int place = inclusive_sum(matches, lane);
    int start = 0;
    if (lane == 31 && place > 0) start = atomicAdd(&list_n, place);
    place += __shfl_sync(kFull, start, 31) - matches;
    auto put = [&](uint32_t key) {
      if (place < kRanked) list[place++] = (int)key;  // (always, unless the weights change)
    };
    if (matches == 1) put(match);
    if (matches > 1)
      for_keys([&](uint32_t key) {
        if ((key & known) == prefix) put(key);
      });
    const int* ranked = list;
    if (clusters > 1) {
      // every CTA collects the lists of all of them
      ranked = all;
      cluster_sync();
#pragma unroll 1
      for (int t = threadIdx.x; t < kRanked; t += blockDim.x) {
        int j = t, from = -1, key = 0;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          const int n = c < clusters ? min(max(ld_cluster(&list_n, c), 0), kRanked) : 0;
          if (from < 0 && j < n)
            from = c;
          else if (from < 0)
            j -= n;
        }
        if (from >= 0) key = ld_cluster(list + j, from);
        all[t] = key;
      }
    }
    __syncthreads();
#pragma unroll 1
    for (int t = threadIdx.x; t < size; t += blockDim.x) {
      const uint32_t own = (uint32_t)ranked[t];
      int above = 0, same = 0;  // (the list's last vector is padded with 0)
      auto meet = [&](int key) {
        above += (uint32_t)key > own;
        same += (uint32_t)key == own;
      };
#pragma unroll 4
      for (int j = 0; j < size; j += 4) {
        const int4 four = *reinterpret_cast<const int4*>(ranked + j);
        meet(four.x);
        meet(four.y);
        meet(four.z);
        meet(four.w);
      }
      if (above < left && left <= above + same) {  // (equal keys write the same)
        found[0] = (int)own;
        found[1] = left - above;
        found[2] = same;
      }
    }
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
      gt += key > (prefix | ~known);
      eq += key - prefix <= ~known;
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
    for (int c = 0; c < (int)rank; ++c) {
      ngt += cta_gt[c];
      neq += cta_eq[c];
    }
  }
  int32_t* kept = p.kept + ((int64_t)i * p.num_kv_heads + h) * p.max_keep;
  float* out = p.out ? p.out + at : nullptr;
  const uint32_t below = (1u << lane) - 1;
  ngt += whole ? neq : min(neq, left);  // the keys kept before this warp's share
  // A group's kept keys go through shared memory, so that the lanes write them
  // side by side: their indices where the group was staged, their keys where
  // the histograms were (no CTA reads those any more).
  int* heavy = &hist[0][0] + warp * 128;
  for (int g = 0; g < groups; ++g) {  // in step with the whole warp
    uint4 four;
    if (Staged) {
      four = mine[g * 32];
    } else {
      float4 x[2];
      load_two(g, x);
      four = keys_of(g, x[0]);
    }
    int* at_k = reinterpret_cast<int*>(staged) + (Staged ? warp * groups + g : warp) * 128;
    const uint32_t key[4] = {four.x, four.y, four.z, four.w};
    bool keep_it[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) keep_it[j] = key[j] >= prefix;
    if (!whole) {
      int n = neq;  // matching keys before the lane's
#pragma unroll
      for (int j = 0; j < 4; ++j)
        n += __popc(__ballot_sync(kFull, key[j] - prefix <= ~known) & below);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (key[j] - prefix <= ~known && n++ >= left) keep_it[j] = false;
      neq = __shfl_sync(kFull, n, 31);
    }
    int o = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) o += __popc(__ballot_sync(kFull, keep_it[j]) & below);
    __syncwarp();  // the keys of this group, and the buffers of the last one, have been read
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (keep_it[j]) {
        at_k[o] = base + g * 128 + lane * 4 + j;
        heavy[o] = (int)key[j];
        ++o;
      }
    const int n = __shfl_sync(kFull, o, 31);
    __syncwarp();
    for (int t = lane; t < n; t += 32) {
      const int k = at_k[t];
      if (ngt + t >= keep) break;  // (never, unless the weights change while they are read)
      kept[ngt + t] = k;
      if (out) {
        // (a key does not tell a zero's sign, a NaN's bits, a protected weight)
        const float x = key_weight((uint32_t)heavy[t]);
        out[ngt + t] = isfinite(x) && x != 0.f ? x : __ldg(w + k);
      }
    }
    ngt += n;
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

// How many clusters of 1 to kMaxCluster CTAs the device holds at one CTA an SM
// (the SMs of a cluster lie in one of its GPCs, which differ in size).
class ClusterRoom {
 public:
  cudaError_t get(const int** fit) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!done_[dev].load(std::memory_order_acquire)) {
      std::lock_guard<std::mutex> lock(mu_);
      if (!done_[dev].load(std::memory_order_relaxed)) {
        e = fill(fit_[dev]);
        if (e != cudaSuccess) return e;
        done_[dev].store(true, std::memory_order_release);
      }
    }
    *fit = fit_[dev];
    return cudaSuccess;
  }

 private:
  static cudaError_t fill(int* fit);
  static constexpr int kMaxDevices = 64;
  std::mutex mu_;
  std::atomic<bool> done_[kMaxDevices] = {};
  int fit_[kMaxDevices][kMaxCluster + 1] = {};
};
ClusterRoom cluster_room;

template <bool Staged>
cudaError_t launch_select(const EvictSelectParams& p, int clusters, int threads, int staged,
                          cudaStream_t stream) {
  auto kernel = evict_select_kernel<Staged>;
  static SmemLimit limit;
  const cudaError_t e = limit.ensure(reinterpret_cast<const void*>(kernel), kStaged * 4);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg =
      config(dim3((unsigned)(p.num_kv_heads * clusters), (unsigned)p.num_seqs), threads, stream,
             attr);
  cfg.dynamicSmemBytes = (size_t)staged * 4;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)clusters;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p, clusters);
}

cudaError_t ClusterRoom::fill(int* fit) {
  auto kernel = evict_select_kernel<true>;
  cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kStaged * 4);
  for (int c = 1; e == cudaSuccess && c <= kMaxCluster; ++c) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = config(dim3((unsigned)c), 1024, nullptr, attr);
    cfg.dynamicSmemBytes = kStaged * 4;  // over half of an SM's
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    e = cudaOccupancyMaxActiveClusters(&fit[c], kernel, &cfg);
  }
  return e;
}

}  // namespace

cudaError_t launch_evict_select(const EvictSelectParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.num_seqs * p.num_kv_heads, L = p.max_seq_len;
  const int* fit = nullptr;
  cudaError_t e = cluster_room.get(&fit);
  if (e != cudaSuccess) return e;
  // Clusters for rows of over 8192 keys that would leave SMs without work: the
  // most CTAs a row, of 2048 keys at least, for which every CTA has an SM of its
  // own (128K keys: 16 rows in clusters of 6: 18 us, of 8, of which 15 fit:
  // 23 us, of 4: 24 us; 128 rows of 24K: one CTA each 12 us, clusters 17 us).
  int clusters = 1;
  if (L > 8192)
    for (int c = 2; c <= kMaxCluster; ++c)
      if (rows <= fit[c] && L >= 2048 * c) clusters = c;
  const bool alone = rows * clusters <= fit[1];
  // And for somewhat more rows than SMs, too long for one CTA to stage: some SMs
  // would have two of them and end last (192 rows of 25K to 100K keys in
  // clusters of 5: 51.7 us, a CTA each 74.8; 160 rows of 50K to 60K, of 3: 34.7
  // and 51.6; but 256 rows of 128K, of 7: 151 and 139).
  if (!alone && L > kStaged && rows * 2 < (int64_t)fit[1] * 3) {
    const int64_t c = (L + kStaged / 2 - 1) / (kStaged / 2);
    clusters = c < kMaxCluster ? (int)c : kMaxCluster;
  }
  // Threads: 1024 where a CTA has its SM alone (128 rows of 4096 keys: 6.1 us,
  // with 512 7.3 us) or a long row (512 rows of 24K: 40 against 45 us), else 512
  // (512 rows of 4096: 12 us, with 1024 15.8, with 256 14.4 us), fewer for
  // short rows (1600 rows of 150 to 600 keys: 10.2 us, with 512 15.9).
  const int64_t share_of = L / clusters;
  int threads = 512;
  if (clusters > 1)
    threads = alone && share_of > 8192 ? 1024 : 512;
  else if (share_of > (alone ? 2048 : 16384))
    threads = 1024;
  else if (!alone && share_of <= 2048)
    threads = 256;
  const int64_t per_group = (int64_t)clusters * threads * 4;
  const int64_t share = (L + per_group - 1) / per_group * threads * 4;
  if (share <= kStaged) return launch_select<true>(p, clusters, threads, (int)share, stream);
  return launch_select<false>(p, clusters, threads, threads * 4, stream);
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
