// key_weights_tc.cu -- accumulated attention weights of the cached keys for
// requests with many queries (prompts and chunks), on the 5th-generation
// tensor cores. The formula stands in key_weights.cu.
//
// S^T = K Q^T is computed with the keys as the rows of the accumulator: a
// TMEM lane is a key, and since the log-sum-exp of every query is known, a
// key's sum runs along its own lane: no reduction between threads, no
// rescaling, no second pass.
//
//   * work: (request, KV head, 256 keys), two 128-row tiles of K resident in
//     shared memory, against every tile of 128 / G queries x G heads that can
//     see them. Each Q tile is used by both K tiles: 128 x 128 x 128 products
//     read 16 KB of Q, half of what the SMs' L2 bandwidth would allow at the
//     tensor cores' full rate with one K tile;
//   * a cluster of 1, 2, 4 or 8 CTAs splits an item's Q tiles when a batch has
//     few items (one prompt: the first keys are seen by every query, the last
//     by few); the partial sums meet in the first CTA's shared memory and are
//     added in a fixed order;
//   * warp 8 issues the TMA copies (Q ring of 4 tiles), warp 9 the MMAs
//     (two accumulators of 128 columns per K tile: 512 TMEM columns), warp 10
//     loads the columns' -log2e * lse, warps 0-7 turn scores into weights: a
//     packed fma, ex2 and a packed add per pair of scores, no mask in
//     groups of 32 columns that every key of the warp sees;
//   * a tile's sum runs in eight chains and joins the total with a
//     compensated add, so a sum over 10^5 columns stays within a few 2^-24.
//
// Bound: one ex2 a score (32 a cycle and SM) and 2 D flops a score
// (8192 a cycle and SM dense): 512 cycles each for 128 x 128 at D = 128.
#include <math.h>

#include "key_weights.cuh"

namespace pkv {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kTM = 128;                 // keys per K tile (TMEM lanes)
constexpr int kKT = 2;                   // K tiles per item
constexpr int kTN = 128;                 // columns per Q tile
constexpr int kStages = 4;               // Q ring
constexpr int kEpiWarps = kKT * 4;       // warps 0 .. 7
constexpr int kTmaWarp = kEpiWarps, kMmaWarp = kTmaWarp + 1, kLseWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kLseWarp + 1);
constexpr int kMaxCluster = 8;
constexpr uint32_t kTmemCols = 512;
static_assert(kKT * 2 * kTN <= (int)kTmemCols, "two accumulators per K tile fit in TMEM");

struct Bars {
  uint64_t k_full;
  uint64_t q_full[kStages], q_empty[kStages];
  uint64_t l_full[kStages], l_empty[kStages];
  uint64_t s_full[kKT][2], s_free[kKT][2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int32_t abort;
  uint32_t masked[kStages];  // bit g: some column of the tile's group g of 32 adds nothing
};

template <int D>
struct Layout {
  static constexpr int NCH = D / 64;               // 128-byte column chunks of a row
  static constexpr int CH_BYTES = 128 * 128;       // one chunk of 128 rows
  static constexpr int TILE_BYTES = NCH * CH_BYTES;
  static constexpr int K_OFF = 0;
  static constexpr int Q_OFF = K_OFF + kKT * TILE_BYTES;
  static constexpr int LSE_OFF = Q_OFF + kStages * TILE_BYTES;     // [kStages][kTN] float
  static constexpr int RED_OFF = LSE_OFF + kStages * kTN * 4;      // [kMaxCluster][256] float
  static constexpr int BAR_OFF = RED_OFF + kMaxCluster * kKT * kTM * 4;
  static constexpr int NEED = 1024 + BAR_OFF + (int)sizeof(Bars);
  // one CTA per SM: each allocates all 512 TMEM columns
  static constexpr int BYTES = NEED > 120 * 1024 ? NEED : 120 * 1024;
};
static_assert(Layout<128>::BYTES <= 227 * 1024, "the stages fit a CTA");

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float to the same shared-memory offset of cluster CTA `rank`.
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t rank, float v) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(remote), "f"(v) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                          const __grid_constant__ CUtensorMap k_map, const KeyWeightsParams p,
                          const int clusters) {
  using Lay = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + Lay::BAR_OFF);

  griddep_wait();
  griddep_launch_dependents();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.z, h = blockIdx.y;
  const int key0 = (int)(blockIdx.x / clusters) * (kKT * kTM);
  const int rank = blockIdx.x % clusters;
  const int G = p.num_heads / p.num_kv_heads;
  // the CTAs of a cluster share (request, head, keys): these exits are uniform
  KeyRequest r;
  if (!key_request(p, i, threadIdx.x == 0 && blockIdx.x == 0 && h == 0, &r)) return;
  if (r.qlen <= p.short_max_q) {  // on the mma.sync grid
    if (p.no_short && threadIdx.x == 0 && blockIdx.x == 0 && h == 0)
      set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  if (key0 >= r.L) return;
  const int nk = min(kKT, (r.L - key0 + kTM - 1) / kTM);  // K tiles with keys
  const int QT = kTN / G;                                 // queries per Q tile
  const int qpos0 = r.L - r.qlen;
  const int j0 = max(0, key0 - qpos0);                    // the first query that sees key0
  const int all_tiles = (r.qlen - j0 + QT - 1) / QT;
  const int n = (all_tiles - rank + clusters - 1) / clusters;  // tiles rank, rank + clusters, ...

  if (warp == kTmaWarp && lane == 0) {
    mbar_init(smem_addr(&bars->k_full), 1);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&bars->q_full[s]), 1);
      mbar_init(smem_addr(&bars->q_empty[s]), 1);
      mbar_init(smem_addr(&bars->l_full[s]), 32);
      mbar_init(smem_addr(&bars->l_empty[s]), 4 * nk);
    }
    for (int x = 0; x < kKT; ++x)
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&bars->s_full[x][b]), 1);
        mbar_init(smem_addr(&bars->s_free[x][b]), 4);
      }
    mbar_init(smem_addr(&bars->mma_done), 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&bars->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (clusters > 1) cluster_arrive();  // waited for before the first remote store
  const uint32_t tmem = bars->tmem_base;
  volatile int32_t* abort = &bars->abort;
  const uint32_t k_s = smem_addr(smem + Lay::K_OFF), q_s = smem_addr(smem + Lay::Q_OFF);
  float* lse_s = reinterpret_cast<float*>(smem + Lay::LSE_OFF);
  const int32_t* table = p.block_table + (int64_t)i * p.max_blocks;
  float total = 0.f;  // an epilogue thread's key

  if (warp == kTmaWarp) {
    // ---- K boxes of 16 keys: lane b looks up box b's page; bad pages and
    // boxes past the context stay unloaded (their rows are never written out)
    const int key = key0 + lane * 16;
    const bool in = lane < kKT * kTM / 16 && key < r.L && n > 0;
    const int32_t id = in ? __ldg(table + key / p.block_size) : -1;
    const bool good = in && id >= 0 && id < p.num_blocks;
    const uint32_t load = __ballot_sync(kFull, good);
    const int32_t row = good ? id * p.block_size + key % p.block_size : 0;
    if (__any_sync(kFull, in && !good) && lane == 0 && rank == 0)
      set_status(p.status, PKV_DEV_BAD_BLOCK);
    if (lane == 0) {
      prefetch_tmap(&k_map);
      prefetch_tmap(&q_map);
      mbar_arrive_expect_tx(smem_addr(&bars->k_full), __popc(load) * Lay::NCH * 16 * 128);
    }
    __syncwarp();
    if (good)
      for (int c = 0; c < Lay::NCH; ++c)
        tma_load_4d(k_s + (lane >> 3) * Lay::TILE_BYTES + c * Lay::CH_BYTES +
                        (lane & 7) * 16 * 128,
                    &k_map, smem_addr(&bars->k_full), 0, row, h, c);
    if (lane == 0) {
      const uint32_t bytes = (uint32_t)(Lay::NCH * QT * G * 128);
      int t = 0;
      for (; t < n; ++t) {
        const int s = t % kStages;
        if (t >= kStages &&
            !mbar_wait(smem_addr(&bars->q_empty[s]), (t / kStages - 1) & 1, p.status, abort))
          break;
        mbar_arrive_expect_tx(smem_addr(&bars->q_full[s]), bytes);
        const int j = r.t0 + j0 + (rank + t * clusters) * QT;
        for (int c = 0; c < Lay::NCH; ++c)
          tma_load_3d(q_s + s * Lay::TILE_BYTES + c * Lay::CH_BYTES, &q_map,
                      smem_addr(&bars->q_full[s]), c * 64, h * G, j);
      }
      // copies in flight land before the CTA can exit
      for (int g = max(0, t - kStages); g < t; ++g)
        mbar_wait(smem_addr(&bars->q_full[g % kStages]), (g / kStages) & 1, nullptr);
      mbar_wait(smem_addr(&bars->k_full), 0, nullptr);
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0 && n > 0) {
      const int cols = min(kTN, min(QT, r.qlen - j0) * G);
      const uint32_t idesc = umma_idesc_bf16(kTM, (uint32_t)((cols + 15) & ~15), false, false);
      const uint64_t kd = smem_desc_sw128(k_s, 16, 1024), qd = smem_desc_sw128(q_s, 16, 1024);
      bool ok = mbar_wait(smem_addr(&bars->k_full), 0, p.status, abort);
      for (int t = 0; ok && t < n; ++t) {
        const int s = t % kStages, b = t & 1;
        ok = mbar_wait(smem_addr(&bars->q_full[s]), (t / kStages) & 1, p.status, abort);
        for (int x = 0; ok && x < nk; ++x) {
          if (t >= 2)
            ok = mbar_wait(smem_addr(&bars->s_free[x][b]), ((t >> 1) - 1) & 1, p.status, abort);
          if (!ok) break;
          tc_fence_after();
          const uint32_t acc = tmem + (uint32_t)((x * 2 + b) * kTN);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * Lay::CH_BYTES + (kk & 3) * 32) >> 4;
            umma_ss(acc, kd + (uint32_t)((x * Lay::TILE_BYTES) >> 4) + off,
                    qd + (uint32_t)((s * Lay::TILE_BYTES) >> 4) + off, idesc, kk > 0);
          }
          umma_commit(smem_addr(&bars->s_full[x][b]));
        }
        if (ok) umma_commit(smem_addr(&bars->q_empty[s]));
      }
      // every MMA issued has completed before TMEM is released
      umma_commit(smem_addr(&bars->mma_done));
      mbar_wait(smem_addr(&bars->mma_done), 0, nullptr);
    }
  } else if (warp == kLseWarp) {
    // ---- the columns' -log2e * lse; -inf marks a column that adds nothing.
    // Values of the next kStages tiles are in flight in registers.
    constexpr int E = kTN / 32;
    int dj[E];
    const float* src[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = e * 32 + lane;
      dj[e] = c < QT * G ? c / G : 1 << 30;
      src[e] = p.lse + (int64_t)r.t0 * p.num_heads + h * G + c % G;
    }
    auto fetch = [&](int t, float (&v)[E]) {
      const int j = j0 + (rank + t * clusters) * QT;
#pragma unroll
      for (int e = 0; e < E; ++e)
        v[e] = t < n && dj[e] < r.qlen - j
                   ? __ldg(src[e] + (int64_t)(j + dj[e]) * p.num_heads) : -INFINITY;
    };
    float v[kStages][E];
#pragma unroll
    for (int s = 0; s < kStages; ++s) fetch(s, v[s]);
    bool ok = true;
    for (int t0 = 0; ok && t0 < n; t0 += kStages) {
#pragma unroll
      for (int s = 0; s < kStages; ++s) {
        if (!ok || t0 + s >= n) break;
        if (t0 > 0) {
          ok = __all_sync(kFull, mbar_wait(smem_addr(&bars->l_empty[s]),
                                           (t0 / kStages - 1) & 1, p.status, abort));
          if (!ok) break;
        }
        uint32_t empty = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool none = v[s][e] == -INFINITY;
          empty |= __any_sync(kFull, none) ? 1u << e : 0u;
          lse_s[s * kTN + e * 32 + lane] = none ? -INFINITY : -kLog2e * v[s][e];
        }
        if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&bars->masked[s]) = empty;
        __syncwarp();
        mbar_arrive(smem_addr(&bars->l_full[s]));
        fetch(t0 + s + kStages, v[s]);
      }
    }
  } else if ((warp >> 2) < nk) {
    // ---- weights of tile x's keys: thread = TMEM lane = key
    const int x = warp >> 2;
    const int wkey = key0 + x * kTM + (warp & 3) * 32;  // the warp's first key
    const int key = wkey + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const float2 sc = make_float2(p.scale_log2, p.scale_log2);
    float comp = 0.f;  // of the compensated total
    bool ok = true;
    for (int t = 0; t < n; ++t) {
      const int s = t % kStages, b = t & 1;
      ok = __all_sync(kFull, mbar_wait(smem_addr(&bars->l_full[s]), (t / kStages) & 1, p.status,
                                       abort) &&
                                 mbar_wait(smem_addr(&bars->s_full[x][b]), (t >> 1) & 1, p.status,
                                           abort));
      if (!ok) break;
      tc_fence_after();
      const int jt = j0 + (rank + t * clusters) * QT;
      const int cols = min(QT, r.qlen - jt) * G;
      // the first column that sees the key, and the warp's first and last key
      // (32 bits: key - qpos0 - jt is below 256 and at least -qlen)
      const int first = (key - qpos0 - jt) * G;
      const int first_lo = (wkey - qpos0 - jt) * G;
      const int first_hi = (wkey + 31 - qpos0 - jt) * G;
      const uint32_t masked = *reinterpret_cast<volatile uint32_t*>(&bars->masked[s]);
      const uint32_t acc = tmem + lanes + (uint32_t)((x * 2 + b) * kTN);
      const float* nl = lse_s + s * kTN;
      float2 a0 = make_float2(0.f, 0.f), a1 = a0, a2 = a0, a3 = a0;
      uint32_t u[2][32];
      PKV_TMEM_LD32(acc, u[0]);
      tmem_wait_ld();
#pragma unroll
      for (int g = 0; g < kTN / 32; ++g) {
        const int c0 = g * 32;
        uint32_t(&cur)[32] = u[g & 1];
        if (g + 1 < kTN / 32) PKV_TMEM_LD32(acc + c0 + 32, u[(g + 1) & 1]);
        if (c0 < cols && first_lo < c0 + 32) {  // some column is there and sees some key
          if (c0 >= first_hi && !((masked >> g) & 1u)) {
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 l4 = *reinterpret_cast<const float4*>(nl + c0 + c);
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(cur[c]),
                                                      __uint_as_float(cur[c + 1])),
                                          sc, make_float2(l4.x, l4.y));
              const float2 z = __ffma2_rn(make_float2(__uint_as_float(cur[c + 2]),
                                                      __uint_as_float(cur[c + 3])),
                                          sc, make_float2(l4.z, l4.w));
              const float2 ey = make_float2(fast_exp2(y.x), fast_exp2(y.y));
              const float2 ez = make_float2(fast_exp2(z.x), fast_exp2(z.y));
              if (c & 4) {
                a2 = __fadd2_rn(a2, ey);
                a3 = __fadd2_rn(a3, ez);
              } else {
                a0 = __fadd2_rn(a0, ey);
                a1 = __fadd2_rn(a1, ez);
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float l = nl[c0 + c];
              const float w = fast_exp2(fmaf(__uint_as_float(cur[c]), p.scale_log2, l));
              // selected, not multiplied: the score of an empty or hidden
              // column may be anything
              const float add = (l == -INFINITY || c0 + c < first) ? 0.f : w;
              if (c & 1)
                a1.x += add;
              else
                a0.x += add;
            }
          }
        }
        tmem_wait_ld();
        if (g == kTN / 32 - 2) {  // the tile is in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&bars->s_free[x][b]));
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars->l_empty[s]));
      const float2 a = __fadd2_rn(__fadd2_rn(a0, a1), __fadd2_rn(a2, a3));
      const float y = (a.x + a.y) - comp;
      const float sum = total + y;
      // infinite or NaN sums stay what they are
      comp = isfinite(sum) ? (sum - total) - y : 0.f;
      total = sum;
    }
  }

  // ---- the cluster's partial sums, added in rank order
  float* red = reinterpret_cast<float*>(smem + Lay::RED_OFF);  // [clusters][256]
  if (clusters > 1) {
    __syncwarp();
    cluster_wait();  // every CTA of the cluster has started
    if (rank != 0 && threadIdx.x < kKT * kTM)
      st_cluster(smem_addr(red + rank * (kKT * kTM) + threadIdx.x), 0, total);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  if (rank == 0 && threadIdx.x < kKT * kTM) {
    const int key = key0 + (int)threadIdx.x;
    if (key < r.L) {
      const int32_t id = __ldg(table + key / p.block_size);
      if (id >= 0 && id < p.num_blocks) {
        for (int c = 1; c < clusters; ++c) total += red[c * (kKT * kTM) + threadIdx.x];
        const int64_t at = ((int64_t)r.row * p.num_kv_heads + h) * p.row_len + key;
        p.out[at] = key < r.prior && p.decay != 0.f ? fmaf(p.decay, p.in[at], total) : total;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(const KeyWeightsParams& p, const CUtensorMap& q_map, const CUtensorMap& k_map,
                   cudaStream_t stream) {
  auto kernel = key_weights_tc_kernel<D>;
  static SmemLimit limit;
  cudaError_t e = limit.ensure(reinterpret_cast<const void*>(kernel), Layout<D>::BYTES);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int G = p.num_heads / p.num_kv_heads;
  const int64_t key_tiles = ((int64_t)p.max_seq_len + kKT * kTM - 1) / (kKT * kTM);
  const int64_t items = key_tiles * p.num_kv_heads * p.num_seqs;
  const int q_tiles = (p.max_query_len + kTN / G - 1) / (kTN / G);
  // Split an item's Q tiles while there are fewer than 8 CTAs an SM to even
  // the load out and a CTA keeps at least 8 tiles for its K tiles.
  int clusters = 1;
  while (clusters < kMaxCluster && items * clusters < 8 * sms && q_tiles / clusters >= 16)
    clusters *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(key_tiles * clusters), (unsigned)p.num_kv_heads,
                     (unsigned)p.num_seqs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<D>::BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)clusters;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, q_map, k_map, p, clusters);
}

}  // namespace

cudaError_t launch_key_weights_tc(const KeyWeightsParams& p, const CUtensorMap& q_map,
                                  const CUtensorMap& k_map, cudaStream_t stream) {
  return p.head_dim == 64 ? launch<64>(p, q_map, k_map, stream)
                          : launch<128>(p, q_map, k_map, stream);
}

}  // namespace pkv
