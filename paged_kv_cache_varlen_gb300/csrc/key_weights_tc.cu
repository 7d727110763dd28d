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
//   * a cluster of 1, 2 or 4 CTAs splits an item's Q tiles when a batch has
//     few items (one prompt: the first keys are seen by every query, the last
//     by few); the partial sums meet in the first CTA's shared memory and are
//     added in a fixed order;
//   * warp 16 issues the TMA copies (Q ring of 4 tiles), warp 17 loads the
//     columns' -log2e * lse, warps 18 and 19 issue the MMAs of a K tile each
//     (three accumulators of 64 columns, beside K in the 512 TMEM columns),
//     warps 0-15 turn scores into weights
//     (a warpgroup per K tile and half of the columns): a packed fma, ex2 and
//     a packed add per pair of scores, no mask where every column sees
//     every key of the warp;
//   * a key's sum over 16 tiles runs in eight chains for each half of the
//     columns (four threads, two each), the groups of 16 tiles are added up
//     apart: chains of 128 additions and one for each group, so the additions
//     leave a sum over 10^5 columns within about 2^-16.5 (177 roundings of
//     2^-24). Each addend is off by ex2's 2^-22 and by its exponent's roundings,
//     3 2^-24 (|scale s| + |lse|). Seen against 64 bits: 3.2e-7 of the sums (an
//     8192-token prompt, lse and scores of a few units).
//
// Bound: one ex2 a score (32 a cycle and SM) and 2 D flops a score
// (8192 a cycle and SM dense): 512 cycles each for 128 x 128 at D = 128, so
// 1024 a Q tile against 256 keys; the epilogue's warps alone take 1240 with
// their other instructions, and about 1600 beside the issuing and copying
// warps that wait. Measured: one 8192-token prompt, 32 query and 8 KV heads of
// 128, three sets of inputs in turn: 223 us, 1.25 PFLOP/s (65 % of the measured
// bf16 rate; 204 us in a burst of 30 calls); 512 queries over 32K keys 128 us;
// 64 single tokens of 64 or 128 heads on one KV head of 64 (128) dimensions: 26
// (33) us. (One warp issuing for both K tiles took a quarter longer.)
#include <math.h>
#include <stddef.h>

#include "key_weights.cuh"

#ifdef PKV_TEST_HOLD_ARRIVAL
// Test builds only: while set, epilogue warp 0 of CTA 0 withholds its release
// of its first accumulator, so that an issuing warp's bounded wait runs out.
__device__ int g_pkv_test_hold_key_weights;
extern "C" int pkv_test_hold_key_weights(int on) {
  return (int)cudaMemcpyToSymbol(g_pkv_test_hold_key_weights, &on, sizeof(int));
}
#endif

namespace pkv {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kTM = 128;                 // keys per K tile (TMEM lanes)
constexpr int kKT = 2;                   // K tiles per item
constexpr int kTN = 128;                 // columns per Q tile
constexpr int kHalf = kTN / 2;           // columns of one epilogue warpgroup
constexpr int kStages = 4;               // Q ring
constexpr int kEpiWarps = kKT * 2 * 4;   // warps 0 .. 15: (column half, K tile, lane quarter)
constexpr int kTmaWarp = kEpiWarps, kLseWarp = kTmaWarp + 1;
constexpr int kMmaWarp = kLseWarp + 1;   // one for each K tile
constexpr int kThreads = 32 * (kMmaWarp + kKT);
constexpr int kMaxCluster = 4;
constexpr uint32_t kTmemCols = 512;
constexpr int kAcc = 3;                  // accumulators of kHalf columns per K tile, in turn
constexpr uint32_t kKCol = kKT * kAcc * kHalf;  // then the K tiles: bf16 pairs, D / 2 columns each
static_assert(kKCol + kKT * 64 <= kTmemCols, "accumulators and K tiles fit in TMEM");

struct Bars {  // kNumBars barriers, the rest, and s_full
  uint64_t k_land, k_read;     // K in shared memory; read by the epilogue warps
  uint64_t k_full[kKT];        // K in tensor memory
  uint64_t q_full[kStages], q_empty[kStages];
  uint64_t l_full[kStages], l_empty[kStages];
  uint64_t s_free[kKT][kAcc];
  uint64_t mma_done;
  uint32_t tmem_base;
  int32_t abort;
  uint32_t masked[kStages];  // bit g: some column of the tile's group g of 32 adds nothing
  // Two an accumulator: its uses alternate between the column halves, so each
  // half has one of its own and meets every phase of it. (With one, a half would
  // wait for every other phase, all of one parity, and be right only because the
  // product before has arrived by then.) A prompt of 8192 tokens takes 222 us
  // with them here, 225 among the other barriers.
  uint64_t s_full[kKT][2 * kAcc];
};

constexpr uint32_t kNumBars = offsetof(Bars, tmem_base) / 8;
constexpr int kListed = 256;  // requests at most whose items a CTA lists

template <int D>
struct Layout {
  static constexpr int NCH = D / 64;               // 128-byte column chunks of a row
  static constexpr int CH_BYTES = 128 * 128;       // one chunk of 128 rows
  static constexpr int TILE_BYTES = NCH * CH_BYTES;
  static constexpr int Q_OFF = 0;
  static constexpr int LSE_OFF = Q_OFF + kStages * TILE_BYTES;     // [kStages][kTN] float
  static constexpr int RED_OFF = LSE_OFF + kStages * kTN * 4;      // [kMaxCluster][2][256] float
  static constexpr int BAR_OFF = RED_OFF + kMaxCluster * 2 * kKT * kTM * 4;
  static constexpr int LIST_OFF = BAR_OFF + ((int)sizeof(Bars) + 15) / 16 * 16;  // [kListed + 1]
  static constexpr int NEED = 1024 + LIST_OFF + (kListed + 1) * 4;
  // one CTA per SM: each allocates all 512 TMEM columns
  static constexpr int BYTES = NEED > 120 * 1024 ? NEED : 120 * 1024;
};
static_assert(Layout<128>::BYTES <= 227 * 1024, "the stages fit a CTA");

__device__ __forceinline__ void mbar_inval(uint32_t bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
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

// tcgen05.ld of 16 lanes x 32 columns: register 4 c + e of a thread is row
// lane / 4 + 8 (e / 2), column 8 c + 2 (lane % 4) + e % 2.
#define PKV_TMEM_LD_16X256B_X4(taddr, r)                                                         \
  asm volatile(                                                                                  \
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"   \
      "%14,%15}, [%16];"                                                                         \
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),     \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), \
        "=r"(r[14]), "=r"(r[15])                                                                \
      : "r"(taddr))

// Every lane waits for its own barrier (all lanes together: no divergence
// while the barriers are complete, the usual case). False when a wait gave up.
__device__ __noinline__ bool slow_wait(uint32_t bar, uint32_t parity, int32_t* status,
                                       volatile int32_t* abort) {
  const uint64_t t0 = globaltimer();
  while (true) {
    // polls in as few instructions as there are: they share the schedulers
    // with the warps that compute
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .u32 i;\n\tmov.u32 i, 256;\n\t"
        "POLL:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 i, i, 1;\n\tsetp.ne.u32 p, i, 0;\n\t@p bra POLL;\n\t"
        "setp.ne.u32 p, i, 0;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if (abort && *abort) return false;
    if (globaltimer() - t0 > PKV_WAIT_TIMEOUT_NS) {
      set_status(status, PKV_DEV_TIMEOUT);
      if (abort) *abort = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t phase, int32_t* status,
                                          volatile int32_t* abort) {
  bool ok = mbar_try_wait(bar, phase & 1);
  if (__all_sync(kFull, ok)) return true;
  if (!ok) ok = slow_wait(bar, phase & 1, status, abort);
  return __all_sync(kFull, ok) != 0;
}
__device__ __forceinline__ void arrive_if(uint32_t bar, bool yes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"((uint32_t)yes)
      : "memory");
}
__device__ __forceinline__ float4 lds128(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// True for one lane of the (converged) warp, in a form that tells the compiler
// so: the tcgen05 instructions then take their operands from uniform
// registers without a loop over lanes.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Where a column's lse stands in its stage: the four columns 8 c + 2 q + e
// (c = 2 m, 2 m + 1; e = 0, 1) that the epilogue's lanes q = lane % 4 need
// together are one 16-byte vector, [m][q].
__device__ __forceinline__ int lse_slot(int col) {
  return ((col >> 4) << 4) | ((col & 6) << 1) | ((col >> 2) & 2) | (col & 1);
}

// One item: request i, KV head and keys by its place `local` among the
// request's items (every head's first keys, which the most queries see, come
// first), split over `ctas` CTAs of a cluster. Whole CTA. `again`: more items
// may follow; `started`: the CTA has had one before (its tensor memory and
// barriers are there). False when a wait gave up.
template <int D, bool again>
__device__ __forceinline__ bool key_item(const CUtensorMap& q_map, const CUtensorMap& k_map,
                                         const KeyWeightsParams& p, uint8_t* smem, int i,
                                         int local, int rank, int ctas, bool flag,
                                         bool* started) {
  using Lay = Layout<D>;
  Bars* bars = reinterpret_cast<Bars*>(smem + Lay::BAR_OFF);
  // (the shuffle tells the compiler that the warp's number is uniform)
  const int warp = __shfl_sync(kFull, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int h = local % p.num_kv_heads;
  const int key0 = local / p.num_kv_heads * (kKT * kTM);
  const int G = p.num_heads / p.num_kv_heads;
  const int32_t* table = p.block_table + (int64_t)i * p.max_blocks;
  // an epilogue thread's key, and its page: looked up before the request's
  // lengths are known, so that the two loads overlap
  const int my_key = key0 + ((warp >> 2) & 1) * kTM + (warp & 3) * 32 + lane;
  int32_t my_page = -1;
  const int box_key = key0 + (lane & 15) * 16;  // (the copying warp: its lane's 16 keys)
  const int look = warp == kTmaWarp ? box_key : my_key;
  if (warp <= kTmaWarp && look / p.block_size < p.max_blocks)
    my_page = __ldg(table + look / p.block_size);
  // these exits are uniform, for a cluster too
  KeyRequest r;
  if (!key_request(p, i, flag, &r)) return true;
  if (r.qlen <= p.short_max_q) {  // on the mma.sync grid
    if (p.no_short && flag) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return true;
  }
  if (key0 >= r.L) return true;
  const int nk = min(kKT, (r.L - key0 + kTM - 1) / kTM);  // K tiles with keys
  const int QT = kTN / G;                                 // queries per Q tile
  const int qpos0 = r.L - r.qlen;
  const int j0 = max(0, key0 - qpos0);                    // the first query that sees key0
  const int all_tiles = (r.qlen - j0 + QT - 1) / QT;
  const int n = (all_tiles - rank + ctas - 1) / ctas;  // tiles rank, rank + ctas, ...

  if (warp == kTmaWarp && lane == 0) {
    if (!*started) {
      prefetch_tmap(&k_map);
      prefetch_tmap(&q_map);
      bars->abort = 0;
    } else {  // (every arrival on them has been waited for)
      for (uint32_t b = 0; b < kNumBars; ++b) mbar_inval(smem_addr(bars) + b * 8);
      for (uint32_t b = 0; b < kKT * 2 * kAcc; ++b)
        mbar_inval(smem_addr(bars->s_full) + b * 8);
    }
    mbar_init(smem_addr(&bars->k_land), 1);
    mbar_init(smem_addr(&bars->k_read), 8 * nk);
    for (int x = 0; x < kKT; ++x) mbar_init(smem_addr(&bars->k_full[x]), 8);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(&bars->q_full[s]), 1);
      mbar_init(smem_addr(&bars->q_empty[s]), nk);
      mbar_init(smem_addr(&bars->l_full[s]), 32);
      mbar_init(smem_addr(&bars->l_empty[s]), 8 * nk);
    }
    for (int x = 0; x < kKT; ++x)
      for (int b = 0; b < kAcc; ++b) {
        mbar_init(smem_addr(&bars->s_full[x][b]), 1);
        mbar_init(smem_addr(&bars->s_full[x][kAcc + b]), 1);
        mbar_init(smem_addr(&bars->s_free[x][b]), 4);
      }
    mbar_init(smem_addr(&bars->mma_done), nk);
    fence_barrier_init();
  }
  if (warp == kMmaWarp && !*started) {
    tmem_alloc(smem_addr(&bars->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  *started = true;
  if (ctas > 1) cluster_arrive();  // waited for before the first remote store
  const uint32_t tmem = bars->tmem_base;
  volatile int32_t* abort = &bars->abort;
  const uint32_t q_s = smem_addr(smem + Lay::Q_OFF);
  float* lse_s = reinterpret_cast<float*>(smem + Lay::LSE_OFF);
  float total = 0.f;  // of one key, in an epilogue thread

  if (warp == kTmaWarp) {
    // ---- K: 16-key boxes into the last Q stages (K tile x: stage 2 + x),
    // which are free until the epilogue warps have moved K to tensor memory.
    // Bad pages and keys past the context stay unloaded: their rows meet
    // nothing else and are never written out
    const bool in = lane < kKT * kTM / 16 && box_key < r.L && n > 0;
    const bool good = in && my_page >= 0 && my_page < p.num_blocks;
    const uint32_t load = __ballot_sync(kFull, good);
    if (__any_sync(kFull, in && !good) && lane == 0 && rank == 0)
      set_status(p.status, PKV_DEV_BAD_BLOCK);
    if (lane == 0)
      mbar_arrive_expect_tx(smem_addr(&bars->k_land), __popc(load) * Lay::NCH * 16 * 128);
    __syncwarp();
    if (good)
      for (int c = 0; c < Lay::NCH; ++c)
        tma_load_4d(q_s + (2 + (lane >> 3)) * Lay::TILE_BYTES + c * Lay::CH_BYTES +
                        (lane & 7) * 16 * 128,
                    &k_map, smem_addr(&bars->k_land), 0,
                    my_page * p.block_size + box_key % p.block_size, h, c);
    if (lane == 0) {
      const uint32_t bytes = (uint32_t)(Lay::NCH * QT * G * 128);
      int t = 0;
      for (; t < n; ++t) {
        const int s = t % kStages;
        if (t == 2 && !mbar_wait(smem_addr(&bars->k_read), 0, p.status, abort)) break;
        if (t >= kStages &&
            !mbar_wait(smem_addr(&bars->q_empty[s]), (t / kStages - 1) & 1, p.status, abort))
          break;
        mbar_arrive_expect_tx(smem_addr(&bars->q_full[s]), bytes);
        const int j = r.t0 + j0 + (rank + t * ctas) * QT;
        for (int c = 0; c < Lay::NCH; ++c)
          tma_load_3d(q_s + s * Lay::TILE_BYTES + c * Lay::CH_BYTES, &q_map,
                      smem_addr(&bars->q_full[s]), c * 64, h * G, j);
      }
      // copies in flight land before the CTA can exit
      for (int g = max(0, t - kStages); g < t; ++g)
        mbar_wait(smem_addr(&bars->q_full[g % kStages]), (g / kStages) & 1, nullptr);
      mbar_wait(smem_addr(&bars->k_land), 0, nullptr);
      // and, where the barriers will be set up again, so do the issuing warps'
      // last releases of the stages
      if (again && t == n)
        for (int g = max(0, n - kStages); g < n; ++g)
          mbar_wait(smem_addr(&bars->q_empty[g % kStages]), (g / kStages) & 1, p.status, abort);
    }
  } else if (warp >= kMmaWarp) {
    // ---- the products of K tile x. (A lane's next operands wait for the
    // MMAs it has issued, so a warp's barrier waits are not hidden behind its
    // own MMAs: the two warps hide each other's.)
    const int x = warp - kMmaWarp;
    if (x < nk) {
      constexpr uint32_t idesc = umma_idesc_bf16(kTM, kHalf, false, false);
      const uint64_t qd = smem_desc_sw128(q_s, 16, 1024);
      const uint32_t k_tmem = tmem + kKCol + (uint32_t)(x * (D / 2));
      bool ok = n > 0 && warp_wait(smem_addr(&bars->k_full[x]), 0, p.status, abort);
      int b = 0, turn = 0;  // accumulator, and how often each has been used
      for (int t = 0; ok && t < n; ++t) {
        const int s = t % kStages;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // even lanes: the accumulator (before its first use the phase
          // "before the first" counts as complete), odd lanes: the Q tile
          ok = warp_wait((lane & 1) ? smem_addr(&bars->q_full[s]) : smem_addr(&bars->s_free[x][b]),
                         (lane & 1) ? t / kStages : turn + 1, p.status, abort);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off =
                  ((kk >> 2) * Lay::CH_BYTES + (kk & 3) * 32 + half * kHalf * 128) >> 4;
              umma_ts(tmem + (uint32_t)((x * kAcc + b) * kHalf), k_tmem + (uint32_t)(kk * 8),
                      qd + (uint32_t)((s * Lay::TILE_BYTES) >> 4) + off, idesc, kk > 0);
            }
            umma_commit(smem_addr(&bars->s_full[x][b + (turn & 1) * kAcc]));
            if (half == 1) umma_commit(smem_addr(&bars->q_empty[s]));
          }
          __syncwarp();
          if (++b == kAcc) {
            b = 0;
            ++turn;
          }
        }
      }
      // every MMA issued has completed before TMEM is released
      if (elect_one()) umma_commit(smem_addr(&bars->mma_done));
      __syncwarp();
      warp_wait(smem_addr(&bars->mma_done), 0, nullptr, nullptr);
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
      const int j = j0 + (rank + t * ctas) * QT;
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
          ok = warp_wait(smem_addr(&bars->l_empty[s]), t0 / kStages - 1, p.status, abort);
          if (!ok) break;
        }
        uint32_t empty = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool none = v[s][e] == -INFINITY;
          empty |= __any_sync(kFull, none) ? 1u << e : 0u;
          lse_s[s * kTN + lse_slot(e * 32 + lane)] = none ? -INFINITY : -kLog2e * v[s][e];
        }
        if (lane == 0) *reinterpret_cast<volatile uint32_t*>(&bars->masked[s]) = empty;
        __syncwarp();
        mbar_arrive(smem_addr(&bars->l_full[s]));
        fetch(t0 + s + kStages, v[s]);
      }
    }
  } else if (((warp >> 2) & 1) < nk) {
    // ---- weights of tile x's keys in columns [64 half, 64 half + 64). A
    // thread has 4 keys (wkey + lane / 4 + 8 k) and 2 of every 8 columns: a
    // column's lse, read from shared memory, serves 4 scores
    const int x = (warp >> 2) & 1, half = warp >> 3;
    const int wkey = key0 + x * kTM + (warp & 3) * 32;  // the warp's first key
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    bool ok = n > 0 && warp_wait(smem_addr(&bars->k_land), 0, p.status, abort);
    if (ok) {
      // half of the key's row to tensor memory, the A operand
      constexpr int U = D / 16;  // 16-byte units of half a row
      const uint32_t row = (warp & 3) * 32 + lane;
      uint32_t w[D / 4];
#pragma unroll
      for (uint32_t c = 0; c < U; ++c) {
        const uint32_t unit = half * U + c;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[4 * c]), "=r"(w[4 * c + 1]), "=r"(w[4 * c + 2]), "=r"(w[4 * c + 3])
                     : "r"(q_s + (2 + x) * Lay::TILE_BYTES + (unit >> 3) * Lay::CH_BYTES +
                           row * 128 + (((unit & 7) ^ (row & 7)) << 4))
                     : "memory");
      }
      const uint32_t at = tmem + lanes + kKCol + (uint32_t)(x * (D / 2) + half * (D / 4));
      if constexpr (D == 128)
        PKV_TMEM_ST32(at, w);
      else
        PKV_TMEM_ST16(at, w);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      arrive_if(smem_addr(&bars->k_read), lane == 0);
      arrive_if(smem_addr(&bars->k_full[x]), lane == 0);
    }
    const float2 sc = make_float2(p.scale_log2, p.scale_log2);
    const uint32_t nl = smem_addr(lse_s + half * kHalf + 4 * (lane & 3));
    const uint32_t s_full0 = smem_addr(&bars->s_full[x][0]);
    const uint32_t s_free0 = smem_addr(&bars->s_free[x][0]);
    const uint32_t l_full0 = smem_addr(&bars->l_full[0]), l_empty0 = smem_addr(&bars->l_empty[0]);
    const uint32_t masked0 = smem_addr(&bars->masked[0]);
    // sums of a few tiles, in two chains a key, then of the groups of tiles:
    // no chain is longer than a few hundred additions
    float2 a[4];
    float sum4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = make_float2(0.f, 0.f);
    uint32_t b = half, turn = 0;  // the accumulator, and how often it has been used
    // the first column of this half that sees the warp's first key, and the
    // columns there are from this half's first one on (every query sees keys
    // 64 places before it, and the distance times G may pass 32 bits)
    int first = max(wkey - qpos0 - j0 - rank * QT, -64) * G - half * kHalf;
    int left = (r.qlen - j0 - rank * QT) * G - half * kHalf;
    const int step = ctas * QT * G;
    for (int t = 0; ok && t < n; ++t, first -= step, left -= step) {
      const uint32_t s = (uint32_t)t % kStages;
      ok = warp_wait(s_full0 + (b + (turn & 1) * kAcc) * 8, turn >> 1, p.status, abort) &&
           warp_wait(l_full0 + s * 8, (uint32_t)t / kStages, p.status, abort);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + lanes + (x * kAcc + b) * kHalf;
      const uint32_t masked = (lds32(masked0 + s * 4) >> (2 * half)) & 3u;
      const bool plain = first + 31 * G <= 0 && !masked;  // every column sees every key of the warp
      const bool some = left > 0 && first < kHalf;        // some column is there and sees some key
#pragma unroll
      for (int g = 0; g < 2; ++g) {  // 32 columns at a time: fewer registers, no spills
        uint32_t u[2][16];
        PKV_TMEM_LD_16X256B_X4(acc + g * 32, u[0]);
        PKV_TMEM_LD_16X256B_X4(acc + g * 32 + (16u << 16), u[1]);
        float4 l4[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) l4[m] = lds128(nl + s * (kTN * 4) + (2 * g + m) * 64);
        tmem_wait_ld();
        if (g == 1) {  // the tile is in registers, and its lse
          tc_fence_before();
          __syncwarp();
#ifdef PKV_TEST_HOLD_ARRIVAL
          if (!(g_pkv_test_hold_key_weights && blockIdx.x == 0 && blockIdx.y == 0 && warp == 0 &&
                t == 0))
#endif
            arrive_if(s_free0 + b * 8, lane == 0);
          arrive_if(l_empty0 + s * 8, lane == 0);
        }
        if (plain) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 l = l4[c >> 1];
            const float2 l2 = (c & 1) ? make_float2(l.z, l.w) : make_float2(l.x, l.y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 4 * c + 2 * (k & 1);
              const float2 y = __ffma2_rn(make_float2(__uint_as_float(u[k >> 1][e]),
                                                      __uint_as_float(u[k >> 1][e + 1])),
                                          sc, l2);
              a[k] = __fadd2_rn(a[k], make_float2(fast_exp2(y.x), fast_exp2(y.y)));
            }
          }
        } else if (some) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float4 l = l4[c >> 1];
            const float2 l2 = (c & 1) ? make_float2(l.z, l.w) : make_float2(l.x, l.y);
            const int col = g * 32 + 8 * c + 2 * (lane & 3);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 4 * c + 2 * (k & 1);
              const int sees = first + ((lane >> 2) + 8 * k) * G;
              const float y = fast_exp2(fmaf(__uint_as_float(u[k >> 1][e]), p.scale_log2, l2.x));
              const float z =
                  fast_exp2(fmaf(__uint_as_float(u[k >> 1][e + 1]), p.scale_log2, l2.y));
              // selected, not multiplied: the score of an empty or hidden
              // column may be anything
              a[k].x += (l2.x == -INFINITY || col < sees) ? 0.f : y;
              a[k].y += (l2.y == -INFINITY || col + 1 < sees) ? 0.f : z;
            }
          }
        }
      }
      b += 2;
      if (b >= kAcc) {
        b -= kAcc;
        ++turn;
      }
      if ((t & 15) == 15) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sum4[k] += a[k].x + a[k].y;
          a[k] = make_float2(0.f, 0.f);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sum4[k] += a[k].x + a[k].y;
    // the four threads of a key; thread q of them keeps key lane / 4 + 8 q
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v = sum4[k];
      v += __shfl_xor_sync(kFull, v, 1);
      v += __shfl_xor_sync(kFull, v, 2);
      if ((lane & 3) == k) total = v;
    }
  }

  // ---- the partial sums of the column halves and of the cluster's CTAs,
  // added in a fixed order: [cluster rank][column half][256 keys] in rank 0
  float* red = reinterpret_cast<float*>(smem + Lay::RED_OFF);
  constexpr int kKeys = kKT * kTM;
  const int slot = warp < kEpiWarps ? (rank * 2 + (warp >> 3)) * kKeys + (warp & 7) * 32 +
                                          (lane >> 2) + 8 * (lane & 3)
                                    : -1;
  if (ctas > 1) {
    __syncwarp();
    cluster_wait();  // every CTA of the cluster has started
    if (slot >= 0) st_cluster(smem_addr(red + slot), 0, total);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  } else {
    if (slot >= 0) red[slot] = total;
    __syncthreads();
  }
  if (rank == 0 && threadIdx.x < kKeys) {
    if (my_key < r.L && my_page >= 0 && my_page < p.num_blocks) {
      total = red[threadIdx.x];
      for (int c = 1; c < 2 * ctas; ++c) total += red[c * kKeys + threadIdx.x];
      const int64_t at = ((int64_t)r.row * p.num_kv_heads + h) * p.row_len + my_key;
      p.out[at] = my_key < r.prior && p.decay != 0.f ? fmaf(p.decay, p.in[at], total) : total;
    }
  }
  // all of the item's work is complete
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  return *const_cast<volatile int32_t*>(&bars->abort) == 0;
}

// Not Listed: a cluster of `ctas` CTAs for each item (blockIdx.y the request,
// blockIdx.x / ctas its item). Listed: each CTA goes through a share of all
// requests' items, listed in shared memory; every other turn goes backwards
// through the CTAs, so that a CTA's items are of mixed sizes.
template <int D, bool Listed>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_tc_kernel(const __grid_constant__ CUtensorMap q_map,
                          const __grid_constant__ CUtensorMap k_map, const KeyWeightsParams p,
                          const int ctas) {
  using Lay = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));

  griddep_wait();
  griddep_launch_dependents();

  bool started = false;
  if constexpr (!Listed) {
    key_item<D, false>(q_map, k_map, p, smem, blockIdx.y, blockIdx.x / ctas, blockIdx.x % ctas,
                       ctas, threadIdx.x == 0 && blockIdx.x == 0, &started);
  } else {
    int* before = reinterpret_cast<int*>(smem + Lay::LIST_OFF);  // items before each request
    for (int i = threadIdx.x; i < p.num_seqs; i += kThreads) {
      KeyRequest r;
      const bool any = key_request(p, i, blockIdx.x == 0, &r);
      const bool here = any && r.qlen > p.short_max_q;
      if (any && !here && p.no_short && blockIdx.x == 0) set_status(p.status, PKV_DEV_BAD_LENGTHS);
      before[i + 1] = here ? (r.L + kKT * kTM - 1) / (kKT * kTM) * p.num_kv_heads : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      int sum = 0;
      for (int i0 = 0; i0 < p.num_seqs; i0 += 32) {
        const bool in = i0 + lane < p.num_seqs;
        int v = in ? before[i0 + lane + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(kFull, v, o);
          if (lane >= o) v += x;
        }
        if (in) before[i0 + lane + 1] = sum + v;
        sum += __shfl_sync(kFull, v, 31);
      }
      if (lane == 0) before[0] = 0;
    }
    __syncthreads();
    for (int turn = 0;; ++turn) {
      const int64_t at = (int64_t)turn * gridDim.x +
                         ((turn & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      if (at >= before[p.num_seqs]) break;
      int lo = 0, hi = p.num_seqs;  // the last request with before[lo] <= at
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= at)
          lo = mid;
        else
          hi = mid;
      }
      if (!key_item<D, true>(q_map, k_map, p, smem, lo, (int)at - before[lo], 0, 1, false,
                             &started))
        break;
    }
  }
  if (started && __shfl_sync(kFull, threadIdx.x >> 5, 0) == kMmaWarp)
    tmem_dealloc(reinterpret_cast<Bars*>(smem + Lay::BAR_OFF)->tmem_base, kTmemCols);
}

template <int D>
cudaError_t launch(const KeyWeightsParams& p, const CUtensorMap& q_map, const CUtensorMap& k_map,
                   cudaStream_t stream) {
  static SmemLimit limit, limit_listed;
  cudaError_t e = limit.ensure(reinterpret_cast<const void*>(key_weights_tc_kernel<D, false>),
                               Layout<D>::BYTES);
  if (e == cudaSuccess)
    e = limit_listed.ensure(reinterpret_cast<const void*>(key_weights_tc_kernel<D, true>),
                            Layout<D>::BYTES);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int G = p.num_heads / p.num_kv_heads;
  const int64_t key_tiles = ((int64_t)p.max_seq_len + kKT * kTM - 1) / (kKT * kTM);
  // (the work is that of about num_tokens / max_query_len requests of full length)
  const int64_t items =
      key_tiles * p.num_kv_heads * ((p.num_tokens + p.max_query_len - 1) / p.max_query_len);
  const int q_tiles = (p.max_query_len + kTN / G - 1) / (kTN / G);
  // Split an item's Q tiles while there are fewer than two items an SM and a
  // CTA keeps at least 8 tiles for its K tiles. (One 8192-token prompt, 256
  // items of 8 to 256 tiles: 217 us whole, 212 in two, 255 in four; a mixed
  // batch with some 480 items of about 12 tiles: 60 us whole, 85 in two: a
  // cluster waits until all its SMs are free, and every CTA pays about 4 us
  // before its first and after its last product.)
  int clusters = 1;
  while (clusters < kMaxCluster && items * clusters < 2 * sms && q_tiles / clusters >= 16)
    clusters *= 2;
  // Many items: max_seq_len may be far above the requests' lengths, and a CTA
  // that finds no keys takes a turn on an SM like any other (one CTA an SM).
  // CTAs that list the items first skip the empty ones. (32 chunks of 20 to
  // 100 queries, 2560 items in bounds and about half of them there: 59.5 us,
  // 69 with a CTA for each; 512 queries over 32K keys, 1024 items, all there:
  // 136 us, 131 with a CTA for each, which the hardware hands out as SMs fall
  // free; 13 requests, 1040 items in bounds, 484 there: 83 and 59 us, the
  // difference being the single tokens' grid, which then waits to the end.)
  // Not listed are items split over a cluster and batches of more than kListed
  // requests: there every request, a single token too, has its CTAs in bounds,
  // about 1 us each on one SM after the other (64 single tokens and a chunk of
  // 2048, contexts to 4096: 259 us; in calls of their own 46 and 62).
  const int64_t bound = key_tiles * p.num_kv_heads * p.num_seqs;
  const bool listed =
      clusters == 1 && p.num_seqs <= kListed && bound > 12 * sms && bound < (1 << 30);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = listed ? dim3((unsigned)sms)
                       : dim3((unsigned)(key_tiles * p.num_kv_heads * clusters),
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
  return listed ? cudaLaunchKernelEx(&cfg, key_weights_tc_kernel<D, true>, q_map, k_map, p, 1)
                : cudaLaunchKernelEx(&cfg, key_weights_tc_kernel<D, false>, q_map, k_map, p,
                                     clusters);
}

}  // namespace

cudaError_t launch_key_weights_tc(const KeyWeightsParams& p, const CUtensorMap& q_map,
                                  const CUtensorMap& k_map, cudaStream_t stream) {
  return p.head_dim == 64 ? launch<64>(p, q_map, k_map, stream)
                          : launch<128>(p, q_map, k_map, stream);
}

}  // namespace pkv
