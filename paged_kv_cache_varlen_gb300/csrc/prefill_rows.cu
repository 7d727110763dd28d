// prefill_rows.cu -- paged attention for requests of more than 32 (query, head) rows
// through a window, over a bf16 pool or over one held in 8 bits, on the
// 5th-generation tensor cores (tcgen05). The formulas stand in decode_rows.cu.
//
//   * persistent CTAs, one per SM; a work item is (request, KV head, two query
//     tiles A and B of 128 rows, 128 / G queries of G heads each), taken in the
//     order of the heaviest requests from a ticket counter in the workspace. Where
//     there are too few items for the SMs, each CTA has an equal share of all their
//     tiles instead, and the pieces of an item are joined by log-sum-exp;
//   * the keys that some query of an item sees, its sinks' 16-key chunks and then
//     its window's, are numbered through: a tile is consecutive ones of them, wherever
//     they lie in the context, so that a few sinks cost a quarter of a tile and a
//     window no more than its ends. In these numbers a row sees the columns
//     [low, lim] and those before the sinks' end;
//   * S = Q K^T over 64 keys (bf16), O += P V (fp16 P and V), fp32 accumulators in
//     tensor memory: two S and one O of both query tiles fill its 512 columns, P
//     (fp16) lies over the first half of its S;
//   * a warp issues a query tile's products by one elected lane: S(0), S(1), then
//     PV(j), S(j + 2), so that a softmax goes from one tile to the next without
//     waiting for products. (By a lane of a diverged warp each product takes a loop
//     over lanes to get its operands: 171 us for the prompt below, 156 so.);
//   * a softmax thread owns a row: 64 scores in registers, one pass;
//   * K and V arrive by TMA in 16-key boxes, K into two stages of 128 keys, V into five
//     of 64. V becomes fp16 in place (four converter warps); at 8 bits K becomes bf16
//     and V fp16, both exactly, and a block's two scales act on the scores;
//   * bf16 values have a wider range than fp16: the 64 of a stage are multiplied by one
//     power of two, which its weights take up as they do an 8-bit block's scale (the
//     prompt below, in a graph, 156 us; 153 without, which lost values below 2^-17 and
//     refused those from 2^16 on; 160 with a power for every 16 keys: a longer softmax);
//   * every wait is bounded; on a timeout the CTA drains its copies and products,
//     frees its tensor memory and leaves with PKV_DEV_TIMEOUT set.
//
// What bounds it (32 + 8 heads of 128): 64 keys take ~1880 cycles over 8 bits and ~1840
// over bf16, where the products of both query tiles take 1024 and shared memory, at 128
// bytes a cycle, 1536 (Q and K of 64-key products 96 KB, V's products 32, the
// conversions 32, the copies 32). With half of the score products left out 8 and 12 %
// of the time go, without the conversions 6 and 3 %, without the exponentials none: over
// bf16 it is shared memory most of all, over 8 bits the waiting of softmax, products and
// conversions for one another, at 57 % of the issue slots. 8-bit chunks of 1500 to 2048
// tokens over 4096 to 8192 keys: 349 us, 51 % of the bf16 peak; a prompt of 8192 tokens
// through a window of 1024: 158 us, 42 %. Tried (at 349 and 154 us): 128-key tiles with
// one S each (less of shared memory, a longer chain: 358 and 157), the weights formed
// before the maximum is known (373), a half of the next scores loaded between the halves
// of a softmax (392), their barrier asked then (351).
#include <float.h>
#include <math.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "launch.h"
#include "wait.cuh"

namespace pkv {
namespace {

constexpr int kBM = 128;      // rows of a query tile
constexpr int kBN = 128;      // keys of a K stage
constexpr int kSub = 16;      // keys of a TMA box
constexpr int kBoxes = kBN / kSub;
constexpr int kNS = 2;        // stages of the K ring
constexpr int kHalf = 64;     // keys of a score tile, and of a V stage: a stage is copied,
                              // converted and held until both query tiles have used it
constexpr int kHalfBoxes = kHalf / kSub;
constexpr int kVS = 5;        // stages of the V ring
constexpr int kThreads = 512;
// warps: 0-3 softmax of A, 4-7 of B, 8-11 converters, 12 and 13 the products of A
// and of B, 14 tickets and K, 15 Q and V
constexpr int kConvWarp0 = 8, kMmaWarp = 12, kKWarp = 14, kVWarp = 15;
constexpr int kConverters = 128;
// registers a thread: launched with 128; the softmax warpgroups take more of them
constexpr int kSoftmaxRegs = 152, kOtherRegs = 104;
static_assert(2 * kSoftmaxRegs + 2 * kOtherRegs == 4 * (65536 / kThreads),
              "the register split adds up to the launch's registers");
constexpr uint32_t kTmemCols = 512;
constexpr int kRing = 4;  // items announced ahead of their readers
constexpr int kItemReaders = 8 + 4 + 3;  // softmax and converter warps, products, V
constexpr int kSortMax = 768;
// In 64-key tiles' time: what an item costs to begin, what cutting costs a CTA; cycles
// of one, and bytes of the pool that an SM of the decode grid reads in a cycle (for the
// split of the SMs in a call with both kinds of request).
constexpr int kItemTiles = 4;
constexpr float kPieceTiles = 9.f;
constexpr float kTileCycles = 2000.f;
constexpr float kDecodeBytesPerCycle = 40.f;
constexpr int kCutUnits = 2 * kThreads;  // calls of more units are not cut
constexpr int kCutKeys = 1 << 24;        // nor of longer contexts (the sums stay in 32 bits)
constexpr int kMinShare = 4;             // tiles
// p.sched from here on: of each CTA, what it says of the item that begins in its share
// and is cut: 8 warps' counts of finished pieces, or (prefill_join) a record
constexpr int kRecords = 64;
constexpr int kMaxCtas = 152;  // shares at most: their pieces have room in the workspace
// A row's reference moves when a score outgrows it by 2^14: weights up to that stay in
// fp16's range, with their 11 bits, and O is seldom rescaled (8-bit chunks of 2048
// tokens: 349 us, 357 from 2^8 on, 364 from 2^4).
constexpr float kRescaleThreshold = 14.f;
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kMinusInf = 0xff800000u;
constexpr int32_t kBadRow = -2;  // of a box in a block that is not there (-1: of none)

constexpr size_t list_ints(int num_seqs) {
  return (num_seqs <= kSortMax ? 5 : 1) * ((size_t)num_seqs + 1);
}

template <int D>
struct Layout {
  static constexpr int NCH = D / 64;               // 128-byte column chunks of a row
  static constexpr int CH_BYTES = 128 * 128;
  static constexpr int TILE_BYTES = NCH * CH_BYTES;
  static constexpr int VCH_BYTES = kHalf * 128;    // a chunk of a V stage
  static constexpr int VS_BYTES = NCH * VCH_BYTES;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * TILE_BYTES;
  static constexpr int V_OFF = K_OFF + kNS * TILE_BYTES;
  static constexpr int BAR_OFF = V_OFF + kVS * VS_BYTES;
  static constexpr int LIST_OFF = BAR_OFF + 768;
  // one CTA an SM (each takes all of its tensor memory)
  static size_t bytes(int num_seqs) {
    const size_t need = 1024 + LIST_OFF + list_ints(num_seqs) * 4;
    return need > 120 * 1024 ? need : 120 * 1024;
  }
  __device__ static constexpr uint32_t s_col(int x) { return 128u * (uint32_t)x; }  // 2 x 64
  __device__ static constexpr uint32_t o_col(int x) { return 256u + 128u * (uint32_t)x; }
};

// A run of tiles of an item (all of them, where the work is not cut): tiles
// [first, first + n); `pieces` of it from CTA `head` on.
struct Piece {
  int32_t id, first, n, head, pieces;
};

// What the threads of a CTA pass one another while they plan.
struct Sums {
  unsigned long long chunks, row;
  int32_t scan[kThreads / 32];
  int32_t start[3];  // a share's first unit, KV head, place in the item
  int32_t cands;
  int32_t lightest, heaviest;  // the items' lengths
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_landed[kNS], k_full[kNS], k_empty[kNS];  // (landed: 8 bits)
  uint64_t v_landed[kVS], v_full[kVS], v_empty[kVS];
  uint64_t s_full[2][2];   // S(j) of a query tile is there: [x][j & 1]
  uint64_t p_ready[2][2];  // P(j) is stored (and O rescaled)
  uint64_t o_done[2][2];   // PV(j) is done
  uint64_t o_free[2];      // the item's O has been read
  uint64_t mma_done;
  uint64_t v_sized;        // bf16: every converter warp has said how large its rows are
  uint64_t item_full[kRing], item_empty[kRing];
  Piece item[kRing];
  uint32_t tmem_base;
  int32_t abort;
  uint32_t k_mask[kNS], v_mask[kVS];  // boxes of a stage that were loaded
  uint32_t v_top[2][kConverters / 32];
  float2 v_scale[kVS];  // bf16: what undoes the power that a stage's values were scaled by:
                        // its log2, and the power
  Sums sums;
};
static_assert(sizeof(Bars) <= 768, "the barriers fit below the work list");

struct Item {
  int req, kvh, j0, j1, t0;
  // of the piece; columns are counted from its first
  int n;       // score tiles
  int base;    // the item's column that is the piece's first
  int shift;   // from a column behind the sinks' to its key
  int columns; // of the sinks' chunks: columns before it are base less than their keys
  int count;   // 16-key chunks
  int qpos0;   // position of the request's first query
  int sink;    // columns before it are sinks
  int end;     // columns before it are needed keys
  int lo_any;  // no query of the item sees columns [sink, lo_any)

  __device__ __forceinline__ int key(int column) const {
    return column + (column < columns ? base : shift);
  }
};

__device__ __forceinline__ int tiles_of(const AttnParams& p, int first, int end) {
  return (visible_units(p.window, p.num_sink, first, end, kSub).count + kHalfBoxes - 1) /
         kHalfBoxes;
}

// Exclusive prefix sum of one value a thread; *total gets the sum. All threads.
__device__ __forceinline__ int block_scan(int v, int32_t* scan, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int x = scan[w];
    if (w < warp) base += x;
    all += x;
  }
  __syncthreads();
  *total = all;
  return base + incl - v;
}

// The units in the order that they are handed out: position k is request
// order[k] (null: k), units before it pref[k], pref[n] all.
struct List {
  const int *order, *pref;
  int n;
};

// Item `it`, tiles [first, first + n) of it (n < 0: all).
__device__ __forceinline__ Item item_of(const AttnParams& p, const List& list, int QP, int it,
                                        int first_tile, int n_tiles) {
  Item d;
  const int u = it / p.num_kv_heads;
  d.kvh = it - u * p.num_kv_heads;
  int lo = 0, hi = list.n;  // largest lo with pref[lo] <= u
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (list.pref[mid] <= u)
      lo = mid;
    else
      hi = mid;
  }
  d.req = list.order ? list.order[lo] : lo;
  d.t0 = __ldg(p.cu_seqlens + d.req);
  const int n = __ldg(p.cu_seqlens + d.req + 1) - d.t0;
  d.qpos0 = __ldg(p.seq_lens + d.req) - n;
  const int unit = (n + QP - 1) / QP - 1 - (u - list.pref[lo]);  // later (heavier) units first
  d.j0 = unit * QP;
  d.j1 = min(n, d.j0 + QP);
  const int first = d.qpos0 + d.j0, end = d.qpos0 + d.j1;
  const Visible v = visible_units(p.window, p.num_sink, first, end, kSub);
  const int shift = (v.low - v.sink) * kSub;
  d.base = first_tile * kHalf;
  d.shift = shift + d.base;
  d.columns = v.sink * kSub - d.base;
  d.count = v.count - first_tile * kHalfBoxes;
  d.n = n_tiles < 0 ? (v.count + kHalfBoxes - 1) / kHalfBoxes : n_tiles;
  d.sink = p.num_sink - d.base;
  d.end = end - d.shift;
  d.lo_any = max(0, first - p.window + 1) - d.shift;
  return d;
}

// Shares: the items stand in a row, unit after unit, the KV heads of a unit one after
// the other; an item is as long as its tiles and kItemTiles, what it costs to begin
// one. A CTA has the tiles that lie in its share of the row, `ctas` shares of `size` or
// (the first `more`) size + 1.
struct Share {
  uint32_t ctas;      // 0: items are handed out by tickets
  uint32_t size, more;
  uint32_t at, end;   // the CTA's place in the row, and the end of its share
  int unit, kvh;      // where that is
  int in;             // in the item
  int tiles;          // of the unit's items (0: not known yet)

  __device__ __forceinline__ uint32_t start(uint32_t cta) const {
    return cta * size + min(cta, more);
  }
  __device__ __forceinline__ int cta_of(uint32_t x) const {
    const uint32_t longer = more * (size + 1);
    return (int)(x < longer ? x / (size + 1) : more + (x - longer) / size);
  }
};

// The next piece: of the CTA's share, or a whole item by the next ticket. One lane of
// the K warp announces it in a small ring; every other role reads it from there.
template <bool CUT>
__device__ __forceinline__ Piece next_piece(const AttnParams& p, const List& list, int QP,
                                            int items, Share& sh) {
  Piece c{-1, 0, -1, 0, 1};
  if (!CUT || sh.ctas == 0) {
    const int t = atomicAdd(p.sched, 1);
    c.id = t < items ? t : -1;
    return c;
  }
  if (sh.in < kItemTiles) {
    sh.at += kItemTiles - sh.in;
    sh.in = kItemTiles;
  }
  if (sh.at >= sh.end) return c;
  if (sh.tiles == 0) sh.tiles = item_of(p, list, QP, sh.unit * p.num_kv_heads, 0, -1).n;
  c.id = sh.unit * p.num_kv_heads + sh.kvh;
  c.first = sh.in - kItemTiles;
  c.n = min(sh.tiles - c.first, (int)(sh.end - sh.at));
  const uint32_t begin = sh.at - c.first;  // the item's first tile
  c.head = sh.cta_of(begin);
  c.pieces = sh.cta_of(begin + sh.tiles - 1) - c.head + 1;
  sh.at += c.n;
  sh.in += c.n;
  if (c.first + c.n == sh.tiles) {
    sh.in = 0;
    if (++sh.kvh == p.num_kv_heads) {
      sh.kvh = 0;
      sh.tiles = 0;
      ++sh.unit;
    }
  }
  return c;
}
template <bool CUT>
__device__ __forceinline__ Piece take_item(Bars* bars, const AttnParams& p, const List& list,
                                           int QP, int items, Share& sh, int k,
                                           volatile int32_t* abort) {
  const int slot = k % kRing;
  Piece c{-1, 0, -1, 0, 1};
  if (k < kRing ||
      short_wait(smem_addr(&bars->item_empty[slot]), ((k / kRing) - 1) & 1, p.status, abort))
    c = next_piece<CUT>(p, list, QP, items, sh);
  bars->item[slot] = c;  // (before the barrier's release)
  mbar_arrive(smem_addr(&bars->item_full[slot]));
  return c;
}
__device__ __forceinline__ Piece read_item(Bars* bars, const AttnParams& p, int k,
                                           volatile int32_t* abort) {
  const int slot = k % kRing;
  Piece c{-1, 0, -1, 0, 1};
  if (short_wait(smem_addr(&bars->item_full[slot]), (k / kRing) & 1, p.status, abort)) {
    const volatile Piece* x = &bars->item[slot];
    c.id = x->id;
    c.first = x->first;
    c.n = x->n;
    c.head = x->head;
    c.pieces = x->pieces;
  }
  mbar_arrive(smem_addr(&bars->item_empty[slot]));
  return c;
}
template <bool CUT>
__device__ __forceinline__ Piece all_lanes(Piece c) {
  c.id = __shfl_sync(kFull, c.id, 0);
  if (!CUT) return Piece{c.id, 0, -1, 0, 1};
  c.first = __shfl_sync(kFull, c.first, 0);
  c.n = __shfl_sync(kFull, c.n, 0);
  c.head = __shfl_sync(kFull, c.head, 0);
  c.pieces = __shfl_sync(kFull, c.pieces, 0);
  return c;
}

struct Work {
  List list;
  int items;    // units x KV heads
  int active;   // CTAs of the grid that take some
  Share share;
};

// The call's work: the requests with more than decode_max_q queries (any queries, where
// no decode grid runs beside), those with the most tiles in a unit first (batches of more
// than kSortMax requests: as they come; bad lengths flagged by one CTA), the CTAs that
// work on them, and whether their items are cut. All threads of every CTA come to the
// same result.
template <bool EIGHT, bool CUT>
__device__ __noinline__ void plan_work(const AttnParams& p, int QP, int* ints, Sums* sums,
                                       Work* out) {
  const int B = p.num_seqs, tid = threadIdx.x, lane = tid & 31;
  const bool flag = blockIdx.x == 0, sorted = B <= kSortMax;
  int* pref = ints;
  int* order = ints + (B + 1);
  int* cand = order + (B + 1);  // request, units, tiles of its heaviest unit
  // units of request r (0: none, or the decode grid's); the 16-key chunks that one of
  // the latter sees
  auto look = [&](int r, int& weight, int& chunks) {
    const int32_t t0 = __ldg(p.cu_seqlens + r), t1 = __ldg(p.cu_seqlens + r + 1);
    const int32_t L = __ldg(p.seq_lens + r);
    const int32_t n = t1 - t0;
    weight = chunks = 0;
    bool bad = t0 < 0 || t1 < t0 || t1 > p.num_tokens;
    // (a batch padded behind its last request may look as if no request were short)
    const bool short_one = !bad && n <= (p.no_decode ? 0 : p.decode_max_q);
    const bool len_ok = L >= n && L <= p.max_seq_len && L <= p.max_blocks * p.block_size;
    if (short_one) {
      if (n > 0 && len_ok) chunks = visible_units(p.window, p.num_sink, L - n, L, kSub).count;
      return 0;
    }
    bad = bad || n > p.max_query_len || !len_ok;
    if (bad) {
      if (flag) set_status(p.status, PKV_DEV_BAD_LENGTHS);
      return 0;
    }
    weight = tiles_of(p, max(0, L - QP), L);
    return (n + QP - 1) / QP;
  };
  if (tid == 0) {
    *sums = Sums{};
    sums->lightest = INT32_MAX;
  }
  __syncthreads();
  unsigned long long chunks = 0;
  int n, units;
  if (sorted) {
    for (int r = tid; r < B; r += kThreads) {
      int w, c;
      const int u = look(r, w, c);
      chunks += c;
      if (u == 0) continue;
      const int at = atomicAdd(&sums->cands, 1);
      cand[3 * at] = r;
      cand[3 * at + 1] = u;
      cand[3 * at + 2] = w;
    }
    if (p.shared_sms > 0 && chunks > 0) atomicAdd(&sums->chunks, chunks);
    __syncthreads();
    n = sums->cands;
    for (int i = tid; i < n; i += kThreads) {
      const int r = cand[3 * i], u = cand[3 * i + 1], w = cand[3 * i + 2];
      int rank = 0, before = 0;
      for (int j = 0; j < n; ++j) {
        const bool ahead = cand[3 * j + 2] > w || (cand[3 * j + 2] == w && cand[3 * j] < r);
        rank += ahead;
        before += ahead ? cand[3 * j + 1] : 0;
      }
      order[rank] = r;
      pref[rank] = before;
      if (rank == n - 1) pref[n] = before + u;
    }
    if (n == 0 && tid == 0) pref[0] = 0;
    __syncthreads();
    units = pref[n];
  } else {
    n = B;
    const int per = (B + kThreads - 1) / kThreads;
    const int r0 = min(B, tid * per), r1 = min(B, r0 + per);
    int sum = 0, all;
    for (int r = r0; r < r1; ++r) {
      int w, c;
      pref[r] = look(r, w, c);
      sum += pref[r];
      chunks += c;
    }
    if (p.shared_sms > 0 && chunks > 0) atomicAdd(&sums->chunks, chunks);
    int run = block_scan(sum, sums->scan, &all);
    for (int r = r0; r < r1; ++r) {
      const int u = pref[r];
      pref[r] = run;
      run += u;
    }
    if (tid == 0) pref[B] = all;
    __syncthreads();
    units = all;
  }
  const List list{sorted ? order : nullptr, pref, n};
  out->list = list;
  const int items = out->items = units * p.num_kv_heads;
  int active = out->active = (int)gridDim.x;
  Share& sh = out->share;
  sh = Share{};

  // the tiles of the units (and what beginning them costs)
  const int Hkv = p.num_kv_heads;
  const bool may_cut = CUT && units <= kCutUnits && p.max_seq_len <= kCutKeys;
  int before = 0, all = 0;
  int len[2] = {0, 0};
  float row = 0.f;
  if (may_cut) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i)
      if (2 * tid + i < units)
        (i == 0 ? len[0] : len[1]) =
            item_of(p, list, QP, (2 * tid + i) * Hkv, 0, -1).n + kItemTiles;
    const int least = __reduce_min_sync(
        kFull, len[1] > 0 ? min(len[0], len[1]) : len[0] > 0 ? len[0] : INT32_MAX);
    const int most = __reduce_max_sync(kFull, max(len[0], len[1]));
    if (lane == 0) {
      atomicMin(&sums->lightest, least);
      atomicMax(&sums->heaviest, most);
    }
    before = block_scan(len[0] + len[1], sums->scan, &all);
    row = (float)all;
  } else if (p.shared_sms > 0) {
    unsigned long long sum = 0;
    for (int u = tid; u < units; u += kThreads)
      sum += item_of(p, list, QP, u * Hkv, 0, -1).n + kItemTiles;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == 0) atomicAdd(&sums->row, sum);
    __syncthreads();
    row = (float)sums->row;
  }
  if (p.shared_sms > 0) {  // a decode grid works beside: the estimates' shares of the SMs
    const float a = (float)sums->chunks * (float)(kSub * p.num_kv_heads * p.head_dim) *
                    (EIGHT ? 2.f : 4.f) / kDecodeBytesPerCycle;
    const float b = row * (float)Hkv * kTileCycles;
    const int keep = a + b > 0.f ? p.shared_sms - (int)((float)p.shared_sms * a / (a + b) + 0.5f)
                                 : p.shared_sms;
    active = out->active = max(1, min(min(p.shared_sms, (int)gridDim.x), keep));
  }
  // Cut, where the last round of tickets, of which some CTAs get none, costs more than
  // to hand over pieces, about kPieceTiles. (Items that differ fill the rounds better,
  // the light ones last.) 13 requests, 513-key window, 156 items, in a graph: 40.1 us by
  // tickets, 38.2 cut.
  if (!may_cut || units == 0 || (int64_t)all * Hkv >= 1 << 30) return;
  const uint32_t total = (uint32_t)all * Hkv;
  const uint32_t ctas = max(1u, min((uint32_t)min(active, kMaxCtas),
                                    total / (uint32_t)(kItemTiles + kMinShare)));
  const int rounds = (items + active - 1) / active;
  const float light = (float)sums->lightest, ratio = light / (float)sums->heaviest;
  const float idle = ((float)rounds - (float)items / (float)active) * light * ratio * ratio;
  if (idle <= kPieceTiles) return;
  sh.ctas = ctas;
  sh.size = total / ctas;
  sh.more = total - sh.size * ctas;
  if (blockIdx.x >= ctas) return;  // (uniform)
  sh.at = sh.start(blockIdx.x);
  sh.end = sh.start(blockIdx.x + 1);
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const int own = i == 0 ? len[0] : len[1];
    const uint32_t x = sh.at - (uint32_t)before * Hkv;  // (of the unit where the share begins)
    if (sh.at >= (uint32_t)before * Hkv && x < (uint32_t)own * Hkv) {
      sums->start[0] = 2 * tid + i;
      sums->start[1] = x / own;
      sums->start[2] = x % own;
    }
    before += own;
  }
  __syncthreads();
  sh.unit = sums->start[0];
  sh.kvh = sums->start[1];
  sh.in = sums->start[2];
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                      uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// The lowest n bits (none below 0, all from 32 on).
__device__ __forceinline__ uint32_t bits_below(int n) {
  uint32_t r;
  asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(~0u), "r"(max(n, 0)));  // (0 from 32 on)
  return ~r;
}

__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
  float a, b;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(a), "=f"(b)
      : "r"(h));
  return pack_bf16x2(a, b);
}

// 64 rows of a tile, whose boxes were loaded (a bit of `load` each), into the 16-bit
// rows that the products read; 128 threads. Rows not loaded, behind the needed keys or
// hidden from every query ([h0, h1)) become zeros. CH: from one 128-byte chunk of the
// rows to the next.
// bf16 to fp16 in place, in two steps.
template <int D>
constexpr int kBf16Pieces = kHalf * (D / 8) / kConverters;  // of 16 bytes, a thread's
template <int D, int CH>
__device__ __forceinline__ uint32_t bf16_at(uint32_t base, int ct, int e) {
  constexpr int RP = D / 8;  // pieces of a row
  const int pc = ct % RP, k = ct / RP + kConverters / RP * e;
  return base + (pc >> 3) * CH + k * 128 + (((uint32_t)(pc & 7) ^ (uint32_t)(k & 7)) << 4);
}
// First: a thread's pieces of the rows, and the largest magnitude of its warp's, as the
// bits of a bf16.
template <int D, int CH>
__device__ __forceinline__ uint32_t load_bf16(uint32_t base, int ct, uint32_t load, int end, int h0,
                                              int h1, uint4 (&v)[kBf16Pieces<D>]) {
  const bool all =
      end >= kHalf && load == (1u << kHalfBoxes) - 1 && (h0 >= kHalf || h1 <= 0 || h0 >= h1);
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < kBf16Pieces<D>; ++e) v[e] = lds16(bf16_at<D, CH>(base, ct, e));
#pragma unroll
  for (int e = 0; e < kBf16Pieces<D>; ++e) {
    const int k = ct / (D / 8) + kConverters / (D / 8) * e;
    if (!all && !(k < end && ((load >> (k / kSub)) & 1u) && (k < h0 || k >= h1)))
      v[e] = make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("max.u16x2 %0, %0, %1;" : "+r"(top) : "r"(w[j] & 0x7fff7fffu));
  }
  return __reduce_max_sync(kFull, max(top & 0xffffu, top >> 16));
}
// The power of two that the rows are multiplied by, its exponent + 127: brings their
// largest magnitude into [2^14, 2^15) (within [2^-113, 2^64]; rows of zeros: 2^64), which
// leaves values exact down to 2^-17, 2^-31 of the largest.
__device__ __forceinline__ uint32_t bf16_power(uint32_t top) {
  return min(max(14 + 127 + 127 - (int)(top >> 7), 127 - 113), 127 + 64);
}
// Second: the pieces times that power, as fp16.
template <int D, int CH>
__device__ __forceinline__ void store_bf16(uint32_t base, int ct, uint32_t power,
                                           const uint4 (&v)[kBf16Pieces<D>]) {
  const uint32_t times = power << 7 | power << 23;  // as bf16, twice
#pragma unroll
  for (int e = 0; e < kBf16Pieces<D>; ++e) {
    uint32_t w[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(w[j]) : "r"(times));
      w[j] = pack_f16x2(bf16_lo(w[j]), bf16_hi(w[j]));
    }
    sts16(bf16_at<D, CH>(base, ct, e), w[0], w[1], w[2], w[3]);
  }
}
// e4m3 in place: box b landed at 2048 b bytes, its rows D bytes apart, swizzled by
// their length, so that a box lies where the same warp writes its 16 rows: it reads
// them, then writes them. To bf16 (BF) or fp16.
template <int D, bool BF, int CH>
__device__ __forceinline__ void convert_e4m3(uint32_t base, int ct, uint32_t load, int end, int h0,
                                             int h1) {
  constexpr int NP = D / 16;   // 16-byte pieces of a row
  constexpr int N = NP / 2;    // pieces of a thread: 16 rows of them, 32 lanes
  const int box = ct >> 5, lane = ct & 31;
  uint4 w[N];
  // piece e of a lane: 8 lanes take one piece of 8 rows (different bank groups)
  auto row = [&](int e) { return (lane & 7) + 8 * (e & 1); };
  auto part = [&](int e) { return (lane >> 3) + 4 * (e >> 1); };
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int r = row(e), k = box * kSub + r, pc = part(e);
    const uint32_t at = base + box * 2048 + r * D +
                        ((pc ^ (D == 128 ? (r & 7) : ((r >> 1) & 3))) << 4);
    w[e] = make_uint4(0u, 0u, 0u, 0u);
    if (k < end && ((load >> box) & 1u) && (k < h0 || k >= h1)) w[e] = lds16(at);
  }
  __syncwarp();
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int r = row(e), pc = part(e);
    uint32_t x[8] = {e4m3_lo(w[e].x), e4m3_hi(w[e].x), e4m3_lo(w[e].y), e4m3_hi(w[e].y),
                     e4m3_lo(w[e].z), e4m3_hi(w[e].z), e4m3_lo(w[e].w), e4m3_hi(w[e].w)};
    if (BF)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = f16x2_to_bf16x2(x[i]);
    const uint32_t to = base + (pc >> 2) * CH + box * 2048 + r * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      sts16(to + ((((pc & 3) * 2 + h) ^ (r & 7)) << 4), x[4 * h], x[4 * h + 1], x[4 * h + 2],
            x[4 * h + 3]);
  }
}

// Zeros into the boxes of a K stage (a bit of `boxes` each), by a warp.
template <int NCH, int CH>
__device__ __noinline__ void clear_boxes(uint32_t stage, uint32_t boxes) {
#pragma unroll 1
  for (int b = 0; b < kBoxes; ++b)
    if ((boxes >> b) & 1u)
#pragma unroll 1
      for (int e = threadIdx.x & 31; e < NCH * kSub * 8; e += 32)
        st_shared_zero16(stage + b * kSub * 128 + e / (kSub * 8) * CH + e % (kSub * 8) * 16);
  fence_proxy_async_smem();
  __syncwarp();
}

// A warp's part of a piece: O, 4 dimensions of its 32 rows after the other, then m and l.
template <int D>
constexpr int kWarpFloats = 32 * (D + 2);

// 32 values of a row of the output from dimension c on.
template <int D>
__device__ __forceinline__ void put32(const AttnParams& p, int64_t row, int c,
                                      const float (&v)[32]) {
  if (p.out_bf16) {
    uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + row * D + c;
#pragma unroll
    for (int e = 0; e < 32; e += 8)
      *reinterpret_cast<uint4*>(out + e) =
          make_uint4(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]),
                     pack_bf16x2(v[e + 4], v[e + 5]), pack_bf16x2(v[e + 6], v[e + 7]));
  } else {
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      *reinterpret_cast<float4*>(p.out + row * D + c + e) =
          make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  }
}

// The part of warp `warp` of a CTA's piece of an item, of the one that it begins or of
// the one that it continues.
template <int D>
__device__ __forceinline__ float* part_of(const AttnParams& p, int cta, bool begins, int warp) {
  return p.prefill_parts + ((int64_t)(2 * cta + (begins ? 1 : 0)) * 8 + warp) * kWarpFloats<D>;
}

// Dimensions [c0, c0 + N) of a warp's rows from the item's `pieces`, the first of them
// CTA `head`'s, in their order.
template <int D, int N>
__device__ __forceinline__ void join_rows(const AttnParams& p, int head, int pieces, int warp,
                                          int c0, bool valid, int64_t row) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f;
#pragma unroll 4
  for (int i = 0; i < pieces; ++i) {
    const float* from = part_of<D>(p, head + i, i == 0, warp) + 32 * D + lane;
    const float mi = __ldcg(from), li = __ldcg(from + 32);
    const float mn = fmaxf(m, mi), mu = mn == -INFINITY ? 0.f : mn;
    l = fmaf(l, fast_exp2(m - mu), li * fast_exp2(mi - mu));
    m = mn;
  }
  const float mu = m == -INFINITY ? 0.f : m, inv = 1.f / l;
#pragma unroll 1
  for (int c = c0; c < c0 + N; c += 32) {
    float v[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = 0.f;
#pragma unroll 2
    for (int i = 0; i < pieces; ++i) {
      const float* from = part_of<D>(p, head + i, i == 0, warp);
      const float w = fast_exp2(__ldcg(from + 32 * D + lane) - mu) * inv;
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        const float4 o = __ldcg(reinterpret_cast<const float4*>(from) + (c + e) / 4 * 32 + lane);
        v[e] = fmaf(o.x, w, v[e]);
        v[e + 1] = fmaf(o.y, w, v[e + 1]);
        v[e + 2] = fmaf(o.z, w, v[e + 2]);
        v[e + 3] = fmaf(o.w, w, v[e + 3]);
      }
    }
    if (valid) put32<D>(p, row, c, v);
  }
  if (c0 == 0 && valid && p.out_lse) p.out_lse[row] = (m + fast_log2(l)) * kLn2;
}

template <int R>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// The roles of the warps. CUT: items may be cut, their pieces' places are read with them.
template <int D, bool EIGHT, bool CUT>
__device__ __forceinline__ void work_on(const CUtensorMap& q_map, const CUtensorMap& kv_map,
                                        const AttnParams& p, uint8_t* smem, const List& list,
                                        Share& share, int total, uint32_t tmem) {
  using Lay = Layout<D>;
  Bars* bars = reinterpret_cast<Bars*>(smem + Lay::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.num_heads / p.num_kv_heads, QT = kBM / G, QP = 2 * QT;
  volatile int32_t* abort = &bars->abort;
  const uint32_t q_s = smem_addr(smem + Lay::Q_OFF);
  const uint32_t k_s = smem_addr(smem + Lay::K_OFF);
  const uint32_t v_s = smem_addr(smem + Lay::V_OFF);
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return short_wait(smem_addr(bar), parity, p.status, abort);
  };
  // a warp's wait, by every lane; by one lane
  auto all_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(kFull, wait(bar, parity)) != 0;
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    int w = 1;
    if (lane == 0) w = wait(bar, parity);
    return __shfl_sync(kFull, w, 0) != 0;
  };
  auto next_item = [&](int k) {
    Piece c;
    if (lane == 0) c = read_item(bars, p, k, abort);
    return all_lanes<CUT>(c);
  };

  if (warp >= kConvWarp0) {
    fewer_registers<kOtherRegs>();
    if (warp == kKWarp || warp == kVWarp) {
      // ===== copies of K (and the tickets); of Q and V =====
      const bool vrole = warp == kVWarp;
      const int32_t first_row = vrole ? p.num_blocks * p.block_size : 0;
      const uint32_t ring = vrole ? v_s : k_s;
      uint64_t* empty = vrole ? bars->v_empty : bars->k_empty;
      uint64_t* landed = vrole ? bars->v_landed : EIGHT ? bars->k_landed : bars->k_full;
      uint32_t* mask = vrole ? bars->v_mask : bars->k_mask;
      // a stage: a tile of K, half a tile of V
      const int boxes = vrole ? kHalfBoxes : kBoxes, stages = vrole ? kVS : kNS;
      const uint32_t stage_bytes = vrole ? Lay::VS_BYTES : Lay::TILE_BYTES;
      const uint32_t chunk_bytes = vrole ? Lay::VCH_BYTES : Lay::CH_BYTES;
      if (lane == 0) prefetch_tmap(vrole ? &q_map : &kv_map);
      int st = 0, filled = 0, copied = 0;
      uint32_t parity = 1;  // of the stage's last release (none before the first lap)
      bool ok = true, bad_block = false;
      // both tiles of Q. Rows behind the last token read as zeros, rows of the next
      // request belong to no valid output row
      auto copy_q = [&](int k, const Item& d) {
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          if (k > 0) ok = warp_wait(&bars->q_empty[x], (k - 1) & 1);
          if (!ok) break;
          ++copied;
          if (lane == 0) {
            mbar_arrive_expect_tx(smem_addr(&bars->q_full[x]), Lay::NCH * QT * G * 128);
#pragma unroll 1
            for (int c = 0; c < Lay::NCH; ++c)
              tma_load_3d(q_s + x * Lay::TILE_BYTES + c * Lay::CH_BYTES, &q_map,
                          smem_addr(&bars->q_full[x]), c * 64, d.kvh * G, d.t0 + d.j0 + x * QT);
          }
        }
      };
      for (int k = 0; ok; ++k) {
        Piece c;
        if (lane == 0)
          c = vrole ? read_item(bars, p, k, abort)
                    : take_item<CUT>(bars, p, list, QP, total, share, k, abort);
        c = all_lanes<CUT>(c);
        if (c.id < 0) break;
        const Item d = item_of(p, list, QP, c.id, c.first, c.n);
        const int32_t* bt = p.block_table + (int64_t)d.req * p.max_blocks;
        int32_t row = -1;
        if (vrole && k == 0) copy_q(k, d);
#pragma unroll 1
        for (int box0 = 0; box0 < d.n * kHalfBoxes; box0 += boxes) {
          if ((box0 & 31) == 0) {  // the next 32 boxes, one a lane: first row in the pool
            const int box = box0 + lane;
            row = -1;
            if (box < d.count) {
              const int key = d.key(box * kSub);
              const int32_t id = __ldg(bt + key / p.block_size);
              if (id >= 0 && id < p.num_blocks) {
                row = first_row + id * p.block_size + key % p.block_size;
              } else {
                row = kBadRow;
                bad_block = true;
              }
            }
          }
          if (filled >= stages) ok = warp_wait(&empty[st], parity);
          if (!ok) break;
          // keys of a bad block count as zeros (the converters see to the other rows)
          if (!EIGHT && !vrole && __any_sync(kFull, bad_block))
            clear_boxes<Lay::NCH, Lay::CH_BYTES>(
                ring + st * stage_bytes, __ballot_sync(kFull, row == kBadRow) >> (box0 & 31));
          const uint32_t load =
              (__ballot_sync(kFull, row >= 0) >> (box0 & 31)) & ((1u << boxes) - 1);
          if (lane == 0) {
            *reinterpret_cast<volatile uint32_t*>(&mask[st]) = load;
            mbar_arrive_expect_tx(smem_addr(&landed[st]),
                                  __popc(load) * (EIGHT ? kSub * D : Lay::NCH * kSub * 128));
          }
          // a lane a copy: one after the other by one lane they take long enough for
          // the stages to run dry
          const int b = lane & (boxes - 1), c = lane / boxes;
          const int32_t r = __shfl_sync(kFull, row, (box0 & 31) + b);
          if (r >= 0 && c < (EIGHT ? 1 : Lay::NCH)) {
            const uint32_t at = ring + st * stage_bytes + b * kSub * 128 + c * chunk_bytes;
            if (EIGHT)
              tma_load_3d(at, &kv_map, smem_addr(&landed[st]), 0, r, d.kvh);
            else
              tma_load_4d(at, &kv_map, smem_addr(&landed[st]), 0, r, d.kvh, c);
          }
          __syncwarp();
          ++filled;
          st = st + 1 == stages ? 0 : st + 1;
          parity ^= st == 0 ? 1u : 0u;
          // behind the item's first two V tiles (whose stages are free by then): Q, free
          // when the last scores of the item before are there
          if (vrole && k > 0 && box0 == min(1, d.n - 1) * kHalfBoxes) copy_q(k, d);
          if (!ok) break;
        }
      }
      if (bad_block) set_status(p.status, PKV_DEV_BAD_BLOCK);
      // our copies, and the arrivals that they trigger, land before the CTA can exit
      if (lane == 0) {
        for (int x = 0; x < 2; ++x)  // copies of Q: A's of items 0, 1 .., B's
          if (copied > x)
            short_wait(smem_addr(&bars->q_full[x]), ((copied - x + 1) / 2 - 1) & 1, nullptr);
        for (int g = max(0, filled - stages); g < filled; ++g)
          short_wait(smem_addr(&landed[g % stages]), (g / stages) & 1, nullptr);
      }
    } else if (warp < kMmaWarp) {
      // ===== converters =====
      const int ct = threadIdx.x - kConvWarp0 * 32;
      uint32_t most = 0;  // of V
      int gt = 0, vt = 0, vst = 0;
      uint32_t vparity = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const Piece c = next_item(k);
        if (c.id < 0) break;
        const Item d = item_of(p, list, QP, c.id, c.first, c.n);
#pragma unroll 1
        for (int j = 0; ok && j < d.n; ++j) {
          const int c0 = j * kHalf;
          if (EIGHT && (j & 1) == 0) {
            const int st = gt % kNS;
            ok = warp_wait(&bars->k_landed[st], (gt / kNS) & 1);
            if (!ok) break;
            const uint32_t load = *reinterpret_cast<volatile uint32_t*>(&bars->k_mask[st]);
#pragma unroll 1
            for (int h = 0; h < 2; ++h)
              convert_e4m3<D, true, Lay::CH_BYTES>(
                  k_s + st * Lay::TILE_BYTES + h * kHalf * 128, ct, load >> (h * kHalfBoxes),
                  d.end - c0 - h * kHalf, d.sink - c0 - h * kHalf, d.lo_any - c0 - h * kHalf);
            fence_proxy_async_smem();
            mbar_arrive(smem_addr(&bars->k_full[st]));
            ++gt;
          }
          ok = warp_wait(&bars->v_landed[vst], vparity);
          if (!ok) break;
          const uint32_t load = *reinterpret_cast<volatile uint32_t*>(&bars->v_mask[vst]);
          const uint32_t base = v_s + vst * Lay::VS_BYTES;
          if (EIGHT)
            convert_e4m3<D, false, Lay::VCH_BYTES>(base, ct, load, d.end - c0, d.sink - c0,
                                                   d.lo_any - c0);
          else {
            uint4 v[kBf16Pieces<D>];
            uint32_t top = load_bf16<D, Lay::VCH_BYTES>(base, ct, load, d.end - c0, d.sink - c0,
                                                        d.lo_any - c0, v);
            volatile uint32_t* tops = bars->v_top[vt & 1];
            if (lane == 0) {
              tops[ct >> 5] = top;
              mbar_arrive(smem_addr(&bars->v_sized));
            }
            ok = all_wait(&bars->v_sized, vt & 1);
            if (!ok) break;
            ++vt;
#pragma unroll
            for (int w = 0; w < kConverters / 32; ++w) top = max(top, tops[w]);
            most = max(most, top);
            const uint32_t power = bf16_power(top);
            store_bf16<D, Lay::VCH_BYTES>(base, ct, power, v);
            if (ct == 0) {
              volatile float2* scale = &bars->v_scale[vst];
              scale->x = 127.f - (float)power;
              scale->y = __uint_as_float(power << 23);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(smem_addr(&bars->v_full[vst]));
          vst = vst + 1 == kVS ? 0 : vst + 1;
          vparity ^= vst == 0 ? 1u : 0u;
        }
      }
      if (most >= 0x7f80u && ct == 0) set_status(p.status, PKV_DEV_V_RANGE);  // inf, NaN
    } else {
      // ===== the products of query tile x: the warp waits, one lane issues =====
      const int x = warp - kMmaWarp;
      constexpr uint32_t idesc_qk = umma_idesc_bf16(kBM, kHalf, false, false);
      constexpr uint32_t idesc_pv = umma_idesc_f16(kBM, D, false, true);
      const uint64_t qd = smem_desc_sw128(q_s + x * Lay::TILE_BYTES, 16, 1024);
      const uint64_t kd = smem_desc_sw128(k_s, 16, 1024);
      const uint64_t vd = smem_desc_sw128(v_s, Lay::VCH_BYTES, 1024);
      constexpr uint32_t kTile16 = Lay::TILE_BYTES >> 4;
      static_assert(kNS == 2, "two stages");
      const uint32_t s_tm = tmem + Lay::s_col(x), o_tm = tmem + Lay::o_col(x);
      // S(g) of the tile in half h of K stage kt, and what follows it
      auto issue_qk = [&](int g, int kt, int h, bool release, bool last) {
        const uint64_t k = kd + (kt & 1) * kTile16 + h * (uint32_t)((kHalf * 128) >> 4);
        const uint32_t s = s_tm + (uint32_t)((g & 1) * kHalf);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = ((i >> 2) * Lay::CH_BYTES + (i & 3) * 32) >> 4;
            umma_ss(s, qd + off, k + off, idesc_qk, i > 0);
          }
          umma_commit(smem_addr(&bars->s_full[x][g & 1]));
          if (release) umma_commit(smem_addr(&bars->k_empty[kt % kNS]));
          if (last) umma_commit(smem_addr(&bars->q_empty[x]));  // Q is read no more
        }
        __syncwarp();
      };
      int g = 0, kt = 0, vst = 0;  // score tiles, K stages, V stage so far
      uint32_t vparity = 0;
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        const Piece c = next_item(k);
        if (c.id < 0) break;
        const int n = item_of(p, list, QP, c.id, c.first, c.n).n;
        ok = all_wait(&bars->q_full[x], k & 1);
        // tile j's product with P behind tile j + 2's scores' issue, from j = -2 on
#pragma unroll 1
        for (int j = -2; ok && j < n; ++j) {
          if (j >= 0) {
            ok = all_wait(&bars->v_full[vst], vparity) &&
                 all_wait(&bars->p_ready[x][g & 1], (g >> 1) & 1) &&
                 (j > 0 || k == 0 || all_wait(&bars->o_free[x], (k - 1) & 1));
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = vd + vst * (uint32_t)(Lay::VS_BYTES >> 4);
            const uint32_t pt = s_tm + (uint32_t)((g & 1) * kHalf);
            if (elect_one()) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                umma_ts(o_tm, pt + 8u * i, v + (uint32_t)((i * 16 * 128) >> 4), idesc_pv,
                        j > 0 || i > 0);
              umma_commit(smem_addr(&bars->o_done[x][g & 1]));
              umma_commit(smem_addr(&bars->v_empty[vst]));
            }
            __syncwarp();
            vst = vst + 1 == kVS ? 0 : vst + 1;
            vparity ^= vst == 0 ? 1u : 0u;
            ++g;
          }
          const int j2 = j + 2;
          if (j2 >= n) continue;
          const int kt2 = kt + (j2 >> 1);
          ok = (j2 & 1) || all_wait(&bars->k_full[kt2 % kNS], (kt2 / kNS) & 1);
          if (!ok) break;
          // (before the loop's first product g counts no tile of this item yet)
          issue_qk(j >= 0 ? g + 1 : g + j2, kt2, j2 & 1, (j2 & 1) || j2 == n - 1, j2 == n - 1);
        }
        kt += (n + 1) >> 1;
      }
      // every product has completed before tensor memory is released (one lane issued them)
      if (elect_one()) umma_commit(smem_addr(&bars->mma_done));
      __syncwarp();
      short_wait(smem_addr(&bars->mma_done), 0, nullptr);
    }
  } else {
    more_registers<kSoftmaxRegs>();
    // ===== softmax and output: warpgroup x owns query tile x, thread r its row r =====
    const int x = warp >> 2, r = threadIdx.x & (kBM - 1);
    const int rq = r / G, g = r % G;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sa0 = tmem + lanes + Lay::s_col(x), oa = tmem + lanes + Lay::o_col(x);
    const float sl2 = p.scale_log2;
    bool ok = true;
    int gt = 0, vst = 0;
    uint32_t vparity = 0;
    float2 vs = make_float2(0.f, 1.f);  // bf16: the V stage's scale, which the weights take up
    auto score_col = [&](int g) { return sa0 + (uint32_t)((g & 1) * kHalf); };
    auto load_scores = [&](int g, uint32_t (&u)[kHalf]) {
      bool there = wait(&bars->s_full[x][g & 1], (g >> 1) & 1);
      if (!EIGHT) {
        there = there && wait(&bars->v_full[vst], vparity);
        const volatile float2* scale = &bars->v_scale[vst];
        vs.x = scale->x;
        vs.y = scale->y;
        vst = vst + 1 == kVS ? 0 : vst + 1;
        vparity ^= vst == 0 ? 1u : 0u;
      }
      there = __all_sync(kFull, there) != 0;  // (all waits before the loads are under way)
      tc_fence_after();
      if (there) {
        PKV_TMEM_LD32(score_col(g), u);
        PKV_TMEM_LD32(score_col(g) + 32, (u + 32));
        tmem_wait_ld();
      }
      return there;
    };
    for (int k = 0; ok; ++k) {
      const Piece piece = next_item(k);
      if (piece.id < 0) break;
      const Item d = item_of(p, list, QP, piece.id, piece.first, piece.n);
      // (head, pieces, whether it begins the item: in a word over the loop)
      const int cut = piece.head | piece.pieces << 8 | (piece.first == 0 ? 1 << 16 : 0);
      const int qj = d.j0 + x * QT + rq;
      const bool valid = qj < d.j1 && rq < QT;
      // the columns [low, lim] and those before d.sink are visible to the row
      const int lim0 = valid ? d.qpos0 + qj - d.shift : d.end - 1;
      const int low0 = lim0 - p.window + 1;
      float m = -INFINITY, l = 0.f;
      // 8 bits: lane i holds the block id and the scales of the item's 16-key chunk
      // 32 b + i: the scores' factor, log2 of the values' scale, one over it
      auto chunk_id = [&](int box) -> int32_t {
        if (box >= d.count) return -1;
        const int32_t id = __ldg(p.block_table + (int64_t)d.req * p.max_blocks +
                                 d.key(box * kSub) / p.block_size);
        return id < p.num_blocks ? id : -1;
      };
      float sc_a = 0.f, sc_l = 0.f, sc_i = 1.f, nx_a = 0.f, nx_l = 0.f, nx_i = 1.f;
      int32_t nx_id = -1;
      auto chunk_scales = [&](int32_t id) {
        nx_a = nx_i = 1.f;
        nx_l = 0.f;
        if (id >= 0) {
          // (never 0: a hidden score's -inf times it would be NaN)
          nx_a = fmaxf(__ldg(p.scales + (int64_t)id * p.num_kv_heads + d.kvh) * sl2, FLT_MIN);
          // (a scale below 2^-100 as that: its values are nothing beside any other)
          const float v = fmaxf(
              __ldg(p.scales + ((int64_t)p.num_blocks + id) * p.num_kv_heads + d.kvh),
              7.888609e-31f);
          nx_l = fast_log2(v);
          nx_i = 1.f / v;
        }
      };
      if (EIGHT) chunk_scales(chunk_id(lane));
      // the columns [all0, all1] are visible to every row of the warp
      const int all0 = __reduce_max_sync(kFull, low0 <= d.sink ? 0 : low0);
      const int all1 = __reduce_min_sync(kFull, lim0);
      uint32_t u[kHalf];
      ok = load_scores(gt, u);
      if (!ok) break;
#pragma unroll 1
      for (int j = 0; j < d.n; ++j, ++gt) {
        if (EIGHT) {  // in time for the next 8 tiles
          if ((j & 7) == 0) {
            sc_a = nx_a;
            sc_l = nx_l;
            sc_i = nx_i;
            nx_id = chunk_id((j + 8) * kHalfBoxes + lane);
          } else if ((j & 7) == 4) {
            chunk_scales(nx_id);
          }
        }
        const int lim = lim0 - j * kHalf, low = low0 - j * kHalf, sink = d.sink - j * kHalf;
        // hidden scores become -inf
        if (j * kHalf < all0 || j * kHalf + kHalf - 1 > all1) {
#pragma unroll
          for (int c0 = 0; c0 < kHalf; c0 += 32) {
            const uint32_t seen =
                bits_below(lim + 1 - c0) & (~bits_below(low - c0) | bits_below(sink - c0));
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(seen & (1u << c))) u[c0 + c] = kMinusInf;
          }
        }
        // the row's maximum, in log2 units
        float mx, fa[kHalfBoxes], fl[kHalfBoxes];
        const int from = (j & 7) * kHalfBoxes;  // the lane of the tile's first chunk
        if (EIGHT) {
          mx = -INFINITY;
#pragma unroll
          for (int q = 0; q < kHalfBoxes; ++q) {
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int c = 16 * q; c < 16 * q + 16; c += 4) {
              a = max3(a, __uint_as_float(u[c]), __uint_as_float(u[c + 1]));
              b = max3(b, __uint_as_float(u[c + 2]), __uint_as_float(u[c + 3]));
            }
            fa[q] = __shfl_sync(kFull, sc_a, from + q);
            fl[q] = __shfl_sync(kFull, sc_l, from + q);
            mx = fmaxf(mx, fmaf(fmaxf(a, b), fa[q], fl[q]));
          }
        } else {
          float a = -INFINITY, b = -INFINITY;
#pragma unroll
          for (int c = 0; c < kHalf; c += 4) {
            a = max3(a, __uint_as_float(u[c]), __uint_as_float(u[c + 1]));
            b = max3(b, __uint_as_float(u[c + 2]), __uint_as_float(u[c + 3]));
          }
          mx = fmaf(fmaxf(a, b), sl2, vs.x);
        }
        const float mnew = fmaxf(m, mx);
        const bool grow = mnew > m + kRescaleThreshold;
        if (__any_sync(kFull, grow)) {
          const float alpha = grow ? fast_exp2(m - mnew) : 1.f;  // 0 while m is -inf
          if (grow) m = mnew;
          l *= alpha;
          if (j > 0) {  // O once the product before has written it
            ok = all_wait(&bars->o_done[x][(gt - 1) & 1], ((gt - 1) >> 1) & 1);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t v[32];
              PKV_TMEM_LD32(oa + c, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
              PKV_TMEM_ST32(oa + c, v);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : m;
        // weights: the sum takes them before they are rounded to fp16
        float2 sum = make_float2(0.f, 0.f);
        float sum8 = 0.f;
        const float voff = vs.x - mu;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t pk[16];
          if (EIGHT) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int box = 2 * b + q;
              const float off = fl[box] - mu;
              const float fi = __shfl_sync(kFull, sc_i, from + box);
              float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const uint32_t ua = u[16 * box + 2 * c], ub = u[16 * box + 2 * c + 1];
                const float2 y = __ffma2_rn(
                    make_float2(__uint_as_float(ua), __uint_as_float(ub)), make_float2(fa[box], fa[box]),
                    make_float2(off, off));
                const float2 w = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                pk[8 * q + c] = pack_f16x2(w.x, w.y);
                s2 = __fadd2_rn(s2, w);
              }
              sum8 = fmaf(s2.x + s2.y, fi, sum8);
            }
          } else {
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const int e = 32 * b + 2 * c;
              const float2 y = __ffma2_rn(
                  make_float2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])),
                  make_float2(sl2, sl2), make_float2(voff, voff));
              const float2 w = make_float2(fast_exp2(y.x), fast_exp2(y.y));
              pk[c] = pack_f16x2(w.x, w.y);
              sum = __fadd2_rn(sum, w);
            }
          }
          PKV_TMEM_ST16(score_col(gt) + 16 * b, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars->p_ready[x][gt & 1]));
        l = EIGHT ? l + sum8 : fmaf(sum.x + sum.y, vs.y, l);
        // (at the loop's end: 8-bit chunks of 2048 tokens 353 us, 359 at its start)
        if (j + 1 < d.n) ok = load_scores(gt + 1, u);
        if (!ok) break;
      }
      if (!ok) break;
      // ---- the item's rows: O / l, lse
      ok = all_wait(&bars->o_done[x][(gt - 1) & 1], ((gt - 1) >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      const int64_t orow = (int64_t)(d.t0 + qj) * p.num_heads + d.kvh * G + g;
      const int head = cut & 255, pieces = cut >> 8 & 255;
      const bool whole = pieces == 1, begins = cut >> 16;
      if (whole) {
        const float inv = 1.f / l;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          PKV_TMEM_LD32(oa + c, o);
          tmem_wait_ld();
          if (!valid) continue;
          float v[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(o[e]) * inv;
          put32<D>(p, orow, c, v);
        }
        if (valid && p.out_lse) p.out_lse[orow] = (m + fast_log2(l)) * kLn2;
      } else {  // a piece of an item goes to the workspace as it is, with m and l
        float* part = part_of<D>(p, (int)blockIdx.x, begins, warp);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          PKV_TMEM_LD32(oa + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            reinterpret_cast<uint4*>(part)[(c + e) / 4 * 32 + lane] =
                make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        }
        part[32 * D + lane] = m;
        part[32 * D + 32 + lane] = l;
        if (p.prefill_join && begins && threadIdx.x == 0)
          reinterpret_cast<int4*>(p.sched + kRecords)[blockIdx.x] =
              make_int4(d.t0 + d.j0, d.j1 - d.j0, d.kvh, pieces);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&bars->o_free[x]));
      if (whole || p.prefill_join) continue;
      // the warp that comes last joins the pieces
      __threadfence();
      __syncwarp();
      int done = 0;
      if (lane == 0) done = atomicAdd(p.sched + kRecords + head * 8 + warp, 1) + 1;
      if (__shfl_sync(kFull, done, 0) != pieces) continue;
      __threadfence();
      join_rows<D, D>(p, head, pieces, warp, 0, valid, orow);
    }
  }
}

template <int D, bool EIGHT, bool CUT>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_rows_kernel(const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap kv_map, const AttnParams p) {
  using Lay = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + Lay::BAR_OFF);
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int G = p.num_heads / p.num_kv_heads;
  const int QT = kBM / G;  // queries of a tile (rows G QT .. 127 belong to none)
  const int QP = 2 * QT;   // queries of an item

  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_addr(&bars->q_full[x]), 1);
      mbar_init(smem_addr(&bars->q_empty[x]), 1);
      for (int b = 0; b < 2; ++b) {
        mbar_init(smem_addr(&bars->s_full[x][b]), 1);
        mbar_init(smem_addr(&bars->p_ready[x][b]), 4);
        mbar_init(smem_addr(&bars->o_done[x][b]), 1);
      }
      mbar_init(smem_addr(&bars->o_free[x]), 4);
    }
    for (int s = 0; s < kNS; ++s) {
      mbar_init(smem_addr(&bars->k_landed[s]), 1);
      mbar_init(smem_addr(&bars->k_full[s]), EIGHT ? kConverters : 1);
      mbar_init(smem_addr(&bars->k_empty[s]), 2);
    }
    for (int s = 0; s < kVS; ++s) {
      mbar_init(smem_addr(&bars->v_landed[s]), 1);
      mbar_init(smem_addr(&bars->v_full[s]), kConverters);
      mbar_init(smem_addr(&bars->v_empty[s]), 2);
    }
    mbar_init(smem_addr(&bars->mma_done), 2);
    mbar_init(smem_addr(&bars->v_sized), kConverters / 32);
    for (int k = 0; k < kRing; ++k) {
      mbar_init(smem_addr(&bars->item_full[k]), 1);
      mbar_init(smem_addr(&bars->item_empty[k]), kItemReaders);
    }
    bars->abort = 0;
    fence_barrier_init();
  }
  Work work;
  plan_work<EIGHT, CUT>(p, QP, reinterpret_cast<int*>(smem + Lay::LIST_OFF), &bars->sums,
                   &work);  // (synchronises)
  const List list = work.list;
  const int total = work.items;
  Share share = work.share;
  // (uniform; nothing allocated yet)
  if ((int)blockIdx.x >= (share.ctas > 0 ? (int)share.ctas : min(total, work.active))) return;
  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&bars->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  work_on<D, EIGHT, CUT>(q_map, kv_map, p, smem, list, share, total, tmem);

  // ---- the CTA's tcgen05 work is complete: tensor memory is released (its address
  // read again: the roles ran with different register budgets)
  tc_fence_before();
  __syncthreads();
  if ((threadIdx.x >> 5) == kMmaWarp) {
    const Bars* b = reinterpret_cast<const Bars*>(
        ((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023)) +
        Lay::BAR_OFF);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(*reinterpret_cast<const volatile uint32_t*>(&b->tmem_base), kTmemCols);
  }
}

// The items that were cut: CTA (h, x, c) joins 32 dimensions of query tile x of the one
// that begins in CTA h's share, a row a thread.
template <int D>
__global__ void __launch_bounds__(kBM) join_pieces_kernel(const AttnParams p) {
  griddep_wait();  // (no early trigger: as in join_rows_kernel)
  const int4 rec = __ldcg(reinterpret_cast<const int4*>(p.sched + kRecords) + blockIdx.x);
  if (rec.w < 2) return;
  const int x = blockIdx.y, r = threadIdx.x;
  const int G = p.num_heads / p.num_kv_heads, QT = kBM / G;
  const int j = x * QT + r / G;
  const bool valid = r < QT * G && j < rec.y;
  join_rows<D, 32>(p, blockIdx.x, rec.w, x * 4 + (r >> 5), blockIdx.z * 32, valid,
                   (int64_t)(rec.x + j) * p.num_heads + rec.z * G + r % G);
}

template <int D, bool EIGHT, bool CUT>
cudaError_t launch_form(const AttnParams& p, const CUtensorMap& q_map, const CUtensorMap& kv_map,
                     cudaStream_t stream) {
  const size_t smem = Layout<D>::bytes(p.num_seqs);
  if (smem > 227 * 1024) return cudaErrorInvalidValue;
  auto kernel = prefill_rows_kernel<D, EIGHT, CUT>;
  static SmemLimit limit;
  if (cudaError_t e = limit.ensure(reinterpret_cast<const void*>(kernel), 227 * 1024);
      e != cudaSuccess)
    return e;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, q_map, kv_map, p);
}

// Items are cut in calls of up to three rounds of them (the places of the pieces cost
// the loops something: 8 bits, chunks of 2048 tokens, 496 items, 354 us, 365 in the form
// that may cut).
template <int D, bool EIGHT>
cudaError_t launch_d(const AttnParams& p, const CUtensorMap& q_map, const CUtensorMap& kv_map,
                     cudaStream_t stream) {
  const int QP = 2 * (kBM / (p.num_heads / p.num_kv_heads));
  // (items at least, those of requests that the decode grid may take left out)
  const int64_t items =
      ((int64_t)p.num_tokens - (int64_t)p.num_seqs * p.decode_max_q) / QP * p.num_kv_heads;
  return items <= 3 * kMaxCtas ? launch_form<D, EIGHT, true>(p, q_map, kv_map, stream)
                               : launch_form<D, EIGHT, false>(p, q_map, kv_map, stream);
}

}  // namespace

bool prefill_rows_fits(int32_t num_seqs, int32_t head_dim) {
  return num_seqs >= 0 && (head_dim == 128 ? Layout<128>::bytes(num_seqs)
                                           : Layout<64>::bytes(num_seqs)) <= 227 * 1024;
}

size_t prefill_rows_sched() { return (kRecords + 8 * kMaxCtas) * sizeof(int32_t); }

size_t prefill_rows_workspace(int32_t head_dim) {
  return (size_t)kMaxCtas * 2 * 8 * 32 * (head_dim + 2) * sizeof(float);
}

cudaError_t launch_prefill_rows(const AttnParams& p, const CUtensorMap& q_map,
                                const CUtensorMap& kv_map, cudaStream_t stream) {
  if (p.scales)
    return p.head_dim == 128 ? launch_d<128, true>(p, q_map, kv_map, stream)
                             : launch_d<64, true>(p, q_map, kv_map, stream);
  return p.head_dim == 128 ? launch_d<128, false>(p, q_map, kv_map, stream)
                           : launch_d<64, false>(p, q_map, kv_map, stream);
}

bool prefill_rows_join(const AttnParams& p) {
  const int QP = 2 * (kBM / (p.num_heads / p.num_kv_heads));
  const int64_t units = (int64_t)p.num_tokens / QP + p.num_seqs;  // at most
  return units * p.num_kv_heads * 4 <= kMaxCtas;
}

cudaError_t launch_prefill_rows_join(const AttnParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)kMaxCtas, 2, (unsigned)(p.head_dim / 32));
  cfg.blockDim = dim3(kBM);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, p.head_dim == 128 ? join_pieces_kernel<128> : join_pieces_kernel<64>,
                            p);
}

}  // namespace pkv
