// decode_rows.cu -- paged attention for requests of up to 32 (query, head) rows
// (decodes, short verification steps) through a window, over a bf16 pool or over
// one held in 8 bits (e4m3, a scale for each block and KV head).
//
//   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j), j the keys that the
//   query sees;  8 bits: k_j = a_b K_j, v_j = c_b V_j with K_j, V_j the e4m3 values
//   and a_b, c_b the scales of the key's block b.
//
// Neither scale is multiplied into the values: a_b joins the factor of the score
// (fp32), and the weights are formed as c_b w_j = 2^(s_j + log2 c_b - m), whose
// running maximum m is over the scaled weights. What is multiplied with V_j is
// thus at most 2^8 whatever the scales, and a weight that fp16 would flush to zero
// adds less than 2^-24 of the largest to the output. The sum of the weights takes
// them in fp32, divided by c_b.
//
// Bound: HBM, 2 D values a key and KV head. At 8 bits that leaves half of the time
// a key that the bf16 cache leaves, so that the products have to be cheap:
//   * the keys are the rows of the products, S^T = K Q^T (m16n8k16) and
//     O^T = V^T P^T, with the group's heads as the columns: 8 columns waste less
//     of a tile than 16 rows, and one warp has 8 + 8 products per 16 keys of 128
//     dimensions (48 in decode_mma.cu);
//   * 8 bits: both operands are fp16, to which e4m3 converts exactly, two values an
//     instruction; q is converted once, its row scaled by a power of two into
//     fp16's range (bf16's 8 significant bits fit: exact down to 2^-24 of the
//     row's largest value). P is rounded to fp16. 16 bits: bf16 products, P as a
//     bf16 part and a bf16 remainder (p to 2^-16);
//   * the order of the head dimensions inside a product is free as long as K and
//     q agree, and so is that of the output dimensions: a lane takes whole 16-byte
//     units of a K row, and at 8 bits consecutive bytes of four V rows, whose pairs
//     are interleaved by byte permutes before they are converted (16 bits: the
//     transposing load);
//   * P goes from the S^T accumulators to the operand of the second product by an
//     8 x 8 register transpose (movmatrix).
// 4 warps a CTA, each with its own slots of 16 keys of K and of V filled by TMA.
//
// Split: the requests' contexts, counted in 16-key chunks one after the other, are
// cut into equal shares, as many as let every (share, KV head, row group) have one
// of the CTAs that the GPU holds at once: they all stream the same number of bytes
// and end together, whatever the lengths, and the CTAs of one share, which start
// together, read the heads of the same tokens, neighbours in memory, at the same
// time. (Shares that ran through one head after the other took 297 us where these
// take 199 for 8 contexts of 32K to 128K keys.) A CTA goes through its share request
// by request; a context that a cut divides leaves unnormalised partial rows (at most
// two sets a CTA: of its first and its last request), which a second, small grid
// joins.
#include <math.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kChunk = 16;  // keys of a TMA box and of a pipeline stage
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr float kRescaleThreshold = 8.f;
constexpr uint32_t kFull = 0xffffffffu;
// A share is at least this many units, so that short contexts are not cut into pieces
// that cost more than they save (2 contexts of 4096 keys, 8 bits: 14.8 us; 16.4 with
// shares of 8, 16.0 with 32; one of 2048: 12.4, 12.4, 14.6).
constexpr int kMinShare = 16;
// What going over to another request costs a CTA, in units of a chunk's time (64 contexts
// of 512 to 4096 keys, 8 bits: 62.7 us by equal chunks alone, 59.4 with a cost of 9, 56.7
// with 18, 57.8 with 36; contexts of 32K to 128K 204.2, 202.9, 202.4, 202.6).
constexpr int kStartCost = 18;

template <bool EIGHT>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (EIGHT)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Byte offset of 16-byte unit `unit` of row `row` in a 16-row tile written by TMA.
// 8 bits: D-byte rows, 128-byte swizzle for 128-byte rows, 64-byte for 64. 16 bits:
// the rows' first 128-byte halves, then their second, 128-byte swizzle.
template <int D, bool EIGHT>
__device__ __forceinline__ uint32_t swz(int row, int unit) {
  if (EIGHT && D == 64) return (uint32_t)(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
  const int line = EIGHT ? row : (unit >> 3) * kChunk + row;
  return (uint32_t)(line * 128 + (((unit & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// A request as the shares count it.
struct Request {
  int32_t t0, qlen, L;
  Visible vis;
  // kStartCost and the chunks that it sees, or the whole as one; 0: not one of this
  // grid's
  int units;
};

__device__ __forceinline__ Request read_request(const AttnParams& p, int i, bool* bad = nullptr) {
  Request r;
  r.units = 0;
  r.t0 = __ldg(p.cu_seqlens + i);
  const int32_t t1 = __ldg(p.cu_seqlens + i + 1);
  r.L = __ldg(p.seq_lens + i);
  r.qlen = t1 - r.t0;
  if (r.t0 < 0 || t1 < r.t0 || t1 > p.num_tokens) {
    if (bad) *bad = true;
    return r;
  }
  if (r.qlen < 1 || r.qlen > p.decode_max_q) return r;  // longer ones run on the prefill kernel
  if (r.qlen > p.max_query_len || r.L < r.qlen || r.L > p.max_seq_len ||
      r.L > p.max_blocks * p.block_size) {
    if (bad) *bad = true;
    return r;
  }
  r.vis = visible_units(p.window, p.num_sink, r.L - r.qlen, r.L, kChunk);
  r.units = p.whole_segments ? 1 : kStartCost + r.vis.count;
  return r;
}

// Where a share begins, for the grid that joins the pieces: the chunk of the request
// there (0: its start, nothing to join) and its chunks, the share's length, the
// request's first token and its queries.
struct Cut {
  int32_t chunk, chunks, share, t0, qlen;
};

// Partial rows of piece `slot` of CTA `cta`: [COLS][D] sums, [COLS] maxima, [COLS]
// sums of weights.
template <int D, int COLS>
__device__ __forceinline__ float* piece(const AttnParams& p, int cta, int slot) {
  return p.ws_out + (int64_t)(2 * cta + slot) * COLS * (D + 2);
}

template <int D, int NT, bool EIGHT>
struct Form {
  static constexpr int COLS = 8 * NT;
  static constexpr int ROW = EIGHT ? D : 2 * D;  // bytes of a key's K or V
  static constexpr int SLOT = 2 * kChunk * ROW;
  static constexpr int SPW = (EIGHT && NT == 2 ? 3 : 2) * (D == 128 ? 1 : 2);
  static constexpr int SLOTS = kWarps * SPW * SLOT;
  static constexpr int RS = D + 4;  // floats of a column in the reduction, padded
  // at most so many CTAs an SM (their registers), fewer where shared memory ends first
  static constexpr int CTAS = 3;
  static constexpr size_t smem(int rows) {
    return 1024 + SLOTS + kWarps * SPW * sizeof(uint64_t) +
           (size_t)kWarps * (rows < COLS ? rows : COLS) * (RS + 2) * sizeof(float);
  }
  static constexpr int ctas(int rows) {
    // 228 KB an SM, 1 KB of it taken by each CTA beside what it asks for (and 1 KB
    // of its own static memory)
    const int n = (int)(228 * 1024 / (smem(rows) + 2048));
    return n < CTAS ? n : CTAS;
  }
};

// NT: 8-column tiles of (query, head) rows, rows being query-major.
template <int D, int NT, bool EIGHT>
__global__ void __launch_bounds__(kThreads, (Form<D, NT, EIGHT>::CTAS))
    decode_rows_kernel(const __grid_constant__ CUtensorMap kv_map, const AttnParams p) {
  using F = Form<D, NT, EIGHT>;
  constexpr int KS = D / 16;     // k-steps of K Q^T
  constexpr int MT = D / 16;     // row tiles of V^T P^T
  constexpr int COLS = F::COLS, SPW = F::SPW, SLOT = F::SLOT, HALF = SLOT / 2, RS = F::RS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + F::SLOTS);
  __shared__ int64_t s_sums[kWarps];
  __shared__ int64_t s_rem;
  __shared__ int32_t s_req, s_abort;

  if (p.after_prefill) {
    // behind a prefill grid that produces nothing read here: one extra CTA waits
    // for it, so that this grid completes after it (see decode_mma.cu)
    if (blockIdx.x == gridDim.x - 1) {
      griddep_wait();
      return;
    }
  } else {
    griddep_wait();
    griddep_launch_dependents();
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int group = p.num_heads / p.num_kv_heads;
  // the CTA: share `at` of one KV head and one group of rows
  const int subs = (p.decode_max_rows + COLS - 1) / COLS;
  const int at = blockIdx.x / (p.num_kv_heads * subs);
  const int combo = blockIdx.x - at * (p.num_kv_heads * subs);
  const int kvh = combo / subs, row0 = (combo - kvh * subs) * COLS;

  if (lane == 0) {
    for (int s = 0; s < SPW; ++s) mbar_init(smem_addr(&bars[warp * SPW + s]), 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    prefetch_tmap(&kv_map);
    s_abort = 0;
    s_req = -1;
  }

  // ---- the share: units [x0, x1) of the whole step's
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  const int r0 = min(p.num_seqs, (int)threadIdx.x * per), r1 = min(p.num_seqs, r0 + per);
  int64_t sum = 0;
  bool bad = false;
  for (int i = r0; i < r1; ++i) sum += read_request(p, i, &bad).units;
  if (bad && blockIdx.x == 0) set_status(p.status, PKV_DEV_BAD_LENGTHS);
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sums[w];
    total += s_sums[w];
  }
  const int64_t share =
      max((total + p.num_shares - 1) / p.num_shares, (int64_t)(p.whole_segments ? 1 : kMinShare));
  const int64_t x0 = at * share, x1 = min(total, x0 + share);
  if (x0 >= before && x0 < before + sum) {  // one thread: its requests hold the first unit
    int64_t rem = x0 - before;
    int i = r0;
    for (;; ++i) {
      const int w = read_request(p, i).units;
      if (rem < w) break;
      rem -= w;
    }
    s_req = i;
    s_rem = rem;
  }
  __syncthreads();
  int req = s_req;
  Cut* cut = reinterpret_cast<Cut*>(p.ws_lse) + at;
  const bool says = threadIdx.x == 0 && combo == 0 && !p.whole_segments;
  if (x0 >= total || req < 0) {
    if (says) *cut = Cut{0, 0, 0, 0, 0};
    return;
  }
  int64_t rem = s_rem, x = x0;
  const int32_t nrows = p.num_blocks * p.block_size;
  const int bs16 = p.block_size / kChunk;
  // the reduction's buffers, for as many rows as a request may have
  const int red_rows = min(COLS, p.decode_max_rows);
  float* red_o = reinterpret_cast<float*>(bars + kWarps * SPW);  // [kWarps][red_rows][RS]
  float* red_ml = red_o + kWarps * red_rows * RS;                // [kWarps][red_rows][2]

  // One request's part of the share: chunks [c0, c0 + nchunks) of the ones it sees
  struct Piece {
    int32_t req, t0, qlen, L;
    Visible vis;
    int c0, nchunks;
    bool split;
  };
  // The next piece of the share that has rows for this CTA; false: none left
  auto next_piece = [&](Piece& d) -> bool {
    while (x < x1) {
      Request rq = read_request(p, req);
      while (rem >= rq.units) {  // (the next request with work; there is one)
        rem -= rq.units;
        rq = read_request(p, ++req);
      }
      const int ua = (int)rem, ub = (int)min((int64_t)rq.units, ua + (x1 - x));
      // chunks [ca, cb); a cut among the units of the start leaves all of them to
      // the share behind it
      const int ca = max(0, ua - kStartCost), cb = max(0, ub - kStartCost);
      if (x == x0 && says)
        *cut = Cut{ca, rq.vis.count, (int32_t)min(share, (int64_t)INT32_MAX), rq.t0, rq.qlen};
      x += ub - ua;
      rem += ub - ua;
      if (!p.whole_segments && ca == cb) continue;
      d.req = req;
      d.t0 = rq.t0;
      d.qlen = rq.qlen;
      d.L = rq.L;
      d.vis = rq.vis;
      d.c0 = p.whole_segments ? 0 : ca;
      d.nchunks = p.whole_segments ? rq.vis.count : cb - ca;
      d.split = d.nchunks < rq.vis.count;
      if (row0 < rq.qlen * group) return true;
    }
    return false;
  };
  auto chunks_of = [&](const Piece& d) { return max(0, (d.nchunks - warp + kWarps - 1) / kWarps); };
  // lane j: the block id of the warp's chunk kb + j of a piece (-1 behind its last)
  auto load_id = [&](const Piece& d, int kb) -> int32_t {
    const int v = warp + (kb + lane) * kWarps;
    if (v >= d.nchunks) return -1;
    return __ldg(p.block_table + (int64_t)d.req * p.max_blocks + d.vis.unit(d.c0 + v) / bs16);
  };
  // and the chunk's first row in the pool; -1: a bad id
  auto first_row = [&](const Piece& d, int kb, int32_t id) -> int32_t {
    const int u = d.vis.unit(d.c0 + warp + (kb + lane) * kWarps);
    return id >= 0 && id < p.num_blocks ? (id * bs16 + u % bs16) * kChunk : -1;
  };
  // 8 bits: the factor of a chunk's scores, log2 of its values' scale, one over it
  struct Scales {
    float a, lc, ic;
  };
  auto load_scales = [&](int32_t id) {
    Scales s{EIGHT ? 0.f : p.scale_log2, 0.f, 1.f};
    if (EIGHT && id >= 0 && id < p.num_blocks) {
      s.a = __ldg(p.scales + (int64_t)id * p.num_kv_heads + kvh) * p.scale_log2;
      // (a scale below 2^-100 as that: its values are nothing beside any other)
      const float v = fmaxf(
          __ldg(p.scales + ((int64_t)p.num_blocks + id) * p.num_kv_heads + kvh), 7.888609e-31f);
      s.lc = fast_log2(v);
      s.ic = 1.f / v;
    }
    return s;
  };
  // A piece's queries: row g of each tile, the pairs of dimensions that the lane's K
  // words hold: at 8 bits D/4 consecutive ones, at 16 bits units 2 c and 2 c + 1 of
  // each 64 dimensions
  auto load_q = [&](const Piece& d, uint32_t (&w)[NT][KS * 2]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row0 + n * 8 + g;
      if (r < d.qlen * group) {
        const uint16_t* qr =
            p.q + ((int64_t)(d.t0 + r / group) * p.num_heads + kvh * group + r % group) * D;
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
          const int at = EIGHT ? c * (D / 4) + j * 8 : (j >> 1) * 64 + c * 16 + (j & 1) * 8;
          const uint4 y = __ldg(reinterpret_cast<const uint4*>(qr + at));
          w[n][4 * j] = y.x;
          w[n][4 * j + 1] = y.y;
          w[n][4 * j + 2] = y.z;
          w[n][4 * j + 3] = y.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < KS * 2; ++j) w[n][j] = 0u;
      }
    }
  };
  // The warp's slots in turn: the next to fill, and the next to wait for with its
  // parity
  int fill = 0, use = 0;
  uint32_t use_parity = 0;
  auto issue = [&](int32_t row) {  // lane 0 only
    const uint32_t bar = smem_addr(&bars[warp * SPW + fill]);
    if (row < 0) {
      set_status(p.status, PKV_DEV_BAD_BLOCK);
      mbar_arrive(bar);  // no bytes: the chunk is skipped (masked)
      return;
    }
    const uint32_t dst = smem_addr(smem + (warp * SPW + fill) * SLOT);
    mbar_arrive_expect_tx(bar, SLOT);
    if (EIGHT) {
      tma_load_3d(dst, &kv_map, bar, 0, row, kvh);
      tma_load_3d(dst + HALF, &kv_map, bar, 0, row + nrows, kvh);
    } else {
      tma_load_4d(dst, &kv_map, bar, 0, row, kvh, 0);
      tma_load_4d(dst + HALF, &kv_map, bar, 0, row + nrows, kvh, 0);
    }
  };
  auto filled = [&]() { fill = fill + 1 == SPW ? 0 : fill + 1; };

  Piece cur, nxt;
  bool more = next_piece(cur);
  if (!more) return;
  int32_t id_cur = load_id(cur, 0), id_next = load_id(cur, 32);
  int32_t row_cur = first_row(cur, 0, id_cur);
  int in_flight = min(SPW, chunks_of(cur));
  for (int k = 0; k < in_flight; ++k) {
    const int32_t row = __shfl_sync(kFull, row_cur, k);
    if (lane == 0) issue(row);
    filled();
  }
  Scales sc_cur = load_scales(id_cur);
  uint32_t qw[NT][KS * 2];
  load_q(cur, qw);
  while (true) {
    const int my_chunks = chunks_of(cur);
    const int32_t t0 = cur.t0, L = cur.L;
    const int rows = min(COLS, cur.qlen * group - row0);
    const int32_t qpos0 = L - cur.qlen;
    Scales sc_next = sc_cur;
    int32_t row_next = -1;

    // q as the column operand, column g of a tile
    auto row_token = [&](int r) { return t0 + (row0 + r) / group; };
    auto row_head = [&](int r) { return kvh * group + (row0 + r) % group; };
    uint32_t qb[NT][KS][2];
    float qf[NT][2];  // columns 2 c, 2 c + 1 of a tile: what undoes the row's scaling
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t* w = qw[n];
      if (EIGHT) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < KS * 2; ++j)
          top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[j])), fabsf(bf16_hi(w[j]))));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // 2^(14 - exponent): the largest value lands in [2^14, 2^15)
        const int e = min(126, 14 + 127 - (int)(__float_as_uint(top) >> 23));
        const float up = __uint_as_float((uint32_t)(e + 127) << 23);
        const float down = 1.f / up;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int b = 0; b < 2; ++b)
            qb[n][ks][b] = pack_f16x2(bf16_lo(w[2 * ks + b]) * up, bf16_hi(w[2 * ks + b]) * up);
        qf[n][0] = __shfl_sync(kFull, down, (2 * c) * 4);
        qf[n][1] = __shfl_sync(kFull, down, (2 * c + 1) * 4);
      } else {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qb[n][ks][0] = w[2 * ks];
          qb[n][ks][1] = w[2 * ks + 1];
        }
        qf[n][0] = qf[n][1] = 1.f;
      }
    }
    // keys [low, lim) and the first num_sink are visible to a column
    int lim[NT][2], low[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int r = n * 8 + 2 * c + b;
        lim[n][b] = r < rows ? qpos0 + (row0 + r) / group + 1 : 0;
        low[n][b] = lim[n][b] - p.window;
      }
    // every column sees keys [lo_all, lim_all); none sees keys [num_sink, lo_any)
    const int lim_all = qpos0 + row0 / group + 1;
    const int lo_all = max(0, qpos0 + (row0 + rows - 1) / group - p.window + 1);
    const int lo_any = max(0, qpos0 - p.window + 1);

    float o[NT][MT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int t = 0; t < MT; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
    }

    // visible chunks [v0, v1) are seen whole by every column
    const int shift = cur.vis.low - cur.vis.sink;
    const int v0 = max(cur.vis.sink, (lo_all + kChunk - 1) / kChunk - shift);
    const int v1 = lim_all / kChunk - shift;
    int kb = 0;
    bool failed = false;
    // the next piece and its block ids: looked up behind the first chunks, whose
    // successors are then on their way
    int32_t nid_cur = -1, nid_next = -1;
    const int look = min(SPW, max(0, my_chunks - 1));
    auto look_up = [&]() {
      more = next_piece(nxt);
      nid_cur = more ? load_id(nxt, 0) : -1;
      nid_next = more ? load_id(nxt, 32) : -1;
    };
    if (my_chunks == 0) look_up();
    for (int k = 0; k < my_chunks; ++k) {
      if (k == look) look_up();
      if (k - kb == 32) {
        kb += 32;
        id_cur = id_next;
        row_cur = row_next;
        sc_cur = sc_next;
        id_next = load_id(cur, kb + 32);
      }
      if (k - kb == 16) {  // in time for the next 32 chunks, after their ids have arrived
        row_next = first_row(cur, kb + 32, id_next);
        if (EIGHT && k + 16 < my_chunks) sc_next = load_scales(id_next);
      }
      const bool ok = __all_sync(
          kFull, mbar_wait(smem_addr(&bars[warp * SPW + use]), use_parity, p.status));
      if (!ok) {
        failed = true;
        break;
      }
      const int slot = use;
      use = use + 1 == SPW ? 0 : use + 1;
      use_parity ^= use == 0 ? 1u : 0u;
      --in_flight;
      const bool chunk_ok = __shfl_sync(kFull, row_cur, k - kb) >= 0;
      Scales sc = sc_cur;
      if (EIGHT) {
        sc.a = __shfl_sync(kFull, sc_cur.a, k - kb);
        sc.lc = __shfl_sync(kFull, sc_cur.lc, k - kb);
        sc.ic = __shfl_sync(kFull, sc_cur.ic, k - kb);
      }
      const int v = cur.c0 + warp + k * kWarps;
      const bool whole = chunk_ok && v >= v0 && v < v1;
      const uint32_t ka = smem_addr(smem + (warp * SPW + slot) * SLOT), va = ka + HALF;

      // ---- S^T = K Q^T: rows g and g + 8 of the chunk, columns 2 c, 2 c + 1, in
      // two chains of products
      float s2[2][NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s2[0][n][e] = s2[1][n][e] = 0.f;
      if (EIGHT) {
        uint32_t kw[2][KS];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < KS / 4; ++j) {
            const uint4 y = lds16(ka + swz<D, EIGHT>(g + 8 * h, c * (KS / 4) + j));
            kw[h][4 * j] = y.x;
            kw[h][4 * j + 1] = y.y;
            kw[h][4 * j + 2] = y.z;
            kw[h][4 * j + 3] = y.w;
          }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t a0 = e4m3_lo(kw[0][ks]), a1 = e4m3_lo(kw[1][ks]);
          const uint32_t a2 = e4m3_hi(kw[0][ks]), a3 = e4m3_hi(kw[1][ks]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma<EIGHT>(s2[ks & 1][n], a0, a1, a2, a3, qb[n][ks][0], qb[n][ks][1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
          const int unit = (j >> 1) * 8 + 2 * c + (j & 1);
          const uint4 y = lds16(ka + swz<D, EIGHT>(g, unit));
          const uint4 z = lds16(ka + swz<D, EIGHT>(g + 8, unit));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma<EIGHT>(s2[0][n], y.x, z.x, y.y, z.y, qb[n][2 * j][0], qb[n][2 * j][1]);
            mma<EIGHT>(s2[1][n], y.z, z.z, y.w, z.w, qb[n][2 * j + 1][0], qb[n][2 * j + 1][1]);
          }
        }
      }
      // ---- scores in log2 units, with the values' scale; hidden ones -inf
      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[n][e] = fmaf(s2[0][n][e] + s2[1][n][e], sc.a * qf[n][e & 1], sc.lc);
      if (!whole) {
        const int key0 = cur.vis.unit(v) * kChunk;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = key0 + g + (e >> 1) * 8;
            if (!chunk_ok || key >= lim[n][e & 1] || (key < low[n][e & 1] && key >= p.num_sink))
              s[n][e] = -INFINITY;
          }
        // V rows that no query sees may hold anything: their weights are 0, and
        // 0 * NaN is not
        for (int e = lane; e < kChunk * (F::ROW / 16); e += 32) {
          const int row = e / (F::ROW / 16), key = key0 + row;
          if (!chunk_ok || key >= L || (key < lo_any && key >= p.num_sink))
            st_shared_zero16(va + swz<D, EIGHT>(row, e % (F::ROW / 16)));
        }
        __syncwarp();
      }
      // ---- lazy running maximum: it moves only when a score passes it by 8
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) grow |= s[n][e] > m[n][e & 1] + kRescaleThreshold;
      if (__any_sync(kFull, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float mx = fmaxf(s[n][b], s[n][2 + b]);
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
            if (mx > m[n][b] + kRescaleThreshold) {
              const float al = fast_exp2(m[n][b] - mx);  // 0 while m is -inf
              m[n][b] = mx;
              l[n][b] *= al;
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                o[n][t][b] *= al;
                o[n][t][2 + b] *= al;
              }
            }
          }
      }
      // ---- weights, transposed into the operand of the second product. The sum
      // takes them before their rounding (a small scale of the values makes a
      // weight small, not its share of the sum)
      uint32_t pb[NT][2], pl[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
        const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
        const float p0 = fast_exp2(s[n][0] - m0), p1 = fast_exp2(s[n][1] - m1);
        const float p2 = fast_exp2(s[n][2] - m0), p3 = fast_exp2(s[n][3] - m1);
        l[n][0] = fmaf(p0 + p2, sc.ic, l[n][0]);
        l[n][1] = fmaf(p1 + p3, sc.ic, l[n][1]);
        if (EIGHT) {
          pb[n][0] = transpose8(pack_f16x2(p0, p1));
          pb[n][1] = transpose8(pack_f16x2(p2, p3));
        } else {
          const uint32_t a = pack_bf16x2(p0, p1), b = pack_bf16x2(p2, p3);
          pb[n][0] = transpose8(a);
          pb[n][1] = transpose8(b);
          pl[n][0] = transpose8(pack_bf16x2(p0 - bf16_lo(a), p1 - bf16_hi(a)));
          pl[n][1] = transpose8(pack_bf16x2(p2 - bf16_lo(b), p3 - bf16_hi(b)));
        }
      }
      // ---- O^T += V^T P^T
      if (EIGHT) {
        // V rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9: D / 8 bytes from dimension g D / 8;
        // row tile t holds dimensions g D/8 + 2 t (rows 0..7) and + 1 (rows 8..15)
        uint32_t vw[4][MT / 2];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int row = 2 * c + (h & 1) + (h >> 1) * 8;
          if (D == 128) {
            const uint4 y = lds16(va + swz<D, EIGHT>(row, g));
            vw[h][0] = y.x;
            vw[h][1] = y.y;
            vw[h][MT / 2 - 2] = y.z;
            vw[h][MT / 2 - 1] = y.w;
          } else {
            const uint2 y = lds8(va + swz<D, EIGHT>(row, g >> 1) + (g & 1) * 8);
            vw[h][0] = y.x;
            vw[h][1] = y.y;
          }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const uint32_t sel = (t & 1) ? 0x7362u : 0x5140u;
          const uint32_t y = __byte_perm(vw[0][t / 2], vw[1][t / 2], sel);
          const uint32_t z = __byte_perm(vw[2][t / 2], vw[3][t / 2], sel);
          const uint32_t a0 = e4m3_lo(y), a1 = e4m3_hi(y), a2 = e4m3_lo(z), a3 = e4m3_hi(z);
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma<EIGHT>(o[n][t], a0, a1, a2, a3, pb[n][0], pb[n][1]);
        }
      } else {
        // row tile t holds dimensions 16 t + g (rows 0..7) and 16 t + 8 + g
        const int mi = lane >> 3;
        const int row = (lane & 7) + (mi >> 1) * 8;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t a[4];
          ldsm_x4_trans(va + swz<D, EIGHT>(row, 2 * t + (mi & 1)), a);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma<EIGHT>(o[n][t], a[0], a[1], a[2], a[3], pb[n][0], pb[n][1]);
            mma<EIGHT>(o[n][t], a[0], a[1], a[2], a[3], pl[n][0], pl[n][1]);
          }
        }
      }
      __syncwarp();
      const int kn = k + SPW;
      if (kn < my_chunks) {
        const int32_t row = kn - kb < 32 ? __shfl_sync(kFull, row_cur, kn - kb)
                                         : __shfl_sync(kFull, row_next, kn - kb - 32);
        if (lane == 0) {
          fence_proxy_async_smem();  // our accesses of the slot precede the refill
          issue(row);
        }
        filled();
        ++in_flight;
      }
    }
    if (failed) {
      // after an abandoned wait, let this warp's copies in flight land before the
      // CTA leaves (bounded as well)
      for (; in_flight > 0; --in_flight) {
        mbar_wait(smem_addr(&bars[warp * SPW + use]), use_parity, nullptr);
        use = use + 1 == SPW ? 0 : use + 1;
        use_parity ^= use == 0 ? 1u : 0u;
      }
      if (lane == 0) s_abort = 1;
    } else if (more) {
      // the next piece's first chunks, scales and queries are fetched while this
      // one's rows are written
      row_next = first_row(nxt, 0, nid_cur);
      sc_next = load_scales(nid_cur);
      in_flight = min(SPW, chunks_of(nxt));
      if (lane == 0) fence_proxy_async_smem();
      for (int k = 0; k < in_flight; ++k) {
        const int32_t row = __shfl_sync(kFull, row_next, k);
        if (lane == 0) issue(row);
        filled();
      }
    }

    // a column's sum lies in the 8 lanes of the same c
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int y = 4; y < 32; y <<= 1) l[n][b] += __shfl_xor_sync(kFull, l[n][b], y);

    __syncthreads();  // the last piece's rows have been read
    if (s_abort) {    // (uniform: written before the barrier)
      for (; in_flight > 0; --in_flight) {  // the next piece's copies land first
        mbar_wait(smem_addr(&bars[warp * SPW + use]), use_parity, nullptr);
        use = use + 1 == SPW ? 0 : use + 1;
        use_parity ^= use == 0 ? 1u : 0u;
      }
      return;
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int col = n * 8 + 2 * c + b;
        float* dst = red_o + (warp * red_rows + col) * RS;
        if (col < rows) {
          if (EIGHT) {
#pragma unroll
            for (int t = 0; t < MT; t += 2)
              *reinterpret_cast<float4*>(dst + g * (D / 8) + 2 * t) =
                  make_float4(o[n][t][b], o[n][t][2 + b], o[n][t + 1][b], o[n][t + 1][2 + b]);
          } else {
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              dst[16 * t + g] = o[n][t][b];
              dst[16 * t + 8 + g] = o[n][t][2 + b];
            }
          }
        }
        if (g == 0 && col < rows) {
          red_ml[(warp * red_rows + col) * 2] = m[n][b];
          red_ml[(warp * red_rows + col) * 2 + 1] = l[n][b];
        }
      }
    __syncthreads();
    if (more) load_q(nxt, qw);

    float* part = piece<D, COLS>(p, blockIdx.x, cur.c0 > 0 ? 0 : 1);
    for (int idx = threadIdx.x; idx < rows * (D / 2); idx += kThreads) {
      const int r = idx / (D / 2), d = (idx - r * (D / 2)) * 2;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_ml[(w * red_rows + r) * 2]);
      float wsum = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = red_ml[(w * red_rows + r) * 2], lw = red_ml[(w * red_rows + r) * 2 + 1];
        if (lw == 0.f) continue;  // no key (a sum that is NaN goes on)
        const float a = fast_exp2(mw - M);
        wsum += a * lw;
        const float2 y = *reinterpret_cast<const float2*>(red_o + (w * red_rows + r) * RS + d);
        a0 += a * y.x;
        a1 += a * y.y;
      }
      if (cur.split) {
        *reinterpret_cast<float2*>(part + r * D + d) = make_float2(a0, a1);
        if (d == 0) {
          part[COLS * D + r] = M;
          part[COLS * (D + 1) + r] = wsum;
        }
        continue;
      }
      const bool none = wsum == 0.f;
      const float v0 = none ? 0.f : a0 / wsum, v1 = none ? 0.f : a1 / wsum;
      const int64_t orow = (int64_t)row_token(r) * p.num_heads + row_head(r);
      if (p.out_bf16)
        reinterpret_cast<uint32_t*>(p.out)[(orow * D + d) / 2] = pack_bf16x2(v0, v1);
      else
        *reinterpret_cast<float2*>(p.out + orow * D + d) = make_float2(v0, v1);
      if (d == 0 && p.out_lse)
        p.out_lse[orow] = none ? -INFINITY : (M + fast_log2(wsum)) * kLn2;
    }
    if (!more) return;
    cur = nxt;
    id_cur = nid_cur;
    id_next = nid_next;
    row_cur = row_next;
    sc_cur = sc_next;
  }
}

// Contexts that a cut divides: a CTA takes the one that a share begins inside of, if
// it is the context's first cut, for one KV head and one group of rows, a warp a row.
template <int D, int NT, bool EIGHT>
__global__ void __launch_bounds__(256) join_rows_kernel(const AttnParams p) {
  constexpr int COLS = 8 * NT;
  constexpr int E = D / 32;  // values a lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // The next grid may launch only when this one has left the SMs (no early trigger):
  // an attention CTA takes a third of an SM's registers, and CTAs of this grid that
  // leave holes in the register file keep the third one out for a whole share (64
  // contexts of 512 to 4096 keys, 8 bits: 58 us, with the trigger 58 to 68; a window
  // of 1024 keys: 53, with the trigger 54.5 to 59).
  griddep_wait();  // the attention grid and its partial rows are complete
  const int subs = (p.decode_max_rows + COLS - 1) / COLS, combos = p.num_kv_heads * subs;
  const int first = blockIdx.x / combos;  // the share that the context's first piece is in
  const int combo = blockIdx.x - first * combos;
  const int kvh = combo / subs, row0 = (combo - kvh * subs) * COLS;
  const Cut cut = reinterpret_cast<const Cut*>(p.ws_lse)[first + 1];
  // the first cut: the context does not reach back over the whole share before it
  if (cut.chunk == 0 || cut.chunk > cut.share) return;
  const int group = p.num_heads / p.num_kv_heads;
  const int rows = min(COLS, cut.qlen * group - row0);
  const int pieces = 1 + (cut.chunks - cut.chunk + cut.share - 1) / cut.share;
  for (int r = warp; r < rows; r += 8) {
    float M = -INFINITY, wsum = 0.f;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    constexpr int U = 4;  // pieces in flight
    for (int b = 0; b < pieces; b += U) {
      float mm[U], ll[U], v[U][E];
#pragma unroll
      for (int y = 0; y < U; ++y) {
        const bool there = b + y < pieces;
        const float* part = piece<D, COLS>(p, (first + (there ? b + y : 0)) * combos + combo,
                                           b + y == 0 ? 1 : 0);
        mm[y] = there ? __ldcg(part + COLS * D + r) : -INFINITY;
        ll[y] = there ? __ldcg(part + COLS * (D + 1) + r) : 0.f;
        if (E == 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(part + r * D) + lane);
          v[y][0] = f.x;
          v[y][1] = f.y;
          v[y][E - 2] = f.z;
          v[y][E - 1] = f.w;
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(part + r * D) + lane);
          v[y][0] = f.x;
          v[y][1] = f.y;
        }
      }
#pragma unroll
      for (int y = 0; y < U; ++y) {
        if (ll[y] == 0.f) continue;  // no key (a sum that is NaN goes on)
        if (mm[y] > M) {
          const float a = fast_exp2(M - mm[y]);  // 0 while M is -inf
          wsum *= a;
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] *= a;
          M = mm[y];
        }
        const float w = fast_exp2(mm[y] - M);
        wsum += w * ll[y];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] += w * v[y][e];
      }
    }
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    const int64_t orow =
        (int64_t)(cut.t0 + (row0 + r) / group) * p.num_heads + kvh * group + (row0 + r) % group;
    if (p.out_bf16) {
      uint32_t* out = reinterpret_cast<uint32_t*>(p.out) + (orow * D + lane * E) / 2;
#pragma unroll
      for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) p.out[orow * D + lane * E + e] = acc[e] * inv;
    }
    if (lane == 0 && p.out_lse)
      p.out_lse[orow] = wsum == 0.f ? -INFINITY : (M + fast_log2(wsum)) * kLn2;
  }
}

// Shares of a step of `combos` (KV head, group of rows): what the GPU's 152 SMs hold
// at once.
template <int D, int NT, bool EIGHT>
int rows_shares(int num_kv_heads, int max_rows, int64_t* combos) {
  using F = Form<D, NT, EIGHT>;
  *combos = (int64_t)num_kv_heads * ((max_rows + F::COLS - 1) / F::COLS);
  const int64_t n = 152 * F::ctas(max_rows) / *combos;
  return n < 1 ? 1 : (int)n;
}

template <class... A>
cudaError_t launch(void (*kernel)(A...), unsigned grid, int threads, size_t smem,
                   cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, int NT, bool EIGHT>
cudaError_t launch_form(AttnParams p, const CUtensorMap& kv_map, cudaStream_t stream) {
  using F = Form<D, NT, EIGHT>;
  auto kernel = decode_rows_kernel<D, NT, EIGHT>;
  static SmemLimit limit;
  if (cudaError_t e =
          limit.ensure(reinterpret_cast<const void*>(kernel), (int)F::smem(F::COLS), 100);
      e != cudaSuccess)
    return e;
  // (the small grid behind it asks for the same split between shared memory and L1:
  // an SM that has to change it waits until it is empty)
  static SmemLimit join_limit;
  if (cudaError_t e = join_limit.ensure(
          reinterpret_cast<const void*>(join_rows_kernel<D, NT, EIGHT>), 0, 100);
      e != cudaSuccess)
    return e;
  int64_t combos = 0;
  p.num_shares = rows_shares<D, NT, EIGHT>(p.num_kv_heads, p.decode_max_rows, &combos);
  cudaError_t e = launch(kernel, (unsigned)(p.num_shares * combos + (p.after_prefill ? 1 : 0)),
                         kThreads, F::smem(p.decode_max_rows), stream, kv_map, p);
  if (e != cudaSuccess || p.whole_segments || p.num_shares < 2) return e;
  return launch(join_rows_kernel<D, NT, EIGHT>, (unsigned)((p.num_shares - 1) * combos), 256, 0,
                stream, p);
}

template <int D, int NT, bool EIGHT>
size_t form_workspace(int num_kv_heads, int max_rows, size_t* cuts) {
  int64_t combos = 0;
  const int64_t shares = rows_shares<D, NT, EIGHT>(num_kv_heads, max_rows, &combos);
  // (one share: nothing is divided)
  *cuts = shares < 2 ? 0 : shares * combos * 2 * 8 * NT * (D + 2) * sizeof(float);
  return *cuts + shares * sizeof(Cut);
}

}  // namespace

size_t decode_rows_workspace(int32_t num_kv_heads, int32_t max_rows, int32_t head_dim, bool eight,
                             size_t* cuts) {
  const bool one = max_rows <= 8;
  if (eight) {
    if (head_dim == 128)
      return one ? form_workspace<128, 1, true>(num_kv_heads, max_rows, cuts)
                 : form_workspace<128, 2, true>(num_kv_heads, max_rows, cuts);
    return one ? form_workspace<64, 1, true>(num_kv_heads, max_rows, cuts)
               : form_workspace<64, 2, true>(num_kv_heads, max_rows, cuts);
  }
  if (head_dim == 128)
    return one ? form_workspace<128, 1, false>(num_kv_heads, max_rows, cuts)
               : form_workspace<128, 2, false>(num_kv_heads, max_rows, cuts);
  return one ? form_workspace<64, 1, false>(num_kv_heads, max_rows, cuts)
             : form_workspace<64, 2, false>(num_kv_heads, max_rows, cuts);
}

cudaError_t launch_decode_rows(const AttnParams& p, const CUtensorMap& kv_map,
                               cudaStream_t stream) {
  const bool one = p.decode_max_rows <= 8;
  if (p.scales) {
    if (p.head_dim == 128)
      return one ? launch_form<128, 1, true>(p, kv_map, stream)
                 : launch_form<128, 2, true>(p, kv_map, stream);
    return one ? launch_form<64, 1, true>(p, kv_map, stream)
               : launch_form<64, 2, true>(p, kv_map, stream);
  }
  if (p.head_dim == 128)
    return one ? launch_form<128, 1, false>(p, kv_map, stream)
               : launch_form<128, 2, false>(p, kv_map, stream);
  return one ? launch_form<64, 1, false>(p, kv_map, stream)
             : launch_form<64, 2, false>(p, kv_map, stream);
}

}  // namespace pkv
