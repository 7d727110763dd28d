// decode_fp8.cu -- paged attention over an 8-bit cache (e4m3, a scale for each
// block and KV head) for requests of up to 32 (query, head) rows: decodes and
// short verification steps.
//
//   out = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j),  k_j = a_b K_j,
//   v_j = c_b V_j, with K_j, V_j the e4m3 values and a_b, c_b the scales of the
//   key's block b.
//
// Neither scale is multiplied into the values: a_b joins the factor of the score
// (fp32), and the weights are formed as c_b w_j = 2^(s_j + log2 c_b - m), whose
// running maximum m is over the scaled weights. What is multiplied with V_j is
// thus at most 2^8 whatever the scales, and a weight that fp16 would flush to zero
// adds less than 2^-24 of the largest to the output. The sum of the weights takes
// them in fp32, divided by c_b.
//
// Bound: HBM, 2 D bytes a key and KV head, half of the bf16 cache's. What that
// leaves is half the time a key, so that the products have to be cheap:
//   * the keys are the rows of the products, S^T = K Q^T (m16n8k16) and
//     O^T = V^T P^T, with the group's heads as the columns: 8 columns waste less
//     of a tile than 16 rows, and one warp has 8 + 8 products per 16 keys of 128
//     dimensions (48 in the bf16 kernel);
//   * both operands are fp16, to which e4m3 converts exactly, two values an
//     instruction; q is converted once, its row scaled by a power of two into
//     fp16's range (bf16's 8 significant bits fit: exact down to 2^-24 of the
//     row's largest value);
//   * the order of the head dimensions inside a product is free as long as K and
//     q agree, and so is that of the output dimensions: a lane takes 16 or 32
//     consecutive bytes of a K row and 8 or 16 of four V rows with one or two
//     wide shared-memory loads each, and needs no transposing loads: pairs of V
//     rows are interleaved by byte permutes before they are converted;
//   * P goes from the S^T accumulators to the operand of the second product by an
//     8 x 8 register transpose (movmatrix).
// The pipeline is that of decode_mma.cu: 4 warps, each with its own slots of 16
// keys of K and of V filled by TMA.
#include <math.h>

#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kChunk = 16;  // keys of a TMA box and of a pipeline stage
constexpr int kWarps = 4;
constexpr float kRescaleThreshold = 8.f;
constexpr uint32_t kFull = 0xffffffffu;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two e4m3 values (the low or the high half of w) as fp16x2, exactly.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Byte offset of 16-byte unit `unit` of row `row` in a 16-row tile of D-byte
// rows written by TMA: 128-byte swizzle for 128-byte rows, 64-byte for 64.
template <int D>
__device__ __forceinline__ uint32_t swz(int row, int unit) {
  if (D == 128) return (uint32_t)(row * 128 + ((unit ^ (row & 7)) << 4));
  return (uint32_t)(row * 64 + ((unit ^ ((row >> 1) & 3)) << 4));
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

// NT: 8-column tiles of (query, head) rows, rows being query-major.
template <int D, int NT, int SPW>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 4 : 3)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap kv_map, const AttnParams p) {
  constexpr int KS = D / 16;     // k-steps of K Q^T
  constexpr int MT = D / 16;     // row tiles of V^T P^T
  constexpr int HALF = kChunk * D;
  constexpr int SLOT = 2 * HALF;
  constexpr int COLS = 8 * NT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * SPW * SLOT);

  if (p.after_prefill) {
    // behind a prefill grid that produces nothing read here: one extra CTA waits
    // for it, so that this grid completes after it (see decode_mma.cu)
    if ((int)blockIdx.z >= p.num_seqs) {
      if (blockIdx.x == 0 && blockIdx.y == 0) griddep_wait();
      return;
    }
  } else {
    griddep_wait();
    griddep_launch_dependents();
  }

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int group = p.num_heads / p.num_kv_heads;
  const int nsub = (p.decode_max_rows + COLS - 1) / COLS;
  const int kvh = blockIdx.x / nsub;
  const int sub = blockIdx.x - kvh * nsub;
  const int part = blockIdx.y;
  const int i = blockIdx.z;
  const bool leader = blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0;

  const int32_t t0 = __ldg(p.cu_seqlens + i), t1 = __ldg(p.cu_seqlens + i + 1);
  const int32_t L = __ldg(p.seq_lens + i);
  if (t0 < 0 || t1 < t0 || t1 > p.num_tokens) {
    if (leader) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int32_t qlen = t1 - t0;
  if (qlen < 1 || qlen > p.decode_max_q) return;  // longer requests run on the prefill kernel
  if (qlen > p.max_query_len || L < qlen || L > p.max_seq_len ||
      L > p.max_blocks * p.block_size) {
    if (leader) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return;
  }
  const int row0 = sub * COLS;
  if (row0 >= qlen * group) return;
  const int rows = min(COLS, qlen * group - row0);
  const int32_t qpos0 = L - qlen;
  const Visible vis = visible_units(p.window, p.num_sink, qpos0, L, kChunk);
  const int per_part = p.part_size / kChunk;
  const int c0 = part * per_part;  // the partition's first visible chunk
  if (c0 >= vis.count) return;
  const int nchunks = min(per_part, vis.count - c0);
  const int my_chunks = (nchunks - warp + kWarps - 1) / kWarps;

  // lane j of the warp holds the block id and the scales of the warp's chunk
  // kb + j: the factor of its scores, log2 of its values' scale, and one over it
  const int32_t* bt = p.block_table + (int64_t)i * p.max_blocks;
  auto chunk_at = [&](int k) { return vis.unit(c0 + warp + k * kWarps); };
  auto load_id = [&](int kb) -> int32_t {
    const int k = kb + lane;
    return k < my_chunks ? __ldg(bt + (int64_t)chunk_at(k) * kChunk / p.block_size) : -1;
  };
  struct Scales {
    float a, lc, ic;
  };
  auto load_scales = [&](int32_t id) {
    Scales s{0.f, 0.f, 1.f};
    if (id >= 0 && id < p.num_blocks) {
      s.a = __ldg(p.scales + (int64_t)id * p.num_kv_heads + kvh) * p.scale_log2;
      // (a scale below 2^-100 as that: its values are nothing beside any other)
      const float v = fmaxf(
          __ldg(p.scales + ((int64_t)p.num_blocks + id) * p.num_kv_heads + kvh), 7.888609e-31f);
      s.lc = fast_log2(v);
      s.ic = 1.f / v;
    }
    return s;
  };
  int32_t id_cur = load_id(0);
  int32_t id_next = load_id(32);

  if (lane == 0) {
    for (int s = 0; s < SPW; ++s) mbar_init(smem_addr(&bars[warp * SPW + s]), 1);
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) prefetch_tmap(&kv_map);
  __syncwarp();

  const int32_t nrows = p.num_blocks * p.block_size;
  auto issue = [&](int k, int32_t id) {  // lane 0 only
    const int slot = k % SPW;
    const uint32_t bar = smem_addr(&bars[warp * SPW + slot]);
    if (id < 0 || id >= p.num_blocks) {
      set_status(p.status, PKV_DEV_BAD_BLOCK);
      mbar_arrive(bar);  // no bytes: the chunk is skipped (masked)
      return;
    }
    const uint32_t dst = smem_addr(smem + (warp * SPW + slot) * SLOT);
    const int32_t row = id * p.block_size + chunk_at(k) * kChunk % p.block_size;
    mbar_arrive_expect_tx(bar, SLOT);
    tma_load_3d(dst, &kv_map, bar, 0, row, kvh);
    tma_load_3d(dst + HALF, &kv_map, bar, 0, row + nrows, kvh);
  };
  int issued = 0;
  for (int k = 0; k < SPW && k < my_chunks; ++k) {
    const int32_t id = __shfl_sync(kFull, id_cur, k);
    if (lane == 0) issue(k, id);
    ++issued;
  }
  Scales sc_cur = load_scales(id_cur);
  Scales sc_next = sc_cur;

  // q as the column operand: column g of a tile, dimensions c D/4 .. + D/4 - 1
  // (the bytes of a K row that the lane takes), a k-step taking 4 of them
  auto row_token = [&](int r) { return t0 + (row0 + r) / group; };
  auto row_head = [&](int r) { return kvh * group + (row0 + r) % group; };
  uint32_t qb[NT][KS][2];
  float qf[NT][2];  // columns 2 c, 2 c + 1 of a tile: what undoes the row's scaling
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = n * 8 + g;
    uint32_t w[KS * 2];
    if (r < rows) {
      const uint4* q = reinterpret_cast<const uint4*>(
          p.q + ((int64_t)row_token(r) * p.num_heads + row_head(r)) * D + c * (D / 4));
#pragma unroll
      for (int j = 0; j < KS / 2; ++j) {
        const uint4 x = __ldg(q + j);
        w[4 * j] = x.x;
        w[4 * j + 1] = x.y;
        w[4 * j + 2] = x.z;
        w[4 * j + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < KS * 2; ++j) w[j] = 0u;
    }
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
  }
  // keys [low, lim) and the first num_sink are visible to a column
  int lim[NT][2], low[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int r = n * 8 + 2 * c + b;
      lim[n][b] = r < rows ? qpos0 + (row0 + r) / group + 1 : 0;
      low[n][b] = p.window > 0 ? lim[n][b] - p.window : 0;
    }
  // every column sees keys [lo_all, lim_all); none sees keys [num_sink, lo_any)
  const int lim_all = qpos0 + row0 / group + 1;
  const int last_q = qpos0 + (row0 + rows - 1) / group;
  const int lo_all = p.window > 0 ? max(0, last_q - p.window + 1) : 0;
  const int lo_any = p.window > 0 ? max(0, qpos0 - p.window + 1) : 0;

  float o[NT][MT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int t = 0; t < MT; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
  }

  int kb = 0, consumed = 0;
  for (int k = 0; k < my_chunks; ++k) {
    if (k - kb == 32) {
      kb += 32;
      id_cur = id_next;
      sc_cur = sc_next;
      id_next = load_id(kb + 32);
    }
    // (in time for the next 32 chunks, after their ids have arrived)
    if (k - kb == 16 && k + 16 < my_chunks) sc_next = load_scales(id_next);
    const int slot = k % SPW;
    const bool ok =
        __all_sync(kFull, mbar_wait(smem_addr(&bars[warp * SPW + slot]), (k / SPW) & 1, p.status));
    if (!ok) break;
    consumed = k + 1;
    const int32_t id = __shfl_sync(kFull, id_cur, k - kb);
    const float fa = __shfl_sync(kFull, sc_cur.a, k - kb);
    const float flc = __shfl_sync(kFull, sc_cur.lc, k - kb);
    const float fic = __shfl_sync(kFull, sc_cur.ic, k - kb);
    const int key0 = chunk_at(k) * kChunk;
    const bool chunk_ok = id >= 0 && id < p.num_blocks;
    const bool whole = chunk_ok && key0 + kChunk <= lim_all &&
                       (key0 >= lo_all || key0 + kChunk <= p.num_sink);
    const uint32_t ka = smem_addr(smem + (warp * SPW + slot) * SLOT), va = ka + HALF;

    // ---- S^T = K Q^T: rows g and g + 8 of the chunk, columns 2 c, 2 c + 1
    uint32_t kw[2][KS];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < KS / 4; ++j) {
        const uint4 x = lds16(ka + swz<D>(g + 8 * h, c * (KS / 4) + j));
        kw[h][4 * j] = x.x;
        kw[h][4 * j + 1] = x.y;
        kw[h][4 * j + 2] = x.z;
        kw[h][4 * j + 3] = x.w;
      }
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint32_t a0 = e4m3_lo(kw[0][ks]), a1 = e4m3_lo(kw[1][ks]);
      const uint32_t a2 = e4m3_hi(kw[0][ks]), a3 = e4m3_hi(kw[1][ks]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(s[n], a0, a1, a2, a3, qb[n][ks][0], qb[n][ks][1]);
    }
    // V rows 2 c, 2 c + 1, 2 c + 8, 2 c + 9: D / 8 bytes from dimension g D / 8
    uint32_t vw[4][MT / 2];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int row = 2 * c + (h & 1) + (h >> 1) * 8;
      if (D == 128) {
        const uint4 x = lds16(va + swz<D>(row, g));
        vw[h][0] = x.x;
        vw[h][1] = x.y;
        vw[h][MT / 2 - 2] = x.z;
        vw[h][MT / 2 - 1] = x.w;
      } else {
        const uint2 x = lds8(va + swz<D>(row, g >> 1) + (g & 1) * 8);
        vw[h][0] = x.x;
        vw[h][1] = x.y;
      }
    }

    // ---- scores in log2 units, with the values' scale; hidden ones -inf
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = fmaf(s[n][e], fa * qf[n][e & 1], flc);
    if (!whole) {
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
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int key = key0 + 2 * c + (h & 1) + (h >> 1) * 8;
        if (!chunk_ok || key >= L || (key < lo_any && key >= p.num_sink))
#pragma unroll
          for (int j = 0; j < MT / 2; ++j) vw[h][j] = 0u;
      }
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
    // ---- weights in fp16, transposed into the operand of the second product; the
    // sum takes them before that rounding (a small scale of the values makes a
    // weight small, not its share of the sum)
    uint32_t pb[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float m0 = m[n][0] == -INFINITY ? 0.f : m[n][0];
      const float m1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
      const float p0 = fast_exp2(s[n][0] - m0), p1 = fast_exp2(s[n][1] - m1);
      const float p2 = fast_exp2(s[n][2] - m0), p3 = fast_exp2(s[n][3] - m1);
      l[n][0] = fmaf(p0 + p2, fic, l[n][0]);
      l[n][1] = fmaf(p1 + p3, fic, l[n][1]);
      pb[n][0] = transpose8(pack_f16x2(p0, p1));
      pb[n][1] = transpose8(pack_f16x2(p2, p3));
    }
    // ---- O^T += V^T P^T: row tile t holds dimensions g D/8 + 2 t (rows 0..7)
    // and g D/8 + 2 t + 1 (rows 8..15)
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const uint32_t sel = (t & 1) ? 0x7362u : 0x5140u;
      const uint32_t x = __byte_perm(vw[0][t / 2], vw[1][t / 2], sel);
      const uint32_t y = __byte_perm(vw[2][t / 2], vw[3][t / 2], sel);
      const uint32_t a0 = e4m3_lo(x), a1 = e4m3_hi(x), a2 = e4m3_lo(y), a3 = e4m3_hi(y);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma_f16(o[n][t], a0, a1, a2, a3, pb[n][0], pb[n][1]);
    }
    __syncwarp();
    const int kn = k + SPW;
    if (kn < my_chunks) {
      const int32_t idn = (kn - kb < 32) ? __shfl_sync(kFull, id_cur, kn - kb)
                                         : __shfl_sync(kFull, id_next, kn - kb - 32);
      if (lane == 0) {
        fence_proxy_async_smem();  // our reads of the slot precede the refill
        issue(kn, idn);
      }
      ++issued;
    }
  }
  // After an abandoned wait, let this warp's copies in flight land before the
  // CTA leaves (bounded as well).
  for (int k = consumed; k < issued; ++k)
    mbar_wait(smem_addr(&bars[warp * SPW + (k % SPW)]), (k / SPW) & 1, nullptr);

  // a column's sum lies in the 8 lanes of the same c
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[n][b] += __shfl_xor_sync(kFull, l[n][b], x);

  __syncthreads();  // every warp is done with its slots: reuse them
  constexpr int RS = D + 4;  // floats per column, padded
  static_assert((size_t)kWarps * COLS * (RS + 2) * sizeof(float) <= (size_t)kWarps * SPW * SLOT,
                "the reduction buffers fit in the slots they reuse");
  float* red_o = reinterpret_cast<float*>(smem);  // [kWarps][COLS][RS]
  float* red_ml = red_o + kWarps * COLS * RS;     // [kWarps][COLS][2]
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int col = n * 8 + 2 * c + b;
      float* dst = red_o + (warp * COLS + col) * RS + g * (D / 8);
      if (col < rows) {
#pragma unroll
        for (int t = 0; t < MT; t += 2)
          *reinterpret_cast<float4*>(dst + 2 * t) =
              make_float4(o[n][t][b], o[n][t][2 + b], o[n][t + 1][b], o[n][t + 1][2 + b]);
      }
      if (g == 0) {
        red_ml[(warp * COLS + col) * 2] = m[n][b];
        red_ml[(warp * COLS + col) * 2 + 1] = l[n][b];
      }
    }
  __syncthreads();

  const int parts_i = (vis.count + per_part - 1) / per_part;
  for (int idx = threadIdx.x; idx < rows * (D / 2); idx += kWarps * 32) {
    const int r = idx / (D / 2), d = (idx - r * (D / 2)) * 2;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_ml[(w * COLS + r) * 2]);
    float wsum = 0.f, a0 = 0.f, a1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = red_ml[(w * COLS + r) * 2], lw = red_ml[(w * COLS + r) * 2 + 1];
      if (lw == 0.f) continue;  // no key (a sum that is NaN goes on)
      const float a = fast_exp2(mw - M);
      wsum += a * lw;
      const float2 x = *reinterpret_cast<const float2*>(red_o + (w * COLS + r) * RS + d);
      a0 += a * x.x;
      a1 += a * x.y;
    }
    const bool none = wsum == 0.f;
    const float v0 = none ? 0.f : a0 / wsum, v1 = none ? 0.f : a1 / wsum;
    const float lse = none ? -INFINITY : (M + fast_log2(wsum)) * kLn2;
    if (parts_i == 1) {
      const int64_t orow = (int64_t)row_token(r) * p.num_heads + row_head(r);
      if (p.out_bf16)
        reinterpret_cast<uint32_t*>(p.out)[(orow * D + d) / 2] = pack_bf16x2(v0, v1);
      else
        *reinterpret_cast<float2*>(p.out + orow * D + d) = make_float2(v0, v1);
      if (d == 0 && p.out_lse) p.out_lse[orow] = lse;
    } else {
      const int64_t rr = (((int64_t)part * p.num_seqs + i) * p.ws_q + (row0 + r) / group) *
                             p.num_heads + row_head(r);
      *reinterpret_cast<float2*>(p.ws_out + rr * D + d) = make_float2(v0, v1);
      if (d == 0) p.ws_lse[rr] = lse;
    }
  }
}

// Rows of split requests: the partitions' normalised outputs combined by their
// log-sum-exp. WPR warps share a row's partitions (one row a CTA when WPR > 1,
// else four); a lane holds 2 or 4 of the row's values.
template <int D, int WPR>
__global__ void __launch_bounds__(WPR == 1 ? 128 : WPR * 32)
    merge_rows_kernel(const AttnParams p) {
  constexpr int R = WPR == 1 ? 4 : 1;
  constexpr int RS = D + 4;
  constexpr int E = D / 32;  // values a lane
  __shared__ __align__(16) float red[WPR > 1 ? WPR * RS : 4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = (int64_t)blockIdx.x * R + (R > 1 ? warp : 0);  // (request, query, head)
  const int h = (int)(row % p.num_heads);
  const int64_t iq = row / p.num_heads;
  const int j = (int)(iq % p.ws_q);
  const int64_t i = iq / p.ws_q;
  const bool in = i < p.num_seqs;
  // the lengths are inputs, final since every attention CTA has begun; the
  // attention grid does not write them
  const int32_t t0 = in ? __ldcg(p.cu_seqlens + i) : 0;
  const int32_t t1 = in ? __ldcg(p.cu_seqlens + i + 1) : 0;
  const int32_t L = in ? __ldcg(p.seq_lens + i) : 0;
  griddep_wait();  // the attention grid and its partials are complete
  griddep_launch_dependents();
  // (uniform over the CTA when WPR > 1) rows that do not exist, and requests that
  // the attention kernel rejected, left to the prefill kernel or did not split
  if (!in || t0 < 0 || t1 < t0 || t1 > p.num_tokens) return;
  const int32_t qlen = t1 - t0;
  if (j >= qlen || qlen > p.decode_max_q || qlen > p.max_query_len) return;
  if (L < qlen || L > p.max_seq_len || L > p.max_blocks * p.block_size) return;
  const Visible vis = visible_units(p.window, p.num_sink, L - qlen, L, 16);
  const int per_part = p.part_size / 16;
  const int parts = (vis.count + per_part - 1) / per_part;
  if (parts < 2) return;
  const int64_t stride = (int64_t)p.num_seqs * p.ws_q * p.num_heads;
  const int wr = R > 1 ? 0 : warp;
  float M = -INFINITY, wsum = 0.f;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  constexpr int U = 8;  // partitions in flight a warp
  for (int base = wr; base < parts; base += U * WPR) {
    float l[U];
    float ov[U][E];
#pragma unroll
    for (int x = 0; x < U; ++x) {
      const int pp = base + x * WPR;
      const bool there = pp < parts;
      const int64_t rr = row + pp * stride;
      l[x] = there ? __ldcg(p.ws_lse + rr) * kLog2e : -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) ov[x][e] = 0.f;
      if (there) {
        if (E == 4) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ws_out + rr * D) + lane);
          ov[x][0] = v.x;
          ov[x][1] = v.y;
          ov[x][E - 2] = v.z;
          ov[x][E - 1] = v.w;
        } else {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(p.ws_out + rr * D) + lane);
          ov[x][0] = v.x;
          ov[x][1] = v.y;
        }
      }
    }
#pragma unroll
    for (int x = 0; x < U; ++x) {
      if (l[x] == -INFINITY) continue;  // past the last partition, or empty
      if (l[x] > M) {
        const float a = fast_exp2(M - l[x]);  // 0 while M is -inf
        wsum *= a;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] *= a;
        M = l[x];
      }
      const float w = fast_exp2(l[x] - M);
      wsum += w;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += w * ov[x][e];
    }
  }
  if (WPR > 1) {
    float* mine = red + warp * RS;
#pragma unroll
    for (int e = 0; e < E; ++e) mine[lane * E + e] = acc[e];
    if (lane == 0) {
      mine[D] = M;
      mine[D + 1] = wsum;
    }
    __syncthreads();
    if (warp != 0) return;
    float Mt = -INFINITY;
#pragma unroll
    for (int w = 0; w < WPR; ++w) Mt = fmaxf(Mt, red[w * RS + D]);
    wsum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      const float mw = red[w * RS + D];
      if (red[w * RS + D + 1] == 0.f) continue;  // nothing (a sum that is NaN goes on)
      const float a = fast_exp2(mw - Mt);
      wsum += a * red[w * RS + D + 1];
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += a * red[w * RS + lane * E + e];
    }
    M = Mt;
  }
  const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
  const int64_t orow = (int64_t)(t0 + j) * p.num_heads + h;
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

void config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, dim3 grid, int threads, size_t smem,
            cudaStream_t stream) {
  cfg->gridDim = grid;
  cfg->blockDim = dim3(threads);
  cfg->dynamicSmemBytes = smem;
  cfg->stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg->attrs = attr;
  cfg->numAttrs = 1;
}

template <int D, int NT>
cudaError_t launch_nt(const AttnParams& p, const CUtensorMap& kv_map, cudaStream_t stream) {
  constexpr int SPW = D == 128 ? 3 : 6;  // 48 KB of slots a CTA
  constexpr size_t SLOT = 2 * kChunk * D;
  const size_t smem = 1024 + kWarps * SPW * SLOT + kWarps * SPW * sizeof(uint64_t) + 16;
  auto kernel = decode_fp8_kernel<D, NT, SPW>;
  static SmemLimit limit;
  if (cudaError_t e = limit.ensure(reinterpret_cast<const void*>(kernel), (int)smem);
      e != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const int nsub = (p.decode_max_rows + 8 * NT - 1) / (8 * NT);
  config(&cfg, attr,
         dim3(p.num_kv_heads * nsub, p.num_parts, p.num_seqs + (p.after_prefill ? 1 : 0)),
         kWarps * 32, smem, stream);
  return cudaLaunchKernelEx(&cfg, kernel, kv_map, p);
}

template <int D>
cudaError_t launch_merge_d(const AttnParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.num_seqs * p.ws_q * p.num_heads;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  // few partitions, or many rows: a warp a row; else eight warps share a row's
  if (p.num_parts <= 8 || rows > 152 * 64) {
    config(&cfg, attr, dim3((unsigned)((rows + 3) / 4)), 128, 0, stream);
    return cudaLaunchKernelEx(&cfg, merge_rows_kernel<D, 1>, p);
  }
  config(&cfg, attr, dim3((unsigned)rows), 256, 0, stream);
  return cudaLaunchKernelEx(&cfg, merge_rows_kernel<D, 8>, p);
}

}  // namespace

cudaError_t launch_merge_rows(const AttnParams& p, cudaStream_t stream) {
  return p.head_dim == 128 ? launch_merge_d<128>(p, stream) : launch_merge_d<64>(p, stream);
}

cudaError_t launch_decode_fp8(const AttnParams& p, const CUtensorMap& kv_map, cudaStream_t stream) {
  const bool one = p.decode_max_rows <= 8;
  cudaError_t e;
  if (p.head_dim == 128)
    e = one ? launch_nt<128, 1>(p, kv_map, stream) : launch_nt<128, 2>(p, kv_map, stream);
  else
    e = one ? launch_nt<64, 1>(p, kv_map, stream) : launch_nt<64, 2>(p, kv_map, stream);
  if (e != cudaSuccess || p.num_parts < 2) return e;
  return launch_merge_rows(p, stream);
}

}  // namespace pkv
