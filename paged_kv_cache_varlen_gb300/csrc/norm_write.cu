// norm_write.cu -- the norms of the query and key heads, the rotary positions
// and the cache write in one pass: into a bf16 pool, or into a pool held in 8
// bits (e4m3) with a scale for each block of tokens and KV head.
//
// A head x of D dimensions, its weights w, a pair (a, b) of the normed head at
// position m with the pair's frequency f:
//   y = x (mean(x^2) + eps)^(-1/2) (w + offset),   t = m f,
//   (a, b) -> factor * (a cos t - b sin t, b cos t + a sin t),
// all in fp32, rounded once. The angle is formed as in rope_write.cu.
//
// 8 bits: a block's scale for one KV head is the power of two
//   s = 2^ceil(log2(max |y| / 448)), 448 the largest e4m3 value,
// over its rows. e4m3 is a floating-point type, so a scale that is no power of
// two would give no closer values; and where a later token makes a block's
// scale grow, the rows that are there are rescaled without a second rounding
// (but for values that fall below the type's normal range).
//
// A head is held by a group of lanes, two 16-byte vectors a lane, so that the
// sum of squares meets in a few shuffles and the halves of a pair in one lane.
#include "common.cuh"
#include "launch.h"
#include "rope.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xffffffffu;

// Where a pair's two dimensions are: kHalves p and p + r / 2, with r / 2 a
// multiple of 8 (two vectors of one lane); kPairs 2p and 2p + 1 (one vector);
// kAny halves of any length (met through shared memory).
enum Turn { kHalves, kPairs, kAny };

// Lanes of a head's group: a power of two with two vectors a lane.
__host__ __device__ constexpr int group_lanes(int head_dim) {
  int g = 1;
  while (g * 16 < head_dim) g *= 2;
  return g;
}

// The vectors of lane u of a head: first and second, -1 where there is none.
struct LaneVecs {
  int a, b;
  bool turn;  // kHalves: the two are the halves of 8 pairs
};
template <int MODE>
__device__ __forceinline__ LaneVecs lane_vecs(int u, int V, int half) {
  LaneVecs l;
  l.turn = false;
  if (MODE == kHalves) {
    const int U = half / 8;
    l.turn = u < U;
    l.a = l.turn ? u : 2 * U + 2 * (u - U);
    l.b = l.turn ? u + U : l.a + 1;
  } else {
    l.a = 2 * u;
    l.b = 2 * u + 1;
  }
  if (l.a >= V) l.a = -1;
  if (l.b >= V) l.b = -1;
  return l;
}

__device__ __forceinline__ void unpack8(const Vec8& v, float* y) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = bf16_lo(v.w[i]);
    y[2 * i + 1] = bf16_hi(v.w[i]);
  }
}
__device__ __forceinline__ Vec8 pack8(const float* y) {
  Vec8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v.w[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
  return v;
}

// The factor of a head's norm, from a lane's share of its values; all lanes of
// the warp call this.
__device__ __forceinline__ float norm_factor(const float (&y)[16], int GS, float inv_dim,
                                             float eps) {
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) ss = fmaf(y[i], y[i], ss);
  for (int o = 1; o < GS; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
  return rsqrtf(fmaf(ss, inv_dim, eps));
}

// A lane's 16 values turned; c, s: the cosines and sines of its 8 pairs (kHalves,
// kPairs). kAny: cs, sn those of all pairs, st room for the head's values.
template <int MODE>
__device__ __forceinline__ void turn16(float (&y)[16], const float (&c)[8], const float (&s)[8],
                                       const LaneVecs& l, int u, int half, const float* cs,
                                       const float* sn, float* st) {
  if (MODE == kHalves) {
    if (l.turn) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = y[i], b = y[8 + i];
        y[i] = a * c[i] - b * s[i];
        y[8 + i] = b * c[i] + a * s[i];
      }
    }
  } else if (MODE == kPairs) {
    const int pairs = half - u * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1];
      if (i < pairs) {
        y[2 * i] = a * c[i] - b * s[i];
        y[2 * i + 1] = b * c[i] + a * s[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<float4*>(st + u * 16 + i) =
          make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int d = u * 16 + i;
      if (d < half)
        y[i] = y[i] * cs[d] - st[d + half] * sn[d];
      else if (d < 2 * half)
        y[i] = y[i] * cs[d - half] + st[d - half] * sn[d - half];
    }
    __syncwarp();
  }
}

__device__ __forceinline__ void load_cs(float (&c)[8], float (&s)[8], const float* cs,
                                        const float* sn, int u) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + u * 8 + i);
    *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(sn + u * 8 + i);
  }
}

// Weight i of a norm (bf16 or fp32), 1 where there is none.
__device__ __forceinline__ float weight_at(const void* w, int f32, float offset, int i) {
  if (!w) return 1.f;
  const float x = f32 ? __ldg(static_cast<const float*>(w) + i)
                      : bf16_lo(__ldg(static_cast<const uint16_t*>(w) + i));
  return x + offset;
}

// A lane's 16 weights from shared memory (vectors that it has none of: 0).
__device__ __forceinline__ void load_weights(float (&w)[16], const float* ws, const LaneVecs& l) {
#pragma unroll
  for (int i = 0; i < 8; i += 4) {
    const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 a = l.a >= 0 ? *reinterpret_cast<const float4*>(ws + l.a * 8 + i) : z;
    const float4 b = l.b >= 0 ? *reinterpret_cast<const float4*>(ws + l.b * 8 + i) : z;
    *reinterpret_cast<float4*>(w + i) = a;
    *reinterpret_cast<float4*>(w + 8 + i) = b;
  }
}

// Into a bf16 pool through slots: `parts` warps share a token, as in
// rope_write.cu.
template <int MODE>
__global__ void __launch_bounds__(kThreads, 2) norm_rope_kernel(const NormRopeParams p,
                                                                const int parts) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = p.head_dim, H = p.num_heads, Hkv = p.num_kv_heads;
  const int half = p.rotary_dim / 2;
  const int V = D / 8, GS = group_lanes(D);
  const int slots = 32 / GS;          // heads at a time
  const int pad = 8 * GS;             // pairs, rounded up
  uint64_t* frac = reinterpret_cast<uint64_t*>(smem);                // [pad]
  float* wq = reinterpret_cast<float*>(frac + pad);                  // [2 pad]
  float* wk = wq + 2 * pad;                                          // [2 pad]
  float* cs = wk + 2 * pad + warp * 2 * pad;                         // [pad]
  float* sn = cs + pad;
  float* st = wk + 2 * pad + kWarps * 2 * pad + warp * 512;          // [512] (kAny)
  griddep_wait();
  griddep_launch_dependents();
  int lost = 0;  // whether some frequency is no number
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double f = __ldg(p.inv_freq + i);
    frac[i] = turn_fraction(f);
    lost |= no_number(f);
  }
  for (int i = threadIdx.x; i < D; i += kThreads) {
    wq[i] = weight_at(p.q_weight, p.weight_f32, p.weight_offset, i);
    wk[i] = weight_at(p.k_weight, p.weight_f32, p.weight_offset, i);
  }
  lost = __syncthreads_or(lost);
  const int u = lane % GS, head_slot = lane / GS;
  const LaneVecs l = lane_vecs<MODE>(u, V, half);
  const float inv_dim = 1.f / (float)D;
  const int64_t row = (int64_t)Hkv * D;
  const int vecs = (int)(row / 8);
  const int units = p.num_tokens * parts;  // (below 2^31: the host bounds parts by the tokens)
  for (int unit = blockIdx.x * kWarps + warp; unit < units; unit += gridDim.x * kWarps) {
    const int t = unit / parts, part = unit - t * parts;
    const int32_t pos = __ldg(p.positions + t);
    const int64_t slot = __ldg(p.slots + t);
    if (pos < 0) {  // uniform: the token is skipped
      if (lane == 0 && part == 0) set_status(p.status, PKV_DEV_BAD_POSITION);
      continue;
    }
    const bool write = slot >= 0 && slot < p.num_slots;
    if (!write && slot != -1 && lane == 0 && part == 0) set_status(p.status, PKV_DEV_BAD_SLOT);
    const uint16_t* q = p.q + (int64_t)t * p.q_stride;
    const uint16_t* k = p.k + (int64_t)t * p.k_stride;
    uint16_t* qo = p.q_out + (int64_t)t * H * D;
    uint16_t* ko = static_cast<uint16_t*>(p.pool) + (write ? slot : 0) * row;
    const int heads = write ? H + Hkv : H;
    // the warp's share: heads [h0, h1) of q's and then k's, vectors of v
    const int h0 = (int)((int64_t)heads * part / parts);
    const int h1 = (int)((int64_t)heads * (part + 1) / parts);

    __syncwarp();  // the last token's angles have been read
    for (int i = lane; i < half; i += 32) {
      const float2 a = rope_angle(frac[i], (uint32_t)pos, p.factor);
      cs[i] = a.x;
      sn[i] = a.y;
    }
    if (lost)
      for (int i = lane; i < half; i += 32)
        if (no_number(__ldg(p.inv_freq + i))) cs[i] = sn[i] = __uint_as_float(kNan);
    __syncwarp();
    float c[8], s[8];
    load_cs(c, s, cs, sn, u);
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {  // queries, keys
      const int a0 = kind == 0 ? h0 : max(h0, H) - H, a1 = kind == 0 ? min(h1, H) : h1 - H;
      if (a0 >= a1) continue;
      const uint16_t* in = kind == 0 ? q : k;
      uint16_t* out = kind == 0 ? qo : ko;
      const bool normed = (kind == 0 ? p.q_weight : p.k_weight) != nullptr;
      float w[16];
      load_weights(w, kind == 0 ? wq : wk, l);
      constexpr int B = MODE == kAny ? 1 : 2;  // loads of so many heads in flight
      for (int hb = a0; hb < a1; hb += B * slots) {
        Vec8 xa[B], xb[B];
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int h = hb + i * slots + head_slot;
          xa[i] = xb[i] = Vec8{{0u, 0u, 0u, 0u}};
          if (h < a1 && l.a >= 0) xa[i] = load8(in + h * D + l.a * 8);
          if (h < a1 && l.b >= 0) xb[i] = load8(in + h * D + l.b * 8);
        }
#pragma unroll
        for (int i = 0; i < B; ++i) {
          const int h = hb + i * slots + head_slot;
          float y[16];
          unpack8(xa[i], y);
          unpack8(xb[i], y + 8);
          if (normed) {
            const float r = norm_factor(y, GS, inv_dim, p.eps);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = y[j] * r * w[j];
          }
          turn16<MODE>(y, c, s, l, u, half, cs, sn, st + head_slot * (GS * 16));
          if (h < a1 && l.a >= 0) store8(out + h * D + l.a * 8, pack8(y));
          if (h < a1 && l.b >= 0) store8(out + h * D + l.b * 8, pack8(y + 8));
        }
      }
    }
    if (write) {
      const uint16_t* v = p.v + (int64_t)t * p.v_stride;
      uint16_t* vo = ko + p.num_slots * row;
      const int v1 = (int)((int64_t)vecs * (part + 1) / parts);
      constexpr int B = 4;
      for (int i = (int)((int64_t)vecs * part / parts) + lane; i < v1; i += B * 32) {
        Vec8 a[B];
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (i + j * 32 < v1) a[j] = load8(v + (int64_t)(i + j * 32) * 8);
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (i + j * 32 < v1) store8(vo + (int64_t)(i + j * 32) * 8, a[j]);
      }
    }
  }
}

template <int MODE>
cudaError_t launch_norm_rope_mode(const NormRopeParams& p, cudaStream_t stream) {
  const int pad = 8 * group_lanes(p.head_dim);
  size_t smem = (size_t)pad * 8 + 4 * pad * sizeof(float) + kWarps * 2 * pad * sizeof(float);
  if (MODE == kAny) smem += kWarps * 512 * sizeof(float);
  // (at most 40 KB, at head_dim 512)
  // warps per token: enough to spread a step over the GPU, no more than leave
  // a warp about four heads
  const int heads = p.num_heads + p.num_kv_heads;
  int parts = 1;
  while (parts < 16 && parts * 8 <= heads && (int64_t)p.num_tokens * parts < 152 * 16) parts *= 2;
  const int64_t units = (int64_t)p.num_tokens * parts;
  int64_t ctas = (units + kWarps - 1) / kWarps;
  const int64_t most = 152 * 8;  // CTAs that stay for several tokens share what they set up
  if (ctas > most) ctas = most;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_kernel<MODE>, p, parts);
}

// ---------------------------------------------------------------------------
// Into an 8-bit pool
// ---------------------------------------------------------------------------

// Four values as e4m3 (round to nearest even; beyond the range +-448; NaN stays
// NaN), the first in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
// The e4m3 pair in the low half of w as floats.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)w));
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// 2^ceil(log2(top / 448)), at least 2^-100, for a finite top >= 0: with top in
// [2^e, 2^(e + 1)) and 448 = 1.75 2^8, the exponent is e - 8, one more where the
// significand is above 1.75.
__device__ __forceinline__ float block_scale(float top) {
  const uint32_t bits = __float_as_uint(top);
  const int e = (int)(bits >> 23) - 127;
  const int k = max(-100, e - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0));
  return __uint_as_float((uint32_t)(k + 127) << 23);
}

__device__ __forceinline__ float finite_magnitude(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// One CTA: the rows that the step adds to one block of one request, a share of
// the heads. A warp holds the rows of one head, 16 at a time, in registers: their
// largest magnitude gives the scale, and they are written without being read
// again (blocks of more than 16 rows read them twice, the second time from L2).
template <int D, int MODE>
__global__ void __launch_bounds__(kThreads, 2) append_fp8_kernel(const NormRopeParams p,
                                                                 const int parts) {
  constexpr int V = D / 8, GS = group_lanes(D);
  constexpr int RP = 32 / GS;   // rows at a time
  constexpr int NP = 16 / RP;   // of 16
  constexpr int PAD = D / 2;    // pairs, rounded up
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.num_heads, Hkv = p.num_kv_heads, BS = p.block_size;
  const int half = p.rotary_dim / 2;
  float* wq = reinterpret_cast<float*>(smem);  // [D]
  float* wk = wq + D;                          // [D]
  float* st = wk + D + warp * 512;             // [512] (kAny)
  float* cs = wk + D + (MODE == kAny ? kWarps * 512 : 0);  // [BS][PAD], then the sines
  float* sn = cs + BS * PAD;
  griddep_wait();
  griddep_launch_dependents();
  const int item = blockIdx.x / parts, part = blockIdx.x - item * parts;

  // Item x of the grid belongs to the request r with f(r) <= x < f(r + 1), where
  // f(r) = cu[r] / BS + 2 r leaves each request room for every block it touches.
  int r = item, local = 0;
  if (p.max_query_len > 1) {
    int count = 0;
    for (int base = 0; base < p.num_seqs; base += kThreads) {
      const int i = base + threadIdx.x;
      const bool at = i < p.num_seqs && __ldg(p.cu_seqlens + i) / BS + 2 * i <= item;
      const int n = __syncthreads_count(at);
      count += n;
      if (n < kThreads) break;
    }
    r = count - 1;
    if (r < 0) return;
    local = item - (__ldg(p.cu_seqlens + r) / BS + 2 * r);
  }
  auto bad_lengths = [&](int i) {
    const int32_t a = __ldg(p.cu_seqlens + i), b = __ldg(p.cu_seqlens + i + 1);
    if (a < 0 || b < a || b > p.num_tokens) return true;
    const int32_t len = __ldg(p.seq_lens + i);
    return b > a && (len < b - a || b - a > p.max_query_len || len > p.max_blocks * BS);
  };
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.num_seqs; i += kThreads)
      if (bad_lengths(i)) set_status(p.status, PKV_DEV_BAD_LENGTHS);
  if (bad_lengths(r)) return;
  const int32_t t0 = __ldg(p.cu_seqlens + r), qlen = __ldg(p.cu_seqlens + r + 1) - t0;
  const int32_t L = __ldg(p.seq_lens + r);
  const int32_t start = L - qlen;  // the position of the first new token
  const int32_t block = start / BS + local;
  if (qlen < 1 || block > (L - 1) / BS) return;
  const int first = max(0, start - block * BS), last = min(BS, L - block * BS);  // its new rows
  const int32_t tok0 = t0 + block * BS - start;  // the token of row 0 (of row r: tok0 + r)
  const int32_t id = __ldg(p.block_table + (int64_t)r * p.max_blocks + block);
  const bool write = id >= 0 && id < p.num_blocks;
  if (!write && threadIdx.x == 0) set_status(p.status, PKV_DEV_BAD_BLOCK);

  for (int i = threadIdx.x; i < D; i += kThreads) {
    wq[i] = weight_at(p.q_weight, p.weight_f32, p.weight_offset, i);
    wk[i] = weight_at(p.k_weight, p.weight_f32, p.weight_offset, i);
  }
  if (half > 0)
    for (int e = threadIdx.x; e < (last - first) * half; e += kThreads) {
      const int row = first + e / half, i = e % half;
      const double f = __ldg(p.inv_freq + i);
      const int32_t pos = __ldg(p.positions + tok0 + row);
      float2 a = rope_angle(turn_fraction(f), (uint32_t)pos, p.factor);
      if (no_number(f)) a.x = a.y = __uint_as_float(kNan);
      cs[row * PAD + i] = a.x;
      sn[row * PAD + i] = a.y;
    }
  __syncthreads();

  const int u = lane % GS, row_slot = lane / GS;
  const LaneVecs l = lane_vecs<MODE>(u, V, half);
  constexpr float inv_dim = 1.f / (float)D;
  const int g0 = first / 16, g1 = (last - 1) / 16;  // groups of 16 rows
  // whether a row is one of the new ones (and its position good)
  auto is_new = [&](int row) {
    return row >= first && row < last &&
           (!p.positions || __ldg(p.positions + tok0 + row) >= 0);
  };
  if (p.positions && part == 0)
    for (int row = first + threadIdx.x; row < last; row += kThreads)
      if (__ldg(p.positions + tok0 + row) < 0) set_status(p.status, PKV_DEV_BAD_POSITION);
  // rows of group g of one head, normed and turned
  auto rows_of = [&](const uint16_t* in, int64_t stride, bool normed, const float* ws, bool turned,
                     int g, float (&y)[NP][16], bool (&ok)[NP]) {
    Vec8 xa[NP], xb[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int row = g * 16 + i * RP + row_slot;
      ok[i] = is_new(row);
      xa[i] = xb[i] = Vec8{{0u, 0u, 0u, 0u}};
      const uint16_t* x = in + (int64_t)(tok0 + row) * stride;
      if (ok[i] && l.a >= 0) xa[i] = load8(x + l.a * 8);
      if (ok[i] && l.b >= 0) xb[i] = load8(x + l.b * 8);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      unpack8(xa[i], y[i]);
      unpack8(xb[i], y[i] + 8);
    }
    if (normed) {
      float w[16];
      load_weights(w, ws, l);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float f = norm_factor(y[i], GS, inv_dim, p.eps);
#pragma unroll
        for (int j = 0; j < 16; ++j) y[i][j] = y[i][j] * f * w[j];
      }
    }
    if (turned)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int row = min(max(g * 16 + i * RP + row_slot, first), last - 1);
        float c[8], s[8];
        if (MODE != kAny) load_cs(c, s, cs + row * PAD, sn + row * PAD, u);
        turn16<MODE>(y[i], c, s, l, u, half, cs + row * PAD, sn + row * PAD,
                     st + row_slot * (GS * 16));
      }
  };

  const int jobs = (write ? 2 * Hkv : 0) + (p.q ? H : 0);
  for (int job = part * kWarps + warp; job < jobs; job += parts * kWarps) {
    const int kv = write ? 2 * Hkv : 0;
    float y[NP][16];
    bool ok[NP];
    if (job >= kv) {  // a query head
      const int h = job - kv;
      for (int g = g0; g <= g1; ++g) {
        rows_of(p.q + h * D, p.q_stride, p.q_weight != nullptr, wq, half > 0, g, y, ok);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int row = g * 16 + i * RP + row_slot;
          uint16_t* out = p.q_out + ((int64_t)(tok0 + row) * H + h) * D;
          if (ok[i] && l.a >= 0) store8(out + l.a * 8, pack8(y[i]));
          if (ok[i] && l.b >= 0) store8(out + l.b * 8, pack8(y[i] + 8));
        }
      }
      continue;
    }
    const bool key = job < Hkv;
    const int h = key ? job : job - Hkv;
    const uint16_t* in = (key ? p.k : p.v) + h * D;
    const int64_t stride = key ? p.k_stride : p.v_stride;
    const bool normed = key && p.k_weight != nullptr, turned = key && half > 0;
    float top = 0.f;
    for (int g = g0; g <= g1; ++g) {
      rows_of(in, stride, normed, wk, turned, g, y, ok);
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (ok[i]) top = fmaxf(top, finite_magnitude(y[i][j]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    // the scale: a block that holds rows already keeps its own where that is larger
    float* scale_at = p.scales + ((int64_t)(key ? 0 : p.num_blocks) + id) * Hkv + h;
    const float old = first > 0 ? *scale_at : 0.f;
    const float scale = fmaxf(old, block_scale(top));
    uint8_t* rows = static_cast<uint8_t*>(p.pool) +
                    (((int64_t)(key ? 0 : p.num_blocks) + id) * BS * Hkv + h) * D;
    const int64_t step = (int64_t)Hkv * D;
    if (first > 0 && scale != old) {
      const float ratio = old > 0.f ? old / scale : 0.f;
      for (int e = lane; e < first * (D / 4); e += 32) {
        uint32_t* at = reinterpret_cast<uint32_t*>(rows + (e / (D / 4)) * step) + e % (D / 4);
        const float2 a = unpack_e4m3x2(*at), b = unpack_e4m3x2(*at >> 16);
        *at = pack_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
      }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0 && scale != old) *scale_at = scale;
    // a power of two (every scale of these writes): its reciprocal is exact
    const bool exact = (__float_as_uint(scale) & 0x7fffffu) == 0;
    const float inv = 1.f / scale;
    for (int g = g0; g <= g1; ++g) {
      if (g0 != g1) rows_of(in, stride, normed, wk, turned, g, y, ok);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint8_t* out = rows + (g * 16 + i * RP + row_slot) * step;
        if (!exact)
#pragma unroll
          for (int j = 0; j < 16; ++j) y[i][j] = __fdiv_rn(y[i][j], scale);
        else
#pragma unroll
          for (int j = 0; j < 16; ++j) y[i][j] *= inv;
        if (ok[i] && l.a >= 0)
          *reinterpret_cast<uint2*>(out + l.a * 8) =
              make_uint2(pack_e4m3x4(y[i][0], y[i][1], y[i][2], y[i][3]),
                         pack_e4m3x4(y[i][4], y[i][5], y[i][6], y[i][7]));
        if (ok[i] && l.b >= 0)
          *reinterpret_cast<uint2*>(out + l.b * 8) =
              make_uint2(pack_e4m3x4(y[i][8], y[i][9], y[i][10], y[i][11]),
                         pack_e4m3x4(y[i][12], y[i][13], y[i][14], y[i][15]));
      }
    }
  }
}

template <int D, int MODE>
cudaError_t launch_append_mode(const NormRopeParams& p, cudaStream_t stream) {
  size_t smem = 2 * D * sizeof(float) + (MODE == kAny ? kWarps * 512 * sizeof(float) : 0);
  if (p.rotary_dim > 0) smem += (size_t)p.block_size * D * sizeof(float);
  auto kernel = append_fp8_kernel<D, MODE>;
  if (smem > 48 * 1024) {
    static SmemLimit limit;
    cudaError_t e = limit.ensure(reinterpret_cast<const void*>(kernel), 200 * 1024);
    if (e != cudaSuccess) return e;
  }
  const int64_t items = p.max_query_len == 1
                            ? p.num_seqs
                            : (int64_t)p.num_tokens / p.block_size + 2 * (int64_t)p.num_seqs;
  // shares of a block's heads: enough CTAs for the GPU, no more than leave a
  // warp one head
  const int jobs = 2 * p.num_kv_heads + (p.q ? p.num_heads : 0);
  const int64_t blocks = p.num_tokens / p.block_size + p.num_seqs;  // about
  int parts = 1;
  while (parts * kWarps < jobs && blocks * parts < 152 * 4) ++parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, parts);
}

template <int D>
cudaError_t launch_append_d(const NormRopeParams& p, cudaStream_t stream) {
  if (p.interleaved || p.rotary_dim == 0) return launch_append_mode<D, kPairs>(p, stream);
  if ((p.rotary_dim / 2) % 8 == 0) return launch_append_mode<D, kHalves>(p, stream);
  return launch_append_mode<D, kAny>(p, stream);
}

}  // namespace

cudaError_t launch_append_fp8(const NormRopeParams& p, cudaStream_t stream) {
  if (p.head_dim == 128) return launch_append_d<128>(p, stream);
  if (p.head_dim == 64) return launch_append_d<64>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
  if (p.interleaved || p.rotary_dim == 0) return launch_norm_rope_mode<kPairs>(p, stream);
  if ((p.rotary_dim / 2) % 8 == 0) return launch_norm_rope_mode<kHalves>(p, stream);
  return launch_norm_rope_mode<kAny>(p, stream);
}

}  // namespace pkv
