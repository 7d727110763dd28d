// norm_write.cu -- the norms of the query and key heads, the rotary positions
// and the cache write in one pass: into a bf16 pool, or into a pool held in 8
// bits (e4m3) with a scale for each block of tokens and KV head.
//
// A head x of D dimensions, its weights w, a pair (a, b) of the normed head at
// position m with the pair's frequency f:
//   y = x (mean(x^2) + eps)^(-1/2) (w + offset),   t = m f,
//   (a, b) -> factor * (a cos t - b sin t, b cos t + a sin t),
// all in fp32, rounded once. The angle is formed modulo a turn as in rope_write.cu.
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
//
// What bounds them: bytes, for prompts (8192 tokens of 32 + 8 heads of 128: 201 MB
// into a bf16 pool, 36 us, 5.6 TB/s; 185 MB into an 8-bit one, 44 us, 4.2 TB/s, where
// the angles, the magnitudes and the roundings keep the issue slots half busy);
// latency, for single tokens (3.4 us for one, 5.3 us for 64 of them at 8 bits: a chain
// of lengths, block, scale, rows).
#include "common.cuh"
#include "launch.h"
#include "rope.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kAhead = 3;  // passes whose copies are under way (5: as fast)
// CTAs an SM; three of them spill (8192 tokens: 36 us, 41 with three)
constexpr int kRowCtas = 2;

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
#pragma unroll
  for (int o = 1; o < GS; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
  // (a Newton step takes the root's 2 ulp to less than one; not where it is 0 or no number)
  const float v = fmaf(ss, inv_dim, eps), r = rsqrtf(v), e = fmaf(-v * r, r, 1.f);
  return fabsf(e) < 1e-3f ? fmaf(0.5f * r, e, r) : r;
}

// The same to about half an ulp, for keys that are rounded to 8 bits (of 168M, 104 fall
// to the other side of a rounding boundary, 133 by the form above; 8192 tokens 44.2 us,
// 43.3): the factor as r + lo (float2), its products with the weights with their
// remainders, one rounding a value. Both kernels that write 8 bits norm keys so: a key's
// bits do not depend on what else is in its step.
__device__ __forceinline__ float2 near_factor(const float (&y)[16], int GS, float inv_dim,
                                              float eps) {
  float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) s4[i & 3] = fmaf(y[i], y[i], s4[i & 3]);
  float ss = (s4[0] + s4[1]) + (s4[2] + s4[3]);
#pragma unroll
  for (int o = 1; o < GS; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
  const float v = fmaf(ss, inv_dim, eps), r = rsqrtf(v), e = fmaf(-v * r, r, 1.f);
  return make_float2(r, fabsf(e) < 1e-3f ? 0.5f * r * e : 0.f);
}
__device__ __forceinline__ void near_scale16(float (&y)[16], float2 f, const float* ws,
                                             const LaneVecs& l) {
  const float* wa = ws + max(l.a, 0) * 8;
  const float* wb = ws + max(l.b, 0) * 8;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 w4 = *reinterpret_cast<const float4*>((i < 8 ? wa : wb) + i % 8);
    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q = f.x * w[j], rest = fmaf(f.y, w[j], fmaf(f.x, w[j], -q));
      y[i + j] = fmaf(y[i + j], q, y[i + j] * rest);
    }
  }
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
      for (int i = 0; i < 8; i += 2) {  // two pairs an instruction
        const float2 a = make_float2(y[i], y[i + 1]), b = make_float2(y[8 + i], y[9 + i]);
        const float2 cc = make_float2(c[i], c[i + 1]), ss = make_float2(s[i], s[i + 1]);
        const float2 n = __fmul2_rn(b, ss);
        const float2 x = __ffma2_rn(a, cc, make_float2(-n.x, -n.y));
        const float2 z = __ffma2_rn(b, cc, __fmul2_rn(a, ss));
        y[i] = x.x;
        y[i + 1] = x.y;
        y[8 + i] = z.x;
        y[9 + i] = z.y;
      }
    }
  } else if (MODE == kPairs) {
    const int pairs = half - u * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1];
      if (i < pairs) {
        y[2 * i] = fmaf(a, c[i], -(b * s[i]));  // (in every kernel the same bits)
        y[2 * i + 1] = fmaf(a, s[i], b * c[i]);
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
        y[i] = fmaf(y[i], cs[d], -(st[d + half] * sn[d]));
      else if (d < 2 * half)
        y[i] = fmaf(y[i], cs[d - half], st[d - half] * sn[d - half]);
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

// A lane's values times the norm's factor and the weights, from shared memory.
__device__ __forceinline__ void scale16(float (&y)[16], float f, const float* ws,
                                        const LaneVecs& l) {
  const float* wa = ws + max(l.a, 0) * 8;  // (of a vector that the lane has not: any)
  const float* wb = ws + max(l.b, 0) * 8;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 w = *reinterpret_cast<const float4*>((i < 8 ? wa : wb) + i % 8);
    y[i] = y[i] * f * w.x;
    y[i + 1] = y[i + 1] * f * w.y;
    y[i + 2] = y[i + 2] * f * w.z;
    y[i + 3] = y[i + 3] * f * w.w;
  }
}

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

// Eight values over a scale, as e4m3. The scale of every one of these writes is a power of
// two: its reciprocal is exact (one that was there before need not be).
__device__ __forceinline__ uint2 quantise8(const float* y, float scale) {
  float z[8];
  if ((__float_as_uint(scale) & 0x7fffffu) == 0) {
    const float inv = 1.f / scale;
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = y[j] * inv;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = __fdiv_rn(y[j], scale);
  }
  return make_uint2(pack_e4m3x4(z[0], z[1], z[2], z[3]), pack_e4m3x4(z[4], z[5], z[6], z[7]));
}
// Four stored values under a scale that is `ratio` times smaller than the new one.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  const float2 a = unpack_e4m3x2(w), b = unpack_e4m3x2(w >> 16);
  return pack_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// Rows of their own: into a bf16 pool through slots, or (EIGHT) one token a request
// into an 8-bit pool. A pass of a warp takes as many heads as it has groups, of a
// token's query, key and value heads in this order; every warp has an equal run of the
// passes of all tokens. A lane fetches its own vectors kAhead passes early into shared
// memory, where only it reads them: nothing has to be waited for but the lane's own
// copies, which start before the angles are formed. DIM: the heads' size, 0 for any.
template <int DIM, int MODE, bool EIGHT>
__global__ void __launch_bounds__(kThreads, kRowCtas) norm_rope_kernel(const NormRopeParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = DIM ? DIM : p.head_dim;
  const int H = EIGHT && !p.q ? 0 : p.num_heads, Hkv = p.num_kv_heads;
  const int half = p.rotary_dim / 2;
  const int V = D / 8, GS = group_lanes(D);
  const int slots = 32 / GS;          // heads of a pass
  const int pad = 8 * GS;             // pairs, rounded up
  uint64_t* frac = reinterpret_cast<uint64_t*>(smem);                // [pad]
  float* wq = reinterpret_cast<float*>(frac + pad);                  // [2 pad]
  float* wk = wq + 2 * pad;                                          // [2 pad]
  float* cs = wk + 2 * pad + warp * 2 * pad;                         // [pad]
  float* sn = cs + pad;
  uint8_t* ring = reinterpret_cast<uint8_t*>(wk + 2 * pad + kWarps * 2 * pad) +
                  warp * (kAhead + 1) * 1024 + lane * 16;            // [kAhead + 1][2][32][16]
  float* st = wk + 2 * pad + kWarps * 2 * pad + kWarps * (kAhead + 1) * 256 + warp * 512;  // kAny
  griddep_wait();
  griddep_launch_dependents();
  const int u = lane % GS, head_slot = lane / GS;
  const LaneVecs l = lane_vecs<MODE>(u, V, half);
  const bool has_a = DIM || l.a >= 0, has_b = DIM || l.b >= 0;
  const float inv_dim = 1.f / (float)D;
  const int64_t row = (int64_t)Hkv * D;
  const int passes = (H + 2 * Hkv + slots - 1) / slots;
  // the warp's run: n passes from pass `pass` of row t on
  const int64_t total = (int64_t)(EIGHT ? p.num_seqs : p.num_tokens) * passes;
  const int64_t warps = min(total, (int64_t)gridDim.x * kWarps);
  const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t begin = w < warps ? total * w / warps : 0;
  const int n = w < warps ? (int)(total * (w + 1) / warps - begin) : 0;
  int t = (int)(begin / passes), pass = (int)(begin - (int64_t)t * passes);

  // EIGHT: request r's token, -1 where it has none (or lengths that are no good)
  auto token_of = [&](int r, int32_t& len, bool& bad) -> int {
    const int32_t a = __ldg(p.cu_seqlens + r), b = __ldg(p.cu_seqlens + r + 1);
    len = __ldg(p.seq_lens + r);
    bad = a < 0 || b < a || b > p.num_tokens ||
          (b > a && (len < 1 || b - a > 1 || len > p.max_blocks * p.block_size));
    return bad || b == a ? -1 : a;
  };
  struct Row {
    int token;     // -1: none
    int32_t pos;
    int64_t slot;  // the pool's row
    int32_t id;    // EIGHT: the block, the rows that it held
    int held;
    bool bad;
  };
  auto look = [&](int i) {
    Row x;
    x.bad = false;
    x.id = -1;
    x.held = 0;
    x.slot = -1;
    if (EIGHT) {
      int32_t len;
      x.token = token_of(i, len, x.bad);
      if (x.token >= 0) {
        const int block = (len - 1) / p.block_size;
        x.id = __ldg(p.block_table + (int64_t)i * p.max_blocks + block);
        x.held = len - 1 - block * p.block_size;
        if (x.id >= 0 && x.id < p.num_blocks) x.slot = (int64_t)x.id * p.block_size + x.held;
      }
    } else {
      x.token = i;
      x.slot = __ldg(p.slots + i);
    }
    x.pos = (!EIGHT || p.positions) && x.token >= 0 ? __ldg(p.positions + x.token) : 0;
    return x;
  };

  // the copies' place in the run
  int left = n, ft = t, fpass = pass, to = 0, ftok = -1;
  const uint16_t *fq = nullptr, *fk = nullptr, *fv = nullptr;  // of the row, less heads before
  auto fetch = [&] {
    if (left > 0) {
      if (left == n || fpass == 0) {
        int32_t len;
        bool bad;
        ftok = EIGHT ? token_of(ft, len, bad) : ft;
        fq = p.q + ftok * p.q_stride;
        fk = p.k + ftok * p.k_stride - H * D;
        fv = p.v + ftok * p.v_stride - (H + Hkv) * D;
      }
      const int h = fpass * slots + head_slot;
      const uint16_t* x = (h < H ? fq : h < H + Hkv ? fk : fv) + h * D;
      const uint32_t at = smem_addr(ring + to * 1024);
      if (ftok >= 0 && h < H + 2 * Hkv) {
        if (has_a) cp_async_16(at, x + l.a * 8, 16);
        if (has_b) cp_async_16(at + 512, x + l.b * 8, 16);
      }
      --left;
      if (++fpass == passes) {
        fpass = 0;
        ++ft;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    to = to == kAhead ? 0 : to + 1;
  };
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) fetch();
  Row next{};
  if (n > 0) next = look(t);

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

  Row now{};
  bool good = false, write = false;
  uint16_t *oq = nullptr, *ok = nullptr, *ov = nullptr;  // where the row goes, less heads before
  uint8_t *ek = nullptr, *ev = nullptr;                  // (EIGHT)
  float c[8], s[8];
  float had = 0.f;  // EIGHT: the scale that the lane's head of the next pass finds
  // EIGHT: where the scale of the lane's head of a pass is
  auto scale_of = [&](int i) -> float* {
    const int h = i * slots + head_slot - H;
    if (!write || h < 0 || h >= 2 * Hkv) return nullptr;
    return p.scales + (h < Hkv ? (int64_t)now.id * Hkv + h
                               : ((int64_t)p.num_blocks + now.id) * Hkv + h - Hkv);
  };
  int from = 0;
#pragma unroll 1
  for (int i = 0; i < n; ++i, ++pass) {
    if (pass == passes) pass = 0;
    if (i == 0 || pass == 0) {  // the next row
      now = next;
      good = now.token >= 0 && now.pos >= 0;
      write = now.token >= 0 && now.slot >= 0 && now.slot < p.num_slots;
      if (lane == 0 && pass == 0) {
        if (now.bad) set_status(p.status, PKV_DEV_BAD_LENGTHS);
        if (now.token >= 0 && now.pos < 0) set_status(p.status, PKV_DEV_BAD_POSITION);
        if (EIGHT && now.token >= 0 && !write) set_status(p.status, PKV_DEV_BAD_BLOCK);
        if (!EIGHT && good && !write && now.slot != -1) set_status(p.status, PKV_DEV_BAD_SLOT);
      }
      oq = p.q_out + (int64_t)now.token * H * D;
      const int64_t first = (write ? now.slot : 0) * row - H * D;
      if (EIGHT) {
        ek = static_cast<uint8_t*>(p.pool) + first;
        ev = ek + p.num_slots * row - Hkv * D;
      } else {
        ok = static_cast<uint16_t*>(p.pool) + first;
        ov = ok + p.num_slots * row - Hkv * D;
      }
      if (EIGHT && now.held > 0 && scale_of(pass)) had = *scale_of(pass);
      ++t;
      if (i + passes - pass < n) next = look(t);
      __syncwarp();  // the last row's angles have been read
      for (int e = lane; e < half; e += 32) {
        const float2 a = near_angle(frac[e], (uint32_t)now.pos, p.factor);
        cs[e] = a.x;
        sn[e] = a.y;
      }
      if (lost)
        for (int e = lane; e < half; e += 32)
          if (no_number(__ldg(p.inv_freq + e))) cs[e] = sn[e] = __uint_as_float(kNan);
      __syncwarp();
      load_cs(c, s, cs, sn, u);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    Vec8 xa = Vec8{{0u, 0u, 0u, 0u}}, xb = xa;
    if (has_a) xa = load8(reinterpret_cast<const uint16_t*>(ring + from * 1024));
    if (has_b) xb = load8(reinterpret_cast<const uint16_t*>(ring + from * 1024 + 512));
    from = from == kAhead ? 0 : from + 1;
    fetch();  // (into the stage read in the pass before)
    const int h = pass * slots + head_slot;
    const bool query = h < H, key = !query && h < H + Hkv;
    const bool store = good && h < H + 2 * Hkv && (query || write);
    float y[16];
    if (EIGHT || pass * slots < H + Hkv) {  // uniform: not bf16 values alone
      const bool normed = query ? p.q_weight != nullptr : key && p.k_weight != nullptr;
      unpack8(xa, y);
      unpack8(xb, y + 8);
      if (pass * slots < H + Hkv) {
        const float f = norm_factor(y, GS, inv_dim, p.eps);
        float2 near = make_float2(0.f, 0.f);
        if (EIGHT && (pass + 1) * slots > H) near = near_factor(y, GS, inv_dim, p.eps);
        if (normed && EIGHT && key)
          near_scale16(y, near, wk, l);
        else if (normed)
          scale16(y, f, query ? wq : wk, l);
        turn16<MODE>(y, c, s, l, u, half, cs, sn, st + head_slot * (GS * 16));
        if (EIGHT && !query && !key) {  // a value beside keys
          unpack8(xa, y);
          unpack8(xb, y + 8);
        }
      }
    }
    if (!EIGHT || pass * slots < H) {
      if (query || (!EIGHT && key)) {
        xa = pack8(y);
        xb = pack8(y + 8);
      }
      uint16_t* out = (query ? oq : EIGHT ? nullptr : key ? ok : ov) + h * D;
      if (store && (!EIGHT || query)) {
        if (has_a) store8(out + l.a * 8, xa);
        if (has_b) store8(out + l.b * 8, xb);
      }
    }
    if (EIGHT) {
      float top = 0.f;
      if (good)
#pragma unroll
        for (int j = 0; j < 16; ++j) top = fmaxf(top, finite_magnitude(y[j]));
      for (int o = 1; o < GS; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      const float old = had;
      float* scale_at = scale_of(pass);
      had = now.held > 0 && pass + 1 < passes && scale_of(pass + 1) ? *scale_of(pass + 1) : 0.f;
      if (scale_at) {
        const float scale = fmaxf(old, block_scale(top));
        uint8_t* rows = (key ? ek : ev) + h * D;
        if (scale != old) {
          const float ratio = old > 0.f ? old / scale : 0.f;
          for (int e = 1; e <= now.held; ++e) {  // 16 bytes of each of the block's rows
            uint4* o = reinterpret_cast<uint4*>(rows - e * row + u * 16);
            const uint4 x = *o;
            *o = make_uint4(rescale4(x.x, ratio), rescale4(x.y, ratio), rescale4(x.z, ratio),
                            rescale4(x.w, ratio));
          }
          if (u == 0) *scale_at = scale;
        }
        if (store && has_a) *reinterpret_cast<uint2*>(rows + l.a * 8) = quantise8(y, scale);
        if (store && has_b) *reinterpret_cast<uint2*>(rows + l.b * 8) = quantise8(y + 8, scale);
      }
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int DIM, int MODE, bool EIGHT>
cudaError_t launch_rows_mode(const NormRopeParams& p, cudaStream_t stream) {
  const int pad = 8 * group_lanes(p.head_dim), slots = 32 / group_lanes(p.head_dim);
  size_t smem = (size_t)pad * 8 + 4 * pad * sizeof(float) + kWarps * 2 * pad * sizeof(float) +
                kWarps * (kAhead + 1) * 1024;
  if (MODE == kAny) smem += kWarps * 512 * sizeof(float);
  auto kernel = norm_rope_kernel<DIM, MODE, EIGHT>;
  if (smem > 48 * 1024) {  // (at most 72 KB, at head_dim 512)
    static SmemLimit limit;
    cudaError_t e = limit.ensure(reinterpret_cast<const void*>(kernel), 80 * 1024);
    if (e != cudaSuccess) return e;
  }
  const int passes = ((EIGHT && !p.q ? 0 : p.num_heads) + 2 * p.num_kv_heads + slots - 1) / slots;
  const int64_t total = (int64_t)(EIGHT ? p.num_seqs : p.num_tokens) * passes;
  const int64_t ctas = (total + kWarps - 1) / kWarps, most = 152 * kRowCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas < most ? ctas : most));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int DIM, bool EIGHT>
cudaError_t launch_rows_dim(const NormRopeParams& p, cudaStream_t stream) {
  if (p.interleaved || p.rotary_dim == 0) return launch_rows_mode<DIM, kPairs, EIGHT>(p, stream);
  if ((p.rotary_dim / 2) % 8 == 0) return launch_rows_mode<DIM, kHalves, EIGHT>(p, stream);
  return launch_rows_mode<DIM, kAny, EIGHT>(p, stream);
}
// The common head sizes have kernels of their own: all vectors are there, and loops
// over lanes unroll.
template <bool EIGHT>
cudaError_t launch_rows(const NormRopeParams& p, cudaStream_t stream) {
  if (p.head_dim == 128) return launch_rows_dim<128, EIGHT>(p, stream);
  if (p.head_dim == 64) return launch_rows_dim<64, EIGHT>(p, stream);
  if (EIGHT) return cudaErrorInvalidValue;
  return launch_rows_dim<0, false>(p, stream);
}

// ---------------------------------------------------------------------------
// Into an 8-bit pool, several tokens of a request
// ---------------------------------------------------------------------------

// One CTA: the rows that the step adds to one block of one request, a share of
// the heads. A warp holds a group of rows of one head in registers: their largest
// magnitude gives the scale, and they are written without being read again. The groups
// of a longer block have a warp each, TEAM of them, who tell one another the largest
// (blocks of more than four groups read their rows twice, the second time from L2). The
// next rows come into shared memory meanwhile. 8192 tokens of 32 + 8 heads of 128 in
// blocks of 16, 32, 64: 44, 55, 62 us; 44, 62, 76 when one warp goes through a block's
// groups twice; 50 for blocks of 16 when nothing is fetched ahead. CTAs of 4 warps, so
// that their setups overlap (blocks of 16: 46 us with 8, 47 with 2), 8 for teams of 4,
// as the angles of their blocks leave room for fewer.
template <int TEAM>
constexpr int kBlockWarps = TEAM == 4 ? 8 : 4;

template <int D, int MODE, int NP, int TEAM>
__global__ void __launch_bounds__(kBlockWarps<TEAM> * 32, 16 / kBlockWarps<TEAM>)
    append_fp8_kernel(const NormRopeParams p, const int parts) {
  constexpr int W = kBlockWarps<TEAM>, kBlockThreads = 32 * W;
  constexpr int V = D / 8, GS = group_lanes(D);
  constexpr int RP = 32 / GS;   // rows at a time
  constexpr int RG = NP * RP;   // of a group
  constexpr int PAD = D / 2;    // pairs, rounded up
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int H = p.num_heads, Hkv = p.num_kv_heads, BS = p.block_size;
  const int half = p.rotary_dim / 2;
  float* wq = reinterpret_cast<float*>(smem);  // [D]
  float* wk = wq + D;                          // [D]
  float* st = wk + D + warp * 512;             // [512] (kAny)
  // the warp's ring: [2][NP][2][32][16], a lane's vectors of the rows of a head
  uint8_t* ring = reinterpret_cast<uint8_t*>(wk + D + (MODE == kAny ? W * 512 : 0)) +
                  warp * 2 * NP * 1024 + lane * 16;
  uint8_t* good = reinterpret_cast<uint8_t*>(wk + D + (MODE == kAny ? W * 512 : 0)) +
                  W * 2 * NP * 1024;             // [256]: whether a row's position is good
  float* cs = reinterpret_cast<float*>(good + 256);   // [BS][PAD], then the sines
  float* sn = cs + BS * PAD;
  griddep_wait();
  griddep_launch_dependents();

  // The items, the blocks that the requests' new tokens reach, stand in a row, request
  // after request. Each request is looked at by itself: one whose lengths are no good
  // (cu_seqlens that falls, say) has none and moves no other's.
  // Request i: its first token, the position of it, its length; its items, -1 where the
  // lengths are no good.
  auto items_of = [&](int i, int32_t& t0, int32_t& start, int32_t& len) -> int {
    t0 = __ldg(p.cu_seqlens + i);
    const int32_t t1 = __ldg(p.cu_seqlens + i + 1);
    len = __ldg(p.seq_lens + i);
    if (t0 < 0 || t1 < t0 || t1 > p.num_tokens) return -1;
    if (t1 == t0) return 0;
    if (len < t1 - t0 || t1 - t0 > p.max_query_len || len > p.max_blocks * BS) return -1;
    start = len - (t1 - t0);
    return (len - 1) / BS - start / BS + 1;
  };
  // (every warp for itself, a run of requests a lane: no barrier until the angles)
  const int per = (p.num_seqs + 31) / 32;
  const int r0 = min(p.num_seqs, lane * per), r1 = min(p.num_seqs, r0 + per);
  int32_t t0 = 0, start = 0, len = 0;
  constexpr uint32_t kMost = INT32_MAX;  // (sums stop here; the grid has fewer items)
  uint32_t behind = 0;                   // items before the lane's last, it among them
#pragma unroll 4
  for (int i = r0; i < r1; ++i) {
    const int n = items_of(i, t0, start, len);
    if (n < 0 && blockIdx.x == 0 && warp == 0) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    behind = min(behind + max(n, 0), kMost);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(kFull, behind, o);
    if (lane >= o) behind = min(behind + x, kMost);
  }
  const uint32_t total = __shfl_sync(kFull, behind, 31);
  uint32_t before = __shfl_up_sync(kFull, behind, 1);
  if (lane == 0) before = 0;
  const int u = lane % GS, row_slot = lane / GS;
  const LaneVecs l = lane_vecs<MODE>(u, V, half);
  constexpr float inv_dim = 1.f / (float)D;
  const int team = warp / TEAM, member = warp % TEAM;
  __shared__ float tops[2][W];
  int from = 0, to = 0, turn = 0;
  bool loaded = false;  // the weights
  // (one item a CTA, but where requests count the same tokens)
  const int part = blockIdx.x % parts;
  const uint32_t step_items = gridDim.x / parts;
  for (uint32_t item = blockIdx.x / parts; item < total; item += step_items) {
    int r = r0;
    uint32_t rest = item - before;
    const bool holds = item >= before && item < behind;  // one lane: it has the item's request
    if (per > 1 && holds)
      for (;; ++r) {
        const uint32_t n = max(0, items_of(r, t0, start, len));
        if (rest < n) break;
        rest -= n;
      }
    const int from_lane = __ffs(__ballot_sync(kFull, holds)) - 1;
    r = __shfl_sync(kFull, r, from_lane);
    const int32_t pos0 = __shfl_sync(kFull, start, from_lane);  // of its first new token
    const int32_t block = __shfl_sync(kFull, start / BS + (int)rest, from_lane);
    const int32_t end = __shfl_sync(kFull, len, from_lane);
    // its new rows
    const int first = max(0, pos0 - block * BS), last = min(BS, end - block * BS);
    // the token of row 0 (of row r: tok0 + r)
    const int32_t tok0 = __shfl_sync(kFull, t0, from_lane) + block * BS - pos0;
    const int32_t id = __ldg(p.block_table + (int64_t)r * p.max_blocks + block);
    const bool write = id >= 0 && id < p.num_blocks;
    if (!write && threadIdx.x == 0) set_status(p.status, PKV_DEV_BAD_BLOCK);

    const int g0 = first / RG, g1 = (last - 1) / RG;  // groups of rows
    // A job is a head: of the keys, the values, the queries. The rows of one come into
    // the ring while those before are worked on.
    const int kv = write ? 2 * Hkv : 0, jobs = kv + (p.q ? H : 0);
    const int job0 = part * (W / TEAM) + team, stride_jobs = parts * (W / TEAM);
    const int own0 = g0 + member;         // the warp's first group (of none: past g1)
    const bool again = own0 + TEAM <= g1;  // it has several: keys and values are read twice
    auto sweeps = [&](int job) { return job < kv && again ? 2 : 1; };
    int fjob = own0 <= g1 ? job0 : jobs, fg = own0, fsweep = 0;
    auto fetch = [&] {
      if (fjob < jobs) {
        const bool query = fjob >= kv, key = !query && fjob < Hkv;
        const int h = query ? fjob - kv : key ? fjob : fjob - Hkv;
        const int64_t stride = query ? p.q_stride : key ? p.k_stride : p.v_stride;
        const uint16_t* x = (query ? p.q : key ? p.k : p.v) + h * D;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int row = fg * RG + i * RP + row_slot;
          if (row < first || row >= last) continue;
          const uint16_t* at = x + (tok0 + row) * stride;
          const uint32_t dst = smem_addr(ring + (to * NP + i) * 1024);
          cp_async_16(dst, at + l.a * 8, 16);
          cp_async_16(dst + 512, at + l.b * 8, 16);
        }
        fg += TEAM;
        if (fg > g1) {
          fg = own0;
          if (++fsweep == sweeps(fjob)) {
            fsweep = 0;
            fjob += stride_jobs;
          }
        }
        to ^= 1;
      }
    };
    fetch();

    for (int i = loaded ? D : threadIdx.x; i < D; i += kBlockThreads) {
      wq[i] = weight_at(p.q_weight, p.weight_f32, p.weight_offset, i);
      wk[i] = weight_at(p.k_weight, p.weight_f32, p.weight_offset, i);
    }
    loaded = true;
    for (int row = first + threadIdx.x; row < last; row += kBlockThreads) {
      const bool ok = !p.positions || __ldg(p.positions + tok0 + row) >= 0;
      good[row] = ok;
      if (!ok && part == 0) set_status(p.status, PKV_DEV_BAD_POSITION);
    }
    if (half > 0)
      for (int e = threadIdx.x; e < (last - first) * half; e += kBlockThreads) {
        const int row = first + e / half, i = e % half;
        const double f = __ldg(p.inv_freq + i);
        const int32_t pos = __ldg(p.positions + tok0 + row);
        float2 a = near_angle(turn_fraction(f), (uint32_t)pos, p.factor);
        if (no_number(f)) a.x = a.y = __uint_as_float(kNan);
        cs[row * PAD + i] = a.x;
        sn[row * PAD + i] = a.y;
      }
    __syncthreads();

    // the next rows of the ring, group g of one head, normed and turned
    auto rows_of = [&](bool normed, bool key, bool turned, int g, float (&y)[NP][16],
                       bool (&ok)[NP]) {
      cp_async_wait_all();
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int row = g * RG + i * RP + row_slot;
        ok[i] = row >= first && row < last && good[row];
        const uint8_t* at = ring + (from * NP + i) * 1024;
        const Vec8 none = Vec8{{0u, 0u, 0u, 0u}};
        unpack8(ok[i] ? load8(reinterpret_cast<const uint16_t*>(at)) : none, y[i]);
        unpack8(ok[i] ? load8(reinterpret_cast<const uint16_t*>(at + 512)) : none, y[i] + 8);
      }
      from ^= 1;
      fetch();  // (into the stage read before this one)
      if (normed)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (key)
            near_scale16(y[i], near_factor(y[i], GS, inv_dim, p.eps), wk, l);
          else
            scale16(y[i], norm_factor(y[i], GS, inv_dim, p.eps), wq, l);
        }
      if (turned)
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int row = min(max(g * RG + i * RP + row_slot, first), last - 1);
          float c[8], s[8];
          if (MODE != kAny) load_cs(c, s, cs + row * PAD, sn + row * PAD, u);
          turn16<MODE>(y[i], c, s, l, u, half, cs + row * PAD, sn + row * PAD,
                       st + row_slot * (GS * 16));
        }
    };

    for (int job = job0; job < jobs; job += stride_jobs) {
      float y[NP][16];
      bool ok[NP];
      if (job >= kv) {  // a query head
        const int h = job - kv;
        for (int g = own0; g <= g1; g += TEAM) {
          rows_of(p.q_weight != nullptr, false, half > 0, g, y, ok);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const int row = g * RG + i * RP + row_slot;
            uint16_t* out = p.q_out + ((int64_t)(tok0 + row) * H + h) * D;
            if (ok[i]) store8(out + l.a * 8, pack8(y[i]));
            if (ok[i]) store8(out + l.b * 8, pack8(y[i] + 8));
          }
        }
        continue;
      }
      const bool key = job < Hkv;
      const int h = key ? job : job - Hkv;
      const bool normed = key && p.k_weight != nullptr, turned = key && half > 0;
      // the scale: a block that holds rows already keeps its own where that is larger
      float* scale_at = p.scales + ((int64_t)(key ? 0 : p.num_blocks) + id) * Hkv + h;
      const float old = first > 0 ? *scale_at : 0.f;
      float top = 0.f;
      for (int g = own0; g <= g1; g += TEAM) {
        rows_of(normed, true, turned, g, y, ok);
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (ok[i]) top = fmaxf(top, finite_magnitude(y[i][j]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      if (TEAM > 1) {
        if (lane == 0) tops[turn][warp] = top;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * TEAM) : "memory");
#pragma unroll
        for (int w = 0; w < TEAM; ++w) top = fmaxf(top, tops[turn][team * TEAM + w]);
        turn ^= 1;  // (who writes there again has met the others at the next barrier)
      }
      const float scale = fmaxf(old, block_scale(top));
      uint8_t* rows = static_cast<uint8_t*>(p.pool) +
                      (((int64_t)(key ? 0 : p.num_blocks) + id) * BS * Hkv + h) * D;
      const int64_t step = (int64_t)Hkv * D;
      if (first > 0 && scale != old) {
        const float ratio = old > 0.f ? old / scale : 0.f;
        for (int e = member * 32 + lane; e < first * (D / 4); e += 32 * TEAM) {
          uint32_t* at = reinterpret_cast<uint32_t*>(rows + (e / (D / 4)) * step) + e % (D / 4);
          *at = rescale4(*at, ratio);
        }
      }
      __syncwarp();  // every lane (and at the barrier every warp) has read the old scale
      if (member == 0 && lane == 0 && scale != old) *scale_at = scale;
      for (int g = own0; g <= g1; g += TEAM) {
        if (again) rows_of(normed, true, turned, g, y, ok);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          uint8_t* out = rows + (g * RG + i * RP + row_slot) * step;
          if (ok[i]) *reinterpret_cast<uint2*>(out + l.a * 8) = quantise8(y[i], scale);
          if (ok[i])
            *reinterpret_cast<uint2*>(out + l.b * 8) = quantise8(y[i] + 8, scale);
        }
      }
    }
    if (item + step_items < total) __syncthreads();  // the angles have been read
  }
}

template <int D, int MODE, int NP, int TEAM>
cudaError_t launch_append_rows(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int W = kBlockWarps<TEAM>;
  size_t smem = 2 * D * sizeof(float) + (MODE == kAny ? W * 512 * sizeof(float) : 0) +
                W * 2 * NP * 1024 + 256;
  if (p.rotary_dim > 0) smem += (size_t)p.block_size * D * sizeof(float);
  auto kernel = append_fp8_kernel<D, MODE, NP, TEAM>;
  if (smem > 48 * 1024) {
    static SmemLimit limit;
    cudaError_t e = limit.ensure(reinterpret_cast<const void*>(kernel), 226 * 1024);
    if (e != cudaSuccess) return e;
  }
  const int64_t items = (int64_t)p.num_tokens / p.block_size + 2 * (int64_t)p.num_seqs;
  // shares of a block's heads: enough CTAs for the GPU, no more than leave a team of
  // warps one head
  const int jobs = 2 * p.num_kv_heads + (p.q ? p.num_heads : 0);
  const int64_t blocks = p.num_tokens / p.block_size + p.num_seqs;  // about
  int parts = 1;
  while (parts * (W / TEAM) < jobs && blocks * parts < 152 * 4) ++parts;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * parts));
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, parts);
}

// A group of rows: 16 at 128 dimensions, and at 64 where the blocks are no longer; 32
// at 64 dimensions otherwise (8192 tokens of 32 + 8 heads of 64: blocks of 16 26 us, 35
// by groups of 32; blocks of 32 31 us, 34 by groups of 16).
template <int D, int MODE>
cudaError_t launch_append_mode(const NormRopeParams& p, cudaStream_t stream) {
  constexpr int kRows = D == 64 ? 32 : 16;
  if constexpr (D == 64) {
    if (p.block_size == 16) return launch_append_rows<D, MODE, 2, 1>(p, stream);
  }
  if constexpr (MODE != kAny) {
    if (D == 128 && p.block_size > 2 * kRows) return launch_append_rows<128, MODE, 4, 4>(p, stream);
    if (p.block_size > kRows) return launch_append_rows<D, MODE, 4, 2>(p, stream);
  }
  return launch_append_rows<D, MODE, 4, 1>(p, stream);
}

template <int D>
cudaError_t launch_append_d(const NormRopeParams& p, cudaStream_t stream) {
  if (p.interleaved || p.rotary_dim == 0) return launch_append_mode<D, kPairs>(p, stream);
  if ((p.rotary_dim / 2) % 8 == 0) return launch_append_mode<D, kHalves>(p, stream);
  return launch_append_mode<D, kAny>(p, stream);
}

}  // namespace

cudaError_t launch_append_fp8(const NormRopeParams& p, cudaStream_t stream) {
  // a token a request: by rows (64 requests of 32 + 8 heads: 5.3 us; 10.0 by blocks,
  // most of whose lanes hold rows that there are not)
  if (p.max_query_len == 1) return launch_rows<true>(p, stream);
  if (p.head_dim == 128) return launch_append_d<128>(p, stream);
  if (p.head_dim == 64) return launch_append_d<64>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_norm_rope(const NormRopeParams& p, cudaStream_t stream) {
  return launch_rows<false>(p, stream);
}

}  // namespace pkv
