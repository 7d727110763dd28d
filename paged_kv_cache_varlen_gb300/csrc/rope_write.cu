// rope_write.cu -- rotary positions fused with the KV-cache write: a step's
// queries and keys are rotated by their positions on the way to q_out and to
// the paged pool, the values are copied beside them.
//
// A pair (a, b) of a head at position m, with the pair's frequency f:
//   t = m f,   (a, b) -> factor * (a cos t - b sin t, b cos t + a sin t);
// pairs are (p, p + r/2) or (2p, 2p + 1) of the first r = rotary_dim
// dimensions; the others pass through.
//
// The angle: m f in fp32 would lose the fraction of a turn for far positions
// (m = 10^6 leaves 0.06 rad). The frequency is turned into a 64-bit fixed-
// point fraction of a turn instead, so that m f modulo a turn is one integer
// product that wraps by itself: off by at most |m| |f| 2^-63 / 2 pi + |m| 2^-64
// turns. Its top 32 bits become the argument of sincospif. The fraction comes
// out of the double's bits by an integer product with 2 / pi: the few FP64
// units of this GPU would take longer for a prompt's angles than its bytes.
//
// Bound: every byte moves once (q, k, v in, q_out and the pool's rows out):
// HBM for prompts, launch and memory latency for single tokens. A warp takes
// a token, or a share of its heads when the tokens are few; the token's sines
// and cosines, two or so a lane, meet in shared memory, and in the layout of
// halves a lane keeps those of its 8 pairs for all its heads.
// Measured: 8192 tokens of 32 + 8 heads of 128: 35.0 us, 5.8 TB/s (85 % of the
// measured copy rate); 64 tokens: 4.5 us a call, most of it the host's. Halves
// of any length (40 of the 128 dimensions rotated): 64 tokens 4.3, 1024 9.8,
// 8192 60.7 us, a CTA a token and two trips through shared memory.
#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The fraction of a turn that a position advances: frac(f / 2 pi) 2^64, rounded
// down, from the bits of f (a finite double).
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)((bits >> 52) & 2047) - 1023;  // |f| in [2^e, 2^(e + 1))
  const uint64_t m = (bits << 11) | (1ull << 63);   // |f| 2^(63 - e)
  const uint64_t kTwoOverPi = 0xA2F9836E4E441529ull;  // 2 / pi 2^64 = 2^66 / 2 pi
  const uint64_t hi = __umul64hi(m, kTwoOverPi), lo = m * kTwoOverPi;
  // |f| / 2 pi = (hi 2^64 + lo) 2^(e - 129)
  const int s = 65 - e;
  uint64_t r = 0;
  if (s >= 128 || s <= -64)
    r = 0;
  else if (s >= 64)
    r = hi >> (s - 64);
  else if (s > 0)
    r = (hi << (64 - s)) | (lo >> s);
  else
    r = lo << -s;
  return (bits >> 63) ? 0 - r : r;
}

// An infinite or NaN frequency: its pair becomes NaN (a fraction of a turn cannot
// say so).
__device__ __forceinline__ bool no_number(double f) {
  return ((uint64_t)__double_as_longlong(f) >> 52 & 2047) == 2047;
}
constexpr uint32_t kNan = 0x7fffffffu;

// cos and sin of pos turns of `frac` 2^-64 each, times factor.
__device__ __forceinline__ float2 rope_angle(uint64_t frac, uint32_t pos, float factor) {
  const int32_t hi = (int32_t)((frac * pos) >> 32);  // fraction of a turn, as a signed 32-bit one
  float s, c;
  sincospif((float)hi * 4.656612873077393e-10f, &s, &c);  // 2 pi hi / 2^32 = pi hi / 2^31
  return make_float2(c * factor, s * factor);
}

struct Vec8 {
  uint32_t w[4];
};
__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  return Vec8{{v.x, v.y, v.z, v.w}};
}
__device__ __forceinline__ void store8(uint16_t* p, const Vec8& v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

__device__ __forceinline__ void rotate8(Vec8& a, Vec8& b, const float (&c)[8],
                                        const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a0 = bf16_lo(a.w[i]), a1 = bf16_hi(a.w[i]);
    const float b0 = bf16_lo(b.w[i]), b1 = bf16_hi(b.w[i]);
    a.w[i] = pack_bf16x2(a0 * c[2 * i] - b0 * s[2 * i], a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
    b.w[i] = pack_bf16x2(b0 * c[2 * i] + a0 * s[2 * i], b1 * c[2 * i + 1] + a1 * s[2 * i + 1]);
  }
}

// kInter false: halves with rotary_dim / 2 a multiple of 8 (pairs of vectors);
// true: adjacent pairs (within a vector). `parts` warps share a token.
template <bool kInter>
__global__ void __launch_bounds__(kThreads, 4) rope_warp_kernel(const RopeWriteParams p,
                                                                const int parts) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = p.head_dim, H = p.num_heads, Hkv = p.num_kv_heads;
  const int half = p.rotary_dim / 2;
  const int pad = (half + 3) & ~3;
  uint64_t* frac = reinterpret_cast<uint64_t*>(smem);                     // [pad]
  float* cs = reinterpret_cast<float*>(frac + pad) + warp * 2 * pad;      // cos [pad], sin [pad]
  float* sn = cs + pad;
  griddep_wait();
  griddep_launch_dependents();
  int lost = 0;  // whether some frequency is no number
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double f = __ldg(p.inv_freq + i);
    frac[i] = turn_fraction(f);
    lost |= no_number(f);
  }
  lost = __syncthreads_or(lost);
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
    auto in_of = [&](int h) { return h < H ? q + h * D : k + (h - H) * D; };
    auto out_of = [&](int h) { return h < H ? qo + h * D : ko + (h - H) * D; };

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
    if (!kInter) {
      const int U = half / 8;                // vector pairs per head
      const int P = (D - p.rotary_dim) / 8;  // vectors per head that pass through
      const int step = 32 / U;               // heads at a time (U is at most 32)
      const int u = lane % U;
      if (lane < step * U) {
        float c[8], s[8];
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          *reinterpret_cast<float4*>(c + i) = *reinterpret_cast<const float4*>(cs + u * 8 + i);
          *reinterpret_cast<float4*>(s + i) = *reinterpret_cast<const float4*>(sn + u * 8 + i);
        }
        constexpr int B = 2;  // loads of so many heads in flight
        for (int h = h0 + lane / U; h < h1; h += B * step) {
          Vec8 a[B], b[B];
#pragma unroll
          for (int i = 0; i < B; ++i)
            if (h + i * step < h1) {
              const uint16_t* in = in_of(h + i * step) + u * 8;
              a[i] = load8(in);
              b[i] = load8(in + half);
            }
#pragma unroll
          for (int i = 0; i < B; ++i)
            if (h + i * step < h1) {
              uint16_t* out = out_of(h + i * step) + u * 8;
              rotate8(a[i], b[i], c, s);
              store8(out, a[i]);
              store8(out + half, b[i]);
            }
        }
      }
      for (int i = lane; i < (h1 - h0) * P; i += 32) {
        const int h = h0 + i / P, o = p.rotary_dim + (i % P) * 8;
        store8(out_of(h) + o, load8(in_of(h) + o));
      }
    } else {
      // lane v of a head's V vectors, as many heads at a time as fit the warp
      const int V = D / 8;
      const int step = V < 32 ? 32 / V : 1;
      const int v0 = V < 32 ? lane % V : lane;
      for (int u = v0; u < V && (V >= 32 || lane < step * V); u += 32) {
        float c[4], s[4];  // of the vector's pairs; a pair past the rotated ones is left alone
        const int pairs = min(4, max(0, half - u * 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          c[e] = e < pairs ? cs[u * 4 + e] : 1.f;
          s[e] = e < pairs ? sn[u * 4 + e] : 0.f;
        }
        constexpr int B = 4;
        for (int h = h0 + (V < 32 ? lane / V : 0); h < h1; h += B * step) {
          Vec8 a[B];
#pragma unroll
          for (int i = 0; i < B; ++i)
            if (h + i * step < h1) a[i] = load8(in_of(h + i * step) + u * 8);
#pragma unroll
          for (int i = 0; i < B; ++i)
            if (h + i * step < h1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float y = bf16_lo(a[i].w[e]), z = bf16_hi(a[i].w[e]);
                const uint32_t r = pack_bf16x2(y * c[e] - z * s[e], z * c[e] + y * s[e]);
                if (e < pairs) a[i].w[e] = r;
              }
              store8(out_of(h + i * step) + u * 8, a[i]);
            }
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

// Halves of any length: one CTA per token, whose heads are staged in shared
// memory so that each output vector gathers its partners (and q_out may be q).
__global__ void __launch_bounds__(kThreads) rope_staged_kernel(const RopeWriteParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x;
  const int D = p.head_dim, H = p.num_heads, Hkv = p.num_kv_heads;
  const int half = p.rotary_dim / 2;
  const int pad = (half + 3) & ~3;
  float* cs = reinterpret_cast<float*>(smem);  // cos [pad], sin [pad]
  float* sn = cs + pad;
  uint16_t* st = reinterpret_cast<uint16_t*>(sn + pad);  // [heads][D]
  const int32_t pos = __ldg(p.positions + t);
  const int64_t slot = __ldg(p.slots + t);
  if (pos < 0) {  // uniform: the token is skipped
    if (threadIdx.x == 0) set_status(p.status, PKV_DEV_BAD_POSITION);
    return;
  }
  const bool write = slot >= 0 && slot < p.num_slots;
  if (!write && slot != -1 && threadIdx.x == 0) set_status(p.status, PKV_DEV_BAD_SLOT);
  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double f = __ldg(p.inv_freq + i);
    const float2 a = rope_angle(turn_fraction(f), (uint32_t)pos, p.factor);
    cs[i] = no_number(f) ? __uint_as_float(kNan) : a.x;
    sn[i] = no_number(f) ? __uint_as_float(kNan) : a.y;
  }
  const uint16_t* q = p.q + (int64_t)t * p.q_stride;
  const uint16_t* k = p.k + (int64_t)t * p.k_stride;
  uint16_t* qo = p.q_out + (int64_t)t * H * D;
  const int64_t row = (int64_t)Hkv * D;
  uint16_t* ko = static_cast<uint16_t*>(p.pool) + (write ? slot : 0) * row;
  const int heads = write ? H + Hkv : H;
  const int V = D / 8;  // vectors per head
  if (write) {
    const uint16_t* v = p.v + (int64_t)t * p.v_stride;
    uint16_t* vo = ko + p.num_slots * row;
    for (int i = threadIdx.x; i < Hkv * V; i += kThreads) store8(vo + i * 8, load8(v + i * 8));
  }
  for (int i = threadIdx.x; i < heads * V; i += kThreads)
    store8(st + i * 8, load8(i < H * V ? q + i * 8 : k + (i - H * V) * 8));
  __syncthreads();
  for (int i = threadIdx.x; i < heads * V; i += kThreads) {
    const int o = (i % V) * 8;
    Vec8 a = load8(st + i * 8);
    const uint16_t* head = st + i * 8 - o;
    auto turn = [&](int d, uint32_t bits) {  // dimension d, its bf16 bits
      if (d >= 2 * half) return bits;
      const int pr = d < half ? d : d - half;
      const float x = __uint_as_float(bits << 16);
      const float y = __uint_as_float((uint32_t)head[d < half ? d + half : pr] << 16);
      const float r = d < half ? x * cs[pr] - y * sn[pr] : x * cs[pr] + y * sn[pr];
      return pack_bf16x2(r, 0.f) & 0xffffu;
    };
#pragma unroll
    for (int j = 0; j < 4; ++j)
      a.w[j] = turn(o + 2 * j, a.w[j] & 0xffffu) | (turn(o + 2 * j + 1, a.w[j] >> 16) << 16);
    store8(i < H * V ? qo + i * 8 : ko + (i - H * V) * 8, a);
  }
}

cudaLaunchConfig_t config(int64_t ctas, size_t smem, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

cudaError_t launch_rope_write(const RopeWriteParams& p, cudaStream_t stream) {
  const int half = p.rotary_dim / 2;
  const size_t pad = (size_t)((half + 3) & ~3);
  cudaLaunchAttribute attr[1];
  if (!p.interleaved && half % 8 != 0) {
    const size_t smem = pad * 8 + (size_t)(p.num_heads + p.num_kv_heads) * p.head_dim * 2;
    if (smem > 48 * 1024) {
      static SmemLimit limit;
      cudaError_t e = limit.ensure(reinterpret_cast<const void*>(rope_staged_kernel), 200 * 1024);
      if (e != cudaSuccess) return e;
    }
    const cudaLaunchConfig_t cfg = config(p.num_tokens, smem, stream, attr);
    return cudaLaunchKernelEx(&cfg, rope_staged_kernel, p);
  }
  // warps per token: enough to spread a step over the GPU, no more than leave
  // a warp about four heads
  const int heads = p.num_heads + p.num_kv_heads;
  int parts = 1;
  while (parts < 16 && parts * 8 <= heads && (int64_t)p.num_tokens * parts < 152 * 16) parts *= 2;
  const int64_t units = (int64_t)p.num_tokens * parts;
  int64_t ctas = (units + kWarps - 1) / kWarps;
  // CTAs that stay for several tokens share the fractions of a turn (8192
  // tokens, 32 + 8 heads of 128: 47 us with a CTA a token, 35 us this way)
  const int64_t most = 152 * 8;
  if (ctas > most) ctas = most;
  const size_t smem = pad * 8 + kWarps * 2 * pad * sizeof(float);
  const cudaLaunchConfig_t cfg = config(ctas, smem, stream, attr);
  return p.interleaved ? cudaLaunchKernelEx(&cfg, rope_warp_kernel<true>, p, parts)
                       : cudaLaunchKernelEx(&cfg, rope_warp_kernel<false>, p, parts);
}

}  // namespace pkv
