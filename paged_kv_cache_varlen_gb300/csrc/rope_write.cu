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
// product that wraps by itself: off by at most |m| (2^-53 |f| / 2 pi + 2^-64)
// turns. Its top 32 bits become the argument of sincospif.
//
// Bound: every byte moves once (q, k, v in, q_out and the pool's rows out):
// HBM for prompts, launch and memory latency for single tokens. One CTA per
// token; a thread keeps one group of 8 pairs for all its heads, so their
// sines and cosines stay in registers (head halves), and moves 16-byte vectors.
#include "common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;

// cos and sin of pos * inv_freq, times factor.
__device__ __forceinline__ float2 rope_angle(double inv_freq, uint32_t pos, float factor) {
  const double turns = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
  const uint64_t frac = __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
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

// kMode 0: halves with rotary_dim / 2 a multiple of 8 (pairs of vectors);
// 1: adjacent pairs (within a vector); 2: halves of any length, the token's
// heads staged in shared memory so that each output vector gathers its
// partners (and q_out may be q).
template <int kMode>
__global__ void __launch_bounds__(kThreads) rope_write_kernel(const RopeWriteParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x;
  const int D = p.head_dim, H = p.num_heads, Hkv = p.num_kv_heads;
  const int half = p.rotary_dim / 2;
  float* cs = reinterpret_cast<float*>(smem);  // cos [half], sin [half], 16-byte aligned each
  const int hpad = (half + 3) & ~3;
  float* sn = cs + hpad;

  const int32_t pos = __ldg(p.positions + t);
  const int64_t slot = __ldg(p.slots + t);
  if (pos < 0) {  // uniform: the token is skipped
    if (threadIdx.x == 0) set_status(p.status, PKV_DEV_BAD_POSITION);
    return;
  }
  const bool write = slot >= 0 && slot < p.num_slots;
  if (!write && slot != -1 && threadIdx.x == 0) set_status(p.status, PKV_DEV_BAD_SLOT);

  for (int i = threadIdx.x; i < half; i += kThreads) {
    const float2 a = rope_angle(__ldg(p.inv_freq + i), (uint32_t)pos, p.factor);
    cs[i] = a.x;
    sn[i] = a.y;
  }

  const uint16_t* q = p.q + (int64_t)t * p.q_stride;
  const uint16_t* k = p.k + (int64_t)t * p.k_stride;
  uint16_t* qo = p.q_out + (int64_t)t * H * D;
  const int64_t row = (int64_t)Hkv * D;
  uint16_t* ko = static_cast<uint16_t*>(p.pool) + slot * row;  // used only when `write`
  const int heads = write ? H + Hkv : H;

  if (write) {
    const uint16_t* v = p.v + (int64_t)t * p.v_stride;
    uint16_t* vo = ko + p.num_slots * row;
    for (int i = threadIdx.x; i < Hkv * D / 8; i += kThreads) store8(vo + i * 8, load8(v + i * 8));
  }

  if (kMode == 0) {
    __syncthreads();
    const int U = half / 8;                 // vector pairs per head
    const int P = (D - p.rotary_dim) / 8;   // vectors per head that pass through
    const int u = threadIdx.x % U, step = kThreads / U;
    if (threadIdx.x < step * U) {
      float c[8], s[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = cs[u * 8 + i];
        s[i] = sn[u * 8 + i];
      }
      for (int h = threadIdx.x / U; h < heads; h += step) {
        const uint16_t* in = h < H ? q + h * D : k + (h - H) * D;
        uint16_t* out = h < H ? qo + h * D : ko + (h - H) * D;
        Vec8 a = load8(in + u * 8), b = load8(in + half + u * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a0 = bf16_lo(a.w[i]), a1 = bf16_hi(a.w[i]);
          const float b0 = bf16_lo(b.w[i]), b1 = bf16_hi(b.w[i]);
          a.w[i] = pack_bf16x2(a0 * c[2 * i] - b0 * s[2 * i],
                               a1 * c[2 * i + 1] - b1 * s[2 * i + 1]);
          b.w[i] = pack_bf16x2(b0 * c[2 * i] + a0 * s[2 * i],
                               b1 * c[2 * i + 1] + a1 * s[2 * i + 1]);
        }
        store8(out + u * 8, a);
        store8(out + half + u * 8, b);
      }
    }
    for (int i = threadIdx.x; i < heads * P; i += kThreads) {
      const int h = i / P, o = p.rotary_dim + (i % P) * 8;
      store8((h < H ? qo + h * D : ko + (h - H) * D) + o,
             load8((h < H ? q + h * D : k + (h - H) * D) + o));
    }
  } else {
    const int V = D / 8;  // vectors per head
    uint16_t* st = reinterpret_cast<uint16_t*>(sn + hpad);  // kMode 2: [heads][D]
    if (kMode == 2) {
      for (int i = threadIdx.x; i < heads * V; i += kThreads)
        store8(st + i * 8, load8(i < H * V ? q + i * 8 : k + (i - H * V) * 8));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < heads * V; i += kThreads) {
      const int o = (i % V) * 8;
      const bool isq = i < H * V;
      uint16_t* out = isq ? qo + i * 8 : ko + (i - H * V) * 8;
      Vec8 a = load8(kMode == 2 ? st + i * 8 : (isq ? q + i * 8 : k + (i - H * V) * 8));
      if (kMode == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pr = o / 2 + j;  // the pair's index
          if (pr < half) {
            const float x = bf16_lo(a.w[j]), y = bf16_hi(a.w[j]);
            a.w[j] = pack_bf16x2(x * cs[pr] - y * sn[pr], y * cs[pr] + x * sn[pr]);
          }
        }
      } else {
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
      }
      store8(out, a);
    }
  }
}

SmemLimit g_limit2;

}  // namespace

cudaError_t launch_rope_write(const RopeWriteParams& p, cudaStream_t stream) {
  const int half = p.rotary_dim / 2;
  const int mode = p.interleaved ? 1 : (half % 8 == 0 ? 0 : 2);
  size_t smem = (size_t)((half + 3) & ~3) * 2 * sizeof(float);
  if (mode == 2) {
    smem += (size_t)(p.num_heads + p.num_kv_heads) * p.head_dim * 2;
    if (smem > 48 * 1024) {
      cudaError_t e = g_limit2.ensure(reinterpret_cast<const void*>(rope_write_kernel<2>),
                                      200 * 1024);
      if (e != cudaSuccess) return e;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.num_tokens);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (mode == 0) return cudaLaunchKernelEx(&cfg, rope_write_kernel<0>, p);
  if (mode == 1) return cudaLaunchKernelEx(&cfg, rope_write_kernel<1>, p);
  return cudaLaunchKernelEx(&cfg, rope_write_kernel<2>, p);
}

}  // namespace pkv
