// key_weights.cu -- the softmax weight that each cached key received in a
// step's attention, added to its running sum:
//
//   out[r][h][p] = (p < prior ? decay * in[r][h][p] : 0)
//     + sum over queries j with pos_j >= p, heads a of the KV head h, of
//       2^(scale log2e q[j][a] . K[p][h] - log2e lse[j][a]).
//
// The attention call has already reduced over the keys (its lse), so a key's
// sum needs nothing from other keys: keys are the rows of S^T = K Q^T, the
// (query, head) pairs its columns, and a key's sum runs along its own row.
//
// A warp takes 16-key tiles of one (request, KV head): the tile's K rows are
// the A operand of mma.m16n8k16, straight from global memory into registers.
// The order of the dimensions inside a dot product is free as long as both
// operands agree, so a lane's 16-byte vector (8 consecutive dimensions of a
// row) serves as the A fragments of two MMAs and no shared memory or
// transposition is needed. K is read once; single-token steps are bound by
// that read.
#include <math.h>

#include "key_weights.cuh"

namespace pkv {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kChunk = 128;  // keys of one warp's unit of work

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: 8-column tiles held in registers at a time; ONE: every column of a
// request fits in them (single tokens and short steps), so Q is loaded once.
template <int D, int NT, bool ONE>
__global__ void __launch_bounds__(kWarps * 32) key_weights_kernel(const KeyWeightsParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int h = unit % p.num_kv_heads;
  const int key0 = (unit / p.num_kv_heads) * kChunk;
  const int i = blockIdx.y;
  KeyRequest r;
  if (!key_request(p, i, unit == 0 && lane == 0, &r)) return;
  if (key0 >= r.L) return;
  const int G = p.num_heads / p.num_kv_heads;
  const int cols = r.qlen * G;
  if (ONE && cols > NT * 8) return;  // a longer step: the tcgen05 grid takes it
  const int qpos0 = r.L - r.qlen;
  const int row = lane >> 2, quad = lane & 3;
  constexpr int KB = D / 32;  // 32-dimension blocks of a row: one vector a lane
  uint4 qf[NT][KB];
  float lse2[NT][2];
  int last[NT][2];  // last key that the column sees, -1: no such column

  auto load_columns = [&](int c0) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int c = c0 + n * 8 + row;
      const bool in = c < cols;
      const int j = in ? c / G : 0;
      const uint16_t* q = p.q + ((int64_t)(r.t0 + j) * p.num_heads + h * G + (in ? c % G : 0)) * D;
#pragma unroll
      for (int b = 0; b < KB; ++b)
        qf[n][b] = in ? __ldg(reinterpret_cast<const uint4*>(q + b * 32 + quad * 8))
                      : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int ce = c0 + n * 8 + quad * 2 + e;
        float l = 0.f;
        int lim = -1;
        if (ce < cols) {
          const int je = ce / G;
          l = __ldg(p.lse + (int64_t)(r.t0 + je) * p.num_heads + h * G + ce % G);
          lim = l == -INFINITY ? -1 : qpos0 + je;
        }
        lse2[n][e] = l * kLog2e;
        last[n][e] = lim;
      }
    }
  };
  if (ONE) load_columns(0);

  // block ids of the chunk's 16-key tiles, one a lane
  const int32_t* table = p.block_table + (int64_t)i * p.max_blocks;
  int32_t ids = -1;
  if (lane < kChunk / 16 && key0 + lane * 16 < r.L)
    ids = __ldg(table + (key0 + lane * 16) / p.block_size);
  float* out = p.out + ((int64_t)r.row * p.num_kv_heads + h) * p.row_len;
  const float* in = p.in + ((int64_t)r.row * p.num_kv_heads + h) * p.row_len;
  bool bad = false;
  for (int t = 0; t < kChunk / 16; ++t) {
    const int k0 = key0 + t * 16;
    if (k0 >= r.L) break;
    const int32_t id = __shfl_sync(kFull, ids, t);
    if (id < 0 || id >= p.num_blocks) {
      bad = true;
      continue;
    }
    const uint16_t* k = p.pool + (((int64_t)id * p.block_size + k0 % p.block_size + row) *
                                      p.num_kv_heads + h) * D;
    uint4 ka[KB], kb[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      ka[b] = *reinterpret_cast<const uint4*>(k + b * 32 + quad * 8);
      kb[b] = *reinterpret_cast<const uint4*>(k + (int64_t)8 * p.num_kv_heads * D + b * 32 +
                                              quad * 8);
    }
    float s0 = 0.f, s1 = 0.f;  // keys k0 + row, k0 + row + 8
    // the first column group that sees the tile's first key
    const int c_first = ONE ? 0 : max(0, k0 - qpos0) * G / (NT * 8) * (NT * 8);
    for (int c0 = c_first; c0 < cols; c0 += NT * 8) {
      if (!ONE) load_columns(c0);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          mma_bf16(c, ka[b].x, kb[b].x, ka[b].y, kb[b].y, qf[n][b].x, qf[n][b].y);
          mma_bf16(c, ka[b].z, kb[b].z, ka[b].w, kb[b].w, qf[n][b].z, qf[n][b].w);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float w0 = fast_exp2(fmaf(c[e], p.scale_log2, -lse2[n][e]));
          const float w1 = fast_exp2(fmaf(c[2 + e], p.scale_log2, -lse2[n][e]));
          s0 += k0 + row <= last[n][e] ? w0 : 0.f;
          s1 += k0 + row + 8 <= last[n][e] ? w1 : 0.f;
        }
      }
      if (ONE) break;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      s0 += __shfl_xor_sync(kFull, s0, o);
      s1 += __shfl_xor_sync(kFull, s1, o);
    }
    if (quad < 2) {
      const int key = k0 + row + quad * 8;
      if (key < r.L) {
        const float s = quad ? s1 : s0;
        out[key] = key < r.prior && p.decay != 0.f ? fmaf(p.decay, in[key], s) : s;
      }
    }
  }
  if (bad && lane == 0) set_status(p.status, PKV_DEV_BAD_BLOCK);
}

template <int D, int NT, bool ONE>
cudaError_t launch(const KeyWeightsParams& p, cudaStream_t stream) {
  const int64_t units = ((int64_t)p.max_seq_len + kChunk - 1) / kChunk * p.num_kv_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units + kWarps - 1) / kWarps), (unsigned)p.num_seqs);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_kernel<D, NT, ONE>, p);
}

template <int D>
cudaError_t launch_d(const KeyWeightsParams& p, int64_t cols, cudaStream_t stream) {
  if (cols <= 8) return launch<D, 1, true>(p, stream);
  if (cols <= 16) return launch<D, 2, true>(p, stream);
  if (cols <= 32) return launch<D, 4, true>(p, stream);
  return launch<D, 2, false>(p, stream);
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams& p, cudaStream_t stream) {
  // columns of the longest request that this grid takes
  const int G = p.num_heads / p.num_kv_heads;
  int64_t cols = (int64_t)p.max_query_len * G;
  if (p.short_max_q > 0 && p.short_max_q < p.max_query_len) cols = (int64_t)p.short_max_q * G;
  return p.head_dim == 64 ? launch_d<64>(p, cols, stream) : launch_d<128>(p, cols, stream);
}

}  // namespace pkv
