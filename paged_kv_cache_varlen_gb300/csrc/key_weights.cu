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
// A warp takes a run of 16-key tiles of one (request, KV head): the tile's K
// rows are the A operand of mma.m16n8k16, straight from global memory into
// registers. The order of the dimensions inside a dot product is free as long
// as both operands agree, so a lane's 16-byte vector (8 consecutive
// dimensions of a row) serves as the A fragments of two MMAs and no shared
// memory or transposition is needed. The next tile's loads go out as soon as
// the MMAs have taken this one's registers, before its exponentials. K is read
// once; single-token steps are bound by that read.
// Measured (32 query and 8 KV heads of 128): 64 contexts of 512 to 4096 keys
// 49.5 us, 6.3 TB/s (92 % of the measured copy rate); 8 contexts of 32K to 128K
// 236 us, 6.7 TB/s (98 %). The same with the tile staged by TMA, four 4 KB
// slots a warp: 66.7 and 280 us (a third of the warps fit); with the next tile
// in a second set of registers: 57.4 and 257 us. Steps of 4 and 8 tokens over
// contexts like the first ones (16 and 32 columns): 55 and 81 us; 64 single
// tokens of 256 heads on one KV head of 64 (128) dimensions, whose Q is read
// again for every 16 keys: 108 (125) us.
#include <math.h>

#include "key_weights.cuh"

namespace pkv {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kWarps = 4;
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes that no other warp reads again.
__device__ __forceinline__ uint4 ld_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// NT: 8-column tiles held in registers at a time; ONE: every column of a
// request fits in them (single tokens and short steps), so Q is loaded once;
// LOOP: a warp goes on to further units of its head (without, it has one: 13
// registers fewer, 49.5 us for 56.3 on the first batch above).
template <int D, int NT, bool ONE, bool LOOP>
__global__ void __launch_bounds__(kWarps * 32)
    key_weights_kernel(const KeyWeightsParams p, const int chunk) {
  // Behind the tcgen05 grid of the same call (which started once everything
  // before it had finished) the CTAs do not wait for it, so that they fill the
  // SMs it leaves; those of one extra slice do, and with them this grid's
  // completion.
  if (!p.after_tc || blockIdx.y == p.num_seqs) griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.y == p.num_seqs) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // a warp's units are the same head's: the stride is a multiple of the heads
  const int unit = blockIdx.x * kWarps + warp, stride = gridDim.x * kWarps;
  const int h = unit % p.num_kv_heads;
  int key0 = (unit / p.num_kv_heads) * chunk;
  const int step = stride / p.num_kv_heads * chunk;
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
  const int32_t* table = p.block_table + (int64_t)i * p.max_blocks;
  float* out = p.out + ((int64_t)r.row * p.num_kv_heads + h) * p.row_len;
  const float* in = p.in + ((int64_t)r.row * p.num_kv_heads + h) * p.row_len;

  int32_t ids = -1;  // block ids of the chunk's 16-key tiles, one a lane
  uint4 ka[KB], kb[KB];  // rows row and row + 8 of a tile
  auto fetch = [&](int t) {
    const int32_t id = __shfl_sync(kFull, ids, t);
    if (id < 0) return;  // not in the pool: computed on what is there, not stored
    const uint16_t* src =
        p.pool + (((int64_t)id * p.block_size + (key0 + t * 16) % p.block_size + row) *
                      p.num_kv_heads + h) * D + quad * 8;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      ka[b] = ld_once(src + b * 32);
      kb[b] = ld_once(src + (int64_t)8 * p.num_kv_heads * D + b * 32);
    }
  };
  // c += K (16 keys) Q^T (8 columns of tile n)
  auto scores = [&](int n, float (&c)[4]) {
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      mma_bf16(c, ka[b].x, kb[b].x, ka[b].y, kb[b].y, qf[n][b].x, qf[n][b].y);
      mma_bf16(c, ka[b].z, kb[b].z, ka[b].w, kb[b].w, qf[n][b].z, qf[n][b].w);
    }
  };
  auto weights = [&](int n, const float (&c)[4], int k0, float& s0, float& s1) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float w0 = fast_exp2(fmaf(c[e], p.scale_log2, -lse2[n][e]));
      const float w1 = fast_exp2(fmaf(c[2 + e], p.scale_log2, -lse2[n][e]));
      s0 += k0 + row <= last[n][e] ? w0 : 0.f;
      s1 += k0 + row + 8 <= last[n][e] ? w1 : 0.f;
    }
  };
#pragma unroll
  for (int b = 0; b < KB; ++b) ka[b] = kb[b] = make_uint4(0, 0, 0, 0);
  if (ONE && LOOP) load_columns(0);
  do {
    const int tiles = (min(chunk, r.L - key0) + 15) / 16;
    ids = lane < tiles ? __ldg(table + (key0 + lane * 16) / p.block_size) : -1;
    const bool lost = lane < tiles && (ids < 0 || ids >= p.num_blocks);
    if (lost) ids = -1;
    if (__any_sync(kFull, lost) && lane == 0) set_status(p.status, PKV_DEV_BAD_BLOCK);
    fetch(0);
    if (ONE && !LOOP) load_columns(0);
    for (int t = 0; t < tiles; ++t) {
      const int k0 = key0 + t * 16;
      const bool there = __shfl_sync(kFull, ids, t) >= 0;
      const int key = k0 + row + quad * 8;
      const bool mine = there && quad < 2 && key < r.L;
      float before = 0.f;
      if (mine && key < r.prior && p.decay != 0.f) before = p.decay * in[key];
      float s0 = 0.f, s1 = 0.f;  // keys k0 + row, k0 + row + 8
      if (ONE) {
        float c[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
          scores(n, c[n]);
        }
        if (t + 1 < tiles) fetch(t + 1);
#pragma unroll
        for (int n = 0; n < NT; ++n) weights(n, c[n], k0, s0, s1);
      } else {
        // From the first column group that sees the tile's first key. The sums
        // of 64 groups are added up apart, so that no chain is longer than 256
        // additions and one for every 1024 columns (a single one drifts: equal
        // addends round to the same side for a whole octave of the sum; 2000
        // queries of 256 heads were off by 9e-4).
        float all0 = 0.f, all1 = 0.f;
        for (int c0 = max(0, k0 - qpos0) * G / (NT * 8) * (NT * 8); c0 < cols; c0 += NT * 8) {
          load_columns(c0);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            scores(n, c);
            weights(n, c, k0, s0, s1);
          }
          if ((c0 / (NT * 8) & 63) == 63) {
            all0 += s0;
            all1 += s1;
            s0 = s1 = 0.f;
          }
        }
        s0 += all0;
        s1 += all1;
        if (t + 1 < tiles) fetch(t + 1);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        s0 += __shfl_xor_sync(kFull, s0, o);
        s1 += __shfl_xor_sync(kFull, s1, o);
      }
      if (mine) out[key] = before + (quad ? s1 : s0);
    }
    key0 += step;
  } while (LOOP && key0 < r.L);
}

template <int D, int NT, bool ONE, bool LOOP = false>
cudaError_t launch(const KeyWeightsParams& p, cudaStream_t stream) {
  // Keys of a warp's unit: 128 amortise its start (64 x 512-4096 keys, 8 KV
  // heads: 49.5 us; 64 keys 50.3, 256 54.2); fewer while that leaves less
  // than about two units for each of the GPU's resident warps (13 requests of
  // up to 5000 keys, 4 KV heads, beside chunks: 66.0 us with 64, 69.4 with 128).
  int chunk = 128;
  auto units_of = [&](int c) { return ((int64_t)p.max_seq_len + c - 1) / c * p.num_kv_heads; };
  while (chunk > 16 && units_of(chunk) * p.num_seqs < 8192) chunk /= 2;
  const int64_t units = units_of(chunk);
  int64_t ctas = (units + kWarps - 1) / kWarps;
  if constexpr (ONE && !LOOP) {
    // max_seq_len may be far above the requests' lengths: past so many CTAs,
    // fewer of them go on to further units (64 x 512-4096 keys under a bound
    // of 131072: 57 us, 141 with a warp for each unit in bounds)
    if (ctas * p.num_seqs > 32768) return launch<D, NT, ONE, true>(p, stream);
  }
  if (LOOP) {
    const int64_t hkv = p.num_kv_heads;
    ctas = 8192 / p.num_seqs > 0 ? 8192 / p.num_seqs : 1;
    ctas = (ctas + hkv - 1) / hkv * hkv;  // a warp's stride is a multiple of the heads
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)p.num_seqs + (p.after_tc ? 1u : 0u));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_kernel<D, NT, ONE, LOOP>, p, chunk);
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
