// key_weights.cuh -- what the two key-weight kernels share: a request's
// checked lengths and the split of a batch between the kernels.
#pragma once

#include "common.cuh"
#include "launch.h"

namespace pkv {

struct KeyRequest {
  int t0, qlen, L, prior, row;
};

// A request's lengths, checked; false when it has no work (no queries, or
// inconsistent entries, flagged by the thread with `flag`).
__device__ __forceinline__ bool key_request(const KeyWeightsParams& p, int i, bool flag,
                                            KeyRequest* r) {
  const int32_t t0 = __ldg(p.cu_seqlens + i), t1 = __ldg(p.cu_seqlens + i + 1);
  const int32_t L = __ldg(p.seq_lens + i);
  const int32_t row = p.rows ? __ldg(p.rows + i) : i;
  const int32_t qlen = t1 - t0;
  if (t0 < 0 || t1 < t0 || t1 > p.num_tokens ||
      (qlen > 0 && (qlen > p.max_query_len || L < qlen || L > p.max_seq_len ||
                    L > p.max_blocks * p.block_size))) {
    if (flag) set_status(p.status, PKV_DEV_BAD_LENGTHS);
    return false;
  }
  if (qlen == 0) return false;
  if (row < 0 || row >= p.num_rows) {
    if (flag) set_status(p.status, PKV_DEV_BAD_ROW);
    return false;
  }
  const int32_t prior = p.prior_lens ? __ldg(p.prior_lens + i) : L - qlen;
  *r = KeyRequest{t0, qlen, L, prior, row};
  return true;
}

}  // namespace pkv
