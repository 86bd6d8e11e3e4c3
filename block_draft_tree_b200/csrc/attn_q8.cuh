// attn_q8.cuh -- parameters shared by the attention kernels over the 8-bit cache.
#pragma once

#include "q8_common.cuh"

namespace ddt {

struct AttnQ8Params {
  Q8View c;
  const uint16_t *q, *kt, *vt;
  const int32_t *ctx_len, *n_nodes;
  const uint32_t* mask;
  int max_ctx, batch, n_max, hq, g, W;
  float scale_log2;     // softmax scale * log2(e)
  uint16_t* out;
  float* lse_out;
  int32_t* status;
  int nsplit;
  int steps_per_split;  // steps of a KV split
  int box_rows;         // tokens of a TMA box of codes
  long long wait_cycles;  // bound of every wait on a copy
  float* part_o;        // [batch*hkv][nsplit][R][d], R = n_max * g
  float2* part_ml;      // [batch*hkv][nsplit][R]: (reference, sum)
};

// Live tree rows and context tokens of sequence b (clamped as ddt_tree_attn does).
__device__ __forceinline__ void attn_q8_lengths(const AttnQ8Params& p, int b, bool tell, int& n, int& T) {
  n = min(max(p.n_nodes[b], 1), p.n_max);
  T = p.ctx_len[b];
  if (T < 0 || T > p.max_ctx) {
    if (tell) raise_status(p.status, DDT_ERR_INVALID_ARG);
    T = min(max(T, 0), p.max_ctx);
  }
}

Q8View q8_view(const ddt_q8_cache* c);

}  // namespace ddt
