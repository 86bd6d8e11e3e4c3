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

// The (sequence, kv head) group of a block's z index: longest contexts first,
// so that the last blocks to start are short ones (measured on 16 trees of 129
// rows over 1024 .. 16384 tokens: 439 us in order, 380 us so).  Batches beyond
// kOrdered run in order.
constexpr int kOrdered = 256;
__device__ __forceinline__ int group_of(const AttnQ8Params& p, int z, int* s_pick) {
  if (p.batch == 1 || p.batch > kOrdered) return z;
  const int want = z / p.c.hkv;
  for (int t = threadIdx.x; t < p.batch; t += blockDim.x) {
    const int mine = p.ctx_len[t];
    int before = 0;
    for (int j = 0; j < p.batch; ++j) {
      const int other = __ldg(p.ctx_len + j);
      before += other > mine || (other == mine && j < t);
    }
    if (before == want) *s_pick = t;
  }
  __syncthreads();
  return *s_pick * p.c.hkv + z % p.c.hkv;
}

// What a converter thread of the wide kernel reads of KV tile `tile` (128 tokens)
// in pass q (0..7): token 32 (q / 2) + tok, tok < 32, of the tile.  Rows behind the
// context are never touched: a cache's length need not be a multiple of 16, so
// they may lie past its end.  left: the context's tokens from the thread's
// first one on; group_row: the first cache row of the token's group of 16 (-1: a
// page that is not there, or nothing of the context).
__host__ __device__ constexpr int q8_wide_left(int T, int tile, int tok) { return T - tile * 128 - tok; }
__host__ __device__ constexpr bool q8_wide_reads(int group_row, int q, int left) {
  return group_row >= 0 && (q >> 1) * 32 < left;
}

Q8View q8_view(const ddt_q8_cache* c);

}  // namespace ddt
