// cache_q8.cu -- the 8-bit key/value cache: quantising rows as they are
// written (prompts, single tokens, the accepted rows of a draft tree) and
// reading positions back as bf16.
//
// Mathematics.  A block of tokens of one kv head holds code * 2^e with e4m3
// codes.  Writing takes the smallest e with amax <= 448 * 2^e over the block's
// new rows; amax is a bf16 number 1.m * 2^x, so e = x - 8 when 1.m <= 1.75 and
// x - 7 above: integer arithmetic on its bits.  A block that had tokens keeps
// max(e, old e) and rounds its older codes once more if that grew: the scales
// are powers of two, so only codes that become e4m3 subnormals lose bits.
//
// Layout.  One unit of work is (block, kv head, K or V): block x d elements,
// held in registers (16 rows a warp, so a block of 16 needs no shared memory
// and one of 128 takes a CTA), loaded once, reduced to amax, converted and
// stored: each input byte is read once and each code written once, which is
// what bounds a prompt (3 bytes per element); a single token is a launch's
// latency.  Measured: 4 prompts of up to 8192 tokens, 8 heads of 128, written
// and read back in 61 us (0.87 of the copy rate), 8 contexts of up to 32768
// tokens read in 209 .. 219 us (0.96 .. 1.0 of it); both were bound by their
// issue slots (80 us, 232 us) until magnitudes and multiplies went two at a time.
#include "launch.h"
#include "q8_common.cuh"

namespace ddt {
namespace {

constexpr int kThreads = 256;

struct WriteParams {
  Q8View c;
  const uint4 *k_new, *v_new;  // [batch][n_max][hkv][d] bf16
  const int32_t* n_new;        // null: n_max
  const int32_t* acc_len;      // commit: rows = acc_len + 1 (n_new unused)
  const int32_t* acc_nodes;    // commit: [batch][L]
  int L;
  const int32_t* ctx_len;
  int32_t* ctx_len_out;
  int batch, n_max, units;     // units per sequence
  int32_t* status;
};

// Rows that sequence b gets (clamped); bad: the device value was out of range.
__device__ __forceinline__ int rows_of(const WriteParams& p, int b, bool* bad) {
  int n, most;
  if (p.acc_len) {
    n = p.acc_len[b] + 1;
    most = p.L + 1;
    *bad = n < 1 || n > most;
    return min(max(n, 1), most);
  }
  n = p.n_new ? p.n_new[b] : p.n_max;
  most = p.n_max;
  *bad = n < 0 || n > most;
  return min(max(n, 0), most);
}

template <int D, int BLOCK>
__global__ void __launch_bounds__(kThreads) write_q8_kernel(WriteParams p) {
  constexpr int CH = D / 8;               // 16-byte chunks of a bf16 row
  constexpr int TU = 32 * (BLOCK / 16);   // threads of a unit: 16 rows a warp
  constexpr int RP = TU / CH;             // rows a pass
  constexpr int NP = BLOCK / RP;          // passes: 8 (d = 128) or 4
  __shared__ uint32_t s_max[kThreads / 32];
  const int tid = threadIdx.x, b = blockIdx.y;
  const int unit = blockIdx.x * (kThreads / TU) + tid / TU;
  const int tu = tid % TU;
  pdl_wait();
  const int64_t ctx = p.ctx_len[b];
  bool bad;
  const int n = rows_of(p, b, &bad);
  if ((bad || ctx < 0) && blockIdx.x == 0 && tid == 0) raise_status(p.status, DDT_ERR_INVALID_ARG);
  const int hkv = p.c.hkv;
  const int h = unit % hkv, kv = (unit / hkv) & 1;
  const int64_t pos0 = ((ctx >> p.c.block_log2) + unit / (2 * hkv)) << p.c.block_log2;
  bool on = unit < p.units && ctx >= 0 && pos0 < ctx + n;
  // the rows are asked for before the place that they go to is looked up
  const int64_t limit = p.c.page_table ? ctx + n : p.c.t_max;
  const int64_t end = min(ctx + n, limit);
  const uint4* src = (kv ? p.v_new : p.k_new) + ((int64_t)b * p.n_max * hkv + h) * CH + tu % CH;
  uint4 x[NP];
  uint32_t fresh = 0, older = 0;  // bit i: pass i holds a new row / an older code
  uint32_t amax = 0;  // the largest magnitudes' bits, of even and odd elements
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int64_t pos = pos0 + tu / CH + i * RP;
    x[i] = make_uint4(0, 0, 0, 0);
    if (on && pos < min(ctx, limit)) {
      older |= 1u << i;
    } else if (on && pos < end) {
      int64_t r = pos - ctx;
      if (p.acc_len && r > 0) r = p.acc_nodes[(int64_t)b * p.L + r - 1];
      if (r >= 0 && r < p.n_max) {
        fresh |= 1u << i;
        x[i] = ld_stream_v4(src + r * hkv * CH);
      } else if (tu % CH == 0) {
        raise_status(p.status, DDT_ERR_INVALID_ARG);
      }
    }
  }
  Q8Place at{-1, -1};
  if (on) {
    at = q8_place(p.c, b, pos0);
    if (at.row < 0) {
      if (tu == 0) raise_status(p.status, DDT_ERR_INVALID_ARG);
      on = false;
      fresh = 0;
    }
  }
  if (on && end < ctx + n && pos0 + BLOCK > end && tu == 0)
    raise_status(p.status, DDT_ERR_INVALID_ARG);  // a dense block cut off by t_max
  uint8_t* codes = (kv ? p.c.vc : p.c.kc) + (at.row * hkv + h) * D + (tu % CH) * 8;
  int8_t* exps = (kv ? p.c.ve : p.c.ke) + at.blk * hkv + h;
  const bool had = on && pos0 < ctx;
  const int e_was = had ? *exps : DDT_Q8_EXP_MIN;
  const int e_old = q8_exp(e_was);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    amax = max_bf16x2(max_bf16x2(max_bf16x2(max_bf16x2(amax, x[i].x), x[i].y), x[i].z), x[i].w);
  }
  amax = max_bf16(amax);
  // bit 31: some row is new (so that an all-zero block still gets its exponent)
  amax = __reduce_max_sync(0xFFFFFFFFu, amax | (fresh ? 0x80000000u : 0u));
  if (TU > 32) {
    if ((tid & 31) == 0) s_max[tid / 32] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TU / 32; ++w) amax = max(amax, s_max[tid / TU * (TU / 32) + w]);
  }
  pdl_trigger();
  if (!(amax >> 31)) return;
  amax &= 0x7FFFu;
  const bool nan = amax >= 0x7F80u || e_was == DDT_Q8_EXP_NAN;
  // amax = 1.m * 2^(E - 127): 448 = 1.75 * 2^8 and 1.75 is m = 96 of 128
  int e = amax ? (int)(amax >> 7) - 127 - ((amax & 0x7Fu) <= 96u ? 8 : 7) : DDT_Q8_EXP_MIN;
  e = min(max(e, DDT_Q8_EXP_MIN), DDT_Q8_EXP_MAX);
  e = max(e, e_old);
  const float inv = pow2i(-e);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    if (!((fresh >> i) & 1u)) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float lo, hi;
      unpack2(fmul2(pack2(bf16_lo(w[q]), bf16_hi(w[q])), pack2(inv, inv)), lo, hi);
      c[q] = nan ? 0u : f32x2_to_e4m3x2(lo, hi);
    }
    *(uint2*)(codes + (int64_t)(tu / CH + i * RP) * hkv * D) =
        make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  }
  if (e > e_old && older && !nan) {
    const float down = pow2i(e_old - e);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (!((older >> i) & 1u)) continue;
      uint2* at_c = (uint2*)(codes + (int64_t)(tu / CH + i * RP) * hkv * D);
      const uint2 o = *at_c;
      const uint32_t w[2] = {o.x, o.y};
      uint32_t c[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float2 a = f16x2_to_f32x2(codes_lo(w[q])), z = f16x2_to_f32x2(codes_hi(w[q]));
        c[q] = f32x2_to_e4m3x2(a.x * down, a.y * down) | (f32x2_to_e4m3x2(z.x * down, z.y * down) << 16);
      }
      *at_c = make_uint2(c[0], c[1]);
    }
  }
  if (tu == 0) *exps = (int8_t)(nan ? DDT_Q8_EXP_NAN : e);
}

__global__ void __launch_bounds__(kThreads) advance_kernel(WriteParams p) {
  const int b = blockIdx.x * kThreads + threadIdx.x;
  pdl_wait();
  pdl_trigger();
  if (b >= p.batch) return;
  bool bad;
  p.ctx_len_out[b] = p.ctx_len[b] + rows_of(p, b, &bad);
}

struct ReadParams {
  Q8View c;
  const int32_t *ctx_len, *first;
  uint4 *k_out, *v_out;
  int n_max, rows;            // output rows of a sequence, of a CTA
  int32_t* status;
};

constexpr int kReadRows = 32;  // output rows of a CTA, at most

// 8 codes -> 8 bf16; s: the block's scale.
__device__ __forceinline__ uint4 decode8(uint2 c, float s) {
  const uint32_t w[2] = {c.x, c.y};
  uint32_t o[4];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const float2 a = f16x2_to_f32x2(codes_lo(w[q])), z = f16x2_to_f32x2(codes_hi(w[q]));
    float b[4];
    unpack2(fmul2(pack2(a.x, a.y), pack2(s, s)), b[0], b[1]);
    unpack2(fmul2(pack2(z.x, z.y), pack2(s, s)), b[2], b[3]);
    o[2 * q] = f32x2_to_bf16x2(b[0], b[1]);
    o[2 * q + 1] = f32x2_to_bf16x2(b[2], b[3]);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kThreads) read_q8_kernel(ReadParams p) {
  __shared__ Q8Place s_at[kReadRows];
  const int tid = threadIdx.x, b = blockIdx.y, kv = blockIdx.z;
  const int r0 = blockIdx.x * p.rows;
  pdl_wait();
  if (tid < p.rows) {
    Q8Place at{-1, -1};
    const int64_t first = p.first ? p.first[b] : 0;
    const int64_t pos = first + r0 + tid;
    if (r0 + tid < p.n_max) {
      if (first < 0 && r0 + tid == 0) raise_status(p.status, DDT_ERR_INVALID_ARG);
      if (pos >= 0 && pos < p.ctx_len[b]) {
        at = q8_place(p.c, b, pos);
        if (at.row < 0) raise_status(p.status, DDT_ERR_INVALID_ARG);
      }
    }
    s_at[tid] = at;
  }
  __syncthreads();
  pdl_trigger();
  const int vecs = p.c.hkv * p.c.d / 8;  // 8-code vectors of a row: a warp writes 512 bytes in a row
  const int head_log2 = p.c.d == 128 ? 4 : 3;
  const uint2* codes = (const uint2*)(kv ? p.c.vc : p.c.kc);
  const int8_t* exps = kv ? p.c.ve : p.c.ke;
  const int rows = min(p.rows, p.n_max - r0);
  const int items = rows * vecs;
  uint4* out = (kv ? p.v_out : p.k_out) + ((int64_t)b * p.n_max + r0) * vecs;
  constexpr int kFly = 8;  // vectors in flight per thread
  // item i = row r, vector x of it, stepped without divisions
  const int dr = kThreads / vecs, dx = kThreads % vecs;
  int r = tid / vecs, x = tid % vecs;
  for (int i0 = tid; i0 < items; i0 += kThreads * kFly) {
    uint2 v[kFly];
    int e[kFly];
#pragma unroll
    for (int q = 0; q < kFly; ++q) {
      v[q] = make_uint2(0, 0);
      e[q] = 0;
      if (r < rows) {
        const Q8Place at = s_at[r];
        if (at.row >= 0) {
          v[q] = __ldcs(codes + at.row * vecs + x);
          e[q] = __ldg(exps + at.blk * p.c.hkv + (x >> head_log2));
        }
      }
      r += dr;
      x += dx;
      if (x >= vecs) {
        x -= vecs;
        ++r;
      }
    }
#pragma unroll
    for (int q = 0; q < kFly; ++q) {
      const int i = i0 + q * kThreads;
      if (i < items) __stcs(out + i, decode8(v[q], q8_scale(e[q])));
    }
  }
}

template <int D>
cudaError_t launch_write(const WriteParams& p, int block, dim3 grid, cudaStream_t stream) {
  switch (block) {
    case 16: return launch_pdl(write_q8_kernel<D, 16>, grid, dim3(kThreads), 0, stream, 0, p);
    case 32: return launch_pdl(write_q8_kernel<D, 32>, grid, dim3(kThreads), 0, stream, 0, p);
    case 64: return launch_pdl(write_q8_kernel<D, 64>, grid, dim3(kThreads), 0, stream, 0, p);
    default: return launch_pdl(write_q8_kernel<D, 128>, grid, dim3(kThreads), 0, stream, 0, p);
  }
}

ddt_status run_write(WriteParams& p, const ddt_q8_cache* c, int max_rows, cudaStream_t stream) {
  // blocks that max_rows rows can touch from any starting position
  const int64_t blocks = ((int64_t)max_rows + c->block - 2) / c->block + 1;
  const int64_t units = blocks * 2 * c->hkv;
  if (units > INT32_MAX) return DDT_ERR_UNSUPPORTED;
  p.units = (int)units;
  const int per_cta = 128 / c->block;
  const dim3 grid((unsigned)((units + per_cta - 1) / per_cta), (unsigned)p.batch);
  const cudaError_t e = c->d == 128 ? launch_write<128>(p, c->block, grid, stream)
                                    : launch_write<64>(p, c->block, grid, stream);
  if (e != cudaSuccess) return DDT_ERR_CUDA;
  if (p.ctx_len_out) {
    if (launch_pdl(advance_kernel, dim3((p.batch + kThreads - 1) / kThreads), dim3(kThreads), 0, stream, 0,
                   p) != cudaSuccess)
      return DDT_ERR_CUDA;
  }
  return DDT_OK;
}

}  // namespace

Q8View q8_view(const ddt_q8_cache* c) {
  Q8View v;
  v.kc = (uint8_t*)c->k_cache;
  v.vc = (uint8_t*)c->v_cache;
  v.ke = c->k_exp;
  v.ve = c->v_exp;
  v.page_table = c->page_table;
  v.page_size = c->page_size;
  v.max_pages = c->max_pages;
  v.num_pages = c->num_pages;
  v.page_log2 = -1;
  for (int i = 0; i < 31; ++i)
    if (c->page_size == 1 << i) v.page_log2 = i;
  v.t_max = c->t_max;
  v.hkv = c->hkv;
  v.d = c->d;
  v.block_log2 = c->block == 16 ? 4 : c->block == 32 ? 5 : c->block == 64 ? 6 : 7;
  v.blocks_per = c->page_table ? c->page_size / c->block : (c->t_max + c->block - 1) / c->block;
  return v;
}

ddt_status launch_kv_append_q8(const ddt_kv_append_q8_args* a, cudaStream_t stream) {
  if (a->batch == 0) return DDT_OK;
  WriteParams p = {};
  p.c = q8_view(&a->cache);
  p.k_new = (const uint4*)a->k_new;
  p.v_new = (const uint4*)a->v_new;
  p.n_new = a->n_new;
  p.ctx_len = a->ctx_len;
  p.ctx_len_out = a->ctx_len_out;
  p.batch = a->batch;
  p.n_max = a->n_max;
  p.status = a->dev_status;
  return run_write(p, &a->cache, a->n_max, stream);
}

ddt_status launch_kv_commit_q8(const ddt_kv_commit_q8_args* a, cudaStream_t stream) {
  if (a->batch == 0) return DDT_OK;
  WriteParams p = {};
  p.c = q8_view(&a->cache);
  p.k_new = (const uint4*)a->k_tree;
  p.v_new = (const uint4*)a->v_tree;
  p.acc_len = a->acc_len;
  p.acc_nodes = a->acc_nodes;
  p.L = a->L;
  p.ctx_len = a->ctx_len;
  p.ctx_len_out = a->ctx_len_out;
  p.batch = a->batch;
  p.n_max = a->n_max;
  p.status = a->dev_status;
  return run_write(p, &a->cache, a->L + 1, stream);
}

ddt_status launch_kv_read_q8(const ddt_kv_read_q8_args* a, cudaStream_t stream) {
  if (a->batch == 0 || a->n_max == 0) return DDT_OK;
  ReadParams p;
  p.c = q8_view(&a->cache);
  p.ctx_len = a->ctx_len;
  p.first = a->first;
  p.k_out = (uint4*)a->k_out;
  p.v_out = (uint4*)a->v_out;
  p.n_max = a->n_max;
  p.status = a->dev_status;
  // 32 rows a CTA where that still gives every SM several (32 contexts of up to
  // 8192 tokens, 2 heads of 128: 80 us, 123 us with 16 and 209 us with 8 rows; 8
  // contexts of up to 32768 tokens, 8 heads: 219, 209 and 281 us), 8 where the
  // call is small
  const int64_t ctas = (int64_t)((a->n_max + kReadRows - 1) / kReadRows) * a->batch * 2;
  p.rows = ctas >= 8 * device_sm_count() ? kReadRows : kReadRows / 4;
  const dim3 grid((a->n_max + p.rows - 1) / p.rows, a->batch, 2);
  return launch_pdl(read_q8_kernel, grid, dim3(kThreads), 0, stream, 0, p) == cudaSuccess ? DDT_OK
                                                                                          : DDT_ERR_CUDA;
}

}  // namespace ddt
