// attn_q8.cu -- tree attention over the 8-bit key/value cache, for few query
// rows per kv head (an ordinary decoding step, a small tree) and for every
// shape that the wide kernel does not serve.
//
// Mathematics.  With code c_j, exponents a_j (K) and e_j (V) of token j and
// s_j = scale * log2(e) * 2^a_j * (q . ck_j), the output is
//   sum_j 2^s_j 2^e_j cv_j / sum_j 2^s_j.
// The V exponents join the softmax's reference: with t_j = s_j + e_j and m a
// running bound on t_j, P_j = 2^(t_j - m) weighs the bare codes and the
// denominator adds P_j 2^-e_j.  So the codes meet the tensor cores as f16
// (exact: e4m3 is a subset of f16), scales cost one multiply-add per score,
// and P as f16 (11 bits, error 2^-11) keeps every block's share whatever its
// scale.  m lags the true maximum by up to 2^4 and P's range begins at 2^11 for
// a new maximum: weights reach 2^15 at most, and f16's subnormal step (2^-24)
// is 2^-35 of the maximum, below any sum over a long tail.  Queries become f16
// under a power of two per row, exact down to 2^-39 of the row's largest.
//
// What bounds it: with R <= 32 rows per kv head the K/V codes are read once
// for 2R multiply-adds each, so HBM.  A warp takes 32 tokens a step; its lane
// 0 copies the step's K and V codes by TMA into a private ring of two steps
// (12 warps an SM: 96 KB in flight), so no lane computes an address and no
// barrier joins the warps before the end.  The places and exponents of the
// next 16 steps are looked up by 32 lanes at once and handed out by shuffles.
// The products are S^T = K Q^T and O^T = V^T P^T, so that query rows are the
// m16n8k16's narrow side: 8 rows (a decoding step of 8 heads per kv head) pad
// nothing.  A lane reads its own fragments: for K, lane (g, c) holds tokens g,
// g + 8 and two 16-byte chunks, with the d index permuted alike in Q's
// fragments; for V, lane (g, c) holds tokens 2c, 2c+1, 8+2c, 9+2c and chunk g,
// whose pairs one byte permute interleaves for the conversion to f16;
// P^T turns between the products by movmatrix.
// Tree rows become f16 under a power of two per row, for K and V apart.
// Measured, calls in turn: one row of 32 ragged sequences of 1024 .. 32768 tokens,
// 32/8 heads, 64-token pages, 196 .. 210 us in several runs, 0.83 .. 0.89 of the
// copy rate; 4 x 131072 tokens, 16/1 heads, 35 us with the merge of 111 splits.
#include <algorithm>
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_q8.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace ddt {
cudaError_t launch_attn_q8_wide(const AttnQ8Params& p, int pairs, cudaStream_t stream);
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
}
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 2;             // steps in the ring of a warp
constexpr int kHalf = 16;              // tokens that share a place and an exponent
constexpr int kStep = 2 * kHalf;       // tokens of a step
constexpr float kSlack = 4.f;          // the reference moves when a score passes it by 2^4
constexpr float kHead = 11.f;          // P of a new maximum is 2^11
// Rows per kv head beyond which d = 128 takes the wide kernel (4 x 16384 tokens:
// 40 rows 90 us there and 100 us here, 80 rows 92 us and 137 us; 20 x 2736 tokens:
// 125 us and 76 us, 125 us and 131 us; up to 32 rows are one pass here).  So trees
// of few rows more than 32 in a large batch would be better off here; the rule
// looks at rows alone.
constexpr long kWideRows = 32;

// D += A (16x16, row) * B (16x8, col), f16 inputs, f32 accumulators.
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held as a fragment.
__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

template <int D, int NR>
struct Smem {
  static constexpr int kHalfBytes = kHalf * D;           // K (or V) codes of 16 tokens
  static constexpr int kStageBytes = 4 * kHalfBytes;     // K then V of a step
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kQ = 8 * NR * D * 2;              // Q's f16 fragments, [NR][D / 16][32 lanes] x 8 bytes
  static constexpr int kORow = D + 4;                    // f32 a row of a warp's O, padded
  static constexpr int kMerge = kWarps * 8 * NR * (kORow * 4 + 8);
  static constexpr int kBody = kRing > kMerge ? kRing : kMerge;  // 1024-byte aligned
  static constexpr int kTotal = 1024 + kBody + kQ + 8 * NR * 4 + kWarps * kStages * 8 + 16;
};

// Row qr of sequence b and kv head kvh: its place in q / out.
__device__ __forceinline__ int64_t row_index(const AttnQ8Params& p, int b, int kvh, int qr) {
  return ((int64_t)b * p.n_max + qr / p.g) * p.hq + kvh * p.g + qr % p.g;
}

template <int D, int NR>  // NR: tiles of 8 query rows
__global__ void __launch_bounds__(kThreads, NR <= 2 ? 3 : 2)
    attn_q8_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const AttnQ8Params p) {
  using S = Smem<D, NR>;
  constexpr int KH = D / 64;       // 16-byte chunks of a K row that a lane holds
  constexpr int NT = D / 16;       // m-tiles of O^T
  constexpr int RT = 8 * NR;       // query rows of a CTA
  constexpr int KS = D / 16;       // k-steps of QK
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* sQ = ring + S::kBody;
  float* sRow = (float*)(ring + S::kBody + S::kQ);  // score multiplier of each row
  uint64_t* bars = (uint64_t*)(sRow + RT);     // [kWarps][kStages]
  int* s_abort = (int*)(bars + kWarps * kStages);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int tile = blockIdx.x, split = blockIdx.y;
  const int R = p.n_max * p.g;
  const int q0 = tile * RT;
  uint64_t* full = bars + warp * kStages;
  if (tid == 0) *s_abort = 0;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  pdl_wait();
  const int grp = blockIdx.z;
  const int b = grp / p.c.hkv, kvh = grp % p.c.hkv;
  int n, T;
  attn_q8_lengths(p, b, tile == 0 && split == 0 && kvh == 0 && tid == 0, n, T);
  const int nhalf = (T + kHalf - 1) / kHalf;     // 16-token pieces of the context
  const int nctx = (T + kStep - 1) / kStep;
  const int nall = nctx + (n + kHalf - 1) / kHalf;  // then the tree, 16 rows a step
  const int lo = min(split * p.steps_per_split, nall);
  const int hi = min(lo + p.steps_per_split, nall);
  const bool dead = q0 >= n * p.g;  // every row past the tree
  const bool idle = dead || lo >= hi;
  const int chi = min(hi, nctx);
  const int64_t stride = (int64_t)p.c.hkv * D;

  // ---- context steps of this warp: lo + warp + it * kWarps, it < steps
  const int first = lo + warp;
  const int steps = idle || first >= chi ? 0 : (chi - first + kWarps - 1) / kWarps;
  // Lane l's look-up for iterations 16 k ..: half l & 1 of iteration 16 k + l / 2.
  // row: the half's first cache row (-1: none); ek, ev: its stored exponents.
  struct LookUp {
    int row, ek, ev;
  };
  auto look_up = [&](int k) -> LookUp {
    LookUp u{-1, 0, 0};
    const int it = 16 * k + (lane >> 1);
    const int half = 2 * (first + it * kWarps) + (lane & 1);
    if (it < steps && half < nhalf) {
      const Q8Place at = q8_place(p.c, b, (int64_t)half * kHalf);
      if (at.row < 0) {
        raise_status(p.status, DDT_ERR_INVALID_ARG);
      } else {
        u.row = (int)at.row;
        const int64_t e = at.blk * p.c.hkv + kvh;
        u.ek = __ldg(p.c.ke + e);
        u.ev = __ldg(p.c.ve + e);
      }
    }
    return u;
  };
  // What a K code counts for, and the V exponent: NaN for
  // a block of NaN, -inf for a half that is not there (its weights are then 0).
  auto k_scale = [](const LookUp& u) { return q8_scale(u.ek); };
  auto v_exp = [](const LookUp& u) {
    return u.row < 0 ? -INFINITY
                     : u.ev == DDT_Q8_EXP_NAN ? __int_as_float(0x7FC00000) : (float)q8_exp(u.ev);
  };
  unsigned char* my = ring + warp * kStages * S::kStageBytes;
  // Issue iteration `it` (its look-up in `row`) into its stage.
  auto copy = [&](int it, int row) {
    const int r0 = __shfl_sync(0xFFFFFFFFu, row, (it & 15) * 2);
    const int r1 = __shfl_sync(0xFFFFFFFFu, row, (it & 15) * 2 + 1);
    if (lane != 0) return;
    unsigned char* dst = my + it % kStages * S::kStageBytes;
    uint64_t* bar = &full[it % kStages];
    if (p.box_rows == kStep) {
      if (r0 >= 0) {
        mbar_expect_tx(bar, S::kStageBytes);
        tma_load_3d(dst, &tm_k, 0, kvh, r0, bar);
        tma_load_3d(dst + 2 * S::kHalfBytes, &tm_v, 0, kvh, r0, bar);
      } else {
        mbar_arrive(bar);
      }
      return;
    }
    mbar_expect_tx(bar, ((r0 >= 0) + (r1 >= 0)) * 2 * S::kHalfBytes);
    if (r0 >= 0) {
      tma_load_3d(dst, &tm_k, 0, kvh, r0, bar);
      tma_load_3d(dst + 2 * S::kHalfBytes, &tm_v, 0, kvh, r0, bar);
    }
    if (r1 >= 0) {
      tma_load_3d(dst + S::kHalfBytes, &tm_k, 0, kvh, r1, bar);
      tma_load_3d(dst + 3 * S::kHalfBytes, &tm_v, 0, kvh, r1, bar);
    }
  };
  LookUp now = look_up(0), then = now;  // this batch of 16 iterations and the next
  for (int it = 0; it < kStages && it < steps; ++it) copy(it, now.row);
  float now_k, now_v;               // the exponents, converted once they are needed
  if (!idle) {
  // ---- Q as f16 under a power of two per row
    constexpr int LPR = D / 8;         // lanes of a row: 8 elements each
    for (int r = tid / LPR; r < RT; r += kThreads / LPR) {
      const int qr = q0 + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (qr < R) v = __ldg((const uint4*)(p.q + row_index(p, b, kvh, qr) * D) + tid % LPR);
      uint32_t m = max_finite_bf16(max_finite_bf16(max_finite_bf16(max_finite_bf16(0, v.x), v.y), v.z), v.w);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const int e = m ? max(f16_exponent(m, 14), -126) : 0;
      const float inv = pow2i(-e);
      // 4 elements of word w of chunk ch: k-step (ch % KH) * 4 + w of lane (row % 8, ch / KH)
      const int ch = tid % LPR / 2, w0 = tid % LPR % 2 * 2;
      uint2* at = (uint2*)sQ + (r / 8 * KS + ch % KH * 4 + w0) * 32 + (r % 8) * 4 + ch / KH;
      at[0] = make_uint2(bf16x2_to_f16x2(v.x, inv), bf16x2_to_f16x2(v.y, inv));
      at[32] = make_uint2(bf16x2_to_f16x2(v.z, inv), bf16x2_to_f16x2(v.w, inv));
      if (tid % LPR == 0) sRow[r] = p.scale_log2 * pow2i(e);
    }
  }
  __syncthreads();

  float o[NR][NT][4];  // O^T: elements g * D / 8 + 2 i (+ 1: third and fourth) of rows 2c, 2c + 1
  float m_ref[NR][2], l[NR][2], mul[NR][2];
#pragma unroll
  for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nr][i][e] = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      m_ref[nr][r] = -INFINITY;
      l[nr][r] = 0.f;
      mul[nr][r] = idle ? 0.f : sRow[nr * 8 + 2 * c + r];
    }
  }
  auto q_frag = [&](int nr, int ks) { return ((const uint2*)sQ)[(nr * KS + ks) * 32 + lane]; };

  // The softmax of a step for row tile nr: scores sc (f32 fragments of NH
  // halves: tokens g, g + 8 of rows 2c, 2c + 1) to the f16 fragments of P^T.
  // kmul, what a K product counts for, and ev, the V exponent: of each half, or
  // for one half (tree rows) of each of its two tokens.
  // bits[r]: the tokens that row 2c + r sees, unless it sees all.
  auto softmax = [&](auto nh, int nr, float (*sc)[4], const float* kmul, const float* ev, bool all,
                     const uint32_t* bits, uint32_t (*pt)[2]) {
    constexpr int NH = decltype(nh)::value;
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = NH == 1 ? e >> 1 : h;
        sc[h][e] = fmaf(sc[h][e], mul[nr][e & 1] * kmul[at], ev[at]);
      }
    if (!all) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((bits[e & 1] >> (h * kHalf + g + (e >> 1) * 8)) & 1u)) sc[h][e] = -INFINITY;
    }
    float top[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(sc[0][r], sc[0][2 + r]);
#pragma unroll
      for (int h = 1; h < NH; ++h) top[r] = fmax3(top[r], sc[h][r], sc[h][2 + r]);
    }
    // (differences: where scores are so large that their last place is above 1, a sum would round past f16's range)
    if (__any_sync(0xFFFFFFFFu, top[0] - m_ref[nr][0] > kSlack + kHead || top[1] - m_ref[nr][1] > kSlack + kHead)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], x));
        float alpha = 1.f;
        if (top[r] - m_ref[nr][r] > kSlack + kHead) {
          const float to = reference_below(top[r], kHead, kSlack);
          alpha = m_ref[nr][r] == -INFINITY ? 0.f : ex2(m_ref[nr][r] - to);
          m_ref[nr][r] = to;
        }
        l[nr][r] *= alpha;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          o[nr][i][r] *= alpha;
          o[nr][i][2 + r] *= alpha;
        }
      }
    }
    float m[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) m[r] = m_ref[nr][r] == -INFINITY ? 0.f : m_ref[nr][r];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = ex2(sc[h][e] - m[e & 1]);
      if (NH == 1) {
        const float down[2] = {ex2(-ev[0]), ex2(-ev[1])};
#pragma unroll
        for (int r = 0; r < 2; ++r) l[nr][r] = fmaf(w[r], down[0], fmaf(w[2 + r], down[1], l[nr][r]));
      } else {
        // (a half that is not there has weights 0 and must not meet 2^inf)
        const float down = ex2(fminf(-ev[h], 126.f));
#pragma unroll
        for (int r = 0; r < 2; ++r) l[nr][r] = fmaf(w[r] + w[2 + r], down, l[nr][r]);
      }
      pt[h][0] = movmatrix(f32x2_to_f16x2(w[0], w[1]));
      pt[h][1] = movmatrix(f32x2_to_f16x2(w[2], w[3]));
    }
  };

  // ---- context steps
  // byte offsets of this lane's fragments in a stage, under TMA's swizzle (16-byte
  // chunk ^ row & 7 in 128-byte rows, ^ row / 2 & 3 in 64-byte rows)
  int koff[KH], voff[2];
#pragma unroll
  for (int h = 0; h < KH; ++h) koff[h] = g * D + (D == 128 ? ((2 * c + h) ^ g) * 16 : (c ^ (g >> 1)) * 16);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    voff[i] = (2 * c + i) * D + (D == 128 ? (g ^ (2 * c + i)) * 16 : ((g >> 1) ^ c) * 16 + (g & 1) * 8);
  now_k = k_scale(now);
  now_v = v_exp(now);
  int it = 0;
  for (; it < steps; ++it) {
    if ((it & 15) == 0) then = look_up((it >> 4) + 1);  // used from iteration it + 14 on
    float kmul[2], ev[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kmul[h] = __shfl_sync(0xFFFFFFFFu, now_k, (it & 15) * 2 + h);
      ev[h] = __shfl_sync(0xFFFFFFFFu, now_v, (it & 15) * 2 + h);
    }
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[it % kStages], (uint32_t)(it / kStages) & 1u, s_abort,
                                                   p.wait_cycles)))
      break;
    const unsigned char* dk = my + it % kStages * S::kStageBytes;
    const unsigned char* dv = dk + 2 * S::kHalfBytes;
    float sc[NR][2][4];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nr][h][e] = 0.f;
#pragma unroll
    for (int h = 0; h < KH; ++h) {
      uint4 k[4];  // tokens g, g + 8, g + 16, g + 24
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = *(const uint4*)(dk + koff[h] + j * 8 * D);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint2 q[NR];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) q[nr] = q_frag(nr, h * 4 + w);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t x = word(k[2 * j], w), y = word(k[2 * j + 1], w);
          const uint32_t a[4] = {codes_lo(x), codes_lo(y), codes_hi(x), codes_hi(y)};
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) mma16816(sc[nr][j], a, q[nr].x, q[nr].y);
        }
      }
    }
    const int have = T - (first + it * kWarps) * kStep;
    uint32_t bits = have >= kStep ? 0xFFFFFFFFu : (1u << have) - 1u;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (ev[h] == -INFINITY) bits &= h ? 0xFFFFu : 0xFFFF0000u;  // a page that is not there
    const bool all = bits == 0xFFFFFFFFu;
    const uint32_t see[2] = {bits, bits};
    uint32_t pt[NR][2][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
      softmax(std::integral_constant<int, 2>(), nr, sc[nr], kmul, ev, all, see, pt[nr]);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t v[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned char* src = dv + voff[i & 1] + half * S::kHalfBytes + (i >> 1) * 8 * D;
        if (D == 128) {
          const uint4 x = *(const uint4*)src;
          v[i][0] = x.x;
          v[i][1] = x.y;
          v[i][D / 32 - 2] = x.z;
          v[i][D / 32 - 1] = x.w;
        } else {
          const uint2 x = *(const uint2*)src;
          v[i][0] = x.x;
          v[i][1] = x.y;
        }
      }
      if (!all) {  // codes outside the context may be anything, NaN too
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (!((bits >> (half * kHalf + (i >> 1) * 8 + 2 * c + (i & 1))) & 1u)) {
#pragma unroll
            for (int w = 0; w < D / 32; ++w) v[i][w] = 0u;
          }
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t a0[4] = {codes_of<0>(v[0][w], v[1][w]), codes_of<1>(v[0][w], v[1][w]),
                                codes_of<0>(v[2][w], v[3][w]), codes_of<1>(v[2][w], v[3][w])};
        const uint32_t a1[4] = {codes_of<2>(v[0][w], v[1][w]), codes_of<3>(v[0][w], v[1][w]),
                                codes_of<2>(v[2][w], v[3][w]), codes_of<3>(v[2][w], v[3][w])};
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          mma16816(o[nr][2 * w], a0, pt[nr][half][0], pt[nr][half][1]);
          mma16816(o[nr][2 * w + 1], a1, pt[nr][half][0], pt[nr][half][1]);
        }
      }
    }
    if (it + kStages < steps) {  // every lane has read the stage: refill it
      __syncwarp();
      copy(it + kStages, ((it + kStages) >> 4) == (it >> 4) ? now.row : then.row);
    }
    if ((it & 15) == 15) {
      now = then;
      now_k = k_scale(now);
      now_v = v_exp(now);
    }
  }
  if (it < steps) {  // a wait gave up: let the copies in flight land
    int keep_going = 0;
    for (int i = it; i < it + kStages && i < steps; ++i)
      mbar_wait_bounded(&full[i % kStages], (uint32_t)(i / kStages) & 1u, &keep_going, kDrainCycles);
    if (lane == 0) raise_status(p.status, DDT_ERR_TIMEOUT);
  }

  // ---- tree steps: the rows' own bf16 K/V, as f16 under a power of two per tree
  // row, so that no row's size shows in another's (the mask may hide it)
  const int tfirst = first >= nctx ? first : first + (nctx - first + kWarps - 1) / kWarps * kWarps;
  for (int s = tfirst; !idle && s < hi; s += kWarps) {
    const int t0 = (s - nctx) * kHalf;
    const int cnt = min(kHalf, n - t0);
    const uint16_t* kt = p.kt + (((int64_t)b * p.n_max + t0) * p.c.hkv + kvh) * D;
    const uint16_t* vt = p.vt + (((int64_t)b * p.n_max + t0) * p.c.hkv + kvh) * D;
    uint32_t kmax[2] = {0, 0};  // of tokens g, g + 8
    uint4 kw[2][KH][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < KH; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int t = j * 8 + g;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (t < cnt) x = __ldg((const uint4*)(kt + t * stride + (c * KH + h) * 16) + q);
          kmax[j] = max_finite_bf16(max_finite_bf16(max_finite_bf16(max_finite_bf16(kmax[j], x.x), x.y), x.z), x.w);
          kw[j][h][q] = x;
        }
    float kmul[2], kinv[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int o = 1; o < 4; o *= 2) kmax[j] = max(kmax[j], __shfl_xor_sync(0xFFFFFFFFu, kmax[j], o));
      const int ek = tree_exponent(kmax[j]);
      kmul[j] = pow2i(ek);
      kinv[j] = pow2i(-ek);
    }
    float sc[NR][1][4];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[nr][0][e] = 0.f;
#pragma unroll
    for (int h = 0; h < KH; ++h)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint4 &x = kw[0][h][w >> 1], &y = kw[1][h][w >> 1];
        const uint32_t a[4] = {bf16x2_to_f16x2(word(x, (w & 1) * 2), kinv[0]),
                               bf16x2_to_f16x2(word(y, (w & 1) * 2), kinv[1]),
                               bf16x2_to_f16x2(word(x, (w & 1) * 2 + 1), kinv[0]),
                               bf16x2_to_f16x2(word(y, (w & 1) * 2 + 1), kinv[1])};
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
          const uint2 q = q_frag(nr, h * 4 + w);
          mma16816(sc[nr][0], a, q.x, q.y);
        }
      }
    // V: tokens 2c, 2c+1, 8+2c, 9+2c, elements g*D/8 ..
    uint32_t v[4][D / 16];
    uint32_t vmax[4] = {0, 0, 0, 0};
    bool odd = false;  // a wild element
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = (i >> 1) * 8 + 2 * c + (i & 1);
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (t < cnt) x = __ldg((const uint4*)(vt + t * stride + g * (D / 8)) + q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t w = word(x, e);
          odd |= has_wild(w);
          v[i][q * 4 + e] = tame_bf16x2(w);
          vmax[i] = max(vmax[i], max_bf16(v[i][q * 4 + e]));
        }
      }
    }
    odd = __any_sync(0xFFFFFFFFu, odd);
    float ev[2];  // of tokens g, g + 8, from a lane that holds their V
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int o = 4; o < 32; o *= 2) vmax[i] = max(vmax[i], __shfl_xor_sync(0xFFFFFFFFu, vmax[i], o));
      const int e = tree_exponent(vmax[i]);
#pragma unroll
      for (int w = 0; w < D / 16; ++w) v[i][w] = bf16x2_to_f16x2(v[i][w], pow2i(-e));
      const float other = (float)__shfl_sync(0xFFFFFFFFu, e, g >> 1);
      if ((g & 1) == (i & 1)) ev[i >> 1] = other;
    }
    uint32_t pt[NR][1][2];
    const uint32_t cbits = cnt >= kHalf ? 0xFFFFu : (1u << cnt) - 1u;
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      uint32_t see[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int j = (q0 + nr * 8 + 2 * c + r) / p.g;
        see[r] = j < n ? (__ldg(p.mask + ((int64_t)b * p.n_max + j) * p.W + (t0 >> 5)) >> (t0 & 31)) & cbits : 0u;
      }
      softmax(std::integral_constant<int, 1>(), nr, sc[nr], kmul, ev, false, see, pt[nr]);
      if (odd) {
        // a wild V element reaches the rows that see its token, and no others
        for (int t = 0; t < cnt; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if ((see[r] >> t) & 1u) {
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint16_t x = vt[t * stride + g * (D / 8) + 2 * i + e];
                  if (is_wild(x)) o[nr][i][2 * e + r] += wild_value(x);
                }
            }
      }
    }
#pragma unroll
    for (int w = 0; w < NT; ++w) {
      const uint32_t a[4] = {prmt(v[0][w], v[1][w], 0x5410), prmt(v[0][w], v[1][w], 0x7632),
                             prmt(v[2][w], v[3][w], 0x5410), prmt(v[2][w], v[3][w], 0x7632)};
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) mma16816(o[nr][w], a, pt[nr][0][0], pt[nr][0][1]);
    }
  }

  // ---- merge the warps, write rows or partials
  float* sO = (float*)ring;                                   // [kWarps][RT][kORow]
  float2* sML = (float2*)(ring + kWarps * RT * S::kORow * 4);  // [kWarps][RT]
  __syncthreads();  // every warp is done with its ring
  if (!idle) {
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = nr * 8 + 2 * c + r;
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[nr][r] += __shfl_xor_sync(0xFFFFFFFFu, l[nr][r], x);
        // (a row of NaN scores alone has no reference: any number carries its NaN on)
        if (g == 0)
          sML[warp * RT + row] = make_float2(l[nr][r] != l[nr][r] ? 0.f : m_ref[nr][r], l[nr][r]);
        float* dst = sO + (warp * RT + row) * S::kORow + g * (D / 8);
#pragma unroll
        for (int i = 0; i < NT; ++i) *(float2*)(dst + 2 * i) = make_float2(o[nr][i][r], o[nr][i][2 + r]);
      }
  }
  __syncthreads();
  pdl_trigger();
  constexpr int LPR = D / 4;  // threads of a row: 4 elements each
  for (int r = tid / LPR; r < RT; r += kThreads / LPR) {
    const int qr = q0 + r;
    if (qr >= R) break;
    const int d0 = tid % LPR * 4;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!idle && qr < n * p.g) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sML[w * RT + r].x);
      if (M != -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 ml = sML[w * RT + r];
          if (ml.x == -INFINITY) continue;
          const float a = ex2(ml.x - M);
          const float4 x = *(const float4*)(sO + (w * RT + r) * S::kORow + d0);
          L = fmaf(ml.y, a, L);
          acc.x = fmaf(x.x, a, acc.x);
          acc.y = fmaf(x.y, a, acc.y);
          acc.z = fmaf(x.z, a, acc.z);
          acc.w = fmaf(x.w, a, acc.w);
        }
      }
    }
    if (p.nsplit > 1) {
      const int64_t row = ((int64_t)grp * p.nsplit + split) * R + qr;
      if (M != -INFINITY) *(float4*)(p.part_o + row * D + d0) = acc;
      if (d0 == 0) p.part_ml[row] = make_float2(M, L);
    } else {
      const float inv = M == -INFINITY ? 0.f : 1.f / L;
      const int64_t at = row_index(p, b, kvh, qr);
      *(uint2*)(p.out + at * D + d0) = make_uint2(f32x2_to_bf16x2(acc.x * inv, acc.y * inv),
                                                  f32x2_to_bf16x2(acc.z * inv, acc.w * inv));
      if (p.lse_out && d0 == 0)
        p.lse_out[at] = M == -INFINITY ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
    }
  }
}

// Merge the splits' partials.  WPR = 1: a warp per query row (many rows of few
// splits: large trees).  WPR = 8: the CTA's warps take one row's splits in turn
// and join (few rows of many splits: long contexts).
constexpr int kCombineWarps = 8;
template <int D, int WPR>
__global__ void __launch_bounds__(32 * kCombineWarps) attn_q8_combine(const AttnQ8Params p) {
  constexpr int E = D / 32;  // elements a lane
  __shared__ float s_o[kCombineWarps][D];
  __shared__ float2 s_ml[kCombineWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.n_max * p.g;
  const int qr = blockIdx.x * (kCombineWarps / WPR) + (WPR == 1 ? warp : 0);
  const int grp = blockIdx.y, b = grp / p.c.hkv, kvh = grp % p.c.hkv;
  pdl_wait();
  pdl_trigger();
  if (WPR == 1 && qr >= R) return;
  int n, T;
  attn_q8_lengths(p, b, false, n, T);
  const bool live = qr < n * p.g;
  float M = -INFINITY, L = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const int64_t row = (int64_t)grp * p.nsplit * R + qr;
  constexpr int kFly = 4;
  for (int s0 = WPR == 1 ? 0 : warp; live && s0 < p.nsplit; s0 += kFly * WPR) {
    float2 ml[kFly];
    float v[kFly][E];
#pragma unroll
    for (int f = 0; f < kFly; ++f) {
      const int s = s0 + f * WPR;
      ml[f] = make_float2(-INFINITY, 0.f);
      if (s < p.nsplit) {
        const int64_t at = row + (int64_t)s * R;
        ml[f] = p.part_ml[at];
        const float* src = p.part_o + at * D + lane * E;
        if (E == 4) {
          const float4 x = *(const float4*)src;
          v[f][0] = x.x;
          v[f][1] = x.y;
          v[f][E - 2] = x.z;
          v[f][E - 1] = x.w;
        } else {
          const float2 x = *(const float2*)src;
          v[f][0] = x.x;
          v[f][1] = x.y;
        }
      }
    }
    float to = M;
#pragma unroll
    for (int f = 0; f < kFly; ++f) to = fmaxf(to, ml[f].x);
    if (to == -INFINITY) continue;
    const float back = M == -INFINITY ? 0.f : ex2(M - to);
    L *= back;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= back;
#pragma unroll
    for (int f = 0; f < kFly; ++f)
      if (ml[f].x != -INFINITY) {  // (an empty split's partial was not written)
        const float a = ex2(ml[f].x - to);
        L = fmaf(ml[f].y, a, L);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(v[f][e], a, acc[e]);
      }
    M = to;
  }
  if (WPR > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = acc[e];
    if (lane == 0) s_ml[warp] = make_float2(M, L);
    __syncthreads();
    if (warp != 0) return;
    M = -INFINITY;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kCombineWarps; ++w) M = fmaxf(M, s_ml[w].x);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kCombineWarps; ++w)
      if (s_ml[w].x != -INFINITY) {
        const float a = ex2(s_ml[w].x - M);
        L = fmaf(s_ml[w].y, a, L);
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(s_o[w][lane * E + e], a, acc[e]);
      }
  }
  const float inv = M == -INFINITY ? 0.f : 1.f / L;
  const int64_t at = row_index(p, b, kvh, qr);
  uint32_t* dst = (uint32_t*)(p.out + at * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) dst[e / 2] = f32x2_to_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (p.lse_out && lane == 0)
    p.lse_out[at] = M == -INFINITY ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
}

template <int D>
cudaError_t launch_combine(const AttnQ8Params& p, cudaStream_t stream) {
  const unsigned groups = (unsigned)(p.batch * p.c.hkv), R = (unsigned)(p.n_max * p.g);
  const dim3 block(32 * kCombineWarps);
  if (p.nsplit > 8) return launch_pdl(attn_q8_combine<D, kCombineWarps>, dim3(R, groups), block, 0, stream, 0, p);
  return launch_pdl(attn_q8_combine<D, 1>, dim3((R + kCombineWarps - 1) / kCombineWarps, groups), block, 0,
                    stream, 0, p);
}

struct Plan {
  int nr;  // tiles of 8 query rows a CTA; 0: the wide kernel
  int tiles, nsplit, steps_per_split;
};

// The wide kernel's pairs of row tiles and KV splits (steps: tiles of 128
// tokens): the fewest waves x tiles of a CTA, a split's partials and their
// merge counted as kMergeTiles tiles (measured on 16 ragged trees of 129 rows:
// 418 us in three splits, 380 us in one).  The steps are those of max_ctx: a bound
// far above the contexts leaves most splits empty (one tree of 65 rows over 4096
// tokens: 37 us with a bound of 4096, 115 us with 131072).
Plan plan_wide(const ddt_attn_q8_args* a, long R) {
  constexpr long kMergeTiles = 8;
  Plan pl = {};
  pl.tiles = (int)((R + 255) / 256);
  const long base = (long)pl.tiles * a->batch * a->cache.hkv, sms = device_sm_count();
  const long tiles = (a->max_ctx + 127) / 128 + (a->n_max + 127) / 128;
  long best = -1;
  for (long s = 1; s <= 64 && s <= tiles; ++s) {
    const long ts = (tiles + s - 1) / s, sp = (tiles + ts - 1) / ts;
    const long cost = (base * sp + sms - 1) / sms * (ts + (sp > 1 ? kMergeTiles : 0));
    if (best < 0 || cost < best) {
      best = cost;
      pl.steps_per_split = (int)ts;
      pl.nsplit = (int)sp;
    }
  }
  return pl;
}

// d = 128 with more than kWideRows rows per kv head takes the wide kernel,
// anything else row tiles of 8, 16, 24 or 32 rows and KV splits of this file's.
Plan plan_of(const ddt_attn_q8_args* a) {
  const long R = (long)a->n_max * (a->hq / a->cache.hkv);
  if (a->cache.d == 128 && R > kWideRows) return plan_wide(a, R);
  Plan pl;
  pl.nr = (int)std::min(4L, (R + 7) / 8);
  pl.tiles = (int)((R + 8 * pl.nr - 1) / (8 * pl.nr));
  const long base = (long)pl.tiles * a->batch * a->cache.hkv;
  const long steps = (a->max_ctx + kStep - 1) / kStep + (a->n_max + kHalf - 1) / kHalf;
  const long slots = (long)device_sm_count() * (pl.nr <= 2 ? 3 : 2);
  // as many splits as fill the device, of at least 2 steps a warp; long
  // contexts in splits of at most kLong steps, so that ragged ones even out (32
  // ragged sequences: 233 us so, 303 us without; at the step that took it, 40 to
  // 128 steps were alike, and 32 cut 4 x 131072 tokens into more than one wave: 50
  // us against 37 us)
  constexpr long kLong = 64;
  long ns = std::max(1L, slots / std::max(1L, base));
  ns = std::min(ns, std::max(1L, steps / (2 * kWarps)));
  ns = std::max(ns, steps / kLong);
  ns = std::min(ns, 65535L);
  pl.steps_per_split = (int)((steps + ns - 1) / ns);
  pl.nsplit = (int)((steps + pl.steps_per_split - 1) / pl.steps_per_split);
  return pl;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The codes as rows of one kv head: d bytes x hkv x all tokens, boxes of box_rows tokens.
bool encode_codes(CUtensorMap* m, const void* codes, const ddt_q8_cache* c, int batch, int box_rows) {
  auto fn = tc::encode_fn();
  if (!fn) return false;
  const cuuint64_t rows =
      c->page_table ? (cuuint64_t)c->num_pages * c->page_size : (cuuint64_t)batch * (cuuint64_t)c->t_max;
  const cuuint64_t dims[3] = {(cuuint64_t)c->d, (cuuint64_t)c->hkv, rows};
  const cuuint64_t str[2] = {(cuuint64_t)c->d, (cuuint64_t)c->hkv * c->d};
  const cuuint32_t box[3] = {(cuuint32_t)c->d, 1, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(codes), dims, str, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, c->d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NR>
cudaError_t launch_rows(const CUtensorMap& mk, const CUtensorMap& mv, const AttnQ8Params& p, int tiles,
                          cudaStream_t stream) {
  const size_t smem = Smem<D, NR>::kTotal;
  cudaError_t e = ensure_smem_attr((const void*)attn_q8_kernel<D, NR>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_q8_kernel<D, NR>, dim3(tiles, p.nsplit, p.batch * p.c.hkv), dim3(kThreads), smem, stream,
                    0, mk, mv, p);
}

template <int D>
cudaError_t launch_narrow(const CUtensorMap& mk, const CUtensorMap& mv, const AttnQ8Params& p, const Plan& pl,
                          cudaStream_t stream) {
  switch (pl.nr) {
    case 1: return launch_rows<D, 1>(mk, mv, p, pl.tiles, stream);
    case 2: return launch_rows<D, 2>(mk, mv, p, pl.tiles, stream);
    case 3: return launch_rows<D, 3>(mk, mv, p, pl.tiles, stream);
    default: return launch_rows<D, 4>(mk, mv, p, pl.tiles, stream);
  }
}

}  // namespace

size_t attn_q8_workspace_size(const ddt_attn_q8_args* a) {
  if (a->batch == 0) return 0;
  const Plan pl = plan_of(a);
  if (pl.nsplit <= 1) return 0;
  const size_t rows = (size_t)a->batch * a->cache.hkv * pl.nsplit * a->n_max * (a->hq / a->cache.hkv);
  return align256(rows * a->cache.d * sizeof(float)) + rows * sizeof(float2);
}

ddt_status launch_attn_q8(const ddt_attn_q8_args* a, void* ws, cudaStream_t stream) {
  if (a->batch == 0) return DDT_OK;
  AttnQ8Params p;
  p.c = q8_view(&a->cache);
  p.q = (const uint16_t*)a->q;
  p.kt = (const uint16_t*)a->k_tree;
  p.vt = (const uint16_t*)a->v_tree;
  p.ctx_len = a->ctx_len;
  p.n_nodes = a->n_nodes;
  p.mask = a->mask;
  p.max_ctx = a->max_ctx;
  p.batch = a->batch;
  p.n_max = a->n_max;
  p.hq = a->hq;
  p.g = a->hq / a->cache.hkv;
  p.W = (a->n_max + 31) / 32;
  p.scale_log2 = a->scale * kLog2e;
  p.out = (uint16_t*)a->out;
  p.lse_out = a->lse_out;
  p.status = a->dev_status;
  p.wait_cycles = wait_limit_cycles();
  const Plan pl = plan_of(a);
  p.nsplit = pl.nsplit;
  p.steps_per_split = pl.steps_per_split;
  const size_t rows = (size_t)a->batch * a->cache.hkv * pl.nsplit * a->n_max * p.g;
  p.part_o = pl.nsplit > 1 ? (float*)ws : nullptr;
  p.part_ml = pl.nsplit > 1 ? (float2*)((char*)ws + align256(rows * a->cache.d * sizeof(float))) : nullptr;
  cudaError_t e;
  if (pl.nr == 0) {
    p.box_rows = 0;
    e = launch_attn_q8_wide(p, pl.tiles, stream);
  } else {
    // a box never leaves its page, and steps begin at multiples of 32 tokens
    p.box_rows = a->cache.page_table && a->cache.page_size % kStep ? kHalf : kStep;
    CUtensorMap mk = {}, mv = {};
    if (a->max_ctx > 0 && (!encode_codes(&mk, a->cache.k_cache, &a->cache, a->batch, p.box_rows) ||
                           !encode_codes(&mv, a->cache.v_cache, &a->cache, a->batch, p.box_rows)))
      return DDT_ERR_CUDA;
    e = a->cache.d == 128 ? launch_narrow<128>(mk, mv, p, pl, stream) : launch_narrow<64>(mk, mv, p, pl, stream);
  }
  if (e != cudaSuccess) return DDT_ERR_CUDA;
  if (pl.nsplit > 1) {
    e = a->cache.d == 128 ? launch_combine<128>(p, stream) : launch_combine<64>(p, stream);
    if (e != cudaSuccess) return DDT_ERR_CUDA;
  }
  return DDT_OK;
}

}  // namespace ddt
