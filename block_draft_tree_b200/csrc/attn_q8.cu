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
// and P as f16 (11 bits, error 2^-12) keeps every block's share whatever its
// scale.  m lags the true maximum by up to 2^8 and P's range begins at 2^7 for
// a new maximum: weights reach 2^15 at most, and f16's subnormal step (2^-24)
// is 2^-31 of the maximum, below any sum over a long tail.  Queries become f16
// under a power of two per row, exact down to 2^-39 of the row's largest.
//
// What bounds it: with R <= 32 rows per kv head the K/V codes are read once
// for 2R multiply-adds each, so HBM.  A warp takes 16 tokens a step; thread-
// private 16-byte cp.async copies (a lane later reads what it copied itself:
// no barrier) keep kStages - 1 steps in flight.  The copies are laid out so
// that a lane's bytes are its own m16n8k16 fragments: for K lane (g, c) holds
// token g and a 16-byte chunk c, with the d index permuted alike in Q's
// fragments; for V lane (g, c) holds tokens 2c, 2c+1, 8+2c, 9+2c and chunk g,
// whose pairs one byte permute interleaves.  One cvt turns two codes into an
// f16 pair, so nothing is transposed and nothing is staged twice.
#include <algorithm>

#include "attn_q8.cuh"
#include "launch.h"

namespace ddt {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;             // steps in the ring of a warp
constexpr int kStep = 16;              // tokens of a step
constexpr float kSlack = 8.f;          // the reference moves when a score passes it by 2^8
constexpr float kHead = 7.f;           // P of a new maximum is 2^7

__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async8(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// D += A (16x16, row) * B (16x8, col), f16 inputs, f32 accumulators.
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Exponent e with amax (bf16 magnitude bits, finite) * 2^-e in [2^top, 2^(top+1)).
__device__ __forceinline__ int f16_exponent(uint32_t amax_bits, int top) {
  return amax_bits < 0x80u ? -126 - top : (int)(amax_bits >> 7) - 127 - top;
}
// Two packed bf16 -> two f16 scaled by `inv` (a power of two).
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float inv) {
  return f32x2_to_f16x2(bf16_lo(w) * inv, bf16_hi(w) * inv);
}
// Same, non-finite elements as 0.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2_finite(uint32_t w, float inv) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return bf16x2_to_f16x2(w, inv);
}

template <int D, int MT>
struct Smem {
  static constexpr int kKSlots = 2 * (D / 64);           // 16-byte copies of K a lane makes per step
  static constexpr int kVSlots = 4;                      // V: 4 tokens, D/8 bytes each
  static constexpr int kVBytes = D / 8;                  // 16 or 8
  static constexpr int kStageBytes = 32 * (kKSlots * 16 + kVSlots * kVBytes);
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kQRow = D + 8;                    // f16 a row, padded by 16 bytes
  static constexpr int kQ = 16 * MT * kQRow * 2;
  static constexpr int kORow = D + 4;                    // f32 a row of a warp's O, padded
  static constexpr int kMerge = kWarps * 16 * MT * (kORow * 4 + 8);
  static constexpr int kTotal = kQ + 16 * MT * 4 + (kRing > kMerge ? kRing : kMerge);
};

// Row qr of sequence b and kv head kvh: its place in q / out.
__device__ __forceinline__ int64_t row_index(const AttnQ8Params& p, int b, int kvh, int qr) {
  return ((int64_t)b * p.n_max + qr / p.g) * p.hq + kvh * p.g + qr % p.g;
}

template <int D, int MT>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 3 : 2) attn_q8_kernel(const AttnQ8Params p) {
  using S = Smem<D, MT>;
  constexpr int KH = D / 64;       // 64-wide halves of d
  constexpr int NT = D / 8;        // n-tiles of O
  constexpr int KS = D / 16;       // k-steps of QK
  extern __shared__ __align__(16) unsigned char smem[];
  __half* sQ = (__half*)smem;
  float* sRow = (float*)(smem + S::kQ);  // score multiplier of each row
  unsigned char* ring = smem + S::kQ + 16 * MT * 4;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int tile = blockIdx.x, split = blockIdx.y, grp = blockIdx.z;
  const int b = grp / p.c.hkv, kvh = grp % p.c.hkv;
  const int R = p.n_max * p.g;
  const int q0 = tile * 16 * MT;
  pdl_wait();
  int n, T;
  attn_q8_lengths(p, b, tile == 0 && split == 0 && kvh == 0 && tid == 0, n, T);
  const int nctx = (T + kStep - 1) / kStep;
  const int nall = nctx + (n + kStep - 1) / kStep;
  const int lo = min(split * p.steps_per_split, nall);
  const int hi = min(lo + p.steps_per_split, nall);
  const bool dead = q0 >= n * p.g;  // every row past the tree
  const bool idle = dead || lo >= hi;
  const int chi = min(hi, nctx);

  // ---- the ring's producer: this lane's own fragments of context step `s`
  const uint8_t* kbase = p.c.kc + (int64_t)kvh * D;
  const uint8_t* vbase = p.c.vc + (int64_t)kvh * D;
  const int64_t stride = (int64_t)p.c.hkv * D;
  unsigned char* my = ring + warp * kStages * S::kStageBytes + lane * 16;
  unsigned char* myv = ring + warp * kStages * S::kStageBytes + 32 * S::kKSlots * 16 + lane * S::kVBytes;
  auto place = [&](int s) -> Q8Place { return s < chi ? q8_place(p.c, b, (int64_t)s * kStep) : Q8Place{-1, -1}; };
  auto copy = [&](int s, int stage, const Q8Place& at) {
    if (s >= chi) return;
    const int t0 = s * kStep;
    const int have = at.row < 0 ? 0 : T - t0;  // tokens of the step that exist
    const int64_t base = max(at.row, (int64_t)0) * stride;
    unsigned char* dk = my + stage * S::kStageBytes;
    unsigned char* dv = myv + stage * S::kStageBytes;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = j * 8 + g;
      const bool ok = t < have;
      const uint8_t* src = kbase + base + (ok ? t : 0) * stride + c * 16;
#pragma unroll
      for (int h = 0; h < KH; ++h) cp_async16(dk + (j * KH + h) * 512, src + h * 64, ok ? 16 : 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = (i >> 1) * 8 + 2 * c + (i & 1);
      const bool ok = t < have;
      const uint8_t* src = vbase + base + (ok ? t : 0) * stride + g * S::kVBytes;
      if (D == 128)
        cp_async16(dv + i * 512, src, ok ? 16 : 0);
      else
        cp_async8(dv + i * 256, src, ok ? 8 : 0);
    }
  };
  auto exps = [&](const Q8Place& at, int& ek, int& ev) {
    ek = ev = 0;
    if (at.row >= 0) {
      ek = p.c.ke[at.blk * p.c.hkv + kvh];
      ev = p.c.ve[at.blk * p.c.hkv + kvh];
    }
  };

  int s_mine = lo + warp;              // this warp's steps: lo + warp, + kWarps, ...
  int ek_ring[kStages], ev_ring[kStages];
  Q8Place next{-1, -1};
  if (!idle) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const int s = s_mine + i * kWarps;
      const Q8Place at = place(s);
      if (s < chi && at.row < 0 && lane == 0) raise_status(p.status, DDT_ERR_INVALID_ARG);
      copy(s, i, at);
      exps(at, ek_ring[i], ev_ring[i]);
      cp_commit();
    }
    ek_ring[kStages - 1] = ev_ring[kStages - 1] = 0;
    next = place(s_mine + (kStages - 1) * kWarps);

    // ---- Q as f16 under a power of two per row
    constexpr int LPR = D / 8;         // lanes of a row: 8 elements each
    for (int r = tid / LPR; r < 16 * MT; r += kThreads / LPR) {
      const int qr = q0 + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (qr < R) v = __ldg((const uint4*)(p.q + row_index(p, b, kvh, qr) * D) + tid % LPR);
      uint32_t m = max_finite_bf16(max_finite_bf16(max_finite_bf16(max_finite_bf16(0, v.x), v.y), v.z), v.w);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const int e = m ? max(f16_exponent(m, 14), -126) : 0;
      const float inv = pow2i(-e);
      *(uint4*)(sQ + r * S::kQRow + tid % LPR * 8) =
          make_uint4(bf16x2_to_f16x2(v.x, inv), bf16x2_to_f16x2(v.y, inv), bf16x2_to_f16x2(v.z, inv),
                     bf16x2_to_f16x2(v.w, inv));
      if (tid % LPR == 0) sRow[r] = p.scale_log2 * pow2i(e);
    }
  }
  __syncthreads();

  float o[MT][NT][4];
  float m_ref[MT][2], l[MT][2], mul[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][i][e] = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      m_ref[mt][r] = -INFINITY;
      l[mt][r] = 0.f;
      mul[mt][r] = idle ? 0.f : sRow[mt * 16 + r * 8 + g];
    }
  }
  // Q's fragments: one row tile keeps them in registers
  uint32_t qf[MT == 1 ? KS : 1][4];
  auto q_frag = [&](int mt, int ks, uint32_t* a) {  // k-step ks covers d = (ks/4)*64 + c*16 + (ks%4)*4 + 0..3
    const int d0 = (ks >> 2) * 64 + c * 16 + (ks & 3) * 4;
    const uint2 x = *(const uint2*)(sQ + (mt * 16 + g) * S::kQRow + d0);
    const uint2 y = *(const uint2*)(sQ + (mt * 16 + 8 + g) * S::kQRow + d0);
    a[0] = x.x;
    a[1] = y.x;
    a[2] = x.y;
    a[3] = y.y;
  };
  if (MT == 1 && !idle) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q_frag(0, ks, qf[ks]);
  }

  // The softmax of one step for row tile mt: scores sc (f32 fragments of two
  // 8-token tiles) to P's f16 fragments.  kmul: 2^(K exponent); ev: V exponent;
  // see[r]: the step's visible tokens for row r * 8 + g.
  auto softmax = [&](int mt, float sc[2][4], float kmul, int ev, const uint32_t* see, bool all, uint32_t* pa) {
    const float fev = (float)ev, down = pow2i(-ev);
    float t[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[j][e] = fmaf(sc[j][e], mul[mt][e >> 1] * kmul, fev);
        if (!all && !((see[e >> 1] >> (j * 8 + 2 * c + (e & 1))) & 1u)) t[j][e] = -INFINITY;
      }
    const float top0 = fmaxf(fmaxf(t[0][0], t[0][1]), fmaxf(t[1][0], t[1][1]));
    const float top1 = fmaxf(fmaxf(t[0][2], t[0][3]), fmaxf(t[1][2], t[1][3]));
    const bool move = top0 > m_ref[mt][0] + (kSlack + kHead) || top1 > m_ref[mt][1] + (kSlack + kHead);
    if (__any_sync(0xFFFFFFFFu, move)) {
      float top[2] = {top0, top1};
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 2));
        float alpha = 1.f;
        if (top[r] > m_ref[mt][r] + (kSlack + kHead)) {
          const float to = top[r] - kHead;
          alpha = m_ref[mt][r] == -INFINITY ? 0.f : ex2(m_ref[mt][r] - to);
          m_ref[mt][r] = to;
        }
        l[mt][r] *= alpha;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          o[mt][i][2 * r] *= alpha;
          o[mt][i][2 * r + 1] *= alpha;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float m = m_ref[mt][r] == -INFINITY ? 0.f : m_ref[mt][r];
      float w[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) w[j][e] = ex2(t[j][2 * r + e] - m);
      l[mt][r] = fmaf((w[0][0] + w[0][1]) + (w[1][0] + w[1][1]), down, l[mt][r]);
      pa[r] = f32x2_to_f16x2(w[0][0], w[0][1]);
      pa[2 + r] = f32x2_to_f16x2(w[1][0], w[1][1]);
    }
  };

  // ---- context steps
  int it = 0;
  for (; !idle && s_mine < chi; s_mine += kWarps, ++it) {
    const int stage = it % kStages;
    {  // refill the stage that the last step freed
      const int s = s_mine + (kStages - 1) * kWarps;
      if (s < chi && next.row < 0 && lane == 0) raise_status(p.status, DDT_ERR_INVALID_ARG);
      copy(s, (it + kStages - 1) % kStages, next);
      exps(next, ek_ring[kStages - 1], ev_ring[kStages - 1]);
      cp_commit();
      next = place(s + kWarps);
    }
    cp_wait<kStages - 1>();
    const float kmul = pow2i(q8_exp((int8_t)ek_ring[0]));
    const int ev = q8_exp((int8_t)ev_ring[0]);
    const unsigned char* dk = my + stage * S::kStageBytes;
    float sc[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[mt][j][e] = 0.f;
#pragma unroll
    for (int h = 0; h < KH; ++h) {
      const uint4 k0 = *(const uint4*)(dk + h * 512);
      const uint4 k1 = *(const uint4*)(dk + (KH + h) * 512);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t w0 = word(k0, w), w1 = word(k1, w);
        const uint32_t b00 = e4m3x2_to_f16x2((uint16_t)w0), b01 = e4m3x2_to_f16x2((uint16_t)(w0 >> 16));
        const uint32_t b10 = e4m3x2_to_f16x2((uint16_t)w1), b11 = e4m3x2_to_f16x2((uint16_t)(w1 >> 16));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t a[4];
          if (MT == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = qf[h * 4 + w][e];
          } else {
            q_frag(mt, h * 4 + w, a);
          }
          mma16816(sc[mt][0], a, b00, b01);
          mma16816(sc[mt][1], a, b10, b11);
        }
      }
    }
    const int left = T - s_mine * kStep;
    const uint32_t bits = left >= kStep ? 0xFFFFu : (1u << left) - 1u;
    const uint32_t see[2] = {bits, bits};
    uint32_t pa[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) softmax(mt, sc[mt], kmul, ev, see, left >= kStep, pa[mt]);
    const unsigned char* dv = myv + stage * S::kStageBytes;
    uint32_t v[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (D == 128) {
        const uint4 x = *(const uint4*)(dv + i * 512);
        v[i][0] = x.x;
        v[i][1] = x.y;
        v[i][D / 32 - 2] = x.z;
        v[i][D / 32 - 1] = x.w;
      } else {
        const uint2 x = *(const uint2*)(dv + i * 256);
        v[i][0] = x.x;
        v[i][1] = x.y;
      }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t x = __byte_perm(v[0][w], v[1][w], half ? 0x7362 : 0x5140);
        const uint32_t y = __byte_perm(v[2][w], v[3][w], half ? 0x7362 : 0x5140);
        const uint32_t x0 = e4m3x2_to_f16x2((uint16_t)x), x1 = e4m3x2_to_f16x2((uint16_t)(x >> 16));
        const uint32_t y0 = e4m3x2_to_f16x2((uint16_t)y), y1 = e4m3x2_to_f16x2((uint16_t)(y >> 16));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816(o[mt][w * 4 + half * 2], pa[mt], x0, y0);
          mma16816(o[mt][w * 4 + half * 2 + 1], pa[mt], x1, y1);
        }
      }
    }
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) {
      ek_ring[i] = ek_ring[i + 1];
      ev_ring[i] = ev_ring[i + 1];
    }
  }
  cp_wait<0>();

  // ---- tree steps: the rows' own bf16 K/V, as f16 under a power of two per step
  for (; !idle && s_mine < hi; s_mine += kWarps) {
    const int t0 = (s_mine - nctx) * kStep;
    const int cnt = min(kStep, n - t0);
    const uint16_t* kt = p.kt + (((int64_t)b * p.n_max + t0) * p.c.hkv + kvh) * D;
    const uint16_t* vt = p.vt + (((int64_t)b * p.n_max + t0) * p.c.hkv + kvh) * D;
    uint32_t kmax = 0;
    uint4 kw[2][KH][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int h = 0; h < KH; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int t = j * 8 + g;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (t < cnt) x = __ldg((const uint4*)(kt + t * stride + h * 64 + c * 16) + q);
          kmax = max_finite_bf16(max_finite_bf16(max_finite_bf16(max_finite_bf16(kmax, x.x), x.y), x.z), x.w);
          kw[j][h][q] = x;
        }
    kmax = __reduce_max_sync(0xFFFFFFFFu, kmax);
    const int ek = min(max(f16_exponent(kmax, 8), DDT_Q8_EXP_MIN), DDT_Q8_EXP_MAX);
    const float kinv = pow2i(-ek);
    float sc[MT][2][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[mt][j][e] = 0.f;
#pragma unroll
    for (int h = 0; h < KH; ++h)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t bb[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint4& x = kw[j][h][w >> 1];
          bb[j][0] = bf16x2_to_f16x2(word(x, (w & 1) * 2), kinv);
          bb[j][1] = bf16x2_to_f16x2(word(x, (w & 1) * 2 + 1), kinv);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t a[4];
          if (MT == 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = qf[h * 4 + w][e];
          } else {
            q_frag(mt, h * 4 + w, a);
          }
          mma16816(sc[mt][0], a, bb[0][0], bb[0][1]);
          mma16816(sc[mt][1], a, bb[1][0], bb[1][1]);
        }
      }
    // V: tokens 2c, 2c+1, 8+2c, 9+2c, elements g*D/8 ..
    uint32_t v[4][D / 16];
    uint32_t vmax = 0;
    bool odd = false;  // a non-finite element
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
          vmax = max_finite_bf16(vmax, w);
          odd |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
          v[i][q * 4 + e] = w;
        }
      }
    }
    vmax = __reduce_max_sync(0xFFFFFFFFu, vmax);
    odd = __any_sync(0xFFFFFFFFu, odd);
    const int ev = min(max(f16_exponent(vmax, 8), DDT_Q8_EXP_MIN), DDT_Q8_EXP_MAX);
    const float vinv = pow2i(-ev);
    uint32_t pa[MT][4];
    const uint32_t cbits = cnt >= kStep ? 0xFFFFu : (1u << cnt) - 1u;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      uint32_t see[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int j = (q0 + mt * 16 + r * 8 + g) / p.g;
        see[r] = j < n ? (__ldg(p.mask + ((int64_t)b * p.n_max + j) * p.W + (t0 >> 5)) >> (t0 & 31)) & cbits : 0u;
      }
      softmax(mt, sc[mt], pow2i(ek), ev, see, false, pa[mt]);
      if (odd) {
        // a non-finite V element reaches the rows that see its token, and no others
        for (int t = 0; t < cnt; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if ((see[r] >> t) & 1u) {
#pragma unroll
              for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint16_t x = vt[t * stride + (2 * c + e) * (D / 8) + i];
                  if ((x & 0x7F80u) == 0x7F80u) o[mt][i][2 * r + e] += bf16_to_f32(x);
                }
            }
      }
    }
#pragma unroll
    for (int w = 0; w < D / 16; ++w) {
      const uint32_t x0 = bf16x2_to_f16x2_finite(v[0][w], vinv), x1 = bf16x2_to_f16x2_finite(v[1][w], vinv);
      const uint32_t y0 = bf16x2_to_f16x2_finite(v[2][w], vinv), y1 = bf16x2_to_f16x2_finite(v[3][w], vinv);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        mma16816(o[mt][2 * w], pa[mt], __byte_perm(x0, x1, 0x5410), __byte_perm(y0, y1, 0x5410));
        mma16816(o[mt][2 * w + 1], pa[mt], __byte_perm(x0, x1, 0x7632), __byte_perm(y0, y1, 0x7632));
      }
    }
  }

  // ---- merge the warps, write rows or partials
  float* sO = (float*)ring;                                   // [kWarps][16 MT][kORow]
  float2* sML = (float2*)(ring + kWarps * 16 * MT * S::kORow * 4);  // [kWarps][16 MT]
  __syncthreads();  // every lane is done with its ring
  if (!idle) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = mt * 16 + r * 8 + g;
        l[mt][r] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][r], 1);
        l[mt][r] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][r], 2);
        // (a row of NaN scores alone has no reference: any number carries its NaN on)
        if (c == 0)
          sML[warp * 16 * MT + row] = make_float2(l[mt][r] != l[mt][r] ? 0.f : m_ref[mt][r], l[mt][r]);
        float* dst = sO + (warp * 16 * MT + row) * S::kORow;
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) dst[(2 * c + e) * (D / 8) + i] = o[mt][i][2 * r + e];
      }
  }
  __syncthreads();
  pdl_trigger();
  constexpr int LPR = D / 4;  // threads of a row: 4 elements each
  for (int r = tid / LPR; r < 16 * MT; r += kThreads / LPR) {
    const int qr = q0 + r;
    if (qr >= R) break;
    const int d0 = tid % LPR * 4;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!idle && qr < n * p.g) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sML[w * 16 * MT + r].x);
      if (M != -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 ml = sML[w * 16 * MT + r];
          if (ml.x == -INFINITY) continue;
          const float a = ex2(ml.x - M);
          const float4 x = *(const float4*)(sO + (w * 16 * MT + r) * S::kORow + d0);
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

// Merge the splits' partials: D/4 threads a row, 4 elements each.
template <int D>
__global__ void __launch_bounds__(128) attn_q8_combine(const AttnQ8Params p) {
  constexpr int LPR = D / 4;
  const int R = p.n_max * p.g;
  const int qr = blockIdx.x * (128 / LPR) + threadIdx.x / LPR;
  const int grp = blockIdx.y, b = grp / p.c.hkv, kvh = grp % p.c.hkv;
  const int d0 = threadIdx.x % LPR * 4;
  pdl_wait();
  pdl_trigger();
  if (qr >= R) return;
  int n, T;
  attn_q8_lengths(p, b, false, n, T);
  const int64_t at = row_index(p, b, kvh, qr);
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (qr < n * p.g) {
    const int64_t row = (int64_t)grp * p.nsplit * R + qr;
    constexpr int kFly = 8;
    for (int s0 = 0; s0 < p.nsplit; s0 += kFly) {
      float2 ml[kFly];
      float4 v[kFly];
#pragma unroll
      for (int e = 0; e < kFly; ++e)
        ml[e] = s0 + e < p.nsplit ? p.part_ml[row + (int64_t)(s0 + e) * R] : make_float2(-INFINITY, 0.f);
      float Mg = M;
#pragma unroll
      for (int e = 0; e < kFly; ++e) {
        Mg = fmaxf(Mg, ml[e].x);
        if (ml[e].x != -INFINITY) v[e] = *(const float4*)(p.part_o + (row + (int64_t)(s0 + e) * R) * D + d0);
      }
      if (Mg == -INFINITY) continue;
      const float back = M == -INFINITY ? 0.f : ex2(M - Mg);
      L *= back;
      acc.x *= back;
      acc.y *= back;
      acc.z *= back;
      acc.w *= back;
#pragma unroll
      for (int e = 0; e < kFly; ++e)
        if (ml[e].x != -INFINITY) {
          const float a = ex2(ml[e].x - Mg);
          L = fmaf(ml[e].y, a, L);
          acc.x = fmaf(v[e].x, a, acc.x);
          acc.y = fmaf(v[e].y, a, acc.y);
          acc.z = fmaf(v[e].z, a, acc.z);
          acc.w = fmaf(v[e].w, a, acc.w);
        }
      M = Mg;
    }
  }
  const float inv = M == -INFINITY ? 0.f : 1.f / L;
  *(uint2*)(p.out + at * D + d0) =
      make_uint2(f32x2_to_bf16x2(acc.x * inv, acc.y * inv), f32x2_to_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse_out && d0 == 0)
    p.lse_out[at] = M == -INFINITY ? -INFINITY : (M + __log2f(L)) * 0.69314718055994531f;
}

struct Plan {
  int mt, tiles, nsplit, steps_per_split;
};

// Row tiles of 16 (or 32 when there are more rows) and KV splits.
Plan plan_of(const ddt_attn_q8_args* a) {
  Plan pl;
  const long R = (long)a->n_max * (a->hq / a->cache.hkv);
  pl.mt = R > 16 ? 2 : 1;
  pl.tiles = (int)((R + 16 * pl.mt - 1) / (16 * pl.mt));
  const long base = (long)pl.tiles * a->batch * a->cache.hkv;
  const long steps = (a->max_ctx + kStep - 1) / kStep + (a->n_max + kStep - 1) / kStep;
  const long slots = (long)device_sm_count() * (pl.mt == 1 ? 3 : 2);
  // as many splits as fill the device, of at least 4 steps a warp
  long ns = std::max(1L, slots / std::max(1L, base));
  ns = std::min(ns, std::max(1L, steps / (4 * kWarps)));
  ns = std::min(ns, 65535L);
  pl.steps_per_split = (int)((steps + ns - 1) / ns);
  pl.nsplit = (int)((steps + pl.steps_per_split - 1) / pl.steps_per_split);
  return pl;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

template <int D, int MT>
cudaError_t launch_narrow(const AttnQ8Params& p, int tiles, cudaStream_t stream) {
  const size_t smem = Smem<D, MT>::kTotal;
  cudaError_t e = ensure_smem_attr((const void*)attn_q8_kernel<D, MT>, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_q8_kernel<D, MT>, dim3(tiles, p.nsplit, p.batch * p.c.hkv), dim3(kThreads), smem, stream,
                    0, p);
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
  const Plan pl = plan_of(a);
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
  p.nsplit = pl.nsplit;
  p.steps_per_split = pl.steps_per_split;
  const size_t rows = (size_t)a->batch * a->cache.hkv * pl.nsplit * a->n_max * p.g;
  p.part_o = pl.nsplit > 1 ? (float*)ws : nullptr;
  p.part_ml = pl.nsplit > 1 ? (float2*)((char*)ws + align256(rows * a->cache.d * sizeof(float))) : nullptr;
  cudaError_t e;
  if (a->cache.d == 128)
    e = pl.mt == 1 ? launch_narrow<128, 1>(p, pl.tiles, stream) : launch_narrow<128, 2>(p, pl.tiles, stream);
  else
    e = pl.mt == 1 ? launch_narrow<64, 1>(p, pl.tiles, stream) : launch_narrow<64, 2>(p, pl.tiles, stream);
  if (e != cudaSuccess) return DDT_ERR_CUDA;
  if (pl.nsplit > 1) {
    const int per = 128 / (a->cache.d / 4);
    const dim3 grid((a->n_max * p.g + per - 1) / per, a->batch * a->cache.hkv);
    e = a->cache.d == 128 ? launch_pdl(attn_q8_combine<128>, grid, dim3(128), 0, stream, 0, p)
                          : launch_pdl(attn_q8_combine<64>, grid, dim3(128), 0, stream, 0, p);
    if (e != cudaSuccess) return DDT_ERR_CUDA;
  }
  return DDT_OK;
}

}  // namespace ddt
