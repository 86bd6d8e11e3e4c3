// attn_q8_wide.cu -- tree attention over the 8-bit key/value cache on the
// tcgen05 tensor cores: d = 128 and more than 32 query rows per kv head.
//
// Mathematics: as in attn_q8.cu (codes as f16, K exponents on the scores, V
// exponents in the softmax's reference, queries f16 under a power of two per
// row); each tree row becomes f16 under its own powers of two for K and V, which
// the softmax's reference takes as it takes the blocks'.  P is f16 too, so
// kind::f16 takes both products with f16 operands.
//
// What bounds it: R rows of a kv head want 4 R d flops per context token, so
// the tensor pipe, and beside it the 2^x of every score (MUFU) and the shared
// memory that feeds the MMAs.  One CTA per SM takes two tiles of 128 rows
// (A, B) of a kv head and KV tiles of 128 tokens, each converted once for both:
//   * warpgroups 3 and 4 convert K and V: codes come from global memory into
//     registers (the next tile's loads are issued as the last one's registers
//     are used up), become f16, and go to a ring of two 32 KB slots each in
//     the 128-byte swizzle that the MMAs read; tree rows likewise.  The codes
//     never pass through a staging buffer, and any page size works, since no
//     box has to fit a page; what is not in the context is not read;
//   * warp 1 issues the MMAs by steps of 64 tokens, PV_A(j), QK_A(j+2), PV_B(j),
//     QK_B(j+2): a tile's scores have two buffers, so the softmax of step j + 1
//     runs while the products around step j do;
//   * warpgroups 1 and 2 are the softmax of A and B, a row per thread: the 64
//     scores in registers, the context bound and the ancestor bitset as masks,
//     P over the scores' columns, O rescaled only when the reference moves; tree
//     rows, with scales and mask bits of their own, in a second loop.
// Registers go to where they are needed by setmaxnreg: 40 + 2 x 120 + 2 x 96.
// KV splits write (O, m, l) partials that attn_q8_combine merges.  Every wait
// is bounded; one that gives up raises DDT_ERR_TIMEOUT.
// Measured, one call behind a flush of L2 / back to back for 2 s: 8 trees of 257
// rows over 8192 tokens, 64/8 heads, 623 / 576 us = 0.71 / 0.77 PFLOP/s, under
// half of cuBLAS's bf16 rate (the bf16 kernel over the same context: 526 / 516
// us); 16 ragged trees of 129 rows 393 / 354 us (bf16: 469 / 450 us).  Under the
// power cap, in longer runs, up to 670 us and 435 us.  The MMAs are busy two
// thirds of a step, MUFU and the issue slots half of it each.
#include <cfloat>

#include "attn_q8.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace ddt {
namespace {

constexpr int BM = 128, BN = 128, D = 128;
constexpr int kThreads = 640;
constexpr int kRegs0 = 40, kRegsSoftmax = 120, kRegsConvert = 96;  // of a thread of each warpgroup
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;   // tile t: S of step j at 128 t + 64 (j & 1), O at 256 + 128 t
constexpr int kHalfTile = BN * 128;          // a 64-wide slice: 128 rows x 128 bytes
constexpr int kTile = 2 * kHalfTile;         // 32 KB
constexpr int kSlots = 4;
constexpr float kSlack = 6.f;                // the reference moves when a score passes it by 2^6
constexpr float kHead = 9.f;                 // P of a new maximum is 2^9: at most 2^15 in f16
constexpr float kFar = 1048576.f;            // references from here on have a last place of 2^-3 and more
constexpr int kGroup = 16;                   // tokens that share a place and an exponent
constexpr int kGroups = BN / kGroup;
constexpr int SN = 64;                       // tokens of a softmax step: half a KV tile

struct __align__(16) Shared {
  uint64_t q_full;
  uint64_t kv_full[kSlots], kv_empty[kSlots];
  uint64_t sc_full[4];        // the scales of tile i (ring of 4 tiles)
  uint64_t s_full[2][2], p_full[2][2];  // [tile][step & 1]
  uint64_t o_full, drain;
  long long wait_cycles;
  uint32_t tmem_base;
  int abort, pick;
  float2 scales[4][kGroups];  // context tile: (what a K product counts for, V exponent) of each group
  // tree tile: the same of each row, and 2^-(V exponent)
  __align__(16) float row_k[4][BN], row_v[4][BN], row_d[4][BN];
  uint32_t odd[32];           // tree rows with a wild V element
};

__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, Shared* sh) {
  return mbar_wait_bounded(b, parity, &sh->abort, sh->wait_cycles);
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// kind::f16, f16 x f16 -> f32, M = 128, A K-major; B K-major or MN-major.
constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);
}
// One lane of a converged warp (the MMA issuer's: 661 us for 8 trees of 257 rows
// over 8192 tokens, 681 us under `lane == 0`, at the step that took it).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// A shared-memory descriptor from its varying low word (128-byte swizzle, 1024
// bytes between groups of 8 rows), so that the issuer's registers hold one word each.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  return ((uint64_t)((1024u >> 4) | (1u << 14) | (2u << 29)) << 32) | lo;
}
__device__ __forceinline__ uint32_t desc_lo(const void* at, uint32_t lbo_bytes) {
  return ((smem_u32(at) >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);
}
// Byte offset of 16-byte chunk `ch` (0..15) of row r in a tile of two 64-wide slices.
__device__ __forceinline__ uint32_t tile_at(int r, int ch) {
  return (uint32_t)((ch >> 3) * kHalfTile + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

__global__ void __launch_bounds__(kThreads, 1) attn_q8_wide_kernel(const AttnQ8Params p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = (unsigned char*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  unsigned char* sQ = smem;                // [2 tiles]
  unsigned char* sKV = smem + 2 * kTile;   // [kSlots]
  Shared* sh = (Shared*)(sKV + kSlots * kTile);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
  const int pair = blockIdx.x, split = blockIdx.y;
  if (tid == 0) {
    mbar_init(&sh->q_full, 8);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sh->kv_full[s], 4);
      mbar_init(&sh->kv_empty[s], 1);
      mbar_init(&sh->sc_full[s], 8);
    }
    for (int t = 0; t < 2; ++t)
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sh->s_full[t][h], 1);
        mbar_init(&sh->p_full[t][h], 4);
      }
    mbar_init(&sh->o_full, 1);
    mbar_init(&sh->drain, 1);
    sh->wait_cycles = p.wait_cycles;
    sh->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < 32) sh->odd[tid] = 0;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&sh->tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  const int grp = group_of(p, blockIdx.z, &sh->pick);
  const int b = grp / p.c.hkv, kvh = grp % p.c.hkv;
  const int g = p.g, R = p.n_max * g, q0 = pair * 2 * BM;
  int n, T;
  attn_q8_lengths(p, b, pair == 0 && split == 0 && kvh == 0 && tid == 0, n, T);
  // a tile works when one of its rows belongs to a tree row
  const int live = n * g;
  const bool has_a = q0 < live, has_b = q0 + BM < live;
  const int nct = (T + BN - 1) / BN;
  const int ntt = (n + BN - 1) / BN;
  const int t_lo = min(split * p.steps_per_split, nct + ntt);
  const int t_hi = min(t_lo + p.steps_per_split, nct + ntt);
  const int ntiles = has_a ? t_hi - t_lo : 0;

  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (wg == 0) {
    regs_dec<kRegs0>();
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    if (warp == 1 && ntiles > 0 && elect_one()) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t kIdQK = idesc_f16(SN, false), kIdPV = idesc_f16(D, true);
      const int nt = has_b ? 2 : 1, steps = 2 * ntiles;
      const uint32_t q_lo = desc_lo(sQ, 16), k_lo = desc_lo(sKV, 16), v_lo = desc_lo(sKV, kHalfTile);
      // S_x(j) = Q_x K^T for step j: tokens 64 (j & 1) .. of tile j / 2
      auto qk = [&](int x, int j) {
        const uint32_t q = q_lo + x * (kTile >> 4);
        const uint32_t k = k_lo + (j & 2) * (kTile >> 4) + (j & 1) * (SN * 128 >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (uint32_t)((kk >> 2) * kHalfTile + (kk & 3) * 32) >> 4;
          mma_ss(tm + kColS + 128 * x + SN * (j & 1), desc_of(q + off), desc_of(k + off), kIdQK, kk > 0 ? 1u : 0u);
        }
      };
      auto pv = [&](int x, int j) {  // O_x += P_x V, P_x in the first half of S_x(j)'s columns
        const uint32_t v = v_lo + ((j & 2) + 1) * (kTile >> 4) + (j & 1) * (SN * 128 >> 4);
#pragma unroll
        for (int kk = 0; kk < SN / 16; ++kk)
          mma_ts(tm + kColO + 128 * x, tm + kColS + 128 * x + SN * (j & 1) + kk * 8, desc_of(v + kk * (2048 >> 4)),
                 kIdPV, (j > 0 || kk > 0) ? 1u : 0u);
      };
      bool go = wait(&sh->q_full, 0, sh) && wait(&sh->kv_full[0], 0, sh);
      if (go) {
        fence_after();
        for (int j = 0; j < 2; ++j)
          for (int x = 0; x < nt; ++x) {
            qk(x, j);
            mma_commit(&sh->s_full[x][j]);
          }
        mma_commit(&sh->kv_empty[0]);  // K_0
      }
      // Tile i's slots: K at 2 i & 2, V behind it.  S_x(j + 2) follows PV_x(j),
      // whose P shares its columns; S_x(j + 1) is there meanwhile, so the softmax
      // of a step never waits for its own product.
      for (int j = 0; go && j < steps; ++j) {
        const int i = j >> 1;
        const bool next = j + 2 < steps;
        if ((j & 1) == 0)
          go = wait(&sh->kv_full[(j & 2) + 1], (uint32_t)(i >> 1) & 1u, sh) &&
               (!next || wait(&sh->kv_full[(j + 2) & 2], (uint32_t)((i + 1) >> 1) & 1u, sh));
        for (int x = 0; go && x < nt; ++x) {
          go = wait(&sh->p_full[x][j & 1], (uint32_t)i & 1u, sh);
          if (!go) break;
          fence_after();
          pv(x, j);
          if (next) qk(x, j + 2);
          mma_commit(&sh->s_full[x][j & 1]);  // (also when there is no S: PV_x(j) is complete behind it)
        }
        if (!go) break;
        if (j & 1) {
          mma_commit(&sh->kv_empty[(j & 2) + 1]);           // V_i: every PV of tile i issued
          if (next) mma_commit(&sh->kv_empty[(j + 2) & 2]);  // K_{i+1}
        }
      }
      if (go) mma_commit(&sh->o_full);
      if (*(volatile int*)&sh->abort) {
        int keep_going = 0;
        mma_commit(&sh->drain);
        mbar_wait_bounded(&sh->drain, 0u, &keep_going, kDrainCycles);
      }
    }
  } else if (wg >= 3) {
    // ------------------------------------------------------------ converters
    static_assert(kRegsConvert == 96, "what the block is launched with");
    const int kind = wg - 3;  // K, V
    const int cw = warp & 3, ct = tid & 127;
    const int tok = ct >> 2, c4 = ct & 3;  // of 32 tokens; 16 elements of a 64-wide slice
    const uint32_t stride = (uint32_t)p.c.hkv * D;
    const int nctx = min(max(nct - t_lo, 0), ntiles);  // context tiles of this CTA
    // places and exponents of the 16-token groups of 4 tiles, a group a lane; a
    // group that is not there (row -1) is zeros and weighs nothing
    struct LookUp {
      int row, e;
    };
    constexpr int kMissing = 1 << 16;  // exponent of a group that is not there
    const int8_t* exps = kind ? p.c.ve : p.c.ke;
    auto look_up = [&](int i) -> LookUp {  // of tiles i .. i + 3
      LookUp u{-1, kMissing};
      const int64_t pos = ((int64_t)(t_lo + i) * kGroups + lane) * kGroup;
      if (i + (lane >> 3) < nctx && pos < T) {
        const Q8Place at = q8_place(p.c, b, pos);
        if (at.row < 0) {
          if (warp == 12) raise_status(p.status, DDT_ERR_INVALID_ARG);
        } else {
          u.row = (int)at.row;
          u.e = exps[at.blk * p.c.hkv + kvh];
        }
      }
      return u;
    };
    // codes of the next tile to convert: pass q holds slice q & 1 of tokens
    // 32 (q / 2) + tok, of group 2 (q / 2) + (cw >= 2); what is not in the context
    // is neither read nor anything but 0 (codes there may be anything, NaN too)
    uint4 x[8];
    const uint8_t* lane_src =
        (kind ? p.c.vc : p.c.kc) + (int64_t)kvh * D + (tok & 15) * (int64_t)stride + c4 * 16;
    auto load = [&](const LookUp& u, int i, int q, int left) {
      const int r = __shfl_sync(0xFFFFFFFFu, u.row, (i & 3) * 8 + (q >> 1) * 2 + (cw >> 1));
      x[q] = ld_stream_v4_if(lane_src + (uint64_t)(uint32_t)r * stride + (q & 1) * 64,
                             q8_wide_reads(r, q, left));
    };
    // 16 elements as f16 to their two chunks of row r (of rows of two parities
    // a quarter warp writes, the swizzle gives eight different banks)
    auto store = [&](unsigned char* dst, int r, int slice, uint4 lo, uint4 hi) {
      *(uint4*)(dst + tile_at(r, slice * 8 + 2 * c4)) = lo;
      *(uint4*)(dst + tile_at(r, slice * 8 + 2 * c4 + 1)) = hi;
    };
    auto slot_of = [&](int i) { return (2 * i + kind) & 3; };
    auto slot_free = [&](int i) {
      return __all_sync(0xFFFFFFFFu, wait(&sh->kv_empty[slot_of(i)], ((uint32_t)(i >> 1) & 1u) ^ 1u, sh));
    };
    auto done = [&](int i) {  // tile i is in its slot
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->kv_full[slot_of(i)]);
    };
    bool go = true;
    LookUp now = {}, then = {};
    if (nctx > 0) {
      now = look_up(0);
#pragma unroll
      for (int q = 0; q < 8; ++q) load(now, 0, q, q8_wide_left(T, t_lo, tok));
    }
    for (int i = 0; go && i < nctx; ++i) {
      const int e = __shfl_sync(0xFFFFFFFFu, now.e, (i & 3) * 8 + (lane & 7));
      if (cw == 0 && lane < kGroups) {
        // what a K code counts for; the V exponent
        if (kind == 0)
          sh->scales[i & 3][lane].x = e == kMissing ? 1.f : q8_scale(e);
        else
          sh->scales[i & 3][lane].y = e == kMissing ? -INFINITY
                                                    : e == DDT_Q8_EXP_NAN ? __int_as_float(0x7FC00000)
                                                                          : (float)q8_exp(e);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->sc_full[i & 3]);
      if ((i & 3) == 1) then = look_up((i & ~3) + 4);
      if ((i & 3) == 3) now = then;  // from here on for tile i + 1
      go = slot_free(i);
      if (!go) break;
      unsigned char* dst = sKV + slot_of(i) * kTile;
      const int left = q8_wide_left(T, t_lo + i + 1, tok);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint4 v = x[q];
        if (i + 1 < nctx) load(now, i + 1, q, left);
        store(dst, (q >> 1) * 32 + tok, q & 1, make_uint4(codes_lo(v.x), codes_hi(v.x), codes_lo(v.y), codes_hi(v.y)),
              make_uint4(codes_lo(v.z), codes_hi(v.z), codes_lo(v.w), codes_hi(v.w)));
      }
      done(i);
    }
    for (int i = nctx; go && i < ntiles; ++i) {
      // ---- a tile of tree rows: bf16 to f16 under a power of two per row, so that
      // no row's size shows in another's (the mask may hide it)
      const int row0 = (t_lo + i - nct) * BN;
      const uint16_t* src = (kind ? p.vt : p.kt) + (((int64_t)b * p.n_max + row0) * p.c.hkv + kvh) * D + c4 * 16;
      unsigned char* dst = sKV + slot_of(i) * kTile;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {  // 64 rows
        uint4 w[4][2];  // pass q as for the codes
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = half * 64 + (q >> 1) * 32 + tok;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            w[q][h] = make_uint4(0, 0, 0, 0);
            if (row0 + r < n) w[q][h] = __ldg((const uint4*)(src + (int64_t)r * stride + (q & 1) * 64) + h);
          }
        }
        float inv[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {  // a row: four lanes, two slices
          uint32_t m = 0;
          bool odd = false;
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint4& v = w[2 * q + (h >> 1)][h & 1];
            if (kind) {  // wild V elements go to their rows at the end, and to no others
              odd |= has_wild(v.x) || has_wild(v.y) || has_wild(v.z) || has_wild(v.w);
              v = make_uint4(tame_bf16x2(v.x), tame_bf16x2(v.y), tame_bf16x2(v.z), tame_bf16x2(v.w));
            }
            m = max_finite_bf16(max_finite_bf16(max_finite_bf16(max_finite_bf16(m, v.x), v.y), v.z), v.w);
          }
          const int r = half * 64 + q * 32 + tok;
          if (odd) atomicOr(&sh->odd[(row0 + r) >> 5], 1u << ((row0 + r) & 31));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
          m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
          const int e = tree_exponent(m);
          inv[q] = pow2i(-e);
          if (c4 == 0) {
            if (kind == 0) {
              sh->row_k[i & 3][r] = pow2i(e);
            } else {
              sh->row_v[i & 3][r] = (float)e;
              sh->row_d[i & 3][r] = inv[q];
            }
          }
        }
        if (half) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->sc_full[i & 3]);
        } else {
          go = slot_free(i);
          if (!go) break;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 f[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t u[4] = {w[q][h].x, w[q][h].y, w[q][h].z, w[q][h].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) u[z] = bf16x2_to_f16x2(u[z], inv[q >> 1]);
            f[h] = make_uint4(u[0], u[1], u[2], u[3]);
          }
          store(dst, half * 64 + (q >> 1) * 32 + tok, q & 1, f[0], f[1]);
        }
      }
      if (go) done(i);
    }
    asm volatile("bar.arrive 2, 512;" ::: "memory");
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<kRegsSoftmax>();
    const int t = wg - 1;                            // softmax tile
    const int row = (warp & 3) * 32 + lane;
    const int qr = q0 + t * BM + row, jq = qr / g;
    const bool tile_live = t == 0 ? has_a : has_b;
    const bool row_valid = tile_live && qr < live;
    const int qr0 = q0 + t * BM + (warp & 3) * 32;   // the warp's first row
    auto out_row = [&](int q) { return ((int64_t)b * p.n_max + q / g) * p.hq + kvh * g + q % g; };
    // ---- Q as f16 under a power of two per row: half a warp loads a row
    float mul = 0.f;
    if (tile_live && ntiles > 0) {
      unsigned char* dst = sQ + t * kTile;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 16) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + 2 * i + (lane >> 4);
          v[i] = make_uint4(0, 0, 0, 0);
          if (qr0 + r < live) v[i] = __ldg((const uint4*)(p.q + out_row(qr0 + r) * D) + (lane & 15));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = r0 + 2 * i + (lane >> 4);
          uint32_t m = max_finite_bf16(max_finite_bf16(max_finite_bf16(max_finite_bf16(0, v[i].x), v[i].y), v[i].z), v[i].w);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          const int e = m ? max(f16_exponent(m, 14), -126) : 0;
          const float inv = pow2i(-e);
          *(uint4*)(dst + tile_at((warp & 3) * 32 + r, lane & 15)) =
              make_uint4(bf16x2_to_f16x2(v[i].x, inv), bf16x2_to_f16x2(v[i].y, inv), bf16x2_to_f16x2(v[i].z, inv),
                         bf16x2_to_f16x2(v[i].w, inv));
          const float f = __shfl_sync(0xFFFFFFFFu, p.scale_log2 * pow2i(e), (lane & 1) * 16);
          if ((lane >> 1) == (r0 >> 1) + i) mul = f;  // lanes 2 i, 2 i + 1 own these two rows
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->q_full);
    float m_ref = -INFINITY, l = 0.f;
    bool ok = true;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_col = lane_base + kColS + 128 * t, o_col = lane_base + kColO + 128 * t;
    const uint32_t* mrow = p.mask + ((int64_t)b * p.n_max + (row_valid ? jq : 0)) * p.W;
    // the scores of step j are there
    auto scores_of = [&](int j) {
      const int i = j >> 1, half = j & 1;
      const bool there = __all_sync(0xFFFFFFFFu, (half || wait(&sh->sc_full[i & 3], (uint32_t)(i >> 2) & 1u, sh)) &&
                                                     wait(&sh->s_full[t][half], (uint32_t)i & 1u, sh));
      if (there) fence_after();
      return there;
    };
    // the reference, and with it l, for a step whose largest t is `top`: what O has to be multiplied by
    auto refer = [&](float top, bool& move) {
      float alpha = 1.f;
      move = top - m_ref > kSlack + kHead;
      if (move) {
        const float to = reference_below(top, kHead, kSlack);
        alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - to);
        m_ref = to;
        l *= alpha;
      }
      return alpha;
    };
    // P of step j is written: O under the reference, then the product may begin
    auto hand_over = [&](int j, float alpha, bool move) {
      const int half = j & 1;
      if (j > 0 && __any_sync(0xFFFFFFFFu, move)) {
        // PV_t(j - 1) is complete behind the next commit on the other half's S
        if (!__all_sync(0xFFFFFFFFu, wait(&sh->s_full[t][half ^ 1], (uint32_t)((j + 1) >> 1) & 1u, sh))) return false;
        fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(o_col + 32 * c, o);
        }
      }
      tmem_st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full[t][half]);
      return true;
    };

    const int ctx_steps = 2 * min(max(nct - t_lo, 0), ntiles);
    for (int j = 0; tile_live && j < ctx_steps; ++j) {
      const int i = j >> 1, half = j & 1;
      const int cnt = min(SN, T - (t_lo + i) * BN - half * SN);
      ok = scores_of(j);
      if (!ok) break;
      const float2* scale = &sh->scales[i & 3][half * (SN / kGroup)];
      uint32_t r[SN];
#pragma unroll
      for (int c = 0; c < SN / 32; ++c) tmem_ld32(s_col + half * SN + 32 * c, r + 32 * c);
      tmem_ld_wait();
      if (cnt < SN) {
#pragma unroll
        for (int e = 0; e < SN; ++e)
          if (e >= cnt) r[e] = 0xFF800000u;  // -inf
      }
      // t = f s + V exponent; its largest from the largest s of each group (f > 0)
      float f[SN / kGroup], ev[SN / kGroup], top = -INFINITY;
#pragma unroll
      for (int q = 0; q < SN / kGroup; ++q) {
        const float2 sc = scale[q];
        f[q] = mul * sc.x;
        if (f[q] < FLT_MIN) f[q] = FLT_MIN;  // (all that it multiplies is nothing then; -inf has to stay -inf)
        ev[q] = sc.y;
        float m2[2] = {__uint_as_float(r[q * 16]), __uint_as_float(r[q * 16 + 1])};
#pragma unroll
        for (int e = 2; e < kGroup; e += 2)
          m2[(e >> 1) & 1] = fmax3(m2[(e >> 1) & 1], __uint_as_float(r[q * 16 + e]), __uint_as_float(r[q * 16 + e + 1]));
        top = fmaxf(top, fmaf(fmaxf(m2[0], m2[1]), f[q], ev[q]));
      }
      bool move;
      const float alpha = refer(top, move);
      const float m = m_ref == -INFINITY ? 0.f : m_ref;
      float c_of[SN / kGroup];  // P = 2^(f s + c)
#pragma unroll
      for (int q = 0; q < SN / kGroup; ++q) c_of[q] = ev[q] - m;
      if (fabsf(m) > kFar) {
        // t rounded first, as its maximum was: in one fma with m, P could pass f16's range
#pragma unroll
        for (int q = 0; q < SN / kGroup; ++q) {
#pragma unroll
          for (int e = 0; e < kGroup; ++e)
            r[16 * q + e] = __float_as_uint(fmaf(__uint_as_float(r[16 * q + e]), f[q], ev[q]) - m);
          f[q] = 1.f;
          c_of[q] = 0.f;
        }
      }
      // P = 2^(t - m) as f16 pairs over the scores, its sum weighted by 2^-(V
      // exponent).  (A quarter of the 2^x on the FMA pipe instead of MUFU gave
      // 1 %, more of them lost: the issue slots are as scarce.)
#pragma unroll
      for (int c = 0; c < SN / 32; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int gq = 2 * c + q;
          const uint64_t f2 = pack2(f[gq], f[gq]), c2 = pack2(c_of[gq], c_of[gq]);
          uint64_t s2[2] = {0ull, 0ull};
#pragma unroll
          for (int e = 0; e < kGroup; e += 2) {
            const int at = 16 * gq + e;
            const uint64_t x2 = ffma2(pack2(__uint_as_float(r[at]), __uint_as_float(r[at + 1])), f2, c2);
            float a, z;
            unpack2(x2, a, z);
            a = ex2(a);
            z = ex2(z);
            s2[(e >> 1) & 1] = fadd2(s2[(e >> 1) & 1], pack2(a, z));
            pk[8 * q + (e >> 1)] = f32x2_to_f16x2(a, z);
          }
          float a, z;
          unpack2(fadd2(s2[0], s2[1]), a, z);
          l = fmaf(a + z, ev[gq] == -INFINITY ? 0.f : ex2(-ev[gq]), l);  // (a group that is not there: nothing)
        }
        tmem_st16(s_col + half * SN + 16 * c, pk);
      }
      ok = hand_over(j, alpha, move);
      if (!ok) break;
    }
    // Tree rows: scales by the row, masks by the bit.  Few steps of many, so in two
    // passes over 32 scores at a time, which leaves the context's steps their
    // registers (8 trees of 257 rows over 8192 tokens: 614 us, 596 us with a scale
    // per 16 rows, 757 us with the rows' scales in the body of every step).
    for (int j = ctx_steps; tile_live && ok && j < 2 * ntiles; ++j) {
      const int i = j >> 1, half = j & 1;
      const int base = (t_lo + i - nct) * BN + half * SN;
      ok = scores_of(j);
      if (!ok) break;
      // t of row base + e, -inf where the mask hides it, back over its score
      float top = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < SN / 32; ++c) {
        const int have = n - base - 32 * c;
        if (have <= 0) break;
        uint32_t bits = row_valid ? __ldg(mrow + (base >> 5) + c) : 0u;
        if (have < 32) bits &= (1u << have) - 1u;
        const float4* k4 = (const float4*)&sh->row_k[i & 3][half * SN + 32 * c];
        const float4* v4 = (const float4*)&sh->row_v[i & 3][half * SN + 32 * c];
        uint32_t r[32];
        tmem_ld32(s_col + half * SN + 32 * c, r);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float k[4] = {k4[e / 4].x, k4[e / 4].y, k4[e / 4].z, k4[e / 4].w};
          const float v[4] = {v4[e / 4].x, v4[e / 4].y, v4[e / 4].z, v4[e / 4].w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {  // (FLT_MIN: all that a smaller factor multiplies is nothing)
            const float x = fmaf(__uint_as_float(r[e + z]), fmaxf(mul * k[z], FLT_MIN), v[z]);
            r[e + z] = (bits >> (e + z)) & 1u ? __float_as_uint(x) : 0xFF800000u;
          }
          top = fmax3(top, __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
          top = fmax3(top, __uint_as_float(r[e + 2]), __uint_as_float(r[e + 3]));
        }
        tmem_st32(s_col + half * SN + 32 * c, r);
      }
      tmem_st_wait();
      bool move;
      const float alpha = refer(top, move);
      const float m = m_ref == -INFINITY ? 0.f : m_ref;
#pragma unroll 1
      for (int c = 0; c < SN / 32; ++c) {
        const float4* d4 = (const float4*)&sh->row_d[i & 3][half * SN + 32 * c];
        uint32_t r[32], pk[16];
        if (n - base - 32 * c <= 0) {  // no rows: no weights
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0u;
          tmem_st16(s_col + half * SN + 16 * c, pk);
          continue;
        }
        tmem_ld32(s_col + half * SN + 32 * c, r);
        tmem_ld_wait();
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float d[4] = {d4[e / 4].x, d4[e / 4].y, d4[e / 4].z, d4[e / 4].w};
          float w[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            w[z] = ex2(__uint_as_float(r[e + z]) - m);
            sum[z] = fmaf(w[z], d[z], sum[z]);
          }
          pk[e / 2] = f32x2_to_f16x2(w[0], w[1]);
          pk[e / 2 + 1] = f32x2_to_f16x2(w[2], w[3]);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st16(s_col + half * SN + 16 * c, pk);
      }
      ok = hand_over(j, alpha, move);
    }
    if (tile_live && ok && ntiles > 0) ok = __all_sync(0xFFFFFFFFu, wait(&sh->o_full, 0, sh));
    asm volatile("bar.sync 2, 512;" ::: "memory");  // the converter's marks in sh->odd are complete
    fence_after();

    // ---- epilogue: O rows to the output or to a split's partial
    if (l != l)
      m_ref = 0.f;  // a row of NaN scores alone has no reference: any number carries its NaN on
    else if (m_ref == -INFINITY)
      l = 0.f;      // a row that saw nothing
    const bool final_out = p.nsplit == 1;
    const bool has = ok && row_valid && ntiles > 0 && l != 0.f;  // (NaN counts as a sum)
    const float inv = has ? 1.f / l : 0.f;
    const bool writes = final_out ? qr < R : row_valid;
    const int64_t part0 = ((int64_t)grp * p.nsplit + split) * R;
    unsigned char* stage = smem + (t * 4 + (warp & 3)) * (32 * D * 4);
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      if (tile_live && ntiles > 0) {  // (warp-collective)
        tmem_ld32(o_col + 32 * c, o);
        tmem_ld_wait();
      }
      if (!has) {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      } else if (t_hi > nct) {
        // wild V elements of the tree rows that this row sees, in this CTA's tiles
        const int w_lo = max(t_lo - nct, 0) * 4, w_hi = min((t_hi - nct) * 4, p.W);
#pragma unroll 1
        for (int w = w_lo; w < w_hi; ++w) {
          uint32_t bits = sh->odd[w];
          if (bits) bits &= __ldg(p.mask + ((int64_t)b * p.n_max + jq) * p.W + w);
          while (bits) {
            const int tr = w * 32 + __ffs(bits) - 1;
            bits &= bits - 1;
            const uint16_t* v = p.vt + (((int64_t)b * p.n_max + tr) * p.c.hkv + kvh) * D + 32 * c;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint16_t z = v[e];
              if (is_wild(z)) o[e] = __float_as_uint(__uint_as_float(o[e]) + wild_value(z));
            }
          }
        }
      }
      if (final_out) {
        if (writes) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = f32x2_to_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          uint4* dst = (uint4*)(p.out + out_row(qr) * D + 32 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
        }
      } else {
        // through shared memory (every product has read it), so that a warp writes whole rows
#pragma unroll
        for (int e = 0; e < 8; ++e)
          *(uint4*)(stage + lane * 512 + (((8 * c + e) ^ lane) << 4)) =
              make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
    }
    __syncwarp();  // lanes read one another's rows from here on (a vote orders no memory)
    const uint32_t write_rows = __ballot_sync(0xFFFFFFFFu, writes && !final_out);
    if (write_rows) {
      float* dst = p.part_o + (part0 + qr0) * D + 4 * lane;
#pragma unroll 8
      for (int r = 0; r < 32; ++r)
        if ((write_rows >> r) & 1u) *(float4*)(dst + r * D) = *(const float4*)(stage + r * 512 + ((lane ^ r) << 4));
    }
    if (writes && final_out) {
      if (p.lse_out) p.lse_out[out_row(qr)] = has ? (m_ref + __log2f(l)) * 0.69314718055994531f : -INFINITY;
    } else if (writes) {
      p.part_ml[part0 + qr] = has ? make_float2(m_ref, l) : make_float2(-INFINITY, 0.f);
    }
  }
  pdl_trigger();
  fence_before();
  __syncthreads();
  if (tid == 0 && sh->abort) raise_status(p.status, DDT_ERR_TIMEOUT);
  if (warp == 0) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

}  // namespace

cudaError_t launch_attn_q8_wide(const AttnQ8Params& p, int pairs, cudaStream_t stream) {
  // the warpgroups' shares have to come out of what the block is launched with
  static_assert(kRegs0 + 2 * kRegsSoftmax + 2 * kRegsConvert <= 96 * kThreads / 128, "register split");
  static const int regs = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, attn_q8_wide_kernel) == cudaSuccess ? fa.numRegs : 0;
  }();
  if (regs < 96) return cudaErrorInvalidConfiguration;
  const size_t smem = 1024 + (size_t)(2 + kSlots) * kTile + sizeof(Shared);
  const cudaError_t e = ensure_smem_attr((const void*)attn_q8_wide_kernel, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_q8_wide_kernel, dim3(pairs, p.nsplit, p.batch * p.c.hkv), dim3(kThreads), smem, stream, 0, p);
}

}  // namespace ddt
