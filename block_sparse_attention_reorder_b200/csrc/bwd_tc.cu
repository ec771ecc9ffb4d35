// dQ of the block-sparse attention backward on the 5th-generation tensor
// cores (tcgen05, TMEM accumulators, TMA-fed shared memory). The gradient of
// the trainable block-sparse attention ("Faster Video Diffusion with
// Trainable Sparse Attention", reproducibility record, Research Type row):
//   dQ_i = scale * sum_j dS_ij K_j,  dS_ij = P_ij * (dO_i V_j^T - Delta_i),
//   P_ij = 2^(scale log2(e) Q_i K_j^T - lse_i log2(e)),  Delta = rowsum(dO * O).
//
// Work unit, as in the forward kernel: a 128-row block of two 64-row chunks.
// With 64-token tiles, two adjacent query tiles (along t for top-k and top-p,
// the window's widest axis for a window) walking the union of their kept lists (a key tile
// kept by only one of the two gives zero dS to the other's rows); with tiles
// of several chunks, chunks 2b and 2b + 1 of one query tile walking every
// real chunk of each kept key tile.
//
// Roles (320 threads, one CTA per SM):
//   warps 0-7  warps w and w + 4 own query rows 32 (w % 4) .. (TMEM lanes);
//              warp w takes keys 0-31 of a step, warp w + 4 keys 32-63 (the
//              log-sum-exp is known, so the halves need no exchange). Each
//              reads its half of S and dP from TMEM, forms dS = P (dP - Delta)
//              in fp32 and writes it as bf16 over the first 16 columns of its
//              half of S.
//   warp 8     TMA producer: Q and dO blocks once, then K_j and V_j together
//              into a ring of three stages (a stage is released by the dQ MMA
//              that last reads K_j); with score rules of four stages where the
//              lists leave room (released by the S product two steps on).
//   warp 9     MMA issuer (the warp runs as a whole, one elected lane issues,
//              3.46 -> 2.69 ms with the rules; csrc/attn_mod_tc.cu has the
//              reason): S_n = Q K_n^T and dP_n = dO V_n^T (both SS, N = 64)
//              into double buffers, two steps ahead of the softmax side; dQ +=
//              dS_n K_n (dS from TMEM, K_n as an MN-major shared-memory
//              operand).
// TMEM (512 columns): S [0,64) and [64,128), dP [128,192) and [192,256), dQ
// [256, 256+D); with score rules dP [128,192), S's block operand [192,256), G
// [384, 384+D). Every mbarrier wait is bounded; on expiry the CTA sets the
// device error word, raises an abort flag, lets issued copies land, drains its
// MMAs and frees TMEM.
//
// Under score rules dQ is computed first and corrects Delta on the way: the
// rounding of O to bf16 puts an error eps_i into Delta_i, which costs dQ and
// dK more than all other roundings where the softmax is sharp. In a row of
// probabilities eps_i = sum_j P_ij (dP_ij - Delta_i), so the kernel sums that
// next to a second accumulator G_i = sum_j P_ij (1 - tanh^2) K_j (one more
// product a step) and writes dQ_i = scale (dQ_i - eps_i G_i) and -(Delta_i +
// eps_i), which the dK pass then reads.
//
// With the rules S takes its block operand (Q, or K) from TMEM, which leaves
// room for one dP buffer only; it is released as soon as the softmax side has
// read it, and dS and P go over the two halves of S. On one B200 the backward
// of the Wan-1.3B shape takes 2.48 ms without a rule, 3.01 with the cap, 3.54
// with cap and bias (3.53 by attn_backward, two dP buffers, one product fewer).
//
// Score rules (MOD, score_mod.cuh): P is recomputed from the capped, biased
// and masked scores; the step lists are filtered as in the forward. Hidden
// pairs take no part through selects (their scores may be NaN), and the rows
// of hidden tokens in a step's tiles are zeroed in shared memory before the
// product that sums over them.
#include <cudaTypedefs.h>

#include <math.h>

#include <type_traits>

#include "internal.h"
#include "score_mod.cuh"
#include "steps.cuh"
#include "tc_common.cuh"

namespace {

constexpr int kThreads = 320;
constexpr int kSoftmaxThreads = 256;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColDP = 128, kColOp = 192, kColDQ = 256, kColG = 384;
constexpr long long kWaitLimit = 4000000000LL;  // SM cycles (~2 s)

// A CTA's share of an accumulator row (fp32, the columns of half `part`), zeros
// where the row is no visible token or nothing was summed.
template <int D>
__device__ __forceinline__ void store_share(float* dst, uint32_t src, int part, bool summed, bool live) {
#pragma unroll
  for (int col = part * (D / 2); col < (part + 1) * (D / 2); col += 32) {
    uint32_t o[32];
    if (summed) tc::tmem_ld32_wait(src + col, o);
    if (!summed || !live) {
#pragma unroll
      for (int q = 0; q < 32; ++q) o[q] = 0u;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      reinterpret_cast<uint4*>(dst + col)[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
  }
}

// Row r of a 128-row block in shared memory (128-byte swizzled 64-column
// blocks of 16 KB) as an A operand in TMEM, two bf16 a column: the half that
// `part` names, by the warps that own the row's lanes.
template <int D>
__device__ __forceinline__ bool operand_to_tmem(const uint8_t* block, uint32_t dst, int part, int r, uint32_t bar_loaded,
                                                uint32_t bar_op, volatile int* abort_flag) {
  if (!__all_sync(0xffffffffu, tc::mbar_wait(bar_loaded, 0, abort_flag, kWaitLimit))) return false;
  if (part < D / 64) {
    uint32_t w[32];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4*>(w + 4 * c) =
          *reinterpret_cast<const uint4*>(block + part * 128 * 128 + r * 128 + ((c ^ (r & 7)) << 4));
    tc::tmem_st32(dst + 32 * part, w);
    tc::tmem_wait_st();
  }
  tc::fence_before_sync();
  tc::mbar_arrive(bar_op);
  return true;
}

struct DqParams {
  Geom g;
  const int32_t* idx;
  const int32_t* cnt;
  const float* lse;    // tiled [B, Hh, N, 64], natural log
  const float* delta;  // tiled [B, Hh, N, 64]
  int kmax;
  __nv_bfloat16* dq;
  float scale;
  float scale_log2;
  int* err;
  int umax;
  int bm_words;
  int pair_axis;
  int pdim[3];
};

struct DqParamsMod : DqParams {
  ModParams mod;
  float* neg_delta;    // gets -(Delta + eps) of every row, 0 where no gradient passes
  float* neg_lse2;     // gets -lse log2(e) of every row, -inf where no gradient passes
  float* slope_parts;  // null, or [B * heads, backward_slope_items]: the slope gradient's parts
  int shares;          // CTAs that share a query block's steps
  float* part_q;       // shares > 1: [blocks, shares, 2, 128, D] dQ and G
  float4* part_s;      // [blocks, shares, 128] (sum w, sum w dist, sum P dist, -Delta) of each row
};

template <int D, bool MOD, int kStages>
struct DqCfg {
  static constexpr int QRB = D * 2;                  // row bytes
  static constexpr int QBLK = QRB / 128;             // 128-byte column blocks
  static constexpr int NKS = QRB / 32;               // K = 16 MMAs per product
  static constexpr int BLK_BYTES = 128 * QRB;        // 128-row block (Q, dO)
  static constexpr int T_BYTES = 64 * QRB;           // one 64-row tile (K, V)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = OFF_Q + BLK_BYTES;
  static constexpr int OFF_K = OFF_DO + BLK_BYTES;
  static constexpr int OFF_V = OFF_K + kStages * T_BYTES;
  static constexpr int OFF_BAR = OFF_V + kStages * T_BYTES;
  // barriers: q, full[S], empty[S], sfull[2], pfull[2], final
  static constexpr int NBAR = 1 + 2 * kStages + 5 + (MOD ? 2 : 0);  // score rules: operand in TMEM, dP read
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tmem base, abort, L, zero
  static constexpr int OFF_COL = OFF_MISC + 16;        // 64 packed in-tile coordinates
  static constexpr int OFF_SCAN = OFF_COL + 256;
  static constexpr int OFF_TAB = OFF_SCAN + 64;        // score rules: row offsets, chunk origins
  static constexpr int OFF_DYN = OFF_TAB + (MOD ? (int)sizeof(ModTab) : 0);  // bitmaps, step list, extents
  static_assert(OFF_TAB % 16 == 0, "float4 reads of the table");
  static constexpr int O_PITCH = D * 2 + 16;           // epilogue staging pitch
  static_assert(128 * O_PITCH <= OFF_BAR - OFF_K, "epilogue staging fits in the rings");
};

template <int D, bool MOD, int kStages>
__global__ void __launch_bounds__(kThreads, 1)
bwd_dq_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                 const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const __grid_constant__ std::conditional_t<MOD, DqParamsMod, DqParams> P) {
  using C = DqCfg<D, MOD, kStages>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = tc::smem_addr(smem);
  const uint32_t bar_q = sb + C::OFF_BAR;
  auto bar_full = [&](int s) { return sb + C::OFF_BAR + 8u * (1 + s); };
  auto bar_empty = [&](int s) { return sb + C::OFF_BAR + 8u * (1 + kStages + s); };
  auto bar_sfull = [&](int b) { return sb + C::OFF_BAR + 8u * (1 + 2 * kStages + b); };
  auto bar_pfull = [&](int b) { return sb + C::OFF_BAR + 8u * (3 + 2 * kStages + b); };
  const uint32_t bar_final = sb + C::OFF_BAR + 8u * (5 + 2 * kStages);
  // Score rules: one commit a step. The products that last read the stage of
  // step m - kStages precede the S and dP products of step m - kStages + 2, so
  // the stage is free when those are full. The wait starts with step 0's, two
  // loads earlier than the ring needs it, so that every phase of the barrier
  // is seen; none can be missed, because with at most four stages its next
  // phase needs the load that waits here.
  static_assert(!MOD || kStages <= 4, "the producer would miss a phase");
  const uint32_t bar_op = bar_final + 8, bar_ld = bar_final + 16;  // score rules only
  auto released = [](int m) { return m - kStages + 2; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* never = reinterpret_cast<volatile int*>(misc + 3);
  uint32_t* colc = reinterpret_cast<uint32_t*>(smem + C::OFF_COL);
  int* scan = reinterpret_cast<int*>(smem + C::OFF_SCAN);
  uint32_t* bmA = reinterpret_cast<uint32_t*>(smem + C::OFF_DYN);
  uint32_t* bmB = bmA + P.bm_words;
  uint32_t* ulist = bmB + P.bm_words;
  uint32_t* uext = ulist + P.umax;

  const Geom& g = P.g;
  int i0, i1, c0 = 0, c1 = 0;
  int item = blockIdx.x, share = 0;
  if constexpr (MOD) {  // causal order: the longest lists first, as in the forward
    if (P.mod.causal) item = gridDim.x - 1 - blockIdx.x;
    share = item % P.shares;
    item /= P.shares;
  }
  block_halves(g, P.pair_axis, P.pdim, item, &i0, &i1, &c0, &c1);
  const int head = blockIdx.y, b = blockIdx.z;
  const size_t bh = (size_t)b * g.Hh + head;
  const bool has1 = i1 >= 0;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be uniform
  // First tiled-layout row of chunk c of tile j.
  auto tile_row = [&](int j, int c) -> int { return (int)((bh * g.N + j) * g.V) + 64 * c; };

  // ------------------------------------------------------------ setup
  if (tid == 0) {
    tc::mbar_init(bar_q, 1);
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(bar_full(s), 1);
      tc::mbar_init(bar_empty(s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(bar_sfull(x), 1);
      tc::mbar_init(bar_pfull(x), kSoftmaxThreads);
    }
    tc::mbar_init(bar_final, 1);
    if (MOD) {
      tc::mbar_init(bar_op, kSoftmaxThreads);
      tc::mbar_init(bar_ld, kSoftmaxThreads);
    }
    misc[1] = 0;
    misc[3] = 0;
    tc::mbar_fence_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(sb + C::OFF_MISC, kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid < 64) colc[tid] = chunk_row_code(g, tid);  // in-chunk (t, h, w) offsets of each chunk row
  ModTab* tab = reinterpret_cast<ModTab*>(smem + C::OFF_TAB);  // score rules only
  int prefix = 0;
  if constexpr (MOD) {
    if (P.mod.prefix) prefix = __ldg(P.mod.prefix + b);
  }
  for (int w = tid; w < 2 * P.bm_words; w += kThreads) bmA[w] = 0u;
  if (!has1) {  // rows 64..127 have no tile: zero their Q and dO
    for (int x = tid; x < C::QBLK * 64 * 128 / 16; x += kThreads) {
      const int cb = x / (64 * 128 / 16), off = x % (64 * 128 / 16);
      reinterpret_cast<uint4*>(smem + C::OFF_Q + cb * 128 * 128 + 64 * 128)[off] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(smem + C::OFF_DO + cb * 128 * 128 + 64 * 128)[off] = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  auto load_block = [&]() {
    tc::tma_prefetch_desc(&tmQ);
    tc::tma_prefetch_desc(&tmDO);
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
    tc::mbar_arrive_expect_tx(bar_q, (has1 ? 2 : 1) * 2 * 64 * C::QRB);
    for (int x = 0; x < (has1 ? 2 : 1); ++x) {
      const int row = x ? tile_row(i1, c1) : tile_row(i0, c0);
#pragma unroll
      for (int cb = 0; cb < C::QBLK; ++cb) {
        const uint32_t d = cb * 128 * 128 + x * 64 * 128;
        tc::tma_load_2d(sb + C::OFF_Q + d, &tmQ, bar_q, cb * 64, row);
        tc::tma_load_2d(sb + C::OFF_DO + d, &tmDO, bar_q, cb * 64, row);
      }
    }
  };
  __syncthreads();
  if (MOD) {  // while the list is made
    if (warp == 8 && lane == 0) load_block();
    __syncwarp();
  }

  // Union of the two kept lists, ascending, one step per real 64-key chunk:
  // key tile in bits 0-20, chunk in bits 21-29, bit 30 (31) when the first
  // (second) query half keeps the tile; uext holds the key chunk's real
  // extent from its first token (t, h, w bytes) and bit 31 when it has
  // padded keys.
  int nA = P.cnt[bh * g.N + i0];
  int nB = has1 ? P.cnt[bh * g.N + i1] : 0;
  if (nA < 0 || nA > P.kmax || nB < 0 || nB > P.kmax) {
    if (tid == 0) atomicOr(P.err, BSATTN_DEVERR_BAD_INDEX);
    nA = min(max(nA, 0), P.kmax);
    nB = min(max(nB, 0), P.kmax);
  }
  {
    const int32_t* lA = P.idx + (bh * g.N + i0) * (size_t)P.kmax;
    const int32_t* lB = has1 ? P.idx + (bh * g.N + i1) * (size_t)P.kmax : lA;
    for (int e = tid; e < nA + nB; e += kThreads) {
      const int j = e < nA ? __ldg(lA + e) : __ldg(lB + (e - nA));
      if (j < 0 || j >= g.N) {
        atomicOr(P.err, BSATTN_DEVERR_BAD_INDEX);
        continue;
      }
      atomicOr(e < nA ? &bmA[j >> 5] : &bmB[j >> 5], 1u << (j & 31));
    }
  }
  __syncthreads();
  if constexpr (!MOD) {
    compact_steps<kThreads>(g, bmA, bmB, P.bm_words, ulist, uext, P.umax, scan, misc + 2);
  } else {
    list_steps<kThreads>(g, bmA, bmB, P.bm_words, ulist, P.umax, scan, misc + 2);
    fill_modtab<kThreads>(g, tab, colc);
    __syncthreads();
    const int steps = (int)misc[2];
    int left = mod::filter_steps<kThreads, false>(g, P.mod, b, prefix, i0, i1, c0, c1, ulist, uext, steps, scan,
                                                       tab->origin);
    __syncthreads();
    if (P.shares > 1) left = take_share<kThreads>(ulist, uext, left, share, P.shares);
    if (tid == 0) misc[2] = (uint32_t)left;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
  const int L = __shfl_sync(0xffffffffu, (int)misc[2], 0);

  // ------------------------------------------------------------ roles
  if (warp == 8) {
    if (lane == 0 && L > 0) {
      if (!MOD) load_block();
      int last[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) last[s] = -1;
      for (int m = 0; m < L; ++m) {
        const int s = m % kStages;
        if (m >= (MOD ? kStages - 2 : kStages) && !(MOD ? tc::mbar_wait(bar_sfull(released(m) & 1), (released(m) >> 1) & 1, abort_flag, kWaitLimit)
                                  : tc::mbar_wait(bar_empty(s), ((m / kStages) - 1) & 1, abort_flag, kWaitLimit))) {
          *abort_flag = 1;
          atomicOr(P.err, BSATTN_DEVERR_TIMEOUT);
          break;
        }
        const int krow = tile_row((int)(ulist[m] & 0x1FFFFFu), (int)((ulist[m] >> 21) & 0x1FFu));
        tc::mbar_arrive_expect_tx(bar_full(s), 2 * C::T_BYTES);
#pragma unroll
        for (int cb = 0; cb < C::QBLK; ++cb) {
          tc::tma_load_2d(sb + C::OFF_K + s * C::T_BYTES + cb * 64 * 128, &tmK, bar_full(s), cb * 64, krow);
          tc::tma_load_2d(sb + C::OFF_V + s * C::T_BYTES + cb * 64 * 128, &tmV, bar_full(s), cb * 64, krow);
        }
        last[s] = m;
      }
      if (*abort_flag) {
        tc::mbar_wait(bar_q, 0, never, kWaitLimit);
        for (int s = 0; s < kStages; ++s)
          if (last[s] >= 0) tc::mbar_wait(bar_full(s), (last[s] / kStages) & 1, never, kWaitLimit);
      }
    }
    if (MOD && lane == 0 && L == 0) tc::mbar_wait(bar_q, 0, never, kWaitLimit);  // the block's load lands first
  } else if (warp == 9) {
    if (L > 0) {
      const uint32_t lead = tc::elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, kWaitLimit));
      };
      constexpr uint32_t idS = tc::instr_desc(1, 1, 0, 0, 64, 128);   // bf16, K-major A and B, N = 64
      constexpr uint32_t idQ = tc::instr_desc(1, 1, 0, 1, D, 128);    // B (K tile) MN-major, N = D
      bool ok = wait(bar_q, 0);
      // S_m = Q K_m^T and dP_m = dO V_m^T into buffer m & 1.
      auto issue_sdp = [&](int m) -> bool {
        const int s = m % kStages;
        if (!wait(bar_full(s), (m / kStages) & 1)) return false;
        tc::fence_after_sync();
        const uint32_t dS = tmem + kColS + (m & 1) * 64, dP = tmem + kColDP + (m & 1) * 64;
#pragma unroll
        for (int kk = 0; kk < C::NKS; ++kk) {
          const int cb = kk / 4, within = kk % 4;
          const uint32_t aoff = cb * 128 * 128 + within * 32, boff = s * C::T_BYTES + cb * 64 * 128 + within * 32;
          tc::mma_ss_f16_warp(lead, dS, tc::smem_desc(sb + C::OFF_Q + aoff, 16, 1024, tc::kLayoutSW128),
                         tc::smem_desc(sb + C::OFF_K + boff, 16, 1024, tc::kLayoutSW128), idS, kk > 0 ? 1u : 0u);
          tc::mma_ss_f16_warp(lead, dP, tc::smem_desc(sb + C::OFF_DO + aoff, 16, 1024, tc::kLayoutSW128),
                         tc::smem_desc(sb + C::OFF_V + boff, 16, 1024, tc::kLayoutSW128), idS, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit_warp(lead, bar_sfull(m & 1));
        return true;
      };
      // Score rules: S_m = Q K_m^T with Q from TMEM, and dP_m, whose one
      // buffer is free once the softmax side has read dP_{m-1}.
      auto issue_mod = [&](int m) -> bool {
        const int s = m % kStages;
        if (!wait(bar_full(s), (m / kStages) & 1)) return false;
        tc::fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < C::NKS; ++kk)
          tc::mma_ts_f16_warp(lead, tmem + kColS + (m & 1) * 64, tmem + kColOp + kk * 8,
                         tc::smem_desc(sb + C::OFF_K + s * C::T_BYTES + (kk / 4) * 64 * 128 + (kk % 4) * 32, 16, 1024,
                                       tc::kLayoutSW128),
                         idS, kk > 0 ? 1u : 0u);
        if (m > 0 && !wait(bar_ld, (m - 1) & 1)) return false;
        tc::fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < C::NKS; ++kk) {
          const int cb = kk / 4, within = kk % 4;
          tc::mma_ss_f16_warp(lead, tmem + kColDP, tc::smem_desc(sb + C::OFF_DO + cb * 128 * 128 + within * 32, 16, 1024, tc::kLayoutSW128),
                         tc::smem_desc(sb + C::OFF_V + s * C::T_BYTES + cb * 64 * 128 + within * 32, 16, 1024, tc::kLayoutSW128),
                         idS, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit_warp(lead, bar_sfull(m & 1));
        return true;
      };
      if (MOD) {
        ok = ok && wait(bar_op, 0);
        tc::fence_after_sync();
      }
      if (ok) ok = MOD ? issue_mod(0) : issue_sdp(0);
      if (!MOD && ok && L > 1) ok = issue_sdp(1);
      for (int n = 0; ok && n < L; ++n) {
        const int s = n % kStages;
        if (MOD && n + 1 < L && !issue_mod(n + 1)) {
          ok = false;
          break;
        }
        if (!wait(bar_pfull(n & 1), (n >> 1) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        // dS_n (bf16): keys 0-31 in S_n's columns 0-15, keys 32-63 in 32-47.
        const uint32_t dsA = tmem + kColS + (n & 1) * 64;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // 16 keys per MMA: 2048 bytes of the K tile
          const uint64_t dk = tc::smem_desc(sb + C::OFF_K + s * C::T_BYTES + kk * 2048, 8192, 1024, tc::kLayoutSW128);
          const uint32_t acol = kk < 2 ? kk * 8 : 32 + (kk - 2) * 8, acc = (n > 0 || kk > 0) ? 1u : 0u;
          tc::mma_ts_f16_warp(lead, tmem + kColDQ, dsA + acol, dk, idQ, acc);
          if (MOD) tc::mma_ts_f16_warp(lead, tmem + kColG, dsA + 16 + acol, dk, idQ, acc);
        }
        if (!MOD) tc::mma_commit_warp(lead, bar_empty(s));
        if (!MOD && n + 2 < L && !issue_sdp(n + 2)) {
          ok = false;
          break;
        }
      }
      if (!ok && lead) {
        *abort_flag = 1;
        atomicOr(P.err, BSATTN_DEVERR_TIMEOUT);
      }
      tc::mma_commit_warp(lead, bar_final);
      tc::mbar_wait(bar_final, 0, never, kWaitLimit);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- dS
    const int quad = warp & 3, part = warp >> 2;  // lane quadrant, key half
    const int r = quad * 32 + lane;
    const int half = r >> 6;
    const bool row_exists = half == 0 || has1;
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const size_t lrow = row_exists ? (size_t)(half ? tile_row(i1, c1) : tile_row(i0, c0)) + (r & 63) : 0;
    const float lse2 = row_exists ? P.lse[lrow] * 1.4426950408889634f : 0.f;
    const float dlt = row_exists ? P.delta[lrow] : 0.f;
    const float c = P.scale_log2;
    bool ok = true;
    if constexpr (MOD) {
      if (L > 0) ok = operand_to_tmem<D>(smem + C::OFF_Q, tmem + lane_base + kColOp, part, r, bar_q, bar_op, abort_flag);
    }
    mod::Row row{};
    float kc = 0.f;  // takes raw scores to the argument of tanh
    float slope = 0.f;
    float2 sw2 = mod::bc(0.f), swd2 = sw2, spd2 = sw2;  // sums of w = P (dP - Delta), w dist, P dist
    float nlse2 = -lse2, ndlt = -dlt;
    if constexpr (MOD) {
      if (row_exists) row = mod::row_of(g, P.mod, b, half ? i1 : i0, half ? c1 : c0, colc[r & 63], r & 63);
      if (!row.live || nlse2 == INFINITY) {  // no key seen: P = 0
        nlse2 = -INFINITY;
        ndlt = 0.f;
      }
      if (P.mod.slopes) slope = __ldg(P.mod.slopes + head);
      if (P.mod.cap > 0.f) kc = P.scale / P.mod.cap;
    }
    for (int n = 0; n < L; ++n) {
      const uint32_t e = ulist[n], ext = uext[n];
      const bool keep = row_exists && ((e >> (30 + half)) & 1u) != 0;  // uniform within the warp
      if (!__all_sync(0xffffffffu, tc::mbar_wait(bar_sfull(n & 1), (n >> 1) & 1, abort_flag, kWaitLimit))) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const uint32_t sbuf = tmem + lane_base + kColS + (n & 1) * 64 + 32 * part;
      const uint32_t pbuf = tmem + lane_base + kColDP + (MOD ? 0 : (n & 1) * 64) + 32 * part;
      uint32_t dsw[16];
      uint32_t gw[MOD ? 16 : 1];  // P (1 - tanh^2)
      if constexpr (MOD) {
        if ((ext & mod::kHidden) && tid < 64) {  // K rows of hidden tokens (S has been formed)
          const size_t first = ((size_t)b * g.N + (e & 0x1FFFFFu)) * g.V + 64 * ((e >> 21) & 0x1FFu);
          if (__ldg(P.mod.doc_rows + first + tid) < 0)
            mod::zero_row(smem + C::OFF_K + (n % kStages) * C::T_BYTES, C::QBLK, tid);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      }
      if (MOD && keep) {
        if constexpr (MOD) {
          const ModParams& M = P.mod;
          // (Rows without a token need no mask: P is 0 through neg_lse2 there.)
          mod::Coord f{};
          uint32_t vis = 0xffffffffu;
          bool partial = false;
          if (M.slopes || (ext & mod::kSpecial)) f = mod::chunk_first(g, M, ext, tab->at((int)((e >> 21) & 0x1FFu)));
          if (ext & mod::kSpecial) {
            int vt = g.T - f.t;
            if (M.causal) vt = min(vt, max(row.at.t + 1, prefix) - f.t);
            unsigned long long all = mod::visible_box(g, &tab->col, 0, vt, g.H - f.h, g.W - f.w);
            if (ext & mod::kDoc)
              all &= mod::visible_doc(M, ((size_t)b * g.N + (e & 0x1FFFFFu)) * g.nchunk + ((e >> 21) & 0x1FFu), row.id);
            vis = (uint32_t)(all >> (32 * part));
            partial = __any_sync(0xffffffffu, vis != 0xffffffffu);
          }
          uint32_t sr[32], pr[32];
          tc::tmem_ld32x2_wait(sbuf, sr, pbuf, pr);
          tc::fence_before_sync();
          tc::mbar_arrive(bar_ld);
          // log2 of P = raw scores (or tanh values) times c2, bias, minus the log-sum-exp.
          float c2 = c;
          if (M.cap > 0.f) {
            c2 = M.cap * mod::kLog2e;
            if (partial) mod::set_unseen<32>(sr, vis, 0.f);
            mod::tanh_scores<32>(sr, kc);
          }
          float far[32];
          if (M.slopes) {
            mod::add_distance<32, true>(g, far, &tab->col, 32 * part, mod::make_dist(g, M, row.at, f, 1.f));
          }
          const float2 cc2 = mod::bc(c2), ss2 = mod::bc(-slope * mod::kLog2e), nl2 = mod::bc(nlse2), nd2 = mod::bc(ndlt);
          auto form = [&](auto masked, auto cap, auto bias) {
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              float2 th = mod::pair(sr + 2 * q), dp = mod::pair(pr + 2 * q);
              const bool v0 = (vis >> (2 * q)) & 1u, v1 = (vis >> (2 * q + 1)) & 1u;
              if (masked) {  // whatever hidden rows left in S and dP
                th = make_float2(v0 ? th.x : 0.f, v1 ? th.y : 0.f);
                dp = make_float2(v0 ? dp.x : 0.f, v1 ? dp.y : 0.f);
              }
              float2 y = __ffma2_rn(th, cc2, nl2);
              const float2 d = bias ? make_float2(far[2 * q], far[2 * q + 1]) : mod::bc(0.f);
              if (bias) y = __ffma2_rn(d, ss2, y);
              float2 p = make_float2(tc::ex2(y.x), tc::ex2(y.y));
              if (masked) p = make_float2(v0 ? p.x : 0.f, v1 ? p.y : 0.f);
              float2 w = __fmul2_rn(p, __fadd2_rn(dp, nd2));
              sw2 = __fadd2_rn(sw2, w);
              if (bias) {
                swd2 = __ffma2_rn(w, d, swd2);
                spd2 = __ffma2_rn(p, d, spd2);
              }
              if (cap) {
                const float2 gain = __ffma2_rn(make_float2(-th.x, -th.y), th, mod::bc(1.f));
                w = __fmul2_rn(w, gain);
                p = __fmul2_rn(p, gain);
              }
              dsw[q] = mod::pack(w);
              gw[q] = mod::pack(p);
            }
          };
          mod::dispatch(partial, M.cap > 0.f, M.slopes != nullptr, form);
        }
      } else if (!MOD && keep) {
        const bool edge = (ext >> 31) != 0;
        const int vt = (int)(ext & 0xffu), vh = (int)((ext >> 8) & 0xffu), vw = (int)((ext >> 16) & 0xffu);
        uint32_t sr[32], pr[32];
        tc::tmem_ld32_wait(sbuf, sr);
        tc::tmem_ld32_wait(pbuf, pr);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float d2[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            bool real = true;
            if (edge) {
              const uint32_t cc = colc[32 * part + 2 * q + u];
              real = (int)(cc & 0xffu) < vt && (int)((cc >> 8) & 0xffu) < vh && (int)((cc >> 16) & 0xffu) < vw;
            }
            const float p = real ? tc::ex2(__uint_as_float(sr[2 * q + u]) * c - lse2) : 0.f;
            d2[u] = p * (__uint_as_float(pr[2 * q + u]) - dlt);
          }
          __nv_bfloat162 hv = __floats2bfloat162_rn(d2[0], d2[1]);
          dsw[q] = *reinterpret_cast<uint32_t*>(&hv);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) dsw[q] = 0u;
        if constexpr (MOD) {
#pragma unroll
          for (int q = 0; q < 16; ++q) gw[q] = 0u;
          tc::mbar_arrive(bar_ld);
        }
      }
      if constexpr (MOD) tc::tmem_st16(sbuf + 16, gw);  // P (1 - tanh^2) over the second 16
      tc::tmem_st16(sbuf, dsw);  // dS of this half over the first 16 columns of its S
      tc::tmem_wait_st();
      tc::fence_before_sync();
      tc::mbar_arrive(bar_pfull(n & 1));
    }
    if (!ok) {
      *abort_flag = 1;
      atomicOr(P.err, BSATTN_DEVERR_TIMEOUT);
    }
    // ---------------------------------------------------------- epilogue
    if (ok && L > 0) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(bar_final, 0, abort_flag, kWaitLimit))) {
        *abort_flag = 1;
        atomicOr(P.err, BSATTN_DEVERR_TIMEOUT);
        ok = false;
      }
      tc::fence_after_sync();
    }
    float eps = 0.f;
    if constexpr (MOD) {
      // The two halves' sums. With w = P (dP - Delta) for any Delta and sum P
      // = 1: eps = sum w, and the row's share of -sum dZ dist is eps (sum P
      // dist) - sum w dist.
      const float sw = sw2.x + sw2.y, swd = swd2.x + swd2.y, spd = spd2.x + spd2.y;
      float* red = reinterpret_cast<float*>(smem + C::OFF_V);  // the V ring is no longer read
      const bool use = ok && L > 0;
      if (use) {
        red[3 * tid] = sw;
        red[3 * tid + 1] = swd;
        red[3 * tid + 2] = spd;
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
      float v = 0.f;
      const int o = 3 * (tid ^ 128);
      if (use && row.live) eps = sw + red[o];
      if (P.shares > 1) {
        // The block's sums are complete only where its shares are joined.
        const size_t at = ((bh * (gridDim.x / P.shares) + item) * P.shares + share) * 128 + r;
        if (part == 0) {
          P.part_s[at] = use && row.live ? make_float4(eps, swd + red[o + 1], spd + red[o + 2], ndlt)
                                         : make_float4(0.f, 0.f, 0.f, ndlt);
          if (share == 0 && row_exists) P.neg_lse2[lrow] = nlse2;
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          float* dst = P.part_q + (((at - r) * 2 + which * 128) + r) * D;
          store_share<D>(dst, tmem + lane_base + (which ? kColG : kColDQ), part, ok && L > 0, row.live);
        }
      } else if (part == 0 && row_exists) {
        P.neg_delta[lrow] = ndlt - eps;
        P.neg_lse2[lrow] = nlse2;
        if (use && row.live) v = eps * (spd + red[o + 2]) - (swd + red[o + 1]);
      }
      if (P.slope_parts && P.shares == 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (part == 0 && lane == 0) scan[warp] = __float_as_int(v);
        asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
        if (tid == 0)
          P.slope_parts[bh * gridDim.x + item] = (__int_as_float(scan[0]) + __int_as_float(scan[1])) +
                                                       (__int_as_float(scan[2]) + __int_as_float(scan[3]));
      }
    }
    bool whole = true;
    if constexpr (MOD) whole = P.shares == 1;
    if (whole) {
      uint8_t* stage = smem + C::OFF_K + r * C::O_PITCH;
      constexpr int OC = D / 2;  // dQ columns this warp writes
#pragma unroll
      for (int col = part * OC; col < part * OC + OC; col += 32) {
        uint32_t o[32];
        if (ok && L > 0) {
          tc::tmem_ld32_wait(tmem + lane_base + kColDQ + col, o);
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] = 0u;
        }
        if constexpr (MOD) {
          if (ok && L > 0) {
            uint32_t gr[32];
            tc::tmem_ld32_wait(tmem + lane_base + kColG + col, gr);
#pragma unroll
            for (int q = 0; q < 32; ++q)
              o[q] = __float_as_uint(fmaf(-eps, __uint_as_float(gr[q]), __uint_as_float(o[q])));
          }
          if (!row.live) {
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = 0u;
          }
        }
        uint32_t w[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          __nv_bfloat162 hv = __floats2bfloat162_rn(__uint_as_float(o[2 * q]) * P.scale,
                                                    __uint_as_float(o[2 * q + 1]) * P.scale);
          w[q] = *reinterpret_cast<uint32_t*>(&hv);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<uint4*>(stage + col * 2)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
      constexpr int CPR = D / 8;
      const int rows = has1 ? 128 : 64;
      for (int e2 = tid; e2 < rows * CPR; e2 += kSoftmaxThreads) {
        const int rr = e2 / CPR, cc = e2 % CPR;
        const uint4 val = *reinterpret_cast<const uint4*>(smem + C::OFF_K + rr * C::O_PITCH + cc * 16);
        uint4* og = reinterpret_cast<uint4*>(P.dq + (size_t)(rr >> 6 ? tile_row(i1, c1) : tile_row(i0, c0)) * D);
        og[(rr & 63) * CPR + cc] = val;
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the shares of each query block (small grids): eps = sum of the shares'
// eps, dQ = scale (sum dQ - eps sum G), and each CTA's part of the slope
// gradient. D / 8 threads a row, eight features each, kJoinRows rows a CTA,
// every load of a thread in flight at once; sums in the order of the shares.
constexpr int kMaxShares = 8, kJoinRows = 16, kJoinBlocks = 128 / kJoinRows;
__device__ __forceinline__ void add8(float* s, const float* src) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  s[0] += a.x; s[1] += a.y; s[2] += a.z; s[3] += a.w;
  s[4] += b.x; s[5] += b.y; s[6] += b.z; s[7] += b.w;
}
__device__ __forceinline__ uint4 pack8(const float* s, float mul) {
  return make_uint4(mod::pack(make_float2(s[0] * mul, s[1] * mul)), mod::pack(make_float2(s[2] * mul, s[3] * mul)),
                    mod::pack(make_float2(s[4] * mul, s[5] * mul)), mod::pack(make_float2(s[6] * mul, s[7] * mul)));
}
template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 8) bwd_dq_join_kernel(const __grid_constant__ DqParamsMod P) {
  __shared__ float sums[kJoinRows];
  const Geom& g = P.g;
  const int item = blockIdx.x / kJoinBlocks, items = gridDim.x / kJoinBlocks, piece = threadIdx.x % (D / 8);
  const int r = blockIdx.x % kJoinBlocks * kJoinRows + threadIdx.x / (D / 8), half = r >> 6;
  const size_t bh = (size_t)blockIdx.z * g.Hh + blockIdx.y;
  int i0, i1, c0 = 0, c1 = 0;
  block_halves(g, P.pair_axis, P.pdim, item, &i0, &i1, &c0, &c1);
  float v = 0.f;
  if (half == 0 || i1 >= 0) {
    const size_t at = (bh * items + item) * P.shares;
    float4 s[kMaxShares];
    float dq[8] = {}, gr[8] = {};
#pragma unroll
    for (int p = 0; p < kMaxShares; ++p) {
      if (p >= P.shares) continue;
      s[p] = P.part_s[(at + p) * 128 + r];
      const float* src = P.part_q + ((at + p) * 256 + r) * D + 8 * piece;
      add8(dq, src);
      add8(gr, src + 128 * D);
    }
    float eps = 0.f, wd = 0.f, pd = 0.f;
#pragma unroll
    for (int p = 0; p < kMaxShares; ++p) {
      if (p >= P.shares) continue;
      eps += s[p].x;
      wd += s[p].y;
      pd += s[p].z;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) dq[q] = fmaf(-eps, gr[q], dq[q]);
    const size_t row = (bh * g.N + (half ? i1 : i0)) * g.V + 64 * (half ? c1 : c0) + (r & 63);
    reinterpret_cast<uint4*>(P.dq + row * D)[piece] = pack8(dq, P.scale);
    if (piece == 0) P.neg_delta[row] = s[0].w - eps;
    v = eps * pd - wd;
  }
  if (!P.slope_parts) return;
  if (piece == 0) sums[threadIdx.x / (D / 8)] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    float t = 0.f;
    for (int i = 0; i < kJoinRows; ++i) t += sums[i];
    P.slope_parts[bh * gridDim.x + blockIdx.x] = t;
  }
}

template <int D, bool MOD, int kStages>
bsattn_status run_dq(const bsattn_plan* p, const void* q, const void* k, const void* v, const void* d_o,
                     const std::conditional_t<MOD, DqParamsMod, DqParams>& prm, cudaStream_t st) {
  using C = DqCfg<D, MOD, kStages>;
  const uint64_t rows = (uint64_t)p->desc.B * p->desc.heads * p->N * p->V;
  if (rows + 128 >= (1ull << 31)) return BSATTN_ERR_UNSUPPORTED;
  CUtensorMap mq, mdo, mk, mv;
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!bsattn_make_map_2d(&mq, q, bf, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !bsattn_make_map_2d(&mdo, d_o, bf, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !bsattn_make_map_2d(&mk, k, bf, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !bsattn_make_map_2d(&mv, v, bf, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return BSATTN_ERR_CUDA;
  const size_t smem = 1024 + C::OFF_DYN + (size_t)prm.bm_words * 8 + (size_t)prm.umax * 8;
  if (smem > 227 * 1024) return BSATTN_ERR_UNSUPPORTED;
  auto kern = bwd_dq_tc_kernel<D, MOD, kStages>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return BSATTN_ERR_CUDA;
  const int items = attention_items(p);
  dim3 grid(items, p->desc.heads, p->desc.B);
  if constexpr (MOD) grid.x *= prm.shares;
  kern<<<grid, kThreads, smem, st>>>(mq, mdo, mk, mv, prm);
  if constexpr (MOD) {
    if (prm.shares > 1)
      bwd_dq_join_kernel<D><<<dim3(items * kJoinBlocks, p->desc.heads, p->desc.B), kJoinRows * D / 8, 0, st>>>(prm);
  }
  return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

// ---------------------------------------------------------------- dK, dV
// Two adjacent key tiles j0, j1 stacked into one 128-row block walk the union
// of their transposed lists (the query tiles that keep them), on the same
// pattern with rows and columns exchanged:
//   S^T = K Q_i^T and dP^T = V dO_i^T (SS, N = 64) into TMEM double buffers;
//   P^T = 2^(S^T scale log2(e) - lse_i log2(e)) per query column,
//   dS^T = P^T (dP^T - Delta_i), both written back as bf16 over the first 16
//   columns of each key half of their buffers by eight warps;
//   dV += P^T dO_i and dK += dS^T Q_i (A from TMEM, dO_i and Q_i as MN-major
//   shared-memory operands), accumulated in TMEM; dK is scaled at the end.
// Per step the TMA warp brings Q_i, dO_i and the 64 lse and Delta values of
// query tile i into a ring of three stages, with score rules of four where the
// lists leave room.
struct KvParams {
  Geom g;
  const int32_t* idxT;  // [B, Hh, N, N] query tiles keeping each key tile, ascending
  const int32_t* cntT;  // [B, Hh, N]
  const float* lse;    // with score rules: -lse log2(e)
  const float* delta;  // with score rules: -Delta
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  float scale;
  float scale_log2;
  int* err;
  int umax;
  int bm_words;
  int pair_axis;
  int pdim[3];
};

struct KvParamsMod : KvParams {
  ModParams mod;
  int shares;          // CTAs that share a key block's steps
  float* part_kv;      // shares > 1: [blocks, shares, 2, 128, D] dK (not yet scaled) and dV
};

template <int D, bool MOD, int kStages>
struct KvCfg {
  static constexpr int QRB = D * 2;
  static constexpr int QBLK = QRB / 128;
  static constexpr int NKS = QRB / 32;
  static constexpr int BLK_BYTES = 128 * QRB;   // K or V block (two key tiles)
  static constexpr int T_BYTES = 64 * QRB;      // Q or dO tile
  static constexpr int STAGE = 2 * T_BYTES + 1024;  // Q, dO, lse (256 B), Delta (256 B), pad
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + BLK_BYTES;
  static constexpr int OFF_RING = OFF_V + BLK_BYTES;
  static constexpr int OFF_BAR = OFF_RING + kStages * STAGE;
  // kv, full[S], empty[S], sfull[2], pfull[2], final; score rules: operand in TMEM, dP read
  static constexpr int NBAR = 1 + 2 * kStages + 5 + (MOD ? 2 : 0);
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int OFF_COL = OFF_MISC + 16;
  static constexpr int OFF_SCAN = OFF_COL + 256;
  static constexpr int OFF_TAB = OFF_SCAN + 64;
  static constexpr int OFF_DYN = OFF_TAB + (MOD ? (int)sizeof(ModTab) : 0);
  static_assert(OFF_TAB % 16 == 0, "float4 reads of the table");
  static constexpr int O_PITCH = D * 2 + 16;
  static_assert(STAGE % 1024 == 0, "stage alignment");
  static_assert(2 * 128 * O_PITCH <= OFF_BAR - OFF_RING, "epilogue staging fits in the ring");
};

template <int D, bool MOD, int kStages>
__global__ void __launch_bounds__(kThreads, 1)
bwd_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmDO,
                   const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ std::conditional_t<MOD, KvParamsMod, KvParams> P) {
  using C = KvCfg<D, MOD, kStages>;
  constexpr uint32_t kColST = 0, kColDPT = 128, kColOp = 192, kColDV = 256, kColDK = 256 + D;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = tc::smem_addr(smem);
  const uint32_t bar_kv = sb + C::OFF_BAR;
  auto bar_full = [&](int s) { return sb + C::OFF_BAR + 8u * (1 + s); };
  auto bar_empty = [&](int s) { return sb + C::OFF_BAR + 8u * (1 + kStages + s); };
  auto bar_sfull = [&](int b) { return sb + C::OFF_BAR + 8u * (1 + 2 * kStages + b); };
  auto bar_pfull = [&](int b) { return sb + C::OFF_BAR + 8u * (3 + 2 * kStages + b); };
  const uint32_t bar_final = sb + C::OFF_BAR + 8u * (5 + 2 * kStages);
  // Score rules: one commit a step. The products that last read the stage of
  // step m - kStages precede the S and dP products of step m - kStages + 2, so
  // the stage is free when those are full. The wait starts with step 0's, two
  // loads earlier than the ring needs it, so that every phase of the barrier
  // is seen; none can be missed, because with at most four stages its next
  // phase needs the load that waits here.
  static_assert(!MOD || kStages <= 4, "the producer would miss a phase");
  const uint32_t bar_op = bar_final + 8, bar_ld = bar_final + 16;  // score rules only
  auto released = [](int m) { return m - kStages + 2; };
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* never = reinterpret_cast<volatile int*>(misc + 3);
  uint32_t* colc = reinterpret_cast<uint32_t*>(smem + C::OFF_COL);
  int* scan = reinterpret_cast<int*>(smem + C::OFF_SCAN);
  uint32_t* bmA = reinterpret_cast<uint32_t*>(smem + C::OFF_DYN);
  uint32_t* bmB = bmA + P.bm_words;
  uint32_t* ulist = bmB + P.bm_words;
  uint32_t* uext = ulist + P.umax;

  const Geom& g = P.g;
  int j0, j1, kc0 = 0, kc1 = 0;
  int item = blockIdx.x, share = 0;
  if constexpr (MOD) {
    share = item % P.shares;
    item /= P.shares;
  }
  block_halves(g, P.pair_axis, P.pdim, item, &j0, &j1, &kc0, &kc1);
  const int head = blockIdx.y, b = blockIdx.z;
  const size_t bh = (size_t)b * g.Hh + head;
  const bool has1 = j1 >= 0;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be uniform
  // First tiled-layout row of chunk c of tile j.
  auto tile_row = [&](int j, int c) -> int { return (int)((bh * g.N + j) * g.V) + 64 * c; };
  // Whether row q of chunk c of tile j is a real token.
  auto row_is_real = [&](int j, int c, int q) -> bool {
    const ChunkOrigin o = chunk_origin(g, c);
    const int bt = j / (g.nH * g.nW), bhh = (j / g.nW) % g.nH, bw = j % g.nW;
    const uint32_t cc = colc[q];
    return bt * g.tt + o.dt + (int)(cc & 0xffu) < g.T && bhh * g.th + o.dh + (int)((cc >> 8) & 0xffu) < g.H &&
           bw * g.tw + o.dw + (int)((cc >> 16) & 0xffu) < g.W;
  };

  // ------------------------------------------------------------ setup
  if (tid == 0) {
    tc::mbar_init(bar_kv, 1);
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(bar_full(s), 1);
      tc::mbar_init(bar_empty(s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(bar_sfull(x), 1);
      tc::mbar_init(bar_pfull(x), kSoftmaxThreads);
    }
    tc::mbar_init(bar_final, 1);
    if (MOD) {
      tc::mbar_init(bar_op, kSoftmaxThreads);
      tc::mbar_init(bar_ld, kSoftmaxThreads);
    }
    misc[1] = 0;
    misc[3] = 0;
    tc::mbar_fence_init();
  }
  if (warp == 9) {
    tc::tmem_alloc(sb + C::OFF_MISC, kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid < 64) colc[tid] = chunk_row_code(g, tid);  // in-chunk (t, h, w) offsets of each chunk row
  ModTab* tab = reinterpret_cast<ModTab*>(smem + C::OFF_TAB);  // score rules only
  int prefix = 0;
  if constexpr (MOD) {
    if (P.mod.prefix) prefix = __ldg(P.mod.prefix + b);
  }
  for (int w = tid; w < 2 * P.bm_words; w += kThreads) bmA[w] = 0u;
  if (!has1) {  // rows 64..127 have no key tile: zero their K and V
    for (int x = tid; x < C::QBLK * 64 * 128 / 16; x += kThreads) {
      const int cb = x / (64 * 128 / 16), off = x % (64 * 128 / 16);
      reinterpret_cast<uint4*>(smem + C::OFF_K + cb * 128 * 128 + 64 * 128)[off] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(smem + C::OFF_V + cb * 128 * 128 + 64 * 128)[off] = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  auto load_block = [&]() {
    tc::tma_prefetch_desc(&tmQ);
    tc::tma_prefetch_desc(&tmDO);
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
    tc::mbar_arrive_expect_tx(bar_kv, (has1 ? 2 : 1) * 2 * 64 * C::QRB);
    for (int x = 0; x < (has1 ? 2 : 1); ++x) {
      const int row = x ? tile_row(j1, kc1) : tile_row(j0, kc0);
#pragma unroll
      for (int cb = 0; cb < C::QBLK; ++cb) {
        const uint32_t d = cb * 128 * 128 + x * 64 * 128;
        tc::tma_load_2d(sb + C::OFF_K + d, &tmK, bar_kv, cb * 64, row);
        tc::tma_load_2d(sb + C::OFF_V + d, &tmV, bar_kv, cb * 64, row);
      }
    }
  };
  __syncthreads();
  if (MOD) {  // while the list is made
    if (warp == 8 && lane == 0) load_block();
    __syncwarp();
  }

  // Union of the two transposed lists, ascending, one step per real chunk of
  // each listed query tile: query tile in bits 0-20, chunk in bits 21-29, bit
  // 30 (31) when it keeps j0 (j1); uext holds the query chunk's real extent
  // and bit 31 when it has padded rows.
  {
    const int nA = min(max(P.cntT[bh * g.N + j0], 0), g.N);
    const int nB = has1 ? min(max(P.cntT[bh * g.N + j1], 0), g.N) : 0;
    const int32_t* lA = P.idxT + (bh * g.N + j0) * (size_t)g.N;
    const int32_t* lB = has1 ? P.idxT + (bh * g.N + j1) * (size_t)g.N : lA;
    for (int e = tid; e < nA + nB; e += kThreads) {
      const int i = e < nA ? __ldg(lA + e) : __ldg(lB + (e - nA));
      if (i < 0 || i >= g.N) continue;  // the transposed lists are built in range
      atomicOr(e < nA ? &bmA[i >> 5] : &bmB[i >> 5], 1u << (i & 31));
    }
  }
  __syncthreads();
  if constexpr (!MOD) {
    compact_steps<kThreads>(g, bmA, bmB, P.bm_words, ulist, uext, P.umax, scan, misc + 2);
  } else {
    list_steps<kThreads>(g, bmA, bmB, P.bm_words, ulist, P.umax, scan, misc + 2);
    fill_modtab<kThreads>(g, tab, colc);
    __syncthreads();
    const int steps = (int)misc[2];
    int left = mod::filter_steps<kThreads, true>(g, P.mod, b, prefix, j0, j1, kc0, kc1, ulist, uext, steps, scan,
                                                       tab->origin);
    __syncthreads();
    if (P.shares > 1) left = take_share<kThreads>(ulist, uext, left, share, P.shares);
    if (tid == 0) misc[2] = (uint32_t)left;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
  const int L = __shfl_sync(0xffffffffu, (int)misc[2], 0);

  // ------------------------------------------------------------ roles
  if (warp == 8) {
    if (lane == 0 && L > 0) {
      if (!MOD) load_block();
      int last[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) last[s] = -1;
      for (int m = 0; m < L; ++m) {
        const int s = m % kStages;
        if (m >= (MOD ? kStages - 2 : kStages) && !(MOD ? tc::mbar_wait(bar_sfull(released(m) & 1), (released(m) >> 1) & 1, abort_flag, kWaitLimit)
                                  : tc::mbar_wait(bar_empty(s), ((m / kStages) - 1) & 1, abort_flag, kWaitLimit))) {
          *abort_flag = 1;
          atomicOr(P.err, BSATTN_DEVERR_TIMEOUT);
          break;
        }
        const int qrow = tile_row((int)(ulist[m] & 0x1FFFFFu), (int)((ulist[m] >> 21) & 0x1FFu));
        const uint32_t st = sb + C::OFF_RING + s * C::STAGE;
        tc::mbar_arrive_expect_tx(bar_full(s), 2 * C::T_BYTES + 512);
#pragma unroll
        for (int cb = 0; cb < C::QBLK; ++cb) {
          tc::tma_load_2d(st + cb * 64 * 128, &tmQ, bar_full(s), cb * 64, qrow);
          tc::tma_load_2d(st + C::T_BYTES + cb * 64 * 128, &tmDO, bar_full(s), cb * 64, qrow);
        }
        tc::bulk_load(st + 2 * C::T_BYTES, P.lse + qrow, 256, bar_full(s));
        tc::bulk_load(st + 2 * C::T_BYTES + 256, P.delta + qrow, 256, bar_full(s));
        last[s] = m;
      }
      if (*abort_flag) {
        tc::mbar_wait(bar_kv, 0, never, kWaitLimit);
        for (int s = 0; s < kStages; ++s)
          if (last[s] >= 0) tc::mbar_wait(bar_full(s), (last[s] / kStages) & 1, never, kWaitLimit);
      }
    }
    if (MOD && lane == 0 && L == 0) tc::mbar_wait(bar_kv, 0, never, kWaitLimit);  // the block's load lands first
  } else if (warp == 9) {
    if (L > 0) {
      const uint32_t lead = tc::elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, kWaitLimit));
      };
      constexpr uint32_t idS = tc::instr_desc(1, 1, 0, 0, 64, 128);  // K-major A and B, N = 64
      constexpr uint32_t idG = tc::instr_desc(1, 1, 0, 1, D, 128);   // B MN-major, N = D
      bool ok = wait(bar_kv, 0);
      auto issue_sdp = [&](int m) -> bool {
        const int s = m % kStages;
        if (!wait(bar_full(s), (m / kStages) & 1)) return false;
        tc::fence_after_sync();
        const uint32_t st = sb + C::OFF_RING + s * C::STAGE;
        const uint32_t dS = tmem + kColST + (m & 1) * 64, dP = tmem + kColDPT + (m & 1) * 64;
#pragma unroll
        for (int kk = 0; kk < C::NKS; ++kk) {
          const int cb = kk / 4, within = kk % 4;
          const uint32_t aoff = cb * 128 * 128 + within * 32, boff = cb * 64 * 128 + within * 32;
          tc::mma_ss_f16_warp(lead, dS, tc::smem_desc(sb + C::OFF_K + aoff, 16, 1024, tc::kLayoutSW128),
                         tc::smem_desc(st + boff, 16, 1024, tc::kLayoutSW128), idS, kk > 0 ? 1u : 0u);
          tc::mma_ss_f16_warp(lead, dP, tc::smem_desc(sb + C::OFF_V + aoff, 16, 1024, tc::kLayoutSW128),
                         tc::smem_desc(st + C::T_BYTES + boff, 16, 1024, tc::kLayoutSW128), idS, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit_warp(lead, bar_sfull(m & 1));
        return true;
      };
      // Score rules: S^T_m = K Q_m^T with K from TMEM, and dP^T_m, whose one
      // buffer is free once the softmax side has read dP^T_{m-1}.
      auto issue_mod = [&](int m) -> bool {
        const int s = m % kStages;
        if (!wait(bar_full(s), (m / kStages) & 1)) return false;
        tc::fence_after_sync();
        const uint32_t st = sb + C::OFF_RING + s * C::STAGE;
#pragma unroll
        for (int kk = 0; kk < C::NKS; ++kk)
          tc::mma_ts_f16_warp(lead, tmem + kColST + (m & 1) * 64, tmem + kColOp + kk * 8,
                         tc::smem_desc(st + (kk / 4) * 64 * 128 + (kk % 4) * 32, 16, 1024, tc::kLayoutSW128), idS,
                         kk > 0 ? 1u : 0u);
        if (m > 0 && !wait(bar_ld, (m - 1) & 1)) return false;
        tc::fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < C::NKS; ++kk) {
          const int cb = kk / 4, within = kk % 4;
          tc::mma_ss_f16_warp(lead, tmem + kColDPT, tc::smem_desc(sb + C::OFF_V + cb * 128 * 128 + within * 32, 16, 1024, tc::kLayoutSW128),
                         tc::smem_desc(st + C::T_BYTES + cb * 64 * 128 + within * 32, 16, 1024, tc::kLayoutSW128), idS,
                         kk > 0 ? 1u : 0u);
        }
        tc::mma_commit_warp(lead, bar_sfull(m & 1));
        return true;
      };
      if (MOD) {
        ok = ok && wait(bar_op, 0);
        tc::fence_after_sync();
      }
      if (ok) ok = MOD ? issue_mod(0) : issue_sdp(0);
      if (!MOD && ok && L > 1) ok = issue_sdp(1);
      for (int n = 0; ok && n < L; ++n) {
        const int s = n % kStages;
        if (MOD && n + 1 < L && !issue_mod(n + 1)) {
          ok = false;
          break;
        }
        if (!wait(bar_pfull(n & 1), (n >> 1) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t st = sb + C::OFF_RING + s * C::STAGE;
        // P^T and dS^T (bf16): queries 0-31 in columns 0-15, 32-63 in 32-47.
        const uint32_t pA = tmem + kColST + (n & 1) * 64, dsA = MOD ? pA + 16 : tmem + kColDPT + (n & 1) * 64;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {  // 16 queries per MMA: 2048 bytes of the dO / Q tile
          const uint32_t acol = kk < 2 ? kk * 8 : 32 + (kk - 2) * 8;
          const uint32_t acc = (n > 0 || kk > 0) ? 1u : 0u;
          tc::mma_ts_f16_warp(lead, tmem + kColDV, pA + acol,
                         tc::smem_desc(st + C::T_BYTES + kk * 2048, 8192, 1024, tc::kLayoutSW128), idG, acc);
          tc::mma_ts_f16_warp(lead, tmem + kColDK, dsA + acol, tc::smem_desc(st + kk * 2048, 8192, 1024, tc::kLayoutSW128),
                         idG, acc);
        }
        if (!MOD) tc::mma_commit_warp(lead, bar_empty(s));
        if (!MOD && n + 2 < L && !issue_sdp(n + 2)) {
          ok = false;
          break;
        }
      }
      if (!ok && lead) {
        *abort_flag = 1;
        atomicOr(P.err, BSATTN_DEVERR_TIMEOUT);
      }
      tc::mma_commit_warp(lead, bar_final);
      tc::mbar_wait(bar_final, 0, never, kWaitLimit);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- P^T, dS^T
    const int quad = warp & 3, part = warp >> 2;  // lane quadrant, query half
    const int r = quad * 32 + lane;                // key row of the block
    const int half = r >> 6;                       // 0: tile j0, 1: tile j1
    const bool row_exists = half == 0 || has1;
    const bool key_real = row_exists && (half ? row_is_real(j1, kc1, r & 63) : row_is_real(j0, kc0, r & 63));
    const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
    const float c = P.scale_log2;
    bool ok = true;
    if constexpr (MOD) {
      if (L > 0) ok = operand_to_tmem<D>(smem + C::OFF_K, tmem + lane_base + kColOp, part, r, bar_kv, bar_op, abort_flag);
    }
    mod::Row row{};
    float kc = 0.f;  // takes raw scores to the argument of tanh
    float slope = 0.f;
    if constexpr (MOD) {
      if (row_exists) row = mod::row_of(g, P.mod, b, half ? j1 : j0, half ? kc1 : kc0, colc[r & 63], r & 63);
      if (P.mod.slopes) slope = __ldg(P.mod.slopes + head);
      if (P.mod.cap > 0.f) kc = P.scale / P.mod.cap;
    }
    for (int n = 0; n < L; ++n) {
      const uint32_t e = ulist[n], ext = uext[n];
      const bool keep = row_exists && ((e >> (30 + half)) & 1u) != 0;  // uniform within the warp
      if (!__all_sync(0xffffffffu, tc::mbar_wait(bar_sfull(n & 1), (n >> 1) & 1, abort_flag, kWaitLimit))) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const uint32_t sbuf = tmem + lane_base + kColST + (n & 1) * 64 + 32 * part;
      const uint32_t pbuf = tmem + lane_base + kColDPT + (MOD ? 0 : (n & 1) * 64) + 32 * part;
      // lse and Delta of this step's query tile came with its TMA copies:
      // observe their barrier before reading them.
      if (!__all_sync(0xffffffffu, tc::mbar_wait(bar_full(n % kStages), (n / kStages) & 1, abort_flag, kWaitLimit))) {
        ok = false;
        break;
      }
      uint32_t pw[16], dw[16];
      if constexpr (MOD) {
        if ((ext & mod::kHidden) && tid < 64) {  // Q and dO rows of hidden tokens (S and dP have been formed)
          const size_t first = ((size_t)b * g.N + (e & 0x1FFFFFu)) * g.V + 64 * ((e >> 21) & 0x1FFu);
          if (__ldg(P.mod.doc_rows + first + tid) < 0) {
            uint8_t* tile = smem + C::OFF_RING + (n % kStages) * C::STAGE;
            mod::zero_row(tile, C::QBLK, tid);
            mod::zero_row(tile + C::T_BYTES, C::QBLK, tid);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
      }
      if (MOD && keep) {
        if constexpr (MOD) {
          const ModParams& M = P.mod;
          const float* ld = reinterpret_cast<const float*>(smem + C::OFF_RING + (n % kStages) * C::STAGE + 2 * C::T_BYTES);
          // (Rows without a token need no mask: their gradients are not written.)
          mod::Coord f{};
          uint32_t vis = 0xffffffffu;
          bool partial = false;
          if (M.slopes || (ext & mod::kSpecial)) f = mod::chunk_first(g, M, ext, tab->at((int)((e >> 21) & 0x1FFu)));
          if (ext & mod::kSpecial) {
            // Queries at or behind the key's frame, all of them for a key of the prefix.
            const int lo = M.causal && row.at.t >= prefix ? row.at.t - f.t : 0;
            unsigned long long all = mod::visible_box(g, &tab->col, lo, g.T - f.t, g.H - f.h, g.W - f.w);
            if (ext & mod::kDoc)
              all &= mod::visible_doc(M, ((size_t)b * g.N + (e & 0x1FFFFFu)) * g.nchunk + ((e >> 21) & 0x1FFu), row.id);
            vis = (uint32_t)(all >> (32 * part));
            partial = __any_sync(0xffffffffu, vis != 0xffffffffu);
          }
          uint32_t sr[32], pr[32];
          tc::tmem_ld32x2_wait(sbuf, sr, pbuf, pr);
          tc::fence_before_sync();
          tc::mbar_arrive(bar_ld);
          float c2 = c;
          if (M.cap > 0.f) {
            c2 = M.cap * mod::kLog2e;
            if (partial) mod::set_unseen<32>(sr, vis, 0.f);
            mod::tanh_scores<32>(sr, kc);
          }
          float y[32];  // -lse log2(e) of the queries, plus the bias
#pragma unroll
          for (int q = 0; q < 8; ++q) *reinterpret_cast<float4*>(y + 4 * q) = reinterpret_cast<const float4*>(ld + 32 * part)[q];
          if (M.slopes) {
            mod::add_distance<32>(g, y, &tab->col, 32 * part, mod::make_dist(g, M, row.at, f, -slope * mod::kLog2e));
          }
          const float2 cc2 = mod::bc(c2);
          auto form = [&](auto masked, auto cap, auto) {
#pragma unroll
            for (int q4 = 0; q4 < 8; ++q4) {
              const float4 nd = reinterpret_cast<const float4*>(ld + 64 + 32 * part)[q4];  // -Delta of four queries
#pragma unroll
              for (int q = 2 * q4; q < 2 * q4 + 2; ++q) {
                float2 th = mod::pair(sr + 2 * q), dp = mod::pair(pr + 2 * q);
                const bool v0 = (vis >> (2 * q)) & 1u, v1 = (vis >> (2 * q + 1)) & 1u;
                if (masked) {
                  th = make_float2(v0 ? th.x : 0.f, v1 ? th.y : 0.f);
                  dp = make_float2(v0 ? dp.x : 0.f, v1 ? dp.y : 0.f);
                }
                const float2 e = __ffma2_rn(th, cc2, make_float2(y[2 * q], y[2 * q + 1]));
                float2 p = make_float2(tc::ex2(e.x), tc::ex2(e.y));
                if (masked) p = make_float2(v0 ? p.x : 0.f, v1 ? p.y : 0.f);
                pw[q] = mod::pack(p);
                float2 w = __fmul2_rn(p, __fadd2_rn(dp, q & 1 ? make_float2(nd.z, nd.w) : make_float2(nd.x, nd.y)));
                if (cap) w = __fmul2_rn(w, __ffma2_rn(make_float2(-th.x, -th.y), th, mod::bc(1.f)));
                dw[q] = mod::pack(w);
              }
            }
          };
          mod::dispatch(partial, M.cap > 0.f, false, form);
        }
      } else if (!MOD && keep) {
        const float* ld = reinterpret_cast<const float*>(smem + C::OFF_RING + (n % kStages) * C::STAGE + 2 * C::T_BYTES);
        const bool edge = (ext >> 31) != 0;
        const int vt = (int)(ext & 0xffu), vh = (int)((ext >> 8) & 0xffu), vw = (int)((ext >> 16) & 0xffu);
        uint32_t sr[32], pr[32];
        tc::tmem_ld32_wait(sbuf, sr);
        tc::tmem_ld32_wait(pbuf, pr);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          float pp[2], d2[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int qc = 32 * part + 2 * q + u;  // query column
            bool real = key_real;
            if (edge) {
              const uint32_t cc = colc[qc];
              real = real && (int)(cc & 0xffu) < vt && (int)((cc >> 8) & 0xffu) < vh && (int)((cc >> 16) & 0xffu) < vw;
            }
            const float p = real ? tc::ex2(__uint_as_float(sr[2 * q + u]) * c - ld[qc] * 1.4426950408889634f) : 0.f;
            pp[u] = p;
            d2[u] = p * (__uint_as_float(pr[2 * q + u]) - ld[64 + qc]);
          }
          __nv_bfloat162 hp = __floats2bfloat162_rn(pp[0], pp[1]), hd = __floats2bfloat162_rn(d2[0], d2[1]);
          pw[q] = *reinterpret_cast<uint32_t*>(&hp);
          dw[q] = *reinterpret_cast<uint32_t*>(&hd);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) pw[q] = dw[q] = 0u;
        if (MOD) tc::mbar_arrive(bar_ld);
      }
      tc::tmem_st16(sbuf, pw);  // P^T over the first 16 columns of this half of S^T
      // dS^T over the first 16 columns of this half of dP^T; with rules over the
      // second 16 of S^T, so that dP^T is free as soon as it is read.
      tc::tmem_st16(MOD ? sbuf + 16 : pbuf, dw);
      tc::tmem_wait_st();
      tc::fence_before_sync();
      tc::mbar_arrive(bar_pfull(n & 1));
    }
    if (!ok) {
      *abort_flag = 1;
      atomicOr(P.err, BSATTN_DEVERR_TIMEOUT);
    }
    // ---------------------------------------------------------- epilogue
    if (ok && L > 0) {
      if (!__all_sync(0xffffffffu, tc::mbar_wait(bar_final, 0, abort_flag, kWaitLimit))) {
        *abort_flag = 1;
        atomicOr(P.err, BSATTN_DEVERR_TIMEOUT);
        ok = false;
      }
      tc::fence_after_sync();
    }
    bool whole = true;
    if constexpr (MOD) {
      whole = P.shares == 1;
      if (!whole) {
        float* dst = P.part_kv + (((bh * (gridDim.x / P.shares) + item) * P.shares + share) * 2 * 128 + r) * D;
        store_share<D>(dst, tmem + lane_base + kColDK, part, ok && L > 0, row.live);
        store_share<D>(dst + 128 * D, tmem + lane_base + kColDV, part, ok && L > 0, row.live);
      }
    }
    if (whole) {
      // dK (scaled) and dV rows staged in the ring: dK at rows 0-127, dV at 128-255.
      constexpr int OC = D / 2;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        uint8_t* stage = smem + C::OFF_RING + (which * 128 + r) * C::O_PITCH;
        const float mul = which == 0 ? P.scale : 1.f;
        const uint32_t base = which == 0 ? kColDK : kColDV;
#pragma unroll
        for (int col = part * OC; col < part * OC + OC; col += 32) {
          uint32_t o[32];
          if (ok && L > 0) {
            tc::tmem_ld32_wait(tmem + lane_base + base + col, o);
          } else {
#pragma unroll
            for (int q = 0; q < 32; ++q) o[q] = 0u;
          }
          if constexpr (MOD) {
            if (!row.live) {
#pragma unroll
              for (int q = 0; q < 32; ++q) o[q] = 0u;
            }
          }
          uint32_t w[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            __nv_bfloat162 hv = __floats2bfloat162_rn(__uint_as_float(o[2 * q]) * mul, __uint_as_float(o[2 * q + 1]) * mul);
            w[q] = *reinterpret_cast<uint32_t*>(&hv);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            reinterpret_cast<uint4*>(stage + col * 2)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
      constexpr int CPR = D / 8;
      const int rows = has1 ? 128 : 64;
      for (int e2 = tid; e2 < 2 * rows * CPR; e2 += kSoftmaxThreads) {
        const int which = e2 / (rows * CPR), rem = e2 % (rows * CPR);
        const int rr = rem / CPR, cc = rem % CPR;
        const uint4 val = *reinterpret_cast<const uint4*>(smem + C::OFF_RING + (which * 128 + rr) * C::O_PITCH + cc * 16);
        __nv_bfloat16* dst = which == 0 ? P.dk : P.dv;
        uint4* og = reinterpret_cast<uint4*>(dst + (size_t)(rr >> 6 ? tile_row(j1, kc1) : tile_row(j0, kc0)) * D);
        og[(rr & 63) * CPR + cc] = val;
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the shares of each key block, as bwd_dq_join_kernel.
template <int D>
__global__ void __launch_bounds__(kJoinRows * D / 8) bwd_dkdv_join_kernel(const __grid_constant__ KvParamsMod P) {
  const Geom& g = P.g;
  const int item = blockIdx.x / kJoinBlocks, items = gridDim.x / kJoinBlocks, piece = threadIdx.x % (D / 8);
  const int r = blockIdx.x % kJoinBlocks * kJoinRows + threadIdx.x / (D / 8), half = r >> 6;
  const size_t bh = (size_t)blockIdx.z * g.Hh + blockIdx.y;
  int j0, j1, c0 = 0, c1 = 0;
  block_halves(g, P.pair_axis, P.pdim, item, &j0, &j1, &c0, &c1);
  if (half && j1 < 0) return;
  const size_t at = (bh * items + item) * P.shares;
  float dk[8] = {}, dv[8] = {};
#pragma unroll
  for (int p = 0; p < kMaxShares; ++p) {
    if (p >= P.shares) continue;
    const float* src = P.part_kv + ((at + p) * 256 + r) * D + 8 * piece;
    add8(dk, src);
    add8(dv, src + 128 * D);
  }
  const size_t row = (bh * g.N + (half ? j1 : j0)) * g.V + 64 * (half ? c1 : c0) + (r & 63);
  reinterpret_cast<uint4*>(P.dk + row * D)[piece] = pack8(dk, P.scale);
  reinterpret_cast<uint4*>(P.dv + row * D)[piece] = pack8(dv, 1.f);
}

template <int D, bool MOD, int kStages>
bsattn_status run_dkdv(const bsattn_plan* p, const void* q, const void* k, const void* v, const void* d_o,
                       const std::conditional_t<MOD, KvParamsMod, KvParams>& prm, cudaStream_t st) {
  using C = KvCfg<D, MOD, kStages>;
  const uint64_t rows = (uint64_t)p->desc.B * p->desc.heads * p->N * p->V;
  if (rows + 128 >= (1ull << 31)) return BSATTN_ERR_UNSUPPORTED;
  CUtensorMap mq, mdo, mk, mv;
  const auto bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!bsattn_make_map_2d(&mq, q, bf, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !bsattn_make_map_2d(&mdo, d_o, bf, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !bsattn_make_map_2d(&mk, k, bf, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !bsattn_make_map_2d(&mv, v, bf, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return BSATTN_ERR_CUDA;
  const size_t smem = 1024 + C::OFF_DYN + (size_t)prm.bm_words * 8 + (size_t)prm.umax * 8;
  if (smem > 227 * 1024) return BSATTN_ERR_UNSUPPORTED;
  auto kern = bwd_dkdv_tc_kernel<D, MOD, kStages>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return BSATTN_ERR_CUDA;
  const int items = attention_items(p);
  dim3 grid(items, p->desc.heads, p->desc.B);
  if constexpr (MOD) grid.x *= prm.shares;
  kern<<<grid, kThreads, smem, st>>>(mq, mdo, mk, mv, prm);
  if constexpr (MOD) {
    if (prm.shares > 1)
      bwd_dkdv_join_kernel<D><<<dim3(items * kJoinBlocks, p->desc.heads, p->desc.B), kJoinRows * D / 8, 0, st>>>(prm);
  }
  return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace

// Whether the step lists fit: shared memory of a launch is the configuration's
// fixed part, two list bitmaps and two words per step. Under score rules a
// stage is released by the S product two steps on, which leaves three ring
// stages one step for a load's latency and four stages two, so four are taken
// where they fit.
template <class C>
static bool fits(const bsattn_plan* p, int steps) {
  return 1024 + C::OFF_DYN + (size_t)((p->N + 31) / 32) * 8 + (size_t)steps * 8 <= 227 * 1024;
}

// Most steps of a key block: all query tiles times their chunks.
static int key_steps(const bsattn_plan* p) { return p->N * p->nchunk; }
// Under score rules, on grids that leave half of the SMs or more idle, up to
// eight CTAs share a block's steps, one per SM over the grid and four steps
// each at least, and a second kernel joins their sums. A step takes 1.2 us
// there and the join 6 to 8, so the shares must save eight steps. On one B200
// with cap and bias (all launches of a backward): 2,048 tokens of one head 127
// us alone, 70 shared; two heads of 8 x 16 x 16 tokens in a (3,3,3) window 80
// and 55; 18 (6,8,8) tiles of one head 174 and 81.
static int backward_shares(const bsattn_plan* p, int steps) {
  const long long blocks = (long long)attention_items(p) * p->desc.heads * p->desc.B;
  long long n = 148 / blocks;
  if (n > steps / 4) n = steps / 4;
  if (n > kMaxShares) n = kMaxShares;
  return n < 2 || steps - steps / n < 8 ? 1 : (int)n;
}
static size_t share_rows(const bsattn_plan* p, int shares) {
  return shares == 1 ? 0 : (size_t)attention_items(p) * p->desc.heads * p->desc.B * shares * 128;
}
size_t backward_mod_workspace_bytes(const bsattn_plan* p) {
  const size_t d = p->desc.head_dim, nq = share_rows(p, backward_shares(p, attention_steps(p))),
               nk = share_rows(p, backward_shares(p, key_steps(p)));
  const size_t a = nq * (2 * d * sizeof(float) + sizeof(float4)), b = nk * 2 * d * sizeof(float);
  return a > b ? a : b;  // the passes follow one another
}
int backward_slope_items(const bsattn_plan* p) {
  return attention_items(p) * (backward_shares(p, attention_steps(p)) > 1 ? kJoinBlocks : 1);
}

bsattn_status check_backward_mod(const bsattn_plan* p) {
  if (tiled_rows(p) + 128 >= (1ull << 31)) return BSATTN_ERR_UNSUPPORTED;
  if (p->desc.B > 65535 || p->desc.heads > 65535) return BSATTN_ERR_UNSUPPORTED;  // grid
  const int q = attention_steps(p), k = key_steps(p);
  const bool ok = p->desc.head_dim == 128 ? fits<DqCfg<128, true, 3>>(p, q) && fits<KvCfg<128, true, 3>>(p, k)
                                          : fits<DqCfg<64, true, 3>>(p, q) && fits<KvCfg<64, true, 3>>(p, k);
  return ok ? BSATTN_OK : BSATTN_ERR_UNSUPPORTED;
}

bsattn_status launch_backward_dq_tc(const bsattn_plan* p, const void* q, const void* k, const void* v,
                                    const void* d_o, const float* lse, float* delta, const int32_t* idx,
                                    const int32_t* cnt, void* dq, cudaStream_t st, const ModParams* mod,
                                    float* neg_lse2, float* slope_parts, void* shares) {
  DqParamsMod prm;
  prm.g = make_geom(p);
  prm.idx = idx;
  prm.cnt = cnt;
  prm.lse = lse;
  prm.delta = delta;
  prm.kmax = p->kmax;
  prm.dq = (__nv_bfloat16*)dq;
  prm.scale = p->scale;
  prm.scale_log2 = p->scale * 1.4426950408889634f;
  prm.err = p->d_err;
  prm.umax = attention_steps(p);
  prm.bm_words = (p->N + 31) / 32;
  prm.pair_axis = pair_axis_of(p);
  const int nd[3] = {p->nT, p->nH, p->nW};
  for (int a = 0; a < 3; ++a) prm.pdim[a] = a == prm.pair_axis ? (nd[a] + 1) / 2 : nd[a];
  const bool d128 = p->desc.head_dim == 128;
  if (mod) {
    prm.mod = *mod;
    prm.neg_delta = delta;
    prm.neg_lse2 = neg_lse2;
    prm.slope_parts = slope_parts;
    prm.shares = backward_shares(p, prm.umax);
    prm.part_q = (float*)shares;
    prm.part_s = (float4*)(prm.part_q + share_rows(p, prm.shares) * 2 * p->desc.head_dim);
    if (d128)
      return fits<DqCfg<128, true, 4>>(p, prm.umax) ? run_dq<128, true, 4>(p, q, k, v, d_o, prm, st)
                                                    : run_dq<128, true, 3>(p, q, k, v, d_o, prm, st);
    return fits<DqCfg<64, true, 4>>(p, prm.umax) ? run_dq<64, true, 4>(p, q, k, v, d_o, prm, st)
                                                 : run_dq<64, true, 3>(p, q, k, v, d_o, prm, st);
  }
  return d128 ? run_dq<128, false, 3>(p, q, k, v, d_o, prm, st) : run_dq<64, false, 3>(p, q, k, v, d_o, prm, st);
}

bsattn_status launch_backward_dkdv_tc(const bsattn_plan* p, const void* q, const void* k, const void* v,
                                      const void* d_o, const float* lse, const float* delta, const int32_t* idxT,
                                      const int32_t* cntT, void* dk, void* dv, cudaStream_t st,
                                      const ModParams* mod, void* shares) {
  KvParamsMod prm;
  prm.g = make_geom(p);
  prm.idxT = idxT;
  prm.cntT = cntT;
  prm.lse = lse;
  prm.delta = delta;
  prm.dk = (__nv_bfloat16*)dk;
  prm.dv = (__nv_bfloat16*)dv;
  prm.scale = p->scale;
  prm.scale_log2 = p->scale * 1.4426950408889634f;
  prm.err = p->d_err;
  prm.umax = key_steps(p);
  prm.bm_words = (p->N + 31) / 32;
  prm.pair_axis = pair_axis_of(p);
  const int nd[3] = {p->nT, p->nH, p->nW};
  for (int a = 0; a < 3; ++a) prm.pdim[a] = a == prm.pair_axis ? (nd[a] + 1) / 2 : nd[a];
  const bool d128 = p->desc.head_dim == 128;
  if (mod) {
    prm.mod = *mod;
    prm.shares = backward_shares(p, prm.umax);
    prm.part_kv = (float*)shares;
    if (d128)
      return fits<KvCfg<128, true, 4>>(p, prm.umax) ? run_dkdv<128, true, 4>(p, q, k, v, d_o, prm, st)
                                                    : run_dkdv<128, true, 3>(p, q, k, v, d_o, prm, st);
    return fits<KvCfg<64, true, 4>>(p, prm.umax) ? run_dkdv<64, true, 4>(p, q, k, v, d_o, prm, st)
                                                 : run_dkdv<64, true, 3>(p, q, k, v, d_o, prm, st);
  }
  return d128 ? run_dkdv<128, false, 3>(p, q, k, v, d_o, prm, st) : run_dkdv<64, false, 3>(p, q, k, v, d_o, prm, st);
}
