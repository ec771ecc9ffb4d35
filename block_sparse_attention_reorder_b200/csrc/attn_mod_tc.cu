// Block-sparse attention forward under score rules (tanh cap, distance bias,
// causal, prefix and document masks) on the 5th-generation tensor cores.
//
// Work unit, step list, rings and TMEM layout are those of the forward
// without rules (csrc/attn_tc.cu): a 128-row query block of two 64-row chunks
// walks the union of their kept key chunks, S = Q K^T (N = 64) and O += P V
// per step, two CTAs per SM (one where the plan's lists are longer than 1,300
// steps at D = 128: list, coordinates and the table of chunk origins then take
// more than half of the shared memory; 7,200 at D = 64, e4m3 3,500 and 6,200).
// Different is what stands between the products:
//
//  * The step list is filtered by the rules at set-up (score_mod.cuh): chunks
//    hidden from the whole block are never loaded, and only steps that need
//    element masks evaluate them, from shared bit tables.
//  * The rules cost 3 to 10 FMA-pipe operations a score on top of the
//    softmax's four; masks and their tables are fetched while S is computed.
//  * The reference m of 2^(x - m) is set by the first step that shows the row
//    a key and moves only when a score grows by more than 2^70, for which
//    fp32's exponent range has room in the sums and in bf16 P. So no step
//    waits for its row maximum: the step's sum shows whether a term was too
//    large, and then, hardly ever, the step is taken again with the maximum,
//    and O rescaled.
//  * The MMA warp runs its code as a whole and one elected lane issues, so
//    that descriptors stay in uniform registers. Issued from one lane's
//    branch, a product took 70 to 85 cycles of operand moves, whatever its
//    size, and the twelve of a step bounded the kernel (737 -> 650 us).
//
// Measured on one B200 (12 heads, Wan-1.3B shape, top-k 46 of 364, tiled
// layout, 421 GFLOP on kept pairs): no rule 0.59 ms, cap 0.79, bias 0.76, both
// 1.09; the Wan-14B shape in (6,8,8) tiles with cap and frame-causal mask 12.7
// ms. Bound now by the softmax warps: a step's 64 x 128 exponentials take 512
// of its ~1,050 SM cycles on the SFU, the cap another 384 to 512 on the FMA
// pipe. Eight softmax warps of 32 columns were slower (1,000 against 757 us):
// the per-step scalar work doubles.
//
// A CTA of two steps takes about 9 us of set-up, first loads and epilogue, as
// much as nine more steps, so short lists are bound by that chain: quotients
// by reciprocal, tables a thread per entry and Q loaded while the list is made
// took 16K tokens in 1,024 such CTAs from 50.6 to 41.4 us, and tile windows of
// twelve steps from 228 to 213 us.
//
// Roles (192 threads): warps 0-3 rules and softmax (thread r owns query row
// r), warp 4 TMA producer, warp 5 MMA issuer. Every mbarrier wait is bounded;
// on expiry the CTA sets the device error word, lets issued copies land,
// drains its MMAs and frees TMEM.
#include <cudaTypedefs.h>
#include <math.h>

#include "internal.h"
#include "score_mod.cuh"
#include "steps.cuh"
#include "tc_common.cuh"

namespace {

constexpr int kThreads = 192;
constexpr int kSoftmaxThreads = 128;
constexpr int kStages = 2;
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColS0 = 0, kColS1 = 64, kColO = 128;
constexpr long long kWaitLimit = 4000000000LL;  // SM cycles (~2 s)
constexpr long long kTestWaitLimit = 2000000LL;  // ~1 ms, with the testing hook on
// A row's reference m is put kAbove over a maximum and stays until a score
// exceeds m by kRaise (log2 units), i.e. until the maximum grows by 70: fp32
// sums and bf16 P, both with fp32's exponent range, hold all of 2^-40 .. 2^30
// with values of V from 2^-80 to 2^80, and terms that fall below the range are
// under 2^-86 of the largest.
constexpr float kAbove = 40.f, kRaise = 30.f;
constexpr float kSumLimit = 0x1p30f;  // no term of a smaller sum exceeds m + kRaise
constexpr float kAboveUnit = 0x1p40f;
constexpr float kLeastUnit = 1e-30f;

struct Params {
  Geom g;
  ModParams mod;
  const float* qs;
  const float* ks;
  const int32_t* idx;
  const int32_t* cnt;
  int kmax;
  __nv_bfloat16* o;
  float* lse;
  float scale;
  int* err;
  int umax;      // step list capacity
  int bm_words;  // bitmap words per list
  int pair_axis;
  int pdim[3];
  long long wait_limit;
  int stall;  // testing: the MMA thread first waits on a barrier nothing arrives at
  int parts;  // CTAs that share a query block's steps
  float* part_o;   // parts > 1: [blocks, parts, 128, D] unnormalised O
  float2* part_ml; // [blocks, parts, 128] (m, l) of each row; l = 0: saw no key
};

// A work item's halves; with natural outputs chunks of padded rows only are
// left out. False: nothing to do.
template <bool NAT>
__device__ __forceinline__ bool work_halves(const Params& P, int item, int* i0, int* i1, int* c0, int* c1) {
  const Geom& g = P.g;
  block_halves(g, P.pair_axis, P.pdim, item, i0, i1, c0, c1);
  if (NAT && g.nchunk > 1) {
    if (*i1 >= 0 && !chunk_is_real(g, *i1, *c1)) *i1 = -1;
    if (!chunk_is_real(g, *i0, *c0)) {
      if (*i1 < 0) return false;
      *c0 = *c1;
      *i1 = -1;
    }
  }
  return true;
}

template <int D, bool FP8>
struct Cfg {
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int QRB = D * ESZ;        // Q/K row bytes
  static constexpr int SWB = QRB >= 128 ? 128 : 64;
  static constexpr uint32_t LAYOUT = SWB == 128 ? tc::kLayoutSW128 : tc::kLayoutSW64;
  static constexpr int QBLK = QRB / SWB;     // column blocks of Q/K
  static constexpr int NKS = QRB / 32;       // S MMAs (32 bytes of K each)
  static constexpr int KS_PER_BLK = SWB / 32;
  static constexpr int K_BYTES = 64 * QRB;
  static constexpr int V_BYTES = 64 * D * 2;
  static constexpr int VBLK = D / 64;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 128 * QRB;
  static constexpr int OFF_V = OFF_K + kStages * K_BYTES;
  static constexpr int OFF_BAR = OFF_V + kStages * V_BYTES;
  // barriers: q, kfull[S], vfull[S], sfull[2], pfull[2], pvdone[2], final
  static constexpr int NBAR = 1 + 2 * kStages + 7;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;  // tmem base, abort, steps, zero
  static constexpr int OFF_COL = OFF_MISC + 16;        // 64 packed row codes
  static constexpr int OFF_SCAN = OFF_COL + 256;
  static constexpr int OFF_TOK = OFF_SCAN + 64;        // epilogue: natural token of each block row
  static constexpr int OFF_TAB = OFF_TOK + 512;
  static constexpr int OFF_DYN = OFF_TAB + (int)sizeof(ModTab);  // bitmaps, step list, coordinates
  static constexpr int O_PITCH = D * 2 + 16;
  static_assert(OFF_TAB % 16 == 0, "float4 reads of the table");
  static_assert(128 * O_PITCH <= OFF_BAR - OFF_K, "epilogue staging fits in the rings");
};

__device__ __forceinline__ void record_timeout(volatile int* abort_flag, int* err) {
  *abort_flag = 1;
  atomicOr(err, BSATTN_DEVERR_TIMEOUT);
}

__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// CAP and BIAS: whether scores are capped and biased. Masks need no variant:
// steps that need none skip them by one flag test. Branches and scalar work
// per step are what a softmax warp cannot hide (two divisions a step cost
// 20% of the time), so what the call fixes is fixed at compile time or ahead
// of the loop.
template <int D, bool FP8, bool NAT, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kThreads, 2)
attn_mod_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params P) {
  using C = Cfg<D, FP8>;
  // Cap and bias together: 32 columns at a time in a loop, with P in two
  // halves (16 columns each, 32 apart). Straight-line code for all 64 stalls
  // on instruction fetch (1.7 warps a cycle, against 0.8 with the cap alone):
  // 1,380 us against 1,177 us at the Wan-1.3B shape.
  constexpr bool kHalves = CAP && BIAS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sb = tc::smem_addr(smem);
  const uint32_t bar_q = sb + C::OFF_BAR;
  auto bar_kfull = [&](int s) { return sb + C::OFF_BAR + 8u * (1 + s); };
  auto bar_vfull = [&](int s) { return sb + C::OFF_BAR + 8u * (1 + kStages + s); };
  auto bar_sfull = [&](int b) { return sb + C::OFF_BAR + 8u * (1 + 2 * kStages + b); };
  auto bar_pfull = [&](int b) { return sb + C::OFF_BAR + 8u * (3 + 2 * kStages + b); };
  auto bar_pvdone = [&](int b) { return sb + C::OFF_BAR + 8u * (5 + 2 * kStages + b); };
  const uint32_t bar_final = sb + C::OFF_BAR + 8u * (7 + 2 * kStages);
  uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  volatile int* never = reinterpret_cast<volatile int*>(misc + 3);  // stays 0: waits that ignore abort
  uint32_t* colc = reinterpret_cast<uint32_t*>(smem + C::OFF_COL);
  int* scan = reinterpret_cast<int*>(smem + C::OFF_SCAN);
  ModTab* tab = reinterpret_cast<ModTab*>(smem + C::OFF_TAB);
  uint32_t* bmA = reinterpret_cast<uint32_t*>(smem + C::OFF_DYN);
  uint32_t* bmB = bmA + P.bm_words;
  uint32_t* ulist = bmB + P.bm_words;
  uint32_t* uext = ulist + P.umax;                        // packed coordinates and flags of each step
  float* uks = reinterpret_cast<float*>(uext + P.umax);   // e4m3: each step's key-tile scale

  const Geom& g = P.g;
  const ModParams& M = P.mod;
  // Causal order: the last frames see the most keys, so they start first and
  // the short lists fill the end of the grid.
  const int first = M.causal ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
  const int item = first / P.parts, part = first % P.parts;
  int i0, i1, c0, c1;
  if (!work_halves<NAT>(P, item, &i0, &i1, &c0, &c1)) return;  // uniform over the CTA, before any set-up
  const int head = blockIdx.y, b = blockIdx.z;
  const size_t bh = (size_t)b * g.Hh + head;
  const bool has1 = i1 >= 0;
  // First tiled-layout row of chunk c of tile j.
  auto tiled_row = [&](int j, int c) -> int { return (int)((bh * g.N + j) * g.V) + 64 * c; };
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // known to be uniform

  // The list counts and this thread's first entry of each list come first, so
  // that their latency overlaps the set-up (entries at and beyond a count are
  // read but not used).
  const int32_t* lA = P.idx + (bh * g.N + i0) * (size_t)P.kmax;
  const int32_t* lB = has1 ? P.idx + (bh * g.N + i1) * (size_t)P.kmax : lA;
  int nA = P.cnt[bh * g.N + i0];
  int nB = has1 ? P.cnt[bh * g.N + i1] : 0;
  int jA = tid < P.kmax ? __ldg(lA + tid) : 0;
  int jB = has1 && tid < P.kmax ? __ldg(lB + tid) : 0;

  // ------------------------------------------------------------ setup
  if (tid == 0) {
    tc::mbar_init(bar_q, 1);
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init(bar_kfull(s), 1);
      tc::mbar_init(bar_vfull(s), 1);
    }
    for (int x = 0; x < 2; ++x) {
      tc::mbar_init(bar_sfull(x), 1);
      tc::mbar_init(bar_pfull(x), kSoftmaxThreads);
      tc::mbar_init(bar_pvdone(x), 1);
    }
    tc::mbar_init(bar_final, 1);
    misc[1] = 0;
    misc[3] = 0;
    tc::mbar_fence_init();
  }
  if (warp == 5) {
    tc::tmem_alloc(sb + C::OFF_MISC, kTmemCols);
    tc::tmem_relinquish();
  }
  if (tid < 64) colc[tid] = chunk_row_code(g, tid);
  if (g.cr < 64) {
    // Tiles of fewer than 64 tokens: natural-layout loads fill only the
    // chunk box's rows; the rest of every V slot must hold finite values.
    for (int x = tid; x < kStages * C::V_BYTES / 16; x += kThreads)
      reinterpret_cast<uint4*>(smem + C::OFF_V)[x] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  for (int w = tid; w < 2 * P.bm_words; w += kThreads) bmA[w] = 0u;
  if (!has1) {  // rows 64..127 of the query block have no chunk
    for (int x = tid; x < C::QBLK * 64 * C::SWB / 16; x += kThreads) {
      const int cb = x / (64 * C::SWB / 16), off = x % (64 * C::SWB / 16);
      reinterpret_cast<uint4*>(smem + C::OFF_Q + cb * 128 * C::SWB + 64 * C::SWB)[off] = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  const int prefix = M.prefix ? __ldg(M.prefix + b) : 0;
  // A natural-layout load fills the chunk box's rows (cr of them).
  const int qrows = NAT && !FP8 ? g.cr : 64, kvrows = NAT ? g.cr : 64;
  // One chunk (64 tokens x 64 columns) of a natural-layout tensor: the
  // box {64 columns, cw, ch, ct, 1} at the chunk's first token.
  auto load_nat = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int col, mod::Coord p) {
    tc::tma_load_5d(dst, map, bar, col, p.w, p.h, p.t, b);
  };
  if (warp == 4 && lane == 0) {
    tc::tma_prefetch_desc(&tmQ);
    tc::tma_prefetch_desc(&tmK);
    tc::tma_prefetch_desc(&tmV);
  }
  __syncthreads();
  if (warp == 4 && lane == 0) {  // the block's Q, while the list is made
    tc::mbar_arrive_expect_tx(bar_q, (has1 ? 2 : 1) * qrows * C::QRB);
    for (int x = 0; x < (has1 ? 2 : 1); ++x) {
      const int tile = x ? i1 : i0, chunk = x ? c1 : c0;
      const mod::Coord qp = mod::chunk_first(g, M, mod::pack_tile(g, M, tile), mod::origin_of(g, chunk));
#pragma unroll
      for (int cb = 0; cb < C::QBLK; ++cb) {
        const uint32_t dst = sb + C::OFF_Q + cb * 128 * C::SWB + x * 64 * C::SWB;
        if (NAT && !FP8)
          load_nat(dst, &tmQ, bar_q, head * D + cb * 64, qp);
        else
          tc::tma_load_2d(dst, &tmQ, bar_q, cb * C::SWB / C::ESZ, tiled_row(tile, chunk));
      }
    }
  }
  __syncwarp();
  if (nA < 0 || nA > P.kmax || nB < 0 || nB > P.kmax) {
    if (tid == 0) atomicOr(P.err, BSATTN_DEVERR_BAD_INDEX);
    nA = min(max(nA, 0), P.kmax);
    nB = min(max(nB, 0), P.kmax);
  }
  {
    for (int e = tid; e < max(nA, nB); e += kThreads) {
      if (e != tid) {
        jA = e < nA ? __ldg(lA + e) : 0;
        jB = e < nB ? __ldg(lB + e) : 0;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (e >= (x ? nB : nA)) continue;
        const int j = x ? jB : jA;
        if (j < 0 || j >= g.N) {
          atomicOr(P.err, BSATTN_DEVERR_BAD_INDEX);
          continue;
        }
        atomicOr(x ? &bmB[j >> 5] : &bmA[j >> 5], 1u << (j & 31));
      }
    }
  }
  __syncthreads();
  list_steps<kThreads>(g, bmA, bmB, P.bm_words, ulist, P.umax, scan, misc + 2);
  fill_modtab<kThreads>(g, tab, colc);
  __syncthreads();
  {
    const int steps = (int)misc[2];
    int left = mod::filter_steps<kThreads, false>(g, M, b, prefix, i0, i1, c0, c1, ulist, uext, steps, scan,
                                                       tab->origin);
    __syncthreads();
    if (BIAS) nearest_first<kThreads>(ulist, uext, left, i0);
    if (P.parts > 1) left = take_share<kThreads>(ulist, uext, left, part, P.parts);
    if (tid == 0) misc[2] = (uint32_t)left;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, misc[0], 0);
  const int L = __shfl_sync(0xffffffffu, (int)misc[2], 0);

  // ------------------------------------------------------------ roles
  if (warp == 4) {
    if (lane == 0 && L > 0) {
      // K_m is issued as soon as S_{m-2} has released its slot, V_{m-1} once
      // PV_{m-3} has: K runs one step ahead of V.
      int lastk[kStages], lastv[kStages];
#pragma unroll
      for (int s = 0; s < kStages; ++s) lastk[s] = lastv[s] = -1;
      for (int m = 0; m <= L; ++m) {
        if (m < L) {
          const int s = m % kStages;
          if (m >= kStages &&
              !tc::mbar_wait(bar_sfull(s), ((m / kStages) - 1) & 1, abort_flag, P.wait_limit)) {
            record_timeout(abort_flag, P.err);
            break;
          }
          const int kt = (int)(ulist[m] & 0x1FFFFFu), kc = (int)((ulist[m] >> 21) & 0x1FFu);
          tc::mbar_arrive_expect_tx(bar_kfull(s), FP8 ? C::K_BYTES : kvrows * C::QRB);
          const mod::Coord kp = mod::chunk_first(g, M, uext[m], tab->at(kc));
#pragma unroll
          for (int cb = 0; cb < C::QBLK; ++cb) {
            const uint32_t dst = sb + C::OFF_K + s * C::K_BYTES + cb * 64 * C::SWB;
            if (NAT && !FP8)
              load_nat(dst, &tmK, bar_kfull(s), head * D + cb * 64, kp);
            else
              tc::tma_load_2d(dst, &tmK, bar_kfull(s), cb * C::SWB / C::ESZ, tiled_row(kt, kc));
          }
          lastk[s] = m;
        }
        if (m >= 1) {
          const int v = m - 1, s = v % kStages;
          if (v >= kStages &&
              !tc::mbar_wait(bar_pvdone(s), ((v / kStages) - 1) & 1, abort_flag, P.wait_limit)) {
            record_timeout(abort_flag, P.err);
            break;
          }
          const int vt = (int)(ulist[v] & 0x1FFFFFu), vc = (int)((ulist[v] >> 21) & 0x1FFu);
          tc::mbar_arrive_expect_tx(bar_vfull(s), kvrows * D * 2);
          const mod::Coord vp = mod::chunk_first(g, M, uext[v], tab->at(vc));
#pragma unroll
          for (int vb = 0; vb < C::VBLK; ++vb) {
            const uint32_t dst = sb + C::OFF_V + s * C::V_BYTES + vb * 8192;
            if (NAT)
              load_nat(dst, &tmV, bar_vfull(s), head * D + vb * 64, vp);
            else
              tc::tma_load_2d(dst, &tmV, bar_vfull(s), vb * 64, tiled_row(vt, vc));
          }
          lastv[s] = v;
        }
      }
      if (*abort_flag) {
        // Let copies already issued land before the CTA's memory goes away.
        for (int s = 0; s < kStages; ++s) {
          if (lastk[s] >= 0) tc::mbar_wait(bar_kfull(s), (lastk[s] / kStages) & 1, never, kWaitLimit);
          if (lastv[s] >= 0) tc::mbar_wait(bar_vfull(s), (lastv[s] / kStages) & 1, never, kWaitLimit);
        }
      }
    }
    if (lane == 0 && (L == 0 || *abort_flag)) tc::mbar_wait(bar_q, 0, never, kWaitLimit);  // the block's load too
  } else if (warp == 5) {
    if (L > 0) {
      const uint32_t lead = tc::elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, tc::mbar_wait(bar, parity, abort_flag, P.wait_limit));
      };
      constexpr uint32_t idS = FP8 ? tc::instr_desc(0, 0, 0, 0, 64, 128) : tc::instr_desc(1, 1, 0, 0, 64, 128);
      constexpr uint32_t idPV = tc::instr_desc(1, 1, 0, 1, D, 128);
      // Testing hook: bar_final gets its first arrival only from the final
      // commit below, so this wait runs out and the CTA takes the timeout path.
      bool ok = !P.stall || wait(bar_final, 0);
      ok = ok && wait(bar_q, 0);
      auto issue_S = [&](int m) -> bool {
        const int s = m % kStages;
        if (!wait(bar_kfull(s), (m / kStages) & 1)) return false;
        tc::fence_after_sync();
        const uint32_t dS = tmem + ((m & 1) ? kColS1 : kColS0);
#pragma unroll
        for (int kk = 0; kk < C::NKS; ++kk) {
          const int cb = kk / C::KS_PER_BLK, within = kk % C::KS_PER_BLK;
          const uint64_t da = tc::smem_desc(sb + C::OFF_Q + cb * 128 * C::SWB + within * 32, 16, 8 * C::SWB, C::LAYOUT);
          const uint64_t db =
              tc::smem_desc(sb + C::OFF_K + s * C::K_BYTES + cb * 64 * C::SWB + within * 32, 16, 8 * C::SWB, C::LAYOUT);
          if (FP8)
            tc::mma_ss_f8_warp(lead, dS, da, db, idS, kk > 0 ? 1u : 0u);
          else
            tc::mma_ss_f16_warp(lead, dS, da, db, idS, kk > 0 ? 1u : 0u);
        }
        tc::mma_commit_warp(lead, bar_sfull(m & 1));
        return true;
      };
      if (ok) ok = issue_S(0);
      if (ok && L > 1) ok = issue_S(1);
      for (int n = 0; ok && n < L; ++n) {
        const int s = n % kStages;
        if (!wait(bar_pfull(n & 1), (n >> 1) & 1) || !wait(bar_vfull(s), (n / kStages) & 1)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t pA = tmem + ((n & 1) ? kColS1 : kColS0);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t dv = tc::smem_desc(sb + C::OFF_V + s * C::V_BYTES + kk * 2048, 8192, 1024, tc::kLayoutSW128);
          tc::mma_ts_f16_warp(lead, tmem + kColO, pA + (kHalves && kk >= 2 ? 16 : 0) + kk * 8, dv, idPV, (n > 0 || kk > 0) ? 1u : 0u);
        }
        tc::mma_commit_warp(lead, bar_pvdone(n & 1));
        if (n + 2 < L && !issue_S(n + 2)) {
          ok = false;
          break;
        }
      }
      if (!ok && lead) record_timeout(abort_flag, P.err);
      // Every MMA issued so far has finished before TMEM is released.
      tc::mma_commit_warp(lead, bar_final);
      tc::mbar_wait(bar_final, 0, never, kWaitLimit);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------- softmax
    const int r = tid;         // query row of the block
    const int half = r >> 6;   // 0: first chunk, 1: second
    const bool row_exists = half == 0 || has1;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const float qsc = (FP8 && row_exists) ? P.qs[bh * g.N + (half ? i1 : i0)] : 1.f;
    if (FP8) {
      for (int n = tid; n < L; n += kSoftmaxThreads) uks[n] = __ldg(P.ks + bh * g.N + (ulist[n] & 0x1FFFFFu));
      sync_softmax();
    }
    mod::Row row{};
    if (row_exists) row = mod::row_of(g, M, b, half ? i1 : i0, half ? c1 : c0, colc[r & 63], r & 63);
    const float cap = CAP ? M.cap : 1.f;
    // Scores stay in units of `unit`: the raw products (unit = the scale, with
    // the tile scales on the e4m3 path), or tanh values (unit = the cap); the
    // bias is added in the same units, and one FMA per score applies
    // c = unit log2(e). `kq` takes raw products to the argument of tanh.
    const float slope = BIAS ? __ldg(M.slopes + head) : 0.f;
    // e4m3 tiles of tiny values: a unit below kLeastUnit, whose scores (448^2 D
    // units at most) are no more than 1e-22, is taken for it, so that the bias
    // stays finite in it.
    constexpr bool kFloor = FP8 && BIAS && !CAP;
    const float sq = kFloor ? fmaxf(P.scale * qsc, kLeastUnit) : P.scale * qsc, kq = sq / cap;
    const float least_ks = kFloor ? kLeastUnit / sq : 0.f;
    const float c_fix = (CAP ? cap : sq) * mod::kLog2e;     // c, without the key tile's scale
    const float nslope = -slope / (CAP ? cap : sq);         // likewise
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    auto step_chunk = [&](uint32_t e) -> size_t {  // a step's chunk among all of the batch's
      return ((size_t)b * g.N + (e & 0x1FFFFFu)) * g.nchunk + ((e >> 21) & 0x1FFu);
    };
    // Rescales what this row has accumulated before step n by alpha.
    auto rescale = [&](int n, float alpha) -> bool {
      // O holds PV_0..PV_{n-1} once PV_{n-1} has completed.
      if (!__all_sync(0xffffffffu, tc::mbar_wait(bar_pvdone((n - 1) & 1), ((n - 1) >> 1) & 1, abort_flag, P.wait_limit)))
        return false;
      tc::fence_after_sync();
#pragma unroll 1
      for (int col = 0; col < D; col += 16) {
        uint32_t o[16];
        tc::tmem_ld16_wait(tmem + lane_base + kColO + col, o);
#pragma unroll
        for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * alpha);
        tc::tmem_st16(tmem + lane_base + kColO + col, o);
      }
      return true;
    };
    // Whether scores of the warp may hold anything in masked places without
    // hidden keys: rows that are no visible token, and, in chunks of fewer than
    // 64 tokens, key rows that no load fills. They must not pick the form of
    // tanh.
    const bool odd_rows = __any_sync(0xffffffffu, !row.live) || g.cr < 64;
    bool fresh = true;  // some row of the warp has seen no key yet
    uint32_t e = L > 0 ? ulist[0] : 0u, ext = L > 0 ? uext[0] : 0u;
    for (int n = 0; n < L; ++n) {
      const bool keep = ((e >> (30 + half)) & 1u) != 0;  // uniform within the warp
      unsigned long long vis = ~0ull;
      bool partial = false, clear = false;
      mod::Dist dist{};
      if (BIAS || (ext & mod::kSpecial)) {
        const mod::Coord f = mod::chunk_first(g, M, ext, tab->at((int)((e >> 21) & 0x1FFu)));
        if (BIAS) dist = mod::make_dist(g, M, row.at, f, kFloor ? nslope / fmaxf(uks[n], least_ks) : nslope);
        if (ext & mod::kSpecial) {
          if ((ext & mod::kHidden) && warp < 2) {
            // V rows of hidden tokens become zeros before the product reads them.
            // Only once S_n is there: S_n follows PV_{n-2}, so the slot's barrier is
            // past V_{n-2}, whose phase has the parity that stands for V_n's before.
            const bool hidden = __ldg(M.doc_rows + 64 * step_chunk(e) + tid) < 0;
            ok = __all_sync(0xffffffffu,
                            tc::mbar_wait(bar_sfull(n & 1), (n >> 1) & 1, abort_flag, P.wait_limit) &&
                                tc::mbar_wait(bar_vfull(n % kStages), (n / kStages) & 1, abort_flag, P.wait_limit));
            if (ok && hidden) mod::zero_row(smem + C::OFF_V + (n % kStages) * C::V_BYTES, C::VBLK, tid);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          if (keep) {
            int vt = g.T - f.t;
            if (M.causal) vt = min(vt, max(row.at.t + 1, prefix) - f.t);
            vis = mod::visible_box(g, &tab->col, 0, vt, g.H - f.h, g.W - f.w);
            if (ext & mod::kDoc) vis &= mod::visible_doc(M, step_chunk(e), row.id);
            if (!row.live) vis = 0;
            partial = __any_sync(0xffffffffu, vis != ~0ull);
            clear = partial && ((ext & mod::kHidden) || odd_rows);
          }
        }
      }
      const float ksc = kFloor ? fmaxf(uks[n], least_ks) : FP8 ? uks[n] : 1.f;
      const int n1 = min(n + 1, L - 1);
      e = ulist[n1];
      ext = uext[n1];
      ok = ok && __all_sync(0xffffffffu, tc::mbar_wait(bar_sfull(n & 1), (n >> 1) & 1, abort_flag, P.wait_limit));
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t sbuf = tmem + lane_base + ((n & 1) ? kColS1 : kColS0);
      if constexpr (kHalves) {
        const float k = FP8 ? kq * ksc : kq;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
          if (keep) {
            uint32_t sr[32];
            const uint32_t see = (uint32_t)(vis >> (32 * h));
            tc::tmem_ld32_wait(sbuf + 32 * h, sr);
            if (clear) mod::set_unseen<32>(sr, see, 0.f);
            mod::tanh_scores<32>(sr, k);
            mod::add_distance<32>(g, reinterpret_cast<float*>(sr), &tab->col, 32 * h, dist);
            if (partial) mod::set_unseen<32>(sr, see, -INFINITY);
            float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int q = 0; q < 16; ++q)
              mx4[q & 3] = tc::fmax3(mx4[q & 3], __uint_as_float(sr[2 * q]), __uint_as_float(sr[2 * q + 1]));
            const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * c_fix;
            const bool raise = mx > m + kRaise;  // m = -inf: the row has seen no key and its O row is zero
            if (__any_sync(0xffffffffu, raise)) {
              const float alpha = raise && m != -INFINITY ? tc::ex2(m - (mx + kAbove)) : 1.f;
              if (raise) m = mx + kAbove;
              if (__any_sync(0xffffffffu, alpha != 1.f)) {
                // What the first half stored is read again below: its P, and O
                // where the reference moved there too. Stores and loads of
                // tensor memory are ordered by a wait only.
                tc::tmem_wait_st();
                l *= alpha;
                if (n > 0) ok = rescale(n, alpha);
                if (h == 1) {  // this step's first 32 probabilities
                  tc::tmem_ld16_wait(sbuf, pk);
#pragma unroll
                  for (int q = 0; q < 16; ++q) {
                    const float2 p = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&pk[q]));
                    pk[q] = mod::pack(make_float2(p.x * alpha, p.y * alpha));
                  }
                  tc::tmem_st16(sbuf, pk);
                }
              }
            }
            // A row that has seen no key yet has m = -inf and only -inf scores.
            const float2 c2 = mod::bc(c_fix), nm2 = mod::bc(m == -INFINITY ? 0.f : -m);
            float2 ls2[2] = {mod::bc(0.f), mod::bc(0.f)};
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float2 x = __ffma2_rn(mod::pair(sr + 2 * q), c2, nm2);
              const float2 p = make_float2(tc::ex2(x.x), tc::ex2(x.y));
              ls2[q & 1] = __fadd2_rn(ls2[q & 1], p);
              pk[q] = mod::pack(p);
            }
            const float2 ls = __fadd2_rn(ls2[0], ls2[1]);
            l += ls.x + ls.y;
          } else {
#pragma unroll
            for (int q = 0; q < 16; ++q) pk[q] = 0u;
          }
          tc::tmem_st16(sbuf + 32 * h, pk);  // P over the first 16 columns of its half of S_n
        }
        if (!ok) break;
      } else {
        uint32_t pk[32];
        float alpha = 1.f;
        if (keep) {
          const float c = FP8 && !CAP ? c_fix * ksc : c_fix, k = FP8 ? kq * ksc : kq;
          float sum;
          uint32_t sr[64];
          // P and its sum from the modified scores.
          auto exponentials = [&]() {
            // A row that has seen no key yet has m = -inf and only -inf scores.
            const float2 c2 = mod::bc(c), nm2 = mod::bc(m == -INFINITY ? 0.f : -m);
            float2 ls2[4] = {mod::bc(0.f), mod::bc(0.f), mod::bc(0.f), mod::bc(0.f)};
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              const float2 x = __ffma2_rn(mod::pair(sr + 2 * q), c2, nm2);
              const float2 p = make_float2(tc::ex2(x.x), tc::ex2(x.y));
              ls2[q & 3] = __fadd2_rn(ls2[q & 3], p);
              pk[q] = mod::pack(p);
            }
            const float2 ls = __fadd2_rn(__fadd2_rn(ls2[0], ls2[1]), __fadd2_rn(ls2[2], ls2[3]));
            sum = ls.x + ls.y;
          };
          // Once more with the row maxima when a score turns out to be far above
          // its row's reference.
          bool done = false;
          for (bool measure = fresh; !done; measure = true) {
            tc::tmem_ld64_wait(sbuf, sr);
            if (CAP) {
              if (clear) mod::set_unseen<64>(sr, vis, 0.f);
              mod::tanh_scores<64>(sr, k);
            }
            if (BIAS) mod::add_distance<64>(g, reinterpret_cast<float*>(sr), &tab->col, 0, dist);
            if (partial) mod::set_unseen<64>(sr, vis, -INFINITY);
            if (measure) {
              float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int q = 0; q < 32; ++q)
                mx4[q & 3] = tc::fmax3(mx4[q & 3], __uint_as_float(sr[2 * q]), __uint_as_float(sr[2 * q + 1]));
              const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * c;
              if (mx > m + kRaise) {  // m = -inf: the row has seen no key and its O row is zero
                if (m != -INFINITY) alpha = tc::ex2(m - (mx + kAbove));
                m = mx + kAbove;
              }
              fresh = __any_sync(0xffffffffu, m == -INFINITY);
            }
            exponentials();
            done = measure || __all_sync(0xffffffffu, sum <= kSumLimit);
          }
          l = l * alpha + sum;
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) pk[q] = 0u;
        }
        tc::tmem_st32(sbuf, pk);  // P_n over the first 32 columns of S_n
        if (__any_sync(0xffffffffu, alpha != 1.f) && !rescale(n, alpha)) {
          ok = false;
          break;
        }
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      tc::mbar_arrive(bar_pfull(n & 1));
    }
    if (!ok) record_timeout(abort_flag, P.err);
    // ---------------------------------------------------------- epilogue
    if (ok && L > 0) {
      if (!__all_sync(0xffffffffu,
                      tc::mbar_wait(bar_pvdone((L - 1) & 1), ((L - 1) >> 1) & 1, abort_flag, P.wait_limit))) {
        record_timeout(abort_flag, P.err);
        ok = false;
      }
      tc::fence_after_sync();
    }
    int* tokrow = reinterpret_cast<int*>(smem + C::OFF_TOK);
    if (NAT) {
      const bool real = row_exists && (r & 63) < g.cr && row.at.t < g.T && row.at.h < g.H && row.at.w < g.W;
      tokrow[r] = real ? (row.at.t * g.H + row.at.h) * g.W + row.at.w : -1;
    }
    if (!row.live || !ok) l = 0.f;  // padded or hidden: a zero row
    if (P.parts > 1) {
      const size_t at = (((bh * (gridDim.x / P.parts) + item) * P.parts + part) * 128 + r);
      P.part_ml[at] = make_float2(m, l);
      if (ok && L > 0) {
#pragma unroll
        for (int col = 0; col < D; col += 16) {
          uint32_t o[16];
          tc::tmem_ld16_wait(tmem + lane_base + kColO + col, o);
          if (l == 0.f) continue;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            reinterpret_cast<uint4*>(P.part_o + at * D + col)[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
    } else {
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a sum that is no number stays one, as where parts are joined
      uint8_t* stage = smem + C::OFF_K + r * C::O_PITCH;
#pragma unroll
      for (int col = 0; col < D; col += 32) {
        uint32_t o[32];
        if (ok && L > 0) {
          tc::tmem_ld32_wait(tmem + lane_base + kColO + col, o);
        }
        if (!(ok && L > 0 && row.live)) {  // whatever the row holds, NaN included
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] = 0u;
        }
        uint32_t w[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) w[q] = mod::pack(__fmul2_rn(mod::pair(o + 2 * q), mod::bc(inv)));
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<uint4*>(stage + col * 2)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
      }
      if (P.lse && row_exists) {
        // In terms of the maximum, so that no rounding of m's size enters.
        const float lse_r = l == 0.f ? -INFINITY : ((m - kAbove) + log2f(l * kAboveUnit)) * 0.69314718055994531f;
        if (NAT) {
          if (tokrow[r] >= 0) P.lse[bh * (size_t)g.L + (size_t)tokrow[r]] = lse_r;
        } else {
          P.lse[(size_t)tiled_row(half ? i1 : i0, half ? c1 : c0) + (r & 63)] = lse_r;
        }
      }
      sync_softmax();
      constexpr int CPR = D / 8;  // 16-byte pieces per row
      const int rows = has1 ? 128 : 64;
      for (int e2 = tid; e2 < rows * CPR; e2 += kSoftmaxThreads) {
        const int rr = e2 / CPR, cc = e2 % CPR;
        const uint4 val = *reinterpret_cast<const uint4*>(smem + C::OFF_K + rr * C::O_PITCH + cc * 16);
        if (NAT) {
          const int n = tokrow[rr];
          if (n >= 0) reinterpret_cast<uint4*>(P.o + (((size_t)b * g.L + n) * g.Hh + head) * D)[cc] = val;
        } else {
          uint4* og = reinterpret_cast<uint4*>(P.o + (size_t)tiled_row(rr >> 6 ? i1 : i0, rr >> 6 ? c1 : c0) * D);
          og[(rr & 63) * CPR + cc] = val;
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of each query block: with M the greatest m + log2(l), w =
// 2^(m - M), l = sum w l, O = sum w O / l. D / 8 threads a row, eight features
// each; a CTA takes kJoinRows rows, every load of a thread in flight at once.
constexpr int kMaxParts = 8, kJoinRows = 16;
template <int D, bool NAT>
__global__ void __launch_bounds__(kJoinRows * D / 8) attn_join_kernel(const __grid_constant__ Params P) {
  const Geom& g = P.g;
  const int head = blockIdx.y, b = blockIdx.z, item = blockIdx.x / (128 / kJoinRows);
  const size_t bh = (size_t)b * g.Hh + head;
  const int r = blockIdx.x % (128 / kJoinRows) * kJoinRows + threadIdx.x / (D / 8), piece = threadIdx.x % (D / 8);
  const int half = r >> 6;
  int i0, i1, c0, c1;
  if (!work_halves<NAT>(P, item, &i0, &i1, &c0, &c1) || (half && i1 < 0)) return;
  const size_t at = ((bh * (gridDim.x / (128 / kJoinRows)) + item) * P.parts) * 128 + r;
  float2 ml[kMaxParts];
  float4 x[kMaxParts], y[kMaxParts];
#pragma unroll
  for (int p = 0; p < kMaxParts; ++p) {
    ml[p] = p < P.parts ? P.part_ml[at + p * 128] : make_float2(0.f, 0.f);
    if (p < P.parts) {  // unwritten where l = 0, and not used then
      const float4* src = reinterpret_cast<const float4*>(P.part_o + (at + p * 128) * D) + 2 * piece;
      x[p] = src[0];
      y[p] = src[1];
    }
  }
  const int tile = half ? i1 : i0, chunk = half ? c1 : c0;
  size_t out;  // row of O and lse
  if (NAT) {
    const uint32_t code = chunk_row_code(g, r & 63);
    const mod::Coord f = mod::chunk_first(g, P.mod, mod::pack_tile(g, P.mod, tile), chunk_origin(g, chunk));
    const int t = f.t + (int)(code & 0xffu), h = f.h + (int)((code >> 8) & 0xffu), w = f.w + (int)((code >> 16) & 0xffu);
    if ((r & 63) >= g.cr || t >= g.T || h >= g.H || w >= g.W) return;
    out = (size_t)(t * g.H + h) * g.W + w;
  } else {
    out = (bh * g.N + tile) * g.V + 64 * chunk + (r & 63);
  }
  float M = -INFINITY;
#pragma unroll
  for (int p = 0; p < kMaxParts; ++p)
    if (ml[p].y != 0.f) M = fmaxf(M, ml[p].x + log2f(ml[p].y));
  float l = 0.f;
  float2 o[4] = {mod::bc(0.f), mod::bc(0.f), mod::bc(0.f), mod::bc(0.f)};
#pragma unroll
  for (int p = 0; p < kMaxParts; ++p) {
    if (ml[p].y == 0.f) continue;
    const float w = exp2f(ml[p].x - M);
    const float2 w2 = mod::bc(w);
    l = fmaf(w, ml[p].y, l);
    o[0] = __ffma2_rn(w2, make_float2(x[p].x, x[p].y), o[0]);
    o[1] = __ffma2_rn(w2, make_float2(x[p].z, x[p].w), o[1]);
    o[2] = __ffma2_rn(w2, make_float2(y[p].x, y[p].y), o[2]);
    o[3] = __ffma2_rn(w2, make_float2(y[p].z, y[p].w), o[3]);
  }
  const float2 inv = mod::bc(l == 0.f ? 0.f : 1.f / l);
  __nv_bfloat16* dst = P.o + (NAT ? (((size_t)b * g.L + out) * g.Hh + head) * D : out * D);
  reinterpret_cast<uint4*>(dst)[piece] = make_uint4(mod::pack(__fmul2_rn(o[0], inv)), mod::pack(__fmul2_rn(o[1], inv)),
                                                    mod::pack(__fmul2_rn(o[2], inv)), mod::pack(__fmul2_rn(o[3], inv)));
  if (P.lse && piece == 0)
    P.lse[NAT ? bh * (size_t)g.L + out : out] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
}

// Fixed part, two list bitmaps, step list, coordinates and (e4m3) scales.
template <int D, bool FP8>
size_t smem_bytes(const bsattn_plan* p) {
  const size_t smem = 1024 + Cfg<D, FP8>::OFF_DYN + (size_t)((p->N + 31) / 32) * 8 +
                      (size_t)attention_steps(p) * (FP8 ? 12 : 8);
  return smem < 80 * 1024 ? 80 * 1024 : smem;  // at most two CTAs (2 x 256 TMEM columns) per SM
}

template <int D, bool FP8, bool NAT, bool CAP, bool BIAS>
bsattn_status run(const bsattn_plan* p, const void* q, const void* k, const __nv_bfloat16* v, const Params& prm,
                  cudaStream_t st) {
  using C = Cfg<D, FP8>;
  const uint64_t rows = tiled_rows(p);
  CUtensorMap mq, mk, mv;
  const CUtensorMapDataType dqk = FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUtensorMapSwizzle sw = C::SWB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (NAT && !FP8 ? !bsattn_make_map_nat(&mq, q, p) || !bsattn_make_map_nat(&mk, k, p)
                  : !bsattn_make_map_2d(&mq, q, dqk, C::ESZ, D, rows, C::SWB / C::ESZ, 64, sw) ||
                        !bsattn_make_map_2d(&mk, k, dqk, C::ESZ, D, rows, C::SWB / C::ESZ, 64, sw))
    return BSATTN_ERR_CUDA;
  if (NAT ? !bsattn_make_map_nat(&mv, v, p)
          : !bsattn_make_map_2d(&mv, v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, D, rows, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B))
    return BSATTN_ERR_CUDA;
  const size_t smem = smem_bytes<D, FP8>(p);
  auto kern = attn_mod_tc_kernel<D, FP8, NAT, CAP, BIAS>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return BSATTN_ERR_CUDA;
  const int items = attention_items(p);
  kern<<<dim3(items * prm.parts, p->desc.heads, p->desc.B), kThreads, smem, st>>>(mq, mk, mv, prm);
  if (prm.parts > 1)
    attn_join_kernel<D, NAT><<<dim3(items * (128 / kJoinRows), p->desc.heads, p->desc.B), kJoinRows * D / 8, 0, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

template <int D, bool FP8, bool NAT>
bsattn_status run(const bsattn_plan* p, const void* q, const void* k, const __nv_bfloat16* v, const Params& prm,
                  cudaStream_t st) {
  if (prm.mod.cap > 0.f)
    return prm.mod.slopes ? run<D, FP8, NAT, true, true>(p, q, k, v, prm, st)
                          : run<D, FP8, NAT, true, false>(p, q, k, v, prm, st);
  return prm.mod.slopes ? run<D, FP8, NAT, false, true>(p, q, k, v, prm, st)
                        : run<D, FP8, NAT, false, false>(p, q, k, v, prm, st);
}

}  // namespace

// Few query blocks leave most of the GPU idle while each walks its list: up to
// eight CTAs then share a block's steps, two per SM at most over the grid and
// four steps each at least, and a second kernel joins their parts (two heads
// of 8 x 16 x 16 tokens, about 20 steps a block: 40 us alone, 21 us shared).
static int attention_parts(const bsattn_plan* p) {
  const long long blocks = (long long)attention_items(p) * p->desc.heads * p->desc.B;
  long long parts = 2 * 148 / blocks;
  if (parts > attention_steps(p) / 4) parts = attention_steps(p) / 4;
  return parts < 2 ? 1 : parts > kMaxParts ? kMaxParts : (int)parts;
}
size_t attention_mod_workspace_bytes(const bsattn_plan* p) {
  const int parts = attention_parts(p);
  if (parts == 1) return 0;
  const size_t rows = (size_t)attention_items(p) * p->desc.heads * p->desc.B * parts * 128;
  return rows * ((size_t)p->desc.head_dim * sizeof(float) + sizeof(float2));
}

bsattn_status check_attention_mod(const bsattn_plan* p) {
  if (p->N > 32768 || tiled_rows(p) + 128 >= (1ull << 31)) return BSATTN_ERR_UNSUPPORTED;
  if (p->desc.B > 65535 || p->desc.heads > 65535) return BSATTN_ERR_UNSUPPORTED;  // grid
  const bool fp8 = p->desc.qk_fp8 != 0, d128 = p->desc.head_dim == 128;
  const size_t smem = d128 ? (fp8 ? smem_bytes<128, true>(p) : smem_bytes<128, false>(p))
                           : (fp8 ? smem_bytes<64, true>(p) : smem_bytes<64, false>(p));
  return smem > 227 * 1024 ? BSATTN_ERR_UNSUPPORTED : BSATTN_OK;
}

bsattn_status launch_attention_mod(const bsattn_plan* p, const ModParams& mod, const void* q, const void* k,
                                   const float* qs, const float* ks, const __nv_bfloat16* v, const int32_t* idx,
                                   const int32_t* cnt, __nv_bfloat16* o, float* lse, void* ws, cudaStream_t st,
                                   AttnLayout lay) {
  Params prm;
  prm.g = make_geom(p);
  prm.mod = mod;
  prm.qs = qs;
  prm.ks = ks;
  prm.idx = idx;
  prm.cnt = cnt;
  prm.kmax = p->kmax;
  prm.o = o;
  prm.lse = lse;
  prm.scale = p->scale;
  prm.err = p->d_err;
  prm.umax = attention_steps(p);
  prm.parts = ws ? attention_parts(p) : 1;
  prm.part_o = (float*)ws;
  prm.part_ml = nullptr;
  if (prm.parts > 1)
    prm.part_ml = (float2*)(prm.part_o + (size_t)attention_items(p) * p->desc.heads * p->desc.B * prm.parts * 128 *
                                             p->desc.head_dim);
  prm.bm_words = (p->N + 31) / 32;
  prm.pair_axis = pair_axis_of(p);
  prm.stall = bsattn_testing_timeout_forced() ? 1 : 0;
  prm.wait_limit = prm.stall ? kTestWaitLimit : kWaitLimit;
  const int nd[3] = {p->nT, p->nH, p->nW};
  for (int a = 0; a < 3; ++a) prm.pdim[a] = a == prm.pair_axis ? (nd[a] + 1) / 2 : nd[a];
  const bool fp8 = p->desc.qk_fp8 != 0, d128 = p->desc.head_dim == 128;
  if (lay == AttnLayout::Natural)
    return d128 ? (fp8 ? run<128, true, true>(p, q, k, v, prm, st) : run<128, false, true>(p, q, k, v, prm, st))
                : (fp8 ? run<64, true, true>(p, q, k, v, prm, st) : run<64, false, true>(p, q, k, v, prm, st));
  return d128 ? (fp8 ? run<128, true, false>(p, q, k, v, prm, st) : run<128, false, false>(p, q, k, v, prm, st))
              : (fp8 ? run<64, true, false>(p, q, k, v, prm, st) : run<64, false, false>(p, q, k, v, prm, st));
}
