// Rotary positions on natural bf16 tensors, with the tile means of the result.
//
// Pair (x, y) of a token at position pos turns by pos * f (f per pair):
//   (x, y) -> m (x cos - y sin, x sin + y cos),
// the transpose with -sin. f / 2 pi is a 64-bit binary fraction, so that
// pos * f wraps modulo one turn by itself in integer arithmetic, exactly for
// every int32 position; its upper 32 bits go to fp32 sine and cosine. One
// rounding to bf16 at the end.
//
// Memory bound: every tensor is read and written once. Angles depend on a row
// only through its coordinate along the pair's axis: a CTA takes one 64-row
// chunk of a tile (with tile means: one tile, chunk by chunk) and a few heads,
// and fills a shared table [coordinate within the chunk's box][pair] of (cos,
// sin), 4 x 64 entries for a (4, 4, 4) chunk and at most 64 x 64. Explicit
// positions give one table row per token row. A thread owns the same features
// (its unit) of every rg-th row and of kHeads heads: the angles it reads from
// the table serve all of its heads, a pair's two features meet in one thread
// (in-place calls are safe), and its share of a tile's sum stays in
// registers until one exchange at the end, in a fixed order.
//
// Measured on one B200 (measured copy rate 6,528 GB/s): Q and K of the
// Wan-1.3B-shaped layer with means 59 us (291 MB, 0.75 of the copy rate; 3.7
// waves of CTAs), the Wan-14B-shaped gradient in the half layout 560-597 us
// (3.10 GB, 0.79-0.85), one token 3.8 us; at that size explicit positions take
// 670-740 us (a table row per token row) and half layouts with R no multiple
// of 8 980 us (features two by two). A thread per column of all heads, with
// angles from fp64, took 84 us, 669 us and 4-36 us; two heads a thread
// instead of four 743 us in the half layout (twice the table reads per
// feature, half the contiguous bytes).
#include "internal.h"

#include <math.h>

namespace {

constexpr int kThreads = 128;

struct RopeParams {
  Geom g;
  const __nv_bfloat16* x[2];
  __nv_bfloat16* y[2];
  float* pooled[2];
  const int32_t* pos;   // [B, L, 3] or null
  const int32_t* doc;   // [B, L] or null: tokens with a negative id become zeros and count in no mean
  int off[3];
  RopeTurns turn;
  float amp;
  float sign;           // -1: transposed rotation
  int hblk;             // head blocks per tensor
  int by_tile;          // a CTA takes a whole tile (tile means)
  int nu, rg;           // units per head, rows taken at once
};

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  __nv_bfloat162 h = *reinterpret_cast<__nv_bfloat162*>(&w);
  return __bfloat1622float2(h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// A unit, what a thread owns of a head:
//   kInterleaved: 8 neighbouring features (4 pairs)                  D / 8 units
//   kHalf8:       features [8u, 8u + 8) and [R + 8u, R + 8u + 8) (8
//                 pairs), R a multiple of 8; 8 passed features each   (D - R) / 8 units
//   kPair:        two features: a pair, or two passed ones; for half
//                 layouts whose R is not a multiple of 8, where a
//                 pair's features share no 16-byte alignment (2-byte
//                 accesses: 980 us where kHalf8 with R = 40 takes 560) D / 2 units
enum Mode { kInterleaved, kHalf8, kPair };
constexpr int kHeads = 4;  // heads of a CTA
constexpr uint32_t kHiddenRow = 1u << 31;

template <int MODE, bool POOL>
__global__ void __launch_bounds__(kThreads, POOL ? (MODE == kHalf8 ? 3 : 4) : (MODE == kHalf8 ? 5 : 7))
rope_kernel(const __grid_constant__ RopeParams P) {
  constexpr int NV = MODE == kPair ? 2 : MODE == kHalf8 ? 16 : 8;  // features of a unit
  constexpr int NP = NV / 2;
  constexpr int kRows = MODE == kHalf8 ? 1 : 2;                    // rows in flight: eight 16-byte loads a thread
  extern __shared__ float2 table[];   // [value][pair]
  __shared__ int rowtok[64];          // token of each row of the chunk, -1 for a padded slot
  __shared__ uint32_t rowval[64];     // its table rows along t, h, w; kHiddenRow set for a hidden token
  __shared__ int rowpos[3][64];       // explicit positions of each row
  __shared__ int seen;                // tokens in the sums
  __shared__ float part[POOL ? kThreads * kHeads * NV : 1];
  const Geom& g = P.g;
  const int D = g.D, R = P.turn.npairs, tid = threadIdx.x;
  // Head blocks vary fastest, so that CTAs that run together read whole token
  // rows (all heads of a token are contiguous).
  const int tensor = blockIdx.z, b = blockIdx.y, head0 = blockIdx.x % P.hblk * kHeads, item = blockIdx.x / P.hblk;
  const int j = P.by_tile ? item : item / g.nchunk;
  const int ch0 = P.by_tile ? 0 : item % g.nchunk, ch1 = P.by_tile ? g.nchunk : ch0 + 1;
  const __nv_bfloat16* x = P.x[tensor];
  __nv_bfloat16* y = P.y[tensor];
  const int bt = j / (g.nH * g.nW), bh = (j / g.nW) % g.nH, bw = j % g.nW;
  const int u = tid % P.nu, grp = tid / P.nu;
  const bool active = grp < P.rg;
  // First feature of each part, first pair (-1: passed unchanged).
  int fa, fb = 0, p0;
  if (MODE == kInterleaved) {
    fa = 8 * u;
    p0 = 4 * u < R ? 4 * u : -1;
  } else if (MODE == kHalf8) {
    const bool turned = 8 * u < R;
    fa = turned ? 8 * u : R + 8 * u;
    fb = R + 8 * u;
    p0 = turned ? 8 * u : -1;
  } else {
    const bool turned = u < R;
    fa = turned ? u : 2 * u;
    fb = turned ? u + R : 2 * u + 1;
    p0 = turned ? u : -1;
  }
  const int np = p0 < 0 ? 0 : min(NP, R - p0);  // turned pairs among the thread's (interleaved: a unit may end mid-way)
  // Shift that takes a pair's axis out of rowval.
  uint32_t shift[NP];
#pragma unroll
  for (int e = 0; e < NP; ++e) shift[e] = p0 + e < P.turn.split[0] ? 0 : p0 + e < P.turn.split[1] ? 8 : 16;
  const size_t row_el = (size_t)g.Hh * D;
  const size_t base = (size_t)b * g.L * row_el + (size_t)head0 * D;
  const int nh = min(kHeads, g.Hh - head0);
  float acc[POOL ? kHeads : 1][POOL ? NV : 1];
  if (POOL) {
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
#pragma unroll
      for (int e = 0; e < NV; ++e) acc[h][e] = 0.f;
    if (tid == 0) seen = 0;
  }

  for (int ch = ch0; ch < ch1; ++ch) {
    const ChunkOrigin o = chunk_origin(g, ch);
    const int t0 = bt * g.tt + o.dt, h0 = bh * g.th + o.dh, w0 = bw * g.tw + o.dw;
    if (t0 >= g.T || h0 >= g.H || w0 >= g.W) continue;  // padding only (uniform over the CTA)
    __syncthreads();  // the previous chunk's table and rows are read
    if (tid < 64) {
      const uint32_t cc = chunk_row_code(g, tid);
      const int t = t0 + (int)(cc & 0xffu), h = h0 + (int)((cc >> 8) & 0xffu), w = w0 + (int)((cc >> 16) & 0xffu);
      const bool real = tid < g.cr && t < g.T && h < g.H && w < g.W;
      const int n = real ? (t * g.H + h) * g.W + w : -1;
      uint32_t val = P.pos ? (uint32_t)tid * 0x10101u : cc;
      if (P.doc && real && P.doc[(size_t)b * g.L + n] < 0) val |= kHiddenRow;
      rowtok[tid] = n;
      rowval[tid] = val;
      if (POOL) {
        const uint32_t in = __ballot_sync(0xffffffffu, real && !(val & kHiddenRow));
        if (tid % 32 == 0) atomicAdd(&seen, __popc(in));
      }
    }
    if (P.pos) {
      __syncthreads();
      for (int e = tid; e < 3 * g.cr; e += kThreads) {
        const int a = e / g.cr, r = e % g.cr;
        rowpos[a][r] = rowtok[r] >= 0 ? P.pos[((size_t)b * g.L + rowtok[r]) * 3 + a] : 0;
      }
      __syncthreads();
    }
    // The table: thread tid takes pair tid % 64 of every second value.
    const int p = tid % 64;
    if (p < R) {
      const int a = p < P.turn.split[0] ? 0 : p < P.turn.split[1] ? 1 : 2;
      const int vals = P.pos ? g.cr : a == 0 ? g.ct : a == 1 ? g.ch : g.cw;
      const unsigned long long f = P.turn.turns[p];
      const long long at0 = (long long)P.off[a] + (a == 0 ? t0 : a == 1 ? h0 : w0);
      for (int v = tid / 64; v < vals; v += kThreads / 64) {
        const long long at = P.pos ? rowpos[a][v] : at0 + v;
        const int hi = (int)(((unsigned long long)at * f) >> 32);  // the turn in [-1/2, 1/2), in 2^-32
        // fp32 holds 24 of the 32 bits; the rest turns (cos, sin) to first order.
        const float top = (float)hi;
        const float rest = (float)(int)((long long)hi - (long long)top) * (float)(M_PI * 0x1p-31);
        float s, c;
        sincospif(top * 0x1p-31f, &s, &c);
        const float s1 = fmaf(c, rest, s), c1 = fmaf(-s, rest, c);
        table[v * R + p] = make_float2(c1 * P.amp, s1 * P.amp * P.sign);
      }
    }
    __syncthreads();
    if (!active) continue;
#pragma unroll 1
    for (int r0 = grp; r0 < g.cr; r0 += kRows * P.rg) {
      uint4 va[kRows][kHeads], vb[MODE == kHalf8 ? kRows : 1][kHeads];
      float sa[MODE == kPair ? kRows : 1][kHeads], sb[MODE == kPair ? kRows : 1][kHeads];
      int tok[kRows];
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int r = r0 + i * P.rg;
        tok[i] = r < g.cr ? rowtok[r] : -1;
        if (tok[i] < 0) continue;
        const __nv_bfloat16* src = x + base + (size_t)tok[i] * row_el;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          if (h >= nh) continue;
          if (MODE == kPair) {
            sa[i][h] = __bfloat162float(src[h * D + fa]);
            sb[i][h] = __bfloat162float(src[h * D + fb]);
          } else {
            va[i][h] = *reinterpret_cast<const uint4*>(src + h * D + fa);
            if (MODE == kHalf8 && p0 >= 0) vb[i][h] = *reinterpret_cast<const uint4*>(src + h * D + fb);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (tok[i] < 0) continue;
        const uint32_t val = rowval[r0 + i * P.rg];
        float2 cs[NP];
#pragma unroll
        for (int e = 0; e < NP; ++e)
          cs[e] = e < np ? table[((val >> shift[e]) & 0xffu) * R + p0 + e] : make_float2(1.f, 0.f);
        __nv_bfloat16* dst = y + base + (size_t)tok[i] * row_el;
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          if (h >= nh) continue;
          if (val & kHiddenRow) {  // zeros, whatever the row holds
            if (MODE == kPair) {
              sa[i][h] = sb[i][h] = 0.f;
            } else {
              va[i][h] = make_uint4(0, 0, 0, 0);
              if (MODE == kHalf8) vb[i][h] = make_uint4(0, 0, 0, 0);
            }
          }
          float f[NV];
          if (MODE == kPair) {
            f[0] = np ? sa[i][h] * cs[0].x - sb[i][h] * cs[0].y : sa[i][h];
            f[1] = np ? sa[i][h] * cs[0].y + sb[i][h] * cs[0].x : sb[i][h];
            dst[h * D + fa] = __float2bfloat16_rn(f[0]);
            dst[h * D + fb] = __float2bfloat16_rn(f[1]);
          } else if (MODE == kInterleaved) {
            const uint32_t w[4] = {va[i][h].x, va[i][h].y, va[i][h].z, va[i][h].w};
            uint32_t q[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 a = unpack2(w[e]);
              f[2 * e] = a.x;
              f[2 * e + 1] = a.y;
              if (e < np) {  // not by cos 1, sin 0: 0 * inf
                f[2 * e] = a.x * cs[e].x - a.y * cs[e].y;
                f[2 * e + 1] = a.x * cs[e].y + a.y * cs[e].x;
              }
              q[e] = pack2(f[2 * e], f[2 * e + 1]);
            }
            *reinterpret_cast<uint4*>(dst + h * D + fa) = make_uint4(q[0], q[1], q[2], q[3]);
          } else {
            const uint32_t w[4] = {va[i][h].x, va[i][h].y, va[i][h].z, va[i][h].w};
            if (p0 < 0) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 a = unpack2(w[e]);
                f[2 * e] = a.x;
                f[2 * e + 1] = a.y;
              }
              *reinterpret_cast<uint4*>(dst + h * D + fa) = va[i][h];
            } else {
              const uint32_t z[4] = {vb[i][h].x, vb[i][h].y, vb[i][h].z, vb[i][h].w};
              uint32_t q[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 a = unpack2(w[e]), c = unpack2(z[e]);
                const float2 k0 = cs[(2 * e) % NP], k1 = cs[(2 * e + 1) % NP];
                f[2 * e] = a.x * k0.x - c.x * k0.y;
                f[2 * e + 1] = a.y * k1.x - c.y * k1.y;
                f[(8 + 2 * e) % NV] = a.x * k0.y + c.x * k0.x;
                f[(9 + 2 * e) % NV] = a.y * k1.y + c.y * k1.x;
                q[e] = pack2(f[2 * e], f[2 * e + 1]);
                q[4 + e] = pack2(f[(8 + 2 * e) % NV], f[(9 + 2 * e) % NV]);
              }
              *reinterpret_cast<uint4*>(dst + h * D + fa) = make_uint4(q[0], q[1], q[2], q[3]);
              *reinterpret_cast<uint4*>(dst + h * D + fb) = make_uint4(q[4], q[5], q[6], q[7]);
            }
          }
          if (POOL) {
#pragma unroll
            for (int e = 0; e < NV; ++e)
              if (MODE != kHalf8 || e < 8 || p0 >= 0) acc[h][e] += f[e];
          }
        }
      }
    }
  }
  if (POOL) {
    // part[group][head][value][unit]: sums over the groups in order.
    if (active) {
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
#pragma unroll
        for (int e = 0; e < NV; ++e) part[((grp * kHeads + h) * NV + e) * P.nu + u] = acc[h][e];
    }
    __syncthreads();
    const float n = (float)max(seen, 1);
    const int per = NV * P.nu;
    for (int o = tid; o < nh * per; o += kThreads) {
      const int h = o / per, e = o % per / P.nu, v = o % P.nu;
      float s = 0.f;
      for (int k = 0; k < P.rg; ++k) s += part[(k * kHeads + h) * per + o % per];
      int feat;
      if (MODE == kInterleaved) {
        feat = 8 * v + e;
      } else if (MODE == kHalf8) {
        if (8 * v >= R && e >= 8) continue;  // passed units have eight features
        feat = 8 * v < R ? 8 * v + e + (e >= 8 ? R - 8 : 0) : R + 8 * v + e;
      } else {
        feat = v < R ? v + e * R : 2 * v + e;
      }
      P.pooled[tensor][(((size_t)b * g.Hh + head0 + h) * g.N + j) * D + feat] = __fdiv_rn(s, n);
    }
  }
}

template <int MODE>
bsattn_status run(RopeParams& prm, int ntensor, bool pool, cudaStream_t st) {
  const Geom& g = prm.g;
  prm.nu = MODE == kInterleaved ? g.D / 8 : MODE == kHalf8 ? (g.D - prm.turn.npairs) / 8 : g.D / 2;
  prm.rg = kThreads / prm.nu;  // nu <= 64
  prm.hblk = (g.Hh + kHeads - 1) / kHeads;
  prm.by_tile = pool ? 1 : 0;
  const long long gx = (pool ? g.N : (long long)g.N * g.nchunk) * prm.hblk;
  if (g.B > 65535 || gx > 0x7fffffffLL) return BSATTN_ERR_UNSUPPORTED;
  const int box = g.ct > g.ch ? (g.ct > g.cw ? g.ct : g.cw) : (g.ch > g.cw ? g.ch : g.cw);
  const size_t smem = (size_t)(prm.pos ? g.cr : box) * prm.turn.npairs * sizeof(float2);  // <= 32 KB
  if (pool && smem > 14 * 1024) {  // with the exchange buffer (33 KB at most) above the default 48 KB
    if (cudaFuncSetAttribute(rope_kernel<MODE, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, 32 * 1024) != cudaSuccess)
      return BSATTN_ERR_CUDA;
  }
  dim3 grid((unsigned)gx, g.B, ntensor);
  if (pool)
    rope_kernel<MODE, true><<<grid, kThreads, smem, st>>>(prm);
  else
    rope_kernel<MODE, false><<<grid, kThreads, smem, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace

// x modulo 1 (x >= 0), in units of 2^-64.
static unsigned long long fraction64(double x) {
  x -= floor(x);
  const double hi = floor(x * 0x1p32);
  const double lo = floor((x * 0x1p32 - hi) * 0x1p32);
  return ((unsigned long long)hi << 32) | (unsigned long long)lo;
}

bsattn_status check_rope(const bsattn_plan* p, const bsattn_rope* r, RopeTurns* out) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (r->layout != BSATTN_ROPE_INTERLEAVED && r->layout != BSATTN_ROPE_HALF) return BSATTN_ERR_INVALID_ARG;
  if (r->scaling < BSATTN_ROPE_SCALE_NONE || r->scaling > BSATTN_ROPE_SCALE_BY_PARTS) return BSATTN_ERR_INVALID_ARG;
  long long sum = 0;
  for (int a = 0; a < 3; ++a) {
    if (r->dim[a] < 0 || r->dim[a] % 2 != 0) return BSATTN_ERR_INVALID_ARG;
    sum += r->dim[a];
  }
  if (sum < 2 || sum > p->desc.head_dim) return BSATTN_ERR_INVALID_ARG;
  if (!(r->base > 1.0) || !isfinite(r->base) || !isfinite((float)r->amplitude)) return BSATTN_ERR_INVALID_ARG;
  if (r->scaling != BSATTN_ROPE_SCALE_NONE)
    for (int a = 0; a < 3; ++a)
      if (!(r->factor[a] > 0.0) || !isfinite(r->factor[a])) return BSATTN_ERR_INVALID_ARG;
  if (r->scaling == BSATTN_ROPE_SCALE_BY_PARTS) {
    for (int a = 0; a < 3; ++a)
      if (!(r->original[a] > 0.0) || !isfinite(r->original[a])) return BSATTN_ERR_INVALID_ARG;
    if (!(r->slow >= 0.0) || !(r->fast > r->slow) || !isfinite(r->fast)) return BSATTN_ERR_INVALID_ARG;
  }
  if (r->pos && !aligned16(r->pos)) return BSATTN_ERR_INVALID_ARG;
  int np = 0;
  for (int a = 0; a < 3; ++a) {
    const int d = r->dim[a];
    if (a > 0) out->split[a - 1] = np;
    const double s = r->factor[a];
    double base = r->base;
    if (r->scaling == BSATTN_ROPE_SCALE_NTK && d > 2) base *= pow(s, (double)d / (d - 2));
    // Frequencies of 53 bits: up to 1 they are within 4e-7 of a radian at position
    // 2^31 (3.1e-7 is the most that bases of 100 to 10^6 give unscaled).
    const double per_pair = d > 0 ? -2.0 * log2(base) / d : 0.0;
    for (int i = 0; i < d / 2; ++i) {
      double f = exp2(per_pair * i);
      if (r->scaling == BSATTN_ROPE_SCALE_LINEAR) f /= s;
      if (r->scaling == BSATTN_ROPE_SCALE_BY_PARTS) {
        double keep = (r->original[a] * f / kTwoPi - r->slow) / (r->fast - r->slow);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        f *= keep + (1.0 - keep) / s;
      }
      const double turn = f / kTwoPi;
      if (!isfinite(turn)) return BSATTN_ERR_INVALID_ARG;  // extreme factors
      out->turns[np++] = fraction64(turn);
    }
  }
  out->npairs = np;
  return BSATTN_OK;
}

bsattn_status launch_rope(const bsattn_plan* p, const bsattn_rope* r, const RopeTurns& turns, const __nv_bfloat16* x0,
                          __nv_bfloat16* y0, const __nv_bfloat16* x1, __nv_bfloat16* y1, float* pooled0, float* pooled1,
                          bool transpose, const int32_t* doc, cudaStream_t st) {
  RopeParams prm{};
  prm.g = make_geom(p);
  prm.doc = doc;
  if (r) {
    prm.pos = r->pos;
    prm.amp = r->amplitude == 0.0 ? 1.f : (float)r->amplitude;
    prm.sign = transpose ? -1.f : 1.f;
    for (int a = 0; a < 3; ++a) prm.off[a] = r->offset[a];
    prm.turn = turns;
  }
  const int np = prm.turn.npairs;
  const bool interleaved = !r || r->layout == BSATTN_ROPE_INTERLEAVED;
  // One launch when both tensors want the same outputs (the usual call), else one each.
  const bool one = x1 && (pooled0 != nullptr) == (pooled1 != nullptr);
  for (int l = 0; l < (x1 && !one ? 2 : 1); ++l) {
    prm.x[0] = l ? x1 : x0; prm.y[0] = l ? y1 : y0; prm.pooled[0] = l ? pooled1 : pooled0;
    prm.x[1] = x1; prm.y[1] = y1; prm.pooled[1] = pooled1;
    const int nt = one ? 2 : 1;
    const bool pool = prm.pooled[0] != nullptr;
    const bsattn_status s = interleaved ? run<kInterleaved>(prm, nt, pool, st)
                            : np % 8 == 0 ? run<kHalf8>(prm, nt, pool, st)
                                          : run<kPair>(prm, nt, pool, st);
    if (s) return s;
  }
  return BSATTN_OK;
}

extern "C" bsattn_status attn_rope(const bsattn_plan* p, const bsattn_rope* r, const void* x0, void* y0, const void* x1,
                                   void* y1, float* pooled0, float* pooled1, int transpose, void* stream) {
  auto ok = [](const void* x) { return x != nullptr && aligned16(x); };
  if (!p || !r || !ok(x0) || !ok(y0) || (x1 == nullptr) != (y1 == nullptr) || (x1 && (!ok(x1) || !ok(y1))))
    return BSATTN_ERR_INVALID_ARG;
  if ((pooled0 && !aligned16(pooled0)) || (pooled1 && (!aligned16(pooled1) || !x1))) return BSATTN_ERR_INVALID_ARG;
  if (transpose != 0 && transpose != 1) return BSATTN_ERR_INVALID_ARG;
  RopeTurns turns{};
  bsattn_status s = check_rope(p, r, &turns);
  if (s) return s;
  DeviceGuard dev(p->device);
  if (dev.status) return dev.status;
  return launch_rope(p, r, turns, (const __nv_bfloat16*)x0, (__nv_bfloat16*)y0, (const __nv_bfloat16*)x1, (__nv_bfloat16*)y1,
                     pooled0, pooled1, transpose != 0, nullptr, (cudaStream_t)stream);
}
