// Rotary positions on natural bf16 tensors, with the tile means of the result.
//
// Pair (x, y) of a token at position pos turns by pos * f (f per pair):
//   (x, y) -> m (x cos - y sin, x sin + y cos),
// the transpose with -sin. The angle is formed in turns in fp64 (pos * f / 2pi
// minus its nearest integer), so that far positions keep fp32's accuracy in
// sine and cosine; one rounding to bf16 at the end.
//
// Memory bound: every tensor is read and written once. A CTA takes one 64-row
// chunk of a tile (with tile means: one tile, chunk by chunk) and a block of
// columns of the token rows, thread c owning the same features of every row,
// so that rows are read coalesced, a pair's two features meet in one thread
// (in-place calls are safe) and the tile's sum needs no exchange. Angles
// depend on a row only through its coordinate along the pair's axis: the CTA
// fills a shared table [coordinate within the chunk's box][pair] of (cos, sin)
// once, at most 64 x 64 entries (12 x 21 for a (4, 4, 4) chunk), instead of
// one sine per token, pair and head. Explicit positions give one table row
// per token row.
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
  int npairs;           // R
  int split[2];         // first pair of the h and w axes
  float amp;
  float sign;           // -1: transposed rotation
  int ncblk;            // column blocks per tensor
  int by_tile;          // a CTA takes a whole tile (tile means)
  double turns[64];     // f / (2 pi) of each pair
};

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  __nv_bfloat162 h = *reinterpret_cast<__nv_bfloat162*>(&w);
  return __bfloat1622float2(h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// What a thread owns of every token row. Units are numbered over a head's
// features, then heads:
//   kInterleaved: 8 neighbouring features (4 pairs)                  D / 8 units
//   kHalf8:       features [8u, 8u + 8) and [R + 8u, R + 8u + 8) (8
//                 pairs), R a multiple of 8; 8 passed features each   (D - R) / 8 units
//   kPair:        two features: a pair, or two passed ones; for half
//                 layouts whose R is not a multiple of 8 (2-byte
//                 accesses: 4x the load instructions of kHalf8)       D / 2 units
constexpr uint32_t kHiddenRow = 1u << 31;
enum Mode { kInterleaved, kHalf8, kPair };

template <int MODE, bool POOL>
__global__ void __launch_bounds__(kThreads)
rope_kernel(const __grid_constant__ RopeParams P) {
  constexpr int NV = MODE == kPair ? 2 : MODE == kHalf8 ? 16 : 8;  // features a thread owns
  constexpr int NP = NV / 2;
  constexpr int kRowsInFlight = MODE == kHalf8 ? 4 : 8;  // eight 16-byte loads in flight a thread
  extern __shared__ float2 table[];   // [value][pair]
  __shared__ int rowtok[64];          // token of each row of the chunk, -1 for a padded slot
  __shared__ uint32_t rowval[64];     // its table rows along t, h, w; kHiddenRow set for a hidden token
  const Geom& g = P.g;
  const int D = g.D, R = P.npairs;
  const int tensor = blockIdx.z / P.ncblk, cblk = blockIdx.z % P.ncblk, b = blockIdx.y;
  const int j = P.by_tile ? blockIdx.x : blockIdx.x / g.nchunk;
  const int ch0 = P.by_tile ? 0 : blockIdx.x % g.nchunk, ch1 = P.by_tile ? g.nchunk : ch0 + 1;
  const __nv_bfloat16* x = P.x[tensor];
  __nv_bfloat16* y = P.y[tensor];
  const int bt = j / (g.nH * g.nW), bh = (j / g.nW) % g.nH, bw = j % g.nW;
  const int nu = MODE == kInterleaved ? D / 8 : MODE == kHalf8 ? (D - R) / 8 : D / 2;
  const int unit = cblk * kThreads + threadIdx.x;
  const int head = unit / nu, u = unit % nu;
  const bool active = head < g.Hh;
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
  const size_t row_el = (size_t)g.Hh * D;
  const size_t base = (size_t)b * g.L * row_el + (size_t)head * D;
  float acc[POOL ? NV : 1];
  int seen = 0;  // tokens in the sums
  if (POOL) {
#pragma unroll
    for (int e = 0; e < NV; ++e) acc[e] = 0.f;
  }

  for (int ch = ch0; ch < ch1; ++ch) {
    const ChunkOrigin o = chunk_origin(g, ch);
    const int t0 = bt * g.tt + o.dt, h0 = bh * g.th + o.dh, w0 = bw * g.tw + o.dw;
    if (t0 >= g.T || h0 >= g.H || w0 >= g.W) continue;  // padding only (uniform over the CTA)
    __syncthreads();  // the previous chunk's table and rows are read
    if (threadIdx.x < 64) {
      const uint32_t cc = chunk_row_code(g, threadIdx.x);
      const int t = t0 + (int)(cc & 0xffu), h = h0 + (int)((cc >> 8) & 0xffu), w = w0 + (int)((cc >> 16) & 0xffu);
      const bool real = threadIdx.x < g.cr && t < g.T && h < g.H && w < g.W;
      rowtok[threadIdx.x] = real ? (t * g.H + h) * g.W + w : -1;
      uint32_t val = P.pos ? (uint32_t)threadIdx.x * 0x10101u : cc;
      if (P.doc && real && P.doc[(size_t)b * g.L + (t * g.H + h) * g.W + w] < 0) val |= kHiddenRow;
      rowval[threadIdx.x] = val;
    }
    __syncthreads();
    const int vals = P.pos ? 64 : max(g.ct, max(g.ch, g.cw));
    for (int e = threadIdx.x; e < vals * R; e += kThreads) {
      const int v = e / R, p = e % R;
      const int a = p < P.split[0] ? 0 : p < P.split[1] ? 1 : 2;
      double at;
      if (P.pos) {
        const int n = rowtok[v];
        if (n < 0) continue;
        at = (double)P.pos[((size_t)b * g.L + n) * 3 + a];
      } else {
        if (v >= (a == 0 ? g.ct : a == 1 ? g.ch : g.cw)) continue;
        at = (double)P.off[a] + (double)((a == 0 ? t0 : a == 1 ? h0 : w0) + v);
      }
      double turn = at * P.turns[p];
      turn -= rint(turn);
      float s, c;
      sincospif((float)(2.0 * turn), &s, &c);
      table[v * R + p] = make_float2(c * P.amp, s * P.amp * P.sign);
    }
    __syncthreads();
    if (!active) continue;
#pragma unroll 1
    for (int r0 = 0; r0 < g.cr; r0 += kRowsInFlight) {
      uint4 va[kRowsInFlight], vb[MODE == kHalf8 ? kRowsInFlight : 1];
      float sa[MODE == kPair ? kRowsInFlight : 1], sb[MODE == kPair ? kRowsInFlight : 1];
#pragma unroll
      for (int i = 0; i < kRowsInFlight; ++i) {
        const int n = r0 + i < g.cr ? rowtok[r0 + i] : -1;
        if (n < 0) continue;
        const __nv_bfloat16* src = x + base + (size_t)n * row_el;
        if (MODE == kPair) {
          sa[i] = __bfloat162float(src[fa]);
          sb[i] = __bfloat162float(src[fb]);
        } else {
          va[i] = *reinterpret_cast<const uint4*>(src + fa);
          if (MODE == kHalf8 && p0 >= 0) vb[i] = *reinterpret_cast<const uint4*>(src + fb);
        }
      }
#pragma unroll
      for (int i = 0; i < kRowsInFlight; ++i) {
        const int n = r0 + i < g.cr ? rowtok[r0 + i] : -1;
        if (n < 0) continue;
        const uint32_t val = rowval[r0 + i];
        if (val & kHiddenRow) {  // zeros, whatever the row holds
          if (MODE == kPair) {
            sa[i] = sb[i] = 0.f;
          } else {
            va[i] = make_uint4(0, 0, 0, 0);
            if (MODE == kHalf8) vb[i] = make_uint4(0, 0, 0, 0);
          }
        } else {
          ++seen;
        }
        auto turn = [&](int p) -> float2 {
          const uint32_t v = p < P.split[0] ? val & 0xffu : p < P.split[1] ? (val >> 8) & 0xffu : (val >> 16) & 0xffu;
          return table[v * R + p];
        };
        __nv_bfloat16* dst = y + base + (size_t)n * row_el;
        float f[NV];
        if (MODE == kPair) {
          f[0] = sa[i];
          f[1] = sb[i];
          if (np) {
            const float2 cs = turn(p0);
            f[0] = sa[i] * cs.x - sb[i] * cs.y;
            f[1] = sa[i] * cs.y + sb[i] * cs.x;
          }
          dst[fa] = __float2bfloat16_rn(f[0]);
          dst[fb] = __float2bfloat16_rn(f[1]);
        } else if (MODE == kInterleaved) {
          const uint32_t w[4] = {va[i].x, va[i].y, va[i].z, va[i].w};
          uint32_t q[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = unpack2(w[e]);
            f[2 * e] = a.x;
            f[2 * e + 1] = a.y;
            if (e < np) {
              const float2 cs = turn(p0 + e);
              f[2 * e] = a.x * cs.x - a.y * cs.y;
              f[2 * e + 1] = a.x * cs.y + a.y * cs.x;
            }
            q[e] = pack2(f[2 * e], f[2 * e + 1]);
          }
          *reinterpret_cast<uint4*>(dst + fa) = make_uint4(q[0], q[1], q[2], q[3]);
        } else {
          const uint32_t w[4] = {va[i].x, va[i].y, va[i].z, va[i].w};
          if (p0 < 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 a = unpack2(w[e]);
              f[2 * e] = a.x;
              f[2 * e + 1] = a.y;
            }
            *reinterpret_cast<uint4*>(dst + fa) = va[i];
          } else {
            const uint32_t z[4] = {vb[i].x, vb[i].y, vb[i].z, vb[i].w};
            uint32_t q[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 a = unpack2(w[e]), c = unpack2(z[e]);
              const float2 k0 = turn(p0 + 2 * e), k1 = turn(p0 + 2 * e + 1);
              f[2 * e] = a.x * k0.x - c.x * k0.y;
              f[2 * e + 1] = a.y * k1.x - c.y * k1.y;
              f[(8 + 2 * e) % NV] = a.x * k0.y + c.x * k0.x;
              f[(9 + 2 * e) % NV] = a.y * k1.y + c.y * k1.x;
              q[e] = pack2(f[2 * e], f[2 * e + 1]);
              q[4 + e] = pack2(f[(8 + 2 * e) % NV], f[(9 + 2 * e) % NV]);
            }
            *reinterpret_cast<uint4*>(dst + fa) = make_uint4(q[0], q[1], q[2], q[3]);
            *reinterpret_cast<uint4*>(dst + fb) = make_uint4(q[4], q[5], q[6], q[7]);
          }
        }
        if (POOL) {
#pragma unroll
          for (int e = 0; e < NV; ++e)
            if (MODE != kHalf8 || e < 8 || p0 >= 0) acc[e] += f[e];
        }
      }
    }
  }
  if (POOL && active) {
    const float n = (float)max(seen, 1);
    float* out = P.pooled[tensor] + (((size_t)b * g.Hh + head) * g.N + j) * D;
    if (MODE == kPair) {
      out[fa] = __fdiv_rn(acc[0], n);
      out[fb] = __fdiv_rn(acc[1 % NV], n);
    } else {
#pragma unroll
      for (int q = 0; q < NV / 4; ++q) {
        if (q >= 2 && p0 < 0) break;
        *reinterpret_cast<float4*>(out + (q < 2 ? fa : fb) + 4 * (q & 1)) =
            make_float4(__fdiv_rn(acc[4 * q], n), __fdiv_rn(acc[4 * q + 1], n), __fdiv_rn(acc[4 * q + 2], n),
                        __fdiv_rn(acc[4 * q + 3], n));
      }
    }
  }
}

template <int MODE>
bsattn_status run(RopeParams& prm, int ntensor, bool pool, cudaStream_t st) {
  const Geom& g = prm.g;
  const int nu = MODE == kInterleaved ? g.D / 8 : MODE == kHalf8 ? (g.D - prm.npairs) / 8 : g.D / 2;
  prm.ncblk = (g.Hh * nu + kThreads - 1) / kThreads;
  prm.by_tile = pool ? 1 : 0;
  const long long gx = pool ? g.N : (long long)g.N * g.nchunk;
  if (g.B > 65535 || prm.ncblk * ntensor > 65535 || gx > 0x7fffffffLL) return BSATTN_ERR_UNSUPPORTED;
  const int box = g.ct > g.ch ? (g.ct > g.cw ? g.ct : g.cw) : (g.ch > g.cw ? g.ch : g.cw);
  const size_t smem = (size_t)(prm.pos ? 64 : box) * prm.npairs * sizeof(float2);  // <= 32 KB
  dim3 grid((unsigned)gx, g.B, prm.ncblk * ntensor);
  if (pool)
    rope_kernel<MODE, true><<<grid, kThreads, smem, st>>>(prm);
  else
    rope_kernel<MODE, false><<<grid, kThreads, smem, st>>>(prm);
  return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace

bsattn_status check_rope(const bsattn_plan* p, const bsattn_rope* r) {
  if (r->layout != BSATTN_ROPE_INTERLEAVED && r->layout != BSATTN_ROPE_HALF) return BSATTN_ERR_INVALID_ARG;
  if (r->scaling < BSATTN_ROPE_SCALE_NONE || r->scaling > BSATTN_ROPE_SCALE_BY_PARTS) return BSATTN_ERR_INVALID_ARG;
  long long sum = 0;
  for (int a = 0; a < 3; ++a) {
    if (r->dim[a] < 0 || r->dim[a] % 2 != 0) return BSATTN_ERR_INVALID_ARG;
    sum += r->dim[a];
  }
  if (sum < 2 || sum > p->desc.head_dim) return BSATTN_ERR_INVALID_ARG;
  if (!(r->base > 1.0) || !isfinite(r->base) || !isfinite(r->amplitude)) return BSATTN_ERR_INVALID_ARG;
  if (r->scaling != BSATTN_ROPE_SCALE_NONE)
    for (int a = 0; a < 3; ++a)
      if (!(r->factor[a] > 0.0) || !isfinite(r->factor[a])) return BSATTN_ERR_INVALID_ARG;
  if (r->scaling == BSATTN_ROPE_SCALE_BY_PARTS) {
    for (int a = 0; a < 3; ++a)
      if (!(r->original[a] > 0.0) || !isfinite(r->original[a])) return BSATTN_ERR_INVALID_ARG;
    if (!(r->slow >= 0.0) || !(r->fast > r->slow) || !isfinite(r->fast)) return BSATTN_ERR_INVALID_ARG;
  }
  if (r->pos && !aligned16(r->pos)) return BSATTN_ERR_INVALID_ARG;
  return BSATTN_OK;
}

bsattn_status launch_rope(const bsattn_plan* p, const bsattn_rope* r, const __nv_bfloat16* x0, __nv_bfloat16* y0,
                          const __nv_bfloat16* x1, __nv_bfloat16* y1, float* pooled0, float* pooled1, bool transpose,
                          const int32_t* doc, cudaStream_t st) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  RopeParams prm{};
  prm.g = make_geom(p);
  prm.doc = doc;
  int np = 0;
  if (r) {
    prm.pos = r->pos;
    prm.amp = r->amplitude == 0.0 ? 1.f : (float)r->amplitude;
    prm.sign = transpose ? -1.f : 1.f;
    for (int a = 0; a < 3; ++a) {
      prm.off[a] = r->offset[a];
      const int d = r->dim[a];
      if (a > 0) prm.split[a - 1] = np;
      const double s = r->factor[a];
      double base = r->base;
      if (r->scaling == BSATTN_ROPE_SCALE_NTK && d > 2) base *= pow(s, (double)d / (d - 2));
      for (int i = 0; i < d / 2; ++i) {
        double f = pow(base, -2.0 * i / d);
        if (r->scaling == BSATTN_ROPE_SCALE_LINEAR) f /= s;
        if (r->scaling == BSATTN_ROPE_SCALE_BY_PARTS) {
          double keep = (r->original[a] * f / kTwoPi - r->slow) / (r->fast - r->slow);
          keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
          f *= keep + (1.0 - keep) / s;
        }
        prm.turns[np++] = f / kTwoPi;
      }
    }
  }
  prm.npairs = np;
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
  bsattn_status s = check_rope(p, r);
  if (s) return s;
  DeviceGuard dev(p->device);
  if (dev.status) return dev.status;
  return launch_rope(p, r, (const __nv_bfloat16*)x0, (__nv_bfloat16*)y0, (const __nv_bfloat16*)x1, (__nv_bfloat16*)y1,
                     pooled0, pooled1, transpose != 0, nullptr, (cudaStream_t)stream);
}
