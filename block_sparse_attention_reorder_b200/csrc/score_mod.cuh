// Score rules inside the attention kernels: capping by tanh, distance bias,
// causal, prefix and document masks (the definitions stand at
// bsattn_score_mod in bsattn.h). Shared by the forward and the backward.
#pragma once

#include <math.h>

#include "internal.h"
#include "tc_common.cuh"

namespace mod {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHiddenDoc = -2;  // a query id that equals no key's

// tanh for |u| <= kSmall: u + u^3 P(u^2), P of degree 4 fitted to
// (tanh(u) / u - 1) / u^2 for the least maximum relative error of tanh
// (Lawson's iteratively reweighted least squares): 3.2e-8, 1.0e-7 evaluated
// in fp32. Eight FMA-pipe operations, four on packed pairs.
constexpr float kSmall = 0.75f;
__device__ __forceinline__ float2 tanh_small2(float2 u) {
  const float2 v = __fmul2_rn(u, u);
  float2 p = __ffma2_rn(make_float2(-0.004769490100443363f, -0.004769490100443363f), v,
                        make_float2(0.019664913415908813f, 0.019664913415908813f));
  p = __ffma2_rn(p, v, make_float2(-0.0533902570605278f, -0.0533902570605278f));
  p = __ffma2_rn(p, v, make_float2(0.13326521217823029f, 0.13326521217823029f));
  p = __ffma2_rn(p, v, make_float2(-0.3333306908607483f, -0.3333306908607483f));
  return __ffma2_rn(__fmul2_rn(v, u), p, u);
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh for any u: 1 - 2 / (e^(2u) + 1), two SFU operations; its absolute
// error is about 2e-7, so it stands in where |u| is not small.
__device__ __forceinline__ float tanh_any(float u) {
  return fmaf(-2.f, rcp(tc::ex2(u * (2.f * kLog2e)) + 1.f), 1.f);
}

// Replaces raw scores s[] by u = tanh(k s) (k = scale / cap). The polynomial
// serves a whole warp's values when all are small, which usual scores under a
// usual cap are; else the SFU form does, and the polynomial where |u| is
// small, so that a value's tanh does not depend on its neighbours.
template <int N>
__device__ __forceinline__ void tanh_scores(uint32_t* s, float k) {
  float mx = 0.f;
#pragma unroll
  for (int q = 0; q < N; ++q) mx = fmaxf(mx, fabsf(__uint_as_float(s[q])));
  const bool small = mx * fabsf(k) <= kSmall;
  const float2 k2 = make_float2(k, k);
  if (__all_sync(0xffffffffu, small)) {
#pragma unroll
    for (int q = 0; q < N; q += 2) {
      const float2 t = tanh_small2(__fmul2_rn(make_float2(__uint_as_float(s[q]), __uint_as_float(s[q + 1])), k2));
      s[q] = __float_as_uint(t.x);
      s[q + 1] = __float_as_uint(t.y);
    }
  } else {
#pragma unroll
    for (int q = 0; q < N; q += 2) {
      const float2 u = __fmul2_rn(make_float2(__uint_as_float(s[q]), __uint_as_float(s[q + 1])), k2);
      const float2 t = tanh_small2(u);
      s[q] = __float_as_uint(fabsf(u.x) <= kSmall ? t.x : tanh_any(u.x));
      s[q + 1] = __float_as_uint(fabsf(u.y) <= kSmall ? t.y : tanh_any(u.y));
    }
  }
}

// A step's key chunk as the kernels keep it: tile coordinates packed with the
// plan's bit widths (at most 18 bits: N <= 32768) and flags.
constexpr uint32_t kEdge = 1u << 31;    // padded rows
constexpr uint32_t kCausal = 1u << 30;  // some pair of the block and the chunk is hidden by time
constexpr uint32_t kDoc = 1u << 29;     // ids differ somewhere
constexpr uint32_t kHidden = 1u << 28;  // tokens with a negative id

struct Coord {
  int t, h, w;
};
__device__ __forceinline__ uint32_t pack_tile(const Geom& g, const ModParams& m, int j) {
  const int bt = j / (g.nH * g.nW), rem = j - bt * (g.nH * g.nW);
  const int bh = rem / g.nW, bw = rem - bh * g.nW;
  return ((uint32_t)bt << (m.sh_h + m.sh_w)) | ((uint32_t)bh << m.sh_w) | (uint32_t)bw;
}
// First token of the chunk at in-tile offset o of the packed tile.
__device__ __forceinline__ Coord chunk_first(const Geom& g, const ModParams& m, uint32_t packed, const ChunkOrigin& o) {
  const uint32_t x = packed & 0xFFFFFFu;
  return Coord{(int)(x >> (m.sh_h + m.sh_w)) * g.tt + o.dt, (int)((x >> m.sh_w) & ((1u << m.sh_h) - 1u)) * g.th + o.dh,
               (int)(x & ((1u << m.sh_w) - 1u)) * g.tw + o.dw};
}

// One half (64 rows) of a block: the range of its frames and of its ids.
struct Half {
  int lo, hi;        // frames
  int4 ids;          // (least, greatest, tokens with an id, tokens without); all 0 ids without documents
};
__device__ __forceinline__ Half half_of(const Geom& g, const ModParams& m, int b, int tile, int chunk) {
  const ChunkOrigin o = chunk_origin(g, chunk);
  const int t0 = tile / (g.nH * g.nW) * g.tt + o.dt;
  Half r{t0, min(t0 + g.ct - 1, g.T - 1), make_int4(0, 0, 1, 0)};
  if (m.doc_chunks) r.ids = __ldg(m.doc_chunks + ((size_t)b * g.N + tile) * g.nchunk + chunk);
  return r;
}

// Whether queries q see any token of the keys k, by the ranges alone (never
// false when one pair is visible), and which element masks the pair needs.
__device__ __forceinline__ bool sees(const ModParams& m, int prefix, const Half& q, const Half& k, uint32_t* flags) {
  if (m.causal) {
    if (k.lo > q.hi && k.lo >= prefix) return false;
    if (k.hi > q.lo && k.hi >= prefix) *flags |= kCausal;
  }
  if (m.doc_chunks) {
    if (q.ids.z == 0 || k.ids.z == 0 || k.ids.x > q.ids.y || q.ids.x > k.ids.y) return false;
    if (q.ids.x != q.ids.y || k.ids.x != k.ids.y || k.ids.w != 0 || q.ids.w != 0) *flags |= kDoc;
  }
  return true;
}

// Takes the steps that the rules hide from the block out of the compacted
// step list (in place, order kept) and writes each step's packed coordinates
// and flags to ext. One side of every pair is the block's halves (queries, or
// keys with SWAP), the other the step's chunk. All NT threads take part;
// returns the steps left. org (several-chunk tiles, forward) moves along.
template <int NT, bool SWAP>
__device__ __forceinline__ int filter_steps(const Geom& g, const ModParams& m, int b, int prefix, int i0, int i1, int c0,
                                            int c1, uint32_t* list, uint32_t* ext, uint32_t* org, int steps, int* scan) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Half h0 = half_of(g, m, b, i0, c0), h1 = i1 >= 0 ? half_of(g, m, b, i1, c1) : h0;
  int kept = 0;
  for (int base = 0; base < steps; base += NT) {
    const int n = base + tid;
    uint32_t e = 0, x = 0, og = 0;
    if (n < steps) {
      e = list[n];
      const int j = (int)(e & 0x1FFFFFu), c = (int)((e >> 21) & 0x1FFu);
      if (org) og = org[n];
      const Half k = half_of(g, m, b, j, c);
      if (e >> 30 & 1u && !(SWAP ? sees(m, prefix, k, h0, &x) : sees(m, prefix, h0, k, &x))) e &= ~(1u << 30);
      if (e >> 31 & 1u && !(SWAP ? sees(m, prefix, k, h1, &x) : sees(m, prefix, h1, k, &x))) e &= ~(1u << 31);
      x |= pack_tile(g, m, j);
      const ChunkOrigin o = chunk_origin(g, c);
      const Coord f = chunk_first(g, m, x, o);
      if (g.T - f.t < g.ct || g.H - f.h < g.ch || g.W - f.w < g.cw || g.cr < 64) x |= kEdge;
      if (k.ids.w) x |= kHidden;
    }
    const bool keep = (e >> 30) != 0;
    const uint32_t vote = __ballot_sync(0xffffffffu, keep);
    __syncthreads();  // this round's entries are read, the last round's counts too
    if (lane == 0) scan[warp] = __popc(vote);
    __syncthreads();
    int pos = kept + __popc(vote & ((1u << lane) - 1u));
#pragma unroll
    for (int i = 0; i < NT / 32; ++i) {
      pos += i < warp ? scan[i] : 0;
      kept += scan[i];
    }
    if (keep) {  // pos <= n: no entry of a later round is overwritten
      list[pos] = e;
      ext[pos] = x;
      if (org) org[pos] = og;
    }
  }
  return kept;
}

// A row of the block: its grid coordinates, its id (kHiddenDoc: sees and is
// seen by nothing) and whether it is a token that is not hidden.
struct Row {
  Coord at;
  int id;
  bool live;
};
__device__ __forceinline__ Row row_of(const Geom& g, const ModParams& m, int b, int tile, int chunk, uint32_t code,
                                      int r) {
  const ChunkOrigin o = chunk_origin(g, chunk);
  Row x;
  x.at = Coord{tile / (g.nH * g.nW) * g.tt + o.dt + (int)(code & 0xffu),
               tile / g.nW % g.nH * g.th + o.dh + (int)((code >> 8) & 0xffu), tile % g.nW * g.tw + o.dw + (int)((code >> 16) & 0xffu)};
  x.live = r < g.cr && x.at.t < g.T && x.at.h < g.H && x.at.w < g.W;
  x.id = 0;
  if (m.doc_rows) {
    x.id = x.live ? __ldg(m.doc_rows + ((size_t)b * g.N + tile) * g.V + 64 * chunk + r) : -1;
    if (x.id < 0) x.live = false;
  }
  if (!x.live) x.id = kHiddenDoc;
  return x;
}

// Shared tables of a chunk's 64 rows: offsets from its first token along each
// axis, as fp32.
struct ColTab {
  float d[3][64];
};
__device__ __forceinline__ void fill_coltab(const Geom& g, ColTab* tab, int r) {
  const uint32_t c = chunk_row_code(g, r);
  tab->d[0][r] = (float)(c & 0xffu);
  tab->d[1][r] = (float)((c >> 8) & 0xffu);
  tab->d[2][r] = (float)((c >> 16) & 0xffu);
}

// y[q] += sum over the axes of nw[a] |at[a] - d[a][first + q]|: the distance
// bias of a token at offset `at` from the chunk's first token, or, with
// y = 0 and positive weights, the distance itself. Axes of weight zero are
// passed over.
template <int N>
__device__ __forceinline__ void add_distance(float* y, const ColTab* tab, int first, const float* at, const float* nw) {
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    if (nw[a] == 0.f) continue;
    const float4* d4 = reinterpret_cast<const float4*>(tab->d[a] + first);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float4 d = d4[q];
      y[4 * q] = fmaf(fabsf(at[a] - d.x), nw[a], y[4 * q]);
      y[4 * q + 1] = fmaf(fabsf(at[a] - d.y), nw[a], y[4 * q + 1]);
      y[4 * q + 2] = fmaf(fabsf(at[a] - d.z), nw[a], y[4 * q + 2]);
      y[4 * q + 3] = fmaf(fabsf(at[a] - d.w), nw[a], y[4 * q + 3]);
    }
  }
}

// Which of 32 columns (rows first .. of the chunk whose codes colc holds) a
// row sees: offset along t in [lo, vt), along h and w below vh and vw, and,
// where docs is given (the chunk's ids in row order), the row's id.
__device__ __forceinline__ uint32_t visible32(const uint32_t* colc, int first, int lo, int vt, int vh, int vw,
                                              const int32_t* docs, int id) {
  uint32_t vis = 0;
#pragma unroll
  for (int q = 0; q < 32; ++q) {
    const uint32_t cc = colc[first + q];
    const int t = (int)(cc & 0xffu);
    vis |= (t >= lo && t < vt && (int)((cc >> 8) & 0xffu) < vh && (int)((cc >> 16) & 0xffu) < vw ? 1u : 0u) << q;
  }
  if (docs) {
    const int4* d4 = reinterpret_cast<const int4*>(docs + first);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int4 d = __ldg(d4 + q);
      const uint32_t same = (d.x == id ? 1u : 0u) | (d.y == id ? 2u : 0u) | (d.z == id ? 4u : 0u) | (d.w == id ? 8u : 0u);
      vis &= ~((~same & 0xFu) << (4 * q));
    }
  }
  return vis;
}

// Zeroes a 64-row operand tile's rows of hidden tokens (128-byte swizzle: a
// row is 128 contiguous bytes of each 64-column block), so that what such
// rows hold cannot reach the product. The caller fences for the async proxy.
__device__ __forceinline__ void zero_row(uint8_t* tile, int blocks, int r) {
  for (int cb = 0; cb < blocks; ++cb)
#pragma unroll
    for (int q = 0; q < 8; ++q)
      reinterpret_cast<uint4*>(tile + cb * 8192 + r * 128)[q] = make_uint4(0, 0, 0, 0);
}

}  // namespace mod
