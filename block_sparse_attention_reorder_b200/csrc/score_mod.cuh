// Score rules inside the attention kernels: capping by tanh, distance bias,
// causal, prefix and document masks (the definitions stand at
// bsattn_score_mod in bsattn.h). Shared by the forward and the backward.
#pragma once

#include <math.h>

#include <type_traits>

#include "internal.h"
#include "tc_common.cuh"

namespace mod {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kHiddenDoc = -2;  // a query id that equals no key's

// tanh for small |u|: u (1 + v P(v)), v = u^2, P fitted to (tanh(u) / u - 1)
// / v for the least maximum relative error of tanh (Lawson's iteratively
// reweighted least squares): degree 2 on |u| <= 0.375 (7.0e-8; 1.3e-7 with
// fp32 evaluation), degree 4 on |u| <= 0.75 (3.2e-8; 1.0e-7), degree 7 on |u|
// <= 1.5 (1.2e-7; 3.0e-7). Six, eight and eleven FMA-pipe operations on
// packed pairs; the SFU stays free for the softmax.
constexpr float kTiny = 0.375f, kSmall = 0.75f, kWide = 1.5f;
__device__ __forceinline__ float2 bc(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair(const uint32_t* r) { return make_float2(__uint_as_float(r[0]), __uint_as_float(r[1])); }
__device__ __forceinline__ uint32_t pack(float2 v) {
  __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<uint32_t*>(&h);
}
// f(a, b, c) with the three conditions (uniform over the warp) as constants,
// so that one straight loop runs per step.
template <class F>
__device__ __forceinline__ void dispatch(bool a, bool b, bool c, F&& f) {
  constexpr std::true_type Y{};
  constexpr std::false_type N{};
  if (a) {
    if (b) c ? f(Y, Y, Y) : f(Y, Y, N);
    else c ? f(Y, N, Y) : f(Y, N, N);
  } else {
    if (b) c ? f(N, Y, Y) : f(N, Y, N);
    else c ? f(N, N, Y) : f(N, N, N);
  }
}
__device__ __forceinline__ float2 tanh_tiny2(float2 u) {
  const float2 v = __fmul2_rn(u, u);
  float2 p = __ffma2_rn(bc(-0.04848729074001312f), v, bc(0.1328972578048706f));
  p = __ffma2_rn(p, v, bc(-0.33332332968711853f));
  return __fmul2_rn(u, __ffma2_rn(p, v, bc(1.f)));
}
__device__ __forceinline__ float2 tanh_small2(float2 u) {
  const float2 v = __fmul2_rn(u, u);
  float2 p = __ffma2_rn(bc(-0.004769490100443363f), v, bc(0.019664913415908813f));
  p = __ffma2_rn(p, v, bc(-0.0533902570605278f));
  p = __ffma2_rn(p, v, bc(0.13326521217823029f));
  p = __ffma2_rn(p, v, bc(-0.3333306908607483f));
  return __fmul2_rn(u, __ffma2_rn(p, v, bc(1.f)));
}
__device__ __forceinline__ float2 tanh_wide2(float2 u) {
  const float2 v = __fmul2_rn(u, u);
  float2 p = __ffma2_rn(bc(2.621273961267434e-05f), v, bc(-0.000327014276990667f));
  p = __ffma2_rn(p, v, bc(0.0018979610176756978f));
  p = __ffma2_rn(p, v, bc(-0.007121095899492502f));
  p = __ffma2_rn(p, v, bc(0.0207283403724432f));
  p = __ffma2_rn(p, v, bc(-0.053532831370830536f));
  p = __ffma2_rn(p, v, bc(0.13325031101703644f));
  p = __ffma2_rn(p, v, bc(-0.3333278000354767f));
  return __fmul2_rn(u, __ffma2_rn(p, v, bc(1.f)));
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

// Replaces raw scores s[] by tanh(k s) (k = scale / cap) in the form that TIER
// names: 0, 1 and 2 the polynomials, 3 the SFU form. The forms agree to about
// 3e-7 absolute.
template <int TIER, int N>
__device__ __forceinline__ void tanh_form(uint32_t* s, float k) {
  const float2 k2 = bc(k);
#pragma unroll
  for (int q = 0; q < N; q += 2) {
    const float2 u = __fmul2_rn(pair(s + q), k2);
    const float2 t = TIER == 0   ? tanh_tiny2(u)
                     : TIER == 1 ? tanh_small2(u)
                     : TIER == 2 ? tanh_wide2(u)
                                 : make_float2(tanh_any(u.x), tanh_any(u.y));
    s[q] = __float_as_uint(t.x);
    s[q + 1] = __float_as_uint(t.y);
  }
}
// Greatest |s|; a NaN is passed over.
template <int N>
__device__ __forceinline__ float greatest(const uint32_t* s) {
  float mx4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < N; q += 2)
    mx4[(q / 2) & 3] = tc::fmax3(mx4[(q / 2) & 3], fabsf(__uint_as_float(s[q])), fabsf(__uint_as_float(s[q + 1])));
  return fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
}
// Sets the scores of unseen pairs (bits of see) to x.
template <int N>
__device__ __forceinline__ void set_unseen(uint32_t* s, unsigned long long see, float x) {
  const uint32_t w[2] = {(uint32_t)see, (uint32_t)(see >> 32)};
#pragma unroll
  for (int q = 0; q < N; ++q)
    if (!((w[q / 32] >> (q % 32)) & 1u)) s[q] = __float_as_uint(x);
}
// The cheapest form that covers all of the warp's values (those of unseen
// pairs are zero by then: what hidden rows hold picks no form).
template <int N>
__device__ __forceinline__ void tanh_scores(uint32_t* s, float k) {
  const float mx = greatest<N>(s) * fabsf(k);
  if (__all_sync(0xffffffffu, mx <= kTiny))
    tanh_form<0, N>(s, k);
  else if (__all_sync(0xffffffffu, mx <= kSmall))
    tanh_form<1, N>(s, k);
  else if (__all_sync(0xffffffffu, mx <= kWide))
    tanh_form<2, N>(s, k);
  else
    tanh_form<3, N>(s, k);
}

// A step's key chunk as the kernels keep it: tile coordinates packed with the
// plan's bit widths (at most 23 bits for N <= 2^20 tiles) and flags.
constexpr uint32_t kEdge = 1u << 31;    // padded rows
constexpr uint32_t kCausal = 1u << 30;  // some pair of the block and the chunk is hidden by time
constexpr uint32_t kDoc = 1u << 29;     // ids differ somewhere
constexpr uint32_t kHidden = 1u << 28;  // tokens with a negative id
constexpr uint32_t kSpecial = kEdge | kCausal | kDoc | kHidden;

struct Coord {
  int t, h, w;
};
// a / d for 0 <= a < 2^23 with inv = 1 / d: the estimate is off by one at most.
// A CTA's set-up is a chain of such steps: the filter of a two-step list, with
// some twenty integer divisions in a row, took 2,200 cycles.
__device__ __forceinline__ int quotient(int a, int d, float inv) {
  const int q = (int)((float)a * inv), r = a - q * d;
  return q + (r >= d ? 1 : 0) - (r < 0 ? 1 : 0);
}
// In-tile origin of a chunk (the first at once: tiles of one chunk are the usual ones).
__device__ __forceinline__ ChunkOrigin origin_of(const Geom& g, int c) {
  return c == 0 ? ChunkOrigin{0, 0, 0} : chunk_origin(g, c);
}
__device__ __forceinline__ ChunkOrigin unpack_origin(uint32_t v) {
  return ChunkOrigin{(int)(v & 0x3FFu), (int)((v >> 10) & 0x3FFu), (int)(v >> 20)};
}
struct Tile {
  int t, h, w;
};
__device__ __forceinline__ Tile tile_of(const Geom& g, const ModParams& m, int j) {
  const int t = quotient(j, g.nH * g.nW, m.per_plane), rem = j - t * (g.nH * g.nW);
  const int h = quotient(rem, g.nW, m.per_row);
  return Tile{t, h, rem - h * g.nW};
}
__device__ __forceinline__ uint32_t pack_tile(const Geom& g, const ModParams& m, int j) {
  const Tile x = tile_of(g, m, j);
  const int bt = x.t, bh = x.h, bw = x.w;
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
__device__ __forceinline__ Half half_of(const Geom& g, const ModParams& m, int b, int tile, int chunk,
                                        const ChunkOrigin& o) {
  const int t0 = quotient(tile, g.nH * g.nW, m.per_plane) * g.tt + o.dt;
  Half r{t0, min(t0 + g.ct - 1, g.T - 1), make_int4(0, 0, 1, 0)};
  if (m.doc_chunks) r.ids = __ldg(&m.doc_chunks[((size_t)b * g.N + tile) * g.nchunk + chunk].range);
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

// Takes chunks of padding and the steps that the rules hide from the block out
// of the step list (in place, order kept) and writes each step's packed coordinates
// and flags to ext. One side of every pair is the block's halves (queries, or
// keys with SWAP), the other the step's chunk. All NT threads take part;
// returns the steps left. origin: every chunk's packed in-tile origin (shared).
template <int NT, bool SWAP>
__device__ __forceinline__ int filter_steps(const Geom& g, const ModParams& m, int b, int prefix, int i0, int i1, int c0,
                                            int c1, uint32_t* list, uint32_t* ext, int steps, int* scan,
                                            const uint32_t* origin) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Half h0 = half_of(g, m, b, i0, c0, unpack_origin(origin[c0]));
  const Half h1 = i1 >= 0 ? half_of(g, m, b, i1, c1, unpack_origin(origin[c1])) : h0;
  int kept = 0;
  for (int base = 0; base < steps; base += NT) {
    const int n = base + tid;
    uint32_t e = 0, x = 0;
    if (n < steps) {
      e = list[n];
      const int j = (int)(e & 0x1FFFFFu), c = (int)((e >> 21) & 0x1FFu);
      const ChunkOrigin o = unpack_origin(origin[c]);
      const Half k = half_of(g, m, b, j, c, o);
      if (e >> 30 & 1u && !(SWAP ? sees(m, prefix, k, h0, &x) : sees(m, prefix, h0, k, &x))) e &= ~(1u << 30);
      if (e >> 31 & 1u && !(SWAP ? sees(m, prefix, k, h1, &x) : sees(m, prefix, h1, k, &x))) e &= ~(1u << 31);
      x |= pack_tile(g, m, j);
      const Coord f = chunk_first(g, m, x, o);
      if (g.T - f.t < g.ct || g.H - f.h < g.ch || g.W - f.w < g.cw || g.cr < 64) x |= kEdge;
      if (k.ids.w) x |= kHidden;
      if (f.t >= g.T || f.h >= g.H || f.w >= g.W) e = 0;  // a chunk of padding
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
  const ChunkOrigin o = origin_of(g, chunk);
  const Tile i = tile_of(g, m, tile);
  Row x;
  x.at = Coord{i.t * g.tt + o.dt + (int)(code & 0xffu), i.h * g.th + o.dh + (int)((code >> 8) & 0xffu),
               i.w * g.tw + o.dw + (int)((code >> 16) & 0xffu)};
  x.live = r < g.cr && x.at.t < g.T && x.at.h < g.H && x.at.w < g.W;
  x.id = 0;
  if (m.doc_rows) {
    x.id = x.live ? __ldg(m.doc_rows + ((size_t)b * g.N + tile) * g.V + 64 * chunk + r) : -1;
    if (x.id < 0) x.live = false;
  }
  if (!x.live) x.id = kHiddenDoc;
  return x;
}

// Shared tables of a chunk's 64 rows (columns of a step).
struct Table {
  float d[3][64];              // offsets from the chunk's first token along each axis
  float4 group[16];            // the same for rows 4g (t, h, w)
  unsigned long long below[3][68];  // rows whose offset along the axis is below v, v = 0 .. box extent
};
// Filled by all NT threads; codes of the rows in colc (shared, visible).
template <int NT>
__device__ __forceinline__ void fill_table(const Geom& g, Table* tab, const uint32_t* colc) {
  const int tid = threadIdx.x;
  if (tid < 64) {
    const uint32_t c = colc[tid];
    const float4 d = make_float4((float)(c & 0xffu), (float)((c >> 8) & 0xffu), (float)((c >> 16) & 0xffu), 0.f);
    tab->d[0][tid] = d.x;
    tab->d[1][tid] = d.y;
    tab->d[2][tid] = d.z;
    if (tid % 4 == 0) tab->group[tid / 4] = d;
  }
  // A thread per entry: rows are ordered (t, h, w), so the first v steps of an
  // axis are v times the inner extents' product of each of its periods.
  const int n0 = g.ct + 1, n1 = n0 + g.ch + 1, n2 = n1 + g.cw + 1;
  for (int e = tid; e < n2; e += NT) {
    const int a = e < n0 ? 0 : e < n1 ? 1 : 2, v = e - (a == 0 ? 0 : a == 1 ? n0 : n1);
    const int inner = a == 0 ? g.ch * g.cw : a == 1 ? g.cw : 1, period = a == 0 ? g.cr : a == 1 ? g.ch * g.cw : g.cw;
    unsigned long long m = v * inner >= 64 ? ~0ull : (1ull << (v * inner)) - 1ull;
    for (int p = period; p < g.cr; p *= 2) m |= m << p;
    tab->below[a][v] = g.cr < 64 ? m & ((1ull << g.cr) - 1ull) : m;
  }
}

// Which rows of a chunk a token sees by coordinates: offset along t in
// [lo, vt), along h and w below vh and vw (any integers).
__device__ __forceinline__ unsigned long long visible_box(const Geom& g, const Table* tab, int lo, int vt, int vh, int vw) {
  return tab->below[0][min(max(vt, 0), g.ct)] & ~tab->below[0][min(max(lo, 0), g.ct)] &
         tab->below[1][min(max(vh, 0), g.ch)] & tab->below[2][min(max(vw, 0), g.cw)];
}

// Which rows of a chunk carry the token's id.
__device__ __forceinline__ unsigned long long visible_doc(const ModParams& m, size_t chunk, int id) {
  const DocChunk* c = m.doc_chunks + chunk;
  const int4 ids = __ldg(&c->id);
  const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(c->rows)), b = __ldg(reinterpret_cast<const ulonglong2*>(c->rows + 2));
  unsigned long long vis = (ids.x == id ? a.x : 0ull) | (ids.y == id ? a.y : 0ull) | (ids.z == id ? b.x : 0ull);
  if (ids.w != kManyIds) return vis | (ids.w == id ? b.y : 0ull);
  // More than four ids in 64 tokens: the rows themselves.
  const int4* d4 = reinterpret_cast<const int4*>(m.doc_rows + 64 * chunk);
  vis = 0;
  for (int q = 0; q < 16; ++q) {
    const int4 d = __ldg(d4 + q);
    vis |= (unsigned long long)((d.x == id ? 1u : 0u) | (d.y == id ? 2u : 0u) | (d.z == id ? 4u : 0u) | (d.w == id ? 8u : 0u)) << (4 * q);
  }
  return vis;
}

// Distance bias of a token at offset (t, h, w) from the chunk's first token,
// weights nt, nh, nw (0 for an axis of one token): y[q] += sum of weight times
// |offset - the row's|; with SET and positive weights y becomes the distance.
struct Dist {
  float t, h, w, nt, nh, nw;
};
__device__ __forceinline__ Dist make_dist(const Geom& g, const ModParams& m, const Coord& at, const Coord& first,
                                          float scale) {
  return Dist{(float)(at.t - first.t), (float)(at.h - first.h), (float)(at.w - first.w),
              g.T > 1 ? scale * m.dist[0] : 0.f, g.H > 1 ? scale * m.dist[1] : 0.f, g.W > 1 ? scale * m.dist[2] : 0.f};
}
// y[q .. q + 3] += u + w terms (SET: = instead), on packed pairs.
template <bool SET>
__device__ __forceinline__ void add4(float* y, float u, float w0, float w1, float w2, float w3) {
  float2 a = __fadd2_rn(bc(u), make_float2(w0, w1)), b = __fadd2_rn(bc(u), make_float2(w2, w3));
  if (!SET) {
    a = __fadd2_rn(make_float2(y[0], y[1]), a);
    b = __fadd2_rn(make_float2(y[2], y[3]), b);
  }
  y[0] = a.x; y[1] = a.y; y[2] = b.x; y[3] = b.y;
}
template <int N>
__device__ __forceinline__ void axis_distance(float* y, const float* d, float at, float nw) {
  const float4* d4 = reinterpret_cast<const float4*>(d);
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const float4 x = d4[q];
    y[4 * q] = fmaf(fabsf(at - x.x), nw, y[4 * q]);
    y[4 * q + 1] = fmaf(fabsf(at - x.y), nw, y[4 * q + 1]);
    y[4 * q + 2] = fmaf(fabsf(at - x.z), nw, y[4 * q + 2]);
    y[4 * q + 3] = fmaf(fabsf(at - x.w), nw, y[4 * q + 3]);
  }
}
// In chunks whose rows of four or eight lie along w the t and h terms are one
// value for four columns and the w terms four or eight values per step: three
// operations a column. Chunks that are a line (sequences) take two; with all 64 columns
// at a time one where no query of the warp stands among them (the distance is
// linear there, two packed operations a pair: 8 x 16K tokens 1,300 -> 1,195 us;
// beside the cap's 32 columns at a time the larger code costs 4%). Axis
// after axis, seven with the table reads, serves the other shapes and passes
// over axes of weight zero.
template <int N, bool SET = false>
__device__ __forceinline__ void add_distance(const Geom& g, float* y, const Table* tab, int first, const Dist& p) {
  if (g.cw == 4 || g.cw == 8) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = p.nw * fabsf(p.w - (float)i);
    const bool wide = g.cw == 8;
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float2 d = *reinterpret_cast<const float2*>(&tab->group[first / 4 + q]);
      const float u = fmaf(p.nh, fabsf(p.h - d.y), p.nt * fabsf(p.t - d.x));
      if ((q & 1) && wide)
        add4<SET>(y + 4 * q, u, w[4], w[5], w[6], w[7]);
      else
        add4<SET>(y + 4 * q, u, w[0], w[1], w[2], w[3]);
    }
    return;
  }
  if (g.ct == 64 || g.cw == 64) {  // 64 tokens in a line along t or w: the offset is the column
    const float at = g.ct == 64 ? p.t : p.w, n = g.ct == 64 ? p.nt : p.nw;
    const float u = fmaf(p.nh, fabsf(p.h), g.ct == 64 ? p.nw * fabsf(p.w) : p.nt * fabsf(p.t));
    const float a0 = at - (float)first;
    if (N == 64 && __all_sync(0xffffffffu, a0 >= (float)(N - 1) || a0 <= 0.f)) {  // every row before or behind the columns
      const float k = a0 <= 0.f ? n : -n;  // |a0 - q| n = k q - k a0
      const float2 k2 = bc(k), base = bc(fmaf(-k, a0, u));
#pragma unroll
      for (int q = 0; q < N; q += 2) {
        float2 x = __ffma2_rn(k2, make_float2((float)q, (float)(q + 1)), base);
        if (!SET) x = __fadd2_rn(make_float2(y[q], y[q + 1]), x);
        y[q] = x.x;
        y[q + 1] = x.y;
      }
      return;
    }
#pragma unroll
    for (int q = 0; q < N; ++q) y[q] = SET ? fabsf(a0 - (float)q) * n : fmaf(fabsf(a0 - (float)q), n, y[q]);
    if (u != 0.f) {
#pragma unroll
      for (int q = 0; q < N; ++q) y[q] += u;
    }
    return;
  }
  if (SET) {
#pragma unroll
    for (int q = 0; q < N; ++q) y[q] = 0.f;
  }
  if (p.nt != 0.f) axis_distance<N>(y, tab->d[0] + first, p.t, p.nt);
  if (p.nh != 0.f) axis_distance<N>(y, tab->d[1] + first, p.h, p.nh);
  if (p.nw != 0.f) axis_distance<N>(y, tab->d[2] + first, p.w, p.nw);
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
