// Score rules: their checks and entry points, document ids brought into tile
// order, the rules on block scores, and the sum of the slope gradient's parts.
// The rules inside the attention kernels are in score_mod.cuh.
#include "score_mod.cuh"

#include <float.h>
#include <limits.h>

namespace {

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct Carve {
  uint8_t* base;
  size_t off = 0;
  explicit Carve(void* b) : base((uint8_t*)b) {}
  void* take(size_t bytes) {
    void* r = base ? base + off : nullptr;
    off += align_up(bytes, 256);
    return r;
  }
};

// Ids in tile order, and their ranges per 64-row chunk and per tile.
struct DocWs {
  int32_t* rows;  // [B, N, V]
  DocChunk* chunks;  // [B, N, nchunk]
};

DocWs carve_doc(const bsattn_plan* p, Carve& c) {
  const size_t bn = (size_t)p->desc.B * p->N;
  DocWs w;
  w.rows = (int32_t*)c.take(bn * p->V * sizeof(int32_t));
  w.chunks = (DocChunk*)c.take(bn * p->nchunk * sizeof(DocChunk));
  return w;
}

struct BwdModWs {
  DocWs doc;
  float* slope_parts;
  float* neg_lse2;
  void* shares;
  BackwardWs b;
};
BwdModWs carve_backward_mod(const bsattn_plan* p, Carve& c) {
  const size_t rows = (size_t)p->desc.B * p->desc.heads * p->N;
  BwdModWs w;
  w.doc = carve_doc(p, c);
  w.slope_parts = (float*)c.take((size_t)p->desc.B * p->desc.heads * backward_slope_items(p) * sizeof(float));
  w.neg_lse2 = (float*)c.take(rows * p->V * sizeof(float));
  w.shares = c.take(backward_mod_workspace_bytes(p));
  w.b.delta = (float*)c.take(rows * p->V * sizeof(float));
  w.b.bm = (uint32_t*)c.take(rows * ((p->N + 31) / 32) * sizeof(uint32_t));
  w.b.idxT = (int32_t*)c.take(rows * p->N * sizeof(int32_t));
  w.b.cntT = (int32_t*)c.take(rows * sizeof(int32_t));
  return w;
}

struct FwdModWs {
  DocWs doc;
  void* parts;
};
FwdModWs carve_forward_mod(const bsattn_plan* p, Carve& c) {
  FwdModWs w;
  w.doc = carve_doc(p, c);
  w.parts = c.take(attention_mod_workspace_bytes(p));
  return w;
}

struct LayerModWs {
  DocWs doc;
  void* parts;
  __nv_bfloat16 *q, *k;  // rotated
  uint8_t *qc, *kc;      // e4m3 tile codes
  float *qs, *ks;
  float *pq, *pk, *S;
  int32_t *idx, *cnt;
};
LayerModWs carve_layer_mod(const bsattn_plan* p, Carve& c) {
  const size_t bh = (size_t)p->desc.B * p->desc.heads, D = p->desc.head_dim;
  const bool route = p->rule.kind != BSATTN_RULE_WINDOW;
  const size_t codes = p->desc.qk_fp8 ? bh * p->N * p->V * D : 0;
  LayerModWs w;
  w.doc = carve_doc(p, c);
  w.parts = c.take(attention_mod_workspace_bytes(p));
  w.q = (__nv_bfloat16*)c.take(bh * p->L * D * 2);
  w.k = (__nv_bfloat16*)c.take(bh * p->L * D * 2);
  w.qc = (uint8_t*)c.take(codes);
  w.kc = (uint8_t*)c.take(codes);
  w.qs = (float*)c.take(p->desc.qk_fp8 ? bh * p->N * sizeof(float) : 0);
  w.ks = (float*)c.take(p->desc.qk_fp8 ? bh * p->N * sizeof(float) : 0);
  w.pq = (float*)c.take(route ? bh * p->N * D * sizeof(float) : 0);
  w.pk = (float*)c.take(route ? bh * p->N * D * sizeof(float) : 0);
  w.S = (float*)c.take(route ? bh * p->N * p->N * sizeof(float) : 0);
  w.idx = (int32_t*)c.take(bh * p->N * p->kmax * sizeof(int32_t));
  w.cnt = (int32_t*)c.take(bh * p->N * sizeof(int32_t));
  return w;
}

// One warp per (64-row chunk, batch), two rows a lane: the ids in tile order,
// their range, and up to four ids with their rows. A few bytes per token;
// bound by its launch.
constexpr int kPrepWarps = 4;
__global__ void __launch_bounds__(32 * kPrepWarps) doc_prep_kernel(Geom g, const int32_t* __restrict__ doc, DocWs w) {
  const int lane = threadIdx.x % 32, b = blockIdx.y;
  const long long n = (long long)blockIdx.x * kPrepWarps + threadIdx.x / 32;  // chunk of the batch
  if (n >= (long long)g.N * g.nchunk) return;
  const int j = (int)(n / g.nchunk), c = (int)(n % g.nchunk);
  const ChunkOrigin o = chunk_origin(g, c);
  const int t0 = j / (g.nH * g.nW) * g.tt + o.dt, h0 = j / g.nW % g.nH * g.th + o.dh, w0 = j % g.nW * g.tw + o.dw;
  int id[2];
  int without = 0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = lane + 32 * x;
    const uint32_t code = chunk_row_code(g, r);
    const int t = t0 + (int)(code & 0xffu), h = h0 + (int)((code >> 8) & 0xffu), v = w0 + (int)((code >> 16) & 0xffu);
    const bool real = r < g.cr && t < g.T && h < g.H && v < g.W;
    id[x] = real ? doc[(size_t)b * g.L + (t * g.H + h) * g.W + v] : -1;
    if (id[x] < 0) {
      id[x] = -1;
      without += real ? 1 : 0;
    }
    w.rows[((size_t)b * g.N + j) * g.V + 64 * c + r] = id[x];
  }
  const unsigned all = 0xffffffffu;
  DocChunk k;
  k.range.x = __reduce_min_sync(all, min(id[0] < 0 ? INT_MAX : id[0], id[1] < 0 ? INT_MAX : id[1]));
  k.range.y = __reduce_max_sync(all, max(id[0], id[1]));
  k.range.z = __reduce_add_sync(all, (id[0] >= 0) + (id[1] >= 0));
  k.range.w = __reduce_add_sync(all, without);
  int ids[4];
  int left[2] = {id[0], id[1]};
#pragma unroll
  for (int e = 0; e < 4; ++e) {  // the least id not yet taken; greatest int as an id shares the code of "none left"
    const int next = __reduce_min_sync(all, min(left[0] < 0 ? INT_MAX : left[0], left[1] < 0 ? INT_MAX : left[1]));
    const uint32_t lo = __ballot_sync(all, left[0] == next), hi = __ballot_sync(all, left[1] == next);
    ids[e] = lo | hi ? next : kNoId;
    k.rows[e] = ((unsigned long long)hi << 32) | lo;
    if (left[0] == next) left[0] = -1;
    if (left[1] == next) left[1] = -1;
  }
  if (__any_sync(all, left[0] >= 0 || left[1] >= 0)) ids[3] = kManyIds;
  k.id = make_int4(ids[0], ids[1], ids[2], ids[3]);
  if (lane == 0) w.chunks[((size_t)b * g.N + j) * g.nchunk + c] = k;
}

// Least and greatest id >= 0 of each tile (INT_MAX, -1: none), from its chunks.
__device__ __forceinline__ int2 tile_ids(const Geom& g, const DocChunk* chunks, int b, int j) {
  int2 r = make_int2(INT_MAX, -1);
  for (int c = 0; c < g.nchunk; ++c) {
    const int4 x = __ldg(&chunks[((size_t)b * g.N + j) * g.nchunk + c].range);
    r.x = min(r.x, x.x);
    r.y = max(r.y, x.y);
  }
  return r;
}

// The rules on block scores, S' from S. Memory bound (8 bytes an entry): a
// thread owns four neighbouring key tiles, whose mean coordinates and ranges
// it keeps in registers (no division per entry), and walks kScoreRows query
// tiles, whose own come from shared memory, four rows' loads in flight. On one
// B200 128-133 us for the Wan-14B-shaped layer (40 x 1440 x 1440, 664 MB) with
// every rule, 0.77-0.79 of the measured copy rate; one row at a time 154-164.
constexpr int kScoreRows = 32;
constexpr int kScoreThreads = 128;

struct TileMeta {
  float4 mean;  // mean (t, h, w) of the real tokens
  int4 range;   // first and last frame, least and greatest id
};
__device__ __forceinline__ TileMeta tile_meta(const Geom& g, int j, int b, const DocChunk* ids) {
  const int t0 = j / (g.nH * g.nW) * g.tt, h0 = j / g.nW % g.nH * g.th, w0 = j % g.nW * g.tw;
  const int vt = min(g.tt, g.T - t0), vh = min(g.th, g.H - h0), vw = min(g.tw, g.W - w0);
  TileMeta m{make_float4(t0 + 0.5f * (vt - 1), h0 + 0.5f * (vh - 1), w0 + 0.5f * (vw - 1), 0.f),
             make_int4(t0, t0 + vt - 1, 0, 0)};
  if (ids) {
    const int2 r = tile_ids(g, ids, b, j);
    m.range.z = r.x;
    m.range.w = r.y;
  }
  return m;
}

template <bool VEC>
__global__ void __launch_bounds__(kScoreThreads)
mod_scores_kernel(Geom g, ModParams m, const float* S, float* out) {
  __shared__ float4 row_mean[kScoreRows];
  __shared__ int4 row_range[kScoreRows];
  const DocChunk* ids = m.doc_chunks;
  const int N = g.N, bh = blockIdx.z, b = bh / g.Hh, head = bh % g.Hh;
  const int i0 = blockIdx.y * kScoreRows, rows = min(kScoreRows, N - i0);
  const int j0 = 4 * (blockIdx.x * kScoreThreads + threadIdx.x);
  if (threadIdx.x < rows) {
    const TileMeta q = tile_meta(g, i0 + threadIdx.x, b, ids);
    row_mean[threadIdx.x] = q.mean;
    row_range[threadIdx.x] = q.range;
  }
  __syncthreads();
  if (j0 >= N) return;
  const int prefix = m.prefix ? __ldg(m.prefix + b) : 0;
  TileMeta km[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    km[e] = tile_meta(g, min(j0 + e, N - 1), b, ids);
    if (!m.causal || km[e].range.x < prefix) km[e].range.x = INT_MIN;  // never behind a query's last frame
  }
  const float slope = m.slopes ? __ldg(m.slopes + head) : 0.f;
  const float inv = m.cap > 0.f ? 1.f / m.cap : 0.f;
  const float* src = S + ((size_t)bh * N + i0) * N + j0;
  float* dst = out + ((size_t)bh * N + i0) * N + j0;
  const int ne = min(4, N - j0);
  constexpr int kBatch = 4;
#pragma unroll 1
  for (int ib = 0; ib < rows; ib += kBatch) {
    float v[kBatch][4];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int i = min(ib + x, rows - 1);  // the last row again, not stored
      if (VEC) {
        const float4 y = *reinterpret_cast<const float4*>(src + (size_t)i * N);
        v[x][0] = y.x; v[x][1] = y.y; v[x][2] = y.z; v[x][3] = y.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[x][e] = e < ne ? src[(size_t)i * N + e] : 0.f;
      }
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int i = ib + x;
      if (i >= rows) break;
      if (m.cap > 0.f) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 u = __fmul2_rn(make_float2(v[x][e], v[x][e + 1]), mod::bc(inv));
          const float2 t = mod::tanh_small2(u);
          v[x][e] = m.cap * (fabsf(u.x) <= mod::kSmall ? t.x : mod::tanh_any(u.x));
          v[x][e + 1] = m.cap * (fabsf(u.y) <= mod::kSmall ? t.y : mod::tanh_any(u.y));
        }
      }
      if (m.slopes) {
        const float4 q = row_mean[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float far = m.dist[0] * fabsf(q.x - km[e].mean.x);
          far = fmaf(m.dist[1], fabsf(q.y - km[e].mean.y), far);
          far = fmaf(m.dist[2], fabsf(q.z - km[e].mean.z), far);
          v[x][e] = fmaf(-slope, far, v[x][e]);
        }
      }
      const int4 q = row_range[i];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (km[e].range.x > q.y || km[e].range.z > q.w || q.z > km[e].range.w) v[x][e] = -FLT_MAX;
      if (VEC) {
        *reinterpret_cast<float4*>(dst + (size_t)i * N) = make_float4(v[x][0], v[x][1], v[x][2], v[x][3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < ne) dst[(size_t)i * N + e] = v[x][e];
      }
    }
  }
}

// d_slopes[head] = sum of the head's parts over batches and CTAs, in a fixed
// order in fp64.
__global__ void __launch_bounds__(256) slope_sum_kernel(const float* __restrict__ parts, int B, int heads, int items,
                                                        float* __restrict__ d_slopes) {
  __shared__ double red[256];
  const int head = blockIdx.x;
  double s = 0.0;
  for (int b = 0; b < B; ++b)
    for (int x = threadIdx.x; x < items; x += 256) s += (double)parts[((size_t)b * heads + head) * items + x];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) d_slopes[head] = (float)red[0];
}

bool ok_ptr(const void* x) { return x != nullptr && aligned16(x); }

bsattn_status check_mod(const bsattn_score_mod* m) {
  if (!m) return BSATTN_ERR_INVALID_ARG;
  if (m->softcap != 0.f && !(m->softcap >= 1e-6f && m->softcap <= 1e30f)) return BSATTN_ERR_INVALID_ARG;
  const float d[3] = {m->dist_t, m->dist_h, m->dist_w};
  for (float x : d)
    if (!(x >= 0.f) || !isfinite(x)) return BSATTN_ERR_INVALID_ARG;
  if (m->causal != 0 && m->causal != 1) return BSATTN_ERR_INVALID_ARG;
  if (m->prefix && !m->causal) return BSATTN_ERR_INVALID_ARG;
  if (!aligned16(m->slopes) || !aligned16(m->prefix) || !aligned16(m->doc)) return BSATTN_ERR_INVALID_ARG;
  return BSATTN_OK;
}

int bits_of(int n) {  // bits of 0 .. n - 1
  int b = 0;
  while ((1 << b) < n) ++b;
  return b;
}

ModParams device_mod(const bsattn_plan* p, const bsattn_score_mod* m, const DocWs& w) {
  ModParams d;
  d.cap = m->softcap;
  d.slopes = m->slopes;
  d.dist[0] = m->dist_t; d.dist[1] = m->dist_h; d.dist[2] = m->dist_w;
  d.causal = m->causal;
  d.prefix = m->prefix;
  d.doc_rows = m->doc ? w.rows : nullptr;
  d.doc_chunks = m->doc ? w.chunks : nullptr;
  d.sh_h = bits_of(p->nH);
  d.sh_w = bits_of(p->nW);
  d.per_plane = 1.f / ((float)p->nH * (float)p->nW);
  d.per_row = 1.f / (float)p->nW;
  return d;
}

bsattn_status launch_doc_prep(const bsattn_plan* p, const bsattn_score_mod* m, const DocWs& w, cudaStream_t st) {
  if (!m->doc) return BSATTN_OK;
  const long long chunks = (long long)p->N * p->nchunk;
  doc_prep_kernel<<<dim3((unsigned)((chunks + kPrepWarps - 1) / kPrepWarps), p->desc.B), 32 * kPrepWarps, 0, st>>>(
      make_geom(p), m->doc, w);
  return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

bsattn_status launch_mod_scores(const bsattn_plan* p, const ModParams& d, const float* S, float* out, cudaStream_t st) {
  const Geom g = make_geom(p);
  dim3 grid((g.N + 4 * kScoreThreads - 1) / (4 * kScoreThreads), (g.N + kScoreRows - 1) / kScoreRows, g.B * g.Hh);
  if (g.N % 4 == 0)  // every row starts on 16 bytes
    mod_scores_kernel<true><<<grid, kScoreThreads, 0, st>>>(g, d, S, out);
  else
    mod_scores_kernel<false><<<grid, kScoreThreads, 0, st>>>(g, d, S, out);
  return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

// What the rules on block scores refuse, asked before a call enqueues anything
// (as check_attention_mod and check_backward_mod).
bsattn_status check_scores(const bsattn_plan* p) {
  return p->N > 2048 || (long long)p->desc.B * p->desc.heads > 65535 ? BSATTN_ERR_UNSUPPORTED : BSATTN_OK;
}

// The workspace of calls that need one for documents only.
bsattn_status carve_call_doc(const bsattn_plan* p, const bsattn_score_mod* m, void* ws, size_t ws_bytes, DocWs* w) {
  if (!m->doc) {
    *w = DocWs{};
    return BSATTN_OK;
  }
  Carve size(nullptr);
  carve_doc(p, size);
  if (!ws || !aligned16(ws) || ws_bytes < size.off) return BSATTN_ERR_WORKSPACE;
  Carve c(ws);
  *w = carve_doc(p, c);
  return BSATTN_OK;
}

bsattn_status forward_mod(const bsattn_plan* p, const bsattn_score_mod* m, const void* q, const void* k, const float* qs,
                          const float* ks, const void* v, const int32_t* idx, const int32_t* cnt, void* o, float* lse,
                          void* ws, size_t ws_bytes, void* stream, AttnLayout lay) {
  if (!p || !ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(idx) || !ok_ptr(cnt) || !ok_ptr(o) ||
      (lse && !aligned16(lse)))
    return BSATTN_ERR_INVALID_ARG;
  if (p->desc.qk_fp8 && (!ok_ptr(qs) || !ok_ptr(ks))) return BSATTN_ERR_INVALID_ARG;
  bsattn_status s = check_mod(m);
  if (s) return s;
  Carve size(nullptr);
  carve_forward_mod(p, size);
  FwdModWs w{};
  if (ws || m->doc) {
    if (!ws || !aligned16(ws) || ws_bytes < size.off) return BSATTN_ERR_WORKSPACE;
    Carve c(ws);
    w = carve_forward_mod(p, c);
  }
  if ((s = check_attention_mod(p))) return s;
  DeviceGuard dev(p->device);
  if (dev.status) return dev.status;
  if ((s = launch_doc_prep(p, m, w.doc, (cudaStream_t)stream))) return s;
  const ModParams d = device_mod(p, m, w.doc);
  return launch_attention_mod(p, d, q, k, qs, ks, (const __nv_bfloat16*)v, idx, cnt, (__nv_bfloat16*)o, lse,
                              w.parts, (cudaStream_t)stream, lay);
}

}  // namespace

extern "C" {

bsattn_status attn_mod_info(const bsattn_plan* p, bsattn_mod_info* o) {
  if (!p || !o) return BSATTN_ERR_INVALID_ARG;
  Carve a(nullptr), f(nullptr), b(nullptr), c(nullptr);
  carve_doc(p, a);
  carve_forward_mod(p, f);
  carve_backward_mod(p, b);
  carve_layer_mod(p, c);
  o->scores_workspace_bytes = a.off;
  o->forward_workspace_bytes = f.off;
  o->backward_workspace_bytes = b.off;
  o->layer_workspace_bytes = c.off;
  return BSATTN_OK;
}

bsattn_status attn_mod_scores(const bsattn_plan* p, const bsattn_score_mod* m, const float* S, float* out, void* ws,
                              size_t ws_bytes, void* stream) {
  if (!p || !ok_ptr(S) || !ok_ptr(out)) return BSATTN_ERR_INVALID_ARG;
  bsattn_status s = check_mod(m);
  if (s) return s;
  if ((s = check_scores(p))) return s;
  DocWs w;
  if ((s = carve_call_doc(p, m, ws, ws_bytes, &w))) return s;
  DeviceGuard dev(p->device);
  if (dev.status) return dev.status;
  if ((s = launch_doc_prep(p, m, w, (cudaStream_t)stream))) return s;
  return launch_mod_scores(p, device_mod(p, m, w), S, out, (cudaStream_t)stream);
}

bsattn_status attn_forward_mod(const bsattn_plan* p, const bsattn_score_mod* m, const void* q, const void* k,
                               const float* qs, const float* ks, const void* v, const int32_t* idx, const int32_t* cnt,
                               void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  return forward_mod(p, m, q, k, qs, ks, v, idx, cnt, o, lse, ws, ws_bytes, stream, AttnLayout::Tiled);
}

bsattn_status attn_forward_natural_mod(const bsattn_plan* p, const bsattn_score_mod* m, const void* q, const void* k,
                                       const float* qs, const float* ks, const void* v_nat, const int32_t* idx,
                                       const int32_t* cnt, void* o_nat, float* lse_nat, void* ws, size_t ws_bytes,
                                       void* stream) {
  return forward_mod(p, m, q, k, qs, ks, v_nat, idx, cnt, o_nat, lse_nat, ws, ws_bytes, stream, AttnLayout::Natural);
}

bsattn_status attn_backward_mod(const bsattn_plan* p, const bsattn_score_mod* m, const void* q, const void* k,
                                const void* v, const void* o, const void* d_o, const float* lse, const int32_t* idx,
                                const int32_t* cnt, void* dq, void* dk, void* dv, float* d_slopes, void* ws,
                                size_t ws_bytes, void* stream) {
  if (!p || !ok_ptr(q) || !ok_ptr(k) || !ok_ptr(v) || !ok_ptr(o) || !ok_ptr(d_o) || !ok_ptr(lse) || !ok_ptr(idx) ||
      !ok_ptr(cnt) || !ok_ptr(dq) || !ok_ptr(dk) || !ok_ptr(dv) || !aligned16(d_slopes))
    return BSATTN_ERR_INVALID_ARG;
  bsattn_status s = check_mod(m);
  if (s) return s;
  if (d_slopes && !m->slopes) return BSATTN_ERR_INVALID_ARG;
  if (p->desc.qk_fp8) return BSATTN_ERR_UNSUPPORTED;
  Carve size(nullptr);
  carve_backward_mod(p, size);
  if (!ws || !aligned16(ws) || ws_bytes < size.off) return BSATTN_ERR_WORKSPACE;
  if ((s = check_backward_mod(p))) return s;
  DeviceGuard dev(p->device);
  if (dev.status) return dev.status;
  cudaStream_t st = (cudaStream_t)stream;
  Carve c(ws);
  const BwdModWs w = carve_backward_mod(p, c);
  if ((s = launch_doc_prep(p, m, w.doc, st))) return s;
  const ModParams d = device_mod(p, m, w.doc);
  if ((s = launch_backward(p, q, k, v, o, d_o, lse, idx, cnt, dq, dk, dv, w.b, st, &d, w.neg_lse2,
                           d_slopes ? w.slope_parts : nullptr, w.shares)))
    return s;
  if (!d_slopes) return BSATTN_OK;
  slope_sum_kernel<<<p->desc.heads, 256, 0, st>>>(w.slope_parts, p->desc.B, p->desc.heads, backward_slope_items(p),
                                                d_slopes);
  return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

bsattn_status attn_layer_mod(const bsattn_plan* p, const bsattn_rope* rope, const bsattn_score_mod* m,
                             const void* q_nat, const void* k_nat, const void* v_nat, void* o_nat, float* lse_nat,
                             int32_t* idx_out, int32_t* cnt_out, void* ws, size_t ws_bytes, void* stream) {
  if (!p || !ok_ptr(q_nat) || !ok_ptr(k_nat) || !ok_ptr(v_nat) || !ok_ptr(o_nat) || !aligned16(lse_nat) ||
      !aligned16(idx_out) || !aligned16(cnt_out) || ((idx_out == nullptr) != (cnt_out == nullptr)))
    return BSATTN_ERR_INVALID_ARG;
  bsattn_status s = BSATTN_OK;
  RopeTurns turns{};
  if (rope && (s = check_rope(p, rope, &turns))) return s;
  if (m && (s = check_mod(m))) return s;
  Carve size(nullptr);
  carve_layer_mod(p, size);
  if (!ws || !aligned16(ws) || ws_bytes < size.off) return BSATTN_ERR_WORKSPACE;
  const bool route = p->rule.kind != BSATTN_RULE_WINDOW;
  if ((s = m ? check_attention_mod(p) : check_attention(p))) return s;
  if (m && route && (s = check_scores(p))) return s;
  DeviceGuard dev(p->device);
  if (dev.status) return dev.status;
  cudaStream_t st = (cudaStream_t)stream;
  Carve c(ws);
  const LayerModWs w = carve_layer_mod(p, c);
  const Geom g = make_geom(p);
  int32_t* idx = idx_out ? idx_out : w.idx;
  int32_t* cnt = cnt_out ? cnt_out : w.cnt;
  const int32_t* doc = m ? m->doc : nullptr;
  const void *q = q_nat, *k = k_nat;
  if (m && (s = launch_doc_prep(p, m, w.doc, st))) return s;
  // Rotated copies with their tile means; documents need them too where tile
  // means or tile scales are taken, because hidden tokens must not enter those.
  if (rope || (doc && (route || p->desc.qk_fp8))) {
    if ((s = launch_rope(p, rope, turns, (const __nv_bfloat16*)q_nat, w.q, (const __nv_bfloat16*)k_nat, w.k,
                         route ? w.pq : nullptr, route ? w.pk : nullptr, false, doc, st)))
      return s;
    q = w.q;
    k = w.k;
  } else if (route) {
    if ((s = launch_pool(g, (const __nv_bfloat16*)q, w.pq, (const __nv_bfloat16*)k, w.pk, st))) return s;
  }
  const ModParams d = m ? device_mod(p, m, w.doc) : ModParams{};
  if (route) {
    if ((s = launch_block_scores(g, w.pq, w.pk, p->scale, w.S, p->d_err, st))) return s;
    if (m && (s = launch_mod_scores(p, d, w.S, w.S, st))) return s;
  }
  if ((s = attn_select_from_scores(p, w.S, idx, cnt, stream))) return s;
  const void *qa = q, *ka = k;
  if (p->desc.qk_fp8) {
    if ((s = launch_reorder_quant(g, (const __nv_bfloat16*)q, (const __nv_bfloat16*)k, w.qc, w.kc, w.qs, w.ks, st)))
      return s;
    qa = w.qc;
    ka = w.kc;
  }
  if (m)
    return launch_attention_mod(p, d, qa, ka, w.qs, w.ks, (const __nv_bfloat16*)v_nat, idx, cnt, (__nv_bfloat16*)o_nat,
                                lse_nat, w.parts, st, AttnLayout::Natural);
  return launch_attention(p, qa, ka, w.qs, w.ks, (const __nv_bfloat16*)v_nat, idx, cnt, (__nv_bfloat16*)o_nat, lse_nat,
                          nullptr, 0, st, AttnLayout::Natural);
}

}  // extern "C"
