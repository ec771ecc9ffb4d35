// Step lists of the attention kernels: a work item's two 64-row halves, and
// the union of their kept lists compacted to 64-row chunks.
#pragma once

#include "score_mod.cuh"

// Work item -> its two (tile, chunk) halves; i1 = -1 when the second half is
// absent. 64-token tiles: adjacent tiles along the pair axis. Tiles of several
// chunks: chunks 2b and 2b + 1 of one tile (padding-only chunks included, so
// that their rows of the tiled gradients are written, as zeros).
__device__ __forceinline__ void block_halves(const Geom& g, int pair_axis, const int* pdim, int item, int* i0,
                                             int* i1, int* c0, int* c1) {
  if (g.nchunk > 1) {
    const int per = (g.nchunk + 1) / 2;
    *i0 = *i1 = item / per;
    *c0 = 2 * (item % per);
    *c1 = *c0 + 1;
    if (*c1 >= g.nchunk) *i1 = -1;
    return;
  }
  const int nd[3] = {g.nT, g.nH, g.nW};
  int c[3], rem = item;
  c[2] = rem % pdim[2];
  rem /= pdim[2];
  c[1] = rem % pdim[1];
  c[0] = rem / pdim[1];
  c[pair_axis] *= 2;
  *i0 = (c[0] * g.nH + c[1]) * g.nW + c[2];
  c[pair_axis] += 1;
  *i1 = c[pair_axis] < nd[pair_axis] ? (c[0] * g.nH + c[1]) * g.nW + c[2] : -1;
  *c0 = *c1 = 0;
}

// Whether chunk c of tile j holds a real token (its first row is in the grid).
__device__ __forceinline__ bool chunk_is_real(const Geom& g, int j, int c) {
  const ChunkOrigin o = chunk_origin(g, c);
  const int bt = j / (g.nH * g.nW), bhh = (j / g.nW) % g.nH, bw = j % g.nW;
  return bt * g.tt + o.dt < g.T && bhh * g.th + o.dh < g.H && bw * g.tw + o.dw < g.W;
}

// Compacts the union of two tile bitmaps into the ascending step list, one
// step per real 64-row chunk of each listed tile: tile in bits 0-20, chunk in
// bits 21-29, bit 30 (31) from the first (second) bitmap; ext gets the
// chunk's real extent from its first token (t, h, w bytes, capped at 255) and
// bit 31 when the chunk has padded rows. *count = steps (capped at cap). All
// threads of the CTA take part; the block-scan scratch holds one int per warp.
template <int NT>
__device__ __forceinline__ void compact_steps(const Geom& g, const uint32_t* bmA, const uint32_t* bmB, int words,
                                              uint32_t* list, uint32_t* ext, int cap, int* scan, uint32_t* count) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int wpt = (words + NT - 1) / NT;
  const int w0 = min(tid * wpt, words), w1 = min(w0 + wpt, words);
  int mine = 0;
  for (int w = w0; w < w1; ++w) {
    uint32_t bits = bmA[w] | bmB[w];
    if (g.nchunk == 1) {
      mine += __popc(bits);
    } else {
      while (bits) {
        const int j = w * 32 + __ffs(bits) - 1;
        for (int c = 0; c < g.nchunk; ++c) mine += chunk_is_real(g, j, c) ? 1 : 0;
        bits &= bits - 1;
      }
    }
  }
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  int off = 0, tot = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    off += i < warp ? scan[i] : 0;
    tot += scan[i];
  }
  int pos = off + x - mine;
  for (int w = w0; w < w1; ++w) {
    const uint32_t a = bmA[w], bb = bmB[w];
    uint32_t bits = a | bb;
    while (bits) {
      const int bit = __ffs(bits) - 1;
      bits &= bits - 1;
      const int j = w * 32 + bit;
      const uint32_t e = (uint32_t)j | (((a >> bit) & 1u) << 30) | (((bb >> bit) & 1u) << 31);
      const int bt = j / (g.nH * g.nW), bhh = (j / g.nW) % g.nH, bw = j % g.nW;
      for (int c = 0; c < g.nchunk; ++c) {
        if (g.nchunk > 1 && !chunk_is_real(g, j, c)) continue;
        if (pos < cap) {
          const ChunkOrigin o = chunk_origin(g, c);
          const int vt = min(g.T - bt * g.tt - o.dt, 255), vh = min(g.H - bhh * g.th - o.dh, 255),
                    vw = min(g.W - bw * g.tw - o.dw, 255);
          const bool edge = vt < g.ct || vh < g.ch || vw < g.cw || g.cr < 64;
          list[pos] = e | ((uint32_t)c << 21);
          ext[pos] = (uint32_t)vt | ((uint32_t)vh << 8) | ((uint32_t)vw << 16) | (edge ? 1u << 31 : 0u);
        }
        ++pos;
      }
    }
  }
  if (tid == 0) *count = (uint32_t)min(tot, cap);
}

// The same for mod::filter_steps, which looks at every entry anyway: chunks
// of padding are listed too, and no coordinates are formed, so that a thread
// only counts and writes. It takes the bitmaps by bytes: a dense list's words
// would keep a few threads busy with 32 entries each.
template <int NT>
__device__ __forceinline__ void list_steps(const Geom& g, const uint32_t* bmA, const uint32_t* bmB, int words,
                                           uint32_t* list, int cap, int* scan, uint32_t* count) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nb = 4 * words, per = (nb + NT - 1) / NT;
  const int b0 = min(tid * per, nb), b1 = min(b0 + per, nb);
  int mine = 0;
  for (int q = b0; q < b1; ++q) mine += __popc(((bmA[q >> 2] | bmB[q >> 2]) >> (8 * (q & 3))) & 0xffu) * g.nchunk;
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scan[warp] = x;
  __syncthreads();
  int pos = x - mine, tot = 0;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) {
    pos += i < warp ? scan[i] : 0;
    tot += scan[i];
  }
  for (int q = b0; q < b1; ++q) {
    const uint32_t a = (bmA[q >> 2] >> (8 * (q & 3))) & 0xffu, b = (bmB[q >> 2] >> (8 * (q & 3))) & 0xffu;
    for (uint32_t bits = a | b; bits; bits &= bits - 1) {
      const int bit = __ffs(bits) - 1;
      const uint32_t e = (uint32_t)(8 * q + bit) | (((a >> bit) & 1u) << 30) | (((b >> bit) & 1u) << 31);
      for (int c = 0; c < g.nchunk; ++c, ++pos)
        if (pos < cap) list[pos] = e | ((uint32_t)c << 21);
    }
  }
  if (tid == 0) *count = (uint32_t)min(tot, cap);
}

// Turns the first part of an ascending list, the steps up to the block's first
// query tile, around: a walk then starts there and leaves it in both
// directions, so that under a distance bias the nearest keys come first and a
// row's reference, set by its first keys, seldom has to move. (Rows of the
// block's second tile start at their neighbour.)
template <int NT>
__device__ __forceinline__ void nearest_first(uint32_t* list, uint32_t* ext, int steps, int tile) {
  int lo = 0, hi = steps;  // steps of tiles <= tile
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if ((int)(list[mid] & 0x1FFFFFu) <= tile) lo = mid + 1;
    else hi = mid;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < lo / 2; e += NT) {
    const int f = lo - 1 - e;
    const uint32_t a = list[e], x = ext[e];
    list[e] = list[f];
    ext[e] = ext[f];
    list[f] = a;
    ext[f] = x;
  }
  __syncthreads();
}

// Brings one of `shares` equal parts of the list to its front; returns its steps.
template <int NT>
__device__ __forceinline__ int take_share(uint32_t* list, uint32_t* ext, int steps, int share, int shares) {
  const int lo = steps * share / shares, n = steps * (share + 1) / shares - lo;
  for (int base = 0; lo > 0 && base < n; base += NT) {
    const int i = base + threadIdx.x;
    uint32_t e = 0, x = 0;
    if (i < n) {
      e = list[lo + i];
      x = ext[lo + i];
    }
    __syncthreads();
    if (i < n) {  // entries of later rounds lie behind this round's places
      list[i] = e;
      ext[i] = x;
    }
    __syncthreads();
  }
  return n;
}

// Score rules: a chunk's row offsets, and every chunk's in-tile origin
// (packed 10 bits per axis), so that a step needs no division.
struct ModTab {
  mod::Table col;
  uint32_t origin[kMaxChunks];
  __device__ __forceinline__ ChunkOrigin at(int c) const { return mod::unpack_origin(origin[c]); }
};
template <int NT>
__device__ __forceinline__ void fill_modtab(const Geom& g, ModTab* tab, const uint32_t* colc) {
  mod::fill_table<NT>(g, &tab->col, colc);
  for (int c = threadIdx.x; c < g.nchunk; c += NT) {
    const ChunkOrigin o = mod::origin_of(g, c);
    tab->origin[c] = (uint32_t)o.dt | ((uint32_t)o.dh << 10) | ((uint32_t)o.dw << 20);
  }
}
