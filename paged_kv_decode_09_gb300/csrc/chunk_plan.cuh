// chunk_plan.cuh — how a ragged chunk's attention is cut into work: tiles of
// queries, blocks of 128 cached tokens, and contiguous ranges of (KV head,
// tile, block) units, one range per CTA.
#pragma once

#include <cstdint>

#include "chunk_device.cuh"

namespace pkv {

constexpr int kTileRows = 256;   // (query, query head) rows of a tile: 256 / G queries
constexpr int kBlockTok = 128;   // cached tokens of a block
constexpr int kPlanThreads = 384;
constexpr int kPlanWarps = kPlanThreads / 32;

// A tile: queries tile * QT .. of a row, and the blocks they attend to.
struct TileGeom {
  int nq;    // queries
  int P0;    // position of the first
  int t_lo;  // tokens [t_lo, t_hi) that some query of the tile attends to
  int t_hi;
  int kb;    // first block
  int nb;    // blocks
};
__device__ __forceinline__ TileGeom tile_geom(const RowInfo& r, int t, int QT, int W, int F) {
  TileGeom g;
  const int j0 = t * QT;
  g.nq = min(QT, r.n - j0);
  g.P0 = r.L - r.n + j0;
  g.t_lo = seen_from(g.P0, W);
  g.t_hi = seen_to(g.P0 + g.nq - 1, r.L, F);
  g.kb = g.t_lo / kBlockTok;
  g.nb = (g.t_hi + kBlockTok - 1) / kBlockTok - g.kb;
  return g;
}
__device__ __forceinline__ int tiles_of(const RowInfo& r, int QT) { return r.L >= 0 ? (r.n + QT - 1) / QT : 0; }

// A place in the work: block `off` of tile `tile` (counted over the batch;
// tile t of row i) for KV head h.  The end of all work is {n_kv, 0, .., 0}.
struct Place {
  int h, tile, i, t, off;
};
__device__ __forceinline__ bool before(const Place& a, const Place& b) {
  return a.h != b.h ? a.h < b.h : a.tile != b.tile ? a.tile < b.tile : a.off < b.off;
}

// Exclusive prefix sum over the CTA's threads and the total; `tmp` holds
// kPlanWarps + 1 values.  Ends with a barrier.
template <typename T>
__device__ __forceinline__ T cta_scan(T x, T* tmp, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) tmp[warp] = v;
  __syncthreads();
  T pre = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) pre += tmp[w];
    sum += tmp[w];
  }
  total = sum;
  __syncthreads();
  return pre + v - x;
}

// The plan of the call, made by every CTA (kPlanThreads threads, all of them
// call it; `scratch` holds num_rows + 1 ints and may be reused afterwards).
// The U units of the batch are cut into C = min(chunks, U) ranges, range k from
// floor(k U / C); a boundary closer than `snap` blocks to an end of its tile
// moves there, since a split tile costs a partial state and its merge.  Writes
// the boundaries blockIdx.x and blockIdx.x + 1 to bounds[0], bounds[1], and
// returns the number of tiles.  A thread shares out the tiles in contiguous
// runs, so that its work is the same whatever the rows' lengths.
struct PlanScratch {
  long long wide[kPlanWarps + 1];
  int narrow[kPlanWarps + 1];
};
__device__ __forceinline__ int chunk_plan(const ChunkRows& rows, int n_kv, int QT, int W, const int32_t* prefix_lens,
                                          int chunks, int snap, int* tile_start, PlanScratch* tmp, Place* bounds) {
  const int tid = threadIdx.x;
  const int per = (rows.num_rows + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * per, rows.num_rows), r1 = min(r0 + per, rows.num_rows);
  int mine = 0;
  for (int i = r0; i < r1; ++i) mine += tiles_of(row_info(rows, i, nullptr), QT);
  int T;
  int pre = cta_scan(mine, tmp->narrow, T);
  for (int i = r0; i < r1; ++i) {
    tile_start[i] = pre;
    pre += tiles_of(row_info(rows, i, nullptr), QT);
  }
  if (tid == 0) tile_start[rows.num_rows] = T;
  if (tid < 2) bounds[tid] = Place{n_kv, 0, 0, 0, 0};
  __syncthreads();
  // this thread's run of tiles
  const int run = (T + kPlanThreads - 1) / kPlanThreads;
  const int a = min(tid * run, T), b = min(a + run, T);
  int i0 = 0;
  if (a < b) {  // the last row that starts at or before tile a
    int lo = 0, hi = rows.num_rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_start[mid] <= a) lo = mid; else hi = mid;
    }
    i0 = lo;
  }
  long long cost = 0;
  {
    int i = i0;
    RowInfo r{0, 0, 0};
    int F = 0, seen = -1;
    for (int x = a; x < b; ++x) {
      while (x >= tile_start[i + 1]) ++i;
      if (i != seen) {
        r = row_info(rows, i, nullptr);
        F = prefix_lens ? __ldg(prefix_lens + i) : 0;
        seen = i;
      }
      cost += tile_geom(r, x - tile_start[i], QT, W, F).nb;
    }
  }
  long long U1;
  const long long first = cta_scan(cost, tmp->wide, U1);
  const long long U = U1 * n_kv;
  const long long C = U < chunks ? U : chunks;
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const long long k = static_cast<long long>(blockIdx.x) + e;
    if (k >= C) continue;  // at or behind the end
    const long long u = k * U / C;
    const int h = static_cast<int>(u / U1);
    const long long rem = u - h * U1;
    if (rem < first || rem >= first + cost) continue;
    long long at = first;
    int i = i0;
    for (int x = a; x < b; ++x) {
      while (x >= tile_start[i + 1]) ++i;
      const RowInfo r = row_info(rows, i, nullptr);
      const int F = prefix_lens ? __ldg(prefix_lens + i) : 0;
      const int nb = tile_geom(r, x - tile_start[i], QT, W, F).nb;
      if (rem < at + nb) {
        Place p{h, x, i, x - tile_start[i], static_cast<int>(rem - at)};
        if (p.off < snap) {
          p.off = 0;
        } else if (nb - p.off < snap) {  // the next tile's start
          p.off = 0;
          if (++p.tile == T) {
            p.tile = 0;
            ++p.h;
          }
          // its row: the last that starts at or before it
          int lo = 0, hi = rows.num_rows;
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tile_start[mid] <= p.tile) lo = mid; else hi = mid;
          }
          p.i = lo;
          p.t = p.tile - tile_start[lo];
        }
        bounds[e] = p;
        break;
      }
      at += nb;
    }
  }
  __syncthreads();
  return T;
}

}  // namespace pkv
