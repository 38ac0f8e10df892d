// chunk_plan.cuh — how the work on a ragged chunk is cut: every row has tiles
// (of its queries, or of its cached tokens), every tile blocks, and the batch
// is a line of (KV head, tile, block) units of which each CTA takes a range.
#pragma once

#include <cstdint>

#include "chunk_device.cuh"

namespace pkv {

constexpr int kPlanThreads = 384;  // the first threads of a CTA make its plan
constexpr int kPlanWarps = kPlanThreads / 32;

// What a kernel tells the plan (Geo below):
//   int tiles(const RowInfo&)                 tiles of a row
//   int blocks(const RowInfo&, int F, int t)  blocks of its tile t
//   weight(const RowInfo&, int t)             units of each of its blocks
//   kMostWeight                               the largest weight
//   lead(int weight)                          units a tile costs besides its
//                                             blocks, at least kMostWeight
// F is prefix_lens[i], or 0 without.

// A place in the work: tile `tile` (counted over the batch; tile t of row i)
// for KV head h, and the block `off` that comes next.  The end of all work is
// {n_kv, 0, .., 0}.
struct Place {
  int h, tile, i, t, off;
};
__device__ __forceinline__ bool before(const Place& a, const Place& b) {
  return a.h != b.h ? a.h < b.h : a.tile != b.tile ? a.tile < b.tile : a.off < b.off;
}

// Exclusive prefix sum over the first kPlanThreads threads and its total (any
// further threads call it too, with 0); `tmp` holds kPlanWarps values.  Ends
// with a barrier.
template <typename T>
__device__ __forceinline__ T cta_scan(T x, T* tmp, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31 && warp < kPlanWarps) tmp[warp] = v;
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

// The block that comes next at unit u of a tile.
__device__ __forceinline__ int block_of(unsigned u, unsigned lead, unsigned w) {
  return u < lead ? 0 : static_cast<int>((u - lead) / w);
}
struct PlanScratch {
  long long wide[kPlanWarps];
  int narrow[kPlanWarps];
};
__device__ __forceinline__ int row_of_tile(const int* tile_start, int rows, int x) {
  int lo = 0, hi = rows;  // the last row that starts at or before tile x
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile_start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// The plan of the call, made by every CTA (all its threads, kPlanThreads or
// more, call it; `tile_start` holds num_rows + 1 ints and may be reused
// afterwards).  The U units of the batch are cut into C = min(chunks, U /
// kMostWeight) ranges, range k from floor(k U / C), so that no two boundaries
// fall on one block.  A boundary less than `snap` blocks from an end of its tile
// moves there, since a split tile costs a partial state and its merge (1: none
// does, a boundary being at a block's start).  Writes the boundaries blockIdx.x
// and blockIdx.x + 1 to bounds[0], bounds[1], and returns the number of tiles.
// The threads share out the tiles in contiguous runs, so that their work is the
// same whatever the rows' lengths.
template <typename Geo>
__device__ __forceinline__ int chunk_plan(const ChunkRows& rows, int n_kv, const Geo& geo, const int32_t* prefix_lens,
                                          int chunks, int snap, int* tile_start, PlanScratch* tmp, Place* bounds) {
  const int tid = threadIdx.x;
  const int per = (rows.num_rows + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(tid * per, rows.num_rows), r1 = min(r0 + per, rows.num_rows);
  int mine = 0;
  for (int i = r0; i < r1; ++i) {
    const int n = geo.tiles(row_info(rows, i, nullptr));
    tile_start[i] = n;
    mine += n;
  }
  int T;
  int pre = cta_scan(mine, tmp->narrow, T);
  for (int i = r0; i < r1; ++i) {
    const int n = tile_start[i];
    tile_start[i] = pre;
    pre += n;
  }
  if (tid == 0) tile_start[rows.num_rows] = T;
  if (tid < 2) bounds[tid] = Place{n_kv, 0, 0, 0, 0};
  __syncthreads();
  // this thread's run of tiles
  const int run = (T + kPlanThreads - 1) / kPlanThreads;
  const int a = min(tid * run, T), b = min(a + run, T);
  const int i0 = a < b ? row_of_tile(tile_start, rows.num_rows, a) : 0;
  long long cost = 0;
  {
    int i = i0, seen = -1, F = 0;
    RowInfo r{0, 0, 0};
    for (int x = a; x < b; ++x) {
      while (x >= tile_start[i + 1]) ++i;
      if (i != seen) {
        r = row_info(rows, i, nullptr);
        F = prefix_lens ? __ldg(prefix_lens + i) : 0;
        seen = i;
      }
      const int w = geo.weight(r, x - tile_start[i]);
      cost += geo.lead(w) + w * geo.blocks(r, F, x - tile_start[i]);
    }
  }
  long long U1;
  const long long first = cta_scan(cost, tmp->wide, U1);
  const long long U = U1 * n_kv;
  const long long C = min(static_cast<long long>(chunks), U / Geo::kMostWeight);
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    const long long k = static_cast<long long>(blockIdx.x) + e;
    if (k >= C) continue;  // at or behind the end
    // in 32 bits where they hold the products: a division of 64-bit integers is
    // a software routine of some 500 cycles
    long long u;
    int h;
    if (U < (1ll << 31) / 4096) {
      u = static_cast<int>(k) * static_cast<int>(U) / static_cast<int>(C);
      h = static_cast<int>(u) / static_cast<int>(U1);
    } else {
      u = k * U / C;
      h = static_cast<int>(u / U1);
    }
    const long long rem = u - h * U1;
    if (rem < first || rem >= first + cost) continue;
    long long at = first;
    int i = i0;
    for (int x = a; x < b; ++x) {
      while (x >= tile_start[i + 1]) ++i;
      const int F = prefix_lens ? __ldg(prefix_lens + i) : 0;
      const RowInfo r = row_info(rows, i, nullptr);
      const int w = geo.weight(r, x - tile_start[i]), nb = geo.blocks(r, F, x - tile_start[i]);
      const long long units = geo.lead(w) + static_cast<long long>(w) * nb;
      if (rem < at + units) {
        Place p{h, x, i, x - tile_start[i], block_of(static_cast<unsigned>(rem - at), geo.lead(w), w)};
        if (p.off < snap) {
          p.off = 0;
        } else if (nb - p.off < snap) {  // the next tile's start
          p.off = 0;
          if (++p.tile == T) {
            p.tile = 0;
            ++p.h;
          }
          p.i = row_of_tile(tile_start, rows.num_rows, p.tile);
          p.t = p.tile - tile_start[p.i];
        }
        bounds[e] = p;
        break;
      }
      at += units;
    }
  }
  __syncthreads();
  return T;
}

// The same for a few rows of a few tiles each (num_rows <= 32), by one warp, a
// row per lane, without shared memory or barriers: 1700 cycles where the CTA's
// plan takes 5600, at the front of calls that last 20 us.
template <typename Geo>
__device__ __forceinline__ int chunk_plan_warp(const ChunkRows& rows, int n_kv, const Geo& geo,
                                               const int32_t* prefix_lens, int chunks, int snap, Place& begin,
                                               Place& end) {
  const int lane = threadIdx.x & 31;
  RowInfo r{0, 0, -1};
  int F = 0;
  if (lane < rows.num_rows) {
    r = row_info(rows, lane, nullptr);
    if (prefix_lens) F = __ldg(prefix_lens + lane);
  }
  const int n = r.L >= 0 ? geo.tiles(r) : 0;
  long long cost = 0;
  for (int t = 0; t < n; ++t) {
    const int w = geo.weight(r, t);
    cost += geo.lead(w) + w * geo.blocks(r, F, t);
  }
  int tiles = n;
  long long units = cost;  // inclusive prefix sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, tiles, o);
    const long long y = __shfl_up_sync(kFull, units, o);
    if (lane >= o) {
      tiles += x;
      units += y;
    }
  }
  const int T = __shfl_sync(kFull, tiles, 31);
  const long long U1 = __shfl_sync(kFull, units, 31), U = U1 * n_kv,
                  C = min(static_cast<long long>(chunks), U / Geo::kMostWeight);
#pragma unroll 1
  for (int e = 0; e < 2; ++e) {
    Place p{n_kv, 0, 0, 0, 0};
    const long long k = static_cast<long long>(blockIdx.x) + e;
    if (k < C) {
      long long u;
      if (U < (1ll << 31) / 4096) {
        u = static_cast<int>(k) * static_cast<int>(U) / static_cast<int>(C);
        p.h = static_cast<int>(u) / static_cast<int>(U1);
      } else {
        u = k * U / C;
        p.h = static_cast<int>(u / U1);
      }
      const long long rem = u - p.h * U1;
      const bool here = rem >= units - cost && rem < units;
      if (here) {  // in one lane
        long long off = rem - (units - cost);
        int t = 0, nb, w;
        while (true) {
          nb = geo.blocks(r, F, t);
          w = geo.weight(r, t);
          const long long tile = geo.lead(w) + static_cast<long long>(w) * nb;
          if (off < tile) break;
          off -= tile;
          ++t;
        }
        p.i = lane;
        p.t = t;
        p.off = block_of(static_cast<unsigned>(off), geo.lead(w), w);
        if (p.off < snap) {
          p.off = 0;
        } else if (nb - p.off < snap) {  // the next tile's start
          p.off = 0;
          ++p.t;
        }
        p.tile = tiles - n + p.t;
      }
      const int owner = __ffs(__ballot_sync(kFull, here)) - 1;
      p.tile = __shfl_sync(kFull, p.tile, owner);
      p.i = __shfl_sync(kFull, p.i, owner);
      p.t = __shfl_sync(kFull, p.t, owner);
      p.off = __shfl_sync(kFull, p.off, owner);
      if (p.tile == T) {
        p.tile = 0;
        ++p.h;
      }
      // the row of the tile, which may be the next one's first
      const unsigned at = __ballot_sync(kFull, n > 0 && tiles - n <= p.tile && p.tile < tiles);
      p.i = __ffs(at) - 1;
      p.t = p.tile - __shfl_sync(kFull, tiles - n, p.i);
    }
    if (e == 0) begin = p; else end = p;
  }
  return T;
}

// Walks the tiles of a range (one warp, all lanes): the rows are read 32 at a
// time, one per lane.
template <typename Geo>
struct Walk {
  const ChunkRows& rows;
  const Geo& geo;
  const int32_t* prefix_lens;
  int T;
  Place at, end;
  RowInfo r;  // the row of `at`
  int F;
  int base;
  RowInfo mine;
  int mineF;
  __device__ __forceinline__ Walk(const ChunkRows& rows_, const Geo& geo_, const int32_t* prefix, int T_,
                                  const Place& begin, const Place& end_)
      : rows(rows_), geo(geo_), prefix_lens(prefix), T(T_), at(begin), end(end_), base(-1) {
    if (more()) load(at.i);
  }
  __device__ __forceinline__ void load(int i) {
    if (base < 0 || i < base || i >= base + 32) {
      base = i;
      mine = RowInfo{0, 0, -1};
      mineF = 0;
      const int lane = threadIdx.x & 31;
      if (base + lane < rows.num_rows) {
        mine = row_info(rows, base + lane, nullptr);
        if (prefix_lens) mineF = __ldg(prefix_lens + base + lane);
      }
    }
    r.start = __shfl_sync(kFull, mine.start, i - base);
    r.n = __shfl_sync(kFull, mine.n, i - base);
    r.L = __shfl_sync(kFull, mine.L, i - base);
    F = __shfl_sync(kFull, mineF, i - base);
  }
  __device__ __forceinline__ bool more() const { return before(at, end); }
  // the range ends within this tile, or at its start
  __device__ __forceinline__ bool ends_here() const { return at.h == end.h && at.tile == end.tile; }
  // the tile's blocks in the range: [from, to) of its nb
  __device__ __forceinline__ int from() const { return at.off; }
  __device__ __forceinline__ int to(int nb) const { return ends_here() ? end.off : nb; }
  // to the next tile; `end` is not in the tile just left
  __device__ __forceinline__ void next() {
    at.off = 0;
    ++at.t;
    if (++at.tile == T) {
      at.tile = 0;
      ++at.h;
      at.i = 0;
      at.t = 0;
      if (!more()) return;
      load(0);
    }
    while (at.t >= geo.tiles(r)) {
      ++at.i;
      at.t = 0;
      load(at.i);
    }
  }
};

}  // namespace pkv
