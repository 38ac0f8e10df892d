// attention_mass.cu — paged_attention_mass: the softmax weight that each cached
// token receives from a chunk's queries, on the fifth-generation tensor cores
// (tcgen05, accumulators in tensor memory).
//
// With the lse of each (query, query head) row known, the weights need no
// running maximum and no second pass: for 128 cached tokens and 128 rows c,
//     S = K Q^T             128 tokens x 128 rows, K the first operand
//     sum_t += sum_c 2^(y(S[t][c]) - lse2_c)
// so a token is a lane of tensor memory and a thread sums its own token's
// weights: no exchange between threads, and a fixed order of additions.  The
// K of 256 tokens of one (row, KV head) (a tile, in two halves m of 128) stay
// in shared memory while the row's queries stream past, 128 rows a block.
// q8_0 keys enter as two f16 parts, hi and lo (q8_tiles.cuh), two products.  A
// token with a value beyond f16's range gets a sum that is not a number; it is
// left out, and summed in fp32 after the pipeline has drained (mend_tokens).
// Such tokens are rare, and looking for them earlier costs every call: votes of
// the splitting warps 49 -> 51.5 us for the last queries' call, a warp of its own
// 58.7; scaling them down for the products and their scores back up 186 -> 194
// for whole chunks.
//
// Warps: 0-3 and 4-7 sum the weights of half 0 and 1, 8 walks the work, 9
// issues the products, 10 copies K pages, 11 copies queries and stages their
// lse; with q8_0, 12-15 split the codes instead of warp 10.  Each half has two
// score buffers (all 512 columns of tensor memory), so that the products run
// ahead of the exponentials.  A block of 256 x 128 takes 1024 cycles of
// products and as many of exponentials (four cycles a warp's row each), and in
// fact some 2500: two warps a scheduler take 450 cycles for a group of 32
// columns, four warps a scheduler (the columns shared out) no less in all.  Two
// chunks of 1800 tokens over 5600 and 4500: 158 us, 775 TFLOP/s; the last 32
// queries of four rows of 5K to 23K tokens, which K's bytes bound (15 us): 28.5.
//
// The work is the line of (KV head, tile, block) units of chunk_plan.cuh; a
// tile cut by a boundary leaves its 256 partial sums in the workspace, which
// the second kernel adds in order.
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "attend_row.cuh"
#include "chunk_device.cuh"
#include "chunk_plan.cuh"
#include "q8_tiles.cuh"
#include "score32.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kMassTok = 256;                        // tokens of a tile
constexpr uint32_t kBuf = 32768;                     // 128 tokens or 128 query rows
constexpr int kKBufs = 4;                            // K buffers (q8_0: two of hi and lo)
constexpr int kQSlots = 2;
constexpr int kLseSlots = 4;
constexpr int kTileCost = 1;  // units of a tile besides its blocks (chunk_plan)
constexpr uint32_t kQRing = kKBufs * kBuf;
constexpr uint32_t kMassTail = kQRing + kQSlots * kBuf;
constexpr int kDescs = 4;

enum : int {
  kBKFull = 0,
  kBKEmpty = kBKFull + kKBufs,
  kBQFull = kBKEmpty + kKBufs,
  kBQEmpty = kBQFull + kQSlots,
  kBQLand = kBQEmpty + kQSlots,  // queries that are cleared behind the row's
  kBLse = kBQLand + 1,
  kBLseEmpty = kBLse + kLseSlots,
  kBS = kBLseEmpty + kLseSlots,  // [half][buffer]
  kBSFree = kBS + 4,
  kBDesc = kBSFree + 4,
  kBDescEmpty = kBDesc + kDescs,
  kBDrain = kBDescEmpty + kDescs,
  kBStall,
  kNumBars,
};

// A piece: blocks b0 .. b0 + nb - 1 (128 rows of queries each) of one tile.
struct Piece {
  int i, h, t0;     // row, KV head, first token
  int tok, nq, P0;  // first query that counts: its token, how many, its position
  int L, n, F;
  int b0, nb;
  int slot;  // partial slot, -1: the whole tile
  int last;
  int pad[3];
};
static_assert(sizeof(Piece) == 64, "");

struct Tail {
  uint64_t bars[kNumBars];
  Piece piece[kDescs];
  alignas(16) float lse2[kLseSlots][128];  // minus the lse of a block's rows in base 2, -inf: not counted
  int odd[kLseSlots];          // the block has a row that is not counted
  volatile int ctl[2];  // abort; q8_0: sums were left out
  uint32_t tmem;
  int tiles;        // of the batch
  Place bounds[2];  // the CTA's range
  PlanScratch scratch;
  int tile_start[PKV_MAX_ROWS + 1];
};
constexpr size_t kSmemBytes = 1024 + kMassTail + sizeof(Tail);
static_assert(offsetof(Tail, lse2) % 16 == 0 && kMassTail % 16 == 0, "read four at a time");
static_assert(kSmemBytes <= 232448, "");

// Tokens t * 256 .. of a row, and the blocks of the queries that attend to
// any of them (a tile without any still has its weights carried over).
struct TokenTiles {
  int QT, W, last, stride;
  __device__ __forceinline__ int tiles(const RowInfo& r) const {
    return r.L >= 0 && r.L <= stride ? (r.L + kMassTok - 1) / kMassTok : 0;
  }
  __device__ __forceinline__ int first_query(const RowInfo& r) const { return last > 0 ? max(0, r.n - last) : 0; }
  // blocks [b0, b1) of 128 / G queries from first_query on
  __device__ __forceinline__ void range(const RowInfo& r, int F, int t, int& b0, int& b1) const {
    const int t0 = t * kMassTok, past = r.L - r.n, j0 = first_query(r);
    const int ja = t0 < F ? j0 : max(j0, t0 - past);
    const long long end = W > 0 ? static_cast<long long>(min(t0 + kMassTok, r.L)) - 1 + W - past : r.n;
    const int jb = static_cast<int>(min(static_cast<long long>(r.n), end));
    b0 = b1 = 0;
    if (ja < jb) {
      b0 = (ja - j0) / QT;
      b1 = (jb - 1 - j0) / QT + 1;
    }
  }
  __device__ __forceinline__ int blocks(const RowInfo& r, int F, int t) const {
    int b0, b1;
    range(r, F, t, b0, b1);
    return b1 - b0;
  }
  static constexpr int kMostWeight = 1;
  __device__ __forceinline__ int weight(const RowInfo&, int) const { return 1; }
  __device__ __forceinline__ int lead(int) const { return kTileCost; }
};

struct Rec {
  int inside;  // the boundary cuts a tile
  int h, tile, i, t0, L, n, pad;
};
__host__ __device__ inline size_t rec_bytes(int chunks) {
  return (static_cast<size_t>(chunks + 1) * sizeof(Rec) + 255) & ~size_t(255);
}
__device__ __forceinline__ float* slot_sums(const MassArgs& a, int slot) {
  return reinterpret_cast<float*>(a.workspace + rec_bytes(a.chunks)) + static_cast<size_t>(slot) * kMassTok;
}

template <int DT>
constexpr int kMassThreads = DT == PKV_KV_Q8_0 ? 512 : 384;

// The partial slot of blocks [from, to) of a tile's in this CTA's range, -1: all.
__device__ __forceinline__ int slot_of(int from, int to, int blocks) {
  const int cta = static_cast<int>(blockIdx.x);
  return from > 0 ? 2 * cta : to < blocks ? 2 * cta + 1 : -1;
}

// The sum of token t of row i (of L tokens, n of them new) and KV head h, over
// a whole tile or the part of it in `slot`.
__device__ __forceinline__ void store_sum(const MassArgs& a, int slot, int i, int h, int t, int L, int n, float sum) {
  if (slot >= 0) {
    slot_sums(a, slot)[t % kMassTok] = sum;
  } else {
    const long long at = (static_cast<long long>(i) * a.pool.n_kv + h) * a.mass_stride + t;
    a.mass_out[at] = (a.mass_in && t < L - n ? a.mass_in[at] : 0.0f) + sum;
  }
}

// Token t of row i as a row of 128 dims in the pool's layer, for KV head h.
__device__ __forceinline__ long long token_row(const MassArgs& a, int i, int h, int t) {
  int pg = __ldg(a.rows.block_table + static_cast<long long>(i) * a.rows.bt_stride + t / kPage);
  if (pg < 0 || pg >= a.pool.num_pages) pg = 0;  // as the products read it
  return (static_cast<long long>(pg) * a.pool.n_kv + h) * kPage + t % kPage;
}

// Dims 4 u .. 4 u + 3 of a q8_0 token; one is beyond what q8_split8 takes (as
// one that is not finite is).
__device__ __forceinline__ bool key4(const MassArgs& a, long long row, int u, float (&k)[4]) {
  const float scale = __half2float(__ldg(reinterpret_cast<const __half*>(a.pool.k_scales) + 4 * row + (u >> 3)));
  const uint32_t codes = __ldg(reinterpret_cast<const uint32_t*>(a.pool.k_data + row * kD) + u);
  bool beyond = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    k[e] = scale * (static_cast<float>((codes >> (8 * e)) & 255u) - 128.0f);
    beyond = beyond || !(fabsf(k[e]) < 65520.0f);
  }
  return beyond;
}

// A thread's token t has such a value: its sum is left to mend_tokens.  (Where no
// query attends to the token its sum is 0, in both.)
__device__ __noinline__ bool token_beyond(const MassArgs& a, int i, int h, int t) {
  const long long row = token_row(a, i, h, t);
  bool beyond = false;
#pragma unroll 1
  for (int u = 0; u < kD / 4; ++u) {
    float k[4];
    beyond = key4(a, row, u, k) || beyond;
  }
  return beyond;
}

// The sums of such tokens over the range [begin, end), in fp32 from the stored
// codes: a token by each warp of the CTA (all of them call it), 4 dims a lane.
__device__ __noinline__ void mend_tokens(const MassArgs& a, const TokenTiles& geo, const Place& begin,
                                         const Place& end, int T) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int G = a.n_q / a.pool.n_kv;
  Walk<TokenTiles> w(a.rows, geo, a.sc.prefix_lens, T, begin, end);
  while (w.more()) {
    const RowInfo& r = w.r;
    const int i = w.at.i, h = w.at.h;
    int b0, b1;
    geo.range(r, w.F, w.at.t, b0, b1);
    const int from = w.from(), to = w.to(b1 - b0), slot = slot_of(from, to, b1 - b0);
    const int j0 = geo.first_query(r) + (b0 + from) * geo.QT, j1 = min(r.n, j0 + (to - from) * geo.QT);
#pragma unroll 1
    for (int t = w.at.t * kMassTok + warp; to > from && t < min(r.L, (w.at.t + 1) * kMassTok); t += warps) {
      float k[4];
      if (!__any_sync(kFull, key4(a, token_row(a, i, h, t), lane, k))) continue;
      // 32 (query, head) columns at a time, whose loads go out together; lane u
      // weighs column u and sums its own
      float sum = 0.0f, lost = 0.0f;
#pragma unroll 1
      for (int c0 = j0 * G; c0 < j1 * G; c0 += 32) {
        const int c = c0 + lane, j = c / G, g = h * G + c % G, P = r.L - r.n + j;
        float lse = INFINITY, mine = 0.0f;
        if (c < j1 * G && t >= seen_from(P, geo.W) && t < seen_to(P, r.L, w.F))
          lse = __ldg(a.lse + static_cast<long long>(r.start + j) * a.n_q + g);
        const bool counts = fabsf(lse) <= 3.0e38f;
        if (!__any_sync(kFull, counts)) continue;
        const int n = min(32, j1 * G - c0);
#pragma unroll 8
        for (int u = 0; u < n; ++u) {
          const int cu = c0 + u;
          const uint2 q = __ldg(reinterpret_cast<const uint2*>(
              a.q + ((r.start + cu / G) * a.q_stride + static_cast<long long>(h * G + cu % G) * kD + 4 * lane) * 2));
          const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&q.x));
          const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&q.y));
          float dot = fmaf(hi.y, k[3], fmaf(hi.x, k[2], fmaf(lo.y, k[1], lo.x * k[0])));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
          mine = u == lane ? dot : mine;
        }
        if (counts) {
          const float s =
              score2(mine, a.sc.scale, a.sc.softcap, a.sc.slopes ? __ldg(a.sc.slopes + g) : 0.0f, abs(P - t));
          const float y = exp2f(s - lse * kLog2e) - lost, z = sum + y;
          lost = (z - sum) - y;
          sum = z;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (lane == 0) store_sum(a, slot, i, h, t, r.L, r.n, sum);
    }
    if (w.ends_here()) break;
    w.next();
  }
}

// GEN: 0 plain scores; 1 capped; 2 with a distance bias, capped or not.
template <int DT, int GEN>
__global__ void __launch_bounds__(kMassThreads<DT>, 1)
    attention_mass_kernel(const __grid_constant__ MassArgs a, const __grid_constant__ TileMaps maps,
                          const __grid_constant__ CUtensorMap qmap) {
  constexpr bool kQ8 = DT == PKV_KV_Q8_0;
  constexpr int kNB = kQ8 ? kKBufs / 2 : kKBufs;           // K buffers, and their bytes
  constexpr uint32_t kKBytes = kQ8 ? 2 * kBuf : kBuf;
  constexpr int kReaders = 8 + 1 + 1 + (kQ8 ? 4 : 1);      // sums, products, queries, keys
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Tail& tail = *reinterpret_cast<Tail*>(smem + kMassTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = smem_addr(tail.bars);
  auto bar = [&](int b) { return bars + 8u * static_cast<uint32_t>(b); };
  volatile int* ctl = tail.ctl;
  const int G = a.n_q / a.pool.n_kv, QT = 128 / G;

  if (tid == 0) {
    prefetch_tensormap(&maps.kp);
    prefetch_tensormap(&qmap);
    tail.ctl[0] = 0;
    tail.ctl[1] = 0;
  }
  if (tid < kNumBars) {
    const int b = tid;
    int count = 1;
    if (b < kBKEmpty && kQ8) count = 4;
    if (b >= kBLseEmpty && b < kBS) count = 8;
    if (b >= kBSFree && b < kBDesc) count = 4;
    if (b >= kBDescEmpty && b < kBDrain) count = kReaders;
    mbar_init(bar(b), count);
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tail.tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc::fence_before();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const TokenTiles geo{QT, a.pool.window, a.last_queries, a.mass_stride};
  // a small call's plan is made by the one warp that walks the work
  const bool small = a.rows.num_rows <= 32 && min(a.mass_stride, a.rows.bt_stride * kPage) <= 16 * kMassTok;
  int T = 0;
  if (small)
    __syncthreads();
  else
    T = chunk_plan(a.rows, a.pool.n_kv, geo, a.sc.prefix_lens, a.chunks, 1, tail.tile_start, &tail.scratch,
                           tail.bounds);
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tail.tmem);
  Place begin = tail.bounds[0], end = tail.bounds[1];  // of a small call: made by warp 8
  if (warp == 8) {  // before the test hook: the merge reads every range's record
    if (small) T = chunk_plan_warp(a.rows, a.pool.n_kv, geo, a.sc.prefix_lens, a.chunks, 1, begin, end);
    if (lane == 0) {  // the range, for mend_tokens, and the boundary at its start, for the merge
      tail.tiles = T;
      tail.bounds[0] = begin;
      tail.bounds[1] = end;
      Rec x{};
      x.inside = begin.h < a.pool.n_kv && begin.off > 0;
      if (x.inside) {
        const RowInfo r = row_info(a.rows, begin.i, nullptr);
        x.h = begin.h;
        x.tile = begin.tile;
        x.i = begin.i;
        x.t0 = begin.t * kMassTok;
        x.L = r.L;
        x.n = r.n;
      }
      reinterpret_cast<Rec*>(a.workspace)[blockIdx.x] = x;
    }
    __syncwarp();
  }
  const bool stalled = test_stall(bar(kBStall), a.pool.test_stall_ns, ctl, a.pool.status);

  auto wait = [&](int b, uint32_t parity) { return tc::warp_wait(bar(b), parity & 1u, ctl, a.pool.status); };

  if (stalled) {
    // test hook: every warp gave up
  } else if (warp == 8) {
    // ------------------------------------------------------------- pieces ----
    Walk<TokenTiles> w(a.rows, geo, a.sc.prefix_lens, T, begin, end);
    int p = 0;
    bool ok = true;
    while (w.more()) {
      const RowInfo& r = w.r;
      int b0, b1;
      geo.range(r, w.F, w.at.t, b0, b1);
      const int from = w.from(), to = w.to(b1 - b0);
      const int x = p % kDescs;
      if (p >= kDescs && !(ok = wait(kBDescEmpty + x, p / kDescs - 1))) break;
      if (lane == 0) {
        Piece& d = tail.piece[x];
        const int j0 = geo.first_query(r);
        d.i = w.at.i;
        d.h = w.at.h;
        d.t0 = w.at.t * kMassTok;
        d.tok = r.start + j0;
        d.nq = r.n - j0;
        d.P0 = r.L - r.n + j0;
        d.L = r.L;
        d.n = r.n;
        d.F = w.F;
        d.b0 = b0 + from;
        d.nb = to - from;
        d.slot = slot_of(from, to, b1 - b0);
        d.last = 0;
        mbar_arrive(bar(kBDesc + x));
      }
      __syncwarp();
      ++p;
      if (w.ends_here()) break;
      w.next();
    }
    if (ok) {
      const int x = p % kDescs;
      if (p < kDescs || wait(kBDescEmpty + x, p / kDescs - 1)) {
        if (lane == 0) {
          tail.piece[x].last = 1;
          mbar_arrive(bar(kBDesc + x));
        }
        __syncwarp();
      }
    }
    // rows that are skipped, once each
    for (int i = blockIdx.x * 32 + lane; i < a.rows.num_rows; i += gridDim.x * 32) {
      const RowInfo r = row_info(a.rows, i, a.pool.status);
      if (r.L > a.mass_stride) record_status(a.pool.status, PKV_DEV_BAD_LENGTH);
    }
  } else if (!kQ8 && warp == 10) {
    // ------------------------------------------------------------ K pages ----
    int kp = 0;  // K buffers filled
    uint32_t my_bar = 0, my_par = 0;
    bool ok = true;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      if (d.nb > 0) {
        const int32_t* bt = a.rows.block_table + static_cast<long long>(d.i) * a.rows.bt_stride;
        const int first = d.t0 / kPage, np = min(kMassTok / kPage, (d.L + kPage - 1) / kPage - first);
        int pg = lane < np ? __ldg(bt + first + lane) : 0;
        if (lane < np && (pg < 0 || pg >= a.pool.num_pages)) {
          record_status(a.pool.status, PKV_DEV_BAD_PAGE);
          pg = 0;
        }
#pragma unroll
        for (int m = 0; m < 2; ++m, ++kp) {
          const int s = kp % kNB;
          if (kp >= kNB && !(ok = wait(kBKEmpty + s, kp / kNB - 1))) break;
          const int n = max(0, min(8, np - 8 * m));
          if (lane == s) {
            my_bar = bar(kBKFull + s);
            my_par = static_cast<uint32_t>(kp / kNB) & 1u;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(kBKFull + s), static_cast<uint32_t>(n) * 4096u);
          __syncwarp();
          const int q = lane - 8 * m;
          if (q >= 0 && q < n) tc::load_tile(sbase + s * kBuf + q * 4096u, &maps.kp, pg * a.pool.n_kv + d.h, bar(kBKFull + s));
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
    }
    const int zero = 0;
    if (my_bar) mbar_wait_bounded(my_bar, my_par, &zero);
    __syncwarp();
  } else if (kQ8 && warp >= 12) {
    // ------------------------------------------- q8_0 keys as two f16 parts ----
    const int u = tid - 384;           // 8 threads a token, 16 codes each
    const int row = u >> 3, col = u & 7;
    int kp = 0;
    bool ok = true;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      if (d.nb > 0) {
        const int32_t* bt = a.rows.block_table + static_cast<long long>(d.i) * a.rows.bt_stride;
        const int first = d.t0 / kPage, np = min(kMassTok / kPage, (d.L + kPage - 1) / kPage - first);
        int pg = lane < np ? __ldg(bt + first + lane) : 0;
        if (lane < np && (pg < 0 || pg >= a.pool.num_pages)) {
          record_status(a.pool.status, PKV_DEV_BAD_PAGE);
          pg = 0;
        }
#pragma unroll 1
        for (int m = 0; m < 2; ++m, ++kp) {
          const int s = kp % kNB;
          uint4 code[8];
          __half sc[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {  // page 8 m + e, its token `row`
            const int pe = __shfl_sync(kFull, pg, 8 * m + e);
            code[e] = make_uint4(0u, 0u, 0u, 0u);
            sc[e] = __float2half_rn(0.0f);
            if (8 * m + e < np) {
              const long long at = (static_cast<long long>(pe) * a.pool.n_kv + d.h) * kPage + row;
              code[e] = __ldg(reinterpret_cast<const uint4*>(a.pool.k_data + at * kD) + col);
              sc[e] = __ldg(reinterpret_cast<const __half*>(a.pool.k_scales) + at * (kD / kQBlock) + (col >> 1));
            }
          }
          if (kp >= kNB && !(ok = wait(kBKEmpty + s, kp / kNB - 1))) break;
          uint8_t* hi = smem + s * kKBytes;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2 s2 = __half2half2(sc[e]);
            uint4 h0, l0, h1, l1;
            q8_split8(make_uint2(code[e].x, code[e].y), s2, h0, l0);
            q8_split8(make_uint2(code[e].z, code[e].w), s2, h1, l1);
            const uint32_t o0 = tile_vec(16 * e + row, 2 * col), o1 = tile_vec(16 * e + row, 2 * col + 1);
            *reinterpret_cast<uint4*>(hi + o0) = h0;
            *reinterpret_cast<uint4*>(hi + o1) = h1;
            *reinterpret_cast<uint4*>(hi + kBuf + o0) = l0;
            *reinterpret_cast<uint4*>(hi + kBuf + o1) = l1;
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBKFull + s));
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
    }
  } else if (warp == 11) {
    // ---------------------------------------------------- queries and lse ----
    int gq = 0;
    uint32_t landed = 0;   // blocks that were cleared
    bool landing = false;  // the wait for one was given up
    bool ok = true;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      for (int b = 0; b < d.nb; ++b, ++gq) {
        const int s = gq % kQSlots;
        const int j = (d.b0 + b) * QT;  // first query of the block, from d.tok
        const int own = (d.nq - j) * G;  // rows of the row's queries
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 4 * lane + e, jj = j + c / G;
          v[e] = jj < d.nq ? __ldg(a.lse + static_cast<long long>(d.tok + jj) * a.n_q + d.h * G + c % G) : INFINITY;
        }
        if (gq >= kQSlots && !(ok = wait(kBQEmpty + s, gq / kQSlots - 1))) break;
        // A cap's arithmetic is chosen by the scores of a block, so the rows behind
        // (another row's queries, or tokens of no row) are cleared first.
        const bool clear = GEN == 1 && own < 128;
        if (lane == 0) {
          const uint32_t to = clear ? bar(kBQLand) : bar(kBQFull + s);
          mbar_arrive_expect_tx(to, kBuf);
          tc::load_rows(sbase + kQRing + s * kBuf, &qmap, d.h * G, d.tok + j, to);
        }
        if (clear) {
          __syncwarp();
          ok = wait(kBQLand, landed);
          landing = !ok;
          if (!ok) break;
          ++landed;
          uint8_t* rows = smem + kQRing + s * kBuf;  // 128 bytes of a row in either half
          for (int e = 8 * own + lane; e < 8 * 128; e += 32) {
            reinterpret_cast<uint4*>(rows)[e] = make_uint4(0u, 0u, 0u, 0u);
            reinterpret_cast<uint4*>(rows + kBuf / 2)[e] = make_uint4(0u, 0u, 0u, 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBQFull + s));
        }
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool fine = fabsf(v[e]) <= 3.0e38f;  // neither infinite nor NaN
          odd = odd || !fine;
          v[e] = fine ? -v[e] * kLog2e : -INFINITY;
        }
        const int ls = gq % kLseSlots;
        if (gq >= kLseSlots && !(ok = wait(kBLseEmpty + ls, gq / kLseSlots - 1))) {
          ++gq;  // its copy is in flight
          break;
        }
        *reinterpret_cast<float4*>(&tail.lse2[ls][4 * lane]) = make_float4(v[0], v[1], v[2], v[3]);
        const bool any = __any_sync(kFull, odd);
        if (lane == 0) tail.odd[ls] = any;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBLse + ls));
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
    }
    const int zero = 0;  // the last copies land before the CTA ends
    if (lane == 0 && landing) mbar_wait_bounded(bar(kBQLand), landed & 1u, &zero);
    if (lane == 0)
      for (int g = max(0, gq - kQSlots); g < gq; ++g)
        mbar_wait_bounded(bar(kBQFull + g % kQSlots), (g / kQSlots) & 1, &zero);
    __syncwarp();
  } else if (warp == 9) {
    // ----------------------------------------------------------- products ----
    // converged and uniform throughout: see tcgen05.cuh
    const uint32_t lead = tc::elect_one();
    const uint32_t tm = tc::uniform(tmem);
    constexpr uint32_t id = tc::idesc(128, 128, false, false, DT == PKV_KV_BF16 ? 1u : 0u);
    constexpr uint32_t kHiK = tc::desc_hi(2048), kHiQ = tc::desc_hi(1024);
    const uint32_t k_lo = tc::desc_lo(sbase, 16), q_lo = tc::desc_lo(sbase + kQRing, 16);
    int gq = 0, kp = 0;
    uint32_t used[2] = {0, 0};  // score buffers filled per half
    bool ok = true, any = false;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece& d = tail.piece[x];
      if (tc::uniform(d.last)) break;
      const bool two = tc::uniform(d.t0) + 128 < tc::uniform(d.L);
      const int nb = tc::uniform(d.nb);
      for (int b = 0; b < nb && ok; ++b, ++gq) {
        const int s = gq % kQSlots;
        any = true;
        if (!(ok = wait(kBQFull + s, gq / kQSlots))) break;
        const uint32_t qd = q_lo + s * (kBuf >> 4);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int ks = (kp + m) % kNB;
          if (b == 0 && !(ok = wait(kBKFull + ks, (kp + m) / kNB))) break;
          if (m == 0 || two) {
            const int buf = used[m] & 1;
            if (used[m] >= 2 && !(ok = wait(kBSFree + 2 * m + buf, used[m] / 2 - 1))) break;
            ++used[m];
            tc::fence_after();
            const uint32_t kd = k_lo + ks * (kKBytes >> 4);
#pragma unroll
            for (int part = 0; part < (kQ8 ? 2 : 1); ++part)
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc::mma_ss<kHiK, kHiQ>(tm + 256 * m + 128 * buf,
                                       kd + ((part * kBuf + (kk >> 2) * 1024 + (kk & 3) * 32) >> 4),
                                       qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4), id, part > 0 || kk > 0, lead);
            tc::commit(bar(kBS + 2 * m + buf), lead);
          }
          if (b + 1 == nb) tc::commit(bar(kBKEmpty + ks), lead);
        }
        if (!ok) break;
        tc::commit(bar(kBQEmpty + s), lead);
      }
      if (!ok) break;
      if (nb > 0) kp += 2;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
      __syncwarp();
    }
    if (any) {  // every product issued completes before the tensor memory is freed
      const int zero = 0;
      tc::commit(bar(kBDrain), lead);
      __syncwarp();
      if (lane == 0) mbar_wait_bounded(bar(kBDrain), 0, &zero);
      __syncwarp();
    }
  } else if (warp < 8) {
    // --------------------------------------------------------------- sums ----
    const int m = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const float c1 = a.sc.scale * kLog2e;
    const float cap_k = a.sc.softcap > 0.0f ? a.sc.scale / a.sc.softcap : 0.0f;
    const float cap2 = a.sc.softcap * kLog2e;
    const NearCap cap(cap_k, cap2);
    const int lg = G == 4 ? 2 : G == 2 ? 1 : 0;
    int gq = 0;
    uint32_t used = 0;
    bool ok = true;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      const bool mine = m == 0 || d.t0 + 128 < d.L;
      const int t = d.t0 + 128 * m + 32 * quarter + lane;
      // queries [jlo, jhi) from d.tok attend to t
      const int past = d.P0;
      const int jlo = t < d.F ? 0 : max(0, t - past);
      const long long jend = a.pool.window > 0 ? static_cast<long long>(t) + a.pool.window - past : d.nq;
      const int jhi = static_cast<int>(max(0ll, min(static_cast<long long>(d.nq), jend)));
      float slope2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (GEN == 2) {
#pragma unroll
          for (int e = 0; e < 4; ++e) slope2[e] = __ldg(a.sc.slopes + d.h * G + (e & (G - 1))) * kLog2e;
      }
      float sum = 0.0f, lost = 0.0f;  // the sum over blocks and its rounding error so far
      for (int b = 0; b < d.nb; ++b, ++gq) {
        const int s = gq % kLseSlots;
        // the block's lse staged (a half without tokens takes part in the
        // slots' hand-overs all the same)
        if (!(ok = wait(kBLse + s, gq / kLseSlots))) break;
        if (mine) {
          if (!(ok = wait(kBS + 2 * m + (used & 1), used >> 1))) break;
          tc::fence_after();
          const uint32_t tS = tmem + lanes + 256 * m + 128 * (used & 1);
          const int j = (d.b0 + b) * QT;
          const int from = min(128, max(0, (jlo - j) * G)), to = min(128, max(0, (jhi - j) * G));
          const bool fast = __all_sync(kFull, from == 0 && to == 128) && *(volatile int*)&tail.odd[s] == 0;
          float2 acc[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[e] = make_float2(0.0f, 0.0f);
          // the weights of columns 32 q ..: 2^(c1 s - lse2).  The masked form is
          // code of its own: a test per column would cut the arithmetic into
          // pieces too short to hide each other's latency (two chunks of 1800
          // tokens 223 us instead of 163).
          auto weigh = [&](float (&v)[32], int q) {
            float2 mul = make_float2(c1, c1);
            float cq[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // GEN 1: the factor is q(v^2)
            if constexpr (GEN == 1) {
              if (__builtin_expect(cap.beyond(v, cap.limit(t < d.L)), 0)) {
                cap32(v, tS + 32 * q, cap_k, cap2);
                cq[0] = 1.0f;
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) cq[e] = cap.q[e];
              }
            }
            if constexpr (GEN == 2) {
              if (a.sc.softcap > 0.0f) {
                cap32(v, tS + 32 * q, cap_k, cap2);
                mul = make_float2(1.0f, 1.0f);
              }
            }
            if constexpr (GEN == 2) {
              const float dist0 = static_cast<float>(past + j - t + ((32 * q) >> lg));  // P - t of the first column
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float step = lg == 2 ? static_cast<float>(e >> 2) : lg == 1 ? static_cast<float>(e >> 1) : static_cast<float>(e);
                v[e] = fmaf(-slope2[e & 3], fabsf(dist0 + step), v[e] * mul.x);
              }
              mul = make_float2(1.0f, 1.0f);
            }
            const float4* lse4 = reinterpret_cast<const float4*>(&tail.lse2[s][32 * q]);
            float2 y[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float4 l = lse4[e];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float2 x = make_float2(v[4 * e + 2 * h], v[4 * e + 2 * h + 1]);
                float2 f = mul;
                if constexpr (GEN == 1) {
                  const float2 xx = tc::fma2(x, x, make_float2(0.0f, 0.0f));
                  f = tc::fma2(xx, make_float2(cq[3], cq[3]), make_float2(cq[2], cq[2]));
                  f = tc::fma2(xx, f, make_float2(cq[1], cq[1]));
                  f = tc::fma2(xx, f, make_float2(cq[0], cq[0]));
                }
                y[2 * e + h] = tc::fma2(x, f, h ? make_float2(l.z, l.w) : make_float2(l.x, l.y));
              }
            }
            if (!fast) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int c = 32 * q + 2 * e;
                const float2 l = *reinterpret_cast<const float2*>(&tail.lse2[s][c]);
                y[e].x = c >= from && c < to && l.x > -INFINITY ? y[e].x : -INFINITY;
                y[e].y = c + 1 >= from && c + 1 < to && l.y > -INFINITY ? y[e].y : -INFINITY;
              }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e & 3] = tc::add2(acc[e & 3], make_float2(tc::ex2(y[e].x), tc::ex2(y[e].y)));
          };
          auto release = [&] {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kBSFree + 2 * m + (used & 1)));
          };
          if constexpr (GEN != 0) {  // one copy of the longer code
            float v[32];
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              tc::ld32(tS + 32 * q, v);
              tc::wait_ld();
              weigh(v, q);
            }
            release();
          } else {  // one load from tensor memory ahead of the arithmetic
            float v0[32], v1[32];
            tc::ld32(tS, v0);
            tc::wait_ld();
            tc::ld32(tS + 32, v1);
            weigh(v0, 0);
            tc::wait_ld();
            tc::ld32(tS + 64, v0);
            weigh(v1, 1);
            tc::wait_ld();
            tc::ld32(tS + 96, v1);
            weigh(v0, 2);
            tc::wait_ld();
            release();
            weigh(v1, 3);
          }
          ++used;
          const float2 a2 = tc::add2(tc::add2(acc[0], acc[1]), tc::add2(acc[2], acc[3]));
          // compensated: a tile may see hundreds of blocks
          const float y = (a2.x + a2.y) - lost, z = sum + y;
          lost = (z - sum) - y;
          sum = z;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBLseEmpty + s));
      }
      if (!ok) break;
      if (mine && t < d.L) {
        if (kQ8 && __builtin_expect(!(fabsf(sum) <= 3.0e38f), 0) && token_beyond(a, d.i, d.h, t))
          ctl[1] = 1;
        else
          store_sum(a, d.slot, d.i, d.h, t, d.L, d.n, sum);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
    }
  }

  tc::fence_before();
  __syncthreads();
  if (warp == 9) {
    tc::fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if constexpr (kQ8) {
    if (ctl[1] && !ctl[0]) mend_tokens(a, geo, tail.bounds[0], tail.bounds[1], tail.tiles);
  }
}

// CTA k: if boundary k + 1 is the first to cut its tile, the tile's sums from
// its pieces, in order: the end of range k and the starts of the ranges whose
// boundaries cut it.
__global__ void __launch_bounds__(kMassTok) mass_merge_kernel(const __grid_constant__ MassArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  const Rec* rec = reinterpret_cast<const Rec*>(a.workspace);
  const int k0 = blockIdx.x + 1;
  const Rec me = rec[k0], prev = rec[k0 - 1];
  if (!me.inside || (prev.inside && prev.h == me.h && prev.tile == me.tile)) return;
  const int t = me.t0 + threadIdx.x;
  if (t >= me.L) return;
  float sum = slot_sums(a, 2 * (k0 - 1) + 1)[threadIdx.x];
  for (int k = k0; k < a.chunks; ++k) {
    const Rec n = rec[k];
    if (!n.inside || n.h != me.h || n.tile != me.tile) break;
    sum += slot_sums(a, 2 * k)[threadIdx.x];
  }
  const long long at = (static_cast<long long>(me.i) * a.pool.n_kv + me.h) * a.mass_stride + t;
  a.mass_out[at] = (a.mass_in && t < me.L - me.n ? a.mass_in[at] : 0.0f) + sum;
}

template <int DT, int GEN>
cudaError_t launch_mass_t(const MassArgs& a, const TileMaps& maps, const CUtensorMap& qmap, cudaStream_t st) {
  static std::atomic<int> granted[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !granted[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(attention_mass_kernel<DT, GEN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) granted[dev].store(1, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.chunks);
  cfg.blockDim = dim3(kMassThreads<DT>);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, attention_mass_kernel<DT, GEN>, a, maps, qmap);
  if (e != cudaSuccess) return e;
  if (a.chunks > 1) {
    cfg.gridDim = dim3(a.chunks - 1);
    cfg.blockDim = dim3(kMassTok);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, mass_merge_kernel, a);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_mass_g(const MassArgs& a, const TileMaps& maps, const CUtensorMap& qmap, cudaStream_t st) {
  if (a.sc.slopes) return launch_mass_t<DT, 2>(a, maps, qmap, st);
  if (a.sc.softcap > 0.0f) return launch_mass_t<DT, 1>(a, maps, qmap, st);
  return launch_mass_t<DT, 0>(a, maps, qmap, st);
}

}  // namespace

size_t attention_mass_workspace(int chunks) {
  return rec_bytes(chunks) + 2 * static_cast<size_t>(chunks) * kMassTok * sizeof(float);
}

cudaError_t launch_attention_mass(const MassArgs& a, const TileMaps& maps, cudaStream_t st) {
  const int G = a.n_q / a.pool.n_kv;
  CUtensorMap qmap;
  cudaError_t e = encode_query_map(&qmap, a.pool.dtype == PKV_KV_BF16, a.q, a.q_stride, a.n_q, G,
                                   a.rows.total_tokens, 128 / G);
  if (e != cudaSuccess) return e;
  if (a.pool.dtype == PKV_KV_F16) return launch_mass_g<PKV_KV_F16>(a, maps, qmap, st);
  if (a.pool.dtype == PKV_KV_BF16) return launch_mass_g<PKV_KV_BF16>(a, maps, qmap, st);
  return launch_mass_g<PKV_KV_Q8_0>(a, maps, qmap, st);
}

}  // namespace pkv
