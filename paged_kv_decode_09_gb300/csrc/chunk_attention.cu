// chunk_attention.cu — paged_chunk_attention on the fifth-generation tensor
// cores (tcgen05, accumulators in tensor memory).
//
// For one (row, KV head), the (query, query head) pairs are rows of a matrix
// product: a tile is 256 of them, 256 / G queries, as two halves m of 128.
// Over the tile's blocks of N cached tokens (128; q8_0: 64),
//     S_m = Q_m K^T             128 x N, both from shared memory
//     P_m = 2^(y - max)         y the base-2 score, one thread per row
//     O_m += P_m V              128 x 128, P_m from tensor memory
// with one pass over K and V and the running maximum and sum of the softmax
// in the row's thread.  The maximum is raised, and O rescaled, only when a
// block exceeds it by more than 8 (a factor of 256, which f16 and bf16 hold).
// P_m overwrites S_m in tensor memory as 16-bit pairs: S_0, S_1, O_0 and O_1
// take all 512 columns.  The halves alternate on the tensor cores: while one
// is in its softmax, the other's products run.  A tile of up to 128 rows (a
// token of a row, the end of a chunk) would leave half 1 idle and each block
// waiting for the one before: there the halves hold the same rows and take the
// blocks in turn, and half 0 joins the two states at the end (8 rows of one
// token 28.5 -> 23.3 us).
// q8_0 keys and values enter as two f16 parts, hi and lo (q8_tiles.cuh), two
// products each.
//
// Warps: 0-3 and 4-7 the softmax of half 0 and 1, 8 walks the work and copies
// Q, 9 issues the products, 10 copies K and V pages (one tensor copy each)
// into a ring of five 32 KiB slots, 11 mends V blocks that hold tokens no
// query of the tile attends to; with q8_0, 10 copies codes and scales into a
// ring of their own, and 12-15 split them into the ring of slots.  Hand-overs
// by shared-memory barriers:
//   dfull, dempty[x]  descriptor x of a piece (a tile's blocks in this range)
//   qfull[m], qempty  Q_m landed; the piece's last scores are computed
//   full, empty[s]    K or V block in ring slot s
//   raw, rawempty[s]  codes and scales of a K or V block (q8_0)
//   land[s]           a V block that warp 11 passes on to full[s]
//   sfull[m]          S_m computed (and every product issued before it)
//   pready[m]         P_m written, S_m read
//   ofull[m]          O_m of the piece complete
//   half, joined      half 1's maximum and sum are in shared memory; half 0 has
//                     read them and O_1
// Every wait is bounded; a warp that gives up sets the abort flag, which ends
// the other waits, and its copies and products are awaited before the CTA ends.
//
// What bounds it: the products of a block of 256 x 128 take 2048 cycles, a block
// some 3200.  A half's softmax (four groups of 32 columns, 400 to 500 cycles
// each while the other half's warps compete for the schedulers) and its own two
// products follow one another, and there is no tensor memory left for a second
// S_m.  Scores in steps of 64 tokens, each computed while the step before is in
// its softmax, take that chain apart, but the scores' products then cost half
// as much again and the steps their own hand-overs: 381 us instead of 376.
// 8191 tokens of 32 heads in bf16 373 us, 1475 TFLOP/s; with a window of 4096
// over rows of 14K to 16K 194 us, 1240 TFLOP/s; 2048 tokens over 32049 in q8_0
// 1.37 ms (twice the products; 761 TFLOP/s of useful work).  Single tokens of 8
// rows of 1K to 6K in f16 are bound by K and V's bytes: 22.1 us, 4.2 TB/s, of
// which some 10 are the launches, the plan, the last blocks and the merge.  In
// q8_0 they take 45.8 us for half the bytes: no turns, blocks of 64 tokens, and
// the splitting of each block stands in its chain.  The CTAs of the prompt are
// busy for 351 to 364 us, 356 in the mean.
//
// The work of the batch is a line of (KV head, tile, block) units, cut into
// equal ranges, one per CTA (chunk_plan.cuh).  A tile that crosses a boundary
// leaves partial states (m, l, O) in the workspace, which the second kernel
// merges.
//
// A token that some rows of a tile attend to and others do not gets weight 0
// in the latter, but 0 times a value that is not finite is not 0.  Warp 11
// looks for such values in the blocks that are masked for part of the tile.
// With q8_0, a block's scale of 512 or more may take a value out of f16's range
// (q8_tiles.cuh): scores or outputs of the rows that meet it are not finite.
// Where there is either, the rows of the piece that ended up not finite are
// computed again from the tokens they attend to alone (mend_rows), after the
// pipeline has drained: a query takes a warp microseconds per 32 tokens, so that
// inside the pipeline a tile of a long row would run the other warps' waits out
// of their limit.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cudaTypedefs.h>

#include "attend_row.cuh"
#include "chunk_device.cuh"
#include "chunk_plan.cuh"
#include "q8_tiles.cuh"
#include "score32.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kTileRows = 256;   // (query, query head) rows of a tile: 256 / G queries
template <int DT>
constexpr int kBlockTok = DT == PKV_KV_Q8_0 ? 64 : 128;  // cached tokens of a block
template <int DT>
constexpr int kAttnThreads = DT == PKV_KV_Q8_0 ? 512 : kPlanThreads;
// How far from a tile's end a boundary moves there, in blocks (chunk_plan): with
// q8_0's blocks of 64 tokens, from one block away; with blocks of 128, never.
template <int DT>
constexpr int kSplitSnap = 128 / kBlockTok<DT>;
template <int DT>
constexpr int kSlots = DT == PKV_KV_Q8_0 ? 4 : 5;    // ring slots
constexpr int kMaxSlots = 5;
constexpr uint32_t kHalf = 32768;                    // bytes of Q_m, and of a ring slot
constexpr uint32_t kRing = 2 * kHalf;                // the ring, behind Q
// q8_0: a ring of K or V codes of a block as they are stored, and their scales
constexpr int kRaws = 3;
constexpr uint32_t kRawBytes = 64 * kD;
constexpr uint32_t kRaw = kRing + kSlots<PKV_KV_Q8_0> * kHalf;
constexpr uint32_t kRawScales = kRaw + kRaws * kRawBytes;
constexpr uint32_t kRawScaleBytes = 64 * (kD / kQBlock) * 2;
constexpr uint32_t kTail = kRing + kMaxSlots * kHalf;   // barriers and descriptors
static_assert(kRawScales + kRaws * kRawScaleBytes <= kTail, "");
constexpr int kDescs = 4;
constexpr int kMendBits = 1024;                      // pieces of a range told apart by mend_rows
constexpr uint32_t kTmemS = 0, kTmemO = 256;         // S_m at 128 m, O_m at 256 + 128 m

// barriers
enum : int {
  kBFull = 0,
  kBEmpty = kBFull + kMaxSlots,
  kBLand = kBEmpty + kMaxSlots,
  kBRaw = kBLand + kMaxSlots,
  kBRawEmpty = kBRaw + kRaws,
  kBS = kBRawEmpty + kRaws,
  kBP = kBS + 2,
  kBO = kBP + 2,
  kBQ = kBO + 2,
  kBQEmpty = kBQ + 2,
  kBDesc = kBQEmpty + 1,
  kBDescEmpty = kBDesc + kDescs,
  kBHalf = kBDescEmpty + kDescs,  // alternating halves: half 1's state handed over, half 0's epilogue over
  kBJoined,
  kBDrain,
  kBStall,
  kNumBars,
};
template <int DT>
constexpr int kDescReaders = DT == PKV_KV_Q8_0 ? 14 : 11;  // softmax, products, copies, and mending or splitting

// A piece: blocks kb .. kb + nb - 1 of one tile for KV head h.
struct Piece {
  int i, h, tok, nq, P0, L, F, kb, nb, t_lo, t_hi;
  int full_lo, full_hi;  // [full_lo, full_hi): tokens every query of the tile attends to
  int slot;              // partial slot, -1: the whole tile
  int last;              // no piece: the end
  int pad;
};
static_assert(sizeof(Piece) == 64, "");

struct Tail {
  uint64_t bars[kNumBars];
  Piece piece[kDescs];
  volatile int ctl[2];  // abort; there may be rows to compute again
  uint32_t tmem;
  int tiles;           // of the batch
  uint32_t notes[kMendBits / 32];  // the pieces with such rows (note_piece)
  float2 half[kTileRows / 2];  // half 1's maximum and sum of each row
  Place bounds[2];     // the CTA's range
  PlanScratch scratch;
};
constexpr size_t kSmemBytes = 1024 + kTail + sizeof(Tail);
static_assert(kSmemBytes <= 232448, "");

// A tile: queries t * QT .. of a row, and the blocks they attend to.
struct TileGeom {
  int nq;    // queries
  int P0;    // position of the first
  int t_lo;  // tokens [t_lo, t_hi) that some query of the tile attends to
  int t_hi;
  int kb;    // first block
  int nb;    // blocks
};
template <int DT>
struct QueryTiles {
  int QT, W;
  __device__ __forceinline__ int tiles(const RowInfo& r) const { return r.L >= 0 ? (r.n + QT - 1) / QT : 0; }
  __device__ __forceinline__ TileGeom tile(const RowInfo& r, int F, int t) const {
    TileGeom g;
    const int j0 = t * QT;
    g.nq = min(QT, r.n - j0);
    g.P0 = r.L - r.n + j0;
    g.t_lo = seen_from(g.P0, W);
    g.t_hi = seen_to(g.P0 + g.nq - 1, r.L, F);
    g.kb = g.t_lo / kBlockTok<DT>;
    g.nb = (g.t_hi + kBlockTok<DT> - 1) / kBlockTok<DT> - g.kb;
    return g;
  }
  __device__ __forceinline__ int blocks(const RowInfo& r, int F, int t) const { return tile(r, F, t).nb; }
  // Units: 4 a block, 2 in a tile of up to 128 rows (half the arithmetic); 12
  // and 10 a tile.  A batch of two chunks and 30 single tokens takes 122 us, 142
  // at 3 units for the smaller blocks, 156 at 4.  q8_0 has no turns to gain by.
  // (Measured on plain scores; with a cap or a bias a block costs up to half as
  // much again.)
  static constexpr int kMostWeight = 4;
  __device__ __forceinline__ int weight(const RowInfo& r, int t) const {
    return DT == PKV_KV_Q8_0 || 2 * (r.n - t * QT) > QT ? 4 : 2;
  }
  __device__ __forceinline__ int lead(int weight) const {
    return (weight == 4 ? 12 : 10) * (128 / kBlockTok<DT>);
  }
};

// ------------------------------------------------------------ workspace ----
// Records of the boundaries (Rec), then two partial slots per chunk: slot 2k
// for the piece at the start of range k, 2k + 1 for the one at its end.  A
// slot: (m, l) of its 256 rows, then O as [32 groups of 4 dims][256 rows].
struct __align__(16) Rec {
  int inside;  // the boundary cuts a tile
  int h, tile, tok, nq, pad[3];
};
constexpr size_t kSlotMl = kTileRows * 8;
constexpr size_t kSlotFull = kSlotMl + static_cast<size_t>(kTileRows) * kD * 4;
__host__ __device__ inline size_t rec_bytes(int chunks) {
  return (static_cast<size_t>(chunks + 1) * sizeof(Rec) + 255) & ~size_t(255);
}
__device__ __forceinline__ float2* slot_ml(const ChunkAttnArgs& a, int slot) {
  return reinterpret_cast<float2*>(a.workspace + rec_bytes(a.chunks) + slot * kSlotFull);
}
__device__ __forceinline__ float4* slot_acc(const ChunkAttnArgs& a, int slot) {
  return reinterpret_cast<float4*>(a.workspace + rec_bytes(a.chunks) + slot * kSlotFull + kSlotMl);
}

template <int DT>
struct Io {
  static constexpr int kType = DT == PKV_KV_BF16 ? PKV_KV_BF16 : PKV_KV_F16;
  [[maybe_unused]] static constexpr uint32_t kFormat = DT == PKV_KV_BF16 ? 1u : 0u;
  // P is scaled by 2^kShift: f16 weights far below the maximum stay normal
  // (the largest, 2^(8 + 7), is still below f16's 65504); bf16 has the range.
  [[maybe_unused]] static constexpr float kShift = DT == PKV_KV_BF16 ? 0.0f : 7.0f;
  [[maybe_unused]] static constexpr float kScale = DT == PKV_KV_BF16 ? 1.0f : 128.0f;
  // two packed values times f
  static __device__ __forceinline__ uint32_t scale(uint32_t w, float f) {
    if constexpr (kType == PKV_KV_BF16) {
      const __nv_bfloat162 h = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w), __float2bfloat162_rn(f));
      return *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __hmul2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(f));
      return *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  static __device__ __forceinline__ float2 values(uint32_t w) {
    if constexpr (kType == PKV_KV_BF16)
      return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else
      return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    if constexpr (kType == PKV_KV_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
      return *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x, y);
      return *reinterpret_cast<const uint32_t*>(&h);
    }
  }
};

// Blocks [b0, b1) of tile g, where the walk of this CTA's range stands.
template <int DT>
__device__ __forceinline__ Piece piece_of(const Walk<QueryTiles<DT>>& w, const TileGeom& g, int b0, int b1) {
  Piece d;
  d.i = w.at.i;
  d.h = w.at.h;
  d.tok = w.r.start + w.at.t * w.geo.QT;
  d.nq = g.nq;
  d.P0 = g.P0;
  d.L = w.r.L;
  d.F = w.F;
  d.kb = g.kb + b0;
  d.nb = b1 - b0;
  d.t_lo = g.t_lo;
  d.t_hi = g.t_hi;
  d.full_lo = seen_from(g.P0 + g.nq - 1, w.geo.W);
  d.full_hi = seen_to(g.P0, w.r.L, w.F);
  d.slot = b0 > 0 ? 2 * static_cast<int>(blockIdx.x) : b1 < g.nb ? 2 * static_cast<int>(blockIdx.x) + 1 : -1;
  d.last = 0;
  d.pad = 0;
  return d;
}

// ------------------------------------------------- queries, once more ----
// The pieces of the range with something to mend: a bit each, those from the last
// bit on together.
__device__ __forceinline__ void note_piece(uint32_t* notes, int p) {
  const int b = min(p, kMendBits - 1);
  atomicOr(notes + b / 32, 1u << (b % 32));
}

// The rows of the noted pieces of the range [begin, end) that were stored as not
// finite, computed again in fp32 from the tokens they attend to: a query by each
// of the first kMendWarps warps (all of them call it, behind a barrier after the
// range's last store).
constexpr int kMendWarps = 8;
template <int DT>
__device__ __noinline__ void mend_rows(const ChunkAttnArgs& a, const uint32_t* notes, const Place& begin,
                                       const Place& end, int T) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_q / a.pool.n_kv;
  const QueryTiles<DT> geo{kTileRows / G, a.pool.window};
  Walk<QueryTiles<DT>> w(a.rows, geo, a.sc.prefix_lens, T, begin, end);
  for (int p = 0; w.more(); ++p) {
    const TileGeom g = geo.tile(w.r, w.F, w.at.t);
    const Piece d = piece_of<DT>(w, g, w.from(), w.to(g.nb));
    const int bit = min(p, kMendBits - 1);
    const int queries = notes[bit / 32] >> (bit % 32) & 1u ? d.nq : 0;
#pragma unroll 1
    for (int j = warp; j < queries; j += kMendWarps) {
      const long long row = static_cast<long long>(d.tok + j) * a.n_q + d.h * G;  // of its first head
      unsigned bad = 0;  // heads
#pragma unroll 1
      for (int u = 0; u < G; ++u) {
        float x[4];  // four dims of the row
        if (d.slot >= 0) {
          const float4 v = slot_acc(a, d.slot)[lane * kTileRows + j * G + u];
          x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(a.out + ((row + u) * kD + 4 * lane) * 2);
          const float2 lo = Io<DT>::values(v.x), hi = Io<DT>::values(v.y);
          x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
        }
        float watch = 0.0f;  // NaN once a value is not finite
#pragma unroll
        for (int e = 0; e < 4; ++e) watch = fmaf(x[e], 0.0f, watch);
        bad |= __any_sync(kFull, watch != 0.0f) ? 1u << u : 0u;
      }
      if (!bad) continue;
      const int P = d.P0 + j;
      const int t0 = max(seen_from(P, a.pool.window), d.kb * kBlockTok<DT>);
      const int t1 = min(seen_to(P, d.L, d.F), (d.kb + d.nb) * kBlockTok<DT>);
      float m[4], l[4], acc[4][4];
      attend_query<DT>(a.pool, a.rows, a.sc, d.i, d.h, G, P,
                       a.q + ((d.tok + j) * a.q_stride + static_cast<long long>(d.h) * G * kD) * 2, t0, t1, m, l, acc);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!(bad >> u & 1u)) continue;
        if (d.slot >= 0) {
          const int r = j * G + u;
          slot_acc(a, d.slot)[lane * kTileRows + r] = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
          if (lane == 0) slot_ml(a, d.slot)[r] = make_float2(m[u], l[u]);
        } else {
          const float inv = 1.0f / l[u];
          *reinterpret_cast<uint2*>(a.out + ((row + u) * kD + 4 * lane) * 2) = make_uint2(
              Io<DT>::pack(acc[u][0] * inv, acc[u][1] * inv), Io<DT>::pack(acc[u][2] * inv, acc[u][3] * inv));
          if (a.lse && lane == 0) a.lse[row + u] = (m[u] + log2f(l[u])) * kLn2;
        }
      }
    }
    if (w.ends_here()) break;
    w.next();
  }
}

// The rare end of a raised maximum, kept out of the softmax's loop: the rows'
// weights of the block so far (`groups` of 32 columns in P) and, with `o`, their
// O, times al.
template <int DT>
__device__ __forceinline__ void rescale_here(uint32_t tP, uint32_t tO, int groups, bool o, float al) {
#pragma unroll 1
  for (int e = 0; e < groups; ++e) {
    uint32_t w[16];
    tc::ld16w(tP + 16 * e, w);
    tc::wait_ld();
#pragma unroll
    for (int u = 0; u < 16; ++u) w[u] = Io<DT>::scale(w[u], al);
    tc::st16(tP + 16 * e, w);
  }
#pragma unroll 1
  for (int e = 0; o && e < 8; ++e) {
    uint32_t w[16];
    tc::ld16w(tO + 16 * e, w);
    tc::wait_ld();
#pragma unroll
    for (int u = 0; u < 16; ++u) w[u] = __float_as_uint(__uint_as_float(w[u]) * al);
    tc::st16(tO + 16 * e, w);
  }
  tc::wait_st();
}
template <int DT>
__device__ __noinline__ void rescale(uint32_t tP, uint32_t tO, int groups, bool o, float al) {
  rescale_here<DT>(tP, tO, groups, o, al);
}

// Zeros and an lse of -inf for the queries of rows that are skipped (one warp).
__device__ __forceinline__ void fill_skipped(const ChunkAttnArgs& a) {
  const int lane = threadIdx.x & 31;
  for (int i = blockIdx.x; i < a.rows.num_rows; i += gridDim.x) {
    const RowInfo r = row_info(a.rows, i, lane == 0 ? a.pool.status : nullptr);
    if (r.L >= 0 || r.n == 0) continue;
    uint4* out = reinterpret_cast<uint4*>(a.out + static_cast<long long>(r.start) * a.n_q * kD * 2);
    const long long rows = static_cast<long long>(r.n) * a.n_q;
    for (long long e = lane; e < rows * (kD / 8); e += 32) out[e] = make_uint4(0u, 0u, 0u, 0u);
    if (a.lse)
      for (long long e = lane; e < rows; e += 32) a.lse[static_cast<long long>(r.start) * a.n_q + e] = -INFINITY;
  }
}

// GEN: 0 plain scores; 1 capped (at most 1e9); 2 with a distance bias, capped
// or not, with a scale that is not positive, or a higher cap.
template <int DT, int GEN>
__global__ void __launch_bounds__(kAttnThreads<DT>, 1)
    chunk_attention_kernel(const __grid_constant__ ChunkAttnArgs a, const __grid_constant__ TileMaps maps,
                           const __grid_constant__ CUtensorMap qmap) {
  using F = Io<DT>;
  constexpr bool kQ8 = DT == PKV_KV_Q8_0;
  constexpr int kS = kSlots<DT>;
  constexpr int N = kBlockTok<DT>;                   // tokens of a block
  constexpr int kPages = N / kPage;                  // its pages
  constexpr uint32_t kPart = N * kD * 2;             // bytes of one part of it
  // The halves take a smaller tile's blocks in turn (q8_0: no registers left)
  constexpr bool kTurns = !kQ8;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Tail& tail = *reinterpret_cast<Tail*>(smem + kTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_addr(smem);
  const uint32_t bars = smem_addr(tail.bars);
  auto bar = [&](int b) { return bars + 8u * static_cast<uint32_t>(b); };
  volatile int* ctl = tail.ctl;
  const int G = a.n_q / a.pool.n_kv, QT = kTileRows / G;

  if (tid == 0) {
    prefetch_tensormap(&maps.kp);
    prefetch_tensormap(&maps.vp);
    prefetch_tensormap(&qmap);
    tail.ctl[0] = 0;
    tail.ctl[1] = 0;
  }
  if (tid < kMendBits / 32) tail.notes[tid] = 0;
  if (tid < kNumBars) {
    const int b = tid;
    int count = 1;
    if ((b < kBEmpty && kQ8) || (b >= kBRawEmpty && b < kBS)) count = 4;
    if ((b >= kBP && b < kBO) || b == kBHalf || b == kBJoined) count = 4;
    if (b >= kBDescEmpty && b < kBDescEmpty + kDescs) count = kDescReaders<DT>;
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
  const QueryTiles<DT> geo{QT, a.pool.window};
  // a small call's plan is made by the one warp that walks the work
  const bool small = a.rows.num_rows <= 32 && a.rows.total_tokens <= 32 * QT;
  int T = 0;
  if (small)
    __syncthreads();
  else
    T = chunk_plan(a.rows, a.pool.n_kv, geo, a.sc.prefix_lens, a.chunks, kSplitSnap<DT>,
                           reinterpret_cast<int*>(smem + kRing), &tail.scratch, tail.bounds);
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tail.tmem);
  Place begin, end;
  if (!small) {
    begin = tail.bounds[0];
    end = tail.bounds[1];
    // the ring is written next by the async proxy, after the plan's plain accesses
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  if (warp == 8) {  // before the test hook: the merge reads every range's record
    if (small)
      T = chunk_plan_warp(a.rows, a.pool.n_kv, geo, a.sc.prefix_lens, a.chunks, kSplitSnap<DT>, begin, end);
    if (lane == 0) {  // the range, for mend_rows, and the boundary at its start, for the merge
      tail.tiles = T;
      tail.bounds[0] = begin;
      tail.bounds[1] = end;
      Rec x{};
      x.inside = begin.h < a.pool.n_kv && begin.off > 0;
      if (x.inside) {
        const RowInfo r = row_info(a.rows, begin.i, nullptr);
        const TileGeom g = geo.tile(r, 0, begin.t);
        x.h = begin.h;
        x.tile = begin.tile;
        x.tok = r.start + begin.t * QT;
        x.nq = g.nq;
      }
      reinterpret_cast<Rec*>(a.workspace)[blockIdx.x] = x;
    }
    __syncwarp();
  }
  // test hook: every warp gives up here, before any copy
  const bool stalled = test_stall(bar(kBStall), a.pool.test_stall_ns, ctl, a.pool.status);

  auto wait = [&](int b, uint32_t parity) { return tc::warp_wait<!kQ8>(bar(b), parity & 1u, ctl, a.pool.status); };
  // block b of a piece: with a bias from the last one back, where the scores
  // are highest (a steep bias would raise the maximum with every group of 32
  // columns otherwise: 1100 us instead of 474 for a prompt of 8191 tokens)
  auto block = [](int kb, int nb, int b) { return GEN == 2 ? kb + nb - 1 - b : kb + b; };
  auto pages_of = [&](const Piece& p, int b, int& lo, int& hi) {  // pages of a block that are read
    const int first = block(p.kb, p.nb, b) * kPages;
    lo = max(first, p.t_lo / kPage);
    hi = min(first + kPages, (p.t_hi + kPage - 1) / kPage);
  };
  // V blocks that warp 11 sees: with tokens outside [t_lo, t_hi) in their
  // pages (zeroed), or masked for part of the tile (searched)
  auto mended = [&](const Piece& p, int b) {
    const int t0 = block(p.kb, p.nb, b) * N;
    return t0 < p.full_lo || t0 + N > p.full_hi;
  };

  if (kQ8 && warp >= 12) {
    // 3 x 144 + 80 = 4 x 128 registers a thread, what the launch has
    if constexpr (kQ8) tc::more_registers<144>();
    // ------------------------------ q8_0 keys and values as two f16 parts ----
    const int row = (tid - 384) >> 3, col = (tid - 384) & 7;  // 8 threads a token, 16 codes each
    int gs = 0;
    bool ok = !stalled;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      for (int b = 0; b < d.nb && ok; ++b) {
        const bool mend = mended(d, b);
        const int t0 = block(d.kb, d.nb, b) * N;
#pragma unroll
        for (int v = 0; v < 2; ++v, ++gs) {
          const int rs = gs % kRaws, s = gs % kS;
          if (!(ok = wait(kBRaw + rs, gs / kRaws))) break;
          const uint8_t* raw = smem + kRaw + rs * kRawBytes + row * kD + ((col ^ (row & 7)) << 4);
          const __half* rsc = reinterpret_cast<const __half*>(smem + kRawScales + rs * kRawScaleBytes) +
                              row * (kD / kQBlock) + (col >> 1);
          uint4 code[kPages];
          __half2 sc[kPages];
          bool odd = false, large = false;
#pragma unroll
          for (int e = 0; e < kPages; ++e) {  // token `row` of page e; 0 where no query of the tile attends
            const int t = t0 + e * kPage + row;
            const bool in = t >= d.t_lo && t < d.t_hi;
            code[e] = *reinterpret_cast<const uint4*>(raw + e * (kPage * kD));
            const __half f = in ? rsc[e * kPage * (kD / kQBlock)] : __float2half_rn(0.0f);
            const unsigned bits = __half_as_ushort(f) & 0x7FFFu;
            odd = odd || bits >= kNotFinite;
            large = large || (bits >= kLargeScale && bits < kNotFinite);
            sc[e] = __half2half2(f);
          }
          if (gs >= kS && !(ok = wait(kBEmpty + s, gs / kS - 1))) break;
          uint8_t* hi = smem + kRing + s * kHalf;
#pragma unroll
          for (int e = 0; e < kPages; ++e) {
            uint4 h0, l0, h1, l1;
            q8_split8(make_uint2(code[e].x, code[e].y), sc[e], h0, l0);
            q8_split8(make_uint2(code[e].z, code[e].w), sc[e], h1, l1);
            const uint32_t o0 = tile_vec(kPage * e + row, 2 * col), o1 = tile_vec(kPage * e + row, 2 * col + 1);
            *reinterpret_cast<uint4*>(hi + o0) = h0;
            *reinterpret_cast<uint4*>(hi + o1) = h1;
            *reinterpret_cast<uint4*>(hi + kPart + o0) = l0;
            *reinterpret_cast<uint4*>(hi + kPart + o1) = l1;
          }
          if (large || (v == 1 && mend && odd)) {
            ctl[1] = 1;
            note_piece(tail.notes, p);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(kBFull + s));
            mbar_arrive(bar(kBRawEmpty + rs));
          }
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
    }
    if (warp == 12) fill_skipped(a);
  } else if (warp >= 8) {
  if constexpr (kQ8) tc::fewer_registers<80>();
  if (stalled) {
    // test hook: every warp gave up
  } else if (warp == 8) {
    // ------------------------------------------------- pieces and queries ----
    Walk<QueryTiles<DT>> w(a.rows, geo, a.sc.prefix_lens, T, begin, end);
    int p = 0;
    bool ok = true;
    uint32_t q1 = 0;  // pieces with both halves so far
    while (w.more()) {
      const Place& c = w.at;
      const RowInfo& r = w.r;
      const TileGeom g = geo.tile(r, w.F, c.t);
      const int b0 = w.from(), b1 = w.to(g.nb);
      const int x = p % kDescs;
      const int tok = r.start + c.t * QT;
      if (p >= kDescs && !(ok = wait(kBDescEmpty + x, p / kDescs - 1))) break;
      if (lane == 0) {
        tail.piece[x] = piece_of<DT>(w, g, b0, b1);
        mbar_arrive(bar(kBDesc + x));
      }
      __syncwarp();
      const bool two = g.nq * G > kTileRows / 2;
      if (p > 0 && !(ok = wait(kBQEmpty, p - 1))) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(kBQ), kHalf);
        tc::load_rows(sbase, &qmap, c.h * G, tok, bar(kBQ));
        if (two) {
          mbar_arrive_expect_tx(bar(kBQ + 1), kHalf);
          tc::load_rows(sbase + kHalf, &qmap, c.h * G, tok + QT / 2, bar(kBQ + 1));
        }
      }
      __syncwarp();
      q1 += two ? 1 : 0;
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
    // the last copies land before the CTA ends
    const int zero = 0;
    if (lane == 0 && p > 0) {
      mbar_wait_bounded(bar(kBQ), (p - 1) & 1, &zero);
      if (q1 > 0) mbar_wait_bounded(bar(kBQ + 1), (q1 - 1) & 1, &zero);
    }
    __syncwarp();
  } else if (!kQ8 && warp == 10) {
    // ------------------------------------------------------ K and V pages ----
    int gs = 0;              // slots filled
    uint32_t landed = 0;     // parity of each slot's land barrier
    uint32_t my_bar = 0, my_par = 0;  // lane s: the last copy's barrier of slot s
    bool ok = true;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      const int32_t* bt = a.rows.block_table + static_cast<long long>(d.i) * a.rows.bt_stride;
      int lo, hi;
      pages_of(d, 0, lo, hi);
      auto entry = [&](int b) {
        int l0, h0;
        pages_of(d, b, l0, h0);
        return lane < h0 - l0 ? __ldg(bt + l0 + lane) : 0;
      };
      int next = entry(0);
      for (int b = 0; b < d.nb; ++b) {
        int pg = next;
        pages_of(d, b, lo, hi);
        if (b + 1 < d.nb) next = entry(b + 1);
        const int n = hi - lo;
        if (lane < n && (pg < 0 || pg >= a.pool.num_pages)) {
          record_status(a.pool.status, PKV_DEV_BAD_PAGE);
          pg = 0;
        }
        const uint32_t in_slot = (lo & (kPages - 1)) * 4096u + lane * 4096u;
        const bool mend = mended(d, b);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int s = (gs + v) % kS;
          if (gs + v >= kS && !wait(kBEmpty + s, (gs + v) / kS - 1)) {
            ok = false;
            break;
          }
          const int to = v == 1 && mend ? kBLand + s : kBFull + s;
          const uint32_t par = v == 1 && mend ? (landed >> s) & 1u : static_cast<uint32_t>((gs + v) / kS) & 1u;
          if (v == 1 && mend) landed ^= 1u << s;
          if (lane == s) {
            my_bar = bar(to);
            my_par = par;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(to), static_cast<uint32_t>(n) * 4096u);
          __syncwarp();
          if (lane < n)
            tc::load_tile(sbase + kRing + s * kHalf + in_slot, v ? &maps.vp : &maps.kp, pg * a.pool.n_kv + d.h,
                          bar(to));
        }
        if (!ok) break;
        gs += 2;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
    }
    const int zero = 0;
    if (my_bar) mbar_wait_bounded(my_bar, my_par, &zero);
    __syncwarp();
  } else if (kQ8 && warp == 10) {
    // ----------------------------------------- q8_0 codes and scales, raw ----
    int gs = 0;
    uint32_t my_bar = 0, my_par = 0;  // lane s: the last copy's barrier of stage s
    bool ok = true;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      const int32_t* bt = a.rows.block_table + static_cast<long long>(d.i) * a.rows.bt_stride;
      auto entry = [&](int b) {  // lane e: page e of the block, -1 where it is not read
        int lo, hi;
        pages_of(d, b, lo, hi);
        const int q = block(d.kb, d.nb, b) * kPages + lane;
        return lane < kPages && q >= lo && q < hi ? __ldg(bt + q) : -1;
      };
      int next = entry(0);
      for (int b = 0; b < d.nb && ok; ++b) {
        int pg = next;
        if (b + 1 < d.nb) next = entry(b + 1);
        int lo, hi;
        pages_of(d, b, lo, hi);
        const int q = block(d.kb, d.nb, b) * kPages + lane;
        const bool mine = lane < kPages && q >= lo && q < hi;
        if (mine && (pg < 0 || pg >= a.pool.num_pages)) {
          record_status(a.pool.status, PKV_DEV_BAD_PAGE);
          pg = 0;
        }
#pragma unroll
        for (int v = 0; v < 2; ++v, ++gs) {
          const int rs = gs % kRaws;
          if (gs >= kRaws && !(ok = wait(kBRawEmpty + rs, gs / kRaws - 1))) break;
          if (lane == rs) {
            my_bar = bar(kBRaw + rs);
            my_par = static_cast<uint32_t>(gs / kRaws) & 1u;
          }
          if (lane == 0)
            mbar_arrive_expect_tx(bar(kBRaw + rs), static_cast<uint32_t>(hi - lo) * (kPage * kD + kPage * 8));
          __syncwarp();
          if (mine) {
            const long long tile = static_cast<long long>(pg) * a.pool.n_kv + d.h;
            tc::load_page(sbase + kRaw + rs * kRawBytes + lane * (kPage * kD), v ? &maps.vp : &maps.kp,
                          static_cast<int>(tile), bar(kBRaw + rs));
            tc::load_bytes(sbase + kRawScales + rs * kRawScaleBytes + lane * (kPage * 8),
                           (v ? a.pool.v_scales : a.pool.k_scales) + tile * (kPage * 8), kPage * 8, bar(kBRaw + rs));
          }
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
    }
    const int zero = 0;
    if (my_bar) mbar_wait_bounded(my_bar, my_par, &zero);
    __syncwarp();
  } else if (!kQ8 && warp == 11) {
    // ------------------------------------------------------------ mending ----
    int gs = 0;
    uint32_t landed = 0;
    bool ok = true;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      for (int b = 0; b < d.nb; ++b, gs += 2) {
        if (!mended(d, b)) continue;
        const int s = (gs + 1) % kS;
        if (!wait(kBLand + s, (landed >> s) & 1u)) {
          ok = false;
          break;
        }
        landed ^= 1u << s;
        uint8_t* v = smem + kRing + s * kHalf;
        const int t0 = block(d.kb, d.nb, b) * N;
        int lo, hi;
        pages_of(d, b, lo, hi);
        // tokens of the pages read that no query of the tile attends to
        for (int t = lo * kPage + lane; t < hi * kPage; t += 32) {
          if (t >= d.t_lo && t < d.t_hi) continue;
          const int u = t - t0;  // token of the block: page u / 16, group (u / 8) % 2
          uint4* row = reinterpret_cast<uint4*>(v + (u >> 3) * 2048 + (u & 7) * 128);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            row[e] = make_uint4(0u, 0u, 0u, 0u);
            row[64 + e] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        __syncwarp();
        // 0 * x is NaN for the others
        uint32_t bits = 0;
        const uint4* w = reinterpret_cast<const uint4*>(v + (lo & (kPages - 1)) * 4096);
        const int n16 = (hi - lo) * 256;
        if constexpr (DT == PKV_KV_BF16) {
          __nv_bfloat162 acc = __floats2bfloat162_rn(0.f, 0.f);
          const __nv_bfloat162 z = acc;
#pragma unroll 8
          for (int e = lane; e < n16; e += 32) {
            const uint4 q = w[e];
            acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&q.x), z, acc);
            acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&q.y), z, acc);
            acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&q.z), z, acc);
            acc = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&q.w), z, acc);
          }
          bits = *reinterpret_cast<const uint32_t*>(&acc);
        } else {
          __half2 acc = __floats2half2_rn(0.f, 0.f);
          const __half2 z = acc;
#pragma unroll 8
          for (int e = lane; e < n16; e += 32) {
            const uint4 q = w[e];
            acc = __hfma2(*reinterpret_cast<const __half2*>(&q.x), z, acc);
            acc = __hfma2(*reinterpret_cast<const __half2*>(&q.y), z, acc);
            acc = __hfma2(*reinterpret_cast<const __half2*>(&q.z), z, acc);
            acc = __hfma2(*reinterpret_cast<const __half2*>(&q.w), z, acc);
          }
          bits = *reinterpret_cast<const uint32_t*>(&acc);
        }
        if (__any_sync(kFull, (bits & 0x7FFF7FFFu) != 0u) && lane == 0) {
          ctl[1] = 1;
          note_piece(tail.notes, p);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the zeroed rows
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBFull + s));
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
    }
    fill_skipped(a);
  } else if (warp == 9) {
    // ----------------------------------------------------------- products ----
    // converged and uniform throughout: see tcgen05.cuh
    const uint32_t lead = tc::elect_one();
    const uint32_t tm = tc::uniform(tmem);
    constexpr uint32_t id_s = tc::idesc(128, 128, false, false, F::kFormat);
    constexpr uint32_t id_o = tc::idesc(128, 128, false, true, F::kFormat);
    constexpr uint32_t kHiQ = tc::desc_hi(1024), kHiKV = tc::desc_hi(2048);
    const uint32_t q_lo = tc::desc_lo(sbase, 16), k_lo = tc::desc_lo(sbase + kRing, 16),
                   v_lo = tc::desc_lo(sbase + kRing, 1024);
    // scores S_m of the K block in slot s (q8_0: 64 columns with the hi parts,
    // and 64 with the lo parts, which the softmax adds)
    auto issue_s = [&](int m, int s, int q) {
      const uint32_t qd = q_lo + q * (kHalf >> 4), kd = k_lo + s * (kHalf >> 4);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        tc::mma_ss<kHiQ, kHiKV>(tm + kTmemS + 128 * m, qd + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4),
                                kd + (((kk >> 2) * 1024 + (kk & 3) * 32) >> 4), id_s, kk > 0, lead);
      tc::commit(bar(kBS + m), lead);
    };
    // the block whose values product is due
    struct {
      int s, lo, n, m;       // V slot, first page in it, pages; the (first) half
      bool first, last, two;
    } v{0, 0, 0, 0, false, false, false};
    bool due = false;
    uint32_t np[2] = {0, 0};  // blocks of P consumed per half
    int gs = 0;
    bool ok = true, any = false;
    // O_m of the due block, whose V is in its slot, once P_m is written
    auto issue_o = [&](int m) {
      const uint32_t vd = v_lo + v.s * (kHalf >> 4);
      const uint32_t to = tm + kTmemO + 128 * m, tp = tm + kTmemS + 128 * m;
      const int fresh = v.first ? 0 : 1;
      if (!wait(kBP + m, np[m])) return false;
      ++np[m];
      tc::fence_after();
      if (v.n == kPages) {
#pragma unroll
        for (int kk = 0; kk < kPages; ++kk) {
          tc::mma_ts<kHiKV>(to, tp + 8 * kk, vd + kk * (4096 >> 4), id_o, kk > 0 ? 1 : fresh, lead);
          if constexpr (kQ8) tc::mma_ts<kHiKV>(to, tp + 8 * kk, vd + ((kPart + kk * 4096) >> 4), id_o, 1, lead);
        }
      } else {
#pragma unroll 1
        for (int kk = v.lo; kk < v.lo + v.n; ++kk) {
          tc::mma_ts<kHiKV>(to, tp + 8 * kk, vd + kk * (4096 >> 4), id_o, kk > v.lo ? 1 : fresh, lead);
          if constexpr (kQ8) tc::mma_ts<kHiKV>(to, tp + 8 * kk, vd + ((kPart + kk * 4096) >> 4), id_o, 1, lead);
        }
      }
      if (v.last) tc::commit(bar(kBO + m), lead);
      return true;
    };
    auto finish_o = [&] { return (v.m == 1 || issue_o(0)) && (!(v.two || v.m == 1) || issue_o(1)); };
    uint32_t q1 = 0;
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) { ok = false; break; }
      const Piece& d = tail.piece[x];
      if (tc::uniform(d.last)) break;
      const int nb = tc::uniform(d.nb), t_lo = tc::uniform(d.t_lo), t_hi = tc::uniform(d.t_hi),
                kb = tc::uniform(d.kb);
      const bool two = tc::uniform(d.nq) * G > kTileRows / 2;
      any = true;
      for (int b = 0; b < nb && ok; ++b) {
        // gs: the slot of this block's K; gs - 1 that of the due block's V.
        // What lands early is waited for first: once P_m is there, its product
        // and the next scores go out without another wait.  The halves are
        // constants everywhere: with a variable half the products' addresses
        // are not uniform registers (438 us instead of 405 for the prompt).
        const int s = gs % kS;
        if (due && !(ok = wait(kBFull + v.s, static_cast<uint32_t>(gs - 1) / kS))) break;
        if (b == 0) {
          // the piece before is finished while this one's queries land
          if (due) {
            if (!(ok = finish_o())) break;
            tc::commit(bar(kBEmpty + v.s), lead);
            due = false;
          }
          if (!(ok = wait(kBQ, p) && (!two || wait(kBQ + 1, q1)))) break;
        }
        if (!(ok = wait(kBFull + s, gs / kS))) break;
        if (!kTurns || two) {
          if (due) {
            if (!(ok = issue_o(0))) break;
          } else {
            tc::fence_after();
          }
          issue_s(0, s, 0);
          if (due) {
            if (v.two && !(ok = issue_o(1))) break;
            tc::commit(bar(kBEmpty + v.s), lead);
          }
          if (two) issue_s(1, s, 1);
        } else {
          // the scores go out before the product of the block before, whose
          // weights are still made
          tc::fence_after();
          if (b & 1) {
            issue_s(1, s, 0);
            if (due && !(ok = issue_o(0))) break;
          } else {
            issue_s(0, s, 0);
            if (due && !(ok = issue_o(1))) break;
          }
          if (due) tc::commit(bar(kBEmpty + v.s), lead);
        }
        tc::commit(bar(kBEmpty + s), lead);
        if (b + 1 == nb) tc::commit(bar(kBQEmpty), lead);
        const int first = block(kb, nb, b) * kPages;
        const int lo = max(first, t_lo / kPage), hi = min(first + kPages, (t_hi + kPage - 1) / kPage);
        v.s = (gs + 1) % kS;
        v.lo = lo & (kPages - 1);
        v.n = hi - lo;
        v.m = kTurns && !two ? b & 1 : 0;
        v.first = b < (!kTurns || two ? 1 : 2);
        v.last = b + (!kTurns || two ? 1 : 2) >= nb;
        v.two = two;
        due = true;
        gs += 2;
      }
      if (!ok) break;
      q1 += two ? 1 : 0;
      if (lane == 0) mbar_arrive(bar(kBDescEmpty + x));
      __syncwarp();
    }
    if (ok && due && wait(kBFull + v.s, static_cast<uint32_t>(gs - 1) / kS)) finish_o();
    // every product issued completes before the tensor memory is freed
    if (any) {
      const int zero = 0;
      tc::commit(bar(kBDrain), lead);
      __syncwarp();
      if (lane == 0) mbar_wait_bounded(bar(kBDrain), 0, &zero);
      __syncwarp();
    }
  }
  } else {
    // ------------------------------------------------------------ softmax ----
    if constexpr (kQ8) tc::more_registers<144>();
    const int m = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t tS = tmem + lanes + kTmemS + 128 * m, tO = tS + (kTmemO - kTmemS);
    const int r_half = 32 * quarter + lane, jq_full = (r_half + 128 * m) / G;
    uint32_t blocks = 0, pieces = 0, joins = 0;
    bool ok = !stalled;
    const float c1 = a.sc.scale * kLog2e;
    const float cap_k = a.sc.softcap > 0.0f ? a.sc.scale / a.sc.softcap : 0.0f, cap2 = a.sc.softcap * kLog2e;
    const NearCap cap(cap_k, cap2);
    for (int p = 0; ok; ++p) {
      const int x = p % kDescs;
      if (!wait(kBDesc + x, p / kDescs)) break;
      const Piece d = tail.piece[x];
      if (d.last) break;
      const bool two = d.nq * G > kTileRows / 2;
      // A tile of up to 128 rows: the halves take its blocks in turn, so that
      // one's scores are made while the other's go through the softmax.
      const bool join = kTurns && !two && d.nb > 1;
      bool begun = false;  // O holds an earlier block
      const int r = kTurns && !two ? r_half : r_half + 128 * m;  // row of the tile
      const int jq = kTurns ? r / G : jq_full;                   // its query
      const int every = !kTurns || two ? 1 : 2;
      if (m == 0 || two || join) {
        const bool valid = jq < d.nq;
        const bool any = __any_sync(kFull, valid);
        const int P = d.P0 + jq, g = d.h * G + r % G;
        const int lo = valid ? seen_from(P, a.pool.window) : 0;
        const int hi = valid ? seen_to(P, d.L, d.F) : 0x7FFFFFFF;
        float slope2 = 0.0f;
        bool behind = true;
        if constexpr (GEN == 2) {
          slope2 = a.sc.slopes ? __ldg(a.sc.slopes + g) * kLog2e : 0.0f;
          behind = __all_sync(kFull, !valid || hi <= P + 1);
        }
        constexpr float kMasked = GEN == 1 ? -1e15f : -INFINITY, kNone = GEN == 1 ? -1e14f : -INFINITY;
        float mx = kNone;      // the maximum in force, base 2
        float sub = 0.0f;      // what is taken off the scores: mx - shift (0 before a first score)
        float l = 0.0f;
        float most = -1.0f;    // a group's sum beyond which its maximum is looked at
        for (int b = !kTurns || two ? 0 : m; b < d.nb; b += every, ++blocks, begun = true) {
          const int t0 = block(d.kb, d.nb, b) * N;
          const bool fast = __all_sync(kFull, t0 >= lo && t0 + N <= hi);
          const float near = GEN == 1 ? cap.limit(valid, fast) : 0.0f;
          if (!(ok = wait(kBS + m, blocks))) break;
          tc::fence_after();
          if (any) {
            // The block goes by in groups of 32 columns, in a loop of one group:
            // its code has to stay in the instruction caches that six other
            // loops share (two groups, the loads from tensor memory one ahead of
            // the arithmetic: 395 us instead of 377 for 8191 tokens).  A group's exponentials start under the maximum in force.
            // Should their sum exceed 256 (or a row have no maximum yet), the
            // group's own maximum is found; if that exceeds the one in force by
            // more than 8 (rare after a tile's first block) the maximum is raised
            // and they are taken again.  Raises are by whole powers of two, so
            // that the weights already written for the block are rescaled
            // without another rounding.  The maximum of every group costs 8 us of
            // 403 beside the exponentials, and 450 cycles a block before them.
            auto raise_to = [&](float bm, int group) {
              const bool raise = bm > mx + 8.0f;  // also from none
              float al = 1.0f;
              if (raise) {
                const float to = mx == kNone ? bm : mx + ceilf(bm - mx);
                al = tc::ex2(mx - to);  // a power of two, or 0
                mx = to;
                sub = to - F::kShift;
                l *= al;
                most = 256.0f * F::kScale;
              }
              // the block's weights so far, and O: the values products before
              // are complete, S was issued after them
              tc::wait_ld();
              if (group > 0 || (kTurns ? begun : b > 0)) {
                if constexpr (kQ8) rescale_here<DT>(tS, tO, group, b > 0, al);  // no registers for a call
                else rescale<DT>(tS, tO, group, begun, al);
              }
            };
            // With a bias the scores get slope (t - P) with the exponentials'
            // subtraction, -slope (t - P) for tokens after the query; a cap
            // is their factor there, q(v^2) instead of c1: there a masked
            // score is one far below the cap's, whose square is finite.
            auto weigh = [&](float (&v)[32], int group) {
              float2 mul = make_float2(c1, c1);
              float bias = 0.0f, step = 0.0f;  // of the group's first column; per column
              float cq[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              if constexpr (GEN == 1) {
                if (__builtin_expect(cap.beyond(v, near), 0)) {
                  cap32(v, tS + 32 * group, cap_k, cap2);
                  cq[0] = 1.0f;
                } else {
#pragma unroll
                  for (int e = 0; e < 4; ++e) cq[e] = cap.q[e];
                }
              }
              if constexpr (GEN == 2) {
                if (a.sc.softcap > 0.0f) {
                  cap32(v, tS + 32 * group, cap_k, cap2);
                  mul = make_float2(1.0f, 1.0f);
                } else if (!(c1 > 0.0f)) {  // the mask's -inf has to stay one
#pragma unroll
                  for (int e = 0; e < 32; ++e) v[e] *= c1;
                  mul = make_float2(1.0f, 1.0f);
                }
              }
              if constexpr (GEN == 2) {
                const float dist0 = static_cast<float>(t0 + 32 * group - P);  // t - P of the first column
                const bool before = behind || dist0 <= -31.0f, after = dist0 >= 0.0f;
                if (__builtin_expect(__any_sync(kFull, valid && !before && !after), 0)) {  // seen on both sides
#pragma unroll
                  for (int e = 0; e < 32; ++e) v[e] = fmaf(-slope2, fabsf(dist0 + static_cast<float>(e)), v[e] * mul.x);
                  mul = make_float2(1.0f, 1.0f);
                } else {
                  step = before ? slope2 : -slope2;
                  bias = step * dist0;
                }
              }
              if (__builtin_expect(!fast, 0)) {
                const int from = lo - t0 - 32 * group, to = hi - t0 - 32 * group;
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = e >= from && e < to ? v[e] : kMasked;
              }
              uint32_t w[16];
              float2 lb[2];
              float group_sum;
#pragma unroll 1
              while (true) {
                float2 off[4];  // of columns 2u, 2u + 1 and every eighth after
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  off[u] = make_float2(bias - sub, bias - sub);
                  if constexpr (GEN == 2) off[u] = make_float2(fmaf(step, 2.0f * u, off[u].x), fmaf(step, 2.0f * u + 1.0f, off[u].y));
                }
                const float2 next = make_float2(8.0f * step, 8.0f * step);
                float x0 = -INFINITY, x1 = -INFINITY;
                lb[0] = lb[1] = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                  const float2 x = make_float2(v[2 * u], v[2 * u + 1]);
                  float2 f = mul;
                  if constexpr (GEN == 1) {
                    const float2 xx = tc::fma2(x, x, make_float2(0.0f, 0.0f));
                    f = tc::fma2(xx, make_float2(cq[3], cq[3]), make_float2(cq[2], cq[2]));
                    f = tc::fma2(xx, f, make_float2(cq[1], cq[1]));
                    f = tc::fma2(xx, f, make_float2(cq[0], cq[0]));
                  }
                  const float2 y = tc::fma2(x, f, off[u & 3]);
                  if constexpr (GEN == 2) off[u & 3] = tc::add2(off[u & 3], next);
                  if constexpr (GEN != 0) {
                    if (u & 1) x1 = tc::max3(x1, y.x, y.y); else x0 = tc::max3(x0, y.x, y.y);
                  }
                  const float2 pr = make_float2(tc::ex2(y.x), tc::ex2(y.y));
                  lb[u & 1] = tc::add2(lb[u & 1], pr);
                  w[u] = F::pack(pr.x, pr.y);
                }
                const float2 both = tc::add2(lb[0], lb[1]);
                group_sum = both.x + both.y;
                if constexpr (GEN == 0) {
                  if (__builtin_expect(!__any_sync(kFull, group_sum > most), 1)) break;
#pragma unroll
                  for (int u = 0; u < 16; ++u) {
                    if (u & 1) x1 = tc::max3(x1, v[2 * u], v[2 * u + 1]); else x0 = tc::max3(x0, v[2 * u], v[2 * u + 1]);
                  }
                }
                const float bm = GEN != 0 ? fmaxf(x0, x1) + sub : fmaxf(x0, x1) * c1;
                if (__builtin_expect(!__any_sync(kFull, bm > mx + 8.0f), 1)) break;
                raise_to(bm, group);
              }
              l += group_sum;
              tc::st16(tS + 16 * group, w);
            };
            float v[32];
            float more[kQ8 ? 32 : 1];  // q8_0: the lo parts' scores
            auto load = [&](float (&v)[32], int group) {
              tc::ld32(tS + 32 * group, v);
              if constexpr (kQ8) tc::ld32(tS + 64 + 32 * group, more);
            };
            auto arrived = [&](float (&v)[32]) {
              tc::wait_ld();
              if constexpr (kQ8) {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] += more[e];
              }
            };
#pragma unroll 1
            for (int group = 0; group < N / 32; ++group) {
              load(v, group);
              arrived(v);
              weigh(v, group);
            }
            tc::wait_st();
          }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBP + m));
        }
        if (!ok || !(ok = wait(kBO + m, pieces))) break;
        ++pieces;
        tc::fence_after();
        float f0 = 1.0f, f1 = 0.0f;  // the halves' factors
        if (join && m == 1) {  // O_1 is complete, and half 0 reads it
          tail.half[32 * quarter + lane] = make_float2(sub, l);
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBHalf));
          if (!(ok = wait(kBJoined, joins))) break;  // before the next piece's P_1
          ++joins;
        } else if (join) {
          if (!(ok = wait(kBHalf, joins))) break;
          ++joins;
          tc::fence_after();
          const float2 o = tail.half[32 * quarter + lane];
          // a half without tokens of the row weighs nothing
          const float top = !(o.y > 0.0f) ? sub : !(l > 0.0f) ? o.x : fmaxf(sub, o.x);
          f0 = l == 0.0f ? 0.0f : tc::ex2(sub - top);
          f1 = o.y == 0.0f ? 0.0f : tc::ex2(o.x - top);
          l = fmaf(f0, l, f1 * o.y);
          sub = top;
        }
        if (any && (two || m == 0)) {
          const float inv = d.slot >= 0 ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
          f0 *= inv;
          f1 *= inv;
          const long long row = static_cast<long long>(d.tok + jq) * a.n_q + g;
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            float o[32];
            tc::ld32(tO + 32 * e, o);
            tc::wait_ld();
#pragma unroll
            for (int u = 0; u < 32; ++u) o[u] *= f0;
            if (join) {
              float o1[32];
              tc::ld32(tO + 128 + 32 * e, o1);
              tc::wait_ld();
#pragma unroll
              for (int u = 0; u < 32; ++u) o[u] = fmaf(f1, o1[u], o[u]);
            }
            if (valid) {
              if (d.slot >= 0) {
                float4* acc = slot_acc(a, d.slot) + r;
#pragma unroll
                for (int u = 0; u < 8; ++u)
                  acc[(8 * e + u) * kTileRows] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
              } else {
                uint4* to = reinterpret_cast<uint4*>(a.out + (row * kD + 32 * e) * 2);
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  to[u] = make_uint4(F::pack(o[8 * u], o[8 * u + 1]), F::pack(o[8 * u + 2], o[8 * u + 3]),
                                     F::pack(o[8 * u + 4], o[8 * u + 5]), F::pack(o[8 * u + 6], o[8 * u + 7]));
              }
            }
          }
          tc::fence_before();  // O read before the next piece's first values product
          if (valid) {
            if (d.slot >= 0)
              slot_ml(a, d.slot)[r] = make_float2(l > 0.0f ? sub : -INFINITY, l);
            else if (a.lse)
              a.lse[row] = (sub + log2f(l)) * kLn2;
          }
        }
        if (join && m == 0) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBJoined));
        }
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
  // (the warps with registers for it; a range that was given up has stored nothing to go by)
  if (warp < kMendWarps && ctl[1] && !ctl[0]) mend_rows<DT>(a, tail.notes, tail.bounds[0], tail.bounds[1], tail.tiles);
}

// ---------------------------------------------------------------- merge ----
// CTA (k, y): if boundary k + 1 is the first to cut its tile, the tile's rows
// 32 y .. from its pieces: the end of range k and the starts of the ranges
// whose boundaries cut it.  A thread takes 16 dims of a row; the records, and
// then the pieces four at a time, are loaded together, so that a merge of a few
// pieces is three trips to memory.
constexpr int kMergeThreads = 256;
template <int DT>
__global__ void __launch_bounds__(kMergeThreads) chunk_merge_kernel(const __grid_constant__ ChunkAttnArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int k0 = blockIdx.x + 1;
  grid_dependency_wait();
  grid_launch_dependents();
  const Rec* rec = reinterpret_cast<const Rec*>(a.workspace);
  auto load_rec = [&](int k) { return *reinterpret_cast<const int4*>(rec + k); };
  const int4 prev = load_rec(k0 - 1), me = load_rec(k0);  // inside, h, tile, tok
  const int nq = rec[k0].nq;
  int4 ahead = make_int4(0, 0, 0, 0);  // lane l: boundary k0 + 1 + l
  if (k0 + 1 + lane < a.chunks) ahead = load_rec(k0 + 1 + lane);
  if (!me.x || (prev.x && prev.y == me.y && prev.z == me.z)) return;
  const int G = a.n_q / a.pool.n_kv;
  const int r = 32 * blockIdx.y + lane;
  if (32 * static_cast<int>(blockIdx.y) >= nq * G) return;
  // the boundaries after k0 that cut the tile
  int cuts = 0;
  for (int base = k0 + 1;; base += 32) {
    const unsigned same = __ballot_sync(kFull, ahead.x && ahead.y == me.y && ahead.z == me.z);
    if (same != kFull) {
      cuts += __ffs(~same) - 1;
      break;
    }
    cuts += 32;
    ahead = base + 32 + lane < a.chunks ? load_rec(base + 32 + lane) : make_int4(0, 0, 0, 0);
  }
  if (r >= nq * G) return;
  // piece 0: slot 2 (k0 - 1) + 1; piece u: slot 2 (k0 + u - 1)
  const int pieces = cuts + 2;
  float M = -INFINITY, Lsum = 0.0f;
  float4 acc[4];  // dims 16 warp ..
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int u0 = 0; u0 < pieces; u0 += 4) {
    float2 ml[4];
    float4 v[4][4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      ml[u] = make_float2(-INFINITY, 0.0f);
      if (u0 + u < pieces) {
        const int s = u0 + u == 0 ? 2 * k0 - 1 : 2 * (k0 + u0 + u - 1);
        ml[u] = slot_ml(a, s)[r];
        const float4* src = slot_acc(a, s) + r;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[u][e] = src[(4 * warp + e) * kTileRows];
      }
    }
    float m = M;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (ml[u].y != 0.0f) m = fmaxf(m, ml[u].x);
    if (m == -INFINITY) m = 0.0f;  // no token of the row so far
    const float keep = tc::ex2(M - m);
    Lsum *= keep;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[e].x *= keep;
      acc[e].y *= keep;
      acc[e].z *= keep;
      acc[e].w *= keep;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (ml[u].y == 0.0f) continue;  // no token of the row in the piece (or no piece)
      const float w = tc::ex2(ml[u].x - m);
      Lsum = fmaf(w, ml[u].y, Lsum);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[e].x = fmaf(w, v[u][e].x, acc[e].x);
        acc[e].y = fmaf(w, v[u][e].y, acc[e].y);
        acc[e].z = fmaf(w, v[u][e].z, acc[e].z);
        acc[e].w = fmaf(w, v[u][e].w, acc[e].w);
      }
    }
    if (Lsum != 0.0f) M = m;
  }
  const float inv = 1.0f / Lsum;
  const long long row = static_cast<long long>(me.w + r / G) * a.n_q + me.y * G + r % G;
  uint4* to = reinterpret_cast<uint4*>(a.out + (row * kD + 16 * warp) * 2);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float4 p = acc[2 * e], q = acc[2 * e + 1];
    to[e] = make_uint4(Io<DT>::pack(p.x * inv, p.y * inv), Io<DT>::pack(p.z * inv, p.w * inv),
                       Io<DT>::pack(q.x * inv, q.y * inv), Io<DT>::pack(q.z * inv, q.w * inv));
  }
  if (a.lse && warp == 0) a.lse[row] = (M + log2f(Lsum)) * kLn2;
}

// ------------------------------------------------------------- launchers ----
template <int DT, int GEN>
cudaError_t launch_attention_t(const ChunkAttnArgs& a, const TileMaps& maps, const CUtensorMap& qmap, cudaStream_t st) {
  static std::atomic<int> granted[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !granted[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(chunk_attention_kernel<DT, GEN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) granted[dev].store(1, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.chunks);
  cfg.blockDim = dim3(kAttnThreads<DT>);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, chunk_attention_kernel<DT, GEN>, a, maps, qmap);
  if (e != cudaSuccess) return e;
  if (a.chunks > 1) {
    cfg.gridDim = dim3(a.chunks - 1, kTileRows / 32);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, chunk_merge_kernel<DT>, a);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_attention_g(const ChunkAttnArgs& a, const TileMaps& maps, const CUtensorMap& qmap, cudaStream_t st) {
  if (a.sc.slopes || !(a.sc.scale > 0.0f) || a.sc.softcap > 1e9f) return launch_attention_t<DT, 2>(a, maps, qmap, st);
  if (a.sc.softcap > 0.0f) return launch_attention_t<DT, 1>(a, maps, qmap, st);
  return launch_attention_t<DT, 0>(a, maps, qmap, st);
}

}  // namespace

size_t chunk_attention_workspace(int n_q, int n_kv, int chunks) {
  (void)n_q;
  (void)n_kv;
  return rec_bytes(chunks) + 2 * static_cast<size_t>(chunks) * kSlotFull;
}

cudaError_t launch_chunk_attention(const ChunkAttnArgs& a, const TileMaps& maps, cudaStream_t st) {
  CUtensorMap qmap;
  cudaError_t e = encode_query_map(&qmap, a.pool.dtype == PKV_KV_BF16, a.q, a.q_stride, a.n_q, a.n_q / a.pool.n_kv,
                                   a.rows.total_tokens, 128 / (a.n_q / a.pool.n_kv));
  if (e != cudaSuccess) return e;
  if (a.pool.dtype == PKV_KV_F16) return launch_attention_g<PKV_KV_F16>(a, maps, qmap, st);
  if (a.pool.dtype == PKV_KV_BF16) return launch_attention_g<PKV_KV_BF16>(a, maps, qmap, st);
  return launch_attention_g<PKV_KV_Q8_0>(a, maps, qmap, st);
}

// The queries as a 4-D tensor {64 dims, heads, tokens, 2 halves of the dims},
// box {64, G, queries, 2}: a copy lands [half][query, head][64 dims] under the
// 128-byte swizzle, the K-major layout of a product's first operand.  Tokens
// behind the last read as zeros.
cudaError_t encode_query_map(CUtensorMap* m, bool bf16, const void* q, long long stride, int heads, int group,
                             int tokens, int queries) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!fn) return cudaErrorNotSupported;
  const cuuint64_t dims[4] = {64u, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens), 2u};
  const cuuint64_t strides[3] = {kD * 2, static_cast<cuuint64_t>(stride) * 2, 128u};
  const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(queries), 2u};
  const cuuint32_t estride[4] = {1u, 1u, 1u, 1u};
  const CUresult r = fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                        const_cast<void*>(q), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace pkv
