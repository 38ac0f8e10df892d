// evict.cu — kv_evict: shorten rows to their budget per KV head, keeping the
// tokens that received the most attention.
//
// Selecting.  A token's key is its weight as an unsigned integer of the same
// order (NaN lowest; the protected first and recent tokens highest), so the B
// kept tokens of a (row, KV head) are the B largest keys with ties to the
// lowest index.  The B-th largest key T is found digit by digit from the top
// (11, 11 and 10 bits): a histogram of the digit over the keys that match the
// digits found so far, and the digit at which the count from above reaches B.
// Then token t is kept if its key exceeds T, or equals T with fewer than
// (B - #greater) equals before it; its place among the kept is
//     #greater before t + min(#equal before t, B - #greater),
// two prefix sums.  A cluster of CTAs shares one (row, KV head), each with a
// contiguous slice of its tokens; the histograms and the slices' counts meet
// through distributed shared memory.  The keys are read once and kept in
// shared memory while the slice fits, and re-read (from L2) beyond.
//
// Gathering.  The kept tokens go to fresh pages, so every copy is independent:
// a CTA takes 64 kept tokens of a head and moves their K and V in 16-byte
// pieces.  Bound by memory: the bytes are the kept K and V, read and written
// once; the weights of the whole row are a few percent of them.
#include <cstdint>

#include "chunk_device.cuh"

namespace pkv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kCachedKeys = 8192;  // a slice of this many keys stays in shared memory
constexpr int kGatherTokens = 64;
constexpr int kGatherThreads = 256;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrive and wait with release / acquire order over the cluster's threads.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of CTA `rank`'s shared memory, at the place `addr` has in this CTA's.
__device__ __forceinline__ uint32_t peer_load(uint32_t addr, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// The row's tokens L and budget B, clamped to what the tables hold.
__device__ __forceinline__ void row_budget(const EvictArgs& a, int i, int32_t* status, int& L, int& B) {
  const long long cap = min(static_cast<long long>(a.bt_stride) * kPage, static_cast<long long>(a.mass_stride));
  L = __ldg(a.seq_lens + i);
  if (L < 0 || L > cap) {
    record_status(status, PKV_DEV_BAD_LENGTH);
    L = L < 0 ? 0 : static_cast<int>(cap);
  }
  const long long room = min(static_cast<long long>(a.dst_bt_stride) * kPage, static_cast<long long>(a.keep_stride));
  B = min(L, __ldg(a.keep_lens + i));
  if (B < 0 || B > room) {
    record_status(status, PKV_DEV_BAD_LENGTH);
    B = B < 0 ? 0 : static_cast<int>(room);
  }
}

// Unsigned key of the same order as x: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b >> 31) ? ~b : (b | 0x80000000u);
}

struct SelShared {
  uint32_t hist[kBins];
  uint32_t scan[kSelWarps];
  uint32_t pick[2];      // the digit, and the count above it
  uint32_t totals[2];    // greater and equal keys of this CTA's slice
  uint32_t seg[2][kSelWarps];
};

template <int CS>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];  // [kCachedKeys]
  __shared__ SelShared sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = CS > 1 ? cluster_rank() : 0u;
  const int seg = blockIdx.x / CS;  // (row, KV head)
  const int i = seg / a.pool.n_kv, h = seg - i * a.pool.n_kv;
  grid_dependency_wait();
  grid_launch_dependents();
  int L, B;
  row_budget(a, i, (h == 0 && rank == 0 && tid == 0) ? a.pool.status : nullptr, L, B);
  const float* mass = a.mass + static_cast<long long>(seg) * a.mass_stride;
  int32_t* keep = a.keep_idx + static_cast<long long>(seg) * a.keep_stride;
  float* kept_mass = a.dst_mass ? a.dst_mass + static_cast<long long>(seg) * a.keep_stride : nullptr;
  if (h == 0 && rank == 0 && tid == 0) a.new_lens[i] = B;
  if (B == L || B == 0) {  // uniform over the cluster: everything kept, or nothing
    for (int t = static_cast<int>(rank) * kSelThreads + tid; t < B; t += CS * kSelThreads) {
      keep[t] = t;
      if (kept_mass) kept_mass[t] = mass[t];
    }
    return;
  }
  const int recent = min(a.recent, B), first = min(a.first, B - recent);
  // this CTA's slice [s0, s1), cut at multiples of 32
  const int groups = (L + 31) / 32, per = (groups + CS - 1) / CS;
  const int s0 = min(L, static_cast<int>(rank) * per * 32), s1 = min(L, s0 + per * 32);
  const bool cached = s1 - s0 <= kCachedKeys;
  auto fetch = [&](int t) {
    if (t < first || t >= L - recent) return 0xFFFFFFFFu;
    return key_of(__ldg(mass + t));
  };
  auto key = [&](int t) { return cached ? keys[t - s0] : fetch(t); };
  if (cached)
    for (int t = s0 + tid; t < s1; t += kSelThreads) keys[t - s0] = fetch(t);

  uint32_t prefix = 0, mask = 0;  // the digits of T found so far
  uint32_t want = static_cast<uint32_t>(B);
  const uint32_t hist_at = smem_addr(sm.hist);
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
    for (int b = tid; b < kBins; b += kSelThreads) sm.hist[b] = 0u;
    __syncthreads();
    for (int t = s0 + tid; t < s1; t += kSelThreads) {
      const uint32_t x = key(t);
      if ((x & mask) == prefix) atomicAdd(&sm.hist[(x >> shift) & digit_mask], 1u);
    }
    if (CS > 1) cluster_sync(); else __syncthreads();
    // thread tid holds two bins, counted from the top
    const int b0 = kBins - 1 - 2 * tid, b1 = b0 - 1;
    uint32_t c0 = 0, c1 = 0;
#pragma unroll
    for (int r = 0; r < CS; ++r) {
      c0 += CS > 1 ? peer_load(hist_at + 4 * b0, r) : sm.hist[b0];
      c1 += CS > 1 ? peer_load(hist_at + 4 * b1, r) : sm.hist[b1];
    }
    uint32_t v = c0 + c1;  // inclusive scan of the pairs
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) sm.scan[warp] = v;
    __syncthreads();
    uint32_t before = lane < warp ? sm.scan[lane] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(kFull, before, o);
    const uint32_t above0 = before + v - c0 - c1, above1 = above0 + c0;
    if (above0 < want && want <= above0 + c0) {
      sm.pick[0] = static_cast<uint32_t>(b0);
      sm.pick[1] = above0;
    } else if (above1 < want && want <= above1 + c1) {
      sm.pick[0] = static_cast<uint32_t>(b1);
      sm.pick[1] = above1;
    }
    if (CS > 1) cluster_sync(); else __syncthreads();  // every peer has read this CTA's counts
    prefix |= sm.pick[0] << shift;
    mask |= digit_mask << shift;
    want -= sm.pick[1];
    __syncthreads();
  }
  // want: how many keys equal to T = prefix are kept.  Each warp takes a
  // contiguous part of the slice.
  const int len = s1 - s0;
  const int wgroups = ((len + 31) / 32 + kSelWarps - 1) / kSelWarps;
  const int w0 = min(s1, s0 + warp * wgroups * 32), w1 = min(s1, w0 + wgroups * 32);
  uint32_t ngt = 0, neq = 0;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const uint32_t x = t < w1 ? key(t) : 0u;
    ngt += __popc(__ballot_sync(kFull, t < w1 && x > prefix));
    neq += __popc(__ballot_sync(kFull, t < w1 && x == prefix));
  }
  if (lane == 0) {
    sm.seg[0][warp] = ngt;
    sm.seg[1][warp] = neq;
  }
  __syncthreads();
  uint32_t gt = lane < warp ? sm.seg[0][lane] : 0u, eq = lane < warp ? sm.seg[1][lane] : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(kFull, gt, o);
    eq += __shfl_xor_sync(kFull, eq, o);
  }
  if (CS > 1) {
    if (warp == kSelWarps - 1 && lane == 0) {
      sm.totals[0] = gt + ngt;
      sm.totals[1] = eq + neq;
    }
    cluster_sync();
    const uint32_t at = smem_addr(sm.totals);
    for (uint32_t r = 0; r < rank; ++r) {
      gt += peer_load(at, r);
      eq += peer_load(at + 4, r);
    }
  }
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const uint32_t x = t < w1 ? key(t) : 0u;
    const bool is_gt = t < w1 && x > prefix, is_eq = t < w1 && x == prefix;
    const unsigned mg = __ballot_sync(kFull, is_gt), me = __ballot_sync(kFull, is_eq);
    const unsigned below = (1u << lane) - 1u;
    const uint32_t g = gt + __popc(mg & below), e = eq + __popc(me & below);
    if (is_gt || (is_eq && e < want)) {
      const uint32_t to = g + min(e, want);
      keep[to] = t;
      if (kept_mass) kept_mass[to] = mass[t];
    }
    gt += __popc(mg);
    eq += __popc(me);
  }
  if (CS > 1) cluster_sync();  // no CTA leaves while a peer may read its totals
}

// K and V of 64 kept tokens of one (row, KV head).
template <int DT>
__global__ void __launch_bounds__(kGatherThreads) evict_gather_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ long long src_at[kGatherTokens], dst_at[kGatherTokens];  // token rows in the pool, -1: no copy
  constexpr int kUnits = DT == PKV_KV_Q8_0 ? 8 : DT == PKV_KV_F32 ? 32 : 16;  // 16-byte pieces of a token
  const int tid = threadIdx.x;
  const int i = blockIdx.z, h = blockIdx.y, b0 = blockIdx.x * kGatherTokens;
  grid_dependency_wait();
  grid_launch_dependents();
  int L, B;
  row_budget(a, i, nullptr, L, B);
  if (b0 >= B) return;
  const int n = min(kGatherTokens, B - b0);
  if (tid < n) {
    const int b = b0 + tid;
    const int t = a.keep_idx[(static_cast<long long>(i) * a.pool.n_kv + h) * a.keep_stride + b];
    const int sp = __ldg(a.block_table + static_cast<long long>(i) * a.bt_stride + t / kPage);
    const int dp = __ldg(a.dst_block_table + static_cast<long long>(i) * a.dst_bt_stride + b / kPage);
    const bool ok = sp >= 0 && sp < a.pool.num_pages && dp >= 0 && dp < a.pool.num_pages;
    if (!ok) record_status(a.pool.status, PKV_DEV_BAD_PAGE);
    const long long s = (static_cast<long long>(sp) * a.pool.n_kv + h) * kPage + t % kPage;
    const long long d = (static_cast<long long>(dp) * a.pool.n_kv + h) * kPage + b % kPage;
    src_at[tid] = ok && s != d ? s : -1;
    dst_at[tid] = d;
  }
  __syncthreads();
  const int total = n * kUnits;  // a piece of K and the same piece of V
  for (int e0 = 0; e0 < total; e0 += 2 * kGatherThreads) {
    uint4 kv[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int e = e0 + x * kGatherThreads + tid;
      if (e < total && src_at[e / kUnits] >= 0) {
        const long long s = src_at[e / kUnits] * kUnits + e % kUnits;
        kv[x][0] = reinterpret_cast<const uint4*>(a.pool.k_data)[s];
        kv[x][1] = reinterpret_cast<const uint4*>(a.pool.v_data)[s];
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int e = e0 + x * kGatherThreads + tid;
      if (e < total && src_at[e / kUnits] >= 0) {
        const long long d = dst_at[e / kUnits] * kUnits + e % kUnits;
        reinterpret_cast<uint4*>(a.pool.k_data)[d] = kv[x][0];
        reinterpret_cast<uint4*>(a.pool.v_data)[d] = kv[x][1];
      }
    }
  }
  if constexpr (DT == PKV_KV_Q8_0) {
    if (tid < n && src_at[tid] >= 0) {  // 4 scales, 8 bytes, a token
      const uint2 k = reinterpret_cast<const uint2*>(a.pool.k_scales)[src_at[tid]];
      const uint2 v = reinterpret_cast<const uint2*>(a.pool.v_scales)[src_at[tid]];
      reinterpret_cast<uint2*>(a.pool.k_scales)[dst_at[tid]] = k;
      reinterpret_cast<uint2*>(a.pool.v_scales)[dst_at[tid]] = v;
    }
  }
}

template <int CS>
cudaError_t launch_select(const EvictArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_rows) * a.pool.n_kv * CS);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kCachedKeys * sizeof(uint32_t);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CS > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel<CS>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DT>
cudaError_t launch_gather(const EvictArgs& a, cudaStream_t st) {
  const long long most = a.keep_stride < static_cast<long long>(a.dst_bt_stride) * kPage
                             ? a.keep_stride
                             : static_cast<long long>(a.dst_bt_stride) * kPage;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((most + kGatherTokens - 1) / kGatherTokens), a.pool.n_kv, a.num_rows);
  cfg.blockDim = dim3(kGatherThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_gather_kernel<DT>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) {
  // The CTAs that share a (row, KV head), by the longest row the tables allow.
  const long long cap = a.mass_stride < static_cast<long long>(a.bt_stride) * kPage
                            ? a.mass_stride
                            : static_cast<long long>(a.bt_stride) * kPage;
  cudaError_t e = cap <= 4096 ? launch_select<1>(a, st) : launch_select<4>(a, st);
  if (e != cudaSuccess) return e;
  if (a.pool.dtype == PKV_KV_F16 || a.pool.dtype == PKV_KV_BF16) return launch_gather<PKV_KV_F16>(a, st);
  if (a.pool.dtype == PKV_KV_F32) return launch_gather<PKV_KV_F32>(a, st);
  return launch_gather<PKV_KV_Q8_0>(a, st);
}

}  // namespace pkv
