// evict.cu — kv_evict: shorten rows to their budget per KV head, keeping the
// tokens that received the most attention.
//
// Selecting.  A token's key is its weight as an unsigned integer of the same
// order (NaN lowest; the protected first and recent tokens highest), so the B
// kept tokens of a (row, KV head) are the B largest keys with ties to the
// lowest index.  One CTA holds the keys in shared memory and finds the B-th
// largest key T digit by digit from the top (11, 11 and 10 bits): a histogram of
// the digit over the keys that match the digits found so far, in four copies to
// spread its atomics, and the digit at which the count from above reaches B.
// Then token t is kept if its key exceeds T, or equals T with fewer than
// (B - #greater) equals before it; its place among the kept is
//     #greater before t + min(#equal before t, B - #greater),
// prefix sums of votes over groups of 32 tokens in order.  Rows longer than the
// shared memory holds re-read their weights (from L2) in every pass.  Each loop
// runs once over the keys, from a cold instruction cache: they are loops of a
// few instructions (with the keys in registers and the loops unrolled, the code
// took 32 us to fetch, whatever the rows' lengths).  18 us for 32768 tokens a
// row, 7 for 2048; a cluster of two CTAs a row and head gains one of them, one
// of four loses nine to its meetings.
//
// Gathering.  The kept tokens go to fresh pages, so every copy is independent:
// a CTA takes 64 kept tokens of a head and moves their K and V in 16-byte
// pieces.  Bound by memory: the bytes are the kept K and V, read and written
// once; the weights of the whole row are a few percent of them.  Eight rows to
// 4096 tokens of 8 heads each, 273 MB: 40 us, 6.8 TB/s; with the selection 58.
#include <atomic>
#include <cstdint>

#include "chunk_device.cuh"

namespace pkv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kCopies = 4;
constexpr int kKeys = 47 * 1024;  // 188 KiB beside the histograms' 32
constexpr int kGatherTokens = 64;
constexpr int kGatherThreads = 256;

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

// CACHED: the keys stay in shared memory (kKeys at most).
template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) uint32_t hist[kCopies][kBins];
  __shared__ uint32_t bin_sums[kSelWarps];
  __shared__ uint32_t pick[2];  // the digit, and the count above it
  __shared__ uint2 votes[kSelWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int seg = blockIdx.x;  // (row, KV head)
  const int i = seg / a.pool.n_kv, h = seg - i * a.pool.n_kv;
  grid_dependency_wait();
  grid_launch_dependents();
  int L, B;
  row_budget(a, i, (h == 0 && tid == 0) ? a.pool.status : nullptr, L, B);
  const float* mass = a.mass + static_cast<long long>(seg) * a.mass_stride;
  int32_t* keep = a.keep_idx + static_cast<long long>(seg) * a.keep_stride;
  if (h == 0 && tid == 0) a.new_lens[i] = B;
  if (B == L || B == 0) {  // everything kept, or nothing
    for (int t = tid; t < B; t += kSelThreads) keep[t] = t;
    return;
  }
  const int recent = min(a.recent, B), first = min(a.first, B - recent);
  auto fetch = [&](int t) {
    const float x = __ldg(mass + t);
    return t < first || t >= L - recent ? 0xFFFFFFFFu : key_of(x);
  };
  auto key = [&](int t) { return CACHED ? keys[t] : fetch(t); };
  uint32_t* mine = hist[warp % kCopies];
  auto clear = [&] {
#pragma unroll 1
    for (int e = tid; e < kCopies * kBins / 4; e += kSelThreads)
      reinterpret_cast<uint4*>(hist)[e] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  };
  clear();
  if constexpr (CACHED) {  // the keys, and the first digit's histogram with them
#pragma unroll 1
    for (int t0 = 0; t0 < L; t0 += 8 * kSelThreads) {  // eight loads in flight
      float x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = __ldg(mass + min(t0 + u * kSelThreads + tid, L - 1));
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int t = t0 + u * kSelThreads + tid;
        if (t < L) {
          const uint32_t y = t < first || t >= L - recent ? 0xFFFFFFFFu : key_of(x[u]);
          keys[t] = y;
          atomicAdd(&mine[y >> 21], 1u);
        }
      }
    }
  }
  uint32_t T = 0, mask = 0;  // the digits of T found so far
  int want = B;              // how many of the keys that match them are kept
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t digit = pass == 2 ? 1023u : 2047u;
    if (pass > 0) clear();
    if (!CACHED || pass > 0) {
#pragma unroll 4
      for (int t = tid; t < L; t += kSelThreads) {
        const uint32_t x = key(t);
        if ((x & mask) == T) atomicAdd(&mine[(x >> shift) & digit], 1u);
      }
    }
    __syncthreads();
    // a thread's bins, from the top: 2 consecutive ones
    constexpr int kPer = kBins / kSelThreads;
    static_assert(kPer == 2, "");
    const int b0 = kBins - kPer * (tid + 1);
    uint32_t c[kPer] = {0u, 0u};
#pragma unroll
    for (int r = 0; r < kCopies; ++r) {
      const uint2 v = *reinterpret_cast<const uint2*>(&hist[r][b0]);
      c[1] += v.x;
      c[0] += v.y;
    }
    const uint32_t sum = c[0] + c[1];
    uint32_t run = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(kFull, run, o);
      if (lane >= o) run += u;
    }
    if (lane == 31) bin_sums[warp] = run;
    __syncthreads();
    uint32_t above = run - sum + __reduce_add_sync(kFull, lane < warp ? bin_sums[lane & (kSelWarps - 1)] : 0u);
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      if (above < static_cast<uint32_t>(want) && static_cast<uint32_t>(want) <= above + c[u]) {
        pick[0] = static_cast<uint32_t>(b0 + kPer - 1 - u);
        pick[1] = above;
      }
      above += c[u];
    }
    __syncthreads();
    T |= pick[0] << shift;
    mask |= digit << shift;
    want -= static_cast<int>(pick[1]);
  }
  // each warp takes a contiguous part of the tokens, in groups of 32
  const int groups = (L + 31) / 32, per = (groups + kSelWarps - 1) / kSelWarps;
  const int w0 = min(L, warp * per * 32), w1 = min(L, w0 + per * 32);
  uint32_t gt = 0, eq = 0;
#pragma unroll 4
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const int t = t0 + lane;
    const uint32_t x = t < w1 ? key(t) : 0u;
    gt += __popc(__ballot_sync(kFull, t < w1 && x > T));
    eq += __popc(__ballot_sync(kFull, t < w1 && x == T));
  }
  if (lane == 0) votes[warp] = make_uint2(gt, eq);
  __syncthreads();
  const uint2 v = lane < warp ? votes[lane & (kSelWarps - 1)] : make_uint2(0u, 0u);
  gt = __reduce_add_sync(kFull, v.x);
  eq = __reduce_add_sync(kFull, v.y);
  const unsigned below = (1u << lane) - 1u;
#pragma unroll 4
  for (int t0 = w0; t0 < w1; t0 += 32) {
    const int t = t0 + lane;
    const uint32_t x = t < w1 ? key(t) : 0u;
    const bool is_gt = t < w1 && x > T, is_eq = t < w1 && x == T;
    const unsigned mg = __ballot_sync(kFull, is_gt), me = __ballot_sync(kFull, is_eq);
    const uint32_t g = gt + __popc(mg & below), e = eq + __popc(me & below);
    if (is_gt || (is_eq && e < static_cast<uint32_t>(want))) keep[g + min(e, static_cast<uint32_t>(want))] = t;
    gt += __popc(mg);
    eq += __popc(me);
  }
}

// K, V and the weights of 64 kept tokens of one (row, KV head).
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
    if (a.dst_mass) {
      const long long seg = static_cast<long long>(i) * a.pool.n_kv + h;
      a.dst_mass[seg * a.keep_stride + b] = __ldg(a.mass + seg * a.mass_stride + t);
    }
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

template <bool CACHED>
cudaError_t launch_select(const EvictArgs& a, size_t smem, cudaStream_t st) {
  if (smem > 8192) {  // above the default limit with the static arrays
    static std::atomic<int> granted[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !granted[dev].load(std::memory_order_relaxed)) {
      e = cudaFuncSetAttribute(evict_select_kernel<CACHED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kKeys * static_cast<int>(sizeof(uint32_t)));
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) granted[dev].store(1, std::memory_order_relaxed);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_rows) * a.pool.n_kv);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel<CACHED>, a);
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
  // Shared memory for the keys of the longest row the tables allow.
  const long long cap = a.mass_stride < static_cast<long long>(a.bt_stride) * kPage
                            ? a.mass_stride
                            : static_cast<long long>(a.bt_stride) * kPage;
  cudaError_t e = cap <= kKeys ? launch_select<true>(a, static_cast<size_t>(cap) * sizeof(uint32_t), st)
                               : launch_select<false>(a, 0, st);
  if (e != cudaSuccess) return e;
  if (a.pool.dtype == PKV_KV_F16 || a.pool.dtype == PKV_KV_BF16) return launch_gather<PKV_KV_F16>(a, st);
  if (a.pool.dtype == PKV_KV_F32) return launch_gather<PKV_KV_F32>(a, st);
  return launch_gather<PKV_KV_Q8_0>(a, st);
}

}  // namespace pkv
