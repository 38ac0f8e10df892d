// rope_append.cu — kv_rope_append: a ragged chunk's queries and keys turned by
// their positions, its keys and values stored in the rows' pages.
//
// Pair u of a head is turned by a = positions[axis(u)][token] * inv_freq[u]:
//     x' = x cos a - y sin a,   y' = x sin a + y cos a.
// The angle is the same for every head of a token, so a CTA computes the
// cosines and sines of its tokens once, into shared memory, and then streams
// the heads.  The product of an int32 position and an fp32 frequency has up to
// 55 significant bits; it is formed and reduced to a fraction of a turn in 64
// bits (one product of 64 pairs a token: a few double operations against 48
// heads of memory traffic), which leaves an fp32 argument in [-1, 1] half turns
// for sincospif.
//
// A thread takes 16 elements of a head: two 8-element vectors A and B whose
// elements pair up with one another (halves: dims 8c and R/2 + 8c) or among
// themselves (interleaved: dims 16c and 16c + 8), so that 8 threads cover a
// head with 16-byte loads and stores and no exchange.  Each pair is read and
// written by one thread, which is why q_out may be q.
//
// Bound by memory: it reads the three projections and writes q and the cache
// once; everything else stays in registers and 2 KiB of shared memory.
#include <cstdint>

#include "chunk_device.cuh"

namespace pkv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxTok = 4;  // tokens of a CTA

struct TokenSlot {
  long long tile;  // first token row of the token's page for KV head 0, or -1: not stored
  int slot;        // its slot in the page
  int queries;     // the token belongs to a row: its queries are rotated
};

// The vectors of thread j (of the 8 of a head): dims 8 va .. and 8 vb ..
__device__ __forceinline__ void vectors_of(int j, int half, int interleaved, int& va, int& vb) {
  const int rot = half / 8;  // threads with pairs
  if (j < rot) {
    va = interleaved ? 2 * j : j;
    vb = interleaved ? 2 * j + 1 : rot + j;
  } else {
    va = rot + j;  // the 8 - rot vectors from 2 rot on, then as many more
    vb = 8 + j;
  }
}

template <int DT, int TOK>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 turn[TOK][64];
  __shared__ TokenSlot where[TOK];
  __shared__ float maxima[DT == PKV_KV_Q8_0 ? kRopeThreads / 8 : 1][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tok0 = blockIdx.x * TOK;
  const int ntok = min(TOK, a.rows.total_tokens - tok0);
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0) report_rows(a.rows, a.pool.status);
  // the page slot of each token
  if (warp < ntok) {
    const int tok = tok0 + warp;
    const int i = row_of_token(a.rows, tok);
    TokenSlot w{-1, 0, 0};
    if (i >= 0) {
      const RowInfo r = row_info(a.rows, i, nullptr);
      w.queries = r.n > 0;
      if (r.L >= 0) {
        const int P = r.L - r.n + (tok - r.start);
        const int pg = __ldg(a.rows.block_table + static_cast<long long>(i) * a.rows.bt_stride + P / kPage);
        if (pg >= 0 && pg < a.pool.num_pages) {
          w.tile = static_cast<long long>(pg) * a.pool.n_kv * kPage;
          w.slot = P % kPage;
        } else if (lane == 0) {
          record_status(a.pool.status, PKV_DEV_BAD_PAGE);
        }
      }
    }
    if (lane == 0) where[warp] = w;
  }
  // the turns of each (token, pair)
  for (int e = tid; e < ntok * a.half; e += kRopeThreads) {
    const int t = e / a.half, u = e - t * a.half;
    int axis = 0;
#pragma unroll
    for (int x = 0; x + 1 < PKV_MAX_ROPE_AXES; ++x) axis += u >= a.axis_end[x] ? 1 : 0;
    const int pos = __ldg(a.positions + static_cast<long long>(axis) * a.rows.total_tokens + tok0 + t);
    const double half_turns = static_cast<double>(pos) * static_cast<double>(__ldg(a.inv_freq + u)) *
                              0.31830988618379067154;  // 1 / pi
    const double r = half_turns - 2.0 * rint(0.5 * half_turns);  // in [-1, 1]
    float s, c;
    sincospif(static_cast<float>(r), &s, &c);
    turn[t][u] = make_float2(c, s);
  }
  __syncthreads();
  const int heads = a.n_q + 2 * a.pool.n_kv;
  const int items = ntok * heads * 8;  // 8 threads a head
  const int rounds = (items + kRopeThreads - 1) / kRopeThreads;
  for (int rd = 0; rd < rounds; ++rd) {
    const int it = rd * kRopeThreads + tid;
    const bool on = it < items;
    const int j = it & 7, row = it >> 3;
    const int t = on ? row / heads : 0, hh = on ? row - t * heads : 0;
    const TokenSlot w = where[t];
    const bool is_q = hh < a.n_q, is_k = !is_q && hh < a.n_q + a.pool.n_kv;
    const bool live = on && (is_q ? w.queries != 0 : w.tile >= 0);
    int va, vb;
    vectors_of(j, a.half, a.interleaved, va, vb);
    float A[8], B[8];
    if (live) {
      const int h = is_q ? hh : (is_k ? hh - a.n_q : hh - a.n_q - a.pool.n_kv);
      const uint8_t* src = is_q ? a.q : (is_k ? a.k : a.v);
      const long long stride = is_q ? a.q_stride : (is_k ? a.k_stride : a.v_stride);
      const long long at = (tok0 + t) * stride + static_cast<long long>(h) * kD;
      load8(src, at + 8 * va, a.in_dtype, A);
      load8(src, at + 8 * vb, a.in_dtype, B);
      if ((is_q || is_k) && j < a.half / 8) {
        const float2* cs = &turn[t][8 * j];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c0 = cs[e], c1 = cs[4 + e];
            const float x = A[2 * e], y = A[2 * e + 1], z = B[2 * e], q = B[2 * e + 1];
            A[2 * e] = x * c0.x - y * c0.y;
            A[2 * e + 1] = x * c0.y + y * c0.x;
            B[2 * e] = z * c1.x - q * c1.y;
            B[2 * e + 1] = z * c1.y + q * c1.x;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 c = cs[e];
            const float x = A[e], y = B[e];
            A[e] = x * c.x - y * c.y;
            B[e] = x * c.y + y * c.x;
          }
        }
      }
      if (is_q) {
        const long long to = (static_cast<long long>(tok0 + t) * a.n_q + h) * kD;
        store8(a.q_out, to + 8 * va, a.q_dtype, A);
        store8(a.q_out, to + 8 * vb, a.q_dtype, B);
      } else if constexpr (DT != PKV_KV_Q8_0) {
        uint8_t* data = is_k ? a.pool.k_data : a.pool.v_data;
        const long long to = (w.tile + static_cast<long long>(h) * kPage + w.slot) * kD;
        store8(data, to + 8 * va, DT, A);
        store8(data, to + 8 * vb, DT, B);
      }
    }
    if constexpr (DT == PKV_KV_Q8_0) {
      // The four vectors of a 32-wide block may sit in different threads of
      // the head's 8: their maxima meet in shared memory.
      const bool enc = live && !is_q;
      float ma = 0.f, mb = 0.f;
      if (enc) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ma = fmaxf(ma, fabsf(A[e]));
          mb = fmaxf(mb, fabsf(B[e]));
        }
      }
      float* mx = maxima[tid >> 3];
      __syncwarp();
      mx[va] = ma;
      mx[vb] = mb;
      __syncwarp();
      if (enc) {
        const int h = is_k ? hh - a.n_q : hh - a.n_q - a.pool.n_kv;
        uint8_t* data = is_k ? a.pool.k_data : a.pool.v_data;
        uint8_t* sc = is_k ? a.pool.k_scales : a.pool.v_scales;
        const long long to = w.tile + static_cast<long long>(h) * kPage + w.slot;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int vec = half ? vb : va, blk = vec >> 2;
          const float amax = fmaxf(fmaxf(mx[4 * blk], mx[4 * blk + 1]), fmaxf(mx[4 * blk + 2], mx[4 * blk + 3]));
          const float dq = amax / 127.0f;  // IEEE division, as kv_append
          uint32_t code[2] = {0u, 0u};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = half ? B[e] : A[e];
            float c = 0.0f;
            if (dq != 0.0f) c = fminf(fmaxf(roundf(x / dq), -127.0f), 127.0f);
            code[e >> 2] |= static_cast<uint32_t>(static_cast<int>(c) + 128) << (8 * (e & 3));
          }
          *reinterpret_cast<uint2*>(data + to * kD + 8 * vec) = make_uint2(code[0], code[1]);
          if ((vec & 3) == 0) reinterpret_cast<__half*>(sc)[to * (kD / kQBlock) + blk] = __float2half_rn(dq);
        }
      }
    }
  }
}

template <int DT>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int n = a.rows.total_tokens;
  cudaError_t e;
  if (n >= 4096) {
    cfg.gridDim = dim3((n + kMaxTok - 1) / kMaxTok);
    e = cudaLaunchKernelEx(&cfg, rope_append_kernel<DT, kMaxTok>, a);
  } else {
    cfg.gridDim = dim3(n);
    e = cudaLaunchKernelEx(&cfg, rope_append_kernel<DT, 1>, a);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t st) {
  if (a.pool.dtype == PKV_KV_F16) return launch_rope_t<PKV_KV_F16>(a, st);
  if (a.pool.dtype == PKV_KV_BF16) return launch_rope_t<PKV_KV_BF16>(a, st);
  if (a.pool.dtype == PKV_KV_F32) return launch_rope_t<PKV_KV_F32>(a, st);
  return launch_rope_t<PKV_KV_Q8_0>(a, st);
}

}  // namespace pkv
