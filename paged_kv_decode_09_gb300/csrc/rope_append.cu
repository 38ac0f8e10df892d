// rope_append.cu — kv_rope_append: a ragged chunk's queries and keys turned by
// their positions, its keys and values stored in the rows' pages.
//
// Pair u of a head is turned by a = positions[axis(u)][token] * inv_freq[u]:
//     x' = x cos a - y sin a,   y' = x sin a + y cos a.
// The angle is the same for every head of a token, so a CTA computes the
// cosines and sines of its tokens once, into shared memory, and then streams
// the heads.  An angle is reduced without rounding: a frequency is kept as a
// 64-bit fraction of a turn (one product in 64 bits per pair and CTA), and
// position times fraction modulo 2^64 is the fraction of a turn that is left,
// whose upper half goes to sincospif.  At positions near 2^31 the fraction's
// own rounding leaves 2.4e-7 radians.
//
// A thread takes 16 elements of a head: two 8-element vectors A and B whose
// elements pair up with one another (halves: dims 8c and R/2 + 8c) or among
// themselves (interleaved: dims 16c and 16c + 8), so that 8 threads cover a
// head with 16-byte loads and stores and no exchange.  Each pair is read and
// written by one thread, which is why q_out may be q.
//
// Bound by memory: it reads the three projections and writes q and the cache
// once; everything else stays in registers and 2 KiB of shared memory.  10560
// tokens of 32 + 8 + 8 heads in bf16, 260 MB: 43.6 us, 5950 GB/s.  What that
// took: a CTA of four tokens (one: their angles, the row search and two barriers
// come too often; eight: 50 us), five CTAs an SM by keeping only the next
// round's vectors in flight (three rounds in flight and three CTAs: 60 us;
// seven CTAs spill: 69 us), and turns laid out for the threads that read them
// together (in order, a quarter of the shared memory's rate).
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

// Where pair u's turn is kept: the pairs of one step of the 8 threads of a head
// side by side (in order, the threads would meet in two of the banks).
__device__ __forceinline__ int turn_at(int u) { return (u & 7) * 8 + (u >> 3); }

// One 8-element vector of a token array, as loaded.
template <int IN>
struct Raw {
  uint4 w[IN == PKV_KV_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t* base, long long elem) {
    const uint4* p = reinterpret_cast<const uint4*>(base + elem * (IN == PKV_KV_F32 ? 4 : 2));
    w[0] = p[0];
    if constexpr (IN == PKV_KV_F32) w[1] = p[1];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if constexpr (IN == PKV_KV_F32) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[4 * e] = __uint_as_float(w[e].x);
        x[4 * e + 1] = __uint_as_float(w[e].y);
        x[4 * e + 2] = __uint_as_float(w[e].z);
        x[4 * e + 3] = __uint_as_float(w[e].w);
      }
    } else {
      const uint32_t v[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (IN == PKV_KV_BF16) {
          x[2 * e] = __uint_as_float(v[e] << 16);
          x[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
          x[2 * e] = f.x;
          x[2 * e + 1] = f.y;
        }
      }
    }
  }
};

template <int DT, int IN, int TOK>
__global__ void __launch_bounds__(kRopeThreads, IN == PKV_KV_F32 || DT == PKV_KV_Q8_0 ? 4 : 5) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ unsigned long long fraction[64];
  __shared__ float2 turn[TOK][64];
  __shared__ TokenSlot where[TOK];
  __shared__ float maxima[DT == PKV_KV_Q8_0 ? kRopeThreads / 8 : 1][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tok0 = blockIdx.x * TOK;
  const int ntok = min(TOK, a.rows.total_tokens - tok0);
  const int heads = a.n_q + 2 * a.pool.n_kv;
  const int items = ntok * heads * 8;  // 8 threads a head
  const int j = tid & 7;
  int va, vb;
  vectors_of(j, a.half, a.interleaved, va, vb);
  // item -> (token, head): q heads, then k, then v
  auto place = [&](int rd, int& t, int& hh) {
    const int row = rd * (kRopeThreads / 8) + (tid >> 3);
    t = 0;
#pragma unroll
    for (int u = 1; u < TOK; ++u) t += row >= u * heads ? 1 : 0;
    hh = row - t * heads;
    return rd * kRopeThreads + tid < items;
  };
  Raw<IN> A, B;  // of the next round
  auto fetch = [&](int rd) {
    int t, hh;
    if (!place(rd, t, hh)) return;
    const bool is_q = hh < a.n_q, is_k = !is_q && hh < a.n_q + a.pool.n_kv;
    const int h = is_q ? hh : (is_k ? hh - a.n_q : hh - a.n_q - a.pool.n_kv);
    const uint8_t* src = is_q ? a.q : (is_k ? a.k : a.v);
    const long long stride = is_q ? a.q_stride : (is_k ? a.k_stride : a.v_stride);
    const long long at = (tok0 + t) * stride + static_cast<long long>(h) * kD;
    A.load(src, at + 8 * va);
    B.load(src, at + 8 * vb);
  };
  grid_dependency_wait();
  grid_launch_dependents();
  fetch(0);
  if (blockIdx.x == 0) report_rows(a.rows, a.pool.status);
  if (tid >= kRopeThreads - 64 && tid - (kRopeThreads - 64) < a.half) {
    const int u = tid - (kRopeThreads - 64);
    const double turns = static_cast<double>(__ldg(a.inv_freq + u)) * 0.15915494309189533577;  // 1 / 2 pi
    fraction[u] = __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
  }
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
  __syncthreads();
  // the turns of each (token, pair)
  for (int e = tid; e < ntok * 64; e += kRopeThreads) {
    const int t = e >> 6, u = e & 63;
    if (u < a.half) {
      int axis = 0;
#pragma unroll
      for (int x = 0; x + 1 < PKV_MAX_ROPE_AXES; ++x) axis += u >= a.axis_end[x] ? 1 : 0;
      const long long pos = __ldg(a.positions + static_cast<long long>(axis) * a.rows.total_tokens + tok0 + t);
      const unsigned long long left = static_cast<unsigned long long>(pos) * fraction[u];
      // the fraction as a signed one, in half turns: [-1, 1]
      const float half_turns = static_cast<float>(static_cast<int>((left + (1ull << 31)) >> 32)) * 4.656612873077393e-10f;
      float s, c;
      sincospif(half_turns, &s, &c);
      turn[t][turn_at(u)] = make_float2(c, s);
    }
  }
  __syncthreads();
  const int rounds = (items + kRopeThreads - 1) / kRopeThreads;
  for (int rd = 0; rd < rounds; ++rd) {
    int t, hh;
    const bool on = place(rd, t, hh);
    if (!on) t = 0;
    const TokenSlot w = where[t];
    const bool is_q = hh < a.n_q, is_k = !is_q && hh < a.n_q + a.pool.n_kv;
    const bool live = on && (is_q ? w.queries != 0 : w.tile >= 0);
    const int h = is_q ? hh : (is_k ? hh - a.n_q : hh - a.n_q - a.pool.n_kv);
    float x[8], y[8];
    if (live) {
      A.values(x);
      B.values(y);
    }
    fetch(rd + 1);
    if (live) {
      if ((is_q || is_k) && j < a.half / 8) {
        const float2* cs = &turn[t][turn_at(8 * j)];
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c0 = cs[8 * e], c1 = cs[8 * (4 + e)];
            const float p = x[2 * e], q = x[2 * e + 1], u = y[2 * e], v = y[2 * e + 1];
            x[2 * e] = p * c0.x - q * c0.y;
            x[2 * e + 1] = p * c0.y + q * c0.x;
            y[2 * e] = u * c1.x - v * c1.y;
            y[2 * e + 1] = u * c1.y + v * c1.x;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 c = cs[8 * e];
            const float p = x[e], q = y[e];
            x[e] = p * c.x - q * c.y;
            y[e] = p * c.y + q * c.x;
          }
        }
      }
      if (is_q) {
        const long long to = (static_cast<long long>(tok0 + t) * a.n_q + h) * kD;
        store8(a.q_out, to + 8 * va, a.q_dtype, x);
        store8(a.q_out, to + 8 * vb, a.q_dtype, y);
      } else if constexpr (DT != PKV_KV_Q8_0) {
        uint8_t* data = is_k ? a.pool.k_data : a.pool.v_data;
        const long long to = (w.tile + static_cast<long long>(h) * kPage + w.slot) * kD;
        store8(data, to + 8 * va, DT, x);
        store8(data, to + 8 * vb, DT, y);
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
          ma = fmaxf(ma, fabsf(x[e]));
          mb = fmaxf(mb, fabsf(y[e]));
        }
      }
      float* mx = maxima[tid >> 3];
      __syncwarp();
      mx[va] = ma;
      mx[vb] = mb;
      __syncwarp();
      if (enc) {
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
            const float v = half ? y[e] : x[e];
            float c = 0.0f;
            if (dq != 0.0f) c = fminf(fmaxf(roundf(v / dq), -127.0f), 127.0f);
            code[e >> 2] |= static_cast<uint32_t>(static_cast<int>(c) + 128) << (8 * (e & 3));
          }
          *reinterpret_cast<uint2*>(data + to * kD + 8 * vec) = make_uint2(code[0], code[1]);
          if ((vec & 3) == 0) reinterpret_cast<__half*>(sc)[to * (kD / kQBlock) + blk] = __float2half_rn(dq);
        }
      }
    }
  }
}

template <int DT, int IN>
cudaError_t launch_rope_in(const RopeArgs& a, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Four tokens a CTA share their angles' setup; one a CTA fills the SMs with
  // fewer tokens.  One and four, of 32 + 8 + 8 heads: f16 and bf16 3.3 and 4.9 us
  // for 256 tokens, 6.1 and 6.0 for 1024, 9.3 and 10.1 for 2048, 19.4 and 16.8 for
  // 4095, 49.4 and 43.1 for 10560; q8_0 4.5 and 7.2, 8.8 and 8.8, 16.1 and 13.1,
  // 28.6 and 22.1, 72.3 and 53.6; f32 4.2 and 5.4, 10.1 and 9.1, 16.9 and 17.1,
  // 34.3 and 34.6, 81.5 and 80.1.
  const int n = a.rows.total_tokens;
  cudaError_t e;
  if (n >= 4096) {
    cfg.gridDim = dim3((n + kMaxTok - 1) / kMaxTok);
    e = cudaLaunchKernelEx(&cfg, rope_append_kernel<DT, IN, kMaxTok>, a);
  } else {
    cfg.gridDim = dim3(n);
    e = cudaLaunchKernelEx(&cfg, rope_append_kernel<DT, IN, 1>, a);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int DT>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t st) {
  if (a.in_dtype == PKV_KV_F16) return launch_rope_in<DT, PKV_KV_F16>(a, st);
  if (a.in_dtype == PKV_KV_BF16) return launch_rope_in<DT, PKV_KV_BF16>(a, st);
  return launch_rope_in<DT, PKV_KV_F32>(a, st);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t st) {
  if (a.pool.dtype == PKV_KV_F16) return launch_rope_t<PKV_KV_F16>(a, st);
  if (a.pool.dtype == PKV_KV_BF16) return launch_rope_t<PKV_KV_BF16>(a, st);
  if (a.pool.dtype == PKV_KV_F32) return launch_rope_t<PKV_KV_F32>(a, st);
  return launch_rope_t<PKV_KV_Q8_0>(a, st);
}

}  // namespace pkv
