// tcgen05.cuh — inline-PTX wrappers of the fifth-generation tensor core
// instructions (products with accumulators in tensor memory), of the tensor
// copies that feed them, and of packed fp32 arithmetic, for the long-prompt
// kernels.
#pragma once

#include <cstdint>

#include "pkv_device.cuh"

namespace pkv {
namespace tc {

// Shared-memory matrix descriptor under the 128-byte swizzle: start address
// and two byte offsets in units of 16 bytes.  K-major operands (rows of 64
// elements, 8 rows per 1024-byte atom): sbo = bytes between 8-row groups, lbo
// unused.  MN-major operands: lbo = bytes between the 64-element parts of the
// M or N extent, sbo = bytes between groups of 8 rows along K.  The high word
// does not depend on the address, and an offset of x bytes adds x / 16 to the
// low word (addresses stay below 2^18), so products take the words apart.
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo) { return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
// Instruction descriptor of kind::f16, fp32 accumulation; A and B both f16
// (format 0) or both bf16 (format 1).
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool a_mn_major, bool b_mn_major, uint32_t format) {
  return (1u << 4) | (format << 7) | (format << 10) | (a_mn_major ? (1u << 15) : 0u) | (b_mn_major ? (1u << 16) : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Products and their commits are instructions of one thread, but they take
// their operands from the warp's uniform registers.  The whole warp runs the
// code around them, converged and on values that are the same in every lane
// (uniform() below), and `lead`, non-zero in one lane, guards the instruction
// itself: in a branch of one lane every operand of every product is first
// moved to a uniform register, which made a product cost 63 cycles to issue
// (one of 128 x 128 x 16 computes for 64).

// x, known to the compiler to be the same in every lane.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(kFull, x, 0); }
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(kFull, x, 0); }

// D (tensor memory) = A B (+ D): A and B in shared memory, their descriptors'
// low words and (constant) high words.
template <uint32_t A_HI, uint32_t B_HI>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, int accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %7};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accumulate), "r"(lead), "n"(A_HI), "n"(B_HI)
      : "memory");
}
// The same with A in tensor memory: lane = row of A, a 32-bit column two
// consecutive elements along K.
template <uint32_t B_HI>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, int accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accumulate), "r"(lead), "n"(B_HI)
      : "memory");
}
// Arrive on `bar` once every product the leading thread has issued is complete.
__device__ __forceinline__ void commit(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 consecutive 32-bit columns of the warp's 32 lanes (lane = thread).
__device__ __forceinline__ void ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int u = 0; u < 32; ++u) v[u] = __uint_as_float(r[u]);
}
__device__ __forceinline__ void st32(uint32_t taddr, const float* v) {
  uint32_t r[32];
#pragma unroll
  for (int u = 0; u < 32; ++u) r[u] = __float_as_uint(v[u]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void ld16w(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// 2^x by the hardware approximation (about 22 correct bits; 2^-inf = 0,
// results below 2^-126 flushed to 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest of three.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Registers a thread of the (whole, converged) warpgroup may use from here on.
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 values a b + c, one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t x, y, z, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t x, y, d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
  return r;
}

// Non-zero in one lane of the (converged) warp.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t pred;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(pred));
  return pred;
}

// Tensor copies global -> shared, completing on `bar`: the 5-D box at {0, 0,
// 0, 0, v} (a page tile), and the 4-D box at {0, y, z, 0} (query rows).
__device__ __forceinline__ void load_tile(uint32_t dst, const void* tmap, int v, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %2, %3}], "
      "[%4];" ::"r"(dst),
      "l"(tmap), "r"(0), "r"(v), "r"(bar)
      : "memory");
}
// The 3-D box at {0, 0, z} (a page of codes), and `bytes` contiguous bytes.
__device__ __forceinline__ void load_page(uint32_t dst, const void* tmap, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %3}], [%4];" ::"r"(
          dst),
      "l"(tmap), "r"(0), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void load_rows(uint32_t dst, const void* tmap, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %2}], "
      "[%5];" ::"r"(dst),
      "l"(tmap), "r"(0), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// The long end of a wait: false once *abort is set or after kWaitLimitNs.
__device__ __forceinline__ bool wait_on_here(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  const unsigned long long t0 = global_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(kFull, *abort != 0 || global_ns() - t0 > kWaitLimitNs)) break;
  }
  if ((threadIdx.x & 31) == 0 && !*abort) {
    *abort = 1;
    record_status(status, PKV_DEV_TIMEOUT);
  }
  return false;
}

// The same as a call, which keeps it out of the callers' loops.
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  return wait_on_here(bar, parity, abort, status);
}

// A wait by every lane of a warp, its outcome the same for all.  False once
// *abort is set or after kWaitLimitNs; it then has set *abort and recorded
// PKV_DEV_TIMEOUT.  A wait that has nothing to wait for is on many critical
// paths: a poll, a vote and a branch (some 35 cycles; a loop that lets lanes
// leave one by one took 157), and the clock is left to wait_on.  CALL: as a
// call, where the caller has registers for one.
template <bool CALL = true>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
#pragma unroll 1
  for (int i = 0; i < 512; ++i)
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
  if constexpr (CALL) return wait_on(bar, parity, abort, status);
  return wait_on_here(bar, parity, abort, status);
}

}  // namespace tc
}  // namespace pkv
