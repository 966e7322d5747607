// cached_tc.cuh -- what the cache's tcgen05 kernels share: operand descriptors,
// 8-bit products, bulk copies, a query row as two 8-bit parts.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache.cuh"
#include "ptx.cuh"

namespace bdlm {

// Shared-memory descriptors (see sdesc_sw128) as their two words: the upper
// one is a constant of the layout, the lower one the start address (and, for an
// MN-major operand, the panel stride), so that the issuing thread holds one
// register per operand.  128-byte (SW = 2) or 64-byte (SW = 4) swizzle.
__host__ __device__ constexpr uint32_t desc_hi(int sw, int sbo) {
  return (uint32_t)(sbo >> 4) | (1u << 14) | ((uint32_t)sw << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, int lbo) {
  return ((addr & 0x3FFFFu) >> 4) | ((uint32_t)(lbo >> 4) << 16);
}

// D[tmem] (+)= A[smem] B[smem]: 8-bit types, K = 32 (F8), or bf16, K = 16.
template <bool F8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                       uint32_t idesc, uint32_t acc) {
  if (F8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\t"
        "mov.b64 b, {%3, %4};\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
        : "memory");
}
// D[tmem] (+)= A[tmem] B[smem], 16-bit types, K = 16.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t bhi, uint32_t idesc,
                                       uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(blo), "r"(bhi), "r"(idesc), "r"(acc)
      : "memory");
}
// Waits for three barriers, asked side by side: shared memory takes some 200 cycles to
// answer beside the MMAs, whether a barrier is complete or not.  (The issuing thread's
// three waits for a cached tile one after the other / side by side, in a graph, warm: blocks of
// 32 / 128 / 512 85.2 / 224 / 492 and 83.1 / 221 / 487 us; trees of 60 rows over 8 sequences of
// 16384 290 / 282.)
__device__ __forceinline__ bool mbar_wait3(uint32_t b0, uint32_t p0, uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2,
                                           const Watchdog& wd, uint32_t s0, uint32_t s1, uint32_t s2) {
  const uint32_t x = mbar_try_wait(b0, p0), y = mbar_try_wait(b1, p1), z = mbar_try_wait(b2, p2);
  return (x & y & z) || (mbar_wait(b0, p0, wd, s0) && mbar_wait(b1, p1, wd, s1) && mbar_wait(b2, p2, wd, s2));
}

// kind::f8f6f4, fp32 accumulator, both operands K-major, each of its own format:
// e4m3 (0) or e5m2 (1).
constexpr int kE4m3 = 0, kE5m2 = 1;
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, int a, int b) {
  return (1u << 4) | ((uint32_t)a << 7) | ((uint32_t)b << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Contiguous copy into shared memory (16-byte aligned, a multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
// 16 bytes into shared memory, `bytes` (0 or 16) of them read and the rest zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Sixteen values of a bf16 query row, times f, as the 16-byte chunks of its two
// parts: hi the nearest e4m3 values, lo what that left, in e5m2.  A bf16 value has
// 8 significant bits, hi rounds to 4: the rest is at most 8 units of the 8th bit,
// which e5m2's 3 bits hold.  So the parts are exact for values from 2^-6 on, e4m3's
// smallest normal one; below, hi's step is 2^-9, the rest at most 2^-10, and its
// 3 bits leave 2^-14 at most.  Of a row's largest value, 2^7 to 2^8, that is: exact
// down to 2^-13, off by 2^-21 below.  (lo in e4m3, whose smallest step is 2^-9:
// exact down to 2^-9, off by 2^-17.  In fp16 the scaled values are exact down to
// 2^-17 and off by 2^-25 below.)
__device__ __forceinline__ void split_f8(const uint32_t* w, float f, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const __half2 v =
        __floats2half2_rn(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xffff0000u) * f);
    const uint32_t h = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
    const uint32_t back = e4m3x2_to_half2(h);
    const __half2 d = __hsub2(v, *reinterpret_cast<const __half2*>(&back));
    const uint32_t l = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(d), __NV_SATFINITE, __NV_E5M2);
    hi[k >> 1] = k & 1 ? hi[k >> 1] | h << 16 : h;
    lo[k >> 1] = k & 1 ? lo[k >> 1] | l << 16 : l;
  }
}

// The power of two that puts a row of largest magnitude `amax` (bf16 bits) into
// [128, 256), and its inverse; NaN for a row that is not finite (e4m3 has no
// infinity: such a row reads NaN).
__device__ __forceinline__ float row_factor(uint32_t amax, float& inv) {
  int e = 7 + 127 - (int)(amax >> 7);
  if (amax >= 0x7f80u || amax == 0) e = 0;
  e = min(e, 126);
  inv = __uint_as_float((uint32_t)(127 - e) << 23);
  return amax >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

// Byte offset of 16-byte chunk i of row r in a K-major 8-bit tile of HD columns
// (128-byte swizzle; 64-byte for HD = 64).
template <int HD>
__device__ __forceinline__ uint32_t e4m3_chunk(int r, int i) {
  return HD == 128 ? (uint32_t)(r * 128 + ((i ^ (r & 7)) << 4)) : (uint32_t)(r * 64 + ((i ^ ((r >> 1) & 3)) << 4));
}

}  // namespace bdlm
