// mma.cuh — warp matrix instructions: m16n8k16 products of binary16 with binary32 sums, and the
// copies and transposes that feed them. With g = lane / 4 and c = lane % 4 a thread holds
//   A (16 x 16): a[0] row g, columns 2c, 2c+1; a[1] row g+8; a[2] row g, columns 2c+8, 2c+9; a[3] row g+8
//   B (16 x 8):  b[0] rows 2c, 2c+1 of column g; b[1] rows 2c+8, 2c+9
//   C (16 x 8):  c[0], c[1] row g, columns 2c, 2c+1; c[2], c[3] row g+8
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace fmoe {

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum: d = a b.
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// d += a b over 8 of the sum, tf32 operands (the upper 19 bits of binary32): a[0] row g, column c; a[1] row g+8;
// a[2] row g, column c+4; a[3] row g+8; b[0] row c of column g, b[1] row c+4; d as above.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// A binary32 value as two tf32 parts, each rounded to nearest: together within 2^-23 of it. (The
// product reads no more than the upper 19 bits. Additions, as the conversion instruction is slow: 16384 tokens,
// 64 heads 1650 us so, 1750 us with it.)
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;
}

// Transposes an 8 x 8 matrix of 16-bit values: in, a thread holds row g, columns 2c, 2c+1.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Asynchronous 16-byte copies from global to shared memory.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
// What binary16 leaves of two values after `hi` = pack_half2 of them, as binary16 again: together
// they hold 22 bits of each value (while it is above 2^-14 in magnitude; 2^-25 absolute below).
__device__ __forceinline__ uint32_t rest_half2(float lo, float hi, uint32_t packed) {
  const float2 f = unpack_half2(packed);
  return pack_half2(lo - f.x, hi - f.y);
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// The exponent e of the largest power of two <= |x| (x finite and normal; else the range's end).
__device__ __forceinline__ int exponent(float x) { return (int)((__float_as_uint(x) >> 23) & 255u) - 127; }

}  // namespace fmoe
