// cp_fp4.cuh -- the 4-bit format and the register-level helpers that the
// 4-bit operators share.
//
// A value is s * c with c one of the sixteen E2M1 numbers (+-0, 0.5, 1, 1.5,
// 2, 3, 4, 6) and s the bfloat16 scale of its group.  s = bf16(max |x| * r), r
// the float32 number nearest to 1/6, the product rounded to float32 and then to
// bfloat16, both to nearest even (the same as bf16(max |x| / 6) for bfloat16 and
// fp16 inputs and for all but 21 of the 2^23 significands of float32, where it is
// the next bfloat16 number); c is the E2M1 number nearest to x / s, ties to the even code.  The float32 quotient decides like the exact one: a tie
// point is s times a number of at most three bits, hence a float32 number,
// and for any other x the quotient differs from the tie point by more than
// half an ulp.  A group that holds an infinity or a NaN gets a NaN scale (all
// its values read back as NaN); a group whose scale rounds to zero reads back
// as zeros.
//
// E2M1 is what the converter unit of sm_103a turns into two fp16 numbers with
// one instruction (about 42 lanes per clock and SM measured in a mix with as
// many integer instructions; 4-bit integers by bit tricks take 9
// instructions for 8 values), and every E2M1 number is exact in fp16, so the
// products run on fp16 mma.sync with float32 accumulators without rounding
// the weights or the cache.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "cp_common.cuh"

namespace cpk {

// Element types of the 4-bit operators (values of the C ABI).
enum : int { kF32 = 0, kBF16 = 1, kF16 = 2 };
inline __host__ __device__ int elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }

// Two codes of a byte (low nibble first) -> fp16x2, for the four bytes of w.
__device__ __forceinline__ void e2m1_to_half2x4(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Nearest E2M1 codes of lo (low nibble) and hi (high nibble), ties to even,
// saturating; neither may be a NaN.
__device__ __forceinline__ uint32_t float2_to_e2m1(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t, z;\n .reg .b16 h;\n mov.b16 h, 0;\n mov.b16 {z, t}, h;\n"
      " cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n mov.b32 %0, {t, z, z, z};\n}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}

constexpr float kSixth = 0x1.555556p-3f;  // 1/6 rounded to float32

// Bits of the scale of a group whose largest finite magnitude is amax;
// `bad`: the group holds an infinity or a NaN.
__device__ __forceinline__ uint32_t fp4_scale_bits(float amax, bool bad) {
  if (bad) return 0x7FC0u;
  return (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(amax, kSixth)));
}
__device__ __forceinline__ float bf16_bits_f32(uint32_t b) { return __uint_as_float(b << 16); }

// x / s for the code of x: zero where the group's scale is zero or NaN.
__device__ __forceinline__ float fp4_quotient(float x, float s) { return s > 0.0f ? __fdiv_rn(x, s) : 0.0f; }

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 tile of 16-bit elements held one row pair per thread.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

template <int N>
__device__ __forceinline__ void cp_async_wait_group() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Four consecutive elements k0 .. k0 + 3 of a row as float32, zeros at and
// past `n`.  `vec`: the row's address and k0 allow one wide load.
__device__ __forceinline__ float4 load4(const void* row, int dtype, long long k0, long long n, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (dtype == kF32) {
    const float* p = static_cast<const float*>(row) + k0;
    if (vec && k0 + 3 < n) return *reinterpret_cast<const float4*>(p);
    if (k0 < n) v.x = p[0];
    if (k0 + 1 < n) v.y = p[1];
    if (k0 + 2 < n) v.z = p[2];
    if (k0 + 3 < n) v.w = p[3];
    return v;
  }
  const uint16_t* p = static_cast<const uint16_t*>(row) + k0;
  uint32_t a = 0, b = 0;
  if (vec && k0 + 3 < n) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    a = u.x;
    b = u.y;
  } else {
    if (k0 < n) a = p[0];
    if (k0 + 1 < n) a |= (uint32_t)p[1] << 16;
    if (k0 + 2 < n) b = p[2];
    if (k0 + 3 < n) b |= (uint32_t)p[3] << 16;
  }
  if (dtype == kBF16) {
    const float2 lo = bf16x2_to_f2(a), hi = bf16x2_to_f2(b);
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  }
  const float2 lo = unpack_half2(a), hi = unpack_half2(b);
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// Bits of |x|, or 0 where x is an infinity or a NaN.
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
  return u < 0x7F800000u ? u : 0u;
}

// The power of two 2^k, 2^-k that brings a largest magnitude (its float32
// bits) into [2^14, 2^15), within the exponents that float32 holds as normal
// numbers both ways.  fp16 of x * 2^k then keeps eleven bits of every element
// down to 2^-29 of the largest one.
__device__ __forceinline__ void pow2_normaliser(uint32_t amax_bits, float* up, float* down) {
  int k = 14 - ((int)(amax_bits >> 23) - 127);
  if (amax_bits == 0) k = 0;
  k = k > 126 ? 126 : k;
  *up = __uint_as_float((uint32_t)(127 + k) << 23);
  *down = __uint_as_float((uint32_t)(127 - k) << 23);
}

// fp16 parts of v: hi = fp16(v), lo = fp16(v - hi) (zero where hi is not
// finite).  Together they hold 22 bits of v.
__device__ __forceinline__ float fp16_rest(float v) {
  const float h = __half2float(__float2half_rn(v));
  return fabsf(h) <= 65504.0f ? v - h : 0.0f;
}

__device__ __forceinline__ void store_elem(void* p, long long i, int dtype, float v) {
  if (dtype == kF32) static_cast<float*>(p)[i] = v;
  else if (dtype == kBF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

}  // namespace cpk
