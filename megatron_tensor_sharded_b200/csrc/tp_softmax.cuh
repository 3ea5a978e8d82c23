// Softmax arithmetic shared by the attention kernels: 2^x on the MUFU unit and
// on the FMA pipe, three-input maxima, bf16 pairs.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <cstring>

#include "tp_device.cuh"

namespace tpk {

constexpr unsigned kErrWaitAttn = 1u << 6;      // attention: Q, scores, probabilities or output

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  uint32_t u;
  memcpy(&u, &v, 4);
  return u;
}

// The softmax's hot loops use the packed fp32 pair helpers f2_* of
// tp_device.cuh (sm_100 FFMA2 / FADD2: two lanes per instruction).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 2^x on the FMA pipe, for part of the probabilities so that the MUFU unit
// (16 exp2 per clock per SM) is not the only one computing them: range
// reduction to the nearest integer n (x = n + f, |f| <= 1/2, by the
// 1.5 * 2^23 rounding constant), a degree-4 polynomial for 2^f whose
// coefficients were fitted to minimise the relative error on [-1/2, 1/2]
// (iteratively reweighted least squares; max relative error of the fit
// 2.6e-6, of the fp32 evaluation below at most 2.7e-6 on [-126, 0]), and n
// added to the exponent field.  x is clamped to >= -126, or, MASKED, to
// -126.9999: the polynomial is 1 + 6.9e-5 there and the bits come to 8e-43, so
// -inf gives a number that is 0 as bf16 (2^-126 is not, and would count beside
// a value of 2^127).  (At -127 itself the polynomial is just below 1 and the
// bits would be a NaN's.)  Two lanes per call.
template <bool MASKED>
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x2) {
  constexpr float kLeast = MASKED ? -126.9999f : -126.0f;
  float x0, x1;
  f2_unpack(x2, x0, x1);
  x2 = f2_pack(fmaxf(x0, kLeast), fmaxf(x1, kLeast));
  const uint64_t magic = f2_pack(12582912.0f, 12582912.0f);
  const uint64_t t = f2_add(x2, magic);
  const uint64_t n = f2_add(t, f2_pack(-12582912.0f, -12582912.0f));
  const uint64_t f = f2_fma(n, f2_pack(-1.0f, -1.0f), x2);
  uint64_t p = f2_fma(f2_pack(0.009570101276040077f, 0.009570101276040077f), f,
                      f2_pack(0.05591785907745361f, 0.05591785907745361f));
  p = f2_fma(p, f, f2_pack(0.240247443318367f, 0.240247443318367f));
  p = f2_fma(p, f, f2_pack(0.6931217908859253f, 0.6931217908859253f));
  p = f2_fma(p, f, f2_pack(0.9999992847442627f, 0.9999992847442627f));
  float p0, p1, t0, t1;
  f2_unpack(p, p0, p1);
  f2_unpack(t, t0, t1);
  return f2_pack(__int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23)),
                 __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23)));
}

// The same maximum, NaN if an operand is one.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 2^x of two lanes on the FMA pipe as exp2_poly2, by a polynomial of degree 5
// fitted the same way (relative error of the fit 7.5e-8, in fp32 2.1e-7: the
// log of a row's sum is kept in fp32).  NAN_SAFE: NaN for a NaN -- the power
// of two is multiplied in (its exponent field is built apart), where adding
// to the bits of a NaN would give a number.  Otherwise the clamp lies at -127,
// where the polynomial is 1 + 2^-23 and the bits come to 2^-149: -inf gives a
// number that is 0 as bf16.  (2^-126 is not: a key that a row does not see
// would add 2^-126 times its value, which may be 2^127.)  Between -127 and
// -126 the result lies between 0 and 2^-126.
template <bool NAN_SAFE>
__device__ __forceinline__ uint64_t exp2_poly5(uint64_t x2) {
  float x0, x1;
  f2_unpack(x2, x0, x1);
  if (NAN_SAFE)
    x2 = f2_pack(max3_nan(x0, -126.0f, -126.0f), max3_nan(x1, -126.0f, -126.0f));
  else
    x2 = f2_pack(fmaxf(x0, -127.0f), fmaxf(x1, -127.0f));
  const uint64_t magic = f2_pack(12582912.0f, 12582912.0f);
  const uint64_t t = f2_add(x2, magic);
  const uint64_t n = f2_add(t, f2_pack(-12582912.0f, -12582912.0f));
  const uint64_t f = f2_fma(n, f2_pack(-1.0f, -1.0f), x2);
  uint64_t p = f2_fma(f2_pack(0.001327647129073739f, 0.001327647129073739f), f, f2_pack(0.009675540961325169f, 0.009675540961325169f));
  p = f2_fma(p, f, f2_pack(0.05550713092088699f, 0.05550713092088699f));
  p = f2_fma(p, f, f2_pack(0.24022120237350464f, 0.24022120237350464f));
  p = f2_fma(p, f, f2_pack(0.6931469440460205f, 0.6931469440460205f));
  p = f2_fma(p, f, f2_pack(1.0000001192092896f, 1.0000001192092896f));
  float t0, t1;
  f2_unpack(t, t0, t1);
  if (NAN_SAFE)
    return f2_mul(p, f2_pack(__int_as_float((__float_as_int(t0) << 23) + 0x3f800000),
                             __int_as_float((__float_as_int(t1) << 23) + 0x3f800000)));
  float p0, p1;
  f2_unpack(p, p0, p1);
  return f2_pack(__int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23)),
                 __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23)));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace tpk
