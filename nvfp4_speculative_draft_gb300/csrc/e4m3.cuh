// e4m3.cuh -- E4M3 codes of correctly rounded quotients, shared by the FP8
// quantisers: code = E4M3_RNE_SATFINITE(fl32(x / s)).
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace nvfp4 {
namespace e4m3 {

__device__ __forceinline__ uint4 ld_u4(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t mag_max8(uint4 v) {
  return __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                  __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
}

// Eight codes by one correctly rounded division each; code byte j is
// element j (even elements in the low BF16 half of each word).
__device__ __forceinline__ uint2 codes_exact(uint4 v, float s) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = (j & 1) ? (u[j >> 1] & 0xFFFF0000u) : (u[j >> 1] << 16);
    const float q = __fdiv_rn(__uint_as_float(b), s);
    const uint32_t c = (uint32_t)__nv_cvt_float_to_fp8(q, __NV_SATFINITE, __NV_E4M3);
    out[j >> 2] |= c << (8 * (j & 3));
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ uint32_t e4m3_pair(float a_even, float a_odd) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a_even, a_odd), __NV_SATFINITE,
                                            __NV_E4M3);
}

// Two BF16 pairs -> four code bytes.  With rlo <= 1/s and rhi >= (1 + 2^-22)/s,
// RZ(x rlo) and RZ(x rhi) carry the sign of x and bracket the magnitude of
// fl32(x/s); the monotone, sign-keeping RNE satfinite conversion of the two
// bounds then brackets its code.  Returns false when the bracket holds two
// codes.
__device__ __forceinline__ uint64_t f32x2_of_bf16x2(uint32_t u) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(u << 16), "r"(u & 0xFFFF0000u));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_splat(float a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(a));
  return r;
}
// packed binary32 product of two pairs, rounded toward zero (sm_100+ f32x2)
__device__ __forceinline__ uint64_t mul_rz_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_pair2(uint64_t q) {
  float e, o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(e), "=f"(o) : "l"(q));
  return e4m3_pair(e, o);
}

__device__ __forceinline__ bool codes_fast_word(uint32_t u0, uint32_t u1, uint64_t rlo2,
                                                uint64_t rhi2, uint32_t& out) {
  const uint64_t x01 = f32x2_of_bf16x2(u0), x23 = f32x2_of_bf16x2(u1);
  const uint32_t lo = e4m3_pair2(mul_rz_f32x2(x01, rlo2)) |
                      e4m3_pair2(mul_rz_f32x2(x23, rlo2)) << 16;
  const uint32_t hi = e4m3_pair2(mul_rz_f32x2(x01, rhi2)) |
                      e4m3_pair2(mul_rz_f32x2(x23, rhi2)) << 16;
  out = lo;
  return lo == hi;
}

__device__ __forceinline__ uint2 codes_of(uint4 v, float s, bool fast, uint64_t rlo2,
                                          uint64_t rhi2) {
  if (s == 0.0f) return make_uint2(0u, 0u);
  if (fast) {
    uint2 r;
    const bool ok0 = codes_fast_word(v.x, v.y, rlo2, rhi2, r.x);
    const bool ok1 = codes_fast_word(v.z, v.w, rlo2, rhi2, r.y);
    if (ok0 && ok1) return r;
  }
  return codes_exact(v, s);
}

// ---- block scales: quotients without a division per element
//
// s = RN(amax / 448), and each code from q = q0 + (x - s q0) y with y = 1/s to within
// an ulp, q0 = RN(x y) (one step of Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990): the remainder is exact to 2^-23 of
// an ulp of q, so q = RN(x/s + e), |e| < 2^-20 ulp.  For BF16 x and amax that is
// fl32(x/s) wherever it decides a code: x and amax have 8 bits and a code border M
// five, so where x/s is nearer than 2^-13 to M it is M (amax/448)/s, whose distance
// from M in ulps is a multiple of about 2^-8 and never half of one.  For FP32 x (a
// normalised row) q is fl32(x/s) but for a share of about 2^-20 of the quotients that
// lie next to a border, themselves about 2^-19 of all.
// fast: amax in [2^-80, 2^127), where no remainder that can decide a code
// (|q| >= 2^-10) leaves binary32's normal range; divisions otherwise.
// (A rounding test with a division in doubt, as above, costs more here: up to a per
// cent of the quotients of BF16 values by a BF16 maximum lie on a border exactly.)
// The steps form -q, from -y: the remainder of x = +-0 is +0, and the last step's
// (+0)(-y) + (-q0) is then -q0 for either sign, where (+0) y + q0 would lose the sign of
// -0.  Conversion to E4M3 is symmetric, so a code's sign bit is flipped instead.
struct Scale {
  float s;
  bool fast;
  uint64_t neg_y, pair;  // -1/s and s, as pairs
};
__device__ __forceinline__ Scale scale_of(float amax) {
  Scale o;
  o.fast = amax >= 0x1p-80f && amax < 0x1p127f;
  constexpr float c = 1.0f / 448.0f;
  const float q = amax * c;
  o.s = o.fast ? fmaf(fmaf(-448.0f, q, amax), c, q) : __fdiv_rn(amax, 448.0f);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(o.s));
  o.neg_y = f32x2_splat(-y);
  o.pair = f32x2_splat(o.s);
  return o;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
// Eight codes of four pairs (first element in the lowest byte).
__device__ __forceinline__ uint2 codes_of(const uint64_t (&x)[4], const Scale& sc) {
  uint32_t c[4];
  if (sc.fast) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t nq = mul_f32x2(x[j], sc.neg_y);  // -q0
      c[j] = e4m3_pair2(fma_f32x2(fma_f32x2(sc.pair, nq, x[j]), sc.neg_y, nq));
    }
    return make_uint2((c[0] | c[1] << 16) ^ 0x80808080u, (c[2] | c[3] << 16) ^ 0x80808080u);
  } else if (sc.s == 0.0f) {
    return make_uint2(0u, 0u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      unpack_f32x2(x[j], a, b);
      c[j] = e4m3_pair(__fdiv_rn(a, sc.s), __fdiv_rn(b, sc.s));
    }
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
__device__ __forceinline__ void pairs_of(uint4 v, uint64_t (&x)[4]) {  // eight BF16 as FP32
  x[0] = f32x2_of_bf16x2(v.x);
  x[1] = f32x2_of_bf16x2(v.y);
  x[2] = f32x2_of_bf16x2(v.z);
  x[3] = f32x2_of_bf16x2(v.w);
}

__device__ __forceinline__ uint2 codes_of(uint4 v, const Scale& sc) {
  uint64_t x[4];
  pairs_of(v, x);
  return codes_of(x, sc);
}

}  // namespace e4m3
}  // namespace nvfp4
