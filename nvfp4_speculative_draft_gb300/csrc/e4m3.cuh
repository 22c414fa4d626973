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

// The same for eight binary32 values y (fast: s in [2^-126, 2^126]).
__device__ __forceinline__ uint2 codes_of(const float (&y)[8], float s, bool fast, uint64_t rlo2,
                                          uint64_t rhi2) {
  if (s == 0.0f) return make_uint2(0u, 0u);
  uint32_t lo[4], hi[4];
  bool ok = fast;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint64_t y2;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y2) : "f"(y[2 * j]), "f"(y[2 * j + 1]));
    lo[j] = e4m3_pair2(mul_rz_f32x2(y2, rlo2));
    hi[j] = e4m3_pair2(mul_rz_f32x2(y2, rhi2));
    ok = ok && lo[j] == hi[j];
  }
  if (!ok) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      lo[j] = e4m3_pair(__fdiv_rn(y[2 * j], s), __fdiv_rn(y[2 * j + 1], s));
  }
  return make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
}

// The scale of a block or row group and the reciprocal bounds its codes are
// decided with.  With s in [2^-126, 2^126], 1/s is normal and finite and
// rlo <= 1/s, rhi >= (1 + 2^-22)/s.
struct Scale {
  float s;
  bool fast;
  uint64_t rlo, rhi;
};
__device__ __forceinline__ Scale scale_of(float amax) {
  Scale r;
  r.s = __fdiv_rn(amax, 448.0f);
  r.fast = r.s >= 0x1p-126f && r.s <= 0x1p126f;
  r.rlo = f32x2_splat(r.fast ? __frcp_rd(r.s) : 0.0f);
  r.rhi = f32x2_splat(r.fast ? __fmul_ru(__frcp_ru(r.s), 1.0f + 0x1p-22f) : 0.0f);
  return r;
}

}  // namespace e4m3
}  // namespace nvfp4
