// Eight consecutive values of a row in registers, and the sigmoid, shared by the channels-last kernels.
#pragma once

#include "gated.cuh"

namespace la {

// Eight values as loaded; converted where they are used, so that rows in flight cost few registers.
template <typename T>
struct Raw {
  uint4 a[sizeof(T) / 2];
  __device__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) a[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ void zero() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) a[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ void get(float2 (&o)[4]) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = sizeof(T) == 2 ? make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u))
                            : make_float2(__uint_as_float(w[(2 * e) % (2 * sizeof(T))]),
                                          __uint_as_float(w[(2 * e + 1) % (2 * sizeof(T))]));
  }
};
__device__ __forceinline__ void put8(float *p, const float2 (&o)[4]) {
  st4(p, o[0].x, o[0].y, o[1].x, o[1].y);
  st4(p + 4, o[2].x, o[2].y, o[3].x, o[3].y);
}
__device__ __forceinline__ void put8(__nv_bfloat16 *p, const float2 (&o)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[e].x, o[e].y);
    w[e] = *reinterpret_cast<const uint32_t *>(&x);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// e^-x and 1 / (1 + e^-x), two at a time: e^-x overflows to inf below -88, where the quotient is 0 as it
// should be.  The approximate instructions are taken without their care for subnormal numbers (there 1 + e^-x
// is 1, and the quotient below 1e-38): issue slots, 70 % of them taken, bound the group norm's forward
// beside HBM: 68 to 65 us.
struct Sigmoid2 {
  float2 e, s;
  __device__ __forceinline__ explicit Sigmoid2(float2 x) {
    const float2 t = __fmul2_rn(x, both(-1.44269504f));  // -log2 e
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    const float2 d = __fadd2_rn(e, both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(d.y));
  }
  // 1 - s as e^-x s, which keeps its bits where s is near 1 (a gate of 1e4 multiplies what 1 - s would
  // have lost); inf * 0 is NaN, of which the minimum takes the 1.
  __device__ __forceinline__ float2 one_less() const {
    const float2 o = __fmul2_rn(e, s);
    return make_float2(fminf(o.x, 1.f), fminf(o.y, 1.f));
  }
};

}  // namespace la
