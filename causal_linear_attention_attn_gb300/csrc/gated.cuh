// Device helpers shared by the gated linear attention kernels.
#pragma once

#include "common.cuh"

namespace la {

// Running sums of log2 decays, in 64-bit fixed point with 40 fraction bits: a chunk full of resets
// sums to 128 * 173, where fp32 resolves 2^-9 only, and the FP64 unit of this GPU is slow enough to
// set the pace of a whole kernel (a warp's scan of 128 doubles took 8000 cycles, this one under 1000).
//
// e^g below e^-120 is zero in fp32, and so is every product of it with a state the recurrence could
// hold; clamping there gives the same results and keeps differences of sums finite (a log decay of
// -inf, i.e. a reset of the state, would give inf - inf).  Above e^120 it is inf in fp32 as well.
__device__ __forceinline__ long long fixed_log2_decay(float g) {
  const float x = fminf(fmaxf(g, -120.f), 120.f);  // a NaN is dealt with apart (nan_before)
  const float l2e = 1.44269504f, l2e_lo = 1.92596303e-8f;  // log2(e) in two parts
  const float p = x * l2e, e = fmaf(x, l2e_lo, fmaf(x, l2e, -p));
  return __float2ll_rn(p * 1099511627776.f) + __float2ll_rn(e * 1099511627776.f);
}

// A sum as hi (a multiple of 1/64, exact in fp32) plus lo, so that (hi_i - hi_j) + (lo_i - lo_j) is
// c_i - c_j to 2^-30.
struct Cum {
  float hi, lo;
};
__device__ __forceinline__ Cum split_cum(long long c, bool nan) {
  const int h = (int)((c + (1ll << 33)) >> 34);
  const int rem = (int)((c - ((long long)h << 34)) >> 3);
  return Cum{nan ? __int_as_float(0x7fffffff) : (float)h * 0.015625f, (float)rem * 7.275957614183426e-12f};
}

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// fp32 sums that carry their rounding errors along (two-sum), for the long sums behind dg.
struct Sum2 {
  float s, e;
  __device__ __forceinline__ void add(float x, float xe = 0.f) {
    const float t = s + x, b = t - s;
    e += ((s - (t - b)) + (x - b)) + xe;
    s = t;
  }
};
// Sum over the lanes below (kDown: above) this one, this lane's x not included.
template <bool kDown>
__device__ __forceinline__ Sum2 warp_scan_others(Sum2 x, int lane) {
  // shift by one lane first, then an inclusive scan
  Sum2 y{kDown ? __shfl_down_sync(0xffffffffu, x.s, 1) : __shfl_up_sync(0xffffffffu, x.s, 1),
         kDown ? __shfl_down_sync(0xffffffffu, x.e, 1) : __shfl_up_sync(0xffffffffu, x.e, 1)};
  if (kDown ? lane == 31 : lane == 0) y = Sum2{0.f, 0.f};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float s = kDown ? __shfl_down_sync(0xffffffffu, y.s, o) : __shfl_up_sync(0xffffffffu, y.s, o);
    const float e = kDown ? __shfl_down_sync(0xffffffffu, y.e, o) : __shfl_up_sync(0xffffffffu, y.e, o);
    if (kDown ? lane + o < 32 : lane >= o) y.add(s, e);
  }
  return y;
}

// Tokens of batch row b that take part.
__device__ __forceinline__ long row_length(const int *lengths, long b, long N) {
  if (!lengths) return N;
  const long n = lengths[b];
  return n < 0 ? 0 : (n > N ? N : n);
}

__device__ __forceinline__ void st4(float *p, float a, float b, float c, float d) {
  *reinterpret_cast<float4 *>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void st4(__nv_bfloat16 *p, float a, float b, float c, float d) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  *reinterpret_cast<uint2 *>(p) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}

}  // namespace la
