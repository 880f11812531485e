// Device helpers shared by the gated linear attention kernels.
#pragma once

#include "common.cuh"

namespace la {

// log2 of a token's decay.  e^g below e^-120 is zero in fp32, and so is every product of it with
// a state the recurrence could hold; clamping there gives the same results and keeps differences
// of running sums finite (a log decay of -inf, i.e. a reset of the state, would give inf - inf).
// A NaN stays a NaN.
__device__ __forceinline__ double log2_decay(float g) {
  return (double)(g < -120.f ? -120.f : g) * 1.4426950408889634074;
}

// Running sums c of log2 decays reach 128 * 173 in a chunk full of resets, where fp32 resolves
// 2^-9 only.  They are summed in 64 bits and kept as hi (a multiple of 1/64, exact in fp32) plus
// lo, so that (hi_i - hi_j) + (lo_i - lo_j) is c_i - c_j to 2^-30.
struct Cum {
  float hi, lo;
};
__device__ __forceinline__ Cum split_cum(double c) {
  const float hi = (float)(rint(c * 64.0) * 0.015625);
  return Cum{hi, (float)(c - (double)hi)};
}

__device__ __forceinline__ double warp_scan(double x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
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
