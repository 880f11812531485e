// Device helpers shared by the gated linear attention kernels.
#pragma once

#include "common.cuh"

namespace la {

// Running sums of log2 decays, in 64-bit fixed point with 40 fraction bits: a chunk full of strong decays
// sums to 128 * 150, where fp32 resolves 2^-9 only, and the FP64 unit of this GPU is slow enough to
// set the pace of a whole kernel (a warp's scan of 128 doubles took 8000 cycles, this one under 1000).
//
// A decay that is zero in fp32 (e^-104 < 2^-150; a log decay of -inf among them) is a cut: the recurrence
// reads nothing across it, whatever follows.  It counts as 2^-32768: decays above e^120 are taken as that
// (inf in fp32 as well), so the 127 other tokens of a chunk grow by 2^21986 at most, and every weight across a
// cut is zero.  The state, which may be inf or NaN, is dropped there and not multiplied by zero.
// (The floats are chosen from, not the sums: choosing between those cost 3 of the prefill's 148 us.)
__device__ __forceinline__ bool is_cut(float g) { return g < -104.f; }
__device__ __forceinline__ long long fixed_log2_decay(float g) {
  const float x = is_cut(g) ? -22713.f : fminf(g, 120.f);  // a NaN is dealt with apart (split_cum)
  const float l2e = 1.44269504f, l2e_lo = 1.92596303e-8f;  // log2(e) in two parts
  const float p = x * l2e, e = fmaf(x, l2e_lo, fmaf(x, l2e, -p));
  return __float2ll_rn(p * 1099511627776.f) + __float2ll_rn(e * 1099511627776.f);
}

// A sum as hi (a multiple of 1/4, exact in fp32: 128 cuts are 2^22) plus lo, so that
// (hi_i - hi_j) + (lo_i - lo_j) is c_i - c_j to 2^-27.
struct Cum {
  float hi, lo;
};
__device__ __forceinline__ Cum split_cum(long long c, bool nan) {
  const int h = (int)((c + (1ll << 37)) >> 38);
  const int rem = (int)((c - ((long long)h << 38)) >> 7);
  return Cum{nan ? __int_as_float(0x7fffffff) : (float)h * 0.25f, (float)rem * 1.1641532182693481e-10f};
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
