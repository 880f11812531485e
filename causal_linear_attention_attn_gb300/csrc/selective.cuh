// Pieces shared by the selective scan, its gradient and its step.
//
//   delta = softplus(dt + dt_bias),  h_t = e^{delta A} h_{t-1} + (delta x_t) B_t,
//   y_t = sum_n C_t,n h_t,n + D x_t,  out_t = y_t silu(z_t)
//
// per channel, with ds state components each; B_t and C_t belong to all channels.
#pragma once

#include "vec8.cuh"

namespace la {

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float2 exp2_approx(float2 x) { return make_float2(exp2_approx(x.x), exp2_approx(x.y)); }

// A log2 e.  A = -inf, a component that forgets at once, becomes the lowest finite number: a token without a step, padding
// among them, still changes nothing.
__device__ __forceinline__ float rate(float A) {
  constexpr float kLowest = -3.402823466e38f;
  const float r = A * kLog2e;
  return r < kLowest ? kLowest : r;
}
__device__ __forceinline__ float2 rate(float2 A) { return make_float2(rate(A.x), rate(A.y)); }

// A state's decay e^{delta A}, A as rate(A).  The instruction's results are low on average, measured over each
// power of two of the exponent: by 0.5e-8 to 2.6e-8 of their value above 2^-1/8, 5e-8 below.  A state that remembers a
// thousand tokens is a product of as many, so the exponent leans up by what centres those (2^kLean is still exactly 1: a
// token without a step changes nothing).  2 x 4096 x 512 x 16: the gradient of A is
// off by 0.8e-6 (1.8e-6 without; plain 32-bit exponentials 1.5e-6), the state by 2.7e-7 (5.7e-7; 4.1e-7).
constexpr float kLean = 2.2e-8f;
__device__ __forceinline__ float2 decay(float2 delta, float2 A) { return exp2_approx(__ffma2_rn(delta, A, make_float2(kLean, kLean))); }

// log(1 + e^v) = max(v, 0) + log1p(e^-|v|), two at a time.  log1p(e) = e P(e) on [0, 1], P of degree 9 (least
// largest relative error, 5e-9; 1.5e-7 with the rounding of its steps): small steps delta keep their bits, which a
// logarithm of 1 + e would lose.
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 m = make_float2(-fabsf(v.x), -fabsf(v.y));
  const float2 e = exp2_approx(__fmul2_rn(m, both(kLog2e)));
  float2 p = both(-0.0032440247f);
  p = __ffma2_rn(p, e, both(0.0198514629f));
  p = __ffma2_rn(p, e, both(-0.0569595397f));
  p = __ffma2_rn(p, e, both(0.106036559f));
  p = __ffma2_rn(p, e, both(-0.153055936f));
  p = __ffma2_rn(p, e, both(0.196759403f));
  p = __ffma2_rn(p, e, both(-0.249541342f));
  p = __ffma2_rn(p, e, both(0.333299637f));
  p = __ffma2_rn(p, e, both(-0.499999017f));
  p = __ffma2_rn(p, e, both(1.f));
  // (max passes over a NaN, e does not: it is NaN then)
  return __ffma2_rn(p, e, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

// Where two channels' steps are: eight lanes that write four neighbours each meet no bank twice.
__device__ __forceinline__ int step_slot(int pair) { return pair ^ (pair >> 3 & 3); }

// Named barriers between kinds of warps: all kThreads threads, some of which wait.
template <int kThreads>
__device__ __forceinline__ void bar_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}
template <int kThreads>
__device__ __forceinline__ void bar_arrive(int id) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "n"(kThreads) : "memory");
}

// Sums over the lanes of aligned groups of kLanes (a power of two) of kVals values a lane, which end up
// spread over the group: each round halves the lanes that still add the same values and the values a lane holds, so
// kVals values cost about kVals shuffles and not kVals log2(kLanes).  `stride`: lanes of a group are that far apart.
// Afterwards v[0 .. max(1, kVals / kLanes) - 1] hold values  index(lane) + kLanes * i  (kVals >= kLanes),
// or every kVals lanes the same value (kVals < kLanes), index(lane) = lane's number in the group mod kVals.
template <int kLanes, int kVals, int kStride>
__device__ __forceinline__ void spread_sum(float (&v)[kVals], int number) {
  int have = kVals;
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    if (have > 1) {
      const bool up = number & o;
#pragma unroll
      for (int i = 0; i < kVals / 2; ++i) {
        if (2 * i + 1 < have) {
          const float give = up ? v[2 * i] : v[2 * i + 1], keep = up ? v[2 * i + 1] : v[2 * i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o * kStride);
        }
      }
      have >>= 1;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o * kStride);
    }
  }
}

}  // namespace la
