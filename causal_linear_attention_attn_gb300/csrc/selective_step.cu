// One token of the selective scan per served row, on states in a pool: a read-modify-write of the states,
// bound by HBM (8 bytes a component; delta, x and the gate are a channel's, B and C a row's).
//
// A thread owns four components of a channel (16 bytes, neighbours in memory for neighbouring lanes), ds / 4 lanes
// a channel, and loads all of its states before it uses the first.  A slot out of range, or one that an
// earlier row of the batch already has, leaves its state alone (two rows on one state would race).
#include "internal.h"
#include "selective.cuh"

namespace la {

__device__ unsigned int g_scan_step_status;

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 4;  // states a thread

template <typename T, int DS>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(const __grid_constant__ ScanStepProblem p, int per_row) {
  constexpr int kLanes = DS / 4;
  const int b = blockIdx.x / per_row, part = blockIdx.x - b * per_row;
  const int slot = p.slots ? p.slots[b] : b;
  const bool bad = slot < 0 || slot >= p.n_slots;
  const int q = threadIdx.x % kLanes;
  const long quads = (long)p.D * kLanes, first = (long)part * kThreads * kPer + threadIdx.x;
  float4 *S = bad ? nullptr : reinterpret_cast<float4 *>(p.S) + (long)slot * quads;
  float4 h[kPer], A[kPer];
  float dt[kPer], x[kPer], z[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const long i = first + u * kThreads;
    if (bad || i >= quads) continue;
    const long c = i / kLanes;
    h[u] = __ldcs(S + i);
    A[u] = __ldg(reinterpret_cast<const float4 *>(p.A) + i);
    dt[u] = ldf((const T *)p.delta + b * p.ldt + c) + (p.dt_bias ? p.dt_bias[c] : 0.f);
    x[u] = ldf((const T *)p.x + b * p.ldx + c);
    z[u] = p.z ? ldf((const T *)p.z + b * p.ldz + c) : 0.f;
  }
  const float4 B = ld4((const T *)p.Bm + b * p.ldb + 4 * q), C = ld4((const T *)p.Cm + b * p.ldc + 4 * q);
  int again = 0;
  if (p.slots && !bad)
    for (int o = threadIdx.x; o < b; o += kThreads) again |= p.slots[o] == slot;
  const bool skip = __syncthreads_or(again) || bad;
  if (skip && slot >= 0 && threadIdx.x == 0) atomicOr(&g_scan_step_status, kStatusBadSlot);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const long i = first + u * kThreads, c = i / kLanes;
    const bool in = i < quads;  // the channels' lanes stay together: quads is a multiple of kLanes
    float y = 0.f;
    if (in && !skip) {
      const float d = p.softplus ? softplus2(both(dt[u])).x : dt[u], du = d * x[u], d2 = d * kLog2e;
      h[u].x = fmaf(exp2_approx(d2 * A[u].x), h[u].x, du * B.x);
      h[u].y = fmaf(exp2_approx(d2 * A[u].y), h[u].y, du * B.y);
      h[u].z = fmaf(exp2_approx(d2 * A[u].z), h[u].z, du * B.z);
      h[u].w = fmaf(exp2_approx(d2 * A[u].w), h[u].w, du * B.w);
      __stcs(S + i, h[u]);
      y = fmaf(h[u].x, C.x, fmaf(h[u].y, C.y, fmaf(h[u].z, C.z, h[u].w * C.w)));
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (in && q == 0) {
      if (!skip) {
        if (p.Dskip) y = fmaf(p.Dskip[c], x[u], y);
        if (p.z) y *= z[u] * Sigmoid2(both(z[u])).s.x;
      }
      T *to = (T *)p.out + (long)b * p.D + c;
      if constexpr (sizeof(T) == 2)
        *to = __float2bfloat16(y);
      else
        *to = y;
    }
  }
}

template <typename T, int DS>
cudaError_t launch_t(const ScanStepProblem &p) {
  const int per_row = (int)(((long)p.D * (DS / 4) + kThreads * kPer - 1) / (kThreads * kPer));
  LaunchTimer timer(kKSelectiveStep, p.stream);
  scan_step_kernel<T, DS><<<(unsigned)((long)per_row * p.B), kThreads, 0, p.stream>>>(p, per_row);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T>
cudaError_t launch_ds(const ScanStepProblem &p) {
  return p.ds == 8 ? launch_t<T, 8>(p) : p.ds == 16 ? launch_t<T, 16>(p) : p.ds == 32 ? launch_t<T, 32>(p) : launch_t<T, 64>(p);
}

}  // namespace

cudaError_t launch_selective_step(const ScanStepProblem &p) {
  return p.dt == LA_F32 ? launch_ds<float>(p) : launch_ds<__nv_bfloat16>(p);
}

cudaError_t read_and_clear_scan_step_status(unsigned int *value) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_scan_step_status, sizeof(unsigned int));
  if (e == cudaSuccess && *value) e = cudaMemcpyToSymbol(g_scan_step_status, &zero, sizeof(unsigned int));
  return e;
}

}  // namespace la
