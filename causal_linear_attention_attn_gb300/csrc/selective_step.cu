// One token of the selective scan per served row, on states in a pool: a read-modify-write of the states,
// bound by HBM (8 bytes a component; delta, x and the gate are a channel's, B and C a row's).  512 rows of 2048 x 16 in
// 35 us in bf16, 4.1 TB/s (fp32 39 us, 3.9 TB/s): a block loads, waits, stores and ends, and nothing loads the next rows
// meanwhile.  28 us call by call on the same states, which L2 then holds in part (one row a block, and every lane its
// channel's step: 49 us).
//
// A thread owns four components of a channel (16 bytes, neighbours in memory for neighbouring lanes), ds / 4 lanes
// a channel, in two places of the state and, with many rows, in four rows, so that it reads A once for them and has
// eight loads of states under way before it uses the first.  Meanwhile the block works out what belongs to whole
// channels, a thread a channel and row: the step, its product with x, the gate.  A slot out of range, or one that an earlier row of the
// batch already has, leaves its state alone (two rows on one state would race).
#include <algorithm>

#include "internal.h"
#include "selective.cuh"

namespace la {

__device__ unsigned int g_scan_step_status;

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 2;  // places a thread

template <typename T, int DS, int kRows>
__global__ void __launch_bounds__(kThreads, 3) scan_step_kernel(const __grid_constant__ ScanStepProblem p, int per_row) {
  constexpr int kLanes = DS / 4;
  constexpr int kCols = kThreads * kPer / kLanes;  // channels a block
  struct Item {
    float d, du, gate, skip;  // delta, delta x, silu(z), D x
  };
  __shared__ Item items[kRows][kCols];
  __shared__ __align__(16) float bc[kRows][2][DS];
  __shared__ int twice[kRows];
  const int group = blockIdx.x / per_row, part = blockIdx.x - group * per_row, b0 = group * kRows;
  const int q = threadIdx.x % kLanes;
  const long quads = (long)p.D * kLanes;
  const int first = part * kThreads * kPer + threadIdx.x;  // (at most 2^29 quads a row)
  if (threadIdx.x < kRows) twice[threadIdx.x] = 0;
  int slot[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int b = b0 + r;
    slot[r] = b < p.B ? (p.slots ? p.slots[b] : b) : -1;
    if (slot[r] >= p.n_slots) slot[r] = -2;
  }
  float4 h[kRows][kPer], A[kPer];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (slot[r] >= 0 && first + u * kThreads < quads)
        h[r][u] = __ldcs(reinterpret_cast<const float4 *>(p.S) + slot[r] * quads + first + u * kThreads);
#pragma unroll
  for (int u = 0; u < kPer; ++u)
    if (first + u * kThreads < quads) A[u] = __ldg(reinterpret_cast<const float4 *>(p.A) + first + u * kThreads);
  for (int i = threadIdx.x; i < kRows * kCols; i += kThreads) {
    const int r = i / kCols, j = i % kCols, c = part * kCols + j;
    const long b = b0 + r;
    if (b >= p.B || c >= p.D) continue;
    const float x = ldf((const T *)p.x + b * p.ldx + c);
    float d = ldf((const T *)p.delta + b * p.ldt + c) + (p.dt_bias ? p.dt_bias[c] : 0.f);
    const float z = p.z ? ldf((const T *)p.z + b * p.ldz + c) : 0.f;
    if (p.softplus) d = softplus2(both(d)).x;
    items[r][j] = Item{d, d * x, p.z ? z * Sigmoid2(both(z)).s.x : 1.f, p.Dskip ? p.Dskip[c] * x : 0.f};
  }
  for (int i = threadIdx.x; i < kRows * 2 * DS; i += kThreads) {
    const int r = i / (2 * DS), j = i % (2 * DS);
    const long b = b0 + r;
    if (b < p.B) bc[r][j / DS][j % DS] = j < DS ? ldf((const T *)p.Bm + b * p.ldb + j) : ldf((const T *)p.Cm + b * p.ldc + j - DS);
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) A[u] = make_float4(rate(A[u].x), rate(A[u].y), rate(A[u].z), rate(A[u].w));
  __syncthreads();
  if (p.slots) {
    for (int o = threadIdx.x; o < min(b0 + kRows, p.B) - 1; o += kThreads) {
      const int s = p.slots[o];
#pragma unroll
      for (int r = 0; r < kRows; ++r)
        if (o < b0 + r && s == slot[r]) twice[r] = 1;
    }
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int b = b0 + r;
    if (b >= p.B) break;
    const bool again = p.slots && slot[r] >= 0 && twice[r], skip_row = slot[r] < 0 || again;
    if ((again || slot[r] == -2) && (!p.slots || p.slots[b] >= 0) && threadIdx.x == 0) atomicOr(&g_scan_step_status, kStatusBadSlot);
    const float4 B = ld4(&bc[r][0][4 * q]), C = ld4(&bc[r][1][4 * q]);
    float4 *S = reinterpret_cast<float4 *>(p.S) + slot[r] * quads + first;
    T *out = (T *)p.out + (long)b * p.D;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const int i = first + u * kThreads, c = i / kLanes;
      const bool in = i < quads;  // a channel's lanes stay together: quads is a multiple of kLanes
      float y = 0.f;
      const Item &it = items[r][(threadIdx.x + u * kThreads) / kLanes];
      if (in && !skip_row) {
        const float d = it.d, du = it.du;
        float4 &s = h[r][u];
        s.x = fmaf(exp2_approx(fmaf(d, A[u].x, kLean)), s.x, du * B.x);
        s.y = fmaf(exp2_approx(fmaf(d, A[u].y, kLean)), s.y, du * B.y);
        s.z = fmaf(exp2_approx(fmaf(d, A[u].z, kLean)), s.z, du * B.z);
        s.w = fmaf(exp2_approx(fmaf(d, A[u].w, kLean)), s.w, du * B.w);
        __stcs(S + u * kThreads, s);
        y = fmaf(s.x, C.x, fmaf(s.y, C.y, fmaf(s.z, C.z, s.w * C.w)));
      }
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      if (in && q == 0) {
        y = skip_row ? 0.f : (y + it.skip) * it.gate;
        if constexpr (sizeof(T) == 2)
          out[c] = __float2bfloat16(y);
        else
          out[c] = y;
      }
    }
  }
}

template <typename T, int DS, int kRows>
cudaError_t launch_rows(const ScanStepProblem &p) {
  const int per_row = (int)(((long)p.D * (DS / 4) + kThreads * kPer - 1) / (kThreads * kPer));
  LaunchTimer timer(kKSelectiveStep, p.stream);
  scan_step_kernel<T, DS, kRows><<<(unsigned)((long)per_row * ((p.B + kRows - 1) / kRows)), kThreads, 0, p.stream>>>(p, per_row);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

// Four rows a block once that leaves two blocks an SM.
template <typename T, int DS>
cudaError_t launch_t(const ScanStepProblem &p) {
  const long quads = (long)p.B * p.D * (DS / 4);
  return quads >= 4L * kThreads * kPer * 2 * std::max(1, device_info(-1).sm_count) ? launch_rows<T, DS, 4>(p) : launch_rows<T, DS, 1>(p);
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
