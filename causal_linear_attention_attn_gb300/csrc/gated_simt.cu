// Gated linear attention on CUDA cores, fp32 throughout: the path of fp32 inputs and of head sizes
// the tensor-core kernels do not take.
//
//   S_t = a_t S_{t-1} + k_t v_t^T,  out_t = q_t^T S_t,  a_t = e^{g_t}
//
// Over a chunk of T tokens (local rows i, j; c the running sum of log2 decays, inclusive) that
// starts from the state S:
//   out_i = 2^{c_i} q_i^T S + sum_{j <= i} 2^{c_i - c_j} (q_i . k_j) v_j
//   S'    = 2^{c_T} S + sum_j 2^{c_T - c_j} k_j v_j^T
// Every exponent is a difference of running sums of a token and an earlier one, so no weight
// exceeds 1 for g <= 0, however fast the decay.  Backward, with R the gradient of S' :
//   dq_i = 2^{c_i} S do_i + sum_{j <= i} D_ij k_j,        D_ij = 2^{c_i - c_j} (do_i . v_j)
//   dk_j = 2^{c_T - c_j} R v_j + sum_{i >= j} D_ij q_i
//   dv_j = 2^{c_T - c_j} R^T k_j + sum_{i >= j} 2^{c_i - c_j} (q_i . k_j) do_i
//   R_prev = 2^{c_T} R + sum_i 2^{c_i} q_i do_i^T
// and dg_t is the sum over all pairs (i, j) with j < t <= i of their share of the loss, written
// without differences of large terms as
//   sum_{j < t <= i} D_ij (q_i . k_j)                    both in the chunk
//   + sum_{i >= t} 2^{c_i} q_i^T S do_i                  j before it
//   + sum_{j < t} 2^{c_T - c_j} k_j^T R v_j              i behind it
//   + 2^{c_T} <S, R>                                     both outside.
//
// Three phases of one cooperative launch (small calls, which are most of this path's, are bound by
// launches): each chunk's own sum of k v^T (and q do^T); a scan over a head's chunks, one thread for
// four elements of the state; each chunk's outputs or gradients.  The states between the phases cost
// 4 dk dv / T bytes per token each way; in exchange a single long sequence fills the device, where
// one CTA per head would leave it idle.  Measured in fp32: 1 x 2 x 256 tokens at d = 32 in 12 us on
// the device (launch latency and two grid barriers), the gradient at 2 x 4 x 333 tokens, 64 x 32, in
// 35 us (latency of a chunk's loops: 88 blocks).
#include <cooperative_groups.h>

#include <algorithm>

#include "gated.cuh"
#include "internal.h"
#include "per_device.h"

namespace la {
namespace {

constexpr int kT = 32;  // tokens per chunk: one warp holds a chunk's decays
constexpr int kThreads = 256;

struct Args {
  const void *q, *k, *v, *dout;
  const float *g;
  const int *lengths;
  void *out, *dq, *dk_, *dv_;
  float *dg;
  const float *S0, *dS;
  float *S, *dS0;
  float *buf, *rbuf;  // [BH][n][dk][dv] chunk sums, then the state before (rbuf: gradient behind) each chunk
  float *tot;         // [BH][n] log2 decay of each chunk
  int H, dk, dv;
  long N, n;
};

// Running sum of the log2 decays up to token `lane` of the chunk (tokens past the end decay by 1).
__device__ __forceinline__ Cum chunk_scan(const Args &a, long bh, long t0, int tv, int lane) {
  const float g = lane < tv ? a.g[bh * a.N + t0 + lane] : 0.f;
  const bool nan = __ballot_sync(0xffffffffu, isnan(g)) & (0xffffffffu >> (31 - lane));
  return split_cum(warp_scan(fixed_log2_decay(g), lane), nan);
}
__device__ __forceinline__ Cum last_lane(Cum c) {
  return Cum{__shfl_sync(0xffffffffu, c.hi, 31), __shfl_sync(0xffffffffu, c.lo, 31)};
}
__device__ __forceinline__ float decay_between(Cum from, Cum to) {
  return exp2f((to.hi - from.hi) + (to.lo - from.lo));
}

template <typename Tin>
__device__ __forceinline__ void load_rows(float *dst, int ld, const Tin *src, int d, int tv) {
  const int quads = d / 4;
  for (int e = threadIdx.x; e < kT * quads; e += kThreads) {
    const int t = e / quads, c = (e - t * quads) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < tv) x = ld4(src + (long)t * d + c);
    *reinterpret_cast<float4 *>(dst + t * ld + c) = x;
  }
}

// Chunk sums: blockIdx.z 0: sum_t 2^{c_T - c_t} k_t v_t^T; 1: sum_t 2^{c_t} q_t do_t^T.
template <typename Tin>
__device__ __forceinline__ void chunk_sums(const Args &a, float *sm, long item, bool rev) {
  const int dk = a.dk, dv = a.dv;
  float *A = sm, *B = A + kT * dk, *w = B + kT * dv;
  const long bh = item / a.n, ch = item - bh * a.n, t0 = ch * kT;
  const int tid = threadIdx.x;
  const long len = row_length(a.lengths, bh / a.H, a.N);
  if (t0 >= len) return;  // the scan stops before this chunk
  const int tv = (int)min((long)kT, len - t0);
  if (tid < 32) {
    const Cum c = chunk_scan(a, bh, t0, tv, tid), T = last_lane(c);
    w[tid] = rev ? exp2f(c.hi + c.lo) : decay_between(c, T);
    if (tid == 0 && !rev) a.tot[bh * a.n + ch] = T.hi + T.lo;
  }
  const long row = bh * a.N + t0;
  load_rows(A, dk, (const Tin *)(rev ? a.q : a.k) + row * dk, dk, tv);
  load_rows(B, dv, (const Tin *)(rev ? a.dout : a.v) + row * dv, dv, tv);
  __syncthreads();
  float *dst = (rev ? a.rbuf : a.buf) + (bh * a.n + ch) * (long)dk * dv;
  const int cq = dv / 4;
  for (int e = tid; e < (dk / 4) * cq; e += kThreads) {
    const int i = (e / cq) * 4, c = (e % cq) * 4;
    float acc[4][4] = {};
    for (int t = 0; t < tv; ++t) {
      const float4 x = *reinterpret_cast<const float4 *>(A + t * dk + i);
      const float4 y = *reinterpret_cast<const float4 *>(B + t * dv + c);
      const float wt = w[t], xs[4] = {x.x * wt, x.y * wt, x.z * wt, x.w * wt};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        acc[r][0] = fmaf(xs[r], y.x, acc[r][0]), acc[r][1] = fmaf(xs[r], y.y, acc[r][1]);
        acc[r][2] = fmaf(xs[r], y.z, acc[r][2]), acc[r][3] = fmaf(xs[r], y.w, acc[r][3]);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) st4(dst + (long)(i + r) * dv + c, acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  }
}

// Scan over a head's chunks, elements [e, e + 4) of head bh's state.  Forward: chunk sums -> state
// before each chunk, final state to S; rev: sums -> gradient of the state behind each chunk, initial
// state's gradient to dS0.
__device__ __forceinline__ void chunk_scan_states(const Args &a, long bh, long e, bool rev) {
  const long dd = (long)a.dk * a.dv;
  const long len = row_length(a.lengths, bh / a.H, a.N);
  const int n = (int)((len + kT - 1) / kT);
  const float *first = rev ? a.dS : a.S0;
  float4 s = first ? *reinterpret_cast<const float4 *>(first + bh * dd + e) : make_float4(0.f, 0.f, 0.f, 0.f);
  float *buf = (rev ? a.rbuf : a.buf) + bh * a.n * dd + e;
  const float *tot = a.tot + bh * a.n;
  constexpr int kAhead = 8;  // chunk sums in flight per thread
  for (int c0 = 0; c0 < n; c0 += kAhead) {
    float4 x[kAhead];
    float f[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (c0 + u < n) {
        const int c = rev ? n - 1 - (c0 + u) : c0 + u;
        x[u] = *reinterpret_cast<const float4 *>(buf + c * dd);
        f[u] = tot[c];
      }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (c0 + u < n) {
        const int c = rev ? n - 1 - (c0 + u) : c0 + u;
        *reinterpret_cast<float4 *>(buf + c * dd) = s;
        const float w = exp2f(f[u]);
        s = make_float4(fmaf(w, s.x, x[u].x), fmaf(w, s.y, x[u].y), fmaf(w, s.z, x[u].z), fmaf(w, s.w, x[u].w));
      }
  }
  float *last = rev ? a.dS0 : a.S;
  if (last) *reinterpret_cast<float4 *>(last + bh * dd + e) = s;
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}

// X[i][j] = (A_i . B_j) for a [kT x kT] tile, rows of d floats with stride ld.
__device__ __forceinline__ void tile_dots(float *X, const float *A, const float *B, int d, int ld) {
  const int i = threadIdx.x >> 3, j = threadIdx.x & 7;
  float s[4] = {};
  for (int x = 0; x < d; x += 4) {
    const float4 u = *reinterpret_cast<const float4 *>(A + i * ld + x);
#pragma unroll
    for (int m = 0; m < 4; ++m) s[m] = dot4(u, *reinterpret_cast<const float4 *>(B + (j + 8 * m) * ld + x), s[m]);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) X[i * (kT + 1) + j + 8 * m] = s[m];
}

// acc[r][m] += sum_x A[i + r][x] M[x][c + m] (M row-major in global memory).
__device__ __forceinline__ void rows_times(float (&acc)[4][4], const float *A, int ld, const float *M, int dx, int dm,
                                           int i, int c) {
  for (int x = 0; x < dx; ++x) {
    const float4 y = *reinterpret_cast<const float4 *>(M + (long)x * dm + c);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float u = A[(i + r) * ld + x];
      acc[r][0] = fmaf(u, y.x, acc[r][0]), acc[r][1] = fmaf(u, y.y, acc[r][1]);
      acc[r][2] = fmaf(u, y.z, acc[r][2]), acc[r][3] = fmaf(u, y.w, acc[r][3]);
    }
  }
}
// acc[r][m] += sum_c A[i + r][c] M[x + m][c].
__device__ __forceinline__ void rows_times_t(float (&acc)[4][4], const float *A, int ld, const float *M, int dc, int i,
                                             int x) {
  for (int c = 0; c < dc; c += 4) {
    float4 y[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) y[m] = *reinterpret_cast<const float4 *>(M + (long)(x + m) * dc + c);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float4 u = *reinterpret_cast<const float4 *>(A + (i + r) * ld + c);
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[r][m] = dot4(u, y[m], acc[r][m]);
    }
  }
}

template <typename Tin>
__device__ __forceinline__ void chunk_out(const Args &a, float *sm, long item) {
  const int dk = a.dk, dv = a.dv, lk = dk + 4;
  float *Q = sm, *K = Q + kT * lk, *V = K + kT * lk, *P = V + kT * dv;
  float *hi = P + kT * (kT + 1), *lo = hi + kT;
  const long bh = item / a.n, ch = item - bh * a.n, t0 = ch * kT;
  const int tid = threadIdx.x;
  const long len = row_length(a.lengths, bh / a.H, a.N);
  if (t0 >= len) return;
  const int tv = (int)min((long)kT, len - t0);
  if (tid < 32) {
    const Cum c = chunk_scan(a, bh, t0, tv, tid);
    hi[tid] = c.hi;
    lo[tid] = c.lo;
  }
  const long row = bh * a.N + t0;
  load_rows(Q, lk, (const Tin *)a.q + row * dk, dk, tv);
  load_rows(K, lk, (const Tin *)a.k + row * dk, dk, tv);
  load_rows(V, dv, (const Tin *)a.v + row * dv, dv, tv);
  __syncthreads();
  tile_dots(P, Q, K, dk, lk);
  __syncthreads();
  for (int e = tid; e < kT * kT; e += kThreads) {
    const int i = e / kT, j = e % kT;
    float *x = P + i * (kT + 1) + j;
    *x = j <= i ? *x * exp2f((hi[i] - hi[j]) + (lo[i] - lo[j])) : 0.f;
  }
  __syncthreads();
  const float *S = a.buf + (bh * a.n + ch) * (long)dk * dv;
  Tin *o = (Tin *)a.out + row * dv;
  const int cq = dv / 4;
  for (int e = tid; e < (kT / 4) * cq; e += kThreads) {
    const int i = (e / cq) * 4, c = (e % cq) * 4;
    float acc[4][4] = {};
    rows_times(acc, Q, lk, S, dk, dv, i, c);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = exp2f(hi[i + r] + lo[i + r]);
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[r][m] *= f;
    }
    rows_times(acc, P, kT + 1, V, kT, dv, i, c);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (i + r < tv) st4(o + (long)(i + r) * dv + c, acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  }
}

template <typename Tin>
__device__ __forceinline__ void chunk_grad(const Args &a, float *sm, long item) {
  const int dk = a.dk, dv = a.dv, lk = dk + 4, lv = dv + 4;
  float *Q = sm, *K = Q + kT * lk, *V = K + kT * lk, *dO = V + kT * lv;
  float *P = dO + kT * lv, *D = P + kT * (kT + 1), *M = D + kT * (kT + 1);
  float *hi = M + kT * (kT + 1), *lo = hi + kT, *ew = lo + kT;
  float *left = ew + kT, *right = left + kT * 33, *red = right + kT * 33;  // [kT][33] partial dots, [8] warp sums
  const long bh = item / a.n, ch = item - bh * a.n, t0 = ch * kT;
  const int tid = threadIdx.x, lane = tid & 31;
  const long len = row_length(a.lengths, bh / a.H, a.N);
  const int rows = (int)min((long)kT, a.N - t0);
  const int tv = (int)max(0L, min((long)kT, len - t0));
  const long row = bh * a.N + t0;
  Tin *dq = (Tin *)a.dq + row * dk, *dkp = (Tin *)a.dk_ + row * dk, *dvp = (Tin *)a.dv_ + row * dv;
  float *dg = a.dg + row;
  const int kq = dk / 4, vq = dv / 4;
  if (tv == 0) {  // padding only: zero gradients
    for (int e = tid; e < rows * kq; e += kThreads) st4(dq + 4 * (long)e, 0, 0, 0, 0), st4(dkp + 4 * (long)e, 0, 0, 0, 0);
    for (int e = tid; e < rows * vq; e += kThreads) st4(dvp + 4 * (long)e, 0, 0, 0, 0);
    if (tid < rows) dg[tid] = 0.f;
    return;
  }
  float total = 0.f;
  if (tid < 32) {
    const Cum c = chunk_scan(a, bh, t0, tv, tid), T = last_lane(c);
    hi[tid] = c.hi;
    lo[tid] = c.lo;
    ew[tid] = decay_between(c, T);
    total = exp2f(T.hi + T.lo);
  }
  load_rows(Q, lk, (const Tin *)a.q + row * dk, dk, tv);
  load_rows(K, lk, (const Tin *)a.k + row * dk, dk, tv);
  load_rows(V, lv, (const Tin *)a.v + row * dv, dv, tv);
  load_rows(dO, lv, (const Tin *)a.dout + row * dv, dv, tv);
  const long dd = (long)dk * dv;
  const float *S = a.buf + (bh * a.n + ch) * dd, *R = a.rbuf + (bh * a.n + ch) * dd;
  // <S, R>, in a fixed order
  float sr = 0.f;
  for (long e = tid * 4; e < dd; e += kThreads * 4)
    sr = dot4(*reinterpret_cast<const float4 *>(S + e), *reinterpret_cast<const float4 *>(R + e), sr);
  sr = warp_sum(sr);
  if (lane == 0) red[tid >> 5] = sr;
  __syncthreads();
  tile_dots(P, Q, K, dk, lk);
  tile_dots(D, dO, V, dv, lv);
  __syncthreads();
  for (int e = tid; e < kT * kT; e += kThreads) {
    const int i = e / kT, j = e % kT, x = i * (kT + 1) + j;
    const float w = j <= i ? exp2f((hi[i] - hi[j]) + (lo[i] - lo[j])) : 0.f;
    const float p = j <= i ? P[x] : 0.f, d = j <= i ? D[x] * w : 0.f;
    M[x] = j < i ? p * d : 0.f;
    P[x] = p * w;
    D[x] = d;
  }
  __syncthreads();

  // dq and the reads' share of the state before the chunk
  for (int e = tid; e < (kT / 4) * kq; e += kThreads) {
    const int i = (e / kq) * 4, x = (e % kq) * 4;
    float acc[4][4] = {};
    rows_times_t(acc, dO, lv, S, dv, i, x);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = exp2f(hi[i + r] + lo[i + r]);
      float s = 0.f;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        acc[r][m] *= f;
        s = fmaf(acc[r][m], Q[(i + r) * lk + x + m], s);
      }
      left[(i + r) * 33 + x / 4] = s;
    }
    rows_times(acc, D, kT + 1, K, kT, lk, i, x);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (i + r < rows) {
        const bool in = i + r < tv;  // padding rows: zero, whatever the states hold
        st4(dq + (long)(i + r) * dk + x, in ? acc[r][0] : 0.f, in ? acc[r][1] : 0.f, in ? acc[r][2] : 0.f,
            in ? acc[r][3] : 0.f);
      }
  }
  // dk and the keys' share of the gradient behind the chunk
  for (int e = tid; e < (kT / 4) * kq; e += kThreads) {
    const int j = (e / kq) * 4, x = (e % kq) * 4;
    float acc[4][4] = {};
    rows_times_t(acc, V, lv, R, dv, j, x);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float s = 0.f;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        acc[r][m] *= ew[j + r];
        s = fmaf(acc[r][m], K[(j + r) * lk + x + m], s);
      }
      right[(j + r) * 33 + x / 4] = s;
    }
    for (int i = 0; i < kT; ++i) {
      const float4 y = *reinterpret_cast<const float4 *>(Q + i * lk + x);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float u = D[i * (kT + 1) + j + r];
        acc[r][0] = fmaf(u, y.x, acc[r][0]), acc[r][1] = fmaf(u, y.y, acc[r][1]);
        acc[r][2] = fmaf(u, y.z, acc[r][2]), acc[r][3] = fmaf(u, y.w, acc[r][3]);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (j + r < rows) {
        const bool in = j + r < tv;
        st4(dkp + (long)(j + r) * dk + x, in ? acc[r][0] : 0.f, in ? acc[r][1] : 0.f, in ? acc[r][2] : 0.f,
            in ? acc[r][3] : 0.f);
      }
  }
  for (int e = tid; e < (kT / 4) * vq; e += kThreads) {
    const int j = (e / vq) * 4, c = (e % vq) * 4;
    float acc[4][4] = {};
    rows_times(acc, K, lk, R, dk, dv, j, c);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[r][m] *= ew[j + r];
    for (int i = 0; i < kT; ++i) {
      const float4 y = *reinterpret_cast<const float4 *>(dO + i * lv + c);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float u = P[i * (kT + 1) + j + r];
        acc[r][0] = fmaf(u, y.x, acc[r][0]), acc[r][1] = fmaf(u, y.y, acc[r][1]);
        acc[r][2] = fmaf(u, y.z, acc[r][2]), acc[r][3] = fmaf(u, y.w, acc[r][3]);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (j + r < rows) {
        const bool in = j + r < tv;
        st4(dvp + (long)(j + r) * dv + c, in ? acc[r][0] : 0.f, in ? acc[r][1] : 0.f, in ? acc[r][2] : 0.f,
            in ? acc[r][3] : 0.f);
      }
  }
  __syncthreads();
  if (tid < 32) {
    // what token `lane` adds to every dg_t with t <= lane, and with t > lane
    Sum2 ends{0.f, 0.f}, rgt{0.f, 0.f};
    for (int j = 0; j < kT; ++j) {
      ends.add(M[lane * (kT + 1) + j]);
      ends.add(-M[j * (kT + 1) + lane]);
    }
    for (int x = 0; x < kq; ++x) {
      ends.add(left[lane * 33 + x]);
      rgt.add(right[lane * 33 + x]);
    }
    float over = 0.f;
    for (int x = 0; x < kThreads / 32; ++x) over += red[x];
    Sum2 all = warp_scan_others<true>(ends, lane);
    const Sum2 upto = warp_scan_others<false>(rgt, lane);
    all.add(ends.s, ends.e);
    all.add(upto.s, upto.e);
    all.add(total * over);
    if (lane < rows) dg[lane] = lane < tv ? all.s + all.e : 0.f;
  }
}

template <typename Tin, bool kGrad>
__global__ void __launch_bounds__(kThreads) gated_simt_kernel(const __grid_constant__ Args a, long BH) {
  extern __shared__ float sm[];
  const cooperative_groups::grid_group grid = cooperative_groups::this_grid();
  const long items = BH * a.n;
  for (long x = blockIdx.x; x < items * (kGrad ? 2 : 1); x += gridDim.x) {
    chunk_sums<Tin>(a, sm, x % items, x >= items);
    __syncthreads();  // shared memory is free for the next chunk
  }
  grid.sync();
  const long quads = (long)a.dk * a.dv / 4, all = BH * quads;
  for (long x = (long)blockIdx.x * kThreads + threadIdx.x; x < all * (kGrad ? 2 : 1); x += (long)gridDim.x * kThreads) {
    const long y = x % all;
    chunk_scan_states(a, y / quads, (y % quads) * 4, x >= all);
  }
  grid.sync();
  for (long x = blockIdx.x; x < items; x += gridDim.x) {
    if (kGrad)
      chunk_grad<Tin>(a, sm, x);
    else
      chunk_out<Tin>(a, sm, x);
    __syncthreads();
  }
}

size_t state_floats(long BH, long N, int dk, int dv) { return (size_t)BH * ((N + kT - 1) / kT) * dk * dv; }

template <typename Tin, bool kGrad>
cudaError_t launch_t(Args a, long BH, cudaStream_t stream) {
  const int dk = a.dk, dv = a.dv;
  const size_t sm_sums = sizeof(float) * (kT * (dk + dv) + kT);
  const size_t sm_out = sizeof(float) * (2 * kT * (dk + 4) + kT * dv + kT * (kT + 1) + 2 * kT);
  const size_t sm_grad = sizeof(float) * (2 * kT * (dk + 4) + 2 * kT * (dv + 4) + 3 * kT * (kT + 1) + 3 * kT + 2 * kT * 33 + 8);
  const size_t smem = std::max(sm_sums, kGrad ? sm_grad : sm_out);
  const void *fn = (const void *)gated_simt_kernel<Tin, kGrad>;
  cudaError_t e = ensure_smem_optin(fn, (int)smem);
  if (e != cudaSuccess) return e;
  // blocks that fit on the device at once, looked up once per device and size
  static PerDeviceCache<size_t, int> fits;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const long room = fits.get(dev, smem, [&] {
    int per_sm = 0;
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, kThreads, smem);
    return std::max(1, per_sm) * std::max(1, device_info(dev).sm_count);
  });
  // enough blocks for the chunks and for the scan, all of them resident
  const long want = std::max(BH * a.n * (kGrad ? 2 : 1), BH * dk * dv / 4 * (kGrad ? 2 : 1) / kThreads);
  LaunchTimer timer(kGrad ? kKGatedBackward : kKGated, stream);
  void *args[] = {&a, &BH};
  e = cudaLaunchCooperativeKernel(fn, dim3((unsigned)std::max(1L, std::min(room, want))), dim3(kThreads), args, smem, stream);
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

Args make_args(const GatedProblem &p, bool grad) {
  Args a = {};
  a.q = p.q, a.k = p.k, a.v = p.v, a.g = p.g, a.lengths = p.lengths, a.out = p.out, a.S0 = p.S0, a.S = p.S;
  a.H = p.H, a.dk = p.dk, a.dv = p.dv, a.N = p.N, a.n = (p.N + kT - 1) / kT;
  a.buf = (float *)p.ws;
  float *end = a.buf + state_floats(p.BH(), p.N, p.dk, p.dv);
  if (grad) a.rbuf = end, end += state_floats(p.BH(), p.N, p.dk, p.dv);
  a.tot = end;
  return a;
}

}  // namespace

size_t gated_simt_workspace(long BH, long N, int dk, int dv, bool grad) {
  return sizeof(float) * (state_floats(BH, N, dk, dv) * (grad ? 2 : 1) + (size_t)BH * ((N + kT - 1) / kT));
}

cudaError_t launch_gated_simt(const GatedProblem &p) {
  const Args a = make_args(p, false);
  return p.dt == LA_F32 ? launch_t<float, false>(a, p.BH(), p.stream)
                        : launch_t<__nv_bfloat16, false>(a, p.BH(), p.stream);
}

cudaError_t launch_gated_grad_simt(const GatedGradProblem &b) {
  Args a = make_args(b.p, true);
  a.dout = b.dout, a.dS = b.dS, a.dq = b.dq, a.dk_ = b.dk, a.dv_ = b.dv, a.dg = b.dg, a.dS0 = b.dS0;
  a.S = nullptr;
  return b.p.dt == LA_F32 ? launch_t<float, true>(a, b.p.BH(), b.p.stream)
                          : launch_t<__nv_bfloat16, true>(a, b.p.BH(), b.p.stream);
}

}  // namespace la
