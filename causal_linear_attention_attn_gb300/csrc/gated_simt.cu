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
// Three phases of one cooperative launch (small calls are bound by launches; heads of one chunk need
// no barrier and no scan): each chunk's own sum of k v^T (and q do^T); a scan over a head's chunks,
// one thread for an element of the state; each chunk's outputs or gradients.  The states between the
// phases cost 4 dk dv / T bytes per token each way; in exchange a single long sequence fills the
// device, where one CTA per head would leave it idle.  Measured in fp32, whole calls: 2 x 4 x 4096
// tokens at d = 64 in 71 us and the gradient in 161 us (shared-memory reads of the products),
// 1 x 1 x 16384 in 69 and 121 us (the scan's rounds of loads), 4 x 4 x 300 in 24 and 50 us (latency
// of a chunk's loops).
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
  float *tot;         // [BH][n] decay over each chunk
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

// Chunk sums: sum_t 2^{c_T - c_t} k_t v_t^T; rev: sum_t 2^{c_t} q_t do_t^T.
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
    if (tid == 0 && !rev) a.tot[bh * a.n + ch] = exp2f(T.hi + T.lo);
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

// Scan over a head's chunks, element e of head bh's state.  Forward: chunk sums -> state before each
// chunk, final state to S; rev: sums -> gradient of the state behind each chunk, initial state's
// gradient to dS0.  One element a thread and 32 chunks in flight: with few heads the chain of loads is
// what this phase costs.
__device__ __forceinline__ void chunk_scan_states(const Args &a, long bh, long e, bool rev) {
  const long dd = (long)a.dk * a.dv;
  const long len = row_length(a.lengths, bh / a.H, a.N);
  const int n = (int)((len + kT - 1) / kT);
  const float *first = rev ? a.dS : a.S0;
  float s = first ? first[bh * dd + e] : 0.f;
  const long step = rev ? -dd : dd;
  const int dt = rev ? -1 : 1;
  float *at = (rev ? a.rbuf : a.buf) + (bh * a.n + (rev ? n - 1 : 0)) * dd + e;
  const float *tot = a.tot + bh * a.n + (rev ? n - 1 : 0);
  constexpr int kAhead = 32;  // chunks in flight: 4096 tokens at d = 64 take 69 us; 16 71, factors not ahead 90
  for (int c0 = 0; c0 < n; c0 += kAhead) {
    float x[kAhead], f[kAhead];
    const float *src = at;
#pragma unroll
    for (int u = 0; u < kAhead; ++u, src += step)
      if (c0 + u < n) x[u] = *src, f[u] = tot[u * dt];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (c0 + u < n) {
        *at = s;
        s = f[u] == 0.f ? x[u] : fmaf(f[u], s, x[u]);
        at += step;
      }
    tot += kAhead * dt;
  }
  float *last = rev ? a.dS0 : a.S;
  if (last) last[bh * dd + e] = s;
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float s) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}

constexpr int kTp = kT + 4;  // row stride of a [kT x kT] tile: whole float4s

// X[i][j] = (A_i . B_j) for a [kT x kT] tile, rows of d floats with stride ld.
__device__ __forceinline__ void tile_dots(float *X, const float *A, const float *B, int d, int ld) {
  const int i = threadIdx.x >> 3, j = threadIdx.x & 7;
  float s[4] = {};
#pragma unroll 2
  for (int x = 0; x < d; x += 4) {
    const float4 u = *reinterpret_cast<const float4 *>(A + i * ld + x);
#pragma unroll
    for (int m = 0; m < 4; ++m) s[m] = dot4(u, *reinterpret_cast<const float4 *>(B + (j + 8 * m) * ld + x), s[m]);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) X[i * kTp + j + 8 * m] = s[m];
}

__device__ __forceinline__ void fma4(float (&acc)[4], float u, float4 y) {
  acc[0] = fmaf(u, y.x, acc[0]), acc[1] = fmaf(u, y.y, acc[1]), acc[2] = fmaf(u, y.z, acc[2]), acc[3] = fmaf(u, y.w, acc[3]);
}
__device__ __forceinline__ void scale(float (&acc)[4], float f) {  // across a cut: nothing, not even a NaN
#pragma unroll
  for (int m = 0; m < 4; ++m) acc[m] = f == 0.f ? 0.f : acc[m] * f;
}

// acc[r][m] += sum_x A[i + r][x] M[x][c + m], four x at a time (dx a multiple of 4).
__device__ __forceinline__ void rows_times(float (&acc)[4][4], const float *A, int ld, const float *M, int dx, int ldm,
                                           int i, int c) {
#pragma unroll 4
  for (int x = 0; x < dx; x += 4) {
    float4 y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = *reinterpret_cast<const float4 *>(M + (long)(x + e) * ldm + c);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float4 u = *reinterpret_cast<const float4 *>(A + (i + r) * ld + x);
      fma4(acc[r], u.x, y[0]), fma4(acc[r], u.y, y[1]), fma4(acc[r], u.z, y[2]), fma4(acc[r], u.w, y[3]);
    }
  }
}
// acc[r][m] += sum_c A[i + r][c] M[x + m][c].
__device__ __forceinline__ void rows_times_t(float (&acc)[4][4], const float *A, int ld, const float *M, int dc, int ldm,
                                             int i, int x) {
#pragma unroll 2
  for (int c = 0; c < dc; c += 4) {
    float4 y[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) y[m] = *reinterpret_cast<const float4 *>(M + (x + m) * ldm + c);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float4 u = *reinterpret_cast<const float4 *>(A + (i + r) * ld + c);
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[r][m] = dot4(u, y[m], acc[r][m]);
    }
  }
}
// acc[r][m] += sum_i A[i][j + r] M[i][c + m] over the tile's kT rows.
__device__ __forceinline__ void cols_times(float (&acc)[4][4], const float *A, const float *M, int ldm, int j, int c) {
#pragma unroll 4
  for (int i = 0; i < kT; ++i) {
    const float4 u = *reinterpret_cast<const float4 *>(A + i * kTp + j);
    const float4 y = *reinterpret_cast<const float4 *>(M + i * ldm + c);
    fma4(acc[0], u.x, y), fma4(acc[1], u.y, y), fma4(acc[2], u.z, y), fma4(acc[3], u.w, y);
  }
}

// S: the state before the chunk (null: zero).
template <typename Tin>
__device__ __forceinline__ void chunk_out(const Args &a, float *sm, long item, const float *S) {
  const int dk = a.dk, dv = a.dv, lk = dk + 4;
  float *Q = sm, *K = Q + kT * lk, *V = K + kT * lk, *P = V + kT * dv;
  float *hi = P + kT * kTp, *lo = hi + kT;
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
    float *x = P + i * kTp + j;
    *x = j <= i ? *x * exp2f((hi[i] - hi[j]) + (lo[i] - lo[j])) : 0.f;
  }
  __syncthreads();
  Tin *o = (Tin *)a.out + row * dv;
  const int cq = dv / 4;
  for (int e = tid; e < (kT / 4) * cq; e += kThreads) {
    const int i = (e / cq) * 4, c = (e % cq) * 4;
    float acc[4][4] = {};
    if (S) rows_times(acc, Q, lk, S, dk, dv, i, c);
#pragma unroll
    for (int r = 0; r < 4; ++r) scale(acc[r], exp2f(hi[i + r] + lo[i + r]));
    rows_times(acc, P, kTp, V, kT, dv, i, c);
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (i + r < tv) st4(o + (long)(i + r) * dv + c, acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
  }
}

// S, R: the state before the chunk and the gradient behind it (null: zero).
template <typename Tin>
__device__ __forceinline__ void chunk_grad(const Args &a, float *sm, long item, const float *S, const float *R) {
  const int dk = a.dk, dv = a.dv, lk = dk + 4, lv = dv + 4;
  float *Q = sm, *K = Q + kT * lk, *V = K + kT * lk, *dO = V + kT * lv;
  float *P = dO + kT * lv, *D = P + kT * kTp, *M = D + kT * kTp;  // M: [kT][kT + 1]
  float *hi = M + kT * (kT + 1), *lo = hi + kT, *ew = lo + kT;
  float *left = ew + kT, *right = left + kT * 33, *red = right + kT * 33;  // [kT][33] partial dots, [8] warp sums
  float *St = red + 8;  // [dk][lv] the state before the chunk, then the gradient behind it
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
#pragma unroll 4
  for (int e = tid; e < dk * vq; e += kThreads) {
    const int x = e / vq, c = (e - x * vq) * 4;
    *reinterpret_cast<float4 *>(St + x * lv + c) =
        S ? *reinterpret_cast<const float4 *>(S + (long)e * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  tile_dots(P, Q, K, dk, lk);
  tile_dots(D, dO, V, dv, lv);
  __syncthreads();
  for (int e = tid; e < kT * kT; e += kThreads) {
    const int i = e / kT, j = e % kT, x = i * kTp + j;
    const float w = j <= i ? exp2f((hi[i] - hi[j]) + (lo[i] - lo[j])) : 0.f;
    const float p = j <= i ? P[x] : 0.f, d = j <= i ? D[x] * w : 0.f;
    P[x] = p * w;
    D[x] = d;
    // M[i][t]: the query's sum over the keys before t (a warp has a row)
    float m = j < i ? p * d : 0.f;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, m, o);
      if (j >= o) m += y;
    }
    M[i * (kT + 1) + j + 1] = m;
    if (j == 0) M[i * (kT + 1)] = 0.f;
  }
  __syncthreads();

  auto put = [&](Tin *dst, int t, int col, int d, const float (&acc)[4][4]) {  // padding rows: zero, whatever the states hold
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (t + r < rows) {
        const bool in = t + r < tv;
        st4(dst + (long)(t + r) * d + col, in ? acc[r][0] : 0.f, in ? acc[r][1] : 0.f, in ? acc[r][2] : 0.f, in ? acc[r][3] : 0.f);
      }
  };
  // dq and the reads' share of the state before the chunk
  for (int e = tid; e < (kT / 4) * kq; e += kThreads) {
    const int i = (e / kq) * 4, x = (e % kq) * 4;
    float acc[4][4] = {};
    rows_times_t(acc, dO, lv, St, dv, lv, i, x);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      scale(acc[r], exp2f(hi[i + r] + lo[i + r]));
      left[(i + r) * 33 + x / 4] = dot4(make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]),
                                        *reinterpret_cast<const float4 *>(Q + (i + r) * lk + x), 0.f);
    }
    rows_times(acc, D, kTp, K, kT, lk, i, x);
    put(dq, i, x, dk, acc);
  }
  __syncthreads();
  // the gradient behind the chunk takes the state's place; <S, R> on the way, in a fixed order
  float sr = 0.f;
#pragma unroll 4
  for (int e = tid; e < dk * vq; e += kThreads) {
    const int x = e / vq, c = (e - x * vq) * 4;
    float4 *at = reinterpret_cast<float4 *>(St + x * lv + c);
    const float4 y = R ? *reinterpret_cast<const float4 *>(R + (long)e * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    sr = dot4(*at, y, sr);
    *at = y;
  }
  sr = warp_sum(sr);
  if (lane == 0) red[tid >> 5] = sr;
  __syncthreads();
  // dk and the keys' share of the gradient behind the chunk; dv
  const int nk = (kT / 4) * kq, nv = (kT / 4) * vq;
  for (int e = tid; e < nk + nv; e += kThreads) {
    float acc[4][4] = {};
    if (e < nk) {
      const int j = (e / kq) * 4, x = (e % kq) * 4;
      rows_times_t(acc, V, lv, St, dv, lv, j, x);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        scale(acc[r], ew[j + r]);
        right[(j + r) * 33 + x / 4] = dot4(make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]),
                                           *reinterpret_cast<const float4 *>(K + (j + r) * lk + x), 0.f);
      }
      cols_times(acc, D, Q, lk, j, x);
      put(dkp, j, x, dk, acc);
    } else {
      const int j = ((e - nk) / vq) * 4, c = ((e - nk) % vq) * 4;
      rows_times(acc, K, lk, St, dk, lv, j, c);
#pragma unroll
      for (int r = 0; r < 4; ++r) scale(acc[r], ew[j + r]);
      cols_times(acc, P, dO, lv, j, c);
      put(dvp, j, c, dv, acc);
    }
  }
  __syncthreads();
  if (tid < 32) {
    // pairs in the chunk on both sides of token `lane`: keys before it (summed above), queries from it on
    // (row sums less column sums, added from the end, would cancel all pairs behind it)
    float in = 0.f;
#pragma unroll
    for (int i = 0; i < kT; ++i) in += i >= lane ? M[i * (kT + 1) + lane] : 0.f;
    // what token `lane` adds to every dg_t with t <= lane, and with t > lane
    Sum2 ends{0.f, 0.f}, rgt{0.f, 0.f};
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
    all.add(total == 0.f ? 0.f : total * over);
    all.add(in);
    if (lane < rows) dg[lane] = lane < tv ? all.s + all.e : 0.f;
  }
}

// Two blocks an SM, 128 registers a thread (the prefill spills 4 bytes): the gradient took 170 us at
// 2 x 4 x 4096, d = 64, where one block and all its registers took 220.
template <typename Tin, bool kGrad>
__global__ void __launch_bounds__(kThreads, 2) gated_simt_kernel(const __grid_constant__ Args a, long BH) {
  extern __shared__ float sm[];
  const long items = BH * a.n, dd = (long)a.dk * a.dv;
  if (a.n == 1) {
    // one chunk a head: its CTA has all it needs, and nothing waits for another.  The gradient of
    // 1 x 2 x 30 tokens takes 25 us this way, with the barriers 31 us.
    for (long bh = blockIdx.x; bh < BH; bh += gridDim.x) {
      const bool rows = row_length(a.lengths, bh / a.H, a.N) > 0;
      const float *S0 = a.S0 ? a.S0 + bh * dd : nullptr, *dS = a.dS ? a.dS + bh * dd : nullptr;
      float *sum = (kGrad ? a.rbuf : a.buf) + bh * dd, *last = kGrad ? a.dS0 : a.S;
      chunk_sums<Tin>(a, sm, bh, false);
      __syncthreads();
      if (kGrad) {
        chunk_sums<Tin>(a, sm, bh, true);
        __syncthreads();
        chunk_grad<Tin>(a, sm, bh, S0, dS);
      } else {
        chunk_out<Tin>(a, sm, bh, S0);
      }
      __syncthreads();  // the initial state is read: the result may take its place
      if (last) {
        const float *first = kGrad ? dS : S0;
        const float f = rows ? a.tot[bh] : 1.f;
        for (long e = threadIdx.x; e < dd; e += kThreads)
          last[bh * dd + e] = fmaf(f, first && f != 0.f ? first[e] : 0.f, rows ? sum[e] : 0.f);
      }
    }
    return;
  }
  const cooperative_groups::grid_group grid = cooperative_groups::this_grid();
  for (long x = blockIdx.x; x < items * (kGrad ? 2 : 1); x += gridDim.x) {
    chunk_sums<Tin>(a, sm, x % items, x >= items);
    __syncthreads();  // shared memory is free for the next chunk
  }
  grid.sync();
  const long all = BH * dd;
  for (long x = (long)blockIdx.x * kThreads + threadIdx.x; x < all * (kGrad ? 2 : 1); x += (long)gridDim.x * kThreads) {
    const long y = x % all;
    chunk_scan_states(a, y / dd, y % dd, x >= all);
  }
  grid.sync();
  for (long x = blockIdx.x; x < items; x += gridDim.x) {
    if (kGrad)
      chunk_grad<Tin>(a, sm, x, a.buf + x * dd, a.rbuf + x * dd);
    else
      chunk_out<Tin>(a, sm, x, a.buf + x * dd);
    __syncthreads();
  }
}

size_t state_floats(long BH, long N, int dk, int dv) { return (size_t)BH * ((N + kT - 1) / kT) * dk * dv; }

template <typename Tin, bool kGrad>
cudaError_t launch_t(Args a, long BH, cudaStream_t stream) {
  const int dk = a.dk, dv = a.dv;
  const size_t sm_sums = sizeof(float) * (kT * (dk + dv) + kT);
  const size_t sm_out = sizeof(float) * (2 * kT * (dk + 4) + kT * dv + kT * kTp + 2 * kT);
  const size_t sm_grad = sizeof(float) * (2 * kT * (dk + 4) + 2 * kT * (dv + 4) + 2 * kT * kTp + kT * (kT + 1) + 3 * kT +
                                          2 * kT * 33 + 8 + (size_t)dk * (dv + 4));
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
  const long want = std::max(BH * a.n * (kGrad ? 2 : 1), BH * dk * dv * (kGrad ? 2 : 1) / kThreads);
  LaunchTimer timer(kGrad ? kKGatedBackward : kKGated, stream);
  void *args[] = {&a, &BH};
  if (a.n == 1)
    e = cudaLaunchKernel(fn, dim3((unsigned)BH), dim3(kThreads), args, smem, stream);
  else
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
