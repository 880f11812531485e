// Group norm of each head's channels with an affine map and a SiLU gate, and its gradient: the
// "gated normalization" that retention and its kin put in place of the denominator.
//
// Per token and head, over the d channels:  h = (x - mean) / sqrt(var + eps),
//   y = (h w + b) silu(gate),  silu(g) = g sigmoid(g).
// With u = dy silu(gate) w:
//   dx    = (u - mean(u) - h mean(u h)) / sqrt(var + eps)
//   dgate = dy (h w + b) sigmoid(g) (1 + g (1 - sigmoid(g)))
//   dw    = sum over tokens of dy silu(gate) h,   db = sum over tokens of dy silu(gate).
//
// x is the attention output's layout [B, H, N, d]; y, gate and their gradients are channels last
// [B, N, H d], the layout of the projections around the layer, so the transposition between the two
// costs no pass of its own.  HBM bounds it: every tensor is read or written once (the gradient
// recomputes the statistics instead of storing them).
//
// A thread owns eight channels of one head; the d/8 threads of a head meet in shuffles; the threads
// of a block cover up to 2048 channels of one token or the same channels of several tokens.  So
// channels-last rows move in runs of up to 4 KB, and every thread keeps its channels while the block
// walks over tokens: the column sums dw, db stay in registers until the block's end.  Each block
// writes its column sums once and a second kernel adds them in a fixed order (no atomics, so the
// gradient is the same from run to run).
#include <algorithm>

#include "gated.cuh"
#include "internal.h"

namespace la {
namespace {

constexpr int kMaxThreads = 256;

__device__ __forceinline__ void st8(float *p, const float (&o)[8]) {
  st4(p, o[0], o[1], o[2], o[3]);
  st4(p + 4, o[4], o[5], o[6], o[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16 *p, const float (&o)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t *>(&x);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over the aligned group of D / 8 lanes of one head.
template <int D>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// How a launch cuts [B * N tokens][H * d channels]: a block covers `heads` heads of `rows` tokens at
// a time (blockIdx.y: which heads) and walks over tokens with stride gridDim.x * rows.
struct Cut {
  int heads, rows, threads, slabs;
};
Cut make_cut(int H, int d) {
  Cut c;
  c.heads = std::min(H, kMaxThreads / (d / 8));
  c.slabs = (H + c.heads - 1) / c.heads;
  const int per_row = c.heads * (d / 8);
  c.rows = kMaxThreads / per_row;
  c.threads = (c.rows * per_row + 31) / 32 * 32;  // whole warps; the spare lanes idle
  return c;
}

template <int D>
struct Place {  // what a thread owns
  int h, c, row;
  bool live;
  __device__ Place(const Cut &cut, int H) {
    constexpr int kLanes = D / 8;
    const int grp = threadIdx.x / kLanes;
    row = grp / cut.heads;
    h = blockIdx.y * cut.heads + grp % cut.heads;
    c = (threadIdx.x % kLanes) * 8;
    live = row < cut.rows && h < H;
  }
};

template <int D>
__device__ __forceinline__ void normalize(float (&x)[8], float eps, float &rstd) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += x[e];
  const float mean = group_sum<D>(s) * (1.f / D);
  s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] -= mean;
    s = fmaf(x[e], x[e], s);
  }
  rstd = rsqrtf(group_sum<D>(s) * (1.f / D) + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= rstd;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + __expf(-x)); }

template <typename T, int D, int kRowsAhead>
__global__ void __launch_bounds__(kMaxThreads)
    group_norm_kernel(const __grid_constant__ NormProblem p, const __grid_constant__ Cut cut) {
  const Place<D> me(cut, p.H);
  const long tokens = (long)p.B * p.N, stride = (long)gridDim.x * cut.rows, HD = (long)p.H * D;
  float w[8], b[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 1.f, b[e] = 0.f;
  const long col = (long)me.h * D + me.c;
  if (me.live && p.weight) ld8(p.weight + col, w);
  if (me.live && p.bias) ld8(p.bias + col, b);
  // every lane of a warp runs the same number of turns: the shuffles need all of them
  for (long r0 = (long)blockIdx.x * cut.rows; r0 < tokens; r0 += kRowsAhead * stride) {
    float x[kRowsAhead][8], g[kRowsAhead][8];
    bool in[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const long r = r0 + u * stride + me.row;
      in[u] = me.live && r < tokens;
      if (in[u]) {
        const long bi = r / p.N, n = r - bi * p.N;
        ld8((const T *)p.x + ((bi * p.H + me.h) * p.N + n) * D + me.c, x[u]);
        if (p.gate) ld8((const T *)p.gate + r * HD + col, g[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      float rstd;
      normalize<D>(x[u], p.eps, rstd);
      if (!in[u]) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float y = fmaf(x[u][e], w[e], b[e]);
        if (p.gate) y *= g[u][e] * sigmoid(g[u][e]);
        x[u][e] = y;
      }
      st8((T *)p.y + (r0 + u * stride + me.row) * HD + col, x[u]);
    }
  }
}

template <typename T, int D, int kRowsAhead>
__global__ void __launch_bounds__(kMaxThreads)
    group_norm_grad_kernel(const __grid_constant__ NormGradProblem q, const __grid_constant__ Cut cut) {
  __shared__ float sums[kMaxThreads][16 + 1];
  const NormProblem &p = q.p;
  const Place<D> me(cut, p.H);
  const long tokens = (long)p.B * p.N, stride = (long)gridDim.x * cut.rows, HD = (long)p.H * D;
  float w[8], b[8], dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = 1.f, b[e] = dw[e] = db[e] = 0.f;
  const long col = (long)me.h * D + me.c;
  if (me.live && p.weight) ld8(p.weight + col, w);
  if (me.live && p.bias) ld8(p.bias + col, b);
  for (long r0 = (long)blockIdx.x * cut.rows; r0 < tokens; r0 += kRowsAhead * stride) {
    float x[kRowsAhead][8], g[kRowsAhead][8], dy[kRowsAhead][8];
    long at[kRowsAhead];
    bool in[kRowsAhead];
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      const long r = r0 + u * stride + me.row;
      in[u] = me.live && r < tokens;
      at[u] = 0;
      if (in[u]) {
        const long bi = r / p.N, n = r - bi * p.N;
        at[u] = ((bi * p.H + me.h) * p.N + n) * D + me.c;
        ld8((const T *)p.x + at[u], x[u]);
        ld8((const T *)q.dy + r * HD + col, dy[u]);
        if (p.gate) ld8((const T *)p.gate + r * HD + col, g[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[u][e] = dy[u][e] = g[u][e] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      float rstd, o[8];
      normalize<D>(x[u], p.eps, rstd);
      float su = 0.f, suh = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float t = dy[u][e];
        if (p.gate) {
          const float gg = g[u][e], sg = sigmoid(gg);
          o[e] = t * fmaf(x[u][e], w[e], b[e]) * sg * fmaf(gg, 1.f - sg, 1.f);
          t *= gg * sg;
        }
        dw[e] = fmaf(t, x[u][e], dw[e]);
        db[e] += t;
        t *= w[e];
        dy[u][e] = t;
        su += t;
        suh = fmaf(t, x[u][e], suh);
      }
      if (p.gate && in[u]) st8((T *)q.dgate + (r0 + u * stride + me.row) * HD + col, o);
      su = group_sum<D>(su) * (1.f / D);
      suh = group_sum<D>(suh) * (1.f / D);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = rstd * (dy[u][e] - su - x[u][e] * suh);
      if (in[u]) st8((T *)q.dx + at[u], o);
    }
  }
  if (!q.ws) return;
  // the block's column sums over its token rows, rows added in order
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = dw[e], sums[threadIdx.x][8 + e] = db[e];
  __syncthreads();
  if (me.live && me.row == 0) {
    const int per_row = cut.heads * (D / 8);
    for (int r = 1; r < cut.rows; ++r)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[e] += sums[threadIdx.x + r * per_row][e];
        db[e] += sums[threadIdx.x + r * per_row][8 + e];
      }
    float *dst = q.ws + (long)blockIdx.x * 2 * HD + col;
    st8(dst, dw);
    st8(dst + HD, db);
  }
}

// Column sums of the blocks' sums [blocks][2][HD], a warp per column pair set: thread = column.
__global__ void __launch_bounds__(128) norm_columns_kernel(const float *ws, int blocks, long HD, float *dw, float *db) {
  __shared__ float part[4][32];
  const long col = (long)blockIdx.x * 32 + (threadIdx.x & 31);
  const int grp = threadIdx.x >> 5;
  float s = 0.f;
  if (col < 2 * HD)
    for (int i = grp; i < blocks; i += 4) s += ws[(long)i * 2 * HD + col];
  part[grp][threadIdx.x & 31] = s;
  __syncthreads();
  if (grp == 0 && col < 2 * HD) {
    s = (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
    if (col < HD) {
      if (dw) dw[col] = s;
    } else if (db) {
      db[col - HD] = s;
    }
  }
}

// Blocks over the tokens: as many as fill the SMs at `per_sm` blocks each, no more than there are turns.
int token_blocks(const Cut &c, long tokens, int per_sm, int ahead) {
  const int sms = std::max(1, device_info(-1).sm_count);
  const long turns = (tokens + (long)c.rows * ahead - 1) / ((long)c.rows * ahead);
  return (int)std::max(1L, std::min<long>(turns, std::max(1, sms * per_sm / c.slabs)));
}

constexpr int kAheadFwd = 4, kAheadGrad = 2, kPerSmGrad = 4;

template <typename T, int D>
cudaError_t launch_fwd(const NormProblem &p) {
  const Cut c = make_cut(p.H, D);
  LaunchTimer timer(kKGroupNorm, p.stream);
  const dim3 grid((unsigned)token_blocks(c, (long)p.B * p.N, 1 << 20, kAheadFwd), (unsigned)c.slabs);
  group_norm_kernel<T, D, kAheadFwd><<<grid, c.threads, 0, p.stream>>>(p, c);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T, int D>
cudaError_t launch_grad(const NormGradProblem &q) {
  const NormProblem &p = q.p;
  const Cut c = make_cut(p.H, D);
  const int blocks = token_blocks(c, (long)p.B * p.N, kPerSmGrad, kAheadGrad);
  cudaError_t e;
  {
    LaunchTimer timer(kKGroupNormBackward, p.stream);
    group_norm_grad_kernel<T, D, kAheadGrad><<<dim3((unsigned)blocks, (unsigned)c.slabs), c.threads, 0, p.stream>>>(q, c);
    e = cudaGetLastError();
    timer.done(e);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  if (!q.ws) return e;
  const long HD = (long)p.H * D;
  LaunchTimer timer(kKGroupNormBackward, p.stream);
  norm_columns_kernel<<<(unsigned)((2 * HD + 31) / 32), 128, 0, p.stream>>>(q.ws, blocks, HD, q.dweight, q.dbias);
  e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t launch_group_norm(const NormProblem &p) {
  if (p.dt == LA_F32)
    return p.d == 32 ? launch_fwd<float, 32>(p) : p.d == 64 ? launch_fwd<float, 64>(p) : launch_fwd<float, 128>(p);
  return p.d == 32   ? launch_fwd<__nv_bfloat16, 32>(p)
         : p.d == 64 ? launch_fwd<__nv_bfloat16, 64>(p)
                     : launch_fwd<__nv_bfloat16, 128>(p);
}

size_t norm_grad_workspace(int B, int H, long N, int d) {
  const Cut c = make_cut(H, d);
  return sizeof(float) * 2 * (size_t)H * d * token_blocks(c, (long)B * N, kPerSmGrad, kAheadGrad);
}

cudaError_t launch_group_norm_grad(const NormGradProblem &q) {
  if (q.p.dt == LA_F32)
    return q.p.d == 32 ? launch_grad<float, 32>(q) : q.p.d == 64 ? launch_grad<float, 64>(q) : launch_grad<float, 128>(q);
  return q.p.d == 32   ? launch_grad<__nv_bfloat16, 32>(q)
         : q.p.d == 64 ? launch_grad<__nv_bfloat16, 64>(q)
                       : launch_grad<__nv_bfloat16, 128>(q);
}

}  // namespace la
