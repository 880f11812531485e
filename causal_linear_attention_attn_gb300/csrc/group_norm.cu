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
// Two rows a thread are in flight, each loaded again as soon as its values are taken.  Measured in bf16
// with gate and affine map, d = 128: 4 x 16 x 8192 tokens forward in 65 us (6.2 TB/s), 4 x 16 x 4096
// tokens of the gradient in 73 us (4.6 TB/s); loads and use in turns took 77 and 78, other numbers of
// rows and of blocks an SM 66 to 120 and 72 to 105 (three rows in the gradient: fp32 69 to 87), the
// affine map read again for each row 83.
//
// A thread owns eight channels of one head; the d/8 threads of a head meet in shuffles; the threads
// of a block cover up to 2048 channels of one token or the same channels of several tokens.  So
// channels-last rows move in runs of up to 4 KB, and every thread keeps its channels while the block
// walks over tokens: the column sums dw, db stay in registers until the block's end.  Each block
// writes its column sums once and, behind a grid barrier (a cooperative launch: the blocks are resident
// anyway), they are added in a fixed order: no atomics, so the gradient is the same from run to run.
#include <cooperative_groups.h>

#include <algorithm>

#include "gated.cuh"
#include "internal.h"
#include "vec8.cuh"

namespace la {
namespace {

constexpr int kMaxThreads = 256;
// rows in flight a thread, blocks an SM
constexpr int kAheadFwd = 2, kPerSmFwd = 4, kAheadGrad = 2, kPerSmGrad = 2;

// Sum over the aligned group of D / 8 lanes of one head.
template <int D>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// How a launch cuts [B * N tokens][H * d channels]: a block covers `heads` heads of `rows` tokens at
// a time (a slab of heads), two such groups of consecutive tokens in flight.
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
  __device__ Place(const Cut &cut, int H, int slab) {
    constexpr int kLanes = D / 8;
    const int grp = threadIdx.x / kLanes;
    row = grp / cut.heads;
    h = slab * cut.heads + grp % cut.heads;
    c = (threadIdx.x % kLanes) * 8;
    live = row < cut.rows && h < H;
  }
};

__device__ __forceinline__ float sum8(const float2 (&x)[4]) {
  const float2 s = __fadd2_rn(__fadd2_rn(x[0], x[1]), __fadd2_rn(x[2], x[3]));
  return s.x + s.y;
}
__device__ __forceinline__ float dot8(const float2 (&x)[4], const float2 (&y)[4]) {
  const float2 s = __ffma2_rn(x[0], y[0], __ffma2_rn(x[1], y[1], __ffma2_rn(x[2], y[2], __fmul2_rn(x[3], y[3]))));
  return s.x + s.y;
}

// x - mean over the head, scaled to unit variance: the mean first, then the squared deviations (one
// pass with the mean of the squares would cancel for rows far from zero).
template <int D>
__device__ __forceinline__ float normalize(float2 (&x)[4], float eps) {
  const float mean = group_sum<D>(sum8(x)) * (1.f / D);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __fadd2_rn(x[e], both(-mean));
  const float rstd = rsqrtf(group_sum<D>(dot8(x, x)) * (1.f / D) + eps);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __fmul2_rn(x[e], both(rstd));
  return rstd;
}

// Quotients by N of numbers below 2^31 (round-up multiplier; add and shift).
struct Divider {
  uint32_t n, mul, shift;
  __device__ uint32_t of(uint32_t x) const { return (__umulhi(x, mul) + x) >> shift; }
};
Divider make_divider(uint32_t n) {
  Divider d{n, 0, 0};
  while ((1ull << d.shift) < n) ++d.shift;
  d.mul = (uint32_t)(((1ull << 32) * ((1ull << d.shift) - n)) / n + 1);
  return d;
}

template <typename T, int D, bool kGate, int kRowsAhead>
__global__ void __launch_bounds__(kMaxThreads, kPerSmFwd)
    group_norm_kernel(const __grid_constant__ NormProblem p, const __grid_constant__ Cut cut,
                      const __grid_constant__ Divider by_n) {
  const uint32_t tokens = (uint32_t)((long)p.B * p.N);
  const long HD = (long)p.H * D;
  const Place<D> me(cut, p.H, blockIdx.y);
  const long col = (long)me.h * D + me.c;
  float2 w[4], b[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = both(1.f), b[e] = both(0.f);
  if (me.live && p.weight) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = reinterpret_cast<const float2 *>(p.weight + col)[e];
  }
  if (me.live && p.bias) {
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = reinterpret_cast<const float2 *>(p.bias + col)[e];
  }
  const long step = (long)gridDim.x * cut.rows * kRowsAhead;
  Raw<T> x[kRowsAhead], g[kRowsAhead];
  auto load = [&](int u, long r) {
    x[u].zero();
    if (me.live && r < tokens) {
      const uint32_t bi = by_n.of((uint32_t)r), n = (uint32_t)r - bi * by_n.n;
      x[u].load((const T *)p.x + (((long)bi * p.H + me.h) * p.N + n) * D + me.c);
      if (kGate) g[u].load((const T *)p.gate + r * HD + col);
    }
  };
  long r0 = (long)blockIdx.x * cut.rows * kRowsAhead;
#pragma unroll
  for (int u = 0; u < kRowsAhead; ++u) load(u, r0 + u * cut.rows + me.row);
  // every lane of a warp runs the same number of turns: the shuffles need all of them
  for (; r0 < tokens; r0 += step) {
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) {
      float2 y[4], t[4];
      x[u].get(y);
      if (kGate) g[u].get(t);
      const long r = r0 + u * cut.rows + me.row;
      load(u, r + step);
      normalize<D>(y, p.eps);
      if (!(me.live && r < tokens)) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = __ffma2_rn(y[e], w[e], b[e]);
      if (kGate) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = __fmul2_rn(y[e], __fmul2_rn(t[e], Sigmoid2(t[e]).s));
      }
      put8((T *)p.y + r * HD + col, y);
    }
  }
}

template <typename T, int D, bool kGate, int kRowsAhead>
__global__ void __launch_bounds__(kMaxThreads, kPerSmGrad)
    group_norm_grad_kernel(const __grid_constant__ NormGradProblem q, const __grid_constant__ Cut cut,
                           const __grid_constant__ Divider by_n) {
  __shared__ float sums[kMaxThreads][16 + 1];
  const NormProblem &p = q.p;
  const uint32_t tokens = (uint32_t)((long)p.B * p.N);
  const long HD = (long)p.H * D;
  for (int slab = blockIdx.y; slab < cut.slabs; slab += gridDim.y) {
    const Place<D> me(cut, p.H, slab);
    const long col = (long)me.h * D + me.c;
    float2 w[4], b[4], dw[4], db[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = both(1.f), b[e] = dw[e] = db[e] = both(0.f);
    if (me.live && p.weight) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = reinterpret_cast<const float2 *>(p.weight + col)[e];
    }
    if (me.live && p.bias) {
#pragma unroll
      for (int e = 0; e < 4; ++e) b[e] = reinterpret_cast<const float2 *>(p.bias + col)[e];
    }
    const long step = (long)gridDim.x * cut.rows * kRowsAhead;
    Raw<T> x[kRowsAhead], g[kRowsAhead], dy[kRowsAhead];
    auto load = [&](int u, long r) {
      x[u].zero(), dy[u].zero(), g[u].zero();
      if (me.live && r < tokens) {
        const uint32_t bi = by_n.of((uint32_t)r), n = (uint32_t)r - bi * by_n.n;
        x[u].load((const T *)p.x + (((long)bi * p.H + me.h) * p.N + n) * D + me.c);
        dy[u].load((const T *)q.dy + r * HD + col);
        if (kGate) g[u].load((const T *)p.gate + r * HD + col);
      }
    };
    long r0 = (long)blockIdx.x * cut.rows * kRowsAhead;
#pragma unroll
    for (int u = 0; u < kRowsAhead; ++u) load(u, r0 + u * cut.rows + me.row);
    for (; r0 < tokens; r0 += step) {
#pragma unroll
      for (int u = 0; u < kRowsAhead; ++u) {
        const long r = r0 + u * cut.rows + me.row;
        const bool in = me.live && r < tokens;
        float2 h[4], t[4], gg[4];
        x[u].get(h);
        dy[u].get(t);
        if (kGate) g[u].get(gg);
        load(u, r + step);
        const float rstd = normalize<D>(h, p.eps);
        if (kGate) {
          float2 o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const Sigmoid2 sg(gg[e]);
            const float2 silu = __fmul2_rn(gg[e], sg.s);
            const float2 ds = __ffma2_rn(silu, sg.one_less(), sg.s);  // silu' = s + silu (1 - s)
            o[e] = __fmul2_rn(__fmul2_rn(t[e], __ffma2_rn(h[e], w[e], b[e])), ds);
            t[e] = __fmul2_rn(t[e], silu);
          }
          if (in) put8((T *)q.dgate + r * HD + col, o);
        }
        if (in) {  // (past the last token h is 0 / 0 when eps is 0)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dw[e] = __ffma2_rn(t[e], h[e], dw[e]);
            db[e] = __fadd2_rn(db[e], t[e]);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = __fmul2_rn(t[e], w[e]);
        const float su = group_sum<D>(sum8(t)) * (-1.f / D), suh = group_sum<D>(dot8(t, h)) * (-1.f / D);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = __fmul2_rn(__fadd2_rn(__ffma2_rn(h[e], both(suh), t[e]), both(su)), both(rstd));
        if (in) {
          const uint32_t bi = by_n.of((uint32_t)r), n = (uint32_t)r - bi * by_n.n;
          put8((T *)q.dx + (((long)bi * p.H + me.h) * p.N + n) * D + me.c, t);
        }
      }
    }
    if (!q.ws) continue;
    // the block's column sums over its token rows, rows added in order
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sums[threadIdx.x][2 * e] = dw[e].x, sums[threadIdx.x][2 * e + 1] = dw[e].y;
      sums[threadIdx.x][8 + 2 * e] = db[e].x, sums[threadIdx.x][9 + 2 * e] = db[e].y;
    }
    __syncthreads();
    if (me.live && me.row == 0) {
      const int per_row = cut.heads * (D / 8);
      float o[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] = sums[threadIdx.x][e];
      for (int r = 1; r < cut.rows; ++r)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] += sums[threadIdx.x + r * per_row][e];
      float *dst = q.ws + (long)blockIdx.x * 2 * HD + col;
#pragma unroll
      for (int e = 0; e < 16; e += 4) st4(dst + (e >> 3) * HD + (e & 7), o[e], o[e + 1], o[e + 2], o[e + 3]);
    }
    __syncthreads();  // the sums' place is free for the next slab
  }
  if (!q.ws) return;
  cooperative_groups::this_grid().sync();
  // 32 columns a turn, a warp for every eighth row of blocks
  const int warps = blockDim.x / 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long flat = (long)blockIdx.y * gridDim.x + blockIdx.x, all = (long)gridDim.x * gridDim.y;
  for (long c0 = flat * 32; c0 < 2 * HD; c0 += all * 32) {
    const long c = c0 + lane;
    float s = 0.f;
    if (c < 2 * HD)
      for (int i = warp; i < (int)gridDim.x; i += warps) s += __ldcg(q.ws + (long)i * 2 * HD + c);
    __syncthreads();
    (&sums[0][0])[threadIdx.x] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * HD) {
      for (int w2 = 1; w2 < warps; ++w2) s += (&sums[0][0])[w2 * 32 + lane];
      if (c < HD) {
        if (q.dweight) q.dweight[c] = s;
      } else if (q.dbias) {
        q.dbias[c - HD] = s;
      }
    }
  }
}

// Blocks over the tokens: as many as fill the SMs at `per_sm` blocks each, no more than there are turns.
int token_blocks(const Cut &c, long tokens, int per_sm, int ahead) {
  const int sms = std::max(1, device_info(-1).sm_count);
  const long turns = (tokens + (long)c.rows * ahead - 1) / ((long)c.rows * ahead);
  return (int)std::max(1L, std::min<long>(turns, std::max(1, sms * per_sm / c.slabs)));
}

template <typename T, int D>
cudaError_t launch_fwd(const NormProblem &p) {
  const Cut c = make_cut(p.H, D);
  LaunchTimer timer(kKGroupNorm, p.stream);
  const dim3 grid((unsigned)token_blocks(c, (long)p.B * p.N, kPerSmFwd, kAheadFwd), (unsigned)c.slabs);
  const Divider by_n = make_divider((uint32_t)p.N);
  if (p.gate)
    group_norm_kernel<T, D, true, kAheadFwd><<<grid, c.threads, 0, p.stream>>>(p, c, by_n);
  else
    group_norm_kernel<T, D, false, kAheadFwd><<<grid, c.threads, 0, p.stream>>>(p, c, by_n);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T, int D>
cudaError_t launch_grad(const NormGradProblem &q) {
  const NormProblem &p = q.p;
  const Cut c = make_cut(p.H, D);
  const Divider by_n = make_divider((uint32_t)p.N);
  const int sms = std::max(1, device_info(-1).sm_count);
  const dim3 grid((unsigned)token_blocks(c, (long)p.B * p.N, kPerSmGrad, kAheadGrad),
                  (unsigned)std::min(c.slabs, sms * kPerSmGrad));
  const void *fn = p.gate ? (const void *)group_norm_grad_kernel<T, D, true, kAheadGrad>
                          : (const void *)group_norm_grad_kernel<T, D, false, kAheadGrad>;
  LaunchTimer timer(kKGroupNormBackward, p.stream);
  void *args[] = {const_cast<NormGradProblem *>(&q), const_cast<Cut *>(&c), const_cast<Divider *>(&by_n)};
  cudaError_t e;
  if (q.ws)  // column sums: a grid barrier; all blocks are resident (kPerSmGrad an SM)
    e = cudaLaunchCooperativeKernel(fn, grid, dim3(c.threads), args, 0, p.stream);
  else
    e = cudaLaunchKernel(fn, grid, dim3(c.threads), args, 0, p.stream);
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
