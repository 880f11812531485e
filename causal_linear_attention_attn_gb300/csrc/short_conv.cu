// Short causal convolution along the tokens, one window of K weights per channel, with a SiLU; its
// gradient; and its step for single tokens on a pool of windows.
//
//   u_t = bias + sum_{j<K} w_j x_{t-K+1+j},   y_t = silu(u_t) (or u_t),   x_{-K+1..-1} the carried window.
//   g_t = dy_t silu'(u_t),  dx_t = sum_j w_j g_{t+K-1-j},  dw_j = sum_t g_t x_{t-K+1+j},  db = sum_t g_t.
//
// Tokens are rows of D channels (channels last, the projections' layout), so neighbouring threads own
// neighbouring channels and walk down the rows of a run of tokens: the window (and, in the gradient, the
// last K values of g) stays in registers, every row is loaded once a run, plus K - 1 rows in front of it
// (which another thread reads too, so they come from L2) and, in the gradient, K - 1 behind it.  Four
// rows are in flight.  HBM bounds it: x and y (gradient: x, dy, dx) once each.
//
// Column sums dw, db leave each run once and are added in a fixed order by a second kernel.
#include <algorithm>

#include "internal.h"
#include "vec8.cuh"

namespace la {

__device__ unsigned int g_conv_step_status;

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // rows in flight a thread

// V consecutive channels as loaded.
template <typename T, int V>
struct Row {
  static constexpr int kBytes = V * (int)sizeof(T);
  uint32_t w[kBytes / 4];
  __device__ __forceinline__ void load(const T *p) {
    if (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
        w[(4 * i) % (kBytes / 4)] = v.x, w[(4 * i + 1) % (kBytes / 4)] = v.y;
        w[(4 * i + 2) % (kBytes / 4)] = v.z, w[(4 * i + 3) % (kBytes / 4)] = v.w;
      }
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if (kBytes == 8) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[(4 * i) % (kBytes / 4)], w[(4 * i + 1) % (kBytes / 4)],
                                                     w[(4 * i + 2) % (kBytes / 4)], w[(4 * i + 3) % (kBytes / 4)]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kBytes / 4; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float2 pair(int e) const {
    return sizeof(T) == 2
               ? make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u))
               : make_float2(__uint_as_float(w[(2 * e) % (kBytes / 4)]), __uint_as_float(w[(2 * e + 1) % (kBytes / 4)]));
  }
  __device__ __forceinline__ void set(int e, float2 v) {
    if (sizeof(T) == 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
      w[e] = *reinterpret_cast<const uint32_t *>(&h);
    } else {
      w[(2 * e) % (kBytes / 4)] = __float_as_uint(v.x), w[(2 * e + 1) % (kBytes / 4)] = __float_as_uint(v.y);
    }
  }
};

// The weights of V channels, [V][K] in memory, as pairs of channels per tap.
template <int K, int V>
__device__ __forceinline__ void load_weights(const float *weight, const float *bias, long c, float2 (&w)[K][V / 2],
                                             float2 (&b)[V / 2]) {
  float f[K * V];
#pragma unroll
  for (int i = 0; i < K * V; i += 4) {
    const float4 v = *reinterpret_cast<const float4 *>(weight + c * K + i);
    f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
  }
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
#pragma unroll
    for (int j = 0; j < K; ++j) w[j][e] = make_float2(f[2 * e * K + j], f[(2 * e + 1) * K + j]);
    b[e] = bias ? *reinterpret_cast<const float2 *>(bias + c + 2 * e) : both(0.f);
  }
}

// A thread's channels and run of tokens.
struct Run {
  long b, n;
  long t0, t1, tN;  // its tokens that count, and the end of its rows
  int seg, g;
  bool live;
  __device__ Run(const ConvProblem &p, long unit, int groups, int segs, int len) {
    g = (int)(unit % groups);
    const long r = unit / groups;
    seg = (int)(r % segs);
    b = r / segs;
    live = b < p.B;
    if (!live) b = 0;
    n = row_length(p.lengths, b, p.N);
    t0 = (long)seg * len;
    tN = min(t0 + len, p.N);
    t1 = min(tN, n);
  }
};

template <typename T, int K>
__global__ void __launch_bounds__(kThreads) short_conv_kernel(const __grid_constant__ ConvProblem p, int segs, int len) {
  constexpr int V = 8;
  const int groups = p.D / V;
  const Run me(p, (long)blockIdx.x * kThreads + threadIdx.x, groups, segs, len);
  if (!me.live || (me.t0 >= me.n && me.seg > 0)) return;
  const long c = (long)me.g * V;
  const T *x = (const T *)p.x + me.b * p.N * p.ldx + c;
  T *S = (T *)p.S + me.b * (K - 1) * p.D + c;
  Row<T, V> win[K - 1];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const long t = me.t0 - (K - 1) + i;
    win[i].zero();
    if (t >= 0)
      win[i].load(x + t * p.ldx);
    else if (p.from_state)
      win[i].load(S + (t + K - 1) * p.D);
  }
  if (me.seg == 0) {  // the window to carry on, written by the thread that has read the one in its place
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const long t = me.n - (K - 1) + i;
      Row<T, V> r;
      if (t >= 0) {
        r.load(x + t * p.ldx);
      } else {
        r = win[0];
#pragma unroll
        for (int o = 1; o < K - 1; ++o)
          if (t + K - 1 == o) r = win[o];
      }
      r.store(S + i * p.D);
    }
  }
  if (me.t0 >= me.t1) return;
  float2 w[K][V / 2], bias[V / 2], v[K][V / 2];
  load_weights<K, V>(p.weight, p.bias, c, w, bias);
#pragma unroll
  for (int i = 0; i < K - 1; ++i)
#pragma unroll
    for (int e = 0; e < V / 2; ++e) v[i][e] = win[i].pair(e);
  T *out = (T *)p.out + me.b * p.N * p.D + c;
  Row<T, V> r[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (me.t0 + u < me.t1) r[u].load(x + (me.t0 + u) * p.ldx);
  for (long t = me.t0; t < me.t1; t += kAhead) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (t + u >= me.t1) break;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) v[K - 1][e] = r[u].pair(e);
      if (t + u + kAhead < me.t1) r[u].load(x + (t + u + kAhead) * p.ldx);
      Row<T, V> o;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        float2 a = bias[e];
#pragma unroll
        for (int j = 0; j < K; ++j) a = __ffma2_rn(w[j][e], v[j][e], a);
        if (p.silu) a = __fmul2_rn(a, Sigmoid2(a).s);
        o.set(e, a);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) v[j][e] = v[j + 1][e];
      }
      o.store(out + (t + u) * p.D);
    }
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(kThreads)
    short_conv_grad_kernel(const __grid_constant__ ConvGradProblem q, int segs, int len, float *sums) {
  constexpr int V = 4;
  const ConvProblem &p = q.p;
  const int groups = p.D / V;
  const Run me(p, (long)blockIdx.x * kThreads + threadIdx.x, groups, segs, len);
  if (!me.live) return;
  const long c = (long)me.g * V;
  const T *x = (const T *)p.x + me.b * p.N * p.ldx + c;
  const T *dy = (const T *)q.dout + me.b * p.N * p.D + c;
  T *dx = (T *)q.dx + me.b * p.N * p.D + c;
  const T *S0 = q.S0 ? (const T *)q.S0 + me.b * (K - 1) * p.D + c : nullptr;
  const T *dS = q.dS ? (const T *)q.dS + me.b * (K - 1) * p.D + c : nullptr;
  T *dS0 = q.dS0 ? (T *)q.dS0 + me.b * (K - 1) * p.D + c : nullptr;
  float2 w[K][V / 2], bias[V / 2], v[K][V / 2], g[K][V / 2], dw[K][V / 2], db[V / 2];
  load_weights<K, V>(p.weight, p.bias, c, w, bias);
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    db[e] = both(0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = g[j][e] = both(0.f);
  }
  if (me.t0 < me.t1 || (me.seg == 0 && dS0)) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const long t = me.t0 - (K - 1) + i;
      Row<T, V> r;
      r.zero();
      if (t >= 0)
        r.load(x + t * p.ldx);
      else if (S0)
        r.load(S0 + (t + K - 1) * p.D);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) v[i][e] = r.pair(e);
    }
    Row<T, V> rx[kAhead], ry[kAhead];
    auto load = [&](int u, long t) {
      rx[u].zero(), ry[u].zero();
      if (t < me.n) rx[u].load(x + t * p.ldx), ry[u].load(dy + t * p.D);
    };
    // row t of dx is complete with g of token t + K - 1; rows in front of the first are the carried window's
    const long end = max(me.t1, me.t0) + K - 1;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) load(u, me.t0 + u);
    for (long s0 = me.t0; s0 < end; s0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const long s = s0 + u, t = s - (K - 1);
        if (s >= end) break;
        float2 dyv[V / 2];
#pragma unroll
        for (int e = 0; e < V / 2; ++e) v[K - 1][e] = rx[u].pair(e), dyv[e] = ry[u].pair(e);
        load(u, s + kAhead < end ? s + kAhead : me.n);
        const bool put = t >= me.t0 || (me.seg == 0 && (t >= 0 || dS0));
        Row<T, V> o, ds;
        ds.zero();
        const long from_end = t - (me.n - (K - 1));  // the window that the call carries on gives its gradient
        if (dS && put && from_end >= 0 && from_end < K - 1) ds.load(dS + from_end * p.D);
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
          float2 gg = dyv[e];
          if (p.silu) {
            float2 a = bias[e];
#pragma unroll
            for (int j = 0; j < K; ++j) a = __ffma2_rn(w[j][e], v[j][e], a);
            const Sigmoid2 sg(a);
            gg = __fmul2_rn(gg, __ffma2_rn(__fmul2_rn(a, sg.s), sg.one_less(), sg.s));
          }
          if (s >= me.n) gg = both(0.f);  // nothing is there, and bias alone may not be finite
          if (s < me.t1) {
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][e] = __ffma2_rn(gg, v[j][e], dw[j][e]);
            db[e] = __fadd2_rn(db[e], gg);
          }
#pragma unroll
          for (int j = 0; j < K - 1; ++j) g[j][e] = g[j + 1][e], v[j][e] = v[j + 1][e];
          g[K - 1][e] = gg;
          float2 d = ds.pair(e);
#pragma unroll
          for (int j = 0; j < K; ++j) d = __ffma2_rn(w[j][e], g[K - 1 - j][e], d);
          o.set(e, d);
        }
        if (put) o.store(t >= 0 ? dx + t * p.D : dS0 + (t + K - 1) * p.D);
      }
    }
  }
  Row<T, V> none;
  none.zero();
  for (long t = max(me.t0, me.n); t < me.tN; ++t) none.store(dx + t * p.D);
  if (!sums) return;
  float *to = sums + (me.b * segs + me.seg) * (K + 1) * p.D + c;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    const float2 a = j < K ? dw[j % K][0] : db[0], b = j < K ? dw[j % K][1] : db[1];
    st4(to + (long)j * p.D, a.x, a.y, b.x, b.y);
  }
}

// One token a row on the window of its slot: a block a row, a thread eight channels.
template <typename T, int K>
__global__ void __launch_bounds__(kThreads) short_conv_step_kernel(const __grid_constant__ ConvStepProblem p, int per_row) {
  constexpr int V = 8;
  const int b = blockIdx.x / per_row, part = blockIdx.x - b * per_row;
  const int slot = p.slots ? p.slots[b] : b;
  const bool bad = slot < 0 || slot >= p.n_slots;
  int again = 0;
  if (p.slots && !bad)
    for (int o = threadIdx.x; o < b; o += kThreads) again |= p.slots[o] == slot;
  const long c = ((long)part * kThreads + threadIdx.x) * V;
  const bool live = c < p.D;
  Row<T, V> r[K];
  T *S = bad ? nullptr : (T *)p.S + (long)slot * (K - 1) * p.D + c;
  if (live && !bad) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) r[i].load(S + (long)i * p.D);
    r[K - 1].load((const T *)p.x + (long)b * p.ldx + c);
  }
  const bool skip = __syncthreads_or(again) || bad;
  if (skip && slot >= 0 && threadIdx.x == 0) atomicOr(&g_conv_step_status, kStatusBadSlot);
  if (!live) return;
  Row<T, V> o;
  o.zero();
  if (!skip) {
    float2 w[K][V / 2], bias[V / 2];
    load_weights<K, V>(p.weight, p.bias, c, w, bias);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
      float2 a = bias[e];
#pragma unroll
      for (int j = 0; j < K; ++j) a = __ffma2_rn(w[j][e], r[j].pair(e), a);
      if (p.silu) a = __fmul2_rn(a, Sigmoid2(a).s);
      o.set(e, a);
    }
#pragma unroll
    for (int i = 0; i < K - 1; ++i) r[i + 1].store(S + (long)i * p.D);
  }
  o.store((T *)p.out + (long)b * p.D + c);
}

// Runs of tokens: enough threads to fill the SMs (1024 each), but at least kMinRun tokens a run, whose
// K - 1 extra rows then cost at most a fifth more reads, from L2.
constexpr int kMinRun = 16;
int run_length(const ConvProblem &p, int v) {
  const long threads = (long)std::max(1, device_info(-1).sm_count) * 1024;
  const long len = ((long)p.B * (p.D / v) * p.N + threads - 1) / threads;
  return (int)std::max<long>(kMinRun, std::min<long>(len, p.N));
}

template <typename T, int K>
cudaError_t launch_fwd(const ConvProblem &p) {
  const int len = run_length(p, 8), segs = (int)((p.N + len - 1) / len);
  const long units = (long)p.B * segs * (p.D / 8);
  LaunchTimer timer(kKShortConv, p.stream);
  short_conv_kernel<T, K><<<(unsigned)((units + kThreads - 1) / kThreads), kThreads, 0, p.stream>>>(p, segs, len);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T, int K>
cudaError_t launch_grad(const ConvGradProblem &q) {
  const ConvProblem &p = q.p;
  const int len = run_length(p, 4), segs = (int)((p.N + len - 1) / len);
  const long units = (long)p.B * segs * (p.D / 4);
  const bool sums = q.dweight || q.dbias;
  LaunchTimer timer(kKShortConvBackward, p.stream);
  short_conv_grad_kernel<T, K>
      <<<(unsigned)((units + kThreads - 1) / kThreads), kThreads, 0, p.stream>>>(q, segs, len, sums ? q.ws : nullptr);
  cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e != cudaSuccess) return e;
  count_launch();
  if (!sums) return e;
  ColumnSums s{q.ws, (long)p.B * segs, (long)(K + 1) * p.D, {}};
  s.part[0] = {q.dweight, (long)K * p.D, K};
  s.part[1] = {q.dbias, (long)(K + 1) * p.D, 1};
  s.part[2] = {nullptr, (long)(K + 1) * p.D, 1};
  return launch_column_sums(s, kKShortConvBackward, p.stream);
}

template <typename T, int K>
cudaError_t launch_step(const ConvStepProblem &p) {
  LaunchTimer timer(kKShortConvStep, p.stream);
  const int per_row = (p.D / 8 + kThreads - 1) / kThreads;
  short_conv_step_kernel<T, K><<<(unsigned)((long)per_row * p.B), kThreads, 0, p.stream>>>(p, per_row);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

cudaError_t launch_short_conv(const ConvProblem &p) {
  if (p.dt == LA_F32)
    return p.K == 2 ? launch_fwd<float, 2>(p) : p.K == 3 ? launch_fwd<float, 3>(p) : launch_fwd<float, 4>(p);
  return p.K == 2   ? launch_fwd<__nv_bfloat16, 2>(p)
         : p.K == 3 ? launch_fwd<__nv_bfloat16, 3>(p)
                    : launch_fwd<__nv_bfloat16, 4>(p);
}

size_t short_conv_grad_workspace(const ConvProblem &p) {
  const int len = run_length(p, 4);
  return sizeof(float) * (size_t)p.B * ((p.N + len - 1) / len) * (p.K + 1) * p.D;
}

cudaError_t launch_short_conv_grad(const ConvGradProblem &q) {
  const int K = q.p.K;
  if (q.p.dt == LA_F32)
    return K == 2 ? launch_grad<float, 2>(q) : K == 3 ? launch_grad<float, 3>(q) : launch_grad<float, 4>(q);
  return K == 2   ? launch_grad<__nv_bfloat16, 2>(q)
         : K == 3 ? launch_grad<__nv_bfloat16, 3>(q)
                  : launch_grad<__nv_bfloat16, 4>(q);
}

cudaError_t launch_short_conv_step(const ConvStepProblem &p) {
  if (p.dt == LA_F32)
    return p.K == 2 ? launch_step<float, 2>(p) : p.K == 3 ? launch_step<float, 3>(p) : launch_step<float, 4>(p);
  return p.K == 2   ? launch_step<__nv_bfloat16, 2>(p)
         : p.K == 3 ? launch_step<__nv_bfloat16, 3>(p)
                    : launch_step<__nv_bfloat16, 4>(p);
}

cudaError_t read_and_clear_conv_step_status(unsigned int *value) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, g_conv_step_status, sizeof(unsigned int));
  if (e == cudaSuccess && *value) e = cudaMemcpyToSymbol(g_conv_step_status, &zero, sizeof(unsigned int));
  return e;
}

}  // namespace la
