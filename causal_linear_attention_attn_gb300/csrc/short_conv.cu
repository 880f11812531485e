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
// rows are in flight.  HBM bounds it, x and y (gradient: x, dy, dx) once each, beside instruction issue: steps inside a
// run have no checks and no 64-bit products.  In bf16, K = 4: 4 x up to 8192 x 2048 forward in 42 us (4.5 TB/s), 4 x 8192 x
// 2048 of the gradient in 95 us (4.3 TB/s; with checks at every step 330).
//
// Column sums dw, db leave each run once and are added in a fixed order by a second kernel.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "vec8.cuh"

namespace la {

__device__ unsigned int g_conv_step_status;

namespace {

constexpr int kThreads = 256, kGradThreads = 128;
constexpr int kV = 4;      // channels a thread of the passes over tokens
constexpr int kAhead = 4;  // rows in flight a thread
// Blocks an SM, and threads an SM that the tokens are cut for.  The forward wants many short runs (its registers leave
// four blocks; 1024 threads an SM 52 us, 2048 47, 4096 42 at 4 x up to 8192 x 2048), the gradient one long run for
// each thread that is resident (128 registers; 512 threads 96 us, 1024 104, 2048 123; three blocks of more
// registers 122).
constexpr int kPerSm = 4, kCutThreads = 4096, kCutThreadsGrad = 512;
// A run of the gradient adds its tokens' shares of dweight and dbias one behind the other: at most so many, whatever the
// batch (a sum of thousands loses the low bits of every share).  Blocks that end early cost large batches less than runs
// of theirs that end late: in bf16, 16 x 8192 x 2048 and 64 x 8192 x 2048 take 359 and 1290 us, 368 and 1331 with 256
// tokens, 421 and 1360 with 1024, 421 and 1555 with no limit.
constexpr long kMostGrad = 512;

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
__global__ void __launch_bounds__(kThreads, kPerSm) short_conv_kernel(const __grid_constant__ ConvProblem p, int segs, int len) {
  constexpr int V = kV;
  const Run me(p, (long)blockIdx.x * kThreads + threadIdx.x, p.D / V, segs, len);
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
  const int count = (int)(me.t1 - me.t0);
  if (count <= 0) return;
  float2 w[K][V / 2], bias[V / 2], v[K][V / 2];
  load_weights<K, V>(p.weight, p.bias, c, w, bias);
#pragma unroll
  for (int i = 0; i < K - 1; ++i)
#pragma unroll
    for (int e = 0; e < V / 2; ++e) v[i][e] = win[i].pair(e);
  T *out = (T *)p.out + (me.b * p.N + me.t0) * p.D + c;
  x += me.t0 * p.ldx;
  Row<T, V> r[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (u < count) r[u].load(x + u * p.ldx);
  for (int i0 = 0; i0 < count; i0 += kAhead) {
    x += kAhead * p.ldx;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i0 + u < count) {
#pragma unroll
        for (int e = 0; e < V / 2; ++e) v[K - 1][e] = r[u].pair(e);
        if (i0 + u + kAhead < count) r[u].load(x + u * p.ldx);
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
        o.store(out + (long)u * p.D);
      }
    }
    out += (long)kAhead * p.D;
  }
}

template <typename T, int K>
__global__ void __launch_bounds__(kGradThreads, kPerSm)
    short_conv_grad_kernel(const __grid_constant__ ConvGradProblem q, int segs, int len, float *sums) {
  constexpr int V = kV, kRows = sizeof(T) == 4 ? 2 : kAhead;  // (fp32: four spill registers, 222 us for 155)
  const ConvProblem &p = q.p;
  const Run me(p, (long)blockIdx.x * kGradThreads + threadIdx.x, p.D / V, segs, len);
  if (!me.live) return;
  const long c = (long)me.g * V;
  const T *x = (const T *)p.x + me.b * p.N * p.ldx + c;
  T *dx = (T *)q.dx + me.b * p.N * p.D + c;
  const T *S0 = q.S0 ? (const T *)q.S0 + me.b * (K - 1) * p.D + c : nullptr;
  const T *dS = q.dS ? (const T *)q.dS + me.b * (K - 1) * p.D + c : nullptr;
  T *dS0 = q.dS0 ? (T *)q.dS0 + me.b * (K - 1) * p.D + c : nullptr;
  float2 dw[K][V / 2], db[V / 2];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    db[e] = both(0.f);
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j][e] = both(0.f);
  }
  const int count = (int)max(me.t1 - me.t0, 0L);
  if (count > 0 || (me.seg == 0 && dS0)) {
    float2 w[K][V / 2], bias[V / 2], v[K][V / 2], g[K][V / 2];
    load_weights<K, V>(p.weight, p.bias, c, w, bias);
#pragma unroll
    for (int e = 0; e < V / 2; ++e)
#pragma unroll
      for (int j = 0; j < K; ++j) g[j][e] = both(0.f);
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
    // Step i takes token t0 + i and completes row t0 + i - (K - 1) of dx, which lacks no later g.  The rows in front
    // of the first are the carried window's, and the K - 1 last steps only finish rows.
    const int steps = count + K - 1, there = (int)min(me.n - me.t0, (long)steps);
    const int carried = dS ? (int)min(me.n - me.t0, 0x3fffffffL) : 0x3fffffff;  // from that step on dS adds
    const T *xi = x + me.t0 * p.ldx, *yi = (const T *)q.dout + (me.b * p.N + me.t0) * p.D + c;
    T *o = dx + (me.t0 - (K - 1)) * p.D;
    Row<T, V> rx[kRows], ry[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      rx[u].zero(), ry[u].zero();
      if (u < there) rx[u].load(xi + u * p.ldx), ry[u].load(yi + (long)u * p.D);
    }
    // one step; kInside: nothing about it is special
    auto step = [&](auto inside, int i, int u) {
      constexpr bool kInside = decltype(inside)::value;
      float2 gg[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) v[K - 1][e] = rx[u].pair(e), gg[e] = ry[u].pair(e);
      if (i + kRows < there) {
        rx[u].load(xi + u * p.ldx), ry[u].load(yi + (long)u * p.D);
      } else if (!kInside) {
        rx[u].zero(), ry[u].zero();
      }
      Row<T, V> ds, to;
      if (!kInside) {
        ds.zero();
        if (i >= carried && i - carried < K - 1) ds.load(dS + (long)(i - carried) * p.D);
      }
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        if (p.silu) {
          float2 a = bias[e];
#pragma unroll
          for (int j = 0; j < K; ++j) a = __ffma2_rn(w[j][e], v[j][e], a);
          const Sigmoid2 sg(a);
          gg[e] = __fmul2_rn(gg[e], __ffma2_rn(__fmul2_rn(a, sg.s), sg.one_less(), sg.s));
        }
        if (!kInside && i >= there) gg[e] = both(0.f);  // nothing is there, and bias alone may not be finite
        if (kInside || i < count) {
#pragma unroll
          for (int j = 0; j < K; ++j) dw[j][e] = __ffma2_rn(gg[e], v[j][e], dw[j][e]);
          db[e] = __fadd2_rn(db[e], gg[e]);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) g[j][e] = g[j + 1][e], v[j][e] = v[j + 1][e];
        g[K - 1][e] = gg[e];
        float2 d = kInside ? both(0.f) : ds.pair(e);
#pragma unroll
        for (int j = 0; j < K; ++j) d = __ffma2_rn(w[j][e], g[K - 1 - j][e], d);
        to.set(e, d);
      }
      if (kInside || i >= K - 1)
        to.store(o + (long)u * p.D);
      else if (me.seg == 0 && dS0)
        to.store(dS0 + (long)i * p.D);
    };
    for (int i0 = 0; i0 < steps; i0 += kRows) {
      xi += kRows * p.ldx, yi += (long)kRows * p.D;
      if (i0 >= K - 1 && i0 + kRows <= min(count, carried)) {
#pragma unroll
        for (int u = 0; u < kRows; ++u) step(std::true_type{}, i0 + u, u);
      } else {
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (i0 + u < steps) step(std::false_type{}, i0 + u, u);
      }
      o += (long)kRows * p.D;
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

// Runs of tokens: at least kMinRun, so that the rows a run shares with its neighbours cost at most a fifth more reads, from
// L2 (the gradient, K - 1 rows of x on both sides and of dout behind: 9 for 32, 28 %); at most `most`.
constexpr int kMinRun = 16;
int run_length(const ConvProblem &p, int per_sm, long most) {
  const long threads = (long)std::max(1, device_info(-1).sm_count) * per_sm;
  const long len = ((long)p.B * (p.D / kV) * p.N + threads - 1) / threads;
  return (int)std::max<long>(kMinRun, std::min({len, p.N, most}));
}
int forward_run(const ConvProblem &p) { return run_length(p, kCutThreads, p.N); }
int gradient_run(const ConvProblem &p) { return run_length(p, kCutThreadsGrad, kMostGrad); }

template <typename T, int K>
cudaError_t launch_fwd(const ConvProblem &p) {
  const int len = forward_run(p), segs = (int)((p.N + len - 1) / len);
  const long units = (long)p.B * segs * (p.D / kV);
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
  const int len = gradient_run(p), segs = (int)((p.N + len - 1) / len);
  const long units = (long)p.B * segs * (p.D / kV);
  const bool sums = q.dweight || q.dbias;
  LaunchTimer timer(kKShortConvBackward, p.stream);
  short_conv_grad_kernel<T, K>
      <<<(unsigned)((units + kGradThreads - 1) / kGradThreads), kGradThreads, 0, p.stream>>>(q, segs, len, sums ? q.ws : nullptr);
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
  const int len = gradient_run(p);
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
