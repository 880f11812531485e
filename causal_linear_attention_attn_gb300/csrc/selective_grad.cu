// Gradient of the selective state space scan.
//
// With a_t = e^{delta_t A}, dy = dout silu(z) and G_t the gradient of h_t (formulas of the forward in selective.cuh):
//   G_t = C_t dy_t + a_{t+1} G_{t+1},  behind the last token G = dS
//   dC_t,n = sum_c h dy,  dB_t,n = sum_c G delta x,  s1 = sum_n G B_n,  s2 = sum_n G (a h_{t-1}) A_n
//   dx = D dy + delta s1,  ddt = (x s1 + s2) softplus'(dt + bias),  dz = dout y silu'(z)
//   dA_n = sum_{b,t} G (a h_{t-1}) delta,  dD = sum dy x,  dbias = sum ddt,  dS0 = a_0 G_0.
//
// The states are not kept by the forward: a pass of the scan leaves the state in front of every chunk, and
// this kernel goes through the chunks from the last to the first.  In each it runs the recurrence again, with
// the scan's layout (a lane: four components of a channel), keeping a_t h_{t-1} of the chunk's tokens in shared
// memory (16 bytes a lane and token, read back by the lane that wrote it), then walks back with G in registers.
// Sums over the components are spread over a channel's lanes; the sums of dB and dC over channels are
// spread over a warp's channels, added over the block's warps, and leave as one partial sum a block of 32
// channels, which a last kernel adds in order.  No atomics: the gradient is the same from run to run.
//
// Three exponentials and about twenty issue slots a component, channel and token bound it.
#include <algorithm>

#include "internal.h"
#include "selective.cuh"

namespace la {
namespace {

constexpr int kCols = 32;        // channels a block
constexpr int kRow = kCols + 8;  // floats between tokens of the sums' places

// Tokens a chunk: a h of a token takes 128 ds bytes of shared memory, and two blocks an SM fit (ds = 64: one).
constexpr int chunk_tokens(int ds) { return ds <= 16 ? 32 : ds == 32 ? 16 : 8; }

template <int DS>
struct Smem {
  static constexpr int kTok = chunk_tokens(DS), kThreads = 8 * DS;
  float4 ah[kTok][kThreads];
  float2 steps[kTok][kCols];  // delta; delta x
  float dy[kTok][kCols];
  float B[kTok][DS], C[kTok][DS];
  float s1[kTok][kRow], s2[kTok][kRow], y[kTok][kRow];
  float bc[kTok][kThreads / 32][2 * DS];  // dB, dC of each warp's channels
};

template <typename T, int DS, bool kGate>
__global__ void __launch_bounds__(8 * DS) scan_grad_kernel(const __grid_constant__ ScanGradProblem g, const __grid_constant__ ScanSplit s) {
  constexpr int kThreads = 8 * DS, kLanes = DS / 4, kPerWarp = 32 / kLanes, kTok = Smem<DS>::kTok;
  constexpr int kGroups = (kTok * 4 + kThreads - 1) / kThreads;
  constexpr int kStep = kLanes < 4 ? 4 : kLanes > kTok ? kTok : kLanes;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Smem<DS> &m = *reinterpret_cast<Smem<DS> *>(raw_smem);
  const ScanProblem &p = g.p;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = (p.D + kCols - 1) / kCols;
  const int cb = blockIdx.x % nb;
  const long rest = blockIdx.x / nb;
  const int seg = (int)(rest % s.segs);
  const long b = rest / s.segs;
  const long n = row_length(p.lengths, b, p.N);
  const long begin = (long)seg * s.len, stop = min(begin + s.len, p.N), end = min(stop, n);

  const int q = lane % kLanes, num = lane / kLanes, ch = warp * kPerWarp + num;
  const int c = cb * kCols + ch;
  const long at = (long)c * DS + 4 * q, state = (long)p.D * DS;
  const bool mine = c < p.D;
  float2 A[2] = {both(0.f), both(0.f)}, G[2] = {both(0.f), both(0.f)}, dA[2] = {both(0.f), both(0.f)};
  if (mine) {
    const float4 a = *reinterpret_cast<const float4 *>(p.A + at);
    A[0] = __fmul2_rn(make_float2(a.x, a.y), both(kLog2e)), A[1] = __fmul2_rn(make_float2(a.z, a.w), both(kLog2e));
    const float *from = s.segs > 1 ? s.rev_starts + (b * s.segs + seg) * state : g.dS ? g.dS + b * state : nullptr;
    if (from) {
      const float4 v = *reinterpret_cast<const float4 *>(from + at);
      G[0] = make_float2(v.x, v.y), G[1] = make_float2(v.z, v.w);
    }
  }

  const int c8 = cb * kCols + (tid & 3) * 8;
  const bool live = c8 < p.D;
  float2 bias[4], skip[4], dD[4], dbias[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bias[e] = live && p.dt_bias ? reinterpret_cast<const float2 *>(p.dt_bias + c8)[e] : both(0.f);
    skip[e] = live && p.Dskip ? reinterpret_cast<const float2 *>(p.Dskip + c8)[e] : both(0.f);
    dD[e] = dbias[e] = both(0.f);
  }
  const T *x = (const T *)p.x + b * p.N * p.ldx + c8, *dt = (const T *)p.delta + b * p.N * p.ldt + c8;
  const T *z = kGate ? (const T *)p.z + b * p.N * p.ldz + c8 : nullptr;
  const T *dout = (const T *)g.dout + b * p.N * p.D + c8;
  const long out0 = b * p.N * p.D + c8;
  // tokens past the row's end: zero gradients
  for (long i = tid; i < (stop - max(begin, end)) * 4; i += kThreads) {
    const long o = out0 + (max(begin, end) + (i >> 2)) * p.D;
    const float2 zero[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
    if (!live) break;
    put8((T *)g.dx + o, zero), put8((T *)g.ddt + o, zero);
    if (kGate) put8((T *)g.dz + o, zero);
  }

  Raw<T> rx[kGroups], rt[kGroups], rz[kGate ? kGroups : 1], rd[kGroups], rb;
  constexpr int kPieces = kTok * DS / 8, kPerRow = DS / 8;
  const bool with_c = tid >= kPieces;
  const int piece = with_c ? tid - kPieces : tid, brow = piece / kPerRow, bcol = piece % kPerRow * 8;
  const bool has_bc = tid < 2 * kPieces;
  const T *bc = with_c ? (const T *)p.Cm + b * p.N * p.ldc + bcol : (const T *)p.Bm + b * p.N * p.ldb + bcol;
  const long ldbc = with_c ? p.ldc : p.ldb;
  float4 h0 = make_float4(0.f, 0.f, 0.f, 0.f);
  auto load = [&](long t0) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int k = tid + i * kThreads;
      const long t = t0 + (k >> 2);
      rx[i].zero(), rt[i].zero(), rd[i].zero();
      if (kGate) rz[i].zero();
      if (k < kTok * 4 && live && t < end) {
        rx[i].load(x + t * p.ldx), rt[i].load(dt + t * p.ldt), rd[i].load(dout + t * p.D);
        if (kGate) rz[i].load(z + t * p.ldz);
      }
    }
    rb.zero();
    if (has_bc && t0 + brow < end) rb.load(bc + (t0 + brow) * ldbc);
    if (mine) h0 = *reinterpret_cast<const float4 *>(s.chunk_states + (b * s.all_chunks + t0 / kTok) * state + at);
  };
  const long chunks = end > begin ? (end - begin + kTok - 1) / kTok : 0;
  if (chunks) load(begin + (chunks - 1) * kTok);
  for (long k = chunks - 1; k >= 0; --k) {
    const long t0 = begin + k * kTok;
    Raw<T> kx[kGroups], kt[kGroups], kz[kGate ? kGroups : 1], kd[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int j = tid + i * kThreads;
      if (j >= kTok * 4) break;
      const bool in = t0 + (j >> 2) < end;
      kx[i] = rx[i], kt[i] = rt[i], kd[i] = rd[i];
      float2 xv[4], tv[4], dv[4], zv[4];
      rx[i].get(xv), rt[i].get(tv), rd[i].get(dv);
      if (kGate) kz[i] = rz[i], rz[i].get(zv);
      const int row = j >> 2, col = (tid & 3) * 8;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 d = __fadd2_rn(tv[e], bias[e]);
        if (p.softplus) d = softplus2(d);
        float2 u = __fmul2_rn(d, xv[e]);
        if (!in) d = u = both(0.f);
        reinterpret_cast<float4 *>(&m.steps[row][col])[e] = make_float4(d.x, u.x, d.y, u.y);
        if (kGate) dv[e] = __fmul2_rn(dv[e], __fmul2_rn(zv[e], Sigmoid2(zv[e]).s));
        reinterpret_cast<float2 *>(&m.dy[row][col])[e] = in ? dv[e] : both(0.f);
      }
    }
    if (has_bc) {
      float2 v[4];
      rb.get(v);
      put8(with_c ? &m.C[brow][bcol] : &m.B[brow][bcol], v);
    }
    float2 h[2] = {make_float2(h0.x, h0.y), make_float2(h0.z, h0.w)};
    if (k > 0) load(t0 - kTok);
    __syncthreads();
    // the chunk's states again
#pragma unroll 1
    for (int i0 = 0; i0 < kTok; i0 += kStep) {
      float y[kStep];
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const int i = i0 + j;
        const float2 d = m.steps[i][ch];
        const float4 bv = *reinterpret_cast<const float4 *>(&m.B[i][4 * q]);
        const float2 a0 = __fmul2_rn(exp2_approx(__fmul2_rn(both(d.x), A[0])), h[0]);
        const float2 a1 = __fmul2_rn(exp2_approx(__fmul2_rn(both(d.x), A[1])), h[1]);
        m.ah[i][tid] = make_float4(a0.x, a0.y, a1.x, a1.y);
        h[0] = __ffma2_rn(both(d.y), make_float2(bv.x, bv.y), a0);
        h[1] = __ffma2_rn(both(d.y), make_float2(bv.z, bv.w), a1);
        if (kGate) {
          const float4 cv = *reinterpret_cast<const float4 *>(&m.C[i][4 * q]);
          const float2 yy = __ffma2_rn(h[1], make_float2(cv.z, cv.w), __fmul2_rn(h[0], make_float2(cv.x, cv.y)));
          y[j] = yy.x + yy.y;
        }
      }
      if (kGate) {
        spread_sum<kLanes, kStep, 1>(y, q);
#pragma unroll
        for (int v = 0; v < (kStep > kLanes ? kStep / kLanes : 1); ++v)
          if (q < kStep) m.y[i0 + v * kLanes + q][ch] = y[v];
      }
    }
    // and back
#pragma unroll 1
    for (int i0 = kTok - kStep; i0 >= 0; i0 -= kStep) {
      float s1[kStep], s2[kStep];
#pragma unroll
      for (int j = kStep - 1; j >= 0; --j) {
        const int i = i0 + j;
        const float2 d = m.steps[i][ch];
        const float dy = m.dy[i][ch];
        const float4 bv = *reinterpret_cast<const float4 *>(&m.B[i][4 * q]);
        const float4 cv = *reinterpret_cast<const float4 *>(&m.C[i][4 * q]);
        const float4 av = m.ah[i][tid];
        const float2 b0 = make_float2(bv.x, bv.y), b1 = make_float2(bv.z, bv.w);
        const float2 ah0 = make_float2(av.x, av.y), ah1 = make_float2(av.z, av.w);
        G[0] = __ffma2_rn(make_float2(cv.x, cv.y), both(dy), G[0]);
        G[1] = __ffma2_rn(make_float2(cv.z, cv.w), both(dy), G[1]);
        const float2 B0 = __fmul2_rn(G[0], both(d.y)), B1 = __fmul2_rn(G[1], both(d.y));
        const float2 C0 = __fmul2_rn(__ffma2_rn(both(d.y), b0, ah0), both(dy));
        const float2 C1 = __fmul2_rn(__ffma2_rn(both(d.y), b1, ah1), both(dy));
        const float2 t1 = __ffma2_rn(G[1], b1, __fmul2_rn(G[0], b0));
        const float2 w0 = __fmul2_rn(G[0], ah0), w1 = __fmul2_rn(G[1], ah1);
        const float2 t2 = __ffma2_rn(w1, A[1], __fmul2_rn(w0, A[0]));
        s1[j] = t1.x + t1.y, s2[j] = t2.x + t2.y;
        dA[0] = __ffma2_rn(w0, both(d.x), dA[0]), dA[1] = __ffma2_rn(w1, both(d.x), dA[1]);
        G[0] = __fmul2_rn(exp2_approx(__fmul2_rn(both(d.x), A[0])), G[0]);
        G[1] = __fmul2_rn(exp2_approx(__fmul2_rn(both(d.x), A[1])), G[1]);
        float v[8] = {B0.x, B0.y, B1.x, B1.y, C0.x, C0.y, C1.x, C1.y};
        spread_sum<kPerWarp, 8, kLanes>(v, num);
        // value k of a lane's four components' dB (k < 4) and dC
#pragma unroll
        for (int r = 0; r < (kPerWarp < 8 ? 8 / kPerWarp : 1); ++r) {
          const int k8 = num + r * kPerWarp;
          if (k8 < 8) m.bc[i][warp][(k8 >> 2) * DS + 4 * q + (k8 & 3)] = v[r];
        }
      }
      spread_sum<kLanes, kStep, 1>(s1, q);
      spread_sum<kLanes, kStep, 1>(s2, q);
#pragma unroll
      for (int v = 0; v < (kStep > kLanes ? kStep / kLanes : 1); ++v)
        if (q < kStep) m.s1[i0 + v * kLanes + q][ch] = s1[v], m.s2[i0 + v * kLanes + q][ch] = s2[v];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const int j = tid + i * kThreads, row = j >> 2, col = (tid & 3) * 8;
      const long t = t0 + row;
      if (j >= kTok * 4 || !live || t >= end) break;
      float2 xv[4], tv[4], dv[4], zv[4], ox[4], ot[4], oz[4];
      kx[i].get(xv), kt[i].get(tv), kd[i].get(dv);
      if (kGate) kz[i].get(zv);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 s1 = *reinterpret_cast<const float2 *>(&m.s1[row][col + 2 * e]);
        const float2 s2 = *reinterpret_cast<const float2 *>(&m.s2[row][col + 2 * e]);
        const float2 dy = *reinterpret_cast<const float2 *>(&m.dy[row][col + 2 * e]);
        const float4 st = reinterpret_cast<const float4 *>(&m.steps[row][col])[e];
        ox[e] = __ffma2_rn(make_float2(st.x, st.z), s1, __fmul2_rn(skip[e], dy));
        ot[e] = __ffma2_rn(xv[e], s1, __fmul2_rn(s2, both(0.693147181f)));  // A carries log2 e
        if (p.softplus) ot[e] = __fmul2_rn(ot[e], Sigmoid2(__fadd2_rn(tv[e], bias[e])).s);
        dD[e] = __ffma2_rn(dy, xv[e], dD[e]);
        dbias[e] = __fadd2_rn(dbias[e], ot[e]);
        if (kGate) {
          const float2 y = __ffma2_rn(skip[e], xv[e], *reinterpret_cast<const float2 *>(&m.y[row][col + 2 * e]));
          const Sigmoid2 sg(zv[e]);
          const float2 slope = __ffma2_rn(__fmul2_rn(zv[e], sg.s), sg.one_less(), sg.s);
          oz[e] = __fmul2_rn(__fmul2_rn(dv[e], y), slope);
        }
      }
      const long o = out0 + t * p.D;
      put8((T *)g.dx + o, ox), put8((T *)g.ddt + o, ot);
      if (kGate) put8((T *)g.dz + o, oz);
    }
    for (int i = tid; i < kTok * 2 * DS; i += kThreads) {
      const int row = i / (2 * DS), col = i % (2 * DS);
      float v = m.bc[row][0][col];
#pragma unroll
      for (int w = 1; w < kThreads / 32; ++w) v += m.bc[row][w][col];
      if (t0 + row < end) s.bc[((long)cb * p.B * p.N + b * p.N + t0 + row) * (2 * DS) + col] = v;
    }
    __syncthreads();
  }
  if (seg == 0 && g.dS0 && mine) *reinterpret_cast<float4 *>(g.dS0 + b * state + at) = make_float4(G[0].x, G[0].y, G[1].x, G[1].y);
  float *to = s.columns + (b * s.segs + seg) * (long)p.D * (DS + 2);
  if (mine) *reinterpret_cast<float4 *>(to + at) = make_float4(dA[0].x, dA[0].y, dA[1].x, dA[1].y);
  __syncthreads();
  float *part = reinterpret_cast<float *>(raw_smem);  // [warp][dD, dbias][32 channels]
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      dD[e].x += __shfl_xor_sync(0xffffffffu, dD[e].x, o), dD[e].y += __shfl_xor_sync(0xffffffffu, dD[e].y, o);
      dbias[e].x += __shfl_xor_sync(0xffffffffu, dbias[e].x, o), dbias[e].y += __shfl_xor_sync(0xffffffffu, dbias[e].y, o);
    }
    if (lane < 4) {
      float *at8 = part + warp * 2 * kCols + lane * 8 + 2 * e;
      at8[0] = dD[e].x, at8[1] = dD[e].y, at8[kCols] = dbias[e].x, at8[kCols + 1] = dbias[e].y;
    }
  }
  __syncthreads();
  if (tid < 2 * kCols && cb * kCols + tid % kCols < p.D) {
    float v = part[tid];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) v += part[w * 2 * kCols + tid];
    to[state + (long)(tid / kCols) * p.D + cb * kCols + tid % kCols] = v;
  }
}

// dB and dC from the partial sums of the blocks of channels: a thread a token and component.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(const __grid_constant__ ScanGradProblem g, const __grid_constant__ ScanSplit s) {
  const ScanProblem &p = g.p;
  const int ds2 = 2 * p.ds, nb = (p.D + kCols - 1) / kCols;
  const long rows = (long)p.B * p.N, all = rows * ds2, i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= all) return;
  const long row = i / ds2, b = row / p.N;
  const int col = (int)(i - row * ds2);
  float v = 0.f;
  if (row - b * p.N < row_length(p.lengths, b, p.N)) {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    int k = 0;
    for (; k + 4 <= nb; k += 4)
#pragma unroll
      for (int u = 0; u < 4; ++u) a[u] += s.bc[(k + u) * all + i];
    for (; k < nb; ++k) a[0] += s.bc[k * all + i];
    v = (a[0] + a[1]) + (a[2] + a[3]);
  }
  T *to = col < p.ds ? (T *)g.dB + row * p.ds + col : (T *)g.dC + row * p.ds + col - p.ds;
  if constexpr (sizeof(T) == 2)
    *to = __float2bfloat16(v);
  else
    *to = v;
}

template <typename T, int DS>
cudaError_t launch_grad(const ScanGradProblem &g, const ScanSplit &s) {
  const ScanProblem &p = g.p;
  const void *fn = p.z ? (const void *)scan_grad_kernel<T, DS, true> : (const void *)scan_grad_kernel<T, DS, false>;
  cudaError_t e = ensure_smem_optin(fn, sizeof(Smem<DS>));
  if (e != cudaSuccess) return e;
  const long blocks = (long)p.B * s.segs * ((p.D + kCols - 1) / kCols);
  {
    LaunchTimer timer(kKSelectiveBackward, p.stream);
    void *args[] = {const_cast<ScanGradProblem *>(&g), const_cast<ScanSplit *>(&s)};
    e = cudaLaunchKernel(fn, dim3((unsigned)blocks), dim3(8 * DS), args, sizeof(Smem<DS>), p.stream);
    timer.done(e);
    if (e != cudaSuccess) return e;
    count_launch();
  }
  LaunchTimer timer(kKSelectiveBackward, p.stream);
  scan_bc_kernel<T><<<(unsigned)(((long)p.B * p.N * 2 * DS + 255) / 256), 256, 0, p.stream>>>(g, s);
  e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T>
cudaError_t launch_ds(const ScanGradProblem &g, const ScanSplit &s) {
  return g.p.ds == 8    ? launch_grad<T, 8>(g, s)
         : g.p.ds == 16 ? launch_grad<T, 16>(g, s)
         : g.p.ds == 32 ? launch_grad<T, 32>(g, s)
                        : launch_grad<T, 64>(g, s);
}

// The workspace's parts, in floats; every one is a multiple of 32 bytes.
struct Parts {
  size_t starts, total, rev_starts, rev_total, chunk_states, bc, columns, all;
};
Parts parts(const ScanProblem &p, const ScanSplit &s) {
  const size_t state = (size_t)p.D * p.ds, rows = (size_t)p.B * s.segs;
  Parts q{};
  size_t o = 0;
  auto take = [&](size_t n) {
    const size_t at = o;
    o += n;
    return at;
  };
  const size_t split = s.segs > 1 ? rows : 0;
  q.starts = take(split * state);
  q.total = take(split * p.D);
  q.rev_starts = take(split * state);
  q.rev_total = take(split * p.D);
  q.chunk_states = take((size_t)p.B * s.all_chunks * state);
  q.bc = take((size_t)((p.D + kCols - 1) / kCols) * p.B * p.N * 2 * p.ds);
  q.columns = take(rows * p.D * (p.ds + 2));
  q.all = o;
  return q;
}
ScanSplit grad_split(const ScanProblem &p) {
  ScanSplit s = scan_split(p);
  s.chunk = chunk_tokens(p.ds);
  s.all_chunks = (p.N + s.chunk - 1) / s.chunk;
  return s;
}

}  // namespace

size_t scan_grad_workspace(const ScanProblem &p) { return sizeof(float) * parts(p, grad_split(p)).all; }

cudaError_t launch_selective_scan_grad(const ScanGradProblem &g) {
  const ScanProblem &p = g.p;
  ScanSplit s = grad_split(p);
  const Parts at = parts(p, s);
  float *ws = (float *)p.ws;
  s.chunk_states = ws + at.chunk_states;
  s.bc = ws + at.bc;
  s.columns = ws + at.columns;
  cudaError_t e = cudaSuccess;
  if (s.segs > 1) {
    s.starts = ws + at.starts, s.total = ws + at.total, s.rev_starts = ws + at.rev_starts, s.rev_total = ws + at.rev_total;
    e = launch_scan_starts(p, s);
    if (e != cudaSuccess) return e;
    ScanProblem r = p;
    r.x = g.dout, r.ldx = p.D;
    e = launch_scan_reverse_starts(r, s, g.dS);
    if (e != cudaSuccess) return e;
  }
  e = launch_scan_states(p, s);
  if (e == cudaSuccess) e = p.dt == LA_F32 ? launch_ds<float>(g, s) : launch_ds<__nv_bfloat16>(g, s);
  if (e != cudaSuccess) return e;
  const long state = (long)p.D * p.ds;
  ColumnSums c{s.columns, (long)p.B * s.segs, state + 2L * p.D, {}};
  c.part[0] = {g.dA, state, 1};
  c.part[1] = {g.dD, state + p.D, 1};
  c.part[2] = {g.dbias, state + 2L * p.D, 1};
  return launch_column_sums(c, kKSelectiveBackward, p.stream);
}

}  // namespace la
