// Selective state space scan: outputs, and the states in front of chunks or at the ends of segments.
//
// Formulas in selective.cuh.  A lane owns four state components of one channel, ds/4 neighbouring lanes
// a channel: the state stays in registers while the lane walks over the tokens, one fused multiply-add after
// another, and the exponentials of later tokens do not wait for it.  A block takes 32 channels (64 bytes of
// a bf16 row) and goes through the tokens in chunks of 32:
//   1. threads as (token, eight channels): delta = softplus(dt + bias) and delta x to shared memory, B and C in
//      32 bits beside them; the next chunk's rows are loaded meanwhile;
//   2. lanes as (channel, four components): the recurrence, and C . h spread over the channel's lanes
//      (spread_sum: every lane ends up with one token's sum);
//   3. threads as in 1 again: + D x, times silu(z), rows out.
//
// One exponential a component, channel and token (plus three for softplus and the gate of each channel) on the
// special-function pipe, and about four issue slots a component, bound it, before HBM does.
//
// When batch and channels alone do not fill the SMs, the tokens are cut into segments: a first pass leaves
// each segment's end state from zero and its sum of delta (the decay of the whole segment is e^{A sum}), a second
// one joins them, and the outputs' pass starts every segment from its own state.
#include <algorithm>

#include "internal.h"
#include "selective.cuh"

namespace la {
namespace {

constexpr int kTok = 32;         // tokens a chunk
constexpr int kCols = 32;        // channels a block
constexpr int kRow = kCols + 8;  // floats between tokens of the sums' place: four tokens of eight channels meet no bank twice

enum Mode { kOutputs, kEnds, kStates, kReverseEnds };

// kOutputs: out, and the last segment's end state to S.  kEnds: each segment's end state from zero and sum of
// delta.  kStates: the state in front of each chunk of s.chunk tokens.  kReverseEnds: the same as kEnds for the
// recurrence of the state's gradient, from a segment's last token to its first: G <- a_t (G + C_t dy_t).
template <typename T, int DS, int kMode>
__global__ void __launch_bounds__(8 * DS) scan_kernel(const __grid_constant__ ScanProblem p, const __grid_constant__ ScanSplit s) {
  constexpr int kThreads = 8 * DS, kLanes = DS / 4, kPerWarp = 32 / kLanes;
  constexpr int kGroups = (kTok * 4 + kThreads - 1) / kThreads;  // (token, eight channels) a thread
  constexpr bool kRev = kMode == kReverseEnds;
  __shared__ __align__(16) float2 steps[kTok][kCols];  // delta; delta x (reverse: dy)
  __shared__ __align__(16) float sB[kTok][DS];         // (reverse: C)
  __shared__ __align__(16) float sC[kMode == kOutputs ? kTok : 1][DS];
  __shared__ __align__(16) float sums[kMode == kOutputs ? kTok : 1][kRow];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nb = (p.D + kCols - 1) / kCols;
  const int cb = blockIdx.x % nb;
  const long rest = blockIdx.x / nb;
  const int seg = (int)(rest % s.launched) + (kRev ? 1 : 0);
  const long b = rest / s.launched;
  const long n = row_length(p.lengths, b, p.N);
  const long begin = (long)seg * s.len, end = min(begin + s.len, n);
  const long chunks = end > begin ? (end - begin + kTok - 1) / kTok : 0;

  // as (channel, components)
  const int q = lane % kLanes, ch = warp * kPerWarp + lane / kLanes;
  const int c = cb * kCols + ch;
  const long at = (long)c * DS + 4 * q;  // in a state
  const long state = (long)p.D * DS;
  float2 A[2] = {both(0.f), both(0.f)}, h[2] = {both(0.f), both(0.f)};
  if (c < p.D) {
    const float4 a = *reinterpret_cast<const float4 *>(p.A + at);
    A[0] = __fmul2_rn(make_float2(a.x, a.y), both(kLog2e)), A[1] = __fmul2_rn(make_float2(a.z, a.w), both(kLog2e));
    const float *from = nullptr;
    if (kMode == kOutputs || kMode == kStates) from = s.starts ? s.starts + (b * s.segs + seg) * state : p.S0 ? p.S0 + b * state : nullptr;
    if (from) {
      const float4 v = *reinterpret_cast<const float4 *>(from + at);
      h[0] = make_float2(v.x, v.y), h[1] = make_float2(v.z, v.w);
    }
  }

  // as (token, eight channels): every group of a thread has the same channels
  const int c8 = cb * kCols + (tid & 3) * 8;
  const bool live = c8 < p.D;
  float2 bias[4], skip[4], total[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    bias[e] = live && p.dt_bias ? reinterpret_cast<const float2 *>(p.dt_bias + c8)[e] : both(0.f);
    skip[e] = live && p.Dskip && kMode == kOutputs ? reinterpret_cast<const float2 *>(p.Dskip + c8)[e] : both(0.f);
    total[e] = both(0.f);
  }
  const T *x = (const T *)p.x + b * p.N * p.ldx + c8, *dt = (const T *)p.delta + b * p.N * p.ldt + c8;
  const T *z = p.z ? (const T *)p.z + b * p.N * p.ldz + c8 : nullptr;
  constexpr bool kNeedZ = kMode == kOutputs || kRev;
  Raw<T> rx[kGroups], rt[kGroups], rz[kNeedZ ? kGroups : 1], rb, rc;
  // rows of B (and C): eight components a thread, as many threads as kTok * DS / 8
  constexpr int kPieces = kTok * DS / 8, kPerRow = DS / 8;
  const bool with_c = kMode == kOutputs && tid >= kPieces;
  const int piece = with_c ? tid - kPieces : tid, brow = piece / kPerRow, bcol = piece % kPerRow * 8;
  const T *bc = with_c || kRev ? (const T *)p.Cm + b * p.N * p.ldc + bcol : (const T *)p.Bm + b * p.N * p.ldb + bcol;
  const long ldbc = with_c || kRev ? p.ldc : p.ldb;
  const bool has_bc = kMode == kOutputs ? tid < 2 * kPieces : tid < kPieces;
  static_assert(2 * kPieces == kThreads, "a piece a thread");
  auto load = [&](long t0) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int i = tid + g * kThreads;
      const long t = t0 + (i >> 2);
      rx[g].zero(), rt[g].zero();
      if (kNeedZ) rz[g].zero();
      if (i < kTok * 4 && live && t < end) {
        rx[g].load(x + t * p.ldx);
        rt[g].load(dt + t * p.ldt);
        if (kNeedZ && z) rz[g].load(z + t * p.ldz);
      }
    }
    rb.zero();
    if (has_bc && t0 + brow < end) rb.load(bc + (t0 + brow) * ldbc);
  };
  (void)rc;
  auto first_of = [&](long k) { return begin + (kRev ? chunks - 1 - k : k) * kTok; };
  if (chunks) load(first_of(0));
  for (long k = 0; k < chunks; ++k) {
    const long t0 = first_of(k);
    Raw<T> kx[kMode == kOutputs ? kGroups : 1], kz[kMode == kOutputs ? kGroups : 1];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int i = tid + g * kThreads;
      if (i >= kTok * 4) break;
      const long t = t0 + (i >> 2);
      if (kMode == kOutputs) kx[g] = rx[g], kz[g] = rz[g];
      float2 xv[4], tv[4], zv[4];
      rx[g].get(xv), rt[g].get(tv);
      if (kRev) rz[g].get(zv);
      float4 *to = reinterpret_cast<float4 *>(&steps[i >> 2][(tid & 3) * 8]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 d = __fadd2_rn(tv[e], bias[e]);
        if (p.softplus) d = softplus2(d);
        if (t >= end) d = both(0.f);
        if (kMode == kEnds || kRev) total[e] = __fadd2_rn(total[e], d);
        float2 u = kRev ? xv[e] : __fmul2_rn(d, xv[e]);
        if (kRev && z) u = __fmul2_rn(u, __fmul2_rn(zv[e], Sigmoid2(zv[e]).s));
        if (t >= end) u = both(0.f);
        to[e] = make_float4(d.x, u.x, d.y, u.y);
      }
    }
    if (has_bc) {
      float2 v[4];
      rb.get(v);
      float *to = with_c ? &sC[kMode == kOutputs ? brow : 0][bcol] : &sB[brow][bcol];
      put8(to, v);
    }
    if (k + 1 < chunks) load(first_of(k + 1));
    if (kMode == kStates && c < p.D && (t0 - begin) % s.chunk == 0)
      *reinterpret_cast<float4 *>(s.chunk_states + (b * s.all_chunks + t0 / s.chunk) * state + at) =
          make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    __syncthreads();
#pragma unroll 1
    for (int i0 = 0; i0 < kTok; i0 += kLanes < 4 ? 4 : kLanes) {
      constexpr int kStep = kLanes < 4 ? 4 : kLanes;
      float y[kStep];
#pragma unroll
      for (int j = 0; j < kStep; ++j) {
        const int i = kRev ? kTok - 1 - (i0 + j) : i0 + j;
        if (kMode == kStates && j % 8 == 0 && s.chunk < kTok && i > 0 && i % s.chunk == 0 && c < p.D && t0 + i < end)
          *reinterpret_cast<float4 *>(s.chunk_states + (b * s.all_chunks + (t0 + i) / s.chunk) * state + at) =
              make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
        const float2 d = steps[i][ch];
        const float4 bv = *reinterpret_cast<const float4 *>(&sB[i][4 * q]);
        const float2 a0 = exp2_approx(__fmul2_rn(both(d.x), A[0])), a1 = exp2_approx(__fmul2_rn(both(d.x), A[1]));
        const float2 u0 = __fmul2_rn(both(d.y), make_float2(bv.x, bv.y)), u1 = __fmul2_rn(both(d.y), make_float2(bv.z, bv.w));
        if (kRev) {
          h[0] = __fmul2_rn(a0, __fadd2_rn(h[0], u0)), h[1] = __fmul2_rn(a1, __fadd2_rn(h[1], u1));
        } else {
          h[0] = __ffma2_rn(a0, h[0], u0), h[1] = __ffma2_rn(a1, h[1], u1);
        }
        if (kMode == kOutputs) {
          const float4 cv = *reinterpret_cast<const float4 *>(&sC[i][4 * q]);
          const float2 yy = __ffma2_rn(h[1], make_float2(cv.z, cv.w), __fmul2_rn(h[0], make_float2(cv.x, cv.y)));
          y[j] = yy.x + yy.y;
        }
      }
      if (kMode == kOutputs) {
        spread_sum<kLanes, kStep, 1>(y, q);
        if (kLanes >= 4) {
          sums[i0 + q][ch] = y[0];
        } else {
          sums[i0 + q][ch] = y[0];
          sums[i0 + 2 + q][ch] = y[1];
        }
      }
    }
    __syncthreads();
    if (kMode == kOutputs) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const int i = tid + g * kThreads;
        const long t = t0 + (i >> 2);
        if (i >= kTok * 4 || !live || t >= end) break;
        const float4 y0 = *reinterpret_cast<const float4 *>(&sums[i >> 2][(tid & 3) * 8]);
        const float4 y1 = *reinterpret_cast<const float4 *>(&sums[i >> 2][(tid & 3) * 8 + 4]);
        float2 y[4] = {make_float2(y0.x, y0.y), make_float2(y0.z, y0.w), make_float2(y1.x, y1.y), make_float2(y1.z, y1.w)};
        float2 xv[4], zv[4];
        kx[g].get(xv), kz[g].get(zv);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = __ffma2_rn(skip[e], xv[e], y[e]);
          if (z) y[e] = __fmul2_rn(y[e], __fmul2_rn(zv[e], Sigmoid2(zv[e]).s));
        }
        put8((T *)p.out + (b * p.N + t) * p.D + c8, y);
      }
    }
  }
  const float4 hv = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
  if (kMode == kOutputs) {
    if (seg == s.segs - 1 && c < p.D) *reinterpret_cast<float4 *>(p.S + b * state + at) = hv;
  } else if (kMode == kEnds || kRev) {
    if (c < p.D) *reinterpret_cast<float4 *>((kRev ? s.rev_starts : s.starts) + (b * s.segs + seg) * state + at) = hv;
    // sums of delta: the threads of the same eight channels in order
    float *part = &steps[0][0].x;
    static_assert(8 * kThreads <= 2 * kTok * kCols * (kThreads > 256 ? 2 : 1), "place for the sums");
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // neighbours in a warp first: lanes 4 apart have the same channels
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        total[e].x += __shfl_xor_sync(0xffffffffu, total[e].x, o);
        total[e].y += __shfl_xor_sync(0xffffffffu, total[e].y, o);
      }
      if (lane < 4) {
        part[warp * kCols + lane * 8 + 2 * e] = total[e].x;
        part[warp * kCols + lane * 8 + 2 * e + 1] = total[e].y;
      }
    }
    __syncthreads();
    if (tid < kCols && cb * kCols + tid < p.D) {
      float v = part[tid];
#pragma unroll
      for (int w = 1; w < kThreads / 32; ++w) v += part[w * kCols + tid];
      (kRev ? s.rev_total : s.total)[(b * s.segs + seg) * p.D + cb * kCols + tid] = v;
    }
  }
}

// Segment ends to segment starts, in place: starts[s] <- h, h <- e^{A total[s]} h + starts[s] (old), from S0; the
// state's gradient the same way from the last segment, from dS.  A thread a component.
__global__ void __launch_bounds__(256) scan_join_kernel(const __grid_constant__ ScanSplit s, const float *A,
                                                        const float *S0, int B, int D, int ds, bool reverse) {
  const long state = (long)D * ds, i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= B * state) return;
  const long b = i / state, r = i - b * state, c = r / ds;
  const float a = A[r] * kLog2e;
  float h = S0 ? S0[i] : 0.f;
  float *starts = (reverse ? s.rev_starts : s.starts) + b * s.segs * state + r;
  const float *total = (reverse ? s.rev_total : s.total) + b * s.segs * D + c;
  constexpr int kAhead = 8;
  for (int k0 = 0; k0 < s.segs; k0 += kAhead) {
    float v[kAhead], d[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = reverse ? s.segs - 1 - (k0 + u) : k0 + u;
      const bool has = k0 + u < s.segs - 1;  // the last one's end starts no other segment
      v[u] = has ? starts[k * state] : 0.f;
      d[u] = has ? total[(long)k * D] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = reverse ? s.segs - 1 - (k0 + u) : k0 + u;
      if (k0 + u >= s.segs) break;
      starts[k * state] = h;
      h = fmaf(exp2f(a * d[u]), h, v[u]);
    }
  }
}

template <typename T, int DS>
cudaError_t launch_mode(const ScanProblem &p, ScanSplit s, int mode) {
  s.launched = mode == kEnds || mode == kReverseEnds ? s.segs - 1 : s.segs;
  const long blocks = (long)p.B * s.launched * ((p.D + kCols - 1) / kCols);
  LaunchTimer timer(mode == kOutputs ? kKSelectiveScan : kKSelectiveState, p.stream);
  if (mode == kOutputs)
    scan_kernel<T, DS, kOutputs><<<(unsigned)blocks, 8 * DS, 0, p.stream>>>(p, s);
  else if (mode == kEnds)
    scan_kernel<T, DS, kEnds><<<(unsigned)blocks, 8 * DS, 0, p.stream>>>(p, s);
  else if (mode == kStates)
    scan_kernel<T, DS, kStates><<<(unsigned)blocks, 8 * DS, 0, p.stream>>>(p, s);
  else
    scan_kernel<T, DS, kReverseEnds><<<(unsigned)blocks, 8 * DS, 0, p.stream>>>(p, s);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

template <typename T>
cudaError_t launch_ds(const ScanProblem &p, const ScanSplit &s, int mode) {
  return p.ds == 8    ? launch_mode<T, 8>(p, s, mode)
         : p.ds == 16 ? launch_mode<T, 16>(p, s, mode)
         : p.ds == 32 ? launch_mode<T, 32>(p, s, mode)
                      : launch_mode<T, 64>(p, s, mode);
}

cudaError_t launch(const ScanProblem &p, const ScanSplit &s, int mode) {
  return p.dt == LA_F32 ? launch_ds<float>(p, s, mode) : launch_ds<__nv_bfloat16>(p, s, mode);
}

cudaError_t join(const ScanProblem &p, const ScanSplit &s, const float *from, bool reverse) {
  const long all = (long)p.B * p.D * p.ds;
  LaunchTimer timer(kKSelectiveState, p.stream);
  scan_join_kernel<<<(unsigned)((all + 255) / 256), 256, 0, p.stream>>>(s, p.A, from, p.B, p.D, p.ds, reverse);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

// One segment where the batch's channels fill the SMs' schedulers with a warp each (the first pass costs two thirds
// of the outputs' pass); otherwise enough for two warps each, of at least 256 tokens.
ScanSplit scan_split(const ScanProblem &p) {
  ScanSplit s{};
  const long schedulers = 4L * std::max(1, device_info(-1).sm_count);
  const long warps = (long)p.B * ((p.D + kCols - 1) / kCols) * (p.ds / 4);
  long segs = 1;
  if (warps < schedulers) segs = std::max(1L, std::min((2 * schedulers + warps - 1) / warps, p.N / 256));
  s.len = (p.N + segs - 1) / segs;
  s.len = (s.len + kTok - 1) / kTok * kTok;
  s.segs = (int)std::max(1L, (p.N + s.len - 1) / s.len);
  return s;
}

size_t scan_workspace(const ScanProblem &p) {
  const ScanSplit s = scan_split(p);
  return s.segs == 1 ? 0 : sizeof(float) * (size_t)p.B * s.segs * p.D * (p.ds + 1);
}

cudaError_t launch_scan_starts(const ScanProblem &p, const ScanSplit &s) {
  const cudaError_t e = launch(p, s, kEnds);
  return e != cudaSuccess ? e : join(p, s, p.S0, false);
}

cudaError_t launch_scan_reverse_starts(const ScanProblem &p, const ScanSplit &s, const float *dS) {
  const cudaError_t e = launch(p, s, kReverseEnds);
  return e != cudaSuccess ? e : join(p, s, dS, true);
}

cudaError_t launch_scan_states(const ScanProblem &p, const ScanSplit &s) { return launch(p, s, kStates); }

cudaError_t launch_selective_scan(const ScanProblem &p) {
  ScanSplit s = scan_split(p);
  if (s.segs > 1) {
    s.starts = (float *)p.ws;
    s.total = s.starts + (size_t)p.B * s.segs * p.D * p.ds;
    const cudaError_t e = launch_scan_starts(p, s);
    if (e != cudaSuccess) return e;
  }
  return launch(p, s, kOutputs);
}

}  // namespace la
