// Selective state space scan: outputs, and the states in front of chunks or at the ends of segments.
//
// Formulas in selective.cuh.  A lane owns four state components (or two: launch_mode) of two channels, ds/4 (ds/2)
// neighbouring lanes a pair of channels: the states stay in registers while the lane walks over the tokens.  (Every load
// from shared memory costs its port the lanes' bytes, broadcast or not: with two channels a lane B and C are read half as
// often as with one, which had the port 72 % taken and took 516 us for 488.)  A block takes 64 channels (ds = 64: 32) and goes through the
// tokens in chunks of 32, on two kinds of warps a chunk apart:
//   - around the recurrence, threads as (token, eight channels): rows in, delta = softplus(dt + bias) and delta x to shared
//     memory, B and C in 32 bits beside them; a chunk later + D x, times silu(z), rows out;
//   - the recurrence, and C . h spread over the channel's lanes (spread_sum: every lane ends up with one token's
//     sum).
//
// One exponential a component, channel and token and about six issue slots bound it, before HBM does: 4 x 8192 x 2048 x 16
// in bf16 in 413 us (79 us at the copy rate), where a block an SM is all there is and one warp a scheduler leaves half
// of the slots; 16 x 2048 tokens, two blocks an SM, in 347 us, where shared memory's port is 75 % taken.  Scalar
// instead of packed arithmetic: 585 for 488 us.
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

// Channels a block: as many as keep it within 512 threads.
constexpr int scan_cols(int ds) { return ds == 64 ? 32 : 64; }

// Threads of the recurrence with `comp` components of two channels each.
constexpr int scan_threads(int ds, int comp) { return scan_cols(ds) / 2 * ds / comp; }

enum Mode { kOutputs, kEnds, kStates, kReverseEnds };

template <int DS, int kMode>
struct Smem {
  static constexpr int kCols = scan_cols(DS), kRow = kCols + 8;  // floats between tokens of the sums' place
  float4 steps[kTok][kCols / 2];  // of two channels: delta, delta x (reverse: dy); at step_slot
  float B[kTok][DS];          // (reverse: C)
  float C[kMode == kOutputs ? kTok : 1][DS];
  float sums[kMode == kOutputs ? kTok : 1][kRow];
};

// kOutputs: out, and the last segment's end state to S.  kEnds: each segment's end state from zero and sum of
// delta.  kStates: the state in front of each chunk of s.chunk tokens.  kReverseEnds: the same as kEnds for the
// recurrence of the state's gradient, from a segment's last token to its first: G <- a_t (G + C_t dy_t).
// kAround: threads around the recurrence, (token, eight channels) in turns.  kComp: components a lane.  `block`
// of the mode's blocks.
template <typename T, int DS, int kMode, int kAround, int kComp>
__device__ __forceinline__ void scan_block(const ScanProblem &p, const ScanSplit &s, unsigned block) {
  constexpr int kCols = Smem<DS, kMode>::kCols, kTurns = kTok * kCols / 8 / kAround;
  constexpr int kScan = kCols / 2 * DS / kComp, kThreads = kScan + kAround, kLanes = DS / kComp, kPerWarp = 64 / kLanes;
  constexpr int kP = kComp / 2;  // pairs of components
  constexpr bool kRev = kMode == kReverseEnds;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Smem<DS, kMode> *m = reinterpret_cast<Smem<DS, kMode> *>(raw_smem);
  __shared__ float part[kAround / 32][Smem<DS, kMode>::kCols];
  const int tid = threadIdx.x, lane = tid & 31;
  const int nb = (p.D + kCols - 1) / kCols;
  const int cb = block % nb;
  const long rest = block / nb;
  const int seg = (int)(rest % s.launched) + (kRev ? 1 : 0);
  const long b = rest / s.launched;
  const long n = row_length(p.lengths, b, p.N);
  const long begin = (long)seg * s.len, end = min(begin + s.len, n);
  const int chunks = end > begin ? (int)((end - begin + kTok - 1) / kTok) : 0;
  auto first_of = [&](int k) { return begin + (long)(kRev ? chunks - 1 - k : k) * kTok; };

  if (tid >= kScan) {
    // around the recurrence
    const int at = tid - kScan, col = (at % (kCols / 8)) * 8, c8 = cb * kCols + col, row0 = at / (kCols / 8);
    constexpr int kRows = kAround / (kCols / 8);  // tokens between a thread's turns
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
    T *out = (T *)p.out + b * p.N * p.D + c8;
    // rows of B (and C), eight components a piece
    constexpr int kPerRow = DS / 8, kOne = kTok * kPerRow, kPieces = kMode == kOutputs ? 2 * kOne : kOne;
    constexpr int kEach = (kPieces + kAround - 1) / kAround;
    const T *Bm = (const T *)(kRev ? p.Cm : p.Bm) + b * p.N * (kRev ? p.ldc : p.ldb), *Cm = (const T *)p.Cm + b * p.N * p.ldc;
    // Rows of the chunk that goes in, and of the next one, which are on their way all the while (an iteration's time is
    // about the latency of HBM: asked for only behind this chunk's work they cost 488 us for 390); x and z of the chunk
    // that comes out are read again, from L2.
    struct Rows {
      Raw<T> x[kTurns], t[kTurns], z[kTurns], b[kEach];
    } now, next;
    Raw<T> ox[kTurns], oz[kTurns];
    auto load = [&](Rows &r, long t0) {
#pragma unroll
      for (int u = 0; u < kTurns; ++u) {
        const long t = t0 + row0 + u * kRows;
        r.x[u].zero(), r.t[u].zero(), r.z[u].zero();
        if (live && t < end) {
          r.x[u].load(x + t * p.ldx), r.t[u].load(dt + t * p.ldt);
          if (kRev && z) r.z[u].load(z + t * p.ldz);
        }
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int k = at + i * kAround, which = k >= kOne, j = which ? k - kOne : k;
        r.b[i].zero();
        if (k < kPieces && t0 + j / kPerRow < end)
          r.b[i].load((which ? Cm : Bm) + (t0 + j / kPerRow) * (which ? p.ldc : kRev ? p.ldc : p.ldb) + j % kPerRow * 8);
      }
    };
    if (chunks) load(next, first_of(0));
    for (int k = 0; k <= chunks; ++k) {
      if (kMode == kOutputs && k > 0) {
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
          const long t = first_of(k - 1) + row0 + u * kRows;
          ox[u].zero(), oz[u].zero();
          if (live && t < end) {
            if (p.Dskip) ox[u].load(x + t * p.ldx);
            if (z) oz[u].load(z + t * p.ldz);
          }
        }
      }
      now = next;
      if (k + 1 < chunks) load(next, first_of(k + 1));
      if (k < chunks) {
        Smem<DS, kMode> &to = m[k & 1];
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
          const int row = row0 + u * kRows;
          const bool in = first_of(k) + row < end;
          float2 xv[4], tv[4], zv[4];
          now.x[u].get(xv), now.t[u].get(tv);
          if (kRev) now.z[u].get(zv);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 d = __fadd2_rn(tv[e], bias[e]);
            if (p.softplus) d = softplus2(d);
            if (!in) d = both(0.f);
            if (kMode == kEnds || kRev) total[e] = __fadd2_rn(total[e], d);
            float2 v = kRev ? xv[e] : __fmul2_rn(d, xv[e]);
            if (kRev && z) v = __fmul2_rn(v, __fmul2_rn(zv[e], Sigmoid2(zv[e]).s));
            if (!in) v = both(0.f);
            to.steps[row][step_slot(col / 2 + e)] = make_float4(d.x, v.x, d.y, v.y);
          }
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const int q = at + i * kAround, which = q >= kOne, j = which ? q - kOne : q;
          float2 v[4];
          now.b[i].get(v);
          if (q < kPieces) put8((which ? &to.C[0][0] : &to.B[0][0]) + j * 8, v);
        }
        bar_arrive<kThreads>(1 + (k & 1));
      }
      if (k > 0) {
        bar_sync<kThreads>(3 + ((k - 1) & 1));
        const Smem<DS, kMode> &from = m[(k - 1) & 1];
#pragma unroll
        for (int u = 0; u < kTurns; ++u) {
          const int row = row0 + u * kRows;
          const long t = first_of(k - 1) + row;
          if (kMode == kOutputs && live && t < end) {
            const float4 y0 = *reinterpret_cast<const float4 *>(&from.sums[row][col]);
            const float4 y1 = *reinterpret_cast<const float4 *>(&from.sums[row][col + 4]);
            float2 y[4] = {make_float2(y0.x, y0.y), make_float2(y0.z, y0.w), make_float2(y1.x, y1.y), make_float2(y1.z, y1.w)};
            float2 xv[4], zv[4];
            ox[u].get(xv), oz[u].get(zv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[e] = __ffma2_rn(skip[e], xv[e], y[e]);
              if (z) y[e] = __fmul2_rn(y[e], __fmul2_rn(zv[e], Sigmoid2(zv[e]).s));
            }
            put8(out + t * p.D, y);
          }
        }
      }
    }
    if (kMode == kEnds || kRev) {
      // sums of delta: lanes 8 apart have the same channels, then the warps in order
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int o = kCols / 8; o < 32; o <<= 1) {
          total[e].x += __shfl_xor_sync(0xffffffffu, total[e].x, o);
          total[e].y += __shfl_xor_sync(0xffffffffu, total[e].y, o);
        }
        if (lane < kCols / 8) *reinterpret_cast<float2 *>(&part[at >> 5][col + 2 * e]) = total[e];
      }
      bar_sync<kAround>(5);
      if (at < kCols && cb * kCols + at < p.D) {
        float v = part[0][at];
#pragma unroll
        for (int w = 1; w < kAround / 32; ++w) v += part[w][at];
        (kRev ? s.rev_total : s.total)[(b * s.segs + seg) * p.D + cb * kCols + at] = v;
      }
    }
    return;
  }

  // the recurrence
  const int q = lane % kLanes, ch = (tid >> 5) * kPerWarp + lane / kLanes * 2;
  const int c = cb * kCols + ch;  // and the next one; D is even
  const int slot = step_slot(ch / 2);
  const bool mine = c < p.D;
  const long at = (long)c * DS + kComp * q;  // in a state
  const long state = (long)p.D * DS;
  float2 A[2 * kP], h[2 * kP];  // of the first channel, of the second
  auto read = [](float2 *v, const float *from) {  // kComp values at once
    if constexpr (kP == 2) {
      const float4 f = *reinterpret_cast<const float4 *>(from);
      v[0] = make_float2(f.x, f.y), v[1] = make_float2(f.z, f.w);
    } else {
      v[0] = *reinterpret_cast<const float2 *>(from);
    }
  };
  auto get = [&](float2 (&v)[2 * kP], const float *from) {
#pragma unroll
    for (int i = 0; i < 2; ++i) read(&v[kP * i], from + at + i * DS);
  };
  auto put = [&](float *to) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (kP == 2)
        st4(to + at + i * DS, h[2 * i].x, h[2 * i].y, h[2 * i + 1].x, h[2 * i + 1].y);
      else
        *reinterpret_cast<float2 *>(to + at + i * DS) = h[i];
    }
  };
#pragma unroll
  for (int i = 0; i < 2 * kP; ++i) A[i] = h[i] = both(0.f);
  if (mine) {
    get(A, p.A);
    const float *from = nullptr;
    if (kMode == kOutputs || kMode == kStates) from = s.starts ? s.starts + (b * s.segs + seg) * state : p.S0 ? p.S0 + b * state : nullptr;
    if (from) get(h, from);
  }
#pragma unroll
  for (int i = 0; i < 2 * kP; ++i) A[i] = rate(A[i]);
  for (int k = 0; k < chunks; ++k) {
    Smem<DS, kMode> &in = m[k & 1];
    const long t0 = first_of(k);
    bar_sync<kThreads>(1 + (k & 1));
    // two tokens' values ahead of their use: the compiler does not move loads across the stores of sums
    struct Two {
      float4 d[2];
      float2 b[2][kP], c[kMode == kOutputs ? 2 : 1][kP];
    };
    auto token = [](int i) { return kRev ? kTok - 1 - i : i; };
    auto fetch = [&](Two &v, int i0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v.d[j] = in.steps[token(i0 + j)][slot];
        read(v.b[j], &in.B[token(i0 + j)][kComp * q]);
        if (kMode == kOutputs) read(v.c[j], &in.C[token(i0 + j)][kComp * q]);
      }
    };
    constexpr int kStep = kLanes < 4 ? 4 : kLanes;
    Two now, then;
    fetch(now, 0);
#pragma unroll
    for (int i0 = 0; i0 < kTok; i0 += kStep) {
      float y[2 * kStep];  // of the first channel, of the second
#pragma unroll
      for (int f = 0; f < kStep; f += 2) {
        if (i0 + f + 2 < kTok) fetch(then, i0 + f + 2);
        float2 a[2][2 * kP];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 2 * kP; ++i) a[j][i] = decay(both(i < kP ? now.d[j].x : now.d[j].z), A[i]);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (kMode == kStates && (f + j) % 8 == 0) {
            const int i = i0 + f + j;
            if (i % s.chunk == 0 && mine && t0 + i < end) put(s.chunk_states + (b * s.all_chunks + (t0 + i) / s.chunk) * state);
          }
#pragma unroll
          for (int i = 0; i < 2 * kP; ++i) {
            const float2 u = both(i < kP ? now.d[j].y : now.d[j].w), bv = now.b[j][i % kP];
            h[i] = kRev ? __fmul2_rn(a[j][i], __ffma2_rn(u, bv, h[i])) : __ffma2_rn(a[j][i], h[i], __fmul2_rn(u, bv));
          }
          if (kMode == kOutputs) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float2 yy = __fmul2_rn(h[kP * i], now.c[j][0]);
              if (kP == 2) yy = __ffma2_rn(h[kP * i + kP - 1], now.c[j][kP - 1], yy);
              y[i * kStep + f + j] = yy.x + yy.y;
            }
          }
        }
        now = then;
      }
      if (kMode == kOutputs) {
        spread_sum<kLanes, 2 * kStep, 1>(y, q);
        constexpr int kHave = kStep / kLanes;
#pragma unroll
        for (int v = 0; v < kHave; ++v)
          *reinterpret_cast<float2 *>(&in.sums[i0 + v * kLanes + q][ch]) = make_float2(y[v], y[kHave + v]);
      }
    }
    bar_arrive<kThreads>(3 + (k & 1));
  }
  if (kMode == kOutputs) {
    if (seg == s.segs - 1 && mine) put(p.S + b * state);
  } else if (kMode == kEnds || kRev) {
    if (mine) put((kRev ? s.rev_starts : s.starts) + (b * s.segs + seg) * state);
  }
}

template <typename T, int DS, int kMode, int kAround, int kComp>
__global__ void __launch_bounds__(scan_threads(DS, kComp) + kAround) scan_kernel(const __grid_constant__ ScanProblem p, const __grid_constant__ ScanSplit s) {
  scan_block<T, DS, kMode, kAround, kComp>(p, s, blockIdx.x);
}

// The ends of segments in both directions, side by side: the second half of the blocks runs q, whose x is the gradient of
// the outputs.
template <typename T, int DS>
__global__ void __launch_bounds__(scan_threads(DS, 4) + 128)
    scan_ends_kernel(const __grid_constant__ ScanProblem p, const __grid_constant__ ScanProblem q, const __grid_constant__ ScanSplit s) {
  const unsigned half = gridDim.x / 2;
  if (blockIdx.x < half)
    scan_block<T, DS, kEnds, 128, 4>(p, s, blockIdx.x);
  else
    scan_block<T, DS, kReverseEnds, 128, 4>(q, s, blockIdx.x - half);
}

// 2^exponent h + v.  A segment that grows (negative steps, A > 0) may do so beyond 2^128 while the state it starts from, zero
// or small, has a finite product: the power is split then, and its whole part goes straight into the product's exponent.
__device__ __forceinline__ float grown(float exponent, float h, float v) {
  if (!(exponent > 126.f)) return fmaf(exp2f(exponent), h, v);
  const float whole = rintf(fminf(exponent, 1024.f));  // (2^1024 takes the smallest number beyond the largest)
  return ldexpf(exp2f(fminf(exponent, 1024.f) - whole) * h, (int)whole) + v;
}

// Segment ends to segment starts, in place: starts[s] <- h, h <- e^{A total[s]} h + starts[s] (old), from S0; the
// state's gradient (blockIdx.y = 1) the same way from the last segment, from dS.  A thread a component.
__global__ void __launch_bounds__(256) scan_join_kernel(const __grid_constant__ ScanSplit s, const float *A,
                                                        const float *S0, const float *dS, int B, int D, int ds) {
  const bool reverse = blockIdx.y;
  const long state = (long)D * ds, i = (long)blockIdx.x * 256 + threadIdx.x;
  if (i >= B * state) return;
  const long b = i / state, r = i - b * state, c = r / ds;
  const float a = rate(A[r]);
  const float *from = reverse ? dS : S0;
  float h = from ? from[i] : 0.f;
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
      h = grown(a * d[u], h, v[u]);
    }
  }
}

template <typename T, int DS, int kMode, int kAround, int kComp>
cudaError_t launch_kernel(const ScanProblem &p, const ScanSplit &s, long blocks) {
  const void *fn = (const void *)scan_kernel<T, DS, kMode, kAround, kComp>;
  constexpr int kSmem = 2 * (int)sizeof(Smem<DS, kMode>);
  cudaError_t e = kSmem > 48 * 1024 ? ensure_smem_optin(fn, kSmem) : cudaSuccess;
  if (e != cudaSuccess) return e;
  LaunchTimer timer(kMode == kOutputs ? kKSelectiveScan : kKSelectiveState, p.stream);
  void *args[] = {const_cast<ScanProblem *>(&p), const_cast<ScanSplit *>(&s)};
  e = cudaLaunchKernel(fn, dim3((unsigned)blocks), dim3(scan_threads(DS, kComp) + kAround), args, kSmem, p.stream);
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

// Outputs: where a block an SM is all there is, the work around its recurrence gets twice the warps (4 x 8192 x 2048 x 16:
// 445 us to 413); with more blocks an SM their registers are worth more (16 x 2048 tokens: 347 us, with them 415).
// With a block an SM, two components a lane instead of four are twice the warps of the recurrence: states in front of
// chunks, 4 x 4096 x 2048 x 16, 198 us to 163, outputs of 8 components 357 to 340; outputs of 16 need the steps
// and C twice as often from shared memory then (413 us, with two 453).  With two blocks an SM four are as good or better
// (states of 16 x 1024 tokens 159 us, with two 167; outputs of 8 components in fp32 287, with two 472).
template <typename T, int DS>
cudaError_t launch_mode(const ScanProblem &p, ScanSplit s, int mode) {
  s.launched = mode == kEnds ? s.segs - 1 : s.segs;
  const long blocks = (long)p.B * s.launched * ((p.D + scan_cols(DS) - 1) / scan_cols(DS));
  if (mode == kEnds) return launch_kernel<T, DS, kEnds, 128, 4>(p, s, blocks);
  const bool one = blocks <= device_info(-1).sm_count;
  if constexpr (scan_cols(DS) == 64) {
    if (one && mode == kOutputs) return launch_kernel<T, DS, kOutputs, 256, DS == 8 ? 2 : 4>(p, s, blocks);
  }
  if constexpr (DS <= 16) {
    if (one && mode == kStates) return launch_kernel<T, DS, kStates, 128, 2>(p, s, blocks);
  }
  if (mode == kStates) return launch_kernel<T, DS, kStates, 128, 4>(p, s, blocks);
  return launch_kernel<T, DS, kOutputs, 128, 4>(p, s, blocks);
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

template <typename T, int DS>
cudaError_t launch_ends(const ScanProblem &p, const ScanProblem &q, ScanSplit s) {
  s.launched = s.segs - 1;
  constexpr int kSmem = 2 * (int)sizeof(Smem<DS, kEnds>);
  static_assert(kSmem <= 48 * 1024, "no opt-in needed");
  const long blocks = 2L * p.B * s.launched * ((p.D + scan_cols(DS) - 1) / scan_cols(DS));
  LaunchTimer timer(kKSelectiveState, p.stream);
  scan_ends_kernel<T, DS><<<(unsigned)blocks, scan_threads(DS, 4) + 128, kSmem, p.stream>>>(p, q, s);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}
template <typename T>
cudaError_t launch_ends_ds(const ScanProblem &p, const ScanProblem &q, const ScanSplit &s) {
  return p.ds == 8    ? launch_ends<T, 8>(p, q, s)
         : p.ds == 16 ? launch_ends<T, 16>(p, q, s)
         : p.ds == 32 ? launch_ends<T, 32>(p, q, s)
                      : launch_ends<T, 64>(p, q, s);
}

cudaError_t join(const ScanProblem &p, const ScanSplit &s, const float *dS, int directions) {
  const long all = (long)p.B * p.D * p.ds;
  LaunchTimer timer(kKSelectiveState, p.stream);
  scan_join_kernel<<<dim3((unsigned)((all + 255) / 256), directions), 256, 0, p.stream>>>(s, p.A, p.S0, dS, p.B, p.D, p.ds);
  const cudaError_t e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

}  // namespace

// Segments of at least 256 tokens, in front of which the blocks of channels (of `cols`) take the fewest turns on the SMs,
// `per_sm` blocks each: a turn of two blocks an SM takes half as long again as one of one block, and the passes over
// segments' ends as long as 0.3 turns over all tokens.  Rows of a padded batch end early, whole blocks of theirs have
// nothing to do: two turns' worth of segments then (4 x up to 1021 x 520 x 32, gradient: 162 us for 219).
ScanSplit scan_split(const ScanProblem &p, int cols, int per_sm) {
  ScanSplit s{};
  const long sms = std::max(1, device_info(-1).sm_count), blocks = (long)p.B * ((p.D + cols - 1) / cols);
  const long most = std::max(1L, std::min(2 * per_sm * sms / blocks, p.N / 256));
  long segs = 1;
  if (p.lengths) {
    segs = most;
  } else {
    float least = 1e30f;
    for (long n = 1; n <= most; ++n) {
      const long all = blocks * n, turns = (all + per_sm * sms - 1) / (per_sm * sms);
      const float cost = (all <= sms ? 1.f : (per_sm == 2 ? 1.5f : 1.f) * turns) / n + (n > 1 ? 0.3f : 0.f);
      if (cost < least) least = cost, segs = n;
    }
  }
  s.len = (p.N + segs - 1) / segs;
  s.len = (s.len + kTok - 1) / kTok * kTok;
  s.segs = (int)std::max(1L, (p.N + s.len - 1) / s.len);
  return s;
}
namespace {
ScanSplit forward_split(const ScanProblem &p) { return scan_split(p, scan_cols(p.ds), 2); }
}  // namespace

size_t scan_workspace(const ScanProblem &p) {
  const ScanSplit s = forward_split(p);
  return s.segs == 1 ? 0 : sizeof(float) * (size_t)p.B * s.segs * p.D * (p.ds + 1);
}
size_t scan_workspace_any(ScanProblem p, size_t (*need)(const ScanProblem &)) {
  static const int some = 0;
  p.lengths = nullptr;
  const size_t plain = need(p);
  p.lengths = &some;  // whether there are lengths is all that counts
  return std::max(plain, need(p));
}

cudaError_t launch_scan_starts(const ScanProblem &p, const ScanSplit &s) {
  const cudaError_t e = launch(p, s, kEnds);
  return e != cudaSuccess ? e : join(p, s, nullptr, 1);
}

cudaError_t launch_scan_both_starts(const ScanProblem &p, const ScanSplit &s, const void *dout, const float *dS) {
  ScanProblem q = p;
  q.x = dout, q.ldx = p.D;
  const cudaError_t e = p.dt == LA_F32 ? launch_ends_ds<float>(p, q, s) : launch_ends_ds<__nv_bfloat16>(p, q, s);
  return e != cudaSuccess ? e : join(p, s, dS, 2);
}

cudaError_t launch_scan_states(const ScanProblem &p, const ScanSplit &s) { return launch(p, s, kStates); }

cudaError_t launch_selective_scan(const ScanProblem &p) {
  ScanSplit s = forward_split(p);
  if (s.segs > 1) {
    s.starts = (float *)p.ws;
    s.total = s.starts + (size_t)p.B * s.segs * p.D * p.ds;
    const cudaError_t e = launch_scan_starts(p, s);
    if (e != cudaSuccess) return e;
  }
  return launch(p, s, kOutputs);
}

}  // namespace la
