// Gradient of the selective state space scan.
//
// With a_t = e^{delta_t A}, dy = dout silu(z) and G_t the gradient of h_t (formulas of the forward in selective.cuh):
//   G_t = C_t dy_t + a_{t+1} G_{t+1},  behind the last token G = dS
//   dC_t,n = sum_c h dy,  dB_t,n = sum_c G delta x,  s1 = sum_n G B_n,  s2 = sum_n G (a h_{t-1}) A_n
//   dx = D dy + delta s1,  ddt = (x s1 + s2) softplus'(dt + bias),  dz = dout y silu'(z)
//   dA_n = sum_{b,t} G (a h_{t-1}) delta,  dD = sum dy x,  dbias = sum ddt,  dS0 = a_0 G_0.
//
// The states are not kept by the forward: a pass of the scan leaves the state in front of every chunk of 16 tokens, and
// this kernel goes through the chunks from the last to the first, with the scan's layout (a lane: four components, of
// d_state = 64 eight, of two channels) and three kinds of warps, a chunk apart:
//   1. around: rows in, steps, dy, B and C to shared memory; later dx, ddt, dz out, and dB, dC added over the warps;
//   2. forward: the recurrence again, leaving a_t h_{t-1} of every token in shared memory, y, and h dy summed to dC;
//   3. backward: G in registers, and what depends on it.  A lane reads the a h that its like wrote.
// Sums over the components are spread over a channel's lanes; the sums of dB and dC over channels are
// spread over a warp's channels, added over the block's warps, and leave as one partial sum a block of channels, which a
// last kernel adds in order.  No atomics: the gradient is the same from run to run.
//
// Shared memory's port bounds it (60 of its cycles a token and pair of warps, 81 % taken on the 128 SMs that have a block
// of 4 x 4096 x 2048 x 16), and two exponentials and about twenty issue slots a component: 833 us in bf16 (launches timed
// one by one: 650 here, 163 in the scan of states, 28 in the sums).  With one kind of warps and one channel a lane it took 1337 us; with
// results out before the next rows in, 944.  With y and dC in the third kind of warps 8 components took 826 us for 738,
// 16 876 for 866 (both with 35 us more in the scan of states than now).
#include <algorithm>

#include "internal.h"
#include "selective.cuh"

namespace la {
namespace {

constexpr int kAround = 128;  // threads of the first kind

// Tokens a chunk and channels a block: as many as keep the a h of two chunks within shared memory.
constexpr int grad_tokens(int ds) { return ds == 64 ? 8 : 16; }
__host__ __device__ constexpr int grad_cols(int ds) { return ds <= 16 ? 64 : 32; }

template <int DS>
struct Layout {
  static constexpr int kTok = grad_tokens(DS), kCols = grad_cols(DS), kRow = kCols + 8;  // floats between tokens of the sums' places
  static constexpr int kSN = DS == 64 ? 8 : 4;                   // components a lane
  static constexpr int kLanes = DS / kSN, kScan = kCols / 2 * kLanes, kWarps = kScan / 32;
  static constexpr int kThreads = kAround + 2 * kScan;
};

template <int DS>
struct Smem {
  using L = Layout<DS>;
  static constexpr int kTok = L::kTok;
  float4 ah[2][kTok][L::kSN / 2][L::kScan];
  struct In {
    float4 steps[kTok][L::kCols / 2];  // of two channels: delta, delta x; at step_slot
    float dy[kTok][L::kCols];
    float B[kTok][DS], C[kTok][DS];
  } in[3];
  struct Out {
    float s1[kTok][L::kRow], s2[kTok][L::kRow], y[kTok][L::kRow];
    float bc[kTok][L::kWarps][2 * DS];  // dB, dC of each warp's channels
  } out[2];
  float sums[2][kAround][8];  // dD, dbias of each thread around
};
// Chunks whose shares of dD and dbias a thread adds in registers, and then to its place in `sums`: chains of additions stay
// short in long sequences (over 65536 tokens equal shares lost 3e-5 of their sum).  834 us at 4 x 4096 x 2048 x 16 as without
// the places, 0.6 to 1.6 % more with 8, 32 and 64 components; both levels in registers 855 us, a loop around 32 chunks 838
// but in fp32 3 % more.
constexpr int kSumChunks = 32;

// Where channel c's sums and dy are in a token's row: eight threads that read eight channels each, four at a
// time, meet no bank twice.
__device__ __forceinline__ int row_place(int c) { return c ^ (c >> 3 & 4); }

// Barriers between the kinds of warps.
enum Bar { kIn = 1, kAhFull = 4, kAhFree = 6, kOutFull = 8, kOutFree = 10, kOwn = 12 };

// A sum that carries its rounding errors along.
__device__ __forceinline__ void add_carry(float2 &s, float2 &e, float2 x) {
  const float2 t = __fadd2_rn(s, x), b = __fadd2_rn(t, __fmul2_rn(s, both(-1.f)));
  const float2 rest = __fadd2_rn(s, __fmul2_rn(__fadd2_rn(t, __fmul2_rn(b, both(-1.f))), both(-1.f)));
  e = __fadd2_rn(e, __fadd2_rn(rest, __fadd2_rn(x, __fmul2_rn(b, both(-1.f)))));
  s = t;
}

template <typename T, int DS, bool kGate>
__global__ void __launch_bounds__(Layout<DS>::kThreads) scan_grad_kernel(const __grid_constant__ ScanGradProblem g, const __grid_constant__ ScanSplit s) {
  using L = Layout<DS>;
  constexpr int kTok = L::kTok, kCols = L::kCols, kScan = L::kScan, kLanes = L::kLanes, kSN = L::kSN, kPerWarp = 32 / kLanes;
  constexpr int kPairs = kSN / 2;                                // of components, a channel
  constexpr int kStep = kLanes < 4 ? 4 : kLanes;  // tokens whose sums over components are spread together
  constexpr int kBatch = 16 / kSN;                 // the same for sums over channels: the more, the fewer waits
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Smem<DS> &m = *reinterpret_cast<Smem<DS> *>(raw_smem);
  const ScanProblem &p = g.p;
  const int tid = threadIdx.x, lane = tid & 31;
  const int nb = (p.D + kCols - 1) / kCols;
  const int cb = blockIdx.x % nb;
  const long rest = blockIdx.x / nb;
  const int seg = (int)(rest % s.segs);
  const long b = rest / s.segs;
  const long n = row_length(p.lengths, b, p.N);
  const long begin = (long)seg * s.len, stop = min(begin + s.len, p.N), end = min(stop, n);
  const int chunks = end > begin ? (int)((end - begin + kTok - 1) / kTok) : 0;
  auto first_of = [&](int i) { return begin + (long)(chunks - 1 - i) * kTok; };  // the i-th chunk from the end
  const long state = (long)p.D * DS;
  float *columns = s.columns + (b * s.segs + seg) * (long)p.D * (DS + 2);

  if (tid < kAround) {
    constexpr int kPerRow = kCols / 8;  // threads a token
    const int row = tid / kPerRow, col = tid % kPerRow * 8, c8 = cb * kCols + col;
    const bool live = c8 < p.D && row < kTok;
    float2 bias[4], skip[4], dD[4], dbias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      bias[e] = live && p.dt_bias ? reinterpret_cast<const float2 *>(p.dt_bias + c8)[e] : both(0.f);
      skip[e] = live && p.Dskip ? reinterpret_cast<const float2 *>(p.Dskip + c8)[e] : both(0.f);
      dD[e] = dbias[e] = both(0.f);
    }
    put8(m.sums[0][tid], dD), put8(m.sums[1][tid], dbias);
    auto put_by = [&](float *to, float2 (&v)[4]) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = __fadd2_rn(v[e], reinterpret_cast<const float2 *>(to)[e]);
        reinterpret_cast<float2 *>(to)[e] = v[e];
        v[e] = both(0.f);
      }
    };
    const T *x = (const T *)p.x + b * p.N * p.ldx + c8, *dt = (const T *)p.delta + b * p.N * p.ldt + c8;
    const T *z = kGate ? (const T *)p.z + b * p.N * p.ldz + c8 : nullptr;
    const long out0 = b * p.N * p.D + c8;
    const T *dout = (const T *)g.dout + out0;
    if (live) {  // tokens past the row's end: zero gradients
      const float2 zero[4] = {both(0.f), both(0.f), both(0.f), both(0.f)};
      for (long t = max(begin, end) + row; t < stop; t += kTok) {
        put8((T *)g.dx + out0 + t * p.D, zero), put8((T *)g.ddt + out0 + t * p.D, zero);
        if (kGate) put8((T *)g.dz + out0 + t * p.D, zero);
      }
    }
    // rows of B and C, eight components a piece
    constexpr int kPieces = 2 * kTok * DS / 8, kEach = (kPieces + kAround - 1) / kAround, kPR = DS / 8;
    struct Rows {
      Raw<T> x, t, z, d;
    } next, done;  // of the chunk that goes in next; of the one that comes out (read again, from L2: there is no place)
    Raw<T> rb[kEach];
    auto rows_of = [&](Rows &r, long t) {
      r.x.zero(), r.t.zero(), r.z.zero(), r.d.zero();
      if (live && t < end) {
        r.x.load(x + t * p.ldx), r.t.load(dt + t * p.ldt), r.d.load(dout + t * p.D);
        if (kGate) r.z.load(z + t * p.ldz);
      }
    };
    auto load = [&](long t0) {
      rows_of(next, t0 + row);
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int k = tid + i * kAround, which = k >= kPieces / 2, j = which ? k - kPieces / 2 : k;
        rb[i].zero();
        if (k < kPieces && t0 + j / kPR < end)
          rb[i].load((which ? (const T *)p.Cm + (b * p.N + t0 + j / kPR) * p.ldc : (const T *)p.Bm + (b * p.N + t0 + j / kPR) * p.ldb) +
                     j % kPR * 8);
      }
    };
    if (chunks) load(first_of(0));
    int at = 0;  // i mod 3
    for (int i = 0; i < chunks + 2; ++i) {
      if (i < chunks) {
        typename Smem<DS>::In &to = m.in[at];
        if (row < kTok) {
          const bool in = first_of(i) + row < end;
          float2 xv[4], tv[4], dv[4], zv[4];
          next.x.get(xv), next.t.get(tv), next.d.get(dv);
          if (kGate) next.z.get(zv);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 d = __fadd2_rn(tv[e], bias[e]);
            if (p.softplus) d = softplus2(d);
            float2 u = __fmul2_rn(d, xv[e]);
            if (!in) d = u = both(0.f);
            to.steps[row][step_slot(col / 2 + e)] = make_float4(d.x, u.x, d.y, u.y);
            if (kGate) dv[e] = __fmul2_rn(dv[e], __fmul2_rn(zv[e], Sigmoid2(zv[e]).s));
            if (!in) dv[e] = both(0.f);
          }
#pragma unroll
          for (int e = 0; e < 4; e += 2) st4(&to.dy[row][row_place(col + 2 * e)], dv[e].x, dv[e].y, dv[e + 1].x, dv[e + 1].y);
        }
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const int k = tid + j * kAround;
          float2 v[4];
          rb[j].get(v);
          if (k < kPieces) put8((k >= kPieces / 2 ? &to.C[0][0] + (k - kPieces / 2) * 8 : &to.B[0][0] + k * 8), v);
        }
        if (i + 1 < chunks) load(first_of(i + 1));
        bar_arrive<kAround + kScan>(kIn + at);
      }
      if (i >= 2) {
        const int o = i - 2;
        const long t0 = first_of(o), t = t0 + row;
        rows_of(done, t);
        if (o % kSumChunks == 0) put_by(m.sums[0][tid], dD), put_by(m.sums[1][tid], dbias);  // while this chunk is waited for
        bar_sync<kAround + kScan>(kOutFull + (o & 1));
        const typename Smem<DS>::Out &from = m.out[o & 1];
        const typename Smem<DS>::In &in = m.in[at == 2 ? 0 : at + 1];
        if (live && t < end) {
          float2 xv[4], tv[4], dv[4], zv[4], ox[4], ot[4], oz[4], s1v[4], s2v[4], yv[4], dyv[4];
          auto row8 = [&](float2 (&v)[4], const float *of) {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float4 f = *reinterpret_cast<const float4 *>(of + row_place(col + 2 * e));
              v[e] = make_float2(f.x, f.y), v[e + 1] = make_float2(f.z, f.w);
            }
          };
          row8(s1v, from.s1[row]), row8(s2v, from.s2[row]), row8(dyv, in.dy[row]);
          if (kGate) row8(yv, from.y[row]);
          done.x.get(xv), done.t.get(tv), done.d.get(dv);
          if (kGate) done.z.get(zv);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 s1 = s1v[e], s2 = s2v[e], dy = dyv[e];
            const float4 st = in.steps[row][step_slot(col / 2 + e)];
            ox[e] = __ffma2_rn(make_float2(st.x, st.z), s1, __fmul2_rn(skip[e], dy));
            ot[e] = __ffma2_rn(xv[e], s1, __fmul2_rn(s2, both(0.693147181f)));  // A carries log2 e
            if (p.softplus) ot[e] = __fmul2_rn(ot[e], Sigmoid2(__fadd2_rn(tv[e], bias[e])).s);
            dD[e] = __ffma2_rn(dy, xv[e], dD[e]);
            dbias[e] = __fadd2_rn(dbias[e], ot[e]);
            if (kGate) {
              const float2 y = __ffma2_rn(skip[e], xv[e], yv[e]);
              const Sigmoid2 sg(zv[e]);
              const float2 slope = __ffma2_rn(__fmul2_rn(zv[e], sg.s), sg.one_less(), sg.s);
              oz[e] = __fmul2_rn(__fmul2_rn(dv[e], y), slope);
            }
          }
          const long to = out0 + t * p.D;
          put8((T *)g.dx + to, ox), put8((T *)g.ddt + to, ot);
          if (kGate) put8((T *)g.dz + to, oz);
        }
        for (int j = tid; j < kTok * 2 * DS; j += kAround) {
          const int r = j / (2 * DS), k = j % (2 * DS);
          float v = from.bc[r][0][k];
#pragma unroll
          for (int w = 1; w < L::kWarps; ++w) v += from.bc[r][w][k];
          if (t0 + r < end) s.bc[((long)cb * p.B * p.N + b * p.N + t0 + r) * (2 * DS) + k] = v;
        }
        if (i < chunks) bar_arrive<kAround + kScan>(kOutFree + (o & 1));
      }
      at = at == 2 ? 0 : at + 1;
    }
    // dD and the bias's gradient: threads of the same channels in order
    put_by(m.sums[0][tid], dD), put_by(m.sums[1][tid], dbias);
    bar_sync<kAround>(kOwn);
    for (int j = tid; j < 2 * kCols; j += kAround) {
      const int which = j / kCols, c = j % kCols;
      if (cb * kCols + c >= p.D) continue;
      float v = 0.f;
      for (int r = 0; r < kTok; ++r) v += m.sums[which][r * kPerRow + c / 8][c % 8];
      columns[state + (long)which * p.D + cb * kCols + c] = v;
    }
    return;
  }

  const bool forward = tid < kAround + kScan;
  const int me = tid - kAround - (forward ? 0 : kScan), warp = me >> 5;
  const int q = lane % kLanes, num = lane / kLanes, ch = (warp * kPerWarp + num) * 2;
  const int c = cb * kCols + ch, slot = step_slot(ch / 2), place = row_place(ch);  // and the next channel; D is even
  const bool mine = c < p.D;
  const long at = (long)c * DS + kSN * q;  // in a state
  float2 A[2][kPairs];
  auto get = [&](float2 (&v)[2][kPairs], const float *from) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < kPairs; e += 2) {
        const float4 f = mine && from ? *reinterpret_cast<const float4 *>(from + at + i * DS + 2 * e) : make_float4(0.f, 0.f, 0.f, 0.f);
        v[i][e] = make_float2(f.x, f.y), v[i][e + 1] = make_float2(f.z, f.w);
      }
  };
  auto put = [&](float *to, const float2 (&v)[2][kPairs]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < kPairs; e += 2) st4(to + at + i * DS + 2 * e, v[i][e].x, v[i][e].y, v[i][e + 1].x, v[i][e + 1].y);
  };
  auto read = [&](float2 (&v)[kPairs], const float *from) {
#pragma unroll
    for (int e = 0; e < kPairs; e += 2) {
      const float4 f = *reinterpret_cast<const float4 *>(from + 2 * e);
      v[e] = make_float2(f.x, f.y), v[e + 1] = make_float2(f.z, f.w);
    }
  };
  get(A, p.A);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < kPairs; ++e) A[i][e] = rate(A[i][e]);

  // Sums over the warp's channels of kSN values of each of kBatch tokens from t0 on: dB (first = 0) or dC (first = DS).
  auto put_sums = [&](float (&v)[kBatch * kSN], typename Smem<DS>::Out &out, int t0, int first) {
    spread_sum<kPerWarp, kBatch * kSN, kLanes>(v, num);
#pragma unroll
    for (int r = 0; r < kBatch * kSN / kPerWarp; ++r) {
      const int k = num + r * kPerWarp;
      out.bc[t0 + k / kSN][warp][first + kSN * q + k % kSN] = v[r];
    }
  };

  if (forward) {
    float2 h[2][kPairs], next[2][kPairs];
    auto states_of = [&](int i) { return s.chunk_states + (b * s.all_chunks + first_of(i) / kTok) * state; };
    if (chunks) get(next, states_of(0));
    int buf = 0;
    for (int i = 0; i < chunks; ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < kPairs; ++e) h[k][e] = next[k][e];
      if (i + 1 < chunks) get(next, states_of(i + 1));
      bar_sync<kAround + kScan>(kIn + buf);
      if (i >= 2) {
        bar_sync<2 * kScan>(kAhFree + (i & 1));
        bar_sync<kAround + kScan>(kOutFree + (i & 1));
      }
      const typename Smem<DS>::In &in = m.in[buf];
      typename Smem<DS>::Out &out = m.out[i & 1];
      auto &ah = m.ah[i & 1];
      struct Token {  // as below
        float4 d;
        float2 dy, B[kPairs], C[kPairs];
      } now, then;
      auto fetch = [&](Token &v, int t) {
        v.d = in.steps[t][slot];
        v.dy = *reinterpret_cast<const float2 *>(&in.dy[t][place]);
        read(v.B, &in.B[t][kSN * q]);
        read(v.C, &in.C[t][kSN * q]);
      };
      fetch(now, 0);
#pragma unroll 4
      for (int i0 = 0; i0 < kTok; i0 += kStep) {
        float y[2 * kStep], sums[kBatch * kSN];  // of the two channels; of dC
#pragma unroll
        for (int j = 0; j < kStep; ++j) {
          const int t = i0 + j;
          if (t + 1 < kTok) fetch(then, t + 1);
          float2 dC[kPairs];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float2 dd = both(k ? now.d.z : now.d.x), u = both(k ? now.d.w : now.d.y), dyk = both(k ? now.dy.y : now.dy.x);
            float2 v[kPairs], t3 = both(0.f);
#pragma unroll
            for (int e = 0; e < kPairs; ++e) {
              v[e] = __fmul2_rn(decay(dd, A[k][e]), h[k][e]);
              h[k][e] = __ffma2_rn(u, now.B[e], v[e]);
              dC[e] = k ? __ffma2_rn(h[k][e], dyk, dC[e]) : __fmul2_rn(h[k][e], dyk);
              if (kGate) t3 = e ? __ffma2_rn(h[k][e], now.C[e], t3) : __fmul2_rn(h[k][e], now.C[e]);
            }
            if (kGate) y[k * kStep + j] = t3.x + t3.y;
#pragma unroll
            for (int e = 0; e < kPairs; e += 2) ah[t][(k * kPairs + e) / 2][me] = make_float4(v[e].x, v[e].y, v[e + 1].x, v[e + 1].y);
          }
#pragma unroll
          for (int e = 0; e < kPairs; ++e) sums[j % kBatch * kSN + 2 * e] = dC[e].x, sums[j % kBatch * kSN + 2 * e + 1] = dC[e].y;
          if (j % kBatch == kBatch - 1) put_sums(sums, out, t - (kBatch - 1), DS);
          now = then;
        }
        if (kGate) {
          spread_sum<kLanes, 2 * kStep, 1>(y, q);
          constexpr int kHave = kStep / kLanes;
#pragma unroll
          for (int v = 0; v < kHave; ++v) *reinterpret_cast<float2 *>(&out.y[i0 + v * kLanes + q][place]) = make_float2(y[v], y[kHave + v]);
        }
      }
      bar_arrive<2 * kScan>(kAhFull + (i & 1));
      buf = buf == 2 ? 0 : buf + 1;
    }
    return;
  }
  float2 G[2][kPairs], dA[2][kPairs], lost[2][kPairs];
  get(G, s.segs > 1 ? s.rev_starts + (b * s.segs + seg) * state : g.dS ? g.dS + b * state : nullptr);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < kPairs; ++e) dA[k][e] = lost[k][e] = both(0.f);
  int buf = 0;
  for (int i = 0; i < chunks; ++i) {
    bar_sync<2 * kScan>(kAhFull + (i & 1));
    const typename Smem<DS>::In &in = m.in[buf];
    typename Smem<DS>::Out &out = m.out[i & 1];
    const auto &ah = m.ah[i & 1];
    float2 part[2][kPairs];  // of dA
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < kPairs; ++e) part[k][e] = both(0.f);
    // a token's values are on their way while the one behind it is worked on (the compiler does not move these loads
    // across the stores of sums)
    struct Token {
      float4 d;
      float2 dy, B[kPairs], C[kPairs], ah[2][kPairs];
    } now, then;
    auto fetch = [&](Token &v, int t) {
      v.d = in.steps[t][slot];
      v.dy = *reinterpret_cast<const float2 *>(&in.dy[t][place]);
      read(v.B, &in.B[t][kSN * q]);
      read(v.C, &in.C[t][kSN * q]);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < kPairs; e += 2) {
          const float4 f = ah[t][(k * kPairs + e) / 2][me];
          v.ah[k][e] = make_float2(f.x, f.y), v.ah[k][e + 1] = make_float2(f.z, f.w);
        }
    };
    fetch(now, kTok - 1);
#pragma unroll 1
    for (int i0 = kTok - kStep; i0 >= 0; i0 -= kStep) {
      float s1[2 * kStep], s2[2 * kStep];  // of the first channel, of the second
      float sums[kBatch * kSN];            // of dB
#pragma unroll
      for (int j = kStep - 1; j >= 0; --j) {
        const int t = i0 + j;
        if (t > 0) fetch(then, t - 1);
        const float4 d = now.d;
        const float2 dy = now.dy;
        const auto &B = now.B, &C = now.C;
        float2 dB[kPairs];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float2 dd = both(k ? d.z : d.x), u = both(k ? d.w : d.y), dyk = both(k ? dy.y : dy.x);
          const auto &v = now.ah[k];
          float2 t1 = both(0.f), t2 = both(0.f);
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            G[k][e] = __ffma2_rn(C[e], dyk, G[k][e]);
            dB[e] = k ? __ffma2_rn(G[k][e], u, dB[e]) : __fmul2_rn(G[k][e], u);
            t1 = e ? __ffma2_rn(G[k][e], B[e], t1) : __fmul2_rn(G[k][e], B[e]);
            const float2 w = __fmul2_rn(G[k][e], v[e]);
            t2 = e ? __ffma2_rn(w, A[k][e], t2) : __fmul2_rn(w, A[k][e]);
            part[k][e] = __ffma2_rn(w, dd, part[k][e]);
            G[k][e] = __fmul2_rn(decay(dd, A[k][e]), G[k][e]);
          }
          s1[k * kStep + j] = t1.x + t1.y, s2[k * kStep + j] = t2.x + t2.y;
        }
#pragma unroll
        for (int e = 0; e < kPairs; ++e) sums[j % kBatch * kSN + 2 * e] = dB[e].x, sums[j % kBatch * kSN + 2 * e + 1] = dB[e].y;
        if (j % kBatch == 0) put_sums(sums, out, t, 0);
        now = then;
      }
      spread_sum<kLanes, 2 * kStep, 1>(s1, q);
      spread_sum<kLanes, 2 * kStep, 1>(s2, q);
      constexpr int kHave = kStep / kLanes;
#pragma unroll
      for (int v = 0; v < kHave; ++v) {
        const int t = i0 + v * kLanes + q;
        *reinterpret_cast<float2 *>(&out.s1[t][place]) = make_float2(s1[v], s1[kHave + v]);
        *reinterpret_cast<float2 *>(&out.s2[t][place]) = make_float2(s2[v], s2[kHave + v]);
      }
    }
    if (i + 2 < chunks) bar_arrive<2 * kScan>(kAhFree + (i & 1));
    bar_arrive<kAround + kScan>(kOutFull + (i & 1));
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < kPairs; ++e) add_carry(dA[k][e], lost[k][e], part[k][e]);
    buf = buf == 2 ? 0 : buf + 1;
  }
  if (!mine) return;
  if (seg == 0 && g.dS0) put(g.dS0 + b * state, G);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < kPairs; ++e) dA[k][e] = __fadd2_rn(dA[k][e], lost[k][e]);
  put(columns, dA);
}

// dB and dC from the partial sums of the blocks of channels: a thread a token and component.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(const __grid_constant__ ScanGradProblem g, const __grid_constant__ ScanSplit s) {
  const ScanProblem &p = g.p;
  const int cols = grad_cols(p.ds), ds2 = 2 * p.ds, nb = (p.D + cols - 1) / cols;
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
  constexpr int kCols = grad_cols(DS);
  const long blocks = (long)p.B * s.segs * ((p.D + kCols - 1) / kCols);
  {
    LaunchTimer timer(kKSelectiveBackward, p.stream);
    void *args[] = {const_cast<ScanGradProblem *>(&g), const_cast<ScanSplit *>(&s)};
    e = cudaLaunchKernel(fn, dim3((unsigned)blocks), dim3(Layout<DS>::kThreads), args, sizeof(Smem<DS>), p.stream);
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
  const int cols = grad_cols(p.ds);
  q.bc = take((size_t)((p.D + cols - 1) / cols) * p.B * p.N * 2 * p.ds);
  q.columns = take(rows * p.D * (p.ds + 2));
  q.all = o;
  return q;
}
ScanSplit grad_split(const ScanProblem &p) {
  ScanSplit s = scan_split(p, grad_cols(p.ds), 1);
  s.chunk = grad_tokens(p.ds);
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
    e = launch_scan_both_starts(p, s, g.dout, g.dS);
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
