// Gradient of gated linear attention on the sm_103a tensor cores (bf16, d_k = d_v = D in {64, 128}).
//
// The state pass (gated_state_tc.cu) leaves, for every chunk of 128 tokens, the state S before it and
// the gradient R of the state behind it, both as bf16 pairs.  Then every chunk is independent; one
// CTA takes one chunk at a time.  With W_ij = 2^{c_i - c_j} for j <= i, else 0:
//   P^T = K Q^T,  D^T = V dO^T                              fp32 in tensor memory, keys in the lanes
//   dQ  = 2^{c_i} (dO S^T)        + (W D) K
//   dK  = 2^{c_T - c_j} (V R^T)   + (W D)^T Q
//   dV  = 2^{c_T - c_j} (K R)     + (W P)^T dO
//   dg_t = sum_{j < t <= i} W_ij P_ij D_ij + sum_{i >= t} q_i . [2^{c_i} S do_i]
//          + sum_{j < t} k_j . [2^{c_T - c_j} R v_j] + 2^{c_T} <S, R>
// dg is an fp32 result: its first term comes from the fp32 products before any rounding, the next
// two from dQ's and dK's first products, which take S and R as pairs, the last from the stored pairs.
// The first term adds only pairs on both sides of t, in blocks of 32 tokens: pairs of earlier keys and
// later queries by block, t's own block's keys and queries by row and column sums, and inside the block by
// each key's sums over the queries from t on.  (Row sums less column sums, summed from the end, would cancel all
// pairs behind t: a strong decay's gradient is small beside them, and a reset's is 0.)  So no term is a
// difference of larger ones, and no error is carried from chunk to chunk.  dQ, dK and dV
// are bf16: W D, W P and dV's R are rounded to bf16 once.
//
// Tensor memory holds P^T and D^T, dQ and dK; W P overwrites P^T and dV takes D^T's columns.  The
// first products are scaled by row in tensor memory, then the second ones accumulate on top.
// HBM bounds it at 14 D bytes a token of inputs and results plus 8 D of states (D = 128: 8.1 us a
// chunk at an SM's share); the tensor work is 13 products of 128 x 128 x D.  Measured at 4 x 16 x 8192,
// D = 128: 260 us (5.6 TB/s).  Of these dg's pairs by blocks take 4 and the test for cuts 2; before these two
// it took as long without the score warps' work, and 34 us less without the second reading of the states for
// <S, R> (from L2).  At D = 64 a chunk's chain of steps bounds it, 16000 cycles; two chunks' tokens in shared
// memory and a place for results beside W D's, for which there is room, took 3 % off and were not kept.
//
// Every warp runs its code once a chunk, out of a cold instruction cache (the first of a score warp's
// four equal turns takes 4000 cycles, the others 1500): less code is faster.  32-bit quotients in place
// of 64-bit ones took 269 to 258 us, turns of a loop unrolled by two 280.
//
// Two chunks overlap: the score warps weigh a chunk's products while the row warps still write the
// previous chunk's results; the score columns are free for it as soon as dV is read.
//
// Warps: 0 TMA, 1 MMA and TMEM owner, 2 running sums and dg, 3-6 <S, R>, 7-14 scores, 15-22 rows
// (scales, dot products, results).
// Every wait is bounded (tc_ptx.cuh).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "gated_tc.cuh"

namespace la {
namespace {
using namespace gtc;

constexpr int kThreads = 736;
constexpr int kWarpGate = 2, kWarpDot = 3, kWarpScore = 7, kWarpRow = 15;
constexpr uint32_t kBarScore = 1;
constexpr int kRing = 2;

template <int D>
struct Lay {
  static constexpr uint32_t kTile = D / 64 * kBlk;  // 128 tokens
  static constexpr uint32_t kState = D * D * 2;     // S or R, hi or lo
  static constexpr uint32_t Q = 0;
  static constexpr uint32_t K = Q + kTile;
  static constexpr uint32_t dO = K + kTile;
  static constexpr uint32_t V = dO + kTile;
  static constexpr uint32_t Ring = V + kTile;
  static constexpr uint32_t WD = Ring + kRing * kState;  // W D [keys][queries] bf16; then results on their way out
  static constexpr uint32_t Gate = WD + 2 * kBlk;        // hi 128, lo 128
  static constexpr uint32_t Buf = Gate + 2 * kC * 4;     // 320 floats
  static constexpr uint32_t Red = Buf + 320 * 4;         // 4 floats
  static constexpr uint32_t Bars = Red + 16;
  static constexpr int kNumBars = 3 + 2 * kRing + 17;
  static constexpr uint32_t Misc = Bars + kNumBars * 8;
  static constexpr uint32_t Bytes = Misc + 16;
};
static_assert(Lay<128>::Bytes <= 232448, "shared memory budget");
constexpr uint32_t kColP = 0, kColD = 128, kColQ = 256, kColK = 384;  // dV in D's columns

struct Params {
  CUtensorMap tq, tk, tv, td;  // boxes of 64 x 128
  CUtensorMap ts, tr;          // tiles of S and R, boxes of one part
  CUtensorMap oq, ok, ov;      // dq, dk, dv: boxes of 64 x 32
  const float *g;
  const int *lengths;
  const uint8_t *s_tiles, *r_tiles;
  __nv_bfloat16 *dq, *dk, *dv;
  float *dg;
  float *mail;  // [CTAs][4][128] a token's dg inside the chunk (two chunks in turn), what it adds up to it, and behind it
  long N;
  uint32_t n, items;  // chunks a head, all chunks (below 2^31)
  int H;
  bool wide;  // dq, dk, dv are 32-byte aligned
};

// Place of what the keys [32 q, 32 q + 32) add to query i > 32 q + 31, packed.  The first 32 places of
// each q hold, by key, what the other half of the queries adds.
__device__ __forceinline__ int part_at(int q, int i) { return q * 128 - 16 * q * (q - 1) + i - 32 * q; }

// Sum over the warp's lanes of x[c], returned by lanes c and c + 16.
__device__ __forceinline__ float column_sums(uint32_t (&x)[16], int lane) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < o; ++k) {
      const bool up = lane & o;
      const uint32_t give = up ? x[k] : x[k + o], keep = up ? x[k + o] : x[k];
      x[k] = __float_as_uint(__uint_as_float(keep) + __uint_as_float(__shfl_xor_sync(0xffffffffu, give, o)));
    }
  const float s = __uint_as_float(x[0]);
  return s + __shfl_xor_sync(0xffffffffu, s, 16);
}

// Dot of 32 fp32 values (raw bits) with 32 bf16 values of a swizzled row.
__device__ __forceinline__ float dot_row32(const uint32_t (&r)[32], const uint8_t *blk, int row, int col0) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint4 x = *reinterpret_cast<const uint4 *>(blk + sw128_offset(row, col0 + 8 * e));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int m = 0; m < 4; ++m)
      s = __ffma2_rn(make_float2(__uint_as_float(w[m] << 16), __uint_as_float(w[m] & 0xffff0000u)),
                     make_float2(__uint_as_float(r[8 * e + 2 * m]), __uint_as_float(r[8 * e + 2 * m + 1])), s);
  }
  return s.x + s.y;
}

__device__ __forceinline__ float dot_pairs(uint4 ah, uint4 al, uint4 bh, uint4 bl, float s) {
  const uint32_t a[4] = {ah.x, ah.y, ah.z, ah.w}, b[4] = {al.x, al.y, al.z, al.w}, c[4] = {bh.x, bh.y, bh.z, bh.w},
                 d[4] = {bl.x, bl.y, bl.z, bl.w};
  float2 t = make_float2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    auto f2 = [](uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); };
    t = __ffma2_rn(__fadd2_rn(f2(a[e]), f2(b[e])), __fadd2_rn(f2(c[e]), f2(d[e])), t);
  }
  return s + (t.x + t.y);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) gated_grad_tc_kernel(const __grid_constant__ Params p) {
  using L = Lay<D>;
  constexpr uint32_t kState = L::kState;
  extern __shared__ __align__(1024) uint8_t sm[];
  if (smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_gated_status, kAbortMisaligned);
    return;
  }
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::Bars);
  uint64_t *full_kq = bars, *full_v = bars + 1, *full_d = bars + 2, *ring_full = bars + 3, *ring_free = ring_full + kRing,
           *b0 = ring_free + kRing, *tok_free = b0, *gate_full = b0 + 1, *e_full = b0 + 2, *el_done = b0 + 3,
           *q_in = b0 + 4, *k_in = b0 + 5, *v_in = b0 + 6, *x_ready = b0 + 7, *out_full = b0 + 8, *out_free = b0 + 9,
           *dg_in = b0 + 10, *dot_full = b0 + 11, *dot_free = b0 + 12,
           *v_free = b0 + 13, *d_free = b0 + 14, *in_full = b0 + 15;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::Misc);
  volatile uint32_t *abort_word = reinterpret_cast<volatile uint32_t *>(sm + L::Misc + 4);
  uint64_t *drain = reinterpret_cast<uint64_t *>(sm + L::Misc + 8);
  unsigned int *status = &g_gated_status;
  float *hi = reinterpret_cast<float *>(sm + L::Gate), *lo = hi + kC;
  float *buf = reinterpret_cast<float *>(sm + L::Buf), *red = reinterpret_cast<float *>(sm + L::Red);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(full_kq, 1);
    mbar_init(full_v, 1);
    mbar_init(full_d, 1);
    mbar_init(v_free, 1);
    for (int s = 0; s < kRing; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_free[s], 1);
    }
    mbar_init(tok_free, 1);
    mbar_init(gate_full, 32);
    mbar_init(e_full, 1);
    mbar_init(el_done, 256);
    mbar_init(q_in, 1);
    mbar_init(k_in, 1);
    mbar_init(v_in, 1);
    mbar_init(x_ready, 256);
    mbar_init(out_full, 1);
    mbar_init(out_free, 256);
    mbar_init(d_free, 256);
    mbar_init(dg_in, 256 + 256);
    mbar_init(&in_full[0], 128);  // by parity: the gate warp may still have a chunk to wait for when the next is through
    mbar_init(&in_full[1], 128);
    mbar_init(dot_full, 4);
    mbar_init(dot_free, 32);
    mbar_init(drain, 1);
    *abort_word = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the states are the previous kernel's

  // every role walks over the same chunks; `it` counts those with tokens
  struct Item {
    long bh, t0;
    int tv;
  };
  // (32-bit quotients: every warp's code is run once a chunk, out of a cold instruction cache)
  auto item = [&](uint32_t x) -> Item {
    Item r;
    const uint32_t bh = x / p.n;
    r.bh = bh;
    r.t0 = (long)(x - bh * p.n) * kC;
    const long len = p.lengths ? row_length(p.lengths, bh / (uint32_t)p.H, p.N) : p.N;
    r.tv = (int)max(0L, min((long)kC, len - r.t0));
    return r;
  };

  if (warp == 0) {
    if (lane == 0) {
      int it = 0, ring = 0;
      int kq = 0, vd = 0;  // tiles issued
      bool ok = true;
      auto piece = [&](const CUtensorMap *map, uint32_t x, int part) {
        const int s = ring % kRing;
        if (ring >= kRing) ok = ok && mbar_wait(&ring_free[s], (ring / kRing - 1) & 1, abort_word, status);
        if (!ok) return;
        mbar_arrive_expect_tx(&ring_full[s], kState);
        tma_load_3d(sm + L::Ring + s * kState, map, &ring_full[s], 0, 0, (int)(2 * x + part) * (D / 64));
        ++ring;
      };
      auto tile = [&](uint32_t at, const CUtensorMap *map, uint64_t *bar, const Item &w) {
        for (int b = 0; b < D / 64; ++b) tma_load_3d(sm + at + b * kBlk, map, bar, 64 * b, (int)w.t0, (int)w.bh);
      };
      for (uint32_t x = blockIdx.x; x < p.items && ok; x += gridDim.x) {
        const Item w = item(x);
        if (w.tv == 0) continue;
        piece(&p.ts, x, 0);
        piece(&p.ts, x, 1);
        if (ok && it > 0) ok = mbar_wait(v_free, (it - 1) & 1, abort_word, status);
        if (!ok) break;
        mbar_arrive_expect_tx(full_v, L::kTile);
        tile(L::V, &p.tv, full_v, w);
        vd = it + 1;
        if (it > 0) ok = mbar_wait(tok_free, (it - 1) & 1, abort_word, status);
        if (!ok) break;
        mbar_arrive_expect_tx(full_kq, 2 * L::kTile);
        tile(L::K, &p.tk, full_kq, w);
        tile(L::Q, &p.tq, full_kq, w);
        mbar_arrive_expect_tx(full_d, L::kTile);
        tile(L::dO, &p.td, full_d, w);
        kq = ++it;
        piece(&p.tr, x, 0);
        piece(&p.tr, x, 1);
      }
      for (int r = max(0, ring - kRing); r < ring; ++r) wait_drain(&ring_full[r % kRing], (r / kRing) & 1, status);
      if (kq) wait_drain(full_kq, (kq - 1) & 1, status), wait_drain(full_d, (kq - 1) & 1, status);
      if (vd) wait_drain(full_v, (vd - 1) & 1, status);
    }
  } else if (warp == 1) {
    constexpr uint32_t iE = idesc_bf16_f32(128, 128, 0, 0), iKK = idesc_bf16_f32(128, D, 0, 0),
                       iKM = idesc_bf16_f32(128, D, 0, 1), iMM = idesc_bf16_f32(128, D, 1, 1);
    constexpr int kDs = D / 16;
    constexpr uint32_t kSBlk = D * 128;  // a 64-column block of S or R
    const bool leader = elect_one();
    const uint32_t tP = tmem + kColP, tD = tmem + kColD, tQ = tmem + kColQ, tK = tmem + kColK;
    const uint32_t sQ = smem_u32(sm + L::Q), sK = smem_u32(sm + L::K), sV = smem_u32(sm + L::V),
                   sO = smem_u32(sm + L::dO), sW = smem_u32(sm + L::WD), sR = smem_u32(sm + L::Ring);
    int it = 0;
    for (uint32_t x = blockIdx.x; x < p.items; x += gridDim.x) {
      if (item(x).tv == 0) continue;
      const uint32_t ph = it & 1;
      // the chunk's pieces S hi, S lo, R hi, R lo take the ring's two places in turn
      static_assert(kRing == 2, "places by parity");
      if (p.lengths && !warp_wait(gate_full, ph, abort_word)) break;  // padding tokens are cleared
      if (!warp_wait(full_kq, ph, abort_word)) break;
      // the columns of P: the previous W P is read by the previous dV's product, in issue order
      tc_fence_after();
      if (leader) product<kDs, kK, kK>(tP, kbase(sK), kbase(sQ), iE, false);
      __syncwarp();
      if (!warp_wait(full_v, ph, abort_word) || !warp_wait(full_d, ph, abort_word)) break;
      if (it > 0 && !warp_wait(d_free, ph ^ 1, abort_word)) break;
      tc_fence_after();
      if (leader) {
        product<kDs, kK, kK>(tD, kbase(sV), kbase(sO), iE, false);
        mma_commit(e_full);
      }
      __syncwarp();
      if (it > 0 && !warp_wait(out_free, ph ^ 1, abort_word)) break;
      // dQ = dO S^T, both parts of S
      if (!warp_wait(&ring_full[0], 0, abort_word)) break;
      tc_fence_after();
      if (leader) {
        product<kDs, kK, kK, kBlk, kSBlk>(tQ, kbase(sO), kbase(sR), iKK, false);
        mma_commit(&ring_free[0]);
      }
      __syncwarp();
      if (!warp_wait(&ring_full[1], 0, abort_word)) break;
      if (leader) {
        product<kDs, kK, kK, kBlk, kSBlk>(tQ, kbase(sO), kbase(sR + kState), iKK, true);
        mma_commit(&ring_free[1]);
        mma_commit(q_in);
      }
      __syncwarp();
      // dK = V R^T; R's high part stays for dV
      if (!warp_wait(&ring_full[0], 1, abort_word)) break;
      if (leader) product<kDs, kK, kK, kBlk, kSBlk>(tK, kbase(sV), kbase(sR), iKK, false);
      __syncwarp();
      if (!warp_wait(&ring_full[1], 1, abort_word)) break;
      if (leader) {
        product<kDs, kK, kK, kBlk, kSBlk>(tK, kbase(sV), kbase(sR + kState), iKK, true);
        mma_commit(&ring_free[1]);
        mma_commit(v_free);
        mma_commit(k_in);
      }
      __syncwarp();
      // dV = K R, over D^T once that is read
      if (!warp_wait(el_done, ph, abort_word)) break;
      tc_fence_after();
      if (leader) {
        product<kDs, kK, kMN, kBlk, kSBlk>(tD, kbase(sK), mnbase(sR, kSBlk), iKM, false);
        mma_commit(&ring_free[0]);
        mma_commit(v_in);
      }
      __syncwarp();
      if (!warp_wait(x_ready, ph, abort_word)) break;
      tc_fence_after();
      if (leader) {
        product_ts<kMN>(tD, tP, mnbase(sO), iKM, true);
        product<8, kK, kMN>(tK, kbase(sW), mnbase(sQ), iKM, true);
        product<8, kMN, kMN>(tQ, mnbase(sW), mnbase(sK), iMM, true);
        mma_commit(tok_free);
        mma_commit(out_full);
      }
      __syncwarp();
      ++it;
    }
    if (leader) {
      mma_commit(drain);
      wait_drain(drain, 0, status);
    }
  } else if (warp == kWarpGate) {
    // ---- running sums for the next chunk, dg of the current one ----
    int it = 0;
    auto fetch = [&](const Item &w) { return load_gates(p.g + w.bh * p.N + w.t0, w.tv, lane); };
    auto gates = [&](const Item &w, float4 g) -> bool {
      scan_gates(g, lane, hi, lo);
      if (p.lengths && w.tv < kC) {
        // padding tokens are contracted over: clear whatever they hold
        if (!warp_wait(full_kq, it & 1, abort_word) || !warp_wait(full_v, it & 1, abort_word) ||
            !warp_wait(full_d, it & 1, abort_word))
          return false;
        for (int e = w.tv * (D / 8) + lane; e < kC * (D / 8); e += 32) {
          const int row = e / (D / 8), ch = e % (D / 8);
          const uint32_t off = (ch >> 3) * kBlk + sw128_offset(row, (ch & 7) * 8);
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4 *>(sm + L::Q + off) = z;
          *reinterpret_cast<uint4 *>(sm + L::K + off) = z;
          *reinterpret_cast<uint4 *>(sm + L::V + off) = z;
          *reinterpret_cast<uint4 *>(sm + L::dO + off) = z;
        }
        fence_async_smem();
      }
      __syncwarp();
      mbar_arrive(gate_full);
      return true;
    };
    auto next = [&](uint32_t x) -> uint32_t {
      while (x < p.items && item(x).tv == 0) x += gridDim.x;
      return x;
    };
    uint32_t x = next(blockIdx.x);
    bool ok = x < p.items;
    if (ok) ok = gates(item(x), fetch(item(x)));
    while (ok && x < p.items) {
      const Item w = item(x);
      const float total = exp2f(hi[kC - 1] + lo[kC - 1]);
      x = next(x + gridDim.x);
      Item w2 = w;
      float4 g2 = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x < p.items) w2 = item(x), g2 = fetch(w2);
      if (!warp_wait(dg_in, it & 1, abort_word) || !warp_wait(dot_full, it & 1, abort_word)) break;
      const float *mail = p.mail + (long)blockIdx.x * 4 * kC + 4 * lane;
      const float4 l4 = __ldcg(reinterpret_cast<const float4 *>(mail + 2 * kC)), r4 = __ldcg(reinterpret_cast<const float4 *>(mail + 3 * kC));
      const float over = total == 0.f ? 0.f : total * ((red[0] + red[1]) + (red[2] + red[3]));
      __syncwarp();
      mbar_arrive(dot_free);
      ++it;
      if (x < p.items) ok = gates(w2, g2);  // the next chunk waits for these, nothing waits for dg
      const int done = it - 1;
      if (!warp_wait(&in_full[done & 1], (done >> 1) & 1, abort_word)) break;
      const float4 s4 = __ldcg(reinterpret_cast<const float4 *>(mail + (done & 1) * kC));
      // suffix sums of what the state gives queries at or behind t, prefix sums of what keys before t give it
      const float e[4] = {l4.x, l4.y, l4.z, l4.w}, r[4] = {r4.x, r4.y, r4.z, r4.w}, in[4] = {s4.x, s4.y, s4.z, s4.w};
      Sum2 es{0.f, 0.f}, rs{0.f, 0.f};
#pragma unroll
      for (int m = 0; m < 4; ++m) es.add(e[m]), rs.add(r[m]);
      Sum2 behind = warp_scan_others<true>(es, lane), before = warp_scan_others<false>(rs, lane);
      float dgv[4];
#pragma unroll
      for (int m = 3; m >= 0; --m) {
        behind.add(e[m]);
        Sum2 v = behind;
        Sum2 b = before;
#pragma unroll
        for (int k = 0; k < m; ++k) b.add(r[k]);
        v.add(b.s, b.e);
        v.add(over);
        v.add(in[m]);
        dgv[m] = v.s + v.e;
      }
      float *dg = p.dg + w.bh * p.N + w.t0;
      const int rows = (int)min((long)kC, p.N - w.t0);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const int t = 4 * lane + m;
        if (t < rows) dg[t] = t < w.tv ? dgv[m] : 0.f;
      }
    }
  } else if (warp < kWarpScore) {
    // ---- <S, R> of the stored pairs ----
    int it = 0;
    for (uint32_t x = blockIdx.x; x < p.items; x += gridDim.x) {
      if (item(x).tv == 0) continue;
      const uint4 *S = reinterpret_cast<const uint4 *>(p.s_tiles + x * (size_t)(2 * kState));
      const uint4 *R = reinterpret_cast<const uint4 *>(p.r_tiles + x * (size_t)(2 * kState));
      constexpr int kQ = kState / 16;
      float s = 0.f;
#pragma unroll 4
      for (int e = threadIdx.x - kWarpDot * 32; e < kQ; e += 128) s = dot_pairs(S[e], S[e + kQ], R[e], R[e + kQ], s);
      s = warp_sum(s);
      if (it > 0 && !warp_wait(dot_free, (it - 1) & 1, abort_word)) break;
      if (lane == 0) {
        red[warp - kWarpDot] = s;
        mbar_arrive(dot_full);
      }
      ++it;
    }
  } else if (warp < kWarpRow) {
    // ---- scores: key T (lane) against 64 queries ----
    const int q = warp & 3, half = (warp - kWarpScore) >> 2, T = q * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
    float *mail = p.mail + (long)blockIdx.x * 4 * kC;
    int it = 0;
    for (uint32_t x = blockIdx.x; x < p.items; x += gridDim.x) {
      if (item(x).tv == 0) continue;
      const uint32_t ph = it & 1;
      bool ok = mbar_wait(gate_full, ph, abort_word, status) && mbar_wait(e_full, ph, abort_word, status);
      ok = ok && (it == 0 || mbar_wait(out_free, ph ^ 1, abort_word, status));  // W D's place is free
      if (bar_or(kBarScore, 256, !ok)) break;  // also: the last chunk's partial sums are read
      tc_fence_after();
      // W P to tensor memory, W D to shared memory, and W P D's share of dg
      const float hi_j = hi[T], lo_j = lo[T];
      float2 col = make_float2(0.f, 0.f);  // this key's sum over the queries of later blocks
      float own = 0.f;                     // pairs of this block on both sides of token T
#pragma unroll 1
      for (int b = 0; b < 4; ++b) {
        const int i0 = 64 * half + 16 * b;  // 16 queries: none of them, all, or those from the key on
        const bool some = i0 + 15 >= 32 * q, cut = i0 < 32 * q + 32;
        uint32_t o[8];
        uint4 wd[2];
        uint32_t *wdw = reinterpret_cast<uint32_t *>(wd);
        if (!some) {
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = wdw[e] = 0u;
        } else {
          uint32_t pr[16], dr[16];
          tmem_ld16x2(tl + kColP + i0, tl + kColD + i0, pr, dr);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 h = *reinterpret_cast<const float4 *>(hi + i0 + 4 * e), l = *reinterpret_cast<const float4 *>(lo + i0 + 4 * e);
            float f[4];
            decay4(h, l, hi_j, lo_j, 1.f, f);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const int c = 4 * e + k;
              const float2 pp = make_float2(__uint_as_float(pr[c]), __uint_as_float(pr[c + 1]));
              float2 pw = __fmul2_rn(pp, make_float2(f[k], f[k + 1]));
              float2 dw = __fmul2_rn(make_float2(__uint_as_float(dr[c]), __uint_as_float(dr[c + 1])), make_float2(f[k], f[k + 1]));
              float2 m = __fmul2_rn(pp, dw);
              if (cut) {  // queries before the key: nothing; its own: no part in dg
                const int i = i0 + c;
                pw = make_float2(i >= T ? pw.x : 0.f, i + 1 >= T ? pw.y : 0.f);
                dw = make_float2(i >= T ? dw.x : 0.f, i + 1 >= T ? dw.y : 0.f);
                m = make_float2(i > T ? m.x : 0.f, i + 1 > T ? m.y : 0.f);
              }
              if (!cut) col = __fadd2_rn(col, m);
              o[c / 2] = pack_bf16(pw.x, pw.y);
              wdw[c / 2] = pack_bf16(dw.x, dw.y);
              pr[c] = __float_as_uint(m.x), pr[c + 1] = __float_as_uint(m.y);
            }
          }
          const int sub = b & 1;  // which half of its block of 32
          if (cut) {              // the keys' own block: for each token t of it, queries from t on of keys before t
#pragma unroll
            for (int c = 14; c >= 0; --c)
              pr[c] = __float_as_uint(__uint_as_float(pr[c]) + __uint_as_float(pr[c + 1]));
            if (sub) {  // and for the tokens of its first half, all of these queries
              float pre = __shfl_up_sync(0xffffffffu, __uint_as_float(pr[0]), 1);
              if (lane == 0) pre = 0.f;
#pragma unroll
              for (int k = 1; k < 16; k <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, pre, k);
                if (lane >= k) pre += y;
              }
              if (lane < 16) own = pre + own;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c)
              if (lane >= 16 * sub + c) pr[c] = 0u;
          }
          const float s = column_sums(pr, lane);
          if (cut)
            own += lane >> 4 == sub ? s : 0.f;
          else if (lane < 16)
            buf[part_at(q, i0 + lane)] = s;
        }
        tmem_st8_nowait(tl + kColP + 64 * half + 8 * b, o);  // over columns this warp alone reads, and has read
        uint8_t *W = sm + L::WD + half * kBlk;
        *reinterpret_cast<uint4 *>(W + sw128_offset(T, 16 * b)) = wd[0];
        *reinterpret_cast<uint4 *>(W + sw128_offset(T, 16 * b + 8)) = wd[1];
      }
      tmem_wait_st();
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(el_done);
      mbar_arrive(dg_in);  // the running sums are read; what follows has time until the next chunk's
      // token T's dg inside the chunk, by the half that has its block
      const bool mine = half == q >> 1;
      if (!mine) buf[part_at(q, T)] = col.x + col.y;
      named_bar(kBarScore, 256);
      if (mine) {
        const float keys = (col.x + col.y) + buf[part_at(q, T)];
        float row = 0.f, across = 0.f;  // of this query from earlier blocks; of later blocks' queries from earlier blocks' keys
        for (int k = 0; k < q; ++k) {
          row += buf[part_at(k, T)];
          for (int i = T + 32; i < kC; i += 32) across += buf[part_at(k, i)];
        }
        // queries from T on, keys before T
        float before = __shfl_up_sync(0xffffffffu, keys, 1);
        if (lane == 0) before = 0.f;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const float r = __shfl_down_sync(0xffffffffu, row, k), u = __shfl_up_sync(0xffffffffu, before, k);
          if (lane + k < 32) row += r;
          if (lane >= k) before += u;
        }
        __stcg(mail + ph * kC + T, (own + warp_sum(across)) + (row + before));
        mbar_arrive(&in_full[ph]);
      }
      ++it;
    }
  } else {
    // ---- rows: scale the first products, their dot products, results ----
    // half 0: dQ (and dV's first half of columns), half 1: dK (and the second)
    const int q = warp & 3, half = (warp - kWarpRow) >> 2, T = q * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16), tX = tl + (half ? kColK : kColQ);
    const uint8_t *X = sm + (half ? L::K : L::Q);
    float *mail = p.mail + (long)blockIdx.x * 4 * kC + (2 + half) * kC;
    __nv_bfloat16 *dx = half ? p.dk : p.dq;
    int it = 0;
    for (uint32_t x = blockIdx.x; x < p.items; x += gridDim.x) {
      const Item w = item(x);
      const int rows = (int)min((long)kC, p.N - w.t0);
      const long at = (w.bh * p.N + w.t0 + T) * D;
      if (w.tv == 0) {  // padding only: zero gradients
        const uint4 z[4] = {};
        if (T < rows) {
          for (int cb = 0; cb < D / 32; ++cb) store_row64(dx + at + cb * 32, z, p.wide);
          for (int cb = 0; cb < D / 64; ++cb) store_row64(p.dv + at + half * (D / 2) + cb * 32, z, p.wide);
          if (half == 0) p.dg[w.bh * p.N + w.t0 + T] = 0.f;
        }
        continue;
      }
      const uint32_t ph = it & 1;
      if (!warp_wait(gate_full, ph, abort_word)) break;
      const float ew = exp2f((hi[kC - 1] - hi[T]) + (lo[kC - 1] - lo[T])), f = half ? ew : exp2f(hi[T] + lo[T]);
      if (!warp_wait(half ? k_in : q_in, ph, abort_word)) break;
      tc_fence_after();
      drop_cut_rows(tX, D, f);
      float dot = 0.f;
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        uint32_t r[32];
        tmem_ld32(tX + cb * 32, r);
        scale32(r, f);
        tmem_st32(tX + cb * 32, r);
        dot += dot_row32(r, X + (cb >> 1) * kBlk, T, (cb & 1) * 32);
      }
      __stcg(mail + T, dot);
      mbar_arrive(dg_in);
      if (!warp_wait(v_in, ph, abort_word)) break;
      tc_fence_after();
      drop_cut_rows(tl + kColD + half * (D / 2), D / 2, ew);
#pragma unroll
      for (int cb = 0; cb < D / 64; ++cb) {
        uint32_t r[32];
        tmem_ld32(tl + kColD + half * (D / 2) + cb * 32, r);
        scale32(r, ew);
        tmem_st32(tl + kColD + half * (D / 2) + cb * 32, r);
      }
      tc_fence_before();
      mbar_arrive(x_ready);
      // Results leave through W D's place, which its products have left: 32 rows of 64 columns a copy
      // and warp (half 0: dV's first block and dQ; half 1: its second and dK).  Rows past N are clipped,
      // padding rows (T >= tv) are zero whatever the states hold.
      uint8_t *stage = sm + L::WD + (half * 4 + q) * 4096;
      auto put = [&](uint32_t col, const CUtensorMap *map, int c0) {
        if (lane == 0) bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint32_t r[32];
          uint4 v[4];
          tmem_ld32(col + 32 * b, r);
          to_bf16x32(r, v);
          if (T >= w.tv) v[0] = v[1] = v[2] = v[3] = make_uint4(0u, 0u, 0u, 0u);
          stage_row32(stage, lane, b, v);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && q * 32 < rows) {
          tma_store_3d(map, stage, c0, (int)w.t0 + q * 32, (int)w.bh);
          bulk_commit();
        }
      };
      // (the place is W D's until every product that reads it is done)
      if (!warp_wait(out_full, ph, abort_word)) break;
      tc_fence_after();
      // dV's block first: its columns are the next chunk's D
#pragma unroll 1
      for (int cb = -1; cb < D / 64; ++cb) {
        if (D == 128 || half == 0 || cb >= 0)
          put(cb < 0 ? tl + kColD + half * 64 : tX + cb * 64, cb < 0 ? &p.ov : half ? &p.ok : &p.oq,
              64 * (cb < 0 ? half : cb));
        if (cb < 0) {
          tc_fence_before();
          mbar_arrive(d_free);
        }
      }
      if (lane == 0) bulk_wait_read();
      __syncwarp();
      tc_fence_before();
      mbar_arrive(out_free);
      ++it;
    }
    if (lane == 0) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Segments of the state pass: one CTA an SM, one per head and direction; few heads are cut further (the
// sums of the segments first, then the states), down to four chunks a segment.
struct Plan {
  long n, segs, seg_chunks;
};
Plan make_plan(long BH, long N) {
  const long slots = std::max(1, device_info(-1).sm_count), ctas = BH * 2;
  Plan t;
  t.n = (N + kC - 1) / kC;
  t.segs = std::max(1L, std::min(slots / std::max(1L, ctas), t.n / 4));
  t.seg_chunks = (t.n + t.segs - 1) / t.segs;
  t.segs = (t.n + t.seg_chunks - 1) / t.seg_chunks;
  return t;
}

template <int D>
cudaError_t launch_chunks(const Params &cp, cudaStream_t stream) {
  cudaError_t e = ensure_smem_optin((const void *)gated_grad_tc_kernel<D>, (int)Lay<D>::Bytes);
  if (e != cudaSuccess) return e;
  const long sms = std::max(1, device_info(-1).sm_count);
  return launch_gated_kernel(gated_grad_tc_kernel<D>, cp, dim3((unsigned)std::min(sms, (long)cp.items)), kThreads, Lay<D>::Bytes, true,
                             kKGatedBackward, stream);
}

}  // namespace

cudaError_t read_and_clear_gated_grad_status(unsigned int *value) {
  return read_and_clear_status_word((const void *)&g_gated_status, value);
}

size_t gated_tc_grad_workspace(long BH, long N, int D) {
  const Plan t = make_plan(BH, N);
  const size_t tiles = 2 * (size_t)BH * t.n * gated_tile_bytes(D);
  const size_t mail = sizeof(float) * 4 * kC * std::max(1, device_info(-1).sm_count);
  return tiles + mail + (t.segs > 1 ? sizeof(float) * (size_t)BH * t.segs * (2 * (size_t)D * D + 1) : 0);
}

cudaError_t launch_gated_grad_tc(const GatedGradProblem &b) {
  const GatedProblem &p = b.p;
  const int D = p.dk;
  const long BH = p.BH();
  const Plan t = make_plan(BH, p.N);
  const size_t mail = sizeof(float) * 4 * kC * std::max(1, device_info(-1).sm_count);
  uint8_t *ws = (uint8_t *)p.ws + mail;
  const size_t tiles = (size_t)BH * t.n * gated_tile_bytes(D);
  GatedStateParams sp;
  memset(&sp, 0, sizeof sp);
  if (!gated_map(&sp.ta[0], p.k, BH, p.N, D, kC) || !gated_map(&sp.tb[0], p.v, BH, p.N, D, kC) ||
      !gated_map(&sp.ta[1], p.q, BH, p.N, D, kC) || !gated_map(&sp.tb[1], b.dout, BH, p.N, D, kC))
    return cudaErrorInvalidValue;
  sp.g = p.g, sp.lengths = p.lengths, sp.N = p.N, sp.n = t.n, sp.H = p.H;
  sp.segs = sp.run_segs = (int)t.segs, sp.seg_chunks = (int)t.seg_chunks;
  cudaError_t e;
  if (t.segs > 1) {
    float *sums = (float *)(ws + 2 * tiles), *rsums = sums + (size_t)BH * t.segs * D * D,
          *tot = rsums + (size_t)BH * t.segs * D * D;
    sp.fin[0] = sums, sp.fin[1] = rsums, sp.seg_tot = tot;
    e = launch_gated_states(sp, D, BH, 2, false, p.stream);
    if (e != cudaSuccess) return e;
    GatedSegScan sc = {};
    sc.sums[0] = sums, sc.sums[1] = rsums, sc.tot = tot, sc.first[0] = p.S0, sc.first[1] = b.dS;
    sc.last[1] = b.dS0, sc.segs = (int)t.segs, sc.dd = D * D;
    e = launch_gated_seg_scan(sc, BH, 2, p.stream);
    if (e != cudaSuccess) return e;
    sp.init[0] = sums, sp.init[1] = rsums, sp.fin[0] = sp.fin[1] = nullptr, sp.seg_tot = nullptr;
  } else {
    sp.init[0] = p.S0, sp.init[1] = b.dS, sp.fin[1] = b.dS0;
  }
  sp.tiles[0] = ws, sp.tiles[1] = ws + tiles;
  if (!gated_tile_map(&sp.to[0], sp.tiles[0], BH * t.n, D, 32, 1) || !gated_tile_map(&sp.to[1], sp.tiles[1], BH * t.n, D, 32, 1))
    return cudaErrorInvalidValue;
  e = launch_gated_states(sp, D, BH, 2, t.segs > 1, p.stream);
  if (e != cudaSuccess) return e;
  Params cp;
  memset(&cp, 0, sizeof cp);
  cp.tk = sp.ta[0], cp.tv = sp.tb[0], cp.tq = sp.ta[1], cp.td = sp.tb[1];
  if (!gated_tile_map(&cp.ts, ws, BH * t.n, D, D, D / 64) || !gated_tile_map(&cp.tr, ws + tiles, BH * t.n, D, D, D / 64) ||
      !gated_map(&cp.oq, b.dq, BH, p.N, D, 32) || !gated_map(&cp.ok, b.dk, BH, p.N, D, 32) ||
      !gated_map(&cp.ov, b.dv, BH, p.N, D, 32))
    return cudaErrorInvalidValue;
  cp.g = p.g, cp.lengths = p.lengths, cp.s_tiles = sp.tiles[0], cp.r_tiles = sp.tiles[1];
  cp.dq = (__nv_bfloat16 *)b.dq, cp.dk = (__nv_bfloat16 *)b.dk, cp.dv = (__nv_bfloat16 *)b.dv, cp.dg = b.dg;
  cp.mail = (float *)p.ws;
  cp.wide = (((uintptr_t)b.dq | (uintptr_t)b.dk | (uintptr_t)b.dv) & 31) == 0;
  cp.N = p.N, cp.n = (uint32_t)t.n, cp.items = (uint32_t)(BH * t.n), cp.H = p.H;
  return D == 64 ? launch_chunks<64>(cp, p.stream) : launch_chunks<128>(cp, p.stream);
}

}  // namespace la
