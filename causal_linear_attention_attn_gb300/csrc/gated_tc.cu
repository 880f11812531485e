// Gated linear attention on the sm_103a tensor cores (bf16, d_k = d_v = D in {64, 128}).
//
// A CTA owns a segment of one head and carries its state S through chunks of 128 tokens.  Per chunk
// (local rows i, j; c the inclusive running sum of log2 decays, kept as hi + lo, see gated.cuh):
//   P   = Q K^T                             fp32 in tensor memory
//   P'  = bf16(2^{c_i - c_j} P), j <= i     one rounding; written back as the A operand
//   O   = 2^{c_i} (Q bf16(S)) + P' V        two accumulators, joined when they are read
//   S  <- 2^{c_T} S + (w k)^T V             w_j = 2^{c_T - c_j}; w k as a bf16 pair, S fp32
// The outputs are bf16, so one rounding of the weights and of the state the queries read keeps their
// error near the outputs' own; S is an fp32 result and takes its keys as a pair (2^-17).  Weighting
// scores by differences of running sums (not queries and keys by their own) costs an exponential per
// score, half of them masked, and holds for every decay: no factor exceeds 1.
//
// Long sequences with few heads are cut into segments; the state before each comes from the state
// pass (gated_state_tc.cu) over the earlier ones and a scan over their sums.
//
// HBM is its floor (8 D bytes per token in and out, 40 flops a byte at D = 128); built, a chunk takes
// about 5500 cycles, of which the one thread that issues its 40 MMAs is busy for most: they take 64
// cycles each alone and about twice that beside 26 busy warps.  Measured at 4 x 16 x 8192, D = 128:
// 102 us for this pass (5.3 TB/s of its bytes), 149 us with the state pass and scan before it.
//
// Warps: 0 TMA, 1 MMA and TMEM owner, 2 running sums, 4-11 weights of the scores, 12-19 weighted keys,
// 20-23 state (bf16 copy, decay), 24-27 outputs.  Every wait is bounded (tc_ptx.cuh).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>

#include "gated_tc.cuh"
#include "register_shares.h"

namespace la {
namespace {
using namespace gtc;

constexpr int kThreads = 896;
constexpr int kWarpGate = 2, kWarpP = 4, kWarpK = 12, kWarpS = 20, kWarpO = 24;
constexpr uint32_t kBarS = 1;
// Registers a thread: the launch gives every warpgroup 72; the state and the outputs, which pass
// through in blocks, take what the others leave.
constexpr int kRegs = 72, kRegs0 = 48, kRegsK = 64, kRegsS = 96, kRegsO = 88;
static_assert(kRegs0 + 2 * kRegs + 2 * kRegsK + kRegsS + kRegsO <= 7 * kRegs, "warpgroups' shares within the launch's");

template <int D>
struct Lay {
  static constexpr uint32_t kTile = D / 64 * kBlk;  // 128 tokens
  static constexpr uint32_t Q = 0;
  static constexpr uint32_t K = Q + kTile;
  static constexpr uint32_t Khi = K + kTile;
  static constexpr uint32_t Klo = Khi + kTile;
  static constexpr uint32_t V = Klo + kTile;  // 2 stages
  static constexpr uint32_t Sb = V + 2 * kTile;
  static constexpr uint32_t Sum = Sb + 128 * D * 2;  // D = 64: low rows of the state [64][65] fp32
  static constexpr uint32_t Gate = Sum + (D == 64 ? 64 * 65 * 4 : 0);
  static constexpr uint32_t Bars = Gate + 2 * 2 * kC * 4;
  static constexpr int kNumBars = 19;
  static constexpr uint32_t Misc = Bars + kNumBars * 8;
  static constexpr uint32_t Bytes = Misc + 16;
};
static_assert(Lay<128>::Bytes <= 232448, "shared memory budget");
constexpr uint32_t kColS = 0, kColP = 128, kColI = 256, kColA = 384;  // state, scores, Q S, P' V

struct Params {
  CUtensorMap tq, tk, tv;  // boxes of 64 x 128
  CUtensorMap to;          // boxes of 64 x 32
  const float *g;
  const int *lengths;
  const float *init;  // state before each segment: [BH][init_segs][D][D], segment s at s * init_step; null: zero
  __nv_bfloat16 *out;
  float *S;
  long N;
  int H, segs, seg_chunks, init_segs, init_step;
  bool wide;  // out is 32-byte aligned
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) gated_tc_kernel(const __grid_constant__ Params p) {
  using L = Lay<D>;
  extern __shared__ __align__(1024) uint8_t sm[];
  if (smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_gated_status, kAbortMisaligned);
    return;
  }
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::Bars);
  uint64_t *full_v = bars, *v_free = bars + 2, *gate_full = bars + 4, *gate_free = bars + 6, *full_q = bars + 8,
           *q_free = bars + 9, *full_k = bars + 10, *k_free = bars + 11, *p_full = bars + 12, *k_ready = bars + 13,
           *pp_ready = bars + 14, *sb_ready = bars + 15, *s_full = bars + 16, *o_full = bars + 17, *o_free = bars + 18;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::Misc);
  volatile uint32_t *abort_word = reinterpret_cast<volatile uint32_t *>(sm + L::Misc + 4);
  uint64_t *drain = reinterpret_cast<uint64_t *>(sm + L::Misc + 8);
  unsigned int *status = &g_gated_status;
  float *gate = reinterpret_cast<float *>(sm + L::Gate);  // [2][hi 128, lo 128]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long bh = blockIdx.x / p.segs;
  const int seg = (int)(blockIdx.x - bh * p.segs);
  const long len = row_length(p.lengths, bh / p.H, p.N);
  const long nb = (len + kC - 1) / kC;
  const long c_lo = min(nb, (long)seg * p.seg_chunks);
  const int nc = (int)(min(nb, c_lo + p.seg_chunks) - c_lo);
  auto valid = [&](int c) -> int { return (int)min((long)kC, len - (c_lo + c) * kC); };

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&full_v[b], 1);
      mbar_init(&v_free[b], 4);  // the outputs' warps, when their rows have left it
      mbar_init(&gate_full[b], 32);
      mbar_init(&gate_free[b], 768);
    }
    mbar_init(full_k, 1);
    mbar_init(k_free, 1 + 256);  // the scores' product and the weighted keys' warps
    mbar_init(full_q, 1);
    mbar_init(q_free, 1);
    mbar_init(p_full, 1);
    mbar_init(k_ready, 256);
    mbar_init(pp_ready, 256);
    mbar_init(sb_ready, 128);
    mbar_init(s_full, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, 128);
    mbar_init(drain, 1);
    *abort_word = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the states before the segments are the previous kernels'

  if (warp < 4) {
    reg_dec<kRegs0>();
    if (warp == 0 && lane == 0) {
      prefetch_tmap(&p.tq);
      prefetch_tmap(&p.tk);
      prefetch_tmap(&p.tv);
      auto load = [&](uint32_t at, const CUtensorMap *map, uint64_t *bar, int tok) {
        mbar_arrive_expect_tx(bar, L::kTile);
        for (int b = 0; b < D / 64; ++b) tma_load_3d(sm + at + b * kBlk, map, bar, 64 * b, tok, (int)bh);
      };
      int k_issued = 0, q_issued = 0, v_issued = 0;
      for (int c = 0; c < nc; ++c) {
        const int s = c & 1, tok = (int)((c_lo + c) * kC);
        if (c >= 1 && !mbar_wait(k_free, (c - 1) & 1, abort_word, status)) break;
        load(L::K, &p.tk, full_k, tok);
        k_issued = c + 1;
        if (c >= 2 && !mbar_wait(&v_free[s], ((c >> 1) - 1) & 1, abort_word, status)) break;
        load(L::V + s * L::kTile, &p.tv, &full_v[s], tok);
        v_issued = c + 1;
        if (c >= 1 && !mbar_wait(q_free, (c - 1) & 1, abort_word, status)) break;
        load(L::Q, &p.tq, full_q, tok);
        q_issued = c + 1;
        if (c + 1 < nc)  // (values have a second stage)
          for (int b = 0; b < D / 64; ++b) {
            tma_prefetch_3d(&p.tk, 64 * b, tok + kC, (int)bh);
            tma_prefetch_3d(&p.tq, 64 * b, tok + kC, (int)bh);
          }
      }
      for (int c = max(0, v_issued - 2); c < v_issued; ++c) wait_drain(&full_v[c & 1], (c >> 1) & 1, status);
      if (k_issued) wait_drain(full_k, (k_issued - 1) & 1, status);
      if (q_issued) wait_drain(full_q, (q_issued - 1) & 1, status);
    } else if (warp == 1) {
      constexpr uint32_t iP = idesc_bf16_f32(128, 128, 0, 0), iO = idesc_bf16_f32(128, D, 0, 1), iS = idesc_bf16_f32(128, D, 1, 1);
      constexpr int kDs = D / 16;
      const bool leader = elect_one();
      const uint32_t tS = tmem + kColS, tP = tmem + kColP, tI = tmem + kColI, tA = tmem + kColA;
      const uint32_t sQ = smem_u32(sm + L::Q), sK = smem_u32(sm + L::K), sSb = smem_u32(sm + L::Sb),
                     sKhi = smem_u32(sm + L::Khi), sKlo = smem_u32(sm + L::Klo);
      for (int c = 0; c < nc; ++c) {
        const int s = c & 1;
        const uint32_t v = smem_u32(sm + L::V) + s * L::kTile;
        if (!warp_wait(full_q, c & 1, abort_word)) break;
        if (!warp_wait(full_k, c & 1, abort_word)) break;
        tc_fence_after();
        // the scores' columns are free: the previous P' V reads them before, in issue order
        if (leader) {
          product<kDs, kK, kK>(tP, kbase(sQ), kbase(sK), iP, false);
          mma_commit(p_full);
          mma_commit(k_free);
        }
        __syncwarp();
        // The update before the read: the read waits for the last outputs to be read out, the update
        // only for the state's warps (the read takes the state from their copy).
        if (!warp_wait(k_ready, c & 1, abort_word)) break;
        if (!warp_wait(sb_ready, c & 1, abort_word)) break;
        if (!warp_wait(&full_v[s], (c >> 1) & 1, abort_word)) break;
        tc_fence_after();
        if (leader) {
          if (D == 128) {
            product<8, kMN, kMN>(tS, mnbase(sKhi), mnbase(v), iS, true);
            product<8, kMN, kMN>(tS, mnbase(sKlo), mnbase(v), iS, true);
          } else {
            product<8, kMN, kMN>(tS, mnbase(sKhi, L::kTile), mnbase(v), iS, true);  // rows: hi, then lo
          }
          mma_commit(s_full);
        }
        __syncwarp();
        if (c > 0 && !warp_wait(o_free, (c - 1) & 1, abort_word)) break;
        tc_fence_after();
        if (leader) {
          product<kDs, kK, kMN>(tI, kbase(sQ), mnbase(sSb), iO, false);
          if (D == 64) product<kDs, kK, kMN>(tI, kbase(sQ), mnbase(sSb + 64 * 128), iO, true);  // the low keys' part
          mma_commit(q_free);
        }
        __syncwarp();
        if (!warp_wait(pp_ready, c & 1, abort_word)) break;
        tc_fence_after();
        if (leader) {
          product_ts<kMN>(tA, tP, mnbase(v), iO, false);
          mma_commit(o_full);
        }
        __syncwarp();
      }
      if (leader) {
        mma_commit(drain);
        wait_drain(drain, 0, status);
      }
    } else if (warp == kWarpGate) {
      const float *g = p.g + bh * p.N + c_lo * kC;
      float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
      if (nc > 0) cur = load_gates(g, valid(0), lane);
      for (int c = 0; c < nc; ++c) {
        float4 nxt = cur;
        if (c + 1 < nc) nxt = load_gates(g + (c + 1) * kC, valid(c + 1), lane);
        if (c >= 2 && !warp_wait(&gate_free[c & 1], ((c >> 1) - 1) & 1, abort_word)) break;
        float *hi = gate + (c & 1) * 2 * kC;
        scan_gates(cur, lane, hi, hi + kC);
        mbar_arrive(&gate_full[c & 1]);
        cur = nxt;
      }
    }
  } else if (warp < kWarpK) {
    // ---- weights of the scores: row i of this thread, keys [64 half, 64 half + 64) ----
    const int q = warp & 3, i = q * 32 + lane, half = (warp - kWarpP) >> 2;
    const uint32_t tP = tmem + ((uint32_t)(q * 32) << 16) + kColP + 64 * half;
    for (int c = 0; c < nc; ++c) {
      if (!warp_wait(&gate_full[c & 1], (c >> 1) & 1, abort_word)) break;
      if (!warp_wait(p_full, c & 1, abort_word)) break;
      tc_fence_after();
      const float *hi = gate + (c & 1) * 2 * kC, *lo = hi + kC;
      const float hi_i = hi[i], lo_i = lo[i];
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const int cb = 2 * half + b;  // 32 keys: none, all, or (cb == q) those up to the query
        uint32_t o[16];
        if (cb > q) {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0u;
        } else {
          uint32_t r[32];
          tmem_ld32(tP + b * 32, r);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 h = *reinterpret_cast<const float4 *>(hi + cb * 32 + 4 * e),
                         l = *reinterpret_cast<const float4 *>(lo + cb * 32 + 4 * e);
            float f[4];
            decay4(h, l, hi_i, lo_i, -1.f, f);
            float2 x = __fmul2_rn(make_float2(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1])), make_float2(f[0], f[1]));
            float2 y = __fmul2_rn(make_float2(__uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3])), make_float2(f[2], f[3]));
            if (cb == q) {
              const int j = 4 * e;
              x = make_float2(j <= lane ? x.x : 0.f, j + 1 <= lane ? x.y : 0.f);
              y = make_float2(j + 2 <= lane ? y.x : 0.f, j + 3 <= lane ? y.y : 0.f);
            }
            o[2 * e] = pack_bf16(x.x, x.y);
            o[2 * e + 1] = pack_bf16(y.x, y.y);
          }
        }
        tmem_st16(tP + b * 16, o);  // over scores that this warp alone reads
      }
      tc_fence_before();
      mbar_arrive(pp_ready);
      mbar_arrive(&gate_free[c & 1]);
    }
  } else if (warp < kWarpS) {
    // ---- weighted keys as a pair, in tiles of their own: the last update has read them ----
    reg_dec<kRegsK>();
    const int r = (threadIdx.x - kWarpK * 32) & 127, half = (threadIdx.x - kWarpK * 32) >> 7;
    for (int c = 0; c < nc; ++c) {
      const int s = c & 1;
      if (!warp_wait(&gate_full[c & 1], (c >> 1) & 1, abort_word)) break;
      const float *hi = gate + (c & 1) * 2 * kC, *lo = hi + kC;
      const float w = exp2f((hi[kC - 1] - hi[r]) + (lo[kC - 1] - lo[r]));
      const int tv = valid(c);
      mbar_arrive(&gate_free[c & 1]);
      if (!warp_wait(full_k, c & 1, abort_word)) break;
      if (c > 0 && !warp_wait(s_full, (c - 1) & 1, abort_word)) break;
      // a thread's half of the row: one 64-feature block (D = 128) or half of the only one
      const uint32_t blk = D == 128 ? half * kBlk : 0;
      const int c0 = D == 128 ? 0 : half * 4;
      const uint8_t *K = sm + L::K + blk;
      uint8_t *Khi = sm + L::Khi + blk, *Klo = sm + L::Klo + blk;
#pragma unroll 4
      for (int e = 0; e < D / 16; ++e) {
        const uint32_t off = sw128_offset(r, (c0 + e) * 8);
        uint4 h = make_uint4(0u, 0u, 0u, 0u), l = h;
        if (r < tv) split8p(*reinterpret_cast<const uint4 *>(K + off), w, h, l);
        *reinterpret_cast<uint4 *>(Khi + off) = h;
        *reinterpret_cast<uint4 *>(Klo + off) = l;
      }
      mbar_arrive(k_free);
      if (tv < kC) {  // padding tokens: a zero weight does not clear a NaN of the values
        if (!warp_wait(&full_v[s], (c >> 1) & 1, abort_word)) break;
        uint8_t *V = sm + L::V + s * L::kTile + blk;
        if (r >= tv)
          for (int e = 0; e < D / 16; ++e)
            *reinterpret_cast<uint4 *>(V + sw128_offset(r, (c0 + e) * 8)) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      mbar_arrive(k_ready);
    }
  } else if (warp < kWarpO) {
    // ---- state: bf16 copy for the queries, then decayed in place for the update ----
    reg_inc<kRegsS>();
    const int q = warp & 3, T = q * 32 + lane;
    const int row = D == 64 ? T & 63 : T;
    const bool main_row = D == 128 || q < 2;  // D = 64: lanes from 64 on hold the low keys' part
    const uint32_t tS = tmem + ((uint32_t)(q * 32) << 16) + kColS;
    float *sum = reinterpret_cast<float *>(sm + L::Sum);
    uint32_t r[2][32];
    const long dd = (long)D * D;
    const float *init = p.init ? p.init + (bh * p.init_segs + (long)seg * p.init_step) * dd + (long)row * D : nullptr;
    auto load_init = [&](int cb) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (init && main_row) x = reinterpret_cast<const float4 *>(init + cb * 64 + b * 32)[e];
          r[b][4 * e] = __float_as_uint(x.x), r[b][4 * e + 1] = __float_as_uint(x.y);
          r[b][4 * e + 2] = __float_as_uint(x.z), r[b][4 * e + 3] = __float_as_uint(x.w);
        }
    };
    auto join = [&]() {  // D = 64: the two parts meet in the rows of the first two warps
      if (D == 128) return;
      if (!main_row)
#pragma unroll
        for (int e = 0; e < 64; ++e) sum[row * 65 + e] = __uint_as_float(r[e >> 5][e & 31]);
      named_bar(kBarS, 128);
      if (main_row)
#pragma unroll
        for (int e = 0; e < 64; ++e)
          r[e >> 5][e & 31] = __float_as_uint(__uint_as_float(r[e >> 5][e & 31]) + sum[row * 65 + e]);
    };
    bool ok = true;
    for (int c = 0; c < nc; ++c) {
      bool w = mbar_wait(&gate_full[c & 1], (c >> 1) & 1, abort_word, status);
      if (w && c > 0) w = mbar_wait(s_full, (c - 1) & 1, abort_word, status);
      if (bar_or(kBarS, 128, !w)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float *hi = gate + (c & 1) * 2 * kC;
      const float f = exp2f(hi[kC - 1] + hi[2 * kC - 1]);
      mbar_arrive(&gate_free[c & 1]);
#pragma unroll 1
      for (int cb = 0; cb < D / 64; ++cb) {
        if (c == 0)
          load_init(cb);
        else
          tmem_ld32x2(tS + cb * 64, tS + cb * 64 + 32, r[0], r[1]);
        tmem_st_scaled(tS + cb * 64, r, f);
        if (cb == 0 && c > 0) {  // the last read of the copy is done
          const bool qw = mbar_wait(q_free, (c - 1) & 1, abort_word, status);
          if (bar_or(kBarS, 128, !qw)) {
            ok = false;
            break;
          }
        }
        // (D = 64: the low keys' part is the copy's rows from 64 on; the queries read both)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          uint4 h[4];
          to_bf16x32(r[b], h);
          stage_row32(sm + L::Sb + cb * kBlk, T, b, h);
        }
      }
      if (!ok) break;
      tmem_wait_st();
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(sb_ready);
    }
    if (seg == p.segs - 1 && ok) {
      const bool w = nc == 0 || mbar_wait(s_full, (nc - 1) & 1, abort_word, status);
      if (!bar_or(kBarS, 128, !w)) {
        tc_fence_after();
        float *dst = p.S + bh * dd + (long)row * D;
#pragma unroll 1
        for (int cb = 0; cb < D / 64; ++cb) {
          if (nc == 0)
            load_init(cb);
          else
            tmem_ld32x2(tS + cb * 64, tS + cb * 64 + 32, r[0], r[1]);
          join();
          if (main_row)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              reinterpret_cast<float4 *>(dst + cb * 64)[e] =
                  make_float4(__uint_as_float(r[e >> 3][4 * (e & 7)]), __uint_as_float(r[e >> 3][4 * (e & 7) + 1]),
                              __uint_as_float(r[e >> 3][4 * (e & 7) + 2]), __uint_as_float(r[e >> 3][4 * (e & 7) + 3]));
        }
      }
    }
  } else {
    // ---- outputs: row i, 2^{c_i} (Q S) + P' V ----
    reg_inc<kRegsO>();
    const int q = warp & 3, i = q * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)(q * 32) << 16);
    for (int c = 0; c < nc; ++c) {
      if (!warp_wait(&gate_full[c & 1], (c >> 1) & 1, abort_word)) break;
      const float *hi = gate + (c & 1) * 2 * kC;
      const float f = exp2f(hi[i] + hi[kC + i]);
      mbar_arrive(&gate_free[c & 1]);
      if (!warp_wait(o_full, c & 1, abort_word)) break;
      tc_fence_after();
      // The rows leave through the chunk's values, which are read by now: 32 rows of 64 columns a copy.
      // (Stored from registers, a row a lane, they took 30 of the pass's 125 us at 4 x 16 x 8192.)  A
      // chunk cut by its row's length, not by N where the copy is clipped, stores its rows itself.
      const int tv = valid(c), s = c & 1;
      const long t0 = (c_lo + c) * kC;
      const bool whole = tv == (int)min((long)kC, p.N - t0);
      uint8_t *stage = sm + L::V + s * L::kTile + q * 4096;
      __nv_bfloat16 *dst = p.out + (bh * p.N + t0 + i) * D;
#pragma unroll 1
      for (int cb = 0; cb < D / 32; ++cb) {
        uint4 o[4];
        uint32_t *ow = reinterpret_cast<uint32_t *>(o);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[16], y[16];
          tmem_ld16x2(tl + kColI + cb * 32 + 16 * h, tl + kColA + cb * 32 + 16 * h, x, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 z = add_scaled(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])),
                                        make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), f);
            ow[8 * h + e] = pack_bf16(z.x, z.y);
          }
        }
        if (cb == D / 32 - 1) {
          tc_fence_before();
          mbar_arrive(o_free);
        }
        if (whole)
          stage_row32(stage + (cb >> 1) * kBlk, lane, cb & 1, o);
        else if (i < tv)
          store_row64(dst + cb * 32, o, p.wide);
        if (whole && (cb & 1)) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0 && q * 32 < tv) {
            tma_store_3d(&p.to, stage + (cb >> 1) * kBlk, (cb >> 1) * 64, (int)(t0 + q * 32), (int)bh);
            bulk_commit();
          }
        }
      }
      if (lane == 0) {
        bulk_wait_read();
        mbar_arrive(&v_free[s]);
      }
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

// How a prefill is cut: G segments of seg_chunks chunks per head in the main pass; the states before
// them come from sub-segments of seg_chunks / step chunks (the state pass's CTAs).
struct Plan {
  long n, G, seg_chunks, step;
  long init_segs() const { return (G - 1) * step + 1; }
  bool split() const { return G > 1; }
};
Plan make_plan(long BH, long N) {
  const long sms = std::max(1, device_info(-1).sm_count);
  Plan t;
  t.n = (N + kC - 1) / kC;
  // enough CTAs to cover the SMs once, at least four chunks each: a segment costs a second reading of
  // its keys and values
  t.G = std::max(1L, std::min(sms / std::max(1L, BH), t.n / 4));
  t.seg_chunks = (t.n + t.G - 1) / t.G;
  // the state pass's CTAs, one an SM: parts a segment for the fewest turns of an SM, a CTA's start and
  // end counted as two chunks
  t.step = 1;
  if (t.G > 1) {
    long best = -1;
    for (long step = 1; step <= 8 && step <= t.seg_chunks; ++step) {
      const long cost = (BH * (t.G - 1) * step + sms - 1) / sms * ((t.seg_chunks + step - 1) / step + 2);
      if (best < 0 || cost < best) best = cost, t.step = step;
    }
    t.seg_chunks = (t.seg_chunks + t.step - 1) / t.step * t.step;
    t.G = (t.n + t.seg_chunks - 1) / t.seg_chunks;
    if (t.G == 1) t.step = 1;
  }
  return t;
}

template <int D>
cudaError_t launch_main(const Params &mp, long BH, cudaStream_t stream) {
  cudaError_t e = ensure_smem_optin((const void *)gated_tc_kernel<D>, (int)Lay<D>::Bytes);
  if (e != cudaSuccess) return e;
  return launch_gated_kernel(gated_tc_kernel<D>, mp, dim3((unsigned)(BH * mp.segs)), kThreads, Lay<D>::Bytes, mp.segs > 1, kKGated,
                             stream);
}

template <int D>
bool shares_fit() {
  static RegisterShares shares;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  return shares.fit(dev, kRegs, [] {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, gated_tc_kernel<D>) == cudaSuccess) return a.numRegs;
    cudaGetLastError();
    return -1;
  });
}

}  // namespace

bool gated_tc_supported(int dk, int dv, la_dtype dt, bool grad) {
  if (dt != LA_BF16 || dk != dv || (dk != 64 && dk != 128)) return false;
  const DeviceInfo di = device_info(-1);
  if (di.cc_major != 10 || di.cc_minor != 3 || tensor_map_encoder() == nullptr) return false;
  return grad || (dk == 64 ? shares_fit<64>() : shares_fit<128>());  // the prefill alone splits its registers
}

cudaError_t read_and_clear_gated_status(unsigned int *value) {
  return read_and_clear_status_word((const void *)&g_gated_status, value);
}

size_t gated_tc_prefill_workspace(long BH, long N, int D) {
  const Plan t = make_plan(BH, N);
  return t.split() ? sizeof(float) * (size_t)BH * t.init_segs() * ((size_t)D * D + 1) : 0;
}

cudaError_t launch_gated_tc(const GatedProblem &p) {
  const int D = p.dk;
  const long BH = p.BH();
  const Plan t = make_plan(BH, p.N);
  Params mp;
  memset(&mp, 0, sizeof mp);
  if (!gated_map(&mp.tq, p.q, BH, p.N, D, kC) || !gated_map(&mp.tk, p.k, BH, p.N, D, kC) ||
      !gated_map(&mp.tv, p.v, BH, p.N, D, kC) || !gated_map(&mp.to, p.out, BH, p.N, D, 32))
    return cudaErrorInvalidValue;
  mp.g = p.g, mp.lengths = p.lengths, mp.out = (__nv_bfloat16 *)p.out, mp.S = p.S, mp.N = p.N, mp.H = p.H;
  mp.segs = (int)t.G, mp.seg_chunks = (int)t.seg_chunks, mp.init_segs = 1, mp.init_step = 0;
  mp.init = p.S0;
  mp.wide = ((uintptr_t)p.out & 31) == 0;
  cudaError_t e = cudaSuccess;
  if (t.split()) {
    float *sums = (float *)p.ws, *tot = sums + (size_t)BH * t.init_segs() * D * D;
    GatedStateParams sp;
    memset(&sp, 0, sizeof sp);
    sp.ta[0] = mp.tk, sp.tb[0] = mp.tv;
    sp.g = p.g, sp.lengths = p.lengths, sp.N = p.N, sp.n = t.n, sp.H = p.H;
    sp.segs = (int)t.init_segs(), sp.run_segs = sp.segs - 1, sp.seg_chunks = (int)(t.seg_chunks / t.step);
    sp.fin[0] = sums, sp.seg_tot = tot;
    e = launch_gated_states(sp, D, BH, 1, false, p.stream);
    if (e != cudaSuccess) return e;
    GatedSegScan sc = {};
    sc.sums[0] = sums, sc.tot = tot, sc.first[0] = p.S0, sc.segs = sp.segs, sc.dd = D * D, sc.skip_last = true;
    e = launch_gated_seg_scan(sc, BH, 1, p.stream);
    if (e != cudaSuccess) return e;
    mp.init = sums, mp.init_segs = sp.segs, mp.init_step = (int)t.step;
  }
  return D == 64 ? launch_main<64>(mp, BH, p.stream) : launch_main<128>(mp, BH, p.stream);
}

}  // namespace la
