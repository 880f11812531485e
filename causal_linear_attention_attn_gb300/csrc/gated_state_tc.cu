// States of gated linear attention at chunk borders, on the sm_103a tensor cores.
//
//   X <- 2^{c_T} X + sum_t w_t a_t b_t^T      over chunks of 128 tokens,
// forward: a = k, b = v, w_t = 2^{c_T - c_t} (the state); backward, from the last chunk: a = q,
// b = dout, w_t = 2^{c_t} (the gradient of the state).  The state stays fp32 in tensor memory.  The
// weighted a_t reach the MMAs as a bf16 pair (hi + lo, 2^-17 relative): the state is an fp32 result
// and feeds the decays' gradient, and one bf16 rounding (2^-9) would show in both.
//
// A CTA owns one segment of one head and direction.  The chunks are a chain, state -> MMA -> state;
// what is not on the chain (loads, weights, the bf16 pairs that are stored) runs beside it: the state
// warps read the state, write it back decayed for the next MMA, and only then split and store it.
// Where only a segment's sum is wanted (kSum: the pass before the prefill's segments), the weights run
// to the segment's end instead of the chunk's, 2^{c_end - c_t}, from the last chunk to the first: then
// nothing is decayed between chunks, there is no chain, and the state warps weigh every other chunk.
// At D = 64 hi and lo make up the 128 rows of one MMA, [hi | lo]^T b, and meet when the state is read.
// HBM bounds it: per token 4 D bytes in and, when tiles are written, 4 D bytes out per direction.
// Measured at 4 x 16 x 8192, D = 128, both directions with tiles: 170 us (6.3 TB/s); with the tiles
// stored from registers, a row a lane, 209 us.
//
// Warps: 0 TMA, 1 MMA and TMEM owner, 2-9 weights (hi in place, lo beside it), 10-17 state, 18
// running sums of the decays.  Every wait is bounded (tc_ptx.cuh).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>

#include "gated_tc.cuh"

namespace la {

namespace {
using namespace gtc;

constexpr int kThreads = 608;
constexpr int kWarpXform = 2, kWarpState = 10, kWarpGate = 18;
constexpr uint32_t kBarState = 1;

template <int D, bool kSum>
struct Lay {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kLo = D == 128 && !kSum ? 1 : 2;  // buffers of low parts
  static constexpr uint32_t kTile = D / 64 * kBlk;       // 128 tokens
  static constexpr uint32_t A = 0;
  static constexpr uint32_t Lo = A + kStages * kTile;
  static constexpr uint32_t B = Lo + kLo * kTile;
  // tiles on their way out: 32 rows of 64 columns, hi and lo, for each state warp (D = 64: each of two)
  static constexpr uint32_t Stage = B + kStages * kTile;
  static constexpr uint32_t Sum = Stage + (kSum ? 0 : (D == 128 ? 8 : 2) * 8192);  // D = 64: low rows of the state [64][65] fp32
  static constexpr uint32_t Gate = Sum + (D == 64 ? 64 * 65 * 4 : 0);              // [2][hi 128, lo 128]
  static constexpr uint32_t Bars = Gate + 2 * 2 * kC * 4;
  static constexpr int kNumBars = 3 * kStages + 2 + 4 + 3;
  static constexpr uint32_t Misc = Bars + kNumBars * 8;
  static constexpr uint32_t Bytes = Misc + 16;
};
static_assert(Lay<128, true>::Bytes <= 232448 && Lay<128, false>::Bytes <= 232448, "shared memory budget");

template <int D, bool kSum>
__global__ void __launch_bounds__(kThreads, 1) gated_state_tc_kernel(const __grid_constant__ GatedStateParams p) {
  using L = Lay<D, kSum>;
  constexpr int kStages = L::kStages, kLo = L::kLo;
  extern __shared__ __align__(1024) uint8_t sm[];
  if (smem_u32(sm) & 1023u) {
    if (threadIdx.x == 0) atomicOr(&g_gated_status, kAbortMisaligned);
    return;
  }
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::Bars);
  uint64_t *full = bars, *done = full + kStages, *empty = done + kStages, *lo_free = empty + kStages,
           *gate_full = lo_free + 2, *gate_free = gate_full + 2, *x_ready = gate_free + 2, *x_full = x_ready + 1,
           *drain = x_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::Misc);
  volatile uint32_t *abort_word = reinterpret_cast<volatile uint32_t *>(sm + L::Misc + 4);
  unsigned int *status = &g_gated_status;
  float *gate = reinterpret_cast<float *>(sm + L::Gate);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int dir = blockIdx.y;
  const long bh = blockIdx.x / p.run_segs;
  const int seg = (int)(blockIdx.x - bh * p.run_segs);
  const long len = row_length(p.lengths, bh / p.H, p.N);
  const long nb = (len + kC - 1) / kC;  // the row's chunks
  const long c_lo = min(nb, (long)seg * p.seg_chunks), c_hi = min(nb, c_lo + p.seg_chunks);
  const int nc = (int)(c_hi - c_lo);
  float *fin = p.fin[dir];
  // the last chunk is folded in only if the state behind it is wanted
  const int run = kSum || fin ? nc : max(0, nc - 1);
  auto chunk = [&](int i) -> long { return (dir != 0) != kSum ? c_hi - 1 - i : c_lo + i; };
  auto valid = [&](int i) -> int { return (int)min((long)kC, len - chunk(i) * kC); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&done[s], 256);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&lo_free[b], 1);
      mbar_init(&gate_full[b], 32);
      mbar_init(&gate_free[b], kSum ? 256 : 512);
    }
    mbar_init(x_ready, 256);
    mbar_init(x_full, 1);
    mbar_init(drain, 1);
    *abort_word = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, D);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // after the tensor-memory allocation: the next kernel's CTAs, which allocate too and wait for this
  // grid, must not take columns that a CTA of this grid still needs
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();  // init may be the previous kernel's

  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int i = 0; i < run; ++i) {
        const int s = i % kStages, tok = (int)(chunk(i) * kC);
        if (i >= kStages && !mbar_wait(&empty[s], (i / kStages - 1) & 1, abort_word, status)) break;
        mbar_arrive_expect_tx(&full[s], 2 * L::kTile);
        for (int b = 0; b < D / 64; ++b) {
          tma_load_3d(sm + L::A + s * L::kTile + b * kBlk, &p.ta[dir], &full[s], 64 * b, tok, (int)bh);
          tma_load_3d(sm + L::B + s * L::kTile + b * kBlk, &p.tb[dir], &full[s], 64 * b, tok, (int)bh);
        }
        issued = i + 1;
      }
      for (int i = max(0, issued - kStages); i < issued; ++i) wait_drain(&full[i % kStages], (i / kStages) & 1, status);
    }
  } else if (warp == 1) {
    constexpr uint32_t iMM = idesc_bf16_f32(128, D, 1, 1);
    const bool leader = elect_one();
    const uint32_t sA = smem_u32(sm + L::A), sLo = smem_u32(sm + L::Lo), sB = smem_u32(sm + L::B);
    for (int i = 0; i < run; ++i) {
      const int s = i % kStages;
      if (!warp_wait(&done[s], (i / kStages) & 1, abort_word)) break;
      if (!kSum && !warp_wait(x_ready, i & 1, abort_word)) break;
      const bool add = !kSum || i > 0;
      tc_fence_after();
      const uint32_t a = sA + s * L::kTile, lo = sLo + i % kLo * L::kTile, b = sB + s * L::kTile;
      if (leader) {
        if (D == 128) {
          product<8, kMN, kMN>(tmem, mnbase(a), mnbase(b), iMM, add);
          product<8, kMN, kMN>(tmem, mnbase(lo), mnbase(b), iMM, true);
        } else {
          product<8, kMN, kMN>(tmem, mnbase(a, lo - a), mnbase(b), iMM, add);  // rows: hi, then lo
        }
        mma_commit(&empty[s]);
        mma_commit(&lo_free[i % kLo]);
        if (!kSum || i + 1 == run) mma_commit(x_full);
      }
      __syncwarp();
    }
    if (leader) {
      mma_commit(drain);
      wait_drain(drain, 0, status);
    }
  } else if (warp < kWarpGate) {
    if (kSum || warp < kWarpState) {
      // weights: token r of the chunk, half of its features
      const int t = threadIdx.x - (warp < kWarpState ? kWarpXform : kWarpState) * 32, r = t & 127, half = t >> 7;
      constexpr int kChunks = D / 16;  // 16-byte chunks per thread
      const int blk = D == 128 ? half * kBlk : 0, c0 = D == 128 ? 0 : half * 4;
      for (int i = kSum && warp >= kWarpState; i < run; i += kSum ? 2 : 1) {
        const int s = i % kStages;
        bool ok = mbar_wait(&gate_full[i & 1], (i >> 1) & 1, abort_word, status);
        ok = ok && mbar_wait(&full[s], (i / kStages) & 1, abort_word, status);
        if (ok && i >= kLo) ok = mbar_wait(&lo_free[i % kLo], (i / kLo - 1) & 1, abort_word, status);
        if (!__all_sync(0xffffffffu, ok)) break;
        const float *hi = gate + (i & 1) * 2 * kC, *lo = hi + kC;
        const bool in = r < valid(i);
        const float w = kSum || dir ? exp2f(hi[r] + lo[r]) : exp2f((hi[kC - 1] - hi[r]) + (lo[kC - 1] - lo[r]));
        mbar_arrive(&gate_free[i & 1]);
        uint8_t *A = sm + L::A + s * L::kTile + blk, *Lo = sm + L::Lo + i % kLo * L::kTile + blk;
#pragma unroll 4
        for (int e = 0; e < kChunks; ++e) {
          const uint32_t off = sw128_offset(r, (c0 + e) * 8);
          uint4 h = make_uint4(0u, 0u, 0u, 0u), l = h;
          if (in) split8p(*reinterpret_cast<const uint4 *>(A + off), w, h, l);
          *reinterpret_cast<uint4 *>(A + off) = h;
          *reinterpret_cast<uint4 *>(Lo + off) = l;
        }
        if (!in) {  // padding tokens: a zero weight does not clear a NaN of the other operand
          uint8_t *B = sm + L::B + s * L::kTile + blk;
          for (int e = 0; e < kChunks; ++e)
            *reinterpret_cast<uint4 *>(B + sw128_offset(r, (c0 + e) * 8)) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_smem();
        mbar_arrive(&done[s]);
      }
    }
    if (warp >= kWarpState) {
      const int q = warp & 3, T = q * 32 + lane;  // tensor-memory lane: a row of the state (D = 64: from 64 on, its low part)
      const int col0 = ((warp - kWarpState) >> 2) * (D / 2);
      constexpr int kB = D / 64;  // blocks of 32 columns
      const uint32_t tx = tmem + ((uint32_t)(q * 32) << 16) + col0;
      const int row = D == 64 ? T & 63 : T;
      const bool main_row = D == 128 || q < 2;
      float *sum = reinterpret_cast<float *>(sm + L::Sum);
      uint32_t r[kB][32];
      const long dd = (long)D * D;
      const float *init = !kSum && p.init[dir] ? p.init[dir] + (bh * p.segs + seg) * dd + (long)row * D + col0 : nullptr;
#pragma unroll
      for (int b = 0; b < kB; ++b) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (init && main_row) x = reinterpret_cast<const float4 *>(init + b * 32)[e];
          r[b][4 * e] = __float_as_uint(x.x), r[b][4 * e + 1] = __float_as_uint(x.y);
          r[b][4 * e + 2] = __float_as_uint(x.z), r[b][4 * e + 3] = __float_as_uint(x.w);
        }
      }
      // D = 64: the two parts meet in the rows of the first two lane quarters
      auto join = [&]() {
        if (D == 128) return;
        if (!main_row)
#pragma unroll
          for (int e = 0; e < 32; ++e) sum[row * 65 + col0 + e] = __uint_as_float(r[0][e]);
        named_bar(kBarState, 256);
        if (main_row)
#pragma unroll
          for (int e = 0; e < 32; ++e) r[0][e] = __float_as_uint(__uint_as_float(r[0][e]) + sum[row * 65 + col0 + e]);
      };
      bool ok = true;
      for (int i = 0; !kSum && i < nc && ok; ++i) {
        if (D == 64 && lane == 0) bulk_wait_read();
        bool w = i == 0 || mbar_wait(x_full, (i - 1) & 1, abort_word, status);
        if (w && i < run) w = mbar_wait(&gate_full[i & 1], (i >> 1) & 1, abort_word, status);
        if (bar_or(kBarState, 256, !w)) {  // D = 64: also, the last joined columns are read
          ok = false;
          break;
        }
        tc_fence_after();
        if (i > 0) {
          if constexpr (kB == 2)
            tmem_ld32x2(tx, tx + 32, r[0], r[kB - 1]);
          else
            tmem_ld32(tx, r[0]);
        }
        if (i < run) {
          const float *hi = gate + (i & 1) * 2 * kC;
          const float f = exp2f(hi[kC - 1] + hi[2 * kC - 1]);
          mbar_arrive(&gate_free[i & 1]);
          tmem_st_scaled(tx, r, f);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(x_ready);
        }
        // the tile: 32 rows of 64 columns a copy, read out of shared memory by the next chunk
        if constexpr (!kSum) {
          const int z = (int)((bh * p.n + chunk(i)) * 2 * (D / 64)) + (col0 >> 6);
          uint8_t *stage = sm + L::Stage + (D == 128 ? warp - kWarpState : q & 1) * 8192;
          if (D == 128) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
          }
          join();
          if (main_row) {
#pragma unroll 1
            for (int part = 0; part < 2; ++part)
#pragma unroll
              for (int b = 0; b < kB; ++b) {
                uint4 v[4];
                if (part)
                  rest_bf16x32(r[b], v);
                else
                  to_bf16x32(r[b], v);
                stage_row32(stage + part * 4096, lane, D == 128 ? b : col0 >> 5, v);
              }
          }
          fence_async_smem();
          if (D == 128)
            __syncwarp();
          else
            named_bar(kBarState, 256);
          if (lane == 0 && main_row && col0 % 64 == 0) {
            tma_store_3d(&p.to[dir], stage, 0, q * 32, z);
            tma_store_3d(&p.to[dir], stage + 4096, 0, q * 32, z + D / 64);
            bulk_commit();
          }
        }
      }
      if (!kSum && lane == 0) bulk_wait_all();
      if (fin && ok) {
        const bool w = run == 0 || mbar_wait(x_full, kSum ? 0 : (run - 1) & 1, abort_word, status);
        if (!bar_or(kBarState, 256, !w)) {
          tc_fence_after();
          if (run > 0) {
            if constexpr (kB == 2)
              tmem_ld32x2(tx, tx + 32, r[0], r[kB - 1]);
            else
              tmem_ld32(tx, r[0]);
          }
          join();
          float *dst = fin + (bh * p.segs + seg) * dd + (long)row * D + col0;
          if (main_row)
#pragma unroll
            for (int b = 0; b < kB; ++b)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                reinterpret_cast<float4 *>(dst + b * 32)[e] =
                    make_float4(__uint_as_float(r[b][4 * e]), __uint_as_float(r[b][4 * e + 1]),
                                __uint_as_float(r[b][4 * e + 2]), __uint_as_float(r[b][4 * e + 3]));
        }
      }
    }
  } else {
    const float *g = p.g + bh * p.N;
    float4 cur = make_float4(0.f, 0.f, 0.f, 0.f);
    // kSum: decay of the chunks taken so far, which is what lies between this chunk and the segment's
    // end.  Behind a cut, or below 2^-32768, nothing comes back: it stays at 2^-65536, whatever the chunks
    // that follow.  Growth is held at 2^8192, inf as well, which a cut of a chunk's own still outweighs.
    long long beyond = 0;
    bool beyond_nan = false, gone = false;
    constexpr long long kLeast = -(1ll << 55), kGone = -(1ll << 56), kMost = 1ll << 53;
    if (run > 0) cur = load_gates(g + chunk(0) * kC, valid(0), lane);
    for (int i = 0; i < run; ++i) {
      float4 nxt = cur;
      if (i + 1 < run) nxt = load_gates(g + chunk(i + 1) * kC, valid(i + 1), lane);
      if (i >= 2 && !warp_wait(&gate_free[i & 1], ((i >> 1) - 1) & 1, abort_word)) break;
      float *hi = gate + (i & 1) * 2 * kC;
      if constexpr (kSum) {
        GateSums u(cur, lane);
        const long long all = __shfl_sync(0xffffffffu, u.c[3], 31);
        const bool all_nan = __shfl_sync(0xffffffffu, (int)u.nan[3], 31);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u.c[e] = beyond + (dir ? u.c[e] : all - u.c[e]);
          u.nan[e] = !gone && (beyond_nan || (dir ? u.nan[e] : all_nan));
        }
        store_cums(u.c, u.nan, lane, hi, hi + kC);
        beyond_nan = !gone && (beyond_nan || all_nan);
        beyond += all;
        gone = gone || __any_sync(0xffffffffu, u.cut) || beyond < kLeast;
        beyond = gone ? kGone : min(beyond, kMost);
      } else {
        scan_gates(cur, lane, hi, hi + kC);
      }
      mbar_arrive(&gate_full[i & 1]);
      cur = nxt;
    }
    if (kSum && dir == 0 && lane == 0) {
      const Cum t = split_cum(beyond, beyond_nan);
      p.seg_tot[bh * p.segs + seg] = t.hi + t.lo;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, D);
  }
}

constexpr int kScanThreads = 256;

__global__ void __launch_bounds__(kScanThreads) gated_seg_scan_kernel(const __grid_constant__ GatedSegScan a) {
  if (threadIdx.x == 0) pdl_trigger();
  pdl_wait();
  const int dir = blockIdx.z, parts = a.dd / (4 * kScanThreads);
  const int bh = blockIdx.x / parts;
  const int e = ((blockIdx.x - bh * parts) * kScanThreads + threadIdx.x) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.first[dir]) s = *reinterpret_cast<const float4 *>(a.first[dir] + (long)bh * a.dd + e);
  float *at = a.sums[dir] + (long)bh * a.segs * a.dd + e;
  const float *tot = a.tot + (long)bh * a.segs;
  constexpr int kAhead = 8;  // sums in flight per thread
  for (int i0 = 0; i0 < a.segs; i0 += kAhead) {
    float4 x[kAhead];
    float w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u, g = dir ? a.segs - 1 - i : i;
      const bool has = i < a.segs && !(a.skip_last && i == a.segs - 1);
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      w[u] = 0.f;
      if (has) {
        x[u] = *reinterpret_cast<const float4 *>(at + (long)g * a.dd);
        w[u] = tot[g];
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u, g = dir ? a.segs - 1 - i : i;
      if (i >= a.segs) break;
      *reinterpret_cast<float4 *>(at + (long)g * a.dd) = s;
      const float f = exp2f(w[u]);
      if (f == 0.f) s = make_float4(0.f, 0.f, 0.f, 0.f);  // a cut: not even a NaN stays
      s = make_float4(fmaf(f, s.x, x[u].x), fmaf(f, s.y, x[u].y), fmaf(f, s.z, x[u].z), fmaf(f, s.w, x[u].w));
    }
  }
  if (a.last[dir]) *reinterpret_cast<float4 *>(a.last[dir] + (long)bh * a.dd + e) = s;
}

template <int D, bool kSum>
cudaError_t launch_t(const GatedStateParams &sp, long BH, int dirs, bool pdl, cudaStream_t stream) {
  cudaError_t e = ensure_smem_optin((const void *)gated_state_tc_kernel<D, kSum>, (int)Lay<D, kSum>::Bytes);
  if (e != cudaSuccess) return e;
  return launch_gated_kernel(gated_state_tc_kernel<D, kSum>, sp, dim3((unsigned)(BH * sp.run_segs), (unsigned)dirs), kThreads,
                             Lay<D, kSum>::Bytes, pdl, kKGatedState, stream);
}

}  // namespace

bool gated_map(CUtensorMap *m, const void *base, long BH, long N, int D, uint32_t rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)N, (cuuint64_t)BH};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)N * D * 2};
  cuuint32_t box[3] = {64, rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool gated_tile_map(CUtensorMap *m, const void *base, long chunks, int D, uint32_t rows, uint32_t blocks) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {64, (cuuint64_t)D, (cuuint64_t)(2 * chunks * (D / 64))};
  cuuint64_t strides[2] = {128, (cuuint64_t)D * 128};
  cuuint32_t box[3] = {64, rows, blocks};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_gated_states(const GatedStateParams &sp, int D, long BH, int dirs, bool pdl, cudaStream_t stream) {
  if (!sp.tiles[0]) {
    if (!sp.fin[0] || (dirs == 2 && !sp.fin[1]) || !sp.seg_tot) return cudaErrorInvalidValue;
    return D == 64 ? launch_t<64, true>(sp, BH, dirs, pdl, stream) : launch_t<128, true>(sp, BH, dirs, pdl, stream);
  }
  return D == 64 ? launch_t<64, false>(sp, BH, dirs, pdl, stream) : launch_t<128, false>(sp, BH, dirs, pdl, stream);
}

cudaError_t read_and_clear_gated_state_status(unsigned int *value) {
  return read_and_clear_status_word((const void *)&g_gated_status, value);
}

cudaError_t launch_gated_seg_scan(const GatedSegScan &a, long BH, int dirs, cudaStream_t stream) {
  return launch_gated_kernel(gated_seg_scan_kernel, a, dim3((unsigned)(BH * (a.dd / (4 * kScanThreads))), 1, (unsigned)dirs), kScanThreads, 0,
                             true, kKGatedState, stream);
}

}  // namespace la
