// Device helpers of the tensor-core kernels of gated linear attention (bf16, d_k = d_v = D).
#pragma once

#include "gated.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace la {

// Bounded-wait timeouts (see tc_ptx.cuh), one word per translation unit.
static __device__ unsigned int g_gated_status;
inline cudaError_t read_and_clear_status_word(const void *symbol, unsigned int *value) {
  unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(value, symbol, sizeof zero);
  if (e == cudaSuccess && *value) e = cudaMemcpyToSymbol(symbol, &zero, sizeof zero);
  return e;
}

namespace gtc {
using namespace tc;

constexpr int kC = 128;                    // tokens per chunk
constexpr uint32_t kBlk = 16384;           // [128 rows x 128 bytes], 128-byte swizzled
constexpr uint32_t kAbortMisaligned = 2u;  // status bit: shared memory base not 1024-aligned

// Operand descriptors.  K-major: rows are M or N, the K index runs along 64-element blocks `blk`
// bytes apart.  MN-major: rows are the K index, 64-wide M or N blocks `blk` bytes apart.
__device__ __forceinline__ uint64_t kdesc(uint32_t tile, int ks, uint32_t blk = kBlk) {
  return sw128_desc(tile + (ks >> 2) * blk + (ks & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t mndesc(uint32_t tile, int ks, uint32_t blk = kBlk) {
  return sw128_desc(tile + ks * 2048, blk, 1024);
}

// All lanes wait; false for the whole warp if any lane's wait gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_word) {
  const bool ok = mbar_wait(bar, parity, abort_word, &g_gated_status);
  return __all_sync(0xffffffffu, ok);
}

// Running sums of a chunk's log2 decays (one warp, four tokens a lane; tokens from tv on decay by 1).
__device__ __forceinline__ void scan_gates(const float *g, int tv, int lane, float *hi, float *lo) {
  double x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = 4 * lane + e < tv ? log2_decay(g[4 * lane + e]) : 0.0;
#pragma unroll
  for (int e = 1; e < 4; ++e) x[e] += x[e - 1];
  const double before = warp_scan(x[3], lane) - x[3];
  Cum c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] = split_cum(before + x[e]);
  *reinterpret_cast<float4 *>(hi + 4 * lane) = make_float4(c[0].hi, c[1].hi, c[2].hi, c[3].hi);
  *reinterpret_cast<float4 *>(lo + 4 * lane) = make_float4(c[0].lo, c[1].lo, c[2].lo, c[3].lo);
}

// 32 fp32 values (raw bits) as bf16, four 16-byte chunks.
__device__ __forceinline__ void to_bf16x32(const uint32_t (&r)[32], uint4 (&o)[4]) {
  const float *v = reinterpret_cast<const float *>(r);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = make_uint4(pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                      pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
}
// The same as a pair: hi = bf16(x), lo = bf16(x - hi).
__device__ __forceinline__ void split_bf16x32(const uint32_t (&r)[32], uint4 (&hi)[4], uint4 (&lo)[4]) {
  const float *v = reinterpret_cast<const float *>(r);
  uint32_t *h = reinterpret_cast<uint32_t *>(hi), *l = reinterpret_cast<uint32_t *>(lo);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    h[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    l[e] = pack_bf16(v[2 * e] - __uint_as_float(h[e] << 16), v[2 * e + 1] - __uint_as_float(h[e] & 0xffff0000u));
  }
}

__device__ __forceinline__ void scale32(uint32_t (&r)[32], float f) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 y = __fmul2_rn(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), make_float2(f, f));
    r[2 * e] = __float_as_uint(y.x);
    r[2 * e + 1] = __float_as_uint(y.y);
  }
}

// Contiguous copy of `bytes` (a multiple of 16) into shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

}  // namespace gtc

// [BH][N][D] bf16 as a 3-D tensor with boxes of 64 features x `rows` tokens, 128-byte swizzle.
bool gated_map(CUtensorMap *m, const void *base, long BH, long N, int D, uint32_t rows);

// The state pass (gated_state_tc.cu).  For each of `dirs` directions (0: forward, K and V, from the
// first chunk; 1: backward, Q and dout, from the last) and each segment of seg_chunks chunks of
// each head, starting from init: X = 2^{c_T} X + sum_t w_t a_t b_t^T per chunk, w_t = 2^{c_T - c_t}
// (forward) or 2^{c_t} (backward).  tiles: X before each chunk as a bf16 pair in the shared-memory
// image of the MMAs that read it (gated_tile_bytes a chunk, hi then lo); fin: X behind the segment.
struct GatedStateParams {
  CUtensorMap ta[2], tb[2];  // boxes of 64 x 64
  const float *g;
  const int *lengths;
  long N, n;  // tokens and chunks per head
  int H, segs, seg_chunks, run_segs;  // segments [0, run_segs) of segs are run
  const float *init[2];               // [BH][segs][D][D], null: zero
  float *fin[2];                      // [BH][segs][D][D], nullable
  float *seg_tot;                     // [BH][segs] log2 decay of each segment (written with fin), nullable
  uint8_t *tiles[2];                  // [BH][n] tiles, nullable
};
constexpr size_t gated_tile_bytes(int D) { return (size_t)D * D * 4; }
// pdl: may start while the previous kernel of the stream, one of this file's family, still runs.
cudaError_t launch_gated_states(const GatedStateParams &sp, int D, long BH, int dirs, bool pdl, cudaStream_t stream);
// Segment sums -> state before each segment, in place; the running state behind the last one to last.
struct GatedSegScan {
  float *sums[2];      // [BH][segs][D][D]
  const float *tot;    // [BH][segs]
  const float *first[2];
  float *last[2];      // nullable
  int segs, dd;
  bool skip_last;      // the last segment (forward) has no sum: its start is written, nothing behind it
};
cudaError_t launch_gated_seg_scan(const GatedSegScan &a, long BH, int dirs, cudaStream_t stream);

}  // namespace la
