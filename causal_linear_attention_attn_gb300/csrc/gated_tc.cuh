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

// Matrix products.  One thread issues a kernel's MMAs, beside five or six busy warps on its scheduler:
// the instructions between two MMAs set the tensor core's pace.  So the whole warp walks through the
// loop (its values stay in uniform registers, where the MMA takes them), one elected lane issues, and
// a product's descriptors are a base and constant steps.  Measured: 104 MMAs of the gradient in 9700
// cycles instead of 15000 with lane 0 in a loop of its own and descriptors built per MMA.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// Operands.  K-major: rows are M or N, the K index runs along 64-element blocks `blk` bytes apart.
// MN-major: rows are the K index, 64-wide M or N blocks `blk` bytes apart.
__device__ __forceinline__ uint64_t kbase(uint32_t tile) { return sw128_desc(tile, 16, 1024); }
__device__ __forceinline__ uint64_t mnbase(uint32_t tile, uint32_t blk = kBlk) { return sw128_desc(tile, blk, 1024); }
enum Major { kK, kMN };
template <Major kMajor, uint32_t kBlock>
__device__ __forceinline__ constexpr uint64_t op_step(int ks) {  // 16 K elements on
  return kMajor == kK ? ((ks >> 2) * kBlock + (ks & 3) * 32) >> 4 : (ks * 2048) >> 4;
}
// D (+)= A B over kSteps steps of 16; A in shared memory.
template <int kSteps, Major kA, Major kB, uint32_t kBlkA = kBlk, uint32_t kBlkB = kBlk>
__device__ __forceinline__ void product(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
#pragma unroll
  for (int ks = 0; ks < kSteps; ++ks)
    mma_bf16(d, a + op_step<kA, kBlkA>(ks), b + op_step<kB, kBlkB>(ks), idesc, (ks > 0 || add) ? 1u : 0u);
}
// A in tensor memory, 64 K elements from each of two column groups 64 apart (see the scores' warps).
template <Major kB>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    mma_bf16_ts(d, a + (ks < 4 ? 8 * ks : 32 + 8 * ks), b + op_step<kB, kBlk>(ks), idesc, (ks > 0 || add) ? 1u : 0u);
}

// A tile into L2 ahead of its load: shared memory has no room for a second stage of everything, and a
// load that starts when its place frees up then waits for L2 and not for DRAM.
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}

// Registers of a warpgroup (four warps, aligned).
template <int kN>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kN));
}
template <int kN>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kN));
}

// All lanes wait; false for the whole warp if any lane's wait gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_word) {
  const bool ok = mbar_wait(bar, parity, abort_word, &g_gated_status);
  return __all_sync(0xffffffffu, ok);
}

// A chunk's log decays, four consecutive tokens a lane (tokens from tv on decay by 1).
__device__ __forceinline__ float4 load_gates(const float *g, int tv, int lane) {
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = 4 * lane + e < tv ? g[4 * lane + e] : 0.f;
  return make_float4(x[0], x[1], x[2], x[3]);
}
// Their inclusive running sums in base 2 (one warp).
struct GateSums {
  long long c[4];  // fixed point
  bool nan[4];
  bool cut;  // any of this lane's four
  __device__ __forceinline__ GateSums(float4 g, int lane) {
    const float v[4] = {g.x, g.y, g.z, g.w};
    cut = is_cut(fminf(fminf(g.x, g.y), fminf(g.z, g.w)));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = fixed_log2_decay(v[e]) + (e ? c[e - 1] : 0);
      nan[e] = isnan(v[e]) || (e && nan[e - 1]);
    }
    const long long before = warp_scan(c[3], lane) - c[3];
    const bool nan_before = __ballot_sync(0xffffffffu, nan[3]) & ((1u << lane) - 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] += before, nan[e] = nan[e] || nan_before;
  }
};
__device__ __forceinline__ void store_cums(const long long (&c)[4], const bool (&nan)[4], int lane, float *hi, float *lo) {
  Cum u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) u[e] = split_cum(c[e], nan[e]);
  *reinterpret_cast<float4 *>(hi + 4 * lane) = make_float4(u[0].hi, u[1].hi, u[2].hi, u[3].hi);
  *reinterpret_cast<float4 *>(lo + 4 * lane) = make_float4(u[0].lo, u[1].lo, u[2].lo, u[3].lo);
}
__device__ __forceinline__ void scan_gates(float4 g, int lane, float *hi, float *lo) {
  const GateSums s(g, lane);
  store_cums(s.c, s.nan, lane, hi, lo);
}

// Two loads of 16 columns with a single wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t a, uint32_t b, uint32_t (&r)[16], uint32_t (&s)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(s[0]),
        "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7]), "=r"(s[8]), "=r"(s[9]),
        "=r"(s[10]), "=r"(s[11]), "=r"(s[12]), "=r"(s[13]), "=r"(s[14]), "=r"(s[15])
      : "r"(a), "r"(b)
      : "memory");
}

// Store 16 consecutive columns of this warp's 32 lanes; a tmem_wait_st() must follow.
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// A state's columns times f, the whole warp's factor, without the wait.  Zero is a cut: not even a NaN stays.
template <int kBlocks>
__device__ __forceinline__ void tmem_st_scaled(uint32_t taddr, const uint32_t (&r)[kBlocks][32], float f) {
  if (f != 0.f) {
#pragma unroll
    for (int h = 0; h < 2 * kBlocks; ++h) {
      uint32_t y[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(r[h >> 1][16 * (h & 1) + e]) * f);
      tmem_st16_nowait(taddr + 16 * h, y);
    }
  } else {
    const uint32_t y[16] = {};
#pragma unroll
    for (int h = 0; h < 2 * kBlocks; ++h) tmem_st16_nowait(taddr + 16 * h, y);
  }
}

__device__ __forceinline__ void tmem_st8_nowait(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// f = 2^{sign (c_t - c)} for the running sums c_t = h + l of four tokens and c = hi + lo.
__device__ __forceinline__ void decay4(float4 h, float4 l, float hi, float lo, float sign, float (&f)[4]) {
  const float2 s = make_float2(sign, sign), a = make_float2(-sign * hi, -sign * hi), b = make_float2(-sign * lo, -sign * lo);
  const float2 x = __fadd2_rn(__ffma2_rn(make_float2(h.x, h.y), s, a), __ffma2_rn(make_float2(l.x, l.y), s, b));
  const float2 y = __fadd2_rn(__ffma2_rn(make_float2(h.z, h.w), s, a), __ffma2_rn(make_float2(l.z, l.w), s, b));
  f[0] = ex2_approx(x.x), f[1] = ex2_approx(x.y), f[2] = ex2_approx(y.x), f[3] = ex2_approx(y.y);
}

// Eight packed bf16 values times f as a bf16 pair (split8 of tc_ptx.cuh in packed arithmetic).
__device__ __forceinline__ void split8p(uint4 x, float f, uint4 &hi, uint4 &lo) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = __fmul2_rn(make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)), make_float2(f, f));
    h[e] = pack_bf16(v.x, v.y);
    const float2 d = __ffma2_rn(make_float2(__uint_as_float(h[e] << 16), __uint_as_float(h[e] & 0xffff0000u)),
                                make_float2(-1.f, -1.f), v);
    l[e] = pack_bf16(d.x, d.y);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// y + f x, and y where f is zero, whatever x holds.  Measured in the prefill's outputs (148 us): a
// predicate costs 1 us, clearing x first 3 to 4.
__device__ __forceinline__ float2 add_scaled(float2 y, float2 x, float f) {
  asm("{\n.reg .pred p;\n.reg .b64 a, b, c;\nsetp.neu.f32 p, %4, 0f00000000;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %4};\n"
      "mov.b64 c, {%0, %1};\n@p fma.rn.f32x2 c, a, b, c;\nmov.b64 {%0, %1}, c;\n}"
      : "+f"(y.x), "+f"(y.y)
      : "f"(x.x), "f"(x.y), "f"(f));
  return y;
}

// 32 fp32 values (raw bits) as bf16, four 16-byte chunks.
__device__ __forceinline__ void to_bf16x32(const uint32_t (&r)[32], uint4 (&o)[4]) {
  const float *v = reinterpret_cast<const float *>(r);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = make_uint4(pack_bf16(v[8 * q], v[8 * q + 1]), pack_bf16(v[8 * q + 2], v[8 * q + 3]),
                      pack_bf16(v[8 * q + 4], v[8 * q + 5]), pack_bf16(v[8 * q + 6], v[8 * q + 7]));
}
// What bf16 leaves of them, as bf16: bf16(x - bf16(x)).
__device__ __forceinline__ void rest_bf16x32(const uint32_t (&r)[32], uint4 (&o)[4]) {
  const float *v = reinterpret_cast<const float *>(r);
  uint32_t *l = reinterpret_cast<uint32_t *>(o);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint32_t h = pack_bf16(v[2 * e], v[2 * e + 1]);
    const float2 d = __ffma2_rn(make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)),
                                make_float2(-1.f, -1.f), make_float2(v[2 * e], v[2 * e + 1]));
    l[e] = pack_bf16(d.x, d.y);
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

// Rows whose factor is zero, which is a cut, cleared: times zero an inf or a NaN would stay.  (A test in
// scale32 cost the gradient's chunks 10 us of 254 where no row is cut, one for all of a row's columns 2.)
__device__ __forceinline__ void drop_cut_rows(uint32_t taddr, int columns, float f) {
  if (!__any_sync(0xffffffffu, f == 0.f)) return;
#pragma unroll 1
  for (int c = 0; c < columns; c += 32) {
    uint32_t r[32];
    tmem_ld32(taddr + c, r);
#pragma unroll
    for (int e = 0; e < 32; ++e) r[e] = f == 0.f ? 0u : r[e];
    tmem_st32(taddr + c, r);
  }
}

// A lane's row of 32 bf16 into a [rows x 128 bytes] block of shared memory, 128-byte swizzled.
__device__ __forceinline__ void stage_row32(uint8_t *blk, int row, int half, const uint4 (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) *reinterpret_cast<uint4 *>(blk + sw128_offset(row, half * 32 + 8 * e)) = v[e];
}

// 64 bytes of a lane's own row, for what is not worth a copy through shared memory: every lane is in
// another row, an instruction touches 32 lines (20 bytes a cycle and SM; a bulk copy moves 27, beside
// the warp's other work).
__device__ __forceinline__ void store_row64(void *p, const uint4 (&v)[4], bool wide) {
  if (wide) {
#pragma unroll
    for (int e = 0; e < 4; e += 2)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint4 *>(p) + e),
                   "r"(v[e].x), "r"(v[e].y), "r"(v[e].z), "r"(v[e].w), "r"(v[e + 1].x), "r"(v[e + 1].y), "r"(v[e + 1].z),
                   "r"(v[e + 1].w)
                   : "memory");
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) reinterpret_cast<uint4 *>(p)[e] = v[e];
  }
}

}  // namespace gtc

// One launch; pdl: it may start while the previous kernel of the stream, one of this family, still
// runs (that kernel lets it in after its tensor-memory allocation, and it waits for that kernel's
// results before it reads any).
template <typename P>
cudaError_t launch_gated_kernel(void (*fn)(P), const P &p, dim3 grid, int threads, uint32_t smem, bool pdl, int kernel_id,
                                cudaStream_t stream) {
  LaunchTimer timer(kernel_id, stream);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  timer.done(e);
  if (e == cudaSuccess) count_launch();
  return e;
}

// [BH][N][D] bf16 as a 3-D tensor with boxes of 64 features x `rows` tokens, 128-byte swizzle.
bool gated_map(CUtensorMap *m, const void *base, long BH, long N, int D, uint32_t rows);

// The state pass's tiles as [blocks][D][64] bf16 with boxes of `rows` rows of `blocks` blocks.
bool gated_tile_map(CUtensorMap *m, const void *base, long chunks, int D, uint32_t rows, uint32_t blocks);

// The state pass (gated_state_tc.cu).  For each of `dirs` directions (0: forward, K and V, from the
// first chunk; 1: backward, Q and dout, from the last) and each segment of seg_chunks chunks of
// each head, starting from init: X = 2^{c_T} X + sum_t w_t a_t b_t^T per chunk, w_t = 2^{c_T - c_t}
// (forward) or 2^{c_t} (backward).  tiles: X before each chunk as a bf16 pair (gated_tile_bytes a
// chunk: hi then lo, each in blocks of 64 columns, [D][64] row-major); fin: X behind the segment.
// Without tiles only the segments' own sums are wanted (init is not read, fin is given).
struct GatedStateParams {
  CUtensorMap ta[2], tb[2];  // boxes of 64 x 128
  CUtensorMap to[2];         // of tiles, boxes of 32 rows
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
