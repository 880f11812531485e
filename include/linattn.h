/*
 * linattn.h — C ABI of the GB300 (sm_103a) normalized linear attention
 * library (liblinattn.so).
 *
 * The method: similarity sim(q, k) = phi(q)^T phi(k) with the feature map
 * phi(x) = ELU(x) + 1 (alpha = 1: x + 1 for x > 0, exp(x) otherwise),
 * applied separately to every query and key vector.  Keys and values are
 * summarized in a state S = sum_j phi(k_j) v_j^T ([m, d_v], m = d_k) and a
 * normalizer z = sum_j phi(k_j) ([m]); a query reads
 *     o = phi(q)^T S / (phi(q)^T z + eps).
 * Sources: "线性注意力从头到尾讲清楚" (lilfry09.github.io) §4 (eps-normalized
 * read), §5 (matrix form), §7 (causal recurrence), §8 (phi = elu + 1,
 * [B,H,N,.] layout); "Linear Attention Math" (aicassindra.com), "The
 * associativity trick, written out", "The recurrent form", "Feature maps:
 * elu+1"; "Linear Attention: Accumulating KV in a Fixed-Size State"
 * (ai-systems-engineering.com), "Summarize state updates and reads with
 * equations".
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Pointers are DEVICE pointers on the current CUDA device, except where a
 * comment says otherwise.  Tensors are contiguous row-major, last index
 * fastest:
 *     q, k : [B, H, N, d_k]        v, out : [B, H, N, d_v]
 *     S    : [B, H, d_k, d_v]      z      : [B, H, d_k]
 * (the decode step drops the N axis).  Rows of S are key-feature
 * components, columns value components.  q, k, v have the dtype given by
 * `dt`; out, S and z are always float32.
 *
 * Ownership: the caller owns every buffer.  The library keeps no pointer
 * after a call returns and never frees caller memory.  `out` must not
 * overlap q, k, v, S or z.  Calls only enqueue work on `stream` (a
 * cudaStream_t; NULL = the legacy default stream) and never synchronize
 * the host; errors raised by kernels that were enqueued successfully
 * surface at the caller's next synchronization.
 *
 * Errors: every entry point validates its arguments before touching the
 * GPU and returns a la_status; nothing is launched on error and no output
 * is modified.  LA_ERR_INVALID_VALUE: a NULL pointer where data is
 * needed, B, H, N < 0, d_k or d_v <= 0, or eps negative / not finite.
 * LA_ERR_UNSUPPORTED: d_k or d_v not in {32, 64, 128}, or an unknown
 * dtype.  LA_ERR_MISALIGNED: a pointer not 16-byte aligned.
 * LA_ERR_NO_DEVICE: no usable CUDA device.  LA_ERR_OUT_OF_MEMORY:
 * stream-ordered scratch could not be allocated.  LA_ERR_LAUNCH: a kernel
 * launch failed (cudaGetLastError).
 *
 * Thread safety: calls may be made concurrently from several host threads;
 * the only shared state is a per-device table of attributes filled once.
 */
#ifndef LINATTN_H
#define LINATTN_H

#include <stddef.h>

#if defined(__GNUC__)
#define LA_API __attribute__((visibility("default")))
#else
#define LA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LA_F32 = 0,  /* q, k, v are float32 */
  LA_BF16 = 1  /* q, k, v are bfloat16 */
} la_dtype;

typedef enum {
  LA_OK = 0,
  LA_ERR_INVALID_VALUE = 1,
  LA_ERR_UNSUPPORTED = 2,
  LA_ERR_MISALIGNED = 3,
  LA_ERR_OUT_OF_MEMORY = 4,
  LA_ERR_LAUNCH = 5,
  LA_ERR_TIMEOUT = 6,
  LA_ERR_NO_DEVICE = 7,
  LA_ERR_TOO_LARGE = 8
} la_status;

/*
 * Global (non-causal) linear attention: every position reads the state of
 * the whole sequence,
 *     S = sum_{j<N} phi(k_j) v_j^T,  z = sum_{j<N} phi(k_j),
 *     out_i = phi(q_i)^T S / (phi(q_i)^T z + eps)      for every i.
 * Source: "线性注意力从头到尾讲清楚" §5 (matrix form) and §8 (the einsum
 * sketch); "Linear Attention Math", "The associativity trick, written out".
 *
 * q, k: [B,H,N,d_k]; v: [B,H,N,d_v] (dtype dt).  out: [B,H,N,d_v] float32,
 * written.  S: [B,H,d_k,d_v], z: [B,H,d_k] float32, OVERWRITTEN with the
 * whole-sequence state (the zero state when N == 0).  May allocate
 * stream-ordered scratch on `stream`.  B*H == 0 is a no-op returning LA_OK.
 */
LA_API la_status la_global(const void *q, const void *k, const void *v, float *out, float *S, float *z,
                    int B, int H, int N, int d_k, int d_v, float eps, la_dtype dt, void *stream);

/*
 * Causal prefill: position t reads the prefix state that INCLUDES token t,
 *     S_t = S_{t-1} + phi(k_t) v_t^T,  z_t = z_{t-1} + phi(k_t),
 *     out_t = phi(q_t)^T S_t / (phi(q_t)^T z_t + eps),   S_{-1} = 0, z_{-1} = 0.
 * Source: "线性注意力从头到尾讲清楚" §7; "Linear Attention Math", "The
 * recurrent form"; "Linear Attention: Accumulating KV in a Fixed-Size
 * State" (token t joins the state before its query reads it).  Computed in
 * chunks ("Linear Attention: From Pairwise Reads to a Recurrent State",
 * "A recurrence need not force token-serial training").
 *
 * Arguments as la_global.  S, z are OVERWRITTEN with the final prefix state
 * S_{N-1}, z_{N-1}, ready to be passed to la_decode_step.
 */
LA_API la_status la_causal(const void *q, const void *k, const void *v, float *out, float *S, float *z,
                    int B, int H, int N, int d_k, int d_v, float eps, la_dtype dt, void *stream);

/*
 * Causal prefill that continues from a given state: as la_causal, but the
 * recurrence starts from the caller's S, z instead of zero (chunked prefill
 * continuation; N new tokens appended to a sequence whose state is S, z).
 * S, z are read, then OVERWRITTEN with the state after the N new tokens.
 * With N == 0 the state is left unchanged.
 * Source: the causal recurrence above applied to a persistent state
 * ("线性注意力从头到尾讲清楚" §7, last paragraph: only S_t, z_t are kept).
 */
LA_API la_status la_causal_with_state(const void *q, const void *k, const void *v, float *out, float *S,
                               float *z, int B, int H, int N, int d_k, int d_v, float eps,
                               la_dtype dt, void *stream);

/*
 * la_causal without any device memory allocation.  The pages have no
 * counterpart to this call; it exists for callers that must not allocate
 * device memory once they are running: serving runtimes that reserve all of
 * their memory up front and forbid allocation after warm-up (so that memory
 * use and latency stay flat), and processes in which another framework's
 * caching allocator already holds nearly all device memory, so that a
 * stream-ordered allocation made by la_causal could fail mid-run.
 *
 * Same arguments, results and errors as la_causal.  The partial states that
 * la_causal allocates per call (for long sequences split into segments: at
 * most two 128x128 fp32 states per first-pass CTA, at most one CTA per SM) live here
 * in one fixed 20 MiB device array inside the library instead; every GPU
 * that loads the library keeps that array until the process exits.  It holds
 * the partial states of 158 first-pass CTAs.  The planner gives the first pass
 * at most one CTA per SM, so on a GB300 (152 SMs) every problem fits; only on
 * a device with more than 158 SMs can a problem need more (B * H * (segments
 * - 1) > 158), and there the call returns LA_ERR_TOO_LARGE and launches
 * nothing.  All calls share the array, so
 * calls whose work overlaps on the GPU (different streams, or different host
 * threads on the same device) race on it and give wrong results: order them.
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  Everything else is enqueued on `stream`; the
 * leading-token pass runs on `stream` too (no second stream is used).
 */
LA_API la_status la_causal_noalloc(const void *q, const void *k, const void *v, float *out, float *S,
                                   float *z, int B, int H, int N, int d_k, int d_v, float eps, la_dtype dt,
                                   void *stream);

/*
 * Positive random features (FAVOR+): for every row x of x ([B,H,N,d]) and the
 * m projections w_r (the rows of W, [m, d]),
 *     phi[b,h,t,r] = exp(w_r . x - |x|^2 / 2) / sqrt(m),
 * so that E[phi(q) . phi(k)] = exp(q . k) for w_r ~ N(0, I).  Source:
 * "Linear Attention Math", "Feature maps: elu+1 and positive random
 * features"; "线性注意力从头到尾讲清楚" §9 (approximating the softmax kernel
 * exp(q^T k / sqrt(d_k)): scale q and k by d_k^(-1/4) first).  W is an input
 * (random or orthogonal random projections, drawn by the caller).
 *
 * x: [B,H,N,d], W: [m,d], phi: [B,H,N,m], all of dtype dt (phi is written).
 * d in {32, 64, 128}; m in {32, 64, 128, 256} (the page notes that more
 * features give a closer approximation; m = 256 is m = 2d at d = 128).
 * Tensor cores for bf16 with m in {128, 256} and d in {64, 128} (one launch
 * per 128 features, each reading x); CUDA cores otherwise.  Allocates
 * nothing.  Errors as la_causal.
 * The features feed la_causal_features (or la_global / la_causal with any
 * caller-side map) as phi(q), phi(k).
 */
LA_API la_status la_favor_features(const void *x, const void *W, void *phi, int B, int H, int N, int d, int m,
                                   la_dtype dt, void *stream);

/*
 * Causal prefill on features the caller has already applied: as la_causal
 * with phi the identity, i.e. out_t = phi_q_t^T S_t / (phi_q_t^T z_t + eps),
 * S_t = sum_{j<=t} phi_k_j v_j^T, z_t = sum_{j<=t} phi_k_j.  For any
 * non-negative feature map, e.g. la_favor_features ("Linear Attention Math",
 * "Feature maps: elu+1 and positive random features": the normalized read
 * needs non-negative features).  phi_q, phi_k: [B,H,N,m] (dtype dt, m in
 * {32, 64, 128}, or 256 with d_v <= 128); S: [B,H,m,d_v]; z: [B,H,m]; other
 * arguments, results and errors as la_causal.  The tensor-core path (bf16,
 * m = d_v = 128) takes the features as given, so no leading tokens are
 * recomputed in fp32; every other size runs the exact fp32 CUDA-core pass
 * (32-token chunks at m = 256, where a 64-token chunk and the 128 KB state
 * would not fit in shared memory).
 */
LA_API la_status la_causal_features(const void *phi_q, const void *phi_k, const void *v, float *out, float *S,
                                    float *z, int B, int H, int N, int m, int d_v, float eps, la_dtype dt,
                                    void *stream);

/*
 * Global (non-causal) read on features the caller has already applied: as
 * la_global with phi the identity.  Arguments, results and errors as
 * la_causal_features.  Computed in fp32 on CUDA cores: the tensor-core
 * global read takes the state as one bf16 operand, which heavy-tailed
 * features (a few keys dominating each read while the state sums all of
 * them) do not tolerate.
 */
LA_API la_status la_global_features(const void *phi_q, const void *phi_k, const void *v, float *out, float *S,
                                    float *z, int B, int H, int N, int m, int d_v, float eps, la_dtype dt,
                                    void *stream);

/*
 * Retention: the causal recurrence with an explicit per-head decay and no
 * denominator,
 *     S_t = gamma_h S_{t-1} + k_t v_t^T,   out_t = q_t^T S_t,   S_{-1} = 0,
 * q and k used as given (no feature map), the read taken after the update as
 * in la_causal.  Source: "Linear Attention Math", "The kernel cousins: SSMs
 * and RetNet" (linear attention plus a decay gamma < 1, fixed or one per
 * head, without the denominator).  The pages' gated normalization that
 * replaces the denominator is a separate layer on top of out and is not
 * part of this call.
 *
 * q, k: [B,H,N,d_k]; v: [B,H,N,d_v] (dtype dt); out: [B,H,N,d_v] float32;
 * S: [B,H,d_k,d_v] float32, OVERWRITTEN with S_{N-1} (zeroed when N == 0).
 * gamma: HOST array of H floats, head h (of every batch row) decaying by
 * gamma[h]; read during the call only.
 *
 * Supported: dt LA_F32 or LA_BF16, d_k and d_v each 32, 64 or 128, H <= 128,
 * every gamma[h] in [0, 1] (gamma = 0 keeps only the current token);
 * anything else returns LA_ERR_UNSUPPORTED.  LA_ERR_INVALID_VALUE for a NULL
 * gamma or a gamma that is not finite; other errors as la_causal.
 *
 * Two kernels serve it.  bf16 with d_k == d_v == 128 on an sm_103 device and
 * every gamma[h] >= 0.75 runs on the tensor cores: that chunked kernel weighs
 * a key 128 tokens ahead by gamma^-128, which must stay well inside float
 * range, and it allocates stream-ordered scratch on `stream` for long
 * sequences split into segments.  Everything else runs on CUDA cores, exact
 * fp32 in 64-token chunks whose decay powers never exceed 1, one CTA per
 * head, allocating nothing.
 */
LA_API la_status la_retention(const void *q, const void *k, const void *v, float *out, float *S,
                              const float *gamma, int B, int H, int N, int d_k, int d_v, la_dtype dt,
                              void *stream);

/*
 * Retention continuing from a given state: as la_retention, but the
 * recurrence starts from the caller's S, which is read and then OVERWRITTEN
 * with the state after the N new tokens (N == 0 leaves it unchanged).
 */
LA_API la_status la_retention_with_state(const void *q, const void *k, const void *v, float *out, float *S,
                                         const float *gamma, int B, int H, int N, int d_k, int d_v,
                                         la_dtype dt, void *stream);

/*
 * Gradient of la_causal / la_causal_with_state.  The pages name training
 * through the chunked causal form ("Linear Attention: From Pairwise Reads to
 * a Recurrent State", "A recurrence need not force token-serial training")
 * but write no backward pass; this is the derivative of the causal
 * definition above.  With den_t = phi(q_t)^T z_t + eps, o_t the output and
 * dO_t its upstream gradient:
 *     gnum_t = dO_t / den_t,   gden_t = -(dO_t . o_t) / den_t
 *     dq_t = (S_t gnum_t + z_t gden_t) * phi'(q_t)
 *     dk_j = (U_j v_j + u_j) * phi'(k_j),   dv_j = U_j^T phi(k_j)
 *     U_j = dS + sum_{t >= j} phi(q_t) gnum_t^T,   u_j = dz + sum_{t >= j} phi(q_t) gden_t
 * and the initial state's gradient is (U_0, u_0).  phi'(x) = 1 for x > 0,
 * exp(x) otherwise.
 *
 * q, k: [B,H,N,d_k]; v: [B,H,N,d_v] (dtype dt), the forward's inputs.
 * dout: [B,H,N,d_v] float32, the gradient of the forward's out.  S0, z0
 * (nullable, each independently; NULL = zero): the forward's initial state.
 * dS, dz (nullable; NULL = zero): the gradient of the forward's final state.
 * dq, dk: [B,H,N,d_k], dv: [B,H,N,d_v] float32, written.  dS0: [B,H,d_k,d_v],
 * dz0: [B,H,d_k] float32 (nullable), written with the initial state's gradient.
 * The forward output is neither read nor formed: dO_t . o_t comes from the
 * state read dO S^T and the chunk's scores.  Allocates stream-ordered scratch
 * on `stream`: B*H*(N*(d_v+1) + 2*64*64*ceil(N/64)) floats (gnum, gden, and
 * each 64-token chunk's masked scores and score gradients), plus, when heads
 * are cut into segments, at most 4 * (SM count) * (d_k*d_v + d_k) floats of
 * segment part sums.  Errors as la_causal; every non-NULL pointer must be
 * 16-byte aligned.  B*H == 0 is a no-op.
 */
LA_API la_status la_causal_backward(const void *q, const void *k, const void *v, const float *dout,
                                    const float *S0, const float *z0, const float *dS, const float *dz,
                                    float *dq, float *dk, float *dv, float *dS0, float *dz0, int B, int H,
                                    int N, int d_k, int d_v, float eps, la_dtype dt, void *stream);

/*
 * One recurrent decode step per (b,h) on a persistent state: update, then
 * read the updated state,
 *     S += phi(k) v^T;  z += phi(k);  out = phi(q)^T S / (phi(q)^T z + eps).
 * Source: "线性注意力从头到尾讲清楚" §7 (inference keeps only S_t, z_t);
 * "Linear Attention Math", "The recurrent form" (O(1) time and memory per
 * generated token).
 *
 * q, k: [B,H,d_k]; v: [B,H,d_v] (dtype dt).  out: [B,H,d_v] float32,
 * written.  S: [B,H,d_k,d_v], z: [B,H,d_k] float32, read and written IN
 * PLACE.  Allocates nothing.
 */
LA_API la_status la_decode_step(const void *q, const void *k, const void *v, float *out, float *S,
                         float *z, int B, int H, int d_k, int d_v, float eps, la_dtype dt,
                         void *stream);

/*
 * One recurrent retention step per (b,h) on a persistent state: decay,
 * update, then read,
 *     S = gamma_h S + k v^T;   out = q^T S,
 * q and k used as given, no normalizer.  Source: "Linear Attention Math",
 * "The kernel cousins: SSMs and RetNet" (the recurrent form of retention).
 * Continues the state left by la_retention / la_retention_with_state.
 *
 * q, k: [B,H,d_k]; v: [B,H,d_v] (dtype dt).  out: [B,H,d_v] float32,
 * written.  S: [B,H,d_k,d_v] float32, read and written IN PLACE.  gamma:
 * HOST array of H floats (head h decays by gamma[h]), read during the call.
 * Allocates nothing.
 *
 * Supported: dt LA_F32 or LA_BF16; d_k, d_v in {32, 64, 128}; H <= 128;
 * every gamma[h] in [0, 1] (else LA_ERR_UNSUPPORTED).  LA_ERR_INVALID_VALUE
 * for a NULL pointer or a gamma that is not finite; LA_ERR_MISALIGNED for a
 * pointer that is not 16-byte aligned.  B*H == 0 is a no-op returning LA_OK.
 */
LA_API la_status la_retention_decode_step(const void *q, const void *k, const void *v, float *out, float *S,
                                          const float *gamma, int B, int H, int d_k, int d_v, la_dtype dt,
                                          void *stream);

/*
 * Gated linear attention: retention whose decay is data, one per token and
 * head,
 *     S_t = e^{g_t} S_{t-1} + k_t v_t^T,   out_t = q_t^T S_t,   S_{-1} = 0,
 * q and k used as given, the read taken after the update.  Source: "Linear
 * Attention Math", "The kernel cousins: SSMs and RetNet" (the decayed update
 * without a denominator); "Linear Attention: From Pairwise Reads to a
 * Recurrent State" (gated unnormalized states).  la_group_norm is the
 * normalization that takes the denominator's place.
 *
 * q, k: [B,H,N,d_k]; v, out: [B,H,N,d_v], all of dtype dt (out too, unlike
 * the normalized forms: the next layer takes the inputs' type).  g:
 * [B,H,N] float32 DEVICE array of natural-log decays, meant to be <= 0.  -inf,
 * and everything below -104 (e^g is zero in float32), resets the state: nothing
 * before the token is read at or after it, whatever the state held and however
 * later decays grow it.  A positive value grows the state; where the growth of
 * up to 128 tokens passes float32's range, or after a decay that is NaN, results
 * may be inf or NaN until a reset in a later chunk.  Chunks are 128 tokens (32 off
 * the tensor cores), and a masked product in one is a product with zero: q, k, v
 * and dout have to be finite, an inf or NaN among them may reach every result of
 * its chunk, those of earlier tokens and behind a reset included.
 * S: [B,H,d_k,d_v] float32, OVERWRITTEN with the
 * final state.  lengths: [B] int32 DEVICE array or NULL (every row has N
 * tokens): tokens t >= lengths[b] of batch row b take no part, whatever they
 * hold; out is left as it was there and S is the state after the last token
 * that does.  Values outside [0, N] are taken as the nearer bound.
 *
 * workspace: at least la_gated_workspace(..., 0) bytes of device memory,
 * 256-byte aligned, free for other use when the call's work on `stream` is done; calls that may run
 * at the same time (two streams, two graphs) need one each.  Nothing is
 * allocated.  d_k, d_v in {32, 64, 128}; dt LA_F32 or LA_BF16; LA_ERR_MISALIGNED
 * for g or lengths off 4 bytes, the workspace off 256 or another pointer off 16; LA_ERR_INVALID_VALUE
 * for a workspace that is too small (NULL where 0 bytes are needed is fine); other errors as la_causal.
 * N == 0 zeroes S.
 */
LA_API la_status la_gated(const void *q, const void *k, const void *v, const float *g, const int *lengths,
                          void *out, float *S, int B, int H, int N, int d_k, int d_v, la_dtype dt,
                          void *workspace, size_t workspace_bytes, void *stream);

/*
 * Gated linear attention continuing from a given state: as la_gated, but the
 * recurrence starts from the caller's S, which is read and then OVERWRITTEN
 * with the state after the new tokens (unchanged for a row without any).
 */
LA_API la_status la_gated_with_state(const void *q, const void *k, const void *v, const float *g,
                                     const int *lengths, void *out, float *S, int B, int H, int N, int d_k,
                                     int d_v, la_dtype dt, void *workspace, size_t workspace_bytes,
                                     void *stream);

/*
 * Workspace bytes of la_gated / la_gated_with_state (backward == 0) or of
 * la_gated_backward (backward != 0) on the current device; 0 when the sizes
 * are invalid or there is nothing to do.
 */
LA_API size_t la_gated_workspace(int B, int H, int N, int d_k, int d_v, la_dtype dt, int backward);

/*
 * Gradient of la_gated / la_gated_with_state: with R_t the gradient of S_t,
 *     R_t = q_t dout_t^T + e^{g_{t+1}} R_{t+1},   R_{N-1} = q dout^T + dS,
 *     dq_t = S_t dout_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,
 *     dg_t = e^{g_t} <S_{t-1}, R_t>,  dS0 = e^{g_0} R_0.
 * q, k, v, g, lengths: the forward's inputs.  dout: [B,H,N,d_v] of dtype dt.
 * S0 (NULL = zero): the forward's initial state.  dS (NULL = zero): gradient
 * of its final state.  Written: dq, dk: [B,H,N,d_k], dv: [B,H,N,d_v], dtype
 * dt; dg: [B,H,N] float32; dS0 (nullable): [B,H,d_k,d_v] float32, gradient of
 * the initial state, which may be dS itself.  No output may overlap an input
 * otherwise (LA_ERR_INVALID_VALUE for dS0 on S0 or on a part of dS).  Rows
 * t >= lengths[b] get zero gradients.  Workspace, sizes and errors as la_gated,
 * with la_gated_workspace(..., 1).
 */
LA_API la_status la_gated_backward(const void *q, const void *k, const void *v, const float *g,
                                   const int *lengths, const void *dout, const float *S0, const float *dS,
                                   void *dq, void *dk, void *dv, float *dg, float *dS0, int B, int H, int N,
                                   int d_k, int d_v, la_dtype dt, void *workspace, size_t workspace_bytes,
                                   void *stream);

/*
 * One recurrent step of gated linear attention per (row, head), on states
 * that live in a pool:
 *     S = e^{g} S + k v^T;   out = q^T S,   S the state of row b's slot.
 * q, k: [B,H,d_k]; v, out: [B,H,d_v], dtype dt; g: [B,H] float32.  S:
 * [n_slots,H,d_k,d_v] float32, the slots of this batch read and written IN
 * PLACE, the others untouched.  A g below -104 (-inf) starts the state anew, also
 * in a slot that was never written.  slots: [B] int32 DEVICE array or NULL (row b
 * uses slot b; n_slots >= B).  A negative slot marks an unused row: no state
 * is touched and its out is zero.  A slot >= n_slots, or one that an earlier
 * row of the batch has, is treated the same way and also makes the next
 * la_device_status return LA_ERR_INVALID_VALUE (two rows on one state have no
 * defined order).  Allocates nothing.  Sizes and errors as la_gated.
 */
LA_API la_status la_gated_decode_step(const void *q, const void *k, const void *v, const float *g, float *S,
                                      const int *slots, void *out, int B, int H, int n_slots, int d_k, int d_v,
                                      la_dtype dt, void *stream);

/*
 * Group norm of each head's channels with an affine map and a SiLU gate, the
 * "gated normalization" that replaces retention's denominator ("Linear
 * Attention Math", "The kernel cousins: SSMs and RetNet"): per token and
 * head, over its d channels,
 *     y = ((x - mean) / sqrt(var + eps) * weight + bias) * gate * sigmoid(gate),
 * var the mean squared deviation.  x: [B,H,N,d] (the attention output's
 * layout); gate (nullable: no gating), y: [B,N,H*d], channels last; all of
 * dtype dt.  weight, bias: [H*d] float32, each nullable (1 and 0).  d in
 * {32, 64, 128}, eps >= 0.  Statistics in fp32.  Every pointer 16-byte
 * aligned; y must not overlap an input.  B*H*N == 0 is a no-op.
 */
LA_API la_status la_group_norm(const void *x, const void *gate, const float *weight, const float *bias, void *y,
                               int B, int H, int N, int d, float eps, la_dtype dt, void *stream);

/*
 * Gradient of la_group_norm for dy ([B,N,H*d], dtype dt).  Written: dx
 * [B,H,N,d] and dgate [B,N,H*d] (given exactly when gate is) of dtype dt;
 * dweight, dbias [H*d] float32, each nullable, whether or not the forward had
 * weight and bias.  No output may overlap an input.  The column sums are added in
 * a fixed order, over all rows: rows of padding tokens need finite x and gate and
 * zeros in dy.  workspace:
 * la_group_norm_workspace bytes when dweight or dbias is wanted (NULL
 * otherwise); calls that may run at the same time need one each.
 */
LA_API la_status la_group_norm_backward(const void *x, const void *dy, const void *gate, const float *weight,
                                        const float *bias, void *dx, void *dgate, float *dweight, float *dbias,
                                        int B, int H, int N, int d, float eps, la_dtype dt, void *workspace,
                                        size_t workspace_bytes, void *stream);
LA_API size_t la_group_norm_workspace(int B, int H, int N, int d);

/*
 * Short causal convolution along the tokens, one window of K weights per
 * channel, the layer in front of the selective scan:
 *     u_t = bias + sum_{j<K} weight_j x_{t-K+1+j},   out_t = silu(u_t)
 * (silu == 0: out_t = u_t), with x_t = 0 before the first token.  Channels
 * last: x: [B,N,D] of dtype dt, whose token rows are ldx elements apart (D
 * when contiguous, more for one part of a wider projection; batch rows N * ldx
 * apart); out: [B,N,D], dtype dt.  weight: [D,K], bias: [D] (nullable), float32.
 * S: [B,K-1,D], dtype dt, the last K - 1 inputs, written.  lengths (nullable,
 * [B] int32, device): tokens t >= lengths[b] take no part and their rows of out
 * are not written.  D a multiple of 8, K in {2, 3, 4}.
 * la_short_conv_with_state starts from the window in S and updates it in
 * place.  Sums in fp32.  Pointers 16-byte aligned (lengths 4), ldx >= D and a
 * multiple of 16 bytes.  out and S must overlap neither an input nor each other.
 * N == 0 leaves the carried window (zeros without one).
 */
LA_API la_status la_short_conv(const void *x, long ldx, const float *weight, const float *bias, const int *lengths,
                               void *out, void *S, int B, int N, int D, int K, int silu, la_dtype dt, void *stream);
LA_API la_status la_short_conv_with_state(const void *x, long ldx, const float *weight, const float *bias,
                                          const int *lengths, void *out, void *S, int B, int N, int D, int K, int silu,
                                          la_dtype dt, void *stream);

/*
 * Gradient of la_short_conv(_with_state): dout [B,N,D], dtype dt, contiguous;
 * S0 (NULL = zero) the forward's window, dS (NULL = zero) the gradient of the
 * one it left, both [B,K-1,D], dtype dt.  Written: dx [B,N,D] and dS0 (nullable)
 * of dtype dt; dweight [D,K], dbias [D] float32, each nullable, added in a fixed
 * order.  Rows t >= lengths[b] of dx are zero.  No output may overlap an input
 * (dS0: neither S0 nor dS) or another output.  workspace: la_short_conv_workspace bytes, 256-byte aligned, when dweight
 * or dbias is wanted (NULL otherwise); calls that may run at the same time need
 * one each.
 */
LA_API la_status la_short_conv_backward(const void *x, long ldx, const float *weight, const float *bias,
                                        const int *lengths, const void *dout, const void *S0, const void *dS, void *dx,
                                        float *dweight, float *dbias, void *dS0, int B, int N, int D, int K, int silu,
                                        la_dtype dt, void *workspace, size_t workspace_bytes, void *stream);
LA_API size_t la_short_conv_workspace(int B, int N, int D, int K);

/*
 * One token of la_short_conv per batch row, on windows that live in a pool S
 * [n_slots,K-1,D], dtype dt, read and written in place: row b works on
 * S[slots[b]].  x: [B,D], rows ldx apart; out: [B,D].  slots as in
 * la_gated_decode_step (unused, bad and repeated ones too).  out and S must overlap
 * neither an input nor each other.  Allocates nothing.
 */
LA_API la_status la_short_conv_step(const void *x, long ldx, const float *weight, const float *bias, void *S,
                                    const int *slots, void *out, int B, int n_slots, int D, int K, int silu, la_dtype dt,
                                    void *stream);

/*
 * Selective state space scan, per channel with d_state components ("Linear
 * Attention Math", "The kernel cousins: SSMs and RetNet", with steps and
 * projections that depend on the token):
 *     delta = softplus(dt + dt_bias)  (softplus == 0: dt + dt_bias)
 *     h_t = e^{delta A} h_{t-1} + (delta x_t) B_t
 *     out_t = (C_t . h_t + D x_t) silu(z_t)
 * x, delta (dt above), z (nullable: no gate): [B,N,D]; Bm, Cm (B_t and C_t, shared by
 * all channels): [B,N,d_state]; all of dtype dt, token rows ld* elements apart
 * (parts of wider projections; batch rows N * ld* apart).  A: [D,d_state], Dskip
 * (nullable: 0) and dt_bias (nullable: 0): [D], float32.  Written: out [B,N,D],
 * dtype dt; S [B,D,d_state] float32, the final state.  lengths as in
 * la_short_conv.  la_selective_scan_with_state starts from S and updates it in
 * place.  Steps, states and sums in fp32.  D a multiple of 8, d_state in {8, 16,
 * 32, 64}; pointers 16-byte aligned (lengths 4), every ld at least its row and a
 * multiple of 16 bytes.  out and S must overlap neither an input nor each other.  workspace:
 * la_selective_scan_workspace(..., 0) bytes, 256-byte aligned (NULL if that is 0);
 * calls that may run at the same time need one each.  N == 0 leaves the carried
 * state (zeros without one).
 */
LA_API la_status la_selective_scan(const void *x, long ldx, const void *delta, long ld_delta, const float *A,
                                   const void *Bm, long ldb, const void *Cm, long ldc, const float *Dskip, const void *z,
                                   long ldz, const float *dt_bias, const int *lengths, void *out, float *S, int B, int N,
                                   int D, int d_state, int softplus, la_dtype dt, void *workspace,
                                   size_t workspace_bytes, void *stream);
LA_API la_status la_selective_scan_with_state(const void *x, long ldx, const void *delta, long ld_delta, const float *A,
                                              const void *Bm, long ldb, const void *Cm, long ldc, const float *Dskip,
                                              const void *z, long ldz, const float *dt_bias, const int *lengths,
                                              void *out, float *S, int B, int N, int D, int d_state, int softplus,
                                              la_dtype dt, void *workspace, size_t workspace_bytes, void *stream);
LA_API size_t la_selective_scan_workspace(int B, int N, int D, int d_state, la_dtype dt, int backward);

/*
 * Gradient of la_selective_scan(_with_state): with dy = dout silu(z) and G_t the
 * gradient of h_t,
 *     G_t = C_t dy_t + e^{delta_{t+1} A} G_{t+1},  behind the last token G = dS,
 *     dx = D dy + delta (G . B),  d delta = x (G . B) + (G e^{delta A} h_{t-1}) . A,
 *     dB_t = sum over channels of G delta x,  dC_t = sum over channels of h dy.
 * dout [B,N,D], dtype dt, contiguous; S0 (NULL = zero) the forward's initial state,
 * dS (NULL = zero) the gradient of its final one.  Written, contiguous: dx, ddelta
 * (of dt, before its bias) [B,N,D], dB, dC [B,N,d_state], dz [B,N,D] (given
 * exactly when z is), dtype dt; dA [D,d_state], dDskip, ddt_bias [D], dS0
 * [B,D,d_state] (which may be dS itself), float32, each nullable.  Rows t >=
 * lengths[b] are zero.  All sums in a fixed order.  No output may overlap an input
 * or another output otherwise.  workspace: la_selective_scan_workspace(..., 1) bytes, 256-byte
 * aligned; calls that may run at the same time need one each.
 */
LA_API la_status la_selective_scan_backward(const void *x, long ldx, const void *delta, long ld_delta, const float *A,
                                            const void *Bm, long ldb, const void *Cm, long ldc, const float *Dskip,
                                            const void *z, long ldz, const float *dt_bias, const int *lengths,
                                            const void *dout, const float *S0, const float *dS, void *dx, void *ddelta,
                                            float *dA, void *dB, void *dC, float *dDskip, void *dz, float *ddt_bias,
                                            float *dS0, int B, int N, int D, int d_state, int softplus, la_dtype dt,
                                            void *workspace, size_t workspace_bytes, void *stream);

/*
 * One token of la_selective_scan per batch row, on states that live in a pool S
 * [n_slots,D,d_state] float32, read and written in place: row b works on
 * S[slots[b]].  x, delta, z: [B,D]; Bm, Cm: [B,d_state]; rows ld* apart; out
 * [B,D].  slots as in la_gated_decode_step (unused, bad and repeated ones too).  out
 * and S must overlap neither an input nor each other.
 */
LA_API la_status la_selective_scan_step(const void *x, long ldx, const void *delta, long ld_delta, const float *A,
                                        const void *Bm, long ldb, const void *Cm, long ldc, const float *Dskip,
                                        const void *z, long ldz, const float *dt_bias, float *S, const int *slots,
                                        void *out, int B, int n_slots, int D, int d_state, int softplus, la_dtype dt,
                                        void *stream);

/*
 * Beam search, selection: of each group's W beams with accumulated log
 * probabilities `scores` ([G,W] float32, finite or -inf) and next-token logits
 * ([G,W,V], dtype dt, rows ld elements apart), the k best continuations by
 *     scores_w + logits_{w,v} - log sum_v' e^{logits_{w,v'}},
 * best first, ties to the lowest w V + v.  Within a beam the logits decide.  Between
 * beams the scores are added and compared in 64 bits, but for the sum over v', whose
 * exponentials are float32 and added in float32: its logarithm was off by 4e-7 at
 * most where measured (up to 131072 tokens, any spread), and is by no more than
 * 2^-22 + (28 + 3 log V + 8 ceil(V / 4096)) 2^-24, 2e-5 at 131072 tokens.
 * Continuations of different beams nearer than twice that may change places; beams
 * of equal logits have equal sums and tie.  Written, [G,k]: out_scores
 * float32, parents (w) and tokens (v) int32.  finished (nullable, [G,W], one byte
 * each): a finished beam has one continuation, token eos, and keeps its score.
 * Everything else is -inf: a logit of -inf or NaN, all continuations of a beam
 * whose score is -inf or NaN; where nothing else is left these are chosen too, with
 * score -inf.  Infinite logits count as the largest finite number.  1 <= k <=
 * min(64, W V), W <= 64, 0 <= eos < V, ld >= V.  logits 16-byte aligned, the other
 * pointers 4 (finished 1).  workspace: la_beam_select_workspace bytes, 256-byte
 * aligned; calls that may run at the same time need one each.  No output may
 * overlap an input or another output.
 */
LA_API la_status la_beam_select(const void *logits, long ld, const float *scores, const unsigned char *finished,
                                float *out_scores, int *parents, int *tokens, int G, int W, int k, int V, int eos,
                                la_dtype dt, void *workspace, size_t workspace_bytes, void *stream);
LA_API size_t la_beam_select_workspace(int G, int W, int k, int V, la_dtype dt);

/*
 * Beam search, states: pools of states follow the beams that were chosen.
 * slots [G,W] int32: the slot of each beam's state in every pool; parents [G,W]
 * int32: the beam that each new beam continues.  The first child of a beam keeps
 * its slot; the others get the slots of the group's childless beams, lowest beam
 * first, and a copy of their parent's row there, in place, in each of n_pools
 * pools (host arrays of device pointers [n_slots, row_bytes] and row sizes, a
 * multiple of 16 bytes each; pools 16-byte aligned).  new_slots [G,W] int32,
 * written, not overlapping slots, parents or a pool, nor may a pool overlap these.
 * A negative parent takes a childless beam's slot
 * without a copy, and nothing is copied from or to a negative slot.  A parent >= W,
 * a slot >= n_slots that a copy reads or writes, and a slot to be written that
 * another beam of the call has too: no copy, and the next la_device_status returns
 * LA_ERR_INVALID_VALUE.  W <= 64.  Allocates nothing.
 */
LA_API la_status la_beam_reorder(void *const *pools, const size_t *row_bytes, int n_pools, const int *slots,
                                 const int *parents, int *new_slots, int G, int W, int n_slots, void *stream);

/*
 * Synchronizes `stream`, then reads and clears the library's device status
 * word on the current device.  Returns LA_ERR_TIMEOUT if a bounded
 * device-side wait inside one of the library's kernels gave up since the
 * last check, LA_ERR_LAUNCH if a kernel refused to run on this device
 * configuration (its shared-memory base was not 1024-byte aligned); in both
 * cases that call's outputs are not valid.  LA_ERR_INVALID_VALUE if a
 * la_gated_decode_step, la_short_conv_step or la_selective_scan_step skipped a
 * row, or a la_beam_reorder a copy, whose slot was out of range or repeated.
 * LA_OK otherwise, or the error of the synchronization itself.
 */
LA_API la_status la_device_status(void *stream);

/*
 * Diagnostics, for measuring the carry of the causal prefill: fixes how many
 * segments each head is cut into by the tensor-core passes of la_causal,
 * la_causal_with_state, la_causal_features and la_retention (1 = one CTA
 * carries each head's state through all of its chunks; G > 1 = G segments
 * whose starting states come from the first pass over the earlier ones),
 * clamped to the number of 128-token chunks.  0 restores the planner's
 * choice (enough segments to cover the SMs once, at least 4 chunks each).
 * Process-wide; results are the same up to rounding for every value.
 * la_causal_noalloc ignores it.  LA_ERR_INVALID_VALUE outside [0, 4096].
 */
LA_API la_status la_diag_force_segments(int segments);
/*
 * Testing only: exercises the bounded-wait failure path on the GPU without a
 * fault.  Arms a one-shot injection taken by the NEXT launch of the
 * tensor-core causal pass (la_causal, la_causal_with_state or
 * la_causal_noalloc with bf16 inputs and d_k = d_v = 128), from any host
 * thread: in that launch the first CTA (segment 0 of head 0) does not issue
 * the key load of chunk `chunk` (128-token chunks of its segment), and every
 * mbarrier wait of the launch gives up after wait_us microseconds instead of
 * 4 s.  The waits that depend on the missing load run out; the CTA raises its
 * abort word, drains the copies and tensor-core work already issued, frees its
 * tensor memory and exits, and the next la_device_status returns
 * LA_ERR_TIMEOUT.  That call's outputs are not valid; later calls are
 * unaffected.  If the chunk does not exist in that launch nothing is left out.
 * LA_ERR_INVALID_VALUE for chunk < 0 or wait_us outside [1, 1000000].  No
 * counterpart in the pages: it tests this library's error reporting.
 */
LA_API la_status la_test_inject_missing_load(int chunk, unsigned int wait_us);
/* Static English description of a status code (never NULL). */
LA_API const char *la_status_string(la_status s);

/* Library ABI version: (major << 16) | minor. */
LA_API int la_version(void);

/*
 * Diagnostics: name and description of the CUDA runtime error behind the
 * last LA_ERR_LAUNCH / LA_ERR_OUT_OF_MEMORY / LA_ERR_NO_DEVICE returned to
 * the calling host thread ("no error" if none).  Static storage; never NULL.
 */
LA_API const char *la_last_error_detail(void);

/*
 * Diagnostics: number of kernels this library has enqueued in this process
 * (all devices, all threads; a relaxed atomic counter incremented at every
 * successful launch).  Read it before and after a region to count the
 * library's launches inside it.
 */
LA_API unsigned long long la_kernel_launches(void);

/* Kernels whose device time la_profile_read reports. */
typedef enum {
  LA_KERNEL_CAUSAL_MAIN = 0,   /* tensor-core causal pass (bf16, d_k = d_v = 128) */
  LA_KERNEL_CAUSAL_STATE = 1,  /* its state-only first pass over earlier segments */
  LA_KERNEL_EXACT_HEAD = 2,    /* exact fp32 pass over each head's leading tokens */
  LA_KERNEL_CAUSAL_SIMT = 3,   /* fp32 chunked causal kernel (other shapes) */
  LA_KERNEL_GLOBAL_STATE = 4,  /* global form: state build */
  LA_KERNEL_GLOBAL_READ = 5,   /* global form: read */
  LA_KERNEL_DECODE = 6,         /* recurrent decode step */
  LA_KERNEL_RETENTION_MAIN = 7,   /* tensor-core retention pass */
  LA_KERNEL_RETENTION_STATE = 8,  /* its first pass over earlier segments */
  LA_KERNEL_RETENTION_DECODE = 9, /* recurrent retention step */
  LA_KERNEL_BACKWARD = 10,        /* causal backward */
  LA_KERNEL_FAVOR = 11,           /* positive random features */
  LA_KERNEL_GLOBAL_FUSED = 12,    /* global form in one pass: a CTA per head (d = 64, heads >= 80 % of SMs) */
  LA_KERNEL_GATED = 13,           /* gated linear attention: outputs */
  LA_KERNEL_GATED_STATE = 14,     /* its passes over chunk states, forward and backward */
  LA_KERNEL_GATED_BACKWARD = 15,  /* its gradient */
  LA_KERNEL_GATED_DECODE = 16,    /* its recurrent step */
  LA_KERNEL_GROUP_NORM = 17,      /* gated group norm */
  LA_KERNEL_GROUP_NORM_BACKWARD = 18, /* its gradient */
  LA_KERNEL_SHORT_CONV = 19,          /* short causal convolution */
  LA_KERNEL_SHORT_CONV_BACKWARD = 20, /* its gradient */
  LA_KERNEL_SHORT_CONV_STEP = 21,     /* its step */
  LA_KERNEL_SELECTIVE_SCAN = 22,      /* selective scan: outputs */
  LA_KERNEL_SELECTIVE_STATE = 23,     /* its passes over states, forward and backward */
  LA_KERNEL_SELECTIVE_BACKWARD = 24,  /* its gradient */
  LA_KERNEL_SELECTIVE_STEP = 25,      /* its step */
  LA_KERNEL_BEAM_SELECT = 26,         /* beam selection */
  LA_KERNEL_BEAM_REORDER = 27         /* states following their beams */
} la_kernel;

/*
 * Diagnostics: per-kernel device time.  la_profile_enable(1) clears the
 * totals and from then on brackets every launch of this library with a CUDA
 * event pair recorded on the launch's own stream (two event creations and
 * records per launch: host cost only, nothing is added to the kernels);
 * la_profile_enable(0) stops recording.  la_profile_read waits for the
 * recorded pairs to complete and returns, for one kernel, the summed
 * milliseconds between its events and the number of timed launches since
 * the last enable.  A kernel that shares the GPU with a concurrent one (the
 * exact leading-token pass runs beside the tensor-core pass) is timed as it
 * ran, contention included.  Thread-safe.  Errors: LA_ERR_INVALID_VALUE for an
 * unknown kernel or NULL outputs; a failed event query maps like a launch
 * error (the totals still hold the pairs that completed).
 */
LA_API la_status la_profile_enable(int on);
LA_API la_status la_profile_read(la_kernel kernel, double *ms_total, long long *launches);

#ifdef __cplusplus
}
#endif

#endif /* LINATTN_H */
