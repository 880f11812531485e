// C ABI of the short convolution, the selective scan and beam search: argument validation and dispatch
// (see linattn.h for the contract of each call).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>
#include <utility>

#include "internal.h"
#include "linattn.h"

namespace la {
namespace {

bool aligned(std::initializer_list<const void *> ptrs, uintptr_t to) {
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return false;
  return true;
}
bool missing(std::initializer_list<const void *> ptrs) {
  for (const void *p : ptrs)
    if (!p) return true;
  return false;
}
bool overlap(const void *a, const void *b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && (x < y ? y - x : x - y) < bytes;
}
// Memory of `an` bytes at a and of `bn` at b.
bool meets(const void *a, size_t an, const void *b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && an && bn && x < y + bn && y < x + an;
}
int bytes_of(la_dtype dt) { return dt == LA_F32 ? 4 : 2; }

// Rows of `width` values, `ld` apart: long enough and 16-byte aligned, and the whole tensor addressable.
la_status rows_ok(long ld, long width, la_dtype dt) {
  if (ld < width || ld > 0x7fffffffL) return LA_ERR_INVALID_VALUE;
  return ld * bytes_of(dt) % 16 ? LA_ERR_MISALIGNED : LA_OK;
}
la_status all_rows_ok(std::initializer_list<std::pair<long, long>> rows, la_dtype dt) {
  la_status st = LA_OK;
  for (const auto &r : rows) {
    const la_status s = rows_ok(r.first, r.second, dt);
    if (s == LA_ERR_INVALID_VALUE) return s;
    if (s != LA_OK) st = s;
  }
  return st;
}

// Memory that a call reads or writes; null: none.
struct Span {
  const void *at;
  size_t bytes;
};
// `count` rows (one at least) of `width` values, `ld` apart.
Span rows(const void *at, long count, long ld, long width, la_dtype dt) {
  return {at, ((count - 1) * (size_t)ld + width) * bytes_of(dt)};
}
Span floats(const void *at, long count) { return {at, sizeof(float) * (size_t)count}; }
// Whether an output meets an input or another output.
bool over(std::initializer_list<Span> outputs, std::initializer_list<Span> inputs) {
  for (const Span *o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Span &i : inputs)
      if (meets(o->at, o->bytes, i.at, i.bytes)) return true;
    for (const Span *q = outputs.begin(); q != o; ++q)
      if (meets(o->at, o->bytes, q->at, q->bytes)) return true;
  }
  return false;
}

// Every launch counts its blocks, of at least eight channels and a token each, in 31 bits.
la_status sizes(int B, long N, int D, la_dtype dt) {
  if (B < 0 || N < 0 || D <= 0) return LA_ERR_INVALID_VALUE;
  if (B > 0 && ((long)D * B > 0x7fffffffL || (long)B * D / 8 * ((N + 15) / 16) > 0x7fffffffL || (long)B * N > 0x3ffffffffL / 8))
    return LA_ERR_INVALID_VALUE;
  if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_UNSUPPORTED;
  return D % 8 ? LA_ERR_UNSUPPORTED : LA_OK;
}
la_status conv_sizes(int B, long N, int D, int K, la_dtype dt) {
  if (K <= 0) return LA_ERR_INVALID_VALUE;
  const la_status st = sizes(B, N, D, dt);
  return st != LA_OK ? st : K < 2 || K > 4 ? LA_ERR_UNSUPPORTED : LA_OK;
}
la_status scan_sizes(int B, long N, int D, int ds, la_dtype dt) {
  if (ds <= 0) return LA_ERR_INVALID_VALUE;
  const la_status st = sizes(B, N, D, dt);
  if (st != LA_OK) return st;
  if (ds != 8 && ds != 16 && ds != 32 && ds != 64) return LA_ERR_UNSUPPORTED;
  return (long)D * ds > 0x7fffffffL || (long)B * N * ds > 0x7fffffffL * 64 ? LA_ERR_INVALID_VALUE : LA_OK;
}

// A carried state that no token changes: zero, or as it is.
la_status empty(void *S, size_t bytes, bool from_state, void *stream) {
  if (from_state) return LA_OK;
  const la_status st = api_device();
  return st != LA_OK ? st : api_status(cudaMemsetAsync(S, 0, bytes, (cudaStream_t)stream));
}
// Its gradient.
cudaError_t pass_through(void *dS0, const void *dS, size_t bytes, cudaStream_t s) {
  if (!dS0 || dS0 == dS) return cudaSuccess;
  return dS ? cudaMemcpyAsync(dS0, dS, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dS0, 0, bytes, s);
}

la_status conv(const void *x, long ldx, const float *weight, const float *bias, const int *lengths, void *out, void *S,
               int B, int N, int D, int K, int silu, la_dtype dt, void *stream, bool from_state) {
  la_status st = conv_sizes(B, N, D, K, dt);
  if (st != LA_OK) return st;
  if (B == 0) return LA_OK;
  if (!S || (N > 0 && missing({x, weight, out}))) return LA_ERR_INVALID_VALUE;
  if ((st = rows_ok(ldx, D, dt)) != LA_OK) return st;
  if (!aligned({x, weight, bias, out, S}, 16) || !aligned({lengths}, 4)) return LA_ERR_MISALIGNED;
  if (N == 0) return empty(S, (size_t)B * (K - 1) * D * bytes_of(dt), from_state, stream);
  const long tokens = (long)B * N;
  if (over({rows(out, tokens, D, D, dt), rows(S, (long)B * (K - 1), D, D, dt)},
           {rows(x, tokens, ldx, D, dt), floats(weight, (long)D * K), floats(bias, D), floats(lengths, B)}))
    return LA_ERR_INVALID_VALUE;
  if ((st = api_device()) != LA_OK) return st;
  return api_status(launch_short_conv(
      {x, ldx, weight, bias, lengths, from_state, out, S, B, N, D, K, silu != 0, dt, (cudaStream_t)stream}));
}

la_status scan(const void *x, long ldx, const void *delta, long ldt, const float *A, const void *Bm, long ldb,
               const void *Cm, long ldc, const float *Dskip, const void *z, long ldz, const float *dt_bias,
               const int *lengths, void *out, float *S, int B, int N, int D, int ds, int softplus, la_dtype dt, void *ws,
               size_t ws_bytes, void *stream, bool from_state) {
  la_status st = scan_sizes(B, N, D, ds, dt);
  if (st != LA_OK) return st;
  if (B == 0) return LA_OK;
  if (!S || (N > 0 && missing({x, delta, A, Bm, Cm, out}))) return LA_ERR_INVALID_VALUE;
  if ((st = all_rows_ok({{ldx, D}, {ldt, D}, {ldb, ds}, {ldc, ds}, {z ? ldz : ldx, D}}, dt)) != LA_OK) return st;
  if (!aligned({x, delta, A, Bm, Cm, Dskip, z, dt_bias, out, S}, 16) || !aligned({ws}, 256) || !aligned({lengths}, 4))
    return LA_ERR_MISALIGNED;
  if (N == 0) return empty(S, sizeof(float) * (size_t)B * D * ds, from_state, stream);
  const long tokens = (long)B * N;
  if (over({rows(out, tokens, D, D, dt), floats(S, (long)B * D * ds)},
           {rows(x, tokens, ldx, D, dt), rows(delta, tokens, ldt, D, dt), rows(z, tokens, ldz, D, dt),
            rows(Bm, tokens, ldb, ds, dt), rows(Cm, tokens, ldc, ds, dt), floats(A, (long)D * ds), floats(Dskip, D),
            floats(dt_bias, D), floats(lengths, B)}))
    return LA_ERR_INVALID_VALUE;
  if ((st = api_device()) != LA_OK) return st;
  const ScanProblem p{x, delta, z, Bm, Cm, ldx, ldt, ldz, ldb, ldc, A, Dskip, dt_bias, lengths, from_state ? S : nullptr,
                      out, S, B, N, D, ds, softplus != 0, dt, ws, (cudaStream_t)stream};
  const size_t need = scan_workspace(p);
  if (ws_bytes < need || (need && !ws)) return LA_ERR_INVALID_VALUE;
  return api_status(launch_selective_scan(p));
}

la_status beam_sizes(int G, int W, int k, long V, la_dtype dt) {
  if (G < 0 || W <= 0 || V <= 0 || k <= 0 || k > (long)W * V) return LA_ERR_INVALID_VALUE;
  if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_UNSUPPORTED;
  if (W > 64 || k > 64) return LA_ERR_UNSUPPORTED;
  return (long)G * W * ((V + kBeamChunk - 1) / kBeamChunk + 1) > 0x7fffffffL ? LA_ERR_INVALID_VALUE : LA_OK;
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

la_status la_short_conv(const void *x, long ldx, const float *weight, const float *bias, const int *lengths, void *out,
                        void *S, int B, int N, int D, int K, int silu, la_dtype dt, void *stream) {
  return conv(x, ldx, weight, bias, lengths, out, S, B, N, D, K, silu, dt, stream, false);
}

la_status la_short_conv_with_state(const void *x, long ldx, const float *weight, const float *bias, const int *lengths,
                                   void *out, void *S, int B, int N, int D, int K, int silu, la_dtype dt, void *stream) {
  return conv(x, ldx, weight, bias, lengths, out, S, B, N, D, K, silu, dt, stream, true);
}

size_t la_short_conv_workspace(int B, int N, int D, int K) {
  if (conv_sizes(B, N, D, K, LA_F32) != LA_OK || B == 0 || N == 0) return 0;
  ConvProblem p{};
  p.B = B, p.N = N, p.D = D, p.K = K;
  return short_conv_grad_workspace(p);
}

la_status la_short_conv_backward(const void *x, long ldx, const float *weight, const float *bias, const int *lengths,
                                 const void *dout, const void *S0, const void *dS, void *dx, float *dweight,
                                 float *dbias, void *dS0, int B, int N, int D, int K, int silu, la_dtype dt,
                                 void *workspace, size_t workspace_bytes, void *stream) {
  la_status st = conv_sizes(B, N, D, K, dt);
  if (st != LA_OK) return st;
  if (B > 0 && N > 0 && missing({x, weight, dout, dx})) return LA_ERR_INVALID_VALUE;
  if (B > 0 && (st = rows_ok(ldx, D, dt)) != LA_OK) return st;
  if (!aligned({x, weight, bias, dout, S0, dS, dx, dS0}, 16) || !aligned({workspace}, 256) ||
      !aligned({lengths, dweight, dbias}, 4))
    return LA_ERR_MISALIGNED;
  const size_t window = (size_t)B * (K - 1) * D * bytes_of(dt);
  if (dS != dS0 && overlap(dS, dS0, window)) return LA_ERR_INVALID_VALUE;
  // a run of tokens reads what belongs to the ones beside it, and runs are in no order
  const long tokens = (long)B * N;
  if (tokens > 0 && over({rows(dx, tokens, D, D, dt), {dS0, window}, floats(dweight, (long)D * K), floats(dbias, D)},
                         {rows(x, tokens, ldx, D, dt), rows(dout, tokens, D, D, dt), {S0, window}, {dS, window},
                          floats(weight, (long)D * K), floats(bias, D), floats(lengths, B)}))
    return LA_ERR_INVALID_VALUE;
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = api_device()) != LA_OK) return st;
  if (B == 0 || N == 0) {  // the sums are empty, the window passes through
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)D * K, s);
    if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, sizeof(float) * (size_t)D, s);
    if (B > 0 && e == cudaSuccess) e = pass_through(dS0, dS, window, s);
    return api_status(e);
  }
  const ConvGradProblem q{{x, ldx, weight, bias, lengths, false, nullptr, nullptr, B, N, D, K, silu != 0, dt, s},
                          dout, S0, dS, dx, dweight, dbias, dS0, (float *)workspace};
  if ((dweight || dbias) && (!workspace || workspace_bytes < short_conv_grad_workspace(q.p))) return LA_ERR_INVALID_VALUE;
  return api_status(launch_short_conv_grad(q));
}

la_status la_short_conv_step(const void *x, long ldx, const float *weight, const float *bias, void *S, const int *slots,
                             void *out, int B, int n_slots, int D, int K, int silu, la_dtype dt, void *stream) {
  la_status st = conv_sizes(B, 1, D, K, dt);
  if (st != LA_OK) return st;
  if (n_slots < 0 || (!slots && n_slots < B)) return LA_ERR_INVALID_VALUE;
  if (B == 0) return LA_OK;
  if (missing({x, weight, out}) || (!S && n_slots > 0)) return LA_ERR_INVALID_VALUE;
  if ((st = rows_ok(ldx, D, dt)) != LA_OK) return st;
  if (!aligned({x, weight, bias, S, out}, 16) || !aligned({slots}, 4)) return LA_ERR_MISALIGNED;
  if (over({rows(out, B, D, D, dt), {S, (size_t)n_slots * (K - 1) * D * bytes_of(dt)}},
           {rows(x, B, ldx, D, dt), floats(weight, (long)D * K), floats(bias, D), floats(slots, B)}))
    return LA_ERR_INVALID_VALUE;
  if ((st = api_device()) != LA_OK) return st;
  return api_status(launch_short_conv_step(
      {x, ldx, weight, bias, S, slots, out, B, D, K, n_slots, silu != 0, dt, (cudaStream_t)stream}));
}

la_status la_selective_scan(const void *x, long ldx, const void *delta, long ld_delta, const float *A, const void *Bm,
                            long ldb, const void *Cm, long ldc, const float *Dskip, const void *z, long ldz,
                            const float *dt_bias, const int *lengths, void *out, float *S, int B, int N, int D,
                            int d_state, int softplus, la_dtype dt, void *workspace, size_t workspace_bytes,
                            void *stream) {
  return scan(x, ldx, delta, ld_delta, A, Bm, ldb, Cm, ldc, Dskip, z, ldz, dt_bias, lengths, out, S, B, N, D, d_state,
              softplus, dt, workspace, workspace_bytes, stream, false);
}

la_status la_selective_scan_with_state(const void *x, long ldx, const void *delta, long ld_delta, const float *A,
                                       const void *Bm, long ldb, const void *Cm, long ldc, const float *Dskip,
                                       const void *z, long ldz, const float *dt_bias, const int *lengths, void *out,
                                       float *S, int B, int N, int D, int d_state, int softplus, la_dtype dt,
                                       void *workspace, size_t workspace_bytes, void *stream) {
  return scan(x, ldx, delta, ld_delta, A, Bm, ldb, Cm, ldc, Dskip, z, ldz, dt_bias, lengths, out, S, B, N, D, d_state,
              softplus, dt, workspace, workspace_bytes, stream, true);
}

size_t la_selective_scan_workspace(int B, int N, int D, int d_state, la_dtype dt, int backward) {
  if (scan_sizes(B, N, D, d_state, dt) != LA_OK || B == 0 || N == 0) return 0;
  ScanProblem p{};
  p.B = B, p.N = N, p.D = D, p.ds = d_state, p.dt = dt;
  return scan_workspace_any(p, backward ? scan_grad_workspace : scan_workspace);
}

la_status la_selective_scan_backward(const void *x, long ldx, const void *delta, long ld_delta, const float *A,
                                     const void *Bm, long ldb, const void *Cm, long ldc, const float *Dskip,
                                     const void *z, long ldz, const float *dt_bias, const int *lengths, const void *dout,
                                     const float *S0, const float *dS, void *dx, void *ddelta, float *dA, void *dB,
                                     void *dC, float *dDskip, void *dz, float *ddt_bias, float *dS0, int B, int N, int D,
                                     int d_state, int softplus, la_dtype dt, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  la_status st = scan_sizes(B, N, D, d_state, dt);
  if (st != LA_OK) return st;
  if (B > 0 && N > 0 && (missing({x, delta, A, Bm, Cm, dout, dx, ddelta, dB, dC}) || (z != nullptr) != (dz != nullptr)))
    return LA_ERR_INVALID_VALUE;
  if (B > 0 && (st = all_rows_ok({{ldx, D}, {ld_delta, D}, {ldb, d_state}, {ldc, d_state}, {z ? ldz : ldx, D}}, dt)) != LA_OK)
    return st;
  if (!aligned({x, delta, A, Bm, Cm, Dskip, z, dt_bias, dout, S0, dS, dx, ddelta, dB, dC, dz, dS0}, 16) ||
      !aligned({workspace}, 256) || !aligned({lengths, dA, dDskip, ddt_bias}, 4))
    return LA_ERR_MISALIGNED;
  const size_t bytes = sizeof(float) * (size_t)B * D * d_state;
  if (dS != dS0 && overlap(dS, dS0, bytes)) return LA_ERR_INVALID_VALUE;
  // rows are read again when a chunk's results go out, by every block of channels at its own pace; the state and its
  // gradient are walked in opposite directions, neither waits for the other
  const long tokens = (long)B * N;
  if (tokens > 0 &&
      over({rows(dx, tokens, D, D, dt), rows(ddelta, tokens, D, D, dt), rows(dz, tokens, D, D, dt),
            rows(dB, tokens, d_state, d_state, dt), rows(dC, tokens, d_state, d_state, dt), floats(dA, (long)D * d_state),
            floats(dDskip, D), floats(ddt_bias, D), {dS0, bytes}},
           {rows(x, tokens, ldx, D, dt), rows(delta, tokens, ld_delta, D, dt), rows(z, tokens, ldz, D, dt),
            rows(Bm, tokens, ldb, d_state, dt), rows(Cm, tokens, ldc, d_state, dt), rows(dout, tokens, D, D, dt),
            floats(A, (long)D * d_state), floats(Dskip, D), floats(dt_bias, D), floats(lengths, B), {S0, bytes},
            {dS == dS0 ? nullptr : dS, bytes}}))
    return LA_ERR_INVALID_VALUE;
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = api_device()) != LA_OK) return st;
  if (B == 0 || N == 0) {  // the sums are empty, the state passes through
    cudaError_t e = cudaSuccess;
    if (dA) e = cudaMemsetAsync(dA, 0, sizeof(float) * (size_t)D * d_state, s);
    if (dDskip && e == cudaSuccess) e = cudaMemsetAsync(dDskip, 0, sizeof(float) * (size_t)D, s);
    if (ddt_bias && e == cudaSuccess) e = cudaMemsetAsync(ddt_bias, 0, sizeof(float) * (size_t)D, s);
    if (B > 0 && e == cudaSuccess) e = pass_through(dS0, dS, bytes, s);
    return api_status(e);
  }
  const ScanGradProblem g{{x, delta, z, Bm, Cm, ldx, ld_delta, ldz, ldb, ldc, A, Dskip, dt_bias, lengths, S0, nullptr,
                           nullptr, B, N, D, d_state, softplus != 0, dt, workspace, s},
                          dout, dS, dx, ddelta, dB, dC, dz, dA, dDskip, ddt_bias, dS0};
  if (!workspace || workspace_bytes < scan_grad_workspace(g.p)) return LA_ERR_INVALID_VALUE;
  return api_status(launch_selective_scan_grad(g));
}

la_status la_selective_scan_step(const void *x, long ldx, const void *delta, long ld_delta, const float *A,
                                 const void *Bm, long ldb, const void *Cm, long ldc, const float *Dskip, const void *z,
                                 long ldz, const float *dt_bias, float *S, const int *slots, void *out, int B,
                                 int n_slots, int D, int d_state, int softplus, la_dtype dt, void *stream) {
  la_status st = scan_sizes(B, 1, D, d_state, dt);
  if (st != LA_OK) return st;
  if (n_slots < 0 || (!slots && n_slots < B)) return LA_ERR_INVALID_VALUE;
  if (B == 0) return LA_OK;
  if (missing({x, delta, A, Bm, Cm, out}) || (!S && n_slots > 0)) return LA_ERR_INVALID_VALUE;
  if ((st = all_rows_ok({{ldx, D}, {ld_delta, D}, {ldb, d_state}, {ldc, d_state}, {z ? ldz : ldx, D}}, dt)) != LA_OK) return st;
  if (!aligned({x, delta, A, Bm, Cm, Dskip, z, dt_bias, S, out}, 16) || !aligned({slots}, 4)) return LA_ERR_MISALIGNED;
  if (over({rows(out, B, D, D, dt), floats(S, (long)n_slots * D * d_state)},
           {rows(x, B, ldx, D, dt), rows(delta, B, ld_delta, D, dt), rows(z, B, ldz, D, dt), rows(Bm, B, ldb, d_state, dt),
            rows(Cm, B, ldc, d_state, dt), floats(A, (long)D * d_state), floats(Dskip, D), floats(dt_bias, D), floats(slots, B)}))
    return LA_ERR_INVALID_VALUE;
  if ((st = api_device()) != LA_OK) return st;
  return api_status(launch_selective_step({x, delta, z, Bm, Cm, ldx, ld_delta, ldz, ldb, ldc, A, Dskip, dt_bias, S, slots,
                                           out, B, D, d_state, n_slots, softplus != 0, dt, (cudaStream_t)stream}));
}

size_t la_beam_select_workspace(int G, int W, int k, int V, la_dtype dt) {
  if (beam_sizes(G, W, k, V, dt) != LA_OK || G == 0) return 0;
  return beam_split(G, W, k, V).bytes;
}

la_status la_beam_select(const void *logits, long ld, const float *scores, const unsigned char *finished,
                         float *out_scores, int *parents, int *tokens, int G, int W, int k, int V, int eos, la_dtype dt,
                         void *workspace, size_t workspace_bytes, void *stream) {
  la_status st = beam_sizes(G, W, k, V, dt);
  if (st != LA_OK) return st;
  if (eos < 0 || eos >= V || ld < V) return LA_ERR_INVALID_VALUE;
  if (G == 0) return LA_OK;
  if (missing({logits, scores, out_scores, parents, tokens})) return LA_ERR_INVALID_VALUE;
  if (!aligned({logits}, 16) || !aligned({workspace}, 256) || !aligned({scores, out_scores, parents, tokens}, 4))
    return LA_ERR_MISALIGNED;
  const long beams = (long)G * W, chosen = (long)G * k;
  if (over({floats(out_scores, chosen), floats(parents, chosen), floats(tokens, chosen)},
           {rows(logits, beams, ld, V, dt), floats(scores, beams), {finished, (size_t)beams}}))
    return LA_ERR_INVALID_VALUE;
  if ((st = api_device()) != LA_OK) return st;
  if (!workspace || workspace_bytes < beam_split(G, W, k, V).bytes) return LA_ERR_INVALID_VALUE;
  return api_status(launch_beam_select(
      {logits, ld, scores, finished, out_scores, parents, tokens, G, W, k, V, eos, dt, workspace, (cudaStream_t)stream}));
}

la_status la_beam_reorder(void *const *pools, const size_t *row_bytes, int n_pools, const int *slots, const int *parents,
                          int *new_slots, int G, int W, int n_slots, void *stream) {
  if (G < 0 || W <= 0 || n_slots < 0 || n_pools < 0 || (n_pools > 0 && (!pools || !row_bytes))) return LA_ERR_INVALID_VALUE;
  if (W > 64) return LA_ERR_UNSUPPORTED;
  if (G > (1 << 24)) return LA_ERR_INVALID_VALUE;
  if (G == 0) return LA_OK;
  const Span slots_of = floats(slots, (long)G * W), parents_of = floats(parents, (long)G * W);
  if (missing({slots, parents, new_slots}) || over({floats(new_slots, (long)G * W)}, {slots_of, parents_of}))
    return LA_ERR_INVALID_VALUE;
  if (!aligned({slots, parents, new_slots}, 4)) return LA_ERR_MISALIGNED;
  for (int i = 0; i < n_pools; ++i) {
    if (!pools[i] && row_bytes[i] > 0 && n_slots > 0) return LA_ERR_INVALID_VALUE;
    // blocks of the largest row are counted in 31 bits
    if (row_bytes[i] > (size_t)1 << 40 || (long)G * W * (long)(row_bytes[i] / kReorderPiece + 1) * kMaxPools > 0x7fffffffL)
      return LA_ERR_INVALID_VALUE;
    if (!aligned({pools[i]}, 16) || row_bytes[i] % 16) return LA_ERR_MISALIGNED;
    if (over({{pools[i], row_bytes[i] * n_slots}, floats(new_slots, (long)G * W)}, {slots_of, parents_of}))
      return LA_ERR_INVALID_VALUE;
  }
  la_status st = api_device();
  if (st != LA_OK) return st;
  for (int at = 0; at == 0 || at < n_pools; at += kMaxPools) {
    ReorderProblem p{};
    p.pools = std::min(n_pools - at, kMaxPools);
    for (int i = 0; i < p.pools; ++i) p.pool[i] = pools[at + i], p.row_bytes[i] = (long)row_bytes[at + i];
    p.first = at == 0;
    p.slots = slots, p.parents = parents, p.new_slots = new_slots;
    p.G = G, p.W = W, p.n_slots = n_pools ? n_slots : 0x7fffffff, p.stream = (cudaStream_t)stream;
    if ((st = api_status(launch_beam_reorder(p))) != LA_OK) return st;
  }
  return LA_OK;
}

}  // extern "C"
