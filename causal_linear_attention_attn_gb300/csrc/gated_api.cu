// C ABI of gated linear attention, its gradient and serving step, and of the gated group norm:
// argument validation and dispatch (see linattn.h for the contract of each call).
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>
#include <initializer_list>

#include "internal.h"
#include "linattn.h"

namespace la {
namespace {

bool dim_ok(int d) { return d == 32 || d == 64 || d == 128; }

bool aligned(std::initializer_list<const void *> ptrs, uintptr_t to) {
  for (const void *p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & (to - 1)) return false;
  return true;
}

bool overlap(const void *a, const void *b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && (x < y ? y - x : x - y) < bytes;
}

la_status sizes(int B, int H, long N, int dk, int dv, la_dtype dt) {
  if (B < 0 || H < 0 || N < 0 || dk <= 0 || dv <= 0) return LA_ERR_INVALID_VALUE;
  // every launch indexes chunks of a head in one 31-bit grid dimension
  if ((long)B * H > 0x3ffffffL || (long)B * H * ((N + 31) / 32) > 0x7fffffffL) return LA_ERR_INVALID_VALUE;
  if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_UNSUPPORTED;
  if (!dim_ok(dk) || !dim_ok(dv)) return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

size_t workspace(int B, int H, long N, int dk, int dv, la_dtype dt, bool grad) {
  const long BH = (long)B * H;
  if (gated_tc_supported(dk, dv, dt, grad))
    return grad ? gated_tc_grad_workspace(BH, N, dk) : gated_tc_prefill_workspace(BH, N, dk);
  return gated_simt_workspace(BH, N, dk, dv, grad);
}

la_status gated(const void *q, const void *k, const void *v, const float *g, const int *lengths, void *out, float *S,
                int B, int H, int N, int dk, int dv, la_dtype dt, void *ws, size_t ws_bytes, void *stream,
                bool from_state) {
  la_status st = sizes(B, H, N, dk, dv, dt);
  if (st != LA_OK) return st;
  if ((long)B * H == 0) return LA_OK;
  if (!S || (N > 0 && (!q || !k || !v || !g || !out))) return LA_ERR_INVALID_VALUE;
  if (!aligned({q, k, v, out, S}, 16) || !aligned({ws}, 256) || !aligned({g, lengths}, 4)) return LA_ERR_MISALIGNED;
  GatedProblem p{q, k, v, g, lengths, from_state ? S : nullptr, out, S, B, H, N, dk, dv, dt, ws, (cudaStream_t)stream};
  if (N == 0) {
    if (from_state) return LA_OK;
    if ((st = api_device()) != LA_OK) return st;
    return api_status(cudaMemsetAsync(S, 0, sizeof(float) * (size_t)p.BH() * dk * dv, p.stream));
  }
  if ((st = api_device()) != LA_OK) return st;
  const size_t need = workspace(B, H, N, dk, dv, dt, false);
  if (ws_bytes < need || (need && !ws)) return LA_ERR_INVALID_VALUE;
  return api_status(gated_tc_supported(dk, dv, dt, false) ? launch_gated_tc(p) : launch_gated_simt(p));
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

size_t la_gated_workspace(int B, int H, int N, int d_k, int d_v, la_dtype dt, int backward) {
  if (sizes(B, H, N, d_k, d_v, dt) != LA_OK || (long)B * H == 0 || N == 0) return 0;
  return workspace(B, H, N, d_k, d_v, dt, backward != 0);
}

la_status la_gated(const void *q, const void *k, const void *v, const float *g, const int *lengths, void *out,
                   float *S, int B, int H, int N, int d_k, int d_v, la_dtype dt, void *workspace,
                   size_t workspace_bytes, void *stream) {
  return gated(q, k, v, g, lengths, out, S, B, H, N, d_k, d_v, dt, workspace, workspace_bytes, stream, false);
}

la_status la_gated_with_state(const void *q, const void *k, const void *v, const float *g, const int *lengths,
                              void *out, float *S, int B, int H, int N, int d_k, int d_v, la_dtype dt,
                              void *workspace, size_t workspace_bytes, void *stream) {
  return gated(q, k, v, g, lengths, out, S, B, H, N, d_k, d_v, dt, workspace, workspace_bytes, stream, true);
}

la_status la_gated_backward(const void *q, const void *k, const void *v, const float *g, const int *lengths,
                            const void *dout, const float *S0, const float *dS, void *dq, void *dk, void *dv,
                            float *dg, float *dS0, int B, int H, int N, int d_k, int d_v, la_dtype dt,
                            void *workspace, size_t workspace_bytes, void *stream) {
  la_status st = sizes(B, H, N, d_k, d_v, dt);
  if (st != LA_OK) return st;
  if ((long)B * H == 0) return LA_OK;
  if (N > 0 && (!q || !k || !v || !g || !dout || !dq || !dk || !dv || !dg)) return LA_ERR_INVALID_VALUE;
  if (!aligned({q, k, v, dout, S0, dS, dq, dk, dv, dS0}, 16) || !aligned({workspace}, 256) || !aligned({g, dg, lengths}, 4))
    return LA_ERR_MISALIGNED;
  const size_t bytes = sizeof(float) * (size_t)B * H * d_k * d_v;
  // the state and its gradient are walked in opposite directions, neither waits for the other
  if ((N > 0 && overlap(S0, dS0, bytes)) || (dS != dS0 && overlap(dS, dS0, bytes))) return LA_ERR_INVALID_VALUE;
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = api_device()) != LA_OK) return st;
  if (N == 0) {  // the state passes through
    if (!dS0 || dS0 == dS) return LA_OK;
    return api_status(dS ? cudaMemcpyAsync(dS0, dS, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(dS0, 0, bytes, s));
  }
  if (!workspace || workspace_bytes < la::workspace(B, H, N, d_k, d_v, dt, true)) return LA_ERR_INVALID_VALUE;
  GatedGradProblem b{{q, k, v, g, lengths, S0, nullptr, nullptr, B, H, N, d_k, d_v, dt, workspace, s},
                     dout, dS, dq, dk, dv, dg, dS0};
  return api_status(gated_tc_supported(d_k, d_v, dt, true) ? launch_gated_grad_tc(b) : launch_gated_grad_simt(b));
}

la_status la_gated_decode_step(const void *q, const void *k, const void *v, const float *g, float *S, const int *slots,
                               void *out, int B, int H, int n_slots, int d_k, int d_v, la_dtype dt, void *stream) {
  la_status st = sizes(B, H, 1, d_k, d_v, dt);
  if (st != LA_OK) return st;
  if (n_slots < 0 || (!slots && n_slots < B)) return LA_ERR_INVALID_VALUE;
  if ((long)B * H == 0) return LA_OK;
  if (!q || !k || !v || !g || !out || (!S && n_slots > 0)) return LA_ERR_INVALID_VALUE;
  if (!aligned({q, k, v, out, S}, 16) || !aligned({g, slots}, 4)) return LA_ERR_MISALIGNED;
  if ((st = api_device()) != LA_OK) return st;
  return api_status(launch_gated_decode({q, k, v, g, S, slots, out, B, H, n_slots, d_k, d_v, dt, (cudaStream_t)stream}));
}

static la_status norm_sizes(int B, int H, long N, int d, float eps, la_dtype dt) {
  if (B < 0 || H < 0 || N < 0 || d <= 0 || !std::isfinite(eps) || eps < 0.f) return LA_ERR_INVALID_VALUE;
  if ((long)B * N > 0x7fffffffL || (long)H * d > 0x3fffffffL || H > 65535 * 16) return LA_ERR_INVALID_VALUE;
  if ((dt != LA_F32 && dt != LA_BF16) || !dim_ok(d)) return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

la_status la_group_norm(const void *x, const void *gate, const float *weight, const float *bias, void *y, int B,
                        int H, int N, int d, float eps, la_dtype dt, void *stream) {
  la_status st = norm_sizes(B, H, N, d, eps, dt);
  if (st != LA_OK) return st;
  if ((long)B * H * N == 0) return LA_OK;
  if (!x || !y) return LA_ERR_INVALID_VALUE;
  if (!aligned({x, gate, weight, bias, y}, 16)) return LA_ERR_MISALIGNED;
  if ((st = api_device()) != LA_OK) return st;
  return api_status(launch_group_norm({x, gate, weight, bias, y, B, H, N, d, eps, dt, (cudaStream_t)stream}));
}

size_t la_group_norm_workspace(int B, int H, int N, int d) {
  if (norm_sizes(B, H, N, d, 0.f, LA_F32) != LA_OK || (long)B * H * N == 0) return 0;
  return norm_grad_workspace(B, H, N, d);
}

la_status la_group_norm_backward(const void *x, const void *dy, const void *gate, const float *weight,
                                 const float *bias, void *dx, void *dgate, float *dweight, float *dbias, int B,
                                 int H, int N, int d, float eps, la_dtype dt, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  la_status st = norm_sizes(B, H, N, d, eps, dt);
  if (st != LA_OK) return st;
  if (H == 0 || (long)B * N == 0) {  // no tokens: the column sums are empty
    if (H == 0 || (!dweight && !dbias)) return LA_OK;
    if ((st = api_device()) != LA_OK) return st;
    cudaError_t e = cudaSuccess;
    if (dweight) e = cudaMemsetAsync(dweight, 0, sizeof(float) * (size_t)H * d, (cudaStream_t)stream);
    if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, sizeof(float) * (size_t)H * d, (cudaStream_t)stream);
    return api_status(e);
  }
  if (!x || !dy || !dx || (gate != nullptr) != (dgate != nullptr)) return LA_ERR_INVALID_VALUE;
  if (!aligned({x, dy, gate, weight, bias, dx, dgate, workspace}, 16) || !aligned({dweight, dbias}, 4))
    return LA_ERR_MISALIGNED;
  if ((st = api_device()) != LA_OK) return st;
  const bool sums = dweight || dbias;
  if (sums && (!workspace || workspace_bytes < norm_grad_workspace(B, H, N, d))) return LA_ERR_INVALID_VALUE;
  return api_status(launch_group_norm_grad({{x, gate, weight, bias, nullptr, B, H, N, d, eps, dt, (cudaStream_t)stream},
                                            dy, dx, dgate, dweight, dbias, sums ? (float *)workspace : nullptr}));
}

}  // extern "C"
