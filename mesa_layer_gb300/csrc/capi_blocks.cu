// capi_blocks.cu -- the extern "C" entry points of the gated delta rule and the block norm:
// argument validation, workspace carve-up and dispatch.  No allocation, no synchronisation.
#include <math.h>

#include "../../include/mesa.h"
#include "block_norm.h"
#include "gated_delta.h"
#include "launch.h"

namespace {

constexpr size_t kMaxUnits = 65535;  // (batch, head) units index a grid dimension
constexpr size_t kStatusBytes = 256;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }
template <typename... P>
bool all_aligned16(const P *...p) {
  return (... && aligned16(p));
}
// The tensor-core path of the delta rule: bf16 with dk = dv = 128.
bool rule_tc(int dtype, int dk, int dv) { return dtype == MESA_BF16 && dk == 128 && dv == 128; }
// The forward's: a few tokens are quicker as a recurrence (us on the tensor cores, as a recurrence: 16 units,
// 1 token 14.4, 6.2; 16 tokens 14.5, 8.3; 64 tokens 14.9, 18.7; 128 units, 16 tokens 16.4, 15.7; 32 tokens 16.4, 25.8).  The
// backward's recurrence is slower at any length (16 units, 1 token 30.8, 81.5).
bool rule_tc_forward(int dtype, int dk, int dv, int T) { return T > 16 && rule_tc(dtype, dk, dv); }
bool dtype_ok(int dtype) { return dtype == MESA_F32 || dtype == MESA_BF16; }

// The checks the two sequence forms share.
int check_sizes(int B, int H, int Hk, int T, int dk, int dv, int dtype, float scale) {
  if (B < 0 || H < 0 || Hk < 0 || T < 0 || !dtype_ok(dtype) || !isfinite(scale)) return MESA_ERR_INVALID_ARG;
  if (H > 0 && (Hk == 0 || H % Hk != 0)) return MESA_ERR_INVALID_ARG;
  if (!dim_ok(dk) || !dim_ok(dv)) return MESA_ERR_UNSUPPORTED;
  if ((size_t)B * H > kMaxUnits) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

// Backward workspace of the CUDA-core path: [status | S | dS | e | du | per-head dq, dk | segments].
constexpr int kBwdParts = 7;
size_t backward_parts(int B, int H, int Hk, int T, int dk, int dv, size_t *off) {
  const size_t U = (size_t)B * H, NC = ((size_t)T + mesa::kRuleChunk - 1) / mesa::kRuleChunk;
  const size_t st = U * NC * dv * dk * sizeof(float), rows = U * T * dv * sizeof(float);
  const size_t part = Hk != H ? U * T * dk * sizeof(float) : 0;
  const size_t sizes[kBwdParts] = {st, st, rows, rows, part, part, mesa::rule_scan_workspace(B * H, T, dk, dv, true)};
  size_t at = kStatusBytes;
  for (int i = 0; i < kBwdParts; i++) {
    off[i] = at;
    at += align256(sizes[i]);
  }
  return at;
}

// Backward workspace of the tensor-core path: [status | records | S | A | u | du | their scales (4) |
// per-head dq, dk].
constexpr int kTcParts = 10;
size_t backward_tc_parts(int B, int H, int Hk, int T, size_t *off) {
  const size_t U = (size_t)B * H, n = U * (((size_t)T + 63) / 64);
  const size_t part = Hk != H ? U * T * 128 * sizeof(float) : 0;
  const size_t sizes[kTcParts + 1] = {mesa::rule_tc_workspace(B * H, T, true), n * 32768, n * 32768, n * 16384, n * 16384,
                                      n * 4, n * 4, n * 4, n * 4, part, part};
  size_t at = kStatusBytes;
  for (int i = 0; i <= kTcParts; i++) {
    off[i] = at;
    at += align256(sizes[i]);
  }
  return at;
}

}  // namespace

extern "C" {

size_t mesa_delta_workspace_size(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  if (check_sizes(B, H, Hk, T, dk, dv, dtype, 1.0f) != MESA_OK) return 0;
  return kStatusBytes + (rule_tc_forward(dtype, dk, dv, T) ? mesa::rule_tc_workspace(B * H, T, false)
                                                            : mesa::rule_scan_workspace(B * H, T, dk, dv, false));
}

int mesa_delta_forward_chunked(int B, int H, int Hk, int T, int dk, int dv, int dtype, const void *q,
                               const void *k, const void *v, const float *gamma, const float *beta,
                               float scale, void *out, const float *S0, float *S_final,
                               void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  const int bad = check_sizes(B, H, Hk, T, dk, dv, dtype, scale);
  if (bad != MESA_OK) return bad;
  const size_t U = (size_t)B * H;
  if (U == 0) return MESA_OK;
  if (!all_aligned16(q, k, v, out, S0, S_final)) return MESA_ERR_INVALID_ARG;
  if (T == 0) {  // nothing to compute; the final state is the initial state
    if (!S_final || S_final == S0) return MESA_OK;
    const size_t bytes = U * dv * dk * sizeof(float);
    const cudaError_t e = S0 ? cudaMemcpyAsync(S_final, S0, bytes, cudaMemcpyDeviceToDevice, stream)
                             : cudaMemsetAsync(S_final, 0, bytes, stream);
    return e == cudaSuccess ? MESA_OK : MESA_ERR_CUDA;
  }
  if (!q || !k || !v || !gamma || !beta || !out) return MESA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < mesa_delta_workspace_size(B, H, Hk, T, dk, dv, dtype) ||
      ((uintptr_t)workspace & 255))
    return MESA_ERR_WORKSPACE;
  mesa::RuleArgs a{B, H, Hk, T, dk, dv, dtype, q, k, v, gamma, beta, scale};
  a.out = out;
  a.S0 = S0;
  a.S_final = S_final;
  a.status = (unsigned *)workspace;
  a.wait_limit = mesa::wait_limit();
  if (cudaMemsetAsync(a.status, 0, sizeof(unsigned), stream) != cudaSuccess) return MESA_ERR_CUDA;
  char *rest = (char *)workspace + kStatusBytes;
  const int rc = rule_tc_forward(dtype, dk, dv, T)
                     ? mesa::launch_rule_forward_tc(a, rest, stream)
                     : mesa::launch_rule_forward(a, mesa::rule_scan_parts(B * H, T, dk, dv, false, rest), stream);
  return rc == 0 ? MESA_OK : MESA_ERR_CUDA;
}

size_t mesa_delta_backward_workspace_size(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  dtype &= ~MESA_GATE_GRADS_F32;  // (the same workspace)
  if (check_sizes(B, H, Hk, T, dk, dv, dtype, 1.0f) != MESA_OK) return 0;
  size_t off[kTcParts + 1];
  return rule_tc(dtype, dk, dv) ? backward_tc_parts(B, H, Hk, T, off) : backward_parts(B, H, Hk, T, dk, dv, off);
}

int mesa_delta_backward_chunked(int B, int H, int Hk, int T, int dk, int dv, int dtype, const void *q,
                                const void *k, const void *v, const float *gamma, const float *beta,
                                float scale, const void *dout, const float *S0, const float *dS_final,
                                void *dq, void *dk_out, void *dv_out, void *dgamma, void *dbeta,
                                float *dS0, void *workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
  const bool gates_f32 = (dtype & MESA_GATE_GRADS_F32) != 0;
  dtype &= ~MESA_GATE_GRADS_F32;
  const int bad = check_sizes(B, H, Hk, T, dk, dv, dtype, scale);
  if (bad != MESA_OK) return bad;
  const size_t U = (size_t)B * H;
  if (U == 0) return MESA_OK;
  if (!all_aligned16(q, k, v, dout, S0, dS_final, dq, dk_out, dv_out, dS0)) return MESA_ERR_INVALID_ARG;
  if (T == 0) {  // no token: the state's gradient passes through
    if (!dS0 || dS0 == dS_final) return MESA_OK;
    const size_t bytes = U * dv * dk * sizeof(float);
    const cudaError_t e = dS_final ? cudaMemcpyAsync(dS0, dS_final, bytes, cudaMemcpyDeviceToDevice, stream)
                                   : cudaMemsetAsync(dS0, 0, bytes, stream);
    return e == cudaSuccess ? MESA_OK : MESA_ERR_CUDA;
  }
  if (!q || !k || !v || !gamma || !beta || !dout || !dq || !dk_out || !dv_out || !dgamma || !dbeta)
    return MESA_ERR_INVALID_ARG;
  size_t off[kTcParts + 1];
  const bool tc = rule_tc(dtype, dk, dv);
  const size_t need = tc ? backward_tc_parts(B, H, Hk, T, off) : backward_parts(B, H, Hk, T, dk, dv, off);
  if (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255)) return MESA_ERR_WORKSPACE;
  char *w = (char *)workspace;
  mesa::RuleArgs a{B, H, Hk, T, dk, dv, dtype, q, k, v, gamma, beta, scale};
  a.S0 = S0;
  a.dout = dout;
  a.dS_final = dS_final;
  a.dq = dq;
  a.dk_out = dk_out;
  a.dv_out = dv_out;
  a.gates_f32 = gates_f32 || dtype == MESA_F32;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.dS0 = dS0;
  a.status = (unsigned *)workspace;
  a.wait_limit = mesa::wait_limit();
  if (cudaMemsetAsync(a.status, 0, sizeof(unsigned), stream) != cudaSuccess) return MESA_ERR_CUDA;
  if (tc) {
    auto f = [&](int i) { return (float *)(w + off[i]); };
    auto b8 = [&](int i) { return (uint8_t *)(w + off[i]); };
    const mesa::RuleOperands so{b8(1), b8(3), f(5), f(6)}, ao{b8(2), b8(4), f(7), f(8)};
    const mesa::RuleSegments sg = mesa::rule_tc_segments(a.units(), T, true, b8(0));
    const bool ok = mesa::launch_rule_prep(a, b8(0), sg, false, stream) == 0 &&
                    mesa::launch_rule_adjoint_tails(a, b8(0), sg, stream) == 0 &&
                    mesa::launch_rule_states_tc(a, b8(0), sg, so, stream) == 0 &&
                    mesa::launch_rule_adjoint_tc(a, b8(0), sg, ao, stream) == 0 &&
                    mesa::launch_rule_grads_tc(a, b8(0), so, ao, Hk != H ? f(9) : nullptr, Hk != H ? f(10) : nullptr,
                                               stream) == 0;
    return ok ? MESA_OK : MESA_ERR_CUDA;
  }
  mesa::RuleBwdWorkspace ws{(float *)(w + off[0]), (float *)(w + off[1]), (float *)(w + off[2]),
                            (float *)(w + off[3]), Hk != H ? (float *)(w + off[4]) : nullptr,
                            Hk != H ? (float *)(w + off[5]) : nullptr};
  const mesa::RuleScanSegments sg = mesa::rule_scan_parts(B * H, T, dk, dv, true, w + off[6]);
  return mesa::launch_rule_backward(a, ws, sg, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

int mesa_delta_step(int N, int H, int Hk, int dk, int dv, int dtype, float *S_state, const void *q,
                    const void *k, const void *v, const float *gamma, const float *beta, float scale,
                    void *out, cudaStream_t stream) {
  if (N < 0 || H < 0 || Hk < 0 || !dtype_ok(dtype) || !isfinite(scale)) return MESA_ERR_INVALID_ARG;
  if (H > 0 && (Hk == 0 || H % Hk != 0)) return MESA_ERR_INVALID_ARG;
  if (!dim_ok(dk) || !dim_ok(dv)) return MESA_ERR_UNSUPPORTED;
  if ((size_t)N * H == 0) return MESA_OK;
  if ((size_t)N * H > 0x7fffffff) return MESA_ERR_UNSUPPORTED;
  if (!S_state || !q || !k || !v || !gamma || !beta || !out) return MESA_ERR_INVALID_ARG;
  if (!all_aligned16(S_state, q, k)) return MESA_ERR_INVALID_ARG;
  mesa::RuleStepArgs a{N, H, Hk, dk, dv, dtype, S_state, q, k, v, gamma, beta, scale, out, mesa::decode_status_word()};
  if (!a.status) return MESA_ERR_CUDA;
  return mesa::launch_rule_step(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

int mesa_block_norm(int N, int D, int dtype, const void *x, const void *y, const void *gate,
                    const float *w_post, const float *res_scale, const float *w_pre, float eps,
                    void *x_out, void *h_out, cudaStream_t stream) {
  if (N < 0 || D < 1 || !dtype_ok(dtype) || !(eps >= 0.0f) || !isfinite(eps)) return MESA_ERR_INVALID_ARG;
  if (D > mesa::kNormMaxD) return MESA_ERR_UNSUPPORTED;
  if (N == 0) return MESA_OK;
  if (!y || (!x_out && !w_pre) || (w_pre && !h_out)) return MESA_ERR_INVALID_ARG;
  mesa::NormArgs a{N, D, dtype, x, y, gate, w_post, res_scale, w_pre, eps};
  a.x_out = x_out;
  a.h_out = w_pre ? h_out : nullptr;
  return mesa::launch_block_norm(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

size_t mesa_block_norm_backward_workspace_size(int N, int D) {
  if (N < 0 || D < 1 || D > mesa::kNormMaxD) return 0;
  return align256((size_t)mesa::norm_bwd_ctas(N, D) * 3 * D * sizeof(float));
}

int mesa_block_norm_backward(int N, int D, int dtype, const void *x, const void *y, const void *gate,
                             const float *w_post, const float *res_scale, const float *w_pre,
                             float eps, const void *dx_out, const void *dh, void *dx, void *dy,
                             void *dgate, float *dw_post, float *dres_scale, float *dw_pre,
                             void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (N < 0 || D < 1 || !dtype_ok(dtype) || !(eps >= 0.0f) || !isfinite(eps)) return MESA_ERR_INVALID_ARG;
  if (D > mesa::kNormMaxD) return MESA_ERR_UNSUPPORTED;
  if ((dw_post && !w_post) || (dres_scale && !res_scale) || (dw_pre && !w_pre) || (dgate && !gate))
    return MESA_ERR_INVALID_ARG;  // a gradient of something the forward did not have
  const bool sums = dw_post || dres_scale || dw_pre;
  if (N == 0) {  // empty sums
    for (float *p : {dw_post, dres_scale, dw_pre})
      if (p && cudaMemsetAsync(p, 0, sizeof(float) * D, stream) != cudaSuccess) return MESA_ERR_CUDA;
    return MESA_OK;
  }
  if (!y || !dy) return MESA_ERR_INVALID_ARG;
  if (sums && (!workspace || workspace_bytes < mesa_block_norm_backward_workspace_size(N, D) ||
               ((uintptr_t)workspace & 255)))
    return MESA_ERR_WORKSPACE;
  mesa::NormArgs a{N, D, dtype, x, y, gate, w_post, res_scale, w_pre, eps};
  a.dx_out = dx_out;
  a.dh = w_pre ? dh : nullptr;
  a.dx = dx;
  a.dy = dy;
  a.dgate = dgate;
  a.dw_post = dw_post;
  a.dres_scale = dres_scale;
  a.dw_pre = dw_pre;
  a.partial = sums ? (float *)workspace : nullptr;
  return mesa::launch_block_norm_backward(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

}  // extern "C"
