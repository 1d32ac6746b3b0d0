// capi_mixer.cu -- the extern "C" entry points of the selective scan, the causal convolution and the norm and rotation of
// queries and keys: argument validation, workspace carve-up and dispatch.  No allocation, no synchronisation.
#include <math.h>

#include "../../include/mesa.h"
#include "launch.h"
#include "mixer_ops.h"
#include "ssm.h"

namespace {

constexpr size_t kMaxUnits = 65535;  // (batch, head) units index a grid dimension
constexpr size_t kStatusBytes = 256;

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool dtype_ok(int dtype) { return dtype == MESA_F32 || dtype == MESA_BF16; }
template <typename... P>
bool all_aligned16(const P *...p) {
  return (... && (((uintptr_t)p & 15) == 0));
}
bool workspace_ok(const void *w, size_t bytes, size_t need) { return w && bytes >= need && !((uintptr_t)w & 255); }
bool bad_memset(void *p, size_t bytes, cudaStream_t st) { return p && cudaMemsetAsync(p, 0, bytes, st) != cudaSuccess; }

int check_scan(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  if (B < 0 || H < 0 || Hk < 0 || T < 0 || !dtype_ok(dtype)) return MESA_ERR_INVALID_ARG;
  if (H > 0 && (Hk == 0 || H % Hk != 0)) return MESA_ERR_INVALID_ARG;
  if (!dim_ok(dk) || !dim_ok(dv)) return MESA_ERR_UNSUPPORTED;
  if ((size_t)B * H > kMaxUnits || T > 0x7fffff00) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

// The tensor-core path: bf16, dk = 128 and dv 64 or 128, or both 64.  (us on it, on the CUDA cores, forward / backward:
// 8 x 16 x 4096, both 64: 87, 700 / 300, 1610.)
bool scan_tc(int dtype, int dk, int dv) {
  return dtype == MESA_BF16 && ((dk == 128 && (dv == 64 || dv == 128)) || (dk == 64 && dv == 64));
}

// Workspace of the CUDA-core path: [status | S | decay], and for the backward [R | sums | per-head dq, dk].
size_t scan_parts(int B, int H, int Hk, int T, int dk, int dv, bool backward, mesa::SsmWorkspace *ws, char *base) {
  const size_t U = (size_t)B * H, NC = ((size_t)T + mesa::kSsmChunk - 1) / mesa::kSsmChunk;
  const size_t state = U * NC * dv * dk * sizeof(float);
  size_t at = kStatusBytes;
  auto take = [&](float **p, size_t bytes) {
    if (ws) *p = bytes ? (float *)(base + at) : nullptr;
    at += align256(bytes);
  };
  mesa::SsmWorkspace none;
  mesa::SsmWorkspace &w = ws ? *ws : none;
  take(&w.S, state);
  take(&w.decay, U * NC * sizeof(float));
  if (!backward) return at;
  take(&w.R, state);
  take(&w.sums, 3 * U * NC * sizeof(float));
  const size_t part = Hk != H ? U * T * dk * sizeof(float) : 0;
  take(&w.dqp, part);
  take(&w.dkp, part);
  return at;
}

}  // namespace

extern "C" {

size_t mesa_ssm_workspace_size(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  if (check_scan(B, H, Hk, T, dk, dv, dtype) != MESA_OK) return 0;
  if (scan_tc(dtype, dk, dv)) return kStatusBytes + mesa::ssm_tc_workspace(B * H, T, dv);
  return scan_parts(B, H, Hk, T, dk, dv, false, nullptr, nullptr);
}

int mesa_ssm_forward_chunked(int B, int H, int Hk, int T, int dk, int dv, int dtype, const void *q, const void *k,
                             const void *v, const float *dt, const float *A, const float *dt_bias,
                             const float *skip, const uint8_t *starts, void *out, const float *S0,
                             float *S_final, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  const int bad = check_scan(B, H, Hk, T, dk, dv, dtype);
  if (bad != MESA_OK) return bad;
  const size_t U = (size_t)B * H, state = U * dv * dk * sizeof(float);
  if (U == 0) return MESA_OK;
  if (!all_aligned16(q, k, v, out, S0, S_final)) return MESA_ERR_INVALID_ARG;
  if (T == 0) {  // nothing to compute; the final state is the initial state
    if (!S_final || S_final == S0) return MESA_OK;
    if (!S0) return bad_memset(S_final, state, stream) ? MESA_ERR_CUDA : MESA_OK;
    return cudaMemcpyAsync(S_final, S0, state, cudaMemcpyDeviceToDevice, stream) == cudaSuccess ? MESA_OK : MESA_ERR_CUDA;
  }
  if (!q || !k || !v || !dt || !A || !out) return MESA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, mesa_ssm_workspace_size(B, H, Hk, T, dk, dv, dtype))) return MESA_ERR_WORKSPACE;
  mesa::SsmArgs a{B, H, Hk, T, dk, dv, dtype, q, k, v, dt, A, dt_bias, skip, starts};
  a.out = out;
  a.S0 = S0;
  a.S_final = S_final;
  a.status = (unsigned *)workspace;
  a.wait_limit = mesa::wait_limit();
  if (scan_tc(dtype, dk, dv))
    return mesa::launch_ssm_forward_tc(a, (char *)workspace + kStatusBytes, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
  mesa::SsmWorkspace ws;
  scan_parts(B, H, Hk, T, dk, dv, false, &ws, (char *)workspace);
  return mesa::launch_ssm_forward(a, ws, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

size_t mesa_ssm_backward_workspace_size(int B, int H, int Hk, int T, int dk, int dv, int dtype) {
  dtype &= ~MESA_GATE_GRADS_F32;  // (the same workspace)
  if (check_scan(B, H, Hk, T, dk, dv, dtype) != MESA_OK) return 0;
  if (scan_tc(dtype, dk, dv)) return kStatusBytes + mesa::ssm_tc_backward_workspace(B, H, Hk, T, dk, dv);
  return scan_parts(B, H, Hk, T, dk, dv, true, nullptr, nullptr);
}

int mesa_ssm_backward_chunked(int B, int H, int Hk, int T, int dk, int dv, int dtype, const void *q, const void *k,
                              const void *v, const float *dt, const float *A, const float *dt_bias,
                              const float *skip, const uint8_t *starts, const void *dout, const float *S0,
                              const float *dS_final, void *dq, void *dk_out, void *dv_out, void *ddt, void *dA,
                              void *ddt_bias, void *dskip, float *dS0, void *workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
  const bool gates_f32 = (dtype & MESA_GATE_GRADS_F32) != 0;
  dtype &= ~MESA_GATE_GRADS_F32;
  const int bad = check_scan(B, H, Hk, T, dk, dv, dtype);
  if (bad != MESA_OK) return bad;
  if ((ddt_bias && !dt_bias) || (dskip && !skip)) return MESA_ERR_INVALID_ARG;  // what the forward did not have
  const size_t U = (size_t)B * H, state = U * dv * dk * sizeof(float);
  const size_t param = (size_t)H * (gates_f32 || dtype == MESA_F32 ? 4 : 2);
  if (!all_aligned16(q, k, v, dout, S0, dS_final, dq, dk_out, dv_out, dS0)) return MESA_ERR_INVALID_ARG;
  if (U == 0 || T == 0) {  // empty sums (of a key head without value heads, too); the state's gradient passes through
    const size_t qk = H == 0 ? (size_t)B * Hk * T * dk * (dtype == MESA_F32 ? 4 : 2) : 0;
    if (qk > 0 && (!dq || !dk_out)) return MESA_ERR_INVALID_ARG;
    if (qk > 0 && (bad_memset(dq, qk, stream) || bad_memset(dk_out, qk, stream))) return MESA_ERR_CUDA;
    for (void *p : {dA, ddt_bias, dskip})
      if (H > 0 && bad_memset(p, param, stream)) return MESA_ERR_CUDA;
    if (U == 0 || !dS0 || dS0 == dS_final) return MESA_OK;
    if (!dS_final) return bad_memset(dS0, state, stream) ? MESA_ERR_CUDA : MESA_OK;
    return cudaMemcpyAsync(dS0, dS_final, state, cudaMemcpyDeviceToDevice, stream) == cudaSuccess ? MESA_OK : MESA_ERR_CUDA;
  }
  if (!q || !k || !v || !dt || !A || !dout || !dq || !dk_out || !dv_out || !ddt) return MESA_ERR_INVALID_ARG;
  if (!workspace_ok(workspace, workspace_bytes, mesa_ssm_backward_workspace_size(B, H, Hk, T, dk, dv, dtype)))
    return MESA_ERR_WORKSPACE;
  mesa::SsmArgs a{B, H, Hk, T, dk, dv, dtype, q, k, v, dt, A, dt_bias, skip, starts};
  a.S0 = S0;
  a.dout = dout;
  a.dS_final = dS_final;
  a.dq = dq;
  a.dk_out = dk_out;
  a.dv_out = dv_out;
  a.ddt = ddt;
  a.dA = dA;
  a.dbias = ddt_bias;
  a.dskip = dskip;
  a.gates_f32 = gates_f32 || dtype == MESA_F32;
  a.dS0 = dS0;
  a.status = (unsigned *)workspace;
  a.wait_limit = mesa::wait_limit();
  if (scan_tc(dtype, dk, dv))
    return mesa::launch_ssm_backward_tc(a, (char *)workspace + kStatusBytes, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
  mesa::SsmWorkspace ws;
  scan_parts(B, H, Hk, T, dk, dv, true, &ws, (char *)workspace);
  return mesa::launch_ssm_backward(a, ws, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

int mesa_ssm_step(int N, int H, int Hk, int dk, int dv, int dtype, float *S_state, const void *q, const void *k,
                  const void *v, const float *dt, const float *A, const float *dt_bias, const float *skip,
                  void *out, cudaStream_t stream) {
  if (N < 0 || H < 0 || Hk < 0 || !dtype_ok(dtype)) return MESA_ERR_INVALID_ARG;
  if (H > 0 && (Hk == 0 || H % Hk != 0)) return MESA_ERR_INVALID_ARG;
  if (!dim_ok(dk) || !dim_ok(dv)) return MESA_ERR_UNSUPPORTED;
  if ((size_t)N * H == 0) return MESA_OK;
  if ((size_t)N * H > 0x7fffffff) return MESA_ERR_UNSUPPORTED;
  if (!S_state || !q || !k || !v || !dt || !A || !out) return MESA_ERR_INVALID_ARG;
  if (!all_aligned16(S_state, q, k)) return MESA_ERR_INVALID_ARG;
  mesa::SsmStepArgs a{N, H, Hk, dk, dv, dtype, S_state, q, k, v, dt, A, dt_bias, skip, out, mesa::decode_status_word()};
  if (!a.status) return MESA_ERR_CUDA;
  return mesa::launch_ssm_step(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

static int check_conv(int B, int H, int T, int d, int W, int dtype) {
  if (B < 0 || H < 0 || T < 0 || d < 1 || W < 1 || !dtype_ok(dtype)) return MESA_ERR_INVALID_ARG;
  if (d % 8 != 0 || d > 65536 || W > mesa::kConvMaxW || (size_t)B * H > kMaxUnits || T > 0x7fffff00) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

int mesa_causal_conv(int B, int H, int T, int d, int W, int dtype, int silu, const void *x, const float *w,
                     const float *bias, const uint8_t *starts, const float *state0, float *state_final, void *out,
                     cudaStream_t stream) {
  const int bad = check_conv(B, H, T, d, W, dtype);
  if (bad != MESA_OK) return bad;
  const size_t U = (size_t)B * H, state = U * (W - 1) * d * sizeof(float);
  if (U == 0) return MESA_OK;
  if (!all_aligned16(x, out, state0, state_final)) return MESA_ERR_INVALID_ARG;
  if (state0 && state0 == state_final) return MESA_ERR_INVALID_ARG;  // (read while it is written)
  if (T == 0) {  // the window stays where it is
    if (!state_final || W == 1) return MESA_OK;
    if (!state0) return bad_memset(state_final, state, stream) ? MESA_ERR_CUDA : MESA_OK;
    return cudaMemcpyAsync(state_final, state0, state, cudaMemcpyDeviceToDevice, stream) == cudaSuccess ? MESA_OK : MESA_ERR_CUDA;
  }
  if (!x || !w || !out || x == out) return MESA_ERR_INVALID_ARG;
  mesa::ConvArgs a{B, H, T, d, W, dtype, silu != 0, x, w, bias, starts, state0, state_final};
  a.out = out;
  return mesa::launch_causal_conv(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

int mesa_causal_conv_step(int N, int H, int d, int W, int dtype, int silu, const void *x, const float *w,
                          const float *bias, float *conv_state, void *out, cudaStream_t stream) {
  const int bad = check_conv(N, 1, 1, d, W, dtype) == MESA_ERR_INVALID_ARG ? MESA_ERR_INVALID_ARG : check_conv(0, 0, 0, d, W, dtype);
  if (bad != MESA_OK || H < 0) return bad != MESA_OK ? bad : MESA_ERR_INVALID_ARG;
  if ((size_t)N * H == 0) return MESA_OK;
  if ((size_t)N * H > 0x7fffffff / ((size_t)d / 4)) return MESA_ERR_UNSUPPORTED;
  if (!x || !w || !out || (W > 1 && !conv_state) || !all_aligned16(x, out, conv_state)) return MESA_ERR_INVALID_ARG;
  mesa::ConvArgs a{N, H, 1, d, W, dtype, silu != 0, x, w, bias, nullptr, nullptr, conv_state};
  a.out = out;
  return mesa::launch_causal_conv_step(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

size_t mesa_causal_conv_backward_workspace_size(int B, int H, int T, int d, int W) {
  if (check_conv(B, H, T, d, W, MESA_F32) != MESA_OK || (size_t)B * H == 0 || T == 0) return 0;
  return align256((size_t)mesa::conv_bwd_parts(B, H, T, d, W) * H * d * (W + 1) * sizeof(float));
}

int mesa_causal_conv_backward(int B, int H, int T, int d, int W, int dtype, int silu, const void *x, const float *w,
                              const float *bias, const uint8_t *starts, const void *dout, void *dx, float *dw,
                              float *dbias, void *workspace, size_t workspace_bytes, cudaStream_t stream) {
  const int bad = check_conv(B, H, T, d, W, dtype);
  if (bad != MESA_OK) return bad;
  if (dbias && !bias) return MESA_ERR_INVALID_ARG;  // a gradient of something the forward did not have
  if ((size_t)B * H == 0 || T == 0) {  // empty sums
    return bad_memset(dw, (size_t)H * d * W * sizeof(float), stream) || bad_memset(dbias, (size_t)H * d * sizeof(float), stream)
               ? MESA_ERR_CUDA
               : MESA_OK;
  }
  if (!x || !w || !dout || !dx || dx == x || dx == dout || !all_aligned16(x, dout, dx)) return MESA_ERR_INVALID_ARG;
  const bool sums = dw || dbias;
  if (sums && !workspace_ok(workspace, workspace_bytes, mesa_causal_conv_backward_workspace_size(B, H, T, d, W)))
    return MESA_ERR_WORKSPACE;
  mesa::ConvArgs a{B, H, T, d, W, dtype, silu != 0, x, w, bias, starts, nullptr, nullptr};
  a.dout = dout;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.partial = sums ? (float *)workspace : nullptr;
  return mesa::launch_causal_conv_backward(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

static int check_rotary(const mesa::RotaryArgs &a) {
  if (a.B < 0 || a.H < 0 || a.Hk < 0 || a.T < 0 || a.R < 0 || a.R % 2 != 0 || a.R > a.d || !dtype_ok(a.dtype))
    return MESA_ERR_INVALID_ARG;
  if (!(a.eps >= 0.0f) || !isfinite(a.eps) || !isfinite(a.rot_scale)) return MESA_ERR_INVALID_ARG;
  if (!a.norm && (a.wq || a.wk)) return MESA_ERR_INVALID_ARG;
  if (!dim_ok(a.d) || (size_t)a.H + a.Hk > kMaxUnits || (size_t)a.B * a.T > 0x7fffffff) return MESA_ERR_UNSUPPORTED;
  if (!a.positions && ((long long)a.offset + a.T > 0x7fffffff)) return MESA_ERR_UNSUPPORTED;
  return MESA_OK;
}

int mesa_qk_norm_rotary(int B, int H, int Hk, int T, int d, int R, int dtype, int interleaved, int norm, const void *q,
                        const void *k, const float *wq, const float *wk, const float *inv_freq,
                        const int32_t *positions, int offset, float rot_scale, float eps, void *q_out, void *k_out,
                        cudaStream_t stream) {
  const mesa::RotaryArgs a{B, H, Hk, T, d, R, dtype, interleaved != 0, norm != 0, q, k, wq, wk, inv_freq, positions, offset,
                           rot_scale, eps, q_out, k_out};
  const int bad = check_rotary(a);
  if (bad != MESA_OK) return bad;
  if ((size_t)B * T == 0 || H + Hk == 0) return MESA_OK;
  if ((H > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out)) || (R > 0 && !inv_freq)) return MESA_ERR_INVALID_ARG;
  if (!all_aligned16(q, k, q_out, k_out)) return MESA_ERR_INVALID_ARG;
  return mesa::launch_qk_norm_rotary(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

size_t mesa_qk_norm_rotary_backward_workspace_size(int B, int H, int Hk, int T, int d) {
  if (B < 0 || H < 0 || Hk < 0 || T < 0 || !dim_ok(d)) return 0;
  return align256((size_t)mesa::rotary_bwd_parts(B, T, d) * 2 * d * sizeof(float));
}

int mesa_qk_norm_rotary_backward(int B, int H, int Hk, int T, int d, int R, int dtype, int interleaved, int norm,
                                 const void *q, const void *k, const float *wq, const float *wk, const float *inv_freq,
                                 const int32_t *positions, int offset, float rot_scale, float eps, const void *dq_out,
                                 const void *dk_out, void *dq, void *dk, float *dwq, float *dwk, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream) {
  mesa::RotaryArgs a{B, H, Hk, T, d, R, dtype, interleaved != 0, norm != 0, q, k, wq, wk, inv_freq, positions, offset,
                     rot_scale, eps, dq, dk};
  const int bad = check_rotary(a);
  if (bad != MESA_OK) return bad;
  if ((dwq && !wq) || (dwk && !wk)) return MESA_ERR_INVALID_ARG;  // a gradient of something the forward did not have
  if ((size_t)B * T == 0 || H + Hk == 0) {  // empty sums
    return bad_memset(dwq, d * sizeof(float), stream) || bad_memset(dwk, d * sizeof(float), stream) ? MESA_ERR_CUDA : MESA_OK;
  }
  if ((H > 0 && (!dq_out || !dq || (norm && !q))) || (Hk > 0 && (!dk_out || !dk || (norm && !k))) || (R > 0 && !inv_freq))
    return MESA_ERR_INVALID_ARG;
  if (!all_aligned16(q, k, dq_out, dk_out, dq, dk)) return MESA_ERR_INVALID_ARG;
  const bool sums = dwq || dwk;
  if (sums && !workspace_ok(workspace, workspace_bytes, mesa_qk_norm_rotary_backward_workspace_size(B, H, Hk, T, d)))
    return MESA_ERR_WORKSPACE;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.dwq = dwq;
  a.dwk = dwk;
  a.partial = sums ? (float *)workspace : nullptr;
  return mesa::launch_qk_norm_rotary_backward(a, stream) == 0 ? MESA_OK : MESA_ERR_CUDA;
}

}  // extern "C"
