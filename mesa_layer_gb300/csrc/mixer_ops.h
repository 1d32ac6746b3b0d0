// mixer_ops.h -- argument bundles and launchers of the causal convolution and of the norm and rotation of queries
// and keys (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mesa {

constexpr int kConvMaxW = 8;
struct ConvArgs {
  int B, H, T, d, W, dtype, silu;
  const void *x;           // [B, H, T, d] (step: [B, H, d])
  const float *w, *bias;   // [H, d, W], [H, d] or nullptr
  const uint8_t *starts;   // [B, T] or nullptr
  const float *state0;     // [B, H, W - 1, d] or nullptr
  float *state;            // the window after the last token, or nullptr (step: in place)
  void *out = nullptr;
  const void *dout = nullptr;
  void *dx = nullptr;
  float *dw = nullptr, *dbias = nullptr;
  float *partial = nullptr;  // [parts][H, d, W + 1]
};
int conv_bwd_parts(int B, int H, int T, int d, int W);  // CTAs that share a head's channels in the backward
int launch_causal_conv(const ConvArgs &a, cudaStream_t st);
int launch_causal_conv_step(const ConvArgs &a, cudaStream_t st);
int launch_causal_conv_backward(const ConvArgs &a, cudaStream_t st);

struct RotaryArgs {
  int B, H, Hk, T, d, R, dtype, interleaved, norm;
  const void *q, *k;            // [B, H, T, d], [B, Hk, T, d] (Hk = 0: no k)
  const float *wq, *wk;         // [d] or nullptr
  const float *inv_freq;        // [R / 2]
  const int32_t *positions;     // [B, T] or nullptr: offset + t
  int offset;
  float rot_scale, eps;
  void *q_out, *k_out;          // backward: dq, dk
  const void *dq_out = nullptr, *dk_out = nullptr;
  float *dwq = nullptr, *dwk = nullptr;
  float *partial = nullptr;     // [parts][2][d]
};
int rotary_bwd_parts(int B, int T, int d);  // CTAs of the backward at most
int launch_qk_norm_rotary(const RotaryArgs &a, cudaStream_t st);
int launch_qk_norm_rotary_backward(const RotaryArgs &a, cudaStream_t st);

}  // namespace mesa
