// block_norm.h -- argument bundle and launchers of the block norm (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mesa {

struct NormArgs {
  int N, D, dtype;
  const void *x, *y, *gate;                       // [N, D]; x and gate may be nullptr
  const float *w_post, *res_scale, *w_pre;        // [D] or nullptr
  float eps;
  void *x_out = nullptr, *h_out = nullptr;        // forward: [N, D] (h_out nullptr without w_pre)
  // backward
  const void *dx_out = nullptr, *dh = nullptr;    // [N, D] (nullptr: zero)
  void *dx = nullptr, *dy = nullptr, *dgate = nullptr;
  float *dw_post = nullptr, *dres_scale = nullptr, *dw_pre = nullptr;
  float *partial = nullptr;                       // [ctas][3][D] column sums
};

constexpr int kNormMaxD = 8192;
// Threads of a row: 8 channels a thread, a power of two from 8 to 1024.
inline int norm_group(int D) {
  int g = 8;
  while (8 * g < D) g *= 2;
  return g;
}
// Rows of a CTA at a time (CTAs of at least 128 threads).
inline int norm_rows(int D) {
  const int g = norm_group(D);
  return g < 128 ? 128 / g : 1;
}
// CTAs of the backward kernel: its column sums are kept per CTA.  A fixed count (as many as are resident
// on a GB300's 152 SMs), so that the workspace size needs no device.
inline int norm_bwd_ctas(int N, int D) {
  const int g = norm_group(D), most = 152 * (g <= 128 ? 4 : g == 256 ? 2 : 1);
  const size_t want = ((size_t)N + norm_rows(D) - 1) / norm_rows(D);
  return want < (size_t)most ? (int)want : most;
}

int launch_block_norm(const NormArgs &a, cudaStream_t st);
int launch_block_norm_backward(const NormArgs &a, cudaStream_t st);

}  // namespace mesa
