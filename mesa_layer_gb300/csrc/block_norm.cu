// block_norm.cu -- the norms around a block, with its output gate and residual scale, in one
// pass.  Per row of D channels (each part optional):
//     z = y rsqrt(mean(y^2) + eps) w_post            (the block's output, normalised)
//     x' = x + res_scale silu(gate) z                (gated and scaled into the residual stream)
//     h = x' rsqrt(mean(x'^2) + eps) w_pre           (the next block's input)
// Arithmetic and both means are fp32; h is taken from x' before its rounding to dtype.
//
// Bound by memory: x, y and gate are read once and x' and h written once; the row stays in
// registers (eight channels a thread) across both means, the weights across a CTA's rows.
#include <initializer_list>

#include "block_norm.cuh"
#include "launch.h"

namespace mesa {

namespace {

template <typename T, int VEC, int G>
__global__ void __launch_bounds__(G < 128 ? 128 : G) mesa_block_norm_kernel(NormArgs a) {
  using namespace norm;
  constexpr int RPC = G < 128 ? 128 / G : 1;
  __shared__ float red[2][1][32];
  const int lane = threadIdx.x % G, sub = threadIdx.x / G, D = a.D;
  const float inv_d = 1.0f / (float)D;
  float wp[EPT], rs[EPT], wn[EPT];
  load_weights<VEC, G>(a.w_post, lane, D, 1.0f, wp);
  load_weights<VEC, G>(a.res_scale, lane, D, 1.0f, rs);
  load_weights<VEC, G>(a.w_pre, lane, D, 0.0f, wn);
  const T *x = (const T *)a.x, *y = (const T *)a.y, *gate = (const T *)a.gate;
  int buf = 0;
  for (size_t base = (size_t)blockIdx.x * RPC; base < (size_t)a.N; base += (size_t)gridDim.x * RPC) {
    const size_t row = base + sub, at = row * D;
    const bool in = row < (size_t)a.N;
    float yv[EPT], gv[EPT], xv[EPT];
    load_row<VEC, G>(y + at, lane, D, in, yv);
    load_row<VEC, G>(gate + at, lane, D, in && gate, gv);
    load_row<VEC, G>(x + at, lane, D, in && x, xv);
    float r = 1.0f;
    if (a.w_post) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < EPT; i++) ss[0] = fmaf(yv[i], yv[i], ss[0]);
      row_sums<G>(ss, red, buf);
      r = rsqrtf(fmaf(ss[0], inv_d, a.eps));
    }
#pragma unroll
    for (int i = 0; i < EPT; i++) {
      float z = yv[i] * r * wp[i];
      if (gate) z *= gv[i] / (1.0f + expf(-gv[i]));
      xv[i] = fmaf(rs[i], z, xv[i]);
    }
    if (a.x_out) store_row<VEC, G>((T *)a.x_out + at, lane, D, in, xv);
    if (a.w_pre) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < EPT; i++) ss[0] = fmaf(xv[i], xv[i], ss[0]);
      row_sums<G>(ss, red, buf);
      const float rn = rsqrtf(fmaf(ss[0], inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < EPT; i++) xv[i] *= rn * wn[i];
      store_row<VEC, G>((T *)a.h_out + at, lane, D, in, xv);
    }
  }
}

template <typename T, int VEC, int G>
struct Forward {
  static int run(const NormArgs &a, cudaStream_t st) {
    constexpr int RPC = G < 128 ? 128 / G : 1;
    const size_t want = ((size_t)a.N + RPC - 1) / RPC;
    int sms = sm_count();
    if (sms <= 0) sms = 152;
    const size_t most = (size_t)sms * (G <= 128 ? 12 : 2048 / G);
    timing_mark_begin(K_NORM, st);
    mesa_block_norm_kernel<T, VEC, G><<<(unsigned)(want < most ? want : most), G < 128 ? 128 : G, 0, st>>>(a);
    timing_mark_end(K_NORM, st);
    return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
  }
};

}  // namespace

int launch_block_norm(const NormArgs &a, cudaStream_t st) {
  return norm::dispatch<Forward>(a, norm::vec_of(a.D, a.dtype, {a.x, a.y, a.gate, a.x_out, a.h_out}), st);
}

}  // namespace mesa
