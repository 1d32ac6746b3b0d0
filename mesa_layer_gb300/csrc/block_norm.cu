// block_norm.cu -- the norms around a block, with its output gate and residual scale, in one
// pass.  Per row of D channels (each part optional):
//     z = y rsqrt(mean(y^2) + eps) w_post            (the block's output, normalised)
//     x' = x + res_scale silu(gate) z                (gated and scaled into the residual stream)
//     h = x' rsqrt(mean(x'^2) + eps) w_pre           (the next block's input)
// Arithmetic and both means are fp32; h is taken from x' before its rounding to dtype.
//
// Bound by memory: x, y and gate are read once and x' and h written once; the row stays in
// registers (eight channels a thread) across both means, the weights across a CTA's rows, and the
// next row is on its way while one is worked on: 109 us at 32768 x 2048 bf16 with every part, 6.1 TB/s
// (without that 143 us).
#include <initializer_list>

#include "block_norm.cuh"
#include "launch.h"

namespace mesa {

namespace {

template <typename T, int VEC, int G>
__global__ void __launch_bounds__(G < 128 ? 128 : G, G <= 128 ? 6 : G == 256 ? 3 : 1) mesa_block_norm_kernel(NormArgs a) {
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
  const size_t N = (size_t)a.N, step = (size_t)gridDim.x * RPC;
  Raw<T, VEC> ry, rg, rx;
  auto fetch = [&](size_t row) {
    const bool in = row < N;
    ry.template load<G>(y + row * D, lane, D, in);
    rg.template load<G>(gate + row * D, lane, D, in && gate);
    rx.template load<G>(x + row * D, lane, D, in && x);
  };
  fetch((size_t)blockIdx.x * RPC + sub);
  for (size_t base = (size_t)blockIdx.x * RPC; base < N; base += step) {
    const size_t row = base + sub, at = row * D;
    const bool in = row < N;
    float yv[EPT], gv[EPT], xv[EPT];
    ry.widen(yv);
    rg.widen(gv);
    rx.widen(xv);
    fetch(row + step);
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
      if (gate) z *= gv[i] * sigmoid<T>(gv[i]);
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
    const size_t most = 152 * (G <= 128 ? 6 : G == 256 ? 3 : 1);  // (a GB300's SMs)
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
