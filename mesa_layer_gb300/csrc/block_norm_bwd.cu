// block_norm_bwd.cu -- the gradients of the block norm (block_norm.cu).  With
// a = silu(gate), t = a z, X = x' and xh = X rsqrt(mean(X^2) + eps), yh = y rsqrt(mean(y^2) + eps):
//     dX = dx' + r_x (w_pre dh - xh mean(w_pre dh xh)),          dw_pre = sum dh xh,
//     dx = dX,   dres_scale = sum dX t,   dgate = dX res_scale z silu'(gate),
//     dz = dX res_scale a,   dw_post = sum dz yh,   dy = r_y (w_post dz - yh mean(w_post dz yh)),
// silu'(g) = s (1 + g (1 - s)), s = 1 / (1 + e^-g); sums over the rows.
//
// Bound by memory: the five row inputs are read once and the three row gradients written once;
// a row stays in registers across its three sums.  The column sums stay in registers over a
// CTA's rows and are written once per CTA; a second kernel adds them in a fixed order, so the
// result does not vary from run to run.
#include <initializer_list>

#include "block_norm.cuh"
#include "launch.h"

namespace mesa {

namespace {

template <typename T, int VEC, int G>
__global__ void __launch_bounds__(G < 128 ? 128 : G) mesa_block_norm_bwd_kernel(NormArgs a) {
  using namespace norm;
  constexpr int RPC = G < 128 ? 128 / G : 1;
  __shared__ float red[2][1][32], red2[2][2][32];
  extern __shared__ float cols[];  // [3][D] when a CTA holds several rows
  const int lane = threadIdx.x % G, sub = threadIdx.x / G, D = a.D;
  const float inv_d = 1.0f / (float)D;
  float wp[EPT], rs[EPT], wn[EPT];
  load_weights<VEC, G>(a.w_post, lane, D, 1.0f, wp);
  load_weights<VEC, G>(a.res_scale, lane, D, 1.0f, rs);
  load_weights<VEC, G>(a.w_pre, lane, D, 0.0f, wn);
  const T *x = (const T *)a.x, *y = (const T *)a.y, *gate = (const T *)a.gate;
  const T *dxo = (const T *)a.dx_out, *dh = (const T *)a.dh;
  const bool pre = a.w_pre && dh;
  // d - xh mean(d xh), the part of a norm's gradient across the row.  A row of one channel has
  // xh^2 = 1 - eps r^2: the difference, d eps r^2, is taken as such (in fp32 it would cancel).
  const bool one = D == 1;
  const float eps = a.eps;
  auto along = [one, eps](float d, float xh, float m, float r) {
    return one ? d * (eps * r * r) : fmaf(-xh, m, d);
  };
  float cpost[EPT] = {}, cscale[EPT] = {}, cpre[EPT] = {};
  int buf = 0, buf2 = 0;
  for (size_t base = (size_t)blockIdx.x * RPC; base < (size_t)a.N; base += (size_t)gridDim.x * RPC) {
    const size_t row = base + sub, at = row * D;
    const bool in = row < (size_t)a.N;
    float yv[EPT], gv[EPT], X[EPT], dX[EPT], dhv[EPT];
    load_row<VEC, G>(y + at, lane, D, in, yv);
    load_row<VEC, G>(gate + at, lane, D, in && gate, gv);
    load_row<VEC, G>(x + at, lane, D, in && x && pre, X);
    load_row<VEC, G>(dxo + at, lane, D, in && dxo, dX);
    load_row<VEC, G>(dh + at, lane, D, in && pre, dhv);
    float r = 1.0f;
    if (a.w_post) {
      float ss[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < EPT; i++) ss[0] = fmaf(yv[i], yv[i], ss[0]);
      row_sums<G>(ss, red, buf);
      r = rsqrtf(fmaf(ss[0], inv_d, a.eps));
    }
    float act[EPT], dact[EPT];
#pragma unroll
    for (int i = 0; i < EPT; i++) {
      yv[i] *= r;  // y normalised
      if (gate) {
        const float s = 1.0f / (1.0f + expf(-gv[i]));
        act[i] = gv[i] * s;
        dact[i] = s * fmaf(gv[i], 1.0f - s, 1.0f);
      } else {
        act[i] = 1.0f;
        dact[i] = 0.0f;
      }
    }
    if (pre) {
      float ss[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < EPT; i++) {
        X[i] = fmaf(rs[i], yv[i] * wp[i] * act[i], X[i]);
        ss[0] = fmaf(X[i], X[i], ss[0]);
        ss[1] = fmaf(dhv[i] * wn[i], X[i], ss[1]);
      }
      row_sums<G>(ss, red2, buf2);
      const float rn = rsqrtf(fmaf(ss[0], inv_d, a.eps));
      const float m = ss[1] * rn * inv_d;  // mean(w_pre dh xh)
#pragma unroll
      for (int i = 0; i < EPT; i++) {
        const float xh = X[i] * rn;
        cpre[i] = fmaf(dhv[i], xh, cpre[i]);
        dX[i] = fmaf(rn, along(dhv[i] * wn[i], xh, m, rn), dX[i]);
      }
    }
    if (a.dx) store_row<VEC, G>((T *)a.dx + at, lane, D, in, dX);
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < EPT; i++) {
      const float z = yv[i] * wp[i];
      cscale[i] = fmaf(dX[i], act[i] * z, cscale[i]);
      const float d = dX[i] * rs[i];
      gv[i] = d * z * dact[i];  // dgate
      const float dz = d * act[i];
      cpost[i] = fmaf(dz, yv[i], cpost[i]);
      dX[i] = dz * wp[i];
      ss[0] = fmaf(dX[i], yv[i], ss[0]);
    }
    if (a.dgate) store_row<VEC, G>((T *)a.dgate + at, lane, D, in, gv);
    if (a.w_post) {
      row_sums<G>(ss, red, buf);
      const float m = ss[0] * inv_d;
#pragma unroll
      for (int i = 0; i < EPT; i++) dX[i] = r * along(dX[i], yv[i], m, r);
    }
    store_row<VEC, G>((T *)a.dy + at, lane, D, in, dX);
  }
  if (!a.partial) return;
  float *out = a.partial + (size_t)blockIdx.x * 3 * D;
  auto each = [&](auto f) {  // f(channel, register)
#pragma unroll
    for (int i = 0; i < EPT / VEC; i++)
#pragma unroll
      for (int k = 0; k < VEC; k++) {
        const int c = (lane + i * G) * VEC + k;
        if (c < D) f(c, i * VEC + k);
      }
  };
  if constexpr (RPC == 1) {
    each([&](int c, int i) {
      out[c] = cpost[i];
      out[D + c] = cscale[i];
      out[2 * D + c] = cpre[i];
    });
  } else {
    // the rows of a CTA in turn
    for (int s = 0; s < RPC; s++) {
      if (sub == s)
        each([&](int c, int i) {
          cols[c] = cpost[i] + (s ? cols[c] : 0.0f);
          cols[D + c] = cscale[i] + (s ? cols[D + c] : 0.0f);
          cols[2 * D + c] = cpre[i] + (s ? cols[2 * D + c] : 0.0f);
        });
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 3 * D; c += blockDim.x) out[c] = cols[c];
  }
}

// Column c of the three sums: 8 partial sums over the CTAs, then their sum.  Block 32 x 8.
__global__ void __launch_bounds__(256) mesa_block_norm_cols_kernel(NormArgs a, int ctas) {
  __shared__ float sh[8][32];
  const int cx = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx, n = 3 * a.D;
  float s = 0.0f;
  if (c < n)
    for (int r = part; r < ctas; r += 8) s += a.partial[(size_t)r * n + c];
  sh[part][cx] = s;
  __syncthreads();
  if (part != 0 || c >= n) return;
#pragma unroll
  for (int p = 1; p < 8; p++) s += sh[p][cx];
  float *dst = c < a.D ? a.dw_post : c < 2 * a.D ? a.dres_scale : a.dw_pre;
  if (dst) dst[c % a.D] = s;
}

template <typename T, int VEC, int G>
struct Backward {
  static int run(const NormArgs &a, cudaStream_t st) {
    const int ctas = norm_bwd_ctas(a.N, a.D);
    const int smem = G < 128 ? 3 * a.D * (int)sizeof(float) : 0;
    timing_mark_begin(K_NORM_BWD, st);
    mesa_block_norm_bwd_kernel<T, VEC, G><<<ctas, G < 128 ? 128 : G, smem, st>>>(a);
    timing_mark_end(K_NORM_BWD, st);
    if (a.partial) {
      timing_mark_begin(K_NORM_COLS, st);
      mesa_block_norm_cols_kernel<<<(3 * a.D + 31) / 32, 256, 0, st>>>(a, ctas);
      timing_mark_end(K_NORM_COLS, st);
    }
    return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
  }
};

}  // namespace

int launch_block_norm_backward(const NormArgs &a, cudaStream_t st) {
  return norm::dispatch<Backward>(
      a, norm::vec_of(a.D, a.dtype, {a.x, a.y, a.gate, a.dx_out, a.dh, a.dx, a.dy, a.dgate}), st);
}

}  // namespace mesa
