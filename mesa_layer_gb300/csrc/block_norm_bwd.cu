// block_norm_bwd.cu -- the gradients of the block norm (block_norm.cu).  With
// a = silu(gate), t = a z, X = x' and xh = X rsqrt(mean(X^2) + eps), yh = y rsqrt(mean(y^2) + eps):
//     dX = dx' + r_x (w_pre dh - xh mean(w_pre dh xh)),          dw_pre = sum dh xh,
//     dx = dX,   dres_scale = sum dX t,   dgate = dX res_scale z silu'(gate),
//     dz = dX res_scale a,   dw_post = sum dz yh,   dy = r_y (w_post dz - yh mean(w_post dz yh)),
// silu'(g) = s (1 + g (1 - s)), s = 1 / (1 + e^-g); sums over the rows.
//
// Bound by memory: the five row inputs are read once and the three row gradients written once;
// a row stays in registers across its three sums, the next one is on its
// way, and the weights wait in shared memory (in registers they cost half the resident rows).  The column sums stay in registers over a
// CTA's rows and are written once per CTA; a second kernel adds them in a fixed order, so the
// result does not vary from run to run.
#include <initializer_list>

#include "block_norm.cuh"
#include "launch.h"

namespace mesa {

namespace {

template <typename T, int VEC, int G>
__global__ void __launch_bounds__(G < 128 ? 128 : G, G <= 128 ? 4 : G == 256 ? 2 : 1) mesa_block_norm_bwd_kernel(NormArgs a) {
  using namespace norm;
  constexpr int RPC = G < 128 ? 128 / G : 1;
  __shared__ float red[2][1][32], red2[2][2][32];
  constexpr int BLOCK = G < 128 ? 128 : G;
  extern __shared__ __align__(16) float wsm[];  // three weights of a row's channels, as the threads hold them
  const int lane = threadIdx.x % G, sub = threadIdx.x / G, D = a.D;
  const float inv_d = 1.0f / (float)D;
  // weight k's channels of a thread: wsm[(k EPT + i) G + lane]
  for (int t = threadIdx.x; t < 3 * G; t += BLOCK) {
    const int k = t / G, l = t % G;
    float v[EPT];
    load_weights<VEC, G>(k == 0 ? a.w_post : k == 1 ? a.res_scale : a.w_pre, l, D, k == 2 ? 0.0f : 1.0f, v);
#pragma unroll
    for (int i = 0; i < EPT; i++) wsm[(k * EPT + i) * G + l] = v[i];
  }
  __syncthreads();
  const float *wp = wsm + lane, *rs = wp + EPT * G, *wn = rs + EPT * G;
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
  const size_t N = (size_t)a.N, step = (size_t)gridDim.x * RPC;
  Raw<T, VEC> ry, rg, rx, rd, rh;
  auto fetch = [&](size_t row) {
    const bool in = row < N;
    ry.template load<G>(y + row * D, lane, D, in);
    rg.template load<G>(gate + row * D, lane, D, in && gate);
    rx.template load<G>(x + row * D, lane, D, in && x && pre);
    rd.template load<G>(dxo + row * D, lane, D, in && dxo);
    rh.template load<G>(dh + row * D, lane, D, in && pre);
  };
  fetch((size_t)blockIdx.x * RPC + sub);
  for (size_t base = (size_t)blockIdx.x * RPC; base < N; base += step) {
    const size_t row = base + sub, at = row * D;
    const bool in = row < N;
    float yv[EPT], gv[EPT], X[EPT], dX[EPT], dhv[EPT];
    ry.widen(yv);
    rg.widen(gv);
    rx.widen(X);
    rd.widen(dX);
    rh.widen(dhv);
    fetch(row + step);
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
        const float s = sigmoid<T>(gv[i]);
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
        X[i] = fmaf(rs[i * G], yv[i] * wp[i * G] * act[i], X[i]);
        ss[0] = fmaf(X[i], X[i], ss[0]);
        ss[1] = fmaf(dhv[i] * wn[i * G], X[i], ss[1]);
      }
      row_sums<G>(ss, red2, buf2);
      const float rn = rsqrtf(fmaf(ss[0], inv_d, a.eps));
      const float m = ss[1] * rn * inv_d;  // mean(w_pre dh xh)
#pragma unroll
      for (int i = 0; i < EPT; i++) {
        const float xh = X[i] * rn;
        cpre[i] = fmaf(dhv[i], xh, cpre[i]);
        dX[i] = fmaf(rn, along(dhv[i] * wn[i * G], xh, m, rn), dX[i]);
      }
    }
    if (a.dx) store_row<VEC, G>((T *)a.dx + at, lane, D, in, dX);
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < EPT; i++) {
      const float z = yv[i] * wp[i * G];
      cscale[i] = fmaf(dX[i], act[i] * z, cscale[i]);
      const float d = dX[i] * rs[i * G];
      gv[i] = d * z * dact[i];  // dgate
      const float dz = d * act[i];
      cpost[i] = fmaf(dz, yv[i], cpost[i]);
      dX[i] = dz * wp[i * G];
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
  if constexpr (G < 32) {  // the rows of a warp
#pragma unroll
    for (int i = 0; i < EPT; i++)
#pragma unroll
      for (int o = G; o < 32; o *= 2) {
        cpost[i] += __shfl_xor_sync(0xffffffffu, cpost[i], o);
        cscale[i] += __shfl_xor_sync(0xffffffffu, cscale[i], o);
        cpre[i] += __shfl_xor_sync(0xffffffffu, cpre[i], o);
      }
  }
  constexpr int W = G < 32 ? 32 : G, PARTS = BLOCK / W;  // threads that hold one sum; sums left in the CTA
  if constexpr (PARTS > 1) {  // in turn, through the weights' place ([3][EPT][G])
    float *cols = wsm;
    const int part = threadIdx.x / W;
    for (int p = PARTS - 1; p >= 0; p--) {
      __syncthreads();
      if (part == p && threadIdx.x % W < G) {
#pragma unroll
        for (int i = 0; i < EPT; i++) {
          float *c = cols + i * G + lane;
          if (p < PARTS - 1) {
            cpost[i] += c[0];
            cscale[i] += c[EPT * G];
            cpre[i] += c[2 * EPT * G];
          }
          c[0] = cpost[i];
          c[EPT * G] = cscale[i];
          c[2 * EPT * G] = cpre[i];
        }
      }
    }
    if (part != 0) return;
  }
  if (threadIdx.x % W < G)
    each([&](int c, int i) {
      out[c] = cpost[i];
      out[D + c] = cscale[i];
      out[2 * D + c] = cpre[i];
    });
}

// Column c of the three sums: 32 partial sums over the CTAs, then their sum.  Block 32 x 32.
__global__ void __launch_bounds__(1024) mesa_block_norm_cols_kernel(NormArgs a, int ctas) {
  __shared__ float sh[32][33];
  const int cx = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx, n = 3 * a.D;
  float s = 0.0f;
  if (c < n)
    for (int r = part; r < ctas; r += 32) s += a.partial[(size_t)r * n + c];
  sh[part][cx] = s;
  __syncthreads();
  s = warp_sum(sh[cx][part]);  // column `part` of the block
  const int d = blockIdx.x * 32 + part;
  if (cx != 0 || d >= n) return;
  float *dst = d < a.D ? a.dw_post : d < 2 * a.D ? a.dres_scale : a.dw_pre;
  if (dst) dst[d % a.D] = s;
}

template <typename T, int VEC, int G>
struct Backward {
  static int run(const NormArgs &a, cudaStream_t st) {
    const int ctas = norm_bwd_ctas(a.N, a.D);
    constexpr int smem = 3 * norm::EPT * G * (int)sizeof(float);
    if (smem > 48 * 1024 && cudaFuncSetAttribute(mesa_block_norm_bwd_kernel<T, VEC, G>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return -1;
    timing_mark_begin(K_NORM_BWD, st);
    mesa_block_norm_bwd_kernel<T, VEC, G><<<ctas, G < 128 ? 128 : G, smem, st>>>(a);
    timing_mark_end(K_NORM_BWD, st);
    if (a.partial) {
      timing_mark_begin(K_NORM_COLS, st);
      mesa_block_norm_cols_kernel<<<(3 * a.D + 31) / 32, 1024, 0, st>>>(a, ctas);
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
