// block_norm_bwd.cu -- the gradients of the block norm (block_norm.cu).  With
// a = silu(gate), t = a z, X = x' and xh = X rsqrt(mean(X^2) + eps), yh = y rsqrt(mean(y^2) + eps):
//     dX = dx' + r_x (w_pre dh - xh mean(w_pre dh xh)),          dw_pre = sum dh xh,
//     dx = dX,   dres_scale = sum dX t,   dgate = dX res_scale z silu'(gate),
//     dz = dX res_scale a,   dw_post = sum dz yh,   dy = r_y (w_post dz - yh mean(w_post dz yh)),
// silu'(g) = s (1 + g (1 - s)), s = 1 / (1 + e^-g); sums over the rows.
//
// Bound by memory: the five row inputs are read once and the three row gradients written once;
// a row stays in registers across its three sums, the next one is on its
// way, and the weights wait in shared memory (in registers they cost half the resident rows).  With
// every part: 222 us at 32768 x 2048 bf16, 4.8 TB/s (issue slots 58 %, two CTAs of 256 threads per SM; fp32
// pairs saved 10 %); 338 us at 65536 x 1024 fp32, 6.4 TB/s.  The column sums stay in registers over
// a CTA's rows and are written once per CTA; a second kernel adds them in a fixed order, so the
// result does not vary from run to run.
#include <initializer_list>

#include "block_norm.cuh"
#include "launch.h"

namespace mesa {

namespace {

// CTAs on an SM (fp32 rows of up to 1024 channels: three, 338 us at 65536 x 1024; with four what is read
// ahead spills, 360).
template <typename T, int G>
constexpr int resident() {
  return G <= 128 ? (sizeof(T) == 4 ? 3 : 4) : G == 256 ? 2 : 1;
}
template <typename T, int VEC, int G>
__global__ void __launch_bounds__(G < 128 ? 128 : G, resident<T, G>()) mesa_block_norm_bwd_kernel(NormArgs a) {
  using namespace norm;
  constexpr int RPC = G < 128 ? 128 / G : 1;
  __shared__ float red[2][1][32], red2[2][2][32];
  constexpr int BLOCK = G < 128 ? 128 : G, P = EPT / 2;
  extern __shared__ __align__(16) float wsm[];  // three weights of a row's channels, as the threads hold them
  const int lane = threadIdx.x % G, sub = threadIdx.x / G, D = a.D;
  const float inv_d = 1.0f / (float)D;
  // weight k's channels of a thread, two at a time: the pair at wsm + 2 ((k EPT / 2 + i) G + lane)
  for (int t = threadIdx.x; t < 3 * G; t += BLOCK) {
    const int k = t / G, l = t % G;
    float v[EPT];
    load_weights<VEC, G>(k == 0 ? a.w_post : k == 1 ? a.res_scale : a.w_pre, l, D, k == 2 ? 0.0f : 1.0f, v);
#pragma unroll
    for (int i = 0; i < EPT; i++) wsm[2 * ((k * (EPT / 2) + i / 2) * G + l) + (i & 1)] = v[i];
  }
  __syncthreads();
  const u64 *wp = reinterpret_cast<const u64 *>(wsm) + lane, *rs = wp + P * G, *wn = rs + P * G;
  const T *x = (const T *)a.x, *y = (const T *)a.y, *gate = (const T *)a.gate;
  const T *dxo = (const T *)a.dx_out, *dh = (const T *)a.dh;
  const bool pre = a.w_pre && dh;
  // d - xh mean(d xh), the part of a norm's gradient across the row.  A row of one channel has
  // xh^2 = 1 - eps r^2: the difference, d eps r^2, is taken as such (in fp32 it would cancel).
  const bool one = D == 1;
  auto along = [&](u64 d, u64 xh, float m, float r) -> u64 {
    const float e = a.eps * r * r;
    return one ? mul2(d, pack2(e, e)) : fma2(xh, pack2(-m, -m), d);
  };
  u64 cpost[P] = {}, cscale[P] = {}, cpre[P] = {};
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
    u64 yv[P], gv[P], X[P], dX[P], dhv[P];
    ry.pairs(yv);
    rg.pairs(gv);
    rx.pairs(X);
    rd.pairs(dX);
    rh.pairs(dhv);
    fetch(row + step);
    float r = 1.0f;
    if (a.w_post) {
      u64 t = 0;
#pragma unroll
      for (int i = 0; i < P; i++) t = fma2(yv[i], yv[i], t);
      float ss[1] = {sum2(t)};
      row_sums<G>(ss, red, buf);
      r = rsqrtf(fmaf(ss[0], inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < P; i++) yv[i] = mul2(yv[i], pack2(r, r));  // y normalised
    }
    u64 act[P], dact[P];
#pragma unroll
    for (int i = 0; i < P; i++) {
      act[i] = pack2(1.0f, 1.0f);
      dact[i] = 0;
      if (gate) {
        float g0, g1;
        unpack2(gv[i], g0, g1);
        const u64 s = pack2(sigmoid<T>(g0), sigmoid<T>(g1));
        dact[i] = mul2(s, fma2(gv[i], sub2(act[i], s), act[i]));
        act[i] = mul2(gv[i], s);
      }
    }
    u64 az[P];  // act z
#pragma unroll
    for (int i = 0; i < P; i++) az[i] = mul2(act[i], mul2(yv[i], wp[i * G]));
    if (pre) {
      u64 t0 = 0, t1 = 0;
#pragma unroll
      for (int i = 0; i < P; i++) {
        X[i] = fma2(rs[i * G], az[i], X[i]);
        t0 = fma2(X[i], X[i], t0);
        t1 = fma2(mul2(dhv[i], wn[i * G]), X[i], t1);
      }
      float ss[2] = {sum2(t0), sum2(t1)};
      row_sums<G>(ss, red2, buf2);
      const float rn = rsqrtf(fmaf(ss[0], inv_d, a.eps));
      const float m = ss[1] * rn * inv_d;  // mean(w_pre dh xh)
      const u64 rn2 = pack2(rn, rn);
#pragma unroll
      for (int i = 0; i < P; i++) {
        const u64 xh = mul2(X[i], rn2);
        cpre[i] = fma2(dhv[i], xh, cpre[i]);
        dX[i] = fma2(rn2, along(mul2(dhv[i], wn[i * G]), xh, m, rn), dX[i]);
      }
    }
    if (a.dx) store_pairs<VEC, G>((T *)a.dx + at, lane, D, in, dX);
    u64 t = 0;
#pragma unroll
    for (int i = 0; i < P; i++) {
      cscale[i] = fma2(dX[i], az[i], cscale[i]);
      const u64 d = mul2(dX[i], rs[i * G]), dz = mul2(d, act[i]), w = wp[i * G];
      gv[i] = mul2(mul2(d, dact[i]), mul2(yv[i], w));  // dgate
      cpost[i] = fma2(dz, yv[i], cpost[i]);
      dX[i] = mul2(dz, w);
      t = fma2(dX[i], yv[i], t);
    }
    if (a.dgate) store_pairs<VEC, G>((T *)a.dgate + at, lane, D, in, gv);
    if (a.w_post) {
      float ss[1] = {sum2(t)};
      row_sums<G>(ss, red, buf);
      const float m = ss[0] * inv_d;
#pragma unroll
      for (int i = 0; i < P; i++) dX[i] = mul2(along(dX[i], yv[i], m, r), pack2(r, r));
    }
    store_pairs<VEC, G>((T *)a.dy + at, lane, D, in, dX);
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
  float cp[EPT], cs[EPT], cn[EPT];
#pragma unroll
  for (int i = 0; i < P; i++) {
    unpack2(cpost[i], cp[2 * i], cp[2 * i + 1]);
    unpack2(cscale[i], cs[2 * i], cs[2 * i + 1]);
    unpack2(cpre[i], cn[2 * i], cn[2 * i + 1]);
  }
  if constexpr (G < 32) {  // the rows of a warp
#pragma unroll
    for (int i = 0; i < EPT; i++)
#pragma unroll
      for (int o = G; o < 32; o *= 2) {
        cp[i] += __shfl_xor_sync(0xffffffffu, cp[i], o);
        cs[i] += __shfl_xor_sync(0xffffffffu, cs[i], o);
        cn[i] += __shfl_xor_sync(0xffffffffu, cn[i], o);
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
            cp[i] += c[0];
            cs[i] += c[EPT * G];
            cn[i] += c[2 * EPT * G];
          }
          c[0] = cp[i];
          c[EPT * G] = cs[i];
          c[2 * EPT * G] = cn[i];
        }
      }
    }
    if (part != 0) return;
  }
  if (threadIdx.x % W < G)
    each([&](int c, int i) {
      out[c] = cp[i];
      out[D + c] = cs[i];
      out[2 * D + c] = cn[i];
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
    const int most = norm_bwd_ctas(a.N, a.D), ctas = most < 152 * resident<T, G>() ? most : 152 * resident<T, G>();
    constexpr int smem = 3 * norm::EPT * G * (int)sizeof(float);
    // (48 KB without being asked for, the row sums' static part among them: rows of more than 2048 channels)
    if (smem >= 48 * 1024 && cudaFuncSetAttribute(mesa_block_norm_bwd_kernel<T, VEC, G>,
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
