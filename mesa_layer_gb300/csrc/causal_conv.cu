// causal_conv.cu -- short causal depthwise convolution with bias and SiLU: forward, one decode step, gradients.
//
//     y_t = bias + sum_{s < W} w_s x_{t-s},   o_t = silu(y_t) or y_t,
// taps that would reach before a document's first token left out.  A thread owns a few channels and walks a run of
// tokens with the last W - 1 inputs in registers (the run's own W - 1 predecessors are read again), so that every
// input is read about once and nothing goes through shared memory.  Bound by memory.
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "mixer_ops.h"
#include "overlap.cuh"
#include "packed.cuh"

namespace mesa {

namespace {

constexpr int kBlock = 256, kFwdBlock = 128;

// VEC consecutive channels as fp32 pairs.
template <typename TIO, int VEC>
struct Vec;
template <>
struct Vec<float, 4> {
  using Raw = float4;
  __device__ static void unpack(Raw r, u64 (&v)[2]) { v[0] = pack2(r.x, r.y), v[1] = pack2(r.z, r.w); }
  __device__ static Raw pack(const u64 (&v)[2]) {
    Raw r;
    unpack2(v[0], r.x, r.y);
    unpack2(v[1], r.z, r.w);
    return r;
  }
};
__device__ __forceinline__ u64 bf2(uint32_t w) { return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t to_bf2(u64 v) {
  float x, y;
  unpack2(v, x, y);
  const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t *>(&b);
}
template <>
struct Vec<__nv_bfloat16, 4> {
  using Raw = uint2;
  __device__ static void unpack(Raw r, u64 (&v)[2]) { v[0] = bf2(r.x), v[1] = bf2(r.y); }
  __device__ static Raw pack(const u64 (&v)[2]) { return make_uint2(to_bf2(v[0]), to_bf2(v[1])); }
};
// The taps of VEC channels from channel c0 of head h on, and their bias.
template <int VEC, int W>
__device__ __forceinline__ void load_taps(const ConvArgs &a, int h, int c0, u64 (&w)[W][VEC / 2], u64 (&bias)[VEC / 2]) {
  const float *wh = a.w + ((size_t)h * a.d + c0) * W;
#pragma unroll
  for (int p = 0; p < VEC / 2; p++) {
#pragma unroll
    for (int s = 0; s < W; s++) w[s][p] = pack2(wh[2 * p * W + s], wh[(2 * p + 1) * W + s]);
    bias[p] = a.bias ? pack2(a.bias[(size_t)h * a.d + c0 + 2 * p], a.bias[(size_t)h * a.d + c0 + 2 * p + 1]) : pack2(0.0f, 0.0f);
  }
}
// sigmoid(y) from the hardware's exponential and division (2^-21 relative error).
__device__ __forceinline__ u64 sigmoid2(u64 y) {
  float p, q;
  unpack2(mul2(y, pack2(-1.4426950408889634f, -1.4426950408889634f)), p, q);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(p));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(q));
  unpack2(add2(pack2(p, q), pack2(1.0f, 1.0f)), p, q);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(p));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(q));
  return pack2(p, q);
}
__device__ __forceinline__ u64 silu2(u64 y) { return mul2(y, sigmoid2(y)); }

// The inputs before token t0 of unit u that tap windows from there reach: x[s] the one s tokens back, s = 1 .. W - 1,
// zero across a document's start.  Returns how many of them belong to token t0 - 1's document.
template <typename TIO, int VEC, int W>
__device__ __forceinline__ int load_window(const ConvArgs &a, int u, int t0, int c0, u64 (&x)[W][VEC / 2]) {
  using V = Vec<TIO, VEC>;
  const TIO *src = static_cast<const TIO *>(a.x) + (size_t)u * a.T * a.d + c0;
  const uint8_t *starts = a.starts ? a.starts + (size_t)(u / a.H) * a.T : nullptr;
  int alive = 0;
  bool on = true;
#pragma unroll
  for (int s = 1; s < W; s++) {
    const int t = t0 - s;
    if (s > 1 && t + 1 >= 0 && starts && on) on = starts[t + 1] == 0;
#pragma unroll
    for (int p = 0; p < VEC / 2; p++) x[s][p] = pack2(0.0f, 0.0f);
    if (!on) continue;
    if (t >= 0) {
      V::unpack(*reinterpret_cast<const typename V::Raw *>(src + (size_t)t * a.d), x[s]);
      alive = s;
    } else if (a.state0) {
      const float *h = a.state0 + ((size_t)u * (W - 1) + (-t - 1)) * a.d + c0;
#pragma unroll
      for (int p = 0; p < VEC / 2; p++) x[s][p] = pack2(h[2 * p], h[2 * p + 1]);
      alive = s;
    }
  }
  return alive;
}

// Thread (unit, run, channel group) over runs of `run` tokens; the next AHEAD tokens' inputs are on their way while the
// present ones are worked on.
// (Seven CTAs per SM where that fits: 60 -> 58 us at 8 x 16 x 4096 x 128.)
template <typename TIO, int VEC, int W, bool PACKED>
__global__ void __launch_bounds__(kFwdBlock, sizeof(TIO) == 2 && W <= 4 && !PACKED ? 7 : 1) mesa_causal_conv_kernel(ConvArgs a, int run, int runs) {
  using V = Vec<TIO, VEC>;
  constexpr int AHEAD = 4, P = VEC / 2;
  const int groups = a.d / VEC;
  const size_t i = (size_t)blockIdx.x * kFwdBlock + threadIdx.x, total = (size_t)a.B * a.H * runs * groups;
  if (i >= total) return;
  const int c0 = (int)(i % groups) * VEC, r = (int)(i / groups % runs), u = (int)(i / groups / runs);
  const int t0 = r * run, t1 = min(t0 + run, a.T);
  const TIO *src = static_cast<const TIO *>(a.x) + (size_t)u * a.T * a.d + c0;
  TIO *dst = static_cast<TIO *>(a.out) + (size_t)u * a.T * a.d + c0;
  const uint8_t *starts = PACKED ? a.starts + (size_t)(u / a.H) * a.T : nullptr;
  u64 w[W][P], bias[P], x[W][P];
  typename V::Raw raw[2][AHEAD];
  bool cut[2][AHEAD];
  auto load = [&](int t, typename V::Raw (&x)[AHEAD], bool (&c)[AHEAD], bool whole) {
#pragma unroll
    for (int j = 0; j < AHEAD; j++)
      if (whole || t + j < t1) {
        x[j] = *reinterpret_cast<const typename V::Raw *>(src + (size_t)(t + j) * a.d);
        if (PACKED) c[j] = starts[t + j];
      }
  };
  auto work = [&](int t, typename V::Raw (&raw)[AHEAD], bool (&cut)[AHEAD], bool whole) {
#pragma unroll
    for (int j = 0; j < AHEAD; j++) {
      if (!whole && t + j >= t1) break;
      if (PACKED && cut[j]) {
#pragma unroll
        for (int s = 1; s < W; s++)
#pragma unroll
          for (int p = 0; p < P; p++) x[s][p] = 0;
      }
      V::unpack(raw[j], x[0]);
      u64 y[P];
#pragma unroll
      for (int p = 0; p < P; p++) {
        y[p] = fma2(w[0][p], x[0][p], bias[p]);
#pragma unroll
        for (int s = 1; s < W; s++) y[p] = fma2(w[s][p], x[s][p], y[p]);
        if (a.silu) y[p] = silu2(y[p]);
      }
      *reinterpret_cast<typename V::Raw *>(dst + (size_t)(t + j) * a.d) = V::pack(y);
#pragma unroll
      for (int s = W - 1; s > 0; s--)
#pragma unroll
        for (int p = 0; p < P; p++) x[s][p] = x[s - 1][p];
    }
  };
  load(t0, raw[0], cut[0], false);
  load_window<TIO, VEC, W>(a, u, t0, c0, x);
  load_taps<VEC, W>(a, u % a.H, c0, w, bias);
  int t = t0;
#pragma unroll 1
  for (; t + 3 * AHEAD <= t1; t += 2 * AHEAD) {
    load(t + AHEAD, raw[1], cut[1], true);
    work(t, raw[0], cut[0], true);
    load(t + 2 * AHEAD, raw[0], cut[0], true);
    work(t + AHEAD, raw[1], cut[1], true);
  }
#pragma unroll 1
  for (; t < t1; t += AHEAD) {  // the last tokens
    work(t, raw[0], cut[0], false);
    load(t + AHEAD, raw[0], cut[0], false);
  }
  if (W > 1 && a.state && t1 == a.T) {
#pragma unroll
    for (int s = 1; s < W; s++)
#pragma unroll
      for (int p = 0; p < P; p++)
        *reinterpret_cast<u64 *>(a.state + ((size_t)u * (W - 1) + s - 1) * a.d + c0 + 2 * p) = x[s][p];
  }
}

// One token of B x H units; the window [B, H, W - 1, d] moves on in place.
template <typename TIO, int W>
__global__ void __launch_bounds__(128) mesa_causal_conv_step_kernel(ConvArgs a) {
  using V = Vec<TIO, 4>;
  const int groups = a.d / 4;
  const size_t i = (size_t)blockIdx.x * 128 + threadIdx.x, total = (size_t)a.B * a.H * groups;
  if (i >= total) return;
  const int c0 = (int)(i % groups) * 4;
  const size_t u = i / groups;
  u64 w[W][2], bias[2], x[W][2];
  V::unpack(*reinterpret_cast<const typename V::Raw *>(static_cast<const TIO *>(a.x) + u * a.d + c0), x[0]);
  float *hist = a.state + u * (W - 1) * a.d + c0;
#pragma unroll
  for (int s = 1; s < W; s++) {
    const ulonglong2 h = *reinterpret_cast<const ulonglong2 *>(hist + (size_t)(s - 1) * a.d);
    x[s][0] = h.x, x[s][1] = h.y;
  }
  load_taps<4, W>(a, (int)(u % a.H), c0, w, bias);
  u64 y[2];
#pragma unroll
  for (int p = 0; p < 2; p++) {
    y[p] = fma2(w[0][p], x[0][p], bias[p]);
#pragma unroll
    for (int s = 1; s < W; s++) y[p] = fma2(w[s][p], x[s][p], y[p]);
    if (a.silu) y[p] = silu2(y[p]);
  }
  *reinterpret_cast<typename V::Raw *>(static_cast<TIO *>(a.out) + u * a.d + c0) = V::pack(y);
#pragma unroll
  for (int s = 1; s < W; s++)
    *reinterpret_cast<ulonglong2 *>(hist + (size_t)(s - 1) * a.d) = make_ulonglong2(x[s - 1][0], x[s - 1][1]);
}

// ---- gradients ---------------------------------------------------------------------------------------
// dy_t = do_t silu'(y_t),   dx_t = sum_s w_s dy_{t+s} (inside the document),   dw_s = sum_t dy_t x_{t-s}.
// Block: GX channel groups of four x rows of runs; part p of a head's (batch, run) pairs; sums over a part's tokens stay
// in registers, those of the parts are added by mesa_causal_conv_cols_kernel, both in a fixed order.
constexpr int kBwdRun = 64;
constexpr int kBwdVec = 4;  // channels a thread (two: half the registers, but 153 us)
__host__ __device__ inline int bwd_gx(int d) { return d / kBwdVec < 32 ? d / kBwdVec : 32; }

// (Two CTAs per SM: 203 -> 140 us at 8 x 16 x 4096 x 128; runs of 64 tokens instead of 32: 138.)
template <typename TIO, int W, bool PACKED>
__global__ void __launch_bounds__(kBlock, 2) mesa_causal_conv_bwd_kernel(ConvArgs a, int parts, int runs) {
  using V = Vec<TIO, kBwdVec>;
  constexpr int AHEAD = 4, VEC = kBwdVec, P = VEC / 2, N = VEC * (W + 1);
  extern __shared__ float sm[];
  const int gx = bwd_gx(a.d), rows = kBlock / gx, g = threadIdx.x % gx, row = threadIdx.x / gx;
  const int h = blockIdx.z, c0 = (blockIdx.y * gx + g) * VEC, pairs = a.B * runs;
  const bool on = row < rows && c0 < a.d;
  u64 dw[W][P] = {}, db[P] = {};
  if (on) {
    u64 w[W][P], bias[P];
    load_taps<VEC, W>(a, h, c0, w, bias);
    for (int pr = blockIdx.x * rows + row; pr < pairs; pr += parts * rows) {
      const int b = pr / runs, u = b * a.H + h, t0 = pr % runs * kBwdRun, t1 = min(t0 + kBwdRun, a.T);
      const size_t base = (size_t)u * a.T * a.d + c0;
      const TIO *src = static_cast<const TIO *>(a.x) + base, *dout = static_cast<const TIO *>(a.dout) + base;
      TIO *dx = static_cast<TIO *>(a.dx) + base;
      const uint8_t *starts = PACKED ? a.starts + (size_t)b * a.T : nullptr;
      u64 x[W][P], pend[W][P] = {};  // pend[s]: what the tokens so far give dx_{t-s}
      int age;  // tokens before t of its document, W - 1 at most
      struct Token {
        typename V::Raw x, g;
        bool cut;
      };
      auto load = [&](int t, Token &in) {
        in.x = *reinterpret_cast<const typename V::Raw *>(src + (size_t)t * a.d);
        in.g = *reinterpret_cast<const typename V::Raw *>(dout + (size_t)t * a.d);
        if (PACKED) in.cut = starts[t];
      };
      // Token t: dx of token t - (W - 1) is complete (EMIT: it is the run's own); MINE: so is t.
      auto token = [&](int t, const Token &in, auto mine, auto emit) {
        if (PACKED && in.cut) {
          age = 0;
#pragma unroll
          for (int s = 1; s < W; s++)
#pragma unroll
            for (int p = 0; p < P; p++) x[s][p] = 0;
        }
        u64 dy[P];
        V::unpack(in.x, x[0]);
        V::unpack(in.g, dy);
        if (a.silu) {
#pragma unroll
          for (int p = 0; p < P; p++) {
            u64 y = fma2(w[0][p], x[0][p], bias[p]);
#pragma unroll
            for (int s = 1; s < W; s++) y = fma2(w[s][p], x[s][p], y);
            const u64 one = pack2(1.0f, 1.0f), g = sigmoid2(y);  // silu' = g (1 + y (1 - g))
            dy[p] = mul2(dy[p], mul2(g, fma2(y, sub2(one, g), one)));
          }
        }
        if constexpr (decltype(mine)::value) {
#pragma unroll
          for (int p = 0; p < P; p++) {
            db[p] = add2(db[p], dy[p]);
#pragma unroll
            for (int s = 0; s < W; s++) dw[s][p] = fma2(dy[p], x[s][p], dw[s][p]);
          }
        }
        if (!PACKED || age >= W - 1) {
#pragma unroll
          for (int p = 0; p < P; p++)
#pragma unroll
            for (int s = W - 1; s > 0; s--) pend[s][p] = fma2(w[s][p], dy[p], pend[s - 1][p]);
        } else {  // a document's first tokens: nothing of theirs reaches the one before
#pragma unroll
          for (int p = 0; p < P; p++)
#pragma unroll
            for (int s = W - 1; s > 0; s--) pend[s][p] = age < s ? pend[s - 1][p] : fma2(w[s][p], dy[p], pend[s - 1][p]);
        }
#pragma unroll
        for (int p = 0; p < P; p++) pend[0][p] = mul2(w[0][p], dy[p]);
        if constexpr (decltype(emit)::value)
          *reinterpret_cast<typename V::Raw *>(dx + (size_t)(t - (W - 1)) * a.d) = V::pack(pend[W - 1]);
        if (PACKED) age = min(age + 1, W - 1);
#pragma unroll
        for (int s = W - 1; s > 0; s--)
#pragma unroll
          for (int p = 0; p < P; p++) x[s][p] = x[s - 1][p];
      };
      constexpr std::true_type yes{};
      constexpr std::false_type no{};
      Token in[2][AHEAD];
      int t = t0;
      age = load_window<TIO, VEC, W>(a, u, t0, c0, x);
      const int lead = min(t0 + W - 1, t1);
#pragma unroll 1
      for (; t < lead; t++) {  // nothing of the run's own is complete yet
        load(t, in[0][0]);
        token(t, in[0][0], yes, no);
      }
      if (t + 2 * AHEAD <= t1) {
#pragma unroll
        for (int j = 0; j < AHEAD; j++) load(t + j, in[0][j]);
#pragma unroll 1
        for (; t + 3 * AHEAD <= t1; t += 2 * AHEAD) {  // (the next tokens are on their way)
#pragma unroll
          for (int j = 0; j < AHEAD; j++) load(t + AHEAD + j, in[1][j]);
#pragma unroll
          for (int j = 0; j < AHEAD; j++) token(t + j, in[0][j], yes, yes);
#pragma unroll
          for (int j = 0; j < AHEAD; j++) load(t + 2 * AHEAD + j, in[0][j]);
#pragma unroll
          for (int j = 0; j < AHEAD; j++) token(t + AHEAD + j, in[1][j], yes, yes);
        }
#pragma unroll
        for (int j = 0; j < AHEAD; j++) token(t + j, in[0][j], yes, yes);
        t += AHEAD;
      }
#pragma unroll 1
      for (; t < t1; t++) {
        load(t, in[0][0]);
        token(t, in[0][0], yes, yes);
      }
#pragma unroll 1
      for (; t < t1 + W - 1 && t < a.T; t++) {  // the next run's first tokens
        load(t, in[0][0]);
        token(t, in[0][0], no, yes);
      }
#pragma unroll
      for (int s = W - 1; s >= 1; s--)  // the sequence's end (t = T): token t - s's sum is in pend[s - 1]
        if (t < t1 + W - 1 && t - s >= t0 && t - s < t1)
          *reinterpret_cast<typename V::Raw *>(dx + (size_t)(t - s) * a.d) = V::pack(pend[s - 1]);
    }
  }
  may_follow();
  if (!a.partial) return;
  // the rows' sums: [row][value][group]
#pragma unroll
  for (int p = 0; p < P; p++)
#pragma unroll
    for (int s = 0; s <= W; s++) {
      float lo, hi;
      unpack2(s < W ? dw[s < W ? s : 0][p] : db[p], lo, hi);
      if (row < rows) {
        sm[(row * N + 2 * p * (W + 1) + s) * gx + g] = lo;
        sm[(row * N + (2 * p + 1) * (W + 1) + s) * gx + g] = hi;
      }
    }
  __syncthreads();
  float *dst = a.partial + (size_t)blockIdx.x * a.H * a.d * (W + 1);
  for (int i = threadIdx.x; i < N * gx; i += kBlock) {
    const int gg = i % gx, v = i / gx, c = (blockIdx.y * gx + gg) * VEC + v / (W + 1);
    if (c >= a.d) continue;
    float x = 0.0f;
    for (int r = 0; r < rows; r++) x += sm[(r * N + v) * gx + gg];
    dst[((size_t)h * a.d + c) * (W + 1) + v % (W + 1)] = x;
  }
}

// Eight lanes a value over the parts' sums.
__global__ void __launch_bounds__(kBlock) mesa_causal_conv_cols_kernel(ConvArgs a, int parts) {
  const int n = a.H * a.d * (a.W + 1), i = (blockIdx.x * kBlock + threadIdx.x) / 8, l = threadIdx.x & 7;
  ahead_done();
  float x = 0.0f;
  if (i < n)
    for (int p = l; p < parts; p += 8) x += a.partial[(size_t)p * n + i];
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (i >= n || l != 0) return;
  const int s = i % (a.W + 1), c = i / (a.W + 1);
  if (s == a.W) {
    if (a.dbias) a.dbias[c] = x;
  } else if (a.dw) {
    a.dw[(size_t)c * a.W + s] = x;
  }
}

template <typename F>
int by_width(int W, F f) {
  switch (W) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    default: return f(std::integral_constant<int, 8>());
  }
}
int done() { return cudaPeekAtLastError() == cudaSuccess ? 0 : -1; }

template <typename TIO, int VEC>
int forward(const ConvArgs &a, cudaStream_t st) {
  // runs of 64 tokens (W - 1 are read twice), shorter ones where that leaves SMs idle
  const size_t lanes = (size_t)a.B * a.H * (a.d / VEC);
  int run = 64;
  while (run > 8 && lanes * ((a.T + run - 1) / run) < 152 * 1024) run /= 2;
  const int runs = (a.T + run - 1) / run;
  const size_t blocks = (lanes * runs + kFwdBlock - 1) / kFwdBlock;
  if (blocks > 0x7fffffff) return -1;
  return by_width(a.W, [&](auto w) {
    timing_mark_begin(K_CONV, st);
    if (a.starts)
      mesa_causal_conv_kernel<TIO, VEC, decltype(w)::value, true><<<(unsigned)blocks, kFwdBlock, 0, st>>>(a, run, runs);
    else
      mesa_causal_conv_kernel<TIO, VEC, decltype(w)::value, false><<<(unsigned)blocks, kFwdBlock, 0, st>>>(a, run, runs);
    timing_mark_end(K_CONV, st);
    return done();
  });
}

template <typename TIO>
int backward(const ConvArgs &a, cudaStream_t st) {
  const int parts = conv_bwd_parts(a.B, a.H, a.T, a.d), gx = bwd_gx(a.d), runs = (a.T + kBwdRun - 1) / kBwdRun;
  return by_width(a.W, [&](auto w) {
    constexpr int W = decltype(w)::value;
    const size_t smem = a.partial ? (size_t)(kBlock / gx) * gx * kBwdVec * (W + 1) * sizeof(float) : 0;
    timing_mark_begin(K_CONV_BWD, st);
    const dim3 grid(parts, (a.d / kBwdVec + gx - 1) / gx, a.H);
    if (a.starts)
      mesa_causal_conv_bwd_kernel<TIO, W, true><<<grid, kBlock, smem, st>>>(a, parts, runs);
    else
      mesa_causal_conv_bwd_kernel<TIO, W, false><<<grid, kBlock, smem, st>>>(a, parts, runs);
    timing_mark_end(K_CONV_BWD, st);
    if (a.partial) {
      timing_mark_begin(K_CONV_COLS, st);
      const bool ok = launch_after(mesa_causal_conv_cols_kernel, (unsigned)(((size_t)a.H * a.d * (W + 1) * 8 + kBlock - 1) / kBlock), kBlock, 0,
                                   st, a, parts);
      timing_mark_end(K_CONV_COLS, st);
      if (!ok) return -1;
    }
    return done();
  });
}

template <typename TIO>
int step(const ConvArgs &a, cudaStream_t st) {
  const size_t blocks = ((size_t)a.B * a.H * (a.d / 4) + 127) / 128;
  if (blocks > 0x7fffffff) return -1;
  return by_width(a.W, [&](auto w) {
    timing_mark_begin(K_CONV_STEP, st);
    mesa_causal_conv_step_kernel<TIO, decltype(w)::value><<<(unsigned)blocks, 128, 0, st>>>(a);
    timing_mark_end(K_CONV_STEP, st);
    return done();
  });
}

}  // namespace

// Two CTAs for each of a GB300's 152 SMs (what their registers allow at once) over all heads and channels, no more than
// there are runs.  (us of 8 x 16 x 4096 x 128: two 166, three 221, four 189, six 192)
int conv_bwd_parts(int B, int H, int T, int d) {
  const int gx = bwd_gx(d), rows = kBlock / gx, slabs = (d / kBwdVec + gx - 1) / gx;
  const size_t pairs = (size_t)B * ((T + kBwdRun - 1) / kBwdRun), most = (pairs + rows - 1) / rows;
  size_t n = 152 * 2 / ((size_t)H * slabs);
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

int launch_causal_conv(const ConvArgs &a, cudaStream_t st) {
  return a.dtype == 1 ? forward<__nv_bfloat16, 4>(a, st) : forward<float, 4>(a, st);
}
int launch_causal_conv_step(const ConvArgs &a, cudaStream_t st) {
  return a.dtype == 1 ? step<__nv_bfloat16>(a, st) : step<float>(a, st);
}
int launch_causal_conv_backward(const ConvArgs &a, cudaStream_t st) {
  return a.dtype == 1 ? backward<__nv_bfloat16>(a, st) : backward<float>(a, st);
}

}  // namespace mesa
