// causal_conv.cu -- short causal depthwise convolution with bias and SiLU: forward, one decode step, gradients.
//
//     y_t = bias + sum_{s < W} w_s x_{t-s},   o_t = silu(y_t) or y_t,
// taps that would reach before a document's first token left out.  A thread owns a few channels and walks a run of
// tokens with the last W - 1 inputs in registers (the run's own W - 1 predecessors are read again), so that every
// input is read about once; nothing is shared between threads but the gradients' last sums.
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
// sigmoid(y) from the hardware's exponential and division: 2^-21 relative error for fp32 outputs, down to 2^-120 (0 below).  For
// bf16 ones, whose own rounding is 2^-9, without what the exponent's rounding leaves out (|y| 2^-24: 2^-17 at y = -88; with it an
// fp32 forward of 8 x 16 x 4096 x 128 takes 97 us instead of 89, the gradients 145 instead of 141).
template <typename TIO>
__device__ __forceinline__ u64 sigmoid2(u64 y) {
  constexpr bool F32 = std::is_same<TIO, float>::value;
  const u64 c = pack2(-1.4426950408889634f, -1.4426950408889634f);
  float p, q;
  if constexpr (F32) {  // (beyond these it is 0 or 1, and what is infinite has no rest; NaN comes back with y)
    unpack2(y, p, q);
    y = pack2(fminf(fmaxf(p, -88.0f), 88.0f), fminf(fmaxf(q, -88.0f), 88.0f));
  }
  const u64 x = mul2(y, c);
  unpack2(x, p, q);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(p));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(q));
  u64 e = pack2(p, q);
  if constexpr (F32) {  // 2^(x + r) = 2^x (1 + r ln 2); r: the product's rounding and the constant's
    const u64 r = fma2(y, pack2(-1.9259629911266175e-8f, -1.9259629911266175e-8f), fma2(y, c, mul2(x, pack2(-1.0f, -1.0f))));
    e = fma2(e, mul2(r, pack2(0.69314718f, 0.69314718f)), e);
  }
  unpack2(add2(e, pack2(1.0f, 1.0f)), p, q);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(p));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(q));
  return pack2(p, q);
}
template <typename TIO>
__device__ __forceinline__ u64 silu2(u64 y) {
  return mul2(y, sigmoid2<TIO>(y));
}

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
// (Seven CTAs per SM for bf16 and up to four taps without documents, though four taps then leave 36 bytes a thread in local
// memory: 60 -> 58 us at 8 x 16 x 4096 x 128.)
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
        if (a.silu) y[p] = silu2<TIO>(y[p]);
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
    if (a.silu) y[p] = silu2<TIO>(y[p]);
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
constexpr int kBwdBlock = 128;
constexpr int kBwdVec = 4;  // channels a thread (two: half the registers, but 153 us)
__host__ __device__ inline int bwd_gx(int d) { return d / kBwdVec < 32 ? d / kBwdVec : 32; }

// As many CTAs as a GB300's 152 SMs hold at once (bwd_ctas: what keeps taps, windows and sums in registers, but for 4 to 20
// bytes a thread with documents and W = 5, 7, or 2 in fp32; four tokens' chains interleave, and more warps with values in local memory lose: W = 4 with
// three, four, five, six CTAs an SM 95, 93, 116, 136 us at 8 x 16 x 4096 x 128; W = 8 with two, three 172, 212), shared by all heads and channels; and runs of which
// every row takes as many as the others, as nearly as that goes (in parts of a sequence of 16 tokens at least; a run costs
// about four tokens more than it has).  us of 8 x 16 x 4001 x 128: runs of 64 tokens, three or four a row, 137; this, the
// inputs on their way in shared memory instead of registers, and no case distinction while no document starts, 98 (75 % of a copy's rate at W = 2 and in fp32; at W = 4 the packed products' pipe
// and the exponentials' latency, 45 % of the issue slots).
struct BwdSplit {
  int parts, run, runs;  // CTAs that share a head's channels; tokens a run, runs a sequence
};
constexpr int bwd_ctas(int W) { return W <= 2 ? 6 : W <= 5 ? 4 : W <= 7 ? 3 : 2; }
BwdSplit bwd_split(int B, int H, int T, int d, int W) {
  const int gx = bwd_gx(d), rows = kBwdBlock / gx, slabs = (d / kBwdVec + gx - 1) / gx;
  const int n = max(152 * bwd_ctas(W) / (H * slabs), 1), slots = n * rows;
  BwdSplit best{1, T > 0 ? T : 1, 1};
  double least = 1e30;
  for (int each = 1; each <= 8; each++) {
    long long runs = max(1LL, (long long)each * slots / B);  // (tokens and a run's length together may pass 32 bits)
    const int run = max((int)((T + runs - 1) / runs), 16);
    runs = max(1LL, ((long long)T + run - 1) / run);
    const long long all = B * runs;
    const double cost = (double)((all + slots - 1) / slots) * (run + 4);
    if (cost < least) {
      least = cost;
      best = {(int)min((all + rows - 1) / rows, (long long)n), run, (int)runs};
    }
  }
  return best;
}

// 8 or 16 bytes to shared memory, in flight until the wait for their group.
template <int N>
__device__ __forceinline__ void copy_ahead(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// A thread's inputs come through shared memory of its own, kRing groups of kGroup tokens: [ring][token][x, dout][thread].
constexpr int kGroup = 4;
constexpr int kRing = 2;  // (three or four: the same times)
template <typename TIO>
constexpr uint32_t kRingBytes = kRing * kGroup * 2 * kBwdBlock * kBwdVec * sizeof(TIO);

template <typename TIO, int W, bool PACKED>
__global__ void __launch_bounds__(kBwdBlock, bwd_ctas(W)) mesa_causal_conv_bwd_kernel(ConvArgs a, int parts, int run, int runs) {
  using V = Vec<TIO, kBwdVec>;
  using Raw = typename V::Raw;
  constexpr int VEC = kBwdVec, P = VEC / 2, N = VEC * (W + 1), RING = kRing;
  extern __shared__ __align__(16) uint8_t ring[];
  const int gx = bwd_gx(a.d), rows = kBwdBlock / gx, g = threadIdx.x % gx, row = threadIdx.x / gx;
  const int h = blockIdx.z, c0 = (blockIdx.y * gx + g) * VEC, pairs = a.B * runs;
  const bool on = row < rows && c0 < a.d;
  u64 dw[W][P] = {}, db[P] = {};
  if (on) {
    u64 w[W][P], bias[P];
    load_taps<VEC, W>(a, h, c0, w, bias);
    Raw *const mine_at = reinterpret_cast<Raw *>(ring) + threadIdx.x;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(mine_at);
#pragma unroll 1
    for (int pr = blockIdx.x * rows + row; pr < pairs; pr += parts * rows) {
      const int b = pr / runs, u = b * a.H + h, t0 = pr % runs * run, t1 = t0 + min(run, a.T - t0), end = min(t1 + W - 1, a.T);
      const size_t base = (size_t)u * a.T * a.d + c0;
      const TIO *src = static_cast<const TIO *>(a.x) + base, *dout = static_cast<const TIO *>(a.dout) + base;
      TIO *dx = static_cast<TIO *>(a.dx) + base;
      const uint8_t *starts = PACKED ? a.starts + (size_t)b * a.T : nullptr;
      u64 x[W][P], pend[W][P] = {};  // pend[s]: what the tokens so far give dx_{t-s}
      auto fetch = [&](int t, int slot) {
#pragma unroll
        for (int j = 0; j < kGroup; j++)
          if (t + j < end) {
            const uint32_t at = to + ((slot * kGroup + j) * 2 * kBwdBlock) * (uint32_t)sizeof(Raw);
            copy_ahead<sizeof(Raw)>(at, src + (size_t)(t + j) * a.d);
            copy_ahead<sizeof(Raw)>(at + kBwdBlock * (uint32_t)sizeof(Raw), dout + (size_t)(t + j) * a.d);
          }
        copies_commit();
      };
      auto any_start = [&](int t) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < kGroup; j++)
          if (PACKED && t + j < end) any |= starts[t + j] != 0;
        return any;
      };
#pragma unroll
      for (int k = 0; k < RING - 1; k++) fetch(t0 + k * kGroup, k);
      bool later = any_start(t0);
      int age = load_window<TIO, VEC, W>(a, u, t0, c0, x);  // tokens before t of its document, W - 1 at most
      // Token t: dx of token t - (W - 1) is complete (emit: it is the run's own); mine: so is t.  fresh: it may be among the
      // first W - 1 of its document.
      auto token = [&](int t, const Raw *in, bool fresh, bool mine, bool emit) {
        if (fresh && starts[t]) {
          age = 0;
#pragma unroll
          for (int s = 1; s < W; s++)
#pragma unroll
            for (int p = 0; p < P; p++) x[s][p] = 0;
        }
        u64 dy[P];
        V::unpack(in[0], x[0]);
        V::unpack(in[kBwdBlock], dy);
        if (a.silu) {
#pragma unroll
          for (int p = 0; p < P; p++) {
            u64 y = fma2(w[0][p], x[0][p], bias[p]);
#pragma unroll
            for (int s = 1; s < W; s++) y = fma2(w[s][p], x[s][p], y);
            const u64 one = pack2(1.0f, 1.0f), g = sigmoid2<TIO>(y);  // silu' = g (1 + y (1 - g))
            dy[p] = mul2(dy[p], mul2(g, fma2(y, sub2(one, g), one)));
          }
        }
        if (mine) {
#pragma unroll
          for (int p = 0; p < P; p++) {
            db[p] = add2(db[p], dy[p]);
#pragma unroll
            for (int s = 0; s < W; s++) dw[s][p] = fma2(dy[p], x[s][p], dw[s][p]);
          }
        }
        if (!fresh || age >= W - 1) {
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
        if (emit) *reinterpret_cast<Raw *>(dx + (size_t)(t - (W - 1)) * a.d) = V::pack(pend[W - 1]);
        if (fresh) age = min(age + 1, W - 1);
#pragma unroll
        for (int s = W - 1; s > 0; s--)
#pragma unroll
          for (int p = 0; p < P; p++) x[s][p] = x[s - 1][p];
      };
      int slot = 0;
#pragma unroll 1
      for (int t = t0; t < end; t += kGroup) {
        fetch(t + (RING - 1) * kGroup, slot == 0 ? RING - 1 : slot - 1);
        const bool fresh = PACKED && (later || age < W - 1);
        later = any_start(t + kGroup);
        copies_wait<RING - 1>();
        const Raw *in = mine_at + slot * kGroup * 2 * kBwdBlock;
        if (t >= t0 + W - 1 && t + kGroup <= t1 && !fresh) {
#pragma unroll
          for (int j = 0; j < kGroup; j++) token(t + j, in + j * 2 * kBwdBlock, false, true, true);
        } else {  // (the run's first tokens and the next one's, a document's first ones)
#pragma unroll 1
          for (int j = 0; j < kGroup && t + j < end; j++)
            token(t + j, in + j * 2 * kBwdBlock, PACKED, t + j < t1, t + j >= t0 + W - 1);
        }
        if (++slot == RING) slot = 0;
      }
#pragma unroll
      for (int s = W - 1; s >= 1; s--)  // the sequence's end (end = T): token T - s's sum is in pend[s - 1]
        if (end < t1 + W - 1 && end - s >= t0 && end - s < t1)
          *reinterpret_cast<Raw *>(dx + (size_t)(end - s) * a.d) = V::pack(pend[s - 1]);
    }
  }
  may_follow();
  if (!a.partial) return;
  // the rows' sums: [row][value][group]
  float *const sm = reinterpret_cast<float *>(ring);
  __syncthreads();  // (every row has read its inputs)
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
  for (int i = threadIdx.x; i < N * gx; i += kBwdBlock) {
    const int gg = i % gx, v = i / gx, c = (blockIdx.y * gx + gg) * VEC + v / (W + 1);
    if (c >= a.d) continue;
    float x = 0.0f;
    for (int r = 0; r < rows; r++) x += sm[(r * N + v) * gx + gg];
    dst[((size_t)h * a.d + c) * (W + 1) + v % (W + 1)] = x;
  }
}

// Eight lanes a value over the parts' sums.
__global__ void __launch_bounds__(kBlock) mesa_causal_conv_cols_kernel(ConvArgs a, int parts) {
  // (64 bits: heads of 65536 channels pass 32 with eight taps from 3641 heads on, eight lanes a value from 911 on)
  const size_t n = (size_t)a.H * a.d * (a.W + 1), i = ((size_t)blockIdx.x * kBlock + threadIdx.x) / 8;
  const int l = threadIdx.x & 7;
  ahead_done();
  float x = 0.0f;
  if (i < n)
    for (int p = l; p < parts; p += 8) x += a.partial[p * n + i];
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (i >= n || l != 0) return;
  const size_t c = i / (a.W + 1);
  const int s = (int)(i - c * (a.W + 1));
  if (s == a.W) {
    if (a.dbias) a.dbias[c] = x;
  } else if (a.dw) {
    a.dw[c * a.W + s] = x;
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
  const BwdSplit split = bwd_split(a.B, a.H, a.T, a.d, a.W);
  const int parts = split.parts, gx = bwd_gx(a.d);
  return by_width(a.W, [&](auto w) {
    constexpr int W = decltype(w)::value;
    const size_t sums = a.partial ? (size_t)(kBwdBlock / gx) * gx * kBwdVec * (W + 1) * sizeof(float) : 0;
    const size_t smem = sums > kRingBytes<TIO> ? sums : kRingBytes<TIO>;
    timing_mark_begin(K_CONV_BWD, st);
    const dim3 grid(parts, (a.d / kBwdVec + gx - 1) / gx, a.H);
    auto kernel = a.starts ? mesa_causal_conv_bwd_kernel<TIO, W, true> : mesa_causal_conv_bwd_kernel<TIO, W, false>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return -1;
    kernel<<<grid, kBwdBlock, smem, st>>>(a, parts, split.run, split.runs);
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

int conv_bwd_parts(int B, int H, int T, int d, int W) { return bwd_split(B, H, T, d, W).parts; }

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
