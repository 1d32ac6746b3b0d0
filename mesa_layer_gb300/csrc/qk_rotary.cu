// qk_rotary.cu -- norms of queries and keys per head with the position rotation in the same pass, and their gradients.
//
// Per row x of d channels: n = x rsqrt(mean(x^2) + eps) w; the first R channels turn by the angles pos f_j,
//     o_a = s (n_a cos - n_b sin),   o_b = s (n_b cos + n_a sin),
// in pairs (a, b) = (j, j + R/2) or (2j, 2j + 1).  So o_c = n_c C_c + n_{pair(c)} S_c with C = s cos, S = -s sin for
// a, s sin for b, and C = 1, S = 0 past R.  L = d / VEC lanes hold a row; a lane takes the angles of its channels once for a token and
// walks over heads, so that the sines cost little and what bounds it is memory.  Gradients turn back
// (n_c <- g_c C_c - g_{pair(c)} S_c) and go through the norm:
//     dx = r (m - xn mean(m xn)),   m = dn w,   xn = x r,   dw = sum over rows of dn xn.
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "mixer_ops.h"
#include "overlap.cuh"

namespace mesa {

namespace {

constexpr int kBlock = 256, kFwdBlock = 128;
enum Pairs { kNone = 0, kNeighbours = 1, kHalves = 2, kAnyHalves = 3 };  // kHalves: R/2 a multiple of a lane's channels

template <typename TIO>
struct Row;
template <>
struct Row<float> {
  static constexpr int VEC = 4;
  using Raw = uint4;
  __device__ static void unpack(Raw r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
  __device__ static Raw pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
};
template <>
struct Row<__nv_bfloat16> {
  static constexpr int VEC = 8;
  using Raw = uint4;
  __device__ static void unpack(Raw r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; i++) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  __device__ static Raw pack(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// cos and sin of pos f, for any 32-bit position: the turns pos f / (2 pi) as a sum of exact parts (the position in two
// pieces of 19 and 12 bits, f / (2 pi) in two fp32 values), whole turns taken out of each.
__device__ __forceinline__ void rotation(int pos, float f, float &c, float &s) {
  constexpr float kHi = 0.15915494f, kLo = 6.4206383e-9f;  // 1 / (2 pi) = kHi + kLo
  const float g = f * kHi, gl = fmaf(f, kHi, -g) + f * kLo;
  const float a = (float)(pos & ~4095), b = (float)(pos & 4095);
  float p = a * g, q = b * g;
  const float e = (fmaf(a, g, -p) + fmaf(b, g, -q)) + (a * gl + b * gl);
  p -= rintf(p);
  q -= rintf(q);
  float t = (p + q) + e;
  t -= rintf(t);
  sincospif(2.0f * t, &s, &c);
}

// A lane's share of a token's rotation: C and S of its channels c0 ..
template <int VEC, int PAIRS>
__device__ __forceinline__ void token_angles(const RotaryArgs &a, size_t token, int c0, float (&C)[VEC], float (&S)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; i++) C[i] = 1.0f, S[i] = 0.0f;
  if constexpr (PAIRS == kNone) return;
  const int pos = a.positions ? a.positions[token] : a.offset + (int)(token % a.T), half = a.R / 2;
  float co, si;
  if constexpr (PAIRS == kNeighbours) {
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      if (c0 + i >= a.R) continue;
      rotation(pos, a.inv_freq[(c0 + i) / 2], co, si);
      C[i] = C[i + 1] = a.rot_scale * co;
      S[i] = -a.rot_scale * si;
      S[i + 1] = a.rot_scale * si;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i++) {
      const int c = c0 + i;
      if (c >= a.R) continue;
      rotation(pos, a.inv_freq[c < half ? c : c - half], co, si);
      C[i] = a.rot_scale * co;
      S[i] = c < half ? -a.rot_scale * si : a.rot_scale * si;
    }
  }
}

// The pairs' values of this lane's channels of one row (raw: the lane's own; row: the row in memory); 0 for channels that do
// not turn (their S is 0, but 0 times what is not finite would not be).
template <typename TIO, int PAIRS>
__device__ __forceinline__ void pairs_of(const RotaryArgs &a, const TIO *row, uint4 raw, int c0, float (&p)[Row<TIO>::VEC]) {
  constexpr int VEC = Row<TIO>::VEC;
  const int half = a.R / 2;
  if constexpr (PAIRS == kNeighbours) {
    float v[VEC];
    Row<TIO>::unpack(raw, v);
#pragma unroll
    for (int i = 0; i < VEC; i++) p[i] = c0 + i < a.R ? v[i ^ 1] : 0.0f;
  } else if constexpr (PAIRS == kHalves) {  // another lane's channels, in the same places
    const int lane = threadIdx.x & 31, from = c0 < half ? lane + half / VEC : c0 < a.R ? lane - half / VEC : lane;
    raw.x = __shfl_sync(0xffffffffu, raw.x, from);
    raw.y = __shfl_sync(0xffffffffu, raw.y, from);
    raw.z = __shfl_sync(0xffffffffu, raw.z, from);
    raw.w = __shfl_sync(0xffffffffu, raw.w, from);
    if (c0 >= a.R) raw = make_uint4(0, 0, 0, 0);
    Row<TIO>::unpack(raw, p);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i++) {
      const int c = c0 + i;
      p[i] = c < half ? ld(row, c + half) : c < a.R ? ld(row, c - half) : 0.0f;
    }
  }
}
// The channel that c turns with.
template <int PAIRS>
__device__ __forceinline__ int pair_of(const RotaryArgs &a, int c) {
  if constexpr (PAIRS == kNeighbours) return c ^ 1;
  return c < a.R / 2 ? c + a.R / 2 : c < a.R ? c - a.R / 2 : c;
}

// L lanes a token, grid.y groups of `heads` heads (the query heads, then the key heads).  The lanes past the last
// token work on it and write nothing.  Outputs may replace inputs: a warp reads its rows before it writes.
// (Four rows in flight a lane, eight CTAs of 128 threads per SM.  us of 8 x (16 + 16) x 4096 x 128, pairs of halves /
// neighbours: CTAs of 256 threads without a bound of registers 127 / 96, with it 109 / 90; so, 105 / 88.)
template <typename TIO, int D, int PAIRS>
__global__ void __launch_bounds__(kFwdBlock, 8) mesa_qk_norm_rotary_kernel(RotaryArgs a, int heads) {
  using R = Row<TIO>;
  constexpr int VEC = R::VEC, BATCH = 4, L = D / VEC;
  const int c0 = (threadIdx.x % L) * VEC;
  const size_t tokens = (size_t)a.B * a.T, mine = ((size_t)blockIdx.x * kFwdBlock + threadIdx.x) / L;
  const bool in = mine < tokens;
  const size_t token = in ? mine : tokens - 1, b = token / a.T, t = token % a.T;
  float C[VEC], S[VEC];
  token_angles<VEC, PAIRS>(a, token, c0, C, S);
  const int first = blockIdx.y * heads, last = min(first + heads, a.H + a.Hk);
#pragma unroll
  for (int which = 0; which < 2; which++) {
    const int H = which == 0 ? a.H : a.Hk, h0 = which == 0 ? first : max(first - a.H, 0), h1 = which == 0 ? min(last, H) : last - a.H;
    const TIO *src = static_cast<const TIO *>(which == 0 ? a.q : a.k);
    TIO *dst = static_cast<TIO *>(which == 0 ? a.q_out : a.k_out);
    const float *w = which == 0 ? a.wq : a.wk;
    float cw[VEC], sw[VEC];  // C and S times the weights
#pragma unroll
    for (int j = 0; j < VEC; j++) {
      cw[j] = w ? C[j] * w[c0 + j] : C[j];
      sw[j] = w && PAIRS != kNone ? S[j] * w[pair_of<PAIRS>(a, c0 + j)] : S[j];
    }
#pragma unroll 1
    for (int h = h0; h < h1; h += BATCH) {
      uint4 raw[BATCH];
      float far[PAIRS == kAnyHalves ? BATCH : 1][VEC];
      size_t at[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        at[i] = ((b * H + min(h + i, h1 - 1)) * a.T + t) * D;
        raw[i] = *reinterpret_cast<const uint4 *>(src + at[i] + c0);
        if constexpr (PAIRS == kAnyHalves) pairs_of<TIO, PAIRS>(a, src + at[i], raw[i], c0, far[i]);
      }
      if constexpr (PAIRS == kAnyHalves) __syncwarp();  // (the row is read: it may be written)
      float r[BATCH];
      if (a.norm) {
#pragma unroll
        for (int i = 0; i < BATCH; i++) {
          float x[VEC];
          R::unpack(raw[i], x);
          r[i] = 0.0f;
#pragma unroll
          for (int j = 0; j < VEC; j++) r[i] = fmaf(x[j], x[j], r[i]);
        }
#pragma unroll
        for (int i = 0; i < BATCH; i++) r[i] = rsqrtf(fmaf(group_sum<L>(r[i]), 1.0f / D, a.eps));
      }
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        float x[VEC], p[VEC];
        R::unpack(raw[i], x);
        if constexpr (PAIRS == kNeighbours || PAIRS == kHalves) pairs_of<TIO, PAIRS>(a, src, raw[i], c0, p);
        const float f = a.norm ? r[i] : 1.0f;
#pragma unroll
        for (int j = 0; j < VEC; j++)
          x[j] = f * (PAIRS == kNone ? x[j] * cw[j] : fmaf(PAIRS == kAnyHalves ? far[PAIRS == kAnyHalves ? i : 0][j] : p[j], sw[j], x[j] * cw[j]));
        if (in && h + i < h1) *reinterpret_cast<uint4 *>(dst + at[i] + c0) = R::pack(x);
      }
    }
  }
}

// (Four rows in flight a lane, two CTAs per SM: 166 / 152 us, halves / neighbours; two rows and four CTAs 185 / 188.)
// A resident grid walks over the tokens; sums of the weights' gradients stay in registers until the end.
template <typename TIO, int D, int PAIRS>
__global__ void __launch_bounds__(kBlock, 2) mesa_qk_norm_rotary_bwd_kernel(RotaryArgs a) {
  using R = Row<TIO>;
  constexpr int VEC = R::VEC, BATCH = 4, L = D / VEC, per = kBlock / L;
  __shared__ float sums[kBlock][VEC + 1];
  const int c0 = (threadIdx.x % L) * VEC;
  const size_t tokens = (size_t)a.B * a.T;
  float dw[2][VEC] = {};
  for (size_t first = (size_t)blockIdx.x * per; first < tokens; first += (size_t)gridDim.x * per) {
    const size_t mine = first + threadIdx.x / L;
    const bool in = mine < tokens;
    const size_t token = in ? mine : tokens - 1, b = token / a.T, t = token % a.T;
    float C[VEC], S[VEC];
    token_angles<VEC, PAIRS>(a, token, c0, C, S);
#pragma unroll
    for (int which = 0; which < 2; which++) {
      const int H = which == 0 ? a.H : a.Hk;
      const TIO *xs = static_cast<const TIO *>(which == 0 ? a.q : a.k), *gs = static_cast<const TIO *>(which == 0 ? a.dq_out : a.dk_out);
      TIO *ds = static_cast<TIO *>(which == 0 ? a.q_out : a.k_out);
      const float *w = which == 0 ? a.wq : a.wk;
      float wc[VEC];
#pragma unroll
      for (int j = 0; j < VEC; j++) wc[j] = w ? w[c0 + j] : 1.0f;
#pragma unroll 1
      for (int h = 0; h < H; h += BATCH) {
        uint4 xr[BATCH], gr[BATCH];
        float far[PAIRS == kAnyHalves ? BATCH : 1][VEC];
        size_t at[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; i++) {
          at[i] = ((b * H + min(h + i, H - 1)) * a.T + t) * D;
          gr[i] = *reinterpret_cast<const uint4 *>(gs + at[i] + c0);
          if (a.norm) xr[i] = *reinterpret_cast<const uint4 *>(xs + at[i] + c0);
          if constexpr (PAIRS == kAnyHalves) pairs_of<TIO, PAIRS>(a, gs + at[i], gr[i], c0, far[i]);
        }
        if constexpr (PAIRS == kAnyHalves) __syncwarp();  // (the row is read: it may be written)
#pragma unroll
        for (int i = 0; i < BATCH; i++) {
          const bool on = in && h + i < H;
          float g[VEC];
          R::unpack(gr[i], g);
          if constexpr (PAIRS != kNone) {
            float p[VEC];
            if constexpr (PAIRS != kAnyHalves) pairs_of<TIO, PAIRS>(a, gs, gr[i], c0, p);
#pragma unroll
            for (int j = 0; j < VEC; j++) g[j] = fmaf(PAIRS == kAnyHalves ? -far[PAIRS == kAnyHalves ? i : 0][j] : -p[j], S[j], g[j] * C[j]);
          }
          if (a.norm) {
            float x[VEC], ss = 0.0f, mx = 0.0f;
            R::unpack(xr[i], x);
#pragma unroll
            for (int j = 0; j < VEC; j++) {
              ss = fmaf(x[j], x[j], ss);
              mx = fmaf(g[j] * wc[j], x[j], mx);
            }
            ss = group_sum<L>(ss);
            mx = group_sum<L>(mx);
            const float r = rsqrtf(fmaf(ss, 1.0f / D, a.eps)), mean = mx * r * (1.0f / D), rr = on ? r : 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; j++) {
              dw[which][j] = fmaf(g[j] * rr, x[j], dw[which][j]);
              g[j] = r * fmaf(-(x[j] * r), mean, g[j] * wc[j]);
            }
          }
          if (on) *reinterpret_cast<uint4 *>(ds + at[i] + c0) = R::pack(g);
        }
      }
    }
  }
  may_follow();
  if (!a.partial) return;
#pragma unroll
  for (int which = 0; which < 2; which++) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < VEC; j++) sums[threadIdx.x][j] = dw[which][j];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kBlock) {
      float x = 0.0f;
      for (int r = 0; r < per; r++) x += sums[r * L + c / VEC][c % VEC];
      a.partial[((size_t)blockIdx.x * 2 + which) * D + c] = x;
    }
  }
}

// A warp a channel over the CTAs' sums.
__global__ void __launch_bounds__(kBlock) mesa_qk_norm_rotary_cols_kernel(RotaryArgs a, int parts) {
  const int i = (blockIdx.x * kBlock + threadIdx.x) / 32, lane = threadIdx.x & 31;
  ahead_done();
  if (i >= 2 * a.d) return;
  float x = 0.0f;
  for (int p = lane; p < parts; p += 32) x += a.partial[(size_t)p * 2 * a.d + i];
  x = warp_sum(x);
  float *dst = i < a.d ? a.dwq : a.dwk;
  if (lane == 0 && dst) dst[i % a.d] = x;
}

int pairs_kind(const RotaryArgs &a) {
  const int vec = a.dtype == 1 ? 8 : 4;
  return a.R == 0 ? kNone : a.interleaved ? kNeighbours : a.R / 2 % vec == 0 ? kHalves : kAnyHalves;
}
// f(channels, kind of pairs)
template <typename F>
int by_pairs(const RotaryArgs &a, F f) {
  auto d = [&](auto pairs) {
    switch (a.d) {
      case 16: return f(std::integral_constant<int, 16>(), pairs);
      case 32: return f(std::integral_constant<int, 32>(), pairs);
      case 64: return f(std::integral_constant<int, 64>(), pairs);
      default: return f(std::integral_constant<int, 128>(), pairs);
    }
  };
  switch (pairs_kind(a)) {
    case kNone: return d(std::integral_constant<int, kNone>());
    case kNeighbours: return d(std::integral_constant<int, kNeighbours>());
    case kHalves: return d(std::integral_constant<int, kHalves>());
    default: return d(std::integral_constant<int, kAnyHalves>());
  }
}
int done() { return cudaPeekAtLastError() == cudaSuccess ? 0 : -1; }

template <typename TIO>
int forward(const RotaryArgs &a, cudaStream_t st) {
  const size_t blocks = ((size_t)a.B * a.T * (a.d / Row<TIO>::VEC) + kFwdBlock - 1) / kFwdBlock;
  if (blocks > 0x7fffffff) return -1;
  // all heads of a token in one thread (its angles serve them all) where that fills the SMs, else fewer
  int heads = a.H + a.Hk;
  while (heads > 4 && blocks * ((a.H + a.Hk + heads - 1) / heads) < 152 * 8) heads = (heads + 1) / 2;
  if (heads <= 4 && blocks * ((a.H + a.Hk + heads - 1) / heads) < 152 * 8) heads = 1;
  return by_pairs(a, [&](auto d, auto p) {
    timing_mark_begin(K_ROTARY, st);
    mesa_qk_norm_rotary_kernel<TIO, decltype(d)::value, decltype(p)::value>
        <<<dim3((unsigned)blocks, (a.H + a.Hk + heads - 1) / heads), kFwdBlock, 0, st>>>(a, heads);
    timing_mark_end(K_ROTARY, st);
    return done();
  });
}
// Two CTAs for each of a GB300's 152 SMs, no more than there are tokens for (d = 128: a CTA takes 16 of bf16, 8 of fp32).
int bwd_parts(int B, int T, int d, int vec) {
  const size_t n = ((size_t)B * T * (d / vec) + kBlock - 1) / kBlock;
  return n < 1 ? 1 : n < 152 * 2 ? (int)n : 152 * 2;
}
template <typename TIO>
int backward(const RotaryArgs &a, cudaStream_t st) {
  const int parts = bwd_parts(a.B, a.T, a.d, Row<TIO>::VEC);
  return by_pairs(a, [&](auto d, auto p) {
    timing_mark_begin(K_ROTARY_BWD, st);
    mesa_qk_norm_rotary_bwd_kernel<TIO, decltype(d)::value, decltype(p)::value><<<parts, kBlock, 0, st>>>(a);
    timing_mark_end(K_ROTARY_BWD, st);
    if (a.partial) {
      timing_mark_begin(K_ROTARY_COLS, st);
      const bool ok = launch_after(mesa_qk_norm_rotary_cols_kernel, (2 * a.d * 32 + kBlock - 1) / kBlock, kBlock, 0, st, a, parts);
      timing_mark_end(K_ROTARY_COLS, st);
      if (!ok) return -1;
    }
    return done();
  });
}

}  // namespace

// (For the workspace, whose size goes by either type: fp32 has more.)
int rotary_bwd_parts(int B, int T, int d) { return bwd_parts(B, T, d, Row<float>::VEC); }

int launch_qk_norm_rotary(const RotaryArgs &a, cudaStream_t st) {
  return a.dtype == 1 ? forward<__nv_bfloat16>(a, st) : forward<float>(a, st);
}
int launch_qk_norm_rotary_backward(const RotaryArgs &a, cudaStream_t st) {
  return a.dtype == 1 ? backward<__nv_bfloat16>(a, st) : backward<float>(a, st);
}

}  // namespace mesa
