// ssm_tc.cuh -- what the tensor-core kernels of the selective scan share (bf16, dk = 128, dv = P in {64, 128}, chunks of
// L = 128 tokens).
//
// Rows of q, k, v (and of the output's gradient) are bf16 operands as they come from memory.  What is formed on the way
// is rounded to bf16 where only bf16 outputs depend on it (the pairs' weights M, the state as an operand: 2^-9 of a
// term each, as much as the output's own rounding), and to two bf16 values (2^-17) where it enters a state, which is
// fp32 in tensor memory from chunk to chunk.  bf16 has fp32's range, so no scales are needed.
// States lie transposed, S^T [dk lanes][dv columns]: the same 128 lanes for either dv.
#pragma once

#include "gated_delta_tc.cuh"
#include "ssm.h"
#include "ssm_common.cuh"

namespace mesa {
namespace ssm {

using rule::elect_one;
using rule::group_or;
using rule::mbar_arrive;
using rule::step128;
using rule::step_mn;
using rule::tensor_g2s_3d;
using rule::tensor_s2g_3d;
using rule::tile_off;
using rule::wait;

constexpr int L = 128, DK = 128;
constexpr uint32_t QK_TILE = L * DK * 2;              // 128 rows of 128 bf16: two halves of 64 columns
constexpr uint32_t HALF = L * 64 * 2;
template <int P>
constexpr uint32_t V_TILE = L * P * 2;

// Instruction descriptor: bf16 operands, fp32 sums.
__device__ __forceinline__ uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return tc::idesc_f16(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);
}
__device__ __forceinline__ uint32_t bf2(float a, float b) {  // two bf16 values, a in the low half
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&x);
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A token's gates inside its chunk, thread t of a group of 128: its step; its log2 decay from the chunk's start and from
// its warp's first token's; the last start up to it (-1: none in the chunk).
struct Token {
  float step;
  Two l, local;
  int s;
  Two before, end;  // log2 decay from the chunk's start to before the warp's first token, to the chunk's end
  int s_warp, s_end;  // the last start in the warp's tokens and before, in the chunk
};
struct WarpTotals {
  float hi[4], lo[4];
  int s[4];
};
struct TokenIn {
  float raw;
  bool start;
};
// Token t0 + t of unit u (past the end: nothing is forgotten, nothing written).
__device__ __forceinline__ TokenIn token_load(const SsmArgs &a, int u, int t) {
  TokenIn x = {-INFINITY, false};
  if (t < a.T) {
    x.raw = a.dt[(size_t)u * a.T + t];
    x.start = a.starts && a.starts[(size_t)(u / a.H) * a.T + t];
  }
  return x;
}
// group: named barrier of the 128 threads; true when one of them gave up.  `tot` is another one in the next call.
__device__ __forceinline__ bool token_gates(Token &g, TokenIn in, float bias, float A, WarpTotals &tot, int t, int group, bool ok) {
  const int lane = t & 31, w = t >> 5;
  g.step = softplus(in.raw + bias);
  Two l = in.start ? Two{0.0f, 0.0f} : log2_decay(g.step, A);
  int s = in.start ? t : -1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two p = {__shfl_up_sync(0xffffffffu, l.hi, o), __shfl_up_sync(0xffffffffu, l.lo, o)};
    const int ps = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) {
      l = two_add(p, l);
      s = max(s, ps);
    }
  }
  if (lane == 31) tot.hi[w] = l.hi, tot.lo[w] = l.lo, tot.s[w] = s;
  const bool stop = group_or(group, 128, !ok);
  g.local = l;
  g.before = Two{0.0f, 0.0f};
  g.s = s;
  g.s_warp = -1;
  Two sum = {0.0f, 0.0f};
  int last = -1;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if (i == w) g.before = sum, g.s = max(g.s, last);
    sum = two_add(sum, Two{tot.hi[i], tot.lo[i]});
    last = max(last, tot.s[i]);
    if (i == w) g.s_warp = last;
  }
  g.l = two_add(g.before, l);
  g.end = sum;
  g.s_end = last;
  return stop;
}
__device__ __forceinline__ float exp2_of(Two x) { return exp2f(x.hi + x.lo); }

// Row t of a 128-row tile of 128 columns times w: rounded to bf16 in place, what that leaves as bf16 pairs in `rest`.
__device__ __forceinline__ void weigh_row(uint8_t *tile, int t, float w, uint4 (&rest)[16]) {
#pragma unroll
  for (int c = 0; c < 16; c++) {
    uint4 *at = reinterpret_cast<uint4 *>(tile + tile_off(t, c, L));
    const uint4 x = *at;
    auto one = [w](uint32_t v, uint32_t &r) {
      const float a = lo_of(v) * w, b = hi_of(v) * w;
      const uint32_t h = bf2(a, b);
      r = bf2(a - lo_of(h), b - hi_of(h));
      return h;
    };
    *at = make_uint4(one(x.x, rest[c].x), one(x.y, rest[c].y), one(x.z, rest[c].z), one(x.w, rest[c].w));
  }
}
__device__ __forceinline__ void put_row(uint8_t *tile, int t, const uint4 (&x)[16]) {
#pragma unroll
  for (int c = 0; c < 16; c++) *reinterpret_cast<uint4 *>(tile + tile_off(t, c, L)) = x[c];
}

// Lane n's P columns of the state in tensor memory (from global memory [P][dk], or zero, where `first`) become the
// operand row n at `op` (nullptr: none), and are multiplied by `all` where they lie.
template <int P>
__device__ __forceinline__ void state_step(uint32_t tS, uint8_t *op, int n, float all, bool first, const float *S0) {
#pragma unroll
  for (int h = 0; h < P / 32; h++) {
    float x[32];
    if (first) {
#pragma unroll
      for (int i = 0; i < 32; i++) x[i] = S0 ? S0[(size_t)(32 * h + i) * DK + n] : 0.0f;
    } else {
      tc::tmem_ld32(tS + 32 * h, x);
      tc::tmem_ld_wait();
    }
    if (op) {
#pragma unroll
      for (int c = 0; c < 4; c++)
        *reinterpret_cast<uint4 *>(op + tile_off(n, 4 * h + c, L)) =
            make_uint4(bf2(x[8 * c], x[8 * c + 1]), bf2(x[8 * c + 2], x[8 * c + 3]), bf2(x[8 * c + 4], x[8 * c + 5]),
                       bf2(x[8 * c + 6], x[8 * c + 7]));
    }
#pragma unroll
    for (int i = 0; i < 32; i++) x[i] = all == 0.0f ? 0.0f : x[i] * all;  // (a start: nothing of it is left)
    tc::tmem_st32(tS + 32 * h, x);
  }
  tc::tmem_st_wait();
}
template <int P>
__device__ __forceinline__ void state_out(uint32_t tS, float *dst, int n) {
#pragma unroll
  for (int h = 0; h < P / 32; h++) {
    float x[32];
    tc::tmem_ld32(tS + 32 * h, x);
    tc::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; i++) dst[(size_t)(32 * h + i) * DK + n] = x[i];
  }
}

// The halves of 64 channels of 128 tokens' rows of unit z, from token y on.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const void *map, int y, int z, uint32_t bar) {
#pragma unroll
  for (int h = 0; h < D / 64; h++) tensor_g2s_3d(dst + h * HALF, map, 64 * h, y, z, bar);
}

}  // namespace ssm

// Long sequences of few units: n segments of `per` chunks that run side by side.
struct SsmSegments {
  int n = 1, per = 0;
  float *S = nullptr, *decay = nullptr;  // [U, n][dv, dk] what a segment leaves, then the state before it; [U, n]
  float *R = nullptr;                    // the same of the adjoint
};

}  // namespace mesa
