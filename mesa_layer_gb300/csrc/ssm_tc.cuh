// ssm_tc.cuh -- what the tensor-core kernels of the selective scan share (bf16, dk = N = 128 and dv = P in {64, 128}, or N =
// P = 64; chunks of L = 128 tokens).
//
// Rows of q, k, v (and of the output's gradient) are bf16 operands as they come from memory.  What is formed on the way
// is rounded to bf16 where only bf16 outputs depend on it (the pairs' weights M, the state as an operand: 2^-9 of a
// term each, as much as the output's own rounding), and to two bf16 values (2^-17) where it enters a state, which is
// fp32 in tensor memory from chunk to chunk.  bf16 has fp32's range, so no scales are needed.  (A third value would take the
// final state's error from 2.3e-6 to 3e-7, near fp32's own 1.2e-7, but eight more products stand in every chunk's chain: us of
// 8 x 16 x 4096 forward 113 to 131, 128 x 64 98 to 111, 64 x 64 89 to 105, 1 x 16 x 65536 293 to 325.  The outputs do not change.
// As a walk of its own over the tokens that a final state still holds: 111 to 127, 175 with heads that hardly forget, 16 x 512
// 20 to 30.  And where heads hardly forget, it is the tensor cores' sums that count, which cut what does not fit.)
// States lie transposed, S^T [dk lanes][dv columns]: the same 128 lanes for every size.  N = 64 uses tiles of 128 columns
// whose second half is zero from the start and stays so (a gradient put there is zero, too): half of the products is
// idle.  64 x 64 states take 80 % of the time of 128 x 128 for half of the bytes: a chunk's chain has the same steps.
#pragma once

#include "gated_delta_tc.cuh"
#include "overlap.cuh"
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

constexpr int L = 128, DK = 128;                      // tokens of a chunk; columns of a q or k tile, lanes of the state
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
__device__ __forceinline__ u64 of_bf2(uint32_t w) { return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t bf2(u64 x) {
  float a, b;
  unpack2(x, a, b);
  return bf2(a, b);
}

// A chunk's gates, one record of floats [U, NC]: for each token the decay from it to the end of its warp's 32 tokens and
// from before them to it (0 across a start), log2 of the latter (R_LO: what its rounding to fp32 left, as bf16: 2^-21 where a
// warp's tokens forget all that they can), the step's length, the last start up to it inside the chunk (a byte, -1: none); then
// the decays from before warp w to ... [w][b]: from the end of warp b's tokens (b < w), FIRST[w]: from
// before the chunk to before warp w, LAST[w]: from the end of warp w to the chunk's end, ALL: across the chunk.
constexpr int R_OUT = 0, R_IN = L, R_LOG = 2 * L, R_STEP = 3 * L, R_START = 4 * L, R_LO = R_START + L / 4, R_BETWEEN = R_LO + L / 2,
              R_FIRST = R_BETWEEN + 16, R_LAST = R_FIRST + 4, R_ALL = R_LAST + 4, REC = R_BETWEEN + 32;
__device__ __forceinline__ int start_of(const float *r, int t) { return reinterpret_cast<const int8_t *>(r + R_START)[t]; }
__device__ __forceinline__ float lo_of(const float *r, int t) { return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(r + R_LO)[t]); }
__device__ __forceinline__ const float *record(const float *records, int u, int NC, int c) {
  return records + ((size_t)u * NC + c) * REC;
}

// Loops over a row's pieces stay loops: unrolled, the parts of a chain's warps do not fit the instruction cache together
// (a third of all cycles went by waiting for instructions).

// Columns 8 c0 .. 8 c1 - 1 of row t of a 128-row tile times w: rounded to bf16 in place, what that leaves as bf16 to `rest`.
__device__ __forceinline__ void weigh_row(uint8_t *tile, uint8_t *rest, int t, float w, int c0, int c1) {
  const u64 w2 = pack2(w, w);
#pragma unroll 2
  for (int c = c0; c < c1; c++) {
    const uint32_t at = tile_off(t, c, L);
    const uint4 x = *reinterpret_cast<const uint4 *>(tile + at);
    uint4 h, r;
    auto one = [w2](uint32_t v, uint32_t &h, uint32_t &r) {
      const u64 p = mul2(of_bf2(v), w2);
      h = bf2(p);
      r = bf2(sub2(p, of_bf2(h)));
    };
    one(x.x, h.x, r.x);
    one(x.y, h.y, r.y);
    one(x.z, h.z, r.z);
    one(x.w, h.w, r.w);
    *reinterpret_cast<uint4 *>(tile + at) = h;
    *reinterpret_cast<uint4 *>(rest + at) = r;
  }
}

// What is not finite in a token's row must not reach the outputs (or gradients) of tokens on the other side of it, but a matrix
// product multiplies it by their zeros.  So the chunks that hold any (rare) have it taken out of the tile (zeros) before the
// product, with a mark for each column from which row, or up to which, the product's column is not finite: NaN is put there after.
constexpr int kNoRow = 128;
__device__ __forceinline__ bool odd_word(uint32_t x) { return (x & 0x7f80u) == 0x7f80u; }  // a bf16 value that is not finite
__device__ __forceinline__ bool odd_words(uint4 x) {
  const uint32_t m = rule::absmax_words(0, x);
  return max(m & 0xffffu, m >> 16) >= 0x7f80u;
}
__device__ __forceinline__ uint16_t *word_at(uint8_t *tile, int row, int column) {
  return reinterpret_cast<uint16_t *>(tile + tile_off(row, column >> 3, L)) + (column & 7);
}

// Columns 32 h0 .. 32 h1 - 1 of lane n of the state in tensor memory (from global memory [P][dk], or zero, where `first`)
// become the operand row n at `op` (nullptr: none), and are multiplied by `all` where they lie.
template <int N>
__device__ __forceinline__ void state_step(uint32_t tS, uint8_t *op, int n, float all, bool first, const float *S0, int h0, int h1) {
  const u64 all2 = pack2(all, all);
#pragma unroll 1
  for (int h = h0; h < h1; h++) {
    float x[32];
    if (first) {
#pragma unroll
      for (int i = 0; i < 32; i++) x[i] = S0 && n < N ? S0[(size_t)(32 * h + i) * N + n] : 0.0f;
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
    for (int i = 0; i < 32; i += 2) unpack2(mul2(pack2(x[i], x[i + 1]), all2), x[i], x[i + 1]);
    tc::tmem_st32(tS + 32 * h, x);
  }
  tc::tmem_st_wait();
}
template <int N>
__device__ __forceinline__ void state_out(uint32_t tS, float *dst, int n, int h0, int h1) {
#pragma unroll 1
  for (int h = h0; h < h1; h++) {
    float x[32];
    tc::tmem_ld32(tS + 32 * h, x);
    tc::tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; i++)
      if (n < N) dst[(size_t)(32 * h + i) * N + n] = x[i];
  }
}

// Zeros where tiles of 64 channels leave theirs, `n` tiles from `tiles` on, by the whole block.
__device__ __forceinline__ void clear_halves(uint8_t *tiles, int n) {
  for (int i = threadIdx.x; i < n * (int)(HALF / 16); i += blockDim.x)
    *reinterpret_cast<uint4 *>(tiles + (i / (HALF / 16)) * QK_TILE + HALF + (i % (HALF / 16)) * 16) = make_uint4(0, 0, 0, 0);
  tc::fence_smem_to_async();
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
  float *records = nullptr;              // [U, NC] the chunks' gates
};

// workspace nullptr: the bytes alone.
SsmSegments ssm_segments(int U, int T, int dv, bool backward, void *workspace, size_t *bytes);

// The backward's workspace: [U, NC] operand tiles of the states before the chunks and the adjoints after them; [3][U, 4 NC]
// sums for the parameters; per-unit dq, dk [U, T, dk] (nullptr when every head has its own q, k).
struct SsmTcBwd {
  uint8_t *S, *R;
  float *sums, *dqp, *dkp;
};
int launch_ssm_gates(const SsmArgs &a, const SsmSegments &sg, cudaStream_t st);
int launch_ssm_chains_tc(const SsmArgs &a, const SsmSegments &sg, const SsmTcBwd &ws, cudaStream_t st);

}  // namespace mesa
