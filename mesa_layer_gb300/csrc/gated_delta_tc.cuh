// gated_delta_tc.cuh -- what the tensor-core kernels of the gated delta rule share (bf16,
// dk = dv = 128, chunks of 64 tokens).
//
// A chunk's algebra, rows = tokens, S0 the state before it, D_ij the decay from token j to i,
// f_i the decay from the chunk's start to i, c_j from j to its end:
//     (I + A) U = diag(beta) (V - diag(f) K S0^T),   A = diag(beta) (K K^T o D), strictly lower,
//     O = scale (diag(f) Q S0^T + (Q K^T o D) U),    S = f_last S0 + (diag(c) U)^T K.
// (I + A) is unit lower triangular: its inverse comes from substitution, which keeps the
// accuracy of the recurrence (powers of A would cancel).
//
// Operands of the matrix products are fp16 with power-of-two scales, accumulated in fp32: q
// and k are bf16, exact in fp16 but for elements 2^14 below their tile's largest; states, u and
// the triangular factors are rounded to 2^-12 relative to their row's largest element, well
// inside the 2^-9 of the bf16 outputs.  The states themselves stay fp32 in registers, so
// the operand rounding of one chunk is not carried on but as an input error.
#pragma once

#include "common.cuh"
#include "gated_delta.h"
#include "launch.h"
#include "packed.cuh"
#include "tc_common.cuh"

namespace mesa {
namespace rule {

constexpr int C = 64, D = 128;               // tokens per chunk; dk = dv
constexpr uint32_t TILE = 2 * C * D * 2;     // fp16 [128 x 128] operand: K rows, then Q rows
constexpr uint32_t SQ = C * C * 2;           // fp16 [64 x 64] operand
constexpr uint32_t ROWS64 = C * D * 2;       // 64 bf16 rows
// A chunk's record in the workspace: the factor T or T diag(beta) and P = (Q K^T o D), both as
// swizzled K-major operands, then f and c.
constexpr uint32_t REC_P = SQ, REC_F = 2 * SQ, REC_C = REC_F + 4 * C, REC = REC_C + 4 * C;
static_assert(REC % 128 == 0, "records are bulk copied");

// Operand scale of a tile with largest element m: a power of two with m s in (0.5, 1], limited
// so that its square stays finite.
__device__ __forceinline__ float tile_scale(float m) {
  return fminf(fmaxf(tc::rcp_pow2_ceil(m), 8.6736174e-19f), 1.1529215e18f);  // 2^-60 .. 2^60
}

// Eight bf16 values times s as fp16.
__device__ __forceinline__ uint4 to_half8(uint4 raw, u64 s2) {
  const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const u64 x = mul2(pack2(__uint_as_float(in[i] << 16), __uint_as_float(in[i] & 0xffff0000u)), s2);
    float a, b;
    unpack2(x, a, b);
    const __half2 h = __floats2half2_rn(a, b);
    out[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}
__device__ __forceinline__ float absmax8(uint4 raw) {  // largest |x| of eight bf16 values
  const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; i++)
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(in[i] << 16)), fabsf(__uint_as_float(in[i] & 0xffff0000u))));
  return m;
}
__device__ __forceinline__ float half2_bits(float a, float b) {  // two fp16 values as a 32-bit register
  const __half2 h = __floats2half2_rn(a, b);
  return __uint_as_float(*reinterpret_cast<const uint32_t *>(&h));
}

// Offset in a swizzled K-major [rows x 128] fp16 tile of the 16 bytes holding columns
// 8 c8 .. 8 c8 + 7 of row r.
__device__ __forceinline__ uint32_t tile_off(int r, int c8, int rows) { return tc::sw128_offset(r, 8 * c8, rows); }

// Barrier of the first `n` arriving threads of group `id`, with the OR of their flags.
__device__ __forceinline__ bool group_or(int id, int n, bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)flag), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// Untiled bulk copy of this CTA's shared memory to global memory (both 16-byte aligned).
__device__ __forceinline__ void bulk_s2g(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n" ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
// Bounded wait that also gives up when another warp of the CTA has (its limit is then not
// waited for twice).
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, unsigned limit, const volatile int *gave_up) {
  for (unsigned i = 0; i < limit; i++) {
    if (tc::mbar_wait(bar, parity, 1)) return true;
    if (*gave_up) return false;
  }
  return false;
}

// Decays of a chunk's tokens in log2, with closed gates counted apart: the decay from token j
// to token i >= j is 2^(l_i - l_j) if z_i = z_j, else 0.  Lane l of a whole warp handles
// tokens 2l and 2l + 1; gates past the end are 1.  Gates below e^-80 count as closed.
struct GatePair {
  float l0, l1;
  int z0, z1;
};
__device__ __forceinline__ GatePair gate_scan(const float *gamma, int n, int lane) {
  const float ga = 2 * lane < n ? gamma[2 * lane] : 1.0f, gb = 2 * lane + 1 < n ? gamma[2 * lane + 1] : 1.0f;
  const bool sa = ga < 1.8048514e-35f, sb = gb < 1.8048514e-35f;
  const float a = sa ? 0.0f : log2f(ga), b = sb ? 0.0f : log2f(gb);
  float l = a + b;
  int z = (int)sa + (int)sb;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float pl = __shfl_up_sync(0xffffffffu, l, o);
    const int pz = __shfl_up_sync(0xffffffffu, z, o);
    if (lane >= o) {
      l += pl;
      z += pz;
    }
  }
  return GatePair{l - b, l, z - (int)sb, z};
}

// Workspace of the tensor-core forward: records and operand scales {s_k, s_q} of every chunk.
struct TcWorkspace {
  uint8_t *rec;     // [U, NC] records
  float2 *scales;   // [U, NC]
};

}  // namespace rule
}  // namespace mesa
