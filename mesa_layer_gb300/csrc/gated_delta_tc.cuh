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
// Operands of the matrix products are fp16 with power-of-two scales, sums are fp32: q and k are
// bf16, exact in fp16 but for elements 2^16 below their tile's largest; the state, R, U and the
// factors are rounded to 2^-12, well inside the 2^-9 of the bf16 outputs (bf16 operands would
// double the output's error).  Row scales come from bounds rather than from the largest
// element: fp16 covers 2^29 in full precision, so a bound 2^15 above the values costs nothing.
// The state itself stays fp32 in registers, so a chunk's operand rounding enters the next
// one only through u.  The inverse is formed in fp32 (diagonal blocks) and from fp16 blocks with
// fp32 sums (the rest), A's blocks as two fp16 values each: where keys are alike the inverse is a small sum of
// large products of A's entries (keys of cosine 0.9, beta 1 to 2: rounded once they cost T 2.4e-3, so 5e-4; its
// other roundings cost 2e-4).
#pragma once

#include "common.cuh"
#include "gated_delta.h"
#include "launch.h"
#include "packed.cuh"
#include "tc_common.cuh"

namespace mesa {
namespace rule {

constexpr int C = 64, D = 128;               // tokens per chunk; dk = dv
constexpr uint32_t TILE = 2 * C * D * 2;     // [128 x 128] operand: K rows, then Q rows
constexpr uint32_t SQ = C * C * 2;           // [64 x 64] operand
constexpr uint32_t ROWS64 = C * D * 2;       // 64 rows of bf16
// A chunk's record: the factor T or T diag(beta) and P = Q K^T o D, swizzled K-major operands, then
// minus f, c, beta, and {1 / scale of K, of Q, scale of K, of Q; a power of two that no decay in the chunk
// exceeds (1 but for gates above one), 1 / it: P is times that}.  REC_PAD: its place in shared memory.
constexpr uint32_t REC_P = SQ, REC_F = 2 * SQ, REC_C = REC_F + 4 * C, REC_B = REC_C + 4 * C, REC_S = REC_B + 4 * C,
                   REC = REC_S + 128, REC_PAD = 18 * 1024;
static_assert(REC % 16 == 0 && REC <= REC_PAD, "records are bulk copied");
__device__ __forceinline__ float half2_bits(float a, float b) {  // two fp16 values as a 32-bit register
  const __half2 h = __floats2half2_rn(a, b);
  return __uint_as_float(*reinterpret_cast<const uint32_t *>(&h));
}
__device__ __forceinline__ float half2_bits(u64 x) {
  float a, b;
  unpack2(x, a, b);
  return half2_bits(a, b);
}
// The power of two s with 2^(top-1) < bound s < 2^top (bound taken as at least 2^-63 and at most
// 2^63), and 1 / s.
__device__ __forceinline__ float bound_scale(float bound, int top, float &inv) {
  const int e = min(max((int)(__float_as_uint(bound) >> 23), 64), 190);
  inv = __uint_as_float((uint32_t)(e + 1 - top) << 23);
  return __uint_as_float((uint32_t)(253 + top - e) << 23);
}
constexpr int kTopRow = 15;   // state rows, R and U rows: bound to 2^15
constexpr float kLittle = -40.0f;  // log2 of what is left of a state at the end of a segment's tail
constexpr float kMostGrowth = 8.0f;  // log2 of what a chunk's gates above one multiply to, at most
constexpr int kTopTile = 3;   // K and Q tiles: 128 products of two stay below 2^13
// Largest |x| of 2 x 16-bit bf16 words, as an integer (the order of positive floats is theirs).
__device__ __forceinline__ uint32_t absmax_words(uint32_t m, uint4 x) {
  constexpr uint32_t k = 0x7fff7fffu;
  return __vimax3_u16x2(__vimax3_u16x2(m, x.x & k, x.y & k), x.z & k, x.w & k);
}
__device__ __forceinline__ uint32_t absmax_fold(uint32_t m) {  // over the two halves and the warp
  m = max(m & 0xffffu, m >> 16);
  return __reduce_max_sync(0xffffffffu, m);
}
// Eight bf16 values times s as fp16.
__device__ __forceinline__ uint4 to_half8(uint4 raw, u64 s2) {
  auto two = [s2](uint32_t w) {
    return __float_as_uint(half2_bits(mul2(pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), s2)));
  };
  return make_uint4(two(raw.x), two(raw.y), two(raw.z), two(raw.w));
}
// Tiled load of a box of a 3-D tensor map (channel x, token y, unit z); tokens past the end
// read as zero.
__device__ __forceinline__ void tensor_g2s_3d(uint32_t dst, const void *map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Offset in a swizzled K-major [rows x 128] 16-bit tile of the 16 bytes holding columns
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
// tokens 2l and 2l + 1 (gates past the end: 1).  Gates below e^-80 count as closed; a negative one has no
// logarithm (NaN, and so is all that it decays).
struct GatePair {
  float l0, l1;
  int z0, z1;
};
__device__ __forceinline__ GatePair gate_scan(float2 gamma, int lane) {
  const bool sa = fabsf(gamma.x) < 1.8048514e-35f, sb = fabsf(gamma.y) < 1.8048514e-35f;
  const float a = sa ? 0.0f : log2f(gamma.x), b = sb ? 0.0f : log2f(gamma.y);
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

// 2^x (a PTX instruction; 2^-22 relative error).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B of one 16 x 8 x 16 product (fp16 operands, fp32 sums): the blocks of the triangular
// inverse, too small and too sequential for the 128-row products.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One lane of a converged warp.  The products' operands are warp-uniform registers: behind a plain
// thread test (not this, under a warp-uniform condition) each product took 130 cycles to issue,
// whatever its size; so, 56 (N = 64) to 74 (N = 128).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}\n" : "=r"(p));
  return p != 0;
}
// K-step s of 16 added to a K-major descriptor of a 128-row tile, of a 64-row tile with 64 columns, and
// to an MN-major one, in the descriptor's 16-byte units.
__device__ __forceinline__ uint64_t step128(int s) { return (uint64_t)((s >> 2) * 1024 + (s & 3) * 2); }
__device__ __forceinline__ uint64_t step64(int s) { return (uint64_t)(2 * s); }
__device__ __forceinline__ uint64_t step_mn(int s) { return (uint64_t)(128 * s); }

// Register shares of warp groups (setmaxnreg; a whole group of four warps).
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
// 64 columns of 16 tensor-memory lanes as 8-column fragments: for columns 8 j .. 8 j + 7 this thread gets
// lane T / 4, columns 2 (T % 4) and the next, in r[4 j], r[4 j + 1]; lane T / 4 + 8 in the next two.
__device__ __forceinline__ void tmem_ld_frag64(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}
// Four 8 x 8 blocks of 16-bit fragments to shared memory, transposed: lane l gives the address of row
// l % 8 (the fragments' column) of block l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// The same of 16 columns, pairs together: v[2 j + e] is lane T / 4 + 8 e, columns 8 j + 2 (T % 4) and the next.
__device__ __forceinline__ void tmem_ld_frag16(uint32_t taddr, u64 (&v)[4]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 4; i++) v[i] = (u64)r[2 * i] | (u64)r[2 * i + 1] << 32;
}
// 8 x 8 blocks of 16-bit fragments to shared memory (lane l % 8: row of block l / 8), one of them also transposed.
__device__ __forceinline__ void stmatrix_x4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void stmatrix_x1(uint32_t addr, uint32_t a) {
  asm volatile("stmatrix.sync.aligned.m8n8.x1.shared.b16 [%0], {%1};\n" ::"r"(addr), "r"(a) : "memory");
}
__device__ __forceinline__ void stmatrix_x1_trans(uint32_t addr, uint32_t a) {
  asm volatile("stmatrix.sync.aligned.m8n8.x1.trans.shared.b16 [%0], {%1};\n" ::"r"(addr), "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t a) {  // an 8 x 8 block of fragments
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
  return d;
}
// Tiled store of a box of a 3-D tensor map; tokens past the end are not written.
__device__ __forceinline__ void tensor_s2g_3d(const void *map, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];\n" ::"l"(map), "r"(src),
               "r"(x), "r"(y), "r"(z)
               : "memory");
}

// ---- the factors of a chunk, by 128 threads ------------------------------------------------------
struct Factor {
  __half Ah[C - 16][56]; // A's blocks below the diagonal, fp16 (from row 16 on; the rest of it: factor_rows)
  float Ad[C][20];       // its diagonal 16 x 16 blocks: row i, columns of block i / 16
  __half Tb[4][16][24];  // inverses of the diagonal blocks of I + A, and their transposes
  __half Yb[4][16][24];
  float l[C], beta[C];
  int z[C];
};
// Decays from the gates of one warp's scan: l, z, minus f (chunk start to token) and c (token to
// end); most[0] a power of two that none exceeds (all gates above one together; 64 gates of up to 2^0.001
// stay inside the scales' factor of two), most[1] 1 / it.  The scales take it into account, up to 2^8: three
// such bounds multiply in the backward's operands, whose fp16 range is 2^29 (growth of 2^8 in a chunk costs no
// accuracy, 2^10 up to 2e-2 of a gradient).  What grows more has no decays: NaN, and is reported.
__device__ __forceinline__ void factor_gates(Factor &s, GatePair g, float *nf, float *c, float *most, int lane) {
  const float before = __shfl_up_sync(0xffffffffu, g.l1, 1), up0 = g.l0 - (lane > 0 ? before : 0.0f), up1 = g.l1 - g.l0;
  const float up = (up0 > 0.001f ? up0 : 0.0f) + (up1 > 0.001f ? up1 : 0.0f);
  int e = 0;
  if (__any_sync(0xffffffffu, up > 0.0f)) {
    const float all = warp_sum(up);
    e = (int)ceilf(fminf(all, kMostGrowth));
    if (!(all <= kMostGrowth)) g.l0 = g.l1 = NAN;
  }
  if (lane == 0)
    *reinterpret_cast<float2 *>(most) =
        make_float2(__uint_as_float((uint32_t)(127 + e) << 23), __uint_as_float((uint32_t)(127 - e) << 23));
  const float end = __shfl_sync(0xffffffffu, g.l1, 31);
  const int zend = __shfl_sync(0xffffffffu, g.z1, 31);
  *reinterpret_cast<float2 *>(&s.l[2 * lane]) = make_float2(g.l0, g.l1);
  *reinterpret_cast<int2 *>(&s.z[2 * lane]) = make_int2(g.z0, g.z1);
  *reinterpret_cast<float2 *>(nf + 2 * lane) = make_float2(g.z0 == 0 ? -ex2(g.l0) : 0.0f, g.z1 == 0 ? -ex2(g.l1) : 0.0f);
  *reinterpret_cast<float2 *>(c + 2 * lane) =
      make_float2(g.z0 == zend ? ex2(end - g.l0) : 0.0f, g.z1 == zend ? ex2(end - g.l1) : 0.0f);
}
// Thread `tid` (warp w reads tensor-memory lanes 32 w ..): row tid of [K K^T; Q K^T] at tensor
// memory `t`, in operand units (inv_kk: 1 / scale of K, squared).  Rows of A go to s, what their fp16 values
// leave of block (b, k) to block (k, b) of M, which is not used yet; rows of P,
// still in operand units (times p_unit), to the swizzled operand P.  Columns
// right of the diagonal's 32 are skipped.
__device__ __forceinline__ void factor_rows(Factor &s, uint32_t t, float inv_kk, float p_unit, uint8_t *M, uint8_t *P, int tid) {
  const int warp = tid >> 5, i = tid & 63;
  const bool isA = tid < C, low = i >= 32;  // (uniform in a warp)
  const float li = s.l[i], mul = isA ? s.beta[i] * inv_kk : p_unit;
  const int zi = s.z[i], last = isA ? i - 1 : i;  // last column kept
  const bool cut = s.z[C - 1] != 0;                       // a closed gate in the chunk
  const uint32_t tl = t + ((uint32_t)(32 * warp) << 16);
  const u64 li2 = pack2(li, li), mul2x = pack2(mul, mul);
  const int diag = i >> 4;  // the row's diagonal block
  float w[2][16];
  tc::tmem_ld16(tl, w[0]);
#pragma unroll
  for (int h = 0; h < 4; h++) {  // columns 16 h .., the next ones on their way
    if (h >= 2 && !low) break;
    float *v = w[h & 1];
    ulonglong2 lj[4];
#pragma unroll
    for (int k = 0; k < 4; k++) lj[k] = *reinterpret_cast<const ulonglong2 *>(&s.l[16 * h + 4 * k]);
    u64 dec[8];
#pragma unroll
    for (int k = 0; k < 8; k++) {
      float x, y;
      unpack2(sub2(li2, k & 1 ? lj[k / 2].y : lj[k / 2].x), x, y);
      dec[k] = mul2(pack2(ex2(x), ex2(y)), mul2x);
    }
    tc::tmem_ld_wait();
    if (h < 1 || (h < 3 && low)) tc::tmem_ld16(tl + 16 * (h + 1), w[(h + 1) & 1]);
#pragma unroll
    for (int k = 0; k < 8; k++) unpack2(mul2(pack2(v[2 * k], v[2 * k + 1]), dec[k]), v[2 * k], v[2 * k + 1]);
    const int keep = last - 16 * h;
    if (h >= (low ? 2 : 0)) {
#pragma unroll
      for (int k = 0; k < 16; k++)
        if (k > keep) v[k] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const float4 o = make_float4(half2_bits(v[8 * k], v[8 * k + 1]), half2_bits(v[8 * k + 2], v[8 * k + 3]),
                                   half2_bits(v[8 * k + 4], v[8 * k + 5]), half2_bits(v[8 * k + 6], v[8 * k + 7]));
      if (!isA)
        *reinterpret_cast<float4 *>(P + tile_off(i, 2 * h + k, C)) = o;
      else if (h < diag) {
        *reinterpret_cast<float4 *>(&s.Ah[i - 16][16 * h + 8 * k]) = o;
        auto rest = [&](int e, float bits) {
          const uint32_t w = __float_as_uint(bits);
          const float2 hi = __half22float2(*reinterpret_cast<const __half2 *>(&w));
          return half2_bits(v[8 * k + e] - hi.x, v[8 * k + e + 1] - hi.y);
        };
        *reinterpret_cast<float4 *>(M + tile_off(16 * h + (i & 15), 2 * diag + k, C)) =
            make_float4(rest(0, o.x), rest(2, o.y), rest(4, o.z), rest(6, o.w));
      }
    }
    if (isA && h == diag) {  // its part of the diagonal block, in fp32
#pragma unroll
      for (int k = 0; k < 4; k++)
        *reinterpret_cast<float4 *>(&s.Ad[i][4 * k]) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
    }
  }
  if (cut) {  // rare: the entries across a closed gate, in the stored rows
#pragma unroll 1
    for (int j = 0; j < i; j++) {
      if (s.z[j] == zi) continue;
      if (isA) {
        if (j >> 4 == diag) {
          s.Ad[i][j & 15] = 0.0f;
        } else {
          s.Ah[i - 16][j] = __float2half_rn(0.0f);
          *reinterpret_cast<uint16_t *>(M + tc::sw128_offset((j & ~15) + (i & 15), 16 * diag + (j & 15), C)) = 0;
        }
      } else {
        *reinterpret_cast<uint16_t *>(P + tc::sw128_offset(i, j, C)) = 0;
      }
    }
  }
}
// Warp w < 4: the inverse of diagonal block w by substitution in fp32 (lane = column, twice), to
// s and to the swizzled operand M, columns times b (1 or beta).
template <bool WITH_BETA>
__device__ __forceinline__ void factor_diagonal(Factor &s, uint8_t *M, int w, int lane) {
  const int col = lane & 15;
  const float b = WITH_BETA ? s.beta[16 * w + col] : 1.0f;
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; i++) {
    float x[2] = {i == col ? 1.0f : 0.0f, 0.0f};
#pragma unroll
    for (int j4 = 0; j4 < i; j4 += 4) {
      const float4 a = *reinterpret_cast<const float4 *>(&s.Ad[16 * w + i][j4]);
      x[0] = fmaf(-a.x, t[j4], x[0]);
      if (j4 + 1 < i) x[1] = fmaf(-a.y, t[j4 + 1], x[1]);
      if (j4 + 2 < i) x[0] = fmaf(-a.z, t[j4 + 2], x[0]);
      if (j4 + 3 < i) x[1] = fmaf(-a.w, t[j4 + 3], x[1]);
    }
    t[i] = x[0] + x[1];
  }
  if (lane < 16) {
#pragma unroll
    for (int i = 0; i < 16; i++) {
      s.Tb[w][i][col] = __float2half_rn(t[i]);
      *reinterpret_cast<__half *>(M + tc::sw128_offset(16 * w + i, 16 * w + col, C)) = __float2half_rn(t[i] * b);
    }
  } else {
    __align__(16) float y[8];
#pragma unroll
    for (int k = 0; k < 8; k++) y[k] = half2_bits(t[2 * k], t[2 * k + 1]);
    *reinterpret_cast<float4 *>(&s.Yb[w][col][0]) = *reinterpret_cast<const float4 *>(y);
    *reinterpret_cast<float4 *>(&s.Yb[w][col][8]) = *reinterpret_cast<const float4 *>(y + 4);
  }
}
// Warp c < 4: the blocks of column block c below the diagonal, downwards,
//     T_bc = -T_bb sum_{k = c .. b-1} A_bk T_kc,
// in transposed form Y_cb = T_bc^T: a product's sums are then the next one's operand as they lie in
// the registers.
template <bool WITH_BETA>
__device__ __forceinline__ void factor_columns(Factor &s, uint8_t *M, int c, int lane) {
  const int g = lane >> 2, q = 2 * (lane & 3);
  const float be0 = WITH_BETA ? s.beta[16 * c + g] : 1.0f, be1 = WITH_BETA ? s.beta[16 * c + g + 8] : 1.0f;
  uint32_t y[4][4];
  auto word = [](const __half *p) { return *reinterpret_cast<const uint32_t *>(p); };
  auto pack = [](float a, float b) { return __float_as_uint(half2_bits(a, b)); };
#pragma unroll
  for (int b = 0; b < 4; b++) {
    if (b == c) {
      y[b][0] = word(&s.Yb[b][g][q]);
      y[b][1] = word(&s.Yb[b][g + 8][q]);
      y[b][2] = word(&s.Yb[b][g][q + 8]);
      y[b][3] = word(&s.Yb[b][g + 8][q + 8]);
    } else if (b > c) {
      float z0[4] = {}, z1[4] = {};
      auto rest = [&](int k, int row, int col) {  // of A's block (b, k)
        return *reinterpret_cast<const uint32_t *>(M + tc::sw128_offset(16 * k + row, 16 * b + col, C));
      };
#pragma unroll
      for (int k = 0; k < b; k++) {
        if (k < c) continue;
        mma_16816(z0, y[k], rest(k, g, q), rest(k, g, q + 8));
        mma_16816(z1, y[k], rest(k, g + 8, q), rest(k, g + 8, q + 8));
        mma_16816(z0, y[k], word(&s.Ah[16 * b - 16 + g][16 * k + q]), word(&s.Ah[16 * b - 16 + g][16 * k + q + 8]));
        mma_16816(z1, y[k], word(&s.Ah[16 * b - 8 + g][16 * k + q]), word(&s.Ah[16 * b - 8 + g][16 * k + q + 8]));
      }
      const uint32_t za[4] = {pack(-z0[0], -z0[1]), pack(-z0[2], -z0[3]), pack(-z1[0], -z1[1]), pack(-z1[2], -z1[3])};
      float w0[4] = {}, w1[4] = {};
      mma_16816(w0, za, word(&s.Tb[b][g][q]), word(&s.Tb[b][g][q + 8]));
      mma_16816(w1, za, word(&s.Tb[b][g + 8][q]), word(&s.Tb[b][g + 8][q + 8]));
      y[b][0] = pack(w0[0], w0[1]);
      y[b][1] = pack(w0[2], w0[3]);
      y[b][2] = pack(w1[0], w1[1]);
      y[b][3] = pack(w1[2], w1[3]);
      auto put = [&](int row, int col, float t) {
        *reinterpret_cast<__half *>(M + tc::sw128_offset(16 * b + row, 16 * c + col, C)) = __float2half_rn(t);
      };
#pragma unroll
      for (int e = 0; e < 2; e++) {
        put(q + e, g, w0[e] * be0);
        put(q + e, g + 8, w0[2 + e] * be1);
        put(q + 8 + e, g, w1[e] * be0);
        put(q + 8 + e, g + 8, w1[2 + e] * be1);
      }
    }
  }
}
// What lies above the 32-column halves of P is never written: cleared once by 128 threads.
__device__ __forceinline__ void factor_clear(uint8_t *P, int tid) {
  for (int i = tid; i < (int)(SQ / 16); i += 128) reinterpret_cast<uint4 *>(P)[i] = make_uint4(0, 0, 0, 0);
}
// M above its diagonal blocks, once A's rests there have been read.
__device__ __forceinline__ void factor_clear_upper(uint8_t *M, int tid) {
  for (int i = tid; i < 8 * (C - 16); i += 128) {
    const int r = i >> 3, c8 = i & 7;
    if (c8 >= 2 * (r >> 4) + 2) *reinterpret_cast<uint4 *>(M + tile_off(r, c8, C)) = make_uint4(0, 0, 0, 0);
  }
}

}  // namespace rule
}  // namespace mesa
