// gated_delta_tc.cu -- the gated delta rule's chunked forward on the tensor cores (bf16,
// dk = dv = 128; the chunk algebra and the operand formats are in gated_delta_tc.cuh).
//
// One CTA per unit walks the unit's chunks with the state in registers (thread r of the chain
// holds row r, 128 values) and everything laid out by state row, so that a chunk's chain of
// dependent products never crosses threads:
//     D1 = S0 K^T          -> R = V^T - f D1      (row r of the accumulator is thread r's)
//     D2 = R (T beta)^T    -> U
//     dS = (c U) K         -> S = f_last S0 + dS
// with S0, R and U written back to tensor memory as the next product's A operand.  The readout
// O = f (S0 Q^T) + U P^T shares the first product (K and Q rows are one operand tile).  The chain
// bounds the kernel, so all else runs beside it, in warp groups of their own:
//     chain    the three epilogues above;
//     helper   transposes V one chunk ahead, writes the readout of the chunk before;
//     factor   decays, masks and the triangular inverse, one chunk ahead;
//     convert  K and Q as fp16 operands, up to three chunks ahead.
// Each group's first thread issues the products that the group itself waits for.
// The inputs are read once and the output written once; nothing else goes to memory.
#include "gated_delta_tc.cuh"

namespace mesa {

using namespace rule;

namespace {

// shared memory: three K, Q operand tiles | two slots of factors M, P | V^T in fp32 | V | output |
// factor scratch | misc
constexpr uint32_t CH_TILE = 0, CH_FAC = CH_TILE + 3 * TILE, CH_VT = CH_FAC + 4 * SQ, CH_V = CH_VT + 2 * ROWS64;
constexpr uint32_t CH_OUT = CH_V + ROWS64, CH_SCR = CH_OUT + ROWS64;
constexpr uint32_t CH_MISC = CH_SCR + ((sizeof(Factor) + 127) & ~127u);
struct ChainMisc {
  float o1[2][D], o2[2][D];     // units of the readout's accumulators, by state row
  float nf[4][C], c[4][C];    // minus the decays from the chunk's start; those to its end
  float inv_k[3], inv_q[3];   // 1 / operand scales, by tile
  float vmax[4];              // largest |v| of 32 channels
  alignas(16) uint32_t red[16];
  uint64_t tile_full[3], tile_free[3], v_full, vt_full, d0_full, fac_full[2], r_ready, u_ready, o_free;
  uint64_t mma1, mma2, mma3, mma4[2], drain;
  uint32_t tmem;
  int gave_up;
};
constexpr uint32_t CH_SMEM = CH_MISC + sizeof(ChainMisc) + 1024;
static_assert(CH_SMEM <= 232448, "shared memory per block");
// tensor memory columns: dS | S0 operand | D1 (then R, c U and U), O from S0 | D2 | O from U |
// [K K^T; Q K^T]
constexpr uint32_t T_DS = 0, T_S = 128, T_D1 = 192, T_O1 = 256, T_D2 = 320, T_O2 = 384, T_D0 = 448;
constexpr uint32_t T_R = T_D1, T_CU = T_D1, T_U = T_D1 + 32;  // two values a column, each over what has been read

// Offset of tokens 4 ch .. 4 ch + 3 of channel r in the transposed fp32 values (256 bytes a
// channel; permuted so that neither the writes nor a warp's reads of 32 channels meet in a bank).
__device__ __forceinline__ uint32_t vt_off(int r, int ch) { return (uint32_t)(r * 256 + ((ch ^ (r & 7)) << 4)); }

// One lane of a converged warp.  The products' operands are warp-uniform registers: behind a plain
// thread test (not this, under a warp-uniform condition) each product took 130 cycles to issue,
// whatever its size; so, 56 (N = 64) to 74 (N = 128).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Register shares of the four warp groups; the block is launched with 128 a thread.
constexpr int kRegChain = 208, kRegHelper = 104, kRegFactor = 104, kRegConvert = 96;
static_assert(kRegChain + kRegHelper + kRegFactor + kRegConvert <= 4 * 128, "register file");
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// K-step s of 16 added to a K-major descriptor of a 128-row tile, of a 64-row tile with 64 columns, and
// to an MN-major one, in the descriptor's 16-byte units.
__device__ __forceinline__ uint64_t step128(int s) { return (uint64_t)((s >> 2) * 1024 + (s & 3) * 2); }
__device__ __forceinline__ uint64_t step64(int s) { return (uint64_t)(2 * s); }
__device__ __forceinline__ uint64_t step_mn(int s) { return (uint64_t)(128 * s); }

// grid U, 512 threads: warps 0-3 chain, 4-7 helper, 8-11 factor, 12-15 convert.
__global__ void __launch_bounds__(512, 1) mesa_rule_chain_kernel(RuleArgs a, const __grid_constant__ CUtensorMap mapV) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  ChainMisc *m = reinterpret_cast<ChainMisc *>(sm + CH_MISC);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // (warp: uniform)
  const int u = blockIdx.x, T = a.T, NC = (T + C - 1) / C;
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  volatile int *gave_up = &m->gave_up;
  const unsigned limit = a.wait_limit;

  auto fetch_v = [&](int c) {
    const uint32_t b = bar(m->v_full), dst = tc::smem_u32(sm + CH_V);
    tc::mbar_arrive_expect_tx(b, ROWS64);
#pragma unroll
    for (int h = 0; h < 2; h++) tensor_g2s_3d(dst + h * C * 128, &mapV, 64 * h, c * C, u, b);
  };
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 128) {
    for (uint64_t *b : {&m->vt_full, &m->fac_full[0], &m->fac_full[1], &m->r_ready, &m->u_ready, &m->o_free,
                        &m->tile_full[0], &m->tile_full[1], &m->tile_full[2]})
      tc::mbar_init(bar(*b), 4);
    for (uint64_t *b : {&m->tile_free[0], &m->tile_free[1], &m->tile_free[2], &m->v_full, &m->d0_full, &m->mma1, &m->mma2,
                        &m->mma3, &m->mma4[0], &m->mma4[1]})
      tc::mbar_init(bar(*b), 1);
    tc::mbar_init(bar(m->drain), 3);  // the three threads that issue products
    m->gave_up = 0;
    fetch_v(0);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = __shfl_sync(0xffffffffu, m->tmem, 0);
  // one arrival per warp, after what its lanes did
  auto warp_arrive = [&](uint64_t &b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  bool ok = true;
  int v_sent = 1;  // fetches issued (thread 128)

  if (warp < 4) {
    // ---- the chain: thread r holds row r of the state ----
    regs_up<kRegChain>();
    const int r = tid;
    const uint32_t tl = tbase + ((uint32_t)(32 * warp) << 16);
    u64 S[D / 2];
    {
      const float4 *src = a.S0 ? reinterpret_cast<const float4 *>(a.S0 + ((size_t)u * D + r) * D) : nullptr;
#pragma unroll
      for (int g = 0; g < D / 4; g++) {
        const float4 x = src ? src[g] : make_float4(0, 0, 0, 0);
        S[2 * g] = pack2(x.x, x.y);
        S[2 * g + 1] = pack2(x.z, x.w);
      }
    }
    float bS, iS;  // a bound of the row's elements; 1 / scale of the S0 operand
    auto row_max = [&]() {
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < D / 2; i++) {
        float p, q;
        unpack2(S[i], p, q);
        x[i & 3] = fmaxf(x[i & 3], fmaxf(fabsf(p), fabsf(q)));
      }
      bS = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
    };
    row_max();
    {
      const float sS = bound_scale(bS, kTopRow, iS);
      const u64 s2 = pack2(sS, sS);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = half2_bits(mul2(S[8 * k + i], s2));
        tc::tmem_st8(tl + T_S + 8 * k, v);
      }
      tc::tmem_st_wait();
    }
    const uint32_t id64 = tc::idesc_f16(128, C, false, false);    // N = 64, B K-major
    const uint32_t id128 = tc::idesc_f16(128, D, false, false);   // N = 128, B K-major
    const uint32_t idKN = tc::idesc_f16(128, D, false, true);     // N = 128, B MN-major
    // barrier of the chain; true when a wait gave up
    auto meet = [&]() -> bool {
      tc::fence_before_sync();
      const bool stop = group_or(1, 128, !ok);
      tc::fence_after_sync();
      ok &= !stop;
      return stop;
    };
    for (int c = 0; c < NC; c++) {
      const uint32_t ph = c & 1, tile = tc::smem_u32(sm + CH_TILE + (c % 3) * TILE),
                     fac = tc::smem_u32(sm + CH_FAC + 2 * SQ * ph);
      const float *nf = m->nf[c & 3], *cc = m->c[c & 3];
      ok &= wait(bar(m->tile_full[c % 3]), (c / 3) & 1, limit, gave_up);
      if (c > 0) ok &= wait(bar(m->o_free), (c - 1) & 1, limit, gave_up);  // (the last readout is read)
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t kq = tc::kmajor_desc(tile, 128, 0);
#pragma unroll
        for (int s = 0; s < 8; s++)  // S0 K^T and S0 Q^T
          tc::mma_f16_ts(tbase + T_D1, tbase + T_S + 8 * s, kq + step128(s), id128, s > 0);
        tc::mma_commit(bar(m->mma1));
      }
      ok &= wait(bar(m->fac_full[ph]), (c >> 1) & 1, limit, gave_up);
      ok &= wait(bar(m->vt_full), ph, limit, gave_up);
      const float iK = m->inv_k[c % 3], kmax = (float)(1 << kTopTile) * iK;
      m->o1[ph][r] = -a.scale * iS * m->inv_q[c % 3];
      const float w1 = iS * iK;  // units of D1
      float iR;
      const float sR = bound_scale(fmaf((float)D * kmax, bS, m->vmax[warp]), kTopRow, iR);
      const u64 w1_2 = pack2(w1, w1), sR2 = pack2(sR, sR);
      ok &= wait(bar(m->mma1), ph, limit, gave_up);
      tc::fence_after_sync();
      // R = V^T - f D1, 16 tokens at a time (few registers beside the state's 128: what spills
      // here is paid for on the chain)
      {
        const uint8_t *V = sm + CH_VT + r * 256;
#pragma unroll
        for (int h = 0; h < 4; h++) {
          float z[16];
          tc::tmem_ld16(tl + T_D1 + 16 * h, z);
          ulonglong2 vv[4], ff[4];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            ff[k] = *reinterpret_cast<const ulonglong2 *>(nf + 16 * h + 4 * k);
            vv[k] = *reinterpret_cast<const ulonglong2 *>(V + (((4 * h + k) ^ (r & 7)) << 4));
          }
          tc::tmem_ld_wait();
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            v[2 * k] = half2_bits(mul2(fma2(pack2(z[4 * k], z[4 * k + 1]), mul2(ff[k].x, w1_2), vv[k].x), sR2));
            v[2 * k + 1] = half2_bits(mul2(fma2(pack2(z[4 * k + 2], z[4 * k + 3]), mul2(ff[k].y, w1_2), vv[k].y), sR2));
          }
          // (columns 8 h .. 8 h + 7: read by now)
          tc::tmem_st8(tl + T_R + 8 * h, v);
        }
      }
      tc::tmem_st_wait();
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t fm = tc::kmajor_desc(fac, C, 0);
#pragma unroll
        for (int s = 0; s < 4; s++) tc::mma_f16_ts(tbase + T_D2, tbase + T_R + 8 * s, fm + step64(s), id64, s > 0);
        tc::mma_commit(bar(m->mma2));
      }
      warp_arrive(m->r_ready);  // (V^T has been read)
      ok &= wait(bar(m->mma2), ph, limit, gave_up);
      tc::fence_after_sync();
      // U, for the readout, and c U, for the state (over R and what is left of D1)
      float uU = 0.0f, iU;  // the row's largest in units of D2, 1 / scale of the operands
      {
        float mx[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float x[32];
          tc::tmem_ld32(tl + T_D2 + 32 * h, x);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; i += 2) mx[(i >> 1) & 3] = fmaxf(mx[(i >> 1) & 3], fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
        }
        uU = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float sU = bound_scale(uU, kTopRow, iU);
        const u64 sU2 = pack2(sU, sU);
#pragma unroll
        for (int h = 0; h < 4; h++) {
          float x[16], v[8], w[8];
          tc::tmem_ld16(tl + T_D2 + 16 * h, x);
          tc::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(cc + 16 * h + 4 * k);
            const u64 p = mul2(pack2(x[4 * k], x[4 * k + 1]), sU2), q = mul2(pack2(x[4 * k + 2], x[4 * k + 3]), sU2);
            w[2 * k] = half2_bits(mul2(p, ff.x));
            w[2 * k + 1] = half2_bits(mul2(q, ff.y));
            v[2 * k] = half2_bits(p);
            v[2 * k + 1] = half2_bits(q);
          }
          tc::tmem_st8(tl + T_CU + 8 * h, w);
          tc::tmem_st8(tl + T_U + 8 * h, v);
        }
        tc::tmem_st_wait();
      }
      const float w3 = iU * iR * iK;  // units of dS
      m->o2[ph][r] = a.scale * w3 * m->inv_q[c % 3];
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t kt = tc::mnmajor_desc(tile, 128, 0);
#pragma unroll
        for (int s = 0; s < 4; s++) tc::mma_f16_ts(tbase + T_DS, tbase + T_CU + 8 * s, kt + step_mn(s), idKN, s > 0);
        tc::mma_commit(bar(m->mma3));
      }
      warp_arrive(m->u_ready);
      // the state after the chunk
      const u64 w3_2 = pack2(w3, w3);
      // 64 products of |c u| <= |u| and |k| bound what is added
      bS = fmaf(-nf[C - 1], bS, (float)C * uU * iR * kmax);
      const float sS = bound_scale(bS, kTopRow, iS);
      const u64 sS2 = pack2(sS, sS);
      const u64 dec = pack2(-nf[C - 1], -nf[C - 1]);
      ok &= wait(bar(m->mma3), ph, limit, gave_up);
      tc::fence_after_sync();
      if (r == 0) mbar_arrive(bar(m->tile_free[c % 3]));
      {
#pragma unroll
        for (int k = 0; k < 8; k++) {
          float z[16], v[8];
          tc::tmem_ld16(tl + T_DS + 16 * k, z);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; i++) {
            S[8 * k + i] = fma2(pack2(z[2 * i], z[2 * i + 1]), w3_2, mul2(S[8 * k + i], dec));
            v[i] = half2_bits(mul2(S[8 * k + i], sS2));
          }
          tc::tmem_st8(tl + T_S + 8 * k, v);  // the next chunk's operand
        }
        tc::tmem_st_wait();
      }
      if ((c & 7) == 7) row_max();  // (before the bound is loose)
    }
    if (!group_or(1, 128, !ok) && a.S_final) {
      float4 *dst = reinterpret_cast<float4 *>(a.S_final + ((size_t)u * D + r) * D);
#pragma unroll
      for (int g = 0; g < D / 4; g++) {
        float4 x;
        unpack2(S[2 * g], x.x, x.y);
        unpack2(S[2 * g + 1], x.z, x.w);
        dst[g] = x;
      }
    }
  } else if (warp < 8) {
    // ---- transpose the values; write the readout ----
    regs_down<kRegHelper>();
    const int h = tid - 128;
    const uint32_t tl = tbase + ((uint32_t)(32 * (warp - 4)) << 16);
    auto transpose = [&](int c) -> bool {  // chunk c's values (the last chunk's have been used)
      if (group_or(2, 128, !wait(bar(m->v_full), c & 1, limit, gave_up))) return false;
      // channels 32 w .. 32 w + 31 by warp w: eight channels x 32 tokens at a time
      uint32_t mv = 0;
#pragma unroll 1
      for (int g = 0; g < 4; g++) {
        const int ch8 = 4 * (warp - 4) + g;
#pragma unroll
        for (int t = 0; t < 2; t++) {
          uint32_t x[4];
          ldmatrix_x4_trans(x, tc::smem_u32(sm + CH_V + tile_off(32 * t + lane, ch8, C)));
          mv = absmax_words(mv, make_uint4(x[0], x[1], x[2], x[3]));
          const int r = 8 * ch8 + (lane >> 2);
#pragma unroll
          for (int k = 0; k < 4; k++)  // tokens 32 t + 8 k + 2 (lane % 4), + 1
            *reinterpret_cast<float2 *>(sm + CH_VT + vt_off(r, 8 * t + 2 * k + ((lane & 3) >> 1)) + 8 * (lane & 1)) =
                make_float2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u));
        }
      }
      mv = absmax_fold(mv);
      if (lane == 0) m->vmax[warp - 4] = __uint_as_float(mv << 16);  // of this warp's channels
      warp_arrive(m->vt_full);
      group_or(2, 128, false);
      if (c + 1 < NC) {
        if (h == 0) fetch_v(c + 1);
        v_sent++;
      }
      return true;
    };
    const uint32_t id64 = tc::idesc_f16(128, C, false, false);
    u64 nonfinite = 0;  // a NaN once an output was not finite
    ok = transpose(0);
    for (int c = 0; c < NC && ok; c++) {
      if (c + 1 < NC) {
        if (group_or(2, 128, !wait(bar(m->r_ready), c & 1, limit, gave_up)) || !transpose(c + 1)) {
          ok = false;
          break;
        }
      }
      bool got = wait(bar(m->u_ready), c & 1, limit, gave_up);
      got = __all_sync(0xffffffffu, got);
      tc::fence_after_sync();
      if (warp == 4 && got && elect_one()) {  // U P^T
        const uint64_t pd = tc::kmajor_desc(tc::smem_u32(sm + CH_FAC + 2 * SQ * (c & 1) + SQ), C, 0);
#pragma unroll
        for (int s = 0; s < 4; s++) tc::mma_f16_ts(tbase + T_O2, tbase + T_U + 8 * s, pd + step64(s), id64, s > 0);
        tc::mma_commit(bar(m->mma4[c & 1]));
      }
      got &= wait(bar(m->mma4[c & 1]), (c >> 1) & 1, limit, gave_up);
      if (h == 0) tc::bulk_wait_read();  // the last chunk's output has left its buffer
      if (group_or(2, 128, !got)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const float *nf = m->nf[c & 3];
      const float o1 = m->o1[c & 1][h], o2 = m->o2[c & 1][h];
      const u64 w1 = pack2(o1, o1), w2 = pack2(o2, o2);
      __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(sm + CH_OUT) + h;
      float x[64];  // from S0: all at once, the chain's next product writes there
      tc::tmem_ld32(tl + T_O1, *reinterpret_cast<float(*)[32]>(x));
      tc::tmem_ld32(tl + T_O1 + 32, *reinterpret_cast<float(*)[32]>(x + 32));
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      warp_arrive(m->o_free);
#pragma unroll
      for (int g = 0; g < 4; g++) {
        float y[16];
        tc::tmem_ld16(tl + T_O2 + 16 * g, y);
        ulonglong2 ff[4];
#pragma unroll
        for (int k = 0; k < 4; k++) ff[k] = *reinterpret_cast<const ulonglong2 *>(nf + 16 * g + 4 * k);
        tc::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
          const u64 o = fma2(pack2(x[16 * g + k], x[16 * g + k + 1]), mul2(k & 2 ? ff[k / 4].y : ff[k / 4].x, w1),
                             mul2(pack2(y[k], y[k + 1]), w2));
          nonfinite = fma2(o, 0ull, nonfinite);
          float p, q;
          unpack2(o, p, q);
          const __nv_bfloat162 b = __floats2bfloat162_rn(p, q);
          dst[(16 * g + k) * D] = b.x;
          dst[(16 * g + k + 1) * D] = b.y;
        }
      }
      tc::fence_before_sync();
      tc::fence_smem_to_async();
      group_or(2, 128, false);
      if (h == 0) {
        bulk_s2g((__nv_bfloat16 *)a.out + ((size_t)u * T + (size_t)c * C) * D, tc::smem_u32(sm + CH_OUT),
                 (uint32_t)min(C, T - c * C) * D * 2);
        tc::bulk_commit();
      }
    }
    if (!(sum2(nonfinite) == 0.0f)) atomicOr(a.status, tc::kErrNonFinite);
    if (h == 0) tc::bulk_wait_all();
  } else if (warp < 12) {
    // ---- the factors, one chunk ahead of the chain ----
    regs_down<kRegFactor>();
    const int h = tid - 256, w = warp - 8;
    Factor &s = *reinterpret_cast<Factor *>(sm + CH_SCR);
    for (int b = 0; b < 4; b++) factor_clear(sm + CH_FAC + SQ * b, h);
    const size_t g0 = (size_t)u * T;
    // the next chunk's gates: gamma in warp 3, beta in warps 0 and 1
    float2 ga;
    float be = 0.0f;
    auto load_gates = [&](int c) {
      const int n = T - c * C;
      const float *gp = a.gamma + g0 + (size_t)c * C, *bp = a.beta + g0 + (size_t)c * C;
      if (w == 3) ga = make_float2(2 * lane < n ? gp[2 * lane] : 1.0f, 2 * lane + 1 < n ? gp[2 * lane + 1] : 1.0f);
      if (w < 2) be = h < n ? bp[h] : 0.0f;
    };
    const uint32_t id64 = tc::idesc_f16(128, C, false, false);
    auto begin = [&](int c) {  // warp 3: [K K^T; Q K^T] of chunk c, and its decays while that runs
      const bool got = wait(bar(m->tile_full[c % 3]), (c / 3) & 1, limit, gave_up);
      tc::fence_after_sync();
      if (__all_sync(0xffffffffu, got) && elect_one()) {
        const uint64_t t = tc::kmajor_desc(tc::smem_u32(sm + CH_TILE + (c % 3) * TILE), 128, 0);
#pragma unroll
        for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_D0, t + step128(s), t + step128(s), id64, s > 0);
        tc::mma_commit(bar(m->d0_full));
      }
      __syncwarp();
      factor_gates(s, gate_scan(ga, lane), m->nf[c & 3], m->c[c & 3], lane);
    };
    load_gates(0);
    if (w == 3) begin(0);
    for (int c = 0; c < NC; c++) {
      const int b = c & 1;
      uint8_t *M = sm + CH_FAC + 2 * SQ * b, *P = M + SQ;
      const float be_now = be;
      if (c + 1 < NC) load_gates(c + 1);
      // slot b of M and P is free once the readout product of chunk c - 2 is done (and slot c % 4
      // of the decays: that product came after the readout of chunk c - 4)
      bool got = c < 2 || wait(bar(m->mma4[b]), ((c >> 1) - 1) & 1, limit, gave_up);
      got &= wait(bar(m->tile_full[c % 3]), (c / 3) & 1, limit, gave_up);
      got &= wait(bar(m->d0_full), c & 1, limit, gave_up);
      if (group_or(3, 128, !got)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (w < 2) s.beta[h] = be_now;
      factor_rows(s, tbase + T_D0, m->inv_k[c % 3] * m->inv_k[c % 3], P, h);
      tc::fence_before_sync();
      group_or(3, 128, false);
      factor_diagonal<true>(s, M, w, lane);
      group_or(3, 128, false);
      tc::fence_after_sync();
      if (w < 3) {
        factor_columns<true>(s, M, w, lane);
      } else if (c + 1 < NC) {  // (the last column block has nothing below its diagonal block)
        begin(c + 1);
      }
      tc::fence_smem_to_async();
      warp_arrive(m->fac_full[b]);
    }
  } else {
    // ---- K and Q as operands, up to three chunks in flight ----
    regs_down<kRegConvert>();
    const int h = tid - 384, r0 = h >> 4, c8 = h & 15, uk = a.qk_unit(u);  // rows r0, r0 + 8 ..; 8 channels
    const __nv_bfloat16 *kp = (const __nv_bfloat16 *)a.k + ((size_t)uk * T + r0) * D + 8 * c8;
    const __nv_bfloat16 *qp = (const __nv_bfloat16 *)a.q + ((size_t)uk * T + r0) * D + 8 * c8;
    uint4 x[8], y[8];  // the next chunk's rows, on their way while this one's are converted
    auto load = [&](int c) {
      const int n = T - c * C - r0;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        x[i] = y[i] = make_uint4(0, 0, 0, 0);
        if (8 * i < n) {
          x[i] = *reinterpret_cast<const uint4 *>(kp + ((size_t)c * C + 8 * i) * D);
          y[i] = *reinterpret_cast<const uint4 *>(qp + ((size_t)c * C + 8 * i) * D);
        }
      }
    };
    load(0);
    for (int c = 0; c < NC; c++) {
      uint32_t mk = 0, mq = 0;
#pragma unroll
      for (int k = 0; k < 8; k++) {
        mk = absmax_words(mk, x[k]);
        mq = absmax_words(mq, y[k]);
      }
      mk = absmax_fold(mk);
      mq = absmax_fold(mq);
      uint32_t *red = m->red + 8 * (c & 1);
      if (lane == 0) {
        red[warp - 12] = mk;
        red[warp - 8] = mq;
      }
      bool got = true;
      if (c >= 3) got = wait(bar(m->tile_free[c % 3]), (c / 3 - 1) & 1, limit, gave_up);
      if (group_or(4, 128, !got)) {
        ok = false;
        break;
      }
      const uint4 k4 = *reinterpret_cast<const uint4 *>(red), q4 = *reinterpret_cast<const uint4 *>(red + 4);
      float ik, iq;
      const float sk = bound_scale(__uint_as_float(max(max(k4.x, k4.y), max(k4.z, k4.w)) << 16), kTopTile, ik);
      const float sq = bound_scale(__uint_as_float(max(max(q4.x, q4.y), max(q4.z, q4.w)) << 16), kTopTile, iq);
      if (h == 0) {
        m->inv_k[c % 3] = ik;
        m->inv_q[c % 3] = iq;
      }
      const u64 sk2 = pack2(sk, sk), sq2 = pack2(sq, sq);
      uint8_t *dst = sm + CH_TILE + (c % 3) * TILE + tile_off(r0, c8, 128);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        *reinterpret_cast<uint4 *>(dst + 1024 * k) = to_half8(x[k], sk2);
        *reinterpret_cast<uint4 *>(dst + C * 128 + 1024 * k) = to_half8(y[k], sq2);
      }
      tc::fence_smem_to_async();
      warp_arrive(m->tile_full[c % 3]);
      if (c + 1 < NC) load(c + 1);
    }
  }
  if (!ok) *gave_up = 1;
  __syncthreads();
  // a wait gave up: products and copies still in flight finish before the memory is released
  if (*gave_up) {
    // (a product's commit counts for the thread that issued it: the same elected lane)
    if ((warp == 0 || warp == 4 || warp == 8) && elect_one()) tc::mma_commit(bar(m->drain));
    if (tid == 0) {
      unsigned bits = tc::kErrMmaTimeout;
      if (!tc::mbar_wait(bar(m->drain), 0, tc::kWaitLimit)) bits |= tc::kErrDrainTimeout;
      atomicOr(a.status, bits);
    }
    if (tid == 128 && !tc::mbar_wait(bar(m->v_full), (v_sent - 1) & 1, tc::kWaitLimit))
      atomicOr(a.status, tc::kErrDrainTimeout);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 512);
}

}  // namespace

int launch_rule_forward_tc(const RuleArgs &a, cudaStream_t st) {
  CUtensorMap mapV{};
  if (!tmap_units128_bf16(&mapV, a.v, a.units(), a.T)) return -1;
  if (cudaFuncSetAttribute(mesa_rule_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CH_SMEM) !=
      cudaSuccess)
    return -1;
  timing_mark_begin(K_RULE_CHAIN, st);
  mesa_rule_chain_kernel<<<a.units(), 512, CH_SMEM, st>>>(a, mapV);
  timing_mark_end(K_RULE_CHAIN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mesa
