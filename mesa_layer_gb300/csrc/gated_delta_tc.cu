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
// bounds the kernel, so all else runs beside it, in four warp groups:
//     chain    the three epilogues above;
//     helper   converts K and Q and transposes V one chunk ahead, writes the last readout;
//     factor   decays, masks and the triangular inverse, one chunk ahead;
//     issuer   one thread that issues every product in the order the chain needs them.
// The inputs are read once and the output written once; nothing else goes to memory.
#include "gated_delta_tc.cuh"

namespace mesa {

using namespace rule;

namespace {

// shared memory: two K, Q operand tiles | two slots of factors M, P | V^T in fp32 | V, K, Q as read |
// output | factor scratch | misc
constexpr uint32_t CH_TILE = 0, CH_FAC = CH_TILE + 2 * TILE, CH_VT = CH_FAC + 4 * SQ, CH_RAW = CH_VT + 2 * ROWS64;
constexpr uint32_t CH_V = CH_RAW + 2 * ROWS64;
constexpr uint32_t CH_OUT = CH_V + ROWS64, CH_SCR = CH_OUT + ROWS64;
constexpr uint32_t CH_MISC = CH_SCR + ((sizeof(Factor) + 127) & ~127u);
struct ChainMisc {
  float o1[2][D], o2[2][D];     // units of the readout's accumulators, by state row
  float nf[4][C], c[4][C];    // minus the decays from the chunk's start; those to its end
  float inv_k[2], inv_q[2];   // 1 / operand scales, by slot
  float vmax[4];              // largest |v| of 32 channels
  uint32_t red[8];
  uint64_t raw_full, tile_full[2], v_full, vt_full, d0_full, d0_free, fac_full[2], s_ready, r_ready, u_ready, o_free;
  uint64_t mma1, mma2, mma3, mma4, drain;
  uint32_t tmem;
  int gave_up;
};
constexpr uint32_t CH_SMEM = CH_MISC + sizeof(ChainMisc) + 1024;
static_assert(CH_SMEM <= 232448, "shared memory per block");
// tensor memory columns: dS | S0 operand | D1 (then R), O from S0 | D2 (then U and c U) | O from U |
// [K K^T; Q K^T]
constexpr uint32_t T_DS = 0, T_S = 128, T_D1 = 192, T_O1 = 256, T_D2 = 320, T_O2 = 384, T_D0 = 448;
constexpr uint32_t T_R = T_D1;  // R, two values a column, over what of D1 has been read

// Offset of tokens 4 ch .. 4 ch + 3 of channel r in the transposed fp32 values (256 bytes a
// channel; permuted so that neither the writes nor a warp's reads of 32 channels meet in a bank).
__device__ __forceinline__ uint32_t vt_off(int r, int ch) { return (uint32_t)(r * 256 + ((ch ^ (r & 7)) << 4)); }

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Register shares of the warp groups; the block is launched with 128 a thread.
constexpr int kRegChain = 208, kRegHelper = 128, kRegFactor = 128, kRegIssuer = 48;
static_assert(kRegChain + kRegHelper + kRegFactor + kRegIssuer <= 512, "register file");
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// grid U, 512 threads: warps 0-3 chain, 4-7 helper, 8-11 factor, 12 issuer (13-15 idle).
__global__ void __launch_bounds__(512, 1)
    mesa_rule_chain_kernel(RuleArgs a, const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapQ,
                           const __grid_constant__ CUtensorMap mapV) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  ChainMisc *m = reinterpret_cast<ChainMisc *>(sm + CH_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, u = blockIdx.x, T = a.T, NC = (T + C - 1) / C;
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  volatile int *gave_up = &m->gave_up;
  const unsigned limit = a.wait_limit;

  const int uk = a.qk_unit(u);
  auto fetch_kq = [&](int c) {
    const uint32_t b = bar(m->raw_full), dst = tc::smem_u32(sm + CH_RAW);
    tc::mbar_arrive_expect_tx(b, 2 * ROWS64);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      tensor_g2s_3d(dst + h * C * 128, &mapK, 64 * h, c * C, uk, b);
      tensor_g2s_3d(dst + h * C * 128 + ROWS64, &mapQ, 64 * h, c * C, uk, b);
    }
  };
  auto fetch_v = [&](int c) {
    const uint32_t b = bar(m->v_full), dst = tc::smem_u32(sm + CH_V);
    tc::mbar_arrive_expect_tx(b, ROWS64);
#pragma unroll
    for (int h = 0; h < 2; h++) tensor_g2s_3d(dst + h * C * 128, &mapV, 64 * h, c * C, u, b);
  };
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 128) {
    for (uint64_t *b : {&m->vt_full, &m->fac_full[0], &m->fac_full[1], &m->d0_free, &m->s_ready, &m->r_ready,
                        &m->u_ready, &m->o_free})
      tc::mbar_init(bar(*b), 4);
    for (uint64_t *b : {&m->raw_full, &m->v_full, &m->d0_full, &m->mma1, &m->mma2, &m->mma3, &m->mma4, &m->drain})
      tc::mbar_init(bar(*b), 1);
    for (uint64_t *b : {&m->tile_full[0], &m->tile_full[1]}) tc::mbar_init(bar(*b), 4);
    m->gave_up = 0;
    fetch_kq(0);
    fetch_v(0);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = m->tmem;
  // one arrival per warp, after what its lanes did
  auto warp_arrive = [&](uint64_t &b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  bool ok = true;
  int kq_sent = 1, v_sent = 1;  // fetches issued (thread 128)

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
    auto stage_state = [&]() {  // S (this thread's row) as the A operand
      const float sS = bound_scale(bS, kTopRow, iS);
      const u64 s2 = pack2(sS, sS);
#pragma unroll
      for (int k = 0; k < 4; k++) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; i++) v[i] = half2_bits(mul2(S[16 * k + i], s2));
        tc::tmem_st16(tl + T_S + 16 * k, v);
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(m->s_ready);
    };
    stage_state();
    for (int c = 0; c < NC; c++) {
      const uint32_t ph = c & 1;
      const float *nf = m->nf[c & 3], *cc = m->c[c & 3];
      ok &= wait(bar(m->tile_full[ph]), (c >> 1) & 1, limit, gave_up);
      ok &= wait(bar(m->fac_full[ph]), (c >> 1) & 1, limit, gave_up);
      ok &= wait(bar(m->vt_full), ph, limit, gave_up);
      const float iK = m->inv_k[ph], kmax = (float)(1 << kTopTile) * iK;
      m->o1[ph][r] = -a.scale * iS * m->inv_q[ph];
      const float w1 = iS * iK;  // units of D1
      float iR;
      const float sR = bound_scale(fmaf((float)D * kmax, bS, m->vmax[warp]), kTopRow, iR);
      const u64 w1_2 = pack2(w1, w1), sR2 = pack2(sR, sR);
      ok &= wait(bar(m->mma1), ph, limit, gave_up);
      if (__any_sync(0xffffffffu, !ok)) break;
      tc::fence_after_sync();
      // R = V^T - f D1
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float x[32];
        tc::tmem_ld32(tl + T_D1 + 32 * h, x);
        tc::tmem_ld_wait();
        float v[16];
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(nf + 32 * h + 4 * k);
          const ulonglong2 vv = *reinterpret_cast<const ulonglong2 *>(sm + CH_VT + vt_off(r, 8 * h + k));
          v[2 * k] = half2_bits(mul2(fma2(pack2(x[4 * k], x[4 * k + 1]), mul2(ff.x, w1_2), vv.x), sR2));
          v[2 * k + 1] = half2_bits(mul2(fma2(pack2(x[4 * k + 2], x[4 * k + 3]), mul2(ff.y, w1_2), vv.y), sR2));
        }
        tc::tmem_st16(tl + T_R + 16 * h, v);
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(m->r_ready);
      ok &= wait(bar(m->mma2), ph, limit, gave_up);
      if (__any_sync(0xffffffffu, !ok)) break;
      tc::fence_after_sync();
      // U, for the readout, and c U, for the state
      float uU, iU;  // the row's largest in units of D2, 1 / scale of the operands
      {
        float x[32], y[32];
        tc::tmem_ld32(tl + T_D2, x);
        tc::tmem_ld32(tl + T_D2 + 32, y);
        tc::tmem_ld_wait();
        float mx[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 32; i++) mx[i & 3] = fmaxf(mx[i & 3], fmaxf(fabsf(x[i]), fabsf(y[i])));
        uU = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float sU = bound_scale(uU, kTopRow, iU);
        const u64 sU2 = pack2(sU, sU);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float v[16], w[16];
#pragma unroll
          for (int k = 0; k < 8; k++) {
            const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(cc + 32 * h + 4 * k);
            const float *z = (h ? y : x) + 4 * k;
            const u64 p = mul2(pack2(z[0], z[1]), sU2), q = mul2(pack2(z[2], z[3]), sU2);
            w[2 * k] = half2_bits(mul2(p, ff.x));
            w[2 * k + 1] = half2_bits(mul2(q, ff.y));
            v[2 * k] = half2_bits(p);
            v[2 * k + 1] = half2_bits(q);
          }
          tc::tmem_st16(tl + T_D2 + 32 + 16 * h, w);
          tc::tmem_st16(tl + T_D2 + 16 * h, v);
        }
        tc::tmem_st_wait();
      }
      const float w3 = iU * iR * iK;  // units of dS
      m->o2[ph][r] = a.scale * w3 * m->inv_q[ph];
      tc::fence_before_sync();
      warp_arrive(m->u_ready);
      // the state after the chunk
      const u64 w3_2 = pack2(w3, w3);
      const u64 dec = pack2(-nf[C - 1], -nf[C - 1]);
      ok &= wait(bar(m->mma3), ph, limit, gave_up);
      if (__any_sync(0xffffffffu, !ok)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int k = 0; k < 4; k++) {
        float x[32];
        tc::tmem_ld32(tl + T_DS + 32 * k, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i++)
          S[16 * k + i] = fma2(pack2(x[2 * i], x[2 * i + 1]), w3_2, mul2(S[16 * k + i], dec));
      }
      // 64 products of |c u| <= |u| and |k|; the row itself now and then, before the bound is loose
      bS = fmaf(-nf[C - 1], bS, (float)C * uU * iR * kmax);
      if ((c & 7) == 7) row_max();
      if (c + 1 < NC) stage_state();
    }
    if (ok && a.S_final) {
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
    auto convert = [&](int c) -> bool {  // chunk c's K and Q into slot c & 1 (free: its products are done)
      const int b = c & 1;
      if (group_or(2, 128, !wait(bar(m->raw_full), c & 1, limit, gave_up))) return false;
      const uint8_t *raw = sm + CH_RAW + tile_off(h >> 4, h & 15, C);  // rows h / 16, + 8, + 16 ..
      uint8_t *tile = sm + CH_TILE + b * TILE + tile_off(h >> 4, h & 15, 128);
      uint32_t mk = 0, mq = 0;
#pragma unroll
      for (int p = 0; p < 8; p++) {
        mk = absmax_words(mk, *reinterpret_cast<const uint4 *>(raw + 1024 * p));
        mq = absmax_words(mq, *reinterpret_cast<const uint4 *>(raw + ROWS64 + 1024 * p));
      }
      mk = absmax_fold(mk);
      mq = absmax_fold(mq);
      if (lane == 0) {
        m->red[warp - 4] = mk;
        m->red[warp] = mq;
      }
      group_or(2, 128, false);
      mk = max(max(m->red[0], m->red[1]), max(m->red[2], m->red[3]));
      mq = max(max(m->red[4], m->red[5]), max(m->red[6], m->red[7]));
      float ik, iq;
      const float sk = bound_scale(__uint_as_float(mk << 16), kTopTile, ik);
      const float sq = bound_scale(__uint_as_float(mq << 16), kTopTile, iq);
      if (h == 0) {
        m->inv_k[b] = ik;
        m->inv_q[b] = iq;
      }
      const u64 sk2 = pack2(sk, sk), sq2 = pack2(sq, sq);
#pragma unroll
      for (int p = 0; p < 8; p++) {
        *reinterpret_cast<uint4 *>(tile + 1024 * p) = to_half8(*reinterpret_cast<const uint4 *>(raw + 1024 * p), sk2);
        *reinterpret_cast<uint4 *>(tile + C * 128 + 1024 * p) =
            to_half8(*reinterpret_cast<const uint4 *>(raw + ROWS64 + 1024 * p), sq2);
      }
      tc::fence_smem_to_async();
      warp_arrive(m->tile_full[b]);
      group_or(2, 128, false);  // (the raw rows have been read)
      if (c + 1 < NC) {
        if (h == 0) fetch_kq(c + 1);
        kq_sent++;
      }
      return true;
    };
    auto transpose = [&](int c) -> bool {  // chunk c's values (the last chunk's have been used)
      if (group_or(2, 128, !wait(bar(m->v_full), c & 1, limit, gave_up))) return false;
      // channels 32 w .. 32 w + 31 by warp w: eight channels x 32 tokens at a time
      uint32_t mv = 0;
#pragma unroll
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
    u64 nonfinite = 0;  // a NaN once an output was not finite
    ok = convert(0) && transpose(0);
    for (int c = 0; c < NC && ok; c++) {
      if (c + 1 < NC) {
        if (!convert(c + 1) || group_or(2, 128, !wait(bar(m->r_ready), c & 1, limit, gave_up)) || !transpose(c + 1)) {
          ok = false;
          break;
        }
      }
      bool got = wait(bar(m->u_ready), c & 1, limit, gave_up);
      got &= wait(bar(m->mma4), c & 1, limit, gave_up);
      if (h == 0) tc::bulk_wait_read();  // the last chunk's output has left its buffer
      if (group_or(2, 128, !got)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const float *nf = m->nf[c & 3];
      const float o1 = m->o1[c & 1][h], o2 = m->o2[c & 1][h];
      const u64 w1 = pack2(o1, o1), w2 = pack2(o2, o2);
#pragma unroll
      for (int g = 0; g < 2; g++) {
        float x[32], y[32];
        tc::tmem_ld32(tl + T_O1 + 32 * g, x);
        tc::tmem_ld32(tl + T_O2 + 32 * g, y);
        tc::tmem_ld_wait();
        if (g == 1) {
          tc::fence_before_sync();
          warp_arrive(m->o_free);
        }
        __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(sm + CH_OUT) + 32 * g * D + h;
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(nf + 32 * g + k);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const u64 o = fma2(pack2(x[k + e], x[k + e + 1]), mul2(e ? ff.y : ff.x, w1),
                               mul2(pack2(y[k + e], y[k + e + 1]), w2));
            nonfinite = fma2(o, 0ull, nonfinite);
            float p, q;
            unpack2(o, p, q);
            const __nv_bfloat162 b = __floats2bfloat162_rn(p, q);
            dst[(k + e) * D] = b.x;
            dst[(k + e + 1) * D] = b.y;
          }
        }
      }
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
    for (int c = 0; c < NC; c++) {
      const int b = c & 1, n = min(C, T - c * C);
      uint8_t *M = sm + CH_FAC + 2 * SQ * b, *P = M + SQ;
      const size_t t0 = g0 + (size_t)c * C;
      GatePair g;
      float be = 0.0f;
      if (w == 0) g = gate_scan(a.gamma + t0, n, lane);
      if (w >= 2) be = h - 64 < n ? a.beta[t0 + h - 64] : 0.0f;
      // (slot b of M and P is free: the products of chunk c are issued after all of chunk c - 2;
      // slot c % 4 of the decays: its last readout came before one the issuer has waited for)
      bool got = wait(bar(m->tile_full[b]), (c >> 1) & 1, limit, gave_up);
      got &= wait(bar(m->d0_full), c & 1, limit, gave_up);
      if (group_or(3, 128, !got)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (w == 0) factor_gates(s, g, m->nf[c & 3], m->c[c & 3], lane);
      if (w >= 2) s.beta[h - 64] = be;
      group_or(3, 128, false);
      factor_rows(s, tbase + T_D0, m->inv_k[b] * m->inv_k[b], P, h, [&] {
        tc::fence_before_sync();
        warp_arrive(m->d0_free);
      });
      group_or(3, 128, false);
      factor_diagonal<true>(s, M, w, lane);
      group_or(3, 128, false);
      factor_columns<true>(s, M, w, lane);
      tc::fence_smem_to_async();
      warp_arrive(m->fac_full[b]);
    }
  } else {
    regs_down<kRegIssuer>();
    if (warp == 12 && lane == 0) {
      // ---- every product, in the order the chain needs them ----
      const uint32_t id64 = tc::idesc_f16(128, C, false, false);    // N = 64, B K-major
      const uint32_t id128 = tc::idesc_f16(128, D, false, false);   // N = 128, B K-major
      const uint32_t idKN = tc::idesc_f16(128, D, false, true);     // N = 128, B MN-major
      auto products0 = [&](int c) {  // [K K^T; Q K^T] of chunk c
        ok &= wait(bar(m->tile_full[c & 1]), (c >> 1) & 1, limit, gave_up);
        if (c > 0) ok &= wait(bar(m->d0_free), (c - 1) & 1, limit, gave_up);
        if (!ok) return;
        tc::fence_after_sync();
        const uint32_t tile = tc::smem_u32(sm + CH_TILE + (c & 1) * TILE);
#pragma unroll 1
        for (int s = 0; s < 8; s++)
          tc::mma_f16(tbase + T_D0, tc::kmajor_desc(tile, 128, s), tc::kmajor_desc(tile, 128, s), id64, s > 0);
        tc::mma_commit(bar(m->d0_full));
      };
      products0(0);
      for (int c = 0; c < NC && ok; c++) {
        const int b = c & 1;
        const uint32_t tile = tc::smem_u32(sm + CH_TILE + (c & 1) * TILE), fac = tc::smem_u32(sm + CH_FAC + 2 * SQ * b);
        ok &= wait(bar(m->s_ready), c & 1, limit, gave_up);
        if (c > 0) ok &= wait(bar(m->o_free), (c - 1) & 1, limit, gave_up);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll 1
        for (int s = 0; s < 8; s++)  // S0 K^T and S0 Q^T
          tc::mma_f16_ts(tbase + T_D1, tbase + T_S + 8 * s, tc::kmajor_desc(tile, 128, s), id128, s > 0);
        tc::mma_commit(bar(m->mma1));
        ok &= wait(bar(m->r_ready), c & 1, limit, gave_up);
        ok &= wait(bar(m->fac_full[b]), (c >> 1) & 1, limit, gave_up);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll 1
        for (int s = 0; s < 4; s++)
          tc::mma_f16_ts(tbase + T_D2, tbase + T_R + 8 * s, tc::kmajor_desc(fac, C, s), id64, s > 0);
        tc::mma_commit(bar(m->mma2));
        if (c + 1 < NC) products0(c + 1);
        ok &= wait(bar(m->u_ready), c & 1, limit, gave_up);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll 1
        for (int s = 0; s < 4; s++)
          tc::mma_f16_ts(tbase + T_DS, tbase + T_D2 + 32 + 8 * s, tc::mnmajor_desc(tile, 128, s), idKN, s > 0);
        tc::mma_commit(bar(m->mma3));
#pragma unroll 1
        for (int s = 0; s < 4; s++)
          tc::mma_f16_ts(tbase + T_O2, tbase + T_D2 + 8 * s, tc::kmajor_desc(fac + SQ, C, s), id64, s > 0);
        tc::mma_commit(bar(m->mma4));
      }
      if (!ok) tc::mma_commit(bar(m->drain));
    }
    __syncwarp();
  }
  if (!ok) *gave_up = 1;
  __syncthreads();
  // a wait gave up: products and copies still in flight finish before the memory is released
  if (*gave_up) {
    if (tid == 384) {
      unsigned bits = tc::kErrMmaTimeout;
      if (ok) tc::mma_commit(bar(m->drain));  // (the issuer had finished)
      if (!tc::mbar_wait(bar(m->drain), 0, tc::kWaitLimit)) bits |= tc::kErrDrainTimeout;
      atomicOr(a.status, bits);
    }
    if (tid == 128) {
      bool in = tc::mbar_wait(bar(m->v_full), (v_sent - 1) & 1, tc::kWaitLimit);
      in &= tc::mbar_wait(bar(m->raw_full), (kq_sent - 1) & 1, tc::kWaitLimit);
      if (!in) atomicOr(a.status, tc::kErrDrainTimeout);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 512);
}

}  // namespace

int launch_rule_forward_tc(const RuleArgs &a, cudaStream_t st) {
  CUtensorMap mapK{}, mapQ{}, mapV{};
  if (!tmap_units128_bf16(&mapK, a.k, a.B * a.Hk, a.T) || !tmap_units128_bf16(&mapQ, a.q, a.B * a.Hk, a.T) ||
      !tmap_units128_bf16(&mapV, a.v, a.units(), a.T))
    return -1;
  if (cudaFuncSetAttribute(mesa_rule_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CH_SMEM) !=
      cudaSuccess)
    return -1;
  timing_mark_begin(K_RULE_CHAIN, st);
  mesa_rule_chain_kernel<<<a.units(), 512, CH_SMEM, st>>>(a, mapK, mapQ, mapV);
  timing_mark_end(K_RULE_CHAIN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mesa
