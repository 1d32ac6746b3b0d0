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
//     helper   fetches rows, converts K and Q, transposes V one chunk ahead; writes the readout
//              of the chunk before;
//     factor   decays, masks and the triangular inverse, one chunk ahead;
//     issuer   one thread that issues every product in the order the chain needs them.
// The inputs are read once and the output written once; nothing else goes to memory.
#include "gated_delta_tc.cuh"

namespace mesa {

using namespace rule;

namespace {

// shared memory: two operand tiles | two slots of factors M, P | two V^T | raw K, Q, V | output |
// factor scratch | misc
constexpr uint32_t CH_TILE = 0, CH_FAC = CH_TILE + 2 * TILE, CH_VT = CH_FAC + 4 * SQ, CH_RAW = CH_VT + 2 * ROWS64;
constexpr uint32_t CH_OUT = CH_RAW + 3 * ROWS64, CH_SCR = CH_OUT + ROWS64;
constexpr uint32_t CH_MISC = CH_SCR + ((sizeof(Factor) + 127) & ~127u);
struct ChainMisc {
  float f[2][C], c[2][C];     // decays from the chunk's start, to its end
  float2 scales[2];           // of the K and Q operands
  float o1[2][D], o2[2][D];   // factors of the readout's accumulators, by state row
  float red[8];
  uint64_t raw_full, tile_full[2], d0_full, d0_free, fac_full[2], s_ready, r_ready, u_ready, o_free;
  uint64_t mma1, mma2, mma3, mma4, drain;
  uint32_t tmem;
  int gave_up;
};
constexpr uint32_t CH_SMEM = CH_MISC + sizeof(ChainMisc) + 1024;
static_assert(CH_SMEM <= 232448, "shared memory per block");
// tensor memory columns: dS | S0 operand | D1 (then R), O from S0 | D2 (then U and c U) | O from U |
// [K K^T; Q K^T]
constexpr uint32_t T_DS = 0, T_S = 128, T_D1 = 192, T_O1 = 256, T_D2 = 320, T_O2 = 384, T_D0 = 448;

// Offset of the 16 bytes with tokens 8 ch .. 8 ch + 7 of channel r in a transposed value tile
// (128 bytes a channel; permuted so that neither the transposing writes nor a chain warp's reads
// of 32 channels meet in a bank).
__device__ __forceinline__ uint32_t vt_off(int r, int ch) {
  return (uint32_t)(r * 128 + ((ch ^ (r & 7) ^ ((r >> 3) & 7)) << 4));
}

// The largest |x| of N pairs, four at a time (one running maximum would be a chain of N).
template <int N>
__device__ __forceinline__ float pair_absmax(const u64 (&x)[N]) {
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < N; i++) {
    float a, b;
    unpack2(x[i], a, b);
    m[i & 3] = fmaxf(m[i & 3], fmaxf(fabsf(a), fabsf(b)));
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Register shares of the warp groups; the block is launched with 128 a thread.
constexpr int kRegChain = 240, kRegHelper = 104, kRegFactor = 120, kRegIssuer = 40;
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
__global__ void __launch_bounds__(512, 1) mesa_rule_chain_kernel(RuleArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  ChainMisc *m = reinterpret_cast<ChainMisc *>(sm + CH_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, u = blockIdx.x, T = a.T, NC = (T + C - 1) / C;
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  volatile int *gave_up = &m->gave_up;
  const unsigned limit = a.wait_limit;
  const size_t v0 = (size_t)u * T * D, qk0 = (size_t)a.qk_unit(u) * T * D, g0 = (size_t)u * T;

  auto fetch = [&](int c) {  // raw K, Q and V rows of chunk c
    const uint32_t bytes = (uint32_t)min(C, T - c * C) * D * 2, b = bar(m->raw_full);
    const size_t at = (size_t)c * C * D;
    tc::mbar_arrive_expect_tx(b, 3 * bytes);
    tc::bulk_g2s(tc::smem_u32(sm + CH_RAW), (const __nv_bfloat16 *)a.k + qk0 + at, bytes, b);
    tc::bulk_g2s(tc::smem_u32(sm + CH_RAW + ROWS64), (const __nv_bfloat16 *)a.q + qk0 + at, bytes, b);
    tc::bulk_g2s(tc::smem_u32(sm + CH_RAW + 2 * ROWS64), (const __nv_bfloat16 *)a.v + v0 + at, bytes, b);
  };
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 128) {
    tc::mbar_init(bar(m->raw_full), 1);
    for (int b = 0; b < 2; b++) {
      tc::mbar_init(bar(m->tile_full[b]), 1);
      tc::mbar_init(bar(m->fac_full[b]), 4);
    }
    for (uint64_t *b : {&m->d0_free, &m->s_ready, &m->r_ready, &m->u_ready, &m->o_free}) tc::mbar_init(bar(*b), 4);
    for (uint64_t *b : {&m->d0_full, &m->mma1, &m->mma2, &m->mma3, &m->mma4, &m->drain}) tc::mbar_init(bar(*b), 1);
    m->gave_up = 0;
    fetch(0);
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
  int sent = 1;  // fetches issued (helper)

  if (warp < 4) {
    // ---- the chain: thread r holds row r of the state ----
    regs_up<kRegChain>();
    const int r = tid;
    const uint32_t tl = tbase + ((uint32_t)(32 * warp) << 16);
    u64 S[D / 2];
    float sS;  // scale of the S0 operand
    {
      const float4 *src = a.S0 ? reinterpret_cast<const float4 *>(a.S0 + ((size_t)u * D + r) * D) : nullptr;
#pragma unroll
      for (int g = 0; g < D / 4; g++) {
        const float4 x = src ? src[g] : make_float4(0, 0, 0, 0);
        S[2 * g] = pack2(x.x, x.y);
        S[2 * g + 1] = pack2(x.z, x.w);
      }
    }
    auto stage_state = [&]() {  // S (this thread's row) as the fp16 A operand
      sS = tile_scale(pair_absmax(S));
      const u64 s2 = pack2(sS, sS);
#pragma unroll
      for (int k = 0; k < 4; k++) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 16; i++) {
          float x, y;
          unpack2(mul2(S[16 * k + i], s2), x, y);
          v[i] = half2_bits(x, y);
        }
        tc::tmem_st16(tl + T_S + 16 * k, v);
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(m->s_ready);
    };
    stage_state();
    for (int c = 0; c < NC; c++) {
      const int b = c & 1;
      const uint32_t ph = c & 1;
      const float *f = m->f[b], *cc = m->c[b];
      ok &= wait(bar(m->tile_full[b]), (c >> 1) & 1, limit, gave_up);
      ok &= wait(bar(m->fac_full[b]), (c >> 1) & 1, limit, gave_up);
      const float2 sc = m->scales[b];
      ok &= wait(bar(m->mma1), ph, limit, gave_up);
      if (__any_sync(0xffffffffu, !ok)) break;
      tc::fence_after_sync();
      // R = V^T - f D1
      const float d1 = -1.0f / (sS * sc.x);  // (powers of two)
      m->o1[b][r] = a.scale / (sS * sc.y);
      float sR;
      {
        const uint8_t *V = sm + CH_VT + b * ROWS64;
        const u64 w1 = pack2(d1, d1);
        u64 R[C / 2];
#pragma unroll
        for (int h = 0; h < 4; h++) {
          float x[16];
          tc::tmem_ld16(tl + T_D1 + 16 * h, x);
          uint4 vr[2];
#pragma unroll
          for (int k = 0; k < 2; k++) vr[k] = *reinterpret_cast<const uint4 *>(V + vt_off(r, 2 * h + k));
          tc::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(f + 16 * h + k);
            const uint32_t w[2] = {k % 8 ? vr[k / 8].z : vr[k / 8].x, k % 8 ? vr[k / 8].w : vr[k / 8].y};
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const u64 vv = pack2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
              R[8 * h + k / 2 + e] = fma2(pack2(x[k + 2 * e], x[k + 2 * e + 1]), mul2(e ? ff.y : ff.x, w1), vv);
            }
          }
        }
        sR = tile_scale(pair_absmax(R));
        const u64 s2 = pack2(sR, sR);
#pragma unroll
        for (int k = 0; k < 2; k++) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; i++) {
            float p, q;
            unpack2(mul2(R[16 * k + i], s2), p, q);
            v[i] = half2_bits(p, q);
          }
          tc::tmem_st16(tl + T_D1 + 16 * k, v);
        }
        tc::tmem_st_wait();
      }
      tc::fence_before_sync();
      warp_arrive(m->r_ready);
      ok &= wait(bar(m->mma2), ph, limit, gave_up);
      if (__any_sync(0xffffffffu, !ok)) break;
      tc::fence_after_sync();
      // U, for the readout, and c U, for the state
      float sU;  // the operands hold U sU sR
      {
        u64 X[C / 2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float x[32];
          tc::tmem_ld32(tl + T_D2 + 32 * h, x);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; i++) X[16 * h + i] = pack2(x[2 * i], x[2 * i + 1]);
        }
        sU = tile_scale(pair_absmax(X));
        const u64 s2 = pack2(sU, sU);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float v[16], w[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(cc + 32 * h + 2 * k);
#pragma unroll
            for (int e = 0; e < 2; e++) {
              const u64 g = mul2(X[16 * h + k + e], s2);
              float p, q;
              unpack2(mul2(g, e ? ff.y : ff.x), p, q);
              w[k + e] = half2_bits(p, q);
              unpack2(g, p, q);
              v[k + e] = half2_bits(p, q);
            }
          }
          tc::tmem_st16(tl + T_D2 + 32 + 16 * h, w);
          tc::tmem_st16(tl + T_D2 + 16 * h, v);
        }
        tc::tmem_st_wait();
      }
      const float us = sU * sR, ku = 1.0f / (us * sc.x);
      m->o2[b][r] = a.scale * (ku / sc.y);
      tc::fence_before_sync();
      warp_arrive(m->u_ready);
      // the state after the chunk
      const u64 ds = pack2(ku, ku), dec = pack2(f[C - 1], f[C - 1]);
#pragma unroll
      for (int i = 0; i < D / 2; i++) S[i] = mul2(S[i], dec);
      ok &= wait(bar(m->mma3), ph, limit, gave_up);
      if (__any_sync(0xffffffffu, !ok)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int k = 0; k < 4; k++) {
        float x[32];
        tc::tmem_ld32(tl + T_DS + 32 * k, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i++) S[16 * k + i] = fma2(pack2(x[2 * i], x[2 * i + 1]), ds, S[16 * k + i]);
      }
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
    // ---- fetch, convert, transpose; write the readout ----
    regs_down<kRegHelper>();
    const int h = tid - 128;
    const uint32_t tl = tbase + ((uint32_t)(32 * (warp - 4)) << 16);
    auto convert = [&](int c) -> bool {  // chunk c into slot c & 1 (free: its last readout is out)
      const int b = c & 1, n = min(C, T - c * C);
      if (group_or(2, 128, !wait(bar(m->raw_full), c & 1, limit, gave_up))) return false;
      const uint8_t *raw = sm + CH_RAW;
      uint8_t *tile = sm + CH_TILE + b * TILE, *vt = sm + CH_VT + b * ROWS64;
      const int c8 = h & 15;
      auto row16 = [&](uint32_t base, int row) {
        return row < n ? *reinterpret_cast<const uint4 *>(raw + base + row * 256 + c8 * 16) : make_uint4(0, 0, 0, 0);
      };
#pragma unroll
      for (int p = 0; p < 4; p++) {  // tokens i, i + 1 of eight channels
        const int i = 2 * ((h >> 4) + 8 * p);
        const uint4 x = row16(2 * ROWS64, i), y = row16(2 * ROWS64, i + 1);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 8; e++)
          *reinterpret_cast<uint32_t *>(vt + vt_off(8 * c8 + e, i >> 3) + 2 * (i & 7)) =
              __byte_perm(xs[e / 2], ys[e / 2], e & 1 ? 0x7632 : 0x5410);
      }
      float mk = 0.0f, mq = 0.0f;
#pragma unroll
      for (int p = 0; p < 8; p++) {
        mk = fmaxf(mk, absmax8(row16(0, (h >> 4) + 8 * p)));
        mq = fmaxf(mq, absmax8(row16(ROWS64, (h >> 4) + 8 * p)));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
        mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, o));
      }
      if (lane == 0) {
        m->red[warp - 4] = mk;
        m->red[warp] = mq;
      }
      group_or(2, 128, false);
      const float sk = tile_scale(fmaxf(fmaxf(m->red[0], m->red[1]), fmaxf(m->red[2], m->red[3])));
      const float sq = tile_scale(fmaxf(fmaxf(m->red[4], m->red[5]), fmaxf(m->red[6], m->red[7])));
      if (h == 0) m->scales[b] = make_float2(sk, sq);
      const u64 sk2 = pack2(sk, sk), sq2 = pack2(sq, sq);
#pragma unroll 4
      for (int p = 0; p < 8; p++) {
        const int row = (h >> 4) + 8 * p;
        *reinterpret_cast<uint4 *>(tile + tile_off(row, c8, 128)) = to_half8(row16(0, row), sk2);
        *reinterpret_cast<uint4 *>(tile + tile_off(C + row, c8, 128)) = to_half8(row16(ROWS64, row), sq2);
      }
      tc::fence_smem_to_async();
      group_or(2, 128, false);  // (the raw rows are read, too)
      if (h == 0) mbar_arrive(bar(m->tile_full[b]));
      if (c + 1 < NC) {
        if (h == 0) fetch(c + 1);
        sent = c + 2;
      }
      return true;
    };
    float nonfinite[2] = {0.0f, 0.0f};  // NaN once an output was not finite
    ok = convert(0);
    for (int c = 0; c < NC && ok; c++) {
      const int b = c & 1;
      if (c + 1 < NC && !convert(c + 1)) {
        ok = false;
        break;
      }
      bool got = wait(bar(m->u_ready), c & 1, limit, gave_up);
      got &= wait(bar(m->mma4), c & 1, limit, gave_up);
      if (h == 0) tc::bulk_wait_read();  // the last chunk's output has left its buffer
      if (group_or(2, 128, !got)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const u64 w1 = pack2(m->o1[b][h], m->o1[b][h]), w2 = pack2(m->o2[b][h], m->o2[b][h]);
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
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(&m->f[b][32 * g + k]);
#pragma unroll
          for (int e = 0; e < 2; e++) {
            float p, q;
            unpack2(fma2(pack2(x[k + 2 * e], x[k + 2 * e + 1]), mul2(e ? ff.y : ff.x, w1),
                         mul2(pack2(y[k + 2 * e], y[k + 2 * e + 1]), w2)), p, q);
            nonfinite[0] = fmaf(p, 0.0f, nonfinite[0]);
            nonfinite[1] = fmaf(q, 0.0f, nonfinite[1]);
            __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(sm + CH_OUT) + (32 * g + k + 2 * e) * D + h;
            dst[0] = __float2bfloat16_rn(p);
            dst[D] = __float2bfloat16_rn(q);
          }
        }
      }
      tc::fence_smem_to_async();
      group_or(2, 128, false);
      if (h == 0) {
        bulk_s2g((__nv_bfloat16 *)a.out + v0 + (size_t)c * C * D, tc::smem_u32(sm + CH_OUT),
                 (uint32_t)min(C, T - c * C) * D * 2);
        tc::bulk_commit();
      }
    }
    if (!(nonfinite[0] + nonfinite[1] == 0.0f)) atomicOr(a.status, tc::kErrNonFinite);
    if (h == 0) tc::bulk_wait_all();
  } else if (warp < 12) {
    // ---- the factors, one chunk ahead of the chain ----
    regs_down<kRegFactor>();
    const int h = tid - 256, w = warp - 8;
    Factor &s = *reinterpret_cast<Factor *>(sm + CH_SCR);
    for (int b = 0; b < 2; b++) factor_clear(sm + CH_FAC + 2 * SQ * b, h);
    for (int c = 0; c < NC; c++) {
      const int b = c & 1, n = min(C, T - c * C);
      uint8_t *M = sm + CH_FAC + 2 * SQ * b, *P = M + SQ;
      const size_t t0 = g0 + (size_t)c * C;
      // (the last chunk's blocks are done with s: group barrier below)
      GatePair g;
      float be = 0.0f;
      if (w == 0) g = gate_scan(a.gamma + t0, n, lane);
      if (w >= 2) be = h - 64 < n ? a.beta[t0 + h - 64] : 0.0f;
      bool got = wait(bar(m->tile_full[b]), (c >> 1) & 1, limit, gave_up);
      // the products of chunk c come after those of chunk c - 2 in the tensor pipe, and its tile
      // after that chunk's readout: slot b is free
      got &= wait(bar(m->d0_full), c & 1, limit, gave_up);
      if (group_or(3, 128, !got)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (w == 0) factor_gates(s, g, m->f[b], m->c[b], lane);
      if (w >= 2) s.beta[h - 64] = be;
      group_or(3, 128, false);
      factor_rows(s, tbase + T_D0, m->scales[b].x, P, h, [&] {
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
        const uint32_t tile = tc::smem_u32(sm + CH_TILE + b * TILE), fac = tc::smem_u32(sm + CH_FAC + 2 * SQ * b);
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
          tc::mma_f16_ts(tbase + T_D2, tbase + T_D1 + 8 * s, tc::kmajor_desc(fac, C, s), id64, s > 0);
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
    if (tid == 128 && !tc::mbar_wait(bar(m->raw_full), (sent - 1) & 1, tc::kWaitLimit))
      atomicOr(a.status, tc::kErrDrainTimeout);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 512);
}

}  // namespace

int launch_rule_forward_tc(const RuleArgs &a, cudaStream_t st) {
  if (cudaFuncSetAttribute(mesa_rule_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CH_SMEM) !=
      cudaSuccess)
    return -1;
  timing_mark_begin(K_RULE_CHAIN, st);
  mesa_rule_chain_kernel<<<a.units(), 512, CH_SMEM, st>>>(a);
  timing_mark_end(K_RULE_CHAIN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mesa
