// gated_delta_tc.cu -- the gated delta rule's chunked forward on the tensor cores (bf16,
// dk = dv = 128; the chunk algebra and the operand formats are in gated_delta_tc.cuh).
//
// Two kernels.  mesa_rule_prep_kernel, one CTA per chunk: K K^T and Q K^T in one product, decays,
// masks and the triangular inverse, written as a record.  mesa_rule_chain_kernel, one CTA per
// unit, walks the unit's chunks with the state in registers (thread r of the chain holds row r,
// 128 values) and everything laid out by state row, so that a chunk's chain of dependent
// products never crosses threads:
//     D1 = S0 K^T          -> R = V^T - f D1      (row r of the accumulator is thread r's)
//     D2 = R (T beta)^T    -> U
//     dS = (c U) K         -> S = f_last S0 + dS
// with S0, R and U written back to tensor memory as the next product's A operand.  The readout
// O = f (S0 Q^T) + U P^T shares the first product (K and Q rows are one operand tile).  The chain
// bounds the kernel, so all else runs beside it, in warp groups of their own:
//     chain    the three epilogues above;
//     helper   transposes V one chunk ahead, writes the readout of the chunk before;
//     convert  K and Q as fp16 operands, up to three chunks ahead.
// (With the preparation in the same kernel, as a fourth group, nothing but the inputs and the output
// went to memory, but the groups' code no longer fitted the instruction caches and every
// group slowed down: 268 us at 8 x 16 x 4096 against the two kernels' time below.)
#include "gated_delta_tc.cuh"

namespace mesa {

using namespace rule;

namespace {

// ---- per-chunk preparation --------------------------------------------------------------------
// shared memory: the operand tile, and once its products are done record | scratch in its place
// (39 KB: five CTAs on an SM hide each other's substitution) | misc
constexpr uint32_t PR_REC = 0, PR_SCR = REC_PAD;
constexpr uint32_t PR_MISC = (PR_SCR + sizeof(Factor) > TILE ? PR_SCR + sizeof(Factor) : TILE);
static_assert(PR_MISC % 16 == 0, "misc alignment");
struct PrepMisc {
  alignas(16) uint32_t red[8];
  uint64_t mbar, drain;
  uint32_t tmem;
};
constexpr uint32_t PR_SMEM = PR_MISC + sizeof(PrepMisc) + 1024;

// grid (NC, U), 128 threads.  WITH_BETA: the record's factor is T diag(beta), else T.
// Measured (8 x 16 x 4096, 8192 chunks): see the table at the launch.
template <bool WITH_BETA>
__global__ void __launch_bounds__(128, 5) mesa_rule_prep_kernel(RuleArgs a, uint8_t *records) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  PrepMisc *m = reinterpret_cast<PrepMisc *>(sm + PR_MISC);
  Factor &s = *reinterpret_cast<Factor *>(sm + PR_SCR);
  uint8_t *rec = sm + PR_REC;
  float *nf = reinterpret_cast<float *>(rec + REC_F), *cc = nf + C, *inv = reinterpret_cast<float *>(rec + REC_S);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int c = blockIdx.x, u = blockIdx.y, NC = gridDim.x, t0 = c * C, n = min(C, a.T - t0);
  const size_t row0 = (size_t)a.qk_unit(u) * a.T + t0, tok0 = (size_t)u * a.T + t0;

  // rows of K and Q: 16 threads a row, 8 rows a pass
  const int r0 = tid >> 4, c8 = tid & 15;
  uint4 x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    x[i] = y[i] = make_uint4(0, 0, 0, 0);
    if (8 * i + r0 < n) {
      x[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.k + (row0 + r0 + 8 * i) * D + 8 * c8);
      y[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.q + (row0 + r0 + 8 * i) * D + 8 * c8);
    }
  }
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 64);
  if (tid == 32) {
    tc::mbar_init(tc::smem_u32(&m->mbar), 1);
    tc::mbar_init(tc::smem_u32(&m->drain), 1);
  }
  const float be = tid < n && tid < C ? a.beta[tok0 + tid] : 0.0f;
  GatePair g;
  if (warp == 3) {
    const float *gp = a.gamma + tok0;
    g = gate_scan(make_float2(2 * lane < n ? gp[2 * lane] : 1.0f, 2 * lane + 1 < n ? gp[2 * lane + 1] : 1.0f), lane);
  }
  uint32_t mk = 0, mq = 0;
#pragma unroll
  for (int k = 0; k < 8; k++) {
    mk = absmax_words(mk, x[k]);
    mq = absmax_words(mq, y[k]);
  }
  mk = absmax_fold(mk);
  mq = absmax_fold(mq);
  if (lane == 0) {
    m->red[warp] = mk;
    m->red[4 + warp] = mq;
  }
  __syncthreads();
  const uint4 k4 = *reinterpret_cast<const uint4 *>(m->red), q4 = *reinterpret_cast<const uint4 *>(m->red + 4);
  float ik, iq;
  const float sk = bound_scale(__uint_as_float(max(max(k4.x, k4.y), max(k4.z, k4.w)) << 16), kTopTile, ik);
  const float sq = bound_scale(__uint_as_float(max(max(q4.x, q4.y), max(q4.z, q4.w)) << 16), kTopTile, iq);
  const u64 sk2 = pack2(sk, sk), sq2 = pack2(sq, sq);
  uint8_t *dst = sm + tile_off(r0, c8, 128);
#pragma unroll
  for (int k = 0; k < 8; k++) {
    *reinterpret_cast<uint4 *>(dst + 1024 * k) = to_half8(x[k], sk2);
    *reinterpret_cast<uint4 *>(dst + C * 128 + 1024 * k) = to_half8(y[k], sq2);
  }
  tc::fence_smem_to_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = __shfl_sync(0xffffffffu, m->tmem, 0), bar = tc::smem_u32(&m->mbar);
  if (warp == 0 && elect_one()) {  // rows 0..63: K K^T, rows 64..127: Q K^T
    const uint32_t id = tc::idesc_f16(128, C, false, false);
    const uint64_t t = tc::kmajor_desc(tc::smem_u32(sm), 128, 0);
#pragma unroll
    for (int k = 0; k < 8; k++) tc::mma_f16(tbase, t + step128(k), t + step128(k), id, k > 0);
    tc::mma_commit(bar);
  }
  const bool done = tc::mbar_wait(bar, 0, a.wait_limit);
  tc::fence_after_sync();
  if (__syncthreads_or(!done)) {
    if (tid == 0) atomicOr(a.status, tc::kErrMmaTimeout);
    const bool issuer = warp == 0 && elect_one();
    tc::drain_mmas(tc::smem_u32(&m->drain), issuer, a.status);
  } else {
    if (tid == 0) *reinterpret_cast<float4 *>(inv) = make_float4(ik, iq, sk, sq);
    if (tid < C) s.beta[tid] = reinterpret_cast<float *>(rec + REC_B)[tid] = be;
    if (warp == 3) factor_gates(s, g, nf, cc, lane);
    factor_clear(rec, tid);
    factor_clear(rec + SQ, tid);
    __syncthreads();
    factor_rows(s, tbase, ik * ik, rec + SQ, tid);
    tc::fence_before_sync();
    __syncthreads();
    factor_diagonal<WITH_BETA>(s, rec, warp, lane);
    __syncthreads();
    if (warp < 3) factor_columns<WITH_BETA>(s, rec, warp, lane);
    tc::fence_smem_to_async();
    __syncthreads();
    if (tid == 0) {
      bulk_s2g(records + ((size_t)u * NC + c) * REC, tc::smem_u32(rec), REC);
      tc::bulk_commit();
      tc::bulk_wait_all();
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 64);
}

// ---- the chain ----------------------------------------------------------------------------------
// shared memory: three records | V^T in fp32 | V | output | K, Q operand tiles (three; two when the states
// are kept, and a tile for their way out) | misc
constexpr uint32_t CH_REC = 0, CH_VT = CH_REC + 3 * REC_PAD, CH_V = CH_VT + 2 * ROWS64;
constexpr uint32_t CH_OUT = CH_V + ROWS64, CH_TILE = CH_OUT + ROWS64, CH_STAGE = CH_TILE + 2 * TILE, CH_MISC = CH_TILE + 3 * TILE;
struct ChainMisc {
  float o1[2][D], o2[2][D];     // units of the readout's accumulators, by state row
  float vmax[4];              // largest |v| of 32 channels
  float bmax[4], umax[2][4];  // by chain warp: bounds of the state, of |u|
  uint64_t tile_full[3], tile_free[3], rec_full[3], v_full, vt_full, r_ready, u_ready, o_free;
  uint64_t mma1, mma2, mma3, mma4, drain;
  uint32_t tmem;
  int gave_up;
};
constexpr uint32_t CH_SMEM = CH_MISC + sizeof(ChainMisc) + 1024;
static_assert(CH_SMEM <= 232448, "shared memory per block");
// tensor memory columns: dS | S0 operand | D1 (then R, c U and U), O from S0 | D2 | O from U
constexpr uint32_t T_DS = 0, T_S = 128, T_D1 = 192, T_O1 = 256, T_D2 = 320, T_O2 = 384;
constexpr uint32_t T_R = T_D1, T_CU = T_D1, T_U = T_D1 + 32;  // two values a column, each over what has been read

// Offset of tokens 4 ch .. 4 ch + 3 of channel r in the transposed fp32 values (256 bytes a
// channel; permuted so that neither the writes nor a warp's reads of 32 channels meet in a bank).
__device__ __forceinline__ uint32_t vt_off(int r, int ch) { return (uint32_t)(r * 256 + ((ch ^ (r & 7)) << 4)); }

__device__ __forceinline__ uint32_t bf2_bits(u64 x) {  // two bf16 values
  float a, b;
  unpack2(x, a, b);
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Register shares of the three warp groups; the block is launched with 168 a thread.
constexpr int kRegChain = 240, kRegHelper = 136, kRegConvert = 120;
static_assert(kRegChain + kRegHelper + kRegConvert <= 3 * 168, "register file");

// grid U, 384 threads: warps 0-3 chain, 4-7 helper, 8-11 convert.
// FWD: the forward; the records hold T diag(beta).  Otherwise the backward's pass over the states: the
// records hold T, nothing is read out, and the state before each chunk and the chunk's u are kept as
// operands with one scale each (so.S, so.U).
template <bool FWD>
__global__ void __launch_bounds__(384, 1)
    mesa_rule_chain_kernel(RuleArgs a, const uint8_t *records, RuleOperands so, const __grid_constant__ CUtensorMap mapV,
                           const __grid_constant__ CUtensorMap mapO) {
  constexpr int NT = FWD ? 3 : 2;  // operand tiles
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
  auto fetch_rec = [&](int c) {
    const uint32_t b = bar(m->rec_full[c % 3]);
    tc::mbar_arrive_expect_tx(b, REC);
    tc::bulk_g2s(tc::smem_u32(sm + CH_REC + (c % 3) * REC_PAD), records + ((size_t)u * NC + c) * REC, REC, b);
  };
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 128) {
    for (uint64_t *b : {&m->vt_full, &m->r_ready, &m->u_ready, &m->o_free, &m->tile_full[0], &m->tile_full[1], &m->tile_full[2]})
      tc::mbar_init(bar(*b), 4);
    for (uint64_t *b : {&m->tile_free[0], &m->tile_free[1], &m->tile_free[2], &m->rec_full[0], &m->rec_full[1],
                        &m->rec_full[2], &m->v_full, &m->mma1, &m->mma2, &m->mma3, &m->mma4})
      tc::mbar_init(bar(*b), 1);
    tc::mbar_init(bar(m->drain), FWD ? 2 : 1);  // the threads that issue products
    m->gave_up = 0;
    fetch_v(0);
    for (int c = 0; c < min(NC, 3); c++) fetch_rec(c);
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
  int v_sent = 1, rec_sent = min(NC, 3);  // fetches issued (thread 128)

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
    // the bound that scales the operand: the row's, or that of all rows where the operand is kept
    auto all_rows = [&](float b) -> float {  // after a barrier that follows put_rows
      const float4 x = *reinterpret_cast<const float4 *>(m->bmax);
      return FWD ? b : fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
    };
    auto put_rows = [&](float b) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(b));
      if (lane == 0) m->bmax[warp] = __uint_as_float(w);
    };
    auto keep_words = [&](int k, const float (&v)[8]) {  // columns 16 k .. of this row, on their way out
      *reinterpret_cast<float4 *>(sm + CH_STAGE + tile_off(r, 2 * k, 128)) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(sm + CH_STAGE + tile_off(r, 2 * k + 1, 128)) = make_float4(v[4], v[5], v[6], v[7]);
    };
    if constexpr (!FWD) {
      put_rows(bS);
      group_or(1, 128, false);
    }
    {
      const float sS = bound_scale(all_rows(bS), kTopRow, iS);
      const u64 s2 = pack2(sS, sS);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = half2_bits(mul2(S[8 * k + i], s2));
        tc::tmem_st8(tl + T_S + 8 * k, v);
        if constexpr (!FWD) keep_words(k, v);
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
      const uint32_t ph = c & 1, tile = tc::smem_u32(sm + CH_TILE + (c % NT) * TILE),
                     rec = tc::smem_u32(sm + CH_REC + (c % 3) * REC_PAD);
      const float *nf = reinterpret_cast<const float *>(sm + CH_REC + (c % 3) * REC_PAD + REC_F), *cc = nf + C,
                  *inv = reinterpret_cast<const float *>(sm + CH_REC + (c % 3) * REC_PAD + REC_S);
      ok &= wait(bar(m->tile_full[c % NT]), (c / NT) & 1, limit, gave_up);
      if (c > 0) ok &= wait(bar(m->o_free), (c - 1) & 1, limit, gave_up);  // (the last readout is read)
      if constexpr (!FWD) tc::fence_smem_to_async();
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t kq = tc::kmajor_desc(tile, 128, 0);
#pragma unroll
        for (int s = 0; s < 8; s++)  // S0 K^T and S0 Q^T (one product), or the first alone
          tc::mma_f16_ts(tbase + T_D1, tbase + T_S + 8 * s, kq + step128(s), FWD ? id128 : id64, s > 0);
        tc::mma_commit(bar(m->mma1));
      }
      if constexpr (!FWD) {
        if (r == 32) {
          bulk_s2g(so.S + ((size_t)u * NC + c) * TILE, tc::smem_u32(sm + CH_STAGE), TILE);
          tc::bulk_commit();
          so.iS[(size_t)u * NC + c] = iS;
        }
      }
      ok &= wait(bar(m->rec_full[c % 3]), (c / 3) & 1, limit, gave_up);
      ok &= wait(bar(m->vt_full), ph, limit, gave_up);
      const float iK = inv[0], kmax = (float)(1 << kTopTile) * iK, all = -nf[C - 1];  // all: the chunk's decay
      if constexpr (FWD) m->o1[ph][r] = -a.scale * iS * inv[1];
      const float w1 = iS * iK;  // units of D1
      float iR;
      const float sR = bound_scale(fmaf((float)D * kmax, bS, m->vmax[warp]), FWD ? kTopRow : kTopRow - 2, iR);  // (beta < 4)
      const u64 w1_2 = pack2(w1, w1), sR2 = pack2(sR, sR);
      const float *be = cc + C;
      if constexpr (!FWD) m->o1[ph][r] = iR;
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
            ulonglong2 bb = make_ulonglong2(sR2, sR2);
            if constexpr (!FWD) {
              bb = *reinterpret_cast<const ulonglong2 *>(be + 16 * h + 4 * k);
              bb = make_ulonglong2(mul2(bb.x, sR2), mul2(bb.y, sR2));
            }
            v[2 * k] = half2_bits(mul2(fma2(pack2(z[4 * k], z[4 * k + 1]), mul2(ff[k].x, w1_2), vv[k].x), bb.x));
            v[2 * k + 1] = half2_bits(mul2(fma2(pack2(z[4 * k + 2], z[4 * k + 3]), mul2(ff[k].y, w1_2), vv[k].y), bb.y));
          }
          // (columns 8 h .. 8 h + 7: read by now)
          tc::tmem_st8(tl + T_R + 8 * h, v);
        }
      }
      tc::tmem_st_wait();
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t fm = tc::kmajor_desc(rec, C, 0);
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
          if constexpr (FWD) tc::tmem_st8(tl + T_U + 8 * h, v);
        }
        tc::tmem_st_wait();
      }
      const float w3 = iU * iR * iK;  // units of dS
      // 64 products of |c u| <= |u| and |k| bound what is added to the state
      bS = fmaf(all, bS, (float)C * uU * iR * kmax);
      if constexpr (FWD) {
        m->o2[ph][r] = a.scale * w3 * inv[1];
      } else {
        put_rows(bS);
        const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(uU * iR));
        if (lane == 0) m->umax[ph][warp] = __uint_as_float(w);
        if (r == 32) tc::bulk_wait_read();  // the kept state has left its tile
      }
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t kt = tc::mnmajor_desc(tile, 128, 0);
#pragma unroll
        for (int s = 0; s < 4; s++) tc::mma_f16_ts(tbase + T_DS, tbase + T_CU + 8 * s, kt + step_mn(s), idKN, s > 0);
        tc::mma_commit(bar(m->mma3));
      }
      warp_arrive(m->u_ready);  // (and the record has been read)
      // the state after the chunk
      const u64 w3_2 = pack2(w3, w3);
      const float sS = bound_scale(all_rows(bS), kTopRow, iS);
      const u64 sS2 = pack2(sS, sS);
      const u64 dec = pack2(all, all);
      ok &= wait(bar(m->mma3), ph, limit, gave_up);
      tc::fence_after_sync();
      if (r == 0) mbar_arrive(bar(m->tile_free[c % NT]));
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
          if constexpr (!FWD) keep_words(k, v);
        }
        tc::tmem_st_wait();
      }
      if ((c & 7) == 7) row_max();  // (before the bound is loose)
    }
    if constexpr (!FWD) {
      if (r == 32) tc::bulk_wait_all();
    }
    if (!group_or(1, 128, !ok) && FWD && a.S_final) {
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
      bool got = wait(bar(m->rec_full[c % 3]), (c / 3) & 1, limit, gave_up);
      got &= wait(bar(m->u_ready), c & 1, limit, gave_up);
      got = __all_sync(0xffffffffu, got);
      tc::fence_after_sync();
      if (FWD && warp == 4 && got && elect_one()) {  // U P^T
        const uint64_t pd = tc::kmajor_desc(tc::smem_u32(sm + CH_REC + (c % 3) * REC_PAD + REC_P), C, 0);
#pragma unroll
        for (int s = 0; s < 4; s++) tc::mma_f16_ts(tbase + T_O2, tbase + T_U + 8 * s, pd + step64(s), id64, s > 0);
        tc::mma_commit(bar(m->mma4));
      }
      if constexpr (FWD) got &= wait(bar(m->mma4), c & 1, limit, gave_up);
      if (h == 0) tc::bulk_wait_read();  // the last chunk's output has left its buffer
      if (group_or(2, 128, !got)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      const float *nf = reinterpret_cast<const float *>(sm + CH_REC + (c % 3) * REC_PAD + REC_F);
      // 16 channels at a time in fragments of 8 tokens (this thread: channels T / 4 and T / 4 + 8, tokens
      // 2 (T % 4) and the next of each 8), transposed into the swizzled output tile
      constexpr uint32_t first = FWD ? T_O1 : T_D2;
      float x[2][32];  // from S0: all at once, the chain's next product writes there
      tmem_ld_frag64(tl + first, x[0]);
      tmem_ld_frag64(tl + (16u << 16) + first, x[1]);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      warp_arrive(m->o_free);
      const int w = warp - 4, q = 2 * (lane & 3);
      float su = 1.0f, iu = 1.0f;
      if constexpr (!FWD) {
        const float4 b = *reinterpret_cast<const float4 *>(m->umax[c & 1]);
        su = bound_scale(fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)), kTopRow, iu);
      }
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        float y[32];
        if constexpr (FWD) tmem_ld_frag64(tl + ((uint32_t)(16 * hf) << 16) + T_O2, y);
        const int ch = 32 * w + 16 * hf + (lane >> 2);
        const float r1 = m->o1[c & 1][ch] * su, r2 = m->o1[c & 1][ch + 8] * su;
        const u64 a1 = pack2(r1, r1), b1 = pack2(r2, r2), a2 = pack2(m->o2[c & 1][ch], m->o2[c & 1][ch]);
        const u64 b2 = pack2(m->o2[c & 1][ch + 8], m->o2[c & 1][ch + 8]);
        // rows of the four blocks of a store: tokens 16 p + 8 (lane / 16) + lane % 8, channels + 8 ((lane / 8) % 2)
        const int tk = 8 * (lane >> 4) + (lane & 7), c8 = 4 * w + 2 * hf + ((lane >> 3) & 1);
        tc::tmem_ld_wait();
        const float *z = x[hf];
#pragma unroll
        for (int p = 0; p < 4; p++) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int j = 8 * p + 4 * e;
            if constexpr (!FWD) {
              o[2 * e] = __float_as_uint(half2_bits(mul2(pack2(z[j], z[j + 1]), a1)));
              o[2 * e + 1] = __float_as_uint(half2_bits(mul2(pack2(z[j + 2], z[j + 3]), b1)));
              continue;
            }
            const u64 ff = *reinterpret_cast<const u64 *>(nf + 16 * p + 8 * e + q);
            const u64 oa = fma2(pack2(z[j], z[j + 1]), mul2(ff, a1), mul2(pack2(y[j], y[j + 1]), a2));
            const u64 ob = fma2(pack2(z[j + 2], z[j + 3]), mul2(ff, b1), mul2(pack2(y[j + 2], y[j + 3]), b2));
            nonfinite = fma2(oa, 0ull, fma2(ob, 0ull, nonfinite));
            o[2 * e] = bf2_bits(oa);
            o[2 * e + 1] = bf2_bits(ob);
          }
          stmatrix_x4_trans(tc::smem_u32(sm + CH_OUT + tile_off(16 * p + tk, c8, C)), o[0], o[1], o[2], o[3]);
        }
      }
      tc::fence_before_sync();
      tc::fence_smem_to_async();
      group_or(2, 128, false);
      if (h == 0) {
        if constexpr (FWD) {
#pragma unroll
          for (int b = 0; b < 2; b++) tensor_s2g_3d(&mapO, tc::smem_u32(sm + CH_OUT + b * C * 128), 64 * b, c * C, u);
        } else {
          bulk_s2g(so.U + ((size_t)u * NC + c) * ROWS64, tc::smem_u32(sm + CH_OUT), ROWS64);
          so.iU[(size_t)u * NC + c] = iu;
        }
        tc::bulk_commit();
        if (c + 3 < NC) fetch_rec(c + 3);  // (the chain is past this record, and so is the group)
      }
      if (c + 3 < NC) rec_sent++;
    }
    if (!(sum2(nonfinite) == 0.0f)) atomicOr(a.status, tc::kErrNonFinite);
    if (h == 0) tc::bulk_wait_all();
  } else {
    // ---- K and Q as operands, up to three chunks in flight ----
    regs_down<kRegConvert>();
    const int h = tid - 256, r0 = h >> 4, c8 = h & 15, uk = a.qk_unit(u);  // rows r0, r0 + 8 ..; 8 channels
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
          if (FWD) y[i] = *reinterpret_cast<const uint4 *>(qp + ((size_t)c * C + 8 * i) * D);
        }
      }
    };
    load(0);
    for (int c = 0; c < NC; c++) {
      bool got = wait(bar(m->rec_full[c % 3]), (c / 3) & 1, limit, gave_up);
      if (c >= NT) got &= wait(bar(m->tile_free[c % NT]), (c / NT - 1) & 1, limit, gave_up);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      const float4 inv = *reinterpret_cast<const float4 *>(sm + CH_REC + (c % 3) * REC_PAD + REC_S);
      const u64 sk2 = pack2(inv.z, inv.z), sq2 = pack2(inv.w, inv.w);
      uint8_t *dst = sm + CH_TILE + (c % NT) * TILE + tile_off(r0, c8, 128);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        *reinterpret_cast<uint4 *>(dst + 1024 * k) = to_half8(x[k], sk2);
        if (FWD) *reinterpret_cast<uint4 *>(dst + C * 128 + 1024 * k) = to_half8(y[k], sq2);
      }
      tc::fence_smem_to_async();
      warp_arrive(m->tile_full[c % NT]);
      if (c + 1 < NC) load(c + 1);
    }
  }
  if (!ok) *gave_up = 1;
  __syncthreads();
  // a wait gave up: products and copies still in flight finish before the memory is released
  if (*gave_up) {
    // (a product's commit counts for the thread that issued it: the same elected lane)
    if ((warp == 0 || (FWD && warp == 4)) && elect_one()) tc::mma_commit(bar(m->drain));
    if (tid == 0) {
      unsigned bits = tc::kErrMmaTimeout;
      if (!tc::mbar_wait(bar(m->drain), 0, tc::kWaitLimit)) bits |= tc::kErrDrainTimeout;
      atomicOr(a.status, bits);
    }
    if (tid == 128) {
      bool in = tc::mbar_wait(bar(m->v_full), (v_sent - 1) & 1, tc::kWaitLimit);
      for (int c = max(0, rec_sent - 3); c < rec_sent; c++)
        in &= tc::mbar_wait(bar(m->rec_full[c % 3]), (c / 3) & 1, tc::kWaitLimit);
      if (!in) atomicOr(a.status, tc::kErrDrainTimeout);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 512);
}

template <bool FWD>
int launch_chain(const RuleArgs &a, const uint8_t *records, const RuleOperands &so, const CUtensorMap &mapV,
                 const CUtensorMap &mapO, cudaStream_t st) {
  auto kfn = mesa_rule_chain_kernel<FWD>;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CH_SMEM) != cudaSuccess) return -1;
  timing_mark_begin(K_RULE_CHAIN, st);
  kfn<<<a.units(), 384, CH_SMEM, st>>>(a, records, so, mapV, mapO);
  timing_mark_end(K_RULE_CHAIN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

size_t rule_tc_workspace(int U, int T) {
  return (size_t)U * (((size_t)T + C - 1) / C) * REC;
}

int launch_rule_prep(const RuleArgs &a, void *records, bool with_beta, cudaStream_t st) {
  auto kfn = with_beta ? mesa_rule_prep_kernel<true> : mesa_rule_prep_kernel<false>;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PR_SMEM) != cudaSuccess) return -1;
  timing_mark_begin(K_RULE_PREP, st);
  kfn<<<dim3((a.T + C - 1) / C, a.units()), 128, PR_SMEM, st>>>(a, (uint8_t *)records);
  timing_mark_end(K_RULE_PREP, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int launch_rule_forward_tc(const RuleArgs &a, void *workspace, cudaStream_t st) {
  CUtensorMap mapV{}, mapO{};
  if (!tmap_units128_bf16(&mapV, a.v, a.units(), a.T) || !tmap_units128_bf16(&mapO, a.out, a.units(), a.T)) return -1;
  if (launch_rule_prep(a, workspace, true, st) != 0) return -1;
  return launch_chain<true>(a, (const uint8_t *)workspace, RuleOperands{}, mapV, mapO, st);
}

int launch_rule_states_tc(const RuleArgs &a, const void *records, const RuleOperands &so, cudaStream_t st) {
  CUtensorMap mapV{};
  if (!tmap_units128_bf16(&mapV, a.v, a.units(), a.T)) return -1;
  return launch_chain<false>(a, (const uint8_t *)records, so, mapV, mapV, st);
}

}  // namespace mesa
