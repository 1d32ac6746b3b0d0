// gated_delta_bwd_tc.cu -- the gated delta rule's backward on the tensor cores (bf16, dk = dv = 128;
// the chunk algebra, the records and the operand formats are in gated_delta_tc.cuh).
//
// After the records (T without beta) and a pass over the states (mesa_rule_chain_kernel<kKeep>, which
// keeps the state S0 before each chunk and the chunk's u), two kernels:
//  - mesa_rule_adjoint_kernel, one CTA per unit (or segment of a unit), walks the chunks backwards with the adjoint A of the
//    state after the chunk in registers, like the forward's chain (g = dL/do, scale in P and Q):
//        R' = (c A K^T + g^T P),   du = R' T,   A <- f_last A + g^T (f Q) - (beta f du)^T K;
//  - mesa_rule_grads_tc_kernel, a resident CTA per SM over all chunks, takes every gradient from S0, A, u, du and the
//    chunk's rows:
//        W = g u^T o D, V = beta du u^T o D (strictly lower),
//        dq = f (g S0) + W K,   dk = W^T Q - (V + V^T) K + c (u A) - f beta (du S0),
//        dv = beta du,          dbeta = du . (v - f S0 k - sum_j D_ij (k_i . k_j) u_j),
//        dgamma_t: every pair (reader i >= t or the state after, writer j < t or the state before)
//        that the gate separates, with the decay between them but for gamma_t's own.
// States, adjoints, u and du go through memory as fp16 operands with one scale a chunk (2^-12 of a
// chunk's largest).  Measured at 8 x 16 x 4096: records 122 us, states 155, adjoint 217 (64 dependent steps of
// 3.4 us), gradients 461 (1.7 GB of operands, rows and gradients: 3.7 TB/s); each bound by the latency of
// its dependent steps on one CTA per SM, the last also by shared memory (its products' operands).
#include "gated_delta_tc.cuh"

namespace mesa {

using namespace rule;

namespace {

constexpr int kRegChain = 240, kRegHelper = 112, kRegConvert = 144;
static_assert(kRegChain + kRegHelper + kRegConvert <= 3 * 168, "register file");

// ---- the adjoint chain ----------------------------------------------------------------------------
// shared memory: three records | two operand tiles (K, f Q) | two g tiles | kept adjoint | du | misc
constexpr uint32_t AD_REC = 0, AD_TILE = 3 * REC_PAD, AD_G = AD_TILE + 2 * TILE, AD_STAGE = AD_G + 2 * ROWS64;
constexpr uint32_t AD_OUT = AD_STAGE + TILE, AD_MISC = AD_OUT + ROWS64;
struct AdjointMisc {
  float iR[2][D];             // units of D2, by row
  float bmax[4], umax[2][4];  // by chain warp: bounds of the adjoint, of |du|
  alignas(16) uint32_t red[8];
  float ig[2];                // 1 / scale of the g tiles
  uint64_t tile_full[2], tile_free[2], rec_full[3], r_ready, u_ready, o_free, upd, dp_full, dq_full;
  uint64_t mma1, mma2, mma3, drain;
  float rest, rest0;  // a bound of what the chunks after can give, of the part of dS_final that can come through
  uint32_t tmem;
  int gave_up;
};
constexpr uint32_t AD_SMEM = AD_MISC + sizeof(AdjointMisc) + 1024;
static_assert(AD_SMEM <= 232448, "shared memory per block");
// tensor memory columns: (beta f du) K | g^T (f Q) | A operand | D1 (then R', then -beta f du) | g^T P | D2
constexpr uint32_t T_DS = 0, T_DQ = 128, T_S = 256, T_D1 = 320, T_DP = 384, T_D2 = 448;
constexpr uint32_t T_R = T_D1, T_CU = T_D1;

// grid (U, segments), 384 threads: warps 0-3 chain (thread r: row r of A), 4-7 write du, 8-11 convert.
// SEG, grid (U, segments - 1): what the segments from 1 on give from an adjoint of zero after them (the last: from
// dS_final), nothing kept.  `tail`: of the chunks at the segment's start only those of whose end 2^-40 of an
// adjoint comes through, all there is when the bounds of what follows say that it adds less than 2^-26 of each
// row's largest element (as for the states); not tail: the segments where it was not, in full.
template <bool SEG>
__global__ void __launch_bounds__(384, 1)
    mesa_rule_adjoint_kernel(RuleArgs a, const uint8_t *records, RuleOperands ao, RuleSegments sg, bool tail) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  AdjointMisc *m = reinterpret_cast<AdjointMisc *>(sm + AD_MISC);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // (warp: uniform)
  const int u = blockIdx.x, seg = blockIdx.y + (SEG ? 1 : 0), T = a.T, NCT = (T + C - 1) / C;
  const int c0 = sg.n > 1 ? seg * sg.per : 0;
  int NC = sg.n > 1 ? min(NCT - c0, sg.per) : NCT;  // this CTA's chunks, from c0 on
  const float *start = !SEG && sg.n > 1 ? sg.A + ((size_t)u * sg.n + seg) * D * D  // (nullptr: zero)
                       : a.dS_final && (!SEG || seg == sg.n - 1) ? a.dS_final + (size_t)u * D * D
                                                                 : nullptr;
  if constexpr (SEG) {
    int *whole = sg.whole_adj + (size_t)u * sg.n + seg;
    if (tail) {
      const float2 *left_of = sg.bounds + (size_t)u * NCT;
      float left = 0.0f;
      int n = 0;
      while (n < NC && !(left <= kLittle)) left += left_of[c0 + n++].x;
      if (!(left <= kLittle)) {
        if (tid == 0) *whole = 1;
        return;
      }
      NC = n;
      start = nullptr;
      if (warp == 11) {  // what the chunks after can give: four a lane
        float rest = 0.0f;
        for (int j0 = c0 + NC; j0 < NCT; j0 += 128) {
          const int j = j0 + 4 * lane;
          float l[4], b[4], mine = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            l[i] = j + i < NCT ? left_of[j + i].x : 0.0f;
            b[i] = j + i < NCT ? sg.adds[(size_t)u * NCT + j + i] : 0.0f;
            mine += l[i];
          }
          float run = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += x;
          }
          const float total = __shfl_sync(0xffffffffu, run, 31);
          float before = left + __shfl_up_sync(0xffffffffu, run, 1);
          if (lane == 0) before = left;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            rest = fmaf(b[i], exp2f(before), rest);
            before += l[i];
          }
          left += total;
        }
        rest = warp_sum(rest);
        if (lane == 0) {
          m->rest = rest;
          m->rest0 = exp2f(left);  // of dS_final
        }
      }
    } else if (!*whole) {
      return;
    }
  }
  const int last = c0 + NC - 1;
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  volatile int *gave_up = &m->gave_up;
  const unsigned limit = a.wait_limit;
  // step it works on chunk last - it
  auto fetch_rec = [&](int it) {
    const uint32_t b = bar(m->rec_full[it % 3]);
    tc::mbar_arrive_expect_tx(b, REC);
    tc::bulk_g2s(tc::smem_u32(sm + AD_REC + (it % 3) * REC_PAD), records + ((size_t)u * NCT + last - it) * REC, REC, b);
  };
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 128) {
    for (uint64_t *b : {&m->tile_full[0], &m->tile_full[1], &m->r_ready, &m->u_ready, &m->o_free, &m->upd})
      tc::mbar_init(bar(*b), 4);
    for (uint64_t *b : {&m->tile_free[0], &m->tile_free[1], &m->rec_full[0], &m->rec_full[1], &m->rec_full[2], &m->dp_full,
                        &m->dq_full, &m->mma1, &m->mma2, &m->mma3})
      tc::mbar_init(bar(*b), 1);
    tc::mbar_init(bar(m->drain), 2);  // the threads that issue products
    m->gave_up = 0;
    for (int it = 0; it < min(NC, 3); it++) fetch_rec(it);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = __shfl_sync(0xffffffffu, m->tmem, 0);
  auto warp_arrive = [&](uint64_t &b) {  // one arrival per warp, after what its lanes did
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  bool ok = true;
  int rec_sent = min(NC, 3);  // fetches issued (thread 128)

  if (warp < 4) {
    regs_up<kRegChain>();
    const int r = tid;
    const uint32_t tl = tbase + ((uint32_t)(32 * warp) << 16);
    u64 S[D / 2];
    {
      const float4 *src = start ? reinterpret_cast<const float4 *>(start + (size_t)r * D) : nullptr;
#pragma unroll
      for (int g = 0; g < D / 4; g++) {
        const float4 x = src ? src[g] : make_float4(0, 0, 0, 0);
        S[2 * g] = pack2(x.x, x.y);
        S[2 * g + 1] = pack2(x.z, x.w);
      }
    }
    float bS, iS;  // a bound of the row's elements; 1 / scale of the operand (the same for all rows)
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
    auto all_rows = [&]() -> float {  // after a barrier that follows put_rows
      const float4 x = *reinterpret_cast<const float4 *>(m->bmax);
      return fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
    };
    auto put_rows = [&](float b) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(b));
      if (lane == 0) m->bmax[warp] = __uint_as_float(w);
    };
    auto keep_words = [&](int k, const float (&v)[8]) {  // columns 16 k .. of this row
      tc::tmem_st8(tl + T_S + 8 * k, v);
      if constexpr (SEG) return;
      *reinterpret_cast<float4 *>(sm + AD_STAGE + tile_off(r, 2 * k, 128)) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(sm + AD_STAGE + tile_off(r, 2 * k + 1, 128)) = make_float4(v[4], v[5], v[6], v[7]);
    };
    row_max();
    put_rows(bS);
    group_or(1, 128, false);
    {
      const float sS = bound_scale(all_rows(), kTopRow, iS);
      const u64 s2 = pack2(sS, sS);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = half2_bits(mul2(S[8 * k + i], s2));
        keep_words(k, v);
      }
      tc::tmem_st_wait();
    }
    const uint32_t id64 = tc::idesc_f16(128, C, false, false);    // N = 64, B K-major
    const uint32_t id64n = tc::idesc_f16(128, C, false, true);    // N = 64, B MN-major
    const uint32_t idKN = tc::idesc_f16(128, D, false, true);     // N = 128, B MN-major
    auto meet = [&]() -> bool {  // barrier of the chain; true when a wait gave up
      tc::fence_before_sync();
      const bool stop = group_or(1, 128, !ok);
      tc::fence_after_sync();
      ok &= !stop;
      return stop;
    };
    const float ascale = fabsf(a.scale);
    for (int it = 0; it < NC; it++) {
      const uint32_t ph = it & 1, tile = tc::smem_u32(sm + AD_TILE + ph * TILE), rec = tc::smem_u32(sm + AD_REC + (it % 3) * REC_PAD);
      const float *nf = reinterpret_cast<const float *>(sm + AD_REC + (it % 3) * REC_PAD + REC_F), *cc = nf + C, *be = cc + C;
      ok &= wait(bar(m->tile_full[ph]), (it >> 1) & 1, limit, gave_up);
      tc::fence_smem_to_async();
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t kd = tc::kmajor_desc(tile, 128, 0);
#pragma unroll
        for (int s = 0; s < 8; s++)  // A K^T
          tc::mma_f16_ts(tbase + T_D1, tbase + T_S + 8 * s, kd + step128(s), id64, s > 0);
        tc::mma_commit(bar(m->mma1));
      }
      if (!SEG && r == 32) {  // the adjoint after the chunk
        const size_t at = (size_t)u * NCT + last - it;
        bulk_s2g(ao.S + at * TILE, tc::smem_u32(sm + AD_STAGE), TILE);
        tc::bulk_commit();
        ao.iS[at] = iS;
      }
      ok &= wait(bar(m->rec_full[it % 3]), (it / 3) & 1, limit, gave_up);
      const float4 inv = *reinterpret_cast<const float4 *>(sm + AD_REC + (it % 3) * REC_PAD + REC_S);
      const float iK = inv.x, iQ = inv.y, ig = m->ig[ph], top = (float)(1 << kTopTile);
      const float kmax = top * iK, qmax = top * iQ, gmax = top * ig, all = -nf[C - 1];  // all: the chunk's decay
      const float gm = reinterpret_cast<const float *>(sm + AD_REC + (it % 3) * REC_PAD + REC_S)[4];  // no decay in it is greater
      const float w1 = iS * iK, w2 = a.scale * ig * iK * iQ * gm;  // units of D1 and of g^T P
      float iR;
      const float sR = bound_scale((float)D * gm * kmax * fmaf((float)C * gmax * ascale, qmax, bS), kTopRow, iR);
      m->iR[ph][r] = iR;
      const u64 w1_2 = pack2(w1 * sR, w1 * sR), w2_2 = pack2(w2 * sR, w2 * sR);
      ok &= wait(bar(m->dp_full), ph, limit, gave_up);
      ok &= wait(bar(m->mma1), ph, limit, gave_up);
      tc::fence_after_sync();
      // R' = c D1 + g^T P
#pragma unroll
      for (int h = 0; h < 4; h++) {
        float z[16], y[16], v[8];
        tc::tmem_ld16(tl + T_D1 + 16 * h, z);
        tc::tmem_ld16(tl + T_DP + 16 * h, y);
        ulonglong2 ff[4];
#pragma unroll
        for (int k = 0; k < 4; k++) ff[k] = *reinterpret_cast<const ulonglong2 *>(cc + 16 * h + 4 * k);
        tc::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; k++) {
          v[2 * k] = half2_bits(fma2(pack2(z[4 * k], z[4 * k + 1]), mul2(ff[k].x, w1_2),
                                     mul2(pack2(y[4 * k], y[4 * k + 1]), w2_2)));
          v[2 * k + 1] = half2_bits(fma2(pack2(z[4 * k + 2], z[4 * k + 3]), mul2(ff[k].y, w1_2),
                                         mul2(pack2(y[4 * k + 2], y[4 * k + 3]), w2_2)));
        }
        tc::tmem_st8(tl + T_R + 8 * h, v);  // (columns 8 h ..: read by now)
      }
      tc::tmem_st_wait();
      if (it > 0) ok &= wait(bar(m->o_free), (it - 1) & 1, limit, gave_up);  // (the last du is read)
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t td = tc::mnmajor_desc(rec, C, 0);
#pragma unroll
        for (int s = 0; s < 4; s++) tc::mma_f16_ts(tbase + T_D2, tbase + T_R + 8 * s, td + step_mn(s), id64n, s > 0);
        tc::mma_commit(bar(m->mma2));
      }
      warp_arrive(m->r_ready);  // (g^T P has been read)
      ok &= wait(bar(m->mma2), ph, limit, gave_up);
      tc::fence_after_sync();
      // -beta f du as the next operand (headroom for beta < 4)
      float uU = 0.0f, iU;
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
        const float sU = bound_scale(uU * gm, kTopRow - 2, iU);
        const u64 sU2 = pack2(sU, sU);
#pragma unroll
        for (int h = 0; h < 4; h++) {
          float x[16], w[8];
          tc::tmem_ld16(tl + T_D2 + 16 * h, x);
          tc::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; k++) {
            const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(nf + 16 * h + 4 * k);
            const ulonglong2 bb = *reinterpret_cast<const ulonglong2 *>(be + 16 * h + 4 * k);
            w[2 * k] = half2_bits(mul2(mul2(pack2(x[4 * k], x[4 * k + 1]), sU2), mul2(ff.x, bb.x)));
            w[2 * k + 1] = half2_bits(mul2(mul2(pack2(x[4 * k + 2], x[4 * k + 3]), sU2), mul2(ff.y, bb.y)));
          }
          tc::tmem_st8(tl + T_CU + 8 * h, w);
        }
        tc::tmem_st_wait();
      }
      const float w3 = iU * iR * iK, w4 = a.scale * ig * iQ * gm;  // units of the two sums into A
      bS = fmaf(all, bS, (float)C * gm * fmaf(4.0f * uU * iR, kmax, gmax * qmax * ascale));
      put_rows(bS);
      {
        const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(uU * iR));
        if (lane == 0) m->umax[ph][warp] = __uint_as_float(w);
      }
      if (r == 32) tc::bulk_wait_read();  // the kept adjoint has left its tile
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t kt = tc::mnmajor_desc(tile, 128, 0);
#pragma unroll
        for (int s = 0; s < 4; s++) tc::mma_f16_ts(tbase + T_DS, tbase + T_CU + 8 * s, kt + step_mn(s), idKN, s > 0);
        tc::mma_commit(bar(m->mma3));
      }
      warp_arrive(m->u_ready);  // (and the record has been read)
      const float sS = bound_scale(all_rows(), kTopRow, iS);
      const u64 w3_2 = pack2(w3, w3), w4_2 = pack2(w4, w4), sS2 = pack2(sS, sS), dec = pack2(all, all);
      ok &= wait(bar(m->dq_full), ph, limit, gave_up);
      ok &= wait(bar(m->mma3), ph, limit, gave_up);
      tc::fence_after_sync();
      if (r == 0) mbar_arrive(bar(m->tile_free[ph]));
#pragma unroll
      for (int k = 0; k < 8; k++) {
        float z[16], y[16], v[8];
        tc::tmem_ld16(tl + T_DS + 16 * k, z);
        tc::tmem_ld16(tl + T_DQ + 16 * k, y);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; i++) {
          S[8 * k + i] = fma2(pack2(z[2 * i], z[2 * i + 1]), w3_2,
                              fma2(pack2(y[2 * i], y[2 * i + 1]), w4_2, mul2(S[8 * k + i], dec)));
          v[i] = half2_bits(mul2(S[8 * k + i], sS2));
        }
        keep_words(k, v);  // the next chunk's operand
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(m->upd);
      if ((it & 7) == 7) row_max();  // (before the bound is loose)
    }
    if (r == 32) tc::bulk_wait_all();
    if (SEG && tail) {  // is that all?  (a NaN or an infinity anywhere: no)
      row_max();
      float after = m->rest;
      if (a.dS_final) {
        const float *src = a.dS_final + ((size_t)u * D + r) * D;
        float x = 0.0f;
        for (int j = 0; j < D; j++) x += fabsf(src[j]);
        after = fmaf(x, m->rest0, after);
      }
      const int more = group_or(1, 128, !(after <= 0x1p-26f * bS));
      if (r == 0) sg.whole_adj[(size_t)u * sg.n + seg] = more;
    }
    float *final = SEG              ? sg.adj + ((size_t)u * sg.n + seg) * D * D
                   : a.dS0 && seg == 0 ? a.dS0 + (size_t)u * D * D
                                       : nullptr;
    if (!group_or(1, 128, !ok) && final) {
      float4 *dst = reinterpret_cast<float4 *>(final + (size_t)r * D);
#pragma unroll
      for (int g = 0; g < D / 4; g++) {
        float4 x;
        unpack2(S[2 * g], x.x, x.y);
        unpack2(S[2 * g + 1], x.z, x.w);
        dst[g] = x;
      }
    }
  } else if (warp < 8) {
    // ---- du as an operand: fragments, transposed into a token-major tile ----
    regs_down<kRegHelper>();
    const int h = tid - 128, w = warp - 4;
    const uint32_t tl = tbase + ((uint32_t)(32 * w) << 16);
    for (int it = 0; it < NC; it++) {
      const bool got = wait(bar(m->u_ready), it & 1, limit, gave_up);
      if (h == 0) tc::bulk_wait_read();  // the last chunk's du has left its buffer
      if (group_or(2, 128, !got)) {
        ok = false;
        break;
      }
      if constexpr (SEG) {  // nothing to write
        warp_arrive(m->o_free);
        if (it + 3 < NC) {
          if (h == 0) fetch_rec(it + 3);
          rec_sent++;
        }
        continue;
      }
      tc::fence_after_sync();
      float x[2][32];
      tmem_ld_frag64(tl + T_D2, x[0]);
      tmem_ld_frag64(tl + (16u << 16) + T_D2, x[1]);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      warp_arrive(m->o_free);
      const float4 b = *reinterpret_cast<const float4 *>(m->umax[it & 1]);
      float iu;
      const float su = bound_scale(fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)), kTopRow, iu);
      const int tk = 8 * (lane >> 4) + (lane & 7);
#pragma unroll
      for (int hf = 0; hf < 2; hf++) {
        const int ch = 32 * w + 16 * hf + (lane >> 2), c8 = 4 * w + 2 * hf + ((lane >> 3) & 1);
        const float r1 = m->iR[it & 1][ch] * su, r2 = m->iR[it & 1][ch + 8] * su;
        const u64 a1 = pack2(r1, r1), b1 = pack2(r2, r2);
        const float *z = x[hf];
#pragma unroll
        for (int p = 0; p < 4; p++) {
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int j = 8 * p + 4 * e;
            o[2 * e] = __float_as_uint(half2_bits(mul2(pack2(z[j], z[j + 1]), a1)));
            o[2 * e + 1] = __float_as_uint(half2_bits(mul2(pack2(z[j + 2], z[j + 3]), b1)));
          }
          stmatrix_x4_trans(tc::smem_u32(sm + AD_OUT + tile_off(16 * p + tk, c8, C)), o[0], o[1], o[2], o[3]);
        }
      }
      tc::fence_smem_to_async();
      group_or(2, 128, false);
      if (h == 0) {
        const size_t at = (size_t)u * NCT + last - it;
        bulk_s2g(ao.U + at * ROWS64, tc::smem_u32(sm + AD_OUT), ROWS64);
        tc::bulk_commit();
        ao.iU[at] = iu;
        if (it + 3 < NC) fetch_rec(it + 3);  // (the other groups are past this record)
      }
      if (it + 3 < NC) rec_sent++;
    }
    if (h == 0) tc::bulk_wait_all();
  } else {
    // ---- K, f Q and g as operands; the products of g ----
    regs_down<kRegConvert>();
    const int h = tid - 256, r0 = h >> 4, c8 = h & 15, uk = a.qk_unit(u);  // rows r0, r0 + 8 ..; 8 channels
    const __nv_bfloat16 *kp = (const __nv_bfloat16 *)a.k + ((size_t)uk * T + r0) * D + 8 * c8;
    const __nv_bfloat16 *qp = (const __nv_bfloat16 *)a.q + ((size_t)uk * T + r0) * D + 8 * c8;
    const __nv_bfloat16 *gp = (const __nv_bfloat16 *)a.dout + ((size_t)u * T + r0) * D + 8 * c8;
    uint4 x[8], y[8], z[8];
    auto load = [&](int c) {
      const int n = T - c * C - r0;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        x[i] = y[i] = z[i] = make_uint4(0, 0, 0, 0);
        if (8 * i < n) {
          const size_t at = ((size_t)c * C + 8 * i) * D;
          x[i] = *reinterpret_cast<const uint4 *>(kp + at);
          y[i] = *reinterpret_cast<const uint4 *>(qp + at);
          z[i] = *reinterpret_cast<const uint4 *>(gp + at);
        }
      }
    };
    const uint32_t idP = tc::idesc_f16(128, C, true, true), idQ = tc::idesc_f16(128, D, true, true);
    load(last);
    for (int it = 0; it < NC; it++) {
      const int b = it & 1;
      uint32_t mg = 0;
#pragma unroll
      for (int k = 0; k < 8; k++) mg = absmax_words(mg, z[k]);
      mg = absmax_fold(mg);
      if (lane == 0) m->red[4 * b + warp - 8] = mg;
      bool got = wait(bar(m->rec_full[it % 3]), (it / 3) & 1, limit, gave_up);
      if (it >= 2) got &= wait(bar(m->tile_free[b]), ((it >> 1) - 1) & 1, limit, gave_up);
      if (group_or(4, 128, !got)) {
        ok = false;
        break;
      }
      const uint4 g4 = *reinterpret_cast<const uint4 *>(m->red + 4 * b);
      float ig;
      const float sg = bound_scale(__uint_as_float(max(max(g4.x, g4.y), max(g4.z, g4.w)) << 16), kTopTile, ig);
      if (h == 0) m->ig[b] = ig;
      const float *nf = reinterpret_cast<const float *>(sm + AD_REC + (it % 3) * REC_PAD + REC_F);
      const float4 inv = *reinterpret_cast<const float4 *>(sm + AD_REC + (it % 3) * REC_PAD + REC_S);
      const float f_unit = inv.w * reinterpret_cast<const float *>(sm + AD_REC + (it % 3) * REC_PAD + REC_S)[5];
      const u64 sk2 = pack2(inv.z, inv.z), sg2 = pack2(sg, sg);
      uint8_t *dst = sm + AD_TILE + b * TILE + tile_off(r0, c8, 128), *dg = sm + AD_G + b * ROWS64 + tile_off(r0, c8, C);
#pragma unroll
      for (int k = 0; k < 8; k++) {
        const float fq = -nf[r0 + 8 * k] * f_unit;
        *reinterpret_cast<uint4 *>(dst + 1024 * k) = to_half8(x[k], sk2);
        *reinterpret_cast<uint4 *>(dst + C * 128 + 1024 * k) = to_half8(y[k], pack2(fq, fq));
        *reinterpret_cast<uint4 *>(dg + 1024 * k) = to_half8(z[k], sg2);
      }
      tc::fence_smem_to_async();
      warp_arrive(m->tile_full[b]);
      if (it + 1 < NC) load(last - 1 - it);
      if (warp == 8) {
        const uint64_t gd = tc::mnmajor_desc(tc::smem_u32(sm + AD_G + b * ROWS64), C, 0);
        const uint64_t pd = tc::mnmajor_desc(tc::smem_u32(sm + AD_REC + (it % 3) * REC_PAD + REC_P), C, 0);
        const uint64_t qd = tc::mnmajor_desc(tc::smem_u32(sm + AD_TILE + b * TILE + C * 128), 128, 0);
        got = wait(bar(m->tile_full[b]), (it >> 1) & 1, limit, gave_up);
        if (it > 0) got &= wait(bar(m->r_ready), (it - 1) & 1, limit, gave_up);
        tc::fence_after_sync();
        if (__all_sync(0xffffffffu, got) && elect_one()) {
#pragma unroll
          for (int s = 0; s < 4; s++) tc::mma_f16(tbase + T_DP, gd + step_mn(s), pd + step_mn(s), idP, s > 0);
          tc::mma_commit(bar(m->dp_full));
        }
        __syncwarp();
        if (it > 0) got &= wait(bar(m->upd), (it - 1) & 1, limit, gave_up);
        tc::fence_after_sync();
        if (__all_sync(0xffffffffu, got) && elect_one()) {
#pragma unroll
          for (int s = 0; s < 4; s++) tc::mma_f16(tbase + T_DQ, gd + step_mn(s), qd + step_mn(s), idQ, s > 0);
          tc::mma_commit(bar(m->dq_full));
        }
        __syncwarp();
      }
    }
  }
  if (!ok) *gave_up = 1;
  __syncthreads();
  // a wait gave up: products and copies still in flight finish before the memory is released
  if (*gave_up) {
    if ((warp == 0 || warp == 8) && elect_one()) tc::mma_commit(bar(m->drain));
    if (tid == 0) {
      unsigned bits = tc::kErrMmaTimeout;
      if (!tc::mbar_wait(bar(m->drain), 0, tc::kWaitLimit)) bits |= tc::kErrDrainTimeout;
      atomicOr(a.status, bits);
    }
    if (tid == 128) {
      bool in = true;
      for (int c = max(0, rec_sent - 3); c < rec_sent; c++)
        in &= tc::mbar_wait(bar(m->rec_full[c % 3]), (c / 3) & 1, tc::kWaitLimit);
      if (!in) atomicOr(a.status, tc::kErrDrainTimeout);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 512);
}

// ---- the gradients of a chunk ---------------------------------------------------------------------
// shared memory: [g; du] | u | [Q; K] | S0 | A | products' operand | X | misc.  (u as rows 64 .. 127 of a
// 128-row operand: its descriptor starts 8 KB before it.)  dq and dk leave through the products' operand.
constexpr uint32_t GR_A1 = 0, GR_U = TILE, GR_QK = GR_U + ROWS64, GR_S = GR_QK + TILE, GR_DS = GR_S + TILE, GR_A5 = GR_DS + TILE;
constexpr int X_LD = 72;  // (rows of a fragment in different banks)
constexpr uint32_t GR_X = GR_A5 + TILE, GR_MISC = GR_X + ((C * X_LD * 4 + 127) & ~127);
constexpr int GR_WARPS = 16, GR_SEGS = 8;
struct GradsMisc {
  float l[C], nf[C], c[C], beta[C], gam[C], num[12];  // num: 1 / scale of K, Q, S0, u, A, du; scale of K, Q; gm
  alignas(16) int z[C];
  float duv[C], dbeta[4][C], xin[4][2][C], xout[4][C];
  float head[GR_SEGS][C], pass[GR_SEGS], dgam[2][C];
  alignas(16) uint32_t red[GR_WARPS];
  float cross[GR_WARPS];
  uint64_t load, mma_a, mma_b, mma_c, drain;
  uint32_t tmem;
};
constexpr uint32_t GR_SMEM = GR_MISC + sizeof(GradsMisc) + 1024;
static_assert(GR_SMEM <= 232448, "shared memory per block");
// tensor memory columns: [g; du] S0 | [.; u] A | [g; du] u^T | [Q; K] K^T | [0 W; W^T -(V + V^T)] [Q; K]
constexpr uint32_t T_G1 = 0, T_G2 = 128, T_G3 = 256, T_G4 = 320, T_G5 = 384;

__device__ __forceinline__ float2 half2_at(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

__device__ __forceinline__ void l2_prefetch(const void *p, uint32_t bytes) {  // (16-byte aligned, multiples of 16)
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;\n" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void l2_prefetch(const void *p) { asm volatile("prefetch.global.L2 [%0];\n" ::"l"(p)); }

// 512 threads, one CTA per SM over `chunks` chunks of all units: the warps that share a quarter of the
// tensor memory's lanes take a quarter of the columns each.  A chunk is a row of short steps that wait
// for one another, so the next chunk's rows are on their way (in registers) from the middle of this one's, its states
// and u from where this one's have been read.  (One CTA per chunk, 256 threads, nothing on its way: 875 us
// at 8 x 16 x 4096; so, 461.)
__global__ void __launch_bounds__(32 * GR_WARPS, 1)
    mesa_rule_grads_tc_kernel(RuleArgs a, int NC, int chunks, const uint8_t *records, RuleOperands so, RuleOperands ao,
                              float *dqp, float *dkp, const __grid_constant__ CUtensorMap mapDq,
                              const __grid_constant__ CUtensorMap mapDk) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  GradsMisc *m = reinterpret_cast<GradsMisc *>(sm + GR_MISC);
  float *X = reinterpret_cast<float *>(sm + GR_X);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t bl = tc::smem_u32(&m->load), ba = tc::smem_u32(&m->mma_a), bb = tc::smem_u32(&m->mma_b),
                 bc = tc::smem_u32(&m->mma_c);
  const int r0 = tid >> 4, c8 = tid & 15;  // rows of Q, K, g and v: 16 threads a row, rows r0 and r0 + 32

  // what is read ahead
  uint4 q4[2], k4[2], g4[2], v4[2];
  float tok;
  auto fetch_qk = [&](int at) {
    const int u = at / NC, t0 = (at - u * NC) * C, n = min(C, a.T - t0);
    const size_t first = ((size_t)a.qk_unit(u) * a.T + t0 + r0) * D + 8 * c8;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      q4[i] = k4[i] = make_uint4(0, 0, 0, 0);
      if (r0 + 32 * i < n) {
        q4[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.q + first + 32 * i * D);
        k4[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.k + first + 32 * i * D);
      }
    }
  };
  auto fetch_gv = [&](int at) {
    const int u = at / NC, t0 = (at - u * NC) * C, n = min(C, a.T - t0);
    const size_t tok0 = (size_t)u * a.T + t0, first = (tok0 + r0) * D + 8 * c8;
    const uint8_t *rec = records + (size_t)at * REC;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      g4[i] = v4[i] = make_uint4(0, 0, 0, 0);
      if (r0 + 32 * i < n) {
        g4[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.dout + first + 32 * i * D);
        v4[i] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.v + first + 32 * i * D);
      }
    }
    const int t = tid & (C - 1), which = tid >> 6;  // a token's numbers, one kind to two warps; the chunk's
    const float *src = which < 3 ? reinterpret_cast<const float *>(rec + REC_F) + tid
                       : which == 3 ? a.gamma + tok0 + t
                       : t < 2      ? reinterpret_cast<const float *>(rec + REC_S) + t
                       : t < 6      ? (t == 2 ? so.iS : t == 3 ? so.iU : t == 4 ? ao.iS : ao.iU) + at
                                    : reinterpret_cast<const float *>(rec + REC_S) + t - 4;
    tok = 1.0f;
    if (which < 3 || (which == 3 && t < n) || (which == 4 && t < 9)) tok = *src;
  };
  auto fetch_operands = [&](int at) {  // one thread
    tc::mbar_arrive_expect_tx(bl, 2 * TILE + 2 * ROWS64);
    tc::bulk_g2s(tc::smem_u32(sm + GR_U), so.U + (size_t)at * ROWS64, ROWS64, bl);
#pragma unroll
    for (int h = 0; h < 2; h++)  // du: rows 64 .. of both column halves
      tc::bulk_g2s(tc::smem_u32(sm + GR_A1 + h * ROWS64 + C * 128), ao.U + (size_t)at * ROWS64 + h * C * 128, C * 128, bl);
    tc::bulk_g2s(tc::smem_u32(sm + GR_S), so.S + (size_t)at * TILE, TILE, bl);
    tc::bulk_g2s(tc::smem_u32(sm + GR_DS), ao.S + (size_t)at * TILE, TILE, bl);
  };

  int at = blockIdx.x;
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 32) {
    for (uint32_t b : {bl, ba, bb, bc, tc::smem_u32(&m->drain)}) tc::mbar_init(b, 1);
    fetch_operands(at);
  }
  fetch_qk(at);
  fetch_gv(at);
  int fetched = 1;  // chunks' operands asked for
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = __shfl_sync(0xffffffffu, m->tmem, 0);
  // rows of the token x token products: row < 64: g_i and q_i, else du_i and k_i; a quarter of the columns
  const int quad = warp & 3, part = warp >> 2, row = 32 * quad + lane, i = row & 63;
  const bool upper = row < C;
  const uint32_t tl = tbase + ((uint32_t)(32 * quad) << 16);
  bool stop = false;
  float bad = 0.0f;  // NaN once a gradient was not finite

  for (int it = 0; at < chunks; it++, at += gridDim.x) {
    const uint32_t ph = it & 1;
    const int u = at / NC, t0 = (at - u * NC) * C, n = min(C, a.T - t0);
    const size_t tok0 = (size_t)u * a.T + t0;
    const int next = at + (int)gridDim.x;
    {
      const int t = tid & (C - 1), which = tid >> 6;
      if (which < 4) {
        (which == 0 ? m->nf : which == 1 ? m->c : which == 2 ? m->beta : m->gam)[t] = tok;
      } else if (which == 4 && t < 9) {
        m->num[t] = tok;
      }
    }
    uint32_t mg = 0;
#pragma unroll
    for (int k = 0; k < 2; k++) mg = absmax_words(mg, g4[k]);
    mg = absmax_fold(mg);
    if (lane == 0) m->red[warp] = mg;
    if (tid == 0) tc::bulk_wait_read();  // the last chunk's dq and dk have left their place
    __syncthreads();
    const float ik = m->num[0], iq = m->num[1], iS = m->num[2], iu = m->num[3], iA = m->num[4], idu = m->num[5], gm = m->num[8];
    const float2 sk_sq = *reinterpret_cast<const float2 *>(m->num + 6);
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const int r = r0 + 32 * k;
      *reinterpret_cast<uint4 *>(sm + GR_QK + tile_off(r, c8, 128)) = to_half8(q4[k], pack2(sk_sq.y, sk_sq.y));
      *reinterpret_cast<uint4 *>(sm + GR_QK + tile_off(C + r, c8, 128)) = to_half8(k4[k], pack2(sk_sq.x, sk_sq.x));
    }
    // the products' operand: its block of Q columns for dq is zero
    *reinterpret_cast<uint4 *>(sm + GR_A5 + tile_off(tid >> 3, tid & 7, 128)) = make_uint4(0, 0, 0, 0);
    mg = 0;
#pragma unroll
    for (int w = 0; w < GR_WARPS / 4; w++) {
      const uint4 x = *reinterpret_cast<const uint4 *>(m->red + 4 * w);
      mg = max(mg, max(max(x.x, x.y), max(x.z, x.w)));
    }
    float ig;
    const float sg = bound_scale(__uint_as_float(mg << 16), kTopTile, ig);
#pragma unroll
    for (int k = 0; k < 2; k++)
      *reinterpret_cast<uint4 *>(sm + GR_A1 + tile_off(r0 + 32 * k, c8, 128)) = to_half8(g4[k], pack2(sg, sg));
    if (warp == GR_WARPS - 1) {
      const GatePair g = gate_scan(make_float2(m->gam[2 * lane], m->gam[2 * lane + 1]), lane);
      *reinterpret_cast<float2 *>(&m->l[2 * lane]) = make_float2(g.l0, g.l1);
      *reinterpret_cast<int2 *>(&m->z[2 * lane]) = make_int2(g.z0, g.z1);
      if (lane < GR_SEGS) {
        float x = lane == GR_SEGS - 1 ? 1.0f : m->gam[8 * lane + 8];
#pragma unroll
        for (int k = 1; k < 8; k++) x *= m->gam[8 * lane + k];
        m->pass[lane] = x;
      }
    }
    tc::fence_smem_to_async();
    tc::fence_before_sync();
    const bool loaded = tc::mbar_wait(bl, ph, a.wait_limit);
    stop = __syncthreads_or(!loaded);
    tc::fence_after_sync();
    if (stop) break;
    const uint64_t dA1 = tc::kmajor_desc(tc::smem_u32(sm + GR_A1), 128, 0), dQK = tc::kmajor_desc(tc::smem_u32(sm + GR_QK), 128, 0);
    if (warp == 0 && elect_one()) {
      const uint32_t id64 = tc::idesc_f16(128, C, false, false), idN = tc::idesc_f16(128, D, false, true);
      const uint64_t dU = tc::kmajor_desc(tc::smem_u32(sm + GR_U), C, 0), dUhi = tc::kmajor_desc(tc::smem_u32(sm + GR_U) - C * 128, C, 0);
      const uint64_t dK = tc::kmajor_desc(tc::smem_u32(sm + GR_QK) + C * 128, 128, 0);
      const uint64_t nS = tc::mnmajor_desc(tc::smem_u32(sm + GR_S), 128, 0), nA = tc::mnmajor_desc(tc::smem_u32(sm + GR_DS), 128, 0);
      // (a 64-row tile's second column half is 8 KB on)
      auto step64x128 = [](int s) { return (uint64_t)((s >> 2) * 512 + (s & 3) * 2); };
#pragma unroll
      for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_G3, dA1 + step128(s), dU + step64x128(s), id64, s > 0);
#pragma unroll
      for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_G4, dQK + step128(s), dK + step128(s), id64, s > 0);
      tc::mma_commit(ba);
#pragma unroll
      for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_G1, dA1 + step128(s), nS + step_mn(s), idN, s > 0);
#pragma unroll
      for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_G2, dUhi + step64x128(s), nA + step_mn(s), idN, s > 0);
      tc::mma_commit(bb);
    }
    __syncwarp();
    if (warp == GR_WARPS - 1 && next < chunks) {  // the next chunk comes to the L2 cache
      const int nu = next / NC, nt0 = (next - nu * NC) * C, nn = min(C, a.T - nt0);
      const size_t ntok = (size_t)nu * a.T + nt0, nrow = (size_t)a.qk_unit(nu) * a.T + nt0;
      if (lane < 4) {
        const void *base = lane == 0 ? a.q : lane == 1 ? a.k : lane == 2 ? a.dout : a.v;
        l2_prefetch((const __nv_bfloat16 *)base + (lane < 2 ? nrow : ntok) * D, nn * D * 2);
      } else if (lane < 8) {
        l2_prefetch((lane & 1 ? ao.S : so.S) + (size_t)next * TILE + (lane < 6 ? 0 : TILE / 2), TILE / 2);
      } else if (lane < 10) {
        l2_prefetch((lane & 1 ? ao.U : so.U) + (size_t)next * ROWS64, ROWS64);
      } else if (lane == 10) {
        l2_prefetch(records + (size_t)next * REC + REC_F, REC - REC_F);
      } else if (lane < 15) {
        l2_prefetch((lane == 11 ? so.iS : lane == 12 ? so.iU : lane == 13 ? ao.iS : ao.iU) + next);
      } else if (lane >= 16 && 4 * (lane - 16) < nn) {
        l2_prefetch(a.gamma + ntok + 4 * (lane - 16));
      }
    }
    // dv = beta du, du . v, and <A, S0>, while the products run
#pragma unroll
    for (int p = 0; p < 2; p++) {
      const int r = r0 + 32 * p;
      const uint4 d4 = *reinterpret_cast<const uint4 *>(sm + GR_A1 + tile_off(C + r, c8, 128));
      const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w}, vw[4] = {v4[p].x, v4[p].y, v4[p].z, v4[p].w};
      const float b = m->beta[r] * idu;
      float s = 0.0f;
      __align__(16) __nv_bfloat162 o[4];
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const float2 d = half2_at(dw[k]);
        s = fmaf(d.x, __uint_as_float(vw[k] << 16), fmaf(d.y, __uint_as_float(vw[k] & 0xffff0000u), s));
        o[k] = __floats2bfloat162_rn(b * d.x, b * d.y);
      }
      if (r < n) *reinterpret_cast<uint4 *>((__nv_bfloat16 *)a.dv_out + (tok0 + r) * D + 8 * c8) = *reinterpret_cast<uint4 *>(o);
      s = group_sum<16>(s);
      bad = fmaf(s, 0.0f, bad);
      if (c8 == 0) m->duv[r] = s * idu;
    }
    {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < (int)(TILE / 16 / (32 * GR_WARPS)); k++) {
        const uint4 x = *reinterpret_cast<const uint4 *>(sm + GR_S + 16 * (tid + 32 * GR_WARPS * k));
        const uint4 y = *reinterpret_cast<const uint4 *>(sm + GR_DS + 16 * (tid + 32 * GR_WARPS * k));
        const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float2 p = half2_at(xw[e]), q = half2_at(yw[e]);
          s = fmaf(p.x, q.x, fmaf(p.y, q.y, s));
        }
      }
      s = warp_sum(s);
      if (lane == 0) m->cross[warp] = s * iS * iA;
    }
    const float mul = upper ? a.scale * ig * iu : idu * iu;
    // the operand's units: W alpha, V alpha sq / sk (= op_v), both below 2^15 (|g16| <= 2^3, |u16|, |du16| <= 2^15,
    // 128 products, decays up to gm, beta < 4, V + V^T); in dq's rows, where W stands alone, its own (V can be far
    // larger).  sq / sk has no bound (2^61 for unit keys without queries), so V's units come from V alone: where they are the
    // smaller ones alpha = op_v sk / sq, which may be 0 (W^T Q is then nothing beside (V + V^T) K), and dk's unit
    // is 1 / (op_v sk), not 1 / (alpha sq).
    float ialpha_v, ialpha_q;
    const float vq = sk_sq.y * ik;  // sq / sk
    const float alpha_v = bound_scale(8.0f * gm * idu * iu * 137438953472.0f, kTopRow, ialpha_v);
    const float alpha_q = bound_scale(fabsf(a.scale) * gm * ig * iu * 33554432.0f, kTopRow, ialpha_q);
    const bool of_v = alpha_q * vq > alpha_v;  // (2^77 2^126 at most: infinity is greater, too)
    const float alpha = of_v ? alpha_v * (iq * sk_sq.x) : alpha_q, op_v = of_v ? alpha_v : alpha_q * vq;
    if (next < chunks) fetch_qk(next);
    const bool got_a = tc::mbar_wait(ba, ph, a.wait_limit);
    tc::fence_after_sync();
    stop = __syncthreads_or(!got_a);
    if (stop) break;
    {
      // in fragments of 8 x 8: of the rows 16 h + 8 e + lane / 4 of the warp's 32 (mod 64: i0 ..), columns 16 part +
      // 8 b + 2 (lane % 4) and the next
      const int i0 = 32 * (quad & 1), g = lane >> 2, q = 2 * (lane & 3), col = 16 * part + q;
      u64 x[2][4], y[2][4];  // [h][2 b + e]
#pragma unroll
      for (int h = 0; h < 2; h++) {
        tmem_ld_frag16(tl + ((uint32_t)(16 * h) << 16) + T_G3 + 16 * part, x[h]);
        tmem_ld_frag16(tl + ((uint32_t)(16 * h) << 16) + T_G4 + 16 * part, y[h]);
      }
      const u64 lj[2] = {*reinterpret_cast<const u64 *>(&m->l[col]), *reinterpret_cast<const u64 *>(&m->l[col + 8])};
      const float qk = (upper ? iq : ik) * ik, op0 = upper ? alpha_q : -op_v;  // real q . k, k . k
      const u64 mul2x = pack2(mul, mul), qk2 = pack2(qk, qk);
      const bool closed = m->z[C - 1] != 0;  // a gate in the chunk
      uint32_t p[2][4], pt[2][4];  // the operand's fragments (W: as it stands, and for its transpose)
      const float down = alpha * ialpha_q;
      float db[2][2];
      tc::tmem_ld_wait();
#pragma unroll
      for (int h = 0; h < 2; h++) {
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const int i = i0 + 16 * h + 8 * e + g, keep = upper ? i : i - 1;  // the last column of the operand
          const float li = m->l[i], op = upper ? op0 : op0 * m->beta[i];
          const u64 li2 = pack2(li, li), op2 = pack2(op, op);
          float sum = 0.0f;
#pragma unroll
          for (int b = 0; b < 2; b++) {
            const int j = col + 8 * b;
            float d0, d1, y0, y1, x0, x1;
            unpack2(sub2(li2, lj[b]), d0, d1);
            d0 = j <= keep ? ex2(d0) : 0.0f;
            d1 = j + 1 <= keep ? ex2(d1) : 0.0f;
            if (closed) {
              if (m->z[j] != m->z[i]) d0 = 0.0f;
              if (m->z[j + 1] != m->z[i]) d1 = 0.0f;
            }
            const u64 w = mul2(x[h][2 * b + e], mul2x);
            y[h][2 * b + e] = mul2(w, mul2(y[h][2 * b + e], qk2));  // X's part, without the decay
            unpack2(y[h][2 * b + e], y0, y1);
            unpack2(mul2(mul2(w, op2), pack2(d0, d1)), x0, x1);
            // (columns without a decay are none of the operand's, whatever their products are)
            x0 = j <= keep ? x0 : 0.0f;
            x1 = j + 1 <= keep ? x1 : 0.0f;
            p[h][2 * b + e] = __float_as_uint(half2_bits(x0, x1));
            pt[h][2 * b + e] = __float_as_uint(half2_bits(x0 * down, x1 * down));
            if (j <= keep) sum = fmaf(d0, y0, sum);
            if (j + 1 <= keep) sum = fmaf(d1, y1, sum);
          }
          db[h][e] = sum;
        }
      }
      const int l8 = lane & 7, lb = lane >> 3;  // this lane's row and block of a matrix store
      if (upper) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          // W: row i of dq's, K columns; W^T: row j of dk's, Q columns
          stmatrix_x4(tc::smem_u32(sm + GR_A5 + tile_off(i0 + 16 * h + 8 * (lb & 1) + l8, 8 + 2 * part + (lb >> 1), 128)),
                      p[h][0], p[h][1], p[h][2], p[h][3]);
          stmatrix_x4_trans(tc::smem_u32(sm + GR_A5 + tile_off(C + 16 * part + 8 * (lb >> 1) + l8, (i0 >> 3) + 2 * h + (lb & 1), 128)),
                            pt[h][0], pt[h][1], pt[h][2], pt[h][3]);
#pragma unroll
          for (int e = 0; e < 2; e++)
#pragma unroll
            for (int b = 0; b < 2; b++)
              *reinterpret_cast<u64 *>(&X[(i0 + 16 * h + 8 * e + g) * X_LD + col + 8 * b]) = y[h][2 * b + e];
        }
      } else {
        // -(V + V^T), block by block: a diagonal one is the sum of its two triangles (disjoint), one below is
        // written twice, one above by its mirror image
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int t = 0; t < 4; t++) {
            const int bi = (i0 >> 3) + 2 * h + (t & 1), bj = 2 * part + (t >> 1);
            if (bj > bi) continue;
            const uint32_t f = bj == bi ? p[h][t] | transposed(p[h][t]) : p[h][t];
            stmatrix_x1(tc::smem_u32(sm + GR_A5 + tile_off(C + 8 * bi + l8, 8 + bj, 128)), f);
            if (bj < bi) stmatrix_x1_trans(tc::smem_u32(sm + GR_A5 + tile_off(C + 8 * bj + l8, 8 + bi, 128)), f);
          }
      }
      tc::fence_smem_to_async();
      tc::fence_before_sync();
      __syncthreads();
      tc::fence_after_sync();
      if (warp == 0 && elect_one()) {
        const uint32_t idN = tc::idesc_f16(128, D, false, true);
        const uint64_t dA5 = tc::kmajor_desc(tc::smem_u32(sm + GR_A5), 128, 0), nQK = tc::mnmajor_desc(tc::smem_u32(sm + GR_QK), 128, 0);
#pragma unroll
        for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_G5, dA5 + step128(s), nQK + step_mn(s), idN, s > 0);
        tc::mma_commit(bc);
      }
      __syncwarp();
      if (!upper) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
          for (int e = 0; e < 2; e++) {
            const int i = i0 + 16 * h + 8 * e + g;
            const u64 nb = pack2(-m->beta[i], -m->beta[i]);
#pragma unroll
            for (int b = 0; b < 2; b++) {
              u64 *x1 = reinterpret_cast<u64 *>(&X[i * X_LD + col + 8 * b]);
              *x1 = fma2(nb, y[h][2 * b + e], *x1);
            }
            // du_i against sum_j D_ij (k_i . k_j) u_j
            float sum = db[h][e];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (q == 0) m->dbeta[part][i] = sum;
          }
      }
    }
    if (next < chunks) fetch_gv(next);
    const bool got_b = tc::mbar_wait(bb, ph, a.wait_limit);
    tc::fence_after_sync();
    stop = __syncthreads_or(!got_b);
    if (stop) break;
    if (next < chunks) {  // the states, u and du have been read
      if (tid == 32) fetch_operands(next);
      fetched++;
    }
    {  // rows against q_i or k_i: what the gates and betas need of the state products; columns 32 part ..
      float d1 = 0.0f, d2 = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float x[16], y[16];
        tc::tmem_ld16(tl + T_G1 + 32 * part + 16 * h, x);
        if (!upper) tc::tmem_ld16(tl + T_G2 + 32 * part + 16 * h, y);
        const uint4 p = *reinterpret_cast<const uint4 *>(sm + GR_QK + tile_off(row, 4 * part + 2 * h, 128));
        const uint4 q = *reinterpret_cast<const uint4 *>(sm + GR_QK + tile_off(row, 4 * part + 2 * h + 1, 128));
        const uint32_t w[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
        tc::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const float2 f = half2_at(w[k]);
          d1 = fmaf(x[2 * k], f.x, fmaf(x[2 * k + 1], f.y, d1));
          if (!upper) d2 = fmaf(y[2 * k], f.x, fmaf(y[2 * k + 1], f.y, d2));
        }
      }
      if (upper) {
        m->xin[part][0][i] = d1 * (a.scale * ig * iS * iq);
      } else {
        m->xin[part][1][i] = d1 * (idu * iS * ik);  // (times beta below)
        m->xout[part][i] = d2 * (iu * iA * ik);
      }
    }
    __syncthreads();
    if (tid < C) {
      const float kS = (m->xin[0][1][tid] + m->xin[1][1][tid]) + (m->xin[2][1][tid] + m->xin[3][1][tid]);
      X[tid * X_LD + C - 1] = (m->xin[0][0][tid] + m->xin[1][0][tid]) + (m->xin[2][0][tid] + m->xin[3][0][tid]) - m->beta[tid] * kS;
      m->duv[tid] += m->nf[tid] * kS;
    }
    __syncthreads();
    // columns of X (column j: token j as the writer; the last: the state before the chunk), upwards from the
    // last token: Z_t = X_t + gamma_{t+1} Z_{t+1}, times the decay from the writer to t - 1, summed over the
    // writers before t.  Eight tokens a thread, joined over the segments above.
    {
      const int seg = warp >> 1, col = 32 * (warp & 1) + lane, t8 = 8 * seg, j = col == C - 1 ? -1 : col;
      float Z[8];
#pragma unroll
      for (int k = 0; k < 8; k++) Z[k] = X[(t8 + k) * X_LD + col];
#pragma unroll
      for (int k = 6; k >= 0; k--) Z[k] = fmaf(m->gam[t8 + k + 1], Z[k + 1], Z[k]);
      m->head[seg][col] = Z[0];
      __syncthreads();
      float in;  // Z of the token above the segment
      if (j < 0) {
        in = 0.0f;
#pragma unroll
        for (int w = 0; w < GR_WARPS; w++) in += m->cross[w];
      } else {
        in = (m->xout[0][j] + m->xout[1][j]) + (m->xout[2][j] + m->xout[3][j]);
      }
#pragma unroll
      for (int s = GR_SEGS - 1; s > 0; s--)
        if (s > seg) in = fmaf(m->pass[s], in, m->head[s][col]);
      const float lj = j < 0 ? 0.0f : m->l[j];
      const int zj = j < 0 ? 0 : m->z[j];
      float carry = seg < GR_SEGS - 1 ? m->gam[t8 + 8] * in : in;  // (the last token's gate to the state after: in c)
#pragma unroll
      for (int k = 7; k >= 0; k--) {
        const int t = t8 + k;
        const float lp = t > 0 ? m->l[t - 1] : 0.0f;
        const int zp = t > 0 ? m->z[t - 1] : 0;
        const float z = Z[k] + carry;
        carry *= m->gam[t];
        Z[k] = t > j && zp == zj ? z * ex2(lp - lj) : 0.0f;
      }
      // over the warp's columns: lanes 4 m .. hold token m's
#pragma unroll
      for (int o = 16, w = 4; o >= 4; o >>= 1, w >>= 1) {
        const bool hi = lane & o;
#pragma unroll
        for (int k = 0; k < 4; k++) {
          if (k >= w) continue;
          const float give = hi ? Z[k] : Z[k + w];
          Z[k] = (hi ? Z[k + w] : Z[k]) + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
      float s = Z[0] + __shfl_xor_sync(0xffffffffu, Z[0], 2);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      bad = fmaf(s, 0.0f, bad);
      if ((lane & 3) == 0) m->dgam[warp & 1][t8 + (lane >> 2)] = s;
    }
    const bool got_c = tc::mbar_wait(bc, ph, a.wait_limit);
    tc::fence_after_sync();
    stop = __syncthreads_or(!got_c);
    if (stop) break;
    if (tid < n) {
      st_gate<__nv_bfloat16>(a, a.dgamma, tok0 + tid, m->dgam[0][tid] + m->dgam[1][tid]);
      st_gate<__nv_bfloat16>(
          a, a.dbeta, tok0 + tid,
          m->duv[tid] - ((m->dbeta[0][tid] + m->dbeta[1][tid]) + (m->dbeta[2][tid] + m->dbeta[3][tid])));
    }
    // dq = f (g S0) + W K;  dk = W^T Q - (V + V^T) K + c (u A) - f beta (du S0); columns 32 part ..
    const float f1 = upper ? -m->nf[i] * a.scale * ig * iS : m->nf[i] * m->beta[i] * idu * iS;
    const float f2 = m->c[i] * iu * iA, f5 = upper ? ialpha_q * ik : of_v ? ialpha_v * ik : ialpha_q * iq;
    uint8_t *out = sm + GR_A5 + (upper ? 0 : ROWS64);
    float *sum = upper ? dqp : dkp;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      float x[16], y[16];
      tc::tmem_ld16(tl + T_G5 + 32 * part + 16 * h, x);
      tc::tmem_ld16(tl + T_G1 + 32 * part + 16 * h, y);
      tc::tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 16; k++) x[k] = fmaf(y[k], f1, x[k] * f5);
      if (!upper) {
        tc::tmem_ld16(tl + T_G2 + 32 * part + 16 * h, y);
        tc::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; k++) x[k] = fmaf(y[k], f2, x[k]);
      }
#pragma unroll
      for (int k = 0; k < 16; k++) bad = fmaf(x[k], 0.0f, bad);
      if (sum) {
        if (i < n) {
          float4 *dst = reinterpret_cast<float4 *>(sum + (tok0 + i) * D + 32 * part + 16 * h);
#pragma unroll
          for (int k = 0; k < 4; k++) dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        }
      } else {
        __align__(16) __nv_bfloat162 o[8];
#pragma unroll
        for (int k = 0; k < 8; k++) o[k] = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        *reinterpret_cast<uint4 *>(out + tile_off(i, 4 * part + 2 * h, C)) = *reinterpret_cast<const uint4 *>(o);
        *reinterpret_cast<uint4 *>(out + tile_off(i, 4 * part + 2 * h + 1, C)) = *reinterpret_cast<const uint4 *>(o + 4);
      }
    }
    tc::fence_smem_to_async();
    tc::fence_before_sync();  // (the next chunk's products write what was read)
    __syncthreads();
    if (!dqp && tid == 0) {
#pragma unroll
      for (int h = 0; h < 2; h++) {
        tensor_s2g_3d(&mapDq, tc::smem_u32(sm + GR_A5 + h * C * 128), 64 * h, t0, u);
        tensor_s2g_3d(&mapDk, tc::smem_u32(sm + GR_A5 + ROWS64 + h * C * 128), 64 * h, t0, u);
      }
      tc::bulk_commit();
    }
  }
  if (tid == 0) tc::bulk_wait_all();
  if (!(bad == 0.0f)) atomicOr(a.status, tc::kErrNonFinite);
  if (stop) {  // a wait gave up: what is in flight finishes before the memory is released
    if (tid == 0) atomicOr(a.status, tc::kErrMmaTimeout);
    const bool issuer = warp == 0 && elect_one();
    tc::drain_mmas(tc::smem_u32(&m->drain), issuer, a.status);
    if (tid == 0 && !tc::mbar_wait(bl, (fetched - 1) & 1, tc::kWaitLimit)) atomicOr(a.status, tc::kErrDrainTimeout);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 512);
}

}  // namespace

namespace {
// The adjoint after each segment: A_{y-1} = A_y Tr_y^T + adj_y (A_{n-2} = adj_{n-1}; A_{n-1} is a copy of dS_final: dS0
// may be its memory), sixteen rows by a CTA of 256 threads; grid (8, U).
__global__ void __launch_bounds__(256) mesa_rule_join_adjoint_kernel(RuleSegments sg, const float *dS_final) {
  __shared__ __align__(16) float rows[16][D + 4];
  const int u = blockIdx.y, row0 = 16 * blockIdx.x, tid = threadIdx.x;
  const int r = tid >> 4, c0 = (tid & 15) * 8;  // row r, columns c0 ..
  const size_t own = (size_t)(row0 + r) * D + c0;
  for (int i = 0; i < 8; i++)
    sg.A[((size_t)u * sg.n + sg.n - 1) * D * D + own + i] = dS_final ? dS_final[(size_t)u * D * D + own + i] : 0.0f;
  for (int y = sg.n - 1; y > 0; y--) {
    const size_t at = (size_t)u * sg.n + y;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = sg.adj[at * D * D + own + i];
    if (y < sg.n - 1 && sg.whole_adj[at]) {
      const float *Tr = sg.Tr + at * D * D + (size_t)c0 * D;
#pragma unroll 2
      for (int k = 0; k < D; k += 4) {
        const float4 s = *reinterpret_cast<const float4 *>(&rows[r][k]);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          const float4 p = *reinterpret_cast<const float4 *>(Tr + i * D + k);
          x[i] = fmaf(s.x, p.x, fmaf(s.y, p.y, fmaf(s.z, p.z, fmaf(s.w, p.w, x[i]))));
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; i++) {
      rows[r][c0 + i] = x[i];
      sg.A[(at - 1) * D * D + own + i] = x[i];
    }
    __syncthreads();
  }
}

template <bool SEG>
int launch_adjoint(const RuleArgs &a, const void *records, const RuleOperands &ao, const RuleSegments &sg, bool tail,
                   cudaStream_t st) {
  auto kfn = mesa_rule_adjoint_kernel<SEG>;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)AD_SMEM) != cudaSuccess) return -1;
  const int kind = SEG ? K_RULE_SEGMENT : K_RULE_ADJOINT;
  timing_mark_begin(kind, st);
  kfn<<<dim3(a.units(), SEG ? sg.n - 1 : sg.n), 384, AD_SMEM, st>>>(a, (const uint8_t *)records, ao, sg, tail);
  timing_mark_end(kind, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}
}  // namespace

int launch_rule_adjoint_tails(const RuleArgs &a, const void *records, const RuleSegments &sg, cudaStream_t st) {
  return sg.n == 1 ? 0 : launch_adjoint<true>(a, records, RuleOperands{}, sg, true, st);
}
int launch_rule_adjoint_tc(const RuleArgs &a, const void *records, const RuleSegments &sg, const RuleOperands &ao,
                           cudaStream_t st) {
  if (sg.n > 1) {
    if (launch_adjoint<true>(a, records, RuleOperands{}, sg, false, st) != 0) return -1;
    timing_mark_begin(K_RULE_JOIN, st);
    mesa_rule_join_adjoint_kernel<<<dim3(8, a.units()), 256, 0, st>>>(sg, a.dS_final);
    timing_mark_end(K_RULE_JOIN, st);
    if (cudaPeekAtLastError() != cudaSuccess) return -1;
  }
  return launch_adjoint<false>(a, records, ao, sg, false, st);
}

int launch_rule_grads_tc(const RuleArgs &a, const void *records, const RuleOperands &so, const RuleOperands &ao,
                         float *dqp, float *dkp, cudaStream_t st) {
  CUtensorMap mapDq{}, mapDk{};
  if (!tmap_units128_bf16(&mapDq, a.dq, a.B * a.Hk, a.T) || !tmap_units128_bf16(&mapDk, a.dk_out, a.B * a.Hk, a.T)) return -1;
  if (cudaFuncSetAttribute(mesa_rule_grads_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)GR_SMEM) != cudaSuccess)
    return -1;
  timing_mark_begin(K_RULE_GRADS, st);
  const int NC = (a.T + C - 1) / C, chunks = NC * a.units(), sms = sm_count();
  mesa_rule_grads_tc_kernel<<<chunks < sms ? chunks : sms, 32 * GR_WARPS, GR_SMEM, st>>>(
      a, NC, chunks, (const uint8_t *)records, so, ao, dqp, dkp, mapDq, mapDk);
  timing_mark_end(K_RULE_GRADS, st);
  if (cudaPeekAtLastError() != cudaSuccess) return -1;
  return dqp ? launch_rule_group_sum(a, dqp, dkp, st) : 0;
}

}  // namespace mesa
