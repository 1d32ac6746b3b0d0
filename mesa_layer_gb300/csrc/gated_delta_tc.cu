// gated_delta_tc.cu -- the gated delta rule's chunked forward on the tensor cores (bf16,
// dk = dv = 128; the chunk algebra and the operand formats are in gated_delta_tc.cuh).
//
// Two kernels.  mesa_rule_prep_kernel, one CTA per chunk: K K^T and Q K^T in one product, the
// decays, the inverse factor by substitution.  mesa_rule_chain_kernel, one CTA per unit: walks
// the chunks with the state in registers (thread r holds row r, 128 values) and everything
// laid out by state row, so that the chain of a chunk never crosses threads:
//     D1 = S0 K^T          -> R = V^T - f D1      (row r of the accumulator is thread r's)
//     D2 = R (T beta)^T    -> U
//     dS = (c U) K         -> S = f_last S0 + dS
// with S0, R and U written back to tensor memory as the next product's A operand.  The
// readout O = f (S0 Q^T) + U P^T runs beside the chain and leaves one chunk later, while the next
// chunk's first product runs.  Four more warps fetch the next chunk's rows and convert them.
#include "gated_delta_tc.cuh"

namespace mesa {

using namespace rule;

namespace {

// ---- per-chunk preparation --------------------------------------------------------------------
constexpr int A_LD = 68;  // row stride of the fp32 triangle in shared memory
constexpr uint32_t PREP_TILE = 0, PREP_M = TILE, PREP_P = PREP_M + SQ, PREP_MISC = PREP_P + SQ;
struct PrepMisc {
  float l[C], beta[C], f[C], c[C], red[8];
  int z[C];
  uint64_t mbar, drain;
  uint32_t tmem;
};
constexpr uint32_t PREP_SMEM = PREP_MISC + sizeof(PrepMisc) + 1024;
static_assert(C * A_LD * 4 <= TILE, "the triangle reuses the operand tile");

// Rows FROM .. C-1 of column `col` of (I + A)^-1 by substitution, for a column >= FROM; A in
// shared memory, the same element for every lane of a warp (a broadcast).  put(i, value).
template <int FROM, typename Put>
__device__ __forceinline__ void solve_column(const float *A, int col, Put put) {
  float t[C - FROM];
#pragma unroll
  for (int i = FROM; i < C; i++) {
    float s[4] = {i == col ? 1.0f : 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j4 = FROM; j4 < i; j4 += 4) {
      const float4 a = *reinterpret_cast<const float4 *>(A + i * A_LD + j4);
      s[0] = fmaf(-a.x, t[j4 - FROM], s[0]);
      if (j4 + 1 < i) s[1] = fmaf(-a.y, t[j4 + 1 - FROM], s[1]);
      if (j4 + 2 < i) s[2] = fmaf(-a.z, t[j4 + 2 - FROM], s[2]);
      if (j4 + 3 < i) s[3] = fmaf(-a.w, t[j4 + 3 - FROM], s[3]);
    }
    t[i - FROM] = (s[0] + s[1]) + (s[2] + s[3]);
    put(i, t[i - FROM]);
  }
}

// grid (NC, U), 128 threads.  with_beta: the record's factor is T diag(beta), else T.
__global__ void __launch_bounds__(128) mesa_rule_prep_kernel(RuleArgs a, TcWorkspace ws, bool with_beta) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  PrepMisc *m = reinterpret_cast<PrepMisc *>(sm + PREP_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, u = blockIdx.y, NC = gridDim.x, t0 = c * C, n = min(C, a.T - t0);
  const size_t row0 = (size_t)a.qk_unit(u) * a.T + t0, tok0 = (size_t)u * a.T + t0;

  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 64);
  if (tid == 32) {
    tc::mbar_init(tc::smem_u32(&m->mbar), 1);
    tc::mbar_init(tc::smem_u32(&m->drain), 1);
  }
  if (tid < C) m->beta[tid] = tid < n ? a.beta[tok0 + tid] : 0.0f;
  if (warp == 2) {
    const GatePair g = gate_scan(a.gamma + tok0, n, lane);
    m->l[2 * lane] = g.l0;
    m->l[2 * lane + 1] = g.l1;
    m->z[2 * lane] = g.z0;
    m->z[2 * lane + 1] = g.z1;
    const float end = __shfl_sync(0xffffffffu, g.l1, 31);
    const int zend = __shfl_sync(0xffffffffu, g.z1, 31);
    m->f[2 * lane] = g.z0 == 0 ? exp2f(g.l0) : 0.0f;
    m->f[2 * lane + 1] = g.z1 == 0 ? exp2f(g.l1) : 0.0f;
    m->c[2 * lane] = g.z0 == zend ? exp2f(end - g.l0) : 0.0f;
    m->c[2 * lane + 1] = g.z1 == zend ? exp2f(end - g.l1) : 0.0f;
  }
  // rows of K and Q: 16 threads a row, 8 rows a pass
  const int rr = tid >> 4, c8 = tid & 15;
  uint4 kr[8], qr[8];
  float mk = 0.0f, mq = 0.0f;
#pragma unroll
  for (int p = 0; p < 8; p++) {
    const int r = 8 * p + rr;
    kr[p] = qr[p] = make_uint4(0, 0, 0, 0);
    if (r < n) {
      kr[p] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.k + (row0 + r) * D + 8 * c8);
      qr[p] = *reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.q + (row0 + r) * D + 8 * c8);
    }
    mk = fmaxf(mk, absmax8(kr[p]));
    mq = fmaxf(mq, absmax8(qr[p]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
    mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, o));
  }
  if (lane == 0) {
    m->red[warp] = mk;
    m->red[4 + warp] = mq;
  }
  __syncthreads();
  const float sk = tile_scale(fmaxf(fmaxf(m->red[0], m->red[1]), fmaxf(m->red[2], m->red[3])));
  const float sq = tile_scale(fmaxf(fmaxf(m->red[4], m->red[5]), fmaxf(m->red[6], m->red[7])));
  if (tid == 0) ws.scales[(size_t)u * NC + c] = make_float2(sk, sq);
  const u64 sk2 = pack2(sk, sk), sq2 = pack2(sq, sq);
#pragma unroll
  for (int p = 0; p < 8; p++) {
    const int r = 8 * p + rr;
    *reinterpret_cast<uint4 *>(sm + PREP_TILE + tile_off(r, c8, 128)) = to_half8(kr[p], sk2);
    *reinterpret_cast<uint4 *>(sm + PREP_TILE + tile_off(C + r, c8, 128)) = to_half8(qr[p], sq2);
  }
  tc::fence_smem_to_async();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = m->tmem, bar = tc::smem_u32(&m->mbar);
  if (tid == 0) {  // rows 0..63: K K^T, rows 64..127: Q K^T
    const uint32_t id = tc::idesc_f16(128, C, false, false), at = tc::smem_u32(sm + PREP_TILE);
#pragma unroll
    for (int s = 0; s < 8; s++)
      tc::mma_f16(tbase, tc::kmajor_desc(at, 128, s), tc::kmajor_desc(at, 128, s), id, s > 0);
    tc::mma_commit(bar);
  }
  const bool done = tc::mbar_wait(bar, 0, a.wait_limit);
  tc::fence_after_sync();
  if (__syncthreads_or(!done)) {
    if (tid == 0) atomicOr(a.status, tc::kErrMmaTimeout);
    tc::drain_mmas(tc::smem_u32(&m->drain), tid == 0, a.status);
  } else {
    const int i = tid & 63;
    const float li = m->l[i];
    const int zi = m->z[i];
    const float mul = tid < C ? m->beta[i] / (sk * sk) : 1.0f;
    float *A = reinterpret_cast<float *>(sm + PREP_TILE);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      float v[32];
      tc::tmem_ld32(tbase + ((uint32_t)(32 * warp) << 16) + 32 * h, v);
      tc::tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 32; k++) {
        const int j = 32 * h + k;
        const bool keep = (tid < C ? j < i : j <= i) && m->z[j] == zi;
        v[k] = keep ? v[k] * mul * exp2f(li - m->l[j]) : 0.0f;
      }
      if (tid < C) {
#pragma unroll
        for (int k = 0; k < 8; k++)
          *reinterpret_cast<float4 *>(A + i * A_LD + 32 * h + 4 * k) =
              make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; k++) {
          float4 o;
          o.x = half2_bits(v[8 * k], v[8 * k + 1]);
          o.y = half2_bits(v[8 * k + 2], v[8 * k + 3]);
          o.z = half2_bits(v[8 * k + 4], v[8 * k + 5]);
          o.w = half2_bits(v[8 * k + 6], v[8 * k + 7]);
          *reinterpret_cast<float4 *>(sm + PREP_P + tile_off(i, 4 * h + k, C)) = o;
        }
      }
    }
    tc::fence_before_sync();
    __syncthreads();
    if (tid < C) {
      const float b = with_beta ? m->beta[tid] : 1.0f;
      auto put = [&](int r, float t) {
        *reinterpret_cast<__half *>(sm + PREP_M + tc::sw128_offset(r, tid, C)) = __float2half_rn(t * b);
      };
      if (tid < 32) {
        solve_column<0>(A, tid, put);
      } else {
        for (int r = 0; r < 32; r++) put(r, 0.0f);
        solve_column<32>(A, tid, put);
      }
    }
    tc::fence_smem_to_async();
    __syncthreads();
    uint8_t *rec = ws.rec + ((size_t)u * NC + c) * REC;
    if (tid == 0) {
      bulk_s2g(rec, tc::smem_u32(sm + PREP_M), 2 * SQ);
      tc::bulk_commit();
      tc::bulk_wait_all();
    } else if (tid >= 64) {
      reinterpret_cast<float *>(rec + REC_F)[tid - 64] = m->f[tid - 64];
      reinterpret_cast<float *>(rec + REC_C)[tid - 64] = m->c[tid - 64];
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 64);
}

// ---- the chain ----------------------------------------------------------------------------------
// shared memory: two operand tiles | two records | two value tiles | raw K and Q | output | misc
constexpr uint32_t CH_TILE = 0, CH_REC = CH_TILE + 2 * TILE, CH_RECP = 17 * 1024;
constexpr uint32_t CH_V = CH_REC + 2 * CH_RECP, CH_RAW = CH_V + 2 * ROWS64, CH_OUT = CH_RAW + 2 * ROWS64;
constexpr uint32_t CH_MISC = CH_OUT + ROWS64;
struct ChainMisc {
  uint64_t kq_full, vm_full[2], tile_full[2], slot_free[2], mma1, mma2, mma3, mma4, drain;
  uint32_t tmem;
  int gave_up;
};
constexpr uint32_t CH_SMEM = CH_MISC + sizeof(ChainMisc) + 1024;
static_assert(CH_RECP >= REC && CH_SMEM <= 232448, "shared memory layout");
// tensor memory columns: dS | S0 operand | D1, R | D2, U and c U | O from S0 | O from U
constexpr uint32_t T_DS = 0, T_S = 128, T_D1 = 192, T_D2 = 256, T_O1 = 320, T_O2 = 384;

// grid U, 256 threads: warps 0-3 the chain (thread r: state row r), warps 4-7 fetch and convert.
__global__ void __launch_bounds__(256, 1) mesa_rule_chain_kernel(RuleArgs a, TcWorkspace ws) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  ChainMisc *m = reinterpret_cast<ChainMisc *>(sm + CH_MISC);
  const int tid = threadIdx.x, warp = tid >> 5, u = blockIdx.x, T = a.T, NC = (T + C - 1) / C;
  const uint32_t kqb = tc::smem_u32(&m->kq_full);
  const uint32_t vmb[2] = {tc::smem_u32(&m->vm_full[0]), tc::smem_u32(&m->vm_full[1])};
  const uint32_t tfb[2] = {tc::smem_u32(&m->tile_full[0]), tc::smem_u32(&m->tile_full[1])};
  const uint32_t sfb[2] = {tc::smem_u32(&m->slot_free[0]), tc::smem_u32(&m->slot_free[1])};
  const uint32_t b1 = tc::smem_u32(&m->mma1), b2 = tc::smem_u32(&m->mma2), b3 = tc::smem_u32(&m->mma3),
                 b4 = tc::smem_u32(&m->mma4);
  volatile int *gave_up = &m->gave_up;
  const size_t v0 = (size_t)u * T * D, qk0 = (size_t)a.qk_unit(u) * T * D;

  auto fetch_kq = [&](int c) {
    const uint32_t bytes = (uint32_t)min(C, T - c * C) * D * 2;
    tc::mbar_arrive_expect_tx(kqb, 2 * bytes);
    tc::bulk_g2s(tc::smem_u32(sm + CH_RAW), (const __nv_bfloat16 *)a.k + qk0 + (size_t)c * C * D, bytes, kqb);
    tc::bulk_g2s(tc::smem_u32(sm + CH_RAW + ROWS64), (const __nv_bfloat16 *)a.q + qk0 + (size_t)c * C * D, bytes, kqb);
  };
  auto fetch_vm = [&](int c) {
    const int b = c & 1;
    const uint32_t bytes = (uint32_t)min(C, T - c * C) * D * 2;
    tc::mbar_arrive_expect_tx(vmb[b], bytes + REC);
    tc::bulk_g2s(tc::smem_u32(sm + CH_V + b * ROWS64), (const __nv_bfloat16 *)a.v + v0 + (size_t)c * C * D, bytes, vmb[b]);
    tc::bulk_g2s(tc::smem_u32(sm + CH_REC + b * CH_RECP), ws.rec + ((size_t)u * NC + c) * REC, REC, vmb[b]);
  };
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 128) {
    tc::mbar_init(kqb, 1);
    for (int b = 0; b < 2; b++) {
      tc::mbar_init(vmb[b], 1);
      tc::mbar_init(tfb[b], 1);
      tc::mbar_init(sfb[b], 1);
    }
    for (uint32_t b : {b1, b2, b3, b4, tc::smem_u32(&m->drain)}) tc::mbar_init(b, 1);
    m->gave_up = 0;
    fetch_kq(0);
    fetch_vm(0);
    if (NC > 1) fetch_vm(1);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = m->tmem;
  bool ok = true;
  int kq_sent = 1, vm_sent = min(NC, 2);

  if (warp >= 4) {
    // ---- fetch and convert ----
    const int h = tid - 128;
    float2 sc = ws.scales[(size_t)u * NC];
    for (int c = 0; c < NC; c++) {
      const int b = c & 1, n = min(C, T - c * C);
      ok = wait(kqb, c & 1, a.wait_limit, gave_up);
      if (c >= 2) ok &= wait(sfb[b], ((c >> 1) - 1) & 1, a.wait_limit, gave_up);
      if (group_or(2, 128, !ok)) {
        ok = false;
        break;
      }
      if (h == 0 && c >= 2) fetch_vm(c);
      if (c >= 2) vm_sent++;
      const u64 sk2 = pack2(sc.x, sc.x), sq2 = pack2(sc.y, sc.y);
      if (c + 1 < NC) sc = ws.scales[(size_t)u * NC + c + 1];
      uint8_t *tile = sm + CH_TILE + b * TILE;
#pragma unroll 4
      for (int p = 0; p < 8; p++) {
        const int i = h + 128 * p, r = i >> 4, c8 = i & 15;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (r < n) {
          x = *reinterpret_cast<const uint4 *>(sm + CH_RAW + 16 * i);
          y = *reinterpret_cast<const uint4 *>(sm + CH_RAW + ROWS64 + 16 * i);
        }
        *reinterpret_cast<uint4 *>(tile + tile_off(r, c8, 128)) = to_half8(x, sk2);
        *reinterpret_cast<uint4 *>(tile + tile_off(C + r, c8, 128)) = to_half8(y, sq2);
      }
      // (rows past the end of the values: the factor's columns there are zero, the values have
      // to be finite)
      for (int i = h + n * (D / 8); i < C * (D / 8); i += 128)
        *reinterpret_cast<uint4 *>(sm + CH_V + b * ROWS64 + 16 * i) = make_uint4(0, 0, 0, 0);
      tc::fence_smem_to_async();
      group_or(2, 128, false);
      if (h == 0) mbar_arrive(tfb[b]);
      if (c + 1 < NC) {
        if (h == 0) fetch_kq(c + 1);
        kq_sent++;
      }
    }
    if (!ok && h == 0) m->gave_up = 1;
  } else {
    // ---- the chain ----
    const int r = tid;
    const uint32_t tl = tbase + ((uint32_t)(32 * warp) << 16);
    const uint32_t idKK = tc::idesc_f16(128, C, false, false);   // N = 64 tokens, B K-major
    const uint32_t idKN = tc::idesc_f16(128, D, false, true);    // N = 128 channels, B MN-major
    float2 sc = ws.scales[(size_t)u * NC];
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
    // S (this thread's row) as the fp16 A operand
    auto stage_state = [&]() {
      float mx = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 2; i++) {
        float x, y;
        unpack2(S[i], x, y);
        mx = fmaxf(mx, fmaxf(fabsf(x), fabsf(y)));
      }
      sS = tile_scale(mx);
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
    };
    stage_state();
    tc::tmem_st_wait();

    float o1 = 0.0f, o2 = 0.0f;  // factors of the last chunk's readout accumulators
    float nonfinite = 0.0f;      // NaN once an output was not finite
    // the readout of chunk c: tensor memory -> bf16 rows in shared memory
    auto readout = [&](int c) {
      const float *f = reinterpret_cast<const float *>(sm + CH_REC + (c & 1) * CH_RECP + REC_F);
      const u64 w1 = pack2(o1, o1), w2 = pack2(o2, o2);
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float x[32], y[32];
        tc::tmem_ld32(tl + T_O1 + 32 * h, x);
        tc::tmem_ld32(tl + T_O2 + 32 * h, y);
        tc::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(f + 32 * h + k);
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const u64 w = mul2(e ? ff.y : ff.x, w1);
            float p, q;
            unpack2(fma2(pack2(x[k + e], x[k + e + 1]), w, mul2(pack2(y[k + e], y[k + e + 1]), w2)), p, q);
            nonfinite = fmaf(p, 0.0f, fmaf(q, 0.0f, nonfinite));
            __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(sm + CH_OUT) + (32 * h + k + e) * D + r;
            dst[0] = __float2bfloat16_rn(p);
            dst[D] = __float2bfloat16_rn(q);
          }
        }
      }
    };
    auto send_out = [&](int c) {  // thread 0
      const uint32_t bytes = (uint32_t)min(C, T - c * C) * D * 2;
      bulk_s2g((__nv_bfloat16 *)a.out + v0 + (size_t)c * C * D, tc::smem_u32(sm + CH_OUT), bytes);
      tc::bulk_commit();
    };

    for (int c = 0; c < NC; c++) {
      const int b = c & 1;
      const uint32_t ph = c & 1, tile = tc::smem_u32(sm + CH_TILE + b * TILE),
                     rec = tc::smem_u32(sm + CH_REC + b * CH_RECP);
      const float *f = reinterpret_cast<const float *>(sm + CH_REC + b * CH_RECP + REC_F), *cc = f + C;
      ok &= wait(tfb[b], (c >> 1) & 1, a.wait_limit, gave_up);
      ok &= wait(vmb[b], (c >> 1) & 1, a.wait_limit, gave_up);
      if (r == 0) tc::bulk_wait_read();  // the last chunk's output has left its buffer
      tc::fence_before_sync();
      if (group_or(1, 128, !ok)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (r == 0) {
#pragma unroll
        for (int s = 0; s < 8; s++) tc::mma_f16_ts(tbase + T_D1, tbase + T_S + 8 * s, tc::kmajor_desc(tile, 128, s), idKK, s > 0);
        tc::mma_commit(b1);
      }
      if (c > 0) {  // the last chunk's readout, while the first product runs
        ok &= wait(b4, (c - 1) & 1, a.wait_limit, gave_up);
        tc::fence_after_sync();
        readout(c - 1);
        tc::fence_smem_to_async();
      }
      tc::fence_before_sync();
      if (group_or(1, 128, !ok)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (r == 0) {
        if (c > 0) {
          send_out(c - 1);
          mbar_arrive(sfb[b ^ 1]);  // the last chunk's tiles and records are free
        }
#pragma unroll
        for (int s = 0; s < 8; s++)
          tc::mma_f16_ts(tbase + T_O1, tbase + T_S + 8 * s, tc::kmajor_desc(tile + C * 128, 128, s), idKK, s > 0);
      }
      // R = V^T - f D1
      ok &= wait(b1, ph, a.wait_limit, gave_up);
      tc::fence_after_sync();
      const float d1 = -1.0f / (sS * sc.x);  // (powers of two)
      o1 = a.scale / (sS * sc.y);
      float sR;
      {
        const uint16_t *V = reinterpret_cast<const uint16_t *>(sm + CH_V + b * ROWS64) + r;
        const u64 w1 = pack2(d1, d1);
        u64 R[C / 2];
        float mx = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float x[32];
          tc::tmem_ld32(tl + T_D1 + 32 * h, x);
          tc::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(f + 32 * h + k);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const int i = 32 * h + k + e;
              const u64 vv = pack2(__uint_as_float((uint32_t)V[i * D] << 16), __uint_as_float((uint32_t)V[(i + 1) * D] << 16));
              R[i / 2] = fma2(pack2(x[k + e], x[k + e + 1]), mul2(e ? ff.y : ff.x, w1), vv);
              float p, q;
              unpack2(R[i / 2], p, q);
              mx = fmaxf(mx, fmaxf(fabsf(p), fabsf(q)));
            }
          }
        }
        sR = tile_scale(mx);
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
      if (group_or(1, 128, !ok)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (r == 0) {
#pragma unroll
        for (int s = 0; s < 4; s++)
          tc::mma_f16_ts(tbase + T_D2, tbase + T_D1 + 8 * s, tc::kmajor_desc(rec, C, s), idKK, s > 0);
        tc::mma_commit(b2);
      }
      // U, for the readout, and c U, for the state
      ok &= wait(b2, ph, a.wait_limit, gave_up);
      tc::fence_after_sync();
      float sU;  // the operands hold U sU sR
      {
        float x[32], y[32];
        tc::tmem_ld32(tl + T_D2, x);
        tc::tmem_ld32(tl + T_D2 + 32, y);
        tc::tmem_ld_wait();
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; i++) mx = fmaxf(mx, fmaxf(fabsf(x[i]), fabsf(y[i])));
        sU = tile_scale(mx);
        const u64 s2 = pack2(sU, sU);
#pragma unroll
        for (int h = 0; h < 2; h++) {
          float v[16], w[16];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            const ulonglong2 ff = *reinterpret_cast<const ulonglong2 *>(cc + 32 * h + k);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float *z = h ? y : x;
              const u64 g = mul2(pack2(z[k + e], z[k + e + 1]), s2);
              float p, q;
              unpack2(g, p, q);
              v[(k + e) / 2] = half2_bits(p, q);
              unpack2(mul2(g, e ? ff.y : ff.x), p, q);
              w[(k + e) / 2] = half2_bits(p, q);
            }
          }
          tc::tmem_st16(tl + T_D2 + 16 * h, v);
          tc::tmem_st16(tl + T_D2 + 32 + 16 * h, w);
        }
        tc::tmem_st_wait();
      }
      tc::fence_before_sync();
      if (group_or(1, 128, !ok)) {
        ok = false;
        break;
      }
      tc::fence_after_sync();
      if (r == 0) {
#pragma unroll
        for (int s = 0; s < 4; s++)
          tc::mma_f16_ts(tbase + T_DS, tbase + T_D2 + 32 + 8 * s, tc::mnmajor_desc(tile, 128, s), idKN, s > 0);
        tc::mma_commit(b3);
#pragma unroll
        for (int s = 0; s < 4; s++)
          tc::mma_f16_ts(tbase + T_O2, tbase + T_D2 + 8 * s, tc::kmajor_desc(rec + REC_P, C, s), idKK, s > 0);
        tc::mma_commit(b4);
      }
      // the state after the chunk
      const float us = sU * sR;
      o2 = a.scale / (us * sc.x * sc.y);
      const u64 ds = pack2(1.0f / (us * sc.x), 1.0f / (us * sc.x)), dec = pack2(f[C - 1], f[C - 1]);
      if (c + 1 < NC) sc = ws.scales[(size_t)u * NC + c + 1];
      ok &= wait(b3, ph, a.wait_limit, gave_up);
      tc::fence_after_sync();
#pragma unroll
      for (int k = 0; k < 4; k++) {
        float x[32];
        tc::tmem_ld32(tl + T_DS + 32 * k, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; i++)
          S[16 * k + i] = fma2(pack2(x[2 * i], x[2 * i + 1]), ds, mul2(S[16 * k + i], dec));
      }
      if (c + 1 < NC) {
        stage_state();
        tc::tmem_st_wait();
      }
      if (!ok) *gave_up = 1;  // (the vote is at the next barrier)
    }
    // the last chunk's readout
    if (!group_or(1, 128, !ok)) {
      ok &= wait(b4, (NC - 1) & 1, a.wait_limit, gave_up);
      tc::fence_after_sync();
      if (r == 0) tc::bulk_wait_read();
      ok = !group_or(1, 128, !ok);
      if (ok) {
        readout(NC - 1);
        tc::fence_smem_to_async();
      }
      group_or(1, 128, false);
      if (ok && r == 0) send_out(NC - 1);
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
      if (!(nonfinite == 0.0f)) atomicOr(a.status, tc::kErrNonFinite);
    } else {
      ok = false;
    }
    if (!ok && r == 0) {
      *gave_up = 1;
      atomicOr(a.status, tc::kErrMmaTimeout);
    }
    if (r == 0) tc::bulk_wait_all();
  }
  __syncthreads();
  // a wait gave up: products and copies still in flight finish before the memory is released
  if (*gave_up) {
    tc::drain_mmas(tc::smem_u32(&m->drain), tid == 0, a.status);
    if (tid == 128) {
      bool in = tc::mbar_wait(kqb, (kq_sent - 1) & 1, tc::kWaitLimit);
      for (int s = max(0, vm_sent - 2); s < vm_sent; s++) in &= tc::mbar_wait(vmb[s & 1], (s >> 1) & 1, tc::kWaitLimit);
      if (!in) atomicOr(a.status, tc::kErrDrainTimeout);
      atomicOr(a.status, tc::kErrMmaTimeout);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) tc::tmem_free(tbase, 512);
}

}  // namespace

size_t rule_tc_workspace(int U, int T) {
  const size_t NC = ((size_t)T + C - 1) / C;
  return (size_t)U * NC * REC + (((size_t)U * NC * sizeof(float2) + 255) & ~(size_t)255);
}

int launch_rule_forward_tc(const RuleArgs &a, void *workspace, cudaStream_t st) {
  const int U = a.units(), NC = (a.T + C - 1) / C;
  TcWorkspace ws{(uint8_t *)workspace, (float2 *)((uint8_t *)workspace + (size_t)U * NC * REC)};
  if (cudaFuncSetAttribute(mesa_rule_prep_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PREP_SMEM) !=
          cudaSuccess ||
      cudaFuncSetAttribute(mesa_rule_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CH_SMEM) !=
          cudaSuccess)
    return -1;
  timing_mark_begin(K_RULE_PREP, st);
  mesa_rule_prep_kernel<<<dim3(NC, U), 128, PREP_SMEM, st>>>(a, ws, true);
  timing_mark_end(K_RULE_PREP, st);
  timing_mark_begin(K_RULE_CHAIN, st);
  mesa_rule_chain_kernel<<<U, 256, CH_SMEM, st>>>(a, ws);
  timing_mark_end(K_RULE_CHAIN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mesa
