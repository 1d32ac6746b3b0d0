// gated_delta_tc.cu -- the gated delta rule's chunked forward on the tensor cores (bf16,
// dk = dv = 128; the chunk algebra and the operand formats are in gated_delta_tc.cuh).
//
// Two kernels.  mesa_rule_prep_kernel, one CTA per chunk: K K^T and Q K^T in one product, decays,
// masks and the triangular inverse, written as a record.  mesa_rule_chain_kernel, one CTA per
// unit (or segment of a unit), walks the unit's chunks with the state in registers (thread r of the chain holds row r,
// 128 values) and everything laid out by state row, so that a chunk's chain of dependent
// products never crosses threads:
//     D1 = S0 K^T          -> R = V^T - f D1      (row r of the accumulator is thread r's)
//     D2 = R (T beta)^T    -> U
//     dS = (c U) K         -> S = f_last S0 + dS
// with S0, R and U written back to tensor memory as the next product's A operand.  The readout
// O = f (S0 Q^T) + U P^T shares the first product (K and Q rows are one operand tile).  The chain
// bounds the kernel, so all else runs beside it, in warp groups of their own:
//     chain    the three epilogues above;
//     helper   writes the readout (and with the transposition, too, it held up the chain: 188 us);
//     convert  V transposed one chunk ahead, K and Q as fp16 operands, up to three chunks ahead.
// Measured at 8 x 16 x 4096 (8192 chunks): preparation 120 us (400 MB of rows and records: 3.3 TB/s; the
// substitution's latency and instruction fetch; 10 us of it for the second fp16 value of A's blocks), chain
// 180 us (64 dependent steps of 2.8 us; issue slots
// 37 %, tensor pipe 19 % busy: the latency of four products and three epilogues a step, 128 of 152 SMs).
// (With the preparation in the same kernel, as a fourth group, nothing but the inputs and the output
// went to memory, but the groups' code no longer fitted the instruction caches and every
// group slowed down: at best 268 us, at 8 x 16 x 4096, in some runs 300.)
#include "gated_delta_tc.cuh"

namespace mesa {

using namespace rule;

namespace {

// ---- per-chunk preparation --------------------------------------------------------------------
// shared memory: the operand tile, and once its products are done record | scratch in its place
// (36 KB: six CTAs on an SM hide each other's substitution) | misc
constexpr uint32_t PR_REC = 0, PR_SCR = REC;
constexpr uint32_t PR_MISC = (PR_SCR + sizeof(Factor) > TILE ? PR_SCR + sizeof(Factor) : TILE);
static_assert(PR_MISC % 16 == 0 && PR_SCR % 16 == 0, "alignment");
struct PrepMisc {
  alignas(16) uint32_t red[8];
  float grow[C], give[C];
  uint32_t vmax[4], gmax[4];
  uint64_t mbar, drain;
  uint32_t tmem;
};
constexpr uint32_t PR_SMEM = PR_MISC + sizeof(PrepMisc) + 1024;
static_assert(6 * (PR_SMEM + 1024) <= 228 * 1024, "six CTAs on an SM");

// grid (NC, U), 128 threads.  WITH_BETA: the record's factor is T diag(beta), else T.  bounds [U, NC]
// (or nullptr): log2 of how much of a state the chunk leaves, at most, the product over its tokens of
// gamma max(1, |1 - beta k.k|) (the norm of gamma (I - beta k k^T)); and a bound of the norm of what it adds
// to a row of the state, the largest |v| times the sum of beta |k|.  adds [U, NC] (or nullptr): the same of the
// adjoint before the chunk, from the largest |dout| and |q|.  Numbers that are none (or that could end
// in an overflow) bound nothing: infinity or NaN.
template <bool WITH_BETA>
__global__ void __launch_bounds__(128, 6) mesa_rule_prep_kernel(RuleArgs a, uint8_t *records, float2 *bounds, float *adds) {
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
  if (bounds) {  // the values, on their way during the products
    const uint4 *vp = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.v + tok0 * D);
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = 128 * i + tid < n * (D / 8) ? vp[128 * i + tid] : make_uint4(0, 0, 0, 0);
    if (!WITH_BETA && adds) {  // (the backward's)
      const uint4 *gp = reinterpret_cast<const uint4 *>((const __nv_bfloat16 *)a.dout + tok0 * D);
#pragma unroll
      for (int i = 0; i < 8; i++) y[i] = 128 * i + tid < n * (D / 8) ? gp[128 * i + tid] : make_uint4(0, 0, 0, 0);
    }
  }
  if (warp == 0 && elect_one()) {  // rows 0..63: K K^T, rows 64..127: Q K^T
    const uint32_t id = tc::idesc_f16(128, C, false, false);
    const uint64_t t = tc::kmajor_desc(tc::smem_u32(sm), 128, 0);
#pragma unroll
    for (int k = 0; k < 8; k++) tc::mma_f16(tbase, t + step128(k), t + step128(k), id, k > 0);
    tc::mma_commit(bar);
  }
  const bool done = tc::mbar_wait(bar, 0, a.wait_limit);
  tc::fence_after_sync();
  if (bounds) {
    uint32_t mv = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) mv = absmax_words(mv, x[i]);
    mv = absmax_fold(mv);
    if (lane == 0) m->vmax[warp] = mv;
    if (!WITH_BETA && adds) {
      mv = 0;
#pragma unroll
      for (int i = 0; i < 8; i++) mv = absmax_words(mv, y[i]);
      mv = absmax_fold(mv);
      if (lane == 0) m->gmax[warp] = mv;
    }
  }
  if (__syncthreads_or(!done)) {
    if (tid == 0) atomicOr(a.status, tc::kErrMmaTimeout);
    const bool issuer = warp == 0 && elect_one();
    tc::drain_mmas(tc::smem_u32(&m->drain), issuer, a.status);
  } else {
    if (tid == 0) *reinterpret_cast<float4 *>(inv) = make_float4(ik, iq, sk, sq);
    if (tid < C) s.beta[tid] = reinterpret_cast<float *>(rec + REC_B)[tid] = be;
    if (warp == 3) factor_gates(s, g, nf, cc, inv + 4, lane);
    factor_clear(rec + SQ, tid);
    __syncthreads();
    if (bounds && tid < C) {  // (the diagonal of K K^T: column i of row i)
      float kk = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; h++) {
        float x[16];
        tc::tmem_ld16(tbase + ((uint32_t)(32 * warp) << 16) + 32 * warp + 16 * h, x);
        tc::tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; k++)
          if (16 * h + k == lane) kk = x[k];
      }
      kk *= ik * ik;
      const float grow = fabsf(1.0f - be * kk);  // (0.003: k's rounding to fp16)
      const float up = s.l[tid] - (tid > 0 ? s.l[tid - 1] : 0.0f);  // (of a gate above 1)
      m->grow[tid] = (grow <= 1.0f ? 0.0f : grow < INFINITY ? log2f(grow) + 0.003f : INFINITY) + fmaxf(up, 0.0f);
      m->give[tid] = fabsf(be) * sqrtf(kk) * 1.002f;
    }
    factor_rows(s, tbase, ik * ik, inv[5], rec, rec + SQ, tid);
    tc::fence_before_sync();
    __syncthreads();
    if (bounds && warp == 3) {
      const float grow = warp_sum(m->grow[lane] + m->grow[lane + 32]), give = warp_sum(m->give[lane] + m->give[lane + 32]);
      const float vmax = __uint_as_float(max(max(m->vmax[0], m->vmax[1]), max(m->vmax[2], m->vmax[3])) << 16);
      const float add = vmax * give * exp2f(grow);
      if (lane == 0)
        bounds[(size_t)u * NC + c] = make_float2((s.z[C - 1] != 0 ? -1e30f : s.l[C - 1]) + grow, add < 1e30f ? add : INFINITY);
      if (!WITH_BETA && adds && lane == 0) {
        const float gmax = __uint_as_float(max(max(m->gmax[0], m->gmax[1]), max(m->gmax[2], m->gmax[3])) << 16);
        const float qmax = __uint_as_float(max(max(q4.x, q4.y), max(q4.z, q4.w)) << 16);
        const float g = fabsf(a.scale) * gmax * qmax * exp2f(grow) * (C * 11.4f);  // (C tokens, sqrt(D))
        adds[(size_t)u * NC + c] = g < 1e30f ? g : INFINITY;
      }
    }
    factor_diagonal<WITH_BETA>(s, rec, warp, lane);
    __syncthreads();
    if (warp < 3) factor_columns<WITH_BETA>(s, rec, warp, lane);
    __syncthreads();
    factor_clear_upper(rec, tid);
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
  float rest, rest0;  // a bound of what the chunks before can have left, of the part of S0 that can be left
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
// kFwd: the forward.  kKeep: the backward's pass over the states: the records hold T without beta, nothing
// is read out, and the state before each chunk and the chunk's u are kept as operands with one scale
// each (so.S, so.U).  Grid (U, segments): a segment's CTA starts from the state in sg.
// kSegment: what the segments start from: the state that segment y leaves when it starts from zero (the
// first: from S0), and, where that is not all, the matrix that takes the state before it to its part
// of the state after it (the rows of the identity without values).  First, grid (U, segments - 1): only
// the chunks at the segment's end of which 2^-40 of a state is left, from zero; that is all when the
// bounds of all that went before say that it adds less than 2^-26 of each row's largest element (the
// operands carry 2^-12).  Then, grid (U, segments - 1, 2), the segments where it was not: all their chunks
// (z = 0), the matrix (z = 1).
// kSegmentT: the same from records without beta.
enum ChainMode { kFwd = 0, kKeep = 1, kSegment = 2, kSegmentT = 3 };
template <int MODE>
__global__ void __launch_bounds__(384, 1)
    mesa_rule_chain_kernel(RuleArgs a, const uint8_t *records, RuleOperands so, RuleSegments sg,
                           const __grid_constant__ CUtensorMap mapV, const __grid_constant__ CUtensorMap mapO) {
  constexpr bool FWD = MODE == kFwd, KEEP = MODE == kKeep, SEG = MODE >= kSegment, BETA = KEEP || MODE == kSegmentT;
  constexpr int NT = KEEP ? 2 : 3;  // operand tiles
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = smem_raw + ((1024 - (tc::smem_u32(smem_raw) & 1023)) & 1023);
  ChainMisc *m = reinterpret_cast<ChainMisc *>(sm + CH_MISC);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // (warp: uniform)
  const int u = blockIdx.x, seg = blockIdx.y, T = a.T, NCT = (T + C - 1) / C;
  const bool identity = SEG && blockIdx.z == 1, tail = SEG && gridDim.z == 1;
  // this CTA's chunks: NC of them from c0 on (the loops count them from 0)
  int c0 = sg.n > 1 ? seg * sg.per : 0, NC = sg.n > 1 ? min(NCT - c0, sg.per) : NCT;
  const float *start = !SEG && sg.n > 1 ? sg.S + ((size_t)u * sg.n + seg) * D * D  // (nullptr: zero)
                       : a.S0         ? a.S0 + (size_t)u * D * D
                                      : nullptr;
  if constexpr (SEG) {
    int *whole = sg.whole + (size_t)u * sg.n + seg;
    if (seg > 0 || tail) start = nullptr;
    if (tail) {
      const int end = c0 + NC, lo = c0;
      float left = 0.0f;
      c0 = end;
      while (c0 > lo && !(left <= kLittle)) left += sg.bounds[(size_t)u * NCT + --c0].x;
      NC = end - c0;
      if (!(left <= kLittle)) {
        if (tid == 0) *whole = 1;
        return;
      }
      if (warp == 11) {  // what the chunks before c0 can have left: four a lane, backwards
        float rest = 0.0f;
        for (int j0 = c0; j0 > 0; j0 -= 128) {
          const int j = j0 - 1 - 4 * lane;
          float2 b[4];
#pragma unroll
          for (int i = 0; i < 4; i++) b[i] = j - i >= 0 ? sg.bounds[(size_t)u * NCT + j - i] : make_float2(0, 0);
          const float mine = b[0].x + b[1].x + b[2].x + b[3].x;
          float run = mine;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float x = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += x;
          }
          const float total = __shfl_sync(0xffffffffu, run, 31);
          float after = left + __shfl_up_sync(0xffffffffu, run, 1);
          if (lane == 0) after = left;
#pragma unroll
          for (int i = 0; i < 4; i++) {
            rest = fmaf(b[i].y, exp2f(after), rest);
            after += b[i].x;
          }
          left += total;
        }
        rest = warp_sum(rest);
        if (lane == 0) {
          m->rest = rest;
          m->rest0 = exp2f(left);  // of S0
        }
      }
    } else if (identity ? seg == 0 || (!*whole && !(sg.whole_adj && sg.whole_adj[(size_t)u * sg.n + seg])) : !*whole) {
      return;
    }
  }
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  volatile int *gave_up = &m->gave_up;
  const unsigned limit = a.wait_limit;

  auto fetch_v = [&](int c) {
    const uint32_t b = bar(m->v_full), dst = tc::smem_u32(sm + CH_V);
    tc::mbar_arrive_expect_tx(b, ROWS64);
#pragma unroll
    for (int h = 0; h < 2; h++) tensor_g2s_3d(dst + h * C * 128, &mapV, 64 * h, (c0 + c) * C, u, b);
  };
  auto fetch_rec = [&](int c) {
    const uint32_t b = bar(m->rec_full[c % 3]);
    tc::mbar_arrive_expect_tx(b, REC);
    tc::bulk_g2s(tc::smem_u32(sm + CH_REC + (c % 3) * REC_PAD), records + ((size_t)u * NCT + c0 + c) * REC, REC, b);
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
  int v_sent = 1, rec_sent = min(NC, 3);  // fetches issued (threads 256 and 128)

  if (warp < 4) {
    // ---- the chain: thread r holds row r of the state ----
    regs_up<kRegChain>();
    const int r = tid;
    const uint32_t tl = tbase + ((uint32_t)(32 * warp) << 16);
    u64 S[D / 2];
    {
      const float4 *src = start ? reinterpret_cast<const float4 *>(start + (size_t)r * D) : nullptr;
#pragma unroll
      for (int g = 0; g < D / 4; g++) {
        float4 x = src ? src[g] : make_float4(0, 0, 0, 0);
        if (identity)
          x = make_float4(r == 4 * g ? 1.0f : 0.0f, r == 4 * g + 1 ? 1.0f : 0.0f, r == 4 * g + 2 ? 1.0f : 0.0f,
                          r == 4 * g + 3 ? 1.0f : 0.0f);
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
      return KEEP ? fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) : b;
    };
    auto put_rows = [&](float b) {
      const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(b));
      if (lane == 0) m->bmax[warp] = __uint_as_float(w);
    };
    auto keep_words = [&](int k, const float (&v)[8]) {  // columns 16 k .. of this row, on their way out
      *reinterpret_cast<float4 *>(sm + CH_STAGE + tile_off(r, 2 * k, 128)) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(sm + CH_STAGE + tile_off(r, 2 * k + 1, 128)) = make_float4(v[4], v[5], v[6], v[7]);
    };
    if constexpr (KEEP) {
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
        if constexpr (KEEP) keep_words(k, v);
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
      if constexpr (KEEP) tc::fence_smem_to_async();
      if (meet()) break;
      if (warp == 0 && elect_one()) {
        const uint64_t kq = tc::kmajor_desc(tile, 128, 0);
#pragma unroll
        for (int s = 0; s < 8; s++)  // S0 K^T and S0 Q^T (one product), or the first alone
          tc::mma_f16_ts(tbase + T_D1, tbase + T_S + 8 * s, kq + step128(s), FWD ? id128 : id64, s > 0);
        tc::mma_commit(bar(m->mma1));
      }
      if constexpr (KEEP) {
        if (r == 32) {
          const size_t at = (size_t)u * NCT + c0 + c;
          bulk_s2g(so.S + at * TILE, tc::smem_u32(sm + CH_STAGE), TILE);
          tc::bulk_commit();
          so.iS[at] = iS;
        }
      }
      ok &= wait(bar(m->rec_full[c % 3]), (c / 3) & 1, limit, gave_up);
      ok &= wait(bar(m->vt_full), ph, limit, gave_up);
      // all: the chunk's decay; gm: no decay in it is greater
      const float iK = inv[0], kmax = (float)(1 << kTopTile) * iK, all = -nf[C - 1], gm = inv[4];
      if constexpr (FWD) m->o1[ph][r] = -a.scale * iS * inv[1];
      const float w1 = iS * iK;  // units of D1
      float iR;
      const float sR = bound_scale(fmaf((float)D * kmax * gm, bS, m->vmax[warp]), BETA ? kTopRow - 2 : kTopRow, iR);  // (beta < 4)
      const u64 w1_2 = pack2(w1, w1), sR2 = pack2(sR, sR);
      const float *be = cc + C;
      if constexpr (KEEP) m->o1[ph][r] = iR;
      ok &= wait(bar(m->mma1), ph, limit, gave_up);
      tc::fence_after_sync();
      // R = V^T - f D1, 16 tokens at a time (few registers beside the state's 128: what spills
      // here is paid for on the chain)
      {
        const uint8_t *V = sm + CH_VT + r * 256;
        float y[2][16];
        tc::tmem_ld16(tl + T_D1, y[0]);
#pragma unroll
        for (int h = 0; h < 4; h++) {
          float *z = y[h & 1];
          ulonglong2 vv[4], ff[4];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            ff[k] = *reinterpret_cast<const ulonglong2 *>(nf + 16 * h + 4 * k);
            vv[k] = *reinterpret_cast<const ulonglong2 *>(V + (((4 * h + k) ^ (r & 7)) << 4));
          }
          tc::tmem_ld_wait();
          if (h < 3) tc::tmem_ld16(tl + T_D1 + 16 * (h + 1), y[(h + 1) & 1]);
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; k++) {
            ulonglong2 bb = make_ulonglong2(sR2, sR2);
            if constexpr (BETA) {
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
        const float sU = bound_scale(uU * gm, kTopRow, iU);  // (c U, too)
        const u64 sU2 = pack2(sU, sU);
        float y[2][16];
        tc::tmem_ld16(tl + T_D2, y[0]);
#pragma unroll
        for (int h = 0; h < 4; h++) {
          float v[8], w[8], *x = y[h & 1];
          tc::tmem_ld_wait();
          if (h < 3) tc::tmem_ld16(tl + T_D2 + 16 * (h + 1), y[(h + 1) & 1]);
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
      // 64 products of |c u| <= gm |u| and |k| bound what is added to the state
      bS = fmaf(all, bS, (float)C * gm * uU * iR * kmax);
      if constexpr (FWD) {
        m->o2[ph][r] = a.scale * w3 * gm * inv[1];
      } else if constexpr (KEEP) {
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
        float y[2][16];  // these columns and the next ones, on their way
        tc::tmem_ld16(tl + T_DS, y[0]);
#pragma unroll
        for (int k = 0; k < 8; k++) {
          float v[8], *z = y[k & 1];
          tc::tmem_ld_wait();
          if (k < 7) tc::tmem_ld16(tl + T_DS + 16 * (k + 1), y[(k + 1) & 1]);
#pragma unroll
          for (int i = 0; i < 8; i++) {
            S[8 * k + i] = fma2(pack2(z[2 * i], z[2 * i + 1]), w3_2, mul2(S[8 * k + i], dec));
            v[i] = half2_bits(mul2(S[8 * k + i], sS2));
          }
          tc::tmem_st8(tl + T_S + 8 * k, v);  // the next chunk's operand
          if constexpr (KEEP) keep_words(k, v);
        }
        tc::tmem_st_wait();
      }
      if ((c & 7) == 7) row_max();  // (before the bound is loose)
    }
    if constexpr (KEEP) {
      if (r == 32) tc::bulk_wait_all();
    }
    float *final = SEG ? (identity ? sg.Tr : sg.loc) + ((size_t)u * sg.n + seg) * D * D
                   : FWD && a.S_final && c0 + NC == NCT ? a.S_final + (size_t)u * D * D : nullptr;
    if (SEG && tail) {  // is that all?  (a NaN or an infinity anywhere: no)
      row_max();
      float before = m->rest;
      if (a.S0) {
        const float *src = a.S0 + ((size_t)u * D + r) * D;
        float x = 0.0f;
        for (int j = 0; j < D; j++) x += fabsf(src[j]);
        before = fmaf(x, m->rest0, before);
      }
      const int more = group_or(1, 128, !(before <= 0x1p-26f * bS));
      if (r == 0) sg.whole[(size_t)u * sg.n + seg] = more;
    }
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
    // ---- write the readout ----
    regs_down<kRegHelper>();
    const int h = tid - 128;
    const uint32_t tl = tbase + ((uint32_t)(32 * (warp - 4)) << 16);
    const uint32_t id64 = tc::idesc_f16(128, C, false, false);
    u64 nonfinite = 0;  // a NaN once an output was not finite
    for (int c = 0; c < NC; c++) {
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
      if constexpr (SEG) {  // nothing to write
        warp_arrive(m->o_free);
        if (c + 3 < NC) {
          if (h == 0) fetch_rec(c + 3);
          rec_sent++;
        }
        continue;
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
      if constexpr (KEEP) {
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
            if constexpr (KEEP) {
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
          for (int b = 0; b < 2; b++) tensor_s2g_3d(&mapO, tc::smem_u32(sm + CH_OUT + b * C * 128), 64 * b, (c0 + c) * C, u);
        } else {
          const size_t at = (size_t)u * NCT + c0 + c;
          bulk_s2g(so.U + at * ROWS64, tc::smem_u32(sm + CH_OUT), ROWS64);
          so.iU[at] = iu;
        }
        tc::bulk_commit();
        if (c + 3 < NC) fetch_rec(c + 3);  // (the chain is past this record, and so is the group)
      }
      if (c + 3 < NC) rec_sent++;
    }
    if (!(sum2(nonfinite) == 0.0f)) atomicOr(a.status, tc::kErrNonFinite);
    if (h == 0) tc::bulk_wait_all();
  } else {
    // ---- K and Q as operands, up to three chunks in flight; the values transposed, one ahead ----
    regs_down<kRegConvert>();
    const int h = tid - 256, r0 = h >> 4, c8 = h & 15, uk = a.qk_unit(u);  // rows r0, r0 + 8 ..; 8 channels
    const size_t first = ((size_t)uk * T + (size_t)c0 * C + r0) * D + 8 * c8;
    const __nv_bfloat16 *kp = (const __nv_bfloat16 *)a.k + first, *qp = (const __nv_bfloat16 *)a.q + first;
    uint4 x[8], y[8];  // the next chunk's rows, on their way while this one's are converted,
    float2 scales;     // and its scales (not from the records in shared memory: those come later)
    auto load = [&](int c) {
      const int n = T - (c0 + c) * C - r0;
      scales = *reinterpret_cast<const float2 *>(records + ((size_t)u * NCT + c0 + c) * REC + REC_S + 8);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        x[i] = y[i] = make_uint4(0, 0, 0, 0);
        if (8 * i < n) {
          x[i] = *reinterpret_cast<const uint4 *>(kp + ((size_t)c * C + 8 * i) * D);
          if (FWD) y[i] = *reinterpret_cast<const uint4 *>(qp + ((size_t)c * C + 8 * i) * D);
        }
      }
    };
    auto transpose = [&](int c) -> bool {  // chunk c's values, once the last chunk's have been used
      if (group_or(3, 128, !(wait(bar(m->v_full), c & 1, limit, gave_up) &
                             (c == 0 || wait(bar(m->r_ready), (c - 1) & 1, limit, gave_up))))) return false;
      const uint32_t live = identity ? 0u : 0xffffffffu;  // (rows of the identity take no values)
      // channels 32 w .. 32 w + 31 by warp w: eight channels x 32 tokens at a time
      uint32_t mv = 0;
#pragma unroll 1
      for (int g = 0; g < 4; g++) {
        const int ch8 = 4 * (warp - 8) + g;
#pragma unroll
        for (int t = 0; t < 2; t++) {
          uint32_t x[4];
          ldmatrix_x4_trans(x, tc::smem_u32(sm + CH_V + tile_off(32 * t + lane, ch8, C)));
#pragma unroll
          for (int k = 0; k < 4; k++) x[k] &= live;
          mv = absmax_words(mv, make_uint4(x[0], x[1], x[2], x[3]));
          const int r = 8 * ch8 + (lane >> 2);
#pragma unroll
          for (int k = 0; k < 4; k++)  // tokens 32 t + 8 k + 2 (lane % 4), + 1
            *reinterpret_cast<float2 *>(sm + CH_VT + vt_off(r, 8 * t + 2 * k + ((lane & 3) >> 1)) + 8 * (lane & 1)) =
                make_float2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xffff0000u));
        }
      }
      mv = absmax_fold(mv);
      if (lane == 0) m->vmax[warp - 8] = __uint_as_float(mv << 16);  // of this warp's channels
      warp_arrive(m->vt_full);
      group_or(3, 128, false);
      if (c + 1 < NC) {
        if (h == 0) fetch_v(c + 1);
        v_sent++;
      }
      return true;
    };
    load(0);
    // tile 0, values 0, tiles up to NT - 1, then values c + 1 (once those of c are used) before tile c + NT
    for (int c = 0; c < NC + NT - 1; c++) {
      const int tv = c == 1 ? 0 : c < NT ? -1 : c - NT + 1;
      if (tv >= 0 && !transpose(tv)) {
        ok = false;
        break;
      }
      if (c >= NC) continue;
      const bool got = c < NT || wait(bar(m->tile_free[c % NT]), (c / NT - 1) & 1, limit, gave_up);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      const u64 sk2 = pack2(scales.x, scales.x), sq2 = pack2(scales.y, scales.y);
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
    if (tid == 256 && !tc::mbar_wait(bar(m->v_full), (v_sent - 1) & 1, tc::kWaitLimit)) atomicOr(a.status, tc::kErrDrainTimeout);
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

// The state before each segment from the segments' own: S_{y+1} = S_y Tr_y + loc_y (S_1 = loc_0; S_0 is a
// copy: the last segment may write its final state over the caller's), sixteen rows by a CTA of 256
// threads; grid (8, U).  A chain of steps that read a 64 KB matrix from the L2 cache with nothing on its way: 27 us
// each where matrices are applied, 1.2 where not.
__global__ void __launch_bounds__(256) mesa_rule_join_kernel(RuleSegments sg, const float *S0) {
  __shared__ float rows[16][D + 4];
  const int u = blockIdx.y, row0 = 16 * blockIdx.x, tid = threadIdx.x;
  const int r = tid >> 4, c0 = (tid & 15) * 8;  // row r, columns c0 ..
  for (int i = 0; i < 8; i++) {
    const size_t at = (size_t)(row0 + r) * D + c0 + i;
    sg.S[(size_t)u * sg.n * D * D + at] = S0 ? S0[(size_t)u * D * D + at] : 0.0f;
  }
  for (int y = 0; y + 1 < sg.n; y++) {
    const size_t at = (size_t)u * sg.n + y;
    const float *loc = sg.loc + at * D * D + (size_t)(row0 + r) * D + c0;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = loc[i];
    if (y > 0 && sg.whole[at]) {
      const float *Tr = sg.Tr + at * D * D + c0;
      for (int k = 0; k < D; k++) {
        const float s = rows[r][k];
        const float4 p = *reinterpret_cast<const float4 *>(Tr + (size_t)k * D);
        const float4 q = *reinterpret_cast<const float4 *>(Tr + (size_t)k * D + 4);
        x[0] = fmaf(s, p.x, x[0]);
        x[1] = fmaf(s, p.y, x[1]);
        x[2] = fmaf(s, p.z, x[2]);
        x[3] = fmaf(s, p.w, x[3]);
        x[4] = fmaf(s, q.x, x[4]);
        x[5] = fmaf(s, q.y, x[5]);
        x[6] = fmaf(s, q.z, x[6]);
        x[7] = fmaf(s, q.w, x[7]);
      }
    }
    __syncthreads();
    float *dst = sg.S + (at + 1) * D * D + (size_t)(row0 + r) * D + c0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      rows[r][c0 + i] = x[i];
      dst[i] = x[i];
    }
    __syncthreads();
  }
}

template <int MODE>
int launch_chain(const RuleArgs &a, const uint8_t *records, const RuleOperands &so, const RuleSegments &sg, dim3 grid,
                 const CUtensorMap &mapV, const CUtensorMap &mapO, cudaStream_t st) {
  auto kfn = mesa_rule_chain_kernel<MODE>;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)CH_SMEM) != cudaSuccess) return -1;
  timing_mark_begin(MODE >= kSegment ? K_RULE_SEGMENT : K_RULE_CHAIN, st);
  kfn<<<grid, 384, CH_SMEM, st>>>(a, records, so, sg, mapV, mapO);
  timing_mark_end(MODE >= kSegment ? K_RULE_SEGMENT : K_RULE_CHAIN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// Segments of a unit's NC chunks: as many CTAs as a GB300 has SMs (152), at least 20 chunks each, at most 24.
// They run one pass over a segment's chunks in place of one over the unit's, and the starts: the chunks at each
// segment's end where 20 of them forget (2^-40), else two more passes and the join, a chain of 27 us a
// step (34 in the backward) where matrices are applied.  us of a forward, one chain against n segments, gates
// about 0.98 / above 0.99999: 1 unit x 65536 tokens 2450, 24: 211 / 847, 152: 4090 / 4090; 16 x 65536 2800, 9: 641 /
// 1289; 1 x 8192 312, 6: 123 / 240, 19: 538 / 539; 16 x 8192 366, 6: 169 / 287; 16 x 4096 183, 5: 194 / 196, 9: 279 / 279;
// 16 x 2048 97, 5: 160 / 160.  (The backward likewise: 1 x 65536 5230, 501 / 1947; 16 x 4096 432, 5: 476.)
int segments(int U, int NC) {
  int n = U > 0 ? 152 / U : 1;
  n = n < NC / 20 ? n : NC / 20;
  n = n < 24 ? n : 24;
  return n < 5 ? 1 : n;
}
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// [records | chunk bounds | states before segments, their own states, matrices | matrix flags], and for the backward
// [bounds of the adjoint | adjoints after segments, their own | flags]
size_t rule_tc_workspace(int U, int T, bool backward) {
  const int NC = (T + C - 1) / C, n = segments(U, NC);
  const size_t rec = up256((size_t)U * NC * REC), mats = (size_t)U * n * D * D * 4, flags = up256((size_t)U * n * 4);
  if (n == 1) return rec;
  return rec + up256((size_t)U * NC * 8) + 3 * mats + flags + (backward ? up256((size_t)U * NC * 4) + 2 * mats + flags : 0);
}
RuleSegments rule_tc_segments(int U, int T, bool backward, void *workspace) {
  const int NC = (T + C - 1) / C;
  RuleSegments sg;
  sg.n = segments(U, NC);
  if (sg.n == 1) return sg;
  const size_t mats = (size_t)U * sg.n * D * D, flags = up256((size_t)U * sg.n * 4);
  sg.per = (NC + sg.n - 1) / sg.n;
  sg.n = (NC + sg.per - 1) / sg.per;  // (no empty one; the strides of the arrays are this count's)
  uint8_t *w = (uint8_t *)workspace + up256((size_t)U * NC * REC);
  sg.bounds = (float2 *)w;
  sg.S = (float *)(w + up256((size_t)U * NC * 8));
  sg.loc = sg.S + mats;
  sg.Tr = sg.loc + mats;
  sg.whole = (int *)(sg.Tr + mats);
  if (backward) {
    w = (uint8_t *)sg.whole + flags;
    sg.adds = (float *)w;
    sg.A = (float *)(w + up256((size_t)U * NC * 4));
    sg.adj = sg.A + mats;
    sg.whole_adj = (int *)(sg.adj + mats);
  }
  return sg;
}

int launch_rule_prep(const RuleArgs &a, void *records, const RuleSegments &sg, bool with_beta, cudaStream_t st) {
  auto kfn = with_beta ? mesa_rule_prep_kernel<true> : mesa_rule_prep_kernel<false>;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PR_SMEM) != cudaSuccess) return -1;
  timing_mark_begin(K_RULE_PREP, st);
  kfn<<<dim3((a.T + C - 1) / C, a.units()), 128, PR_SMEM, st>>>(a, (uint8_t *)records, sg.bounds, sg.adds);
  timing_mark_end(K_RULE_PREP, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

namespace {
// What every segment but the first starts from.
template <bool WITH_BETA>
int launch_segments(const RuleArgs &a, const uint8_t *records, const RuleSegments &sg, const CUtensorMap &mapV,
                    cudaStream_t st) {
  if (sg.n == 1) return 0;
  for (int z = 1; z <= 2; z++)
    if (launch_chain<WITH_BETA ? kSegment : kSegmentT>(a, records, RuleOperands{}, sg, dim3(a.units(), sg.n - 1, z), mapV, mapV,
                                                       st) != 0)
      return -1;
  timing_mark_begin(K_RULE_JOIN, st);
  mesa_rule_join_kernel<<<dim3(8, a.units()), 256, 0, st>>>(sg, a.S0);
  timing_mark_end(K_RULE_JOIN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}
}  // namespace

int launch_rule_forward_tc(const RuleArgs &a, void *workspace, cudaStream_t st) {
  const RuleSegments sg = rule_tc_segments(a.units(), a.T, false, workspace);
  const uint8_t *records = (const uint8_t *)workspace;
  CUtensorMap mapV{}, mapO{};
  if (!tmap_units128_bf16(&mapV, a.v, a.units(), a.T) || !tmap_units128_bf16(&mapO, a.out, a.units(), a.T)) return -1;
  if (launch_rule_prep(a, workspace, sg, true, st) != 0 || launch_segments<true>(a, records, sg, mapV, st) != 0) return -1;
  return launch_chain<kFwd>(a, records, RuleOperands{}, sg, dim3(a.units(), sg.n), mapV, mapO, st);
}

int launch_rule_states_tc(const RuleArgs &a, const void *records, const RuleSegments &sg, const RuleOperands &so,
                          cudaStream_t st) {
  CUtensorMap mapV{};
  if (!tmap_units128_bf16(&mapV, a.v, a.units(), a.T)) return -1;
  if (launch_segments<false>(a, (const uint8_t *)records, sg, mapV, st) != 0) return -1;
  return launch_chain<kKeep>(a, (const uint8_t *)records, so, sg, dim3(a.units(), sg.n), mapV, mapV, st);
}

}  // namespace mesa
