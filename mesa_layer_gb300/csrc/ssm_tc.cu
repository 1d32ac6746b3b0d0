// ssm_tc.cu -- the selective state space scan's forward on the tensor cores (bf16, dk = 128 and dv 64 or 128, or both 64; the
// operand formats are in ssm_tc.cuh).
//
// In a chunk of 128 tokens, S the state before it, f_i the decay from before the chunk to token i, E_ij from token j to i:
//     O = f (Q S^T) + M V + skip V,   M = (Q K^T) o E D,     S' = f_end S + (w V)^T K, w_j = E_{end,j} D_j.
// The gates come first, a record for each chunk (2.6 KB beside its 128).  Then one CTA per SM walks a unit's chunks (or
// those of a segment of it) with the state in tensor memory; q, k and v are read and o is written once.  Warps: four turn
// Q K^T into M, four write the outputs, eight turn the state into the next operand and weigh K's rows, one issues the
// products, one the copies.  Two chains run side by side, Q K^T -> M -> M V and state -> Q S^T -> state.
// In M V what is not finite in a value meets the zeros of the tokens before it.  A walk whose outputs are not all finite is
// done over, this time with a look at the values of each chunk before M V (ssm_tc.cuh; in every walk that took 1 to 5 % of its time).
#include <type_traits>

#include "launch.h"
#include "ssm_tc.cuh"

namespace mesa {

using namespace ssm;

namespace {

// grid (half of NC, U), a thread a token of two chunks (one's instructions fill the other's waits): the chunks' records.
// (In the chain's own warps the scan of sums, the exponentials and the logarithm were on its way: 225 us for
// 8 x 16 x 4096, against 200 with this before it.)
__global__ void __launch_bounds__(L) mesa_ssm_gates_kernel(SsmArgs a, float *records, int NC) {
  __shared__ float thi[2][4], tlo[2][4];
  __shared__ int ts[2][4];
  const int u = blockIdx.y, h = u % a.H, t = threadIdx.x, w = t >> 5, lane = t & 31;
  may_follow();
  if (t == 0 && u == 0 && blockIdx.x == 0) *a.status = 0;  // (the call's first kernel; those after it report)
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.0f, A = a.A[h];
  float step[2];
  Two l[2];
  int s[2];
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int at = (2 * blockIdx.x + k) * L + t;
    float raw = -INFINITY;  // (past the end: nothing is forgotten, nothing written)
    bool start = false;
    if (at < a.T) {
      raw = a.dt[(size_t)u * a.T + at] + bias;
      start = a.starts && a.starts[(size_t)(u / a.H) * a.T + at];
    }
    step[k] = softplus(raw);
    l[k] = start ? Two{0.0f, 0.0f} : log2_decay(step[k], A);
    s[k] = start ? t : -1;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const Two p = {__shfl_up_sync(0xffffffffu, l[k].hi, o), __shfl_up_sync(0xffffffffu, l[k].lo, o)};
      const int ps = __shfl_up_sync(0xffffffffu, s[k], o);
      if (lane >= o) {
        l[k] = two_add(p, l[k]);
        s[k] = max(s[k], ps);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; k++)
    if (lane == 31) thi[k][w] = l[k].hi, tlo[k][w] = l[k].lo, ts[k][w] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; k++) {
    const int c = 2 * blockIdx.x + k;
    if (c >= NC) break;
    float *r = records + ((size_t)u * NC + c) * REC;
    const Two end = {__shfl_sync(0xffffffffu, l[k].hi, 31), __shfl_sync(0xffffffffu, l[k].lo, 31)};
    const int send = __shfl_sync(0xffffffffu, s[k], 31);
    r[R_OUT + t] = t >= send ? rule::ex2(two_sub(end, l[k])) : 0.0f;
    r[R_IN + t] = s[k] < 0 ? rule::ex2(l[k].hi + l[k].lo) : 0.0f;
    r[R_LOG + t] = l[k].hi;
    reinterpret_cast<__nv_bfloat16 *>(r + R_LO)[t] = __float2bfloat16_rn(l[k].lo);
    r[R_STEP + t] = step[k];
    int before = -1;
    for (int i = 0; i < w; i++) before = max(before, ts[k][i]);
    reinterpret_cast<int8_t *>(r + R_START)[t] = (int8_t)max(s[k], before);
    if (w == k) {  // decays over whole warps' tokens, from..to
      const int from = lane < 16 ? lane % 4 + 1 : lane < 20 ? 0 : lane < 24 ? lane - 20 + 1 : 0,
                to = lane < 16 ? lane / 4 : lane < 20 ? lane - 16 : 4;
      Two d = {0.0f, 0.0f};
      bool cut = false;
      for (int i = from; i < to; i++) {
        d = two_add(d, Two{thi[k][i], tlo[k][i]});
        cut |= ts[k][i] >= 0;
      }
      r[R_BETWEEN + lane] = cut ? 0.0f : rule::ex2(d.hi + d.lo);
    }
  }
}

constexpr uint32_t T_G = 0, T_Y1 = 128, T_Y2 = 256, T_S = 384;  // tensor memory columns; M replaces Q K^T

// shared memory: two q tiles | two k tiles | two v tiles | the state as an operand, then the rests of K's rows | misc
template <int P>
struct Fwd {
  static constexpr uint32_t K = 2 * QK_TILE, V = 4 * QK_TILE, S = V + 2 * V_TILE<P>, MISC = S + QK_TILE;
};
struct FwdMisc {
  float cw[2][L], log[L], lo[L], step[L];  // step and decay from a token to its warp's end; for the diagonal blocks
  uint8_t marks[2][L];  // (a walk done over) by channel, the first row of the chunk's values that is not finite, kNoRow: none
  int again;            // an output was not finite: another walk
  uint64_t full[2], y_staged[2], st_done[2], g_full, m_full, y_full, y_free, s_full, w_full, cs_done, drain;
  uint32_t tmem;
  int gave_up;
};
template <int P>
constexpr uint32_t kFwdSmem = Fwd<P>::MISC + sizeof(FwdMisc);
static_assert(kFwdSmem<128> <= 232448, "shared memory per block");

// grid (U, segments), 576 threads.
template <int N, int P>
__global__ void __launch_bounds__(576, 1)
    mesa_ssm_forward_tc_kernel(SsmArgs a, SsmSegments sg, const float *records, const __grid_constant__ CUtensorMap mapQ,
                               const __grid_constant__ CUtensorMap mapK, const __grid_constant__ CUtensorMap mapV,
                               const __grid_constant__ CUtensorMap mapO) {
  extern __shared__ __align__(1024) uint8_t sm[];
  if (tc::smem_u32(sm) & 1023) {  // (swizzled tiles need it; the declaration asks for it)
    ahead_done();
    if (threadIdx.x == 0) atomicOr(a.status, tc::kErrMmaTimeout);
    return;
  }
  FwdMisc *m = reinterpret_cast<FwdMisc *>(sm + Fwd<P>::MISC);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;  // (warp: uniform)
  const int u = blockIdx.x, h = u % a.H, seg = blockIdx.y, NCT = (a.T + L - 1) / L;
  const int c0 = seg * sg.per, NC = sg.n > 1 ? min(NCT - c0, sg.per) : NCT;  // this CTA's chunks, from c0 on
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  volatile int *gave_up = &m->gave_up;
  const unsigned limit = a.wait_limit;
  if (N < DK) clear_halves(sm, 4);
  if (warp == 16) tc::tmem_alloc(tc::smem_u32(&m->tmem), 512);
  if (tid == 544) {
    for (uint64_t *b : {&m->full[0], &m->full[1], &m->st_done[0], &m->st_done[1], &m->g_full, &m->y_full, &m->cs_done, &m->drain})
      tc::mbar_init(bar(*b), 1);
    for (uint64_t *b : {&m->m_full, &m->y_free, &m->y_staged[0], &m->y_staged[1]}) tc::mbar_init(bar(*b), 4);
    for (uint64_t *b : {&m->s_full, &m->w_full}) tc::mbar_init(bar(*b), 8);
    m->gave_up = m->again = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = __shfl_sync(0xffffffffu, m->tmem, 0);
  auto warp_arrive = [&](uint64_t &b) {  // one arrival per warp, after what its lanes did
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  // a warp's wait; once a lane has given up, the warp has
  bool ok = true;
  auto need = [&](uint64_t &b, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && wait(bar(b), parity, limit, gave_up));
    tc::fence_after_sync();
    return ok;
  };
  int sent = 0;  // tiles asked for (warp 17)
  const int t = tid & 127, w = warp & 3;  // token, or lane of the state
  const uint32_t tl = tbase + ((uint32_t)(32 * w) << 16);

  if (warp != 17) ahead_done();  // (the records, the segments' states; the copies are of the call's inputs)
  // Step n of the barriers is chunk n - n0: a walk done over goes on with their phases.  (Code of its own: with the same code
  // for both the first walk is 1 to 5 % slower.)
  auto walk = [&](auto over) {
    constexpr bool OVER = decltype(over)::value;
    const int n0 = OVER ? NC : 0;
    if (warp < 4) {
      // ---- M ----
      const float *r = record(records, u, NCT, c0);
      float out = r[R_OUT + t], in = r[R_IN + t], log = r[R_LOG + t], lo = lo_of(r, t), step = r[R_STEP + t];
      int start = start_of(r, t);
      for (int c = 0; c < NC; c++) {
        const int n = n0 + c;
        const uint32_t ph = n & 1;
        const int s = start;
        const float mine = log, mine_lo = lo, from = in;
        const float *between = r + R_BETWEEN + 4 * w;
        m->cw[ph][t] = out * step;
        m->log[t] = log;
        m->lo[t] = lo;
        m->step[t] = step;
        if (c + 1 < NC) {
          r += REC;
          out = r[R_OUT + t], in = r[R_IN + t], log = r[R_LOG + t], lo = lo_of(r, t), step = r[R_STEP + t], start = start_of(r, t);
        }
        if (group_or(1, 128, !ok)) {  // (also: the others' columns)
          ok = false;
          break;
        }
        need(m->g_full, ph);
        if (OVER && t < P) {  // channel t of the values (M V waits for this)
          // (The marks of two chunks before have been used: these scores follow the last chunk's products, and those the outputs.)
          need(m->full[ph], (n >> 1) & 1);
          uint8_t *V = sm + Fwd<P>::V + ph * V_TILE<P>;
          int first = kNoRow;
          for (int i = L - 1; i >= 0; i--) {
            uint16_t *x = word_at(V, i, t);
            if (odd_word(*x)) *x = 0, first = i;
          }
          m->marks[ph][t] = (uint8_t)first;
          tc::fence_smem_to_async();
        }
#pragma unroll 1
        for (int b = 0; b < w; b++) {  // tokens of an earlier warp: through the end of theirs
          float x[32], o[16];
          tc::tmem_ld32(tl + T_G + 32 * b, x);
          const float f = between[b] * from;
          const u64 f2 = pack2(f, f);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(&m->cw[ph][32 * b + 4 * i]);
            o[2 * i] = __uint_as_float(bf2(mul2(pack2(x[4 * i], x[4 * i + 1]), mul2(f2, y.x))));
            o[2 * i + 1] = __uint_as_float(bf2(mul2(pack2(x[4 * i + 2], x[4 * i + 3]), mul2(f2, y.y))));
          }
          tc::tmem_st16(tl + T_G + 16 * b, o);
        }
        {
          float x[32], o[16];
          tc::tmem_ld32(tl + T_G + 32 * w, x);
          const int first = max(s - 32 * w, 0);
          const uint32_t on = (0xffffffffu >> (31 - lane)) & (0xffffffffu << first);  // the columns that count
          const u64 mine2 = pack2(mine, mine), lo2 = pack2(mine_lo, mine_lo);
          tc::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; i++) {
            const ulonglong2 l = *reinterpret_cast<const ulonglong2 *>(&m->log[32 * w + 4 * i]);
            const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(&m->lo[32 * w + 4 * i]);
            const ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(&m->step[32 * w + 4 * i]);
            auto two = [&](int j, u64 lj, u64 kj, u64 sj) {  // columns j and j + 1
              float d0, d1;
              unpack2(add2(sub2(mine2, lj), sub2(lo2, kj)), d0, d1);
              unpack2(mul2(pack2(rule::ex2(d0), rule::ex2(d1)), sj), d0, d1);
              return __uint_as_float(bf2(on >> j & 1 ? x[j] * d0 : 0.0f, on >> (j + 1) & 1 ? x[j + 1] * d1 : 0.0f));
            };
            o[2 * i] = two(4 * i, l.x, k.x, y.x);
            o[2 * i + 1] = two(4 * i + 2, l.y, k.y, y.y);
          }
          tc::tmem_st16(tl + T_G + 16 * w, o);
#pragma unroll
          for (int i = 0; i < 16; i++) o[i] = 0.0f;
#pragma unroll 1
          for (int b = w + 1; b < 4; b++) tc::tmem_st16(tl + T_G + 16 * b, o);
        }
        tc::tmem_st_wait();
        tc::fence_before_sync();
        warp_arrive(m->m_full);
      }
    } else if (warp < 8) {
      // ---- outputs: from tensor memory to the place of Q, and out from there ----
      const float skip = a.skip ? a.skip[h] : 0.0f;
      const u64 skip2 = pack2(skip, skip);
      const float *r = record(records, u, NCT, c0);
      float f = r[R_IN + t] * r[R_FIRST + w];
      uint32_t bad = 0;
      for (int c = 0; c < NC; c++) {
        const int n = n0 + c;
        const uint32_t ph = n & 1;
        uint8_t *X = sm + Fwd<P>::V + ph * V_TILE<P>, *Y = sm + ph * QK_TILE;
        const u64 f2 = pack2(f, f);
        const bool in = (c0 + c) * L + t < a.T;
        if (c + 1 < NC) {
          r += REC;
          f = r[R_IN + t] * r[R_FIRST + w];
        }
        if (!need(m->full[ph], (n >> 1) & 1) || !need(m->y_full, ph)) break;
#pragma unroll 1
        for (int hh = 0; hh < P / 16; hh++) {
          float p[16], q[16];
          tc::tmem_ld16(tl + T_Y1 + 16 * hh, p);
          tc::tmem_ld16(tl + T_Y2 + 16 * hh, q);
          const uint32_t at[2] = {tile_off(t, 2 * hh, L), tile_off(t, 2 * hh + 1, L)};
          const uint4 x[2] = {*reinterpret_cast<const uint4 *>(X + at[0]), *reinterpret_cast<const uint4 *>(X + at[1])};
          tc::tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 2; k++) {
            const uint32_t xs[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
              const int e = 8 * k + 2 * i;
              u64 y = fma2(f2, pack2(p[e], p[e + 1]), pack2(q[e], q[e + 1]));
              if (a.skip) y = fma2(skip2, of_bf2(xs[i]), y);
              o[i] = bf2(y);
            }
            const uint4 y = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(Y + at[k]) = y;
            if (in) bad = rule::absmax_words(bad, y);
          }
        }
        if constexpr (OVER) {
          for (int p = 0; p < P; p++)
            if (m->marks[ph][p] <= t) {
              *word_at(Y, t, p) = 0x7fff;  // NaN
              if (in) bad = 0x7fff;
            }
        }
        tc::fence_before_sync();
        warp_arrive(m->y_free);
        tc::fence_smem_to_async();
        warp_arrive(m->y_staged[ph]);
      }
      if (ok && max(bad & 0xffffu, bad >> 16) >= 0x7f80u) {
        if constexpr (OVER)
          atomicOr(a.status, tc::kErrNonFinite);
        else
          m->again = 1;
      }
    } else if (warp < 16) {
      // ---- the state, then K's rows weighed: two warps for each 32 lanes (rows), half of the columns each ----
      const int hf = warp < 12 ? 0 : 1, h0 = hf * P / 64, h1 = h0 + P / 64;
      const float *S0 = sg.n > 1 ? sg.S + ((size_t)u * sg.n + seg) * P * N : a.S0 ? a.S0 + (size_t)u * P * N : nullptr;
      const float *r = record(records, u, NCT, c0);
      float next = r[R_OUT + t] * r[R_STEP + t] * r[R_LAST + w], left = r[R_ALL];
      for (int c = 0; c < NC; c++) {
        const int n = n0 + c;
        const uint32_t ph = n & 1;
        const float mine = next, all = left;
        if (c + 1 < NC) {
          r += REC;
          next = r[R_OUT + t] * r[R_STEP + t] * r[R_LAST + w];
          left = r[R_ALL];
        }
        if (n > 0 && !need(m->st_done[ph ^ 1], ((n - 1) >> 1) & 1)) break;
        state_step<N>(tl + T_S, sm + Fwd<P>::S, t, all, c == 0, S0, h0, h1);
        tc::fence_smem_to_async();
        tc::fence_before_sync();
        warp_arrive(m->s_full);
        // (Q K^T has read K, Q S^T the state)
        if (!need(m->full[ph], (n >> 1) & 1) || !need(m->cs_done, ph)) break;
        weigh_row(sm + Fwd<P>::K + ph * QK_TILE, sm + Fwd<P>::S, t, mine, 8 * hf, 8 * hf + 8);
        tc::fence_smem_to_async();
        warp_arrive(m->w_full);
      }
      if (ok) need(m->st_done[(n0 + NC - 1) & 1], ((n0 + NC - 1) >> 1) & 1);
    } else if (warp == 16) {
      // ---- products ----
      const uint32_t idG = idesc_bf16(128, 128, false, false), idY = idesc_bf16(128, P, false, true),
                     idS = idesc_bf16(128, P, true, true);
      const uint32_t sS = tc::smem_u32(sm + Fwd<P>::S);
      const uint64_t sd = tc::mnmajor_desc(sS, L, 0);  // (the state, or the rests: the same form)
      auto scores = [&](int n) -> bool {  // Q K^T of step n
        const uint32_t ph = n & 1;
        if (!need(m->full[ph], (n >> 1) & 1)) return false;
        if (elect_one()) {
          const uint64_t q = tc::kmajor_desc(tc::smem_u32(sm + ph * QK_TILE), L, 0),
                         k = tc::kmajor_desc(tc::smem_u32(sm + Fwd<P>::K + ph * QK_TILE), L, 0);
#pragma unroll
          for (int s = 0; s < N / 16; s++) tc::mma_f16(tbase + T_G, q + step128(s), k + step128(s), idG, s > 0);
          tc::mma_commit(bar(m->g_full));
        }
        return true;
      };
      scores(n0);
      for (int n = n0; ok && n < n0 + NC; n++) {
        const uint32_t ph = n & 1, q = tc::smem_u32(sm + ph * QK_TILE), k = tc::smem_u32(sm + Fwd<P>::K + ph * QK_TILE),
                       v = tc::smem_u32(sm + Fwd<P>::V + ph * V_TILE<P>);
        const uint64_t vd = tc::mnmajor_desc(v, L, 0), kd = tc::mnmajor_desc(k, L, 0);
        if (!need(m->s_full, ph) || (n > 0 && !need(m->y_free, ph ^ 1))) break;
        if (elect_one()) {
          const uint64_t qd = tc::kmajor_desc(q, L, 0);
#pragma unroll
          for (int s = 0; s < N / 16; s++) tc::mma_f16(tbase + T_Y1, qd + step128(s), sd + step_mn(s), idY, s > 0);
          tc::mma_commit(bar(m->cs_done));
        }
        if (!need(m->m_full, ph)) break;
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < 8; s++) tc::mma_f16_ts(tbase + T_Y2, tbase + T_G + 8 * s, vd + step_mn(s), idY, s > 0);
          tc::mma_commit(bar(m->y_full));
        }
        if constexpr (OVER) {  // what was taken out of the values belongs in the state: a NaN for each channel that had any
          if (!need(m->y_full, ph)) break;
          for (int p = lane; p < P; p += 32)
            if (m->marks[ph][p] != kNoRow) *word_at(sm + Fwd<P>::V + ph * V_TILE<P>, m->marks[ph][p], p) = 0x7fff;
          tc::fence_smem_to_async();
          __syncwarp();
        }
        if (!need(m->w_full, ph)) break;
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_S, kd + step_mn(s), vd + step_mn(s), idS, true);
#pragma unroll
          for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_S, sd + step_mn(s), vd + step_mn(s), idS, true);
          tc::mma_commit(bar(m->st_done[ph]));
        }
        if (n + 1 < n0 + NC && need(m->y_full, ph)) scores(n + 1);  // (M has been read)
      }
    } else if (lane == 0) {
      // ---- copies ----
      const int uk = a.qk_unit(u);
      auto at = [&](uint32_t where, int c) { return tc::smem_u32(sm + where) + ((n0 + c) & 1) * (where == Fwd<P>::V ? V_TILE<P> : QK_TILE); };
      auto fetch_kv = [&](int c) {
        const uint32_t b = bar(m->full[(n0 + c) & 1]);
        tc::mbar_arrive_expect_tx(b, 2 * L * N * 2 + V_TILE<P>);
        load_tile<N>(at(Fwd<P>::K, c), &mapK, (c0 + c) * L, uk, b);
        load_tile<P>(at(Fwd<P>::V, c), &mapV, (c0 + c) * L, u, b);
      };
      auto fetch_q = [&](int c) { load_tile<N>(at(0, c), &mapQ, (c0 + c) * L, uk, bar(m->full[(n0 + c) & 1])); };
      for (int c = 0; c < min(NC, 2); c++, sent++) {
        fetch_kv(c);
        fetch_q(c);
      }
      ahead_done();
      for (int c = 0; c < NC; c++) {
        const int n = n0 + c;
        const uint32_t ph = n & 1, par = (n >> 1) & 1;
        if (!(ok = wait(bar(m->y_staged[ph]), par, limit, gave_up))) break;
#pragma unroll
        for (int i = 0; i < P / 64; i++) tensor_s2g_3d(&mapO, at(0, c) + i * HALF, 64 * i, (c0 + c) * L, u);
        tc::bulk_commit();
        if (!(ok = wait(bar(m->st_done[ph]), par, limit, gave_up))) break;
        if (c + 2 < NC) {
          fetch_kv(c + 2);
          tc::bulk_wait_read();
          fetch_q(c + 2);
          sent++;
        }
      }
      tc::bulk_wait_all();
    }
    if (!ok) *gave_up = 1;
    __syncthreads();
  };
  walk(std::false_type());
  if (!*gave_up && m->again) walk(std::true_type());
  if (a.S_final && seg == sg.n - 1 && warp >= 8 && warp < 16 && !*gave_up) {
    const int hf = warp < 12 ? 0 : 1;
    state_out<N>(tl + T_S, a.S_final + (size_t)u * P * N, t, hf * P / 64, (hf + 1) * P / 64);
  }
  // a wait gave up: products and copies still in flight finish before the memory is released
  if (*gave_up) {
    if (warp == 16 && elect_one()) tc::mma_commit(bar(m->drain));
    if (tid == 0) {
      unsigned bits = tc::kErrMmaTimeout;
      if (!tc::mbar_wait(bar(m->drain), 0, tc::kWaitLimit)) bits |= tc::kErrDrainTimeout;
      atomicOr(a.status, bits);
    }
    if (tid == 544) {
      bool landed = true;
      for (int c = max(0, sent - 2); c < sent; c++)
        landed &= tc::mbar_wait(bar(m->full[c & 1]), (c >> 1) & 1, tc::kWaitLimit);
      if (!landed) atomicOr(a.status, tc::kErrDrainTimeout);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 16) tc::tmem_free(tbase, 512);
}

// ---- the states alone ------------------------------------------------------------------------------------
// A segment's walk without outputs: from the state before it the states before its chunks as operands (kKeep: 16-bit tiles
// for the backward), or what it leaves of a zero state (kSegment); the adjoints after the chunks the same way, backwards,
// from rows of q and dout (kAdjoint, kAdjointSegment).  What a segment leaves is one sum: its chunks are taken from the end
// on and their rows weighed by the decay that is still to come, so that the state stays in the accumulator (1 x 16 x 65536
// forward 298 -> 294 us; rescaled after each chunk, the state went to registers and back).
enum ChainMode { kSegment, kKeep, kAdjointSegment, kAdjoint };

// shared memory: two row tiles | their rests | two v tiles | the state as an operand (kept) | misc
template <int P>
struct Chain {
  static constexpr uint32_t R = 2 * QK_TILE, V = 4 * QK_TILE, S = V + 2 * V_TILE<P>, MISC = S + V_TILE<P>;
};
struct ChainMisc {
  uint64_t full[2], w_full[2], st_done[2], s_full, kept, sum, drain;  // (sum: the last chunk's products)
  uint32_t tmem;
  int gave_up;
};
template <int P>
constexpr uint32_t kChainSmem = Chain<P>::MISC + sizeof(ChainMisc);

// grid (U, segments (from 1 on for adjoint segments, all but the last for segments)), 448 threads: warps 0-7 weigh
// rows, 8-11 the state, 12 products, 13 copies.  kept: [U, NC][V_TILE] operand tiles.
template <int N, int P, int MODE>
__global__ void __launch_bounds__(448, 1)
    mesa_ssm_chain_tc_kernel(SsmArgs a, SsmSegments sg, const float *records, uint8_t *kept, const __grid_constant__ CUtensorMap mapK,
                             const __grid_constant__ CUtensorMap mapV) {
  constexpr bool ADJ = MODE == kAdjoint || MODE == kAdjointSegment, KEEP = MODE == kKeep || MODE == kAdjoint;
  extern __shared__ __align__(1024) uint8_t sm[];
  if (tc::smem_u32(sm) & 1023) {
    ahead_done();
    if (threadIdx.x == 0) atomicOr(a.status, tc::kErrMmaTimeout);
    return;
  }
  ChainMisc *m = reinterpret_cast<ChainMisc *>(sm + Chain<P>::MISC);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int u = blockIdx.x, seg = blockIdx.y + (MODE == kAdjointSegment ? 1 : 0), NCT = (a.T + L - 1) / L;
  const int c0 = seg * sg.per, NC = sg.n > 1 ? min(NCT - c0, sg.per) : NCT;
  auto chunk = [&](int c) { return ADJ == KEEP ? c0 + NC - 1 - c : c0 + c; };  // of step c
  auto bar = [](uint64_t &b) { return tc::smem_u32(&b); };
  volatile int *gave_up = &m->gave_up;
  const unsigned limit = a.wait_limit;
  if (N < DK) clear_halves(sm, 4);  // (the rests', too)
  if (warp == 12) tc::tmem_alloc(tc::smem_u32(&m->tmem), 128);
  if (tid == 416) {
    for (uint64_t *b : {&m->full[0], &m->full[1], &m->st_done[0], &m->st_done[1], &m->kept, &m->sum, &m->drain}) tc::mbar_init(bar(*b), 1);
    for (uint64_t *b : {&m->w_full[0], &m->w_full[1]}) tc::mbar_init(bar(*b), 8);
    tc::mbar_init(bar(m->s_full), 4);
    m->gave_up = 0;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = __shfl_sync(0xffffffffu, m->tmem, 0);
  auto warp_arrive = [&](uint64_t &b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(b));
  };
  bool ok = true;
  int sent = 0;

  auto need = [&](uint64_t &b, uint32_t parity) {
    ok = __all_sync(0xffffffffu, ok && wait(bar(b), parity, limit, gave_up));
    tc::fence_after_sync();
    return ok;
  };
  const int t = tid & 127, w = warp & 3;  // token, or lane of the state
  const uint32_t tl = tbase + ((uint32_t)(32 * w) << 16);

  may_follow();
  if (warp != 13) ahead_done();  // (the records, the segments' states; the copies are of the call's inputs)
  if (warp < 8) {
    const int hf = warp >> 2;  // two warps for each 32 rows, half of the columns each
    auto weight = [&](int c) {
      const float *r = record(records, u, NCT, chunk(c));
      return ADJ ? r[R_IN + t] * r[R_FIRST + w] : r[R_OUT + t] * r[R_STEP + t] * r[R_LAST + w];
    };
    float next = weight(0), coming = 1.0f, all = KEEP ? 1.0f : record(records, u, NCT, chunk(0))[R_ALL];
    for (int c = 0; c < NC; c++) {
      const uint32_t ph = c & 1;
      const float mine = next * coming;
      if constexpr (!KEEP) coming *= all;
      if (c + 1 < NC) {
        next = weight(c + 1);
        if constexpr (!KEEP) all = record(records, u, NCT, chunk(c + 1))[R_ALL];
      }
      if (c > 1 && !need(m->st_done[ph], ((c - 2) >> 1) & 1)) break;  // (its tiles are free)
      if (!need(m->full[ph], (c >> 1) & 1)) break;
      weigh_row(sm + ph * QK_TILE, sm + Chain<P>::R + ph * QK_TILE, t, mine, 8 * hf, 8 * hf + 8);
      tc::fence_smem_to_async();
      warp_arrive(m->w_full[ph]);
    }
    if (!KEEP && tid == 0) sg.decay[(size_t)u * sg.n + seg] = coming;  // of a state, after the segment
  } else if (warp < 12) {
    if constexpr (KEEP) {
      const float *from = MODE == kKeep ? (sg.n > 1 ? sg.S + ((size_t)u * sg.n + seg) * P * N : a.S0 ? a.S0 + (size_t)u * P * N : nullptr)
                          : sg.n > 1    ? sg.R + ((size_t)u * sg.n + seg) * P * N
                          : a.dS_final  ? a.dS_final + (size_t)u * P * N
                                        : nullptr;
      float next = record(records, u, NCT, chunk(0))[R_ALL];
      for (int c = 0; c < NC; c++) {
        const uint32_t ph = c & 1;
        const float all = next;
        if (c + 1 < NC) next = record(records, u, NCT, chunk(c + 1))[R_ALL];
        if (c > 0 && !need(m->st_done[ph ^ 1], ((c - 1) >> 1) & 1)) break;
        if (c > 0 && !need(m->kept, (c - 1) & 1)) break;  // (the last tile has left)
        state_step<N>(tl + T_G, sm + Chain<P>::S, t, all, c == 0, from, 0, P / 32);
        tc::fence_smem_to_async();
        tc::fence_before_sync();
        warp_arrive(m->s_full);
      }
    }
    float *to = nullptr;
    if constexpr (MODE == kSegment) to = sg.S + ((size_t)u * sg.n + seg) * P * N;
    if constexpr (MODE == kAdjointSegment) to = sg.R + ((size_t)u * sg.n + seg) * P * N;
    if constexpr (MODE == kAdjoint) to = a.dS0 && seg == 0 ? a.dS0 + (size_t)u * P * N : nullptr;
    if (ok && need(m->sum, 0) && to) state_out<N>(tl + T_G, to, t, 0, P / 32);
  } else if (warp == 12) {
    const uint32_t idS = idesc_bf16(128, P, true, true);
    for (int c = 0; c < NC; c++) {
      const uint32_t ph = c & 1;
      if constexpr (KEEP) {
        if (!need(m->s_full, ph)) break;
      }
      if (!need(m->w_full[ph], (c >> 1) & 1)) break;
      if (elect_one()) {
        const uint64_t vd = tc::mnmajor_desc(tc::smem_u32(sm + Chain<P>::V + ph * V_TILE<P>), L, 0),
                       kd = tc::mnmajor_desc(tc::smem_u32(sm + ph * QK_TILE), L, 0),
                       rd = tc::mnmajor_desc(tc::smem_u32(sm + Chain<P>::R + ph * QK_TILE), L, 0);
#pragma unroll
        for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_G, kd + step_mn(s), vd + step_mn(s), idS, KEEP || s > 0 || c > 0);
#pragma unroll
        for (int s = 0; s < 8; s++) tc::mma_f16(tbase + T_G, rd + step_mn(s), vd + step_mn(s), idS, true);
        tc::mma_commit(bar(m->st_done[ph]));
        if (c + 1 == NC) tc::mma_commit(bar(m->sum));
      }
    }
  } else if (lane == 0) {
    const int uk = a.qk_unit(u);
    auto fetch = [&](int c) {
      const uint32_t ph = c & 1, b = bar(m->full[ph]);
      tc::mbar_arrive_expect_tx(b, L * N * 2 + V_TILE<P>);
      load_tile<N>(tc::smem_u32(sm + ph * QK_TILE), &mapK, chunk(c) * L, uk, b);
      load_tile<P>(tc::smem_u32(sm + Chain<P>::V + ph * V_TILE<P>), &mapV, chunk(c) * L, u, b);
      sent++;
    };
    for (int c = 0; c < min(NC, 2); c++) fetch(c);
    ahead_done();
    for (int c = 0; c < NC; c++) {
      if (KEEP) {
        if (!(ok = wait(bar(m->s_full), c & 1, limit, gave_up))) break;
        rule::bulk_s2g(kept + ((size_t)u * NCT + chunk(c)) * V_TILE<P>, tc::smem_u32(sm + Chain<P>::S), V_TILE<P>);
        tc::bulk_commit();
        tc::bulk_wait_read();
        mbar_arrive(bar(m->kept));
      }
      if (!(ok = wait(bar(m->st_done[c & 1]), (c >> 1) & 1, limit, gave_up))) break;
      if (c + 2 < NC) fetch(c + 2);
    }
    if (KEEP) tc::bulk_wait_all();
  }
  if (!ok) *gave_up = 1;
  __syncthreads();
  if (*gave_up) {
    if (warp == 12 && elect_one()) tc::mma_commit(bar(m->drain));
    if (tid == 0) {
      unsigned bits = tc::kErrMmaTimeout;
      if (!tc::mbar_wait(bar(m->drain), 0, tc::kWaitLimit)) bits |= tc::kErrDrainTimeout;
      atomicOr(a.status, bits);
    }
    if (tid == 416) {
      bool landed = true;
      for (int c = max(0, sent - 2); c < sent; c++)
        landed &= tc::mbar_wait(bar(m->full[c & 1]), (c >> 1) & 1, tc::kWaitLimit);
      if (!landed) atomicOr(a.status, tc::kErrDrainTimeout);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 12) tc::tmem_free(tbase, 128);
}

// The states before the segments from what each leaves: S_{y+1} = decay_y S_y + left_y, S_0 the call's (copied: the last
// segment may write its final state over it); the adjoints after them the same way, backwards.  Four elements a thread;
// eight segments' are asked for together (one after the other: 27 us for 16 units in nine segments).
// No decay is too small to carry what is not finite, as in one chain.
__global__ void __launch_bounds__(128) mesa_ssm_join_kernel(SsmArgs a, SsmSegments sg, bool adjoint) {
  constexpr int AHEAD = 8;
  const int n4 = a.dv * a.dk / 4, e = blockIdx.x * 128 + threadIdx.x, u = blockIdx.y, n = sg.n;
  may_follow();
  ahead_done();
  if (e >= n4) return;
  const float4 *from = reinterpret_cast<const float4 *>(adjoint ? a.dS_final : a.S0);
  float4 *x = reinterpret_cast<float4 *>(adjoint ? sg.R : sg.S) + (size_t)u * n * n4 + e;
  const float *decay = sg.decay + (size_t)u * n;
  float4 s = from ? from[(size_t)u * n4 + e] : make_float4(0, 0, 0, 0);
  for (int i0 = 0; i0 < n; i0 += AHEAD) {
    float4 d[AHEAD];
    float w[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; j++) {
      const int y = adjoint ? n - 1 - i0 - j : i0 + j;
      if (i0 + j + 1 < n) {  // (the last one's is not needed)
        d[j] = x[(size_t)y * n4];
        w[j] = decay[y];
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; j++) {
      const int y = adjoint ? n - 1 - i0 - j : i0 + j;
      if (i0 + j < n) {
        x[(size_t)y * n4] = s;
        if (i0 + j + 1 < n)
          s = make_float4(fmaf(w[j], s.x, d[j].x), fmaf(w[j], s.y, d[j].y), fmaf(w[j], s.z, d[j].z), fmaf(w[j], s.w, d[j].w));
      }
    }
  }
}

template <typename K, typename... Args>
bool launch_tc(int kind, K kernel, dim3 grid, int threads, uint32_t smem, cudaStream_t st, const Args &...args) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
  timing_mark_begin(kind, st);
  const bool ok = launch_after(kernel, grid, threads, smem, st, args...);
  timing_mark_end(kind, st);
  return ok && cudaPeekAtLastError() == cudaSuccess;
}

bool launch_join(const SsmArgs &a, const SsmSegments &sg, bool adjoint, cudaStream_t st) {
  timing_mark_begin(K_SSM_SCAN, st);
  const bool ok = launch_after(mesa_ssm_join_kernel, dim3((a.dv * a.dk / 4 + 127) / 128, a.units()), 128, 0, st, a, sg, adjoint);
  timing_mark_end(K_SSM_SCAN, st);
  return ok;
}
template <int N, int P, int MODE>
bool launch_chain(const SsmArgs &a, const SsmSegments &sg, uint8_t *kept, const CUtensorMap &k, const CUtensorMap &v, cudaStream_t st) {
  const int n = MODE == kSegment || MODE == kAdjointSegment ? sg.n - 1 : sg.n;
  return launch_tc(K_SSM_CHAIN, mesa_ssm_chain_tc_kernel<N, P, MODE>, dim3(a.units(), n), 448, kChainSmem<P>, st, a, sg, sg.records, kept, k,
                   v);
}

template <int N, int P>
int forward(const SsmArgs &a, const SsmSegments &sg, cudaStream_t st) {
  CUtensorMap q{}, k{}, v{}, o{};
  if (!tmap_units_bf16(&q, a.q, a.B * a.Hk, a.T, N) || !tmap_units_bf16(&k, a.k, a.B * a.Hk, a.T, N) ||
      !tmap_units_bf16(&v, a.v, a.units(), a.T, P) || !tmap_units_bf16(&o, a.out, a.units(), a.T, P))
    return -1;
  if (sg.n > 1) {
    if (!launch_chain<N, P, kSegment>(a, sg, nullptr, k, v, st) || !launch_join(a, sg, false, st)) return -1;
  }
  return launch_tc(K_SSM_FORWARD, mesa_ssm_forward_tc_kernel<N, P>, dim3(a.units(), sg.n), 576, kFwdSmem<P>, st, a, sg, sg.records, q, k,
                   v, o)
             ? 0
             : -1;
}

// The states before every chunk and the adjoints after it.
template <int N, int P>
int chains(const SsmArgs &a, const SsmSegments &sg, const SsmTcBwd &ws, cudaStream_t st) {
  CUtensorMap q{}, k{}, v{}, g{};
  if (!tmap_units_bf16(&q, a.q, a.B * a.Hk, a.T, N) || !tmap_units_bf16(&k, a.k, a.B * a.Hk, a.T, N) ||
      !tmap_units_bf16(&v, a.v, a.units(), a.T, P) || !tmap_units_bf16(&g, a.dout, a.units(), a.T, P))
    return -1;
  if (sg.n > 1) {
    if (!launch_chain<N, P, kSegment>(a, sg, nullptr, k, v, st) || !launch_join(a, sg, false, st)) return -1;
    if (!launch_chain<N, P, kAdjointSegment>(a, sg, nullptr, q, g, st) || !launch_join(a, sg, true, st)) return -1;
  }
  return launch_chain<N, P, kKeep>(a, sg, ws.S, k, v, st) && launch_chain<N, P, kAdjoint>(a, sg, ws.R, q, g, st) ? 0 : -1;
}

}  // namespace

// Segments: a GB300's 152 SMs hold a CTA each.  A segment's chunks are walked twice (before a forward the second time takes
// half as long), and the two more kernels cost as much as four or five chunks: shorter chains are left whole.  us of one
// chain, of segments, forward / backward, in a graph (units x chunks): 1 x 4 16, 13 / 30, 32 (launched one by one, the two
// kernels more cost the 3 us); 1 x 8 28, 14 / 43, 33; 16 x 16 52, 22 / 78, 55; 24 x 9 (dv = 64) 27, 18 / 50, 44; 48 x 9
// 32, 26 / 66, 72; 70 x 16 54, 49 / 135, 154; 70 x 32 101, 86 / 256, 275; 16 x 512 1489, 283 / 2117, 920.
SsmSegments ssm_segments(int U, int T, int dv, bool backward, void *workspace, size_t *bytes) {
  const int NC = (T + L - 1) / L;
  SsmSegments sg;
  const int most = U > 0 ? 152 / U : 1, n = most < NC ? most : NC;
  sg.per = n > 1 ? (NC + n - 1) / n : NC;
  sg.n = n > 1 && (backward ? 2 * sg.per + 5 <= NC : 3 * sg.per + 8 <= 2 * NC) ? (NC + sg.per - 1) / sg.per : 1;  // (no empty one)
  auto up256 = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t state = sg.n > 1 ? (size_t)U * sg.n * dv * DK * sizeof(float) : 0, decay = up256((size_t)U * sg.n * sizeof(float)),
               recs = up256((size_t)U * NC * REC * sizeof(float));
  if (bytes) *bytes = recs + decay + state * (backward ? 2 : 1);
  if (workspace) {
    sg.records = (float *)workspace;
    sg.decay = (float *)((char *)workspace + recs);
    sg.S = (float *)((char *)sg.decay + decay);
    sg.R = (float *)((char *)sg.S + state);
  }
  return sg;
}

int launch_ssm_gates(const SsmArgs &a, const SsmSegments &sg, cudaStream_t st) {
  timing_mark_begin(K_SSM_GATES, st);
  const int NC = (a.T + L - 1) / L;
  mesa_ssm_gates_kernel<<<dim3((NC + 1) / 2, a.units()), L, 0, st>>>(a, sg.records, NC);
  timing_mark_end(K_SSM_GATES, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int launch_ssm_forward_tc(const SsmArgs &a, void *workspace, cudaStream_t st) {
  const SsmSegments sg = ssm_segments(a.units(), a.T, a.dv, false, workspace, nullptr);
  if (launch_ssm_gates(a, sg, st) != 0) return -1;
  return a.dk == 64 ? forward<64, 64>(a, sg, st) : a.dv == 128 ? forward<128, 128>(a, sg, st) : forward<128, 64>(a, sg, st);
}
int launch_ssm_chains_tc(const SsmArgs &a, const SsmSegments &sg, const SsmTcBwd &ws, cudaStream_t st) {
  return a.dk == 64 ? chains<64, 64>(a, sg, ws, st) : a.dv == 128 ? chains<128, 128>(a, sg, ws, st) : chains<128, 64>(a, sg, ws, st);
}
size_t ssm_tc_workspace(int U, int T, int dv) {
  size_t n;
  ssm_segments(U, T, dv, false, nullptr, &n);
  return n;
}

}  // namespace mesa
