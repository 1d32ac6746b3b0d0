// gated_delta.cu -- the gated delta rule on the CUDA cores: token recurrence for whole
// sequences (forward, and the two sweeps of the backward pass), the backward's per-chunk
// gradients, and the decode step.
//
// Per (batch, head) unit, with the state S [dv, dk]:
//     e_t = v_t - gamma_t S_{t-1} k_t,  u_t = beta_t e_t,  S_t = gamma_t S_{t-1} + u_t k_t^T,
//     o_t = scale S_t q_t.
// Every row of S evolves on its own given k, q and the gates, so rows are split over lanes,
// warps and CTAs without any exchange but the sum over dk.  The adjoint A_t of S_t (from the
// tokens after t) runs the same way in reverse: with g_t = dL/do_t
//     A <- A + scale g_t q_t^T,  du_t = A k_t,  N_t = A - beta_t du_t k_t^T,  A_{t-1} = gamma_t N_t,
// and the gradients are dv_t = beta_t du_t, dbeta_t = du_t . e_t, dgamma_t = <N_t, S_{t-1}>,
// dq_t = scale S_t^T g_t, dk_t = (A + scale g q^T)^T u_t - beta_t gamma_t S_{t-1}^T du_t.
#include "common.cuh"
#include "gated_delta.h"
#include "launch.h"
#include "packed.cuh"

namespace mesa {

namespace {

__device__ __forceinline__ void cp16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ float nonfinite4(const float4 &x, float bad) {  // NaN once one of them was not finite
  return fmaf(x.x, 0.0f, fmaf(x.y, 0.0f, fmaf(x.z, 0.0f, fmaf(x.w, 0.0f, bad))));
}

enum ScanMode { kForward = 0, kStates = 1, kAdjoint = 2, kSegment = 3, kSegAdjoint = 4 };
constexpr int TB = 16;    // tokens staged at a time
constexpr int ROWS = 32;  // state rows per CTA
constexpr int lanes_per_row(int dk) { return dk == 128 ? 4 : 2; }

// One CTA: 32 rows of one unit's state through all tokens.  The recurrence is a dependent
// chain per token (sum over dk, shuffles, rank-one update).  Few lanes a row: the sum's tail (shuffles, gate,
// error) and the reads of k and q then cost fewer instructions beside the products (2 x 4 x 2048 x 64 fp32,
// both passes: four lanes 63 us, two 55; 32 columns, four passes: four 50, two 48, one 56).  k, q and v (or dout)
// of the next 16 tokens arrive by cp.async while a block of 16 is worked on; bf16 is widened once per
// block.  Bound by the chain's latency when units are few, by FMA issue when they are many (packed
// fp32 pairs halve the issue slots).
//   kForward: out, S_final.  kStates: e and the state before each 32-token chunk.
//   kAdjoint: tokens descending; du and the adjoint after each chunk, dS0.
// Few units: the tokens are cut into segments (blockIdx.z) that run side by side, each from the state
// before it, which two more modes and mesa_rule_scan_join_kernel find first.
//   kSegment: what segment z leaves of a state of zero (the first: of S0), and, in the CTAs past the
//   state's rows, of the rows of the identity without values: the matrix that takes the state before
//   the segment to its part of the state after it (and that matrix transposed, which takes the adjoint back).
//   kSegAdjoint: the adjoint before segment z + 1 from zero after it (the last: dS_final).
template <int DK, typename TIO, int MODE>
__global__ void __launch_bounds__(ROWS * lanes_per_row(DK)) mesa_rule_scan_kernel(RuleArgs a, RuleBwdWorkspace ws, RuleScanSegments sg) {
  constexpr bool ADJ = MODE == kAdjoint || MODE == kSegAdjoint, SEG = MODE == kSegment || MODE == kSegAdjoint;
  constexpr int LPR = lanes_per_row(DK), NT = ROWS * LPR, RPW = 32 / LPR;  // threads, rows of a warp
  constexpr int VPL = DK / LPR, NG = VPL / 4;                              // values and 16-byte groups per lane
  constexpr bool WIDE = sizeof(TIO) == 4;
  constexpr bool USEQ = MODE == kForward || ADJ;
  __shared__ __align__(16) TIO kraw[2][TB * DK], qraw[2][USEQ ? TB * DK : 8], xraw[2][TB * ROWS];
  __shared__ __align__(16) float kwide[WIDE ? 4 : TB * DK], qwide[WIDE || !USEQ ? 4 : TB * DK];
  __shared__ __align__(16) float os[TB * ROWS * (MODE == kForward ? LPR : 1)];
  __shared__ float gs[2][TB], bs[2][TB];
  const int u = blockIdx.y, tiles = (a.dv + ROWS - 1) / ROWS, tid = threadIdx.x;
  const bool matrix = MODE == kSegment && (int)blockIdx.x >= tiles;
  const int r0 = (blockIdx.x - (matrix ? tiles : 0)) * ROWS;
  const int r = tid / LPR, j = tid % LPR, nr = min(ROWS, (matrix ? DK : a.dv) - r0);
  const int T = a.T, seg = blockIdx.z + (MODE == kSegAdjoint ? 1 : 0);
  const int b0 = seg * sg.per, b1 = min((T + TB - 1) / TB, b0 + sg.per), nblk = b1 - b0;  // its blocks of tokens
  if (matrix && seg == 0) return;
  const size_t qk0 = (size_t)a.qk_unit(u) * T, tu = (size_t)u * T;
  const TIO *kp = (const TIO *)a.k + qk0 * DK, *qp = (const TIO *)a.q + qk0 * DK;
  const TIO *xp = (const TIO *)(ADJ ? a.dout : a.v) + tu * a.dv + r0;
  const bool rin = r < nr;

  auto fetch = [&](int blk, int buf) {
    const int t0 = blk * TB, n = min(TB, T - t0);
    constexpr int E = 16 / sizeof(TIO), KV = TB * DK / E, XV = ROWS / E;
    const TIO *ks = kp + (size_t)t0 * DK, *qs = qp + (size_t)t0 * DK, *xs = xp + (size_t)t0 * a.dv;
#pragma unroll
    for (int i0 = 0; i0 < KV; i0 += NT) {
      const int i = i0 + tid;
      if (i * E < n * DK) {
        cp16(&kraw[buf][i * E], ks + i * E);
        if (USEQ) cp16(&qraw[buf][i * E], qs + i * E);
      }
    }
#pragma unroll
    for (int i0 = 0; i0 < TB * XV; i0 += NT) {
      const int i = i0 + tid, t = i / XV, c = i % XV * E;
      if (t < n && c < nr && !matrix) cp16(&xraw[buf][t * ROWS + c], xs + (size_t)t * a.dv + c);
    }
    if (tid < n) {
      cp4(&gs[buf][tid], a.gamma + tu + t0 + tid);
      cp4(&bs[buf][tid], a.beta + tu + t0 + tid);
    }
    cp_commit();
  };

  u64 s[2 * NG];
  {
    const bool first = seg == (ADJ ? sg.n - 1 : 0), kept = !SEG && sg.n > 1;  // (first: the sweep starts here)
    const float *init = kept ? (ADJ ? sg.A : sg.S) : first ? (ADJ ? a.dS_final : a.S0) : nullptr;
    const float *src = init ? init + ((kept ? (size_t)u * sg.n + seg : (size_t)u) * a.dv + r0 + r) * DK : nullptr;
#pragma unroll
    for (int g = 0; g < NG; g++) {
      const float4 x = (src && rin) ? *reinterpret_cast<const float4 *>(src + 4 * (j + LPR * g)) : make_float4(0, 0, 0, 0);
      s[2 * g] = pack2(x.x, x.y);
      s[2 * g + 1] = pack2(x.z, x.w);
      if (matrix) {
        const int d = r0 + r - 4 * (j + LPR * g);  // the diagonal's place in this group
        s[2 * g] = pack2(d == 0 ? 1.0f : 0.0f, d == 1 ? 1.0f : 0.0f);
        s[2 * g + 1] = pack2(d == 2 ? 1.0f : 0.0f, d == 3 ? 1.0f : 0.0f);
      }
    }
  }
  auto store_state = [&](float *dst) {  // this lane's part of row r (dst: the unit's matrix)
    if (!rin) return;
#pragma unroll
    for (int g = 0; g < NG; g++)
      *reinterpret_cast<ulonglong2 *>(dst + (size_t)(r0 + r) * DK + 4 * (j + LPR * g)) =
          make_ulonglong2(s[2 * g], s[2 * g + 1]);
  };

  const int NC = (T + kRuleChunk - 1) / kRuleChunk;
  constexpr int BPC = kRuleChunk / TB;  // blocks per chunk
  fetch(ADJ ? b1 - 1 : b0, 0);
  for (int it = 0; it < nblk; it++) {
    const int blk = ADJ ? b1 - 1 - it : b0 + it, buf = it & 1;
    const int t0 = blk * TB, n = min(TB, T - t0);
    cp_wait<0>();
    __syncthreads();  // this block is there, and the last one has been used
    if (it + 1 < nblk) fetch(ADJ ? blk - 1 : blk + 1, buf ^ 1);
    const float *kf, *qf;
    if constexpr (WIDE) {
      kf = kraw[buf];
      qf = qraw[buf];
    } else {
      for (int i = tid; i < TB * DK / 4; i += NT) {
        *reinterpret_cast<float4 *>(&kwide[4 * i]) = load4(kraw[buf], 4 * i);
        if (USEQ) *reinterpret_cast<float4 *>(&qwide[4 * i]) = load4(qraw[buf], 4 * i);
      }
      kf = kwide;
      qf = qwide;
      __syncthreads();
    }
    if (MODE == kStates && blk % BPC == 0) store_state(ws.S + ((size_t)u * NC + blk / BPC) * a.dv * DK);
    if (MODE == kAdjoint && (blk % BPC == BPC - 1 || blk == b1 - 1))
      store_state(ws.dS + ((size_t)u * NC + blk / BPC) * a.dv * DK);
    // a token's key, gates and value are read a token ahead, its query at its start: nothing on the
    // chain waits for shared memory
    struct Token {
      ulonglong2 k[NG];
      float x, g, b;
    } cur, nxt;
    auto load_token = [&](int t, Token &w) {
      const ulonglong2 *kv = reinterpret_cast<const ulonglong2 *>(kf + t * DK);
#pragma unroll
      for (int i = 0; i < NG; i++) w.k[i] = kv[j + LPR * i];
      w.x = matrix ? 0.0f : ld(xraw[buf], t * ROWS + r);
      w.g = gs[buf][t];
      w.b = bs[buf][t];
    };
    auto token = [&](int t, const Token &w) {
      const ulonglong2 *qv = reinterpret_cast<const ulonglong2 *>(qf + t * DK);
      const u64 g2 = pack2(w.g, w.g);
      ulonglong2 qq[NG];
      if constexpr (USEQ) {
#pragma unroll
        for (int i = 0; i < NG; i++) qq[i] = qv[j + LPR * i];
      }
      u64 d[4] = {};  // (four sums: short chains)
      if constexpr (ADJ) {
        const u64 gx = pack2(a.scale * w.x, a.scale * w.x);
#pragma unroll
        for (int i = 0; i < NG; i++) {
          s[2 * i] = fma2(gx, qq[i].x, s[2 * i]);
          s[2 * i + 1] = fma2(gx, qq[i].y, s[2 * i + 1]);
          d[2 * (i & 1)] = fma2(s[2 * i], w.k[i].x, d[2 * (i & 1)]);
          d[2 * (i & 1) + 1] = fma2(s[2 * i + 1], w.k[i].y, d[2 * (i & 1) + 1]);
        }
        float du = sum2(add2(add2(d[0], d[1]), add2(d[2], d[3])));
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) du += __shfl_xor_sync(0xffffffffu, du, o);
        const u64 p = pack2(-w.b * du, -w.b * du);
#pragma unroll
        for (int i = 0; i < NG; i++) {
          s[2 * i] = mul2(g2, fma2(p, w.k[i].x, s[2 * i]));
          s[2 * i + 1] = mul2(g2, fma2(p, w.k[i].y, s[2 * i + 1]));
        }
        if (!SEG && j == 0) os[t * ROWS + r] = du;
      } else {
#pragma unroll
        for (int i = 0; i < NG; i++) {
          d[2 * (i & 1)] = fma2(s[2 * i], w.k[i].x, d[2 * (i & 1)]);
          d[2 * (i & 1) + 1] = fma2(s[2 * i + 1], w.k[i].y, d[2 * (i & 1) + 1]);
          s[2 * i] = mul2(g2, s[2 * i]);
          s[2 * i + 1] = mul2(g2, s[2 * i + 1]);
        }
        float sk = sum2(add2(add2(d[0], d[1]), add2(d[2], d[3])));
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) sk += __shfl_xor_sync(0xffffffffu, sk, o);
        const float e = fmaf(-w.g, sk, w.x), uu = w.b * e;
        const u64 u2 = pack2(uu, uu);
        u64 o[4] = {};
#pragma unroll
        for (int i = 0; i < NG; i++) {
          s[2 * i] = fma2(u2, w.k[i].x, s[2 * i]);
          s[2 * i + 1] = fma2(u2, w.k[i].y, s[2 * i + 1]);
          if constexpr (MODE == kForward) {
            o[2 * (i & 1)] = fma2(s[2 * i], qq[i].x, o[2 * (i & 1)]);
            o[2 * (i & 1) + 1] = fma2(s[2 * i + 1], qq[i].y, o[2 * (i & 1) + 1]);
          }
        }
        if constexpr (MODE == kForward) {
          os[(t * ROWS + r) * LPR + j] = sum2(add2(add2(o[0], o[1]), add2(o[2], o[3])));  // (added over the lanes when the block is written)
        } else {
          if (!SEG && j == 0) os[t * ROWS + r] = e;
        }
      }
    };
    auto nth = [&](int tt) { return ADJ ? max(n - 1 - tt, 0) : min(tt, n - 1); };
    load_token(nth(0), cur);
    if (n == TB) {
#pragma unroll 4
      for (int tt = 0; tt < TB; tt += 2) {
        load_token(nth(tt + 1), nxt);
        token(nth(tt), cur);
        load_token(nth(tt + 2), cur);
        token(nth(tt + 1), nxt);
      }
    } else {
      for (int tt = 0; tt < n; tt++) {
        load_token(nth(tt), cur);
        token(nth(tt), cur);
      }
    }
    if constexpr (!SEG) {  // a warp writes its own rows
      __syncwarp();
      bool bad = false;
#pragma unroll
      for (int i0 = 0; i0 < TB * RPW; i0 += 32) {
        const int i = i0 + (tid & 31), t = i / RPW, rr = (tid >> 5) * RPW + i % RPW;
        if (t < n && rr < nr) {
          const size_t at = (tu + t0 + t) * a.dv + r0 + rr;
          if constexpr (MODE == kForward) {
            float y = 0.0f;
#pragma unroll
            for (int l = 0; l < LPR; l++) y += os[(t * ROWS + rr) * LPR + l];
            y *= a.scale;
            st((TIO *)a.out, at, y);
            bad |= !isfinite(y);
          } else {
            (MODE == kStates ? ws.e : ws.du)[at] = os[t * ROWS + rr];
          }
        }
      }
      if (MODE == kForward && bad) atomicOr(a.status, tc_err_nonfinite());
      __syncwarp();
    }
  }
  if (MODE == kForward && a.S_final && seg == sg.n - 1) store_state(a.S_final + (size_t)u * a.dv * DK);
  if (MODE == kAdjoint && a.dS0 && seg == 0) store_state(a.dS0 + (size_t)u * a.dv * DK);
  if (SEG && !matrix) store_state((ADJ ? sg.adj : sg.loc) + ((size_t)u * sg.n + seg) * a.dv * DK);
  if (matrix) {
    const size_t at = ((size_t)u * sg.n + seg) * DK * DK;
    store_state(sg.Tr + at);
    if (sg.TrT && rin) {
#pragma unroll
      for (int i = 0; i < 2 * NG; i++) {
        const int c = 4 * (j + LPR * (i >> 1)) + 2 * (i & 1);
        float x, y;
        unpack2(s[i], x, y);
        sg.TrT[at + (size_t)c * DK + r0 + r] = x;
        sg.TrT[at + (size_t)(c + 1) * DK + r0 + r] = y;
      }
    }
  }
}

// The state before each segment: start[y + 1] = start[y] M[y] + local[y] (the first: local[0], and start[0] a
// copy of `given`: the final state may be written over it); downwards for the adjoint.  A chain of n short products, so what counts is a step's latency: eight rows by a CTA of
// 256 threads, a thread two rows, DK / 16 columns and a quarter of the sum (so that a matrix is read
// from shared memory four times in a step, not eight, by eight warps), the matrices and local states of the
// next steps on their way by cp.async.  (One row and the whole sum a thread: 1.0 us a step at DK = 64.)
constexpr int JROWS = 8;
template <int DK>
struct JoinBuffers {
  static constexpr int n = DK == 128 ? 3 : 4, bytes = n * (DK * DK + JROWS * DK) * (int)sizeof(float);
};
template <int DK>
__global__ void __launch_bounds__(256) mesa_rule_scan_join_kernel(RuleScanSegments sg, const float *given, int dv, bool adjoint) {
  constexpr int CPT = DK / 16, MAT = DK * DK, BUF = MAT + JROWS * DK, NB = JoinBuffers<DK>::n, KP = DK / 4;
  extern __shared__ __align__(16) float jm[];  // NB buffers: a matrix, the local rows
  __shared__ __align__(16) float rows[JROWS][DK], part[4][JROWS][DK];
  const int u = blockIdx.y, tid = threadIdx.x, row0 = blockIdx.x * JROWS;
  const int kp = tid >> 6, r = (tid >> 4 & 3) * 2, c0 = (tid & 15) * CPT;
  const float *local = adjoint ? sg.adj : sg.loc, *M = adjoint ? sg.TrT : sg.Tr;
  float *start = adjoint ? sg.A : sg.S;
  auto at = [&](int i) { return (size_t)u * sg.n + (adjoint ? sg.n - 1 - i : i); };
  auto fetch = [&](int i) {  // (a step past the last: an empty group)
    if (i + 1 < sg.n) {
      float *buf = jm + (i % NB) * BUF;
      const float *src = M + at(i) * MAT, *lsrc = local + (at(i) * dv + row0) * DK;
      if (i > 0) {
#pragma unroll
        for (int e = 0; e < MAT / 4; e += 256)
          if (e + tid < MAT / 4) cp16(buf + 4 * (e + tid), src + 4 * (e + tid));
      }
      if (tid < JROWS * DK / 4) cp16(buf + MAT + 4 * tid, lsrc + 4 * tid);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < NB - 1; i++) fetch(i);
  for (int e = tid; e < JROWS * DK; e += 256)
    start[(at(0) * dv + row0) * DK + e] = given ? given[((size_t)u * dv + row0) * DK + e] : 0.0f;
  for (int i = 0; i + 1 < sg.n; i++) {
    cp_wait<NB - 2>();
    __syncthreads();  // the rows and this step's buffer are there, the last step's has been read
    fetch(i + NB - 1);
    const float *buf = jm + (i % NB) * BUF;
    if (i > 0) {
      const float *m = buf + kp * KP * DK + c0;
      float x[CPT] = {}, y[CPT] = {};
#pragma unroll
      for (int k = 0; k < KP; k += 4) {
        const float4 p4 = *reinterpret_cast<const float4 *>(&rows[r][kp * KP + k]);
        const float4 q4 = *reinterpret_cast<const float4 *>(&rows[r + 1][kp * KP + k]);
        const float p[4] = {p4.x, p4.y, p4.z, p4.w}, q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int e = 0; e < 4; e++) {
          float w[CPT];
          if constexpr (CPT >= 4) {
#pragma unroll
            for (int c = 0; c < CPT; c += 4)
              *reinterpret_cast<float4 *>(&w[c]) = *reinterpret_cast<const float4 *>(m + (k + e) * DK + c);
          } else {
#pragma unroll
            for (int c = 0; c < CPT; c++) w[c] = m[(k + e) * DK + c];
          }
#pragma unroll
          for (int c = 0; c < CPT; c++) {
            x[c] = fmaf(p[e], w[c], x[c]);
            y[c] = fmaf(q[e], w[c], y[c]);
          }
        }
      }
#pragma unroll
      for (int c = 0; c < CPT; c++) {
        part[kp][r][c0 + c] = x[c];
        part[kp][r + 1][c0 + c] = y[c];
      }
      __syncthreads();
    }
    float *dst = start + ((at(i) + (adjoint ? -1 : 1)) * dv + row0) * DK;
#pragma unroll
    for (int e0 = 0; e0 < JROWS * DK; e0 += 256) {
      const int e = e0 + tid;
      if (e >= JROWS * DK) break;
      const int rr = e / DK, c = e % DK;
      float x = buf[MAT + e];
      if (i > 0) x += (part[0][rr][c] + part[1][rr][c]) + (part[2][rr][c] + part[3][rr][c]);
      rows[rr][c] = x;
      dst[e] = x;
    }
  }
  cp_wait<0>();
}

// The gradients of one 32-token chunk of one unit, from the state before it, the adjoint after
// it, e and du.  With the decay D_ij from token j to token i (a product of gates: exact for
// closed ones), w = scale (g u^T) o D and x = (db u^T) o D (strictly lower), db = beta du:
//     dq = scale D_i0 (g S0) + w K,
//     dk = w^T Q + D_Cj (u dS) - D_i0 (db S0) - (x + x^T) K,
//     dgamma_t = sum over every pair (i >= t > j) that the gate separates, i the state's reader
//                (or dS), j its writer (or S0), each with its decay without gamma_t.
// 256 threads: column groups of four over dk, token groups of four.  Register-tiled products on the CUDA
// cores, several CTAs to an SM: bound by FMA issue and shared memory (300 chunks of d = 32: 33 us).
template <int DK, typename TIO>
__global__ void __launch_bounds__(256) mesa_rule_grads_kernel(RuleArgs a, RuleBwdWorkspace ws) {
  constexpr int C = kRuleChunk, CG = DK / 4, P = C + 1;
  extern __shared__ __align__(16) float sm[];
  const int dv = a.dv, vp = dv + 4, kp = DK + 4;
  float *K = sm, *Q = K + C * kp, *G = Q + C * kp, *Uu = G + C * vp, *Db = Uu + C * vp;
  float *W = Db + C * vp, *V = W + C * P, *X = V + C * P, *D = X + C * P;  // [C][P]
  float *gam = D + C * P, *bet = gam + C, *from0 = bet + C, *xin = from0 + C, *xout = xin + C, *red = xout + C;
  const int u = blockIdx.y, c = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int T = a.T, t0 = c * C, n = min(C, T - t0), NC = gridDim.x;
  const size_t qk0 = ((size_t)a.qk_unit(u) * T + t0) * DK, v0 = ((size_t)u * T + t0) * dv, tu = (size_t)u * T + t0;
  if (tid < C) {
    gam[tid] = tid < n ? a.gamma[tu + tid] : 1.0f;
    bet[tid] = tid < n ? a.beta[tu + tid] : 0.0f;
    xin[tid] = 0.0f;
    xout[tid] = 0.0f;
  }
  __syncthreads();
  for (int i = 4 * tid; i < C * DK; i += 1024) {
    const int t = i / DK, d = i % DK;
    const bool in = t < n;
    *reinterpret_cast<float4 *>(K + t * kp + d) = in ? load4((const TIO *)a.k, qk0 + i) : make_float4(0, 0, 0, 0);
    *reinterpret_cast<float4 *>(Q + t * kp + d) = in ? load4((const TIO *)a.q, qk0 + i) : make_float4(0, 0, 0, 0);
  }
  float bad = 0.0f;  // NaN once a gradient was not finite
  // tokens' rows; dv and dbeta on the way (a warp per token)
  for (int t = warp; t < C; t += 8) {
    float db_sum = 0.0f;
    for (int d = lane; d < dv; d += 32) {
      float g = 0, e = 0, du = 0;
      if (t < n) {
        const size_t at = v0 + (size_t)t * dv + d;
        g = ld((const TIO *)a.dout, at);
        e = ws.e[at];
        du = ws.du[at];
        st((TIO *)a.dv_out, at, bet[t] * du);
        bad = fmaf(bet[t] * du, 0.0f, bad);
      }
      db_sum = fmaf(du, e, db_sum);
      G[t * vp + d] = a.scale * g;
      Uu[t * vp + d] = bet[t] * e;
      Db[t * vp + d] = bet[t] * du;
    }
    db_sum = warp_sum(db_sum);
    bad = fmaf(db_sum, 0.0f, bad);
    if (lane == 0 && t < n) st_gate<TIO>(a, a.dbeta, tu + t, db_sum);
  }
  // decays: D[i][j] = gamma_{j+1} .. gamma_i (j <= i), from0[i] = gamma_0 .. gamma_i
  if (warp == 0) {
    float p = 1.0f, f = 1.0f;
    for (int i = 0; i < C; i++) {
      if (i > lane) p *= gam[i];
      D[i * P + lane] = i >= lane ? p : 0.0f;
      f *= gam[i];
      if (lane == 0) from0[i] = f;
    }
  }
  __syncthreads();
  // token x token products
  {
    const int i0 = tid >> 4, j0 = tid & 15;  // rows i0, i0 + 16; columns j0, j0 + 16
    float gu[2][2] = {}, bu[2][2] = {}, kk[2][2] = {}, qk[2][2] = {};
    for (int d = 0; d < dv; d++) {
      const float ua = Uu[j0 * vp + d], ub = Uu[(j0 + 16) * vp + d];
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const float g = G[(i0 + 16 * x) * vp + d], b = Db[(i0 + 16 * x) * vp + d];
        gu[x][0] = fmaf(g, ua, gu[x][0]);
        gu[x][1] = fmaf(g, ub, gu[x][1]);
        bu[x][0] = fmaf(b, ua, bu[x][0]);
        bu[x][1] = fmaf(b, ub, bu[x][1]);
      }
    }
    for (int d = 0; d < DK; d++) {
      const float ka = K[j0 * kp + d], kb = K[(j0 + 16) * kp + d];
#pragma unroll
      for (int x = 0; x < 2; x++) {
        const float k = K[(i0 + 16 * x) * kp + d], q = Q[(i0 + 16 * x) * kp + d];
        kk[x][0] = fmaf(k, ka, kk[x][0]);
        kk[x][1] = fmaf(k, kb, kk[x][1]);
        qk[x][0] = fmaf(q, ka, qk[x][0]);
        qk[x][1] = fmaf(q, kb, qk[x][1]);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
      for (int y = 0; y < 2; y++) {
        const int i = i0 + 16 * x, j = j0 + 16 * y;
        const float dec = D[i * P + j];
        W[i * P + j] = j <= i ? gu[x][y] * dec : 0.0f;
        V[i * P + j] = j < i ? bu[x][y] * dec : 0.0f;
        X[i * P + j] = gu[x][y] * qk[x][y] - bu[x][y] * kk[x][y];
      }
  }
  __syncthreads();
  // token x state products, then dq and dk: tokens 4 tg .. 4 tg + 3, columns 4 cg .. 4 cg + 3
  const float *S0 = ws.S + ((size_t)u * NC + c) * dv * DK, *dS = ws.dS + ((size_t)u * NC + c) * dv * DK;
  const int cg = tid % CG, tg = tid / CG;
  float cross = 0.0f;  // <dS, S0>
  if (tg < C / 4) {  // (whole warps: 8 CG threads)
    float4 gS[4] = {}, bS[4] = {}, uS[4] = {};
    auto axpy = [](float f, const float4 &x, float4 &y) {
      y.x = fmaf(f, x.x, y.x);
      y.y = fmaf(f, x.y, y.y);
      y.z = fmaf(f, x.z, y.z);
      y.w = fmaf(f, x.w, y.w);
    };
    for (int v = 0; v < dv; v++) {
      const float4 s0 = *reinterpret_cast<const float4 *>(S0 + (size_t)v * DK + 4 * cg);
      const float4 ds = *reinterpret_cast<const float4 *>(dS + (size_t)v * DK + 4 * cg);
      if (tg == 0) cross = fmaf(s0.x, ds.x, fmaf(s0.y, ds.y, fmaf(s0.z, ds.z, fmaf(s0.w, ds.w, cross))));
#pragma unroll
      for (int m = 0; m < 4; m++) {
        axpy(G[(4 * tg + m) * vp + v], s0, gS[m]);
        axpy(Db[(4 * tg + m) * vp + v], s0, bS[m]);
        axpy(Uu[(4 * tg + m) * vp + v], ds, uS[m]);
      }
    }
#pragma unroll
    for (int m = 0; m < 4; m++) {
      const int t = 4 * tg + m;
      const float f0 = from0[t], fC = D[(C - 1) * P + t];
      const float4 q = *reinterpret_cast<const float4 *>(Q + t * kp + 4 * cg);
      const float4 k = *reinterpret_cast<const float4 *>(K + t * kp + 4 * cg);
      float xi = gS[m].x * q.x + gS[m].y * q.y + gS[m].z * q.z + gS[m].w * q.w -
                 (bS[m].x * k.x + bS[m].y * k.y + bS[m].z * k.z + bS[m].w * k.w);
      float xo = uS[m].x * k.x + uS[m].y * k.y + uS[m].z * k.z + uS[m].w * k.w;
#pragma unroll
      for (int o = (CG < 32 ? CG : 32) / 2; o > 0; o >>= 1) {
        xi += __shfl_xor_sync(0xffffffffu, xi, o);
        xo += __shfl_xor_sync(0xffffffffu, xo, o);
      }
      if (cg == 0) {
        xin[t] = xi;
        xout[t] = xo;
      }
      float4 dq = make_float4(f0 * gS[m].x, f0 * gS[m].y, f0 * gS[m].z, f0 * gS[m].w);
      float4 dk = make_float4(fC * uS[m].x - f0 * bS[m].x, fC * uS[m].y - f0 * bS[m].y, fC * uS[m].z - f0 * bS[m].z,
                              fC * uS[m].w - f0 * bS[m].w);
      for (int s = 0; s < C; s++) {
        const float4 ks = *reinterpret_cast<const float4 *>(K + s * kp + 4 * cg);
        const float4 qs = *reinterpret_cast<const float4 *>(Q + s * kp + 4 * cg);
        axpy(W[t * P + s], ks, dq);
        axpy(W[s * P + t], qs, dk);
        axpy(-(V[t * P + s] + V[s * P + t]), ks, dk);
      }
      if (t < n) {
        bad = nonfinite4(dq, nonfinite4(dk, bad));
        if (ws.dqp) {
          const size_t at = (tu + t) * DK + 4 * cg;
          *reinterpret_cast<float4 *>(ws.dqp + at) = dq;
          *reinterpret_cast<float4 *>(ws.dkp + at) = dk;
        } else {
          const size_t at = qk0 + (size_t)t * DK + 4 * cg;
          TIO *dqo = (TIO *)a.dq, *dko = (TIO *)a.dk_out;
          st(dqo, at, dq.x);
          st(dqo, at + 1, dq.y);
          st(dqo, at + 2, dq.z);
          st(dqo, at + 3, dq.w);
          st(dko, at, dk.x);
          st(dko, at + 1, dk.y);
          st(dko, at + 2, dk.z);
          st(dko, at + 3, dk.w);
        }
      }
    }
  }
  cross = warp_sum(cross);
  if (lane == 0) red[warp] = cross;
  __syncthreads();
  cross = 0.0f;
  for (int w = 0; w < 8; w++) cross += red[w];
  // dgamma: a warp per token, lanes over i (readers) or j (writers)
  for (int t = warp; t < n; t += 8) {
    const float prev0 = t > 0 ? from0[t - 1] : 1.0f, toC = D[(C - 1) * P + t];
    const float dprev = lane < t ? D[(t - 1) * P + lane] : 0.0f;
    float col = 0.0f;  // sum over i >= t of D[i][t] X[i][lane]
    for (int i = t; i < C; i++) col = fmaf(D[i * P + t], X[i * P + lane], col);
    float s = (lane < t ? dprev * (col + toC * xout[lane]) : 0.0f) + prev0 * (D[lane * P + t] * xin[lane]);
    s = fmaf(toC * prev0, cross, warp_sum(s));
    bad = fmaf(s, 0.0f, bad);
    if (lane == 0) st_gate<TIO>(a, a.dgamma, tu + t, s);
  }
  if (!(bad == 0.0f)) atomicOr(a.status, tc_err_nonfinite());
}

// The sums over the value heads of a key head, in a fixed order (memory).
template <typename TIO>
__global__ void __launch_bounds__(256) mesa_rule_group_sum_kernel(RuleArgs a, const float *dqp, const float *dkp) {
  const size_t per = (size_t)a.T * a.dk, total = (size_t)a.B * a.Hk * per;
  const int group = a.H / a.Hk;
  float bad = 0.0f;  // NaN once a sum was not finite
  for (size_t i = 4 * ((size_t)blockIdx.x * 256 + threadIdx.x); i < total; i += (size_t)gridDim.x * 1024) {
    const size_t uk = i / per, at = i % per, b = uk / a.Hk, hk = uk % a.Hk;
    float4 q = make_float4(0, 0, 0, 0), k = q;
    for (int g = 0; g < group; g++) {
      const size_t src = (b * a.H + hk * group + g) * per + at;
      const float4 x = *reinterpret_cast<const float4 *>(dqp + src), y = *reinterpret_cast<const float4 *>(dkp + src);
      q = make_float4(q.x + x.x, q.y + x.y, q.z + x.z, q.w + x.w);
      k = make_float4(k.x + y.x, k.y + y.y, k.z + y.z, k.w + y.w);
    }
    TIO *dq = (TIO *)a.dq + i, *dk = (TIO *)a.dk_out + i;
    st(dq, 0, q.x);
    st(dq, 1, q.y);
    st(dq, 2, q.z);
    st(dq, 3, q.w);
    st(dk, 0, k.x);
    st(dk, 1, k.y);
    st(dk, 2, k.z);
    st(dk, 3, k.w);
    bad = nonfinite4(q, nonfinite4(k, bad));
  }
  if (!(bad == 0.0f)) atomicOr(a.status, tc_err_nonfinite());
}

// One decode step.  A lane holds 16 values of a row (float4 groups DK/16 lanes apart, so that
// a group of lanes reads whole 128-byte lines for dk = 128), a warp four rows at a time for
// dk = 128; the state is read and written once and its traffic is the bound (256 x 16 heads, d = 128: 91 us,
// 5.9 TB/s).  A CTA takes 32 rows and more of one unit: small batches spread over many SMs.
template <int DK, typename TIO>
__global__ void __launch_bounds__(128) mesa_rule_step_kernel(RuleStepArgs a) {
  constexpr int LPR = DK / 16, RPW = 32 / LPR, PASS = DK == 128 ? 2 : 1;
  const int u = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = lane % LPR, rs = lane / LPR;
  const int row0 = (blockIdx.y * 4 + warp) * RPW * PASS;
  const int uk = (u / a.H) * a.Hk + (u % a.H) / (a.H / a.Hk);
  float4 s[PASS][4];
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const int row = row0 + p * RPW + rs;
    const float4 *src = reinterpret_cast<const float4 *>(a.S + ((size_t)u * a.dv + row) * DK);
#pragma unroll
    for (int i = 0; i < 4; i++) s[p][i] = row < a.dv ? src[j + LPR * i] : make_float4(0, 0, 0, 0);
  }
  float4 k[4], q[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    k[i] = load4((const TIO *)a.k, (size_t)uk * DK + 4 * (j + LPR * i));
    q[i] = load4((const TIO *)a.q, (size_t)uk * DK + 4 * (j + LPR * i));
  }
  const float g = a.gamma[u], b = a.beta[u];
  auto dot = [&](const float4 (&x)[4], const float4 (&y)[4]) {
    float t[4];
#pragma unroll
    for (int i = 0; i < 4; i++) t[i] = fmaf(x[i].x, y[i].x, fmaf(x[i].y, y[i].y, fmaf(x[i].z, y[i].z, x[i].w * y[i].w)));
    float d = (t[0] + t[1]) + (t[2] + t[3]);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    return d;
  };
#pragma unroll
  for (int p = 0; p < PASS; p++) {
    const int row = row0 + p * RPW + rs;
    const float v = row < a.dv ? ld((const TIO *)a.v, (size_t)u * a.dv + row) : 0.0f;
    const float uu = b * fmaf(-g, dot(s[p], k), v);
    float4 *dst = reinterpret_cast<float4 *>(a.S + ((size_t)u * a.dv + row) * DK);
#pragma unroll
    for (int i = 0; i < 4; i++) {
      s[p][i].x = fmaf(g, s[p][i].x, uu * k[i].x);
      s[p][i].y = fmaf(g, s[p][i].y, uu * k[i].y);
      s[p][i].z = fmaf(g, s[p][i].z, uu * k[i].z);
      s[p][i].w = fmaf(g, s[p][i].w, uu * k[i].w);
      if (row < a.dv) dst[j + LPR * i] = s[p][i];
    }
    const float o = a.scale * dot(s[p], q);
    if (row < a.dv && j == 0) {
      st((TIO *)a.out, (size_t)u * a.dv + row, o);
      if (!isfinite(o)) atomicOr(a.status, tc_err_nonfinite());
    }
  }
}

template <int DK, typename TIO, int MODE>
int launch_scan(const RuleArgs &a, const RuleBwdWorkspace &ws, const RuleScanSegments &sg, cudaStream_t st) {
  const int tiles = (a.dv + ROWS - 1) / ROWS + (MODE == kSegment ? (DK + ROWS - 1) / ROWS : 0);
  const int segs = MODE == kSegment || MODE == kSegAdjoint ? sg.n - 1 : sg.n;
  timing_mark_begin(K_RULE_SCAN, st);
  mesa_rule_scan_kernel<DK, TIO, MODE><<<dim3(tiles, a.units(), segs), ROWS * lanes_per_row(DK), 0, st>>>(a, ws, sg);
  timing_mark_end(K_RULE_SCAN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

template <int DK>
int launch_scan_join(const RuleArgs &a, const RuleScanSegments &sg, bool adjoint, cudaStream_t st) {
  const int smem = JoinBuffers<DK>::bytes;
  auto kfn = mesa_rule_scan_join_kernel<DK>;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -1;
  timing_mark_begin(K_RULE_JOIN, st);
  kfn<<<dim3(a.dv / JROWS, a.units()), 256, smem, st>>>(sg, adjoint ? a.dS_final : a.S0, a.dv, adjoint);  // (dv: a multiple of 16)
  timing_mark_end(K_RULE_JOIN, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// Segments of a unit's tokens: about 256 threads for each of a GB300's 152 SMs (the chain of one CTA leaves most of an
// SM idle; the rows of d = 128 take twice the threads of the others and fill it twice as soon), whole chunks (two at
// least for d = 128), at most 16 (the join is a chain over them); fewer than four are not worth the two more passes.
// us of one scan, of n segments: forward of 2 x 4 x 2048 x 64 fp32 447, 16: 69, 24: 78, 32: 74; forward / backward of 32
// units x 1024, d 128, 219 / 831, four: 307 / 999; of 8 units 219 / 471, eight: 109 / 303, 16: 132 / 348; of one
// unit x 128 36 / 115, four: 35 / 139; 32 units x 1024, d 64, 170 / 473, nine: 86 / 321.
int scan_segments(int U, int T, int dk, int dv) {
  const int NC = (T + kRuleChunk - 1) / kRuleChunk, ctas = U * ((dv + ROWS - 1) / ROWS);
  int n = ctas > 0 ? 152 * 256 / (ctas * ROWS * lanes_per_row(dk)) : 1;
  const int most = dk == 128 ? NC / 2 : NC;
  if (n > most) n = most;
  if (n > 16) n = 16;
  return n < 4 ? 1 : n;
}

template <int DK, typename TIO>
int launch_bwd_t(const RuleArgs &a, const RuleBwdWorkspace &ws, const RuleScanSegments &sg, cudaStream_t st) {
  if (sg.n > 1 && (launch_scan<DK, TIO, kSegment>(a, ws, sg, st) != 0 || launch_scan_join<DK>(a, sg, false, st) != 0 ||
                   launch_scan<DK, TIO, kSegAdjoint>(a, ws, sg, st) != 0 || launch_scan_join<DK>(a, sg, true, st) != 0))
    return -1;
  if (launch_scan<DK, TIO, kStates>(a, ws, sg, st) != 0 || launch_scan<DK, TIO, kAdjoint>(a, ws, sg, st) != 0) return -1;
  const int smem = (2 * kRuleChunk * (DK + 4) + 3 * kRuleChunk * (a.dv + 4) + 4 * kRuleChunk * (kRuleChunk + 1) +
                    5 * kRuleChunk + 8) * (int)sizeof(float);
  auto kfn = mesa_rule_grads_kernel<DK, TIO>;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return -1;
  timing_mark_begin(K_RULE_GRADS, st);
  kfn<<<dim3((a.T + kRuleChunk - 1) / kRuleChunk, a.units()), 256, smem, st>>>(a, ws);
  timing_mark_end(K_RULE_GRADS, st);
  if (cudaPeekAtLastError() != cudaSuccess) return -1;
  return ws.dqp ? launch_rule_group_sum(a, ws.dqp, ws.dkp, st) : 0;
}

template <int DK, typename TIO>
int launch_step_t(const RuleStepArgs &a, cudaStream_t st) {
  constexpr int rows = 4 * (32 / (DK / 16)) * (DK == 128 ? 2 : 1);
  timing_mark_begin(K_RULE_STEP, st);
  mesa_rule_step_kernel<DK, TIO><<<dim3(a.N * a.H, (a.dv + rows - 1) / rows), 128, 0, st>>>(a);
  timing_mark_end(K_RULE_STEP, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

// F<DK, TIO>(...) for the supported key sizes and element types.
#define MESA_RULE_DISPATCH(F, a, ...)                                                          \
  switch (a.dk) {                                                                              \
    case 16: return a.dtype == 1 ? F<16, __nv_bfloat16>(__VA_ARGS__) : F<16, float>(__VA_ARGS__);   \
    case 32: return a.dtype == 1 ? F<32, __nv_bfloat16>(__VA_ARGS__) : F<32, float>(__VA_ARGS__);   \
    case 64: return a.dtype == 1 ? F<64, __nv_bfloat16>(__VA_ARGS__) : F<64, float>(__VA_ARGS__);   \
    case 128: return a.dtype == 1 ? F<128, __nv_bfloat16>(__VA_ARGS__) : F<128, float>(__VA_ARGS__); \
  }                                                                                            \
  return -1

template <int DK, typename TIO>
int launch_fwd_t(const RuleArgs &a, const RuleScanSegments &sg, cudaStream_t st) {
  const RuleBwdWorkspace none{};
  if (sg.n > 1 && (launch_scan<DK, TIO, kSegment>(a, none, sg, st) != 0 || launch_scan_join<DK>(a, sg, false, st) != 0))
    return -1;
  return launch_scan<DK, TIO, kForward>(a, none, sg, st);
}

}  // namespace

size_t rule_scan_workspace(int U, int T, int dk, int dv, bool backward) {
  const size_t n = scan_segments(U, T, dk, dv), mat = (size_t)dk * dk * sizeof(float), state = (size_t)dv * dk * sizeof(float);
  return n == 1 ? 0 : U * n * (2 * state + mat) * (backward ? 2 : 1);
}
RuleScanSegments rule_scan_parts(int U, int T, int dk, int dv, bool backward, void *workspace) {
  const int blocks = kRuleChunk / TB, NC = (T + kRuleChunk - 1) / kRuleChunk;
  RuleScanSegments sg;
  sg.n = scan_segments(U, T, dk, dv);
  sg.per = (NC + sg.n - 1) / sg.n * blocks;
  if (sg.n == 1) return sg;
  const size_t mat = (size_t)U * sg.n * dk * dk, state = (size_t)U * sg.n * dv * dk;
  sg.n = (NC * blocks + sg.per - 1) / sg.per;  // (no empty one)
  sg.S = (float *)workspace;
  sg.loc = sg.S + state;
  sg.Tr = sg.loc + state;
  if (backward) {
    sg.A = sg.Tr + mat;
    sg.adj = sg.A + state;
    sg.TrT = sg.adj + state;
  }
  return sg;
}

int launch_rule_forward(const RuleArgs &a, const RuleScanSegments &sg, cudaStream_t st) {
  MESA_RULE_DISPATCH(launch_fwd_t, a, a, sg, st);
}
int launch_rule_backward(const RuleArgs &a, const RuleBwdWorkspace &ws, const RuleScanSegments &sg, cudaStream_t st) {
  MESA_RULE_DISPATCH(launch_bwd_t, a, a, ws, sg, st);
}
int launch_rule_step(const RuleStepArgs &a, cudaStream_t st) { MESA_RULE_DISPATCH(launch_step_t, a, a, st); }

int launch_rule_group_sum(const RuleArgs &a, const float *dqp, const float *dkp, cudaStream_t st) {
  const size_t total = (size_t)a.B * a.Hk * a.T * a.dk / 4;
  const size_t want = (total + 255) / 256;
  const int grid = (int)(want < 4096 ? want : 4096);
  timing_mark_begin(K_RULE_GROUP, st);
  if (a.dtype == 1)
    mesa_rule_group_sum_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(a, dqp, dkp);
  else
    mesa_rule_group_sum_kernel<float><<<grid, 256, 0, st>>>(a, dqp, dkp);
  timing_mark_end(K_RULE_GROUP, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace mesa
