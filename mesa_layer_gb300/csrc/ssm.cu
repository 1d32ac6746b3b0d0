// ssm.cu -- the selective state space scan on the CUDA cores (every size and type but what the tensor cores take), and
// its decode step.
//
// Per unit, D_t = softplus(dt_t + bias), a_t = e^(D_t A) (0 where a document starts), S_t = a_t S_{t-1} + D_t v_t k_t^T,
// o_t = S_t q_t + skip v_t.  In a chunk of C = 32 tokens, l_i the log-decay from its start:
//     o_i = e^{l_i} S q_i + sum_{j <= i} e^{l_i - l_j} (q_i . k_j) D_j v_j + skip v_i,
//     S' = e^{l_C} S + sum_j e^{l_C - l_j} D_j v_j k_j^T,
// so that nothing but the states runs in sequence: what each chunk adds to the state (all chunks side by side), a
// running sum over the chunks (each element of the state on its own), then the outputs (all chunks side by side).
// Everything is fp32; log-decays are sums of two fp32 values (ssm_common.cuh).  32 tokens: the states that go through
// memory cost 2 dk dv / 32 values a token, the products within a chunk 32 (dk + dv) / 2.
#include <cuda_runtime.h>

#include <type_traits>

#include "launch.h"
#include "ssm_simt.cuh"

namespace mesa {

using namespace ssm;

namespace {

// grid (NC, U, 1 or 2): what chunk c adds to its unit's state, [dv, dk], to ws.S, and ws.decay; z = 1: what it gives the
// adjoint of the state before it, sum_i e^{l_i} g_i q_i^T, to ws.R.
template <int DK, int DV>
__global__ void __launch_bounds__(kThreads) mesa_ssm_states_kernel(SsmArgs a, SsmWorkspace ws) {
  extern __shared__ float4 smem4[];
  float *k = reinterpret_cast<float *>(smem4), *v = k + C * (DK + 4);
  __shared__ Gates g;
  const bool adjoint = blockIdx.z == 1;
  const int u = blockIdx.y, c = blockIdx.x, NC = gridDim.x, t0 = c * C, n = min(C, a.T - t0);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  may_follow();
  load_rows<DK, C, kThreads>(k, adjoint ? a.q : a.k, a.dtype, (size_t)a.qk_unit(u) * a.T + t0, n, a.dk);
  load_rows<DV, C, kThreads>(v, adjoint ? a.dout : a.v, a.dtype, (size_t)u * a.T + t0, n, a.dv);
  if (threadIdx.x < 32) gates_load(g, a, u, t0, n, threadIdx.x);
  __syncthreads();
  for (int i = threadIdx.x; i < C * DV; i += kThreads) {
    const int t = i / DV;
    v[t * (DV + 4) + i % DV] *= adjoint ? g.f[t] : g.c[t] * g.step[t];
  }
  __syncthreads();
  float acc[DV / 16][DK / 16];
  zero(acc);
  mm_outer<C, DV, DK>(acc, v, DV + 4, k, DK + 4, ty, tx);
  ahead_done();
  if (threadIdx.x == 0 && !adjoint) {
    ws.decay[(size_t)u * NC + c] = g.f[C - 1];
    if (ws.clear && c == 0 && u == 0) *a.status = 0;  // (the kernels after this one report)
  }
  float *dst = (adjoint ? ws.R : ws.S) + ((size_t)u * NC + c) * a.dv * a.dk;
#pragma unroll
  for (int i = 0; i < DV / 16; i++) {
    const int p = frag<DV>(ty, i);
    if (p >= a.dv) continue;
    if constexpr (DK >= 64) {  // (dk = DK)
#pragma unroll
      for (int j = 0; j < DK / 16; j += 4)
        *reinterpret_cast<float4 *>(dst + p * a.dk + frag<DK>(tx, j)) = make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < DK / 16; j++)
        if (frag<DK>(tx, j) < a.dk) dst[p * a.dk + frag<DK>(tx, j)] = acc[i][j];
    }
  }
}

// Four elements of a unit's state a thread, chunk after chunk: what a chunk adds is replaced by the state before it
// (from S0 on; what is left after the last goes to S_final), the adjoints' (z = 1) by the adjoint after it, backwards (from
// dS_final to dS0).  Sixteen chunks' values are asked for together: their latency is what this takes.
__global__ void __launch_bounds__(128) mesa_ssm_scan_kernel(SsmArgs a, SsmWorkspace ws, int NC) {
  constexpr int AHEAD = 16;
  const bool adjoint = blockIdx.z == 1;
  const int n4 = a.dv * a.dk / 4, e = blockIdx.x * 128 + threadIdx.x, u = blockIdx.y;
  may_follow();
  ahead_done();
  if (e >= n4) return;
  const float4 *from = reinterpret_cast<const float4 *>(adjoint ? a.dS_final : a.S0);
  float4 *to = reinterpret_cast<float4 *>(adjoint ? a.dS0 : a.S_final);
  float4 *x = reinterpret_cast<float4 *>(adjoint ? ws.R : ws.S) + (size_t)u * NC * n4 + e;
  const float *decay = ws.decay + (size_t)u * NC;
  float4 s = from ? from[(size_t)u * n4 + e] : make_float4(0, 0, 0, 0);
  for (int c0 = 0; c0 < NC; c0 += AHEAD) {
    float4 d[AHEAD];
    float w[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; i++) {
      const int c = adjoint ? NC - 1 - c0 - i : c0 + i;
      if (c0 + i < NC) {
        d[i] = x[(size_t)c * n4];
        w[i] = decay[c];
      }
    }
#pragma unroll
    for (int i = 0; i < AHEAD; i++) {
      const int c = adjoint ? NC - 1 - c0 - i : c0 + i;
      if (c0 + i < NC) {
        x[(size_t)c * n4] = s;
        s = make_float4(fmaf(w[i], s.x, d[i].x), fmaf(w[i], s.y, d[i].y), fmaf(w[i], s.z, d[i].z), fmaf(w[i], s.w, d[i].w));
      }
    }
  }
  if (to) to[(size_t)u * n4 + e] = s;
}

// grid (NC, U): a chunk's outputs from the state before it (of one chunk: S0).
template <int DK, int DV>
__global__ void __launch_bounds__(kFew) mesa_ssm_out_kernel(SsmArgs a, SsmWorkspace ws) {
  constexpr int TY = kFew / 16;
  extern __shared__ float4 smem4[];
  float *q = reinterpret_cast<float *>(smem4), *k = q + C * (DK + 4), *v = k + C * (DK + 4), *S = v + C * (DV + 4),
        *M = S + kPart<DV> * (DK + 4);
  __shared__ Gates g;
  const int u = blockIdx.y, c = blockIdx.x, NC = gridDim.x, t0 = c * C, n = min(C, a.T - t0);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  may_follow();
  const float *state = NC > 1 ? ws.S + ((size_t)u * NC + c) * a.dv * a.dk : a.S0 ? a.S0 + (size_t)u * a.dv * a.dk : nullptr;
  load_rows<DK, C>(q, a.q, a.dtype, (size_t)a.qk_unit(u) * a.T + t0, n, a.dk);
  load_rows<DK, C>(k, a.k, a.dtype, (size_t)a.qk_unit(u) * a.T + t0, n, a.dk);
  load_rows<DV, C>(v, a.v, a.dtype, (size_t)u * a.T + t0, n, a.dv);
  if (threadIdx.x < 32) gates_load(g, a, u, t0, n, threadIdx.x);
  ahead_done();  // (the states)
  constexpr int PART = kPart<DV>;
  if (state) load_rows<DK, PART>(S, state, 0, 0, min(a.dv, PART), a.dk);
  __syncthreads();
  {
    float acc[4][2];
    zero(acc);
    mm_nt<TY, DK>(acc, q, DK + 4, k, DK + 4, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int r = ty + TY * i, t = tx + 16 * j;
        const float d = g.decay(r, t);  // (what lies across a start or above the diagonal is dropped, whatever it is)
        M[r * LDC + t] = t <= r && t >= g.s[r] ? acc[i][j] * d * g.step[t] : 0.0f;
      }
  }
  float acc[4][DV / 16];
  zero(acc);
  if (state) mm_nt<TY, DK, 0, PART / 16>(acc, q, DK + 4, S, DK + 4, ty, tx);
  __syncthreads();
  if constexpr (PART < DV) {
    if (state) {
      load_rows<DK, PART>(S, state, 0, PART, a.dv - PART, a.dk);
      __syncthreads();
      mm_nt<TY, DK, PART / 16, PART / 16>(acc, q, DK + 4, S, DK + 4, ty, tx);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < DV / 16; j++) acc[i][j] = g.s[ty + TY * i] < 0 ? acc[i][j] * g.f[ty + TY * i] : 0.0f;
  mm_lower<TY>(acc, M, LDC, v, DV + 4, ty, tx);
  const float skip = a.skip ? a.skip[u % a.H] : 0.0f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; i++)
#pragma unroll
    for (int j = 0; j < DV / 16; j++) {
      const int r = ty + TY * i, p = tx + 16 * j;
      if (r < n && p < a.dv) {
        const float o = a.skip ? fmaf(skip, v[r * (DV + 4) + p], acc[i][j]) : acc[i][j];
        store(a.out, a.dtype == 0, ((size_t)u * a.T + t0 + r) * a.dv + p, o);
        bad |= !isfinite(o);
      }
    }
  if (bad) atomicOr(a.status, tc_err_nonfinite());
}

template <int DK, int DV>
struct States {
  static int run(const SsmArgs &a, const SsmWorkspace &ws, int NC, bool adjoints, cudaStream_t st) {
    const size_t smem = sizeof(float) * C * (DK + DV + 8);
    const int n = adjoints ? 2 : 1;
    timing_mark_begin(K_SSM_STATES, st);
    bool ok = launch(mesa_ssm_states_kernel<DK, DV>, dim3(NC, a.units(), n), kThreads, smem, ws.clear, st, a, ws);
    timing_mark_end(K_SSM_STATES, st);
    if (!ok) return -1;
    timing_mark_begin(K_SSM_SCAN, st);
    ok = launch_after(mesa_ssm_scan_kernel, dim3((a.dv * a.dk / 4 + 127) / 128, a.units(), n), 128, 0, st, a, ws, NC);
    timing_mark_end(K_SSM_SCAN, st);
    return ok && cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
  }
};
template <int DK, int DV>
struct Out {
  static int run(const SsmArgs &a, const SsmWorkspace &ws, int NC, cudaStream_t st) {
    const size_t smem = sizeof(float) * (C * (2 * DK + DV + 12) + kPart<DV> * (DK + 4) + C * LDC);
    timing_mark_begin(K_SSM_OUT, st);
    const bool ok = launch(mesa_ssm_out_kernel<DK, DV>, dim3(NC, a.units()), kFew, smem, NC == 1, st, a, ws);
    timing_mark_end(K_SSM_OUT, st);
    return ok && cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
  }
};

}  // namespace

// The states before every chunk; with adjoints those after every chunk, too.
int launch_ssm_states(const SsmArgs &a, const SsmWorkspace &ws, bool adjoints, cudaStream_t st) {
  return by_size<States>(a.dk, a.dv, a, ws, (a.T + C - 1) / C, adjoints, st);
}

int launch_ssm_forward(const SsmArgs &a, SsmWorkspace ws, cudaStream_t st) {
  const int NC = (a.T + C - 1) / C;
  ws.clear = NC > 1;
  if (NC > 1) return launch_ssm_states(a, ws, false, st) == 0 ? by_size<Out>(a.dk, a.dv, a, ws, NC, st) : -1;
  // outputs of one chunk come before its state: S_final may be S0's memory
  if (cudaMemsetAsync(a.status, 0, sizeof(unsigned), st) != cudaSuccess || by_size<Out>(a.dk, a.dv, a, ws, NC, st) != 0) return -1;
  return a.S_final ? launch_ssm_states(a, ws, false, st) : 0;
}

// ---- the decode step -------------------------------------------------------------------------------
namespace {

// S <- a S + (D v) k^T, o = S q + skip v for `rows` rows of one unit's state: a row's dk channels lie in L = dk / 4
// lanes, a warp takes 32 / L rows at a time, R of them in flight.  Bound by the states' traffic.
template <int DK, typename TIO>
__global__ void __launch_bounds__(kThreads) mesa_ssm_step_kernel(SsmStepArgs a, int rows) {
  constexpr int L = DK / 4, RW = 32 / L, R = 4;  // lanes a row, rows a warp, steps in flight
  const int u = blockIdx.x, h = u % a.H, p0 = blockIdx.y * rows, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t qk = (size_t)(u / a.H) * a.Hk + h / (a.H / a.Hk);
  const int c = 4 * (lane % L);
  const float4 q = load4(static_cast<const TIO *>(a.q), qk * DK + c), k = load4(static_cast<const TIO *>(a.k), qk * DK + c);
  const float step = softplus(a.dt[u] + (a.dt_bias ? a.dt_bias[h] : 0.0f));
  const Two l = log2_decay(step, a.A[h]);
  const float decay = exp2f(l.hi) * (1.0f + 0.69314718f * l.lo), skip = a.skip ? a.skip[h] : 0.0f;
  const TIO *v = static_cast<const TIO *>(a.v) + (size_t)u * a.dv;
  TIO *out = static_cast<TIO *>(a.out) + (size_t)u * a.dv;
  bool bad = false;
  for (int r0 = warp * RW * R; r0 < rows; r0 += kThreads / 32 * RW * R) {
    float4 S[R];
    float x[R], o[R];
#pragma unroll
    for (int i = 0; i < R; i++) {
      const int p = r0 + i * RW + lane / L;
      if (p < rows) {
        S[i] = *reinterpret_cast<const float4 *>(a.S + ((size_t)u * a.dv + p0 + p) * DK + c);
        x[i] = ld(v, p0 + p);
      }
    }
#pragma unroll
    for (int i = 0; i < R; i++) {
      const int p = r0 + i * RW + lane / L;
      const float w = step * x[i];
      S[i] = make_float4(fmaf(w, k.x, decay * S[i].x), fmaf(w, k.y, decay * S[i].y), fmaf(w, k.z, decay * S[i].z),
                         fmaf(w, k.w, decay * S[i].w));
      if (p < rows) *reinterpret_cast<float4 *>(a.S + ((size_t)u * a.dv + p0 + p) * DK + c) = S[i];
      o[i] = fmaf(S[i].x, q.x, fmaf(S[i].y, q.y, fmaf(S[i].z, q.z, S[i].w * q.w)));
    }
#pragma unroll
    for (int i = 0; i < R; i++) o[i] = group_sum<L>(o[i]);
#pragma unroll
    for (int i = 0; i < R; i++) {
      const int p = r0 + i * RW + lane / L;
      if (p < rows && lane % L == 0) {
        const float y = a.skip ? fmaf(skip, x[i], o[i]) : o[i];
        st(out, p0 + p, y);
        bad |= !isfinite(y);
      }
    }
  }
  if (bad) atomicOr(a.status, tc_err_nonfinite());
}

template <typename TIO>
int step_by_size(const SsmStepArgs &a, cudaStream_t st) {
  const int U = a.N * a.H;
  const int rows = a.dv < 32 ? a.dv : 32;  // (a unit's rows on several CTAs: one sequence's few units fill more SMs)
  const dim3 grid(U, a.dv / rows);
  timing_mark_begin(K_SSM_STEP, st);
  switch (a.dk) {
    case 16: mesa_ssm_step_kernel<16, TIO><<<grid, kThreads, 0, st>>>(a, rows); break;
    case 32: mesa_ssm_step_kernel<32, TIO><<<grid, kThreads, 0, st>>>(a, rows); break;
    case 64: mesa_ssm_step_kernel<64, TIO><<<grid, kThreads, 0, st>>>(a, rows); break;
    default: mesa_ssm_step_kernel<128, TIO><<<grid, kThreads, 0, st>>>(a, rows); break;
  }
  timing_mark_end(K_SSM_STEP, st);
  return cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace

int launch_ssm_step(const SsmStepArgs &a, cudaStream_t st) {
  return a.dtype == 1 ? step_by_size<__nv_bfloat16>(a, st) : step_by_size<float>(a, st);
}

}  // namespace mesa
