// ssm_bwd.cu -- gradients of the selective state space scan on the CUDA cores.
//
// With S the state before a chunk of 32 tokens, R the adjoint of the state after it (both from ssm.cu's passes), g =
// dL/do, E_ij = e^{l_i - l_j} (0 for j > i and across starts), f_i the decay from before the chunk, c_j to its end:
//     W = (g V^T) o E D,   dq = f (g S) + W K,   dk = W^T Q + c D (V R),
//     du = ((Q K^T) o E)^T g + c (K R^T),   dv = D du + skip g,
//     d log a_t = sum over readers i >= t (or the state after) and writers j < t (or the state before) of what passes
//     between them: (Q K^T o W) inside the chunk, f (g S) . q into it, c D (V R) . k out of it, <R, S> across,
//     d dt = (du . v + A d log a) sigmoid(dt + bias),   dA = sum D d log a.
// The pairs are summed as they are, never as a difference of sums, so that a gate's gradient is as exact as its terms.
#include <cuda_runtime.h>

#include <type_traits>

#include "gated_delta.h"
#include "launch.h"
#include "ssm_simt.cuh"

namespace mesa {

using namespace ssm;

int launch_ssm_states(const SsmArgs &a, const SsmWorkspace &ws, bool adjoints, cudaStream_t st);

namespace {

__device__ __forceinline__ float sum16(float x) {  // over a row's 16 threads
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Threads a chunk: with four rows each of 128 channels their sums leave an SM too few warps (us of 2 x 16 x 4096 fp32, both
// 128, 128 threads 830, 256 threads 729; both 64 239, 260).
template <int DK, int DV>
constexpr int kGradThreads = DK + DV > 192 ? 256 : kFew;

// grid (NC, U)
template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads<DK, DV>) mesa_ssm_grads_kernel(SsmArgs a, SsmWorkspace ws) {
  constexpr int LK = DK + 4, LV = DV + 4, PART = kPart<DV>, TH = kGradThreads<DK, DV>, TY = TH / 16, RI = C / TY;
  extern __shared__ float4 smem4[];
  float *q = reinterpret_cast<float *>(smem4), *k = q + C * LK, *v = k + C * LK, *g = v + C * LV, *S = g + C * LV,
        *M = S + PART * LK, *W = M + C * LDC;
  constexpr int LX = C + 1;  // the pairs' terms, in the states' place until these come
  float *X = S;
  __shared__ Gates ga;
  __shared__ float x_in[C], x_out[C], duv[C], gv[C], pairs[C], across[TH / 32];
  const int u = blockIdx.y, c = blockIdx.x, NC = gridDim.x, t0 = c * C, n = min(C, a.T - t0), h = u % a.H;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, lane = tid & 31, warp = tid >> 5;
  const size_t at = ((size_t)u * NC + c) * a.dv * a.dk;
  may_follow();
  load_rows<DK, C, TH>(q, a.q, a.dtype, (size_t)a.qk_unit(u) * a.T + t0, n, a.dk);
  load_rows<DK, C, TH>(k, a.k, a.dtype, (size_t)a.qk_unit(u) * a.T + t0, n, a.dk);
  load_rows<DV, C, TH>(v, a.v, a.dtype, (size_t)u * a.T + t0, n, a.dv);
  load_rows<DV, C, TH>(g, a.dout, a.dtype, (size_t)u * a.T + t0, n, a.dv);
  if (warp == 0) gates_load(ga, a, u, t0, n, lane);
  __syncthreads();
  {
    float G[RI][2], Hm[RI][2];
    zero(G);
    zero(Hm);
    mm_nt<TY, DK>(G, q, LK, k, LK, ty, tx);
    mm_nt<TY, DV>(Hm, g, LV, v, LV, ty, tx);
#pragma unroll
    for (int i = 0; i < RI; i++)
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int r = ty + TY * i, t = tx + 16 * j;
        const bool on = t <= r && t >= ga.s[r];
        const float d = ga.decay(r, t), w = on ? Hm[i][j] * d * ga.step[t] : 0.0f;
        M[r * LDC + t] = on ? G[i][j] * d : 0.0f;
        W[r * LDC + t] = w;
        X[r * LX + t] = on && t < r ? G[i][j] * w : 0.0f;
        if (r == t) gv[r] = Hm[i][j];
      }
  }
  __syncthreads();
  // X[i][t] <- sum over j < t (a warp: four rows), then for each t the sum over i >= t
#pragma unroll
  for (int i = warp; i < C; i += TH / 32) {
    float x = X[i * LX + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const float before = __shfl_up_sync(0xffffffffu, x, 1);
    X[i * LX + lane] = lane > 0 ? before : 0.0f;
  }
  __syncthreads();
  if (warp == 0) {
    float x = 0.0f;
    for (int i = lane; i < C; i++) x += X[i * LX + lane];
    pairs[lane] = x;
  }
  ahead_done();  // (the states and adjoints)
  __syncthreads();
  const bool own = ws.dqp == nullptr;  // every head has its own q, k
  const size_t krow = (own ? (size_t)a.qk_unit(u) : (size_t)u) * a.T + t0, vrow = (size_t)u * a.T + t0;
  bool bad = false;
  const float skip = a.skip ? a.skip[h] : 0.0f;
  float aq[RI][DK / 16], ak[RI][DK / 16], cross = 0.0f, dots[RI] = {};
  zero(aq);
  zero(ak);
  // the rows of S and R in one or two parts
#pragma unroll
  for (int p0 = 0; p0 < DV; p0 += PART) {
    const int rows = min(a.dv - p0, PART);
    if (p0 > 0) __syncthreads();
    load_rows<DK, PART, TH>(S, ws.S + at, 0, p0, rows, a.dk);
    __syncthreads();
    mm_nn<TY, PART>(aq, g + p0, LV, S, LK, ty, tx);
    __syncthreads();
#pragma unroll 8
    for (int i = 0; i < PART * DK / 4 / TH; i++) {  // R takes S's place, an element its own
      const int e = tid + i * TH, p = e / (DK / 4), cc = 4 * (e % (DK / 4));
      const float4 r = p < rows && cc < a.dk ? *reinterpret_cast<const float4 *>(ws.R + at + (size_t)(p0 + p) * a.dk + cc) : make_float4(0, 0, 0, 0);
      float4 *s = reinterpret_cast<float4 *>(S + p * LK + cc);
      cross = fmaf(r.x, s->x, fmaf(r.y, s->y, fmaf(r.z, s->z, fmaf(r.w, s->w, cross))));
      *s = r;
    }
    __syncthreads();
    mm_nn<TY, PART>(ak, v + p0, LV, S, LK, ty, tx);
    float acc[RI][PART / 16];
    zero(acc);
    mm_nt<TY, DK>(acc, k, LK, S, LK, ty, tx);
#pragma unroll
    for (int i = 0; i < RI; i++)
#pragma unroll
      for (int j = 0; j < PART / 16; j++) acc[i][j] *= ga.c[ty + TY * i];
    mm_lower_t<TY>(acc, M, LDC, g + p0, LV, ty, tx);
#pragma unroll
    for (int i = 0; i < RI; i++) {
      const int row = ty + TY * i;
#pragma unroll
      for (int j = 0; j < PART / 16; j++) {
        const int p = p0 + tx + 16 * j;
        dots[i] = fmaf(acc[i][j], v[row * LV + p], dots[i]);
        if (row < n && p < a.dv) {
          const float o = ga.step[row] * acc[i][j], y = a.skip ? fmaf(skip, g[row * LV + p], o) : o;
          bad |= !isfinite(y);
          store(a.dv_out, a.dtype == 0, (vrow + row) * a.dv + p, y);
        }
      }
    }
  }
  cross = warp_sum(cross);
  if (lane == 0) across[warp] = cross;
#pragma unroll
  for (int i = 0; i < RI; i++) {
    const int row = ty + TY * i;
    const float f = ga.f[row], w = ga.c[row] * ga.step[row], x = sum16(dots[i]);
    float in = 0.0f, out = 0.0f;
#pragma unroll
    for (int j = 0; j < DK / 16; j++) {
      aq[i][j] = ga.s[row] < 0 ? aq[i][j] * f : 0.0f;
      ak[i][j] *= w;
      in = fmaf(aq[i][j], q[row * LK + tx + 16 * j], in);
      out = fmaf(ak[i][j], k[row * LK + tx + 16 * j], out);
    }
    in = sum16(in);
    out = sum16(out);
    if (tx == 0) duv[row] = x, x_in[row] = in, x_out[row] = out;
  }
  mm_lower<TY>(aq, W, LDC, k, LK, ty, tx);
  mm_lower_t<TY>(ak, W, LDC, q, LK, ty, tx);
#pragma unroll
  for (int i = 0; i < RI; i++)
#pragma unroll
    for (int j = 0; j < DK / 16; j++)
      if (ty + TY * i < n && tx + 16 * j < a.dk) {
        const size_t to = (krow + ty + TY * i) * a.dk + tx + 16 * j;
        bad |= !isfinite(aq[i][j]) || !isfinite(ak[i][j]);
        store(own ? a.dq : ws.dqp, !own || a.dtype == 0, to, aq[i][j]);
        store(own ? a.dk_out : ws.dkp, !own || a.dtype == 0, to, ak[i][j]);
      }
  __syncthreads();
  if (warp == 0) {  // token `lane`
    const int t = lane;
    float in = x_in[t], out = x_out[t], all = 0.0f;
#pragma unroll
    for (int i = 0; i < TH / 32; i++) all += across[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {  // readers from t on, writers up to t
      const float y = __shfl_down_sync(0xffffffffu, in, o), z = __shfl_up_sync(0xffffffffu, out, o);
      if (lane + o < 32) in += y;
      if (lane >= o) out += z;
    }
    out = __shfl_up_sync(0xffffffffu, out, 1);
    if (lane == 0) out = 0.0f;
    const bool start = ga.s[t] == t;
    const float left = ga.s[C - 1] < 0 ? ga.f[C - 1] * all : 0.0f;
    const float da = start ? 0.0f : pairs[t] + in + out + left;
    const float dstep = fmaf(a.A[h], da, duv[t]);
    const float draw = t < n ? dstep * sigmoid(ga.raw[t]) : 0.0f;
    if (t < n) {
      bad |= !isfinite(draw);
      store(a.ddt, a.gates_f32 || a.dtype == 0, vrow + t, draw);
    }
    const float sA = warp_sum(t < n ? ga.step[t] * da : 0.0f), sb = warp_sum(draw), sg = warp_sum(t < n ? gv[t] : 0.0f);
    if (lane == 0) {
      const size_t UN = (size_t)gridDim.y * NC, i = (size_t)u * NC + c;
      ws.sums[i] = sA;
      ws.sums[UN + i] = sb;
      ws.sums[2 * UN + i] = sg;
    }
  }
  if (bad) atomicOr(a.status, tc_err_nonfinite());
}

// grid (H, 3): one parameter's gradient of one head, the sum over its units' chunks in a fixed order.
__global__ void __launch_bounds__(256) mesa_ssm_params_kernel(SsmArgs a, const float *sums, int n) {
  __shared__ float part[8];
  const int h = blockIdx.x, which = blockIdx.y;
  void *dst = which == 0 ? a.dA : which == 1 ? a.dbias : a.dskip;
  ahead_done();
  if (!dst) return;
  const size_t U = (size_t)a.units();
  float x = 0.0f;
#pragma unroll 4
  for (size_t i = threadIdx.x; i < (size_t)a.B * n; i += 256) {
    const size_t b = i / n;
    x += sums[(which * U + b * a.H + h) * n + (i - b * n)];
  }
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x == 0) {
    x = 0.0f;
    for (int i = 0; i < 8; i++) x += part[i];
    store(dst, a.gates_f32 || a.dtype == 0, h, x);
  }
}

template <int DK, int DV>
struct Grads {
  static int run(const SsmArgs &a, const SsmWorkspace &ws, int NC, cudaStream_t st) {
    const size_t smem = sizeof(float) * (2 * C * (DK + 4) + 2 * C * (DV + 4) + kPart<DV> * (DK + 4) + 2 * C * LDC);
    timing_mark_begin(K_SSM_GRADS, st);
    const bool ok = launch(mesa_ssm_grads_kernel<DK, DV>, dim3(NC, a.units()), kGradThreads<DK, DV>, smem, false, st, a, ws);
    timing_mark_end(K_SSM_GRADS, st);
    return ok && cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
  }
};

}  // namespace

int launch_ssm_param_sums(const SsmArgs &a, const float *sums, int n, cudaStream_t st) {
  if (!a.dA && !a.dbias && !a.dskip) return 0;
  timing_mark_begin(K_SSM_PARAMS, st);
  const bool ok = launch_after(mesa_ssm_params_kernel, dim3(a.H, 3), 256, 0, st, a, sums, n);
  timing_mark_end(K_SSM_PARAMS, st);
  return ok && cudaPeekAtLastError() == cudaSuccess ? 0 : -1;
}

int launch_ssm_group_sum(const SsmArgs &a, const float *dqp, const float *dkp, cudaStream_t st) {
  RuleArgs r{a.B, a.H, a.Hk, a.T, a.dk, a.dv, a.dtype};  // the same sum as the delta rule's
  r.dq = a.dq;
  r.dk_out = a.dk_out;
  r.status = a.status;
  return launch_rule_group_sum(r, dqp, dkp, st);
}

int launch_ssm_backward(const SsmArgs &a, SsmWorkspace ws, cudaStream_t st) {
  const int NC = (a.T + C - 1) / C;
  ws.clear = true;
  if (launch_ssm_states(a, ws, true, st) != 0 || by_size<Grads>(a.dk, a.dv, a, ws, NC, st) != 0) return -1;
  if (ws.dqp && launch_ssm_group_sum(a, ws.dqp, ws.dkp, st) != 0) return -1;
  return launch_ssm_param_sums(a, ws.sums, NC, st);
}

}  // namespace mesa
