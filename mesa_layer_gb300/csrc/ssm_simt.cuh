// ssm_simt.cuh -- what the CUDA-core kernels of the selective scan share: the gates of a chunk of 32 tokens, rows in
// shared memory as fp32, and small products by 16 x 16 threads.
#pragma once

#include "overlap.cuh"
#include "ssm.h"
#include "ssm_common.cuh"

namespace mesa {
namespace ssm {

constexpr int C = kSsmChunk;  // a warp's lanes: one token each
constexpr int kThreads = 256, kFew = 128;  // of the states' kernel; of those whose threads take four rows each
constexpr int LDC = C + 4;    // row stride of a [C x C] matrix

struct Gates {
  float step[C], hi[C], lo[C];  // lengths of the steps; log2 decay from the chunk's start
  int s[C];                     // the last start up to a token, -1: none in the chunk
  float f[C], c[C];             // decay from before the chunk to a token, from a token to the chunk's end
  float raw[C];
  __device__ __forceinline__ float decay(int i, int j) const {  // from token j to token i >= j
    return j <= i && j >= s[i] ? exp2f((hi[i] - hi[j]) + (lo[i] - lo[j])) : 0.0f;
  }
};

// By one warp: the gates of tokens t0 .. t0 + n - 1 of unit u (the others do nothing).
__device__ __forceinline__ void gates_load(Gates &g, const SsmArgs &a, int u, int t0, int n, int lane) {
  const int h = u % a.H, b = u / a.H;
  const bool in = lane < n;
  const float raw = in ? a.dt[(size_t)u * a.T + t0 + lane] + (a.dt_bias ? a.dt_bias[h] : 0.0f) : 0.0f;
  const float step = in ? softplus(raw) : 0.0f;
  const bool start = in && a.starts && a.starts[(size_t)b * a.T + t0 + lane];
  Two l = start ? Two{0.0f, 0.0f} : log2_decay(step, a.A[h]);
  int s = start ? lane : -1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Two p = {__shfl_up_sync(0xffffffffu, l.hi, o), __shfl_up_sync(0xffffffffu, l.lo, o)};
    const int ps = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) {
      l = two_add(p, l);
      s = max(s, ps);
    }
  }
  const Two end = {__shfl_sync(0xffffffffu, l.hi, 31), __shfl_sync(0xffffffffu, l.lo, 31)};
  const int send = __shfl_sync(0xffffffffu, s, 31);
  g.step[lane] = step;
  g.hi[lane] = l.hi;
  g.lo[lane] = l.lo;
  g.s[lane] = s;
  g.raw[lane] = raw;
  g.f[lane] = s < 0 ? exp2f(l.hi + l.lo) : 0.0f;
  g.c[lane] = lane >= send ? exp2f(two_sub(end, l)) : 0.0f;
}

// n rows of d channels (fp32 or bf16) to fp32 rows of D channels, stride D + 4, what is missing as zeros.  Eight loads of a
// thread are in flight together (one after the other, they were most of the time: 543 us of a 2 x 16 x 4096 x 128 fp32
// forward's outputs, so 345).
template <int D, int ROWS, int TH = kFew>
__device__ __forceinline__ void load_rows(float *dst, const void *src, int dtype, size_t first, int n, int d) {
  constexpr int PER = ROWS * (D / 4) / TH, BATCH = PER < 8 ? PER : 8;
  static_assert(PER % BATCH == 0 && PER * TH == ROWS * (D / 4), "whole batches");
  const bool bf16 = dtype == 1;
#pragma unroll
  for (int i0 = 0; i0 < PER; i0 += BATCH) {
    uint4 x[BATCH];
#pragma unroll
    for (int j = 0; j < BATCH; j++) {
      const int i = threadIdx.x + (i0 + j) * TH, r = i / (D / 4), c = 4 * (i % (D / 4));
      const size_t at = (first + r) * d + c;
      x[j] = make_uint4(0, 0, 0, 0);
      if (r < n && c < d) {
        if (bf16) {
          const uint2 y = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(src) + at);
          x[j].x = y.x, x[j].y = y.y;
        } else {
          x[j] = *reinterpret_cast<const uint4 *>(static_cast<const float *>(src) + at);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < BATCH; j++) {
      const int i = threadIdx.x + (i0 + j) * TH, r = i / (D / 4), c = 4 * (i % (D / 4));
      if (bf16) x[j] = make_uint4(x[j].x << 16, x[j].x & 0xffff0000u, x[j].y << 16, x[j].y & 0xffff0000u);
      *reinterpret_cast<uint4 *>(dst + r * (D + 4) + c) = x[j];
    }
  }
}
__device__ __forceinline__ void store(void *p, bool f32, size_t i, float x) {
  if (f32)
    static_cast<float *>(p)[i] = x;
  else
    static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
}

// Products by TY x 16 threads (ty, tx): this thread's rows ty + TY i, columns tx + 16 j.  A 16-byte load of a warp takes
// four turns of shared memory whatever its lanes share: with two rows a thread the loads take 2.5 times as long as the
// products, with four rows (TY = 8) 1.5 times.
// acc += A B^T, A [.][K], B [.][K] (row strides lda, ldb); with J0, COLS the columns' share acc[.][J0 ..] of COLS alone.
template <int TY, int K, int J0 = 0, int COLS = 0, int RI, int CJ>
__device__ __forceinline__ void mm_nt(float (&acc)[RI][CJ], const float *A, int lda, const float *B, int ldb, int ty, int tx) {
#pragma unroll 4
  for (int k = 0; k < K; k += 4) {
    float4 x[RI];
#pragma unroll
    for (int i = 0; i < RI; i++) x[i] = *reinterpret_cast<const float4 *>(A + (ty + TY * i) * lda + k);
#pragma unroll
    for (int j = J0; j < (COLS ? J0 + COLS : CJ); j++) {
      const float4 y = *reinterpret_cast<const float4 *>(B + (tx + 16 * (j - J0)) * ldb + k);
#pragma unroll
      for (int i = 0; i < RI; i++)
        acc[i][j] = fmaf(x[i].w, y.w, fmaf(x[i].z, y.z, fmaf(x[i].y, y.y, fmaf(x[i].x, y.x, acc[i][j]))));
    }
  }
}
// acc += A B, A [.][K], B [K][.].
template <int TY, int K, int RI, int CJ>
__device__ __forceinline__ void mm_nn(float (&acc)[RI][CJ], const float *A, int lda, const float *B, int ldb, int ty, int tx) {
#pragma unroll 2
  for (int k = 0; k < K; k += 4) {
    float4 x[RI];
#pragma unroll
    for (int i = 0; i < RI; i++) x[i] = *reinterpret_cast<const float4 *>(A + (ty + TY * i) * lda + k);
#pragma unroll
    for (int e = 0; e < 4; e++)
#pragma unroll
      for (int j = 0; j < CJ; j++) {
        const float y = B[(k + e) * ldb + tx + 16 * j];
#pragma unroll
        for (int i = 0; i < RI; i++) acc[i][j] = fmaf(e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w, y, acc[i][j]);
      }
  }
}
// acc += A B of the chunk's tokens, A [C][C] lower triangular: row r takes B's rows up to r alone.  What is not finite in a later
// token's row stays out of it, and 6 of 16 blocks of products are left out (as a loop over all of A with a test: 1 % slower).
template <int TY, int RI, int CJ>
__device__ __forceinline__ void mm_lower(float (&acc)[RI][CJ], const float *A, int lda, const float *B, int ldb, int ty, int tx) {
  static_assert(TY * RI == C, "all rows of the chunk");
#pragma unroll
  for (int b = 0; b < RI; b++)
#pragma unroll
    for (int k = 0; k < TY; k += 4) {
      float4 x[RI];
#pragma unroll
      for (int i = b; i < RI; i++) x[i] = *reinterpret_cast<const float4 *>(A + (ty + TY * i) * lda + TY * b + k);
#pragma unroll
      for (int e = 0; e < 4; e++)
#pragma unroll
        for (int j = 0; j < CJ; j++) {
          const float y = B[(TY * b + k + e) * ldb + tx + 16 * j];
#pragma unroll
          for (int i = b; i < RI; i++)
            acc[i][j] = fmaf(e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w, i > b || k + e <= ty ? y : 0.0f, acc[i][j]);
        }
    }
}
// acc += A^T B, A as above: row r takes B's rows from r on alone.  (In blocks as above the gradients take 2 to 10 % longer.)
template <int TY, int RI, int CJ>
__device__ __forceinline__ void mm_lower_t(float (&acc)[RI][CJ], const float *A, int lda, const float *B, int ldb, int ty, int tx) {
  static_assert(TY * RI == C, "all rows of the chunk");
#pragma unroll 4
  for (int k = 0; k < C; k++) {
    float x[RI], y[CJ];
#pragma unroll
    for (int i = 0; i < RI; i++) x[i] = A[k * lda + ty + TY * i];
#pragma unroll
    for (int j = 0; j < CJ; j++) y[j] = B[k * ldb + tx + 16 * j];
#pragma unroll
    for (int i = 0; i < RI; i++)
#pragma unroll
      for (int j = 0; j < CJ; j++)
        if (k >= ty + TY * i) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
  }
}
// acc += A^T B by 16 x 16 threads, where both rows' elements lie side by side: this thread's rows and columns frag<M>(ty, i), frag<N>(tx, j), in
// groups of four from 64 on (a quarter of the shared-memory instructions).
template <int D>
__device__ __forceinline__ int frag(int t, int i) {
  return D >= 64 ? 64 * (i / 4) + 4 * t + i % 4 : t + 16 * i;
}
template <int D>
__device__ __forceinline__ void load_frag(const float *row, int t, float (&x)[D / 16]) {
  if constexpr (D >= 64) {
#pragma unroll
    for (int g = 0; g < D / 64; g++) {
      const float4 y = *reinterpret_cast<const float4 *>(row + 64 * g + 4 * t);
      x[4 * g] = y.x, x[4 * g + 1] = y.y, x[4 * g + 2] = y.z, x[4 * g + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < D / 16; i++) x[i] = row[t + 16 * i];
  }
}
template <int K, int M, int N>
__device__ __forceinline__ void mm_outer(float (&acc)[M / 16][N / 16], const float *A, int lda, const float *B, int ldb, int ty, int tx) {
#pragma unroll 2
  for (int k = 0; k < K; k++) {
    float x[M / 16], y[N / 16];
    load_frag<M>(A + k * lda, ty, x);
    load_frag<N>(B + k * ldb, tx, y);
#pragma unroll
    for (int i = 0; i < M / 16; i++)
#pragma unroll
      for (int j = 0; j < N / 16; j++) acc[i][j] = fmaf(x[i], y[j], acc[i][j]);
  }
}
template <int RI, int CJ>
__device__ __forceinline__ void zero(float (&acc)[RI][CJ]) {
#pragma unroll
  for (int i = 0; i < RI; i++)
#pragma unroll
    for (int j = 0; j < CJ; j++) acc[i][j] = 0.0f;
}

// Rows of a state that are in shared memory at a time: two CTAs of the largest size fit an SM then.
template <int DV>
constexpr int kPart = DV > 64 ? 64 : DV;

// Sizes are padded to 32, 64 or 128 channels in shared memory (16 to 32).
template <template <int, int> class F, typename... Args>
int by_size(int dk, int dv, Args &&...args) {
  auto k = [&](auto dkc) {
    constexpr int DK = decltype(dkc)::value;
    if (dv <= 32) return F<DK, 32>::run(args...);
    if (dv == 64) return F<DK, 64>::run(args...);
    return F<DK, 128>::run(args...);
  };
  if (dk <= 32) return k(std::integral_constant<int, 32>());
  if (dk == 64) return k(std::integral_constant<int, 64>());
  return k(std::integral_constant<int, 128>());
}

// Launch, the call's first kernel or not, with `smem` bytes of dynamic shared memory (48 KB without being asked for, the static part among them).
template <typename K, typename... Args>
bool launch(K kernel, dim3 grid, int threads, size_t smem, bool first, cudaStream_t st, const Args &...args) {
  if (smem > 32 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return false;
  if (!first) return launch_after(kernel, grid, threads, smem, st, args...);
  kernel<<<grid, threads, smem, st>>>(args...);
  return true;
}

}  // namespace ssm
}  // namespace mesa
