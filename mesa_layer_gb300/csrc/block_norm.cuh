// block_norm.cuh -- what the forward and backward block-norm kernels share: vector access,
// the sums over a row's threads, the choice of the kernel instance.
#pragma once

#include "block_norm.h"
#include "common.cuh"
#include "packed.cuh"

namespace mesa {
namespace norm {

constexpr int EPT = 8;  // channels per thread

template <int VEC>
__device__ __forceinline__ void store_vec(float *p, const float *x) {
  if constexpr (VEC == 4)
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
  else if constexpr (VEC == 2)
    *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
  else
    *p = x[0];
}
template <int VEC>
__device__ __forceinline__ void store_vec(__nv_bfloat16 *p, const float *x) {
  if constexpr (VEC == 1) {
    *p = __float2bfloat16_rn(x[0]);
  } else {
    __align__(16) __nv_bfloat162 b[VEC / 2];
#pragma unroll
    for (int i = 0; i < VEC / 2; i++) b[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    if constexpr (VEC == 8) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(b);
    if constexpr (VEC == 4) *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<const uint2 *>(b);
    if constexpr (VEC == 2) *reinterpret_cast<__nv_bfloat162 *>(p) = b[0];
  }
}

// A thread's eight channels as they lie in memory, so that the next row's can be on their way in few
// registers: vector i of VEC elements (the address aligned to it) starts at channel (lane + i G) VEC.
template <typename T, int VEC>
struct Raw {
  static constexpr int kBytes = VEC * (int)sizeof(T), kWords = kBytes >= 4 ? kBytes / 4 : 1;
  uint32_t w[EPT / VEC * kWords];
  template <int G>
  __device__ __forceinline__ void load(const T *row, int lane, int D, bool in) {
#pragma unroll
    for (int i = 0; i < EPT / VEC; i++) {
      const int c = (lane + i * G) * VEC;
      uint32_t *x = w + i * kWords;
#pragma unroll
      for (int k = 0; k < kWords; k++) x[k] = 0;
      if (in && c < D) {
        if constexpr (kBytes == 16) {
          const uint4 v = *reinterpret_cast<const uint4 *>(row + c);
          x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else if constexpr (kBytes == 8) {
          const uint2 v = *reinterpret_cast<const uint2 *>(row + c);
          x[0] = v.x, x[1] = v.y;
        } else if constexpr (kBytes == 4) {
          x[0] = *reinterpret_cast<const uint32_t *>(row + c);
        } else {
          x[0] = *reinterpret_cast<const uint16_t *>(row + c);
        }
      }
    }
  }
  __device__ __forceinline__ void pairs(u64 (&x)[EPT / 2]) const {
    float v[EPT];
    widen(v);
#pragma unroll
    for (int i = 0; i < EPT / 2; i++) x[i] = pack2(v[2 * i], v[2 * i + 1]);
  }
  __device__ __forceinline__ void widen(float (&x)[EPT]) const {
    if constexpr (sizeof(T) == 4 || kBytes == 2) {
#pragma unroll
      for (int i = 0; i < EPT; i++) x[i] = __uint_as_float(sizeof(T) == 4 ? w[i] : w[i] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < EPT / 2; i++) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
};
template <int VEC, int G, typename T>
__device__ __forceinline__ void store_row(T *row, int lane, int D, bool in, const float (&x)[EPT]) {
#pragma unroll
  for (int i = 0; i < EPT / VEC; i++) {
    const int c = (lane + i * G) * VEC;
    if (in && c < D) store_vec<VEC>(row + c, x + i * VEC);
  }
}
template <int VEC, int G, typename T>
__device__ __forceinline__ void store_pairs(T *row, int lane, int D, bool in, const u64 (&x)[EPT / 2]) {
  float v[EPT];
#pragma unroll
  for (int i = 0; i < EPT / 2; i++) unpack2(x[i], v[2 * i], v[2 * i + 1]);
  store_row<VEC, G>(row, lane, D, in, v);
}
// A [D] fp32 vector's channels of this thread (fill where it is not given).
template <int VEC, int G>
__device__ __forceinline__ void load_weights(const float *w, int lane, int D, float fill, float (&x)[EPT]) {
#pragma unroll
  for (int i = 0; i < EPT / VEC; i++)
#pragma unroll
    for (int k = 0; k < VEC; k++) {
      const int c = (lane + i * G) * VEC + k;
      x[i * VEC + k] = w && c < D ? w[c] : fill;
    }
}

// 1 / (1 + e^-g).  For bf16 rows by the approximate exponential and division (each within 2^-20 for
// |g| < 10, far below the outputs' 2^-9): with the exact ones the arithmetic, not memory, set the
// backward's pace.
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 2) return __fdividef(1.0f, 1.0f + __expf(-g));
  return 1.0f / (1.0f + expf(-g));
}

// Sums over a row's G threads, every thread getting them.  Rows wider than a warp go through
// shared memory with one barrier; `buf` alternates, so that a buffer is rewritten only after
// the barrier of the sum in between.
template <int G, int NS>
__device__ __forceinline__ void row_sums(float (&v)[NS], float (*red)[NS][32], int &buf) {
#pragma unroll
  for (int s = 0; s < NS; s++) {
#pragma unroll
    for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) v[s] += __shfl_xor_sync(0xffffffffu, v[s], o);
  }
  if constexpr (G > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
#pragma unroll
      for (int s = 0; s < NS; s++) red[buf][s][warp] = v[s];
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < NS; s++) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < G / 32; w++) t += red[buf][s][threadIdx.x / G * (G / 32) + w];
      v[s] = t;
    }
    buf ^= 1;
  }
}

// Elements of the widest vector that fits every row: D a multiple of it and the [N, D] arrays
// aligned to it (16 bytes at most).
inline int vec_of(int D, int dtype, std::initializer_list<const void *> ptrs) {
  const int esz = dtype == 1 ? 2 : 4;
  int vec = 16 / esz;
  while (vec > 1 && D % vec) vec /= 2;
  for (const void *p : ptrs)
    while (vec > 1 && ((uintptr_t)p % (vec * esz))) vec /= 2;
  return vec;
}

// L::run<T, VEC, G>(a, grid-independent arguments) for the call's type, vector and row width.
template <template <typename, int, int> class L, typename T, int VEC>
int dispatch_group(const NormArgs &a, cudaStream_t st) {
  switch (norm_group(a.D)) {
    case 8: return L<T, VEC, 8>::run(a, st);
    case 16: return L<T, VEC, 16>::run(a, st);
    case 32: return L<T, VEC, 32>::run(a, st);
    case 64: return L<T, VEC, 64>::run(a, st);
    case 128: return L<T, VEC, 128>::run(a, st);
    case 256: return L<T, VEC, 256>::run(a, st);
    case 512: return L<T, VEC, 512>::run(a, st);
    case 1024: return L<T, VEC, 1024>::run(a, st);
  }
  return -1;
}
template <template <typename, int, int> class L>
int dispatch(const NormArgs &a, int vec, cudaStream_t st) {
  if (a.dtype == 1) {
    switch (vec) {
      case 8: return dispatch_group<L, __nv_bfloat16, 8>(a, st);
      case 4: return dispatch_group<L, __nv_bfloat16, 4>(a, st);
      case 2: return dispatch_group<L, __nv_bfloat16, 2>(a, st);
      default: return dispatch_group<L, __nv_bfloat16, 1>(a, st);
    }
  }
  switch (vec) {
    case 4: return dispatch_group<L, float, 4>(a, st);
    case 2: return dispatch_group<L, float, 2>(a, st);
    default: return dispatch_group<L, float, 1>(a, st);
  }
}

}  // namespace norm
}  // namespace mesa
