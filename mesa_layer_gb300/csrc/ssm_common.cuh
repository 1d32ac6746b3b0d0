// ssm_common.cuh -- steps and log-decays of the selective scan, shared by its kernels.
#pragma once

#include "common.cuh"

namespace mesa {
namespace ssm {

constexpr float kLog2e = 1.4426950408889634f;

// softplus and its derivative's argument: log(1 + e^x), for any x (0 at -inf).
__device__ __forceinline__ float softplus(float x) { return fmaxf(x, 0.0f) + log1pf(expf(-fabsf(x))); }
__device__ __forceinline__ float sigmoid(float x) {
  const float e = expf(-fabsf(x));
  return (x >= 0.0f ? 1.0f : e) / (1.0f + e);
}

// A sum of fp32 values kept to twice their precision: hi the rounded sum, lo what that left out.  Differences of
// log-decays far from the chunk's start keep the accuracy of the steps between (|l| reaches hundreds where a head
// forgets within a few tokens; one fp32 sum would then be 2^-17 off).
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_add(Two a, Two b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
  const float h = s + e;
  return {h, e - (h - s)};
}
__device__ __forceinline__ float two_sub(Two a, Two b) { return (a.hi - b.hi) + (a.lo - b.lo); }

// log2 of a token's decay, e^(step A), as a sum of two.  Decays below 2^-150 count as that (they leave nothing in
// fp32), so that differences of sums stay finite; a NaN stays one.
__device__ __forceinline__ Two log2_decay(float step, float A) {
  const float p = step * A, e = fmaf(step, A, -p);
  const float h = p * kLog2e;
  if (h < -150.0f) return {-150.0f, 0.0f};
  return {h, fmaf(p, kLog2e, -h) + fmaf(p, 1.9259629911266175e-8f, e * kLog2e)};  // (log2(e) - kLog2e)
}

}  // namespace ssm
}  // namespace mesa
