// ssm.h -- argument bundle and launchers of the selective state space scan (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mesa {

// One bundle for the sequence forms.  Units u = b H + h; unit u reads the query / key head
// b Hk + h / (H / Hk).
struct SsmArgs {
  int B, H, Hk, T, dk, dv, dtype;
  const void *q, *k, *v;          // [B, Hk, T, dk] x 2, [B, H, T, dv]
  const float *dt;                // [B, H, T]
  const float *A;                 // [H]
  const float *dt_bias, *skip;    // [H] or nullptr
  const uint8_t *starts;          // [B, T] or nullptr
  void *out = nullptr;            // [B, H, T, dv] (forward)
  const float *S0 = nullptr;      // [B, H, dv, dk] or nullptr
  float *S_final = nullptr;
  // backward
  const void *dout = nullptr;     // [B, H, T, dv]
  const float *dS_final = nullptr;
  void *dq = nullptr, *dk_out = nullptr, *dv_out = nullptr, *ddt = nullptr, *dA = nullptr, *dbias = nullptr, *dskip = nullptr;
  bool gates_f32 = false;         // ddt, dA, dbias, dskip in fp32 (else of dtype)
  float *dS0 = nullptr;
  unsigned *status = nullptr;
  unsigned wait_limit = 0;
  __host__ __device__ int units() const { return B * H; }
  __host__ __device__ int qk_unit(int u) const { return (u / H) * Hk + (u % H) / (H / Hk); }
};

// The CUDA-core path works on chunks of kSsmChunk tokens.
constexpr int kSsmChunk = 32;
struct SsmWorkspace {
  float *S = nullptr;      // [U, NC, dv, dk] what each chunk adds, then the states before the chunks
  float *R = nullptr;      // the same of the adjoints (after the chunks)
  float *decay = nullptr;  // [U, NC] what is left of a state after each chunk
  float *sums = nullptr;   // [3][U, NC] what each chunk adds to dA, dbias, dskip
  float *dqp = nullptr, *dkp = nullptr;  // [U, T, dk] per-unit dq, dk (nullptr when every head has its own q, k)
  bool clear = false;      // the states' kernel is the call's first: it clears the status word
};

struct SsmStepArgs {
  int N, H, Hk, dk, dv, dtype;
  float *S;
  const void *q, *k, *v;
  const float *dt, *A, *dt_bias, *skip;
  void *out;
  unsigned *status;  // the device's status word of the decode steps
};

// Each returns 0 when every launch was enqueued, -1 otherwise.
int launch_ssm_forward(const SsmArgs &a, SsmWorkspace ws, cudaStream_t st);
int launch_ssm_backward(const SsmArgs &a, SsmWorkspace ws, cudaStream_t st);
int launch_ssm_step(const SsmStepArgs &a, cudaStream_t st);
// The tensor-core path (bf16, dk = 128 and dv 64 or 128, or both 64).
size_t ssm_tc_workspace(int U, int T, int dv);
int launch_ssm_forward_tc(const SsmArgs &a, void *workspace, cudaStream_t st);
size_t ssm_tc_backward_workspace(int B, int H, int Hk, int T, int dk, int dv);
int launch_ssm_backward_tc(const SsmArgs &a, void *workspace, cudaStream_t st);
// dA, dbias, dskip from n sums a unit, [3][U, n].
int launch_ssm_param_sums(const SsmArgs &a, const float *sums, int n, cudaStream_t st);
// dq, dk [B, Hk, T, dk] = sums of the per-unit fp32 parts over the value heads of a key head.
int launch_ssm_group_sum(const SsmArgs &a, const float *dqp, const float *dkp, cudaStream_t st);

}  // namespace mesa
