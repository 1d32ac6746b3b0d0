// gated_delta.h -- argument bundle and launchers of the gated delta rule (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mesa {

// One bundle for the sequence forms.  Units u = b H + h; unit u reads the query / key head
// b Hk + h / (H / Hk).
struct RuleArgs {
  int B, H, Hk, T, dk, dv, dtype;
  const void *q, *k, *v;               // [B, Hk, T, dk] x 2, [B, H, T, dv]
  const float *gamma, *beta;           // [B, H, T]
  float scale;
  void *out = nullptr;                 // [B, H, T, dv] (forward)
  const float *S0 = nullptr;           // [B, H, dv, dk] or nullptr
  float *S_final = nullptr;
  // backward
  const void *dout = nullptr;          // [B, H, T, dv]
  const float *dS_final = nullptr;     // [B, H, dv, dk] or nullptr
  void *dq = nullptr, *dk_out = nullptr, *dv_out = nullptr, *dgamma = nullptr, *dbeta = nullptr;
  bool gates_f32 = false;              // dgamma, dbeta [B, H, T] in fp32 (else of dtype)
  float *dS0 = nullptr;
  unsigned *status = nullptr;
  unsigned wait_limit = 0;
  __host__ __device__ int units() const { return B * H; }
  __host__ __device__ int qk_unit(int u) const { return (u / H) * Hk + (u % H) / (H / Hk); }
};

// A gate's gradient, in fp32 or in the call's type TIO.
template <typename TIO>
__device__ __forceinline__ void st_gate(const RuleArgs &a, void *p, size_t i, float x) {
  if (a.gates_f32)
    static_cast<float *>(p)[i] = x;
  else
    static_cast<TIO *>(p)[i] = TIO(x);
}

// CUDA-core path: chunks of kRuleChunk tokens in the backward pass.
constexpr int kRuleChunk = 32;
struct RuleBwdWorkspace {
  float *S, *dS;       // [U, NC, dv, dk] states before / adjoints after each chunk
  float *e, *du;       // [U, T, dv]
  float *dqp, *dkp;    // [U, T, dk] per-unit dq, dk (nullptr when every head has its own q, k)
};

// Few units: n segments of `per` blocks of tokens that run side by side (one: nothing is used).
struct RuleScanSegments {
  int n = 1, per = 0;
  float *S = nullptr, *loc = nullptr;   // [U, n][dv, dk] the state before a segment; what it leaves from zero
  float *A = nullptr, *adj = nullptr;   // [U, n][dv, dk] the adjoint after a segment; what it gives from zero
  float *Tr = nullptr, *TrT = nullptr;  // [U, n][dk, dk] the matrix from the state before to the state after
};

struct RuleStepArgs {
  int N, H, Hk, dk, dv, dtype;
  float *S;
  const void *q, *k, *v;
  const float *gamma, *beta;
  float scale;
  void *out;
  unsigned *status;  // the device's status word of the decode steps
};

// Each returns 0 when every launch was enqueued, -1 otherwise.
size_t rule_scan_workspace(int U, int T, int dk, int dv, bool backward);
RuleScanSegments rule_scan_parts(int U, int T, int dk, int dv, bool backward, void *workspace);
int launch_rule_forward(const RuleArgs &a, const RuleScanSegments &sg, cudaStream_t st);
int launch_rule_backward(const RuleArgs &a, const RuleBwdWorkspace &ws, const RuleScanSegments &sg, cudaStream_t st);
int launch_rule_step(const RuleStepArgs &a, cudaStream_t st);
// The tensor-core path (bf16, dk = dv = 128): workspace bytes, the chunks' records (with_beta: the
// forward's), the forward.
// What the two chains of the backward pass keep, as fp16 operands of 64-token chunks, each with 1 /
// its scale: states (or their adjoints) S [U, NC][128 x 128] and u (or du) U [U, NC][64 x 128].
struct RuleOperands {
  uint8_t *S = nullptr, *U = nullptr;
  float *iS = nullptr, *iU = nullptr;
};
// Segments of long sequences with few units: n segments of `per` chunks.
struct RuleSegments {
  int n = 1, per = 0;
  float2 *bounds = nullptr;  // [U, NC] log2 of what a chunk leaves of a state; what it adds to a row (bounds)
  float *S = nullptr, *loc = nullptr, *Tr = nullptr;  // [U, n][128 x 128] the state before; what it leaves
  int *whole = nullptr;  // [U, n] whether what went before counts (Tr is there and to be applied)
  // the backward's: what a chunk adds to a row of the adjoint (bounds), the adjoints after the segments, what
  // they give from zero, whether what comes after counts
  float *adds = nullptr, *A = nullptr, *adj = nullptr;
  int *whole_adj = nullptr;
};
size_t rule_tc_workspace(int U, int T, bool backward);
RuleSegments rule_tc_segments(int U, int T, bool backward, void *workspace);
int launch_rule_prep(const RuleArgs &a, void *records, const RuleSegments &sg, bool with_beta, cudaStream_t st);
int launch_rule_forward_tc(const RuleArgs &a, void *workspace, cudaStream_t st);
// The backward on the tensor cores, from the records (without beta): the states and u before the
// adjoint chain, the adjoint chain, the gradients.
int launch_rule_states_tc(const RuleArgs &a, const void *records, const RuleSegments &sg, const RuleOperands &so,
                          cudaStream_t st);
int launch_rule_adjoint_tails(const RuleArgs &a, const void *records, const RuleSegments &sg, cudaStream_t st);  // (first)
int launch_rule_adjoint_tc(const RuleArgs &a, const void *records, const RuleSegments &sg, const RuleOperands &ao,
                           cudaStream_t st);
int launch_rule_grads_tc(const RuleArgs &a, const void *records, const RuleOperands &so, const RuleOperands &ao,
                         float *dqp, float *dkp, cudaStream_t st);
// dq, dk [B, Hk, T, dk] = sums of the per-unit fp32 parts over the value heads of a key head.
int launch_rule_group_sum(const RuleArgs &a, const float *dqp, const float *dkp, cudaStream_t st);

}  // namespace mesa
