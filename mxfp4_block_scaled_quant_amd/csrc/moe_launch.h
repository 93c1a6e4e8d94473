// Internal launchers of the routing and experts' kernels.  Arguments are
// already validated by the caller; each returns the HIP launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace mxfp4 {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;

// One moe_route call.
struct RouteArgs {
  const void* logits;  // bf16 or fp32 [tokens, experts], row stride ld elements
  int64_t ld;
  const float* bias;   // [experts] or nullptr
  float* weights;      // [tokens, top_k], row stride ldw
  int64_t ldw;
  int32_t* ids;        // [tokens, top_k], row stride ldi
  int64_t ldi;
  int64_t tokens;
  int experts, top_k;
  int groups, kept, group_top;  // groups == 1: no choice of groups
  int renormalize;
  float scale;
};

hipError_t launch_moe_route(const RouteArgs& p, bool f32, bool sigmoid, hipStream_t stream);

// What a plan found: blocks in its list, 16-row strips in all.
struct MoeHead {
  int blocks, strips;
};

// A run of one expert's rows that one workgroup (or row of tiles) takes:
// `rows` rows from the first of 16-row strip `strip` on.
struct MoeBlock {
  int expert, strip, rows, pad;
};

// One mxfp4_moe call.  A pair is (token t, choice j), number t * top_k + j; it
// counts if its id is in [0, experts).  The pairs of each expert are gathered
// in rows of their own, from a whole 16-row strip on, in the GEMM layouts.
struct MoeArgs {
  const uint16_t* x;  // bf16 [tokens, hidden], row stride ldx elements
  int64_t ldx;
  const int32_t* ids;  // [tokens, top_k]
  int64_t ldi;
  const float* weights;  // [tokens, top_k]
  int64_t ldw;
  const uint8_t *up, *up_scales;  // preshuffled [experts, rows_up, hidden]
  const uint16_t* up_bias;        // bf16 [experts, rows_up] or nullptr
  const uint8_t *down, *down_scales;  // preshuffled [experts, hidden, inner]
  const uint16_t* down_bias;          // bf16 [experts, hidden] or nullptr
  const uint16_t* residual;           // bf16 [tokens, hidden] or nullptr
  int64_t ldr;
  uint16_t* out;  // bf16 [tokens, hidden]
  int64_t ldo;
  int64_t tokens;
  int top_k, experts, hidden, inner, gated, act;
  int cus;
  uint8_t* work;
};

size_t moe_workspace_bytes(int64_t tokens, int64_t top_k, int64_t experts, int64_t hidden, int64_t inner);
hipError_t launch_moe(const MoeArgs& p, hipStream_t stream);

}  // namespace mxfp4
