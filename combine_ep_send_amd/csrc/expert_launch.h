// Launchers of the expert-side calls (include/epdc_expert.h), after the C-ABI
// layer has validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "expert_rules.h"

namespace epdc {

constexpr int kFewSlots = 1024;    // slots (token, k) or rows of one call
constexpr int kFewExperts = 1024;

// One kind of weights of the few-row products.
// kWBf16Stream: bf16 read with the non-temporal hint, chosen at the launch.
enum WeightKind : int {
  kWBf16 = 0, kWFp4 = 1, kWInt4G32 = 2, kWInt4G64 = 3, kWInt4G128 = 4, kWBf16Stream = 5
};

struct Weights {
  WeightKind kind;
  const void* q;
  const void* scale;
};

// What a layer's first launch finds out about the routing, for its second:
// the experts in use in ascending order, and the slots sorted by expert.
struct FewPlan {
  int32_t active;
  int32_t pad[63];
  int32_t expert[kFewExperts];
  int32_t first[kFewExperts];      // index into order of the expert's first slot
  int32_t count[kFewExperts];
  int32_t order[kFewSlots];
};

struct FewArgs {
  // rows: slot s reads row s / top of x; its expert is ids64[s] - first_expert
  // (a layer), ids32[s] (rows), or 0 when both are null
  const void* x;
  const int64_t* ids64;
  const int32_t* ids32;
  int64_t first_expert;
  int slots;                       // 1..kFewSlots
  int top;                         // slots per row of x
  int rows;                        // rows of x
  int per_token;                   // rows of x a token has (a layer's second launch: K)
  int experts;
  int N;                           // output channels (a layer's first launch: I of the 2I rows)
  int K;                           // input channels
  Weights w;                       // [experts, N (first launch: 2N), K]
  void* y;                         // [slots, N] bf16 (a layer's first launch: [slots, 2, N],
                                   // the two bf16 parts of h)
  FewPlan* plan;                   // written by a layer's first launch
};
hipError_t launch_few_rows(const FewArgs& a, bool gated, hipStream_t s);

struct DownArgs {
  const FewPlan* plan;
  const void* h;                   // [slots, 2, I] bf16, the two parts of h
  Weights w;                       // [experts, H, I]
  int experts;
  const int64_t* ids64;
  int64_t first_expert;
  const float* topk_weights;
  int T, K, H, I;
  const void* bias0;
  const void* bias1;
  void* out;
  float* y;                        // [slots, H], where the sum is a launch of its own
};
// The products go through y in the workspace unless few_down_joined.
hipError_t launch_few_down(const DownArgs& a, hipStream_t s);

struct QuantArgs {
  const void* w;
  int64_t rows;
  int channels;
  bool fp4;
  int group;
  void* q;
  void* scale;
};
hipError_t launch_quantize_w4(const QuantArgs& a, hipStream_t s);

struct SwigluArgs {
  const void* gate_up;             // forward: bf16 in; backward: null
  const void* dh;                  // backward
  int64_t rows;
  int inner;
  const int32_t* row_count;        // or null
  void* h;
  void* q;                         // forward: out; backward: in
  float* scale;
  void* d_gate_up;
};
hipError_t launch_swiglu_fp8(const SwigluArgs& a, hipStream_t s);
hipError_t launch_swiglu_fp8_backward(const SwigluArgs& a, hipStream_t s);

struct CombineBackwardArgs {
  const void* dout;
  const void* y;
  int64_t R;
  const int32_t* token_row;
  const float* w;                  // or null: unweighted
  int64_t T;
  int K;
  int H;
  void* dy;
  float* dw;                       // or null
};
hipError_t launch_combine_backward(const CombineBackwardArgs& a, hipStream_t s);

}  // namespace epdc
