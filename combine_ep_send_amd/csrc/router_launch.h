// Launchers of the calls before the dispatch (include/epdc_router.h), after the
// C-ABI layer has validated every argument.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "router_rules.h"

namespace epdc {

struct NormArgs {
  const void* x;                   // backward: s
  const void* residual;            // or null; backward: d_residual
  const void* weight;              // [H] bf16, or fp32 with w32
  bool w32;
  int64_t T;
  int H;
  float eps;
  void* residual_out;              // or null
  void* out;                       // or null; backward: dx
  void* q;                         // or null
  float* scale;
  bool pow2;
  float* rstd;                     // or null; backward: in
  const void* dy;                  // backward
  float* dweight;                  // backward, or null
  float* part;                     // backward: [norm_groups, H] fp32
};
hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s);
hipError_t launch_rms_norm_backward(const NormArgs& a, hipStream_t s);

struct RouteArgs {
  const float* logits;
  int64_t T;
  int E;
  int K;
  bool sigmoid;
  const float* bias;               // or null
  int groups;                      // 1 where all groups stay
  int kept;
  int group_top;
  bool renorm;
  float scale;
  const int32_t* token_count;      // or null
  int64_t* topk_idx;               // backward: in
  float* topk_weights;
  const float* dweights;           // backward
  float* dlogits;                  // backward
};
hipError_t launch_route(const RouteArgs& a, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s);

struct LogitsArgs {
  const void* x;                   // [T, H] bf16
  const void* w;                   // [E, H] bf16
  int64_t T;
  int E;
  int H;
  float* logits;
  void* ws;
  const float* dlogits;            // backward
  void* dx;                        // or null
  float* dw;                       // or null
};
hipError_t launch_router_logits(const LogitsArgs& a, hipStream_t s);
hipError_t launch_router_logits_backward(const LogitsArgs& a, hipStream_t s);

}  // namespace epdc
