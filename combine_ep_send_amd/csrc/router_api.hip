// C ABI of the calls before the dispatch (include/epdc_router.h): argument
// validation on the host, then launches.  Nothing here allocates, frees or
// synchronizes.
#include <math.h>
#include <stdint.h>

#include "../../include/epdc_router.h"
#include "epdc_launch.h"
#include "router_launch.h"

namespace {

using namespace epdc;

constexpr int64_t kMaxRows = int64_t(1) << 30;

static_assert(kRouterChannels == EPDC_ROUTER_CHANNELS && kNormChannels == EPDC_NORM_CHANNELS,
              "limits");

bool is_aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}
bool array_ok(const void* p, int64_t count, uintptr_t a) {
  return count == 0 || (p != nullptr && is_aligned(p, a));
}
bool maybe_ok(const void* p, uintptr_t a) { return p == nullptr || is_aligned(p, a); }
int launched(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_LAUNCH; }

int check_tokens(int64_t tokens, int hidden, int most) {
  if (tokens < 0 || hidden <= 0 || hidden % 8 != 0) return EP_ERR_INVALID_ARG;
  if (tokens >= kMaxRows || hidden > most) return EP_ERR_UNSUPPORTED;
  return EP_OK;
}

int check_logits(int64_t tokens, int experts, int hidden) {
  const int st = check_tokens(tokens, hidden, EPDC_ROUTER_CHANNELS);
  if (st != EP_OK) return st;
  return experts < 1 ? EP_ERR_INVALID_ARG : experts > EPDC_MAX_BINS ? EP_ERR_UNSUPPORTED : EP_OK;
}

int check_route(int64_t tokens, int experts, int topk, int score, float scale) {
  if (tokens < 0 || experts < 1 || topk < 1 || !isfinite(scale)) return EP_ERR_INVALID_ARG;
  if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID) return EP_ERR_INVALID_ARG;
  if (tokens >= kMaxRows || experts > EPDC_MAX_BINS || topk > EPDC_MAX_TOPK)
    return EP_ERR_UNSUPPORTED;
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_router_abi_version(void) { return EPDC_ROUTER_ABI_VERSION; }

int ep_rms_norm(const void* x, const void* residual, const void* weight, int weight_type,
                int64_t num_tokens, int hidden, float eps, void* residual_out, void* out, void* q,
                float* scale, int scale_fmt, float* rstd, hipStream_t stream) {
  const int st = check_tokens(num_tokens, hidden, EPDC_NORM_CHANNELS);
  if (st != EP_OK) return st;
  if (weight_type != EP_NORM_W_BF16 && weight_type != EP_NORM_W_F32) return EP_ERR_INVALID_ARG;
  if (scale_fmt != EP_SCALE_F32 && scale_fmt != EP_SCALE_POW2) return EP_ERR_INVALID_ARG;
  if (!isfinite(eps) || eps < 0.0f) return EP_ERR_INVALID_ARG;
  if (!array_ok(weight, 1, 16)) return EP_ERR_INVALID_ARG;
  if (!array_ok(x, num_tokens, 16) || !maybe_ok(residual, 16) || !maybe_ok(residual_out, 16) ||
      !maybe_ok(out, 16) || !maybe_ok(q, 16) || !maybe_ok(scale, 4) || !maybe_ok(rstd, 4))
    return EP_ERR_INVALID_ARG;
  if (q && hidden % EPDC_FP8_GROUP != 0) return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  if (!residual != !residual_out || (!out && !q) || !q != !scale) return EP_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.w32 = weight_type == EP_NORM_W_F32;
  a.T = num_tokens;
  a.H = hidden;
  a.eps = eps;
  a.residual_out = residual_out;
  a.out = out;
  a.q = q;
  a.scale = scale;
  a.pow2 = scale_fmt == EP_SCALE_POW2;
  a.rstd = rstd;
  return launched(launch_rms_norm(a, stream));
}

size_t ep_rms_norm_backward_workspace_bytes(int64_t num_tokens, int hidden) {
  if (check_tokens(num_tokens, hidden, EPDC_NORM_CHANNELS) != EP_OK) return 0;
  // one row even for no tokens, so that 0 says refused
  return size_t(num_tokens ? norm_groups(num_tokens, hidden) : 1) * size_t(hidden) * 4;
}

int ep_rms_norm_backward(const void* dy, const void* s, const void* weight, int weight_type,
                         const float* rstd, const void* d_residual, int64_t num_tokens, int hidden,
                         void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  const int st = check_tokens(num_tokens, hidden, EPDC_NORM_CHANNELS);
  if (st != EP_OK) return st;
  if (weight_type != EP_NORM_W_BF16 && weight_type != EP_NORM_W_F32) return EP_ERR_INVALID_ARG;
  if (!array_ok(weight, 1, 16)) return EP_ERR_INVALID_ARG;
  if (!array_ok(dy, num_tokens, 16) || !array_ok(s, num_tokens, 16) ||
      !array_ok(rstd, num_tokens, 4) || !maybe_ok(d_residual, 16) ||
      !array_ok(dx, num_tokens, 16) || !maybe_ok(dweight, 4))
    return EP_ERR_INVALID_ARG;
  if (dweight && (!workspace || !is_aligned(workspace, 256) ||
                  workspace_bytes < ep_rms_norm_backward_workspace_bytes(num_tokens, hidden)))
    return EP_ERR_WORKSPACE;
  if (num_tokens == 0 && !dweight) return EP_OK;
  NormArgs a{};
  a.dy = dy;
  a.x = s;
  a.weight = weight;
  a.w32 = weight_type == EP_NORM_W_F32;
  a.rstd = const_cast<float*>(rstd);
  a.residual = d_residual;
  a.T = num_tokens;
  a.H = hidden;
  a.out = dx;
  a.dweight = dweight;
  a.part = static_cast<float*>(workspace);
  return launched(launch_rms_norm_backward(a, stream));
}

size_t ep_router_logits_workspace_bytes(int64_t num_tokens, int num_experts, int hidden) {
  if (check_logits(num_tokens, num_experts, hidden) != EP_OK) return 0;
  return logits_ws_bytes(num_tokens, num_experts, hidden);
}

int ep_router_logits(const void* x, const void* w, int64_t num_tokens, int num_experts, int hidden,
                     float* logits, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int st = check_logits(num_tokens, num_experts, hidden);
  if (st != EP_OK) return st;
  if (!array_ok(w, 1, 16) || !array_ok(x, num_tokens, 16) || !array_ok(logits, num_tokens, 4))
    return EP_ERR_INVALID_ARG;
  if (!workspace || !is_aligned(workspace, 256) ||
      workspace_bytes < logits_ws_bytes(num_tokens, num_experts, hidden))
    return EP_ERR_WORKSPACE;
  if (num_tokens == 0) return EP_OK;
  LogitsArgs a{};
  a.x = x;
  a.w = w;
  a.T = num_tokens;
  a.E = num_experts;
  a.H = hidden;
  a.logits = logits;
  a.ws = workspace;
  return launched(launch_router_logits(a, stream));
}

size_t ep_router_logits_backward_workspace_bytes(int64_t num_tokens, int num_experts,
                                                 int hidden) {
  if (check_logits(num_tokens, num_experts, hidden) != EP_OK) return 0;
  return logits_backward_space(num_tokens, num_experts, hidden).total;
}

int ep_router_logits_backward(const float* dlogits, const void* x, const void* w,
                              int64_t num_tokens, int num_experts, int hidden, void* dx, float* dw,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const int st = check_logits(num_tokens, num_experts, hidden);
  if (st != EP_OK) return st;
  if (!array_ok(dlogits, num_tokens, 4) || !maybe_ok(x, 16) || !maybe_ok(w, 16) ||
      !maybe_ok(dx, 16) || !maybe_ok(dw, 16) || (dx && !w) || (dw && !x && num_tokens > 0))
    return EP_ERR_INVALID_ARG;
  if (num_tokens > 0 && !dx && !dw) return EP_ERR_INVALID_ARG;
  if (!workspace || !is_aligned(workspace, 256) ||
      workspace_bytes < logits_backward_space(num_tokens, num_experts, hidden).total)
    return EP_ERR_WORKSPACE;
  if (num_tokens == 0 && !dw) return EP_OK;
  LogitsArgs a{};
  a.dlogits = dlogits;
  a.x = x;
  a.w = w;
  a.T = num_tokens;
  a.E = num_experts;
  a.H = hidden;
  a.dx = num_tokens ? dx : nullptr;
  a.dw = dw;
  a.ws = workspace;
  return launched(launch_router_logits_backward(a, stream));
}

int ep_route(const float* logits, int64_t num_tokens, int num_experts, int num_topk, int score,
             const float* bias, int num_groups, int topk_groups, int group_top, int renormalize,
             float scale, const int32_t* token_count, int64_t* topk_idx, float* topk_weights,
             hipStream_t stream) {
  const int st = check_route(num_tokens, num_experts, num_topk, score, scale);
  if (st != EP_OK) return st;
  if (num_groups < 1 || topk_groups < 1 || topk_groups > num_groups || group_top < 1 ||
      group_top > 2 || num_experts % num_groups != 0)
    return EP_ERR_INVALID_ARG;
  if (num_groups > EPDC_MAX_GROUPS) return EP_ERR_UNSUPPORTED;
  if (!array_ok(logits, num_tokens, 4) || !maybe_ok(bias, 4) || !maybe_ok(token_count, 4) ||
      !array_ok(topk_idx, num_tokens, 8) || !array_ok(topk_weights, num_tokens, 4))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  RouteArgs a{};
  a.logits = logits;
  a.T = num_tokens;
  a.E = num_experts;
  a.K = num_topk;
  a.sigmoid = score == EP_SCORE_SIGMOID;
  a.bias = bias;
  a.groups = topk_groups == num_groups ? 1 : num_groups;
  a.kept = topk_groups;
  a.group_top = group_top;
  a.renorm = renormalize != 0;
  a.scale = scale;
  a.token_count = token_count;
  a.topk_idx = topk_idx;
  a.topk_weights = topk_weights;
  return launched(launch_route(a, stream));
}

int ep_route_backward(const float* dweights, const float* logits, const int64_t* topk_idx,
                      int64_t num_tokens, int num_experts, int num_topk, int score,
                      int renormalize, float scale, float* dlogits, hipStream_t stream) {
  const int st = check_route(num_tokens, num_experts, num_topk, score, scale);
  if (st != EP_OK) return st;
  if (!array_ok(dweights, num_tokens, 4) || !array_ok(logits, num_tokens, 4) ||
      !array_ok(topk_idx, num_tokens, 8) || !array_ok(dlogits, num_tokens, 4))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  RouteArgs a{};
  a.dweights = dweights;
  a.logits = logits;
  a.topk_idx = const_cast<int64_t*>(topk_idx);
  a.T = num_tokens;
  a.E = num_experts;
  a.K = num_topk;
  a.sigmoid = score == EP_SCORE_SIGMOID;
  a.renorm = renormalize != 0;
  a.scale = scale;
  a.dlogits = dlogits;
  return launched(launch_route_backward(a, stream));
}

int ep_dispatch_permute_quantized(const void* q, const void* scale, int scale_words,
                                  int64_t num_tokens, int hidden, const int32_t* token_row,
                                  int num_topk, int64_t num_send_capacity, void* send_q,
                                  void* send_scale, hipStream_t stream) {
  if (num_tokens < 0 || num_topk < 1 || num_send_capacity < 0 || scale_words < 0 || hidden <= 0 ||
      hidden % EPDC_FP8_GROUP != 0)
    return EP_ERR_INVALID_ARG;
  if (num_tokens >= kMaxRows || num_topk > EPDC_MAX_TOPK || num_send_capacity > INT32_MAX ||
      hidden > (1 << 26) || scale_words > (1 << 26))
    return EP_ERR_UNSUPPORTED;
  const int64_t words = scale_words;
  if (!array_ok(q, num_tokens, 16) || !array_ok(scale, num_tokens * words, 4) ||
      !array_ok(token_row, num_tokens, 4) || !array_ok(send_q, num_send_capacity, 16) ||
      !array_ok(send_scale, num_send_capacity * words, 4))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0 || num_send_capacity == 0) return EP_OK;
  QuantRowArgs a{};
  a.q = q;
  a.scale = scale;
  a.words = scale_words;
  a.T = num_tokens;
  a.H = hidden;
  a.token_row = token_row;
  a.K = num_topk;
  a.capacity = num_send_capacity;
  a.out = send_q;
  a.out_scale = send_scale;
  return launched(launch_permute_quantized(a, stream));
}

}  // extern "C"
