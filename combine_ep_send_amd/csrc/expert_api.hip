// C ABI of the expert-side calls (include/epdc_expert.h): argument validation
// on the host, then launches.  Nothing here allocates, frees or synchronizes.
#include <stdint.h>

#include "../../include/epdc_expert.h"
#include "expert_launch.h"

namespace {

using namespace epdc;

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr size_t kPlanBytes = (sizeof(FewPlan) + 255) / 256 * 256;

static_assert(kFewSlots == EPDC_FEW_SLOTS && kFewExperts == EPDC_MAX_BINS, "limits");

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool arr_ok(const void* p, int64_t count, uintptr_t a) {
  return count == 0 || (p != nullptr && aligned(p, a));
}
int launch_status(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_LAUNCH; }

// Format and group of a 4-bit matrix with `channels` channels a row.
int check_w4(int fmt, int group, int channels) {
  if (fmt != EP_W_INT4 && fmt != EP_W_FP4) return EP_ERR_INVALID_ARG;
  if (group != 32 && (fmt == EP_W_FP4 || (group != 64 && group != 128)))
    return EP_ERR_INVALID_ARG;
  if (channels <= 0 || channels % 128 != 0) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

// `experts` matrices [out, in], and their pointers.
int check_weights(int fmt, int group, int out, int in, const void* w, const void* scale) {
  if (out <= 0 || in <= 0 || out % 8 != 0 || in % 8 != 0) return EP_ERR_INVALID_ARG;
  if (fmt == EP_W_BF16) {
    if (group != 0) return EP_ERR_INVALID_ARG;
  } else {
    const int st = check_w4(fmt, group, in);
    if (st != EP_OK) return st;
  }
  if (in > EPDC_FEW_CHANNELS || out > 2 * EPDC_FEW_CHANNELS) return EP_ERR_UNSUPPORTED;
  const int64_t bytes = fmt == EP_W_BF16 ? int64_t(out) * in * 2 : int64_t(out) * in / 2;
  if (bytes > EPDC_FEW_MATRIX_BYTES) return EP_ERR_UNSUPPORTED;
  if (!arr_ok(w, 1, 16) || (fmt != EP_W_BF16 && !arr_ok(scale, 1, 16))) return EP_ERR_INVALID_ARG;
  return EP_OK;
}

// Whether a matrix [out, in], both within EPDC_FEW_CHANNELS (out: twice), has a
// format that check_weights takes.
bool some_format(int out, int in) {
  if (out % 8 != 0 || in % 8 != 0) return false;
  const int64_t channels = int64_t(out) * in;
  return (in % 128 == 0 ? channels / 2 : channels * 2) <= EPDC_FEW_MATRIX_BYTES;
}

// The activations h in two bf16 parts, 256-byte aligned at their end.
size_t h_bytes(size_t slots, int inner) { return (slots * size_t(inner) * 4 + 255) / 256 * 256; }

Weights weights(int fmt, int group, const void* w, const void* scale) {
  const WeightKind kind = fmt == EP_W_BF16 ? kWBf16
                          : fmt == EP_W_FP4 ? kWFp4
                          : group == 32 ? kWInt4G32
                          : group == 64 ? kWInt4G64 : kWInt4G128;
  return Weights{kind, w, scale};
}

// Rows and channels of a row kernel of the training side.
int check_rows(int64_t rows, int channels, int step) {
  if (rows < 0 || channels <= 0 || channels % step != 0) return EP_ERR_INVALID_ARG;
  if (rows >= kMaxRows || channels > (1 << 26)) return EP_ERR_UNSUPPORTED;
  return EP_OK;
}

}  // namespace

extern "C" {

int ep_expert_abi_version(void) { return EPDC_EXPERT_ABI_VERSION; }

int ep_quantize_w4(const void* w, int64_t num_rows, int channels, int weight_fmt, int group,
                   void* q, void* scale, hipStream_t stream) {
  int st = check_w4(weight_fmt, group, channels);
  if (st != EP_OK) return st;
  st = check_rows(num_rows, channels, 128);
  if (st != EP_OK) return st;
  if (!arr_ok(w, num_rows, 16) || !arr_ok(q, num_rows, 16) || !arr_ok(scale, num_rows, 16))
    return EP_ERR_INVALID_ARG;
  if (num_rows == 0) return EP_OK;
  QuantArgs a{};
  a.w = w;
  a.rows = num_rows;
  a.channels = channels;
  a.fp4 = weight_fmt == EP_W_FP4;
  a.group = group;
  a.q = q;
  a.scale = scale;
  return launch_status(launch_quantize_w4(a, stream));
}

int ep_expert_matvec(const void* x, const int32_t* row_expert, int64_t num_rows, int num_experts,
                     int out_channels, int channels, int weight_fmt, int group, const void* w,
                     const void* w_scale, void* y, hipStream_t stream) {
  if (num_rows < 0 || num_experts < 1) return EP_ERR_INVALID_ARG;
  if (num_rows > EPDC_FEW_SLOTS || num_experts > EPDC_MAX_BINS) return EP_ERR_UNSUPPORTED;
  const int st = check_weights(weight_fmt, group, out_channels, channels, w, w_scale);
  if (st != EP_OK) return st;
  if (out_channels > EPDC_FEW_CHANNELS) return EP_ERR_UNSUPPORTED;
  if (!arr_ok(x, num_rows, 16) || !arr_ok(y, num_rows, 16) ||
      (row_expert ? !aligned(row_expert, 4) : num_rows > 0 && num_experts != 1))
    return EP_ERR_INVALID_ARG;
  if (num_rows == 0) return EP_OK;
  FewArgs a{};
  a.x = x;
  a.ids32 = row_expert;
  a.slots = int(num_rows);
  a.top = 1;
  a.rows = int(num_rows);
  a.per_token = 1;
  a.experts = num_experts;
  a.N = out_channels;
  a.K = channels;
  a.w = weights(weight_fmt, group, w, w_scale);
  a.y = y;
  return launch_status(launch_few_rows(a, false, stream));
}

size_t ep_moe_tokens_workspace_bytes(int64_t num_tokens, int num_topk, int hidden, int inner) {
  if (num_tokens < 0 || num_topk < 1 || hidden < 1 || inner < 1) return 0;
  if (num_tokens > EPDC_FEW_TOKENS || num_topk > EPDC_MAX_TOPK ||
      num_tokens * num_topk > EPDC_FEW_SLOTS || hidden > EPDC_FEW_CHANNELS ||
      inner > EPDC_FEW_CHANNELS)
    return 0;
  if (!some_format(2 * inner, hidden) || !some_format(hidden, inner)) return 0;
  const size_t slots = size_t(num_tokens) * size_t(num_topk);
  return kPlanBytes + h_bytes(slots, inner) +
         (few_down_joined(int(slots), hidden, inner) ? 0 : slots * size_t(hidden) * 4);
}

int ep_moe_tokens(const void* x, const int64_t* topk_idx, const float* topk_weights,
                  int64_t num_tokens, int num_topk, int hidden, int inner, int first_expert,
                  int num_local_experts, int w13_fmt, int w13_group, const void* w13,
                  const void* w13_scale, int w2_fmt, int w2_group, const void* w2,
                  const void* w2_scale, const void* bias0, const void* bias1, void* out,
                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (num_tokens < 0 || num_topk < 1 || num_local_experts < 1 || first_expert < 0 || hidden <= 0 ||
      inner <= 0)
    return EP_ERR_INVALID_ARG;
  if (num_tokens > EPDC_FEW_TOKENS || num_topk > EPDC_MAX_TOPK ||
      num_tokens * num_topk > EPDC_FEW_SLOTS || num_local_experts > EPDC_MAX_BINS ||
      hidden > EPDC_FEW_CHANNELS || inner > EPDC_FEW_CHANNELS)
    return EP_ERR_UNSUPPORTED;
  // 2I before I: an odd I passes neither
  int st = inner % 8 != 0 ? int(EP_ERR_INVALID_ARG)
                          : check_weights(w13_fmt, w13_group, 2 * inner, hidden, w13, w13_scale);
  if (st != EP_OK) return st;
  st = check_weights(w2_fmt, w2_group, hidden, inner, w2, w2_scale);
  if (st != EP_OK) return st;
  if (!arr_ok(x, num_tokens, 16) || !arr_ok(topk_idx, num_tokens, 8) ||
      !arr_ok(topk_weights, num_tokens, 4) || !arr_ok(out, num_tokens, 16) ||
      (bias0 && !aligned(bias0, 16)) || (bias1 && !aligned(bias1, 16)))
    return EP_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, 256) ||
      workspace_bytes < ep_moe_tokens_workspace_bytes(num_tokens, num_topk, hidden, inner))
    return EP_ERR_WORKSPACE;
  if (num_tokens == 0) return EP_OK;
  FewPlan* plan = static_cast<FewPlan*>(workspace);
  void* h = static_cast<char*>(workspace) + kPlanBytes;
  FewArgs a{};
  a.x = x;
  a.ids64 = topk_idx;
  a.first_expert = first_expert;
  a.slots = int(num_tokens) * num_topk;
  a.top = num_topk;
  a.rows = int(num_tokens);
  a.per_token = 1;
  a.experts = num_local_experts;
  a.N = inner;
  a.K = hidden;
  a.w = weights(w13_fmt, w13_group, w13, w13_scale);
  a.y = h;
  a.plan = plan;
  if (launch_few_rows(a, true, stream) != hipSuccess) return EP_ERR_LAUNCH;
  DownArgs d{};
  d.plan = plan;
  d.h = h;
  d.w = weights(w2_fmt, w2_group, w2, w2_scale);
  d.experts = num_local_experts;
  d.ids64 = topk_idx;
  d.first_expert = first_expert;
  d.topk_weights = topk_weights;
  d.T = int(num_tokens);
  d.K = num_topk;
  d.H = hidden;
  d.I = inner;
  d.bias0 = bias0;
  d.bias1 = bias1;
  d.out = out;
  d.y = reinterpret_cast<float*>(static_cast<char*>(h) + h_bytes(size_t(a.slots), inner));
  return launch_status(launch_few_down(d, stream));
}

int ep_swiglu_fp8(const void* gate_up, int64_t num_rows, int inner, const int32_t* row_count,
                  void* h, void* q, float* scale, hipStream_t stream) {
  const int st = check_rows(num_rows, inner, EPDC_FP8_GROUP);
  if (st != EP_OK) return st;
  if (!arr_ok(gate_up, num_rows, 16) || !arr_ok(h, num_rows, 16) || !arr_ok(q, num_rows, 16) ||
      !arr_ok(scale, num_rows, 4) || (row_count && !aligned(row_count, 4)))
    return EP_ERR_INVALID_ARG;
  if (num_rows == 0) return EP_OK;
  SwigluArgs a{};
  a.gate_up = gate_up;
  a.rows = num_rows;
  a.inner = inner;
  a.row_count = row_count;
  a.h = h;
  a.q = q;
  a.scale = scale;
  return launch_status(launch_swiglu_fp8(a, stream));
}

int ep_swiglu_fp8_backward(const void* dh, const void* q, const float* scale, int64_t num_rows,
                           int inner, const int32_t* row_count, void* d_gate_up, void* h,
                           hipStream_t stream) {
  const int st = check_rows(num_rows, inner, EPDC_FP8_GROUP);
  if (st != EP_OK) return st;
  if (!arr_ok(dh, num_rows, 16) || !arr_ok(q, num_rows, 16) || !arr_ok(scale, num_rows, 4) ||
      !arr_ok(d_gate_up, num_rows, 16) || (h && !aligned(h, 16)) ||
      (row_count && !aligned(row_count, 4)))
    return EP_ERR_INVALID_ARG;
  if (num_rows == 0) return EP_OK;
  SwigluArgs a{};
  a.dh = dh;
  a.rows = num_rows;
  a.inner = inner;
  a.row_count = row_count;
  a.h = h;
  a.q = const_cast<void*>(q);
  a.scale = const_cast<float*>(scale);
  a.d_gate_up = d_gate_up;
  return launch_status(launch_swiglu_fp8_backward(a, stream));
}

int ep_combine_backward(const void* dout, const void* y, int64_t num_rows,
                        const int32_t* token_row, const float* topk_weights, int64_t num_tokens,
                        int num_topk, int hidden, void* dy, float* dw, hipStream_t stream) {
  if (num_tokens < 0 || num_topk < 1 || num_rows < 0) return EP_ERR_INVALID_ARG;
  if (num_topk > EPDC_MAX_TOPK) return EP_ERR_UNSUPPORTED;
  const int st = check_rows(num_tokens, hidden, 8);
  if (st != EP_OK) return st;
  if (num_rows > INT32_MAX) return EP_ERR_UNSUPPORTED;
  if (dw && !topk_weights && num_tokens > 0) return EP_ERR_INVALID_ARG;
  if (!arr_ok(dout, num_tokens, 16) || !arr_ok(token_row, num_tokens, 4) ||
      (topk_weights && !aligned(topk_weights, 4)) || (dw && !aligned(dw, 4)) ||
      (dw ? !arr_ok(y, num_rows, 16) : y && !aligned(y, 16)) || !arr_ok(dy, num_rows, 16))
    return EP_ERR_INVALID_ARG;
  if (num_tokens == 0) return EP_OK;
  CombineBackwardArgs a{};
  a.dout = dout;
  a.y = y;
  a.R = num_rows;
  a.token_row = token_row;
  a.w = topk_weights;
  a.T = num_tokens;
  a.K = num_topk;
  a.H = hidden;
  a.dy = dy;
  a.dw = dw;
  return launch_status(launch_combine_backward(a, stream));
}

}  // extern "C"
