// C ABI of the general routing, the router losses and their gradient: argument checks and
// launches. Contracts are in include/moe.h.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/moe.h"
#include "moe_internal.h"

namespace moe {

moe_status_t fail_with(moe_status_t code, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  set_error_message(msg);
  return code;
}

moe_status_t launched(cudaError_t e, const char* where) {
  if (e == cudaSuccess) return MOE_OK;
  return fail_with(MOE_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

moe_status_t check_aligned(const void* p, const char* name, size_t align, bool nullable) {
  if (!p) return nullable ? MOE_OK : fail_with(MOE_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % align)
    return fail_with(MOE_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
  return MOE_OK;
}

// moe_routing_t -> Routing. full: the selection rule is checked too.
moe_status_t check_routing(const moe_routing_t* in, bool full, Routing* out) {
  if (!in) return fail_with(MOE_ERR_INVALID_ARG, "routing is NULL");
  if (in->num_tokens < 0 || in->num_tokens > (int64_t)1 << 30)
    return fail_with(MOE_ERR_INVALID_ARG, "num_tokens must be in [0, 2^30] (got %lld)",
                     (long long)in->num_tokens);
  if (in->num_experts < 1 || in->num_experts > 512)
    return fail_with(MOE_ERR_UNSUPPORTED, "num_experts must be in [1, 512] (got %d)",
                     in->num_experts);
  if (in->num_experts_per_tok < 1 || in->num_experts_per_tok > 32 ||
      in->num_experts_per_tok > in->num_experts)
    return fail_with(MOE_ERR_UNSUPPORTED,
                     "num_experts_per_tok must be in [1, min(32, num_experts)] (got %d)",
                     in->num_experts_per_tok);
  if (in->logits_stride < in->num_experts)
    return fail_with(MOE_ERR_INVALID_ARG, "logits_stride must be >= num_experts (got %lld)",
                     (long long)in->logits_stride);
  if (in->scoring != MOE_SCORING_SOFTMAX && in->scoring != MOE_SCORING_SIGMOID)
    return fail_with(MOE_ERR_INVALID_ARG,
                     "scoring must be MOE_SCORING_SOFTMAX or MOE_SCORING_SIGMOID (got %d)",
                     in->scoring);
  if (in->logits_bf16 != 0 && in->logits_bf16 != 1)
    return fail_with(MOE_ERR_INVALID_ARG, "logits_bf16 must be 0 or 1 (got %d)", in->logits_bf16);
  if (in->renormalize != 0 && in->renormalize != 1)
    return fail_with(MOE_ERR_INVALID_ARG, "renormalize must be 0 or 1 (got %d)", in->renormalize);
  if (!isfinite(in->weight_scale))
    return fail_with(MOE_ERR_INVALID_ARG, "weight_scale must be finite");
  if (full) {
    const int g = in->num_groups;
    if (g < 1 || g > 32 || in->num_experts % g)
      return fail_with(MOE_ERR_UNSUPPORTED,
                       "num_groups must be in [1, 32] and divide num_experts (got %d)", g);
    if (in->topk_groups < 1 || in->topk_groups > g)
      return fail_with(MOE_ERR_INVALID_ARG, "topk_groups must be in [1, num_groups] (got %d)",
                       in->topk_groups);
    if (in->group_top < 1 || in->group_top > in->num_experts / g || (g == 1 && in->group_top != 1))
      return fail_with(MOE_ERR_INVALID_ARG,
                       "group_top must be in [1, experts of a group], 1 with one group (got %d)",
                       in->group_top);
    if (in->num_experts_per_tok > in->topk_groups * (in->num_experts / g))
      return fail_with(MOE_ERR_INVALID_ARG,
                       "num_experts_per_tok is above the %d experts of topk_groups groups",
                       in->topk_groups * (in->num_experts / g));
  }
  out->T = in->num_tokens;
  out->stride = in->logits_stride;
  out->E = in->num_experts;
  out->k = in->num_experts_per_tok;
  out->sigmoid = in->scoring == MOE_SCORING_SIGMOID;
  out->groups = full ? in->num_groups : 1;
  out->topk_groups = full ? in->topk_groups : 1;
  out->group_top = full ? in->group_top : 1;
  out->renorm = in->renormalize;
  out->bf16 = in->logits_bf16;
  out->scale = in->weight_scale;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

#define MOE_TRY(x)               \
  do {                           \
    moe_status_t _s = (x);       \
    if (_s != MOE_OK) return _s; \
  } while (0)

namespace {

// Scratch of the losses: per block E + 1 double sums, then E + 1 int32 counts.
struct LossLayout {
  size_t count, end;
};
LossLayout loss_layout(const Routing& r) {
  const size_t n = (size_t)router_loss_blocks(r) * (r.E + 1);
  LossLayout l;
  l.count = (n * 8 + 255) / 256 * 256;
  l.end = l.count + (n * 4 + 255) / 256 * 256 + 256;
  return l;
}

}  // namespace

extern "C" {

moe_status_t moe_route(const moe_routing_t* routing, const void* logits, const float* select_bias,
                       int32_t* topk_idx, float* topk_w, moe_stream_t stream) {
  set_error_message("");
  Routing r;
  MOE_TRY(check_routing(routing, true, &r));
  if (r.T == 0) return MOE_OK;
  MOE_TRY(check_aligned(logits, "logits", r.bf16 ? 2 : 4, false));
  MOE_TRY(check_aligned(select_bias, "select_bias", 4, true));
  MOE_TRY(check_aligned(topk_idx, "topk_idx", 4, false));
  MOE_TRY(check_aligned(topk_w, "topk_w", 4, false));
  return launched(launch_route(r, logits, select_bias, topk_idx, topk_w, (cudaStream_t)stream),
                  "routing launch");
}

size_t moe_router_losses_workspace(const moe_routing_t* routing) {
  set_error_message("");
  Routing r;
  if (check_routing(routing, false, &r) != MOE_OK) return 0;
  return loss_layout(r).end;
}

moe_status_t moe_router_losses(const moe_routing_t* routing, const void* logits,
                               const int32_t* topk_idx, const uint8_t* token_mask, float* losses,
                               int32_t* counts, float* prob_mean, void* ws, size_t ws_bytes,
                               moe_stream_t stream) {
  set_error_message("");
  Routing r;
  MOE_TRY(check_routing(routing, false, &r));
  MOE_TRY(check_aligned(logits, "logits", r.bf16 ? 2 : 4, r.T == 0));
  MOE_TRY(check_aligned(topk_idx, "topk_idx", 4, r.T == 0));
  MOE_TRY(check_aligned(losses, "losses", 4, false));
  MOE_TRY(check_aligned(counts, "counts", 4, false));
  MOE_TRY(check_aligned(prob_mean, "prob_mean", 4, false));
  const LossLayout l = loss_layout(r);
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256)
    return fail_with(MOE_ERR_WORKSPACE, "workspace is NULL or not 256-byte aligned");
  if (ws_bytes < l.end)
    return fail_with(MOE_ERR_WORKSPACE, "workspace too small: need %zu bytes, got %zu", l.end,
                     ws_bytes);
  return launched(launch_router_losses(r, logits, topk_idx, token_mask, losses, counts, prob_mean,
                                       static_cast<double*>(ws),
                                       reinterpret_cast<int32_t*>(static_cast<char*>(ws) + l.count),
                                       (cudaStream_t)stream),
                  "router losses launch");
}

moe_status_t moe_route_backward(const moe_routing_t* routing, const void* logits,
                                const int32_t* topk_idx, const float* d_topk_w,
                                const int32_t* counts, const float* d_losses,
                                const uint8_t* token_mask, void* d_logits, moe_stream_t stream) {
  set_error_message("");
  Routing r;
  MOE_TRY(check_routing(routing, false, &r));
  if ((counts == nullptr) != (d_losses == nullptr))
    return fail_with(MOE_ERR_INVALID_ARG, "counts and d_losses go together: both or neither NULL");
  if (r.T == 0) return MOE_OK;
  MOE_TRY(check_aligned(logits, "logits", r.bf16 ? 2 : 4, false));
  MOE_TRY(check_aligned(topk_idx, "topk_idx", 4, d_topk_w == nullptr));
  MOE_TRY(check_aligned(d_topk_w, "d_topk_w", 4, true));
  MOE_TRY(check_aligned(counts, "counts", 4, true));
  MOE_TRY(check_aligned(d_losses, "d_losses", 4, true));
  MOE_TRY(check_aligned(d_logits, "d_logits", r.bf16 ? 2 : 4, false));
  return launched(launch_route_backward(r, logits, topk_idx, d_topk_w, counts, d_losses, token_mask,
                                        d_logits, (cudaStream_t)stream),
                  "routing backward launch");
}

}  // extern "C"
