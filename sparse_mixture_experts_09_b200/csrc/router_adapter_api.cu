// C ABI of the general routing, the router losses, the gradients and the low-rank adapters:
// argument checks and launches. Contracts are in include/moe.h.
#include <cuda_runtime.h>
#include <math.h>
#include <limits.h>
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
  l.end = l.count + (n * 4 + 255) / 256 * 256;
  return l;
}

moe_status_t check_lora(const moe_lora_t* in, Lora* out) {
  if (!in) return fail_with(MOE_ERR_INVALID_ARG, "lora is NULL");
  if (in->num_rows < 0 || in->num_rows > 1 << 24)
    return fail_with(MOE_ERR_INVALID_ARG, "num_rows must be in [0, 2^24] (got %lld)",
                     (long long)in->num_rows);
  if (in->in_features <= 0 || in->in_features % 8 || in->out_features <= 0 || in->out_features % 8 ||
      in->in_features > 1 << 20 || in->out_features > 1 << 20)
    return fail_with(MOE_ERR_UNSUPPORTED,
                     "in_features and out_features must be positive multiples of 8, at most 2^20 "
                     "(got %d and %d)", in->in_features, in->out_features);
  if (in->rank < 8 || in->rank > 128 || in->rank % 8)
    return fail_with(MOE_ERR_UNSUPPORTED, "rank must be a multiple of 8 in [8, 128] (got %d)", in->rank);
  if (in->num_adapters < 1 || in->num_adapters > kLoraMaxAdapters)
    return fail_with(MOE_ERR_UNSUPPORTED, "num_adapters must be in [1, %d] (got %d)",
                     kLoraMaxAdapters, in->num_adapters);
  if (in->x_stride < in->in_features || in->x_stride % 8 || in->base_stride < in->out_features ||
      in->base_stride % 8 || in->out_stride < in->out_features || in->out_stride % 8)
    return fail_with(MOE_ERR_INVALID_ARG,
                     "the row strides must be multiples of 8, at least the row's length");
  if (in->out_fp32 != 0 && in->out_fp32 != 1)
    return fail_with(MOE_ERR_INVALID_ARG, "out_fp32 must be 0 or 1 (got %d)", in->out_fp32);
  out->R = in->num_rows;
  out->x_stride = in->x_stride;
  out->base_stride = in->base_stride;
  out->out_stride = in->out_stride;
  out->H = in->in_features;
  out->N = in->out_features;
  out->rank = in->rank;
  out->G = in->num_adapters;
  out->fp32 = in->out_fp32;
  return MOE_OK;
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
  if (l.end && (!ws || reinterpret_cast<uintptr_t>(ws) % 256))
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

moe_status_t moe_combine_backward(const moe_bf16_t* d_out, const float* y_perm,
                                  const int32_t* row_of, const float* topk_w,
                                  const int32_t* expert_counts, const int32_t* expert_offsets,
                                  float* dy_perm, float* d_topk_w, int64_t num_tokens, int k,
                                  int hidden, int num_experts, int64_t num_rows,
                                  moe_stream_t stream) {
  set_error_message("");
  if (num_tokens < 0 || num_rows < 0 || num_rows > INT_MAX)
    return fail_with(MOE_ERR_INVALID_ARG, "num_tokens and num_rows must be in [0, 2^31)");
  if (k < 1 || k > 8) return fail_with(MOE_ERR_UNSUPPORTED, "k must be in [1, 8] (got %d)", k);
  if (num_tokens > ((int64_t)1 << 30) / k)
    return fail_with(MOE_ERR_UNSUPPORTED, "num_tokens * k must be <= 2^30");
  if (hidden <= 0 || hidden % 8)
    return fail_with(MOE_ERR_UNSUPPORTED, "hidden must be a positive multiple of 8 (got %d)", hidden);
  if (num_experts < 1 || num_experts > 512)
    return fail_with(MOE_ERR_UNSUPPORTED, "num_experts must be in [1, 512] (got %d)", num_experts);
  const bool none = num_tokens == 0;
  MOE_TRY(check_aligned(d_out, "d_out", 16, none));
  MOE_TRY(check_aligned(row_of, "row_of", 4, none));
  MOE_TRY(check_aligned(dy_perm, "dy_perm", 16, true));
  MOE_TRY(check_aligned(d_topk_w, "d_topk_w", 4, true));
  MOE_TRY(check_aligned(y_perm, "y_perm", 16, none || !d_topk_w || num_rows == 0));
  MOE_TRY(check_aligned(topk_w, "topk_w", 4, none || !dy_perm));
  MOE_TRY(check_aligned(expert_counts, "expert_counts", 4, !dy_perm));
  MOE_TRY(check_aligned(expert_offsets, "expert_offsets", 4, !dy_perm));
  if (!dy_perm && !d_topk_w) return MOE_OK;
  CombineBwd c;
  c.d_out = d_out;
  c.y = y_perm;
  c.row_of = row_of;
  c.w = topk_w;
  c.counts = expert_counts;
  c.offsets = expert_offsets;
  c.dy = dy_perm;
  c.d_w = d_topk_w;
  c.T = num_tokens;
  c.rows = num_rows;
  c.k = k;
  c.H = hidden;
  c.E = num_experts;
  return launched(launch_combine_bwd(c, (cudaStream_t)stream), "combine backward launch");
}

size_t moe_lora_workspace(const moe_lora_t* lora) {
  set_error_message("");
  Lora l = {};
  if (check_lora(lora, &l) != MOE_OK) return 0;
  return lora_workspace(l);
}

moe_status_t moe_lora_add(const moe_lora_t* lora, const void* base, const moe_bf16_t* x,
                          const moe_bf16_t* a, const moe_bf16_t* b, const int32_t* adapter,
                          const float* scale, void* out, void* ws, size_t ws_bytes,
                          moe_stream_t stream) {
  set_error_message("");
  Lora l = {};
  MOE_TRY(check_lora(lora, &l));
  if (l.R == 0) return MOE_OK;
  MOE_TRY(check_aligned(base, "base", 16, false));
  MOE_TRY(check_aligned(x, "x", 16, false));
  MOE_TRY(check_aligned(a, "a", 16, false));
  MOE_TRY(check_aligned(b, "b", 16, false));
  MOE_TRY(check_aligned(adapter, "adapter", 4, false));
  MOE_TRY(check_aligned(scale, "scale", 4, true));
  MOE_TRY(check_aligned(out, "out", 16, false));
  if (out == base && l.out_stride != l.base_stride)
    return fail_with(MOE_ERR_INVALID_ARG, "out is base, but their strides differ");
  const size_t need = lora_workspace(l);
  if (need && (!ws || reinterpret_cast<uintptr_t>(ws) % 256))
    return fail_with(MOE_ERR_WORKSPACE, "workspace is NULL or not 256-byte aligned");
  if (ws_bytes < need)
    return fail_with(MOE_ERR_WORKSPACE, "workspace too small: need %zu bytes, got %zu", need, ws_bytes);
  l.x = x;
  l.a = a;
  l.b = b;
  l.adapter = adapter;
  l.scale = scale;
  l.base = base;
  l.out = out;
  return launched(launch_lora(l, ws, (cudaStream_t)stream), "adapter launch");
}

moe_status_t moe_lora_rows(const int32_t* token_of_row, const int32_t* expert_offsets,
                           const int32_t* adapter, int64_t num_tokens, int64_t num_rows,
                           int num_experts, int num_adapters, int32_t* row_adapter,
                           moe_stream_t stream) {
  set_error_message("");
  if (num_tokens < 0 || num_rows < 0 || num_rows > INT_MAX)
    return fail_with(MOE_ERR_INVALID_ARG, "num_tokens and num_rows must be in [0, 2^31)");
  if (num_experts < 1 || num_experts > 512)
    return fail_with(MOE_ERR_UNSUPPORTED, "num_experts must be in [1, 512] (got %d)", num_experts);
  if (num_adapters < 1 || num_adapters > kLoraMaxAdapters / num_experts)
    return fail_with(MOE_ERR_UNSUPPORTED,
                     "num_adapters must be >= 1 and num_adapters * num_experts <= %d (got %d)",
                     kLoraMaxAdapters, num_adapters);
  if (num_rows == 0) return MOE_OK;
  MOE_TRY(check_aligned(token_of_row, "token_of_row", 4, false));
  MOE_TRY(check_aligned(expert_offsets, "expert_offsets", 4, false));
  MOE_TRY(check_aligned(adapter, "adapter", 4, num_tokens == 0));
  MOE_TRY(check_aligned(row_adapter, "row_adapter", 4, false));
  return launched(launch_lora_rows(token_of_row, expert_offsets, adapter, num_tokens, num_rows,
                                   num_experts, num_adapters, row_adapter, (cudaStream_t)stream),
                  "row adapter launch");
}

moe_status_t moe_swiglu_rows(const float* gate, const float* up, const int32_t* expert_offsets,
                             int num_experts, int64_t num_rows, int intermediate, moe_bf16_t* h,
                             moe_stream_t stream) {
  set_error_message("");
  if (num_rows < 0 || num_rows > INT_MAX)
    return fail_with(MOE_ERR_INVALID_ARG, "num_rows must be in [0, 2^31)");
  if (num_experts < 1 || num_experts > 512)
    return fail_with(MOE_ERR_UNSUPPORTED, "num_experts must be in [1, 512] (got %d)", num_experts);
  if (intermediate <= 0 || intermediate % 8)
    return fail_with(MOE_ERR_UNSUPPORTED, "intermediate must be a positive multiple of 8 (got %d)",
                     intermediate);
  if (num_rows == 0) return MOE_OK;
  MOE_TRY(check_aligned(gate, "gate", 16, false));
  MOE_TRY(check_aligned(up, "up", 16, false));
  MOE_TRY(check_aligned(expert_offsets, "expert_offsets", 4, false));
  MOE_TRY(check_aligned(h, "h", 16, false));
  return launched(launch_swiglu_rows(gate, up, expert_offsets, num_experts, num_rows, intermediate, h,
                                     (cudaStream_t)stream),
                  "activation launch");
}

}  // extern "C"
