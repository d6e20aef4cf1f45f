// C ABI of the scored router: argument validation, workspace carving, launches.
#include <cmath>

#include "api_util.h"
#include "score.h"

using namespace moe::api;

namespace {

int validate_score(const moe_score_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID, "desc must not be NULL");
  if (d->tokens < 1) return fail(MOE_ERR_INVALID, "tokens must be >= 1 (got %d)", d->tokens);
  if (d->tokens > 1 << 22)
    return fail(MOE_ERR_UNSUPPORTED, "tokens must be <= 2^22 (got %d)", d->tokens);
  if (d->d_model < 1) return fail(MOE_ERR_INVALID, "d_model must be >= 1 (got %d)", d->d_model);
  if (d->d_model % 128)
    return fail(MOE_ERR_UNSUPPORTED, "d_model (%d) must be a multiple of 128", d->d_model);
  if (d->n_experts < 1) return fail(MOE_ERR_INVALID, "n_experts must be >= 1 (got %d)", d->n_experts);
  if (d->n_experts > moe::kScoreMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "n_experts must be <= %d (got %d)", moe::kScoreMaxExperts,
                d->n_experts);
  if (d->dtype != MOE_DTYPE_F32 && d->dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_INVALID, "dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  if (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID, "score must be MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID");
  if (d->n_groups < 1 || d->n_experts % d->n_groups)
    return fail(MOE_ERR_INVALID, "n_groups (%d) must divide n_experts (%d)", d->n_groups,
                d->n_experts);
  if (d->n_groups > 64)
    return fail(MOE_ERR_UNSUPPORTED, "n_groups must be <= 64 (got %d)", d->n_groups);
  const int per = d->n_experts / d->n_groups;
  if (d->top_groups < 1 || d->top_groups > d->n_groups)
    return fail(MOE_ERR_INVALID, "top_groups must be in [1, n_groups] (got %d)", d->top_groups);
  if ((d->group_top != 1 && d->group_top != 2) || d->group_top > per)
    return fail(MOE_ERR_INVALID, "group_top must be 1 or 2 and at most the experts of a group (got %d)",
                d->group_top);
  if (d->top_k < 1 || d->top_k > d->top_groups * per)
    return fail(MOE_ERR_INVALID, "top_k must be in [1, experts of top_groups groups] (got %d)", d->top_k);
  if (d->top_k > 8) return fail(MOE_ERR_UNSUPPORTED, "top_k must be <= 8 (got %d)", d->top_k);
  if (d->renormalize != 0 && d->renormalize != 1)
    return fail(MOE_ERR_INVALID, "renormalize must be 0 or 1");
  if (!std::isfinite(d->scale)) return fail(MOE_ERR_INVALID, "scale must be finite");
  if (d->d_model > 1 << 20)
    return fail(MOE_ERR_UNSUPPORTED, "d_model must be <= 2^20 (got %d)", d->d_model);
  return MOE_OK;
}

moe::ScoreShape shape_of(const moe_score_desc* d) {
  return {d->dtype == MOE_DTYPE_BF16, d->tokens, d->d_model, d->n_experts, d->top_k};
}

// The forward and the backward use the same bytes, one call at a time.
struct ScoreLayout {
  size_t part, psum, pload, pz, share, done;   // forward
  size_t dl, pb, pw;              // backward
  size_t total;
};

ScoreLayout layout_of(const moe_score_desc* d) {
  ScoreLayout L{};
  const moe::ScoreShape s = shape_of(d);
  const size_t T = s.T, E = s.E;
  size_t p = 0;
  auto take = [&](size_t bytes) { size_t at = p; p += up256(bytes); return at; };
  L.part = take((size_t)moe::score_parts(s) * T * E * 4);
  const size_t sums = T < 256 ? T : 256;              // blocks with partial sums, at most
  L.psum = take(sums * E * 8);
  L.pload = take(sums * E * 4);
  L.pz = take(sums * 8);
  L.share = take(E * 8);
  L.done = take(4);
  L.total = p;
  p = 0;
  L.dl = take(moe::score_dl_bytes(s));
  L.pb = take((size_t)moe::score_grad_sum_blocks(s.T) * E * 8);
  L.pw = take((size_t)moe::score_grad_slices(s) * E * s.d * 4);
  if (p > L.total) L.total = p;
  return L;
}

int check_ws(const moe_score_desc* d, void* ws, size_t bytes, ScoreLayout& L) {
  L = layout_of(d);
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace must not be NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (bytes < L.total)
    return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, L.total);
  return MOE_OK;
}

size_t elem(const moe_score_desc* d) { return d->dtype == MOE_DTYPE_BF16 ? 2 : 4; }

}  // namespace

extern "C" {

int moe_score_workspace_size(const moe_score_desc* desc, size_t* bytes) {
  if (int st = validate_score(desc)) return st;
  if (!bytes) return fail(MOE_ERR_INVALID, "bytes must not be NULL");
  *bytes = layout_of(desc).total;
  return ok();
}

int moe_score_route(const moe_score_desc* desc, const void* x, const void* w_router,
                    const float* b_router, const float* b_select, moe_score_out* out, void* ws,
                    size_t ws_bytes, void* stream) {
  if (int st = validate_score(desc)) return st;
  MOE_REQUIRE_PTR(x, "x");
  MOE_REQUIRE_PTR(w_router, "w_router");
  MOE_OPTIONAL_PTR(b_router, "b_router");
  MOE_OPTIONAL_PTR(b_select, "b_select");
  if (!out) return fail(MOE_ERR_INVALID, "out must not be NULL");
  MOE_REQUIRE_PTR(out->topk_idx, "out->topk_idx");
  MOE_REQUIRE_PTR(out->topk_w, "out->topk_w");
  MOE_OPTIONAL_PTR(out->logits, "out->logits");
  MOE_OPTIONAL_PTR(out->load, "out->load");
  MOE_OPTIONAL_PTR(out->prob_mean, "out->prob_mean");
  MOE_OPTIONAL_PTR(out->aux, "out->aux");
  MOE_OPTIONAL_PTR(out->z_loss, "out->z_loss");
  ScoreLayout L;
  if (int st = check_ws(desc, ws, ws_bytes, L)) return st;
  const size_t T = desc->tokens, D = desc->d_model, E = desc->n_experts, k = desc->top_k;
  {
    Spans o, in;
    o.add(out->topk_idx, T * k * 4, "topk_idx");
    o.add(out->topk_w, T * k * 4, "topk_w");
    o.add(out->logits, T * E * 4, "logits");
    o.add(out->load, E * 4, "load");
    o.add(out->prob_mean, E * 4, "prob_mean");
    o.add(out->aux, 4, "aux");
    o.add(out->z_loss, 4, "z_loss");
    o.add(ws, ws_bytes, "workspace");
    in.add(x, T * D * elem(desc), "x");
    in.add(w_router, E * D * elem(desc), "w_router");
    in.add(b_router, E * 4, "b_router");
    in.add(b_select, E * 4, "b_select");
    if (int st = check_alias(o, in)) return st;
  }
  moe::ScoreArgs a{};
  a.sh = shape_of(desc);
  a.x = x;
  a.w = w_router;
  a.b_router = b_router;
  a.b_select = b_select;
  a.sigmoid = desc->score == MOE_SCORE_SIGMOID;
  a.groups = desc->n_groups;
  a.top_groups = desc->top_groups;
  a.group_top = desc->group_top;
  a.renorm = desc->renormalize;
  a.scale = desc->scale;
  a.topk_idx = out->topk_idx;
  a.topk_w = out->topk_w;
  a.logits = out->logits;
  a.load = out->load;
  a.prob_mean = out->prob_mean;
  a.aux = out->aux;
  a.z_loss = out->z_loss;
  a.part = at<float>(ws, L.part);
  a.psum = at<double>(ws, L.psum);
  a.pload = at<int32_t>(ws, L.pload);
  a.pz = at<double>(ws, L.pz);
  a.share = at<double>(ws, L.share);
  a.done = at<uint32_t>(ws, L.done);
  return hip_status(moe::launch_score(a, static_cast<hipStream_t>(stream)), "scored router launch");
}

int moe_score_backward(const moe_score_desc* desc, const void* x, const void* w_router,
                       const moe_score_out* fwd, const float* d_topk_w, const float* d_aux,
                       const float* d_z_loss, moe_score_grads* grads, void* ws, size_t ws_bytes,
                       void* stream) {
  if (int st = validate_score(desc)) return st;
  if (!fwd) return fail(MOE_ERR_INVALID, "fwd must not be NULL");
  if (!grads) return fail(MOE_ERR_INVALID, "grads must not be NULL");
  MOE_REQUIRE_PTR(fwd->topk_idx, "fwd->topk_idx");
  MOE_REQUIRE_PTR(fwd->logits, "fwd->logits");
  if (d_aux) MOE_REQUIRE_PTR(fwd->load, "fwd->load");
  MOE_OPTIONAL_PTR(d_topk_w, "d_topk_w");
  MOE_OPTIONAL_PTR(d_aux, "d_aux");
  MOE_OPTIONAL_PTR(d_z_loss, "d_z_loss");
  if (!grads->d_x && !grads->d_w_router && !grads->d_b_router && !grads->d_logits)
    return fail(MOE_ERR_INVALID, "grads asks for nothing");
  MOE_OPTIONAL_PTR(grads->d_x, "grads->d_x");
  MOE_OPTIONAL_PTR(grads->d_w_router, "grads->d_w_router");
  MOE_OPTIONAL_PTR(grads->d_b_router, "grads->d_b_router");
  MOE_OPTIONAL_PTR(grads->d_logits, "grads->d_logits");
  if (grads->d_w_router) MOE_REQUIRE_PTR(x, "x");
  if (grads->d_x) MOE_REQUIRE_PTR(w_router, "w_router");
  ScoreLayout L;
  if (int st = check_ws(desc, ws, ws_bytes, L)) return st;
  const size_t T = desc->tokens, D = desc->d_model, E = desc->n_experts, k = desc->top_k;
  {
    Spans o, in;
    o.add(grads->d_x, T * D * elem(desc), "d_x");
    o.add(grads->d_w_router, E * D * 4, "d_w_router");
    o.add(grads->d_b_router, E * 4, "d_b_router");
    o.add(grads->d_logits, T * E * 4, "d_logits");
    o.add(ws, ws_bytes, "workspace");
    if (grads->d_w_router) in.add(x, T * D * elem(desc), "x");
    if (grads->d_x) in.add(w_router, E * D * elem(desc), "w_router");
    in.add(fwd->topk_idx, T * k * 4, "topk_idx");
    in.add(fwd->logits, T * E * 4, "logits");
    if (d_aux) in.add(fwd->load, E * 4, "load");
    in.add(d_topk_w, T * k * 4, "d_topk_w");
    in.add(d_aux, 4, "d_aux");
    in.add(d_z_loss, 4, "d_z_loss");
    if (int st = check_alias(o, in)) return st;
  }
  moe::ScoreGradArgs a{};
  a.sh = shape_of(desc);
  a.sigmoid = desc->score == MOE_SCORE_SIGMOID;
  a.renorm = desc->renormalize;
  a.scale = desc->scale;
  a.x = x;
  a.w = w_router;
  a.topk_idx = fwd->topk_idx;
  a.logits = fwd->logits;
  a.load = fwd->load;
  a.d_topk_w = d_topk_w;
  a.d_aux = d_aux;
  a.d_z = d_z_loss;
  a.d_x = grads->d_x;
  a.d_w = grads->d_w_router;
  a.d_b = grads->d_b_router;
  a.d_logits = grads->d_logits;
  a.dl = at<float>(ws, L.dl);
  a.pb = at<double>(ws, L.pb);
  a.pw = at<float>(ws, L.pw);
  return hip_status(moe::launch_score_grad(a, static_cast<hipStream_t>(stream)),
                    "scored router backward launch");
}

}  // extern "C"
