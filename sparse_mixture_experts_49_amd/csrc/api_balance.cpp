// C ABI of the balance loss by sequence: argument validation, workspace carving, launches.
#include "api_util.h"
#include "balance.h"

using namespace moe::api;

namespace {

int validate_balance(const moe_balance_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID, "desc must not be NULL");
  if (d->tokens < 1) return fail(MOE_ERR_INVALID, "tokens must be >= 1 (got %d)", d->tokens);
  if (d->tokens > 1 << 22) return fail(MOE_ERR_UNSUPPORTED, "tokens must be <= 2^22 (got %d)", d->tokens);
  if (d->n_experts < 1) return fail(MOE_ERR_INVALID, "n_experts must be >= 1 (got %d)", d->n_experts);
  if (d->n_experts > moe::kBalanceMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "n_experts must be <= %d (got %d)", moe::kBalanceMaxExperts, d->n_experts);
  if (d->top_k < 1 || d->top_k > d->n_experts)
    return fail(MOE_ERR_INVALID, "top_k must be in [1, n_experts] (got %d)", d->top_k);
  if (d->top_k > 8) return fail(MOE_ERR_UNSUPPORTED, "top_k must be <= 8 (got %d)", d->top_k);
  if (d->n_seqs < 1) return fail(MOE_ERR_INVALID, "n_seqs must be >= 1 (got %d)", d->n_seqs);
  if (d->n_seqs > 1 << 20) return fail(MOE_ERR_UNSUPPORTED, "n_seqs must be <= 2^20 (got %d)", d->n_seqs);
  if (d->score != MOE_SCORE_SOFTMAX && d->score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID, "score must be MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID");
  return MOE_OK;
}

moe::BalanceShape shape_of(const moe_balance_desc* d) {
  return {d->tokens, d->n_experts, d->top_k, d->n_seqs, d->score == MOE_SCORE_SIGMOID};
}

struct BalanceLayout {
  size_t pq, pload, pvalid, part, total;
};

BalanceLayout layout_of(const moe_balance_desc* d) {
  BalanceLayout L{};
  const moe::BalanceShape s = shape_of(d);
  const size_t pieces = (size_t)moe::balance_chunks(s) + s.S, E = s.E;
  size_t p = 0;
  auto take = [&](size_t bytes) { size_t at = p; p += up256(bytes); return at; };
  L.pq = take(pieces * E * 4);
  L.pload = take(pieces * E * 4);
  L.pvalid = take(pieces * 4);
  L.part = take((size_t)s.S * moe::balance_blocks(s.E) * 8);
  L.total = p;
  return L;
}

}  // namespace

extern "C" {

int moe_balance_workspace_size(const moe_balance_desc* desc, size_t* bytes) {
  if (int st = validate_balance(desc)) return st;
  if (!bytes) return fail(MOE_ERR_INVALID, "bytes must not be NULL");
  *bytes = layout_of(desc).total;
  return ok();
}

int moe_balance_loss(const moe_balance_desc* desc, const float* logits, const int32_t* topk_idx,
                     const int32_t* seq_offsets, const uint8_t* token_mask, moe_balance_out* out, void* ws,
                     size_t ws_bytes, void* stream) {
  if (int st = validate_balance(desc)) return st;
  MOE_REQUIRE_PTR(logits, "logits");
  MOE_REQUIRE_PTR(topk_idx, "topk_idx");
  MOE_REQUIRE_PTR(seq_offsets, "seq_offsets");
  MOE_OPTIONAL_PTR(token_mask, "token_mask");
  if (!out) return fail(MOE_ERR_INVALID, "out must not be NULL");
  MOE_REQUIRE_PTR(out->load, "out->load");
  MOE_REQUIRE_PTR(out->valid, "out->valid");
  MOE_OPTIONAL_PTR(out->prob_mean, "out->prob_mean");
  MOE_OPTIONAL_PTR(out->seq_loss, "out->seq_loss");
  MOE_OPTIONAL_PTR(out->loss, "out->loss");
  MOE_OPTIONAL_PTR(out->total_load, "out->total_load");
  const BalanceLayout L = layout_of(desc);
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace must not be NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < L.total) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, L.total);
  const size_t T = desc->tokens, E = desc->n_experts, S = desc->n_seqs;
  {
    Spans o, in;
    o.add(out->load, S * E * 4, "load");
    o.add(out->valid, (S + 1) * 4, "valid");
    o.add(out->prob_mean, S * E * 4, "prob_mean");
    o.add(out->seq_loss, S * 4, "seq_loss");
    o.add(out->loss, 4, "loss");
    o.add(out->total_load, E * 4, "total_load");
    o.add(ws, ws_bytes, "workspace");
    in.add(logits, T * E * 4, "logits");
    in.add(topk_idx, T * desc->top_k * 4, "topk_idx");
    in.add(seq_offsets, (S + 1) * 4, "seq_offsets");
    in.add(token_mask, T, "token_mask");
    if (int st = check_alias(o, in)) return st;
  }
  moe::BalanceArgs a{};
  a.sh = shape_of(desc);
  a.logits = logits;
  a.topk_idx = topk_idx;
  a.offsets = seq_offsets;
  a.mask = token_mask;
  a.load = out->load;
  a.valid = out->valid;
  a.prob_mean = out->prob_mean;
  a.seq_loss = out->seq_loss;
  a.loss = out->loss;
  a.total_load = out->total_load;
  a.pq = at<float>(ws, L.pq);
  a.pload = at<int32_t>(ws, L.pload);
  a.pvalid = at<int32_t>(ws, L.pvalid);
  a.part = at<double>(ws, L.part);
  return hip_status(moe::launch_balance(a, static_cast<hipStream_t>(stream)), "balance loss launch");
}

int moe_balance_backward(const moe_balance_desc* desc, const float* logits, const int32_t* seq_offsets,
                         const uint8_t* token_mask, const moe_balance_out* fwd, const float* d_loss,
                         const float* d_seq_loss, float* d_logits, void* stream) {
  if (int st = validate_balance(desc)) return st;
  MOE_REQUIRE_PTR(logits, "logits");
  MOE_REQUIRE_PTR(seq_offsets, "seq_offsets");
  MOE_OPTIONAL_PTR(token_mask, "token_mask");
  if (!fwd) return fail(MOE_ERR_INVALID, "fwd must not be NULL");
  MOE_REQUIRE_PTR(fwd->load, "fwd->load");
  MOE_REQUIRE_PTR(fwd->valid, "fwd->valid");
  MOE_OPTIONAL_PTR(d_loss, "d_loss");
  MOE_OPTIONAL_PTR(d_seq_loss, "d_seq_loss");
  if (!d_loss && !d_seq_loss) return fail(MOE_ERR_INVALID, "d_loss and d_seq_loss are both NULL");
  MOE_REQUIRE_PTR(d_logits, "d_logits");
  const size_t T = desc->tokens, E = desc->n_experts, S = desc->n_seqs;
  {
    Spans o, in;
    o.add(d_logits, T * E * 4, "d_logits");
    in.add(logits, T * E * 4, "logits");
    in.add(seq_offsets, (S + 1) * 4, "seq_offsets");
    in.add(token_mask, T, "token_mask");
    in.add(fwd->load, S * E * 4, "load");
    in.add(fwd->valid, (S + 1) * 4, "valid");
    in.add(d_loss, 4, "d_loss");
    in.add(d_seq_loss, S * 4, "d_seq_loss");
    if (int st = check_alias(o, in)) return st;
  }
  moe::BalanceGradArgs a{};
  a.sh = shape_of(desc);
  a.logits = logits;
  a.offsets = seq_offsets;
  a.mask = token_mask;
  a.load = fwd->load;
  a.valid = fwd->valid;
  a.d_loss = d_loss;
  a.d_seq_loss = d_seq_loss;
  a.d_logits = d_logits;
  return hip_status(moe::launch_balance_grad(a, static_cast<hipStream_t>(stream)), "balance loss backward launch");
}

}  // extern "C"
