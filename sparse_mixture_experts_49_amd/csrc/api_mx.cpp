// C ABI of the MXFP4 experts: argument validation, workspace carving, launches.
#include <limits>

#include "api_util.h"
#include "kernels.h"
#include "mx.h"

using namespace moe::api;

namespace {

int validate_mx(const moe_mx_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID, "desc must not be NULL");
  if (d->tokens < 1) return fail(MOE_ERR_INVALID, "tokens must be >= 1 (got %d)", d->tokens);
  if (d->n_experts < 1) return fail(MOE_ERR_INVALID, "n_experts must be >= 1 (got %d)", d->n_experts);
  if (d->n_experts > moe::kMxMaxExperts)
    return fail(MOE_ERR_UNSUPPORTED, "n_experts must be <= %d (got %d)", moe::kMxMaxExperts, d->n_experts);
  if (d->top_k < 1 || d->top_k > d->n_experts)
    return fail(MOE_ERR_INVALID, "top_k must be in [1, n_experts] (got %d)", d->top_k);
  if (d->top_k > 8) return fail(MOE_ERR_UNSUPPORTED, "top_k must be <= 8 (got %d)", d->top_k);
  if (d->d_model < 1 || d->d_ff < 1) return fail(MOE_ERR_INVALID, "d_model and d_ff must be >= 1");
  if (d->d_model % 128 || d->d_ff % 128)
    return fail(MOE_ERR_UNSUPPORTED, "d_model (%d) and d_ff (%d) must be multiples of 128", d->d_model,
                d->d_ff);
  if (d->act != MOE_MX_ACT_BF16 && d->act != MOE_MX_ACT_MXFP4)
    return fail(MOE_ERR_INVALID, "act must be MOE_MX_ACT_BF16 or MOE_MX_ACT_MXFP4");
  if (d->has_expert_bias != 0 && d->has_expert_bias != 1)
    return fail(MOE_ERR_INVALID, "has_expert_bias must be 0 or 1");
  const long long most = std::numeric_limits<int32_t>::max();
  const long long widest = d->d_model > d->d_ff ? d->d_model : d->d_ff;
  if ((long long)d->tokens * d->top_k * widest > most)
    return fail(MOE_ERR_UNSUPPORTED, "tokens * top_k * max(d_model, d_ff) exceeds int32");
  if ((long long)d->d_model * d->d_ff > most)
    return fail(MOE_ERR_UNSUPPORTED, "one expert's d_model * d_ff exceeds int32");
  return MOE_OK;
}

struct MxLayout {
  size_t act, partial, blk_hist, blk_base;          // every call
  size_t counts, offsets, dest, src, topk_idx, topk_w, h, o;   // moe_mx_forward
  size_t total;
};

MxLayout layout_of(const moe_mx_desc* d) {
  MxLayout L{};
  const int T = d->tokens, k = d->top_k, E = d->n_experts, D = d->d_model, F = d->d_ff;
  const bool fp4 = d->act == MOE_MX_ACT_MXFP4;
  const size_t A = (size_t)T * k, nb = moe::mx_dispatch_blocks((int)A);
  size_t p = 0;
  auto take = [&](size_t bytes) { size_t at = p; p += up256(bytes); return at; };
  auto larger = [](size_t a, size_t b) { return a > b ? a : b; };
  L.act = take(larger(moe::mx_act_bytes(T, k, E, F, D, fp4), moe::mx_act_bytes(T, k, E, D, F, fp4)));
  L.partial = take(larger(moe::mx_partial_bytes(T, k, E, F, D), moe::mx_partial_bytes(T, k, E, D, F)));
  L.blk_hist = take(nb * E * 4);
  L.blk_base = take(nb * E * 4);
  L.counts = take((size_t)E * 4);
  L.offsets = take((size_t)(E + 1) * 4);
  L.dest = take(A * 4);
  L.src = take(A * 4);
  L.topk_idx = take(A * 4);
  L.topk_w = take(A * 4);
  L.h = take(A * F * 2);
  L.o = take(A * D * 4);
  L.total = p;
  return L;
}

int check_ws(const moe_mx_desc* d, void* ws, size_t bytes, size_t more, MxLayout& L) {
  L = layout_of(d);
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace must not be NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (bytes < L.total + more)
    return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, L.total + more);
  return MOE_OK;
}

int validate_weights(const moe_mx_desc* d, const moe_mx_weights* w, bool up, bool down) {
  if (!w) return fail(MOE_ERR_INVALID, "weights must not be NULL");
  if (up) {
    MOE_REQUIRE_PTR(w->w1, "w1");
    MOE_REQUIRE_PTR(w->s1, "s1");
    if (d->has_expert_bias) MOE_REQUIRE_PTR(w->b1, "b1");
  }
  if (down) {
    MOE_REQUIRE_PTR(w->w2, "w2");
    MOE_REQUIRE_PTR(w->s2, "s2");
    if (d->has_expert_bias) MOE_REQUIRE_PTR(w->b2, "b2");
  }
  if (!d->has_expert_bias && (w->b1 || w->b2))
    return fail(MOE_ERR_INVALID, "b1/b2 given but has_expert_bias == 0");
  return MOE_OK;
}

void add_weights(Spans& in, const moe_mx_desc* d, const moe_mx_weights* w, bool up, bool down) {
  const size_t E = d->n_experts, n = E * d->d_model * d->d_ff;
  if (up) {
    in.add(w->w1, n / 2, "w1");
    in.add(w->s1, n / 32, "s1");
    in.add(w->b1, E * d->d_ff * 2, "b1");
  }
  if (down) {
    in.add(w->w2, n / 2, "w2");
    in.add(w->s2, n / 32, "s2");
    in.add(w->b2, E * d->d_model * 2, "b2");
  }
}

int launch_product(const moe_mx_desc* d, bool up, const void* a, const int32_t* src,
                   const int32_t* offsets, const moe_mx_weights* w, void* out, void* ws,
                   const MxLayout& L, hipStream_t s) {
  moe::MxFfnArgs f{};
  f.up = up;
  f.fp4 = d->act == MOE_MX_ACT_MXFP4;
  f.a = a;
  f.a_rows = (up && src) ? d->tokens : (int64_t)d->tokens * d->top_k;
  f.src = src;
  f.offsets = offsets;
  f.w = up ? w->w1 : w->w2;
  f.ws = up ? w->s1 : w->s2;
  f.bias = d->has_expert_bias ? (up ? w->b1 : w->b2) : nullptr;
  f.out = out;
  f.T = d->tokens;
  f.k = d->top_k;
  f.E = d->n_experts;
  f.N = up ? d->d_ff : d->d_model;
  f.K = up ? d->d_model : d->d_ff;
  f.act = at<uint8_t>(ws, L.act);
  f.partial = at<float>(ws, L.partial);
  return hip_status(moe::launch_mx_ffn(f, s), up ? "mx up launch" : "mx down launch");
}

int launch_dispatch(const moe_mx_desc* d, const int32_t* idx, int32_t* counts, int32_t* offsets,
                    int32_t* dest, int32_t* src, void* ws, const MxLayout& L, hipStream_t s) {
  moe::MxDispatchArgs a{};
  a.topk_idx = idx;
  a.A = d->tokens * d->top_k;
  a.E = d->n_experts;
  a.counts = counts;
  a.offsets = offsets;
  a.dest = dest;
  a.src = src;
  a.blk_hist = at<int32_t>(ws, L.blk_hist);
  a.blk_base = at<int32_t>(ws, L.blk_base);
  return hip_status(moe::launch_mx_dispatch(a, s), "mx dispatch launch");
}

// Rows of a quantisation call.
int validate_rows(int dtype, int64_t rows, int64_t cols, int64_t stride) {
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_INVALID, "dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  if (rows < 0) return fail(MOE_ERR_INVALID, "rows must be >= 0");
  if (cols < 32 || cols % 32) return fail(MOE_ERR_INVALID, "cols must be a positive multiple of 32");
  if (stride < cols) return fail(MOE_ERR_INVALID, "row_stride must be >= cols");
  if (stride % (dtype == MOE_DTYPE_BF16 ? 8 : 4))
    return fail(MOE_ERR_INVALID, "row_stride must be a multiple of 16 bytes");
  // One thread per 8 values, and a launch takes under 2^32 threads.
  if (cols > std::numeric_limits<int32_t>::max() || rows > (int64_t(1) << 34) / cols)
    return fail(MOE_ERR_UNSUPPORTED, "rows * cols must be at most 2^34");
  return MOE_OK;
}

size_t rows_bytes(int dtype, int64_t rows, int64_t cols, int64_t stride) {
  return rows ? ((size_t)(rows - 1) * stride + cols) * (dtype == MOE_DTYPE_BF16 ? 2 : 4) : 0;
}

// The layer on tokens x, its workspace carved as L with the router's behind it; shared [T][d] fp32
// or null is added to y.
int run_layer(const moe_score_desc* route, const moe_mx_desc* desc, const void* x, const void* w_router,
              const float* b_router, const float* b_select, const moe_mx_weights* w, const float* shared, float* y,
              moe_score_out r, void* ws, const MxLayout& L, size_t route_bytes, void* stream) {
  if (!r.topk_idx) r.topk_idx = at<int32_t>(ws, L.topk_idx);
  if (!r.topk_w) r.topk_w = at<float>(ws, L.topk_w);
  hipStream_t s = static_cast<hipStream_t>(stream);
  int32_t *counts = at<int32_t>(ws, L.counts), *offsets = at<int32_t>(ws, L.offsets),
          *dest = at<int32_t>(ws, L.dest), *src = at<int32_t>(ws, L.src);
  void* h = at<void>(ws, L.h);
  float* o = at<float>(ws, L.o);
  if (int st = moe_score_route(route, x, w_router, b_router, b_select, &r, at<void>(ws, L.total),
                               route_bytes, stream))
    return st;
  if (int st = launch_dispatch(desc, r.topk_idx, counts, offsets, dest, src, ws, L, s)) return st;
  if (int st = launch_product(desc, true, x, src, offsets, w, h, ws, L, s)) return st;
  if (int st = launch_product(desc, false, h, nullptr, offsets, w, o, ws, L, s)) return st;
  moe::CombineArgs c{};
  c.o = o;
  c.dest = dest;
  c.topk_w = r.topk_w;
  c.shared = shared;
  c.y = y;
  c.T = desc->tokens;
  c.d = desc->d_model;
  c.k = desc->top_k;
  return hip_status(moe::launch_combine(c, s), "combine launch");
}

// Routing, experts and shared expert of a block agree in tokens and width; where its workspace's
// parts begin.
struct BlockLayout {
  size_t xn, shared, lora, layer, total;
  size_t route_bytes, lora_bytes;
};

int validate_pairing(const moe_score_desc* route, const moe_mx_desc* desc) {
  if (route->tokens != desc->tokens || route->d_model != desc->d_model || route->n_experts != desc->n_experts ||
      route->top_k != desc->top_k)
    return fail(MOE_ERR_INVALID, "route and desc differ in tokens, d_model, n_experts or top_k");
  if (route->dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "moe_mx_forward takes bf16 tokens (route->dtype)");
  return MOE_OK;
}

int validate_block(const moe_mx_block* b, BlockLayout& B) {
  B = BlockLayout{};
  if (!b) return fail(MOE_ERR_INVALID, "block must not be NULL");
  size_t bytes = 0;
  if (int st = moe_norm_workspace_size(b->norm, &bytes)) return st;
  if (int st = moe_score_workspace_size(b->route, &B.route_bytes)) return st;
  if (int st = validate_mx(b->experts)) return st;
  if (int st = validate_pairing(b->route, b->experts)) return st;
  if (b->norm->rows != b->experts->tokens || b->norm->d != b->experts->d_model)
    return fail(MOE_ERR_INVALID, "norm and experts differ in tokens or d_model");
  if (b->norm->dtype != MOE_DTYPE_BF16) return fail(MOE_ERR_UNSUPPORTED, "norm->dtype must be MOE_DTYPE_BF16");
  if (!b->up != !b->down) return fail(MOE_ERR_INVALID, "up and down must both be given, or neither");
  const size_t T = b->experts->tokens, D = b->experts->d_model;
  size_t p = 0;
  auto take = [&](size_t n) { size_t at = p; p += up256(n); return at; };
  B.xn = take(T * D * 2);
  if (b->up) {
    if (int st = moe_lora_shared_workspace_size(b->up, b->down, &B.lora_bytes)) return st;
    if (b->up->tokens != b->experts->tokens || b->up->d_in != b->experts->d_model)
      return fail(MOE_ERR_INVALID, "up and experts differ in tokens or d_model");
    B.shared = take(T * D * 4);
    B.lora = take(B.lora_bytes);
  }
  B.layer = take(layout_of(b->experts).total + B.route_bytes);
  B.total = p;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_mx_quantize(const void* x, int dtype, int64_t rows, int64_t cols, int64_t row_stride,
                    uint8_t* codes, uint8_t* scales, void* stream) {
  if (int st = validate_rows(dtype, rows, cols, row_stride)) return st;
  if (rows == 0) return ok();
  MOE_REQUIRE_PTR(x, "x");
  MOE_REQUIRE_PTR(codes, "codes");
  MOE_REQUIRE_PTR(scales, "scales");
  {
    Spans o, in;
    o.add(codes, (size_t)rows * cols / 2, "codes");
    o.add(scales, (size_t)rows * cols / 32, "scales");
    in.add(x, rows_bytes(dtype, rows, cols, row_stride), "x");
    if (int st = check_alias(o, in)) return st;
  }
  return hip_status(moe::launch_mx_quantize(x, dtype == MOE_DTYPE_BF16, rows, cols, row_stride, codes,
                                            scales, static_cast<hipStream_t>(stream)),
                    "mx quantize launch");
}

int moe_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                      int dtype, void* out, int64_t row_stride, void* stream) {
  if (int st = validate_rows(dtype, rows, cols, row_stride)) return st;
  if (rows == 0) return ok();
  MOE_REQUIRE_PTR(codes, "codes");
  MOE_REQUIRE_PTR(scales, "scales");
  MOE_REQUIRE_PTR(out, "out");
  {
    Spans o, in;
    o.add(out, rows_bytes(dtype, rows, cols, row_stride), "out");
    in.add(codes, (size_t)rows * cols / 2, "codes");
    in.add(scales, (size_t)rows * cols / 32, "scales");
    if (int st = check_alias(o, in)) return st;
  }
  return hip_status(moe::launch_mx_dequantize(codes, scales, rows, cols, dtype == MOE_DTYPE_BF16, out,
                                              row_stride, static_cast<hipStream_t>(stream)),
                    "mx dequantize launch");
}

int moe_mx_workspace_size(const moe_mx_desc* desc, size_t* bytes) {
  if (int st = validate_mx(desc)) return st;
  if (!bytes) return fail(MOE_ERR_INVALID, "bytes must not be NULL");
  *bytes = layout_of(desc).total;
  return ok();
}

int moe_mx_dispatch(const moe_mx_desc* desc, moe_routing* r, void* ws, size_t ws_bytes, void* stream) {
  if (int st = validate_mx(desc)) return st;
  if (!r) return fail(MOE_ERR_INVALID, "r must not be NULL");
  MOE_REQUIRE_PTR(r->topk_idx, "r->topk_idx");
  MOE_REQUIRE_PTR(r->counts, "r->counts");
  MOE_REQUIRE_PTR(r->offsets, "r->offsets");
  MOE_REQUIRE_PTR(r->dest, "r->dest");
  MOE_REQUIRE_PTR(r->src, "r->src");
  MxLayout L;
  if (int st = check_ws(desc, ws, ws_bytes, 0, L)) return st;
  const size_t A = (size_t)desc->tokens * desc->top_k, E = desc->n_experts;
  {
    Spans o, in;
    o.add(r->counts, E * 4, "counts");
    o.add(r->offsets, (E + 1) * 4, "offsets");
    o.add(r->dest, A * 4, "dest");
    o.add(r->src, A * 4, "src");
    o.add(ws, ws_bytes, "workspace");
    in.add(r->topk_idx, A * 4, "topk_idx");
    if (int st = check_alias(o, in)) return st;
  }
  return launch_dispatch(desc, r->topk_idx, r->counts, r->offsets, r->dest, r->src, ws, L,
                         static_cast<hipStream_t>(stream));
}

int moe_mx_ffn_up(const moe_mx_desc* desc, const void* x, const int32_t* src, const int32_t* offsets,
                  const moe_mx_weights* w, void* h, void* ws, size_t ws_bytes, void* stream) {
  if (int st = validate_mx(desc)) return st;
  MOE_REQUIRE_PTR(x, "x");
  MOE_OPTIONAL_PTR(src, "src");
  MOE_REQUIRE_PTR(offsets, "offsets");
  MOE_REQUIRE_PTR(h, "h");
  if (int st = validate_weights(desc, w, true, false)) return st;
  MxLayout L;
  if (int st = check_ws(desc, ws, ws_bytes, 0, L)) return st;
  const size_t A = (size_t)desc->tokens * desc->top_k;
  {
    Spans o, in;
    o.add(h, A * desc->d_ff * 2, "h");
    o.add(ws, ws_bytes, "workspace");
    in.add(x, (src ? (size_t)desc->tokens : A) * desc->d_model * 2, "x");
    in.add(src, A * 4, "src");
    in.add(offsets, (size_t)(desc->n_experts + 1) * 4, "offsets");
    add_weights(in, desc, w, true, false);
    if (int st = check_alias(o, in)) return st;
  }
  return launch_product(desc, true, x, src, offsets, w, h, ws, L, static_cast<hipStream_t>(stream));
}

int moe_mx_ffn_down(const moe_mx_desc* desc, const void* h, const int32_t* offsets,
                    const moe_mx_weights* w, float* o, void* ws, size_t ws_bytes, void* stream) {
  if (int st = validate_mx(desc)) return st;
  MOE_REQUIRE_PTR(h, "h");
  MOE_REQUIRE_PTR(offsets, "offsets");
  MOE_REQUIRE_PTR(o, "o");
  if (int st = validate_weights(desc, w, false, true)) return st;
  MxLayout L;
  if (int st = check_ws(desc, ws, ws_bytes, 0, L)) return st;
  const size_t A = (size_t)desc->tokens * desc->top_k;
  {
    Spans out, in;
    out.add(o, A * desc->d_model * 4, "o");
    out.add(ws, ws_bytes, "workspace");
    in.add(h, A * desc->d_ff * 2, "h");
    in.add(offsets, (size_t)(desc->n_experts + 1) * 4, "offsets");
    add_weights(in, desc, w, false, true);
    if (int st = check_alias(out, in)) return st;
  }
  return launch_product(desc, false, h, nullptr, offsets, w, o, ws, L, static_cast<hipStream_t>(stream));
}

int moe_mx_forward(const moe_score_desc* route, const moe_mx_desc* desc, const void* x,
                   const void* w_router, const float* b_router, const float* b_select,
                   const moe_mx_weights* w, float* y, moe_score_out* out, void* ws, size_t ws_bytes,
                   void* stream) {
  size_t route_bytes = 0;
  if (int st = moe_score_workspace_size(route, &route_bytes)) return st;
  if (int st = validate_mx(desc)) return st;
  if (int st = validate_pairing(route, desc)) return st;
  MOE_REQUIRE_PTR(x, "x");
  MOE_REQUIRE_PTR(y, "y");
  if (int st = validate_weights(desc, w, true, true)) return st;
  MxLayout L;
  if (int st = check_ws(desc, ws, ws_bytes, route_bytes, L)) return st;
  const size_t T = desc->tokens, D = desc->d_model, E = desc->n_experts;
  moe_score_out r{};
  if (out) r = *out;
  {
    // y against everything else; the router's own call checks its arguments (its outputs
    // against the expert weights here).
    Spans o, in;
    o.add(y, T * D * 4, "y");
    o.add(r.topk_idx, T * desc->top_k * 4, "topk_idx");
    o.add(r.topk_w, T * desc->top_k * 4, "topk_w");
    o.add(r.logits, T * E * 4, "logits");
    o.add(r.load, E * 4, "load");
    o.add(r.prob_mean, E * 4, "prob_mean");
    o.add(r.aux, 4, "aux");
    o.add(r.z_loss, 4, "z_loss");
    o.add(ws, ws_bytes, "workspace");
    in.add(x, T * D * 2, "x");
    in.add(w_router, E * D * 2, "w_router");
    in.add(b_router, E * 4, "b_router");
    in.add(b_select, E * 4, "b_select");
    add_weights(in, desc, w, true, true);
    if (int st = check_alias(o, in)) return st;
  }
  return run_layer(route, desc, x, w_router, b_router, b_select, w, nullptr, y, r, ws, L, route_bytes, stream);
}

int moe_mx_block_workspace_size(const moe_mx_block* block, size_t* bytes) {
  BlockLayout B;
  if (int st = validate_block(block, B)) return st;
  if (!bytes) return fail(MOE_ERR_INVALID, "bytes must not be NULL");
  *bytes = B.total;
  return ok();
}

int moe_mx_block_forward(const moe_mx_block* block, const moe_rows* x, const moe_rows* add, const moe_rows* x_out,
                         float* y, moe_score_out* out, void* ws, size_t ws_bytes, void* stream) {
  BlockLayout B;
  if (int st = validate_block(block, B)) return st;
  const moe_mx_block& b = *block;
  const moe_mx_desc* desc = b.experts;
  const size_t T = desc->tokens, D = desc->d_model, E = desc->n_experts;
  // Everything is checked before the first launch: no call below then finds a fault.
  auto rows = [&](const moe_rows* r, const char* name, bool needed) -> int {
    if (!r || !r->data) return needed ? fail(MOE_ERR_INVALID, "%s must not be NULL", name) : MOE_OK;
    if (!aligned16(r->data)) return fail(MOE_ERR_INVALID, "%s must be 16-byte aligned", name);
    if (T > 1 && r->stride < (int64_t)D) return fail(MOE_ERR_INVALID, "%s: stride must be >= d", name);
    if (T > 1 && r->stride > (int64_t(1) << 40) / (int64_t)T)
      return fail(MOE_ERR_UNSUPPORTED, "%s: rows * stride must be <= 2^40", name);
    return MOE_OK;
  };
  if (int st = rows(x, "x", true)) return st;
  if (int st = rows(add, "add", false)) return st;
  if (int st = rows(x_out, "x_out", false)) return st;
  MOE_OPTIONAL_PTR(b.weight, "weight");
  MOE_OPTIONAL_PTR(b.bias, "bias");
  MOE_REQUIRE_PTR(b.w_router, "w_router");
  MOE_OPTIONAL_PTR(b.b_router, "b_router");
  MOE_OPTIONAL_PTR(b.b_select, "b_select");
  if (int st = validate_weights(desc, b.w, true, true)) return st;
  MOE_REQUIRE_PTR(y, "y");
  moe_score_out r{};
  if (out) r = *out;
  MOE_OPTIONAL_PTR(r.topk_idx, "out->topk_idx");
  MOE_OPTIONAL_PTR(r.topk_w, "out->topk_w");
  MOE_OPTIONAL_PTR(r.logits, "out->logits");
  MOE_OPTIONAL_PTR(r.load, "out->load");
  MOE_OPTIONAL_PTR(r.prob_mean, "out->prob_mean");
  MOE_OPTIONAL_PTR(r.aux, "out->aux");
  MOE_OPTIONAL_PTR(r.z_loss, "out->z_loss");
  if (b.up) {
    MOE_REQUIRE_PTR(b.adapter, "adapter");
    const moe_lora_weights* both[2] = {b.w_up, b.w_down};
    const moe_lora_desc* of[2] = {b.up, b.down};
    for (int i = 0; i < 2; ++i) {
      const moe_lora_weights* w = both[i];
      if (!w) return fail(MOE_ERR_INVALID, "w_up and w_down must not be NULL");
      MOE_REQUIRE_PTR(w->w, "w");
      MOE_REQUIRE_PTR(w->a, "a");
      MOE_REQUIRE_PTR(w->b, "b");
      MOE_OPTIONAL_PTR(w->scale, "scale");
      if (of[i]->has_bias) MOE_REQUIRE_PTR(w->bias, "bias");
      if (!of[i]->has_bias && w->bias) return fail(MOE_ERR_INVALID, "bias given but has_bias == 0");
    }
  }
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace must not be NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (ws_bytes < B.total) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, B.total);
  {
    auto reach = [&](const moe_rows* m, size_t e) { return m && m->data ? (T - 1) * (size_t)m->stride * e + D * e : 0; };
    auto data = [](const moe_rows* m) -> const void* { return m ? m->data : nullptr; };
    const size_t pe = b.norm->param_dtype == MOE_DTYPE_BF16 ? 2 : 4, ae = b.norm->add_dtype == MOE_DTYPE_BF16 ? 2 : 4;
    Spans o, in, xo;
    o.add(y, T * D * 4, "y");
    xo.add(data(x_out), T > 1 ? reach(x_out, 2) : D * 2, "x_out");
    o.add(r.topk_idx, T * desc->top_k * 4, "topk_idx");
    o.add(r.topk_w, T * desc->top_k * 4, "topk_w");
    o.add(r.logits, T * E * 4, "logits");
    o.add(r.load, E * 4, "load");
    o.add(r.prob_mean, E * 4, "prob_mean");
    o.add(r.aux, 4, "aux");
    o.add(r.z_loss, 4, "z_loss");
    o.add(ws, ws_bytes, "workspace");
    in.add(b.weight, D * pe, "weight");
    in.add(b.bias, D * pe, "bias");
    in.add(b.w_router, E * D * 2, "w_router");
    in.add(b.b_router, E * 4, "b_router");
    in.add(b.b_select, E * 4, "b_select");
    add_weights(in, desc, b.w, true, true);
    if (b.up) {
      in.add(b.adapter, T * 4, "adapter");
      const moe_lora_weights* both[2] = {b.w_up, b.w_down};
      const moe_lora_desc* of[2] = {b.up, b.down};
      for (int i = 0; i < 2; ++i) {
        const size_t N = of[i]->n_adapters, rank = of[i]->rank, n = of[i]->d_out, k = of[i]->d_in;
        in.add(both[i]->w, n * k * 2, "w");
        in.add(both[i]->bias, n * 2, "bias");
        in.add(both[i]->a, N * rank * k * 2, "a");
        in.add(both[i]->b, N * rank * n * 2, "b");
        in.add(both[i]->scale, N * 4, "scale");
      }
    }
    // x_out may lie beside x and add in one buffer's rows: moe_layer_norm, the first launch, tells them apart.
    if (int st = check_alias(xo, in)) return st;
    in.add(data(x), T > 1 ? reach(x, 2) : D * 2, "x");
    in.add(data(add), T > 1 ? reach(add, ae) : D * ae, "add");
    in.add(data(x_out), T > 1 ? reach(x_out, 2) : D * 2, "x_out");
    if (int st = check_alias(o, in)) return st;
  }
  void* xn = at<void>(ws, B.xn);
  const moe_rows normed{xn, (int64_t)D};
  if (int st = moe_layer_norm(b.norm, x, add, b.weight, b.bias, x_out, &normed, nullptr, nullptr, stream)) return st;
  float* shared = nullptr;
  if (b.up) {
    shared = at<float>(ws, B.shared);
    if (int st = moe_lora_shared_ffn(b.up, b.down, xn, b.adapter, b.w_up, b.w_down, shared, at<void>(ws, B.lora),
                                     B.lora_bytes, stream))
      return st;
  }
  return run_layer(b.route, desc, xn, b.w_router, b.b_router, b.b_select, b.w, shared, y, r, at<void>(ws, B.layer),
                   layout_of(desc), B.route_bytes, stream);
}

}  // extern "C"
