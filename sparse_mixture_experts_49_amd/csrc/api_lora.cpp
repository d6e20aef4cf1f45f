// C ABI of the shared projection with low-rank adapters: validation, workspace, launches.
#include <limits>

#include "api_util.h"
#include "lora.h"

using namespace moe::api;

namespace {

int validate_lora(const moe_lora_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID, "desc must not be NULL");
  if (d->tokens < 1) return fail(MOE_ERR_INVALID, "tokens must be >= 1 (got %d)", d->tokens);
  if (d->d_in < 1 || d->d_out < 1) return fail(MOE_ERR_INVALID, "d_in and d_out must be >= 1");
  if (d->d_in % 128 || d->d_out % 128)
    return fail(MOE_ERR_UNSUPPORTED, "d_in (%d) and d_out (%d) must be multiples of 128", d->d_in, d->d_out);
  if (d->rank < 1) return fail(MOE_ERR_INVALID, "rank must be >= 1 (got %d)", d->rank);
  if (d->rank % 8 || d->rank > moe::kLoraMaxRank)
    return fail(MOE_ERR_UNSUPPORTED, "rank must be a multiple of 8 and <= %d (got %d)", moe::kLoraMaxRank, d->rank);
  if (d->n_adapters < 1) return fail(MOE_ERR_INVALID, "n_adapters must be >= 1 (got %d)", d->n_adapters);
  if (d->n_adapters > moe::kLoraMaxAdapters)
    return fail(MOE_ERR_UNSUPPORTED, "n_adapters must be <= %d (got %d)", moe::kLoraMaxAdapters, d->n_adapters);
  if (d->act != MOE_LORA_ACT_NONE && d->act != MOE_LORA_ACT_GELU)
    return fail(MOE_ERR_INVALID, "act must be MOE_LORA_ACT_NONE or MOE_LORA_ACT_GELU");
  if (d->out_dtype != MOE_DTYPE_F32 && d->out_dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_INVALID, "out_dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  if (d->has_bias != 0 && d->has_bias != 1) return fail(MOE_ERR_INVALID, "has_bias must be 0 or 1");
  const long long most = std::numeric_limits<int32_t>::max();
  const long long widest = d->d_in > d->d_out ? d->d_in : d->d_out;
  if (d->tokens * widest > most) return fail(MOE_ERR_UNSUPPORTED, "tokens * max(d_in, d_out) exceeds int32");
  if ((long long)d->d_in * d->d_out > most) return fail(MOE_ERR_UNSUPPORTED, "d_in * d_out exceeds int32");
  return MOE_OK;
}

moe::LoraShape shape_of(const moe_lora_desc* d) {
  return {d->tokens, d->d_in, d->d_out, d->rank, d->n_adapters, d->act == MOE_LORA_ACT_GELU,
          d->out_dtype == MOE_DTYPE_F32};
}

int check_ws(void* ws, size_t bytes, size_t need) {
  if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace must not be NULL");
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", bytes, need);
  return MOE_OK;
}

int validate_weights(const moe_lora_desc* d, const moe_lora_weights* w, const char* which) {
  if (!w) return fail(MOE_ERR_INVALID, "%s must not be NULL", which);
  MOE_REQUIRE_PTR(w->w, "w");
  MOE_REQUIRE_PTR(w->a, "a");
  MOE_REQUIRE_PTR(w->b, "b");
  MOE_OPTIONAL_PTR(w->scale, "scale");
  if (d->has_bias) MOE_REQUIRE_PTR(w->bias, "bias");
  if (!d->has_bias && w->bias) return fail(MOE_ERR_INVALID, "bias given but has_bias == 0");
  return MOE_OK;
}

void add_weights(Spans& in, const moe_lora_desc* d, const moe_lora_weights* w) {
  const size_t N = d->n_adapters, r = d->rank;
  in.add(w->w, (size_t)d->d_in * d->d_out * 2, "w");
  in.add(w->bias, (size_t)d->d_out * 2, "bias");
  in.add(w->a, N * r * d->d_in * 2, "a");
  in.add(w->b, N * r * d->d_out * 2, "b");
  in.add(w->scale, N * 4, "scale");
}

size_t out_bytes(const moe_lora_desc* d) {
  return (size_t)d->tokens * d->d_out * (d->out_dtype == MOE_DTYPE_F32 ? 4 : 2);
}

int launch(const moe_lora_desc* d, const void* x, const int32_t* adapter, const moe_lora_weights* w, void* y,
           void* u, void* stream) {
  moe::LoraArgs a{};
  a.sh = shape_of(d);
  a.x = static_cast<const uint16_t*>(x);
  a.adapter = adapter;
  a.w = static_cast<const uint16_t*>(w->w);
  a.bias = static_cast<const uint16_t*>(w->bias);
  a.a = static_cast<const uint16_t*>(w->a);
  a.b = static_cast<const uint16_t*>(w->b);
  a.scale = w->scale;
  a.y = y;
  a.u = u;
  return hip_status(moe::launch_lora(a, static_cast<hipStream_t>(stream)), "adapter projection launch");
}

// The two products of a shared expert as descriptors; h lies between them.
int validate_pair(const moe_lora_desc* up, const moe_lora_desc* down) {
  if (int st = validate_lora(up)) return st;
  if (int st = validate_lora(down)) return st;
  if (up->tokens != down->tokens || up->d_out != down->d_in || up->d_in != down->d_out)
    return fail(MOE_ERR_INVALID, "up and down differ in tokens, or up's widths are not down's reversed");
  if (up->act != MOE_LORA_ACT_GELU || up->out_dtype != MOE_DTYPE_BF16)
    return fail(MOE_ERR_INVALID, "up must have act MOE_LORA_ACT_GELU and out_dtype MOE_DTYPE_BF16");
  if (down->act != MOE_LORA_ACT_NONE || down->out_dtype != MOE_DTYPE_F32)
    return fail(MOE_ERR_INVALID, "down must have act MOE_LORA_ACT_NONE and out_dtype MOE_DTYPE_F32");
  return MOE_OK;
}

size_t u_bytes(const moe_lora_desc* d) { return up256(moe::lora_u_bytes(shape_of(d))); }
size_t h_bytes(const moe_lora_desc* up) { return up256(out_bytes(up)); }

}  // namespace

extern "C" {

int moe_lora_workspace_size(const moe_lora_desc* desc, size_t* bytes) {
  if (int st = validate_lora(desc)) return st;
  if (!bytes) return fail(MOE_ERR_INVALID, "bytes must not be NULL");
  *bytes = u_bytes(desc);
  return ok();
}

int moe_lora_linear(const moe_lora_desc* desc, const void* x, const int32_t* adapter, const moe_lora_weights* w,
                    void* y, void* ws, size_t ws_bytes, void* stream) {
  if (int st = validate_lora(desc)) return st;
  MOE_REQUIRE_PTR(x, "x");
  MOE_REQUIRE_PTR(adapter, "adapter");
  if (int st = validate_weights(desc, w, "weights")) return st;
  MOE_REQUIRE_PTR(y, "y");
  if (int st = check_ws(ws, ws_bytes, u_bytes(desc))) return st;
  {
    Spans out, in;
    out.add(y, out_bytes(desc), "y");
    out.add(ws, ws_bytes, "workspace");
    in.add(x, (size_t)desc->tokens * desc->d_in * 2, "x");
    in.add(adapter, (size_t)desc->tokens * 4, "adapter");
    add_weights(in, desc, w);
    if (int st = check_alias(out, in)) return st;
  }
  return launch(desc, x, adapter, w, y, ws, stream);
}

int moe_lora_shared_workspace_size(const moe_lora_desc* up, const moe_lora_desc* down, size_t* bytes) {
  if (int st = validate_pair(up, down)) return st;
  if (!bytes) return fail(MOE_ERR_INVALID, "bytes must not be NULL");
  *bytes = h_bytes(up) + (u_bytes(up) > u_bytes(down) ? u_bytes(up) : u_bytes(down));
  return ok();
}

int moe_lora_shared_ffn(const moe_lora_desc* up, const moe_lora_desc* down, const void* x, const int32_t* adapter,
                        const moe_lora_weights* w_up, const moe_lora_weights* w_down, float* o_shared, void* ws,
                        size_t ws_bytes, void* stream) {
  size_t need = 0;
  if (int st = moe_lora_shared_workspace_size(up, down, &need)) return st;
  MOE_REQUIRE_PTR(x, "x");
  MOE_REQUIRE_PTR(adapter, "adapter");
  if (int st = validate_weights(up, w_up, "w_up")) return st;
  if (int st = validate_weights(down, w_down, "w_down")) return st;
  MOE_REQUIRE_PTR(o_shared, "o_shared");
  if (int st = check_ws(ws, ws_bytes, need)) return st;
  {
    Spans out, in;
    out.add(o_shared, out_bytes(down), "o_shared");
    out.add(ws, ws_bytes, "workspace");
    in.add(x, (size_t)up->tokens * up->d_in * 2, "x");
    in.add(adapter, (size_t)up->tokens * 4, "adapter");
    add_weights(in, up, w_up);
    add_weights(in, down, w_down);
    if (int st = check_alias(out, in)) return st;
  }
  void* u = at<void>(ws, h_bytes(up));
  if (int st = launch(up, x, adapter, w_up, ws, u, stream)) return st;
  return launch(down, ws, adapter, w_down, o_shared, u, stream);
}

}  // extern "C"
