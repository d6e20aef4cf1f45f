// C ABI of the layer norm: argument validation, workspace carving, launches.
#include <cmath>

#include "api_util.h"
#include "norm.h"

using namespace moe::api;

namespace {

bool dtype_ok(int dtype) { return dtype == MOE_DTYPE_F32 || dtype == MOE_DTYPE_BF16; }
size_t elem(int dtype) { return dtype == MOE_DTYPE_BF16 ? 2 : 4; }

int validate_norm(const moe_norm_desc* d) {
  if (!d) return fail(MOE_ERR_INVALID, "desc must not be NULL");
  if (d->rows < 0) return fail(MOE_ERR_INVALID, "rows must be >= 0 (got %lld)", (long long)d->rows);
  if (d->d < 1) return fail(MOE_ERR_INVALID, "d must be >= 1 (got %d)", d->d);
  if (d->d > moe::kNormMaxWidth)
    return fail(MOE_ERR_UNSUPPORTED, "d must be <= %d (got %d)", moe::kNormMaxWidth, d->d);
  if (d->rows > (int64_t(1) << 40) / d->d)
    return fail(MOE_ERR_UNSUPPORTED, "rows * d must be <= 2^40 (got %lld x %d)", (long long)d->rows, d->d);
  if (!dtype_ok(d->dtype) || !dtype_ok(d->param_dtype) || !dtype_ok(d->add_dtype))
    return fail(MOE_ERR_INVALID, "dtype, param_dtype and add_dtype must be MOE_DTYPE_F32 or MOE_DTYPE_BF16");
  if (!std::isfinite(d->eps) || d->eps < 0.f) return fail(MOE_ERR_INVALID, "eps must be finite and >= 0");
  return MOE_OK;
}

moe::NormShape shape_of(const moe_norm_desc* d) {
  return {d->rows, d->d, d->dtype == MOE_DTYPE_BF16, d->param_dtype == MOE_DTYPE_BF16,
          d->add_dtype == MOE_DTYPE_BF16, d->eps};
}

size_t need_of(const moe_norm_desc* d) {
  const size_t n = up256(moe::norm_grad_part_bytes(shape_of(d)));
  return n ? n : 256;
}

// A matrix argument: its rows' bytes and the distance between them.
struct Matrix {
  uintptr_t p;
  size_t row, pitch;
  int64_t rows;
  const char* name;
};

size_t reach(const Matrix& m) { return m.rows ? (size_t)(m.rows - 1) * m.pitch + m.row : 0; }

// Whether two matrices share a byte.  Rows of the same pitch may lie side by side in one
// buffer (columns of a wider matrix); otherwise the whole ranges count.
bool share(const Matrix& a, const Matrix& b) {
  if (!a.p || !b.p || !a.rows || !b.rows) return false;
  if (a.p >= b.p + reach(b) || b.p >= a.p + reach(a)) return false;
  if (a.pitch != b.pitch || a.rows <= 1 || b.rows <= 1) return true;
  const uintptr_t off = a.p > b.p ? (a.p - b.p) % a.pitch : (b.p - a.p) % a.pitch;
  const size_t first = a.p > b.p ? b.row : a.row, second = a.p > b.p ? a.row : b.row;
  return off < first || off + second > a.pitch;
}

struct Matrices {
  Matrix m[12];
  int n = 0;
};

int add_matrix(Matrices& to, const moe_rows* r, const moe_norm_desc* d, int dtype, const char* name, bool needed,
               bool& given) {
  given = r && r->data;
  if (!given) return needed && d->rows > 0 ? fail(MOE_ERR_INVALID, "%s must not be NULL", name) : MOE_OK;
  if (!aligned16(r->data)) return fail(MOE_ERR_INVALID, "%s must be 16-byte aligned", name);
  if (d->rows > 1) {
    if (r->stride < d->d)
      return fail(MOE_ERR_INVALID, "%s: stride must be >= d (got %lld)", name, (long long)r->stride);
    if (r->stride > (int64_t(1) << 40) / d->rows)
      return fail(MOE_ERR_UNSUPPORTED, "%s: rows * stride must be <= 2^40", name);
  }
  to.m[to.n++] = Matrix{reinterpret_cast<uintptr_t>(r->data), (size_t)d->d * elem(dtype),
                        d->rows > 1 ? (size_t)r->stride * elem(dtype) : (size_t)d->d * elem(dtype), d->rows, name};
  return MOE_OK;
}

void add_vector(Matrices& to, const void* p, size_t bytes, const char* name) {
  if (p && bytes) to.m[to.n++] = Matrix{reinterpret_cast<uintptr_t>(p), bytes, bytes, 1, name};
}

int check_apart(const Matrices& outs, const Matrices& ins) {
  for (int i = 0; i < outs.n; ++i) {
    for (int j = i + 1; j < outs.n; ++j)
      if (share(outs.m[i], outs.m[j]))
        return fail(MOE_ERR_INVALID, "%s overlaps %s", outs.m[i].name, outs.m[j].name);
    for (int j = 0; j < ins.n; ++j)
      if (share(outs.m[i], ins.m[j]))
        return fail(MOE_ERR_INVALID, "%s overlaps %s", outs.m[i].name, ins.m[j].name);
  }
  return MOE_OK;
}

template <typename P>
moe::Rows<P> rows_of(const moe_rows* r, bool given) {
  return given ? moe::Rows<P>{r->data, r->stride} : moe::Rows<P>{nullptr, 0};
}

}  // namespace

extern "C" {

int moe_norm_workspace_size(const moe_norm_desc* desc, size_t* bytes) {
  if (int st = validate_norm(desc)) return st;
  if (!bytes) return fail(MOE_ERR_INVALID, "bytes must not be NULL");
  *bytes = need_of(desc);
  return ok();
}

int moe_layer_norm(const moe_norm_desc* desc, const moe_rows* x, const moe_rows* add, const void* weight,
                   const void* bias, const moe_rows* x_out, const moe_rows* y, float* mean, float* rstd,
                   void* stream) {
  if (int st = validate_norm(desc)) return st;
  Matrices out, in;
  bool has_x, has_add, has_out, has_y;
  if (int st = add_matrix(in, x, desc, desc->dtype, "x", true, has_x)) return st;
  if (int st = add_matrix(in, add, desc, desc->add_dtype, "add", false, has_add)) return st;
  if (int st = add_matrix(out, x_out, desc, desc->dtype, "x_out", false, has_out)) return st;
  if (int st = add_matrix(out, y, desc, desc->dtype, "y", true, has_y)) return st;
  MOE_OPTIONAL_PTR(weight, "weight");
  MOE_OPTIONAL_PTR(bias, "bias");
  MOE_OPTIONAL_PTR(mean, "mean");
  MOE_OPTIONAL_PTR(rstd, "rstd");
  add_vector(in, weight, (size_t)desc->d * elem(desc->param_dtype), "weight");
  add_vector(in, bias, (size_t)desc->d * elem(desc->param_dtype), "bias");
  add_vector(out, mean, (size_t)desc->rows * 4, "mean");
  add_vector(out, rstd, (size_t)desc->rows * 4, "rstd");
  if (int st = check_apart(out, in)) return st;
  moe::NormArgs a{};
  a.sh = shape_of(desc);
  a.x = rows_of<const void>(x, has_x);
  a.add = rows_of<const void>(add, has_add);
  a.weight = weight;
  a.bias = bias;
  a.x_out = rows_of<void>(x_out, has_out);
  a.y = rows_of<void>(y, has_y);
  a.mean = mean;
  a.rstd = rstd;
  return hip_status(moe::launch_norm(a, static_cast<hipStream_t>(stream)), "layer norm launch");
}

int moe_layer_norm_backward(const moe_norm_desc* desc, const moe_rows* dy, const moe_rows* x, const void* weight,
                            const float* mean, const float* rstd, const moe_rows* d_x_out, const moe_rows* d_x,
                            float* d_weight, float* d_bias, void* ws, size_t ws_bytes, void* stream) {
  if (int st = validate_norm(desc)) return st;
  Matrices out, in;
  bool has_dy, has_x, has_res, has_dx;
  if (int st = add_matrix(in, dy, desc, desc->dtype, "dy", true, has_dy)) return st;
  if (int st = add_matrix(in, x, desc, desc->dtype, "x", true, has_x)) return st;
  if (int st = add_matrix(in, d_x_out, desc, desc->dtype, "d_x_out", false, has_res)) return st;
  if (int st = add_matrix(out, d_x, desc, desc->dtype, "d_x", false, has_dx)) return st;
  MOE_OPTIONAL_PTR(weight, "weight");
  if (desc->rows > 0) {
    MOE_REQUIRE_PTR(mean, "mean");
    MOE_REQUIRE_PTR(rstd, "rstd");
  }
  MOE_OPTIONAL_PTR(d_weight, "d_weight");
  MOE_OPTIONAL_PTR(d_bias, "d_bias");
  if (desc->rows > 0 && !has_dx && !d_weight && !d_bias) return fail(MOE_ERR_INVALID, "d_x, d_weight and d_bias are all NULL");
  if (has_res && !has_dx) return fail(MOE_ERR_INVALID, "d_x_out given without d_x");
  const size_t need = need_of(desc);
  if (d_weight || d_bias) {
    if (!ws) return fail(MOE_ERR_WORKSPACE, "workspace must not be NULL");
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
      return fail(MOE_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (ws_bytes < need) return fail(MOE_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    add_vector(out, ws, ws_bytes, "workspace");
  }
  add_vector(in, weight, (size_t)desc->d * elem(desc->param_dtype), "weight");
  add_vector(in, mean, (size_t)desc->rows * 4, "mean");
  add_vector(in, rstd, (size_t)desc->rows * 4, "rstd");
  add_vector(out, d_weight, (size_t)desc->d * 4, "d_weight");
  add_vector(out, d_bias, (size_t)desc->d * 4, "d_bias");
  if (int st = check_apart(out, in)) return st;
  moe::NormGradArgs a{};
  a.sh = shape_of(desc);
  a.dy = rows_of<const void>(dy, has_dy);
  a.x = rows_of<const void>(x, has_x);
  a.d_x_out = rows_of<const void>(d_x_out, has_res);
  a.weight = weight;
  a.mean = mean;
  a.rstd = rstd;
  a.d_x = rows_of<void>(d_x, has_dx);
  a.d_weight = d_weight;
  a.d_bias = d_bias;
  a.part = static_cast<float*>(ws);
  return hip_status(moe::launch_norm_grad(a, static_cast<hipStream_t>(stream)), "layer norm backward launch");
}

}  // extern "C"
