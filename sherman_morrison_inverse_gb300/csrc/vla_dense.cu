// C entry points of the products and layer norms: argument checks and dispatch.
#include "vla.h"
#include "vla_dense.cuh"
#include "vla_handle.cuh"

#include <exception>

using namespace vla::api;

namespace {

constexpr long long kMaxWidth = 32768;          // D of the norm
constexpr long long kMaxSide = 1LL << 30;       // M, N, K of a product: tiles and coordinates are 32-bit

template <typename... P>
bool to_values(size_t size, P... p) { return ((reinterpret_cast<uintptr_t>(p) | ...) & (size - 1)) == 0; }
size_t size_of(vla_dtype_t t) { return t == VLA_BF16 ? 2 : 4; }
size_t size_of(vla_mat_t t) { return t == VLA_MAT_F32 ? 4 : t == VLA_MAT_BF16 ? 2 : 1; }
bool known(vla_dtype_t t) { return t == VLA_F32 || t == VLA_BF16; }
bool stride_ok(long long v) { return v >= 0 && v < (1LL << 40); }
bool rows_apart(long long n, long long row, long long width) { return n <= 1 || row >= width; }
// Whether an output starts where none of the others does: the overlap that a call is likely to have by mistake.
template <typename... P>
bool elsewhere(const void* out, P... p) { return !out || ((out != static_cast<const void*>(p)) && ...); }

vla_err_t check_sizes(vla_handle_t h, const std::string& f, long long M, long long N, long long K) {
  if (M < 0 || N < 0 || K < 0) return fail(h, VLA_ERR_INVALID_ARG, f + ": negative size");
  if (M > kMaxSide || N > kMaxSide || K > kMaxSide)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": sizes must be at most 2^30");
  return VLA_OK;
}

vla_err_t check_strides(vla_handle_t h, const std::string& f, const long long* rows, int n) {
  if (!rows) return fail(h, VLA_ERR_INVALID_ARG, f + ": NULL pointer");
  for (int i = 0; i < n; ++i)
    if (!stride_ok(rows[i])) return fail(h, VLA_ERR_INVALID_ARG, f + ": stride out of range");
  return VLA_OK;
}

vla_err_t check_ws(vla_handle_t h, const std::string& f, const void* ws, size_t have, size_t need) {
  if (need > 0 && (!ws || have < need || !aligned16(ws)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": workspace missing, misaligned or smaller than " + f + "_workspace says");
  return VLA_OK;
}

vla_err_t check_types(vla_handle_t h, const std::string& f, vla_mat_t in, vla_dtype_t out) {
  if (in != VLA_MAT_F32 && in != VLA_MAT_BF16 && in != VLA_MAT_E4M3)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown operand type");
  if (!known(out)) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown output type");
  if (in == VLA_MAT_F32 && out != VLA_F32)
    return fail(h, VLA_ERR_UNSUPPORTED, f + ": float32 operands have a float32 result");
  return VLA_OK;
}

size_t up16(size_t n) { return (n + 15) / 16 * 16; }

vla::ProductArgs linear_product(vla_handle_t h, const void* x, const void* w, long long M, long long N, long long K,
                                const long long* rows) {
  vla::ProductArgs p{};
  p.a = x; p.b = w;
  p.M = M; p.N = N; p.Kd = K;
  p.a_row = rows[0]; p.b_row = rows[1];
  p.sm_count = h->sm_count;
  p.status = h->status;
  p.wait_limit = h->wait_limit;
  return p;
}

// The two products of a gradient and what they share of the workspace: g, the partial sums of db.
struct BackPlan {
  vla::ProductArgs dx, dw, run[2];   // run: those that are asked for
  int count;
  vla::SlopeArgs slope;
  size_t g_bytes, part_bytes, ws_bytes;
};

BackPlan back_plan(vla_handle_t h, const void* dy, const void* x, const void* w, bool want_dx, bool want_dw, bool want_db,
                   long long M, long long N, long long K, const long long* rows, bool act, vla_dtype_t io) {
  BackPlan b{};
  const long long size = (long long)size_of(io);
  const bool need_g = act && (want_dx || want_dw);
  b.slope.M = M; b.slope.N = N; b.slope.dy_row = rows[0]; b.slope.pre_row = rows[3];
  b.slope.g_row = (N + 7) / 8 * 8;   // rows on 16-byte boundaries
  b.slope.sm_count = h->sm_count;
  b.g_bytes = need_g ? up16((size_t)(M * b.slope.g_row * size)) : 0;
  b.part_bytes = want_db ? up16(vla::slope_ws(M, N, h->sm_count)) : 0;
  // g's place in the workspace is not known yet: an aligned address that is not one
  const void* g = need_g ? reinterpret_cast<const void*>(uintptr_t{256}) : dy;
  const long long g_row = need_g ? b.slope.g_row : rows[0];
  b.dx.a = g; b.dx.a_row = g_row;
  b.dx.b = w; b.dx.b_row = rows[2]; b.dx.b_mn = true;
  b.dx.M = M; b.dx.N = K; b.dx.Kd = N;
  b.dw.a = g; b.dw.a_row = g_row; b.dw.a_mn = true;
  b.dw.b = x; b.dw.b_row = rows[1]; b.dw.b_mn = true;
  b.dw.M = N; b.dw.N = K; b.dw.Kd = M;
  b.dx.sm_count = b.dw.sm_count = h->sm_count;
  b.dx.status = b.dw.status = h->status;
  b.dx.wait_limit = b.dw.wait_limit = h->wait_limit;
  b.dx.out.y_bf16 = b.dw.out.y_bf16 = io == VLA_BF16;
  b.count = 0;
  if (want_dx) b.run[b.count++] = b.dx;
  if (want_dw) b.run[b.count++] = b.dw;
  b.ws_bytes = b.g_bytes + b.part_bytes;
  if (b.count) b.ws_bytes += vla::products_ws(b.run, b.count, io == VLA_BF16 ? VLA_MAT_BF16 : VLA_MAT_F32);
  return b;
}

}  // namespace

extern "C" {

vla_err_t vla_linear(vla_handle_t h, const void* x, const void* w, const float* x_scale, const float* w_scale,
                     const float* bias, const void* residual, void* pre, void* y, long long M, long long N, long long K,
                     const long long* rows, vla_act_t act, vla_mat_t in, vla_dtype_t out, void* workspace,
                     size_t workspace_bytes, void* stream) try {
  const std::string f = "vla_linear";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  vla_err_t err = check_types(h, f, in, out);
  if (err == VLA_OK) err = check_sizes(h, f, M, N, K);
  if (err != VLA_OK) return err;
  if (act != VLA_ACT_NONE && act != VLA_ACT_SILU && act != VLA_ACT_GELU)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown activation");
  if ((x_scale || w_scale) && in != VLA_MAT_E4M3)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": scales go with e4m3 operands");
  if (M == 0 || N == 0) return VLA_OK;
  if ((err = check_strides(h, f, rows, 5)) != VLA_OK) return err;
  if (!y || (K > 0 && (!x || !w))) return fail(h, VLA_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!to_values(size_of(in), x, w) || !to_values(size_of(out), residual, pre, y) || !to_values(4, x_scale, w_scale, bias))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": misaligned pointer");
  if (!rows_apart(M, rows[4], N) || (pre && !rows_apart(M, rows[3], N)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": rows of y or pre overlap");
  if (!elsewhere(y, pre) || !elsewhere(pre, residual) || (K > 0 && (!elsewhere(y, x, w) || !elsewhere(pre, x, w))))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": y and pre must not be an input (y may be the residual) or each other");
  if (residual == y && M > 1 && rows[2] != rows[4])
    return fail(h, VLA_ERR_INVALID_ARG, f + ": y may be the residual only with the same rows");
  vla::ProductArgs p = linear_product(h, x, w, M, N, K, rows);
  vla::Epilogue& o = p.out;
  o.x_scale = x_scale; o.w_scale = w_scale; o.bias = bias; o.residual = residual; o.pre = pre; o.y = y;
  o.res_row = rows[2]; o.pre_row = rows[3]; o.y_row = rows[4];
  o.act = act; o.y_bf16 = out == VLA_BF16;
  if ((err = check_ws(h, f, workspace, workspace_bytes, vla::products_ws(&p, 1, in))) != VLA_OK) return err;
  p.ws = workspace;
  cudaError_t e = on_device(h->device, [&]() { return vla::launch_products(&p, 1, in, static_cast<cudaStream_t>(stream)); });
  if (e != cudaSuccess) return fail(h, VLA_ERR_CUDA, cuda_msg("vla_linear: launch", e));
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_linear_workspace(vla_handle_t h, const void* x, const void* w, long long M, long long N, long long K,
                               const long long* rows, vla_mat_t in, vla_dtype_t out, size_t* bytes) try {
  const std::string f = "vla_linear_workspace";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (!bytes) return fail(h, VLA_ERR_INVALID_ARG, f + ": bytes is NULL");
  vla_err_t err = check_types(h, f, in, out);
  if (err == VLA_OK) err = check_sizes(h, f, M, N, K);
  if (err != VLA_OK) return err;
  *bytes = 0;
  if (M == 0 || N == 0) return VLA_OK;
  if ((err = check_strides(h, f, rows, 2)) != VLA_OK) return err;
  vla::ProductArgs p = linear_product(h, x, w, M, N, K, rows);
  p.out.y_bf16 = out == VLA_BF16;
  *bytes = vla::products_ws(&p, 1, in);
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_linear_backward(vla_handle_t h, const void* dy, const void* x, const void* w, const void* pre, void* dx,
                              void* dw, float* db, long long M, long long N, long long K, const long long* rows,
                              vla_act_t act, vla_dtype_t io_dtype, void* workspace, size_t workspace_bytes,
                              void* stream) try {
  const std::string f = "vla_linear_backward";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (!known(io_dtype)) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown io_dtype");
  if (act != VLA_ACT_NONE && act != VLA_ACT_SILU && act != VLA_ACT_GELU)
    return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown activation");
  vla_err_t err = check_sizes(h, f, M, N, K);
  if (err == VLA_OK) err = check_strides(h, f, rows, 6);
  if (err != VLA_OK) return err;
  if (M == 0 || K == 0) dx = nullptr;   // nothing to write
  if (N == 0 || K == 0) dw = nullptr;
  if (N == 0) db = nullptr;
  if (!dx && !dw && !db) return VLA_OK;
  const bool has_act = act != VLA_ACT_NONE, terms = M > 0 && N > 0;
  if (terms && (!dy || (has_act && !pre) || (dx && !w) || (dw && !x)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!to_values(size_of(io_dtype), dy, x, w, dx, dw) || !to_values(4, db) ||
      (has_act && !to_values(size_of(io_dtype), pre)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": misaligned pointer");
  if ((dx && !rows_apart(M, rows[4], K)) || (dw && !rows_apart(N, rows[5], K)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": rows of dx or dw overlap");
  if (terms && (!elsewhere(dx, dy, x, w, dw, has_act ? pre : nullptr) || !elsewhere(dw, dy, x, w, has_act ? pre : nullptr)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": dx and dw must not be an input or each other");
  BackPlan b = back_plan(h, dy, x, w, dx, dw, db, M, N, K, rows, has_act, io_dtype);
  if ((err = check_ws(h, f, workspace, workspace_bytes, b.ws_bytes)) != VLA_OK) return err;
  char* ws = static_cast<char*>(workspace);
  b.slope.dy = dy; b.slope.pre = has_act ? pre : nullptr; b.slope.act = act; b.slope.db = db;
  b.slope.partial = reinterpret_cast<float*>(ws + b.g_bytes);
  if (b.g_bytes) b.slope.g = ws;
  for (int i = 0; i < b.count; ++i) {
    vla::ProductArgs& p = b.run[i];
    if (b.g_bytes) p.a = ws;
    p.ws = ws + b.g_bytes + b.part_bytes;
    p.follows = terms && (b.g_bytes || db);
    p.out.y = p.a_mn ? dw : dx;
    p.out.y_row = rows[p.a_mn ? 5 : 4];
  }
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = io_dtype == VLA_BF16;
  const int mat = bf16 ? VLA_MAT_BF16 : VLA_MAT_F32;
  cudaError_t e = on_device(h->device, [&]() {
    cudaError_t r = cudaSuccess;
    if (terms && (b.g_bytes || db)) r = vla::launch_slope(b.slope, bf16, s);
    if (r == cudaSuccess && !terms && db) r = cudaMemsetAsync(db, 0, (size_t)N * 4, s);
    if (r == cudaSuccess && b.count) r = vla::launch_products(b.run, b.count, mat, s);
    return r;
  });
  if (e != cudaSuccess) return fail(h, VLA_ERR_CUDA, cuda_msg("vla_linear_backward: launch", e));
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_linear_backward_workspace(vla_handle_t h, const void* dy, const void* x, const void* w, int dx, int dw,
                                        int db, long long M, long long N, long long K, const long long* rows,
                                        vla_act_t act, vla_dtype_t io_dtype, size_t* bytes) try {
  const std::string f = "vla_linear_backward_workspace";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (!bytes) return fail(h, VLA_ERR_INVALID_ARG, f + ": bytes is NULL");
  if (!known(io_dtype)) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown io_dtype");
  vla_err_t err = check_sizes(h, f, M, N, K);
  if (err == VLA_OK) err = check_strides(h, f, rows, 6);
  if (err != VLA_OK) return err;
  *bytes = back_plan(h, dy, x, w, dx && M && K, dw && N && K, db && N, M, N, K, rows, act != VLA_ACT_NONE, io_dtype).ws_bytes;
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_layer_norm(vla_handle_t h, const void* x, const float* w, const float* b, void* residual, void* y,
                         float* stats, long long rows, long long D, long long x_row, long long res_row, long long y_row,
                         float eps, vla_dtype_t io_dtype, vla_dtype_t res_dtype, void* stream) try {
  const std::string f = "vla_layer_norm";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (!known(io_dtype)) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown io_dtype");
  if (residual && !known(res_dtype)) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown res_dtype");
  if (!(eps >= 0.f)) return fail(h, VLA_ERR_INVALID_ARG, f + ": eps must be >= 0 (NaN rejected)");
  if (rows < 0 || D < 0) return fail(h, VLA_ERR_INVALID_ARG, f + ": negative size");
  if (!stride_ok(x_row) || !stride_ok(res_row) || !stride_ok(y_row))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": stride out of range");
  if (rows == 0 || D == 0) return VLA_OK;
  if (D > kMaxWidth) return fail(h, VLA_ERR_UNSUPPORTED, f + ": built for D up to 32768");
  if (!x || !w || !y) return fail(h, VLA_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!to_values(size_of(io_dtype), x, y) || !to_values(4, w, b, stats) || (residual && !to_values(size_of(res_dtype), residual)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": misaligned pointer");
  if (!rows_apart(rows, y_row, D) || (residual && !rows_apart(rows, res_row, D)))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": rows of y or the residual overlap");
  if (!elsewhere(y, residual)) return fail(h, VLA_ERR_INVALID_ARG, f + ": y must not be the residual");
  vla::LayerNormArgs a{};
  a.x = x; a.w = w; a.b = b; a.residual = residual; a.y = y; a.stats = stats;
  a.rows = rows; a.D = D; a.x_row = x_row; a.res_row = res_row; a.y_row = y_row;
  a.eps = eps; a.res_bf16 = res_dtype == VLA_BF16;
  a.sm_count = h->sm_count;
  cudaError_t e = on_device(h->device, [&]() {
    return vla::launch_layer_norm(a, io_dtype == VLA_BF16, static_cast<cudaStream_t>(stream));
  });
  if (e != cudaSuccess) return fail(h, VLA_ERR_CUDA, cuda_msg("vla_layer_norm: launch", e));
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_layer_norm_backward(vla_handle_t h, const void* dy, const void* x, const float* w, const float* stats,
                                  const void* dresidual, void* dx, float* dw, float* db, long long rows, long long D,
                                  const long long* strides, vla_dtype_t dy_dtype, vla_dtype_t x_dtype, void* workspace,
                                  size_t workspace_bytes, void* stream) try {
  const std::string f = "vla_layer_norm_backward";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (!known(dy_dtype) || !known(x_dtype)) return fail(h, VLA_ERR_INVALID_ARG, f + ": unknown type");
  if (rows < 0 || D < 0) return fail(h, VLA_ERR_INVALID_ARG, f + ": negative size");
  if (D == 0) return VLA_OK;
  vla_err_t err = check_strides(h, f, strides, 4);
  if (err != VLA_OK) return err;
  if (D > kMaxWidth) return fail(h, VLA_ERR_UNSUPPORTED, f + ": built for D up to 32768");
  if (!dw || (rows > 0 && (!dy || !x || !w || !stats || !dx))) return fail(h, VLA_ERR_INVALID_ARG, f + ": NULL pointer");
  if (!to_values(size_of(dy_dtype), dy) || !to_values(size_of(x_dtype), x, dresidual, dx) || !to_values(4, w, stats, dw, db))
    return fail(h, VLA_ERR_INVALID_ARG, f + ": misaligned pointer");
  if (!rows_apart(rows, strides[3], D)) return fail(h, VLA_ERR_INVALID_ARG, f + ": rows of dx overlap");
  if (rows > 0 && !elsewhere(dx, dy, x)) return fail(h, VLA_ERR_INVALID_ARG, f + ": dx must not be dy or x");
  if ((err = check_ws(h, f, workspace, workspace_bytes, rows ? vla::layer_norm_back_ws(rows, D, h->sm_count) : 0)) != VLA_OK) return err;
  vla::LayerNormBackArgs a{};
  a.dy = dy; a.x = x; a.w = w; a.stats = stats; a.dres = dresidual; a.dx = dx; a.dw = dw; a.db = db;
  a.partial = static_cast<float*>(workspace);
  a.rows = rows; a.D = D; a.dy_row = strides[0]; a.x_row = strides[1]; a.dres_row = strides[2]; a.dx_row = strides[3];
  a.sm_count = h->sm_count;
  a.status = h->status;
  a.wait_limit = h->wait_limit;
  cudaError_t e = on_device(h->device, [&]() {
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows > 0) return vla::launch_layer_norm_back(a, dy_dtype == VLA_BF16, x_dtype == VLA_BF16, s);
    cudaError_t r = cudaMemsetAsync(dw, 0, (size_t)D * 4, s);
    return r == cudaSuccess && db ? cudaMemsetAsync(db, 0, (size_t)D * 4, s) : r;
  });
  if (e != cudaSuccess) return fail(h, VLA_ERR_CUDA, cuda_msg("vla_layer_norm_backward: launch", e));
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

vla_err_t vla_layer_norm_backward_workspace(vla_handle_t h, long long rows, long long D, size_t* bytes) try {
  const std::string f = "vla_layer_norm_backward_workspace";
  if (!h) return fail(nullptr, VLA_ERR_INVALID_ARG, f + ": handle is NULL");
  h->last_error.clear();
  if (!bytes) return fail(h, VLA_ERR_INVALID_ARG, f + ": bytes is NULL");
  if (rows < 0 || D < 0) return fail(h, VLA_ERR_INVALID_ARG, f + ": negative size");
  *bytes = rows && D ? vla::layer_norm_back_ws(rows, D, h->sm_count) : 0;
  return VLA_OK;
} catch (const std::exception&) {   // no memory for a message
  return VLA_ERR_NOMEM;
}

}  // extern "C"
