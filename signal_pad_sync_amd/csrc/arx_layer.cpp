// arx_layer.cpp — host side of the layer operators declared in arx.h: argument
// checks, workspaces, launches. Nothing is kept between calls.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstdint>

#include "arx.h"
#include "arx_internal.h"
#include "arx_layer.h"

namespace {

using arx::Plane;
using arx::PlaneOut;
using arx::set_error;

constexpr size_t kMaxSize = 0x7FFFFFFF;
// Of the linear calls: a tile's rows lie within 32-bit offsets of each other,
// and a launch has fewer than 2^32 threads.
constexpr size_t kMaxTokens = (size_t)1 << 29, kMaxWidth = ((size_t)1 << 22) - 8;

size_t size_of(int dtype) { return dtype == ARX_F32 ? 4 : 2; }
size_t round_up(size_t n) { return (n + 255) & ~(size_t)255; }

// One operand of a call: a plane of rows, or a vector (one row).
struct Operand {
  const char* name;
  const void* p;
  size_t rows, cols, ld, size;
  bool output, in_place;  // in_place (inputs): an output may have just this place
};

// Bytes from the first element to the end of the last.
size_t extent(const Operand& o) { return ((o.rows - 1) * o.ld + o.cols) * o.size; }

bool overlaps(const Operand& a, const Operand& b) {
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  if (x + extent(a) <= y || y + extent(b) <= x) return false;
  // Column slices of one buffer lie between each other's rows: with one row
  // distance, rows meet only where their bytes do, modulo that distance.
  const size_t step = a.ld * a.size;
  if (a.rows > 1 && b.rows > 1 && step == b.ld * b.size) {
    const size_t off = y >= x ? (y - x) % step : (step - (x - y) % step) % step;
    if (off >= a.cols * a.size && off + b.cols * b.size <= step) return false;
  }
  return true;
}

// Shapes, alignment and overlaps of a call's operands; absent ones have a null
// address and are let pass, empty ones are not looked at.
template <size_t N>
int check(const Operand (&ops)[N]) {
  for (const Operand& o : ops) {
    if (!o.p) continue;
    if ((uintptr_t)o.p % o.size) return set_error(ARX_EINVAL, "%s is not aligned to its elements", o.name);
    if (o.rows > 1 && o.ld < o.cols)
      return set_error(ARX_EINVAL, "%s: row distance %zu below its %zu columns", o.name, o.ld, o.cols);
    if (o.ld > kMaxSize) return set_error(ARX_EINVAL, "%s: row distance %zu above %zu", o.name, o.ld, kMaxSize);
  }
  for (size_t i = 0; i < N; ++i) {
    const Operand& o = ops[i];
    if (!o.output || !o.p || o.rows == 0 || o.cols == 0) continue;
    for (size_t j = 0; j < N; ++j) {
      const Operand& q = ops[j];
      if (j == i || !q.p || q.rows == 0 || q.cols == 0 || (q.output && j < i)) continue;
      const bool same = q.p == o.p && q.rows == o.rows && q.cols == o.cols && q.size == o.size &&
                        (q.ld == o.ld || o.rows == 1);
      if (same && q.in_place) continue;
      if (overlaps(o, q)) return set_error(ARX_EINVAL, "%s overlaps %s", o.name, q.name);
    }
  }
  return ARX_OK;
}

Operand in(const char* name, const void* p, size_t rows, size_t cols, size_t ld, size_t size, bool in_place = false) {
  return {name, p, rows, cols, ld, size, false, in_place};
}
Operand out(const char* name, const void* p, size_t rows, size_t cols, size_t ld, size_t size) {
  return {name, p, rows, cols, ld, size, true, false};
}

int need(const char* name, const void* p, bool wanted = true) {
  return wanted && !p ? set_error(ARX_EINVAL, "null %s", name) : ARX_OK;
}

int check_sizes(size_t a, size_t b, size_t c = 0) {
  if (a > kMaxSize || b > kMaxSize || c > kMaxSize)
    return set_error(ARX_EINVAL, "a size above %zu", kMaxSize);
  return ARX_OK;
}

int check_types(int dtype, int wdtype) {
  if (dtype != ARX_BF16 && dtype != ARX_F16 && dtype != ARX_F32)
    return set_error(ARX_EINVAL, "dtype %d unknown", dtype);
  if (wdtype != dtype && wdtype != ARX_F32)
    return set_error(ARX_EINVAL, "wdtype %d is neither the rows' type nor ARX_F32", wdtype);
  return ARX_OK;
}

int check_eps(double eps) {
  return eps >= 0.0 && std::isfinite(eps) ? ARX_OK : set_error(ARX_EINVAL, "eps %g is not a finite value >= 0", eps);
}

int check_workspace(const void* p, size_t bytes, size_t wanted) {
  if (wanted == 0) return ARX_OK;
  if (!p || bytes < wanted)
    return set_error(ARX_EINVAL, "workspace of %zu bytes, %zu needed", p ? bytes : (size_t)0, wanted);
  if ((uintptr_t)p & 15u) return set_error(ARX_EINVAL, "workspace is not 16-byte aligned");
  return ARX_OK;
}

int make_drop(double p, uint64_t seed, uint64_t offset, arx::Drop* d) {
  if (!(p >= 0.0 && p <= 1.0)) return set_error(ARX_EINVAL, "p %g not in [0, 1]", p);
  d->threshold = (uint32_t)llrint(65536.0 * p);
  d->scale = d->threshold < 65536u ? 65536.0f / (float)(65536u - d->threshold) : 0.0f;
  d->seed = seed;
  d->offset = offset;
  return ARX_OK;
}

int launched(hipError_t e, const char* what) {
  return e == hipSuccess ? ARX_OK : set_error(ARX_EHIP, "%s: %s", what, hipGetErrorString(e));
}

#define TRY(call)                \
  do {                           \
    const int rc_ = (call);      \
    if (rc_ != ARX_OK) return rc_; \
  } while (0)

Plane plane(const void* p, size_t ld) { return {p, (int64_t)ld}; }
PlaneOut plane_out(void* p, size_t ld) { return {p, (int64_t)ld}; }

// The backward pass's workspace: g, the operands that have to be copied, then
// what the bias's column sums and the two products need one after another.
struct LinearSpace {
  size_t g = 0, pads = 0, rest = 0;
  size_t total() const { return g + pads + rest; }
};
LinearSpace linear_space(size_t m, size_t n, size_t k, int act, bool aligned) {
  const uint32_t m_ = (uint32_t)m, n_ = (uint32_t)n, k_ = (uint32_t)k;
  LinearSpace s;
  if (act != ARX_ACT_NONE) s.g = round_up(m * ((n + 7) & ~(size_t)7) * 2);
  else if (!aligned || n % 8) s.pads += arx::padded_bytes(m_, n_);
  if (!aligned || k % 8) s.pads += arx::padded_bytes(m_, k_) + arx::padded_bytes(n_, k_);
  const size_t parts[3] = {arx::act_grad_workspace(m, n), arx::gemm_splits_workspace(m_, k_, n_, false, true),
                           arx::gemm_splits_workspace(n_, k_, m_, true, true)};
  for (size_t b : parts) s.rest = b > s.rest ? b : s.rest;
  return s;
}

// Whether a plane's rows all start on 16-byte boundaries, near enough for a
// tile's 32-bit offsets.
bool on_lines(const void* p, size_t ld) { return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0 && ld < ((size_t)1 << 22); }

int check_linear(size_t m, size_t n, size_t k, int act, int dtype) {
  if (m > kMaxTokens) return set_error(ARX_EINVAL, "size m %zu above %zu", m, kMaxTokens);
  if (n > kMaxWidth || k > kMaxWidth)
    return set_error(ARX_EINVAL, "a size above %zu: n %zu, k %zu", kMaxWidth, n, k);
  if (dtype != ARX_BF16 && dtype != ARX_F16) return set_error(ARX_EINVAL, "dtype %d: ARX_BF16 or ARX_F16", dtype);
  if (act < ARX_ACT_NONE || act > ARX_ACT_SILU) return set_error(ARX_EINVAL, "act %d unknown", act);
  return ARX_OK;
}

}  // namespace

extern "C" {

size_t arx_linear_workspace(size_t m, size_t n, size_t k, int aligned) {
  if (m > kMaxTokens || n > kMaxWidth || k > kMaxWidth) return 0;
  return arx::gemm_workspace((uint32_t)m, (uint32_t)n, (uint32_t)k, aligned != 0);
}

int arx_linear(const void* x, const void* w, const void* bias, const void* residual, void* y, void* z, size_t m,
               size_t n, size_t k, size_t ldx, size_t ldw, size_t ldr, size_t ldy, size_t ldz, int act, int dtype,
               void* workspace, size_t workspace_bytes, hipStream_t stream) {
  TRY(check_linear(m, n, k, act, dtype));
  if (m == 0 || n == 0) return ARX_OK;
  TRY(need("x", x, k > 0));
  TRY(need("w", w, k > 0));
  TRY(need("y", y));
  TRY(check({in("x", x, m, k, ldx, 2), in("w", w, n, k, ldw, 2), in("bias", bias, 1, n, n, 2),
             in("residual", residual, m, n, ldr, 2, true), out("y", y, m, n, ldy, 2), out("z", z, m, n, ldz, 2)}));
  TRY(check_workspace(workspace, workspace_bytes,
                      arx_linear_workspace(m, n, k, on_lines(x, ldx) && on_lines(w, ldw))));
  arx::GemmArgs g{};
  g.a = x;
  g.b = w;
  g.lda = (int64_t)ldx;
  g.ldb = (int64_t)ldw;
  g.m = (uint32_t)m;
  g.n = (uint32_t)n;
  g.k = (uint32_t)k;
  g.bias = bias;
  g.residual = plane(residual, ldr);
  g.y = plane_out(y, ldy);
  g.z = plane_out(z, ldz);
  g.act = act;
  g.workspace = workspace;
  return launched(arx::launch_gemm(g, dtype, stream), "arx_linear");
}

size_t arx_linear_backward_workspace(size_t m, size_t n, size_t k, int act, int aligned) {
  if (m > kMaxTokens || n > kMaxWidth || k > kMaxWidth) return 0;
  return linear_space(m, n, k, act, aligned != 0).total();
}

int arx_linear_backward(const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw, void* dbias,
                        size_t m, size_t n, size_t k, size_t lddy, size_t ldx, size_t ldw, size_t ldz, size_t lddx,
                        size_t lddw, int act, int dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  TRY(check_linear(m, n, k, act, dtype));
  if (m == 0 || k == 0) dx = nullptr;
  if (n == 0 || k == 0) dw = nullptr;
  if (n == 0) dbias = nullptr;
  if (!dx && !dw && !dbias) return ARX_OK;
  const bool some = m > 0 && n > 0;
  TRY(need("dy", dy, some));
  TRY(need("x", x, dw && some));
  TRY(need("w", w, dx && some));
  TRY(need("z", z, act != ARX_ACT_NONE && some));
  if (act == ARX_ACT_NONE) z = nullptr;
  TRY(check({in("dy", dy, m, n, lddy, 2), in("x", dw ? x : nullptr, m, k, ldx, 2),
             in("w", dx ? w : nullptr, n, k, ldw, 2), in("z", z, m, n, ldz, 2), out("dx", dx, m, k, lddx, 2),
             out("dw", dw, n, k, lddw, 2), out("dbias", dbias, 1, n, n, 2)}));
  const LinearSpace s = linear_space(m, n, k, act, on_lines(dy, lddy) && on_lines(x, ldx) && on_lines(w, ldw));
  TRY(check_workspace(workspace, workspace_bytes, s.total()));
  char* const pads = static_cast<char*>(workspace) + s.g;
  char* const rest = pads + s.pads;

  const bool slope = act != ARX_ACT_NONE && (dx || dw);
  if (slope || dbias) {
    arx::ActGradArgs a{};
    a.dy = plane(dy, lddy);
    a.z = plane(z, ldz);
    a.g = slope ? workspace : nullptr;
    a.dbias = dbias;
    a.m = (uint32_t)m;
    a.n = (uint32_t)n;
    a.partial = reinterpret_cast<float*>(rest);
    TRY(launched(arx::launch_act_grad(a, act, dtype, stream), "arx_linear_backward"));
  }
  if (!dx && !dw) return ARX_OK;

  arx::Lines l[3] = {{slope ? workspace : dy, (int64_t)(slope ? (n + 7) & ~(size_t)7 : lddy), (uint32_t)m, (uint32_t)n, slope},
                     {dx && some ? w : nullptr, (int64_t)ldw, (uint32_t)n, (uint32_t)k, false},
                     {dw && some ? x : nullptr, (int64_t)ldx, (uint32_t)m, (uint32_t)k, false}};
  if (some) TRY(launched(arx::launch_pad(l, 3, dtype, pads, stream), "arx_linear_backward"));
  arx::GemmArgs gx{};
  gx.a = l[0].p;
  gx.lda = l[0].ld;
  gx.a_whole = gx.b_whole = true;
  gx.act = ARX_ACT_NONE;
  gx.workspace = rest;
  arx::GemmArgs gw = gx;
  gx.b = l[1].p;
  gx.ldb = l[1].ld;
  gx.b_rows_k = true;
  gx.m = (uint32_t)m;
  gx.n = (uint32_t)k;
  gx.k = (uint32_t)n;
  gx.y = plane_out(dx, lddx);
  gw.b = l[2].p;
  gw.ldb = l[2].ld;
  gw.a_rows_k = gw.b_rows_k = true;
  gw.m = (uint32_t)n;
  gw.n = (uint32_t)k;
  gw.k = (uint32_t)m;
  gw.y = plane_out(dw, lddw);
  if (dx && dw) return launched(arx::launch_gemm_pair(gx, gw, dtype, stream), "arx_linear_backward");
  return launched(arx::launch_gemm(dx ? gx : gw, dtype, stream), "arx_linear_backward");
}

int arx_layer_norm(const void* x, const void* weight, const void* shift, void* y, float* mean, float* rstd,
                   size_t rows, size_t cols, size_t ldx, size_t ldy, double eps, int dtype, int wdtype,
                   hipStream_t stream) {
  TRY(check_sizes(rows, cols));
  TRY(check_types(dtype, wdtype));
  TRY(check_eps(eps));
  if (rows == 0 || (cols == 0 && !mean && !rstd)) return ARX_OK;
  TRY(need("x", x, cols > 0));
  TRY(need("y", y, cols > 0));
  const size_t e = size_of(dtype), we = size_of(wdtype);
  TRY(check({in("x", x, rows, cols, ldx, e, true), in("weight", weight, 1, cols, cols, we),
             in("shift", shift, 1, cols, cols, we), out("y", y, rows, cols, ldy, e), out("mean", mean, 1, rows, rows, 4),
             out("rstd", rstd, 1, rows, rows, 4)}));
  arx::RowsArgs a{};
  a.x = plane(x, ldx);
  a.weight = weight;
  a.shift = shift;
  a.y = plane_out(y, ldy);
  a.mean = mean;
  a.rstd = rstd;
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.eps = (float)eps;
  return launched(arx::launch_norm(a, false, dtype, wdtype, stream), "arx_layer_norm");
}

size_t arx_rows_workspace(size_t rows, size_t cols, int sums) {
  if (rows > kMaxSize || cols > kMaxSize || sums < 1 || sums > 3) return 0;
  return arx::rows_workspace(rows, cols, sums);
}

int arx_layer_norm_backward(const void* dy, const void* x, const float* mean, const float* rstd, const void* weight,
                            void* dx, void* dweight, void* dshift, size_t rows, size_t cols, size_t lddy, size_t ldx,
                            size_t lddx, int dtype, int wdtype, void* workspace, size_t workspace_bytes,
                            hipStream_t stream) {
  TRY(check_sizes(rows, cols));
  TRY(check_types(dtype, wdtype));
  if (cols == 0) return ARX_OK;
  TRY(need("dy", dy, rows > 0));
  TRY(need("x", x, rows > 0));
  TRY(need("mean", mean, rows > 0));
  TRY(need("rstd", rstd, rows > 0));
  TRY(need("dx", dx, rows > 0));
  const size_t e = size_of(dtype), we = size_of(wdtype);
  TRY(check({in("dy", dy, rows, cols, lddy, e, true), in("x", x, rows, cols, ldx, e, true),
             in("mean", mean, 1, rows, rows, 4), in("rstd", rstd, 1, rows, rows, 4),
             in("weight", weight, 1, cols, cols, we), out("dx", dx, rows, cols, lddx, e),
             out("dweight", dweight, 1, cols, cols, we), out("dshift", dshift, 1, cols, cols, we)}));
  TRY(check_workspace(workspace, workspace_bytes, arx_rows_workspace(rows, cols, 2)));
  arx::RowsGradArgs a{};
  a.dy = plane(dy, lddy);
  a.x = plane(x, ldx);
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.dx = plane_out(dx, lddx);
  a.dweight = dweight;
  a.dshift = dshift;
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.partial = static_cast<float*>(workspace);
  return launched(arx::launch_norm_backward(a, false, dtype, wdtype, stream), "arx_layer_norm_backward");
}

int arx_dropout_add(const void* x, const void* bias, const void* residual, void* h, size_t rows, size_t cols,
                    size_t ldx, size_t ldr, size_t ldh, double p, uint64_t seed, uint64_t offset, int dtype,
                    hipStream_t stream) {
  TRY(check_sizes(rows, cols));
  TRY(check_types(dtype, dtype));
  arx::RowsArgs a{};
  TRY(make_drop(p, seed, offset, &a.drop));
  if (rows == 0 || cols == 0) return ARX_OK;
  TRY(need("x", x));
  TRY(need("h", h));
  const size_t e = size_of(dtype);
  TRY(check({in("x", x, rows, cols, ldx, e, true), in("bias", bias, 1, cols, cols, e),
             in("residual", residual, rows, cols, ldr, e, true), out("h", h, rows, cols, ldh, e)}));
  a.x = plane(x, ldx);
  a.bias = bias;
  a.residual = plane(residual, ldr);
  a.h = plane_out(h, ldh);
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  return launched(arx::launch_dropout_add(a, dtype, stream), "arx_dropout_add");
}

int arx_dropout_add_backward(const void* dh, void* dx, void* dbias, size_t rows, size_t cols, size_t lddh, size_t lddx,
                             double p, uint64_t seed, uint64_t offset, int dtype, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  TRY(check_sizes(rows, cols));
  TRY(check_types(dtype, dtype));
  arx::RowsGradArgs a{};
  TRY(make_drop(p, seed, offset, &a.drop));
  if (cols == 0 || (rows == 0 && !dbias) || (!dx && !dbias)) return ARX_OK;
  TRY(need("dh", dh, rows > 0));
  const size_t e = size_of(dtype);
  TRY(check({in("dh", dh, rows, cols, lddh, e, true), out("dx", dx, rows, cols, lddx, e),
             out("dbias", dbias, 1, cols, cols, e)}));
  TRY(check_workspace(workspace, workspace_bytes, dbias ? arx_rows_workspace(rows, cols, 1) : 0));
  a.dh = plane(dh, lddh);
  a.dx = plane_out(dx, lddx);
  a.dbias = dbias;
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.partial = static_cast<float*>(workspace);
  return launched(arx::launch_dropout_add_backward(a, dtype, stream), "arx_dropout_add_backward");
}

int arx_dropout_add_norm(const void* x, const void* bias, const void* residual, const void* weight,
                         const void* shift, void* h, void* y, float* mean, float* rstd, size_t rows, size_t cols,
                         size_t ldx, size_t ldr, size_t ldh, size_t ldy, double eps, double p, uint64_t seed,
                         uint64_t offset, int dtype, int wdtype, hipStream_t stream) {
  TRY(check_sizes(rows, cols));
  TRY(check_types(dtype, wdtype));
  TRY(check_eps(eps));
  arx::RowsArgs a{};
  TRY(make_drop(p, seed, offset, &a.drop));
  if (rows == 0 || (cols == 0 && !mean && !rstd)) return ARX_OK;
  TRY(need("x", x, cols > 0));
  TRY(need("y", y, cols > 0));
  const size_t e = size_of(dtype), we = size_of(wdtype);
  TRY(check({in("x", x, rows, cols, ldx, e, true), in("bias", bias, 1, cols, cols, e),
             in("residual", residual, rows, cols, ldr, e, true), in("weight", weight, 1, cols, cols, we),
             in("shift", shift, 1, cols, cols, we), out("h", h, rows, cols, ldh, e), out("y", y, rows, cols, ldy, e),
             out("mean", mean, 1, rows, rows, 4), out("rstd", rstd, 1, rows, rows, 4)}));
  a.x = plane(x, ldx);
  a.residual = plane(residual, ldr);
  a.bias = bias;
  a.weight = weight;
  a.shift = shift;
  a.h = plane_out(h, ldh);
  a.y = plane_out(y, ldy);
  a.mean = mean;
  a.rstd = rstd;
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.eps = (float)eps;
  return launched(arx::launch_norm(a, true, dtype, wdtype, stream), "arx_dropout_add_norm");
}

int arx_dropout_add_norm_backward(const void* dy, const void* dh, const void* h, const float* mean, const float* rstd,
                                  const void* weight, void* dx, void* dresidual, void* dbias, void* dweight,
                                  void* dshift, size_t rows, size_t cols, size_t lddy, size_t lddh, size_t ldh,
                                  size_t lddx, size_t lddr, double p, uint64_t seed, uint64_t offset, int dtype,
                                  int wdtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  TRY(check_sizes(rows, cols));
  TRY(check_types(dtype, wdtype));
  arx::RowsGradArgs a{};
  TRY(make_drop(p, seed, offset, &a.drop));
  if (cols == 0) return ARX_OK;
  TRY(need("dy", dy, rows > 0));
  TRY(need("h", h, rows > 0));
  TRY(need("mean", mean, rows > 0));
  TRY(need("rstd", rstd, rows > 0));
  TRY(need("dx", dx, rows > 0));
  const size_t e = size_of(dtype), we = size_of(wdtype);
  TRY(check({in("dy", dy, rows, cols, lddy, e, true), in("dh", dh, rows, cols, lddh, e, true),
             in("h", h, rows, cols, ldh, e, true), in("mean", mean, 1, rows, rows, 4),
             in("rstd", rstd, 1, rows, rows, 4), in("weight", weight, 1, cols, cols, we),
             out("dx", dx, rows, cols, lddx, e), out("dresidual", dresidual, rows, cols, lddr, e),
             out("dbias", dbias, 1, cols, cols, e), out("dweight", dweight, 1, cols, cols, we),
             out("dshift", dshift, 1, cols, cols, we)}));
  TRY(check_workspace(workspace, workspace_bytes, arx_rows_workspace(rows, cols, 3)));
  a.dy = plane(dy, lddy);
  a.dh = plane(dh, lddh);
  a.x = plane(h, ldh);
  a.mean = mean;
  a.rstd = rstd;
  a.weight = weight;
  a.dx = plane_out(dx, lddx);
  a.dresidual = plane_out(dresidual, lddr);
  a.dbias = dbias;
  a.dweight = dweight;
  a.dshift = dshift;
  a.rows = (uint32_t)rows;
  a.cols = (uint32_t)cols;
  a.partial = static_cast<float*>(workspace);
  return launched(arx::launch_norm_backward(a, true, dtype, wdtype, stream), "arx_dropout_add_norm_backward");
}

}  // extern "C"
