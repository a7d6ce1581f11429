// C ABI of the microscaled operators (declared in include/nvfp4.h): argument
// validation on the host before any HIP call, then the gfx950 kernels.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "../../include/nvfp4.h"
#include "launchers.h"

namespace {

using nvfp4::clear_error;
using nvfp4::device_ok;

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return nvfp4::set_error(status, buf);
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
hipStream_t hs(void* s) { return reinterpret_cast<hipStream_t>(s); }

// Launches stay below 2^32 work-items: the quantizer runs a thread per 32
// elements in workgroups of 8192.
constexpr int64_t kMaxElems = ((int64_t)1 << 37) - (1 << 20);
constexpr int64_t kMaxTokens = (int64_t)1 << 22;  // rows of a product's activations: 64 rows per grid row
constexpr int64_t kMaxRows = (int64_t)1 << 27;    // weight rows: 512 threads per 16 of them
constexpr int64_t kMaxK = (int64_t)1 << 30;
constexpr int64_t kMaxNormK = 65536;  // 8 pieces of 8 elements for each of 1024 threads, one workgroup per row

int check_mk(int64_t m, int64_t k, const char* rows) {
  if (m < 0 || k < 0)
    return fail(NVFP4_ERR_INVALID_VALUE, "negative dimension (%s=%lld, k=%lld)", rows, (long long)m, (long long)k);
  if (k % 32 != 0)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "k=%lld is not a multiple of 32", (long long)k);
  if (k > kMaxK || m > kMaxElems || (k > 0 && m > kMaxElems / k))
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "matrix too large (%s=%lld, k=%lld)", rows, (long long)m, (long long)k);
  return NVFP4_OK;
}

int check_format(int format) {
  if (format != NVFP4_MXFP4 && format != NVFP4_MXFP8)
    return fail(NVFP4_ERR_INVALID_VALUE, "format %d is not a NVFP4_MXFP* value", format);
  return NVFP4_OK;
}

int check_type(int t, const char* name) {
  if (t != NVFP4_BF16 && t != NVFP4_F32) return fail(NVFP4_ERR_INVALID_VALUE, "%s %d", name, t);
  return NVFP4_OK;
}

int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return NVFP4_OK;
  if (bytes < need)
    return fail(NVFP4_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu required", bytes, need);
  if (!workspace) return fail(NVFP4_ERR_INVALID_VALUE, "workspace is NULL");
  if (!aligned(workspace, 16)) return fail(NVFP4_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  return NVFP4_OK;
}

int check_product(int64_t m, int64_t n, int64_t k, int out_dtype) {
  int st = check_mk(m, k, "m");
  if (st) return st;
  if ((st = check_mk(n, k, "n"))) return st;
  if (m > kMaxTokens || n >= kMaxRows || (m > 0 && n > kMaxElems / m))
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "product too large (m=%lld, n=%lld)", (long long)m, (long long)n);
  return check_type(out_dtype, "out_dtype");
}

bool product_sizes_ok(int64_t m, int64_t n, int64_t k) {
  return m > 0 && n > 0 && k > 0 && k % 32 == 0 && k <= kMaxK && m <= kMaxTokens && n < kMaxRows &&
         m <= kMaxElems / k && n <= kMaxElems / k && n <= kMaxElems / m;
}

int check_norm(int64_t m, int64_t k, int weight_dtype) {
  int st = check_mk(m, k, "m");
  if (st) return st;
  if (k == 0 || k > kMaxNormK)
    return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "k=%lld: 32 .. %lld", (long long)k, (long long)kMaxNormK);
  // a row of more than 16384 elements has a workgroup of 1024 threads
  if (m >= kMaxTokens) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "m=%lld too large", (long long)m);
  return check_type(weight_dtype, "weight_dtype");
}

// A buffer of a call; NULL or no bytes: none.
struct Buffer {
  const void* p;
  int64_t bytes;
  const char* name;
};

bool overlap(const Buffer& a, const Buffer& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// An output that shares memory with an input or another output is written by one workgroup while another reads or
// writes it: refused, but where the output is that whole buffer and every thread reads what it then writes (`in_place`).
int check_outputs(std::initializer_list<Buffer> outputs, std::initializer_list<Buffer> inputs,
                  std::initializer_list<Buffer> in_place) {
  for (const Buffer* o = outputs.begin(); o != outputs.end(); ++o) {
    for (const Buffer& i : inputs)
      if (overlap(*o, i)) return fail(NVFP4_ERR_INVALID_VALUE, "%s overlaps %s", o->name, i.name);
    for (const Buffer* q = outputs.begin(); q != o; ++q)
      if (overlap(*o, *q)) return fail(NVFP4_ERR_INVALID_VALUE, "%s overlaps %s", o->name, q->name);
    for (const Buffer& i : in_place)
      if (overlap(*o, i) && !(o == outputs.begin() && o->p == i.p))
        return fail(NVFP4_ERR_INVALID_VALUE, "%s overlaps %s", o->name, i.name);
  }
  return NVFP4_OK;
}

int done(hipError_t e, const char* where) { return e == hipSuccess ? NVFP4_OK : nvfp4::set_hip_error(e, where); }

}  // namespace

extern "C" {

NVFP4_API int nvfp4_mx_quantize(const void* x, int x_dtype, int64_t m, int64_t k, int format, uint8_t* codes,
                                uint8_t* scales, void* stream) {
  clear_error();
  int st = check_mk(m, k, "m");
  if (st || (st = check_type(x_dtype, "x_dtype")) || (st = check_format(format))) return st;
  if (m == 0 || k == 0) return NVFP4_OK;
  if (!x || !codes || !scales) return fail(NVFP4_ERR_INVALID_VALUE, "x, codes and scales are required");
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16))
    return fail(NVFP4_ERR_MISALIGNED, "x, codes and scales must be 16-byte aligned");
  if ((st = device_ok())) return st;
  return done(nvfp4::launch_mx_quantize(x, x_dtype == NVFP4_F32, m, k, format, codes, scales, hs(stream)),
              "mx_quantize launch");
}

NVFP4_API int nvfp4_mx_dequant(const uint8_t* codes, const uint8_t* scales, void* out, int64_t m, int64_t k,
                               int format, int out_dtype, void* stream) {
  clear_error();
  int st = check_mk(m, k, "m");
  if (st || (st = check_type(out_dtype, "out_dtype")) || (st = check_format(format))) return st;
  if (m == 0 || k == 0) return NVFP4_OK;
  if (!codes || !scales || !out) return fail(NVFP4_ERR_INVALID_VALUE, "codes, scales and out are required");
  if (!aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16))
    return fail(NVFP4_ERR_MISALIGNED, "codes, scales and out must be 16-byte aligned");
  if ((st = device_ok())) return st;
  return done(nvfp4::launch_mx_dequant(codes, scales, out, m, k, format, out_dtype == NVFP4_F32, hs(stream)),
              "mx_dequant launch");
}

NVFP4_API size_t nvfp4_mx_gemm_workspace_size(int64_t m, int64_t n, int64_t k, int a_format) {
  if (!product_sizes_ok(m, n, k) || (a_format != NVFP4_MXFP4 && a_format != NVFP4_MXFP8)) return 0;
  return nvfp4::plan_mx_gemm(m, n, k, a_format).ws_bytes;
}

NVFP4_API int nvfp4_mx_gemm_path(int64_t m, int64_t n, int64_t k, int a_format) {
  if (!product_sizes_ok(m, n, k) || (a_format != NVFP4_MXFP4 && a_format != NVFP4_MXFP8)) return -1;
  return nvfp4::plan_mx_gemm(m, n, k, a_format).tile;
}

NVFP4_API int nvfp4_mx_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int a_format, const uint8_t* w_codes,
                            const uint8_t* w_scales, void* y, int64_t m, int64_t n, int64_t k, int out_dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  int st = check_product(m, n, k, out_dtype);
  if (st || (st = check_format(a_format))) return st;
  if (m == 0 || n == 0) return NVFP4_OK;
  if (!y) return fail(NVFP4_ERR_INVALID_VALUE, "y is required");
  if (k > 0 && (!a_codes || !a_scales || !w_codes || !w_scales))
    return fail(NVFP4_ERR_INVALID_VALUE, "a_codes, a_scales, w_codes and w_scales are required");
  if (!aligned(y, 16) ||
      (k > 0 && (!aligned(a_codes, 16) || !aligned(a_scales, 16) || !aligned(w_codes, 16) || !aligned(w_scales, 16))))
    return fail(NVFP4_ERR_MISALIGNED, "a_codes, a_scales, w_codes, w_scales and y must be 16-byte aligned");
  const nvfp4::MxPlan plan = nvfp4::plan_mx_gemm(m, n, k, a_format);
  if ((st = check_workspace(workspace, workspace_bytes, plan.ws_bytes)) || (st = device_ok())) return st;
  return done(nvfp4::launch_mx_gemm(a_codes, a_scales, a_format, w_codes, w_scales, y, m, n, k,
                                    out_dtype == NVFP4_F32, plan, workspace, hs(stream)),
              "mx_gemm launch");
}

NVFP4_API size_t nvfp4_mx_gemm_dx_workspace_size(int64_t m, int64_t n, int64_t k) {
  return product_sizes_ok(m, n, k) ? nvfp4::plan_mx_dx(m, n, k).ws_bytes : 0;
}

NVFP4_API int nvfp4_mx_gemm_dx_path(int64_t m, int64_t n, int64_t k) {
  return product_sizes_ok(m, n, k) ? nvfp4::plan_mx_dx(m, n, k).tile : -1;
}

NVFP4_API int nvfp4_mx_gemm_dx(const void* dy, const uint8_t* w_codes, const uint8_t* w_scales, void* dx, int64_t m,
                               int64_t n, int64_t k, int out_dtype, void* workspace, size_t workspace_bytes,
                               void* stream) {
  clear_error();
  int st = check_product(m, n, k, out_dtype);
  if (st) return st;
  if (m == 0 || k == 0) return NVFP4_OK;
  if (!dx) return fail(NVFP4_ERR_INVALID_VALUE, "dx is required");
  if (n > 0 && (!dy || !w_codes || !w_scales))
    return fail(NVFP4_ERR_INVALID_VALUE, "dy, w_codes and w_scales are required");
  if (!aligned(dx, 16) || (n > 0 && (!aligned(dy, 16) || !aligned(w_codes, 16) || !aligned(w_scales, 16))))
    return fail(NVFP4_ERR_MISALIGNED, "dy, w_codes, w_scales and dx must be 16-byte aligned");
  const nvfp4::MxPlan plan = nvfp4::plan_mx_dx(m, n, k);
  if ((st = check_workspace(workspace, workspace_bytes, plan.ws_bytes)) || (st = device_ok())) return st;
  return done(nvfp4::launch_mx_dx(static_cast<const uint16_t*>(dy), w_codes, w_scales, dx, m, n, k,
                                       out_dtype == NVFP4_F32, plan, workspace, hs(stream)),
              "mx_gemm_dx launch");
}

NVFP4_API int nvfp4_add_rmsnorm_mx(const void* x, const void* residual, const void* weight, int weight_dtype,
                                   float eps, int64_t m, int64_t k, int format, void* residual_out, float* rstd,
                                   uint8_t* codes, uint8_t* scales, void* stream) {
  clear_error();
  int st = check_norm(m, k, weight_dtype);
  if (st || (st = check_format(format))) return st;
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(NVFP4_ERR_INVALID_VALUE, "eps must be finite and >= 0");
  if ((residual == nullptr) != (residual_out == nullptr) && m > 0)
    return fail(NVFP4_ERR_INVALID_VALUE, "residual and residual_out go together");
  if (m == 0) return NVFP4_OK;
  if (!x || !weight || !codes || !scales)
    return fail(NVFP4_ERR_INVALID_VALUE, "x, weight, codes and scales are required");
  if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(residual_out, 16) ||
      !aligned(codes, 16) || !aligned(scales, 16))
    return fail(NVFP4_ERR_MISALIGNED, "x, residual, weight, residual_out, codes and scales must be 16-byte aligned");
  if (!aligned(rstd, 4)) return fail(NVFP4_ERR_MISALIGNED, "rstd must be 4-byte aligned");
  const int64_t row = 2 * m * k, wide = weight_dtype == NVFP4_F32 ? 4 * k : 2 * k;
  if ((st = check_outputs({{residual_out, row, "residual_out"},
                           {rstd, 4 * m, "rstd"},
                           {codes, format == NVFP4_MXFP4 ? m * k / 2 : m * k, "codes"},
                           {scales, m * k / 32, "scales"}},
                          {{weight, wide, "weight"}}, {{x, row, "x"}, {residual, row, "residual"}})))
    return st;
  if ((st = device_ok())) return st;
  return done(nvfp4::launch_add_rmsnorm_mx(x, residual, weight, weight_dtype == NVFP4_F32, (double)eps, m, k, format,
                                           residual_out, rstd, codes, scales, hs(stream)),
              "add_rmsnorm launch");
}

NVFP4_API size_t nvfp4_add_rmsnorm_backward_workspace_size(int64_t m, int64_t k) {
  if (m <= 0 || k <= 0 || k % 32 != 0 || k > kMaxNormK || m >= kMaxTokens) return 0;
  return (size_t)nvfp4::rmsnorm_backward_planes(m, k) * (size_t)k * sizeof(float);
}

NVFP4_API int nvfp4_add_rmsnorm_backward(const void* dh, const void* s, const void* weight, int weight_dtype,
                                         const float* rstd, const void* ds, void* dx, float* dweight, int64_t m,
                                         int64_t k, void* workspace, size_t workspace_bytes, void* stream) {
  clear_error();
  int st = check_norm(m, k, weight_dtype);
  if (st) return st;
  if (!dweight) return fail(NVFP4_ERR_INVALID_VALUE, "dweight is required");
  if (m > 0 && (!dh || !s || !weight || !rstd || !dx))
    return fail(NVFP4_ERR_INVALID_VALUE, "dh, s, weight, rstd and dx are required");
  if (!aligned(dweight, 16) || (m > 0 && (!aligned(dh, 16) || !aligned(s, 16) || !aligned(weight, 16) ||
                                          !aligned(ds, 16) || !aligned(dx, 16))))
    return fail(NVFP4_ERR_MISALIGNED, "dh, s, weight, ds, dx and dweight must be 16-byte aligned");
  if (m > 0 && !aligned(rstd, 4)) return fail(NVFP4_ERR_MISALIGNED, "rstd must be 4-byte aligned");
  const int64_t need = (int64_t)nvfp4_add_rmsnorm_backward_workspace_size(m, k);
  if ((st = check_workspace(workspace, workspace_bytes, (size_t)need))) return st;
  const int64_t row = 2 * m * k, wide = weight_dtype == NVFP4_F32 ? 4 * k : 2 * k;
  if (m > 0 && (st = check_outputs({{dx, row, "dx"}, {dweight, 4 * k, "dweight"}, {need > 0 ? workspace : nullptr, need, "workspace"}},
                                   {{dh, row, "dh"}, {s, row, "s"}, {weight, wide, "weight"}, {rstd, 4 * m, "rstd"}},
                                   {{ds, row, "ds"}})))
    return st;
  if ((st = device_ok())) return st;
  return done(nvfp4::launch_rmsnorm_backward(dh, s, weight, weight_dtype == NVFP4_F32, rstd, ds, dx, dweight, m, k,
                                             workspace, hs(stream)),
              "add_rmsnorm_backward launch");
}

}  // extern "C"
