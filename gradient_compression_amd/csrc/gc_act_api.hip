// gc_act_api.hip -- host side of the activation operators of include/gc.h: layouts, argument
// checks and launches.  Nothing is allocated and nothing is kept between calls.
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <numeric>
#include <utility>

#include "gc.h"

#include "gc_act_internal.h"

namespace {

constexpr int64_t kMostRows = (int64_t)1 << 25;      // threads of a launch stay below 2^32
constexpr int64_t kMostCodes = (int64_t)1 << 34;
constexpr int64_t kMostCols = (int64_t)1 << 27;
constexpr int64_t kMostWeights = ((int64_t)1 << 31) - 1;

int64_t groups_of(int64_t cols) { return cols / 32 + (cols % 32 != 0); }
bool valid_dtype(int32_t d) { return d == GC_F32 || d == GC_BF16 || d == GC_F16; }
int64_t size_of(int32_t d) { return d == GC_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// What a call touches through one pointer: `rows` pieces of `width` bytes, `pitch` bytes apart.
struct Area {
  const void* p;
  int64_t rows, width, pitch;
  bool out;
};
Area matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int32_t dtype, bool out) {
  if (!p || !rows || !cols) return {nullptr, 0, 0, 0, out};   // whatever ld is
  return {p, rows, cols * size_of(dtype), ld * size_of(dtype), out};
}
Area flat(const void* p, int64_t bytes, bool out) { return {p, bytes > 0, bytes, bytes, out}; }

bool share_bytes(const Area& a, const Area& b) {
  if (!a.p || !b.p || !a.rows || !b.rows || !a.width || !b.width) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t a1 = a0 + (a.rows - 1) * a.pitch + a.width;
  const uintptr_t b1 = b0 + (b.rows - 1) * b.pitch + b.width;
  if (a0 >= b1 || b0 >= a1) return false;
  // Their spans meet.  Pieces at one pitch (column blocks of a wider matrix), at multiples of one
  // pitch (of every row of it and of every other one), or one piece against rows, still share nothing
  // where they lie in the rows' gaps.  (Pitches whose common divisor leaves no room for both, such as
  // 100 and 101 elements, are taken to meet: nothing that lies in one matrix has them.)
  if (a.rows == 1 && b.rows > 1) return share_bytes(b, a);
  if (a.rows == 1) return true;
  const int64_t pitch = b.rows == 1 ? a.pitch : std::gcd(a.pitch, b.pitch);
  int64_t d = ((int64_t)b0 - (int64_t)a0) % pitch;   // b's place in a's row, 0 <= d < pitch
  if (d < 0) d += pitch;
  return d < a.width || d + b.width > pitch;
}

bool same(const Area& a, const Area& b) {
  return a.p == b.p && a.width == b.width && (a.pitch == b.pitch || a.rows <= 1);
}

// True when an output shares a byte with another buffer, but for the pairs of the same matrix
// that `may` names (indices into `areas`).
bool clash(std::initializer_list<Area> areas, std::initializer_list<std::pair<int, int>> may) {
  const Area* v = areas.begin();
  const int n = (int)areas.size();
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j) {
      if (!v[i].out && !v[j].out) continue;
      if (!share_bytes(v[i], v[j])) continue;
      bool allowed = false;
      for (const auto& m : may)
        allowed = allowed || (((m.first == i && m.second == j) || (m.first == j && m.second == i)) &&
                              same(v[i], v[j]));
      if (!allowed) return true;
    }
  return false;
}

int check_sizes(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0) return GC_ERR_INVALID_ARG;
  if (rows > kMostRows || cols > kMostCols) return GC_ERR_UNSUPPORTED;
  if (rows * groups_of(cols) * 32 > kMostCodes) return GC_ERR_UNSUPPORTED;   // < 2^57: no wrap
  return GC_OK;
}

// A matrix argument: present, aligned to its element, rows that do not overlap; a span that
// 63-bit byte offsets hold.
bool valid_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, int32_t dtype) {
  if (rows == 0 || cols == 0) return true;
  return p && aligned(p, size_of(dtype)) && ld >= cols && ld <= ((int64_t)1 << 34);
}

bool valid_checkpoint(const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols) {
  return rows == 0 || cols == 0 || (codes && exps && aligned(codes, 16));
}

gc::ActRound rounding_of(int32_t rounding, uint64_t seed, uint64_t step) {
  return {rounding == GC_ROUND_STOCHASTIC, (uint32_t)seed, (uint32_t)(seed >> 32), (uint32_t)step};
}

int status(hipError_t e) { return e == hipSuccess ? GC_OK : GC_ERR_HIP; }

gc::Mat mat(const void* p, int64_t ld) { return {const_cast<void*>(p), ld}; }

}  // namespace

extern "C" {

int gc_act_layout(int64_t cols, int64_t* pitch, int64_t* groups) {
  if (cols < 0) return GC_ERR_INVALID_ARG;
  if (cols > kMostCols) return GC_ERR_UNSUPPORTED;
  if (pitch) *pitch = groups_of(cols) * 32;
  if (groups) *groups = groups_of(cols);
  return GC_OK;
}

int gc_act_quant(const void* x, int64_t ld_x, int32_t dtype, int64_t rows, int64_t cols,
                 int32_t rounding, uint64_t seed, uint64_t step, int8_t* codes, uint8_t* exps,
                 void* stream) {
  if (!valid_dtype(dtype) || (rounding != GC_ROUND_NEAREST && rounding != GC_ROUND_STOCHASTIC))
    return GC_ERR_INVALID_ARG;
  if (int rc = check_sizes(rows, cols)) return rc;
  if (!valid_matrix(x, ld_x, rows, cols, dtype) || !valid_checkpoint(codes, exps, rows, cols))
    return GC_ERR_INVALID_ARG;
  const int64_t g = groups_of(cols);
  if (clash({matrix(x, ld_x, rows, cols, dtype, false), flat(codes, rows * g * 32, true),
             flat(exps, rows * g, true)}, {}))
    return GC_ERR_INVALID_ARG;
  return status(gc::launch_act_quant(mat(x, ld_x), dtype, rows, (int32_t)cols,
                                     rounding_of(rounding, seed, step), codes, exps,
                                     static_cast<hipStream_t>(stream)));
}

int gc_act_restore(const int8_t* codes, const uint8_t* exps, int64_t rows, int64_t cols,
                   void* out, int64_t ld_out, int32_t dtype, void* stream) {
  if (!valid_dtype(dtype)) return GC_ERR_INVALID_ARG;
  if (int rc = check_sizes(rows, cols)) return rc;
  if (!valid_matrix(out, ld_out, rows, cols, dtype) || !valid_checkpoint(codes, exps, rows, cols))
    return GC_ERR_INVALID_ARG;
  const int64_t g = groups_of(cols);
  if (clash({matrix(out, ld_out, rows, cols, dtype, true), flat(codes, rows * g * 32, false),
             flat(exps, rows * g, false)}, {}))
    return GC_ERR_INVALID_ARG;
  return status(gc::launch_act_restore(codes, exps, rows, (int32_t)cols, mat(out, ld_out), dtype,
                                       static_cast<hipStream_t>(stream)));
}

int gc_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
               int32_t dtype, int64_t rows, int64_t cols, const void* weight,
               int32_t weight_dtype, float eps, void* h, int64_t ld_h, void* y, int64_t ld_y,
               float* rstd, int8_t* codes, uint8_t* exps, int32_t rounding, uint64_t seed,
               uint64_t step, void* stream) {
  if (!valid_dtype(dtype) || (weight && !valid_dtype(weight_dtype)) || !(eps >= 0.0f) ||
      std::isinf(eps) || (rounding != GC_ROUND_NEAREST && rounding != GC_ROUND_STOCHASTIC))
    return GC_ERR_INVALID_ARG;
  if (int rc = check_sizes(rows, cols)) return rc;
  if (cols > gc::kNormMostCols) return GC_ERR_UNSUPPORTED;
  if ((codes == nullptr) != (exps == nullptr)) return GC_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GC_OK;
  if (!y && !codes) return GC_ERR_INVALID_ARG;
  if (!valid_matrix(x, ld_x, rows, cols, dtype) ||
      (residual && !valid_matrix(residual, ld_residual, rows, cols, dtype)) ||
      (h && !valid_matrix(h, ld_h, rows, cols, dtype)) ||
      (y && !valid_matrix(y, ld_y, rows, cols, dtype)) ||
      (codes && !valid_checkpoint(codes, exps, rows, cols)) ||
      (weight && !aligned(weight, size_of(weight_dtype))) || !aligned(rstd, 4))
    return GC_ERR_INVALID_ARG;
  const int64_t g = groups_of(cols);
  if (clash({matrix(x, ld_x, rows, cols, dtype, false),
             matrix(residual, ld_residual, rows, cols, dtype, false),
             matrix(h, ld_h, rows, cols, dtype, true), matrix(y, ld_y, rows, cols, dtype, true),
             flat(weight, weight ? cols * size_of(weight_dtype) : 0, false),
             flat(rstd, rows * 4, true), flat(codes, rows * g * 32, true),
             flat(exps, rows * g, true)},
            {{0, 2}, {1, 2}, {0, 3}, {1, 3}}))
    return GC_ERR_INVALID_ARG;
  gc::NormArgs a{};
  a.dtype = dtype;
  a.weight_dtype = weight_dtype;
  a.rows = rows;
  a.cols = (int32_t)cols;
  a.x = mat(x, ld_x);
  a.res = mat(residual, ld_residual);
  a.h = mat(h, ld_h);
  a.y = mat(y, ld_y);
  a.weight = weight;
  a.eps = eps;
  a.rstd = rstd;
  a.codes = codes;
  a.exps = exps;
  a.round = rounding_of(rounding, seed, step);
  return status(gc::launch_rmsnorm(a, static_cast<hipStream_t>(stream)));
}

int gc_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
  if (!bytes) return GC_ERR_INVALID_ARG;
  if (int rc = check_sizes(rows, cols)) return rc;
  if (cols > gc::kNormMostCols) return GC_ERR_UNSUPPORTED;
  *bytes = gc::norm_grad_blocks(rows, (int32_t)cols) * groups_of(cols) * 32 * 4;
  return GC_OK;
}

int gc_rmsnorm_backward(const void* dy, int64_t ld_dy, int32_t dtype, int64_t rows, int64_t cols,
                        const int8_t* codes, const uint8_t* exps, const float* rstd,
                        const void* weight, int32_t weight_dtype, const void* dres,
                        int64_t ld_dres, void* dx, int64_t ld_dx, float* dweight, int accumulate,
                        void* workspace, int64_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype) || (weight && !valid_dtype(weight_dtype))) return GC_ERR_INVALID_ARG;
  int64_t need = 0;
  if (int rc = gc_rmsnorm_backward_workspace(rows, cols, &need)) return rc;
  if (!dweight) need = 0;
  if (workspace_bytes < need || (need && !workspace) || !aligned(workspace, 16))
    return GC_ERR_INVALID_ARG;
  if (!valid_matrix(dy, ld_dy, rows, cols, dtype) || !valid_matrix(dx, ld_dx, rows, cols, dtype) ||
      (dres && !valid_matrix(dres, ld_dres, rows, cols, dtype)) ||
      !valid_checkpoint(codes, exps, rows, cols) ||
      (rows && cols && (!rstd || !aligned(rstd, 4))) ||
      (weight && !aligned(weight, size_of(weight_dtype))) || !aligned(dweight, 4))
    return GC_ERR_INVALID_ARG;
  const int64_t g = groups_of(cols);
  if (clash({matrix(dy, ld_dy, rows, cols, dtype, false),
             matrix(dres, ld_dres, rows, cols, dtype, false),
             matrix(dx, ld_dx, rows, cols, dtype, true), flat(codes, rows * g * 32, false),
             flat(exps, rows * g, false), flat(rstd, rows * 4, false),
             flat(weight, weight ? cols * size_of(weight_dtype) : 0, false),
             flat(dweight, cols * 4, true), flat(workspace, need, true)},
            {{0, 2}, {1, 2}}))
    return GC_ERR_INVALID_ARG;
  gc::NormGradArgs a{};
  a.dtype = dtype;
  a.weight_dtype = weight_dtype;
  a.rows = rows;
  a.cols = (int32_t)cols;
  a.dy = mat(dy, ld_dy);
  a.dres = mat(dres, ld_dres);
  a.dx = mat(dx, ld_dx);
  a.codes = codes;
  a.exps = exps;
  a.rstd = rstd;
  a.weight = weight;
  a.dweight = dweight;
  a.accumulate = accumulate != 0;
  a.ws = static_cast<float*>(workspace);
  return status(gc::launch_rmsnorm_backward(a, static_cast<hipStream_t>(stream)));
}

int gc_act_weight_grad_workspace(int64_t rows, int64_t n_out, int64_t cols, int32_t dtype,
                                 int64_t* bytes) {
  if (!bytes || !valid_dtype(dtype) || n_out < 0) return GC_ERR_INVALID_ARG;
  if (int rc = check_sizes(rows, cols)) return rc;
  if (n_out > kMostCols || n_out * cols > kMostWeights) return GC_ERR_UNSUPPORTED;
  const int splits = gc::wgrad_splits(rows, (int32_t)n_out, (int32_t)cols, dtype);
  *bytes = splits > 1 ? (int64_t)splits * n_out * cols * 4 : 0;
  return GC_OK;
}

int gc_act_weight_grad(const void* dy, int64_t ld_dy, int32_t dtype, int64_t rows, int64_t n_out,
                       int64_t cols, const int8_t* codes, const uint8_t* exps,
                       const void* col_scale, int32_t scale_dtype, float* dweight, int accumulate,
                       void* workspace, int64_t workspace_bytes, void* stream) {
  if (col_scale && !valid_dtype(scale_dtype)) return GC_ERR_INVALID_ARG;
  int64_t need = 0;
  if (int rc = gc_act_weight_grad_workspace(rows, n_out, cols, dtype, &need)) return rc;
  if (n_out == 0 || cols == 0) return GC_OK;
  if (workspace_bytes < need || (need && !workspace) || !aligned(workspace, 16))
    return GC_ERR_INVALID_ARG;
  if (!valid_matrix(dy, ld_dy, rows, n_out, dtype) || !valid_checkpoint(codes, exps, rows, cols) ||
      !dweight || !aligned(dweight, 4) ||
      (col_scale && !aligned(col_scale, size_of(scale_dtype))))
    return GC_ERR_INVALID_ARG;
  const int64_t g = groups_of(cols);
  if (clash({matrix(dy, ld_dy, rows, n_out, dtype, false), flat(codes, rows * g * 32, false),
             flat(exps, rows * g, false),
             flat(col_scale, col_scale ? cols * size_of(scale_dtype) : 0, false),
             flat(dweight, n_out * cols * 4, true), flat(workspace, need, true)}, {}))
    return GC_ERR_INVALID_ARG;
  gc::WgradArgs a{};
  a.dtype = dtype;
  a.scale_dtype = scale_dtype;
  a.rows = rows;
  a.n_out = (int32_t)n_out;
  a.cols = (int32_t)cols;
  a.dy = mat(dy, ld_dy);
  a.codes = codes;
  a.exps = exps;
  a.col_scale = rows ? col_scale : nullptr;   // a sum of no rows is 0, whatever its scale
  a.dw = dweight;
  a.accumulate = accumulate != 0;
  a.ws = static_cast<float*>(workspace);
  return status(gc::launch_wgrad(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
