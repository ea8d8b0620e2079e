// gc_grads_api.hip -- host side of the operators over many tensors of include/gc.h: argument checks,
// the tables of tensors and the launches.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <vector>

#include "gc.h"

#include "gc_grads.h"

namespace {

constexpr int64_t kMostElements = (int64_t)1 << 44;   // of a tensor, and of a call
constexpr int32_t kMostTensors = 1 << 20;
// Results of more than this are stored non-temporally, as no cache would keep them for their reader and the
// tensors stay in it instead: 391 tensors of 335 M elements into fp32 540 us in place of 562, 1.07e9 elements
// 1596 in place of 1636.
constexpr int64_t kCache = (int64_t)256 << 20;

bool valid_dtype(int32_t d) { return d == GC_F32 || d == GC_BF16 || d == GC_F16; }
int64_t size_of(int32_t d) { return d == GC_F32 ? 4 : 2; }
bool aligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
int64_t chunks_of(int64_t n) { return (n + gc::kGradChunk - 1) / gc::kGradChunk; }
int status(hipError_t e) { return e == hipSuccess ? GC_OK : GC_ERR_HIP; }

int check_sizes(const int64_t* sizes, int32_t n) {
  if (n < 0 || (n > 0 && !sizes)) return GC_ERR_INVALID_ARG;
  if (n > kMostTensors) return GC_ERR_UNSUPPORTED;
  int64_t total = 0;
  for (int32_t t = 0; t < n; ++t) {
    if (sizes[t] < 0) return GC_ERR_INVALID_ARG;
    if (sizes[t] > kMostElements) return GC_ERR_UNSUPPORTED;
    total += sizes[t];   // at most twice kMostElements
    if (total > kMostElements) return GC_ERR_UNSUPPORTED;
  }
  return GC_OK;
}

bool valid_tensors(const void* const* p, const int64_t* sizes, const int32_t* dtypes, int32_t n) {
  if (n > 0 && (!p || !dtypes)) return false;
  for (int32_t t = 0; t < n; ++t)
    if (!valid_dtype(dtypes[t]) || (sizes[t] && (!p[t] || !aligned(p[t], size_of(dtypes[t])))))
      return false;
  return true;
}

// A piece of memory that a call reads or writes.
struct Piece {
  uintptr_t begin, end;
  bool out;
};

Piece piece(const void* p, int64_t bytes, bool out) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + (p ? (uintptr_t)bytes : 0), out};
}

bool meet(const Piece& a, const Piece& b) {   // share a byte
  return a.begin < b.end && b.begin < a.end;
}

// True when an output shares a byte with another piece.
bool clash(std::vector<Piece>& v) {
  auto before = [](const Piece& a, const Piece& b) { return a.begin < b.begin; };
  if (!std::is_sorted(v.begin(), v.end(), before)) std::sort(v.begin(), v.end(), before);
  const Piece *out = nullptr, *in = nullptr;   // the pieces so far that reach farthest
  for (const Piece& p : v) {
    if ((out && meet(*out, p)) || (p.out && in && meet(*in, p))) return true;
    const Piece*& far = p.out ? out : in;
    if (!far || p.end > far->end) far = &p;
  }
  return false;
}

// Calls f(first, count, chunks) for each launch's run of tensors, at most `most` of them.
template <typename F>
hipError_t each_launch(const int64_t* sizes, int32_t n, int most, F f) {
  for (int32_t first = 0; first < n; first += most) {
    const int32_t count = std::min(most, n - first);
    int64_t chunks = 0;
    for (int32_t t = 0; t < count; ++t) chunks += chunks_of(sizes[first + t]);
    if (hipError_t e = f(first, count, chunks)) return e;
  }
  return hipSuccess;
}

uint32_t blocks_of(int64_t chunks) {
  return (uint32_t)std::max<int64_t>(1, std::min<int64_t>(chunks, gc::kGradBlocks));
}

// The part of a table that both kernels have.
template <typename Table>
void fill(Table& t, const void* const* p, const int64_t* sizes, const int32_t* dtypes, int32_t first,
          int32_t count, int64_t chunks) {
  uint32_t c = 0;
  for (int32_t i = 0; i < count; ++i) {
    const int64_t n = sizes[first + i], k = chunks_of(n);
    t.p[i] = p[first + i];
    t.first[i] = c;
    t.tail[i] = (uint32_t)(n - (k ? k - 1 : 0) * gc::kGradChunk) | (uint32_t)dtypes[first + i] << 16;
    c += (uint32_t)k;
  }
  t.first[count] = c;
  t.n = count;
  t.blocks = blocks_of(chunks);
}

// Partial sums of a call: 8 bytes each, and behind them where each tensor's are.
int64_t sums_of(const int64_t* sizes, int32_t n) {
  int64_t total = 0;
  each_launch(sizes, n, gc::kNormTensors, [&](int32_t, int32_t count, int64_t chunks) {
    total += blocks_of(chunks) + count;
    return hipSuccess;
  });
  return total;
}

}  // namespace

extern "C" {

int gc_grad_norm_workspace(const int64_t* sizes, int32_t n, int64_t* bytes) {
  if (!bytes) return GC_ERR_INVALID_ARG;
  if (int rc = check_sizes(sizes, n)) return rc;
  *bytes = (sums_of(sizes, n) + n) * 8;
  return GC_OK;
}

int gc_grad_norm(const void* const* tensors, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                 float* norm, float* norms, void* workspace, int64_t workspace_bytes, void* stream) {
  int64_t need = 0;
  if (int rc = gc_grad_norm_workspace(sizes, n, &need)) return rc;
  if (!valid_tensors(tensors, sizes, dtypes, n) || !norm || !aligned(norm, 4) ||
      !aligned(norms, 4) || workspace_bytes < need || (need && !workspace) || !aligned(workspace, 16))
    return GC_ERR_INVALID_ARG;
  const Piece outs[3] = {piece(norm, 4, true), piece(norms, (int64_t)n * 4, true),
                         piece(workspace, need, true)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(outs[j], outs[i])) return GC_ERR_INVALID_ARG;
    for (int32_t t = 0; t < n; ++t)
      if (meet(piece(tensors[t], sizes[t] * size_of(dtypes[t]), false), outs[i]))
        return GC_ERR_INVALID_ARG;
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  double* sums = static_cast<double*>(workspace);
  gc::GradSums* of = reinterpret_cast<gc::GradSums*>(sums + (need / 8 - n));
  uint32_t base = 0;
  hipError_t e = each_launch(
      sizes, n, gc::kNormTensors, [&](int32_t first, int32_t count, int64_t chunks) -> hipError_t {
        gc::NormTable t;
        fill(t, tensors, sizes, dtypes, first, count, chunks);
        if (hipError_t r = gc::launch_grad_squares(t, sums + base, of + first, base, st)) return r;
        base += t.blocks + (uint32_t)count;
        return hipSuccess;
      });
  if (e == hipSuccess) e = gc::launch_grad_roots(sums, base, of, n, norm, norms, st);
  return status(e);
}

int gc_grad_clip(const void* const* tensors, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                 void* const* out, const int32_t* out_dtypes, float max_norm, const float* norm,
                 float* factors, int64_t n_factors, void* stream) {
  if (int rc = check_sizes(sizes, n)) return rc;
  if (n_factors < 0 || !(max_norm >= 0.0f)) return GC_ERR_INVALID_ARG;
  if (n_factors > kMostElements) return GC_ERR_UNSUPPORTED;
  if (!factors) n_factors = 0;
  if (!valid_tensors(tensors, sizes, dtypes, n) ||
      !valid_tensors(out, sizes, out_dtypes, n) || !norm || !aligned(norm, 4) || !aligned(factors, 4))
    return GC_ERR_INVALID_ARG;
  try {
    std::vector<Piece> v;
    v.reserve(2 * (size_t)n + 2);
    auto add = [&](const Piece& p) {
      if (p.end > p.begin) v.push_back(p);
    };
    for (int32_t t = 0; t < n; ++t) {
      // an output in its tensor's place has to be of its type: then the two are one piece
      if (out[t] != tensors[t])
        add(piece(tensors[t], sizes[t] * size_of(dtypes[t]), false));
      else if (sizes[t] && out_dtypes[t] != dtypes[t])
        return GC_ERR_INVALID_ARG;
      add(piece(out[t], sizes[t] * size_of(out_dtypes[t]), true));
    }
    add(piece(norm, 4, false));
    add(piece(factors, n_factors * 4, true));
    if (clash(v)) return GC_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return GC_ERR_OOM;
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
  int64_t written = 0;
  for (int32_t t = 0; t < n; ++t) written += sizes[t] * size_of(out_dtypes[t]);
  hipError_t e = each_launch(
      sizes, n, gc::kClipTensors, [&](int32_t first, int32_t count, int64_t chunks) -> hipError_t {
        if (!chunks) return hipSuccess;
        gc::ClipTable t;
        fill(t, tensors, sizes, dtypes, first, count, chunks);
        for (int32_t i = 0; i < count; ++i) {
          t.out[i] = out[first + i];
          t.tail[i] |= (uint32_t)out_dtypes[first + i] << 18 |
                       (uint32_t)(out[first + i] == tensors[first + i]) << 20;
        }
        return gc::launch_grad_clip(t, written > kCache, max_norm, norm, st);
      });
  if (e == hipSuccess && n_factors)
    e = gc::launch_grad_factors(max_norm, norm, factors, n_factors, st);
  return status(e);
}

}  // extern "C"
