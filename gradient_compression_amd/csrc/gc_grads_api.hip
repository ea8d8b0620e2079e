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

// Whether the outputs lie one behind the other, as in a flat gradient, and no input between the first and
// the last: the common case, told without sorting, as a first launch waits for the checks.
bool apart(const std::vector<Piece>& v) {
  const Piece *first = nullptr, *last = nullptr;
  for (const Piece& p : v)
    if (p.out) {
      if (last && p.begin < last->end) return false;
      if (!first) first = &p;
      last = &p;
    }
  if (!first) return true;
  const Piece all = {first->begin, last->end, true};
  for (const Piece& p : v)
    if (!p.out && meet(all, p)) return false;
  return true;
}

// True when an output shares a byte with another piece.
bool clash(std::vector<Piece>& v) {
  if (apart(v)) return false;
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

// Bytes of a call's partial sums, 8 each, and behind them where each tensor's are.
int64_t workspace_of(const int64_t* sizes, int32_t n) {
  int64_t total = 0;
  each_launch(sizes, n, gc::kNormTensors, [&](int32_t, int32_t count, int64_t chunks) {
    total += blocks_of(chunks) + count;
    return hipSuccess;
  });
  return (total + n) * 8;
}

// A call's tensors.
struct Tensors {
  const void* const* p;
  const int64_t* sizes;
  const int32_t* dtypes;
  int32_t n;
};

// What gc_grad_norm refuses; the workspace it needs.
int check_norm(const Tensors& in, const float* norm, const float* norms, const void* workspace,
               int64_t workspace_bytes, int64_t* need) {
  if (int rc = check_sizes(in.sizes, in.n)) return rc;
  *need = workspace_of(in.sizes, in.n);
  if (!valid_tensors(in.p, in.sizes, in.dtypes, in.n) || !norm || !aligned(norm, 4) ||
      !aligned(norms, 4) || workspace_bytes < *need || (*need && !workspace) || !aligned(workspace, 16))
    return GC_ERR_INVALID_ARG;
  const Piece outs[3] = {piece(norm, 4, true), piece(norms, (int64_t)in.n * 4, true),
                         piece(workspace, *need, true)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(outs[j], outs[i])) return GC_ERR_INVALID_ARG;
    for (int32_t t = 0; t < in.n; ++t)
      if (meet(piece(in.p[t], in.sizes[t] * size_of(in.dtypes[t]), false), outs[i]))
        return GC_ERR_INVALID_ARG;
  }
  return GC_OK;
}

hipError_t run_norm(const Tensors& in, float* norm, float* norms, void* workspace, int64_t need,
                    hipStream_t st) {
  double* sums = static_cast<double*>(workspace);
  gc::GradSums* of = reinterpret_cast<gc::GradSums*>(sums + (need / 8 - in.n));
  uint32_t base = 0;
  hipError_t e = each_launch(
      in.sizes, in.n, gc::kNormTensors, [&](int32_t first, int32_t count, int64_t chunks) -> hipError_t {
        gc::NormTable t;
        fill(t, in.p, in.sizes, in.dtypes, first, count, chunks);
        if (hipError_t r = gc::launch_grad_squares(t, sums + base, of + first, base, st)) return r;
        base += t.blocks + (uint32_t)count;
        return hipSuccess;
      });
  return e == hipSuccess ? gc::launch_grad_roots(sums, base, of, in.n, norm, norms, st) : e;
}

// What the scaling writes.
struct Scaled {
  void* const* p;
  const int32_t* dtypes;
  float max_norm;
  float* factors;
  int64_t n_factors;
};

// What gc_grad_clip refuses.
int check_clip(const Tensors& in, const Scaled& out, const float* norm) {
  if (int rc = check_sizes(in.sizes, in.n)) return rc;
  if (out.n_factors < 0 || !(out.max_norm >= 0.0f)) return GC_ERR_INVALID_ARG;
  if (out.n_factors > kMostElements) return GC_ERR_UNSUPPORTED;
  if (!valid_tensors(in.p, in.sizes, in.dtypes, in.n) ||
      !valid_tensors(out.p, in.sizes, out.dtypes, in.n) || !norm || !aligned(norm, 4) ||
      !aligned(out.factors, 4))
    return GC_ERR_INVALID_ARG;
  try {
    std::vector<Piece> v;
    v.reserve(2 * (size_t)in.n + 2);
    auto add = [&](const Piece& p) {
      if (p.end > p.begin) v.push_back(p);
    };
    for (int32_t t = 0; t < in.n; ++t) {
      // an output in its tensor's place has to be of its type: then the two are one piece
      if (out.p[t] != in.p[t])
        add(piece(in.p[t], in.sizes[t] * size_of(in.dtypes[t]), false));
      else if (in.sizes[t] && out.dtypes[t] != in.dtypes[t])
        return GC_ERR_INVALID_ARG;
      add(piece(out.p[t], in.sizes[t] * size_of(out.dtypes[t]), true));
    }
    add(piece(norm, 4, false));
    add(piece(out.factors, out.n_factors * 4, true));
    return clash(v) ? GC_ERR_INVALID_ARG : GC_OK;
  } catch (const std::bad_alloc&) {
    return GC_ERR_OOM;
  }
}

hipError_t run_clip(const Tensors& in, const Scaled& out, const float* norm, hipStream_t st) {
  int64_t written = 0;
  for (int32_t t = 0; t < in.n; ++t) written += in.sizes[t] * size_of(out.dtypes[t]);
  hipError_t e = each_launch(
      in.sizes, in.n, gc::kClipTensors, [&](int32_t first, int32_t count, int64_t chunks) -> hipError_t {
        if (!chunks) return hipSuccess;
        gc::ClipTable t;
        fill(t, in.p, in.sizes, in.dtypes, first, count, chunks);
        for (int32_t i = 0; i < count; ++i) {
          t.out[i] = out.p[first + i];
          t.tail[i] |= (uint32_t)out.dtypes[first + i] << 18 |
                       (uint32_t)(out.p[first + i] == in.p[first + i]) << 20;
        }
        return gc::launch_grad_clip(t, written > kCache, out.max_norm, norm, st);
      });
  if (e == hipSuccess && out.factors && out.n_factors)
    e = gc::launch_grad_factors(out.max_norm, norm, out.factors, out.n_factors, st);
  return e;
}

}  // namespace

extern "C" {

int gc_grad_norm_workspace(const int64_t* sizes, int32_t n, int64_t* bytes) {
  if (!bytes) return GC_ERR_INVALID_ARG;
  if (int rc = check_sizes(sizes, n)) return rc;
  *bytes = workspace_of(sizes, n);
  return GC_OK;
}

int gc_grad_norm(const void* const* tensors, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                 float* norm, float* norms, void* workspace, int64_t workspace_bytes, void* stream) {
  const Tensors in = {tensors, sizes, dtypes, n};
  int64_t need = 0;
  if (int rc = check_norm(in, norm, norms, workspace, workspace_bytes, &need)) return rc;
  return status(run_norm(in, norm, norms, workspace, need, static_cast<hipStream_t>(stream)));
}

int gc_grad_clip(const void* const* tensors, const int64_t* sizes, const int32_t* dtypes, int32_t n,
                 void* const* out, const int32_t* out_dtypes, float max_norm, const float* norm,
                 float* factors, int64_t n_factors, void* stream) {
  const Tensors in = {tensors, sizes, dtypes, n};
  const Scaled to = {out, out_dtypes, max_norm, factors, n_factors};
  if (int rc = check_clip(in, to, norm)) return rc;
  return status(run_clip(in, to, norm, static_cast<hipStream_t>(stream)));
}

int gc_clip_grad_norm(const void* const* tensors, const int64_t* sizes, const int32_t* dtypes,
                      int32_t n, void* const* out, const int32_t* out_dtypes, float max_norm,
                      float* norm, float* norms, float* factors, int64_t n_factors, void* workspace,
                      int64_t workspace_bytes, void* stream) {
  const Tensors in = {tensors, sizes, dtypes, n};
  const Scaled to = {out, out_dtypes, max_norm, factors, n_factors};
  int64_t need = 0;
  if (int rc = check_norm(in, norm, norms, workspace, workspace_bytes, &need)) return rc;
  if (int rc = check_clip(in, to, norm)) return rc;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = run_norm(in, norm, norms, workspace, need, st);
  return status(e == hipSuccess ? run_clip(in, to, norm, st) : e);
}

}  // extern "C"
