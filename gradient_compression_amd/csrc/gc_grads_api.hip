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
    total += sizes[t];   // at most 2^20 * 2^44
  }
  return total > kMostElements ? GC_ERR_UNSUPPORTED : GC_OK;
}

bool valid_tensors(const void* const* p, const int64_t* sizes, const int32_t* dtypes, int32_t n) {
  if (n > 0 && (!p || !dtypes)) return false;
  for (int32_t t = 0; t < n; ++t)
    if (!valid_dtype(dtypes[t]) || (sizes[t] && (!p[t] || !aligned(p[t], size_of(dtypes[t])))))
      return false;
  return true;
}

// A piece of memory that a call reads or writes; `of`: the tensor that it is, or -1.
struct Piece {
  uintptr_t begin, end;
  int32_t of;
  bool out;
};

void add(std::vector<Piece>& v, const void* p, int64_t bytes, int32_t of, bool out) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  if (p && bytes > 0) v.push_back({b, b + (uintptr_t)bytes, of, out});
}

// True when an output shares a byte with another piece, but for an output that is its own tensor.
bool clash(std::vector<Piece>& v) {
  std::sort(v.begin(), v.end(),
            [](const Piece& a, const Piece& b) { return a.begin < b.begin; });
  // the pieces so far that reach farthest: of the outputs, and of the inputs
  const Piece* out = nullptr;
  const Piece* in = nullptr;
  const Piece* in2 = nullptr;   // the farthest input of another tensor than `in`
  auto meet = [](const Piece* a, const Piece& b) {
    return a && a->end > b.begin &&
           !(a->of >= 0 && a->of == b.of && a->out != b.out && a->begin == b.begin &&
             a->end == b.end);
  };
  for (const Piece& p : v) {
    if (meet(out, p) || (p.out && (meet(in, p) || meet(in2, p)))) return true;
    if (p.out) {
      if (!out || p.end > out->end) out = &p;
    } else if (!in || p.end > in->end) {
      if (in && in->of != p.of) in2 = in;
      in = &p;
    } else if (p.of != in->of && (!in2 || p.end > in2->end)) {
      in2 = &p;
    }
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
  try {
    std::vector<Piece> v;
    v.reserve(n + 3);
    for (int32_t t = 0; t < n; ++t) add(v, tensors[t], sizes[t] * size_of(dtypes[t]), t, false);
    add(v, norm, 4, -1, true);
    add(v, norms, (int64_t)n * 4, -1, true);
    add(v, workspace, need, -1, true);
    if (clash(v)) return GC_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return GC_ERR_OOM;
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
    for (int32_t t = 0; t < n; ++t) {
      // an output in its tensor's place has to be of its type: then the two pieces are alike
      add(v, tensors[t], sizes[t] * size_of(dtypes[t]), t, false);
      add(v, out[t], sizes[t] * size_of(out_dtypes[t]), t, true);
      if (sizes[t] && out[t] == tensors[t] && out_dtypes[t] != dtypes[t]) return GC_ERR_INVALID_ARG;
    }
    add(v, norm, 4, -1, false);
    add(v, factors, n_factors * 4, -1, true);
    if (clash(v)) return GC_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return GC_ERR_OOM;
  }
  const hipStream_t st = static_cast<hipStream_t>(stream);
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
        return gc::launch_grad_clip(t, max_norm, norm, st);
      });
  if (e == hipSuccess && n_factors)
    e = gc::launch_grad_factors(max_norm, norm, factors, n_factors, st);
  return status(e);
}

}  // extern "C"
