// gc_grads.hip -- the l2 norm over many tensors of any of the types, and their scaling by one factor.
//
// Both are streams: the norm reads every tensor once, the scaling reads it again (part of it from the
// 256 MB cache) and writes the result.  Squares and sums are in double, so that neither the range
// of fp32 nor the length of the sum matters; the order of a sum depends on the tensors' sizes alone.
// A block of 4 waves takes a run of 16384-element chunks, so that many small tensors load it as evenly as a
// large one; it has 4 accesses of 16 bytes a lane in flight (8 gained nothing).
//
// Measured: 1.07e9 bf16 elements into one fp32 tensor 1605 us in all, of which the norm reads at 5.9 TB/s and the
// scaling moves 5.2 TB/s (a plain read reaches 7.1, a plain copy 5.4); 335 M elements in 391 tensors 540 us;
// 335 M in place under the limit, which nothing is written for, 238 us (5.65 TB/s), and scaled 789 us.  161
// tensors of 25 M elements take the GPU 28 us, and the host 60 to 64 us to look at.  Going through the tensors
// from their end when scaling, where the cache still holds the last ones, gained 1 % at most.
#include <type_traits>

#include "gc_grads.h"

#include "gc_act_internal.h"

#include "gc_act.h"

namespace gc {
namespace {

constexpr int kThreadsGrad = 256;

// First tensor of the launch whose chunks reach beyond c (a tensor of no chunks never does).
template <typename Table>
__device__ __forceinline__ int tensor_of(const Table& t, uint32_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid + 1] > c)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ uint32_t chunk_of(uint32_t block, uint32_t chunks, uint32_t blocks) {
  return (uint32_t)((uint64_t)block * chunks / blocks);
}

// N elements from p on as fp32, and back: one access of 8 or 16 bytes a lane, at any element.
template <int DT, int N>
__device__ __forceinline__ void load_n(const typename Elt<DT>::T* p, float (&v)[N]) {
  typename Elt<DT>::T t[N];
  __builtin_memcpy(t, p, sizeof t);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = to_float(t[j]);
}
template <int DT, bool STREAM, int N>
__device__ __forceinline__ void store_n(typename Elt<DT>::T* p, const float (&v)[N]) {
  typename Elt<DT>::T t[N];
#pragma unroll
  for (int j = 0; j < N; ++j) t[j] = round_to<DT>(v[j]);
  if constexpr (STREAM && sizeof t == 16) {
    u4 w;
    __builtin_memcpy(&w, t, sizeof w);
    __builtin_nontemporal_store(w, reinterpret_cast<u4_at_any*>(p));
  } else {
    __builtin_memcpy(p, t, sizeof t);
  }
}

constexpr int kFlight = 4;   // a lane's accesses on their way at once

// Sum of squares of n elements from p on, this thread's share.
template <int DT>
__device__ __forceinline__ double squares(const typename Elt<DT>::T* p, int n) {
  constexpr int N = DT == kF32 ? 4 : 8;   // 16 bytes
  double s[4] = {};
  int i = threadIdx.x * N;
  auto pass = [&](auto flight) {
    constexpr int U = decltype(flight)::value, kNext = kThreadsGrad * N;
    for (; i + (U - 1) * kNext + N <= n; i += U * kNext) {
      float v[U][N];
#pragma unroll
      for (int u = 0; u < U; ++u) load_n<DT>(p + i + u * kNext, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < N; ++j) s[j & 3] = fma((double)v[u][j], (double)v[u][j], s[j & 3]);
    }
  };
  pass(std::integral_constant<int, kFlight>());
  pass(std::integral_constant<int, 1>());
  for (int j = i; j < n && j < i + N; ++j) {
    const double v = to_float(p[j]);
    s[0] = fma(v, v, s[0]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ double block_sum(double v, double* tmp) {
  v = wave_sum(v);
  if (lane_id() == 0) tmp[wave_id()] = v;
  __syncthreads();
  const double r = (tmp[0] + tmp[1]) + (tmp[2] + tmp[3]);
  __syncthreads();
  return r;
}

__global__ __launch_bounds__(kThreadsGrad) void k_grad_squares(NormTable t, double* sums,
                                                               GradSums* of, uint32_t base) {
  __shared__ double s_tmp[kThreadsGrad / 64];
  const uint32_t b = blockIdx.x, chunks = t.first[t.n];
  const uint32_t from = chunk_of(b, chunks, t.blocks), to = chunk_of(b + 1, chunks, t.blocks);
  int at = tensor_of(t, from);
  // the slots before this block's first one that are nobody's
  if (b == 0)
    for (int i = threadIdx.x; i < at; i += kThreadsGrad) sums[i] = 0.0;
  if (from == to && threadIdx.x == 0) sums[b + at] = 0.0;   // a launch without chunks
  uint32_t c = from;
  while (c < to) {
    const uint32_t first = t.first[at], next = t.first[at + 1], end = next < to ? next : to;
    const uint32_t info = t.tail[at];
    double s = 0.0;
    for (; c < end; ++c) {
      const int n = c + 1 == next ? (int)(info & 0xFFFFu) : (int)kGradChunk;
      const int64_t off = (int64_t)(c - first) * kGradChunk;
      switch ((info >> 16) & 3) {
        case kF32: s += squares<kF32>(static_cast<const float*>(t.p[at]) + off, n); break;
        case kBF16: s += squares<kBF16>(static_cast<const __bf16*>(t.p[at]) + off, n); break;
        default: s += squares<kF16>(static_cast<const _Float16*>(t.p[at]) + off, n);
      }
    }
    s = block_sum(s, s_tmp);
    if (threadIdx.x == 0) sums[b + at] = s;
    if (c < to) ++at;
  }
  // and those up to the next block's first one
  const int64_t stop = b + 1 < t.blocks ? (int64_t)b + 1 + tensor_of(t, to) : (int64_t)t.blocks + t.n;
  for (int64_t i = (int64_t)b + at + 1 + threadIdx.x; i < stop; i += kThreadsGrad) sums[i] = 0.0;
  if (b == 0)
    for (int i = threadIdx.x; i < t.n; i += kThreadsGrad) {
      const uint32_t c0 = t.first[i], c1 = t.first[i + 1];
      GradSums g = {base, 0};
      if (c1 > c0) {   // chunk c is block ceil((c + 1) * blocks / chunks) - 1's
        const uint32_t b0 = (uint32_t)((((uint64_t)c0 + 1) * t.blocks + chunks - 1) / chunks) - 1;
        const uint32_t b1 = (uint32_t)(((uint64_t)c1 * t.blocks + chunks - 1) / chunks) - 1;
        g = {base + b0 + (uint32_t)i, b1 - b0 + 1};
      }
      of[i] = g;
    }
}

// Block 0: the norm of all; the others: a tensor a wave.
__global__ __launch_bounds__(kThreadsGrad) void k_grad_roots(const double* sums, uint32_t total,
                                                             const GradSums* of, int32_t n,
                                                             float* norm, float* norms) {
  __shared__ double s_tmp[kThreadsGrad / 64];
  double s = 0.0;
  if (blockIdx.x == 0) {
    for (uint32_t i = threadIdx.x; i < total; i += kThreadsGrad) s += sums[i];
    s = block_sum(s, s_tmp);
    if (threadIdx.x == 0) *norm = (float)sqrt(s);
    return;
  }
  const int64_t t = (int64_t)(blockIdx.x - 1) * (kThreadsGrad / 64) + wave_id();
  if (t >= n) return;
  const GradSums g = of[t];
  for (uint32_t i = lane_id(); i < g.count; i += 64) s += sums[g.first + i];
  s = wave_sum(s);
  if (lane_id() == 0) norms[t] = (float)sqrt(s);
}

// 1 where the norm is not above the limit, and where it is Inf or NaN (nothing sensible to scale by).
__device__ __forceinline__ float clip_factor(float norm, float max_norm) {
  return norm > max_norm && norm <= 3.402823466e38f ? max_norm / norm : 1.0f;
}

// 16 bytes of the wider type a lane, so that what a wave stores lies without gaps (bf16 to fp32 by 8
// elements a lane, in two stores with gaps: 1409 us in place of 1286 for 1.07e9 elements).
template <int DI, int DO, bool STREAM>
__device__ __forceinline__ void scale(const typename Elt<DI>::T* p, typename Elt<DO>::T* out, int n,
                                      float f) {
  constexpr int N = DI == kF32 || DO == kF32 ? 4 : 8;
  int i = threadIdx.x * N;
  auto pass = [&](auto flight) {
    constexpr int U = decltype(flight)::value, kNext = kThreadsGrad * N;
    for (; i + (U - 1) * kNext + N <= n; i += U * kNext) {
      float v[U][N];
#pragma unroll
      for (int u = 0; u < U; ++u) load_n<DI>(p + i + u * kNext, v[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[u][j] *= f;
        store_n<DO, STREAM>(out + i + u * kNext, v[u]);
      }
    }
  };
  pass(std::integral_constant<int, kFlight>());
  pass(std::integral_constant<int, 1>());
  for (int j = i; j < n && j < i + N; ++j) out[j] = round_to<DO>(to_float(p[j]) * f);
}

template <int DI, bool STREAM>
__device__ __forceinline__ void scale(const void* p, int64_t off, void* out, int dtype, int n,
                                      float f) {
  typedef const typename Elt<DI>::T* P;
  if (dtype == kF32)
    scale<DI, kF32, STREAM>(static_cast<P>(p) + off, static_cast<float*>(out) + off, n, f);
  else if (dtype == kBF16)
    scale<DI, kBF16, STREAM>(static_cast<P>(p) + off, static_cast<__bf16*>(out) + off, n, f);
  else
    scale<DI, kF16, STREAM>(static_cast<P>(p) + off, static_cast<_Float16*>(out) + off, n, f);
}

template <bool STREAM>
__global__ __launch_bounds__(kThreadsGrad) void k_grad_clip(ClipTable t, float max_norm,
                                                            const float* norm) {
  const float f = clip_factor(*norm, max_norm);
  const uint32_t chunks = t.first[t.n];
  const uint32_t from = chunk_of(blockIdx.x, chunks, t.blocks);
  const uint32_t to = chunk_of(blockIdx.x + 1, chunks, t.blocks);
  int at = tensor_of(t, from);
  for (uint32_t c = from; c < to; ++c) {
    while (c >= t.first[at + 1]) ++at;
    const uint32_t info = t.tail[at];
    if (f == 1.0f && (info >> 20 & 1)) continue;   // it is where it belongs already
    const int n = c + 1 == t.first[at + 1] ? (int)(info & 0xFFFFu) : (int)kGradChunk;
    const int64_t off = (int64_t)(c - t.first[at]) * kGradChunk;
    const int dtype = (info >> 18) & 3;
    switch ((info >> 16) & 3) {
      case kF32: scale<kF32, STREAM>(t.p[at], off, t.out[at], dtype, n, f); break;
      case kBF16: scale<kBF16, STREAM>(t.p[at], off, t.out[at], dtype, n, f); break;
      default: scale<kF16, STREAM>(t.p[at], off, t.out[at], dtype, n, f);
    }
  }
}

__global__ __launch_bounds__(kThreadsGrad) void k_grad_factors(float max_norm, const float* norm,
                                                               float* factors, int64_t n) {
  const float f = clip_factor(*norm, max_norm);
  for (int64_t i = (int64_t)blockIdx.x * kThreadsGrad + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * kThreadsGrad)
    factors[i] = f;
}

}  // namespace

hipError_t launch_grad_squares(const NormTable& t, double* sums, GradSums* of, uint32_t base,
                               hipStream_t st) {
  k_grad_squares<<<t.blocks, kThreadsGrad, 0, st>>>(t, sums, of, base);
  return hipGetLastError();
}

hipError_t launch_grad_roots(const double* sums, uint32_t total, const GradSums* of, int32_t n,
                             float* norm, float* norms, hipStream_t st) {
  const unsigned grid = 1 + (norms ? blocks_for(n, kThreadsGrad / 64) : 0);
  k_grad_roots<<<grid, kThreadsGrad, 0, st>>>(sums, total, of, n, norm, norms);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const ClipTable& t, bool stream, float max_norm, const float* norm,
                            hipStream_t st) {
  if (stream)
    k_grad_clip<true><<<t.blocks, kThreadsGrad, 0, st>>>(t, max_norm, norm);
  else
    k_grad_clip<false><<<t.blocks, kThreadsGrad, 0, st>>>(t, max_norm, norm);
  return hipGetLastError();
}

hipError_t launch_grad_factors(float max_norm, const float* norm, float* factors, int64_t n,
                               hipStream_t st) {
  const int64_t blocks = (n + kThreadsGrad - 1) / kThreadsGrad;
  k_grad_factors<<<(unsigned)(blocks < 1024 ? blocks : 1024), kThreadsGrad, 0, st>>>(max_norm, norm,
                                                                                     factors, n);
  return hipGetLastError();
}

}  // namespace gc
