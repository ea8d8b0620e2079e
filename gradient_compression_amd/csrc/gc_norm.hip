// gc_norm.hip -- root-mean-square norm with the residual's addition and the 8-bit checkpoint of
// its normalised rows, and its backward pass from that checkpoint.
//
// Forward, per row of K columns:
//   h = round(x + residual);  rstd = fl32(1 / sqrt(sum(h^2) / K + eps)), the sum in double;
//   z = fl(h * rstd);  y = round(z * w);  codes and exponents of z.
// Backward, with z as the checkpoint restores it:
//   t = dy * w;  c = mean(t * z);  dx = rstd * (t - z * c) + dres;  dw = sum over rows of dy * z.
//
// Both are streams (4 s + 1.03 and 3 s + 1.03 bytes an element), so HBM bounds them: a row stays
// in registers between its sum and its outputs, everything is read once.  The square sum is in
// double because the codes next to a rounding border follow rstd's last bit (and so that no
// finite row overflows); it costs one double operation an element, hidden under the loads.
#include "gc_act_internal.h"

#include "gc_act.h"

namespace gc {
namespace {

// Sums over the threads that hold one row (a wave, or the whole block of TPR threads); valid in
// every one of them.  The order is fixed.
template <int TPR, typename S>
__device__ __forceinline__ S row_sum(S v, S* s_part) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  if (TPR == 64) return v;
  if (lane_id() == 0) s_part[wave_id()] = v;
  __syncthreads();
  S t = s_part[0];
#pragma unroll
  for (int i = 1; i < TPR / 64; ++i) t += s_part[i];
  __syncthreads();
  return t;
}

// Threads of a block: rows of up to 64 * NV octets take one wave each, four to a block.
template <int TPR>
constexpr int block_threads() {
  return TPR == 64 ? 256 : TPR;
}

template <int DT, bool kVec, bool kRandom, int TPR, int NV>
__global__ __launch_bounds__(block_threads<TPR>()) void k_rmsnorm(NormArgs a) {
  typedef typename Elt<DT>::T T;
  __shared__ double s_part[16];
  constexpr int kRows = block_threads<TPR>() / TPR;
  const int t = TPR == 64 ? lane_id() : threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * kRows + (TPR == 64 ? wave_id() : 0);
  if (row >= a.rows) return;   // a whole wave (TPR 64) or nobody
  const int cols = a.cols, octets = (cols + kActGroup - 1) / kActGroup * (kActGroup / 8);
  const T* x = static_cast<const T*>(a.x.p) + row * a.x.ld;
  const T* res = a.res.p ? static_cast<const T*>(a.res.p) + row * a.res.ld : nullptr;
  T* hp = a.h.p ? static_cast<T*>(a.h.p) + row * a.h.ld : nullptr;
  T* yp = a.y.p ? static_cast<T*>(a.y.p) + row * a.y.ld : nullptr;

  float h[NV][8];
  double ss = 0.0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = (t + v * TPR) * 8;
    load8<DT, kVec>(x, col, cols, h[v]);
  }
  if (res) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (t + v * TPR) * 8;
      float r[8];
      load8<DT, kVec>(res, col, cols, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = to_float(round_to<DT>(h[v][j] + r[j]));
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (hp) store8<DT, kVec>(hp, (t + v * TPR) * 8, cols, h[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)h[v][j], (double)h[v][j], ss);
  }
  ss = row_sum<TPR>(ss, s_part);
  const float rstd = (float)(1.0 / sqrt(ss / (double)cols + (double)a.eps));
  if (t == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int octet = t + v * TPR, col = octet * 8;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      h[v][j] = h[v][j] * rstd;
      const float w = a.weight && col + j < cols ? load_any(a.weight, a.weight_dtype, col + j)
                                                 : 1.0f;
      y[j] = h[v][j] * w;
    }
    if (yp) store8<DT, kVec>(yp, col, cols, y);
    if (a.codes && octet < octets) {   // whole quads at a time
      // columns past the row hold 0 * rstd: 0, or NaN where rstd is Inf, which must not reach
      // the last group's scale
      if (col + 8 > cols)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col + j >= cols) h[v][j] = 0.0f;
      const int64_t i = row * octets + octet;
      uint32_t e;
      const u2 q = encode8<kRandom>(h[v], (uint64_t)i * 2, a.round.seed_lo, a.round.seed_hi,
                                    a.round.step_lo, &e);
      reinterpret_cast<u2*>(a.codes)[i] = q;
      if ((octet & 3) == 0) a.exps[i >> 2] = (uint8_t)e;
    }
  }
}

template <int DT, bool kVec, int TPR, int NV>
__global__ __launch_bounds__(block_threads<TPR>()) void k_rmsnorm_backward(NormGradArgs a,
                                                                           int64_t workers) {
  typedef typename Elt<DT>::T T;
  __shared__ float s_part[16];
  constexpr int kRows = block_threads<TPR>() / TPR;
  const int t = TPR == 64 ? lane_id() : threadIdx.x;
  const int64_t worker = (int64_t)blockIdx.x * kRows + (TPR == 64 ? wave_id() : 0);
  if (worker >= workers) return;   // a whole wave (TPR 64) or nobody
  const int cols = a.cols, octets = (cols + kActGroup - 1) / kActGroup * (kActGroup / 8);
  float dw[NV][8] = {};
  for (int64_t row = worker; row < a.rows; row += workers) {
    const T* dy = static_cast<const T*>(a.dy.p) + row * a.dy.ld;
    const T* dres = a.dres.p ? static_cast<const T*>(a.dres.p) + row * a.dres.ld : nullptr;
    T* dx = static_cast<T*>(a.dx.p) + row * a.dx.ld;
    float g[NV][8], z[NV][8];
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int octet = t + v * TPR, col = octet * 8;
      load8<DT, kVec>(dy, col, cols, g[v]);
      if (octet < octets) {
        const int64_t i = row * octets + octet;
        decode8(reinterpret_cast<const u2*>(a.codes)[i], exponent_scale(a.exps[i >> 2]), z[v]);
      }
      // the padding of the last octets is not part of the row, whatever its group restores to
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j >= cols) z[v][j] = 0.0f;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (t + v * TPR) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[v][j] = fmaf(g[v][j], z[v][j], dw[v][j]);
        const float w = a.weight && col + j < cols ? load_any(a.weight, a.weight_dtype, col + j)
                                                   : 1.0f;
        g[v][j] = g[v][j] * w;
        s = fmaf(g[v][j], z[v][j], s);
      }
    }
    const float c = row_sum<TPR>(s, s_part) / (float)cols;
    const float rstd = a.rstd[row];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (t + v * TPR) * 8;
      float r[8];
      if (dres) load8<DT, kVec>(dres, col, cols, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = rstd * fmaf(-z[v][j], c, g[v][j]);
        g[v][j] = dres ? d + r[j] : d;
      }
      store8<DT, kVec>(dx, col, cols, g[v]);
    }
  }
  if (!a.dweight) return;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int octet = t + v * TPR;
    if (octet >= octets) continue;
    f4* p = reinterpret_cast<f4*>(a.ws + (worker * octets + octet) * 8);
    p[0] = f4{dw[v][0], dw[v][1], dw[v][2], dw[v][3]};
    p[1] = f4{dw[v][4], dw[v][5], dw[v][6], dw[v][7]};
  }
}

// dw[k] (+)= the workers' partial sums, added in a fixed order: slice s of 32 sums the workers
// s, s + 32, ... of a column, then the slices are joined.
__global__ __launch_bounds__(1024) void k_norm_dweight(const float* ws, int64_t workers,
                                                       int32_t pitch, int32_t cols, float* dw,
                                                       int accumulate) {
  __shared__ float s_sum[32][33];
  const int c = threadIdx.x & 31, s = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;    // below pitch, a multiple of 32
  float acc = 0.0f;
  for (int64_t i = s; i < workers; i += 32) acc += ws[i * pitch + col];
  s_sum[s][c] = acc;
  __syncthreads();
  if (s == 0 && col < cols) {
    float t = s_sum[0][c];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += s_sum[i][c];
    dw[col] = accumulate ? dw[col] + t : t;
  }
}

bool vectors(const Mat& a, int dtype) {
  const int64_t bytes = dtype == kF32 ? 4 : 2;
  return (reinterpret_cast<uintptr_t>(a.p) & 15) == 0 && (a.ld * bytes & 15) == 0;
}

// Calls f with the threads per row and the octets per thread as constants.  Rows of up to 2048
// columns take a wave, which needs no barrier; longer ones a block.
template <typename F>
void by_columns(int32_t cols, F&& f) {
  const int octets = (cols + 7) / 8;
  if (octets <= 64)
    f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  else if (octets <= 128)
    f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  else if (octets <= 256)
    f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
  else if (octets <= 512)
    f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  else if (octets <= 1024)
    f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
  else if (octets <= 2048)
    f(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
  else
    f(std::integral_constant<int, 1024>(), std::integral_constant<int, 4>());
}

template <int DT, bool kVec, bool kRandom>
void forward(const NormArgs& a, hipStream_t st) {
  by_columns(a.cols, [&](auto tpr, auto nv) {
    constexpr int nt = block_threads<tpr>();
    k_rmsnorm<DT, kVec, kRandom, tpr, nv>
        <<<blocks_for(a.rows, nt / tpr), nt, 0, st>>>(a);
  });
}

template <int DT>
void forward(const NormArgs& a, hipStream_t st) {
  const bool vec = vectors(a.x, DT) && (!a.res.p || vectors(a.res, DT)) &&
                   (!a.h.p || vectors(a.h, DT)) && (!a.y.p || vectors(a.y, DT));
  if (vec)
    a.round.random ? forward<DT, true, true>(a, st) : forward<DT, true, false>(a, st);
  else
    a.round.random ? forward<DT, false, true>(a, st) : forward<DT, false, false>(a, st);
}

template <int DT, bool kVec>
void backward(const NormGradArgs& a, hipStream_t st) {
  const int64_t workers = norm_grad_workers(a.rows, a.cols);
  by_columns(a.cols, [&](auto tpr, auto nv) {
    constexpr int nt = block_threads<tpr>();
    k_rmsnorm_backward<DT, kVec, tpr, nv>
        <<<blocks_for(workers, nt / tpr), nt, 0, st>>>(a, workers);
  });
}

template <int DT>
void backward(const NormGradArgs& a, hipStream_t st) {
  const bool vec = vectors(a.dy, DT) && (!a.dres.p || vectors(a.dres, DT)) && vectors(a.dx, DT);
  vec ? backward<DT, true>(a, st) : backward<DT, false>(a, st);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  a.dtype == kF32 ? forward<kF32>(a, st) : a.dtype == kBF16 ? forward<kBF16>(a, st)
                                                            : forward<kF16>(a, st);
  return hipGetLastError();
}

int64_t norm_grad_workers(int64_t rows, int32_t cols) {
  (void)cols;
  return rows < 1024 ? rows : 1024;
}

hipError_t launch_rmsnorm_backward(const NormGradArgs& a, hipStream_t st) {
  if (a.cols == 0) return hipSuccess;
  if (a.rows) {
    a.dtype == kF32 ? backward<kF32>(a, st) : a.dtype == kBF16 ? backward<kBF16>(a, st)
                                                               : backward<kF16>(a, st);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.dweight && !(a.rows == 0 && a.accumulate)) {
    const int32_t pitch = (a.cols + kActGroup - 1) / kActGroup * kActGroup;
    k_norm_dweight<<<pitch / 32, 1024, 0, st>>>(a.ws, norm_grad_workers(a.rows, a.cols), pitch,
                                                a.cols, a.dweight, a.accumulate);
  }
  return hipGetLastError();
}

}  // namespace gc
