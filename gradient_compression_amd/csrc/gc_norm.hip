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
// in registers between its sum and its outputs (but for the backward pass of rows of more than 16384
// columns), everything is read once.  The square sum is in
// double because the codes next to a rounding border follow rstd's last bit (and so that no
// finite row overflows); it costs one double operation an element, hidden under the loads.
// Measured on 8192 x 4096 bf16: forward 54 us (5.6 TB/s; a copy of 4 GiB reaches 5.0), with stochastic
// codes 59; backward 47 us and 4.9 us of its column sums (4.5 TB/s).  fp32: forward 132 us (4.3 TB/s),
// backward 94 (4.6).  Rows of more than 16384 columns do not fit a block's registers in the backward
// pass: 181 (16-bit types) and 425 (fp32) values a thread go through scratch memory in every row, and
// 2048 x 32768 takes 187 and 342 us (2.5 TB/s; 4096 x 16384 109 and 185 us, 4.4 and 4.7 TB/s).
#include "gc_act_internal.h"

#include "gc_act.h"

namespace gc {
namespace {

// Sums over the threads that hold one row (a wave, or the whole block of TPR threads); valid in
// every one of them.  The order is fixed.
template <int TPR, typename S>
__device__ __forceinline__ S row_sum(S v, S* s_part) {
  v = wave_sum(v);
  if (TPR == 64) return v;
  if (lane_id() == 0) s_part[wave_id()] = v;
  __syncthreads();
  S t = s_part[0];
#pragma unroll
  for (int i = 1; i < TPR / 64; ++i) t += s_part[i];
  __syncthreads();
  return t;
}

// This thread's wave, known to be the same in the whole wave: row addresses then stay in scalar registers.
__device__ __forceinline__ int uniform_wave() { return __builtin_amdgcn_readfirstlane(wave_id()); }

// Threads of a block: rows of up to 64 * NV octets take one wave each, four to a block.
template <int TPR>
constexpr int block_threads() {
  return TPR == 64 ? 256 : TPR;
}

template <int DT, bool kRandom, int TPR, int NV, bool kStream>
__global__ __launch_bounds__(block_threads<TPR>()) void k_rmsnorm(NormArgs a) {
  typedef typename Elt<DT>::T T;
  __shared__ double s_part[16];
  constexpr int kRows = block_threads<TPR>() / TPR;
  const int t = TPR == 64 ? lane_id() : threadIdx.x;
  const int64_t row = (int64_t)blockIdx.x * kRows + (TPR == 64 ? uniform_wave() : 0);
  if (row >= a.rows) return;   // a whole wave (TPR 64) or nobody
  const int cols = a.cols, octets = (cols + kActGroup - 1) / kActGroup * (kActGroup / 8);
  const T* x = static_cast<const T*>(a.x.p) + row * a.x.ld;
  const T* res = a.res.p ? static_cast<const T*>(a.res.p) + row * a.res.ld : nullptr;
  T* hp = a.h.p ? static_cast<T*>(a.h.p) + row * a.h.ld : nullptr;
  T* yp = a.y.p ? static_cast<T*>(a.y.p) + row * a.y.ld : nullptr;

  float h[NV][8], w[NV][8];
  double ss = 0.0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int col = (t + v * TPR) * 8;
    load8<DT>(x, col, cols, h[v]);
  }
  if (res) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (t + v * TPR) * 8;
      float r[8];
      load8<DT>(res, col, cols, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = to_float(round_to<DT>(h[v][j] + r[j]));
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (hp) store8<DT, kStream>(hp, (t + v * TPR) * 8, cols, h[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)h[v][j], (double)h[v][j], ss);
  }
  if (yp)
#pragma unroll
    for (int v = 0; v < NV; ++v)
      load8_any(a.weight, a.weight_dtype, (t + v * TPR) * 8, cols, w[v]);
  ss = row_sum<TPR>(ss, s_part);
  const float rstd = (float)(1.0 / sqrt(ss / (double)cols + (double)a.eps));
  if (t == 0 && a.rstd) a.rstd[row] = rstd;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int octet = t + v * TPR, col = octet * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) h[v][j] = h[v][j] * rstd;
    if (yp) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = h[v][j] * w[v][j];
      store8<DT, kStream>(yp, col, cols, y);
    }
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
      // non-temporal at any pitch: they are read in the backward pass (norm alone of 8192 x 4096 bf16
      // into codes 20.3 us against 23.5, 31775 x 1056, whose rows are not whole blocks, 24.2 against
      // 28.3; with y and h 55.5 against 55.9 and 61.4 against 62.5)
      __builtin_nontemporal_store(q, reinterpret_cast<u2*>(a.codes) + i);
      if ((octet & 3) == 0) a.exps[i >> 2] = (uint8_t)e;
    }
  }
}

// Waves of a SIMD that the backward pass's registers are held to: two blocks of 512 threads a CU as
// long as that costs no more than a few spilled registers (9 in 16-bit rows of 3 octets a thread, 12
// and 19 in fp32 rows of 2 and 3).  Blocks of 1024 threads have 128 registers a thread in any case.
template <int TPR, int NV>
constexpr int backward_waves() {
  return TPR == 512 && NV <= 3 ? 4 : 1;
}

// What a thread holds of one row of the backward pass, as it lies in memory.
template <int DT, int NV>
struct GradRow {
  Raw<DT> dy[NV], dres[NV];
  u2 codes[NV];
  uint32_t exps[NV];
  float rstd;
};

// A worker (a wave or a block, as in the forward pass) takes the rows worker, worker + workers, ...
// Its threads keep their columns' weights and partial sums of dw in registers, and with up to 2 octets
// the next row, loaded before the current one is reduced.  A row is held as it was loaded and expanded
// twice: its floats would cost half of the waves.
template <int DT, int TPR, int NV, bool kStream>
__global__ __launch_bounds__(block_threads<TPR>(), (backward_waves<TPR, NV>())) void k_rmsnorm_backward(NormGradArgs a) {
  typedef typename Elt<DT>::T T;
  constexpr int kRows = block_threads<TPR>() / TPR, kWavesN = TPR / 64;
  constexpr bool kAhead = NV <= 2;
  __shared__ float s_part[2][kWavesN];
  __shared__ float s_dw[kRows > 1 ? kRows : 1][kRows > 1 ? TPR * NV * 8 : 1];
  const int t = TPR == 64 ? lane_id() : threadIdx.x;
  const int64_t workers = (int64_t)gridDim.x * kRows;
  const int64_t worker = (int64_t)blockIdx.x * kRows + (TPR == 64 ? uniform_wave() : 0);
  const int cols = a.cols, octets = (cols + kActGroup - 1) / kActGroup * (kActGroup / 8);
  const bool has_res = a.dres.p != nullptr;

  float dw[NV][8] = {}, w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) load8_any(a.weight, a.weight_dtype, (t + v * TPR) * 8, cols, w[v]);
  auto load = [&](int64_t row, GradRow<DT, NV>& r) {
    const T* dy = static_cast<const T*>(a.dy.p) + row * a.dy.ld;
    const T* dres = static_cast<const T*>(a.dres.p) + row * a.dres.ld;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int octet = t + v * TPR, col = octet * 8;
      // past the row's end dy is 0, so whatever the codes are there adds nothing (a bad last group
      // makes the row NaN by its own columns)
      r.dy[v] = load_raw<DT, kStream>(dy, col, cols);
      if (has_res) r.dres[v] = load_raw<DT, kStream>(dres, col, cols);
      r.codes[v] = u2{0, 0};
      r.exps[v] = 0;
      if (octet < octets) {
        const int64_t i = row * octets + octet;
        r.codes[v] = reinterpret_cast<const u2*>(a.codes)[i];
        r.exps[v] = a.exps[i >> 2];
      }
    }
    r.rstd = a.rstd[row];
  };
  GradRow<DT, NV> cur = {}, nxt = {};   // no dres: zeros are added
  int turn = 0;
  if (worker < a.rows) load(worker, cur);
  for (int64_t row = worker; row < a.rows; row += workers) {
    if (kAhead && row + workers < a.rows) load(row + workers, nxt);
    if (!kAhead && row != worker) load(row, cur);
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float g[8], z[8];
      to_float8<DT>(cur.dy[v], g);
      decode8(cur.codes[v], exponent_scale(cur.exps[v]), z);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[v][j] = fmaf(g[j], z[j], dw[v][j]);
        asm("" : "+v"(dw[v][j]));   // now, or g and z are kept for it until the row's end
        s = fmaf(g[j] * w[v][j], z[j], s);
      }
    }
    // the waves' sums alternate between two places, so that one meeting a row is enough
    s = wave_sum(s);
    if (kWavesN > 1) {
      if (lane_id() == 0) s_part[turn][wave_id()] = s;
      __syncthreads();
      s = s_part[turn][0];
#pragma unroll
      for (int i = 1; i < kWavesN; ++i) s += s_part[turn][i];
      turn ^= 1;
    }
    const float c = s / (float)cols;
    // what was loaded made opaque, or the compiler keeps the floats of the first expansion instead
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      asm("" : "+v"(cur.codes[v]), "+v"(cur.exps[v]));
#pragma unroll
      for (int j = 0; j < Raw<DT>::kWords; ++j) asm("" : "+v"(cur.dy[v].w[j]));
    }
    T* dx = static_cast<T*>(a.dx.p) + row * a.dx.ld;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int col = (t + v * TPR) * 8;
      float g[8], z[8], r[8];
      to_float8<DT>(cur.dy[v], g);
      decode8(cur.codes[v], exponent_scale(cur.exps[v]), z);
      to_float8<DT>(cur.dres[v], r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] = cur.rstd * fmaf(-z[j], c, g[j] * w[v][j]) + r[j];
      }
      store8<DT>(dx, col, cols, g);
    }
    if (kAhead) cur = nxt;
  }
  if (!a.dweight) return;
  // One row of partial sums a block: the waves of a block with several workers are joined first.
  if (kRows > 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s_dw[wave_id()][(v * 8 + j) * 64 + t] = dw[v][j];
    __syncthreads();
    if (wave_id() != 0) return;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 1; i < kRows; ++i) dw[v][j] += s_dw[i][(v * 8 + j) * 64 + t];
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int octet = t + v * TPR;
    if (octet >= octets) continue;
    f4* p = reinterpret_cast<f4*>(a.ws + ((int64_t)blockIdx.x * octets + octet) * 8);
    p[0] = f4{dw[v][0], dw[v][1], dw[v][2], dw[v][3]};
    p[1] = f4{dw[v][4], dw[v][5], dw[v][6], dw[v][7]};
  }
}

// dw[k] (+)= the blocks' partial sums in a fixed order.  A workgroup takes 32 columns: 128 slices of
// 8 lanes (4 columns each) add up every 128th row, the slices are joined in the waves, then in LDS.
__global__ __launch_bounds__(1024) void k_norm_dweight(const float* ws, int blocks, int32_t pitch,
                                                       int32_t cols, float* dw, int accumulate) {
  __shared__ f4 s_sum[16][8];
  const int q = threadIdx.x & 7, s = threadIdx.x >> 3;
  const float* p = ws + blockIdx.x * 32 + q * 4;
  f4 acc = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int i = s; i < blocks; i += 128) acc += *reinterpret_cast<const f4*>(p + (int64_t)i * pitch);
#pragma unroll
  for (int d = 8; d < 64; d <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], d, 64);
  if (lane_id() < 8) s_sum[wave_id()][q] = acc;
  __syncthreads();
  const int col = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && col < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s_sum[i][threadIdx.x >> 2][threadIdx.x & 3];
    dw[col] = accumulate ? dw[col] + t : t;
  }
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

template <int DT, bool kRandom>
void forward(const NormArgs& a, hipStream_t st) {
  const bool stream = (!a.h.p || whole_blocks(a.h, DT)) && (!a.y.p || whole_blocks(a.y, DT));
  by_columns(a.cols, [&](auto tpr, auto nv) {
    constexpr int nt = block_threads<tpr>();
    if (stream)
      k_rmsnorm<DT, kRandom, tpr, nv, true><<<blocks_for(a.rows, nt / tpr), nt, 0, st>>>(a);
    else
      k_rmsnorm<DT, kRandom, tpr, nv, false><<<blocks_for(a.rows, nt / tpr), nt, 0, st>>>(a);
  });
}

template <int DT>
void forward(const NormArgs& a, hipStream_t st) {
  a.round.random ? forward<DT, true>(a, st) : forward<DT, false>(a, st);
}

// The backward pass's threads and octets: 512 threads as long as they do, which leaves a thread
// twice the registers of 1024.
template <typename F>
void by_columns_backward(int32_t cols, F&& f) {
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
    f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
  else if (octets <= 1536)
    f(std::integral_constant<int, 512>(), std::integral_constant<int, 3>());
  else if (octets <= 2048)
    f(std::integral_constant<int, 512>(), std::integral_constant<int, 4>());
  else
    f(std::integral_constant<int, 1024>(), std::integral_constant<int, 4>());
}

template <int DT>
void backward(const NormGradArgs& a, hipStream_t st) {
  const unsigned blocks = (unsigned)norm_grad_blocks(a.rows, a.cols);
  // dy and dres of 32 MB each are not in a cache any more: non-temporal loads then take 39.4 us in
  // place of 44.6 for 4096 x 4096 bf16 and a reader of dx, 72.2 in place of 75.6 for 8192 x 4096, 36.2
  // in place of 41.0 for 16384 x 1024, but 25.2 in place of 24.5 for 2048 x 4096.  In fp32 they gain
  // nothing at 32 MB (27.7 us either way) and lose at 128 MB (8192 x 4096 95.8 us against 89.5).
  const bool stream = a.rows * a.cols * (int64_t)sizeof(typename Elt<DT>::T) >= (int64_t)32 << 20;
  by_columns_backward(a.cols, [&](auto tpr, auto nv) {
    if (stream)
      k_rmsnorm_backward<DT, tpr, nv, true><<<blocks, block_threads<tpr>(), 0, st>>>(a);
    else
      k_rmsnorm_backward<DT, tpr, nv, false><<<blocks, block_threads<tpr>(), 0, st>>>(a);
  });
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st) {
  if (a.rows == 0 || a.cols == 0) return hipSuccess;
  a.dtype == kF32 ? forward<kF32>(a, st) : a.dtype == kBF16 ? forward<kBF16>(a, st)
                                                            : forward<kF16>(a, st);
  return hipGetLastError();
}

// Blocks of a backward call: at least 4 rows a worker, so that the partial sums stay small beside
// the rows, but one block a CU first; at most 1024 threads a CU.
int64_t norm_grad_blocks(int64_t rows, int32_t cols) {
  int64_t per = 1, most = 256;
  by_columns_backward(cols, [&](auto tpr, auto) {
    per = block_threads<tpr>() / tpr;   // workers of a block
    most = 256 * 1024 / block_threads<tpr>();
  });
  const int64_t need = (rows + per - 1) / per, want = (rows + 4 * per - 1) / (4 * per);
  const int64_t blocks = want < 256 ? 256 : want > most ? most : want;
  return blocks < need ? blocks : need;
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
    k_norm_dweight<<<pitch / 32, 1024, 0, st>>>(a.ws, (int)norm_grad_blocks(a.rows, a.cols), pitch,
                                                a.cols, a.dweight, a.accumulate);
  }
  return hipGetLastError();
}

}  // namespace gc
