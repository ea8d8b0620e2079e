// gc_act_internal.h -- what the host side of the activation operators (gc_act_api.hip) and their
// kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gc {

// Element types, in the numbering of gc_dtype.
constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;

// A rows x cols matrix with unit column stride and a row pitch in elements.
struct Mat {
  void* p;
  int64_t ld;
};

// Whether a matrix's rows all start on whole 64-byte blocks: stores of it may be non-temporal then.
// (Of others they are not: a block written in two pieces goes to memory twice.  4096 x 8191 fp32:
// 50 us in place of 36 to restore.)
inline bool whole_blocks(const Mat& a, int dtype) {
  const int64_t bytes = dtype == kF32 ? 4 : 2;
  return ((reinterpret_cast<uintptr_t>(a.p) | (uintptr_t)(a.ld * bytes)) & 63) == 0;
}

struct ActRound {              // how codes are rounded
  int random;                  // 0: to nearest even
  uint32_t seed_lo, seed_hi, step_lo;
};

struct NormArgs {
  int32_t dtype, weight_dtype;
  int64_t rows;
  int32_t cols;
  Mat x, res, h, y;            // res, h, y: p may be null
  const void* weight;          // [cols] or null
  float eps;
  float* rstd;                 // [rows] or null
  int8_t* codes;               // with exps, or null
  uint8_t* exps;
  ActRound round;
};

struct NormGradArgs {
  int32_t dtype, weight_dtype;
  int64_t rows;
  int32_t cols;
  Mat dy, dres, dx;            // dres: p may be null
  const int8_t* codes;
  const uint8_t* exps;
  const float* rstd;
  const void* weight;          // or null
  float* dweight;              // [cols] or null
  int accumulate;
  float* ws;                   // [blocks][pitch] partial sums, with dweight
};

struct WgradArgs {
  int32_t dtype, scale_dtype;
  int64_t rows;
  int32_t n_out, cols;
  Mat dy;
  const int8_t* codes;
  const uint8_t* exps;
  const void* col_scale;       // [cols] or null
  float* dw;                   // [n_out][cols]
  int accumulate;
  float* ws;                   // [splits][n_out][cols] where splits > 1
};

constexpr int64_t kNormMostCols = 32768;

hipError_t launch_act_quant(const Mat& x, int dtype, int64_t rows, int32_t cols,
                            const ActRound& r, int8_t* codes, uint8_t* exps, hipStream_t st);
hipError_t launch_act_restore(const int8_t* codes, const uint8_t* exps, int64_t rows,
                              int32_t cols, const Mat& out, int dtype, hipStream_t st);
hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st);
// Blocks of a backward call, each of which writes a row of partial sums of the weight gradient.
int64_t norm_grad_blocks(int64_t rows, int32_t cols);
hipError_t launch_rmsnorm_backward(const NormGradArgs& a, hipStream_t st);
// Parts into which a weight gradient's sum over the rows is split.
int wgrad_splits(int64_t rows, int32_t n_out, int32_t cols, int dtype);
hipError_t launch_wgrad(const WgradArgs& a, hipStream_t st);

}  // namespace gc
