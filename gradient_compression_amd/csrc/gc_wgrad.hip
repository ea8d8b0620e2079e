// gc_wgrad.hip -- the weight gradient of a linear layer whose input was kept as an 8-bit
// checkpoint: dW[n][k] (+)= s[k] * sum over rows m of dY[m][n] * Z[m][k], Z = code * 2^e.
//
// A restored value has at most 7 bits and a sign, so it is exact in bf16 and the product runs on
// the bf16 matrix cores with exact operands: dY in bf16 as it is, in fp16 as two bf16 parts, in
// fp32 as three (8 bits each, cut off the top one after the other, so that their sum is the value).
// Products of two bf16 are exact in fp32, the sums are in fp32.
#include "gc_act_internal.h"

#include "gc_act.h"

namespace gc {
namespace {

typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s4 lds_s4;

constexpr int kTileN = 128, kTileK = 128, kStep = 32, kThreadsW = 256;
// 64 bytes past the row: the four rows of a transposing read start in different quarters of the banks
constexpr int kPitchN = kTileN + 32, kPitchK = kTileK + 32;

// The parts of a value of the type: bf16 1, fp16 2, fp32 3.
template <int DT>
constexpr int parts() {
  return DT == kBF16 ? 1 : DT == kF16 ? 2 : 3;
}

__device__ __forceinline__ uint32_t pack_high(float a, float b) {   // their upper halves
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
}

// One 32x32x16 operand of a wave: 8 rows of the tile for each lane's column, read across the rows of LDS.
__device__ __forceinline__ b8 fragment(const short* base, int pitch) {
  const int l = lane_id(), b = l >> 4, i = l & 15;
  const short* p = base + (8 * (b >> 1) + (i >> 2)) * pitch + 16 * (b & 1) + 4 * (i & 3);
  const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
  const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 4 * pitch));
  return __builtin_bit_cast(b8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

template <int DT, bool kVec>
__global__ __launch_bounds__(kThreadsW) void k_wgrad(WgradArgs a, int splits) {
  typedef typename Elt<DT>::T T;
  constexpr int NS = parts<DT>();
  __shared__ __align__(16) short s_y[NS][kStep][kPitchN];
  __shared__ __align__(16) short s_z[kStep][kPitchK];
  const int n0 = blockIdx.y * kTileN, k0 = blockIdx.x * kTileK;
  const int wave = wave_id(), lane = lane_id();
  const int wn = (wave >> 1) * 64, wk = (wave & 1) * 64;
  const int groups = (a.cols + kActGroup - 1) / kActGroup, octets = groups * (kActGroup / 8);
  const int64_t steps = (a.rows + kStep - 1) / kStep;
  const int64_t first = steps * blockIdx.z / splits, last = steps * (blockIdx.z + 1) / splits;
  f16v acc[2][2] = {};
  for (int64_t s = first; s < last; ++s) {
    const int64_t m0 = s * kStep;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int o = threadIdx.x + p * kThreadsW, r = o >> 4, c = (o & 15) * 8;
      const int64_t m = m0 + r;
      const bool in = m < a.rows;
      float v[8] = {};
      if (in) load8<DT, kVec>(static_cast<const T*>(a.dy.p) + m * a.dy.ld, n0 + c, a.n_out, v);
      if constexpr (DT == kF32) {   // a NaN whose upper half alone would read as Inf
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (v[j] != v[j]) v[j] = __uint_as_float(0x7FC00000u);
      }
#pragma unroll
      for (int q = 0; q < NS; ++q) {
        u4 w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack_high(v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<u4*>(&s_y[q][r][c]) = w;
        if (q + 1 < NS)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // what is left under the 8 bits just taken; nothing is left of Inf and NaN
            const float top = __uint_as_float(__float_as_uint(v[j]) & 0xFFFF0000u);
            v[j] = mag_key(v[j]) < 0x7F800000u ? v[j] - top : 0.0f;
          }
      }
      float z[8] = {};
      const int octet = k0 / 8 + (o & 15);
      if (in && octet < octets) {
        const int64_t i = m * octets + octet;
        decode8(reinterpret_cast<const u2*>(a.codes)[i], exponent_scale(a.exps[i >> 2]), z);
      }
      u4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_high(z[2 * j], z[2 * j + 1]);
      *reinterpret_cast<u4*>(&s_z[r][c]) = w;
    }
    __syncthreads();
#pragma unroll
    for (int mm = 0; mm < kStep; mm += 16) {
      b8 fz[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) fz[j] = fragment(&s_z[mm][wk + 32 * j], kPitchK);
#pragma unroll
      for (int q = 0; q < NS; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const b8 fy = fragment(&s_y[q][mm][wn + 32 * i], kPitchN);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fy, fz[j], acc[i][j], 0, 0, 0);
        }
    }
  }
  float* out = splits > 1 ? a.ws + (int64_t)blockIdx.z * a.n_out * a.cols : a.dw;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int k = k0 + wk + 32 * j + (lane & 31);
    if (k >= a.cols) continue;
    const float sc = splits == 1 && a.col_scale ? load_any(a.col_scale, a.scale_dtype, k) : 1.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int n = n0 + wn + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
        if (n >= a.n_out) continue;
        float* p = out + (int64_t)n * a.cols + k;
        const float v = acc[i][j][r] * sc;
        *p = splits == 1 && a.accumulate ? *p + v : v;
      }
  }
}

// The parts of the row sum joined in order, scaled and stored.
__global__ __launch_bounds__(256) void k_wgrad_join(WgradArgs a, int splits) {
  const int64_t total = (int64_t)a.n_out * a.cols;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  float v = a.ws[i];
  for (int s = 1; s < splits; ++s) v += a.ws[s * total + i];
  if (a.col_scale) v *= load_any(a.col_scale, a.scale_dtype, i % a.cols);
  a.dw[i] = a.accumulate ? a.dw[i] + v : v;
}

template <int DT>
void wgrad(const WgradArgs& a, int splits, hipStream_t st) {
  const dim3 grid(blocks_for(a.cols, kTileK), blocks_for(a.n_out, kTileN), splits);
  const bool vec = (reinterpret_cast<uintptr_t>(a.dy.p) & 15) == 0 &&
                   (a.dy.ld * (int64_t)sizeof(typename Elt<DT>::T) & 15) == 0;
  if (vec)
    k_wgrad<DT, true><<<grid, kThreadsW, 0, st>>>(a, splits);
  else
    k_wgrad<DT, false><<<grid, kThreadsW, 0, st>>>(a, splits);
}

}  // namespace

int wgrad_splits(int64_t rows, int32_t n_out, int32_t cols, int dtype) {
  (void)dtype;
  const int64_t tiles = ((int64_t)n_out + kTileN - 1) / kTileN * (((int64_t)cols + kTileK - 1) / kTileK);
  const int64_t steps = (rows + kStep - 1) / kStep;
  int64_t s = tiles ? 512 / tiles : 1;
  if (s > steps / 4) s = steps / 4;
  return s < 1 ? 1 : s > 16 ? 16 : (int)s;
}

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t st) {
  if (a.n_out == 0 || a.cols == 0 || (a.rows == 0 && a.accumulate)) return hipSuccess;
  const int splits = wgrad_splits(a.rows, a.n_out, a.cols, a.dtype);
  a.dtype == kF32 ? wgrad<kF32>(a, splits, st) : a.dtype == kBF16 ? wgrad<kBF16>(a, splits, st)
                                                                  : wgrad<kF16>(a, splits, st);
  if (hipError_t e = hipGetLastError()) return e;
  if (splits > 1)
    k_wgrad_join<<<blocks_for((int64_t)a.n_out * a.cols, 256), 256, 0, st>>>(a, splits);
  return hipGetLastError();
}

}  // namespace gc
