// gc_grads.h -- what the host side of the operators over many tensors (gc_grads_api.hip) and their
// kernels (gc_grads.hip) share.
//
// A call's tensors are cut into chunks of kGradChunk elements (each tensor's last one may be short) and
// taken in order by the blocks of a launch, block b the chunks from b * chunks / blocks on.  The table of
// tensors travels in the launch's arguments, whose 4 KB hold kNormTensors or kClipTensors of them; more
// take further launches.  Nothing is copied to the device and nothing is kept, so that a captured call
// holds its own table.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gc {

constexpr int64_t kGradChunk = 16384;
constexpr uint32_t kGradBlocks = 2048;       // of a launch: 8 of 4 waves on each CU
constexpr int kNormTensors = 240, kClipTensors = 160;

// tail[t]: elements of tensor t's last chunk (bits 0-15), its type (16-17), the output's type (18-19),
// whether the output is the tensor itself (20).
template <int N, bool OUT>
struct GradTable {
  const void* p[N];
  void* out[OUT ? N : 1];
  uint32_t first[N + 1];    // chunk at which tensor t starts; first[n]: chunks of the launch
  uint32_t tail[N];
  int32_t n;
  uint32_t blocks;
};
typedef GradTable<kNormTensors, false> NormTable;
typedef GradTable<kClipTensors, true> ClipTable;

// Where a tensor's partial sums lie among all of the call's.
struct GradSums {
  uint32_t first, count;
};

// The table's tensors' sums of squares: block b's share of tensor t goes to sums[b + t], zeros in
// between (blocks + n of them); of[t] says where tensor t's are, counted from `base`.
hipError_t launch_grad_squares(const NormTable& t, double* sums, GradSums* of, uint32_t base,
                               hipStream_t st);
// norm = sqrt of all `total` sums; norms[t] (where given) = sqrt of tensor t's.
hipError_t launch_grad_roots(const double* sums, uint32_t total, const GradSums* of, int32_t n,
                             float* norm, float* norms, hipStream_t st);
// stream: what is written is more than the cache holds.
hipError_t launch_grad_clip(const ClipTable& t, bool stream, float max_norm, const float* norm,
                            hipStream_t st);
hipError_t launch_grad_factors(float max_norm, const float* norm, float* factors, int64_t n,
                               hipStream_t st);

}  // namespace gc
