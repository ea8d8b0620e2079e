// gc_act.hip -- writing an activation matrix as an 8-bit checkpoint, and reading it back.
//
// Both are streams: s + 1.03 bytes an element (s the type's size) and about 6 operations, so HBM
// bounds them.  A lane takes one octet (one 16-byte load of a 16-bit type); a group's largest
// magnitude is found inside its quad of lanes, so nothing goes through LDS.  Measured on 8192 x 11008
// bf16: written in 49 us (5.6 TB/s; a copy of 4 GiB reaches 5.0), read back in 43 us (6.3 TB/s; 48 us
// without non-temporal stores).  The codes' writer does not use such stores, which keeps the codes in
// the cache for a reader that follows at once and costs a writer alone: 8192 x 4096 written and read
// 38 us against 41, 4096 x 4096 19.0 against 21.5; written only 22.0 against 19.5 and 10.0 against 10.6
// (8192 x 11008: 49 us either way).  Stochastic rounding is bound by its draws (two Philox blocks for
// 8 columns): 77 us.
#include "gc_act_internal.h"

#include "gc_act.h"

namespace gc {
namespace {

constexpr int kThreadsAct = 256;

RowMap row_map(int64_t rows, int32_t cols) {
  RowMap m;
  m.rows = rows;
  m.cols = cols;
  m.octets = (cols + kActGroup - 1) / kActGroup * (kActGroup / 8);
  m.chunks = (m.octets + 63) / 64;
  m.lanes = 64;
  if (m.chunks == 1)
    while (m.lanes > 4 && m.lanes / 2 >= m.octets) m.lanes /= 2;
  m.units = m.chunks > 1 ? rows * m.chunks : (rows + 64 / m.lanes - 1) / (64 / m.lanes);
  return m;
}

// Row and octet of this lane in wave unit u; false where it has none.
__device__ __forceinline__ bool place(const RowMap& m, int64_t u, int64_t* row, int* octet) {
  const int lane = lane_id();
  if (u >= m.units) return false;
  if (m.chunks > 1) {
    *row = u / m.chunks;
    *octet = (int)(u - *row * m.chunks) * 64 + lane;
  } else {
    const int per = 64 / m.lanes;
    *row = u * per + lane / m.lanes;
    *octet = lane & (m.lanes - 1);
  }
  return *row < m.rows && *octet < m.octets;
}

template <int DT, bool kRandom>
__global__ __launch_bounds__(kThreadsAct) void k_act_quant(RowMap m,
                                                           const typename Elt<DT>::T* x,
                                                           int64_t ld, ActRound r, int8_t* codes,
                                                           uint8_t* exps) {
  const int64_t u = (int64_t)blockIdx.x * (kThreadsAct / 64) + wave_id();
  int64_t row;
  int octet;
  if (!place(m, u, &row, &octet)) return;   // whole quads at a time
  float v[8];
  load8<DT>(x + row * ld, octet * 8, m.cols, v);
  const int64_t i = (row * m.octets + octet);
  uint32_t e;
  const u2 q = encode8<kRandom>(v, (uint64_t)i * 2, r.seed_lo, r.seed_hi, r.step_lo, &e);
  reinterpret_cast<u2*>(codes)[i] = q;
  if ((octet & 3) == 0) exps[i >> 2] = (uint8_t)e;
}

template <int DT, bool kStream>
__global__ __launch_bounds__(kThreadsAct) void k_act_restore(RowMap m, const int8_t* codes,
                                                             const uint8_t* exps,
                                                             typename Elt<DT>::T* out,
                                                             int64_t ld) {
  const int64_t u = (int64_t)blockIdx.x * (kThreadsAct / 64) + wave_id();
  int64_t row;
  int octet;
  if (!place(m, u, &row, &octet)) return;
  const int64_t i = row * m.octets + octet;
  float v[8];
  decode8(reinterpret_cast<const u2*>(codes)[i], exponent_scale(exps[i >> 2]), v);
  store8<DT, kStream>(out + row * ld, octet * 8, m.cols, v);
}

template <int DT>
void quant(const RowMap& m, const Mat& x, const ActRound& r, int8_t* codes, uint8_t* exps,
           hipStream_t st) {
  typedef const typename Elt<DT>::T* P;
  const unsigned grid = blocks_for(m.units, kThreadsAct / 64);
  if (r.random)
    k_act_quant<DT, true><<<grid, kThreadsAct, 0, st>>>(m, (P)x.p, x.ld, r, codes, exps);
  else
    k_act_quant<DT, false><<<grid, kThreadsAct, 0, st>>>(m, (P)x.p, x.ld, r, codes, exps);
}

template <int DT>
void restore(const RowMap& m, const int8_t* codes, const uint8_t* exps, const Mat& out,
             hipStream_t st) {
  typedef typename Elt<DT>::T* P;
  const unsigned grid = blocks_for(m.units, kThreadsAct / 64);
  if (whole_blocks(out, DT))
    k_act_restore<DT, true><<<grid, kThreadsAct, 0, st>>>(m, codes, exps, (P)out.p, out.ld);
  else
    k_act_restore<DT, false><<<grid, kThreadsAct, 0, st>>>(m, codes, exps, (P)out.p, out.ld);
}

}  // namespace

hipError_t launch_act_quant(const Mat& x, int dtype, int64_t rows, int32_t cols,
                            const ActRound& r, int8_t* codes, uint8_t* exps, hipStream_t st) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const RowMap m = row_map(rows, cols);
  if (dtype == kF32)
    quant<kF32>(m, x, r, codes, exps, st);
  else if (dtype == kBF16)
    quant<kBF16>(m, x, r, codes, exps, st);
  else
    quant<kF16>(m, x, r, codes, exps, st);
  return hipGetLastError();
}

hipError_t launch_act_restore(const int8_t* codes, const uint8_t* exps, int64_t rows,
                              int32_t cols, const Mat& out, int dtype, hipStream_t st) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const RowMap m = row_map(rows, cols);
  if (dtype == kF32)
    restore<kF32>(m, codes, exps, out, st);
  else if (dtype == kBF16)
    restore<kBF16>(m, codes, exps, out, st);
  else
    restore<kF16>(m, codes, exps, out, st);
  return hipGetLastError();
}

}  // namespace gc
