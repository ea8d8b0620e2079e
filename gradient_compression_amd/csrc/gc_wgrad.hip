// gc_wgrad.hip -- the weight gradient of a linear layer whose input was kept as an 8-bit
// checkpoint: dW[n][k] (+)= s[k] * sum over rows m of dY[m][n] * Z[m][k], Z = code * 2^e.
//
// A restored value has at most 7 bits and a sign, so it is exact in bf16 and the product runs on
// the bf16 matrix cores with exact operands: dY in bf16 as it is, in fp16 as two bf16 parts, in
// fp32 as three (8 bits each, cut off the top one after the other, so that their sum is the value).
// Products of two bf16 are exact in fp32, the sums are in fp32.
//
// Both operands have the summed dimension as their slow one, so they are staged in LDS as they lie
// in memory, the codes restored on the way (once for a tile's 256 columns of dY), and read across
// their rows by LDS's transposing reads.  Measured: 8192 x 11008 x 4096 bf16 in 0.67 to 0.77 ms (960 to
// 1100 TFLOP/s; added to what is there 0.73 ms; a library product of bf16 operands in this layout
// reaches 950 on that shape), 4096 x 4096 x 4096 in 0.13 to 0.15 ms; fp16 in 1.23 and 0.22 ms, fp32 in
// 1.95 and 0.33 (two and three products a value: 600 and 620, 380 and 420 TFLOP/s).  The matrix cores are busy
// for 56 % of the cycles; LDS (no bank conflicts) for 35 %; the clock is held at 1.8 to 1.9 GHz by the
// card's power, so that the energy of a step sets its time more than its schedule does: tiles with more
// loads a product (256 x 128) took 11 % longer, without any restoring a step took 7 % less.
#include <type_traits>

#include "gc_act_internal.h"

#include "gc_act.h"

namespace gc {
namespace {

typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s4 lds_s4;

// The parts of a value of the type: bf16 1, fp16 2, fp32 3.
template <int DT>
constexpr int parts() {
  return DT == kBF16 ? 1 : DT == kF16 ? 2 : 3;
}

// A workgroup's tile of dW, kTN x kTK, shared by kWN x kWK waves; BM rows of dY and Z a step.
template <int TN, int TK, int WN, int WK, int BM>
struct Tile {
  static constexpr int kTN = TN, kTK = TK, kWN = WN, kWK = WK, kBM = BM;
  static constexpr int kThreads = 64 * WN * WK;
  static constexpr int kFN = TN / WN / 32, kFK = TK / WK / 32;   // 32x32 products of a wave
  // 64 bytes past a row: the four rows of a transposing read start in different quarters of the banks
  static constexpr int kPitchN = TN + 32, kPitchK = TK + 32;
  static constexpr int kSlices = BM / 16;   // rows of one matrix instruction
  // Staging: an item is one octet a thread, kRowsN rows of a step's dY or kRowsK rows of its Z.
  static constexpr int kRowsN = kThreads / (TN / 8), kRowsK = kThreads / (TK / 8);
  static constexpr int kItemsN = BM / kRowsN, kItemsK = BM / kRowsK;
  static_assert(BM % kRowsN == 0 && BM % kRowsK == 0, "whole items");
};

__device__ __forceinline__ uint32_t pack_high(float a, float b) {   // their upper halves
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
}

// One 32x32x16 operand of a wave: 8 rows of the slice for each lane's column, read across the
// rows of LDS.
__device__ __forceinline__ b8 fragment(const short* p, int pitch) {
  const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)p);
  const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(p + 4 * pitch));
  return __builtin_bit_cast(b8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The bf16 parts of 8 values, part q at y + q * plane.
template <int DT>
__device__ __forceinline__ void store_parts(short* y, int plane, const Raw<DT>& r) {
  if constexpr (DT == kBF16) {
    *reinterpret_cast<u4*>(y) = r.w[0];
  } else {
    float v[8];
    to_float8<DT>(r, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // a NaN whose upper half alone would read as Inf
      if (DT == kF32 && v[j] != v[j]) v[j] = __uint_as_float(0x7FC00000u);
    }
#pragma unroll
    for (int q = 0; q < parts<DT>(); ++q) {
      u4 w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_high(v[2 * j], v[2 * j + 1]);
      *reinterpret_cast<u4*>(y + q * plane) = w;
      if (q + 1 < parts<DT>())
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // what is left under the 8 bits just taken; nothing is left of Inf (Inf - Inf) and NaN,
          // and what is left of a finite value is finite
          v[j] = v[j] - __uint_as_float(__float_as_uint(v[j]) & 0xFFFF0000u);
          if (q == 0 && v[j] != v[j]) v[j] = 0.0f;
        }
    }
  }
}

// Tile of this workgroup.  Workgroups go to the 8 XCDs in turn: each XCD gets a contiguous range of
// the order below, in which kBand tiles along n share their part of Z, and its L2 holds what they
// share.  The 32 large tiles that run on an XCD read least where they are 4 along n (2 or 4 bytes an
// element) by 8 along k (1 byte): 1096 us for 8192 x 8192 x 8192 bf16, with 8 along n 1108, with 2
// 1114.
constexpr int kBand = 4;
__device__ __forceinline__ void tile_of(int tiles_n, int tiles_k, int* tn, int* tk) {
  const int total = tiles_n * tiles_k, id = blockIdx.x;
  const int q = total / 8, r = total % 8, xcd = id % 8, i = id / 8;
  const int t = xcd < r ? xcd * (q + 1) + i : r * (q + 1) + (xcd - r) * q + i;
  const int band = t / (kBand * tiles_k), high = min(kBand, tiles_n - kBand * band);
  const int in = t - band * kBand * tiles_k;
  *tn = kBand * band + in % high;
  *tk = in / high;
}

template <int DT, typename C>
__global__ __launch_bounds__(C::kThreads, 2) void k_wgrad(WgradArgs a, int splits) {
  typedef typename Elt<DT>::T T;
  constexpr int NS = parts<DT>(), kPieces = NS * C::kSlices;
  constexpr int NY = C::kItemsN, NZ = C::kItemsK;
  constexpr int kPlane = C::kBM * C::kPitchN, kStage = NS * kPlane + C::kBM * C::kPitchK;
  __shared__ __align__(16) short s_mem[2 * kStage];   // two stages: the parts of dY, then Z
  int tn, tk;
  tile_of((a.n_out + C::kTN - 1) / C::kTN, (a.cols + C::kTK - 1) / C::kTK, &tn, &tk);
  const int n0 = tn * C::kTN, k0 = tk * C::kTK;
  const int wave = wave_id(), lane = lane_id();
  const int wn = (wave / C::kWK) * (C::kTN / C::kWN), wk = (wave % C::kWK) * (C::kTK / C::kWK);
  const int groups = (a.cols + kActGroup - 1) / kActGroup, octets = groups * (kActGroup / 8);
  const int64_t ld = a.dy.ld;
  const int64_t steps = (a.rows + C::kBM - 1) / C::kBM;
  const int64_t first = steps * blockIdx.y / splits, last = steps * (blockIdx.y + 1) / splits;
  // Whole steps: their rows are all there and their 16-byte loads stay inside dY whatever the column,
  // as a load that starts in a row before the last one ends before the matrix does.  The lanes of
  // columns past n_out or the pitch read some other column there; what they add up is not stored.
  const bool wide = n0 + C::kTN <= a.n_out;
  const int64_t whole = ld < 8 || ld > (1 << 24) || octets > (1 << 22) ? 0
                        : (wide ? a.rows : a.rows - 1) / C::kBM;

  // This thread stages row r, octet c of every item.
  const int ry = threadIdx.x / (C::kTN / 8), cy = threadIdx.x % (C::kTN / 8);
  const int rz = threadIdx.x / (C::kTK / 8), cz = threadIdx.x % (C::kTK / 8);
  const int my_octet = min(k0 / 8 + cz, octets - 1);
  const uint32_t y_off = (uint32_t)(ry * ld + min(n0 + 8 * cy, a.n_out - 1)) * (uint32_t)sizeof(T);
  const uint32_t z_off = (uint32_t)(rz * octets + my_octet) * 8u;
  const uint32_t e_off = (uint32_t)(rz * groups + (my_octet >> 2));
  Raw<DT> y[NY];
  u2 z[NZ];
  uint32_t e[NZ];
  // Loads item p of a step: dY's first, then Z's.  The rows' base is the same in all lanes.
  auto load_whole = [&](int64_t step, int p) {
    if (p < NY) {
      const int64_t m = step * C::kBM + C::kRowsN * p;
      y[p] = load_raw<DT>(static_cast<const char*>(a.dy.p) + m * ld * (int64_t)sizeof(T) + y_off);
    } else {
      const int64_t m = step * C::kBM + C::kRowsK * (p - NY);
      z[p - NY] = *reinterpret_cast<const u2*>(reinterpret_cast<const char*>(a.codes) +
                                               m * octets * 8 + z_off);
      e[p - NY] = (a.exps + m * groups)[e_off];
    }
  };
  // The same of any step, without a branch: the last row in place of the rows behind it, and the row's
  // last 8 columns where an octet ends behind them; mend() puts that right.
  auto load_edge = [&](int64_t step, int p) {
    if (p < NY) {
      const int64_t m = min(step * C::kBM + C::kRowsN * p + ry, a.rows - 1);
      const T* row = static_cast<const T*>(a.dy.p) + m * ld;
      if (a.n_out >= 8)
        y[p] = load_raw<DT>(row + min(n0 + 8 * cy, a.n_out - 8));
      else
        y[p] = load_raw<DT>(row, n0 + 8 * cy, a.n_out);
    } else {
      const int64_t m = min(step * C::kBM + C::kRowsK * (p - NY) + rz, a.rows - 1);
      z[p - NY] = reinterpret_cast<const u2*>(a.codes)[m * octets + my_octet];
      e[p - NY] = a.exps[m * groups + (my_octet >> 2)];
    }
  };
  // Moves such an octet into place, and clears the rows behind the last one.
  auto mend = [&](int64_t step, int p) {
    if (p < NY) {
      const int over = a.n_out >= 8 ? max(n0 + 8 * cy - (a.n_out - 8), 0) : 0;
      uint32_t d[4 * Raw<DT>::kWords];
      __builtin_memcpy(d, &y[p], sizeof d);
      shift_down<4 * Raw<DT>::kWords>(d, (uint32_t)min(over, 7) * (sizeof(T) / 2));
      __builtin_memcpy(&y[p], d, sizeof d);
      if (step * C::kBM + C::kRowsN * p + ry >= a.rows) y[p] = Raw<DT>{};
    } else if (step * C::kBM + C::kRowsK * (p - NY) + rz >= a.rows) {
      z[p - NY] = u2{0, 0};
      e[p - NY] = 0;
    }
  };
  auto store = [&](short* stage, int p) {
    if (p < NY) {
      store_parts<DT>(stage + (C::kRowsN * p + ry) * C::kPitchN + 8 * cy, kPlane, y[p]);
      return;
    }
    p -= NY;
    float v[8];
    decode8(z[p], exponent_scale(e[p]), v);
    u4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_high(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<u4*>(stage + NS * kPlane + (C::kRowsK * p + rz) * C::kPitchK + 8 * cz) = w;
  };
  // The lane's place in a transposing read.
  const int fr = 8 * (lane >> 5) + ((lane & 15) >> 2), fc = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const int fz_at = NS * kPlane + fr * C::kPitchK + wk + fc, fy_at = fr * C::kPitchN + wn + fc;
  auto read_z = [&](const short* stage, int p, b8 (&f)[C::kFK]) {
#pragma unroll
    for (int j = 0; j < C::kFK; ++j)
      f[j] = fragment(stage + fz_at + 16 * p * C::kPitchK + 32 * j, C::kPitchK);
  };
  auto read_y = [&](const short* stage, int p, int q, b8 (&f)[C::kFN]) {
#pragma unroll
    for (int i = 0; i < C::kFN; ++i)
      f[i] = fragment(stage + fy_at + q * kPlane + 16 * p * C::kPitchN + 32 * i, C::kPitchN);
  };

  // The straight loop below stores the steps first + 1 to lim - 2 and loads up to lim - 1, all whole.
  const int64_t lim = whole < last ? whole : last;
  auto loaded_whole = [&](int64_t step) { return first + 2 < lim && step > first && step < lim; };

  f16v acc[C::kFN][C::kFK] = {};
  b8 fz[C::kFK], fy[C::kFN];
  short *cur = s_mem, *nxt = s_mem + kStage;
  // One step: its slices are multiplied, each piece (a slice, a part of dY) while the operands of
  // the next are read.  The next step's rows, loaded a step ago, go to the other stage during all
  // pieces but the last, and the rows of the step after it are loaded.  Before the last piece all
  // waves meet: the other stage is complete then, and nobody reads this one any more.
  auto step = [&](int64_t s, auto all) {
    const bool more1 = all || s + 1 < last, more2 = all || s + 2 < last;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = i / NS, q = i % NS;
      b8 ny[C::kFN], nz[C::kFK];
      if (i + 1 < kPieces) {
        if (q + 1 == NS) read_z(cur, p + 1, nz);
        read_y(cur, (i + 1) / NS, (i + 1) % NS, ny);
      } else {
        __syncthreads();
        if (more1) {
          read_z(nxt, 0, nz);
          read_y(nxt, 0, 0, ny);
        }
      }
#pragma unroll
      for (int t = 0; t < NY + NZ; ++t)
        if (t * (kPieces - 1) / (NY + NZ) == i) {
          if (!all && more1 && !loaded_whole(s + 1)) mend(s + 1, t);
          if (more1) store(nxt, t);
          if (all)
            load_whole(s + 2, t);
          else if (more2)
            load_edge(s + 2, t);
        }
#pragma unroll
      for (int u = 0; u < C::kFN; ++u)
#pragma unroll
        for (int j = 0; j < C::kFK; ++j)
          acc[u][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fy[u], fz[j], acc[u][j], 0, 0, 0);
      // each matrix instruction followed by a share of the rest, which runs beside it
#pragma unroll
      for (int g = 0; g < C::kFN * C::kFK; ++g) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // matrix
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);   // vector
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // loads
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);   // LDS writes
      }
#pragma unroll
      for (int u = 0; u < C::kFN; ++u) fy[u] = ny[u];
      if (q + 1 == NS)
#pragma unroll
        for (int j = 0; j < C::kFK; ++j) fz[j] = nz[j];
    }
    short* t = cur;
    cur = nxt;
    nxt = t;
  };
  if (first < last) {
#pragma unroll
    for (int p = 0; p < NY + NZ; ++p) load_edge(first, p);
#pragma unroll
    for (int p = 0; p < NY + NZ; ++p) {
      mend(first, p);
      store(cur, p);
    }
    if (loaded_whole(first + 1)) {
#pragma unroll
      for (int p = 0; p < NY + NZ; ++p) load_whole(first + 1, p);
    } else if (first + 1 < last) {
#pragma unroll
      for (int p = 0; p < NY + NZ; ++p) load_edge(first + 1, p);
    }
    __syncthreads();
    read_z(cur, 0, fz);
    read_y(cur, 0, 0, fy);
    int64_t s = first;
    // nothing in flight: the loop's own waits then count its own loads only, in their order
    __builtin_amdgcn_s_waitcnt(0x0F70);
    for (; s + 2 < lim; ++s) step(s, std::true_type());
    for (; s < last; ++s) step(s, std::false_type());
  }

  // Register r of a 32x32 product holds its row 8 * (r / 4) + 4 * (lane / 32) + r % 4, column
  // lane % 32.  Only an accumulating call loads: its values one product ahead of the stores, which a
  // wait for a load would otherwise wait for too.
  float* out = splits > 1 ? a.ws + (int64_t)blockIdx.y * a.n_out * a.cols : a.dw;
  const bool add = splits == 1 && a.accumulate, scaled = splits == 1 && a.col_scale;
  const bool inside = wide && k0 + C::kTK <= a.cols;
  const int n_wave = n0 + wn + 4 * (lane >> 5), k_wave = k0 + wk + (lane & 31);
  float* lane_out = out + (int64_t)n_wave * a.cols + k_wave;
  constexpr int kProducts = C::kFN * C::kFK;
  auto row = [](int t, int r) { return 32 * (t / C::kFK) + 8 * (r >> 2) + (r & 3); };
  auto at = [&](int t, int r) { return lane_out + (int64_t)row(t, r) * a.cols + 32 * (t % C::kFK); };
  auto within = [&](int t, int r) {
    return n_wave + row(t, r) < a.n_out && k_wave + 32 * (t % C::kFK) < a.cols;
  };
  if (scaled)
#pragma unroll
    for (int j = 0; j < C::kFK; ++j) {
      const float sc = load_any(a.col_scale, a.scale_dtype, min(k_wave + 32 * j, a.cols - 1));
#pragma unroll
      for (int i = 0; i < C::kFN; ++i) acc[i][j] *= sc;
    }
  if (add) {
    float old[2][16] = {};
#pragma unroll
    for (int t = 0; t <= kProducts; ++t) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (t < kProducts && within(t, r)) old[t & 1][r] = *at(t, r);
      if (t == 0) continue;
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (within(t - 1, r))
          *at(t - 1, r) = old[(t - 1) & 1][r] + acc[(t - 1) / C::kFK][(t - 1) % C::kFK][r];
    }
  } else if (inside) {
#pragma unroll
    for (int t = 0; t < kProducts; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) *at(t, r) = acc[t / C::kFK][t % C::kFK][r];
  } else {
#pragma unroll
    for (int t = 0; t < kProducts; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (within(t, r)) *at(t, r) = acc[t / C::kFK][t % C::kFK][r];
  }
}

// The parts of the row sum joined in order, scaled and stored: kV neighbouring elements of a row a
// thread.
template <int kV>
__global__ __launch_bounds__(256) void k_wgrad_join(WgradArgs a, int splits) {
  const uint32_t total = (uint32_t)a.n_out * (uint32_t)a.cols;   // below 2^31
  const uint32_t i = (blockIdx.x * 256u + threadIdx.x) * kV;
  if (i >= total) return;
  float v[kV] = {}, w[kV];
  for (int s = 0; s < splits; s += 8) {   // 8 parts in flight
    float u[8][kV] = {};
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (s + t < splits) __builtin_memcpy(u[t], a.ws + (int64_t)(s + t) * total + i, sizeof w);
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int j = 0; j < kV; ++j) v[j] += u[t][j];
  }
  if (a.col_scale)
#pragma unroll
    for (int j = 0; j < kV; ++j)
      v[j] *= load_any(a.col_scale, a.scale_dtype, i % (uint32_t)a.cols + j);
  if (a.accumulate) {
    __builtin_memcpy(w, a.dw + i, sizeof w);
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] += w[j];
  }
  __builtin_memcpy(a.dw + i, v, sizeof v);
}

// Values of several parts take half the rows a step, so that two stages fit the 160 KB of LDS.
template <int DT>
using Large = Tile<256, 256, 2, 4, DT == kBF16 ? 64 : 32>;
template <int DT>
using Small = Tile<128, 128, 2, 2, DT == kBF16 ? 64 : 32>;
template <int DT>
using Tiny = Tile<64, 64, 2, 2, DT == kBF16 ? 64 : 32>;

enum TileKind { kLarge, kSmall, kTiny };
constexpr int kTileSize[3] = {256, 128, 64};

struct Shape {
  TileKind tile;
  int splits;
};

int64_t tiles_of(int32_t n_out, int32_t cols, int t) {
  return (((int64_t)n_out + t - 1) / t) * (((int64_t)cols + t - 1) / t);
}

// A large tile needs the fewest loads and restores the fewest codes a product, but leaves CUs idle
// where the matrix is small; a sum over many rows can be split over CUs, at the price of writing and
// joining its parts.  The tile and the split with the least estimated time are taken.  A step of a
// tile takes, with 1, 2 and 3 workgroups on its CU, in tenths of a microsecond (measured; a CU holds
// 1 large, 2 small or 3 tiny ones):
//              large   small      tiny
//   bf16        17     9 14     5  8 11    (64 rows a step)
//   fp16        14     9 11     5  6  8    (32 rows, 2 parts)
//   fp32        25    12 17     8 10 13    (32 rows, 3 parts)
// A call costs 4 us besides, a join 4 us, 0.1 us a part and its bytes (written and read) at 6 TB/s, or
// at 4 where the parts pass 100 MB.  Three shapes were measured against every other choice: 512 rows
// of 1024 x 1024 bf16 take tiny tiles, 7.9 us (small 11.5, small in 4 parts 19.3); 8192 rows of 2048 x
// 2048 large ones in 4 parts, 84 us (small 115, tiny 152); 4096 rows of 512 x 512 tiny ones in 8 parts,
// 15.5 us (whole 33.6).  Estimates against measured times: 2048 rows of 2048 x 2048 bf16 33 and 33 us,
// 8192 of 1024 x 1024 43 and 40, 1531 of 1025 x 1000 fp32 30 and 28, 4096 of 4096 x 4096 fp32 324 and
// 326; large tiles on every CU for long, whose clock the card's power lowers, take more than estimated
// in the 16-bit types: 4096 of 4096 x 4096 bf16 113 and 132, fp16 183 and 220, 8192 of 11008 x 4096
// 657 and 700, 1079 and 1230.
Shape shape_of(int64_t rows, int32_t n_out, int32_t cols, int dtype) {
  constexpr int kPerCU[3] = {1, 2, 3};
  constexpr double kStepTime[3][3][3] = {   // by type (kF32, kBF16, kF16), tile, workgroups on the CU
      {{2.5}, {1.2, 1.7}, {0.8, 1.0, 1.3}},
      {{1.7}, {0.9, 1.4}, {0.5, 0.8, 1.1}},
      {{1.4}, {0.9, 1.1}, {0.5, 0.6, 0.8}}};
  constexpr int64_t kCUs = 256;
  const int64_t bm = dtype == kBF16 ? 64 : 32, steps = (rows + bm - 1) / bm;
  Shape best = {kTiny, 1};
  double least = 1e300;
  for (int t = 0; t < 3; ++t) {
    const int64_t tiles = tiles_of(n_out, cols, kTileSize[t]);
    for (int s = 1; s <= 64 && (s == 1 || s <= steps); s += s < 4 ? 1 : s / 2) {
      const int64_t groups = tiles * s, full = groups / (kCUs * kPerCU[t]);
      const int64_t rest = groups - full * kCUs * kPerCU[t];
      const double* step = kStepTime[dtype][t];
      double us = full * step[kPerCU[t] - 1];
      if (rest) us += step[(rest + kCUs - 1) / kCUs - 1];
      us = us * (double)((steps + s - 1) / s) + 4.0;
      const double bytes = 4.0 * s * (double)n_out * (double)cols;
      if (s > 1) us += 4.0 + 0.1 * s + 2.0 * bytes / (bytes > 100e6 ? 4e6 : 6e6);
      if (us < least) {
        least = us;
        best = {(TileKind)t, s};
      }
    }
  }
  return best;
}

template <int DT, typename C>
hipError_t wgrad(const WgradArgs& a, int splits, hipStream_t st) {
  const dim3 grid((unsigned)tiles_of(a.n_out, a.cols, C::kTN), splits);
  k_wgrad<DT, C><<<grid, C::kThreads, 0, st>>>(a, splits);
  return hipGetLastError();
}

template <int DT>
hipError_t wgrad(const WgradArgs& a, const Shape& s, hipStream_t st) {
  return s.tile == kLarge   ? wgrad<DT, Large<DT>>(a, s.splits, st)
         : s.tile == kSmall ? wgrad<DT, Small<DT>>(a, s.splits, st)
                            : wgrad<DT, Tiny<DT>>(a, s.splits, st);
}

}  // namespace

int wgrad_splits(int64_t rows, int32_t n_out, int32_t cols, int dtype) {
  return shape_of(rows, n_out, cols, dtype).splits;
}

hipError_t launch_wgrad(const WgradArgs& a, hipStream_t st) {
  if (a.n_out == 0 || a.cols == 0 || (a.rows == 0 && a.accumulate)) return hipSuccess;
  const Shape s = shape_of(a.rows, a.n_out, a.cols, a.dtype);
  if (hipError_t e = a.dtype == kF32    ? wgrad<kF32>(a, s, st)
                     : a.dtype == kBF16 ? wgrad<kBF16>(a, s, st)
                                        : wgrad<kF16>(a, s, st))
    return e;
  if (s.splits > 1) {
    const int64_t total = (int64_t)a.n_out * a.cols;
    if (a.cols % 4 == 0)
      k_wgrad_join<4><<<blocks_for(total, 1024), 256, 0, st>>>(a, s.splits);
    else
      k_wgrad_join<1><<<blocks_for(total, 256), 256, 0, st>>>(a, s.splits);
  }
  return hipGetLastError();
}

}  // namespace gc
