// gc_gated.hip -- the gated feed-forward block and its backward pass.
//
//   forward    G = X Wg^T, U = X Wu^T, h = act(G) * U, in one kernel: a workgroup forms the same
//              columns of G and of U, so that their product is taken from its registers.
//   backward   dG = dh * U * act'(G), dU = dh * act(G) of the kept rows of G and U, a stream of
//              five matrices; then dX = dG Wg + dU Wu, one product whose sum runs over the columns of
//              dG and then over those of dU.
//
// The products run on the matrix cores (32x32x16 of 16-bit values; fp32 as three bf16 parts, six products a
// pair) with sums in fp32.  Their first operand is the weight, so that a lane ends up with 16 neighbouring
// columns of one row of the result (the 32 columns of a product are handed out in that order).  Both operands
// come through registers into two stages of LDS, at any alignment; the backward pass's weight, whose rows are
// the summed dimension, is read across its rows by LDS's transposing reads.
//
// Measured, 8192 rows, 4096 x 11008 bf16: forward with gate and up kept 1.19 to 1.24 ms (1190 to 1240 TFLOP/s),
// backward 1.28 to 1.33 ms in all (the stream 0.155, 5.8 TB/s; the product 1.15).  Library products of the
// same sizes, without the activation and its matrices, take 1.11 to 1.22 and 1.06 to 1.09 ms.  The matrix cores
// are busy for 70 and 77 % of the cycles, LDS (hardly a bank conflict) for 47 and 48 %, at a clock of 1.7 GHz;
// the forward pass has its results (541 MB) and activations besides, for which its tiles stand still.
// Loading into LDS directly, 16-byte aligned rows only, was tried first: forward 1.32 ms, backward 1.50.
#include <type_traits>

#include "gc_act_internal.h"

#include "gc_act.h"

namespace gc {
namespace {

typedef short s4 __attribute__((ext_vector_type(4)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s4 lds_s4;

// ------------------------------------------------------------------ the activations
// exp(-(x + low)) for 0 <= x <= 200 and a small correction, within 3 * 2^-24 of it: 2^t of the rounded
// product with 1 / ln 2, and what the rounding left in first order.  (Below 2^-64 the power is taken 2^64
// higher, as the instruction returns no denormals.)
__device__ __forceinline__ float exp_neg(float x, float low = 0.0f) {
  constexpr float kInv = 1.44269502f, kInvLow = 1.92596303e-8f, kLn2 = 0.69314718f;
  const float t = -x * kInv, rest = fmaf(-low, kInv, fmaf(-x, kInvLow, fmaf(-x, kInv, -t)));
  const bool small = t < -64.0f;
  const float e = __builtin_amdgcn_exp2f(small ? t + 64.0f : t);
  return fmaf(e * kLn2, rest, e) * (small ? 0x1p-64f : 1.0f);
}

// act(g) and its derivative, each within 16 * 2^-24 of its terms, gelu_tanh within (16 + 5 |v|) * 2^-24: its
// v is rounded five times before the exponential, which makes an error of |v| of them (as in any fp32 form that
// does not carry v's low part along; 94 * 2^-24 at g = -6.7).  p is the factor that both start from
// (the logistic or the normal distribution function) and q what is left to 1, each formed without
// cancellation.  Arguments are limited to where p is 0 or 1 in fp32 anyway; NaN comes back through g.
// These take about 25 instructions where the library's exponential, error function and division took 65
// and more, which were 14 us of each 256 x 256 tile's time.
template <int ACT>
__device__ __forceinline__ void activate(float g, float* act, float* slope) {
  if (ACT == kGelu) {
    // Phi(-a) = exp(-a^2 / 2) R(a); R, a ninth-degree polynomial in 1 / (1 + a / 4) fitted over 0 <= a
    // <= 15, with these coefficients to 9.7e-8 of its value (at a = 0; 7.7e-8 from a = 1 on)
    const float a = fminf(fabsf(g), 20.0f), half = 0.5f * a, x = half * a;
    const float e = exp_neg(x, fmaf(half, a, -x)), t = __builtin_amdgcn_rcpf(fmaf(0.25f, a, 1.0f));
    float r = 0.024650581181049347f;
    r = fmaf(r, t, -0.14754432439804077f);
    r = fmaf(r, t, 0.28512391448020935f);
    r = fmaf(r, t, -0.19303946197032928f);
    r = fmaf(r, t, 0.19281961023807526f);
    r = fmaf(r, t, 0.03680535778403282f);
    r = fmaf(r, t, 0.10273300111293793f);
    r = fmaf(r, t, 0.0986626073718071f);
    r = fmaf(r, t, 0.09978866577148438f);
    const float q = r * t * e, p = g >= 0.0f ? 1.0f - q : q;
    *act = g * p;
    *slope = fmaf(g, e * 0.39894228f, p);
    return;
  }
  constexpr float k = 1.59576912f;   // 2 sqrt(2 / pi)
  const float c = fminf(fmaxf(g, -30.0f), 30.0f), cubic = fmaf(0.044715f * c * c, c, c);
  const float v = ACT == kSilu ? g : k * cubic;
  const float e = exp_neg(fminf(fabsf(v), 200.0f));
  const float r = __builtin_amdgcn_rcpf(1.0f + e), s = e * r;
  const float p = v >= 0.0f ? r : s, q = v >= 0.0f ? s : r;
  *act = g * p;
  *slope = fmaf(g * p * q, ACT == kSilu ? 1.0f : k * fmaf(0.134145f * c, c, 1.0f), p);
}

// v[r] = act(v[r]) * u[r].  The forward pass stands still for this, so that silu takes a short way where
// |g| <= 16: there exp(-g) needs no correction (its argument's rounding is at most 16 * 2^-24 of it; act is
// within 20 * 2^-24) and stays far from the ends of fp32's range.  Which way is taken goes by the value alone:
// a wave in which some |g| > 16 goes both ways, and each value takes its own.  (8192 rows through 11008 x 4096
// bf16: 1220 us where no wave does, 1264 where all do.)
template <int ACT, int N>
__device__ __forceinline__ void gate(float (&v)[N], const float (&u)[N]) {
  auto near = [](float g) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269502f));
  };
  if (ACT == kSilu) {
    float most = 0.0f;
#pragma unroll
    for (int r = 0; r < N; ++r) most = fmaxf(most, fabsf(v[r]));   // of numbers: NaN stays NaN either way
    if (__ballot(most > 16.0f) == 0) {
#pragma unroll
      for (int r = 0; r < N; ++r) v[r] = near(v[r]) * u[r];
      return;
    }
  }
#pragma unroll
  for (int r = 0; r < N; ++r) {
    float act, slope;
    activate<ACT>(v[r], &act, &slope);
    if (ACT == kSilu) act = fabsf(v[r]) > 16.0f ? act : near(v[r]);
    v[r] = act * u[r];
  }
}

template <int DT, int ACT>
__global__ __launch_bounds__(256) void k_gated_slope(GatedGradArgs a) {
  typedef typename Elt<DT>::T T;
  const int64_t octets = (a.n + 7) / 8, total = a.rows * octets;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const int64_t row = i / octets;
  const int col = (int)(i - row * octets) * 8;
  float dh[8], g[8], u[8], dg[8], du[8];
  load8<DT>(static_cast<const T*>(a.dh.p) + row * a.dh.ld, col, a.n, dh);
  load8<DT>(static_cast<const T*>(a.gate.p) + row * a.gate.ld, col, a.n, g);
  load8<DT>(static_cast<const T*>(a.up.p) + row * a.up.ld, col, a.n, u);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float act, slope;
    activate<ACT>(g[j], &act, &slope);
    dg[j] = dh[j] * u[j] * slope;
    du[j] = dh[j] * act;
  }
  store8<DT>(static_cast<T*>(a.dgate.p) + row * a.dgate.ld, col, a.n, dg);
  store8<DT>(static_cast<T*>(a.dup.p) + row * a.dup.ld, col, a.n, du);
}

// ------------------------------------------------------------------ the products
// What a product of either direction reads and writes: out = sum over the segments s of a[s] b[s].
struct Product {
  int64_t rows;
  int32_t n, depth;      // columns of the result (of one projection), summed columns of a segment
  Mat a[2], b[2];        // forward: x, and the two weights (n x depth); backward: dgate and dup, and
                         // the two weights (depth x n)
  Mat out[3];            // forward: h, gate, up (the last two may be null); backward: dx
  int32_t act;
  int32_t splits;        // parts of the sum; with more than one, part i of result j (forward: gate, up;
  float* ws;             // backward: dx) goes to ws[i][j][rows][n]
};

constexpr int kChunk = 16, kRowBytes = 128, kRowChunks = kRowBytes / kChunk;

// A workgroup's tile, BM rows by BN columns (forward: BN / 2 of each projection), shared by WM x WN
// waves.  A step sums 128 bytes of a row.  PARTS (1, or 3 of fp32): the bf16 values whose sum an element is
// in LDS.  AHEAD: steps from a piece's load to its way into LDS.
template <int DT, bool BACK, int BM, int BN, int WM, int WN, int PARTS = 1, int AHEAD = 1>
struct Tile {
  typedef typename Elt<DT>::T T;
  typedef Tile<DT, BACK, BM, BN, WM, WN> Whole;   // without parts
  static constexpr int kParts = PARTS, kAhead = AHEAD;
  static_assert(AHEAD == 1 || AHEAD == 2, "sets of pieces on their way");
  static constexpr int kBM = BM, kBN = BN, kWM = WM, kWN = WN;
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr int kFM = BM / WM / 32, kFN = BN / WN / 32;
  static constexpr int kElts = kChunk / (int)sizeof(T), kBK = kRowChunks * kElts;
  static constexpr int kCols = BACK ? BN : BN / 2;      // of the result
  static constexpr int kPiecesB = BACK ? BN / kElts : kRowChunks;   // of a row of the second operand
  // In LDS: rows of the summed dimension, or of BN columns (one part after the other).
  static constexpr int kPitch = PARTS == 1 ? kRowBytes : PARTS * kRowBytes / 2;
  static constexpr int kPitchB = !BACK ? kPitch : PARTS == 1 ? kPiecesB * kChunk : BN * 2;
  static constexpr int kBytesA = BM * kPitch, kBytesB = BACK ? PARTS * kBK * kPitchB : BN * kPitchB;
  static constexpr int kStage = kBytesA + kBytesB;
  static constexpr int kSlices = PARTS == 1 ? kRowChunks / 2 : kBK / 16;   // of a step, each one product deep
  // Loading: an item is one piece a thread, kRowsA rows of a step's first or kRowsB of its second operand.
  static constexpr int kRowsA = kThreads / kRowChunks, kRowsB = kThreads / kPiecesB;
  static constexpr int kItemsA = BM * kRowChunks / kThreads;
  static constexpr int kItemsB = (BACK ? kBK : BN) * kPiecesB / kThreads;
  static_assert(BN >= 128 && (BACK || (kFN % 2 == 0 && kRowsB % 16 == 0 && kRowsB <= 64)), "layouts");
};

// Where 16-byte piece c of row r of a tile lies: the pieces of 16 neighbouring rows that a read takes
// at once fall into different banks.  With parts, piece c (of 4) of part q.
template <int PARTS>
__device__ __forceinline__ int piece_at(int r, int c, int q = 0) {
  if (PARTS == 1) return r * kRowBytes + ((c ^ ((r >> 1) & (kRowChunks - 1))) * kChunk);
  return (r * PARTS + q) * (kRowBytes / 2) + ((c ^ ((r >> 2) & 3)) * kChunk);
}

// Where the 64-byte block b of row r lies in a row of the backward pass's second operand: the four rows
// of a transposing read (whole fp32: the two halves of a wave, four rows apart) in different banks.
template <bool WIDE>
__device__ __forceinline__ int block_at(int r, int b) {
  return WIDE ? b ^ ((r >> 1) & 2) : b ^ (r & 3);
}

// The column (of 32) that row i of a product's first operand stands for: a lane's 16 registers hold
// rows 8 * (r / 4) + 4 * (lane / 32) + r % 4, and are to be columns 16 * (lane / 32) + r.
__device__ __forceinline__ int column_of(int i) {
  return 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3);
}

// 16 bytes of the row at p from element k on, zeros from `end` on.  Where the row ends inside them its last
// 16 bytes are loaded and moved into place.
template <typename T>
__device__ __forceinline__ u4 load_piece(const T* p, int k, int end) {
  constexpr int E = 16 / sizeof(T);
  uint32_t d[4] = {};
  if (end >= E) {
    const int at = min(k, end - E), over = min(k - at, E - 1);
    __builtin_memcpy(d, p + at, sizeof d);
    shift_down<4>(d, (uint32_t)over * (sizeof(T) / 2));
  } else {   // a row of less than 16 bytes: from its end, each element under the last
#pragma unroll 1
    for (int j = end - 1; j >= k; --j) {
      uint32_t e = 0;
      __builtin_memcpy(&e, p + j, sizeof(T));
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const uint32_t below = i ? d[i - 1] : (sizeof(T) == 2 ? e << 16 : e);
        d[i] = sizeof(T) == 2 ? (d[i] << 16) | (below >> 16) : below;
      }
    }
  }
  return k < end ? u4{d[0], d[1], d[2], d[3]} : u4{};
}

// The three bf16 values whose sum each of 4 fp32 is, each the nearest to what the ones before it leave (8 bits
// of 24).  Inf and NaN, and what rounds to Inf, leave NaN among them.
__device__ __forceinline__ void parts_of(const u4& w, u2 (&part)[3]) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float a = __uint_as_float(w[2 * h]), b = __uint_as_float(w[2 * h + 1]);
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const uint32_t t = __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, bf2));
      part[q][h] = t;
      a -= __uint_as_float(t << 16);
      b -= __uint_as_float(t & 0xFFFF0000u);
    }
  }
}

// acc += a b for 16 bytes of the summed dimension a lane.
template <int DT>
__device__ __forceinline__ void multiply(const u4& w, const u4& x, f16v& acc) {
  if constexpr (DT == kBF16) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, w),
                                                  __builtin_bit_cast(b8, x), acc, 0, 0, 0);
  } else if constexpr (DT == kF16) {
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, w),
                                                 __builtin_bit_cast(h8, x), acc, 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(w[j]), __uint_as_float(x[j]), acc,
                                                 0, 0, 0);
  }
}

// Stores a block of 32 rows x 32 B columns, of which a lane holds 16 columns of one row (a row of 16 halves
// on two lanes, 32 apart).  Lanes that follow each other in memory are 32 apart in the wave, so that
// stores as they lie took four 16-byte requests for 64 bytes; the block goes through the wave's own part
// of LDS instead, and comes back with 4 and more neighbouring lanes a row.  INSIDE: all columns exist.
template <typename T, int B, bool INSIDE>
__device__ __forceinline__ void store_block(char* lds, T* p, int64_t ld, int64_t row0, int64_t rows,
                                            int col0, int n, const float (&v)[B][16]) {
  constexpr int E = kChunk / sizeof(T), P = 32 * B / E;   // pieces of a row
  static_assert(P <= 16, "a row within the banks");
  const int half = lane_id() >> 5, in = lane_id() & 31;
  // piece c of row r: pieces of neighbouring rows in different banks
  auto at = [&](int r, int c) { return (r * P + (c ^ ((r / (16 / P)) & (P - 1)))) * kChunk; };
  constexpr int DT = sizeof(T) == 4 ? kF32 : std::is_same<T, __bf16>::value ? kBF16 : kF16;
#pragma unroll
  for (int b = 0; b < B; ++b)
#pragma unroll
    for (int q = 0; q < 16 / E; ++q) {
      T t[E];
#pragma unroll
      for (int e = 0; e < E; ++e) t[e] = round_to<DT>(v[b][q * E + e]);
      u4 w;
      __builtin_memcpy(&w, t, sizeof w);
      *reinterpret_cast<u4*>(lds + at(in, (32 * b + 16 * half) / E + q)) = w;
    }
#pragma unroll
  for (int i = 0; i < P / 2; ++i) {
    const int k = i * 64 + lane_id(), r = k / P, c = k % P, col = col0 + c * E;
    const u4 w = *reinterpret_cast<const u4*>(lds + at(r, c));
    if (row0 + r >= rows) continue;
    T* q = p + (row0 + r) * ld + col;
    if (INSIDE || col + E <= n) {
      *reinterpret_cast<u4_at_any*>(q) = w;
    } else {
      T t[E];
      __builtin_memcpy(t, &w, sizeof w);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (col + e < n) q[e] = t[e];
    }
  }
}

// Stores a wave's products: the results, of the forward pass after the activation, or a part of the sums.
template <int DT, bool BACK, typename C, int ACT, bool INSIDE>
__device__ __forceinline__ void finish(const Product& g, const f16v (&acc)[C::kFM][C::kFN], char* lds,
                                       int64_t m0, int n0, int wm, int wn) {
  typedef typename Elt<DT>::T T;
  constexpr int B = BACK ? C::kFN : C::kFN / 2;
  const int col = n0 + (BACK ? wn : wn / 2);
#pragma unroll
  for (int i = 0; i < C::kFM; ++i) {
    const int64_t row = m0 + wm + 32 * i;
    auto put = [&](const Mat& m, const float (&v)[B][16]) {
      store_block<T, B, INSIDE>(lds, static_cast<T*>(m.p), m.ld, row, g.rows, col, g.n, v);
    };
    float v[B][16], u[B][16];
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        v[b][r] = acc[i][BACK ? b : 2 * b][r];
        u[b][r] = acc[i][BACK ? b : 2 * b + 1][r];
      }
    if (g.splits > 1) {
      float* part = g.ws + (int64_t)blockIdx.y * (BACK ? 1 : 2) * g.rows * g.n;
      store_block<float, B, INSIDE>(lds, part, g.n, row, g.rows, col, g.n, v);
      if (!BACK) store_block<float, B, INSIDE>(lds, part + g.rows * g.n, g.n, row, g.rows, col, g.n, u);
    } else if (BACK) {
      put(g.out[0], v);
    } else {
      if (g.out[1].p) put(g.out[1], v);
      if (g.out[2].p) put(g.out[2], u);
#pragma unroll
      for (int b = 0; b < B; ++b) gate<ACT, 16>(v[b], u[b]);
      put(g.out[0], v);
    }
  }
}

// Tile of this workgroup.  Workgroups go to the 8 XCDs in turn: each XCD gets a contiguous range of the
// order below, in which kBand tiles of rows share their part of the second operand, and its L2 holds what
// they share.
constexpr int kBand = 4;
__device__ __forceinline__ void tile_of(int tiles_m, int tiles_n, int* tm, int* tn) {
  const int total = tiles_m * tiles_n, id = blockIdx.x;
  const int q = total / 8, r = total % 8, xcd = id % 8, i = id / 8;
  const int t = xcd < r ? xcd * (q + 1) + i : r * (q + 1) + (xcd - r) * q + i;
  const int band = t / (kBand * tiles_n), high = min(kBand, tiles_m - kBand * band);
  const int in = t - band * kBand * tiles_n;
  *tm = kBand * band + in % high;
  *tn = in / high;
}

// A workgroup's tile from row m0 and column n0 on: `steps` steps of the sum from `first` on.
template <int DT, bool BACK, typename C>
__device__ __forceinline__ void sum_tile(const Product& g, char* s_mem, int64_t m0, int n0, int first,
                                         int steps, f16v (&acc)[C::kFM][C::kFN]) {
  typedef typename Elt<DT>::T T;
  constexpr int E = C::kElts, kItems = C::kItemsA + C::kItemsB, kSlices = C::kSlices;
  constexpr int P = C::kParts;
  constexpr bool kWide = DT == kF32 && P == 1;
  constexpr int64_t kSize = sizeof(T);
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
  const int wm = wave / C::kWN * (C::kFM * 32), wn = wave % C::kWN * (C::kFN * 32);
  const int steps_seg = (g.depth + C::kBK - 1) / C::kBK;

  // Thread t's piece of every item: A's row p * kRowsA + t / kRowChunks, piece piece_a(t) of the step; B's
  // likewise.  Whole elements lie in the order of the threads, so that the piece is the one which belongs
  // there; parts find their places when they are stored.
  auto piece_a = [](int t) {
    const int c = t % kRowChunks;
    return P > 1 ? c : c ^ ((t / kRowChunks >> 1) & 7);
  };
  auto piece_b = [](int t) {
    const int r = t / C::kPiecesB, c = t % C::kPiecesB;
    return P > 1 ? c : BACK ? block_at<kWide>(r, c >> 2) * 4 + (c & 3) : c ^ ((r >> 1) & 7);
  };
  // Where the rows of the items lie from the tile's first (rows past the last one read it; what they add
  // up is not stored).
  auto row_a = [&](int t, int p) {
    return min(m0 + p * C::kRowsA + t / kRowChunks, g.rows - 1) - m0;
  };
  auto row_b = [&](int t, int p) {
    const int r = p * C::kRowsB + t / C::kPiecesB;
    return (int64_t)(BACK ? r : min(n0 + (r >> 6) * 32 + column_of(r & 31), g.n - 1) - n0);
  };
  int seg = 0, left = 0;   // of the sum, from the next step on: the segment, what is left of it
  // Forward: a wave loads 8 rows at a time, of one of the weights: always the same, or by the item.
  auto weight = [&](int p) {
    return BACK ? seg : C::kRowsB == 64 ? (wave >> 2) & 1 : (p * C::kRowsB >> 5) & 1;
  };
  // The place of the next step to be loaded, the same in all lanes, and from it the byte offset of each
  // item's piece (columns past the last one are the tile's first).
  const char *pa, *pb[2];
  int64_t next_b;
  uint32_t off_a[C::kItemsA], off_b[C::kItemsB];
  auto start = [&](int which, int from) {
    seg = which;
    const Mat& a = g.a[seg];
    left = g.depth - from * C::kBK;
    pa = static_cast<const char*>(a.p) + m0 * a.ld * kSize + (int64_t)from * kRowBytes;
    next_b = BACK ? C::kBK * g.b[seg].ld * kSize : kRowBytes;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const Mat& b = g.b[BACK ? seg : C::kRowsB == 64 ? (wave >> 2) & 1 : i];
      pb[i] = static_cast<const char*>(b.p) + (BACK ? (int64_t)n0 : n0 * b.ld) * kSize + from * next_b;
    }
#pragma unroll
    for (int p = 0; p < C::kItemsA; ++p)
      off_a[p] = (uint32_t)(row_a(threadIdx.x, p) * a.ld * kSize) + piece_a(threadIdx.x) * kChunk;
#pragma unroll
    for (int p = 0; p < C::kItemsB; ++p)
      off_b[p] = (uint32_t)(row_b(threadIdx.x, p) * g.b[weight(p)].ld * kSize) +
                 (BACK && n0 + piece_b(threadIdx.x) * E >= g.n ? 0 : piece_b(threadIdx.x) * kChunk);
  };
  auto base_b = [&](int p) { return pb[BACK || C::kRowsB == 64 ? 0 : (p * C::kRowsB >> 5) & 1]; };
  auto advance = [&] {
    pa += kRowBytes;
    pb[0] += next_b;
    pb[1] += next_b;
    left -= C::kBK;
  };
  // Item p of the next step, A's first: of a step that is whole (all of its pieces are there), and of
  // any: what lies behind the sum's end is 0.
  auto load_whole = [&](int p) {
    const char* q = p < C::kItemsA ? pa + off_a[p] : base_b(p - C::kItemsA) + off_b[p - C::kItemsA];
    return u4(*reinterpret_cast<const u4_at_any*>(q));
  };
  auto load_edge = [&](int p) {
    // where this thread's pieces lie is found anew: kept through the steps before, it would take registers that
    // the large tiles do not have (70 values of a thread went to memory and back, 0.2 GB in a call of 8192 rows)
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    if (p < C::kItemsA) {
      const char* q = pa + row_a(t, p) * g.a[seg].ld * kSize;
      return load_piece(reinterpret_cast<const T*>(q), piece_a(t) * E, left);
    } else {
      const int b = p - C::kItemsA;
      const int64_t row = BACK ? min(row_b(t, b), (int64_t)left - 1) : row_b(t, b);
      const char* q = base_b(b) + row * g.b[weight(b)].ld * kSize;
      const u4 w = load_piece(reinterpret_cast<const T*>(q), piece_b(t) * E, BACK ? g.n - n0 : left);
      return BACK && row_b(t, b) >= left ? u4{} : w;
    }
  };
  auto store = [&](char* stage, int p, const u4& w) {
    if constexpr (P == 1) {
      *reinterpret_cast<u4*>(stage + (p * C::kThreads + threadIdx.x) * kChunk) = w;
    } else {
      const int ra = threadIdx.x / kRowChunks, sa = threadIdx.x % kRowChunks;
      const int rb = threadIdx.x / C::kPiecesB, sb = threadIdx.x % C::kPiecesB;
      u2 part[3];
      parts_of(w, part);
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const int b = p - C::kItemsA;
        char* to = stage;
        if (p < C::kItemsA)
          to += piece_at<P>(p * C::kRowsA + ra, sa >> 1, q) + (sa & 1) * 8;
        else if (!BACK)
          to += C::kBytesA + piece_at<P>(b * C::kRowsB + rb, sb >> 1, q) + (sb & 1) * 8;
        else
          to += C::kBytesA + (q * C::kBK + b * C::kRowsB + rb) * C::kPitchB +
                block_at<false>(rb, sb >> 3) * 64 + (sb & 7) * 8;
        *reinterpret_cast<u2*>(to) = part[q];
      }
    }
  };
  // Steps that can be loaded whole from here on: none where the offsets in a tile pass 32 bits.  (A piece
  // that starts inside a row of the backward pass's weight but ends behind it reads on into the next row,
  // which the last one has not.)
  auto whole_steps = [&] {
    const int64_t widest = max(g.a[seg].ld, max(g.b[BACK ? seg : 0].ld, g.b[BACK ? seg : 1].ld));
    if (widest >= (1 << 21) || (BACK && g.b[seg].ld < E)) return 0;
    return (BACK && n0 + C::kBN > g.n ? left - 1 : left) / C::kBK;
  };

  const int half = lane >> 5, in = lane & 31;
  auto read_a = [&](const char* stage, int s, u4 (&f)[P][C::kFM]) {
#pragma unroll
    for (int q = 0; q < P; ++q)
#pragma unroll
      for (int i = 0; i < C::kFM; ++i)
        f[q][i] = *reinterpret_cast<const u4*>(stage + piece_at<P>(wm + 32 * i + in, 2 * s + half, q));
  };
  auto read_b = [&](const char* stage, int s, u4 (&f)[P][C::kFN]) {
#pragma unroll
    for (int t = 0; t < P * C::kFN; ++t) {
      const int q = t / C::kFN, j = t % C::kFN;
      const char* from = stage + C::kBytesA + (BACK ? q * C::kBK * C::kPitchB : 0);
      if constexpr (!BACK) {
        f[q][j] = *reinterpret_cast<const u4*>(from + piece_at<P>(wn + 32 * j + in, 2 * s + half, q));
      } else if constexpr (kWide) {
        const int r = (2 * s + half) * E, c = (wn + 32 * j) * 4 + column_of(in) * 4;
        from += r * C::kPitchB + block_at<kWide>(r, c >> 6) * 64 + (c & 63);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[q][j][e] = *reinterpret_cast<const uint32_t*>(from + e * C::kPitchB);
      } else {
        // four rows of 16 columns for 16 lanes; the lanes' groups of 4 columns in the products' order
        const int group = 4 * ((lane >> 4) & 1) + (lane & 3), r4 = (lane & 15) >> 2;
        from += ((2 * s + half) * 8 + r4) * C::kPitchB + block_at<kWide>(r4, (wn + 32 * j) >> 5) * 64 +
                (16 * (group & 1) + 4 * (group >> 1)) * 2;
        const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)from);
        const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(from + 4 * C::kPitchB));
        f[q][j] = __builtin_bit_cast(u4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  };

  // The next step, whichever it is.
  auto load_step = [&](u4 (&to)[kItems]) {
    if (BACK && left <= 0 && seg == 0) start(1, 0);
#pragma unroll
    for (int p = 0; p < kItems; ++p) {
      to[p] = load_edge(p);
      __builtin_amdgcn_sched_barrier(0);   // one after the other: few registers
    }
    advance();
  };

#pragma unroll
  for (int i = 0; i < C::kFM; ++i)
#pragma unroll
    for (int j = 0; j < C::kFN; ++j) acc[i][j] = f16v{};
  char *cur = s_mem, *nxt = s_mem + C::kStage;
  constexpr int R = C::kAhead;
  u4 reg[R][kItems];     // the pieces of the steps after the next: reg[0] is the first to be stored
  u4 fa[P][C::kFM], fb[P][C::kFN];
  if (steps > 0) {
    start(first >= steps_seg, first >= steps_seg ? first - steps_seg : first);
    u4 now[kItems];
    if (steps > R && whole_steps() > R) {   // all on their way at once
#pragma unroll
      for (int i = 0; i <= R; ++i) {
#pragma unroll
        for (int p = 0; p < kItems; ++p) (i ? reg[i - 1] : now)[p] = load_whole(p);
        advance();
      }
    } else {
      load_step(now);
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i + 1 < steps) load_step(reg[i]);
    }
#pragma unroll
    for (int p = 0; p < kItems; ++p) store(cur, p, now[p]);
    __syncthreads();
    read_b(cur, 0, fb);
    read_a(cur, 0, fa);
  }
  // One step: each slice is multiplied while the operands of the next are read.  During all slices but the
  // last the next step's pieces, loaded kAhead steps ago, go to the other stage, each followed by the load
  // of a piece of the step kAhead after it, where that is whole.  Before the last slice all waves meet: the other
  // stage is complete then, and nobody reads this one any more.
  int step = 0;
  auto turn = [&] {      // the set that was stored last is loaded last
#pragma unroll
    for (int p = 0; p < kItems; ++p)
      if (R == 2) {
        const u4 w = reg[0][p];
        reg[0][p] = reg[R - 1][p];
        reg[R - 1][p] = w;
      }
  };
  auto multiply_step = [&](auto load, auto which) {
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      u4 na[P][C::kFM], nb[P][C::kFN];
      if (s + 1 == kSlices) __syncthreads();
      read_b(s + 1 < kSlices ? cur : nxt, (s + 1) % kSlices, nb);
      read_a(s + 1 < kSlices ? cur : nxt, (s + 1) % kSlices, na);
#pragma unroll
      for (int p = 0; p < kItems; ++p)
        if (p * (kSlices - 1) / kItems == s) {
          store(nxt, p, reg[which][p]);
          if (load) reg[which][p] = load_whole(p);
        }
      // all pairs of parts but those below 2^-23 of the product, the smallest first
#pragma unroll
      for (int d = P - 1; d >= 0; --d)
#pragma unroll
        for (int q = 0; q <= d; ++q)
#pragma unroll
          for (int i = 0; i < C::kFM; ++i)
#pragma unroll
            for (int j = 0; j < C::kFN; ++j)
              multiply<P == 1 ? DT : kBF16>(fb[q][j], fa[d - q][i], acc[i][j]);
      // each matrix instruction followed by a share of the rest, which runs beside it
#pragma unroll
      for (int u = 0; u < C::kFM * C::kFN * P * (P + 1) / 2; ++u) {
        __builtin_amdgcn_sched_group_barrier(0x008, kWide ? 4 : 1, 0);   // matrix
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);               // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x002, P == 1 ? 4 : 8, 0);  // vector
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);               // loads
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);               // LDS writes
      }
#pragma unroll
      for (int q = 0; q < P; ++q) {
#pragma unroll
        for (int i = 0; i < C::kFM; ++i) fa[q][i] = na[q][i];
#pragma unroll
        for (int j = 0; j < C::kFN; ++j) fb[q][j] = nb[q][j];
      }
    }
    if (load) advance();
    char* t = cur;
    cur = nxt;
    nxt = t;
    ++step;
  };
  while (step < steps) {
    if (BACK && left <= 0 && seg == 0) start(1, 0);
    int n = min(whole_steps(), steps - 1 - R - step);
    if constexpr (R == 2)
      for (; n > 1; n -= 2) {   // the two sets in turn
        multiply_step(std::true_type(), std::integral_constant<int, 0>());
        multiply_step(std::true_type(), std::integral_constant<int, 1>());
      }
    for (; n > 0; --n) {
      multiply_step(std::true_type(), std::integral_constant<int, 0>());
      turn();
    }
    if (BACK && left <= 0 && seg == 0 && step + 1 + R < steps) continue;
    multiply_step(std::false_type(), std::integral_constant<int, 0>());
    if (step + R < steps) load_step(reg[0]);   // step is one further now
    turn();
  }
}

template <int DT, bool BACK, typename C, int ACT>
__global__ __launch_bounds__(C::kThreads, 2) void k_product(Product g) {
  __shared__ __align__(16) char s_mem[2 * C::kStage];
  int tm, tn;
  tile_of((int)((g.rows + C::kBM - 1) / C::kBM), (g.n + C::kCols - 1) / C::kCols, &tm, &tn);
  const int64_t m0 = (int64_t)tm * C::kBM;
  const int n0 = tn * C::kCols;
  const int wave = __builtin_amdgcn_readfirstlane(wave_id());
  const int wm = wave / C::kWN * (C::kFM * 32), wn = wave % C::kWN * (C::kFN * 32);
  const int all = (BACK ? 2 : 1) * ((g.depth + C::kBK - 1) / C::kBK);
  const int first = (int)((int64_t)all * blockIdx.y / g.splits);
  const int steps = (int)((int64_t)all * (blockIdx.y + 1) / g.splits) - first;
  f16v acc[C::kFM][C::kFN];
  sum_tile<DT, BACK, C>(g, s_mem, m0, n0, first, steps, acc);
  if constexpr (C::kParts > 1) {
    // Parts do not multiply Inf as it is, and the first of them may overflow where the value does not: what
    // came out as Inf or NaN is what the sum of whole elements says.
    bool again = false;
    auto each = [&](auto&& f) {
#pragma unroll
      for (int i = 0; i < C::kFM; ++i)
#pragma unroll
        for (int j = 0; j < C::kFN; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) f(i, j, r);
    };
    auto finite = [](float v) { return fabsf(v) <= 3.402823466e38f; };   // NaN is not
    each([&](int i, int j, int r) { again |= !finite(acc[i][j][r]); });
    if (__syncthreads_or(again)) {
      f16v whole[C::kFM][C::kFN];
      sum_tile<DT, BACK, typename C::Whole>(g, s_mem, m0, n0, first, steps, whole);
      each([&](int i, int j, int r) {
        if (!finite(acc[i][j][r])) acc[i][j][r] = whole[i][j][r];
      });
    }
  }
  // each wave's own part of LDS, which all have stopped reading
  constexpr int kPart = 2 * C::kStage / (C::kThreads / 64);
  static_assert(kPart >= 32 * 32 * (BACK ? C::kFN : C::kFN / 2) * 4, "a block of fp32");
  char* lds = s_mem + wave * kPart;
  if (n0 + C::kCols <= g.n)
    finish<DT, BACK, C, ACT, true>(g, acc, lds, m0, n0, wm, wn);
  else
    finish<DT, BACK, C, ACT, false>(g, acc, lds, m0, n0, wm, wn);
}

// The parts of the sums joined in order, 8 columns a thread.
template <int DT, bool BACK, int ACT>
__global__ __launch_bounds__(256) void k_product_join(Product g) {
  typedef typename Elt<DT>::T T;
  const int octets = (g.n + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = i / octets;
  if (row >= g.rows) return;
  const int col = (int)(i - row * octets) * 8;
  const int64_t part = (BACK ? 1 : 2) * g.rows * g.n;
  float v[8] = {}, u[8] = {};
  auto add = [&](const float* p, float (&sum)[8]) {
    for (int s = 0; s < g.splits; s += 4) {   // 4 parts in flight
      float w[4][8] = {};
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (s + t < g.splits) load8<kF32>(p + (s + t) * part, col, g.n, w[t]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += w[t][j];
    }
  };
  add(g.ws + row * g.n, v);
  if (!BACK) add(g.ws + (g.rows + row) * g.n, u);
  auto put = [&](const Mat& m, const float (&w)[8]) {
    store8<DT>(static_cast<T*>(m.p) + row * m.ld, col, g.n, w);
  };
  if (!BACK) {
    if (g.out[1].p) put(g.out[1], v);
    if (g.out[2].p) put(g.out[2], u);
    gate<ACT, 8>(v, u);
  }
  put(g.out[0], v);
}

// ------------------------------------------------------------------ few rows
// The forward pass of up to 32 rows, as in serving: the weights are read once and everything else is small.
// A workgroup forms 16 columns of each projection, which are the 32 rows of one operand; its 8 waves share
// the sum, 128 bytes of the rows at a time, each operand straight from memory, and join their parts in
// LDS: many workgroups, no second launch.  One row through 4096 x 1024 bf16 takes 4.3 us of the GPU (tiles
// 8.6), through 11008 x 4096 31 (5.8 TB/s; 32.5), both with the weights in the 256 MB cache.
constexpr int kFewRows = 32, kFewWaves = 8, kFewColumns = 16;

template <int DT, int ACT>
__global__ __launch_bounds__(64 * kFewWaves) void k_gated_few(Product g) {
  typedef typename Elt<DT>::T T;
  constexpr int E = kChunk / sizeof(T), kDeep = kRowChunks * E, kPieces = kRowChunks / 2;
  __shared__ float s_sum[kFewWaves][32][33];   // 33: the columns of a row in different banks
  const int lane = lane_id(), wave = wave_id(), half = lane >> 5, in = lane & 31;
  const int n0 = blockIdx.x * kFewColumns;
  const Mat& w = g.b[in >> 4];
  const T* pw = static_cast<const T*>(w.p) + min(n0 + (in & 15), g.n - 1) * w.ld;
  const T* px = static_cast<const T*>(g.a[0].p) + min((int64_t)in, g.rows - 1) * g.a[0].ld;
  f16v acc = {};
  u4 fw[kPieces], fx[kPieces];
  auto load = [&](int k0) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int k = k0 + (2 * j + half) * E;
      if (k0 + kDeep <= g.depth) {
        fw[j] = *reinterpret_cast<const u4_at_any*>(pw + k);
        fx[j] = *reinterpret_cast<const u4_at_any*>(px + k);
      } else {
        fw[j] = load_piece(pw, k, g.depth);
        fx[j] = load_piece(px, k, g.depth);
      }
    }
  };
  int k0 = wave * kDeep;
  if (k0 < g.depth) load(k0);
  while (k0 < g.depth) {
    u4 cw[kPieces], cx[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      cw[j] = fw[j];
      cx[j] = fx[j];
    }
    k0 += kFewWaves * kDeep;
    if (k0 < g.depth) load(k0);
#pragma unroll
    for (int j = 0; j < kPieces; ++j) multiply<DT>(cw[j], cx[j], acc);
  }
#pragma unroll
  for (int r = 0; r < 16; ++r) s_sum[wave][8 * (r >> 2) + 4 * half + (r & 3)][in] = acc[r];
  __syncthreads();
  static_assert(64 * kFewWaves == kFewRows * kFewColumns, "a thread for each result");
  const int i = threadIdx.x % kFewColumns, row = threadIdx.x / kFewColumns, col = n0 + i;
  if (col >= g.n || row >= g.rows) return;
  float v[1] = {}, u[1] = {};
#pragma unroll
  for (int k = 0; k < kFewWaves; ++k) {
    v[0] += s_sum[k][i][row];
    u[0] += s_sum[k][16 + i][row];
  }
  auto put = [&](const Mat& m, float x) {
    static_cast<T*>(m.p)[row * m.ld + col] = round_to<DT>(x);
  };
  if (g.out[1].p) put(g.out[1], v[0]);
  if (g.out[2].p) put(g.out[2], u[0]);
  gate<ACT, 1>(v, u);
  put(g.out[0], v[0]);
}

template <int DT, bool BACK, int ACT, typename C>
hipError_t product(const Product& g, hipStream_t st) {
  const int64_t tiles = (g.rows + C::kBM - 1) / C::kBM * ((g.n + C::kCols - 1) / C::kCols);
  k_product<DT, BACK, C, ACT><<<dim3((unsigned)tiles, g.splits), C::kThreads, 0, st>>>(g);
  return hipGetLastError();
}

template <int DT, bool BACK>
using Large = std::conditional_t<DT == kF32, Tile<DT, BACK, 256, 128, 4, 2, 3>,
                                 Tile<DT, BACK, 256, 256, 2, 4>>;
template <int DT, bool BACK>
using Small = Tile<DT, BACK, 128, 128, 2, 2, DT == kF32 ? 3 : 1>;
template <int DT, bool BACK, int AHEAD = 1>
using Tiny = Tile<DT, BACK, 64, 128, 2, 2, DT == kF32 ? 3 : 1, AHEAD>;

enum TileKind { kLarge, kSmall, kTiny, kFew };   // kFew: the forward pass of few rows

struct Shape {
  TileKind tile;
  int splits, ahead;   // ahead: of tiny 16-bit tiles
};

// A large tile needs the fewest loads a product, but leaves CUs idle where the result is small; a long sum
// can be split over CUs, at the price of writing and joining its parts.  The tile and the split with the
// least estimated time are taken.  A step (64 summed columns of the 16-bit types, 32 of fp32) of a tile
// takes, with 1, 2 and 3 workgroups on its CU, in microseconds (measured; a CU holds 1 large tile, of the
// 16-bit types 2 small or 3 tiny ones, of fp32 1 and 2):
//              large          small       tiny
//   16 bits    1.15 or 1.72   0.53 1.0    0.43 0.69 1.05
//   fp32       1.6 or 2.4     1.4         0.84 1.47         (large: on up to half of the CUs, or all)
// and a round of tiles 16, 7 or 4 us (fp32 9, 7, 5) besides (launch, first loads, the results' way); a join
// 6 us (the host's share among them), 0.5 us a part and their bytes (written and read) at 5 TB/s.  Where
// the 16-bit types' rows are not whole 16 bytes wide, as where they start anywhere, a large step takes 1.15
// times and the others 1.45 times as long.  Measured against every other choice over 80 drawn sizes, the rule's
// takes 3 % longer than the best.
//
// Up to 2 tiny 16-bit tiles a CU load their pieces two steps ahead, which the third workgroup's registers
// would pay for: at 1 a CU the step waits for its loads (0.50 us one step ahead; with the weights from memory
// 0.75 against 0.5: 27 rows through 4096 x 4096 bf16 47 and 33 us), at 3 others fill the time.  Sums of fewer
// than 8 steps gain nothing and begin later (123 rows through 6963 x 158 8.2 and 10.9 us).
//
// Where one tile holds all rows nothing shares the weights' loads, which come from memory then: a tiny
// tile's 16-bit step takes 0.5, 1.0 and 1.6 us, a small one's 0.75 and 1.3 (27 rows through 11008 x 4096 bf16,
// the weights not in any cache: whole sums 44.7 us, in 4 parts 41.5; the rule, to which the whole sums are 64
// steps of 0.5 and 4 us, takes them).  These steps go by the rows alone, whatever the weights' size.
//
// Up to 32 rows of a forward pass may go without tiles: 3.5 us, and for each 1 KB of a row's sum 1.65 us (fp32
// 1.85, ragged 16-bit rows 2.9; less on part of the CUs) and a little more with the rows, with the
// workgroups in as many turns as fill the CUs.  Weights not in any cache, one row through 4096 x 4096 bf16
// 16.0 us (tiles 21.2), 11008 x 4096 44.7 (37.9), 8192 x 1000 11.0 (15.9); 32 rows through 4096 x 4096 27.4
// (22.2).
Shape shape_of(int64_t rows, int32_t n, int32_t depth, bool back, int dtype) {
  struct Costs {
    int columns, per_cu[3], bk;
    double few, round[3], step[3][3];
  };
  constexpr Costs k16 = {
      256, {1, 2, 3}, 64, 1.15, {16.0, 7.0, 4.0}, {{1.72}, {0.53, 1.0}, {0.43, 0.69, 1.05}}};
  constexpr Costs k16far = {
      256, {1, 2, 3}, 64, 1.15, {16.0, 7.0, 4.0}, {{1.72}, {0.75, 1.3}, {0.5, 1.0, 1.6}}};
  constexpr Costs k32 = {128, {1, 1, 2}, 32, 1.6, {9.0, 7.0, 5.0}, {{2.4}, {1.4}, {0.84, 1.47}}};
  constexpr int kRows[3] = {256, 128, 64};
  constexpr int64_t kCUs = 256;
  const Costs& k = dtype == kF32 ? k32 : rows <= 128 ? k16far : k16;
  const int64_t steps = (back ? 2 : 1) * (((int64_t)depth + k.bk - 1) / k.bk);
  const bool ragged = dtype != kF32 && (depth % 8 || (back && n % 8));
  Shape best = {kTiny, 1, 1};
  double least = 1e300;
  if (!back && rows <= kFewRows && n < 1 << 26) {   // a launch's threads are counted in 32 bits
    // a turn: 1 KB of each row for the 8 waves; of less, most have nothing to do
    const double turns = depth > 8 * k.bk ? (double)((depth - 1) / (8 * k.bk) + 1)
                         : depth > 2 * k.bk ? depth / (8.0 * k.bk) : 0.3;
    const double groups = (double)((n + kFewColumns - 1) / kFewColumns) / kCUs;
    const double some = groups < 1.0 ? groups : 1.0;
    least = 3.5 + turns * (groups / some) *
                      (dtype == kF32 ? 1.5 + 0.35 * some + 0.04 * rows
                       : ragged      ? 2.0 + 0.9 * some + 0.075 * rows
                                     : 1.0 + 0.65 * some + 0.055 * rows);
    best = {kFew, 1, 1};
  }
  for (int t = 0; t < 3; ++t) {
    const int columns = (t == kLarge ? k.columns : 128) / (back ? 1 : 2);
    const int64_t tiles = (rows + kRows[t] - 1) / kRows[t] * ((n + columns - 1) / columns);
    const double slower = !ragged ? 1.0 : t == kLarge ? 1.15 : 1.45;
    for (int s = 1; s <= 32 && (s == 1 || 4 * s <= steps); s += s < 4 ? 1 : s / 2) {
      const int64_t at_once = kCUs * k.per_cu[t], groups = tiles * s, full = groups / at_once;
      const int64_t rest = groups - full * at_once;
      const double part = (double)((steps + s - 1) / s) * slower;
      double us = full * (part * k.step[t][k.per_cu[t] - 1] + k.round[t]);
      if (rest)
        us += k.round[t] + part * (t == kLarge && groups <= kCUs / 2 ? k.few
                                                                    : k.step[t][(rest - 1) / kCUs]);
      if (s > 1) us += 6.0 + 0.5 * s + 2.0 * 4.0 * s * (double)rows * n * (back ? 1 : 2) / 5e6;
      if (us < least) {
        least = us;
        best = {(TileKind)t, s, t == kTiny && dtype != kF32 && groups <= 2 * kCUs && steps >= 8 * s ? 2 : 1};
      }
    }
  }
  return best;
}

int64_t workspace_of(int64_t rows, int32_t n, int32_t depth, bool back, int dtype) {
  if (rows == 0 || n == 0) return 0;
  const int s = shape_of(rows, n, depth, back, dtype).splits;
  return s > 1 ? (int64_t)s * (back ? 1 : 2) * rows * n * 4 : 0;
}

template <int DT, bool BACK, int ACT>
hipError_t product(Product g, hipStream_t st) {
  const Shape s = shape_of(g.rows, g.n, g.depth, BACK, DT);
  g.splits = s.splits;
  if constexpr (!BACK)
    if (s.tile == kFew) {
      const unsigned grid = (g.n + kFewColumns - 1) / kFewColumns;
      k_gated_few<DT, ACT><<<grid, 64 * kFewWaves, 0, st>>>(g);
      return hipGetLastError();
    }
  hipError_t e = hipSuccess;
  if (s.tile == kLarge)
    e = product<DT, BACK, ACT, Large<DT, BACK>>(g, st);
  else if (s.tile == kSmall)
    e = product<DT, BACK, ACT, Small<DT, BACK>>(g, st);
  else if (s.ahead == 2)
    e = product<DT, BACK, ACT, Tiny<DT, BACK, DT == kF32 ? 1 : 2>>(g, st);
  else
    e = product<DT, BACK, ACT, Tiny<DT, BACK>>(g, st);
  if (e || g.splits == 1) return e;
  k_product_join<DT, BACK, ACT><<<blocks_for(g.rows * ((g.n + 7) / 8), 256), 256, 0, st>>>(g);
  return hipGetLastError();
}

template <int DT>
hipError_t forward(const Product& g, hipStream_t st) {
  return g.act == kSilu   ? product<DT, false, kSilu>(g, st)
         : g.act == kGelu ? product<DT, false, kGelu>(g, st)
                          : product<DT, false, kGeluTanh>(g, st);
}

template <int DT>
hipError_t slope(const GatedGradArgs& a, hipStream_t st) {
  const unsigned grid = blocks_for(a.rows * ((a.n + 7) / 8), 256);
  if (a.act == kSilu)
    k_gated_slope<DT, kSilu><<<grid, 256, 0, st>>>(a);
  else if (a.act == kGelu)
    k_gated_slope<DT, kGelu><<<grid, 256, 0, st>>>(a);
  else
    k_gated_slope<DT, kGeluTanh><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace

int64_t gated_workspace(int64_t rows, int32_t n, int32_t cols, int dtype) {
  return workspace_of(rows, n, cols, false, dtype);
}

int64_t gated_grad_workspace(int64_t rows, int32_t n, int32_t cols, int dtype) {
  return workspace_of(rows, cols, n, true, dtype);
}

hipError_t launch_gated(const GatedArgs& a, hipStream_t st) {
  if (a.rows == 0 || a.n == 0) return hipSuccess;
  Product g{};
  g.rows = a.rows;
  g.n = a.n;
  g.depth = a.cols;
  g.a[0] = a.x;
  g.b[0] = a.w_gate;
  g.b[1] = a.w_up;
  g.out[0] = a.h;
  g.out[1] = a.gate;
  g.out[2] = a.up;
  g.act = a.act;
  g.ws = static_cast<float*>(a.ws);
  return a.dtype == kF32    ? forward<kF32>(g, st)
         : a.dtype == kBF16 ? forward<kBF16>(g, st)
                            : forward<kF16>(g, st);
}

hipError_t launch_gated_backward(const GatedGradArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (a.n)
    if (hipError_t e = a.dtype == kF32    ? slope<kF32>(a, st)
                       : a.dtype == kBF16 ? slope<kBF16>(a, st)
                                          : slope<kF16>(a, st))
      return e;
  if (!a.dx.p || a.cols == 0) return hipSuccess;
  Product g{};
  g.rows = a.rows;
  g.n = a.cols;
  g.depth = a.n;
  g.a[0] = a.dgate;
  g.a[1] = a.dup;
  g.b[0] = a.w_gate;
  g.b[1] = a.w_up;
  g.out[0] = a.dx;
  g.ws = static_cast<float*>(a.ws);
  return a.dtype == kF32    ? product<kF32, true, kSilu>(g, st)
         : a.dtype == kBF16 ? product<kBF16, true, kSilu>(g, st)
                            : product<kF16, true, kSilu>(g, st);
}

}  // namespace gc
