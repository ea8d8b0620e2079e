// gc_gated.hip -- the gated feed-forward block and its backward pass.
//
//   forward    G = X Wg^T, U = X Wu^T, h = act(G) * U, in one kernel: a workgroup forms the same
//              columns of G and of U, so that their product is taken from its registers.
//   backward   dG = dh * U * act'(G), dU = dh * act(G) of the kept rows of G and U, a stream of
//              five matrices; then dX = dG Wg + dU Wu, one product whose sum runs over the columns of
//              dG and then over those of dU.
//
// The products run on the matrix cores (32x32x16 for the 16-bit types, 32x32x2 fp32) with sums in
// fp32.  Their first operand is the weight, so that a lane ends up with 16 neighbouring columns of one
// row of the result (the 32 columns of a product are handed out in that order) and stores them in
// 16-byte pieces.
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
// act(g) and its derivative.  p is the factor that both start from (the logistic or the normal
// distribution function) and q what is left to 1, each formed without cancellation.
template <int ACT>
__device__ __forceinline__ void activate(float g, float* act, float* slope) {
  if (ACT == kGelu) {
    const float p = 0.5f * erfcf(g * -0.70710678f);
    *act = g * p;
    *slope = fmaf(g * 0.39894228f, expf(-0.5f * g * g), p);
    return;
  }
  constexpr float k = 1.59576912f;   // 2 sqrt(2 / pi)
  const float v = ACT == kSilu ? g : k * fmaf(0.044715f * g * g, g, g);
  const float e = expf(-fabsf(v)), r = 1.0f / (1.0f + e), s = e * r;
  const float p = v >= 0.0f ? r : s, q = v >= 0.0f ? s : r;
  *act = g * p;
  const float t = g * p * q;
  if (ACT == kSilu)
    *slope = p + t;
  else   // beyond the numbers that g's square holds, t is 0
    *slope = t == 0.0f ? p : fmaf(t, k * fmaf(0.134145f * g, g, 1.0f), p);
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
};

constexpr int kChunk = 16, kRowBytes = 128, kRowChunks = kRowBytes / kChunk;

// A workgroup's tile, BM rows by BN columns (forward: BN / 2 of each projection), shared by WM x WN
// waves.  A step sums 128 bytes of a row.
template <int DT, bool BACK, int BM, int BN, int WM, int WN>
struct Tile {
  typedef typename Elt<DT>::T T;
  static constexpr int kBM = BM, kBN = BN, kWM = WM, kWN = WN;
  static constexpr int kThreads = 64 * WM * WN;
  static constexpr int kFM = BM / WM / 32, kFN = BN / WN / 32;
  static constexpr int kElts = kChunk / (int)sizeof(T), kBK = kRowChunks * kElts;
  static constexpr int kCols = BACK ? BN : BN / 2;      // of the result
  // backward: 64 bytes past a row, so that the four rows of a transposing read start in different
  // quarters of the banks
  static constexpr int kPitchB = BACK ? BN * (int)sizeof(T) + 64 : kRowBytes;
  static constexpr int kBytesA = BM * kRowBytes, kBytesB = (BACK ? kBK : BN) * kPitchB;
  static constexpr int kItemsA = BM * kRowChunks / kThreads;
  static constexpr int kItemsB = BACK ? kBK * (BN / kElts) / kThreads : BN * kRowChunks / kThreads;
};

// Where 16-byte piece c of row r of a tile lies: the pieces of 16 neighbouring rows that a read takes
// at once fall into different banks.
__device__ __forceinline__ int piece_at(int r, int c) {
  return r * kRowBytes + ((c ^ ((r >> 1) & (kRowChunks - 1))) * kChunk);
}

// The column (of 32) that row i of a product's first operand stands for: a lane's 16 registers hold
// rows 8 * (r / 4) + 4 * (lane / 32) + r % 4, and are to be columns 16 * (lane / 32) + r.
__device__ __forceinline__ int column_of(int i) {
  return 16 * ((i >> 2) & 1) + 4 * (i >> 3) + (i & 3);
}

// 16 bytes of the row at p from element k on, zeros from `end` on.
template <typename T>
__device__ __forceinline__ u4 load_piece(const T* p, int k, int end) {
  constexpr int E = 16 / sizeof(T);
  if (k + E <= end) return *reinterpret_cast<const u4_at_any*>(p + k);
  T v[E] = {};
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (k + j < end) v[j] = p[k + j];
  u4 w;
  __builtin_memcpy(&w, v, sizeof w);
  return w;
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

// Rounds and stores a wave's products, of the forward pass after the activation.
template <int DT, bool BACK, typename C, int ACT>
__device__ __forceinline__ void finish(const Product& g, const f16v (&acc)[C::kFM][C::kFN],
                                       int64_t m0, int n0, int wm, int wn) {
  typedef typename Elt<DT>::T T;
  const int half = lane_id() >> 5, in = lane_id() & 31;
#pragma unroll
  for (int i = 0; i < C::kFM; ++i) {
    const int64_t row = m0 + wm + 32 * i + in;
    if (row >= g.rows) continue;
    auto put = [&](const Mat& m, int col, const float (&v)[8]) {
      store8<DT>(static_cast<T*>(m.p) + row * m.ld, col, g.n, v);
    };
#pragma unroll
    for (int j = 0; j < C::kFN; j += BACK ? 1 : 2)
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        const int col = n0 + (BACK ? wn + 32 * j : wn / 2 + 16 * j) + 16 * half + 8 * o;
        if (col >= g.n) continue;
        float v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) v[r] = acc[i][j][8 * o + r];
        if constexpr (BACK) {
          put(g.out[0], col, v);
        } else {
          float u[8];
#pragma unroll
          for (int r = 0; r < 8; ++r) u[r] = acc[i][j + 1][8 * o + r];
          if (g.out[1].p) put(g.out[1], col, v);
          if (g.out[2].p) put(g.out[2], col, u);
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            float act, slope;
            activate<ACT>(v[r], &act, &slope);
            v[r] = act * u[r];
          }
          put(g.out[0], col, v);
        }
      }
  }
}

template <int DT, bool BACK, typename C, int ACT>
__global__ __launch_bounds__(C::kThreads) void k_product(Product g) {
  typedef typename Elt<DT>::T T;
  constexpr int E = C::kElts;
  __shared__ __align__(16) char s_mem[2 * (C::kBytesA + C::kBytesB)];
  const int tiles_m = (int)((g.rows + C::kBM - 1) / C::kBM);
  const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * C::kBM;
  const int n0 = (int)(blockIdx.x / tiles_m) * C::kCols;
  const int lane = lane_id(), wave = wave_id();
  const int wm = wave / C::kWN * (C::kFM * 32), wn = wave % C::kWN * (C::kFN * 32);
  const int steps_seg = (g.depth + C::kBK - 1) / C::kBK, steps = BACK ? 2 * steps_seg : steps_seg;

  u4 ra[C::kItemsA], rb[C::kItemsB];
  auto load = [&](int step) {
    const int seg = BACK && step >= steps_seg, k0 = (step - seg * steps_seg) * C::kBK;
#pragma unroll
    for (int p = 0; p < C::kItemsA; ++p) {
      const int at = p * C::kThreads + threadIdx.x, r = at / kRowChunks, c = at % kRowChunks;
      const int64_t row = min(m0 + r, g.rows - 1);
      ra[p] = load_piece(static_cast<const T*>(g.a[seg].p) + row * g.a[seg].ld, k0 + c * E, g.depth);
    }
#pragma unroll
    for (int p = 0; p < C::kItemsB; ++p) {
      const int at = p * C::kThreads + threadIdx.x;
      if (BACK) {
        const int r = k0 + at / (C::kBN / E), c = at % (C::kBN / E);
        rb[p] = r < g.depth ? load_piece(static_cast<const T*>(g.b[seg].p) + (int64_t)r * g.b[seg].ld,
                                         n0 + c * E, g.n)
                            : u4{};
      } else {
        const int r = at / kRowChunks, c = at % kRowChunks, w = (r >> 5) & 1;
        const int row = min(n0 + (r >> 6) * 32 + column_of(r & 31), g.n - 1);
        rb[p] = load_piece(static_cast<const T*>(g.b[w].p) + (int64_t)row * g.b[w].ld, k0 + c * E,
                           g.depth);
      }
    }
  };
  auto store = [&](char* stage) {
#pragma unroll
    for (int p = 0; p < C::kItemsA; ++p) {
      const int at = p * C::kThreads + threadIdx.x;
      *reinterpret_cast<u4*>(stage + piece_at(at / kRowChunks, at % kRowChunks)) = ra[p];
    }
#pragma unroll
    for (int p = 0; p < C::kItemsB; ++p) {
      const int at = p * C::kThreads + threadIdx.x;
      char* q = stage + C::kBytesA;
      if (BACK)
        q += at / (C::kBN / E) * C::kPitchB + at % (C::kBN / E) * kChunk;
      else
        q += piece_at(at / kRowChunks, at % kRowChunks);
      *reinterpret_cast<u4*>(q) = rb[p];
    }
  };
  const int half = lane >> 5, in = lane & 31;
  auto read_a = [&](const char* stage, int s, int i) {
    return *reinterpret_cast<const u4*>(stage + piece_at(wm + 32 * i + in, 2 * s + half));
  };
  auto read_b = [&](const char* stage, int s, int j) {
    const char* q = stage + C::kBytesA;
    if constexpr (!BACK) {
      return *reinterpret_cast<const u4*>(q + piece_at(wn + 32 * j + in, 2 * s + half));
    } else if constexpr (DT == kF32) {
      q += (2 * s + half) * E * C::kPitchB + (wn + 32 * j + column_of(in)) * 4;
      u4 w;
#pragma unroll
      for (int t = 0; t < 4; ++t) w[t] = *reinterpret_cast<const uint32_t*>(q + t * C::kPitchB);
      return w;
    } else {
      // four rows of 16 columns for 16 lanes; the lanes' groups of 4 columns in the products' order
      const int group = 4 * ((lane >> 4) & 1) + (lane & 3);
      q += ((2 * s + half) * E + ((lane & 15) >> 2)) * C::kPitchB +
           (wn + 32 * j + 16 * (group & 1) + 4 * (group >> 1)) * 2;
      const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)q);
      const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(q + 4 * C::kPitchB));
      return __builtin_bit_cast(u4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };

  f16v acc[C::kFM][C::kFN] = {};
  char *cur = s_mem, *nxt = s_mem + C::kBytesA + C::kBytesB;
  if (steps) {
    load(0);
    store(cur);
  }
  __syncthreads();
  for (int step = 0; step < steps; ++step) {
    if (step + 1 < steps) load(step + 1);
#pragma unroll
    for (int s = 0; s < kRowChunks / 2; ++s) {
      u4 fa[C::kFM], fb[C::kFN];
#pragma unroll
      for (int i = 0; i < C::kFM; ++i) fa[i] = read_a(cur, s, i);
#pragma unroll
      for (int j = 0; j < C::kFN; ++j) fb[j] = read_b(cur, s, j);
#pragma unroll
      for (int i = 0; i < C::kFM; ++i)
#pragma unroll
        for (int j = 0; j < C::kFN; ++j) multiply<DT>(fb[j], fa[i], acc[i][j]);
    }
    if (step + 1 < steps) store(nxt);
    __syncthreads();
    char* t = cur;
    cur = nxt;
    nxt = t;
  }

  finish<DT, BACK, C, ACT>(g, acc, m0, n0, wm, wn);
}

// ------------------------------------------------------------------ whole pieces: loaded into LDS directly
// The same product where every row of an operand starts on 16 bytes and holds whole 16-byte pieces:
// the loads write LDS themselves, a wave 1024 bytes of a stage at a time, in the order of the lanes; so
// what a lane loads is what belongs into its place, and the places of a row's pieces are permuted as
// above without a gap between rows.
__device__ const u4 g_zeros = {0, 0, 0, 0};

typedef __attribute__((address_space(1))) const void global_void;
typedef __attribute__((address_space(3))) void lds_void;

template <int DT, bool BACK, int BM, int BN, int WM, int WN>
struct DirectTile : Tile<DT, BACK, BM, BN, WM, WN> {
  typedef Tile<DT, BACK, BM, BN, WM, WN> Base;
  // pieces of a row of the second operand's stage
  static constexpr int kPiecesB = BACK ? BN / Base::kElts : kRowChunks;
  static constexpr int kPitchB = kPiecesB * kChunk;
  static constexpr int kBytesB = (BACK ? Base::kBK : BN) * kPitchB, kStage = Base::kBytesA + kBytesB;
  static constexpr int kRowsA = Base::kThreads / kRowChunks, kRowsB = Base::kThreads / kPiecesB;
};

// Where the 64-byte block b of row r lies in a row of the second operand (backward): the four rows of a
// transposing read (fp32: the two halves of a wave, four rows apart) in different banks.
template <int DT>
__device__ __forceinline__ int block_at(int r, int b) {
  return DT == kF32 ? b ^ ((r >> 1) & 2) : b ^ (r & 3);
}

template <int DT, bool BACK, typename C, int ACT>
__global__ __launch_bounds__(C::kThreads, 2) void k_product_direct(Product g) {
  typedef typename Elt<DT>::T T;
  constexpr int E = C::kElts;
  __shared__ __align__(16) char s_mem[2 * C::kStage];
  const int tiles_m = (int)((g.rows + C::kBM - 1) / C::kBM);
  const int64_t m0 = (int64_t)(blockIdx.x % tiles_m) * C::kBM;
  const int n0 = (int)(blockIdx.x / tiles_m) * C::kCols;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(wave_id());
  const int wm = wave / C::kWN * (C::kFM * 32), wn = wave % C::kWN * (C::kFN * 32);
  const int steps_seg = (g.depth + C::kBK - 1) / C::kBK, steps = BACK ? 2 * steps_seg : steps_seg;

  // This thread's piece of every item: A's row p * kRowsA + ra, piece ca of the step; B's likewise.
  const int ra = threadIdx.x / kRowChunks, ca = (threadIdx.x % kRowChunks) ^ ((ra >> 1) & 7);
  const int rb = threadIdx.x / C::kPiecesB, sb = threadIdx.x % C::kPiecesB;
  const int cb = BACK ? block_at<DT>(rb, sb >> 2) * 4 + (sb & 3) : sb ^ ((rb >> 1) & 7);
  // The place of the next step to be fetched, the same in all lanes, and from it the byte offset of each
  // item's row (rows past the last one read it, columns past the last one the tile's first; what they
  // add up is not stored).
  const char *pa, *pb[2];
  int64_t next_b;
  uint32_t off_a[C::kItemsA], off_b[C::kItemsB];
  int left;              // of the segment's sum, from the next step on
  auto start = [&](int seg) {
    const Mat& a = g.a[seg];
    left = g.depth;
    pa = static_cast<const char*>(a.p) + m0 * a.ld * (int64_t)sizeof(T);
    if (BACK) {
      pb[0] = static_cast<const char*>(g.b[seg].p) + n0 * (int64_t)sizeof(T);
      next_b = C::kBK * g.b[seg].ld * (int64_t)sizeof(T);
    } else {
      // a wave loads 8 rows at a time, of one of the weights: always the same or each in turn
      const int w = C::kRowsB == 64 ? (wave >> 2) & 1 : 0;
      pb[0] = static_cast<const char*>(g.b[w].p) + n0 * g.b[w].ld * (int64_t)sizeof(T);
      pb[1] = static_cast<const char*>(g.b[1].p) + n0 * g.b[1].ld * (int64_t)sizeof(T);
      next_b = kRowBytes;
    }
#pragma unroll
    for (int p = 0; p < C::kItemsA; ++p)
      off_a[p] = (uint32_t)((min(m0 + p * C::kRowsA + ra, g.rows - 1) - m0) * a.ld *
                            (int64_t)sizeof(T)) + ca * kChunk;
#pragma unroll
    for (int p = 0; p < C::kItemsB; ++p) {
      const int r = p * C::kRowsB + rb;
      const int64_t pitch = g.b[BACK ? seg : (r >> 5) & 1].ld * (int64_t)sizeof(T);
      if (BACK)
        off_b[p] = (uint32_t)(r * pitch) + (n0 + cb * E < g.n ? cb * kChunk : 0);
      else
        off_b[p] = (uint32_t)((min(n0 + (r >> 6) * 32 + column_of(r & 31), g.n - 1) - n0) * pitch) +
                   cb * kChunk;
    }
  };
  auto item = [&](char* stage, const char* src, int p) {
    __builtin_amdgcn_global_load_lds(
        (global_void*)src, (lds_void*)(stage + wave * (64 * kChunk) + p * C::kThreads * kChunk),
        kChunk, 0, 0);
  };
  auto from_b = [&](int p) { return pb[BACK || C::kRowsB == 64 ? 0 : p & 1] + off_b[p]; };
  auto advance = [&] {
    pa += kRowBytes;
    pb[0] += next_b;
    if (!BACK) pb[1] += next_b;
    left -= C::kBK;
  };
  // The next step into a stage: one that is whole, and any; pieces behind the sum's end come from zeros.
  auto fetch_whole = [&](char* stage) {
#pragma unroll
    for (int p = 0; p < C::kItemsA; ++p) item(stage, pa + off_a[p], p);
#pragma unroll
    for (int p = 0; p < C::kItemsB; ++p) item(stage, from_b(p), C::kItemsA + p);
    advance();
  };
  auto fetch = [&](char* stage) {
    if (BACK && left <= 0) start(1);
    const char* none = reinterpret_cast<const char*>(&g_zeros);
#pragma unroll
    for (int p = 0; p < C::kItemsA; ++p) item(stage, ca * E < left ? pa + off_a[p] : none, p);
#pragma unroll
    for (int p = 0; p < C::kItemsB; ++p)
      item(stage, (BACK ? p * C::kRowsB + rb : cb * E) < left ? from_b(p) : none, C::kItemsA + p);
    advance();
  };

  const int half = lane >> 5, in = lane & 31;
  auto read_a = [&](const char* stage, int s, u4 (&f)[C::kFM]) {
#pragma unroll
    for (int i = 0; i < C::kFM; ++i)
      f[i] = *reinterpret_cast<const u4*>(stage + piece_at(wm + 32 * i + in, 2 * s + half));
  };
  auto read_b = [&](const char* stage, int s, u4 (&f)[C::kFN]) {
    const char* q = stage + C::kBytesA;
#pragma unroll
    for (int j = 0; j < C::kFN; ++j) {
      if constexpr (!BACK) {
        f[j] = *reinterpret_cast<const u4*>(q + piece_at(wn + 32 * j + in, 2 * s + half));
      } else if constexpr (DT == kF32) {
        const int r = (2 * s + half) * E, c = (wn + 32 * j) * 4 + column_of(in) * 4;
        const char* t = q + r * C::kPitchB + block_at<DT>(r, c >> 6) * 64 + (c & 63);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          f[j][e] = *reinterpret_cast<const uint32_t*>(t + e * C::kPitchB);
      } else {
        const int group = 4 * ((lane >> 4) & 1) + (lane & 3), r4 = (lane & 15) >> 2;
        const char* t = q + ((2 * s + half) * E + r4) * C::kPitchB +
                        block_at<DT>(r4, (wn + 32 * j) >> 5) * 64 +
                        (16 * (group & 1) + 4 * (group >> 1)) * 2;
        const s4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)t);
        const s4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4*)(t + 4 * C::kPitchB));
        f[j] = __builtin_bit_cast(u4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
  };

  constexpr int kItems = C::kItemsA + C::kItemsB, kSlices = kRowChunks / 2;
  static_assert(BACK || C::kRowsB == 64 || C::kRowsB == 32, "an item's rows of a wave are of one weight");
  f16v acc[C::kFM][C::kFN] = {};
  char *cur = s_mem, *nxt = s_mem + C::kStage;
  u4 fa[C::kFM], fb[C::kFN];
  if (steps) {
    start(0);
    fetch(cur);
    asm volatile("" ::: "memory");
    if (steps > 1) {
      fetch(nxt);
      // the first stage's loads are done when at most the second's are left
      asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kItems) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
    }
    read_a(cur, 0, fa);
    read_b(cur, 0, fb);
  }
  // One step: each slice is multiplied while the operands of the next are read.  Before the last one all
  // waves meet: the next stage has arrived then and nobody reads this one any more, so that the step
  // after the next goes there.
  int step = 0;
  auto multiply_step = [&](auto whole) {
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      u4 na[C::kFM], nb[C::kFN];
      if (s + 1 < kSlices) {
        read_b(cur, s + 1, nb);
        read_a(cur, s + 1, na);
      } else {
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        read_b(nxt, 0, nb);
        read_a(nxt, 0, na);
        if (whole)
          fetch_whole(cur);
        else if (step + 2 < steps)
          fetch(cur);
      }
#pragma unroll
      for (int i = 0; i < C::kFM; ++i)
#pragma unroll
        for (int j = 0; j < C::kFN; ++j) multiply<DT>(fb[j], fa[i], acc[i][j]);
      // each matrix instruction followed by a share of the rest, which runs beside it
#pragma unroll
      for (int u = 0; u < C::kFM * C::kFN; ++u) {
        __builtin_amdgcn_sched_group_barrier(0x008, DT == kF32 ? 4 : 1, 0);   // matrix
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);                    // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);                    // vector
        __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);                    // loads
      }
#pragma unroll
      for (int i = 0; i < C::kFM; ++i) fa[i] = na[i];
#pragma unroll
      for (int j = 0; j < C::kFN; ++j) fb[j] = nb[j];
    }
    char* t = cur;
    cur = nxt;
    nxt = t;
    ++step;
  };
  while (step < steps) {
    for (int n = min(left / C::kBK, steps - 2 - step); n > 0; --n) multiply_step(std::true_type());
    multiply_step(std::false_type());
  }
  finish<DT, BACK, C, ACT>(g, acc, m0, n0, wm, wn);
}

// Whether an operand's rows are whole 16-byte pieces whose offsets in a tile fit 32 bits.
bool whole_pieces(const Mat& m, int width, int size) {
  return (reinterpret_cast<uintptr_t>(m.p) | (uintptr_t)(m.ld * size) | (uintptr_t)(width * size)) %
                 kChunk == 0 && m.ld < (1 << 20);
}

template <int DT, bool BACK, int ACT>
hipError_t product(const Product& g, hipStream_t st) {
  constexpr int kSize = sizeof(typename Elt<DT>::T);
  const int width_b = BACK ? g.n : g.depth;
  if (whole_pieces(g.a[0], g.depth, kSize) && (!BACK || whole_pieces(g.a[1], g.depth, kSize)) &&
      whole_pieces(g.b[0], width_b, kSize) && whole_pieces(g.b[1], width_b, kSize)) {
    typedef DirectTile<DT, BACK, 256, 256, 2, 4> C;
    const int64_t tiles = (g.rows + C::kBM - 1) / C::kBM * ((g.n + C::kCols - 1) / C::kCols);
    k_product_direct<DT, BACK, C, ACT><<<(unsigned)tiles, C::kThreads, 0, st>>>(g);
    return hipGetLastError();
  }
  typedef Tile<DT, BACK, 128, 128, 2, 2> C;
  const int64_t tiles = (g.rows + C::kBM - 1) / C::kBM * ((g.n + C::kCols - 1) / C::kCols);
  k_product<DT, BACK, C, ACT><<<(unsigned)tiles, C::kThreads, 0, st>>>(g);
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
  (void)rows, (void)n, (void)cols, (void)dtype;
  return 0;
}

int64_t gated_grad_workspace(int64_t rows, int32_t n, int32_t cols, int dtype) {
  (void)rows, (void)n, (void)cols, (void)dtype;
  return 0;
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
  return a.dtype == kF32    ? product<kF32, true, kSilu>(g, st)
         : a.dtype == kBF16 ? product<kBF16, true, kSilu>(g, st)
                            : product<kF16, true, kSilu>(g, st);
}

}  // namespace gc
