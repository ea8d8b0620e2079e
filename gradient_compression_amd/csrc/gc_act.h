// gc_act.h -- device-side building blocks of the activation operators: the element types, the
// 8-bit checkpoint format (groups of 32 columns, a power-of-two scale each) and the lane layout
// that its writers share.
//
// An octet is 8 consecutive columns of a row, held by one lane: one 16-byte load of a 16-bit
// type, 8 bytes of codes.  A group is the 4 octets of 4 neighbouring lanes, so its largest
// magnitude is two steps inside the quad.
#pragma once

#include "gc_random.h"

namespace gc {
namespace {

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));

constexpr int kActGroup = 32;          // columns that share a scale
constexpr uint32_t kExpLowest = 7;     // 2^-120: every restored value is a normal number (or 0)
constexpr uint32_t kExpHighest = 248;  // 2^121: 127 * 2^121 is finite
constexpr uint32_t kExpBad = 255;      // 2^128 = Inf, with codes 0: the group restores to NaN
constexpr uint32_t kActTag = 0x54u;    // Philox counter tag of the stochastic rounding

template <int DT>
struct Elt;
template <>
struct Elt<kF32> {
  typedef float T;
};
template <>
struct Elt<kBF16> {
  typedef __bf16 T;
};
template <>
struct Elt<kF16> {
  typedef _Float16 T;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(_Float16 x) { return (float)x; }
// bf16 is the upper half of the binary32 bits
__device__ __forceinline__ float to_float(__bf16 x) {
  return __uint_as_float((uint32_t)__builtin_bit_cast(uint16_t, x) << 16);
}

// 8 values as they lie in memory, kept in whole registers.  They may start at any element: a
// 16-byte load bears that.
template <int DT>
struct Raw {
  static constexpr int kWords = sizeof(typename Elt<DT>::T) / 2;   // of 16 bytes
  u4 w[kWords];
};
typedef u4 __attribute__((aligned(2))) u4_at_any;
// kStream: marked non-temporal, for what is read once and is too large to be in a cache.
template <int DT, bool kStream = false>
__device__ __forceinline__ Raw<DT> load_raw(const void* p) {
  Raw<DT> r;
#pragma unroll
  for (int i = 0; i < Raw<DT>::kWords; ++i) {
    const u4_at_any* q = static_cast<const u4_at_any*>(p) + i;
    r.w[i] = kStream ? __builtin_nontemporal_load(q) : *q;
  }
  return r;
}
// Moves the words down by n halves of a word (n < 2 N), zeros from the top.
template <int N>
__device__ __forceinline__ void shift_down(uint32_t (&d)[N], uint32_t n) {
#pragma unroll
  for (int q = N / 2; q >= 1; q >>= 1)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t from = j + q < N ? d[j + q] : 0u;
      d[j] = n & (2 * q) ? from : d[j];
    }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t next = j + 1 < N ? d[j + 1] : 0u;
    d[j] = n & 1 ? (d[j] >> 16) | (next << 16) : d[j];
  }
}

// 8 columns from col of the row at p, zeros from `cols` on.  Where the row ends inside the octet its
// last 8 columns are loaded and moved into place: one load, as everywhere else.
template <int DT, bool kStream = false>
__device__ __forceinline__ Raw<DT> load_raw(const typename Elt<DT>::T* p, int col, int cols) {
  constexpr int kWords = 4 * Raw<DT>::kWords, kHalves = sizeof(typename Elt<DT>::T) / 2;
  if (col + 8 <= cols) return load_raw<DT, kStream>(p + col);
  Raw<DT> r = {};
  if (col >= cols) return r;
  uint32_t d[kWords] = {};
  if (cols >= 8) {
    __builtin_memcpy(d, p + cols - 8, sizeof d);
    shift_down<kWords>(d, (uint32_t)(col + 8 - cols) * kHalves);
  } else {   // a row of fewer than 8 columns: from its end, each column under the last
#pragma unroll 1
    for (int j = cols - 1; j >= 0; --j) {
      uint32_t e;
      if constexpr (kHalves == 1)
        e = __builtin_bit_cast(uint16_t, p[j]);
      else
        e = __builtin_bit_cast(uint32_t, p[j]);
#pragma unroll
      for (int i = kWords - 1; i >= 0; --i) {
        const uint32_t below = i ? d[i - 1] : (kHalves == 1 ? e << 16 : e);
        d[i] = kHalves == 1 ? (d[i] << 16) | (below >> 16) : below;
      }
    }
  }
  __builtin_memcpy(&r, d, sizeof r);
  return r;
}
template <int DT>
__device__ __forceinline__ void to_float8(const Raw<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (DT == kF32)
      v[j] = __uint_as_float(r.w[j / 4][j % 4]);
    else if constexpr (DT == kBF16)
      v[j] = __uint_as_float(j % 2 ? r.w[0][j / 2] & 0xFFFF0000u : r.w[0][j / 2] << 16);
    else
      v[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.w[0][j / 2] >> (16 * (j % 2))));
  }
}
template <int DT>
__device__ __forceinline__ void load8(const typename Elt<DT>::T* p, int col, int cols,
                                      float (&v)[8]) {
  to_float8<DT>(load_raw<DT>(p, col, cols), v);
}

// One value, and 8, of a vector over the columns whose type is only known at run time; ones for
// no vector.
__device__ __forceinline__ float load_any(const void* p, int dtype, int64_t i) {
  return dtype == kF32    ? static_cast<const float*>(p)[i]
         : dtype == kBF16 ? to_float(static_cast<const __bf16*>(p)[i])
                          : (float)static_cast<const _Float16*>(p)[i];
}
__device__ __forceinline__ void load8_any(const void* p, int dtype, int col, int cols,
                                          float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.0f;
  } else if (dtype == kF32) {
    load8<kF32>(static_cast<const float*>(p), col, cols, v);
  } else if (dtype == kBF16) {
    load8<kBF16>(static_cast<const __bf16*>(p), col, cols, v);
  } else {
    load8<kF16>(static_cast<const _Float16*>(p), col, cols, v);
  }
}

// A fp32 value rounded to the type, nearest even.  For fp16 the value is made opaque first: the
// compiler otherwise joins a product and its conversion into one instruction that rounds once,
// and the stored value would not be the rounded fp32 product.
template <int DT>
__device__ __forceinline__ typename Elt<DT>::T round_to(float x) {
  if (DT == kF16) asm("" : "+v"(x));
  return (typename Elt<DT>::T)x;
}

// Rounds v to the type and stores the columns below `cols`, non-temporal where kStream.
template <int DT, bool kStream = false>
__device__ __forceinline__ void store8(typename Elt<DT>::T* p, int col, int cols,
                                       const float (&v)[8]) {
  typename Elt<DT>::T raw[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) raw[j] = round_to<DT>(v[j]);
  if (col + 8 <= cols) {
    Raw<DT> r;
    __builtin_memcpy(&r, raw, sizeof r);
#pragma unroll
    for (int i = 0; i < Raw<DT>::kWords; ++i) {
      u4_at_any* q = reinterpret_cast<u4_at_any*>(p + col) + i;
      if (kStream)
        __builtin_nontemporal_store(r.w[i], q);
      else
        *q = r.w[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + j < cols) p[col + j] = raw[j];
  }
}

// Largest of a value over the lane's quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // lanes 1,0,3,2
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // 2,3,0,1
}

// Biased exponent of the group's scale from its largest magnitude's bits: the smallest
// e >= -120 with A <= 127 * 2^e.  With A = f * 2^p and f in [1, 2), e = p - 6 where
// f <= 127/64 (mantissa bits <= 0x7E0000) and p - 5 above it: adding 0x1FFFF carries into the
// exponent just there.  Inf, NaN and anything above 127 * 2^121 give kExpBad.
__device__ __forceinline__ uint32_t group_exponent(uint32_t amax) {
  const uint32_t e = ((amax + 0x1FFFFu) >> 23);
  return e < kExpLowest + 6 ? kExpLowest : e > kExpHighest + 6 ? kExpBad : e - 6;
}

__device__ __forceinline__ float exponent_scale(uint32_t e) { return __uint_as_float(e << 23); }

// The octet's codes (column order = byte order) and its group's exponent.  Every lane of the
// quad calls it.  x * 2^-e is exact, so the code of a value is the same however it was formed:
// rounded to nearest even by adding 1.5 * 2^23, whose unit is 1; or, with kRandom, floor or
// ceiling of the magnitude by the 24-bit draws of blocks `block` and `block + 1` (4 columns each).
// The draw is compared with what the floor leaves in the value's own unit, u * 2^(e - 24) < |x| -
// floor * 2^e, where both sides are exact; |x| / 2^e itself would be 0 where it is below 2^-149.
template <bool kRandom>
__device__ __forceinline__ u2 encode8(const float (&v)[8], uint64_t block, uint32_t seed_lo,
                                      uint32_t seed_hi, uint32_t step_lo, uint32_t* exponent) {
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, mag_key(v[j]));
  const uint32_t e = group_exponent(quad_max(amax));
  *exponent = e;
  uint32_t q[8];
  if (kRandom) {
    uint32_t w[8];
    uint32_t w0[4], w1[4];
    philox4((uint32_t)block, (uint32_t)(block >> 32), step_lo, kActTag, seed_lo, seed_hi, w0);
    ++block;
    philox4((uint32_t)block, (uint32_t)(block >> 32), step_lo, kActTag, seed_lo, seed_hi, w1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = w0[j] >> 8;
      w[4 + j] = w1[j] >> 8;
    }
    const float inv = __uint_as_float((254u - min(e, kExpHighest)) << 23);
    const float scale = exponent_scale(min(e, kExpHighest)), unit = scale * 0x1p-24f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = floorf(fabsf(v[j]) * inv);
      const int m = (int)f + ((float)w[j] * unit < fmaf(-f, scale, fabsf(v[j])) ? 1 : 0);
      q[j] = (uint32_t)(signbit(v[j]) ? -m : m);
    }
  } else {
    const float inv = __uint_as_float((254u - min(e, kExpHighest)) << 23);
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __float_as_uint(v[j] * inv + 12582912.0f);
  }
  u2 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t* p = q + 4 * h;
    const uint32_t lo = __builtin_amdgcn_perm(p[1], p[0], 0x0C0C0400);
    const uint32_t hi = __builtin_amdgcn_perm(p[3], p[2], 0x0C0C0400);
    r[h] = lo | (hi << 16);
  }
  return e == kExpBad ? u2{0, 0} : r;
}

// code * scale for 8 codes, exact (7 bits and a sign times a power of two).  u = 127 - code is a byte
// (the code's low 7 bits flipped), which one instruction makes a float, and 127 * scale - u * scale
// rounds nothing: 127 times the largest scale is finite.  For a bad group it is Inf - Inf, the NaN
// that it stands for.
__device__ __forceinline__ void decode8(u2 c, float scale, float (&v)[8]) {
  const float top = 127.0f * scale;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u = c[h] ^ 0x7F7F7F7Fu;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * h + j] = fmaf((float)((u >> (8 * j)) & 0xFFu), -scale, top);
  }
}

// A value from another lane of the row of 16 (DPP control word), for 4- and 8-byte types.
template <int kCtrl, typename S>
__device__ __forceinline__ S from_lane(S v) {
  int w[sizeof(S) / 4];
  __builtin_memcpy(w, &v, sizeof v);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(S) / 4); ++i)
    w[i] = __builtin_amdgcn_mov_dpp(w[i], kCtrl, 0xF, 0xF, true);
  __builtin_memcpy(&v, w, sizeof v);
  return v;
}
template <typename S>
__device__ __forceinline__ S read_lane(S v, int lane) {
  int w[sizeof(S) / 4];
  __builtin_memcpy(w, &v, sizeof v);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(S) / 4); ++i) w[i] = __builtin_amdgcn_readlane(w[i], lane);
  __builtin_memcpy(&v, w, sizeof v);
  return v;
}
// Sum over the wave's 64 lanes, all active, in a fixed order: neighbours, pairs, halves of a row
// of 16, its two halves, then the four rows.
template <typename S>
__device__ __forceinline__ S wave_sum(S v) {
  v += from_lane<0xB1>(v);    // lane ^ 1
  v += from_lane<0x4E>(v);    // lane ^ 2
  v += from_lane<0x141>(v);   // mirrored in the half row
  v += from_lane<0x140>(v);   // mirrored in the row
  return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}

// How the writers and readers of whole rows spread octets over waves: a row has `octets`
// octets; rows of fewer than 64 share a wave (64 / lanes rows of `lanes` lanes, a power of two of
// at least 4), longer ones take `chunks` wave units of 64 octets each.
struct RowMap {
  int64_t rows, units;   // wave units in all
  int32_t cols, octets, chunks, lanes;
};

}  // namespace
}  // namespace gc
