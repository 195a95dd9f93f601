// kvc_cache_device.h -- device helpers shared by the kernels of the resident
// 8-bit cache: which sequence a work unit belongs to, code and type
// conversions, wave-wide reductions.
#pragma once

#include "kvc_arch.h"
#include "kvc_cache.h"

namespace kvc {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t C_FP8 = KVC_FP8_DYNAMIC, C_INT8 = KVC_INT8;

// ------------------------------------------------------------------ batch
struct Seq {
  uint32_t b;             // sequence
  uint32_t unit;          // the unit's number within it
  int r0, n, len, start;  // rows [r0, r0 + n) are positions [start, len); start may be negative
  bool ok;                // its rows and its length are within the batch's bounds
};

__device__ __forceinline__ void flag_seq(const BatchView& b, uint32_t seq, uint32_t bit) {
  if (b.flags && (threadIdx.x & 63) == 0) atomicOr(b.flags + seq, bit);
}

__device__ __forceinline__ void load_seq(const BatchView& v, uint32_t b, Seq& s) {
  // the wave's own values: what follows from them stays scalar
  const int r0 = __builtin_amdgcn_readfirstlane(v.cu[b]), r1 = __builtin_amdgcn_readfirstlane(v.cu[b + 1]),
            len = __builtin_amdgcn_readfirstlane(v.lengths[b]);
  s.b = b;
  s.r0 = r0;
  s.n = r1 - r0;
  s.len = len;
  s.start = len - s.n;
  s.ok = r0 >= 0 && r1 >= r0 && (uint32_t)r1 <= v.n_rows && (uint32_t)(r1 - r0) <= v.max_rows && len >= 0 &&
         (uint32_t)len <= v.max_len;
}

// The sequence of unit u.  With per_seq units for every sequence it is a
// division; else sequence b's units begin at cu[b] * unit_mul / unit_div +
// b * unit_add, which leaves each sequence the units it needs (unit_add
// covers what the floors cut off), and the wave finds b by a 64-ary search:
// every step is one load a lane, two steps up to 4096 sequences.  Sequence
// numbers stay below n_seqs whatever cu holds.
__device__ __forceinline__ Seq seq_of_unit(const BatchView& v, uint32_t u) {
  Seq s;
  if (v.per_seq) {
    const uint32_t b = u / v.per_seq;
    load_seq(v, b, s);
    s.unit = u - b * v.per_seq;
  } else {
    const uint32_t lane = threadIdx.x & 63;
    auto first = [&v](uint32_t b) {
      const uint32_t r = (uint32_t)min(max(v.cu[b], 0), (int)v.n_rows);
      return (uint32_t)((uint64_t)r * v.unit_mul / v.unit_div) + b * v.unit_add;
    };
    uint32_t lo = 0, n = v.n_seqs;
    while (n > 1) {
      const uint32_t step = (n + 63) / 64, at = lane * step;
      const bool below = at < n && first(lo + min(at, n - 1)) <= u;
      const uint32_t cnt = max((uint32_t)__popcll(__ballot(below)), 1u);
      lo += (cnt - 1) * step;
      n = min(step, n - (cnt - 1) * step);
    }
    lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)lo);
    load_seq(v, lo, s);
    const uint32_t f = first(lo);
    s.unit = u - f;
    s.ok = s.ok && u >= f;
    if (u < v.n_seqs) {   // a unit for every sequence, to report the bad ones
      Seq t;
      load_seq(v, u, t);
      if (!t.ok) flag_seq(v, u, KVC_SEQ_BAD_RANGE);
    }
  }
  if (!s.ok) flag_seq(v, s.b, KVC_SEQ_BAD_RANGE);
  return s;
}

// ------------------------------------------------------------------ conversions
template <int DT>
__device__ __forceinline__ f32x2 unpack2(uint32_t w) {
  if constexpr (DT == KVC_BF16) {
    f32x2 r = {__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
    return r;
  } else {
    return __builtin_convertvector(__builtin_bit_cast(f16x2, w), f32x2);
  }
}
// two floats -> packed pair, round to nearest even
template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  f32x2 v = {a, b};
  if constexpr (DT == KVC_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}
// |x| bits of a 16-bit value at or above this: infinity or NaN
template <int DT>
constexpr uint32_t kNonfinite = DT == KVC_BF16 ? 0x7F80u : 0x7C00u;

// four quotients -> four codes; NaN becomes 0, larger magnitudes the largest code
template <uint32_t CODEC>
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d) {
  float x[4] = {a, b, c, d};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float top = CODEC == C_FP8 ? 448.0f : 127.0f;
    x[i] = x[i] == x[i] ? x[i] : 0.0f;
    if constexpr (CODEC == C_INT8) x[i] = rintf(x[i]);
    x[i] = fminf(fmaxf(x[i], -top), top);
  }
  if constexpr (CODEC == C_FP8) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
  } else {
    return ((uint32_t)(int)x[0] & 0xFFu) | (((uint32_t)(int)x[1] & 0xFFu) << 8) |
           (((uint32_t)(int)x[2] & 0xFFu) << 16) | ((uint32_t)(int)x[3] << 24);
  }
}
// the value of code byte I of w
template <uint32_t CODEC, int I>
__device__ __forceinline__ float code_f32(uint32_t w) {
  if constexpr (CODEC == C_FP8) return __builtin_amdgcn_cvt_f32_fp8((int)w, I);
  else return (float)((int)(w << (24 - 8 * I)) >> 24);
}
template <uint32_t CODEC>
__device__ __forceinline__ void codes4(uint32_t w, float* x) {
  x[0] = code_f32<CODEC, 0>(w);
  x[1] = code_f32<CODEC, 1>(w);
  x[2] = code_f32<CODEC, 2>(w);
  x[3] = code_f32<CODEC, 3>(w);
}

// ------------------------------------------------------------------ wave reductions
// partners of lane ^ 16 and lane ^ 32 (row swaps, no LDS)
__device__ __forceinline__ float max_across_groups(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float y = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(y), __float_as_uint(y), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_across_groups(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const float y = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(y), __float_as_uint(y), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
__device__ __forceinline__ float wave_fmax(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = fmaxf(v, __shfl_xor(v, m));
  return v;
}
__device__ __forceinline__ float wave_fsum(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}

}  // namespace kvc
