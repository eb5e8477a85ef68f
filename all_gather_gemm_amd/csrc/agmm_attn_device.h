// Device code shared by the kernels of agmm_attn.h.
#pragma once

#include <type_traits>

#include "agmm_attn_internal.h"

namespace agmm {
namespace {

typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef __bf16 b8_t __attribute__((ext_vector_type(8)));
typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// 16 bytes at any 2-byte address: one global_load / store_dwordx4, which the hardware serves at
// any alignment
typedef u32x4 u32x4_any __attribute__((aligned(2)));

__device__ inline uint32_t operator/(uint32_t n, const FastDiv& f) {
  return (__umulhi(f.mul, n) + n) >> f.shift;
}

// Bytes from the pools' starts (of one head) to a row, and to its scales.
__device__ inline int64_t row_at(const CacheView& c, uint32_t page, uint32_t row) {
  return (int64_t)((uint64_t)page * c.page + (uint64_t)row * c.row);
}
__device__ inline int64_t scales_at(const CacheView& c, uint32_t page, uint32_t row) {
  return (int64_t)((uint64_t)page * c.s_page + (uint64_t)row * c.s_row);
}

__device__ inline u32x4 load16(const uint16_t* p) {
  return *reinterpret_cast<const u32x4_any*>(p);
}
__device__ inline void store16(uint16_t* p, u32x4 v) { *reinterpret_cast<u32x4_any*>(p) = v; }

// The 16-bit types: the values of a packed pair, and two floats rounded (RNE) to a packed pair.
//
// split: two floats >= 0 as a pair cut to the type and a pair of what that leaves, 22 bits (fp16) or 16
// (bf16) of each together. What is left is kept above 0 (at the type's least power of 2 that matrix
// instructions take, or the number itself if that is less): as a factor of an infinite value 0 would
// make the sum of the two products NaN.
template <int DT>
struct T16;

template <>
struct T16<AGMM_F16> {
  __device__ static inline float lo(uint32_t w) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
  }
  __device__ static inline float hi(uint32_t w) { return lo(w >> 16); }
  __device__ static inline uint32_t pack(float a, float b) {
    h2_t v;
    v.x = (_Float16)a;
    v.y = (_Float16)b;
    return __builtin_bit_cast(uint32_t, v);
  }
  __device__ static inline u32x2 split(float a, float b) {
    const uint32_t cut = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(a, b));
    return u32x2{cut, pack(__builtin_amdgcn_fmed3f(a - lo(cut), 0x1p-24f, a),
                           __builtin_amdgcn_fmed3f(b - hi(cut), 0x1p-24f, b))};
  }
  __device__ static inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8_t, a),
                                                  __builtin_bit_cast(h8_t, b), c, 0, 0, 0);
  }
  // two codes times 2^(exponent of s - 127), exact
  template <int HALF>
  __device__ static inline uint32_t from_fp8(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, s, HALF));
  }
  template <int BYTE>
  __device__ static inline uint32_t from_fp4(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, s, BYTE));
  }
};

template <>
struct T16<AGMM_BF16> {
  __device__ static inline float lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
  __device__ static inline float hi(uint32_t w) {
    return __builtin_bit_cast(float, w & 0xffff0000u);
  }
  __device__ static inline uint32_t pack(float a, float b) {
    b2_t v;
    v.x = (__bf16)a;
    v.y = (__bf16)b;
    return __builtin_bit_cast(uint32_t, v);
  }
  __device__ static inline u32x2 split(float a, float b) {
    const uint32_t cut = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b),
                                               __builtin_bit_cast(uint32_t, a), 0x07060302u);
    return u32x2{cut, pack(__builtin_amdgcn_fmed3f(a - lo(cut), 0x1p-126f, a),
                           __builtin_amdgcn_fmed3f(b - hi(cut), 0x1p-126f, b))};
  }
  __device__ static inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8_t, a),
                                                   __builtin_bit_cast(b8_t, b), c, 0, 0, 0);
  }
  template <int HALF>
  __device__ static inline uint32_t from_fp8(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, HALF));
  }
  template <int BYTE>
  __device__ static inline uint32_t from_fp4(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, BYTE));
  }
};

// The scale that byte s (0..255) stands for, as the conversions above take it: only the exponent
// field counts, and 255 in it makes every value NaN.
__device__ inline float scale_of(uint32_t s) {
  return __builtin_bit_cast(float, s << 23);
}

// 8 codes (fp8: two words, fp4: one) as 8 packed 16-bit values.
template <int DT>
__device__ inline u32x4 from_fp8x8(uint32_t w0, uint32_t w1, float s) {
  u32x4 r;
  r[0] = T16<DT>::template from_fp8<0>(w0, s);
  r[1] = T16<DT>::template from_fp8<1>(w0, s);
  r[2] = T16<DT>::template from_fp8<0>(w1, s);
  r[3] = T16<DT>::template from_fp8<1>(w1, s);
  return r;
}
template <int DT>
__device__ inline u32x4 from_fp4x8(uint32_t w, float s) {
  u32x4 r;
  r[0] = T16<DT>::template from_fp4<0>(w, s);
  r[1] = T16<DT>::template from_fp4<1>(w, s);
  r[2] = T16<DT>::template from_fp4<2>(w, s);
  r[3] = T16<DT>::template from_fp4<3>(w, s);
  return r;
}

}  // namespace
}  // namespace agmm
