// Rows in chunks of 16 bytes at any alignment (layer norm, SwiGLU): loads, stores, and the decoding of MXFP8
// codes. The hardware takes 16-byte accesses at any address; only the chunk in which a row ends needs care.
#pragma once
#include "mx_device.h"

namespace mxf {

__device__ __forceinline__ uint32_t bits_of(uint16_t v) { return v; }
__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }

template <class T>
struct Elem;
template <>
struct Elem<uint16_t> {  // BF16 bit patterns
  static constexpr int VEC = 8;
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t put(float f) { return (uint16_t)bf16_bits(f); }
  static __device__ __forceinline__ void unpack(u32x4_t v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(v[i]);
      f[2 * i + 1] = bf16_hi(v[i]);
    }
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    return (u32x4_t){bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]), bf16x2_bits(f[4], f[5]), bf16x2_bits(f[6], f[7])};
  }
};
template <>
struct Elem<float> {
  static constexpr int VEC = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float f) { return f; }
  static __device__ __forceinline__ void unpack(u32x4_t v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ u32x4_t pack(const float* f) {
    return (u32x4_t){__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
  }
};

// How rows end: on a whole chunk; inside one; inside their first. TINY, element by element, is right for any width: SwiGLU
// takes it wherever rows do not end on a chunk.
enum Ends { EXACT, INSIDE, TINY };

// v >> bits (bits < 128, per lane) of a 128-bit value.
__device__ __forceinline__ u32x4_t shr128(u32x4_t v, uint32_t bits) {
  const uint32_t b = bits & 31;
  u32x4_t r = {__builtin_amdgcn_alignbit(v[1], v[0], b), __builtin_amdgcn_alignbit(v[2], v[1], b),
               __builtin_amdgcn_alignbit(v[3], v[2], b), v[3] >> b};
  if (bits & 32) r = (u32x4_t){r[1], r[2], r[3], 0};
  if (bits & 64) r = (u32x4_t){r[2], r[3], 0, 0};
  return r;
}

// 16 bytes at column c of a row, without a branch: after one the compiler cannot count the loads in flight and
// waits for all of them. The chunk in which a row ends is loaded from the row's end backwards and shifted where it
// is used (chunk_of); a lane past the end loads one that exists, and is left out or zeroed there. TINY
// goes element by element.
template <class T, Ends E>
__device__ __forceinline__ u32x4_t load_chunk(const T* row, int c, int cols) {
  u32x4_t v = {0, 0, 0, 0};
  const int n = cols - c;
  if constexpr (E == EXACT) {
    __builtin_memcpy(&v, row + (n > 0 ? c : 0), 16);
  } else if constexpr (E == INSIDE) {
    __builtin_memcpy(&v, row + min(c, cols - Elem<T>::VEC), 16);
  } else if (n > 0) {
    uint32_t e[Elem<T>::VEC];
#pragma unroll
    for (int i = 0; i < Elem<T>::VEC; ++i) e[i] = i < n ? bits_of(row[c + i]) : 0u;
    if constexpr (sizeof(T) == 4)
      v = (u32x4_t){e[0], e[1], e[2], e[3]};
    else
      v = (u32x4_t){e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16};
  }
  return v;
}
// The loaded chunk's elements that exist, then zeros; n: elements from column c to the row's end.
template <class T, Ends E>
__device__ __forceinline__ u32x4_t chunk_of(u32x4_t v, int n) {
  if constexpr (E == INSIDE) {
    constexpr int VEC = Elem<T>::VEC;
    if (n < VEC) v = n > 0 ? shr128(v, (uint32_t)(VEC - n) * (128 / VEC)) : (u32x4_t){0, 0, 0, 0};
  }
  return v;
}

// (past the caches' retention: y and dx are larger than the caches when it matters. 16384 x 2048 backward from
// the checkpoint 36 against 39 us, 8192 x 7168 forward 66 against 69; loads gain nothing from it.)
typedef u32x4_t u32x4_any __attribute__((aligned(1)));
template <class T, Ends E>
__device__ __forceinline__ void store_chunk(T* p, const float* f, int n) {
  constexpr int VEC = Elem<T>::VEC;
  if (E == EXACT ? n > 0 : n >= VEC) {
    __builtin_nontemporal_store(Elem<T>::pack(f), reinterpret_cast<u32x4_any*>(p));
  } else if (E != EXACT) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (i < n) p[i] = Elem<T>::put(f[i]);
  }
}

__device__ __forceinline__ uint32_t dpp_half_mirror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false);
}

// The E8M0 scale's value, and a code word's four decoded values (exact: a code has four significant bits).
__device__ __forceinline__ float ckpt_scale(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}
__device__ __forceinline__ float ckpt_value(const uint32_t* k, int i, float sc) {
  const int w = (int)k[i / 4];
  const float f = i % 4 == 0   ? __builtin_amdgcn_cvt_f32_fp8(w, 0)
                  : i % 4 == 1 ? __builtin_amdgcn_cvt_f32_fp8(w, 1)
                  : i % 4 == 2 ? __builtin_amdgcn_cvt_f32_fp8(w, 2)
                               : __builtin_amdgcn_cvt_f32_fp8(w, 3);
  return f * sc;
}

}  // namespace mxf
