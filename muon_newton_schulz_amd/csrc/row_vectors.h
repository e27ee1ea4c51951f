// Pieces of a row of bfloat16 or float32, at any alignment of the type and cut at the row's end.
#pragma once
#include "lds_dma.h"

namespace mns {
namespace {

// 16 bytes from any address of T's alignment, of which the first `valid` elements exist; the
// others read as zero and are not touched. (A whole chunk is one 16-byte load: this part loads
// from any address.) For the end of a buffer: a partial chunk is read element by element and waited for.
template <typename T>
__device__ __forceinline__ u32x4 load_chunk(const T* p, int valid) {
  constexpr int VEC = 16 / sizeof(T);
  u32x4 v = {0u, 0u, 0u, 0u};
  if (valid >= VEC) {
    __builtin_memcpy(&v, p, 16);
  } else if (valid > 0) {
    T e[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = i < valid ? p[i] : (T)0.f;
    __builtin_memcpy(&v, e, 16);
  }
  return v;
}

// The same for a piece of a row of a larger buffer that ends at `end`: one 16-byte load wherever the buffer
// has that much left, so that a partial chunk costs no wait of its own (input gradient of 1021 rows, 5
// experts of 513 x 1277, bfloat16: 23.6 -> 22.7 us). The elements behind the first `valid` are then
// whatever follows in the buffer: unspecified.
template <typename T, bool STREAM = false>
__device__ __forceinline__ u32x4 load_piece_of_row(const T* p, int valid, const T* end);

// Zeros behind the first `valid` elements.
template <typename T>
__device__ __forceinline__ u32x4 cut_chunk(u32x4 v, int valid) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    if constexpr (sizeof(T) == 4)
      v[d] = d < valid ? v[d] : 0u;
    else
      v[d] = 2 * d + 1 < valid ? v[d] : 2 * d < valid ? v[d] & 0xFFFFu : 0u;
  }
  return v;
}

// The same 16 bytes past the caches, for calls whose data does not fit the 256 MB last-level cache.
constexpr double kStreamBytes = double(256 << 20);
typedef u32x4 u32x4_any __attribute__((aligned(2)));
template <typename T>
__device__ __forceinline__ u32x4 load_streaming(const T* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}
template <typename T>
__device__ __forceinline__ void store_streaming(T* p, const void* v) {
  u32x4 x;
  __builtin_memcpy(&x, v, 16);
  __builtin_nontemporal_store(x, reinterpret_cast<u32x4_any*>(p));
}

template <typename T, bool STREAM>
__device__ __forceinline__ u32x4 load_piece_of_row(const T* p, int valid, const T* end) {
  constexpr int VEC = 16 / sizeof(T);
  u32x4 v = {0u, 0u, 0u, 0u};
  if (valid > 0) {
    if (p + VEC <= end) {
      if (STREAM) v = load_streaming(p);
      else __builtin_memcpy(&v, p, 16);
    } else {
      v = load_chunk(p, valid);
    }
  }
  return v;
}

// Eight consecutive elements of a row; load() leaves those behind `valid` unspecified.
template <typename T>
struct Eight {
  static constexpr int VEC = 16 / sizeof(T);
  u32x4 r[sizeof(T) / 2];
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const T* p, int valid, const T* end) {
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h)
      r[h] = load_piece_of_row<T, STREAM>(p + h * VEC, valid - h * VEC, end);
  }
  template <bool STREAM = false>
  __device__ __forceinline__ void store(T* p, int valid) const {
    T e[8];
    __builtin_memcpy(e, r, sizeof(e));
#pragma unroll
    for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
      if (STREAM && valid >= (h + 1) * VEC) {
        store_streaming(p + h * VEC, &r[h]);
      } else if (valid >= (h + 1) * VEC) {
        __builtin_memcpy(p + h * VEC, &r[h], 16);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (h * VEC + i < valid) p[h * VEC + i] = e[h * VEC + i];
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    T e[8];
    __builtin_memcpy(e, r, sizeof(e));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)e[i];
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = (T)v[i];
    __builtin_memcpy(r, e, sizeof(e));
  }
};

}  // namespace
}  // namespace mns
