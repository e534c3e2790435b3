// Eight elements of a row per thread, loaded without a branch: a row's last, partly filled
// chunk is read as the eight elements that end with the row, and shifted to its place when
// it is used.  With a branch around a chunk (get_row8) the compiler waits for each before
// it asks for the next.
#pragma once

#include "../layers/rows.hpp"

namespace pgemm {
namespace blocks {

using layers::u32x4;

// As they are stored.
template <typename T>
struct Stored8 {
  u32x4 v[sizeof(T) / 2];
};

// What rows8 hands to its function: chunk c .. c + 7 of the row at `row`, c at most n behind
// the row's end or anywhere beyond it (which gives zeros, once settled).
template <typename T>
struct Window {
  int n;
  __device__ __forceinline__ Stored8<T> operator()(const void* base, long long row, int c) const {
    const T* p = static_cast<const T*>(base) + row + (c <= n - 8 ? c : n - 8);
    Stored8<T> s;
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) s.v[k] = layers::load16(p + k * 16 / sizeof(T));
    return s;
  }
};
template <typename T>
struct Singles {
  int n;
  __device__ __forceinline__ Stored8<T> operator()(const void* base, long long row, int c) const {
    const T* p = static_cast<const T*>(base) + row + c;
    T t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = c + j < n ? p[j] : (T)0.0f;
    Stored8<T> s;
    __builtin_memcpy(&s, t, sizeof(s));
    return s;
  }
};

// f with the load for rows of n elements (the same for the launch; a window needs eight).
template <typename T, typename F>
__device__ __forceinline__ void rows8(int n, F f) {
  if (n >= 8) f(Window<T>{n});
  else f(Singles<T>{n});
}

// The chunk at c in its place, zeros behind the row's end.
template <typename T>
__device__ __forceinline__ void settle8(Stored8<T>& s, int c, int n) {
  if (c <= n - 8 || n < 8) return;
  const int by = c - (n - 8) < 8 ? c - (n - 8) : 8;
  constexpr int PER = 4 / sizeof(T), D = 8 / PER;    // elements of a dword, dwords
  uint32_t x[D];
  __builtin_memcpy(x, &s, sizeof(s));
#pragma unroll
  for (int step = D; step >= 1; step >>= 1)
#pragma unroll
    for (int j = 0; j < D; ++j) {
      const uint32_t from = j + step < D ? x[j + step] : 0;
      if (by / PER & step) x[j] = from;
    }
  if constexpr (PER == 2) {
#pragma unroll
    for (int j = 0; j < D; ++j) {
      const uint32_t from = x[j] >> 16 | (j + 1 < D ? x[j + 1] << 16 : 0);
      if (by & 1) x[j] = from;
    }
  }
  __builtin_memcpy(&s, x, sizeof(s));
}

template <typename T>
__device__ __forceinline__ void widen8(const Stored8<T>& s, float* v) {
  T t[8];
  __builtin_memcpy(t, &s, sizeof(s));
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = (float)t[j];
}

}  // namespace blocks
}  // namespace pgemm
