// Loads and stores of V neighbouring elements of a row as floats, in one
// access of V elements. The address need only be aligned to an element: global
// accesses of up to 16 bytes may lie anywhere on this GPU (the compiler's
// default for it), so rows of odd widths and offsets take the same path.
// store() is non-temporal (long results that the kernel does not read again: 4%
// faster forward recurrence at 4 x 8192 x 4096), keep() is not (states that the
// next step reads, pieces of cache lines).
#pragma once

#include "common.h"

namespace ret {

template <typename T, int V>
struct Pack;

template <int V>
struct Pack<float, V> {
  typedef float raw __attribute__((ext_vector_type(V)));
  typedef raw anywhere __attribute__((aligned(4)));
  static __device__ __forceinline__ raw load(const float* p) { return *reinterpret_cast<const anywhere*>(p); }
  static __device__ __forceinline__ void unpack(const raw& r, float (&x)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = r[j];
  }
  static __device__ __forceinline__ raw pack(const float (&x)[V]) {
    raw r;
#pragma unroll
    for (int j = 0; j < V; ++j) r[j] = x[j];
    return r;
  }
  static __device__ __forceinline__ raw all(float v) { return raw(v); }
  static __device__ __forceinline__ void store(float* p, const float (&x)[V]) {
    // Eight floats are two accesses, each of which fills half of the lines it
    // touches: these go through the caches (residual norm backward with an
    // fp32 stream, 16384 x 4096: 235 us against 247).
    if constexpr (V == 8) keep(p, x);
    else __builtin_nontemporal_store(pack(x), reinterpret_cast<anywhere*>(p));
  }
  static __device__ __forceinline__ void keep(float* p, const float (&x)[V]) {
    *reinterpret_cast<anywhere*>(p) = pack(x);
  }
};

template <>
struct Pack<float, 1> {
  typedef float raw;
  static __device__ __forceinline__ raw load(const float* p) { return *p; }
  static __device__ __forceinline__ void unpack(const raw& r, float (&x)[1]) { x[0] = r; }
  static __device__ __forceinline__ raw all(float v) { return v; }
  static __device__ __forceinline__ void store(float* p, const float (&x)[1]) { *p = x[0]; }
  static __device__ __forceinline__ void keep(float* p, const float (&x)[1]) { *p = x[0]; }
};

// bf16: V / 2 words of two elements.
template <int V>
struct Pack<uint16_t, V> {
  typedef uint32_t raw __attribute__((ext_vector_type(V / 2)));
  typedef raw anywhere __attribute__((aligned(2)));
  static __device__ __forceinline__ raw load(const uint16_t* p) { return *reinterpret_cast<const anywhere*>(p); }
  static __device__ __forceinline__ void unpack(const raw& r, float (&x)[V]) {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      x[2 * j] = __uint_as_float(r[j] << 16);
      x[2 * j + 1] = __uint_as_float(r[j] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ raw pack(const float (&x)[V]) {
    raw r;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) r[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    return r;
  }
  static __device__ __forceinline__ raw all(float v) { return raw(pack_bf16x2(v, v)); }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&x)[V]) {
    __builtin_nontemporal_store(pack(x), reinterpret_cast<anywhere*>(p));
  }
  static __device__ __forceinline__ void keep(uint16_t* p, const float (&x)[V]) {
    *reinterpret_cast<anywhere*>(p) = pack(x);
  }
};

template <>
struct Pack<uint16_t, 1> {
  typedef uint16_t raw;
  static __device__ __forceinline__ raw load(const uint16_t* p) { return *p; }
  static __device__ __forceinline__ void unpack(const raw& r, float (&x)[1]) { x[0] = bf16_to_f32(r); }
  static __device__ __forceinline__ raw all(float v) { return f32_to_bf16(v); }
  static __device__ __forceinline__ void store(uint16_t* p, const float (&x)[1]) { *p = f32_to_bf16(x[0]); }
  static __device__ __forceinline__ void keep(uint16_t* p, const float (&x)[1]) { *p = f32_to_bf16(x[0]); }
};

}  // namespace ret
