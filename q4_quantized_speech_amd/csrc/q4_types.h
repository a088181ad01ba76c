// Element types of the adapter operators' activations and parameters: float32,
// binary16 and bfloat16 in memory, float32 in registers.  A store rounds once,
// to nearest even.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_device.h"

namespace q4 {

// Codes of the ABI's element types (the numbers GGUF uses).
constexpr int TYPE_F32 = 0, TYPE_F16 = 1, TYPE_BF16 = 30;

inline bool type_ok(int t) { return t == TYPE_F32 || t == TYPE_F16 || t == TYPE_BF16; }
inline int type_bytes(int t) { return t == TYPE_F32 ? 4 : 2; }

// f called with a value of the type's C++ type.
template <typename F>
void with_type(int t, F f) {
  if (t == TYPE_F32) f(float{});
  else if (t == TYPE_F16) f(_Float16{});
  else f(__bf16{});
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return static_cast<float>(v); }
__device__ __forceinline__ float to_f32(__bf16 v) { return static_cast<float>(v); }

// V consecutive elements at p (p aligned to V elements), as float32.
template <int V, typename T>
__device__ __forceinline__ void load_f32(const T* p, float (&v)[V]) {
  typedef T vec __attribute__((ext_vector_type(V)));
  const vec a = *reinterpret_cast<const vec*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = to_f32(static_cast<T>(a[i]));
}

// V consecutive elements at any element address (the hardware takes vector
// accesses of any alignment in global memory).
template <int V, typename T>
__device__ __forceinline__ auto load_any(const T* p) {
  typedef T vec __attribute__((ext_vector_type(V)));
  typedef T loose __attribute__((ext_vector_type(V), aligned(sizeof(T))));
  const loose a = *reinterpret_cast<const loose*>(p);
  return static_cast<vec>(a);
}
template <int V, typename T>
__device__ __forceinline__ void load_any_f32(const T* p, float (&v)[V]) {
  const auto a = load_any<V>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = to_f32(static_cast<T>(a[i]));
}

template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  return static_cast<T>(v);
}

// V consecutive elements at p (aligned to V elements), each rounded once.
template <int V, typename T>
__device__ __forceinline__ void store_f32(T* p, const float (&v)[V]) {
  typedef T vec __attribute__((ext_vector_type(V)));
  vec a;
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = from_f32<T>(v[i]);
  *reinterpret_cast<vec*>(p) = a;
}

// ... to any element address.
template <int V, typename T>
__device__ __forceinline__ void store_any_f32(T* p, const float (&v)[V]) {
  typedef T loose __attribute__((ext_vector_type(V), aligned(sizeof(T))));
  loose a;
#pragma unroll
  for (int i = 0; i < V; ++i) a[i] = from_f32<T>(v[i]);
  *reinterpret_cast<loose*>(p) = a;
}

}  // namespace q4
