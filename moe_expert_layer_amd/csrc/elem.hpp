// Tensor element types of the operators beside the layer: bfloat16, float16, float32.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace moe {

// 16 bytes of a row at the alignment of its elements: the hardware takes any alignment, the type
// tells the compiler not to assume 16 bytes (odd row lengths and strides)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <int A> struct Aligned;
template <> struct Aligned<1> { typedef u32x4 type __attribute__((aligned(1))); };
template <> struct Aligned<2> { typedef u32x4 type __attribute__((aligned(2))); };
template <> struct Aligned<4> { typedef u32x4 type __attribute__((aligned(4))); };
template <typename T>
__device__ __forceinline__ u32x4 load16(const T* p) { return *reinterpret_cast<const typename Aligned<sizeof(T)>::type*>(p); }
template <typename T>
__device__ __forceinline__ void store16(T* p, u32x4 v) { *reinterpret_cast<typename Aligned<sizeof(T)>::type*>(p) = v; }

struct Bf16 { uint16_t b; };
struct F16 { uint16_t b; };

template <typename T> struct Elem;  // kVec: elements of a 16-byte chunk
template <> struct Elem<Bf16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(Bf16 v) { return __uint_as_float((uint32_t)v.b << 16); }
  static __device__ __forceinline__ Bf16 put(float f) {
    return Bf16{__builtin_bit_cast(uint16_t, (__bf16)f)};  // round to nearest even
  }
  static __device__ __forceinline__ void unpack(u32x4 w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Elem<F16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ float get(F16 v) { return (float)__builtin_bit_cast(_Float16, v.b); }
  static __device__ __forceinline__ F16 put(float f) { return F16{__builtin_bit_cast(uint16_t, (_Float16)f)}; }
  static __device__ __forceinline__ void unpack(u32x4 w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = get(F16{(uint16_t)(w[i] & 0xffffu)});
      f[2 * i + 1] = get(F16{(uint16_t)(w[i] >> 16)});
    }
  }
};
template <> struct Elem<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float f) { return f; }
  static __device__ __forceinline__ void unpack(u32x4 w, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  }
};

template <typename T>
__device__ __forceinline__ u32x4 pack16(const float (&f)[Elem<T>::kVec]) {
  T v[Elem<T>::kVec];
#pragma unroll
  for (int i = 0; i < Elem<T>::kVec; ++i) v[i] = Elem<T>::put(f[i]);
  return __builtin_bit_cast(u32x4, v);
}

}  // namespace moe
