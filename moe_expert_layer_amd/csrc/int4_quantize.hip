// 4-bit weights with a scale, and on demand a zero point, for each group of G consecutive ones of a row: quantisation of
// bf16 / f16 / f32 rows and the values back.
//
// With l the group's least value or 0 and h its largest or 0:  s = max(-l, h) / 7, q = round(v / s) + 8 in
// [0, 15]; or s = (h - l) / 15, z = round(-l / s), q = round(v / s) + z in [0, 15].  s is the float32 quotient rounded to the
// scales' type, and codes are rounded by the exact quotient by that s, ties to even, so results are fully determined: v
// times the reciprocal is at most 4e-6 off the quotient, and where that could change the rounding the remainder
// v - q s, which float32 holds exactly there, decides.
//
// Both directions are bound by HBM.  A lane takes 8 values (one or two 16-byte loads) and leaves 4 bytes of codes; 4, 8 or
// 16 lanes hold a group of 32, 64 or 128.  Larger groups are walked 128 values at a time by 16 lanes, twice, the second
// time from the caches.  16384 x 7168 float32 values with groups of 128 and zero points, and
// back to bf16: 158 to 167 us for the two (109 and 57 traced), 156 at a copy's rate, values read once and values written going past the caches
// (182 us through them).
#include <hip/hip_runtime.h>
#include <cstdint>

#include "device_common.hpp"
#include "elem.hpp"
#include "operators.hpp"

namespace moe {

namespace {

// 16 bytes that are read or written once, past the caches
template <typename T>
__device__ __forceinline__ void store_past(T* p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<typename Aligned<sizeof(T)>::type*>(p));
}
template <bool ONCE, typename T>
__device__ __forceinline__ u32x4 load16_of(const T* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const typename Aligned<sizeof(T)>::type*>(p));
  else return load16(p);
}

template <bool ONCE, typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    const u32x4 a = load16_of<ONCE>(p), b = load16_of<ONCE>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __uint_as_float(a[i]);
      f[4 + i] = __uint_as_float(b[i]);
    }
  } else {
    Elem<T>::unpack(load16_of<ONCE>(p), f);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, false));
}
// f over the LG lanes of a group, the result in each of them
template <int LG, typename F>
__device__ __forceinline__ float over_lanes(float v, F f) {
  v = f(v, dpp<0xB1>(v));                       // quad_perm [1,0,3,2]
  v = f(v, dpp<0x4E>(v));                       // quad_perm [2,3,0,1]
  if constexpr (LG >= 8) v = f(v, dpp<0x141>(v));   // row_half_mirror
  if constexpr (LG >= 16) v = f(v, dpp<0x140>(v));  // row_mirror
  return v;
}

// scales of any of the three types (0 bf16, 1 f16, 2 f32)
__device__ __forceinline__ float scale_get(const void* p, long long i, int dtype) {
  if (dtype == 2) return static_cast<const float*>(p)[i];
  const uint16_t b = static_cast<const uint16_t*>(p)[i];
  return dtype == 0 ? Elem<Bf16>::get(Bf16{b}) : Elem<F16>::get(F16{b});
}
__device__ __forceinline__ float scale_round(float s, int dtype) {
  if (dtype == 2) return s;
  return dtype == 0 ? Elem<Bf16>::get(Elem<Bf16>::put(s)) : Elem<F16>::get(Elem<F16>::put(s));
}
__device__ __forceinline__ void scale_put(void* p, long long i, int dtype, float s) {
  if (dtype == 2) static_cast<float*>(p)[i] = s;
  else if (dtype == 0) static_cast<Bf16*>(p)[i] = Elem<Bf16>::put(s);
  else static_cast<F16*>(p)[i] = Elem<F16>::put(s);
}

// round(v / s), ties to even, for s > 0 and |v / s| < 32 (15 and, where s is a subnormal float16, up to half more), inv
// being 1 / s rounded.  v inv is off by less than 32 * 2^-23 = 2^-18; v - q s, at most s and a multiple of the smaller
// of the two units, is exact.
__device__ __forceinline__ float nearest(float v, float s, float inv) {
  const float r = v * inv;
  float q = rintf(r);
  if (fabsf(r - q) > 0.5f - 0x1p-17f) {
    const float t = 2.f * fmaf(-q, s, v);
    const bool odd = ((int)q & 1) != 0;
    if (t > s || (t == s && odd)) q += 1.f;
    else if (t < -s || (t == -s && odd)) q -= 1.f;
  }
  return q;
}

// How a group's values become codes
struct Coder {
  float s, inv, up;  // up: a power of two that brings a tiny scale and its values into the range of 1 / s
  float lo, hi;
  float scale;             // as stored
  int z;
  bool some;               // the scale is a positive number; else every code is that of 0
  __device__ __forceinline__ void set(float l, float h, float bad, int sdt, bool zeros) {
    scale = zeros ? (float)(((double)h - (double)l) / 15.0) : fmaxf(-l, h) / 7.f;
    scale = scale_round(scale, sdt);
    if (bad != 0.f || !(scale < INFINITY)) scale = __uint_as_float(0x7fc00000u);
    some = scale > 0.f;
    up = scale < 0x1p-100f ? 0x1p100f : 1.f;
    s = some ? scale * up : 1.f;
    inv = 1.f / s;
    z = zeros ? (int)fminf(fmaxf(nearest(-l * up, s, inv), 0.f), 15.f) : 8;
    if (!some && zeros) z = 0;
    lo = (float)-z;
    hi = (float)(15 - z);
  }
  __device__ __forceinline__ uint32_t code(float v) const {
    return (uint32_t)((int)fminf(fmaxf(nearest(v * up, s, inv), lo), hi) + z);
  }
};

// grid-stride over the groups of all rows, LG lanes on each; MULTI: groups of several times 128
template <typename T, int LG, bool MULTI>
__global__ __launch_bounds__(256) void quantize_int4_kernel(const T* __restrict__ src, long long stride, long long ngroups,
                                                            int K, int G, int per_row, int sdt, uint8_t* __restrict__ codes,
                                                            void* __restrict__ scales, uint8_t* __restrict__ zeros) {
  constexpr int GW = 64 / LG;  // groups of a wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int off = lane / LG, l8 = (lane & (LG - 1)) * 8;
  const int steps = MULTI ? G / 128 : 1;
  for (long long g0 = ((long long)blockIdx.x * 4 + wave) * GW; g0 < ngroups; g0 += (long long)gridDim.x * 4 * GW) {
    // the wave's first group by one long division, the others from there
    const long long r0 = g0 / per_row;
    const unsigned at = (unsigned)(g0 - r0 * per_row) + off;
    const long long r = r0 + at / (unsigned)per_row;
    const int g = (int)(at % (unsigned)per_row);
    const bool live = g0 + off < ngroups;
    const T* p = src + (live ? r * stride + (long long)g * G : 0) + l8;
    float f[8], l = 0.f, h = 0.f, bad = 0.f;
    for (int i = 0; i < steps; ++i) {
      load8<!MULTI>(p + (live ? i * 128 : 0), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        l = fminf(l, f[j]);
        h = fmaxf(h, f[j]);
        bad = fmaf(f[j], 0.f, bad);  // NaN from an infinity or a NaN
      }
    }
    l = over_lanes<LG>(l, [](float a, float b) { return fminf(a, b); });
    h = over_lanes<LG>(h, [](float a, float b) { return fmaxf(a, b); });
    bad = over_lanes<LG>(bad, [](float a, float b) { return a + b; });
    Coder c;
    c.set(l, h, bad, sdt, zeros != nullptr);
    if (!live) continue;
    const long long row_at = r * (K / 2) + (long long)g * (G / 2) + l8 / 2;
    for (int i = 0; i < steps; ++i) {
      if constexpr (MULTI) load8<false>(p + i * 128, f);
      uint32_t q = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) q |= c.code(f[j]) << (4 * j);
      *reinterpret_cast<uint32_t*>(codes + row_at + i * 64) = c.some ? q : 0x11111111u * c.z;
    }
    if (l8 == 0) {
      const long long k = r * per_row + g;
      scale_put(scales, k, sdt, c.scale);
      if (zeros != nullptr) zeros[k] = (uint8_t)c.z;
    }
  }
}

// grid-stride over 8-value chunks of all rows
template <typename T>
__global__ __launch_bounds__(256) void dequantize_int4_kernel(const uint8_t* __restrict__ codes,
                                                              const void* __restrict__ scales,
                                                              const uint8_t* __restrict__ zeros, long long nchunks, int K,
                                                              int G, int sdt, T* __restrict__ dst, long long stride) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned per_row = K / 8, per_group = G / 8, groups = K / G;
  for (long long c0 = ((long long)blockIdx.x * 4 + wave) * 64; c0 < nchunks; c0 += (long long)gridDim.x * 256) {
    const long long r0 = c0 / per_row;
    const unsigned at = (unsigned)(c0 - r0 * per_row) + lane;
    const long long r = r0 + at / per_row;
    const unsigned c = at % per_row;
    if (c0 + lane >= nchunks) continue;
    const uint32_t q = reinterpret_cast<const uint32_t*>(codes)[c0 + lane];
    const long long k = r * groups + c / per_group;
    const float s = scale_get(scales, k, sdt);
    const int z = zeros != nullptr ? zeros[k] : 8;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f[j] = (float)((int)((q >> (4 * j)) & 15u) - z) * s;
      asm("" : "+v"(f[j]));  // a float32 product: with a float16 result the compiler would round once, by another instruction
    }
    T* p = dst + r * stride + (long long)c * 8;
    if constexpr (sizeof(T) == 4) {
      store_past(p, __builtin_bit_cast(u32x4, (v4f{f[0], f[1], f[2], f[3]})));
      store_past(p + 4, __builtin_bit_cast(u32x4, (v4f{f[4], f[5], f[6], f[7]})));
    } else {
      store_past(p, pack16<T>(f));
    }
  }
}

unsigned grid_of(long long waves) {
  const long long n = (waves + 3) / 4;
  return (unsigned)(n < (1 << 20) ? n : (1 << 20));
}

template <typename T>
hipError_t quantize(const Int4Shape& d, const void* src, uint8_t* codes, void* scales, uint8_t* zeros, hipStream_t s) {
  const int per_row = d.K / d.G;
  const long long n = (long long)d.M * per_row;
  const auto launch = [&](auto kern, int groups_per_wave) {
    kern<<<grid_of((n + groups_per_wave - 1) / groups_per_wave), 256, 0, s>>>(
        static_cast<const T*>(src), d.stride, n, d.K, d.G, per_row, d.scale_dtype, codes, scales, d.zeros ? zeros : nullptr);
    return hipGetLastError();
  };
  if (d.G == 32) return launch(quantize_int4_kernel<T, 4, false>, 16);
  if (d.G == 64) return launch(quantize_int4_kernel<T, 8, false>, 8);
  if (d.G == 128) return launch(quantize_int4_kernel<T, 16, false>, 4);
  return launch(quantize_int4_kernel<T, 16, true>, 4);
}

template <typename T>
hipError_t dequantize(const Int4Shape& d, const uint8_t* codes, const void* scales, const uint8_t* zeros, void* dst,
                      hipStream_t s) {
  const long long n = (long long)d.M * (d.K / 8);
  dequantize_int4_kernel<T><<<grid_of((n + 63) / 64), 256, 0, s>>>(codes, scales, d.zeros ? zeros : nullptr, n, d.K, d.G,
                                                                  d.scale_dtype, static_cast<T*>(dst), d.stride);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_int4(const Int4Shape& d, const void* src, uint8_t* codes, void* scales, uint8_t* zeros,
                                hipStream_t s) {
  if (d.dtype == 0) return quantize<Bf16>(d, src, codes, scales, zeros, s);
  if (d.dtype == 1) return quantize<F16>(d, src, codes, scales, zeros, s);
  return quantize<float>(d, src, codes, scales, zeros, s);
}

hipError_t launch_dequantize_int4(const Int4Shape& d, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                                  void* dst, hipStream_t s) {
  if (d.dtype == 0) return dequantize<Bf16>(d, codes, scales, zeros, dst, s);
  if (d.dtype == 1) return dequantize<F16>(d, codes, scales, zeros, dst, s);
  return dequantize<float>(d, codes, scales, zeros, dst, s);
}

}  // namespace moe
