// Microscaled 4-bit floating point (OCP MX: E2M1 values, one UE8M0 scale per 32 along a row):
// quantisation of bf16 / f16 / f32 rows and the values back.
//
// The scale of a block is 2^e with the smallest integer e such that 6 * 2^e >= amax (6 is E2M1's
// largest value; the rule the layer uses for E4M3 with 448), byte e + 127 clamped to [0, 254], 127 for
// a block of zeros; codes are v * 2^-e rounded to nearest even, so nothing saturates.  E2M1 has no
// NaN: a block with a NaN or an infinity gets scale byte 255 (UE8M0's NaN) and codes 0, and its
// values, and what the matrix cores make of them, are NaN.  Scaling is by a power of two and every
// input is exact in float32, so results are fully determined.
//
// Both directions are bound by HBM (2 to 4 bytes in, 17/32 out per value).  A workgroup takes 512
// columns of 8 rows; a lane 8 values of a row (one or two 16-byte loads), so 4 lanes hold a block
// and its amax is a two-step DPP maximum.  The scale bytes of the tile meet in LDS and leave as
// runs in either layout: words of 8 consecutive rows (packed int32 MN-major), or 16 bytes of a row.
// Measured: 16384 x 7168 float32 quantised in 101 to 107 us (5.0 TB/s; 128 us with 32-row tiles, whose packed
// words fill whole lines but whose waves are half as many; 116 us without the non-temporal loads),
// values back as bfloat16 in 50 to 51 us (5.8 TB/s); 129 x 7168 bfloat16: 3.4 us each.
#include <hip/hip_runtime.h>
#include <cstdint>

#include "device_common.hpp"
#include "elem.hpp"
#include "operators.hpp"

namespace moe {

constexpr int kTileCols = 512, kTileRows = 8;

// amax = 1.m * 2^(E - 127) and 6 = 1.5 * 2^2: e = E - 129 when 1.m <= 1.5, else E - 128
__device__ __forceinline__ int ue8m0_for_amax6(uint32_t amax_bits) {
  if (amax_bits == 0u) return 127;
  if (amax_bits >= 0x7f800000u) return 255;
  const int byte = (int)(amax_bits >> 23) - 2 + ((amax_bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return byte < 0 ? 0 : byte;
}

// 8 consecutive values as float32
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    // float32 is what master weights are held in: read once, so not kept in the caches (where the codes stay)
    const u32x4 a = __builtin_nontemporal_load(reinterpret_cast<const Aligned<4>::type*>(p));
    const u32x4 b = __builtin_nontemporal_load(reinterpret_cast<const Aligned<4>::type*>(p + 4));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __uint_as_float(a[i]);
      f[4 + i] = __uint_as_float(b[i]);
    }
  } else {
    Elem<T>::unpack(load16(p), f);
  }
}

// s_sf byte of (row r of the tile, block b of its 16): words of four blocks, rows consecutive
__device__ __forceinline__ int sf_at(int r, int b) { return ((b >> 2) * kTileRows + r) * 4 + (b & 3); }

template <typename T>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const T* __restrict__ src, long long stride, int M, int K,
                                                             uint8_t* __restrict__ codes, uint8_t* __restrict__ sf,
                                                             int AM, long long ntiles, int ctiles) {
  constexpr int TR = kTileRows, RW = TR / 4;  // rows per wave
  __shared__ __attribute__((aligned(16))) uint8_t s_sf[TR * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int G = K / 32;
  for (long long tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
    const int c0 = (int)(tile % ctiles) * kTileCols;
    const long long r0 = tile / ctiles * TR;
    const int c = c0 + lane * 8;
    float f[RW][8];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const long long r = r0 + wave * RW + i;
      if (r < M && c < K) load8(src + r * stride + c, f[i]);
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const long long r = r0 + wave * RW + i;
      int byte = 0;
      if (r < M && c < K) {  // K is a multiple of 32: the 4 lanes of a block go together
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t a = __float_as_uint(f[i][j]) & 0x7fffffffu;
          m = m > a ? m : a;
        }
        m = umax_dpp<0xB1>(m);  // quad_perm [1,0,3,2]
        m = umax_dpp<0x4E>(m);  // quad_perm [2,3,0,1]
        byte = ue8m0_for_amax6(m);
        const float inv = inv_scale_of(byte == 255 ? 127 : byte);
        uint32_t q = 0;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[i][0] * inv, f[i][1] * inv, 1.f, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[i][2] * inv, f[i][3] * inv, 1.f, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[i][4] * inv, f[i][5] * inv, 1.f, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[i][6] * inv, f[i][7] * inv, 1.f, 3);
        *reinterpret_cast<uint32_t*>(codes + r * (K / 2) + c / 2) = byte == 255 ? 0u : q;
      }
      if ((lane & 3) == 0) s_sf[sf_at(wave * RW + i, lane >> 2)] = (uint8_t)byte;  // 0 in the padding
    }
    __syncthreads();
    if (AM > 0) {  // packed: word (row m, j) at j * AM + m, padding words and bytes zero
      for (int i = tid; i < TR * 4; i += 256) {
        const int j = c0 / 128 + i / TR;
        const long long m = r0 + i % TR;
        if (j < (G + 3) / 4 && m < AM)
          reinterpret_cast<uint32_t*>(sf)[(long long)j * AM + m] = reinterpret_cast<const uint32_t*>(s_sf)[i];
      }
    } else {
      for (int i = tid; i < TR * 16; i += 256) {
        const int r = i >> 4, g = c0 / 32 + (i & 15);
        if (r0 + r < M && g < G) sf[(r0 + r) * G + g] = s_sf[sf_at(r, i & 15)];
      }
    }
    __syncthreads();
  }
}

template <typename T>
__global__ __launch_bounds__(256) void dequantize_mxfp4_kernel(const uint8_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ sf, int AM, int M, int K,
                                                               T* __restrict__ dst, long long stride, long long ntiles,
                                                               int ctiles) {
  constexpr int TR = kTileRows, RW = TR / 4;
  __shared__ __attribute__((aligned(16))) uint8_t s_sf[TR * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int G = K / 32;
  for (long long tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
    const int c0 = (int)(tile % ctiles) * kTileCols;
    const long long r0 = tile / ctiles * TR;
    const int c = c0 + lane * 8;
    uint32_t q[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const long long r = r0 + wave * RW + i;
      if (r < M && c < K) q[i] = *reinterpret_cast<const uint32_t*>(codes + r * (K / 2) + c / 2);
    }
    if (AM > 0) {
      for (int i = tid; i < TR * 4; i += 256) {
        const int j = c0 / 128 + i / TR;
        const long long m = r0 + i % TR;
        if (j < (G + 3) / 4 && m < M)
          reinterpret_cast<uint32_t*>(s_sf)[i] = reinterpret_cast<const uint32_t*>(sf)[(long long)j * AM + m];
      }
    } else {
      for (int i = tid; i < TR * 16; i += 256) {
        const int r = i >> 4, g = c0 / 32 + (i & 15);
        if (r0 + r < M && g < G) s_sf[sf_at(r, i & 15)] = sf[(r0 + r) * G + g];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const long long r = r0 + wave * RW + i;
      if (r < M && c < K) {
        const uint32_t b = s_sf[sf_at(wave * RW + i, lane >> 2)];
        const float scale = __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23);
        float f[8];
        auto two = [&](auto v, int j) {
          f[j] = v[0] * scale;
          f[j + 1] = v[1] * scale;
        };
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.f, 0), 0);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.f, 1), 2);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.f, 2), 4);
        two(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], 1.f, 3), 6);
        T* p = dst + r * stride + c;
        if constexpr (sizeof(T) == 4) {
          store16(p, __builtin_bit_cast(u32x4, (v4f{f[0], f[1], f[2], f[3]})));
          store16(p + 4, __builtin_bit_cast(u32x4, (v4f{f[4], f[5], f[6], f[7]})));
        } else {
          store16(p, pack16<T>(f));
        }
      }
    }
    __syncthreads();
  }
}

namespace {

struct Tiles {
  long long n;
  int cols;
  unsigned grid;
};

Tiles tiles_of(int M, int K) {
  Tiles t;
  t.cols = (K + kTileCols - 1) / kTileCols;
  t.n = ((long long)M + kTileRows - 1) / kTileRows * t.cols;
  t.grid = (unsigned)(t.n < (1 << 20) ? t.n : (1 << 20));
  return t;
}

template <typename T>
hipError_t quantize(const void* src, long long stride, int M, int K, uint8_t* codes, uint8_t* sf, int AM,
                    hipStream_t s) {
  const Tiles t = tiles_of(M, K);
  quantize_mxfp4_kernel<T><<<t.grid, 256, 0, s>>>(static_cast<const T*>(src), stride, M, K, codes, sf, AM, t.n,
                                                      t.cols);
  return hipGetLastError();
}

template <typename T>
hipError_t dequantize(const uint8_t* codes, const uint8_t* sf, int AM, int M, int K, void* dst, long long stride,
                      hipStream_t s) {
  const Tiles t = tiles_of(M, K);
  dequantize_mxfp4_kernel<T><<<t.grid, 256, 0, s>>>(codes, sf, AM, M, K, static_cast<T*>(dst), stride, t.n, t.cols);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_mxfp4(const void* src, int dtype, long long stride, int M, int K, uint8_t* codes,
                                 uint8_t* sf, int AM, hipStream_t s) {
  if (dtype == 0) return quantize<Bf16>(src, stride, M, K, codes, sf, AM, s);
  if (dtype == 1) return quantize<F16>(src, stride, M, K, codes, sf, AM, s);
  return quantize<float>(src, stride, M, K, codes, sf, AM, s);
}

hipError_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* sf, int AM, int M, int K, void* dst, int dtype,
                                   long long stride, hipStream_t s) {
  if (dtype == 0) return dequantize<Bf16>(codes, sf, AM, M, K, dst, stride, s);
  if (dtype == 1) return dequantize<F16>(codes, sf, AM, M, K, dst, stride, s);
  return dequantize<float>(codes, sf, AM, M, K, dst, stride, s);
}

}  // namespace moe
