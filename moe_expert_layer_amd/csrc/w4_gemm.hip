// Grouped product of 16-bit rows with 4-bit weights that have a scale for each group of G along K:
//   C[r, n] = sum_g s[n, g] sum_{k in g} A[r, k] (q[n, k] - z[n, g])   for the rows r of expert e
// (MXFP4: E2M1 values instead of q - z, scales 2^(b - 127)), or the SwiGLU of two such sums.
//
// For few rows: the weights are read once and are what bounds it, about 0.55 bytes a weight from HBM, so a weight may
// cost some two instructions.  The codes become exact 16-bit floats in a lane's registers and go straight into the
// 16x16x32 matrix instruction, whose float32 sums of one group are then scaled:
//   bf16  16 + q is the bits 0x4180 | q << 3 (no conversion); sum x (q - z) = sum x (16 + q) - (16 + z) sum x, the sum of x
//         from one more matrix instruction, with ones
//   f16   1024 + q is 0x6400 | q, and subtracting 1024 + z is exact
//   E2M1  the conversion instruction
// The weights are the instruction's second operand, so a lane's results, and the scale and zero point that it
// needs, belong to the one weight row whose codes it loads: row lane % 16.  Quarter lane / 16 loads 16 bytes, 32 codes.
// With groups of 128 or more, the four quarters' codes are of one group, and step j multiplies dword j of
// each; with groups of 32 or 64 the dwords are transposed between the quarters first, so that step j has the
// codes of quarter j, a run of 32.
//
// A workgroup takes 16 NT weight rows of one expert; its NW waves every NW-th 128 of K, and their sums meet in LDS, in
// wave order.
#include <hip/hip_runtime.h>
#include <cstdint>

#include "device_common.hpp"
#include "elem.hpp"
#include "operators.hpp"

namespace moe {

namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

enum Format { kInt4 = 0, kMxfp4 = 1 };

__device__ __forceinline__ v4f mfma(Bf16, u32x4 a, u32x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma(F16, u32x4 a, u32x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// bytes I of a and of b as the low bytes of a pair of 16-bit halves
template <int I>
__device__ __forceinline__ uint32_t byte_pair(uint32_t b, uint32_t a) {
  return __builtin_amdgcn_perm(b, a, 0x0c040c00u + 0x00010001u * I);
}

// eight codes as 16-bit floats: 16 + q (bf16), q - z (f16; zh: 1024 + z twice), E2M1 values
template <typename XT, int FMT>
__device__ __forceinline__ u32x4 widen(uint32_t q, uint32_t zh) {
  u32x4 w;
  if constexpr (FMT == kMxfp4) {
    if constexpr (sizeof(XT) && __is_same(XT, Bf16)) {
      w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 0));
      w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 1));
      w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 2));
      w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.f, 3));
    } else {
      w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.f, 0));
      w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.f, 1));
      w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.f, 2));
      w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.f, 3));
    }
  } else if constexpr (__is_same(XT, Bf16)) {
    const uint32_t lo = q << 3, hi = q >> 1;  // low and high nibbles in bits 3 to 6 of each byte
    w[0] = (byte_pair<0>(hi, lo) & 0x00780078u) | 0x41804180u;
    w[1] = (byte_pair<1>(hi, lo) & 0x00780078u) | 0x41804180u;
    w[2] = (byte_pair<2>(hi, lo) & 0x00780078u) | 0x41804180u;
    w[3] = (byte_pair<3>(hi, lo) & 0x00780078u) | 0x41804180u;
  } else {
    const uint32_t hi = q >> 4;
    const f16x2 z = __builtin_bit_cast(f16x2, zh);
    w[0] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (byte_pair<0>(hi, q) & 0x000f000fu) | 0x64006400u) - z);
    w[1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (byte_pair<1>(hi, q) & 0x000f000fu) | 0x64006400u) - z);
    w[2] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (byte_pair<2>(hi, q) & 0x000f000fu) | 0x64006400u) - z);
    w[3] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, (byte_pair<3>(hi, q) & 0x000f000fu) | 0x64006400u) - z);
  }
  return w;
}

// out_j of quarter i = d_i of quarter j
__device__ __forceinline__ u32x4 transpose_quarters(u32x4 d) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false));
  const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false));
  const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false));
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// a stored scale's bits as a float (0 bf16, 1 f16, 2 f32; MXFP4: the UE8M0 byte)
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t raw, int dtype) {
  if constexpr (FMT == kMxfp4) return __uint_as_float(raw == 0 ? 0x00400000u : raw == 255 ? 0x7fc00000u : raw << 23);
  return dtype == 2 ? __uint_as_float(raw) : dtype == 0 ? __uint_as_float(raw << 16) : Elem<F16>::get(F16{(uint16_t)raw});
}

// N consecutive items of SIZE bytes, each in a register of its own; the last `have` < N only
template <int N, int SIZE>
__device__ __forceinline__ void load_items(const void* base, long long at, int have, uint32_t (&v)[N]) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + at * SIZE;
  if (have >= N) {
    if constexpr (SIZE == 4) {
      typedef uint32_t vec __attribute__((ext_vector_type(N == 1 ? 2 : N)));
      typedef vec at4 __attribute__((aligned(4)));
      if constexpr (N == 1) {
        v[0] = *reinterpret_cast<const uint32_t*>(p);
      } else {
        const vec w = *reinterpret_cast<const at4*>(p);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = w[i];
      }
    } else if constexpr (SIZE == 2) {
      if constexpr (N == 1) {
        v[0] = *reinterpret_cast<const uint16_t*>(p);
      } else if constexpr (N == 2) {
        typedef uint32_t at2 __attribute__((aligned(2)));
        const uint32_t w = *reinterpret_cast<const at2*>(p);
        v[0] = w & 0xffffu;
        v[1] = w >> 16;
      } else {
        typedef u32x2 at2 __attribute__((aligned(2)));
        const u32x2 w = *reinterpret_cast<const at2*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
      }
    } else {
      if constexpr (N == 1) {
        v[0] = *p;
      } else if constexpr (N == 2) {
        typedef uint16_t at1 __attribute__((aligned(1)));
        const uint32_t w = *reinterpret_cast<const at1*>(p);
        v[0] = w & 0xffu;
        v[1] = w >> 8;
      } else {
        typedef uint32_t at1 __attribute__((aligned(1)));
        const uint32_t w = *reinterpret_cast<const at1*>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (w >> (8 * i)) & 0xffu;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0;
      if (i < have) {
        if constexpr (SIZE == 4) v[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else if constexpr (SIZE == 2) v[i] = reinterpret_cast<const uint16_t*>(p)[i];
        else v[i] = p[i];
      }
    }
  }
}

__device__ __forceinline__ int2 expert_rows(const int32_t* __restrict__ offsets, int e, int rows) {
  if (offsets == nullptr) return make_int2(0, rows);
  const int lo = min(max(offsets[e], 0), rows);
  return make_int2(lo, min(max(offsets[e + 1], lo), rows));
}

// One sum by the definition.  16 + q times an infinity is infinite whatever q is, and its zero point's part is infinite too,
// so where the sums by 16 + q are not finite, they are taken like this.
__device__ __noinline__ float plain_sum(const Bf16* x, const uint8_t* q, const void* scales, const uint8_t* zeros,
                                        long long at, int K, int G, int scale_dtype) {
  float acc = 0.f;
  for (int k0 = 0; k0 < K; k0 += G, ++at) {
    const float z = zeros != nullptr ? (float)zeros[at] : 8.f;
    float sum = 0.f;
    for (int k = k0; k < k0 + G; ++k)
      sum = fmaf(Elem<Bf16>::get(x[k]), (float)((q[k >> 1] >> (4 * (k & 1))) & 15) - z, sum);
    const uint32_t raw = scale_dtype == 2 ? static_cast<const uint32_t*>(scales)[at] : static_cast<const uint16_t*>(scales)[at];
    acc = fmaf(scale_value<kInt4>(raw, scale_dtype), sum, acc);
  }
  return acc;
}

__device__ __forceinline__ float activate(const W4GemmArgs& g, float gate, float up) {
  float alpha = 1.f;
  if (g.act == 1) {
    // clamps that keep NaN
    gate = gate > g.clamp ? g.clamp : gate;
    up = up > g.clamp ? g.clamp : up < -g.clamp ? -g.clamp : up;
    up += g.bias;
    alpha = g.alpha;
  }
  return gate / (1.f + expf(-alpha * gate)) * up;
}

// what a wave needs of 128 of K for NT weight rows of each lane
template <int FOLD, int NT>
struct Block {
  u32x4 q[NT];
  uint32_t s[NT][4 / FOLD], z[NT][4 / FOLD];
};

// rows [m0, m_end) of one expert, at most 16 RT of them, by 16 NT weight rows.  FOLD: 32-wide steps that go under one scale
template <typename XT, int FMT, int FOLD, int RT, int NT, int NW, int MAXR>
__device__ __forceinline__ void rows_tile(const W4GemmArgs& g, float (*part)[MAXR][NT * 16 + 1], int e, int n0, int m0,
                                          int m_end) {
  constexpr int NS = 4 / FOLD;  // scales of a block
  constexpr bool kOnes = FMT == kInt4 && __is_same(XT, Bf16);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r16 = lane & 15, q4 = lane >> 4;
  const int nblk = (g.K + 127) / 128, ng = g.K / g.G, steps = g.G / 32;
  const long long ld = g.K / 2;
  const long long b_rows = g.act >= 0 ? 2LL * g.N : g.N;  // weight rows of an expert
  const uint8_t* bq[NT];
  long long brow[NT];
  const XT* x[RT];
  bool live[RT];
#pragma unroll
  for (int m = 0; m < RT; ++m) {
    live[m] = m0 + m * 16 + r16 < m_end;
    x[m] = static_cast<const XT*>(g.A) + (long long)(live[m] ? m0 + m * 16 + r16 : m0) * g.a_stride;
  }
#pragma unroll
  for (int s = 0; s < NT; ++s) {
    const int n = g.act >= 0 ? min(n0 + r16, g.N - 1) + (s ? g.N : 0) : min(n0 + s * 16 + r16, g.N - 1);
    brow[s] = e * b_rows + n;
    bq[s] = g.B + brow[s] * ld;
  }
  v4f acc[RT][NT];
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int s = 0; s < NT; ++s) acc[m][s] = v4f{0.f, 0.f, 0.f, 0.f};

  const auto load = [&](int b, Block<FOLD, NT>& t) {
    const int k = b * 128 + q4 * 32;
    const int g0 = b * 4 / steps;            // first group of the block
    const int have = min(NS, ng - g0);       // groups inside K
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      t.q[s] = u32x4{0, 0, 0, 0};
      if (FOLD == 4 || k < g.K) t.q[s] = *reinterpret_cast<const u32x4*>(bq[s] + k / 2);
      const long long at = brow[s] * ng + g0;
      if constexpr (FMT == kMxfp4) load_items<NS, 1>(g.scales, at, have, t.s[s]);
      else if (g.scale_dtype == 2) load_items<NS, 4>(g.scales, at, have, t.s[s]);
      else load_items<NS, 2>(g.scales, at, have, t.s[s]);
      if (FMT == kInt4 && g.zeros != nullptr) {
        load_items<NS, 1>(g.zeros, at, have, t.z[s]);
      } else {
#pragma unroll
        for (int i = 0; i < NS; ++i) t.z[s][i] = 8;
      }
    }
  };

  Block<FOLD, NT> next;
  if (wave < nblk) load(wave, next);
  for (int b = wave; b < nblk; b += NW) {
    Block<FOLD, NT> t = next;
    u32x4 xv[RT][4];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = FOLD == 4 ? b * 128 + q4 * 32 + j * 8 : b * 128 + j * 32 + q4 * 8;
        xv[m][j] = u32x4{0, 0, 0, 0};
        if (live[m] && (FOLD == 4 || k < g.K)) xv[m][j] = load16(x[m] + k);
      }
    if (b + NW < nblk) load(b + NW, next);
    if constexpr (FOLD < 4) {
#pragma unroll
      for (int s = 0; s < NT; ++s) t.q[s] = transpose_quarters(t.q[s]);
    }
#pragma unroll
    for (int f = 0; f < NS; ++f) {
      v4f p[RT][NT], ones[RT];
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        ones[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NT; ++s) p[m][s] = v4f{0.f, 0.f, 0.f, 0.f};
      }
#pragma unroll
      for (int i = 0; i < FOLD; ++i) {
        const int j = f * FOLD + i;
        u32x4 w[NT];
#pragma unroll
        for (int s = 0; s < NT; ++s) w[s] = widen<XT, FMT>(t.q[s][j], 0x64006400u + t.z[s][f] * 0x00010001u);
#pragma unroll
        for (int m = 0; m < RT; ++m) {
#pragma unroll
          for (int s = 0; s < NT; ++s) p[m][s] = mfma(XT{}, xv[m][j], w[s], p[m][s]);
          if constexpr (kOnes)
            ones[m] = mfma(XT{}, xv[m][j], u32x4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}, ones[m]);
        }
      }
#pragma unroll
      for (int s = 0; s < NT; ++s) {
        const float scale = scale_value<FMT>(t.s[s][f], g.scale_dtype);
        const float z = -16.f - (float)t.z[s][f];
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = kOnes ? fmaf(z, ones[m][i], p[m][s][i]) : p[m][s][i];
            acc[m][s][i] = fmaf(scale, v, acc[m][s][i]);
          }
      }
    }
  }
  // a lane holds rows 4 q4 + i, column r16 of each 16 x 16 tile
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][m * 16 + 4 * q4 + i][s * 16 + r16] = acc[m][s][i];
  __syncthreads();
  const int rows = min(RT * 16, m_end - m0);
  const auto total = [&](int r, int c, int n) {
    float v = part[0][r][c];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += part[w][r][c];
    if constexpr (kOnes)
      if (!(fabsf(v) < INFINITY))
        v = plain_sum(static_cast<const Bf16*>(g.A) + (long long)(m0 + r) * g.a_stride, g.B + (e * b_rows + n) * ld,
                      g.scales, g.zeros, (e * b_rows + n) * ng, g.K, g.G, g.scale_dtype);
    return v;
  };
  const int cols = g.act >= 0 ? 16 : NT * 16;
  for (int i = tid; i < rows * cols; i += NW * 64) {
    const int r = i / cols, c = i % cols, n = n0 + c;
    if (n >= g.N) continue;
    const float v = g.act >= 0 ? activate(g, total(r, c, n), total(r, 16 + c, g.N + n)) : total(r, c, n);
    const long long at = (long long)(m0 + r) * g.c_stride + n;
    if (g.out_dtype == 2) static_cast<float*>(g.C)[at] = v;
    else if (g.out_dtype == 0) static_cast<Bf16*>(g.C)[at] = Elem<Bf16>::put(v);
    else static_cast<F16*>(g.C)[at] = Elem<F16>::put(v);
  }
  __syncthreads();
}

// grid (column tiles, experts, row tiles)
template <typename XT, int FMT, int FOLD, int NT, int NW, int MAXR>
__global__ __launch_bounds__(NW * 64) void w4_rows_kernel(W4GemmArgs g) {
  __shared__ float part[NW][MAXR][NT * 16 + 1];
  const int e = blockIdx.y, n0 = blockIdx.x * (g.act >= 0 ? 16 : NT * 16);
  const int2 rr = expert_rows(g.offsets, e, g.rows);
  for (long long m = rr.x + (long long)blockIdx.z * MAXR; m < rr.y; m += (long long)gridDim.z * MAXR) {
    const int m0 = (int)m, rows = rr.y - m0;
    if (MAXR == 16 || rows <= 16) rows_tile<XT, FMT, FOLD, 1, NT, NW, MAXR>(g, part, e, n0, m0, rr.y);
    else if (rows <= 32) rows_tile<XT, FMT, FOLD, 2, NT, NW, MAXR>(g, part, e, n0, m0, rr.y);
    else rows_tile<XT, FMT, FOLD, MAXR / 16, NT, NW, MAXR>(g, part, e, n0, m0, rr.y);
  }
}

template <typename XT, int FMT, int FOLD>
hipError_t launch(const W4GemmArgs& g, hipStream_t s) {
  const auto go = [&](auto kern, int nt, int nw, int maxr) {
    const int cols = g.act >= 0 ? 16 : nt * 16;
    const int z = g.groups == 1 ? (g.rows + maxr - 1) / maxr : 1;
    kern<<<dim3((g.N + cols - 1) / cols, g.groups, z < 1024 ? z : 1024), nw * 64, 0, s>>>(g);
    return hipGetLastError();
  };
  const bool few = g.rows <= 16 * g.groups;
  if (g.act >= 0) {
    return few ? go(w4_rows_kernel<XT, FMT, FOLD, 2, 4, 16>, 2, 4, 16) : go(w4_rows_kernel<XT, FMT, FOLD, 2, 4, 64>, 2, 4, 64);
  }
  return few ? go(w4_rows_kernel<XT, FMT, FOLD, 1, 8, 16>, 1, 8, 16) : go(w4_rows_kernel<XT, FMT, FOLD, 2, 4, 64>, 2, 4, 64);
}

template <typename XT>
hipError_t by_group(const W4GemmArgs& g, bool mxfp4, hipStream_t s) {
  if (mxfp4) return launch<XT, kMxfp4, 1>(g, s);
  if (g.G == 32) return launch<XT, kInt4, 1>(g, s);
  if (g.G == 64) return launch<XT, kInt4, 2>(g, s);
  return launch<XT, kInt4, 4>(g, s);
}

}  // namespace

hipError_t launch_w4_gemm(const W4GemmArgs& g, int dtype, bool mxfp4, hipStream_t s) {
  return dtype == 0 ? by_group<Bf16>(g, mxfp4, s) : by_group<F16>(g, mxfp4, s);
}

}  // namespace moe
