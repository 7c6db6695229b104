// Grouped product of 16-bit rows with 4-bit weights that have a scale for each group of G along K:
//   C[r, n] = sum_g s[n, g] sum_{k in g} A[r, k] (q[n, k] - z[n, g])   for the rows r of expert e
// (MXFP4: E2M1 values instead of q - z, scales 2^(b - 127)), or the SwiGLU of two such sums.
//
// The codes become 16-bit floats in a lane's registers and go straight into the 16x16x32 matrix instruction, whose float32 sums
// over one group are then scaled.  A weight read from HBM at its rate leaves time for about three vector instructions a
// code, so what they cost is what counts: E2M1 has a conversion instruction for two codes, and so has E4M3, whose byte 0000qqqq is
// q 2^-9 for every q (subnormal to 7, the first binade from 8), so that with a scale of 2^9 it gives q.  The zero
// point comes off the sums: sum x (q - z) = sum x q - z sum x, the sum of x from one more matrix instruction, with ones.
//
// The weights are the instruction's second operand, so a lane's results, and the scale and zero point that it
// needs, belong to the one weight row whose codes it loads: row lane % 16.  Quarter lane / 16 loads 16 bytes, 32 codes.
// With groups of 128 or more, the four quarters' codes are of one group, and step j multiplies dword j of
// each; with groups of 32 or 64 the dwords are transposed between the quarters first, so that step j has the
// codes of quarter j, a run of 32.
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

enum Format { kInt4 = 0, kMxfp4 = 1 };

__device__ __forceinline__ v4f mfma(Bf16, u32x4 a, u32x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ v4f mfma(F16, u32x4 a, u32x4 b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <typename XT> __device__ __forceinline__ u32x4 ones() {
  constexpr uint32_t one = __is_same(XT, Bf16) ? 0x3f803f80u : 0x3c003c00u;
  return u32x4{one, one, one, one};
}

// two values from half H (0, 1) of four E4M3 bytes, times 2^9; from byte B of eight E2M1 codes
template <typename XT, bool H>
__device__ __forceinline__ uint32_t from_e4m3(uint32_t v) {
  if constexpr (__is_same(XT, Bf16)) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 512.f, H));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 512.f, H));
}
template <typename XT, int B>
__device__ __forceinline__ uint32_t from_e2m1(uint32_t v) {
  if constexpr (__is_same(XT, Bf16)) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, 1.f, B));
  else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(v, 1.f, B));
}

// eight codes as 16-bit floats, in their order
template <typename XT, int FMT>
__device__ __forceinline__ u32x4 widen(uint32_t q) {
  if constexpr (FMT == kMxfp4) {
    return u32x4{from_e2m1<XT, 0>(q), from_e2m1<XT, 1>(q), from_e2m1<XT, 2>(q), from_e2m1<XT, 3>(q)};
  } else {
    const uint32_t even = q & 0x0f0f0f0fu, odd = (q >> 4) & 0x0f0f0f0fu;
    const uint32_t a = __builtin_amdgcn_perm(odd, even, 0x05010400u), b = __builtin_amdgcn_perm(odd, even, 0x07030602u);
    return u32x4{from_e4m3<XT, false>(a), from_e4m3<XT, true>(a), from_e4m3<XT, false>(b), from_e4m3<XT, true>(b)};
  }
}

// out_j of quarter i = d_i of quarter j
__device__ __forceinline__ u32x4 transpose_quarters(u32x4 d) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false));
  const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false));
  const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false));
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// a stored scale's bits as a float: a UE8M0 byte, float16 or bfloat16, float32
template <int SIZE>
__device__ __forceinline__ float scale_value(uint32_t raw, int dtype) {
  if constexpr (SIZE == 1) return __uint_as_float(raw == 0 ? 0x00400000u : raw == 255 ? 0x7fc00000u : raw << 23);
  if constexpr (SIZE == 4) return __uint_as_float(raw);
  float h = Elem<F16>::get(F16{(uint16_t)raw}), b = __uint_as_float(raw << 16);
  asm("" : "+v"(h), "+v"(b));  // both and a choice, not a branch
  return dtype == 0 ? b : h;
}

// Addresses of global memory (known to be so, or the compiler takes the loads that also serve LDS), a uniform one in scalar
// registers and a lane's own in vector registers, as they are: left to itself the compiler keeps a 64-bit vector address for each
// load of the loop and spills them
#define MOE_GLOBAL __attribute__((address_space(1)))
typedef const MOE_GLOBAL uint8_t* gptr;
__device__ __forceinline__ gptr scalar(const uint8_t* p) {
  gptr v = (gptr)p;
  asm("" : "+s"(v));
  return v;
}
template <typename T>
__device__ __forceinline__ gptr vector(const T* p) {
  gptr v = (gptr) reinterpret_cast<const uint8_t*>(p);
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ uint32_t vector(uint32_t v) {
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ u32x4 load_row16(gptr p) {  // 16 bytes of a row of 16-bit values
  typedef u32x4 at2 __attribute__((aligned(2)));
  return *(const MOE_GLOBAL at2*)p;
}

// N (1, 2 or 4) consecutive items of SIZE bytes at any alignment of theirs, as they lie; `have`: the first ones only
template <int N, int SIZE>
struct Items {
  static constexpr int kWords = (N * SIZE + 3) / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(gptr p) {
    if constexpr (N * SIZE == 1) {
      w[0] = *p;
    } else if constexpr (N * SIZE == 2) {
      typedef uint16_t at1 __attribute__((aligned(1)));
      w[0] = *(const MOE_GLOBAL at1*)p;
    } else if constexpr (N * SIZE == 4) {
      typedef uint32_t at1 __attribute__((aligned(1)));
      w[0] = *(const MOE_GLOBAL at1*)p;
    } else {
      typedef uint32_t vec __attribute__((ext_vector_type(kWords)));
      typedef vec at2 __attribute__((aligned(2)));
      const vec v = *(const MOE_GLOBAL at2*)p;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = v[i];
    }
  }
  __device__ __forceinline__ void load(gptr p, int have) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < have) {
        if constexpr (SIZE == 4) w[i] = ((const MOE_GLOBAL uint32_t*)p)[i];
        else if constexpr (SIZE == 2) w[i >> 1] |= (uint32_t)((const MOE_GLOBAL uint16_t*)p)[i] << (16 * (i & 1));
        else w[0] |= (uint32_t)p[i] << (8 * i);
      }
  }
  __device__ __forceinline__ uint32_t get(int i) const {
    if constexpr (SIZE == 4) return w[i];
    else if constexpr (SIZE == 2) return (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
    else return (w[0] >> (8 * i)) & 0xffu;
  }
};

__device__ __forceinline__ int2 expert_rows(const int32_t* __restrict__ offsets, int e, int rows) {
  if (offsets == nullptr) return make_int2(0, rows);
  const int lo = min(max(offsets[e], 0), rows);
  return make_int2(lo, min(max(offsets[e + 1], lo), rows));
}

// One sum by the definition.  q times an infinity is infinite or NaN whatever z is, and so is z times the sum of x,
// so where the sums taken apart are not finite, they are taken like this.
template <typename XT>
__device__ __forceinline__ float plain_sum(const XT* x, const uint8_t* q, const void* scales, const uint8_t* zeros,
                                        long long at, int K, int G, int scale_dtype) {
  float acc = 0.f;
  for (int k0 = 0; k0 < K; k0 += G, ++at) {
    const float z = zeros != nullptr ? (float)zeros[at] : 8.f;
    float sum = 0.f;
    for (int k = k0; k < k0 + G; ++k)
      sum = fmaf(Elem<XT>::get(x[k]), (float)((q[k >> 1] >> (4 * (k & 1))) & 15) - z, sum);
    const float s = scale_dtype == 2 ? scale_value<4>(static_cast<const uint32_t*>(scales)[at], 2)
                                     : scale_value<2>(static_cast<const uint16_t*>(scales)[at], scale_dtype);
    acc = fmaf(s, sum, acc);
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

// Where a wave's weight rows lie: NT tiles of 16, or a gate and an up tile.  Uniform addresses, and 32-bit offsets of the lane's
// row (cut to the expert's last one)
template <int SIZE, int NT>
struct Columns {
  const uint8_t *q[NT], *s[NT], *z[NT];
  uint32_t q_off[NT], s_off[NT], z_off[NT], z_mul;
  long long first[NT];  // first weight row of each tile, of all experts' rows
  int n0;               // first column of C

  __device__ __forceinline__ void init(const W4GemmArgs& g, int e, int column) {
    n0 = column;
    const int r16 = threadIdx.x & 15, q4 = (threadIdx.x >> 4) & 3, ng = g.K / g.G;
    const long long rows = g.act >= 0 ? 2LL * g.N : g.N;
    z_mul = g.zeros != nullptr ? 1 : 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int n = g.act >= 0 ? n0 : min(n0 + i * 16, g.N - 1);
      first[i] = e * rows + n + (g.act >= 0 && i ? g.N : 0);
      const uint32_t lane = min(r16, g.N - 1 - n);
      q[i] = uniform(g.B + first[i] * (g.K / 2));
      s[i] = uniform(static_cast<const uint8_t*>(g.scales) + first[i] * ng * SIZE);
      z[i] = uniform(g.zeros != nullptr ? g.zeros + first[i] * ng : g.B);  // without zero points one byte is read for all, and not used
      q_off[i] = lane * (uint32_t)(g.K / 2) + q4 * 16u;
      s_off[i] = lane * (uint32_t)(ng * SIZE);
      z_off[i] = lane * (uint32_t)ng * z_mul;
    }
  }
};

// What a wave needs of the weights for 128 of K.  FOLD: 32-wide steps that go under one scale; SIZE: a scale's bytes
template <int FMT, int SIZE, int FOLD, int NT>
struct Codes {
  static constexpr int NS = 4 / FOLD;  // scales
  u32x4 q[NT];
  Items<NS, SIZE> s[NT];
  Items<NS, 1> z[NT];

  // block b of K; FULL: all 128 are there.  per_group: 2^32 over the blocks of a group, rounded up
  template <bool FULL>
  __device__ __forceinline__ void load(const W4GemmArgs& g, const Columns<SIZE, NT>& c, int b, uint64_t per_group) {
    const int g0 = FOLD < 4 ? b * NS : (int)((uint32_t)b * per_group >> 32);
    const int have = g.K / g.G - g0, q4 = (threadIdx.x >> 4) & 3;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      q[i] = u32x4{0, 0, 0, 0};
      if (FULL || b * 128 + q4 * 32 < g.K) q[i] = *(const MOE_GLOBAL u32x4*)(scalar(c.q[i] + (long long)b * 64) + vector(c.q_off[i]));
      const gptr sp = scalar(c.s[i] + g0 * SIZE) + vector(c.s_off[i]);
      const gptr zp = scalar(c.z[i] + g0 * c.z_mul) + vector(c.z_off[i]);
      if constexpr (FULL) s[i].load(sp);
      else s[i].load(sp, have);
      if constexpr (FMT == kInt4) {
        if constexpr (FULL) z[i].load(zp);
        else z[i].load(zp, have);
      }
    }
  }
};

// acc += the products of 128 of K.  x(m, j): rows 16 m + lane % 16, the eight values of step j of this lane's quarter
template <typename XT, int FMT, int SIZE, int FOLD, int RT, int NT, typename X>
__device__ __forceinline__ void multiply(const W4GemmArgs& g, Codes<FMT, SIZE, FOLD, NT>& t, X x, v4f (&acc)[RT][NT]) {
  if constexpr (FOLD < 4) {
#pragma unroll
    for (int s = 0; s < NT; ++s) t.q[s] = transpose_quarters(t.q[s]);
  }
#pragma unroll
  for (int f = 0; f < 4 / FOLD; ++f) {
    v4f p[RT][NT], sum[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      sum[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NT; ++s) p[m][s] = v4f{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int i = 0; i < FOLD; ++i) {
      const int j = f * FOLD + i;
      __builtin_amdgcn_sched_barrier(0);  // one step's values in registers at a time
      u32x4 w[NT];
#pragma unroll
      for (int s = 0; s < NT; ++s) w[s] = widen<XT, FMT>(t.q[s][j]);
#pragma unroll
      for (int m = 0; m < RT; ++m) {
        const u32x4 v = x(m, j);
#pragma unroll
        for (int s = 0; s < NT; ++s) p[m][s] = mfma(XT{}, v, w[s], p[m][s]);
        if constexpr (FMT == kInt4) sum[m] = mfma(XT{}, v, ones<XT>(), sum[m]);
      }
    }
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      const float scale = scale_value<SIZE>(t.s[s].get(f), g.scale_dtype);
      const float z = FMT != kInt4 ? 0.f : g.zeros != nullptr ? -(float)t.z[s].get(f) : -8.f;
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = FMT == kInt4 ? fmaf(z, sum[m][i], p[m][s][i]) : p[m][s][i];
          acc[m][s][i] = fmaf(scale, v, acc[m][s][i]);
        }
    }
  }
}

__device__ __forceinline__ void store(const W4GemmArgs& g, float v, long long r, int n) {
  const long long at = r * g.c_stride + n;
  if (g.out_dtype == 2) static_cast<float*>(g.C)[at] = v;
  else if (g.out_dtype == 0) static_cast<Bf16*>(g.C)[at] = Elem<Bf16>::put(v);
  else static_cast<F16*>(g.C)[at] = Elem<F16>::put(v);
}

// result (r, n) by the definition; brow: its weight row, of all experts' rows
template <typename XT>
__device__ __noinline__ void plain_result(W4GemmArgs g, int r, int n, long long brow) {
  const auto sum = [&](long long row) {
    return plain_sum(static_cast<const XT*>(g.A) + r * g.a_stride, g.B + row * (g.K / 2), g.scales, g.zeros,
                     row * (g.K / g.G), g.K, g.G, g.scale_dtype);
  };
  const float v = sum(brow);
  store(g, g.act >= 0 ? activate(g, v, sum(brow + g.N)) : v, r, n);
}

__device__ __forceinline__ bool finite(float v) { return fabsf(v) < INFINITY; }

// a wave's tiles, straight from its registers: lane holds rows 4 q4 + i, column r16 of each
template <typename XT, int FMT, int SIZE, int RT, int NT>
__device__ __forceinline__ void finish(const W4GemmArgs& g, const v4f (&acc)[RT][NT], const Columns<SIZE, NT>& c, int m0,
                                       int m_end) {
  const int r16 = threadIdx.x & 15, q4 = (threadIdx.x >> 4) & 3;
  bool good = true;
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = m0 + m * 16 + 4 * q4 + i;
      if (r >= m_end) continue;
#pragma unroll
      for (int s = 0; s < NT; ++s) good = good && finite(acc[m][s][i]);
      if (g.act >= 0) {
        if (c.n0 + r16 < g.N) store(g, activate(g, acc[m][0][i], acc[m][NT - 1][i]), r, c.n0 + r16);
      } else {
#pragma unroll
        for (int s = 0; s < NT; ++s)
          if (c.n0 + s * 16 + r16 < g.N) store(g, acc[m][s][i], r, c.n0 + s * 16 + r16);
      }
    }
  if (FMT == kInt4 && !good)
    for (int s = 0; s < (g.act >= 0 ? 1 : NT); ++s)
      for (int i = 0; i < RT * 4; ++i) {
        const int r = m0 + i / 4 * 16 + 4 * q4 + i % 4, n = c.n0 + s * 16 + r16;
        if (r < m_end && n < g.N) plain_result<XT>(g, r, n, c.first[0] + s * 16 + r16);
      }
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// At most 16 rows at a time.  WK = 1: a workgroup of four waves, each with its own 16 NT weight rows; WK > 1: the WK waves
// share theirs, each takes every WK-th 128 of K, and their sums meet in LDS, in wave order.  The rows' values come straight from
// the caches; lanes past the last row read that one, and their results are not stored.  grid (column tiles, experts, row
// tiles)
template <typename XT, int FMT, int SIZE, int FOLD, int NT, int WK>
__global__ __launch_bounds__(WK == 1 ? 256 : WK * 64, 4) void w4_few_kernel(W4GemmArgs g, uint64_t per_group) {
  __shared__ float part[WK > 1 ? WK : 1][16][NT * 16 + 1];
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4, wave = wave_id();
  const int e = blockIdx.y, cols = g.act >= 0 ? 16 : NT * 16;
  const int2 rr = expert_rows(g.offsets, e, g.rows);
  const long long column = (long long)(WK == 1 ? blockIdx.x * 4 + wave : blockIdx.x) * cols;
  if (column >= g.N || rr.x >= rr.y) return;
  Columns<SIZE, NT> c;
  c.init(g, e, (int)column);
  const int nfull = g.K / 128;
  for (long long m = rr.x + (long long)blockIdx.z * 16; m < rr.y; m += (long long)gridDim.z * 16) {
    const int m0 = (int)m;
    const XT* xp = static_cast<const XT*>(g.A) + (long long)min(m0 + r16, rr.y - 1) * g.a_stride + (FOLD == 4 ? q4 * 32 : q4 * 8);
    struct Block {
      Codes<FMT, SIZE, FOLD, NT> t;
      u32x4 x[4];
    } b0, b1;
    const auto load = [&](int b, Block& k) {
      k.t.template load<true>(g, c, b, per_group);
      const gptr xb = vector(xp + b * 128);
#pragma unroll
      for (int j = 0; j < 4; ++j) k.x[j] = load_row16(xb + (FOLD == 4 ? j * 16 : j * 64));
    };
    v4f acc[1][NT];
#pragma unroll
    for (int s = 0; s < NT; ++s) acc[0][s] = v4f{0.f, 0.f, 0.f, 0.f};
    const auto mul = [&](Block& k) {
      multiply<XT, FMT, SIZE, FOLD, 1, NT>(g, k.t, [&](int, int j) { return k.x[j]; }, acc);
    };
    // two blocks in turn, the next one's loads in flight; none of them under a condition, which would make the wait for
    // one block's a wait for all
    int b = WK > 1 ? wave : 0;
    if (b < nfull) load(b, b0);
    for (; b + 2 * WK < nfull; b += 2 * WK) {
      load(b + WK, b1);
      mul(b0);
      load(b + 2 * WK, b0);
      mul(b1);
    }
    if (b + WK < nfull) {
      load(b + WK, b1);
      mul(b0);
      mul(b1);
    } else if (b < nfull) {
      mul(b0);
    }
    if (FOLD < 4 && nfull * 128 < g.K && (WK == 1 || nfull % WK == wave)) {
      b0.t.template load<false>(g, c, nfull, per_group);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b0.x[j] = u32x4{0, 0, 0, 0};
        if (nfull * 128 + j * 32 < g.K) b0.x[j] = load16(xp + nfull * 128 + j * 32);
      }
      mul(b0);
    }
    if constexpr (WK == 1) {
      finish<XT, FMT>(g, acc, c, m0, rr.y);
    } else {
#pragma unroll
      for (int s = 0; s < NT; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][4 * q4 + i][s * 16 + r16] = acc[0][s][i];
      __syncthreads();
      const int rows = min(16, rr.y - m0);
      const auto total = [&](int r, int col) {
        float v = part[0][r][col];
#pragma unroll
        for (int w = 1; w < WK; ++w) v += part[w][r][col];
        return v;
      };
      for (int i = threadIdx.x; i < rows * cols; i += WK * 64) {
        const int r = i / cols, col = i % cols;
        if (c.n0 + col >= g.N) continue;
        float v = total(r, col), up = 0.f;
        if (g.act >= 0) up = total(r, NT * 16 - 16 + col);
        if (FMT == kInt4 && !(finite(v) && finite(up))) plain_result<XT>(g, m0 + r, c.n0 + col, c.first[0] + col);
        else store(g, g.act >= 0 ? activate(g, v, up) : v, m0 + r, c.n0 + col);
      }
      __syncthreads();
    }
  }
}

// Up to 64 rows at a time: a workgroup of four waves, 32 weight rows each, the rows' values brought to LDS by all four, 128 of
// K at a time into one of two slots.
template <typename XT, int FMT, int SIZE, int FOLD, int RT>
__device__ __forceinline__ void tile_rows(const W4GemmArgs& g, uint64_t per_group, uint8_t (*lds)[64 * 256],
                                          const Columns<SIZE, 2>& c, bool mine, int m0, int m_end) {
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4, tid = threadIdx.x;
  const int nfull = g.K / 128;
  // thread: 16-byte chunk tid % 16 of rows tid / 16 + 16 m; in LDS a row's chunks are turned by its number, so that 16 rows' equal
  // chunks lie in different banks
  const int srow = tid >> 4, chunk = tid & 15;
  const XT* src[RT];
#pragma unroll
  for (int m = 0; m < RT; ++m)
    src[m] = static_cast<const XT*>(g.A) + (long long)min(m0 + m * 16 + srow, m_end - 1) * g.a_stride + chunk * 8;
  u32x4 stage[RT];
  Codes<FMT, SIZE, FOLD, 2> next;
  const auto fetch = [&](int b) {
#pragma unroll
    for (int m = 0; m < RT; ++m) stage[m] = load_row16(vector(src[m] + b * 128));
    next.template load<true>(g, c, b, per_group);
  };
  const auto put = [&](int b) {
#pragma unroll
    for (int m = 0; m < RT; ++m)
      *reinterpret_cast<u32x4*>(lds[b & 1] + (m * 16 + srow) * 256 + ((chunk ^ srow) & 15) * 16) = stage[m];
  };
  v4f acc[RT][2];
#pragma unroll
  for (int m = 0; m < RT; ++m)
#pragma unroll
    for (int s = 0; s < 2; ++s) acc[m][s] = v4f{0.f, 0.f, 0.f, 0.f};
  const auto step = [&](int b, Codes<FMT, SIZE, FOLD, 2>& codes) {
    const uint8_t* at = lds[b & 1] + r16 * 256;
    multiply<XT, FMT, SIZE, FOLD, RT, 2>(g, codes, [&](int m, int j) {
      const int k = FOLD == 4 ? q4 * 4 + j : j * 4 + q4;
      return *reinterpret_cast<const u32x4*>(at + m * 16 * 256 + (k ^ r16) * 16);
    }, acc);
  };
  if (nfull > 0) {
    fetch(0);
    put(0);
    for (int b = 0; b + 1 < nfull; ++b) {
      __syncthreads();  // this block's slot is written, and the other one's readers are done
      Codes<FMT, SIZE, FOLD, 2> now = next;
      fetch(b + 1);
      step(b, now);
      put(b + 1);
    }
    __syncthreads();
    step(nfull - 1, next);
  }
  if (FOLD < 4 && nfull * 128 < g.K) {  // the last, partial block
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      stage[m] = u32x4{0, 0, 0, 0};
      if (nfull * 128 + chunk * 8 < g.K) stage[m] = load16(src[m] + nfull * 128);
    }
    next.template load<false>(g, c, nfull, per_group);
    put(nfull);
    __syncthreads();
    step(nfull, next);
  }
  if (mine) finish<XT, FMT>(g, acc, c, m0, m_end);
  __syncthreads();
}

template <typename XT, int FMT, int SIZE, int FOLD>
__global__ __launch_bounds__(256, 2) void w4_tile_kernel(W4GemmArgs g, uint64_t per_group) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][64 * 256];
  const int e = blockIdx.y, cols = g.act >= 0 ? 16 : 32;
  const int2 rr = expert_rows(g.offsets, e, g.rows);
  const long long column = (long long)(blockIdx.x * 4 + wave_id()) * cols;
  const bool mine = column < g.N;  // a wave without columns helps with the rows
  Columns<SIZE, 2> c;
  c.init(g, e, mine ? (int)column : 0);
  for (long long m = rr.x + (long long)blockIdx.z * 64; m < rr.y; m += (long long)gridDim.z * 64) {
    const int m0 = (int)m, rows = rr.y - m0;
    if (rows <= 16) tile_rows<XT, FMT, SIZE, FOLD, 1>(g, per_group, lds, c, mine, m0, rr.y);
    else if (rows <= 32) tile_rows<XT, FMT, SIZE, FOLD, 2>(g, per_group, lds, c, mine, m0, rr.y);
    else tile_rows<XT, FMT, SIZE, FOLD, 4>(g, per_group, lds, c, mine, m0, rr.y);
  }
}

template <typename XT, int FMT, int SIZE, int FOLD>
hipError_t launch(const W4GemmArgs& g, hipStream_t s) {
  const int bpg = g.G / 128;
  const uint64_t per_group = bpg > 0 ? (0x100000000ULL + bpg - 1) / bpg : 0;
  const auto go = [&](auto kern, int columns, int threads, int rows) {
    const int z = (g.rows + rows - 1) / rows, most = g.groups == 1 ? 1024 : 4;
    kern<<<dim3((g.N + columns - 1) / columns, g.groups, z < most ? z : most), threads, 0, s>>>(g, per_group);
    return hipGetLastError();
  };
  const bool act = g.act >= 0;
  if (g.rows > 16 && g.rows > 8LL * g.groups) return go(w4_tile_kernel<XT, FMT, SIZE, FOLD>, act ? 64 : 128, 256, 64);
  // tiles of 32 weight rows; while they fill the GPU's waves, one wave for each
  const long long tiles = (long long)g.groups * ((g.N + 15) / 16) * (act ? 2 : 1) / 2;
  if (tiles >= 2048) return go(w4_few_kernel<XT, FMT, SIZE, FOLD, 2, 4>, act ? 16 : 32, 256, 16);
  if (act || tiles >= 512) return go(w4_few_kernel<XT, FMT, SIZE, FOLD, 2, 8>, act ? 16 : 32, 512, 16);
  return go(w4_few_kernel<XT, FMT, SIZE, FOLD, 1, 16>, 16, 1024, 16);
}

template <typename XT, int SIZE>
hipError_t int4_by_group(const W4GemmArgs& g, hipStream_t s) {
  if (g.G == 32) return launch<XT, kInt4, SIZE, 1>(g, s);
  if (g.G == 64) return launch<XT, kInt4, SIZE, 2>(g, s);
  return launch<XT, kInt4, SIZE, 4>(g, s);
}
template <typename XT>
hipError_t by_weights(const W4GemmArgs& g, bool mxfp4, hipStream_t s) {
  if (mxfp4) return launch<XT, kMxfp4, 1, 1>(g, s);
  return g.scale_dtype == 2 ? int4_by_group<XT, 4>(g, s) : int4_by_group<XT, 2>(g, s);
}

}  // namespace

hipError_t launch_w4_gemm(const W4GemmArgs& g, int dtype, bool mxfp4, hipStream_t s) {
  return dtype == 0 ? by_weights<Bf16>(g, mxfp4, s) : by_weights<F16>(g, mxfp4, s);
}

}  // namespace moe
