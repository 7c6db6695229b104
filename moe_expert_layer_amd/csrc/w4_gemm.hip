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
//
// Three kernels: few rows with K split over waves, few rows by many weight rows, and tiles of up to 64 rows (launch has the rule).  With few
// rows HBM is the bound: 128 rows in 32 experts of 4096 x 7168 take 95 to 97 us with groups of 128 and zero points (5.1 TB/s; a copy runs at 4.9),
// MXFP4 weights of 7168 x 2048 61 us (4.2 TB/s: four scales a block of 128 and their sums).  One row through 4096 x 7168 takes 7 us, nearly
// all of them the kernel's: 3 at a copy's rate, but a workgroup a CU has some 8 KB of loads under way, too few for that.  Tiles are bound by
// instructions: 2000 rows through 32 experts of 4096 x 4096 with groups of 64 take 164 to 173 us, 65 at a copy's rate; of a SIMD's cycles the
// matrix instructions take 24% and the vector ones 45% (the scaled additions two fifths of those), and two waves a SIMD, all that the
// registers allow, leave much of the rest empty.  64 rows in each of those experts: 143 us with groups of 128 or MXFP4 weights, 172 with
// groups of 64 (4 to 8 vector registers spilled), 455 with groups of 32 (110 to 113: four sets of sums and scales a block live beside the
// sums over K).  The kernel of many weight rows spills 10 and 27 with float32 scales and groups of 32 and 64.
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

// Eight codes as 16-bit floats; INT4: even ones, then odd ones, as the nibbles come, the rows' values being put in that order once for many
// weights (turn)
template <typename XT, int FMT>
__device__ __forceinline__ u32x4 widen(uint32_t q) {
  if constexpr (FMT == kMxfp4)
    return u32x4{from_e2m1<XT, 0>(q), from_e2m1<XT, 1>(q), from_e2m1<XT, 2>(q), from_e2m1<XT, 3>(q)};
  const uint32_t even = q & 0x0f0f0f0fu, odd = (q >> 4) & 0x0f0f0f0fu;
  return u32x4{from_e4m3<XT, false>(even), from_e4m3<XT, true>(even), from_e4m3<XT, false>(odd), from_e4m3<XT, true>(odd)};
}
template <int FMT>
__device__ __forceinline__ u32x4 turn(u32x4 x) {
  if constexpr (FMT == kMxfp4) return x;
  constexpr uint32_t lo = 0x05040100u, hi = 0x07060302u;
  return u32x4{__builtin_amdgcn_perm(x[1], x[0], lo), __builtin_amdgcn_perm(x[3], x[2], lo),
               __builtin_amdgcn_perm(x[1], x[0], hi), __builtin_amdgcn_perm(x[3], x[2], hi)};
}

// out_j of quarter i = d_i of quarter j
__device__ __forceinline__ u32x4 transpose_quarters(u32x4 d) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false));
  const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false));
  const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false));
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// a stored scale's bits as a float: a UE8M0 byte (255, NaN, becomes an infinity, which makes the results not finite, and those
// are taken again), float16 or bfloat16, float32
template <int SIZE>
__device__ __forceinline__ float scale_value(uint32_t raw, int dtype) {
  if constexpr (SIZE == 1) {
    const uint32_t v = raw << 23;
    return __uint_as_float(v > 0x00400000u ? v : 0x00400000u);
  }
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

// Scales and zero points lie in LDS as bytes that are written in one width and read in another, so both go through types that may
// alias; and what a lane reads there other lanes of its wave wrote, so a fence stands between.  A wave's LDS instructions run in
// order: the fence keeps the compiler's order and makes no instruction.
typedef uint32_t __attribute__((may_alias)) lds_u32;
typedef uint16_t __attribute__((may_alias)) lds_u16;
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// N (a power of two) consecutive items of SIZE bytes at any alignment of theirs, as they lie
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
      constexpr int kStep = kWords < 4 ? kWords : 4;
      typedef uint32_t vec __attribute__((ext_vector_type(kStep)));
      typedef vec at1 __attribute__((aligned(1)));
#pragma unroll
      for (int j = 0; j < kWords; j += kStep) {
        const vec v = *(const MOE_GLOBAL at1*)(p + 4 * j);
#pragma unroll
        for (int i = 0; i < kStep; ++i) w[j + i] = v[i];
      }
    }
  }
  __device__ __forceinline__ void load_lds(const uint8_t* p) {
    if constexpr (N * SIZE == 1) w[0] = *p;
    else if constexpr (N * SIZE == 2) w[0] = *reinterpret_cast<const lds_u16*>(p);
    else
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const lds_u32*>(p)[i];
  }
  __device__ __forceinline__ uint32_t get(int i) const {
    if constexpr (SIZE == 4) return w[i];
    else if constexpr (SIZE == 2) return (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
    else return (w[i >> 2] >> (8 * (i & 3))) & 0xffu;
  }
};

__device__ __forceinline__ int2 expert_rows(const int32_t* __restrict__ offsets, int e, int rows) {
  if (offsets == nullptr) return make_int2(0, rows);
  const int lo = min(max(offsets[e], 0), rows);
  return make_int2(lo, min(max(offsets[e + 1], lo), rows));
}

// One sum by the definition.  q times an infinity is infinite or NaN whatever z is, and so is z times the sum of x,
// so where the sums taken apart are not finite, they are taken like this.
template <typename XT, int FMT>
__device__ __forceinline__ float plain_sum(const XT* x, const uint8_t* q, const void* scales, const uint8_t* zeros,
                                           long long at, int K, int G, int scale_dtype) {
  float acc = 0.f;
  for (int k0 = 0; k0 < K; k0 += G, ++at) {
    const float z = zeros != nullptr ? (float)zeros[at] : 8.f;
    float sum = 0.f, s;
    for (int k = k0; k < k0 + G; ++k) {
      const int c = (q[k >> 1] >> (4 * (k & 1))) & 15;
      float w = (float)c - z;
      if (FMT == kMxfp4) {
        const int m = c & 7;
        w = m < 4 ? m * 0.5f : m < 6 ? m - 2.f : 2.f * m - 8.f;  // 0 .5 1 1.5 2 3 4 6
        w = c > 7 ? -w : w;
      }
      sum = fmaf(Elem<XT>::get(x[k]), w, sum);
    }
    if (FMT == kMxfp4) {
      const uint32_t b = static_cast<const uint8_t*>(scales)[at];
      s = b == 255 ? __uint_as_float(0x7fc00000u) : scale_value<1>(b, 0);
    } else {
      s = scale_dtype == 2 ? scale_value<4>(static_cast<const uint32_t*>(scales)[at], 2)
                           : scale_value<2>(static_cast<const uint16_t*>(scales)[at], scale_dtype);
    }
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

// Where a wave's weight rows lie: NT tiles of 16, or NT / 2 gate tiles and as many up tiles.  Uniform addresses, and 32-bit offsets of the lane's
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
      const bool up = g.act >= 0 && i >= NT / 2;
      const int n = min(n0 + (up ? i - NT / 2 : i) * 16, g.N - 1);
      first[i] = e * rows + n + (up ? g.N : 0);
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

// Sums of a wave's tiles.  One group's sums wait until the matrix instructions of the next have been issued before they are
// scaled and added, so that those few instructions do not wait for the matrix cores (with RT > 1 rows' tiles there are
// enough of them in flight)
template <int FMT, int RT, int NT>
struct Sums {
  static constexpr bool kWait = RT == 1;
  v4f acc[RT][NT], p[RT][NT], x[RT];  // x: of the rows' values
  float scale[NT], zero[NT];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      x[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NT; ++s) acc[m][s] = p[m][s] = v4f{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int s = 0; s < NT; ++s) scale[s] = zero[s] = 0.f;
  }
  __device__ __forceinline__ void add(const v4f (&q)[RT][NT], const v4f (&sx)[RT], const float (&sc)[NT], const float (&z)[NT]) {
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float v = FMT == kInt4 ? fmaf(-z[s], sx[m][i], q[m][s][i]) : q[m][s][i];
          acc[m][s][i] = fmaf(sc[s], v, acc[m][s][i]);
        }
  }
  __device__ __forceinline__ void finish() {
    if (kWait) add(p, x, scale, zero);
  }
};

// The products of 128 of K.  q: codes; x(m, j): rows 16 m + lane % 16, the eight values of step j of this lane's quarter (asked for
// a step ahead; v has those of step 0, and on return those of step 4); scale_of(s, f), zero_of(s, f): of tile s and fold f
template <typename XT, int FMT, int FOLD, int RT, int NT, typename X, typename S, typename Z>
__device__ __forceinline__ void multiply(u32x4 (&q)[NT], u32x4 (&v)[RT], X x, S scale_of, Z zero_of, Sums<FMT, RT, NT>& sums) {
  if constexpr (FOLD < 4) {
#pragma unroll
    for (int s = 0; s < NT; ++s) q[s] = transpose_quarters(q[s]);
  }
#pragma unroll
  for (int f = 0; f < 4 / FOLD; ++f) {
    v4f p[RT][NT], sx[RT];
    float scale[NT], zero[NT];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      sx[m] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < NT; ++s) p[m][s] = v4f{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int i = 0; i < FOLD; ++i) {
      const int j = f * FOLD + i;
      __builtin_amdgcn_sched_barrier(0);  // one step's values in registers at a time
      u32x4 w[NT], ahead[RT];
#pragma unroll
      for (int m = 0; m < RT; ++m) ahead[m] = x(m, j + 1);
#pragma unroll
      for (int s = 0; s < NT; ++s) {
        w[s] = widen<XT, FMT>(q[s][j]);
        if constexpr (RT > 1) asm("" : "+v"(w[s]));  // once for all rows' tiles: the compiler widens again for each
      }
#pragma unroll
      for (int m = 0; m < RT; ++m) {
#pragma unroll
        for (int s = 0; s < NT; ++s) p[m][s] = mfma(XT{}, v[m], w[s], p[m][s]);
        if constexpr (FMT == kInt4) sx[m] = mfma(XT{}, v[m], ones<XT>(), sx[m]);
        v[m] = ahead[m];
      }
      if (Sums<FMT, RT, NT>::kWait && i == 0) {
        __builtin_amdgcn_sched_barrier(0);
        sums.add(sums.p, sums.x, sums.scale, sums.zero);
      }
    }
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      scale[s] = scale_of(s, f);
      zero[s] = FMT == kInt4 ? zero_of(s, f) : 0.f;
    }
    if (!Sums<FMT, RT, NT>::kWait) {
      sums.add(p, sx, scale, zero);
    } else {
#pragma unroll
      for (int s = 0; s < NT; ++s) {
        sums.p[0][s] = p[0][s];
        sums.scale[s] = scale[s];
        sums.zero[s] = zero[s];
      }
      sums.x[0] = sx[0];
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
template <typename XT, int FMT>
__device__ __noinline__ void plain_result(W4GemmArgs g, int r, int n, long long brow) {
  const auto sum = [&](long long row) {
    return plain_sum<XT, FMT>(static_cast<const XT*>(g.A) + r * g.a_stride, g.B + row * (g.K / 2), g.scales, g.zeros,
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
#pragma unroll
      for (int s = 0; s < NT; ++s) {
        const int n = c.n0 + s * 16 + r16;
        if (n >= g.N || (g.act >= 0 && s >= NT / 2)) continue;
        store(g, g.act >= 0 ? activate(g, acc[m][s][i], acc[m][s < NT / 2 ? s + NT / 2 : s][i]) : acc[m][s][i], r, n);
      }
    }
  if (!good)
    for (int s = 0; s < (g.act >= 0 ? NT / 2 : NT); ++s)
      for (int i = 0; i < RT * 4; ++i) {
        const int r = m0 + i / 4 * 16 + 4 * q4 + i % 4, n = c.n0 + s * 16 + r16;
        if (r < m_end && n < g.N) plain_result<XT, FMT>(g, r, n, c.first[0] + s * 16 + r16);
      }
}

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// The scales and zero points of a wave's weight rows, kUnit groups at a time: each quarter of the lanes loads a quarter of them of its
// row, runs of 64 bytes and more between them, and the wave's own part of LDS gives them out as they are needed.  (Loaded in
// place, a few bytes of each row at a time, they took 15 of 132 us.)  Rows whose number of groups is no multiple of four are
// copied item by item.
template <int FMT, int SIZE, int NT, int kUnit>
struct ScaleLoad {
  static constexpr int kPart = kUnit / 4;
  Items<kPart, SIZE> s[NT];
  Items<kPart, 1> z[NT];

  // groups past the row's last one are not used: the last ones again
  __device__ __forceinline__ void load(const W4GemmArgs& g, const Columns<SIZE, NT>& c, int base) {
    const int ng = g.K / g.G, first = base + ((threadIdx.x >> 4) & 3) * kPart;
#pragma unroll
    for (int i = 0; i < kPart / 4; ++i) {
      const uint32_t at = max(min(first + 4 * i, ng - 4), 0);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        Items<4, SIZE> v;
        v.load(scalar(c.s[t]) + vector(c.s_off[t] + at * SIZE));
#pragma unroll
        for (int j = 0; j < SIZE; ++j) s[t].w[i * SIZE + j] = v.w[j];
        if constexpr (FMT == kInt4) {
          Items<4, 1> y;
          y.load(scalar(c.z[t]) + vector(c.z_off[t] + at * c.z_mul));
          z[t].w[i] = y.w[0];
        }
      }
    }
  }
};
template <int FMT, int SIZE, int NT, int kUnit>
struct ScaleLds {
  // a row's items and a few bytes, so that 16 rows' equal ones lie in different banks
  static constexpr int kPart = kUnit / 4;
  static constexpr int kS = kUnit * SIZE + (SIZE == 1 ? 4 : 8), kZ = FMT == kInt4 ? kUnit + 4 : 0, kBytes = NT * 16 * (kS + kZ);
  uint8_t* at;  // this lane's row

  __device__ __forceinline__ uint8_t* scales(int t) const { return at + t * 16 * kS; }
  __device__ __forceinline__ uint8_t* zeros(int t) const { return at + NT * 16 * kS + t * 16 * kZ - (threadIdx.x & 15) * (kS - kZ); }
  __device__ __forceinline__ void put(const ScaleLoad<FMT, SIZE, NT, kUnit>& l) const {
    const int q4 = (threadIdx.x >> 4) & 3;
    wave_fence();  // the lanes have read what was there
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < Items<kPart, SIZE>::kWords; ++i) reinterpret_cast<lds_u32*>(scales(t) + q4 * kPart * SIZE)[i] = l.s[t].w[i];
      if constexpr (FMT == kInt4) {
#pragma unroll
        for (int i = 0; i < kPart / 4; ++i) reinterpret_cast<lds_u32*>(zeros(t) + q4 * kPart)[i] = l.z[t].w[i];
      }
    }
    wave_fence();
  }
  __device__ __forceinline__ void copy(const W4GemmArgs& g, const Columns<SIZE, NT>& c, int base) const {
    const int ng = g.K / g.G, q4 = (threadIdx.x >> 4) & 3;
    wave_fence();
    for (int i = 0; i < kPart; ++i) {
      const uint32_t at = min(base + q4 * kPart + i, ng - 1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        Items<1, SIZE> v;
        v.load(scalar(c.s[t]) + vector(c.s_off[t] + at * SIZE));
        uint8_t* to = scales(t) + (q4 * kPart + i) * SIZE;
        if constexpr (SIZE == 4) *reinterpret_cast<lds_u32*>(to) = v.w[0];
        else if constexpr (SIZE == 2) *reinterpret_cast<lds_u16*>(to) = (uint16_t)v.w[0];
        else *to = (uint8_t)v.w[0];
        if constexpr (FMT == kInt4) {
          Items<1, 1> y;
          y.load(scalar(c.z[t]) + vector(c.z_off[t] + at * c.z_mul));
          zeros(t)[q4 * kPart + i] = (uint8_t)y.w[0];
        }
      }
    }
    wave_fence();
  }
};

// At most 16 rows at a time by 16 NT weight rows a workgroup: its WK waves share those, each takes a run of blocks of 128 of K, and their
// sums meet in LDS, in wave order.
//
// What counts here is how many cache lines a load touches: a lane's part of the rows or of the scales, loaded where it is needed, touches
// as many lines for a few bytes of each as its codes do.  So each wave brings scales and rows' values in longer runs, through
// parts of LDS that are its own.  CH: 16-byte chunks of the rows' values that a lane brings, for 4 CH rows.
template <typename XT, int FMT, int SIZE, int FOLD, int NT, int CH, typename Lds>
__device__ __forceinline__ void few_rows(const W4GemmArgs& g, uint64_t per_group, const Columns<SIZE, NT>& c, const Lds& sl,
                                         uint8_t* xl, int m0, int m_end, int first, int last, Sums<FMT, 1, NT>& sums) {
  constexpr int F = FOLD > 4 ? 4 : FOLD, NS = 4 / F, kUnit = Lds::kPart * 4;  // NS: scales of a block
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4;
  const int ng = g.K / g.G;
  // lane: chunk lane % 16 of rows lane / 16 + 4 i; a chunk's number is turned by the row's, so that 16 rows' equal chunks lie in
  // different banks
  const XT* src[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) src[i] = static_cast<const XT*>(g.A) + (long long)min(m0 + q4 + 4 * i, m_end - 1) * g.a_stride + r16 * 8;
  const int xrow = min(r16, 4 * CH - 1);
  int xoff[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) xoff[j] = xrow * 256 + (((F == 4 ? q4 * 4 + j : j * 4 + q4) ^ xrow) & 15) * 16;
  struct Block {
    u32x4 q[NT], x[CH];
  } b0, b1;
  const auto load = [&](int b, Block& k) {
#pragma unroll
    for (int t = 0; t < NT; ++t) k.q[t] = *(const MOE_GLOBAL u32x4*)(scalar(c.q[t] + (long long)b * 64) + vector(c.q_off[t]));
#pragma unroll
    for (int i = 0; i < CH; ++i) k.x[i] = load_row16(vector(src[i] + b * 128));
  };
  const auto group_of = [&](int b) { return FOLD > 4 ? (int)((uint32_t)b * per_group >> 32) : b * NS; };
  int base = 0;  // first group in LDS
  const auto mul = [&](int b, Block& k) {
    wave_fence();
#pragma unroll
    for (int i = 0; i < CH; ++i)
      *reinterpret_cast<u32x4*>(xl + (q4 + 4 * i) * 256 + ((r16 ^ (q4 + 4 * i)) & 15) * 16) = turn<FMT>(k.x[i]);
    wave_fence();
    Items<NS, SIZE> s[NT];
    Items<NS, 1> z[NT];
    const int at = group_of(b) - base;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      s[t].load_lds(sl.scales(t) + at * SIZE);
      if constexpr (FMT == kInt4) z[t].load_lds(sl.zeros(t) + at);
    }
    const auto x = [&](int, int j) { return *reinterpret_cast<const u32x4*>(xl + xoff[j & 3]); };
    u32x4 xv[1] = {x(0, 0)};
    multiply<XT, FMT, F, 1, NT>(
        k.q, xv, x, [&](int t, int f) { return scale_value<SIZE>(s[t].get(f), g.scale_dtype); },
        [&](int t, int f) { return g.zeros != nullptr ? (float)z[t].get(f) : 8.f; }, sums);
  };
  // as many blocks as kUnit - 4 groups make, or fewer, at a time
  constexpr int kBlocks = (kUnit - 4) / NS;
  for (int b = first; b < last;) {
    const int end = min(b + kBlocks, last);
    const bool full = end * 128 <= g.K;  // else the last block is partial
    const int whole = full ? end : end - 1;
    if (b < whole) load(b, b0);
    base = group_of(b) & ~3;
    if ((ng & 3) == 0) {
      ScaleLoad<FMT, SIZE, NT, kUnit> sc;
      sc.load(g, c, base);
      sl.put(sc);
    } else {
      sl.copy(g, c, base);
    }
    // two blocks in turn, the next one's loads in flight; none of them under a condition, which would make the wait for
    // one block's a wait for all
    for (; b + 2 < whole; b += 2) {
      load(b + 1, b1);
      mul(b, b0);
      load(b + 2, b0);
      mul(b + 1, b1);
    }
    if (b + 1 < whole) {
      load(b + 1, b1);
      mul(b, b0);
      mul(b + 1, b1);
    } else if (b < whole) {
      mul(b, b0);
    }
    if (FOLD < 4 && !full) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        b0.q[t] = u32x4{0, 0, 0, 0};
        if (whole * 128 + q4 * 32 < g.K) b0.q[t] = *reinterpret_cast<const u32x4*>(c.q[t] + whole * 64LL + c.q_off[t]);
      }
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        b0.x[i] = u32x4{0, 0, 0, 0};
        if (whole * 128 + r16 * 8 < g.K) b0.x[i] = load16(src[i] + whole * 128);
      }
      mul(whole, b0);
    }
    b = end;
  }
}

// grid (column tiles, experts, row tiles)
template <typename XT, int FMT, int SIZE, int FOLD, int NT, int WK>
__global__ __launch_bounds__(WK * 64, NT == 1 ? 3 : 2) void w4_few_kernel(W4GemmArgs g, uint64_t per_group) {
  using Lds = ScaleLds<FMT, SIZE, NT, 32>;
  __shared__ float part[WK][16][NT * 16 + 1];
  __shared__ __attribute__((aligned(16))) uint8_t x_lds[WK][4096], scale_lds[WK][Lds::kBytes];
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4, wave = wave_id();
  const int e = blockIdx.y, cols = g.act >= 0 ? NT * 8 : NT * 16;
  const int2 rr = expert_rows(g.offsets, e, g.rows);
  if (rr.x >= rr.y) return;
  Columns<SIZE, NT> c;
  c.init(g, e, blockIdx.x * cols);
  const Lds sl{scale_lds[wave] + r16 * Lds::kS};
  // runs of blocks as even as they can be
  const int nblk = (g.K + 127) / 128, first = (int)((long long)nblk * wave / WK), last = (int)((long long)nblk * (wave + 1) / WK);
  for (long long m = rr.x + (long long)blockIdx.z * 16; m < rr.y; m += (long long)gridDim.z * 16) {
    const int m0 = (int)m, rows = min(16, rr.y - m0);
    Sums<FMT, 1, NT> sums;
    sums.clear();
    if (rows <= 4) few_rows<XT, FMT, SIZE, FOLD, NT, 1>(g, per_group, c, sl, x_lds[wave], m0, rr.y, first, last, sums);
    else if (rows <= 8) few_rows<XT, FMT, SIZE, FOLD, NT, 2>(g, per_group, c, sl, x_lds[wave], m0, rr.y, first, last, sums);
    else few_rows<XT, FMT, SIZE, FOLD, NT, 4>(g, per_group, c, sl, x_lds[wave], m0, rr.y, first, last, sums);
    sums.finish();
#pragma unroll
    for (int s = 0; s < NT; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[wave][4 * q4 + i][s * 16 + r16] = sums.acc[0][s][i];
    __syncthreads();
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
      if (g.act >= 0) up = total(r, NT * 8 + col);
      if (!(finite(v) && finite(up))) plain_result<XT, FMT>(g, m0 + r, c.n0 + col, c.first[0] + col);
      else store(g, g.act >= 0 ? activate(g, v, up) : v, m0 + r, c.n0 + col);
    }
    __syncthreads();
  }
}

// At most 16 rows at a time by many weight rows: a workgroup of four waves, 16 NT weight rows each.  The rows' values go through
// LDS, 16 KB of them at a time into one of two slots; the codes come from memory 512 of K ahead.  grid (column tiles, experts, row
// tiles)
template <typename XT, int FMT, int SIZE, int FOLD, int NT>
__global__ __launch_bounds__(256, 2) void w4_stream_kernel(W4GemmArgs g, uint64_t per_group) {
  constexpr int F = FOLD > 4 ? 4 : FOLD, NS = 4 / F, kSlot = 16384;  // NS: scales of a block of 128
  constexpr int kUnit = FOLD < 4 ? 64 : 32;
  using Lds = ScaleLds<FMT, SIZE, NT, kUnit>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][kSlot];
  __shared__ __attribute__((aligned(16))) uint8_t scale_lds[4][Lds::kBytes];
  const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15, q4 = lane >> 4;
  const int e = blockIdx.y, cols = g.act >= 0 ? 8 * NT : 16 * NT;
  const int2 rr = expert_rows(g.offsets, e, g.rows);
  const long long column = (long long)(blockIdx.x * 4 + wave_id()) * cols;
  const bool mine = column < g.N;  // a wave without columns helps with the rows
  Columns<SIZE, NT> c;
  c.init(g, e, mine ? (int)column : 0);
  const Lds sl{scale_lds[wave_id()] + r16 * Lds::kS};
  const int nfull = g.K / 512, nsb = (g.K + 511) / 512, nblk = (g.K + 127) / 128, ng = g.K / g.G;
  for (long long m = rr.x + (long long)blockIdx.z * 16; m < rr.y; m += (long long)gridDim.z * 16) {
    const int m0 = (int)m, rows = min(16, rr.y - m0);
    // a slot holds 16 KB / rows (rounded up to a power of two) of each row
    const int row_log2 = rows <= 1 ? 0 : 32 - __builtin_clz(rows - 1);
    const int sb_log2 = 4 - row_log2, nslots = (nsb + (1 << sb_log2) - 1) >> sb_log2;
    // thread: 16-byte chunk at[i] of a row's part of a slot
    const XT* src[4];
    int at[4], to[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = tid + 256 * i, row = id >> (6 + sb_log2);
      at[i] = (id & ((64 << sb_log2) - 1)) * 8;
      src[i] = static_cast<const XT*>(g.A) + (long long)(m0 + min(row, rows - 1)) * g.a_stride;
      to[i] = (id ^ (row & 7)) * 16;
    }
    u32x4 stage[4];
    const auto fetch = [&](int slot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = (slot << sb_log2) * 512 + at[i];
        stage[i] = load_row16(vector(src[i] + min(k, g.K - 8)));
        if (k >= g.K) stage[i] = u32x4{0, 0, 0, 0};
      }
    };
    const auto put = [&](int slot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4*>(lds[slot & 1] + to[i]) = turn<FMT>(stage[i]);
    };
    // where a lane's values of step j lie in a block: the low three bits of a chunk's number are turned by the row's
    const int xrow = min(r16, rows - 1);
    int xoff[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      xoff[j] = (xrow << (10 + sb_log2)) + (((F == 4 ? q4 * 4 + j : j * 4 + q4) ^ (xrow & 7)) * 16);
    Sums<FMT, 1, NT> sums;
    sums.clear();
    u32x4 q[4][NT], xv[1];
    ScaleLoad<FMT, SIZE, NT, kUnit> sc;
    constexpr int kLast = FOLD > 4 ? 1 : 4 / NS;
    Items<kLast * NS, SIZE> bs[NT];
    Items<kLast * NS, 1> bz[NT];
    const bool quads = (ng & 3) == 0;
    // two blocks, 128 bytes of each row, together: asked for one at a time, a cache line's second half came so late that it had to be
    // fetched again
    const auto codes = [&](int b, u32x4 (&v)[NT], u32x4 (&w)[NT]) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const gptr p = scalar(c.q[t] + (long long)b * 64) + vector(c.q_off[t]);
        v[t] = *(const MOE_GLOBAL u32x4*)p;
        w[t] = *(const MOE_GLOBAL u32x4*)(p + 64);
      }
    };
    const auto group_of = [&](int b) { return FOLD > 4 ? (int)((uint32_t)b * per_group >> 32) : b * NS; };
    // block i of the 512 of K at sb
    const auto block = [&](int slot, int sb, int i) {
      const uint8_t* base = lds[slot & 1] + (sb & ((1 << sb_log2) - 1)) * 1024;
      const auto x = [&](int, int j) {  // past the 512 (not used, but in the slot) the first ones
        return *reinterpret_cast<const u32x4*>(base + xoff[j & 3] + ((i + j / 4) & 3) * 256);
      };
      if (i == 0) xv[0] = x(0, 0);
      // scales and zero points of as many blocks as four groups make, or of one block where they are larger
      if (i % kLast == 0) {
        const int at = group_of(sb * 4 + i) & (kUnit - 1);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          bs[t].load_lds(sl.scales(t) + at * SIZE);
          if constexpr (FMT == kInt4) bz[t].load_lds(sl.zeros(t) + at);
        }
      }
      multiply<XT, FMT, F, 1, NT>(
          q[i], xv, x, [&](int t, int f) { return scale_value<SIZE>(bs[t].get(i % kLast * NS + f), g.scale_dtype); },
          [&](int t, int f) { return g.zeros != nullptr ? (float)bz[t].get(i % kLast * NS + f) : 8.f; }, sums);
    };
    // the scales where the 512 of K at sb are the first that need them, and the next ones' loads
    int unit = 0;
    const auto turn_scales = [&](int sb) {
      if (group_of(sb * 4) / kUnit == unit) {
        if (quads) sl.put(sc);
        else sl.copy(g, c, unit * kUnit);
        ++unit;
        if (quads && unit * kUnit < ng) sc.load(g, c, unit * kUnit);
      }
    };
    fetch(0);
    if (quads) sc.load(g, c, 0);
    if (nfull > 0) {
      codes(0, q[0], q[1]);
      codes(2, q[2], q[3]);
    }
    put(0);
    for (int slot = 0, sb = 0; slot < nslots; ++slot) {
      __syncthreads();  // this slot is written, and the other one's readers are done
      fetch(min(slot + 1, nslots - 1));
      const int end = min((slot + 1) << sb_log2, nfull);
      for (; sb < end; ++sb) {
        turn_scales(sb);
        const int next = min(sb + 1, nfull - 1);  // past the end the last ones again, so that no load of codes is under a condition
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          block(slot, sb, i);
          if (i & 1) codes(next * 4 + i - 1, q[i - 1], q[i]);
        }
      }
      if (slot == nslots - 1 && nfull < nsb) {  // less than 512 at the end
        turn_scales(nfull);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            q[i][t] = u32x4{0, 0, 0, 0};
            if (nfull * 512 + i * 128 + q4 * 32 < g.K) q[i][t] = *reinterpret_cast<const u32x4*>(c.q[t] + (nfull * 4 + i) * 64LL + c.q_off[t]);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (nfull * 4 + i < nblk) block(slot, nfull, i);
      }
      put(slot + 1);
    }
    sums.finish();
    if (mine) finish<XT, FMT>(g, sums.acc, c, m0, rr.y);
    __syncthreads();
  }
}

// Up to kTileRows rows at a time: a workgroup of four waves, 32 weight rows each.  The rows' values are brought to LDS by all four, 128 of
// K at a time into one of two slots; the codes come a block of 128 ahead of that.
constexpr int kTileRows = 64;
template <typename XT, int FMT, int SIZE, int FOLD, int RT, typename Lds>
__device__ __forceinline__ void tile_rows(const W4GemmArgs& g, uint64_t per_group, uint8_t (*lds)[kTileRows * 256], const Lds& sl,
                                          const Columns<SIZE, 2>& c, bool mine, int m0, int m_end) {
  constexpr int F = FOLD > 4 ? 4 : FOLD, NS = 4 / F, kUnit = Lds::kPart * 4;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4, tid = threadIdx.x;
  const int nfull = g.K / 128, ng = g.K / g.G;
  // thread: 16-byte chunk tid % 16 of a block of rows tid / 16 + 16 m; a chunk's number is turned by the row's, so that 16 rows' equal
  // chunks lie in different banks
  const int srow = tid >> 4, chunk = tid & 15;
  const XT* src[RT];
#pragma unroll
  for (int m = 0; m < RT; ++m)
    src[m] = static_cast<const XT*>(g.A) + (long long)min(m0 + m * 16 + srow, m_end - 1) * g.a_stride + chunk * 8;
  u32x4 stage[RT];
  const auto fetch = [&](int b) {  // the rows' values of block b
#pragma unroll
    for (int m = 0; m < RT; ++m) stage[m] = load_row16(vector(src[m] + b * 128));
  };
  const auto put = [&](int b) {
    uint8_t* at = lds[b & 1] + srow * 256 + ((chunk ^ srow) & 15) * 16;
#pragma unroll
    for (int m = 0; m < RT; ++m) *reinterpret_cast<u32x4*>(at + m * 16 * 256) = turn<FMT>(stage[m]);
  };
  int xoff[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) xoff[j] = r16 * 256 + (((F == 4 ? q4 * 4 + j : j * 4 + q4) ^ r16) * 16);
  Sums<FMT, RT, 2> sums;
  sums.clear();
  const auto codes = [&](int b, u32x4 (&q)[2]) {
#pragma unroll
    for (int t = 0; t < 2; ++t) q[t] = *(const MOE_GLOBAL u32x4*)(scalar(c.q[t] + (long long)b * 64) + vector(c.q_off[t]));
  };
  const auto group_of = [&](int b) { return FOLD > 4 ? (int)((uint32_t)b * per_group >> 32) : b * NS; };
  int base = -kUnit;  // first group in LDS
  const auto step = [&](int b, u32x4 (&q)[2]) {
    if (group_of(b) >= base + kUnit) {
      base += kUnit;
      if ((ng & 3) == 0) {
        ScaleLoad<FMT, SIZE, 2, kUnit> sc;
        sc.load(g, c, base);
        sl.put(sc);
      } else {
        sl.copy(g, c, base);
      }
    }
    Items<NS, SIZE> s[2];
    Items<NS, 1> z[2];
    const int at = group_of(b) - base;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t].load_lds(sl.scales(t) + at * SIZE);
      if constexpr (FMT == kInt4) z[t].load_lds(sl.zeros(t) + at);
    }
    const uint8_t* p = lds[b & 1];
    const auto x = [&](int m, int j) { return *reinterpret_cast<const u32x4*>(p + m * 16 * 256 + xoff[j & 3]); };
    u32x4 v[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) v[m] = x(m, 0);
    multiply<XT, FMT, F, RT, 2>(
        q, v, x, [&](int t, int f) { return scale_value<SIZE>(s[t].get(f), g.scale_dtype); },
        [&](int t, int f) { return g.zeros != nullptr ? (float)z[t].get(f) : 8.f; }, sums);
  };
  // no load of codes or rows is under a condition: past the last whole block the same one is read again
  u32x4 q0[2], q1[2];
  if (nfull > 0) {
    fetch(0);
    codes(0, q0);
    codes(min(1, nfull - 1), q1);
    put(0);
  }
  const auto turn_block = [&](int b, u32x4 (&q)[2]) {
    __syncthreads();  // this slot is written, and the other one's readers are done
    fetch(min(b + 1, nfull - 1));
    step(b, q);
    codes(min(b + 2, nfull - 1), q);
    put(b + 1);
  };
  int b = 0;
  for (; b + 1 < nfull; b += 2) {
    turn_block(b, q0);
    turn_block(b + 1, q1);
  }
  if (b < nfull) turn_block(b, q0);
  if (FOLD < 4 && nfull * 128 < g.K) {  // the last, partial block, zeros past K
    __syncthreads();
    const bool in = nfull * 128 + chunk * 8 < g.K;
#pragma unroll
    for (int m = 0; m < RT; ++m) {
      stage[m] = u32x4{0, 0, 0, 0};
      if (in) stage[m] = load_row16(vector(src[m] + nfull * 128));
    }
    put(nfull);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      q0[t] = u32x4{0, 0, 0, 0};
      if (nfull * 128 + q4 * 32 < g.K) q0[t] = *reinterpret_cast<const u32x4*>(c.q[t] + nfull * 64LL + c.q_off[t]);
    }
    step(nfull, q0);
  }
  sums.finish();
  if (mine) finish<XT, FMT>(g, sums.acc, c, m0, m_end);
  __syncthreads();
}

template <typename XT, int FMT, int SIZE, int FOLD>
__global__ __launch_bounds__(256, 2) void w4_tile_kernel(W4GemmArgs g, uint64_t per_group) {
  using Lds = ScaleLds<FMT, SIZE, 2, 32>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][kTileRows * 256];
  __shared__ __attribute__((aligned(16))) uint8_t scale_lds[4][Lds::kBytes];
  const int e = blockIdx.y, cols = g.act >= 0 ? 16 : 32;
  const int2 rr = expert_rows(g.offsets, e, g.rows);
  const long long column = (long long)(blockIdx.x * 4 + wave_id()) * cols;
  const bool mine = column < g.N;  // a wave without columns helps with the rows
  Columns<SIZE, 2> c;
  c.init(g, e, mine ? (int)column : 0);
  const Lds sl{scale_lds[wave_id()] + (threadIdx.x & 15) * Lds::kS};
  // an expert's rows in as few parts as there can be, of equal numbers of tiles of 16
  const int all = (int)(((long long)rr.y - rr.x + 15) / 16), parts = (all + kTileRows / 16 - 1) / (kTileRows / 16);
  const int most = 16 * ((all + max(parts, 1) - 1) / max(parts, 1));
  for (long long m = rr.x + (long long)blockIdx.z * most; m < rr.y; m += (long long)gridDim.z * most) {
    const int m0 = (int)m, rows = min(most, rr.y - m0), end = m0 + rows;
    if (rows <= 16) tile_rows<XT, FMT, SIZE, FOLD, 1>(g, per_group, lds, sl, c, mine, m0, end);
    else if (rows <= 32) tile_rows<XT, FMT, SIZE, FOLD, 2>(g, per_group, lds, sl, c, mine, m0, end);
    else if (rows <= 48) tile_rows<XT, FMT, SIZE, FOLD, 3>(g, per_group, lds, sl, c, mine, m0, end);
    else tile_rows<XT, FMT, SIZE, FOLD, 4>(g, per_group, lds, sl, c, mine, m0, end);
  }
}

template <typename XT, int FMT, int SIZE, int FOLD>
hipError_t launch(const W4GemmArgs& g, hipStream_t s) {
  const int bpg = g.G / 128;
  const uint64_t per_group = bpg > 0 ? (0x100000000ULL + bpg - 1) / bpg : 0;
  // Rows' parts beyond those of evenly filled experts are taken in turn; where parts are large, by one more workgroup (32 experts, 62.5
  // rows on average, 42% of them above 64: 207 -> 194 us)
  const auto go = [&](auto kern, int columns, int threads, int rows) {
    const long long z = (g.rows + (long long)rows * g.groups - 1) / ((long long)rows * g.groups) + (rows > 16 && g.groups > 1);
    kern<<<dim3((g.N + columns - 1) / columns, g.groups, z < 1024 ? z : 1024), threads, 0, s>>>(g, per_group);
    return hipGetLastError();
  };
  const bool act = g.act >= 0;
  // Up to 16 rows an expert the weights are read once either way.  Above, the tile kernel reads them once for 64 rows, but its workgroups are
  // long: with less than one for each CU the few-rows kernel, a round for every 16 rows, is faster up to 64 rows an expert (64 rows through
  // 8192 x 8192: 40 us and 64; 128 rows: 79 and 64; 24 rows in each of 32 experts of 4096 x 4096: 143 and 110).
  const long long avg = (g.rows + g.groups - 1) / g.groups, wide = act ? 64 : 128;
  const long long workgroups = g.groups * ((g.N + wide - 1) / wide);
  if (avg > 64 || (avg > 16 && workgroups >= 256)) return go(w4_tile_kernel<XT, FMT, SIZE, FOLD>, (int)wide, 256, kTileRows);
  // Each wave of the stream kernel reads its own rows' whole length, the few-rows kernel's waves share a row: many weight rows keep the
  // card busy with the first, fewer with the second.  K = 7168, stream and few: 131072 weight rows (32 experts of 4096), 1 row of each expert 66
  // and 69 us, 4 rows 95 and 109, 16 rows 160 and 178; 114688 (16 of 7168) 65 and 61, 88 and 96, 133 and 145; 100352 (14 of 7168) 60 and
  // 56, 84 and 85, 129 and 136.  One row of each expert changes sides at some 120000, more rows below 100000: the border suits those.
  // A workgroup of the few-rows kernel has 32 weight rows or, where that gives too few workgroups, 16.  K = 7168, 32 and 16: 10000
  // weight rows (2 experts), 1 row 8.5 and 8.2, 4 rows 11.1 and 10.4; 16384 in 8 experts 11.7 and 9.8, 14.4 and 16.9, in one 12.8 and 15.9,
  // 13.5 and 16.1; 32768 in 16 experts 18.8 and 19.8, 32.7 and 37.1.  One border for all of them is coarse: up to a sixth either way
  // between 8192 and 16384.
  const long long weight_rows = (long long)g.groups * g.N * (act ? 2 : 1);
  if (weight_rows >= 98304) return go(w4_stream_kernel<XT, FMT, SIZE, FOLD, 2>, (int)wide, 256, 16);
  if (act || weight_rows > 8192) return go(w4_few_kernel<XT, FMT, SIZE, FOLD, 2, 4>, act ? 16 : 32, 256, 16);
  return go(w4_few_kernel<XT, FMT, SIZE, FOLD, 1, 4>, 16, 256, 16);
}

template <typename XT, int SIZE>
hipError_t int4_by_group(const W4GemmArgs& g, hipStream_t s) {
  if (g.G == 32) return launch<XT, kInt4, SIZE, 1>(g, s);
  if (g.G == 64) return launch<XT, kInt4, SIZE, 2>(g, s);
  if (g.G == 128) return launch<XT, kInt4, SIZE, 4>(g, s);
  return launch<XT, kInt4, SIZE, 8>(g, s);
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
