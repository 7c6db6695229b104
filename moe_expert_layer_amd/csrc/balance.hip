// The router's balance loss: per-expert counts, probability sums, the loss of each sequence, and the gradient of the
// routing logits.
//
// With p[t, e] a token's probabilities (the softmax of its logits, or their sigmoids over the sum of them), c[s, e] how
// often the N_s tokens of sequence s chose expert e, and P[s, e] the sum of their p[t, e]:
//   balance[s] = E / (k N_s^2) sum_e c[s, e] P[s, e]          z[s] = 1 / N_s sum_t (log sum_e exp l[t, e])^2
//   dl[t, e]   = g E / (k N_s^2) p q (c[s, e] - sum_i p_i c[s, i]) + gz 2 / N_s p lse
// with q = 1, or 1 - sigmoid(l) where the probabilities are sigmoids over their sum.  The probabilities sum to 1, so
// that difference is the same with any constant taken off every count: k N_s / E, their mean, is taken off in whole
// numbers first, which keeps the bits that counts near their mean would cancel.
//
// Both directions read the logits once, and the gradient writes as many values: HBM bounds the large calls, the latency of a
// launch the small ones.  A group of LPT lanes holds a token, R chunks of four columns each: with 16 lanes (64
// columns a chunk row) a token's maximum and sum are four DPP steps each, for four tokens of a wave at once; a whole wave on a
// token would take six steps for one.  Sums over tokens stay in the lanes' registers, over all tokens that a lane sees
// of a piece (the tokens of one workgroup's chunk in one sequence), then over a wave's groups, then over waves.
//
// 65536 tokens of 256 float32 logits: forward 22 us, some 6.5 of them to join the pieces (14 us at a copy's rate), gradient with another one added
// to it 39 us (41); 128 tokens of 32: 3.6 us, 6.2 to 6.8 with the call.
#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

#include "elem.hpp"
#include "operators.hpp"

namespace moe {

namespace {

constexpr float kLog2e = 1.44269504088896341f;

// value with the one of the lane that a DPP control names
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, false));
}

// maximum and sum over a group of LPT lanes, the same bits in each of them
template <int LPT>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));                       // quad_perm [1,0,3,2]
  v = fmaxf(v, dpp<0x4E>(v));                       // quad_perm [2,3,0,1]
  if constexpr (LPT >= 8) v = fmaxf(v, dpp<0x141>(v));   // row_half_mirror: the other quad of 8
  if constexpr (LPT >= 16) v = fmaxf(v, dpp<0x140>(v));  // row_mirror: the other 8 of 16
  if constexpr (LPT == 64) v = fmaxf(v, __shfl_xor(v, 16));
  if constexpr (LPT == 64) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}
template <int LPT>
__device__ __forceinline__ float group_sum(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  if constexpr (LPT >= 8) v += dpp<0x141>(v);
  if constexpr (LPT >= 16) v += dpp<0x140>(v);
  if constexpr (LPT == 64) v += __shfl_xor(v, 16);
  if constexpr (LPT == 64) v += __shfl_xor(v, 32);
  return v;
}

// Four consecutive logits at any alignment of their elements, as loaded and as float32
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <typename T> struct Quad {  // 16-bit types
  typedef u32x2 raw;
  typedef u32x2 at2 __attribute__((aligned(2)));
  static __device__ __forceinline__ raw load(const T* p) { return *reinterpret_cast<const at2*>(p); }
  static __device__ __forceinline__ void get(raw v, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = Elem<T>::get(T{(uint16_t)(v[i >> 1] >> (16 * (i & 1)))});
  }
};

template <> struct Quad<float> {
  typedef u32x4 raw;
  static __device__ __forceinline__ raw load(const float* p) { return load16(p); }
  static __device__ __forceinline__ void get(raw v, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
};

// A group's columns: chunk g + r LPT holds columns 4 c .. 4 c + 3.  The last chunk of a row whose length is no multiple
// of four is read as the row's last four columns, of which the first ones belong to the chunk before it; rows of
// less than four columns are read one by one.
template <typename T, int LPT, int R>
struct Columns {
  int base[R];     // first column read
  unsigned live;   // bit 4 r + i: column base[r] + i is this lane's
  static_assert(R <= 8, "a bit for each column");
  __device__ __forceinline__ void init(int E, int g) {
    live = 0;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = 4 * (g + r * LPT);
      base[r] = c + 4 <= E ? c : E >= 4 ? E - 4 : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (base[r] + i >= c && base[r] + i < E) live |= 1u << (4 * r + i);
    }
  }
  __device__ __forceinline__ bool has(int r, int i) const { return (live >> (4 * r + i)) & 1; }
  __device__ __forceinline__ void load(const T* row, int E, typename Quad<T>::raw (&v)[R]) const {
    if (E >= 4) {
#pragma unroll
      for (int r = 0; r < R; ++r) v[r] = Quad<T>::load(row + base[r]);
    } else {
      T e[8 / sizeof(T) * 2] = {};
      for (int i = 0; i < 4; ++i)
        if (i < E) e[i] = row[i];
      v[0] = Quad<T>::load(e);
    }
  }
};

// One token's probabilities.  x: logits, -inf in columns that are not this lane's; on return p[r][i] unscaled
// and 1 / their sum (0 where every logit is -inf).  The difference to the largest logit, its product with log2 e and that constant are
// float32, so an exponential is off by up to some 2.3 |x - m| 2^-24 of itself (1.3 where x - m is exact), which is most for the
// shares that matter least; a base-2 exponent in two parts would take that off for some four more vector instructions a logit.
template <int LPT, int R>
__device__ __forceinline__ float probabilities(const float (&x)[R][4], float (&p)[R][4], bool sigmoid, float& top,
                                               float& sum) {
  float m = x[0][0];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, x[r][i]);
  m = group_max<LPT>(m);
  m = m == -INFINITY ? 0.f : m;
  float n = 0.f;
  if (!sigmoid) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[r][i] = __builtin_amdgcn_exp2f((x[r][i] - m) * kLog2e);
        n += p[r][i];
      }
  } else {
    // sigmoid(l) e^-c with c = min(m, 0), the numerator e^(min(l, 0) - c), so that tokens whose sigmoids all
    // underflow keep their shares
    const float c = fminf(m, 0.f);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float l = x[r][i], t = __builtin_amdgcn_exp2f(-fabsf(l) * kLog2e);
        const float low = l > 0.f ? 0.f : l;  // NaN stays
        p[r][i] = __builtin_amdgcn_exp2f((low - c) * kLog2e) * __builtin_amdgcn_rcpf(1.f + t);
        n += p[r][i];
      }
  }
  n = group_sum<LPT>(n);
  top = m;
  sum = n;
  return n == 0.f ? 0.f : 1.f / n;
}

// the sequence that holds token t: the number of offsets[1..S] at or below it (S: none)
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ offsets, int S, int t) {
  if (offsets == nullptr) return 0;
  int lo = 0, hi = S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ int2 sequence(const int32_t* __restrict__ offsets, int s, int T) {
  if (offsets == nullptr) return make_int2(0, T);
  const int lo = min(max(offsets[s], 0), T);
  return make_int2(lo, min(max(offsets[s + 1], lo), T));
}

// What a call leaves in its workspace: for each piece, a row of probability sums and one of counts, the sum of squared
// logarithms and the number of tokens.  Piece (chunk c, sequence s) is row c + s: going through the tokens, each
// next piece has the next chunk, a later sequence or both.
struct Parts {
  float* psum;    // [rows][E]
  int32_t* count;
  float* z;       // [rows]
  int32_t* n;
  double* loss;   // [S][slices]
  int32_t* done;  // [S]
};

constexpr int kSlice = 8;  // columns that a workgroup of the second kernel adds up, or 32

// A piece's tokens [a, b): probability sums, counts, sum of squared logarithms and tokens, in LDS (psum, hist) and in
// every thread (z, n).  A workgroup of NW waves, all of them here.
template <typename T, int LPT, int R, int NW>
struct Piece {
  static constexpr int GPW = 64 / LPT, TW = NW * GPW;  // tokens at a time
  float (*psum)[LPT * R * 4];                          // [NW]
  int32_t* hist;
  float* zs;    // [NW]
  int32_t* ns;  // [NW]

  __device__ __forceinline__ void run(const BalanceShape& b, const Columns<T, LPT, R>& cols, const T* __restrict__ logits,
                                      const int32_t* __restrict__ ids, const uint8_t* __restrict__ mask, int a, int e,
                                      bool want_z, float& z, int& n) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane & (LPT - 1);
    int t = a + wave * GPW + lane / LPT;
    typename Quad<T>::raw next[R] = {};
    bool counted = t < e && (mask == nullptr || mask[t]);
    if (t < e) cols.load(logits + (long long)t * b.logit_stride, b.E, next);
    for (int i = tid; i < b.E; i += NW * 64) hist[i] = 0;
    __syncthreads();
    for (long long i = (long long)a * b.k + tid; i < (long long)e * b.k; i += NW * 64) {
      const int id = ids[i];
      if ((unsigned)id < (unsigned)b.E && (mask == nullptr || mask[(unsigned)i / (unsigned)b.k])) atomicAdd(&hist[id], 1);
    }
    float acc[R][4], zacc = 0.f;
    int nacc = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][i] = 0.f;
    while (__any(t < e)) {
      float x[R][4], p[R][4], top, sum;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        Quad<T>::get(next[r], x[r]);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[r][i] = cols.has(r, i) ? x[r][i] : -INFINITY;
      }
      const bool use = counted;
      t += TW;
      counted = t < e && (mask == nullptr || mask[t]);
      if (t < e) cols.load(logits + (long long)t * b.logit_stride, b.E, next);
      const float inv = probabilities<LPT, R>(x, p, b.sigmoid, top, sum);
      if (use) {
        ++nacc;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][i] = fmaf(p[r][i], inv, acc[r][i]);
        if (want_z && sum != 0.f) {
          const float lse = top + logf(sum);
          zacc = fmaf(lse, lse, zacc);
        }
      }
    }
    // over the wave's groups, then over the waves
#pragma unroll
    for (int off = LPT; off < 64; off <<= 1) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][i] += __shfl_xor(acc[r][i], off);
      zacc += __shfl_xor(zacc, off);
      nacc += __shfl_xor(nacc, off);
    }
    if (lane < LPT) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (cols.has(r, i)) psum[wave][cols.base[r] + i] = acc[r][i];
    }
    if (lane == 0) {
      zs[wave] = zacc;
      ns[wave] = nacc;
    }
    __syncthreads();
    z = 0.f;
    n = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      z += zs[w];
      n += ns[w];
    }
  }
  __device__ __forceinline__ float sum(int e) const {
    float v = psum[0][e];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += psum[w][e];
    return v;
  }
};

template <typename T, int LPT, int R, int NW>
struct PieceLds {
  float psum[NW][LPT * R * 4];
  int32_t hist[LPT * R * 4];
  float zs[NW];
  int32_t ns[NW];
};

// workgroup c: the pieces of tokens [c C, c C + C)
template <typename T, int LPT, int R, int NW>
__global__ __launch_bounds__(NW * 64) void balance_parts_kernel(BalanceShape b, const T* __restrict__ logits,
                                                                const int32_t* __restrict__ ids,
                                                                const uint8_t* __restrict__ mask,
                                                                const int32_t* __restrict__ offsets, int C, bool want_z,
                                                                Parts parts) {
  __shared__ PieceLds<T, LPT, R, NW> lds;
  Piece<T, LPT, R, NW> piece{lds.psum, lds.hist, lds.zs, lds.ns};
  const int tid = threadIdx.x;
  Columns<T, LPT, R> cols;
  cols.init(b.E, tid & (LPT - 1));
  if (blockIdx.x == 0)
    for (int s = tid; s < b.S; s += NW * 64) parts.done[s] = 0;
  const int t0 = blockIdx.x * C, t1 = min(b.T - t0, C) + t0;
  for (int s = sequence_of(offsets, b.S, t0); s < b.S; ++s) {
    const int2 range = sequence(offsets, s, b.T);
    if (range.x >= t1) break;
    const int lo = max(range.x, t0), hi = min(range.y, t1);
    if (lo >= hi) continue;
    float z;
    int n;
    piece.run(b, cols, logits, ids, mask, lo, hi, want_z, z, n);
    const long long row = blockIdx.x + s;
    for (int e = tid; e < b.E; e += NW * 64) {
      parts.psum[row * b.E + e] = piece.sum(e);
      parts.count[row * b.E + e] = lds.hist[e];
    }
    if (tid == 0) {
      parts.z[row] = z;
      parts.n[row] = n;
    }
    __syncthreads();  // before the next piece writes LDS
  }
}

__device__ __forceinline__ double block_sum(double v, double* scratch, int waves) {
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < waves; ++w) v += scratch[w];
  return v;
}

__device__ __forceinline__ float balance_of(double cp, int E, int k, double n) {
  return n == 0.0 ? 0.f : (float)(cp * (double)E / ((double)k * n * n));
}

// workgroup (slice, s): sums the pieces of SL columns of sequence s, in float64; the last workgroup of a sequence to
// end adds up the slices' parts of its loss, in their order
template <int SL>
__global__ __launch_bounds__(512) void balance_join_kernel(BalanceShape b, const int32_t* __restrict__ offsets, int C,
                                                           Parts parts, int32_t* __restrict__ counts,
                                                           int32_t* __restrict__ tokens, float* __restrict__ psum,
                                                           float* __restrict__ balance, float* __restrict__ zloss) {
  constexpr int NR = 512 / SL;
  __shared__ double sums[NR][SL + 1];
  __shared__ int32_t cnts[NR][SL];
  __shared__ double scratch[8];
  __shared__ int last;
  const int tid = threadIdx.x, col = tid % SL, rl = tid / SL, s = blockIdx.y;
  const int e = blockIdx.x * SL + col;
  const int2 range = sequence(offsets, s, b.T);
  const int c0 = range.x / C, c1 = range.y > range.x ? (range.y - 1) / C + 1 : c0;
  double p = 0.0;
  int n = 0;
  if (e < b.E)
#pragma unroll 4
    for (int c = c0 + rl; c < c1; c += NR) {
      const long long row = c + s;
      p += (double)parts.psum[row * b.E + e];
      n += parts.count[row * b.E + e];
    }
  sums[rl][col] = p;
  cnts[rl][col] = n;
  __syncthreads();
  double part = 0.0;
  if (tid < SL) {
    for (int r = 1; r < NR; ++r) {
      p += sums[r][col];
      n += cnts[r][col];
    }
    if (e < b.E) {
      counts[(long long)s * b.E + e] = n;
      psum[(long long)s * b.E + e] = (float)p;
      part = (double)n * p;
    }
  }
  part = block_sum(part, scratch, 8);
  double* slot = parts.loss + (long long)s * gridDim.x;
  if (tid == 0) {
    __hip_atomic_store(slot + blockIdx.x, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = __hip_atomic_fetch_add(parts.done + s, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  double z = 0.0, nt = 0.0;
  for (int c = c0 + tid; c < c1; c += 512) {
    z += (double)parts.z[c + s];
    nt += (double)parts.n[c + s];
  }
  z = block_sum(z, scratch, 8);
  nt = block_sum(nt, scratch, 8);
  double cp = 0.0;
  for (unsigned i = tid; i < gridDim.x; i += 512) cp += __hip_atomic_load(slot + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  cp = block_sum(cp, scratch, 8);
  if (tid == 0) {
    tokens[s] = (int)nt;
    balance[s] = balance_of(cp, b.E, b.k, nt);
    if (zloss != nullptr) zloss[s] = nt == 0.0 ? 0.f : (float)(z / nt);
  }
}

// few tokens: workgroup s has a sequence to itself, and nothing to join
template <typename T, int LPT, int R, int NW>
__global__ __launch_bounds__(NW * 64) void balance_small_kernel(BalanceShape b, const T* __restrict__ logits,
                                                                const int32_t* __restrict__ ids,
                                                                const uint8_t* __restrict__ mask,
                                                                const int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ counts, int32_t* __restrict__ tokens,
                                                                float* __restrict__ psum, float* __restrict__ balance,
                                                                float* __restrict__ zloss) {
  __shared__ PieceLds<T, LPT, R, NW> lds;
  __shared__ double scratch[NW];
  Piece<T, LPT, R, NW> piece{lds.psum, lds.hist, lds.zs, lds.ns};
  const int tid = threadIdx.x, s = blockIdx.x;
  Columns<T, LPT, R> cols;
  cols.init(b.E, tid & (LPT - 1));
  const int2 range = sequence(offsets, s, b.T);
  float z;
  int n;
  piece.run(b, cols, logits, ids, mask, range.x, range.y, zloss != nullptr, z, n);
  double part = 0.0;
  for (int e = tid; e < b.E; e += NW * 64) {
    const float p = piece.sum(e);
    const int c = lds.hist[e];
    counts[(long long)s * b.E + e] = c;
    psum[(long long)s * b.E + e] = p;
    part += (double)c * (double)p;
  }
  part = block_sum(part, scratch, NW);
  if (tid == 0) {
    tokens[s] = n;
    balance[s] = balance_of(part, b.E, b.k, (double)n);
    if (zloss != nullptr) zloss[s] = n == 0 ? 0.f : (float)((double)z / (double)n);
  }
}

// Gradient: groups of LPT lanes take the workgroup's tokens in turn, and keep the counts of their sequence.  What is read or written once
// goes past the caches (65536 tokens of 256, 1024 workgroups: 47.4 -> 39.8 us; the logits too: 42.5, and the forward pass has just read them).
typedef u32x4 at4 __attribute__((aligned(4)));
template <typename T, int LPT, int R>
__global__ __launch_bounds__(256) void balance_backward_kernel(BalanceShape b, const T* __restrict__ logits,
                                                               const uint8_t* __restrict__ mask,
                                                               const int32_t* __restrict__ offsets,
                                                               const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ tokens,
                                                               const float* __restrict__ dbalance,
                                                               const float* __restrict__ dz, const float* add,
                                                               float* dlogits, int C) {
  constexpr int TW = 256 / LPT;
  const int g = threadIdx.x & (LPT - 1);
  const int t0 = blockIdx.x * C, t1 = min(b.T - t0, C) + t0;
  Columns<T, LPT, R> cols;
  cols.init(b.E, g);
  int t = t0 + threadIdx.x / LPT, s = -1, lo = 0, hi = 0;
  float w[R][4], wb = 0.f, wz = 0.f;
  typename Quad<T>::raw next[R] = {};
  if (t < t1) cols.load(logits + (long long)t * b.logit_stride, b.E, next);
  while (__any(t < t1)) {
    float x[R][4], p[R][4], top, sum;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      Quad<T>::get(next[r], x[r]);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[r][i] = cols.has(r, i) ? x[r][i] : -INFINITY;
    }
    const int now = t;
    t += TW;
    if (t < t1) cols.load(logits + (long long)t * b.logit_stride, b.E, next);
    bool counted = now < t1 && (mask == nullptr || mask[now]);
    if (counted && (s < 0 || now >= hi)) {  // another sequence's counts
      s = sequence_of(offsets, b.S, now);
      if (s < b.S) {
        const int2 range = sequence(offsets, s, b.T);
        lo = range.x;
        hi = range.y;
        const long long n = tokens[s] > 0 ? tokens[s] : 1, mean = n * b.k / b.E;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[r][i] = cols.has(r, i) ? (float)(counts[(long long)s * b.E + cols.base[r] + i] - mean) : 0.f;
        wb = (float)((double)dbalance[s] * b.E / ((double)b.k * n * n));
        wz = dz != nullptr ? (float)(2.0 * dz[s] / n) : 0.f;
      } else {
        lo = hi = b.T;  // behind the last sequence
      }
    }
    counted = counted && now >= lo && now < hi;
    const float inv = probabilities<LPT, R>(x, p, b.sigmoid, top, sum);
    float dot = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[r][i] *= inv;
        dot = counted ? fmaf(p[r][i], w[r][i], dot) : 0.f;
      }
    dot = group_sum<LPT>(dot);
    const float zl = dz != nullptr && sum != 0.f ? wz * (top + logf(sum)) : 0.f;
    if (now < t1) {
      float* out = dlogits + (long long)now * b.grad_stride;
      const float* in = add != nullptr ? add + (long long)now * b.grad_stride : nullptr;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float q = wb * (w[r][i] - dot);
          if (b.sigmoid) {  // 1 - sigmoid(l) = 1 / (1 + e^l)
            const float t = __builtin_amdgcn_exp2f(-fabsf(x[r][i]) * kLog2e);
            q *= (x[r][i] > 0.f ? t : 1.f) * __builtin_amdgcn_rcpf(1.f + t);
          }
          d[i] = counted ? p[r][i] * (q + zl) : 0.f;
        }
        if (((cols.live >> (4 * r)) & 15u) == 15u) {
          if (in != nullptr) {
            float f[4];
            Quad<float>::get(__builtin_nontemporal_load(reinterpret_cast<const at4*>(in + cols.base[r])), f);
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] += f[i];
          }
          __builtin_nontemporal_store(pack16<float>(d), reinterpret_cast<at4*>(out + cols.base[r]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (cols.has(r, i)) out[cols.base[r] + i] = d[i] + (in != nullptr ? in[cols.base[r] + i] : 0.f);
        }
      }
    }
  }
}

constexpr int kWaves = 8;     // waves of the forward kernels
// At most this many tokens: one workgroup a sequence, and no second kernel.  One sequence of float32 logits, in one workgroup and in pieces, us:
// 32 experts, 128 tokens 7.2 and 9.5, 512 7.6 and 9.5, 1024 12.3 and 9.5; 256 experts, 128 tokens 7.8 and 10.8, 256 11.8 and 10.9, 1024 36
// and 11; 1024 experts, 64 tokens 11.6 and 13, 128 19.5 and 13, 1024 131 and 14.  So one workgroup is the better up to eight rounds of the
// tokens that it takes at a time (128 with up to 16 experts, 8 above 512), and this border is far past that for many experts in one sequence;
// with many sequences their workgroups run side by side.
constexpr int kSmall = 1024;

// Tokens of a workgroup's chunk: for 256 chunks, one for each CU (256, 512, 1024 of them: 22, 24, 29 us for 65536 tokens of 256, the pieces being
// joined after), but no fewer than 32, which a workgroup takes at a time with 33 to 512 experts (128 with up to 16, 64 with up to 32, where
// some of its waves then have none, and 8 above), and no more than leave 1024 to the sums of one lane
int chunk_of(int T) {
  const long long c = ((long long)T + 255) / 256;
  return (int)(c < 32 ? 32 : c > 8192 ? 8192 : c);
}
int chunks_of(int T) { return (int)(((long long)T + chunk_of(T) - 1) / chunk_of(T)); }
// the most chunks that T tokens or fewer make, which is what the workspace holds: 8192 tokens are 256 chunks of 32, 8193 are 249 of 33
int most_chunks(int T) {
  const long long n = T <= 256 * 8192 ? ((long long)T + 31) / 32 : ((long long)T + 8191) / 8192;
  return (int)(T <= 256 * 8192 && n > 256 ? 256 : n);
}

// The shapes: columns a token's lanes hold.  f(lanes per token, chunks per lane)
template <int V> struct Int { static constexpr int value = V; };
template <typename F>
hipError_t by_columns(int E, F f) {
  if (E <= 16) return f(Int<4>(), Int<1>());
  if (E <= 32) return f(Int<8>(), Int<1>());
  if (E <= 64) return f(Int<16>(), Int<1>());
  if (E <= 128) return f(Int<16>(), Int<2>());
  if (E <= 192) return f(Int<16>(), Int<3>());
  if (E <= 256) return f(Int<16>(), Int<4>());
  if (E <= 384) return f(Int<16>(), Int<6>());
  if (E <= 512) return f(Int<16>(), Int<8>());
  return f(Int<64>(), Int<4>());
}

struct WorkspaceLayout {
  size_t psum, count, z, n, loss, done, total;
};
WorkspaceLayout layout_of(int T, int E, int S) {
  WorkspaceLayout L{};
  L.total = 256;  // never nothing: an allocator may give NULL for that, which the call refuses
  if (T <= kSmall) return L;
  const size_t rows = (size_t)most_chunks(T) + S;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  L.psum = take(rows * E * 4);
  L.count = take(rows * E * 4);
  L.z = take(rows * 4);
  L.n = take(rows * 4);
  L.loss = take((size_t)S * ((E + kSlice - 1) / kSlice) * 8);
  L.done = take((size_t)S * 4);
  L.total = at;
  return L;
}

template <typename T>
hipError_t forward(const BalanceShape& b, const void* logits, const int32_t* ids, const uint8_t* mask,
                   const int32_t* offsets, int32_t* counts, int32_t* tokens, float* psum, float* balance, float* z,
                   void* ws, hipStream_t s) {
  return by_columns(b.E, [&](auto lanes, auto chunks) {
    constexpr int LPT = decltype(lanes)::value, R = decltype(chunks)::value;
    const T* l = static_cast<const T*>(logits);
    if (b.T <= kSmall) {
      balance_small_kernel<T, LPT, R, kWaves><<<b.S, kWaves * 64, 0, s>>>(b, l, ids, mask, offsets, counts, tokens, psum,
                                                                          balance, z);
      return hipGetLastError();
    }
    const WorkspaceLayout L = layout_of(b.T, b.E, b.S);
    char* w = static_cast<char*>(ws);
    const Parts parts{reinterpret_cast<float*>(w + L.psum), reinterpret_cast<int32_t*>(w + L.count),
                      reinterpret_cast<float*>(w + L.z),    reinterpret_cast<int32_t*>(w + L.n),
                      reinterpret_cast<double*>(w + L.loss), reinterpret_cast<int32_t*>(w + L.done)};
    const int C = chunk_of(b.T);
    balance_parts_kernel<T, LPT, R, kWaves><<<chunks_of(b.T), kWaves * 64, 0, s>>>(b, l, ids, mask, offsets, C,
                                                                                  z != nullptr, parts);
    if (const hipError_t e = hipGetLastError()) return e;
    // Pieces in the hundreds for a sequence are read by more lanes a column (65536 tokens of 256 experts in one: 8 columns a workgroup 22 us
    // for the two kernels, 32 columns 31); of a few pieces it takes longer to join the slices (16385 tokens of 129 experts in 24: 22.5 us and 16.6)
    const auto join = [&](auto slice) {
      constexpr int SL = decltype(slice)::value;
      balance_join_kernel<SL><<<dim3((b.E + SL - 1) / SL, b.S), 512, 0, s>>>(b, offsets, C, parts, counts, tokens, psum, balance, z);
      return hipGetLastError();
    };
    return chunks_of(b.T) >= 64 * b.S ? join(Int<kSlice>()) : join(Int<32>());
  });
}

template <typename T>
hipError_t backward(const BalanceShape& b, const void* logits, const uint8_t* mask, const int32_t* offsets,
                    const int32_t* counts, const int32_t* tokens, const float* dbalance, const float* dz, const float* add,
                    float* dlogits, hipStream_t s) {
  return by_columns(b.E, [&](auto lanes, auto chunks) {
    constexpr int LPT = decltype(lanes)::value, R = decltype(chunks)::value;
    constexpr int TW = 256 / LPT;  // tokens a workgroup has at a time
    // four workgroups a CU, as many as the registers hold at once (65536 tokens of 256: 512, 1024, 1536, 2048, 4096 workgroups 52, 44, 51, 51,
    // 60 us)
    const long long c = ((long long)b.T + 1023) / 1024;
    const int C = (int)((c + TW - 1) / TW * TW);
    balance_backward_kernel<T, LPT, R><<<(unsigned)(((long long)b.T + C - 1) / C), 256, 0, s>>>(
        b, static_cast<const T*>(logits), mask, offsets, counts, tokens, dbalance, dz, add, dlogits, C);
    return hipGetLastError();
  });
}

}  // namespace

size_t balance_workspace(int T, int E, int S) { return layout_of(T, E, S).total; }

hipError_t launch_balance(const BalanceShape& b, const void* logits, const int32_t* ids, const uint8_t* mask,
                          const int32_t* offsets, int32_t* counts, int32_t* tokens, float* psum, float* balance, float* z,
                          void* ws, hipStream_t s) {
  if (b.dtype == 0) return forward<Bf16>(b, logits, ids, mask, offsets, counts, tokens, psum, balance, z, ws, s);
  if (b.dtype == 1) return forward<F16>(b, logits, ids, mask, offsets, counts, tokens, psum, balance, z, ws, s);
  return forward<float>(b, logits, ids, mask, offsets, counts, tokens, psum, balance, z, ws, s);
}

hipError_t launch_balance_backward(const BalanceShape& b, const void* logits, const uint8_t* mask, const int32_t* offsets,
                                   const int32_t* counts, const int32_t* tokens, const float* dbalance, const float* dz,
                                   const float* add, float* dlogits, hipStream_t s) {
  if (b.dtype == 0) return backward<Bf16>(b, logits, mask, offsets, counts, tokens, dbalance, dz, add, dlogits, s);
  if (b.dtype == 1) return backward<F16>(b, logits, mask, offsets, counts, tokens, dbalance, dz, add, dlogits, s);
  return backward<float>(b, logits, mask, offsets, counts, tokens, dbalance, dz, add, dlogits, s);
}

}  // namespace moe
