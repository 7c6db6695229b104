// Tokens sorted by expert and brought back with their routing weights, and both gradients.
//
// With r(t, j) = slot_to_row[t k + j], the row of slot j of token t (none when the slot's expert is
// not local, or its row lies at or past the rows the caller's tensors hold):
//   dispatch           xs[r(t, j)] = x[t]
//   dispatch backward  dx[t]       = sum_j dxs[r(t, j)]
//   combine            y[t]        = sum_j w[t, j] ys[r(t, j)]
//   combine backward   dys[r(t, j)] = w[t, j] dy[t],   dw[t, j] = <dy[t], ys[r(t, j)]> (0: no row)
//                      dlogits[t, e] = sum over j with ids[t, j] = e of w_j (dw_j - sum_i w_i dw_i)
// Every sum is taken in float32 in slot order (the dot products: per lane, then over lanes, then over
// waves, all in a fixed order) and rounded once to the tensors' type; every output element has one
// writer, so results do not depend on scheduling.
//
// All four move rows and do next to no arithmetic: what bounds them is HBM (large calls) or the
// latency of one chain map -> row -> store (small ones).  A workgroup takes one token at a time, or,
// where rows are short, each wave or pair of waves one of its own: the first k lanes of every wave load
// its map entries in one instruction, a ballot compacts the slots that have a row, and the row loads are
// issued before any of them is used.
#include <hip/hip_runtime.h>
#include <cstdint>

#include "device_common.hpp"
#include "elem.hpp"
#include "operators.hpp"

namespace moe {

// The rows of the first n slots of token t, in lane j's register for slot j (any wave); the mask has bit j
// set when slot j has a row below max_rows (a map entry outside [0, max_rows) counts as none).
__device__ __forceinline__ uint64_t token_rows(const int32_t* __restrict__ s2r, long long t, int k, int n, int max_rows,
                                               int lane, int& row) {
  row = lane < n ? s2r[t * k + lane] : -1;
  return __ballot((unsigned)row < (unsigned)max_rows);
}

// grid (column chunks, tokens): 256 threads on 1, 2 or 4 tokens, PER 16-byte chunks of a row each, read once
// and stored to every row the token has (a kernel by rows would read a token up to k times).  128 tokens of
// 14 KB, 125 rows: 2.5 to 3 us, the latency of map -> row -> store; 4096 tokens, 4136 rows: 16 us, 7.3 TB/s from the
// caches, 30900 rows: 98 us, 5.1 TB/s; 32768 tokens, 32600 rows of 21600 of them: 152 us, 5.1 TB/s.
template <int PER>
__global__ __launch_bounds__(256) void dispatch_kernel(const uint8_t* __restrict__ x, long long x_pitch,
                                                       const int32_t* __restrict__ s2r, int T, int k, int max_rows,
                                                       int waves_log2, long long row_bytes, uint8_t* __restrict__ xs,
                                                       long long xs_pitch) {
  const int lane = threadIdx.x & 63, lanes = 64 << waves_log2, pitch = lanes * 16;
  const long long c0 = ((long long)blockIdx.x * (lanes * PER) + (threadIdx.x & (lanes - 1))) * 16;
  // the row's last, partial chunk, where it is one of this lane's
  long long last = row_bytes;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (c0 + i * pitch == (row_bytes & ~15LL)) last = c0 + i * pitch;
  const int tg = __builtin_amdgcn_readfirstlane(threadIdx.x >> (6 + waves_log2)), tokens = 4 >> waves_log2;
  for (int t0 = blockIdx.y * tokens; t0 < T; t0 += gridDim.y * tokens) {
    const int t = t0 + tg;
    int row;
    if (t >= T) break;
    uint64_t mask = token_rows(s2r, t, k, k, max_rows, lane, row);
    if (mask == 0) continue;
    const uint8_t* src = x + (long long)t * x_pitch;
    u32x4 v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (c0 + i * pitch + 16 <= row_bytes) v[i] = load16(src + c0 + i * pitch);
    while (mask) {
      const int j = __builtin_ctzll(mask);
      mask &= mask - 1;
      uint8_t* dst = xs + (long long)__builtin_amdgcn_readlane(row, j) * xs_pitch;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (c0 + i * pitch + 16 <= row_bytes) store16(dst + c0 + i * pitch, v[i]);
      if (last < row_bytes)
        for (long long b = last; b < row_bytes; ++b) dst[b] = src[b];
    }
  }
}

// y[t] = sum over the token's rows of weight * row (WEIGHTED) or of the rows themselves.
// grid (column chunks, tokens): 256 threads on 1, 2 or 4 tokens, one 16-byte chunk each; the rows are taken four at a
// time, their loads issued before the sum.  32768 tokens of 7168 bfloat16 values with 32700 rows:
// 193 to 200 us, 4.7 to 4.9 TB/s, what a copy of 2 GiB reaches; 4097 tokens of 2050 float32 values, 4 rows each:
// 34 us, 4.9 TB/s; one token: 3.0 to 3.3 us.
template <typename T, bool WEIGHTED>
__global__ __launch_bounds__(256) void combine_rows_kernel(const T* __restrict__ ys, long long ys_stride,
                                                           const int32_t* __restrict__ s2r,
                                                           const float* __restrict__ w, int ntok, int k, int max_rows,
                                                           int waves_log2, int H, T* __restrict__ y,
                                                           long long y_stride) {
  constexpr int V = Elem<T>::kVec;
  const int lane = threadIdx.x & 63, lanes = 64 << waves_log2;
  const int c = (blockIdx.x * lanes + (threadIdx.x & (lanes - 1))) * V;
  const bool whole = c + V <= H;
  const int tg = __builtin_amdgcn_readfirstlane(threadIdx.x >> (6 + waves_log2)), tokens = 4 >> waves_log2;
  for (int t0 = blockIdx.y * tokens; t0 < ntok; t0 += gridDim.y * tokens) {
    const int t = t0 + tg;
    if (t >= ntok) break;
    int row;
    uint64_t mask = token_rows(s2r, t, k, k, max_rows, lane, row);
    const float wl = WEIGHTED && lane < k ? w[(long long)t * k + lane] : 1.f;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    while (mask) {
      long long src[4];
      float wt[4];
      int n = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (mask) {
          const int j = __builtin_ctzll(mask);
          mask &= mask - 1;
          src[q] = (long long)__builtin_amdgcn_readlane(row, j) * ys_stride + c;
          wt[q] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), j));
          n = q + 1;
        }
      if (whole) {
        u32x4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < n) v[q] = load16(ys + src[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < n) {
            float f[V];
            Elem<T>::unpack(v[q], f);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = WEIGHTED ? fmaf(wt[q], f[i], acc[i]) : acc[i] + f[i];
          }
      } else if (c < H) {
        for (int q = 0; q < n; ++q)
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (c + i < H) {
              const float f = Elem<T>::get(ys[src[q] + i]);
              acc[i] = WEIGHTED ? fmaf(wt[q], f, acc[i]) : acc[i] + f;
            }
      }
    }
    T* dst = y + (long long)t * y_stride + c;
    if (whole) {
      store16(dst, pack16<T>(acc));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < H) dst[i] = Elem<T>::put(acc[i]);
    }
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// G groups of NW waves in a workgroup, each with a token of its own.  With n rows the waves of a group
// split into n parts of P = NW / n: each part takes one row, each of its waves every P-th 64-chunk piece
// of it, so the work is spread whether a token has one local row or all k of them.  (n > NW: the waves
// take the rows in turn.)  dy is read by every part, from the L1 after the first.  16384 tokens of 4096 bfloat16 values, 8 rows each:
// 454 to 461 us, 5.0 TB/s, what a copy reaches; 512 tokens of 2048 float16 values, 4 rows each: 6.6 us.
template <typename T, int NW, int G>
__global__ __launch_bounds__(NW * G * 64) void combine_backward_kernel(
    const T* __restrict__ dy, long long dy_stride, const T* __restrict__ ys, long long row_stride,
    const int32_t* __restrict__ s2r, const float* __restrict__ w, int ntok, int k, int max_rows, int H,
    T* __restrict__ dys, float* __restrict__ dw, const int32_t* __restrict__ ids, int E, float* __restrict__ dlogits) {
  constexpr int V = Elem<T>::kVec, U = 4;  // chunks in flight per lane
  __shared__ float part[NW > 1 ? G : 1][16][NW];  // [token][slot][wave of its part]
  __shared__ float gs[NW > 1 ? G : 1][16];
  __shared__ int gids[NW > 1 ? G : 1][16];
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), tg = wid / NW, wave = wid % NW;
  const int nchunk = H / V;  // whole 16-byte chunks of a row
  for (int t0 = blockIdx.x * G; t0 < ntok; t0 += gridDim.x * G) {
    const int t = t0 + tg;
    const bool live = t < ntok;
    int row;
    const uint64_t mask = token_rows(s2r, live ? t : 0, k, live ? k : 0, max_rows, lane, row);
    const float wl = live && lane < k ? w[(long long)t * k + lane] : 0.f;
    const int n = __popcll(mask);
    const int P = n == 0 ? 1 : n < NW ? NW / n : 1;
    const T* dyt = dy + (long long)t * dy_stride;
    float d = 0.f;  // lane j: the dot product of slot j
    for (int q = wave / P; q < n; q += NW / P) {  // q-th slot with a row; one pass unless n > NW
      uint64_t m = mask;
      for (int i = 0; i < q; ++i) m &= m - 1;
      const int j = __builtin_ctzll(m), p = wave % P;
      const long long r = __builtin_amdgcn_readlane(row, j);
      const float wt = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), j));
      const T* src = ys + r * row_stride;
      T* dst = dys + r * row_stride;
      float dot = 0.f;
      for (int c0 = p * 64 + lane; c0 < nchunk; c0 += P * 64 * U) {
        u32x4 a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * P * 64;
          if (c < nchunk) {
            a[u] = load16(dyt + (long long)c * V);
            b[u] = load16(src + (long long)c * V);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int c = c0 + u * P * 64;
          if (c < nchunk) {
            float fa[V], fb[V], o[V];
            Elem<T>::unpack(a[u], fa);
            Elem<T>::unpack(b[u], fb);
#pragma unroll
            for (int i = 0; i < V; ++i) {
              dot = fmaf(fa[i], fb[i], dot);
              o[i] = wt * fa[i];
            }
            store16(dst + (long long)c * V, pack16<T>(o));
          }
        }
      }
      if (p == 0) {  // the elements after the last whole chunk
        const int c = nchunk * V + lane;
        if (c < H) {
          const float fa = Elem<T>::get(dyt[c]);
          dot = fmaf(fa, Elem<T>::get(src[c]), dot);
          dst[c] = Elem<T>::put(wt * fa);
        }
      }
      dot = wave_sum(dot);
      if (NW == 1)
        d = lane == j ? dot : d;
      else if (lane == 0)
        part[tg][j][p] = dot;
    }
    if (NW > 1) __syncthreads();
    float gl = 0.f;
    int id = 0;
    if (wave == 0 && live) {
      if (NW > 1 && lane < k && ((mask >> lane) & 1))
        for (int p = 0; p < P; ++p) d += part[tg][lane][p];
      if (lane < k) dw[(long long)t * k + lane] = d;
      if (dlogits != nullptr) {
        float s = 0.f;  // sum_i w_i dw_i in slot order, over the slots with a row: w may be anything on the others
        for (uint64_t m = mask; m; m &= m - 1) {
          const int i = __builtin_ctzll(m);
          s = fmaf(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wl), i)),
                   __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(d), i)), s);
        }
        if (lane < k) {
          gl = wl * (d - s);
          id = ids[(long long)t * k + lane];
          if (NW > 1) {
            gs[tg][lane] = gl;
            gids[tg][lane] = id;
          }
        }
      }
    }
    if (NW > 1) __syncthreads();
    if (dlogits != nullptr && live) {
      float* out = dlogits + (long long)t * E;
      for (int e = wave * 64 + lane; e < E; e += NW * 64) {
        float v = 0.f;
        for (int i = 0; i < k; ++i) {
          const int at = NW > 1 ? gids[tg][i] : __builtin_amdgcn_readlane(id, i);
          const float x = NW > 1 ? gs[tg][i] : __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(gl), i));
          v += at == e ? x : 0.f;
        }
        out[e] = v;
      }
    }
    // part, gs and gids are rewritten only after the next tokens' barriers: part before the first
    // (its readers, each group's wave 0, are past the second), gs and gids between them
    if (NW > 1) __syncthreads();
  }
}

// log2 of the waves a token's row of that many 16-byte chunks takes in dispatch and combine: 1, 2 or all 4 of a
// workgroup.  32768 tokens of 512 bfloat16 values, 2 rows each: 16 and 17 us; with 4 waves each 25 and 28.
static int waves_log2(long long chunks) { return chunks <= 64 ? 0 : chunks <= 128 ? 1 : 2; }

// workgroups for T tokens, `tokens` in each at a time (the kernels' loops stay in 32 bits past the last one)
static unsigned token_grid(int T, int tokens) {
  const int n = (T + tokens - 1) / tokens, most = 65535 / tokens;
  return (unsigned)(n < most ? n : most);
}

hipError_t launch_dispatch(const DispatchShape& d, const void* x, const int32_t* s2r, void* xs, hipStream_t s) {
  const long long es = dtype_bytes(d.dtype), row_bytes = (long long)d.H * es;
  const int wl = waves_log2((row_bytes + 15) / 16);
  const auto launch = [&](auto kern, int per) {
    const long long cols = (1024LL << wl) * per;
    const dim3 grid((unsigned)((row_bytes + cols - 1) / cols), token_grid(d.T, 4 >> wl));
    kern<<<grid, 256, 0, s>>>(static_cast<const uint8_t*>(x), d.token_stride * es, s2r, d.T, d.k, d.max_rows, wl,
                              row_bytes, static_cast<uint8_t*>(xs), d.row_stride * es);
    return hipGetLastError();
  };
  // few tokens: one chunk per thread, as many workgroups as can be (128 tokens of 14 KB 2.5 us, with four 4.0;
  // 1024: 5.8 and 6.0); many: a workgroup per 16 KB, which most tokens of an expert share leave at once (4096
  // tokens of 14 KB, 249 rows: 4.8 us, with one chunk 9.1; 4136 rows: 16.3 and 17.5)
  return d.T <= 1024 ? launch(dispatch_kernel<1>, 1) : launch(dispatch_kernel<4>, 4);
}

template <typename T, bool WEIGHTED>
static hipError_t combine_rows(const DispatchShape& d, const void* ys, const int32_t* s2r, const float* w, void* y,
                               hipStream_t s) {
  constexpr int V = Elem<T>::kVec;
  const int wl = waves_log2((d.H + V - 1) / V), cols = (64 << wl) * V;
  const dim3 grid((unsigned)((d.H + cols - 1) / cols), token_grid(d.T, 4 >> wl));
  combine_rows_kernel<T, WEIGHTED><<<grid, 256, 0, s>>>(
      static_cast<const T*>(ys), d.row_stride, s2r, w, d.T, d.k, d.max_rows, wl, d.H, static_cast<T*>(y),
      d.token_stride);
  return hipGetLastError();
}

hipError_t launch_combine_rows(const DispatchShape& d, const void* ys, const int32_t* s2r, const float* w, void* y,
                               hipStream_t s) {
  if (d.dtype == 0) return w ? combine_rows<Bf16, true>(d, ys, s2r, w, y, s) : combine_rows<Bf16, false>(d, ys, s2r, w, y, s);
  if (d.dtype == 1) return w ? combine_rows<F16, true>(d, ys, s2r, w, y, s) : combine_rows<F16, false>(d, ys, s2r, w, y, s);
  return w ? combine_rows<float, true>(d, ys, s2r, w, y, s) : combine_rows<float, false>(d, ys, s2r, w, y, s);
}

template <typename T>
static hipError_t combine_backward(const DispatchShape& d, const void* dy, const void* ys, const int32_t* s2r,
                                   const float* w, void* dys, float* dw, const int32_t* ids, float* dlogits,
                                   hipStream_t s) {
  const auto launch = [&](auto kern, int waves, int tokens) {
    kern<<<token_grid(d.T, tokens), waves * tokens * 64, 0, s>>>(
        static_cast<const T*>(dy), d.token_stride, static_cast<const T*>(ys), d.row_stride, s2r, w, d.T, d.k,
        d.max_rows, d.H, static_cast<T*>(dys), dw, ids, d.E, dlogits);
    return hipGetLastError();
  };
  // A wave takes a token by itself where the token's rows are at most 512 16-byte chunks (8 per lane) and there are
  // tokens enough to fill the GPU: 32768 tokens of 512 bfloat16 values, 2 rows each, 27 instead of 99 us; 2048 tokens
  // of 512, 4 rows each, 6.2 instead of 8.9.  (1024 tokens of 512, 8 rows each: 8.3, with eight waves 6.4; 16384
  // tokens of 2048, 4 rows each: 122, with eight waves 115.)
  const long long chunks = (long long)d.k * ((d.H + Elem<T>::kVec - 1) / Elem<T>::kVec);
  if (d.T >= 2048 && chunks <= 512) return launch(combine_backward_kernel<T, 1, 4>, 1, 4);
  return launch(combine_backward_kernel<T, 8, 1>, 8, 1);
}

hipError_t launch_combine_backward(const DispatchShape& d, const void* dy, const void* ys, const int32_t* s2r,
                                   const float* w, void* dys, float* dw, const int32_t* ids, float* dlogits,
                                   hipStream_t s) {
  if (d.dtype == 0) return combine_backward<Bf16>(d, dy, ys, s2r, w, dys, dw, ids, dlogits, s);
  if (d.dtype == 1) return combine_backward<F16>(d, dy, ys, s2r, w, dys, dw, ids, dlogits, s);
  return combine_backward<float>(d, dy, ys, s2r, w, dys, dw, ids, dlogits, s);
}

}  // namespace moe
