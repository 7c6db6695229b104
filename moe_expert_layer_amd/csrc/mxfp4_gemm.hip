// Grouped product of MXFP4 rows with MXFP4 weights (E2M1 values, one UE8M0 scale per 32 along K):
//   C[r, n] = sum_k A[r, k] * B[e, n, k]   for the rows r of group e, offsets[e] <= r < offsets[e + 1]
// on the scaled FP4 matrix instructions, which multiply the codes, apply both blocks' scales and sum
// in float32 (measured: within 2e-7 of the exact sum, as a sequential float32 sum is, for scales
// spread over 2^20).  The result is rounded once to C's type.
//
// A lane of the 16x16x128 instruction holds one 32-wide block of one row: row lane % 16, block
// lane / 16 of four.  Since the sum over K takes its blocks in any order, as long as both operands
// take the same, quarter q of the lanes works through the four blocks of the 128-wide scale word q of
// a 512-wide stretch in four instructions: a lane then needs one scale word and one 64-byte run of
// codes per operand row and stretch, and names the byte of the word in the instruction.
#include <hip/hip_runtime.h>
#include <cstdint>

#include "device_common.hpp"
#include "elem.hpp"
#include "moe_internal.hpp"

namespace moe {

// the rows of group e, inside [0, rows) whatever the offsets hold
__device__ __forceinline__ int2 group_rows(const int32_t* __restrict__ offsets, int e, int rows) {
  if (offsets == nullptr) return make_int2(0, rows);
  const int lo = min(max(offsets[e], 0), rows);
  return make_int2(lo, min(max(offsets[e + 1], lo), rows));
}

__device__ __forceinline__ v8i fp4_operand(uint4 q) {
  return v8i{(int)q.x, (int)q.y, (int)q.z, (int)q.w, 0, 0, 0, 0};
}

// One group's 16 * NS weight rows against MT * 16 token rows at a time; the NW waves take every
// NW-th 512-wide stretch of K and their partial sums meet in LDS, in wave order.
template <typename T, int NW, int NS, int MT>
__global__ __launch_bounds__(NW * 64) void mxfp4_gemm_rows_kernel(Mxfp4GemmArgs g) {
  __shared__ float part[NW][MT * 16][NS * 16 + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.y, n0 = blockIdx.x * (NS * 16);
  const int2 rr = group_rows(g.offsets, e, g.rows);
  const int r16 = lane & 15, q = lane >> 4;
  const int nblk = g.K / 32, nwords = (nblk + 3) / 4, nst = (nwords + 3) / 4;
  const long long ld = g.K / 2;
  const uint8_t* bp[NS];
  const uint8_t* bs[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const long long row = (long long)e * g.N + min(n0 + s * 16 + r16, g.N - 1);
    bp[s] = g.B + row * ld;
    bs[s] = g.B_sf + row * g.b_row_mul;
  }
  for (int m0 = rr.x; m0 < rr.y; m0 += MT * 16) {
    const uint8_t* ap[MT];
    const uint8_t* as[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const long long row = min(m0 + m * 16 + r16, rr.y - 1);
      ap[m] = g.A + row * ld;
      as[m] = g.A_sf + row * g.a_row_mul;
    }
    v4f acc[MT][NS];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < NS; ++s) acc[m][s] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int st = wave; st < nst; st += NW) {
      const int j = st * 4 + q;  // this lane's scale word
      const int jc = min(j, nwords - 1);
      const int left = nblk - 4 * j;  // blocks of the word inside K (<= 0: none)
      int sa[MT], sb[NS];
#pragma unroll
      for (int m = 0; m < MT; ++m) sa[m] = *reinterpret_cast<const int*>(as[m] + (long long)jc * g.a_word_mul);
#pragma unroll
      for (int s = 0; s < NS; ++s) sb[s] = *reinterpret_cast<const int*>(bs[s] + (long long)jc * g.b_word_mul);
      uint4 a[MT][4], b[NS][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const long long at = i < left ? (long long)j * 64 + i * 16 : 0;
#pragma unroll
        for (int m = 0; m < MT; ++m) a[m][i] = *reinterpret_cast<const uint4*>(ap[m] + at);
#pragma unroll
        for (int s = 0; s < NS; ++s) b[s][i] = *reinterpret_cast<const uint4*>(bp[s] + at);
      }
      if (left < 4) {  // past K: zero codes and scales of 1
        const int keep = left <= 0 ? 0 : (1 << (8 * left)) - 1;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          sa[m] = (sa[m] & keep) | (0x7f7f7f7f & ~keep);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i >= left) a[m][i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) sb[s] = (sb[s] & keep) | (0x7f7f7f7f & ~keep);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          // the scale byte's index is an immediate
          acc[m][s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][0]), fp4_operand(b[s][0]),
                                                                       acc[m][s], 4, 4, 0, sa[m], 0, sb[s]);
          acc[m][s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][1]), fp4_operand(b[s][1]),
                                                                       acc[m][s], 4, 4, 1, sa[m], 1, sb[s]);
          acc[m][s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][2]), fp4_operand(b[s][2]),
                                                                       acc[m][s], 4, 4, 2, sa[m], 2, sb[s]);
          acc[m][s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a[m][3]), fp4_operand(b[s][3]),
                                                                       acc[m][s], 4, 4, 3, sa[m], 3, sb[s]);
        }
    }
    // lane holds rows 4 q + i, column r16 of each 16 x 16 tile
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[wave][m * 16 + 4 * q + i][s * 16 + r16] = acc[m][s][i];
    __syncthreads();
    for (int i = tid; i < MT * 16 * NS * 16; i += NW * 64) {
      const int r = i / (NS * 16), c = i % (NS * 16);
      float v = part[0][r][c];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += part[w][r][c];
      if (m0 + r < rr.y && n0 + c < g.N)
        static_cast<T*>(g.C)[(long long)(m0 + r) * g.c_stride + n0 + c] = Elem<T>::put(v);
    }
    __syncthreads();
  }
}

template <typename T>
static hipError_t launch(const Mxfp4GemmArgs& g, hipStream_t s) {
  mxfp4_gemm_rows_kernel<T, 4, 2, 2><<<dim3((unsigned)((g.N + 31) / 32), (unsigned)g.groups), 256, 0, s>>>(g);
  return hipGetLastError();
}

hipError_t launch_mxfp4_gemm(const Mxfp4GemmArgs& g, int out_dtype, int variant, hipStream_t s) {
  (void)variant;
  if (out_dtype == 0) return launch<Bf16>(g, s);
  if (out_dtype == 1) return launch<F16>(g, s);
  return launch<float>(g, s);
}

}  // namespace moe
