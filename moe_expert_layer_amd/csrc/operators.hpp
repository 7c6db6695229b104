// Internal launch interface of the operators beside the layer.  Apart from the layer's own, so that a change here
// leaves the layer's kernels, and what was measured of them, as they are.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace moe {

// tokens in expert order and back ----------------------------------------------
// dtype: moe_dtype (0 bf16, 1 f16, 2 f32, 3 bytes); strides in elements; a map entry outside
// [0, max_rows) means the slot has no row
struct DispatchShape {
  int T, H, E, k, dtype, max_rows;
  long long token_stride, row_stride;
};
constexpr long long dtype_bytes(int dtype) { return dtype == 2 ? 4 : dtype == 3 ? 1 : 2; }
hipError_t launch_dispatch(const DispatchShape& d, const void* x, const int32_t* slot_to_row, void* xs, hipStream_t s);
// w null: the plain sum of the token's rows (the gradient of launch_dispatch)
hipError_t launch_combine_rows(const DispatchShape& d, const void* ys, const int32_t* slot_to_row, const float* w,
                               void* y, hipStream_t s);
hipError_t launch_combine_backward(const DispatchShape& d, const void* dy, const void* ys, const int32_t* slot_to_row,
                                   const float* w, void* dys, float* dw, const int32_t* ids, float* dlogits,
                                   hipStream_t s);

// microscaled 4-bit floating point ------------------------------------------------
// AM: 0 for row-major scale bytes [M, K/32], else the packed layout's aligned row count
hipError_t launch_quantize_mxfp4(const void* src, int dtype, long long stride, int M, int K, uint8_t* codes,
                                 uint8_t* sf, int AM, hipStream_t s);
hipError_t launch_dequantize_mxfp4(const uint8_t* codes, const uint8_t* sf, int AM, int M, int K, void* dst, int dtype,
                                   long long stride, hipStream_t s);

struct Mxfp4GemmArgs {
  const uint8_t* A;        // codes [rows, K/2]
  const uint8_t* A_sf;     // scale word j (128 of K) of row r at r * a_row_mul + j * a_word_mul bytes
  const uint8_t* B;        // codes [groups, N, K/2]
  const uint8_t* B_sf;     // row e * N + n
  const int32_t* offsets;  // [groups + 1], or null: one group of all rows
  void* C;                 // [rows, N], rows c_stride elements apart
  long long a_row_mul, a_word_mul, b_row_mul, b_word_mul, c_stride;
  int rows, N, K, groups;
};
hipError_t launch_mxfp4_gemm(const Mxfp4GemmArgs& g, int out_dtype, int variant, hipStream_t s);

}  // namespace moe
