// fp4.cuh -- block-scaled 4-bit floating point as the kernels store it.
//   element code: sign, then the index of 0, 0.5, 1, 1.5, 2, 3, 4, 6; element 2 i of a row in the
//     low half of byte i; a row takes 16 bytes per 32 elements, the last ones padded with zeros
//   scales: of tiles of 128 rows by 4 scales, tile (i, j) at 512 (i groups + j), the scale of row
//     r and block b at 16 (r % 32) + 4 (r / 32 % 4) + b % 4 in it, the order in which the tensor
//     cores take them from tensor memory; padding is zero
#pragma once

#include "common.cuh"

namespace svk {

constexpr int kScaleTile = 512;

__host__ __device__ inline int fp4_block(spec_fp4_format f) { return f == SPEC_FP4_MX ? 32 : 16; }
// Bytes of a row of codes.
__host__ __device__ inline int64_t fp4_row_bytes(int64_t cols) { return (cols + 31) / 32 * 16; }
// Scale tiles along a row, and along the rows.
__host__ __device__ inline int fp4_groups(int cols, spec_fp4_format f) {
  const int n = fp4_block(f) * 4;
  return (int)(((int64_t)cols + n - 1) / n);
}
__host__ __device__ inline int fp4_row_tiles(int rows) { return (int)(((int64_t)rows + 127) / 128); }
// Where the scale of row r's block b lies.
__device__ __forceinline__ int64_t fp4_scale_at(int r, int b, int groups) {
  return ((int64_t)(r >> 7) * groups + (b >> 2)) * kScaleTile + (r & 31) * 16 + ((r >> 5) & 3) * 4 +
         (b & 3);
}

// A power of two within 2^-100 .. 2^100 (a tensor scale).
inline bool fp4_tensor_scale_ok(float s) {
  uint32_t u;
  __builtin_memcpy(&u, &s, 4);
  const int e = (int)(u >> 23);
  return (u & 0x7fffffu) == 0 && e >= 27 && e <= 227;
}

// Eight values (already divided by their scale) as codes, the first in the lowest bits.
__device__ __forceinline__ uint32_t fp4_codes(const float (&y)[8]) {
  uint32_t d;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(d)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return d;
}

// The launches behind the entry points, arguments checked (quantize.cu, fp4_linear.cu).
cudaError_t launch_fp4_quantize(const void* x, spec_dtype dtype, int rows, int cols,
                                int64_t row_pitch, spec_fp4_format format, float tensor_scale,
                                void* codes, void* scales, cudaStream_t s);
cudaError_t launch_fp4_linear(const void* a_codes, const void* a_scales, const void* w_codes,
                              const void* w_scales, spec_fp4_format format, int R, int V, int K,
                              float alpha, void* out, spec_dtype dtype, int64_t pitch, int stall,
                              cudaStream_t s);

}  // namespace svk
