// quantize.cu -- rows of fp32 or bf16 numbers as block-scaled 4-bit floating point, and back.
//   mx (OCP Microscaling Formats MX 1.0, MXFP4): blocks of 32, scale S = 2^(floor(log2 max|x|) - 2)
//   nv: blocks of 16, scale S = s ts, s = max|x| / (6 ts) rounded to e4m3, ts the matrix's own scale
//   an element's code: x / S rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (halves to the even
//   code, beyond 6 to 6)
// Every rounding is that of the exact quotient.  In mx 1 / S is a power of two.  In nv S has four
// significant bits: ts is a power of two, and max|x| / 6 is rounded to odd before it is rounded to
// e4m3.  x / S is the product with 1 / S, corrected by its exact remainder (the quotient's
// correction of Markstein, IBM Journal of Research and Development 34, 1990), which is the fp32
// number nearest to the quotient; and no quotient of a 24-bit number by a 4-bit one lies so near to
// a midpoint between two codes that rounding it to fp32 first would take it there: the midpoints
// times S are fp32 numbers themselves.
//
// 8 elements per thread, 16-byte loads and 4-byte stores side by side, rows in groups of four loads in
// flight.  128256 x 4096 (GB300): mx bf16 202 us, memory-bound (96 % of the copy bandwidth), f32 350; nv
// bf16 353 us, bound by issue slots (86 % active: twice mx's instructions), f32 459; back 190, 446 (f32's
// two stores a lane), 193, 469 us.  Blocks share their maximum over 4 (nv: 2) lanes; the scales of four
// blocks in four rows are transposed over lanes and go out as four words.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"

namespace svk {

namespace {

constexpr int kQThreads = 256;
constexpr int kQRows = 4;  // rows of a warp, whose loads go out together
constexpr int kQTileRows = kQRows * kQThreads / 32;
constexpr int kQTileCols = 256;

struct QuantJob {
  const void* x;
  int64_t pitch_bytes;
  int R, K, groups, segments;
  float ts;
  uint8_t* codes;
  int64_t row_bytes;
  uint8_t* scales;
};

// Elements c .. c + 7 of a row as they are stored; 0 from K on.
template <typename T>
struct Raw8 {
  static constexpr int kUnits = sizeof(T) / 2;
  uint4 u[kUnits];
};
template <typename T>
__device__ __forceinline__ void load8(const void* row, int c, int K, Raw8<T>& x) {
  constexpr int U = Raw8<T>::kUnits;
  if (c + 8 <= K) {
#pragma unroll
    for (int i = 0; i < U; ++i) x.u[i] = __ldcs(reinterpret_cast<const uint4*>(row) + c / 8 * U + i);
    return;
  }
  uint32_t w[4 * U];
#pragma unroll
  for (int q = 0; q < 4 * U; ++q) {
    if constexpr (sizeof(T) == 2) {
      const uint16_t* p = static_cast<const uint16_t*>(row) + c + 2 * q;
      w[q] = (c + 2 * q < K ? (uint32_t)p[0] : 0u) | (c + 2 * q + 1 < K ? (uint32_t)p[1] << 16 : 0u);
    } else {
      w[q] = c + q < K ? static_cast<const uint32_t*>(row)[c + q] : 0u;
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) x.u[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& x, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    Elt<T>::unpack(x.u[0], f);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(&x.u[0]), b = *reinterpret_cast<const float4*>(&x.u[1]);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

__device__ __forceinline__ float abs_max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(d) : "f"(a), "f"(fabsf(b)));
  return d;
}

// Scale byte of a block with the largest magnitude `top`, and the codes of this lane's 8 elements.
template <spec_fp4_format F>
__device__ __forceinline__ uint32_t encode8(float (&f)[8], float top, float ts, uint32_t& byte) {
  const uint32_t bits = __float_as_uint(top);
  if constexpr (F == SPEC_FP4_MX) {
    if (bits >= 0x7f800000u) {  // NaN or infinity: the scale that stands for NaN
      byte = 255u;
      return 0u;
    }
    const int e = max((int)(bits >> 23) - 2, 0);
    byte = (uint32_t)e;
    const float inv = __uint_as_float((uint32_t)(254 - e) << 23);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= inv;
  } else {
    if (bits >= 0x7f800000u) {
      byte = 127u;
      return 0u;
    }
    // top / (6 ts), truncated with a sticky last bit
    const float t = fminf(top * (1.0f / ts), 1e30f);
    float v = __fdiv_rz(t, 6.0f);
    if (fmaf(-v, 6.0f, t) != 0.f) v = __uint_as_float(__float_as_uint(v) | 1u);
    uint16_t two;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(two) : "f"(0.f), "f"(v));
    byte = two & 0xffu;
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"(two));
    const float s = __low2float(*reinterpret_cast<const __half2*>(&h)) * ts;
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    const bool far = top > 8.f * s;  // a scale at its largest: quotients may leave fp32's range
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y = f[i] * inv;
      if (far) y = fminf(fmaxf(y, -8.f), 8.f);
      f[i] = fmaf(fmaf(-y, s, f[i]), inv, y);
    }
  }
  return fp4_codes(f);
}

template <typename T, spec_fp4_format F>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 2 && F == SPEC_FP4_MX ? 6 : 5) quantize_kernel(QuantJob job) {
  constexpr int kLanes = F == SPEC_FP4_MX ? 4 : 2;  // lanes of a block
  constexpr int kRows = sizeof(T) == 2 ? kQRows : kQRows / 2;  // in flight
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");  // a product may line up
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tile = blockIdx.x / (unsigned)job.segments;
  const int c = (int)(blockIdx.x % (unsigned)job.segments) * kQTileCols + lane * 8;
  const int K = job.K;
  const int r0 = (int)(tile * kQTileRows) + warp;
  constexpr int kStep = kQThreads / 32;  // between this warp's rows
  const char* x = static_cast<const char*>(job.x) + (int64_t)r0 * job.pitch_bytes;
  uint8_t* out = job.codes + (int64_t)r0 * job.row_bytes + c / 2;
  const bool in_row = c < K, in_codes = c < 2 * job.row_bytes;
  uint32_t bytes = 0u;  // this lane's block's scale in each of the rows
#pragma unroll
  for (int i0 = 0; i0 < kQRows; i0 += kRows) {
    Raw8<T> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (in_row && r0 + (i0 + i) * kStep < job.R) {
        load8<T>(x, c, K, raw[i]);
      } else {
#pragma unroll
        for (int u = 0; u < Raw8<T>::kUnits; ++u) raw[i].u[u] = make_uint4(0u, 0u, 0u, 0u);
      }
      x += kStep * job.pitch_bytes;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const bool real = r0 + (i0 + i) * kStep < job.R;
      float f[8];
      unpack8<T>(raw[i], f);
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = abs_max_nan(top, f[e]);
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) top = abs_max_nan(top, __shfl_xor_sync(kFull, top, o));
      uint32_t byte;
      const uint32_t codes = encode8<F>(f, top, job.ts, byte);
      if (real && in_codes) *reinterpret_cast<uint32_t*>(out) = codes;
      // past the row's end, and in rows past the last, scales are zero
      if (in_row && real) bytes |= byte << (8 * (i0 + i));
      out += kStep * job.row_bytes;
    }
  }
  // the four scales of a tile's row as one word: of the lanes of four blocks the first four each
  // take one of the rows
  constexpr int kSpan = 4 * kLanes;
  const int mine = lane & (kSpan - 1), from = lane & ~(kSpan - 1), g = c / (kLanes * 32);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = __shfl_sync(kFull, bytes, from + q * kLanes);
  const uint32_t pick = (uint32_t)(mine & 3) * 0x11u + 0x40u;  // this row's byte of two words
  const uint32_t word = __byte_perm(__byte_perm(w[0], w[1], pick), __byte_perm(w[2], w[3], pick), 0x5410u);
  if (mine < 4 && g < job.groups)
    *reinterpret_cast<uint32_t*>(job.scales + fp4_scale_at(r0 + mine * kStep, 4 * g, job.groups)) = word;
}

struct DequantJob {
  const uint8_t* codes;
  int64_t row_bytes;
  const uint8_t* scales;
  int R, K, groups, segments;
  float ts;
  void* out;
  int64_t pitch_bytes;
};

template <typename T, spec_fp4_format F>
__global__ void __launch_bounds__(kQThreads) dequantize_kernel(DequantJob job) {
  constexpr int kLanes = F == SPEC_FP4_MX ? 4 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tile = blockIdx.x / (unsigned)job.segments;
  const int c = (int)(blockIdx.x % (unsigned)job.segments) * kQTileCols + lane * 8;
  const int K = job.K;
  const int r0 = (int)(tile * kQTileRows) + warp;
  if (c >= K) return;
  uint32_t codes[kQRows];
  uint32_t byte[kQRows];
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    const int r = r0 + i * (kQThreads / 32);
    codes[i] = byte[i] = 0u;
    if (r < job.R) {
      codes[i] = __ldg(reinterpret_cast<const uint32_t*>(job.codes + (int64_t)r * job.row_bytes + c / 2));
      byte[i] = __ldg(job.scales + fp4_scale_at(r, c / (kLanes * 8), job.groups));
    }
  }
#pragma unroll
  for (int i = 0; i < kQRows; ++i) {
    const int r = r0 + i * (kQThreads / 32);
    if (r >= job.R) return;
    float s;
    if constexpr (F == SPEC_FP4_MX) {
      s = __uint_as_float(byte[i] == 255u ? 0x7fffffffu : byte[i] == 0u ? 0x00400000u : byte[i] << 23);
    } else {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h) : "h"((uint16_t)byte[i]));
      s = __low2float(*reinterpret_cast<const __half2*>(&h)) * job.ts;
    }
    float f[8];
    uint32_t h[4];
    asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
        " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes[i]));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[q]));
      f[2 * q] = v.x * s;
      f[2 * q + 1] = v.y * s;
    }
    char* row = static_cast<char*>(job.out) + (int64_t)r * job.pitch_bytes;
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
        w[q] = *reinterpret_cast<const uint32_t*>(&b);
      }
      if (c + 8 <= K) {
        *reinterpret_cast<uint4*>(row + c * 2) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < K) reinterpret_cast<uint16_t*>(row)[c + e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
      }
    } else {
      if (c + 8 <= K) {
        float4* d = reinterpret_cast<float4*>(row + c * 4);
        d[0] = make_float4(f[0], f[1], f[2], f[3]);
        d[1] = make_float4(f[4], f[5], f[6], f[7]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < K) reinterpret_cast<float*>(row)[c + e] = f[e];
      }
    }
  }
}

int check_matrix(spec_dtype dtype, int32_t rows, int32_t cols, int64_t row_pitch,
                 spec_fp4_format format, float tensor_scale) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_UNSUPPORTED_DTYPE;
  if (format != SPEC_FP4_MX && format != SPEC_FP4_NV) return SPEC_ERR_UNSUPPORTED_DTYPE;
  if (rows < 0 || cols < 1 || row_pitch < cols) return SPEC_ERR_INVALID_ARG;
  if (!fp4_tensor_scale_ok(tensor_scale)) return SPEC_ERR_INVALID_ARG;
  if (format == SPEC_FP4_MX && tensor_scale != 1.0f) return SPEC_ERR_INVALID_ARG;
  if (rows > SPEC_FP4_MAX_DIM || cols > SPEC_FP4_MAX_DIM || row_pitch > INT64_MAX / 8)
    return SPEC_ERR_TOO_LARGE;
  // tiles of the launch
  if ((int64_t)fp4_row_tiles(rows) * (128 / kQTileRows) * ((cols + kQTileCols - 1) / kQTileCols) > INT32_MAX)
    return SPEC_ERR_TOO_LARGE;
  return SPEC_OK;
}

bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

}  // namespace

cudaError_t launch_fp4_quantize(const void* x, spec_dtype dtype, int rows, int cols,
                                int64_t row_pitch, spec_fp4_format format, float tensor_scale,
                                void* codes, void* scales, cudaStream_t s) {
  QuantJob job{};
  job.x = x;
  job.pitch_bytes = row_pitch * (dtype == SPEC_BF16 ? 2 : 4);
  job.R = rows;
  job.K = cols;
  job.groups = fp4_groups(cols, format);
  const int span = (int)fp4_row_bytes(cols) * 2;  // elements, the codes' padding included
  job.segments = (span + kQTileCols - 1) / kQTileCols;
  job.ts = tensor_scale;
  job.codes = static_cast<uint8_t*>(codes);
  job.row_bytes = fp4_row_bytes(cols);
  job.scales = static_cast<uint8_t*>(scales);
  const int64_t tiles = (int64_t)fp4_row_tiles(rows) * 128 / kQTileRows;
  const unsigned grid = (unsigned)(tiles * job.segments);
  if (format == SPEC_FP4_MX) {
    if (dtype == SPEC_BF16) quantize_kernel<uint16_t, SPEC_FP4_MX><<<grid, kQThreads, 0, s>>>(job);
    else quantize_kernel<float, SPEC_FP4_MX><<<grid, kQThreads, 0, s>>>(job);
  } else {
    if (dtype == SPEC_BF16) quantize_kernel<uint16_t, SPEC_FP4_NV><<<grid, kQThreads, 0, s>>>(job);
    else quantize_kernel<float, SPEC_FP4_NV><<<grid, kQThreads, 0, s>>>(job);
  }
  return cudaGetLastError();
}

}  // namespace svk

using namespace svk;

extern "C" size_t spec_fp4_code_bytes(int32_t rows, int32_t cols) {
  if (rows < 0 || cols < 1 || rows > SPEC_FP4_MAX_DIM || cols > SPEC_FP4_MAX_DIM) return 0;
  return (size_t)rows * (size_t)fp4_row_bytes(cols);
}

extern "C" size_t spec_fp4_scale_bytes(int32_t rows, int32_t cols, spec_fp4_format format) {
  if (rows < 0 || cols < 1 || rows > SPEC_FP4_MAX_DIM || cols > SPEC_FP4_MAX_DIM) return 0;
  if (format != SPEC_FP4_MX && format != SPEC_FP4_NV) return 0;
  return (size_t)fp4_row_tiles(rows) * (size_t)fp4_groups(cols, format) * kScaleTile;
}

extern "C" int spec_fp4_quantize(const void* x, spec_dtype dtype, int32_t rows, int32_t cols,
                                 int64_t row_pitch, spec_fp4_format format, float tensor_scale,
                                 void* codes, void* scales, spec_stream_t stream) {
  const int rc = check_matrix(dtype, rows, cols, row_pitch, format, tensor_scale);
  if (rc != SPEC_OK) return rc;
  if (rows == 0) return SPEC_OK;
  if (!x || !codes || !scales) return SPEC_ERR_INVALID_ARG;
  if (misaligned16(x) || misaligned16(codes) || misaligned16(scales) ||
      row_pitch * (dtype == SPEC_BF16 ? 2 : 4) % 16 != 0)
    return SPEC_ERR_MISALIGNED;
  return launch_fp4_quantize(x, dtype, rows, cols, row_pitch, format, tensor_scale, codes, scales,
                             reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

extern "C" int spec_fp4_dequantize(const void* codes, const void* scales, int32_t rows, int32_t cols,
                                   spec_fp4_format format, float tensor_scale, void* out,
                                   spec_dtype dtype, int64_t row_pitch, spec_stream_t stream) {
  const int rc = check_matrix(dtype, rows, cols, row_pitch, format, tensor_scale);
  if (rc != SPEC_OK) return rc;
  if (rows == 0) return SPEC_OK;
  if (!out || !codes || !scales) return SPEC_ERR_INVALID_ARG;
  if (misaligned16(out) || misaligned16(codes) || misaligned16(scales) ||
      row_pitch * (dtype == SPEC_BF16 ? 2 : 4) % 16 != 0)
    return SPEC_ERR_MISALIGNED;
  DequantJob job{};
  job.codes = static_cast<const uint8_t*>(codes);
  job.row_bytes = fp4_row_bytes(cols);
  job.scales = static_cast<const uint8_t*>(scales);
  job.R = rows;
  job.K = cols;
  job.groups = fp4_groups(cols, format);
  job.segments = (cols + kQTileCols - 1) / kQTileCols;
  job.ts = tensor_scale;
  job.out = out;
  job.pitch_bytes = row_pitch * (dtype == SPEC_BF16 ? 2 : 4);
  const int64_t tiles = ((int64_t)rows + kQTileRows - 1) / kQTileRows;
  const unsigned grid = (unsigned)(tiles * job.segments);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (format == SPEC_FP4_MX) {
    if (dtype == SPEC_BF16) dequantize_kernel<uint16_t, SPEC_FP4_MX><<<grid, kQThreads, 0, s>>>(job);
    else dequantize_kernel<float, SPEC_FP4_MX><<<grid, kQThreads, 0, s>>>(job);
  } else {
    if (dtype == SPEC_BF16) dequantize_kernel<uint16_t, SPEC_FP4_NV><<<grid, kQThreads, 0, s>>>(job);
    else dequantize_kernel<float, SPEC_FP4_NV><<<grid, kQThreads, 0, s>>>(job);
  }
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
