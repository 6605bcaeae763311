// fp4.cuh -- the layout of a matrix in microscaled 4-bit floating point, and
// conversions to and from e2m1.
#pragma once

#include <stdint.h>

#include "dspark.h"

namespace dspark {
namespace fp4 {

constexpr int kChunk = 256;  // columns that the scales' tiles of one 128-row group advance by
constexpr int kRows = 128;   // rows of a scale tile

__host__ __device__ constexpr int block_of(int format) { return format == DSPARK_NVFP4 ? 16 : 32; }
__host__ __device__ constexpr int64_t row_bytes(int K) { return (int64_t)(K + 31) / 32 * 16; }
// bytes of the scales of 128 rows by kChunk columns
__host__ __device__ constexpr int chunk_bytes(int format) { return kRows * (kChunk / block_of(format)); }
__host__ __device__ constexpr int chunks_of(int K) { return (K + kChunk - 1) / kChunk; }
// byte of the scale of block b of row r
__host__ __device__ __forceinline__ int64_t scale_at(int format, int K, int r, int b) {
  const int nb = kChunk / block_of(format), i = r % kRows;
  return ((int64_t)(r / kRows) * chunks_of(K) + b / nb) * chunk_bytes(format) + (b % nb) / 4 * 512 + (i % 32) * 16 +
         (i / 32) * 4 + b % 4;
}

inline bool dims_ok(const dspark_fp4_dims* d) {
  return d && d->rows >= 0 && d->rows <= (1 << 24) && d->K >= 1 && d->K <= 65536 &&
         (d->format == DSPARK_NVFP4 || d->format == DSPARK_MXFP4);
}
inline bool data_ok(const dspark_fp4_dims* d, const dspark_fp4_data* m) {
  if (!m || !m->codes || !m->scales) return false;
  uintptr_t a = reinterpret_cast<uintptr_t>(m->codes) | reinterpret_cast<uintptr_t>(m->scales);
  if (d->format == DSPARK_NVFP4) {
    if (!m->rowf) return false;
    a |= reinterpret_cast<uintptr_t>(m->rowf);
  }
  return (a & 15u) == 0;
}

// Eight values to e2m1 (nearest, ties to even, at most 6 in magnitude), the first lowest.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* v) {
  uint32_t d;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(d)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return d;
}
// Eight e2m1 codes to the values that they are, the first lowest.
__device__ __forceinline__ void from_e2m1x8(uint32_t c, float* v) {
  uint32_t h[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(c));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
        : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
        : "r"(h[i]));
}
// x >= 0 to e4m3 (nearest, ties to even, at most 448), and back.
__device__ __forceinline__ uint32_t to_e4m3(float x) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(x));
  return d & 0xFFu;
}
__device__ __forceinline__ float from_e4m3(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)b));
  float x;
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %1;\n cvt.f32.f16 %0, a;\n}" : "=f"(x) : "r"(h));
  return x;
}
// 2^e as fp32, e in [-149, 127]
__device__ __forceinline__ float two_to(int e) {
  return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}
// the value of an e8m0 scale (255: NaN)
__device__ __forceinline__ float from_e8m0(uint32_t b) {
  return b == 255u ? __int_as_float(0x7FC00000) : two_to((int)b - 127);
}

}  // namespace fp4
}  // namespace dspark
