// k_fp4.cu -- matrices in microscaled 4-bit floating point: quantisation of
// rows, and rows looked up as values.
//
// A block's scale s comes from its largest magnitude, its values are
// RNE_e2m1(x / (s f)). Both roundings are those of the exact quotients. A bf16 x
// that is not on a border of two e2m1 numbers is 2^-8 of itself off it (8 bits
// against a border of 7 in the scale's units), so its product with the scale's
// rounded reciprocal only has to be brought back to borders that it is on: rounded
// to multiples of 2^-10, by the addition of 1.5 2^13. An fp32 product within two
// units of a border (five in a million) is decided by the remainder instead.
//
// Both kernels move each byte once; quantisation has 3 to 6 instructions a value,
// most of them its largest magnitude's and the products', on two values at a time.
// 129280 x 4096 bf16 into nvfp4 231 us (1.36 GB at 5.9 TB/s; schedulers issue in 79% of
// the cycles: as near the arithmetic's bound as memory's), into mxfp4 195 (6.9 TB/s, memory);
// fp32 409 and 458 (5.9 and 5.3 TB/s). All its rows as bf16 237 us (5.7 TB/s), 262144 rows of 256
// by token 26 us (6.5 TB/s, the table from L2 in part).
#include <math.h>
#include <stdio.h>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "fp4.cuh"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

using namespace fp4;

constexpr int kQuThreads = 256;  // of a CTA whose rows take less

template <typename T>
__device__ __forceinline__ float up(T x);
template <>
__device__ __forceinline__ float up<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ float up<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// q, the fp32 number nearest to a / s, moved off a border of a format with few bits if a / s
// is not on it. rem has the sign of a / s - q; `low` are the bits that are 0 on every border.
__device__ __forceinline__ float off_border(float q, float rem, uint32_t low) {
  const uint32_t b = __float_as_uint(q);
  if ((b & low) != 0 || rem == 0.f) return q;
  const bool more = (rem > 0.f) == (q > 0.f);  // in magnitude
  return __uint_as_float(more ? b + 1 : b - 1);
}

struct QuArgs {
  const void* X;
  int64_t ldx;
  const int32_t* count;  // rows from here on are zeros
  uint8_t* codes;
  uint8_t* scales;
  float* rowf;
  int rows, K, lanes, per_cta;  // lanes of a row; rows of a CTA
  int vec;                      // rows of X on 16 bytes
  int* status;
};

// A row takes `lanes` threads (a power of two up to 32, or whole warps), each
// up to BPL blocks, `lanes` blocks apart, so that neighbours read and write
// neighbouring blocks and four of them make a word of scales.
template <typename T, int FMT, int BPL>
__global__ void __launch_bounds__(FMT == DSPARK_NVFP4 ? 512 : 1024) k_fp4_quant(QuArgs a) {
  constexpr int B = block_of(FMT), W = B * (int)sizeof(T) / 4;  // words of a block
  __shared__ uint32_t s_max[32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid % a.lanes;
  const int64_t r = (int64_t)blockIdx.x * a.per_cta + tid / a.lanes;
  const bool row = r < a.rows;
  const bool held = row && (!a.count || r < __ldg(a.count));
  const T* x = static_cast<const T*>(a.X) + (held ? r : 0) * a.ldx;
  uint32_t w[BPL][W], top[BPL];
  uint32_t rtop = 0;
#pragma unroll
  for (int j = 0; j < BPL; ++j) {
    const int c = (lane + j * a.lanes) * B, left = held ? a.K - c : 0;
    if (a.vec && left >= B) {
      const uint4* p = reinterpret_cast<const uint4*>(x + c);
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint4 q = __ldg(p + i);
        w[j][4 * i] = q.x;
        w[j][4 * i + 1] = q.y;
        w[j][4 * i + 2] = q.z;
        w[j][4 * i + 3] = q.w;
      }
    } else {
      T v[B];
#pragma unroll
      for (int i = 0; i < B; ++i) v[i] = i < left ? x[c + i] : T(0.f);
#pragma unroll
      for (int i = 0; i < W; ++i) w[j][i] = reinterpret_cast<const uint32_t*>(v)[i];
    }
  }
  // the block's largest magnitude by its bits: a NaN is above an infinity is above the rest
#pragma unroll
  for (int j = 0; j < BPL; ++j) {
    uint32_t m = 0;
    if (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < W; ++i) m = max(m, w[j][i] & 0x7FFFFFFFu);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) m = __vmaxu2(m, w[j][i] & 0x7FFF7FFFu);
      m = max(m & 0xFFFF0000u, m << 16);
    }
    top[j] = m;
    if (m < 0x7F800000u) rtop = max(rtop, m);
  }
  float inv_f = 1.f, f = 1.f;
  if (FMT == DSPARK_NVFP4) {
    for (int o = min(a.lanes, 32) / 2; o > 0; o >>= 1) rtop = max(rtop, __shfl_xor_sync(0xFFFFFFFFu, rtop, o));
    if (a.lanes > 32) {  // one row a CTA
      if ((tid & 31) == 0) s_max[tid >> 5] = rtop;
      __syncthreads();
      for (int i = 0; i < a.lanes / 32; ++i) rtop = max(rtop, s_max[i]);
    }
    if (rtop != 0) {
      // the least e with rtop <= 2688 * 2^e = 1.3125 * 2^(11 + e); a subnormal's is below the limit of -100
      const int e = (int)(rtop >> 23) - 127 - 11 + ((rtop & 0x7FFFFFu) > 0x280000u ? 1 : 0);
      const int ec = max(e, -100);
      f = two_to(ec);
      inv_f = two_to(-ec);
    }
    if (row && lane == 0) a.rowf[r] = f;
  }
  bool bad = false;
  const int64_t ldc = row_bytes(a.K);
#pragma unroll
  for (int j = 0; j < BPL; ++j) {
    const int b = lane + j * a.lanes;
    if (top[j] >= 0x7F800000u) bad = true;
    uint32_t code;  // the scale's
    float s, inv;   // the scale, with f, and what x is multiplied by
    if (FMT == DSPARK_NVFP4) {
      const float t = __uint_as_float(top[j]) * inv_f;  // exact: f is a power of two
      float q = __fdiv_rn(t, 6.f);
      q = off_border(q, fmaf(-q, 6.f, t), 0x7FFFFu);
      code = top[j] >= 0x7F800000u ? 0x7Fu : to_e4m3(q);
      s = from_e4m3(code);
      inv = s == 0.f ? 0.f : __frcp_rn(s) * inv_f;
      s *= f;
    } else {
      const int e = top[j] >= 0x00800000u ? (int)(top[j] >> 23) - 127 : top[j] ? 31 - __clz(top[j]) - 149 : -149;
      const int es = max(e - 2, -127);
      code = top[j] >= 0x7F800000u ? 0xFFu : (uint32_t)(es + 127);
      s = two_to(es);
      inv = two_to(-es);
    }
    const int c = b * B;
    if (row && c < (int)(2 * ldc)) {
      uint32_t o[B / 8];
      const unsigned long long inv2 = tc::f2pack(inv, inv);
      uint32_t near = ~0u;
#pragma unroll
      for (int g = 0; g < B / 8; ++g) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const int k = 8 * g + i;
          const float x0 = sizeof(T) == 4 ? __uint_as_float(w[j][k]) : __uint_as_float(w[j][k / 2] << 16);
          const float x1 = sizeof(T) == 4 ? __uint_as_float(w[j][k + 1]) : __uint_as_float(w[j][k / 2] & 0xFFFF0000u);
          unsigned long long q;
          if (FMT == DSPARK_NVFP4 && sizeof(T) == 2) {
            const float m = 12288.f;
            q = tc::add2(tc::fma2(tc::f2pack(x0, x1), inv2, tc::f2pack(m, m)), tc::f2pack(-m, -m));
          } else {
            q = tc::mul2(tc::f2pack(x0, x1), inv2);  // mxfp4: exact
          }
          tc::f2unpack(q, v[i], v[i + 1]);
          if (FMT == DSPARK_NVFP4 && sizeof(T) == 4)
            near = min(near, min((__float_as_uint(v[i]) + 2u) & 0xFFFFFu, (__float_as_uint(v[i + 1]) + 2u) & 0xFFFFFu));
        }
        o[g] = to_e2m1x8(v);
      }
      if (FMT == DSPARK_NVFP4 && sizeof(T) == 4 && near <= 4u && s != 0.f) {
#pragma unroll
        for (int g = 0; g < B / 8; ++g) {
          float v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = __uint_as_float(w[j][8 * g + i]);
            float q = x * inv;
            q = fmaf(fmaf(-q, s, x), inv, q);  // the nearest to x / s
            v[i] = off_border(q, fmaf(-q, s, x), 0xFFFFFu);
          }
          o[g] = to_e2m1x8(v);
        }
      }
      uint8_t* p = a.codes + r * ldc + c / 2;
      if (B == 16) {
        *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
      } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[B / 8 - 2], o[B / 8 - 1]);
      }
    }
    // four neighbours' scales are a word of the tile
    code |= __shfl_down_sync(0xFFFFFFFFu, code, 1) << 8;
    code |= __shfl_down_sync(0xFFFFFFFFu, code, 2) << 16;
    const int64_t rows_up = ((int64_t)a.rows + kRows - 1) / kRows * kRows;
    if ((b & 3) == 0 && r < rows_up && b < chunks_of(a.K) * (kChunk / B))
      *reinterpret_cast<uint32_t*>(a.scales + scale_at(FMT, a.K, (int)r, b)) = code;
  }
  if (bad) raise_status(a.status, DSPARK_ENUMERIC);
}

struct RoArgs {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* rowf;
  int rows, K;
  const int32_t* idx;
  int N;
  void* out;
  int64_t ldo;
  int vec, shift;
  int* status;
};

// 16 bytes of a row: eight bf16 or four fp32.
template <typename T>
__device__ __forceinline__ void put16(T* p, const float* v, bool vec, int left) {
  constexpr int kVals = 16 / (int)sizeof(T);
  uint4 q;
  if (sizeof(T) == 4) {
    q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  } else {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  }
  if (vec && left >= kVals) {
    *reinterpret_cast<uint4*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (i < left) p[i] = reinterpret_cast<const T*>(&q)[i];
  }
}

// A thread takes 16 bytes of the output at a time, 4 or 2 bytes of codes and a scale in, and four of
// these together, whose loads are in flight at once: of four rows, or of one where a row is wider than 256 threads
// (WIDE). 2^shift threads a row.
constexpr int kRoEach = 4;
template <typename T, int FMT, bool WIDE>
__global__ void __launch_bounds__(256) k_fp4_rows(RoArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kNb = kChunk / block_of(FMT), kVals = 16 / (int)sizeof(T);
  const int groups = (a.K + kVals - 1) / kVals, per = 256 >> a.shift;
  const int n0 = blockIdx.x * (WIDE ? 1 : per * kRoEach) + (int)(threadIdx.x >> a.shift);
  const int g0 = threadIdx.x & ((1 << a.shift) - 1);
  for (int gg = g0; gg < groups; gg += WIDE ? 256 * kRoEach : groups) {
    uint32_t c[kRoEach], sb[kRoEach];
    float f[kRoEach];
    int r[kRoEach];
#pragma unroll
    for (int u = 0; u < kRoEach; ++u) {
      const int n = WIDE ? n0 : n0 + u * per;
      r[u] = n >= a.N ? -1 : a.idx ? __ldg(a.idx + n) : n;
    }
#pragma unroll
    for (int u = 0; u < kRoEach; ++u) {
      const int g = WIDE ? gg + u * 256 : gg;
      c[u] = sb[u] = 0;
      f[u] = 0.f;
      if (r[u] >= 0 && r[u] < a.rows && (!WIDE || g < groups)) {
        const int b = kVals * g / block_of(FMT);
        const uint8_t* row = a.codes + r[u] * row_bytes(a.K);
        c[u] = kVals == 8 ? __ldg(reinterpret_cast<const uint32_t*>(row) + g)
                          : __ldg(reinterpret_cast<const unsigned short*>(row) + g);
        sb[u] = __ldg(a.scales + scale_at(FMT, a.K, r[u], 0) + b / kNb * chunk_bytes(FMT) + b % kNb / 4 * 512 + b % 4);
        f[u] = FMT == DSPARK_NVFP4 ? __ldg(a.rowf + r[u]) : 1.f;
      } else if (r[u] != -1 && g == 0 && !(r[u] >= 0 && r[u] < a.rows)) {
        raise_status(a.status, DSPARK_ERANGE);
      }
    }
#pragma unroll
    for (int u = 0; u < kRoEach; ++u) {
      const int n = WIDE ? n0 : n0 + u * per, g = WIDE ? gg + u * 256 : gg;
      if (n >= a.N || (WIDE && g >= groups)) continue;
      // a row without a token: codes and scale 0
      const float s = FMT == DSPARK_NVFP4 ? from_e4m3(sb[u]) * f[u] : f[u] == 0.f ? 0.f : from_e8m0(sb[u]);
      float v[8];
      from_e2m1x8(c[u], v);
#pragma unroll
      for (int i = 0; i < kVals; ++i) v[i] *= s;
      put16<T>(static_cast<T*>(a.out) + n * a.ldo + kVals * g, v, a.vec, a.K - kVals * g);
    }
  }
}

dspark_status fp4_fail(cudaError_t e) {
  if (e == cudaSuccess) return DSPARK_OK;
  fprintf(stderr, "dspark: CUDA error %s\n", cudaGetErrorString(e));
  return DSPARK_ECUDA;
}
bool type_ok(int t) { return t == DSPARK_F32 || t == DSPARK_BF16; }
bool on_type(const void* p, int type) {
  return p && (reinterpret_cast<uintptr_t>(p) & (type == DSPARK_BF16 ? 1u : 3u)) == 0;
}
bool on_16(const void* p, int64_t ld, int type) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * (type == DSPARK_BF16 ? 2 : 4) % 16 == 0;
}

template <typename T, int FMT>
cudaError_t quant(QuArgs a, cudaStream_t st) {
  // blocks with those that only fill up the last tile of scales
  const int nb = chunks_of(a.K) * (kChunk / block_of(FMT));
  // An nvfp4 row belongs to one CTA (its largest value goes into every scale): four blocks a thread, whose loads are
  // in flight together (129280 rows of 256: 20.6 us with one, 15.6 with four), one where that leaves SMs without work,
  // five where those fit the row (320 blocks: 346 us with four, of which one in six is idle, 300 with five), eight
  // past 2048 blocks. Four elsewhere, where one in eight is idle too (65536 rows of 5376, bf16 and fp32: 186 and 333 us
  // with four, 276 and 401 with one, 238 and 358 with five, 292 and 530 with eight; of 4096: 120 and 211, 181 and 242,
  // 154 and 226, 142 and 313). mxfp4's blocks have twice the values. Eight of fp32 and two of mxfp4's (K above
  // 32768) do not fit the registers of so many threads: 380 and 188 bytes a thread go to memory.
  const bool few = (int64_t)a.rows * nb < 152 * 2048;
  const int bpl = FMT == DSPARK_NVFP4 ? (nb <= 512 && few ? 1 : nb > 2048 ? 8 : nb % 160 == 0 ? 5 : 4)
                                      : (nb <= 1024 ? 1 : 2);
  int lanes = 4;
  if (nb > 32 * bpl) {
    lanes = (nb + 32 * bpl - 1) / (32 * bpl) * 32;
  } else {
    while (lanes * bpl < nb) lanes *= 2;
  }
  a.lanes = lanes;
  a.per_cta = lanes <= 32 ? kQuThreads / lanes : 1;
  const int64_t rows_up = ((int64_t)a.rows + kRows - 1) / kRows * kRows;
  const dim3 grid((unsigned)((rows_up + a.per_cta - 1) / a.per_cta)), block(lanes * a.per_cta);
  constexpr int kMore = FMT == DSPARK_NVFP4 ? 4 : 2, kMost = FMT == DSPARK_NVFP4 ? 8 : 2;
  constexpr int kFive = FMT == DSPARK_NVFP4 ? 5 : 2;
  return launch_ex(bpl == 1       ? k_fp4_quant<T, FMT, 1>
                   : bpl == kMore ? k_fp4_quant<T, FMT, kMore>
                   : bpl == kFive ? k_fp4_quant<T, FMT, kFive>
                                  : k_fp4_quant<T, FMT, kMost>,
                   grid, block, 0, st, true, a);
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_fp4_code_bytes(const dspark_fp4_dims* d) {
  if (!fp4::dims_ok(d)) return 0;
  return (size_t)(d->rows > 0 ? d->rows : 1) * fp4::row_bytes(d->K);
}

extern "C" size_t dspark_fp4_scale_bytes(const dspark_fp4_dims* d) {
  if (!fp4::dims_ok(d)) return 0;
  const size_t groups = ((size_t)(d->rows > 0 ? d->rows : 1) + fp4::kRows - 1) / fp4::kRows;
  return groups * fp4::chunks_of(d->K) * fp4::chunk_bytes(d->format);
}

extern "C" dspark_status dspark_fp4_quant(const dspark_fp4_dims* d, const void* X, dspark_wdtype type, int64_t ldx,
                                          const int32_t* count, const dspark_fp4_data* out, int32_t* device_status,
                                          dspark_stream_t stream) {
  if (!fp4::dims_ok(d) || !type_ok(type) || !device_status || ldx < d->K) return DSPARK_EINVAL;
  if (d->rows == 0) return DSPARK_OK;
  if (!on_type(X, type) || !fp4::data_ok(d, out) || (reinterpret_cast<uintptr_t>(count) & 3u) != 0) return DSPARK_EINVAL;
  QuArgs a = {};
  a.X = X;
  a.ldx = ldx;
  a.count = count;
  a.codes = static_cast<uint8_t*>(out->codes);
  a.scales = static_cast<uint8_t*>(out->scales);
  a.rowf = out->rowf;
  a.rows = d->rows;
  a.K = d->K;
  a.vec = on_16(X, ldx, type);
  a.status = device_status;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  typedef __nv_bfloat16 bf;
  if (d->format == DSPARK_NVFP4)
    return fp4_fail(type == DSPARK_BF16 ? quant<bf, DSPARK_NVFP4>(a, st) : quant<float, DSPARK_NVFP4>(a, st));
  return fp4_fail(type == DSPARK_BF16 ? quant<bf, DSPARK_MXFP4>(a, st) : quant<float, DSPARK_MXFP4>(a, st));
}

extern "C" dspark_status dspark_fp4_rows(const dspark_fp4_dims* d, const dspark_fp4_data* m, const int32_t* idx, int N,
                                         void* out, dspark_wdtype type, int64_t ldo, int32_t* device_status,
                                         dspark_stream_t stream) {
  if (!fp4::dims_ok(d) || d->rows < 1 || !type_ok(type) || !device_status || ldo < d->K) return DSPARK_EINVAL;
  if (N < 0 || N > (1 << 24) || (!idx && N > d->rows)) return DSPARK_EINVAL;
  if (N == 0) return DSPARK_OK;
  if (!on_type(out, type) || !fp4::data_ok(d, m) || (reinterpret_cast<uintptr_t>(idx) & 3u) != 0) return DSPARK_EINVAL;
  RoArgs a = {};
  a.codes = static_cast<const uint8_t*>(m->codes);
  a.scales = static_cast<const uint8_t*>(m->scales);
  a.rowf = m->rowf;
  a.rows = d->rows;
  a.K = d->K;
  a.idx = idx;
  a.N = N;
  a.out = out;
  a.ldo = ldo;
  a.vec = on_16(out, ldo, type);
  a.status = device_status;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int vals = type == DSPARK_BF16 ? 8 : 4;
  while (a.shift < 8 && (vals << a.shift) < d->K) ++a.shift;
  const bool wide = d->K > vals * 256;
  const int per = wide ? 1 : (256 >> a.shift) * kRoEach;
  const dim3 grid((unsigned)((N + per - 1) / per)), block(256);
  typedef __nv_bfloat16 bf;
  auto go = [&](auto narrow_kernel, auto wide_kernel) {
    return launch_ex(wide ? wide_kernel : narrow_kernel, grid, block, 0, st, true, a);
  };
  cudaError_t e;
  if (d->format == DSPARK_NVFP4)
    e = type == DSPARK_BF16 ? go(k_fp4_rows<bf, DSPARK_NVFP4, false>, k_fp4_rows<bf, DSPARK_NVFP4, true>)
                            : go(k_fp4_rows<float, DSPARK_NVFP4, false>, k_fp4_rows<float, DSPARK_NVFP4, true>);
  else
    e = type == DSPARK_BF16 ? go(k_fp4_rows<bf, DSPARK_MXFP4, false>, k_fp4_rows<bf, DSPARK_MXFP4, true>)
                            : go(k_fp4_rows<float, DSPARK_MXFP4, false>, k_fp4_rows<float, DSPARK_MXFP4, true>);
  return fp4_fail(e);
}
