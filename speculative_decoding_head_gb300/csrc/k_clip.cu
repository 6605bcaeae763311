// k_clip.cu -- the 2-norm over many gradient tensors, and their scaling to a
// largest norm:
//   norm = sqrt(sum over tensors and values of x^2),
//   out  = x * min(1, max_norm / (norm + 1e-6)).
//
// Two launches over the same list of pieces (16384 values of one tensor each):
// the first leaves a partial sum of squares per CTA, the second adds those in
// order (every CTA the same way) and scales. The list of tensors travels in the
// kernel's parameters, so a call keeps nothing on the device. Bound by memory,
// read twice and written once: 400 M values in 301 tensors 494 us, 95% of the
// measured copy rate; the head's 141 MB 77 us (81%: the two kernels' start and end
// are 6 us of it; L2 keeps nothing from the first pass to the second, in any
// order of the pieces).
//
// A matrix whose rows lie apart (a gradient with padded rows) is cut into pieces of
// whole rows, or of 16384 columns of one; such lists have kernels of their own, so
// that the others' parameters stay small. 50257 x 4100 bf16 in rows of 4104: 508 us
// (fp32 493), where the whole buffer as one tensor takes 199 (377): bound by finding
// each 16 bytes' row and by the two CTAs per SM that 96 registers leave.
//
// Squares are summed in fp32 over 16 or 32 values whose largest magnitude lies in
// [2^-50, 2^60], where no square that counts is lost or overflows, and those
// sums in fp64; other groups (and groups with an infinity) are squared in fp64.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <type_traits>

#include "dspark_common.cuh"
#include "dspark_internal.h"

namespace dspark {

namespace {

constexpr int kClThreads = 256;
constexpr int kClPiece = 16384;    // values of a piece
constexpr int kClCtas = 152 * 8;   // CTAs of a full grid; partial sums of a launch
constexpr int kClLaunch = 512;     // tensors of one launch

struct ClTensor {
  const void* in;
  void* out;
  long long n;
  int first;   // index of its first piece
  int bf16;
};
// a tensor, or a matrix of rows `cols` long (cols 0: contiguous values)
struct ClMatrix : ClTensor {
  long long cols, ldi, ldo;  // n is its rows, ldi and ldo what they lie apart
  // rows of a piece
  __host__ __device__ int per_piece() const { return cols < kClPiece ? kClPiece / (int)cols : 1; }
};
template <int MAXT, bool ROWS>
struct ClList {
  std::conditional_t<ROWS, ClMatrix, ClTensor> t[MAXT];
  int count, pieces;
};

__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// the tensor that piece i belongs to (tensors without values have no piece)
template <int MAXT, bool ROWS>
__device__ __forceinline__ int cl_find(const ClList<MAXT, ROWS>& l, int i) {
  int lo = 0, hi = l.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (l.t[mid].first <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// sum of squares of K values: fp32 where their range allows, else fp64
template <int K>
__device__ __forceinline__ double cl_squares(const float* x) {
  float s[4] = {0.f, 0.f, 0.f, 0.f}, m = 0.f;
#pragma unroll
  for (int i = 0; i < K; ++i) {
    s[i & 3] = fmaf(x[i], x[i], s[i & 3]);
    m = fmaxf(m, fabsf(x[i]));
  }
  if (m == 0.f || (m >= 0x1p-50f && m <= 0x1p60f)) return (double)((s[0] + s[1]) + (s[2] + s[3]));
  double d = 0.0;
  for (int i = 0; i < K; ++i) d += (double)x[i] * (double)x[i];
  return d;
}

// the CTA's sum of x, in every thread: lanes, then warps, in a fixed order
__device__ __forceinline__ double cl_block_sum(double x) {
  __shared__ double red[kClThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  x = 0.0;
#pragma unroll
  for (int w = 0; w < kClThreads / 32; ++w) x += red[w];
  return x;
}

// Piece i of a matrix: nr rows of nc columns each from row r0 and column c0 on, a
// unit of W columns (16 bytes) per thread at a time, units numbered along the rows.
struct ClSpan {
  long long r0, c0;
  int nc, per, units;
  __device__ __forceinline__ ClSpan(const ClMatrix& t, int i, int W) {
    const long long blocks = (t.cols + kClPiece - 1) / kClPiece, at = i - t.first, row = at / blocks;
    const int rows = t.per_piece();
    r0 = row * rows;
    c0 = (at - row * blocks) * kClPiece;
    nc = (int)min((long long)kClPiece, t.cols - c0);
    per = (nc + W - 1) / W;
    units = (int)min((long long)rows, t.n - r0) * per;
  }
  // unit u's row, and its first column in the piece
  __device__ __forceinline__ long long row(int u, int W, int& c) const {
    const int r = u / per;
    c = (u - r * per) * W;
    return r0 + r;
  }
};
// a unit's values: 16 bytes at once (vec, and the unit is whole), or the `left` that there are
template <typename T, int W>
__device__ __forceinline__ void cl_load(const T* p, bool vec, int left, T* x) {
  if (vec && left >= W) {
    *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) x[e] = e < left ? p[e] : T(0.f);
  }
}
__device__ __forceinline__ float cl_up(float x) { return x; }
__device__ __forceinline__ float cl_up(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void cl_down(float x, float* o) { *o = x; }
__device__ __forceinline__ void cl_down(float x, __nv_bfloat16* o) { *o = __float2bfloat16_rn(x); }

constexpr int kClAhead = 4;  // units a thread has on their way

template <typename T>
__device__ __forceinline__ double cl_rows_squares(const ClMatrix& t, int i) {
  constexpr int W = 16 / sizeof(T);
  const ClSpan s(t, i, W);
  const T* in = static_cast<const T*>(t.in) + s.c0;
  const bool vec = ((reinterpret_cast<uintptr_t>(t.in) | (uintptr_t)(t.ldi * sizeof(T))) & 15u) == 0;
  double acc = 0.0;
  for (int u = threadIdx.x; u < s.units; u += kClAhead * kClThreads) {
    __align__(16) T x[kClAhead][W];
#pragma unroll
    for (int k = 0; k < kClAhead; ++k) {
      int c = 0;
      const int v = u + k * kClThreads;
      const long long row = s.row(v < s.units ? v : 0, W, c);
      cl_load<T, W>(in + row * t.ldi + c, vec, v < s.units ? s.nc - c : 0, x[k]);
    }
    float f[kClAhead * W];
#pragma unroll
    for (int k = 0; k < kClAhead * W; ++k) f[k] = cl_up(x[k / W][k % W]);
    acc += cl_squares<kClAhead * W>(f);
  }
  return acc;
}

template <typename T>
__device__ __forceinline__ void cl_rows_scale(const ClMatrix& t, int i, float coef) {
  constexpr int W = 16 / sizeof(T);
  const ClSpan s(t, i, W);
  const T* in = static_cast<const T*>(t.in) + s.c0;
  T* out = static_cast<T*>(t.out) + s.c0;
  const bool vec = ((reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out) |
                     (uintptr_t)((t.ldi | t.ldo) * sizeof(T))) & 15u) == 0;
  for (int u = threadIdx.x; u < s.units; u += kClAhead * kClThreads) {
    __align__(16) T x[kClAhead][W];
#pragma unroll
    for (int k = 0; k < kClAhead; ++k) {
      int c = 0;
      const int v = u + k * kClThreads;
      const long long row = s.row(v < s.units ? v : 0, W, c);
      cl_load<T, W>(in + row * t.ldi + c, vec, v < s.units ? s.nc - c : 0, x[k]);
    }
#pragma unroll
    for (int k = 0; k < kClAhead; ++k) {
      const int v = u + k * kClThreads;
      if (v >= s.units) break;
      int c = 0;
      const long long row = s.row(v, W, c);
      T* o = out + row * t.ldo + c;
#pragma unroll
      for (int e = 0; e < W; ++e) cl_down(coef * cl_up(x[k][e]), &x[k][e]);
      if (vec && s.nc - c >= W) {
        *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(x[k]);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
          if (e < s.nc - c) o[e] = x[k][e];
      }
    }
  }
}

template <int MAXT, bool ROWS>
__global__ void __launch_bounds__(kClThreads)
    k_clip_norm(const __grid_constant__ ClList<MAXT, ROWS> l, double* __restrict__ part) {
  double acc = 0.0;
  pdl_wait();
  for (int i = blockIdx.x; i < l.pieces; i += gridDim.x) {
    const auto& t = l.t[cl_find(l, i)];
    if constexpr (ROWS)
      if (t.cols) {
        acc += t.bf16 ? cl_rows_squares<__nv_bfloat16>(t, i) : cl_rows_squares<float>(t, i);
        continue;
      }
    const long long off = (long long)(i - t.first) * kClPiece;
    const int n = (int)min((long long)kClPiece, t.n - off);
    int done = 0;
    if (t.bf16) {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(t.in) + off;
      if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        const int m = n / 8;
        for (int u = threadIdx.x; u < m; u += 4 * kClThreads) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = u + k * kClThreads < m ? __ldg(q + u + k * kClThreads) : make_uint4(0, 0, 0, 0);
          float x[32];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[k * 8 + 2 * e] = bf_lo(w[e]);
              x[k * 8 + 2 * e + 1] = bf_hi(w[e]);
            }
          }
          acc += cl_squares<32>(x);
        }
        done = m * 8;
      }
      for (int e = done + threadIdx.x; e < n; e += kClThreads) {
        const float x[1] = {__bfloat162float(p[e])};
        acc += cl_squares<1>(x);
      }
    } else {
      const float* p = static_cast<const float*>(t.in) + off;
      if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        const float4* q = reinterpret_cast<const float4*>(p);
        const int m = n / 4;
        for (int u = threadIdx.x; u < m; u += 4 * kClThreads) {
          float x[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 v = u + k * kClThreads < m ? __ldg(q + u + k * kClThreads) : make_float4(0.f, 0.f, 0.f, 0.f);
            x[4 * k] = v.x;
            x[4 * k + 1] = v.y;
            x[4 * k + 2] = v.z;
            x[4 * k + 3] = v.w;
          }
          acc += cl_squares<16>(x);
        }
        done = m * 4;
      }
      for (int e = done + threadIdx.x; e < n; e += kClThreads) {
        const float x[1] = {p[e]};
        acc += cl_squares<1>(x);
      }
    }
  }

  acc = cl_block_sum(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

template <int MAXT, bool ROWS>
__global__ void __launch_bounds__(kClThreads)
    k_clip_scale(const __grid_constant__ ClList<MAXT, ROWS> l, const double* __restrict__ part, int parts, float max_norm,
                 int write_norm, float* __restrict__ norm_out, int* status) {
  pdl_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClThreads) s += part[i];
  s = cl_block_sum(s);
  const double norm = sqrt(s);
  const float nf = (float)norm;
  // a norm that is not finite scales nothing: the caller sees it and skips the step
  const bool finite = isfinite(nf);
  const float coef = finite ? (float)fmin(1.0, (double)max_norm / (norm + 1e-6)) : 1.f;
  if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) {
    *norm_out = nf;
    if (!finite) raise_status(status, DSPARK_ENUMERIC);
  }
  for (int i = blockIdx.x; i < l.pieces; i += gridDim.x) {
    const auto& t = l.t[cl_find(l, i)];
    if (coef == 1.f && t.in == t.out) continue;  // in place and within the norm: nothing to do
    if constexpr (ROWS)
      if (t.cols) {
        if (t.bf16)
          cl_rows_scale<__nv_bfloat16>(t, i, coef);
        else
          cl_rows_scale<float>(t, i, coef);
        continue;
      }
    const long long off = (long long)(i - t.first) * kClPiece;
    const int n = (int)min((long long)kClPiece, t.n - off);
    int done = 0;
    if (t.bf16) {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(t.in) + off;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(t.out) + off;
      if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & 15u) == 0) {
        const uint4* q = reinterpret_cast<const uint4*>(p);
        uint4* r = reinterpret_cast<uint4*>(o);
        const int m = n / 8;
        for (int u = threadIdx.x; u < m; u += 4 * kClThreads) {
          uint4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (u + k * kClThreads < m) v[k] = q[u + k * kClThreads];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (u + k * kClThreads >= m) break;
            uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b = __floats2bfloat162_rn(coef * bf_lo(w[e]), coef * bf_hi(w[e]));
              w[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
            r[u + k * kClThreads] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        done = m * 8;
      }
      for (int e = done + threadIdx.x; e < n; e += kClThreads) o[e] = __float2bfloat16_rn(coef * __bfloat162float(p[e]));
    } else {
      const float* p = static_cast<const float*>(t.in) + off;
      float* o = static_cast<float*>(t.out) + off;
      if (((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(o)) & 15u) == 0) {
        const float4* q = reinterpret_cast<const float4*>(p);
        float4* r = reinterpret_cast<float4*>(o);
        const int m = n / 4;
        for (int u = threadIdx.x; u < m; u += 4 * kClThreads) {
          float4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (u + k * kClThreads < m) v[k] = q[u + k * kClThreads];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (u + k * kClThreads >= m) break;
            r[u + k * kClThreads] = make_float4(coef * v[k].x, coef * v[k].y, coef * v[k].z, coef * v[k].w);
          }
        }
        done = m * 4;
      }
      for (int e = done + threadIdx.x; e < n; e += kClThreads) o[e] = coef * p[e];
    }
  }
}

int cl_launches(int count) { return count > 0 ? (count + kClLaunch - 1) / kClLaunch : 1; }

// The call's list: tensors of numel values, or (rows given) matrices.
struct ClCall {
  int count;
  const void* const* in;
  void* const* out;
  const int64_t* numel;
  const int64_t *rows, *cols, *ldi, *ldo;
  const int32_t* types;

  // matrix i's rows lie one after the other, or there is one: its values are contiguous
  bool flat(int i) const { return !rows || rows[i] == 1 || (ldi[i] == cols[i] && ldo[i] == cols[i]); }
  int64_t values(int i) const { return rows ? rows[i] * cols[i] : numel[i]; }
};

// the tensors [a, b) of the call as a launch's list
template <int MAXT, bool ROWS>
bool cl_list(ClList<MAXT, ROWS>& l, const ClCall& c, int a, int b) {
  memset(&l, 0, sizeof(l));
  long long at = 0;
  for (int i = a; i < b; ++i) {
    if (c.values(i) == 0) continue;
    auto& t = l.t[l.count++];
    t.in = c.in[i];
    t.out = c.out[i];
    t.n = c.values(i);
    t.first = (int)at;
    t.bf16 = c.types[i] == DSPARK_BF16;
    long long pieces = (t.n + kClPiece - 1) / kClPiece;
    if constexpr (ROWS)
      if (!c.flat(i)) {
        t.n = c.rows[i];
        t.cols = c.cols[i];
        t.ldi = c.ldi[i];
        t.ldo = c.ldo[i];
        pieces = (t.n + t.per_piece() - 1) / t.per_piece() * ((t.cols + kClPiece - 1) / kClPiece);
      }
    at += pieces;
    if (at > 0x7FFF0000ll) return false;
  }
  l.pieces = (int)at;
  return true;
}

template <int MAXT, bool ROWS>
cudaError_t cl_run(bool scale, const ClList<MAXT, ROWS>& l, double* part, int parts, float max_norm, bool last,
                   float* norm, int* status, cudaStream_t st) {
  const dim3 grid(l.pieces < 1 ? 1 : l.pieces < kClCtas ? l.pieces : kClCtas), block(kClThreads);
  return scale ? launch_ex(k_clip_scale<MAXT, ROWS>, grid, block, 0, st, true, l, part, parts, max_norm, last ? 1 : 0,
                           norm, status)
               : launch_ex(k_clip_norm<MAXT, ROWS>, grid, block, 0, st, true, l, part);
}

int cl_grid(int64_t pieces) { return pieces < 1 ? 1 : pieces < kClCtas ? (int)pieces : kClCtas; }

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_clip_grads_scratch_bytes(int count) {
  if (count < 0) return 0;
  return sizeof(double) * (size_t)kClCtas * cl_launches(count);
}

namespace {

// MAXT tensors a launch (all launches' partial sums in one run, then the scaling launches on all of them)
template <int MAXT, bool ROWS>
dspark_status cl_call(const ClCall& c, float max_norm, float* norm, double* part, int* status, cudaStream_t st) {
  ClList<MAXT, ROWS> l;
  const int launches = c.count > MAXT ? (c.count + MAXT - 1) / MAXT : 1;
  cudaError_t e = cudaSuccess;
  int parts = 0;
  for (int k = 0; k < launches && e == cudaSuccess; ++k) {
    const int a = k * MAXT, b = a + MAXT < c.count ? a + MAXT : c.count;
    if (!cl_list(l, c, a, b)) return DSPARK_EUNSUPPORTED;
    e = cl_run(false, l, part + parts, 0, max_norm, false, norm, status, st);
    parts += cl_grid(l.pieces);
  }
  for (int k = launches - 1; k >= 0 && e == cudaSuccess; --k) {
    const int a = k * MAXT, b = a + MAXT < c.count ? a + MAXT : c.count;
    if (launches > 1 && !cl_list(l, c, a, b)) return DSPARK_EUNSUPPORTED;
    e = cl_run(true, l, part, parts, max_norm, k == launches - 1, norm, status, st);
  }
  if (e == cudaSuccess) return DSPARK_OK;
  fprintf(stderr, "dspark: CUDA error %s\n", cudaGetErrorString(e));
  return DSPARK_ECUDA;
}

dspark_status cl_clip(const ClCall& c, float max_norm, float* norm, void* scratch, int32_t* device_status,
                      dspark_stream_t stream) {
  if (!norm || !scratch || !device_status || (reinterpret_cast<uintptr_t>(scratch) & 7u) != 0) return DSPARK_EINVAL;
  if (!(max_norm >= 0.f)) return DSPARK_EINVAL;
  bool flat = true;
  for (int i = 0; i < c.count; ++i) {
    if (c.types[i] != DSPARK_F32 && c.types[i] != DSPARK_BF16) return DSPARK_EINVAL;
    const int64_t most = (int64_t)1 << 44;
    if (c.rows) {
      if (c.rows[i] < 0 || c.cols[i] < 0 || c.rows[i] > most || c.cols[i] > most) return DSPARK_EINVAL;
      if (c.cols[i] > 0 && c.rows[i] > most / c.cols[i]) return DSPARK_EINVAL;
    } else if (c.numel[i] < 0 || c.numel[i] > most) {
      return DSPARK_EINVAL;
    }
    if (c.values(i) == 0) continue;
    if (!c.in[i] || !c.out[i]) return DSPARK_EINVAL;
    const uintptr_t mask = c.types[i] == DSPARK_BF16 ? 1u : 3u;
    if (((reinterpret_cast<uintptr_t>(c.in[i]) | reinterpret_cast<uintptr_t>(c.out[i])) & mask) != 0)
      return DSPARK_EINVAL;
    if (c.flat(i)) continue;
    if (c.ldi[i] < c.cols[i] || c.ldo[i] < c.cols[i] || c.ldi[i] > most || c.ldo[i] > most) return DSPARK_EINVAL;
    if (c.in[i] == c.out[i] && c.ldi[i] != c.ldo[i]) return DSPARK_EINVAL;
    flat = false;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(scratch);
  if (flat)
    return c.count <= 32 ? cl_call<32, false>(c, max_norm, norm, part, device_status, st)
                         : cl_call<kClLaunch, false>(c, max_norm, norm, part, device_status, st);
  return c.count <= 32 ? cl_call<32, true>(c, max_norm, norm, part, device_status, st)
                       : cl_call<kClLaunch, true>(c, max_norm, norm, part, device_status, st);
}

}  // namespace

extern "C" dspark_status dspark_clip_grads(int count, const void* const* in, void* const* out, const int64_t* numel,
                                           const int32_t* types, float max_norm, float* norm, void* scratch,
                                           int32_t* device_status, dspark_stream_t stream) {
  if (count < 0 || (count > 0 && (!in || !out || !numel || !types))) return DSPARK_EINVAL;
  const ClCall c{count, in, out, numel, nullptr, nullptr, nullptr, nullptr, types};
  return cl_clip(c, max_norm, norm, scratch, device_status, stream);
}

extern "C" dspark_status dspark_clip_grads_rows(int count, const void* const* in, void* const* out, const int64_t* rows,
                                                const int64_t* cols, const int64_t* ldi, const int64_t* ldo,
                                                const int32_t* types, float max_norm, float* norm, void* scratch,
                                                int32_t* device_status, dspark_stream_t stream) {
  if (count < 0 || (count > 0 && (!in || !out || !rows || !cols || !ldi || !ldo || !types))) return DSPARK_EINVAL;
  const ClCall c{count, in, out, nullptr, rows, cols, ldi, ldo, types};
  return cl_clip(c, max_norm, norm, scratch, device_status, stream);
}
