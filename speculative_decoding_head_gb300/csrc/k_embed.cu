// k_embed.cu -- rows of a table looked up by token, and the table's gradient.
//
//   out[n] = s E[idx_n],   dE[v] = base[v] + s sum_{n: idx_n = v} dout[n]
//
// The lookup moves each row once: a warp takes 4 rows x 64 pieces of 16 bytes
// at a time, its loads in flight together.
//
// The gradient sorts the rows by token (a stable radix sort of (token, row)
// pairs, digits of at most 10 bits: two passes up to V = 2^20) and then sums
// the sorted rows, so that dout is read once, no atomics touch dE, and the
// order of every sum is that of the rows: the same result each time. A CTA
// takes 256 consecutive sorted rows whatever tokens they hold (frequent tokens
// own long runs, rare ones short runs, most of a large vocabulary none), so the
// work is even: runs inside the CTA are written at once, a run that crosses CTAs
// leaves fp32 partial sums that the last kernel adds in order. The same launch
// writes the rows of the tokens that do not occur.
#include <math.h>
#include <stdio.h>

#include "dspark_common.cuh"
#include "dspark_internal.h"

namespace dspark {

namespace {

template <typename T>
struct Num;
template <>
struct Num<float> {
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <>
struct Num<__nv_bfloat16> {
  static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};

// Eight values of a row per lane. Rows on 16 bytes: columns c .. c + 7 with
// c = 8 lane, whole 16-byte pieces; others: columns lane + 32 i, one by one.
template <typename T, bool VEC>
__device__ __forceinline__ int col_of(int lane, int i) {
  return VEC ? lane * 8 + i : lane + 32 * i;
}
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int lane, int left, T* v) {
  if (VEC && lane * 8 + 8 <= left) {
    const uint4* p = reinterpret_cast<const uint4*>(row + lane * 8);
    uint4* o = reinterpret_cast<uint4*>(v);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) o[i] = p[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<T, VEC>(lane, i);
      v[i] = c < left ? row[c] : Num<T>::down(0.f);
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* row, int lane, int left, const T* v) {
  if (VEC && lane * 8 + 8 <= left) {
    uint4* p = reinterpret_cast<uint4*>(row + lane * 8);
    const uint4* o = reinterpret_cast<const uint4*>(v);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) p[i] = o[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<T, VEC>(lane, i);
      if (c < left) row[c] = v[i];
    }
  }
}

constexpr int kEmSpan = 256;     // columns a warp covers at a time
constexpr int kEmRows = 4;       // rows a warp of the lookup has in flight

// ---------------------------------------------------------------- lookup
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
    k_embed(const T* __restrict__ E, int64_t lde, int V, int D, const int32_t* __restrict__ idx, int N, float scale,
            T* __restrict__ out, int64_t ldo, int* status) {
  const int lane = threadIdx.x & 31;
  const int64_t spans = (D + kEmSpan - 1) / kEmSpan, groups = (N + kEmRows - 1) / kEmRows;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= spans * groups) return;
  const int g = (int)(t / spans), c0 = (int)(t - (int64_t)g * spans) * kEmSpan, left = D - c0;
  __align__(16) T v[kEmRows][8];
  int id[kEmRows];
#pragma unroll
  for (int r = 0; r < kEmRows; ++r) {
    const int n = g * kEmRows + r;
    id[r] = n < N ? idx[n] : -1;
    if (id[r] < -1 || id[r] >= V) {
      if (lane == 0) raise_status(status, DSPARK_ERANGE);
      id[r] = -1;
    }
  }
#pragma unroll
  for (int r = 0; r < kEmRows; ++r) {
    if (id[r] >= 0) {
      load8<T, VEC>(E + id[r] * lde + c0, lane, left, v[r]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][i] = Num<T>::down(0.f);
    }
  }
#pragma unroll
  for (int r = 0; r < kEmRows; ++r) {
    const int n = g * kEmRows + r;
    if (n >= N) break;
    if (id[r] >= 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][i] = Num<T>::down(scale * Num<T>::up(v[r][i]));
    }
    store8<T, VEC>(out + n * ldo + c0, lane, left, v[r]);
  }
}

// ---------------------------------------------------------------- sort
constexpr int kSoThreads = 512;
constexpr int kSoWarps = kSoThreads / 32;
constexpr int kSoBits = 10;
constexpr int kSoBins = 1 << kSoBits;
constexpr int kSoTile = 4096;    // rows of a CTA, while that leaves at most kSoCtas CTAs
constexpr int kSoCtas = 64;
constexpr size_t kSoSmem = sizeof(int) * (size_t)kSoWarps * kSoBins;

// One pass's input: the tokens themselves (rows without one are left out) or
// the pairs of the pass before.
struct SoIn {
  const int32_t* idx;
  const int2* pairs;   // (token, row)
  const int* count;    // pairs in all
  int N, V;
};
__device__ __forceinline__ int so_n(const SoIn& in) { return in.idx ? in.N : *in.count; }
__device__ __forceinline__ bool so_load(const SoIn& in, int i, int n, int2& p) {
  if (i >= n) return false;
  if (!in.idx) {
    p = in.pairs[i];
    return true;
  }
  p = make_int2(in.idx[i], i);
  return p.x >= 0 && p.x < in.V;
}

// Counts of each warp's rows by digit, in warp order: hist [warps][bins].
__device__ __forceinline__ void so_count(const SoIn& in, int a, int b, int n, int shift, int mask, int* hist,
                                         int bins) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSoWarps * bins; i += kSoThreads) hist[i] = 0;
  __syncthreads();
  const int per = (b - a + kSoWarps - 1) / kSoWarps, wa = min(b, a + warp * per), wb = min(b, wa + per);
  for (int i = wa; i < wb; i += 32) {
    int2 p;
    const bool has = i + lane < wb && so_load(in, i + lane, n, p);
    if (has) atomicAdd(&hist[warp * bins + ((p.x >> shift) & mask)], 1);
  }
  __syncthreads();
}

// The rows of [a, b) to their places: hist holds each warp's first place per digit.
__device__ __forceinline__ void so_place(const SoIn& in, int a, int b, int n, int shift, int mask, int* hist, int bins,
                                         int2* out, int32_t* rows, int32_t* toks) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (b - a + kSoWarps - 1) / kSoWarps, wa = min(b, a + warp * per), wb = min(b, wa + per);
  for (int i = wa; i < wb; i += 32) {
    int2 p;
    const bool has = i + lane < wb && so_load(in, i + lane, n, p);
    const int d = has ? (p.x >> shift) & mask : bins;  // lanes without a row match one another only
    const unsigned same = __match_any_sync(0xFFFFFFFFu, d);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int at = 0;
    if (has) at = hist[warp * bins + d] + rank;
    __syncwarp();
    if (has && rank == 0) hist[warp * bins + d] += __popc(same);
    __syncwarp();
    if (has) {
      if (out)
        out[at] = p;
      else {
        toks[at] = p.x;
        rows[at] = p.y;
      }
    }
  }
}

// Exclusive prefix of one value per thread over the first `bins` values of
// bin totals held by threads two apart; tot[bins] in shared memory, returns the sum.
__device__ __forceinline__ int so_scan(int* tot, int bins, int* wsum) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int i0 = 2 * tid, x0 = i0 < bins ? tot[i0] : 0, x1 = i0 + 1 < bins ? tot[i0 + 1] : 0;
  int s = x0 + x1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
    if (lane >= o) s += y;
  }
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  if (warp == 0) {
    int w = lane < kSoWarps ? wsum[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, w, o);
      if (lane >= o) w += y;
    }
    if (lane < kSoWarps) wsum[lane] = w;
  }
  __syncthreads();
  const int before = s - x0 - x1 + (warp > 0 ? wsum[warp - 1] : 0);
  if (i0 < bins) tot[i0] = before;
  if (i0 + 1 < bins) tot[i0 + 1] = before + x0;
  const int all = wsum[kSoWarps - 1];
  __syncthreads();
  return all;
}

// Warp counts -> first places: base[d] (start of the CTA's rows of digit d) plus the earlier warps' counts.
__device__ __forceinline__ void so_offsets(int* hist, int bins, const int* base) {
  for (int d = threadIdx.x; d < bins; d += kSoThreads) {
    int at = base[d];
    for (int w = 0; w < kSoWarps; ++w) {
      const int c = hist[w * bins + d];
      hist[w * bins + d] = at;
      at += c;
    }
  }
  __syncthreads();
}

struct SoPass {
  SoIn in;
  int shift, mask, bins;
  int per;              // rows of a CTA
  int* cta;             // [CTAs][bins] counts
  int2* out;            // pairs, or null in the last pass:
  int32_t* rows;        // [N] sorted rows
  int32_t* toks;        // [N] their tokens
  int* total;           // pairs in all (written by the first pass)
  unsigned char* seen;  // [V] token occurs (cleared by the first count, set by the first placement)
  int V;
  int* status;
};

// Bounds of a token and its mark: the first pass alone reads the tokens.
__device__ __forceinline__ void so_mark(const SoPass& p, int a, int b) {
  for (int i = a + (int)threadIdx.x; i < b; i += kSoThreads) {
    const int t = p.in.idx[i];
    if (t >= 0 && t < p.V) p.seen[t] = 1;
    if (t < -1 || t >= p.V) raise_status(p.status, DSPARK_ERANGE);
  }
}

__global__ void __launch_bounds__(kSoThreads) k_sort_count(SoPass p) {
  extern __shared__ int so_hist[];
  const int n = so_n(p.in), a = min(n, (int)blockIdx.x * p.per), b = min(n, a + p.per);
  if (p.in.idx)
    for (int i = blockIdx.x * kSoThreads + threadIdx.x; i < p.V; i += gridDim.x * kSoThreads) p.seen[i] = 0;
  so_count(p.in, a, b, n, p.shift, p.mask, so_hist, p.bins);
  for (int d = threadIdx.x; d < p.bins; d += kSoThreads) {
    int s = 0;
    for (int w = 0; w < kSoWarps; ++w) s += so_hist[w * p.bins + d];
    p.cta[blockIdx.x * p.bins + d] = s;
  }
}

__global__ void __launch_bounds__(kSoThreads) k_sort_place(SoPass p) {
  extern __shared__ int so_hist[];
  __shared__ int tot[kSoBins], mine[kSoBins], wsum[kSoWarps];
  const int n = so_n(p.in), a = min(n, (int)blockIdx.x * p.per), b = min(n, a + p.per);
  for (int d = threadIdx.x; d < p.bins; d += kSoThreads) {
    int s = 0, before = 0;
#pragma unroll 8
    for (int c = 0; c < (int)gridDim.x; ++c) {
      if (c == (int)blockIdx.x) before = s;
      s += p.cta[c * p.bins + d];
    }
    tot[d] = s;
    mine[d] = before;
  }
  so_count(p.in, a, b, n, p.shift, p.mask, so_hist, p.bins);
  const int all = so_scan(tot, p.bins, wsum);
  for (int d = threadIdx.x; d < p.bins; d += kSoThreads) mine[d] += tot[d];
  __syncthreads();
  so_offsets(so_hist, p.bins, mine);
  so_place(p.in, a, b, n, p.shift, p.mask, so_hist, p.bins, p.out, p.rows, p.toks);
  if (p.in.idx) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.total = all;
    so_mark(p, a, b);
  }
}

// All passes in one CTA, for few rows.
struct SoSmall {
  SoPass first;
  int passes, bits;
  int2* buf[2];
};

__global__ void __launch_bounds__(kSoThreads) k_sort_small(SoSmall q) {
  extern __shared__ int so_hist[];
  __shared__ int tot[kSoBins], wsum[kSoWarps];
  SoPass p = q.first;
  for (int i = threadIdx.x; i < p.V; i += kSoThreads) p.seen[i] = 0;
  int n = p.in.N;
  for (int k = 0; k < q.passes; ++k) {
    p.shift = k * q.bits;
    so_count(p.in, 0, n, n, p.shift, p.mask, so_hist, p.bins);  // its barriers order the clearing of `seen`
    for (int d = threadIdx.x; d < p.bins; d += kSoThreads) {
      int s = 0;
      for (int w = 0; w < kSoWarps; ++w) s += so_hist[w * p.bins + d];
      tot[d] = s;
    }
    __syncthreads();
    const int all = so_scan(tot, p.bins, wsum);
    so_offsets(so_hist, p.bins, tot);
    int2* out = k + 1 < q.passes ? q.buf[k & 1] : nullptr;
    so_place(p.in, 0, n, n, p.shift, p.mask, so_hist, p.bins, out, p.rows, p.toks);
    if (k == 0) {
      if (threadIdx.x == 0) *p.total = all;
      so_mark(p, 0, n);
      n = all;
    }
    __syncthreads();
    p.in.idx = nullptr;
    p.in.pairs = out;
    p.in.count = p.total;
  }
}

// ---------------------------------------------------------------- sums
constexpr int kSuRows = 256;     // sorted rows of a CTA (32 per warp)
constexpr int kSuFly = 8;        // rows a warp has in flight
constexpr int kSuFill = 32;      // vocabulary rows a CTA fills where tokens do not occur

struct SuArgs {
  const int32_t* rows;
  const int32_t* toks;
  const int* total;
  const unsigned char* seen;
  int V, D, chunks;        // chunks: CTAs of sorted rows (the others fill)
  int64_t ldd, ldb, lde;
  float scale;
  float* head;             // [chunks][D] sums of a run that begins in an earlier CTA
  float* tail;             // [chunks][D] sums of a run that goes on in the next CTA
  int has_base, fill;
};

template <typename TO, bool VEC>
__device__ __forceinline__ void su_finish(const SuArgs& a, const TO* base, TO* dE, int v, int c0, int lane, int left,
                                          const float* acc) {
  __align__(16) TO o[8];
  if (a.has_base) load8<TO, VEC>(base + v * a.ldb + c0, lane, left, o);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = a.scale * acc[i];
    o[i] = Num<TO>::down(a.has_base ? Num<TO>::up(o[i]) + s : s);
  }
  store8<TO, VEC>(dE + v * a.lde + c0, lane, left, o);
}

template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(256)
    k_embed_sum(SuArgs a, const TI* __restrict__ dout, const TO* base, TO* dE) {
  __shared__ float hd[8][kEmSpan], tl[8][kEmSpan];
  __shared__ int kfirst[8], klast[8], whole[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.y * kEmSpan, left = a.D - c0;
  if ((int)blockIdx.x >= a.chunks) {
    // tokens that do not occur: zero, or what is there already
    const int v0 = ((int)blockIdx.x - a.chunks) * kSuFill;
    __align__(16) TO o[4][8];
    int v[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      v[r] = v0 + warp * 4 + r;
      if (v[r] >= a.V || a.seen[v[r]]) v[r] = -1;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (a.has_base && v[r] >= 0) {
        load8<TO, VEC>(base + v[r] * a.ldb + c0, lane, left, o[r]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[r][i] = Num<TO>::down(0.f);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (v[r] >= 0) store8<TO, VEC>(dE + v[r] * a.lde + c0, lane, left, o[r]);
    return;
  }
  const int ns = *a.total, p0 = blockIdx.x * kSuRows;
  if (p0 >= ns) return;
  const int w0 = p0 + warp * 32, cnt = max(0, min(32, ns - w0));
  if (cnt > 0) {
    const int tok = lane < cnt ? a.toks[w0 + lane] : -1;
    const int64_t row = lane < cnt ? a.rows[w0 + lane] : 0;
    const int first = __shfl_sync(0xFFFFFFFFu, tok, 0), last = __shfl_sync(0xFFFFFFFFu, tok, cnt - 1);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    int cur = first;
    bool inner = false;  // the run began after this warp's first row
    for (int r0 = 0; r0 < cnt; r0 += kSuFly) {
      __align__(16) TI x[kSuFly][8];
#pragma unroll
      for (int f = 0; f < kSuFly; ++f) {
        const int64_t n = __shfl_sync(0xFFFFFFFFu, row, r0 + f);
        if (r0 + f < cnt) load8<TI, VEC>(dout + n * a.ldd + c0, lane, left, x[f]);
      }
#pragma unroll
      for (int f = 0; f < kSuFly; ++f) {
        const int t = __shfl_sync(0xFFFFFFFFu, tok, r0 + f);
        if (r0 + f < cnt) {
          if (t != cur) {
            if (inner) {
              su_finish<TO, VEC>(a, base, dE, cur, c0, lane, left, acc);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) hd[warp][col_of<TI, VEC>(lane, i)] = acc[i];
            }
            inner = true;
            cur = t;
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += Num<TI>::up(x[f][i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) (inner ? tl : hd)[warp][col_of<TI, VEC>(lane, i)] = acc[i];
    if (lane == 0) {
      kfirst[warp] = first;
      klast[warp] = last;
      whole[warp] = !inner;
    }
  }
  __syncthreads();
  // the warps' first and last runs, joined in order, one column per thread
  const int c = threadIdx.x;
  if (c >= left) return;
  const int nw = min(8, (ns - p0 + 31) / 32);
  float cur = 0.f;
  int key = kfirst[0];
  bool begun = p0 == 0 || a.toks[p0 - 1] != key;  // the run begins in this CTA
  auto flush = [&]() {
    if (!begun) {
      a.head[(int64_t)blockIdx.x * a.D + c0 + c] = cur;
      return;
    }
    TO* o = dE + key * a.lde + c0 + c;
    const float s = a.scale * cur;
    *o = Num<TO>::down(a.has_base ? Num<TO>::up(base[key * a.ldb + c0 + c]) + s : s);
  };
  for (int w = 0; w < nw; ++w) {
    if (w > 0 && kfirst[w] != key) {
      flush();
      cur = 0.f;
      key = kfirst[w];
      begun = true;
    }
    cur += hd[w][c];
    if (!whole[w]) {
      flush();
      cur = tl[w][c];
      key = klast[w];
      begun = true;
    }
  }
  const bool on = p0 + kSuRows < ns && a.toks[p0 + kSuRows] == key;  // it goes on in the next CTA
  if (on && begun)
    a.tail[(int64_t)blockIdx.x * a.D + c0 + c] = cur;
  else if (on)
    a.head[(int64_t)blockIdx.x * a.D + c0 + c] = cur;
  else
    flush();
}

// Runs that cross CTAs: the CTA of the chunk where one begins adds the tail
// there and the heads of the chunks that follow, four quarters side by side,
// each in order.
template <typename TO>
__global__ void __launch_bounds__(1024)
    k_embed_join(SuArgs a, const TO* base, TO* dE) {
  __shared__ float part[4][kEmSpan];
  const int ns = *a.total, ch = blockIdx.x, p0 = ch * kSuRows, p1 = p0 + kSuRows;
  if (p1 >= ns) return;
  const int key = a.toks[p1];
  if (a.toks[p1 - 1] != key) return;                                             // no run crosses here
  if (a.toks[p0] == key && p0 > 0 && a.toks[p0 - 1] == key) return;              // it began earlier
  // last chunk whose first row is still this token's
  int lo = ch + 1, hi = (ns - 1) / kSuRows;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.toks[mid * kSuRows] == key)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int c = threadIdx.x & (kEmSpan - 1), g = threadIdx.x / kEmSpan, col = blockIdx.y * kEmSpan + c;
  const int m = lo - ch, per = (m + 3) / 4, i0 = ch + 1 + min(m, g * per), i1 = ch + 1 + min(m, (g + 1) * per);
  float s = 0.f;
  if (col < a.D) {
#pragma unroll 8
    for (int i = i0; i < i1; ++i) s += a.head[(int64_t)i * a.D + col];
  }
  part[g][c] = s;
  __syncthreads();
  if (g != 0 || col >= a.D) return;
  float t = a.tail[(int64_t)ch * a.D + col];
#pragma unroll
  for (int q = 0; q < 4; ++q) t += part[q][c];
  t *= a.scale;
  dE[key * a.lde + col] = Num<TO>::down(a.has_base ? Num<TO>::up(base[key * a.ldb + col]) + t : t);
}

// ---------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct EmScratch {
  size_t rows, toks, bufa, bufb, cta, total, seen, head, tail, all;
  int chunks;
};
EmScratch em_scratch(int N, int V, int D) {
  EmScratch s;
  size_t off = 0;
  auto carve = [&](size_t bytes) {
    const size_t o = off;
    off += up256(bytes > 0 ? bytes : 1);
    return o;
  };
  s.chunks = (N + kSuRows - 1) / kSuRows;
  s.rows = carve(4 * (size_t)N);
  s.toks = carve(4 * (size_t)N);
  s.bufa = carve(8 * (size_t)N);
  s.bufb = carve(8 * (size_t)N);
  s.cta = carve(sizeof(int) * (size_t)kSoCtas * kSoBins);
  s.total = carve(4);
  s.seen = carve((size_t)V);
  s.head = carve(4 * (size_t)s.chunks * D);
  s.tail = carve(4 * (size_t)s.chunks * D);
  s.all = off;
  return s;
}

bool em_dims_ok(int N, int V, int D) {
  return N >= 0 && N <= (1 << 24) && V >= 1 && V <= (1 << 24) && D >= 1 && D <= (1 << 20);
}
bool em_type_ok(int t) { return t == DSPARK_F32 || t == DSPARK_BF16; }
bool em_ptr_ok(const void* p, int type) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (type == DSPARK_BF16 ? 1u : 3u)) == 0;
}
bool em_vec(const void* p, int64_t ld, int type) {
  const int64_t size = type == DSPARK_BF16 ? 2 : 4;
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * size) % 16 == 0;
}

dspark_status em_fail(cudaError_t e) {
  if (e == cudaSuccess) return DSPARK_OK;
  fprintf(stderr, "dspark: CUDA error %s\n", cudaGetErrorString(e));
  return DSPARK_ECUDA;
}

cudaError_t em_sort(const int32_t* idx, int N, int V, char* base, const EmScratch& s, int* status, cudaStream_t st) {
  static bool configured = false;
  if (!configured) {
    cudaError_t e = cudaFuncSetAttribute(k_sort_count, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSoSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_sort_place, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSoSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k_sort_small, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSoSmem);
    if (e != cudaSuccess) return e;
    configured = true;
  }
  int width = 1;
  while (width < 24 && (1 << width) < V) ++width;
  const int passes = (width + kSoBits - 1) / kSoBits, bits = (width + passes - 1) / passes;
  int2* buf[2] = {reinterpret_cast<int2*>(base + s.bufa), reinterpret_cast<int2*>(base + s.bufb)};
  SoPass p;
  p.in.idx = idx;
  p.in.pairs = nullptr;
  p.in.count = nullptr;
  p.in.N = N;
  p.in.V = V;
  p.bins = 1 << bits;
  p.mask = p.bins - 1;
  p.shift = 0;
  p.cta = reinterpret_cast<int*>(base + s.cta);
  p.rows = reinterpret_cast<int32_t*>(base + s.rows);
  p.toks = reinterpret_cast<int32_t*>(base + s.toks);
  p.total = reinterpret_cast<int*>(base + s.total);
  p.seen = reinterpret_cast<unsigned char*>(base + s.seen);
  p.V = V;
  p.status = status;
  p.out = nullptr;
  p.per = N;
  const size_t smem = sizeof(int) * (size_t)kSoWarps * p.bins;
  if (N <= 2 * kSoTile) {
    SoSmall q{p, passes, bits, {buf[0], buf[1]}};
    k_sort_small<<<1, kSoThreads, smem, st>>>(q);
    return cudaGetLastError();
  }
  int ctas = (N + kSoTile - 1) / kSoTile;
  if (ctas > kSoCtas) ctas = kSoCtas;
  p.per = (N + ctas - 1) / ctas;
  cudaError_t e = cudaSuccess;
  for (int k = 0; k < passes && e == cudaSuccess; ++k) {
    p.shift = k * bits;
    p.out = k + 1 < passes ? buf[k & 1] : nullptr;
    k_sort_count<<<ctas, kSoThreads, smem, st>>>(p);
    k_sort_place<<<ctas, kSoThreads, smem, st>>>(p);
    e = cudaGetLastError();
    p.in.idx = nullptr;
    p.in.pairs = p.out;
    p.in.count = p.total;
  }
  return e;
}

template <typename TI, typename TO, bool VEC>
cudaError_t em_sum(const SuArgs& a, const void* dout, const void* base, void* dE, cudaStream_t st) {
  const int fills = a.fill ? (a.V + kSuFill - 1) / kSuFill : 0;
  const int spans = (a.D + kEmSpan - 1) / kEmSpan;
  if (a.chunks + fills > 0)
    k_embed_sum<TI, TO, VEC><<<dim3(a.chunks + fills, spans), 256, 0, st>>>(
        a, static_cast<const TI*>(dout), static_cast<const TO*>(base), static_cast<TO*>(dE));
  if (a.chunks > 1)
    k_embed_join<TO><<<dim3(a.chunks - 1, spans), 1024, 0, st>>>(a, static_cast<const TO*>(base),
                                                                  static_cast<TO*>(dE));
  return cudaGetLastError();
}
template <typename TI, typename TO>
cudaError_t em_sum_v(bool vec, const SuArgs& a, const void* dout, const void* base, void* dE, cudaStream_t st) {
  return vec ? em_sum<TI, TO, true>(a, dout, base, dE, st) : em_sum<TI, TO, false>(a, dout, base, dE, st);
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_embed(const void* E, dspark_wdtype type, int64_t lde, int V, int D, const int32_t* idx,
                                      int N, float scale, void* out, int64_t ldo, int32_t* device_status,
                                      dspark_stream_t stream) {
  if (!em_dims_ok(N, V, D) || !em_type_ok(type) || !device_status || lde < D || ldo < D) return DSPARK_EINVAL;
  if (N == 0) return DSPARK_OK;
  if (!em_ptr_ok(E, type) || !em_ptr_ok(out, type) || !em_ptr_ok(idx, DSPARK_F32)) return DSPARK_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool vec = em_vec(E, lde, type) && em_vec(out, ldo, type);
  const int64_t warps = (int64_t)((N + kEmRows - 1) / kEmRows) * ((D + kEmSpan - 1) / kEmSpan);
  const unsigned grid = (unsigned)((warps + 7) / 8);
  if (type == DSPARK_BF16) {
    const auto* e = static_cast<const __nv_bfloat16*>(E);
    auto* o = static_cast<__nv_bfloat16*>(out);
    if (vec)
      k_embed<__nv_bfloat16, true><<<grid, 256, 0, st>>>(e, lde, V, D, idx, N, scale, o, ldo, device_status);
    else
      k_embed<__nv_bfloat16, false><<<grid, 256, 0, st>>>(e, lde, V, D, idx, N, scale, o, ldo, device_status);
  } else {
    const auto* e = static_cast<const float*>(E);
    auto* o = static_cast<float*>(out);
    if (vec)
      k_embed<float, true><<<grid, 256, 0, st>>>(e, lde, V, D, idx, N, scale, o, ldo, device_status);
    else
      k_embed<float, false><<<grid, 256, 0, st>>>(e, lde, V, D, idx, N, scale, o, ldo, device_status);
  }
  return em_fail(cudaGetLastError());
}

extern "C" size_t dspark_embed_grad_scratch_bytes(int N, int V, int D) {
  if (!em_dims_ok(N, V, D)) return 0;
  return em_scratch(N, V, D).all;
}

extern "C" dspark_status dspark_embed_grad(const void* dout, dspark_wdtype type, int64_t ldd, const int32_t* idx, int N,
                                           int V, int D, float scale, const void* base, int64_t ldb, void* dE,
                                           dspark_wdtype grad_type, int64_t lde, void* scratch, int32_t* device_status,
                                           dspark_stream_t stream) {
  if (!em_dims_ok(N, V, D) || !em_type_ok(type) || !em_type_ok(grad_type) || !device_status) return DSPARK_EINVAL;
  if (ldd < D || lde < D || (base && ldb < D)) return DSPARK_EINVAL;
  if (!em_ptr_ok(dE, grad_type) || (base && !em_ptr_ok(base, grad_type))) return DSPARK_EINVAL;
  if (base == dE && base && ldb != lde) return DSPARK_EINVAL;
  if (N > 0 && (!em_ptr_ok(dout, type) || !em_ptr_ok(idx, DSPARK_F32))) return DSPARK_EINVAL;
  if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u) != 0) return DSPARK_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const EmScratch s = em_scratch(N, V, D);
  char* b = static_cast<char*>(scratch);
  const cudaError_t e = em_sort(idx, N, V, b, s, device_status, st);
  if (e != cudaSuccess) return em_fail(e);
  SuArgs a;
  a.rows = reinterpret_cast<const int32_t*>(b + s.rows);
  a.toks = reinterpret_cast<const int32_t*>(b + s.toks);
  a.total = reinterpret_cast<const int*>(b + s.total);
  a.seen = reinterpret_cast<const unsigned char*>(b + s.seen);
  a.V = V;
  a.D = D;
  a.chunks = s.chunks;
  a.ldd = ldd;
  a.ldb = ldb;
  a.lde = lde;
  a.scale = scale;
  a.head = reinterpret_cast<float*>(b + s.head);
  a.tail = reinterpret_cast<float*>(b + s.tail);
  a.has_base = base != nullptr;
  a.fill = base != dE;  // added in place: the other rows stay as they are
  const bool vec = em_vec(dout, ldd, type) && em_vec(dE, lde, grad_type) && (!base || em_vec(base, ldb, grad_type));
  typedef __nv_bfloat16 bf;
  if (type == DSPARK_BF16)
    return em_fail(grad_type == DSPARK_BF16 ? em_sum_v<bf, bf>(vec, a, dout, base, dE, st)
                                            : em_sum_v<bf, float>(vec, a, dout, base, dE, st));
  return em_fail(grad_type == DSPARK_BF16 ? em_sum_v<float, bf>(vec, a, dout, base, dE, st)
                                          : em_sum_v<float, float>(vec, a, dout, base, dE, st));
}
