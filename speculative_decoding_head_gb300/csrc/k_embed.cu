// k_embed.cu -- rows of a table looked up by token, and the table's gradient.
//
//   out[n] = s E[idx_n],   dE[v] = base[v] + s sum_{n: idx_n = v} dout[n]
//
// The lookup moves each row once: a warp takes 4 rows and one or two spans of 256
// columns at a time (more rows where they are short), its loads in flight together. 16384 rows of 5120 bf16: 43 us,
// 81% of the measured copy rate (one span a warp: 59 us); small calls are one
// launch's latency (4.2 us on the device).
//
// The gradient sorts the rows by token (a stable radix sort of (token, row)
// pairs, digits of at most 10 bits: two passes up to V = 2^20) and then sums
// the sorted rows, so that dout is read once, no atomics touch dE, and the
// order of every sum is that of the rows: the same result each time. A CTA
// takes up to 256 consecutive sorted rows whatever tokens they hold (frequent
// tokens own long runs, rare ones short runs, most of a large vocabulary none),
// so the work is even: runs inside the CTA are written at once, a run that
// crosses CTAs leaves fp32 partial sums that the last kernel adds in order. That
// kernel also writes the rows of the tokens that do not occur.
//
// 262144 rows of 256 bf16 into V = 129280: 66.5 us, 2.4 times the floor of its
// bytes: 22 us of sort (four launches, each a chain of latencies: load, count,
// add up, place), 32 us of sums (512-byte rows in random order, 4.7 TB/s) and
// 12 us of joins and absent rows.
#include <math.h>
#include <stdio.h>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "tc_ptx.cuh"

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
// c = 8 lane, whole 16-byte pieces; others: columns lane + LANES i, one by one
// (LANES lanes to a row).
template <typename T, bool VEC, int LANES = 32>
__device__ __forceinline__ int col_of(int lane, int i) {
  return VEC ? lane * 8 + i : lane + LANES * i;
}
template <typename T, bool VEC, int LANES = 32>
__device__ __forceinline__ void load8(const T* row, int lane, int left, T* v) {
  if (VEC && lane * 8 + 8 <= left) {
    const uint4* p = reinterpret_cast<const uint4*>(row + lane * 8);
    uint4* o = reinterpret_cast<uint4*>(v);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) o[i] = p[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<T, VEC, LANES>(lane, i);
      v[i] = c < left ? row[c] : Num<T>::down(0.f);
    }
  }
}
template <typename T, bool VEC, int LANES = 32>
__device__ __forceinline__ void store8(T* row, int lane, int left, const T* v) {
  if (VEC && lane * 8 + 8 <= left) {
    uint4* p = reinterpret_cast<uint4*>(row + lane * 8);
    const uint4* o = reinterpret_cast<const uint4*>(v);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) p[i] = o[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = col_of<T, VEC, LANES>(lane, i);
      if (c < left) row[c] = v[i];
    }
  }
}

constexpr int kEmSpan = 256;     // columns a warp covers at a time
constexpr int kEmRows = 4;       // rows a lane of the lookup has in flight

// ---------------------------------------------------------------- lookup
// LANES lanes to a row: CH spans of 8 LANES columns of four rows each, all loads
// in flight together. Fewer than 32 lanes where rows are short and many (192139
// rows, 32 lanes and as chosen: 9 bf16 27.1 and 5.9 us, 64 bf16 31.7 and 6.8, 128
// bf16 31.7 and 11.7; 4000 rows of 16 fp32: 2.2 with 32 lanes, 3.1 with two).
constexpr int kEmMany = 8192;
template <typename T, bool VEC, int CH, int LANES>
__global__ void __launch_bounds__(256)
    k_embed(const T* __restrict__ E, int64_t lde, int V, int D, const int32_t* __restrict__ idx, int N, float scale,
            T* __restrict__ out, int64_t ldo, int* status) {
  constexpr int kSpan = 8 * LANES, kCols = CH * kSpan;
  const int lane = threadIdx.x & (LANES - 1);
  const int spans = (D + kCols - 1) / kCols, groups = (N + kEmRows - 1) / kEmRows;
  const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  pdl_wait();
  if (t >= (int64_t)spans * groups) return;
  // a group's rows lie `stride` apart, so that the groups of a warp read and write rows side by side
  const int g = (int)(t / spans), c0 = (int)(t - (int64_t)g * spans) * kCols, left = D - c0;
  const int stride = LANES < 32 ? groups : 1, n0 = LANES < 32 ? g : g * kEmRows;
  __align__(16) T v[kEmRows][CH][8];
  int id[kEmRows];
#pragma unroll
  for (int r = 0; r < kEmRows; ++r) {
    const int n = n0 + r * stride;
    id[r] = n < N ? idx[n] : -1;
    if (id[r] < -1 || id[r] >= V) {
      if (lane == 0) raise_status(status, DSPARK_ERANGE);
      id[r] = -1;
    }
  }
#pragma unroll
  for (int r = 0; r < kEmRows; ++r)
#pragma unroll
    for (int h = 0; h < CH; ++h) {
      if (id[r] >= 0) {
        load8<T, VEC, LANES>(E + id[r] * lde + c0 + h * kSpan, lane, left - h * kSpan, v[r][h]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[r][h][i] = Num<T>::down(0.f);
      }
    }
#pragma unroll
  for (int r = 0; r < kEmRows; ++r) {
    const int n = n0 + r * stride;
    if (n >= N) break;
#pragma unroll
    for (int h = 0; h < CH; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[r][h][i] = Num<T>::down(id[r] >= 0 ? scale * Num<T>::up(v[r][h][i]) : 0.f);
      store8<T, VEC, LANES>(out + n * ldo + c0 + h * kSpan, lane, left - h * kSpan, v[r][h]);
    }
  }
}

template <typename T, bool VEC, int CH, int LANES>
cudaError_t em_lookup_as(const void* E, int64_t lde, int V, int D, const int32_t* idx, int N, float scale, void* out,
                         int64_t ldo, int* status, cudaStream_t st) {
  const int64_t groups = (int64_t)((N + kEmRows - 1) / kEmRows) * ((D + 8 * LANES * CH - 1) / (8 * LANES * CH));
  return launch_ex(k_embed<T, VEC, CH, LANES>, dim3((unsigned)((groups * LANES + 255) / 256)), dim3(256), 0, st, true,
                   static_cast<const T*>(E), lde, V, D, idx, N, scale, static_cast<T*>(out), ldo, status);
}
template <typename T, bool VEC>
cudaError_t em_lookup_v(const void* E, int64_t lde, int V, int D, const int32_t* idx, int N, float scale, void* out,
                        int64_t ldo, int* status, cudaStream_t st) {
  const auto f = D > kEmSpan && sizeof(T) == 2 ? em_lookup_as<T, VEC, 2, 32>
                 : D > 128 || N < kEmMany      ? em_lookup_as<T, VEC, 1, 32>
                 : D > 64                      ? em_lookup_as<T, VEC, 1, 16>
                 : D > 16                      ? em_lookup_as<T, VEC, 1, 4>
                                               : em_lookup_as<T, VEC, 1, 2>;
  return f(E, lde, V, D, idx, N, scale, out, ldo, status, st);
}
template <typename T>
cudaError_t em_lookup(bool vec, const void* E, int64_t lde, int V, int D, const int32_t* idx, int N, float scale,
                      void* out, int64_t ldo, int* status, cudaStream_t st) {
  return (vec ? em_lookup_v<T, true> : em_lookup_v<T, false>)(E, lde, V, D, idx, N, scale, out, ldo, status, st);
}

// ---------------------------------------------------------------- sort
constexpr int kSoThreads = 1024;
constexpr int kSoWarps = kSoThreads / 32;
constexpr int kSoBits = 10;
constexpr int kSoBins = 1 << kSoBits;
constexpr int kSoCtas = 128;
constexpr int kSoAhead = 32;                            // counts of other CTAs a thread has on their way
constexpr size_t kSoSmem = sizeof(int) * (size_t)kSoWarps * kSoBins;

// One pass's input: the tokens themselves (rows without one are left out) or
// the pairs of the pass before.
struct SoPass {
  const int32_t* idx;   // [N], or null:
  const int2* pairs;    // (token, row)
  int N, V;
  int shift, bins;
  int per;              // pairs of a CTA (whole tiles of kSoThreads * KEYS)
  int* cta;             // [CTAs][bins] counts
  int2* out;            // pairs, or null in the last pass:
  int32_t* rows;        // [N] sorted rows
  int32_t* toks;        // [N] their tokens
  int* total;           // pairs in all (written by the first pass)
  unsigned char* seen;  // [V] token occurs (cleared here, set where the rows are summed; room for whole 16 bytes)
  int* status;
};

// A warp's pairs of the tile that begins at a: KEYS runs of 32 in order. A
// row without a token has digit -1.
template <int KEYS>
struct SoKeys {
  int2 p[KEYS];
  int d[KEYS];
};
template <int KEYS>
__device__ __forceinline__ void so_load(const SoPass& q, int a, int n, SoKeys<KEYS>& k) {
  const int w0 = a + (threadIdx.x >> 5) * (32 * KEYS) + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const int at = w0 + 32 * i;
    k.p[i] = make_int2(-1, at);
    if (at < n) {
      if (q.idx)
        k.p[i].x = q.idx[at];
      else
        k.p[i] = q.pairs[at];
    }
  }
#pragma unroll
  for (int i = 0; i < KEYS; ++i)
    k.d[i] = k.p[i].x >= 0 && k.p[i].x < q.V ? (k.p[i].x >> q.shift) & (q.bins - 1) : -1;
}

// Counts of each warp's pairs by digit into hist [warps][bins].
template <int KEYS>
__device__ __forceinline__ void so_count(const SoKeys<KEYS>& k, int* hist, int bins) {
  for (int i = threadIdx.x; i < kSoWarps * bins; i += kSoThreads) hist[i] = 0;
  __syncthreads();
  int* h = hist + (threadIdx.x >> 5) * bins;
#pragma unroll
  for (int i = 0; i < KEYS; ++i)
    if (k.d[i] >= 0) atomicAdd(h + k.d[i], 1);
  __syncthreads();
}

// The pairs to their places: hist holds each warp's first place per digit.
template <int KEYS>
__device__ __forceinline__ void so_place(const SoPass& q, const SoKeys<KEYS>& k, int* hist) {
  const int lane = threadIdx.x & 31;
  int* h = hist + (threadIdx.x >> 5) * q.bins;
#pragma unroll
  for (int i = 0; i < KEYS; ++i) {
    const unsigned same = __match_any_sync(0xFFFFFFFFu, k.d[i]);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int at = 0;
    if (k.d[i] >= 0) at = h[k.d[i]] + rank;
    __syncwarp();
    if (k.d[i] >= 0 && rank == 0) h[k.d[i]] += __popc(same);
    __syncwarp();
    if (k.d[i] < 0) continue;
    if (q.out) {
      q.out[at] = k.p[i];
    } else {
      q.toks[at] = k.p[i].x;
      q.rows[at] = k.p[i].y;
    }
  }
}

// Tokens out of range reported (first pass).
template <int KEYS>
__device__ __forceinline__ void so_check(const SoPass& q, const SoKeys<KEYS>& k) {
#pragma unroll
  for (int i = 0; i < KEYS; ++i)
    if (k.d[i] < 0 && k.p[i].x != -1) raise_status(q.status, DSPARK_ERANGE);
}

// tot[bins] in shared memory to its exclusive prefix; returns the sum.
__device__ __forceinline__ int so_scan(int* tot, int bins, int* wsum) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int x0 = tid < bins ? tot[tid] : 0;
  int s = x0;
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
  if (tid < bins) tot[tid] = s - x0 + (warp > 0 ? wsum[warp - 1] : 0);
  const int all = wsum[kSoWarps - 1];
  __syncthreads();
  return all;
}

// Warp counts -> first places from base[d] on; base[d] moves past the tile's pairs.
__device__ __forceinline__ void so_offsets(int* hist, int bins, int* base) {
  for (int d = threadIdx.x; d < bins; d += kSoThreads) {
    int at = base[d];
#pragma unroll 8
    for (int w = 0; w < kSoWarps; ++w) {
      const int c = hist[w * bins + d];
      hist[w * bins + d] = at;
      at += c;
    }
    base[d] = at;
  }
  __syncthreads();
}

__device__ __forceinline__ int so_n(const SoPass& q) { return q.idx ? q.N : *q.total; }

template <int KEYS>
__global__ void __launch_bounds__(kSoThreads) k_sort_count(SoPass q) {
  extern __shared__ int so_hist[];
  pdl_wait();
  if (q.idx)
    for (int i = blockIdx.x * kSoThreads + threadIdx.x; i < (q.V + 15) / 16; i += gridDim.x * kSoThreads)
      reinterpret_cast<uint4*>(q.seen)[i] = make_uint4(0, 0, 0, 0);
  const int n = so_n(q), a = min(n, (int)blockIdx.x * q.per), b = min(n, a + q.per);
  for (int i = threadIdx.x; i < q.bins; i += kSoThreads) so_hist[i] = 0;
  __syncthreads();
  for (int t = a; t < b; t += kSoThreads * KEYS) {
    SoKeys<KEYS> k;
    so_load(q, t, b, k);
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
      if (k.d[i] >= 0) atomicAdd(so_hist + k.d[i], 1);
    if (q.idx) so_check(q, k);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < q.bins; d += kSoThreads) q.cta[blockIdx.x * q.bins + d] = so_hist[d];
}

template <int KEYS>
__global__ void __launch_bounds__(kSoThreads) k_sort_place(SoPass q) {
  extern __shared__ int so_hist[];
  __shared__ int tot[kSoBins], mine[kSoBins], wsum[kSoWarps];
  pdl_wait();
  const int n = so_n(q), a = min(n, (int)blockIdx.x * q.per), b = min(n, a + q.per);
  SoKeys<KEYS> k;
  so_load(q, a, b, k);
  // a digit's counts of all CTAs: kSoThreads / bins threads share them; the first
  // ones are on their way while the first tile is counted
  const int digit = threadIdx.x & (q.bins - 1), share = kSoThreads / q.bins;
  const int span = ((int)gridDim.x + share - 1) / share, i0 = threadIdx.x / q.bins * span;
  const int i1 = min((int)gridDim.x, i0 + span);
  const int* c = q.cta + digit;
  int x[kSoAhead];
#pragma unroll
  for (int i = 0; i < kSoAhead; ++i) x[i] = i0 + i < i1 ? c[(i0 + i) * q.bins] : 0;
  for (int d = threadIdx.x; d < q.bins; d += kSoThreads) tot[d] = mine[d] = 0;
  so_count(k, so_hist, q.bins);
  int s = 0, before = 0;
#pragma unroll
  for (int i = 0; i < kSoAhead; ++i) {
    before += i0 + i < (int)blockIdx.x ? x[i] : 0;
    s += x[i];
  }
#pragma unroll 16
  for (int i = i0 + kSoAhead; i < i1; ++i) {
    const int y = c[i * q.bins];
    before += i < (int)blockIdx.x ? y : 0;
    s += y;
  }
  atomicAdd(&tot[digit], s);
  atomicAdd(&mine[digit], before);
  __syncthreads();
  const int all = so_scan(tot, q.bins, wsum);
  for (int d = threadIdx.x; d < q.bins; d += kSoThreads) mine[d] += tot[d];
  if (q.idx && blockIdx.x == 0 && threadIdx.x == 0) *q.total = all;
  for (int t = a; t < b; t += kSoThreads * KEYS) {
    if (t > a) {
      so_load(q, t, b, k);
      so_count(k, so_hist, q.bins);
    }
    so_offsets(so_hist, q.bins, mine);
    so_place(q, k, so_hist);
    __syncthreads();
  }
}

// All passes in one launch, for up to 32768 rows: a cluster of eight CTAs of up
// to four pairs a thread, which read one another's counts in shared memory. The
// call with 8190 rows of 1001 fp32 into V = 32000: 67.7 us; with a launch per step
// 74. 4096 rows: 33 us; in one CTA 36.5.
constexpr int kScCtas = 8;
struct ScArgs {
  SoPass first;
  int passes, bits;
  int2* buf[2];
};

template <int KEYS>
__global__ void __cluster_dims__(kScCtas, 1, 1) __launch_bounds__(kSoThreads) k_sort_cluster(ScArgs s) {
  extern __shared__ int so_hist[];
  __shared__ int cnt[kSoBins], tot[kSoBins], mine[kSoBins], wsum[kSoWarps];
  const int rank = blockIdx.x, d = threadIdx.x;
  pdl_wait();
  SoPass q = s.first;
  for (int i = rank * kSoThreads + d; i < (q.V + 15) / 16; i += kScCtas * kSoThreads)
    reinterpret_cast<uint4*>(q.seen)[i] = make_uint4(0, 0, 0, 0);
  int n = q.N;
  for (int pass = 0; pass < s.passes; ++pass) {
    q.shift = pass * s.bits;
    q.out = pass + 1 < s.passes ? s.buf[pass & 1] : nullptr;
    SoKeys<KEYS> k;
    so_load(q, rank * kSoThreads * KEYS, n, k);
    so_count(k, so_hist, q.bins);
    if (d < q.bins) {
      int c = 0;
#pragma unroll
      for (int w = 0; w < kSoWarps; ++w) c += so_hist[w * q.bins + d];
      cnt[d] = c;
    }
    tc::cluster_sync();
    if (d < q.bins) {
      int all = 0, before = 0;
#pragma unroll
      for (int c = 0; c < kScCtas; ++c) {
        const int x = tc::ld_rank(tc::smem_u32(cnt + d), c);
        before += c < rank ? x : 0;
        all += x;
      }
      tot[d] = all;
      mine[d] = before;
    }
    const int all = so_scan(tot, q.bins, wsum);
    if (d < q.bins) mine[d] += tot[d];
    so_offsets(so_hist, q.bins, mine);
    so_place(q, k, so_hist);
    if (pass == 0) {
      so_check(q, k);
      if (rank == 0 && d == 0) *q.total = all;
      n = all;
    }
    tc::cluster_sync();  // the pairs are there, and cnt has been read
    q.idx = nullptr;
    q.pairs = q.out;
  }
}

// ---------------------------------------------------------------- sums
constexpr int kSuWarp = 32;      // sorted rows of a warp at most (8 warps a CTA)
constexpr int kSuGroup = 4;      // rows asked for together
constexpr int kSuGroups = 2;     // groups a warp has on their way or at hand
constexpr int kSuFill = 64;      // vocabulary rows a CTA of the last launch fills where tokens do not occur

struct SuArgs {
  const int32_t* rows;
  const int32_t* toks;
  const int* total;
  unsigned char* seen;
  int V, D, chunks;        // chunks: CTAs of sorted rows
  int fills;               // CTAs that fill
  int64_t ldp;             // of head and tail: D rounded up to 4
  int64_t ldd, ldb, lde;
  float scale;
  float* head;             // [chunks][ldp] sums of a run that begins in an earlier CTA
  float* tail;             // [chunks][ldp] sums of a run that goes on in the next CTA
  int rpw;                 // sorted rows of a warp
  int has_base;
};

// o: the base's values of the row (with has_base), taken over by the result
template <typename TO, bool VEC>
__device__ __forceinline__ void su_finish(const SuArgs& a, TO* o, TO* dE, int v, int c0, int lane, int left,
                                          const float* acc) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = a.scale * acc[i];
    o[i] = Num<TO>::down(a.has_base ? Num<TO>::up(o[i]) + s : s);
  }
  store8<TO, VEC>(dE + v * a.lde + c0, lane, left, o);
}

template <typename TI>
constexpr size_t su_smem() {
  return (size_t)8 * kSuGroups * kSuGroup * kEmSpan * sizeof(TI);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Eight values of a row (a lane's) to shared memory, from where the same lane
// takes them: asynchronously where the row's pieces lie on 16 bytes.
template <typename TI, bool VEC>
__device__ __forceinline__ void su_stage(const TI* row, int lane, int left, TI* to) {
  if (VEC && lane * 8 + 8 <= left) {
    const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(to));
#pragma unroll
    for (int i = 0; i < (int)sizeof(TI) / 2; ++i) cp_async16(d + 16 * i, row + lane * 8 + 16 / sizeof(TI) * i);
  } else {
    __align__(16) TI x[8];
    load8<TI, VEC>(row, lane, left, x);
#pragma unroll
    for (int i = 0; i < (int)sizeof(TI) / 2; ++i)
      reinterpret_cast<uint4*>(to)[i] = reinterpret_cast<const uint4*>(x)[i];
  }
}

template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(256, sizeof(TI) == 2 ? 4 : 2)
    k_embed_sum(SuArgs a, const TI* __restrict__ dout, const TO* base, TO* dE) {
  extern __shared__ __align__(16) unsigned char su_ring[];
  __shared__ __align__(16) float hd[8][kEmSpan], tl[8][kEmSpan];
  __shared__ int kfirst[8], klast[8], whole[8];
  constexpr int G = kSuGroups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = blockIdx.y * kEmSpan, left = a.D - c0;
  TI* ring = reinterpret_cast<TI*>(su_ring) + (size_t)warp * G * kSuGroup * kEmSpan + lane * 8;
  pdl_wait();
  const int ns = *a.total, crows = 8 * a.rpw, p0 = blockIdx.x * crows;
  if (p0 >= ns) return;
  const int w0 = p0 + warp * a.rpw, cnt = max(0, min(a.rpw, ns - w0));
  if (cnt > 0) {
    const int tok = lane < cnt ? a.toks[w0 + lane] : -1;
    const int row = lane < cnt ? a.rows[w0 + lane] : 0;
    const int left_tok = __shfl_up_sync(0xFFFFFFFFu, tok, 1);
    if (blockIdx.y == 0 && lane < cnt && (lane == 0 || tok != left_tok)) a.seen[tok] = 1;
    const int first = __shfl_sync(0xFFFFFFFFu, tok, 0), last = __shfl_sync(0xFFFFFFFFu, tok, cnt - 1);
    // ask for the group that begins with row r0 (the last ones: empty groups keep the count)
    auto ask = [&](int r0) {
#pragma unroll
      for (int f = 0; f < kSuGroup; ++f) {
        const int r = r0 + f;
        const int64_t n = __shfl_sync(0xFFFFFFFFu, row, r & 31);
        if (r < cnt)
          su_stage<TI, VEC>(dout + n * a.ldd + c0, lane, left, ring + (r % (G * kSuGroup)) * kEmSpan);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int g = 0; g < G - 1; ++g) ask(g * kSuGroup);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    int cur = first;
    bool inner = false;  // the run began after this warp's first row
    __align__(16) TO o[8];
#pragma unroll 1
    for (int r = 0; r < cnt; ++r) {
      if ((r & (kSuGroup - 1)) == 0) {
        ask(r + (G - 1) * kSuGroup);
        asm volatile("cp.async.wait_group %0;" ::"n"(G - 1) : "memory");
      }
      const int t = __shfl_sync(0xFFFFFFFFu, tok, r);
      if (t != cur) {
        if (inner) {
          su_finish<TO, VEC>(a, o, dE, cur, c0, lane, left, acc);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) hd[warp][col_of<TI, VEC>(lane, i)] = acc[i];
        }
        inner = true;
        cur = t;
        if (a.has_base) load8<TO, VEC>(base + cur * a.ldb + c0, lane, left, o);  // needed when the run ends
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      }
      __align__(16) TI x[8];
#pragma unroll
      for (int i = 0; i < (int)sizeof(TI) / 2; ++i)
        reinterpret_cast<uint4*>(x)[i] =
            reinterpret_cast<const uint4*>(ring + (r % (G * kSuGroup)) * kEmSpan)[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += Num<TI>::up(x[i]);
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
  const int nw = min(8, (ns - p0 + a.rpw - 1) / a.rpw);
  // what the rows of the warps' first and last tokens are added to, asked for at once
  TO bfirst[8], blast[8];
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    bfirst[w] = blast[w] = Num<TO>::down(0.f);
    if (a.has_base && w < nw) {
      bfirst[w] = base[kfirst[w] * a.ldb + c0 + c];
      blast[w] = base[klast[w] * a.ldb + c0 + c];
    }
  }
  float cur = 0.f;
  int key = kfirst[0];
  TO kb = bfirst[0];
  bool begun = p0 == 0 || a.toks[p0 - 1] != key;  // the run begins in this CTA
  auto flush = [&]() {
    if (!begun) {
      a.head[(int64_t)blockIdx.x * a.ldp + c0 + c] = cur;
      return;
    }
    TO* o = dE + key * a.lde + c0 + c;
    const float s = a.scale * cur;
    *o = Num<TO>::down(a.has_base ? Num<TO>::up(kb) + s : s);
  };
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w >= nw) break;
    if (w > 0 && kfirst[w] != key) {
      flush();
      cur = 0.f;
      key = kfirst[w];
      kb = bfirst[w];
      begun = true;
    }
    cur += hd[w][c];
    if (!whole[w]) {
      flush();
      cur = tl[w][c];
      key = klast[w];
      kb = blast[w];
      begun = true;
    }
  }
  const bool on = p0 + crows < ns && a.toks[p0 + crows] == key;  // it goes on in the next CTA
  if (on && begun)
    a.tail[(int64_t)blockIdx.x * a.ldp + c0 + c] = cur;
  else if (on)
    a.head[(int64_t)blockIdx.x * a.ldp + c0 + c] = cur;
  else
    flush();
}

// Runs that cross CTAs: the CTA of the chunk where one begins adds the tail
// there and the heads of the chunks that follow, four quarters side by side,
// each in order. The other CTAs write the rows of the tokens that do not occur:
// zero, or what is there already.
template <typename TO, bool VEC>
__global__ void __launch_bounds__(256, 8) k_embed_join(SuArgs a, const TO* base, TO* dE) {
  __shared__ __align__(16) float part[4][kEmSpan];
  pdl_wait();
  const int crows = 8 * a.rpw, joins = (int)gridDim.x - a.fills;
  if ((int)blockIdx.x >= joins) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = blockIdx.y * kEmSpan, left = a.D - c0;
    const int v0 = ((int)blockIdx.x - joins) * kSuFill + warp * (kSuFill / 8);
    const unsigned absent =
        __ballot_sync(0xFFFFFFFFu, lane < kSuFill / 8 && v0 + lane < a.V && !a.seen[min(v0 + lane, a.V - 1)]);
#pragma unroll
    for (int q = 0; q < kSuFill / 8; q += 2) {
      __align__(16) TO o[2][8];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        if (a.has_base && (absent >> (q + r) & 1)) {
          load8<TO, VEC>(base + (v0 + q + r) * a.ldb + c0, lane, left, o[r]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[r][i] = Num<TO>::down(0.f);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (absent >> (q + r) & 1) store8<TO, VEC>(dE + (v0 + q + r) * a.lde + c0, lane, left, o[r]);
    }
    return;
  }
  const int ns = *a.total, ch = (int)blockIdx.x, p0 = ch * crows, p1 = p0 + crows;
  if (p1 >= ns) return;
  const int key = a.toks[p1], last = a.toks[p1 - 1], first = a.toks[p0], before = p0 > 0 ? a.toks[p0 - 1] : -1;
  if (last != key) return;                    // no run crosses here
  if (first == key && before == key) return;  // it began earlier
  // last chunk whose first row is still this token's
  int lo = ch + 1, hi = (ns - 1) / crows;
  if (lo < hi && a.toks[(lo + 1) * crows] != key) hi = lo;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.toks[mid * crows] == key)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int c = (threadIdx.x & 63) * 4, g = threadIdx.x >> 6, col = blockIdx.y * kEmSpan + c;
  const int m = lo - ch, per = (m + 3) / 4, i0 = ch + 1 + min(m, g * per), i1 = ch + 1 + min(m, (g + 1) * per);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < a.D) {
    const float* p = a.head + (int64_t)i0 * a.ldp + col;
#pragma unroll 4
    for (int i = i0; i < i1; ++i, p += a.ldp) {
      const float4 x = *reinterpret_cast<const float4*>(p);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
  }
  *reinterpret_cast<float4*>(&part[g][c]) = s;
  __syncthreads();
  const int cc = threadIdx.x, cl = blockIdx.y * kEmSpan + cc;
  if (cl >= a.D) return;
  float t = a.tail[(int64_t)ch * a.ldp + cl];
#pragma unroll
  for (int q = 0; q < 4; ++q) t += part[q][cc];
  t *= a.scale;
  dE[key * a.lde + cl] = Num<TO>::down(a.has_base ? Num<TO>::up(base[key * a.ldb + cl]) + t : t);
}

// ---------------------------------------------------------------- few rows
// At most 256 rows: one launch and no sort. A CTA lists the rows whose tokens
// lie in its 32 vocabulary rows, in order; a warp has four of those, sums a
// token's rows eight loads at a time in that order, and writes the others' zeros
// or what is there already.
constexpr int kDiRows = 256, kDiVocab = 32;

template <typename TI, typename TO, bool VEC>
__global__ void __launch_bounds__(256)
    k_embed_few(SuArgs a, const TI* __restrict__ dout, const int32_t* __restrict__ idx, int N, const TO* base, TO* dE,
                int in_place, int* status) {
  __shared__ int ln[kDiRows], lt[kDiRows], wcount[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c0 = blockIdx.y * kEmSpan, left = a.D - c0;
  const int v0 = blockIdx.x * kDiVocab;
  pdl_wait();
  const int t = (int)threadIdx.x < N ? idx[threadIdx.x] : -1;
  if (blockIdx.x == 0 && blockIdx.y == 0 && (t < -1 || t >= a.V)) raise_status(status, DSPARK_ERANGE);
  const bool in = t >= v0 && t < min(v0 + kDiVocab, a.V);
  const unsigned has = __ballot_sync(0xFFFFFFFFu, in);
  if (lane == 0) wcount[warp] = __popc(has);
  __syncthreads();
  int at = __popc(has & ((1u << lane) - 1u)), m = 0;
  for (int w = 0; w < 8; ++w) {
    if (w < warp) at += wcount[w];
    m += wcount[w];
  }
  if (in) {
    ln[at] = threadIdx.x;
    lt[at] = t;
  }
  __syncthreads();
#pragma unroll 1
  for (int r = 0; r < kDiVocab / 8; ++r) {
    const int v = v0 + warp * (kDiVocab / 8) + r;
    if (v >= a.V) break;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    bool any = false;
    for (int i0 = 0; i0 < m; i0 += 32) {
      unsigned rows = __ballot_sync(0xFFFFFFFFu, i0 + lane < m && lt[min(i0 + lane, kDiRows - 1)] == v);
      any |= rows != 0;
      while (rows) {
        __align__(16) TI x[8][8];
        int k = 0;
#pragma unroll
        for (int f = 0; f < 8; ++f) {
          if (rows) {
            const int n = ln[i0 + __ffs(rows) - 1];
            rows &= rows - 1;
            load8<TI, VEC>(dout + n * a.ldd + c0, lane, left, x[f]);
            k = f + 1;
          }
        }
#pragma unroll
        for (int f = 0; f < 8; ++f)
          if (f < k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] += Num<TI>::up(x[f][i]);
          }
      }
    }
    if (!any && in_place) continue;
    __align__(16) TO o[8];
    if (a.has_base) {
      load8<TO, VEC>(base + v * a.ldb + c0, lane, left, o);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = Num<TO>::down(0.f);
    }
    if (any)
      su_finish<TO, VEC>(a, o, dE, v, c0, lane, left, acc);
    else
      store8<TO, VEC>(dE + v * a.lde + c0, lane, left, o);
  }
}

// ---------------------------------------------------------------- host
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct EmScratch {
  size_t rows, toks, bufa, bufb, cta, total, seen, head, tail, all;
  int chunks, rpw;
};
EmScratch em_scratch(int N, int V, int D) {
  EmScratch s;
  size_t off = 0;
  auto carve = [&](size_t bytes) {
    const size_t o = off;
    off += up256(bytes > 0 ? bytes : 1);
    return o;
  };
  // Rows of a warp: whole waves of four CTAs per SM (152 SMs), each warp at most
  // 32 rows; where there is less than a wave, at least 8 (8190 x 1001 took 45 us
  // with 32, when one CTA's rows follow one another).
  const int64_t spans = (D + kEmSpan - 1) / kEmSpan, slots = 152 * 4, work = (int64_t)N * spans;
  const int64_t waves = (work + 8 * kSuWarp * slots - 1) / (8 * kSuWarp * slots);
  const int64_t rpw = (work + 8 * slots * (waves > 0 ? waves : 1) - 1) / (8 * slots * (waves > 0 ? waves : 1));
  s.rpw = (int)(rpw < 8 ? 8 : rpw > kSuWarp ? kSuWarp : rpw);
  s.chunks = (N + 8 * s.rpw - 1) / (8 * s.rpw);
  s.rows = carve(4 * (size_t)N);
  s.toks = carve(4 * (size_t)N);
  s.bufa = carve(8 * (size_t)N);
  s.bufb = carve(8 * (size_t)N);
  s.cta = carve(sizeof(int) * (size_t)kSoCtas * kSoBins);
  s.total = carve(4);
  s.seen = carve((size_t)V);
  const size_t ldp = ((size_t)D + 3) / 4 * 4;
  s.head = carve(4 * (size_t)s.chunks * ldp);
  s.tail = carve(4 * (size_t)s.chunks * ldp);
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
  static std::atomic<uint64_t> done{0};
  const cudaError_t c = once_per_device(done, [] {
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(k_sort_place<2>, attr, (int)kSoSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_sort_place<4>, attr, (int)kSoSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_sort_cluster<1>, attr, (int)kSoSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_sort_cluster<4>, attr, (int)kSoSmem);
    return e;
  });
  if (c != cudaSuccess) return c;
  int width = 1;
  while (width < 24 && (1 << width) < V) ++width;
  const int passes = (width + kSoBits - 1) / kSoBits, bits = (width + passes - 1) / passes;
  int2* buf[2] = {reinterpret_cast<int2*>(base + s.bufa), reinterpret_cast<int2*>(base + s.bufb)};
  SoPass q = {};
  q.idx = idx;
  q.pairs = nullptr;
  q.N = N;
  q.V = V;
  q.bins = 1 << bits;
  q.shift = 0;
  q.cta = reinterpret_cast<int*>(base + s.cta);
  q.rows = reinterpret_cast<int32_t*>(base + s.rows);
  q.toks = reinterpret_cast<int32_t*>(base + s.toks);
  q.total = reinterpret_cast<int*>(base + s.total);
  q.seen = reinterpret_cast<unsigned char*>(base + s.seen);
  q.status = status;
  q.out = nullptr;
  const size_t smem = sizeof(int) * (size_t)kSoWarps * q.bins;
  if (N <= kScCtas * 4 * kSoThreads) {
    const ScArgs a{q, passes, bits, {buf[0], buf[1]}};
    return launch_ex(N <= kScCtas * kSoThreads ? k_sort_cluster<1> : k_sort_cluster<4>, dim3(kScCtas),
                     dim3(kSoThreads), smem, st, true, a);
  }
  // two pairs a thread while 128 CTAs hold them all at once, else four (99306 rows of
  // 19 fp32 into 63744: 60 us with four, 55 with two; 2 M rows of 16 bf16 360 and 372)
  const bool few = N <= kSoCtas * 2 * kSoThreads;
  const int tile = few ? 2 * kSoThreads : 4 * kSoThreads;
  q.per = ((N + kSoCtas - 1) / kSoCtas + tile - 1) / tile * tile;
  const int ctas = (N + q.per - 1) / q.per;
  cudaError_t e = cudaSuccess;
  for (int k = 0; k < passes && e == cudaSuccess; ++k) {
    q.shift = k * bits;
    q.out = k + 1 < passes ? buf[k & 1] : nullptr;
    e = launch_ex(few ? k_sort_count<2> : k_sort_count<4>, dim3(ctas), dim3(kSoThreads),
                  sizeof(int) * (size_t)q.bins, st, true, q);
    if (e == cudaSuccess)
      e = launch_ex(few ? k_sort_place<2> : k_sort_place<4>, dim3(ctas), dim3(kSoThreads), smem, st, true, q);
    q.idx = nullptr;
    q.pairs = q.out;
  }
  return e;
}

template <typename TI, typename TO, bool VEC>
cudaError_t em_sum(const SuArgs& a, const void* dout, const int32_t* idx, int N, const void* base, void* dE,
                   int* status, cudaStream_t st) {
  if (N <= kDiRows)
    return launch_ex(k_embed_few<TI, TO, VEC>, dim3((a.V + kDiVocab - 1) / kDiVocab, (a.D + kEmSpan - 1) / kEmSpan),
                     dim3(256), 0, st, true, a, static_cast<const TI*>(dout), idx, N, static_cast<const TO*>(base),
                     static_cast<TO*>(dE), base == dE ? 1 : 0, status);
  static std::atomic<uint64_t> done{0};
  const cudaError_t c = once_per_device(done, [] {
    return cudaFuncSetAttribute(k_embed_sum<TI, TO, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)su_smem<TI>());
  });
  if (c != cudaSuccess) return c;
  const int spans = (a.D + kEmSpan - 1) / kEmSpan;
  const TO* b = static_cast<const TO*>(base);
  TO* o = static_cast<TO*>(dE);
  cudaError_t e = cudaSuccess;
  if (a.chunks > 0)
    e = launch_ex(k_embed_sum<TI, TO, VEC>, dim3(a.chunks, spans), dim3(256), su_smem<TI>(), st, true, a,
                  static_cast<const TI*>(dout), b, o);
  const int last = a.fills + (a.chunks > 1 ? a.chunks - 1 : 0);
  if (e == cudaSuccess && last > 0)
    e = launch_ex(k_embed_join<TO, VEC>, dim3(last, spans), dim3(256), 0, st, true, a, b, o);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename TI, typename TO>
cudaError_t em_sum_v(bool vec, const SuArgs& a, const void* dout, const int32_t* idx, int N, const void* base,
                     void* dE, int* status, cudaStream_t st) {
  return vec ? em_sum<TI, TO, true>(a, dout, idx, N, base, dE, status, st)
             : em_sum<TI, TO, false>(a, dout, idx, N, base, dE, status, st);
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
  return em_fail(type == DSPARK_BF16
                     ? em_lookup<__nv_bfloat16>(vec, E, lde, V, D, idx, N, scale, out, ldo, device_status, st)
                     : em_lookup<float>(vec, E, lde, V, D, idx, N, scale, out, ldo, device_status, st));
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
  if (N > kDiRows) {
    const cudaError_t e = em_sort(idx, N, V, b, s, device_status, st);
    if (e != cudaSuccess) return em_fail(e);
  }
  SuArgs a;
  a.rows = reinterpret_cast<const int32_t*>(b + s.rows);
  a.toks = reinterpret_cast<const int32_t*>(b + s.toks);
  a.total = reinterpret_cast<const int*>(b + s.total);
  a.seen = reinterpret_cast<unsigned char*>(b + s.seen);
  a.rpw = s.rpw;
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
  a.fills = base != dE ? (V + kSuFill - 1) / kSuFill : 0;  // added in place: the other rows stay as they are
  a.ldp = ((int64_t)D + 3) / 4 * 4;
  const bool vec = em_vec(dout, ldd, type) && em_vec(dE, lde, grad_type) && (!base || em_vec(base, ldb, grad_type));
  typedef __nv_bfloat16 bf;
  if (type == DSPARK_BF16)
    return em_fail(grad_type == DSPARK_BF16 ? em_sum_v<bf, bf>(vec, a, dout, idx, N, base, dE, device_status, st)
                                            : em_sum_v<bf, float>(vec, a, dout, idx, N, base, dE, device_status, st));
  return em_fail(grad_type == DSPARK_BF16 ? em_sum_v<float, bf>(vec, a, dout, idx, N, base, dE, device_status, st)
                                          : em_sum_v<float, float>(vec, a, dout, idx, N, base, dE, device_status, st));
}
