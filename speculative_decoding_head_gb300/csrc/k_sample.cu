// k_sample.cu -- drawing a token from a row of logits after temperature, top-k,
// top-p and min-p, and the distribution that they make as log-probabilities.
//
// A cluster of CTAs takes a row: each holds its part in shared memory, so that
// the logits are read from memory once and every later pass runs on chip
// (vocabularies that sixteen CTAs cannot hold are read again each pass). With
// m the row's maximum, a token's mass is the whole number
//   W = round(2^Q 2^((z - m) log2(e) / T)),   Q = min(46, 62 - ceil(log2 V)),
// taken to a relative 2^-31 (see weight()), so that masses are added in any order
// with one result, and a border of the top-p set or of the draw is missed by 1e-10
// of the mass at the most: next to nothing against one token's share.
//
// top-k and top-p are one search, for the last token of a prefix of the row sorted by
// falling z (then by index): the first whose running sum, of ones or of masses,
// reaches a target. A histogram of 2048 bins of m - z gives the bin that holds
// it; the bin's tokens (some hundreds of a flat row of 129280) are brought to one CTA, sorted and
// added up. A bin of more than 2048 tokens (many equal logits) is instead narrowed by three
// histograms of the bits of z, down to one value, whose tokens are counted by index.
// What is kept is z > cut, or z == cut and index <= last: the stricter of the three settings' pairs.
#include <math.h>
#include <stdio.h>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

typedef unsigned long long u64;

constexpr int kSpThreads = 512, kSpWarps = kSpThreads / 32;
constexpr int kSpMaxC = 16;     // CTAs of a cluster
constexpr int kSpBins = 2048;
constexpr int kSpList = 2048;   // tokens of a bin that are sorted
constexpr int kSpChunk = 512;   // tokens that a warp takes at a time
constexpr int kSpMaxChunks = 2048;
constexpr float kSpMasked = -1e29f;
constexpr int kSpHist = kSpBins * 8;  // bytes: the histogram, the list or the chunks' sums

struct SpArgs {
  const void* Z;
  int64_t ldz;
  int N, V, requests;
  const int32_t* row_off;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* token;
  float* logp;
  float* out;
  int64_t ldo;
  float fill;
  int part;      // tokens of a CTA, a multiple of kSpChunk
  int q;         // Q
  int vec, vec_out;
  int* status;
};

// Of the row, in every CTA of its cluster.
struct SpRow {
  float m, c_hi, c_lo;  // maximum; log2(e) / T as a sum of two
  float inv_t;
  int q;
};

struct SpCut {
  float z;
  int last;  // of the tokens with this z, those up to this index are kept
};

struct SpShared {
  uint2 exp2[64];              // 2^(i/64): times 2^31 as a whole number and as fp32
  u64 slot[2][kSpMaxC][2];     // what each CTA tells the others
  u64 res[2];                  // a search's answer: bin and sum before it, or a cut
  u64 warp[kSpWarps], warp2[kSpWarps];
  u64 bcast[2];
  float c_hi, c_lo, inv_t, min_z, p, u;
  int k, n, bad;
};

// round(2^31 2^(i/64))
__constant__ uint32_t kSpExp2[64] = {
    2147483648u, 2170868212u, 2194507417u, 2218404036u, 2242560872u, 2266980759u, 2291666561u, 2316621173u,
    2341847524u, 2367348571u, 2393127307u, 2419186755u, 2445529972u, 2472160047u, 2499080105u, 2526293303u,
    2553802834u, 2581611923u, 2609723834u, 2638141863u, 2666869345u, 2695909648u, 2725266179u, 2754942382u,
    2784941738u, 2815267765u, 2845924021u, 2876914102u, 2908241642u, 2939910317u, 2971923842u, 3004285971u,
    3037000500u, 3070071267u, 3103502151u, 3137297074u, 3171459999u, 3205994934u, 3240905930u, 3276197082u,
    3311872529u, 3347936457u, 3384393094u, 3421246719u, 3458501653u, 3496162267u, 3534232978u, 3572718252u,
    3611622603u, 3650950594u, 3690706840u, 3730896002u, 3771522796u, 3812591987u, 3854108391u, 3896076880u,
    3938502376u, 3981389855u, 4024744348u, 4068570940u, 4112874773u, 4157661043u, 4202935003u, 4248701965u};

__device__ __forceinline__ uint32_t ordered(float z) {
  const uint32_t b = __float_as_uint(z);
  return b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o ^ ((int32_t)o < 0 ? 0x80000000u : 0xFFFFFFFFu));
}

// The mass of a token. The exponent y = (z - m) log2(e) / T is carried as a sum
// of two fp32 (z - m with its rounding error, by Knuth's two-sum; the product with its error by
// an fma), split into n + i/64 + r, |r| <= 1/128, and
//   2^y = 2^n 2^(i/64) (1 + r l + (r l)^2 / 2 + (r l)^3 / 6),  l = ln 2,
// Taylor's next term being 2^-35 of it. The bracket less one is fp32, at most
// 2^-7.5, so its rounding is 2^-31 of the mass; 2^(i/64) is held in 32 bits.
__device__ __forceinline__ u64 weight(float z, const SpRow& r, const uint2* tab) {
  const float s = z - r.m;
  const float y = s * r.c_hi;
  if (!(y > -(float)(r.q + 1))) return 0;
  const float a = s + r.m, b = s - a;
  const float e = (z - a) + (-r.m - b);
  const float lo = fmaf(s, r.c_hi, -y) + fmaf(s, r.c_lo, e * r.c_hi);
  const float magic = 196608.f;  // 1.5 * 2^17: a step of 1/64
  const float t = y + magic;
  const int yi = __float_as_int(t) - __float_as_int(magic);
  const float f = (y - (t - magic)) + lo;
  const uint2 w = tab[yi & 63];
  const float p = f * fmaf(f, fmaf(f, 0.05550411f, 0.24022651f), 0.69314718f);
  const uint32_t mant = w.x + (uint32_t)__float2int_rn(__uint_as_float(w.y) * p);
  const int sh = -(yi >> 6) - (r.q - 31);  // mant 2^31 stands for 1
  if (sh <= 0) return (u64)mant << -sh;
  if (sh > 32) return 0;
  return ((u64)mant + (1ull << (sh - 1))) >> sh;
}

__device__ __forceinline__ void st_rank(void* p, uint32_t rank, u64 x) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tc::map_rank(tc::smem_u32(p), rank)), "l"(x) : "memory");
}
__device__ __forceinline__ int add_rank(int* p, uint32_t rank, int x) {
  int old;
  asm volatile("atom.shared::cluster.add.s32 %0, [%1], %2;"
               : "=r"(old)
               : "r"(tc::map_rank(tc::smem_u32(p), rank)), "r"(x)
               : "memory");
  return old;
}

__device__ __forceinline__ u64 warp_sum64(u64 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}
__device__ __forceinline__ u64 warp_scan64(u64 x) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// floor(x a) and ceil(x a) for 0 <= a < 1
__device__ __forceinline__ u64 mul_floor(u64 x, float a, bool ceil) {
  const uint32_t b = __float_as_uint(a), e = b >> 23;
  const uint32_t mant = e ? (b & 0x7FFFFFu) | 0x800000u : b;
  const int sh = 150 - (int)(e ? e : 1);  // a = mant 2^-sh
  const unsigned __int128 v = (unsigned __int128)x * mant;
  if (sh >= 127) return ceil && v != 0;
  const unsigned __int128 q = v >> sh;
  return (u64)q + (ceil && (q << sh) != v ? 1 : 0);
}

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
// masked tokens are -inf, -0 is 0
__device__ __forceinline__ float clean(float z) { return z <= kSpMasked ? -INFINITY : z + 0.f; }

// One row's work in one CTA. RES: its part lies in shared memory.
template <typename T, bool RES>
struct Row {
  static constexpr int kPer = 16 / (int)sizeof(T);  // values of 16 bytes
  const SpArgs& a;
  SpShared& sh;
  uint8_t* buf;        // kSpHist bytes
  T* part;             // RES: the row's part
  const T* row;        // the whole row, in global memory
  int tid, warp, lane;
  uint32_t rank, C;
  int start, count, chunks;  // the part's first token, its tokens, its chunks
  int par = 0;
  SpRow r;
  SpCut cut{-INFINITY, -1};

  __device__ Row(const SpArgs& a_, SpShared& s_) : a(a_), sh(s_) {}

  // place of value i of a lane in a chunk
  __device__ __forceinline__ int at(int ch, int i) const {
    return ch * kSpChunk + i / kPer * (32 * kPer) + lane * kPer + i % kPer;
  }
  __device__ __forceinline__ void unpack(const uint4& q, float* v) const {
    const T* t = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = up<T>(t[i]);
  }
  // 16 / kPer * kPer = 16 tokens of a lane, from global memory; past the end -inf
  __device__ __forceinline__ void fetch(int ch, float* v) const {
#pragma unroll
    for (int g = 0; g < 16 / kPer; ++g) {
      const int l = at(ch, g * kPer);
      if (a.vec && l + kPer <= count) {
        unpack(__ldg(reinterpret_cast<const uint4*>(row + start + l)), v + g * kPer);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) v[g * kPer + i] = l + i < count ? up<T>(row[start + l + i]) : -INFINITY;
      }
    }
  }
  __device__ __forceinline__ void values(int ch, float* v) const {
    if (RES) {
#pragma unroll
      for (int g = 0; g < 16 / kPer; ++g) unpack(*reinterpret_cast<const uint4*>(part + at(ch, g * kPer)), v + g * kPer);
    } else {
      fetch(ch, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = clean(v[i]);
    }
  }
  __device__ __forceinline__ float value(int l) const {
    if (RES) return up<T>(part[l]);
    return l < count ? clean(up<T>(row[start + l])) : -INFINITY;
  }
  __device__ __forceinline__ bool kept(float z, int l) const {
    return z > cut.z || (z == cut.z && start + l <= cut.last);
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int ch = warp; ch < chunks; ch += kSpWarps) {
      float v[16];
      values(ch, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) f(v[i], at(ch, i));
    }
  }
  // Every CTA's thread 0 tells x, y to all; all see them in slot[][].
  __device__ __forceinline__ const u64 (*tell(u64 x, u64 y))[2] {
    if (tid == 0) {
      sh.bcast[0] = x;
      sh.bcast[1] = y;
    }
    __syncthreads();
    if (tid < (int)C) {
      st_rank(&sh.slot[par][rank][0], tid, sh.bcast[0]);
      st_rank(&sh.slot[par][rank][1], tid, sh.bcast[1]);
    }
    tc::cluster_sync();
    const u64(*s)[2] = sh.slot[par];
    par ^= 1;
    return s;
  }
  __device__ __forceinline__ u64 block_sum(u64 x) {  // in every thread
    x = warp_sum64(x);
    __syncthreads();
    if (lane == 0) sh.warp[warp] = x;
    __syncthreads();
    u64 t = 0;
#pragma unroll
    for (int i = 0; i < kSpWarps; ++i) t += sh.warp[i];
    return t;
  }
  // sum of the threads before this one; every thread takes part
  __device__ __forceinline__ u64 block_before(u64 x) {
    const u64 inc = warp_scan64(x);
    __syncthreads();
    if (lane == 31) sh.warp2[warp] = inc;
    __syncthreads();
    u64 t = inc - x;
    for (int i = 0; i < warp; ++i) t += sh.warp2[i];
    return t;
  }

  __device__ __forceinline__ uint32_t* lo() const { return reinterpret_cast<uint32_t*>(buf); }
  __device__ __forceinline__ uint32_t* hi() const { return reinterpret_cast<uint32_t*>(buf) + kSpBins; }
  __device__ __forceinline__ void clear() {
    for (int i = tid; i < kSpBins * 2; i += kSpThreads) lo()[i] = 0;
    __syncthreads();
  }
  template <bool MASS>
  __device__ __forceinline__ void add(int bin, float z) {
    if (!MASS) {
      atomicAdd(lo() + bin, 1u);
    } else {
      const u64 w = weight(z, r, sh.exp2);
      const uint32_t l = (uint32_t)w, old = atomicAdd(lo() + bin, l);
      const uint32_t h = (uint32_t)(w >> 32) + (old + l < old ? 1u : 0u);
      if (h) atomicAdd(hi() + bin, h);
    }
  }
  // With every CTA's histogram filled: the first bin at which before + the sum up to it reaches the
  // target, and the sum before it. target 0: ceil(p of all of it), at least 1.
  __device__ __forceinline__ void find(u64& target, u64& before, int& bin) {
    tc::cluster_sync();
    const int seg = kSpBins / (int)C, per = (seg + kSpThreads - 1) / kSpThreads;
    u64 v[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0;
      const int b = tid * per + i;
      if (i < per && b < seg) {
        const int g = (int)rank * seg + b;
        for (uint32_t c = 0; c < C; ++c)
          v[i] += (u64)(uint32_t)tc::ld_rank(tc::smem_u32(lo() + g), c) +
                  ((u64)(uint32_t)tc::ld_rank(tc::smem_u32(hi() + g), c) << 32);
      }
      sum += v[i];
    }
    const u64 mine = block_before(sum);
    const u64 all = block_sum(sum);
    const u64(*s)[2] = tell(all, 0);
    u64 total = 0, pre = before;
    for (uint32_t c = 0; c < C; ++c) {
      if (c == rank) pre += total;
      total += s[c][0];
    }
    if (target == 0) {
      target = mul_floor(total, sh.p, true);
      if (target == 0) target = 1;
    }
    u64 t = pre + mine;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t < target && t + v[i] >= target) {
        for (uint32_t c = 0; c < C; ++c) {
          st_rank(&sh.res[0], c, (u64)(rank * seg + tid * per + i));
          st_rank(&sh.res[1], c, t);
        }
      }
      t += v[i];
    }
    tc::cluster_sync();
    bin = (int)sh.res[0];
    before = sh.res[1];
  }

  // Tightens the cut to the first of the kept tokens, in order, whose running
  // count (MASS: mass) reaches the target.
  template <bool MASS>
  __device__ void select(u64 target, float beta) {
    auto bin_of = [&](float z) { return min(kSpBins - 1, (int)((r.m - z) * beta)); };
    clear();
    if (tid == 0) sh.n = 0;
    each([&](float z, int l) {
      if (kept(z, l)) add<MASS>(bin_of(z), z);
    });
    u64 before = 0;
    int bin;
    find(target, before, bin);
    // the bin's tokens to CTA 0, sorted by falling z, then by index
    u64* list = reinterpret_cast<u64*>(buf);
    each([&](float z, int l) {
      if (kept(z, l) && bin_of(z) == bin) {
        const int n = add_rank(&sh.n, 0, 1);
        if (n < kSpList) st_rank(list + n, 0, (u64)~ordered(z) << 32 | (uint32_t)(start + l));
      }
    });
    tc::cluster_sync();
    const int n = tc::ld_rank(tc::smem_u32(&sh.n), 0);
    if (n <= kSpList) {
      if (rank == 0) cut_of_list<MASS>(n, target, before);
    } else {
      narrow<MASS>(bin_of, bin, target, before);
    }
    tc::cluster_sync();
    cut.z = unordered((uint32_t)(sh.res[0] >> 32));
    cut.last = (int)(uint32_t)sh.res[0];
  }

  template <bool MASS>
  __device__ void cut_of_list(int n, u64 target, u64 before) {
    u64* list = reinterpret_cast<u64*>(buf);
    int size = 32;
    while (size < n) size *= 2;
    for (int i = n + tid; i < size; i += kSpThreads) list[i] = ~0ull;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2) {
      for (int j = k / 2; j > 0; j /= 2) {
        for (int i = tid; i < size / 2; i += kSpThreads) {
          const int x = 2 * i - (i & (j - 1)), y = x + j;
          const u64 p = list[x], q = list[y];
          if ((p > q) == ((x & k) == 0)) {
            list[x] = q;
            list[y] = p;
          }
        }
        __syncthreads();
      }
    }
    u64 w[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = tid * 4 + i;
      w[i] = e >= n ? 0 : !MASS ? 1 : weight(unordered(~(uint32_t)(list[e] >> 32)), r, sh.exp2);
      sum += w[i];
    }
    u64 t = before + block_before(sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (t < target && t + w[i] >= target) {
        const u64 e = list[tid * 4 + i];
        for (uint32_t c = 0; c < C; ++c) st_rank(&sh.res[0], c, (u64)~(uint32_t)(e >> 32) << 32 | (uint32_t)e);
      }
      t += w[i];
    }
  }

  // The same by the bits of z: 11, 11 and 10 of them, then by index among equals.
  template <bool MASS, typename B>
  __device__ void narrow(B bin_of, int bin, u64 target, u64 before) {
    uint32_t prefix = 0;
    for (int level = 0; level < 3; ++level) {
      const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
      tc::cluster_sync();
      clear();
      each([&](float z, int l) {
        if (!kept(z, l) || bin_of(z) != bin) return;
        const uint32_t key = ~ordered(z);
        if (level > 0 && (key >> (shift + bits)) != prefix) return;
        add<MASS>((int)(key >> shift) & ((1 << bits) - 1), z);
      });
      int digit;
      find(target, before, digit);
      prefix = prefix << bits | (uint32_t)digit;
    }
    const float zc = unordered(~prefix);
    const u64 w = MASS ? weight(zc, r, sh.exp2) : 1;
    u64 keep = (target - before + w - 1) / w;  // the sum reached the target here, so w > 0
    // how many equals each CTA's chunks hold
    u64* cnt = reinterpret_cast<u64*>(buf);
    u64 mine = 0;
    for (int ch = warp; ch < chunks; ch += kSpWarps) {
      float v[16];
      values(ch, v);
      u64 c = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) c += v[i] == zc && kept(v[i], at(ch, i)) ? 1 : 0;
      c = warp_sum64(c);
      if (lane == 0) cnt[ch] = c;
      mine += c;
    }
    mine = block_sum(lane == 0 ? mine : 0);
    const u64(*s)[2] = tell(mine, 0);
    u64 pre = 0;
    for (uint32_t c = 0; c < rank; ++c) pre += s[c][0];
    if (pre >= keep || pre + mine < keep) return;
    keep -= pre;
    int ch = 0;
    while (keep > cnt[ch]) keep -= cnt[ch++];
    if (warp == 0) {
      for (int g = 0; g < kSpChunk / 32; ++g) {
        const int l = ch * kSpChunk + g * 32 + lane;
        const float z = value(l);
        const uint32_t hit = __ballot_sync(0xFFFFFFFFu, z == zc && kept(z, l));
        const int here = __popc(hit);
        if (keep <= (u64)here) {
          const int last = start + ch * kSpChunk + g * 32 + (int)__fns(hit, 0, (int)keep);
          if (lane < (int)C) st_rank(&sh.res[0], lane, (u64)ordered(zc) << 32 | (uint32_t)last);
          break;
        }
        keep -= here;
      }
    }
  }
};

// DIST: the whole distribution is written; otherwise a token is drawn.
template <typename T, bool RES, bool DIST>
__global__ void __launch_bounds__(kSpThreads, 2) k_sample(SpArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ SpShared sh;
  Row<T, RES> w(a, sh);
  w.tid = threadIdx.x;
  w.warp = w.tid >> 5;
  w.lane = w.tid & 31;
  w.rank = tc::cluster_ctarank();
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(w.C));
  const int tid = w.tid;
  const int n = (int)(blockIdx.x / w.C);
  w.buf = smem;
  w.part = reinterpret_cast<T*>(smem + kSpHist);
  w.row = static_cast<const T*>(a.Z) + (int64_t)n * a.ldz;
  w.start = (int)min((int64_t)w.rank * a.part, (int64_t)a.V);
  w.count = min(a.part, a.V - w.start);
  w.chunks = (w.count + kSpChunk - 1) / kSpChunk;
  w.r.q = a.q;
  if (tid < 64) sh.exp2[tid] = make_uint2(kSpExp2[tid], __float_as_uint((float)kSpExp2[tid]));
  pdl_wait();
  pdl_trigger();

  // the row's settings
  int b = n;
  if (a.row_off) {
    // the last request that begins at or before the row; the cluster's CTAs decide alike
    if (__ldg(a.row_off) > n) return;
    b = 0;
    for (int i = 0; i < a.requests; i += kSpThreads)
      b += __syncthreads_count(i + tid < a.requests && __ldg(a.row_off + i + tid + 1) <= n);
    if (b >= a.requests) return;
  }
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");  // this CTA has begun: the others may write to it
  if (tid == kSpThreads - 1) {
    float t = a.temperature ? __ldg(a.temperature + b) : 1.f;
    const float p = a.top_p ? __ldg(a.top_p + b) : 1.f, mp = a.min_p ? __ldg(a.min_p + b) : 0.f;
    const float u = DIST ? 0.f : __ldg(a.u + n);
    int k = a.top_k ? __ldg(a.top_k + b) : 0;
    sh.bad = !(t >= 0.f && t < INFINITY && p >= 0.f && p <= 1.f && mp >= 0.f && mp <= 1.f && u >= 0.f && u < 1.f);
    if (t == 0.f) {
      t = 1.f;
      k = 1;
    }
    t = fmaxf(t, 1e-30f);
    // log2(e) / T, its rounding error with it
    const float l_hi = 1.44269502f, l_lo = 1.92596303e-08f;
    sh.c_hi = l_hi / t;
    sh.c_lo = (fmaf(-sh.c_hi, t, l_hi) + l_lo) / t;
    sh.inv_t = 1.f / t;
    sh.bcast[0] = __double_as_longlong(mp > 0.f ? (double)t * log((double)mp) : -INFINITY);
    sh.p = p;
    sh.u = u;
    sh.k = k;
  }

  // the row's part: to shared memory, its maximum and the sum of its logits on the way
  float top = -INFINITY, sum = 0.f;
  u64 seen = 0;  // tokens not masked; above them, whether there is a NaN or +inf
  for (int ch = w.warp; ch < w.chunks; ch += kSpWarps) {
    float v[16];
    w.fetch(ch, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (!(v[i] < INFINITY)) seen |= 1ull << 40;
      v[i] = clean(v[i]);
      top = fmaxf(top, v[i]);
      if (v[i] > -INFINITY) {
        sum += fmaxf(v[i], -1e4f);
        ++seen;
      }
    }
    if (RES) {
#pragma unroll
      for (int g = 0; g < 16 / Row<T, RES>::kPer; ++g) {
        T t[Row<T, RES>::kPer];
#pragma unroll
        for (int i = 0; i < Row<T, RES>::kPer; ++i) t[i] = T(v[g * Row<T, RES>::kPer + i]);
        *reinterpret_cast<uint4*>(w.part + w.at(ch, g * Row<T, RES>::kPer)) = *reinterpret_cast<const uint4*>(t);
      }
    }
  }
  top = warp_max(top);
  sum = warp_sum(sum);
  const u64 bad_here = (u64)__any_sync(0xFFFFFFFFu, seen >> 40 != 0) << 40;
  seen = (warp_sum64(seen & 0xFFFFFFFFFFull) & 0xFFFFFFFFFFull) | bad_here;
  if (w.lane == 0) {
    sh.warp[w.warp] = (u64)ordered(top) << 32 | __float_as_uint(sum);
    sh.warp2[w.warp] = seen;
  }
  __syncthreads();
  const double t_log = __longlong_as_double((long long)sh.bcast[0]);
  if (tid == 0) {
    uint32_t o = 0;
    u64 c = 0;
    float s = 0.f;
    for (int i = 0; i < kSpWarps; ++i) {
      o = max(o, (uint32_t)(sh.warp[i] >> 32));
      s += __uint_as_float((uint32_t)sh.warp[i]);
      c = ((c | sh.warp2[i]) & (1ull << 40)) | ((c & 0xFFFFFFFFFFull) + (sh.warp2[i] & 0xFFFFFFFFFFull));
    }
    sh.warp[0] = (u64)o << 32 | __float_as_uint(s);
    sh.warp2[0] = c;
  }
  __syncthreads();
  uint32_t o = 0;
  u64 live = 0;
  float all = 0.f;
  bool bad = sh.bad;
  asm volatile("barrier.cluster.wait;" ::: "memory");
  {
    const u64(*s)[2] = w.tell(sh.warp[0], sh.warp2[0]);
    for (uint32_t c = 0; c < w.C; ++c) {
      o = max(o, (uint32_t)(s[c][0] >> 32));
      all += __uint_as_float((uint32_t)s[c][0]);
      live += s[c][1] & 0xFFFFFFFFFFull;
      bad |= s[c][1] >> 40 != 0;
    }
  }
  const bool none = bad || live == 0;
  if (none) {
    if (bad && w.rank == 0 && tid == 0) raise_status(a.status, DSPARK_ENUMERIC);
    if (DIST) {
      float* out = a.out + (int64_t)n * a.ldo + w.start;
      for (int i = tid; i < w.count; i += kSpThreads) out[i] = a.fill;
    } else if (w.rank == 0 && tid == 0) {
      a.token[n] = -1;
      if (a.logp) a.logp[n] = bad ? NAN : -INFINITY;
    }
    tc::cluster_sync();  // no CTA ends while another may still write to it
    return;
  }
  w.r.m = unordered(o);
  w.r.c_hi = sh.c_hi;
  w.r.c_lo = sh.c_lo;
  w.r.inv_t = sh.inv_t;

  // top-k: bins up to four times the mean distance from the maximum (half of the tokens lie within two)
  if (sh.k > 0 && (u64)sh.k < live) {
    const float mean = w.r.m - all / (float)live;
    w.template select<false>((u64)sh.k, mean > 0.f ? kSpBins / (4.f * mean) : 0.f);
  }
  // top-p: bins of 1/64 bit of mass
  if (sh.p < 1.f) w.template select<true>(0, kSpBins / 32 * w.r.c_hi);
  if (t_log > -INFINITY) {
    const double t = (double)w.r.m + t_log;
    float z = __double2float_ru(t);
    if (z > w.cut.z) w.cut = SpCut{z, a.V};
  }

  // the kept mass
  u64 S = 0, before = 0;
  if (DIST) {
    u64 t = 0;
    w.each([&](float z, int l) {
      if (w.kept(z, l)) t += weight(z, w.r, sh.exp2);
    });
    const u64 mine = w.block_sum(t);
    const u64(*s)[2] = w.tell(mine, 0);
    for (uint32_t c = 0; c < w.C; ++c) S += s[c][0];
    const float ls = logf((float)S * exp2f(-(float)a.q));
    float* out = a.out + (int64_t)n * a.ldo + w.start;
    for (int ch = w.warp; ch < w.chunks; ch += kSpWarps) {
      float v[16];
      w.values(ch, v);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = w.kept(v[i], w.at(ch, i)) ? fmaf(v[i] - w.r.m, w.r.inv_t, -ls) : a.fill;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int l = w.at(ch, g * 4);
        if (a.vec_out && l + 4 <= w.count) {
          __stcs(reinterpret_cast<float4*>(out + l), make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (l + i < w.count) out[l + i] = v[4 * g + i];
        }
      }
    }
  } else {
    u64* chunk = reinterpret_cast<u64*>(w.buf);
    for (int ch = w.warp; ch < w.chunks; ch += kSpWarps) {
      float v[16];
      w.values(ch, v);
      u64 t = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (w.kept(v[i], w.at(ch, i))) t += weight(v[i], w.r, sh.exp2);
      t = warp_sum64(t);
      if (w.lane == 0) chunk[ch] = t;
    }
    __syncthreads();
    constexpr int kEach = kSpMaxChunks / kSpThreads;
    u64 t = 0;
    for (int i = 0; i < kEach; ++i) t += tid * kEach + i < w.chunks ? chunk[tid * kEach + i] : 0;
    const u64 mine_before = w.block_before(t);
    const u64 mine = w.block_sum(t);
    const u64(*s)[2] = w.tell(mine, 0);
    for (uint32_t c = 0; c < w.C; ++c) {
      if (c == w.rank) before = S;
      S += s[c][0];
    }
    const u64 target = mul_floor(S, sh.u, false);
    if (target >= before && target < before + mine) {
      u64 x = before + mine_before;
      for (int i = 0; i < kEach; ++i) {
        const int ch = tid * kEach + i;
        const u64 here = ch < w.chunks ? chunk[ch] : 0;
        if (target >= x && target < x + here) {
          sh.bcast[0] = (u64)ch;
          sh.bcast[1] = target - x;
        }
        x += here;
      }
      __syncthreads();
      const int ch = (int)sh.bcast[0];
      const u64 rest = sh.bcast[1];
      // 32 tokens of the chunk a warp
      const int l = ch * kSpChunk + w.warp * 32 + w.lane;
      const float z = w.value(l);
      const u64 own = w.kept(z, l) ? weight(z, w.r, sh.exp2) : 0;
      const u64 inc = warp_scan64(own);
      __syncthreads();
      if (w.lane == 31) sh.warp[w.warp] = inc;
      __syncthreads();
      u64 y = inc - own;
      for (int i = 0; i < w.warp; ++i) y += sh.warp[i];
      if (rest >= y && rest < y + own) {
        a.token[n] = w.start + l;
        if (a.logp)
          a.logp[n] = (float)((double)(z - w.r.m) * (double)w.r.inv_t - (double)logf((float)S * exp2f(-(float)a.q)));
      }
    }
  }
  tc::cluster_sync();  // no CTA ends while another may still write to it
}

bool type_ok(int t) { return t == DSPARK_F32 || t == DSPARK_BF16; }
bool on(const void* p, int size) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(size - 1)) == 0; }

template <typename T, bool RES, bool DIST>
cudaError_t launch(const SpArgs& a, int C, size_t smem, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = once_per_device(done, [] {
    cudaError_t x = cudaFuncSetAttribute(k_sample<T, RES, DIST>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (x == cudaSuccess)
      x = cudaFuncSetAttribute(k_sample<T, RES, DIST>, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
    return x;
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((int64_t)a.N * C));
  cfg.blockDim = dim3(kSpThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_sample<T, RES, DIST>, a);
}

template <bool DIST>
dspark_status sample(const dspark_sample_args* s, const void* Z, SpArgs a, int32_t* device_status,
                     dspark_stream_t stream) {
  if (!s || s->N < 0 || s->N > (1 << 24) || s->V < 1 || s->V > (1 << 24) || !type_ok(s->type) || s->ldz < s->V ||
      !device_status || (s->row_off && s->requests < 1))
    return DSPARK_EINVAL;
  if (!on(s->row_off, 4) || !on(s->temperature, 4) || !on(s->top_k, 4) || !on(s->top_p, 4) || !on(s->min_p, 4))
    return DSPARK_EINVAL;
  if (s->N == 0) return DSPARK_OK;
  const int size = s->type == DSPARK_BF16 ? 2 : 4;
  if (!Z || !on(Z, size)) return DSPARK_EINVAL;
  if (DIST ? (!a.out || !on(a.out, 4) || a.ldo < s->V) : (!a.u || !a.token || !on(a.u, 4) || !on(a.token, 4) || !on(a.logp, 4)))
    return DSPARK_EINVAL;
  a.Z = Z;
  a.ldz = s->ldz;
  a.N = s->N;
  a.V = s->V;
  a.requests = s->requests;
  a.row_off = s->row_off;
  a.temperature = s->temperature;
  a.top_k = s->top_k;
  a.top_p = s->top_p;
  a.min_p = s->min_p;
  a.status = device_status;
  a.vec = on(Z, 16) && s->ldz * size % 16 == 0;
  a.vec_out = DIST && on(a.out, 16) && a.ldo % 4 == 0;
  int bits = 0;
  while ((1 << bits) < a.V) ++bits;
  a.q = 62 - bits < 46 ? 62 - bits : 46;
  // The smallest cluster whose parts leave room for two CTAs on an SM, and more CTAs where the rows do
  // not fill the SMs, down to 2048 tokens a CTA.
  auto part = [&](int C) { return ((a.V + C - 1) / C + kSpChunk - 1) / kSpChunk * kSpChunk; };
  int C = 1;
  while (C < kSpMaxC && (size_t)part(C) * size > 92 * 1024) C *= 2;
  while (C < kSpMaxC && (int64_t)a.N * C < 152 && part(C) > 2048) C *= 2;
  a.part = part(C);
  const bool res = (size_t)a.part * size <= 180 * 1024;
  const size_t smem = kSpHist + (res ? (size_t)a.part * size : 0);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  typedef __nv_bfloat16 bf;
  cudaError_t e;
  if (s->type == DSPARK_BF16)
    e = res ? launch<bf, true, DIST>(a, C, smem, st) : launch<bf, false, DIST>(a, C, smem, st);
  else
    e = res ? launch<float, true, DIST>(a, C, smem, st) : launch<float, false, DIST>(a, C, smem, st);
  if (e != cudaSuccess) fprintf(stderr, "dspark: CUDA error %s\n", cudaGetErrorString(e));
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_sample(const dspark_sample_args* args, const void* Z, const float* u, int32_t* token,
                                       float* logp, int32_t* device_status, dspark_stream_t stream) {
  SpArgs a = {};
  a.u = u;
  a.token = token;
  a.logp = logp;
  return sample<false>(args, Z, a, device_status, stream);
}

extern "C" dspark_status dspark_sample_logprobs(const dspark_sample_args* args, const void* Z, float fill, float* out,
                                                int64_t ldo, int32_t* device_status, dspark_stream_t stream) {
  SpArgs a = {};
  a.out = out;
  a.ldo = ldo;
  a.fill = fill;
  return sample<true>(args, Z, a, device_status, stream);
}
