// k_sample.cu -- drawing a token from a row of logits after temperature, top-k,
// top-p and min-p, and the distribution that they make as log-probabilities.
//
// A cluster of CTAs takes a row: each holds its part in shared memory, so that
// the logits are read from memory once and every later pass runs on chip
// (vocabularies that sixteen CTAs cannot hold are read again each pass).
//
// A token's mass, with m the row's maximum, is 2^y, y = (z - m) log2(e) / T, as a
// whole number `mant` of 31 bits times 2^(-e-30), to a relative 2^-26.5 at the worst
// and 2^-30 in the mean square, with next to no bias (see Mass). Masses are added as whole
// numbers, so in any order with one result. A border of the top-p set or of the draw is
// missed by half of that, 6e-9 of the mass, between a few heavy tokens (less than
// half a step of u or p), by some 1e-10 where a hundred logits and more share the mass.
//
// top-k and top-p are one search, for the first token of the row sorted by
// falling z (then by index) at which the running sum, of ones or of masses,
// reaches a target. A histogram of 1088 bins of z (for masses 1/32 of an octave
// each, so that a bin's tokens share e and their mants are added as they are) gives
// the bin; its tokens (some hundreds of a flat row of 129280) are brought to one
// CTA, which splits them into 256 narrower bins, again and again until few are
// left. A bin of more than 1088 tokens (many equal logits) is instead narrowed by
// four histograms of the bits of z, down to one value, whose tokens are counted by
// index. What is kept is z >= cut; tokens that equal the cut but come after its last
// index are masked in shared memory. Few tokens of a top-k are listed at once, and one
// CTA does all the rest with them. A draw takes the CTA, then 512 tokens, then the token
// that the target mass falls in.
//
// Three CTAs share an SM (64 KB of a row each, 256 threads), so that a row's
// barriers and loads pass under the others' arithmetic. Two CTAs, 320 to 512
// threads, and parts read again from L2 were slower or the same; clusters that take
// row after row (one launch's worth of CTAs) spilled and took 20% more.
//
// 768 rows of 129280, fp32, as log-probabilities (794 MB): temperature alone 215 us
// (3.7 TB/s), top-k 229, top-k and top-p 236, top-p 372 us (2.1 TB/s); bf16
// (596 MB) 172, 152, 159 and 315. Drawn: 195, 182, 198 and 372 us; bf16 141, 111, 121 and
// 308 (settings of each row its own). One row 8 to 20 us. With top-p a CTA spends 6 of its 23 us on the histogram (two
// shared additions a token, 1.6 ns for 32 of them) and 10 in five meetings of the
// cluster; schedulers issue in 46% of the cycles. 51 clusters of eight run at once (of 57
// that SMs have room for), and a place stays empty for 15% of the time between two.
#include <math.h>
#include <stdio.h>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

typedef unsigned long long u64;

constexpr int kSpThreads = 256, kSpWarps = kSpThreads / 32;
constexpr int kSpMaxC = 16;       // CTAs of a cluster
constexpr int kSpBins = 1088;     // 34 octaves of 32 bins, the last one for what lies below
constexpr int kSpNone = 1504;     // from here on (2^-47) a mass is nothing
constexpr int kSpLowQ = 60;      // masses of the last bin are multiples of 2^-60
constexpr int kSpSeg = kSpBins / 8;
constexpr int kSpList = kSpBins;      // tokens of a bin that are brought together,
constexpr int kSpOwn = kSpSeg * 4 / 2; // and of one CTA: half of the histogram's lower words
constexpr int kSpChunk = 512;     // tokens that a warp takes at a time
constexpr float kSpMasked = -1e29f;      // masked tokens are at most this,
constexpr float kSpLeast = -9.9999994e28f;  // the others at least this
constexpr int kSpHist = kSpBins * 8;  // bytes: the histogram, the list or the chunks' sums
constexpr float kSpMagic = 12582912.f;     // 1.5 * 2^23: sums with it round to whole numbers
constexpr uint32_t kSpMagicBits = 0x4B400000u;

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
  int q, fine;   // sums of masses are multiples of 2^-q, of a lane or a chunk of 2^-fine
  int vec, vec_out;
  int* status;
};

// A rounding of z to bins: the whole number nearest to (z - sub) hi + mb - kSpMagic, at most 0 for the maximum.
struct SpScale {
  float sub, hi, mb;
};

struct SpCut {
  float z;
  int last;  // of the tokens with this z, those up to this index are kept
};

struct alignas(128) SpShared {
  uint2 exp2[16];              // kSpExp2 as a whole number and as fp32 (its address has no bits below 128)
  u64 slot[2][kSpMaxC][2];     // what each CTA tells the others
  u64 res[2];                  // a cut and the raw sum of its bin up to it
  u64 found[3];                // a search's bin, the sum before it and what is missing in it
  u64 segs[kSpMaxC][8];        // each CTA's sums of its histogram's eighths
  u64 warp[kSpWarps], warp2[kSpWarps];
  u64 bcast[2];
  u64 few[32];
  float c_hi, c_lo, inv_t, p, u;
  int k, n, m, bad;
  int counts[kSpMaxC];         // tokens of the bin in each CTA
};

// round(2^30 2^(i / 16))
__constant__ uint32_t kSpExp2[16] = {
    1073741824u, 1121280436u, 1170923762u, 1222764986u, 1276901417u, 1333434672u, 1392470869u, 1454120821u,
    1518500250u, 1585730000u, 1655936265u, 1729250827u, 1805811301u, 1885761398u, 1969251188u, 2056437387u};

__device__ __forceinline__ uint32_t ordered(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 is 0
  return b ^ ((int32_t)b < 0 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o ^ ((int32_t)o < 0 ? 0x80000000u : 0xFFFFFFFFu));
}

// Shared memory by 32-bit addresses, the histogram's updates under a predicate in place of a branch.
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 q;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(p) : "memory");
  return q;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {  // of what no one changes
  uint2 q;
  asm("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "r"(p));
  return q;
}
__device__ __forceinline__ void count_if(uint32_t p, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.s32 p, %1, 0;\n @p red.shared.add.u32 [%0], 1;\n}" ::"r"(p), "r"((int)on)
               : "memory");
}
// A sum of numbers of 31 bits as two words kSpBins apart, of their lower 16 bits and of the rest: neither
// overflows with up to 65536 numbers. Where v >= cut and t > low.
__device__ __forceinline__ void add_if(uint32_t p, uint32_t x, float v, float cut, int t, int low) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .u32 l, h;\n setp.ge.f32 p, %2, %3;\n setp.gt.and.s32 p, %4, %5, p;\n"
      " and.b32 l, %1, 65535;\n shr.u32 h, %1, 16;\n @p red.shared.add.u32 [%0], l;\n"
      " @p red.shared.add.u32 [%0 + %6], h;\n}" ::"r"(p),
      "r"(x), "f"(v), "f"(cut), "r"(t), "r"(low), "n"(kSpBins * 4)
      : "memory");
}
// The same where t > low alone.
__device__ __forceinline__ void add_over(uint32_t p, uint32_t x, int t, int low) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .u32 l, h;\n setp.gt.s32 p, %2, %3;\n"
      " and.b32 l, %1, 65535;\n shr.u32 h, %1, 16;\n @p red.shared.add.u32 [%0], l;\n"
      " @p red.shared.add.u32 [%0 + %4], h;\n}" ::"r"(p),
      "r"(x), "r"(t), "r"(low), "n"(kSpBins * 4)
      : "memory");
}
// The same of any many numbers, 32 bits in the lower word: a carry goes to the upper one.
__device__ __forceinline__ void add_carry(uint32_t p, uint32_t x) {
  uint32_t old;
  asm volatile("atom.shared.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(p), "r"(x) : "memory");
  if (old + x < old) asm volatile("red.shared.add.u32 [%0 + %1], 1;" ::"r"(p), "n"(kSpBins * 4) : "memory");
}

// The mass of tokens, of two at a time where it matters. In units of 1/32 octave y is
//   x = (z - sub) (hi + lo) - B,   hi + lo = 32 log2(e) / T,   B = mb's whole number,
// J = round(x) <= 0 names the token's bin, q = J rounded down to an even number its
// table entry and octave (e = -floor(q / 32)), and with r = x - q in [-1/2, 3/2],
//   2^(x/32) = 2^-e T[q mod 32 / 2] (1 + w + w^2/2 + w^3/6 + w^4/24),  w = r ln(2) / 32,
// Taylor's next term being 2^-31.5 at the most. x is never rounded: the fma of z hi with -(q + B) is
// exact up to its own rounding of r, 2^-24 of 1/32 octave, and the bracket less one is at
// most 2^-4.9 in fp32: its roundings and r's are 2^-29 each, 2^-26.9 together at the worst of 33 million
// logits, 2^-29.9 in the mean square, -2^-36 in the mean. sub is 0; where the maximum is so many octaves from 0 that B would not fit (2^16)
// it is the maximum, and z - m is exact for every z whose mass counts (it is within 1/300 of m).
// The table's sixteen entries of 8 bytes take a bank each: reads of it never conflict.
struct Mass {
  SpScale s;
  float lo;
  __device__ __forceinline__ void poly(float r, float tf, uint32_t ti, uint32_t& mant) const {
    const float p = r * fmaf(r, fmaf(r, fmaf(r, 9.1725627e-09f, 1.69385097e-06f), 0.000234596198f), 0.0216608494f);
    mant = ti + (uint32_t)__float2int_rn(tf * p);
  }
  __device__ __forceinline__ uint32_t one(float z, uint32_t tab, int& J) const {
    const float x = z - s.sub;
    const uint32_t t = __float_as_uint(fmaf(x, s.hi, s.mb));
    const uint32_t tq = t & ~1u;
    float r = fmaf(x, s.hi, fmaf(__uint_as_float(tq), -1.f, s.mb));
    r = fmaf(x, lo, r);
    const uint2 w = lds64(tab | (tq << 2 & 0x78u));
    uint32_t mant;
    poly(r, __uint_as_float(w.y), w.x, mant);
    J = (int)(t - kSpMagicBits);
    return mant;
  }
  // the same of two tokens; t: the bits of kSpMagic + J
  template <bool FAR>
  __device__ __forceinline__ void two(float z0, float z1, uint32_t tab, uint32_t* t, uint32_t* mant) const {
    const u64 x = FAR ? tc::add2(tc::f2pack(z0, z1), tc::f2pack(-s.sub, -s.sub)) : tc::f2pack(z0, z1);
    const u64 hi = tc::f2pack(s.hi, s.hi), mb = tc::f2pack(s.mb, s.mb);
    float a, b;
    tc::f2unpack(tc::fma2(x, hi, mb), a, b);
    t[0] = __float_as_uint(a);
    t[1] = __float_as_uint(b);
    const uint32_t q0 = t[0] & ~1u, q1 = t[1] & ~1u;
    u64 r = tc::fma2(tc::f2pack(__uint_as_float(q0), __uint_as_float(q1)), tc::f2pack(-1.f, -1.f), mb);
    r = tc::fma2(x, hi, r);
    r = tc::fma2(x, tc::f2pack(lo, lo), r);
    u64 p = tc::fma2(r, tc::f2pack(9.1725627e-09f, 9.1725627e-09f), tc::f2pack(1.69385097e-06f, 1.69385097e-06f));
    p = tc::fma2(r, p, tc::f2pack(0.000234596198f, 0.000234596198f));
    p = tc::fma2(r, p, tc::f2pack(0.0216608494f, 0.0216608494f));
    p = tc::mul2(r, p);
    tc::f2unpack(p, a, b);
    const uint2 w0 = lds64(tab | (q0 << 2 & 0x78u)), w1 = lds64(tab | (q1 << 2 & 0x78u));
    mant[0] = w0.x + (uint32_t)__float2int_rn(__uint_as_float(w0.y) * a);
    mant[1] = w1.x + (uint32_t)__float2int_rn(__uint_as_float(w1.y) * b);
  }
};
// bin -J: the octave of its masses
__device__ __forceinline__ int octave(int bin) { return (((bin + 1) & ~1) + 31) >> 5; }
// Raw mants of octave e as a multiple of 2^-q, cut off, so that a sum's is at least its parts' together (and with
// some hundred bins and CTAs 2^-34 less at the most); and the least raw sum that reaches `need`.
__device__ __forceinline__ u64 scaled(u64 raw, int e, int q) {
  const int sh = e - (q - 30);
  return sh <= 0 ? raw << -sh : raw >> sh;
}
__device__ __forceinline__ u64 unscaled(u64 need, int e, int q) {
  const int sh = e - (q - 30);
  return sh <= 0 ? (need + (1ull << -sh) - 1) >> -sh : need << sh;
}

__device__ __forceinline__ void st_rank(int* p, uint32_t rank, int x) {
  asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(tc::map_rank(tc::smem_u32(p), rank)), "r"(x) : "memory");
}
__device__ __forceinline__ void st_rank(u64* p, uint32_t rank, u64 x) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(tc::map_rank(tc::smem_u32(p), rank)), "l"(x) : "memory");
}
// not ordered with anything but barriers, so that several are in flight
__device__ __forceinline__ uint32_t ld_rank(uint32_t addr, uint32_t rank) {
  uint32_t x;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(tc::map_rank(addr, rank)));
  return x;
}
__device__ __forceinline__ u64 ld_rank64(uint32_t addr, uint32_t rank) {
  u64 x;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(x) : "r"(tc::map_rank(addr, rank)));
  return x;
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
// maxima that are NaN if one of their inputs is
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// floor(x a) and ceil(x a) for 0 <= a < 1, not -0
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
// One row's work in one CTA. RES: its part lies in shared memory.
template <typename T, bool RES>
struct Row {
  static constexpr int kPer = 16 / (int)sizeof(T);  // values of 16 bytes
  static constexpr int kStep = 8;                   // tokens of a lane that are looked at together
  const SpArgs& a;
  SpShared& sh;
  uint8_t* buf;        // kSpHist bytes
  T* part;             // RES: the row's part
  uint32_t tab, hist, data;  // shared addresses of sh.exp2, buf and part
  const T* row;        // the whole row, in global memory
  int tid, warp, lane;
  uint32_t rank, C;
  int start, count, chunks;  // the part's first token, its tokens, its chunks
  int par = 0;
  float m;                   // the row's maximum
  Mass mass;
  u64 held = 0;              // the mass up to the cut of a search for masses
  u64 own = 0;               // and what of it lies in this CTA (a lane's share, until it is summed)
  bool low_mass = false;     // the search is in the last bin
  SpCut cut{kSpLeast, 0x7FFFFFFF};

  __device__ Row(const SpArgs& a_, SpShared& s_) : a(a_), sh(s_) {}

  // place of value i (< 8) of a lane in step h (0, 1) of a chunk
  __device__ __forceinline__ int at(int ch, int h, int i) const {
    return ch * kSpChunk + h * (32 * kStep) + i / kPer * (32 * kPer) + lane * kPer + i % kPer;
  }
  __device__ __forceinline__ void unpack(const uint4& q, float* v) const {
    const T* t = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = up<T>(t[i]);
  }
  // A lane's tokens of a chunk, from global memory; past the end -inf.
  template <int WORDS>
  __device__ __forceinline__ void fetch(int ch, uint4 (&q)[WORDS], int h = 0) const {
    if (a.vec && (ch + 1) * kSpChunk <= count) {
#pragma unroll
      for (int g = 0; g < WORDS; ++g)
        q[g] = __ldg(reinterpret_cast<const uint4*>(row + start + at(ch, h, 0) + g * (32 * kPer)));
    } else {
#pragma unroll
      for (int g = 0; g < WORDS; ++g) {
        T t[kPer];
        const int l = at(ch, h, 0) + g * (32 * kPer);
#pragma unroll
        for (int i = 0; i < kPer; ++i) t[i] = l + i < count ? row[start + l + i] : T(-INFINITY);
        q[g] = *reinterpret_cast<const uint4*>(t);
      }
    }
  }
  __device__ __forceinline__ void values(int ch, int h, float* v) const {
    uint4 q[kStep / kPer];
    if (RES) {
#pragma unroll
      for (int g = 0; g < kStep / kPer; ++g) q[g] = lds128(data + (uint32_t)(at(ch, h, g * kPer) * (int)sizeof(T)));
    } else {
      fetch(ch, q, h);
    }
#pragma unroll
    for (int g = 0; g < kStep / kPer; ++g) unpack(q[g], v + g * kPer);
  }
  __device__ __forceinline__ float value(int l) const {
    if (RES) return up<T>(part[l]);
    return l < count ? up<T>(row[start + l]) : -INFINITY;
  }
  __device__ __forceinline__ bool kept(float z, int l) const {
    return RES ? z >= cut.z : z > cut.z || (z == cut.z && start + l <= cut.last);
  }
  // f(the eight values of a step, chunk, step)
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int ch = warp; ch < chunks; ch += kSpWarps) {
#pragma unroll 1
      for (int h = 0; h < kSpChunk / (32 * kStep); ++h) {
        float v[kStep];
        values(ch, h, v);
        f(v, ch, h);
      }
    }
  }
  // Every CTA tells x, y, which all of its threads have, to all; all see them in slot[][].
  __device__ __forceinline__ const u64 (*tell(u64 x, u64 y))[2] {
    if (tid < (int)C) {
      st_rank(&sh.slot[par][rank][0], tid, x);
      st_rank(&sh.slot[par][rank][1], tid, y);
    }
    tc::cluster_sync();
    const u64(*s)[2] = sh.slot[par];
    par ^= 1;
    return s;
  }
  // the sum over the CTA's threads, and over those before this one
  __device__ __forceinline__ u64 block_scan(u64 x, u64& before) {
    const u64 inc = warp_scan64(x);
    __syncthreads();
    if (lane == 31) sh.warp[warp] = inc;
    __syncthreads();
    u64 t = 0, b = 0;
#pragma unroll
    for (int i = 0; i < kSpWarps; ++i) {
      if (i == warp) b = t;
      t += sh.warp[i];
    }
    before = b + inc - x;
    return t;
  }

  __device__ __forceinline__ uint32_t* lo() const { return reinterpret_cast<uint32_t*>(buf); }
  __device__ __forceinline__ uint32_t* hi() const { return reinterpret_cast<uint32_t*>(buf) + kSpBins; }
  __device__ __forceinline__ void clear(int n) {
    for (int i = tid; i < n; i += kSpThreads) {
      lo()[i] = 0;
      hi()[i] = 0;
    }
    __syncthreads();
  }
  static constexpr int kUp = RES ? 16 : 32;  // what a bin's upper word counts is 2^kUp
  template <bool MASS>
  __device__ __forceinline__ void add(int bin, uint32_t x) {
    const uint32_t p = hist + 4u * (uint32_t)bin;
    if (!MASS) count_if(p, true);
    else if (RES) add_if(p, x, 0.f, 0.f, 1, 0);
    else add_carry(p, x);
  }
  // With every CTA's histogram filled: the first bin at which the sum up to it reaches the target, the sum before
  // it, and how much of the bin's raw sum is missing there. target 0: ceil(p of all of it), at least 1. Returns
  // whether the sum reaches the target at all. OCT: the bins hold raw mants of their octaves, the last one multiples
  // of 2^-60, and all count as multiples of 2^-q. HIGH: the bins have upper words.
  // Every CTA tells the others its sums of eight segments, so that all know the segment, and all look at its bins:
  // they are not to change before the cluster's next barrier.
  template <bool OCT, bool HIGH>
  __device__ __forceinline__ bool find(u64& target, u64& goal, u64& before, int& bin) {
    constexpr int kEach = (kSpSeg + 31) / 32;
    auto value = [&](u64 v, int g) {
      return !OCT ? v : g < kSpBins - 1 ? scaled(v, octave(g), a.q) : v >> (kSpLowQ - a.q);
    };
    __syncthreads();
    {
      u64 sum = 0;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int b = lane * kEach + i, g = warp * kSpSeg + b;
        if (b < kSpSeg) sum += value((u64)lo()[g] + (HIGH ? (u64)hi()[g] << kUp : 0), g);
      }
      sum = warp_sum64(sum);
      if (lane < (int)C) st_rank(&sh.segs[rank][warp], lane, sum);
    }
    tc::cluster_sync();
    u64 v = 0;
    for (uint32_t c = lane >> 3; c < C; c += 4) v += sh.segs[c][lane & 7];
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
    v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const u64 y = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if ((lane & 7) >= o) v += y;
    }
    const u64 total = __shfl_sync(0xFFFFFFFFu, v, 7);
    if (target == 0) {
      target = mul_floor(total, sh.p, true);
      if (target == 0) target = 1;
    }
    if (target > total) {
      tc::cluster_sync();  // the sums have been read
      return false;
    }
    const int seg = __ffs((int)__ballot_sync(0xFFFFFFFFu, v >= target)) - 1;
    u64 t = __shfl_sync(0xFFFFFFFFu, v, max(seg, 1) - 1);
    if (seg == 0) t = 0;
    const int g = seg * kSpSeg + tid;
    u64 raw = 0, mine;
    if (tid < kSpSeg) {
#pragma unroll
      for (uint32_t c0 = 0; c0 < kSpMaxC; c0 += 8) {
        if (c0 >= C) break;
        uint32_t l[8] = {}, h[8] = {};
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c)
          if (c0 + c < C) {
            l[c] = ld_rank(hist + 4 * g, c0 + c);
            if (HIGH) h[c] = ld_rank(hist + 4 * (g + kSpBins), c0 + c);
          }
#pragma unroll
        for (int c = 0; c < 8; ++c) raw += (u64)l[c] + ((u64)h[c] << kUp);
      }
    }
    const u64 x = value(raw, g);
    block_scan(x, mine);
    t += mine;
    if (t < target && t + x >= target) {
      const u64 need = target - t;
      sh.found[0] = (u64)g;
      sh.found[1] = t;
      sh.found[2] = !OCT ? need : min(g < kSpBins - 1 ? unscaled(need, octave(g), a.q) : need << (kSpLowQ - a.q), raw);
    }
    __syncthreads();
    bin = (int)sh.found[0];
    before = sh.found[1];
    goal = sh.found[2];
    return true;
  }

  // Lists a token of the part.
  __device__ __forceinline__ void note(u64* list, int room, float z, int l) {
    const int n = atomicAdd(&sh.n, 1);
    if (n < room) list[n] = (u64)~ordered(z) << 32 | (uint32_t)(start + l);
  }

  // Greedy: the cut is the lowest token of the row's maximum. MASK: the others are masked.
  template <bool MASK>
  __device__ void first_max() {
    if (tid == 0) {
      sh.n = 0x7FFFFFFF;
      sh.m = 0;
    }
    __syncthreads();
    each([&](const float* v, int ch, int h) {
      uint32_t hits = 0;
#pragma unroll
      for (int i = 0; i < kStep; ++i)
        if (v[i] == m) hits |= 1u << i;
      for (; hits; hits &= hits - 1) {
        atomicMin(&sh.n, start + at(ch, h, __ffs((int)hits) - 1));
        atomicAdd(&sh.m, 1);
      }
    });
    __syncthreads();
    const u64(*s)[2] = tell((u64)(uint32_t)sh.n, (u64)(uint32_t)sh.m);
    u64 first = ~0ull, equals = 0;
    for (uint32_t c = 0; c < C; ++c) {
      first = min(first, s[c][0]);
      equals += s[c][1];
    }
    cut = SpCut{m, (int)first};
    if (MASK && RES && equals > 1) {
      each([&](const float* v, int ch, int h) {
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          if (v[i] == m && start + at(ch, h, i) > cut.last) part[at(ch, h, i)] = T(-INFINITY);
      });
      __syncthreads();
    }
  }

  // Tightens the cut to the first of the kept tokens, in order, at which the running
  // count (MASS: mass) reaches the target. The last bin takes in what lies below the others (its masses
  // are added as multiples of 2^-60). OWN: the CTA's kept mass is wanted too. Returns whether it is known.
  template <bool MASS, bool OWN>
  __device__ bool select(u64 target, const SpScale& b) {
    constexpr int kLow = (int)kSpMagicBits - (kSpBins - 1);
    auto bits_of = [&](float z) { return __float_as_int(fmaf(z - b.sub, b.hi, b.mb)); };
    clear(kSpBins);
    if (tid == 0) sh.n = 0;
    u64 light = 0;
    // what lies between kLow and nothing is one comparison of unsigned numbers
    constexpr uint32_t kNone = kSpMagicBits - kSpNone;
    auto lightest = [&](const float* v, const uint32_t* t, const uint32_t* mant, int ch, int h) {
      uint32_t least = ~0u;
#pragma unroll
      for (int i = 0; i < kStep; i += 2) least = min(least, min(t[i] - kNone, t[i + 1] - kNone));
      if (least <= (uint32_t)kLow - kNone) {
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          if ((int)t[i] <= kLow && kept(v[i], at(ch, h, i))) light += weigh(mant[i], (int)t[i], kSpLowQ);
      }
    };
    if (!MASS) {
      each([&](const float* v, int ch, int h) {
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          count_if(hist + 4u * kSpMagicBits - 4u * (uint32_t)max(bits_of(v[i]), kLow), kept(v[i], at(ch, h, i)));
      });
    } else if (RES && b.sub == 0.f && cut.z == kSpLeast && b.hi > 1e-24f && m > -1e28f) {
      // masked tokens lie 9e28 and more below the maximum, below the bins
      each([&](const float* v, int ch, int h) {
        uint32_t t[kStep], mant[kStep];
#pragma unroll
        for (int i = 0; i < kStep; i += 2) mass.template two<false>(v[i], v[i + 1], tab, t + i, mant + i);
#pragma unroll
        for (int i = 0; i < kStep; ++i) add_over(hist + 4u * kSpMagicBits - 4u * t[i], mant[i], (int)t[i], kLow);
        lightest(v, t, mant, ch, h);
      });
    } else {
      each([&](const float* v, int ch, int h) {
        uint32_t t[kStep], mant[kStep];
#pragma unroll
        for (int i = 0; i < kStep; i += 2) mass.template two<true>(v[i], v[i + 1], tab, t + i, mant + i);
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
          const uint32_t p = hist + 4u * kSpMagicBits - 4u * t[i];
          if (RES) add_if(p, mant[i], v[i], cut.z, (int)t[i], kLow);
          else if ((int)t[i] > kLow && kept(v[i], at(ch, h, i))) add_carry(p, mant[i]);
        }
        lightest(v, t, mant, ch, h);
      });
    }
    if (MASS) {
      light = warp_sum64(light);
      if (lane == 0 && light) {
        constexpr u64 kMask = (1ull << kUp) - 1;
        const uint32_t l = (uint32_t)(light & kMask), old = atomicAdd(lo() + kSpBins - 1, l);
        atomicAdd(hi() + kSpBins - 1, (uint32_t)(light >> kUp) + (old + l < old ? 1u : 0u));
      }
    }
    u64 before, goal;
    int bin;
    if (!find<MASS, MASS>(target, goal, before, bin)) return false;
    const bool low = bin == kSpBins - 1;
    low_mass = MASS && low;
    const int e = octave(bin);
    const int bits = (int)kSpMagicBits - bin;
    auto inside = [&](float z) { return low ? bits_of(z) <= bits : bits_of(z) == bits; };
    auto units = [&](u64 sum) { return low ? sum >> (kSpLowQ - a.q) : scaled(sum, e, a.q); };
    if (OWN) {
      own = 0;
      for (int g = tid; g < bin; g += kSpThreads) own += scaled((u64)lo()[g] + ((u64)hi()[g] << kUp), octave(g), a.q);
      __syncthreads();  // the histogram has been read
    }
    // the CTA's tokens of the bin, into the half of the histogram's lower words that find() leaves alone
    const int at0 = bin < kSpBins / 2 ? kSpBins / 2 * 4 : 0;
    u64* list = reinterpret_cast<u64*>(buf + at0);
    if (low) {
      each([&](const float* v, int ch, int h) {
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          if (inside(v[i]) && kept(v[i], at(ch, h, i))) note(list, kSpOwn, v[i], at(ch, h, i));
      });
    } else {
      const u64 sub = tc::f2pack(-b.sub, -b.sub), up = tc::f2pack(b.hi, b.hi), mb = tc::f2pack(b.mb, b.mb);
      each([&](const float* v, int ch, int h) {
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < kStep; i += 2) {
          float x, y;
          tc::f2unpack(tc::fma2(tc::add2(tc::f2pack(v[i], v[i + 1]), sub), up, mb), x, y);
          if (__float_as_int(x) == bits) hits |= 1u << i;
          if (__float_as_int(y) == bits) hits |= 2u << i;
        }
        for (; hits; hits &= hits - 1) {
          const int l = at(ch, h, __ffs((int)hits) - 1);
          const float z = value(l);
          if (kept(z, l)) note(list, kSpOwn, z, l);
        }
      });
    }
    int n;
    const bool fit = lists_fit(kSpOwn, n);
    if (fit) {
      if (rank == 0) {
        const u64 mine = cut_of_list<MASS>(n, goal, hist + at0);
        if (OWN) own += units(mine);
      }
    } else {
      narrow<MASS>(inside, goal);
    }
    tc::cluster_sync();
    cut.z = unordered((uint32_t)(sh.res[0] >> 32));
    cut.last = (int)(uint32_t)sh.res[0];
    if (MASS) held = before + units(sh.res[1]);
    if (OWN && fit) {
      if (rank != 0) {
        const u64 end = (u64)~(uint32_t)(sh.res[0] >> 32) << 32 | (uint32_t)sh.res[0];
        for (int i = tid; i < sh.n; i += kSpThreads)
          if (list[i] <= end) own += units(raw<MASS>(list[i]));
      }
      u64 ignored;
      own = block_scan(own, ignored);
    }
    if (RES && !fit) {  // settle() has masked the others
      each([&](const float* v, int ch, int h) {
#pragma unroll
        for (int i = 0; i < kStep; ++i)
          if (v[i] == cut.z && start + at(ch, h, i) > cut.last) part[at(ch, h, i)] = T(-INFINITY);
      });
      __syncthreads();
    }
    return OWN && fit;
  }

  template <bool MASS>
  __device__ __forceinline__ uint32_t raw(u64 key) const {
    return MASS ? raw_of(unordered(~(uint32_t)(key >> 32))) : 1;
  }
  __device__ __forceinline__ uint32_t raw_of(float z) const {
    int J;
    const uint32_t mant = mass.one(z, tab, J);
    return low_mass ? (uint32_t)weigh(mant, J + (int)kSpMagicBits, kSpLowQ) : mant;
  }
  // The cut (ordered z, index) and the raw sum up to it, to every CTA.
  __device__ __forceinline__ void answer(u64 key, u64 sum) {
    for (uint32_t c = 0; c < C; ++c) {
      st_rank(&sh.res[0], c, (u64)~(uint32_t)(key >> 32) << 32 | (uint32_t)key);
      st_rank(&sh.res[1], c, sum);
    }
  }

  static constexpr int kOf = (kSpList + kSpThreads - 1) / kSpThreads;  // listed tokens of a thread of CTA 0
  // In CTA 0: the keys (falling z, index) that the CTAs have listed, in any order, each at its shared address `at`.
  __device__ __forceinline__ uint32_t take_list(u64 (&key)[kOf], int n, uint32_t at) {
    uint32_t live = 0;
#pragma unroll
    for (int i = 0; i < kOf; ++i) {
      int e = tid + i * kSpThreads;
      key[i] = ~0ull;
      if (e < n) {
        uint32_t c = 0;
        while (e >= sh.counts[c]) e -= sh.counts[c++];
        key[i] = ld_rank64(at + 8u * (uint32_t)e, c);
        live |= 1u << i;
      }
    }
    return live;
  }
  // The first of the live keys, in order, at which the running sum of weight(key) reaches the goal, in bcast[0] and
  // returned, and the sum there: 256 bins of the keys' range, again and again until 32 are left.
  template <typename W>
  __device__ u64 reach(const u64 (&key)[kOf], uint32_t live, W weight, u64 goal, u64& sum) {
    u64* bins = reinterpret_cast<u64*>(buf);
    u64 base = 0;
    int up = 32;  // keys are told apart by their upper words, falling z, and those of one z by index
    for (;;) {
      uint32_t least = ~0u, most = 0;
#pragma unroll
      for (int i = 0; i < kOf; ++i)
        if (live >> i & 1) {
          least = min(least, (uint32_t)(key[i] >> up));
          most = max(most, (uint32_t)(key[i] >> up));
        }
      least = __reduce_min_sync(0xFFFFFFFFu, least);
      most = __reduce_max_sync(0xFFFFFFFFu, most);
      __syncthreads();  // the list is in registers, and the last turn's words have been read
      if (lane == 0) sh.warp2[warp] = (u64)least << 32 | most;
      if (tid == 0) sh.m = 0;
      bins[tid] = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kSpWarps; ++i) {
        least = min(least, (uint32_t)(sh.warp2[i] >> 32));
        most = max(most, (uint32_t)sh.warp2[i]);
      }
      if (up == 32 && most == least) {
        up = 0;
        continue;
      }
      const int shift = max(0, 32 - __clz(most - least) - 8);
      auto bin_of = [&](u64 k) { return (int)(((uint32_t)(k >> up) - least) >> shift); };
#pragma unroll
      for (int i = 0; i < kOf; ++i)
        if (live >> i & 1) atomicAdd(bins + bin_of(key[i]), weight(key[i]));
      __syncthreads();
      const u64 here = bins[tid];
      u64 before;
      block_scan(here, before);
      before += base;
      if (before < goal && before + here >= goal) {
        sh.bcast[0] = (u64)tid;
        sh.bcast[1] = before;
      }
      __syncthreads();
      base = sh.bcast[1];
#pragma unroll
      for (int i = 0; i < kOf; ++i)
        if (live >> i & 1) {
          if (bin_of(key[i]) == (int)sh.bcast[0]) {
            const int at = atomicAdd(&sh.m, 1);
            if (at < 32) sh.few[at] = key[i];
          } else {
            live &= ~(1u << i);
          }
        }
      __syncthreads();
      if (sh.m <= 32) break;
    }
    if (warp == 0) {
      const u64 mine = lane < sh.m ? sh.few[lane] : ~0ull;
      const u64 w = lane < sh.m ? weight(mine) : 0;
      u64 t = base;
      for (int i = 0; i < sh.m; ++i) {
        const u64 other = __shfl_sync(0xFFFFFFFFu, mine, i), ow = __shfl_sync(0xFFFFFFFFu, w, i);
        if (other < mine) t += ow;
      }
      if (lane < sh.m && t < goal && t + w >= goal) {
        sh.bcast[0] = mine;
        sh.bcast[1] = t + w;
      }
    }
    __syncthreads();
    sum = sh.bcast[1];
    return sh.bcast[0];
  }
  // CTA 0's answer to all: the cut, and the sum up to it. Listed equals of the cut that come after it are masked.
  __device__ __forceinline__ void settle(const u64 (&key)[kOf], int n, u64 end, u64 sum) {
    if (tid == 0) answer(end, sum);
    if (RES) {
#pragma unroll
      for (int i = 0; i < kOf; ++i)
        if (tid + i * kSpThreads < n && key[i] > end && key[i] >> 32 == end >> 32) {
          const int idx = (int)(uint32_t)key[i];
          const uint32_t owner = idx / a.part;
          const uint32_t p = tc::map_rank(data + (uint32_t)((idx - (int)owner * a.part) * (int)sizeof(T)), owner);
          if (sizeof(T) == 4)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(p), "r"(0xFF800000u) : "memory");
          else
            asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(p), "h"((unsigned short)0xFF80u) : "memory");
        }
    }
  }
  // Every CTA's list is complete: their lengths to all. Returns whether they fit, and how many there are.
  __device__ __forceinline__ bool lists_fit(int room, int& n) {
    __syncthreads();
    if (tid < (int)C) st_rank(&sh.counts[rank], tid, sh.n);
    tc::cluster_sync();
    n = 0;
    bool few = true;
    for (uint32_t c = 0; c < C; ++c) {
      n += sh.counts[c];
      few &= sh.counts[c] <= room;
    }
    return few && n <= kSpList;
  }
  // Returns a lane's share of CTA 0's own raw sum up to the cut.
  template <bool MASS>
  __device__ u64 cut_of_list(int n, u64 goal, uint32_t at) {
    u64 key[kOf], sum;
    const uint32_t live = take_list(key, n, at);
    const u64 end = reach(key, live, [&](u64 k) { return (u64)raw<MASS>(k); }, goal, sum);
    settle(key, n, end, sum);
    u64 mine = 0;
#pragma unroll
    for (int i = 0; i < kOf; ++i)
      if (key[i] <= end && (int)(uint32_t)key[i] < a.part) mine += raw<MASS>(key[i]);
    return mine;
  }

  // A row of which top-k keeps few tokens, without looking at all of them twice: the k-th largest of the threads'
  // maxima (`mine`) is at most the k-th largest token, so what is not below its bin holds all that is kept; on flat
  // rows a tenth more than k tokens. Those are listed, and one CTA finds both cuts, leaves out what is below z_min,
  // and draws row_n's token or writes the kept tokens (the others write `fill` meanwhile). Returns false, with
  // nothing done, where they do not fit a list.
  template <bool DIST>
  __device__ bool few(int k, const SpScale& b, float mine, float z_min, int row_n) {
    auto bits_of = [&](float z) { return __float_as_int(fmaf(z - b.sub, b.hi, b.mb)); };
    clear(kSpBins);
    if (tid == 0) sh.n = 0;
    const int t = max(bits_of(mine), (int)kSpMagicBits - (kSpBins - 1));
    if (mine > kSpMasked) add<false>((int)kSpMagicBits - t, 1);
    u64 target = (u64)k, goal, before;
    int bin;
    if (!find<false, false>(target, goal, before, bin)) return false;
    if (bin == kSpBins - 1) {
      tc::cluster_sync();  // the histogram has been read
      return false;
    }
    const int bits = (int)kSpMagicBits - bin;
    const int at0 = bin < kSpBins / 2 ? kSpBins / 2 * 4 : 0;  // away from what find() reads
    u64* list = reinterpret_cast<u64*>(buf + at0);
    const u64 sub = tc::f2pack(-b.sub, -b.sub), up = tc::f2pack(b.hi, b.hi), mb = tc::f2pack(b.mb, b.mb);
    each([&](const float* v, int ch, int h) {
      uint32_t hits = 0;
#pragma unroll
      for (int i = 0; i < kStep; i += 2) {
        float x, y;
        tc::f2unpack(tc::fma2(tc::add2(tc::f2pack(v[i], v[i + 1]), sub), up, mb), x, y);
        if (__float_as_int(x) >= bits) hits |= 1u << i;
        if (__float_as_int(y) >= bits) hits |= 2u << i;
      }
      for (; hits; hits &= hits - 1) {
        const int l = at(ch, h, __ffs((int)hits) - 1);
        note(list, kSpOwn, value(l), l);
      }
    });
    int n;
    if (!lists_fit(kSpOwn, n)) {
      tc::cluster_sync();  // the lengths have been read
      return false;
    }
    u64 key[kOf], sum = 0, ignored;
    uint32_t live = rank == 0 ? take_list(key, n, hist + at0) : 0;
    if (DIST) {
      float* out = a.out + (int64_t)row_n * a.ldo + start;
      if (a.vec_out) {
        for (int i = tid * 4; i + 4 <= count; i += kSpThreads * 4)
          __stcs(reinterpret_cast<float4*>(out + i), make_float4(a.fill, a.fill, a.fill, a.fill));
      }
      for (int i = (a.vec_out ? max(count, 0) & ~3 : 0) + tid; i < count; i += kSpThreads) out[i] = a.fill;
    }
    tc::cluster_arrive();  // the lists have been read, and `fill` written
    if (rank != 0) {
      tc::cluster_wait();
      return true;
    }
    u64 end = reach(key, live, [](u64) { return 1ull; }, (u64)k, sum);
    auto mass_of = [&](u64 x) {
      int J;
      const uint32_t mant = mass.one(unordered(~(uint32_t)(x >> 32)), tab, J);
      return weigh(mant, J + (int)kSpMagicBits, a.q);
    };
    auto mass_up_to = [&](u64 last, float least) {
      u64 all = 0;
#pragma unroll
      for (int i = 0; i < kOf; ++i) {
        if (key[i] > last || unordered(~(uint32_t)(key[i] >> 32)) < least) live &= ~(1u << i);
        if (live >> i & 1) all += mass_of(key[i]);
      }
      return block_scan(all, ignored);
    };
    if (sh.p < 1.f) {
      const u64 goal2 = max(mul_floor(mass_up_to(end, kSpLeast), sh.p, true), 1ull);
      end = reach(key, live, mass_of, goal2, sum);
    }
    const u64 S = mass_up_to(end, z_min);
    if (DIST) {
      const float ls = log_of(S);
      tc::cluster_wait();
#pragma unroll
      for (int i = 0; i < kOf; ++i)
        if (live >> i & 1)
          a.out[(int64_t)row_n * a.ldo + (uint32_t)key[i]] =
              fmaf(unordered(~(uint32_t)(key[i] >> 32)) - m, sh.inv_t, -ls);
    } else {
#pragma unroll
      for (int i = 0; i < kOf; ++i) key[i] = key[i] << 32 | key[i] >> 32;  // by index
      const u64 goal2 = mul_floor(S, sh.u, false) + 1;
      const u64 got = reach(key, live, [&](u64 x) { return mass_of(x << 32 | x >> 32); }, goal2, sum);
      if (tid == 0) put(row_n, (int)(got >> 32), unordered(~(uint32_t)got), S);
      tc::cluster_wait();
    }
    return true;
  }

  // The same of a bin with many tokens, by the bits of z, eight at a time, then by index among equals.
  template <bool MASS, typename B>
  __device__ void narrow(B inside, u64 goal) {
    uint32_t prefix = 0;
    u64 before = 0;
    for (int level = 0; level < 4; ++level) {
      const int shift = 24 - 8 * level;
      tc::cluster_sync();
      clear(kSpBins);
      each([&](const float* v, int ch, int h) {
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
          if (!inside(v[i]) || !kept(v[i], at(ch, h, i))) continue;
          const uint32_t key = ~ordered(v[i]);
          if (level > 0 && key >> (shift + 8) != prefix) continue;
          add<MASS>((int)(key >> shift & 255u), MASS ? raw_of(v[i]) : 1);
        }
      });
      int digit;
      u64 here, rest;
      find<false, MASS>(goal, rest, here, digit);
      goal = rest;
      before += here;
      prefix = prefix << 8 | (uint32_t)digit;
    }
    tc::cluster_sync();
    const u64 end = (u64)prefix << 32;
    const float zc = unordered(~prefix);
    const u64 w = raw<MASS>(end);
    u64 keep = (goal + w - 1) / w;
    before += keep * w;
    // how many equals each CTA's chunks hold
    u64* cnt = reinterpret_cast<u64*>(buf);
    u64 mine = 0;
    for (int ch = warp; ch < chunks; ch += kSpWarps) {
      int c = 0;
      for (int h = 0; h < kSpChunk / (32 * kStep); ++h) {
        float v[kStep];
        values(ch, h, v);
#pragma unroll
        for (int i = 0; i < kStep; ++i) c += v[i] == zc && kept(v[i], at(ch, h, i)) ? 1 : 0;
      }
      c = __reduce_add_sync(0xFFFFFFFFu, c);
      if (lane == 0) {
        cnt[ch] = (u64)c;
        mine += (u64)c;
      }
    }
    u64 ignored;
    mine = block_scan(mine, ignored);
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
          if (lane == 0) answer(end | (uint32_t)(start + ch * kSpChunk + g * 32 + (int)__fns(hit, 0, (int)keep)), before);
          break;
        }
        keep -= here;
      }
    }
  }

  // The logarithm of a kept mass over the maximum's own: of what it has more, so that it is 0 if nothing else is kept.
  __device__ __forceinline__ float log_of(u64 S) const {
    int J;
    const uint32_t mant = mass.one(m, tab, J);
    const u64 w = weigh(mant, J + (int)kSpMagicBits, a.q);
    return log1pf((float)(S > w ? S - w : 0) / (float)w);
  }
  // A row's answer: a token with its z, of kept mass S.
  __device__ __forceinline__ void put(int n, int token, float z, u64 S) const {
    a.token[n] = token;
    if (a.logp) a.logp[n] = (z - m) * sh.inv_t - log_of(S);
  }
  // The kept mass of a lane's tokens of a step: mants times 2^(fine-30-e), added up in two words, of those where that
  // is whole and of the others, times 2^29: all down to 2^-47.
  __device__ __forceinline__ void sum_of(const float* v, int ch, int h, u64& heavy, u64& light) const {
#pragma unroll
    for (int i = 0; i < kStep; i += 2) {
      uint32_t t[2], mant[2];
      mass.template two<true>(v[i], v[i + 1], tab, t, mant);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int n = ((int)t[k] >> 5) - (int)(kSpMagicBits >> 5) + a.fine - 30;
        uint32_t mult;  // 0 for masked tokens and for those that are nothing
        asm("shl.b32 %0, 1, %1;" : "=r"(mult) : "r"(n >= 0 ? n : n + 29));
        if (!kept(v[i + k], at(ch, h, i + k))) mult = 0;
        if (n >= 0) heavy += (u64)mant[k] * mult;
        else light += (u64)mant[k] * mult;
      }
    }
  }
  // Of most rows few tokens are kept: steps without any are passed over. A lane's sum is a multiple of 2^-fine,
  // so that light tokens are not lost one by one.
  __device__ __forceinline__ u64 sum_kept(int ch) const {
    u64 heavy = 0, light = 0;
#pragma unroll 1
    for (int h = 0; h < kSpChunk / (32 * kStep); ++h) {
      float v[kStep];
      values(ch, h, v);
      float top = v[0];
#pragma unroll
      for (int i = 1; i < kStep; ++i) top = fmaxf(top, v[i]);
      if (__any_sync(0xFFFFFFFFu, top >= cut.z)) sum_of(v, ch, h, heavy, light);
    }
    return heavy + ((light + (1ull << 28)) >> 29);
  }
  __device__ __forceinline__ u64 rounded(u64 x) const {
    return (x + (1ull << (a.fine - a.q - 1))) >> (a.fine - a.q);
  }
  // The same of one token: mant 2^(q-30-e), rounded. t: the bits of kSpMagic + J. One product serves both
  // ways: by 2^(q-30-e) where that is whole, else by 2^32 times it, whose upper word is the result.
  __device__ __forceinline__ u64 weigh(uint32_t mant, int t, int q) const {
    const int n = (t >> 5) - (int)(kSpMagicBits >> 5) + q - 30;  // q - 30 - e
    const u64 p = (u64)mant * (1u << (n & 31));
    const u64 w = n >= 0 ? p : (p + 0x80000000ull) >> 32;
    return n >= -32 && t > (int)(kSpMagicBits - kSpNone) ? w : 0;
  }
};

// DIST: the whole distribution is written; otherwise a token is drawn.
template <typename T, bool RES, bool DIST>
__global__ void __launch_bounds__(kSpThreads, 3) k_sample(SpArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ SpShared sh;
  typedef Row<T, RES> R;
  R w(a, sh);
  w.tid = threadIdx.x;
  w.warp = w.tid >> 5;
  w.lane = w.tid & 31;
  w.rank = tc::cluster_ctarank();
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(w.C));
  const int tid = w.tid;
  const int n = (int)(blockIdx.x / w.C);
  w.buf = smem;
  w.part = reinterpret_cast<T*>(smem + kSpHist);
  w.tab = tc::smem_u32(sh.exp2);
  w.hist = tc::smem_u32(smem);
  w.data = w.hist + kSpHist;
  w.row = static_cast<const T*>(a.Z) + (int64_t)n * a.ldz;
  w.start = (int)min((int64_t)w.rank * a.part, (int64_t)a.V);
  w.count = min(a.part, a.V - w.start);
  w.chunks = (w.count + kSpChunk - 1) / kSpChunk;
  if (tid < 16) sh.exp2[tid] = make_uint2(kSpExp2[tid], __float_as_uint((float)kSpExp2[tid]));
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
    t = fmaxf(t, 1e-30f);  // 32 log2(e) / T and 1 / T stay in fp32's range
    // 32 log2(e) / T, its rounding error with it
    const float l_hi = 46.1662407f, l_lo = 6.16308171e-07f;
    sh.c_hi = l_hi / t;
    sh.c_lo = (fmaf(-sh.c_hi, t, l_hi) + l_lo) / t;
    sh.inv_t = 1.f / t;
    sh.bcast[0] = __double_as_longlong(mp > 0.f ? (double)t * log((double)mp) : -INFINITY);
    sh.p = fabsf(p);  // -0 is 0: mul_floor takes its factor's bits
    sh.u = fabsf(u);
    sh.k = k;
  }

  // the row's part: to shared memory, its maximum on the way, and a sample of its logits; a lane has eight loads in flight
  float top = -INFINITY, sum = 0.f, seen = 0.f;
  {
    constexpr int kWords = kSpChunk / (32 * R::kPer), kBatch = 8 / kWords;
    uint32_t pairs = 0xFF80FF80u;  // of bf16: the maximum of the even and of the odd places
    for (int c0 = w.warp; c0 < w.chunks; c0 += kSpWarps * kBatch) {
      uint4 q[kBatch][kWords];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (c0 + b * kSpWarps < w.chunks) w.fetch(c0 + b * kSpWarps, q[b]);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int ch = c0 + b * kSpWarps;
        if (ch >= w.chunks) break;
#pragma unroll
        for (int g = 0; g < kWords; ++g) {
          const uint4 x = q[b][g];
          if (sizeof(T) == 4) {
            top = max_nan(top, __uint_as_float(x.x), __uint_as_float(x.y));
            top = max_nan(top, __uint_as_float(x.z), __uint_as_float(x.w));
          } else {
            pairs = max_nan2(max_nan2(pairs, max_nan2(x.x, x.y)), max_nan2(x.z, x.w));
          }
          if (RES) *reinterpret_cast<uint4*>(w.part + w.at(ch, 0, 0) + g * (32 * R::kPer)) = x;
        }
        const float z = sizeof(T) == 4 ? __uint_as_float(q[b][0].x) : __uint_as_float(q[b][0].x << 16);
        if (z > kSpMasked) {
          sum += fmaxf(z, -1e4f);
          seen += 1.f;
        }
      }
    }
    if (sizeof(T) == 2) top = max_nan(__uint_as_float(pairs << 16), __uint_as_float(pairs & 0xFFFF0000u));
  }
  const float mine = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  sum = warp_sum(sum);
  seen = warp_sum(seen);
  if (w.lane == 0) {
    sh.warp[w.warp] = __float_as_uint(top);
    sh.warp2[w.warp] = (u64)__float_as_uint(sum) << 32 | __float_as_uint(seen);
  }
  __syncthreads();
  const double t_log = __longlong_as_double((long long)sh.bcast[0]);
  bool bad = sh.bad;
  sum = seen = 0.f;
  for (int i = 0; i < kSpWarps; ++i) {
    top = max_nan(top, __uint_as_float((uint32_t)sh.warp[i]));
    sum += __uint_as_float((uint32_t)(sh.warp2[i] >> 32));
    seen += __uint_as_float((uint32_t)sh.warp2[i]);
  }
  asm volatile("barrier.cluster.wait;" ::: "memory");
  {
    const u64(*s)[2] = w.tell(__float_as_uint(top), (u64)__float_as_uint(sum) << 32 | __float_as_uint(seen));
    sum = seen = 0.f;
    for (uint32_t c = 0; c < w.C; ++c) {
      top = max_nan(top, __uint_as_float((uint32_t)s[c][0]));
      sum += __uint_as_float((uint32_t)(s[c][1] >> 32));
      seen += __uint_as_float((uint32_t)s[c][1]);
    }
  }
  bad |= !(top < INFINITY);
  if (bad || top <= kSpMasked) {
    if (bad && w.rank == 0 && tid == 0) raise_status(a.status, DSPARK_ENUMERIC);
    if (DIST) {
      float* out = a.out + (int64_t)n * a.ldo + w.start;
      for (int i = tid; i < w.count; i += kSpThreads) out[i] = a.fill;
    } else if (w.rank == 0 && tid == 0) {
      a.token[n] = -1;
      if (a.logp) a.logp[n] = bad ? NAN : -INFINITY;
    }
    return;  // nothing is written to another CTA after tell()
  }
  w.m = top;
  {
    // the bins' zero: a whole number next to the maximum, one above it, so that its product's rounding error
    // (2^-3 of a bin) leaves J <= 0
    const float at = top * sh.c_hi;
    const bool far = !(fabsf(at) < 2097152.f);
    w.mass.s.sub = far ? top : 0.f;
    w.mass.s.hi = sh.c_hi;
    w.mass.s.mb = kSpMagic - 1.f - (far ? 0.f : rintf(at));
    w.mass.lo = sh.c_lo;
  }

  bool exact = false;  // held is the kept mass
  bool shared_out = false;  // and own the CTA's share of it
  const float z_min = t_log > -INFINITY ? __double2float_ru((double)top + t_log) : kSpLeast;
  const bool greedy = sh.k == 1;
  if (greedy) {
    w.template first_max<DIST>();
    if (!DIST) {  // its probability is 1
      if (w.rank == 0 && tid == 0) {
        a.token[n] = w.cut.last;
        if (a.logp) a.logp[n] = 0.f;
      }
      return;
    }
  } else {
    if (sh.k > 0 && sh.k < a.V) {
      // bins up to four times the mean distance from the maximum: half of the tokens lie within two
      const float mean = top - sum / fmaxf(seen, 1.f);
      const float beta = mean > 0.f ? fminf(kSpBins / (4.f * mean), 1e30f) : 0.f;
      const SpScale b{top, beta, kSpMagic};
      // half as many tokens as threads: up to 1.4 listed for each; 640 of a list's 1088
      if (sh.k <= min((int)w.C * kSpThreads / 2, 640) && w.template few<DIST>(sh.k, b, mine, z_min, n)) return;
      w.template select<false, false>((u64)sh.k, b);
    }
    if (sh.p < 1.f) {
      shared_out = w.template select<true, !DIST>(0, w.mass.s);
      exact = true;
    }
  }
  if (!greedy && z_min > w.cut.z) {
    w.cut = SpCut{z_min, 0x7FFFFFFF};
    exact = shared_out = false;
  }

  if (DIST) {
    u64 S = w.held;
    if (!exact) {
      u64 t = 0, ignored;
      for (int ch = w.warp; ch < w.chunks; ch += kSpWarps) t += w.sum_kept(ch);
      const u64 mine = w.block_scan(w.rounded(t), ignored);
      const u64(*s)[2] = w.tell(mine, 0);
      S = 0;
      for (uint32_t c = 0; c < w.C; ++c) S += s[c][0];
    }
    const float ls = w.log_of(S);
    float* out = a.out + (int64_t)n * a.ldo + w.start;
    w.each([&](const float* v, int ch, int h) {
      float y[R::kStep];
#pragma unroll
      for (int i = 0; i < R::kStep; ++i)
        y[i] = w.kept(v[i], w.at(ch, h, i)) ? fmaf(v[i] - top, sh.inv_t, -ls) : a.fill;
#pragma unroll
      for (int g = 0; g < R::kStep / 4; ++g) {
        const int l = w.at(ch, h, g * 4);
        if (a.vec_out && l + 4 <= w.count) {
          __stcs(reinterpret_cast<float4*>(out + l), make_float4(y[4 * g], y[4 * g + 1], y[4 * g + 2], y[4 * g + 3]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (l + i < w.count) out[l + i] = y[4 * g + i];
        }
      }
    });
  } else {
    u64* chunk = reinterpret_cast<u64*>(w.buf);
    const int kEach = (w.chunks + kSpThreads - 1) / kSpThreads;
    u64 mine_before;
    // the chunks' sums, at least 1 if there is anything; returns the CTA's
    auto sums = [&] {
      for (int ch = w.warp; ch < w.chunks; ch += kSpWarps) {
        const u64 t = warp_sum64(w.sum_kept(ch));
        if (w.lane == 0) chunk[ch] = t ? max(w.rounded(t), 1ull) : 0;
      }
      __syncthreads();
      u64 t = 0;
      for (int i = 0; i < kEach; ++i) t += tid * kEach + i < w.chunks ? chunk[tid * kEach + i] : 0;
      return w.block_scan(t, mine_before);
    };
    u64 mine = shared_out ? w.own : sums(), S = 0, before = 0;
    const u64(*s)[2] = w.tell(mine, 0);
    for (uint32_t c = 0; c < w.C; ++c) {
      if (c == w.rank) before = S;
      S += s[c][0];
    }
    u64 target = mul_floor(S, sh.u, false);
    if (target >= before && target < before + mine) {
      if (shared_out) {  // only here are they looked at: the last bits may differ
        mine = sums();
        target = before + min(target - before, mine - 1);
      }
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
      constexpr int kOwn = kSpChunk / kSpThreads;
      u64 own[kOwn], sum = 0, y;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int l = ch * kSpChunk + tid * kOwn + i;
        const float z = w.value(l);
        int J;
        const uint32_t mant = w.mass.one(z, w.tab, J);
        own[i] = w.kept(z, l) ? w.weigh(mant, J + (int)kSpMagicBits, a.q) : 0;
        sum += own[i];
      }
      u64 total = w.block_scan(sum, y);
      if (total == 0) {  // tokens so light that only their sum is a unit: the first of them
        sum = 0;
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          const int l = ch * kSpChunk + tid * kOwn + i;
          sum += own[i] = w.kept(w.value(l), l) ? 1 : 0;
        }
        w.block_scan(sum, y);
        total = 1;
      }
      // the chunk's sum may be a few units more than its tokens', each rounded by itself
      const u64 rest2 = min(rest, total - 1);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (rest2 >= y && rest2 < y + own[i]) {
          const int l = ch * kSpChunk + tid * kOwn + i;
          w.put(n, w.start + l, w.value(l), S);
        }
        y += own[i];
      }
    }
  }
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
  if (!Z || !on(Z, size) || Z == a.out) return DSPARK_EINVAL;
  if (DIST ? (!a.out || !on(a.out, 4) || a.ldo < s->V)
           : (!a.u || !a.token || !on(a.u, 4) || !on(a.token, 4) || !on(a.logp, 4)))
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
  a.fine = bits <= 20 ? 52 : 49;  // a lane has at most 2^8 tokens, or 2^12, and a chunk 2^9
  // The smallest cluster whose parts leave room for three CTAs on an SM, and more CTAs where the rows do
  // not fill the SMs, down to 4096 tokens a CTA (16 rows of 32000 with top-p: 13.3 us with eight CTAs each, 16.3 with 16).
  auto part = [&](int C) { return ((a.V + C - 1) / C + kSpChunk - 1) / kSpChunk * kSpChunk; };
  int C = 1;
  while (C < kSpMaxC && (size_t)part(C) * size > 64 * 1024) C *= 2;
  while (C < kSpMaxC && (int64_t)a.N * C < 152 && part(C) > 4096) C *= 2;
  a.part = part(C);
  const bool res = (size_t)a.part * size <= 180 * 1024 && a.part <= 65536;  // see add_if
  const size_t sums = (size_t)a.part / kSpChunk * 8;
  const size_t smem = res ? kSpHist + (size_t)a.part * size : sums > kSpHist ? sums : kSpHist;
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
