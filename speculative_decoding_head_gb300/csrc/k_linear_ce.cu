// k_linear_ce.cu -- softmax cross entropy of a linear layer over a large
// vocabulary, with its gradients, without keeping the logits.
//
//   z[n][v] = sum_k X[n][k] W[v][k] (+ U[n][v]),  lse_n = log sum_v e^{z[n][v]}
//   loss_n  = lse_n - z[n][t_n]
//   G[n][v] = w_n (e^{z[n][v] - lse_n} - [v = t_n]),  dX = s G W,  dW = s G^T X
//
// The forward is one product whose epilogue reduces each row of a tile to
// (max, sum of exp), so a logit lives in tensor memory only. The gradient
// goes over the vocabulary in pieces: the product is made again, its epilogue
// turns it into the piece's G in bf16 (the tensor cores' operand type: one
// rounding, at most 2^-8 of each entry, after the softmax's fp32), and two
// more products take G to dX (summed over the pieces in fp32) and to the
// piece's rows of dW.
//
// All four products run in one kernel: 256 x 256 tiles on CTA pairs (tcgen05
// cta_group::2; each CTA holds 128 of the tile's rows and loads 128 of its
// columns, 32 KB per 64-deep stage instead of the 48 KB of a 128 x 256 tile
// per CTA), TMA into a ring of four to ten stages, two accumulators so that the epilogue
// of a tile runs under the next tile's products. An operand whose contraction
// index is its row (W in dX, G in dW) is read in place as an MN-major operand;
// only X is transposed in memory, once, for a long dW (the reason is at
// make_plan), and copied for a short one: dW sees zeros in rows that are left out.
//
//   warp 0      TMA producer (both CTAs; bytes counted on the even CTA)
//   warp 1      allocates TMEM; in the even CTA issues the MMAs of the pair
//   warps 2-17  epilogue, two groups of eight: a TMEM lane quarter and half of
//               the tile's columns each
// Every wait is bounded; a timeout sets DSPARK_ETIMEOUT and every role ends.
//
// What bounds it (one GB300, 1866 TFLOP/s and 6792 GB/s measured): long products
// run at the tensor cores' rate under the power cap (N = 4096, K = 5376,
// V = 129280: forward 2.85 to 2.95 ms, 1930 to 2000 TFLOP/s; gradient 9.9 to
// 10.5 ms for three products, 1630 to 1730). Short ones are bound by a tile's
// fixed cost: with K = 256 a tile's four blocks take 2560 cycles of MMA, its
// epilogue about 2500 to 3500 per group, so two groups in turn keep up (640 x
// 129280, no U: forward 50 us, 850 TFLOP/s; one group of sixteen warps took 79).
// With U the forward streams it at 5.1 TB/s (77 us). Small calls are latency:
// about 5 us a launch, of which 1.2 is the first operand's way from memory.
#include <cudaTypedefs.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

// a lambda whose arrays stay in registers
#define LC_INLINE __attribute__((always_inline))

constexpr int kLcTile = 256;     // rows and columns of a pair's tile
constexpr int kLcHalf = 128;     // rows (A) and columns (B) one CTA loads
constexpr int kLcKb = 64;        // contraction depth of a stage (one 128-byte swizzled row)
constexpr int kLcOpBytes = kLcHalf * kLcKb * 2;   // 16 KB: one operand's half of a stage
constexpr int kLcStageBytes = 2 * kLcOpBytes;  // less with narrow tiles of logits
constexpr int kLcBox = 64 * kLcKb * 2;            // 8 KB: a 64 x 64 box of an MN-major operand
// Epilogue warps: two groups that take tiles in turn (one accumulator each), so
// that one's latencies lie under the other's arithmetic; in a group two warps
// per TMEM lane quarter, 128 columns each in parts of 32.
constexpr int kLcEpiWarps = 16;
constexpr int kLcGroupWarps = 8;
constexpr int kLcWarpCols = 128;
constexpr int kLcPart = 32;
constexpr int kLcThreads = 32 * (2 + kLcEpiWarps);
constexpr int kLcTmemCols = 512;                  // two accumulators of 256 columns
// Shared memory: the operand ring and, from its end, boxes of the epilogue
// warps: 32 rows of 32 fp32 columns of U (4 KB) with U, 32 rows of 64 bytes of
// output (2 KB) in the gradient.
constexpr int kLcMaxStages = 10;
constexpr int kLcUBox = 32 * kLcPart * 4;
constexpr int kLcOBox = 32 * 64;
constexpr int kLcRing = 224 * 1024;
__host__ __device__ constexpr int lc_stages(bool grad, bool u, int stage_bytes) {
  const int n = (kLcRing - (grad ? kLcEpiWarps * kLcOBox : 0) - (u ? kLcEpiWarps * kLcUBox : 0)) / stage_bytes;
  const int most = stage_bytes < kLcStageBytes ? kLcMaxStages : 6;  // seven whole ones: 160 x 1024 x 32000 18.8 -> 19.2 us
  return n < most ? n : most;
}
static_assert(lc_stages(true, true, kLcStageBytes) >= 4, "a ring of four stages at least");
constexpr int kLcAhead = 16;                      // tiles announced: the producer is at most 10 + 2 + 2 ahead
constexpr int kLcBars = 2 * kLcMaxStages + 5 + kLcEpiWarps + kLcAhead + 1;
constexpr int kLcBarBytes = 16 * kLcAhead + 8 * kLcBars + 16;
static_assert(kLcBars % 2 == 0, "16-byte ring entries");
constexpr size_t kLcSmem = (size_t)kLcRing + 1024 + kLcBarBytes;
static_assert(kLcSmem <= 232448, "one CTA's shared memory");
constexpr int kLcPairs = 76;                      // CTA pairs of a full grid (152 SMs)
constexpr int kLcTurnedParts = 16;                // sums per row that a pair leaves of turned logits: one a warp
constexpr float kLcRefMin = -1e29f;               // least log2 reference: what lies below it counts as masked

// One product C[M][Nn] = A B^T over a contraction of nkb blocks of 64.
struct LcJob {
  CUtensorMap ta, tb, tu;
  CUtensorMap to, tacc, tslots;  // stores: result (bf16; G's piece), fp32 sums, parts
  int M, Nn;            // rows and columns of the result
  int nkb;              // contraction blocks
  int mt, nt;           // tiles of 256 rows, of tn columns
  int tn;               // 256, or 128 or 64 where logits have few tiles (see z_cols)
  int split;            // pairs that share the tiles' blocks evenly (0: whole tiles)
  int a_mn, b_mn;       // operand's contraction index is its row (MN-major)
  int a_m0;             // row offset in A's map (turned logits: the piece's first token)
  int b_k0;             // contraction offset in B's map
  int b_n0;             // column offset in B's map (and in U's)
  // logits (statistics, G)
  int has_u;
  int turned;           // the result's rows are tokens (see z_turned)
  const float* u;       // U and its leading dimension, for turned logits
  int64_t ldu;
  int V;                // vocabulary
  float gain;           // makes up for the accumulator's truncation (see logit_gain)
  const int32_t* target;
  const float* lse;
  const float* wt;
  float2* part;         // [M][2 nt] (log2 reference, sum of 2^(z log2 e - reference)) per half tile
  float* zt;            // [M] z at the target
  // gradients
  const float* acc;     // [M][lda] sums so far
  int64_t lda;
  int acc_in;           // acc and slots hold the sums of the pieces before: added to
  int to_out;           // the result is complete: to out (through `to`), scaled; else to acc
  int t_out;            // the result is written transposed: out is [Nn][ldo]
  __nv_bfloat16* out;   // [M][ldo]
  int64_t ldo;
  float scale;
};

// The jobs of a launch: the statistics alone (in place 0), or the gradient's,
// each in a place of its own (a launch may lack some: no tiles, no split), so
// that the epilogue finds its job's values at fixed parameter addresses.
enum : int { kLcDx = 0, kLcDw = 1, kLcMakeG = 2, kLcJobs = 3 };
struct LcParams {
  LcJob job[kLcJobs];
  int tiles[kLcJobs];   // whole tiles of jobs 0 .. i (running totals; split jobs add none)
  int sharing, rounds;  // the first `sharing` pairs take whole tiles from round `rounds` on
  int stages, stage_bytes;
  int* status;
  // beside the first piece's G, where xc is given: X [N][K] to xc, rows `ldc` apart (see lc_live_rows)
  const __nv_bfloat16* x;
  __nv_bfloat16* xc;
  int64_t ldx, ldc;
  int N, K;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// first block of pair p's share of `units` blocks split over `split` pairs
__host__ __device__ __forceinline__ int lc_share(int units, int split, int p) {
  return (int)((long long)units * p / split);
}

// whether row n has a part in the gradients: a target, and a token that is not masked
__device__ __forceinline__ bool lc_live(const int32_t* target, const float* lse, int V, int n) {
  const int t = target[n];
  return t >= 0 && t < V && lse[n] != -INFINITY;
}

// X's rows for dW's product, the ones that are left out as zeros: their rows of G are
// zero, but zero times a NaN or an infinity would reach the feature's gradient of every
// token. All epilogue warps of the launch that makes G share it, a lane four pieces
// of 16 bytes at a time, under the first tile's products: dX and dW of 6 x 80 x 1024
// 13.6 us with and without it, of 706 x 1038 x 1415 26.9 and 26.8; the most where rows
// are many and all else is little, 131072 x 64 x 512: 119 and 104.
__device__ __forceinline__ void lc_live_rows(const LcParams& p, const LcJob& z) {
  const unsigned per = (unsigned)(p.K + 7) / 8, total = (unsigned)p.N * per;
  const unsigned lanes = kLcEpiWarps * 32, first = blockIdx.x * lanes + threadIdx.x - 64, step = gridDim.x * lanes;
#pragma unroll 1
  for (unsigned i = first; i < total; i += 4 * step) {
    uint4 x[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const unsigned j = i + f * step;
      if (j >= total) break;
      const unsigned n = j / per;
      const int k = (int)(j - n * per) * 8;
      const __nv_bfloat16* from = p.x + (int64_t)n * p.ldx + k;
      if (k + 8 <= p.K) {
        x[f] = *reinterpret_cast<const uint4*>(from);
      } else {
        unsigned short v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = k + e < p.K ? __bfloat16_as_ushort(from[e]) : 0;
        x[f] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
      }
      if (!lc_live(z.target, z.lse, z.V, (int)n)) x[f] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const unsigned j = i + f * step;
      if (j >= total) break;
      const unsigned n = j / per;
      *reinterpret_cast<uint4*>(p.xc + (int64_t)n * p.ldc + (j - n * per) * 8) = x[f];
    }
  }
}

// What a pair works on next: its share of the split jobs, then whole tiles of
// the others, one a round (the first rounds without pairs busy with shares). The producer goes through it and announces each
// tile to its CTA's other warps.
struct LcWork {
  int job, m, n, kb0, kb1;
  int slot;  // part of a shared tile: its slot; -1: a whole tile
};
struct LcIter {
  int j, u, uend, r;
  __device__ __forceinline__ LcIter(const LcParams& p, int pair)
      : j(-1), u(0), uend(0), r(pair < p.sharing ? p.rounds : 0) {}
  __device__ __forceinline__ bool next(const LcParams& p, int pair, int npairs, LcWork& w) {
    while (u >= uend && j + 1 < kLcJobs) {
      ++j;
      const LcJob& q = p.job[j];
      if (q.split > pair) {
        const int units = q.mt * q.nt * q.nkb;
        u = lc_share(units, q.split, pair);
        uend = lc_share(units, q.split, pair + 1);
      }
    }
    int tile;
    if (u < uend) {
      const LcJob& q = p.job[j];
      w.job = j;
      tile = u / q.nkb;
      w.kb0 = u - tile * q.nkb;
      w.kb1 = min(q.nkb, w.kb0 + uend - u);
      u += w.kb1 - w.kb0;
      w.slot = w.kb0 == 0 && w.kb1 == q.nkb ? -1 : 2 * pair + (w.kb0 == 0 ? 1 : 0);
    } else {
      const int others = npairs - p.sharing;
      const int t = r < p.rounds ? r * others + pair - p.sharing : p.rounds * others + (r - p.rounds) * npairs + pair;
      ++r;
      if (t >= p.tiles[kLcJobs - 1]) return false;
      int k = 0, before = 0;
      while (t >= p.tiles[k]) before = p.tiles[k++];
      w.job = k;
      w.kb0 = 0;
      w.kb1 = p.job[k].nkb;
      w.slot = -1;
      tile = t - before;
    }
    // column tiles outermost, up to 16 row tiles innermost, so that the tiles
    // in flight share their columns' operand in L2
    const LcJob& q = p.job[w.job];
    int g = 0, gm = q.mt;
    if (gm > 16) {
      g = tile / (16 * q.nt);
      gm = min(16, gm - g * 16);
      tile -= g * 16 * q.nt;
    }
    w.n = tile / gm;
    w.m = g * 16 + tile - w.n * gm;
    return true;
  }
};

// An announced tile: job and slot + 1 (x; -1: no more), row tile, column tile,
// blocks of the contraction.
struct LcTile {
  int job, slot, m, n, nkb;
  __device__ __forceinline__ LcTile() {}
  __device__ __forceinline__ explicit LcTile(int4 a) : job(a.x & 3), slot((a.x >> 2) - 1), m(a.y), n(a.z), nkb(a.w) {}
  static __device__ __forceinline__ int4 pack(const LcWork& w) {
    return make_int4(w.job | (w.slot + 1) << 2, w.m, w.n, w.kb1 - w.kb0);
  }
};

// columns of B the MMA takes for a tile of a result of Nn columns: a multiple of 32
__device__ __forceinline__ int lc_cols(int Nn, int n, int tn) { return min(tn, (Nn - n * tn + 31) & ~31); }

// ring position and the parity of its pass
struct LcRing {
  int s, ph;
  uint32_t at;  // the stage's address
  __device__ __forceinline__ void step(int stages, int bytes, uint32_t base) {
    at += bytes;
    if (++s == stages) {
      s = 0;
      at = base;
      ph ^= 1;
    }
  }
};

template <bool GRAD, bool TURNED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLcThreads, 1)
    k_lce(const __grid_constant__ LcParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = tc::smem_u32(smem);
  const uint32_t bars = sbase + kLcRing;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kLcMaxStages + s); };
  auto tfull = [&](int b) { return bars + 8u * (2 * kLcMaxStages + b); };
  auto tempty = [&](int b) { return bars + 8u * (2 * kLcMaxStages + 2 + b); };
  const uint32_t drain = bars + 8u * (2 * kLcMaxStages + 4);
  auto ufull = [&](int w) { return bars + 8u * (2 * kLcMaxStages + 5 + w); };
  auto told = [&](int i) { return bars + 8u * (2 * kLcMaxStages + 5 + kLcEpiWarps + (i & (kLcAhead - 1))); };
  int4* tile_ring = reinterpret_cast<int4*>(smem + kLcRing + 8 * kLcBars);
  unsigned char* tail = reinterpret_cast<unsigned char*>(tile_ring + kLcAhead);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tail);
  volatile int* abort = reinterpret_cast<volatile int*>(tail + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (warp == 0) {
    // one arrival each; the even CTA's tempty: both CTAs' warps of a group
    for (int i = lane; i < kLcBars; i += 32)
      tc::mbar_init(bars + 8u * i, (i >> 1) == kLcMaxStages + 1 ? 2 * kLcGroupWarps : 1);
    tc::fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    *abort = 0;
    for (int k = 0; k < kLcJobs; ++k) {
      if (p.job[k].mt == 0) continue;
      tc::prefetch_tmap(&p.job[k].ta);
      tc::prefetch_tmap(&p.job[k].tb);
    }
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tc::smem_u32(tmem_holder), kLcTmemCols);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_meet();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  // a small grid leaves SMs on which the next kernel can set up meanwhile
  // (which waits in turn: it reads and writes nothing before this grid has ended)
  const bool early = gridDim.x <= kLcPairs;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      LcRing r{0, 0, sbase};
      int iss = 0;
      bool ok = true;
      LcWork w;
      int tj = 0;
      auto tell = [&](int4 x) {
        tile_ring[tj & (kLcAhead - 1)] = x;
        tc::mbar_arrive(told(tj));
        ++tj;
      };
      LcIter it(p, pair);
      bool more = it.next(p, pair, npairs, w);
      pdl_wait();  // the operands are what earlier kernels of the stream wrote
      if (early) pdl_trigger();
      for (; ok && more; more = it.next(p, pair, npairs, w)) {
        tell(LcTile::pack(w));
        const LcJob& j = p.job[w.job];
        const int half = lc_cols(j.Nn, w.n, j.tn) >> 1;  // columns of B in each CTA
        const int am = j.a_m0 + w.m * kLcTile + (int)rank * kLcHalf, bn = j.b_n0 + w.n * j.tn + (int)rank * half;
        const int bboxes = (half + 63) >> 6;  // boxes of an MN-major B
        const uint32_t bytes = (uint32_t)(kLcOpBytes + (j.b_mn ? bboxes * kLcBox : j.tn * kLcKb));
        const bool a_mn = j.a_mn, b_mn = j.b_mn;
        const int b_k0 = j.b_k0;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          ok = tc::mbar_wait(empty(r.s), r.ph ^ 1, abort);
          if (!ok) break;
          const uint32_t bar = tc::map_rank(full(r.s), 0);
          if (rank == 0) tc::mbar_arrive_expect_tx(full(r.s), 2 * bytes);  // both CTAs' copies
          const uint32_t da = r.at, db = da + kLcOpBytes;
          const int ka = kb * kLcKb, kbn = b_k0 + kb * kLcKb;
          if (a_mn) {
            tc::tma_load_2d_pair(da, &j.ta, am, ka, bar);
            tc::tma_load_2d_pair(da + kLcBox, &j.ta, am + 64, ka, bar);
          } else {
            tc::tma_load_2d_pair(da, &j.ta, ka, am, bar);
          }
          if (b_mn) {
            for (int b = 0; b < bboxes; ++b) tc::tma_load_2d_pair(db + b * kLcBox, &j.tb, bn + b * 64, kbn, bar);
          } else {
            tc::tma_load_2d_pair(db, &j.tb, kbn, bn, bar);
          }
          r.step(p.stages, p.stage_bytes, sbase);
          ++iss;
        }
      }
      // the end, for either group of epilogue warps
      for (int k = 0; k < 2 && ok; ++k) tell(make_int4(-1, 0, 0, 0));
      // the last stages' releases, which the even CTA's MMAs send to both CTAs, have arrived before either exits
      for (int i = min(iss, p.stages); i > 0 && ok; --i) {
        const int k = iss - i;
        ok = tc::mbar_wait(empty(k % p.stages), (k / p.stages) & 1, abort);
      }
      if (!ok) {
        if (!*abort) raise_status(p.status, DSPARK_ETIMEOUT);
        *abort = 1;
        // copies already issued land (they complete on the even CTA's barriers) before the pair can exit
        volatile int never = 0;
        for (int k = max(0, iss - p.stages); k < iss; ++k)
          tc::mbar_wait(full(k % p.stages), (k / p.stages) & 1, &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      bool ok = true;
      LcRing r{0, 0, sbase};
      int tj = 0;
      // its own waits are for this grid's work alone: their limit does not run while an
      // earlier kernel, which may have let this one start, is still at work
      pdl_wait();
      for (;; ++tj) {
        ok = tc::mbar_wait(told(tj), (tj / kLcAhead) & 1, abort);
        if (!ok) break;
        const int4 x = tile_ring[tj & (kLcAhead - 1)];
        if (x.x < 0) break;
        const LcTile w(x);
        const LcJob& j = p.job[w.job];
        const uint32_t idesc = tc::idesc_bf16_f32(kLcTile, lc_cols(j.Nn, w.n, j.tn), j.b_mn) | (j.a_mn ? 1u << 15 : 0u);
        const int ab = tj & 1;
        ok = tc::mbar_wait(tempty(ab), ((tj >> 1) & 1) ^ 1, abort);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(ab * kLcTile);
        const uint32_t a_step = j.a_mn ? 2048 : 32, b_step = j.b_mn ? 2048 : 32;
        const uint32_t a_lbo = j.a_mn ? kLcBox : 16, b_lbo = j.b_mn ? kLcBox : 16;
        for (int kb = 0; kb < w.nkb; ++kb) {
          ok = tc::mbar_wait(full(r.s), r.ph, abort);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t da = r.at, db = da + kLcOpBytes;
#pragma unroll
          for (int kk = 0; kk < kLcKb / 16; ++kk)
            tc::mma_bf16_pair(d, tc::smem_desc(da + kk * a_step, a_lbo, 1024),
                              tc::smem_desc(db + kk * b_step, b_lbo, 1024), idesc, (kb > 0 || kk > 0) ? 1u : 0u);
          tc::mma_commit_pair(empty(r.s));
          r.step(p.stages, p.stage_bytes, sbase);
        }
        if (!ok) break;
        tc::mma_commit_pair(tfull(ab));
      }
      // both CTAs' epilogues have released the last tiles: every MMA is complete, and
      // their arrivals have landed before this CTA exits
      for (int t = max(0, tj - 2); t < tj && ok; ++t) ok = tc::mbar_wait(tempty(t & 1), (t >> 1) & 1, abort);
      if (!ok) {
        if (!*abort) raise_status(p.status, DSPARK_ETIMEOUT);
        *abort = 1;
        tc::mma_commit_pair_own(drain);  // every MMA issued completes before TMEM and the peer's operands go
        volatile int never = 0;
        tc::mbar_wait(drain, 0, &never);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // group grp takes tiles grp, grp + 2, ..; its warp reads lane quarter q and
    // 128 columns (half hf) of the accumulator in parts of 32, the next part on
    // its way while one is worked on
    const int e = warp - 2, grp = e >> 3, q = warp & 3, hf = (e >> 2) & 1;
    // this warp's boxes, from the end of the ring: output (gradient), U before them
    const uint32_t ooff = kLcRing - (kLcEpiWarps - e) * kLcOBox;
    const uint32_t uoff = kLcRing - (GRAD ? kLcEpiWarps * kLcOBox : 0) - (kLcEpiWarps - e) * kLcUBox;
    const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(grp * kLcTile);
    const uint32_t released = tc::map_rank(tempty(grp), 0);
    const LcJob& z = p.job[GRAD ? kLcMakeG : 0];  // the job that makes logits
    const bool has_u = z.has_u != 0;
    const int zn = z.tn;  // columns of a tile of logits
    const int v_off = TURNED ? z.a_m0 : z.b_n0;  // the piece's first token
    // turned: the running sums of row hf 32 + lane over the warp's tokens
    float tref = kLcRefMin, tsum = 0.f;
    // the gain goes to the logits when U is added, else into what they are multiplied by
    const float gain = z.gain, zgain = has_u ? 1.f : gain, l2 = tc::kLog2e * zgain;
    const int row0 = (int)rank * kLcHalf + q * 32;  // the warp's first row in a tile
    bool ok = true;
    int ubox = 0;  // boxes of U taken so far
    pdl_wait();    // rows' data, U and the outputs are other kernels' until they end
    if (GRAD && p.xc != nullptr) lc_live_rows(p, z);

    // the tile announced as number i; a logit tile's target, lse and weight of this
    // lane's row, asked for a tile early where the tile is announced by then
    LcTile w;
    int tgt = -1, row = 0, parts = 0, col = 0, half = 0;  // col, half: the warp's first column in the result; its columns
    float lse = 0.f, wt = 1.f;
    bool is_z = false, has = false, asked = false;
    auto ask = [&](const LcTile& x) LC_INLINE {
      const int r = TURNED ? hf * 32 + lane : x.m * kLcTile + row0 + lane, rows = TURNED ? z.Nn : z.M;
      tgt = -1;
      if ((!GRAD || x.job == kLcMakeG) && r < rows) {
        tgt = z.target[r];
        if (GRAD) {
          lse = z.lse[r];
          wt = z.wt ? z.wt[r] : 1.f;
        }
      }
      if (has_u && (!GRAD || x.job == kLcMakeG) && lane == 0 && r < rows) {
        // its boxes of U on their way to L2
        if (TURNED) {
          const int v = v_off + x.m * kLcTile + row0;
          if (v < z.V) tc::tma_prefetch_2d(&z.tu, v, r);
          return;
        }
        const int c0 = hf * (zn >> 1), n = min(zn >> 1, lc_cols(z.Nn, x.n, zn) - c0);
        for (int c = 0; c < n; c += kLcPart) tc::tma_prefetch_2d(&z.tu, z.b_n0 + x.n * zn + c0 + c, r);
      }
    };
    auto announced = [&](int i) LC_INLINE {
      if (!asked) {
        ok = tc::mbar_wait(told(i), (i / kLcAhead) & 1, abort);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) return false;
      }
      const int4 x = tile_ring[i & (kLcAhead - 1)];
      if (x.x < 0) return false;
      w = LcTile(x);
      if (!asked) ask(w);
      is_z = !GRAD || w.job == kLcMakeG;
      const int M = is_z ? z.M : w.job == kLcDx ? p.job[kLcDx].M : p.job[kLcDw].M;
      const int Nn = is_z ? z.Nn : w.job == kLcDx ? p.job[kLcDx].Nn : p.job[kLcDw].Nn;
      row = w.m * kLcTile + row0 + lane;
      has = row < M;
      // parts of 32 columns this warp has (0: none, or no rows; the same for its lanes)
      const int tn = is_z ? zn : kLcTile;
      half = tn >> 1;
      col = w.n * tn + hf * half;
      parts = row - lane < M ? max(0, min(half, lc_cols(Nn, w.n, tn) - hf * half)) / kLcPart : 0;
      if (TURNED && is_z) {  // 32 tokens by 32 rows, the tokens' lanes turned into the rows'
        col = w.m * kLcTile + row0;
        row = hf * 32 + lane;
        has = row < Nn;
        parts = col < M && hf * 32 < Nn ? 1 : 0;
      }
      return true;
    };
    // the tile's box number b of U into the warp's box
    auto load_u = [&](int b) LC_INLINE {
      if (!TURNED && has_u && is_z && b < parts && lane == 0) {
        tc::mbar_arrive_expect_tx(ufull(e), kLcUBox);
        tc::tma_load_2d(sbase + uoff, &z.tu, v_off + col + b * kLcPart, row - lane, ufull(e),
                        tc::policy_evict_first());
      }
    };
    for (int tj = grp; announced(tj); tj += 2) {
      load_u(0);
      if (is_z && (tgt < -1 || tgt >= z.V)) {
        if (TURNED ? w.m == 0 && row0 == 0 : w.n == 0 && hf == 0) raise_status(p.status, DSPARK_ERANGE);
        tgt = -1;
      }
      // the target's place in the half, the exponent's offset: with the weight in it for G
      const int te = tgt - (v_off + col);
      const bool live = !is_z || (tgt >= 0 && lse != -INFINITY);  // else the row has no G
      const float wr = is_z ? wt : 1.f;
      const float off = GRAD ? fmaf(-lse, tc::kLog2e, log2f(fabsf(wr))) : 0.f;
      const bool plain = __all_sync(0xFFFFFFFFu, live && wr >= 0.f);
      ok = tc::mbar_wait(tfull(grp), (tj >> 1) & 1, abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc::tc_fence_after();
      asked = __all_sync(0xFFFFFFFFu, tc::mbar_test(told(tj + 2), ((tj + 2) / kLcAhead) & 1));
      if (asked) {
        const int4 x = tile_ring[(tj + 2) & (kLcAhead - 1)];
        if (x.x >= 0) ask(LcTile(x));
      }
      auto release = [&]() LC_INLINE {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_cluster_relaxed(released);
      };
      if (parts == 0) {
        release();
        if (!GRAD && !TURNED && has) z.part[(int64_t)row * (2 * z.nt) + 2 * w.n + hf] = make_float2(kLcRefMin, 0.f);
        continue;
      }
      const unsigned long long l2e = tc::f2pack(l2, l2);

      // the warp's parts in order: `use` takes a part's values from v, the next
      // part is asked for and `send` does what is left of this one meanwhile;
      // the accumulator is released with the last part's arrival
      float v[kLcPart];
      auto each_part = [&](auto&& use, auto&& send) LC_INLINE {
        const uint32_t t0 = ta + (uint32_t)(hf * half);
        tc::tmem_ld32(t0, v);
#pragma unroll 1
        for (int h = 0; h < parts; ++h) {
          tc::tmem_wait_ld();
          tc::tmem_tie32(v);
          if (h + 1 == parts) release();
          use(h);
          if (h + 1 < parts) tc::tmem_ld32(t0 + (h + 1) * kLcPart, v);
          send(h);
        }
      };
      // turned: a lane's token by 32 rows to its row by 32 tokens, through the warp's
      // box (no bank is met twice); U is read on the way, lanes side by side
      auto turn = [&]() LC_INLINE {
        if (has_u) {
          const int tok = v_off + col + lane;
          const float* up = z.u + (int64_t)(hf * 32) * z.ldu + tok;
#pragma unroll
          for (int i = 0; i < kLcPart; ++i)
            v[i] = fmaf(v[i], gain, tok < z.V && hf * 32 + i < z.Nn ? up[i * z.ldu] : 0.f);
        }
        float* box = reinterpret_cast<float*>(smem + uoff);
#pragma unroll
        for (int i = 0; i < kLcPart; ++i) box[i * 32 + (lane ^ i)] = v[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kLcPart; ++i) v[i] = box[lane * 32 + (i ^ lane)];
        __syncwarp();
      };
      // U's columns of part h onto its logits
      auto add_u = [&](int h) LC_INLINE {
        ok = ok && tc::mbar_wait(ufull(e), (ubox + h) & 1, abort);
        const unsigned char* box = smem + uoff + lane * 128;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(box + ((c ^ (lane & 7)) << 4));
          v[4 * c] = fmaf(v[4 * c], gain, x.x);
          v[4 * c + 1] = fmaf(v[4 * c + 1], gain, x.y);
          v[4 * c + 2] = fmaf(v[4 * c + 2], gain, x.z);
          v[4 * c + 3] = fmaf(v[4 * c + 3], gain, x.w);
        }
        __syncwarp();  // every lane has read the box before the next one lands on it
        load_u(h + 1);
      };
      // Stores (gradient): 32 rows of 64 bytes through the warp's box in the layout
      // of the store's swizzle (conflict-free both ways) and on by the copy engine,
      // which leaves out what lies past the result's extents
      unsigned char* const obox = smem + ooff + lane * 64;
      const uint32_t osw = (lane >> 1) & 3;
      auto box_free = [&]() LC_INLINE {  // the store before has read the box
        if (lane == 0) tc::bulk_wait_read();
        __syncwarp();
      };
      auto put = [&](const CUtensorMap* tm, int c, int r, bool add = false) LC_INLINE {
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (add)
            tc::tma_add_2d(tm, c, r, sbase + ooff);
          else
            tc::tma_store_2d(tm, c, r, sbase + ooff);
          tc::bulk_commit();
        }
      };
      auto put16 = [&](const uint32_t* r, int h, const CUtensorMap* tm, int Nn, __nv_bfloat16* out, int64_t ldo) LC_INLINE {
        box_free();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(obox + ((k ^ osw) << 4)) = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
        const int oc = col + kLcPart * h;
        if ((Nn & 7) != 0 && oc + kLcPart > Nn) {
          // the copy engine writes whole 16-byte pieces: each lane takes a ragged row's end value by value
          if (has)
            for (int i = 0; i < Nn - oc; ++i)
              out[row * ldo + oc + i] =
                  *reinterpret_cast<const __nv_bfloat16*>(obox + (((i >> 3) ^ osw) << 4) + 2 * (i & 7));
        } else {
          put(tm, oc, row - lane);
        }
      };

      if constexpr (!GRAD) {
        float ref = TURNED ? tref : kLcRefMin, sum = TURNED ? tsum : 0.f;
        each_part([&](int h) LC_INLINE {
          if (TURNED)
            turn();
          else if (has_u)
            add_u(h);
          const int t = te - kLcPart * h, left = z.V - col - kLcPart * h;  // columns past the vocabulary are out
          if (left < kLcPart) {
#pragma unroll
            for (int i = 0; i < kLcPart; ++i)
              if (i >= left) v[i] = -INFINITY;
          }
          if (t >= 0 && t < kLcPart) {
            float x = 0.f;
#pragma unroll
            for (int i = 0; i < kLcPart; ++i) x = i == t ? v[i] : x;
            if (has) z.zt[row] = x * zgain;
          }
          float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int i = 4; i < 28; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = tc::max3f(mx[k], v[i + k], v[i + 4 + k]);
          mx[0] = tc::max3f(mx[0], v[28], v[29]);
          mx[1] = tc::max3f(mx[1], v[30], v[31]);
          // reference: the maximum in log2 units, rounded up to a whole number,
          // so that one fused step gives each exponent with one rounding; what
          // lies below its least value (-inf, the type's lowest value as a
          // mask) adds nothing to the sum
          const float nr = fmaxf(ref, ceilf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * l2));
          sum *= tc::ex2_ftz(ref - nr);
          ref = nr;
          const unsigned long long nref = tc::f2pack(-ref, -ref);
          unsigned long long s2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < kLcPart; i += 2) {
            float a, b;
            tc::f2unpack(tc::fma2(tc::f2pack(v[i], v[i + 1]), l2e, nref), a, b);
            s2[(i >> 1) & 3] = tc::add2(s2[(i >> 1) & 3], tc::f2pack(tc::ex2_ftz(a), tc::ex2_ftz(b)));
          }
          float a, b;
          tc::f2unpack(tc::add2(tc::add2(s2[0], s2[1]), tc::add2(s2[2], s2[3])), a, b);
          sum += a + b;
        }, [](int) {});
        if (TURNED) {
          tref = ref;
          tsum = sum;
        } else if (has) {
          z.part[(int64_t)row * (2 * z.nt) + 2 * w.n + hf] = make_float2(ref, sum);
        }
      } else if (is_z) {
        const unsigned long long off2 = tc::f2pack(off, off);
        uint32_t r[kLcPart / 2];
        each_part([&](int h) LC_INLINE {
          if (TURNED)
            turn();
          else if (has_u)
            add_u(h);
          const int t = te - kLcPart * h;
#pragma unroll
          for (int i = 0; i < kLcPart; i += 2) {
            float a, b;
            tc::f2unpack(tc::fma2(tc::f2pack(v[i], v[i + 1]), l2e, off2), a, b);
            v[i] = tc::ex2_ftz(a);
            v[i + 1] = tc::ex2_ftz(b);
          }
          if (t >= 0 && t < kLcPart) {
#pragma unroll
            for (int i = 0; i < kLcPart; ++i) v[i] = i == t ? v[i] - fabsf(wr) : v[i];
          }
#pragma unroll
          for (int k = 0; k < kLcPart / 2; ++k) r[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
          if (!plain) {  // a row without G, or of negative weight
            const uint32_t keep = live ? 0xFFFFFFFFu : 0u, flip = wr < 0.f ? 0x80008000u : 0u;
#pragma unroll
            for (int k = 0; k < kLcPart / 2; ++k) r[k] = (r[k] ^ flip) & keep;
          }
        }, [&](int h) LC_INLINE { put16(r, h, &z.to, 0, nullptr, 0); });
      } else {
        const LcJob &jx = p.job[kLcDx], &jw = p.job[kLcDw];
        const bool dx = w.job == kLcDx, whole = w.slot < 0;
        auto add_acc = [&](int h) LC_INLINE {  // the sums of the pieces before (rows padded to whole parts)
          const float* ap = (dx ? jx.acc + row * jx.lda : jw.acc + row * jw.lda) + col + kLcPart * h;
#pragma unroll
          for (int i = 0; i < kLcPart; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(ap + i);
            v[i] += x.x;
            v[i + 1] += x.y;
            v[i + 2] += x.z;
            v[i + 3] += x.w;
          }
        };
        const bool acc_in = whole && has && (dx ? jx.acc_in : jw.acc_in);
        if (whole && (dx ? jx.to_out : jw.to_out)) {
          const float f = dx ? jx.scale : jw.scale;
          const int Nn = dx ? jx.Nn : jw.Nn;
          __nv_bfloat16* out = dx ? jx.out : jw.out;
          const int64_t ldo = dx ? jx.ldo : jw.ldo;
          const CUtensorMap* to = dx ? &jx.to : &jw.to;
          uint32_t r[kLcPart / 2];
          auto pack = [&](int h) LC_INLINE {
            if (acc_in) add_acc(h);
#pragma unroll
            for (int k = 0; k < kLcPart / 2; ++k) r[k] = pack_bf16(v[2 * k] * f, v[2 * k + 1] * f);
          };
          if (dx ? jx.t_out : jw.t_out) {
            // a 32 x 32 box with the result's columns as rows: lanes side by side
            const int M = dx ? jx.M : jw.M, r0 = row - lane;
            __nv_bfloat16* tb = reinterpret_cast<__nv_bfloat16*>(smem + ooff);
            each_part(pack, [&](int h) LC_INLINE {
              const int oc = col + kLcPart * h;
              box_free();
#pragma unroll
              for (int k = 0; k < kLcPart; ++k)
                tb[32 * k + lane] = __ushort_as_bfloat16((unsigned short)(r[k / 2] >> (16 * (k & 1))));
              if ((M & 7) != 0 && r0 + 32 > M) {  // a ragged end of the rows written, value by value
                if (has)
                  for (int k = 0; k < min(kLcPart, Nn - oc); ++k) out[(oc + k) * ldo + row] = tb[32 * k + lane];
              } else {
                put(to, r0, oc);
              }
            });
          } else {
            each_part(pack, [&](int h) LC_INLINE { put16(r, h, to, Nn, out, ldo); });
          }
        } else {
          const CUtensorMap* tm = whole ? (dx ? &jx.tacc : &jw.tacc) : (dx ? &jx.tslots : &jw.tslots);
          const int sc = whole ? col : hf * half, sr = whole ? row - lane : w.slot * kLcTile + row0;
          const bool add = dx ? jx.acc_in : jw.acc_in;  // onto the sums of the pieces before
          each_part([&](int h) LC_INLINE {
#pragma unroll
            for (int g = 0; g < 2; ++g) {  // 16 columns at a time
              box_free();
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(obox + ((k ^ osw) << 4)) = make_float4(
                    v[16 * g + 4 * k], v[16 * g + 4 * k + 1], v[16 * g + 4 * k + 2], v[16 * g + 4 * k + 3]);
              put(tm, sc + kLcPart * h + 16 * g, sr, add);
            }
          }, [](int) {});
        }
      }
      if (!TURNED && has_u && is_z) ubox += parts;
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
    }
    if (!GRAD && TURNED && hf * 32 + lane < z.Nn)
      z.part[(int64_t)(hf * 32 + lane) * (kLcTurnedParts * npairs) + kLcTurnedParts * pair + grp * 8 + (int)rank * 4 + q] =
          make_float2(tref, tsum);
    if (!ok && lane == 0) {
      if (!*abort) raise_status(p.status, DSPARK_ETIMEOUT);
      *abort = 1;
      // boxes of U still in flight land before the CTA can exit
      volatile int never = 0;
      for (int b = ubox; !TURNED && b < ubox + kLcWarpCols / kLcPart; ++b)
        tc::mbar_wait(ufull(e), b & 1, &never);
    }
    if (GRAD && lane == 0) tc::bulk_wait_all();
  }
  if (!early) pdl_trigger();
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_meet();  // the peer's MMAs have read this CTA's operands
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, kLcTmemCols);
  }
}

// lse and loss of a row per warp from the half tiles' (reference, sum), joined
// in a fixed order.
constexpr int kLcRowsCta = 4;

// log 2 as a value of 11 significant bits (exact products with whole references below 2^13) and the rest
constexpr float kLn2Hi = 0.693359375f, kLn2Lo = -2.12194440e-4f;

__device__ __forceinline__ float2 lc_join(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return make_float2(m, a.y * tc::ex2_ftz(a.x - m) + b.y * tc::ex2_ftz(b.x - m));
}

__global__ void __launch_bounds__(32 * kLcRowsCta)
    k_lce_rows(const float2* __restrict__ part, const float* __restrict__ zt, const int32_t* __restrict__ target,
               int N, int parts, int V, float* __restrict__ loss, float* __restrict__ lse) {
  const int lane = threadIdx.x & 31, row = blockIdx.x * kLcRowsCta + (threadIdx.x >> 5);
  pdl_wait();
  pdl_trigger();
  if (row >= N) return;
  // two partials per load (parts is even)
  const float4* p = reinterpret_cast<const float4*>(part + (int64_t)row * parts);
  const float2 none = make_float2(kLcRefMin, 0.f);
  float2 a[4] = {none, none, none, none};
  for (int i = lane; i < parts / 2; i += 128) {
    float4 x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = i + 32 * k < parts / 2 ? p[i + 32 * k] : make_float4(kLcRefMin, 0.f, kLcRefMin, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = lc_join(a[k], lc_join(make_float2(x[k].x, x[k].y), make_float2(x[k].z, x[k].w)));
  }
  float2 x = lc_join(lc_join(a[0], a[1]), lc_join(a[2], a[3]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    float2 y;
    y.x = __shfl_xor_sync(0xFFFFFFFFu, x.x, o);
    y.y = __shfl_xor_sync(0xFFFFFFFFu, x.y, o);
    x = lc_join(x, y);
  }
  if (lane == 0) {
    // a row whose every logit is masked has no distribution: lse -inf, loss +inf
    const float v = x.y == 0.f ? -INFINITY : fmaf(x.x, kLn2Hi, fmaf(x.x, kLn2Lo, logf(x.y)));
    const int t = target[row];
    lse[row] = v;
    const float z = t < 0 || t >= V ? 0.f : zt[row];
    loss[row] = t < 0 || t >= V ? 0.f : v == -INFINITY || z <= kLcRefMin ? INFINITY : v - z;
  }
}

// Tiles that several pairs share: their parts (each already summed over the
// pieces of the vocabulary) added in the contraction's order.
struct LcJoin {
  const float* slots;
  int M, Nn, nkb, mt, nt, split;
  __nv_bfloat16* out;
  int64_t ldo;
  int t_out;
  float scale;
};
struct LcJoins {
  LcJoin j[2];
};

// a CTA takes 32 rows x 32 columns of a tile: a float4 per thread
constexpr int kLcJoinDim = 32;

__global__ void __launch_bounds__(256) k_lce_join(const __grid_constant__ LcJoins p) {
  __shared__ float sh[kLcJoinDim][kLcJoinDim + 1];
  pdl_wait();
  pdl_trigger();
  const LcJoin& j = p.j[blockIdx.z];
  int tile = blockIdx.x;
  if (tile >= j.mt * j.nt) return;
  const int units = j.mt * j.nt * j.nkb, u0 = tile * j.nkb, u1 = u0 + j.nkb;
  // the pairs that hold the tile's first and last block
  int pf = (int)((long long)u0 * j.split / units), pl = (int)((long long)(u1 - 1) * j.split / units);
  while (lc_share(units, j.split, pf + 1) <= u0) ++pf;
  while (lc_share(units, j.split, pl + 1) <= u1 - 1) ++pl;
  if (pf == pl) return;  // one pair held all of it and wrote it
  int g = 0, gm = j.mt;
  if (gm > 16) {
    g = tile / (16 * j.nt);
    gm = min(16, gm - g * 16);
    tile -= g * 16 * j.nt;
  }
  const int n = tile / gm, m = g * 16 + tile - n * gm;
  const int lr0 = (blockIdx.y >> 3) * kLcJoinDim, lc0 = (blockIdx.y & 7) * kLcJoinDim;
  const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 4;
  const int row0 = m * kLcTile + lr0, col0 = n * kLcTile + lc0;
  if (row0 >= j.M || col0 >= j.Nn) return;
  const int row = row0 + r, col = col0 + c;
  const bool has = row < j.M && col < j.Nn;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (has) {
    // the first pair's part began with the tile (an odd slot); the others' ranges begin inside it
    const float* sl = j.slots + ((int64_t)(2 * pf + 1) * kLcTile + lr0 + r) * kLcTile + lc0 + c;
    a = *reinterpret_cast<const float4*>(sl);
    sl += kLcTile * kLcTile;
#pragma unroll 8
    for (int q = pf + 1; q <= pl; ++q, sl += 2 * kLcTile * kLcTile) {
      const float4 x = *reinterpret_cast<const float4*>(sl);
      a.x += x.x;
      a.y += x.y;
      a.z += x.z;
      a.w += x.w;
    }
  }
  float f[4] = {a.x * j.scale, a.y * j.scale, a.z * j.scale, a.w * j.scale};
  int orow = row, ocol = col, oN = j.Nn;
  if (j.t_out) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sh[r][c + i] = f[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = sh[c + i][r];
    orow = col0 + r;
    ocol = row0 + c;
    oN = j.M;
    if (orow >= j.Nn) return;
  } else if (!has) {
    return;
  }
  __nv_bfloat16* o = j.out + (int64_t)orow * j.ldo + ocol;
  if (ocol + 4 <= oN) {
    uint2 x;
    x.x = pack_bf16(f[0], f[1]);
    x.y = pack_bf16(f[2], f[3]);
    *reinterpret_cast<uint2*>(o) = x;
  } else {
    for (int e = 0; ocol + e < oN; ++e) o[e] = __float2bfloat16_rn(f[e]);
  }
}

// XT[k][n] = X[n][k] for dW's product, zero for the rows that are left out (see
// lc_live_rows), rows of XT padded to a multiple of 8 (with zeros): 64 x 64 through
// shared memory, 16-byte pieces on both sides.
__global__ void __launch_bounds__(256)
    k_lce_transpose(const __nv_bfloat16* __restrict__ X, int64_t ldx, int N, int K, __nv_bfloat16* __restrict__ XT,
                    int64_t ldt, const int32_t* __restrict__ target, const float* __restrict__ lse, int V) {
  __shared__ __nv_bfloat16 sh[64][66];
  pdl_wait();
  pdl_trigger();
  const int k0 = blockIdx.x * 64, n0 = blockIdx.y * 64;
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int r = i >> 3, c = (i & 7) * 8, n = n0 + r, k = k0 + c;
    __align__(16) __nv_bfloat16 x[8];
    if (n < N && k + 8 <= K) {
      *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(X + n * ldx + k);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = n < N && k + e < K ? X[n * ldx + k + e] : __float2bfloat16_rn(0.f);
    }
    const bool live = n < N && lc_live(target, lse, V, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) sh[r][c + e] = live ? x[e] : __float2bfloat16_rn(0.f);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int r = i >> 3, c = (i & 7) * 8, k = k0 + r, n = n0 + c;
    if (k >= K || n >= N) continue;
    __align__(16) __nv_bfloat16 x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = sh[c + e][r];
    *reinterpret_cast<uint4*>(XT + k * ldt + n) = *reinterpret_cast<const uint4*>(x);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  return fn;
}

// A bf16 matrix of `rows` rows of `cols` values, `ld` apart; boxes 64 wide.
bool encode(CUtensorMap* tm, const void* p, int64_t cols, int64_t rows, int64_t ld, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// The epilogue's boxes of 32 rows: U (128 bytes of fp32, to shared memory), and
// stores of 64 bytes: bf16 results, fp32 sums and parts, or bf16 results turned
// (32 columns as they lie).
enum { kBoxU, kBox16, kBox32, kBoxTurned };
bool encode_box(CUtensorMap* tm, const void* p, int kind, int64_t cols, int64_t rows, int64_t ld) {
  const bool bf16 = kind == kBox16 || kind == kBoxTurned;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {kind == kBox32 ? 16u : 32u, 32};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                     const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     kind == kBoxU        ? CU_TENSOR_MAP_SWIZZLE_128B
                     : kind == kBoxTurned ? CU_TENSOR_MAP_SWIZZLE_NONE
                                          : CU_TENSOR_MAP_SWIZZLE_64B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int tiles_of(int64_t x) { return (int)((x + kLcTile - 1) / kLcTile); }

// Pairs that share a product's tiles block by block: where whole tiles would
// leave more than a quarter of the grid idle in at most two waves, every pair
// gets eight blocks, and the longest pair saves more blocks (a third of a
// microsecond each) than the join's launch costs. Whole tiles run side by side on
// the same stretch of the contraction and share its operands in L2, shares do
// not (1001 x 4100 x 50257, dX of 68 tiles of 786 blocks: the gradient took 813 us
// with shares and 535 with whole tiles). A function of the sizes alone, so the order of the sums does not depend on the device.
int split_of(int tiles, int nkb) {
  const int waves = (tiles + kLcPairs - 1) / kLcPairs;
  if (waves > 2 || 4 * tiles >= 3 * waves * kLcPairs) return 0;
  const int64_t most = (int64_t)tiles * nkb / 8;
  const int s = (int)(most < kLcPairs ? most : kLcPairs);
  return s > tiles && waves * nkb - (int)(((int64_t)tiles * nkb + s - 1) / s) > 12 ? s : 0;
}

// Columns of a tile of logits: narrower where whole tiles would occupy half of
// the pairs or fewer. A short contraction's time is mostly the epilogue's latency
// (6 x 80 x 1024: step 22.1 -> 20.1 us), a long one's the operands', of which the
// ring then holds more stages (234 x 5036 x 846 with U, 4 tiles: gradient of X 58 ->
// 48 us, with 12 us around it).
int z_cols(int64_t N, int64_t cols) {
  const int t = tiles_of(N) * tiles_of(cols);
  return 2 * t > kLcPairs ? kLcTile : 4 * t > kLcPairs ? kLcTile / 2 : kLcTile / 4;
}

// A whole tile's time in blocks: an MN-major B (see make_plan), its start and end.
double tile_cost(int nkb, bool b_mn) { return nkb * (b_mn ? 1.38 : 1.0) + 2.0; }

// The gradient's pieces of the vocabulary and its scratch.
struct LcPlan {
  int piece, pieces;
  int64_t ldg;
  int dx_split, dw_split, dx_nkb;
  int dx_split_dw;  // dX's beside dW
  int64_t dx_lda;
  bool swap;    // the operand whose contraction index is its row goes to A (see make_plan)
  int64_t ldt;  // of X's transpose, or of its copy
  size_t part, zt, fwd_total;                              // forward
  size_t G[2], dx_acc, dx_slots, dw_slots, XT, bwd_total;  // gradient
};

// G's piece: 64 MiB, which stay in L2, where the products are short (K below
// 1024: its 6 bytes of traffic a value take as long as 6 K operations at K = 265),
// else few launches. At least 64 tiles wide where a GiB allows, for long batches at the
// price of L2: narrower pieces
// have too few tiles of dW (K = 256, V = 129280: N = 4096 976 us in pieces of 32
// tiles, 736 of 64; N = 16384 3.94 ms of 8, 2.84 of 64, 2.71 of 128).
constexpr int64_t kLcPieceBytes = 256ll << 20, kLcPieceBytesL2 = 64ll << 20, kLcPieceMost = 1ll << 30;
constexpr int64_t kLcPieceCols = 64 * kLcTile;

// Up to 64 rows of X, the logits' product is made with W's tokens as its 256 rows
// and X's rows as at most 64 columns: rows of X would fill a quarter of the product
// at most, and be what bounds it (6 x 2321 x 141668 with U: forward 193 -> 134 us,
// gradient 534 -> 446; 1 x 256 x 129280 with U and W [K][V] 37.5 -> 29.3 and 69 -> 61,
// all with 12 us around them). The epilogue turns 32 x 32 logits in shared memory and
// goes on as with rows; each warp keeps its running sums to the end. Few tokens
// (7 x 210 x 2676) are 2 us slower that way.
bool z_turned(const dspark_lce_dims& d) { return d.N <= 64 && tiles_of(d.V) >= 16; }

// Sums a row that the statistics leave.
int z_parts(const dspark_lce_dims& d) {
  const int tiles = tiles_of(d.V);
  if (z_turned(d)) return kLcTurnedParts * (tiles < kLcPairs ? tiles : kLcPairs);
  const int n = z_cols(d.N, d.V);
  return 2 * ((d.V + n - 1) / n);
}

LcPlan make_plan(const dspark_lce_dims& d) {
  LcPlan p;
  memset(&p, 0, sizeof(p));
  const int64_t N = d.N, V = d.V, K = d.K;
  size_t off = 0;
  auto carve = [&](int64_t bytes) {
    const size_t o = off;
    off += (size_t)up(bytes > 0 ? bytes : 1, 256);
    return o;
  };
  p.part = carve(8 * N * z_parts(d));
  p.zt = carve(4 * N);
  p.fwd_total = off;
  const int64_t row = 2 * (N > 0 ? N : 1), wide = kLcPieceMost / row < kLcPieceCols ? kLcPieceMost / row : kLcPieceCols;
  int64_t most = (K < 1024 ? kLcPieceBytesL2 : kLcPieceBytes) / row;
  most = (most < wide ? wide : most) / kLcTile * kLcTile;
  most = most < 2048 ? 2048 : most;
  p.pieces = (int)((V + most - 1) / most);
  p.piece = (int)up((V + p.pieces - 1) / p.pieces, kLcTile);
  p.pieces = (int)((V + p.piece - 1) / p.piece);
  const int64_t widest = p.piece < V ? p.piece : V;
  p.ldg = up(widest, 64);
  const int64_t nkb_v = (widest + kLcKb - 1) / kLcKb, nkb_n = (N + kLcKb - 1) / kLcKb;
  p.dx_nkb = (int)nkb_v;
  p.dx_split = split_of(tiles_of(N) * tiles_of(K), (int)nkb_v);
  p.dw_split = split_of(tiles_of(widest) * tiles_of(K), (int)nkb_n);
  // Beside whole tiles of dW, dX goes to as many pairs as its part of the work
  // (those take whole tiles later): each pair more writes another 256 KB of sums
  // a piece. 640 x 256 x 129280 without U: all 76 pairs 167 us, 38 pairs 156;
  // 640 x 256 x 43093 with U 100 and 88, 100 x 512 x 129280 133 and 114. (64 x 4096 x
  // 129280, bound by W's way from HBM, loses 3%.)
  p.dx_split_dw = p.dx_split;
  if (p.dx_split > 0 && p.dw_split == 0) {
    const int tiles = tiles_of(N) * tiles_of(K);
    const double x = (double)tiles * nkb_v, w = (double)tiles_of(widest) * tiles_of(K) * tile_cost((int)nkb_n, false);
    const int s = (int)(kLcPairs * x / (x + w) + 0.5);
    p.dx_split_dw = s <= tiles ? tiles + 1 : s < p.dx_split ? s : p.dx_split;
  }
  // An MN-major B (its contraction index is its row) costs the tensor cores
  // 1.38x the time of a K-major one, an MN-major A nothing (256 x 256 tiles,
  // contraction 5376: 885 against 640 cycles a block). So where the products are
  // long, dX with W [V][K] is made transposed (A = W, B = G) and turned in its
  // epilogue, and dW takes X's transpose, made once, as B. Where they are short
  // the extra launch costs more than it saves (N K V = 2e10: 10 us saved, 3 spent): dW
  // takes a copy of X that the first launch makes.
  p.swap = (double)N * K * V >= 1e10;
  p.ldt = up(p.swap ? N : K, 8);
  p.dx_lda = p.swap && d.layout == DSPARK_W_VK ? up(N, 32) : up(K, 32);
  off = 0;
  p.G[0] = carve(2 * N * p.ldg);
  p.G[1] = p.pieces > 1 ? carve(2 * N * p.ldg) : p.G[0];
  p.dx_acc = carve(p.pieces > 1 ? 4 * p.dx_lda * (p.swap && d.layout == DSPARK_W_VK ? K : N) : 0);
  p.XT = carve(2 * (p.swap ? K : N) * p.ldt);
  p.dx_slots = carve(4ll * 2 * p.dx_split * kLcTile * kLcTile);
  p.dw_slots = carve(4ll * 2 * p.dw_split * kLcTile * kLcTile);
  p.bwd_total = off;
  return p;
}

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool dims_ok(const dspark_lce_dims* d) {
  if (!d || d->N < 0 || d->N > (1 << 20) || d->K < 1 || d->K > 65536 || d->V < 1 || d->V > (1 << 24)) return false;
  return d->layout == DSPARK_W_VK || d->layout == DSPARK_W_KV;
}
// leading dimension of a matrix of `cols` columns: long enough, rows 16-byte aligned
bool ld_ok(int64_t ld, int64_t cols, int mult) { return ld >= cols && ld % mult == 0 && ld < ((int64_t)1 << 32); }

cudaError_t lce_configure() {
  static std::atomic<uint64_t> done{0};
  return once_per_device(done, [] {
    cudaError_t e = cudaSuccess;
    for (const auto k : {k_lce<false, false>, k_lce<false, true>, k_lce<true, false>, k_lce<true, true>})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLcSmem);
    return e;
  });
}

// One launch: the statistics, or up to three of the gradient's products (the
// longest tiles first).
struct LcLaunch {
  LcParams p;
  bool grad, any;
  LcLaunch(bool grad, int* status) : grad(grad), any(false) {
    memset(&p, 0, sizeof(p));
    p.status = status;
  }
  LcJob& add(int place) {
    any = true;
    return p.job[place];
  }
  cudaError_t run(cudaStream_t st) {
    if (!any) return cudaSuccess;
    cudaError_t e = lce_configure();
    if (e != cudaSuccess) return e;
    int pairs = 0, tiles = 0;
    bool u = false, turned = false;
    for (int k = 0; k < kLcJobs; ++k) {
      LcJob& j = p.job[k];
      j.mt = tiles_of(j.M);
      if (j.tn == 0) j.tn = kLcTile;
      j.nt = (j.Nn + j.tn - 1) / j.tn;
      if (j.split == 0) tiles += j.mt * j.nt;
      p.tiles[k] = tiles;
      pairs = pairs > j.split ? pairs : j.split;
      const int b_bytes = j.b_mn ? (j.tn / 2 + 63) / 64 * kLcBox : j.tn * kLcKb;
      if (j.mt > 0 && p.stage_bytes < kLcOpBytes + b_bytes) p.stage_bytes = kLcOpBytes + b_bytes;
      turned = turned || j.turned;
      u = u || j.has_u || j.turned;  // boxes
    }
    p.stages = lc_stages(grad, u, p.stage_bytes);
    // dX's shares and the others' whole tiles on pairs of their own (gradient of 706 x
    // 1038 x 1415: 38.5 -> 32.4 us; of 100 x 1024 x 3000 30.3 -> 32.4)
    const LcJob& x = p.job[kLcDx];
    const bool apart = x.split > 0 && p.job[kLcDw].split == 0;
    pairs = pairs > tiles ? pairs : tiles;
    if (p.xc) {  // X's copy: up to four pieces a lane, on pairs without tiles too
      const int64_t lanes = 2 * kLcEpiWarps * 32, need = ((int64_t)p.N * (p.ldc / 8) + 4 * lanes - 1) / (4 * lanes);
      pairs = pairs > need ? pairs : (int)(need < kLcPairs ? need : kLcPairs);
    }
    if (apart && pairs < x.split + tiles) pairs = x.split + tiles;
    pairs = pairs < kLcPairs ? pairs : kLcPairs;
    // rounds of whole tiles that the other pairs do during one of dX's shares
    if (apart && x.split < pairs) {
      const int others = pairs - x.split;
      double left = (double)x.mt * x.nt * x.nkb / x.split;
      p.sharing = x.split;
      for (int t = 0; t < tiles; t += others, ++p.rounds) {
        const LcJob& j = p.job[t < p.tiles[kLcDw] ? kLcDw : kLcMakeG];
        const double cost = tile_cost(j.nkb, j.b_mn);
        if (left < 0.5 * cost) break;
        left -= cost;
      }
    }
    e = launch_ex(grad ? (turned ? k_lce<true, true> : k_lce<true, false>)
                       : (turned ? k_lce<false, true> : k_lce<false, false>), dim3(2 * pairs), dim3(kLcThreads), kLcSmem, st, true, p);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
};

// The tensor cores' fp32 accumulator is cut, not rounded, once per 16 terms: on
// average by half a unit, 0.36 * 2^-23 of the partial sum (half the mean of 1/m
// over significands m in [1, 2), 1 / (4 log 2)). The partial sums of a logit that
// matters grow evenly towards it, so over n steps it loses 0.36 * 2^-23
// (n + 1) / 2 of itself; the gain puts that back. A logit whose terms all come last
// is then off by as much the other way. Measured on random rows (z of deviation 2,
// V = 8192), in the mean: lse 5.9e-6 too high at K = 4096 where the gain raises it by
// 2.2e-5, 2.2e-5 of 8.8e-5 at 16384; with all terms last 5.8e-5 at 4096.
float logit_gain(int K) { return (float)(1.0 + 0.36 * 0x1p-23 * (K / 16.0 + 1.0) / 2.0); }

// z of the columns [v0, v0 + cols) of the vocabulary (statistics or G)
bool z_job(LcJob& j, const dspark_lce_dims* d, const void* X, const void* W, const float* U, const int32_t* target,
           int v0, int cols) {
  j.turned = z_turned(*d);
  j.M = j.turned ? cols : d->N;
  j.Nn = j.turned ? d->N : cols;
  j.nkb = (d->K + kLcKb - 1) / kLcKb;
  (j.turned ? j.a_mn : j.b_mn) = d->layout == DSPARK_W_KV;
  (j.turned ? j.a_m0 : j.b_n0) = v0;
  j.u = U;
  j.ldu = d->ldu;
  j.has_u = U != nullptr;
  j.target = target;
  j.V = d->V;
  j.gain = logit_gain(d->K);
  j.tn = j.turned ? kLcTile / 4 : z_cols(d->N, cols);
  if (U && !encode_box(&j.tu, U, kBoxU, d->V, d->N, d->ldu)) return false;
  const int w_rows = j.turned ? kLcHalf : j.tn / 2;  // of a box of W [V][K]
  return encode(j.turned ? &j.tb : &j.ta, X, d->K, d->N, d->ldx, j.turned ? j.tn / 2 : kLcHalf) &&
         (d->layout == DSPARK_W_VK ? encode(j.turned ? &j.ta : &j.tb, W, d->K, d->V, d->ldw, w_rows)
                                   : encode(j.turned ? &j.ta : &j.tb, W, d->V, d->K, d->ldw, kLcKb));
}

// Where a gradient's product goes: parts of shared tiles to slots, whole tiles
// to acc (summed over the vocabulary's pieces) or, complete, to out.
bool out_job(LcJob& j, LcJoin& q, float* slots, float* acc, int64_t lda, bool acc_in, bool to_out,
             __nv_bfloat16* out, int64_t ldo, bool t_out, float scale) {
  j.acc = acc;
  j.lda = lda;
  j.acc_in = acc_in;
  j.to_out = to_out;
  j.t_out = t_out;
  j.out = out;
  j.ldo = ldo;
  j.scale = scale;
  q.slots = slots;
  q.M = j.M;
  q.Nn = j.Nn;
  q.nkb = j.nkb;
  q.mt = tiles_of(j.M);
  q.nt = tiles_of(j.Nn);
  q.split = j.split;
  q.out = out;
  q.ldo = ldo;
  q.t_out = t_out;
  q.scale = scale;
  if (j.split && !encode_box(&j.tslots, slots, kBox32, kLcTile, 2ll * j.split * kLcTile, kLcTile)) return false;
  if (!to_out) return encode_box(&j.tacc, acc, kBox32, lda, j.M, lda);
  return t_out ? encode_box(&j.to, out, kBoxTurned, j.M, j.Nn, ldo) : encode_box(&j.to, out, kBox16, j.Nn, j.M, ldo);
}

dspark_status lce_fail(cudaError_t e) {
  if (e == cudaSuccess) return DSPARK_OK;
  fprintf(stderr, "dspark: CUDA error %s\n", cudaGetErrorString(e));
  return DSPARK_ECUDA;
}

dspark_status check_inputs(const dspark_lce_dims* d, const void* X, const void* W, const float* U,
                           const int32_t* target, const void* scratch, const int32_t* device_status) {
  if (!dims_ok(d) || !device_status || !aligned16(W)) return DSPARK_EINVAL;
  if (d->N > 0 && (!aligned16(X) || !aligned16(target))) return DSPARK_EINVAL;
  if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u) != 0) return DSPARK_EINVAL;
  if (!ld_ok(d->ldx, d->K, 8) || !ld_ok(d->ldw, d->layout == DSPARK_W_VK ? d->K : d->V, 8)) return DSPARK_EINVAL;
  if (U && (!aligned16(U) || !ld_ok(d->ldu, d->V, 4))) return DSPARK_EINVAL;
  return DSPARK_OK;
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_linear_ce_scratch_bytes(const dspark_lce_dims* d) {
  if (!dims_ok(d)) return 0;
  const LcPlan p = make_plan(*d);
  return p.fwd_total > p.bwd_total ? p.fwd_total : p.bwd_total;
}

extern "C" dspark_status dspark_linear_ce(const dspark_lce_dims* d, const void* X, const void* W, const float* U,
                                          const int32_t* target, float* loss, float* lse, void* scratch,
                                          int32_t* device_status, dspark_stream_t stream) {
  const dspark_status bad = check_inputs(d, X, W, U, target, scratch, device_status);
  if (bad != DSPARK_OK) return bad;
  if (d->N > 0 && (!aligned16(loss) || !aligned16(lse))) return DSPARK_EINVAL;
  if (!encode_fn()) return DSPARK_ECUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d->N == 0) return DSPARK_OK;
  const LcPlan p = make_plan(*d);
  char* base = static_cast<char*>(scratch);
  float2* part = reinterpret_cast<float2*>(base + p.part);
  float* zt = reinterpret_cast<float*>(base + p.zt);
  LcLaunch l(false, device_status);
  LcJob& j = l.add(0);
  if (!z_job(j, d, X, W, U, target, 0, d->V)) return DSPARK_EINVAL;
  j.part = part;
  j.zt = zt;
  cudaError_t e = l.run(st);
  if (e == cudaSuccess)
    e = launch_ex(k_lce_rows, dim3((d->N + kLcRowsCta - 1) / kLcRowsCta), dim3(32 * kLcRowsCta), 0, st,
                  true, part, zt, target, d->N, z_parts(*d),
                  d->V, loss, lse);
  return lce_fail(e);
}

extern "C" dspark_status dspark_linear_ce_grad(const dspark_lce_dims* d, const void* X, const void* W, const float* U,
                                               const int32_t* target, const float* lse, const float* wt, float scale,
                                               void* dX, void* dW, void* scratch, int32_t* device_status,
                                               dspark_stream_t stream) {
  const dspark_status bad = check_inputs(d, X, W, U, target, scratch, device_status);
  if (bad != DSPARK_OK) return bad;
  const bool vk = d->layout == DSPARK_W_VK;
  if (d->N > 0 && (!aligned16(lse) || (wt && !aligned16(wt)))) return DSPARK_EINVAL;
  if (!dX && !dW && d->N > 0) return DSPARK_EINVAL;  // without rows dX is empty, and may have no address
  if (dX && (!aligned16(dX) || !ld_ok(d->lddx, d->K, 8))) return DSPARK_EINVAL;
  if (dW && (!aligned16(dW) || !ld_ok(d->lddw, vk ? d->K : d->V, 8))) return DSPARK_EINVAL;
  if (!encode_fn()) return DSPARK_ECUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (d->N == 0) {  // no rows: dW is zero
    if (dW)
      e = cudaMemset2DAsync(dW, (size_t)d->lddw * 2, 0, (size_t)(vk ? d->K : d->V) * 2, (size_t)(vk ? d->V : d->K), st);
    return lce_fail(e);
  }
  const LcPlan p = make_plan(*d);
  char* base = static_cast<char*>(scratch);
  if (dW && p.swap)
    e = launch_ex(k_lce_transpose, dim3((d->K + 63) / 64, (d->N + 63) / 64), dim3(256), 0, st, true,
                  static_cast<const __nv_bfloat16*>(X), d->ldx, d->N, d->K, reinterpret_cast<__nv_bfloat16*>(base + p.XT),
                  p.ldt, target, lse, d->V);
  // launch i makes G of piece i beside the gradients' products of piece i - 1
  for (int i = 0; i <= p.pieces && e == cudaSuccess; ++i) {
    LcLaunch l(true, device_status);
    LcJoins joins;
    int njoin = 0, join_tiles = 0;
    if (i > 0) {
      const int v0 = (i - 1) * p.piece, cols = d->V - v0 < p.piece ? d->V - v0 : p.piece;
      const __nv_bfloat16* G = reinterpret_cast<const __nv_bfloat16*>(base + p.G[(i - 1) & 1]);
      if (dX) {
        LcJob& x = l.add(kLcDx);
        const bool t = p.swap && vk;  // dX^T = W^T G^T
        x.M = t ? d->K : d->N;
        x.Nn = t ? d->N : d->K;
        x.nkb = p.dx_nkb;  // every piece's (a narrower last piece reads zeros), so that slots keep their tiles
        x.split = dW ? p.dx_split_dw : p.dx_split;
        if (!out_job(x, joins.j[njoin], reinterpret_cast<float*>(base + p.dx_slots),
                     reinterpret_cast<float*>(base + p.dx_acc), p.dx_lda, i > 1, i == p.pieces,
                     static_cast<__nv_bfloat16*>(dX), d->lddx, t, scale))
          return DSPARK_EINVAL;
        bool ok;
        if (t) {
          x.a_mn = 1;
          ok = encode(&x.ta, static_cast<const __nv_bfloat16*>(W) + (int64_t)v0 * d->ldw, d->K, cols, d->ldw, kLcKb) &&
               encode(&x.tb, G, cols, d->N, p.ldg, kLcHalf);
        } else {
          x.b_mn = vk;
          x.b_k0 = v0;
          ok = encode(&x.ta, G, cols, d->N, p.ldg, kLcHalf) &&
               (vk ? encode(&x.tb, W, d->K, d->V, d->ldw, kLcKb) : encode(&x.tb, W, d->V, d->K, d->ldw, kLcHalf));
        }
        if (!ok) return DSPARK_EINVAL;
        if (x.split && i == p.pieces) {
          ++njoin;
          join_tiles = tiles_of(x.M) * tiles_of(x.Nn);
        }
      }
      if (dW) {
        LcJob& w = l.add(kLcDw);
        const bool rows_v = vk || p.swap;  // the product's rows are tokens (W [K][V]: written transposed)
        w.M = rows_v ? cols : d->K;
        w.Nn = rows_v ? d->K : cols;
        w.nkb = (d->N + kLcKb - 1) / kLcKb;
        // a last piece of fewer tiles than the others shares them only if the others do (its slots are theirs)
        w.split = p.dw_split ? split_of(tiles_of(w.M) * tiles_of(w.Nn), w.nkb) : 0;
        if (!out_job(w, joins.j[njoin], reinterpret_cast<float*>(base + p.dw_slots), nullptr, 0, false, true,
                     static_cast<__nv_bfloat16*>(dW) + (vk ? (int64_t)v0 * d->lddw : v0), d->lddw, rows_v && !vk,
                     scale))
          return DSPARK_EINVAL;
        w.a_mn = 1;
        w.b_mn = !p.swap;
        CUtensorMap* tg = rows_v ? &w.ta : &w.tb;
        CUtensorMap* tx = rows_v ? &w.tb : &w.ta;
        if (!encode(tg, G, cols, d->N, p.ldg, kLcKb) ||
            !(p.swap ? encode(tx, base + p.XT, d->N, d->K, p.ldt, kLcHalf)
                     : encode(tx, base + p.XT, d->K, d->N, p.ldt, kLcKb)))
          return DSPARK_EINVAL;
        if (w.split) {
          ++njoin;
          const int n = tiles_of(w.M) * tiles_of(w.Nn);
          join_tiles = join_tiles > n ? join_tiles : n;
        }
      }
    }
    if (i < p.pieces) {
      const int v0 = i * p.piece, cols = d->V - v0 < p.piece ? d->V - v0 : p.piece;
      LcJob& g = l.add(kLcMakeG);
      if (!z_job(g, d, X, W, U, target, v0, cols)) return DSPARK_EINVAL;
      g.lse = lse;
      g.wt = wt;
      if (!encode_box(&g.to, base + p.G[i & 1], kBox16, cols, d->N, p.ldg)) return DSPARK_EINVAL;
      if (i == 0 && dW && !p.swap) {
        l.p.x = static_cast<const __nv_bfloat16*>(X);
        l.p.xc = reinterpret_cast<__nv_bfloat16*>(base + p.XT);
        l.p.ldx = d->ldx;
        l.p.ldc = p.ldt;
        l.p.N = d->N;
        l.p.K = d->K;
      }
    }
    e = l.run(st);
    if (njoin > 0 && e == cudaSuccess)
      e = launch_ex(k_lce_join, dim3(join_tiles, (kLcTile / kLcJoinDim) * (kLcTile / kLcJoinDim), njoin), dim3(256), 0,
                    st, true, joins);
  }
  return lce_fail(e);
}
