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
// per CTA), TMA into a six-stage ring, two accumulators so that the epilogue
// of a tile runs under the next tile's products. An operand whose contraction
// index is its row (W in dX, G and X in dW) is read in place as an MN-major
// operand; nothing is transposed in memory.
//
//   warp 0      TMA producer (both CTAs; bytes counted on the even CTA)
//   warp 1      allocates TMEM; in the even CTA issues the MMAs of the pair
//   warps 2-9   epilogue: a TMEM lane quarter and half of the tile's columns
// Every wait is bounded; a timeout sets DSPARK_ETIMEOUT and every role ends.
#include <cudaTypedefs.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

constexpr int kLcTile = 256;     // rows and columns of a pair's tile
constexpr int kLcHalf = 128;     // rows (A) and columns (B) one CTA loads
constexpr int kLcKb = 64;        // contraction depth of a stage (one 128-byte swizzled row)
constexpr int kLcStages = 6;
constexpr int kLcOpBytes = kLcHalf * kLcKb * 2;   // 16 KB: one operand's half of a stage
constexpr int kLcStageBytes = 2 * kLcOpBytes;
constexpr int kLcBox = 64 * kLcKb * 2;            // 8 KB: a 64 x 64 box of an MN-major operand
constexpr int kLcEpiWarps = 8;
constexpr int kLcThreads = 32 * (2 + kLcEpiWarps);
constexpr int kLcTmemCols = 512;                  // two accumulators of 256 columns
constexpr size_t kLcSmem = (size_t)kLcStages * kLcStageBytes + 1024 + 256;
constexpr int kLcPairs = 76;                      // CTA pairs of a full grid (152 SMs)

constexpr float kLcMasked = -1e30f;

enum : int { kLcStats = 0, kLcG = 1, kLcOut = 2 };

// One product C[M][Nn] = A B^T over a contraction of nkb blocks of 64.
struct LcJob {
  CUtensorMap ta, tb;
  int mode;
  int M, Nn;            // rows and columns of the result
  int nkb;              // contraction blocks in all
  int slices, per;      // contraction slices and the blocks of each
  int mt, nt;           // tiles of 256 rows, of 256 columns
  int a_mn, b_mn;       // operand's contraction index is its row (MN-major)
  int a_k0, b_k0;       // contraction offset in the operand's map
  int b_n0;             // column offset in B's map (and of U)
  // kLcStats, kLcG
  const float* U;
  int64_t ldu;
  const int32_t* target;
  const float* lse;
  const float* wt;
  float2* part;         // [2 nt][M] (max, sum exp) per half tile
  float* zt;            // [M] z at the target
  __nv_bfloat16* G;     // [M][ldg] the piece's G
  int64_t ldg;
  int V;                // vocabulary
  // kLcOut
  float* acc;           // [slices][M][lda] fp32 partial results, or null
  int64_t lda;
  int acc_in;           // add what acc holds
  __nv_bfloat16* out;   // [M][ldo] the result, or null: acc is written
  int64_t ldo;
  float scale;
};

struct LcParams {
  LcJob job;
  int tiles;
  int* status;
};

__device__ __forceinline__ void st_v8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Tile index -> (row tile, column tile, slice): slices outermost, then column
// tiles, with up to 16 row tiles innermost, so that the tiles in flight share
// their columns' operand in L2.
__device__ __forceinline__ void lc_tile(const LcJob& j, int t, int& m, int& n, int& s) {
  const int per = j.mt * j.nt;
  s = t / per;
  t -= s * per;
  const int g = t / (16 * j.nt), gm = min(16, j.mt - g * 16);
  t -= g * 16 * j.nt;
  n = t / gm;
  m = g * 16 + t - n * gm;
}

// columns of B the MMA takes for a tile: a multiple of 32
__device__ __forceinline__ int lc_cols(const LcJob& j, int n) {
  return min(kLcTile, (j.Nn - n * kLcTile + 31) & ~31);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLcThreads, 1)
    k_lce(const __grid_constant__ LcParams p) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = tc::smem_u32(smem);
  const uint32_t bars = sbase + kLcStages * kLcStageBytes;
  auto full = [&](int s) { return bars + 8u * s; };
  auto empty = [&](int s) { return bars + 8u * (kLcStages + s); };
  auto tfull = [&](int b) { return bars + 8u * (2 * kLcStages + b); };
  auto tempty = [&](int b) { return bars + 8u * (2 * kLcStages + 2 + b); };
  const uint32_t drain = bars + 8u * (2 * kLcStages + 4);
  unsigned char* tail = smem + kLcStages * kLcStageBytes + 8 * (2 * kLcStages + 5);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tail);
  volatile int* abort = reinterpret_cast<volatile int*>(tail + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const LcJob& j = p.job;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kLcStages; ++s) {
      tc::mbar_init(full(s), 1);
      tc::mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tfull(b), 1);
      tc::mbar_init(tempty(b), 2 * kLcEpiWarps);  // both CTAs' epilogue warps, on the even CTA
    }
    tc::mbar_init(drain, 1);
    *abort = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&j.ta);
    tc::prefetch_tmap(&j.tb);
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tc::smem_u32(tmem_holder), kLcTmemCols);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();
  tc::tc_fence_after();
  const uint32_t tmem = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      int iss = 0;
      bool ok = true;
      for (int t = pair; t < p.tiles && ok; t += npairs) {
        int m, n, sl;
        lc_tile(j, t, m, n, sl);
        const int half = lc_cols(j, n) >> 1;  // columns of B in each CTA
        const int am = m * kLcTile + (int)rank * kLcHalf, bn = j.b_n0 + n * kLcTile + (int)rank * half;
        const int kb0 = sl * j.per, kb1 = min(j.nkb, kb0 + j.per);
        const int bboxes = (half + 63) >> 6;  // boxes of an MN-major B
        const uint32_t bytes = (uint32_t)(kLcOpBytes + (j.b_mn ? bboxes * kLcBox : kLcOpBytes));
        for (int kb = kb0; kb < kb1; ++kb, ++iss) {
          const int s = iss % kLcStages;
          ok = tc::mbar_wait(empty(s), ((iss / kLcStages) & 1) ^ 1, abort);
          if (!ok) break;
          const uint32_t bar = tc::map_rank(full(s), 0);
          if (rank == 0) tc::mbar_arrive_expect_tx(full(s), 2 * bytes);  // both CTAs' copies
          const uint32_t da = sbase + s * kLcStageBytes, db = da + kLcOpBytes;
          const int ka = j.a_k0 + kb * kLcKb, kbn = j.b_k0 + kb * kLcKb;
          if (j.a_mn) {
            tc::tma_load_2d_pair(da, &j.ta, am, ka, bar);
            tc::tma_load_2d_pair(da + kLcBox, &j.ta, am + 64, ka, bar);
          } else {
            tc::tma_load_2d_pair(da, &j.ta, ka, am, bar);
          }
          if (j.b_mn) {
            for (int b = 0; b < bboxes; ++b) tc::tma_load_2d_pair(db + b * kLcBox, &j.tb, bn + b * 64, kbn, bar);
          } else {
            tc::tma_load_2d_pair(db, &j.tb, kbn, bn, bar);
          }
        }
      }
      // the last stages' releases, which the even CTA's MMAs send to both CTAs, have arrived before either exits
      for (int i = max(0, iss - kLcStages); i < iss && ok; ++i)
        ok = tc::mbar_wait(empty(i % kLcStages), (i / kLcStages) & 1, abort);
      if (!ok) {
        if (!*abort) raise_status(p.status, DSPARK_ETIMEOUT);
        *abort = 1;
        // copies already issued land (they complete on the even CTA's barriers) before the pair can exit
        volatile int never = 0;
        for (int i = max(0, iss - kLcStages); i < iss; ++i)
          tc::mbar_wait(full(i % kLcStages), (i / kLcStages) & 1, &never);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && rank == 0) {
      bool ok = true;
      int it = 0, tj = 0;
      for (int t = pair; t < p.tiles && ok; t += npairs, ++tj) {
        int m, n, sl;
        lc_tile(j, t, m, n, sl);
        const int cols = lc_cols(j, n), kb0 = sl * j.per, kb1 = min(j.nkb, kb0 + j.per);
        const uint32_t idesc = tc::idesc_bf16_f32(kLcTile, cols, j.b_mn) | (j.a_mn ? 1u << 15 : 0u);
        const int ab = tj & 1;
        ok = tc::mbar_wait(tempty(ab), ((tj >> 1) & 1) ^ 1, abort);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(ab * kLcTile);
        const uint32_t a_step = j.a_mn ? 2048 : 32, b_step = j.b_mn ? 2048 : 32;
        const uint32_t a_lbo = j.a_mn ? kLcBox : 16, b_lbo = j.b_mn ? kLcBox : 16;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % kLcStages;
          ok = tc::mbar_wait(full(s), (it / kLcStages) & 1, abort);
          if (!ok) break;
          tc::tc_fence_after();
          const uint32_t da = sbase + s * kLcStageBytes, db = da + kLcOpBytes;
#pragma unroll
          for (int kk = 0; kk < kLcKb / 16; ++kk)
            tc::mma_bf16_pair(d, tc::smem_desc(da + kk * a_step, a_lbo, 1024),
                              tc::smem_desc(db + kk * b_step, b_lbo, 1024), idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
          tc::mma_commit_pair(empty(s));
        }
        if (ok) tc::mma_commit_pair(tfull(ab));
      }
      if (!ok) {
        if (!*abort) raise_status(p.status, DSPARK_ETIMEOUT);
        *abort = 1;
      }
      tc::mma_commit_pair_own(drain);  // every MMA issued completes before TMEM and the peer's operands go
      volatile int never = 0;
      tc::mbar_wait(drain, 0, &never);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, hf = (warp - 2) >> 2;
    bool ok = true;
    int tj = 0;
    for (int t = pair; t < p.tiles; t += npairs, ++tj) {
      int m, n, sl;
      lc_tile(j, t, m, n, sl);
      const int cols = lc_cols(j, n), ab = tj & 1;
      const int row = m * kLcTile + (int)rank * kLcHalf + q * 32 + lane;
      const bool has = row < j.M;
      const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(ab * kLcTile);
      // this warp's columns of the tile: [c0, c1), in steps of 32
      const int c0 = hf * kLcHalf, c1 = min(cols, c0 + kLcHalf);
      const int col0 = n * kLcTile;
      int tgt = -1;
      float lse = 0.f, w = 0.f;
      if (j.mode != kLcOut && has) {
        tgt = j.target[row];
        if (tgt < -1 || tgt >= j.V) {
          if (n == 0 && hf == 0) raise_status(p.status, DSPARK_ERANGE);
          tgt = -1;
        }
        if (j.mode == kLcG) {
          lse = j.lse[row];
          w = j.wt ? j.wt[row] : 1.f;
        }
      }
      ok = tc::mbar_wait(tfull(ab), (tj >> 1) & 1, abort);
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (!ok) break;
      tc::tc_fence_after();
      const bool any = __any_sync(0xFFFFFFFFu, has);
      if (j.mode == kLcOut) {
        const int64_t o_row = (int64_t)sl * j.M + row;
        for (int c = c0; c < c1 && any; c += 32) {
          float v[32];
          tc::tmem_ld32(ta + (uint32_t)c, v);
          tc::tmem_wait_ld();
          if (!has) continue;
          const int col = col0 + c;
          float* ap = j.acc ? j.acc + o_row * j.lda + col : nullptr;
          if (j.acc_in) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 x = *reinterpret_cast<const float4*>(ap + e);
              v[e] += x.x;
              v[e + 1] += x.y;
              v[e + 2] += x.z;
              v[e + 3] += x.w;
            }
          }
          if (!j.out) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_v8(ap + e, reinterpret_cast<const uint32_t*>(v + e));
          } else {
            __nv_bfloat16* op = j.out + (int64_t)row * j.ldo + col;
            const int left = j.Nn - col;
            if (left >= 32) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint4 x;
                x.x = pack_bf16(v[e] * j.scale, v[e + 1] * j.scale);
                x.y = pack_bf16(v[e + 2] * j.scale, v[e + 3] * j.scale);
                x.z = pack_bf16(v[e + 4] * j.scale, v[e + 5] * j.scale);
                x.w = pack_bf16(v[e + 6] * j.scale, v[e + 7] * j.scale);
                *reinterpret_cast<uint4*>(op + e) = x;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e < left) op[e] = __float2bfloat16_rn(v[e] * j.scale);
            }
          }
        }
      } else {
        // a row's logits, 32 at a time: U added, columns past the vocabulary out
        float mx = -INFINITY, sum = 0.f;
        for (int c = c0; c < c1 && any; c += 32) {
          float v[32];
          tc::tmem_ld32(ta + (uint32_t)c, v);
          tc::tmem_wait_ld();
          const int col = j.b_n0 + col0 + c;  // vocabulary index of v[0]
          const int left = min(32, j.V - col);
          if (j.U && has) {
            const float* up = j.U + (int64_t)row * j.ldu + col;
            if (left == 32) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4*>(up + e));
                v[e] += x.x;
                v[e + 1] += x.y;
                v[e + 2] += x.z;
                v[e + 3] += x.w;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e < left) v[e] += up[e];
            }
            // a mask's finite stand-in (the type's lowest value) masks as -inf does:
            // a row that holds nothing else would lose its sum of exponentials to lse's rounding
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = v[e] <= kLcMasked ? -INFINITY : v[e];
          }
          const int te = tgt - col;  // the target's place among these columns
          if (j.mode == kLcStats) {
            if (left < 32) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e >= left) v[e] = -INFINITY;
            }
            if (te >= 0 && te < 32) {
              float z = 0.f;
#pragma unroll
              for (int e = 0; e < 32; ++e) z = e == te ? v[e] : z;
              j.zt[row] = z;
            }
            float cm = v[0];
#pragma unroll
            for (int e = 1; e < 31; e += 2) cm = tc::max3f(cm, v[e], v[e + 1]);
            cm = tc::max3f(cm, v[31], mx);
            // a row that is -inf so far keeps its sum at 0 (no -inf - -inf)
            const float ref = cm == -INFINITY ? 0.f : cm;
            sum *= tc::ex2_ftz((mx - ref) * tc::kLog2e);
            mx = cm;
            float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 32; ++e) s4[e & 3] += tc::ex2_ftz((v[e] - ref) * tc::kLog2e);
            sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
          } else {
            // G: a row without a target, or with nothing left by its mask, has none
            const bool live = tgt >= 0 && lse != -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float pv = tc::ex2_ftz((v[e] - lse) * tc::kLog2e);
              v[e] = live ? w * (e == te ? pv - 1.f : pv) : 0.f;
            }
            if (has) {
              // the piece's rows are padded to whole 32-column groups
              __nv_bfloat16* gp = j.G + (int64_t)row * j.ldg + col0 + c;
#pragma unroll
              for (int e = 0; e < 32; e += 16) {
                uint32_t r[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) r[i] = pack_bf16(v[e + 2 * i], v[e + 2 * i + 1]);
                st_v8(gp + e, r);
              }
            }
          }
        }
        if (j.mode == kLcStats && has) j.part[(int64_t)(2 * n + hf) * j.M + row] = make_float2(mx, sum);
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_cluster(tc::map_rank(tempty(ab), 0));
    }
    if (!ok && lane == 0) {
      if (!*abort) raise_status(p.status, DSPARK_ETIMEOUT);
      *abort = 1;
    }
  }
  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_sync();  // the peer's MMAs have read this CTA's operands; remote arrivals have landed
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc_pair(tmem, kLcTmemCols);
  }
}

// lse and loss of 32 rows per CTA from the half tiles' (max, sum exp): a
// warp-wide lane of partials per row, joined in a fixed order.
__global__ void __launch_bounds__(1024)
    k_lce_rows(const float2* __restrict__ part, const float* __restrict__ zt, const int32_t* __restrict__ target,
               int N, int parts, int V, float* __restrict__ loss, float* __restrict__ lse) {
  __shared__ float2 sh[32][33];
  const int r = threadIdx.x & 31, g = threadIdx.x >> 5, row = blockIdx.x * 32 + r;
  float m = -INFINITY, s = 0.f;
  if (row < N)
    for (int i = g; i < parts; i += 32) {
      const float2 x = part[(int64_t)i * N + row];
      const float nm = fmaxf(m, x.x), ref = nm == -INFINITY ? 0.f : nm;
      s = s * __expf(m - ref) + x.y * __expf(x.x - ref);
      m = nm;
    }
  sh[g][r] = make_float2(m, s);
  __syncthreads();
  if (g == 0 && row < N) {
    for (int i = 1; i < 32; ++i) {
      const float2 x = sh[i][r];
      const float nm = fmaxf(m, x.x), ref = nm == -INFINITY ? 0.f : nm;
      s = s * __expf(m - ref) + x.y * __expf(x.x - ref);
      m = nm;
    }
    // a row whose every logit is -inf has no distribution: lse -inf, loss +inf
    const float l = (m == -INFINITY && s == 0.f) ? -INFINITY : m + logf(s);
    const int t = target[row];
    lse[row] = l;
    loss[row] = (t < 0 || t >= V) ? 0.f : (l == -INFINITY ? INFINITY : l - zt[row]);
  }
}

// out[m][c] = bf16(scale * sum over slices of acc[s][m][c]), slices in order.
__global__ void __launch_bounds__(256)
    k_lce_join(const float* __restrict__ acc, int slices, int M, int Nn, int64_t lda, float scale,
               __nv_bfloat16* __restrict__ out, int64_t ldo) {
  const int q = (Nn + 3) >> 2;
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= (int64_t)M * q) return;
  const int m = (int)(i / q), c = (int)(i - (int64_t)m * q) * 4;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < slices; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(acc + ((int64_t)s * M + m) * lda + c);
    a.x += x.x;
    a.y += x.y;
    a.z += x.z;
    a.w += x.w;
  }
  __nv_bfloat16* o = out + (int64_t)m * ldo + c;
  if (c + 4 <= Nn) {
    uint2 x;
    x.x = pack_bf16(a.x * scale, a.y * scale);
    x.y = pack_bf16(a.z * scale, a.w * scale);
    *reinterpret_cast<uint2*>(o) = x;
  } else {
    const float v[4] = {a.x, a.y, a.z, a.w};
    for (int e = 0; c + e < Nn; ++e) o[e] = __float2bfloat16_rn(v[e] * scale);
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

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int tiles_of(int64_t x) { return (int)((x + kLcTile - 1) / kLcTile); }

// Slices of a contraction of nkb blocks so that `tiles` tiles fill the grid;
// a slice keeps at least eight blocks. A function of the sizes alone, so the
// order of the sums does not depend on the device.
void slice(int tiles, int nkb, int* slices, int* per) {
  int s = 1;
  if (tiles < kLcPairs) s = kLcPairs / tiles;
  s = s < nkb / 8 ? s : nkb / 8;
  s = s < 1 ? 1 : s;
  *per = (nkb + s - 1) / s;
  *slices = (nkb + *per - 1) / *per;
}

// The gradient's pieces of the vocabulary and its scratch.
struct LcPlan {
  int piece, pieces;
  int64_t ldg;
  int dx_slices, dx_per, dw_slices, dw_per;
  int64_t dx_lda, dw_lda;
  size_t part, zt, fwd_total;            // forward
  size_t G, dx_acc, dw_acc, bwd_total;   // gradient
};

constexpr int64_t kLcPieceBytes = 256ll << 20;

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
  p.part = carve(8 * N * 2 * tiles_of(V));
  p.zt = carve(4 * N);
  p.fwd_total = off;
  int64_t most = kLcPieceBytes / (2 * (N > 0 ? N : 1)) / kLcTile * kLcTile;
  most = most < 2048 ? 2048 : most;
  p.pieces = (int)((V + most - 1) / most);
  p.piece = (int)up((V + p.pieces - 1) / p.pieces, kLcTile);
  p.pieces = (int)((V + p.piece - 1) / p.piece);
  const int64_t widest = p.piece < V ? p.piece : V;
  p.ldg = up(widest, 64);
  const int64_t nkb_v = (widest + kLcKb - 1) / kLcKb, nkb_n = (N + kLcKb - 1) / kLcKb;
  slice(tiles_of(N) * tiles_of(K), (int)nkb_v, &p.dx_slices, &p.dx_per);
  slice(tiles_of(widest) * tiles_of(K), (int)nkb_n, &p.dw_slices, &p.dw_per);
  p.dx_lda = up(K, 32);
  p.dw_lda = d.layout == DSPARK_W_VK ? up(K, 32) : up(widest, 32);
  off = 0;
  p.G = carve(2 * N * p.ldg);
  p.dx_acc = carve(p.dx_slices > 1 || p.pieces > 1 ? 4 * p.dx_slices * N * p.dx_lda : 0);
  p.dw_acc = carve(p.dw_slices > 1 ? 4 * p.dw_slices * (d.layout == DSPARK_W_VK ? widest : K) * p.dw_lda : 0);
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

cudaError_t run_job(LcJob& j, int* status, cudaStream_t st) {
  static bool configured = false;
  if (!configured) {
    const cudaError_t e = cudaFuncSetAttribute(k_lce, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kLcSmem);
    if (e != cudaSuccess) return e;
    configured = true;
  }
  LcParams p;
  memset(&p, 0, sizeof(p));
  j.mt = tiles_of(j.M);
  j.nt = tiles_of(j.Nn);
  p.job = j;
  p.tiles = j.mt * j.nt * j.slices;
  p.status = status;
  const int pairs = p.tiles < kLcPairs ? p.tiles : kLcPairs;
  k_lce<<<2 * pairs, kLcThreads, kLcSmem, st>>>(p);
  return cudaGetLastError();
}

LcJob empty_job() {
  LcJob j;
  memset(&j, 0, sizeof(j));
  j.slices = 1;
  return j;
}

// z of the columns [v0, v0 + cols) of the vocabulary (statistics or G)
bool z_job(LcJob& j, const dspark_lce_dims* d, const void* X, const void* W, const float* U, const int32_t* target,
           int v0, int cols) {
  j.M = d->N;
  j.Nn = cols;
  j.nkb = (d->K + kLcKb - 1) / kLcKb;
  j.per = j.nkb;
  j.b_mn = d->layout == DSPARK_W_KV;
  j.b_n0 = v0;
  j.U = U;
  j.ldu = d->ldu;
  j.target = target;
  j.V = d->V;
  if (!encode(&j.ta, X, d->K, d->N, d->ldx, kLcHalf)) return false;
  return d->layout == DSPARK_W_VK ? encode(&j.tb, W, d->K, d->V, d->ldw, kLcHalf)
                                  : encode(&j.tb, W, d->V, d->K, d->ldw, kLcKb);
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
  LcJob j = empty_job();
  j.mode = kLcStats;
  if (!z_job(j, d, X, W, U, target, 0, d->V)) return DSPARK_EINVAL;
  j.part = part;
  j.zt = zt;
  cudaError_t e = run_job(j, device_status, st);
  if (e == cudaSuccess) {
    k_lce_rows<<<(d->N + 31) / 32, 1024, 0, st>>>(part, zt, target, d->N, 2 * tiles_of(d->V), d->V, loss, lse);
    e = cudaGetLastError();
  }
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
  if (!dX && !dW) return DSPARK_EINVAL;
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
  __nv_bfloat16* G = reinterpret_cast<__nv_bfloat16*>(base + p.G);
  float* dx_acc = reinterpret_cast<float*>(base + p.dx_acc);
  float* dw_acc = reinterpret_cast<float*>(base + p.dw_acc);
  for (int i = 0; i < p.pieces && e == cudaSuccess; ++i) {
    const int v0 = i * p.piece, cols = d->V - v0 < p.piece ? d->V - v0 : p.piece;
    LcJob g = empty_job();
    g.mode = kLcG;
    if (!z_job(g, d, X, W, U, target, v0, cols)) return DSPARK_EINVAL;
    g.lse = lse;
    g.wt = wt;
    g.G = G;
    g.ldg = p.ldg;
    e = run_job(g, device_status, st);
    if (dX && e == cudaSuccess) {
      LcJob x = empty_job();
      x.mode = kLcOut;
      x.M = d->N;
      x.Nn = d->K;
      x.nkb = (cols + kLcKb - 1) / kLcKb;
      x.slices = p.dx_slices;
      x.per = (x.nkb + x.slices - 1) / x.slices;
      x.slices = (x.nkb + x.per - 1) / x.per;  // a short last piece may fill fewer slices; the rest keep their sums
      x.b_mn = vk;
      x.b_k0 = v0;
      x.acc = dx_acc;
      x.lda = p.dx_lda;
      x.acc_in = i > 0;
      x.scale = scale;
      x.ldo = d->lddx;
      if (p.dx_slices == 1 && i == p.pieces - 1) x.out = static_cast<__nv_bfloat16*>(dX);
      if (!encode(&x.ta, G, cols, d->N, p.ldg, kLcHalf)) return DSPARK_EINVAL;
      if (!(vk ? encode(&x.tb, W, d->K, d->V, d->ldw, kLcKb) : encode(&x.tb, W, d->V, d->K, d->ldw, kLcHalf)))
        return DSPARK_EINVAL;
      e = run_job(x, device_status, st);
    }
    if (dW && e == cudaSuccess) {
      LcJob w = empty_job();
      w.mode = kLcOut;
      w.M = vk ? cols : d->K;
      w.Nn = vk ? d->K : cols;
      w.nkb = (d->N + kLcKb - 1) / kLcKb;
      w.slices = p.dw_slices;
      w.per = p.dw_per;
      w.a_mn = w.b_mn = 1;
      w.scale = scale;
      w.ldo = d->lddw;
      w.lda = p.dw_lda;
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(dW) + (vk ? (int64_t)v0 * d->lddw : v0);
      if (p.dw_slices == 1)
        w.out = out;
      else
        w.acc = dw_acc;
      CUtensorMap* tg = vk ? &w.ta : &w.tb;
      CUtensorMap* tx = vk ? &w.tb : &w.ta;
      if (!encode(tg, G, cols, d->N, p.ldg, kLcKb) || !encode(tx, X, d->K, d->N, d->ldx, kLcKb)) return DSPARK_EINVAL;
      e = run_job(w, device_status, st);
      if (p.dw_slices > 1 && e == cudaSuccess) {
        const int64_t n = (int64_t)w.M * ((w.Nn + 3) / 4);
        k_lce_join<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(dw_acc, w.slices, w.M, w.Nn, w.lda, scale, out, w.ldo);
        e = cudaGetLastError();
      }
    }
  }
  if (dX && p.dx_slices > 1 && e == cudaSuccess) {
    const int64_t n = (int64_t)d->N * ((d->K + 3) / 4);
    k_lce_join<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(dx_acc, p.dx_slices, d->N, d->K, p.dx_lda, scale,
                                                            static_cast<__nv_bfloat16*>(dX), d->lddx);
    e = cudaGetLastError();
  }
  return lce_fail(e);
}
