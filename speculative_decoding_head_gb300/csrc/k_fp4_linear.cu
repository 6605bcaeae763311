// k_fp4_linear.cu -- the product of two matrices held in microscaled 4-bit
// floating point, Y[n][v] = sum_k x[n][k] w[v][k] (+ U[n][v]).
//
// The vocabulary is the MMA's M: a tile is 256 rows of w by up to 256 rows of
// x, so that a few tokens make narrow tiles and w streams by once, and a warp of
// the epilogue holds 32 neighbouring v of one token: its stores are whole sectors
// of Y without a transpose. Persistent CTA pairs: each CTA holds half of
// a tile's w and half of its x. A producer warp loads 256 columns of both operands a
// stage (128-byte swizzled boxes) with their scales (contiguous, as
// dspark_fp4_quant lays them out); the MMA warp copies the scales to TMEM and issues
// four block-scaled MMAs of 64 columns; eight warps work off accumulators, 16 tokens
// by 32 v a box of shared memory: U comes in by the copy engine some boxes ahead, the
// result goes out from the same box. Where U's rows are not on 16 bytes its boxes come by
// four-byte copies of the lanes, where Y's are not they leave by plain stores.
//
// TMEM: two accumulators, and 48 columns of scales. Accumulators of more than
// 224 columns overlap in the middle: the epilogue empties the shared columns
// first, and the next tile's MMAs wait for those alone.
//
// Measured at V = 129280, nvfp4: K = 5120, N = 1 to fp32 58 us (w's 372 MB at 6.4 TB/s:
// bound by memory, as up to some 100 tokens); N = 640 163 us (5.2 PFLOP/s; its loads
// alone take 100 us, from L2 at 21 TB/s, without the stores of 331 MB 130);
// N = 4096, K = 5376 to bf16 800 us (7.1 PFLOP/s), 910 in a long run under the
// power limit. mxfp4, K = 256, N = 640 with U 120 us (680 MB at 5.6 TB/s; with plain loads
// and stores 287); V = 50257 53 us, with U's rows, Y's, or both off 16 bytes 74, 78 and 101. Without U 62 us, to
// bf16 56 (nvfp4 64 and 66, with U 150 and 137): the epilogue's work a value, the same for half the bytes.
// More or fewer stages change nothing.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdio.h>

#include <type_traits>

#include "dspark_common.cuh"
#include "dspark_internal.h"
#include "fp4.cuh"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

using namespace fp4;

// How U comes in: not at all, by the copy engine, or by copies of four bytes a lane where its rows are not on 16 bytes.
enum FlU { kFlNoU, kFlBoxU, kFlLaneU };
constexpr int kFlTileV = 256;         // of a pair
constexpr int kFlHalfV = 128;
constexpr int kFlMaxN = 256;          // tokens of a tile
constexpr int kFlThreads = 384;       // producer, MMA, TMEM and a spare warp, eight epilogue warps
constexpr int kFlSfCol = 464;         // TMEM columns of the scales, after the accumulators
constexpr int kFlMaxStages = 12;
constexpr int kFlBoxBytes = 128;      // kChunk values
constexpr int kFlABytes = kFlHalfV * kFlBoxBytes;

struct FlArgs {
  const float* wf;
  const float* xf;
  const float* U;
  void* Y;
  int64_t ldu, ldy;
  int N, K, V;
  int tn;        // tokens of a tile, a multiple of 32
  int vt, nt;    // tiles
  int stages, stage_bytes;
  int acc1, overlap;  // the second accumulator's first column; columns it shares with the first
  int ybox;      // columns of Y that go out by the copy engine: its stores write 16 bytes, so up to a multiple of those
  int* status;
};

struct FlMaps {
  CUtensorMap w, x, ws, xs;  // codes and scales
  CUtensorMap u, y;          // with boxes
};

// Boxes of 16 tokens by 32 v of each epilogue warp: with U four, three of them on their way, else two.
__host__ __device__ constexpr int fl_slots(bool has_u) { return has_u ? 4 : 2; }
__host__ __device__ constexpr int fl_slot_bytes(bool has_u, int size) { return has_u || size == 4 ? 2048 : 1024; }

struct FlBars {
  uint64_t ufull[8][4];
  uint64_t full[kFlMaxStages], empty[kFlMaxStages], tfull[2], tempty[2], over, drain;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ void put(float* p, float y) { __stcs(p, y); }

// 16 columns (tokens n0 .. n0 + 15) of 32 lanes (v), stored.
template <typename T>
__device__ __forceinline__ void fl_store16(const FlArgs& a, float* z, int n0, int nn, int v) {
  if (sizeof(T) == 4) {
    float* y = static_cast<float*>(a.Y) + (int64_t)n0 * a.ldy + v;
    if (v < a.V) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < nn) put(y + i * a.ldy, z[i]);
    }
  } else {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.Y) + (int64_t)n0 * a.ldy;
    const int lane = threadIdx.x & 31, odd = lane & 1;
    const bool pairs = (a.ldy & 1) == 0 && (reinterpret_cast<uintptr_t>(a.Y) & 3u) == 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      // neighbouring lanes trade: the even one stores both v of token i, the odd one of token i + 1
      const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? z[i] : z[i + 1], 1);
      const float lo = odd ? other : z[i], hi = odd ? z[i + 1] : other;
      const int n = i + odd, ve = v - odd;
      __nv_bfloat16* p = y + n * a.ldy + ve;
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      if (n < nn && ve < a.V) {
        if (pairs && ve + 1 < a.V) {
          *reinterpret_cast<__nv_bfloat162*>(p) = h;
        } else {
          p[0] = h.x;
          if (ve + 1 < a.V) p[1] = h.y;
        }
      }
    }
  }
}

// Times w's factor and x's, exactly. A sum is a multiple of 2^-20 below 2^40 and a factor at least 2^-100, so that w's
// may come first up to kFlFar. FAR: one of the warp's rows has a larger one; only what is below 1 of it comes first, then
// x's, then what is above 1, and no step leaves fp32's range where the result does not. (All tiles that way: 640 x 256 x
// 129280 to fp32 65.8 us and to bf16 69.4, with both ways 63.7 and 66.3.)
constexpr float kFlFar = 0x1p80f;
template <bool FAR>
__device__ __forceinline__ void fl_scale16(const FlArgs& a, float* z, int n0, float wf) {
  const float first = FAR ? fminf(wf, 1.f) : wf, last = fmaxf(wf, 1.f);
  const unsigned long long w2 = tc::f2pack(first, first);
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(a.xf + n0 + i));
    tc::f2unpack(tc::mul2(tc::mul2(tc::f2pack(z[i], z[i + 1]), w2), tc::f2pack(f.x, f.y)), z[i], z[i + 1]);
    tc::f2unpack(tc::mul2(tc::mul2(tc::f2pack(z[i + 2], z[i + 3]), w2), tc::f2pack(f.z, f.w)), z[i + 2], z[i + 3]);
  }
  if (FAR)
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] *= last;
}

// The boxes of one epilogue warp, in the order that it takes them.
struct FlUnits {
  int t, i, j;  // tile, its number among the pair's, place in its order
};

template <int FMT, typename T, int U>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kFlThreads, 1)
    k_fp4_linear(const __grid_constant__ FlMaps maps, FlArgs a) {
  constexpr int kSf = chunk_bytes(FMT);         // bytes of a 128-row group's scales of a stage
  constexpr int kQ = kSf / 512;                 // tiles of four blocks in them
  extern __shared__ uint8_t raw[];
  __shared__ FlBars bars;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = tc::smem_u32(base);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tiles = a.vt * a.nt, chunks = chunks_of(a.K);
  const uint32_t rank = tc::cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  volatile int* abort = &bars.abort;
  auto bar = [&](uint64_t* b) { return tc::smem_u32(b); };

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      tc::mbar_init(bar(&bars.full[s]), 1);
      tc::mbar_init(bar(&bars.empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(&bars.tfull[i]), 1);
      tc::mbar_init(bar(&bars.tempty[i]), 16);  // the even CTA's: both CTAs' epilogue warps
    }
    tc::mbar_init(bar(&bars.over), 16);
    for (int i = 0; i < 32; ++i) tc::mbar_init(bar(&bars.ufull[i >> 2][i & 3]), 1);
    tc::mbar_init(bar(&bars.drain), 1);
    bars.abort = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&maps.w);
    tc::prefetch_tmap(&maps.x);
    tc::prefetch_tmap(&maps.ws);
    tc::prefetch_tmap(&maps.xs);
  }
  if (warp == 2) {
    tc::tmem_alloc_pair(tc::smem_u32(&bars.tmem), 512);
    tc::tmem_relinquish_pair();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_meet();
  tc::tc_fence_after();
  const uint32_t tmem = bars.tmem;
  pdl_wait();
  pdl_trigger();

  const int half = a.tn / 2;  // rows of x that a stage has room for in each CTA
  const int b_off = kFlABytes, sa_off = b_off + half * kFlBoxBytes, sb_off = sa_off + kSf;
  bool ok = true;
  // The producer and the MMA warp run their loops whole; one lane issues (see elect_one).
  if (warp == 0) {
    int k = 0, s = 0, ph = 1;
    for (int t = pair; t < tiles && ok; t += pairs) {
      const int v0 = t / a.nt * kFlTileV + (int)rank * kFlHalfV, n0 = t % a.nt * a.tn;
      const int nn = min(a.tn, a.N - n0), nsb = (nn + kRows - 1) / kRows;
      const int nb = n0 + (int)rank * ((nn + 31) / 32 * 16);  // this CTA's first column of B
      const uint32_t bytes = kFlABytes + half * kFlBoxBytes + (1 + nsb) * kSf;
      const int wrow = v0 / kRows * chunks * kQ, xrow = n0 / kRows * chunks * kQ;  // rows of 512 bytes
      for (int c = 0; c < chunks; ++c, ++k) {
        ok = tc::mbar_wait_warp(bar(&bars.empty[s]), ph, abort);
        if (!ok) break;
        if (tc::elect_one()) {
          const uint32_t st = sbase + s * a.stage_bytes, f = tc::map_rank(bar(&bars.full[s]), 0);
          if (rank == 0) tc::mbar_arrive_expect_tx(bar(&bars.full[s]), 2 * bytes);  // both CTAs' copies
          tc::tma_load_2d_pair(st, &maps.w, c * kFlBoxBytes, v0, f);
          tc::tma_load_2d_pair(st + b_off, &maps.x, c * kFlBoxBytes, nb, f);
          tc::tma_load_2d_pair(st + sa_off, &maps.ws, 0, wrow + c * kQ, f);
          tc::tma_load_2d_pair(st + sb_off, &maps.xs, 0, xrow + c * kQ, f);
          if (nsb > 1) tc::tma_load_2d_pair(st + sb_off + kSf, &maps.xs, 0, xrow + (chunks + c) * kQ, f);
        }
        __syncwarp();
        if (++s == a.stages) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    // the last stages' releases, which the even CTA's MMAs send to both CTAs, have arrived before either exits
    for (int j = max(0, k - a.stages); j < k && ok; ++j)
      ok = tc::mbar_wait_warp(bar(&bars.empty[j % a.stages]), j / a.stages & 1, abort);
    if (!ok && lane == 0) {
      *abort = 1;
      raise_status(a.status, DSPARK_ETIMEOUT);
      int never = 0;  // copies in flight (they complete on the even CTA's barriers) land before the pair ends
      if (rank == 0)
        for (int j = max(0, k - a.stages); j < k; ++j)
          tc::mbar_wait(bar(&bars.full[j % a.stages]), j / a.stages & 1, &never);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t sfa = tmem + kFlSfCol, sfb = sfa + 4 * kQ;
      const uint64_t ad0 = tc::smem_desc(sbase, 16, 1024), sd0 = tc::scales_desc(sbase);
      int i = 0, s = 0, ph = 0;
      for (int t = pair; t < tiles && ok; t += pairs, ++i) {
        const int n0 = t % a.nt * a.tn, nn = min(a.tn, a.N - n0), nm = (nn + 31) / 32 * 32;
        const int nsb = (nn + kRows - 1) / kRows, buf = i & 1;
        const uint32_t d = tmem + (buf ? a.acc1 : 0);
        const uint32_t id = tc::idesc_fp4(kFlTileV, nm, FMT == DSPARK_MXFP4, 0);
        ok = tc::mbar_wait_warp(bar(&bars.tempty[buf]), (i >> 1 & 1) ^ 1, abort);
        if (ok && a.overlap && i > 0) ok = tc::mbar_wait_warp(bar(&bars.over), (i - 1) & 1, abort);
        tc::tc_fence_after();
        for (int c = 0; c < chunks && ok; ++c) {
          ok = tc::mbar_wait_warp(bar(&bars.full[s]), ph, abort);
          if (!ok) break;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            const uint32_t off = (uint32_t)(s * a.stage_bytes) >> 4;
            const uint64_t ad = ad0 + off, bd = ad + (b_off >> 4);
            const uint64_t sa = sd0 + off + (sa_off >> 4), sb = sd0 + off + (sb_off >> 4);
#pragma unroll
            for (int q = 0; q < kQ; ++q) tc::cp_scales_pair(sfa + 4 * q, sa + 32 * q);
            if (nsb == 1) {
#pragma unroll
              for (int q = 0; q < kQ; ++q) tc::cp_scales_pair(sfb + 4 * q, sb + 32 * q);
            } else {
#pragma unroll
              for (int q = 0; q < kQ; ++q) {
                tc::cp_scales_pair(sfb + 8 * q, sb + 32 * q);
                tc::cp_scales_pair(sfb + 8 * q + 4, sb + (kSf >> 4) + 32 * q);
              }
            }
            const int steps = min(4, (a.K - c * kChunk + 63) / 64);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < steps) {
                // an nvfp4 step has its own word of scales; two mxfp4 steps share one, by halves
                const int q = FMT == DSPARK_NVFP4 ? kk : kk >> 1;
                const uint32_t part = FMT == DSPARK_NVFP4 ? 0 : (kk & 1) * 2;
                const uint32_t idk = id | part << 4 | part << 29;
                if (FMT == DSPARK_NVFP4)
                  tc::mma_nvfp4_pair(d, ad + 2 * kk, bd + 2 * kk, idk, sfa + 4 * q, sfb + 4 * nsb * q, (c | kk) != 0);
                else
                  tc::mma_mxfp4_pair(d, ad + 2 * kk, bd + 2 * kk, idk, sfa + 4 * q, sfb + 4 * nsb * q, (c | kk) != 0);
              }
            }
            tc::mma_commit_pair(bar(&bars.empty[s]));
            if (c == chunks - 1) tc::mma_commit_pair(bar(&bars.tfull[buf]));
          }
          __syncwarp();
          if (++s == a.stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      // both CTAs' epilogues have released the last tiles: every MMA is complete, and their arrivals have landed
      // before this CTA exits
      for (int j = max(0, i - 2); j < i && ok; ++j) ok = tc::mbar_wait_warp(bar(&bars.tempty[j & 1]), j >> 1 & 1, abort);
      if (ok && a.overlap && i > 0) ok = tc::mbar_wait_warp(bar(&bars.over), (i - 1) & 1, abort);
      if (!ok && lane == 0) {
        *abort = 1;
        raise_status(a.status, DSPARK_ETIMEOUT);
        int never = 0;
        tc::mma_commit_pair_own(bar(&bars.drain));  // every MMA issued completes before TMEM and operands go
        tc::mbar_wait(bar(&bars.drain), 0, &never);
      }
    }
  } else if (warp >= 4) {
    constexpr int kSlots = fl_slots(U != kFlNoU), kSlot = fl_slot_bytes(U != kFlNoU, sizeof(T));
    const int e = warp - 4, q = e & 3, h = e >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t over = tc::map_rank(bar(&bars.over), 0);
    const int units = a.tn / 16, nov = a.overlap / 16;
    const int vq = (int)rank * kFlHalfV + q * 32;  // the warp's first row in a tile
    const uint32_t slots = sbase + a.stages * a.stage_bytes + e * (kSlots * kSlot);
    // the first accumulator's last columns and the second's first are the shared ones: they come first
    auto col = [&](int i, int j) { return 16 * (i & 1 ? j : units - 1 - j); };
    // the next unit of 16 tokens that there are any of, from unit u on
    auto live = [&](FlUnits u) {
      for (; u.t < tiles; u.t += pairs, ++u.i, u.j = h) {
        const int nn = min(a.tn, a.N - u.t % a.nt * a.tn);
        for (; u.j < units; u.j += 2)
          if (col(u.i, u.j) < nn) return u;
      }
      return u;
    };
    int g = 0;  // boxes taken
    FlUnits ahead{pair, 0, h};
    int asked = 0;
    auto ask = [&]() {  // U's next box
      ahead = live(ahead);
      if (ahead.t >= tiles) return;
      const int v = ahead.t / a.nt * kFlTileV + vq, n = ahead.t % a.nt * a.tn + col(ahead.i, ahead.j);
      const uint32_t to = slots + asked % kSlots * kSlot;
      if (U == kFlLaneU) {  // four bytes a lane and token, which that lane reads
        const float* u = a.U + (int64_t)n * a.ldu + v + lane;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const bool there = n + i < a.N && v + lane < a.V;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + i * 128 + lane * 4),
                       "l"(there ? u + i * a.ldu : a.U), "r"(there ? 4 : 0)
                       : "memory");
        }
      } else if (lane == 0) {
        const uint32_t b = bar(&bars.ufull[e][asked % kSlots]);
        tc::mbar_arrive_expect_tx(b, 2048);
        tc::tma_load_2d(to, &maps.u, v, n, b, tc::policy_evict_first());
      }
      ++asked;
      ahead.j += 2;
    };
    auto ask_next = [&]() {
      ask();
      if (U == kFlLaneU) asm volatile("cp.async.commit_group;" ::: "memory");  // an empty one too: they are counted
    };
    if (U != kFlNoU)
      for (int i = 0; i < kSlots - 1; ++i) ask_next();
    // 16 columns: scaled, U added, to their box and out
    auto put = [&](auto far, float* z, int c, int v0, int n0, int nn, float wf) {
      if (FMT == DSPARK_NVFP4) fl_scale16<decltype(far)::value>(a, z, n0 + c, wf);
      const uint32_t box = slots + g % kSlots * kSlot;
      if (U != kFlNoU) {
        if (U == kFlBoxU)  // each lane for itself: no one goes by it before the next tile's vote
          ok = ok && tc::mbar_wait(bar(&bars.ufull[e][g % kSlots]), g / kSlots & 1, abort);
        else
          asm volatile("cp.async.wait_group %0;" ::"n"(kSlots - 2) : "memory");
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float u;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(u) : "r"(box + i * 128 + lane * 4));
          z[i] += u;
        }
        if (sizeof(T) == 2) __syncwarp();  // the box is written with other rows
      } else if (a.ybox) {
        // the store before the last has read this box
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        __syncwarp();
      }
      if (a.ybox) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (sizeof(T) == 4)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(box + i * 128 + lane * 4), "f"(z[i]) : "memory");
          else
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(box + i * 64 + lane * 2),
                         "h"(__bfloat16_as_ushort(__float2bfloat16_rn(z[i])))
                         : "memory");
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tc::tma_store_2d(&maps.y, v0 + vq, n0 + c, box);
          tc::bulk_commit();
          // U's next box goes where the store before this one came from
          if (U != kFlNoU) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        const int v = v0 + vq + lane;
        if (v >= a.ybox && v < a.V) {  // the last columns
          T* y = static_cast<T*>(a.Y) + (int64_t)(n0 + c) * a.ldy + v;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < nn) y[i * a.ldy] = T(z[i]);
        }
      } else {
        fl_store16<T>(a, z, n0 + c, nn - c, v0 + vq + lane);
      }
      if (U != kFlNoU) {
        __syncwarp();
        ask_next();
      }
      ++g;
    };
    // a lane's factor of w in tile t; rows' factors are padded to whole 128-row groups
    auto factor = [&](int t) {
      const int v = t / a.nt * kFlTileV + vq + lane;
      return FMT == DSPARK_NVFP4 && t < tiles && v < (a.V + kRows - 1) / kRows * kRows ? __ldg(a.wf + v) : 1.f;
    };
    int i = 0;
    float wf_next = factor(pair);  // a tile ahead: the choice of a way below does not wait for it
    for (int t = pair; t < tiles; t += pairs, ++i) {
      const int v0 = t / a.nt * kFlTileV, n0 = t % a.nt * a.tn, nn = min(a.tn, a.N - n0), buf = i & 1;
      const float wf = wf_next;
      wf_next = factor(t + pairs);
      ok = __all_sync(0xFFFFFFFFu, ok && tc::mbar_wait(bar(&bars.tfull[buf]), i >> 1 & 1, abort));
      if (!ok) break;
      tc::tc_fence_after();
      const uint32_t d = lanes + (buf ? a.acc1 : 0);
      // two units at a time; their columns are free once they are in registers
      auto out = [&](auto far) {
        for (int j = h; j < units; j += 4) {
          float z[2][16];
          const int c0 = col(i, j), c1 = j + 2 < units ? col(i, j + 2) : kFlMaxN;
          tc::tmem_ld16(d + c0, z[0]);
          if (j + 2 < units) tc::tmem_ld16(d + c1, z[1]);
          tc::tmem_wait_ld();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (nov && j == h) tc::mbar_arrive_cluster_relaxed(over);  // nov <= 4: they are all in registers
            if (j + 4 >= units) tc::mbar_arrive_cluster_relaxed(tc::map_rank(bar(&bars.tempty[buf]), 0));
          }
          if (c0 < nn) put(far, z[0], c0, v0, n0, nn, wf);
          if (c1 < nn) put(far, z[1], c1, v0, n0, nn, wf);
        }
      };
      if (FMT == DSPARK_NVFP4 && __any_sync(0xFFFFFFFFu, wf > kFlFar))
        out(std::true_type{});
      else
        out(std::false_type{});
    }
    // stores are complete, and U's boxes that no one took have come
    if (U == kFlLaneU) asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) {
      asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
      int never = 0;
      if (U == kFlBoxU && !ok)
        for (int x = max(0, asked - kSlots); x < asked; ++x)  // of each slot the last one, taken or not
          tc::mbar_wait(bar(&bars.ufull[e][x % kSlots]), x / kSlots & 1, &never);
    }
    __syncwarp();
    if (!ok) {
      *abort = 1;
      raise_status(a.status, DSPARK_ETIMEOUT);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::cluster_meet();
  tc::tc_fence_after();
  if (warp == 2) tc::tmem_dealloc_pair(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// The codes of `rows` rows; boxes of 256 values (128 bytes) by box_rows.
bool encode(CUtensorMap* tm, const void* codes, int K, int rows, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)row_bytes(K), (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes(K)};
  const cuuint32_t box[2] = {kFlBoxBytes, (cuuint32_t)box_rows};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales as rows of 512 bytes; boxes of one 128-row group's of 256 columns.
bool encode_scales(CUtensorMap* tm, const void* scales, int K, int rows, int format) {
  const cuuint64_t groups = ((cuuint64_t)rows + kRows - 1) / kRows;
  const int per = chunk_bytes(format) / 512;
  const cuuint64_t dims[2] = {128, groups * chunks_of(K) * per};
  const cuuint64_t strides[1] = {512};
  const cuuint32_t box[2] = {128, (cuuint32_t)per};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(tm, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(scales), dims, strides, box, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// U or Y by boxes of 16 rows and 32 columns.
bool encode_boxes(CUtensorMap* tm, const void* p, bool bf16, int V, int N, int64_t ld) {
  const cuuint64_t dims[2] = {(cuuint64_t)V, (cuuint64_t)N};
  const cuuint64_t strides[1] = {(cuuint64_t)ld * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {32, 16};
  const cuuint32_t es[2] = {1, 1};
  return encode_fn()(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                     const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int FMT, typename T, int U>
cudaError_t launch(const FlMaps& maps, const FlArgs& a, int grid, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  constexpr int kMax = 227 * 1024 - 1024;  // the barriers are static
  const cudaError_t c = once_per_device(done, [] {
    return cudaFuncSetAttribute(k_fp4_linear<FMT, T, U>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMax);
  });
  if (c != cudaSuccess) return c;
  const size_t slots = 8 * fl_slots(U != kFlNoU) * fl_slot_bytes(U != kFlNoU, sizeof(T));
  return launch_ex(k_fp4_linear<FMT, T, U>, dim3(grid), dim3(kFlThreads), (size_t)a.stages * a.stage_bytes + slots + 1024,
                   st, true, maps, a);
}
template <int FMT, typename T>
cudaError_t launch_u(int u, const FlMaps& maps, const FlArgs& a, int grid, cudaStream_t st) {
  return u == kFlNoU    ? launch<FMT, T, kFlNoU>(maps, a, grid, st)
         : u == kFlBoxU ? launch<FMT, T, kFlBoxU>(maps, a, grid, st)
                        : launch<FMT, T, kFlLaneU>(maps, a, grid, st);
}
template <int FMT>
cudaError_t launch_t(bool bf16, int u, const FlMaps& maps, const FlArgs& a, int grid, cudaStream_t st) {
  return bf16 ? launch_u<FMT, __nv_bfloat16>(u, maps, a, grid, st) : launch_u<FMT, float>(u, maps, a, grid, st);
}

bool on_type(const void* p, int size) { return p && (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(size - 1)) == 0; }

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" dspark_status dspark_fp4_linear(const dspark_fp4_dims* xd, const dspark_fp4_data* x,
                                           const dspark_fp4_dims* wd, const dspark_fp4_data* w, const float* U,
                                           int64_t ldu, void* Y, dspark_wdtype type, int64_t ldy,
                                           int32_t* device_status, dspark_stream_t stream) {
  if (!fp4::dims_ok(xd) || !fp4::dims_ok(wd) || wd->rows < 1 || xd->K != wd->K || xd->format != wd->format)
    return DSPARK_EINVAL;
  if ((type != DSPARK_F32 && type != DSPARK_BF16) || !device_status || ldy < wd->rows) return DSPARK_EINVAL;
  if (U && (!on_type(U, 4) || ldu < wd->rows)) return DSPARK_EINVAL;
  if (xd->rows == 0) return DSPARK_OK;
  if (!fp4::data_ok(xd, x) || !fp4::data_ok(wd, w) || !on_type(Y, type == DSPARK_BF16 ? 2 : 4)) return DSPARK_EINVAL;
  if (U == Y && (type != DSPARK_F32 || ldu != ldy)) return DSPARK_EINVAL;
  FlArgs a = {};
  a.wf = w->rowf;
  a.xf = x->rowf;
  a.U = U;
  a.Y = Y;
  a.ldu = ldu;
  a.ldy = ldy;
  a.N = xd->rows;
  a.K = xd->K;
  a.V = wd->rows;
  a.status = device_status;
  // one tile of tokens for up to 256 of them; more in tiles of 256 (scales come in groups of 128 rows)
  a.tn = a.N >= kFlMaxN ? kFlMaxN : (a.N + 31) / 32 * 32;
  a.vt = (a.V + kFlTileV - 1) / kFlTileV;
  a.nt = (a.N + a.tn - 1) / a.tn;
  const int64_t tiles = (int64_t)a.vt * a.nt;
  if (tiles > (1ll << 30)) return DSPARK_EUNSUPPORTED;  // they are counted in 32 bits, steps of the grid beyond the last among them
  if (!encode_fn()) return DSPARK_ECUDA;
  const int acc = kFlSfCol / 2 / 16 * 16;  // 224 columns each without overlap
  a.overlap = a.tn > acc ? 2 * a.tn - kFlSfCol : 0;
  a.acc1 = a.tn - a.overlap;
  const int sf = fp4::chunk_bytes(wd->format);
  const int bytes = kFlABytes + a.tn / 2 * kFlBoxBytes + sf * (1 + (a.tn + fp4::kRows - 1) / fp4::kRows);
  a.stage_bytes = (bytes + 1023) / 1024 * 1024;
  const int slots = 8 * fl_slots(U != nullptr) * fl_slot_bytes(U != nullptr, type == DSPARK_BF16 ? 2 : 4);
  a.stages = (227 * 1024 - 2048 - slots) / a.stage_bytes;
  if (a.stages > kFlMaxStages) a.stages = kFlMaxStages;
  FlMaps maps = {};
  if (!encode(&maps.w, w->codes, a.K, a.V, kFlHalfV) || !encode(&maps.x, x->codes, a.K, a.N, a.tn / 2) ||
      !encode_scales(&maps.ws, w->scales, a.K, a.V, wd->format) ||
      !encode_scales(&maps.xs, x->scales, a.K, a.N, wd->format))
    return DSPARK_ECUDA;
  const int size = type == DSPARK_BF16 ? 2 : 4;
  a.ybox = (reinterpret_cast<uintptr_t>(Y) & 15u) == 0 && ldy * size % 16 == 0 ? a.V & ~(16 / size - 1) : 0;
  const int u = !U ? kFlNoU : (reinterpret_cast<uintptr_t>(U) & 15u) == 0 && ldu % 4 == 0 ? kFlBoxU : kFlLaneU;
  if ((a.ybox && !encode_boxes(&maps.y, Y, size == 2, a.ybox, a.N, ldy)) ||
      (u == kFlBoxU && !encode_boxes(&maps.u, U, false, a.V, a.N, ldu)))
    return DSPARK_ECUDA;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int grid = 2 * (int)(tiles < sms / 2 ? tiles : sms / 2);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (e == cudaSuccess)
    e = wd->format == DSPARK_NVFP4 ? launch_t<DSPARK_NVFP4>(type == DSPARK_BF16, u, maps, a, grid, st)
                                   : launch_t<DSPARK_MXFP4>(type == DSPARK_BF16, u, maps, a, grid, st);
  if (e != cudaSuccess) fprintf(stderr, "dspark: CUDA error %s\n", cudaGetErrorString(e));
  return e == cudaSuccess ? DSPARK_OK : DSPARK_ECUDA;
}
