// q8mm.cu -- dense products of 8-bit rows and 8-bit weights,
//   y[m, n] = bf16(sum_g sx[m, g] sw[n / 128, g] sum_{k in group g} x[m, k] w[n, k]),
// groups of 128 columns.
//
// The inner sum is the tensor cores' (tcgen05, kind::f8f6f4: four instructions of 32 columns a group, fp32
// accumulators in TMEM); the outer one, where the scales differ, is an fp32 FMA a group and output in registers.
// Scales may be any fp32 numbers whose products, sx sw, are normal ones: the kernel forms them before it multiplies the
// sums.  (The tensor cores' own block scaling takes powers of two alone, as the quantisers write them; there is no form
// for it.)  Beside a group of a 128 x 256 tile, 512 cycles of MMAs, the sums read TMEM for 256 cycles and have 128 of FMAs,
// two values an instruction.
//
// Orientation: 128 rows of x on the MMA's M side, TN weight rows on its N side.  A TMEM lane is then a row of x, a
// thread's columns lie within one block of 128 weight rows, and the factor of a group is one number a thread.
// Warp 0 issues TMA (both operands K-major, 128-byte swizzle: a stage is one group), warp 1 the MMAs, each group into
// the next of 512 / TN accumulators, warps 2 and 3 bring the scales, multiplied, four groups at a time (a row's scales
// lie far from the next row's: such loads hold up every other access to shared memory of the warp that issues them), and
// warps 4..11 add the groups up: warp w the lanes 32 (w % 4).., half the columns.
//
// Forms:
// - few tiles and many groups: K is split over the CTAs of a cluster (up to 8), each sums its groups, and every rank
//   adds one slice of the columns up over the ranks, by twos and in rank order, through distributed shared memory;
// - else a CTA a tile, and with more tiles than SMs persistent CTAs that take them row tiles first, so that a weight tile
//   is read from HBM once;
// - many rows: pairs of CTAs (cta_group::2) on tiles of 256 x 256, which halves what an SM loads for a product.
//
// Output goes by TMA while the next tile runs where its rows begin on 16 bytes; others are written by the warps, whole
// rows at a time (2440 x 129279 x 1280 503 us; each thread its own row 3036).
//
// What bounds the pairs is the way of a group through two accumulators of 256 columns: by time stamps 830 cycles from an
// accumulator's release to the end of its next group (MMAs 512), 770 until it is read, 100 until that is known, and two
// groups share them, 0.9 K cycles each; the sums' own loop, some 180 instructions a warp and group, takes as long.
// 2440 x 129280 x 1280 413 us (1.95 PFLOP/s), 4879 x 1280 x 7168 57 us.  One CTA a tile of 128 x 256 with two warps that
// issue MMAs: 460 and 63; twice the warps with half the columns each: 479 and 68; accumulators handed over in halves: 417
// and 63; pairs on 256 x 192 with twelve warps 472 and 55, on 256 x 128 with four accumulators 540 and 64.
// All sums are of a fixed order: results are the same from run to run, and up to 256 rows a row's bits do not depend
// on how many rows there are, as a verify pass of several positions a sequence and a decoding step of one want it.
#include <cuda_bf16.h>

#include <atomic>

#include "internal.h"
#include "lsv.h"
#include "ptx.cuh"
#include "q4ptx.cuh"
#include "q8.cuh"
#include "q8ptx.cuh"
#include "tmap.h"

namespace lsv {
namespace {

constexpr int kMmThreads = 384;  // warp 0 TMA, warp 1 MMA, warps 4..11 sums and output
// Registers: what a thread is launched with, and what the first warpgroup keeps and the other two get of the sum (the
// pair's sums take more; at 128 columns the first warpgroup has the more to hold).
constexpr int kMmRegs = 168;
constexpr int mm_regs_few(bool pair) { return pair ? 72 : 88; }
constexpr int mm_regs_many(bool pair) { return pair ? 216 : 208; }
static_assert(128 * mm_regs_few(true) + 256 * mm_regs_many(true) <= 384 * kMmRegs, "register split");
static_assert(128 * mm_regs_few(false) + 256 * mm_regs_many(false) <= 384 * kMmRegs, "register split");
constexpr int kMmTile = 128;     // rows of x a CTA
constexpr int kMmSameRows = 256;  // up to so many rows of x, a row's bits do not depend on their number
constexpr int kMmMaxStages = 12;
constexpr int kMmSmem = 225 * 1024;  // the ring and what lies behind it
constexpr int kMmPanel = 32 * 128;   // bytes of 64 columns of a warp's 32 rows of output
constexpr int kMmBlock = 4;          // groups whose scales are brought at once
constexpr int kMmScaleSlots = 4;     // blocks of scales in shared memory
constexpr int kMmScaleBytes = kMmScaleSlots * kMmBlock * kMmTile * 2 * 4;
constexpr int kMmRowsAtOnce = 8;     // rows of output that a warp holds on their way to where TMA does not store
// What is in flight when a wait has run out is waited for this long, however short the limit of the waits.
constexpr uint64_t kMmDrainNs = 2000000000ull;
// A limit below this is there to run out: then a tile's first stage is waited for awake, so that it does.
constexpr uint64_t kMmShortNs = 1000;

struct MmParams {
  int M, N, K, G;      // G: groups of K
  int nm, nitems;      // row tiles; tiles of the output
  int ns;              // CTAs that share a tile's groups (cluster size; 1 for pairs)
  int stages, a_bytes, stage_bytes;
  int a_last, b_last;  // bytes of the boxes of the last row tile and the last weight tile
  int aligned;         // rows of y start on 16 bytes: they are stored by TMA
  const float* sx;
  const float* sw;
  bf16* y;
  int* err;
  uint64_t wait_ns;
};

struct MmMaps {
  CUtensorMap x, x_last, w, w_last, y;
};

__device__ __forceinline__ uint32_t mm_pack(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// A warp's `rows` x `cols` (64 at most) of output from rows of 128 bytes, 16-byte pieces swizzled, to rows of y that begin
// anywhere.  Where they begin on 8 bytes, two rows at once, four values a lane; else a row at once, two values a lane from
// its first 4-byte boundary on, and the values beside those at the end, a row a lane.  Rows of the panel that do not exist
// are read, and not stored.
__device__ __forceinline__ void store_panel(const uint8_t* panel, bf16* y, int N, int cols, int rows, int lane) {
  if (N % 4 == 0) {
    const int l = lane & 15, h = lane >> 4;
    bf16* to = y + (size_t)h * N + 4 * l;
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 2 * kMmRowsAtOnce) {
      uint2 four[kMmRowsAtOnce];
#pragma unroll
      for (int i = 0; i < kMmRowsAtOnce; ++i) {
        const int r = r0 + 2 * i + h;
        four[i] = *reinterpret_cast<const uint2*>(panel + r * 128 + (((l >> 1) ^ (r & 7)) << 4) + (l & 1) * 8);
      }
#pragma unroll
      for (int i = 0; i < kMmRowsAtOnce; ++i, to += 2 * (size_t)N)
        if (r0 + 2 * i + h < rows && 4 * l < cols) *reinterpret_cast<uint2*>(to) = four[i];
    }
    return;
  }
  // (what depends on where a row begins is the same in every other row)
  const int odd0 = (int)(reinterpret_cast<uintptr_t>(y) >> 1) & 1, odd1 = odd0 ^ (N & 1);
  const bool both[2] = {2 * lane + odd0 + 1 < cols, 2 * lane + odd1 + 1 < cols};
  bf16* to = y + 2 * lane;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += kMmRowsAtOnce) {
    uint32_t two[kMmRowsAtOnce], next[kMmRowsAtOnce];
#pragma unroll
    for (int i = 0; i < kMmRowsAtOnce; ++i)
      two[i] = *reinterpret_cast<const uint32_t*>(panel + (r0 + i) * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4);
#pragma unroll
    for (int i = 0; i < kMmRowsAtOnce; ++i) next[i] = __shfl_down_sync(0xffffffffu, two[i], 1);
#pragma unroll
    for (int i = 0; i < kMmRowsAtOnce; ++i, to += N) {
      const int odd = i & 1 ? odd1 : odd0;
      const uint32_t v = __byte_perm(two[i], next[i], odd ? 0x5432 : 0x3210);
      if (r0 + i < rows && both[i & 1]) *reinterpret_cast<uint32_t*>(to + odd) = v;
    }
  }
  if (N % 2 && lane < rows) {
    const int odd = lane & 1 ? odd1 : odd0, last = cols - 1;
    const uint8_t* row = panel + lane * 128;
    bf16* out = y + (size_t)lane * N;
    if (odd && cols > 0) out[0] = *reinterpret_cast<const bf16*>(row + ((lane & 7) << 4));
    if (cols > odd && (cols - odd) % 2)
      out[last] = *reinterpret_cast<const bf16*>(row + (((last >> 3) ^ (lane & 7)) << 4) + (last & 7) * 2);
  }
}
static_assert(kMmRowsAtOnce % 8 == 0, "the swizzle's period");

// Four groups' scales of a row, those from `g` (a multiple of 4) on that lie within [0, G).
__device__ __forceinline__ float4 load_scales(const float* s, int g, int G) {
  if (G % 4 == 0) {
    const uint4 v = ld_plain128(s + g);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
  }
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  v.x = ld_plain_f32(s + g);
  if (g + 1 < G) v.y = ld_plain_f32(s + g + 1);
  if (g + 2 < G) v.z = ld_plain_f32(s + g + 2);
  if (g + 3 < G) v.w = ld_plain_f32(s + g + 3);
  return v;
}

// TN: weight rows a tile.  PAIR: clusters of two CTAs on tiles of 256 rows; each loads its 128 rows of x and half of
// the weight rows, counts its bytes on the leader's (rank 0's) stage barrier, the leader issues the MMAs of both, and
// its commits release both CTAs' stages and accumulators; each CTA sums its own 128 rows.
// TWO: the CTA's groups are the shares of two CTAs of a split twice as wide, and are added up as those two and then their
// exchange would: share by share (the first one's sums wait in TMEM, in place of the last accumulator), then the two.
template <int TN, bool PAIR, bool TWO>
__global__ void __launch_bounds__(kMmThreads, 1) q8_matmul_kernel(const __grid_constant__ MmMaps maps, const MmParams p) {
  static_assert(!(PAIR && TWO), "a pair has no accumulator to spare");
  constexpr int kTmemCols = 512;
  constexpr int kBufs = kTmemCols / TN - (TWO ? 1 : 0);  // accumulators
  constexpr int kCols = TN / 2;                       // columns a thread
  constexpr int kTileM = PAIR ? 2 * kMmTile : kMmTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[kMmMaxStages], empty[kMmMaxStages], tfull[kBufs], tempty[kBufs], sfull[kMmScaleSlots],
      sempty[kMmScaleSlots], final_bar, recv_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int gave_up, sent[2];  // a wait of this CTA or its pair ran out; groups loaded, of the pair's (sent[0]: own)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool clustered = PAIR || p.ns > 1;
  const uint32_t rank = clustered ? cluster_ctarank() : 0u;
  const bool leader = !PAIR || rank == 0;
  const int size = PAIR ? 2 : p.ns;
  const int first = blockIdx.x / size, step = gridDim.x / size;
  // this CTA's groups of each tile: a split's share, at least one (ns <= G)
  const int g0 = PAIR ? 0 : (int)rank * p.G / p.ns, g1 = PAIR ? p.G : ((int)rank + 1) * p.G / p.ns;
  const int second = (2 * (int)rank + 1) * p.G / (2 * p.ns);  // TWO: where the second share begins
  const int ntn = (p.N + TN - 1) / TN;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < kBufs; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], PAIR ? 16 : 8);
    }
    for (int q = 0; q < kMmScaleSlots; ++q) {
      mbar_init(&sfull[q], 2);
      mbar_init(&sempty[q], 8);
    }
    mbar_init(&final_bar, 1);
    mbar_init(&recv_bar, 1);
    gave_up = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&tmem_slot, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&tmem_slot, kTmemCols);
      tmem_relinquish();
    }
  }
  if (threadIdx.x == 32) {
    tma_prefetch_desc(&maps.x);
    tma_prefetch_desc(&maps.w);
    tma_prefetch_desc(&maps.x_last);
    tma_prefetch_desc(&maps.w_last);
  }
  __syncwarp();
  tc_fence_before_sync();
  if (clustered)
    cluster_sync();  // every CTA's barriers exist before another signals them
  else
    __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = tmem_slot;
  // [slot][group of four][half of the columns][row]
  float* scales = reinterpret_cast<float*>(smem + p.stages * p.stage_bytes);
  uint8_t* behind = reinterpret_cast<uint8_t*>(scales) + kMmScaleBytes;
  const uint64_t drain_ns = p.wait_ns > kMmDrainNs ? p.wait_ns : kMmDrainNs;
  // By one lane of a role whose wait ran out, which issues nothing more; the others' waits run out after it.
  auto give_up = [&]() {
    set_error(p.err, kErrTimeout);
    if constexpr (PAIR) {
      st_shared_cluster_s32(mapa_shared(smem_u32(&gave_up), 0), 1);
      st_shared_cluster_s32(mapa_shared(smem_u32(&gave_up), 1), 1);
    } else {
      gave_up = 1;
    }
  };
  auto group_bytes = [&](int it) {  // of a group of tile `it`, a CTA's
    const int tv = it / p.nm, tr = it - tv * p.nm;
    return (tr == p.nm - 1 ? p.a_last : p.a_bytes) + (tv == ntn - 1 ? p.b_last : TN / (PAIR ? 2 : 1) * 128);
  };
  pdl_trigger();
  pdl_wait();  // x and w may come from the preceding kernels

  if (warp < 4) {
    reg_dec<mm_regs_few(PAIR)>();
    // Both loops are run by the whole warp, and one lane issues.
    if (warp == 0) {
      // ---------------------------------------------------------- TMA
      // weights that one row tile reads come once
      const uint64_t pol_x = l2_policy_evict_last(), pol_w = p.nm == 1 ? l2_policy_evict_first() : l2_policy_evict_last();
      const uint32_t fb0 = PAIR ? mapa_shared(smem_u32(&full[0]), 0) : 0u;
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int it = first; it < p.nitems && ok; it += step) {
        const int tv = it / p.nm, tr = it - tv * p.nm;
        const bool last_r = tr == p.nm - 1, last_v = tv == ntn - 1;
        const CUtensorMap* xm = last_r ? &maps.x_last : &maps.x;
        const CUtensorMap* wm = last_v ? &maps.w_last : &maps.w;
        const int bytes = group_bytes(it);
        const int row = tr * kTileM + (PAIR ? (int)rank * kMmTile : 0);
        const int col = tv * TN + (PAIR ? (int)rank * (TN / 2) : 0);
        for (int g = g0; g < g1; ++g) {
          if (!__all_sync(0xffffffffu, mbar_wait(&empty[stage], phase ^ 1u, p.wait_ns))) {
            ok = false;
            break;
          }
          if (elect_one()) {
            uint8_t* a_s = smem + stage * p.stage_bytes;
            if constexpr (PAIR) {
              if (leader) mbar_arrive_expect_tx(&full[stage], 2 * bytes);
              tma_load_2d_pair(a_s, xm, fb0 + 8 * stage, g * kQ8Group, row, pol_x);
              tma_load_2d_pair(a_s + p.a_bytes, wm, fb0 + 8 * stage, g * kQ8Group, col, pol_w);
            } else {
              mbar_arrive_expect_tx(&full[stage], bytes);
              tma_load_2d(a_s, xm, &full[stage], g * kQ8Group, row, pol_x);
              tma_load_2d(a_s + p.a_bytes, wm, &full[stage], g * kQ8Group, col, pol_w);
            }
          }
          __syncwarp();
          ++issued;
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (lane == 0) {
        if (!ok) give_up();
        if constexpr (PAIR)
          st_shared_cluster_s32(mapa_shared(smem_u32(&sent[rank]), 0), issued);
        else
          sent[0] = issued;
      }
    } else if (warp == 1 && leader) {
      // ---------------------------------------------------------- MMAs (the leader's, for a pair)
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true;
      constexpr uint32_t idesc = idesc_e4m3_f32(kTileM, TN);
      const uint64_t a0 = sdesc_kmajor_sw128(smem_u32(smem)), b0 = sdesc_kmajor_sw128(smem_u32(smem) + p.a_bytes);
      for (int it = first; it < p.nitems && ok; it += step) {
        if (p.wait_ns < kMmShortNs) {
          ok = __all_sync(0xffffffffu, mbar_wait_awake(&full[stage], phase, p.wait_ns));
          if (!ok) break;
        }
        for (int g = g0; g < g1; ++g) {
          // the accumulators last: what they come from is there by then, and nothing is left to ask for between them and
          // the MMAs (the other way round 426 us for 413)
          const bool got =
              mbar_wait(&full[stage], phase, p.wait_ns) && mbar_wait(&tempty[buf], buf_phase ^ 1u, p.wait_ns);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          if (elect_one()) {
            const uint32_t d = tmem_base + (uint32_t)(buf * TN);
            // descriptors hold addresses in units of 16 bytes; a step of 32 columns is two
            const uint64_t at = (uint64_t)(uint32_t)(stage * (p.stage_bytes >> 4));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if constexpr (PAIR)
                umma_e4m3_pair(d, a0 + at + 2 * kk, b0 + at + 2 * kk, idesc, kk ? 1u : 0u);
              else
                umma_e4m3(d, a0 + at + 2 * kk, b0 + at + 2 * kk, idesc, kk ? 1u : 0u);
            }
            if constexpr (PAIR) {
              umma_commit_pair_mc(&tfull[buf], 0x3);
              umma_commit_pair_mc(&empty[stage], 0x3);
            } else {
              umma_commit(&tfull[buf]);
              umma_commit(&empty[stage]);
            }
          }
          __syncwarp();
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++buf == kBufs) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
      }
      // every MMA has completed before TMEM and the ring are given up
      if (elect_one()) {
        if (!ok) give_up();
        if constexpr (PAIR)
          umma_commit_pair_mc(&final_bar, 0x1);
        else
          umma_commit(&final_bar);
        if (!mbar_wait(&final_bar, 0, drain_ns)) set_error(p.err, kErrTimeout);
      }
    }
    if (warp >= 2) {
      // ---------------------------------------------------------- scales: 64 rows a warp, two a lane
      const int r0 = (warp - 2) * 64 + lane;
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int it = first; it < p.nitems && ok; it += step) {
        const int tv = it / p.nm, tr = it - tv * p.nm;
        const int row = tr * kTileM + (PAIR ? (int)rank * kMmTile : 0) + r0;
        const float* sx0 = p.sx + (size_t)min(row, p.M - 1) * p.G;
        const float* sx1 = p.sx + (size_t)min(row + 32, p.M - 1) * p.G;
        const int nb = (p.N - 1) / kQ8Group;
        const float* sw0 = p.sw + (size_t)min(tv * TN / kQ8Group, nb) * p.G;
        const float* sw1 = p.sw + (size_t)min((tv * TN + kCols) / kQ8Group, nb) * p.G;
        for (int g = g0 & ~3; g < g1; g += kMmBlock) {
          const float4 x0 = load_scales(sx0, g, p.G), x1 = load_scales(sx1, g, p.G);
          const float4 w0 = load_scales(sw0, g, p.G), w1 = load_scales(sw1, g, p.G);
          if (!__all_sync(0xffffffffu, mbar_wait(&sempty[slot], phase ^ 1u, p.wait_ns))) {
            ok = false;
            break;
          }
          float* d = scales + slot * (kMmBlock * 2 * kMmTile) + r0;
          const float xs[2][4] = {{x0.x, x0.y, x0.z, x0.w}, {x1.x, x1.y, x1.z, x1.w}};
          const float ws[2][4] = {{w0.x, w0.y, w0.z, w0.w}, {w1.x, w1.y, w1.z, w1.w}};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              d[(2 * i + h) * kMmTile] = xs[0][i] * ws[h][i];
              d[(2 * i + h) * kMmTile + 32] = xs[1][i] * ws[h][i];
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull[slot]);
          if (++slot == kMmScaleSlots) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && lane == 0) give_up();
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ sums over the groups, output
    reg_inc<mm_regs_many(PAIR)>();
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int c0 = half * kCols;
    uint8_t* panel = behind + (warp - 4) * kMmPanel;
    int buf = 0, slot = 0;
    uint32_t buf_phase = 0, slot_phase = 0;
    bool ok = true;
    const uint32_t leaders_tempty = PAIR ? mapa_shared(smem_u32(&tempty[0]), 0) : 0u;
    // The accumulators are read 32 columns at a time, one piece ahead of the sums, from one group into the next and from
    // one tile into the next: a wait for a group and the latency of a read run beside the sums of what was read before.
    // A thread whose row does not exist reads what is there, and stores nothing.
    const uint32_t t_row = tmem_base + ((uint32_t)(32 * quarter) << 16) + (uint32_t)c0;
    constexpr int kPieces = kCols / 32;
    static_assert(kPieces % 2 == 0, "a group begins in r[0]");
    uint32_t r[2][32];
    int left = first < p.nitems ? ((p.nitems - 1 - first) / step + 1) * (g1 - g0) : 0;  // groups not begun
    auto begin = [&]() {
      --left;
      const bool got = mbar_wait(&tfull[buf], buf_phase, p.wait_ns);
      ok = __all_sync(0xffffffffu, got);
      tc_fence_after_sync();
      tmem_ld_32x32b_x32(t_row + (uint32_t)(buf * TN), r[0]);
    };
    if (left > 0) begin();
    // (a split's warps meet behind its one tile, whatever became of their waits)
    for (int it = first; it < p.nitems && (ok || p.ns > 1); it += step) {
      const int tv = it / p.nm, tr = it - tv * p.nm;
      const int row0 = tr * kTileM + (PAIR ? (int)rank * kMmTile : 0) + 32 * quarter;  // the warp's first row
      const int row = row0 + lane;
      const bool any = row0 < p.M, mine = row < p.M;
      const int n0 = tv * TN + c0;
      float2 acc[kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      for (int g = g0; g < g1; ++g) {
        bool got = true;
        if (g == g0 || (g & 3) == 0) got = mbar_wait(&sfull[slot], slot_phase, p.wait_ns);
        const float f = scales[((slot * kMmBlock + (g & 3)) * 2 + half) * kMmTile + 32 * quarter + lane];
        if (!__all_sync(0xffffffffu, got && ok)) {
          ok = false;
          break;
        }
        if constexpr (TWO) {
          if (g == second) {
#pragma unroll
            for (int q = 0; q < kCols / 16; ++q) {
              uint32_t v[16];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                v[2 * j] = __float_as_uint(acc[8 * q + j].x);
                v[2 * j + 1] = __float_as_uint(acc[8 * q + j].y);
                acc[8 * q + j] = make_float2(0.f, 0.f);
              }
              tmem_st_32x32b_x16(t_row + (uint32_t)(kBufs * TN + 16 * q), v);
            }
            tmem_st_wait();
          }
        }
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          tmem_ld_wait_for(r[i & 1]);
          if (i + 1 < kPieces) {
            tmem_ld_32x32b_x32(t_row + (uint32_t)(buf * TN + 32 * (i + 1)), r[(i + 1) & 1]);
          } else {
            // all of the accumulators are read
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
              if (PAIR && !leader)
                mbar_arrive_cluster_relaxed(leaders_tempty + 8 * buf);
              else
                mbar_arrive(&tempty[buf]);
              if ((g & 3) == 3 || g + 1 == g1) mbar_arrive(&sempty[slot]);
            }
            if (++buf == kBufs) {
              buf = 0;
              buf_phase ^= 1u;
            }
            if (left > 0) begin();
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            acc[16 * i + j] = fma2(make_float2(__uint_as_float(r[i & 1][2 * j]), __uint_as_float(r[i & 1][2 * j + 1])),
                                   f2, acc[16 * i + j]);
        }
        if (((g & 3) == 3 || g + 1 == g1) && ++slot == kMmScaleSlots) {
          slot = 0;
          slot_phase ^= 1u;
        }
      }
      if constexpr (TWO) {
#pragma unroll
        for (int q = 0; q < kCols / 16; ++q) {
          uint32_t v[16];
          tmem_ld_32x32b_x16(t_row + (uint32_t)(kBufs * TN + 16 * q), v);
          tmem_ld_wait_for(v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc[8 * q + j] =
                add2(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), acc[8 * q + j]);
        }
      }
      if (PAIR || p.ns == 1) {
        if (ok && any) {
          // to shared memory as 128-byte rows, 16-byte pieces swizzled as TMA has them, and out while the next tile runs
#pragma unroll
          for (int q = 0; q < kCols / 64; ++q) {
            if (p.aligned && lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint32_t v[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = mm_pack(acc[32 * q + 4 * i + j].x, acc[32 * q + 4 * i + j].y);
              *reinterpret_cast<uint4*>(panel + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
            }
            if (p.aligned) fence_proxy_async_shared();
            __syncwarp();
            const int n = n0 + 64 * q;
            if (!p.aligned)
              store_panel(panel, p.y + (size_t)row0 * p.N + n, p.N, min(64, p.N - n), min(32, p.M - row0), lane);
            else if (lane == 0 && n < p.N)
              tma_store_2d(&maps.y, panel, n, row0);
          }
        }
      } else {
        // The tile's columns are dealt to the ranks, TN / ns each.  recv[src][column / 4][row]: four columns a piece,
        // consecutive lanes side by side.  The ring's bytes are free: every MMA that reads them is done before any
        // accumulator of the last group is, and this CTA has one tile.  What a peer sends may come before this CTA's
        // own ring is free, so the receive slots lie behind the ring.
        float4* recv = reinterpret_cast<float4*>(behind);
        const int cols4 = TN / p.ns / 4;
        if (warp == 4 && lane == 0) {
          // the other ranks' sums of this rank's columns, for the rows that exist
          mbar_arrive_expect_tx(&recv_bar, (uint32_t)(p.ns - 1) * cols4 * min(kMmTile, p.M - tr * kTileM) * 16);
        }
#pragma unroll
        for (int j = 0; j < kCols / 4; ++j) {
          const int c4 = c0 / 4 + j, dst = c4 / cols4;
          const int at = ((int)rank * cols4 + c4 - dst * cols4) * kMmTile + 32 * quarter + lane;
          const float4 v = make_float4(acc[2 * j].x, acc[2 * j].y, acc[2 * j + 1].x, acc[2 * j + 1].y);
          if (!mine) continue;
          if (dst == (int)rank)
            recv[at] = v;
          else
            st_async_f4(mapa_shared(smem_u32(recv + at), (uint32_t)dst), v, mapa_shared(smem_u32(&recv_bar), (uint32_t)dst));
        }
        named_bar_sync(1, 256);  // this CTA's own share is there, and the receive barrier is armed
        const bool got = mbar_wait_cluster(&recv_bar, 0, drain_ns);  // (it is also the sums on their way here)
        if (!got) set_error(p.err, kErrTimeout);
        const int tid = threadIdx.x - 128;
        uint8_t* staged = smem;  // where TMA's alignment does not hold: rows of 128 bytes, swizzled, in the free ring
        for (int u = tid; got && u < cols4 * kMmTile; u += 256) {
          const int rl = u & (kMmTile - 1), c4 = u / kMmTile;
          const int m = tr * kTileM + rl, n = tv * TN + ((int)rank * cols4 + c4) * 4;
          if (m >= p.M || n >= p.N) continue;
          // shares by twos, as half as many CTAs have them, and then in rank order
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int q = 0; q < p.ns; q += TWO ? 1 : 2) {
            float4 v = recv[(q * cols4 + c4) * kMmTile + rl];
            if (!TWO) {
              const float4 w = recv[((q + 1) * cols4 + c4) * kMmTile + rl];
              v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
            }
            if (q == 0) {
              s = v;
            } else {
              s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
            }
          }
          const uint2 v = make_uint2(mm_pack(s.x, s.y), mm_pack(s.z, s.w));
          *reinterpret_cast<uint2*>(p.aligned ? reinterpret_cast<uint8_t*>(p.y + (size_t)m * p.N + n)
                                              : staged + rl * 128 + (((c4 >> 1) ^ (rl & 7)) << 4) + (c4 & 1) * 8) = v;
        }
        if (!p.aligned) {
          named_bar_sync(1, 256);
          const int r0 = (warp - 4) * (kMmTile / 8), m = tr * kTileM + r0, n = tv * TN + (int)rank * cols4 * 4;
          if (__all_sync(0xffffffffu, got) && m < p.M)
            store_panel(staged + r0 * 128, p.y + (size_t)m * p.N + n, p.N, min(4 * cols4, p.N - n),
                        min(kMmTile / 8, p.M - m), lane);
        }
      }
    }
    if (!ok && lane == 0) give_up();
    tmem_ld_wait();  // what a wait that ran out left in flight
    if (lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before_sync();
  if (clustered)
    cluster_sync();  // nobody's copies, MMAs or sums go to a CTA that has ended
  else
    __syncthreads();
  if (gave_up) {
    // The copies still in flight land before a CTA ends; nobody issues any more.  A pair's are counted together, on the
    // leader's barriers: there a group that only one of the two asked for is made up for.
    if (threadIdx.x == 0 && leader) {
      const int n = g1 - g0, mine = sent[0], theirs = PAIR ? sent[1] : mine, most = max(mine, theirs);
      for (int q = mine; q < most; ++q)
        mbar_arrive_expect_tx(&full[q % p.stages], group_bytes(first + q / n * step));
      for (int q = theirs; q < most; ++q)
        mbar_complete_tx(&full[q % p.stages], group_bytes(first + q / n * step));
      for (int q = max(0, most - p.stages); q < most; ++q)
        if (!mbar_wait(&full[q % p.stages], (uint32_t)(q / p.stages) & 1u, drain_ns)) set_error(p.err, kErrTimeout);
    }
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after_sync();
    if constexpr (PAIR)
      tmem_dealloc_pair(tmem_base, kTmemCols);
    else
      tmem_dealloc(tmem_base, kTmemCols);
  }
}

// 2-D tensor of bytes [rows, cols] (cols contiguous, a multiple of 16), box = 128 columns x box_rows, 128-byte
// swizzle, zero fill outside the tensor.
bool make_map_bytes(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int round8(int v) { return (v + 7) / 8 * 8; }

template <int TN, bool PAIR, bool TWO>
cudaError_t launch_mm(const uint8_t* x, const uint8_t* w, MmParams p, const DeviceCtx& dc, cudaStream_t s) {
  constexpr int kTileM = PAIR ? 2 * kMmTile : kMmTile, kBox = PAIR ? TN / 2 : TN;
  const int ntn = (p.N + TN - 1) / TN;
  p.nm = (p.M + kTileM - 1) / kTileM;
  p.nitems = p.nm * ntn;
  // Boxes of the last tiles hold what there is: a box that reaches far past its tensor makes every load of it slow.
  // The MMA reads the whole tile; the rows behind a box are what is left of an earlier stage, and their results are
  // never stored.  One row tile alone: the stage is no longer than its box.
  const int tail_m = PAIR ? kMmTile : round8(p.M - (p.nm - 1) * kMmTile);
  const int tail_n = PAIR ? kBox : round8(p.N - (ntn - 1) * TN);
  const int rows = p.nm == 1 ? tail_m : kMmTile;
  p.a_bytes = rows * 128;
  p.a_last = tail_m * 128;
  p.b_last = tail_n * 128;
  p.stage_bytes = p.a_bytes + kBox * 128;
  // behind the ring: the receive slots of a split, or the output's panels; and behind a short stage the MMA reads on, up
  // to a whole tile of rows
  const int behind = kMmScaleBytes + (p.ns > 1 ? kMmTile * TN * 4 : 8 * kMmPanel);
  static_assert(kMmScaleBytes + 8 * kMmPanel >= kMmTile * 128, "room behind the last stage");
  p.stages = (kMmSmem - 1024 - behind) / p.stage_bytes;
  if (p.stages > kMmMaxStages) p.stages = kMmMaxStages;
  const int smem = 1024 + p.stages * p.stage_bytes + behind;
  MmMaps maps;
  if (!make_map_bytes(&maps.x, x, p.M, p.K, (uint32_t)rows) || !make_map_bytes(&maps.w, w, p.N, p.K, kBox))
    return cudaErrorInvalidValue;
  maps.x_last = maps.x;
  maps.w_last = maps.w;
  if ((tail_m != rows && !make_map_bytes(&maps.x_last, x, p.M, p.K, (uint32_t)tail_m)) ||
      (tail_n != kBox && !make_map_bytes(&maps.w_last, w, p.N, p.K, (uint32_t)tail_n)))
    return cudaErrorInvalidValue;
  maps.y = maps.x;
  if (p.aligned && p.ns == 1 && !make_map(&maps.y, p.y, p.M, p.N, 32)) return cudaErrorInvalidValue;
  auto* kernel = q8_matmul_kernel<TN, PAIR, TWO>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem, dc.device);
  if (e != cudaSuccess) return e;
  // a register split above the launch's own would wait for ever
  static std::atomic<bool> split{false};
  if (!split.load(std::memory_order_relaxed)) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kernel);
    if (e != cudaSuccess) return e;
    if (at.numRegs < kMmRegs) return cudaErrorInvalidConfiguration;
    split.store(true, std::memory_order_relaxed);
  }
  const int size = PAIR ? 2 : p.ns;
  const int most = dc.num_sms / size;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size * (p.nitems < most || p.ns > 1 ? p.nitems : most));
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = size;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = size > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

cudaError_t launch_q8_matmul(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw, bf16* y, int M, int N,
                             int K, const DeviceCtx& dc, cudaStream_t s) {
  MmParams p = {};
  p.M = M;
  p.N = N;
  p.K = K;
  p.G = (K + kQ8Group - 1) / kQ8Group;
  p.ns = 1;
  p.aligned = N % 8 == 0;
  p.sx = sx;
  p.sw = sw;
  p.y = y;
  p.err = dc.err;
  p.wait_ns = wait_limit_ns();
  // Pairs save a sixth of the time from some ten groups on and little of few; half of one's rows are idle where the row
  // tiles are odd.  Us with pairs and without: 2440 x 20000 x 1280 71 and 84, x 256 31 and 30; 1100 x 20000 x 1280 40 and 42;
  // 600 x 20000 x 4096 67 and 71, x 512 17 and 15; 300 x 40000 x 1280 35 and 30, 300 x 20000 x 4096 51 and 49.
  const int row_tiles = (M + kMmTile - 1) / kMmTile;
  const long long pairs = (long long)((M + 255) / 256) * ((N + 255) / 256);
  if (row_tiles > 1 && 2 * pairs >= dc.num_sms &&
      (row_tiles % 2 == 0 || (row_tiles > 3 && (long long)row_tiles * p.G >= 64)))
    return launch_mm<256, true, false>(x, w, p, dc, s);
  // A tile's groups over several CTAs, as far as their clusters are on the GPU at once.  A group takes 0.33 us and the
  // exchange 2.5 to 3.  128 x 1280 x K, us with 1, 2, 4 and 8 CTAs: K = 512 4.6, 7.1, 6.3; 1280 6.7, 8.0, 6.7, 7.2; 2048 8.8,
  // 9.0, 7.2, 7.6; 7168 22.6, 15.9, 10.7, 9.2.  Clusters that do not fit at once: 128 x 2048 x 4096 15.3 with 8, 8.9 with 4.
  const long long weight_tiles = (N + 127) / 128, tiles = row_tiles * weight_tiles;
  bool two = false;
  if (p.G >= 12) {
    static ClustersAtOnce at_once;
    const void* split = reinterpret_cast<const void*>(q8_matmul_kernel<128, false, false>);
    const cudaError_t e = ensure_smem_attr(split, kMmSmem, dc.device);
    if (e != cudaSuccess) return e;
    auto fit = [&](long long clusters, int size) {
      return clusters <= at_once.of(split, size, kMmThreads, kMmSmem, dc.device);
    };
    // Up to kMmSameRows the shares that are added up go by N and K alone, as one row tile has them, so that a row's bits do
    // not depend on how many rows there are; where twice as many clusters do not fit, CTAs take two shares each.  It costs
    // 0.9 us and more where the tiles themselves would ask for another split: 256 x 1280 x 7168 12.6 (11.7), 256 x 4096 x
    // 4096 14.1 (12.9), x 1536 10.1 (7.7).  (Pairs, above, have weight tiles for all of the SMs: far more than clusters fit,
    // so that one row tile is not split either.)
    const bool same = M <= kMmSameRows;
    const long long of = same ? weight_tiles : tiles;
    p.ns = p.G >= 24 && fit(of, 8) ? 8 : fit(of, 4) ? 4 : p.G >= 20 && fit(of, 2) ? 2 : 1;
    two = same && p.ns > 1 && !fit(tiles, p.ns);
    if (two) p.ns /= 2;
  }
  return two ? launch_mm<128, false, true>(x, w, p, dc, s) : launch_mm<128, false, false>(x, w, p, dc, s);
}

}  // namespace
}  // namespace lsv

using namespace lsv;

extern "C" lsv_status dense_matmul_q8(const void* x, const float* x_scales, const void* w, const float* w_scales, void* y,
                                      int32_t M, int32_t N, int32_t K, lsv_stream stream) {
  if (M < 0 || N < 0 || K <= 0) return LSV_ERR_INVALID_ARG;
  if (K % 16 || K > kQ8MaxCols || M > kQ8MaxRows || N > kQ8MaxRows ||
      ((long long)M + 127) / 128 * (((long long)N + 127) / 128) >= (1ll << 30))
    return LSV_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return LSV_OK;
  if (!x || !x_scales || !w || !w_scales || !y) return LSV_ERR_INVALID_ARG;
  const void* ptrs[] = {x, x_scales, w, w_scales, y};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 15) return LSV_ERR_MISALIGNED;
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  return launch_q8_matmul(static_cast<const uint8_t*>(x), x_scales, static_cast<const uint8_t*>(w), w_scales,
                          static_cast<bf16*>(y), M, N, K, *dc, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? LSV_OK
             : LSV_ERR_CUDA;
}
