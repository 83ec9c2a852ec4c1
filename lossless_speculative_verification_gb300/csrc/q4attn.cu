// q4attn.cu -- causal attention of the verified positions over the 4-bit paged
// cache (layout: q4.cuh), with query heads that share key heads.
//
// The R = Q * (nh / nkv) query rows of a key head go through m16n8k16 MMAs in
// tiles.  Up to eight rows (NT = 1) are the MMAs' columns and the cached positions
// their rows, S^T = K q^T and O^T = V^T P^T; sixteen (NT = 2) are their rows,
// S = q K^T and O = P V, which needs no transposes and wastes nothing.
//
// Dequantising costs five operations a word of eight codes: a nibble alone in
// the low bits of an f16 is the subnormal n' 2^-24 (n' = n + 8), and 16 times
// that one place higher, so masks alone (and one shift by 8) make MMA operands.
//   keys: the queries are scaled to 2^14 by a power of two of their row, the odd
//   places' share by 1/16; the accumulators start at -8 * 2^-24 * sum(q) of the
//   group, which takes the 8 off; the group's scale multiplies the fp32 sum.
//   values: P times the position's scale is the f16 operand.  sum(P s) of every
//   group, from one more MMA with ones, takes the 8 off every 16 steps, and the
//   rows of the odd places are divided by 16 at the end.
// To keep P s in the range of f16, P is 2^8 at a base, the running maximum of score + exponent of the value scale.
// Where the scales of a step (its positions, both groups) are within 2^8 of each other, one base does for the sum
// of P and for every group: the largest score plus the exponent of the largest scale, at most 2^8 above the largest
// P s.  Elsewhere the sum's base is the largest score, each group's follows the group's own largest P s, and the
// exponent of a scale goes into that of P (wide_step), until the bases are within 2^4 of each other at a step of
// the first kind.  A base follows only where the maximum rises by more than 2^6 (the sums are rescaled in few steps
// then): P s < 2^15, and what loses bits is below 2^-10 of the group's largest term, what is lost below 2^-20.
//
// A CTA's four warps take the steps (32 positions) of one chunk of one key head
// in turn, each from a ring of its own; their states (maximum, sum, output) meet
// in shared memory, those of the chunks as cut_of says.  Which positions are a chunk's goes by the batch, the key
// heads and the capacity, and both forms add in the same order, so in calls of one batch size a row's result does
// not depend on the other rows.
// A step of 16 rows is 580 instructions, 160 of them dequantising; 16 x 32K
// positions of 8 key heads take 131 us, 4.15 TB/s of cache, with 49 % of the issue
// slots, 48 % of the ALU and 45 % of the tensor pipe taken: what bounds it is how
// far three CTAs an SM (168 registers a thread) overlap them.  Where every step is
// a wide one (one group of the values 2^-12 of the other) they take 283 us, where
// one position in 64 is as much smaller 240, one in 4096 136.
#include <limits.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "lsv.h"
#include "ptx.cuh"
#include "q4.cuh"
#include "q4ptx.cuh"

namespace lsv {
namespace {

constexpr int kQaWarps = 4;
constexpr int kQaThreads = kQaWarps * 32;
constexpr float kQaLift = 8.0f;   // log2 of P at the running maximum
constexpr float kQaSlack = 6.0f;  // how far a maximum may rise (log2) before the sums are rescaled
// Value scales (bf16 bits) that one exponent does for: from 2^-64 to 2^64, none more than about 2^8 above another.
constexpr uint32_t kQaScaleLow = (127 - 64) << 7, kQaScaleHigh = (127 + 64) << 7, kQaScaleSpan = 8 << 7;
constexpr float kQaJoin = 4.0f, kQaJoinSum = 64.0f;  // how near (log2) groups' bases, and theirs and the sum's, become one
constexpr float kQaFar = 60.0f;  // how far (log2) a group's base may stand above the sum's in a state
constexpr float kQaLog2e = 1.4426950408889634f;
constexpr uint64_t kQaDrainNs = 2000000000ull;
constexpr int kQaOne = 4, kQaTwo = 3;  // CTAs an SM: up to eight rows, nine to sixteen
constexpr int kQaRound = 32 * kQaWarps;  // positions of a step of a chunk
constexpr int kQaNear = 16;         // steps of chunks that share a CTA, at most
constexpr int kQaCentre = 16;       // steps between two centrings
constexpr int kQaCounters = 16384;  // tiles of rows whose CTAs may be counted; their counters lead the workspace
constexpr int kQaMaxTiles = 8;      // tiles of 16 rows of a key head, at most (8 queries x 16 heads)
constexpr int kQaMaxSteps = 256;    // steps of 128 positions in a chunk, at most: 512 sums in a row in an accumulator

struct QaParams {
  const bf16* q;           // [B, Q, nh, D]
  const uint8_t* pool;
  const int32_t* table;    // [B, M]
  const int32_t* ctx_len;  // [B]
  int B, Q, nh, nkv, grp, R, M, P, page_shift, rblocks;
  int mode;
  int sorted;  // the CTAs take the sequences by falling length
  int nchunk;  // chunks of a sequence
  float scale_log2;   // scale * log2(e)
  bf16* out;          // [B, Q, nh, D]
  int* arrived;       // [B * nkv * rblocks] CTAs that have written their state; 0 before and after a call
  float* o_part;      // [B * nkv, nchunk, R, D]
  float* ml_part;     // [B * nkv, nchunk, R, 2]: maximum (log2 units), sum
  int* err;
  uint64_t wait_ns;
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// How the chunks' states meet: there is one chunk, the chunks' CTAs are a cluster, the last CTA of a tile of rows to
// arrive merges them, or a second kernel does.  (Short ones may be groups of one CTA instead.)
enum : int { kQaDirect = 0, kQaCluster = 1, kQaLast = 2, kQaParts = 3 };
constexpr int kQaWidth = 8, kQaWidthFew = 16;  // chunks of a cluster, at most: where there are many, where few

// A state of four output columns of a row: maximum, sum, unnormalised output.
struct QaState {
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // adds another's (maximum, sum), output; m is the maximum of all already
  __device__ __forceinline__ void add(float2 ml, float4 v) {
    // one that saw nothing adds nothing; one that saw only NaN scores adds them
    const float f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : 1.0f) : ex2_ftz(ml.x - m);
    l = fmaf(ml.y, f, l);
    o.x = fmaf(v.x, f, o.x);
    o.y = fmaf(v.y, f, o.y);
    o.z = fmaf(v.z, f, o.z);
    o.w = fmaf(v.w, f, o.w);
  }
  __device__ __forceinline__ void store(const QaParams& p, int b, int h, int row, int D, int c4) const {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees nothing is zero
    const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
    uint2 v;
    v.x = *reinterpret_cast<const uint32_t*>(&lo);
    v.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(p.out + (((size_t)b * p.Q + row / p.grp) * p.nh + h * p.grp + row % p.grp) * D + 4 * c4) = v;
  }
};

// The chunks' states of four output columns of a row, brought to their common maximum and summed.
constexpr int kQcUnroll = 8;
__device__ __forceinline__ QaState merge_parts(const QaParams& p, int parts, int bh, int row, int D, int c4) {
  const float2* ml = reinterpret_cast<const float2*>(p.ml_part) + (size_t)bh * p.nchunk * p.R;
  const float4* o4 = reinterpret_cast<const float4*>(p.o_part) + (size_t)bh * p.nchunk * p.R * (D / 4);
  QaState all;
  for (int s0 = 0; s0 < parts; s0 += kQcUnroll) {
    float2 a[kQcUnroll];
    float4 v[kQcUnroll];
#pragma unroll
    for (int u = 0; u < kQcUnroll; ++u) {
      const bool in = s0 + u < parts;
      a[u] = in ? __ldcg(ml + (size_t)(s0 + u) * p.R + row) : make_float2(-INFINITY, 0.0f);
      v[u] = in ? __ldcg(o4 + ((size_t)(s0 + u) * p.R + row) * (D / 4) + c4) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    QaState acc;
    acc.m = all.m;
#pragma unroll
    for (int u = 0; u < kQcUnroll; ++u) acc.m = fmaxf(acc.m, a[u].x);
    acc.add(make_float2(all.m, all.l), all.o);
#pragma unroll
    for (int u = 0; u < kQcUnroll; ++u) acc.add(a[u], v[u]);
    all = acc;
  }
  return all;
}

// The range of value scales (bf16 bits); nothing yet.
struct QaRange {
  uint32_t low = 0xFFFFu, high = 0u;
  template <int G>
  __device__ __forceinline__ void add(uint32_t s) {  // a position's scales
    const uint32_t a = s & 0xFFFFu, b = G == 2 ? s >> 16 : a;
    low = min(low, min(a, b));
    high = max(high, max(a, b));
  }
  // One exponent does for them, and so for some or none of them; not for zeros and NaN.
  __device__ __forceinline__ bool near() const {
    return high <= kQaScaleHigh && low >= kQaScaleLow && low + kQaScaleSpan >= high;
  }
};
// Exponent of a normal scale.
__device__ __forceinline__ float exponent_of(uint32_t bits) { return (float)((int)(bits >> 7) - 127); }
// A scale of any kind as mantissa * 2^exponent, the mantissa below 2 (NaN of NaN).
__device__ __forceinline__ float any_exponent(uint32_t bits) {  // (2^23 + the exponent's field) - (2^23 + 127)
  return __uint_as_float(0x4B000000u | max(bits >> 7, 1u)) - 8388735.0f;
}
__device__ __forceinline__ float any_mantissa(float s) {
  const uint32_t bits = __float_as_uint(s), field = bits >> 23;
  return field == 0u ? s * 0x1p126f : field == 255u ? s : __uint_as_float((bits & 0x007FFFFFu) | 0x3F800000u);
}

// The sequence of the given rank by falling length (of equal ones the first comes first), and its length.
__device__ __forceinline__ int2 by_length(const QaParams& p, int rank) {
  __shared__ __align__(16) int len[kQaThreads];
  __shared__ int2 found;
  const int tid = threadIdx.x;
  const int n = tid < p.B ? __ldcg(p.ctx_len + tid) : INT_MIN;
  if (tid < kQaThreads) len[tid] = n;
  __syncthreads();
  if (tid < p.B) {
    int before = 0;
    for (int j = 0; j < p.B; j += 4) {  // (what is behind the last one is not longer than any, and comes later)
      const int4 v = *reinterpret_cast<const int4*>(len + j);
      before += (v.x > n || (v.x == n && j < tid)) + (v.y > n || (v.y == n && j + 1 < tid)) +
                (v.z > n || (v.z == n && j + 2 < tid)) + (v.w > n || (v.w == n && j + 3 < tid));
    }
    if (before == rank) found = make_int2(tid, n);
  }
  __syncthreads();
  return found;
}

// A warp's ring of S stages in shared memory, each the K steps of U blocks that it takes next, filled by untiled
// bulk copies.
template <int D, int NT, int U, int K, int S>
struct QaSmem {
  using L = Q4Block<D>;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStride = D + 4;  // floats between rows of a state, in the ring once it is drained
  static constexpr int kStage = K * U * L::kBytes;
  static constexpr int kRing = S * kStage;
  static constexpr int kMl = kRows * kStride * 4;  // byte offset of (maximum, sum) behind the rows
  static constexpr int kWarp = kRing > kMl + kRows * 8 ? kRing : (kMl + kRows * 8 + 15) / 16 * 16;
  static constexpr int kBars = kQaWarps * kWarp;                     // [warp][S] mbarriers
  static constexpr int kHere = kBars + kQaWarps * S * 8;             // [warp][S] which blocks a stage holds
  static constexpr int kQf = (kHere + kQaWarps * S * 4 + 15) / 16 * 16;  // [W][NT][lane] 16 bytes: the queries
  static constexpr int kCi = kQf + NT * L::W * 512;           // [G][4 or 8] 16 bytes: where the accumulators start
  static constexpr int kFq = kCi + NT * L::G * 64;            // [8 NT] what turns the scaled sums into log2 scores
  static constexpr int kLim = kFq + kRows * 4;                // [8 NT] last position the row sees
  static constexpr int kMlAll = kLim + kRows * 4;             // [8 NT][2] (maximum, sum) of the CTA
  static constexpr int kMg = kMlAll + kRows * 8;              // [warp][G][8 NT] what the groups' sums are relative to
  static constexpr int kTotal = kMg + kQaWarps * L::G * kRows * 4;
};

template <int D, int NT, int U, int K, int S, int kPerSm, int kGroups>
__global__ void __launch_bounds__(kQaThreads * kGroups, kPerSm / kGroups) attn_q4_kernel(const QaParams p) {
  using L = Q4Block<D>;
  using SM = QaSmem<D, NT, U, K, S>;
  constexpr int W = L::W, G = L::G;
  constexpr int kRows = SM::kRows;
  constexpr int kStep = 16 * U;            // positions a warp takes at a time
  constexpr int kBlocks = K * U;           // blocks of a stage
  constexpr int kBatch = 32 / kBlocks;     // stages whose pages the lanes hold
  extern __shared__ __align__(128) uint8_t smem_all[];
  const int group = kGroups > 1 ? (int)threadIdx.x / kQaThreads : 0, tid = (int)threadIdx.x - group * kQaThreads;
  uint8_t* smem = smem_all + group * SM::kTotal;
  auto group_sync = [&]() {
    if (kGroups > 1)
      named_bar_sync(1 + group, kQaThreads);
    else
      __syncthreads();
  };
  const int warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * SM::kWarp;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::kBars) + warp * S;
  int* here = reinterpret_cast<int*>(smem + SM::kHere) + warp * S;
  if (lane < S) mbar_init(&full[lane], 1);
  fence_barrier_init();
  __syncwarp();
  const int tiles = p.nkv * p.rblocks;
  int split = kGroups > 1 ? group : blockIdx.y, b = blockIdx.x / tiles, ht = blockIdx.x - b * tiles, n = 0;
  if (p.sorted) {  // the longest sequence's chunks first
    pdl_wait();
    const int k = blockIdx.y * gridDim.x + blockIdx.x, per = tiles * gridDim.y, rank = k / per;
    if (kGroups == 1) split = (k - rank * per) / tiles;
    ht = k - rank * per - (kGroups == 1 ? split * tiles : 0);
    const int2 s = by_length(p, rank);
    b = s.x;
    n = s.y;
  }
  const int h = ht / p.rblocks, rb = ht - h * p.rblocks, bh = b * p.nkv + h;
  const int r0 = rb * kRows, nrows = min(kRows, p.R - r0);
  const int stride = p.nchunk * kQaRound;
  // step i of this warp is the U blocks from position first + i * stride on, a stage K steps
  const int first = split * kQaRound + warp * kStep;
  const int per_shift = p.page_shift - 4;
  const int cap = p.M << p.page_shift;
  // lane l has block l % kBlocks of stage i + l / kBlocks
  auto pos_of = [&](int i) {
    return first + ((i + lane / kBlocks) * K + lane % kBlocks / U) * stride + 16 * (lane % U);
  };
  auto entry_of = [&](int i) {
    const int pos = pos_of(i);
    return pos < cap ? __ldcg(p.table + (size_t)b * p.M + (pos >> p.page_shift)) : -1;
  };
  if (!p.sorted) {
    pdl_wait();
    n = __ldcg(p.ctx_len + b);
  }
  pdl_trigger();
  int pg_now = entry_of(0);  // beside the length's load, before it is known how many of them there are

  // ---- the queries: warp w < NT makes the operands of tile w; column g is row r0 + 8 w + g, of which this lane
  // has the dims 32 j + 8 t + 0..7
  uint4 xq[W];
  const int qr = 8 * warp + g;
#pragma unroll
  for (int j = 0; j < W; ++j)
    xq[j] = warp < NT && qr < nrows
                ? __ldg(reinterpret_cast<const uint4*>(
                      p.q + (((size_t)b * p.Q + (r0 + qr) / p.grp) * p.nh + h * p.grp + (r0 + qr) % p.grp) * D + 32 * j + 8 * t))
                : make_uint4(0u, 0u, 0u, 0u);

  const bool bad = n < 0 || n > (p.M << p.page_shift);
  if (bad && tid == 0 && split == 0 && h == 0 && rb == 0) set_error(p.err, kErrDeviceIndex);
  const int end = bad ? 0 : n;
  const int parts = bad ? 0 : min((n + kQaRound - 1) / kQaRound, p.nchunk);
  if (kGroups == 1 && p.mode >= kQaLast && split >= max(parts, 1)) return;  // nobody reads a state of it

  // ---- the ring
  const int nsteps = first < end ? (end - first + stride - 1) / stride : 0;
  const int nstages = (nsteps + K - 1) / K;
  auto checked = [&](int pg, int i) {  // the page of this lane's block, -1: none
    if (pos_of(i) >= end) return -1;
    if (pg >= 0 && pg < p.P) return pg;
    set_error(p.err, kErrDeviceIndex);
    return -1;
  };
  pg_now = checked(pg_now, 0);
  int pg_next = -1;
  auto issue = [&](int i, int s) {  // all lanes: stage i of the warp into stage s of the ring
    const int k = i % kBatch;
    if (k == 0) {
      if (i > 0) pg_now = checked(pg_next, i);
      pg_next = entry_of(i + kBatch);
    }
    const int l = lane % kBlocks, pg = __shfl_sync(0xffffffffu, pg_now, k * kBlocks + l);
    const uint32_t there = __ballot_sync(0xffffffffu, lane < kBlocks && pg >= 0);
    if (lane == 0) {
      here[s] = there;
      mbar_arrive_expect_tx(&full[s], __popc(there) * L::kBytes);
    }
    __syncwarp();
    if (there >> lane & 1u) {
      const int blk = ((first + (i * K + l / U) * stride) >> 4) + l % U;
      bulk_load(ring + s * SM::kStage + l * L::kBytes,
                p.pool + ((((size_t)pg * p.nkv + h) << per_shift) + (blk & ((1 << per_shift) - 1))) * L::kBytes, L::kBytes,
                &full[s]);
    }
  };
  // every warp's first stage before anyone's second: with all stages at once the first arrives behind the others'
  // later ones (32 x 4 positions over page-shaped caches: after 4.0 us)
  if (nstages > 0) issue(0, 0);

  uint8_t* qs = smem;
  if (warp < NT) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < W; ++j)
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(xq[j].x & 0x7FFF7FFFu, xq[j].y & 0x7FFF7FFFu),
                               __vmaxu2(xq[j].z & 0x7FFF7FFFu, xq[j].w & 0x7FFF7FFFu)));
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // the largest of the row to 2^14 .. 2^15 (a row below 2^-112 keeps what 2^126 gives it)
    const int e = (int)(m >> 7) - 127;
    const int k = m == 0 ? 0 : min(14 - e, 126);
    const float f = __uint_as_float((uint32_t)(k + 127) << 23);
    float sum[G];
#pragma unroll
    for (int gr = 0; gr < G; ++gr) sum[gr] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const uint32_t xs[4] = {xq[j].x, xq[j].y, xq[j].z, xq[j].w};
      uint32_t v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float fo = (q & 1) ? f * 0.0625f : f;
        v[q] = pack_f16(__uint_as_float(xs[q] << 16) * fo, __uint_as_float(xs[q] & 0xFFFF0000u) * fo);
        const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&v[q]));
        sum[j >> 1] += (back.x + back.y) * ((q & 1) ? 16.0f : 1.0f);
      }
      // NT = 1: the B operands of both halves of a word; NT = 2: the A operands of each, rows g and g + 8 by turns
      if constexpr (NT == 1) {
        *reinterpret_cast<uint4*>(qs + SM::kQf + (j * 32 + lane) * 16) = make_uint4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint32_t*>(qs + SM::kQf + ((2 * j + (q >> 1)) * 32 + lane) * 16 + (2 * (q & 1) + warp) * 4) = v[q];
      }
    }
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 1);
      sum[gr] += __shfl_xor_sync(0xffffffffu, sum[gr], 2);
      // the accumulators start at -8 * 2^-24 * sum of the group's queries: those of the columns 2t', 2t' + 1 twice
      // (NT = 1), or of the row g and the row g + 8 twice each
      float* ci = reinterpret_cast<float*>(qs + SM::kCi + (NT == 1 ? gr * 4 + (g >> 1) : gr * 8 + g) * 16);
      if (t < 2) ci[NT == 1 ? 2 * t + (g & 1) : 2 * warp + t] = sum[gr] * (-8.0f / 16777216.0f);
    }
    if (t == 0) {
      reinterpret_cast<float*>(qs + SM::kFq)[qr] =
          m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : ldexpf(p.scale_log2, 24 - k);
      reinterpret_cast<int*>(qs + SM::kLim)[qr] = qr < nrows ? n - p.Q + (r0 + qr) / p.grp : -1;
    }
  }
  group_sync();
#pragma unroll 1
  for (int i = 1; i < S && i < nstages; ++i) issue(i, i);
  __syncwarp();
  // this lane's two rows: the columns 2t, 2t + 1 (NT = 1), or the rows g and g + 8
  const int row_a = NT == 1 ? 2 * t : g, row_b = NT == 1 ? 2 * t + 1 : g + 8;
  const float fq[2] = {*reinterpret_cast<const float*>(qs + SM::kFq + row_a * 4),
                       *reinterpret_cast<const float*>(qs + SM::kFq + row_b * 4)};

  // NT = 1: tiles of 16 dims, rows g (even places) and g + 8 (odd places), columns 2t, 2t + 1 the query rows.
  // NT = 2: tiles of 8 dims, [4 m + place] column c the dim 32 m + 4 c + place, rows g and g + 8 the query rows.
  constexpr int kTiles = NT == 1 ? 2 * W : 4 * W;
  float o[kTiles][4];
  float cs[G][4];  // sum of P s of every group
  float m_run[2] = {-INFINITY, -INFINITY}, nbase[2] = {0.0f, 0.0f};  // -nbase: what P is 2^0 at
  float l_run[2][NT] = {};  // sums of P over this lane's positions (NT = 2: the even and the odd ones apart, so
                            // that both forms add in the same order)
#pragma unroll
  for (int i = 0; i < kTiles; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.0f;
#pragma unroll
  for (int gr = 0; gr < G; ++gr)
#pragma unroll
    for (int c = 0; c < 4; ++c) cs[gr][c] = 0.0f;

  // One step: the U blocks of a stage from position pos0 on.  Element c of the scores' tile (u, e): NT = 1 (e = 0):
  // position g + 8 (c / 2) and row c % 2; NT = 2: position 8 e + 2t + c % 2 and row c / 2, of this lane's.
  auto row_of = [](int c) { return NT == 1 ? (c & 1) : (c >> 1); };
  auto place_of = [&](int e, int c) { return NT == 1 ? g + 8 * (c >> 1) : 8 * e + 2 * t + (c & 1); };
  // the scales that the elements c and c + 1 of a tile are of
  auto scales_of = [](const uint32_t (&w)[2][G == 2 ? 2 : 1], int e, int c, int gr) {
    if (NT == 1) {
      const float s = q4_scale(w[c >> 1][0], gr);
      return make_float2(s, s);
    }
    return G == 2 ? make_float2(q4_scale(w[e][0], gr), q4_scale(w[e][G - 1], gr))
                  : make_float2(q4_scale(w[e][0], 0), q4_scale(w[e][0], 1));
  };
  // over the lanes that hold a row's elements
  auto row_max = [](auto v, auto f) {
#pragma unroll
    for (int sh = NT == 1 ? 4 : 1; sh < (NT == 1 ? 32 : 4); sh <<= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, sh));
    return v;
  };
  auto larger = [](auto a, auto b) { return max(a, b); };
  auto smaller = [](auto a, auto b) { return min(a, b); };

  // ---- scores, before the row's factor
  auto scores = [&](const uint8_t* blk, float (&x)[U][NT][4]) {
    Q4Words<W> kw[U][2];
    uint32_t ks[U][2][G == 2 ? 2 : 1];  // scales of this lane's positions: G = 2 [position], G = 1 both in one
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint8_t* bk = blk + u * L::kBytes;
        kw[u][e] = q4_load<W>(bk + (32 * e + lane) * (4 * W));
        if constexpr (NT == 1) {
          ks[u][e][0] = q4_load_scales<G>(bk + L::kKs + (g + 8 * e) * 2 * G);
        } else if constexpr (G == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(bk + L::kKs + (8 * e + 2 * t) * 4);
          ks[u][e][0] = v.x, ks[u][e][1] = v.y;
        } else {
          ks[u][e][0] = *reinterpret_cast<const uint32_t*>(bk + L::kKs + (8 * e + 2 * t) * 2);
        }
      }
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      const float4 sv = *reinterpret_cast<const float4*>(qs + SM::kCi + (NT == 1 ? gr * 4 + t : gr * 8 + g) * 16);
      float start[4] = {sv.x, sv.y, sv.z, sv.w};
      float acc[U][NT][4];
#pragma unroll
      for (int j = 2 * gr; j < 2 * gr + 2; ++j) {
        uint4 qf[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) qf[i] = *reinterpret_cast<const uint4*>(qs + SM::kQf + ((NT * j + i) * 32 + lane) * 16);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if constexpr (NT == 1) {
            const uint32_t a = kw[u][0].w[j], c = kw[u][1].w[j], a8 = a >> 8, c8 = c >> 8;
            mma_f16_m16n8k16(acc[u][0], a & 0x000F000Fu, c & 0x000F000Fu, a & 0x00F000F0u, c & 0x00F000F0u, qf[0].x,
                             qf[0].y, j == 2 * gr ? start : acc[u][0]);
            mma_f16_m16n8k16(acc[u][0], a8 & 0x000F000Fu, c8 & 0x000F000Fu, a8 & 0x00F000F0u, c8 & 0x00F000F0u,
                             qf[0].z, qf[0].w, acc[u][0]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t a = kw[u][e].w[j], a8 = a >> 8;
              mma_f16_m16n8k16(acc[u][e], qf[0].x, qf[0].y, qf[0].z, qf[0].w, a & 0x000F000Fu, a & 0x00F000F0u,
                               j == 2 * gr ? start : acc[u][e]);
              mma_f16_m16n8k16(acc[u][e], qf[NT - 1].x, qf[NT - 1].y, qf[NT - 1].z, qf[NT - 1].w, a8 & 0x000F000Fu,
                               a8 & 0x00F000F0u, acc[u][e]);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
          for (int c = 0; c < 4; c += 2) {
            const float2 s = scales_of(ks[u], e, c, gr), a = make_float2(acc[u][e][c], acc[u][e][c + 1]);
            const float2 v = gr == 0 ? mul2(a, s) : fma2(a, s, make_float2(x[u][e][c], x[u][e][c + 1]));
            x[u][e][c] = v.x, x[u][e][c + 1] = v.y;
          }
    }
  };

  // ---- the weighted values: weigh(u, e, gr, scales, w) gives the tile's weights P s of group gr
  auto values = [&](const uint8_t* blk, auto weigh) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint8_t* bk = blk + u * L::kBytes;
      const Q4Words<W> v0 = q4_load<W>(bk + L::kV + lane * (4 * W)), v1 = q4_load<W>(bk + L::kV + (32 + lane) * (4 * W));
      uint32_t vs[2][G == 2 ? 2 : 1];  // like ks
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (NT == 1) {
          vs[e][0] = q4_load_scales<G>(bk + L::kVs + (g + 8 * e) * 2 * G);
        } else if constexpr (G == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(bk + L::kVs + (8 * e + 2 * t) * 4);
          vs[e][0] = v.x, vs[e][1] = v.y;
        } else {
          vs[e][0] = *reinterpret_cast<const uint32_t*>(bk + L::kVs + (8 * e + 2 * t) * 2);
        }
      }
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        uint32_t pp[NT][2];  // P s in f16: [e][row pair]
#pragma unroll
        for (int e = 0; e < NT; ++e) {
          float w[4];
          weigh(u, e, gr, vs, w);
          pp[e][0] = pack_f16(w[0], w[1]);
          pp[e][1] = pack_f16(w[2], w[3]);
        }
        if constexpr (NT == 1) {
          const uint32_t b0 = movmatrix_trans(pp[0][0]), b1 = movmatrix_trans(pp[0][1]);
          mma_f16_m16n8k16(cs[gr], 0x3C003C00u, 0u, 0x3C003C00u, 0u, b0, b1, cs[gr]);
#pragma unroll
          for (int m = 2 * gr; m < 2 * gr + 2; ++m) {
            const uint32_t a = v0.w[m], c = v1.w[m], a8 = a >> 8, c8 = c >> 8;
            mma_f16_m16n8k16(o[2 * m], a & 0x000F000Fu, a & 0x00F000F0u, c & 0x000F000Fu, c & 0x00F000F0u, b0, b1, o[2 * m]);
            mma_f16_m16n8k16(o[2 * m + 1], a8 & 0x000F000Fu, a8 & 0x00F000F0u, c8 & 0x000F000Fu, c8 & 0x00F000F0u, b0, b1,
                             o[2 * m + 1]);
          }
        } else {
          const uint32_t a0 = pp[0][0], a1 = pp[0][1], a2 = pp[NT - 1][0], a3 = pp[NT - 1][1];
          mma_f16_m16n8k16(cs[gr], a0, a1, a2, a3, 0x3C003C00u, 0x3C003C00u, cs[gr]);
#pragma unroll
          for (int m = 2 * gr; m < 2 * gr + 2; ++m) {
            const uint32_t a = v0.w[m], c = v1.w[m], a8 = a >> 8, c8 = c >> 8;
            mma_f16_m16n8k16(o[4 * m], a0, a1, a2, a3, a & 0x000F000Fu, c & 0x000F000Fu, o[4 * m]);
            mma_f16_m16n8k16(o[4 * m + 1], a0, a1, a2, a3, a & 0x00F000F0u, c & 0x00F000F0u, o[4 * m + 1]);
            mma_f16_m16n8k16(o[4 * m + 2], a0, a1, a2, a3, a8 & 0x000F000Fu, c8 & 0x000F000Fu, o[4 * m + 2]);
            mma_f16_m16n8k16(o[4 * m + 3], a0, a1, a2, a3, a8 & 0x00F000F0u, c8 & 0x00F000F0u, o[4 * m + 3]);
          }
        }
      }
    }
  };

  // The elements' positions that their rows do not see (bit 8 u + 4 e + c), as every lane's row limits say.
  auto hidden_of = [&](int pos0, int gone) {
    const int lim[2] = {*reinterpret_cast<const int*>(qs + SM::kLim + row_a * 4),
                        *reinterpret_cast<const int*>(qs + SM::kLim + row_b * 4)};
    uint32_t hidden = 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < NT; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (pos0 + 16 * u + place_of(e, c) > lim[row_of(c)] || (gone >> u & 1)) hidden |= 1u << (8 * u + 4 * e + c);
    return hidden;
  };
  auto scale_at = [&](const uint8_t* blk, int u, int e, int c) {
    return q4_load_scales<G>(blk + u * L::kBytes + L::kVs + place_of(e, c) * 2 * G);
  };

  // Softmax and values of a step whose scales are near each other.  Masked: some row does not see all of it, or a block
  // is not there.  big: the largest scale of the step.
  auto step = [&](auto tag, const uint8_t* blk, int pos0, int gone, uint32_t all_big, float (&x)[U][NT][4]) {
    constexpr bool kMasked = decltype(tag)::value;
    uint32_t hidden = 0;
    uint32_t big[2] = {all_big, all_big};  // of what the row sees
    if (kMasked) {
      hidden = hidden_of(pos0, gone);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        QaRange seen;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < NT; ++e)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (row_of(c) == r && !(hidden >> (8 * u + 4 * e + c) & 1u)) seen.add<G>(scale_at(blk, u, e, c));
        big[r] = row_max(seen.high, larger);
      }
    }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < NT; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!kMasked || !(hidden >> (8 * u + 4 * e + c) & 1u)) top[row_of(c)] = fmaxf(top[row_of(c)], x[u][e][c]);
#pragma unroll
    for (int r = 0; r < 2; ++r) top[r] = fmaf(row_max(top[r], larger), fq[r], exponent_of(big[r]));
    if (__any_sync(0xffffffffu, top[0] > m_run[0] + kQaSlack || top[1] > m_run[1] + kQaSlack)) {
      float corr[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float m = top[r] > m_run[r] + kQaSlack ? top[r] : m_run[r];
        corr[r] = m == -INFINITY ? 1.0f : ex2_ftz(m_run[r] - m);
        m_run[r] = m;
        nbase[r] = m == -INFINITY ? 0.0f : kQaLift - m;
#pragma unroll
        for (int i = 0; i < NT; ++i) l_run[r][i] *= corr[r];
      }
#pragma unroll
      for (int gr = 0; gr < G; ++gr)
#pragma unroll
        for (int c = 0; c < 4; ++c) cs[gr][c] *= corr[row_of(c)];
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][c] *= corr[row_of(c)];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < NT; ++e)
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          const int ra = row_of(c), rb = row_of(c + 1);
          const float2 at = fma2(make_float2(x[u][e][c], x[u][e][c + 1]), make_float2(fq[ra], fq[rb]),
                                 make_float2(nbase[ra], nbase[rb]));
          float2 v = make_float2(ex2_ftz(at.x), ex2_ftz(at.y));
          if (kMasked && (hidden >> (8 * u + 4 * e + c) & 1u)) v.x = 0.0f;
          if (kMasked && (hidden >> (8 * u + 4 * e + c + 1) & 1u)) v.y = 0.0f;
          x[u][e][c] = v.x, x[u][e][c + 1] = v.y;
          float &la = l_run[ra][0], &lb = l_run[rb][NT - 1];
          const float2 l = add2(make_float2(la, lb), v);
          la = l.x, lb = l.y;
        }
    values(blk, [&](int u, int e, int gr, const uint32_t (&vs)[2][G == 2 ? 2 : 1], float (&w)[4]) {
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        const float2 v = mul2(make_float2(x[u][e][c], x[u][e][c + 1]), scales_of(vs, e, c, gr));
        w[c] = v.x, w[c + 1] = v.y;
        if (kMasked && (hidden >> (8 * u + 4 * e + c) & 1u)) w[c] = 0.0f;  // whatever the scale is
        if (kMasked && (hidden >> (8 * u + 4 * e + c + 1) & 1u)) w[c + 1] = 0.0f;
      }
    });
  };

  // The same where they are not, or were not in some step before: the sum of P and the sums of each group have a base
  // of their own, m_run for the first and in shared memory for the others.  Bases that have come near each other become
  // one again at a step whose scales are near each other.  All that goes by the row alone: one whose bases are one gets
  // what `step` gives it at such a step, whatever the rows beside it need.
  float* bases = reinterpret_cast<float*>(smem + SM::kMg) + warp * G * kRows;  // [G][kRows], of use where `wide`
  bool wide = false;
  auto wide_step = [&](auto tag, const uint8_t* blk, int pos0, int gone, bool all_near, uint32_t all_big,
                       const float (&x)[U][NT][4]) {
    constexpr bool kMasked = decltype(tag)::value;
    const uint32_t hidden = kMasked ? hidden_of(pos0, gone) : 0u;
    QaRange seen[2];
    float top[2] = {-INFINITY, -INFINITY}, top_g[G][2];
#pragma unroll
    for (int gr = 0; gr < G; ++gr) top_g[gr][0] = top_g[gr][1] = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < NT; ++e)
#pragma unroll
        for (int j = 0; j < 2; ++j) {  // this lane's positions, each of both rows
          const uint32_t s = scale_at(blk, u, e, NT == 1 ? 2 * j : j);
          float ex[G];  // nothing is relative to zeros and NaN
#pragma unroll
          for (int gr = 0; gr < G; ++gr) {
            const uint32_t sg = gr ? s >> 16 : s & 0xFFFFu;
            ex[gr] = sg == 0u || sg >= 0x7F80u ? -INFINITY : any_exponent(sg);
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int c = NT == 1 ? 2 * j + r : 2 * r + j;
            if (kMasked && (hidden >> (8 * u + 4 * e + c) & 1u)) continue;
            if (kMasked) seen[r].add<G>(s);
            top[r] = fmaxf(top[r], x[u][e][c]);
#pragma unroll
            for (int gr = 0; gr < G; ++gr) top_g[gr][r] = fmaxf(top_g[gr][r], fmaf(x[u][e][c], fq[r], ex[gr]));
          }
        }
    bool one[2];  // one base for all sums of the row
    float corr_g[G][2], nbase_g[G][2];
    bool apart = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = r ? row_b : row_a;
      if (kMasked) {
        seen[r].low = row_max(seen[r].low, smaller);
        seen[r].high = row_max(seen[r].high, larger);
      }
      const bool near = kMasked ? seen[r].near() : all_near, nothing = kMasked && seen[r].low == 0xFFFFu;
      top[r] = row_max(top[r], larger);
      const float near_top = fmaf(top[r], fq[r], exponent_of(kMasked ? seen[r].high : all_big));
      float m_g[G], most = -INFINITY, least = INFINITY;
      one[r] = near;
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        top_g[gr][r] = row_max(top_g[gr][r], larger);
        m_g[gr] = wide ? bases[gr * kRows + row] : m_run[r];
        one[r] = one[r] && m_g[gr] == m_run[r];
        most = fmaxf(most, fmaxf(m_g[gr], near_top));
        least = fminf(least, fmaxf(m_g[gr], near_top));
      }
      const bool join = near && !nothing && !one[r] && most - least <= kQaJoin && fabsf(most - m_run[r]) <= kQaJoinSum;
      const float up = one[r] ? near_top : top[r] * fq[r], m = join ? most : up > m_run[r] + kQaSlack ? up : m_run[r];
      const float corr = m == -INFINITY ? 1.0f : ex2_ftz(m_run[r] - m);
      m_run[r] = m;
      nbase[r] = m == -INFINITY ? 0.0f : kQaLift - m;
#pragma unroll
      for (int i = 0; i < NT; ++i) l_run[r][i] *= corr;
      one[r] = one[r] || join;
#pragma unroll
      for (int gr = 0; gr < G; ++gr) {
        const float mg = one[r] ? m : top_g[gr][r] > m_g[gr] + kQaSlack ? top_g[gr][r] : m_g[gr];
        corr_g[gr][r] = mg == -INFINITY ? 1.0f : ex2_ftz(m_g[gr] - mg);
        nbase_g[gr][r] = mg == -INFINITY ? 0.0f : kQaLift - mg;
        bases[gr * kRows + row] = mg;  // (every lane of the row writes the same)
        apart = apart || mg != m;
      }
    }
    __syncwarp();
    wide = __any_sync(0xffffffffu, apart);
#pragma unroll
    for (int gr = 0; gr < G; ++gr)
#pragma unroll
      for (int c = 0; c < 4; ++c) cs[gr][c] *= corr_g[gr][row_of(c)];
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] *= corr_g[(NT == 1 ? i / 2 : i / 4) >> 1][row_of(c)];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < NT; ++e)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = row_of(c);
          const float v = ex2_ftz(fmaf(x[u][e][c], fq[r], nbase[r]));
          if (!kMasked || !(hidden >> (8 * u + 4 * e + c) & 1u)) l_run[r][NT == 1 ? 0 : c & 1] += v;
        }
    values(blk, [&](int u, int e, int gr, const uint32_t (&vs)[2][G == 2 ? 2 : 1], float (&w)[4]) {
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        const float2 s2 = scales_of(vs, e, c, gr);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // the scale's exponent goes into that of P: neither alone need be in the range of fp32
          const int r = row_of(c + i);
          const float s = i ? s2.y : s2.x, ex = any_exponent(__float_as_uint(s) >> 16), mant = any_mantissa(s);
          const float p = ex2_ftz(fmaf(x[u][e][c + i], fq[r], one[r] ? nbase_g[gr][r] : nbase_g[gr][r] + ex));
          w[c + i] = s == 0.0f || (kMasked && (hidden >> (8 * u + 4 * e + c + i) & 1u)) ? 0.0f : p * (one[r] ? s : mant);
        }
      }
    });
  };

  // Takes the 8 of the nibbles off what is summed so far.  Left to the end, the sums of n + 8 of a long chunk would
  // be hundreds of times those of n, and lose as many times their last bit (32768 positions of about equal weight:
  // 7.2e-3 of the output, against 1.7e-3 of its own rounding).
  auto centre = [&]() {
    constexpr float kEven = -8.0f / 16777216.0f, kOdd = -8.0f / 1048576.0f;
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool odd = NT == 1 ? c >= 2 : (i & 1) != 0;
        const int gr = (NT == 1 ? i / 2 : i / 4) >> 1;
        o[i][c] = fmaf(cs[gr][NT == 1 ? (c & 1) : 2 * (c >> 1)], odd ? kOdd : kEven, o[i][c]);
      }
#pragma unroll
    for (int gr = 0; gr < G; ++gr)
#pragma unroll
      for (int c = 0; c < 4; ++c) cs[gr][c] = 0.0f;
  };

  int done = 0, st = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (; done < nstages; ++done) {
    if (!__all_sync(0xffffffffu, mbar_wait(&full[st], phase, p.wait_ns))) {
      if (lane == 0) set_error(p.err, kErrTimeout);
      break;
    }
    const int there = here[st];
#pragma unroll 1
    for (int k = 0; k < K && done * K + k < nsteps; ++k) {
      const uint8_t* blk = ring + st * SM::kStage + k * (U * L::kBytes);
      const int pos0 = first + (done * K + k) * stride;
      const int gone = ~(there >> (k * U)) & ((1 << U) - 1);  // blocks behind the end, or of a page out of range
      const bool masked = pos0 + kStep - 1 > n - p.Q || gone;
      float x[U][NT][4];
      if (NT == 1) scores(blk, x);  // (page-shaped caches 20.6 us with the scales first; for sixteen rows 130.6, scores first 137)
      QaRange seen;  // by the row that sees most; lane l has position l of two blocks
#pragma unroll
      for (int u = 0; u < U; u += 2) {
        const int ub = U == 1 ? 0 : u + (lane >> 4), at = 16 * ub + (lane & 15);
        const uint32_t s = q4_load_scales<G>(blk + ub * L::kBytes + L::kVs + (lane & 15) * 2 * G);
        if (!masked || (pos0 + at < n && !(gone >> ub & 1))) seen.add<G>(s);
      }
      seen.high = __reduce_max_sync(0xffffffffu, seen.high);
      const bool near = __all_sync(0xffffffffu, seen.near());
      if (NT != 1) scores(blk, x);
      if (__builtin_expect(!near || wide, 0)) {
        // (one form of it where calls are short: what they do not run costs them too, one token 5.05 us, with both 5.2,
        // with neither 4.9)
        if (NT == 1 || masked)
          wide_step(std::true_type{}, blk, pos0, gone, near, seen.high, x);
        else
          wide_step(std::false_type{}, blk, pos0, 0, near, seen.high, x);
      } else if (masked)
        step(std::true_type{}, blk, pos0, gone, seen.high, x);
      else
        step(std::false_type{}, blk, pos0, 0, seen.high, x);
      if ((done * K + k) % kQaCentre == kQaCentre - 1) centre();
    }
    __syncwarp();  // every lane has read the stage
    if (done + S < nstages) issue(done + S, st);
    if (++st == S) {
      st = 0;
      phase ^= 1u;
    }
  }
  // after a wait that ran out: the copies already issued land before the memory is used again (however short the
  // caller's limit is)
  for (int i = done; i < nstages && i < done + S; ++i)
    mbar_wait(&full[i % S], (i / S) & 1, p.wait_ns > kQaDrainNs ? p.wait_ns : kQaDrainNs);
  __syncwarp();

  // ---- the warp's state, in its drained ring
  float* o_w = reinterpret_cast<float*>(ring);
  float* ml_w = reinterpret_cast<float*>(ring + SM::kMl);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = r ? row_b : row_a;
    float l = l_run[r][0], m = m_run[r], back[G];
#pragma unroll
    for (int gr = 0; gr < G; ++gr) back[gr] = 1.0f;
    float back_l = 1.0f;
    if (wide) {  // one base again: the sum's, or as near below the largest group's as keeps the outputs finite
#pragma unroll
      for (int gr = 0; gr < G; ++gr) m = fmaxf(m, bases[gr * kRows + row] - kQaFar);
      if (m != -INFINITY) {
        back_l = ex2_ftz(m_run[r] - m);
#pragma unroll
        for (int gr = 0; gr < G; ++gr) back[gr] = ex2_ftz(bases[gr * kRows + row] - m);
      }
    }
    if constexpr (NT == 1) {
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      if (g == 0) *reinterpret_cast<float2*>(ml_w + 2 * row) = make_float2(m, l * back_l);
    } else {
      l += l_run[r][NT - 1];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (t == 0) *reinterpret_cast<float2*>(ml_w + 2 * row) = make_float2(m, l * back_l);
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = back[w >> 1], off = -8.0f * cs[w >> 1][NT == 1 ? r : 2 * r];
      constexpr float kEven = 16777216.0f, kOdd = 1048576.0f;
      if constexpr (NT == 1) {
        *reinterpret_cast<float4*>(o_w + row * SM::kStride + 32 * w + 4 * g) =
            make_float4(fmaf(o[2 * w][r], kEven, off) * f, fmaf(o[2 * w][r + 2], kOdd, off) * f,
                        fmaf(o[2 * w + 1][r], kEven, off) * f, fmaf(o[2 * w + 1][r + 2], kOdd, off) * f);
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *reinterpret_cast<float4*>(o_w + row * SM::kStride + 32 * w + 8 * t + 4 * c) =
              make_float4(fmaf(o[4 * w][2 * r + c], kEven, off) * f, fmaf(o[(4 * w + 1) % kTiles][2 * r + c], kOdd, off) * f,
                          fmaf(o[(4 * w + 2) % kTiles][2 * r + c], kEven, off) * f,
                          fmaf(o[(4 * w + 3) % kTiles][2 * r + c], kOdd, off) * f);
      }
    }
  }
  group_sync();
  for (int i = tid; i < nrows * (D / 4); i += kQaThreads) {
    const int r = i / (D / 4), c4 = i - r * (D / 4), row = r0 + r;
    float2 ml[kQaWarps];
    float4* at0 = reinterpret_cast<float4*>(smem + (r * SM::kStride + 4 * c4) * 4);
    QaState acc;
#pragma unroll
    for (int w = 0; w < kQaWarps; ++w) {
      ml[w] = *reinterpret_cast<const float2*>(smem + w * SM::kWarp + SM::kMl + 8 * r);
      acc.m = fmaxf(acc.m, ml[w].x);
    }
#pragma unroll
    for (int w = 0; w < kQaWarps; ++w) acc.add(ml[w], *(at0 + w * (SM::kWarp / 16)));
    if (kGroups == 1 && (p.mode == kQaDirect || (p.mode == kQaLast && parts <= 1))) {
      acc.store(p, b, h, row, D, c4);
    } else if (kGroups == 1 && p.mode != kQaCluster) {
      const size_t at = ((size_t)bh * p.nchunk + split) * p.R + row;
      *reinterpret_cast<float4*>(p.o_part + at * D + 4 * c4) = acc.o;
      if (c4 == 0) *reinterpret_cast<float2*>(p.ml_part + at * 2) = make_float2(acc.m, acc.l);
    } else {
      *at0 = acc.o;  // nobody else reads this place of warp 0's state
      if (c4 == 0) *reinterpret_cast<float2*>(smem + SM::kMlAll + 8 * r) = make_float2(acc.m, acc.l);
    }
  }
  if constexpr (kGroups > 1) {  // the chunks are the CTA's groups
    __syncthreads();
    const int live = max(1, parts);
    for (int i = threadIdx.x; i < nrows * (D / 4); i += kQaThreads * kGroups) {
      const int r = i / (D / 4), c4 = i - r * (D / 4);
      float2 ml[kGroups];
      QaState acc;
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        ml[k] = k < live ? *reinterpret_cast<const float2*>(smem_all + k * SM::kTotal + SM::kMlAll + 8 * r)
                         : make_float2(-INFINITY, 0.0f);
        acc.m = fmaxf(acc.m, ml[k].x);
      }
#pragma unroll
      for (int k = 0; k < kGroups; ++k)
        if (k < live)
          acc.add(ml[k], *reinterpret_cast<const float4*>(smem_all + k * SM::kTotal + (r * SM::kStride + 4 * c4) * 4));
      acc.store(p, b, h, r0 + r, D, c4);
    }
    return;
  }
  if constexpr (NT == 1) {
    if (p.mode == kQaLast && parts > 1) {
      __shared__ int last;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        int* count = p.arrived + bh;  // (up to eight rows are one tile)
        last = atomicAdd(count, 1) == parts - 1;
        if (last) *count = 0;  // as the next call wants it
      }
      __syncthreads();
      if (!last) return;
      __threadfence();
      for (int i = threadIdx.x; i < nrows * (D / 4); i += kQaThreads) {
        const int r = i / (D / 4), c4 = i - r * (D / 4);
        merge_parts(p, parts, bh, r0 + r, D, c4).store(p, b, h, r0 + r, D, c4);
      }
    }
  }
  if (p.mode != kQaCluster) return;
  // ---- the chunks' CTAs are a cluster: each takes a share of the outputs and reads it from all of them
  cluster_sync();
  const int live = max(1, parts);
  if (split < live) {
    const uint32_t mine = smem_u32(smem);
    for (int i = split * kQaThreads + threadIdx.x; i < nrows * (D / 4); i += live * kQaThreads) {
      const int r = i / (D / 4), c4 = i - r * (D / 4);
      QaState acc;
      float2 ml[kQcUnroll];
      float4 v[kQcUnroll];
      auto take = [&](int k0) {  // eight states, brought to the common maximum and summed as merge_parts does
        QaState all = acc;
#pragma unroll
        for (int k = 0; k < kQcUnroll; ++k)
          if (k0 + k < live) {
            const uint32_t at = mapa_shared(mine, k0 + k);
            ml[k] = ld_shared_cluster_f2(at + SM::kMlAll + 8 * r);
            v[k] = ld_shared_cluster_f4(at + (r * SM::kStride + 4 * c4) * 4);
            acc.m = fmaxf(acc.m, ml[k].x);
          }
        if (k0 > 0) {
          acc.l = 0.0f;
          acc.o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          acc.add(make_float2(all.m, all.l), all.o);
        }
#pragma unroll
        for (int k = 0; k < kQcUnroll; ++k)
          if (k0 + k < live) acc.add(ml[k], v[k]);
      };
      take(0);
      if (live > kQcUnroll) take(kQcUnroll);
      acc.store(p, b, h, r0 + r, D, c4);
    }
  }
  cluster_sync();  // no CTA leaves while another reads its memory
}

// Per (key head, sequence): the chunks' states merged.
constexpr int kQcThreads = 128;

template <int D>
__global__ void __launch_bounds__(kQcThreads) attn_q4_combine_kernel(const QaParams p) {
  pdl_wait();
  pdl_trigger();
  const int bh = blockIdx.x, b = bh / p.nkv, h = bh - b * p.nkv;
  const int n = __ldcg(p.ctx_len + b);
  const bool bad = n < 0 || n > (p.M << p.page_shift);
  const int parts = bad ? 0 : min((n + kQaRound - 1) / kQaRound, p.nchunk);
  for (int i = blockIdx.y * kQcThreads + threadIdx.x; i < p.R * (D / 4); i += gridDim.y * kQcThreads) {
    const int row = i / (D / 4), c4 = i - row * (D / 4);
    merge_parts(p, parts, bh, row, D, c4).store(p, b, h, row, D, c4);
  }
}

// The cut of a sequence: chunks of a whole number of steps of the four warps (128 positions), and how they meet.
// The lengths are on the device and may be anything up to the capacity, so the cut weighs, in steps of a CTA that has
// a third of an SM: half the capacity's steps and three for every chunk (queries, first loads, the states' meeting),
// spread over the GPU; 0.3 of a chunk's steps, which stay behind when the rest is done, and 0.2 more where no CTA
// waits for another (none is left to fill in); a tenth for every state that a second kernel merges; 0.03 for every
// step of the rounds that full sequences would take.  (Fitted to 44 batches of 1 to 128 sequences of up to 1152 to
// 131072 positions, each cut into 1 to 128 chunks: 3.5 % above the best of each, 17 % at most.  8 sequences of up to
// 32K, 10 key heads: 6 chunks 75.7 us, 10 51.4, 12 44.6, 64 80.3; 64 of up to 8192, 8 key heads and 16 rows: 1 chunk
// 108, 2 80.6, 4 90.5; 32 of up to 9216, 10 key heads: 2 chunks 61.3, 3 47.2, 6 54.1.)
// Where all CTAs are on the GPU at once and a sequence has at most eight, its chunks are a cluster (one of 300, 10 key
// heads: 4 chunks in a cluster 4.8 us, by a kernel 6.5), and so are up to sixteen where two CTAs an SM would do (one
// of 8100, 10 key heads: 8 chunks 11.7 us, 16 10.3, by a kernel 12.0; at 390 CTAs of clusters of eleven some wait: 13
// sequences of 3 to 9000 15.5 for 12.7 with eight); else the last CTA of up to eight merges them, for up to eight
// rows (clusters that wait for room leave SMs idle: 2 chunks of 32 of up to 2304 merged by the last 21.5, by a kernel
// 23.1, in clusters 27.3), and otherwise a second kernel.  All add in the same order.
// A chunk takes every nchunk-th step of the whole sequence: equal shares whatever its length (13 sequences of 3 to 9000
// positions, eight chunks: 12.8 us, one behind the other 13.7; 32 of 360 to 4500, two: 33.1 and 36.9; 24 of 360 to
// 2245, three chunks that last merged: 18.8 and 17.5).
// The cut goes by the batch, the key heads and the capacity and not by Q or the shared heads, so in a batch of one size
// a row is summed in the same order with few queries and with many.
struct Cut {
  int nchunk, steps, mode;  // chunks of a sequence, steps of a chunk, how they meet
};
Cut cut_of(int B, int nkv, long long cap) {
  constexpr int kSlots = 152 * 3, kFew = 152 * 2, kSmall = 16;
  const long long pairs = (long long)B * nkv, steps = (cap + kQaRound - 1) / kQaRound;
  const long long least = (steps + kQaMaxSteps - 1) / kQaMaxSteps;
  auto clustered = [&](long long used) {
    return used <= kQaWidth ? pairs * used <= kSlots : used <= kQaWidthFew && pairs * used <= kFew;
  };
  // up to sixteen chunks, and numbers around the one at which the sum below is least
  const long long mid = (long long)sqrt(40.0 * kSlots * steps / (300.0 * pairs + 10.0 * kSlots));
  long long best = 1ll << 62, at = steps, last = 0;
  for (int i = 1; i <= kSmall + 3; ++i) {
    long long k = i <= kSmall ? i : mid * (i - kSmall + 2) / 4;
    k = k < least ? least : k > steps ? steps : k;
    if (k == last) continue;
    last = k;
    const long long len = (steps + k - 1) / k, used = (steps + len - 1) / len, ctas = pairs * used;
    const long long wait = (10 * ctas <= 11 * kSlots ? 50 : 30) * len, merge = used > kQcUnroll && !clustered(used) ? 10 * used : 0;
    const long long cost = pairs * 50 * steps + ctas * 300 +
                           kSlots * (wait + merge + 3 * ((ctas + kSlots - 1) / kSlots) * (len + 3));
    if (cost < best) best = cost, at = len;
  }
  Cut c;
  c.nchunk = (int)((steps + at - 1) / at);
  c.mode = c.nchunk == 1 ? kQaDirect
           : clustered(c.nchunk) ? kQaCluster
           : c.nchunk <= kQcUnroll && pairs * kQaMaxTiles <= kQaCounters ? kQaLast
                                                                         : kQaParts;
  c.steps = (int)at;
  return c;
}

bool shape_ok(int B, int Q, int M, int page, int nh, int nkv, int d) {
  return B >= 0 && B <= 65535 && Q >= 1 && Q <= kMaxAttnQ && M >= 1 && q4_page_ok(page) && (long long)M * page <= (1ll << 24) &&
         nkv >= 1 && nkv <= 1024 && nh >= nkv && nh % nkv == 0 && nh / nkv <= 16 && q4_dim_ok(d) &&
         (long long)B * nkv <= kAttnMaxPairs && (long long)B * M < (1ll << 31);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// The counters, and the states of the chunks of `pairs` key heads where they meet in memory.
size_t ws_bytes_of(const Cut& cut, size_t pairs, int rows, int d) {
  const size_t parts = cut.mode >= kQaLast ? pairs * cut.nchunk * rows : 0;
  return kQaCounters * 4 + round256(parts * d * 4) + round256(parts * 2 * 4);
}

template <int D, int NT, int U, int K, int S, int kPerSm, int kGroups>
cudaError_t run(const QaParams& p, const DeviceCtx& dc, cudaStream_t s) {
  constexpr int kSmem = QaSmem<D, NT, U, K, S>::kTotal * kGroups;
  auto kernel = attn_q4_kernel<D, NT, U, K, S, kPerSm, kGroups>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kSmem, dc.device);
  if (e != cudaSuccess) return e;
  if (p.mode == kQaCluster && p.nchunk > kQaWidth) {  // to be asked for, once a kernel and device
    static std::atomic<uint64_t> wide{0};
    if (!(wide.load() >> dc.device & 1u)) {
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      wide |= 1ull << dc.device;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.B * p.nkv * p.rblocks, kGroups > 1 ? 1 : p.nchunk);
  cfg.blockDim = dim3(kQaThreads * kGroups);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 1;
  attr[1].val.clusterDim.y = p.nchunk;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kGroups == 1 && p.mode == kQaCluster ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess || kGroups > 1 || p.mode != kQaParts) return e;
  const int slices = (p.R * (D / 4) + kQcThreads - 1) / kQcThreads;
  return launch_pdl(attn_q4_combine_kernel<D>, dim3(p.B * p.nkv, slices), dim3(kQcThreads), 0, s, p);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace
}  // namespace lsv

using namespace lsv;

extern "C" {

size_t spec_q4_attention_workspace_size(int32_t B, int32_t Q, int32_t M, int32_t page, int32_t nh, int32_t nkv,
                                        int32_t d) {
  if (!shape_ok(B, Q, M, page, nh, nkv, d)) return 0;
  return ws_bytes_of(cut_of(B, nkv, (long long)M * page), (size_t)B * nkv, Q * (nh / nkv), d);
}

lsv_status spec_q4_attention(const void* q, const void* pool, const int32_t* table, const int32_t* ctx_len, int32_t B,
                             int32_t Q, int32_t nh, int32_t nkv, int32_t d, int32_t page, int32_t M, int32_t P,
                             float scale, void* out, void* ws, size_t ws_bytes, lsv_stream stream) {
  if (B < 0 || Q < 1 || nh < 1 || nkv < 1 || d < 1 || page < 1 || M < 1 || P < 1 || !(scale > 0.f) || !isfinite(scale))
    return LSV_ERR_INVALID_ARG;
  if (!shape_ok(B, Q, M, page, nh, nkv, d)) return LSV_ERR_UNSUPPORTED;
  if (B == 0) return LSV_OK;
  if (!q || !pool || !table || !ctx_len || !out) return LSV_ERR_INVALID_ARG;
  if (!al16(q) || !al16(pool) || !al16(table) || !al16(ctx_len) || !al16(out)) return LSV_ERR_MISALIGNED;
  const Cut cut = cut_of(B, nkv, (long long)M * page);
  if (!ws || ws_bytes < ws_bytes_of(cut, (size_t)B * nkv, Q * (nh / nkv), d)) return LSV_ERR_WORKSPACE;
  if (!al16(ws)) return LSV_ERR_MISALIGNED;
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  QaParams p;
  p.q = static_cast<const bf16*>(q);
  p.pool = static_cast<const uint8_t*>(pool);
  p.table = table;
  p.ctx_len = ctx_len;
  p.B = B;
  p.Q = Q;
  p.nh = nh;
  p.nkv = nkv;
  p.grp = nh / nkv;
  p.R = Q * p.grp;
  p.M = M;
  p.P = P;
  p.page_shift = 4;
  while ((1 << p.page_shift) < page) ++p.page_shift;
  p.nchunk = cut.nchunk;
  // (merging up to sixteen rows keeps a last CTA for longer than a second kernel takes: 137 us for 133.5)
  p.mode = cut.mode == kQaLast && p.R > 8 ? kQaParts : cut.mode;
  p.scale_log2 = scale * kQaLog2e;
  p.out = static_cast<bf16*>(out);
  const size_t parts = (size_t)B * nkv * p.nchunk * p.R;
  p.arrived = static_cast<int*>(ws);
  p.o_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kQaCounters * 4);
  p.ml_part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kQaCounters * 4 + round256(parts * d * 4));
  p.err = dc->err;
  p.wait_ns = wait_limit_ns();
  // Two or four short chunks of up to eight rows are the groups of one CTA and meet in its shared memory, where neither
  // a state nor a count goes through L2: 32 sequences of up to 2304 positions, two chunks of 9 steps, 20.1 us (merged by
  // the last CTA 23.0), 32 of up to 1152 12.5 (15.0), 16 of up to 4096, four of 8, 18.7 (19.9).  Long chunks are as fast
  // on several SMs, and faster where all are long (32 of 4200 to 4500, two of 18 steps: 51.6, as groups 53.9).
  const bool near = p.R <= 8 && cut.mode >= kQaLast && cut.steps <= kQaNear;
  const int groups = near && (cut.nchunk == 2 || cut.nchunk == 4) ? cut.nchunk : 1;
  const bool two = p.R > 8;  // the rows of an MMA, or its columns (half the MMAs for up to eight rows)
  p.rblocks = two ? (p.R + 15) / 16 : 1;
  // CTAs that find no room at once wait for others to leave: with the longest first, the short ones fill the end (64
  // sequences of up to 2048 positions, 512 CTAs with room for 456: 37.8 -> 33.0 us; 16 of 32K of any length, 896 CTAs:
  // 92 -> 68.5; 80 of about 2048: 55.5 -> 57.3, what sorting costs).  Where nearly all fit, sorting only brings the
  // long ones together on the SMs that are free first (32 of up to 4608, 640 CTAs, room for 608: 34.0 -> 36.5), unless
  // a CTA has half an SM or all of it (32 of up to 2304, 320 CTAs, room for 304: 20.9 -> 20.1).
  const long long ctas = (long long)B * nkv * p.rblocks * p.nchunk;
  const long long room = (long long)dc->num_sms * (two ? kQaTwo : kQaOne);
  p.sorted = B > 1 && B <= kQaThreads && p.mode != kQaCluster && (groups > 1 ? ctas > room : 10 * ctas > 11 * room);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (groups == 2)
    e = d == 128 ? run<128, 1, 2, 1, 3, kQaOne, 2>(p, *dc, s) : run<64, 1, 2, 1, 3, kQaOne, 2>(p, *dc, s);
  else if (groups == 4)
    e = d == 128 ? run<128, 1, 2, 1, 3, kQaOne, 4>(p, *dc, s) : run<64, 1, 2, 1, 3, kQaOne, 4>(p, *dc, s);
  else
    e = d == 128 ? (two ? run<128, 2, 2, 2, 2, kQaTwo, 1>(p, *dc, s) : run<128, 1, 2, 1, 3, kQaOne, 1>(p, *dc, s))
                 : (two ? run<64, 2, 2, 2, 2, kQaTwo, 1>(p, *dc, s) : run<64, 1, 2, 1, 3, kQaOne, 1>(p, *dc, s));
  return e == cudaSuccess ? LSV_OK : LSV_ERR_CUDA;
}

}  // extern "C"
