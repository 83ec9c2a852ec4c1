// q8.cu -- the 8-bit form of rows and weights: quantising, reading back, and the residual + RMSNorm whose
// output is 8-bit rows.
//
// 128 consecutive columns of a row (of a weight: a block of 128 x 128) share a scale s, the smallest power of
// two, 2^-126 at least, with max |x| <= 448 s; a code is e4m3(x / s), nearest, ties to even.  A power of two makes
// the quotient exact, so that a code never depends on how a division was rounded (with max |x| / 448 as the scale,
// bf16 values meet exact ties that the scale's own rounding decides), and it costs no precision: e4m3 is a floating
// format, and only values below 2^-13 of a group's largest lose a bit more than with the finest scale.
//
// All four kernels are bound by their bytes, and have few instructions to spare beside them (values go two at a time
// wherever there is an instruction for it).  16 lanes x 8 columns (one 16-byte load a lane) are a group, so that its
// maximum meets in four shuffles and nothing is read twice.  Of 9760 x 1280, with what is read and written over the
// time: the residual and norm 15.7 us, 5.6 TB/s; quantising 7.6 us, 5.0; reading back 7.0 us, 5.4.  A weight of
// 129280 x 1280 72 us, 6.9.  One row of 1280: 1.6, 1.2 and 0.9 us.
#include <cuda_bf16.h>

#include "internal.h"
#include "lsv.h"
#include "ptx.cuh"
#include "q4ptx.cuh"
#include "q8.cuh"

namespace lsv {
namespace {

constexpr int kQ8Slot = 256;     // columns that a warp takes at once
constexpr int kQ8Vecs = 2;       // slots a warp holds at most
constexpr int kQ8MaxWarps = 32;  // warps a row

// Eight values are four pairs, which the FP32 pipes take two at a time.
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// The sum of two pairs of bf16 values, rounded to bf16 (as their sum in 32 bits rounded would be: where that is not
// exact, one value is below half a step of the other).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 s =
      __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&s);
}

// The largest |x| as bits: ordered like the values, and above 0x7F800000 where one is a NaN.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ uint32_t max8(const float2 (&f)[4]) {
  const float a = max_abs(max_abs(f[0].x, f[0].y), max_abs(f[1].x, f[1].y));
  const float b = max_abs(max_abs(f[2].x, f[2].y), max_abs(f[3].x, f[3].y));
  return __float_as_uint(max_abs(a, b));
}
// The same of eight bf16 values, whose bits are ordered like them too: two at a time.
__device__ __forceinline__ uint32_t max8(const uint4& v) {
  const uint32_t m =
      __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}

// The scale of a group whose largest |x| has these bits, and its reciprocal: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_of(uint32_t amax, float& inv) {
  const int e = max(1, (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0));
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
  return __uint_as_float(amax >= 0x7F800000u ? 0x7FC00000u : (uint32_t)e << 23);
}

__device__ __forceinline__ uint32_t cvt4(float2 a, float2 b) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a.y), "f"(a.x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(b.y), "f"(b.x));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint2 codes8(const float2 (&f)[4], float inv) {
  const float2 by = make_float2(inv, inv);
  return make_uint2(cvt4(mul2(f[0], by), mul2(f[1], by)), cvt4(mul2(f[2], by), mul2(f[3], by)));
}

// ------------------------------------------------------------------------------------------------ rows
// A row is `wpr` warps, `rows` rows are a CTA; warp w of a row takes the slots w, w + wpr, .. of 256 columns, VECS at
// most, and holds them in registers between the sum of squares and the codes, so that x, y and the output move once.
//
// The normalised value is f / sqrt(mean f^2 + eps) with the root's reciprocal as a pair r + r2 (r2: what the
// approximation r left out, from the residual of m r^2), so that h is off by little more than its own rounding: codes
// next to a tie then fall as the formula has them but for 2^-24 of the values next to it.  by_h + by_h2 is 1 / H.
template <int VECS, bool NORM>
__global__ void __launch_bounds__(1024) q8_rows_kernel(const bf16* x, const bf16* __restrict__ y, bf16* x_out,
                                                       const bf16* __restrict__ gain, uint8_t* __restrict__ codes,
                                                       float* __restrict__ scales, int T, int H, float eps,
                                                       float by_h, float by_h2) {
  __shared__ float part[kQ8MaxWarps];
  pdl_wait();
  pdl_trigger();
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, wpr = blockDim.x >> 5, first = threadIdx.y * wpr;
  const int G = (uint32_t)(H + kQ8Group - 1) / kQ8Group;
  const int t = blockIdx.x * blockDim.y + threadIdx.y;
  const bool live = t < T;
  const size_t base = (size_t)t * H;
  uint4 v[VECS], u[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (w + i * wpr) * kQ8Slot + lane * 8;
    v[i] = live && c < H ? ld_stream128(x + base + c) : make_uint4(0, 0, 0, 0);
    if (NORM && y) u[i] = live && c < H ? ld_stream128(y + base + c) : make_uint4(0, 0, 0, 0);
  }
  float r = 1.0f, r2 = 0.0f;
  if constexpr (NORM) {
    float2 sq = make_float2(0.0f, 0.0f);
    if (y) {
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const int c = (w + i * wpr) * kQ8Slot + lane * 8;
        v[i] = make_uint4(add_bf16x2(v[i].x, u[i].x), add_bf16x2(v[i].y, u[i].y), add_bf16x2(v[i].z, u[i].z),
                          add_bf16x2(v[i].w, u[i].w));
        if (live && c < H) *reinterpret_cast<uint4*>(x_out + base + c) = v[i];
      }
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      float2 f[4];
      unpack8(v[i], f);
      // squares of bf16 are exact in 32 bits
#pragma unroll
      for (int j = 0; j < 4; ++j) sq = fma2(f[j], f[j], sq);
    }
    float ss = sq.x + sq.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (wpr > 1) {
      if (lane == 0) part[first + w] = ss;
      __syncthreads();
      const int lanes = 1 << (32 - __clz(wpr - 1)), of = lane & (lanes - 1);  // (as many as hold a value a warp)
      ss = of < wpr ? part[first + of] : 0.0f;
      for (int o = 1; o < lanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float m = fmaf(ss, by_h, fmaf(ss, by_h2, eps));
    r = rsqrtf(m);
    const float q = m * r;
    // 1 - m r^2, exact but for its own rounding; a mean of zero, infinity or NaN has no correction
    const float left = fmaf(-q, r, 1.0f) - fmaf(m, r, -q) * r;
    r2 = 0.5f * r * left;
    if (!(fabsf(r2) < r)) r2 = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int slot = w + i * wpr;
    if (slot * kQ8Slot >= H) break;
    const int c = slot * kQ8Slot + lane * 8;
    float2 f[4];
    uint32_t m;
    unpack8(v[i], f);
    if constexpr (NORM) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = fma2(f[j], make_float2(r2, r2), mul2(f[j], make_float2(r, r)));
      if (gain && c < H) {
        float2 g[4];
        unpack8(ld_plain128(gain + c), g);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], g[j]);
      }
      m = max8(f);
    } else {
      m = max8(v[i]);
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    const float s = scale_of(m, inv);
    if (live && c < H) {
      *reinterpret_cast<uint2*>(codes + base + c) = codes8(f, inv);
      if ((lane & 15) == 0) scales[(size_t)t * G + c / kQ8Group] = s;
    }
  }
}

// ------------------------------------------------------------------------------------------------ weights
// One CTA a block of 128 x 128: 16 lanes a row, eight rows a thread, all of them in registers.
__global__ void __launch_bounds__(256) q8_weight_kernel(const bf16* __restrict__ w, uint8_t* __restrict__ codes,
                                                        float* __restrict__ scales, int N, int K) {
  __shared__ uint32_t part[8];
  pdl_wait();
  const int G = (K + kQ8Group - 1) / kQ8Group;
  const int c = blockIdx.x % G * kQ8Group + (threadIdx.x & 15) * 8;
  const int n0 = blockIdx.x / G * kQ8Group + (threadIdx.x >> 4);
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = c < K && n0 + 16 * i < N ? ld_stream128(w + (size_t)(n0 + 16 * i) * K + c)
                                    : make_uint4(0, 0, 0, 0);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, max8(v[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, part[i]);
  float inv;
  const float s = scale_of(m, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (c >= K || n0 + 16 * i >= N) continue;
    float2 f[4];
    unpack8(v[i], f);
    *reinterpret_cast<uint2*>(codes + (size_t)(n0 + 16 * i) * K + c) = codes8(f, inv);
  }
  if (threadIdx.x == 0) scales[blockIdx.x] = s;
}

// ------------------------------------------------------------------------------------------------ back
constexpr int kQ8ReadPieces = 4;  // 8 codes a piece (a 16-byte store), four pieces a thread

__device__ __forceinline__ uint32_t values2(uint32_t two, float s) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const float2 x = mul2(f, make_float2(s, s));
  return pack2(x.x, x.y);
}

// Quotients of the pieces' places by the pieces a row, `per`, as products with 2^64 / per and 2^32 / per rounded up:
// exact for places whose product with per is below 2^64 and 2^32.  (Divisions took a third of the time: 4879 x 1280
// 5.8 us with them, 4.4 without.)
struct Q8Read {
  long long pieces;
  int per, G, shift;  // shift: 0, or 7 where 128 rows share a scale
  uint64_t by_per64;
  uint32_t by_per32;
};

__global__ void __launch_bounds__(256) q8_read_kernel(const uint8_t* __restrict__ codes,
                                                      const float* __restrict__ scales, bf16* __restrict__ out,
                                                      const Q8Read p) {
  pdl_wait();
  pdl_trigger();
  const long long p0 = (long long)blockIdx.x * (256 * kQ8ReadPieces);
  const int row0 = (int)__umul64hi((uint64_t)p0, p.by_per64);
  const int col0 = (int)(p0 - (long long)row0 * p.per) + (int)threadIdx.x;
  const int left = (int)min(p.pieces - p0, 256ll * kQ8ReadPieces) - (int)threadIdx.x;  // this thread's have places below
  const uint8_t* from = codes + 8 * (p0 + threadIdx.x);
  bf16* to = out + 8 * (p0 + threadIdx.x);
  uint2 v[kQ8ReadPieces];
  float s[kQ8ReadPieces];
#pragma unroll
  for (int i = 0; i < kQ8ReadPieces; ++i) {
    if (256 * i >= left) break;
    const int c = col0 + 256 * i, dr = (int)__umulhi((uint32_t)c, p.by_per32);
    v[i] = ld_stream64(from + 8 * 256 * i);
    s[i] = ld_plain_f32(scales + (size_t)(uint32_t)((row0 + dr) >> p.shift) * p.G +
                        (uint32_t)(c - dr * p.per) / (kQ8Group / 8));
  }
#pragma unroll
  for (int i = 0; i < kQ8ReadPieces; ++i) {
    if (256 * i >= left) break;
    *reinterpret_cast<uint4*>(to + 8 * 256 * i) = make_uint4(values2(v[i].x & 0xFFFFu, s[i]), values2(v[i].x >> 16, s[i]),
                                                             values2(v[i].y & 0xFFFFu, s[i]), values2(v[i].y >> 16, s[i]));
  }
}

cudaError_t launch_rows(bool norm, const bf16* x, const bf16* y, bf16* x_out, const bf16* gain, uint8_t* codes,
                        float* scales, int T, int H, float eps, cudaStream_t s) {
  const int slots = (H + kQ8Slot - 1) / kQ8Slot;
  // One slot a warp for short rows, two for longer ones, which then have fewer warps to meet: the norm of 1500 x 7168
  // takes 16.4 us with one and 14.1 with two, of one row of 1280 1.6 and 1.8, of 9760 x 1280 15.5 with either; quantising
  // 9760 x 1280 alone, where no warp waits for another, 10.5 and 7.6.
  const int vecs = slots > (norm ? 8 : 1) ? kQ8Vecs : 1;
  const int wpr = (slots + vecs - 1) / vecs;
  const int rows = wpr >= 8 ? 1 : 8 / wpr;
  const float by_h = (float)(1.0 / H), by_h2 = (float)(1.0 / H - by_h);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, dim3((T + rows - 1) / rows), dim3(32 * wpr, rows), 0, s, x, y, x_out, gain, codes, scales, T,
                      H, eps, by_h, by_h2);
  };
  if (norm) return vecs > 1 ? go(q8_rows_kernel<kQ8Vecs, true>) : go(q8_rows_kernel<1, true>);
  return vecs > 1 ? go(q8_rows_kernel<kQ8Vecs, false>) : go(q8_rows_kernel<1, false>);
}

// Sizes of an 8-bit matrix.
lsv_status check_q8(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return LSV_ERR_INVALID_ARG;
  if (cols % 16 || cols > kQ8MaxCols || rows > kQ8MaxRows) return LSV_ERR_UNSUPPORTED;
  return LSV_OK;
}

bool aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) & 15) return false;
  return true;
}

}  // namespace
}  // namespace lsv

using namespace lsv;

extern "C" {

lsv_status quantize_q8_rows(const void* x, int32_t R, int32_t C, void* codes, float* scales, lsv_stream stream) {
  const lsv_status st = check_q8(R, C);
  if (st != LSV_OK || R == 0) return st;
  if (!x || !codes || !scales) return LSV_ERR_INVALID_ARG;
  if (!aligned({x, codes, scales})) return LSV_ERR_MISALIGNED;
  return launch_rows(false, static_cast<const bf16*>(x), nullptr, nullptr, nullptr, static_cast<uint8_t*>(codes), scales,
                     R, C, 0.0f, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? LSV_OK
             : LSV_ERR_CUDA;
}

lsv_status rmsnorm_residual_q8(const void* x, const void* y, const void* gain, void* x_out, void* codes, float* scales,
                               int32_t T, int32_t H, float eps, lsv_stream stream) {
  if (!(eps >= 0.0f)) return LSV_ERR_INVALID_ARG;
  const lsv_status st = check_q8(T, H);
  if (st != LSV_OK || T == 0) return st;
  if (!x || !codes || !scales || (y && !x_out)) return LSV_ERR_INVALID_ARG;
  if (!aligned({x, y, gain, x_out, codes, scales})) return LSV_ERR_MISALIGNED;
  return launch_rows(true, static_cast<const bf16*>(x), static_cast<const bf16*>(y), static_cast<bf16*>(x_out),
                     static_cast<const bf16*>(gain), static_cast<uint8_t*>(codes), scales, T, H, eps,
                     reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? LSV_OK
             : LSV_ERR_CUDA;
}

lsv_status quantize_q8_weight(const void* w, int32_t N, int32_t K, void* codes, float* scales, lsv_stream stream) {
  const lsv_status st = check_q8(N, K);
  if (st != LSV_OK || N == 0) return st;
  if (!w || !codes || !scales) return LSV_ERR_INVALID_ARG;
  if (!aligned({w, codes, scales})) return LSV_ERR_MISALIGNED;
  const long long blocks = ((long long)N + kQ8Group - 1) / kQ8Group * ((K + kQ8Group - 1) / kQ8Group);
  return launch_pdl(q8_weight_kernel, dim3((unsigned)blocks), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream),
                    static_cast<const bf16*>(w), static_cast<uint8_t*>(codes), scales, N, K) == cudaSuccess
             ? LSV_OK
             : LSV_ERR_CUDA;
}

lsv_status dequantize_q8(const void* codes, const float* scales, int32_t R, int32_t C, int32_t rows_per_scale, void* out,
                         lsv_stream stream) {
  if (rows_per_scale != 1 && rows_per_scale != kQ8Group) return LSV_ERR_INVALID_ARG;
  const lsv_status st = check_q8(R, C);
  if (st != LSV_OK || R == 0) return st;
  if (!codes || !scales || !out) return LSV_ERR_INVALID_ARG;
  if (!aligned({codes, scales, out})) return LSV_ERR_MISALIGNED;
  Q8Read p;
  p.per = C / 8;
  p.pieces = (long long)R * p.per;
  p.G = (C + kQ8Group - 1) / kQ8Group;
  p.shift = rows_per_scale == 1 ? 0 : 7;
  p.by_per64 = ~0ull / p.per + 1;
  p.by_per32 = ~0u / p.per + 1;
  const long long a_cta = 256 * kQ8ReadPieces;
  return launch_pdl(q8_read_kernel, dim3((unsigned)((p.pieces + a_cta - 1) / a_cta)), dim3(256), 0,
                    reinterpret_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(codes), scales,
                    static_cast<bf16*>(out), p) == cudaSuccess
             ? LSV_OK
             : LSV_ERR_CUDA;
}

}  // extern "C"
