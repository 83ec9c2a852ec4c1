// q8.cu -- the 8-bit form of rows and weights: quantising, reading back, and the residual + RMSNorm whose
// output is 8-bit rows.
//
// 128 consecutive columns of a row (of a weight: a block of 128 x 128) share a scale s, the smallest power of
// two, 2^-126 at least, with max |x| <= 448 s; a code is e4m3(x / s), nearest, ties to even.  A power of two makes
// the quotient exact, so that a code never depends on how a division was rounded (with max |x| / 448 as the scale,
// bf16 values meet exact ties that the scale's own rounding decides), and it costs no precision: e4m3 is a floating
// format, and only values below 2^-13 of a group's largest lose a bit more than with the finest scale.
//
// All four kernels are bound by their bytes.  16 lanes x 8 columns (one 16-byte load a lane) are a group, so that its
// maximum meets in four shuffles and nothing is read twice.
#include <cuda_bf16.h>

#include "internal.h"
#include "lsv.h"
#include "ptx.cuh"
#include "q8.cuh"

namespace lsv {
namespace {

constexpr int kQ8Slot = 256;     // columns that a warp takes at once
constexpr int kQ8Vecs = 2;       // slots a warp holds at most
constexpr int kQ8MaxWarps = 32;  // warps a row

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// |x| as bits: ordered like the values, and at or above 0x7F800000 for an infinity or a NaN.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t max8(const float (&f)[8]) {
  uint32_t m = abs_bits(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, abs_bits(f[i]));
  return m;
}

// The scale of a group whose largest |x| has these bits, and its reciprocal: 448 = 1.75 * 2^8.
__device__ __forceinline__ float scale_of(uint32_t amax, float& inv) {
  const int e = max(1, (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0));
  inv = __uint_as_float((uint32_t)(254 - e) << 23);
  return __uint_as_float(amax >= 0x7F800000u ? 0x7FC00000u : (uint32_t)e << 23);
}

__device__ __forceinline__ uint32_t cvt4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv) {
  return make_uint2(cvt4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    cvt4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// ------------------------------------------------------------------------------------------------ rows
// A row is `wpr` warps, `rows` rows are a CTA; warp w of a row takes the slots w, w + wpr, .. of 256 columns, VECS at
// most, and holds them in registers between the sum of squares and the codes, so that x, y and the output move once.
//
// The normalised value is f / sqrt(mean f^2 + eps) with the root's reciprocal as a pair r + r2 (r2: what rounding r
// to 32 bits left out, from the residual of m r^2), so that h is off by little more than its own rounding: codes
// next to a tie then fall as the formula has them but for 2^-24 of the values next to it.
template <int VECS, bool NORM>
__global__ void __launch_bounds__(1024) q8_rows_kernel(const bf16* x, const bf16* __restrict__ y, bf16* x_out,
                                                       const bf16* __restrict__ gain, uint8_t* __restrict__ codes,
                                                       float* __restrict__ scales, int T, int H, int wpr, int rows,
                                                       float eps) {
  __shared__ float part[kQ8MaxWarps];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rl = warp / wpr, w = warp - rl * wpr;
  const int t = blockIdx.x * rows + rl;
  const bool live = t < T;
  const int G = (H + kQ8Group - 1) / kQ8Group;
  const size_t base = (size_t)t * H;
  uint4 v[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int c = (w + i * wpr) * kQ8Slot + lane * 8;
    v[i] = live && c < H ? ld_stream128(x + base + c) : make_uint4(0, 0, 0, 0);
  }
  float r = 1.0f, r2 = 0.0f;
  if constexpr (NORM) {
    float ss = 0.0f;
    if (y) {
      uint4 u[VECS];
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const int c = (w + i * wpr) * kQ8Slot + lane * 8;
        u[i] = live && c < H ? ld_stream128(y + base + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < VECS; ++i) {
        const int c = (w + i * wpr) * kQ8Slot + lane * 8;
        float a[8], b[8];
        unpack8(v[i], a);
        unpack8(u[i], b);
        v[i] = make_uint4(pack2(a[0] + b[0], a[1] + b[1]), pack2(a[2] + b[2], a[3] + b[3]),
                          pack2(a[4] + b[4], a[5] + b[5]), pack2(a[6] + b[6], a[7] + b[7]));
        if (live && c < H) *reinterpret_cast<uint4*>(x_out + base + c) = v[i];
      }
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      float f[8];
      unpack8(v[i], f);
      // pairwise: squares of bf16 are exact in 32 bits
      const float p0 = fmaf(f[1], f[1], f[0] * f[0]), p1 = fmaf(f[3], f[3], f[2] * f[2]);
      const float p2 = fmaf(f[5], f[5], f[4] * f[4]), p3 = fmaf(f[7], f[7], f[6] * f[6]);
      ss += (p0 + p1) + (p2 + p3);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (wpr > 1) {
      if (lane == 0) part[warp] = ss;
      __syncthreads();
      ss = lane < wpr ? part[rl * wpr + lane] : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float m = ss / (float)H + eps;
    r = 1.0f / sqrtf(m);
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
    float f[8];
    unpack8(v[i], f);
    if constexpr (NORM) {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = fmaf(f[j], r2, f[j] * r);
      if (gain && c < H) {
        float g[8];
        unpack8(ld_plain128(gain + c), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= g[j];
      }
    }
    uint32_t m = max8(f);
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
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8(v[i], f);
    m = max(m, max8(f));
  }
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
    float f[8];
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
  return pack2(f.x * s, f.y * s);
}

__global__ void __launch_bounds__(256) q8_read_kernel(const uint8_t* __restrict__ codes,
                                                      const float* __restrict__ scales, bf16* __restrict__ out,
                                                      int R, int C, int by) {
  pdl_wait();
  pdl_trigger();
  const int per = C / 8, G = (C + kQ8Group - 1) / kQ8Group;
  const long long p0 = (long long)blockIdx.x * (256 * kQ8ReadPieces);
  const int row0 = (int)(p0 / per);
  const int col0 = (int)(p0 - (long long)row0 * per);
  uint2 v[kQ8ReadPieces];
  float s[kQ8ReadPieces];
  size_t at[kQ8ReadPieces];
  bool live[kQ8ReadPieces];
#pragma unroll
  for (int i = 0; i < kQ8ReadPieces; ++i) {
    const int c = col0 + (int)threadIdx.x + 256 * i;
    const int dr = c / per, row = row0 + dr, col = (c - dr * per) * 8;
    live[i] = row < R;
    at[i] = (size_t)row * C + col;
    if (!live[i]) continue;
    v[i] = ld_stream64(codes + at[i]);
    s[i] = ld_plain_f32(scales + (size_t)(row / by) * G + col / kQ8Group);
  }
#pragma unroll
  for (int i = 0; i < kQ8ReadPieces; ++i) {
    if (!live[i]) continue;
    *reinterpret_cast<uint4*>(out + at[i]) =
        make_uint4(values2(v[i].x & 0xFFFFu, s[i]), values2(v[i].x >> 16, s[i]), values2(v[i].y & 0xFFFFu, s[i]),
                   values2(v[i].y >> 16, s[i]));
  }
}

cudaError_t launch_rows(bool norm, const bf16* x, const bf16* y, bf16* x_out, const bf16* gain, uint8_t* codes,
                        float* scales, int T, int H, float eps, const DeviceCtx& dc, cudaStream_t s) {
  const int slots = (H + kQ8Slot - 1) / kQ8Slot;
  // One slot a warp for short rows, two for longer ones, which then have fewer warps to meet: the norm of 9760 x 1280
  // takes 18.1 us with one and 18.5 with two, of 1500 x 7168 18.7 and 18.0; quantising 9760 x 1280 alone, where no warp
  // waits for another, 10.7 and 9.0, and 60000 x 208, a slot a row, 10.7 and 11.4.
  const bool wide = slots > (norm ? 8 : 1);
  const int vecs = wide ? kQ8Vecs : 1;
  const int wpr = (slots + vecs - 1) / vecs;
  const int rows = wpr >= 8 ? 1 : 8 / wpr;
  const dim3 grid((T + rows - 1) / rows), block(32 * wpr * rows);
  auto go = [&](auto kernel) {
    return launch_pdl(kernel, grid, block, 0, s, x, y, x_out, gain, codes, scales, T, H, wpr, rows, eps);
  };
  if (norm) return wide ? go(q8_rows_kernel<kQ8Vecs, true>) : go(q8_rows_kernel<1, true>);
  return wide ? go(q8_rows_kernel<kQ8Vecs, false>) : go(q8_rows_kernel<1, false>);
}

// Sizes of an 8-bit matrix.
lsv_status check_q8(int64_t rows, int64_t cols) {
  if (rows < 0 || cols <= 0) return LSV_ERR_INVALID_ARG;
  if (cols % 16 || cols > kQ8MaxCols || rows * cols >= (1ll << 40)) return LSV_ERR_UNSUPPORTED;
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
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  return launch_rows(false, static_cast<const bf16*>(x), nullptr, nullptr, nullptr, static_cast<uint8_t*>(codes), scales,
                     R, C, 0.0f, *dc, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
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
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  return launch_rows(true, static_cast<const bf16*>(x), static_cast<const bf16*>(y), static_cast<bf16*>(x_out),
                     static_cast<const bf16*>(gain), static_cast<uint8_t*>(codes), scales, T, H, eps, *dc,
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
  const long long pieces = (long long)R * (C / 8), per = 256 * kQ8ReadPieces;
  return launch_pdl(q8_read_kernel, dim3((unsigned)((pieces + per - 1) / per)), dim3(256), 0,
                    reinterpret_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(codes), scales,
                    static_cast<bf16*>(out), R, C, rows_per_scale) == cudaSuccess
             ? LSV_OK
             : LSV_ERR_CUDA;
}

}  // extern "C"
