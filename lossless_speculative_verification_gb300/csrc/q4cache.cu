// q4cache.cu -- writing positions to the 4-bit paged cache and reading them back
// (layout: q4.cuh).
//
// One CTA takes one block (16 positions of a head), each of its warps 8 positions
// of the keys or the values in the lane layout of the cache: a lane quantises what it stores, the maximum of a
// group of 64 dims meets over the 4 lanes of a position (keys) or the 8 lanes
// of a pair of positions (values), and whole words leave as one vector a lane.
// Positions at the edges of the new ones share their block with others: keys and
// scales of a position have bytes of their own, values 16-bit halves, so no
// block is read to be written and two calls on neighbouring positions do not
// touch each other's bytes.
#include <cuda_bf16.h>

#include <type_traits>

#include "internal.h"
#include "lsv.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace lsv {
namespace {

constexpr int kQwWarps = 4;
constexpr uint32_t kSmallScale = 0x0D80u;  // 2^-100 in bf16

// Largest |x| of packed bf16 pairs as bits: ordered like the values, and above 0x7F80 for NaN.
__device__ __forceinline__ uint32_t abs_max2(uint32_t m, uint32_t v) { return __vmaxu2(m, v & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t fold2(uint32_t m) { return max(m & 0xFFFFu, m >> 16); }

// bf16 bits of s = bf16(amax / 7).  With 8 significant bits over 7 the quotient is never within 2^-12 of the
// middle of two bf16 values, so amax * (1 / 7) in fp32, rounded again, is the correctly rounded one.
__device__ __forceinline__ uint32_t scale_bits(uint32_t amax) {
  if (amax >= 0x7F80u) return kQ4NanScale;
  return __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(amax << 16) * (1.0f / 7.0f)));
}

// Scales that 1 / s and 7 steps do for.
__device__ __forceinline__ bool plain_scale(uint32_t bits) { return bits >= kSmallScale && bits < 0x7F80u; }

// A group's scale and its reciprocal (0 for a scale that is not plain: a position beside the new ones has one, and
// must not reach the other half of their word).
struct Step {
  uint32_t bits;
  float s, inv;
};
__device__ __forceinline__ Step step_of(uint32_t bits) {
  Step r;
  r.bits = bits;
  r.s = __uint_as_float(bits << 16);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.inv) : "f"(r.s));
  if (!plain_scale(bits)) r.inv = 0.0f;
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xFFFF0000u); }

// rint(x / s), ties to even, of two values, in the low bits of fp32 that are 1.5 * 2^23 more; the scale is plain.
// x and s have 8 significant bits, so that x / s is k + 1/2 exactly or at least 1/512 away from it:
// x / s = X 2^a / (S 2^b)
// differs by |2^(a+1) X - (2k+1) 2^b S| / (2^(b+1) S), where the numerator is a multiple of 2^b and S < 256, or
// 2^(b-a-1) S >= 256 > X.  x * (1 / s), less than 2^-19 off, is added to 1536 and so becomes a multiple of 2^-13:
// what was k + 1/2 is that again, and nothing else becomes it.  The second addition rounds to a whole number.
// (Eight prompts of 1156 positions are appended in 12.9 us; a quotient corrected by its remainder: 15.5, a division:
// 28.)
constexpr float kSnap = 1536.0f, kRound = 12582912.0f;
__device__ __forceinline__ void whole2(float inv0, float inv1, float x0, float x1, uint32_t* n0, uint32_t* n1) {
  asm("{\n.reg .b64 x, i, c, r;\n"
      "mov.b64 x, {%2, %3};\nmov.b64 i, {%4, %5};\nmov.b64 c, {%6, %6};\nmov.b64 r, {%7, %7};\n"
      "fma.rn.f32x2 x, x, i, c;\nadd.rn.f32x2 x, x, r;\nmov.b64 {%0, %1}, x;\n}"
      : "=r"(*n0), "=r"(*n1)
      : "f"(x0), "f"(x1), "f"(inv0), "f"(inv1), "f"(kSnap), "f"(kRound - kSnap));
}
// Eight of them as the nibbles n + 8 of a word, the first in the lowest place: added up in their places, where the
// bits of 1.5 * 2^23 and the 8s make one constant.
__device__ __forceinline__ uint32_t word_of(const uint32_t (&n)[8]) {
  uint32_t w = n[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) w = (w << 4) + n[i];
  return w + (0x88888888u - 0x4B400000u * 0x11111111u);
}
// One code as a nibble, whatever the scale: of 0 or NaN, n = 0; small scales, whose reciprocal may overflow and whose
// own rounding may leave more than 7 steps, divide.
__device__ __forceinline__ uint32_t any_code(const Step& r, float x) {
  if (r.bits == 0u || r.bits >= 0x7F80u) return 8u;
  return static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(rintf(__fdiv_rn(x, r.s)), -8.0f), 7.0f)) + 8);
}
// The word of eight values x[i] in the steps of r[i / 4].
template <bool kPlain>
__device__ __forceinline__ uint32_t codes8(const Step& r0, const Step& r1, const float (&x)[8]) {
  if (kPlain) {
    uint32_t n[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float inv = i < 4 ? r0.inv : r1.inv;
      whole2(inv, inv, x[i], x[i + 1], &n[i], &n[i + 1]);
    }
    return word_of(n);
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) w |= any_code(i < 4 ? r0 : r1, x[i]) << (4 * i);
  return w;
}

struct QwParams {
  const int32_t* table;    // [B, M]
  const int32_t* ctx_len;  // [B]
  int B, Q, nkv, M, P, page_shift;
  int nblk;  // blocks that Q positions can touch
  int* err;
};

// A CTA's (sequence, block, head), and the entry of the block's page.  The entry's load is only begun here: what
// depends on the length alone (the rows to append) is loaded beside it.
struct QwPlace {
  int b, h, n, p0, block;
  bool any;  // some position of the block exists and is one of the Q
  int pg;
};
__device__ __forceinline__ bool length_ok(const QwParams& p, int n) { return n >= 0 && n <= (p.M << p.page_shift); }
__device__ __forceinline__ QwPlace place(const QwParams& p, int unit) {
  QwPlace w;
  w.h = unit % p.nkv;
  const int r = unit / p.nkv;
  w.b = r / p.nblk;
  const int bi = r - w.b * p.nblk;
  w.n = __ldcg(p.ctx_len + w.b);
  w.p0 = w.n - p.Q;
  w.block = q4_floor_block(w.p0) + bi;
  w.any = length_ok(p, w.n) && w.block >= 0 && (w.block << 4) < w.n;
  w.pg = w.any ? __ldcg(p.table + (size_t)w.b * p.M + ((w.block << 4) >> p.page_shift)) : -1;
  return w;
}
// The block's place in the pool, in blocks.
__device__ __forceinline__ size_t block_of(const QwParams& p, const QwPlace& w) {
  const int per = 1 << (p.page_shift - 4);  // blocks of a page and head
  return ((size_t)w.pg * p.nkv + w.h) * per + (w.block & (per - 1));
}

// Keys of 8 positions: lane (g, t) has the dims 32 j + 8 t + 0..7 of position tk = 8 half + g.
template <int D>
__device__ __forceinline__ void append_keys(const uint4 (&x)[Q4Block<D>::W], bool in, uint8_t* blk, int tk, int t) {
  using L = Q4Block<D>;
  Q4Words<L::W> out;
  uint32_t sc = 0;
  Step st[L::G];
  bool plain = true;
#pragma unroll
  for (int gr = 0; gr < L::G; ++gr) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 2 * gr; j < 2 * gr + 2; ++j) m = abs_max2(abs_max2(abs_max2(abs_max2(m, x[j].x), x[j].y), x[j].z), x[j].w);
    m = fold2(m);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    st[gr] = step_of(scale_bits(m));
    sc |= st[gr].bits << (16 * gr);
    plain = plain && plain_scale(st[gr].bits);
  }
  auto words = [&](auto tag) {
#pragma unroll
    for (int j = 0; j < L::W; ++j) {
      const float v[8] = {lo_f(x[j].x), lo_f(x[j].y), lo_f(x[j].z), lo_f(x[j].w),
                          hi_f(x[j].x), hi_f(x[j].y), hi_f(x[j].z), hi_f(x[j].w)};
      out.w[j] = codes8<decltype(tag)::value>(st[j >> 1], st[j >> 1], v);
    }
  };
  if (__all_sync(0xffffffffu, plain || !in))  // (positions that are not there are not stored)
    words(std::true_type{});
  else
    words(std::false_type{});
  if (in) {
    q4_store<L::W>(blk + tk * (D / 2) + t * (4 * L::W), out);
    if (t == 0) q4_store_scales<L::G>(blk + L::kKs + tk * 2 * L::G, sc);
  }
}

// Values of 8 positions: lane (g, t) has the dims 32 m + 4 g + 0..3 of position 8 half + 2 t and the one after it.
template <int D>
__device__ __forceinline__ void append_values(const uint2 (&x)[2][Q4Block<D>::W], const bool (&in)[2], uint8_t* blk, int half,
                                              int lane) {
  using L = Q4Block<D>;
  const int g = lane >> 2, t = lane & 3;
  Q4Words<L::W> out;
  Step st[2][L::G];
  bool plain = true;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t sc = 0;
#pragma unroll
    for (int gr = 0; gr < L::G; ++gr) {
      uint32_t a = 0;
#pragma unroll
      for (int m = 2 * gr; m < 2 * gr + 2; ++m) a = abs_max2(abs_max2(a, x[e][m].x), x[e][m].y);
      a = fold2(a);
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 4));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 8));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 16));
      st[e][gr] = step_of(scale_bits(a));
      sc |= st[e][gr].bits << (16 * gr);
      plain = plain && (plain_scale(st[e][gr].bits) || !in[e]);
    }
    if (in[e] && g == 0) q4_store_scales<L::G>(blk + L::kVs + (8 * half + 2 * t + e) * 2 * L::G, sc);
  }
  auto words = [&](auto tag) {
#pragma unroll
    for (int m = 0; m < L::W; ++m) {
      const float v[8] = {lo_f(x[0][m].x), hi_f(x[0][m].x), lo_f(x[0][m].y), hi_f(x[0][m].y),
                          lo_f(x[1][m].x), hi_f(x[1][m].x), lo_f(x[1][m].y), hi_f(x[1][m].y)};
      out.w[m] = codes8<decltype(tag)::value>(st[0][m >> 1], st[1][m >> 1], v);
    }
  };
  if (__all_sync(0xffffffffu, plain))
    words(std::true_type{});
  else
    words(std::false_type{});
  uint8_t* at = blk + L::kV + (half * 32 + lane) * (4 * L::W);
  if (in[0] && in[1]) {
    q4_store<L::W>(at, out);
  } else if (in[0] || in[1]) {
#pragma unroll
    for (int m = 0; m < L::W; ++m)
      *reinterpret_cast<uint16_t*>(at + 4 * m + (in[1] ? 2 : 0)) =
          static_cast<uint16_t>(in[1] ? out.w[m] >> 16 : out.w[m] & 0xFFFFu);
  }
}

// Up to twelve CTAs an SM (37 to 40 registers): a CTA is one chain of loads (length, entry and rows, then the codes),
// and what is in flight on an SM is what its CTAs have begun.  Eight prompts of 1156 positions move 60 MB in 12.9 us
// (4.7 TB/s; blocks two or four a CTA: 13.1, 14.0), and are read back in 11.7.
// A warp's share is a half block (8 positions) of the keys or of the values: the four parts of a block are the
// CTA's warps.  32 x 4 positions of 10 heads were written and read back in 17.6 us with whole blocks a warp, in 9.2
// with quarters: the call is as long as one warp's chain of loads, maxima and codes.
template <int D>
__global__ void __launch_bounds__(kQwWarps * 32, 12) q4_append_kernel(const bf16* __restrict__ k_new,
                                                                  const bf16* __restrict__ v_new, uint8_t* pool,
                                                                  const QwParams p) {
  using L = Q4Block<D>;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, half = part & 1;
  const QwPlace w = place(p, blockIdx.x);
  if (!w.any) {
    if (threadIdx.x == 0 && !length_ok(p, w.n)) set_error(p.err, kErrDeviceIndex);
    return;
  }
  const int pos0 = (w.block << 4) + 8 * half, g = lane >> 2, t = lane & 3;
  if (pos0 + 7 < w.p0 || pos0 >= w.n) return;
  const size_t row = (size_t)p.nkv * D;
  const bf16* src = (part < 2 ? k_new : v_new) + (long long)w.b * p.Q * row + (long long)(pos0 - w.p0) * row + w.h * D;
  if (part < 2) {
    const int pos = pos0 + g;
    const bool in = pos >= w.p0 && pos < w.n;
    uint4 x[L::W];
#pragma unroll
    for (int j = 0; j < L::W; ++j)
      x[j] = in ? __ldg(reinterpret_cast<const uint4*>(src + g * (long long)row + 32 * j + 8 * t)) : make_uint4(0u, 0u, 0u, 0u);
    if (w.pg < 0 || w.pg >= p.P) {
      if (lane == 0) set_error(p.err, kErrDeviceIndex);
      return;
    }
    append_keys<D>(x, in, pool + block_of(p, w) * L::kBytes, 8 * half + g, t);
  } else {
    const int pos = pos0 + 2 * t;
    const bool in[2] = {pos >= w.p0 && pos < w.n, pos + 1 >= w.p0 && pos + 1 < w.n};
    uint2 x[2][L::W];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int m = 0; m < L::W; ++m)
        x[e][m] = in[e] ? __ldg(reinterpret_cast<const uint2*>(src + (2 * t + e) * (long long)row + 32 * m + 4 * g))
                        : make_uint2(0u, 0u);
    if (w.pg < 0 || w.pg >= p.P) {
      if (lane == 0) set_error(p.err, kErrDeviceIndex);
      return;
    }
    append_values<D>(x, in, pool + block_of(p, w) * L::kBytes, half, lane);
  }
}

// (n - 8) s of the nibbles in bits 0..3 and 16..19, by the scales in the halves of s: as bf16, 128 + n' is the
// nibble beneath an exponent, less 136 is exact, and the product is rounded once.
__device__ __forceinline__ uint32_t value2(uint32_t w, uint32_t s) {
  const uint32_t b = (w & 0x000F000Fu) | 0x43004300u, o = 0x43084308u;
  const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&b), *reinterpret_cast<const __nv_bfloat162*>(&o)),
                                   *reinterpret_cast<const __nv_bfloat162*>(&s));
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int D>
__global__ void __launch_bounds__(kQwWarps * 32) q4_read_kernel(const uint8_t* __restrict__ pool, bf16* k_out,
                                                                bf16* v_out, const QwParams p) {
  using L = Q4Block<D>;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, half = part & 1, g = lane >> 2, t = lane & 3;
  QwPlace w = place(p, blockIdx.x);
  const bool there = w.any && w.pg >= 0 && w.pg < p.P, bad = !length_ok(p, w.n);
  if (threadIdx.x == 0 && (bad || (w.any && !there))) set_error(p.err, kErrDeviceIndex);
  if (bad) {  // the rows are zeros, laid out as if the last position were the last of a block
    w.n = p.nblk << 4;
    w.p0 = w.n - p.Q;
    w.block = q4_floor_block(w.p0) + (blockIdx.x / p.nkv) % p.nblk;
  }
  const uint8_t* blk = pool + (there ? block_of(p, w) * L::kBytes : 0);
  const int pos0 = w.block * 16 + 8 * half;
  const size_t row = (size_t)p.nkv * D;
  bf16* out = (part < 2 ? k_out : v_out) + (long long)w.b * p.Q * row + (long long)(pos0 - w.p0) * row + w.h * D;
  if (part < 2) {
    const int pos = pos0 + g, tk = 8 * half + g;
    if (pos < w.p0 || pos >= w.n) return;
    uint4* dst = reinterpret_cast<uint4*>(out + g * (long long)row + 8 * t);
    Q4Words<L::W> c = {};
    uint32_t sc = 0;
    if (there) {
      c = q4_load<L::W>(blk + tk * (D / 2) + t * (4 * L::W));
      sc = q4_load_scales<L::G>(blk + L::kKs + tk * 2 * L::G);
    }
#pragma unroll
    for (int j = 0; j < L::W; ++j) {
      const uint32_t s = __byte_perm(sc, 0, (j >> 1) ? 0x3232 : 0x1010);
      dst[4 * j] = there ? make_uint4(value2(c.w[j], s), value2(c.w[j] >> 4, s), value2(c.w[j] >> 8, s), value2(c.w[j] >> 12, s))
                         : make_uint4(0u, 0u, 0u, 0u);
    }
  } else {
    Q4Words<L::W> c = {};
    uint32_t sc[2] = {0u, 0u};
    if (there) {
      c = q4_load<L::W>(blk + L::kV + (half * 32 + lane) * (4 * L::W));
#pragma unroll
      for (int e = 0; e < 2; ++e) sc[e] = q4_load_scales<L::G>(blk + L::kVs + (8 * half + 2 * t + e) * 2 * L::G);
    }
    const int pos = pos0 + 2 * t;
    const bool in[2] = {pos >= w.p0 && pos < w.n, pos + 1 >= w.p0 && pos + 1 < w.n};
    uint2* dst = reinterpret_cast<uint2*>(out + (2 * t) * (long long)row + 4 * g);
#pragma unroll
    for (int m = 0; m < L::W; ++m) {
      // both positions at a time, then apart
      const uint32_t s = __byte_perm(sc[0], sc[1], (m >> 1) ? 0x7632 : 0x5410);
      uint32_t v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = there ? value2(c.w[m] >> (4 * q), s) : 0u;
      if (in[0]) dst[8 * m] = make_uint2(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410));
      if (in[1])
        *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(dst + 8 * m) + row) =
            make_uint2(__byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
    }
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int log2i(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Shared by both calls: sizes, pointers, grid.
lsv_status prepare(const void* a, const void* b, const void* pool, const int32_t* table, const int32_t* ctx_len,
                   int32_t B, int32_t Q, int32_t nkv, int32_t d, int32_t page, int32_t M, int32_t P, QwParams* p,
                   int* grid, bool* empty) {
  *empty = false;
  if (B < 0 || Q < 0 || nkv < 1 || d < 1 || page < 1 || M < 1 || P < 1) return LSV_ERR_INVALID_ARG;
  if (!q4_dim_ok(d) || !q4_page_ok(page) || nkv > 1024 || (long long)M * page > (1ll << 30) || Q > (1 << 30) ||
      (long long)B * M >= (1ll << 31))
    return LSV_ERR_UNSUPPORTED;
  const long long nblk = (Q + 14) / 16 + 1;  // the most blocks that Q consecutive positions touch
  const long long units = (long long)B * nblk * nkv;
  if (units >= (1ll << 31)) return LSV_ERR_UNSUPPORTED;
  if (B == 0 || Q == 0) {
    *empty = true;
    return LSV_OK;
  }
  if (!a || !b || !pool || !table || !ctx_len) return LSV_ERR_INVALID_ARG;
  if (!al16(a) || !al16(b) || !al16(pool) || !al16(table) || !al16(ctx_len)) return LSV_ERR_MISALIGNED;
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  p->table = table;
  p->ctx_len = ctx_len;
  p->B = B;
  p->Q = Q;
  p->nkv = nkv;
  p->M = M;
  p->P = P;
  p->page_shift = log2i(page);
  p->nblk = (int)nblk;
  p->err = dc->err;
  *grid = (int)units;
  return LSV_OK;
}

}  // namespace
}  // namespace lsv

using namespace lsv;

extern "C" {

size_t spec_q4_page_bytes(int32_t nkv, int32_t d, int32_t page) {
  if (nkv < 1 || nkv > 1024 || !q4_dim_ok(d) || !q4_page_ok(page)) return 0;
  return (size_t)nkv * (page / kQ4Block) * q4_block_bytes(d);
}

lsv_status spec_q4_append(const void* k_new, const void* v_new, void* pool, const int32_t* table,
                          const int32_t* ctx_len, int32_t B, int32_t Q, int32_t nkv, int32_t d, int32_t page,
                          int32_t M, int32_t P, lsv_stream stream) {
  QwParams p;
  int grid = 0;
  bool empty;
  const lsv_status st = prepare(k_new, v_new, pool, table, ctx_len, B, Q, nkv, d, page, M, P, &p, &grid, &empty);
  if (st != LSV_OK || empty) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      d == 128 ? launch_pdl(q4_append_kernel<128>, dim3(grid), dim3(kQwWarps * 32), 0, s, static_cast<const bf16*>(k_new),
                            static_cast<const bf16*>(v_new), static_cast<uint8_t*>(pool), p)
               : launch_pdl(q4_append_kernel<64>, dim3(grid), dim3(kQwWarps * 32), 0, s, static_cast<const bf16*>(k_new),
                            static_cast<const bf16*>(v_new), static_cast<uint8_t*>(pool), p);
  return e == cudaSuccess ? LSV_OK : LSV_ERR_CUDA;
}

lsv_status spec_q4_read(const void* pool, const int32_t* table, const int32_t* ctx_len, int32_t B, int32_t N,
                        int32_t nkv, int32_t d, int32_t page, int32_t M, int32_t P, void* k_out, void* v_out,
                        lsv_stream stream) {
  QwParams p;
  int grid = 0;
  bool empty;
  const lsv_status st = prepare(k_out, v_out, pool, table, ctx_len, B, N, nkv, d, page, M, P, &p, &grid, &empty);
  if (st != LSV_OK || empty) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      d == 128 ? launch_pdl(q4_read_kernel<128>, dim3(grid), dim3(kQwWarps * 32), 0, s, static_cast<const uint8_t*>(pool),
                            static_cast<bf16*>(k_out), static_cast<bf16*>(v_out), p)
               : launch_pdl(q4_read_kernel<64>, dim3(grid), dim3(kQwWarps * 32), 0, s, static_cast<const uint8_t*>(pool),
                            static_cast<bf16*>(k_out), static_cast<bf16*>(v_out), p);
  return e == cudaSuccess ? LSV_OK : LSV_ERR_CUDA;
}

}  // extern "C"
