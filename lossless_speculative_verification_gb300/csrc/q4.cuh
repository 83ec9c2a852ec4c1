// q4.cuh -- the paged key/value cache held in 4 bits: its layout.
//
// A group of 64 dims of one position, head and tensor shares a bf16 scale
// s = bf16(max |x| / 7); a code n = rint(x / s) in [-8, 7] stands for n s and is
// stored as the nibble n + 8.  A group that holds a NaN or an infinity has the
// scale NaN, so whatever reads the position reads NaN; a group whose scale is 0
// stands for zeros.
//
// The unit in memory is a block: 16 positions of one head, in the order in
// which a warp's m16n8k16 fragments take them, so that a lane's share is one
// vector load and no shared memory or ldmatrix stands between.  With g = lane / 4
// and t = lane % 4 and W = d / 32 words a lane:
//   keys    [position 16][t 4][W] words: word j of lane t holds the dims
//           32 j + 8 t + 0..7 of its position, nibble r / 2 + 4 (r % 2) the dim r,
//           so that the two halves of a word hold the dims 2 p and 2 p + 1;
//   values  [half 2][g 8][t 4][W] words: the lower 16 bits of word m hold the dims
//           32 m + 4 g + 0..3 of position 8 half + 2 t, the upper ones those of the
//           position after it;
//   key scales [16][d / 64], value scales [16][d / 64] (bf16).
// A page is [kv heads][page / 16][block]; a pool [P][page].
#pragma once

#include <stdint.h>

namespace lsv {

constexpr int kQ4Group = 64;   // dims that share a scale
constexpr int kQ4Block = 16;   // positions of a block
constexpr uint32_t kQ4NanScale = 0x7FC0u;

template <int D>
struct Q4Block {
  static constexpr int W = D / 32;                // 32-bit words of codes a lane and position (keys), or pair of positions (values)
  static constexpr int G = D / kQ4Group;          // scales a position
  static constexpr int kV = kQ4Block * D / 2;     // byte offsets in a block
  static constexpr int kKs = 2 * kV;
  static constexpr int kVs = kKs + kQ4Block * G * 2;
  static constexpr int kBytes = kVs + kQ4Block * G * 2;
};

__host__ __device__ inline int q4_block_bytes(int d) { return kQ4Block * (d + 4 * (d / kQ4Group)); }

// Pages of 16, 32, 64, 128 or 256 positions.
inline bool q4_page_ok(int page) { return page >= 16 && page <= 256 && (page & (page - 1)) == 0; }
inline bool q4_dim_ok(int d) { return d == 64 || d == 128; }

// W consecutive words as one vector access.
template <int W>
struct Q4Words {
  uint32_t w[W];
};
template <int W>
__device__ __forceinline__ Q4Words<W> q4_load(const uint8_t* p) {
  Q4Words<W> r;
  if constexpr (W == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  }
  return r;
}
template <int W>
__device__ __forceinline__ void q4_store(uint8_t* p, const Q4Words<W>& r) {
  if constexpr (W == 4)
    *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
}
// The G scales (bf16 bits) of one position, the first group's in the lower half.
template <int G>
__device__ __forceinline__ uint32_t q4_load_scales(const uint8_t* p) {
  if constexpr (G == 2)
    return *reinterpret_cast<const uint32_t*>(p);
  else
    return *reinterpret_cast<const uint16_t*>(p);
}
template <int G>
__device__ __forceinline__ void q4_store_scales(uint8_t* p, uint32_t s) {
  if constexpr (G == 2)
    *reinterpret_cast<uint32_t*>(p) = s;
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(s);
}
__device__ __forceinline__ float q4_scale(uint32_t s, int g) {
  return __uint_as_float(g ? (s & 0xFFFF0000u) : (s << 16));
}

// floor(a / 16) for any sign
__device__ __forceinline__ int q4_floor_block(int a) { return a >> 4; }

}  // namespace lsv
