// logprobs.cu -- what is read off rows of logits beside their greedy token: the log probability of a given token, the
// entropy of the distribution, and the most likely tokens with their log probabilities.
//
//   m = max_v x_v,  S = sum_v e^(x_v - m),  D = sum_v (x_v - m) e^(x_v - m)
//   log p_t = x_t - m - log S,   entropy = log S - D / S
//
// One pass over the logits with the running maximum, S and D of every thread (rescaled where a maximum rises): some eight
// instructions a logit in the pass, one of them an exponential, and half as many again for what is done once a row.  Many
// rows are bound by their bytes (2440 x 100277 fp32 156 us, 0.92 of the copy's rate; 2440 x 129280 bf16 121 us, 0.77), a
// row an SM by those instructions and the row's chain of steps.
//
// The n most likely tokens come of the same pass.  Values and tokens form one 64-bit key (larger value first, then the
// lower token), so that equal logits, which bf16 makes frequent, are no special case.  They lie in the n vectors (16
// bytes of logits) of the largest maxima, so that vectors are collected, by keys of their maxima and places.  Of the
// first logits of every thread, 64 groups of threads give a bound, the n-th largest of their maxima, which n vectors
// reach and few others; every fourth batch the n-th largest of what has come is the new one (2440 x 100277 fp32 156 us
// with it, 168 without).  Where more come than there is room for, the bound rises by what has come, and the vectors are
// collected again behind the pass: with the first quarter of the row masked, 128 x 129280 with 20 tokens 29 us (12.5
// without a mask; a pass over the row for each token 268), 400 x 50000 with 32 37 us (26; 578).  At the end the vectors,
// some dozens, are ranked by counting, and the logits of the first n of them, from the bound on, once more.
//
// A row is one CTA, or a cluster of up to 16 where there are few rows: its CTAs take a piece each, and rank 0 joins
// their sums and ranks their candidates, through distributed shared memory, in a fixed order.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "internal.h"
#include "lsv.h"
#include "ptx.cuh"
#include "q4ptx.cuh"
#include "q8.cuh"

namespace lsv {
namespace {

constexpr int kLpWide = 512, kLpNarrow = 256, kLpTiny = 128;  // threads a CTA
constexpr int kLpGroups = 64;
constexpr int kLpLong = 8, kLpShort = 4;  // 16-byte vectors a thread takes at once
constexpr int kLpMaxTop = 32;      // most alternatives
constexpr int kLpCandidates = 1024;  // room for the vectors that are collected
constexpr int kLpMaxCluster = 16;
constexpr int kLpFew = 128;          // vectors whose logits are looked at without ranking them first
constexpr int kLpPeriod = 4;         // batches between two looks at how many vectors have come (a power of two)
constexpr float kLpNoBound = -1000.0f;  // a bound that a mask may have left so low
static_assert(kLpMaxTop <= kLpGroups && kLpMaxTop == 32 && kLpMaxCluster <= 2 * kLpNarrow / 32, "lists");

// Larger value first, then the lower token; never 0.  -0 and 0 are equal.
__device__ __forceinline__ uint64_t lp_key(float x, int v) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return ((uint64_t)(u & 0x80000000u ? ~u : u | 0x80000000u) << 32) | (uint32_t)~v;
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t u = (uint32_t)(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// e^(x - m) is 2^l with l = x log2 e + c, c = -m log2 e as it is rounded: one FMA a logit, and what the rounding of c
// leaves out is the same factor in every term (its logarithm to base 2).  For a maximum of 2^16 and more, where that
// factor may be anything, l = (x - m) log2 e, two operations.
__device__ __forceinline__ bool large(float m) { return !(fabsf(m) < 65536.0f); }
__device__ __forceinline__ float left_out(float m) { return large(m) ? 0.0f : fmaf(m, kLog2e, __fmul_rn(-m, kLog2e)); }

// Sums over a part of a row, relative to its maximum m: s = sum 2^l, d = sum l 2^l.  A NaN or +infinity makes s NaN, and
// it stays so.
struct Part {
  float m, s, d;
};
__device__ __forceinline__ void move_to(Part& a, float m) {
  if (a.s != 0.0f) {
    const float by = (a.m - m) * kLog2e + (left_out(m) - left_out(a.m)), c = ex2_ftz(by);
    a.d = c > 0.0f || isnan(c) ? c * fmaf(by, a.s, a.d) : 0.0f;
    a.s *= c;
  }
  a.m = m;
}
// The sums of `width` lanes (a power of two), in each of them: their maximum first, then every lane's share of it.
__device__ __forceinline__ Part join_lanes(Part a, int width) {
  float m = a.m;
  for (int o = width / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  move_to(a, m);
  for (int o = width / 2; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.d += __shfl_xor_sync(0xffffffffu, a.d, o);
  }
  return a;
}
__device__ __forceinline__ void add_one(Part& a, float x) {
  if (!(x <= a.m)) move_to(a, x);
  if (a.m == -INFINITY) return;
  // (-inf counts as e^-1000 = 0, so that it adds 0 and not 0 * inf)
  const float l = max_nan(large(a.m) ? (x - a.m) * kLog2e : fmaf(x, kLog2e, __fmul_rn(-a.m, kLog2e)), -1000.0f);
  const float e = ex2_ftz(l);
  a.s += e;
  a.d = fmaf(l, e, a.d);
}
template <typename T>
struct Vec;
template <>
struct Vec<bf16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;  // -inf, -inf
  static __device__ __forceinline__ float2 two(const uint4& v, int i) {
    const uint32_t w = i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  typedef __nv_bfloat162 Two;
  static __device__ __forceinline__ Two two_max(const uint4& v) {
    const Two* t = reinterpret_cast<const Two*>(&v);
    return __hmax2_nan(__hmax2_nan(t[0], t[1]), __hmax2_nan(t[2], t[3]));
  }
  static __device__ __forceinline__ float max_of(const uint4& v) {
    const Two m = two_max(v);
    return max_nan(__low2float(m), __high2float(m));
  }
  template <int B>
  static __device__ __forceinline__ float max_of(const uint4 (&v)[B]) {
    Two m[B];
#pragma unroll
    for (int i = 0; i < B; ++i) m[i] = two_max(v[i]);
#pragma unroll
    for (int o = 1; o < B; o *= 2)
#pragma unroll
      for (int i = 0; i < B; i += 2 * o) m[i] = __hmax2_nan(m[i], m[i + o]);
    return max_nan(__low2float(m[0]), __high2float(m[0]));
  }
  static __device__ __forceinline__ Two low(float f) { return __float2bfloat162_rn(f); }
  static __device__ __forceinline__ void raise(uint4& v, Two low) {
    Two* t = reinterpret_cast<Two*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = __hmax2_nan(t[i], low);
  }
  static __device__ __forceinline__ float get(const bf16* p) { return __bfloat162float(*p); }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ float2 two(const uint4& v, int i) {
    return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                  : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ float max_of(const uint4& v) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  template <int B>
  static __device__ __forceinline__ float max_of(const uint4 (&v)[B]) {
    float m[B];
#pragma unroll
    for (int i = 0; i < B; ++i) m[i] = max_of(v[i]);
#pragma unroll
    for (int o = 1; o < B; o *= 2)
#pragma unroll
      for (int i = 0; i < B; i += 2 * o) m[i] = max_nan(m[i], m[i + o]);
    return m[0];
  }
  static __device__ __forceinline__ float low(float f) { return f; }
  static __device__ __forceinline__ void raise(uint4& v, float low) {
    float* t = reinterpret_cast<float*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = max_nan(t[i], low);
  }
  static __device__ __forceinline__ float get(const float* p) { return *p; }
};

struct __align__(16) LpSmem {
  uint64_t cand[kLpCandidates];  // at first the threads' largest vectors
  uint64_t last[kLpFew * 8 + 16];
  uint64_t group[kLpGroups];
  uint64_t top[kLpMaxCluster][kLpMaxTop];   // the CTA's largest in order, 0 behind them; rank 0's: every rank's
  Part parts[kLpMaxCluster];                // rank 0's: every rank's sums
  Part warp[kLpWide / 32];
  uint64_t bound;
  int2 ncand;  // vectors, and whether some have been left out for want of room
  int nlast;   // logits at the end
};

// Two lists of 32 keys in falling order, one a lane and the other from its end: the 32 largest, in falling order.
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b_reversed, int lane) {
  uint64_t k = a > b_reversed ? a : b_reversed;  // rises and then falls, or the other way round
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, k, o);
    k = ((lane & o) == 0) == (other > k) ? other : k;
  }
  return k;
}

// The n largest of `cnt` different keys, in order, to dst (0 where there are fewer): each key's place is the number of
// larger ones, counted by 1 to 32 threads.
template <int THREADS>
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int cnt, uint64_t* dst, int n) {
  int log_by = 5;
  while (log_by > 0 && cnt << log_by > THREADS) --log_by;
  const int by = 1 << log_by, each = THREADS >> log_by, part = threadIdx.x & (by - 1);
  // (warps that have no key left are done)
  for (int i0 = 0; i0 + ((int)(threadIdx.x & ~31u) >> log_by) < cnt; i0 += each) {
    const int i = i0 + ((int)threadIdx.x >> log_by);
    const uint64_t k = i < cnt ? keys[i] : 0;
    int r = 0;
#pragma unroll 4
    for (int j = 2 * part; j < cnt; j += 2 * by) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(keys + j);
      r += (two.x > k) + (j + 1 < cnt && two.y > k);
    }
    for (int o = 1; o < by; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    if (part == 0 && k != 0 && r < n) dst[r] = k;
  }
}

// A thread's key to its group's largest (groups of a power of two of lanes); and, a barrier later, the bound from the
// groups, the n-th largest of them, where it is above the one that there is.
__device__ __forceinline__ void to_groups(LpSmem& sm, uint64_t key, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) {
    const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
    key = other > key ? other : key;
  }
  if ((threadIdx.x & (lanes - 1)) == 0 && threadIdx.x < lanes * kLpGroups) sm.group[threadIdx.x / lanes] = key;
}
template <int THREADS>
__device__ __forceinline__ void bound_of_groups(LpSmem& sm, int n, uint64_t bound) {
  constexpr int kInGroup = THREADS / kLpGroups;
  const int mine = threadIdx.x / kInGroup, part = threadIdx.x % kInGroup;  // a group is ranked by so many
  const uint64_t key = sm.group[mine];
  int r = 0;
#pragma unroll
  for (int j = part; j < kLpGroups; j += kInGroup) r += sm.group[j] > key || (sm.group[j] == key && j < mine);
#pragma unroll
  for (int o = 1; o < kInGroup; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  if (part == 0 && r == n - 1 && key > bound) sm.bound = key;
}

// The groups' largest of the vectors that found room.
template <int THREADS>
__device__ __forceinline__ void groups_of_list(LpSmem& sm) {
  uint64_t key = 0;
#pragma unroll 1
  for (int i = threadIdx.x; i < kLpCandidates; i += THREADS) key = sm.cand[i] > key ? sm.cand[i] : key;
  to_groups(sm, key, THREADS / kLpGroups);
}

// More vectors came than there is room for (the row begins far below the rest, as masks leave it, or rises): those of the
// places q0 to q1 once more, from a bound on that leaves few: that of the last ones' groups, and where it leaves too many,
// once the groups' over all of the places.  Every other look leaves out 500 vectors more, at least: the rest of what found
// room.  All threads, after a barrier; the caller takes the bound and the number of vectors from sm.
template <typename T, int THREADS, int BATCH>
__device__ __forceinline__ void collect_again(LpSmem& sm, const T* xv, int q0, int q1, int n) {
  auto keys = [&](auto with) {  // each of this thread's
#pragma unroll 1
    for (int q = q0 + (int)threadIdx.x; q < q1; q += BATCH * THREADS) {
      uint4 w[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (q + i * THREADS < q1) w[i] = ld_plain128(xv + (size_t)(q + i * THREADS) * Vec<T>::N);
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (q + i * THREADS < q1) with(lp_key(Vec<T>::max_of(w[i]), q + i * THREADS));
    }
  };
  bool many = sm.ncand.x > kLpCandidates;  // (else: the bound has been taken from what came before)
#pragma unroll 1
  for (int turn = 0;; ++turn) {
    const uint64_t below = sm.bound;
    if (turn == 1) {
      uint64_t key = 0;
      keys([&](uint64_t other) { key = other > key ? other : key; });
      to_groups(sm, key, THREADS / kLpGroups);
    } else if (many) {
      groups_of_list<THREADS>(sm);
    }
    __syncthreads();
    if (many) bound_of_groups<THREADS>(sm, n, below);
    if (threadIdx.x == 0) sm.ncand.x = 0;
    __syncthreads();
    const uint64_t bound = sm.bound;
    keys([&](uint64_t key) {
      if (key < bound) return;
      const int c = atomicAdd(&sm.ncand.x, 1);
      if (c < kLpCandidates) sm.cand[c] = key;
    });
    __syncthreads();
    many = sm.ncand.x > kLpCandidates;
    if (!many) return;
    __syncthreads();
  }
}

// CTAs of THREADS that take BATCH vectors a thread at once: 16 KB of logits in flight and as much again behind them, four
// CTAs an SM, or 32 KB and two, or 64 KB and one, or 8 KB and eight.
template <typename T, int THREADS, int BATCH>
__global__ void __launch_bounds__(THREADS, 4096 / (THREADS * BATCH))
    logprobs_kernel(const T* logits, const int32_t* tokens, int V, int n, int cs, float* logprob, float* entropy,
                    int32_t* top_ids, float* top_logprobs, int* err) {
  constexpr int N = Vec<T>::N;
  constexpr int kWarps = THREADS / 32, kInGroup = THREADS / kLpGroups;
  __shared__ LpSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / cs, rank = blockIdx.x - row * cs;
  if (cs > 1) cluster_arrive_relaxed();  // all of the cluster run before anything is sent to rank 0
  pdl_wait();
  pdl_trigger();
  const T* x = logits + (size_t)row * V;
  // Whole 16-byte vectors of the row lie from element `head` on; rank 0 takes the elements before them, the last
  // rank those behind them.
  const int head = min(V, (int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T));
  const int nv = (V - head) / N, tail = head + nv * N;
  const T* xv = x + head;
  const int k0 = (int)((long long)nv * rank / cs), k1 = (int)((long long)nv * (rank + 1) / cs);

  // what the end needs of global memory comes meanwhile
  int token = -1;
  float at_token = 0.0f;
  if (logprob && rank == 0 && tid == 0) {
    token = tokens[row];
    if (token >= 0 && token < V) at_token = Vec<T>::get(x + token);
  }

  // ------------------------------------------------------------ one pass: sums, and the candidates
  Part a = {-INFINITY, 0.0f, 0.0f};
  uint4 v[BATCH];
  auto load = [&](int k) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int q = k + i * THREADS;
      v[i] = q < k1 ? ld_stream128(xv + (size_t)q * N)
                    : make_uint4(Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone, Vec<T>::kNone);
    }
  };
  load(k0 + tid);
  if (tid == 0) {
    sm.ncand = make_int2(0, 0);
    sm.nlast = 0;
    sm.bound = 0;
  }
  if (tid < kLpMaxTop) sm.top[0][tid] = 0;
  uint64_t bound = 0;  // the key of a vector: its largest logit, then its place
  float bv = -INFINITY;
  auto set_bound = [&]() {
    bound = sm.bound;
    bv = bound ? key_value(bound) : -INFINITY;
  };
  float2 s2 = make_float2(0.f, 0.f), d2 = s2;
  float c = 0.0f;                   // of l
  auto low = Vec<T>::low(0.0f);
  const int batches = (k1 - k0 + BATCH * THREADS - 1) / (BATCH * THREADS);
#pragma unroll 1
  for (int b = 0; b < batches; ++b) {
    const int k = k0 + tid + b * (BATCH * THREADS);
    uint4 u[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) u[i] = v[i];
    if (b + 1 < batches) load(k + BATCH * THREADS);
    const float bm = Vec<T>::max_of(u);
    if (!(bm <= a.m)) {
      a.s = s2.x + s2.y;
      a.d = d2.x + d2.y;
      move_to(a, bm);
      s2 = make_float2(a.s, 0.f);
      d2 = make_float2(a.d, 0.f);
      c = __fmul_rn(-a.m, kLog2e);
      // logits below it add nothing to s; raised to it they add nothing to d either, where -inf and the type's lowest
      // value would add 0 * inf
      low = Vec<T>::low(a.m - 1000.0f);
    }
    if (b == 0 && n > 0) {
      // The first bound: each thread's vector of the largest maximum, a group's largest of them (of fewer threads where
      // there are few vectors), and the groups' places among themselves, below.
      uint64_t key = 0;
      if (k < k1 && !isnan(bm)) {
        int first = 0;
#pragma unroll
        for (int i = BATCH - 1; i > 0; --i)
          if (Vec<T>::max_of(u[i]) == bm) first = i;
        if (Vec<T>::max_of(u[0]) == bm) first = 0;
        key = lp_key(bm, k + first * THREADS);
      }
      int lanes = 1;
      while (lanes < kInGroup && lanes * kLpGroups < k1 - k0) lanes <<= 1;
      to_groups(sm, key, lanes);
    }
    if (!large(a.m)) {
      const float2 mul = make_float2(kLog2e, kLog2e), add = make_float2(c, c);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        uint4 w = u[i];
        Vec<T>::raise(w, low);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float2 l = fma2(Vec<T>::two(w, j), mul, add);
          const float2 e = make_float2(ex2_ftz(l.x), ex2_ftz(l.y));
          s2 = add2(s2, e);
          d2 = fma2(l, e, d2);
        }
      }
    } else if (a.m != -INFINITY) {  // (nothing but -inf so far)
      // read once more, so that this rare form takes no registers from the other
#pragma unroll 1
      for (int q = k; q < min(k1, k + BATCH * THREADS); q += THREADS) {
        const uint4 w = ld_plain128(xv + (size_t)q * N);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          const float2 f = Vec<T>::two(w, j);
          const float2 l = make_float2(max_nan((f.x - a.m) * kLog2e, -1000.0f), max_nan((f.y - a.m) * kLog2e, -1000.0f));
          const float2 e = make_float2(ex2_ftz(l.x), ex2_ftz(l.y));
          s2 = add2(s2, e);
          d2 = fma2(l, e, d2);
        }
      }
    }
    if (n == 0) continue;
    if (b == 0) {
      __syncthreads();
      bound_of_groups<THREADS>(sm, n, 0);
      __syncthreads();
      set_bound();
    }
    if (bm >= bv) {
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int q = k + i * THREADS;
        const float vm = Vec<T>::max_of(u[i]);
        if (q >= k1 || vm < bv) continue;
        const uint64_t key = lp_key(vm, q);
        if (key < bound) continue;
        const int c = atomicAdd(&sm.ncand.x, 1);
        if (c < kLpCandidates) sm.cand[c] = key;
      }
    }
    if ((b + 1) % kLpPeriod == 0 && b + 1 < batches) {
      __syncthreads();
      const int cnt = sm.ncand.x;
      if (__builtin_expect(cnt > kLpCandidates, 0)) {
        // too many: the bound rises all the same, and they are collected again behind the pass
        groups_of_list<THREADS>(sm);
        __syncthreads();
        bound_of_groups<THREADS>(sm, n, bound);
        if (tid == 0) {
          sm.ncand = make_int2(0, 1);
        }
      } else if (cnt > 2 * n + 8) {
        rank_keys<THREADS>(sm.cand, cnt, sm.group, n);
        __syncthreads();
        if (tid < n) sm.cand[tid] = sm.group[tid];
        if (tid == 0) {
          sm.ncand.x = n;
          sm.bound = sm.group[n - 1];
        }
      }
      __syncthreads();
      set_bound();
    }
  }
  a.s = s2.x + s2.y;
  a.d = d2.x + d2.y;

  // the elements outside whole vectors
  int edge = -1;
  if (rank == 0 && tid < head) edge = tid;
  if (rank == cs - 1 && tid >= 32 && tid - 32 < V - tail) edge = tail + tid - 32;
  const float ex = edge >= 0 ? Vec<T>::get(x + edge) : -INFINITY;
  if (edge >= 0) add_one(a, ex);

  if (n > 0) __syncthreads();  // every candidate is there
  const int2 came = n > 0 ? sm.ncand : make_int2(0, 0);
  int cnt = came.x;
  if (__builtin_expect(came.y != 0 || cnt > kLpCandidates, 0)) {
    collect_again<T, THREADS, BATCH>(sm, xv, k0, k1, n);
    cnt = sm.ncand.x;
    set_bound();
  }
  // The logits of the vectors, of the first n of them where they are many (or theirs would be, above no bound to speak of),
  // from the bound on.
  const uint64_t* from = sm.cand;
  int vectors = cnt;
  if (cnt > (bv < kLpNoBound ? n : kLpFew)) {
    rank_keys<THREADS>(sm.cand, cnt, sm.group, n);
    __syncthreads();
    from = sm.group;
    vectors = n;
    bv = key_value(sm.group[n - 1]);
  }
  int t0 = -1;
  float f0 = 0.0f;
  if (tid < vectors * N) {
    t0 = head + key_token(from[tid / N]) * N + tid % N;
    f0 = Vec<T>::get(x + t0);  // on its way while the lanes' sums are joined
  }
  a = join_lanes(a, 32);
  if (lane == 0) sm.warp[warp] = a;
  if (n > 0) {
    auto offer = [&](float f, int t) {
      if (!(f < bv)) sm.last[atomicAdd(&sm.nlast, 1)] = lp_key(f, t);
    };
    if (t0 >= 0) offer(f0, t0);
    for (int i = tid + THREADS; i < vectors * N; i += THREADS) {
      const int t = head + key_token(from[i / N]) * N + i % N;
      offer(Vec<T>::get(x + t), t);
    }
    if (edge >= 0) offer(ex, edge);
    __syncthreads();
    rank_keys<THREADS>(sm.last, sm.nlast, sm.top[0], n);
  }
  if (n == 0) __syncthreads();  // the warps' sums are there
  if (warp == kWarps - 1) {              // (the others rank)
    a = join_lanes(sm.warp[lane & (kWarps - 1)], kWarps);
    if (lane == 0) sm.parts[0] = a;
  }
  __syncthreads();

  // ------------------------------------------------------------ the cluster's
  if (cs > 1) {
    cluster_wait();
    if (rank > 0 && warp == 0) {
      if (lane == 0) {
        a = sm.parts[0];
        const uint32_t to = mapa_shared(smem_u32(&sm.parts[rank]), 0);
        st_shared_cluster_f32(to, a.m);
        st_shared_cluster_f32(to + 4, a.s);
        st_shared_cluster_f32(to + 8, a.d);
      }
      if (n > 0) {
        const uint32_t to = mapa_shared(smem_u32(&sm.top[rank][lane]), 0);
        const uint64_t k = sm.top[0][lane];
        st_shared_cluster_s32(to, (int)(uint32_t)k);
        st_shared_cluster_s32(to + 4, (int)(uint32_t)(k >> 32));
      }
    }
    cluster_sync();
    if (rank > 0) return;
    if (warp == 0) {
      a = join_lanes(sm.parts[lane & (cs - 1)], cs);
      __syncwarp();
      if (lane == 0) sm.parts[0] = a;
    }
    // the ranks' lists, two by two
    for (int o = 1; n > 0 && o < cs; o *= 2) {
      const int r = 2 * o * warp;
      if (r < cs) sm.top[r][lane] = merge_lists(sm.top[r][lane], sm.top[r + o][31 - lane], lane);
      __syncthreads();
    }
  }
  __syncthreads();

  // ------------------------------------------------------------ out
  a = sm.parts[0];
  const bool bad = isnan(a.s);      // a NaN or +infinity among the logits
  const bool none = a.s == 0.0f;    // nothing but -inf
  const float log_s = logf(a.s), log_sum = log_s - left_out(a.m) * kLn2;
  // What is next to certain has a log probability next to 0, and rounding may put it above (an entropy below): neither
  // leaves the side that it lies on.
  auto log_p = [&](float x) {
    const float p = (x - a.m) - log_sum;
    return p > 0.0f ? 0.0f : p;
  };
  if (tid == 0 && logprob) {
    float p = 0.0f;  // -1: no token
    if (token < -1 || token >= V) {
      set_error(err, kErrDeviceIndex);
      p = NAN;
    } else if (token >= 0) {
      p = bad ? NAN : none ? -INFINITY : log_p(at_token);
    }
    logprob[row] = p;
  }
  if (tid == 32 && entropy) {
    const float h = none ? 0.0f : fmaf(-kLn2, a.d / a.s, log_s);
    entropy[row] = bad ? NAN : h < 0.0f ? 0.0f : h;
  }
  if (tid < n) {
    const uint64_t k = sm.top[0][tid];
    const bool there = k != 0 && !bad;
    top_ids[(size_t)row * n + tid] = there ? key_token(k) : -1;
    top_logprobs[(size_t)row * n + tid] = bad ? NAN : !there || none ? -INFINITY : log_p(key_value(k));
  }
}

template <typename T>
cudaError_t launch_logprobs(const T* logits, const int32_t* tokens, int R, int V, int n, float* logprob, float* entropy,
                            int32_t* top_ids, float* top_logprobs, const DeviceCtx& dc, cudaStream_t s) {
  // Many rows: narrow CTAs, four an SM; up to two rows an SM, so many that they fill it, and a row an SM, half the threads
  // with twice the vectors (wide), which halves what every warp does once a row, in clusters as far as they are on the GPU
  // at once.  Few rows (a quarter of the SMs at most) of less than 3/4 of a wide CTA's batch each: narrow ones again, as
  // many a row (a cluster) as are there at once, each with a vector a thread at least.  Of 129280 bf16 logits and 20
  // tokens: 24 rows 6.8 us (narrow 7.6; of 60000 logits 30 rows 6.3 and 5.9), 32 rows 6.7 (narrow 7.7), 128 rows 12.5
  // (clusters of 4 narrow ones 17.1), 300 rows 21.3 (narrow 24.2), 600 rows and 5 tokens narrow 33.2 (twice the threads
  // 35.3, wide 41.1).  Rows of one batch gain nothing from threads.  Clusters of 16 narrow ones: one row 5.4 us (8: 6.5),
  // 10 rows 6.2 (6.9).
  const long long bytes = (long long)V * (long long)sizeof(T);
  const bool few = 4ll * R <= dc.num_sms;
  auto* wide = logprobs_kernel<T, kLpWide, kLpLong>;
  static ClustersAtOnce at_once;
  int wide_cs = 1;
  while (wide_cs < kLpMaxCluster / 2 && bytes >= 2ll * wide_cs * kLpWide * 16 &&
         R <= at_once.of(reinterpret_cast<const void*>(wide), 2 * wide_cs, kLpWide, 0, dc.device))
    wide_cs *= 2;
  const bool one = R <= dc.num_sms && bytes > kLpNarrow * kLpShort * 16 &&
                   (!few || bytes >= (long long)wide_cs * (kLpWide * kLpLong * 16 * 3 / 4));
  const bool narrow = !one && (few || R > 2 * dc.num_sms || bytes <= kLpNarrow * kLpShort * 16);
  int threads = kLpWide, cs = one ? wide_cs : 1;
  if (narrow) {
    threads = kLpNarrow;
    const int most = 10ll * R <= dc.num_sms ? kLpMaxCluster : kLpMaxCluster / 2;
    while (cs < most && (long long)R * cs * 2 <= 4ll * dc.num_sms && bytes >= 2ll * cs * threads * 16) cs *= 2;
  }
  auto* kernel = narrow ? logprobs_kernel<T, kLpNarrow, kLpShort> : one ? wide : logprobs_kernel<T, kLpWide, kLpShort>;
  // Short rows: what is done once a row is most of it, and tiny CTAs, eight an SM, have twice the rows at it.  Rows of one
  // of their batches (8 KB), or of four where there are more rows than fit at once: 2000 x 200 bf16 11.9 us (narrow 17.5),
  // 2301 x 5910 17.8 (23.9), 2440 x 16384 26.7 (31.5); 700 x 8192 12.3 (9.6).
  if (narrow && cs == 1 && bytes <= (R > 8 * dc.num_sms ? 4 : 1) * kLpTiny * kLpShort * 16) {
    kernel = logprobs_kernel<T, kLpTiny, kLpShort>;
    threads = kLpTiny;
  }
  static std::atomic<bool> asked[64];  // clusters of 16 allowed on the device
  if (cs > 8 && !asked[dc.device].load()) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    asked[dc.device].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)R * cs));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cs;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cs > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, logits, tokens, V, n, cs, logprob, entropy, top_ids, top_logprobs, dc.err);
}

}  // namespace
}  // namespace lsv

using namespace lsv;

extern "C" lsv_status spec_logprobs(const void* logits, int32_t logits_fp32, const int32_t* tokens, int32_t R, int32_t V,
                                    int32_t n, float* logprob, float* entropy, int32_t* top_ids, float* top_logprobs,
                                    lsv_stream stream) {
  if (R < 0 || V <= 0 || n < 0) return LSV_ERR_INVALID_ARG;
  if (n > kLpMaxTop || V > (1 << 30)) return LSV_ERR_UNSUPPORTED;
  if (R == 0) return LSV_OK;
  if (!logits || (logprob && !tokens) || (n > 0 && (!top_ids || !top_logprobs))) return LSV_ERR_INVALID_ARG;
  const void* ptrs[] = {logits, tokens, logprob, entropy, top_ids, top_logprobs};
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 15) return LSV_ERR_MISALIGNED;
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = logits_fp32 ? launch_logprobs(static_cast<const float*>(logits), tokens, R, V, n, logprob, entropy,
                                                      top_ids, top_logprobs, *dc, s)
                                    : launch_logprobs(static_cast<const bf16*>(logits), tokens, R, V, n, logprob, entropy,
                                                      top_ids, top_logprobs, *dc, s);
  return e == cudaSuccess ? LSV_OK : LSV_ERR_CUDA;
}
