// pages.cu -- the pages of a paged cache: giving room and taking it back, copies
// on write, forks, and compaction.
//
// A pool has P pages, each with a count of the table entries that hold it (0:
// free).  A table [B, M] has a row a sequence: entry i is the page of the
// positions i * page .., or -1.  Every layer's cache goes by the same table.
//
// All three calls are scans over the table and the counts.  Nothing depends on
// the order of atomics: new pages are the free ones of lowest number, given out
// in the order (row, entry), and counts are sums of integers.  The calls read
// their inputs as they were before the call, so each output may be its input.
//
// Two grids do the bookkeeping: the first reduces chunks of kPgChunk counts to
// two bits a page (free, shared) and the rows to the number of pages they need;
// the second begins each CTA with the sums of what lies before it.  The page
// contents follow in a third, which streams a list of (source, destination)
// pairs through the whole GPU.  Small tables are planned by one CTA or cluster.
#include "internal.h"
#include "lsv.h"
#include "ptx.cuh"

namespace lsv {
namespace {

constexpr int kErrPages = LSV_ERR_PAGES;  // a pool had fewer free pages than a call needed
constexpr int kPgThreads = 256;
constexpr int kPgWarps = kPgThreads / 32;
constexpr int kPgChunk = 4096;  // pages a CTA reduces
constexpr int kPgChunkWords = kPgChunk / 32;
constexpr int kPgMaxPages = 1 << 24;
constexpr int kPgMaxRows = 1 << 16;
// Forks of few rows, entries and counts are one launch of a cluster instead of two of a grid: 2.9 us for 2.6 on the
// GPU, 7.9 for 9.6 with the host's calls (32 rows of 36).  (A resize in that form took 16.1 us; one CTA plans it in
// 11.0 with its copies.)
constexpr int kPgCluster = 8;        // CTAs of the cluster
constexpr int kPgGroups = 4;         // rows that each takes at a time
constexpr int kPgFewRows = 64;
constexpr int kPgFewInts = 1 << 16;
constexpr int kPgDeep = 4;      // entries of a row a thread has in flight
// Bytes a CTA copies at a time, all of them in flight, and the CTAs an SM has for it: 979 MB of moves take 158 us with
// two CTAs of 32 KB, 166 with four of 16 KB or 32 KB, 167 with two of 64 KB, 188 with one of 32 KB.
constexpr int kPgCopyBytes = 32768;
constexpr int kPgCopyCtas = 2;

struct PgWs {
  int* need;       // [B] pages a row takes
  int* wrong;      // [B] whether a row's bounds or entries are out of range
  int* chunk_n;    // [chunks] free pages (resize) or live pages (compact) of a chunk
  uint32_t* bits;  // [2, words] bit maps: free, shared
  int* list;       // [max(B * M, P)] page numbers in order of rank (new pages; or the pages that move)
  int* list2;      // [max(B, P)] destinations of the copies
  int* src;        // [B] sources of the copies
  int* rank;       // [P] which of the moving pages a page is, -1: none
  int* count;      // copies
  int32_t* table;  // [B, M] the table as it was, where a fork writes it in place
  size_t total;
};

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

PgWs pg_layout(void* base, size_t B, size_t M, size_t P) {
  PgWs w;
  uint8_t* b = static_cast<uint8_t*>(base);
  size_t o = 0;
  auto take = [&](size_t ints) {
    uint8_t* at = b + o;
    o += round256(ints * 4);
    return at;
  };
  const size_t chunks = (P + kPgChunk - 1) / kPgChunk, bm = B * M;
  w.need = reinterpret_cast<int*>(take(B));
  w.wrong = reinterpret_cast<int*>(take(B));
  w.chunk_n = reinterpret_cast<int*>(take(chunks));
  w.bits = reinterpret_cast<uint32_t*>(take(2 * chunks * kPgChunkWords));
  w.list = reinterpret_cast<int*>(take(bm > P ? bm : P));
  w.list2 = reinterpret_cast<int*>(take(B > P ? B : P));
  w.src = reinterpret_cast<int*>(take(B));
  w.rank = reinterpret_cast<int*>(take(P));
  w.count = reinterpret_cast<int*>(take(64));
  w.table = reinterpret_cast<int32_t*>(take(bm));
  w.total = o;
  return w;
}

// A group of kPgThreads threads that takes a row or a chunk: a CTA, or a quarter of one (the cluster form).
struct PgShared {
  int tmp[kPgWarps];
  int before[kPgThreads];        // free pages below each chunk of a tile of chunks
  int fresh[kPgDeep][kPgWarps];  // new pages of each warp's entries
};
template <int kGroups>
struct Group {
  int tid, id;
  PgShared* sh;
  __device__ __forceinline__ explicit Group(PgShared* all)
      : tid((int)threadIdx.x % kPgThreads), id((int)threadIdx.x / kPgThreads), sh(all + id) {}
  __device__ __forceinline__ void sync() const {
    if (kGroups == 1)
      __syncthreads();
    else
      named_bar_sync(1 + id, kPgThreads);
  }
  __device__ __forceinline__ int lane() const { return tid & 31; }
  __device__ __forceinline__ int warp() const { return tid >> 5; }
  // Sum over the group; every thread gets it.
  __device__ __forceinline__ int sum(int v) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    sync();
    if (lane() == 0) sh->tmp[warp()] = v;
    sync();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kPgWarps; ++w) s += sh->tmp[w];
    return s;
  }
  // Exclusive prefix of v over the group's threads; *all the total.
  __device__ __forceinline__ int prefix(int v, int* all) const {
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane() >= o) s += u;
    }
    sync();
    if (lane() == 31) sh->tmp[warp()] = s;
    sync();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kPgWarps; ++w) {
      if (w < warp()) before += sh->tmp[w];
      total += sh->tmp[w];
    }
    *all = total;
    return before + s - v;
  }
  // Sum of a[0..n), and of a[0..upto) in *part.
  __device__ __forceinline__ int sum_upto(const int* a, int n, int upto, int* part) const {
    int all = 0, pre = 0;
    for (int i = tid; i < n; i += kPgThreads) {
      const int v = __ldcg(a + i);
      all += v;
      if (i < upto) pre += v;
    }
    *part = sum(pre);
    return sum(all);
  }
};

// The counts of chunk c, all loads in flight together: refs[k] of lane l is page 32 (warp + k kPgWarps) + l of it.
__device__ __forceinline__ void load_chunk(const Group<1>& g, const int32_t* ref, int P, int c,
                                           int (&refs)[kPgChunkWords / kPgWarps]) {
#pragma unroll
  for (int k = 0; k < kPgChunkWords / kPgWarps; ++k) {
    const int at = c * kPgChunk + 32 * (g.warp() + k * kPgWarps) + g.lane();
    refs[k] = at < P ? __ldcg(ref + at) : -1;
  }
}

// What a turn does with entry i of a row: keep it, give it a new page, copy the old one into the new one.
struct Entry {
  bool held, fresh, copied, gone;
};
__device__ __forceinline__ Entry entry_of(int i, bool held, bool shared, int keep, int cap, int page) {
  Entry e;
  e.held = held;
  const int kept = (keep + page - 1) / page, wanted = (cap + page - 1) / page;
  e.copied = held && shared && i == keep / page && keep % page != 0 && cap > keep;
  e.fresh = i < wanted && (!held || e.copied || (i >= kept && shared));
  e.gone = held && (e.fresh || i >= wanted);
  return e;
}

struct PgResize {
  const int32_t *table, *ref, *keep, *cap;
  int32_t *table_out, *ref_out, *stats;
  int B, M, P, page, chunks;
  PgWs w;
  int* err;
};

// A row's bounds; false: out of range (the row stays as it is).
__device__ __forceinline__ bool row_bounds(const PgResize& p, int b, int* keep, int* cap) {
  *keep = __ldcg(p.keep + b);
  *cap = __ldcg(p.cap + b);
  return *keep >= 0 && *cap >= *keep && *cap <= (long long)p.M * p.page;
}

// Chunk c of the counts: bit maps and the number of free pages; row c of the table: the pages it needs.
__device__ __forceinline__ void resize_count(const Group<1>& g, const PgResize& p, int c) {
  if (c == 0 && g.tid < 64) {
    p.w.count[g.tid] = 0;
    if (p.stats && g.tid < 4) p.stats[g.tid] = 0;
  }
  if (c < p.chunks) {
    int n = 0, refs[kPgChunkWords / kPgWarps];
    load_chunk(g, p.ref, p.P, c, refs);
#pragma unroll
    for (int k = 0; k < kPgChunkWords / kPgWarps; ++k) {
      const int i = g.warp() + k * kPgWarps, at = c * kPgChunk + 32 * i + g.lane(), r = refs[k];
      const uint32_t free = __ballot_sync(0xffffffffu, at < p.P && r <= 0), shared = __ballot_sync(0xffffffffu, r > 1);
      if (g.lane() == 0) {
        p.w.bits[c * kPgChunkWords + i] = free;
        p.w.bits[(p.chunks + c) * kPgChunkWords + i] = shared;
        n += __popc(free);
      }
      if (p.ref_out != p.ref && at < p.P) p.ref_out[at] = r;
    }
    n = g.sum(n);
    if (g.tid == 0) p.w.chunk_n[c] = n;
  }
  if (c < p.B) {
    int keep, cap, n = 0;
    bool wrong = false;
    if (row_bounds(p, c, &keep, &cap)) {
      for (int i0 = 0; i0 < p.M; i0 += kPgThreads * kPgDeep) {
        int pg[kPgDeep], r[kPgDeep];
#pragma unroll
        for (int k = 0; k < kPgDeep; ++k) {
          const int i = i0 + k * kPgThreads + g.tid;
          pg[k] = i < p.M ? __ldcg(p.table + (size_t)c * p.M + i) : -1;
        }
#pragma unroll
        for (int k = 0; k < kPgDeep; ++k) r[k] = pg[k] >= 0 && pg[k] < p.P ? __ldcg(p.ref + pg[k]) : 0;
#pragma unroll
        for (int k = 0; k < kPgDeep; ++k) {
          const int i = i0 + k * kPgThreads + g.tid;
          if (i >= p.M) continue;
          const bool held = pg[k] >= 0 && pg[k] < p.P;
          wrong = wrong || pg[k] < -1 || pg[k] >= p.P || (!held && i < (keep + p.page - 1) / p.page);
          wrong = wrong || (held && r[k] <= 0);  // held, and counted free
          n += entry_of(i, held, r[k] > 1, keep, cap, p.page).fresh;
        }
      }
    } else {
      wrong = true;
    }
    n = g.sum(n);
    wrong = __syncthreads_or(wrong);
    if (g.tid == 0) {
      p.w.need[c] = n;
      p.w.wrong[c] = wrong;
    }
  }
}

// Row b: its new pages' numbers, its entries, the counts.
__device__ __forceinline__ void resize_assign(const Group<1>& g, const PgResize& p, int b) {
  int first, unused;
  const int need = g.sum_upto(p.w.need, p.B, b, &first);
  const int mine = b < p.B ? __ldcg(p.w.need + b) : 0, wrong = b < p.B ? __ldcg(p.w.wrong + b) : 0;
  const int free = g.sum_upto(p.w.chunk_n, p.chunks, 0, &unused);
  if (b == 0 && g.tid == 0) {
    if (p.stats) p.stats[0] = need, p.stats[1] = free;
    if (need > free) set_error(p.err, kErrPages);
  }
  // the error word keeps the first code: that nothing changed must not hide behind what is wrong with one row
  if (wrong && need <= free && g.tid == 0) set_error(p.err, kErrDeviceIndex);
  if (b >= p.B) return;  // no rows at all
  int keep, cap;
  const bool ok = row_bounds(p, b, &keep, &cap) && need <= free;
  const int32_t* row = p.table + (size_t)b * p.M;
  int32_t* out = p.table_out + (size_t)b * p.M;
  if (!ok) {
    if (p.table_out != p.table)
      for (int i = g.tid; i < p.M; i += kPgThreads) out[i] = __ldcg(row + i);
    return;
  }
  int* fresh = p.w.list + first;  // the pages of ranks first .. first + mine - 1
  if (mine > 0) {
    int* before_s = g.sh->before;
    int below = 0;
    for (int c0 = 0; c0 < p.chunks && below < first + mine; c0 += kPgThreads) {
      const int c = c0 + g.tid;
      const int n = c < p.chunks ? __ldcg(p.w.chunk_n + c) : 0;
      int all;
      const int at = below + g.prefix(n, &all);
      before_s[g.tid] = at;
      const int skip = g.sum(c < p.chunks && at + n <= first);  // chunks that end before the row's first
      for (int k = skip; k < kPgThreads && c0 + k < p.chunks && before_s[k] < first + mine; ++k) {
        uint32_t word = g.tid < kPgChunkWords
                            ? __ldcg(p.w.bits + (size_t)(c0 + k) * kPgChunkWords + g.tid) : 0u;
        int in_chunk;
        int rank = before_s[k] + g.prefix(__popc(word), &in_chunk);
        while (word) {
          const int bit = __ffs(word) - 1;
          word &= word - 1;
          if (rank >= first && rank < first + mine) fresh[rank - first] = (c0 + k) * kPgChunk + 32 * g.tid + bit;
          ++rank;
        }
      }
      below += all;
      g.sync();
    }
    g.sync();
  }
  const uint32_t* shared = p.w.bits + (size_t)p.chunks * kPgChunkWords;
  auto& fresh_s = g.sh->fresh;
  const int lane = g.lane(), warp = g.warp();
  int given = 0, gone = 0;
  for (int i0 = 0; i0 < p.M; i0 += kPgThreads * kPgDeep) {
    int pg[kPgDeep];
    uint32_t bit[kPgDeep], ballot[kPgDeep];
    Entry e[kPgDeep];
#pragma unroll
    for (int k = 0; k < kPgDeep; ++k) {
      const int i = i0 + k * kPgThreads + g.tid;
      pg[k] = i < p.M ? __ldcg(row + i) : -1;
    }
#pragma unroll
    for (int k = 0; k < kPgDeep; ++k) bit[k] = pg[k] >= 0 && pg[k] < p.P ? __ldcg(shared + (pg[k] >> 5)) >> (pg[k] & 31) & 1u : 0u;
    g.sync();  // the last round's counts are read
#pragma unroll
    for (int k = 0; k < kPgDeep; ++k) {
      const int i = i0 + k * kPgThreads + g.tid;
      e[k] = entry_of(i, pg[k] >= 0 && pg[k] < p.P, bit[k], keep, cap, p.page);
      if (i >= p.M) e[k].fresh = e[k].gone = e[k].copied = false;
      ballot[k] = __ballot_sync(0xffffffffu, e[k].fresh);
      if (lane == 0) fresh_s[k][warp] = __popc(ballot[k]);
    }
    g.sync();
#pragma unroll
    for (int k = 0; k < kPgDeep; ++k) {
      const int i = i0 + k * kPgThreads + g.tid;
      int rank = given + __popc(ballot[k] & ((1u << lane) - 1u));
#pragma unroll
      for (int w = 0; w < kPgWarps; ++w) {
        if (w < warp) rank += fresh_s[k][w];
        given += fresh_s[k][w];
      }
      if (i >= p.M) continue;
      int to = e[k].held && !e[k].gone ? pg[k] : -1;
      if (e[k].fresh) {
        to = fresh[rank];
        atomicAdd(p.ref_out + to, 1);
        if (e[k].copied) {
          const int at = atomicAdd(p.w.count, 1);  // any order: the copies are apart
          p.w.src[at] = pg[k];
          p.w.list2[at] = to;
        }
      }
      if (e[k].gone) {
        atomicSub(p.ref_out + pg[k], 1);
        ++gone;
      }
      out[i] = to;
    }
  }
  if (p.stats) {
    gone = g.sum(gone);
    if (g.tid == 0 && gone) atomicAdd(p.stats + 3, gone);
  }
}

__global__ void __launch_bounds__(kPgThreads) resize_count_kernel(const PgResize p) {
  __shared__ PgShared sh;
  pdl_wait();
  pdl_trigger();
  resize_count(Group<1>(&sh), p, blockIdx.x);
}

__global__ void __launch_bounds__(kPgThreads) resize_assign_kernel(const PgResize p) {
  __shared__ PgShared sh;
  pdl_wait();
  pdl_trigger();
  resize_assign(Group<1>(&sh), p, blockIdx.x);
}

// A table of few entries over few pages: one CTA plans the whole turn in shared memory, entry k kPgSmall + t by thread t.
// (32 rows of 36, 16 copies of 0.96 MB: 11.0 us with the copies, 13.4 with the two launches above; called from the host
// 12.7 for 14.3.)
constexpr int kPgSmall = 1024;
constexpr int kPgSmallDeep = kPgChunk / kPgSmall;

__global__ void __launch_bounds__(kPgSmall) resize_small_kernel(const PgResize p) {
  __shared__ uint32_t free_s[kPgChunkWords], shared_s[kPgChunkWords];
  __shared__ int free_before[kPgChunkWords];           // free pages before each word's
  __shared__ int fresh_s[kPgSmallDeep * kPgSmall / 32];  // new pages of each warp's entries, then those before them
  __shared__ int list[kPgChunk];                       // the free pages that are given out, in rising order
  __shared__ int need_s, free_n, copies, gone_n;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, total = p.B * p.M;
  pdl_wait();
  pdl_trigger();
  int ref[kPgSmallDeep], pg[kPgSmallDeep], keep[kPgSmallDeep], cap[kPgSmallDeep], entry[kPgSmallDeep];
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const int at = k * kPgSmall + tid, row = at / p.M;
    ref[k] = at < p.P ? __ldcg(p.ref + at) : -1;
    pg[k] = at < total ? __ldcg(p.table + at) : -1;
    keep[k] = at < total ? __ldcg(p.keep + row) : 0;
    cap[k] = at < total ? __ldcg(p.cap + row) : 0;
    entry[k] = at - row * p.M;
  }
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const int at = k * kPgSmall + tid;
    const uint32_t free = __ballot_sync(0xffffffffu, at < p.P && ref[k] <= 0);
    const uint32_t shared = __ballot_sync(0xffffffffu, ref[k] > 1);
    if (lane == 0) {
      free_s[at >> 5] = free;
      shared_s[at >> 5] = shared;
    }
    if (p.ref_out != p.ref && at < p.P) p.ref_out[at] = ref[k];
  }
  if (tid == 0) copies = gone_n = 0;
  __syncthreads();
  Entry e[kPgSmallDeep];
  uint32_t ballot[kPgSmallDeep], stays = 0;  // bit k: the entry's row is out of range and stays as it is
  bool wrong = false;
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const bool in = k * kPgSmall + tid < total, held = pg[k] >= 0 && pg[k] < p.P;
    const bool ok = keep[k] >= 0 && cap[k] >= keep[k] && cap[k] <= (long long)p.M * p.page;
    e[k] = Entry{held, false, false, false};
    if (in && ok) {
      const bool is_free = held && (free_s[pg[k] >> 5] >> (pg[k] & 31) & 1u);
      if (pg[k] < -1 || pg[k] >= p.P || (!held && entry[k] < (keep[k] + p.page - 1) / p.page) || is_free)
        wrong = true;
      e[k] = entry_of(entry[k], held, held && (shared_s[pg[k] >> 5] >> (pg[k] & 31) & 1u), keep[k], cap[k], p.page);
    } else {
      stays |= 1u << k;
      wrong = wrong || in;
    }
    ballot[k] = __ballot_sync(0xffffffffu, e[k].fresh);
    if (lane == 0) fresh_s[k * (kPgSmall / 32) + warp] = __popc(ballot[k]);
  }
  __syncthreads();
  if (warp < 2) {  // prefixes of the 128 counts of new pages, and of free ones
    constexpr int kEach = kPgChunkWords / 32;
    int v[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      v[i] = warp == 0 ? fresh_s[lane * kEach + i] : __popc(free_s[lane * kEach + i]);
      sum += v[i];
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    int before = upto - sum;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      (warp == 0 ? fresh_s : free_before)[lane * kEach + i] = before;
      before += v[i];
    }
    if (lane == 31) (warp == 0 ? need_s : free_n) = upto;
  }
  __syncthreads();
  const int need = need_s;
  const bool enough = need <= free_n;
  if (wrong && enough) set_error(p.err, kErrDeviceIndex);
  if (enough && tid < kPgChunkWords) {
    int rank = free_before[tid];
    for (uint32_t word = free_s[tid]; word && rank < need; word &= word - 1) list[rank++] = 32 * tid + __ffs(word) - 1;
  }
  __syncthreads();
  int gone = 0;
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const int at = k * kPgSmall + tid;
    if (at >= total) continue;
    int to = pg[k];
    if (enough && !(stays >> k & 1u)) {
      to = e[k].held && !e[k].gone ? pg[k] : -1;
      if (e[k].fresh) {
        to = list[fresh_s[k * (kPgSmall / 32) + warp] + __popc(ballot[k] & ((1u << lane) - 1u))];
        atomicAdd(p.ref_out + to, 1);
        if (e[k].copied) {
          const int c = atomicAdd(&copies, 1);  // any order: the copies are apart
          p.w.src[c] = pg[k];
          p.w.list2[c] = to;
        }
      }
      if (e[k].gone) {
        atomicSub(p.ref_out + pg[k], 1);
        ++gone;
      }
    }
    p.table_out[at] = to;
  }
  if (gone) atomicAdd(&gone_n, gone);
  __syncthreads();
  if (tid == 0) {
    p.w.count[0] = copies;
    if (p.stats) p.stats[0] = need, p.stats[1] = free_n, p.stats[2] = copies, p.stats[3] = gone_n;
    if (!enough) set_error(p.err, kErrPages);
  }
}

struct PgCopy {
  uint8_t* pool;  // [layers, P, page_bytes]
  const int *src, *dst, *count;
  int layers, P;
  size_t page_bytes;
  int32_t* copied;  // optional: receives the number of pages
};

// Pieces of kPgCopyBytes of every listed page of every layer, dealt over the grid.
__device__ __forceinline__ void copy_pages(const PgCopy& p) {
  const long long pieces = (long long)((p.page_bytes + kPgCopyBytes - 1) / kPgCopyBytes);
  const long long n = __ldcg(p.count), units = n * p.layers * pieces;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long r = u / pieces, piece = u - r * pieces, k = r / p.layers, l = r - k * p.layers;
    const size_t off = (size_t)piece * kPgCopyBytes;
    const size_t bytes = p.page_bytes - off < kPgCopyBytes ? p.page_bytes - off : kPgCopyBytes;
    const uint4* s = reinterpret_cast<const uint4*>(p.pool + ((size_t)l * p.P + __ldcg(p.src + k)) * p.page_bytes + off);
    uint4* d = reinterpret_cast<uint4*>(p.pool + ((size_t)l * p.P + __ldcg(p.dst + k)) * p.page_bytes + off);
    constexpr int kU = kPgCopyBytes / 16 / kPgThreads;
    uint4 v[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const size_t at = threadIdx.x + i * kPgThreads;
      if (at * 16 < bytes) v[i] = s[at];
    }
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const size_t at = threadIdx.x + i * kPgThreads;
      if (at * 16 < bytes) d[at] = v[i];
    }
  }
}

__global__ void __launch_bounds__(kPgThreads) copy_pages_kernel(const PgCopy p) {
  pdl_wait();
  pdl_trigger();
  if (p.copied && blockIdx.x == 0 && threadIdx.x == 0) *p.copied = __ldcg(p.count);
  copy_pages(p);
}

// ----------------------------------------------------------------------------- fork
struct PgFork {
  const int32_t *table, *ref, *parent;
  int32_t *table_out, *ref_out;
  int B, M, P;
  int32_t* old;  // copy of the table where table_out is table
  int* err;
};

__device__ __forceinline__ void fork_save(const PgFork& p) {
  const size_t step = (size_t)gridDim.x * blockDim.x, at = (size_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (p.table_out == p.table)
    for (size_t i = at; i < (size_t)p.B * p.M; i += step) p.old[i] = __ldcg(p.table + i);
  if (p.ref_out != p.ref)
    for (size_t i = at; i < (size_t)p.P; i += step) p.ref_out[i] = __ldcg(p.ref + i);
}

// Row b: takes its parent's pages; the pages that it held get one count for each of its children, less its own.
template <int N>
__device__ __forceinline__ void fork_row(const Group<N>& g, const PgFork& p, int b) {
  int children = 0;
  for (int i = g.tid; i < p.B; i += kPgThreads) children += __ldcg(p.parent + i) == b;
  const int more = g.sum(children) - 1;
  const int from = __ldcg(p.parent + b);
  const bool has = from >= 0 && from < p.B;
  if ((from < -1 || from >= p.B) && g.tid == 0) set_error(p.err, kErrDeviceIndex);
  const int32_t* table = p.table_out == p.table ? p.old : p.table;
#pragma unroll 4
  for (int i = g.tid; i < p.M; i += kPgThreads) {
    const int mine = __ldcg(table + (size_t)b * p.M + i);
    if (mine >= 0 && mine < p.P) {
      if (more) atomicAdd(p.ref_out + mine, more);
    } else if (mine != -1) {
      set_error(p.err, kErrDeviceIndex);
    }
    p.table_out[(size_t)b * p.M + i] = has ? __ldcg(table + (size_t)from * p.M + i) : -1;
  }
}

__global__ void __launch_bounds__(kPgThreads) fork_save_kernel(const PgFork p) {
  pdl_wait();
  pdl_trigger();
  fork_save(p);
}

__global__ void __launch_bounds__(kPgThreads) fork_rows_kernel(const PgFork p) {
  __shared__ PgShared sh;
  pdl_wait();
  pdl_trigger();
  fork_row(Group<1>(&sh), p, blockIdx.x);
}

__global__ void __cluster_dims__(kPgCluster) __launch_bounds__(kPgGroups * kPgThreads) fork_plan_kernel(const PgFork p) {
  __shared__ PgShared sh[kPgGroups];
  pdl_wait();
  pdl_trigger();
  fork_save(p);
  cluster_sync();
  const Group<kPgGroups> g(sh);
  for (int b = blockIdx.x * kPgGroups + g.id; b < p.B; b += kPgCluster * kPgGroups) fork_row(g, p, b);
}

// ----------------------------------------------------------------------------- compact
struct PgCompact {
  const int32_t *table, *ref;
  int32_t *table_out, *ref_out, *map, *stats;
  int B, M, P, chunks;
  PgWs w;
  PgCopy copy;
  int* err;
};

// Chunk c of the counts: its bit map and the number of live pages.
__device__ __forceinline__ void compact_count(const Group<1>& g, const PgCompact& p, int c) {
  int n = 0, refs[kPgChunkWords / kPgWarps];
  load_chunk(g, p.ref, p.P, c, refs);
#pragma unroll
  for (int k = 0; k < kPgChunkWords / kPgWarps; ++k) {
    const int i = g.warp() + k * kPgWarps;
    const uint32_t live = __ballot_sync(0xffffffffu, refs[k] > 0);
    if (g.lane() == 0) {
      p.w.bits[c * kPgChunkWords + i] = live;
      n += __popc(live);
    }
  }
  n = g.sum(n);
  if (g.tid == 0) p.w.chunk_n[c] = n;
}

__global__ void __launch_bounds__(kPgThreads) compact_count_kernel(const PgCompact p) {
  __shared__ PgShared sh;
  pdl_wait();
  pdl_trigger();
  compact_count(Group<1>(&sh), p, blockIdx.x);
}

// Chunk c: the k-th free page below the live count goes to list2[k], the k-th live one at or above it to
// list[k].  Live pages below the count are as many as the count less the pages that move.
__global__ void __launch_bounds__(kPgThreads) compact_list_kernel(const PgCompact p) {
  __shared__ PgShared sh;
  pdl_wait();
  pdl_trigger();
  const Group<1> g(&sh);
  const int c = blockIdx.x;
  if (p.chunks == 1) {  // a pool of one chunk needs no launch before this one
    compact_count(g, p, 0);
    g.sync();
  }
  int before;
  const int live = g.sum_upto(p.w.chunk_n, p.chunks, c, &before);
  // live pages below number `live`
  int under, all;
  const int cl = live / kPgChunk;  // the chunk of that number (may lie behind the last page)
  g.sum_upto(p.w.chunk_n, p.chunks, cl, &under);
  if (cl < p.chunks) {
    const int word = g.tid, rest = live - cl * kPgChunk - 32 * word;  // pages of this word below the number
    uint32_t v = word < kPgChunkWords ? __ldcg(p.w.bits + cl * kPgChunkWords + word) : 0u;
    if (rest <= 0)
      v = 0u;
    else if (rest < 32)
      v &= (1u << rest) - 1u;
    under += g.sum(__popc(v));
  }
  uint32_t v = g.tid < kPgChunkWords ? __ldcg(p.w.bits + c * kPgChunkWords + g.tid) : 0u;
  int rank = before + g.prefix(__popc(v), &all);  // live pages before this word
  if (g.tid < kPgChunkWords) {
    const int at0 = c * kPgChunk + 32 * g.tid;
    for (int i = 0; i < 32 && at0 + i < p.P; ++i) {
      const bool is = (v >> i) & 1u;
      const bool moves = is && at0 + i >= live;
      if (moves) p.w.list[rank - under] = at0 + i;
      p.w.rank[at0 + i] = moves ? rank - under : -1;
      if (!is && at0 + i < live) p.w.list2[at0 + i - rank] = at0 + i;
      rank += is;
    }
  }
  if (c == 0 && g.tid == 0) {
    p.w.count[0] = live - under;
    p.w.count[1] = live;
    if (p.stats) {
      p.stats[0] = live;
      p.stats[1] = live - under;
      p.stats[2] = p.stats[3] = 0;
    }
  }
}

// New number of a live page: its own below the live count, else that of the free page of its rank; -1: not live.
__device__ __forceinline__ int compact_to(const PgCompact& p, int pg, int live) {
  if (pg < live) return (__ldcg(p.w.bits + (pg >> 5)) >> (pg & 31) & 1u) ? pg : -1;
  const int k = __ldcg(p.w.rank + pg);
  return k >= 0 ? __ldcg(p.w.list2 + k) : -1;
}

__global__ void __launch_bounds__(kPgThreads) compact_move_kernel(const PgCompact p) {
  pdl_wait();
  pdl_trigger();
  const int moves = __ldcg(p.w.count), live = __ldcg(p.w.count + 1);
  copy_pages(p.copy);
  const size_t step = (size_t)gridDim.x * kPgThreads, at = (size_t)blockIdx.x * kPgThreads + threadIdx.x;
  for (size_t i = at; i < (size_t)p.B * p.M; i += step) {
    const int pg = __ldcg(p.table + i);
    const bool in = pg >= 0 && pg < p.P;
    const int to = in ? compact_to(p, pg, live) : -1;
    if (pg != -1 && to < 0) set_error(p.err, kErrDeviceIndex);  // no page, or one that is counted free
    p.table_out[i] = to;
  }
  for (size_t i = at; i < (size_t)p.P; i += step) {
    const bool is = __ldcg(p.w.bits + (i >> 5)) >> (i & 31) & 1u;
    if (p.map) p.map[i] = compact_to(p, (int)i, live);
    // free pages below the live count get their count from the page that moves there
    if (p.ref_out != p.ref && is && (int)i < live) p.ref_out[i] = __ldcg(p.ref + i);
    if ((int)i >= live && !is) p.ref_out[i] = 0;
  }
  for (size_t k = at; k < (size_t)moves; k += step) {
    const int from = __ldcg(p.w.list + k), to = __ldcg(p.w.list2 + k);
    const int r = __ldcg(p.ref + from);
    p.ref_out[to] = r;
    p.ref_out[from] = 0;
  }
}

// A small pool: a cluster, each of whose CTAs plans all of it in shared memory and then does its share.  (300 pages of
// 8.7 KB: 5.8 us for 8.1 with the two launches above; called from one host 14.6 for 16, from others up to 20.)
constexpr long long kPgSmallBytes = 4 << 20;

__global__ void __cluster_dims__(kPgCluster) __launch_bounds__(kPgSmall) compact_small_kernel(const PgCompact p) {
  __shared__ uint32_t bits[kPgChunkWords];
  __shared__ int before[kPgChunkWords];             // live pages before each word's
  __shared__ uint16_t from[kPgChunk], free[kPgChunk];  // the pages that move, the numbers that they get
  __shared__ int16_t to[kPgChunk];                  // new number of a live page, -1
  __shared__ int refs[kPgChunk];
  __shared__ int live_s;
  const int tid = threadIdx.x, lane = tid & 31, c = blockIdx.x;
  pdl_wait();
  pdl_trigger();
  int ref[kPgSmallDeep], rank[kPgSmallDeep];
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const int at = k * kPgSmall + tid;
    ref[k] = at < p.P ? __ldcg(p.ref + at) : 0;
  }
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const int at = k * kPgSmall + tid;
    const uint32_t live = __ballot_sync(0xffffffffu, ref[k] > 0);
    if (lane == 0) bits[at >> 5] = live;
    refs[at] = ref[k];
  }
  __syncthreads();
  if (tid < 32) {
    constexpr int kEach = kPgChunkWords / 32;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sum += __popc(bits[lane * kEach + i]);
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    int b = upto - sum;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      before[lane * kEach + i] = b;
      b += __popc(bits[lane * kEach + i]);
    }
    if (lane == 31) live_s = upto;
  }
  __syncthreads();
  const int live = live_s;
  auto rank_of = [&](int at) { return before[at >> 5] + __popc(bits[at >> 5] & ((1u << (at & 31)) - 1u)); };
  const int under = live < kPgChunk ? rank_of(live) : live;  // live pages below number `live`
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const int at = k * kPgSmall + tid;
    rank[k] = rank_of(at);
    if (ref[k] > 0 && at >= live) from[rank[k] - under] = at;
    if (ref[k] <= 0 && at < live) free[at - rank[k]] = at;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const int at = k * kPgSmall + tid;
    to[at] = ref[k] <= 0 ? -1 : at < live ? at : free[rank[k] - under];
  }
  __syncthreads();
  cluster_sync();  // every CTA has read the counts
#pragma unroll
  for (int k = 0; k < kPgSmallDeep; ++k) {
    const int at = k * kPgSmall + tid;
    if (at >= p.P || (at >> 5) % kPgCluster != c) continue;
    p.ref_out[at] = at >= live ? 0 : ref[k] > 0 ? ref[k] : refs[from[at - rank[k]]];
    if (p.map) p.map[at] = to[at];
  }
  for (int i = c * kPgSmall + tid; i < p.B * p.M; i += kPgCluster * kPgSmall) {
    const int pg = __ldcg(p.table + i), n = pg >= 0 && pg < p.P ? to[pg] : -1;
    if (pg != -1 && n < 0) set_error(p.err, kErrDeviceIndex);  // no page, or one that is counted free
    p.table_out[i] = n;
  }
  if (c == 0 && tid == 0 && p.stats) {
    p.stats[0] = live;
    p.stats[1] = live - under;
    p.stats[2] = p.stats[3] = 0;
  }
  // vectors of every page that moves, in every layer, dealt over the cluster's threads
  const int vecs = (int)(p.copy.page_bytes / 16), per = vecs * p.copy.layers;
  const int all = (live - under) * per;
  for (int i0 = c * kPgSmall + tid; i0 < all; i0 += kPgDeep * kPgCluster * kPgSmall) {
    uint4 v[kPgDeep];
    uint4* dst[kPgDeep];
#pragma unroll
    for (int u = 0; u < kPgDeep; ++u) {
      const int i = i0 + u * kPgCluster * kPgSmall;
      if (i >= all) continue;
      const int k = i / per, l = (i - k * per) / vecs, at = i - k * per - l * vecs;
      uint4* pool = reinterpret_cast<uint4*>(p.copy.pool) + (size_t)l * p.P * vecs + at;
      v[u] = pool[(size_t)from[k] * vecs];
      dst[u] = pool + (size_t)free[k] * vecs;
    }
#pragma unroll
    for (int u = 0; u < kPgDeep; ++u)
      if (i0 + u * kPgCluster * kPgSmall < all) *dst[u] = v[u];
  }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

lsv_status pg_check(int32_t B, int32_t M, int32_t P) {
  if (B < 0 || M < 1 || P < 1) return LSV_ERR_INVALID_ARG;
  if (B > kPgMaxRows || P > kPgMaxPages || (long long)B * M >= (1ll << 31)) return LSV_ERR_UNSUPPORTED;
  return LSV_OK;
}

lsv_status pg_ws(void* ws, size_t bytes, int32_t B, int32_t M, int32_t P, PgWs* w) {
  *w = pg_layout(ws, B, M, P);
  if (!ws || bytes < w->total) return LSV_ERR_WORKSPACE;
  return al16(ws) ? LSV_OK : LSV_ERR_MISALIGNED;
}

lsv_status pool_check(int32_t layers, int64_t page_bytes, int32_t P) {
  if (layers < 1 || page_bytes < 1) return LSV_ERR_INVALID_ARG;
  if (page_bytes % 16 || page_bytes > (1ll << 31) || (double)layers * P * page_bytes > 9e18) return LSV_ERR_UNSUPPORTED;
  return LSV_OK;
}

}  // namespace
}  // namespace lsv

using namespace lsv;

extern "C" {

size_t spec_pages_workspace_size(int32_t B, int32_t M, int32_t P) {
  if (pg_check(B, M, P) != LSV_OK) return 0;
  return pg_layout(nullptr, B, M, P).total;
}

lsv_status spec_pages_resize(void* pool, int32_t layers, int64_t page_bytes, const int32_t* table, const int32_t* ref,
                             const int32_t* keep, const int32_t* cap, int32_t B, int32_t M, int32_t P, int32_t page,
                             int32_t* table_out, int32_t* ref_out, int32_t* stats_opt, void* ws, size_t ws_bytes,
                             lsv_stream stream) {
  lsv_status st = pg_check(B, M, P);
  if (st == LSV_OK) st = pool_check(layers, page_bytes, P);
  if (st != LSV_OK) return st;
  if (page < 1) return LSV_ERR_INVALID_ARG;
  if ((long long)M * page > (1ll << 30)) return LSV_ERR_UNSUPPORTED;
  if (!pool || !ref || !ref_out || (B > 0 && (!table || !keep || !cap || !table_out))) return LSV_ERR_INVALID_ARG;
  if (!al16(pool) || !al16(table) || !al16(ref) || !al16(keep) || !al16(cap) || !al16(table_out) || !al16(ref_out) ||
      !al16(stats_opt))
    return LSV_ERR_MISALIGNED;
  PgResize p;
  st = pg_ws(ws, ws_bytes, B, M, P, &p.w);
  if (st != LSV_OK) return st;
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  p.table = table;
  p.ref = ref;
  p.keep = keep;
  p.cap = cap;
  p.table_out = table_out;
  p.ref_out = ref_out;
  p.stats = stats_opt;
  p.B = B;
  p.M = M;
  p.P = P;
  p.page = page;
  p.chunks = (P + kPgChunk - 1) / kPgChunk;
  p.err = dc->err;
  PgCopy c;
  c.pool = static_cast<uint8_t*>(pool);
  c.src = p.w.src;
  c.dst = p.w.list2;
  c.count = p.w.count;
  c.layers = layers;
  c.P = P;
  c.page_bytes = (size_t)page_bytes;
  c.copied = stats_opt ? stats_opt + 2 : nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (B > 0 && (long long)B * M <= kPgChunk && P <= kPgChunk) {
    e = launch_pdl(resize_small_kernel, dim3(1), dim3(kPgSmall), 0, s, p);
  } else {
    e = launch_pdl(resize_count_kernel, dim3(B > p.chunks ? B : p.chunks), dim3(kPgThreads), 0, s, p);
    if (e == cudaSuccess) e = launch_pdl(resize_assign_kernel, dim3(B > 0 ? B : 1), dim3(kPgThreads), 0, s, p);
  }
  if (e == cudaSuccess && B > 0) e = launch_pdl(copy_pages_kernel, dim3(dc->num_sms * kPgCopyCtas), dim3(kPgThreads), 0, s, c);
  return e == cudaSuccess ? LSV_OK : LSV_ERR_CUDA;
}

lsv_status spec_pages_fork(const int32_t* table, const int32_t* ref, const int32_t* parent, int32_t B, int32_t M,
                           int32_t P, int32_t* table_out, int32_t* ref_out, void* ws, size_t ws_bytes,
                           lsv_stream stream) {
  lsv_status st = pg_check(B, M, P);
  if (st != LSV_OK) return st;
  if (!ref || !ref_out || (B > 0 && (!table || !parent || !table_out))) return LSV_ERR_INVALID_ARG;
  if (!al16(table) || !al16(ref) || !al16(parent) || !al16(table_out) || !al16(ref_out)) return LSV_ERR_MISALIGNED;
  PgWs w;
  st = pg_ws(ws, ws_bytes, B, M, P, &w);
  if (st != LSV_OK) return st;
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  PgFork p;
  p.table = table;
  p.ref = ref;
  p.parent = parent;
  p.table_out = table_out;
  p.ref_out = ref_out;
  p.B = B;
  p.M = M;
  p.P = P;
  p.old = w.table;
  p.err = dc->err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const bool save = table_out == table || ref_out != ref;
  if (save && B <= kPgFewRows && (long long)B * M <= kPgFewInts && P <= kPgFewInts) {
    e = launch_pdl(fork_plan_kernel, dim3(kPgCluster), dim3(kPgGroups * kPgThreads), 0, s, p);
  } else {
    if (save) e = launch_pdl(fork_save_kernel, dim3(dc->num_sms * 4), dim3(kPgThreads), 0, s, p);
    if (e == cudaSuccess && B > 0) e = launch_pdl(fork_rows_kernel, dim3(B), dim3(kPgThreads), 0, s, p);
  }
  return e == cudaSuccess ? LSV_OK : LSV_ERR_CUDA;
}

lsv_status spec_pages_compact(void* pool, int32_t layers, int64_t page_bytes, const int32_t* table, const int32_t* ref,
                              int32_t B, int32_t M, int32_t P, int32_t* table_out, int32_t* ref_out, int32_t* map_opt,
                              int32_t* stats_opt, void* ws, size_t ws_bytes, lsv_stream stream) {
  lsv_status st = pg_check(B, M, P);
  if (st == LSV_OK) st = pool_check(layers, page_bytes, P);
  if (st != LSV_OK) return st;
  if (!pool || !ref || !ref_out || (B > 0 && (!table || !table_out))) return LSV_ERR_INVALID_ARG;
  if (!al16(pool) || !al16(table) || !al16(ref) || !al16(table_out) || !al16(ref_out) || !al16(map_opt) ||
      !al16(stats_opt))
    return LSV_ERR_MISALIGNED;
  PgCompact p;
  st = pg_ws(ws, ws_bytes, B, M, P, &p.w);
  if (st != LSV_OK) return st;
  DeviceCtx* dc = nullptr;
  if (device_ctx(&dc) != cudaSuccess) return LSV_ERR_CUDA;
  p.table = table;
  p.ref = ref;
  p.table_out = table_out;
  p.ref_out = ref_out;
  p.map = map_opt;
  p.stats = stats_opt;
  p.B = B;
  p.M = M;
  p.P = P;
  p.chunks = (P + kPgChunk - 1) / kPgChunk;
  p.err = dc->err;
  p.copy.pool = static_cast<uint8_t*>(pool);
  p.copy.src = p.w.list;
  p.copy.dst = p.w.list2;
  p.copy.count = p.w.count;
  p.copy.layers = layers;
  p.copy.P = P;
  p.copy.page_bytes = (size_t)page_bytes;
  p.copy.copied = nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (P <= kPgChunk && (long long)B * M <= kPgFewInts && (double)layers * P * page_bytes <= (double)kPgSmallBytes) {
    e = launch_pdl(compact_small_kernel, dim3(kPgCluster), dim3(kPgSmall), 0, s, p);
    return e == cudaSuccess ? LSV_OK : LSV_ERR_CUDA;
  }
  if (p.chunks > 1) e = launch_pdl(compact_count_kernel, dim3(p.chunks), dim3(kPgThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(compact_list_kernel, dim3(p.chunks), dim3(kPgThreads), 0, s, p);
  if (e == cudaSuccess) e = launch_pdl(compact_move_kernel, dim3(dc->num_sms * kPgCopyCtas), dim3(kPgThreads), 0, s, p);
  return e == cudaSuccess ? LSV_OK : LSV_ERR_CUDA;
}

}  // extern "C"
