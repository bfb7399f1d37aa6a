// Which pages of the pools are in use, pages for the tokens to come, and moving pages together.
//
// A page is in use if a sequence's table lists it within the sequence's length, or if the caller holds it; nothing
// else is kept from call to call, so a sequence is freed by setting its length to 0, and no count can go wrong.
//
// One kernel works the tables out: it marks the pages, scans them in order and writes the new entries and the list of
// page copies. The marks are one word a page, the largest key of its users: tokens in the page, then the lower sequence.
// A warp takes a contiguous run of pages (or sequences), 32 at a time; ballots count them, and one look at all
// warps' counts tells each where its run starts. The free pages that are wanted become a list, from which each wanted
// entry takes its own. A second kernel copies the pages, over all pools at once, a warp for each 4 KiB.
//
// The tables are bound by latency, so the marks are in one SM's shared memory where they fit (kSmallPages): the table
// and the lengths are then the only trips to memory. After those it is instructions: one of all 32 warps is 8 clocks of
// the SM. So loops are not unrolled (8.0 to 6.5 us for 64 sequences), no warp has both the pages' and the sequences' part
// of a small problem, and the search for a wanted entry's sequence is by all threads, not by the warps whose
// pages are free (6.6 to 5.4). Up to kSmallEntries of the table one CTA does it all (16 sequences of 63 blocks in 1024
// pages compacted: 6.3 us with the copies); larger tables are read by a cluster of 8, each with marks of its own, which the first then gets the largest of (marking there
// from afar: 63 us for 36, 256 sequences of 255 blocks, 31.6 since). What does not fit is marked in the workspace, by the cluster, with
// a barrier between the phases: a page's mark is then a trip to the L2 for each pass over the marks, 32 of a warp at a time. 64
// sequences that grow by a token: 12.1 us in 20000 pages (10k entries in use, the cluster's shared memory), 19.4 in 100000 (50k), 41.8 in
// 350000 (175k); their compaction without pools 24.5, 33.9 and 92.2.
//
// The copies are bound by memory: 1066 MB of moves in 167 us, 0.93 of a plain copy's rate. Chunks of 2 and 8 KiB, and loads
// and stores that pass by the caches, are the same.
#include <cooperative_groups.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kWide = 8;                 // CTAs of the cluster
constexpr int kSmallPages = 28672;       // marks and holes of these fit in one SM's shared memory
constexpr int kSmallEntries = 8192;      // of the table, which one CTA reads
constexpr int kSmallBatch = 2048;
constexpr uint32_t kHeld = 0xffffffffu;
constexpr int kFewPools = 16;
constexpr int kChunk = 4096;             // bytes that a warp copies at a time

// (a table's capacity, and with it every position, fits 31 bits)
__device__ __forceinline__ int blocks_of(int tokens, int page) {
  return (int)(((uint32_t)tokens + (uint32_t)page - 1u) / (uint32_t)page);
}

// Sequence b's length as far as its pages go: a bad one uses all of its row (above the table) or none.
struct Seq {
  int len, want;
  bool bad;
};
__device__ __forceinline__ Seq seq_of(const PagesArgs& a, int len, int want) {
  const int cap = a.max_blocks * a.page_size;
  Seq s{min(max(len, 0), cap), want, len < 0 || len > cap || want > cap};
  if (s.bad || want < s.len) s.want = s.len;
  return s;
}
__device__ __forceinline__ Seq seq_of(const PagesArgs& a, int b) {
  return seq_of(a, __ldg(a.lens + b), a.new_lens ? __ldg(a.new_lens + b) : 0);
}

// The key of a user with so many tokens in the page and behind it.
__device__ __forceinline__ uint32_t key_of(int rest, int page, int b) {
  return (uint32_t)min(rest, page) << 16 | (uint32_t)(65535 - b);
}

// How the CTAs that work on one problem meet, and where they keep what they share.
enum Mode {
  kOne,     // one CTA, its shared memory
  kShared,  // a cluster that reads the table; the first CTA's shared memory, and its warps for what is not the table
  kSpread,  // a cluster; the workspace (past L1, which is an SM's own)
};
template <Mode M>
struct Team {
  static constexpr int kCtas = M == kOne ? 1 : kWide, kAll = kCtas * kThreads;
  static constexpr int kScanCtas = M == kSpread ? kWide : 1, kScanWarps = kScanCtas * kWarps;  // that work on pages and sequences
  uint32_t* key;     // [num_pages]
  uint32_t* own_key;  // kShared: the same of this CTA, else key
  int32_t* counts;   // [3][kScanWarps]
  int32_t* start;    // [batch]: of each sequence among the wanted pages
  uint32_t* from;    // [batch]: its first wanted entry, times 2, and whether that is a copy (all 32 bits: pages of one token)
  int32_t* hole;     // compaction: [num_pages / 2], free pages among the first ones
  int32_t* list;     // reservation, kSpread: the free pages that are wanted, in order
  uint16_t* small_list;  // the same, not kSpread (kSmallPages fit 16 bits; in hole's place)
  int32_t* middle;   // not kSpread: [batch], the page that each sequence is in the middle of
  int32_t* seq;      // not kSpread: [2][batch], this CTA's copy of the sequences' lengths and wanted lengths
  int32_t* moves;    // their number so far; not kSpread: in shared memory
  __device__ __forceinline__ int rank() const { return M == kOne ? 0 : blockIdx.x; }
  __device__ __forceinline__ int me() const { return rank() * kThreads + threadIdx.x; }
  __device__ __forceinline__ int warp() const { return me() >> 5; }
  __device__ __forceinline__ bool scans() const { return rank() < kScanCtas; }
  __device__ __forceinline__ void barrier_all() const {
    if constexpr (M == kOne)
      __syncthreads();
    else
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  __device__ __forceinline__ void barrier() const {  // of those that scan
    if constexpr (M == kSpread)
      barrier_all();
    else
      __syncthreads();
  }
  template <typename T>
  __device__ __forceinline__ T get(const T* p) const {
    if constexpr (M == kSpread)
      return __ldcg(p);
    else
      return *p;
  }
  // Run w [lo, hi) of n things, whole groups of 32; a warp's own run of pages is its own number's.
  __device__ __forceinline__ void run(int n, int w, int& lo, int& hi) const {
    const int per = ((n + 31) / 32 + kScanWarps - 1) / kScanWarps * 32;
    lo = (int)min((int64_t)n, (int64_t)w * per);
    hi = min(n, lo + per);
  }
  // The sum of list `l`'s counts of the runs before run w, and of all.
  __device__ __forceinline__ int before(int l, int w, int& total) const {
    int sum = 0, all = 0;
#pragma unroll 1
    for (int i = threadIdx.x & 31; i < kScanWarps; i += 32) {
      const int v = get(counts + l * kScanWarps + i);
      if (i < w) sum += v;
      all += v;
    }
    total = __reduce_add_sync(0xffffffffu, all);
    return __reduce_add_sync(0xffffffffu, sum);
  }
  __device__ __forceinline__ void set_count(int l, int w, int v) const {
    if ((threadIdx.x & 31) == 0) counts[l * kScanWarps + w] = v;
  }
};

template <Mode M>
__device__ __forceinline__ Team<M> team_of(const PagesArgs& a) {
  Team<M> t;
  if constexpr (M == kSpread) {
    t.counts = a.counts, t.start = a.start, t.from = a.from, t.key = a.key, t.hole = a.move_to;
    t.middle = t.seq = nullptr, t.moves = a.n_moves, t.list = a.list, t.small_list = nullptr;
  } else {
    extern __shared__ int32_t smem[];
    int32_t* at = smem;
    if constexpr (M == kShared) at = cooperative_groups::this_cluster().map_shared_rank(smem, 0);
    t.counts = at;
    t.moves = at + 3 * kWarps;
    t.start = t.moves + 1;
    t.from = reinterpret_cast<uint32_t*>(t.start + a.batch);
    t.middle = t.start + 2 * a.batch;
    t.seq = smem + (t.middle + a.batch - at);
    t.key = reinterpret_cast<uint32_t*>(t.middle + 3 * a.batch);
    t.hole = reinterpret_cast<int32_t*>(t.key + a.num_pages);
    t.list = nullptr, t.small_list = reinterpret_cast<uint16_t*>(t.hole);
    t.own_key = reinterpret_cast<uint32_t*>(smem) + (t.key - reinterpret_cast<uint32_t*>(at));
  }
  if constexpr (M != kShared) t.own_key = t.key;
  return t;
}

// A thread's entries of the table: (row, column), kAll entries further on each time, without a division.
template <Mode M>
struct Walk {
  int rows, columns, b, j;
  __device__ __forceinline__ Walk(const PagesArgs& a, const Team<M>& t)
      : rows(t.kAll / a.max_blocks), columns(t.kAll % a.max_blocks), b(t.me() / a.max_blocks), j(t.me() % a.max_blocks) {}
  __device__ __forceinline__ void next(const PagesArgs& a) {
    b += rows, j += columns;
    if (j >= a.max_blocks) j -= a.max_blocks, ++b;
  }
};

// Marks the pages and copies the table. key[p]: 0 free, kHeld, or the largest key of its users. Not
// kSpread: the sequences are noted, too.
template <Mode M>
__device__ __forceinline__ void mark(const PagesArgs& a, const Team<M>& t) {
  constexpr int U = M == kOne ? 1 : 4;  // entries of a thread in flight, and as many ahead
  const uint32_t entries = (uint32_t)a.batch * (uint32_t)a.max_blocks;  // (below 2^31)
  int p[U], ahead[U];
  auto load = [&](int (&to)[U], uint32_t i) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * t.kAll < entries) to[u] = a.table[i + u * t.kAll];
  };
  constexpr int kStep = M == kSpread ? t.kAll : kThreads, H = 4;  // (kShared: each CTA has marks of its own at first)
  uint8_t held[H];
  auto load_held = [&](int q) {
#pragma unroll
    for (int u = 0; u < H; ++u) held[u] = a.held && t.scans() && q + u * kStep < a.num_pages ? __ldg(a.held + q + u * kStep) : 0;
  };
  int q = M == kSpread ? t.me() : threadIdx.x;
  load(p, t.me());
  load_held(q);
  if constexpr (M != kSpread) {  // (each CTA for itself)
#pragma unroll 1
    for (int b = threadIdx.x; b < a.batch; b += kThreads) {
      const Seq s = seq_of(a, b);
      if (s.bad && t.rank() == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
      t.seq[b] = s.len, t.seq[a.batch + b] = s.want;
    }
  }
#pragma unroll 1
  while (q < a.num_pages) {
#pragma unroll
    for (int u = 0; u < H; ++u)
      if (q + u * kStep < a.num_pages) t.own_key[q + u * kStep] = held[u] ? kHeld : 0u;
    q += H * kStep;
    if (q < a.num_pages) load_held(q);
  }
  if (t.me() == 0) *t.moves = 0;
  Walk<M> at(a, t);
  t.barrier_all();
#pragma unroll 1
  for (uint32_t i0 = t.me(); i0 < entries; i0 += U * t.kAll) {
    load(ahead, i0 + U * t.kAll);
#pragma unroll
    for (int u = 0; u < U; ++u, at.next(a)) {
      const uint32_t i = i0 + u * t.kAll;
      if (i >= entries) break;
      int len;
      if constexpr (M == kSpread) {
        const Seq s = seq_of(a, at.b);
        if (s.bad && at.j == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
        len = s.len;
      } else {
        len = t.seq[at.b];
      }
      if (a.out_table != a.table) a.out_table[i] = p[u];
      const int rest = len - at.j * a.page_size;
      if (rest <= 0) continue;
      if (M != kSpread && rest < a.page_size) t.middle[at.b] = p[u];
      if ((uint32_t)p[u] >= (uint32_t)a.num_pages)
        set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
      else
        atomicMax(t.own_key + p[u], key_of(rest, a.page_size, at.b));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) p[u] = ahead[u];
  }
  t.barrier_all();
  if constexpr (M == kShared) {  // the largest of the CTAs' marks, to the first one's
#pragma unroll 1
    for (int q = t.me(); q < a.num_pages; q += t.kAll) {
      uint32_t k = 0;
#pragma unroll
      for (int c = 0; c < kWide; ++c) k = max(k, *cooperative_groups::this_cluster().map_shared_rank(t.own_key + q, c));
      t.key[q] = k;
    }
    t.barrier_all();
  }
}

// What sequence b asks for: entries [from, to) of its row; whether the first of them is the page that it is in the
// middle of, which others use too and is copied.
struct Want {
  int from, to;
  bool copy;
};
template <Mode M>
__device__ __forceinline__ Want want_of(const PagesArgs& a, const Team<M>& t, int b) {
  Seq s;
  if constexpr (M == kSpread)
    s = seq_of(a, b);
  else
    s = Seq{t.seq[b], t.seq[a.batch + b], false};
  Want w{0, 0, false};
  if (s.want <= s.len) return w;
  const int j = (int)((uint32_t)s.len / (uint32_t)a.page_size), rest = s.len - j * a.page_size;
  w.from = j + (rest > 0), w.to = blocks_of(s.want, a.page_size);
  if (rest > 0) {
    const int p = M == kSpread ? a.table[(int64_t)b * a.max_blocks + j] : t.middle[b];
    if (p >= 0 && p < a.num_pages && t.get(t.key + p) != key_of(rest, a.page_size, b)) w.copy = true, w.from = j;
  }
  return w;
}

template <Mode M>
__global__ void __launch_bounds__(kThreads, 1) reserve_kernel(const PagesArgs a) {
  wait_for_stream();
  let_next_start();
  const Team<M> t = team_of<M>(a);
  mark<M>(a, t);
  if (!t.scans()) return;
  // Pages from the first warp on, sequences from the last: where there are few, no warp has both.
  const int lane = threadIdx.x & 31, seq_run = t.kScanWarps - 1 - t.warp();
  int lo, hi, b_lo, b_hi;
  t.run(a.num_pages, t.warp(), lo, hi);
  t.run(a.batch, seq_run, b_lo, b_hi);
  int free = 0, wanted = 0;
#pragma unroll 1
  for (int p = lo + lane; p < hi; p += 32) free += t.get(t.key + p) == 0;
  t.set_count(0, t.warp(), __reduce_add_sync(0xffffffffu, free));
#pragma unroll 1
  for (int b0 = b_lo; b0 < b_hi; b0 += 32) {  // each sequence's start in its run, for now
    const int b = b0 + lane;
    Want w{0, 0, false};
    if (b < b_hi) w = want_of(a, t, b);
    int x = w.to - w.from;
    const int own = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    if (b < b_hi) t.start[b] = wanted + x - own, t.from[b] = 2u * (uint32_t)w.from + w.copy;
    wanted += __shfl_sync(0xffffffffu, x, 31);
  }
  t.set_count(1, seq_run, wanted);
  t.barrier();
  int n_free, n_want;
  int rank = t.before(0, t.warp(), n_free);
  const int want_before = t.before(1, seq_run, n_want);
#pragma unroll 1
  for (int b = b_lo + lane; b < b_hi; b += 32) t.start[b] += want_before;  // (its own lane's)
  if (t.me() == 0) {
    if (a.count) *a.count = n_free - n_want;
    if (n_want > n_free) set_err(a.err_flag, PKV_DEVERR_NO_PAGES);
  }
  if (n_want > n_free) {  // (the same for all)
    if (M != kSpread && t.me() == 0) *a.n_moves = 0;
    return;
  }
  // the r-th free page is the r-th wanted one
#pragma unroll 1
  for (int p0 = lo; p0 < hi && rank < n_want; p0 += 32) {
    const int p = p0 + lane;
    const bool is = p < hi && t.get(t.key + p) == 0;
    const unsigned mask = __ballot_sync(0xffffffffu, is);
    const int r = rank + __popc(mask & ((1u << lane) - 1u));
    rank += __popc(mask);
    if (!is || r >= n_want) continue;
    if constexpr (M == kSpread)
      t.list[r] = p;
    else
      t.small_list[r] = (uint16_t)p;
  }
  t.barrier();
#pragma unroll 1
  for (int r = t.me(); r < n_want; r += t.kScanCtas * kThreads) {
    int b = 0;  // the last sequence that starts at or before r
#pragma unroll 1
    for (int n = a.batch; n > 1;) {
      const int half = n / 2;
      if (t.get(t.start + b + half) <= r) b += half, n -= half;
      else n = half;
    }
    const int p = M == kSpread ? t.get(t.list + r) : t.small_list[r];
    const uint32_t from = t.get(t.from + b);
    const int i = r - t.get(t.start + b);
    const int64_t at = (int64_t)b * a.max_blocks + (from >> 1) + i;
    if (i == 0 && (from & 1)) {
      const int m = atomicAdd(t.moves, 1);
      a.move_from[m] = M == kSpread ? a.table[at] : t.middle[b], a.move_to[m] = p;
    }
    a.out_table[at] = p;
  }
  if constexpr (M != kSpread) {
    __syncthreads();
    if (threadIdx.x == 0) *a.n_moves = *t.moves;
  }
}

template <Mode M>
__global__ void __launch_bounds__(kThreads, 1) compact_kernel(const PagesArgs a) {
  wait_for_stream();
  let_next_start();
  const Team<M> t = team_of<M>(a);
  mark<M>(a, t);
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = 0, n_used = 0, n_late = 0;
  if (t.scans()) {
    t.run(a.num_pages, t.warp(), lo, hi);
    int used = 0, late = 0;
#pragma unroll 1
    for (int p = lo + lane; p < hi; p += 32) used += t.get(t.key + p) != 0;
    t.set_count(0, t.warp(), __reduce_add_sync(0xffffffffu, used));
    t.barrier();
    int before = t.before(0, t.warp(), n_used);
#pragma unroll 1
    for (int p = lo + lane; p < hi; p += 32) late += p >= n_used && t.get(t.key + p) != 0;
    t.set_count(1, t.warp(), __reduce_add_sync(0xffffffffu, late));
    t.barrier();
    t.before(1, t.warp(), n_late);
    if (t.me() == 0) {
      if (a.count) *a.count = n_used;
      *a.n_moves = n_late;
    }
#pragma unroll 1
    for (int p0 = lo; p0 < hi; p0 += 32) {
      const int p = p0 + lane;
      const bool is = p < hi && t.get(t.key + p) != 0;
      const unsigned mask = __ballot_sync(0xffffffffu, is);
      const int u = before + __popc(mask & ((1u << lane) - 1u));  // pages in use before p
      before += __popc(mask);
      if (p >= hi) continue;
      if (is && p >= n_used) a.move_from[u - (n_used - n_late)] = p;  // (so many of the first n_used pages are in use)
      if (!is && p < n_used) {
        t.hole[p - u] = p;
        if (M != kSpread) a.move_to[p - u] = p;
      }
      if (!is) a.page_map[p] = -1;
      t.key[p] = is ? (uint32_t)u + 1 : 0u;  // (its own lane's: read by no other until the barrier)
    }
  }
  t.barrier_all();
  if (M == kShared) t.before(0, 0, n_used), t.before(1, 0, n_late);
  // where page p in use goes
  auto goes = [&](int p) {
    if (p < n_used) return p;
    return (int)t.get(t.hole + (int)t.get(t.key + p) - 1 - (n_used - n_late));
  };
#pragma unroll 1
  for (int p = lo + lane; p < hi; p += 32)
    if (t.get(t.key + p) != 0) a.page_map[p] = goes(p);
  const uint32_t entries = (uint32_t)a.batch * (uint32_t)a.max_blocks;
  Walk<M> at(a, t);
#pragma unroll 1
  for (uint32_t i = t.me(); i < entries; i += t.kAll, at.next(a)) {
    if (at.j * a.page_size >= (M == kSpread ? seq_of(a, at.b).len : t.seq[at.b])) continue;
    const int p = a.table[i];
    if (p >= 0 && p < a.num_pages) a.out_table[i] = goes(p);
  }
  if (M == kShared) t.barrier_all();  // the first CTA's shared memory is read until here
}

// Pages move_from[m] to move_to[m], m < *n_moves, in every pool. No page is both.
template <int N>
__global__ void __launch_bounds__(256) copy_pages_kernel(const __grid_constant__ PoolsOf<N> pools, const int32_t* move_from,
                                                         const int32_t* move_to, const int32_t* n_moves, int most) {
  wait_for_stream();  // (the next kernel is not let in early: its CTAs would be placed where these leave room)
  const int lane = threadIdx.x & 31;
  int n = most;
  for (int64_t item = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 5; item < (int64_t)n * pools.chunks; item += (int64_t)gridDim.x * 8) {
    const int m = (int)(item / pools.chunks), c = (int)(item % pools.chunks);
    // (the lists have room for `most` moves: an entry is read together with their number, and used if it is one)
    const int from = __ldcg(move_from + m), to = __ldcg(move_to + m);
    n = __ldcg(n_moves);
    if (m >= n) break;
    int q = 0;
    for (int step = N / 2; step > 0; step >>= 1)  // the last pool that begins at or before chunk c
      if (q + step < pools.n && pools.pool[q + step].first_chunk <= c) q += step;
    const PagePool& pool = pools.pool[q];
    const int64_t at = (int64_t)(c - pool.first_chunk) * kChunk;
    const int64_t bytes = min((int64_t)kChunk, pool.page_bytes - at);
    const char* src = static_cast<const char*>(pool.base) + from * pool.page_bytes + at;
    char* dst = static_cast<char*>(pool.base) + to * pool.page_bytes + at;
    if (pool.wide) {
      uint4 v[kChunk / 512];
#pragma unroll
      for (int i = 0; i < kChunk / 512; ++i)
        if (512 * i + 16 * lane < bytes) v[i] = *reinterpret_cast<const uint4*>(src + 512 * i + 16 * lane);
#pragma unroll
      for (int i = 0; i < kChunk / 512; ++i)
        if (512 * i + 16 * lane < bytes) *reinterpret_cast<uint4*>(dst + 512 * i + 16 * lane) = v[i];
    } else {
      for (int64_t i = 4 * lane; i < bytes; i += 128)
        *reinterpret_cast<uint32_t*>(dst + i) = *reinterpret_cast<const uint32_t*>(src + i);
    }
  }
}

int launch_copies(const PagesArgs& a, const PagePools& pools, int most, cudaStream_t stream) {
  if (pools.n == 0 || most == 0) return PKV_OK;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  // How many pages there are to copy is known on the device; a warp that finds nothing to do ends. Four times the CTAs that
  // fit are better than one wave that goes on (169 and 178 us for 1029 MB).
  const int64_t warps = (int64_t)most * pools.chunks;
  const int64_t full = (int64_t)sms * 32, ctas = (warps + 7) / 8 < full ? (warps + 7) / 8 : full;
  auto launch = [&](auto* kernel, const auto& p) {
    return check_launch(launch_overlapped(kernel, dim3((unsigned)ctas), 256, 0, stream, 1, p, (const int32_t*)a.move_from,
                                          (const int32_t*)a.move_to, (const int32_t*)a.n_moves, most));
  };
  if (pools.n > kFewPools) return launch(copy_pages_kernel<PKV_MAX_POOLS>, pools);
  PoolsOf<kFewPools> few;  // (a launch copies its arguments: 6 KiB of them take the host 0.5 us, 4.4 us a call with 16 pools and 4.9 with 17)
  few.n = pools.n, few.chunks = pools.chunks;
  for (int i = 0; i < pools.n; ++i) few.pool[i] = pools.pool[i];
  return launch(copy_pages_kernel<kFewPools>, few);
}

int launch_tables(void (*one)(const PagesArgs), void (*shared)(const PagesArgs), void (*spread)(const PagesArgs),
                  FuncConfigured (&configured)[2], const PagesArgs& a, cudaStream_t stream) {
  if (a.num_pages > kSmallPages || a.batch > kSmallBatch)
    return check_launch(launch_overlapped(spread, dim3(kWide), kThreads, 0, stream, kWide, a));
  constexpr int kMost = 4 * (3 * kWarps + 5 * kSmallBatch + 1 + kSmallPages + kSmallPages / 2);
  static_assert(kMost <= 227 * 1024, "what one SM keeps");
  const bool is_one = (int64_t)a.batch * a.max_blocks <= kSmallEntries;
  if (!configured[is_one].ensure(reinterpret_cast<const void*>(is_one ? one : shared), kMost)) return PKV_ERR_LAUNCH;
  const size_t bytes = 4 * ((size_t)3 * kWarps + 5 * a.batch + 1 + a.num_pages + (a.num_pages + 1) / 2);
  return check_launch(is_one ? launch_overlapped(one, dim3(1), kThreads, bytes, stream, 1, a)
                             : launch_overlapped(shared, dim3(kWide), kThreads, bytes, stream, kWide, a));
}

}  // namespace

size_t pages_layout(PagesArgs* a, char* w, int batch, int num_pages) {
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t head = up(4 * (1 + 3 * kWide * kWarps)), pages = up((size_t)num_pages * 4), seqs = up((size_t)(batch + 1) * 4);
  const size_t moves = pages > seqs ? pages : seqs;  // (a reservation's copies are one a sequence at most)
  if (a) {
    a->n_moves = reinterpret_cast<int32_t*>(w);
    a->counts = a->n_moves + 1;
    a->key = reinterpret_cast<uint32_t*>(w + head);
    a->move_from = reinterpret_cast<int32_t*>(w + head + pages);
    a->move_to = reinterpret_cast<int32_t*>(w + head + pages + moves);
    a->start = reinterpret_cast<int32_t*>(w + head + pages + 2 * moves);
    a->from = reinterpret_cast<uint32_t*>(w + head + pages + 2 * moves + seqs);
    a->list = reinterpret_cast<int32_t*>(w + head + pages + 2 * moves + 2 * seqs);
  }
  return head + 2 * pages + 2 * moves + 2 * seqs;
}

int page_chunks(int64_t page_bytes) { return (int)((page_bytes + kChunk - 1) / kChunk); }

int launch_reserve(const PagesArgs& a, const PagePools& pools, cudaStream_t stream) {
  static FuncConfigured configured[2];
  const int rc = launch_tables(reserve_kernel<kOne>, reserve_kernel<kShared>, reserve_kernel<kSpread>, configured, a, stream);
  return rc != PKV_OK ? rc : launch_copies(a, pools, a.batch, stream);
}

int launch_compact(const PagesArgs& a, const PagePools& pools, cudaStream_t stream) {
  static FuncConfigured configured[2];
  const int rc = launch_tables(compact_kernel<kOne>, compact_kernel<kShared>, compact_kernel<kSpread>, configured, a, stream);
  return rc != PKV_OK ? rc : launch_copies(a, pools, a.num_pages / 2, stream);
}

}  // namespace pkv
