// Attention weight that the keys of a paged cache receive from the queries of a chunk, given
// the log-sum-exps of those queries (as the chunked prefill returns them):
//   sums_out[b, g, t] = decay * sums_in[b, g, t] + sum over queries i >= t - prefix and heads h
//                       of group g of exp(scale q_ih . k_t - lse_ih)
//
// With the lse known there is no softmax to run, only a product and a sum over its rows:
//   S^T [256 keys x 128 columns] = K [256 keys x 128 dims] . Q^T,  a column is a (query, head)
// on the tcgen05 tensor cores, keys as the 128-row operand (two tiles of 8 pages each). A
// thread owns one key, i.e. one TMEM lane, so a key's sum over the columns never leaves its
// thread: no reduction across threads, and a fixed order of additions.
//
// Bound: issue slots. A 256 x 128 step is 32768 exponentials, 1024 clocks of an SM's special-function
// units at 32 a clock, 8.4 MFLOP, about as long on the tensor cores, and three more instructions an
// exponential for the issue slots. A prompt chunk of 2048 queries over 2 x 3-4k keys, 32 heads on 8, takes
// 85.5 us (1.0 PFLOP/s); of the clocks in which an SM works, 68 % issue, 52 % have the
// special-function and 52 % the tensor pipe busy, and the SMs work 80 % of the time: about 230
// unequal items do not divide by 152. Tried and not kept: a share of the exponentials as
// polynomials on the FMA units (12 % slower for each eighth: the issue slots are not free), eight
// exponential warps for sixteen (14 % slower), one warp issuing the products of both tiles (the tensor
// cores idle while it waits), two-wide fp32 arithmetic, tensor memory read in double-buffered
// halves (10 % slower: spills), pages loaded by two warps (no gain).
// With a window of few queries an item is a single step, and what bounds it is the chain of
// barriers, loads and address arithmetic around the step, about 1.8 us of a CTA an item (32 queries
// over 4 x 5k keys: 13.7 us, 3.5 TB/s).
//
// A persistent CTA per SM takes items (sequence, KV head, 256 keys) in an order that pairs long and
// short ones: key tiles slowest (early keys are seen by the most queries), and every other round
// of the CTAs backwards (135 to 108 us against a plain stride). All its threads work its list of
// items out at the start, for every warp to read (16.3 to 13.7 us for the window: each warp working
// them out by itself took longer than its step). Few or uneven items are shared, each by a cluster
// of 2 to 8 CTAs (choose_split), whose partial sums are added in rank order through distributed
// shared memory.
// Warps: 0 and 2 TMA producers (a ring of four K tiles, page by page, and one of two Q tiles), 1
// and 3 MMA issuers of the two key tiles, 4..11 and 12..19 their exponentials and sums. S^T is
// double-buffered per tile: all 512 TMEM columns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "tcgen05.cuh"

namespace pkv {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // prefill.cu

namespace {

constexpr int CD = 128;                // head dim
constexpr int CK = 256;                // keys per item: two 128-row tiles
constexpr int CN = 128;                // columns (queries x heads of the group) per step
// One K stage, 32 KiB: 8-row groups of 2 KiB, each its two 64-dim halves of [8 rows][128 bytes], so
// that a page (16 rows of 256 bytes, contiguous in the pool) is one box and the groups of all pages
// lie at one distance.
constexpr int KSTG = 128 * CD * 2;
constexpr int QSTG = CN * CD * 2;      // one Q stage, 32 KiB: two 64-dim halves
constexpr int HALF = 128 * 128;        // [128 rows][128 bytes]
constexpr int NKS = 4, NQS = 2;
// An item takes two K stages in turn, one for each issuer. A wait by parity cannot tell a phase from the
// one two before, so whoever waits on a barrier has to see all of its phases: with an even number a
// stage is always the same issuer's.
static_assert(NKS % 2 == 0, "a K stage belongs to one issuer");
constexpr int CTHREADS = 640;
// barriers
constexpr int C_KF = 0, C_KE = C_KF + NKS, C_QF = C_KE + NKS, C_QE = C_QF + NQS, C_SF = C_QE + NQS, C_SE = C_SF + 4,
              C_DR = C_SE + 4, C_HF = C_DR + 1, C_NBAR = C_HF + 8 * 3;
constexpr int CITEMS = 256;            // items of a CTA
constexpr int CWARPS = 16;             // exponential warps, four .. nineteen
constexpr int SM_K = 0, SM_Q = SM_K + NKS * KSTG, SM_L = SM_Q + NQS * QSTG, SM_X = SM_L + CWARPS * CN * 4,
              SM_ITEM = SM_X + 4 * CK * 4, SM_BAR = SM_ITEM + CITEMS * 64, SM_MISC = SM_BAR + C_NBAR * 8,
              C_SMEM = SM_MISC + 16 + 1024;
static_assert(C_SMEM <= 232448, "shared memory per CTA");
constexpr float kL2e = 1.4426950408889634f;

struct CMisc {
  uint32_t tmem_base;
  int abort_;
};

// One item, 256 keys and the queries that see any of them, in the form in which it is used.
struct alignas(16) Item {
  int64_t sums_at, table_at, lse_at;  // of its first key's sum, its first page's entry, its first query's lse
  int steps;    // of columns; 0: none (the sums only decay), -1: nothing to do
  int keys;     // up to the end of the sequence (256 or more: all)
  int queries;  // that count and see a key of the item
  int diag;     // key t of the item is seen from query t + diag of them on
  int b, hk, query0;
};
static_assert(sizeof(Item) == 64, "item list");

__device__ __forceinline__ Item make_item(const ChunkWeightsArgs& a, int index, int qpt_log2) {
  const int rows = a.batch * a.n_kv_heads, row = index % rows, key0 = index / rows * CK;
  Item it{};
  it.b = row / a.n_kv_heads;
  it.hk = row % a.n_kv_heads;
  it.steps = -1;
  const int64_t prefix = __ldg(a.prefix_lens + it.b);
  const int64_t n = a.chunk_lens ? __ldg(a.chunk_lens + it.b) : a.chunk_len;
  if (prefix < 0 || n < 0 || n > a.chunk_len || prefix + n > (int64_t)a.max_blocks * a.page_size) {
    if (it.hk == 0 && key0 == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
    return it;
  }
  it.keys = (int)(prefix + n) - key0;
  if (it.keys <= 0) return it;
  const int first = a.window > 0 && a.window < n ? (int)n - a.window : 0;
  it.query0 = max(first, key0 - (int)prefix);
  it.queries = max(0, (int)n - it.query0);
  it.diag = key0 - (int)prefix - it.query0;
  it.steps = (it.queries + (1 << qpt_log2) - 1) >> qpt_log2;
  it.sums_at = (int64_t)row * (a.max_blocks * a.page_size) + key0;
  it.table_at = (int64_t)it.b * a.max_blocks + key0 / 16;
  it.lse_at = (int64_t)row * (a.n_qo_heads / a.n_kv_heads) * a.chunk_len + it.query0;
  return it;
}

// acc += exp2(s * c + nl) over 32 columns; MASKED: columns outside [lo, hi) do not count.
template <bool MASKED>
__device__ __forceinline__ void add_columns(const uint32_t (&s)[32], const float* nl, float c, int col0, int lo, int hi,
                                            float (&acc)[4]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 n4 = *reinterpret_cast<const float4*>(nl + i);
    const float n[4] = {n4.x, n4.y, n4.z, n4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float e = ex2(fmaf(__uint_as_float(s[i + k]), c, n[k]));
      if (MASKED) e = col0 + i + k >= lo && col0 + i + k < hi ? e : 0.0f;
      acc[k] += e;
    }
  }
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// SPLIT: the grid is one cluster per item; CTA r of a cluster of S takes steps r, r + S, ...
template <bool SPLIT>
__global__ void __launch_bounds__(CTHREADS, 1)
chunk_weights_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const ChunkWeightsArgs a, int n_items, int s_log2) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  unsigned char* smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  CMisc* misc = reinterpret_cast<CMisc*>(smem + SM_MISC);
  auto bar = [&](int i) { return sb + SM_BAR + 8 * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_qo_heads / a.n_kv_heads;  // a power of two
  const int g_log2 = 31 - __clz(G), qpt_log2 = 7 - g_log2, qpt = 1 << qpt_log2;  // queries per step
  static_assert(CN == 128, "qpt_log2");
  const int S = SPLIT ? 1 << s_log2 : 1;
  const int rank = SPLIT ? (int)cluster_rank() : 0;  // steps rank, rank + S, ... of the CTA's items
  const int cta = SPLIT ? (int)blockIdx.x >> s_log2 : (int)blockIdx.x;
  const int ctas = SPLIT ? (int)gridDim.x >> s_log2 : (int)gridDim.x;
  // steps of an item that this CTA takes
  auto share_of = [&](int steps) { return SPLIT ? (steps > rank ? (steps - rank + S - 1) >> s_log2 : 0) : steps; };

  // The CTA's items, worked out by all threads at once, so that the warps below only read them. CTA i
  // of P takes i, 2P - 1 - i, 2P + i, ...
  Item* items = reinterpret_cast<Item*>(smem + SM_ITEM);
  const int round = 2 * ctas, back = round - 1 - cta;
  const int count = n_items / round * 2 + (cta < n_items % round) + (back < n_items % round);
  wait_for_stream();
  for (int j = threadIdx.x; j < count; j += CTHREADS)
    items[j] = make_item(a, (j >> 1) * round + (j & 1 ? back : cta), qpt_log2);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C_NBAR; ++i) {
      int cnt = 1;
      if (i >= C_SE && i < C_SE + 4) cnt = 4;  // the four warps that read the buffer
      if ((i >= C_QE && i < C_QE + NQS) || i == C_DR) cnt = 2;  // both issuers
      mbar_init(bar(i), cnt);
    }
    misc->abort_ = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&misc->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem_base;
  volatile int* aborted = &misc->abort_;
  auto give_up = [&]() {
    if (lane == 0) {
      *aborted = 1;
      set_err(a.err_flag, PKV_DEVERR_TIMEOUT);
    }
  };

  // One key of an item: where its sum is, the old sum and its table entry (neither is looked at
  // before the end of the item, when the loads are long done).
  struct Mine {
    int64_t at;
    float before;
    int page;
    bool live;
  };
  auto my_key = [&](const Item& it, int t) {
    Mine m{};
    m.live = t < it.keys;
    if (m.live) {
      m.at = it.sums_at + t;
      m.before = a.sums_in[m.at];
      m.page = __ldg(a.block_table + it.table_at + t / 16);
    }
    return m;
  };
  auto store = [&](const Mine& m, float total) {
    const bool bad = m.page < 0 || m.page >= a.num_pages;
    if (bad) set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
    a.sums_out[m.at] = bad ? NAN : fmaf(a.decay, m.before, total);
  };

  // Registers: 96 a thread at launch; the first warpgroup gives 32 each to the four with the
  // exponentials, 8 more each there (every warp of a warpgroup takes the same setmaxnreg).
  static_assert(128 * 64 + 512 * 104 <= CTHREADS * 96, "register split");
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
    if (warp == 0) {
      // ------------------------------------------------------------------ TMA producer of K tiles
      if (elect_one()) tma_prefetch_desc(&mk);
      __syncwarp();
      uint32_t kc = 0;
      bool ok = true;
      // lane p < 16 holds the table entry of page p of the item; slots past the sequence bring its
      // first page again (their keys are not written), a bad entry page 0 (its keys become NaN).
      // The next item's entries are asked for before this item's copies wait for room.
      auto entry = [&](const Item& it) {
        return lane < 16 && it.steps > 0 ? __ldg(a.block_table + it.table_at + (16 * lane < it.keys ? lane : 0)) : 0;
      };
      Item next{};
      int next_phys = 0;
      if (count > 0) {
        next = items[0];
        next_phys = entry(next);
      }
      for (int j = 0; ok && j < count; ++j) {
        const Item it = next;
        int phys = next_phys;
        if (j + 1 < count) {
          next = items[j + 1];
          next_phys = entry(next);
        }
        if (it.steps <= 0) continue;
        if (__any_sync(0xffffffffu, *aborted)) {
          ok = false;
          break;
        }
        if (phys < 0 || phys >= a.num_pages) phys = 0;
        for (int tile = 0; ok && tile < 2; ++tile, ++kc) {  // lanes 8 tile .. 8 tile + 7 hold its pages
          const uint32_t ks = kc % NKS;
          if (kc >= NKS && !warp_wait(bar(C_KE + ks), (kc / NKS - 1) & 1)) ok = false;
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(C_KF + ks), KSTG);
          __syncwarp();
          if ((lane >> 3) == tile)
            tma_load_4d(sb + SM_K + ks * KSTG + (lane & 7) * 4096, &mk, 0, 0, 0, (phys * a.n_kv_heads + it.hk) * 2,
                        bar(C_KF + ks));
          __syncwarp();
        }
      }
      if (!ok) give_up();
      // every issued copy lands before the shared memory is released
      bool drained = true;
      for (uint32_t s = 0; s < NKS && s < kc; ++s) drained &= warp_wait(bar(C_KF + s), ((kc - 1 - s) / NKS) & 1);
      if (!drained) give_up();
    } else if (warp == 2) {
      // ------------------------------------------------------------------ TMA producer of Q tiles
      if (elect_one()) tma_prefetch_desc(&mq);
      __syncwarp();
      uint32_t qc = 0;
      bool ok = true;
      for (int j = 0; ok && j < count; ++j) {
        const Item it = items[j];
        if (__any_sync(0xffffffffu, *aborted)) ok = false;
        for (int s = rank; ok && s < it.steps; s += S, ++qc) {
          const uint32_t qs = qc % NQS;
          if (qc >= NQS && !warp_wait(bar(C_QE + qs), (qc / NQS - 1) & 1)) ok = false;
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(bar(C_QF + qs), QSTG);
            const uint32_t dst = sb + SM_Q + qs * QSTG;
            tma_load_4d(dst, &mq, 0, it.hk * G, it.query0 + s * qpt, it.b, bar(C_QF + qs));
            tma_load_4d(dst + HALF, &mq, 64, it.hk * G, it.query0 + s * qpt, it.b, bar(C_QF + qs));
          }
          __syncwarp();
        }
      }
      if (!ok) give_up();
      bool drained = true;
      for (uint32_t s = 0; s < NQS && s < qc; ++s) drained &= warp_wait(bar(C_QF + s), ((qc - 1 - s) / NQS) & 1);
      if (!drained) give_up();
    } else if (warp == 1 || warp == 3) {
      // ------------------------------------------------------------------ MMA issuers
      // One warp per key tile: while one waits for its barriers, the other's products run.
      const int tile = warp >> 1;
      const uint32_t idesc = idesc_bf16_f32(128, CN, false, false);
      const uint64_t dk0 = smem_desc(sb + SM_K, 16, 2048, kSwizzle128B);
      const uint64_t dq0 = smem_desc(sb + SM_Q, 16, 1024, kSwizzle128B);
      uint32_t kt = tile, qc = 0;  // this tile's place in the K ring, steps so far
      bool ok = true;
      for (int j = 0; ok && j < count; ++j) {
        const Item it = items[j];
        if (it.steps <= 0) continue;
        const uint32_t ks = kt % NKS;
        const uint64_t dk = dk0 + (uint64_t)((ks * KSTG) >> 4);
        for (int s = rank; ok && s < it.steps; s += S, ++qc) {
          const uint32_t qs = qc % NQS, buf = qc & 1;
          if (s == rank && !warp_wait(bar(C_KF + ks), (kt / NKS) & 1)) ok = false;
          if (ok && !warp_wait(bar(C_QF + qs), (qc / NQS) & 1)) ok = false;
          if (ok && qc >= 2 && !warp_wait(bar(C_SE + 2 * tile + buf), (qc / 2 - 1) & 1)) ok = false;
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dq = dq0 + (uint64_t)((qs * QSTG) >> 4);
  #pragma unroll
            for (int kk = 0; kk < CD / 16; ++kk)
              mma_bf16_ss(tmem + (2 * tile + buf) * CN, dk + (uint64_t)(((kk / 4) * 1024 + (kk % 4) * 32) >> 4),
                          dq + (uint64_t)(((kk / 4) * HALF + (kk % 4) * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
            mma_commit(bar(C_SF + 2 * tile + buf));
            mma_commit(bar(C_QE + qs));
            if (s + S >= it.steps) mma_commit(bar(C_KE + ks));
          }
          __syncwarp();
        }
        kt += 2;
      }
      if (!ok) give_up();
      // every issued product finishes before TMEM is freed
      if (elect_one()) mma_commit(bar(C_DR));
      __syncwarp();
      if (!warp_wait(bar(C_DR), 0)) give_up();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;" ::: "memory");
    // ------------------------------------------------------------------ exponentials and sums
    // Eight warps per key tile, two for each quarter of its TMEM lanes: `half` 0 takes the even
    // steps (S buffer 0), 1 the odd ones, so each buffer goes between the products and its own
    // warps. An item of one step is finished by the warps that take it; of more, by half 0, to
    // which half 1 hands its sums (three slots: a step of an item in between stands before each reuse).
    const int tile = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, wq = warp & 3;
    const int hand_bar = C_HF + (tile * 4 + wq) * 3;
    float* handed = reinterpret_cast<float*>(smem + SM_X);  // [3][CK]
    uint32_t n_hand = 0;
    const int t = tile * 128 + wq * 32 + lane;  // key within the item
    const uint32_t lane_addr = (uint32_t)(wq * 32) << 16;
    const float c = a.scale * kL2e;
    // The lane's four columns of a step, whose log-sum-exps it brings to the warp's own corner of
    // shared memory for all lanes to read; they are asked for one step ahead.
    constexpr int LC = CN / 32;
    float* nl = reinterpret_cast<float*>(smem + SM_L) + (warp - 4) * CN;
    const uint32_t src = tmem + lane_addr + (2 * tile + half) * CN;
    auto lse_of = [&](const Item& it, int s, float (&v)[LC]) {
      if (s >= it.steps) return;
      const float* first = a.lse + it.lse_at + (s << qpt_log2);
      const int left = it.queries - (s << qpt_log2);
#pragma unroll
      for (int k = 0; k < LC; ++k) {
        const int col = 32 * k + lane, query = col >> g_log2;
        v[k] = query < left ? __ldg(first + (int64_t)(col & (G - 1)) * a.chunk_len + query) : 0.0f;
      }
    };
    // look() goes on to the next item that these warps have a part in, and asks for its old sums,
    // table entries and first log-sum-exps, before the steps of the one at hand.
    int at = 0;
    Item it{};
    int steps = 0;         // steps of the item that are this CTA's
    uint32_t next_qc = 0;  // steps before it
    bool more = true, finish = false;
    Mine mine{};
    float ahead[LC] = {};
    auto look = [&]() {
      for (;; ++at) {
        next_qc += steps;
        steps = 0;
        more = at < count;
        if (!more) return;
        it = items[at];
        if (it.steps < 0) continue;
        steps = share_of(it.steps);
        if (steps != 1 || half == (int)(next_qc & 1)) break;
      }
      ++at;
      finish = steps == 1 || half == 0;
      if (finish) mine = my_key(it, t);
      lse_of(it, rank + (int)((half ^ next_qc) & 1) * S, ahead);
    };
    bool ok = true;
    look();
    while (more) {
      const Item now = it;
      const Mine my = mine;
      const int n_steps = steps;
      const uint32_t qc = next_qc;
      const bool fin = finish;
      float v[LC];
#pragma unroll
      for (int k = 0; k < LC; ++k) v[k] = ahead[k];
      look();
      float total = 0.0f;
      const int mine_first = (int)((half ^ qc) & 1);  // of the item's steps, this half takes every other one
      for (int k0 = mine_first; ok && k0 < n_steps; k0 += 2) {
        const int s = rank + k0 * S;
#pragma unroll
        for (int k = 0; k < LC; ++k) nl[32 * k + lane] = -kL2e * v[k];
        __syncwarp();
        lse_of(now, s + 2 * S, v);
        ok = warp_wait(bar(C_SF + 2 * tile + half), ((qc + k0) / 2) & 1);
        if (!ok) break;
        tc_fence_after();
        // columns [lo, hi) count: the causal bound and the end of the chunk
        const int lo = max(now.diag + t - s * qpt, 0) * G, hi = min(qpt, now.queries - s * qpt) * G;
        const bool whole = __all_sync(0xffffffffu, lo == 0) && hi == CN;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < CN / 32; ++k) {
          uint32_t r[32];
          tmem_ld32(src + 32 * k, r);
          tmem_ld_wait();
          if (k == CN / 32 - 1) {  // the buffer is read: the next products may start
            tc_fence_before();
            __syncwarp();
            if (elect_one()) mbar_arrive(bar(C_SE + 2 * tile + half));
            __syncwarp();
          }
          if (whole)
            add_columns<false>(r, nl + 32 * k, c, 32 * k, lo, hi, acc);
          else
            add_columns<true>(r, nl + 32 * k, c, 32 * k, lo, hi, acc);
        }
        __syncwarp();  // every lane has read nl
        // a step's columns are added up on their own first: shorter chains of roundings
        total += (acc[0] + acc[1]) + (acc[2] + acc[3]);
      }
      if (!ok) total = NAN;
      if (n_steps > 1) {
        float* hand = handed + n_hand % 3 * CK + t;
        const uint32_t full = bar(hand_bar + n_hand % 3);
        if (half == 1) {
          *hand = total;
          __syncwarp();
          if (elect_one()) mbar_arrive(full);
          __syncwarp();
        } else {
          if (!warp_wait(full, n_hand / 3 & 1)) ok = false;
          total = ok ? total + *hand : NAN;
        }
        ++n_hand;
      }
      if (!fin) continue;
      if constexpr (SPLIT) {
        reinterpret_cast<float*>(smem + SM_X)[3 * CK + t] = total;
      } else if (my.live) {
        store(my, total);
      }
    }
    if (!ok) give_up();
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (SPLIT) {
    // the cluster's partial sums of the item, added in rank order; every thread of every CTA takes
    // both cluster barriers
    const float* parts = reinterpret_cast<const float*>(smem + SM_X) + 3 * CK;
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int share = CK / S, t = rank * share + (int)threadIdx.x;
    if ((int)threadIdx.x < share) {
      const Item it = items[0];
      const Mine my = my_key(it, t);
      if (it.steps >= 0 && my.live) {
        float total = 0.0f;
        for (int r = 0; r < S; ++r) {
          uint32_t addr;
          float x;
          asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(parts + t)), "r"(r));
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
          total += x;
        }
        store(my, total);
      }
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool encode(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// log2 of the CTAs that share an item, from a chunk that fills the table. Estimated in 10 ns: a step takes
// 100, a CTA's start 700, the next item of a persistent CTA 100 besides its steps; clusters of 2 and 4 can use
// about 95 % of the SMs, of 8 84 %. Measured, whole and shared by 2, 4, 8, in us: 40 items of up to 73 steps 76,
// 42, 26, 37; 128 of up to 128 steps 121, 66, 81, 121; 224 of up to 49 steps 94, 83, 105, 171; 224 of up to 64
// steps 83, 87, 112, 171; 28 of up to 5 steps 12.4, 10.8, 10.7.
int choose_split(const ChunkWeightsArgs& a, int64_t items, int64_t rows, int64_t n_tiles, int n_queries, int qpt, int sms) {
  const int64_t prefix = std::max<int64_t>(0, (int64_t)a.max_blocks * a.page_size - a.chunk_len);
  auto steps_of = [&](int64_t tile) {  // of the items of a key tile
    const int64_t first = std::max<int64_t>(a.chunk_len - n_queries, tile * CK - prefix);
    return first < a.chunk_len ? (a.chunk_len - first + qpt - 1) / qpt : 0;
  };
  const int64_t steps = steps_of(0);
  if (steps < 2) return 0;
  const int64_t seen = std::min<int64_t>(n_tiles, (n_queries + CK - 1) / CK);  // tiles that part of the queries see
  const int64_t total = 100 * rows * (steps * (n_tiles - seen) + steps * seen / 2);
  // whole items: the CTA with the most, exactly where there are few, else the mean
  int64_t best = 0;
  if (items <= 4 * (int64_t)sms) {
    for (int i = 0; i < sms && i < items; ++i) {
      int64_t sum = 0, at = i;
      for (int odd = 0; at < items; odd ^= 1) {
        sum += 100 * steps_of(at / rows) + 100;
        at += odd ? 2 * i + 1 : 2 * (int64_t)sms - 1 - 2 * i;
      }
      best = std::max(best, sum);
    }
    best += 600;
  } else {
    best = 700 + (total + 100 * items) / sms;
  }
  int s_log2 = 0;
  for (int s = 1; s <= 3 && (1 << s) <= steps && items << s <= 0x7fffffffL; ++s) {
    const int64_t part = 100 * ((steps + (1 << s) - 1) >> s) + 700;
    const int64_t cost = std::max(part, (total + 700 * (items << s)) / (sms * (s == 3 ? 84 : 95) / 100) + part / 4);
    if (cost + cost / 20 < best) best = cost, s_log2 = s;  // (the estimate is off by a few per cent)
  }
  return s_log2;
}

}  // namespace

int launch_chunk_weights(const ChunkWeightsArgs& a, cudaStream_t stream) {
  const int G = a.n_qo_heads / a.n_kv_heads;
  CUtensorMap mq, mk;
  {
    // q [B][C][Hq][128] as (128, Hq, C, B): a box is 64 dims of the group's heads of qpt queries
    // (a chunk without queries loads none: any aligned address and length make a map)
    const cuuint64_t chunk = (cuuint64_t)std::max(a.chunk_len, 1);
    cuuint64_t dims[4] = {CD, (cuuint64_t)a.n_qo_heads, chunk, (cuuint64_t)a.batch};
    cuuint64_t strides[3] = {CD * 2, (cuuint64_t)a.n_qo_heads * CD * 2, chunk * a.n_qo_heads * CD * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)(CN / G), 1};
    if (!encode(&mq, a.chunk_len > 0 ? a.q : a.k_pages, 4, dims, strides, box)) return check_launch(cudaErrorInvalidValue);
  }
  {
    // pools as (64 dims, 8 rows, 2 halves, 8-row groups): a box is one (page, KV head) block
    cuuint64_t dims[4] = {64, 8, 2, (cuuint64_t)a.num_pages * a.n_kv_heads * 2};
    cuuint64_t strides[3] = {CD * 2, 128, 8 * CD * 2};
    cuuint32_t box[4] = {64, 8, 2, 2};
    if (!encode(&mk, a.k_pages, 4, dims, strides, box)) return check_launch(cudaErrorInvalidValue);
  }
  const int64_t cap = (int64_t)a.max_blocks * a.page_size;
  const int64_t rows = (int64_t)a.batch * a.n_kv_heads, n_tiles = (cap + CK - 1) / CK;
  if (rows > 0x3fffffffL || n_tiles * rows > 0x7fffffffL) return PKV_ERR_UNSUPPORTED;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  const int n_queries = a.window > 0 && a.window < a.chunk_len ? a.window : a.chunk_len;
  const int s_log2 = choose_split(a, n_tiles * rows, rows, n_tiles, n_queries, CN / G, sms);
  if (s_log2 == 0) {
    // a CTA per SM, more where the list of one cannot hold its share
    const int64_t waves = (n_tiles * rows + (int64_t)sms * (CITEMS - 2) - 1) / ((int64_t)sms * (CITEMS - 2));
    static FuncConfigured configured;
    if (!configured.ensure(reinterpret_cast<const void*>(chunk_weights_kernel<false>), C_SMEM)) return PKV_ERR_LAUNCH;
    const int64_t grid = n_tiles * rows < sms * waves ? n_tiles * rows : sms * waves;
    return check_launch(launch_overlapped(chunk_weights_kernel<false>, dim3((unsigned)grid), CTHREADS, C_SMEM, stream, 1,
                                          mq, mk, a, (int)(n_tiles * rows), 0));
  }
  static FuncConfigured configured;
  if (!configured.ensure(reinterpret_cast<const void*>(chunk_weights_kernel<true>), C_SMEM)) return PKV_ERR_LAUNCH;
  return check_launch(launch_overlapped(chunk_weights_kernel<true>, dim3((unsigned)(n_tiles * rows << s_log2)),
                                        CTHREADS, C_SMEM, stream, 1 << s_log2, mq, mk, a, (int)(n_tiles * rows), s_log2));
}

}  // namespace pkv
