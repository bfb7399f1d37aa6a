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
// Bound: one exponential per (key, query, head). The special-function unit gives 16 a clock and
// SM, 2048 clocks for a 256 x 128 step, and the two products of a step take about 1750 (128 x 128
// products read both operands from shared memory, which is their limit). So a quarter of the
// exponentials are computed as polynomials on the FMA units instead, which leaves the special-
// function unit 1536 clocks and puts the products on the critical path.
//
// A persistent CTA per SM takes items (sequence, KV head, 256 keys) in an order that pairs long and
// short ones: key tiles slowest (early keys are seen by the most queries), and every other round
// of the CTAs backwards. With fewer items than half the SMs an item's steps are shared by a
// cluster of 2 to 8 CTAs, whose partial sums are added in rank order through distributed shared memory.
// Warps: 0 TMA producer (K tiles by page, two items deep; Q tiles, three deep), 1 MMA issuer, 2 the
// columns' log-sum-exps into shared memory, 4..7 and 8..11 the two key tiles' exponentials and
// sums. S^T is double-buffered per tile: all 512 TMEM columns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <cmath>

#include "internal.h"
#include "tcgen05.cuh"

namespace pkv {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // prefill.cu

namespace {

constexpr int CD = 128;                // head dim
constexpr int CK = 256;                // keys per item: two 128-row tiles
constexpr int CN = 128;                // columns (queries x heads of the group) per step
constexpr int KSTG = CK * CD * 2;      // one K stage, 64 KiB: tile 0 halves, tile 1 halves
constexpr int QSTG = CN * CD * 2;      // one Q stage, 32 KiB: two 64-dim halves
constexpr int HALF = 128 * 128;        // [128 rows][128 bytes]
constexpr int NKS = 2, NQS = 3;
constexpr int CTHREADS = 384;
// barriers
constexpr int C_KF = 0, C_KE = 2, C_QF = 4, C_QE = 7, C_LF = 10, C_LE = 13, C_SF = 16, C_SE = 20, C_DR = 24, C_NBAR = 25;
constexpr int SM_K = 0, SM_Q = SM_K + NKS * KSTG, SM_L = SM_Q + NQS * QSTG, SM_BAR = SM_L + NQS * CN * 4,
              SM_MISC = SM_BAR + C_NBAR * 8, C_SMEM = SM_MISC + 16 + 1024;
static_assert(C_SMEM <= 232448, "shared memory per CTA");
constexpr float kL2e = 1.4426950408889634f;

struct CMisc {
  uint32_t tmem_base;
  int abort_;
};

// One item: the keys it covers and the steps of columns that see any of them.
struct Item {
  int b, hk, key0;
  int total;   // keys of the sequence after the chunk; 0: nothing to do; -1: bad lengths
  int prefix;
  int q_begin, q_end;  // queries that count and see a key of the item: [q_begin, q_end)
  int steps;
};

// Where a CTA stands in the items: key tiles slowest, then sequences, then KV heads. CTA i of P
// takes items i, 2P - 1 - i, 2P + i, ...; the two distances are added in turn in mixed radix, so
// that no role divides by run-time sizes for each item.
struct Cursor {
  int tile, b, hk;
  int d_tile[2], d_b[2], d_hk[2], odd;
  __device__ __forceinline__ Cursor(const ChunkWeightsArgs& a, int i, int P) : odd(0) {
    const int rows = a.batch * a.n_kv_heads;
    auto split = [&](int x, int& t, int& b_, int& h) {
      t = x / rows;
      b_ = x % rows / a.n_kv_heads;
      h = x % rows % a.n_kv_heads;
    };
    split(i, tile, b, hk);
    split(2 * P - 1 - 2 * i, d_tile[0], d_b[0], d_hk[0]);
    split(2 * i + 1, d_tile[1], d_b[1], d_hk[1]);
  }
  __device__ __forceinline__ void next(const ChunkWeightsArgs& a) {
    hk += odd ? d_hk[1] : d_hk[0];
    b += odd ? d_b[1] : d_b[0];
    tile += odd ? d_tile[1] : d_tile[0];
    if (hk >= a.n_kv_heads) hk -= a.n_kv_heads, ++b;
    if (b >= a.batch) b -= a.batch, ++tile;
    odd ^= 1;
  }
};

__device__ __forceinline__ Item make_item(const ChunkWeightsArgs& a, const Cursor& c, int qpt_log2) {
  Item it{};
  it.key0 = c.tile * CK;
  it.b = c.b;
  it.hk = c.hk;
  const int64_t prefix = __ldg(a.prefix_lens + it.b);
  const int64_t n = a.chunk_lens ? __ldg(a.chunk_lens + it.b) : a.chunk_len;
  const int64_t cap = (int64_t)a.max_blocks * a.page_size;
  if (prefix < 0 || n < 0 || n > a.chunk_len || prefix + n > cap) {
    it.total = -1;
    return it;
  }
  it.total = (int)(prefix + n);
  it.prefix = (int)prefix;
  if (it.key0 >= it.total) {
    it.total = 0;
    return it;
  }
  const int first = a.window > 0 && a.window < n ? (int)n - a.window : 0;
  it.q_begin = max(first, it.key0 - it.prefix);
  it.q_end = (int)n;
  it.steps = it.q_end > it.q_begin ? (it.q_end - it.q_begin + (1 << qpt_log2) - 1) >> qpt_log2 : 0;
  return it;
}

__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 upk2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2^x of a pair without the special-function unit, x <= 0: x = n + f with n the nearest integer
// (adding 1.5 * 2^23 leaves it in the low bits), 2^f on [-1/2, 1/2] as the degree-5 polynomial of
// least relative error (2e-7 with its fp32 roundings; the exponent unit's is 1e-7), times 2^n
// made from n's bits. Below -126 it stays at 2^-126; NaN stays NaN.
__device__ __forceinline__ uint64_t exp2_poly2(uint64_t x2) {
  constexpr float kRound = 12582912.0f;
  const float2 x = upk2(x2);
  const uint64_t y = pk2(max_nan(x.x, -126.0f), max_nan(x.y, -126.0f));
  const uint64_t t = fadd2(y, pk2(kRound, kRound));
  const uint64_t n = fadd2(t, pk2(-kRound, -kRound));
  const uint64_t f = ffma2(n, pk2(-1.0f, -1.0f), y);
  uint64_t p = pk2(0.0013276472f, 0.0013276472f);
  p = ffma2(p, f, pk2(0.009675541f, 0.009675541f));
  p = ffma2(p, f, pk2(0.05550713f, 0.05550713f));
  p = ffma2(p, f, pk2(0.2402212f, 0.2402212f));
  p = ffma2(p, f, pk2(0.69314694f, 0.69314694f));
  p = ffma2(p, f, pk2(1.0f, 1.0f));
  const float2 b = upk2(t);
  return fmul2(p, pk2(__uint_as_float((__float_as_uint(b.x) << 23) + 0x3f800000u),
                      __uint_as_float((__float_as_uint(b.y) << 23) + 0x3f800000u)));
}

// acc += exp2(s * c + nl) over 32 columns; MASKED: columns outside [lo, hi) do not count.
template <bool MASKED>
__device__ __forceinline__ void add_columns(const uint32_t (&s)[32], const float* nl, uint64_t c2, int col0, int lo,
                                            int hi, uint64_t (&acc)[2]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    uint64_t e[4];
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      const ulonglong2 n = *reinterpret_cast<const ulonglong2*>(nl + i + 2 * k);
      e[k] = ffma2(pk2(__uint_as_float(s[i + 2 * k]), __uint_as_float(s[i + 2 * k + 1])), c2, n.x);
      e[k + 1] = ffma2(pk2(__uint_as_float(s[i + 2 * k + 2]), __uint_as_float(s[i + 2 * k + 3])), c2, n.y);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k == 3) {
        e[k] = exp2_poly2(e[k]);
      } else {
        const float2 x = upk2(e[k]);
        e[k] = pk2(ex2(x.x), ex2(x.y));
      }
      if (MASKED) {
        const float2 x = upk2(e[k]);
        const int c = col0 + i + 2 * k;
        e[k] = pk2(c >= lo && c < hi ? x.x : 0.0f, c + 1 >= lo && c + 1 < hi ? x.y : 0.0f);
      }
      acc[k & 1] = fadd2(acc[k & 1], e[k]);
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
                     const ChunkWeightsArgs a, int n_tiles, int S) {
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
  const int rank = SPLIT ? (int)cluster_rank() : 0;  // steps rank, rank + S, ... of the CTA's items
  const int cta = SPLIT ? (int)blockIdx.x / S : (int)blockIdx.x, ctas = SPLIT ? (int)gridDim.x / S : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C_NBAR; ++i) {
      int cnt = 1;
      if (i >= C_SE && i < C_SE + 4) cnt = 4;  // the four warps of a key tile
      if (i >= C_LE && i < C_LE + NQS) cnt = 8;  // all eight
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

  // One key of an item: where its sum is, the old sum, and whether its page exists.
  struct Mine {
    int64_t at;
    float before;
    bool live, bad_page;
  };
  auto my_key = [&](const Item& it, int t) {
    Mine m{};
    const int key = it.key0 + t;
    m.live = it.total > 0 && key < it.total;
    if (m.live) {
      m.at = ((int64_t)it.b * a.n_kv_heads + it.hk) * ((int64_t)a.max_blocks * a.page_size) + key;
      m.before = a.sums_in[m.at];
      const int page = __ldg(a.block_table + (int64_t)it.b * a.max_blocks + key / 16);
      m.bad_page = page < 0 || page >= a.num_pages;
    }
    return m;
  };
  auto store = [&](const Mine& m, float total) {
    if (m.bad_page) set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
    a.sums_out[m.at] = m.bad_page ? NAN : fmaf(a.decay, m.before, total);
  };
  float part = 0.0f;  // SPLIT: this CTA's share of a key's sum

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (elect_one()) {
      tma_prefetch_desc(&mq);
      tma_prefetch_desc(&mk);
    }
    __syncwarp();
    uint32_t kc = 0, qc = 0;
    bool ok = true;
    // lane p < 16 holds the table entry of page p of the item; slots past the sequence bring its
    // first page again (their keys are not written), a bad entry page 0 (its keys become NaN).
    // The next item's entries are asked for before this item's copies wait for room.
    auto entry = [&](const Item& it) {
      const int pages = min(CK / 16, (it.total - it.key0 + 15) / 16);
      return lane < 16 && it.steps > 0
                 ? __ldg(a.block_table + (int64_t)it.b * a.max_blocks + it.key0 / 16 + (lane < pages ? lane : 0))
                 : 0;
    };
    Cursor at(a, cta, ctas);
    Item next{};
    int next_phys = 0;
    bool more = at.tile < n_tiles;
    if (more) {
      next = make_item(a, at, qpt_log2);
      next_phys = entry(next);
    }
    while (ok && more) {
      const Item it = next;
      int phys = next_phys;
      at.next(a);
      more = at.tile < n_tiles;
      if (more) {
        next = make_item(a, at, qpt_log2);
        next_phys = entry(next);
      }
      if (it.steps == 0) continue;
      const uint32_t ks = kc % NKS;
      if (kc >= NKS && !warp_wait(bar(C_KE + ks), (kc / NKS - 1) & 1)) ok = false;
      if (__any_sync(0xffffffffu, *aborted)) ok = false;
      if (!ok) break;
      if (phys < 0 || phys >= a.num_pages) phys = 0;
      __syncwarp();
      if (lane == 0) mbar_arrive_expect_tx(bar(C_KF + ks), KSTG);
      __syncwarp();
      if (lane < 16) {
        const uint32_t dst = sb + SM_K + ks * KSTG + (lane >> 3) * 2 * HALF + (lane & 7) * 2048;
        const int row = (phys * a.n_kv_heads + it.hk) * 16;
        tma_load_2d(dst, &mk, 0, row, bar(C_KF + ks));
        tma_load_2d(dst + HALF, &mk, 64, row, bar(C_KF + ks));
      }
      __syncwarp();
      ++kc;
      for (int s = rank; s < it.steps; s += S, ++qc) {
        const uint32_t qs = qc % NQS;
        if (qc >= NQS && !warp_wait(bar(C_QE + qs), (qc / NQS - 1) & 1)) ok = false;
        if (__any_sync(0xffffffffu, *aborted)) ok = false;
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(bar(C_QF + qs), QSTG);
          const uint32_t dst = sb + SM_Q + qs * QSTG;
          tma_load_4d(dst, &mq, 0, it.hk * G, it.q_begin + s * qpt, it.b, bar(C_QF + qs));
          tma_load_4d(dst + HALF, &mq, 64, it.hk * G, it.q_begin + s * qpt, it.b, bar(C_QF + qs));
        }
        __syncwarp();
      }
    }
    if (!ok) give_up();
    // every issued copy lands before the shared memory is released
    bool drained = true;
    for (uint32_t s = 0; s < NKS && s < kc; ++s)
      drained &= warp_wait(bar(C_KF + s), ((kc - 1 - s) / NKS) & 1);
    for (uint32_t s = 0; s < NQS && s < qc; ++s)
      drained &= warp_wait(bar(C_QF + s), ((qc - 1 - s) / NQS) & 1);
    if (!drained) give_up();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16_f32(128, CN, false, false);
    const uint64_t dk0 = smem_desc(sb + SM_K, 16, 1024, kSwizzle128B);
    const uint64_t dq0 = smem_desc(sb + SM_Q, 16, 1024, kSwizzle128B);
    uint32_t kc = 0, qc = 0;
    bool ok = true;
    for (Cursor at(a, cta, ctas); ok && at.tile < n_tiles; at.next(a)) {
      const Item it = make_item(a, at, qpt_log2);
      if (it.steps == 0) continue;
      const uint32_t ks = kc % NKS;
      if (!warp_wait(bar(C_KF + ks), (kc / NKS) & 1)) ok = false;
      for (int s = rank; ok && s < it.steps; s += S, ++qc) {
        const uint32_t qs = qc % NQS, buf = qc & 1;
        if (!warp_wait(bar(C_QF + qs), (qc / NQS) & 1)) {
          ok = false;
          break;
        }
        for (int tile = 0; ok && tile < 2; ++tile) {
          if (qc >= 2 && !warp_wait(bar(C_SE + 2 * tile + buf), (qc / 2 - 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dk = dk0 + (uint64_t)((ks * KSTG + tile * 2 * HALF) >> 4);
            const uint64_t dq = dq0 + (uint64_t)((qs * QSTG) >> 4);
#pragma unroll
            for (int kk = 0; kk < CD / 16; ++kk) {
              const uint64_t off = (uint64_t)(((kk / 4) * HALF + (kk % 4) * 32) >> 4);
              mma_bf16_ss(tmem + (2 * tile + buf) * CN, dk + off, dq + off, idesc, kk > 0 ? 1u : 0u);
            }
            mma_commit(bar(C_SF + 2 * tile + buf));
            if (tile == 1) {
              mma_commit(bar(C_QE + qs));
              if (s + S >= it.steps) mma_commit(bar(C_KE + ks));
            }
          }
          __syncwarp();
        }
      }
      ++kc;
    }
    if (!ok) give_up();
    // every issued product finishes before TMEM is freed
    if (elect_one()) mma_commit(bar(C_DR));
    __syncwarp();
    if (!warp_wait(bar(C_DR), 0)) give_up();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ log-sum-exps
    // Step after step through the CTA's items; the values of kAhead steps are on their way, since
    // one step takes less time than one load from the L2.
    constexpr int kAhead = 4;
    // the lane's columns: query and place in lse of a step
    int query[CN / 32];
    int64_t place[CN / 32];
#pragma unroll
    for (int k = 0; k < CN / 32; ++k) {
      const int col = k * 32 + lane;
      query[k] = col >> g_log2;
      place[k] = (int64_t)(col & (G - 1)) * a.chunk_len + query[k];
    }
    Cursor at(a, cta, ctas);
    int s = rank;
    Item it{};
    const float* rows = a.lse;
    auto enter = [&]() {
      it = make_item(a, at, qpt_log2);
      s = rank;
      rows = a.lse + ((int64_t)it.b * a.n_qo_heads + it.hk * G) * a.chunk_len;
    };
    if (at.tile < n_tiles) enter();
    auto load = [&](float (&v)[CN / 32]) -> bool {  // the next step's columns; false: no more steps
      while (at.tile < n_tiles && s >= it.steps) {
        at.next(a);
        if (at.tile < n_tiles) enter();
      }
      if (at.tile >= n_tiles) return false;
      const int q0 = it.q_begin + (s << qpt_log2);
#pragma unroll
      for (int k = 0; k < CN / 32; ++k) v[k] = q0 + query[k] < it.q_end ? __ldg(rows + q0 + place[k]) : 0.0f;
      s += S;
      return true;
    };
    float v[kAhead][CN / 32];
    bool has[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) has[u] = load(v[u]);
    uint32_t qc = 0;
    bool ok = true, more = true;
    while (ok && more) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (!ok || !has[u]) {
          more = false;
          continue;
        }
        const uint32_t qs = qc % NQS;
        if (qc >= NQS && !warp_wait(bar(C_LE + qs), (qc / NQS - 1) & 1)) ok = false;
        if (__any_sync(0xffffffffu, *aborted)) ok = false;
        if (ok) {
          float* dst = reinterpret_cast<float*>(smem + SM_L) + qs * CN;
#pragma unroll
          for (int k = 0; k < CN / 32; ++k) dst[k * 32 + lane] = -kL2e * v[u][k];
          __syncwarp();
          if (elect_one()) mbar_arrive(bar(C_LF + qs));
          __syncwarp();
          ++qc;
          has[u] = load(v[u]);
        }
      }
    }
    if (!ok) give_up();
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ exponentials and sums
    const int tile = (warp - 4) >> 2, wq = warp & 3;
    const int t = tile * 128 + wq * 32 + lane;  // key within the item
    const uint32_t lane_addr = (uint32_t)(wq * 32) << 16;
    const float c = a.scale * kL2e;
    const uint64_t c2 = pk2(c, c);
    uint32_t qc = 0;
    bool ok = true;
    // the next item's lengths, old sum and table entry are asked for before this one's steps
    Cursor at(a, cta, ctas);
    Item it{};
    Mine mine{};
    bool more = at.tile < n_tiles;
    if (more) {
      it = make_item(a, at, qpt_log2);
      mine = my_key(it, t);
    }
    while (more) {
      const Item now = it;
      const Mine my = mine;
      at.next(a);
      more = at.tile < n_tiles;
      if (more) {
        it = make_item(a, at, qpt_log2);
        mine = my_key(it, t);
      }
      if (now.total <= 0) {
        if (now.total < 0 && t == 0 && now.key0 == 0 && now.hk == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
        continue;
      }
      const int key = now.key0 + t;
      float total = 0.0f;
      for (int s = rank; ok && s < now.steps; s += S, ++qc) {
        const uint32_t qs = qc % NQS, buf = qc & 1;
        ok = warp_wait(bar(C_LF + qs), (qc / NQS) & 1) && warp_wait(bar(C_SF + 2 * tile + buf), (qc / 2) & 1);
        if (!ok) break;
        tc_fence_after();
        const float* nl = reinterpret_cast<const float*>(smem + SM_L) + qs * CN;
        const int q0 = now.q_begin + s * qpt;
        // columns [lo, hi) count: the causal bound and the end of the chunk
        const int lo = (key - now.prefix - q0) * G, hi = min(CN, (now.q_end - q0) * G);
        const uint32_t src = tmem + lane_addr + (2 * tile + buf) * CN;
        const bool whole = __all_sync(0xffffffffu, lo <= 0) && hi == CN;
        uint64_t acc[2] = {0ull, 0ull};
        uint32_t r[2][32];
        tmem_ld32(src, r[0]);
#pragma unroll
        for (int k = 0; k < CN / 32; ++k) {
          tmem_ld_wait();
          if (k + 1 < CN / 32) tmem_ld32(src + (k + 1) * 32, r[(k + 1) & 1]);
          if (whole)
            add_columns<false>(r[k & 1], nl + 32 * k, c2, 32 * k, lo, hi, acc);
          else
            add_columns<true>(r[k & 1], nl + 32 * k, c2, 32 * k, lo, hi, acc);
        }
        tc_fence_before();
        __syncwarp();
        if (elect_one()) {
          mbar_arrive(bar(C_SE + 2 * tile + buf));
          mbar_arrive(bar(C_LE + qs));
        }
        __syncwarp();
        // a step's columns are added up on their own first: shorter chains of roundings
        const float2 x = upk2(fadd2(acc[0], acc[1]));
        total += x.x + x.y;
      }
      if (!ok) total = NAN;
      if constexpr (SPLIT) {
        part = total;
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
    float* parts = reinterpret_cast<float*>(smem + SM_L);  // (every step has been read)
    static_assert(NQS * CN >= CK, "one float per key");
    if (warp >= 4) parts[threadIdx.x - 128] = part;
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int share = CK / S, t = rank * share + (int)threadIdx.x;
    if ((int)threadIdx.x < share) {
      const Item it = make_item(a, Cursor(a, cta, ctas), qpt_log2);
      const Mine my = my_key(it, t);
      if (my.live) {
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

}  // namespace

int launch_chunk_weights(const ChunkWeightsArgs& a, cudaStream_t stream) {
  const int G = a.n_qo_heads / a.n_kv_heads;
  CUtensorMap mq, mk;
  {
    // q [B][C][Hq][128] as (128, Hq, C, B): a box is 64 dims of the group's heads of qpt queries
    cuuint64_t dims[4] = {CD, (cuuint64_t)a.n_qo_heads, (cuuint64_t)a.chunk_len, (cuuint64_t)a.batch};
    cuuint64_t strides[3] = {CD * 2, (cuuint64_t)a.n_qo_heads * CD * 2, (cuuint64_t)a.chunk_len * a.n_qo_heads * CD * 2};
    cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)(CN / G), 1};
    if (!encode(&mq, a.q, 4, dims, strides, box)) return check_launch(cudaErrorInvalidValue);
  }
  {
    cuuint64_t dims[2] = {CD, (cuuint64_t)a.num_pages * a.n_kv_heads * 16};
    cuuint64_t strides[1] = {CD * 2};
    cuuint32_t box[2] = {64, 16};
    if (!encode(&mk, a.k_pages, 2, dims, strides, box)) return check_launch(cudaErrorInvalidValue);
  }
  const int64_t cap = (int64_t)a.max_blocks * a.page_size;
  const int64_t rows = (int64_t)a.batch * a.n_kv_heads, n_tiles = (cap + CK - 1) / CK;
  if (rows > 0x3fffffffL || n_tiles * rows > 0x7fffffffL) return PKV_ERR_UNSUPPORTED;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  // Few items: share the steps of each among the largest cluster that fits the SMs and leaves
  // every CTA a step.
  const int n_queries = a.window > 0 && a.window < a.chunk_len ? a.window : a.chunk_len;
  const int64_t steps = ((int64_t)n_queries * G + CN - 1) / CN;
  int S = 1;
  while (S < 8 && 2 * S <= steps && 2 * S * n_tiles * rows <= sms) S *= 2;
  if (S == 1) {
    static FuncConfigured configured;
    if (!configured.ensure(reinterpret_cast<const void*>(chunk_weights_kernel<false>), C_SMEM)) return PKV_ERR_LAUNCH;
    const int grid = (int)(n_tiles * rows < sms ? n_tiles * rows : sms);
    chunk_weights_kernel<false><<<grid, CTHREADS, C_SMEM, stream>>>(mq, mk, a, (int)n_tiles, 1);
    return check_launch(cudaGetLastError());
  }
  static FuncConfigured configured;
  if (!configured.ensure(reinterpret_cast<const void*>(chunk_weights_kernel<true>), C_SMEM)) return PKV_ERR_LAUNCH;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(S * n_tiles * rows), 1, 1);
  cfg.blockDim = dim3(CTHREADS, 1, 1);
  cfg.dynamicSmemBytes = C_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return check_launch(cudaLaunchKernelEx(&cfg, chunk_weights_kernel<true>, mq, mk, a, (int)n_tiles, S));
}

}  // namespace pkv
