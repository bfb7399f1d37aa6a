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
// SM, so a 256 x 128 step takes 2048 clocks of it against 1024 of tensor work.
//
// A persistent CTA per SM takes items (sequence, KV head, 256 keys), those with the most
// queries to see first. Warps: 0 TMA producer (K tiles by page, two items deep; Q tiles, three
// deep), 1 MMA issuer, 2 the columns' log-sum-exps into shared memory, 4..7 and 8..11 the two key
// tiles' exponentials and sums. S^T is double-buffered per tile: all 512 TMEM columns.
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
  int total;   // keys of the sequence after the chunk; 0: nothing to do
  int prefix;
  int q_begin, q_end;  // queries that count and see a key of the item: [q_begin, q_end)
  int steps;
};

__device__ __forceinline__ Item make_item(const ChunkWeightsArgs& a, int id, int qpt) {
  Item it{};
  const int rows = a.batch * a.n_kv_heads;
  it.key0 = (id / rows) * CK;
  const int r = id % rows;
  it.b = r / a.n_kv_heads;
  it.hk = r % a.n_kv_heads;
  const int64_t prefix = __ldg(a.prefix_lens + it.b);
  const int64_t n = a.chunk_lens ? __ldg(a.chunk_lens + it.b) : a.chunk_len;
  const int64_t cap = (int64_t)a.max_blocks * a.page_size;
  if (prefix < 0 || n < 0 || n > a.chunk_len || prefix + n > cap) {
    it.total = -1;  // bad lengths
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
  it.steps = it.q_end > it.q_begin ? (it.q_end - it.q_begin + qpt - 1) / qpt : 0;
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

// acc += exp2(s * c + nl) over 32 columns; MASKED: columns outside [lo, hi) do not count.
template <bool MASKED>
__device__ __forceinline__ void add_columns(const uint32_t (&s)[32], const float* nl, uint64_t c2, int col0, int lo,
                                            int hi, uint64_t (&acc)[2]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const ulonglong2 n = *reinterpret_cast<const ulonglong2*>(nl + i);
    const float2 x0 = upk2(ffma2(pk2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, n.x));
    const float2 x1 = upk2(ffma2(pk2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), c2, n.y));
    float e[4] = {ex2(x0.x), ex2(x0.y), ex2(x1.x), ex2(x1.y)};
    if (MASKED) {
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = col0 + i + k >= lo && col0 + i + k < hi ? e[k] : 0.0f;
    }
    acc[0] = fadd2(acc[0], pk2(e[0], e[1]));
    acc[1] = fadd2(acc[1], pk2(e[2], e[3]));
  }
}

__global__ void __launch_bounds__(CTHREADS, 1)
chunk_weights_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const ChunkWeightsArgs a, int n_items) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  unsigned char* smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  CMisc* misc = reinterpret_cast<CMisc*>(smem + SM_MISC);
  auto bar = [&](int i) { return sb + SM_BAR + 8 * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.n_qo_heads / a.n_kv_heads, qpt = CN / G;  // queries per step

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

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (elect_one()) {
      tma_prefetch_desc(&mq);
      tma_prefetch_desc(&mk);
    }
    __syncwarp();
    uint32_t kc = 0, qc = 0;
    bool ok = true;
    for (int id = blockIdx.x; ok && id < n_items; id += gridDim.x) {
      const Item it = make_item(a, id, qpt);
      if (it.steps == 0) continue;
      const uint32_t ks = kc % NKS;
      if (kc >= NKS && !warp_wait(bar(C_KE + ks), (kc / NKS - 1) & 1)) ok = false;
      if (__any_sync(0xffffffffu, *aborted)) ok = false;
      if (!ok) break;
      // lane p < 16 brings page p of the item; slots past the sequence bring its first page
      // again (their keys are not written), a bad entry page 0 (its keys become NaN)
      const int pages = min(CK / 16, (it.total - it.key0 + 15) / 16);
      int phys = 0;
      if (lane < 16) {
        phys = __ldg(a.block_table + (int64_t)it.b * a.max_blocks + it.key0 / 16 + (lane < pages ? lane : 0));
        if (phys < 0 || phys >= a.num_pages) phys = 0;
      }
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
      for (int s = 0; s < it.steps; ++s, ++qc) {
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
    for (int id = blockIdx.x; ok && id < n_items; id += gridDim.x) {
      const Item it = make_item(a, id, qpt);
      if (it.steps == 0) continue;
      const uint32_t ks = kc % NKS;
      if (!warp_wait(bar(C_KF + ks), (kc / NKS) & 1)) ok = false;
      for (int s = 0; ok && s < it.steps; ++s, ++qc) {
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
              if (s == it.steps - 1) mma_commit(bar(C_KE + ks));
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
    uint32_t qc = 0;
    bool ok = true;
    for (int id = blockIdx.x; ok && id < n_items; id += gridDim.x) {
      const Item it = make_item(a, id, qpt);
      for (int s = 0; ok && s < it.steps; ++s, ++qc) {
        const uint32_t qs = qc % NQS;
        float v[CN / 32];
#pragma unroll
        for (int k = 0; k < CN / 32; ++k) {
          const int col = k * 32 + lane, i = it.q_begin + s * qpt + col / G;
          v[k] = i < it.q_end
                     ? __ldg(a.lse + ((int64_t)it.b * a.n_qo_heads + it.hk * G + col % G) * a.chunk_len + i)
                     : 0.0f;
        }
        if (qc >= NQS && !warp_wait(bar(C_LE + qs), (qc / NQS - 1) & 1)) ok = false;
        if (__any_sync(0xffffffffu, *aborted)) ok = false;
        if (!ok) break;
        float* dst = reinterpret_cast<float*>(smem + SM_L) + qs * CN;
#pragma unroll
        for (int k = 0; k < CN / 32; ++k) dst[k * 32 + lane] = -kL2e * v[k];
        __syncwarp();
        if (elect_one()) mbar_arrive(bar(C_LF + qs));
        __syncwarp();
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
    const int64_t cap = (int64_t)a.max_blocks * a.page_size;
    uint32_t qc = 0;
    bool ok = true;
    for (int id = blockIdx.x; id < n_items; id += gridDim.x) {
      const Item it = make_item(a, id, qpt);
      if (it.total <= 0) {
        if (it.total < 0 && t == 0 && it.key0 == 0 && it.hk == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
        continue;
      }
      const int key = it.key0 + t;
      const bool live = key < it.total;
      const int64_t at = ((int64_t)it.b * a.n_kv_heads + it.hk) * cap + key;
      float before = 0.0f;
      int page = 0;
      if (live) {
        before = a.sums_in[at];
        page = __ldg(a.block_table + (int64_t)it.b * a.max_blocks + key / 16);
      }
      uint64_t acc[2] = {0ull, 0ull};
      float total = 0.0f;
      for (int s = 0; ok && s < it.steps; ++s, ++qc) {
        const uint32_t qs = qc % NQS, buf = qc & 1;
        ok = warp_wait(bar(C_LF + qs), (qc / NQS) & 1) && warp_wait(bar(C_SF + 2 * tile + buf), (qc / 2) & 1);
        if (!ok) break;
        tc_fence_after();
        const float* nl = reinterpret_cast<const float*>(smem + SM_L) + qs * CN;
        const int q0 = it.q_begin + s * qpt;
        // columns [lo, hi) count: the causal bound and the end of the chunk
        const int lo = (key - it.prefix - q0) * G, hi = min(CN, (it.q_end - q0) * G);
        const uint32_t src = tmem + lane_addr + (2 * tile + buf) * CN;
        const bool whole = __all_sync(0xffffffffu, lo <= 0) && hi == CN;
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
        // long sums: a step's columns are added up on their own first
        const float2 x = upk2(fadd2(acc[0], acc[1]));
        total += x.x + x.y;
        acc[0] = acc[1] = 0ull;
      }
      if (live) {
        float out = fmaf(a.decay, before, total);
        if (page < 0 || page >= a.num_pages) {
          set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
          out = NAN;
        }
        a.sums_out[at] = ok ? out : NAN;
      }
    }
    if (!ok) give_up();
  }

  tc_fence_before();
  __syncthreads();
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
  static FuncConfigured configured;
  if (!configured.ensure(reinterpret_cast<const void*>(chunk_weights_kernel), C_SMEM)) return PKV_ERR_LAUNCH;
  const int64_t cap = (int64_t)a.max_blocks * a.page_size;
  const int64_t n_items = (cap + CK - 1) / CK * a.batch * a.n_kv_heads;
  if (n_items > 0x7fffffffL) return PKV_ERR_UNSUPPORTED;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  const unsigned grid = (unsigned)(n_items < sms ? n_items : sms);
  chunk_weights_kernel<<<grid, CTHREADS, C_SMEM, stream>>>(mq, mk, a, (int)n_items);
  return check_launch(cudaGetLastError());
}

}  // namespace pkv
