// Eviction from the paged cache by accumulated attention weight.
//
// Of a sequence's n tokens a KV head keeps min(n, budget): the first n_sink, the last n_recent
// and, of those between, the ones with the largest sums (equal sums: the lower index), in their
// order. The kept rows of K and V are gathered into the pages of a new table, so shared source
// pages stay whole and no row is overwritten before it is read.
//
// Two kernels. The selection is one CTA per (sequence, KV head): a float's order-preserving
// bits are searched for the m-th largest by three passes of 11, 11 and 10 bits, each a
// histogram in shared memory of the values that share the digits found so far; only the first
// pass has every value in it. Then each warp, which holds a contiguous run of tokens, counts
// what it keeps, one scan over the warps places the runs, and the kept indices and sums are
// written in order. The gather is one lane group per kept row, K and V of four rows in flight.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;

// Bits that order as the floats do; both zeros are equal, and NaN is above every number.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Tokens per thread held in registers, E; 0: read again from memory in each pass.
template <int E>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictArgs a) {
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[kSelWarps], s_warp2[kSelWarps];
  __shared__ int s_digit, s_above;
  const int b = blockIdx.y, h = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cap = a.max_blocks * a.page_size, new_cap = a.new_max_blocks * a.page_size;
  int n = __ldg(a.kv_lens + b);
  if (n < 0 || n > cap) {
    if (tid == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
    n = 0;
  }
  const int64_t row = (int64_t)b * a.n_kv_heads + h;
  const float* sums = a.sums + row * cap;
  float* new_sums = a.new_sums + row * new_cap;
  int* kept = a.kept + row * a.budget;
  const int n_new = min(n, a.budget);
  if (h == 0 && tid == 0) a.new_lens[b] = n_new;
  for (int j = n_new + tid; j < a.budget; j += kSelThreads) kept[j] = -1;
  for (int j = n_new + tid; j < new_cap; j += kSelThreads) new_sums[j] = 0.0f;
  if (n <= a.budget) {
    for (int j = tid; j < n; j += kSelThreads) {
      kept[j] = j;
      new_sums[j] = sums[j];
    }
    return;
  }
  // The candidates [lo, hi) and how many of them stay: 0 <= m < hi - lo.
  const int lo = a.n_sink, hi = n - a.n_recent, m = a.budget - a.n_sink - a.n_recent;
  const int per = (n + kSelThreads - 1) / kSelThreads;  // tokens per lane; a warp's are contiguous
  const int first = warp * 32 * per + lane;
  float held[E > 0 ? E : 1];
  if constexpr (E > 0) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int t = first + 32 * e;
      held[e] = e < per && t < n ? __ldg(sums + t) : 0.0f;
    }
  }
  auto value = [&](int e, int t) { return E > 0 ? held[E > 0 ? e : 0] : __ldg(sums + t); };

  // found: the digits of the m-th largest key found so far; need: how many of the keys that
  // share them are kept. Keys above are all kept.
  uint32_t found = 0, mask = 0;
  int need = m;
  if (m > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit_mask = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < (E > 0 ? E : per); ++e) {
        const int t = first + 32 * e;
        if (e < per && t >= lo && t < hi) {
          const uint32_t key = order_bits(value(e, t));
          if ((key & mask) == found) atomicAdd(&s_hist[(key >> shift) & digit_mask], 1);
        }
      }
      __syncthreads();
      // bins from the top: thread i has bins 2047 - 2 i and 2046 - 2 i
      const int c0 = s_hist[kBins - 1 - 2 * tid], c1 = s_hist[kBins - 2 - 2 * tid];
      int incl = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) s_warp[warp] = incl;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < kSelWarps; ++w) before += w < warp ? s_warp[w] : 0;
      const int above = before + incl - c0 - c1;  // keys in the bins above this thread's
      if (above < need && above + c0 >= need) {
        s_digit = kBins - 1 - 2 * tid;
        s_above = above;
      } else if (above + c0 < need && above + c0 + c1 >= need) {
        s_digit = kBins - 2 - 2 * tid;
        s_above = above + c0;
      }
      __syncthreads();
      found |= (uint32_t)s_digit << shift;
      mask |= digit_mask << shift;
      need -= s_above;
    }
  }
  // Kept: sinks, recents, keys above `found`, and the first `need` that equal it (m = 0: the
  // sinks and recents alone).
  int sure = 0, equal = 0;
#pragma unroll
  for (int e = 0; e < (E > 0 ? E : per); ++e) {
    const int t = first + 32 * e;
    const bool in = e < per && t < n;
    const bool cand = in && t >= lo && t < hi;
    const uint32_t key = cand ? order_bits(value(e, t)) : 0u;
    sure += __popc(__ballot_sync(0xffffffffu, in && (!cand || (m > 0 && key > found))));
    equal += __popc(__ballot_sync(0xffffffffu, cand && m > 0 && key == found));
  }
  if (lane == 0) {
    s_warp[warp] = sure;
    s_warp2[warp] = equal;
  }
  __syncthreads();
  int sure_before = 0, eq_before = 0;
  for (int w = 0; w < kSelWarps; ++w) {
    sure_before += w < warp ? s_warp[w] : 0;
    eq_before += w < warp ? s_warp2[w] : 0;
  }
  const uint32_t below = (1u << lane) - 1u;
#pragma unroll
  for (int e = 0; e < (E > 0 ? E : per); ++e) {
    const int t = first + 32 * e;
    const bool in = e < per && t < n;
    const bool cand = in && t >= lo && t < hi;
    const float x = in ? value(e, t) : 0.0f;
    const uint32_t key = cand ? order_bits(x) : 0u;
    const bool is_sure = in && (!cand || (m > 0 && key > found));
    const bool is_eq = cand && m > 0 && key == found;
    const unsigned ms = __ballot_sync(0xffffffffu, is_sure), me = __ballot_sync(0xffffffffu, is_eq);
    const int eq_rank = eq_before + __popc(me & below);
    const int j = sure_before + __popc(ms & below) + min(eq_rank, need);
    if (is_sure || (is_eq && eq_rank < need)) {
      kept[j] = t;
      new_sums[j] = x;
    }
    sure_before += __popc(ms);
    eq_before += __popc(me);
  }
}

constexpr int kGatherThreads = 256;
constexpr int kGatherRows = 4;  // rows of a lane group in flight, K and V each

// ROW: bytes of one K or V row.
template <int ROW>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const EvictArgs a) {
  constexpr int L = ROW / 16;                   // lanes per row
  constexpr int GROUPS = kGatherThreads / L;    // rows at a time
  const int h = blockIdx.y, b = blockIdx.z;
  const int l = threadIdx.x % L, group = threadIdx.x / L;
  const int P = a.page_size;
  const int32_t* kept = a.kept + ((int64_t)b * a.n_kv_heads + h) * a.budget;
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks;
  const int32_t* new_table = a.new_block_table + (int64_t)b * a.new_max_blocks;
  const uint32_t nan = a.dtype == PKV_F32 ? 0x7fc00000u : 0x7fc07fc0u;
  const int j0 = blockIdx.x * (GROUPS * kGatherRows) + group;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int src[kGatherRows];
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u) {
    const int j = j0 + u * GROUPS;
    src[u] = j < a.budget ? __ldcg(kept + j) : -1;
  }
  int64_t from[kGatherRows], to[kGatherRows];
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u) {
    from[u] = to[u] = -1;
    if (src[u] < 0) continue;
    const int j = j0 + u * GROUPS;
    const int p = __ldg(table + src[u] / P), q = __ldg(new_table + j / P);
    if (p >= 0 && p < a.num_pages) from[u] = (((int64_t)p * a.n_kv_heads + h) * P + src[u] % P) * ROW + 16 * l;
    if (q >= 0 && q < a.num_pages) to[u] = (((int64_t)q * a.n_kv_heads + h) * P + j % P) * ROW + 16 * l;
    if (l == 0 && (from[u] < 0 || to[u] < 0)) set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
  }
  uint4 k[kGatherRows], v[kGatherRows];
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u) {
    k[u] = v[u] = make_uint4(nan, nan, nan, nan);  // a bad source page: NaN rows
    if (from[u] >= 0) {
      k[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.k_pages) + from[u]);
      v[u] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.v_pages) + from[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kGatherRows; ++u) {
    if (to[u] >= 0) {
      *reinterpret_cast<uint4*>(static_cast<char*>(a.k_pages) + to[u]) = k[u];
      *reinterpret_cast<uint4*>(static_cast<char*>(a.v_pages) + to[u]) = v[u];
    }
  }
}

template <int ROW>
int launch_gather(const EvictArgs& a, cudaStream_t stream) {
  constexpr int TILE = kGatherThreads / (ROW / 16) * kGatherRows;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((a.budget + TILE - 1) / TILE), (unsigned)a.n_kv_heads, (unsigned)a.batch);
  cfg.blockDim = dim3(kGatherThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return check_launch(cudaLaunchKernelEx(&cfg, gather_kernel<ROW>, a));
}

}  // namespace

int launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t cap = (int64_t)a.max_blocks * a.page_size;
  const dim3 grid((unsigned)a.n_kv_heads, (unsigned)a.batch);
  if (cap <= 8 * kSelThreads)
    select_kernel<8><<<grid, kSelThreads, 0, stream>>>(a);
  else if (cap <= 32 * kSelThreads)
    select_kernel<32><<<grid, kSelThreads, 0, stream>>>(a);
  else
    select_kernel<0><<<grid, kSelThreads, 0, stream>>>(a);
  const int rc = check_launch(cudaGetLastError());
  if (rc != PKV_OK) return rc;
  switch (a.head_dim * (a.dtype == PKV_F32 ? 4 : 2)) {
    case 128: return launch_gather<128>(a, stream);
    case 256: return launch_gather<256>(a, stream);
    case 512: return launch_gather<512>(a, stream);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace pkv
