// Eviction from the paged cache by accumulated attention weight.
//
// Of a sequence's n tokens a KV head keeps min(n, budget): the first n_sink, the last n_recent
// and, of those between, the ones with the largest sums (equal sums: the lower index), in their
// order. The kept rows of K and V are gathered into the pages of a new table, so shared source
// pages stay whole and no row is overwritten before it is read.
//
// Two kernels. The selection is one CTA per (sequence, KV head). A token becomes a 32-bit key,
// once, in shared memory: the sums' order-preserving bits, above them NaN, above all the sinks
// and recents, so that what is kept is the `budget` largest keys. The last of them is searched
// for by passes of 8 bits, each a histogram of the keys that share the digits found so far,
// until a pass needs a whole bin or leaves few keys, which are then compared with one another
// (rows of 20 tokens: 6.1 to 5.0 us a call; rows of 16-32k: 1.5 us of 103). Sums cluster (many are
// equal, most share an exponent) and atomics on one address take turns, so a bin has 8 counters, by
// lane. Then each warp, which holds a contiguous run of tokens, counts what it keeps, one scan over
// the warps places the runs, and the kept indices and sums are written in order. Rows past
// kSmemTokens are read again in each pass.
//
// What bounds the selection: the atomics and the emission of long rows (20 us for 16 x 8 rows of
// 16-32k tokens), for short ones the instructions that every warp runs for a few tokens each, so
// those get 256 threads (5.5 us for rows of 2.3k tokens, 7 with 1024). The gather is one lane group per
// kept row, K and V of four rows in flight, and runs at the copy bandwidth: 82 us for 554 MB.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kDigits = 256;
constexpr int kCopies = 8;                // counters of a bin
constexpr int kGroup = 4;                 // consecutive tokens of a lane
constexpr int kShortTokens = 4096;        // rows up to this length: 256 threads, which hold the keys in registers
constexpr int kFew = 128;                 // candidates that are ranked directly
constexpr int kSmemTokens = 13 * 4096;    // 208 KiB, beside the 8 KiB of counters

constexpr uint32_t kAlways = 0xffffffffu;  // sinks and recents

// Bits that order as the floats do, all above 0; both zeros are equal, NaN is above every number.
__device__ __forceinline__ uint32_t order_bits(float x) {
  if (x != x) return kAlways - 1;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The float of order_bits (a zero comes back positive, a NaN as the canonical one).
__device__ __forceinline__ float from_order_bits(uint32_t k) {
  return __uint_as_float(k == kAlways - 1 ? 0x7fffffffu : (k & 0x80000000u) ? k ^ 0x80000000u : ~k);
}

// Counts in shared memory where `on`, without a branch around the atomic.
__device__ __forceinline__ void count_if(bool on, uint32_t addr) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(addr), "r"((uint32_t)on)
      : "memory");
}

template <bool SMEM, int kSelThreads>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictArgs a) {
  constexpr int kSelWarps = kSelThreads / 32, kWave = kGroup * kSelThreads;
  constexpr int kPerBin = kSelThreads / kDigits;  // threads that add up a bin's counters
  __shared__ __align__(16) int s_hist[kDigits * kCopies];
  __shared__ int s_warp[kSelWarps], s_warp2[kSelWarps];
  __shared__ int s_digit, s_above, s_count;
  __shared__ __align__(16) uint32_t s_few[kFew];
  __shared__ int s_n_few, s_larger;
  __shared__ uint32_t s_last;
  extern __shared__ __align__(16) uint32_t s_row[];
  // A short row's keys, kWaves groups of four a thread
  constexpr bool REG = SMEM && kSelThreads == 256;
  constexpr int kWaves = REG ? kShortTokens / kWave : 1;
  const int b = blockIdx.y, h = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_stream();
  const int cap = a.max_blocks * a.page_size, new_cap = a.new_max_blocks * a.page_size;
  const int64_t row = (int64_t)b * a.n_kv_heads + h;
  const float* sums = a.sums + row * cap;
  int n = __ldg(a.kv_lens + b);
  // The first wave of sums is asked for beside the length (it lies inside the row: rows are
  // 16-byte aligned multiples of 16 tokens).
  auto fetch = [&](int t) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(s_row + t)), "l"(sums + t) : "memory");
  };
  if (SMEM && kGroup * tid < cap) fetch(kGroup * tid);
  for (int i = tid; i < kDigits * kCopies; i += kSelThreads) s_hist[i] = 0;
  if (n < 0 || n > cap) {
    if (tid == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
    n = 0;
  }
  float* new_sums = a.new_sums + row * new_cap;
  int* kept = a.kept + row * a.budget;
  const int n_new = min(n, a.budget);
  if (h == 0 && tid == 0) a.new_lens[b] = n_new;
  for (int j = n_new + tid; j < a.budget; j += kSelThreads) kept[j] = -1;
  for (int j = n_new + tid; j < new_cap; j += kSelThreads) new_sums[j] = 0.0f;
  if (n <= a.budget) {
    for (int j = tid; j < n; j += kSelThreads) {
      kept[j] = j;
      new_sums[j] = __ldg(sums + j);
    }
    if (SMEM) asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  const int lo = a.n_sink, hi = n - a.n_recent;  // [lo, hi): the tokens that are ranked by their sums
  auto key_of = [&](int t, float x) { return t >= n ? 0u : t < lo || t >= hi ? kAlways : order_bits(x); };
  auto keys_of = [&](int t, const float4& x) {
    return make_uint4(key_of(t, x.x), key_of(t + 1, x.y), key_of(t + 2, x.z), key_of(t + 3, x.w));
  };
  const int waves = (n + kWave - 1) / kWave;
  if constexpr (SMEM) {
    for (int t = kWave + kGroup * tid; t < n; t += kWave) fetch(t);
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  // A warp's tokens are contiguous: group e of lane l is tokens first + 128 e .. + 3.
  const int first = warp * (32 * kGroup) * waves + kGroup * lane;
  auto sums_at = [&](int t) {
    if (t >= n) return make_float4(0.f, 0.f, 0.f, 0.f);
    return SMEM ? *reinterpret_cast<const float4*>(s_row + t) : __ldg(reinterpret_cast<const float4*>(sums + t));
  };
  uint4 reg[kWaves];
  auto keys = [&](int e, bool raw) {
    const int t = first + 32 * kGroup * e;
    if (SMEM && !raw) return *reinterpret_cast<const uint4*>(s_row + t);
    const uint4 k = keys_of(t, sums_at(t));
    if (SMEM) *reinterpret_cast<uint4*>(s_row + t) = k;  // the first pass turns the sums into keys
    return k;
  };
  // f(first token, its four keys) for each group of the thread
  auto each = [&](bool raw, auto&& f) {
    if constexpr (REG) {
#pragma unroll
      for (int e = 0; e < kWaves; ++e)
        if (e < waves) f(first + 32 * kGroup * e, reg[e]);
    } else {
#pragma unroll 2
      for (int e = 0; e < waves; ++e) f(first + 32 * kGroup * e, keys(e, raw));
    }
  };

  // found: the digits of the budget-th largest key found so far (those in mask); need: how many
  // of the keys that share them are kept. Keys above are all kept.
  uint32_t found = 0, mask = 0;
  int need = a.budget;
  const uint32_t column = smem_u32(s_hist) + 4 * (lane & (kCopies - 1));
  if (tid == 0) s_n_few = 0, s_larger = 0, s_last = ~0u;
  __syncthreads();
  if constexpr (REG) {
#pragma unroll
    for (int e = 0; e < kWaves; ++e)
      if (e < waves) reg[e] = keys_of(first + 32 * kGroup * e, sums_at(first + 32 * kGroup * e));
  }
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    each(shift == 24, [&](int, const uint4& k4) {
      const uint32_t k[kGroup] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        count_if((k[i] & mask) == found, column + ((k[i] >> shift) & 255u) * (4 * kCopies));
    });
    __syncthreads();
    // kPerBin threads add up a bin's counters (and clear them for the next pass); `above`: the
    // keys in higher bins, first within the warp, then those of the warps above it
    const int bin = tid / kPerBin;
    int c = 0;
    {
      int2* p = reinterpret_cast<int2*>(s_hist) + tid * (kCopies / kPerBin / 2);
#pragma unroll
      for (int i = 0; i < kCopies / kPerBin / 2; ++i) {
        const int2 x = p[i];
        p[i] = make_int2(0, 0);
        c += x.x + x.y;
      }
    }
#pragma unroll
    for (int o = 1; o < kPerBin; o <<= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    int above = c;
#pragma unroll
    for (int o = kPerBin; o < 32; o <<= 1) {
      const int y = __shfl_down_sync(0xffffffffu, above, o);
      if (lane + o < 32) above += y;
    }
    if (lane == 0) s_warp[warp] = above;
    above -= c;
    __syncthreads();
    above += __reduce_add_sync(0xffffffffu, lane > warp && lane < kSelWarps ? s_warp[lane] : 0);
    if (above < need && above + c >= need) {  // one bin in all
      s_digit = bin;
      s_above = above;
      s_count = c;
    }
    __syncthreads();
    found |= (uint32_t)s_digit << shift;
    mask |= 255u << shift;
    need -= s_above;
    if (s_count == need) break;  // the whole bin is kept: its keys need no more digits
    if (shift > 0 && s_count <= kFew) {
      // Few share the digits: each is compared with all of them, and the need-th largest gives the
      // remaining digits at once. (Their order in the list does not matter.)
      each(false, [&](int, const uint4& k4) {
        const uint32_t k[kGroup] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
          if ((k[i] & mask) == found) s_few[atomicAdd(&s_n_few, 1)] = k[i];
      });
      const int few = s_count;
      if (tid >= few && tid < kFew) s_few[tid] = 0;  // (0 is below every key)
      __syncthreads();
      if (warp * 32 < few) {
        const uint32_t mine = tid < few ? s_few[tid] : 0;
        int larger = 0;
#pragma unroll 4
        for (int i = 0; i < few; i += 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(s_few + i);
          larger += (x.x > mine) + (x.y > mine) + (x.z > mine) + (x.w > mine);
        }
        // the keys with fewer than `need` above them are kept: the least of them is the last kept
        const bool kept_key = larger < need;
        const uint32_t last = __reduce_min_sync(0xffffffffu, kept_key ? mine : ~0u);
        const int most = __reduce_max_sync(0xffffffffu, kept_key ? larger : 0);
        if (lane == 0) {
          atomicMin(&s_last, last);
          atomicMax(&s_larger, most);
        }
      }
      __syncthreads();
      found = s_last;
      mask = ~0u;
      need -= s_larger;
      break;
    }
  }
  // Kept: keys whose found digits are above, and the first `need` that share them.
  int sure = 0, equal = 0;
  each(false, [&](int, const uint4& k4) {
    const uint32_t k[kGroup] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      sure += (k[i] & mask) > found;
      equal += (k[i] & mask) == found;
    }
  });
  sure = __reduce_add_sync(0xffffffffu, sure);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    s_warp[warp] = sure;
    s_warp2[warp] = equal;
  }
  __syncthreads();
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0);
  int eq_left = need - __reduce_add_sync(0xffffffffu, lane < warp ? s_warp2[lane] : 0);  // kept of this warp's equal keys
  at += need - max(eq_left, 0);  // where the warp's first kept token goes
  // Only the warp in which the equal keys run out has to count them; before it all are kept.
  const bool count_equal = eq_left > 0 && eq_left < equal;
  // nothing is above kAlways, and this warp has no equal key left to keep
  const bool any = eq_left > 0 || found != kAlways;
  const uint32_t least = eq_left > 0 ? found : found + 1;
  const uint32_t below = (1u << lane) - 1u;
  if (any) each(false, [&](int t, const uint4& k4) {
    const uint32_t full[kGroup] = {k4.x, k4.y, k4.z, k4.w};
    const uint32_t k[kGroup] = {k4.x & mask, k4.y & mask, k4.z & mask, k4.w & mask};
    bool keep[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) keep[i] = k[i] >= least;
    if (count_equal) {
      unsigned m[kGroup];
      int rank = 0, all = 0;
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        m[i] = __ballot_sync(0xffffffffu, k[i] == found);
        rank += __popc(m[i] & below);
        all += __popc(m[i]);
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        keep[i] = k[i] > found || (k[i] == found && rank < eq_left);
        rank += k[i] == found;
      }
      eq_left -= all;
    }
    int j = at;
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const unsigned m = __ballot_sync(0xffffffffu, keep[i]);
      j += __popc(m & below);
      at += __popc(m);
    }
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      if (keep[i]) kept[j] = t + i;
      if (keep[i] && full[i] != kAlways) new_sums[j] = from_order_bits(full[i]);
      j += keep[i];
    }
  });
  // sinks and recents keep their order around the others, so their places are known
  for (int j = tid; j < a.n_sink + a.n_recent; j += kSelThreads) {
    const int back = j < a.n_sink ? 0 : j - a.n_sink - a.n_recent;  // < 0: from the end
    const int to = back < 0 ? a.budget + back : j;
    new_sums[to] = __ldg(sums + (back < 0 ? n + back : j));
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
  wait_for_stream();
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
  const dim3 grid((unsigned)((a.budget + TILE - 1) / TILE), (unsigned)a.n_kv_heads, (unsigned)a.batch);
  return check_launch(launch_overlapped(gather_kernel<ROW>, grid, kGatherThreads, 0, stream, 1, a));
}

}  // namespace

int launch_evict(const EvictArgs& a, cudaStream_t stream) {
  const int64_t cap = (int64_t)a.max_blocks * a.page_size;
  const dim3 grid((unsigned)a.n_kv_heads, (unsigned)a.batch);
  int rc;
  if (cap <= kShortTokens) {
    rc = check_launch(
        launch_overlapped(select_kernel<true, 256>, grid, 256, (size_t)((cap + 1023) / 1024) * 4096, stream, 1, a));
  } else if (cap <= kSmemTokens) {
    static FuncConfigured configured;
    if (!configured.ensure(reinterpret_cast<const void*>(select_kernel<true, 1024>), kSmemTokens * 4))
      return PKV_ERR_LAUNCH;
    rc = check_launch(
        launch_overlapped(select_kernel<true, 1024>, grid, 1024, (size_t)((cap + 4095) / 4096) * 16384, stream, 1, a));
  } else {
    rc = check_launch(launch_overlapped(select_kernel<false, 1024>, grid, 1024, 0, stream, 1, a));
  }
  if (rc != PKV_OK) return rc;
  switch (a.head_dim * (a.dtype == PKV_F32 ? 4 : 2)) {
    case 128: return launch_gather<128>(a, stream);
    case 256: return launch_gather<256>(a, stream);
    case 512: return launch_gather<512>(a, stream);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace pkv
