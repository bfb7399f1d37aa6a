// Tokens of ordinary pages (bf16 or fp32) into 4-bit pages, and back.
//
// To 4 bits, for 16 elements x of a token that share a scale, every step one rounding to nearest even in fp32:
//   y = x * (1 / head scale),  s = e4m3(max |y| * (1 / 6)) (at most 448),  code = e2m1(y * (1 / s)) (at most 6);
// s = 0 gives codes 0, and an x that is not finite (or a y that overflows) gives s = NaN, so that all 16 read as NaN.
// Back: x = (e2m1(code) * e4m3(s)) * head scale, the first product exact, then rounded to the page's type.
//
// Every element is read once and written once. A lane takes one group of two (packing) or four consecutive tokens of a 4-bit
// tile: their codes are 8 bytes each and their scales neighbours, moved at once although a token's are bytes at a
// distance; on the ordinary side a group is 32 or 64 bytes, moved 32 at a time, and eight lanes' groups are a row. The
// tiles' tokens are aligned to the 4-bit page; the ordinary side may start anywhere in its pages. Where there are many
// pages a CTA takes several heads of a page in turn, so that the tables are looked at once for all of them.
//
// Both are bound by memory, packing also by its loads in flight (54 % of the issue slots; 32 warps an SM, for which it spills 16
// bytes from bf16 and 28 from fp32, are 2 to 5 % faster from bf16 than the 28 of its 71 registers, 40 spill more: 44 us for 37.8). 41k
// tokens of 8 heads of 128 packed from bf16: 37.1 us, 215 MB, 5.8 TB/s; from fp32, whose rows are twice the bytes in flight and not
// asked for ahead: 60.9 us, 383 MB, 6.3 TB/s. 64k tokens back to bf16: 55.2 us, 344 MB, 6.2 TB/s; to fp32 96.0, 612 MB, 6.4. Head_dim 64 (half
// the bytes of 41k tokens): 21.7 and 33.8 us. A step's token of each of 64 sequences: 2.9 us, a launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;

// 32 bytes, aligned.
struct Eight {
  uint32_t w[8];
};
__device__ __forceinline__ Eight load32(const void* p) {
  Eight v;
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void store32(void* p, const Eight& v) {
  asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(v.w[0]), "r"(v.w[1]), "r"(v.w[2]), "r"(v.w[3]),
               "r"(v.w[4]), "r"(v.w[5]), "r"(v.w[6]), "r"(v.w[7]), "l"(p)
               : "memory");
}

// Pairs of fp32 numbers in one register pair.
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) { return pair_of(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 split(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 16 consecutive elements of T as eight pairs.
template <typename T>
struct Group16;
template <>
struct Group16<float> {
  Eight v[2];
  __device__ __forceinline__ void load(const char* p) { v[0] = load32(p), v[1] = load32(p + 32); }
  __device__ __forceinline__ void get(uint64_t (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = pair_of(v[i / 4].w[2 * i % 8], v[i / 4].w[2 * i % 8 + 1]);
  }
  static __device__ __forceinline__ void store(char* p, const uint64_t (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      Eight v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = split(x[4 * k + i]);
        v.w[2 * i] = __float_as_uint(f.x), v.w[2 * i + 1] = __float_as_uint(f.y);
      }
      store32(p + 32 * k, v);
    }
  }
};
template <>
struct Group16<__nv_bfloat16> {
  Eight v;
  __device__ __forceinline__ void load(const char* p) { v = load32(p); }
  __device__ __forceinline__ void get(uint64_t (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = pair_of(v.w[i] << 16, v.w[i] & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(char* p, const uint64_t (&x)[8]) {
    Eight v;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = split(x[i]);
      const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
      v.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    store32(p, v);
  }
};

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Eight codes of four pairs, the first in the lowest four bits.
__device__ __forceinline__ uint32_t to_codes(const uint64_t* z) {
  const float2 a = split(z[0]), b = split(z[1]), c = split(z[2]), d = split(z[3]);
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return r;
}

// Codes and scale of 16 elements. The largest |y| is the largest |x| times |inv_head|: a product's rounding keeps
// the order.
__device__ __forceinline__ uint2 quantise(uint64_t (&x)[8], float inv_head, uint32_t& scale) {
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = split(x[i]);
    top = max_abs_nan(top, f.x, f.y);
  }
  top = fabsf(top * inv_head);
  scale = 0x7fu;  // NaN
  if (!(top < INFINITY)) return make_uint2(0, 0);
  unsigned short pair;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.0f), "f"(top * (1.0f / 6.0f)));
  scale = pair & 0xffu;
  if (scale == 0) return make_uint2(0, 0);
  const uint32_t h = e4m3_pair_to_h2(scale);
  const float inv = __frcp_rn(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
  const uint64_t head2 = pair_of(inv_head, inv_head), inv2 = pair_of(inv, inv);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = mul2(mul2(x[i], head2), inv2);
  return make_uint2(to_codes(x), to_codes(x + 4));
}

// What a CTA works on: tokens [lo, hi) of its sequence's 4-bit block.
struct Block {
  int b, block, lo, hi, page, first, row_first;
  bool any;
};

__device__ __forceinline__ Block block_of(const Fp4CopyArgs& a, int per_block) {
  constexpr int P = 16;
  Block k;
  k.b = blockIdx.y;
  const int at = blockIdx.x / per_block;
  k.first = a.first ? __ldg(a.first + k.b) : 0;
  k.row_first = a.row_first ? __ldg(a.row_first + k.b) : 0;
  const int n = __ldg(a.counts + k.b);
  k.any = false;
  if (n < 0 || n > a.max_count || k.first < 0 || k.row_first < 0 || (int64_t)k.first + n > (int64_t)a.max_blocks * P ||
      (int64_t)k.row_first + n > (int64_t)a.row_blocks * P) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
    return k;
  }
  const int64_t block = (int64_t)(k.first / P) + at;  // (past the table only where there is no token)
  const int64_t lo = block * P > k.first ? block * P : k.first, end = (int64_t)k.first + n;
  const int64_t hi = end < (block + 1) * P ? end : (block + 1) * P;
  if (lo >= hi) return k;
  k.block = (int)block, k.lo = (int)lo, k.hi = (int)hi;
  k.page = __ldg(a.block_table + (int64_t)k.b * a.max_blocks + k.block);  // (looked at with the other table's)
  k.any = true;
  return k;
}

// Consecutive tokens of a lane. Packing, two, whose next rows are on their way meanwhile, are 37 us where four are 40 for 41k tokens of
// 8 heads.
constexpr int rows_of_lane(bool pack) { return pack ? 2 : 4; }

template <typename T, int D, bool PACK>
__global__ void __launch_bounds__(kThreads, PACK ? 8 : 10) fp4_copy_kernel(const Fp4CopyArgs a, int per_block, int turns) {
  using Tile = Fp4Tile<D>;
  constexpr int R = rows_of_lane(PACK), kLanes = Tile::kGroups * Tile::kTokens / R;  // lanes of a tile
  constexpr int kTiles = kThreads / kLanes;  // tiles of a CTA at a time: K and V of kTiles / 2 heads
  static_assert(kTiles % 2 == 0, "a lane stays with K or V from turn to turn");
  static_assert(R == (PACK ? 2 : 4), "its scales are one aligned access, a half-word or a word");
  wait_for_stream();  // (the next kernel is not let in early: a decode's CTAs would be placed unevenly, 17.2 us for both, not 14.0)
  const Block k = block_of(a, per_block);
  if (!k.any) return;
  const int unit = (blockIdx.x % per_block) * kTiles * turns + threadIdx.x / kLanes;  // (head, K or V)
  const bool is_v = unit & 1;
  const int l = threadIdx.x % kLanes, grp = l % Tile::kGroups, part = l / Tile::kGroups;
  const float* scales = is_v ? a.v_scale : a.k_scale;
  const int32_t* row_table = a.row_table + (int64_t)k.b * a.row_blocks;
  // where the tokens of head 0 are on the ordinary side; -1: not there
  int64_t at[R];
  int pages[R];
  const int t0 = k.block * 16 + R * part;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int t = t0 + i;
    pages[i] = t >= k.lo && t < k.hi ? __ldg(row_table + (t - k.first + k.row_first) / 16) : 0;
  }
  const bool bad_page = k.page < 0 || k.page >= a.num_pages;
  if (bad_page) {
    if (threadIdx.x == 0) set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
    if (PACK) return;  // (read back, its tokens are NaN)
  }
  constexpr int64_t kRowHead = (int64_t)16 * D * sizeof(T);  // bytes of a head of an ordinary page
#pragma unroll
  for (int i = 0; i < R; ++i) {
    at[i] = -1;
    if (t0 + i < k.lo || t0 + i >= k.hi) continue;
    if (pages[i] >= 0 && pages[i] < a.row_pages)
      at[i] = pages[i] * (a.n_kv_heads * kRowHead) + (((t0 + i - k.first + k.row_first) % 16) * D + grp * Tile::kGroup) * (int)sizeof(T);
    else
      set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
  }
  char* tiles = static_cast<char*>(is_v ? a.v_tiles : a.k_tiles) + (int64_t)k.page * a.n_kv_heads * Tile::kBytes;
  const int codes_at = R * part * Tile::kRow + 8 * grp, scales_at = Tile::kCodes + grp * Tile::kTokens + R * part;
  char* row_pool = static_cast<char*>(is_v ? a.v_rows : a.k_rows);
  constexpr bool kAhead = PACK && sizeof(T) == 2;  // the next turn's rows are asked for before this one's are worked on
  Group16<T> raw[R];
  auto load = [&](Group16<T>(&to)[R], int head) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (at[i] >= 0) to[i].load(row_pool + head * kRowHead + at[i]);
  };
  if (kAhead && (unit >> 1) < a.n_kv_heads) load(raw, unit >> 1);
  for (int turn = 0; turn < turns; ++turn) {
    const int head = (unit + turn * kTiles) >> 1;
    if (head >= a.n_kv_heads) return;
    const float hs = scales ? __ldg(scales + head) : 1.0f;
    char* rows = row_pool + head * kRowHead;
    char* codes = tiles + head * Tile::kBytes + codes_at;
    char* lane_scales = tiles + head * Tile::kBytes + scales_at;
    if constexpr (PACK) {
      Group16<T> now[R];
      if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < R; ++i) now[i] = raw[i];
        if (turn + 1 < turns && head + kTiles / 2 < a.n_kv_heads) load(raw, head + kTiles / 2);
      } else {
        load(now, head);
      }
      const float inv_head = __frcp_rn(hs);
      uint32_t both = 0;
      bool all = true;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (at[i] < 0) {
          all = false;
          continue;
        }
        uint64_t x[8];
        now[i].get(x);
        uint32_t s;
        *reinterpret_cast<uint2*>(codes + i * Tile::kRow) = quantise(x, inv_head, s);
        both |= s << (8 * i);
      }
      if (all) {
        *reinterpret_cast<uint16_t*>(lane_scales) = (uint16_t)both;
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (at[i] >= 0) lane_scales[i] = (char)(both >> (8 * i));
      }
    } else {
      uint32_t s4 = 0x7f7f7f7fu;  // a bad page: NaN
      uint2 c[R] = {};
      if (!bad_page) {
        s4 = __ldg(reinterpret_cast<const uint32_t*>(lane_scales));
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (at[i] >= 0) c[i] = __ldg(reinterpret_cast<const uint2*>(codes + i * Tile::kRow));
      }
      const uint64_t head2 = pair_of(hs, hs);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (at[i] < 0) continue;
        const uint32_t one = (s4 >> (8 * i)) & 0xffu, s = e4m3_pair_to_h2(one | one << 8);
        const uint32_t h[8] = {e2m1x2_to_h2<0>(c[i].x), e2m1x2_to_h2<1>(c[i].x), e2m1x2_to_h2<2>(c[i].x), e2m1x2_to_h2<3>(c[i].x),
                               e2m1x2_to_h2<0>(c[i].y), e2m1x2_to_h2<1>(c[i].y), e2m1x2_to_h2<2>(c[i].y), e2m1x2_to_h2<3>(c[i].y)};
        uint64_t x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t p = mul_h2(h[e], s);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p));
          x[e] = mul2(pair_of(f.x, f.y), head2);
        }
        Group16<T>::store(rows + at[i], x);
      }
    }
  }
}

template <typename T, int D>
int launch_t(const Fp4CopyArgs& a, cudaStream_t stream) {
  const int kTiles = kThreads / (Fp4Tile<D>::kGroups * 16 / rows_of_lane(a.to_fp4));
  // 4-bit blocks that max_count tokens can touch, wherever the first one lies in its block
  const int64_t blocks = ((int64_t)a.max_count + 15) / 16 + (a.first ? 1 : 0);
  const int64_t ctas = (2 * (int64_t)a.n_kv_heads + kTiles - 1) / kTiles;
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  // (packing, 8 turns are 2 % slower than 4 and 2 are 15 %; reading back, 2 are 3 % faster than 4)
  const int64_t most = a.to_fp4 ? 4 : 2;
  const int turns = blocks * ctas * a.batch <= 16 * sms ? 1 : (int)(ctas < most ? ctas : most);
  const int per_block = (int)((ctas + turns - 1) / turns);
  if (blocks * per_block > 0x7fffffffLL) return PKV_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(blocks * per_block), (unsigned)a.batch);
  return check_launch(a.to_fp4
                          ? launch_overlapped(fp4_copy_kernel<T, D, true>, grid, kThreads, 0, stream, 1, a, per_block, turns)
                          : launch_overlapped(fp4_copy_kernel<T, D, false>, grid, kThreads, 0, stream, 1, a, per_block, turns));
}

}  // namespace

int launch_fp4_copy(const Fp4CopyArgs& a, cudaStream_t stream) {
  if (a.dtype == PKV_F32) {
    if (a.head_dim == 64) return launch_t<float, 64>(a, stream);
    if (a.head_dim == 128) return launch_t<float, 128>(a, stream);
  } else {
    if (a.head_dim == 64) return launch_t<__nv_bfloat16, 64>(a, stream);
    if (a.head_dim == 128) return launch_t<__nv_bfloat16, 128>(a, stream);
  }
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace pkv
