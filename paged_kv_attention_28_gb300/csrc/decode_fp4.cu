// Paged single-token decode over 4-bit pages (the tile of fp4.cuh).
//
// One unit of work is (split, KV head, sequence), one CTA of four warps, which take the split's pages in turns of two. A page is
// 18 head_dim bytes of K and V, a quarter of bf16's, so at the memory's rate an SM gets a new page every 100 clocks
// (head_dim 128) and what counts is how few instructions a code costs. Both products run on mma.sync m16n8k16 (f16 in,
// fp32 sums) with the cache as the A operand, straight from the codes: a thread's codes become f16 pairs in its own
// registers (one conversion and one multiplication with the scale for two codes) in the places where the product
// wants them, with no trip through shared memory, which would carry four times the bytes. tcgen05 would need that trip
// (its A operand lies in shared or tensor memory): 88 bytes written and as many read a clock of the 128 an SM
// moves. The products themselves take a third of mma.sync's rate.
//
//   S [16 tokens][8 heads] = K [16 x D] Q^T: the sum over D may be taken in any order, so a thread reads D / 4
//     consecutive elements of its two rows (16 bytes at D = 128) and the query's operand has the same order.
//   P = 2^(S - reference), rounded to f16; an 8 x 8 transposition turns it into the second product's operand.
//   O^T [D][8 heads] += V^T [D x 16 tokens] P: a thread takes D / 8 consecutive elements of four tokens. A pair of
//     tokens has to share a register: the codes of two tokens are interleaved four bits at a time (two instructions
//     for 16 codes) before they are converted.
// Heads past the group's are zero columns: 1 to 8 query heads cost the same.
//
// The query is scaled by a power of two to at most 2^15 per head and held in f16: exact for bf16, but for elements 2^24
// below the head's largest. Softmax statistics are fp32; the reference value lies 2^7 below a maximum on the way, and is
// moved only when a logit passes that maximum by more than 2^8 (a weight is then at most 2^15), which most pages do not.
//
// Each warp has a ring of its own in shared memory, of steps of two pages, filled by 16-byte asynchronous copies, so that
// warps never wait for one another; chunks are placed so that neither product's reads meet in a bank. Two pages a step
// halve what is not work on codes: waits, addresses, the look at the reference value.
//
// A page is 260 instructions and 102 clocks of an SM in the middle of a long split, which is 6.4 TB/s. 151 MB (4 x 32768
// tokens of 8 heads) are 30.6 to 31 us: 1.5 until the first copies are issued, 23.5 of steps, 0.8 for the warps' states, 1.4
// in which only some of an SM's CTAs are left, and the merge of the splits. 170 MB of unequal rows (16 x 512-4096 of 32
// heads) are 37.6, at 56 % of the issue slots while an SM works, 86 % of the time (128 registers a thread at D = 128; ordered by
// length, 4 bytes of them are spilled). A cluster that puts up to 8 splits' states together in
// shared memory, with no second launch, takes 0.2 to 0.7 us less where there are few CTAs, but its CTAs start
// together: the second of these batches was 51 us with it and 41 without. So splits always meet in the merge.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPage = 16;
constexpr int kCols = 8;          // columns of the products: query heads of a group, padded with zeros
constexpr int kGroup = 128;        // (sequence, split) pairs that are put in order, one a thread
// A reference value lies kBelow (in powers of two) below the largest logit that it was taken from, which a later one may
// pass by kHeadroom: a weight is at most 2^15, within f16, and keeps all its bits down to 2^-21 of that logit's (below it, it is
// off by 2^-32 of that logit's at most). Logits of kLarge and more, whose own steps come near the bit that is left, do without
// kBelow; the headroom suffices up to 2^24. Weights in two f16 numbers, both multiplied with V, would be right to 2^-22: 37.7 to 42.6
// us for 16 x 512-4096 tokens of 32 heads, 30.9 to 34.3 for 4 x 32768 of 8, and the same error of the bf16 outputs
// against exact ones to a hundredth (1.70e-3, 1.69e-3).
constexpr float kBelow = 7.0f, kHeadroom = 8.0f, kLarge = 1048576.0f;

template <int D>
struct Cfg {
  using Tile = Fp4Tile<D>;
  static constexpr int kWarps = 4;
  static constexpr int kSteps = D / 16;            // products of 16 along D (K), tiles of 16 along D (V)
  static constexpr int kStages = D == 128 ? 2 : 4;  // steps of a warp's ring
  static constexpr int kCtas = 4;                   // CTAs an SM holds (D = 64: five, with 96 registers, are 4 to 17 % slower)
  static constexpr int kPair = 2 * Tile::kBytes;    // K and V of a page
  static constexpr int kSlot = 2 * kPair;           // of the two pages of a step
  static constexpr int kSmem = kWarps * kStages * kSlot;
  static constexpr int kRow = D + 4;                // floats of a head's sums, as the warps put them together
  static_assert(kWarps * kCols * (kRow + 2) * 4 <= kSmem, "the warps' results fit in their rings");
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
// N words from shared memory, 4 N bytes aligned.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4);
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a) : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(a) : "memory");
  else
    w[0] = lds32(a);
}

// Where 16-byte chunk c of token r's codes lies in a tile in shared memory. Lines of 128 bytes hold 2 (D = 128) or 4
// tokens. A quarter-warp of the K product reads tokens 4 a and 4 a + 1 whole (D = 64: of two a), a half-warp of the V
// product one or two chunks of tokens 4 a + i of every a: the exclusive-or by a's two bits, swapped and doubled, sends
// both to different banks.
template <int D>
__device__ __forceinline__ int chunk_at(int r, int c) {
  constexpr int kPerRow = D / 32, kRows = 8 / kPerRow;
  const int a = (r >> 2) & 3, key = ((a & 1) << 2) | (a & 2);
  return (r / kRows) * 128 + ((((r % kRows) * kPerRow + c) ^ key) << 4);
}

// The rows of a group that has no keys (o = 0, l = -inf) or failed (NaN).
template <int D>
__device__ void write_rows(const DecodeArgs& a, int b, int head, float o, float l) {
  const int G = a.n_qo_heads / a.n_kv_heads;
  const int64_t row = (int64_t)b * a.n_qo_heads + (int64_t)head * G;
  for (int i = threadIdx.x; i < G * D; i += blockDim.x) static_cast<__nv_bfloat16*>(a.out)[row * D + i] = __float2bfloat16_rn(o);
  if (a.lse && threadIdx.x < G) a.lse[row + threadIdx.x] = l;
}

// A KV head's queries in f16, heads past the group's zero, and what takes a product to a logit in powers of two.
template <int D>
struct Queries {
  __half rows[kCols][D];
  float scale[kCols];
};

// 16 threads a head, the CTA's 128 for all; `raw` is the thread's 16 or 8 bytes of its head (zero past the group's).
template <int D>
__device__ __forceinline__ void convert_queries(const DecodeArgs& a, const uint32_t (&raw)[D / 32], float k_scale, Queries<D>& to) {
  const int h = threadIdx.x >> 4, part = threadIdx.x & 15;
  float x[D / 16], mx = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) x[2 * i] = __uint_as_float(raw[i] << 16), x[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) mx = fmaxf(mx, fabsf(x[i]));
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
  const int ex = (int)((__float_as_uint(mx) >> 23) & 0xffu) - 127;
  int sh = mx > 0.0f ? 14 - ex : 0;
  sh = sh > 126 ? 126 : (sh < -126 ? -126 : sh);
  float up = __uint_as_float((uint32_t)(127 + sh) << 23);
  if ((a.scale < 0.0f) != (k_scale < 0.0f)) up = -up;  // (logits are compared before they are scaled)
  uint32_t w[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) w[i] = pack_h2(x[2 * i] * up, x[2 * i + 1] * up);
  uint32_t* row = reinterpret_cast<uint32_t*>(to.rows[h] + part * (D / 16));
  if constexpr (D == 128)
    *reinterpret_cast<uint4*>(row) = make_uint4(w[0], w[1], w[2], w[3]);
  else
    *reinterpret_cast<uint2*>(row) = make_uint2(w[0], w[1]);
  // Not 0, so that a masked product stays -inf as a logit; products are below 2^35, so what 2^-126 makes of them is 0.
  // The scale's power of two goes apart, in two factors: its product with the head's scale may be no fp32 number, or one of
  // few bits, where the query makes an ordinary logit of it.
  const int up_by = a.scale_exponent - sh, half = up_by >> 1;  // (-250 .. 243)
  auto power = [](int e) { return __uint_as_float((uint32_t)(127 + e) << 23); };
  const float unscale = a.scale_fraction * fabsf(k_scale) * power(half) * power(up_by - half);
  if (part == 0) to.scale[h] = unscale < 1.17549435e-38f ? 1.17549435e-38f : unscale;
}

// One warp's attention of a KV head's queries over pages, two a step, from its ring in shared memory.
template <int D>
struct Attention {
  using C = Cfg<D>;
  using Tile = Fp4Tile<D>;
  static constexpr int KS = C::kSteps;
  static constexpr int KW = D / 32, VW = D / 64;     // words of a thread's codes, of a row of K and of a token of V
  static constexpr int KG = KS / 4;                  // groups of a thread's K row
  static constexpr int kRounds = Tile::kCodes / 512;  // of 32 chunks of a tile's codes

  const DecodeArgs& a;
  const int G, lane, g, t;
  const uint32_t ring;
  // copies
  const uint32_t page_bytes;
  const char *k_src, *v_src, *s_src;
  uint32_t code_at[kRounds], scale_at;
  // A thread's rows of K are tokens tok and tok + 2, so that the second product's pairs are tokens 4 t .. 4 t + 3.
  const int tok;
  uint32_t k_at[2], v_at[4];
  const uint32_t ks_at, ks_pick, vs_at;
  // the group's queries, and what takes a product to a logit in powers of two, heads 2 t and 2 t + 1
  uint32_t q[KS][2];
  float qs0, qs1;
  // the reference values (0 while there is none), the product above which they move (-inf while there is none), the sums
  float ref0, ref1, top0, top1, l0, l1;
  float o[KS][4];

  __device__ __forceinline__ Attention(const DecodeArgs& args, uint32_t ring_at)
      : a(args), G(args.n_qo_heads / args.n_kv_heads), lane(threadIdx.x & 31), g((threadIdx.x & 31) >> 2), t(threadIdx.x & 3),
        ring(ring_at), page_bytes((uint32_t)args.n_kv_heads * Tile::kBytes), tok(4 * (g >> 1) + (g & 1)),
        ks_at(ring_at + Tile::kCodes + t * KG * 16 + 4 * (g >> 1)), ks_pick((g & 1) ? 0x31 : 0x20),
        vs_at(ring_at + Tile::kBytes + Tile::kCodes + (g * KS / 8) * 16 + 4 * t) {
    k_src = static_cast<const char*>(a.k_pages) + 16 * lane;
    v_src = static_cast<const char*>(a.v_pages) + 16 * lane;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int c = lane + 32 * i;
      code_at[i] = ring + chunk_at<D>(c / (D / 32), c % (D / 32));
    }
    // 16 bytes of scales a group, K's in the first lanes and V's in the next
    const bool of_v = lane >= Tile::kGroups;
    s_src = (of_v ? v_src - 16 * Tile::kGroups : k_src) + Tile::kCodes;
    scale_at = ring + (of_v ? Tile::kBytes - 16 * Tile::kGroups : 0) + Tile::kCodes + 16 * lane;
#pragma unroll
    for (int i = 0; i < 2; ++i) k_at[i] = ring + chunk_at<D>(tok + 2 * i, t * KW / 4) + (t * KW % 4) * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) v_at[i] = ring + Tile::kBytes + chunk_at<D>(4 * t + i, g * VW / 4) + (g * VW % 4) * 4;
    if constexpr (D == 128) k_at[1] = k_at[0] + 128, v_at[2] = v_at[0] + 128, v_at[3] = v_at[1] + 128;  // (two tokens to a line)
  }

  // K and V of page p (below num_pages) and the head at head_off bytes of it, to `at` in the ring.
  __device__ __forceinline__ void copy_page(int p, uint32_t head_off, uint32_t at) const {
    const uint64_t off = (uint64_t)(uint32_t)p * page_bytes + head_off;
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
      copy16_async(code_at[r] + at, k_src + off + 512 * r);
      copy16_async(code_at[r] + at + Tile::kBytes, v_src + off + 512 * r);
    }
    if (lane < 2 * Tile::kGroups) copy16_async(scale_at + at, s_src + off);
  }

  // The group's queries, as convert_queries left them.
  __device__ __forceinline__ void start(const Queries<D>& from) {
    const float4* f = reinterpret_cast<const float4*>(from.rows[g] + t * (D / 4));
#pragma unroll
    for (int i = 0; i < KS / 2; ++i) {
      const float4 x = f[i];
      q[2 * i][0] = __float_as_uint(x.x), q[2 * i][1] = __float_as_uint(x.y);
      q[2 * i + 1][0] = __float_as_uint(x.z), q[2 * i + 1][1] = __float_as_uint(x.w);
    }
    qs0 = from.scale[2 * t], qs1 = from.scale[2 * t + 1];
    ref0 = ref1 = l0 = l1 = 0.0f, top0 = top1 = -INFINITY;
#pragma unroll
    for (int j = 0; j < KS; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
  }

  // The step at `slot` of the ring, which has `valid` tokens (32 at most).
  __device__ __forceinline__ void step(uint32_t slot, int valid) {
    if (valid < 2 * kPage)
      step_of<true>(slot, valid);
    else
      step_of<false>(slot, valid);
  }

  template <bool PART>
  __device__ __forceinline__ void step_of(uint32_t slot, int valid) {
    // ---- logits: tokens tok, tok + 2 of either page, heads 2 t, 2 t + 1
    float c[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = slot + h * C::kPair;
      uint32_t lo[KW], hi[KW];
      lds_words<KW>(k_at[0] + at, lo);
      lds_words<KW>(k_at[1] + at, hi);
#pragma unroll
      for (int n = 0; n < KG; ++n) {
        const uint32_t pair = e4m3_pair_to_h2(__byte_perm(lds32(ks_at + at + 16 * n), 0, ks_pick));
        const uint32_t sa = __byte_perm(pair, 0, 0x1010), sb = __byte_perm(pair, 0, 0x3232);
#pragma unroll
        for (int w = 0; w < 2; ++w) {  // a word of codes: two products
          const uint32_t x = lo[2 * n + w], y = hi[2 * n + w];
          const int j = 4 * n + 2 * w;
          const uint32_t a0 = mul_h2(e2m1x2_to_h2<0>(x), sa), a1 = mul_h2(e2m1x2_to_h2<0>(y), sb);
          const uint32_t a2 = mul_h2(e2m1x2_to_h2<1>(x), sa), a3 = mul_h2(e2m1x2_to_h2<1>(y), sb);
          if (j == 0)
            mma_first(c[h], a0, a1, a2, a3, q[j][0], q[j][1]);
          else
            mma(c[h], a0, a1, a2, a3, q[j][0], q[j][1]);
          mma(c[h], mul_h2(e2m1x2_to_h2<2>(x), sa), mul_h2(e2m1x2_to_h2<2>(y), sb), mul_h2(e2m1x2_to_h2<3>(x), sa),
              mul_h2(e2m1x2_to_h2<3>(y), sb), q[j + 1][0], q[j + 1][1]);
        }
      }
    }
    uint32_t v_scale[2] = {lds32(vs_at + slot), lds32(vs_at + slot + C::kPair)};
    if constexpr (PART) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (tok + 16 * h >= valid) c[h][0] = c[h][1] = -INFINITY;
        if (tok + 2 + 16 * h >= valid) c[h][2] = c[h][3] = -INFINITY;
        // (what a slot behind the sequence holds may be NaN)
        const int keep = valid - 16 * h - 4 * t;
        v_scale[h] &= keep >= 4 ? 0xffffffffu : keep <= 0 ? 0u : (1u << (8 * keep)) - 1u;
      }
    }

    // ---- softmax
    if (__any_sync(0xffffffffu, c[0][0] > top0 || c[0][1] > top1 || c[0][2] > top0 || c[0][3] > top1 || c[1][0] > top0 ||
                                    c[1][1] > top1 || c[1][2] > top0 || c[1][3] > top1)) {
      float n0 = fmaxf(fmaxf(c[0][0], c[0][2]), fmaxf(c[1][0], c[1][2])), n1 = fmaxf(fmaxf(c[0][1], c[0][3]), fmaxf(c[1][1], c[1][3]));
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, off));
        n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, off));
      }
      // a reference value moves to kBelow the step's maximum, where that is above it or there was none
      const float z0 = n0 * qs0, z1 = n1 * qs1;
      const float m0 = z0 - (fabsf(z0) < kLarge ? kBelow : 0.0f), m1 = z1 - (fabsf(z1) < kLarge ? kBelow : 0.0f);
      const bool up0 = n0 > -INFINITY && (top0 == -INFINITY || m0 > ref0), up1 = n1 > -INFINITY && (top1 == -INFINITY || m1 > ref1);
      const float f0 = up0 ? ex2(ref0 - m0) : 1.0f, f1 = up1 ? ex2(ref1 - m1) : 1.0f;
      const bool any0 = top0 > -INFINITY, any1 = top1 > -INFINITY;  // (else nothing has been summed, and f may be infinite)
      if (up0) ref0 = m0, top0 = (z0 + kHeadroom) / qs0;
      if (up1) ref1 = m1, top1 = (z1 + kHeadroom) / qs1;
      if (any0) l0 *= f0;
      if (any1) l1 *= f1;
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        if (any0) o[j][0] *= f0, o[j][2] *= f0;
        if (any1) o[j][1] *= f1, o[j][3] *= f1;
      }
    }
    uint32_t p[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x0 = ex2(fmaf(c[h][0], qs0, -ref0)), x1 = ex2(fmaf(c[h][1], qs1, -ref1));
      const float x2 = ex2(fmaf(c[h][2], qs0, -ref0)), x3 = ex2(fmaf(c[h][3], qs1, -ref1));
      l0 += x0 + x2, l1 += x1 + x3;
      p[h][0] = transpose8x8(pack_h2(x0, x1)), p[h][1] = transpose8x8(pack_h2(x2, x3));
    }

    // ---- weighted sum of V
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t at = slot + h * C::kPair;
      const uint32_t s01 = e4m3_pair_to_h2(v_scale[h]), s23 = e4m3_pair_to_h2(v_scale[h] >> 16);
      uint32_t w[4][VW];
#pragma unroll
      for (int n = 0; n < 4; ++n) lds_words<VW>(v_at[n] + at, w[n]);
#pragma unroll
      for (int k = 0; k < VW; ++k) {
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        // even and odd elements of tokens 4 t, 4 t + 1 and of 4 t + 2, 4 t + 3: a byte is an element of both
        const uint32_t e01 = (w[0][k] & kLow) | ((w[1][k] << 4) & ~kLow), d01 = ((w[0][k] >> 4) & kLow) | (w[1][k] & ~kLow);
        const uint32_t e23 = (w[2][k] & kLow) | ((w[3][k] << 4) & ~kLow), d23 = ((w[2][k] >> 4) & kLow) | (w[3][k] & ~kLow);
        mma(o[4 * k], mul_h2(e2m1x2_to_h2<0>(e01), s01), mul_h2(e2m1x2_to_h2<0>(d01), s01), mul_h2(e2m1x2_to_h2<0>(e23), s23),
            mul_h2(e2m1x2_to_h2<0>(d23), s23), p[h][0], p[h][1]);
        mma(o[4 * k + 1], mul_h2(e2m1x2_to_h2<1>(e01), s01), mul_h2(e2m1x2_to_h2<1>(d01), s01), mul_h2(e2m1x2_to_h2<1>(e23), s23),
            mul_h2(e2m1x2_to_h2<1>(d23), s23), p[h][0], p[h][1]);
        mma(o[4 * k + 2], mul_h2(e2m1x2_to_h2<2>(e01), s01), mul_h2(e2m1x2_to_h2<2>(d01), s01), mul_h2(e2m1x2_to_h2<2>(e23), s23),
            mul_h2(e2m1x2_to_h2<2>(d23), s23), p[h][0], p[h][1]);
        mma(o[4 * k + 3], mul_h2(e2m1x2_to_h2<3>(e01), s01), mul_h2(e2m1x2_to_h2<3>(d01), s01), mul_h2(e2m1x2_to_h2<3>(e23), s23),
            mul_h2(e2m1x2_to_h2<3>(d23), s23), p[h][0], p[h][1]);
      }
    }
  }

  // The sums over all tokens, on every lane.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, off);
      l1 += __shfl_xor_sync(0xffffffffu, l1, off);
    }
  }
};

// What a CTA works on where the lengths order the CTAs: the splits of 128 (sequence, split) pairs, most pages first, each with
// all its KV heads; then of the next 128 pairs, and what is left over of the batch comes first of all. Those of the SMs' first
// CTAs (sms at a time) are taken from either end in turn, so that no SM gets the longest of all.
struct Place {
  int item, head;  // item: sequence * num_splits + split
};
template <int D>
__device__ __forceinline__ Place place_of(const DecodeArgs& a) {
  __shared__ __align__(16) uint32_t keys[kGroup];
  __shared__ int found;
  const int t = threadIdx.x, p0 = blockIdx.x, layer = p0 / a.sms;
  const int p = layer < Cfg<D>::kCtas && (layer & 1) ? min((int)gridDim.x, (layer + 1) * a.sms) - 1 - (p0 - layer * a.sms) : p0;
  const int place = p / a.n_kv_heads, n = a.batch * a.num_splits, odd = n % kGroup;
  const int begin = place < odd ? 0 : odd + (place - odd) / kGroup * kGroup, count = place < odd ? odd : kGroup;
  wait_for_stream();
  if (a.lets_next) let_next_start();  // (after the wait: the merge reads the lengths at once)
  uint32_t key = 0;
  if (t < count) {
    const int split = (begin + t) % a.num_splits, len = __ldg(a.kv_lens + (begin + t) / a.num_splits);
    const int pages = len < 0 || len > a.max_blocks * kPage ? 0 : (len + kPage - 1) / kPage - split * a.pages_per_split;
    // (no two are equal; a difference past 2^24 pages is none)
    key = (uint32_t)min(max(min(pages, a.pages_per_split), 0), 1 << 24) * kGroup + (kGroup - t);
  }
  keys[t] = key;
  __syncthreads();
  int r0 = 0, r1 = 0, r2 = 0, r3 = 0;
#pragma unroll 8
  for (int i = 0; i < count; i += 4) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + i);
    r0 += k.x > key, r1 += k.y > key, r2 += k.z > key, r3 += k.w > key;
  }
  const int rank = r0 + r1 + r2 + r3;
  if (t < count && rank == place - begin) found = begin + t;
  __syncthreads();
  return Place{found, p % a.n_kv_heads};
}

// One CTA for each (split, KV head, sequence): its warps take the split's steps in turn and put their states together.
template <int D, bool ORDERED>
__global__ void __launch_bounds__(Cfg<D>::kWarps * 32, Cfg<D>::kCtas) decode_fp4_kernel(const DecodeArgs a) {
  using C = Cfg<D>;
  constexpr int KS = C::kSteps, S = C::kStages, NW = C::kWarps;
  extern __shared__ __align__(128) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = a.pages_per_split, G = a.n_qo_heads / a.n_kv_heads;
  int b, head, split;
  if constexpr (ORDERED) {
    const Place at = place_of<D>(a);
    b = at.item / a.num_splits, split = at.item % a.num_splits, head = at.head;
  } else {
    // Every other sequence's CTAs in reverse: those of splits that a sequence has not, which end at once, are then not
    // always on the same SMs (4 x 6000-32768 tokens of 8 heads in 19 splits, one CTA for each place: 30.2 to 24.9 us).
    b = blockIdx.y;
    const int x = b & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    head = x % a.n_kv_heads, split = x / a.n_kv_heads;
    wait_for_stream();
    if (a.lets_next) let_next_start();  // (after the wait: the merge reads the lengths at once)
  }

  __shared__ __align__(16) Queries<D> queries;
  uint32_t raw[D / 32] = {};
  const float k_scale = a.k_scale ? __ldg(a.k_scale + head) : 1.0f, v_scale = a.v_scale ? __ldg(a.v_scale + head) : 1.0f;
  if ((threadIdx.x >> 4) < G) {
    const char* src = static_cast<const char*>(a.q) + (((int64_t)b * a.n_qo_heads + head * G) * D * 2) + threadIdx.x * (D / 8);
    if constexpr (D == 128) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
      raw[0] = x.x, raw[1] = x.y, raw[2] = x.z, raw[3] = x.w;
    } else {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
      raw[0] = x.x, raw[1] = x.y;
    }
  }
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks + (int64_t)split * per;
  // the warp's steps are warp, warp + NW, ...; step i's pages are 2 i and 2 i + 1 of the split. A lane holds one entry of
  // the warp's next 16 steps.
  auto entry_of = [&](int i) { return 2 * (warp + (i + lane / 2) * NW) + (lane & 1); };
  int phys = 0;
  {
    const int at = entry_of(0);
    if (at < per && split * per + at < a.max_blocks) phys = __ldg(table + at);
  }
  const int kv_len = __ldg(a.kv_lens + b);
  Attention<D> w(a, smem_u32(smem) + warp * S * C::kSlot);  // (while the loads are on their way)
  if (kv_len < 0 || kv_len > a.max_blocks * kPage) {
    if (split == 0) {
      if (threadIdx.x == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
      write_rows<D>(a, b, head, NAN, NAN);
    }
    return;
  }
  const int nblk = (kv_len + kPage - 1) / kPage;
  const int n_live = (nblk + per - 1) / per;
  if (n_live == 0) {
    if (split == 0) write_rows<D>(a, b, head, 0.0f, -INFINITY);
    return;
  }
  if (split >= n_live) return;
  const int first = split * per;
  const int n_pages = min(per, nblk - first);
  const int tokens = min(kv_len - first * kPage, n_pages * kPage);  // of the split
  const int n_steps = (n_pages + 1) / 2, mine = n_steps > warp ? (n_steps - warp + NW - 1) / NW : 0;

  const uint32_t head_off = (uint32_t)head * Fp4Tile<D>::kBytes;
  bool bad = false;
  auto check = [&](int i) {  // the entries of the steps from i on: page 0 for a bad one, and rows of NaN in the end
    if (entry_of(i) < n_pages && (phys < 0 || phys >= a.num_pages)) {
      set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
      bad = true;
      phys = 0;
    }
  };
  check(0);
  auto issue = [&](int i, uint32_t slot) {  // the warp's i-th step
    if (i > 0 && i % 16 == 0) {
      phys = entry_of(i) < n_pages ? __ldg(table + entry_of(i)) : 0;
      check(i);
    }
    const int p0 = __shfl_sync(0xffffffffu, phys, 2 * i % 32), p1 = __shfl_sync(0xffffffffu, phys, 2 * i % 32 + 1);
    w.copy_page(p0, head_off, slot);
    if (2 * (warp + i * NW) + 1 < n_pages) w.copy_page(p1, head_off, slot + C::kPair);
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (i < mine) issue(i, i * C::kSlot);
    copy_commit();
  }
  convert_queries<D>(a, raw, k_scale, queries);
  __syncthreads();
  w.start(queries);
  uint32_t slot = 0, ahead = (S - 1) * C::kSlot;
  for (int i = 0; i < mine; ++i) {
    copy_wait<S - 2>();
    __syncwarp();  // step i is there for every lane, and step i - 1 has been read by all
    if (i + S - 1 < mine) issue(i + S - 1, ahead);
    copy_commit();
    ahead = slot;
    w.step(slot, tokens - 2 * (warp + i * NW) * kPage);
    slot = slot + C::kSlot == S * C::kSlot ? 0 : slot + C::kSlot;
  }

  // ---------------------------------------------------------------- the warps' states together
  w.finish();
  const bool poisoned = __syncthreads_or(bad);  // every copy has landed and been read: the rings are free
  const int g = lane >> 2, t = lane & 3;
  float* c_ref = reinterpret_cast<float*>(smem);  // [NW][kCols]
  float* c_l = c_ref + NW * kCols;                // [NW][kCols]
  float* c_o = c_l + NW * kCols;                  // [NW][kCols][kRow]: elements 2 j, 2 j + 1 of lane group g's D / 8 are pair_at(j, g)
  // Pairs of a warp's store (g and t vary) are in different banks, those of a load (g and every other j) two to a bank.
  auto pair_at = [](int j, int g) { return 16 * j + 2 * (g ^ ((j & 2) << 1)); };
  if (g == 0) {
    // (a warp that has summed nothing sets no common reference)
    c_ref[warp * kCols + 2 * t] = w.l0 == 0.0f ? -INFINITY : w.ref0, c_ref[warp * kCols + 2 * t + 1] = w.l1 == 0.0f ? -INFINITY : w.ref1;
    c_l[warp * kCols + 2 * t] = w.l0, c_l[warp * kCols + 2 * t + 1] = w.l1;
  }
#pragma unroll
  for (int j = 0; j < KS; ++j) {
    float* at = c_o + (warp * kCols + 2 * t) * C::kRow + pair_at(j, g);
    if (2 * t < G) *reinterpret_cast<float2*>(at) = make_float2(w.o[j][0], w.o[j][2]);
    if (2 * t + 1 < G) *reinterpret_cast<float2*>(at + C::kRow) = make_float2(w.o[j][1], w.o[j][3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < G * (D / 4); i += NW * 32) {
    const int h = i / (D / 4), d = i % (D / 4) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, c_ref[w * kCols + h]);
    float L = 0.0f, O[4] = {};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ex2(c_ref[w * kCols + h] - M);
      const float lw = c_l[w * kCols + h];
      if (lw != 0.0f) {  // a warp without pages has none
        const float* from = c_o + (w * kCols + h) * C::kRow;
        const float2 x = *reinterpret_cast<const float2*>(from + pair_at(d % (D / 8) / 2, d / (D / 8)));
        const float2 y = *reinterpret_cast<const float2*>(from + pair_at(d % (D / 8) / 2 + 1, d / (D / 8)));
        L += f * lw;
        O[0] += f * x.x, O[1] += f * x.y, O[2] += f * y.x, O[3] += f * y.y;
      }
    }
    const float inv = v_scale / L;
#pragma unroll
    for (int e = 0; e < 4; ++e) O[e] = poisoned ? NAN : O[e] * inv;
    const int64_t row = (int64_t)b * a.n_qo_heads + (int64_t)head * G + h;
    const int64_t part = row * a.num_splits + split;
    if (n_live == 1) {
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * D + d;
#pragma unroll
      for (int e = 0; e < 4; e += 2) *reinterpret_cast<__nv_bfloat162*>(out + e) = __floats2bfloat162_rn(O[e], O[e + 1]);
    } else {
      *reinterpret_cast<float4*>(a.part_o + part * D + d) = make_float4(O[0], O[1], O[2], O[3]);
    }
    if (d == 0) {
      const float lse = poisoned ? NAN : (M + log2f(L)) * kLn2;
      if (n_live > 1)
        a.part_lse[part] = lse;
      else if (a.lse)
        a.lse[row] = lse;
    }
  }
}

// CTAs with pages, where rows are of all lengths.
double live_ctas(int batch, int n_kv_heads, int splits) { return 0.5 * batch * n_kv_heads * (splits + 1.0); }

// Whether the lengths order the CTAs. That saves the last of them running alone, most of the time of a split, and costs
// each CTA a look at the lengths before all else, 0.45 us of an SM: worth it where more CTAs than fit have pages, but not many times
// more, and splits are long. Measured with and without, ragged rows and full ones: 128 x 200-4000 tokens of 8 heads 60.0 and
// 73.1 us, 104 and 100; 16 x 512-4096 of 32 in 2 splits 38.1 and 41.5, 58.5 and 56.1; 100 x 10-3000 of 8 in 2 (9 pages for
// each CTA of an SM: left alone) 44.1 and 48.1, 76.3 and 71.1; 159 x 7-354 of 8 13.6 and 10.5, 17.6 and 13.6.
bool is_ordered(int batch, int n_kv_heads, int splits, int pages_per_split, int sms, int ctas) {
  const double all = (double)batch * n_kv_heads * splits;
  return batch > 1 && live_ctas(batch, n_kv_heads, splits) > (double)sms * ctas && pages_per_split * (double)sms > 16 * all &&
         all < 2147483648.0;
}

template <int D>
int launch_t(DecodeArgs a, cudaStream_t stream) {
  static FuncConfigured configured[2];
  a.sms = device_sm_count();
  if (a.sms <= 0) a.sms = 148;
  // (below 1, so that its product with a head's scale is finite)
  a.scale_fraction = 0.5f * kLog2e * std::frexp(std::fabs(a.scale), &a.scale_exponent);
  ++a.scale_exponent;
  if (a.scale_exponent < -124) a.scale_fraction = std::ldexp(a.scale_fraction, a.scale_exponent + 124), a.scale_exponent = -124;
  const int ctas = a.n_kv_heads * a.num_splits;
  const bool ordered = is_ordered(a.batch, a.n_kv_heads, a.num_splits, a.pages_per_split, a.sms, Cfg<D>::kCtas);
  auto* kernel = ordered ? decode_fp4_kernel<D, true> : decode_fp4_kernel<D, false>;
  if (!configured[ordered].ensure(reinterpret_cast<const void*>(kernel), Cfg<D>::kSmem)) return PKV_ERR_LAUNCH;
  // Whether the stream's next kernel may be placed before this one's end: the merge, or whatever follows a launch of more CTAs than
  // fit. One-wave launches that begin early get their CTAs where the kernel before leaves room, unevenly for good (40 x
  // 100-1000 tokens of 8 heads, calls one after another, 14.4 us and 11.7), so other launches leave the next one alone.
  a.lets_next = a.num_splits > 1 || (int64_t)ctas * a.batch > (int64_t)Cfg<D>::kCtas * a.sms;
  const dim3 grid = ordered ? dim3((unsigned)ctas * a.batch) : dim3((unsigned)ctas, (unsigned)a.batch);
  const int rc = check_launch(launch_overlapped(kernel, grid, Cfg<D>::kWarps * 32, Cfg<D>::kSmem, stream, 1, a));
  if (rc != PKV_OK || a.num_splits == 1) return rc;
  return launch_merge_splits(a, stream);
}

}  // namespace

constexpr double kFixed = 12;

// Estimated time of so many splits, in pages that an SM goes through (65 ns each at head_dim 128, and the same pages are
// counted at head_dim 64, where they take less: see below), where `filled` of the CTAs have pages: each takes its pages and a fixed cost of kFixed (its first loads, the warps' states), fewer than four on an SM
// are slower, and a second launch is kMerge and something for each split. Whole CTAs, or on average.
static double time_of_splits(double units, int max_blocks, int s, double filled, bool whole, int sms, int ctas) {
  constexpr double kMerge = 40;
  const double per = (max_blocks + s - 1) / s, n = filled * units * s, slots = (double)sms * ctas;
  const double waves = std::floor(n / slots), rest = (n - waves * slots) / sms;
  double last = 0;
  if (waves == 0 || rest > 0.02) {
    const double m = whole ? std::ceil(rest) : std::fmax(rest, 1.0);
    last = m * (per * (m > 3.5 ? 1.0 : 1.0 + 0.5 / (m * std::sqrt(m))) + kFixed);
  }
  return waves * ctas * (per + kFixed) + last + (s > 1 ? kMerge + 0.3 * s : 0);
}

// The split count with the least estimated time. Lengths are not known here, only the table's width: the estimate is that
// of full rows and that of rows 3/5 full on average, where the last CTAs run alone for some of their pages, together.
// Measured (us, the chosen one first): 4 x 32768 tokens of 8 heads 30.6 with 19 splits, 33.4 with 32, 33.9 with 38; the same
// with 6000-32768 tokens 24.7 with 19, 25.5 with 32, 28.3 with 38; 16 x 512-4096 of 32 heads 37.8 with 2, 40.2 with 4, 49.9
// with 1; 64 x 100-1000 of 8 15.5 with 1, 19.3 with 2. Head_dim 64, 8 shapes of full rows and of ragged ones: within 9 % of the best
// of up to 20 counts but for 8 x 1000-10000 tokens of 8 heads, 15.0 with 9 splits and 12.5 with 16. CTAs that find the lengths and divide the pages evenly among them
// do so whatever they are, but take 2 us more (33.7, 25.6 and 45.8 us for the first three).
SplitPlan plan_decode_fp4(int batch, int max_blocks, int n_kv_heads, int requested) {
  int S;
  if (requested > 0) {
    S = requested < max_blocks ? requested : max_blocks;
  } else {
    int sms = device_sm_count();
    if (sms <= 0) sms = 148;
    static_assert(Cfg<64>::kCtas == Cfg<128>::kCtas, "one estimate for both");
    const int ctas = Cfg<128>::kCtas, most = max_blocks < 128 ? max_blocks : 128;
    const double units = (double)batch * n_kv_heads;
    double best = -1;
    S = 1;
    for (int s = 1, seen = 0; s <= most; ++s) {
      const int per = (max_blocks + s - 1) / s;
      if (per == seen) continue;  // (no more splits than there were)
      seen = per;
      if (best >= 0 && 1.5 * units * (max_blocks + s * kFixed) / sms > best) break;  // (the work of all alone)
      double cost = time_of_splits(units, max_blocks, s, 1.0, true, sms, ctas) +
                          time_of_splits(units, max_blocks, s, 0.59, false, sms, ctas) + 0.4 * per;
      // more CTAs with pages than fit, in no order: some end up alone
      if (live_ctas(batch, n_kv_heads, s) > (double)sms * ctas && !is_ordered(batch, n_kv_heads, s, per, sms, ctas))
        cost += 0.25 * per;
      if (best < 0 || cost < best) best = cost, S = s;
    }
  }
  const int per = (max_blocks + S - 1) / S;
  return SplitPlan{(max_blocks + per - 1) / per, per};
}

int launch_decode_fp4(const DecodeArgs& a, cudaStream_t stream) {
  if (a.head_dim == 64) return launch_t<64>(a, stream);
  if (a.head_dim == 128) return launch_t<128>(a, stream);
  return PKV_ERR_UNSUPPORTED;
}

}  // namespace pkv
