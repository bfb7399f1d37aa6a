// Linear layer with its epilogue: y[m][n] = act(x[m][k] w[n][k]^T + bias[n]) + residual[m][n].
//
// For few tokens the weights stream through the tensor cores as in the flat GEMM (flat_gemm.cu
// with its epilogue instantiation; launch_linear has the rule). Else this file's kernel: persistent pairs of CTAs, a tile of
// 256 tokens x BN features per pair. One tcgen05 product spans both SMs of the pair: each holds its
// 128 tokens and half of the features, so that a CTA reads half the weights a single one would, and
// the fp32 accumulators of its tokens. Operands come by TMA through a ring of six 64-column blocks;
// the accumulator is double-buffered, so eight epilogue warps read one tile out of tensor memory,
// apply bias, activation and residual in fp32 and store it (one rounding) while the next tile's
// products run.
//
// Bound: the tensor cores, 2 m n k operations; for few tokens the weights' bytes. 4096 x 11008 x 4096 with
// bias and gelu_tanh takes 195 to 200 us in a burst (1.9 PFLOP/s, the rate of the library's plain product; the tensor
// pipe is busy 91 % of the time) and 225 to 229 us under the power limit. BN is the multiple of 32 for which the
// rounds of tiles over the pairs take least (choose_width); what is lost is the last round: 1024 x 4096
// x 4096 takes 24 us where its products are 18. A short product is bound by its epilogue, whose loads
// are a chain: 2611 x 11008 x 256 takes 27 us, 45 to 49 with a residual (46 and 77 with four warps that ask for
// everything when they need it), of which the products with their operands from the L2 are 17. Rows
// that no 16-byte store fits go through shared memory (1152 x 4097 x 1024 with residual: 75 to 31 us, 40 where the
// tensors are not in the L2). Not
// kept: sixteen warps (no faster, small products 3 % slower), y through shared memory and TMA (the same
// time where rows are aligned to 32 bytes).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <cmath>

#include "epilogue.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace pkv {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // prefill.cu

namespace {

constexpr int LBK = 64;              // K per block of a stage: one 128-byte swizzled row
constexpr int BLK = 128 * LBK * 2;   // a CTA's tokens (or most features) of a block
constexpr int LTHREADS = 384;      // TMA, MMA, two idle warps, eight for the epilogue
constexpr int PANEL = 16;  // token tiles walked before the next feature tile: their x stays in L2

struct LinArgs {
  __nv_bfloat16* y;
  Epilogue ep;
  int m, n, n_kc;  // n_kc: stages of K
  int tiles_m, tiles;
  int vec;  // bytes to which the rows of y and of the residual are aligned: 32, 16, or 0 for neither
  int32_t* err_flag;
};

struct LMisc {
  uint32_t tmem_base;
  int abort_;
};

// Tile index -> (token tile, feature tile): panels of PANEL token tiles, token tiles fastest.
__device__ __forceinline__ void tile_at(int i, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per = PANEL * tiles_n;
  const int p = i / per, r = i % per;
  const int rows = min(PANEL, tiles_m - p * PANEL);
  tm = p * PANEL + r % rows;
  tn = r / rows;
}

// 32 features of one token, those from `end` on not stored. `bias` holds theirs (0 from `end` on); `res`
// the residual's, where they are all stored and its rows are aligned.
// All lanes of a warp take part, those of tokens past the last too; `turn` is the warp's own corner of
// shared memory, 32 x 17 floats.
__device__ __forceinline__ void finish_rows(const LinArgs& a, float (&v)[32], const float* bias, const uint4 (&res)[4],
                                            float* turn, int row, int col, int end) {
  constexpr int N = 32;
  const int64_t at = (int64_t)row * a.n + col;
  if (a.ep.bias) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 b = *reinterpret_cast<const float4*>(bias + i);
      v[i] += b.x, v[i + 1] += b.y, v[i + 2] += b.z, v[i + 3] += b.w;
    }
  }
  activate_all(v, a.ep.activation);
  if (a.vec && col + N <= end) {
    if (row >= a.m) return;
    if (a.ep.residual) {
#pragma unroll
      for (int i = 0; i < N; i += 8) {
        const uint4 r = res[i / 8];
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[i + 2 * k] += __uint_as_float(w[k] << 16);
          v[i + 2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
        }
      }
    }
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    if (a.vec == 32) {  // whole 32-byte sectors (half-sector stores cost 4 % of a large product)
#pragma unroll
      for (int i = 0; i < N / 2; i += 8)
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a.y + at + 2 * i), "r"(w[i]),
                     "r"(w[i + 1]), "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]),
                     "r"(w[i + 7])
                     : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; i += 4)
        *reinterpret_cast<uint4*>(a.y + at + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
  } else {
    // Rows that no wide store fits: through shared memory in two halves, so that a warp reads and
    // writes runs of 16 features of two tokens at a time, not 32 tokens' single features.
    constexpr int H = N / 2;
    const int lane = threadIdx.x & 31, row0 = row - lane, c = lane % H;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int f = col + half * H + c;
      const int64_t to = (int64_t)(row0 + lane / H) * a.n + f;  // of the lane's first token
      float add[H] = {};
      if (a.ep.residual) {  // all asked for before any is used: y may be the residual
#pragma unroll
        for (int i = 0; i < H; ++i)
          if (row0 + lane / H + 2 * i < a.m && f < end) add[i] = __bfloat162float(a.ep.residual[to + (int64_t)(2 * i) * a.n]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < H; ++i) turn[lane * (H + 1) + i] = v[half * H + i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float x = turn[(lane / H + 2 * i) * (H + 1) + c];
        if (row0 + lane / H + 2 * i < a.m && f < end)
          a.y[to + (int64_t)(2 * i) * a.n] = __float2bfloat16_rn(a.ep.residual ? x + add[i] : x);
      }
    }
  }
}

constexpr int PBM = 256;  // tokens of a pair's tile, 128 per CTA

// SUB: 64-column blocks per stage. One for wide tiles, whose stage is bound by its products; two
// for narrow ones, where the barriers of a stage weigh more (256 x 4096 x 4096: 22.9 to 16.6 us).
template <int SUB>
struct LinCfg {
  static constexpr int PST = 6 / SUB, STG = SUB * BLK;  // stages; bytes of one operand's stage
  static constexpr int SM_B = PST * STG, SM_BAR = 2 * PST * STG, NBAR = 2 * PST + 5, SM_MISC = SM_BAR + NBAR * 8,
                       SM_BIAS = (SM_MISC + 16 + 15) / 16 * 16,  // [8 warps][4 runs][32]
                       SM_TURN = SM_BIAS + 8 * 4 * 32 * 4,       // [8 warps][32][17]
                       SMEM = SM_TURN + 8 * 32 * 17 * 4 + 1024;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ uint32_t pair_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of the same shared-memory location in the pair's first CTA.
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void pair_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A load into this CTA's shared memory that counts on a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(mbar),
      "h"((unsigned short)3)
      : "memory");
}
// Arrives on a barrier of the pair's first CTA. Relaxed: what it announces is that reads of tensor memory
// are over. tcgen05.wait::ld and the fence before this order the arriving lane's, the __syncwarp between
// them the other lanes', and the issuer's fence after its wait orders the products behind them. A release
// would wait for the tile's stores as well.
__device__ __forceinline__ void arrive_remote(uint32_t mbar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(mbar) : "memory");
}

// A cluster of two CTAs per tile of 256 tokens x bn features. The first CTA's MMA warp issues the
// products of both; loads of both count on its `full` barriers, its commits free the stages of
// both, and the epilogue warps of both hand the accumulators back to it.
template <int SUB>
__global__ void __launch_bounds__(LTHREADS, 1)
linear_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const LinArgs a,
                   int bn) {
  using C = LinCfg<SUB>;
  constexpr int PST = C::PST;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  unsigned char* smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  LMisc* misc = reinterpret_cast<LMisc*>(smem + C::SM_MISC);
  const uint32_t full = sb + C::SM_BAR, empty = full + 8 * PST, acc_full = empty + 8 * PST, acc_empty = acc_full + 16,
                 drain = acc_empty + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)pair_rank(), pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles_n = a.tiles / a.tiles_m;
  const int half = bn / 2;  // features per CTA

  if (threadIdx.x == 0) {
    for (int s = 0; s < PST; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full + 8 * s, 1);
      mbar_init(acc_empty + 8 * s, 16);
    }
    mbar_init(drain, 1);
    misc->abort_ = 0;
    fence_mbar_init();
  }
  // (before tensor memory is taken: an earlier kernel of the stream may still need it)
  wait_for_stream();
  if (warp == 0) {
    __syncwarp();  // the lanes converge after the barriers' initialisation
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&misc->tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // both CTAs' barriers exist before either signals the other's
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
    // ------------------------------------------------------------ TMA producer, one in each CTA
    if (elect_one()) {
      tma_prefetch_desc(&mx);
      tma_prefetch_desc(&mw);
    }
    __syncwarp();
    uint32_t c = 0;
    bool ok = true;
    for (int i = pair; ok && i < a.tiles; i += pairs) {
      int tm, tn;
      tile_at(i, a.tiles_m, tiles_n, tm, tn);
      if (__any_sync(0xffffffffu, *aborted)) ok = false;  // (asked once a tile: the producers' loop is the critical path)
      for (int kc = 0; ok && kc < a.n_kc; ++kc, ++c) {
        const uint32_t s = c % PST;
        if (c >= PST && !warp_wait(empty + 8 * s, (c / PST - 1) & 1)) ok = false;
        if (!ok) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, 2 * SUB * (BLK + half * LBK * 2));
          const uint32_t bar = in_first(full + 8 * s);
#pragma unroll
          for (int h = 0; h < SUB; ++h) {
            const int k0 = (kc * SUB + h) * LBK;  // (columns past k read as 0)
            tma_load_2d_pair(sb + s * C::STG + h * BLK, &mx, k0, tm * PBM + rank * 128, bar);
            tma_load_2d_pair(sb + C::SM_B + s * C::STG + h * BLK, &mw, k0, tn * bn + rank * half, bar);
          }
        }
        __syncwarp();
      }
    }
    if (!ok) give_up();
    // the last signals that free this CTA's stages have come before it may end
    for (uint32_t s = 0; ok && s < (uint32_t)PST && s < c; ++s) ok = warp_wait(empty + 8 * s, ((c - 1 - s) / PST) & 1);
    if (!ok) give_up();
    if (rank == 0) {  // every copy, the other CTA's too, lands before the shared memory is released
      bool drained = true;
      for (uint32_t s = 0; s < (uint32_t)PST && s < c; ++s)
        drained &= warp_wait(full + 8 * s, ((c - 1 - s) / PST) & 1);
      if (!drained) give_up();
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16_f32(PBM, bn, false, false);
    const uint64_t da0 = smem_desc(sb, 16, 1024, kSwizzle128B);
    const uint64_t db0 = smem_desc(sb + C::SM_B, 16, 1024, kSwizzle128B);
    uint32_t c = 0, t = 0;
    bool ok = true;
    for (int i = pair; ok && i < a.tiles; i += pairs, ++t) {
      const uint32_t buf = t & 1;
      if (t >= 2 && !warp_wait(acc_empty + 8 * buf, (t / 2 - 1) & 1)) ok = false;
      tc_fence_after();
      for (int kc = 0; ok && kc < a.n_kc; ++kc, ++c) {
        const uint32_t s = c % PST;
        if (!warp_wait(full + 8 * s, (c / PST) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t da = da0 + (uint64_t)((s * C::STG) >> 4), db = db0 + (uint64_t)((s * C::STG) >> 4);
#pragma unroll
          for (int kk = 0; kk < SUB * LBK / 16; ++kk) {
            const uint64_t off = (uint64_t)((kk / 4 * BLK + kk % 4 * 32) >> 4);
            mma_pair(tmem + buf * 256, da + off, db + off, idesc, (kc > 0 || kk > 0) ? 1u : 0u);
          }
          commit_pair(empty + 8 * s);
          if (kc == a.n_kc - 1) commit_pair(acc_full + 8 * buf);
        }
        __syncwarp();
      }
    }
    if (!ok) give_up();
    if (elect_one())  // every issued product finishes before TMEM is freed
      asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(drain) : "memory");
    __syncwarp();
    if (!warp_wait(drain, 0)) give_up();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    // Two warps for each quarter of the tokens, which take the runs of 32 features in turn. The
    // epilogue of a short product is a chain of loads, so they are asked for early: the bias of a
    // tile in the tile before (through shared memory), the residual's lines come to the L2 in the tile
    // before and to registers two runs ahead.
    const int wq = warp & 3, group = (warp - 4) >> 2;
    float* bias_s = reinterpret_cast<float*>(smem + C::SM_BIAS) + (warp - 4) * 128;
    float* turn_s = reinterpret_cast<float*>(smem + C::SM_TURN) + (warp - 4) * (32 * 17);
    float bias_next[4] = {};
    auto ask_bias = [&](int col0, int end) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int col = col0 + 32 * group + 64 * k + lane;
        bias_next[k] = a.ep.bias && col < end ? __bfloat162float(a.ep.bias[col]) : 0.0f;
      }
    };
    uint32_t t = 0;
    bool ok = true;
    int tm = 0, tn = 0;
    if (pair < a.tiles) {
      tile_at(pair, a.tiles_m, tiles_n, tm, tn);
      ask_bias(tn * bn, min(a.n, (tn + 1) * bn));
    }
    for (int i = pair; i < a.tiles; i += pairs, ++t) {
      const uint32_t buf = t & 1;
      const int row = tm * PBM + rank * 128 + wq * 32 + lane;
      const int end = min(a.n, (tn + 1) * bn), col0 = tn * bn;
#pragma unroll
      for (int k = 0; k < 4; ++k) bias_s[32 * k + lane] = bias_next[k];
      if (i + pairs < a.tiles) {
        tile_at(i + pairs, a.tiles_m, tiles_n, tm, tn);
        const int next0 = tn * bn, next_end = min(a.n, next0 + bn), next_row = tm * PBM + rank * 128 + wq * 32 + lane;
        ask_bias(next0, next_end);
        if (a.ep.residual && next_row < a.m) {
          for (int col = next0 + 64 * group; col < next_end; col += 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.ep.residual + (int64_t)next_row * a.n + col));
        }
      }
      __syncwarp();  // the bias is in
      const uint32_t src = tmem + ((uint32_t)(wq * 32) << 16) + buf * 256;
      const __nv_bfloat16* res_row = a.ep.residual && a.vec && row < a.m ? a.ep.residual + (int64_t)row * a.n + col0 : nullptr;
      auto ask = [&](uint4 (&r)[4], int cc) {
        if (res_row && cc < bn && col0 + cc + 32 <= end) {
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = *reinterpret_cast<const uint4*>(res_row + cc + 8 * k);
        }
      };
      uint4 res[4] = {}, next_res[4] = {};
      ask(res, 32 * group);
      ask(next_res, 32 * group + 64);
      if (ok && !warp_wait(acc_full + 8 * buf, (t / 2) & 1)) ok = false;
      tc_fence_after();
#pragma unroll 1
      for (int cc = 32 * group; cc < bn; cc += 64) {
        uint32_t r[32];
        if (ok) {
          tmem_ld32(src + cc, r);
          tmem_ld_wait();
        }
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = ok ? __uint_as_float(r[k]) : NAN;
        if (col0 + cc < end) finish_rows(a, v, bias_s + cc / 64 * 32, res, turn_s, row, col0 + cc, end);
#pragma unroll
        for (int k = 0; k < 4; ++k) res[k] = next_res[k];
        ask(next_res, cc + 128);
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (ok && elect_one()) arrive_remote(in_first(acc_empty + 8 * buf));
      __syncwarp();
    }
    if (!ok) give_up();
  }
  tc_fence_before();
  __syncthreads();
  pair_sync();  // neither CTA's memory goes while the other's products or signals may touch it
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

bool encode_rows(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_outer) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  cuuint64_t strides[1] = {(cuuint64_t)inner * 2};
  cuuint32_t box[2] = {(cuuint32_t)LBK, box_outer};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The feature width for which the tiles take least. Measured for k = 4096: a round of tiles of
// width 256, 224, 192, 160, 128, 96, 64, 32 takes 20.4, 18.1, 16.0, 14.8, 13.3, 12.2, 11.4, 10.7 us, the
// wide ones their products, the narrow ones the loads and barriers of a stage; the costs below are
// those in 10 ns. What does not fill a round of the pairs is lost. A product over a pair takes
// multiples of 32 from 32 to 256.
int choose_width(int64_t tiles_m, int n, int pairs) {
  int best_w = 256;
  int64_t best = -1;
  for (int w = 256; w >= 32; w -= 32) {
    const int64_t tiles = tiles_m * (((int64_t)n + w - 1) / w);
    const int64_t round = 7 * w + 250 > 3 * w + 1000 ? 7 * w + 250 : 3 * w + 1000;
    const int64_t cost = (tiles + pairs - 1) / pairs * round;
    if (best < 0 || cost < best) {
      best = cost;
      best_w = w;
    }
  }
  return best_w;
}

template <int SUB>
int launch_t(const CUtensorMap& mx, const CUtensorMap& mw, const LinArgs& a, int bn, unsigned grid, cudaStream_t stream) {
  static FuncConfigured configured;
  if (!configured.ensure(reinterpret_cast<const void*>(linear_kernel<SUB>), LinCfg<SUB>::SMEM)) return PKV_ERR_LAUNCH;
  return check_launch(launch_overlapped(linear_kernel<SUB>, dim3(grid), LTHREADS, LinCfg<SUB>::SMEM, stream, 2, mx, mw, a, bn));
}

constexpr int kWide = 224;  // tiles from this width take one block per stage

}  // namespace

int launch_linear(const LinearArgs& p, cudaStream_t stream) {
  // Few tokens stream the weights (flat_gemm.cu) where that is most of the time. Where its plan splits K over a
  // cluster, that and its epilogue, which grows with the tokens, cost more than a tile here for short products, and
  // past 32 tokens for all but long ones. There and here, in us, weights cold: 8 x 1024 x 72 5.8 and 5.2; 64 tokens,
  // 4096 x 512 9.5 and 6.8, 11008 x 1024 14.3 and 10.5, 12288 x 2048 17.8 and 15.8, 8192 x 4096 27 and 21; but 8 x 1024 x
  // 1024 5.5 and 7.0, 32 x 4096 x 4096 11 and 17, 64 x 4096 x 4096 13 and 17, 64 x 1024 x 8192 12 and 28. Without a split
  // (k up to 64, or more tiles than the SMs take at once) it is ahead everywhere: 16 x 22016 x 64 3.8 and 8.1, 64 x 4096
  // x 64 4.1 and 5.2, 64 x 32000 x 1024 14 and 17, x 4096 45 and 50. Over 7 token counts up to 64, 16 n from 256 to 32000 and
  // 9 k from 64 to 8192 the rule is 1 % off the better of the two on average, up to 43 % at single sizes (32 x 6144 x 1024, 13.4
  // there for 9.4: 48 tiles by 6 do not fit the SMs at once; 33 x 12288 x 6144, 35 here for 29).
  // More features than the flat kernel's grid holds run here whatever their time.
  if (p.m <= kFlatGemmMaxM && p.n <= kFlatGemmMaxN) {
    const bool tiled = plan_flat_gemm(p.m, p.n, p.k).splits > 1 &&
                       (p.k <= 128 || (p.m > 32 && (p.k <= 1024 || p.k <= p.n / 2)));
    if (!tiled) return launch_flat_linear(p, stream);
  }
  if (p.m > 0x7fffff00 || p.n > 0x7fffff00) return PKV_ERR_UNSUPPORTED;  // (tile ends fit 32 bits)
  int sms = device_sm_count();
  if (sms <= 1) sms = 148;
  const int pairs = sms / 2;
  const int64_t tm = ((int64_t)p.m + PBM - 1) / PBM;
  const int bn = choose_width(tm, p.n, pairs);
  const int64_t tiles = tm * (((int64_t)p.n + bn - 1) / bn);
  if (tiles > 0x7fffffffL) return PKV_ERR_UNSUPPORTED;
  const uintptr_t rows = reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.residual);
  const int vec = p.n % 16 == 0 && rows % 32 == 0 ? 32 : p.n % 8 == 0 && rows % 16 == 0 ? 16 : 0;
  const int block = bn >= kWide ? LBK : 2 * LBK;
  const LinArgs a{static_cast<__nv_bfloat16*>(p.y),
                  Epilogue{static_cast<const __nv_bfloat16*>(p.bias), static_cast<const __nv_bfloat16*>(p.residual),
                           p.activation},
                  p.m, p.n, (p.k + block - 1) / block, (int)tm, (int)tiles, vec, p.err_flag};
  const unsigned grid = 2u * (unsigned)(tiles < pairs ? tiles : pairs);
  CUtensorMap mx, mw;
  if (!encode_rows(&mx, p.x, (uint64_t)p.k, (uint64_t)p.m, 128) ||
      !encode_rows(&mw, p.w, (uint64_t)p.k, (uint64_t)p.n, (uint32_t)bn / 2))
    return check_launch(cudaErrorInvalidValue);
  return bn >= kWide ? launch_t<1>(mx, mw, a, bn, grid, stream) : launch_t<2>(mx, mw, a, bn, grid, stream);
}

}  // namespace pkv
