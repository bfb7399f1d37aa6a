// Linear layer with its epilogue: y[m][n] = act(x[m][k] w[n][k]^T + bias[n]) + residual[m][n].
//
// Up to 64 tokens the weights stream through the tensor cores as in the flat GEMM (flat_gemm.cu
// with its epilogue instantiation). Above, this file's tiled kernel: a persistent CTA per SM
// multiplies 128 tokens x BN features with tcgen05, fp32 accumulators in tensor memory,
// operands by TMA through a ring of 64-column stages. The accumulator is double-buffered, so the
// four epilogue warps read one tile out of tensor memory, apply bias, activation and residual in
// fp32 and store it (one rounding) while the next tile's products run.
//
// BN is 256 where that still gives every SM a tile, else 128 or 64: a small problem needs
// more tiles than wide ones give, a large one wants the operand reuse of the widest.
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

constexpr int LBM = 128, LBK = 64;
constexpr int ASTG = LBM * LBK * 2;
constexpr int LTHREADS = 256;
constexpr int PANEL = 16;  // token tiles walked before the next feature tile: their x stays in L2

template <int BN>
struct LinCfg {
  static constexpr int BSTG = BN * LBK * 2;
  static constexpr int NST = BN == 256 ? 4 : BN == 128 ? 6 : 8;
  static constexpr int SM_A = 0, SM_B = NST * ASTG, SM_BAR = SM_B + NST * BSTG;
  // barriers: full[NST], empty[NST], acc_full[2], acc_empty[2], drain
  static constexpr int NBAR = 2 * NST + 5;
  static constexpr int SM_MISC = SM_BAR + NBAR * 8, SMEM = SM_MISC + 16 + 1024;
  static constexpr int TMEM = 2 * BN;
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

struct LinArgs {
  __nv_bfloat16* y;
  Epilogue ep;
  int m, n, n_kc;
  int tiles_m, tiles;
  bool vec;  // rows of y and of the residual are 16-byte aligned
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

// 32 consecutive features of one token.
__device__ __forceinline__ void finish_row(const LinArgs& a, float (&v)[32], int row, int col) {
  const __nv_bfloat16* bias = a.ep.bias;
  const int64_t at = (int64_t)row * a.n + col;
  if (a.vec && col + 32 <= a.n) {
    if (bias) {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(bias + col + i));
        v[i] += b.x, v[i + 1] += b.y;
      }
    }
    activate_all(v, a.ep.activation);
    if (a.ep.residual) {
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        const uint4 r = *reinterpret_cast<const uint4*>(a.ep.residual + at + i);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[i + 2 * k] += __uint_as_float(w[k] << 16);
          v[i + 2 * k + 1] += __uint_as_float(w[k] & 0xffff0000u);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 32; i += 8)
      *reinterpret_cast<uint4*>(a.y + at + i) = make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]),
                                                           pack_bf16x2(v[i + 4], v[i + 5]), pack_bf16x2(v[i + 6], v[i + 7]));
  } else {
    if (bias) {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (col + i < a.n) v[i] += __bfloat162float(bias[col + i]);
    }
    activate_all(v, a.ep.activation);
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (col + i < a.n) {
        const float r = a.ep.residual ? __bfloat162float(a.ep.residual[at + i]) : 0.0f;
        a.y[at + i] = __float2bfloat16_rn(a.ep.residual ? v[i] + r : v[i]);
      }
    }
  }
}

template <int BN>
__global__ void __launch_bounds__(LTHREADS, 1)
linear_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mw, const LinArgs a) {
  using C = LinCfg<BN>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw & 1023u)) & 1023u;
  unsigned char* smem = smem_raw + pad;
  const uint32_t sb = raw + pad;
  LMisc* misc = reinterpret_cast<LMisc*>(smem + C::SM_MISC);
  const uint32_t full = sb + C::SM_BAR, empty = full + 8 * C::NST, acc_full = empty + 8 * C::NST,
                 acc_empty = acc_full + 16, drain = acc_empty + 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_n = a.tiles / a.tiles_m;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NST; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(acc_full + 8 * s, 1);
      mbar_init(acc_empty + 8 * s, 4);
    }
    mbar_init(drain, 1);
    misc->abort_ = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&misc->tmem_base), C::TMEM);
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
    // ------------------------------------------------------------ TMA producer
    if (elect_one()) {
      tma_prefetch_desc(&mx);
      tma_prefetch_desc(&mw);
    }
    __syncwarp();
    uint32_t c = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < a.tiles; i += gridDim.x) {
      int tm, tn;
      tile_at(i, a.tiles_m, tiles_n, tm, tn);
      for (int kc = 0; kc < a.n_kc; ++kc, ++c) {
        const uint32_t s = c % C::NST;
        if (c >= C::NST && !warp_wait(empty + 8 * s, (c / C::NST - 1) & 1)) ok = false;
        if (__any_sync(0xffffffffu, *aborted)) ok = false;
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(full + 8 * s, ASTG + C::BSTG);
          tma_load_2d(sb + C::SM_A + s * ASTG, &mx, kc * LBK, tm * LBM, full + 8 * s);
          tma_load_2d(sb + C::SM_B + s * C::BSTG, &mw, kc * LBK, tn * BN, full + 8 * s);
        }
        __syncwarp();
      }
    }
    if (!ok) give_up();
    bool drained = true;  // every issued copy lands before the shared memory is released
    for (uint32_t s = 0; s < (uint32_t)C::NST && s < c; ++s)
      drained &= warp_wait(full + 8 * s, ((c - 1 - s) / C::NST) & 1);
    if (!drained) give_up();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16_f32(LBM, BN, false, false);
    const uint64_t da0 = smem_desc(sb + C::SM_A, 16, 1024, kSwizzle128B);
    const uint64_t db0 = smem_desc(sb + C::SM_B, 16, 1024, kSwizzle128B);
    uint32_t c = 0, t = 0;
    bool ok = true;
    for (int i = blockIdx.x; ok && i < a.tiles; i += gridDim.x, ++t) {
      const uint32_t buf = t & 1;
      if (t >= 2 && !warp_wait(acc_empty + 8 * buf, (t / 2 - 1) & 1)) ok = false;
      tc_fence_after();
      for (int kc = 0; ok && kc < a.n_kc; ++kc, ++c) {
        const uint32_t s = c % C::NST;
        if (!warp_wait(full + 8 * s, (c / C::NST) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t da = da0 + (uint64_t)((s * ASTG) >> 4), db = db0 + (uint64_t)((s * C::BSTG) >> 4);
#pragma unroll
          for (int kk = 0; kk < LBK / 16; ++kk)
            mma_bf16_ss(tmem + buf * BN, da + (uint64_t)(kk * 2), db + (uint64_t)(kk * 2), idesc,
                        (kc > 0 || kk > 0) ? 1u : 0u);
          mma_commit(empty + 8 * s);
          if (kc == a.n_kc - 1) mma_commit(acc_full + 8 * buf);
        }
        __syncwarp();
      }
    }
    if (!ok) give_up();
    if (elect_one()) mma_commit(drain);  // every issued product finishes before TMEM is freed
    __syncwarp();
    if (!warp_wait(drain, 0)) give_up();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int wq = warp & 3;
    uint32_t t = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < a.tiles; i += gridDim.x, ++t) {
      int tm, tn;
      tile_at(i, a.tiles_m, tiles_n, tm, tn);
      const uint32_t buf = t & 1;
      if (ok && !warp_wait(acc_full + 8 * buf, (t / 2) & 1)) ok = false;
      tc_fence_after();
      const int row = tm * LBM + wq * 32 + lane;
      const uint32_t src = tmem + ((uint32_t)(wq * 32) << 16) + buf * BN;
#pragma unroll 1
      for (int cc = 0; cc < BN; cc += 32) {
        uint32_t r[32];
        if (ok) {
          tmem_ld32(src + cc, r);
          tmem_ld_wait();
        }
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = ok ? __uint_as_float(r[k]) : NAN;
        const int col = tn * BN + cc;
        if (row < a.m && col < a.n) finish_row(a, v, row, col);
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (ok && elect_one()) mbar_arrive(acc_empty + 8 * buf);
      __syncwarp();
    }
    if (!ok) give_up();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
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

template <int BN>
int launch_tiled(const LinearArgs& p, int sms, cudaStream_t stream) {
  using C = LinCfg<BN>;
  CUtensorMap mx, mw;
  if (!encode_rows(&mx, p.x, (uint64_t)p.k, (uint64_t)p.m, LBM) ||
      !encode_rows(&mw, p.w, (uint64_t)p.k, (uint64_t)p.n, BN))
    return check_launch(cudaErrorInvalidValue);
  static FuncConfigured configured;
  if (!configured.ensure(reinterpret_cast<const void*>(linear_kernel<BN>), C::SMEM)) return PKV_ERR_LAUNCH;
  const int64_t tm = ((int64_t)p.m + LBM - 1) / LBM, tn = ((int64_t)p.n + BN - 1) / BN;
  if (tm * tn > 0x7fffffffL) return PKV_ERR_UNSUPPORTED;
  const uintptr_t odd = reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.residual);
  const uintptr_t odd_bias = reinterpret_cast<uintptr_t>(p.bias) & 3;
  LinArgs a{static_cast<__nv_bfloat16*>(p.y),
            Epilogue{static_cast<const __nv_bfloat16*>(p.bias), static_cast<const __nv_bfloat16*>(p.residual), p.activation},
            p.m, p.n, (p.k + LBK - 1) / LBK, (int)tm, (int)(tm * tn), p.n % 8 == 0 && (odd & 15) == 0 && odd_bias == 0,
            p.err_flag};
  const unsigned grid = (unsigned)(tm * tn < sms ? tm * tn : sms);
  linear_kernel<BN><<<grid, LTHREADS, C::SMEM, stream>>>(mx, mw, a);
  return check_launch(cudaGetLastError());
}

}  // namespace

int launch_linear(const LinearArgs& a, cudaStream_t stream) {
  if (a.m <= kFlatGemmMaxM) return launch_flat_linear(a, stream);
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  const int64_t tm = ((int64_t)a.m + LBM - 1) / LBM;
  auto tiles = [&](int bn) { return tm * (((int64_t)a.n + bn - 1) / bn); };
  if (tiles(256) >= sms) return launch_tiled<256>(a, sms, stream);
  if (tiles(128) >= sms) return launch_tiled<128>(a, sms, stream);
  return launch_tiled<64>(a, sms, stream);
}

}  // namespace pkv
