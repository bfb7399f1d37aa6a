// Per-head RMS norm of the new queries and keys, their rotary position rotation, and the
// write of the new keys and values into the paged cache, in one pass.
//
// For a head row x of head_dim D (q and k; v is copied):
//   y   = x * rsqrt(mean(x^2) + eps) * w                     (where a norm weight is given)
//   z_a = y_a cos t - y_b sin t,  z_b = y_b cos t + y_a sin t  (each pair (a, b) of rotary_dim)
//   t   = position[axis of the pair] * inv_freq[pair]
// in fp32, rounded once to the row's type. Every element is read once and written once, so
// the call is bound by those bytes.
//
// Angles: a position can be far (10^5 and more) and the angle matters modulo a full turn, so
// an fp32 product loses what is needed (2^-24 of 10^5 rad is 0.006 rad). A pair's frequency is
// kept as a 64-bit fixed-point fraction of a turn, F = frac(inv_freq / 2 pi) * 2^64 (one fp64
// product per pair and CTA); position * F in wrapping 64-bit integers is then the exact phase
// modulo one turn for any int32 position, off only by F's own rounding (2^-53 relative), and
// sincospi of its leading bits gives cos and sin. No fp64 arithmetic per token.
//
// A CTA takes TOK tokens. Its threads first compute the tokens' cos and sin into shared memory,
// one (token, pair) each, so that the rows of all heads share them; then groups of D / 8 lanes
// take the rows (every query, key and value head of every token), 8 elements a lane in two
// runs of 4 chosen so that both elements of a pair are in one lane: no exchange but the norm's
// sum. kRows rows per group are loaded before any is used, to keep enough bytes in flight.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 3;  // rows of a lane group in flight

// Four consecutive elements of T as one access.
template <typename T>
struct Quad;
template <>
struct Quad<float> {
  using Raw = float4;
  static __device__ __forceinline__ void get(const Raw& r, float (&x)[8], int at) {
    x[at] = r.x, x[at + 1] = r.y, x[at + 2] = r.z, x[at + 3] = r.w;
  }
  static __device__ __forceinline__ Raw put(const float (&x)[8], int at) {
    return make_float4(x[at], x[at + 1], x[at + 2], x[at + 3]);
  }
};
template <>
struct Quad<__nv_bfloat16> {
  using Raw = uint2;
  static __device__ __forceinline__ void get(const Raw& r, float (&x)[8], int at) {
    x[at] = __uint_as_float(r.x << 16), x[at + 1] = __uint_as_float(r.x & 0xffff0000u);
    x[at + 2] = __uint_as_float(r.y << 16), x[at + 3] = __uint_as_float(r.y & 0xffff0000u);
  }
  static __device__ __forceinline__ Raw put(const float (&x)[8], int at) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[at], x[at + 1]), b = __floats2bfloat162_rn(x[at + 2], x[at + 3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
};

// What a token of the CTA does.
struct Token {
  int64_t in;    // index in [batch][chunk_len], or -1: nothing (padding)
  int64_t page;  // (page * n_kv_heads) * page_size + slot of its K and V rows, or -1: bad
};

template <typename T, int D, int TOK>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  using Q4 = Quad<T>;
  using Raw = typename Q4::Raw;
  constexpr int L = D / 8;              // lanes per row
  constexpr int GROUPS = kThreads / L;  // rows a CTA works on at a time
  __shared__ uint64_t s_freq[D / 2];
  __shared__ int s_axis[D / 2];
  __shared__ float2 s_cs[TOK][D / 2];
  __shared__ Token s_tok[TOK];
  __shared__ int s_live;
  const int tid = threadIdx.x;
  const int pairs = a.rotary_dim / 2;
  const int64_t n_tokens = (int64_t)a.batch * a.chunk_len;
  const int64_t t0 = (int64_t)blockIdx.x * TOK;

  if (tid == 0) s_live = 0;
  __syncthreads();
  if (tid < TOK && t0 + tid < n_tokens) {
    const int64_t t = t0 + tid;
    const int b = (int)(t / a.chunk_len), i = (int)(t % a.chunk_len);
    const int64_t len = __ldg(a.prefix_lens + b);
    const int64_t n = a.chunk_lens ? __ldg(a.chunk_lens + b) : a.chunk_len;
    Token k{-1, -1};
    if (len < 0 || n < 0 || n > a.chunk_len || len + n > (int64_t)a.max_blocks * a.page_size) {
      set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
      if (n < 0 || n > a.chunk_len || i < n) k.in = t;
    } else if (i < n) {
      const int64_t at = len + i;
      const int page = __ldg(a.block_table + (int64_t)b * a.max_blocks + at / a.page_size);
      k.in = t;
      if (page < 0 || page >= a.num_pages)
        set_err(a.err_flag, PKV_DEVERR_BAD_PAGE);
      else
        k.page = (int64_t)page * a.n_kv_heads * a.page_size + at % a.page_size;
    }
    s_tok[tid] = k;
    if (k.in >= 0) s_live = 1;
  } else if (tid < TOK) {
    s_tok[tid] = Token{-1, -1};
  }
  if (tid >= kThreads - pairs) {  // (pairs <= 64: not the threads that look the tokens up)
    const int p = tid - (kThreads - pairs);
    const float f = __ldg(a.inv_freq + p);
    const double turns = (double)f * 0.15915494309189535;  // 1 / (2 pi)
    s_freq[p] = (uint64_t)((turns - floor(turns)) * 18446744073709551616.0);
    int axis = a.pair_axis ? __ldg(a.pair_axis + p) : 0;
    if (axis < 0 || axis >= a.n_axes) {
      set_err(a.err_flag, PKV_DEVERR_BAD_AXIS);
      axis = -1;
    }
    s_axis[p] = fabsf(f) < INFINITY ? axis : -1;  // -1: the pair's outputs are NaN
  }
  __syncthreads();
  if (!s_live) return;
  for (int x = tid; x < TOK * pairs; x += kThreads) {
    const int k = x / pairs, p = x % pairs;
    const int64_t t = s_tok[k].in;
    if (t < 0) continue;
    const int axis = s_axis[p];
    float2 cs = make_float2(NAN, NAN);
    if (axis >= 0) {
      const int64_t pos = a.positions ? __ldg(a.positions + axis * n_tokens + t)
                                      : (int64_t)__ldg(a.prefix_lens + t / a.chunk_len) + t % a.chunk_len;
      const int64_t phase = (int64_t)((uint64_t)pos * s_freq[p]);  // 2^64 to a turn
      sincospif((float)phase * 1.0842021724855044e-19f, &cs.y, &cs.x);  // 2^-63: half turns
    }
    s_cs[k][p] = cs;
  }
  __syncthreads();

  const int l = tid % L, group = tid / L;
  const int rows = a.n_qo_heads + 2 * a.n_kv_heads;
  // the lane's two runs of four elements, and whether they are rotated
  const bool turned = 8 * l < a.rotary_dim;
  const int o0 = !turned || a.interleaved ? 8 * l : 4 * l;
  const int o1 = !turned || a.interleaved ? 8 * l + 4 : pairs + 4 * l;
  for (int base = 0; base < TOK * rows; base += GROUPS * kRows) {
    Raw lo[kRows], hi[kRows];
    int kind[kRows];  // 0 q, 1 k, 2 v, -1 nothing
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int x = base + u * GROUPS + group;
      const int k = x / rows, r = x % rows;
      kind[u] = -1;
      lo[u] = Raw{}, hi[u] = Raw{};
      if (x < TOK * rows && s_tok[k].in >= 0) {
        const int64_t t = s_tok[k].in;
        kind[u] = r < a.n_qo_heads ? 0 : r < a.n_qo_heads + a.n_kv_heads ? 1 : 2;
        const int h = r - (kind[u] == 0 ? 0 : kind[u] == 1 ? a.n_qo_heads : a.n_qo_heads + a.n_kv_heads);
        const T* src = static_cast<const T*>(kind[u] == 0 ? a.q : kind[u] == 1 ? a.k : a.v) +
                       t * (kind[u] == 0 ? a.q_stride : kind[u] == 1 ? a.k_stride : a.v_stride) + (int64_t)h * D;
        lo[u] = *reinterpret_cast<const Raw*>(src + o0);
        hi[u] = *reinterpret_cast<const Raw*>(src + o1);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int x = base + u * GROUPS + group;
      const int k = min(x / rows, TOK - 1), r = x % rows;
      const T* w = static_cast<const T*>(kind[u] == 0 ? a.q_norm : a.k_norm);
      float v[8];
      Q4::get(lo[u], v, 0);
      Q4::get(hi[u], v, 4);
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
      for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (kind[u] < 0) continue;
      const Token tok = s_tok[k];
      if (kind[u] < 2) {
        if (w) {
          const float s = rsqrtf(ss * (1.0f / D) + a.eps);
          float wv[8];
          Q4::get(*reinterpret_cast<const Raw*>(w + o0), wv, 0);
          Q4::get(*reinterpret_cast<const Raw*>(w + o1), wv, 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = v[e] * s * wv[e];
        }
        if (turned) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 cs = s_cs[k][4 * l + j];
            const float xa = a.interleaved ? v[2 * j] : v[j], xb = a.interleaved ? v[2 * j + 1] : v[j + 4];
            const float za = xa * cs.x - xb * cs.y, zb = xb * cs.x + xa * cs.y;
            if (a.interleaved)
              v[2 * j] = za, v[2 * j + 1] = zb;
            else
              v[j] = za, v[j + 4] = zb;
          }
        }
        if (kind[u] == 0 && tok.page < 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = NAN;
        }
        lo[u] = Q4::put(v, 0);
        hi[u] = Q4::put(v, 4);
      }
      T* dst;
      if (kind[u] == 0) {
        dst = static_cast<T*>(a.q_out) + (tok.in * a.n_qo_heads + r) * D;
      } else {
        if (tok.page < 0) continue;
        const int h = r - a.n_qo_heads - (kind[u] == 2 ? a.n_kv_heads : 0);
        dst = static_cast<T*>(kind[u] == 1 ? a.k_pages : a.v_pages) + (tok.page + (int64_t)h * a.page_size) * D;
      }
      *reinterpret_cast<Raw*>(dst + o0) = lo[u];
      *reinterpret_cast<Raw*>(dst + o1) = hi[u];
    }
  }
}

template <typename T, int D>
int launch_t(const AppendArgs& a, cudaStream_t stream) {
  const int64_t n = (int64_t)a.batch * a.chunk_len;
  // Few tokens: one per CTA, so that they spread over the SMs. Many: four, so that a thread
  // computes about one angle and the rows dominate.
  if (n <= 1024)
    append_kernel<T, D, 1><<<(unsigned)n, kThreads, 0, stream>>>(a);
  else
    append_kernel<T, D, 4><<<(unsigned)((n + 3) / 4), kThreads, 0, stream>>>(a);
  return check_launch(cudaGetLastError());
}

}  // namespace

int launch_append(const AppendArgs& a, cudaStream_t stream) {
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
