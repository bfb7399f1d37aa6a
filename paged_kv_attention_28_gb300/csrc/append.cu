// Per-head RMS norm of the new queries and keys, their rotary position rotation, and the
// write of the new keys and values into the paged cache, in one pass.
//
// For a head row x of head_dim D (q and k; v is copied):
//   y   = x * rsqrt(mean(x^2) + eps) * w                     (where a norm weight is given)
//   z_a = y_a cos t - y_b sin t,  z_b = y_b cos t + y_a sin t  (each pair (a, b) of rotary_dim)
//   t   = position[axis of the pair] * inv_freq[pair]
// in fp32, rounded once to the row's type. Every element is read once and written once, so
// the call is bound by those bytes: 8192 tokens of 48 rows of 128 bf16, 201 MB, take 42 us, 4.8 TB/s, half of
// them (the rest padding) 22 to 30 us, by where the tensors lie in memory; 64 tokens 3.4 us, a launch. 62 % of the issue slots are taken, at 8 bytes an
// access in bf16 and a norm weight loaded and widened for every row: that is this code's, not the work's. Not kept:
// rows asked for two to four batches ahead through shared memory (1 to 15 % slower at twice the
// warps, so it is not the loads' latency), two tokens at a time that share addresses and weights (7 %
// slower: fewer warps).
//
// Angles: a position can be far (10^5 and more) and the angle matters modulo a full turn, so
// an fp32 product loses what is needed (2^-24 of 10^5 rad is 0.006 rad). A pair's frequency is
// taken as a 64-bit fixed-point fraction of a turn, F = frac(inv_freq / 2 pi) * 2^64, by an
// integer product of the fp32 significand with 94 bits of 1 / 2 pi; position * F in wrapping
// 64-bit integers is then the phase modulo one turn for any int32 position, off only by F's last
// bit, and sincospi of its leading bits gives cos and sin. No fp64 arithmetic, whose rate here is
// a 64th of fp32's.
//
// A CTA takes a few consecutive tokens of a sequence. Groups of D / 8 lanes take a token's rows
// (every query, key and value head), kRows each at a time, 8 elements a lane in two runs of 4 chosen
// so that both elements of a pair are in one lane: no exchange but the norm's sum. The next
// rows, the next token's too, are asked for before the present ones are worked on, and one
// thread per pair computes the next token's cos and sin into shared memory, which the rows of
// all heads share.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace pkv {
namespace {

constexpr int kRows = 3;  // rows of a lane group in flight
constexpr int kPage = 16;

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

// frac(f / 2 pi) * 2^64, f finite.
__device__ __forceinline__ uint64_t turn_fraction(float f) {
  // 2^96 / 2 pi, rounded down: 94 bits
  constexpr unsigned __int128 kTurns = ((unsigned __int128)0x28be60dbu << 64) | 0x9391054a7f09d5f4ull;
  const uint32_t u = __float_as_uint(f);
  const int field = (u >> 23) & 0xff;
  const uint32_t m = (u & 0x7fffffu) | (field ? 0x800000u : 0u);
  const int shift = 182 - (field ? field : 1);  // f = m 2^(field - 150), and 96 - 64 bits
  const unsigned __int128 p = kTurns * m;
  const uint64_t v = shift >= 128 ? 0 : shift >= 0 ? (uint64_t)(p >> shift) : shift > -64 ? (uint64_t)p << -shift : 0;
  return (u >> 31) ? 0 - v : v;
}

template <typename T, int D, int THREADS>
__global__ void __launch_bounds__(THREADS) append_kernel(const AppendArgs a, int per_cta) {
  using Q4 = Quad<T>;
  using Raw = typename Q4::Raw;
  constexpr int L = D / 8;             // lanes per row
  constexpr int GROUPS = THREADS / L;  // rows a CTA works on at a time
  __shared__ __align__(16) float s_cos[2][D / 2];
  __shared__ __align__(16) float s_sin[2][D / 2];
  const int tid = threadIdx.x;
  const int pairs = a.rotary_dim / 2;
  const int b = blockIdx.y, first = blockIdx.x * per_cta;
  wait_for_stream();
  const int len = __ldg(a.prefix_lens + b);
  const int n = a.chunk_lens ? __ldg(a.chunk_lens + b) : a.chunk_len;
  const bool bad_n = n < 0 || n > a.chunk_len;
  const int end = min(first + per_cta, bad_n ? a.chunk_len : n);  // tokens [first, end)
  const bool bad_len = bad_n || len < 0 || (int64_t)len + n > (int64_t)a.max_blocks * kPage;
  if (first >= end) {  // padding, perhaps all of the sequence: then nobody else would report its length
    if (bad_len && first == 0 && tid == 0) set_err(a.err_flag, PKV_DEVERR_BAD_LEN);
    return;
  }
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks;
  const int64_t t0 = (int64_t)b * a.chunk_len;  // the sequence's first token
  auto page_of = [&](int i) { return bad_len ? -1 : __ldg(table + (len + i) / kPage); };

  const int l = tid % L, group = tid / L;
  const int rows = a.n_qo_heads + 2 * a.n_kv_heads;
  const int batches = (rows + GROUPS * kRows - 1) / (GROUPS * kRows);  // of a token's rows
  // the lane's two runs of four elements, and whether they are rotated
  const bool turned = 8 * l < a.rotary_dim;
  const int o0 = !turned || a.interleaved ? 8 * l : 4 * l;
  const int o1 = !turned || a.interleaved ? 8 * l + 4 : pairs + 4 * l;
  auto load = [&](Raw (&lo)[kRows], Raw (&hi)[kRows], int i, int batch) {
    const int64_t t = t0 + i;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = (batch * kRows + u) * GROUPS + group;
      lo[u] = Raw{}, hi[u] = Raw{};
      if (r < rows) {
        const bool is_q = r < a.n_qo_heads, is_k = r < a.n_qo_heads + a.n_kv_heads;
        const int h = r - (is_q ? 0 : is_k ? a.n_qo_heads : a.n_qo_heads + a.n_kv_heads);
        const T* src = static_cast<const T*>(is_q ? a.q : is_k ? a.k : a.v) +
                       t * (is_q ? a.q_stride : is_k ? a.k_stride : a.v_stride) + (int64_t)h * D;
        lo[u] = *reinterpret_cast<const Raw*>(src + o0);
        hi[u] = *reinterpret_cast<const Raw*>(src + o1);
      }
    }
  };
  Raw next_lo[kRows], next_hi[kRows];
  load(next_lo, next_hi, first, 0);
  int next_page = page_of(first);

  uint64_t turn = 0;
  int axis = -1;  // -1: the pair's outputs are NaN
  if (tid < pairs) {
    const float f = __ldg(a.inv_freq + tid);
    axis = a.pair_axis ? __ldg(a.pair_axis + tid) : 0;
    if (axis < 0 || axis >= a.n_axes) {
      set_err(a.err_flag, PKV_DEVERR_BAD_AXIS);
      axis = -1;
    }
    if (!(fabsf(f) < INFINITY)) axis = -1;
    turn = turn_fraction(f);
  }
  auto angles = [&](int i) {
    if (tid < pairs) {
      float c = NAN, s = NAN;
      if (axis >= 0) {
        const int64_t pos =
            a.positions ? __ldg(a.positions + axis * ((int64_t)a.batch * a.chunk_len) + t0 + i) : (int64_t)len + i;
        const int64_t phase = (int64_t)((uint64_t)pos * turn);  // 2^64 to a turn
        sincospif((float)phase * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
      }
      s_cos[i & 1][tid] = c;
      s_sin[i & 1][tid] = s;
    }
  };
  angles(first);
  __syncthreads();

  for (int i = first; i < end; ++i) {
    int page = next_page;
    if (page < 0 || page >= a.num_pages) {
      page = -1;
      if (tid == 0) set_err(a.err_flag, bad_len ? PKV_DEVERR_BAD_LEN : PKV_DEVERR_BAD_PAGE);
    }
    const int64_t slot = (int64_t)page * a.n_kv_heads * kPage + (len + i) % kPage;  // of KV head 0
    for (int batch = 0; batch < batches; ++batch) {
      Raw lo[kRows], hi[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) lo[u] = next_lo[u], hi[u] = next_hi[u];
      if (batch + 1 < batches) {
        load(next_lo, next_hi, i, batch + 1);
      } else if (i + 1 < end) {
        load(next_lo, next_hi, i + 1, 0);
        next_page = page_of(i + 1);
        angles(i + 1);
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const int r = (batch * kRows + u) * GROUPS + group;
        const bool is_q = r < a.n_qo_heads, is_k = r < a.n_qo_heads + a.n_kv_heads;
        float v[8];
        Q4::get(lo[u], v, 0);
        Q4::get(hi[u], v, 4);
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (r >= rows) continue;
        if (is_k) {  // (queries too)
          const T* w = static_cast<const T*>(is_q ? a.q_norm : a.k_norm);
          if (w) {
            const float s = rsqrtf(ss * (1.0f / D) + a.eps);
            float wv[8];
            Q4::get(*reinterpret_cast<const Raw*>(w + o0), wv, 0);
            Q4::get(*reinterpret_cast<const Raw*>(w + o1), wv, 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * s * wv[e];
          }
          if (turned) {
            const float4 c4 = *reinterpret_cast<const float4*>(s_cos[i & 1] + 4 * l);
            const float4 s4 = *reinterpret_cast<const float4*>(s_sin[i & 1] + 4 * l);
            const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
            if (a.interleaved) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float xa = v[2 * j], xb = v[2 * j + 1];
                v[2 * j] = xa * c[j] - xb * s[j];
                v[2 * j + 1] = xb * c[j] + xa * s[j];
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float xa = v[j], xb = v[j + 4];
                v[j] = xa * c[j] - xb * s[j];
                v[j + 4] = xb * c[j] + xa * s[j];
              }
            }
          }
          if (is_q && page < 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = NAN;
          }
          lo[u] = Q4::put(v, 0);
          hi[u] = Q4::put(v, 4);
        }
        T* dst;
        if (is_q) {
          dst = static_cast<T*>(a.q_out) + ((t0 + i) * a.n_qo_heads + r) * D;
        } else {
          if (page < 0) continue;
          const int h = r - a.n_qo_heads - (is_k ? 0 : a.n_kv_heads);
          dst = static_cast<T*>(is_k ? a.k_pages : a.v_pages) + (slot + h * kPage) * D;
        }
        *reinterpret_cast<Raw*>(dst + o0) = lo[u];
        *reinterpret_cast<Raw*>(dst + o1) = hi[u];
      }
    }
    __syncthreads();  // the next token's angles are in, and this one's may be overwritten
  }
}

template <typename T, int D>
int launch_t(const AppendArgs& a, cudaStream_t stream) {
  int sms = device_sm_count();
  if (sms <= 0) sms = 148;
  // Few tokens: one per CTA of 256 threads, which puts most rows at work at once. Many: two per CTA
  // of 128 threads (one or four are 3 to 8 % slower, 256 or 64 threads 10 and 30 %).
  if ((int64_t)a.batch * a.chunk_len <= 16 * (int64_t)sms) {
    return check_launch(launch_overlapped(append_kernel<T, D, 256>, dim3((unsigned)a.chunk_len, (unsigned)a.batch), 256,
                                          0, stream, 1, a, 1));
  } else {
    constexpr int kPer = 2;
    const dim3 grid((unsigned)((a.chunk_len + kPer - 1) / kPer), (unsigned)a.batch);
    return check_launch(launch_overlapped(append_kernel<T, D, 128>, grid, 128, 0, stream, 1, a, kPer));
  }
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
