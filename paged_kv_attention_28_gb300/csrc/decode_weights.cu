// Paged decode that also accumulates the attention weight every cached token receives.
//
//   sums_out[b, g, t] = decay * sums_in[b, g, t] + sum over the heads h of group g of
//                       exp(s_ht - lse_h),   s_ht = scale q_h . k_t
//
// A weight needs its row's final log-sum-exp, which is known only after the last key. The
// decode kernel (LOGITS instantiations of the two decode kernels) keeps the logits it computes
// in fp32 scratch, 4 G bytes per key and KV head, written and read, where K and V are 4 D (bf16): for D = 128 1.6 %
// more traffic with one query head per KV head, 6.3 % with four (3.1 and 7.8 with the sums), most of it
// caught by the L2, where a second pass over K would cost half as much again as the decode. One more kernel then merges the split
// states of a row (a CTA each, as the plain decode's merge) and, in its other CTAs, forms the
// weights and updates the sums, reading and writing each once; those take a row's log-sum-exp
// straight from the splits', so that they need not wait for the merge.
//
// Bound: HBM, as the decode. 16 sequences of 0.5-4k tokens with 32 KV heads, 613 MB, take 100 us (6.1
// TB/s): the decode 93, this kernel 7, launched while the decode ends. 4 x 32k tokens with 4 heads on
// each of 8 KV heads, 545 MB: 99 us, the decode 90.
#include "decode_kernel.cuh"
#include "merge.cuh"

namespace pkv {

int dispatch_decode_logits(const DecodeArgs& a, cudaStream_t stream) {
  return dispatch_decode<false, true>(a, stream);
}

namespace {

constexpr int kFinishThreads = 128;
constexpr int kMergeWarps = kFinishThreads / 32;

// The log-sum-exp of n partial ones, by a warp; NaN if any is.
__device__ __forceinline__ float join_lse(const float* part, int n) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int i = lane; i < n; i += 32) m = fmaxf(m, __ldcg(part + i));
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  float l = 0.0f;
  for (int i = lane; i < n; i += 32) l += ex2((__ldcg(part + i) - m) * kLog2e);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
  return m + logf(l);
}

// CTAs [0, merge_rows): the merge of one output row each. The others: 4 kFinishThreads tokens of one
// (sequence, KV head), four consecutive ones a thread. The heads are added in order, so the sums
// do not depend on the launch.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kFinishThreads) finish_weights_kernel(const DecodeWeightsArgs a, int merge_rows,
                                                                        int tiles) {
  __shared__ float s_merge[kMergeWarps * (D + 3)];
  __shared__ float s_lse[G];
  const int P = a.d.page_size;
  const int64_t cap = (int64_t)a.d.max_blocks * P;  // a multiple of 16
  auto splits_of = [&](int len) { return ((len + P - 1) / P + a.d.pages_per_split - 1) / a.d.pages_per_split; };
  if ((int)blockIdx.x < merge_rows) {
    const int row = blockIdx.x;
    const int len = __ldg(a.d.kv_lens + row / a.d.n_qo_heads);
    wait_for_stream();  // (the decode)
    if (len < 0 || len > cap) return;
    const int n = splits_of(len);
    if (n < 2) return;  // the decode wrote the row
    const float* pl = a.d.part_lse + (int64_t)row * a.d.num_splits;
    const float* po = a.d.part_o + (int64_t)row * a.d.num_splits * D;
    merge_row_cta<T, D, kMergeWarps>(
        n, [&](int i) { return __ldcg(pl + i); }, [&](int i) { return po + (int64_t)i * D; },
        static_cast<T*>(a.d.out) + (int64_t)row * D, a.d.lse + row, s_merge);
    return;
  }
  const int idx = blockIdx.x - merge_rows;
  const int tile = idx % tiles, g = idx / tiles % a.d.n_kv_heads, b = idx / tiles / a.d.n_kv_heads;
  const int len = __ldg(a.d.kv_lens + b);  // (an input of the decode, like sums_in)
  const int64_t first = (int64_t)tile * kFinishThreads * 4, t = first + threadIdx.x * 4;
  const bool any = len <= cap && first < len, live = len <= cap && t < len;
  const int64_t at = ((int64_t)b * a.d.n_kv_heads + g) * cap + t;
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) w = *reinterpret_cast<const float4*>(a.sums_in + at);
  wait_for_stream();
  if (!any) return;
  const int64_t row0 = (int64_t)b * a.d.n_qo_heads + (int64_t)g * G;
  float4 x[G];
  if (live) {
#pragma unroll
    for (int h = 0; h < G; ++h) x[h] = __ldcg(reinterpret_cast<const float4*>(a.d.logits + (row0 + h) * cap + t));
  }
  const int n = splits_of(len);
  for (int h = threadIdx.x >> 5; h < G; h += kMergeWarps) {
    const float l = n < 2 ? __ldcg(a.d.lse + row0 + h) : join_lse(a.d.part_lse + (row0 + h) * a.d.num_splits, n);
    if ((threadIdx.x & 31) == 0) s_lse[h] = l;
  }
  __syncthreads();
  if (!live) return;
  w.x *= a.decay, w.y *= a.decay, w.z *= a.decay, w.w *= a.decay;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float m = -s_lse[h];
    w.x += ex2(fmaf(m, kLog2e, x[h].x));
    w.y += ex2(fmaf(m, kLog2e, x[h].y));
    w.z += ex2(fmaf(m, kLog2e, x[h].z));
    w.w += ex2(fmaf(m, kLog2e, x[h].w));
  }
  float* out = a.sums_out + at;
  if (t + 4 <= len) {
    *reinterpret_cast<float4*>(out) = w;
  } else {  // slots at or past the length are left as they were
    out[0] = w.x;
    if (t + 1 < len) out[1] = w.y;
    if (t + 2 < len) out[2] = w.z;
  }
}

template <typename T, int D, int G>
int launch_finish(const DecodeWeightsArgs& a, cudaStream_t stream) {
  const int64_t cap = (int64_t)a.d.max_blocks * a.d.page_size;
  const int64_t tiles = (cap + 4 * kFinishThreads - 1) / (4 * kFinishThreads);
  const int64_t rows = a.d.num_splits > 1 ? (int64_t)a.d.batch * a.d.n_qo_heads : 0;
  const int64_t grid = rows + tiles * a.d.n_kv_heads * a.d.batch;
  if (grid > 0x7fffffffL) return PKV_ERR_UNSUPPORTED;
  return check_launch(launch_overlapped(finish_weights_kernel<T, D, G>, dim3((unsigned)grid), kFinishThreads, 0, stream, 1, a,
                                        (int)rows, (int)tiles));
}

template <typename T, int D>
int launch_finish_any(const DecodeWeightsArgs& a, cudaStream_t stream) {
  switch (a.d.n_qo_heads / a.d.n_kv_heads) {
    case 1: return launch_finish<T, D, 1>(a, stream);
    case 2: return launch_finish<T, D, 2>(a, stream);
    case 4: return launch_finish<T, D, 4>(a, stream);
    case 8: return launch_finish<T, D, 8>(a, stream);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace

int launch_decode_weights(const DecodeWeightsArgs& a, cudaStream_t stream) {
  const int rc = launch_decode_partials(a.d, stream);
  if (rc != PKV_OK) return rc;
  if (a.d.dtype == PKV_F32)
    return a.d.head_dim == 64 ? launch_finish_any<float, 64>(a, stream) : launch_finish_any<float, 128>(a, stream);
  return a.d.head_dim == 64 ? launch_finish_any<__nv_bfloat16, 64>(a, stream)
                            : launch_finish_any<__nv_bfloat16, 128>(a, stream);
}

}  // namespace pkv
