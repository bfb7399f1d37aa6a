// Paged decode that also accumulates the attention weight every cached token receives.
//
//   sums_out[b, g, t] = decay * sums_in[b, g, t] + sum over the heads h of group g of
//                       exp(s_ht - lse_h),   s_ht = scale q_h . k_t
//
// A weight needs its row's final log-sum-exp, which is known only after the last key. The
// decode kernel (LOGITS instantiations of the two decode kernels) keeps the logits it computes
// in fp32 scratch, 4 G bytes per key and KV head where K and V are 4 D (bf16): 3 % more traffic
// for one query head per KV head, 6 % for four, most of it caught by the L2, where a second
// pass over K would cost half as much again as the decode. The pass over the scratch then
// forms the weights and updates the sums, reading and writing each once.
#include "decode_kernel.cuh"

namespace pkv {

int dispatch_decode_logits(const DecodeArgs& a, cudaStream_t stream) {
  return dispatch_decode<false, true>(a, stream);
}

namespace {

constexpr int kFinishThreads = 128;

// One thread: four consecutive tokens of one (sequence, KV head). The heads are added in
// order, so the sums do not depend on the launch.
template <int G>
__global__ void __launch_bounds__(kFinishThreads) finish_weights_kernel(const DecodeWeightsArgs a) {
  const int64_t cap = (int64_t)a.d.max_blocks * a.d.page_size;  // a multiple of 16
  const int b = blockIdx.z, g = blockIdx.y;
  const int64_t t = ((int64_t)blockIdx.x * kFinishThreads + threadIdx.x) * 4;
  const int len = __ldg(a.d.kv_lens + b);  // (an input of the decode, like sums_in)
  const bool live = len <= cap && t < len;
  const int64_t at = ((int64_t)b * a.d.n_kv_heads + g) * cap + t;
  float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
  if (live) w = *reinterpret_cast<const float4*>(a.sums_in + at);
  // launched as a programmatic dependent: the decode and the merge are complete after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) return;
  const int64_t row0 = (int64_t)b * a.d.n_qo_heads + (int64_t)g * G;
  float4 x[G];
  float l[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    x[h] = __ldcg(reinterpret_cast<const float4*>(a.d.logits + (row0 + h) * cap + t));
    l[h] = __ldcg(a.d.lse + row0 + h);
  }
  w.x *= a.decay, w.y *= a.decay, w.z *= a.decay, w.w *= a.decay;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float m = -l[h];
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

template <int G>
int launch_finish(const DecodeWeightsArgs& a, cudaStream_t stream) {
  const int64_t cap = (int64_t)a.d.max_blocks * a.d.page_size;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((cap + 4 * kFinishThreads - 1) / (4 * kFinishThreads)), (unsigned)a.d.n_kv_heads,
                     (unsigned)a.d.batch);
  cfg.blockDim = dim3(kFinishThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return check_launch(cudaLaunchKernelEx(&cfg, finish_weights_kernel<G>, a));
}

}  // namespace

int launch_decode_weights(const DecodeWeightsArgs& a, cudaStream_t stream) {
  const int rc = launch_decode(a.d, stream);
  if (rc != PKV_OK) return rc;
  switch (a.d.n_qo_heads / a.d.n_kv_heads) {
    case 1: return launch_finish<1>(a, stream);
    case 2: return launch_finish<2>(a, stream);
    case 4: return launch_finish<4>(a, stream);
    case 8: return launch_finish<8>(a, stream);
    default: return PKV_ERR_UNSUPPORTED;
  }
}

}  // namespace pkv
