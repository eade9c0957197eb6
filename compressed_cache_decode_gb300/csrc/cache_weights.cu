// cache_weights.cu — attention weights of a decode step summed over the heads
// into one number per cache row, the measure lrkv_evict goes by: the shared
// row serves every head, so a row is worth what all of them looked at it.
//
//   w'[j] = decay w[j] + sum_h exp(s_hj - lse_h)
//
// The scan left every score s_hj (log2 domain, fp32); once the merge has the
// log-sum-exp a thread takes a row, reads its H scores (consecutive threads
// consecutive rows) and adds the weights up in fp32 in the order of the heads:
// no atomics, the same sum every time.  Bound by latency: the scores were
// written just before and come from L2 (33 MB of the 129 MB for 4 x 64K rows
// of 32 heads).  The whole call takes 326 us there, 64 us of them more than the
// cache's bytes at the copy rate.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "cache_weights.h"
#include "decode_common.cuh"
#include "ptx.cuh"

namespace lrkv {

using namespace dec;

namespace {

constexpr int kSumThreads = 256;

}  // namespace

__global__ void __launch_bounds__(kSumThreads)
    lrkv_weights_sum_kernel(int H, int max_len, const int32_t* seq_lens, const float* scores, const float* lse,
                            float decay, const float* weights, float* weights_out) {
  extern __shared__ float s_lse[];  // [H], log2 domain
  pdl_trigger();
  pdl_wait();
  const int b = blockIdx.y;
  const int L = min(max(seq_lens[b], 0), max_len);
  if (static_cast<int>(blockIdx.x) * kSumThreads >= L) return;
  for (int h = threadIdx.x; h < H; h += kSumThreads) s_lse[h] = lse[static_cast<size_t>(b) * H + h] * kLog2e;
  __syncthreads();
  const int j = blockIdx.x * kSumThreads + threadIdx.x;
  if (j >= L) return;
  const float* s = scores + static_cast<size_t>(b) * H * max_len + j;
  float sum = 0.f;
#pragma unroll 8
  for (int h = 0; h < H; ++h) sum += exp2f(s[static_cast<size_t>(h) * max_len] - s_lse[h]);
  const size_t at = static_cast<size_t>(b) * max_len + j;
  // the new token's row has no earlier weight (its slot may hold anything)
  if (decay != 0.f && j < L - 1) sum = fmaf(decay, weights[at], sum);
  weights_out[at] = sum;
}

lrkv_status weights_sum_launch(int B, int H, int max_len, const int32_t* seq_lens, const float* scores,
                               const float* lse, float decay, const float* weights, float* weights_out,
                               void* stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((max_len + kSumThreads - 1) / kSumThreads, B);
  cfg.blockDim = dim3(kSumThreads);
  cfg.dynamicSmemBytes = H * 4;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lrkv_weights_sum_kernel, H, max_len, seq_lens, scores, lse, decay, weights,
                            weights_out) == cudaSuccess
             ? LRKV_OK
             : LRKV_ERR_CUDA;
}

}  // namespace lrkv
