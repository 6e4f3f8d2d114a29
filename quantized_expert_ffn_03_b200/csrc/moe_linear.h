// moe_linear.h -- launch parameters of the dense product with its epilogue
// (moe_linear.cu), shared with the host code that checks the call.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// y[t][n] = act(x[t] . w[n] + bias[n]) [* (x[t] . w_up[n] + bias_up[n])] [+ res[t][n]]
// (8 bytes more of it cost calls of 3 to 8 us 3 to 4 percent.)
struct LinearParams {
  int T, K, N;
  int act;       // MOE_ACT_*
  int out_f32;   // output (and residual) fp32, else the 16-bit input type
  int vec;       // every row of out (and residual) starts on a 16-byte boundary (1), and N features end on one (2)
  int bias_vec;  // the biases start on 16-byte boundaries
  uint32_t err_slot;  // the error word of the call's stream (set by launch_linear)
  const uint16_t* x;
  const uint16_t* w;
  const uint16_t* w_up;  // null: not gated
  const float* bias;
  const float* bias_up;
  const void* res;
  void* out;
  int64_t ldx, ldw, ldw_up, ldr, ldo;
};

// A launch of `kernel` that may start before the kernel ahead of it in the
// stream has ended (it waits for that itself: prior_wait), with clusters of
// `cluster` blocks along x.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                         const A&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[2];
  a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a[0].val.programmaticStreamSerializationAllowed = 1;
  a[1].id = cudaLaunchAttributeClusterDimension;
  a[1].val.clusterDim.x = cluster;
  a[1].val.clusterDim.y = 1;
  a[1].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

// f16: the 16-bit type is fp16, else bf16.  sms: the device's SM count.
cudaError_t launch_linear(LinearParams p, bool f16, int sms, cudaStream_t st);
// Error words of the calls on a device; the word of the stream `st` is read and cleared.
constexpr int kLinearErrSlots = 1024;
cudaError_t read_linear_error(uint32_t* code, cudaStream_t st);
cudaError_t launch_linear_wait_probe(uint64_t limit_ns, cudaStream_t st);

// Expert choice from logits (moe_route.cu).
struct RouteParams {
  int T, E, K;
  int sigmoid;
  int n_groups, topk_groups, top2;
  int per;           // experts of a group
  uint32_t per_inv;  // ceil(2^32 / per): q / per as a high product, for per > 1
  int lane_shift;    // log2 of the lanes that share a group
  int bias_vec;      // the bias starts on a 16-byte boundary
  int vec;           // every row of logits is whole 16-byte pieces on 16-byte boundaries
  int renorm;
  float scale;
  const void* logits;
  int64_t ldl;
  const float* bias;
  int32_t* idx;
  float* w;
};
constexpr int kRouteMaxExperts = 2048;
constexpr int kRouteMaxGroups = 32;
// dtype: MOE_BF16, MOE_F16 or MOE_F32.
cudaError_t launch_route(const RouteParams& p, int dtype, cudaStream_t st);

}  // namespace moe
