// moe_route.cu -- expert choice from router logits (moe_route_from_logits):
// scores, selection bias, groups, top-K, weights.  One warp per token.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include "../../include/moe.h"
#include "moe_linear.h"

namespace moe {

namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load_logit(const __half* p) { return __half2float(*p); }

// Doubles as integers in the same order; zeros of both signs are equal, and no
// value maps to 0, which stands for "none".
__device__ __forceinline__ uint64_t order64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double rank64(double v) { return v != v ? -INFINITY : v; }

// The largest key of the warp and, among its holders, the lowest index.
__device__ __forceinline__ void warp_best(uint64_t& key, int& at) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t k = __shfl_xor_sync(kAll, key, o);
    const int a = __shfl_xor_sync(kAll, at, o);
    if (k > key || (k == key && a < at)) key = k, at = a;
  }
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

template <typename T>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(const RouteParams p) {
  extern __shared__ uint64_t keys_all[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t* key = keys_all + (size_t)warp * p.E;
  const int per = p.E / p.n_groups;
#pragma unroll 1
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < p.T; t += (int64_t)gridDim.x * kRouteWarps) {
    const T* row = static_cast<const T*>(p.logits) + (size_t)t * p.ldl;
    auto logit = [&](int e) {
      const float l = load_logit(row + e);
      return l != l ? -INFINITY : fminf(l, FLT_MAX);
    };
    float top = -INFINITY;
    double sum = 0.0;
    if (!p.sigmoid) {
      for (int e = lane; e < p.E; e += 32) top = fmaxf(top, logit(e));
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
      if (top == -INFINITY) top = 0.f;  // a row of -inf: every score is 0
      for (int e = lane; e < p.E; e += 32) sum += exp((double)logit(e) - (double)top);
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
      if (sum == 0.0) sum = 1.0;
    }
    auto score = [&](float l) { return p.sigmoid ? sigmoid64((double)l) : exp((double)l - (double)top) / sum; };
    const bool by_value = p.bias != nullptr;
    auto value = [&](int e) { return rank64(score(logit(e)) + (by_value ? (double)__ldg(p.bias + e) : 0.0)); };
    // the order of experts: by value, or by logit where the score alone decides
    for (int e = lane; e < p.E; e += 32) key[e] = order64(by_value ? value(e) : (double)logit(e));
    __syncwarp();
    uint32_t kept = kAll;
    if (p.n_groups > 1) {
      uint64_t gk = 0;
      if (lane < p.n_groups) {
        double a = -INFINITY, b = -INFINITY;
        for (int j = 0; j < per; ++j) {
          const double v = value(lane * per + j);
          if (v > a)
            b = a, a = v;
          else if (v > b)
            b = v;
        }
        gk = order64(p.top2 && per > 1 ? rank64(a + b) : a);
      }
      kept = 0;
      for (int i = 0; i < p.topk_groups; ++i) {
        uint64_t k = kept >> lane & 1u ? 0ull : gk;
        int at = lane;
        warp_best(k, at);
        kept |= 1u << at;
      }
    }
    double mine = 0.0, total = 0.0;  // lane k: the score of choice k
    int chosen = 0;
    for (int k = 0; k < p.K; ++k) {
      uint64_t best = 0;
      int at = p.E;
      for (int e = lane; e < p.E; e += 32)
        if (key[e] > best && (p.n_groups == 1 || (kept >> (e / per) & 1u))) best = key[e], at = e;
      warp_best(best, at);
      if (lane == (at & 31)) key[at] = 0;
      const double s = score(logit(at));
      total += s;
      if (lane == k) mine = s, chosen = at;
      __syncwarp();
    }
    if (lane < p.K) {
      const double w = p.renorm ? (total > 0.0 ? mine / total : 0.0) : mine;
      p.idx[(size_t)t * p.K + lane] = chosen;
      p.w[(size_t)t * p.K + lane] = (float)(w * (double)p.scale);
    }
    __syncwarp();
  }
}

template <typename T>
cudaError_t launch_route_t(const RouteParams& p, int sms, cudaStream_t st) {
  const size_t smem = sizeof(uint64_t) * kRouteWarps * (size_t)p.E;
  cudaError_t e = cudaFuncSetAttribute(route_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)(sizeof(uint64_t) * kRouteWarps * kRouteMaxExperts));
  if (e != cudaSuccess) return e;
  const int64_t blocks = ((int64_t)p.T + kRouteWarps - 1) / kRouteWarps;
  const int grid = (int)(blocks < 32 * sms ? blocks : 32 * sms);
  route_kernel<T><<<grid, 32 * kRouteWarps, smem, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int dtype, int sms, cudaStream_t st) {
  if (dtype == MOE_F32) return launch_route_t<float>(p, sms, st);
  if (dtype == MOE_BF16) return launch_route_t<__nv_bfloat16>(p, sms, st);
  return launch_route_t<__half>(p, sms, st);
}

}  // namespace moe
