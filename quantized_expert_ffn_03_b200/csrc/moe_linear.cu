// moe_linear.cu -- dense product with its epilogue (moe_linear_forward):
//   y[t][n] = act(x[t] . w[n] + bias[n]) [* (x[t] . w_up[n] + bias_up[n])] [+ res[t][n]]
// fp32 accumulation and epilogue, one rounding to the output type.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/moe.h"
#include "moe_linear.h"

namespace moe {

namespace {

// ---- epilogue arithmetic ------------------------------------------------------------

// The activation in fp32.  tanh-GELU is v * sigmoid(2u), the same value
// without the cancellation of 1 + tanh(u) at negative u; GELU takes the
// normal CDF for the same reason.  NaN passes through all of them.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case MOE_ACT_SILU:
      return __fdividef(v, 1.f + __expf(-v));
    case MOE_ACT_GELU:
      return v * normcdff(v);
    case MOE_ACT_GELU_TANH:
      return __fdividef(v, 1.f + __expf(-1.5957691216057308f * fmaf(0.044715f * v * v, v, v)));
    case MOE_ACT_RELU:
      return v < 0.f ? 0.f : v;
    default:
      return v;
  }
}

template <bool F16>
__device__ __forceinline__ float from16(uint16_t u) {
  if constexpr (F16)
    return __half2float(__ushort_as_half(u));
  else
    return __uint_as_float((uint32_t)u << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t to16(float v) {
  if constexpr (F16)
    return __half_as_ushort(__float2half_rn(v));
  else
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// One output from its sums: bias, activation, gate, residual, store.  The
// residual is read before the store, so out may be the residual buffer.
template <bool F16>
__device__ __forceinline__ void finish_one(const LinearParams& p, int t, int n, float g, float u) {
  if (p.bias) g += __ldg(p.bias + n);
  float y = activate(g, p.act);
  if (p.w_up) y *= p.bias_up ? u + __ldg(p.bias_up + n) : u;
  const size_t o = (size_t)t * p.ldo + n;
  if (p.out_f32) {
    if (p.res) y += static_cast<const float*>(p.res)[(size_t)t * p.ldr + n];
    static_cast<float*>(p.out)[o] = y;
  } else {
    if (p.res) y += from16<F16>(static_cast<const uint16_t*>(p.res)[(size_t)t * p.ldr + n]);
    static_cast<uint16_t*>(p.out)[o] = to16<F16>(y);
  }
}

// ---- few tokens: weights streamed once through registers ------------------------------

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 elements of a row from column k (a multiple of 8); columns from K on read
// as zero and are never touched in memory.
__device__ __forceinline__ uint4 row8(const uint16_t* row, int k, int K, bool live) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (!live || k >= K) return v;
  if (k + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t h[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (k + i < K) h[i >> 1] |= (uint32_t)__ldg(row + k + i) << (16 * (i & 1));
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// A block takes 16 features (the M of m16n8k16 steps) and 8 tokens; its 8
// warps take the 64-column units of K in turn.  Lane (g, t) of a warp loads
// 16 bytes of rows g and g + 8 at columns 8t.. of a 32-column half unit: the
// order of columns within a sum is free, so those 8 values serve as the
// fragments of two k16 steps without a shuffle, and x is loaded the same way.
constexpr int kRowsFeat = 16, kRowsTok = 8, kRowsWarps = 8;
template <bool F16, bool GATED>
__global__ void __launch_bounds__(32 * kRowsWarps) linear_rows_kernel(const LinearParams p) {
  constexpr int NA = GATED ? 2 : 1;
  __shared__ float red[kRowsWarps][NA][kRowsTok][kRowsFeat + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRowsFeat;
  const int ntt = (p.T + kRowsTok - 1) / kRowsTok;
#pragma unroll 1
  for (int tt = blockIdx.y; tt < ntt; tt += gridDim.y) {
    const int t0 = tt * kRowsTok;
    float acc[NA][4] = {};
    const bool xl = t0 + g < p.T;
    const uint16_t* xr = p.x + (size_t)(xl ? t0 + g : 0) * p.ldx;
    const bool l0 = n0 + g < p.N, l1 = n0 + g + 8 < p.N;
    const uint16_t* w0[NA];
    const uint16_t* w1[NA];
    w0[0] = p.w + (size_t)(l0 ? n0 + g : 0) * p.ldw;
    w1[0] = p.w + (size_t)(l1 ? n0 + g + 8 : 0) * p.ldw;
    if constexpr (GATED) {
      w0[1] = p.w_up + (size_t)(l0 ? n0 + g : 0) * p.ldw_up;
      w1[1] = p.w_up + (size_t)(l1 ? n0 + g + 8 : 0) * p.ldw_up;
    }
#pragma unroll 2
    for (int k = 64 * warp; k < p.K; k += 64 * kRowsWarps) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int kk = k + 32 * h + 8 * t;
        const uint4 xv = row8(xr, kk, p.K, xl);
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          const uint4 v0 = row8(w0[a], kk, p.K, l0), v1 = row8(w1[a], kk, p.K, l1);
          mma16816<F16>(acc[a], v0.x, v1.x, v0.y, v1.y, xv.x, xv.y);
          mma16816<F16>(acc[a], v0.z, v1.z, v0.w, v1.w, xv.z, xv.w);
        }
      }
    }
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      red[warp][a][2 * t][g] = acc[a][0];
      red[warp][a][2 * t + 1][g] = acc[a][1];
      red[warp][a][2 * t][g + 8] = acc[a][2];
      red[warp][a][2 * t + 1][g + 8] = acc[a][3];
    }
    __syncthreads();
    if (threadIdx.x < kRowsFeat * kRowsTok) {
      const int f = threadIdx.x % kRowsFeat, c = threadIdx.x / kRowsFeat;
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) s[a] += red[w][a][c][f];
      if (n0 + f < p.N && t0 + c < p.T) finish_one<F16>(p, t0 + c, n0 + f, s[0], s[1]);
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, bool f16, int sms, cudaStream_t st) {
  (void)sms;
  const int ntt = (p.T + kRowsTok - 1) / kRowsTok;
  const dim3 grid((p.N + kRowsFeat - 1) / kRowsFeat, ntt < 65535 ? ntt : 65535);
  if (p.w_up) {
    if (f16)
      linear_rows_kernel<true, true><<<grid, 32 * kRowsWarps, 0, st>>>(p);
    else
      linear_rows_kernel<false, true><<<grid, 32 * kRowsWarps, 0, st>>>(p);
  } else {
    if (f16)
      linear_rows_kernel<true, false><<<grid, 32 * kRowsWarps, 0, st>>>(p);
    else
      linear_rows_kernel<false, false><<<grid, 32 * kRowsWarps, 0, st>>>(p);
  }
  return cudaGetLastError();
}

// The error word of the calls on a device: the first expired wait's code.
__device__ uint32_t g_linear_err;

cudaError_t read_linear_error(uint32_t* code, cudaStream_t st) {
  uint32_t zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(code, g_linear_err, 4, 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *code) {
    e = cudaMemcpyToSymbolAsync(g_linear_err, &zero, 4, 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

}  // namespace moe
