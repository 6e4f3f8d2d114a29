// moe_linear.cu -- dense product with its epilogue (moe_linear_forward):
//   y[t][n] = act(x[t] . w[n] + bias[n]) [* (x[t] . w_up[n] + bias_up[n])] [+ res[t][n]]
// fp32 accumulation and epilogue, one rounding to the output type.
//
// Three kernels, one per regime of T (choose_* below):
//   rows   few tokens: the weights stream once through registers into
//          m16n8k16 steps (HBM bound);
//   split  up to a few hundred tokens: 128 features x all tokens per cluster,
//          TMA -> tcgen05, K split over the cluster's CTAs and joined through
//          distributed shared memory (HBM / L2 bound);
//   pair   many tokens: persistent pairs of CTAs, 256-token tiles, tcgen05
//          with both CTAs' operands, epilogue under the next tile's MMAs
//          (tensor bound).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_linear.h"
#include "moe_tc.cuh"

namespace moe {

// The error word of the calls on a device: the first expired wait's code.
__device__ uint32_t g_linear_err;

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kKB = 64;  // columns of K per step: 128 bytes, one swizzle row

// ---- epilogue arithmetic ------------------------------------------------------------

// The activation in fp32, one switch for N values (a switch for each value
// fills the instruction cache once the loops around it are unrolled).
// tanh-GELU is v * sigmoid(2u), the same value without the cancellation of
// 1 + tanh(u) at negative u; GELU takes the normal CDF for the same reason.
// NaN passes through all of them.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  switch (act) {
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __fdividef(v[i], 1.f + __expf(-v[i]));
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= normcdff(v[i]);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] = __fdividef(v[i], 1.f + __expf(-1.5957691216057308f * fmaf(0.044715f * v[i] * v[i], v[i], v[i])));
      break;
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
      break;
    default:
      break;
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

// Two values rounded to 16 bits, a in the low half (one instruction, where two
// single conversions go to the slow conversion pipe).
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// One output from its sums: bias, activation, gate, residual, store.  The
// residual is read before the store, so out may be the residual buffer.
template <bool F16>
__device__ __forceinline__ void finish_one(const LinearParams& p, int t, int n, float g, float u) {
  if (p.bias) g += __ldg(p.bias + n);
  float a[1] = {g};
  activate(a, p.act);
  float y = a[0];
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

// W (4 or 8) adjacent values of a row of out or residual, on a boundary of
// their size.
template <bool F16, int W>
__device__ __forceinline__ void load_row(const LinearParams& p, const void* base, size_t at, float (&v)[W]) {
  if (p.out_f32) {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const float4 e = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at + i);
      v[i] = e.x, v[i + 1] = e.y, v[i + 2] = e.z, v[i + 3] = e.w;
    }
  } else {
    uint32_t w[W / 2];
    const uint16_t* src = static_cast<const uint16_t*>(base) + at;
    if constexpr (W == 8) {
      const uint4 e = *reinterpret_cast<const uint4*>(src);
      w[0] = e.x, w[1] = e.y, w[2] = e.z, w[3] = e.w;
    } else {
      const uint2 e = *reinterpret_cast<const uint2*>(src);
      w[0] = e.x, w[1] = e.y;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = from16<F16>((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
  }
}
template <bool F16, int W>
__device__ __forceinline__ void store_row(const LinearParams& p, size_t at, const float (&v)[W]) {
  if (p.out_f32) {
#pragma unroll
    for (int i = 0; i < W; i += 4)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    uint32_t w[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) w[i] = pack16<F16>(v[2 * i], v[2 * i + 1]);
    uint16_t* dst = static_cast<uint16_t*>(p.out) + at;
    if constexpr (W == 8)
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  }
}
// Bias, activation and gate of W adjacent features n .. (those below N).
template <bool GATED, int W>
__device__ __forceinline__ void bias_act_gate(const LinearParams& p, int n, float (&v)[W], const float (&u)[W]) {
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (n + i < p.N) v[i] += __ldg(p.bias + n + i);
  }
  activate(v, p.act);
  if constexpr (GATED) {
    if (p.bias_up) {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] *= n + i < p.N ? u[i] + __ldg(p.bias_up + n + i) : 0.f;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] *= u[i];
    }
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

// A block takes 8 features (the N of m16n8k16 steps) and up to 16 tokens (its
// M; TM of them); its 8 warps take the 64-column units of K in turn.  Lane
// (g, t) of a warp fetches 16 bytes of weight row g at columns 8t.. of each
// 32-column half unit: the order of columns within a sum is free, so those 8
// values serve as fragments of two k16 steps without a shuffle, and x is
// read the same way.  Weights go through a ring of kRowsDepth units of shared
// memory by cp.async, where each lane reads back what it copied itself: no
// barrier, no registers held by loads in flight, and about 190 KB on their
// way per SM (4 blocks of 48 KB).
constexpr int kRowsFeat = 8, kRowsTok = 16, kRowsWarps = 8, kRowsDepth = 6;
constexpr uint32_t kRowsUnit = 1024u;  // bytes of a warp's unit: 8 rows x 64 columns
constexpr uint32_t rows_smem(int na) { return (uint32_t)(kRowsWarps * kRowsDepth * na) * kRowsUnit; }

// 16 bytes of a row from column k; columns from K on read as zero and are
// never touched in memory.
__device__ __forceinline__ void row_copy16(uint32_t dst, const uint16_t* row, int k, int K, bool live) {
  const int left = live ? 2 * (K - k) : 0;
  const uint32_t n = left >= 16 ? 16u : left > 0 ? (uint32_t)left : 0u;
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(n ? row + k : row), "r"(n)
               : "memory");
}
__device__ __forceinline__ uint4 row_load16(const uint16_t* row, int k, int K, bool live) {
  if (!live || k >= K) return make_uint4(0u, 0u, 0u, 0u);
  if (k + 8 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
  uint32_t h[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (k + i < K) h[i >> 1] |= (uint32_t)__ldg(row + k + i) << (16 * (i & 1));
  return make_uint4(h[0], h[1], h[2], h[3]);
}

template <bool F16, bool GATED, int TM>
__global__ void __launch_bounds__(32 * kRowsWarps, 4) linear_rows_kernel(const LinearParams p) {
  constexpr int NA = GATED ? 2 : 1, NX = TM / 8;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ float red[kRowsWarps][NA][TM][kRowsFeat];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRowsFeat;
  const bool wl = n0 + g < p.N;
  const uint16_t* wr[NA];
  wr[0] = p.w + (size_t)(wl ? n0 + g : 0) * p.ldw;
  if constexpr (GATED) wr[1] = p.w_up + (size_t)(wl ? n0 + g : 0) * p.ldw_up;
  const uint32_t ring = smem_u32(smem_raw) + (uint32_t)(warp * kRowsDepth * NA) * kRowsUnit + 16u * (uint32_t)lane;
  const int units = (p.K + kKB - 1) / kKB, mine = (units - warp + kRowsWarps - 1) / kRowsWarps;
  auto fetch = [&](int i) {  // this warp's unit i, or an empty group behind the last
    if (i < mine) {
      const int k = kKB * (warp + kRowsWarps * i) + 8 * t;
      const uint32_t dst = ring + (uint32_t)(i % kRowsDepth * NA) * kRowsUnit;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        row_copy16(dst + (uint32_t)a * kRowsUnit, wr[a], k, p.K, wl);
        row_copy16(dst + (uint32_t)a * kRowsUnit + 512u, wr[a], k + 32, p.K, wl);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kRowsDepth - 1; ++i) fetch(i);

  bool xl[NX];
  const uint16_t* xr[NX];
#pragma unroll
  for (int j = 0; j < NX; ++j) {
    xl[j] = g + 8 * j < p.T;
    xr[j] = p.x + (size_t)(xl[j] ? g + 8 * j : 0) * p.ldx;
  }
  float acc[NA][4] = {};
#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    const int k = kKB * (warp + kRowsWarps * i) + 8 * t;
    uint4 xv[NX][2];
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      xv[j][0] = row_load16(xr[j], k, p.K, xl[j]);
      xv[j][1] = row_load16(xr[j], k + 32, p.K, xl[j]);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kRowsDepth - 2) : "memory");
    const uint32_t src = ring + (uint32_t)(i % kRowsDepth * NA) * kRowsUnit;
    uint4 wv[NA][2];
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(wv[a][h].x), "=r"(wv[a][h].y), "=r"(wv[a][h].z), "=r"(wv[a][h].w)
                     : "r"(src + (uint32_t)a * kRowsUnit + 512u * (uint32_t)h)
                     : "memory");
    fetch(i + kRowsDepth - 1);  // into the slot that the last turn read
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 lo = xv[0][h], hi = NX > 1 ? xv[NX - 1][h] : make_uint4(0u, 0u, 0u, 0u);
        mma16816<F16>(acc[a], lo.x, hi.x, lo.y, hi.y, wv[a][h].x, wv[a][h].y);
        mma16816<F16>(acc[a], lo.z, hi.z, lo.w, hi.w, wv[a][h].z, wv[a][h].w);
      }
  }
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int q = 0; q < 2 * NX; ++q) red[warp][a][g + 8 * (q >> 1)][2 * t + (q & 1)] = acc[a][q];
  __syncthreads();
  const int f = threadIdx.x % kRowsFeat, c = threadIdx.x / kRowsFeat;
  if (c < TM && c < p.T && n0 + f < p.N) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) s[a] += red[w][a][c][f];
    finish_one<F16>(p, c, n0 + f, s[0], s[1]);
  }
}

// ---- bounded waits ------------------------------------------------------------------

constexpr uint64_t kLinearTimeoutNs = 2000000000ull;  // 2 s per wait

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (bar_try(bar, parity)) return true;
    if ((it & 63u) == 0u && globaltimer_ns() - t0 > kLinearTimeoutNs) {
      atomicCAS(&g_linear_err, 0u, 1u);
      return false;
    }
  }
}
// Waits for phase `parity` of an mbarrier; false (and the error word set) on timeout.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
  return bar_try(bar, parity) || bar_wait_slow(bar, parity);
}
// After a wait has expired: time for copies and MMAs already issued to end
// before the block leaves its shared memory and TMEM.
__device__ __noinline__ void let_issued_work_end() {
  const uint64_t t0 = globaltimer_ns();
  for (int i = 0; i < 100000 && globaltimer_ns() - t0 < 5000000ull; ++i) __nanosleep(1000);
}
__device__ __forceinline__ void bar_init(uint32_t a, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(a), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t a, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(a), "r"(bytes) : "memory");
}
__device__ __forceinline__ void sts_f4(uint32_t a, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(a), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

// 8 floats from 16-byte chunks c, c + 1 of a swizzled 128-byte row.
__device__ __forceinline__ void read8(uint32_t row, uint32_t c, uint32_t x, float (&v)[8]) {
  const float4 a = lds_f4(row + ((c ^ x) << 4)), b = lds_f4(row + (((c + 1u) ^ x) << 4));
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

constexpr uint32_t kTile = 128u * 128u;  // bytes of a 128-row operand tile of one stage

// ---- some tokens: a cluster per 128 features, K split over its CTAs --------------------
// The weights are the A operand (128 features), NT tokens the B operand: with
// T < 128 no MMA row is wasted, and an output row of the accumulator is a
// feature, so a warp's loads and stores of out and residual are contiguous.
// Each CTA of the cluster takes a range of K; its accumulators go to its own
// shared memory as fp32, and after a cluster barrier each CTA sums its share
// of the outputs over the cluster in rank order and finishes them.  Nothing
// is exchanged through global memory, so no workspace, and calls on several
// streams share nothing.
constexpr int kSplitEpi = 8;                         // warps that read TMEM
constexpr int kSplitThreads = 32 * (kSplitEpi + 2);  // + a loading and an MMA warp
constexpr int kMaxSplit = 8;                         // CTAs of a cluster (the portable size)
constexpr uint32_t kSplitSmem = 220u * 1024u;

__host__ __device__ constexpr uint32_t split_stage(int nt, int na) { return na * kTile + (uint32_t)nt * 128u; }
__host__ __device__ constexpr int split_stages(int nt, int na) {
  return (int)(kSplitSmem / split_stage(nt, na)) < 12 ? (int)(kSplitSmem / split_stage(nt, na)) : 12;
}
__host__ __device__ constexpr uint32_t tmem_cols(int need) {
  return need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
}

template <bool F16, bool GATED, int NT>
__global__ void __launch_bounds__(kSplitThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_u,
                        const __grid_constant__ CUtensorMap map_x, const LinearParams p) {
  constexpr int NA = GATED ? 2 : 1;
  constexpr int ST = split_stages(NT, NA);
  constexpr uint32_t kStage = split_stage(NT, NA);
  static_assert((uint32_t)NA * NT * 512u <= ST * kStage, "the partial sums reuse the stages");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * ST + 1];
  __shared__ uint32_t tmem_slot;
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8u * ST, accfull = empty + 8u * ST;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc::cluster_rank(), S = gridDim.x;  // the cluster spans x
  const int n0 = blockIdx.y * 128, t0 = blockIdx.z * NT;
  const int KB = (p.K + kKB - 1) / kKB;
  const int kb0 = (int)((int64_t)KB * rank / S), kb1 = (int)((int64_t)KB * (rank + 1) / S);

  if (warp == kSplitEpi && lane == 0) {
    tc::prefetch_map(&map_w);
    tc::prefetch_map(&map_x);
  }
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) bar_init(full + 8u * s, 1), bar_init(empty + 8u * s, 1);
    bar_init(accfull, 1);
    mbar_fence_init();
  }
  if (warp == kSplitEpi + 1) {
    tc::tmem_alloc(smem_u32(&tmem_slot), tmem_cols(NA * NT));
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == kSplitEpi) {
    if (lane == 0) {
      bool ok = true;
#pragma unroll 1
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        const int i = kb - kb0, s = i % ST;
        if (i >= ST) ok = bar_wait(empty + 8u * s, (uint32_t)(i / ST - 1) & 1u);
        if (!ok) break;
        const uint32_t st = s0 + (uint32_t)s * kStage;
        bar_expect(full + 8u * s, kStage);
        tc::tma_2d(st, &map_w, kb * kKB, n0, full + 8u * s);
        if constexpr (GATED) tc::tma_2d(st + kTile, &map_u, kb * kKB, n0, full + 8u * s);
        tc::tma_2d(st + NA * kTile, &map_x, kb * kKB, t0, full + 8u * s);
      }
      if (!ok) let_issued_work_end();
    }
  } else if (warp == kSplitEpi + 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = tc::idesc_f16(128, NT, !F16);
      bool ok = true;
#pragma unroll 1
      for (int kb = kb0; kb < kb1 && ok; ++kb) {
        const int i = kb - kb0, s = i % ST;
        ok = bar_wait(full + 8u * s, (uint32_t)(i / ST) & 1u);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t st = s0 + (uint32_t)s * kStage;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t bd = tc::smem_desc_sw128(st + NA * kTile + 32u * k);
#pragma unroll
          for (int a = 0; a < NA; ++a)
            tc::mma_f16_ss(tmem + (uint32_t)(a * NT), tc::smem_desc_sw128(st + a * kTile + 32u * k), bd, idesc,
                           (i > 0 || k > 0) ? 1u : 0u);
        }
        tc::commit(empty + 8u * s);
      }
      if (ok)
        tc::commit(accfull);
      else
        let_issued_work_end();
    }
  } else {
    // partial sums: [matrix][token][feature] fp32 over the stages, which the
    // completed MMAs no longer read
    const bool ok = __all_sync(kAll, bar_wait(accfull, 0));
    tc::fence_after_sync();
    const int quarter = warp & 3, half = warp >> 2;  // TMEM lanes (features), half of the columns
    const uint32_t dst = s0 + 4u * (uint32_t)(32 * quarter + lane);
    if (ok) {
#pragma unroll 1
      for (int j = 16 * half; j < NA * NT; j += 32) {
        uint32_t v[16];
        tc::ld_32x32b_x16(tmem + ((uint32_t)(32 * quarter) << 16) + (uint32_t)j, v);
        tc::wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + 512u * (uint32_t)(j + q)), "r"(v[q]) : "memory");
      }
    }
    tc::fence_before_sync();
  }
  __syncwarp();
  tc::cluster_arrive();
  tc::cluster_wait();
  tc::fence_after_sync();
  if (warp == kSplitEpi + 1) tc::tmem_dealloc(tmem, tmem_cols(NA * NT));

  // this CTA's share of the outputs: items of 4 adjacent features of a token
  // (item j = floats 4j .. of [token][feature]), a few per turn so that their
  // loads overlap
  constexpr int kTurn = GATED ? 2 : 4;
  const int nt = min(NT, p.T - t0), items = nt * 32;
  const int i0 = (int)((int64_t)items * rank / S), i1 = (int)((int64_t)items * (rank + 1) / S);
#pragma unroll 1
  for (int i = i0 + tid; i < i1; i += kTurn * kSplitThreads) {
    float e[kTurn][4] = {}, v[kTurn][NA][4] = {};
#pragma unroll
    for (int m = 0; m < kTurn; ++m) {
      const int j = i + m * kSplitThreads, c = j >> 5, n = n0 + 4 * (j & 31);
      if (j < i1 && p.res && p.vec && n + 4 <= p.N) load_row<F16>(p, p.res, (size_t)(t0 + c) * p.ldr + n, e[m]);
    }
#pragma unroll
    for (int m = 0; m < kTurn; ++m) {
      const int j = i + m * kSplitThreads;
      if (j >= i1) continue;
      float4 q[NA][kMaxSplit];
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (uint32_t r = 0; r < kMaxSplit; ++r)
          if (r < S) q[a][r] = tc::ld_cluster_f4(tc::map_rank(s0 + 512u * (uint32_t)(a * NT) + 16u * (uint32_t)j, r));
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (uint32_t r = 0; r < kMaxSplit; ++r)
          if (r < S) {
            v[m][a][0] += q[a][r].x, v[m][a][1] += q[a][r].y;
            v[m][a][2] += q[a][r].z, v[m][a][3] += q[a][r].w;
          }
    }
#pragma unroll
    for (int m = 0; m < kTurn; ++m) {
      const int j = i + m * kSplitThreads, t = t0 + (j >> 5), n = n0 + 4 * (j & 31);
      if (j >= i1 || n >= p.N) continue;
      float(&y)[4] = v[m][0];
      if (p.vec && n + 4 <= p.N) {
        bias_act_gate<GATED>(p, n, y, v[m][NA - 1]);
        if (p.res) {
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] += e[m][k];
        }
        store_row<F16>(p, (size_t)t * p.ldo + n, y);
      } else {
        float(&u)[4] = v[m][NA - 1];
#pragma unroll 1
        for (int k = 0; k < 4 && n + k < p.N; ++k) {
          finish_one<F16>(p, t, n + k, y[0], u[0]);
          y[0] = y[1], y[1] = y[2], y[2] = y[3];
          if constexpr (GATED) u[0] = u[1], u[1] = u[2], u[2] = u[3];
        }
      }
    }
  }
  // no CTA leaves while another still reads its partial sums
  __syncwarp();
  tc::cluster_arrive();
  tc::cluster_wait();
}

// ---- many tokens: persistent pairs of CTAs ---------------------------------------------
// A pair owns a tile of 256 tokens x TN accumulator columns: each CTA loads
// its 128 tokens (A) and its half of the weight rows (B), the even CTA issues
// MMAs of M = 256 over both CTAs' operands, and each CTA's TMEM receives its
// tokens' rows.  With a gate, the even CTA's half are rows of w and the odd
// one's the same rows of w_up, so the first TN/2 columns are gates and the
// others their ups: one main loop for both forms.  Two accumulators
// alternate, so the epilogue of a tile runs under the next tile's MMAs.
constexpr int kPairEpi = 8;                            // epilogue warps
constexpr int kPairThreads = 32 * (kPairEpi + 2);      // + a loading and an MMA warp
constexpr uint32_t kPairStage0 = kPairEpi * 32u * 32u * 4u;  // fp32 staging: 32 x 32 per epilogue warp

template <int TN>
struct PairPlan {
  static constexpr uint32_t kBHalf = TN / 2 * 128u;
  static constexpr uint32_t kStage = kTile + kBHalf;
  static constexpr int kStages = TN == 256 ? 6 : 8;
  static constexpr uint32_t kSmem = kPairStage0 + kStages * kStage + 1024u;
};

template <int V>
struct Const {
  __device__ constexpr int operator()() const { return V; }
};

__device__ __forceinline__ void load_bias(const float* bias, int n, int N, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = n + i < N ? __ldg(bias + n + i) : 0.f;
}

// A lane's residual values of one epilogue step, as they lie in memory: 8
// adjacent features of PASS rows.  Only where whole rows move in 16 bytes
// (the other rows read their residual as they are written).
template <bool F16, int FC, int PASS>
struct Residual {
  uint4 raw[PASS][2];
  __device__ __forceinline__ void fetch(const LinearParams& p, int t, int step, int n, int n0) {
    if (!p.vec || n0 + FC > p.N) return;
#pragma unroll
    for (int q = 0; q < PASS; ++q) {
      if (t + q * step >= p.T) continue;
      const size_t at = (size_t)(t + q * step) * p.ldr + n;
      if (p.out_f32) {
        raw[q][0] = *reinterpret_cast<const uint4*>(static_cast<const float*>(p.res) + at);
        raw[q][1] = *reinterpret_cast<const uint4*>(static_cast<const float*>(p.res) + at + 4);
      } else {
        raw[q][0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.res) + at);
      }
    }
  }
  __device__ __forceinline__ void add(const LinearParams& p, int q, float (&v)[8]) const {
    const uint32_t w[8] = {raw[q][0].x, raw[q][0].y, raw[q][0].z, raw[q][0].w,
                           raw[q][1].x, raw[q][1].y, raw[q][1].z, raw[q][1].w};
    if (p.out_f32) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += __uint_as_float(w[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += from16<F16>((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
    }
  }
};

// Tile number -> (token tile, feature tile): columns of 8 token tiles, so that
// the tiles in flight share their operands in L2.
__device__ __forceinline__ void pair_tile(int tile, int MT, int FT, int& mt, int& ft) {
  constexpr int kGroup = 8;
  const int per = kGroup * FT, g = tile / per, in = tile - g * per;
  const int rows = min(kGroup, MT - g * kGroup);
  ft = in / rows;
  mt = g * kGroup + in - ft * rows;
}

template <bool F16, bool GATED, int TN>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_u,
                       const __grid_constant__ CUtensorMap map_x, const LinearParams p) {
  using P = PairPlan<TN>;
  constexpr int ST = P::kStages;
  constexpr int FN = GATED ? TN / 2 : TN;  // features per tile
  constexpr int FC = GATED ? 16 : 32;      // features of an epilogue step
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * ST + 4];
  __shared__ uint32_t tmem_slot;
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t op0 = s0 + kPairStage0;
  const uint32_t full = smem_u32(bars), empty = full + 8u * ST, accfull = empty + 8u * ST, accfree = accfull + 16u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = tc::cluster_rank();
  const int MT = (p.T + 255) / 256, FT = (p.N + FN - 1) / FN;
  const int ntiles = MT * FT, npairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int KB = (p.K + kKB - 1) / kKB;

  if (warp == kPairEpi && lane == 0) {
    tc::prefetch_map(&map_w);
    tc::prefetch_map(&map_x);
  }
  if (tid == 0) {
    for (int s = 0; s < ST; ++s) bar_init(full + 8u * s, 1), bar_init(empty + 8u * s, 1);
    for (int b = 0; b < 2; ++b) bar_init(accfull + 8u * b, 1), bar_init(accfree + 8u * b, 2 * kPairEpi);
    mbar_fence_init();
  }
  if (warp == kPairEpi + 1) {
    tc::tmem_alloc2(smem_u32(&tmem_slot), 2 * TN);
    tc::tmem_relinquish2();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_arrive();
  tc::cluster_wait();
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == kPairEpi) {
    if (lane == 0) {
      bool ok = true;
      uint32_t i = 0;
      const uint32_t full0 = tc::map_rank(full, 0);  // both CTAs' copies count on the even CTA's barriers
      const void* mb = GATED && rank ? &map_u : &map_w;
#pragma unroll 1
      for (int tile = pair; tile < ntiles && ok; tile += npairs) {
        int mt, ft;
        pair_tile(tile, MT, FT, mt, ft);
        const int y_a = mt * 256 + (int)rank * 128;
        const int y_b = ft * FN + (GATED ? 0 : (int)rank * (TN / 2));
#pragma unroll 1
        for (int kb = 0; kb < KB; ++kb, ++i) {
          const uint32_t s = i % ST;
          if (i >= ST) ok = bar_wait(empty + 8u * s, (i / ST - 1u) & 1u);
          if (!ok) break;
          const uint32_t st = op0 + s * P::kStage;
          if (rank == 0) bar_expect(full + 8u * s, 2 * P::kStage);
          tc::tma2_2d(st, &map_x, kb * kKB, y_a, full0 + 8u * s);
          tc::tma2_2d(st + kTile, mb, kb * kKB, y_b, full0 + 8u * s);
        }
      }
      // the last stages' arrivals from the even CTA, before this block may leave
      for (uint32_t j = i > ST ? i - ST : 0; j < i && ok; ++j) ok = bar_wait(empty + 8u * (j % ST), (j / ST) & 1u);
      if (!ok) let_issued_work_end();
    }
  } else if (warp == kPairEpi + 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = tc::idesc_f16(256, TN, !F16);
      bool ok = true;
      uint32_t i = 0, it = 0;
#pragma unroll 1
      for (int tile = pair; tile < ntiles && ok; tile += npairs, ++it) {
        const uint32_t b = it & 1u;
        if (it >= 2) ok = bar_wait(accfree + 8u * b, (it / 2 - 1u) & 1u);
        if (!ok) break;
        tc::fence_after_sync();
#pragma unroll 1
        for (int kb = 0; kb < KB; ++kb, ++i) {
          const uint32_t s = i % ST;
          ok = bar_wait(full + 8u * s, (i / ST) & 1u);
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t st = op0 + s * P::kStage;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma2_f16_ss(tmem + b * TN, tc::smem_desc_sw128(st + 32u * k), tc::smem_desc_sw128(st + kTile + 32u * k),
                            idesc, (kb > 0 || k > 0) ? 1u : 0u);
          tc::commit2(empty + 8u * s);
        }
        if (ok) tc::commit2(accfull + 8u * b);
      }
      if (!ok) let_issued_work_end();
    }
  } else {
    // Epilogue: warp w reads TMEM lanes 32 (w % 4) .. (its tokens) and half
    // w / 4 of the columns, 32 of them at a time (with a gate 16 and their 16
    // ups), in "lane = token" order, and passes the raw sums through a private
    // 32 x 32 fp32 square of shared memory (16-byte chunks XOR-swizzled by
    // token) into "lanes along features" order: a lane then holds 8 adjacent
    // features of a token, and residual and output move in whole sectors.
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t sq = s0 + (uint32_t)warp * 4096u;
    const uint32_t accfree0 = tc::map_rank(accfree, 0);
    constexpr int LR = FC / 8, RP = 32 / LR, PASS = LR;  // lanes of a row, rows of a pass, passes
    const int ch = lane % LR;
    Residual<F16, FC, PASS> res;
    uint32_t it = 0;
    bool ok = true;
#pragma unroll 1
    for (int tile = pair; tile < ntiles; tile += npairs, ++it) {
      int mt, ft;
      pair_tile(tile, MT, FT, mt, ft);
      const uint32_t b = it & 1u;
      const int tok0 = mt * 256 + (int)rank * 128 + 32 * quarter;
      // residual rows are fetched a step ahead, those of the first step while
      // the tile's MMAs still run
      if (p.res) res.fetch(p, tok0 + lane / LR, RP, ft * FN + half * (FN / 2) + 8 * ch, ft * FN + half * (FN / 2));
      ok = __all_sync(kAll, bar_wait(accfull + 8u * b, (it / 2) & 1u));
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t acc = tmem + b * TN + ((uint32_t)(32 * quarter) << 16);
#pragma unroll 1
      for (int c0 = half * (FN / 2); c0 < (half + 1) * (FN / 2); c0 += FC) {
        const int n0 = ft * FN + c0;
        const bool whole = p.vec && n0 + FC <= p.N;
        const int n = n0 + 8 * ch;
        float bg[8], bu[8];
        if (p.bias) load_bias(p.bias, n, p.N, bg);
        if (GATED && p.bias_up) load_bias(p.bias_up, n, p.N, bu);
        {
          uint32_t g[32];
          if constexpr (GATED) {
            uint32_t(&lo)[16] = *reinterpret_cast<uint32_t(*)[16]>(g);
            uint32_t(&hi)[16] = *reinterpret_cast<uint32_t(*)[16]>(g + 16);
            tc::ld_32x32b_x16(acc + (uint32_t)c0, lo);
            tc::ld_32x32b_x16(acc + (uint32_t)(TN / 2 + c0), hi);
          } else {
            tc::ld_32x32b_x32(acc + (uint32_t)c0, g);
          }
          tc::wait_ld();
          if (c0 + FC >= (half + 1) * (FN / 2)) {
            // the last read of this accumulator by this warp
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::arrive_cluster(accfree0 + 8u * b);
          }
          if (n0 >= p.N || tok0 >= p.T) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            sts_f4(sq + (uint32_t)lane * 128u + (((uint32_t)j ^ (lane & 7u)) << 4), __uint_as_float(g[4 * j]),
                   __uint_as_float(g[4 * j + 1]), __uint_as_float(g[4 * j + 2]), __uint_as_float(g[4 * j + 3]));
        }
        __syncwarp();
        // one switch per step: each activation has its own straight-line passes
        auto passes = [&](auto act) {
#pragma unroll
          for (int q = 0; q < PASS; ++q) {
            const int r = lane / LR + q * RP, t = tok0 + r;
            const uint32_t row = sq + (uint32_t)r * 128u, x = (uint32_t)(r & 7);
            float v[8];
            [[maybe_unused]] float u[8];
            read8(row, 2u * ch, x, v);
            if constexpr (GATED) read8(row, 2u * ch + 4u, x, u);
            if (p.bias) {
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] += bg[k];
            }
            activate(v, act());
            if constexpr (GATED) {
              if (p.bias_up) {
#pragma unroll
                for (int k = 0; k < 8; ++k) u[k] += bu[k];
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] *= u[k];
            }
            if (!whole) {
              sts_f4(row + (((2u * ch) ^ x) << 4), v[0], v[1], v[2], v[3]);
              sts_f4(row + (((2u * ch + 1u) ^ x) << 4), v[4], v[5], v[6], v[7]);
            } else if (t < p.T) {
              if (p.res) res.add(p, q, v);
              store_row<F16>(p, (size_t)t * p.ldo + n, v);
            }
          }
        };
        switch (p.act) {
          case MOE_ACT_SILU: passes(Const<MOE_ACT_SILU>()); break;
          case MOE_ACT_GELU: passes(Const<MOE_ACT_GELU>()); break;
          case MOE_ACT_GELU_TANH: passes(Const<MOE_ACT_GELU_TANH>()); break;
          case MOE_ACT_RELU: passes(Const<MOE_ACT_RELU>()); break;
          default: passes(Const<MOE_ACT_NONE>()); break;
        }
        if (p.res && c0 + FC < (half + 1) * (FN / 2)) res.fetch(p, tok0 + lane / LR, RP, n + FC, n0 + FC);
        __syncwarp();
        if (!whole) {
          // rows that start anywhere, or the last features: one element per lane
          const int k = lane % FC, nl = n0 + k;
#pragma unroll 4
          for (int r = lane / FC; r < 32; r += 32 / FC) {
            const int t = tok0 + r;
            if (t >= p.T || nl >= p.N) continue;
            float v;
            asm volatile("ld.shared.f32 %0, [%1];"
                         : "=f"(v)
                         : "r"(sq + (uint32_t)r * 128u + ((uint32_t)((k >> 2) ^ (r & 7)) << 4) + 4u * (uint32_t)(k & 3))
                         : "memory");
            const size_t o = (size_t)t * p.ldo + nl;
            if (p.out_f32) {
              if (p.res) v += static_cast<const float*>(p.res)[(size_t)t * p.ldr + nl];
              static_cast<float*>(p.out)[o] = v;
            } else {
              if (p.res) v += from16<F16>(static_cast<const uint16_t*>(p.res)[(size_t)t * p.ldr + nl]);
              static_cast<uint16_t*>(p.out)[o] = to16<F16>(v);
            }
          }
          __syncwarp();
        }
      }
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  tc::cluster_arrive();
  tc::cluster_wait();
  tc::fence_after_sync();
  if (warp == kPairEpi + 1) tc::tmem_dealloc2(tmem, 2 * TN);
}

// ---- host side --------------------------------------------------------------------------

using EncodeFn = decltype(&cuTensorMapEncodeTiled);

// The driver's tensor-map encoder, looked up once.
EncodeFn encoder() {
  static EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// rows x K elements of 16 bits, ld apart, read in boxes of box_rows x 64
// columns with the 128-byte swizzle; what lies outside reads as zero.
bool make_map(CUtensorMap* m, bool f16, const void* base, int K, int rows, int64_t ld, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
  // one row: any stride will do, and the caller's may be none
  const cuuint64_t strides[1] = {(cuuint64_t)(2 * ld)};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return encoder()(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                   const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Allows a kernel `smem` bytes of dynamic shared memory, once per device.
template <auto Kernel>
cudaError_t allow_smem(uint32_t smem) {
  static bool set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && set[dev])) return e;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) set[dev] = true;
  return e;
}

// A launch with clusters along x.
template <auto Kernel>
cudaError_t launch_cluster(dim3 grid, int threads, int cluster, uint32_t smem, const CUtensorMap& w,
                           const CUtensorMap& u, const CUtensorMap& x, const LinearParams& p, cudaStream_t st) {
  const cudaError_t e = allow_smem<Kernel>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute a[1];
  a[0].id = cudaLaunchAttributeClusterDimension;
  a[0].val.clusterDim.x = cluster;
  a[0].val.clusterDim.y = 1;
  a[0].val.clusterDim.z = 1;
  c.attrs = a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, Kernel, w, u, x, p);
}

template <bool F16, bool GATED, int NT>
cudaError_t launch_split_t(const LinearParams& p, int S, cudaStream_t st) {
  CUtensorMap w, u, x;
  if (!make_map(&w, F16, p.w, p.K, p.N, p.ldw, 128) || !make_map(&x, F16, p.x, p.K, p.T, p.ldx, NT)) return cudaErrorInvalidValue;
  u = w;
  if (GATED && !make_map(&u, F16, p.w_up, p.K, p.N, p.ldw_up, 128)) return cudaErrorInvalidValue;
  constexpr int NA = GATED ? 2 : 1;
  constexpr uint32_t smem = split_stages(NT, NA) * split_stage(NT, NA) + 1024u;
  const dim3 grid(S, (p.N + 127) / 128, (p.T + NT - 1) / NT);
  return launch_cluster<linear_split_kernel<F16, GATED, NT>>(grid, kSplitThreads, S, smem, w, u, x, p, st);
}

template <bool F16, bool GATED>
cudaError_t launch_split(const LinearParams& p, int S, cudaStream_t st) {
  if (p.T <= 16) return launch_split_t<F16, GATED, 16>(p, S, st);
  if (p.T <= 32) return launch_split_t<F16, GATED, 32>(p, S, st);
  if (p.T <= 64) return launch_split_t<F16, GATED, 64>(p, S, st);
  if (GATED || p.T <= 128) return launch_split_t<F16, GATED, 128>(p, S, st);
  if constexpr (!GATED) return launch_split_t<F16, GATED, 256>(p, S, st);
  return cudaErrorInvalidValue;
}

template <bool F16, bool GATED, int TN>
cudaError_t launch_pair_t(const LinearParams& p, int sms, cudaStream_t st) {
  CUtensorMap w, u, x;
  constexpr int FN = GATED ? TN / 2 : TN;
  if (!make_map(&w, F16, p.w, p.K, p.N, p.ldw, TN / 2) || !make_map(&x, F16, p.x, p.K, p.T, p.ldx, 128)) return cudaErrorInvalidValue;
  u = w;
  if (GATED && !make_map(&u, F16, p.w_up, p.K, p.N, p.ldw_up, TN / 2)) return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)((p.T + 255) / 256) * ((p.N + FN - 1) / FN);
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
  return launch_cluster<linear_pair_kernel<F16, GATED, TN>>(dim3(2 * pairs), kPairThreads, 2, PairPlan<TN>::kSmem, w, u,
                                                            x, p, st);
}

template <bool F16, bool GATED, int TM>
cudaError_t launch_rows(const LinearParams& p, cudaStream_t st) {
  constexpr uint32_t smem = rows_smem(GATED ? 2 : 1);
  const cudaError_t e = allow_smem<linear_rows_kernel<F16, GATED, TM>>(smem);
  if (e != cudaSuccess) return e;
  linear_rows_kernel<F16, GATED, TM><<<(p.N + kRowsFeat - 1) / kRowsFeat, 32 * kRowsWarps, smem, st>>>(p);
  return cudaGetLastError();
}

template <bool F16, bool GATED>
cudaError_t launch_any(const LinearParams& p, int sms, cudaStream_t st) {
  if (p.T <= 8) return launch_rows<F16, GATED, 8>(p, st);
  if (p.T <= kRowsTok) return launch_rows<F16, GATED, 16>(p, st);
  if (!encoder()) return cudaErrorNotSupported;
  if (p.T <= 256) {
    const int tiles = (p.N + 127) / 128 * (GATED && p.T > 128 ? 2 : 1), KB = (p.K + kKB - 1) / kKB;
    int S = 1;
    while (S < 8 && 2 * S * tiles <= sms && 2 * S <= KB) S *= 2;
    return launch_split<F16, GATED>(p, S, st);
  }
  return launch_pair_t<F16, GATED, 256>(p, sms, st);
}

}  // namespace

cudaError_t launch_linear(const LinearParams& p, bool f16, int sms, cudaStream_t st) {
  if (p.w_up) return f16 ? launch_any<true, true>(p, sms, st) : launch_any<false, true>(p, sms, st);
  return f16 ? launch_any<true, false>(p, sms, st) : launch_any<false, false>(p, sms, st);
}

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
