// moe_linear.cu -- dense product with its epilogue (moe_linear_forward):
//   y[t][n] = act(x[t] . w[n] + bias[n]) [* (x[t] . w_up[n] + bias_up[n])] [+ res[t][n]]
// fp32 accumulation and epilogue, one rounding to the output type.
//
// Three kernels, by how many tokens there are (linear_way):
//   rows   up to 16: the weights stream once through shared memory into
//          m16n8k16 steps (HBM bound);
//   tile   some hundreds: tiles of up to 128 tokens x 32 to 128 features,
//          TMA -> tcgen05, K split over a cluster whose CTAs join their sums
//          through distributed shared memory (HBM and L2 bound);
//   pair   more: persistent pairs of CTAs, 256 tokens x 128 or 256 columns,
//          tcgen05 on both CTAs' operands, each tile's epilogue under the next
//          one's MMAs (tensor bound).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_linear.h"
#include "moe_linear_way.h"
#include "moe_tc.cuh"

namespace moe {

// Error words of the calls on a device, one per stream (error_slot): the code
// of the first expired wait.
__device__ uint32_t g_linear_err[kLinearErrSlots];

namespace {

constexpr unsigned kAll = 0xffffffffu;
// ---- epilogue arithmetic ------------------------------------------------------------

// 1 / (1 + e^-z), as 2^-64 / (2^-64 + (g 2^-32)^2) with g = e^(-z/2): g stays in
// fp32's range down to z = -131, where the value is below it, and the divisor in
// that of the fast reciprocal (a division by more than 2^126 gives 0, which z
// from -88.7 on reaches where e^-z itself stands in the divisor).  With u =
// 2^-24 off by at most 11 u (g 2.9 u twice, the rest one step each) and 1.3 |z| u
// (z log2 e rounded), about what the rounding of z itself makes of it.  The
// accurate exponential, without the second term, is 8 instructions more, which
// short K shows (2048 x 256 x 4096 tanh-GELU in a run of others: 26 us, 20 so).
__device__ __forceinline__ float logistic(float z) {
  float g, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(g) : "f"(z * -0.72134752f));
  g *= 0x1p-32f;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(g, g, 0x1p-64f)));
  return r * 0x1p-64f;
}

// The activation in fp32, one switch for N values (a switch for each value
// fills the instruction cache once the loops around it are unrolled).
// tanh-GELU is v * logistic(z) with z = 2u, the same value without the
// cancellation of 1 + tanh(u) at negative u; GELU takes the normal CDF for the
// same reason.  SiLU is within 2^-20 (1 + |v| / 8) of the formula, GELU within
// 2^-20, tanh-GELU within 2^-20 (1 + |z| / 2), as z is off by up to 6 u of it (two
// constants, four steps).  NaN passes through all of them.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  switch (act) {
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= logistic(v[i]);
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= normcdff(v[i]);
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] *= logistic(1.5957691216057308f * fmaf(0.044715f * v[i] * v[i], v[i], v[i]));
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
  if (p.bias) g += p.bias[n];
  float a[1] = {g};
  activate(a, p.act);
  float y = a[0];
  if (p.w_up) y *= p.bias_up ? u + p.bias_up[n] : u;
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

// A block takes 8 features (the N of m16n8k16 steps) and up to 16 tokens (its
// M; TM of them); its W warps take the 64-column units of K in turn.  Lane
// (g, t) of a warp fetches 16 bytes of weight row g at columns 8t.. of each
// 32-column half unit: the order of columns within a sum is free, so those 8
// values serve as fragments of two k16 steps without a shuffle, and x is
// read the same way.  Weights go through a ring of units in shared memory by
// cp.async, where each lane reads back what it copied itself: no barrier, and
// no registers held by loads in flight.  32 warps an SM with 3 units each on
// their way (96 KB) suffice; deeper rings take the L1 cache from x (one token,
// 4096 x 4096: 8.3 us with 4 slots, 8.8 with 6, 8.9 with 3).  That is 4.0 TB/s of
// weights, each byte read once; the rest is the launch and the first loads' way.  With few blocks a
// block takes more warps, so that an SM has its 32 all the same (512 features:
// 3.5 us with 32, 4.4 with 8).
constexpr int kRowsFeat = 8;
constexpr uint32_t kRowsUnit = 1024u;  // bytes of a warp's unit: 8 rows x 64 columns
__host__ __device__ constexpr int rows_depth(int na) { return na == 1 ? 4 : 3; }
__host__ __device__ constexpr uint32_t rows_smem(int na, int warps) { return (uint32_t)(warps * rows_depth(na) * na) * kRowsUnit; }

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
  if (k + 8 <= K) return *reinterpret_cast<const uint4*>(row + k);
  uint32_t h[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (k + i < K) h[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
  return make_uint4(h[0], h[1], h[2], h[3]);
}

template <bool F16, bool GATED, int TM, int W>
__global__ void __launch_bounds__(32 * W, 32 / W) linear_rows_kernel(const LinearParams p) {
  constexpr int NA = GATED ? 2 : 1, NX = TM / 8, kDepth = rows_depth(NA);
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ float red[W][NA][TM][kRowsFeat];
  next_may_start();
  prior_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kRowsFeat;
  const bool wl = n0 + g < p.N;
  const uint16_t* wr[NA];
  wr[0] = p.w + (size_t)(wl ? n0 + g : 0) * p.ldw;
  if constexpr (GATED) wr[1] = p.w_up + (size_t)(wl ? n0 + g : 0) * p.ldw_up;
  const uint32_t ring = smem_u32(smem_raw) + (uint32_t)(warp * kDepth * NA) * kRowsUnit + 16u * (uint32_t)lane;
  const int units = (p.K + kKB - 1) / kKB, mine = (units - warp + W - 1) / W;
  auto fetch = [&](int i) {  // this warp's unit i, or an empty group behind the last
    if (i < mine) {
      const int k = kKB * (warp + W * i) + 8 * t;
      const uint32_t dst = ring + (uint32_t)(i % kDepth * NA) * kRowsUnit;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        row_copy16(dst + (uint32_t)a * kRowsUnit, wr[a], k, p.K, wl);
        row_copy16(dst + (uint32_t)a * kRowsUnit + 512u, wr[a], k + 32, p.K, wl);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch(i);

  bool xl[NX];
  const uint16_t* xr[NX];
#pragma unroll
  for (int j = 0; j < NX; ++j) {
    xl[j] = g + 8 * j < p.T;
    xr[j] = p.x + (size_t)(xl[j] ? g + 8 * j : 0) * p.ldx;
  }
  float acc[NA][4] = {};
  // x comes a unit ahead (its way from L2 takes as long as a turn) where the
  // registers for it leave room for 4 blocks per SM
  uint4 next[NX][2];
  auto load_x = [&](int i) {
    const int k = kKB * (warp + W * i) + 8 * t;
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      next[j][0] = row_load16(xr[j], k, p.K, xl[j] && i < mine);
      next[j][1] = row_load16(xr[j], k + 32, p.K, xl[j] && i < mine);
    }
  };
  if (TM == 8) load_x(0);
  // parts of kPart units, added up in red (one part up to 4096 columns and 8
  // warps: the loops are nested since a condition in the inner one costs 0.1
  // to 0.5 us a call)
#pragma unroll 1
  for (int i = 0;;) {
    const int i0 = i, i1 = min(mine, i + kPart);
#pragma unroll 1
    for (; i < i1; ++i) {
      if (TM != 8) load_x(i);
      uint4 xv[NX][2];
#pragma unroll
      for (int j = 0; j < NX; ++j) xv[j][0] = next[j][0], xv[j][1] = next[j][1];
      if (TM == 8) load_x(i + 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 2) : "memory");
      const uint32_t src = ring + (uint32_t)(i % kDepth * NA) * kRowsUnit;
      uint4 wv[NA][2];
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(wv[a][h].x), "=r"(wv[a][h].y), "=r"(wv[a][h].z), "=r"(wv[a][h].w)
                       : "r"(src + (uint32_t)a * kRowsUnit + 512u * (uint32_t)h)
                       : "memory");
      fetch(i + kDepth - 1);  // into the slot that the last turn read
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
    for (int a = 0; a < NA; ++a) {
#pragma unroll
      for (int q = 0; q < 2 * NX; ++q) {
        float& r = red[warp][a][g + 8 * (q >> 1)][2 * t + (q & 1)];
        if (i0)
          r += acc[a][q];
        else
          r = acc[a][q];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[a][q] = 0.f;
    }
    if (i >= mine) break;
  }
  __syncthreads();
  const int f = threadIdx.x % kRowsFeat, c = threadIdx.x / kRowsFeat;
  if (c < TM && c < p.T && n0 + f < p.N) {
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int w = 0; w < W; ++w) s[a] += red[w][a][c][f];
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
__device__ __forceinline__ bool bar_wait_until(uint32_t slot, uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (bar_try(bar, parity)) return true;
    if ((it & 63u) == 0u && globaltimer_ns() - t0 > limit_ns) {
      atomicCAS(&g_linear_err[slot], 0u, 1u);
      return false;
    }
  }
}
__device__ __noinline__ bool bar_wait_slow(uint32_t slot, uint32_t bar, uint32_t parity) {
  return bar_wait_until(slot, bar, parity, kLinearTimeoutNs);
}
// Waits for phase `parity` of an mbarrier; false (and the error word `slot` set) on timeout.
__device__ __forceinline__ bool bar_wait(uint32_t slot, uint32_t bar, uint32_t parity) {
  return bar_try(bar, parity) || bar_wait_slow(slot, bar, parity);
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
__device__ __forceinline__ void bar_arrive(uint32_t a) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(a) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t a, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(a), "r"(bytes) : "memory");
}
__device__ __forceinline__ void sts_v4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

constexpr uint32_t kTile = 128u * 128u;  // bytes of a 128-row operand tile of one stage

// ---- epilogue of the tcgen05 kernels -----------------------------------------------------
// Tokens are the rows of the accumulator (TMEM lanes) and features its
// columns; a warp reads units of 32 tokens x 32 features, a token per lane.
// Bias, activation, gate and residual happen in that order of values; the
// rounded rows go to a square of the warp's shared memory, 16-byte pieces
// XOR-ed by the row as the tensor map's swizzle has it, and leave by a TMA
// store, which also cuts off what lies behind T and N (4096 tokens x 256 ->
// 8192 features: 21 us, of which the bare writing takes 18; with rows written
// by the lanes from accumulator fragments 55).  It cuts off whole 16-byte pieces
// only, so a unit whose rows end inside one, and rows that do not start on
// 16-byte boundaries, are written by the lanes, from the square in row order.
constexpr uint32_t kSquare = 4096u;  // bytes per warp: 32 x 32 fp32, or two of 16 bits

// DIRECT: the lanes write their tokens' 64 bytes themselves, which takes more
// store instructions but no wait for the store to have read shared memory:
// for a block that ends with it.
template <bool F16, bool GATED, bool DIRECT>
struct Epilogue {
  const LinearParams& p;
  const CUtensorMap* map;  // of out, in boxes of 32 x 32
  const int lane;
  const uint32_t square;
  uint32_t turn = 0;
  uint4 raw[4];  // 16-bit residual of the next unit

  __device__ __forceinline__ Epilogue(const LinearParams& p_, const CUtensorMap* map_, int lane_, uint32_t square_)
      : p(p_), map(map_), lane(lane_), square(square_) {}

  // 16-bit residual of the unit at token t0, feature n0, ahead of its use
  __device__ __forceinline__ void fetch(int t0, int n0) {
    if (!p.res || p.out_f32 || !p.vec || n0 + 32 > p.N || t0 + lane >= p.T) return;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.res) + (size_t)(t0 + lane) * p.ldr + n0);
#pragma unroll
    for (int i = 0; i < 4; ++i) raw[i] = src[i];
  }
  // brings the unit's biases into the L1 cache
  __device__ __forceinline__ void touch_bias(int n0) const {
    if (p.bias && n0 + lane < p.N) {
      const float a = p.bias[n0 + lane], b = GATED && p.bias_up ? p.bias_up[n0 + lane] : 0.f;
      asm volatile("" ::"f"(a), "f"(b));
    }
  }
  __device__ __forceinline__ void add_bias(const float* bias, int n0, float (&v)[32]) const {
    if (p.bias_vec && n0 + 32 <= p.N) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 b = reinterpret_cast<const float4*>(bias + n0)[i];
        v[4 * i] += b.x, v[4 * i + 1] += b.y, v[4 * i + 2] += b.z, v[4 * i + 3] += b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (n0 + i < p.N) v[i] += bias[n0 + i];
    }
  }
  // Byte of 16-byte piece j of row r, rows of 64 or of 128 bytes.
  __device__ __forceinline__ static uint32_t piece64(int r, int j) { return (uint32_t)(64 * r + 16 * (j ^ (r >> 1 & 3))); }
  __device__ __forceinline__ static uint32_t piece128(int r, int j) { return (uint32_t)(128 * r + 16 * (j ^ (r & 7))); }

  // Finishes the unit at token t0, feature n0 from its sums (v, u: changed).
  __device__ __forceinline__ void unit(int t0, int n0, float (&v)[32], float (&u)[GATED ? 32 : 1]) {
    if (p.bias) add_bias(p.bias, n0, v);
    activate(v, p.act);
    if constexpr (GATED) {
      if (p.bias_up) add_bias(p.bias_up, n0, u);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] *= u[i];
    }
    // a piece of the residual behind N is not there to be read in 16 bytes
    const bool whole = n0 + 32 <= p.N, live = t0 + lane < p.T;
    if (p.vec == 2 || (p.vec && whole)) {
      if (!p.out_f32) {
        if (p.res) {
          if (whole) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
              for (int k = 0; k < 8; ++k) v[8 * i + k] += from16<F16>((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
            }
          } else if (live) {
            const uint16_t* src = static_cast<const uint16_t*>(p.res) + (size_t)(t0 + lane) * p.ldr + n0;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n0 + i < p.N) v[i] += from16<F16>(src[i]);
          }
        }
        if (DIRECT && whole) {
          if (!live) return;
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + (size_t)(t0 + lane) * p.ldo + n0);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            dst[j] = make_uint4(pack16<F16>(v[8 * j], v[8 * j + 1]), pack16<F16>(v[8 * j + 2], v[8 * j + 3]),
                                pack16<F16>(v[8 * j + 4], v[8 * j + 5]), pack16<F16>(v[8 * j + 6], v[8 * j + 7]));
          return;
        }
        // two squares of 2 KB in turn: the store before the last has been read out
        const uint32_t sq = square + (turn++ & 1u) * (kSquare / 2);
        if (lane == 0) tc::store_wait_read<1>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sts_v4(sq + piece64(lane, j), pack16<F16>(v[8 * j], v[8 * j + 1]), pack16<F16>(v[8 * j + 2], v[8 * j + 3]),
                 pack16<F16>(v[8 * j + 4], v[8 * j + 5]), pack16<F16>(v[8 * j + 6], v[8 * j + 7]));
        send(sq, t0, n0);
      } else {
        if (p.res && live) {
          const float* src = static_cast<const float*>(p.res) + (size_t)(t0 + lane) * p.ldr + n0;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 e = *reinterpret_cast<const float4*>(src + 4 * i);
              v[4 * i] += e.x, v[4 * i + 1] += e.y, v[4 * i + 2] += e.z, v[4 * i + 3] += e.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (n0 + i < p.N) v[i] += src[i];
          }
        }
        if (lane == 0) tc::store_wait_read<0>();
        __syncwarp();
        to_square(v);
        send(square, t0, n0);
      }
      return;
    }
    if (p.vec) {  // stores of units before this one may still read the square
      if (lane == 0) tc::store_wait_read<0>();
      __syncwarp();
    }
    if (p.out_f32) {
      __syncwarp();
      to_square(v);
      __syncwarp();
      if (n0 + lane < p.N) {
#pragma unroll 4
        for (int r = 0; r < 32; ++r) {
          if (t0 + r >= p.T) break;
          float y;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(y) : "r"(square + piece128(r, lane >> 2) + 4u * (lane & 3)) : "memory");
          if (p.res) y += static_cast<const float*>(p.res)[(size_t)(t0 + r) * p.ldr + n0 + lane];
          static_cast<float*>(p.out)[(size_t)(t0 + r) * p.ldo + n0 + lane] = y;
        }
      }
      __syncwarp();
      return;
    }
    // 16-bit rows that start anywhere: a token's values are paired as the
    // 4-byte words of its row in memory fall (from feature 0 or 1), and the
    // words are written two rows at a time; features left over at the ends
    // are written alone
    const uint16_t* res = static_cast<const uint16_t*>(p.res);
    uint16_t* out = static_cast<uint16_t*>(p.out);
    if (res) {
      __syncwarp();
#pragma unroll 1
      for (int r = 0; r < 32; r += 16) {
        uint16_t e[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          e[i] = n0 + lane < p.N && t0 + r + i < p.T ? res[(size_t)(t0 + r + i) * p.ldr + n0 + lane] : (uint16_t)0;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(square + piece64(r + i, lane >> 3) + 2u * (lane & 7)), "h"(e[i])
                       : "memory");
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 q = lds_f4(square + piece64(lane, j));
        const uint32_t w[4] = {__float_as_uint(q.x), __float_as_uint(q.y), __float_as_uint(q.z), __float_as_uint(q.w)};
#pragma unroll
        for (int k = 0; k < 8; ++k) v[8 * j + k] += from16<F16>((uint16_t)(w[k >> 1] >> (16 * (k & 1))));
      }
    }
    auto odd_row = [&](int t) { return (int)((reinterpret_cast<uintptr_t>(out + (size_t)t * p.ldo + n0) >> 1) & 1); };
    const int odd = odd_row(t0 + lane), left = min(32, p.N - n0);
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = pack16<F16>(odd ? v[2 * j + 1] : v[2 * j], odd ? v[j < 15 ? 2 * j + 2 : 31] : v[2 * j + 1]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; ++j) sts_v4(square + piece64(lane, j), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    __syncwarp();
    const int j = lane & 15;
#pragma unroll 4
    for (int r = lane >> 4; r < 32; r += 2) {
      const int o = odd_row(t0 + r);
      uint32_t x;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(square + piece64(r, j >> 2) + 4u * (j & 3)) : "memory");
      if (t0 + r < p.T && 2 * j + o + 1 < left)
        *reinterpret_cast<uint32_t*>(out + (size_t)(t0 + r) * p.ldo + n0 + 2 * j + o) = x;
    }
    if (t0 + lane < p.T) {
      uint16_t* row = out + (size_t)(t0 + lane) * p.ldo + n0;
      if (odd) row[0] = to16<F16>(v[0]);
      const int last = (left - odd) >> 1;  // a word with one feature, if any
      if ((left - odd) & 1) {
        uint16_t x;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(square + piece64(lane, last >> 2) + 4u * (last & 3)) : "memory");
        row[left - 1] = x;
      }
    }
    __syncwarp();
  }
  __device__ __forceinline__ void to_square(const float (&v)[32]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      sts_v4(square + piece128(lane, j), __float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
             __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3]));
  }
  __device__ __forceinline__ void send(uint32_t sq, int t0, int n0) const {
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tc::tma_store_2d(map, n0, t0, sq);
      tc::store_commit();
    }
  }
  // before the block leaves its shared memory
  __device__ __forceinline__ void drain() const {
    if (lane == 0) tc::store_wait_read<0>();
  }
};

// The sums of a unit.
__device__ __forceinline__ void load_unit(uint32_t taddr, float (&v)[32]) {
  tc::ld_32x32b_x32(taddr, reinterpret_cast<uint32_t(&)[32]>(v));
}

// ---- some tokens: a cluster per tile, K split over its CTAs ------------------------------
// Tiles of BT <= 128 tokens x FN features.  Each CTA of the cluster takes a
// range of K and accumulates it in its TMEM.  Then unit u of the tile belongs
// to CTA u % S: the others write their partial sums of it into that CTA's
// shared memory, and after one cluster barrier the owner adds them in rank
// order and finishes the unit.  Nothing is exchanged through global memory, so
// no workspace, and calls on several streams share nothing.
// With T < 128 only BT rows of x are loaded; the MMA reads whatever lies behind
// them as its other rows, whose results nobody reads.
// Bound by the way of a call through its phases (launch, first copies, the
// cluster's exchange, epilogue: 4 to 5 us) and the copies between them, not by
// bytes: 64 x 4096 x 4096 takes 9.8 us, reads 34.2 MB from HBM (weights and x
// once) and keeps the tensor cores busy 19 percent of it; 250 x 1024 x 4096
// takes 5.7 us, 64 x 4096 x 1024 gated 8.1.
//
// SUMS (K beyond longest_sum): the parts go to two
// accumulators in turn, and the epilogue warps add them up in registers while
// the MMAs go on (64 x 4096 x 4096: 11.5 us, 9.8 without).
constexpr int kTileEpi = 8;                         // warps that read TMEM
constexpr int kTileThreads = 32 * (kTileEpi + 2);   // + a loading and an MMA warp
constexpr int kTileStages = 12;                     // at most
constexpr uint32_t kMaxSmem = 227u * 1024u - 512u;  // dynamic shared memory next to the static

// Shared-memory plan of a tile: stages, their bytes, and the slots for other
// CTAs' partial sums behind them.
struct TilePlan {
  int BT, S, stages;
  uint32_t stage, slots, total;
};
__host__ __device__ inline TilePlan tile_plan(int BT, int rows, int na, int fn, int S) {
  TilePlan q;
  q.BT = BT, q.S = S;
  q.stage = (uint32_t)(BT + rows) * 128u;
  const int units = (BT + 31) / 32 * (fn / 32);
  const uint32_t exchange = (uint32_t)((units + S - 1) / S * (S - 1) * na) * kSquare;
  const uint32_t tail = kTile - (uint32_t)BT * 128u > exchange ? kTile - (uint32_t)BT * 128u : exchange;
  const int fit = (int)((kMaxSmem - 1024u - tail) / q.stage);
  q.stages = fit < kTileStages ? fit : kTileStages;
  q.slots = (uint32_t)q.stages * q.stage;
  q.total = 1024u + q.slots + tail;
  return q;
}

template <bool F16, bool GATED, int FN, bool SUMS>
__global__ void __launch_bounds__(kTileThreads, 1)
    linear_tile_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_u,
                       const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_out,
                       const LinearParams p, const TilePlan plan) {
  constexpr int NA = GATED ? 2 : 1, CN = NA * FN, G = FN / 32;
  static_assert(!SUMS || G <= 2, "a warp keeps the sums of one unit");
  constexpr uint32_t kCols = SUMS ? 2 * CN : CN;  // TMEM columns, a power of two from 32
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kTileStages + 4];
  __shared__ uint32_t tmem_slot;
  const uint32_t s0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8u * kTileStages, accfull = empty + 8u * kTileStages;
  const uint32_t accfree = accfull + 16u;  // (two of each; one accumulator: the first accfull alone)
  const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = tc::cluster_rank(), S = (uint32_t)plan.S;  // the cluster spans x
  const int n0 = blockIdx.y * FN, t0 = blockIdx.z * plan.BT;
  const int KB = (p.K + kKB - 1) / kKB;
  const int kb0 = (int)((int64_t)KB * rank / S), kb1 = (int)((int64_t)KB * (rank + 1) / S);

  next_may_start();
  // The loading and the MMA warp run their loops as whole warps, so that
  // addresses and descriptors stay in uniform registers, and one lane issues:
  // with the loops inside a one-lane branch a step took 350 ns whatever its size.
  const bool lead = tc::elect_one();
  auto copy = [&](int kb, uint32_t s) {  // by the loading warp's leader
    const uint32_t st = s0 + s * plan.stage, w = st + (uint32_t)plan.BT * 128u, bar = full + 8u * s;
    bar_expect(bar, plan.stage);
    tc::tma_2d(w, &map_w, kb * kKB, n0, bar);
    if constexpr (GATED) tc::tma_2d(w + FN * 128u, &map_u, kb * kKB, n0, bar);
    tc::tma_2d(st, &map_x, kb * kKB, t0, bar);
  };
  const int first = min(kb1 - kb0, plan.stages);
  if (warp == kTileEpi) {
    // the first copies are on their way before the block has met, and the
    // block does not wait for them to be issued (the copy engine takes in
    // about 50 bytes per clock)
    if (lead) {
      for (int s = 0; s < plan.stages; ++s) bar_init(full + 8u * s, 1), bar_init(empty + 8u * s, 1);
      for (int b = 0; b < 2; ++b) bar_init(accfull + 8u * b, 1), bar_init(accfree + 8u * b, kTileEpi);
      mbar_fence_init();
    }
    __syncwarp();
    asm volatile("bar.arrive 1, %0;" ::"n"(kTileThreads) : "memory");
    prior_wait();
#pragma unroll 1
    for (int i = 0; i < first; ++i) {
      if (lead) copy(kb0 + i, (uint32_t)i);
      __syncwarp();
    }
  }
  if (warp == kTileEpi + 1) {
    tc::tmem_alloc(smem_u32(&tmem_slot), kCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  if (warp != kTileEpi) {
    named_sync(1, kTileThreads);
    prior_wait();
  }
  tc::fence_after_sync();
  if (S > 1) tc::cluster_arrive_relaxed();  // (1) this CTA runs: its shared memory may be written
  const uint32_t tmem = tmem_slot;

  // units of this warp: the tokens of its TMEM quarter, every other group of features
  const int quarter = warp & 3, half = warp >> 2;
  const int tok0 = t0 + 32 * quarter;
  const bool busy = warp < kTileEpi && 32 * quarter < plan.BT && tok0 < p.T;
  const uint32_t acc = tmem + ((uint32_t)(32 * quarter) << 16);
  auto each_unit = [&](auto&& f) {
    if (!busy) return;
#pragma unroll 1
    for (int grp = half; grp < G; grp += 2)
      if (n0 + 32 * grp < p.N) f(grp, (uint32_t)(quarter * G + grp));
  };
  auto load = [&](int grp, float (&v)[32], float (&u)[GATED ? 32 : 1]) {
    load_unit(acc + (uint32_t)(32 * grp), v);
    if constexpr (GATED) load_unit(acc + (uint32_t)(FN + 32 * grp), u);
    tc::wait_ld();
  };
  // the sums of this CTA's range of K: of the warp's unit in registers, or in TMEM
  float sum[SUMS ? 32 : 1] = {}, sum_u[SUMS && GATED ? 32 : 1] = {};
  auto take = [&](int grp, float (&v)[32], float (&u)[GATED ? 32 : 1]) {
    if constexpr (SUMS) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        v[i] = sum[i];
        if constexpr (GATED) u[i] = sum_u[i];
      }
    } else {
      load(grp, v, u);
    }
  };

  Epilogue<F16, GATED, true> epi(p, &map_out, lane, s0 + (uint32_t)warp * kSquare);  // (in the stages, once they are done with)
  int mine = -1;
  if (warp == kTileEpi) {
    bool ok = true;
    uint32_t s = 0, phase = 0;
#pragma unroll 1
    for (int kb = kb0 + first; kb < kb1; ++kb) {
      ok = __all_sync(kAll, bar_wait(p.err_slot, empty + 8u * s, phase));
      if (!ok) break;
      if (lead) copy(kb, s);
      __syncwarp();
      if (++s == (uint32_t)plan.stages) s = 0, phase ^= 1u;
    }
    if (!ok) let_issued_work_end();
    __syncwarp();
    if (S > 1) tc::cluster_wait();  // (1)
  } else if (warp == kTileEpi + 1) {
    constexpr uint32_t idesc = tc::idesc_f16(128, CN, !F16);
    bool ok = true;
    uint32_t s = 0, phase = 0;
#pragma unroll 1
    for (int k0 = kb0, part = 0; k0 < kb1 && ok; ++part) {
      const uint32_t b = (uint32_t)part & 1u;
      if (SUMS && part >= 2) ok = __all_sync(kAll, bar_wait(p.err_slot, accfree + 8u * b, (uint32_t)(part / 2 - 1) & 1u));
      if (!ok) break;
      tc::fence_after_sync();
      const int k1 = SUMS ? min(kb1, k0 + kPart) : kb1;
      // (a commit at the part's end must not stand inside this loop: under a
      // condition there it cost 0.7 us of the 8 to 10 us of a call)
#pragma unroll 1
      for (int kb = k0; kb < k1; ++kb) {
        ok = __all_sync(kAll, bar_wait(p.err_slot, full + 8u * s, phase));
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t st = s0 + s * plan.stage;
        const uint32_t a = tc::desc_lo(st), w = tc::desc_lo(st + (uint32_t)plan.BT * 128u);
        if (lead) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc::mma_f16_lo(tmem + b * CN, a + 2u * k, w + 2u * k, idesc, (kb > k0 || k > 0) ? 1u : 0u);
          tc::commit(empty + 8u * s);
        }
        __syncwarp();
        if (++s == (uint32_t)plan.stages) s = 0, phase ^= 1u;
      }
      if (ok && lead) tc::commit(accfull + 8u * b);
      __syncwarp();
      k0 = k1;
    }
    if (!ok) let_issued_work_end();
    __syncwarp();
    if (S > 1) tc::cluster_wait();  // (1)
  } else {
    if (S > 1) tc::cluster_wait();  // (1)
    // this warp's first unit: its residual and biases come while the MMAs run
    each_unit([&](int grp, uint32_t unit) {
      if (mine >= 0 || unit % S != rank) return;
      mine = grp;
      epi.fetch(tok0, n0 + 32 * grp);
      epi.touch_bias(n0 + 32 * grp);
    });
    bool ok = true;
    if constexpr (SUMS) {
      const int parts = (kb1 - kb0 + kPart - 1) / kPart;
#pragma unroll 1
      for (int part = 0; part < parts && ok; ++part) {
        const uint32_t b = (uint32_t)part & 1u;
        ok = __all_sync(kAll, bar_wait(p.err_slot, accfull + 8u * b, (uint32_t)(part / 2) & 1u));
        if (!ok) break;
        tc::fence_after_sync();
        if (busy && half < G) {
          float v[32], u[GATED ? 32 : 1];
          load_unit(acc + b * CN + (uint32_t)(32 * half), v);
          if constexpr (GATED) load_unit(acc + b * CN + (uint32_t)(FN + 32 * half), u);
          tc::wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            sum[i] += v[i];
            if constexpr (GATED) sum_u[i] += u[i];
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) bar_arrive(accfree + 8u * b);
      }
    } else {
      ok = __all_sync(kAll, bar_wait(p.err_slot, accfull, 0));
      tc::fence_after_sync();
    }
    if (ok && S > 1)
      each_unit([&](int grp, uint32_t unit) {
        const uint32_t owner = unit % S;
        if (owner == rank) return;
        float v[32], u[GATED ? 32 : 1];
        take(grp, v, u);
        const uint32_t slot = unit / S * (S - 1) + (rank < owner ? rank : rank - 1);
        const uint32_t dst = tc::map_rank(s0 + plan.slots + slot * (NA * kSquare) + 16u * (uint32_t)lane, owner);
        auto push = [&](uint32_t at, const float* w) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            tc::st_cluster_v4(at + 512u * i, __float_as_uint(w[4 * i]), __float_as_uint(w[4 * i + 1]),
                              __float_as_uint(w[4 * i + 2]), __float_as_uint(w[4 * i + 3]));
        };
        push(dst, v);
        if constexpr (GATED) push(dst + kSquare, u);
      });
  }
  __syncwarp();
  if (S > 1) {
    tc::cluster_arrive();  // (2) partial sums are where they belong
    tc::cluster_wait();
  }
  if (warp < kTileEpi) {
    each_unit([&](int grp, uint32_t unit) {
      if (unit % S != rank) return;
      if (grp != mine) epi.fetch(tok0, n0 + 32 * grp);
      const uint32_t src = s0 + plan.slots + unit / S * (S - 1) * (NA * kSquare) + 16u * (uint32_t)lane;
      float v[32], u[GATED ? 32 : 1];
      take(grp, v, u);
      if (S > 1) {  // the sum over ranks in their order, whichever of them adds
        auto add = [&](uint32_t at, float* w) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 own = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            float4 sum = rank == 0 ? own : lds_f4(at + 512u * i);
#pragma unroll
            for (uint32_t r = 1; r < kMaxSplit; ++r) {
              if (r >= S) continue;
              const float4 q = r == rank ? own : lds_f4(at + 512u * i + (r < rank ? r : r - 1) * (NA * kSquare));
              sum.x += q.x, sum.y += q.y, sum.z += q.z, sum.w += q.w;
            }
            w[4 * i] = sum.x, w[4 * i + 1] = sum.y, w[4 * i + 2] = sum.z, w[4 * i + 3] = sum.w;
          }
        };
        add(src, v);
        if constexpr (GATED) add(src + kSquare, u);
      }
      epi.unit(tok0, n0 + 32 * grp, v, u);
    });
    epi.drain();
    __syncwarp();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kTileEpi + 1) tc::tmem_dealloc(tmem, kCols);
}

// ---- many tokens: persistent pairs of CTAs ---------------------------------------------
// A pair owns a tile of 256 tokens x TN accumulator columns: each CTA loads
// its 128 tokens (A) and its half of the weight rows (B), the even CTA issues
// MMAs of M = 256 over both CTAs' operands, and each CTA's TMEM receives its
// tokens' rows.  With a gate, the even CTA's half are rows of w and the odd
// one's the same rows of w_up, so the first TN/2 columns are gates and the
// others their ups: one main loop for both forms.  Two accumulators
// alternate, so the epilogue of a tile runs under the next tile's MMAs.
// Bound by the tensor cores: 8192 x 4096 x 8192 runs at 1.57 PFLOP/s (350 us) in
// short runs, at the power limit 1.38 (400 us); 2048 x 4096 x 4096 takes 49 us
// with the tensor pipe 83 percent active and 50 MB read from HBM, the same
// gated 93 us.
constexpr int kPairEpi = 8;                        // epilogue warps
constexpr int kPairThreads = 32 * (kPairEpi + 2);  // + a loading and an MMA warp

template <int TN>
struct PairPlan {
  static constexpr uint32_t kStage = kTile + TN / 2 * 128u;
  static constexpr uint32_t kSquares = kPairEpi * kSquare;
  static constexpr int kStages = (int)((kMaxSmem - 1024u - kSquares) / kStage);
  static constexpr uint32_t kSmem = kStages * kStage + kSquares + 1024u;
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

// (SUMS: as in linear_tile_kernel, the two accumulators alternating by parts of
// K; a warp keeps the sums of its units of the tile in registers, which is why
// TN is 128.  2048 x 4096 x 4096: 58 us, 49 without.)
template <bool F16, bool GATED, int TN, bool SUMS>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_u,
                       const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_out,
                       const LinearParams p) {
  using P = PairPlan<TN>;
  constexpr int ST = P::kStages;
  constexpr int FN = GATED ? TN / 2 : TN;  // features per tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * ST + 4];
  __shared__ uint32_t tmem_slot;
  const uint32_t op0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full = smem_u32(bars), empty = full + 8u * ST, accfull = empty + 8u * ST, accfree = accfull + 16u;
  const int tid = threadIdx.x, warp = __shfl_sync(kAll, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = tc::cluster_rank();
  const int MT = (p.T + 255) / 256, FT = (p.N + FN - 1) / FN;
  const int ntiles = MT * FT, npairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int KB = (p.K + kKB - 1) / kKB, part = SUMS ? kPart : KB;

  next_may_start();
  if (warp == kPairEpi && lane == 0) {
    tc::prefetch_map(GATED && rank ? &map_u : &map_w);
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
  prior_wait();

  // (whole warps run the loops, one lane issues, as in linear_tile_kernel)
  if (warp == kPairEpi) {
    const bool lead = tc::elect_one();
    bool ok = true;
    uint32_t s = 0, phase = 1, filled = 0;
    const uint32_t full0 = tc::map_rank(full, 0);  // both CTAs' copies count on the even CTA's barriers
    const void* mb = GATED && rank ? &map_u : &map_w;
#pragma unroll 1
    for (int tile = pair; tile < ntiles && ok; tile += npairs) {
      int mt, ft;
      pair_tile(tile, MT, FT, mt, ft);
      const int y_a = mt * 256 + (int)rank * 128;
      const int y_b = ft * FN + (GATED ? 0 : (int)rank * (TN / 2));
#pragma unroll 1
      for (int kb = 0; kb < KB; ++kb) {
        if (filled == ST)
          ok = __all_sync(kAll, bar_wait(p.err_slot, empty + 8u * s, phase));
        else
          ++filled;
        if (!ok) break;
        const uint32_t st = op0 + s * P::kStage;
        if (lead) {
          if (rank == 0) bar_expect(full + 8u * s, 2 * P::kStage);
          tc::tma2_2d(st, &map_x, kb * kKB, y_a, full0 + 8u * s);
          tc::tma2_2d(st + kTile, mb, kb * kKB, y_b, full0 + 8u * s);
        }
        __syncwarp();
        if (++s == ST) s = 0, phase ^= 1u;
      }
    }
    // the last stages' arrivals from the even CTA, before this block may leave
    if (filled < ST) s = 0, phase = 0;
    for (uint32_t j = 0; j < filled && ok; ++j) {
      ok = __all_sync(kAll, bar_wait(p.err_slot, empty + 8u * s, phase));
      if (++s == ST) s = 0, phase ^= 1u;
    }
    if (!ok) let_issued_work_end();
  } else if (warp == kPairEpi + 1) {
    if (rank == 0) {
      constexpr uint32_t idesc = tc::idesc_f16(256, TN, !F16);
      const bool lead = tc::elect_one();
      bool ok = true;
      uint32_t s = 0, phase = 0, it = 0;
#pragma unroll 1
      for (int tile = pair, k0 = 0; tile < ntiles && ok; ++it) {
        const uint32_t b = it & 1u;
        if (it >= 2) ok = __all_sync(kAll, bar_wait(p.err_slot, accfree + 8u * b, (it / 2 - 1u) & 1u));
        if (!ok) break;
        tc::fence_after_sync();
        const int k1 = min(KB, k0 + part);
#pragma unroll 1
        for (int kb = k0; kb < k1; ++kb) {
          ok = __all_sync(kAll, bar_wait(p.err_slot, full + 8u * s, phase));
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t st = op0 + s * P::kStage;
          const uint32_t a = tc::desc_lo(st), w = tc::desc_lo(st + kTile);
          if (lead) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc::mma2_f16_lo(tmem + b * TN, a + 2u * k, w + 2u * k, idesc, (kb > k0 || k > 0) ? 1u : 0u);
            tc::commit2(empty + 8u * s);
          }
          __syncwarp();
          if (++s == ST) s = 0, phase ^= 1u;
        }
        if (ok && lead) tc::commit2(accfull + 8u * b);
        __syncwarp();
        k0 = k1;
        if (k0 == KB) k0 = 0, tile += npairs;
      }
      if (!ok) let_issued_work_end();
    }
  } else {
    // Epilogue: warp w has TMEM quarter w % 4 (32 tokens) and half w / 4 of the
    // features, a unit at a time; a unit's residual is fetched one unit ahead,
    // the first one's while the tile's MMAs still run.
    constexpr int UN = FN / 64;  // units of a warp
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t accfree0 = tc::map_rank(accfree, 0);
    Epilogue<F16, GATED, false> epi(p, &map_out, lane, op0 + ST * P::kStage + (uint32_t)warp * kSquare);
    uint32_t it = 0;
#pragma unroll 1
    for (int tile = pair; tile < ntiles; tile += npairs) {
      int mt, ft;
      pair_tile(tile, MT, FT, mt, ft);
      const int tok = mt * 256 + (int)rank * 128 + 32 * quarter, c0 = half * (FN / 2), f0 = ft * FN + c0;
      epi.fetch(tok, f0);
      bool ok = true;
      if constexpr (SUMS) {
        float v[UN][32] = {}, u[GATED ? UN : 1][GATED ? 32 : 1] = {};
#pragma unroll 1
        for (int k0 = 0; k0 < KB; k0 += part, ++it) {
          const uint32_t b = it & 1u;
          ok = __all_sync(kAll, bar_wait(p.err_slot, accfull + 8u * b, (it / 2) & 1u));
          if (!ok) break;
          tc::fence_after_sync();
          const uint32_t acc = tmem + b * TN + ((uint32_t)(32 * quarter) << 16) + (uint32_t)c0;
#pragma unroll
          for (int j = 0; j < UN; ++j) {
            float q[32], z[GATED ? 32 : 1];
            load_unit(acc + 32u * (uint32_t)j, q);
            if constexpr (GATED) load_unit(acc + (uint32_t)(TN / 2 + 32 * j), z);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              v[j][i] += q[i];
              if constexpr (GATED) u[j][i] += z[i];
            }
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::arrive_cluster(accfree0 + 8u * b);
        }
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < UN; ++j) {
          const int n = f0 + 32 * j;
          if (n < p.N && tok < p.T) epi.unit(tok, n, v[j], u[GATED ? j : 0]);
          if (j + 1 < UN) epi.fetch(tok, n + 32);
        }
      } else {
        const uint32_t b = it & 1u;
        ok = __all_sync(kAll, bar_wait(p.err_slot, accfull + 8u * b, (it / 2) & 1u));
        if (!ok) break;
        ++it;
        tc::fence_after_sync();
        const uint32_t acc = tmem + b * TN + ((uint32_t)(32 * quarter) << 16) + (uint32_t)c0;
#pragma unroll 1
        for (int j = 0; j < UN; ++j) {
          const int n = f0 + 32 * j;
          float v[32], u[GATED ? 32 : 1];
          load_unit(acc + 32u * (uint32_t)j, v);
          if constexpr (GATED) load_unit(acc + (uint32_t)(TN / 2 + 32 * j), u);
          tc::wait_ld();
          if (j == UN - 1) {
            // the last read of this accumulator by this warp
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::arrive_cluster(accfree0 + 8u * b);
          }
          if (n < p.N && tok < p.T) epi.unit(tok, n, v, u);
          if (j + 1 < UN) epi.fetch(tok, n + 32);
        }
      }
    }
    epi.drain();
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

// Allows a kernel `smem` bytes of dynamic shared memory, once per device.  Host
// threads that meet here set the same value.
template <auto Kernel>
cudaError_t allow_smem(uint32_t smem) {
  static std::atomic<bool> set[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < 64 && set[dev].load(std::memory_order_acquire))) return e;
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) set[dev].store(true, std::memory_order_release);
  return e;
}

// out in boxes of 32 x 32 elements, swizzled by the box's row length.
bool make_out_map(CUtensorMap* m, bool f16, const LinearParams& p) {
  const cuuint64_t dims[2] = {(cuuint64_t)p.N, (cuuint64_t)p.T};
  const cuuint64_t strides[1] = {(cuuint64_t)((p.out_f32 ? 4 : 2) * p.ldo)};
  const cuuint32_t box[2] = {32, 32}, step[2] = {1, 1};
  return encoder()(m,
                   p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                   : f16     ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                             : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                   2, p.out, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   p.out_f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap w, u, x, out;
};
// Maps of a call: weights in boxes of `rows` rows, x in boxes of BT rows.
template <bool F16, bool GATED>
bool make_maps(const LinearParams& p, int rows, int BT, Maps* m) {
  if (!make_map(&m->w, F16, p.w, p.K, p.N, p.ldw, rows) || !make_map(&m->x, F16, p.x, p.K, p.T, p.ldx, BT)) return false;
  m->u = m->out = m->w;  // (unused ones are valid all the same)
  return (!GATED || make_map(&m->u, F16, p.w_up, p.K, p.N, p.ldw_up, rows)) &&
         (!p.vec || make_out_map(&m->out, F16, p));
}

template <auto Kernel, class... Args>
cudaError_t launch_cluster(dim3 grid, int threads, int cluster, uint32_t smem, cudaStream_t st, const Args&... args) {
  const cudaError_t e = allow_smem<Kernel>(kMaxSmem);
  return e != cudaSuccess ? e : launch_early(Kernel, grid, threads, smem, cluster, st, args...);
}

template <bool F16, bool GATED, int FN, bool SUMS>
cudaError_t launch_tile_t(const LinearParams& p, int BT, int S, cudaStream_t st) {
  Maps m;
  if (!make_maps<F16, GATED>(p, FN, BT, &m)) return cudaErrorInvalidValue;
  constexpr int NA = GATED ? 2 : 1;
  const TilePlan q = tile_plan(BT, NA * FN, NA, FN, S);
  const dim3 grid(S, (p.N + FN - 1) / FN, (p.T + BT - 1) / BT);
  return launch_cluster<linear_tile_kernel<F16, GATED, FN, SUMS>>(grid, kTileThreads, S, q.total, st, m.w, m.u, m.x, m.out,
                                                          p, q);
}

template <bool F16, bool GATED, int TN, bool SUMS>
cudaError_t launch_pair_t(const LinearParams& p, int sms, cudaStream_t st) {
  constexpr int FN = GATED ? TN / 2 : TN;
  Maps m;
  if (!make_maps<F16, GATED>(p, TN / 2, 128, &m)) return cudaErrorInvalidValue;
  const int64_t tiles = (int64_t)((p.T + 255) / 256) * ((p.N + FN - 1) / FN);
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  const int pairs = (int)(tiles < sms / 2 ? tiles : sms / 2);
  return launch_cluster<linear_pair_kernel<F16, GATED, TN, SUMS>>(dim3(2 * pairs), kPairThreads, 2, PairPlan<TN>::kSmem,
                                                                  st, m.w, m.u, m.x, m.out, p);
}

template <bool F16, bool GATED, int TM, int W>
cudaError_t launch_rows_w(const LinearParams& p, cudaStream_t st) {
  constexpr uint32_t smem = rows_smem(GATED ? 2 : 1, W);
  const cudaError_t e = allow_smem<linear_rows_kernel<F16, GATED, TM, W>>(smem);
  if (e != cudaSuccess) return e;
  return launch_early(linear_rows_kernel<F16, GATED, TM, W>, (p.N + kRowsFeat - 1) / kRowsFeat, 32 * W, smem, 1, st, p);
}

// Warps of a block: 32 an SM, as long as there are units of K for them.
template <bool F16, bool GATED, int TM>
cudaError_t launch_rows(const LinearParams& p, int sms, cudaStream_t st) {
  const int blocks = (p.N + kRowsFeat - 1) / kRowsFeat;
  if (blocks <= sms && p.K > 8 * kKB) return launch_rows_w<F16, GATED, TM, 32>(p, st);
  if (blocks <= 2 * sms && p.K > 8 * kKB) return launch_rows_w<F16, GATED, TM, 16>(p, st);
  return launch_rows_w<F16, GATED, TM, 8>(p, st);
}

template <bool F16, bool GATED>
cudaError_t launch_any(const LinearParams& p, int sms, cudaStream_t st) {
  LinearWay w = linear_way(p.T, p.K, p.N, GATED, F16, p.out_f32, sms);
  if (w.tokens > kRowsTok && !encoder()) {
    if (p.T > kRowsTok) return cudaErrorNotSupported;
    w.tokens = kRowsTok;
  }
  if (w.tokens == 8) return launch_rows<F16, GATED, 8>(p, sms, st);
  if (w.tokens == 16) return launch_rows<F16, GATED, 16>(p, sms, st);
  const bool pair = w.tokens == 256;
  if (w.sums) {
    if (pair) return launch_pair_t<F16, GATED, 128, true>(p, sms, st);
    return w.width == 32 ? launch_tile_t<F16, GATED, 32, true>(p, w.tokens, w.split, st)
                         : launch_tile_t<F16, GATED, 64, true>(p, w.tokens, w.split, st);
  }
  if (pair)
    return w.width == 256 ? launch_pair_t<F16, GATED, 256, false>(p, sms, st)
                          : launch_pair_t<F16, GATED, 128, false>(p, sms, st);
  if (w.width == 32) return launch_tile_t<F16, GATED, 32, false>(p, w.tokens, w.split, st);
  if (w.width == 64) return launch_tile_t<F16, GATED, 64, false>(p, w.tokens, w.split, st);
  if constexpr (!GATED) return launch_tile_t<F16, GATED, 128, false>(p, w.tokens, w.split, st);
  return cudaErrorInvalidValue;
}

// A wait on a barrier that nothing arrives at.
__global__ void linear_wait_probe_kernel(uint32_t slot, uint64_t limit_ns) {
  __shared__ __align__(8) uint64_t bar;
  if (threadIdx.x == 0) {
    bar_init(smem_u32(&bar), 1);
    mbar_fence_init();
    bar_wait_until(slot, smem_u32(&bar), 0, limit_ns);
  }
}

// The error word of a stream's calls.  Each stream handle that calls gets a word
// of its own, for good; the default stream, and streams beyond the last free
// word, have the first.
uint32_t error_slot(cudaStream_t st) {
  static std::atomic<uintptr_t> taken[kLinearErrSlots];
  const uintptr_t key = reinterpret_cast<uintptr_t>(st);
  if (st == nullptr || st == cudaStreamLegacy) return 0;
  uint32_t at = (uint32_t)((key >> 4) * 0x9e3779b97f4a7c15ull >> 32);
  for (int n = 0; n < kLinearErrSlots; ++n, ++at) {
    const uint32_t i = at % kLinearErrSlots;
    if (i == 0) continue;
    uintptr_t was = 0;
    if (taken[i].load() == key || taken[i].compare_exchange_strong(was, key) || was == key) return i;
  }
  return 0;
}

}  // namespace

cudaError_t launch_linear(LinearParams p, bool f16, int sms, cudaStream_t st) {
  p.err_slot = error_slot(st);
  if (p.w_up) return f16 ? launch_any<true, true>(p, sms, st) : launch_any<false, true>(p, sms, st);
  return f16 ? launch_any<true, false>(p, sms, st) : launch_any<false, false>(p, sms, st);
}

cudaError_t read_linear_error(uint32_t* code, cudaStream_t st) {
  uint32_t zero = 0;
  const size_t at = 4 * error_slot(st);
  cudaError_t e = cudaMemcpyFromSymbolAsync(code, g_linear_err, 4, at, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *code) {
    e = cudaMemcpyToSymbolAsync(g_linear_err, &zero, 4, at, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

cudaError_t launch_linear_wait_probe(uint64_t limit_ns, cudaStream_t st) {
  linear_wait_probe_kernel<<<1, 32, 0, st>>>(error_slot(st), limit_ns);
  return cudaGetLastError();
}

}  // namespace moe
