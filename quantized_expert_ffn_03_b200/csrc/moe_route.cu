// moe_route.cu -- expert choice from router logits (moe_route_from_logits):
//   s = softmax(l) or sigmoid(l), v = s + bias; the topk_groups groups of the
//   largest value (their largest v, or the sum of their two largest); the top_k
//   of v within them, ties to the lower index; w = scale * s [/ sum of s].
// One warp per token, the row in its registers: lane holds E / 32 values, and
// each choice is one integer maximum over the warp.  A row is read once (DRAM
// 16.8 MB for 16384 x 512 bf16, its size), so what bounds the kernel is the
// chain of a row's dependent steps, top_k rounds of choosing and, with groups,
// their ranking, which the 28 warps of an SM cover in part (0.56 to 0.7
// instructions issued per cycle and scheduler).  16384 tokens, 512 experts, top
// 10: 12.6 us; 4096 tokens, top 8 of 4 of 16 groups: 8.8 us; one token: 2.2 us,
// of which all but some hundred ns is the launch and the way of one load.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include "../../include/moe.h"
#include "moe_device.cuh"
#include "moe_linear.h"

namespace moe {

namespace {

constexpr int kRouteWarps = 4;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
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
__device__ __forceinline__ float logit_of(const T* row, int e) {
  const float l = load_logit(row + e);
  return l != l ? -INFINITY : fminf(l, FLT_MAX);
}

// The warp's largest value; NaN counts as none.
__device__ __forceinline__ float warp_maxf(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// ---- the choice in fp64, for what the fp32 values below leave open ------------------------
// Inlined and not unrolled: as functions of their own they cost every token
// (16384 tokens, 512 experts, top 10: 15.7 us against 12.0), by the registers
// that a call sets aside.

// A row's scores in fp64; top: its largest logit (0 for a row of -inf).
struct Scorer64 {
  bool sigmoid;
  double top, sum;
  __device__ __forceinline__ double operator()(float l) const {
    return sigmoid ? sigmoid64((double)l) : exp((double)l - top) / sum;
  }
};
template <typename T>
__device__ __forceinline__ Scorer64 scorer64(const RouteParams& p, const T* row, float top) {
  Scorer64 s = {p.sigmoid != 0, (double)top, 1.0};
  if (!p.sigmoid) {
    double sum = 0.0;
#pragma unroll 1
    for (int e = threadIdx.x & 31; e < p.E; e += 32) sum += exp((double)logit_of(row, e) - s.top);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if (sum > 0.0) s.sum = sum;
  }
  return s;
}
template <typename T>
__device__ __forceinline__ double value64(const RouteParams& p, const Scorer64& score, const T* row, int e) {
  return rank64(score(logit_of(row, e)) + (p.bias ? (double)p.bias[e] : 0.0));
}

// The rank of this lane's candidate, expert e (the first `count` lanes have one).
template <typename T>
__device__ __forceinline__ int rank_candidates64(const RouteParams& p, const T* row, float top, int e, int count) {
  const double d = value64(p, scorer64(p, row, top), row, e);
  int rank = 0;
  for (int j = 0; j < count; ++j) {
    const double o = __shfl_sync(kAll, d, j);
    const int oe = __shfl_sync(kAll, e, j);
    rank += o > d || (o == d && oe < e);
  }
  return rank;
}

// Whether this lane's group is kept, where the fp32 values leave it open: the
// group's value lies in [least, most], lo is the smallest `least` of the groups
// kept in fp32 and hi the largest `most` of those left out.  fp64 values for
// the groups that these bounds do not decide; first: the lane stands for its
// group.
template <typename T>
__device__ __forceinline__ bool keep_group64(const RouteParams& p, const T* row, float top, float least, float most,
                                             bool first, float lo, float hi) {
  const int lane = threadIdx.x & 31, grp = lane >> p.lane_shift;
  const Scorer64 score = scorer64(p, row, top);
  const bool sure = first && least > hi, near = first && !sure && !(most < lo);
  const int left = p.topk_groups - __popc(__ballot_sync(kAll, sure));
  const uint32_t nears = __ballot_sync(kAll, near);
  double mine = 0.0;
  for (uint32_t m = nears; m; m &= m - 1) {
    const int at = __ffs(m) - 1, g = at >> p.lane_shift;
    double a = -INFINITY, b = -INFINITY;
    for (int j = lane; j < p.per; j += 32) {
      const double v = value64(p, score, row, g * p.per + j);
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) {
      const double a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
      b = fmax(fmax(b, b2), fmin(a, a2));
      a = fmax(a, a2);
    }
    if (lane == at) mine = p.top2 && p.per > 1 ? rank64(a + b) : a;
  }
  int rank = 0;
  for (uint32_t m = nears; m; m &= m - 1) {
    const int at = __ffs(m) - 1;
    const double o = __shfl_sync(kAll, mine, at);
    rank += o > mine || (o == mine && (at >> p.lane_shift) < grp);
  }
  return sure || (near && rank < left);
}

// A whole token.  key: E words of shared memory of this warp; cand: 32 more.
template <typename T>
__device__ __forceinline__ void route_exact(const RouteParams& p, int64_t t, uint64_t* key, int* cand) {
  const int lane = threadIdx.x & 31;
  const T* row = static_cast<const T*>(p.logits) + (size_t)t * p.ldl;
  const bool by_value = p.bias != nullptr;
  float top = 0.f;
  if (!p.sigmoid) {
    top = -INFINITY;
    for (int e = lane; e < p.E; e += 32) top = fmaxf(top, logit_of(row, e));
    top = warp_maxf(top);
    if (top == -INFINITY) top = 0.f;  // a row of -inf: every score is 0
  }
  const Scorer64 score = scorer64(p, row, top);
  __syncwarp();

  // kept groups, a bit each: by their values, or without a bias by their largest logit
  uint32_t kept = kAll;
  if (p.n_groups > 1) {
    double* dv = reinterpret_cast<double*>(key);
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32)
      dv[e] = by_value || p.top2 ? value64(p, score, row, e) : (double)logit_of(row, e);
    __syncwarp();
    const int lanes = 1 << p.lane_shift, grp = lane >> p.lane_shift, sub = lane & (lanes - 1);
    double a = -INFINITY, b = -INFINITY;
    if (grp < p.n_groups)
      for (int j = sub; j < p.per; j += lanes) {
        const double x = dv[grp * p.per + j];
        b = fmax(b, fmin(a, x));
        a = fmax(a, x);
      }
    for (int o = 1; o < lanes; o <<= 1) {
      const double a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
      b = fmax(fmax(b, b2), fmin(a, a2));
      a = fmax(a, a2);
    }
    const double x = p.top2 && p.per > 1 ? rank64(a + b) : a;
    int rank = 0;
    for (int g = 0; g < p.n_groups; ++g) {
      const double o = __shfl_sync(kAll, x, g << p.lane_shift);
      rank += o > x || (o == x && g < grp);
    }
    kept = __reduce_or_sync(kAll, sub == 0 && grp < p.n_groups && rank < p.topk_groups ? 1u << grp : 0u);
    __syncwarp();
  }

  // experts by value, or by logit where the score alone decides; 0: left out
  uint64_t best = 0;
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) {
    const bool in = p.n_groups == 1 || (kept >> (e / p.per) & 1u);
    const uint64_t k = in ? order64(by_value ? value64(p, score, row, e) : (double)logit_of(row, e)) : 0ull;
    key[e] = k;
    best = k > best ? k : best;
  }
  // candidates: those that reach the K-th of the lanes' largest, if they are
  // few enough; all of them count where fewer than K lanes have any
#pragma unroll 1
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll 1
    for (int o = size >> 1; o; o >>= 1) {
      const uint64_t other = __shfl_xor_sync(kAll, best, o);
      const bool keep_max = ((lane & o) == 0) == ((lane & size) == 0);
      best = (other > best) == keep_max ? other : best;
    }
  const uint64_t kth = __shfl_sync(kAll, best, p.K - 1), bound = kth ? kth : 1ull;
  int count = 0;
  for (int e0 = 0; e0 < p.E; e0 += 32) {
    const int e = e0 + lane;
    const bool in = e < p.E && key[e] >= bound;
    const uint32_t m = __ballot_sync(kAll, in);
    const int at = count + __popc(m & ((1u << lane) - 1u));
    if (in && at < 32) cand[at] = e;
    count += __popc(m);
  }
  __syncwarp();
  int chosen = 0, rank = 32;
  if (count <= 32) {
    chosen = lane < count ? cand[lane] : 0;
    const uint64_t mine = lane < count ? key[chosen] : 0ull;
    if (lane < count) {
      rank = 0;
      for (int j = 0; j < count; ++j) {
        const int e = cand[j];
        const uint64_t k = key[e];
        rank += k > mine || (k == mine && e < chosen);
      }
    }
  } else {
    // many equal values: K rounds, lane k keeps the choice of round k
    for (int k = 0; k < p.K; ++k) {
      uint64_t most = 0;
      int at = p.E;
      for (int e = lane; e < p.E; e += 32)
        if (key[e] > most) most = key[e], at = e;
      warp_best(most, at);
      if (lane == (at & 31)) key[at] = 0;
      if (lane == k) chosen = at, rank = k;
      __syncwarp();
    }
  }
  double w = rank < p.K ? score(logit_of(row, chosen)) : 0.0;
  if (p.renorm) {
    double total = w;
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    w = total > 0.0 ? w / total : 0.0;
  }
  if (rank < p.K) {
    p.idx[(size_t)t * p.K + rank] = chosen;
    p.w[(size_t)t * p.K + rank] = (float)(w * (double)p.scale);
  }
}

// ---- one warp per token ------------------------------------------------------------------
// Values are fp32 here.  With s' the fp32 score of s (fast_exp is off by at most
// 2 + 1.16 |x| ulp, a fast division by 2) and u = 2^-24:
//   sigmoid   |s' - s| <= 2^-23 ((1 - s) (2 + 1.16 |l|) s + 1/2 + 2 s) < 2^-21
//   softmax   with x = l - max rounded (u |x|), e^x is off by at most 4 u; the
//             terms of the row's sum together by (4 + 3.3 * 4.9) u of it (4.9:
//             the largest mean |x| that 2048 terms can have, weighted by
//             themselves), its additions by 15 u, the reciprocal and the
//             product by 3 u: 44 u in all, so |s' - s| <= 2^-18 / sum (no score
//             is larger than 1 / sum)
// and v' = s' + bias adds 2^-24 |v'|.  A choice that holds by more than these
// bounds is the fp64 choice; where candidates or groups are closer (a token in
// some hundreds), theirs alone are computed in fp64.  A row with more candidates
// than lanes goes to route_exact.  Without a bias experts are ordered by their
// logits, which needs no bound.
// Weights come from the accurate exponential (2 ulp: 4 u), l - max with its
// rounding made good and divisions to the nearest: under 23 u of the formula.
// Softmax weights that are not renormalised take the sum above, 42 u in all
// (accurate exponentials there would make it 31 and cost 16384 tokens 13.8 us
// instead of 12.6); renormalised ones do not see it, a constant factor.
// Measured in the 2-norm: 6 10^-8 for both.  A chosen score below 2^-100 is no
// longer sure to keep its bits through this, and its row goes to fp64.
//
// Top-K without K rounds over E: each lane's largest value; the K-th largest
// of those 32 is a bound that at least K values reach; the values
// that reach it (a few more than K of E) are gathered one per lane, and each
// lane counts how many beat its own.
__device__ __forceinline__ uint32_t order32(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_order32(uint32_t k) {
  return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ float rank32(float v) { return fmaxf(v, -INFINITY); }  // NaN ranks as -inf
// e^x to within 2 + 1.16 |x| ulp; 0 below fp32's normal range.
__device__ __forceinline__ float fast_exp(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}

// A bound that at least K lanes reach: the K-th largest of the lanes' values, or
// less where some are equal (equal ones leave together).
__device__ __forceinline__ float warp_kth(float v, int K) {
  float m = v;
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    m = warp_maxf(v);
    if (v >= m) v = -INFINITY;
  }
  return m;
}

template <bool LONG>
struct MaskOf {
  using type = uint32_t;
};
template <>
struct MaskOf<true> {
  using type = uint64_t;
};
__device__ __forceinline__ int lowest_bit(uint32_t m) { return __ffs(m) - 1; }
__device__ __forceinline__ int lowest_bit(uint64_t m) { return __ffsll(m) - 1; }

// 16 bytes of logits: W of them.
template <typename T>
struct Wide {
  static constexpr int W = 16 / sizeof(T);
  static __device__ __forceinline__ void load(const T* p, float (&v)[W]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const T* h = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = to_float(h[i]);
  }
  static __device__ __forceinline__ float to_float(float x) { return x; }
  static __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
};

// NV: values per lane, a multiple of Wide<T>::W with 32 NV >= E.
template <typename T, int NV, bool BIAS>
__global__ void __launch_bounds__(32 * kRouteWarps, NV <= 16 ? 7 : NV == 32 ? 5 : 3) route_kernel(const RouteParams p) {
  constexpr int W = Wide<T>::W;
  extern __shared__ uint64_t keys_all[];
  __shared__ int cand_all[kRouteWarps][32];
  __shared__ uint64_t ckey_all[kRouteWarps][32];
  __shared__ float cval_all[kRouteWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  next_may_start();
  prior_wait();
  if (t >= p.T) return;
  uint64_t* key = keys_all + (size_t)warp * p.E;
  float* val = reinterpret_cast<float*>(key);  // groups: the values by expert
  int* cand = cand_all[warp];
  uint64_t* ckey = ckey_all[warp];
  float* cval = cval_all[warp];
  const T* row = static_cast<const T*>(p.logits) + (size_t)t * p.ldl;
  constexpr bool by_value = BIAS;
  // value i of this lane is expert place(i): W adjacent ones per 16-byte load
  auto place = [&](int i) { return W * (lane + 32 * (i / W)) + i % W; };

  // the biases are asked for before the logits are waited for
  float b[BIAS ? NV : 1];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      if (p.vec && p.bias_vec) {
        const float4 q = place(i) < p.E ? *reinterpret_cast<const float4*>(p.bias + place(i)) : make_float4(0.f, 0.f, 0.f, 0.f);
        b[i] = q.x, b[i + 1] = q.y, b[i + 2] = q.z, b[i + 3] = q.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) b[i + j] = place(i + j) < p.E ? p.bias[place(i + j)] : 0.f;
      }
    }
  }

  // ---- logits -> v: what experts are ordered by (values, or logits without a bias) ----
  float v[NV];
  float top = -INFINITY, inv = 1.f;
#pragma unroll
  for (int i = 0; i < NV; i += W) {
    float l[W];
    if (p.vec) {
      if (place(i) < p.E)
        Wide<T>::load(row + place(i), l);
      else
#pragma unroll
        for (int j = 0; j < W; ++j) l[j] = -INFINITY;
    } else {
#pragma unroll
      for (int j = 0; j < W; ++j) l[j] = place(i + j) < p.E ? load_logit(row + place(i + j)) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) v[i + j] = fminf(rank32(l[j]), FLT_MAX);  // (-inf behind the last expert)
  }
  if (!p.sigmoid) {
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, v[i]);
    top = warp_maxf(top);
    if (top == -INFINITY) top = 0.f;  // a row of -inf: every score is 0
    if (by_value || !p.renorm) {
      // (partial sums: at most 10 additions of a lane stand behind each other)
      constexpr int PS = NV <= 16 ? 4 : 8;
      float part[PS] = {};
#pragma unroll
      for (int i = 0; i < NV; ++i) part[i % PS] += fast_exp(v[i] - top);
#pragma unroll
      for (int o = PS / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) part[i] += part[i + o];
      const float sum = warp_sum(part[0]);
      inv = sum > 0.f ? __fdiv_rn(1.f, sum) : 1.f;
    }
  }
  const float eps = p.sigmoid || !by_value ? 0x1p-21f : 0x1p-18f * inv;  // bound of a score's error
  auto score = [&](float l) { return p.sigmoid ? __fdividef(1.f, 1.f + fast_exp(-l)) : fast_exp(l - top) * inv; };
  if (by_value) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      v[i] = place(i) < p.E ? rank32(score(v[i]) + b[BIAS ? i : 0]) : -INFINITY;
  }

  // ---- groups: v becomes the values of the kept groups' experts, entry q of
  // them (value i of a lane: q = lane + 32 i) being expert `expert(q)` ----
  int entries = p.E;
  bool open = false;  // not to be decided here
  int my_group = 0;
  const bool grouped = p.n_groups > 1;
  if (grouped) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (place(i) < p.E) val[place(i)] = v[i];
    __syncwarp();
    // `lanes` lanes per group, each the two largest values of its share, walked
    // from a place of the group's own so that lanes meet different banks
    const int lanes = 1 << p.lane_shift, grp = lane >> p.lane_shift, sub = lane & (lanes - 1);
    float a = -INFINITY, b = -INFINITY;
    const bool plain = by_value || !p.top2;  // no score needed: values, or logits by their largest
    if (grp < p.n_groups) {
      int q = sub + grp * lanes;  // (i + grp * lanes) modulo per
      while (q >= p.per) q -= p.per;
      const float* mine = val + grp * p.per;
#pragma unroll 4
      for (int i = sub; i < p.per; i += lanes) {
        float x = mine[q];
        if (!plain) x = score(x);
        b = fmaxf(b, fminf(a, x));
        a = fmaxf(a, x);
        q += lanes;
        if (q >= p.per) q -= p.per;
      }
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
      b = fmaxf(fmaxf(b, b2), fminf(a, a2));
      a = fmaxf(a, a2);
    }
    // (half the sum, which does not overflow; +inf and -inf together rank as -inf)
    const bool two = p.top2 && p.per > 1;
    const float x = two ? rank32(0.5f * a + 0.5f * b) : a;
    int rank = 0;  // of this lane's group among all
    for (int g = 0; g < p.n_groups; ++g) {
      const float o = __shfl_sync(kAll, x, g << p.lane_shift);
      rank += o > x || (o == x && g < grp);
    }
    const bool first = sub == 0 && grp < p.n_groups;
    bool in = first && rank < p.topk_groups;
    if (by_value || p.top2) {
      // A group's value in fp64 is within `err` of x: a and b are each off by
      // eps and by the rounding of s + bias, 2^-24 |a| and 2^-24 |b|, which do
      // not shrink where a and b cancel, and so the rounding of their sum (the
      // factor of two left over takes in that of the bounds themselves).  An
      // infinite value is exact.  The kept groups have to lead those left out
      // by more than these errors; equal infinities are in their order already.
      float err = eps + 0x1p-22f * fabsf(a);
      if (two) err += 0x1p-22f * fabsf(b);
      if (fabsf(x) == INFINITY) err = 0.f;
      const float least = x - err, most = x + err;
      const float lo = from_order32(__reduce_min_sync(kAll, in ? order32(least) : ~0u));
      const float hi = from_order32(__reduce_max_sync(kAll, first && !in ? order32(most) : 0u));
      if (!(lo > hi || (lo == hi && fabsf(lo) == INFINITY))) in = keep_group64(p, row, top, least, most, first, lo, hi);
    }
    const uint32_t kept = __ballot_sync(kAll, in);
    if (in) cand[__popc(kept & ((1u << lane) - 1u))] = grp;
    entries = p.topk_groups * p.per;
    __syncwarp();
    my_group = lane < p.topk_groups ? cand[lane] : 0;
    __syncwarp();
  }
  auto expert = [&](int q) {  // by the whole warp
    const int g = p.per == 1 ? q : (int)__umulhi((uint32_t)q, p.per_inv);  // q / per
    return __shfl_sync(kAll, my_group, g & 31) * p.per + q - g * p.per;
  };
  if (grouped) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (32 * i >= entries) {
        v[i] = -INFINITY;
      } else {
        const int q = lane + 32 * i, e = expert(q);
        v[i] = q < entries ? val[e] : -INFINITY;
      }
    }
  }

  // ---- candidates ----
  float best = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) best = fmaxf(best, v[i]);
  float bound = warp_kth(best, p.K);
  if (by_value && fabsf(bound) != INFINITY) bound -= 2.f * eps + 0x1p-22f * fabsf(bound);
  using Mask = typename MaskOf<(NV > 32)>::type;
  Mask mask = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (v[i] >= bound) mask |= (Mask)1 << i;
  if (bound == -INFINITY) {  // the places behind the last expert hold -inf too
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((grouped ? lane + 32 * i : place(i)) >= entries) mask &= ~((Mask)1 << i);
  }
  int count = 0;
  for (uint32_t with; (with = __ballot_sync(kAll, mask != 0)) != 0 && count <= 32; mask &= mask - 1) {
    const int at = count + __popc(with & ((1u << lane) - 1u)), i = lowest_bit(mask);
    if (mask && at < 32) cand[at] = grouped ? lane + 32 * i : place(i);
    count += __popc(with);
  }
  if (count > 32) open = true;
  __syncwarp();

  // ---- one candidate per lane: its rank, whether the order is certain ----
  if (!open) {
    const bool live = lane < count;
    int e = live ? cand[lane] : 0;
    if (grouped) e = expert(e);
    // its value again, by the same operations
    const float l = fminf(rank32(load_logit(row + e)), FLT_MAX);
    const float x = by_value ? rank32(score(l) + p.bias[e]) : l;
    const uint64_t mine64 = live ? (uint64_t)order32(x) << 32 | (uint32_t)~e : 0ull;
    ckey[lane] = mine64;
    __syncwarp();
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) rank += ckey[j] > mine64;
    if (by_value) {
      // values in descending order, each against the next: the first K must
      // lead by more than the two errors
      if (live) cval[rank] = x;
      __syncwarp();
      const float hi = cval[lane], lo = cval[(lane + 1) & 31];
      const bool close = lane < p.K && lane + 1 < count && !(hi - lo > fmaf(0x1p-23f, fabsf(hi) + fabsf(lo), 2.f * eps));
      if (__any_sync(kAll, close)) rank = rank_candidates64(p, row, top, e, count);
    }
    const bool in = live && rank < p.K;
    // weights from the accurate exponential; sigmoid by e^-|l|, which does not
    // overflow, softmax with what the rounding of l - top lost put back
    float w;
    if (p.sigmoid) {
      const float q = expf(-fabsf(l));
      w = __fdiv_rn(l < 0.f ? q : 1.f, 1.f + q);
    } else {
      const float d = l - top, back = d - l, lost = (l - (d - back)) - (top + back);
      const float q = expf(d);
      w = (q > 0.f ? fmaf(q, lost, q) : 0.f) * inv;
    }
    // a score of 0 is exact for a logit of -inf alone
    open = __any_sync(kAll, in && w < 0x1p-100f && l > -INFINITY);
    if (p.renorm) {
      const float total = warp_sum(in ? w : 0.f);
      w = __fdiv_rn(w, total);
      open = open || !(total > 0.f);  // none left
    }
    if (!open) {
      if (in) {
        p.idx[(size_t)t * p.K + rank] = e;
        p.w[(size_t)t * p.K + rank] = w * p.scale;
      }
      return;
    }
  }
  route_exact<T>(p, t, key, cand);
}

template <typename T, int NV>
cudaError_t launch_route_nv(const RouteParams& p, cudaStream_t st) {
  const size_t smem = sizeof(uint64_t) * kRouteWarps * (size_t)p.E;
  const auto kernel = p.bias ? route_kernel<T, NV, true> : route_kernel<T, NV, false>;
  if (smem > 40 * 1024) {  // the largest E only: 48 KB is the limit with the static 2 KB
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)(sizeof(uint64_t) * kRouteWarps * kRouteMaxExperts));
    if (e != cudaSuccess) return e;
  }
  return launch_early(kernel, (p.T + kRouteWarps - 1) / kRouteWarps, 32 * kRouteWarps, smem, 1, st, p);
}

template <typename T>
cudaError_t launch_route_t(const RouteParams& p, cudaStream_t st) {
  if (p.E <= 256) return launch_route_nv<T, 8>(p, st);
  if (p.E <= 512) return launch_route_nv<T, 16>(p, st);
  if (p.E <= 1024) return launch_route_nv<T, 32>(p, st);
  return launch_route_nv<T, 64>(p, st);
}

}  // namespace

cudaError_t launch_route(const RouteParams& p, int dtype, cudaStream_t st) {
  if (dtype == MOE_F32) return launch_route_t<float>(p, st);
  if (dtype == MOE_BF16) return launch_route_t<__nv_bfloat16>(p, st);
  return launch_route_t<__half>(p, st);
}

}  // namespace moe
