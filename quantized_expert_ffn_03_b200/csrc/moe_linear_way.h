// moe_linear_way.h -- which kernel and tile a dense product takes, by its sizes
// and types alone (plain C++, host only).
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kKB = 64;        // columns of K per step: 128 bytes, one swizzle row
constexpr int kRowsTok = 16;   // tokens that the rows kernel takes at most
constexpr int kMaxSplit = 4;   // CTAs of a tile's cluster (16 clusters of 8 do not fit the GPCs at once)

// The tensor cores cut what an addition shifts out of the accumulator's 24
// bits, always towards zero, which makes a sum over many columns too small:
// for operands of one sign by 7.9 10^-6 of its size after 4096 columns of one
// accumulator, 6.5 10^-5 after 16384, 3.4 10^-4 after 65536, 1.5 10^-3 after
// 2^18 (measured; mixed signs a quarter of that, but 4.4 10^-6 after 4096).
// Where the output shows that, an accumulator holds kPart steps (512 columns),
// and the parts are added up in fp32, rounding to nearest: 2.4 10^-7 (mixed
// signs 4.8 10^-7) up to K = 16384, below 7.5 10^-7 at 2^20.
constexpr int kPart = 512 / kKB;
// The longest K that one accumulator takes: 512 columns for fp32 outputs, and
// for 16-bit ones what keeps the loss below 1/16 of half a step of the type
// (2^-11 for fp16, 2^-8 for bf16).  Parts need narrower tiles: fp16 2048 x 16384
// x 4096 takes 254 us with them, 193 without.
constexpr int longest_sum(bool out_f32, bool f16) { return out_f32 ? kPart * kKB : f16 ? 1 << 13 : 1 << 15; }

struct LinearWay {
  int tokens;  // of a tile: 8 or 16 (rows), 32 to 128 (tile), 256 (pair)
  int width;   // features of a rows block; of a tile; accumulator columns of a pair
  int split;   // CTAs that share a tile's K (tile), else 1
  bool sums;   // parts of K are added up in fp32 (tile, pair; the rows kernel always does)
  float ns;    // the estimate behind the choice (tile, pair)
};

// How long each way of doing a product takes, in ns, from measurements of the
// parts (steps of 64 columns of K): what a launch and a tile cost besides their
// steps, a step by what its copies move per SM (about 115 bytes per ns) or by
// its MMAs, an epilogue unit.  Against every way tried on 50 sizes (20 to 8192
// tokens, K 64 to 8192, N 512 to 16384) the way it picks is the fastest or
// mostly within 4 percent of it, at the worst 14; no one way is near the fastest
// everywhere (64 x 4096 x 4096: 9.8 us by clusters of 4 against 12.5 unsplit;
// 1024 x 4096 x 4096: 26 us by pairs of 256 columns against 36 by tiles;
// 2048 x 1024 x 1024 gated: 9.7 us by pairs of 128 columns, 10.8 by 256).
// sums: tiles of at most 64 features and pairs of 128 columns alone (those that
// keep sums in registers).
inline LinearWay tensor_way(int T, int K, int N, bool gated, bool sums, int sms) {
  auto max_f = [](float a, float b) { return a > b ? a : b; };
  const int KB = (K + kKB - 1) / kKB, na = gated ? 2 : 1;
  LinearWay best = {0, 0, 1, sums, 1e30f};
  const int BT = T <= 32 ? 32 : T <= 64 ? 64 : 128;
  for (int FN = 32; FN <= (gated || sums ? 64 : 128); FN *= 2) {
    const int64_t tiles = (int64_t)((N + FN - 1) / FN) * ((T + BT - 1) / BT);
    if (tiles > 8 * sms) continue;
    for (int S = 1; S <= kMaxSplit && S <= KB; S *= 2) {
      const int64_t waves = (tiles * S + (S == 4 ? 127 : sms - 1)) / (S == 4 ? 128 : sms);
      const float step = max_f(170.f, (float)(BT + na * FN) * 128.f / 115.f);
      const int units = (FN / 32 + 1) / 2;  // of a warp
      const float tail = S == 1 ? 500.f * units
                                : (S == 4 && BT == 128 ? 2000.f : 1100.f) + 300.f * (S - 1) + 500.f * ((units + S - 1) / S);
      const float ns = (float)waves * (2500.f + (float)((KB + S - 1) / S) * step + na * tail);
      if (ns < best.ns) best = {BT, FN, S, sums, ns};
    }
  }
  for (int TN = 128; TN <= (sums ? 128 : 256); TN *= 2) {
    const int FN = TN / na;
    const int64_t tiles = (int64_t)((T + 255) / 256) * ((N + FN - 1) / FN);
    const int64_t waves = (tiles + sms / 2 - 1) / (sms / 2);
    const float steps = (float)KB * (TN == 256 ? 310.f : 195.f), epilogue = (TN == 256 ? 450.f : 520.f) * FN / 64 * na;
    const float ns = 3300.f + (float)waves * max_f(steps, epilogue) + epilogue;
    if (ns < best.ns) best = {256, TN, 1, sums, ns};
  }
  return best;
}

inline LinearWay linear_way(int T, int K, int N, bool gated, bool f16, bool out_f32, int sms) {
  // 9 to 16 tokens: weights beyond about 40 MB stream faster by TMA (8192 x 8192:
  // 27 us against 35; 4096 x 4096: 9.5 against 9.3)
  const bool heavy = (int64_t)N * K * (gated ? 2 : 1) > (20 << 20);
  if (T <= 8 || (T <= kRowsTok && !heavy)) return {T <= 8 ? 8 : 16, 8, 1, false, 0.f};
  return tensor_way(T, K, N, gated, K > longest_sum(out_f32, f16), sms);
}

}  // namespace moe
