// Which kernel reads the prefix of a shared-prefix decode, and into how many splits prefix and own keys are
// cut.  Host code without CUDA, so that a test can ask which kernel its sizes reach.
#pragma once

#include <algorithm>

namespace fa {

constexpr int kSms = 148;

// Blocks of heads (or rows) that launch_split_rows makes of G, and its CTAs that fit the GPU at once.
inline long long split_blocks(long long G) { return G > 8 ? (G + 15) / 16 : 1; }
inline long long split_slots(long long G) { return (G > 8 ? 2 : 3) * kSms; }

// Whether the prefix, as one sequence of R rows per KV head, goes through the split kernel too (rows in
// blocks of 16, each block reading the cache again from L2) or through the tcgen05 kernel (128 or 256
// rows a tile).  With T tiles of 128 keys per SM, B200, 8 KV heads of 128 dims, INT8:
//   split 10 us + 1.0 T per block of 16 rows;  tcgen05 14 us + 1.45 T, twice that for a block of 256 rows
// (131072 keys, T = 55: 16 rows 70 / 93 us, 32 rows 117 / 95 us; 4096 keys, 48 rows 23 / 25 us, 96 rows
// 29 / 27 us).  At D = 64 a block of 16 costs half, a tcgen05 tile, bound by its softmax, the same.
// More CTAs of the split kernel than half of what fits, beside those of the own keys, would take a second wave.
inline bool shared_through_split(int D, long long R, int Hkv, long long max_keys) {
  const double T = static_cast<double>(Hkv) * ((max_keys + 127) / 128) / kSms;
  const double tile = R <= 128 ? 1.0 : 2.0 * ((R + 255) / 256);
  return Hkv * split_blocks(R) <= split_slots(R) / 2 &&
         split_blocks(R) * T < (D == 128 ? 1.45 : 2.2) * tile * T + 4.0;
}

// Splits of the prefix: the count with the least estimate of tile times, the smaller of equals.  A split
// costs the merge about 0.06 us, 1/17 of the split kernel's tile or 1/25 of the tcgen05 kernel's (one KV head,
// 8 rows, 32768 keys as one paged sequence: 256 / 128 / 64 / 32 splits 19.4 / 12.7 / 11.6 / 12.2 us).  Through the split kernel as many as
// its CTAs find room for beside those of the own keys.  Otherwise one CTA per SM runs a split of one (KV head,
// row block) in about (tiles + 3) tile times (start-up and epilogue count for three), in as many
// waves as the CTAs need on the SMs that it leaves to the own keys' kernel: their share of the work, a
// CTA of own keys a third of an SM for 4.5 us and 1.1 us a stage (half of the longest sequence).
inline int shared_prefix_splits(int D, int B, int Hq, int Hkv, long long max_keys, int own_splits,
                                long long max_own) {
  const long long R = static_cast<long long>(B) * (Hq / Hkv);
  const long long tiles = std::max(1ll, (max_keys + 127) / 128);
  const bool few = shared_through_split(D, R, Hkv, max_keys);
  const long long base = Hkv * (few ? split_blocks(R) : R <= 128 ? 1 : (R + 255) / 256);
  const long long own = static_cast<long long>(B) * Hkv * split_blocks(Hq / Hkv) * own_splits;
  long long limit = kSms, sms = kSms;
  if (few) {
    const long long slots = split_slots(R);
    limit = std::max(1ll, (slots - std::min(own, slots / 2)) / base);
  } else {
    const double stages = std::max(1.0, 0.5 / 128 * max_own / own_splits);
    const double own_time = own * (4.5 + 1.1 * stages) / 3;
    const double time = base * tiles * (R <= 128 ? 1.4 : 2.5) + 9.0 * kSms;
    sms -= std::min<long long>(kSms / 5, static_cast<long long>(kSms * own_time / (own_time + time) + 0.5));
  }
  // by tiles a split, fewest first; of the counts with the same tiles a split, the smallest
  long long best = 1;
  double best_cost = 1e30;
  for (long long per = (tiles + limit - 1) / limit; per <= tiles && per < best_cost; ++per) {
    const long long s = (tiles + per - 1) / per;
    const double cost = few ? per + s / 17.0 : (base * s + sms - 1) / sms * (per + 3.0) + s / 25.0;
    if (cost <= best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return static_cast<int>(best);
}

// Splits of the sequences' own keys where the caller leaves the choice to the library: pieces of 512 keys
// or more (a sequence no longer than that is one piece), as long as all CTAs fit the GPU at once, or
// twice as many, of which about half find nothing to do.  The prefix's kernel runs beside or right
// behind this one on the same SMs, so fewer, longer CTAs beat a full GPU: B200, pieces of 256 / 512 / 1024
// keys, 32 x 32 heads, 1024 own keys 35.0 / 30.9 / 32.9 us; INT4, 13 x 28 heads, 777 keys 24.7 / 22.6 /
// 22.6 us; as many splits as fill the GPU, 12 x 232 heads of 64 dims, 256 keys 39 us for 33.
constexpr int kSharedOwnChunk = 512;
inline int shared_own_splits(int B, int Hq, int Hkv, long long max_keys) {
  const long long ctas = static_cast<long long>(B) * Hkv * split_blocks(Hq / Hkv);
  const long long fit = split_slots(Hq / Hkv) / ctas;
  return static_cast<int>(std::max(
      1ll, std::min(fit == 1 ? 2 : fit, (max_keys + kSharedOwnChunk - 1) / kSharedOwnChunk)));
}

}  // namespace fa
