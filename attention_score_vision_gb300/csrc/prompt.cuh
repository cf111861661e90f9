// Attention over whole prompts: sizes of the launch and parameters of its
// kernel (prompt.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attend.cuh"

namespace tsel {

constexpr int kPromptStep = 64;       // keys of a step
// Units of a CTA up to which they are dealt out; beyond, they come from a counter (a
// memset before the launch). 24 requests of up to 1,370 rows, 14 units a CTA: 180 us
// with it, 197 without.
constexpr int kPromptDealt = 3;
constexpr int kPromptSorted = 256;    // segments up to which units go longest first

// Time of a unit of one row tile, for its keys, in that of one of two. A question of
// 142 rows (16 heads on 8 of 128: two row tiles and one) over 36,973 keys: 60.2 us
// with 0.85, 64.7 with 0.7, 71.3 with 0.6; in equal chunks for both 64.1.
constexpr double kPromptOne = 0.85;
// Chunks of the keys for row blocks of two row tiles (`full` of them, over all KV
// heads and segments) and of one (`light`), `tiles` 128-key tiles each: the counts with
// the least estimated time, in key tiles: a unit's, a block of one row tile taking
// less for each, and three for its start and end, and three for joining (256 rows of
// 256 keys, 4 heads of 64: 9.1 us in one chunk, 10.5 in two).
struct PromptChunks {
  int full, light;   // light <= full
};
inline PromptChunks prompt_chunks(int64_t full, int64_t light, int tiles) {
  PromptChunks best{1, 1};
  double best_cost = double(ceil_div(full + light, kAttWideCtas)) * ((full > 0 ? 1.0 : kPromptOne) * tiles + 3.0);
  for (int n = 1; n <= tiles && n <= 64 && full + n <= 2 * kAttWideCtas; ++n) {
    for (int m = full > 0 ? 1 : n; m <= n; ++m) {
      if (n == 1 && m == 1) continue;
      const int64_t units = full * n + light * m;
      if (units > 2 * kAttWideCtas) break;
      const double two = full > 0 ? double(ceil_div(tiles, n)) : 0.0, one = light > 0 ? kPromptOne * double(ceil_div(tiles, m)) : 0.0;
      const double cost = double(ceil_div(units, kAttWideCtas)) * ((two > one ? two : one) + 3.0) + 3.0 + 0.05 * n;
      if (cost < best_cost) {
        best_cost = cost;
        best = {n, m};
      }
    }
  }
  return best;
}

struct PromptPlan {
  int G, tt;           // query heads per KV head, tokens per 128-row tile
  int chunks, keys;    // key chunks of a segment, keys of one (a multiple of 128),
  int keys_one;        // and of one for a block of one row tile
  int64_t units;       // upper bound
  int slots;           // partial results of a row, 0: written at once
  int64_t lse_off, o_off, total;   // workspace
  bool too_large;
};

// Keys are cut into chunks only while the (segment, KV head, row block) units
// leave SMs idle. `base` estimates the units that have rows as if every segment had
// some and total_q were used up, so a batch padded with many empty segments is cut
// less than its lengths would allow.
inline PromptPlan prompt_plan(int seg, int Tq, int max_q, int max_k, int H, int Hkv, int d) {
  PromptPlan a{};
  a.G = H / Hkv;
  a.tt = kTile / a.G;
  const int64_t blocks = ceil_div(Tq, 2 * a.tt);
  const int64_t base = Hkv * (blocks > seg ? blocks : seg);
  const int tiles = int(ceil_div(max_k, kTile));
  PromptChunks n{1, 1};
  if (base > 0 && base < kAttWideCtas && tiles > 1) {
    // of one sequence the blocks are known; else all count as of two row tiles
    const int rest = max_q % (2 * a.tt);
    const int one = seg == 1 && rest > 0 && rest <= a.tt ? 1 : 0;
    const int64_t all = seg == 1 ? ceil_div(max_q < Tq ? max_q : Tq, 2 * a.tt) * Hkv : base;
    n = prompt_chunks(all - one * Hkv, one * Hkv, tiles);
    if (one == 0) n.light = n.full;
  }
  a.chunks = n.full;
  a.keys = a.chunks > 1 ? int(ceil_div(tiles, n.full)) * kTile : 0x7FFFFF80;
  a.keys_one = a.chunks > 1 ? int(ceil_div(tiles, n.light)) * kTile : a.keys;
  a.units = Hkv * (blocks + seg) * a.chunks;
  a.slots = a.chunks > 1 ? a.chunks : 0;
  a.too_large = double(a.slots) * Tq * H * d > 1e15 || a.units > (1ll << 40);
  if (a.too_large) return a;
  a.lse_off = kWsHeaderBytes;
  a.o_off = align_up(a.lse_off + 4 * int64_t(a.slots) * Tq * H, 256);
  a.total = align_up(a.o_off + 4 * int64_t(a.slots) * Tq * H * d, 256);
  return a;
}

struct PromptParams {
  const void* v;               // also read by threads where V holds infinities or NaN
  int64_t v_stride;            // elements
  const int32_t* cu_q;
  const int32_t* cu_k;
  int seg, Tq, Tk, max_q, max_k;
  int H, Hkv, G, tt;
  int causal;
  int chunks, keys, keys_one;
  float c;                     // softmax_scale * log2(e)
  int32_t* next;               // unit counter, 0 at the start; null: units are dealt out
  float* part_lse;             // [chunks][Tq][H], base 2; null: results are written at once
  float* part_o;               // [chunks][Tq][H][d]
  void* out;
  int64_t out_stride;
  float* lse;                  // [H][Tq] natural log, or null
  uint32_t* status;
  uint64_t timeout_ns;
};

cudaError_t launch_prompt(int head_dim, bool fp16, const CUtensorMap& mq, const CUtensorMap& mk,
                          const CUtensorMap& mv, const PromptParams& p, int ctas, cudaStream_t stream);

}  // namespace tsel
