// Attention of a batch over a shared prefix and each request's own suffix:
// sizes of the launch and parameters of its kernels (attend.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace tsel {

constexpr int kAttMaxChunkKeys = 8192;   // keys of one unit: bounds its page list in shared memory
constexpr int kAttMinPage = 16;
constexpr int kAttMaxPages = kAttMaxChunkKeys / kAttMinPage;
// CTAs resident at once, one per SM. A constant, not a query: the workspace
// size must follow from the sizes alone.
constexpr int kAttCtas = 152;

// How a call is cut into units: (key chunk, KV head, row tiles) of the prefix,
// and (request, KV head, row tile, key chunk) of the suffixes.
struct AttPlan {
  int G;        // query heads per KV head
  int tt;       // tokens per 128-row tile
  int ntg;      // pairs of row tiles over all rows
  int nc, lp;   // prefix chunks and keys per chunk
  int qt;       // pairs of row tiles of one request
  int sc, ls;   // suffix chunks and keys per chunk
  int slots;    // partial results per row: two for each chunk
  int64_t units_p, units_s;
  int64_t lse_off, o_off, total;   // workspace
};

// Chunks for `base` units of `tiles` 128-key tiles each on `ctas` CTAs: the
// count with the least estimated time, in key tiles. A unit costs its tiles
// plus about kAttUnitTiles of start-up and write-out, and joining costs a
// little for each chunk.
constexpr int kAttUnitTiles = 3;
inline int att_chunks(int64_t base, int tiles, int ctas) {
  if (tiles <= 1 || base < 1) return tiles < 1 ? 0 : 1;
  const int least = int(ceil_div(tiles, kAttMaxChunkKeys / kTile));
  int best = least;
  double best_cost = 1e300;
  for (int n = least; n <= tiles && n <= 256; ++n) {
    const int per = int(ceil_div(tiles, n));
    if (n > least && int(ceil_div(tiles, per)) < n) continue;   // the same tiles in fewer chunks
    const double waves = double(ceil_div(base * n, ctas));
    const double cost = waves * (per + kAttUnitTiles) + 0.05 * n;
    if (cost < best_cost) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

inline AttPlan att_plan(int R, int Tq, int max_q, int H, int Hkv, int d, int max_prefix,
                        int max_suffix) {
  AttPlan a{};
  a.G = H / Hkv;
  a.tt = kTile / a.G;
  a.ntg = int(ceil_div(Tq, 2 * a.tt));
  const int kp = int(ceil_div(max_prefix, kTile));
  const int ks = int(ceil_div(max_suffix, kTile));
  a.qt = int(ceil_div(max_q, 2 * a.tt));
  if (Tq > 0) a.nc = att_chunks(int64_t(Hkv) * a.ntg, kp, kAttCtas);
  if (a.nc > 0) a.lp = int(ceil_div(kp, a.nc)) * kTile;
  if (Tq > 0 && R > 0 && a.qt > 0) a.sc = att_chunks(int64_t(R) * Hkv * a.qt, ks, kAttCtas);
  if (a.sc > 0) a.ls = int(ceil_div(ks, a.sc)) * kTile;
  a.slots = 2 * (a.nc + a.sc);
  a.units_p = int64_t(a.nc) * Hkv * a.ntg;
  a.units_s = int64_t(R) * Hkv * a.qt * a.sc;
  a.lse_off = kWsHeaderBytes;
  a.o_off = align_up(a.lse_off + 4 * int64_t(a.slots) * Tq * H, 256);
  a.total = align_up(a.o_off + 4 * int64_t(a.slots) * Tq * H * d, 256);
  return a;
}

struct AttParams {
  const void* q;
  int64_t q_stride;            // elements
  int fp16;                    // q and out: 1 fp16, 0 bf16
  const int32_t* cu_q;
  int R, Tq, max_q;
  const uint8_t* k_pages;
  const uint8_t* v_pages;
  const uint8_t* k_exps;
  const uint8_t* v_exps;
  int num_pages, page_shift;
  const int32_t* prefix_pages;
  const int32_t* prefix_len;   // device scalar
  int max_prefix;
  const int32_t* page_table;
  int64_t table_stride;
  const int32_t* suffix_lens;
  int max_suffix;
  int H, Hkv;
  float c;                     // softmax_scale * log2(e)
  int G, tt, ntg, nc, lp, qt, sc, ls, slots;
  int64_t unit0, units_p;      // this launch's first unit; prefix units of the call
  float* part_lse;             // [slots][Tq][H], base 2
  float* part_o;               // [slots][Tq][H][d]
  void* out;
  int64_t out_stride;
  float* lse;                  // [H][Tq] natural log, or null
  uint32_t* status;
  uint64_t timeout_ns;
};

cudaError_t launch_attend(int head_dim, const AttParams& p, int64_t units, cudaStream_t stream);
cudaError_t launch_attend_join(int head_dim, const AttParams& p, int num_sms, cudaStream_t stream);

}  // namespace tsel
