// Attention of a batch over a shared prefix and each request's own suffix:
// sizes of the launch and parameters of its kernels (attend.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace tsel {

constexpr int kAttMaxChunkKeys = 8192;   // keys of a wide unit: bounds its page list in shared memory
constexpr int kAttMinPage = 16;
constexpr int kAttMaxKeys = 1 << 30;     // of a prefix or a suffix: key numbers and chunk ends stay in 31 bits
constexpr int kAttMaxPages = kAttMaxChunkKeys / kAttMinPage;
// CTAs resident at once on the 152 SMs: one wide CTA per SM, four or three narrow
// ones. Constants, not queries: the workspace size must follow from the sizes alone.
constexpr int kAttWideCtas = 152;
constexpr int kAttNarrowCtas1 = 4 * 152, kAttNarrowCtas2 = 3 * 152;
// Query rows (tokens times query heads per KV head) up to which the narrow
// kernel takes the keys of a prefix or of a request's suffix. More than one
// group of 16 rows reads the keys twice, which pays while start-up counts, or
// while every SM has requests of its own. 8 KV heads of 128, narrow against wide:
// 32 rows over one prefix of 600 keys 11.8 and 13.3 us, of 2,000 15.8 and 17.8,
// of 5,000 18.8 and 17.7, of 12,000 25.0 and 25.4, of 36,831 53.5 and 43.2; 64
// requests of 32 rows with up to 800 keys 42.7 and 59.3, with 3,000 102 and 148;
// 64 rows over 2,000 keys 19.4 and 21.8, over 36,831 75.9 and 47.8. The rule goes
// by rows: past 32 it gives away the 2 us of a short prefix for the 28 of a long
// one. The rows of a suffix are bounded by the longest request of the batch.
constexpr int kAttNarrowRows = 32;
constexpr int kAttNarrowRowsLong = 16;         // past
constexpr int kAttNarrowKeys = 16384;          // this many keys of few requests

constexpr int kAttJoinedTiles = 1024;          // 128-key tiles of suffixes that a prefix's narrow launch takes along

// How the prefix, or the suffixes, are cut into units: (key chunk, KV head, row
// group), for the suffixes of each request.
struct AttPart {
  int narrow;          // attend_narrow.cu with 8 or 16 rows to a unit (1, 2), else attend.cu (0)
  int groups;          // row groups: of 8 or 16 rows, or pairs of 128-row tiles
  int chunks, keys;    // key chunks, keys of one
  int slot0;           // partial results of a row: one for each narrow chunk, two for each wide one
  int64_t units;
};

struct AttPlan {
  int G;               // query heads per KV head
  int tt;              // tokens per 128-row tile
  AttPart pre, suf;
  int slots;
  int64_t lse_off, o_off, total;   // workspace
  bool too_large;      // units or partial results past what is counted in 31 bits or fits any memory
};

// Chunks, at least `least`, for `base` units of `tiles` 128-key tiles each on
// `ctas` CTAs: the count with the least estimated time, in key tiles. A unit
// costs its tiles plus a start-up, and joining costs a little for each chunk.
//   Wide units (start-up 3 tiles) fill their SMs and take equal times: whole
// waves of them count.
//   Narrow units (start-up 1 tile) share theirs. Beyond one full wave they even
// out over the SMs, less half a unit at the end, but a wave that is barely
// exceeded costs half of another: 16 requests with 4,000 keys each, 8 KV heads
// of 128, in 4, 8, 16 chunks: 32.4, 23.2, 27.1 us; 64 such requests in 1, 4, 16
// chunks: 88.8, 65.1, 79.5 us; a prefix of 36,831 keys and 8 rows in 58, 72, 96
// chunks (0.8, 0.9, 1.3 waves): 27.2, 25.3, 29.2 us.
inline int att_chunks(int64_t base, int tiles, int ctas, bool narrow, int least) {
  if (tiles <= 1 || base < 1) return tiles < 1 ? 0 : 1;
  int best = least;
  double best_cost = 1e300;
  int per = 0;
  for (int n = least; n <= tiles && n <= 256 + least; n = per > 1 ? int(ceil_div(tiles, per - 1)) : tiles + 1) {
    per = int(ceil_div(tiles, n));   // the next count is the least that makes it smaller
    const double fill = double(base * n) / ctas;
    const double waves = !narrow ? double(ceil_div(base * n, ctas))
                                 : (fill <= 1.0 ? 1.0 : (fill < 1.5 ? 1.5 : fill)) + 0.5;
    const double cost = waves * (per + (narrow ? 1.0 : 3.0)) + 0.05 * n;
    if (cost < best_cost) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

// `two`: units of 16 rows even where 8 would do.
inline AttPart att_part(int64_t requests, int tokens, int max_keys, int Hkv, int G, int tt, bool two, int* slots) {
  AttPart a{};
  const int64_t rows = int64_t(tokens) * G;
  const bool few = max_keys > kAttNarrowKeys && requests * Hkv < kAttWideCtas;
  a.narrow = rows > (few ? kAttNarrowRowsLong : kAttNarrowRows) ? 0 : (rows > 8 || two ? 2 : 1);
  a.groups = int(a.narrow ? ceil_div(rows, 8 * a.narrow) : ceil_div(tokens, 2 * tt));
  a.slot0 = *slots;
  const int tiles = int(ceil_div(max_keys, kTile));
  const int64_t base = requests * Hkv * a.groups;
  if (base < 1 || tiles < 1) return a;
  if (base > 0x7FFFFFFFll) {   // too large in any number of chunks, and base * chunks could pass 63 bits
    a.units = base;
    return a;
  }
  a.chunks = a.narrow ? att_chunks(base, tiles, a.narrow == 1 ? kAttNarrowCtas1 : kAttNarrowCtas2, true, 1)
                      : att_chunks(base, tiles, kAttWideCtas, false, int(ceil_div(tiles, kAttMaxChunkKeys / kTile)));
  a.keys = int(ceil_div(tiles, a.chunks)) * kTile;
  a.units = base * a.chunks;
  *slots += a.chunks * (a.narrow ? 1 : 2);
  return a;
}

inline AttPlan att_plan(int R, int Tq, int max_q, int H, int Hkv, int d, int max_prefix,
                        int max_suffix) {
  AttPlan a{};
  a.G = H / Hkv;
  a.tt = kTile / a.G;
  a.pre = att_part(1, Tq, max_prefix, Hkv, a.G, a.tt, false, &a.slots);
  // Beside a prefix in units of 16 rows, short suffixes join its launch: 8 users
  // of 1,228 shared keys and up to 142, 1,000, 4,000 of their own on 8 KV heads
  // of 128 take 10.9, 14.1, 23.2 us in one launch and 11.9, 15.9, 21.9 in two
  // (called, not replayed: 24.5, 25.0, 24.4 and 25.9, 26.5, 26.5).
  const bool two = a.pre.narrow == 2 && a.pre.units > 0 &&
                   int64_t(R) * Hkv * ceil_div(max_suffix, kTile) <= kAttJoinedTiles;
  a.suf = att_part(Tq > 0 ? R : 0, max_q, max_suffix, Hkv, a.G, a.tt, two, &a.slots);
  a.too_large = a.pre.units + a.suf.units > 0x7FFFFFFFll || double(a.slots) * Tq * H * d > 1e15;
  if (a.too_large) return a;
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
  int G, tt, slots;
  AttPart pre, suf;
  uint32_t pre_units;          // prefix units of this launch (its first ones); the rest are suffix units
  float* part_lse;             // [slots][Tq][H], base 2
  float* part_o;               // [slots][Tq][H][d]
  void* out;
  int64_t out_stride;
  float* lse;                  // [H][Tq] natural log, or null
  uint32_t* status;
  uint64_t timeout_ns;
};

// Keys [k0, k1) of a page list and the rows that see them: row i of a suffix
// sees the first lim0 + i keys (of the suffix's tokens tok_first ...), rows of
// the prefix the first lim0.
struct AttUnit {
  int kvh, slot, group;
  int tok_first, tok_last;   // tokens [tok_first, tok_last) of the request (prefix: of the batch)
  int k0, k1;
  int lim0;
  int causal;
  const int32_t* pages;
  bool bad;
};

// `per`: rows of a row group; the keys of a suffix unit end where its last row sees no further.
// U is the type that the unit number is divided in. Both give the same numbers;
// what differs is the code that nvcc 13.0 makes of the kernels around them, by no
// rule known here, so each kernel has the one that measures better with it:
// uint32_t the wide one (16 question prefills 390 us, 438 with int64_t), int64_t
// the narrow one (four users of a six-view request 7.9 us, 9.6 with uint32_t;
// other cases within 1%). To be measured again with another compiler.
template <typename U>
__device__ __forceinline__ AttUnit att_unit(const AttParams& p, U u, int per) {
  AttUnit w{};
  if (u < U(p.pre_units)) {
    const U ch = u / U(p.pre.groups);   // neighbouring units share their keys
    w.group = int(u - ch * U(p.pre.groups));
    const int c = int(ch / U(p.Hkv));
    w.kvh = int(ch) - c * p.Hkv;
    w.slot = p.pre.slot0 + c * (p.pre.narrow ? 1 : 2);
    const int n = __ldg(p.prefix_len);
    w.tok_last = __ldg(p.cu_q + p.R);
    w.bad = n < 0 || n > p.max_prefix || w.tok_last < 0 || w.tok_last > p.Tq;
    if (w.bad) return w;
    w.k0 = min(c * p.pre.keys, n);
    w.k1 = min(w.k0 + p.pre.keys, n);
    w.lim0 = n;
    w.pages = p.prefix_pages;
  } else {
    u -= U(p.pre_units);
    const U a1 = u / U(p.suf.chunks), a2 = a1 / U(p.suf.groups);
    const int c = int(u - a1 * U(p.suf.chunks));
    w.group = int(a1 - a2 * U(p.suf.groups));
    const int r = int(a2 / U(p.Hkv));
    w.kvh = int(a2) - r * p.Hkv;
    w.slot = p.suf.slot0 + c * (p.suf.narrow ? 1 : 2);
    const int a = __ldg(p.cu_q + r), b = __ldg(p.cu_q + r + 1);
    const int n = __ldg(p.suffix_lens + r);
    w.bad = a < 0 || b < a || b > p.Tq || b - a > p.max_q || n < 0 || n > p.max_suffix ||
            (r == 0 && a != 0);
    if (w.bad) return w;
    w.tok_first = a;
    w.tok_last = b;
    w.causal = 1;
    w.lim0 = n - (b - a) + 1;
    const int last = min((w.group + 1) * per, (b - a) * p.G);   // rows up to here
    const int seen = max(min(n, w.lim0 + (last - 1) / p.G), 0);
    w.k0 = min(c * p.suf.keys, seen);
    w.k1 = min(w.k0 + p.suf.keys, seen);
    w.pages = p.page_table + r * p.table_stride;
  }
  return w;
}

cudaError_t launch_attend(int head_dim, const AttParams& p, int64_t units, cudaStream_t stream);
cudaError_t launch_attend_narrow(int head_dim, int row_groups, const AttParams& p, int64_t units,
                                 cudaStream_t stream);
cudaError_t launch_attend_join(int head_dim, const AttParams& p, cudaStream_t stream);

}  // namespace tsel
