// Pages of the quantised cache: parameters of the kernels that move cached
// tokens together, share pages and give them out (pages.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace tsel {

constexpr int kMoveThreads = 256;
// 16-byte pieces of a thread in flight, and CTAs of an SM. 36,831 tokens, 8 heads of
// 128, to other pages: 8 pieces and 3 CTAs 34.1 us, 4 and 3 32.9, 4 and 6 30.8,
// 3 and 8 30.1, 2 and 8 35.3.
constexpr int kMoveItems = 3, kMoveCtas = 8;
// The same in place, where a thread holds two chunks' pieces: the 36,831 tokens of one
// request, of 61,385, 177 us with 6 pieces and 2 CTAs, 216 with 5, 267 with 8 (spills).
constexpr int kMoveItemsInPlace = 6, kMoveCtasInPlace = 2;
constexpr int kMoveMaxTokens = 1024;  // of a chunk: 48 KB of row numbers for three
constexpr int kMoveHeads = 32;        // K and V heads of a CTA, at most
// CTAs of a child. 256 children, 8 heads of 128, up to 127 rows copied each, forked,
// grown and freed, without the checks of lists and shared pages (1.3 us): 28.0 us with
// 8, 29.8 with 4, 30.4 with 16, 36.9 with 32.
constexpr int kForkParts = 8;

struct MoveParams {
  uint8_t* k_pages;
  uint8_t* v_pages;
  uint8_t* k_exps;
  uint8_t* v_exps;
  int num_pages, page_shift, Hkv, d;
  const int32_t* table;
  int64_t table_stride;
  int width;                   // pages of a row of it
  const int32_t* dst_table;    // null: in place
  int64_t dst_stride;
  int dst_width;
  const int32_t* starts;       // [R] or null
  const int32_t* bases;        // [R] or null
  const int32_t* keep;
  const int32_t* cu_keep;      // [R + 1]
  int total, max_keep, R;
  int32_t* new_lens;           // [R] or null
  uint32_t* status;
  int heads;                   // K and V heads of a CTA (of 2 Hkv)
  int head_parts;              // CTAs that share the heads
  int pieces, slices;          // 16-byte pieces of a CTA's rows, CTAs that share a row
  int tokens;                  // of a chunk
  int chunks;                  // of a request; 1 in place, where a CTA walks them itself
};

struct PagesParams {
  int32_t* refs;
  int num_pages, page_shift;
  int32_t* table;
  int64_t table_stride;
  int rows, width;
  int32_t* lens;
  const int32_t* new_lens;     // resize
  const int32_t* parents;      // fork
  const int32_t* children;
  int n;
  uint8_t* k_pages;
  uint8_t* v_pages;
  uint8_t* k_exps;
  uint8_t* v_exps;
  int Hkv, d;
  int parts;                   // CTAs of a child
  int32_t* plan;               // [rows + 1]
  int32_t* found;              // [rows * width], [rows] at least
  uint32_t* status;
};

// Sizes of a compaction's launch; CTAs enough for `want` where there is work.
void move_plan(MoveParams& p, int want);
cudaError_t launch_move(const MoveParams& p, cudaStream_t stream);
cudaError_t launch_resize(const PagesParams& p, cudaStream_t stream);
cudaError_t launch_fork(const PagesParams& p, cudaStream_t stream);

}  // namespace tsel
