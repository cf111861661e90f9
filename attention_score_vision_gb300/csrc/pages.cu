// Pages of the quantised cache: the rows of kept tokens moved together (accepted
// drafts, a pruned prompt), pages shared by requests that start from another one,
// and pages given out and back. Dynamic vision-token compression article, section
// 3.2: after pruning the KV cache holds the kept tokens.
//
// cache_move_kernel. Token k of a request's kept list goes from position
// start + keep[k] - base to start + k: cached bytes move unchanged. A thread owns
// one 16-byte piece of rows and has a few of them in flight. A CTA covers some of
// the K and V heads (and, where requests are few, some pieces of their rows) for
// one chunk of tokens; a chunk's row numbers are worked out once in shared memory.
//   In place the destination of one token may be the source of another. Kept
// indices ascend, so a token's source is at or behind its destination and a
// destination is the source of this chunk's tokens or earlier ones', never of
// later ones'. So a CTA takes all the chunks of a request in order and every load
// of a chunk comes before its stores (one barrier); CTAs of other heads or pieces
// touch other bytes. (Through a workspace there would be no order to keep, and twice
// the bytes.)
//   To other pages it is bound by HBM and issue: 36,831 tokens, 8 heads of 128 (152 MB),
// 30.1 us, 5.05 TB/s, 76% of the copy rate; schedulers issue in 80% of the cycles
// (row numbers for 16-byte pieces). In place the chunks of a request follow one
// another, on at most 64 CTAs for one of 8 heads of 128: 177 us for the same tokens,
// five times as long (four requests at once 216), a chunk of 768 tokens every 3.7 us.
//
// cache_resize_kernel, fork_plan_kernel. Reference counts are whole numbers added
// with atomics, so their order does not matter; free pages (count 0) are found by
// one CTA that walks the counts 8,192 at a time until it has enough, and go, lowest
// first, to rows in order: results are deterministic. Pages given back are a launch
// of their own, a CTA for each row: one SM adds about one scattered count a clock
// (256 rows of up to 289 pages freed in the first launch's CTA: 50 us, in CTAs of
// their own 17). A row that grows by a few pages is a thread's, by many a warp's (a
// warp for each of 264 rows: 9.7 us, 4.5 so).
//   What bounds them: chains of dependent loads of one CTA, 4 to 8 us alone in pools of
// some thousand pages with free ones among the first; each 8,192 pages in use in front of
// them are one more round. Forking 16 requests into 64 and 8 into 256 the copies of last
// pages, 6 and 16 us. Forked, grown and freed these take 18.7 and 28.9 us; 1.3 of that
// keep what a caller got wrong from others' pages (children out of order, growth behind
// a shared page).
#include "launch_util.cuh"
#include "pages.cuh"

namespace tsel {

namespace {

__device__ __forceinline__ int ceil_pages(int n, int shift) { return int((int64_t(n) + (1 << shift) - 1) >> shift); }

template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, IN_PLACE ? kMoveCtasInPlace : kMoveCtas) cache_move_kernel(const MoveParams p) {
  constexpr int kItems = IN_PLACE ? kMoveItemsInPlace : kMoveItems;
  extern __shared__ int64_t s_rows[];   // [chunk mod 3][source, destination][tokens]: rows of head 0, -1 none
  pdl_wait();
  pdl_launch_dependents();
  unsigned b = blockIdx.x;
  const int slice = int(b % unsigned(p.slices));
  b /= unsigned(p.slices);
  const int part = int(b % unsigned(p.head_parts));
  b /= unsigned(p.head_parts);
  const int first_chunk = int(b % unsigned(p.chunks)), r = int(b / unsigned(p.chunks));
  const int a = __ldg(p.cu_keep + r), e = __ldg(p.cu_keep + r + 1);
  const int start = p.starts != nullptr ? __ldg(p.starts + r) : 0, base = p.bases != nullptr ? __ldg(p.bases + r) : 0;
  const bool lead = threadIdx.x == 0 && part == 0 && slice == 0 && first_chunk == 0;
  const int64_t room = int64_t(IN_PLACE ? p.width : p.dst_width) << p.page_shift;
  if (a < 0 || e < a || e > p.total || e - a > p.max_keep || (r == 0 && a != 0) || start < 0 || int64_t(start) + (e - a) > room) {
    if (lead) {
      set_status(p.status, TSEL_DEV_REQUESTS);
      if (p.new_lens != nullptr) p.new_lens[r] = -1;
    }
    return;
  }
  const int n = e - a;
  if (lead && p.new_lens != nullptr) p.new_lens[r] = start + n;
  const int chunks = int(ceil_div(n, p.tokens));
  if (first_chunk >= chunks) return;

  const int32_t* table = p.table + r * p.table_stride;
  const int32_t* to = IN_PLACE ? table : p.dst_table + r * p.dst_stride;
  const int mask = (1 << p.page_shift) - 1;
  // Rows of a chunk's tokens: [(page * Hkv) << shift] + place. In place four tokens of
  // a thread at a time, so that their two loads in a row overlap.
  auto find = [&](int c, int64_t* rows) {
    if constexpr (!IN_PLACE) {
      for (int i = threadIdx.x; i < p.tokens; i += kMoveThreads) {
        const int k = c * p.tokens + i;
        int64_t src = -1, dst = -1;
        if (k < n) {
          const int64_t rel = int64_t(__ldg(p.keep + a + k)) - base;
          const int64_t at = start + rel;
          if (rel < k || at >= int64_t(p.width) << p.page_shift || (k > 0 && rel <= int64_t(__ldg(p.keep + a + k - 1)) - base)) {
            set_status(p.status, TSEL_DEV_KEEP_IDX);
          } else {
            const int put = start + k;
            const int pg = __ldg(table + (at >> p.page_shift)), pd = __ldg(to + (put >> p.page_shift));
            if (pg < 0 || pg >= p.num_pages || pd < 0 || pd >= p.num_pages) {
              set_status(p.status, TSEL_DEV_PAGES);
            } else {
              src = ((int64_t(pg) * p.Hkv) << p.page_shift) + (at & mask);
              dst = ((int64_t(pd) * p.Hkv) << p.page_shift) + (put & mask);
            }
          }
        }
        rows[i] = src;
        rows[p.tokens + i] = dst;
      }
    } else {
      for (int i0 = threadIdx.x; i0 < p.tokens; i0 += 4 * kMoveThreads) {
        int64_t rel[4], before[4];
        int pg[4], pd[4];
        unsigned moves = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = i0 + x * kMoveThreads, k = c * p.tokens + i;
          const bool in = i < p.tokens && k < n;
          rel[x] = in ? int64_t(__ldg(p.keep + a + k)) - base : -1;
          before[x] = in && k > 0 ? int64_t(__ldg(p.keep + a + k - 1)) - base : -1;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = i0 + x * kMoveThreads, k = c * p.tokens + i;
          pg[x] = pd[x] = -1;
          if (i >= p.tokens || k >= n) continue;
          if (rel[x] < k || start + rel[x] >= int64_t(p.width) << p.page_shift || (k > 0 && rel[x] <= before[x])) {
            set_status(p.status, TSEL_DEV_KEEP_IDX);
          } else if (rel[x] != k) {
            moves |= 1u << x;
            pg[x] = __ldg(table + ((start + rel[x]) >> p.page_shift));
            pd[x] = __ldg(to + ((start + k) >> p.page_shift));
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int i = i0 + x * kMoveThreads, put = start + c * p.tokens + i;
          if (i >= p.tokens) continue;
          const bool good = pg[x] >= 0 && pg[x] < p.num_pages && pd[x] >= 0 && pd[x] < p.num_pages;
          if (!good && ((moves >> x) & 1u)) set_status(p.status, TSEL_DEV_PAGES);
          rows[i] = good ? ((int64_t(pg[x]) * p.Hkv) << p.page_shift) + ((start + rel[x]) & mask) : -1;
          rows[p.tokens + i] = good ? ((int64_t(pd[x]) * p.Hkv) << p.page_shift) + (put & mask) : -1;
        }
      }
    }
  };

  const int head0 = part * p.heads, heads = min(p.heads, 2 * p.Hkv - head0);
  const int piece0 = slice * p.pieces, pieces = min(p.pieces, p.d / 16 - piece0);
  const int groups = kMoveThreads / p.pieces;
  const int group = int(threadIdx.x) / p.pieces, piece = int(threadIdx.x) - group * p.pieces;
  const bool works = group < groups && piece < pieces;
  const bool scales = works && piece == 0 && slice == 0;   // also moves the row's scale byte
  // item i of this thread: (token, head), head fastest, `groups` apart
  const int tok_step = groups / heads, head_step = groups - tok_step * heads;
  auto rows_of = [&](int c) -> int64_t* { return s_rows + (c % 3) * 2 * p.tokens; };
  auto each = [&](int c, auto&& f) {
    const int left = min(n - c * p.tokens, p.tokens);
    int tok = group / heads, h = group - tok * heads;
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
      if (works && tok < left) f(i, tok, head0 + h);
      tok += tok_step;
      h += head_step;
      if (h >= heads) {
        h -= heads;
        ++tok;
      }
    }
  };
  auto load = [&](int c, const int64_t* rows, uint4 (&data)[kItems], uint8_t (&exps)[kItems]) {
    each(c, [&](int i, int tok, int h) {
      const int64_t row = rows[tok];
      if (row < 0) return;
      const bool v = h >= p.Hkv;
      const int64_t at = row + (int64_t(v ? h - p.Hkv : h) << p.page_shift);
      data[i] = __ldcg(reinterpret_cast<const uint4*>((v ? p.v_pages : p.k_pages) + at * p.d) + piece0 + piece);
      if (scales) exps[i] = __ldcg((v ? p.v_exps : p.k_exps) + at);
    });
  };
  auto store = [&](int c, const int64_t* rows, const uint4 (&data)[kItems], const uint8_t (&exps)[kItems]) {
    each(c, [&](int i, int tok, int h) {
      if (rows[tok] < 0) return;
      const bool v = h >= p.Hkv;
      const int64_t at = rows[p.tokens + tok] + (int64_t(v ? h - p.Hkv : h) << p.page_shift);
      reinterpret_cast<uint4*>((v ? p.v_pages : p.k_pages) + at * p.d)[piece0 + piece] = data[i];
      if (scales) ((v ? p.v_exps : p.k_exps) + at)[0] = exps[i];
    });
  };
  uint4 data[kItems];
  uint8_t exps[kItems];
  if constexpr (!IN_PLACE) {
    find(first_chunk, s_rows);
    __syncthreads();
    load(first_chunk, s_rows, data, exps);
    store(first_chunk, s_rows, data, exps);
  } else {
    // Every load of a chunk comes before its stores: the barrier between them. The
    // next chunk's loads go out before this one's stores. Row numbers are kept for
    // three chunks: the last one's stores may still read theirs.
    uint4 more[kItems];
    uint8_t more_exps[kItems];
    find(0, rows_of(0));
    __syncthreads();
    load(0, rows_of(0), data, exps);
    for (int c = 0;; c += 2) {
      if (c + 1 < chunks) find(c + 1, rows_of(c + 1));
      __syncthreads();
      if (c + 1 < chunks) load(c + 1, rows_of(c + 1), more, more_exps);
      store(c, rows_of(c), data, exps);
      if (c + 1 >= chunks) break;
      if (c + 2 < chunks) find(c + 2, rows_of(c + 2));
      __syncthreads();
      if (c + 2 < chunks) load(c + 2, rows_of(c + 2), data, exps);
      store(c + 1, rows_of(c + 1), more, more_exps);
      if (c + 2 >= chunks) break;
    }
  }
}

// ---------------------------------------------------------------------------
// Counts
// ---------------------------------------------------------------------------

constexpr int kPagesThreads = 1024;
constexpr int kPagesWarps = kPagesThreads / 32;
constexpr int kPagesPerLane = 8;

// Inclusive sums (MAX: largest values) over the block's threads; of all in *total.
template <bool MAX>
__device__ __forceinline__ int block_scan(int mine, int* s_warps, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto both = [](int a, int b) { return MAX ? max(a, b) : a + b; };
  int v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = both(v, y);
  }
  __syncthreads();   // the results of the call before have been read
  if (lane == 31) s_warps[warp] = v;
  __syncthreads();
  int before = s_warps[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before = both(before, y);
  }
  *total = __shfl_sync(0xffffffffu, before, 31);
  const int up_to = __shfl_sync(0xffffffffu, before, max(warp - 1, 0));   // of the warps before
  return warp > 0 ? both(v, up_to) : v;
}
__device__ __forceinline__ int block_sum(int mine, int* s_warps, int* total) { return block_scan<false>(mine, s_warps, total); }

// Writes the lowest `want` free pages into list; returns how many there are (at
// most `want`).
__device__ int free_pages(const int32_t* refs, int num_pages, int want, int32_t* list, int* s_warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int got = 0;
  for (int64_t base = 0; base < num_pages && got < want; base += kPagesThreads * kPagesPerLane) {
    const int64_t first = base + warp * (32 * kPagesPerLane) + lane;
    unsigned free_[kPagesPerLane];
    int count = 0;
#pragma unroll
    for (int i = 0; i < kPagesPerLane; ++i) {
      const int64_t page = first + 32 * i;
      free_[i] = __ballot_sync(0xffffffffu, page < num_pages && __ldcg(refs + page) == 0);
      count += __popc(free_[i]);
    }
    int total;
    int at = got + block_sum(lane == 31 ? count : 0, s_warps, &total);   // lane 31 has the warp's last place
    at = __shfl_sync(0xffffffffu, at, 31) - count;
#pragma unroll
    for (int i = 0; i < kPagesPerLane; ++i) {
      const int place = at + __popc(free_[i] & ((1u << lane) - 1u));
      if (((free_[i] >> lane) & 1u) && place < want) list[place] = int32_t(first + 32 * i);
      at += __popc(free_[i]);
    }
    got = min(got + total, want);
  }
  return got;
}

// Pages that row r holds and needs; false where it is left alone or bad.
__device__ __forceinline__ bool resized_row(const PagesParams& p, int r, int* have, int* need) {
  const int64_t room = int64_t(p.width) << p.page_shift;
  const int now = p.lens[r], then = __ldg(p.new_lens + r);
  if (then < 0) return false;
  if (now < 0 || now > room || then > room) {
    set_status(p.status, TSEL_DEV_REQUESTS);
    return false;
  }
  *have = ceil_pages(now, p.page_shift);
  *need = ceil_pages(then, p.page_shift);
  return true;
}

// Whether row r would grow from inside a page that other rows hold too: what is then
// written behind its length would be theirs as well.
__device__ __forceinline__ bool shared_end(const PagesParams& p, int r) {
  const int now = p.lens[r];
  if (__ldg(p.new_lens + r) <= now || (now & ((1 << p.page_shift) - 1)) == 0) return false;
  const int page = p.table[r * p.table_stride + (now >> p.page_shift)];
  return page >= 0 && page < p.num_pages && __ldcg(p.refs + page) > 1;
}

__global__ void __launch_bounds__(kPagesThreads) cache_resize_kernel(const PagesParams p) {
  __shared__ int s_warps[kPagesWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  int want = 0;   // pages for the rows so far
  for (int base = 0; base < p.rows; base += kPagesThreads) {
    const int r = base + int(threadIdx.x);
    int have = 0, need = 0;
    bool goes = r < p.rows && resized_row(p, r, &have, &need);
    if (goes && shared_end(p, r)) {
      set_status(p.status, TSEL_DEV_REQUESTS);
      goes = false;
    }
    const int more = goes ? max(need - have, 0) : 0;
    int total;
    const int up_to = want + block_sum(more, s_warps, &total);
    if (r < p.rows) p.plan[r] = goes ? up_to - more : -1;   // -1: stays as it is
    want += total;
  }
  const int found = free_pages(p.refs, p.num_pages, want, p.found, s_warps);
  __syncthreads();   // plan, found
  // a thread for each row; rows that grow by many pages are written by the whole warp
  for (int base = 0; base < p.rows; base += kPagesThreads) {
    const int r = base + int(threadIdx.x);
    int have = 0, need = 0, first = 0;
    bool goes = r < p.rows && resized_row(p, r, &have, &need) && need >= have;
    if (goes) first = p.plan[r];
    goes = goes && first >= 0;
    if (goes && need > have && first + (need - have) > found) {   // not enough: the row stays as it is
      set_status(p.status, TSEL_DEV_PAGES);
      goes = false;
    }
    const bool few = need - have <= 4;
    if (goes && few) {
      for (int i = have; i < need; ++i) {
        const int page = p.found[first + i - have];
        p.table[r * p.table_stride + i] = page;
        p.refs[page] = 1;
      }
    }
    for (unsigned many = __ballot_sync(0xffffffffu, goes && !few); many != 0; many &= many - 1) {
      const int src = __ffs(many) - 1;
      const int row = __shfl_sync(0xffffffffu, r, src), from = __shfl_sync(0xffffffffu, have, src);
      const int to = __shfl_sync(0xffffffffu, need, src), at = __shfl_sync(0xffffffffu, first, src);
      for (int i = from + lane; i < to; i += 32) {
        const int page = p.found[at + i - from];
        p.table[row * p.table_stride + i] = page;
        p.refs[page] = 1;
      }
    }
    if (goes) p.lens[r] = __ldg(p.new_lens + r);
  }
}

// The rows that shrink, a CTA each.
__global__ void __launch_bounds__(kMoveThreads) cache_shrink_kernel(const PagesParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int r = int(blockIdx.x);
  int have = 0, need = 0;
  const bool shrinks = resized_row(p, r, &have, &need) && need < have;
  __syncthreads();   // every thread has read the length
  if (!shrinks) return;
  const int32_t* row = p.table + r * p.table_stride;
  for (int i = need + int(threadIdx.x); i < have; i += kMoveThreads) {
    const int page = row[i];
    if (page < 0 || page >= p.num_pages) {
      set_status(p.status, TSEL_DEV_PAGES);
    } else if (atomicSub(p.refs + page, 1) <= 0) {
      atomicAdd(p.refs + page, 1);
      set_status(p.status, TSEL_DEV_PAGES);
    }
  }
  if (threadIdx.x == 0) p.lens[r] = __ldg(p.new_lens + r);
}

// Fresh pages for the children whose parent's last page is not full. plan[i]: that
// page, -1 none needed, -2 no child.
__global__ void __launch_bounds__(kPagesThreads) fork_plan_kernel(const PagesParams p) {
  __shared__ int s_warps[kPagesWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t room = int64_t(p.width) << p.page_shift;
  const int mask = (1 << p.page_shift) - 1;
  // The largest child so far, in the places of the pages found later: a list that
  // ascends whatever the caller's does. A child is taken only where it rises, so none
  // is taken twice, and a parent is looked for in it.
  int* tops = p.found;
  int top = -1;
  for (int base = 0; base < p.n; base += kPagesThreads) {
    const int i = base + int(threadIdx.x);
    int most;
    const int up_to = block_scan<true>(i < p.n ? __ldg(p.children + i) : -1, s_warps, &most);
    if (i < p.n) tops[i] = max(top, up_to);
    top = max(top, most);
  }
  __syncthreads();
  int want = 0;
  for (int base = 0; base < p.n; base += kPagesThreads) {
    const int i = base + int(threadIdx.x);
    int state = -2;   // no child, no page, a page
    if (i < p.n) {
      const int src = __ldg(p.parents + i), dst = __ldg(p.children + i);
      bool ok = src >= 0 && src < p.rows && dst >= 0 && dst < p.rows && dst > (i > 0 ? tops[i - 1] : -1);
      if (ok) {   // no child is a parent
        int lo = 0, hi = p.n;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (tops[mid] < src) lo = mid + 1;
          else hi = mid;
        }
        ok = lo >= p.n || tops[lo] != src;
      }
      const int len = ok ? __ldcg(p.lens + src) : 0;
      ok = ok && len >= 0 && len <= room && __ldcg(p.lens + dst) == 0;
      if (!ok) {
        set_status(p.status, TSEL_DEV_REQUESTS);
      } else if ((len & mask) == 0) {
        state = -1;
      } else {
        const int last = __ldcg(p.table + src * p.table_stride + (len >> p.page_shift));
        if (last < 0 || last >= p.num_pages) set_status(p.status, TSEL_DEV_PAGES);
        else state = 0;
      }
    }
    int total;
    const int up_to = want + block_sum(state == 0 ? 1 : 0, s_warps, &total);
    if (i < p.n) p.plan[i] = state == 0 ? up_to - 1 : state;
    want += total;
  }
  const int found = free_pages(p.refs, p.num_pages, want, p.found, s_warps);
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kPagesThreads) {
    int at = p.plan[i];
    if (at >= found) {
      set_status(p.status, TSEL_DEV_PAGES);
      at = -2;
    } else if (at >= 0) {
      at = p.found[at];
      p.refs[at] = 1;
    }
    p.plan[i] = at;
  }
  // lengths last: a child's own is read above as the sign that it holds nothing
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kPagesThreads)
    if (p.plan[i] != -2) p.lens[__ldg(p.children + i)] = __ldcg(p.lens + __ldg(p.parents + i));
}

// A child's list of pages, their counts, and the rows of its last page.
__global__ void __launch_bounds__(kMoveThreads) fork_copy_kernel(const PagesParams p) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = int(blockIdx.x / unsigned(p.parts)), part = int(blockIdx.x - unsigned(i) * unsigned(p.parts));
  const int fresh = __ldcg(p.plan + i);
  if (fresh == -2) return;
  const int32_t* from = p.table + __ldg(p.parents + i) * p.table_stride;
  const int dst = __ldg(p.children + i);
  int32_t* to = p.table + dst * p.table_stride;
  const int len = __ldcg(p.lens + dst), whole = len >> p.page_shift, rest = len & ((1 << p.page_shift) - 1);
  for (int x = part * kMoveThreads + int(threadIdx.x); x < whole; x += p.parts * kMoveThreads) {
    const int page = __ldcg(from + x);
    to[x] = page;
    if (page < 0 || page >= p.num_pages) set_status(p.status, TSEL_DEV_PAGES);
    else atomicAdd(p.refs + page, 1);
  }
  if (fresh < 0 || rest == 0) return;
  if (part == 0 && threadIdx.x == 0) to[whole] = fresh;
  const int old = __ldcg(from + whole);
  if (old < 0 || old >= p.num_pages) return;
  const int bytes = rest * p.d;
  for (int h = part; h < 2 * p.Hkv; h += p.parts) {   // the rows in use of a head are one piece
    const bool v = h >= p.Hkv;
    const int hh = v ? h - p.Hkv : h;
    uint8_t* pages = v ? p.v_pages : p.k_pages;
    uint8_t* exps = v ? p.v_exps : p.k_exps;
    const int64_t a = (int64_t(old) * p.Hkv + hh) << p.page_shift, b = (int64_t(fresh) * p.Hkv + hh) << p.page_shift;
    const uint4* src = reinterpret_cast<const uint4*>(pages + a * p.d);
    uint4* out = reinterpret_cast<uint4*>(pages + b * p.d);
#pragma unroll 4
    for (int x = threadIdx.x; x < bytes / 16; x += kMoveThreads) out[x] = __ldcg(src + x);
    if (int(threadIdx.x) < rest) exps[b + threadIdx.x] = __ldcg(exps + a + threadIdx.x);
  }
}

}  // namespace

void move_plan(MoveParams& p, int want) {
  const int all = 2 * p.Hkv, row = p.d / 16;
  p.heads = all < kMoveHeads ? all : kMoveHeads;
  p.pieces = row;
  // CTAs of a request: first by heads, then by pieces of 32 bytes or more (a sector)
  auto parts = [&]() { return int64_t(p.R) * ceil_div(all, p.heads) * ceil_div(row, p.pieces); };
  auto size = [&]() {
    const int groups = kMoveThreads / p.pieces;
    p.tokens = groups * (p.dst_table == nullptr ? kMoveItemsInPlace : kMoveItems) / p.heads;
    if (p.tokens > kMoveMaxTokens) p.tokens = kMoveMaxTokens;
    p.chunks = p.dst_table == nullptr ? 1 : int(ceil_div(p.max_keep, p.tokens));
  };
  size();
  if (p.dst_table == nullptr) {
    while (p.heads > 1 && parts() < want) p.heads = (p.heads + 1) / 2;
    while (p.pieces > 2 && parts() < want && p.max_keep > 64) p.pieces = (p.pieces + 1) / 2;
    size();
  }
  p.head_parts = int(ceil_div(all, p.heads));
  p.slices = int(ceil_div(row, p.pieces));
}

cudaError_t launch_move(const MoveParams& p, cudaStream_t stream) {
  const int64_t grid = int64_t(p.R) * p.chunks * p.head_parts * p.slices;
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  const bool in_place = p.dst_table == nullptr;
  const size_t smem = size_t(p.tokens) * 16 * (in_place ? 3 : 1);   // 48 KB at most
  return in_place ? launch_kernel(cache_move_kernel<true>, dim3(unsigned(grid)), kMoveThreads, smem, stream, 1, p)
                  : launch_kernel(cache_move_kernel<false>, dim3(unsigned(grid)), kMoveThreads, smem, stream, 1, p);
}

cudaError_t launch_resize(const PagesParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_kernel(cache_resize_kernel, dim3(1), kPagesThreads, 0, stream, 1, p);
  if (e != cudaSuccess) return e;
  return launch_kernel(cache_shrink_kernel, dim3(unsigned(p.rows)), kMoveThreads, 0, stream, 1, p);
}

cudaError_t launch_fork(const PagesParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_kernel(fork_plan_kernel, dim3(1), kPagesThreads, 0, stream, 1, p);
  if (e != cudaSuccess) return e;
  return launch_kernel(fork_copy_kernel, dim3(unsigned(p.n) * unsigned(p.parts)), kMoveThreads, 0, stream, 1, p);
}

}  // namespace tsel
