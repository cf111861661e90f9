// Host side of the cache entry points of include/tsel.h (rotary positions,
// the quantised paged cache, attention over a shared prefix) and of attention
// over whole prompts: argument checks, the rope table, workspace carving and
// kernel launches. Nothing here allocates or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>

#include "attend.cuh"
#include "common.cuh"
#include "pages.cuh"
#include "prompt.cuh"
#include "rope.cuh"

namespace tsel {
void record_error(const char* msg);
int device_sms(int* out);
uint64_t device_wait_timeout_ns();
bool make_rows_map(CUtensorMap* map, const void* base, bool fp16, int head_dim, int heads, int64_t rows,
                   int64_t row_stride_bytes, int box_heads, int box_rows);
}  // namespace tsel

using namespace tsel;

namespace {

tsel_status fail(tsel_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
tsel_status fail(tsel_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  record_error(buf);
  return s;
}

tsel_status cuda_fail(cudaError_t e, const char* where) {
  return fail(TSEL_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int elem_bytes(int dtype) {
  return dtype == TSEL_FP32 ? 4 : (dtype == TSEL_BF16 || dtype == TSEL_FP16 ? 2 : 0);
}

tsel_status check_header(const void* workspace, size_t bytes) {
  if (workspace == nullptr) return fail(TSEL_ERR_INVALID_VALUE, "null workspace");
  if (!aligned(workspace, 256) || bytes < size_t(kWsHeaderBytes))
    return fail(TSEL_ERR_WORKSPACE, "workspace must be >= %d bytes, 256-byte aligned",
                kWsHeaderBytes);
  return TSEL_OK;
}

// Rows [total][heads][head_dim]: fills in the dense stride, checks the rest.
tsel_status check_rows(const char* name, const void* ptr, int64_t* stride, int64_t width, int elem) {
  if (ptr == nullptr) return fail(TSEL_ERR_INVALID_VALUE, "null %s", name);
  if (*stride == 0) *stride = width;
  if (*stride < width || (*stride * elem) % 16 != 0)
    return fail(TSEL_ERR_INVALID_VALUE, "%s row stride %lld", name, (long long)*stride);
  if (!aligned(ptr, 16)) return fail(TSEL_ERR_INVALID_VALUE, "%s must be 16-byte aligned", name);
  return TSEL_OK;
}

tsel_status check_positions(const int32_t* pos, int pos_dim, const uint64_t* table, int num_pairs,
                            int head_dim) {
  if (num_pairs < 0 || 2 * int64_t(num_pairs) > head_dim)
    return fail(TSEL_ERR_INVALID_VALUE, "num_pairs=%d of head_dim=%d", num_pairs, head_dim);
  if (pos_dim < 0 || pos_dim > 8) return fail(TSEL_ERR_INVALID_VALUE, "pos_dim=%d", pos_dim);
  if (num_pairs > 0 && (pos == nullptr || table == nullptr || pos_dim < 1))
    return fail(TSEL_ERR_INVALID_VALUE, "rotation needs positions and a table");
  if (!aligned(pos, 4) || !aligned(table, 8))
    return fail(TSEL_ERR_INVALID_VALUE, "positions or table misaligned");
  return TSEL_OK;
}

// log2 of a supported page size, -1 otherwise.
int page_shift_of(int page_size) {
  for (int s = 4; s <= 7; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

bool cache_head_dim(int d) { return d == 64 || d == 80 || d == 96 || d == 112 || d == 128; }

tsel_status check_cache(const void* kp, const void* vp, const void* ke, const void* ve,
                        int num_pages, int page_size, int num_kv_heads, int head_dim) {
  if (!cache_head_dim(head_dim))
    return fail(TSEL_ERR_UNSUPPORTED, "head_dim=%d (supported: 64, 80, 96, 112, 128)", head_dim);
  if (page_shift_of(page_size) < 0)
    return fail(TSEL_ERR_UNSUPPORTED, "page_size=%d (supported: 16, 32, 64, 128)", page_size);
  if (num_kv_heads < 1 || num_kv_heads > 256)
    return fail(TSEL_ERR_INVALID_VALUE, "num_kv_heads=%d", num_kv_heads);
  if (num_pages < 0 || int64_t(num_pages) * page_size > 0x7FFFFFFFll)
    return fail(TSEL_ERR_INVALID_VALUE, "num_pages=%d of %d", num_pages, page_size);
  if (num_pages > 0 && (kp == nullptr || vp == nullptr || ke == nullptr || ve == nullptr))
    return fail(TSEL_ERR_INVALID_VALUE, "null cache pointer");
  if (!aligned(kp, 16) || !aligned(vp, 16) || !aligned(ke, 16) || !aligned(ve, 16))
    return fail(TSEL_ERR_INVALID_VALUE, "cache pointers must be 16-byte aligned");
  return TSEL_OK;
}

// Tables of int32 and vectors (one row): rows of `width` entries, `stride` apart.
struct Ints {
  const char* name;
  const void* ptr;
  int64_t rows, stride, width;
  Ints(const char* what, const void* p, int64_t n) : name(what), ptr(p), rows(1), stride(n), width(n) {}
  Ints(const char* what, const void* p, int64_t r, int64_t s, int64_t w) : name(what), ptr(p), rows(r), stride(s), width(w) {}
  bool none() const { return ptr == nullptr || rows <= 0 || width <= 0; }
  uintptr_t at(int64_t row) const { return reinterpret_cast<uintptr_t>(ptr) + uintptr_t(row) * uintptr_t(stride) * 4; }
};

// Whether row r of a, [begin, end), meets a row of b. Rows of b ascend without overlap,
// so only the last one that begins before `end` can.
bool meets(uintptr_t begin, uintptr_t end, const Ints& b) {
  if (b.at(0) >= end) return false;
  int64_t r = b.rows - 1;
  if (b.rows > 1) {
    const int64_t last = int64_t((end - 1 - b.at(0)) / (uintptr_t(b.stride) * 4));
    if (last < r) r = last;
  }
  return b.at(r) + uintptr_t(b.width) * 4 > begin;
}

// What a call writes shares no memory with what it reads or writes besides.
tsel_status check_apart(const Ints& a, const Ints& b) {
  if (a.none() || b.none()) return TSEL_OK;
  const Ints& few = a.rows <= b.rows ? a : b;
  const Ints& many = a.rows <= b.rows ? b : a;
  for (int64_t r = 0; r < few.rows; ++r)
    if (meets(few.at(r), few.at(r) + uintptr_t(few.width) * 4, many))
      return fail(TSEL_ERR_INVALID_VALUE, "%s and %s overlap", a.name, b.name);
  return TSEL_OK;
}

#define TSEL_TRY(expr)                       \
  do {                                       \
    const tsel_status st_ = (expr);          \
    if (st_ != TSEL_OK) return st_;          \
  } while (0)

}  // namespace

extern "C" {

tsel_status tsel_rope_frequencies(double base, const int32_t* sections, int num_axes, int layout,
                                  double* inv_freq, int32_t* axis) {
  if (sections == nullptr || inv_freq == nullptr || axis == nullptr || num_axes < 1 || num_axes > 8)
    return fail(TSEL_ERR_INVALID_VALUE, "null pointer or num_axes=%d", num_axes);
  if (!(base > 0.0) || !std::isfinite(base)) return fail(TSEL_ERR_INVALID_VALUE, "base");
  int64_t total = 0;
  for (int a = 0; a < num_axes; ++a) {
    if (sections[a] < 0) return fail(TSEL_ERR_INVALID_VALUE, "sections[%d]=%d", a, sections[a]);
    total += sections[a];
  }
  if (total > 128) return fail(TSEL_ERR_INVALID_VALUE, "%lld pairs (at most 128)", (long long)total);
  const int pairs = int(total);
  if (layout == TSEL_ROPE_SECTIONED || layout == TSEL_ROPE_PER_AXIS) {
    int i = 0;
    for (int a = 0; a < num_axes; ++a)
      for (int j = 0; j < sections[a]; ++j, ++i) {
        axis[i] = a;
        inv_freq[i] = layout == TSEL_ROPE_SECTIONED ? std::pow(base, -double(i) / pairs)
                                                    : std::pow(base, -double(j) / sections[a]);
      }
    return TSEL_OK;
  }
  if (layout != TSEL_ROPE_INTERLEAVED) return fail(TSEL_ERR_INVALID_VALUE, "layout=%d", layout);
  int first = 0;
  for (int i = 0; i < pairs; ++i) {
    const int a = i % num_axes;
    axis[i] = i / num_axes < sections[a] ? a : 0;
    first += axis[i] == 0;
    inv_freq[i] = std::pow(base, -double(i) / pairs);
  }
  if (first != sections[0])
    return fail(TSEL_ERR_INVALID_VALUE, "sections cannot be interleaved: axis 0 would get %d of %d pairs",
                first, sections[0]);
  return TSEL_OK;
}

tsel_status tsel_rope_table(const double* inv_freq, const int32_t* axis, int num_pairs,
                            uint64_t* table) {
  if (num_pairs < 0 || num_pairs > 128 ||
      (num_pairs > 0 && (inv_freq == nullptr || axis == nullptr || table == nullptr)))
    return fail(TSEL_ERR_INVALID_VALUE, "null pointer or num_pairs=%d", num_pairs);
  // 1 / (2 pi) to twice the precision of a double
  const double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
  for (int i = 0; i < num_pairs; ++i) {
    if (axis[i] < 0 || axis[i] > 7) return fail(TSEL_ERR_INVALID_VALUE, "axis[%d]=%d", i, axis[i]);
    const double f = inv_freq[i];
    if (!(std::fabs(f) <= 1e6)) return fail(TSEL_ERR_INVALID_VALUE, "inv_freq[%d]", i);
    const double turns = f * kHi;
    const double rest = std::fma(f, kHi, -turns) + f * kLo;
    const double frac = std::fmod(turns, 1.0);   // exact, with the sign of turns
    // 2^61 steps to a turn; the sum wraps like the turns it counts
    const uint64_t steps = uint64_t(std::llrint(std::ldexp(frac, 61))) +
                           uint64_t(std::llrint(std::ldexp(rest, 61)));
    table[i] = (steps << 3) | uint64_t(axis[i]);
  }
  return TSEL_OK;
}

size_t tsel_cache_workspace_size(void) { return kWsHeaderBytes; }

tsel_status tsel_rope(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                      const int32_t* pos, int pos_dim, const uint64_t* table, int num_pairs,
                      int total, int num_heads, int num_kv_heads, int head_dim, int dtype,
                      unsigned flags, void* q_out, int64_t q_out_row_stride, void* k_out,
                      int64_t k_out_row_stride, void* workspace, size_t workspace_bytes,
                      void* stream_) {
  const int elem = elem_bytes(dtype);
  if (elem == 0) return fail(TSEL_ERR_UNSUPPORTED, "dtype=%d", dtype);
  if (total < 0 || num_heads < 1 || num_heads > 256 || num_kv_heads < 0 || num_kv_heads > 256)
    return fail(TSEL_ERR_INVALID_VALUE, "total=%d num_heads=%d num_kv_heads=%d", total, num_heads,
                num_kv_heads);
  if (head_dim < 8 || head_dim > 256 || head_dim % 8 != 0)
    return fail(TSEL_ERR_UNSUPPORTED, "head_dim=%d (supported: multiples of 8 to 256)", head_dim);
  if (flags & ~(TSEL_ROPE_ADJACENT | TSEL_ROPE_INVERSE))
    return fail(TSEL_ERR_UNSUPPORTED, "flags=0x%x", flags);
  TSEL_TRY(check_header(workspace, workspace_bytes));
  if (total == 0) return TSEL_OK;
  TSEL_TRY(check_positions(pos, pos_dim, table, num_pairs, head_dim));
  RopeParams p{};
  p.q_stride = q_row_stride;
  p.k_stride = k_row_stride;
  p.q_out_stride = q_out_row_stride;
  p.k_out_stride = k_out_row_stride;
  const int64_t wq = int64_t(num_heads) * head_dim, wk = int64_t(num_kv_heads) * head_dim;
  TSEL_TRY(check_rows("q", q, &p.q_stride, wq, elem));
  TSEL_TRY(check_rows("q_out", q_out, &p.q_out_stride, wq, elem));
  if (num_kv_heads > 0) {
    TSEL_TRY(check_rows("k", k, &p.k_stride, wk, elem));
    TSEL_TRY(check_rows("k_out", k_out, &p.k_out_stride, wk, elem));
  }
  int sms = 0;
  if (device_sms(&sms) != 0) return fail(TSEL_ERR_CUDA, "cannot query the SM count");
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.pos = pos;
  p.pos_dim = pos_dim;
  p.table = table;
  p.num_pairs = num_pairs;
  p.total = total;
  p.H = num_heads;
  p.Hkv = num_kv_heads;
  p.d = head_dim;
  p.adjacent = (flags & TSEL_ROPE_ADJACENT) ? 1 : 0;
  p.inverse = (flags & TSEL_ROPE_INVERSE) ? 1 : 0;
  p.status = &static_cast<WsHeader*>(workspace)->status;
  const cudaError_t e = launch_rope(dtype, p, sms, static_cast<cudaStream_t>(stream_));
  return e == cudaSuccess ? TSEL_OK : cuda_fail(e, "rope launch");
}

tsel_status tsel_cache_write(const void* k, int64_t k_row_stride, const void* v,
                             int64_t v_row_stride, const int32_t* pos, int pos_dim,
                             const uint64_t* table, int num_pairs, const int32_t* slots, int total,
                             int num_kv_heads, int head_dim, int dtype, unsigned flags,
                             uint8_t* k_pages, uint8_t* v_pages, uint8_t* k_exps, uint8_t* v_exps,
                             int num_pages, int page_size, void* workspace,
                             size_t workspace_bytes, void* stream_) {
  const int elem = elem_bytes(dtype);
  if (elem == 0) return fail(TSEL_ERR_UNSUPPORTED, "dtype=%d", dtype);
  if (total < 0) return fail(TSEL_ERR_INVALID_VALUE, "total=%d", total);
  if (flags & ~TSEL_ROPE_ADJACENT) return fail(TSEL_ERR_UNSUPPORTED, "flags=0x%x", flags);
  TSEL_TRY(check_cache(k_pages, v_pages, k_exps, v_exps, num_pages, page_size, num_kv_heads, head_dim));
  TSEL_TRY(check_header(workspace, workspace_bytes));
  if (total == 0) return TSEL_OK;
  TSEL_TRY(check_positions(pos, pos_dim, table, num_pairs, head_dim));
  if (slots == nullptr || !aligned(slots, 4)) return fail(TSEL_ERR_INVALID_VALUE, "slots");
  CacheParams p{};
  p.k_stride = k_row_stride;
  p.v_stride = v_row_stride;
  const int64_t width = int64_t(num_kv_heads) * head_dim;
  TSEL_TRY(check_rows("k", k, &p.k_stride, width, elem));
  TSEL_TRY(check_rows("v", v, &p.v_stride, width, elem));
  int sms = 0;
  if (device_sms(&sms) != 0) return fail(TSEL_ERR_CUDA, "cannot query the SM count");
  p.k = k;
  p.v = v;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.k_exps = k_exps;
  p.v_exps = v_exps;
  p.num_pages = num_pages;
  p.page_shift = page_shift_of(page_size);
  p.slots = slots;
  p.pos = pos;
  p.pos_dim = pos_dim;
  p.table = table;
  p.num_pairs = num_pairs;
  p.total = total;
  p.Hkv = num_kv_heads;
  p.d = head_dim;
  p.adjacent = (flags & TSEL_ROPE_ADJACENT) ? 1 : 0;
  p.status = &static_cast<WsHeader*>(workspace)->status;
  const cudaError_t e = launch_cache_write(dtype, p, sms, static_cast<cudaStream_t>(stream_));
  return e == cudaSuccess ? TSEL_OK : cuda_fail(e, "cache write launch");
}

tsel_status tsel_cache_read(const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_exps,
                            const uint8_t* v_exps, int num_pages, int page_size,
                            const int32_t* slots, int total, int num_kv_heads, int head_dim,
                            int dtype, void* k_out, int64_t k_row_stride, void* v_out,
                            int64_t v_row_stride, void* workspace, size_t workspace_bytes,
                            void* stream_) {
  const int elem = elem_bytes(dtype);
  if (elem == 0) return fail(TSEL_ERR_UNSUPPORTED, "dtype=%d", dtype);
  if (total < 0) return fail(TSEL_ERR_INVALID_VALUE, "total=%d", total);
  TSEL_TRY(check_cache(k_pages, v_pages, k_exps, v_exps, num_pages, page_size, num_kv_heads, head_dim));
  TSEL_TRY(check_header(workspace, workspace_bytes));
  if (total == 0) return TSEL_OK;
  if (slots == nullptr || !aligned(slots, 4)) return fail(TSEL_ERR_INVALID_VALUE, "slots");
  CacheParams p{};
  p.k_stride = k_row_stride;
  p.v_stride = v_row_stride;
  const int64_t width = int64_t(num_kv_heads) * head_dim;
  TSEL_TRY(check_rows("k_out", k_out, &p.k_stride, width, elem));
  TSEL_TRY(check_rows("v_out", v_out, &p.v_stride, width, elem));
  int sms = 0;
  if (device_sms(&sms) != 0) return fail(TSEL_ERR_CUDA, "cannot query the SM count");
  p.k_out = k_out;
  p.v_out = v_out;
  p.k_pages = const_cast<uint8_t*>(k_pages);
  p.v_pages = const_cast<uint8_t*>(v_pages);
  p.k_exps = const_cast<uint8_t*>(k_exps);
  p.v_exps = const_cast<uint8_t*>(v_exps);
  p.num_pages = num_pages;
  p.page_shift = page_shift_of(page_size);
  p.slots = slots;
  p.total = total;
  p.Hkv = num_kv_heads;
  p.d = head_dim;
  p.status = &static_cast<WsHeader*>(workspace)->status;
  const cudaError_t e = launch_cache_read(dtype, p, sms, static_cast<cudaStream_t>(stream_));
  return e == cudaSuccess ? TSEL_OK : cuda_fail(e, "cache read launch");
}

static size_t attend_workspace(bool tree, int num_req, int total_q, int max_seqlen_q, int num_heads, int num_kv_heads,
                               int head_dim, int max_prefix_len, int max_suffix_len) {
  if (num_req < 0 || total_q < 0 || max_seqlen_q < 0 || num_kv_heads < 1 ||
      num_heads < num_kv_heads || num_heads > 256 || num_heads % num_kv_heads != 0 ||
      num_heads / num_kv_heads > kTile || !cache_head_dim(head_dim) || max_prefix_len < 0 ||
      max_suffix_len < 0 || max_prefix_len > kAttMaxKeys || max_suffix_len > kAttMaxKeys ||
      (tree && max_seqlen_q > kAttTreeNodes))
    return 0;
  const AttPlan a = att_plan(num_req, total_q, max_seqlen_q, num_heads, num_kv_heads, head_dim,
                             max_prefix_len, max_suffix_len, tree);
  return a.too_large ? 0 : size_t(a.total);
}

size_t tsel_prefix_attention_workspace_size(int num_req, int total_q, int max_seqlen_q,
                                            int num_heads, int num_kv_heads, int head_dim,
                                            int max_prefix_len, int max_suffix_len) {
  return attend_workspace(false, num_req, total_q, max_seqlen_q, num_heads, num_kv_heads, head_dim,
                          max_prefix_len, max_suffix_len);
}

// Both attentions over the cache; `parents` (and `tree`) are the tree's.
static tsel_status attend_cache(
    const void* q, int64_t q_row_stride, const int32_t* cu_seqlens_q, int num_req, int total_q,
    int max_seqlen_q, bool tree, const int32_t* parents, const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_exps,
    const uint8_t* v_exps, int num_pages, int page_size, const int32_t* prefix_pages,
    const int32_t* prefix_len, int max_prefix_len, const int32_t* page_table,
    int64_t page_table_stride, const int32_t* suffix_lens, int max_suffix_len, int num_heads,
    int num_kv_heads, int head_dim, int dtype, float softmax_scale, void* out,
    int64_t out_row_stride, float* lse, void* workspace, size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (dtype != TSEL_BF16 && dtype != TSEL_FP16)
    return fail(TSEL_ERR_UNSUPPORTED, "dtype=%d (bf16 or fp16)", dtype);
  if (num_req < 0 || total_q < 0 || max_seqlen_q < 0 || max_prefix_len < 0 || max_suffix_len < 0)
    return fail(TSEL_ERR_INVALID_VALUE, "negative size");
  if (num_heads < 1 || num_heads > 256 || num_kv_heads < 1 || num_heads % num_kv_heads != 0)
    return fail(TSEL_ERR_INVALID_VALUE, "num_heads=%d num_kv_heads=%d", num_heads, num_kv_heads);
  if (num_heads / num_kv_heads > kTile)
    return fail(TSEL_ERR_UNSUPPORTED, "%d query heads per KV head (at most %d)",
                num_heads / num_kv_heads, kTile);
  TSEL_TRY(check_cache(k_pages, v_pages, k_exps, v_exps, num_pages, page_size, num_kv_heads, head_dim));
  if (max_prefix_len > kAttMaxKeys || max_suffix_len > kAttMaxKeys)
    return fail(TSEL_ERR_UNSUPPORTED, "prefix of %d or suffix of %d keys (at most %d)", max_prefix_len,
                max_suffix_len, kAttMaxKeys);
  if (!(softmax_scale == softmax_scale) || std::isinf(softmax_scale))
    return fail(TSEL_ERR_INVALID_VALUE, "softmax_scale");
  if (cu_seqlens_q == nullptr) return fail(TSEL_ERR_INVALID_VALUE, "null cu_seqlens_q");
  if (tree && max_seqlen_q > kAttTreeNodes)
    return fail(TSEL_ERR_UNSUPPORTED, "trees of up to %d nodes (at most %d)", max_seqlen_q, kAttTreeNodes);
  if (tree && total_q > 0 && (parents == nullptr || !aligned(parents, 4)))
    return fail(TSEL_ERR_INVALID_VALUE, "parents");
  if (tree && total_q > 0 && max_suffix_len < 1)
    return fail(TSEL_ERR_INVALID_VALUE, "max_suffix_len=%d: the nodes' keys are the suffix's last", max_suffix_len);
  if (max_prefix_len > 0 && (prefix_pages == nullptr || prefix_len == nullptr))
    return fail(TSEL_ERR_INVALID_VALUE, "null prefix_pages or prefix_len");
  if (max_suffix_len > 0 && num_req > 0 && (page_table == nullptr || suffix_lens == nullptr))
    return fail(TSEL_ERR_INVALID_VALUE, "null page_table or suffix_lens");
  if (max_suffix_len > 0 && num_req > 0 && page_table_stride < ceil_div(max_suffix_len, page_size))
    return fail(TSEL_ERR_INVALID_VALUE, "page_table_stride %lld for %d keys",
                (long long)page_table_stride, max_suffix_len);
  TSEL_TRY(check_header(workspace, workspace_bytes));
  const AttPlan a = att_plan(num_req, total_q, max_seqlen_q, num_heads, num_kv_heads, head_dim,
                             max_prefix_len, max_suffix_len, tree);
  if (a.too_large) return fail(TSEL_ERR_UNSUPPORTED, "too many units of work");
  if (workspace_bytes < size_t(a.total))
    return fail(TSEL_ERR_WORKSPACE, "workspace %zu < %lld bytes", workspace_bytes, (long long)a.total);
  if (total_q == 0) return TSEL_OK;
  AttParams p{};
  p.q_stride = q_row_stride;
  p.out_stride = out_row_stride;
  const int64_t width = int64_t(num_heads) * head_dim;
  TSEL_TRY(check_rows("q", q, &p.q_stride, width, 2));
  TSEL_TRY(check_rows("out", out, &p.out_stride, width, 2));
  p.q = q;
  p.fp16 = dtype == TSEL_FP16 ? 1 : 0;
  p.cu_q = cu_seqlens_q;
  p.R = num_req;
  p.Tq = total_q;
  p.max_q = max_seqlen_q;
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.k_exps = k_exps;
  p.v_exps = v_exps;
  p.num_pages = num_pages;
  p.page_shift = page_shift_of(page_size);
  p.prefix_pages = prefix_pages;
  p.prefix_len = prefix_len;
  p.max_prefix = max_prefix_len;
  p.page_table = page_table;
  p.table_stride = page_table_stride;
  p.suffix_lens = suffix_lens;
  p.max_suffix = max_suffix_len;
  p.parents = parents;
  p.H = num_heads;
  p.Hkv = num_kv_heads;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(float(head_dim));
  p.c = scale * 1.4426950408889634f;
  p.G = a.G;
  p.tt = a.tt;
  p.slots = a.slots;
  p.pre = a.pre;
  p.suf = a.suf;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_lse = reinterpret_cast<float*>(ws + a.lse_off);
  p.part_o = reinterpret_cast<float*>(ws + a.o_off);
  p.out = out;
  p.lse = lse;
  p.status = &reinterpret_cast<WsHeader*>(ws)->status;
  p.timeout_ns = device_wait_timeout_ns();
  // The wide launch first, then the few-row ones. Neither reads what the other
  // writes, but a kernel sees earlier kernels' writes (Q, cached rows, lengths)
  // only after its own wait, which is also for the launch before it.
  cudaError_t e;
  for (int kind = 0; kind <= 2; ++kind) {
    const int64_t pre = a.pre.narrow == kind ? a.pre.units : 0, suf = a.suf.narrow == kind ? a.suf.units : 0;
    if (pre + suf == 0) continue;
    p.pre_units = uint32_t(pre);
    e = kind == 0 ? launch_attend(head_dim, p, pre + suf, stream)
                  : launch_attend_narrow(head_dim, kind, p, pre + suf, stream);
    if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  }
  e = launch_attend_join(head_dim, p, stream);
  return e == cudaSuccess ? TSEL_OK : cuda_fail(e, "join launch");
}

tsel_status tsel_prefix_attention(
    const void* q, int64_t q_row_stride, const int32_t* cu_seqlens_q, int num_req, int total_q,
    int max_seqlen_q, const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_exps,
    const uint8_t* v_exps, int num_pages, int page_size, const int32_t* prefix_pages,
    const int32_t* prefix_len, int max_prefix_len, const int32_t* page_table,
    int64_t page_table_stride, const int32_t* suffix_lens, int max_suffix_len, int num_heads,
    int num_kv_heads, int head_dim, int dtype, float softmax_scale, void* out,
    int64_t out_row_stride, float* lse, void* workspace, size_t workspace_bytes, void* stream_) {
  return attend_cache(q, q_row_stride, cu_seqlens_q, num_req, total_q, max_seqlen_q, false, nullptr, k_pages, v_pages, k_exps,
                      v_exps, num_pages, page_size, prefix_pages, prefix_len, max_prefix_len, page_table,
                      page_table_stride, suffix_lens, max_suffix_len, num_heads, num_kv_heads, head_dim, dtype,
                      softmax_scale, out, out_row_stride, lse, workspace, workspace_bytes, stream_);
}

size_t tsel_tree_attention_workspace_size(int num_req, int total_q, int max_nodes, int num_heads, int num_kv_heads,
                                          int head_dim, int max_prefix_len, int max_suffix_len) {
  return attend_workspace(true, num_req, total_q, max_nodes, num_heads, num_kv_heads, head_dim, max_prefix_len,
                          max_suffix_len);
}

tsel_status tsel_tree_attention(
    const void* q, int64_t q_row_stride, const int32_t* cu_seqlens_q, int num_req, int total_q,
    int max_nodes, const int32_t* parents, const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_exps,
    const uint8_t* v_exps, int num_pages, int page_size, const int32_t* prefix_pages,
    const int32_t* prefix_len, int max_prefix_len, const int32_t* page_table,
    int64_t page_table_stride, const int32_t* suffix_lens, int max_suffix_len, int num_heads,
    int num_kv_heads, int head_dim, int dtype, float softmax_scale, void* out,
    int64_t out_row_stride, float* lse, void* workspace, size_t workspace_bytes, void* stream_) {
  return attend_cache(q, q_row_stride, cu_seqlens_q, num_req, total_q, max_nodes, true, parents, k_pages, v_pages, k_exps,
                      v_exps, num_pages, page_size, prefix_pages, prefix_len, max_prefix_len, page_table,
                      page_table_stride, suffix_lens, max_suffix_len, num_heads, num_kv_heads, head_dim, dtype,
                      softmax_scale, out, out_row_stride, lse, workspace, workspace_bytes, stream_);
}

size_t tsel_prompt_attention_workspace_size(int num_seg, int total_q, int max_seqlen_q, int max_seqlen_k,
                                            int num_heads, int num_kv_heads, int head_dim) {
  if (num_seg < 0 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || num_kv_heads < 1 ||
      num_heads < num_kv_heads || num_heads > 256 || num_heads % num_kv_heads != 0 ||
      num_heads / num_kv_heads > kTile || !cache_head_dim(head_dim) || total_q > kAttMaxKeys ||
      max_seqlen_k > kAttMaxKeys)
    return 0;
  const PromptPlan a = prompt_plan(num_seg, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_dim);
  return a.too_large ? 0 : size_t(a.total);
}

tsel_status tsel_prompt_attention(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride,
                                  const void* v, int64_t v_row_stride, const int32_t* cu_seqlens_q,
                                  const int32_t* cu_seqlens_k, int num_seg, int total_q, int total_k,
                                  int max_seqlen_q, int max_seqlen_k, int num_heads, int num_kv_heads,
                                  int head_dim, int dtype, float softmax_scale, unsigned flags, void* out,
                                  int64_t out_row_stride, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream_) {
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (dtype != TSEL_BF16 && dtype != TSEL_FP16)
    return fail(TSEL_ERR_UNSUPPORTED, "dtype=%d (bf16 or fp16)", dtype);
  if (num_seg < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0)
    return fail(TSEL_ERR_INVALID_VALUE, "negative size");
  if (num_heads < 1 || num_heads > 256 || num_kv_heads < 1 || num_heads % num_kv_heads != 0)
    return fail(TSEL_ERR_INVALID_VALUE, "num_heads=%d num_kv_heads=%d", num_heads, num_kv_heads);
  if (num_heads / num_kv_heads > kTile)
    return fail(TSEL_ERR_UNSUPPORTED, "%d query heads per KV head (at most %d)",
                num_heads / num_kv_heads, kTile);
  if (!cache_head_dim(head_dim))
    return fail(TSEL_ERR_UNSUPPORTED, "head_dim=%d (supported: 64, 80, 96, 112, 128)", head_dim);
  if (total_q > kAttMaxKeys || total_k > kAttMaxKeys || max_seqlen_k > kAttMaxKeys)
    return fail(TSEL_ERR_UNSUPPORTED, "more than %d rows or keys", kAttMaxKeys);
  if (flags & ~TSEL_ATT_CAUSAL) return fail(TSEL_ERR_UNSUPPORTED, "flags=0x%x", flags);
  if (!(softmax_scale == softmax_scale) || std::isinf(softmax_scale))
    return fail(TSEL_ERR_INVALID_VALUE, "softmax_scale");
  if (cu_seqlens_q == nullptr || cu_seqlens_k == nullptr || !aligned(cu_seqlens_q, 4) || !aligned(cu_seqlens_k, 4))
    return fail(TSEL_ERR_INVALID_VALUE, "cu_seqlens_q or cu_seqlens_k");
  if (lse != nullptr && !aligned(lse, 4)) return fail(TSEL_ERR_INVALID_VALUE, "lse misaligned");
  TSEL_TRY(check_header(workspace, workspace_bytes));
  const PromptPlan a = prompt_plan(num_seg, total_q, max_seqlen_q, max_seqlen_k, num_heads, num_kv_heads, head_dim);
  if (a.too_large) return fail(TSEL_ERR_UNSUPPORTED, "too many units of work");
  if (workspace_bytes < size_t(a.total))
    return fail(TSEL_ERR_WORKSPACE, "workspace %zu < %lld bytes", workspace_bytes, (long long)a.total);
  if (total_q == 0) return TSEL_OK;
  PromptParams p{};
  int64_t q_stride = q_row_stride, k_stride = k_row_stride;
  p.v_stride = v_row_stride;
  p.out_stride = out_row_stride;
  const int64_t width = int64_t(num_heads) * head_dim, kv_width = int64_t(num_kv_heads) * head_dim;
  TSEL_TRY(check_rows("q", q, &q_stride, width, 2));
  TSEL_TRY(check_rows("out", out, &p.out_stride, width, 2));
  if (total_k > 0) {
    TSEL_TRY(check_rows("k", k, &k_stride, kv_width, 2));
    TSEL_TRY(check_rows("v", v, &p.v_stride, kv_width, 2));
  }
  const bool fp16 = dtype == TSEL_FP16;
  CUtensorMap mq, mk, mv;
  // without keys nothing is loaded through their maps: those of q will do
  if (!make_rows_map(&mq, q, fp16, head_dim, num_heads, total_q, q_stride * 2, a.G, a.tt) ||
      !make_rows_map(&mk, total_k > 0 ? k : q, fp16, head_dim, total_k > 0 ? num_kv_heads : num_heads,
                     total_k > 0 ? total_k : total_q, (total_k > 0 ? k_stride : q_stride) * 2, 1, kPromptStep) ||
      !make_rows_map(&mv, total_k > 0 ? v : q, fp16, head_dim, total_k > 0 ? num_kv_heads : num_heads,
                     total_k > 0 ? total_k : total_q, (total_k > 0 ? p.v_stride : q_stride) * 2, 1, kPromptStep))
    return fail(TSEL_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  int sms = 0;
  if (device_sms(&sms) != 0) return fail(TSEL_ERR_CUDA, "cannot query the SM count");
  p.v = v;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.seg = num_seg;
  p.Tq = total_q;
  p.Tk = total_k;
  p.max_q = max_seqlen_q;
  p.max_k = max_seqlen_k;
  p.H = num_heads;
  p.Hkv = num_kv_heads;
  p.G = a.G;
  p.tt = a.tt;
  p.causal = (flags & TSEL_ATT_CAUSAL) ? 1 : 0;
  p.chunks = a.chunks;
  p.keys = a.keys;
  p.keys_one = a.keys_one;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / std::sqrt(float(head_dim));
  p.c = std::fmax(scale * 1.4426950408889634f, 1e-38f);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (a.slots > 0) {
    p.part_lse = reinterpret_cast<float*>(ws + a.lse_off);
    p.part_o = reinterpret_cast<float*>(ws + a.o_off);
  }
  p.out = out;
  p.lse = lse;
  p.status = &reinterpret_cast<WsHeader*>(ws)->status;
  // a row tile without rows in a unit waits for the whole of it: 100 ns a key are
  // several times what a unit takes
  p.timeout_ns = device_wait_timeout_ns() + 100ull * uint64_t(max_seqlen_k);
  const int ctas = int(a.units < sms ? a.units : sms);
  if (a.units > kPromptDealt * int64_t(ctas) && a.units < (1ll << 30)) {
    p.next = &reinterpret_cast<WsHeader*>(ws)->sched_ctr[0];
    const cudaError_t z = cudaMemsetAsync(p.next, 0, sizeof(int32_t), stream);
    if (z != cudaSuccess) return cuda_fail(z, "unit counter");
  }
  cudaError_t e = launch_prompt(head_dim, fp16, mq, mk, mv, p, ctas, stream);
  if (e != cudaSuccess) return cuda_fail(e, "prompt attention launch");
  if (a.slots == 0) return TSEL_OK;
  AttParams j{};
  j.cu_q = cu_seqlens_q;
  j.cu_k = cu_seqlens_k;
  j.Tk = total_k;
  j.max_k = max_seqlen_k;
  j.R = num_seg;
  j.Tq = total_q;
  j.max_q = max_seqlen_q;
  j.H = num_heads;
  j.slots = a.slots;
  j.part_lse = p.part_lse;
  j.part_o = p.part_o;
  j.out = out;
  j.out_stride = p.out_stride;
  j.fp16 = fp16 ? 1 : 0;
  j.lse = lse;
  j.status = p.status;
  e = launch_attend_join(head_dim, j, stream);
  return e == cudaSuccess ? TSEL_OK : cuda_fail(e, "join launch");
}

tsel_status tsel_cache_compact(uint8_t* k_pages, uint8_t* v_pages, uint8_t* k_exps, uint8_t* v_exps, int num_pages,
                               int page_size, const int32_t* page_table, int64_t page_table_stride, int pages_per_req,
                               const int32_t* dst_table, int64_t dst_table_stride, int dst_pages_per_req,
                               const int32_t* starts, const int32_t* bases, const int32_t* keep_idx,
                               const int32_t* cu_keep, int num_req, int total_keep, int max_keep, int num_kv_heads,
                               int head_dim, int32_t* new_lens, void* workspace, size_t workspace_bytes,
                               void* stream_) {
  if (num_req < 0 || total_keep < 0 || max_keep < 0 || pages_per_req < 0 || (dst_table != nullptr && dst_pages_per_req < 0))
    return fail(TSEL_ERR_INVALID_VALUE, "negative size");
  TSEL_TRY(check_cache(k_pages, v_pages, k_exps, v_exps, num_pages, page_size, num_kv_heads, head_dim));
  TSEL_TRY(check_header(workspace, workspace_bytes));
  if (num_req == 0) return TSEL_OK;
  if (cu_keep == nullptr || !aligned(cu_keep, 4) || !aligned(starts, 4) || !aligned(bases, 4) || !aligned(new_lens, 4))
    return fail(TSEL_ERR_INVALID_VALUE, "cu_keep, starts, bases or new_lens");
  if (total_keep > 0 && (keep_idx == nullptr || !aligned(keep_idx, 4))) return fail(TSEL_ERR_INVALID_VALUE, "keep_idx");
  if (max_keep > 0 && pages_per_req > 0 && (page_table == nullptr || !aligned(page_table, 4)))
    return fail(TSEL_ERR_INVALID_VALUE, "page_table");
  if (page_table_stride < pages_per_req || (dst_table != nullptr && dst_table_stride < dst_pages_per_req))
    return fail(TSEL_ERR_INVALID_VALUE, "table strides %lld, %lld", (long long)page_table_stride, (long long)dst_table_stride);
  if (!aligned(dst_table, 4)) return fail(TSEL_ERR_INVALID_VALUE, "dst_table");
  const Ints lens("new_lens", new_lens, num_req);
  TSEL_TRY(check_apart(lens, Ints("starts", starts, num_req)));
  TSEL_TRY(check_apart(lens, Ints("bases", bases, num_req)));
  TSEL_TRY(check_apart(lens, Ints("keep_idx", keep_idx, total_keep)));
  TSEL_TRY(check_apart(lens, Ints("cu_keep", cu_keep, int64_t(num_req) + 1)));
  TSEL_TRY(check_apart(lens, Ints("page_table", page_table, num_req, page_table_stride, pages_per_req)));
  TSEL_TRY(check_apart(lens, Ints("dst_table", dst_table, num_req, dst_table_stride, dst_pages_per_req)));
  MoveParams p{};
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.k_exps = k_exps;
  p.v_exps = v_exps;
  p.num_pages = num_pages;
  p.page_shift = page_shift_of(page_size);
  p.Hkv = num_kv_heads;
  p.d = head_dim;
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.width = pages_per_req;
  p.dst_table = dst_table;
  p.dst_stride = dst_table_stride;
  p.dst_width = dst_pages_per_req;
  p.starts = starts;
  p.bases = bases;
  p.keep = keep_idx;
  p.cu_keep = cu_keep;
  p.total = total_keep;
  p.max_keep = max_keep > 0 ? max_keep : 1;   // the lengths are written without kept tokens too
  p.R = num_req;
  p.new_lens = new_lens;
  p.status = &static_cast<WsHeader*>(workspace)->status;
  int sms = 0;
  if (device_sms(&sms) != 0) return fail(TSEL_ERR_CUDA, "cannot query the SM count");
  move_plan(p, sms);
  p.max_keep = max_keep;
  if (int64_t(p.R) * p.chunks * p.head_parts * p.slices > 0x7FFFFFFFll)
    return fail(TSEL_ERR_UNSUPPORTED, "too many units of work");
  const cudaError_t e = launch_move(p, static_cast<cudaStream_t>(stream_));
  return e == cudaSuccess ? TSEL_OK : cuda_fail(e, "cache compaction launch");
}

size_t tsel_cache_resize_workspace_size(int num_rows, int pages_per_row) {
  if (num_rows < 0 || pages_per_row < 0 || int64_t(num_rows) * pages_per_row > 0x7FFFFFFFll) return 0;
  const int64_t found = align_up(kWsHeaderBytes + 4 * (int64_t(num_rows) + 1), 256);
  return size_t(found + 4 * align_up(int64_t(num_rows) * (pages_per_row > 0 ? pages_per_row : 1), 64));
}

// What resizing and forking have in common.
static tsel_status pages_params(PagesParams* p, int32_t* refs, int num_pages, int page_size, int32_t* page_table,
                                int64_t page_table_stride, int num_rows, int pages_per_row, int32_t* lens,
                                void* workspace, size_t workspace_bytes) {
  if (page_shift_of(page_size) < 0)
    return fail(TSEL_ERR_UNSUPPORTED, "page_size=%d (supported: 16, 32, 64, 128)", page_size);
  if (num_pages < 0 || int64_t(num_pages) * page_size > 0x7FFFFFFFll)
    return fail(TSEL_ERR_INVALID_VALUE, "num_pages=%d of %d", num_pages, page_size);
  if (num_rows < 0 || pages_per_row < 0 || int64_t(num_rows) * pages_per_row > 0x7FFFFFFFll)
    return fail(TSEL_ERR_INVALID_VALUE, "%d rows of %d pages", num_rows, pages_per_row);
  TSEL_TRY(check_header(workspace, workspace_bytes));
  const size_t need = tsel_cache_resize_workspace_size(num_rows, pages_per_row);
  if (workspace_bytes < need) return fail(TSEL_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, need);
  if (num_rows > 0 && (lens == nullptr || !aligned(lens, 4))) return fail(TSEL_ERR_INVALID_VALUE, "lens");
  if (num_rows > 0 && pages_per_row > 0 && (page_table == nullptr || !aligned(page_table, 4)))
    return fail(TSEL_ERR_INVALID_VALUE, "page_table");
  if (page_table_stride < pages_per_row)
    return fail(TSEL_ERR_INVALID_VALUE, "page_table_stride %lld", (long long)page_table_stride);
  if (num_pages > 0 && (refs == nullptr || !aligned(refs, 4))) return fail(TSEL_ERR_INVALID_VALUE, "refs");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p->refs = refs;
  p->num_pages = num_pages;
  p->page_shift = page_shift_of(page_size);
  p->table = page_table;
  p->table_stride = page_table_stride;
  p->rows = num_rows;
  p->width = pages_per_row;
  p->lens = lens;
  p->plan = reinterpret_cast<int32_t*>(ws + kWsHeaderBytes);
  p->found = reinterpret_cast<int32_t*>(ws + align_up(kWsHeaderBytes + 4 * (int64_t(num_rows) + 1), 256));
  p->status = &reinterpret_cast<WsHeader*>(ws)->status;
  return TSEL_OK;
}

// refs, page_table and lens are written: apart from one another and from `in`.
static tsel_status pages_apart(const PagesParams& p, const Ints* in, int count) {
  const Ints out[3] = {Ints("refs", p.refs, p.num_pages), Ints("page_table", p.table, p.rows, p.table_stride, p.width),
                       Ints("lens", p.lens, p.rows)};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < i; ++j) TSEL_TRY(check_apart(out[j], out[i]));
    for (int j = 0; j < count; ++j) TSEL_TRY(check_apart(out[i], in[j]));
  }
  return TSEL_OK;
}

tsel_status tsel_cache_resize(int32_t* refs, int num_pages, int page_size, int32_t* page_table,
                              int64_t page_table_stride, int num_rows, int pages_per_row, int32_t* lens,
                              const int32_t* new_lens, void* workspace, size_t workspace_bytes, void* stream_) {
  PagesParams p{};
  TSEL_TRY(pages_params(&p, refs, num_pages, page_size, page_table, page_table_stride, num_rows, pages_per_row, lens,
                        workspace, workspace_bytes));
  if (num_rows == 0) return TSEL_OK;
  if (new_lens == nullptr || !aligned(new_lens, 4)) return fail(TSEL_ERR_INVALID_VALUE, "new_lens");
  p.new_lens = new_lens;
  // lens themselves ask for what is there
  const Ints in("new_lens", new_lens == lens ? nullptr : new_lens, num_rows);
  TSEL_TRY(pages_apart(p, &in, 1));
  const cudaError_t e = launch_resize(p, static_cast<cudaStream_t>(stream_));
  return e == cudaSuccess ? TSEL_OK : cuda_fail(e, "cache resize launch");
}

tsel_status tsel_cache_fork(uint8_t* k_pages, uint8_t* v_pages, uint8_t* k_exps, uint8_t* v_exps, int num_pages,
                            int page_size, int num_kv_heads, int head_dim, int32_t* refs, int32_t* page_table,
                            int64_t page_table_stride, int num_rows, int pages_per_row, int32_t* lens,
                            const int32_t* parents, const int32_t* children, int num_forks, void* workspace,
                            size_t workspace_bytes, void* stream_) {
  TSEL_TRY(check_cache(k_pages, v_pages, k_exps, v_exps, num_pages, page_size, num_kv_heads, head_dim));
  PagesParams p{};
  TSEL_TRY(pages_params(&p, refs, num_pages, page_size, page_table, page_table_stride, num_rows, pages_per_row, lens,
                        workspace, workspace_bytes));
  if (num_forks < 0 || num_forks > num_rows)
    return fail(TSEL_ERR_INVALID_VALUE, "num_forks=%d of %d rows", num_forks, num_rows);
  if (num_forks == 0) return TSEL_OK;
  if (parents == nullptr || children == nullptr || !aligned(parents, 4) || !aligned(children, 4))
    return fail(TSEL_ERR_INVALID_VALUE, "parents or children");
  p.parents = parents;
  p.children = children;
  p.n = num_forks;
  const Ints in[2] = {Ints("parents", parents, num_forks), Ints("children", children, num_forks)};
  TSEL_TRY(pages_apart(p, in, 2));
  p.k_pages = k_pages;
  p.v_pages = v_pages;
  p.k_exps = k_exps;
  p.v_exps = v_exps;
  p.Hkv = num_kv_heads;
  p.d = head_dim;
  p.parts = kForkParts;
  if (int64_t(num_forks) * p.parts > 0x7FFFFFFFll) return fail(TSEL_ERR_UNSUPPORTED, "too many units of work");
  const cudaError_t e = launch_fork(p, static_cast<cudaStream_t>(stream_));
  return e == cudaSuccess ? TSEL_OK : cuda_fail(e, "cache fork launch");
}

}  // extern "C"
