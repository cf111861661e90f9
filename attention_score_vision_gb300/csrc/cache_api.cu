// Host side of the cache entry points of include/tsel.h (rotary positions,
// the quantised paged cache, attention over a shared prefix): argument checks,
// the rope table, workspace carving and kernel launches. Nothing here
// allocates or synchronises.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>

#include "attend.cuh"
#include "common.cuh"
#include "rope.cuh"

namespace tsel {
void record_error(const char* msg);
int device_sms(int* out);
uint64_t device_wait_timeout_ns();
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

size_t tsel_prefix_attention_workspace_size(int num_req, int total_q, int max_seqlen_q,
                                            int num_heads, int num_kv_heads, int head_dim,
                                            int max_prefix_len, int max_suffix_len) {
  if (num_req < 0 || total_q < 0 || max_seqlen_q < 0 || num_kv_heads < 1 ||
      num_heads < num_kv_heads || num_heads > 256 || num_heads % num_kv_heads != 0 ||
      num_heads / num_kv_heads > kTile || !cache_head_dim(head_dim) || max_prefix_len < 0 ||
      max_suffix_len < 0 || max_prefix_len > kAttMaxKeys || max_suffix_len > kAttMaxKeys)
    return 0;
  const AttPlan a = att_plan(num_req, total_q, max_seqlen_q, num_heads, num_kv_heads, head_dim,
                             max_prefix_len, max_suffix_len);
  return a.too_large ? 0 : size_t(a.total);
}

tsel_status tsel_prefix_attention(
    const void* q, int64_t q_row_stride, const int32_t* cu_seqlens_q, int num_req, int total_q,
    int max_seqlen_q, const uint8_t* k_pages, const uint8_t* v_pages, const uint8_t* k_exps,
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
  if (max_prefix_len > 0 && (prefix_pages == nullptr || prefix_len == nullptr))
    return fail(TSEL_ERR_INVALID_VALUE, "null prefix_pages or prefix_len");
  if (max_suffix_len > 0 && num_req > 0 && (page_table == nullptr || suffix_lens == nullptr))
    return fail(TSEL_ERR_INVALID_VALUE, "null page_table or suffix_lens");
  if (max_suffix_len > 0 && num_req > 0 && page_table_stride < ceil_div(max_suffix_len, page_size))
    return fail(TSEL_ERR_INVALID_VALUE, "page_table_stride %lld for %d keys",
                (long long)page_table_stride, max_suffix_len);
  TSEL_TRY(check_header(workspace, workspace_bytes));
  const AttPlan a = att_plan(num_req, total_q, max_seqlen_q, num_heads, num_kv_heads, head_dim,
                             max_prefix_len, max_suffix_len);
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

}  // extern "C"
