// The quantised paged cache: K and V rows written as E4M3 codes with one
// power-of-two scale per (token, head), and read back.
//
// The LiteVLM review deploys the language model in FP8, and the dynamic
// vision-token compression article (section 3.2) sends the pruned sequence to
// prefill and the KV cache; neither has code for the cache.
//
// A row x of head_dim elements is stored as codes c_j = RN_e4m3(x_j * 2^-e) and
// the byte e + 127, e the least integer (at least -127) with max|x| <= 448 *
// 2^e. A power of two costs a floating-point code nothing but the lowest part
// of its range, keeps x * 2^-e and c * 2^e exact, and takes one byte instead
// of four. A row with a NaN or an infinity cannot be scaled: it is stored as
// zeros with the byte 255, reads back as NaN, and sets TSEL_DEV_NAN.
//
// Pages are [num_pages][num_kv_heads][page_size][head_dim] codes and
// [num_pages][num_kv_heads][page_size] bytes, so that the keys of one head in
// one page are one contiguous block.
//
// HBM-bound, like the rotation: a warp takes one token (or a share of its
// heads), 16 elements per lane, up to four rows loaded before the first is
// stored. K may be rotated on its way (rope.cuh); it is quantised from the
// fp32 rotation, without a rounding in between.
#include "launch_util.cuh"
#include "rope.cuh"

namespace tsel {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 4;

// Two fp32 values as E4M3 codes (x in the low byte), round to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

// Two E4M3 codes as fp16 (exact).
__device__ __forceinline__ __half2 from_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
  return *reinterpret_cast<__half2*>(&r);
}

// Byte offset of head h's row of a slot, in rows.
__device__ __forceinline__ int64_t cache_row(const CacheParams& p, int slot, int h) {
  const int64_t page = slot >> p.page_shift;
  return ((page * p.Hkv + h) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

// The slot of a token: -1 for none (a padded token, or one out of range,
// which sets the status word).
__device__ __forceinline__ int cache_slot(const CacheParams& p, int64_t t, int lane) {
  const int slot = __ldg(p.slots + t);
  if (int64_t(slot) >= (int64_t(p.num_pages) << p.page_shift)) {
    if (lane == 0) set_status(p.status, TSEL_DEV_PAGES);
    return -1;
  }
  return slot < 0 ? -1 : slot;
}

template <typename T, int V>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
  constexpr int IPL = V == 1 ? 2 : 1;   // items per lane: rows have at most 128 elements
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int items = p.d / (2 * V);
  int lpr = 1;
  while (lpr < items && lpr < 32) lpr <<= 1;
  const int sub = lane / lpr, subs = 32 / lpr, l0 = lane % lpr;
  const int rows = 2 * p.Hkv;   // K heads, then V heads
  const int per = (rows + p.parts - 1) / p.parts;
  const int64_t units = int64_t(p.total) * p.parts;
  const int64_t nwarps = int64_t(gridDim.x) * (kCacheThreads / 32);
  const T* k = static_cast<const T*>(p.k);
  const T* v = static_cast<const T*>(p.v);
  bool any_nan = false;
  for (int64_t u = (int64_t(blockIdx.x) * kCacheThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
    const int64_t t = u / p.parts;
    const int r0 = int(u % p.parts) * per;
    const int r1 = min(r0 + per, rows);
    const int slot = cache_slot(p, t, lane);
    if (slot < 0) continue;
    float c[IPL][V], s[IPL][V];
    const bool turn = p.num_pairs > 0 && r0 < p.Hkv;
    if (turn) {
      bool bad = false;
#pragma unroll
      for (int n = 0; n < IPL; ++n) {
        const int item = l0 + n * lpr;
        if (item * V < p.num_pairs)
          rope_angles<V>(p.table, item, p.pos + t * p.pos_dim, p.pos_dim, c[n], s[n], bad);
      }
      if (bad) set_status(p.status, TSEL_DEV_POSITIONS);
    }
    for (int first = r0; first < r1; first += subs * kCacheRows) {   // the same for the whole warp
      Vec<T, V> a[kCacheRows][IPL], b[kCacheRows][IPL];
#pragma unroll
      for (int i = 0; i < kCacheRows; ++i) {
        const int r = first + sub + i * subs;
        const bool is_k = r < p.Hkv;
        const T* src = is_k ? k + t * p.k_stride + int64_t(r) * p.d
                            : v + t * p.v_stride + int64_t(r - p.Hkv) * p.d;
#pragma unroll
        for (int n = 0; n < IPL; ++n) {
          const int item = l0 + n * lpr;
          if (r < r1 && item < items) {
            int o1, o2;
            rope_item(item, V, is_k ? p.num_pairs : 0, p.adjacent != 0, o1, o2);
            a[i][n].load(src + o1);
            b[i][n].load(src + o2);
          } else {
            a[i][n].zero();
            b[i][n].zero();
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kCacheRows; ++i) {
        const int r = first + sub + i * subs;
        if (first + i * subs >= r1) break;   // no lane of the warp has a row left
        const bool is_k = r < p.Hkv;
        float fa[IPL][V], fb[IPL][V];
        uint32_t top = 0;
#pragma unroll
        for (int n = 0; n < IPL; ++n) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            fa[n][j] = to_f32(a[i][n].e[j]);
            fb[n][j] = to_f32(b[i][n].e[j]);
          }
          if (is_k && turn && (l0 + n * lpr) * V < p.num_pairs)
            rope_turn<V>(fa[n], fb[n], c[n], s[n], p.adjacent != 0);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            top = max(top, __float_as_uint(fa[n][j]) & 0x7FFFFFFFu);
            top = max(top, __float_as_uint(fb[n][j]) & 0x7FFFFFFFu);
          }
        }
        for (int o = lpr >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // e + 127: exponent field - 8 when 1.m <= 1.75 (448 = 1.75 * 2^8), - 7 above
        const bool finite = top < 0x7F800000u;
        int e = int(top >> 23) - ((top & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
        if (e < 0) e = 0;
        const float up = __uint_as_float(uint32_t(254 - e) << 23);   // 2^-(e - 127), normal
        if (r < r1) {
          const int64_t row = cache_row(p, slot, is_k ? r : r - p.Hkv);
          uint8_t* dst = (is_k ? p.k_pages : p.v_pages) + row * p.d;
#pragma unroll
          for (int n = 0; n < IPL; ++n) {
            const int item = l0 + n * lpr;
            if (item >= items) continue;
            int o1, o2;
            rope_item(item, V, is_k ? p.num_pairs : 0, p.adjacent != 0, o1, o2);
            Vec<uint8_t, V> ca, cb;
#pragma unroll
            for (int j = 0; j < V; j += 2) {
              const int j1 = V == 1 ? 0 : j + 1;
              const uint32_t ea = finite ? e4m3x2(fa[n][j] * up, fa[n][j1] * up) : 0u;
              const uint32_t eb = finite ? e4m3x2(fb[n][j] * up, fb[n][j1] * up) : 0u;
              ca.e[j] = uint8_t(ea);
              cb.e[j] = uint8_t(eb);
              if (V > 1) {
                ca.e[j1] = uint8_t(ea >> 8);
                cb.e[j1] = uint8_t(eb >> 8);
              }
            }
            ca.store(dst + o1);
            cb.store(dst + o2);
          }
          if (l0 == 0) (is_k ? p.k_exps : p.v_exps)[row] = finite ? uint8_t(e) : uint8_t(255);
          any_nan = any_nan || !finite;
        }
      }
    }
  }
  if (any_nan) set_status(p.status, TSEL_DEV_NAN);
}

template <typename T>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int items = p.d / 16;   // 4 to 8 pieces of 16 codes
  const int lpr = items <= 4 ? 4 : 8;
  const int sub = lane / lpr, subs = 32 / lpr, item = lane % lpr;
  const int rows = 2 * p.Hkv;
  const int per = (rows + p.parts - 1) / p.parts;
  const int64_t units = int64_t(p.total) * p.parts;
  const int64_t nwarps = int64_t(gridDim.x) * (kCacheThreads / 32);
  T* ko = static_cast<T*>(p.k_out);
  T* vo = static_cast<T*>(p.v_out);
  for (int64_t u = (int64_t(blockIdx.x) * kCacheThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
    const int64_t t = u / p.parts;
    const int r0 = int(u % p.parts) * per;
    const int r1 = min(r0 + per, rows);
    const int slot = cache_slot(p, t, lane);
    for (int first = r0 + sub; first < r1; first += subs * kCacheRows) {
      uint4 w[kCacheRows];
      uint32_t e[kCacheRows];
#pragma unroll
      for (int i = 0; i < kCacheRows; ++i) {
        const int r = first + i * subs;
        w[i] = make_uint4(0, 0, 0, 0);
        e[i] = 0;
        if (r < r1 && item < items && slot >= 0) {
          const bool is_k = r < p.Hkv;
          const int64_t row = cache_row(p, slot, is_k ? r : r - p.Hkv);
          w[i] = *reinterpret_cast<const uint4*>((is_k ? p.k_pages : p.v_pages) + row * p.d + 16 * item);
          e[i] = (is_k ? p.k_exps : p.v_exps)[row];
        }
      }
#pragma unroll
      for (int i = 0; i < kCacheRows; ++i) {
        const int r = first + i * subs;
        if (r < r1 && item < items) {
          const bool is_k = r < p.Hkv;
          // 2^(e - 127); 255 is NaN, 0 is 2^-127 (a denormal float)
          const float scale = e[i] == 255 ? __uint_as_float(0x7FC00000u)
                              : (e[i] == 0 ? 5.8774717541114375e-39f : __uint_as_float(e[i] << 23));
          Vec<T, 16> x;
          const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 lo = __half22float2(from_e4m3x2(ws[j] & 0xFFFFu));
            const float2 hi = __half22float2(from_e4m3x2(ws[j] >> 16));
            x.e[4 * j] = from_f32<T>(lo.x * scale);
            x.e[4 * j + 1] = from_f32<T>(lo.y * scale);
            x.e[4 * j + 2] = from_f32<T>(hi.x * scale);
            x.e[4 * j + 3] = from_f32<T>(hi.y * scale);
          }
          T* dst = is_k ? ko + t * p.k_stride + int64_t(r) * p.d
                        : vo + t * p.v_stride + int64_t(r - p.Hkv) * p.d;
          x.store(dst + 16 * item);
        }
      }
    }
  }
}

// Warps per token: as for the rotation, shared out until about 16 warps per SM.
template <typename Kernel>
cudaError_t launch_cache(Kernel kernel, CacheParams p, int lanes_per_row, int num_sms,
                         cudaStream_t stream) {
  const int max_parts = int(ceil_div(2 * p.Hkv, 32 / lanes_per_row));
  const int64_t want = ceil_div(int64_t(num_sms) * 16, p.total);
  p.parts = int(want < 1 ? 1 : (want > max_parts ? max_parts : want));
  int64_t blocks = ceil_div(int64_t(p.total) * p.parts, kCacheThreads / 32);
  const int64_t most = int64_t(num_sms) * 8;
  if (blocks > most) blocks = most;
  return launch_kernel(kernel, dim3(unsigned(blocks)), kCacheThreads, 0, stream, 1, p);
}

template <typename T, int V>
cudaError_t launch_write_t(const CacheParams& p, int num_sms, cudaStream_t stream) {
  int lpr = 1;
  while (lpr < p.d / (2 * V) && lpr < 32) lpr <<= 1;
  return launch_cache(cache_write_kernel<T, V>, p, lpr, num_sms, stream);
}

template <typename T>
cudaError_t launch_write_v(const CacheParams& p, int num_sms, cudaStream_t stream) {
  switch (rope_vec(p.d, p.num_pairs)) {
    case 8: return launch_write_t<T, 8>(p, num_sms, stream);
    case 4: return launch_write_t<T, 4>(p, num_sms, stream);
    case 2: return launch_write_t<T, 2>(p, num_sms, stream);
    default: return launch_write_t<T, 1>(p, num_sms, stream);
  }
}

}  // namespace

cudaError_t launch_cache_write(int dtype, const CacheParams& p, int num_sms, cudaStream_t stream) {
  switch (dtype) {
    case TSEL_BF16: return launch_write_v<__nv_bfloat16>(p, num_sms, stream);
    case TSEL_FP16: return launch_write_v<__half>(p, num_sms, stream);
    default: return launch_write_v<float>(p, num_sms, stream);
  }
}

cudaError_t launch_cache_read(int dtype, const CacheParams& p, int num_sms, cudaStream_t stream) {
  const int lpr = p.d / 16 <= 4 ? 4 : 8;
  switch (dtype) {
    case TSEL_BF16: return launch_cache(cache_read_kernel<__nv_bfloat16>, p, lpr, num_sms, stream);
    case TSEL_FP16: return launch_cache(cache_read_kernel<__half>, p, lpr, num_sms, stream);
    default: return launch_cache(cache_read_kernel<float>, p, lpr, num_sms, stream);
  }
}

}  // namespace tsel
