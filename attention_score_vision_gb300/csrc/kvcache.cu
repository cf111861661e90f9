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
// heads), a group of lanes one row at a time, 16 elements per lane, two rows
// loaded before the first is stored. K may be rotated on its way (rope.cuh); it
// is quantised from the fp32 rotation, without a rounding in between.
//
// 36,831 tokens on 8 KV heads of 128, bf16 (227 MB): write 42 us, 5.4 TB/s or 79%
// of the copy rate, read 39 us, 85%; 131,072 tokens rotated, written and read
// back (1.6 GB): 302 us, 79% (the rotated write 175, 4.5 TB/s or 66%: schedulers
// issue in 70% of the cycles, the ALU pipe is busy in 63%, and the largest stall
// is the wait for a token's rows, which 30 resident warps with eight rows in
// flight each do not cover); 200 tokens written 2.3 us, 142 read 2.1 us.
#include "launch_util.cuh"
#include "rope.cuh"

namespace tsel {

namespace {

constexpr int kCacheThreads = 256;
constexpr int kCacheWarps = kCacheThreads / 32;
constexpr int kCacheRows = 2;

// Two fp32 values as E4M3 codes (x in the low byte), round to nearest even.
__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}

// Largest magnitude of the three; NaN when one of them is.
__device__ __forceinline__ float max3_abs(float m, float x, float y) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(x), "f"(y));
  return r;
}

// Codes of V values times a power of two; zeros for a row that is not finite.
template <int V>
__device__ __forceinline__ void encode(const float (&f)[V], float up, bool finite, Vec<uint8_t, V>& c) {
  if constexpr (V >= 4) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&c.p[0]);
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float2 up2 = make_float2(up, up);
      const float2 lo = __fmul2_rn(make_float2(f[j], f[j + 1]), up2), hi = __fmul2_rn(make_float2(f[j + 2], f[j + 3]), up2);
      const uint32_t x = e4m3x2(lo.x, lo.y) | (e4m3x2(hi.x, hi.y) << 16);
      w[j / 4] = finite ? x : 0u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) c.e[j] = finite ? uint8_t(e4m3x2(f[j] * up, 0.f)) : uint8_t(0);
  }
}

// Two E4M3 codes as fp16 (exact).
__device__ __forceinline__ __half2 from_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
  return *reinterpret_cast<__half2*>(&r);
}

// Row of a slot's first head; head h's is h << page_shift further on.
__device__ __forceinline__ int64_t cache_row(const CacheParams& p, int slot) {
  const int64_t page = slot >> p.page_shift;
  return ((page * p.Hkv) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
}

// The slot of a token: -1 for none (a padded token, or one out of range,
// which sets the status word).
__device__ __forceinline__ int cache_slot(const CacheParams& p, int slot, int lane) {
  if (int64_t(slot) >= (int64_t(p.num_pages) << p.page_shift)) {
    if (lane == 0) set_status(p.status, TSEL_DEV_PAGES);
    return -1;
  }
  return slot < 0 ? -1 : slot;
}

template <typename T, int V>
__global__ void __launch_bounds__(kCacheThreads, sizeof(T) * V > 16 ? 3 : 4) cache_write_kernel(const CacheParams p) {
  constexpr int IPL = V == 1 ? 2 : 1;   // items per lane: rows have at most 128 elements
  __shared__ __align__(16) float s_cs[kCacheWarps][2 * kRopeMaxPairs];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int items = p.d / (2 * V);
  const int lpr = 1 << p.lane_shift, subs = 32 >> p.lane_shift;
  const int sub = lane >> p.lane_shift, l0 = lane & (lpr - 1);
  const int64_t t = int64_t(blockIdx.x) * kCacheWarps + warp;   // token; blockIdx.y: share of its rows
  if (t >= p.total) return;
  const int r0 = int(blockIdx.y) * p.per;   // K heads, then V heads
  const int r1 = min(r0 + p.per, 2 * p.Hkv);
  int slot = __ldg(p.slots + t);   // looked at once the rows are on their way
  const T* k = static_cast<const T*>(p.k) + t * p.k_stride;
  const T* v = static_cast<const T*>(p.v) + (t * p.v_stride - int64_t(p.Hkv) * p.d);
  int64_t row0 = 0;
  float* cs = s_cs[warp];
  const bool turn = p.num_pairs > 0 && r0 < p.Hkv;
  bool any_nan = false, ready = !turn;
  for (int first = r0; first < r1; first += subs * kCacheRows) {   // the same for the whole warp
    Vec<T, V> a[kCacheRows][IPL], b[kCacheRows][IPL];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      // lanes and rows past the end repeat the last ones: loads without a
      // condition are issued together, and a repeated value changes no maximum
      const int r = min(first + sub + i * subs, r1 - 1);
      const bool is_k = r < p.Hkv;
      const T* src = (is_k ? k : v) + r * p.d;
#pragma unroll
      for (int n = 0; n < IPL; ++n) {
        int o1, o2;
        rope_item(min(l0 + n * lpr, items - 1), V, is_k ? p.num_pairs : 0, p.adjacent != 0, o1, o2);
        a[i][n].load(src + o1);
        b[i][n].load(src + o2);
      }
    }
    if (!ready) {   // the angles, while the rows are on their way
      if (rope_angles(cs, p.table, p.num_pairs, p.pos + t * p.pos_dim, p.pos_dim, 1.f))
        set_status(p.status, TSEL_DEV_POSITIONS);
      __syncwarp();
      ready = true;
    }
    if (first == r0) {
      slot = cache_slot(p, slot, lane);
      if (slot < 0) return;
      row0 = cache_row(p, slot);
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      const int r = first + sub + i * subs;
      if (first + i * subs >= r1) break;   // no lane of the warp has a row left
      const bool is_k = r < p.Hkv;
      float fa[IPL][V], fb[IPL][V];
      float most = 0.f;   // NaN when a value is
#pragma unroll
      for (int n = 0; n < IPL; ++n) {
        const int item = min(l0 + n * lpr, items - 1);
        a[i][n].get(fa[n]);
        b[i][n].get(fb[n]);
        if (min(r, r1 - 1) < p.Hkv && item * V < p.num_pairs) {
          float c[V], s[V];
          rope_fetch<V>(cs, item, c, s);
          rope_turn<V>(fa[n], fb[n], c, s, p.adjacent != 0);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) most = max3_abs(most, fa[n][j], fb[n][j]);
      }
      uint32_t top = __float_as_uint(most);
      for (int o = lpr >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      // e + 127: exponent field - 8 when 1.m <= 1.75 (448 = 1.75 * 2^8), - 7 above
      const bool finite = top < 0x7F800000u;
      int e = int(top >> 23) - ((top & 0x7FFFFFu) <= 0x600000u ? 8 : 7);
      if (e < 0) e = 0;
      const float up = __uint_as_float(uint32_t(254 - e) << 23);   // 2^-(e - 127), normal
      if (r < r1) {
        const int64_t row = row0 + ((is_k ? r : r - p.Hkv) << p.page_shift);
        uint8_t* dst = (is_k ? p.k_pages : p.v_pages) + row * p.d;
#pragma unroll
        for (int n = 0; n < IPL; ++n) {
          const int item = l0 + n * lpr;
          if (item >= items) continue;
          int o1, o2;
          rope_item(item, V, is_k ? p.num_pairs : 0, p.adjacent != 0, o1, o2);
          Vec<uint8_t, V> ca, cb;
          encode<V>(fa[n], up, finite, ca);
          encode<V>(fb[n], up, finite, cb);
          if constexpr (V == 8) {
            if (o2 == o1 + V) {   // V rows and adjacent pairs: 16 bytes in a row
              *reinterpret_cast<uint4*>(dst + o1) = make_uint4(ca.p[0].x, ca.p[0].y, cb.p[0].x, cb.p[0].y);
              continue;
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
  if (any_nan) set_status(p.status, TSEL_DEV_NAN);
}

template <typename T>
__global__ void __launch_bounds__(kCacheThreads, 4) cache_read_kernel(const CacheParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int items = p.d / 16;   // 4 to 8 pieces of 16 codes
  const int sub = lane >> p.lane_shift, subs = 32 >> p.lane_shift, item = lane & ((1 << p.lane_shift) - 1);
  const int64_t t = int64_t(blockIdx.x) * kCacheWarps + (threadIdx.x >> 5);
  if (t >= p.total) return;
  const int r0 = int(blockIdx.y) * p.per;
  const int r1 = min(r0 + p.per, 2 * p.Hkv);
  T* ko = static_cast<T*>(p.k_out) + t * p.k_stride;
  T* vo = static_cast<T*>(p.v_out) + (t * p.v_stride - int64_t(p.Hkv) * p.d);
  const int slot = cache_slot(p, __ldg(p.slots + t), lane);
  const int64_t row0 = slot >= 0 ? cache_row(p, slot) : 0;
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
        const int64_t row = row0 + ((is_k ? r : r - p.Hkv) << p.page_shift);
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
        float f[16];
        const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 lo = __half22float2(from_e4m3x2(ws[j] & 0xFFFFu));
          const float2 hi = __half22float2(from_e4m3x2(ws[j] >> 16));
          f[4 * j] = lo.x * scale;
          f[4 * j + 1] = lo.y * scale;
          f[4 * j + 2] = hi.x * scale;
          f[4 * j + 3] = hi.y * scale;
        }
        x.set(f);
        T* dst = (is_k ? ko : vo) + r * p.d;
        x.store(dst + 16 * item);
      }
    }
  }
}

// Warps per token: as for the rotation, shared out until about 16 warps per SM.
template <typename Kernel>
cudaError_t launch_cache(Kernel kernel, CacheParams p, int lane_shift, int num_sms,
                         cudaStream_t stream) {
  const int rows = 2 * p.Hkv;
  const int max_parts = int(ceil_div(rows, 32 >> lane_shift));
  const int64_t want = ceil_div(int64_t(num_sms) * 16, p.total);
  const int parts = int(want < 1 ? 1 : (want > max_parts ? max_parts : want));
  p.lane_shift = lane_shift;
  p.per = int(ceil_div(rows, parts));
  const dim3 grid(unsigned(ceil_div(p.total, kCacheWarps)), unsigned(ceil_div(rows, p.per)));
  return launch_kernel(kernel, grid, kCacheThreads, 0, stream, 1, p);
}

template <typename T, int V>
cudaError_t launch_write_t(const CacheParams& p, int num_sms, cudaStream_t stream) {
  int shift = 0;
  while ((1 << shift) < p.d / (2 * V) && shift < 5) ++shift;
  return launch_cache(cache_write_kernel<T, V>, p, shift, num_sms, stream);
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
  const int shift = p.d / 16 <= 4 ? 2 : 3;
  switch (dtype) {
    case TSEL_BF16: return launch_cache(cache_read_kernel<__nv_bfloat16>, p, shift, num_sms, stream);
    case TSEL_FP16: return launch_cache(cache_read_kernel<__half>, p, shift, num_sms, stream);
    default: return launch_cache(cache_read_kernel<float>, p, shift, num_sms, stream);
  }
}

}  // namespace tsel
