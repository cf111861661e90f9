// Rotary positions with several axes: the angle of a (token, pair) and the
// vector loads and stores that the rotation and the cache write share.
//
// The angle of pair i of token t is pos[t][axis_i] * f_i. A rope table entry
// holds f_i / (2 pi) modulo one turn as a 61-bit fixed-point fraction, shifted
// left by three, with the pair's axis in the low three bits. The product with
// the position is taken modulo 2^64, that is modulo one turn, exactly: range
// reduction loses nothing (in floating point 32 bits lose 2^-24 of the whole
// angle, and 64-bit arithmetic is slow on this part), and the phase is off by
// the entry's rounding alone, 2^-61 of a turn for each step of position. It is
// then reduced to an eighth of a turn on either side of the nearest quarter in
// integers, and what is left is rounded to fp32's 24 significant bits (not cut
// to a fixed step: the slow pairs' small angles keep their bits; it costs 0.7%
// of the rotation of 61,385 tokens). Sine and cosine are within 4 * 2^-24 of
// their own size: 2^-24 from that rounding, an ulp from the function.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"

namespace tsel {

__device__ __forceinline__ void rope_cos_sin(uint64_t entry, int32_t pos, float& c, float& s) {
  const uint64_t ph = (entry & ~7ull) * uint64_t(int64_t(pos));   // turns * 2^64, modulo one turn
  const uint32_t quad = uint32_t((ph + (1ull << 61)) >> 62);      // nearest quarter turn
  const int64_t rem = int64_t(ph - (uint64_t(quad) << 62));       // [-2^61, 2^61)
  float s0, c0;
  sincospif(__ll2float_rn(rem) * 1.0842021724855044e-19f, &s0, &c0);   // half turns: * 2^-63
  c = (quad & 1) ? s0 : c0;
  s = (quad & 1) ? c0 : s0;
  if (quad == 1 || quad == 2) c = -c;
  if (quad >= 2) s = -s;
}

// V elements of type T as 32-bit floats, loaded and stored in pieces of at
// most 16 bytes (V * sizeof(T) is a power of two; addresses are aligned to the
// piece).
template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Two 16-bit values in one word (the first in the low half).
template <typename T>
__device__ __forceinline__ void to_f32x2(uint32_t w, float& x, float& y) {
  if constexpr (sizeof(T) == 2) {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
      x = f.x, y = f.y;
    } else {
      x = __uint_as_float(w << 16);
      y = __uint_as_float(w & 0xFFFF0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint32_t from_f32x2(float x, float y) {
  uint32_t r = 0;
  if constexpr (std::is_same<T, __half>::value)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

template <int BYTES>
struct Piece;
template <>
struct Piece<16> { using type = uint4; };
template <>
struct Piece<8> { using type = uint2; };
template <>
struct Piece<4> { using type = uint32_t; };
template <>
struct Piece<2> { using type = uint16_t; };
template <>
struct Piece<1> { using type = uint8_t; };

template <typename T, int V>
struct Vec {
  static constexpr int BYTES = V * int(sizeof(T));
  static constexpr int PIECE = BYTES < 16 ? BYTES : 16;
  static constexpr int N = BYTES / PIECE;
  using P = typename Piece<PIECE>::type;
  static constexpr bool WORDS = sizeof(T) == 2 && V >= 2;   // 16-bit types: converted two at a time
  union {
    P p[N];
    T e[V];
    uint32_t w[WORDS ? V / 2 : 1];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void get(float (&f)[V]) const {
    if constexpr (WORDS) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) to_f32x2<T>(w[i], f[2 * i], f[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = to_f32(e[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
    if constexpr (WORDS) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = from_f32x2<T>(f[2 * i], f[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = from_f32<T>(f[i]);
    }
  }
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = reinterpret_cast<const P*>(src)[i];
  }
  __device__ __forceinline__ void store(T* dst) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<P*>(dst)[i] = p[i];
  }
};

// A row of d elements is cut into items of two V-element halves. Items below
// P / V hold V rotated pairs: (i, P + i) in the split layout, neighbouring
// elements in the adjacent one; the items after them hold the columns that are
// not rotated. Every element belongs to one item, so a row may be rotated in
// place.
__device__ __forceinline__ void rope_item(int item, int V, int P, bool adjacent, int& o1, int& o2) {
  const bool split = !adjacent && item * V < P;
  o1 = split ? item * V : 2 * V * item;
  o2 = split ? P + item * V : o1 + V;
}

// Rotates one item's pairs (a, b hold its halves in fp32).
template <int V>
__device__ __forceinline__ void rope_turn(float (&a)[V], float (&b)[V], const float (&c)[V],
                                          const float (&s)[V], bool adjacent) {
  if (!adjacent) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float x = a[j], y = b[j];
      a[j] = x * c[j] - y * s[j];
      b[j] = y * c[j] + x * s[j];
    }
  } else if constexpr (V == 1) {
    const float x = a[0], y = b[0];
    a[0] = x * c[0] - y * s[0];
    b[0] = y * c[0] + x * s[0];
  } else {
    // pair j of the item: elements 2j, 2j + 1 of its 2V
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float& ex = 2 * j < V ? a[2 * j < V ? 2 * j : 0] : b[2 * j < V ? 0 : 2 * j - V];
      float& ey = 2 * j < V ? a[2 * j < V ? 2 * j + 1 : 0] : b[2 * j < V ? 0 : 2 * j + 1 - V];
      const float x = ex, y = ey;
      ex = x * c[j] - y * s[j];
      ey = y * c[j] + x * s[j];
    }
  }
}

constexpr int kRopeMaxPairs = 128;

// Cosines and sines of one token's pairs, shared out over a warp and kept in
// its shared memory cs[2][kRopeMaxPairs] (a lane group per head would compute
// each of them several times over). A table entry whose axis the positions do
// not have returns true and leaves its pair as it is.
__device__ __forceinline__ bool rope_angles(float* cs, const uint64_t* __restrict__ table, int pairs,
                                            const int32_t* __restrict__ pos_row, int pos_dim,
                                            float sign) {
  bool bad = false;
  for (int i = threadIdx.x & 31; i < pairs; i += 32) {
    const uint64_t e = __ldg(table + i);
    const int axis = int(e & 7ull);
    float c = 1.f, s = 0.f;
    if (axis < pos_dim) rope_cos_sin(e, __ldg(pos_row + axis), c, s);
    else bad = true;
    cs[i] = c;
    cs[kRopeMaxPairs + i] = sign * s;
  }
  return bad;
}

// The cosines and sines of an item's V pairs.
template <int V>
__device__ __forceinline__ void rope_fetch(const float* cs, int item, float (&c)[V], float (&s)[V]) {
  if constexpr (V >= 4) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const float4 x = *reinterpret_cast<const float4*>(cs + item * V + j);
      const float4 y = *reinterpret_cast<const float4*>(cs + kRopeMaxPairs + item * V + j);
      c[j] = x.x, c[j + 1] = x.y, c[j + 2] = x.z, c[j + 3] = x.w;
      s[j] = y.x, s[j + 1] = y.y, s[j + 2] = y.z, s[j + 3] = y.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      c[j] = cs[item * V + j];
      s[j] = cs[kRopeMaxPairs + item * V + j];
    }
  }
}

// The widest half that cuts both the rotated pairs and the rest of a row evenly.
// 36,831 tokens, 16 + 8 heads of 128, bf16, with 64, 60, 62, 63 pairs (halves of 8,
// 4, 2, 1 elements): 70, 77, 105, 159 us.
inline int rope_vec(int head_dim, int num_pairs) {
  for (int v = 8; v > 1; v >>= 1)
    if (num_pairs % v == 0 && (head_dim - 2 * num_pairs) % (2 * v) == 0) return v;
  return 1;
}

struct RopeParams {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;   // elements
  const int32_t* pos;
  int pos_dim;
  const uint64_t* table;
  int num_pairs, total, H, Hkv, d;
  int adjacent, inverse;
  int per;                 // heads (Q and K together) a warp takes
  uint32_t* status;
};

struct CacheParams {
  const void* k;           // write: inputs; read: unused
  const void* v;
  void* k_out;             // read: outputs
  void* v_out;
  int64_t k_stride, v_stride;   // elements
  uint8_t* k_pages;
  uint8_t* v_pages;
  uint8_t* k_exps;
  uint8_t* v_exps;
  int num_pages, page_shift;
  const int32_t* slots;
  const int32_t* pos;
  int pos_dim;
  const uint64_t* table;
  int num_pairs, total, Hkv, d;
  int adjacent;
  int lane_shift;          // log2 of the lanes that share a row
  int per;                 // rows (K and V heads together) a warp takes
  uint32_t* status;
};

cudaError_t launch_rope(int dtype, const RopeParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_write(int dtype, const CacheParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_read(int dtype, const CacheParams& p, int num_sms, cudaStream_t stream);

}  // namespace tsel
