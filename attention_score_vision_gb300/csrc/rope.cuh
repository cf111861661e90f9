// Rotary positions with several axes: the angle of a (token, pair) and the
// vector loads and stores that the rotation and the cache write share.
//
// The angle of pair i of token t is pos[t][axis_i] * f_i. A rope table entry
// holds f_i / (2 pi) modulo one turn as a 61-bit fixed-point fraction, shifted
// left by three, with the pair's axis in the low three bits. The product with
// the position is taken modulo 2^64, that is modulo one turn, exactly: a
// position of 2^31 loses nothing to range reduction (in floating point 32 bits
// lose 2^-24 of the whole angle, and 64-bit arithmetic is slow on this part).
// The phase is then reduced to an eighth of a turn on either side of the
// nearest quarter in integers, so the fp32 sine and cosine are good to their
// last bit or two whatever the position.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"

namespace tsel {

__device__ __forceinline__ void rope_cos_sin(uint64_t entry, int32_t pos, float& c, float& s) {
  const uint64_t ph = (entry & ~7ull) * uint64_t(int64_t(pos));   // turns * 2^64, modulo one turn
  const uint32_t quad = uint32_t((ph + (1ull << 61)) >> 62);      // nearest quarter turn
  const int64_t rem = int64_t(ph - (uint64_t(quad) << 62));       // [-2^61, 2^61)
  float s0, c0;
  sincospif(float(int32_t(rem >> 30)) * 1.1641532182693481e-10f, &s0, &c0);   // half turns: * 2^-33
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
  union {
    P p[N];
    T e[V];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = reinterpret_cast<const P*>(src)[i];
  }
  __device__ __forceinline__ void store(T* dst) const {
#pragma unroll
    for (int i = 0; i < N; ++i) reinterpret_cast<P*>(dst)[i] = p[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f32<T>(0.f);
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

// Cosines and sines of the V pairs of an item for one token. A table entry
// whose axis the positions do not have sets `bad` and leaves its pair as it is.
template <int V>
__device__ __forceinline__ void rope_angles(const uint64_t* __restrict__ table, int item,
                                            const int32_t* __restrict__ pos_row, int pos_dim,
                                            float (&c)[V], float (&s)[V], bool& bad) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const uint64_t e = __ldg(table + item * V + j);
    const int axis = int(e & 7ull);
    if (axis < pos_dim) {
      rope_cos_sin(e, __ldg(pos_row + axis), c[j], s[j]);
    } else {
      bad = true;
      c[j] = 1.f;
      s[j] = 0.f;
    }
  }
}

// The widest half that cuts both the rotated pairs and the rest of a row evenly.
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
  int parts;               // warps that share a token's heads
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
  int parts;
  uint32_t* status;
};

cudaError_t launch_rope(int dtype, const RopeParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_write(int dtype, const CacheParams& p, int num_sms, cudaStream_t stream);
cudaError_t launch_cache_read(int dtype, const CacheParams& p, int num_sms, cudaStream_t stream);

}  // namespace tsel
