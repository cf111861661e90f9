// Attention over the cache for few query rows: one decoding step of a request
// (its query heads of one KV head) over its own suffix, or a small batch over
// the prefix. The wide kernel (attend.cu) turns every key into an operand of a
// 128-row product; with 16 rows or fewer that is nearly all waste, and reading
// the codes is what is left to bound the work.
//
// Same quantity and partial results as attend.cu. A CTA of four warps takes 16
// rows of one KV head and a chunk of keys; each warp walks every fourth block of
// 16 keys on its own, with its own running reference, sums and output, and the
// four are added up at the end.
//   - Codes come through cp.async, 16 bytes per lane, four blocks ahead, into
//     places that the same lane reads back: shared memory only lengthens the
//     prefetch (4 KB a block and warp, up to 144 KB in flight per SM), no
//     barrier is needed.
//   - Both products are mma.sync.m16n8k16 on fp16 (rows padded to 16; tcgen05
//     has no shape below 64 rows). The order of the head dimension inside S and
//     of the keys inside P V is free, so each lane takes the elements of one
//     16-byte piece for its fragments and converts them in registers: the codes
//     go from the cache to the tensor cores without a transposition or a store.
//   - A key's scales multiply S (K) and P (V, relative to the largest exponent
//     so far, so that P stays inside fp16).
// HBM-bound: 4 KB of codes per block cost about 260 instructions of one warp.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend.cuh"
#include "imp_pass.cuh"

namespace tsel {

namespace {

constexpr int kNarWarps = 4;
constexpr int kNarThreads = 32 * kNarWarps;
constexpr int kNarStages = 4;
constexpr int kNarKeys = 16;         // keys of a block
constexpr float kNarLift = 6.f;      // P = 2^6 at the row's reference
constexpr float kNarSlack = 9.f;     // the reference may lag the row maximum by 2^9

template <int D>
struct NarCfg {
  static constexpr int H64 = D / 64;               // whole 64-element parts of a row
  static constexpr int TAIL = (D % 64) / 16;       // 4-byte words per lane of the rest
  static constexpr int KSLOTS = H64 + (TAIL ? 1 : 0);
  static constexpr int KSTEPS = D / 16;            // k16 steps of S
  static constexpr int CB = D == 64 ? 8 : 16;      // V columns per lane (consecutive ones)
  static constexpr int SLOTS = 2 * KSLOTS + 4;     // 16-byte places per lane and stage
  static constexpr int STAGE_BYTES = SLOTS * 512 + 32;   // codes, then the 16 exponents of K and of V
  static constexpr int WARP_BYTES = kNarStages * STAGE_BYTES;
  static constexpr int OFF_ROWS = kNarWarps * WARP_BYTES;   // fp32 m, l [warp][16], int vref [warp]
  static constexpr int SMEM_BYTES = OFF_ROWS + kNarWarps * (2 * 16 + 4) * 4;
  static_assert(kNarWarps * 16 * D * 4 <= OFF_ROWS, "the outputs fit the ring");
  static_assert(SMEM_BYTES <= 75 * 1024, "three CTAs per SM");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(ok ? N : 0), "n"(N)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(two)));
  return r;
}

__device__ __forceinline__ uint32_t f16x2(float x, float y) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 2^(e - 127); 255 is NaN, 0 is 2^-127 (a denormal float).
__device__ __forceinline__ float exp_scale(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7FC00000u : (e == 0u ? 0x00400000u : e << 23));
}

template <int D>
__global__ void __launch_bounds__(kNarThreads, 3) attend_narrow_kernel(const AttParams p) {
  using C = NarCfg<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;   // fragment row (and key or column), fragment column pair
  if (!p.late_wait) pdl_wait();
  pdl_launch_dependents();
  // With late_wait the launch before this one is the wide kernel of the same
  // call. It let this one start after its own wait, so the inputs are final;
  // its completion is waited for at the end, for the launch that joins both.
  const AttUnit w = att_unit(p, blockIdx.x, kAttNarrowBlock);
  const int row0 = w.group * kAttNarrowBlock;
  const int rows = w.bad ? 0 : min((w.tok_last - w.tok_first) * p.G - row0, kAttNarrowBlock);
  if (w.bad && threadIdx.x == 0) set_status(p.status, TSEL_DEV_SEQLENS);
  if (rows <= 0) {
    if (p.late_wait) pdl_wait();
    return;
  }
  const int keys = w.k1 - w.k0;
  if (keys <= 0) {   // no visible key in this chunk: an empty partial
    if (p.late_wait) pdl_wait();
    if (int(threadIdx.x) < rows) {
      const int r = row0 + int(threadIdx.x);
      p.part_lse[(int64_t(w.slot) * p.Tq + w.tok_first + r / p.G) * p.H + w.kvh * p.G + r % p.G] = kNegInf;
    }
    return;
  }

  // ---- the warp's blocks: block b of the chunk for b = warp, warp + 4, ...
  const int blocks = (keys + kNarKeys - 1) / kNarKeys;
  const int mine = (blocks - warp + kNarWarps - 1) / kNarWarps;
  const uint32_t ring = smem_u32(smem) + warp * C::WARP_BYTES;
  const uint8_t* ring_ptr = smem + warp * C::WARP_BYTES;
  const int64_t head_row = int64_t(w.kvh) << p.page_shift;
  const int mask = (1 << p.page_shift) - 1;
  int page_of_lane = -1;   // page of this warp's block 32 * (i / 32) + lane
  auto fetch = [&](int i) {   // i-th block of this warp into stage i % kNarStages
    if ((i & 31) == 0) {
      const int key = (warp + (i + lane) * kNarWarps) * kNarKeys;
      page_of_lane = -1;
      if (key < keys) {
        page_of_lane = __ldg(w.pages + ((w.k0 + key) >> p.page_shift));
        if (page_of_lane < 0 || page_of_lane >= p.num_pages) {
          set_status(p.status, TSEL_DEV_PAGES);
          page_of_lane = -1;   // read as zeros
        }
      }
    }
    const int pg = __shfl_sync(0xffffffffu, page_of_lane, i & 31);
    if (i < mine) {
      const int key = (warp + i * kNarWarps) * kNarKeys;
      const int left = pg >= 0 ? keys - key : 0;   // keys of the block inside the chunk
      const int64_t row = (int64_t(max(pg, 0)) * p.Hkv << p.page_shift) + head_row + ((w.k0 + key) & mask);
      const uint8_t* ks = p.k_pages + row * D;
      const uint8_t* vs = p.v_pages + row * D;
      const uint32_t dst = ring + (i % kNarStages) * C::STAGE_BYTES + lane * 16;
#pragma unroll
      for (int t = 0; t < 2; ++t) {   // keys 8 t + g, elements 16 c.. of each 64
        const uint8_t* src = ks + (8 * t + g) * D;
        const bool in = 8 * t + g < left;
#pragma unroll
        for (int h = 0; h < C::H64; ++h)
          cp_async16(dst + (t * C::KSLOTS + h) * 512, src + 64 * h + 16 * c, in);
#pragma unroll
        for (int x = 0; x < C::TAIL; ++x)
          cp_async_small<4>(dst + (t * C::KSLOTS + C::H64) * 512 + 4 * x,
                            src + 64 * C::H64 + 4 * C::TAIL * c + 4 * x, in);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {   // keys 2 c + {0, 1, 8, 9}, columns CB g ..
        const int key_in = 2 * c + (t & 1) + (t >> 1) * 8;
        const bool in = key_in < left && C::CB * g < D;
        const uint8_t* src = vs + (in ? key_in * D + C::CB * g : 0);
        if (C::CB == 16) cp_async16(dst + (2 * C::KSLOTS + t) * 512, src, in);
        else cp_async_small<8>(dst + (2 * C::KSLOTS + t) * 512, src, in);
      }
      if (lane < 2)
        cp_async16(ring + (i % kNarStages) * C::STAGE_BYTES + C::SLOTS * 512 + 16 * lane,
                   (lane == 0 ? p.k_exps : p.v_exps) + row, pg >= 0);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kNarStages - 1; ++i) fetch(i);

  // ---- Q: rows g and g + 8 as A fragments, scaled to fp16 by a power of two
  uint32_t qa[C::KSTEPS][4];
  float qc[2];
  int end[2];   // keys of the chunk that the row sees
  {
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int rr = g + 8 * hi;
      const bool ok = rr < rows;
      const int r = row0 + (ok ? rr : 0);
      const int tok = w.tok_first + r / p.G;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(
          static_cast<const uint16_t*>(p.q) + tok * p.q_stride + int64_t(w.kvh * p.G + r % p.G) * D);
      const int lim = w.causal ? w.lim0 + (tok - w.tok_first) : w.lim0;
      end[hi] = ok ? min(lim, w.k1) - w.k0 : 0;
#pragma unroll
      for (int h = 0; h < C::H64; ++h) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          qa[4 * h + s][hi] = ok ? __ldg(src + 32 * h + 8 * c + 2 * s) : 0u;
          qa[4 * h + s][hi + 2] = ok ? __ldg(src + 32 * h + 8 * c + 2 * s + 1) : 0u;
        }
      }
#pragma unroll
      for (int s = 0; s < C::TAIL; ++s) {
        qa[4 * C::H64 + s][hi] = ok ? __ldg(src + 32 * C::H64 + 2 * C::TAIL * c + 2 * s) : 0u;
        qa[4 * C::H64 + s][hi + 2] = ok ? __ldg(src + 32 * C::H64 + 2 * C::TAIL * c + 2 * s + 1) : 0u;
      }
    }
    auto pair = [&](uint32_t u) -> float2 {
      if (p.fp16) return __half22float2(*reinterpret_cast<__half2*>(&u));
      return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
    };
#pragma unroll
    for (int s = 0; s < C::KSTEPS; ++s) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f = pair(qa[s][x]);
        top[x & 1] = max(top[x & 1], max(__float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu));
      }
    }
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      top[hi] = max(top[hi], __shfl_xor_sync(0xffffffffu, top[hi], 1));
      top[hi] = max(top[hi], __shfl_xor_sync(0xffffffffu, top[hi], 2));
      const int E = max(int(top[hi] >> 23), 14);
      const float up = __uint_as_float(uint32_t(267 - E) << 23);   // largest element into [2^13, 2^14)
      qc[hi] = fmaxf(p.c * __uint_as_float(uint32_t(E - 13) << 23), 1e-38f);   // 2^(E - 140)
#pragma unroll
      for (int s = 0; s < C::KSTEPS; ++s) {
#pragma unroll
        for (int x = hi; x < 4; x += 2) {
          const float2 f = pair(qa[s][x]);
          qa[s][x] = f16x2(f.x * up, f.y * up);
        }
      }
    }
  }
  const int min_end = __reduce_min_sync(0xffffffffu, min(g < rows ? end[0] : 0x7FFFFFFF, g + 8 < rows ? end[1] : 0x7FFFFFFF));

  float o[C::CB][4];
#pragma unroll
  for (int j = 0; j < C::CB; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
  float shift[2] = {0.f, 0.f};
  int vref = 0;

  for (int i = 0; i < mine; ++i) {
    fetch(i + kNarStages - 1);
    cp_async_wait<kNarStages - 1>();
    __syncwarp();   // the exponents were copied by two lanes
    const uint8_t* stage = ring_ptr + (i % kNarStages) * C::STAGE_BYTES;
    const uint8_t* codes = stage + lane * 16;
    const int key0 = (warp + i * kNarWarps) * kNarKeys;
    // ---- S = Q K^T: two tiles of eight keys
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int h = 0; h < C::KSLOTS; ++h) {
        const uint4 u = *reinterpret_cast<const uint4*>(codes + (t * C::KSLOTS + h) * 512);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (4 * h + q < C::KSTEPS) mma_16816(s[t], qa[4 * h + q], e4m3_f16x2(x[q] & 0xFFFFu), e4m3_f16x2(x[q] >> 16));
      }
    }
    // ---- scales of keys 2 c, 2 c + 1 of both tiles
    const uint8_t* ex = stage + C::SLOTS * 512;
    const uint32_t k0e = *reinterpret_cast<const uint16_t*>(ex + 2 * c), k1e = *reinterpret_cast<const uint16_t*>(ex + 8 + 2 * c);
    const uint32_t v0e = *reinterpret_cast<const uint16_t*>(ex + 16 + 2 * c), v1e = *reinterpret_cast<const uint16_t*>(ex + 24 + 2 * c);
    const uint32_t ke[4] = {k0e & 0xFFu, k0e >> 8, k1e & 0xFFu, k1e >> 8};
    uint32_t ve[4] = {v0e & 0xFFu, v0e >> 8, v1e & 0xFFu, v1e >> 8};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float f = exp_scale(ke[x]);
      s[x >> 1][x & 1] *= f;
      s[x >> 1][(x & 1) + 2] *= f;
    }
    const bool full = key0 + kNarKeys <= min_end;
    if (!full) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int key = key0 + 8 * (x >> 1) + 2 * c + (x & 1);
        if (key >= end[0]) s[x >> 1][x & 1] = kNegInf;
        if (key >= end[1]) s[x >> 1][(x & 1) + 2] = kNegInf;
        if (key >= keys) ve[x] = 0;   // whatever the page holds there
      }
    }
    uint32_t vmax = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) vmax = max(vmax, ve[x] == 255u ? 0u : ve[x]);
    float top[2];
#pragma unroll
    for (int hi = 0; hi < 2; ++hi)
      top[hi] = fmaxf(fmaxf(s[0][2 * hi], s[0][2 * hi + 1]), fmaxf(s[1][2 * hi], s[1][2 * hi + 1])) * qc[hi];
    if (__any_sync(0xffffffffu, top[0] > m[0] + kNarSlack || top[1] > m[1] + kNarSlack || int(vmax) > vref)) {
      const int vnew = max(vref, int(__reduce_max_sync(0xffffffffu, vmax)));
      const int dv = vref - vnew;   // V references only grow
      const float sv = dv < -126 ? 0.f : __uint_as_float(uint32_t(127 + dv) << 23);
      vref = vnew;
      float so[2];
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        float t = top[hi];
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
        so[hi] = sv;
        if (t > m[hi] + kNarSlack) {
          const float f = ex2(m[hi] - t);   // 0 at the row's first visible keys
          l[hi] *= f;
          so[hi] *= f;
          m[hi] = t;
          shift[hi] = kNarLift - t;
        }
      }
#pragma unroll
      for (int j = 0; j < C::CB; ++j) {
        o[j][0] *= so[0];
        o[j][1] *= so[0];
        o[j][2] *= so[1];
        o[j][3] *= so[1];
      }
    }
    // ---- P, with V's scales relative to the reference
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int dv = int(ve[x]) - vref;   // <= 0 but for 255
      float f = dv < -126 ? 0.f : __uint_as_float(uint32_t(127 + dv) << 23);
      if (ve[x] == 255u) f = __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        float& e = s[x >> 1][(x & 1) + 2 * hi];
        const float pr = ex2(fmaf(e, qc[hi], shift[hi]));
        l[hi] += pr;
        const bool hidden = !full && key0 + 8 * (x >> 1) + 2 * c + (x & 1) >= end[hi];
        e = hidden ? 0.f : pr * f;   // not 0 * NaN
      }
    }
    const uint32_t pa[4] = {f16x2(s[0][0], s[0][1]), f16x2(s[0][2], s[0][3]), f16x2(s[1][0], s[1][1]),
                            f16x2(s[1][2], s[1][3])};
    // ---- O += P V: column tile j holds columns CB n + j, n = 0..7
    uint4 vr[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) vr[t] = *reinterpret_cast<const uint4*>(codes + (2 * C::KSLOTS + t) * 512);
#pragma unroll
    for (int q = 0; q < C::CB / 4; ++q) {
      const uint32_t a = (&vr[0].x)[q], b = (&vr[1].x)[q], d = (&vr[2].x)[q], e = (&vr[3].x)[q];
      const uint32_t lo01 = __byte_perm(a, b, 0x5140), lo89 = __byte_perm(d, e, 0x5140);
      const uint32_t hi01 = __byte_perm(a, b, 0x7362), hi89 = __byte_perm(d, e, 0x7362);
      mma_16816(o[4 * q], pa, e4m3_f16x2(lo01 & 0xFFFFu), e4m3_f16x2(lo89 & 0xFFFFu));
      mma_16816(o[4 * q + 1], pa, e4m3_f16x2(lo01 >> 16), e4m3_f16x2(lo89 >> 16));
      mma_16816(o[4 * q + 2], pa, e4m3_f16x2(hi01 & 0xFFFFu), e4m3_f16x2(hi89 & 0xFFFFu));
      mma_16816(o[4 * q + 3], pa, e4m3_f16x2(hi01 >> 16), e4m3_f16x2(hi89 >> 16));
    }
    __syncwarp();   // every lane has read the exponents of the stage that the next fetch fills
  }
  cp_async_wait<0>();

  // ---- the four warps' results
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    l[hi] += __shfl_xor_sync(0xffffffffu, l[hi], 1);
    l[hi] += __shfl_xor_sync(0xffffffffu, l[hi], 2);
  }
  float* s_m = reinterpret_cast<float*>(smem + C::OFF_ROWS);
  float* s_l = s_m + kNarWarps * 16;
  int* s_v = reinterpret_cast<int*>(s_l + kNarWarps * 16);
  if (c == 0) {
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      s_m[warp * 16 + g + 8 * hi] = m[hi];
      s_l[warp * 16 + g + 8 * hi] = l[hi];
    }
  }
  if (lane == 0) s_v[warp] = vref;
  __syncthreads();   // also: every warp is done with its ring
  int vtop = 8;
#pragma unroll
  for (int x = 0; x < kNarWarps; ++x) vtop = max(vtop, s_v[x]);
  float* s_o = reinterpret_cast<float*>(smem);   // [warp][16][D]
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int rr = g + 8 * hi;
    float top = kNegInf;
#pragma unroll
    for (int x = 0; x < kNarWarps; ++x) top = fmaxf(top, s_m[x * 16 + rr]);
    const int dv = vref - vtop;
    const float f = m[hi] == kNegInf || dv < -126 ? 0.f : ex2(m[hi] - top) * __uint_as_float(uint32_t(127 + dv) << 23);
    float* dst = s_o + (warp * 16 + rr) * D;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int col = C::CB * (2 * c + n);
      if (col < D) {
#pragma unroll
        for (int j = 0; j < C::CB; j += 4)
          *reinterpret_cast<float4*>(dst + col + j) =
              make_float4(o[j][2 * hi + n] * f, o[j + 1][2 * hi + n] * f, o[j + 2][2 * hi + n] * f, o[j + 3][2 * hi + n] * f);
      }
    }
  }
  __syncthreads();
  if (p.late_wait) pdl_wait();
  for (int x = threadIdx.x; x < rows * (D / 4); x += kNarThreads) {
    const int rr = x / (D / 4), col = 4 * (x - rr * (D / 4));
    float top = kNegInf, sum = 0.f;
#pragma unroll
    for (int y = 0; y < kNarWarps; ++y) top = fmaxf(top, s_m[y * 16 + rr]);
#pragma unroll
    for (int y = 0; y < kNarWarps; ++y)
      if (s_m[y * 16 + rr] != kNegInf) sum += s_l[y * 16 + rr] * ex2(s_m[y * 16 + rr] - top);
      else sum += s_l[y * 16 + rr];   // 0, or NaN from keys that are all NaN
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kNarWarps; ++y) {
      const float4 v = *reinterpret_cast<const float4*>(s_o + (y * 16 + rr) * D + col);
      acc.x += v.x;
      acc.y += v.y;
      acc.z += v.z;
      acc.w += v.w;
    }
    const int r = row0 + rr;
    const int64_t part = (int64_t(w.slot) * p.Tq + w.tok_first + r / p.G) * p.H + w.kvh * p.G + r % p.G;
    if (col == 0) p.part_lse[part] = sum == 0.f ? kNegInf : top + (log2f(sum) - kNarLift);
    if (sum != 0.f) {
      const float inv = 1.f / sum;
      const float vs = exp_scale(uint32_t(vtop));
      *reinterpret_cast<float4*>(p.part_o + part * D + col) =
          make_float4(acc.x * inv * vs, acc.y * inv * vs, acc.z * inv * vs, acc.w * inv * vs);
    }
  }
}

template <int D>
cudaError_t launch_narrow_t(const AttParams& p, int64_t units, cudaStream_t stream) {
  using C = NarCfg<D>;
  auto kern = attend_narrow_kernel<D>;
  static bool attr_set[128] = {};   // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) attr_set[dev] = true;
  }
  return launch_kernel(kern, dim3(unsigned(units)), kNarThreads, size_t(C::SMEM_BYTES), stream, 1, p);
}

}  // namespace

cudaError_t launch_attend_narrow(int head_dim, const AttParams& p, int64_t units, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_narrow_t<64>(p, units, stream);
    case 80: return launch_narrow_t<80>(p, units, stream);
    case 96: return launch_narrow_t<96>(p, units, stream);
    case 112: return launch_narrow_t<112>(p, units, stream);
    case 128: return launch_narrow_t<128>(p, units, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace tsel
