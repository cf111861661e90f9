// Attention over the cache for few query rows: one decoding step of a request
// (its query heads of one KV head) over its own suffix, or a small batch over
// the prefix. The wide kernel (attend.cu) turns every key into an operand of a
// 128-row product; with 16 rows or fewer that is nearly all waste, and reading
// the codes is what is left to bound the work.
//
// Same quantity and partial results as attend.cu. A CTA of four warps takes 8
// or 16 rows of one KV head and a chunk of keys; each warp walks every fourth
// block of 16 keys on its own, with its own running reference, sums and output,
// and the four are added up at the end.
//   - Codes come through cp.async, 16 bytes per lane, blocks ahead, into places
//     that the same lane reads back: shared memory only lengthens the prefetch
//     (4 KB a block and warp), no barrier is needed.
//   - Both products are mma.sync.m16n8k16 on fp16 with the keys (S^T = K Q^T) and
//     the head dimension (O^T = V^T P^T) on the 16 side and the rows on the 8
//     side, where eight rows waste nothing (tcgen05 has no M below 64). The
//     order of the head dimension inside S and of the columns inside O is free,
//     so each lane takes the elements of one 16-byte piece for its fragments
//     and converts them in registers: codes go from the cache to the tensor
//     cores without a transposition or a store. P turns from accumulator to
//     operand with one movmatrix per eight keys.
//   - A key's scales multiply S (K, together with the query's) and P (V, relative
//     to the largest exponent so far, so that P stays inside fp16: the product is
//     rounded to fp16, so it keeps eleven bits while probability times relative
//     scale is at least 2^-20 of the row's reference, and ends at 2^-30 of it).
// Bound by the latency of each warp's instructions (about 230 for a block of
// 4 KB) times the 16 warps that fit an SM's registers, before HBM: 64 requests
// with up to 4,000 keys on 8 KV heads of 128 (253 MB) take 62 us, 4.1 TB/s or
// 60% of the copy rate, with the schedulers issuing in 41% of the cycles; up to
// 1,000 keys 24 us. Five or six CTAs per SM with two stages cost spills (69, 86
// us); two stages with four CTAs are as fast as three; blocks of 32 keys, two
// products interleaved and three CTAs, are slower (65.6 against 63.9 us from a
// graph; 16 such requests 28.3 against 22.9).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend.cuh"
#include "imp_pass.cuh"

namespace tsel {

namespace {

constexpr int kNarWarps = 4;
constexpr int kNarThreads = 32 * kNarWarps;
constexpr int kNarStages = 3;
constexpr int kNarKeys = 16;         // keys of a block
constexpr float kNarLift = 6.f;      // P = 2^6 at the row's reference
constexpr float kNarSlack = 9.f;     // the reference may lag the row maximum by 2^9

// NB: groups of eight rows.
template <int D, int NB>
struct NarCfg {
  static constexpr int H64 = D / 64;               // whole 64-element parts of a row
  static constexpr int TAIL = (D % 64) / 16;       // 4-byte words per lane of the rest
  static constexpr int KSLOTS = H64 + (TAIL ? 1 : 0);
  static constexpr int KSTEPS = D / 16;            // k16 steps of S
  static constexpr int CB = D == 64 ? 8 : 16;      // V columns per lane (consecutive ones)
  static constexpr int SLOTS = 2 * KSLOTS + 4;     // 16-byte places per lane and stage
  static constexpr int STAGE_BYTES = SLOTS * 512 + 32;   // codes, then the 16 exponents of K and of V
  static constexpr int WARP_BYTES = kNarStages * STAGE_BYTES;
  static constexpr int ROWS = 8 * NB;
  static constexpr int OFF_ROWS = kNarWarps * WARP_BYTES;   // fp32 m, l [warp][ROWS], int vref [warp]
  static constexpr int SMEM_BYTES = OFF_ROWS + kNarWarps * (2 * ROWS + 4) * 4;
  static constexpr int CTAS = NB == 1 ? 4 : 3;     // per SM
  static_assert(kNarWarps * ROWS * D * 4 <= OFF_ROWS, "the outputs fit the ring");
  static_assert(CTAS * (SMEM_BYTES + 1024) <= 228 * 1024, "resident CTAs");
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

// Transposes an 8 x 8 matrix of 16-bit values held one word (two columns) per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D, int NB>
__global__ void __launch_bounds__(kNarThreads, NarCfg<D, NB>::CTAS) attend_narrow_kernel(const AttParams p) {
  using C = NarCfg<D, NB>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;   // fragment group and place in it
  pdl_wait();   // also where the launch before is of the same call: only this wait makes earlier kernels' writes visible here
  pdl_launch_dependents();
  const AttUnit w = att_unit<int64_t>(p, blockIdx.x, C::ROWS);
  const int row0 = w.group * C::ROWS;
  const int rows = w.bad ? 0 : min((w.tok_last - w.tok_first) * p.G - row0, C::ROWS);
  if (w.bad && threadIdx.x == 0) set_status(p.status, TSEL_DEV_SEQLENS);
  if (rows <= 0) return;
  const int keys = w.k1 - w.k0;
  if (keys <= 0) {   // no visible key in this chunk: an empty partial
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
  const bool v_in = C::CB * g < D;   // this lane has V columns
  const int k_at = g * D + 16 * c;                                  // key g, elements 16 c ..
  const int t_at = g * D + 64 * C::H64 + 4 * C::TAIL * c;           // ... of the rest of the row
  const int v_at = 2 * c * D + (v_in ? C::CB * g : 0);              // key 2 c, columns CB g ..
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
      const int64_t row = (int64_t(max(pg, 0)) * p.Hkv << p.page_shift) + head_row + ((w.k0 + key) & mask);
      const uint8_t* ks = p.k_pages + row * D;
      const uint8_t* vs = p.v_pages + row * D + v_at;
      const uint32_t stage = ring + (i % kNarStages) * C::STAGE_BYTES, dst = stage + lane * 16;
      const int left = pg >= 0 ? keys - key : 0;   // keys of the block inside the chunk
#pragma unroll
      for (int t = 0; t < 2; ++t) {   // keys 8 t + g
        const bool in = 8 * t + g < left;
#pragma unroll
        for (int h = 0; h < C::H64; ++h)
          cp_async16(dst + (t * C::KSLOTS + h) * 512, ks + k_at + 8 * t * D + 64 * h, in);
#pragma unroll
        for (int x = 0; x < C::TAIL; ++x)
          cp_async_small<4>(dst + (t * C::KSLOTS + C::H64) * 512 + 4 * x, ks + t_at + 8 * t * D + 4 * x, in);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {   // keys 2 c + {0, 1, 8, 9}
        const int j = (t & 1) + (t >> 1) * 8;
        const bool in = v_in && 2 * c + j < left;
        if (C::CB == 16) cp_async16(dst + (2 * C::KSLOTS + t) * 512, vs + j * D, in);
        else cp_async_small<8>(dst + (2 * C::KSLOTS + t) * 512, vs + j * D, in);
      }
      if (lane < 2) cp_async16(stage + C::SLOTS * 512 + 16 * lane, (lane == 0 ? p.k_exps : p.v_exps) + row, pg >= 0);
    }
    cp_async_commit();
  };

  uint32_t qb[NB][C::KSTEPS][2];   // Q rows 8 n + g as B fragments
  float qc[NB][2];                 // of the rows 8 n + 2 c + {0, 1}: scale to logits in base 2
  int end[NB][2];                  // ... and the keys of the chunk that they see
  int min_end = 0x7FFFFFFF;
  float o[NB][C::CB / 2][4];       // [column pair][{column 2 j, row 2 c}, {2 j, 2 c + 1}, {2 j + 1, ..}, ..]
  float m[NB][2], l[NB][2], shift[NB][2];
  int vref = 1;                    // exponent byte of the V reference,
  float vtop = __uint_as_float(1u << 23), vinv = __uint_as_float(253u << 23);   // 2^(vref - 127) and its inverse
#pragma unroll
  for (int n = 0; n < NB; ++n) {
#pragma unroll
    for (int j = 0; j < C::CB / 2; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      m[n][x] = kNegInf;
      l[n][x] = shift[n][x] = 0.f;
    }
  }

  // The first blocks are on their way while Q is loaded; one loop, so that
  // the fetching code is there once (a unit starts with cold instruction caches).
#pragma unroll 1
  for (int i = 1 - kNarStages; i < mine; ++i) {
    fetch(i + kNarStages - 1);
    if (i < 0) {
      if (i == -1) {
        // ---- Q, scaled to fp16 by a power of two of each row
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const int rr = 8 * n + g;
          const bool ok = rr < rows;
          const int r = row0 + (ok ? rr : 0);
          const uint32_t* src = reinterpret_cast<const uint32_t*>(
              static_cast<const uint16_t*>(p.q) + (w.tok_first + r / p.G) * p.q_stride +
              int64_t(w.kvh * p.G + r % p.G) * D);
#pragma unroll
          for (int s = 0; s < C::KSTEPS; ++s) {
            const int at = s < 4 * C::H64 ? 32 * (s / 4) + 8 * c + 2 * (s % 4)
                                          : 32 * C::H64 + 2 * C::TAIL * c + 2 * (s - 4 * C::H64);
            qb[n][s][0] = ok ? __ldg(src + at) : 0u;
            qb[n][s][1] = ok ? __ldg(src + at + 1) : 0u;
          }
          auto pair = [&](uint32_t u) -> float2 {
            if (p.fp16) return __half22float2(*reinterpret_cast<__half2*>(&u));
            return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
          };
          uint32_t top = 0;
#pragma unroll
          for (int s = 0; s < C::KSTEPS; ++s) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 f = pair(qb[n][s][x]);
              top = max(top, max(__float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu));
            }
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int E = max(int(top >> 23), 14);
          const float up = __uint_as_float(uint32_t(267 - E) << 23);   // largest element into [2^13, 2^14)
          const float mine_c = p.c * __uint_as_float(uint32_t(E - 13) << 23);   // 2^(E - 140)
#pragma unroll
          for (int s = 0; s < C::KSTEPS; ++s) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float2 f = pair(qb[n][s][x]);
              qb[n][s][x] = f16x2(f.x * up, f.y * up);
            }
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r2 = 8 * n + 2 * c + x;
            qc[n][x] = __shfl_sync(0xffffffffu, mine_c, 4 * (2 * c + x));
            const int lim = w.causal ? w.lim0 + (row0 + r2) / p.G : w.lim0;
            end[n][x] = r2 < rows ? min(lim, w.k1) - w.k0 : 0;
            if (r2 < rows) min_end = min(min_end, end[n][x]);
          }
        }
        min_end = __reduce_min_sync(0xffffffffu, min_end);
      }
      continue;
    }
    cp_async_wait<kNarStages - 1>();
    __syncwarp();   // the exponents were copied by two lanes
    const uint8_t* stage = ring_ptr + (i % kNarStages) * C::STAGE_BYTES;
    const uint8_t* codes = stage + lane * 16;
    const int key0 = (warp + i * kNarWarps) * kNarKeys;
    // ---- S^T = K Q^T: keys g and g + 8 of the block; even and odd steps apart,
    // which halves the dependent chain
    float s[NB][4], s1[NB][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      s1[n][0] = s1[n][1] = s1[n][2] = s1[n][3] = 0.f;
    }
#pragma unroll
    for (int h = 0; h < C::KSLOTS; ++h) {
      const uint4 u0 = *reinterpret_cast<const uint4*>(codes + h * 512);
      const uint4 u1 = *reinterpret_cast<const uint4*>(codes + (C::KSLOTS + h) * 512);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (4 * h + q >= C::KSTEPS) break;
        const uint32_t x = (&u0.x)[q], y = (&u1.x)[q];
        const uint32_t a[4] = {e4m3_f16x2(x & 0xFFFFu), e4m3_f16x2(y & 0xFFFFu), e4m3_f16x2(x >> 16), e4m3_f16x2(y >> 16)};
#pragma unroll
        for (int n = 0; n < NB; ++n) mma_16816(q & 1 ? s1[n] : s[n], a, qb[n][4 * h + q][0], qb[n][4 * h + q][1]);
      }
    }
    // ---- scales of keys g and g + 8: the byte is a float's exponent; 0 is the
    // denormal 2^-127, 255 makes NaN of the row whatever its codes. The two
    // scales of a logit are multiplied first: with either alone it can leave
    // fp32's range (large keys under small queries).
    const uint8_t* ex = stage + C::SLOTS * 512;
    auto scale = [](uint8_t e) -> float {
      return __uint_as_float(e == 255 ? 0x7FC00000u : max(uint32_t(e) << 23, 0x400000u));
    };
    const float kf[2] = {scale(ex[g]), scale(ex[8 + g])};
    float vf[2] = {scale(ex[16 + g]), scale(ex[24 + g])};
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int x = 0; x < 4; ++x) s[n][x] = (s[n][x] + s1[n][x]) * (kf[x >> 1] * qc[n][x & 1]);
    }
    const bool full = key0 + kNarKeys <= min_end;
    if (!full) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int key = key0 + 8 * x + g;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          if (key >= end[n][0]) s[n][2 * x] = kNegInf;
          if (key >= end[n][1]) s[n][2 * x + 1] = kNegInf;
        }
        if (key >= keys) vf[x] = 0.f;   // whatever the page holds there
      }
    }
    bool move = !(vf[0] <= vtop && vf[1] <= vtop);   // also for a NaN
    bool v_nan = false;   // the block has V rows of scale byte 255
    float top[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        top[n][x] = fmaxf(s[n][x], s[n][2 + x]);
        move = move || top[n][x] > m[n][x] + kNarSlack;
      }
    }
    if (__any_sync(0xffffffffu, move)) {
      v_nan = __any_sync(0xffffffffu, vf[0] != vf[0] || vf[1] != vf[1]);
      // the largest finite scale; V references only grow
      uint32_t ev = 0;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t b = __float_as_uint(vf[x]) >> 23;
        ev = max(ev, b == 255u ? 0u : b);
      }
      const int vnew = max(vref, int(__reduce_max_sync(0xffffffffu, ev)));
      const int dv = vref - vnew;
      const float sv = dv < -126 ? 0.f : __uint_as_float(uint32_t(127 + dv) << 23);
      vref = vnew;
      vtop = __uint_as_float(uint32_t(vnew) << 23);
      vinv = __uint_as_float(max(uint32_t(254 - vnew) << 23, 0x400000u));   // 2^-127 is a denormal
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        float so[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float t = top[n][x];
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
          t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
          so[x] = sv;
          if (t > m[n][x] + kNarSlack) {
            const float f = ex2(m[n][x] - t);   // 0 at the row's first visible keys
            l[n][x] *= f;
            so[x] *= f;
            m[n][x] = t;
            shift[n][x] = kNarLift - t;
          }
        }
#pragma unroll
        for (int j = 0; j < C::CB / 2; ++j) {
#pragma unroll
          for (int x = 0; x < 4; ++x) o[n][j][x] *= so[x & 1];
        }
      }
    }
    // ---- P, with V's scales relative to the reference, as B fragments
    const float vr[2] = {vf[0] * vinv, vf[1] * vinv};   // at most 1, or NaN
    uint32_t pb[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float e[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float pr = ex2(s[n][2 * x + y] + shift[n][y]);
          l[n][y] += pr;
          e[y] = pr * vr[x];
          if (!full && key0 + 8 * x + g >= end[n][y]) e[y] = 0.f;   // not 0 * NaN
        }
        pb[n][x] = transpose8(f16x2(e[0], e[1]));
      }
    }
    // ---- O^T += V^T P^T: tile j holds columns CB n + 2 j (row g) and CB n + 2 j + 1 (row g + 8)
    uint4 vr4[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) vr4[t] = *reinterpret_cast<const uint4*>(codes + (2 * C::KSLOTS + t) * 512);
    if (v_nan) {   // P holds the NaN of the rows that see them; their codes, which may be E4M3's NaN, reach no others
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (ex[16 + 2 * c + (t & 1) + 8 * (t >> 1)] == 255) vr4[t] = make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < C::CB / 4; ++q) {
      const uint32_t a = (&vr4[0].x)[q], b = (&vr4[1].x)[q], d = (&vr4[2].x)[q], e = (&vr4[3].x)[q];
      const uint32_t lo01 = __byte_perm(a, b, 0x5140), lo89 = __byte_perm(d, e, 0x5140);
      const uint32_t hi01 = __byte_perm(a, b, 0x7362), hi89 = __byte_perm(d, e, 0x7362);
      const uint32_t f0[4] = {e4m3_f16x2(lo01 & 0xFFFFu), e4m3_f16x2(lo01 >> 16), e4m3_f16x2(lo89 & 0xFFFFu), e4m3_f16x2(lo89 >> 16)};
      const uint32_t f1[4] = {e4m3_f16x2(hi01 & 0xFFFFu), e4m3_f16x2(hi01 >> 16), e4m3_f16x2(hi89 & 0xFFFFu), e4m3_f16x2(hi89 >> 16)};
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        mma_16816(o[n][2 * q], f0, pb[n][0], pb[n][1]);
        mma_16816(o[n][2 * q + 1], f1, pb[n][0], pb[n][1]);
      }
    }
    __syncwarp();   // every lane has read the exponents of the stage that the next fetch fills
  }
  cp_async_wait<0>();

  // ---- the four warps' results
  float* s_m = reinterpret_cast<float*>(smem + C::OFF_ROWS);
  float* s_l = s_m + kNarWarps * C::ROWS;
  int* s_v = reinterpret_cast<int*>(s_l + kNarWarps * C::ROWS);
#pragma unroll
  for (int n = 0; n < NB; ++n) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], 4);
      l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], 8);
      l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], 16);
      if (g == 0) {
        s_m[warp * C::ROWS + 8 * n + 2 * c + x] = m[n][x];
        s_l[warp * C::ROWS + 8 * n + 2 * c + x] = l[n][x];
      }
    }
  }
  if (lane == 0) s_v[warp] = vref;
  __syncthreads();   // also: every warp is done with its ring
  int vall = 1;
#pragma unroll
  for (int x = 0; x < kNarWarps; ++x) vall = max(vall, s_v[x]);
  float* s_o = reinterpret_cast<float*>(smem);   // [warp][row][D]
#pragma unroll
  for (int n = 0; n < NB; ++n) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int rr = 8 * n + 2 * c + x;
      float top = kNegInf;
#pragma unroll
      for (int y = 0; y < kNarWarps; ++y) top = fmaxf(top, s_m[y * C::ROWS + rr]);
      const int dv = vref - vall;
      const float f = m[n][x] == kNegInf || dv < -126 ? 0.f : ex2(m[n][x] - top) * __uint_as_float(uint32_t(127 + dv) << 23);
      float* dst = s_o + (warp * C::ROWS + rr) * D + C::CB * g;
      if (v_in && rr < rows) {
#pragma unroll
        for (int j = 0; j < C::CB / 2; j += 2)
          *reinterpret_cast<float4*>(dst + 2 * j) =
              make_float4(o[n][j][x] * f, o[n][j][2 + x] * f, o[n][j + 1][x] * f, o[n][j + 1][2 + x] * f);
      }
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < rows * (D / 4); x += kNarThreads) {
    const int rr = x / (D / 4), col = 4 * (x - rr * (D / 4));
    float top = kNegInf, sum = 0.f;
#pragma unroll
    for (int y = 0; y < kNarWarps; ++y) top = fmaxf(top, s_m[y * C::ROWS + rr]);
#pragma unroll
    for (int y = 0; y < kNarWarps; ++y) {
      const float my = s_m[y * C::ROWS + rr], ly = s_l[y * C::ROWS + rr];
      sum += my == kNegInf ? ly : ly * ex2(my - top);   // without a maximum: 0, or NaN from keys that are all NaN
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int y = 0; y < kNarWarps; ++y) {
      const float4 v = *reinterpret_cast<const float4*>(s_o + (y * C::ROWS + rr) * D + col);
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
      const float vs = __uint_as_float(uint32_t(vall) << 23);
      *reinterpret_cast<float4*>(p.part_o + part * D + col) =
          make_float4(acc.x * inv * vs, acc.y * inv * vs, acc.z * inv * vs, acc.w * inv * vs);
    }
  }
}

template <int D, int NB>
cudaError_t launch_narrow_t(const AttParams& p, int64_t units, cudaStream_t stream) {
  using C = NarCfg<D, NB>;
  auto kern = attend_narrow_kernel<D, NB>;
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

cudaError_t launch_attend_narrow(int head_dim, int row_groups, const AttParams& p, int64_t units,
                                 cudaStream_t stream) {
#define TSEL_NAR_CASE(DD)                                                \
  case DD:                                                               \
    return row_groups == 1 ? launch_narrow_t<DD, 1>(p, units, stream)    \
                           : launch_narrow_t<DD, 2>(p, units, stream);
  switch (head_dim) {
    TSEL_NAR_CASE(64)
    TSEL_NAR_CASE(80)
    TSEL_NAR_CASE(96)
    TSEL_NAR_CASE(112)
    TSEL_NAR_CASE(128)
    default:
      return cudaErrorInvalidValue;
  }
#undef TSEL_NAR_CASE
}

}  // namespace tsel
