// Attention of a batch of requests over a prefix that all of them share (the
// kept tokens of the images they ask about) and each one's own suffix, read
// from the quantised paged cache (kvcache.cu).
//
// o_i = sum_j p_ij v_j / sum_j p_ij with p_ij = exp(s q_i . k_j) over the
// prefix and the suffix keys that row i sees. LiteVLM review, "core formulas"
// (softmax(Q K^T / sqrt d) V); the pruned sequence in the KV cache: dynamic
// vision-token compression article, section 3.2.
//
// The prefix is read once for all rows, not once per request: the rows of every
// request and of the query heads that share a KV head form one matrix, cut into
// 128-row tiles. The keys are cut into chunks so that few rows still fill the
// device. A unit is (KV head, pair of row tiles, key chunk); a request's suffix
// is units of the same kind with its own rows. Each unit writes normalised
// partial results and their log-sum-exps, and a last launch joins a row's
// partials in a fixed order (deterministic: no atomics).
//
// A CTA has two pipelines that share the keys: each takes a row tile, or, where
// there is only one, they take the even and the odd key tiles of it. Per
// 128-key tile:
//   - eight converter warps load the E4M3 codes (16 bytes per lane, one tile
//     ahead in registers), turn them into fp16 — exact, with the row's
//     power-of-two scale relative to the tile's largest in one multiplication —
//     and store them to 128-byte-swizzled shared memory: K rows as the K-major B
//     operand of S = Q K^T, V rows as the MN-major B operand of O = P V.
//   - one warp per pipeline issues both products (tcgen05, kind::f16, fp32
//     accumulators in TMEM: two half tiles of 64 columns of S, 128 of O), the S
//     product of one half tile while the softmax is at the other. The whole warp
//     runs that code and one elected lane issues: with the loop inside a branch
//     on one lane, an instruction took 70 to 100 clocks, and the issuer, not the
//     tensor cores, set the pace (483 us for the question prefills below, 413 then).
//   - eight softmax warps per pipeline, two threads to a row, 32 columns each:
//     P = 2^(S c - m + 6) in fp16 lies over its S in TMEM and is the A operand of
//     the second product. The reference m may lag the row's maximum by 2^9; past
//     that (the two warps of a row vote) O is rescaled in TMEM, and then every
//     row of the warp follows, those that could still wait too (408 -> 387 us).
// fp16 throughout: q rows are scaled by a power of two so that their largest
// element is in [2^13, 2^14) (bf16's eight bits fit; elements below 2^-27 of the
// largest lose bits), codes have four bits, and P keeps eleven bits down to
// 2^-20 of the reference and ends at 2^-30. V keeps its codes exactly while a
// row's scale is within 2^-20 of the largest scale so far in its chunk, K while
// within 2^-22 of its tile's largest; smaller rows are rounded on that grid.
//
// What bounds it: per 256 x 128 logits the tensor cores need about 2,050 clocks
// and the instructions (8,000 of the warps, half of them the exponentials and
// what feeds them) 2,000 of each scheduler; a pass takes about 4,600, the rest
// is the chain S product, softmax, O product of each pipeline: P lies over its S,
// so the next S product into those columns waits for the O product that reads
// them. (P takes half the columns of its S; one S and two compact P would fit and
// free the S product of that wait. Not built.) Schedulers issue in 66% of the
// cycles, the tensor pipe is busy in 45%. 16 question prefills of up to 142 tokens
// over 36,831 keys (16 heads on 8 of 128): 366 us of 390 with the join, 0.94
// PFLOP/s, 49% of cuBLAS's bf16 rate; 256 rows over the same keys (a step of 64
// users): 47 us of 79.
// Tried and slower: one row per thread with more registers (setmaxnreg; 515 us),
// P in shared memory (472 to 534), one pipeline with two whole S tiles (535: each
// key tile is then converted for 128 rows instead of 256), whole key tiles
// instead of halves (409), rescaling 16 columns of O at a time (458: spills).
//
// Masked keys never reach a result: V rows past the last visible key of a tile
// are zeros whatever the page holds, S of masked keys is replaced, not added
// to, and a row stored as NaN (scale byte 255) enters through S (K) or P (V) of
// the rows that see it only. Not looked for: a NaN code under another byte in a
// V row that later rows of the same unit see (0 times NaN in the second
// product). The cache write leaves none, and a test of every code would lengthen
// every conversion.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend.cuh"
#include "attend_ops.cuh"
#include "imp_pass.cuh"

namespace tsel {

namespace {

// The converters write a tile's entry before they wait for its stage. While a
// pipeline of a split unit is at tile t, its tile t + 2 is converted but not
// multiplied yet, the other pipeline's t + 3 may be, and t + 4 is entered: five.
constexpr int kAttMetaRing = 8;
constexpr float kAttLift = 6.f;       // P = 2^6 at the row's reference
constexpr float kAttSlack = 9.f;      // the reference may lag the row maximum by 2^9
constexpr int kAttVSlack = 2;         // a moved V reference leaves room for 2^2 larger scales

struct AttTileMeta {
  float k_scale;       // 2^(tile's K reference - 7)
  int v_ref;           // exponent byte of the V reference
  uint32_t v_nan[4];   // keys whose V row is NaN, a bit each
};

template <int D, bool TREE>
struct AttCfg {
  static constexpr int DC = D > 64 ? 2 : 1;                 // 64-element chunks of a row
  static constexpr int TILE_BYTES = DC * kTile * 128;       // one 128-row fp16 operand
  static constexpr int KS = 2;                              // K and V stages
  static constexpr int SOFT_PER_TILE = 8;                   // softmax warps of a row tile: two threads per row
  static constexpr int SOFT_WARPS = 2 * SOFT_PER_TILE;
  static constexpr int MMA_WARP = SOFT_WARPS;               // one issuing thread for each pipeline
  static constexpr int CONV_WARP = MMA_WARP + 2;            // four warps for K, four for V
  static constexpr int WARPS = CONV_WARP + 8;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * TILE_BYTES;
  static constexpr int OFF_V = OFF_K + KS * TILE_BYTES;
  static constexpr int OFF_FAC = OFF_V + KS * TILE_BYTES;   // uint32 [K, V][tile parity][128]
  static constexpr int OFF_PAGES = OFF_FAC + 2 * 2 * kTile * 4;
  static constexpr int OFF_ROW = OFF_PAGES + kAttMaxPages * 4;   // fp32 [row tile][parity][half][128]
  static constexpr int OFF_TREE = OFF_ROW + 2 * 2 * 2 * kTile * 4;   // uint64 [row tile][128]: ancestors
  static constexpr int OFF_META = OFF_TREE + (TREE ? 2 * kTile * 8 : 0);
  static constexpr int NUM_BARS = 4 * KS + 3 * 4;
  static constexpr int OFF_BAR = OFF_META + kAttMetaRing * int(sizeof(AttTileMeta));
  static constexpr int OFF_MISC = OFF_BAR + 8 * NUM_BARS;
  static constexpr int OFF_UNIT = OFF_MISC + 16;            // what the epilogue needs of the unit
  static constexpr int SMEM_USED = OFF_MISC + 64 + 1024;    // + alignment slack
  // one CTA per SM (it holds all of TMEM), also for the smaller heads
  static constexpr int SMEM_BYTES = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static constexpr int STEPS = 4 * DC;                      // 16-code pieces per converter thread and tile
  static_assert(sizeof(AttTileMeta) % 8 == 0 && OFF_META % 8 == 0, "barrier alignment");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// Keeps the compiler from computing x again where it is used.
__device__ __forceinline__ void opaque(int& x) { asm volatile("" : "+r"(x)); }

// Two E4M3 codes times a power of two, as fp16.
__device__ __forceinline__ uint32_t unpack_e4m3(uint32_t two, uint32_t factor) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\t"
      "cvt.rn.f16x2.e4m3x2 t, %1;\n\t"
      "mul.rn.f16x2 %0, t, %2;\n\t}"
      : "=r"(r)
      : "h"(uint16_t(two)), "r"(factor));
  return r;
}

// 2^(7 + exp - ref) in both fp16 halves (exp <= ref): codes of the largest
// row reach 448 * 2^7.
__device__ __forceinline__ uint32_t att_factor(int exp, int ref) {
  const int n = 7 + exp - ref;
  const uint32_t f = n >= -14 ? uint32_t(n + 15) << 10 : (n >= -24 ? 1u << (n + 24) : 0u);
  return f | (f << 16);
}

// Largest of four exponent bytes that are not 255.
__device__ __forceinline__ uint32_t max_byte(uint32_t w) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = (w >> (8 * i)) & 0xFFu;
    m = max(m, b == 255u ? 0u : b);
  }
  return m;
}

// exp2(S * c + shift) of 32 columns, added up in acc and packed to fp16.
__device__ __forceinline__ void att_exp32(const uint32_t (&r)[32], float2 c2, float2 s2, float2& acc,
                                          uint32_t (&h)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 a =
        __ffma2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), c2, s2);
    const float2 e = make_float2(ex2(a.x), ex2(a.y));
    acc = __fadd2_rn(acc, e);
    h[j] = pack_f16(e.x, e.y);
  }
}

// Puts NaN into the visible columns of P whose V row is NaN.
__device__ __forceinline__ void att_poison32(uint32_t (&h)[16], uint32_t nan, int vis) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    if (((nan >> (2 * j)) & 1u) && 2 * j < vis) h[j] = (h[j] & 0xFFFF0000u) | 0x7E00u;
    if (((nan >> (2 * j + 1)) & 1u) && 2 * j + 1 < vis) h[j] = (h[j] & 0xFFFFu) | 0x7E000000u;
  }
}

// The columns of 32 that a row sees where the tree's keys begin at column -s:
// all of those before it, then its ancestors.
__device__ __forceinline__ uint32_t att_seen32(uint64_t tree, int s) {
  if (s >= 64) return 0u;
  if (s >= 0) return uint32_t(tree >> s);
  return s <= -32 ? 0xFFFFFFFFu : uint32_t(tree << -s) | ((1u << -s) - 1u);
}

// TREE: rows of a suffix are nodes of trees.
template <int D, bool TREE>
__global__ void __launch_bounds__(AttCfg<D, TREE>::THREADS, 1) attend_kernel(const AttParams p) {
  using C = AttCfg<D, TREE>;
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = smem_dyn + ((1024u - (smem_u32(smem_dyn) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_full = bars;                  // [KS] K tile converted
  uint64_t* k_free = k_full + C::KS;        // [KS] S products of the tile done
  uint64_t* v_full = k_free + C::KS;        // [KS]
  uint64_t* v_free = v_full + C::KS;        // [KS]
  uint64_t* s_full = v_free + C::KS;        // [pipeline][half tile] S in TMEM
  uint64_t* p_full = s_full + 4;            // P in TMEM
  uint64_t* o_done = p_full + 4;            // O product done
  int32_t* s_pages = reinterpret_cast<int32_t*>(smem + C::OFF_PAGES);
  AttTileMeta* s_meta = reinterpret_cast<AttTileMeta*>(smem + C::OFF_META);
  uint32_t* s_fac = reinterpret_cast<uint32_t*>(smem + C::OFF_FAC);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t T = p.timeout_ns;
  // Before the wait for the earlier kernels: what does not touch their memory.
  // (TMEM may still be held by a CTA of an earlier kernel; none of them waits
  // for this one.)
  if (warp == C::MMA_WARP) {
    if (lane == 0) {
      for (int i = 0; i < C::KS; ++i) {
        mbar_init(&k_full[i], 4);
        mbar_init(&k_free[i], 2);
        mbar_init(&v_full[i], 4);
        mbar_init(&v_free[i], 2);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&p_full[i], C::SOFT_PER_TILE);
        mbar_init(&o_done[i], 1);
      }
      *abort_flag = 0;
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  pdl_wait();   // every input may come from an earlier kernel
  const AttUnit w = att_unit<uint32_t>(p, blockIdx.x, 2 * p.tt * p.G);
  const int tok0 = w.tok_first + w.group * 2 * p.tt;          // of row tile 0
  const int tok_end = min(w.tok_last, tok0 + 2 * p.tt);
  const int tiles = int(ceil_div(w.k1 - w.k0, kTile));
  // Two pipelines x = 0, 1 keep the tensor cores and the softmax warps busy in
  // turn: with two row tiles each takes one and walks every key tile; with one
  // row tile (split) they take the even and the odd key tiles, and their
  // results are two partials.
  const bool split = tok0 + p.tt >= tok_end;
  const int n0 = split ? (tiles + 1) >> 1 : tiles, n1 = split ? tiles >> 1 : tiles;

  // Softmax warps: pipeline x, row (TMEM lane) 32 * (warp % 4) + lane, the 64
  // columns of `half`.
  const int x = (warp >> 3) & 1;
  const int half = (warp >> 2) & 1;
  const int row = int(threadIdx.x) & (kTile - 1);
  const int tok = tok0 + (split ? 0 : x * p.tt) + row / p.G;
  const int head = w.kvh * p.G + row % p.G;
  const bool row_ok = warp < C::SOFT_WARPS && row < p.tt * p.G && tok < tok_end;
  // A row's partial is in slot w.slot; the second pipeline of a split unit has
  // the next one, which is empty otherwise.
  if (row_ok && half == 0) {
    const int64_t next = int64_t(p.Tq) * p.H;
    const int64_t part = (int64_t(w.slot + (split ? x : 0)) * p.Tq + tok) * p.H + head;
    if (!split) p.part_lse[part + next] = kNegInf;
    if ((x == 0 ? n0 : n1) == 0) p.part_lse[part] = kNegInf;
  }
  if (w.bad || tok0 >= tok_end || tiles == 0) {   // bad lengths, no rows, or no visible key in this chunk
    if (w.bad && threadIdx.x == 0) set_status(p.status, TSEL_DEV_SEQLENS);
    __syncthreads();
    pdl_launch_dependents();
    if (warp == C::MMA_WARP) {
      tc_fence_after();
      tmem_dealloc(*tmem_slot, 512);
    }
    return;
  }

  // The converters fetch the chunk's pages (one out of range is read as zeros)
  // and their first tile while the others load Q.
  const int first_page = w.k0 >> p.page_shift;
  if (warp >= C::CONV_WARP) {
    const int n = ((w.k1 - 1) >> p.page_shift) - first_page + 1;
    for (int i = int(threadIdx.x) - 32 * C::CONV_WARP; i < n; i += 32 * 8) {
      const int pg = __ldg(w.pages + first_page + i);
      const bool ok = pg >= 0 && pg < p.num_pages;
      if (!ok) set_status(p.status, TSEL_DEV_PAGES);
      s_pages[i] = ok ? pg : -1;
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
  }
  // Q rows, scaled to fp16, into the K-major A operand (a split unit's rows
  // twice). A warp loads half the columns of its 32 rows, eight lanes to a row;
  // the two warps of a row exchange its largest element.
  float qc = 0.f;   // softmax_scale * log2(e) * 2^(row's exponent)
  float* s_row = reinterpret_cast<float*>(smem + C::OFF_ROW) + x * 4 * kTile;
  if (warp < C::SOFT_WARPS) {
    constexpr int UH = D / 16;   // 16-byte pieces of half a row
    const int unit = lane & 7, quad = 32 * (warp & 3);
    uint4 qv[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = quad + 4 * k + (lane >> 3);
      const int t = tok0 + (split ? 0 : x * p.tt) + r / p.G;
      const bool in = unit < UH && r < p.tt * p.G && t < tok_end;
      qv[k] = in ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + t * p.q_stride +
                                                        int64_t(w.kvh * p.G + r % p.G) * D) + half * UH + unit)
                 : make_uint4(0, 0, 0, 0);
    }
    // magnitudes order like their bits, in both types
    uint32_t* row_top = reinterpret_cast<uint32_t*>(s_row);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t m2 = __vmaxu2(__vmaxu2(qv[k].x & 0x7FFF7FFFu, qv[k].y & 0x7FFF7FFFu),
                             __vmaxu2(qv[k].z & 0x7FFF7FFFu, qv[k].w & 0x7FFF7FFFu));
      uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
      if (unit == 0) row_top[half * kTile + quad + 4 * k + (lane >> 3)] = top;
    }
    asm volatile("bar.sync %0, 64;" ::"r"(3 + x * 4 + (warp & 3)) : "memory");
    // fp32 exponent field of a row's largest element, at least 14
    auto row_exp = [&](int r) -> int {
      const uint32_t top = max(row_top[r], row_top[kTile + r]);
      const uint32_t f = p.fp16 ? __float_as_uint(__half2float(__ushort_as_half(uint16_t(top)))) : top << 16;
      return max(int(f >> 23), 14);
    };
    uint8_t* sq = smem + C::OFF_Q + x * C::TILE_BYTES;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = quad + 4 * k + (lane >> 3), j = half * UH + unit;
      const float up = __uint_as_float(uint32_t(267 - row_exp(r)) << 23);   // largest element into [2^13, 2^14)
      const uint32_t u[4] = {qv[k].x, qv[k].y, qv[k].z, qv[k].w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = p.fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&u[i]))
                                : make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
        h[i] = pack_f16(f.x * up, f.y * up);
      }
      if (unit < UH)
        *reinterpret_cast<uint4*>(sq + (j >> 3) * (kTile * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4)) =
            make_uint4(h[0], h[1], h[2], h[3]);
    }
    qc = p.c * __uint_as_float(uint32_t(row_exp(row) - 13) << 23);   // 2^(E - 140)
    if (TREE && w.causal) {
      const AttAncestors a = att_ancestors(p.parents + w.tok_first, w.tok_last - w.tok_first, p.status);
      const uint64_t bits = att_bits(a, row_ok ? tok - w.tok_first : 0);
      if (half == 0) reinterpret_cast<uint64_t*>(smem + C::OFF_TREE)[x * kTile + row] = row_ok ? bits : 0;
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    int32_t* s_unit = reinterpret_cast<int32_t*>(smem + C::OFF_UNIT);
    s_unit[0] = w.slot;
    s_unit[1] = tok0;
    s_unit[2] = tok_end;
    s_unit[3] = w.kvh;
    s_unit[4] = split ? 1 : 0;
  }
  // Barriers initialised, TMEM allocated, Q in shared memory.
  auto set_up = [&]() {
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
  };

  if (warp < C::SOFT_WARPS) {
    set_up();
    const uint32_t tmem = *tmem_slot;
    // ------------------------------------------------------------ softmax
    const int n = x == 0 ? n0 : n1;
    if (n > 0) {
      const uint32_t lanes = uint32_t((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + lanes + uint32_t(x * 256);   // O: 128 columns on
      const bool any_row = __any_sync(0xffffffffu, row_ok);
      // in a tree: where its keys begin
      const int lim = TREE ? w.lim0 - w.causal : (w.causal ? w.lim0 + (tok - w.tok_first) : w.lim0);
      int end = (row_ok ? min(lim, w.k1) : 0) - w.k0;
      int min_end = int(__reduce_min_sync(0xffffffffu, row_ok ? max(end, 0) : 0x7FFFFFFF));   // of the warp's rows
      // What the loop needs of the row is computed here, once: left alone, the
      // compiler saves registers by dividing rows into tokens again for every tile.
      int keys = w.k1 - w.k0;
      if (TREE) opaque(keys);
      opaque(end);
      opaque(min_end);
      // the two warps of the same 32 rows meet at a barrier of their own
      const int pair_bar = 3 + x * 4 + (warp & 3);
      auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair_bar) : "memory"); };
      auto meet_any = [&](bool mine) -> bool {
        uint32_t any;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.u32 p, %1, 0;\n\t"
            "bar.red.or.pred q, %2, 64, p;\n\t"
            "selp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(any)
            : "r"(uint32_t(mine)), "r"(pair_bar)
            : "memory");
        return any != 0;
      };
      float m = kNegInf, l = 0.f;
      int vref = 0;
      bool ok = true;
#pragma unroll 1
      for (int j = 0; j < 2 * n; ++j) {   // half tiles
        const int i = j >> 1, hh = j & 1, t = split ? 2 * i + x : i;   // key tile
        if (!warp_wait(&s_full[2 * x + hh], uint32_t(i & 1), abort_flag, T)) {
          // the loop goes on (the warps of a row meet in it), its waits return at once
          ok = false;
          if (lane == 0) *abort_flag = 1;
        }
        if (any_row) {
          tc_fence_after();
          const AttTileMeta& meta = s_meta[t & (kAttMetaRing - 1)];
          const int col = 64 * hh + 32 * half;        // first of this thread's columns of the tile
          int vis = end - t * kTile - col;            // visible ones: [0, vis)
          const bool full = t * kTile + col + 32 <= min_end;
          uint32_t r[32];
          tmem_ld32_async(s_at + col, r);
          const float ct = fmaxf(qc * meta.k_scale, 1e-38f);
          const int vnew = meta.v_ref;
          uint32_t nan_v = meta.v_nan[2 * hh + half];
          tmem_wait_ld(r);
          if (TREE && !full && w.causal) {
            const int last = keys - t * kTile - col;   // columns of the chunk
            const uint32_t seen = att_seen32(reinterpret_cast<const uint64_t*>(smem + C::OFF_TREE)[x * kTile + row], -vis) &
                                  (last >= 32 ? 0xFFFFFFFFu : last <= 0 ? 0u : (1u << last) - 1u);
#pragma unroll
            for (int k = 0; k < 32; ++k) r[k] = (seen >> k) & 1u ? r[k] : __float_as_uint(kNegInf);
            nan_v &= seen;
            vis = 32;
          } else if (!full) {
            mask_cols(r, vis);
          }
          float top = cols_max(r) * ct;
          // the two warps of the same rows go the same way
          if (meet_any(top > m + kAttSlack || vnew != vref)) {
            float* mx = s_row + (j & 1) * 2 * kTile;
            mx[half * kTile + row] = top;
            meet();
            top = fmaxf(top, mx[(half ^ 1) * kTile + row]);
            float s = 1.f;
            if (top > m) {   // also the rows that could still wait: once here, it costs nothing
              s = ex2(m - top);   // 0 at the row's first visible keys
              l *= s;
              m = top;
            }
            // V references only grow: 2^(old - new), 0 below 2^-126
            const int dv = vref - vnew;
            s *= dv < -126 ? 0.f : __uint_as_float(uint32_t(127 + dv) << 23);
            vref = vnew;
            if (j > 0) {   // once the O product of the half tile before is complete
              if (!warp_wait(&o_done[2 * x + (hh ^ 1)], uint32_t(((j - 1) >> 1) & 1), abort_flag, T)) {
                ok = false;
                if (lane == 0) *abort_flag = 1;
              }
              tc_fence_after();
#pragma unroll 1
              for (int cc = half * (D / 16); cc < (half + 1) * (D / 16); ++cc) {
                uint32_t o[8];
                tmem_ld8(s_at + 128 + cc * 8, o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * s);
                tmem_st8(s_at + 128 + cc * 8, o);
              }
            }
          }
          const float shift = m == kNegInf ? 0.f : kAttLift - m;
          float2 acc = make_float2(0.f, 0.f);
          uint32_t h[16];
          att_exp32(r, make_float2(ct, ct), make_float2(shift, shift), acc, h);
          if (nan_v) att_poison32(h, nan_v, vis);
          tmem_st16(s_at + col, h);   // over the first of these columns
          l += acc.x + acc.y;
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        mbar_arrive_lane0(&p_full[2 * x + hh], lane);
      }
      if (ok) ok = warp_wait(&o_done[2 * x + 1], uint32_t((n - 1) & 1), abort_flag, T);
      if (!ok && lane == 0) {
        *abort_flag = 1;
        set_status(p.status, TSEL_DEV_TIMEOUT);
      }
      if (any_row) {
        float* sum = s_row;   // the places that the last half tile did not use
        sum[half * kTile + row] = l;
        meet();
        l = half == 0 ? l + sum[kTile + row] : sum[row] + l;
        if (ok) {
          tc_fence_after();
          const int32_t* s_unit = reinterpret_cast<const int32_t*>(smem + C::OFF_UNIT);
          const int tok = s_unit[1] + (s_unit[4] ? 0 : x * p.tt) + row / p.G;
          const bool row_ok = row < p.tt * p.G && tok < s_unit[2];
          const int64_t part = (int64_t(s_unit[0] + (s_unit[4] ? x : 0)) * p.Tq + tok) * p.H + s_unit[3] * p.G + row % p.G;
          if (row_ok && half == 0) p.part_lse[part] = l == 0.f ? kNegInf : m + (log2f(l) - kAttLift);
          // O' * 2^(vref - 134) / l', both with the same lift; -1: not written
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const float vs = __uint_as_float(uint32_t(vref - 7) << 23);
          const int64_t at = row_ok && l != 0.f ? part * D + half * (D / 2) : -1;
          // 32 columns at a time through shared memory (4 KB of Q's, which is
          // done with), so that eight lanes store 128 bytes of a row
          uint8_t* buf = smem + C::OFF_Q + x * C::TILE_BYTES + (warp & 7) * (C::TILE_BYTES / 8 < 4096 ? C::TILE_BYTES / 8 : 4096);
          constexpr int UNITS = C::TILE_BYTES / 8 < 4096 ? 4 : 8;   // 16-byte pieces of a row at a time
#pragma unroll 1
          for (int c0 = 0; c0 < D / 2; c0 += 4 * UNITS) {
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < UNITS / 2; ++i) {
              if (c0 + 8 * i < D / 2) {
                tmem_ld8(s_at + 128 + half * (D / 2) + c0 + 8 * i, o);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  *reinterpret_cast<float4*>(buf + (row & 31) * (16 * UNITS) + (((2 * i + j) ^ (row & (UNITS - 1))) << 4)) =
                      make_float4(__uint_as_float(o[4 * j]) * inv * vs, __uint_as_float(o[4 * j + 1]) * inv * vs,
                                  __uint_as_float(o[4 * j + 2]) * inv * vs, __uint_as_float(o[4 * j + 3]) * inv * vs);
              }
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < UNITS; ++k) {
              const int idx = 32 * k + lane, r = idx / UNITS, u = idx % UNITS;
              const int64_t dst = __shfl_sync(0xffffffffu, at, r);
              if (dst >= 0 && c0 + 4 * u < D / 2)
                *reinterpret_cast<float4*>(p.part_o + dst + c0 + 4 * u) =
                    *reinterpret_cast<const float4*>(buf + r * (16 * UNITS) + ((u ^ (r & (UNITS - 1))) << 4));
            }
            __syncwarp();
          }
        }
      }
    }
  } else if (warp < C::CONV_WARP) {
    // ------------------------------------------------------------ MMA issuer
    // A thread for each pipeline. S has room for two half tiles of 64 keys: the
    // product of one runs while the softmax warps are at the other, so they
    // only wait for the tensor cores when those are behind. P lies over its S,
    // so the O product must have read it before the next S product is issued.
    // Both pipelines read a stage before it is free; where one reads it alone
    // it stands for both.
    set_up();
    const int xx = __shfl_sync(0xffffffffu, warp, 0) - C::MMA_WARP, n = xx == 0 ? n0 : n1;
    if (n > 0) {
      constexpr uint32_t kIdS = idesc_f16_f32(kTile, 64, false);
      constexpr uint32_t kIdO = idesc_f16_f32(kTile, D, true);
      const uint32_t ts = __shfl_sync(0xffffffffu, *tmem_slot, 0) + uint32_t(xx * 256);
      // advanced by (bytes >> 4)
      const uint64_t dq = smem_desc(smem_u32(smem + C::OFF_Q) + xx * C::TILE_BYTES, 2, 1024);
      const uint64_t dk = smem_desc(smem_u32(smem + C::OFF_K), 2, 1024);
      const uint64_t dv = smem_desc_mn(smem_u32(smem + C::OFF_V), kTile * 128, 1024);
      auto s_product = [&](int j) -> bool {
        const int i = j >> 1, hh = j & 1, t = split ? 2 * i + xx : i, st = t % C::KS;
        if (!warp_wait(&k_full[st], uint32_t((t / C::KS) & 1), abort_flag, T) ||
            (i > 0 && !warp_wait(&o_done[2 * xx + hh], uint32_t((i - 1) & 1), abort_flag, T)))
          return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * (kTile * 128) + (kk & 3) * 32;
          mma_ss_elect(ts + 64 * hh, dq + (off >> 4), dk + ((st * C::TILE_BYTES + hh * 8192 + off) >> 4), kIdS, kk > 0);
        }
        commit_elect(&s_full[2 * xx + hh]);
        if (hh == 1) {
          commit_elect(&k_free[st]);
          if (split) commit_elect(&k_free[st]);
        }
        return true;
      };
      bool ok = s_product(0) && s_product(1);
      int done = 0;   // O products issued
#pragma unroll 2
      for (int j = 0; j < 2 * n && ok; ++j) {
        const int i = j >> 1, hh = j & 1, t = split ? 2 * i + xx : i, st = t % C::KS;
        ok = warp_wait(&v_full[st], uint32_t((t / C::KS) & 1), abort_flag, T) &&
             warp_wait(&p_full[2 * xx + hh], uint32_t(i & 1), abort_flag, T);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts_elect(ts + 128, ts + 64 * hh + (kk >> 1) * 32 + (kk & 1) * 8,
                     dv + ((st * C::TILE_BYTES + (4 * hh + kk) * 2048) >> 4), kIdO, j > 0 || kk > 0);
        commit_elect(&o_done[2 * xx + hh]);
        if (hh == 1) {
          commit_elect(&v_free[st]);
          if (split) commit_elect(&v_free[st]);
        }
        done = j + 1;
        if (j + 2 < 2 * n) ok = s_product(j + 2);
      }
      // every MMA this thread issued has completed before TMEM is freed
      if (done > 0) wait_drain(&o_done[2 * xx + ((done - 1) & 1)], uint32_t(((done - 1) >> 1) & 1), T);
      if (!ok) {
        *abort_flag = 1;
        set_status(p.status, TSEL_DEV_TIMEOUT);
        commit_elect(&o_done[2 * xx + (done & 1)]);   // one more phase, for an S product in flight
        wait_drain(&o_done[2 * xx + (done & 1)], uint32_t((done >> 1) & 1), T);
      }
    }
  } else {
    // ------------------------------------------------------------ converters
    const bool do_k = warp < C::CONV_WARP + 4;   // four warps for K, four for V
    const int tid = (int(threadIdx.x) - 32 * C::CONV_WARP) & (kTile - 1);
    const int mask = (1 << p.page_shift) - 1;
    const int keys = w.k1 - w.k0;
    uint32_t* fac_k = s_fac;
    uint32_t* fac_v = s_fac + 2 * kTile;
    // Step i of a thread: row 32 * (i % 4) + tid / 4, piece tid % 4 of chunk
    // i / 4. Four lanes read 64 contiguous bytes of a row; eight lanes store
    // to two neighbouring rows, whose swizzles differ in the lowest bit, so
    // the 16-byte halves of their pieces cover all 32 banks.
    const int r0 = tid >> 2, c0 = tid & 3, sw = r0 & 7;
    const uint8_t* pages = (do_k ? p.k_pages : p.v_pages) + (int64_t(w.kvh) << p.page_shift) * D + 16 * c0;
    const uint32_t page_bytes = uint32_t(p.Hkv << p.page_shift) * uint32_t(D);
    uint4 raw[C::STEPS];   // a tile's codes, loaded one tile ahead
    auto load = [&](int t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = t * kTile + 32 * i + r0;
        const int pg = j < keys ? s_pages[((w.k0 + j) >> p.page_shift) - first_page] : -1;
        const uint8_t* src = pages + uint64_t(uint32_t(pg)) * page_bytes + ((w.k0 + j) & mask) * D;
#pragma unroll
        for (int cc = 0; cc < C::DC; ++cc)
          raw[4 * cc + i] = pg >= 0 && 64 * cc + 16 * c0 < D
                                ? __ldg(reinterpret_cast<const uint4*>(src + 64 * cc))
                                : make_uint4(0, 0, 0, 0);
      }
    };
    // exponent bytes of keys 4 * lane .. + 3 of a tile (0 past the end)
    auto load_exps = [&](int t, const uint8_t* exps) -> uint32_t {
      const int j = t * kTile + 4 * lane;
      const int pg = j < keys ? s_pages[((w.k0 + j) >> p.page_shift) - first_page] : -1;
      if (pg < 0) return 0;
      const int64_t r = ((int64_t(pg) * p.Hkv + w.kvh) << p.page_shift) + ((w.k0 + j) & mask);
      const uint32_t e = __ldg(reinterpret_cast<const uint32_t*>(exps + r));
      const int left = keys - j;   // keys of the four inside the chunk
      return left >= 4 ? e : e & ((1u << (8 * left)) - 1u);
    };
    auto convert = [&](uint8_t* tile, const uint32_t* fac) {
      uint8_t* lo_at = tile + r0 * 128 + (((2 * c0) ^ sw) << 4);
      uint8_t* hi_at = tile + r0 * 128 + (((2 * c0 + 1) ^ sw) << 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t f = fac[32 * i + r0];
#pragma unroll
        for (int cc = 0; cc < C::DC; ++cc) {
          const uint4 u = raw[4 * cc + i];
          if (64 * cc + 16 * c0 < D) {
            const int at = cc * (kTile * 128) + i * (32 * 128);
            *reinterpret_cast<uint4*>(lo_at + at) =
                make_uint4(unpack_e4m3(u.x & 0xFFFFu, f), unpack_e4m3(u.x >> 16, f),
                           unpack_e4m3(u.y & 0xFFFFu, f), unpack_e4m3(u.y >> 16, f));
            *reinterpret_cast<uint4*>(hi_at + at) =
                make_uint4(unpack_e4m3(u.z & 0xFFFFu, f), unpack_e4m3(u.z >> 16, f),
                           unpack_e4m3(u.w & 0xFFFFu, f), unpack_e4m3(u.w >> 16, f));
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    uint32_t ke = do_k ? load_exps(0, p.k_exps) : 0u, ve = load_exps(0, p.v_exps);
    load(0);
    set_up();
    int vref = 0;
    bool ok = true;
    for (int t = 0; t < tiles; ++t) {
      const int st = t % C::KS, par = t & 1;
      // references and factors of the tile; this warp's row is key tid
      const uint32_t kmax = max(8u, __reduce_max_sync(0xffffffffu, max_byte(ke)));
      const int vmax = int(max(8u, __reduce_max_sync(0xffffffffu, max_byte(ve))));
      if (vmax > vref) vref = min(vmax + kAttVSlack, 254);
      const int src_lane = tid >> 2, sh = (tid & 3) * 8;
      const uint32_t kb = (__shfl_sync(0xffffffffu, ke, src_lane) >> sh) & 0xFFu;
      const uint32_t vb = (__shfl_sync(0xffffffffu, ve, src_lane) >> sh) & 0xFFu;
      const unsigned vnan = __ballot_sync(0xffffffffu, vb == 255u);
      if (do_k) {
        fac_k[par * kTile + tid] = kb == 255u ? 0x7E007E00u : att_factor(int(kb), int(kmax));
        AttTileMeta& meta = s_meta[t & (kAttMetaRing - 1)];
        if (lane == 0) meta.v_nan[tid >> 5] = vnan;
        if (tid == 0) {
          meta.k_scale = __uint_as_float((kmax - 7u) << 23);
          meta.v_ref = vref;
        }
      }
      if (!do_k) fac_v[par * kTile + tid] = vb == 255u ? 0u : att_factor(int(vb), vref);
      // the codes of a V row of byte 255 may be E4M3's NaN, which a factor of 0 would let through to rows that do not see it
      const bool drop = __any_sync(0xffffffffu, !do_k && __vcmpeq4(ve, 0xFFFFFFFFu) != 0u);
      // the factors of the next tile go to the other half, so one barrier will do
      if (do_k)
        asm volatile("bar.sync 1, 128;" ::: "memory");
      else
        asm volatile("bar.sync 2, 128;" ::: "memory");
      ke = do_k ? load_exps(t + 1, p.k_exps) : 0u;
      ve = load_exps(t + 1, p.v_exps);
      uint64_t* full = do_k ? k_full : v_full;
      uint64_t* free_ = do_k ? k_free : v_free;
      if (t >= C::KS) ok = ok && warp_wait(&free_[st], uint32_t(((t - C::KS) / C::KS) & 1), abort_flag, T);
      if (ok) {
        if (drop) {   // rows of factor 0, whatever their codes
#pragma unroll
          for (int i = 0; i < 4 * C::DC; ++i)
            if (fac_v[par * kTile + 32 * (i & 3) + r0] == 0u) raw[i] = make_uint4(0, 0, 0, 0);
        }
        convert(smem + (do_k ? C::OFF_K : C::OFF_V) + st * C::TILE_BYTES, (do_k ? fac_k : fac_v) + par * kTile);
        mbar_arrive_lane0(&full[st], lane);
        load(t + 1);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      set_status(p.status, TSEL_DEV_TIMEOUT);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::MMA_WARP) tmem_dealloc(*tmem_slot, 512);
}

// Joins a row's partial results: out = sum_c 2^(lse_c - lse) o_c. WPR warps
// share a row (its partials go round them) and are added up in their order, so
// a row with many partials is not one long chain of loads; D / 4 lanes of four
// columns. Chunks without visible keys have lse = -inf and wrote no columns.
//   PACKED: rows of packed sequences. Only those of segments that keep the bounds have
// partials; a row looks for its segment among all of them, 32 at a time (keys are cut
// into chunks for a few segments alone), since one with bad bounds may lie anywhere.
constexpr int kJoinWarps = 8;

// What is left of a partial too far below the row's largest, its weight 0: its
// NaN, but no number. INF: and its infinities, which are of V rows that the row sees;
// cached rows are finite, so an infinity of theirs is a mean past fp32's range, which
// goes too.
template <bool INF>
__device__ __forceinline__ void keep_special(float& acc, float o) {
  if (INF) {
    if (!(fabsf(o) < __builtin_huge_valf())) acc += o;
  } else if (o != o) {
    acc = o;
  }
}
template <bool INF>
__device__ __forceinline__ void keep_special(float4& acc, const float4& o) {
  keep_special<INF>(acc.x, o.x);
  keep_special<INF>(acc.y, o.y);
  keep_special<INF>(acc.z, o.z);
  keep_special<INF>(acc.w, o.w);
}

// Every lane of the warp calls it.
__device__ __forceinline__ bool join_has_row(const AttParams& p, int64_t tok) {
  const int lane = threadIdx.x & 31;
  for (int first = 0; first < p.R; first += 32) {
    const int g = first + lane;
    bool mine = false;
    if (g < p.R) {
      const int qa = __ldg(p.cu_q + g), nq = __ldg(p.cu_q + g + 1) - qa, ka = __ldg(p.cu_k + g), nk = __ldg(p.cu_k + g + 1) - ka;
      mine = att_segment_ok(g, qa, nq, ka, nk, p.max_q, p.max_k, p.Tq, p.Tk) && tok >= qa && tok < int64_t(qa) + nq;
    }
    if (__any_sync(0xffffffffu, mine)) return true;
  }
  return false;
}

template <int D, int WPR, bool PACKED>
__global__ void __launch_bounds__(32 * kJoinWarps) attend_join_kernel(const AttParams p) {
  __shared__ float s_acc[WPR > 1 ? kJoinWarps : 1][D];
  __shared__ float s_m[kJoinWarps], s_sum[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp % WPR;
  pdl_launch_dependents();
  pdl_wait();
  const int total = __ldg(p.cu_q + p.R);
  // also where no suffix kernel looks at the requests one by one
  if (total < 0 || total > p.Tq || total > int64_t(p.R) * p.max_q) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, TSEL_DEV_SEQLENS);
    if (!PACKED) return;
  }
  const int64_t rows = int64_t(PACKED ? p.Tq : total) * p.H;
  const int64_t step = int64_t(p.Tq) * p.H;
  const int64_t r = int64_t(blockIdx.x) * (kJoinWarps / WPR) + warp / WPR;
  const bool has = r < rows && (!PACKED || join_has_row(p, r / p.H));
  float m = kNegInf, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (has) {
    for (int base = 0; base < p.slots; base += 32 * WPR) {
      const int at = base + lane * WPR + part;   // a lane per partial
      const float mine = at < p.slots ? p.part_lse[at * step + r] : kNegInf;
      unsigned live = __ballot_sync(0xffffffffu, mine != kNegInf);
      float top = mine;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float now = fmaxf(m, top), ref = now == kNegInf ? 0.f : now;
      const float old = m == kNegInf ? 0.f : exp2f(m - ref);
      m = now;
      sum *= old;
      acc.x *= old;
      acc.y *= old;
      acc.z *= old;
      acc.w *= old;
      const float wgt = exp2f(mine - ref);
      while (live != 0) {   // four partials in flight
        float wv[4];
        float4 o[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int c = live != 0 ? __ffs(live) - 1 : -1;
          live &= live - 1;
          wv[x] = c >= 0 ? __shfl_sync(0xffffffffu, wgt, c) : 0.f;
          o[x] = c >= 0 && lane < D / 4
                     ? *reinterpret_cast<const float4*>(p.part_o + ((base + c * WPR + part) * step + r) * D + 4 * lane)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (wv[x] == 0.f) {
            keep_special<PACKED>(acc, o[x]);
            continue;
          }
          sum += wv[x];
          acc.x += wv[x] * o[x].x;
          acc.y += wv[x] * o[x].y;
          acc.z += wv[x] * o[x].z;
          acc.w += wv[x] * o[x].w;
        }
      }
    }
  }
  if (WPR > 1) {
    if (lane < D / 4) *reinterpret_cast<float4*>(&s_acc[warp][4 * lane]) = acc;
    if (lane == 0) {
      s_m[warp] = m;
      s_sum[warp] = sum;
    }
    __syncthreads();
    if (part != 0) return;
    m = kNegInf;
#pragma unroll
    for (int x = 0; x < WPR; ++x) m = fmaxf(m, s_m[warp + x]);
    sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (lane < D / 4) {
#pragma unroll
      for (int x = 0; x < WPR; ++x) {
        // a warp whose partials are all NaN has no maximum, but a NaN sum
        const float f = s_m[warp + x] == kNegInf ? (s_sum[warp + x] == 0.f ? 0.f : 1.f) : exp2f(s_m[warp + x] - m);
        const float4 v = *reinterpret_cast<const float4*>(&s_acc[warp + x][4 * lane]);
        if (f == 0.f) {   // this warp's NaN partials among lower ones: also in its sum
          if (s_sum[warp + x] != s_sum[warp + x]) sum = s_sum[warp + x];
          keep_special<PACKED>(acc, v);
          continue;
        }
        sum += f * s_sum[warp + x];
        acc.x += f * v.x;
        acc.y += f * v.y;
        acc.z += f * v.z;
        acc.w += f * v.w;
      }
    }
  }
  if (!has) return;
  const float ref = m == kNegInf ? 0.f : m;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t tok = r / p.H;
  const int head = int(r - tok * p.H);
  if (lane < D / 4) {
    uint2 o;
    if (p.fp16) {
      o.x = pack_f16(acc.x * inv, acc.y * inv);
      o.y = pack_f16(acc.z * inv, acc.w * inv);
    } else {
      __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      o.x = *reinterpret_cast<uint32_t*>(&a);
      o.y = *reinterpret_cast<uint32_t*>(&b);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + tok * p.out_stride + int64_t(head) * D + 4 * lane) = o;
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[int64_t(head) * p.Tq + tok] = sum == 0.f ? kNegInf : (ref + log2f(sum)) * 0.69314718055994531f;
}

template <int D, bool TREE>
cudaError_t launch_attend_t(const AttParams& p, int64_t units, cudaStream_t stream) {
  using C = AttCfg<D, TREE>;
  auto kern = attend_kernel<D, TREE>;
  static bool attr_set[128] = {};   // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) attr_set[dev] = true;
  }
  return launch_kernel(kern, dim3(unsigned(units)), C::THREADS, size_t(C::SMEM_BYTES), stream, 1, p);
}

}  // namespace

cudaError_t launch_attend(int head_dim, const AttParams& p, int64_t units, cudaStream_t stream) {
  const bool tree = p.parents != nullptr && units > p.pre_units;
#define TSEL_ATT_CASE(DD) \
  case DD:                \
    return tree ? launch_attend_t<DD, true>(p, units, stream) : launch_attend_t<DD, false>(p, units, stream);
  switch (head_dim) {
    TSEL_ATT_CASE(64)
    TSEL_ATT_CASE(80)
    TSEL_ATT_CASE(96)
    TSEL_ATT_CASE(112)
    TSEL_ATT_CASE(128)
    default:
      return cudaErrorInvalidValue;
  }
#undef TSEL_ATT_CASE
}

namespace {
template <int D, bool PACKED>
cudaError_t launch_join_t(const AttParams& p, cudaStream_t stream) {
  // Warps to a row with more than eight partials: all eight while the rows are
  // fewer than the CTAs that fit (64 rows of 73 partials: a call takes 25.7 us,
  // with two 26.9), two while a warp each would leave SMs idle (2,048 rows of 38:
  // 82 us, with eight 85, with one 86); one otherwise (4,544 rows of 17: 90.5
  // us, with two 91.1, with eight 96.3).
  const int64_t rows = int64_t(p.Tq) * p.H;
  const int wpr = p.slots <= 8 || rows > 4096 ? 1 : (rows > 1024 ? 2 : kJoinWarps);
  auto kern = wpr == 1 ? attend_join_kernel<D, 1, PACKED>
                       : (wpr == 2 ? attend_join_kernel<D, 2, PACKED> : attend_join_kernel<D, kJoinWarps, PACKED>);
  return launch_kernel(kern, dim3(unsigned(ceil_div(rows, kJoinWarps / wpr))), 32 * kJoinWarps, 0, stream, 1, p);
}
}  // namespace

cudaError_t launch_attend_join(int head_dim, const AttParams& p, cudaStream_t stream) {
#define TSEL_JOIN_CASE(DD) \
  case DD:                 \
    return p.cu_k != nullptr ? launch_join_t<DD, true>(p, stream) : launch_join_t<DD, false>(p, stream);
  switch (head_dim) {
    TSEL_JOIN_CASE(64)
    TSEL_JOIN_CASE(80)
    TSEL_JOIN_CASE(96)
    TSEL_JOIN_CASE(112)
    TSEL_JOIN_CASE(128)
    default:
      return cudaErrorInvalidValue;
  }
#undef TSEL_JOIN_CASE
}

}  // namespace tsel
