// Attention over whole prompts: packed sequences, causal or not, query heads in
// groups that share a KV head, and the row log-sum-exps that the importance
// scoring takes (TSEL_IMP_LSE_PROVIDED).
//
// o_i = sum_j p_ij v_j / sum_j p_ij with p_ij = exp(s q_i . k_j) over the keys
// that row i sees. LiteVLM review, "core formulas" (softmax(Q K^T / sqrt d) V);
// TLiveOmni article, "Flash-Attention differences" (varlen interface with
// cu_seqlens); dynamic vision-token compression article, section 3.2 (the LSE
// of the attention kernel is used again by the scoring).
//
// The rows of a KV head's query heads form one matrix, token by token, cut into
// 128-row tiles. A unit is (segment, KV head, two row tiles, key chunk); a
// persistent CTA per SM takes units in turn, the ones with most keys first. Keys
// are cut into chunks only where units are few; attend.cu's join then adds the
// chunks up.
//
// Roles of a CTA (12 warps):
//   - producer: decodes units into a ring and loads Q tiles and steps of 64 keys
//     of K and V by TMA (128-byte swizzle; columns past the head dimension and
//     rows past the tensor read as zeros);
//   - two issuers, one for each row tile: S = Q K^T (64 columns) and O += P V, both
//     tcgen05 with fp32 accumulators in TMEM. A row tile has 256 columns: O 128,
//     S 64, and two places of 32 for P, so that the next S product waits only until
//     the softmax has S in registers, never for the O product that reads P;
//   - four softmax warps for each row tile, a thread to a row: P = 2^(S c - m) goes
//     to TMEM as the A operand of the second product. The reference m may lag the
//     row's maximum by 2^9; past that O is rescaled in TMEM;
//   - one warp that passes each V step on: in steps that some row does not see whole,
//     it clears rows past the last visible key and takes infinities and NaN out (a
//     product with P = 0 would make NaN of rows that do not see them). The rows that
//     do see them get them back at the end.
// P is rounded to the type of V (bf16: eight bits; fp16: eleven, down to 2^-20 of
// the reference, ending at 2^-30 of it), since both operands of a product have one
// type; statistics, sums and O are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend_ops.cuh"
#include "imp_pass.cuh"
#include "prompt.cuh"

namespace tsel {

namespace {

constexpr float kPromptSlack = 9.f;   // the reference may lag the row maximum by 2^9
constexpr int kPromptRing = 3;        // units in flight

struct PromptUnit {
  int valid;
  int kvh, chunk;
  int tok0, tok_end;     // tokens of the unit's rows
  int k_base;            // first key of the segment, in K
  int c0, k1;            // keys [c0, k1) of the segment
  int lim;               // token t sees the first lim + (causal ? t : 0) keys of the segment
  int n0, n1, steps;     // steps of the two row tiles, and of the unit
  int fix;               // first step that some row does not see whole
};

template <int D>
struct PromptCfg {
  static constexpr int DC = D > 64 ? 2 : 1;                     // 64-element chunks of a row
  static constexpr int Q_BYTES = DC * kTile * 128;
  static constexpr int ST_BYTES = DC * kPromptStep * 128;       // one step of K or V
  static constexpr int KS = 8 / DC;                             // stages of each
  static constexpr int SOFT_WARPS = 8;
  static constexpr int MMA_WARP = SOFT_WARPS;                   // two
  static constexpr int LOAD_WARP = MMA_WARP + 2;
  static constexpr int FIX_WARP = LOAD_WARP + 1;
  static constexpr int THREADS = 32 * (FIX_WARP + 1);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + KS * ST_BYTES;
  static constexpr int OFF_BAR = OFF_V + KS * ST_BYTES;
  static constexpr int NUM_BARS = 4 + 5 * KS + 4 + 8 + 2 + 2 + 2 * kPromptRing;
  static constexpr int OFF_UNITS = OFF_BAR + 8 * NUM_BARS;
  static constexpr int OFF_BAD = OFF_UNITS + kPromptRing * int(sizeof(PromptUnit));   // int [ring]
  static constexpr int OFF_ORDER = OFF_BAD + 4 * kPromptRing;   // int [sorted], then int [sorted]
  static constexpr int OFF_MISC = (OFF_ORDER + 8 * kPromptSorted + 15) / 16 * 16;
  static constexpr int SMEM_USED = OFF_MISC + 16 + 1024;        // + alignment slack
  // one CTA per SM (it holds all of TMEM), also for the smaller heads
  static constexpr int SMEM_BYTES = SMEM_USED > 120 * 1024 ? SMEM_USED : 120 * 1024;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
};

// Two fp32 values in the type of V (x in the low half).
template <bool FP16>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
  uint32_t r;
  if (FP16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}

// 16 columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 2^(S c + shift) of 32 columns, added up in acc and packed.
template <bool FP16>
__device__ __forceinline__ void prompt_exp32(const uint32_t (&r)[32], float2 c2, float2 s2, float2& acc, uint32_t (&h)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float2 a = __ffma2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), c2, s2);
    const float2 e = make_float2(ex2(a.x), ex2(a.y));
    acc = __fadd2_rn(acc, e);
    h[j] = pack16<FP16>(e.x, e.y);
  }
}

// Two values of V of which one is an infinity or NaN: a mask of those halves.
template <bool FP16>
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) {
  const uint32_t m = FP16 ? 0x7C007C00u : 0x7F807F80u;
  return __vcmpeq2(w & m, m);
}

template <bool FP16>
__device__ __forceinline__ float widen(uint16_t u) {
  return FP16 ? __half2float(__ushort_as_half(u)) : __uint_as_float(uint32_t(u) << 16);
}

template <int D, bool FP16>
__global__ void __launch_bounds__(PromptCfg<D>::THREADS, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, const PromptParams p) {
  using C = PromptCfg<D>;
  constexpr int KS = C::KS;
  constexpr float kLift = FP16 ? 6.f : 0.f;   // P at the row's reference: fp16's range goes further down from there
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = smem_dyn + ((1024u - (smem_u32(smem_dyn) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;              // [row tile]
  uint64_t* q_free = q_full + 2;        // last S product of the unit done
  uint64_t* k_full = q_free + 2;        // [KS] loaded
  uint64_t* k_free = k_full + KS;       // both issuers are done with it
  uint64_t* v_in = k_free + KS;         // loaded
  uint64_t* v_full = v_in + KS;         // looked through
  uint64_t* v_free = v_full + KS;
  uint64_t* s_full = v_free + KS;       // [row tile] S in TMEM
  uint64_t* s_free = s_full + 2;        // S in registers
  uint64_t* p_full = s_free + 2;        // [row tile][place] P in TMEM
  uint64_t* o_done = p_full + 4;        // [row tile][place] O product done
  uint64_t* o_free = o_done + 4;        // [row tile] O of the unit in registers
  uint64_t* drained = o_free + 2;       // [row tile] every product done
  uint64_t* u_full = drained + 2;       // [ring]
  uint64_t* u_free = u_full + kPromptRing;
  PromptUnit* s_units = reinterpret_cast<PromptUnit*>(smem + C::OFF_UNITS);
  volatile int* s_bad = reinterpret_cast<volatile int*>(smem + C::OFF_BAD);   // the unit's V had infinities or NaN taken out
  int* s_order = reinterpret_cast<int*>(smem + C::OFF_ORDER);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t T = p.timeout_ns;
  // Before the wait for earlier kernels: what does not touch their memory.
  if (warp == C::MMA_WARP) {
    if (lane == 0) {
      for (int i = 0; i < KS; ++i) {
        mbar_init(&k_full[i], 1);
        mbar_init(&k_free[i], 2);
        mbar_init(&v_in[i], 1);
        mbar_init(&v_full[i], 1);
        mbar_init(&v_free[i], 2);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&q_full[i], 1);
        mbar_init(&q_free[i], 1);
        mbar_init(&s_full[i], 1);
        mbar_init(&s_free[i], 4);
        mbar_init(&o_free[i], 4);
        mbar_init(&drained[i], 1);
      }
      for (int i = 0; i < 4; ++i) {
        mbar_init(&p_full[i], 4);
        mbar_init(&o_done[i], 1);
      }
      for (int i = 0; i < kPromptRing; ++i) {
        mbar_init(&u_full[i], 1);
        mbar_init(&u_free[i], C::SOFT_WARPS + 2 + 1);   // softmax, issuers, V warp
      }
      *abort_flag = 0;
      fence_barrier_init();
    }
    __syncwarp();
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
    tc_fence_before();
  } else if (warp == C::LOAD_WARP && lane == 0) {
    prefetch_tensormap(&mq);
    prefetch_tensormap(&mk);
    prefetch_tensormap(&mv);
  }
  pdl_wait();
  // Segments by their keys, most first; as they come where there are many.
  const bool sorted = p.seg <= kPromptSorted;
  if (sorted) {
    int* s_len = s_order + kPromptSorted;
    for (int g = threadIdx.x; g < p.seg; g += C::THREADS) s_len[g] = __ldg(p.cu_k + g + 1) - __ldg(p.cu_k + g);
    __syncthreads();
    for (int g = threadIdx.x; g < p.seg; g += C::THREADS) {
      const int n = s_len[g];
      int at = 0;
      for (int i = 0; i < p.seg; ++i) at += s_len[i] > n || (s_len[i] == n && i < g) ? 1 : 0;
      s_order[at] = g;
    }
  }
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;

  if (warp < C::SOFT_WARPS) {
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2;
    const int row = int(threadIdx.x) & (kTile - 1);
    const uint32_t t_o = tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(x * 256);
    const uint32_t t_s = t_o + 128, t_p = t_o + 192;
    uint32_t J = 0, slot = 0, turn = 0;   // steps of this row tile so far, place and turn of the unit ring
    bool ok = true;
    for (;;) {
      if (!warp_wait(&u_full[slot], turn & 1u, abort_flag, T)) {
        ok = false;
        break;
      }
      const PromptUnit& u = s_units[slot];
      if (!u.valid) break;
      const int n = x == 0 ? u.n0 : u.n1, c0 = u.c0;
      const int tok = u.tok0 + x * p.tt + row / p.G;
      const bool row_ok = row < p.tt * p.G && tok < u.tok_end;
      const int end = row_ok ? max(min(u.lim + (p.causal ? tok : 0), u.k1), c0) - c0 : 0;   // visible keys of the chunk
      const int min_end = int(__reduce_min_sync(0xffffffffu, row_ok ? unsigned(end) : 0x7FFFFFFFu));
      float m = kNegInf, l = 0.f;
      for (int j = 0; j < n; ++j, ++J) {
        if (!warp_wait(&s_full[x], J & 1u, abort_flag, T)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r0[32], r1[32];
        tmem_ld32_async(t_s, r0);
        tmem_ld32_async(t_s + 32, r1);
        tmem_wait_ld(r0);
        tmem_wait_ld(r1);
        tc_fence_before();
        __syncwarp();
        mbar_arrive_lane0(&s_free[x], lane);
        if ((j + 1) * kPromptStep > min_end) {
          mask_cols(r0, end - j * kPromptStep);
          mask_cols(r1, end - j * kPromptStep - 32);
        }
        const float top = fmaxf(cols_max(r0), cols_max(r1)) * p.c;
        if (__any_sync(0xffffffffu, top > m + kPromptSlack)) {
          float s = 1.f;
          if (top > m) {   // also the rows that could still wait: once here, it costs nothing
            s = ex2(m - top);   // 0 at the row's first visible keys
            l *= s;
            m = top;
          }
          if (j > 0) {   // once the O product of the step before is complete
            if (!warp_wait(&o_done[2 * x + ((J - 1) & 1u)], ((J - 1) >> 1) & 1u, abort_flag, T)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < D; cc += 16) {
              uint32_t o[16];
              tmem_ld16(t_o + cc, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * s);
              tmem_st16(t_o + cc, o);
            }
          }
        }
        const float shift = m == kNegInf ? 0.f : kLift - m;
        const float2 c2 = make_float2(p.c, p.c), s2 = make_float2(shift, shift);
        float2 a0 = make_float2(0.f, 0.f), a1 = a0;
        uint32_t h0[16], h1[16];
        prompt_exp32<FP16>(r0, c2, s2, a0, h0);
        prompt_exp32<FP16>(r1, c2, s2, a1, h1);
        // the place of P is free once the O product of two steps before is complete
        if (j >= 2 && !warp_wait(&o_done[2 * x + (J & 1u)], ((J >> 1) + 1) & 1u, abort_flag, T)) {
          ok = false;
          break;
        }
        tc_fence_after();
        tmem_st16(t_p + 32 * (J & 1u), h0);
        tmem_st16(t_p + 32 * (J & 1u) + 16, h1);
        a0 = __fadd2_rn(a0, a1);
        l += a0.x + a0.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_lane0(&p_full[2 * x + (J & 1u)], lane);
      }
      if (!ok) break;
      if (n > 0) {
        if (!warp_wait(&o_done[2 * x + ((J - 1) & 1u)], ((J - 1) >> 1) & 1u, abort_flag, T)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      const int head = u.kvh * p.G + row % p.G;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool bad = s_bad[slot] != 0;
      const float lse2 = l == 0.f ? kNegInf : m + (log2f(l) - kLift);
      float* part = nullptr;
      if (p.part_lse != nullptr) {
        const int64_t at = (int64_t(u.chunk) * p.Tq + tok) * p.H + head;
        if (row_ok) p.part_lse[at] = lse2;
        part = p.part_o + at * D;
      } else if (row_ok && p.lse != nullptr) {
        p.lse[int64_t(head) * p.Tq + tok] = lse2 * 0.69314718055994531f;
      }
      uint16_t* out = static_cast<uint16_t*>(p.out) + int64_t(tok) * p.out_stride + int64_t(head) * D;
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 16) {
        uint32_t o[16];
        if (n > 0) tmem_ld16(t_o + cc, o);
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = n > 0 && l != 0.f ? __uint_as_float(o[k]) * inv : 0.f;
        if (bad && row_ok && l != 0.f) {   // infinities and NaN of the V rows that this row sees
          const uint16_t* v = static_cast<const uint16_t*>(p.v) + int64_t(u.k_base + c0) * p.v_stride + int64_t(u.kvh) * D + cc;
          for (int j = u.fix * kPromptStep; j < end; ++j) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float t = widen<FP16>(v[j * p.v_stride + k]);
              if (!(fabsf(t) < __builtin_huge_valf())) f[k] += t;
            }
          }
        }
        if (row_ok) {
          if (part != nullptr) {
            if (l != 0.f) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(part + cc + 4 * k) = make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k)
              *reinterpret_cast<uint4*>(out + cc + 8 * k) =
                  make_uint4(pack16<FP16>(f[8 * k], f[8 * k + 1]), pack16<FP16>(f[8 * k + 2], f[8 * k + 3]),
                             pack16<FP16>(f[8 * k + 4], f[8 * k + 5]), pack16<FP16>(f[8 * k + 6], f[8 * k + 7]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (n > 0) mbar_arrive_lane0(&o_free[x], lane);
      mbar_arrive_lane0(&u_free[slot], lane);
      if (++slot == kPromptRing) {
        slot = 0;
        ++turn;
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      set_status(p.status, TSEL_DEV_TIMEOUT);
    }
  } else if (warp < C::LOAD_WARP) {
    // ------------------------------------------------------------ issuers
    const int x = __shfl_sync(0xffffffffu, warp, 0) - C::MMA_WARP;
    constexpr uint32_t kIdS = idesc_f16_f32(kTile, kPromptStep, false, !FP16);
    constexpr uint32_t kIdO = idesc_f16_f32(kTile, D, true, !FP16);
    const uint32_t t_o = __shfl_sync(0xffffffffu, tmem, 0) + uint32_t(x * 256);
    const uint32_t t_s = t_o + 128, t_p = t_o + 192;
    // advanced by (bytes >> 4)
    const uint64_t dq = smem_desc(smem_u32(smem + C::OFF_Q) + x * C::Q_BYTES, 2, 1024);
    const uint64_t dk = smem_desc(smem_u32(smem + C::OFF_K), 2, 1024);
    const uint64_t dv = smem_desc_mn(smem_u32(smem + C::OFF_V), kPromptStep * 128, 1024);
    uint32_t J = 0, ks = 0, vs = 0, slot = 0, turn = 0;   // steps of this row tile; K and V steps of the CTA; unit ring
    uint32_t live = 0;                                     // units in which this row tile had steps
    bool ok = true;
    for (;;) {
      if (!warp_wait(&u_full[slot], turn & 1u, abort_flag, T)) {
        ok = false;
        break;
      }
      const PromptUnit& u = s_units[slot];
      if (!u.valid) break;
      const int steps = u.steps, n = x == 0 ? u.n0 : u.n1;
      __syncwarp();
      mbar_arrive_lane0(&u_free[slot], lane);
      if (++slot == kPromptRing) {
        slot = 0;
        ++turn;
      }
      // S of step j; steps that this row tile does not see are only let go
      auto s_product = [&](int j) -> bool {
        const uint32_t st = ks % KS;
        if (!warp_wait(&k_full[st], (ks / KS) & 1u, abort_flag, T)) return false;
        ++ks;
        if (j >= n) {
          mbar_arrive_lane0(&k_free[st], lane);
          return true;
        }
        const uint32_t at = J + j;
        if (at > 0 && !warp_wait(&s_free[x], (at - 1) & 1u, abort_flag, T)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t a = (kk >> 2) * (kTile * 128) + (kk & 3) * 32, b = (kk >> 2) * (kPromptStep * 128) + (kk & 3) * 32;
          mma_ss_elect(t_s, dq + (a >> 4), dk + ((st * C::ST_BYTES + b) >> 4), kIdS, kk > 0);
        }
        commit_elect(&s_full[x]);
        commit_elect(&k_free[st]);
        if (j == n - 1) commit_elect(&q_free[x]);
        return true;
      };
      if (n > 0 && !warp_wait(&q_full[x], live & 1u, abort_flag, T)) {
        ok = false;
        break;
      }
      if (steps > 0) ok = s_product(0);
      for (int j = 0; j < steps && ok; ++j) {
        if (j + 1 < steps) ok = s_product(j + 1);
        if (!ok) break;
        const uint32_t st = vs % KS;
        if (!warp_wait(&v_full[st], (vs / KS) & 1u, abort_flag, T)) {
          ok = false;
          break;
        }
        ++vs;
        if (j >= n) {
          mbar_arrive_lane0(&v_free[st], lane);
          continue;
        }
        const uint32_t at = J + j, place = at & 1u;
        if (!warp_wait(&p_full[2 * x + place], (at >> 1) & 1u, abort_flag, T) ||
            (j == 0 && live > 0 && !warp_wait(&o_free[x], (live - 1) & 1u, abort_flag, T))) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kPromptStep / 16; ++kk)
          mma_ts_elect(t_o, t_p + 32 * place + 8 * kk, dv + ((st * C::ST_BYTES + kk * 2048) >> 4), kIdO, j > 0 || kk > 0);
        commit_elect(&o_done[2 * x + place]);
        commit_elect(&v_free[st]);
      }
      if (!ok) break;
      J += uint32_t(n);
      if (n > 0) ++live;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      set_status(p.status, TSEL_DEV_TIMEOUT);
    }
    __syncwarp();
    // every product of this warp has completed before TMEM is freed
    commit_elect(&drained[x]);
    wait_drain(&drained[x], 0, T);
  } else if (warp == C::LOAD_WARP) {
    // ------------------------------------------------------------ producer
    const int64_t per = int64_t(p.Hkv) * p.chunks;   // units of a block of rows
    int first = 0;                                   // segments [first, first + 32) in order,
    int64_t before = 0;                              // units of the ones before
    uint32_t ks = 0, qn[2] = {0, 0}, slot = 0, turn = 0;
    bool ok = true;
    for (int64_t round = 0; ok; ++round) {
      // there and back, so that no CTA has the longer unit of every round
      int64_t i = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      PromptUnit u{};
      while (first < p.seg) {
        const int at = first + lane;
        const int g = at < p.seg ? (sorted ? s_order[at] : at) : -1;
        int qa = 0, nq = 0, ka = 0, nk = 0;
        if (g >= 0) {
          qa = __ldg(p.cu_q + g);
          nq = __ldg(p.cu_q + g + 1) - qa;
          ka = __ldg(p.cu_k + g);
          nk = __ldg(p.cu_k + g + 1) - ka;
          const bool good = qa >= 0 && nq >= 0 && nq <= p.max_q && qa <= p.Tq - nq && ka >= 0 && nk >= 0 && nk <= p.max_k &&
                            ka <= p.Tk - nk && (g > 0 || (qa == 0 && ka == 0));
          if (!good) {
            set_status(p.status, TSEL_DEV_SEQLENS);
            nq = 0;
          }
        }
        int64_t sum = ((int64_t(nq) + 2 * p.tt - 1) / (2 * p.tt)) * per;   // up to this segment
        const int64_t mine = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + sum > i);
        if (past == 0) {
          before += __shfl_sync(0xffffffffu, sum, 31);
          first += 32;
          continue;
        }
        const int src = __ffs(past) - 1;
        qa = __shfl_sync(0xffffffffu, qa, src);
        nq = __shfl_sync(0xffffffffu, nq, src);
        ka = __shfl_sync(0xffffffffu, ka, src);
        nk = __shfl_sync(0xffffffffu, nk, src);
        int64_t v = i - before - __shfl_sync(0xffffffffu, sum - mine, src);
        const int64_t vh = v / p.Hkv, blk = vh / p.chunks;
        u.valid = 1;
        u.kvh = int(v - vh * p.Hkv);
        u.chunk = int(vh - blk * p.chunks);
        const int b = (nq - 1) / (2 * p.tt) - int(blk);   // the last rows see most keys
        u.tok0 = qa + b * 2 * p.tt;
        u.tok_end = min(qa + nq, u.tok0 + 2 * p.tt);
        u.k_base = ka;
        u.lim = p.causal ? nk - nq + 1 - qa : nk;
        auto seen = [&](int tok) { return max(min(u.lim + (p.causal ? tok : 0), nk), 0); };
        const int all = seen(u.tok_end - 1);
        u.c0 = int(min(int64_t(u.chunk) * p.keys, int64_t(all)));
        u.k1 = int(min(int64_t(u.c0) + p.keys, int64_t(all)));
        const int t1 = min(u.tok0 + p.tt, u.tok_end);
        u.n0 = (max(min(seen(t1 - 1), u.k1) - u.c0, 0) + kPromptStep - 1) / kPromptStep;
        u.n1 = u.tok0 + p.tt < u.tok_end ? (u.k1 - u.c0 + kPromptStep - 1) / kPromptStep : 0;
        u.steps = max(u.n0, u.n1);
        u.fix = max(min(seen(u.tok0), u.k1) - u.c0, 0) / kPromptStep;
        break;
      }
      ok = warp_wait(&u_free[slot], (turn & 1u) ^ 1u, abort_flag, T);
      if (!ok) break;
      if (lane == 0) {
        s_units[slot] = u;
        s_bad[slot] = 0;
      }
      __syncwarp();
      mbar_arrive_lane0(&u_full[slot], lane);
      if (++slot == kPromptRing) {
        slot = 0;
        ++turn;
      }
      if (!u.valid) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if ((x == 0 ? u.n0 : u.n1) == 0) continue;
        ok = ok && warp_wait(&q_free[x], (qn[x] & 1u) ^ 1u, abort_flag, T);
        if (ok && lane == 0) {
          mbar_arrive_expect_tx(&q_full[x], uint32_t(C::DC * 128 * p.tt * p.G));
#pragma unroll
          for (int cc = 0; cc < C::DC; ++cc)
            tma_load_3d(smem + C::OFF_Q + x * C::Q_BYTES + cc * (kTile * 128), &mq, &q_full[x], 64 * cc, u.kvh * p.G, u.tok0 + x * p.tt);
        }
        if (ok) ++qn[x];
      }
      for (int j = 0; j < u.steps && ok; ++j) {
        const uint32_t st = ks % KS, par = ((ks / KS) & 1u) ^ 1u;
        const int y = u.k_base + u.c0 + j * kPromptStep;
        ok = warp_wait(&k_free[st], par, abort_flag, T);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&k_full[st], C::ST_BYTES);
#pragma unroll
          for (int cc = 0; cc < C::DC; ++cc)
            tma_load_3d(smem + C::OFF_K + st * C::ST_BYTES + cc * (kPromptStep * 128), &mk, &k_full[st], 64 * cc, u.kvh, y);
        }
        // the V stage before, so that an abort leaves as many of both in flight
        ok = warp_wait(&v_free[st], par, abort_flag, T);
        if (lane == 0 && ok) {
          mbar_arrive_expect_tx(&v_in[st], C::ST_BYTES);
#pragma unroll
          for (int cc = 0; cc < C::DC; ++cc)
            tma_load_3d(smem + C::OFF_V + st * C::ST_BYTES + cc * (kPromptStep * 128), &mv, &v_in[st], 64 * cc, u.kvh, y);
        }
        if (ok) ++ks;
        else wait_drain(&k_full[st], (ks / KS) & 1u, T);
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      set_status(p.status, TSEL_DEV_TIMEOUT);
    }
    // every copy has landed before the CTA's shared memory goes
    for (uint32_t i = ks > KS ? ks - KS : 0; i < ks; ++i) {
      wait_drain(&k_full[i % KS], (i / KS) & 1u, T);
      wait_drain(&v_in[i % KS], (i / KS) & 1u, T);
    }
    for (int x = 0; x < 2; ++x)
      if (qn[x] > 0) wait_drain(&q_full[x], (qn[x] - 1) & 1u, T);
  } else {
    // ------------------------------------------------------------ V
    uint32_t vs = 0, slot = 0, turn = 0;
    bool ok = true;
    for (;;) {
      if (!warp_wait(&u_full[slot], turn & 1u, abort_flag, T)) {
        ok = false;
        break;
      }
      const PromptUnit& u = s_units[slot];
      if (!u.valid) break;
      for (int j = 0; j < u.steps; ++j, ++vs) {
        const uint32_t st = vs % KS;
        if (!warp_wait(&v_in[st], (vs / KS) & 1u, abort_flag, T)) {
          ok = false;
          break;
        }
        if (j >= u.fix) {
          const int left = u.k1 - u.c0 - j * kPromptStep;   // keys that some row sees
          uint32_t found = 0;
          uint8_t* tile = smem + C::OFF_V + st * C::ST_BYTES;
#pragma unroll 4
          for (int i = lane; i < C::DC * kPromptStep * 8; i += 32) {
            uint4* at = reinterpret_cast<uint4*>(tile + 16 * i);
            if (((i >> 3) & (kPromptStep - 1)) >= left) {
              *at = make_uint4(0, 0, 0, 0);
              continue;
            }
            uint4 w = *at;
            const uint4 b = make_uint4(not_finite2<FP16>(w.x), not_finite2<FP16>(w.y), not_finite2<FP16>(w.z), not_finite2<FP16>(w.w));
            const uint32_t any = b.x | b.y | b.z | b.w;
            found |= any;
            if (any) *at = make_uint4(w.x & ~b.x, w.y & ~b.y, w.z & ~b.z, w.w & ~b.w);
          }
          if (found) s_bad[slot] = 1;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        mbar_arrive_lane0(&v_full[st], lane);
      }
      if (!ok) break;
      mbar_arrive_lane0(&u_free[slot], lane);
      if (++slot == kPromptRing) {
        slot = 0;
        ++turn;
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
  if (warp == C::MMA_WARP) tmem_dealloc(tmem, 512);
}

template <int D, bool FP16>
cudaError_t launch_prompt_t(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const PromptParams& p,
                            int ctas, cudaStream_t stream) {
  using C = PromptCfg<D>;
  auto kern = prompt_kernel<D, FP16>;
  static bool attr_set[128] = {};   // per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 128) attr_set[dev] = true;
  }
  return launch_kernel(kern, dim3(unsigned(ctas)), C::THREADS, size_t(C::SMEM_BYTES), stream, 1, mq, mk, mv, p);
}

}  // namespace

cudaError_t launch_prompt(int head_dim, bool fp16, const CUtensorMap& mq, const CUtensorMap& mk,
                          const CUtensorMap& mv, const PromptParams& p, int ctas, cudaStream_t stream) {
#define TSEL_PROMPT_CASE(DD)                                                   \
  case DD:                                                                     \
    return fp16 ? launch_prompt_t<DD, true>(mq, mk, mv, p, ctas, stream)       \
                : launch_prompt_t<DD, false>(mq, mk, mv, p, ctas, stream);
  switch (head_dim) {
    TSEL_PROMPT_CASE(64)
    TSEL_PROMPT_CASE(80)
    TSEL_PROMPT_CASE(96)
    TSEL_PROMPT_CASE(112)
    TSEL_PROMPT_CASE(128)
    default:
      return cudaErrorInvalidValue;
  }
#undef TSEL_PROMPT_CASE
}

}  // namespace tsel
