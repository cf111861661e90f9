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
// Roles of a CTA (15 warps):
//   - producer: decodes units into a ring and loads Q tiles and steps of 64 keys
//     of K and V by TMA (128-byte swizzle; columns past the head dimension and
//     rows past the tensor read as zeros);
//   - four issuers, one for each product of a row tile: S = Q K^T (64 columns) and
//     O += P V, both tcgen05 with fp32 accumulators in TMEM. A row tile has 256
//     columns: O, S (twice for heads of 64) and two places for P, so that the next S
//     product waits only until the softmax has S in registers, never for the O
//     product that reads P;
//   - four softmax warps for each row tile, a thread to a row: P = 2^(S c - m) goes
//     to TMEM as the A operand of the second product. The reference m moves, and O
//     is rescaled in TMEM, only when a row's P of a step add up to more than 2^15: no
//     maximum is looked for before that, and the step is then done again;
//   - two warps that pass each V step on: in steps that some row does not see whole,
//     they clear rows past the last visible key and take infinities and NaN out (a
//     product with P = 0 would make NaN of rows that do not see them). The rows that
//     do see them get them back at the end. (One warp took 3,000 clocks a step of a
//     causal unit's end, two 650.)
// P is rounded to the type of V (bf16: eight bits; fp16: eleven, down to 2^-20 of
// the reference, ending at 2^-30 of it), since both operands of a product have one
// type; statistics, sums and O are fp32.
//
// What bounds it: for heads of 128 the two row tiles need 1,310 clocks of the tensor
// cores for 64 keys (measured alone: 50 for 128 x 64 x 16 with both operands in
// shared memory, 64 for 128 x 128 x 16 with A in TMEM) and a step takes about 1,550: the
// softmax warps' chain, some 350 instructions at four clocks each, of which 64 are
// exponentials (without them a step still took 85% of its time). 36,973 rows, causal,
// 16 heads on 8 of 128: 3.70 ms, 1.51 PFLOP/s, 79% of cuBLAS's bf16 rate; images of
// up to 4,096 tokens, 16 heads of 80: 0.90 ms for 61,585, 0.96 PFLOP/s; a packed
// batch of 24 requests of up to 1,370 (fp16, 32 heads on 8 of 128): 162 us; there a
// unit's end (O out of TMEM and to memory) costs as much as four steps.
// Tried and slower, or no faster: S of 128 keys in one place for both row tiles (a
// step of the batch 25% longer, the others 1 to 4% shorter), two warpgroups to a row
// tile for even and odd steps (5.8 ms: the issuers' waits), two threads to a row (4.05
// ms), more registers for the softmax (setmaxnreg; 3.85), waits that spin (3.87), the
// row tiles half a step apart (3.74), a row's results by its own
// thread instead of four lanes together (the same), 32 columns of O at a time
// (spills: 6.7).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attend_ops.cuh"
#include "imp_pass.cuh"
#include "prompt.cuh"

namespace tsel {

namespace {

// A row's reference moves when its P of a step add up to more than this: none of
// them is then past fp16's range, and the reference lags the row's maximum by
// less than 2^15 (bf16; 2^9 in fp16, whose P are 2^6 at the reference).
constexpr float kPromptMost = 32768.f;
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
  // TMEM columns of a row tile: S (two places where O leaves room), two places for P, O
  static constexpr int NS = D <= 64 ? 2 : 1, NP = 2;
  static constexpr int COL_P = 64 * NS, COL_O = COL_P + 32 * NP;
  static_assert(COL_O + D <= 256, "half of TMEM");
  static constexpr int SOFT_WARPS = 8;
  static constexpr int MMA_WARP = SOFT_WARPS;                   // [product][row tile]
  static constexpr int LOAD_WARP = MMA_WARP + 4;
  static constexpr int FIX_WARP = LOAD_WARP + 1;                // two
  static constexpr int THREADS = 32 * (FIX_WARP + 2);
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = 2 * Q_BYTES;
  static constexpr int OFF_V = OFF_K + KS * ST_BYTES;
  static constexpr int OFF_OUT = OFF_V + KS * ST_BYTES;         // 64 bytes of each row of the softmax warps
  static constexpr int OFF_BAR = OFF_OUT + SOFT_WARPS * 32 * 64;
  static constexpr int NUM_BARS = 4 + 5 * KS + 4 * NS + 4 * NP + 2 + 4 + 2 * kPromptRing;
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

// exp2 of both halves of x, added to acc with one packed add and packed in the type
// of V: in one piece, so that the two results need no moves to become a pair.
template <bool FP16>
__device__ __forceinline__ uint32_t exp_add_pack(float2 x, float2& acc) {
  uint32_t h;
  float2 r;
#define TSEL_EXP_ADD_PACK(CVT)                                \
  asm("{\n\t.reg .f32 e0, e1;\n\t.reg .b64 t, s, d;\n\t"     \
      "ex2.approx.ftz.f32 e0, %3;\n\t"                        \
      "ex2.approx.ftz.f32 e1, %4;\n\t"                        \
      "mov.b64 t, {e0, e1};\n\t"                              \
      "mov.b64 s, {%5, %6};\n\t"                              \
      "add.rn.f32x2 d, s, t;\n\t"                             \
      "mov.b64 {%0, %1}, d;\n\t" CVT " %2, e1, e0;\n\t}"      \
      : "=f"(r.x), "=f"(r.y), "=r"(h)                         \
      : "f"(x.x), "f"(x.y), "f"(acc.x), "f"(acc.y))
  if (FP16) TSEL_EXP_ADD_PACK("cvt.rn.f16x2.f32");
  else TSEL_EXP_ADD_PACK("cvt.rn.bf16x2.f32");
#undef TSEL_EXP_ADD_PACK
  acc = r;
  return h;
}

// 2^(S c + shift) of 32 columns, added up in acc and packed.
template <bool FP16>
__device__ __forceinline__ void prompt_exp32(const uint32_t (&r)[32], float2 c2, float2 s2, float2& acc, uint32_t (&h)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j)
    h[j] = exp_add_pack<FP16>(__ffma2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), c2, s2), acc);
}

// warp_wait() of barriers that have usually come: one test, with the vote taken on
// its predicate, before the bounded waits. (warp_wait alone costs 200 clocks where
// the barrier has come, and a step has several on its way.)
__device__ __forceinline__ bool prompt_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag, uint64_t timeout_ns) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "vote.sync.all.pred p, p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0 || warp_wait(bar, parity, abort_flag, timeout_ns);
}
__device__ __forceinline__ bool prompt_wait2(uint64_t* bar, uint32_t parity, uint64_t* bar2, uint32_t parity2,
                                             const volatile int* abort_flag, uint64_t timeout_ns) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "vote.sync.all.pred p, p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity), "r"(smem_u32(bar2)), "r"(parity2)
      : "memory");
  return done != 0 || (warp_wait(bar, parity, abort_flag, timeout_ns) && warp_wait(bar2, parity2, abort_flag, timeout_ns));
}

// Bits 15 and 31: the half's exponent is all ones (an infinity or NaN).
template <bool FP16>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return (w & (FP16 ? 0x7C007C00u : 0x7F807F80u)) + (FP16 ? 0x04000400u : 0x00800080u);
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
  constexpr int KS = C::KS, NS = C::NS, NP = C::NP;
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
  uint64_t* s_full = v_free + KS;       // [row tile][place] S in TMEM
  uint64_t* s_free = s_full + 2 * NS;   // S in registers
  uint64_t* p_full = s_free + 2 * NS;   // [row tile][place] P in TMEM
  uint64_t* o_done = p_full + 2 * NP;   // O product done
  uint64_t* o_free = o_done + 2 * NP;   // [row tile] O of the unit in registers
  uint64_t* drained = o_free + 2;       // [issuer] every product done
  uint64_t* u_full = drained + 4;       // [ring]
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
        mbar_init(&v_full[i], 2);
        mbar_init(&v_free[i], 2);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&q_full[i], 1);
        mbar_init(&q_free[i], 1);
        mbar_init(&o_free[i], 4);
      }
      for (int i = 0; i < 2 * NS; ++i) {
        mbar_init(&s_full[i], 1);
        mbar_init(&s_free[i], 4);
      }
      for (int i = 0; i < 2 * NP; ++i) {
        mbar_init(&p_full[i], 4);
        mbar_init(&o_done[i], 1);
      }
      for (int i = 0; i < 4; ++i) mbar_init(&drained[i], 1);
      for (int i = 0; i < kPromptRing; ++i) {
        mbar_init(&u_full[i], 1);
        mbar_init(&u_free[i], C::SOFT_WARPS + 4 + 2);   // softmax, issuers, V warps
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
    const uint32_t t_s = tmem + (uint32_t((warp & 3) * 32) << 16) + uint32_t(x * 256);
    const uint32_t t_p = t_s + C::COL_P, t_o = t_s + C::COL_O;
    uint8_t* stage = smem + C::OFF_OUT + warp * (32 * 64);
    uint32_t J = 0, slot = 0, turn = 0;   // steps of this row tile so far, place and turn of the unit ring
    // the O product of step i
    auto o_wait = [&](uint32_t i) -> bool { return prompt_wait(&o_done[NP * x + i % NP], (i / NP) & 1u, abort_flag, T); };
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
        // S, and P's place, free once the O product that read it last is complete (a
        // unit's first steps: the unit before has waited for its own)
        uint64_t* const there = &s_full[NS * x + J % NS];
        if (j < NP ? !prompt_wait(there, (J / NS) & 1u, abort_flag, T)
                   : !prompt_wait2(there, (J / NS) & 1u, &o_done[NP * x + J % NP], (J / NP + 1) & 1u, abort_flag, T)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t r0[32], r1[32];
        tmem_ld32_async(t_s + 64 * (J % NS), r0);
        tmem_ld32_async(t_s + 64 * (J % NS) + 32, r1);
        tmem_wait_ld(r0);
        tmem_wait_ld(r1);
        tc_fence_before();
        __syncwarp();
        mbar_arrive_lane0(&s_free[NS * x + J % NS], lane);
        if ((j + 1) * kPromptStep > min_end) {
          mask_cols(r0, end - j * kPromptStep);
          mask_cols(r1, end - j * kPromptStep - 32);
        }
        // P against the reference that is there; a step that it does not suit is
        // done again, so that no maximum is looked for in the others
        float sum;
        bool moves = j == 0, mine = moves;   // the warp does it again; this row's reference moves
#pragma unroll 1
        for (;;) {
          if (moves) {
            // P goes to the same columns again: stores to TMEM are not ordered among themselves
            if (j > 0) tmem_wait_st();
            const float top = fmaxf(cols_max(r0), cols_max(r1)) * p.c;
            float s = 1.f;
            if (mine && top > m) {   // no other row's: what a row gives does not depend on its neighbours
              s = ex2(m - top);   // 0 at the row's first visible keys
              l *= s;
              m = top;
            }
            if (j > 0) {   // once the O product of the step before is complete
              if (!o_wait(J - 1)) {
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
          uint32_t h[16];
          prompt_exp32<FP16>(r0, c2, s2, a0, h);
          tmem_st16(t_p + 32 * (J % NP), h);
          prompt_exp32<FP16>(r1, c2, s2, a1, h);
          tmem_st16(t_p + 32 * (J % NP) + 16, h);
          a0 = __fadd2_rn(a0, a1);
          sum = a0.x + a0.y;
          if (moves) break;
          mine = end > 0 && ((m == kNegInf && j * kPromptStep < end) || !(sum <= kPromptMost));
          moves = __any_sync(0xffffffffu, mine);
          if (!moves) break;
        }
        if (!ok) break;
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_lane0(&p_full[NP * x + J % NP], lane);
      }
      if (!ok) break;
      if (n > 0) {
        if (!o_wait(J - 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
      }
      const int head = u.kvh * p.G + row % p.G;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const bool bad = s_bad[slot] != 0 && row_ok && l != 0.f;
      const float lse2 = l == 0.f ? kNegInf : m + (log2f(l) - kLift);
      const bool part = p.part_lse != nullptr;
      int64_t at;   // of the row's results, -1: not written
      if (part) {
        const int64_t r = (int64_t(u.chunk) * p.Tq + tok) * p.H + head;
        if (row_ok) p.part_lse[r] = lse2;
        at = row_ok && l != 0.f ? r * D : -1;
      } else {
        if (row_ok && p.lse != nullptr) p.lse[int64_t(head) * p.Tq + tok] = lse2 * 0.69314718055994531f;
        at = row_ok ? int64_t(tok) * p.out_stride + int64_t(head) * D : -1;
      }
      // 64 bytes of each row at a time through shared memory, so that four lanes
      // store them together
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 16) {
        uint32_t o[16];
        if (n > 0) tmem_ld16(t_o + cc, o);
        float f[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = n > 0 && l != 0.f ? __uint_as_float(o[k]) * inv : 0.f;
        if (bad) {   // infinities and NaN of the V rows that this row sees
          const uint16_t* v = static_cast<const uint16_t*>(p.v) + int64_t(u.k_base + c0) * p.v_stride + int64_t(u.kvh) * D + cc;
          for (int j = u.fix * kPromptStep; j < end; ++j) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const float t = widen<FP16>(v[j * p.v_stride + k]);
              if (!(fabsf(t) < __builtin_huge_valf())) f[k] += t;
            }
          }
        }
        auto put = [&](int unit, uint4 w) {
          *reinterpret_cast<uint4*>(stage + lane * 64 + ((unit ^ ((lane >> 1) & 3)) << 4)) = w;
        };
        // `units` 16-byte pieces of each row to dst + row's place
        auto flush = [&](uint8_t* dst, int bytes, int units) {
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int i = 32 * k + lane, r = i / units, un = i - r * units;
            const int64_t to = __shfl_sync(0xffffffffu, at, r & 31);
            if (r < 32 && to >= 0)
              *reinterpret_cast<uint4*>(dst + to * bytes + 16 * un) =
                  *reinterpret_cast<const uint4*>(stage + r * 64 + ((un ^ ((r >> 1) & 3)) << 4));
          }
          __syncwarp();
        };
        if (part) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            put(k, make_uint4(__float_as_uint(f[4 * k]), __float_as_uint(f[4 * k + 1]), __float_as_uint(f[4 * k + 2]), __float_as_uint(f[4 * k + 3])));
          flush(reinterpret_cast<uint8_t*>(p.part_o + cc), 4, 4);
        } else {
          const int odd = (cc >> 4) & 1;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            put(2 * odd + k, make_uint4(pack16<FP16>(f[8 * k], f[8 * k + 1]), pack16<FP16>(f[8 * k + 2], f[8 * k + 3]),
                                        pack16<FP16>(f[8 * k + 4], f[8 * k + 5]), pack16<FP16>(f[8 * k + 6], f[8 * k + 7])));
          if (odd) flush(reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.out) + cc - 16), 2, 4);
          else if (cc + 16 == D) flush(reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.out) + cc), 2, 2);
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
    // A warp for each product of a row tile: with one for both, the next S product
    // waited behind the O product's issue (300 clocks of every step).
    const int who = __shfl_sync(0xffffffffu, warp, 0) - C::MMA_WARP;
    const int x = who & 1;
    const bool second = who >= 2;   // O += P V
    const uint32_t t_s = __shfl_sync(0xffffffffu, tmem, 0) + uint32_t(x * 256);
    const uint32_t t_p = t_s + C::COL_P, t_o = t_s + C::COL_O;
    uint32_t J = 0, st = 0, par = 0, slot = 0, turn = 0;   // steps of this row tile; stage of K or V and its turn; unit ring
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
      if (!second) {
        constexpr uint32_t kIdS = idesc_f16_f32(kTile, kPromptStep, false, !FP16);
        // advanced by (bytes >> 4)
        const uint64_t dq = smem_desc(smem_u32(smem + C::OFF_Q) + x * C::Q_BYTES, 2, 1024);
        const uint64_t dk = smem_desc(smem_u32(smem + C::OFF_K), 2, 1024);
        if (n > 0) ok = prompt_wait(&q_full[x], live & 1u, abort_flag, T);
        for (int j = 0; j < steps && ok; ++j) {
          ok = prompt_wait(&k_full[st], par, abort_flag, T);
          if (!ok) break;
          if (j < n) {
            const uint32_t at = J + j, place = at % NS;
            ok = at < NS || prompt_wait(&s_free[NS * x + place], (at / NS + 1) & 1u, abort_flag, T);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t a = (kk >> 2) * (kTile * 128) + (kk & 3) * 32, b = (kk >> 2) * (kPromptStep * 128) + (kk & 3) * 32;
              mma_ss_elect(t_s + 64 * place, dq + (a >> 4), dk + ((st * C::ST_BYTES + b) >> 4), kIdS, kk > 0);
            }
            commit_elect(&s_full[NS * x + place]);
            commit_elect(&k_free[st]);
            if (j == n - 1) commit_elect(&q_free[x]);
          } else {   // steps that this row tile does not see are only let go
            mbar_arrive_lane0(&k_free[st], lane);
          }
          if (++st == KS) {
            st = 0;
            par ^= 1u;
          }
        }
      } else {
        constexpr uint32_t kIdO = idesc_f16_f32(kTile, D, true, !FP16);
        const uint64_t dv = smem_desc_mn(smem_u32(smem + C::OFF_V), kPromptStep * 128, 1024);
        for (int j = 0; j < steps && ok; ++j) {
          ok = prompt_wait(&v_full[st], par, abort_flag, T);
          if (!ok) break;
          if (j < n) {
            const uint32_t at = J + j, place = at % NP;
            ok = prompt_wait(&p_full[NP * x + place], (at / NP) & 1u, abort_flag, T) &&
                 (j > 0 || live == 0 || prompt_wait(&o_free[x], (live - 1) & 1u, abort_flag, T));
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kPromptStep / 16; ++kk)
              mma_ts_elect(t_o, t_p + 32 * place + 8 * kk, dv + ((st * C::ST_BYTES + kk * 2048) >> 4), kIdO, j > 0 || kk > 0);
            commit_elect(&o_done[NP * x + place]);
            commit_elect(&v_free[st]);
          } else {
            mbar_arrive_lane0(&v_free[st], lane);
          }
          if (++st == KS) {
            st = 0;
            par ^= 1u;
          }
        }
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
    commit_elect(&drained[who]);
    wait_drain(&drained[who], 0, T);
  } else if (warp == C::LOAD_WARP) {
    // ------------------------------------------------------------ producer
    const int64_t per = int64_t(p.Hkv) * p.chunks;   // units of a block of rows
    int first = 0;                                   // segments [first, first + 32) in order,
    int64_t before = 0;                              // units of the ones before
    uint32_t ks = 0, qn[2] = {0, 0}, slot = 0, turn = 0;
    bool ok = true;
    for (int64_t round = 0; ok; ++round) {
      // There and back, so that no CTA has the longer unit of every round; from a
      // counter where there are many, since their times differ.
      int64_t i = round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      if (p.next != nullptr && round > 0) {
        int taken = 0;
        if (lane == 0) taken = atomicAdd(p.next, 1);
        i = int64_t(gridDim.x) + __shfl_sync(0xffffffffu, taken, 0);
      }
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
          if (!att_segment_ok(g, qa, nq, ka, nk, p.max_q, p.max_k, p.Tq, p.Tk)) {
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
        // the last rows see most keys; in chunks, blocks of two row tiles come first
        const int b = p.chunks > 1 ? int(blk) : (nq - 1) / (2 * p.tt) - int(blk);
        u.tok0 = qa + b * 2 * p.tt;
        u.tok_end = min(qa + nq, u.tok0 + 2 * p.tt);
        u.k_base = ka;
        u.lim = p.causal ? nk - nq + 1 - qa : nk;
        auto seen = [&](int tok) { return max(min(u.lim + (p.causal ? tok : 0), nk), 0); };
        const int all = seen(u.tok_end - 1);
        const int keys = u.tok0 + p.tt < u.tok_end ? p.keys : p.keys_one;
        u.c0 = int(min(int64_t(u.chunk) * keys, int64_t(all)));
        u.k1 = int(min(int64_t(u.c0) + keys, int64_t(all)));
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
          // this warp's half of the rows, the pieces of a row in any order
          const int left = u.k1 - u.c0 - j * kPromptStep;   // keys that some row sees
          uint4* tile = reinterpret_cast<uint4*>(smem + C::OFF_V + st * C::ST_BYTES) + (warp - C::FIX_WARP) * (kPromptStep / 2) * 8;
          const int first = (warp - C::FIX_WARP) * (kPromptStep / 2);
          uint32_t found = 0;
#pragma unroll
          for (int cc = 0; cc < C::DC; ++cc) {
#pragma unroll
            for (int i = 0; i < kPromptStep / 2 * 8 / 32; ++i) {
              uint4* at = tile + cc * (kPromptStep * 8) + 32 * i + lane;
              if (first + 4 * i + (lane >> 3) >= left) *at = make_uint4(0, 0, 0, 0);
              const uint4 w = *at;
              found |= not_finite<FP16>(w.x) | not_finite<FP16>(w.y) | not_finite<FP16>(w.z) | not_finite<FP16>(w.w);
            }
          }
          if (found & 0x80008000u) {
            s_bad[slot] = 1;
            for (int i = lane; i < C::DC * (kPromptStep / 2) * 8; i += 32) {
              uint32_t* at = reinterpret_cast<uint32_t*>(tile + (i >> 8) * (kPromptStep * 8) + (i & 255));
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t b = not_finite<FP16>(at[k]);
                at[k] &= ((b & 0x8000u) ? 0u : 0xFFFFu) | ((b & 0x80000000u) ? 0u : 0xFFFF0000u);
              }
            }
          }
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
