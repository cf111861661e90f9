// Rotation of Q and K by positions with several axes (time or image, row,
// column): the step before importance scoring in a vision encoder, and before
// the cache write and attention in the language model, on the position ids
// that the compaction keeps. No page of the sources has code for it; the
// dynamic vision-token compression article (section 3.2) asks that original
// spatial indices and position ids survive pruning, which is what it reads.
//
// (a, b) -> (a cos - b sin, b cos + a sin) per pair; the inverse rotation is
// its transpose, so it is also the gradient.
//
// HBM-bound: every element is read once and written once. A warp takes one
// token (or a share of its heads when there are few tokens); its lanes compute
// the token's angles once, into shared memory, while the first rows are on
// their way. The rows are then cut into pieces of two halves of up to 16 bytes
// that go round the lanes, so no lane idles whatever the head dimension, up to
// three pieces loaded before the first is stored.
//
// 61,385 tokens, 16 + 16 heads of 80, bf16 (629 MB): 110 us, 5.7 TB/s, 84% of
// the copy rate (one row per group of lanes: 227 us); 16,384 tokens, 16 + 8 heads
// of 128, fp32, turned back (403 MB): 71 us, 83%; 64 tokens: 2.5 us.
#include "launch_util.cuh"
#include "rope.cuh"

namespace tsel {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

template <typename T, int V>
__global__ void __launch_bounds__(kRopeThreads, 3) rope_kernel(const RopeParams p) {
  constexpr int kRopeBatch = sizeof(T) * V > 16 ? 2 : 3;   // pieces a lane loads before it stores any
  __shared__ __align__(16) float s_cs[kRopeWarps][2 * kRopeMaxPairs];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = int64_t(blockIdx.x) * kRopeWarps + warp;   // token; blockIdx.y: share of its heads
  if (t >= p.total) return;
  const int items = p.d / (2 * V);
  const int rows = p.H + p.Hkv;
  const int r0 = int(blockIdx.y) * p.per;
  const int pieces = max(min(p.per, rows - r0), 0) * items;
  float* cs = s_cs[warp];
  const bool adjacent = p.adjacent != 0;
  const int gap = adjacent ? V : p.num_pairs;   // from a turned piece's first half to its second
  // row r of the token: q rows first, then k rows (their base is H rows back)
  const T* q = static_cast<const T*>(p.q) + t * p.q_stride;
  const T* k = static_cast<const T*>(p.k) + (t * p.k_stride - int64_t(p.H) * p.d);
  T* qo = static_cast<T*>(p.q_out) + t * p.q_out_stride;
  T* ko = static_cast<T*>(p.k_out) + (t * p.k_out_stride - int64_t(p.H) * p.d);
  const int k_from = p.H * p.d;
  const float inv_items = 1.f / float(items);
  // rounds of at most kRopeBatch pieces per lane, of equal size
  const int steps = (pieces + 31) >> 5, rounds = (steps + kRopeBatch - 1) / kRopeBatch;
  const int batch = rounds > 0 ? (steps + rounds - 1) / rounds : 0;
  for (int round = 0; round < rounds; ++round) {
    Vec<T, V> a[kRopeBatch], b[kRopeBatch];
    int item[kRopeBatch], off[kRopeBatch];   // off: of the first half, in the token's rows; -1 none
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      const int n = (round * batch + i) * 32 + lane;
      off[i] = -1;
      if (i < batch && n < pieces) {
        const int rr = int((float(n) + 0.5f) * inv_items);   // n / items: both below 2^16
        item[i] = n - rr * items;
        const bool turned = item[i] * V < p.num_pairs;
        off[i] = (r0 + rr) * p.d + item[i] * (turned && !adjacent ? V : 2 * V);
        const T* src = (off[i] < k_from ? q : k) + off[i];
        a[i].load(src);
        b[i].load(src + (turned ? gap : V));
      }
    }
    if (round == 0) {   // the angles, while the first rows are on their way
      if (rope_angles(cs, p.table, p.num_pairs, p.pos + t * p.pos_dim, p.pos_dim, p.inverse ? -1.f : 1.f))
        set_status(p.status, TSEL_DEV_POSITIONS);
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < kRopeBatch; ++i) {
      if (off[i] < 0) continue;
      const bool turned = item[i] * V < p.num_pairs;
      if (turned) {
        float c[V], s[V], fa[V], fb[V];
        rope_fetch<V>(cs, item[i], c, s);
        a[i].get(fa);
        b[i].get(fb);
        rope_turn<V>(fa, fb, c, s, adjacent);
        a[i].set(fa);
        b[i].set(fb);
      }
      T* dst = (off[i] < k_from ? qo : ko) + off[i];
      a[i].store(dst);
      b[i].store(dst + (turned ? gap : V));
    }
  }
}

template <typename T, int V>
cudaError_t launch_rope_t(RopeParams p, int num_sms, cudaStream_t stream) {
  // Enough warps to fill the device from few tokens: a token's heads are
  // shared out until there are about 16 warps per SM, each with a piece or more
  // per lane.
  const int rows = p.H + p.Hkv;
  const int max_parts = int(ceil_div(int64_t(rows) * (p.d / (2 * V)), 32));
  const int64_t want = ceil_div(int64_t(num_sms) * 16, p.total);
  int parts = int(want < 1 ? 1 : (want > max_parts ? max_parts : want));
  if (parts > rows) parts = rows;
  p.per = int(ceil_div(rows, parts));
  const dim3 grid(unsigned(ceil_div(p.total, kRopeWarps)), unsigned(ceil_div(rows, p.per)));
  return launch_kernel(rope_kernel<T, V>, grid, kRopeThreads, 0, stream, 1, p);
}

template <typename T>
cudaError_t launch_rope_v(const RopeParams& p, int num_sms, cudaStream_t stream) {
  switch (rope_vec(p.d, p.num_pairs)) {
    case 8: return launch_rope_t<T, 8>(p, num_sms, stream);
    case 4: return launch_rope_t<T, 4>(p, num_sms, stream);
    case 2: return launch_rope_t<T, 2>(p, num_sms, stream);
    default: return launch_rope_t<T, 1>(p, num_sms, stream);
  }
}

}  // namespace

cudaError_t launch_rope(int dtype, const RopeParams& p, int num_sms, cudaStream_t stream) {
  switch (dtype) {
    case TSEL_BF16: return launch_rope_v<__nv_bfloat16>(p, num_sms, stream);
    case TSEL_FP16: return launch_rope_v<__half>(p, num_sms, stream);
    default: return launch_rope_v<float>(p, num_sms, stream);
  }
}

}  // namespace tsel
