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
// token (or a share of its heads when there are few tokens); a lane keeps the
// cosines and sines of its pairs and walks the token's heads with them, the
// loads of up to four rows issued before their stores. The angles are computed
// once per token and lane, not per head.
#include "launch_util.cuh"
#include "rope.cuh"

namespace tsel {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;   // rows a lane loads before it stores any

template <typename T, int V>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int items = p.d / (2 * V);
  int lpr = 1;   // lanes per row
  while (lpr < items && lpr < 32) lpr <<= 1;
  const int sub = lane / lpr, subs = 32 / lpr, l0 = lane % lpr;
  const int rows = p.H + p.Hkv;
  const int per = (rows + p.parts - 1) / p.parts;
  const int64_t units = int64_t(p.total) * p.parts;
  const int64_t nwarps = int64_t(gridDim.x) * (kRopeThreads / 32);
  const T* q = static_cast<const T*>(p.q);
  const T* k = static_cast<const T*>(p.k);
  T* qo = static_cast<T*>(p.q_out);
  T* ko = static_cast<T*>(p.k_out);
  for (int64_t u = (int64_t(blockIdx.x) * kRopeThreads + threadIdx.x) >> 5; u < units; u += nwarps) {
    const int64_t t = u / p.parts;
    const int r0 = int(u % p.parts) * per;
    const int r1 = min(r0 + per, rows);
    for (int item = l0; item < items; item += lpr) {
      int o1, o2;
      rope_item(item, V, p.num_pairs, p.adjacent != 0, o1, o2);
      const bool turned = item * V < p.num_pairs;
      float c[V], s[V];
      if (turned) {
        bool bad = false;
        rope_angles<V>(p.table, item, p.pos + t * p.pos_dim, p.pos_dim, c, s, bad);
        if (bad) set_status(p.status, TSEL_DEV_POSITIONS);
        if (p.inverse) {
#pragma unroll
          for (int j = 0; j < V; ++j) s[j] = -s[j];
        }
      }
      for (int base = r0 + sub; base < r1; base += subs * kRopeRows) {
        Vec<T, V> a[kRopeRows], b[kRopeRows];
#pragma unroll
        for (int i = 0; i < kRopeRows; ++i) {
          const int r = base + i * subs;
          if (r < r1) {
            const T* src = r < p.H ? q + t * p.q_stride + int64_t(r) * p.d
                                   : k + t * p.k_stride + int64_t(r - p.H) * p.d;
            a[i].load(src + o1);
            b[i].load(src + o2);
          }
        }
#pragma unroll
        for (int i = 0; i < kRopeRows; ++i) {
          const int r = base + i * subs;
          if (r < r1) {
            if (turned) {
              float fa[V], fb[V];
#pragma unroll
              for (int j = 0; j < V; ++j) {
                fa[j] = to_f32(a[i].e[j]);
                fb[j] = to_f32(b[i].e[j]);
              }
              rope_turn<V>(fa, fb, c, s, p.adjacent != 0);
#pragma unroll
              for (int j = 0; j < V; ++j) {
                a[i].e[j] = from_f32<T>(fa[j]);
                b[i].e[j] = from_f32<T>(fb[j]);
              }
            }
            T* dst = r < p.H ? qo + t * p.q_out_stride + int64_t(r) * p.d
                             : ko + t * p.k_out_stride + int64_t(r - p.H) * p.d;
            a[i].store(dst + o1);
            b[i].store(dst + o2);
          }
        }
      }
    }
  }
}

template <typename T, int V>
cudaError_t launch_rope_t(RopeParams p, int num_sms, cudaStream_t stream) {
  // Enough warps to fill the device from few tokens: a token's heads are
  // shared out until there are about 16 warps per SM, each with a row or more
  // per lane group.
  const int rows = p.H + p.Hkv;
  int lpr = 1;
  while (lpr < p.d / (2 * V) && lpr < 32) lpr <<= 1;
  const int max_parts = int(ceil_div(rows, 32 / lpr));
  const int64_t want = ceil_div(int64_t(num_sms) * 16, p.total);
  p.parts = int(want < 1 ? 1 : (want > max_parts ? max_parts : want));
  const int64_t warps = int64_t(p.total) * p.parts;
  int64_t blocks = ceil_div(warps, kRopeThreads / 32);
  const int64_t most = int64_t(num_sms) * 8;
  if (blocks > most) blocks = most;
  return launch_kernel(rope_kernel<T, V>, dim3(unsigned(blocks)), kRopeThreads, 0, stream, 1, p);
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
