// Attention of a chunk of new tokens over a paged cache:
//     out = sum_j e^{s_j} v_j / sum_j e^{s_j},  s_j = scale q . k_j,
// over the keys j a row may see (all of the sequence, or up to its own token), optionally joined
// with a part (out0, lse0) attended elsewhere, which counts as one more key of score lse0 and
// value out0. One warp a query row, lane i features 4 i .. 4 i + 3, one key at a time with a
// running maximum and sum.
#include "../paged.h"

namespace jolt {
namespace {

template <typename T>
__device__ __forceinline__ void get4(const T* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const T* h = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = (float)h[i];
}

template <typename T>
__global__ void __launch_bounds__(128) k_paged_attention(const PagedAttnArgs a) {
  const int tok = blockIdx.x, lane = threadIdx.x & 31;
  const int qh = blockIdx.y * 4 + (threadIdx.x >> 5);
  __shared__ int seq_s;
  if (threadIdx.x == 0) seq_s = -1;
  __syncthreads();
  for (int s = threadIdx.x; s < a.b.num_seqs; s += 128)
    if (tok >= a.b.q_start[s] && tok < a.b.q_start[s + 1]) seq_s = s;
  __syncthreads();
  const int s = seq_s;
  if (s < 0 || qh >= a.Hq) return;
  const SeqView v = seq_view(a.b, s);
  if (v.n == 0) return;
  const int h = qh / (a.Hq / a.b.heads), i = tok - v.q0;
  const int lim = a.causal ? v.len - v.n + i : v.len - 1;
  float q[4], o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  get4(reinterpret_cast<const T*>(a.Q) + tok * a.q_ts + qh * a.q_hs + 4 * lane, q);
  float m = -INFINITY, l = 0.0f;
  const int64_t row = (int64_t)tok * a.Hq + qh;
  if (a.pre_lse) {
    m = a.pre_lse[row];
    if (m != -INFINITY) {
      l = 1.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = a.pre_out[row * kD + 4 * lane + e];
    }
  }
  for (int j = 0; j <= lim; ++j) {
    const int pg = page_of(a.b, s, j);
    if (pg < 0) continue;
    const int64_t off = (((int64_t)pg * a.b.heads + h) * a.b.page_size + j % a.b.page_size) * kD + 4 * lane;
    float k[4];
    get4(reinterpret_cast<const T*>(a.K) + off, k);
    float d = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) d = fmaf(q[e], k[e], d);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) d += __shfl_xor_sync(0xffffffffu, d, w);
    d *= a.scale;
    const float mn = fmaxf(m, d), f = m == -INFINITY ? 0.0f : expf(m - mn), p = expf(d - mn);
    get4(reinterpret_cast<const T*>(a.V) + off, k);
    l = fmaf(l, f, p);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = fmaf(o[e], f, p * k[e]);
    m = mn;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  T* out = reinterpret_cast<T*>(a.out) + row * kD + 4 * lane;
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = (T)(o[e] * inv);
  if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t paged_attention(const PagedAttnArgs& a, cudaStream_t s) {
  if (a.b.total_q <= 0 || a.b.num_seqs <= 0) return cudaSuccess;
  const dim3 grid(a.b.total_q, (a.Hq + 3) / 4);
  if (a.dtype == JOLT_BF16) k_paged_attention<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
  else k_paged_attention<__half><<<grid, 128, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace jolt
