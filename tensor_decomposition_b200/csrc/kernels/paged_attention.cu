// Attention of a chunk of new tokens over a paged cache:
//     out = sum_j e^{s_j} v_j / sum_j e^{s_j},  s_j = scale q . k_j,
// over the keys j a row may see (all of the sequence, or up to its own token), optionally joined
// with a part (out0, lse0) attended elsewhere, which counts as one more key of score lse0 and
// value out0. One warp a query row, lane i features 4 i .. 4 i + 3, one key at a time with a
// running maximum and sum.
#include "paged_attention.cuh"

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

namespace {
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t o_bytes(const AttnPlan& p) { return up256((size_t)p.grid * 2 * p.rows * kD * sizeof(float)); }
size_t ml_bytes(const AttnPlan& p) { return up256((size_t)p.grid * 2 * p.rows * sizeof(float2)); }
}  // namespace

// Rows of a chunk that read one KV head: up to 16 run in the kernel for few rows.
AttnPlan paged_attention_plan(const PagedAttnArgs& a, int sms) {
  AttnPlan p;
  const int64_t tokens = (int64_t)a.b.max_pages * a.b.page_size;
  p.decode = (int64_t)a.b.max_q * (a.Hq / a.b.heads) <= 16;
  if (!p.decode) return p;
  const int64_t units = std::max<int64_t>(1, (tokens + 63) / 64) * a.b.heads * a.b.num_seqs;
  p.grid = (int)std::min<int64_t>(2 * (int64_t)sms, units);
  p.rows = 16;
  p.bytes = o_bytes(p) + ml_bytes(p) + up256(p.grid * sizeof(pattn::Split));
  return p;
}

cudaError_t paged_attention(const PagedAttnArgs& a, const AttnPlan& p, void* scratch, cudaStream_t s) {
  if (p.decode) {
    pattn::Workspace w;
    char* at = static_cast<char*>(scratch);
    w.o = reinterpret_cast<float*>(at);
    w.ml = reinterpret_cast<float2*>(at + o_bytes(p));
    w.list = reinterpret_cast<pattn::Split*>(at + o_bytes(p) + ml_bytes(p));
    w.rows = p.rows;
    return attn_decode(a, p, w, s);
  }
  const dim3 grid(a.b.total_q, (a.Hq + 3) / 4);
  if (a.dtype == JOLT_BF16) k_paged_attention<__nv_bfloat16><<<grid, 128, 0, s>>>(a);
  else k_paged_attention<__half><<<grid, 128, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace jolt
