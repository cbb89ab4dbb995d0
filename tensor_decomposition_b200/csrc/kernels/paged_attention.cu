// Attention of a chunk of new tokens over a paged cache:
//     out = sum_j e^{s_j} v_j / sum_j e^{s_j},  s_j = scale q . k_j,
// over the keys j a row may see (all of the sequence, or up to its own token), optionally joined
// with a part (out0, lse0) attended elsewhere, which counts as one more key of score lse0 and
// value out0. Two kernels do the work, one for few rows a KV head (paged_attention_decode.cu), bound
// by HBM, one for many (paged_attention_chunk.cu), bound by the tensor pipe; both divide it into
// equal shares a CTA, whatever the lengths are (but for small calls of few rows, which clusters take item by
// item). This file chooses, and combines the parts of what a share's end has cut.
#include "paged_attention.cuh"

namespace jolt {
namespace {

using namespace pattn;

// The items that lie in several CTAs' shares, the parts weighted by their maxima. Parts of up to 32
// rows lie row by row: four rows a CTA, four warps a row (one warp a row took 0.25 us a part).
constexpr int kSubs = 4;
template <typename T>
__global__ void __launch_bounds__(512) k_attn_combine(const PagedAttnArgs a, const Workspace ws) {
  __shared__ float4 y_s[4][kSubs][32];
  __shared__ float2 ml_s[4][kSubs];
  grid_release();
  grid_wait();
  const Split sp = ws.list[blockIdx.x];
  if (sp.s < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp & 3, rw = warp >> 2;
  const int c0 = blockIdx.x, parts = sp.c_last - c0 + 1;
  const int g = a.g.d, R = sp.rows;
  const int r = blockIdx.y * 4 + rw;
  if ((int)blockIdx.y * 4 >= R) return;
  const int tok = a.g.quot(r);
  const int64_t row = (int64_t)(sp.q0 + tok) * a.Hq + sp.h * g + r - tok * g;
  Prefix pre{};
  if (r < R && sub == 0) pre = load_prefix(a, row, lane);
  float mx = -INFINITY, ls = 0.0f;
  float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (r < R) {
    for (int b0 = 0; b0 < parts; b0 += 8 * kSubs) {   // eight parts in flight
      float2 p[8];
      float4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = b0 + sub + kSubs * i;
        p[i] = make_float2(-INFINITY, 0.0f);
        x[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < parts) {
          const int64_t at = ((int64_t)(c0 + c) * 2 + (c == 0 ? sp.slot : 0)) * ws.rows + r;
          p[i] = ws.ml[at];
          x[i] = *reinterpret_cast<const float4*>(ws.o + at * kD + 4 * lane);
        }
      }
      float mn = mx;
#pragma unroll
      for (int i = 0; i < 8; ++i) mn = fmaxf(mn, p[i].x);
      const float f0 = rescale(mx, mn);
      mx = mn;
      ls *= f0;
      y.x *= f0; y.y *= f0; y.z *= f0; y.w *= f0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = rescale(p[i].x, mn);
        ls = fmaf(p[i].y, f, ls);
        y.x = fmaf(x[i].x, f, y.x);
        y.y = fmaf(x[i].y, f, y.y);
        y.z = fmaf(x[i].z, f, y.z);
        y.w = fmaf(x[i].w, f, y.w);
      }
    }
    y_s[rw][sub][lane] = y;
    if (lane == 0) ml_s[rw][sub] = make_float2(mx, ls);
  }
  __syncthreads();
  if (r >= R || sub != 0) return;
  float mn = mx;
#pragma unroll
  for (int i = 1; i < kSubs; ++i) mn = fmaxf(mn, ml_s[rw][i].x);
  y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  ls = 0.0f;
#pragma unroll
  for (int i = 0; i < kSubs; ++i) {
    const float f = rescale(ml_s[rw][i].x, mn);
    const float4 x = y_s[rw][i][lane];
    ls = fmaf(ml_s[rw][i].y, f, ls);
    y.x = fmaf(x.x, f, y.x);
    y.y = fmaf(x.y, f, y.y);
    y.z = fmaf(x.z, f, y.z);
    y.w = fmaf(x.w, f, y.w);
  }
  finish_row<T>(a, row, lane, y, mn, ls, pre);
}

// The same for blocks of 256 rows, whose parts lie in blocks of four features with the rows next to one
// another: a CTA takes 32 rows, a lane a row and its warp every eighth block of features, and the rows
// come together in shared memory.
constexpr int kBlockWarps = 8;
template <typename T>
__global__ void __launch_bounds__(32 * kBlockWarps) k_attn_combine_blocks(const PagedAttnArgs a, const Workspace ws) {
  constexpr int kN = 32 / kBlockWarps;   // blocks of features of a warp, and its rows
  __shared__ float4 y_s[32][33];
  grid_release();
  grid_wait();
  const Split sp = ws.list[blockIdx.x];
  if (sp.s < 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = blockIdx.x, parts = sp.c_last - c0 + 1;
  const int g = a.g.d, rb = blockIdx.y * 32, R = sp.rows;
  if (rb >= R) return;
  const bool in = rb + lane < R;
  const float4* o = reinterpret_cast<const float4*>(ws.o);
  int64_t row[kN];
  Prefix pre[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int r = sp.m * 256 + min(rb + warp + kBlockWarps * k, R - 1);
    const int tok = a.g.quot(r);
    row[k] = (int64_t)(sp.q0 + tok) * a.Hq + sp.h * g + r - tok * g;
    pre[k] = load_prefix(a, row[k], lane);
  }
  float mx = -INFINITY, ls = 0.0f;
  float4 y[kN] = {};
#pragma unroll 4
  for (int c = 0; c < parts; ++c) {
    if (!in) break;
    const int64_t slot = (int64_t)(c0 + c) * 2 + (c == 0 ? sp.slot : 0);
    const float2 p = ws.ml[slot * 256 + rb + lane];
    float4 x[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) x[k] = o[(slot * 32 + warp + kBlockWarps * k) * 256 + rb + lane];
    const float mn = fmaxf(mx, p.x);
    const float f0 = rescale(mx, mn), f = rescale(p.x, mn);
    mx = mn;
    ls = fmaf(ls, f0, p.y * f);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      y[k].x = fmaf(y[k].x, f0, x[k].x * f);
      y[k].y = fmaf(y[k].y, f0, x[k].y * f);
      y[k].z = fmaf(y[k].z, f0, x[k].z * f);
      y[k].w = fmaf(y[k].w, f0, x[k].w * f);
    }
  }
#pragma unroll
  for (int k = 0; k < kN; ++k) y_s[lane][warp + kBlockWarps * k] = y[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int i = warp + kBlockWarps * k;
    const float m1 = __shfl_sync(0xffffffffu, mx, i), l1 = __shfl_sync(0xffffffffu, ls, i);
    if (rb + i < R) finish_row<T>(a, row[k], lane, y_s[i][lane], m1, l1, pre[k]);
  }
}

template <typename T>
cudaError_t combine(const PagedAttnArgs& a, const AttnPlan& p, const Workspace& w, cudaStream_t s) {
  if (p.decode) return launch_early(k_attn_combine<T>, dim3(p.grid, (p.most + 3) / 4), dim3(512), 0, 1, s, a, w);
  return launch_early(k_attn_combine_blocks<T>, dim3(p.grid, (p.most + 31) / 32), dim3(32 * kBlockWarps), 0, 1, s, a, w);
}

__global__ void k_take_status(int32_t* word, int32_t* out) { *out = atomicExch(word, 0); }

size_t up256(size_t x) { return (x + 255) / 256 * 256; }
size_t o_bytes(const AttnPlan& p) { return up256((size_t)p.grid * 2 * p.rows * kD * sizeof(float)); }
size_t ml_bytes(const AttnPlan& p) { return up256((size_t)p.grid * 2 * p.rows * sizeof(float2)); }

}  // namespace

cudaError_t take_status(int32_t* word, int32_t* out, cudaStream_t s) {
  k_take_status<<<1, 1, 0, s>>>(word, out);
  note_launch();
  return cudaGetLastError();
}

// Up to 8 rows of a chunk reading one KV head run in the kernel for few rows; 9 to 32 do where there are few
// items and short caches, whose fewer steps to the first output count (32 items of 16 rows: 8.1, 8.9, 13.6, 19.6
// and 31.2 us for 128, 512, 2048, 4096 and 6000 keys, in the other kernel 15.3, 16.5, 18.5, 21.5 and 25.8; of 20
// rows: 11.5, 14.9, 22.8 for 128, 512, 2048 and 15.4, 16.9, 18.8; 128 items of 16 rows: 16.9, 25.9, 42, 99 for 128,
// 512, 2048, 8192 and 16.2, 18.1, 35, 93). Both round the output alone up to 128 rows, so the choice is one of time.
// Clusters of 8 CTAs, one for each item, combine by themselves where they all run at once (33 and more do not: 9.0 us
// instead of 5.9) and the table holds few keys (8 items: 5.9 instead of 7.4 us at 1024 keys, 11.8 and 12.2 at 4096, 19.4
// and 14.4 at 8192; one item: 5.9 and 7.7, 11.7 and 9.6, 19.3 and 12.0; 32 items: 7.7 and 10.8, 15.0 and 16.3, 26.4 and
// 29.6). An item's eight CTAs have it whatever the others' lengths are, so longer tables are not for them, where one
// sequence may have nearly all the keys (32 items of 131072, 100, 100 and 100 keys: 271 us, in shares 94; 8192, 100, 100
// and 100: 22 and 15). 9 to 16 rows are in the kernel for few rows where they are in clusters.
constexpr int kTeamTokens = 4096, kTeamItems = 32, kFewTokens32 = 512;
AttnPlan paged_attention_plan(const PagedAttnArgs& a, int sms) {
  AttnPlan p;
  const int64_t tokens = (int64_t)a.b.max_pages * a.b.page_size, rows = (int64_t)std::min(a.b.max_q, a.b.total_q) * (a.Hq / a.b.heads);
  const int64_t items = (int64_t)a.b.heads * a.b.num_seqs;
  p.decode = rows <= 8 || (rows <= 32 && items <= kTeamItems && tokens <= (rows <= 16 ? kTeamTokens : kFewTokens32));
  p.rows = !p.decode ? 256 : rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
  p.most = (int)std::max<int64_t>(1, std::min<int64_t>(rows, p.rows));
  const int fit = p.rows <= 16 ? kTeamItems : kTeamItems / 2;   // two CTAs an SM, or one
  if (p.decode && items <= fit && tokens <= kTeamTokens) {
    p.team = 1;
    p.grid = (int)items * 8;
    return p;
  }
  const int unit = p.decode ? 64 : 128;
  const int64_t per_item = std::max<int64_t>(1, (tokens + unit - 1) / unit) * std::max<int64_t>(1, (rows + p.rows - 1) / p.rows);
  const int64_t most = (p.rows <= 16 ? 3 : p.rows == 32 ? 2 : 1) * (int64_t)sms;
  p.grid = (int)std::min(most, std::min(most, per_item) * items);
  p.bytes = o_bytes(p) + ml_bytes(p) + up256(p.grid * sizeof(Split));
  return p;
}

cudaError_t paged_attention(const PagedAttnArgs& a, const AttnPlan& p, void* scratch, cudaStream_t s) {
  Workspace w;
  char* at = static_cast<char*>(scratch);
  w.o = reinterpret_cast<float*>(at);
  w.ml = reinterpret_cast<float2*>(at + o_bytes(p));
  w.list = reinterpret_cast<Split*>(at + o_bytes(p) + ml_bytes(p));
  w.rows = p.rows;
  const cudaError_t e = p.decode ? attn_decode(a, p, w, s) : attn_chunk(a, p, w, s);
  if (e != cudaSuccess || p.team) return e;
  return a.dtype == JOLT_BF16 ? combine<__nv_bfloat16>(a, p, w, s) : combine<__half>(a, p, w, s);
}

}  // namespace jolt
