// Rows of queries and keys normed and rotated by their position, and the append of keys and values
// to a paged cache. One row is the 128 features of one head of one token:
//     y = w * x / sqrt(mean(x^2) + eps)                        (left out without a weight),
//     (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = position * inv_freq[i],
// over the pairs j = i + rope_dim / 2 (half-split) or (2 i, 2 i + 1) (interleaved) of the first
// rope_dim features. All in float32 and rounded once; the angle is formed in float64 and reduced
// to a part of a turn there, since a float32 angle of position 10^5 is off by 10^-2 rad.
//
// Each row is read and written once, which bounds the kernel for long inputs (HBM); short inputs
// are bound by latency. A CTA takes a tile of tokens, up to 64 rows, 8 lanes a row (two 16-byte runs each) and
// up to four rows a lane in flight at once: with one token a CTA the append of 16 rows a token ran at 1.4
// TB/s, so it runs at 4.4 (tokens of 80 rows, a CTA each, at 5.0, in a short run 5.5). The tile's sines are computed once (a thread each, while the rows are on their
// way) and used by all heads from shared memory; the append's page lookup is one parallel pass over the
// batch's offsets instead of a search. (Persistent CTAs with a ring of asynchronous copies, and tiles of
// two to four times the rows, were 8 to 25 % slower.)
#include <algorithm>

#include "../paged.h"
#include "f32x2.cuh"

namespace jolt {
namespace {

using namespace f32x2;

constexpr int kThreads = 128;
constexpr int kLanes = 8;               // of a row: 16 features each
constexpr int kSlots = kThreads / kLanes;   // rows at a time
// Rows a slot keeps in flight. Where a tile has more rows than the slots hold at once (a token of more than 64
// rows), the next row is loaded as soon as one is taken up, and three do; else all are loaded first and used
// (16384 tokens of 80 rows: 121 us that way and 132 the other in a short run, 134 that way in a sustained one; 64
// tokens of 40 rows: 4.4 and 3.3 us).
template <bool kLong>
constexpr int kBatch = kLong ? 3 : 4;
constexpr int kRows = kSlots * kBatch<false>;   // of a tile, unless one token has more
constexpr int kCtas = 6;                // per SM
constexpr int kMaxTile = 16;            // tokens of a tile

// Elements of a row, as pairs.
__device__ __forceinline__ uint64_t wide(__nv_bfloat16, uint32_t v) {
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
  return pair_of(a.x, a.y);
}
__device__ __forceinline__ uint64_t wide(__half, uint32_t v) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return pair_of(a.x, a.y);
}
__device__ __forceinline__ uint32_t narrow(__nv_bfloat16, uint64_t p) {
  float x, y;
  unpair(p, x, y);
  const __nv_bfloat162 a = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&a);
}
__device__ __forceinline__ uint32_t narrow(__half, uint64_t p) {
  float x, y;
  unpair(p, x, y);
  const __half2 a = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&a);
}
template <typename T>
__device__ __forceinline__ void get8(T, const uint4& v, uint64_t* x) {
  x[0] = wide(T(), v.x);
  x[1] = wide(T(), v.y);
  x[2] = wide(T(), v.z);
  x[3] = wide(T(), v.w);
}
template <typename T>
__device__ __forceinline__ uint4 put8(T, const uint64_t* x) {
  return make_uint4(narrow(T(), x[0]), narrow(T(), x[1]), narrow(T(), x[2]), narrow(T(), x[3]));
}

struct RowsArgs {
  RowsIn A, B;       // A: queries, or the append's keys; B: keys, or the append's values
  RowsOut Ao, Bo;    // outputs (strides of a page row in the append)
  RopeArgs r;
  BatchView b;       // append only
  int32_t tokens, tile;
};

// A lane holds two runs of eight features of its row, from o0 and o1 on, such that it has both members
// of eight rotated pairs (angles 8 l .. 8 l + 7) or sixteen features behind the rotated ones.
template <typename T, bool kPaged, bool kInterleaved, bool kLong>
__global__ void __launch_bounds__(kThreads, kCtas) k_rope_rows(const RowsArgs a) {
  extern __shared__ __align__(16) float trig[];        // [tile][2][64] cosines and sines of the pairs
  __shared__ __align__(16) float w_s[2][kD];           // norm weights
  __shared__ int64_t dst_s[kMaxTile];                  // append: page row in elements from the pages' base; < 0: none
  __shared__ int seq_s[kMaxTile];                      // append: sequence (-1: none)
  grid_release();
  grid_wait();
  const int tid = threadIdx.x, slot = tid / kLanes, l = tid % kLanes;
  const int t0 = blockIdx.x * a.tile, nt = min(a.tile, a.tokens - t0);
  const int nA = a.A.heads, nR = a.A.heads + a.B.heads;
  const int step_t = kSlots / nR, step_r = kSlots % nR;
  const bool rot = a.r.inv_freq != nullptr;
  const bool normA = a.A.w != nullptr, normB = !kPaged && a.B.w != nullptr;
  const int h = a.r.rope_dim >> 1;
  const bool turned = 16 * l < a.r.rope_dim;
  const int o0 = kInterleaved || !turned ? 16 * l : 8 * l, o1 = kInterleaved || !turned ? 16 * l + 8 : 8 * l + h;

  // rows slot, slot + kSlots, ...: token i of the tile, row r of the token
  int i = slot / nR, r = slot - i * nR;
  auto advance = [&](int& ti, int& tr) {
    ti += step_t;
    tr += step_r;
    if (tr >= nR) {
      tr -= nR;
      ++ti;
    }
  };
  uint4 v[kBatch<kLong>][2] = {};
  int li = i, lr = r;        // the next row to load
  auto load = [&](uint4* x) {
    if (li >= nt) return;
    const int t = t0 + li;
    const T* src = lr < nA ? reinterpret_cast<const T*>(a.A.p) + (int64_t)t * a.A.ts + (int64_t)lr * a.A.hs
                           : reinterpret_cast<const T*>(a.B.p) + (int64_t)t * a.B.ts + (int64_t)(lr - nA) * a.B.hs;
    x[0] = *reinterpret_cast<const uint4*>(src + o0);
    x[1] = *reinterpret_cast<const uint4*>(src + o1);
    advance(li, lr);
  };
#pragma unroll
  for (int k = 0; k < kBatch<kLong>; ++k) load(v[k]);

  static_assert(kThreads >= kD, "a thread a weight");
  if (normA && tid < kD) w_s[0][tid] = (float)reinterpret_cast<const T*>(a.A.w)[tid];
  if (normB && tid < kD) w_s[1][tid] = (float)reinterpret_cast<const T*>(a.B.w)[tid];
  // place in its sequence's cache of token t of the tile, below 0 for none (the arrays are in L1 by then)
  auto place = [&](int t) {
    const int s = seq_s[t];
    return s < 0 ? -1 : a.b.kv_len[s] - (a.b.q_start[s + 1] - (t0 + t));
  };
  if (kPaged) {
    if (tid < kMaxTile) seq_s[tid] = -1;
    __syncthreads();
    for (int s = tid; s < a.b.num_seqs; s += kThreads) {
      const int q0 = a.b.q_start[s], q1 = a.b.q_start[s + 1];
      // (the first CTA looks at all of them, so that one whose bounds fit no tile is reported too)
      if (blockIdx.x != 0 && (q0 >= t0 + nt || q1 <= t0)) continue;
      const SeqView sv = seq_view(a.b, s);
      if (sv.n == 0) continue;
      // offsets that fall let several sequences claim a token: the last has it, and its place comes from that one alone
      for (int t = max(q0, t0); t < min(q1, t0 + nt); ++t) atomicMax(&seq_s[t - t0], s);
    }
    __syncthreads();
    if (tid >= kThreads - nt) {   // not the first threads: they have angles to make
      const int t = tid - (kThreads - nt), pos = place(t);
      int64_t d = -1;
      if (pos >= 0) {
        const int pg = page_of(a.b, seq_s[t], pos);
        if (pg >= 0) d = ((int64_t)pg * a.b.heads * a.b.page_size + pos - a.b.by_page.quot(pos) * a.b.page_size) * kD;
      }
      dst_s[t] = d;
    }
  }
  if (rot) {
    for (int u = tid; u < nt * h; u += kThreads) {
      const int t = u / h, f = u - t * h;
      const int pos = kPaged && !a.r.positions ? place(t) : a.r.positions[t0 + t];
      // parts of a turn, in float64 up to the last whole turn
      double turn = (double)pos * ((double)a.r.inv_freq[f] * 0.15915494309189533577);
      turn -= rint(turn);
      sincospif(2.0f * (float)turn, &trig[t * kD + 64 + f], &trig[t * kD + f]);
    }
  }
  __syncthreads();

  const uint32_t mask = 0xffu << (tid & 24);   // the lanes of a row, who take part in its sum
  for (;;) {
#pragma unroll
    for (int k = 0; k < kBatch<kLong>; ++k) {
      if (i >= nt) return;
      const bool isA = r < nA;
      uint4 y0 = v[k][0], y1 = v[k][1];
      if (kLong) load(v[k]);
      if (!kPaged || isA) {     // values of the append go out as they are
        uint64_t x[8];          // features o0 .. o0 + 7, o1 .. o1 + 7
        get8(T(), y0, x);
        get8(T(), y1, x + 4);
        if (isA ? normA : normB) {
          uint64_t q2 = mul2(x[0], x[0]);
#pragma unroll
          for (int e = 1; e < 8; ++e) q2 = fma2(x[e], x[e], q2);
          float q, qb;
          unpair(q2, q, qb);
          q += qb;
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) q += __shfl_xor_sync(mask, q, o, kLanes);
          const float f = rsqrtf(fmaf(q, 1.0f / kD, a.r.eps));
          const float* w = w_s[isA ? 0 : 1];
          const uint64_t f2 = pair_of(f, f);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 u = *reinterpret_cast<const float4*>(w + (e < 2 ? o0 : o1) + 4 * (e & 1));
            x[2 * e] = mul2(x[2 * e], mul2(f2, pair_of(u.x, u.y)));
            x[2 * e + 1] = mul2(x[2 * e + 1], mul2(f2, pair_of(u.z, u.w)));
          }
        }
        if (turned) {
#pragma unroll
          for (int d = 0; d < 2; ++d) {   // four pairs at a time
            const float4 c = *reinterpret_cast<const float4*>(trig + i * kD + 8 * l + 4 * d);
            const float4 s = *reinterpret_cast<const float4*>(trig + i * kD + 64 + 8 * l + 4 * d);
            if (kInterleaved) {     // (u, v) -> (u, v) c + (-v, u) s
              const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float u, w;
                unpair(x[4 * d + e], u, w);
                x[4 * d + e] = fma2(pair_of(w, u), pair_of(-sn[e], sn[e]), mul2(x[4 * d + e], pair_of(cs[e], cs[e])));
              }
            } else {
              const uint64_t c2[2] = {pair_of(c.x, c.y), pair_of(c.z, c.w)}, s2[2] = {pair_of(s.x, s.y), pair_of(s.z, s.w)};
              const uint64_t n2[2] = {pair_of(-s.x, -s.y), pair_of(-s.z, -s.w)};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint64_t u = x[2 * d + e], w = x[4 + 2 * d + e];
                x[2 * d + e] = fma2(w, n2[e], mul2(u, c2[e]));
                x[4 + 2 * d + e] = fma2(u, s2[e], mul2(w, c2[e]));
              }
            }
          }
        }
        y0 = put8(T(), x);
        y1 = put8(T(), x + 4);
      }
      if (!kPaged || dst_s[i] >= 0) {
        T* dst = reinterpret_cast<T*>(isA ? a.Ao.p : a.Bo.p) +
                 (kPaged ? dst_s[i] : (int64_t)(t0 + i) * (isA ? a.Ao.ts : a.Bo.ts)) +
                 (int64_t)(isA ? r : r - nA) * (isA ? a.Ao.hs : a.Bo.hs);
        *reinterpret_cast<uint4*>(dst + o0) = y0;
        *reinterpret_cast<uint4*>(dst + o1) = y1;
      }
      advance(i, r);
    }
    if (!kLong) return;
  }
}

template <bool kPaged>
cudaError_t launch(jolt_dtype t, int tokens, RowsArgs a, int sms, cudaStream_t s) {
  if (tokens <= 0) return cudaSuccess;
  const int64_t nR64 = (int64_t)a.A.heads + a.B.heads;
  if (nR64 * tokens > INT32_MAX) return cudaErrorInvalidValue;   // refused by the caller
  const int nR = (int)nR64;
  // as many tokens as a tile's rows hold, fewer where that would leave the GPU without work
  a.tokens = tokens;
  a.tile = std::max(1, std::min({kMaxTile, kRows / nR, tokens / (2 * sms)}));
  const int grid = (tokens + a.tile - 1) / a.tile, bytes = a.tile * kD * (int)sizeof(float);
  auto go = [&](auto kernel) { return launch_early(kernel, dim3(grid), dim3(kThreads), bytes, 1, s, a); };
  const bool bf16 = t == JOLT_BF16, turn = a.r.interleaved;
  if (nR > kRows)
    return bf16 ? (turn ? go(k_rope_rows<__nv_bfloat16, kPaged, true, true>) : go(k_rope_rows<__nv_bfloat16, kPaged, false, true>))
                : (turn ? go(k_rope_rows<__half, kPaged, true, true>) : go(k_rope_rows<__half, kPaged, false, true>));
  return bf16 ? (turn ? go(k_rope_rows<__nv_bfloat16, kPaged, true, false>) : go(k_rope_rows<__nv_bfloat16, kPaged, false, false>))
              : (turn ? go(k_rope_rows<__half, kPaged, true, false>) : go(k_rope_rows<__half, kPaged, false, false>));
}

}  // namespace

cudaError_t norm_rope(jolt_dtype t, int tokens, const RowsIn& Q, const RowsOut& Qo, const RowsIn& K,
                      const RowsOut& Ko, const RopeArgs& r, int sms, cudaStream_t s) {
  RowsArgs a{};
  a.A = Q;
  a.B = K;
  a.Ao = Qo;
  a.Bo = Ko;
  a.r = r;
  return launch<false>(t, tokens, a, sms, s);
}

cudaError_t paged_append(jolt_dtype t, const BatchView& b, const RowsIn& K, const RowsIn& V, void* K_pages,
                         void* V_pages, const RopeArgs& r, int sms, cudaStream_t s) {
  RowsArgs a{};
  a.A = K;
  a.B = V;
  a.Ao.p = K_pages;
  a.Bo.p = V_pages;
  a.Ao.hs = a.Bo.hs = (int64_t)b.page_size * kD;
  a.r = r;
  a.b = b;
  return launch<true>(t, b.total_q, a, sms, s);
}

}  // namespace jolt
