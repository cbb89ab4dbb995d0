// Rows of queries and keys normed and rotated by their position, and the append of keys and values
// to a paged cache. One row is the 128 features of one head of one token:
//     y = w * x / sqrt(mean(x^2) + eps)                        (left out without a weight),
//     (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = position * inv_freq[i],
// over the pairs j = i + rope_dim / 2 (half-split) or (2 i, 2 i + 1) (interleaved) of the first
// rope_dim features. All in float32 and rounded once; the angle is formed in float64 and reduced
// to a part of a turn there, since a float32 angle of position 10^5 is off by 10^-2 rad.
//
// Each row is read and written once, which bounds the kernel for long inputs (HBM); short inputs
// are bound by latency. A CTA takes a tile of tokens, about 80 rows, 16 lanes a row (16 bytes each) and
// up to five rows a lane in flight at once: with one token a CTA the append of 16 rows a token ran at 1.4
// TB/s. The tile's sines are computed once (a thread each, while the rows are on their way) and used by
// all heads from shared memory; the append's page lookup is one parallel pass over the batch's offsets
// instead of a search.
#include <algorithm>

#include "../paged.h"

namespace jolt {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = kThreads / 16;   // rows at a time
constexpr int kBatch = 5;               // rows a slot keeps in flight
constexpr int kMaxTile = 16;            // tokens of a tile

template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<__half> {
  static __device__ __forceinline__ void get(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

struct RowsArgs {
  RowsIn A, B;       // A: queries, or the append's keys; B: keys, or the append's values
  RowsOut Ao, Bo;    // outputs (strides of a page row in the append)
  RopeArgs r;
  BatchView b;       // append only
  int32_t tokens, tile;
};

__device__ __forceinline__ void get8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

template <typename T, bool kPaged>
__global__ void __launch_bounds__(kThreads) k_rope_rows(const RowsArgs a) {
  extern __shared__ __align__(16) float trig[];        // [tile][2][128]: a feature's cosine, its partner's signed sine
  __shared__ __align__(16) float w_s[2][kD];           // norm weights
  __shared__ int64_t dst_s[kMaxTile];                  // append: page row in elements from the pages' base; < 0: none
  __shared__ int pos_s[kMaxTile], seq_s[kMaxTile];     // append: place in the cache, sequence (-1: none)
  const int tid = threadIdx.x, slot = tid >> 4, l = tid & 15;
  const int t0 = blockIdx.x * a.tile, nt = min(a.tile, a.tokens - t0);
  const int nA = a.A.heads, nR = a.A.heads + a.B.heads, rows = nt * nR;
  const int step_t = kSlots / nR, step_r = kSlots % nR;
  const bool rot = a.r.inv_freq != nullptr;
  const bool normA = a.A.w != nullptr, normB = !kPaged && a.B.w != nullptr;
  const T* A = reinterpret_cast<const T*>(a.A.p) + 8 * l;
  const T* B = reinterpret_cast<const T*>(a.B.p) + 8 * l;

  // rows slot, slot + 16, ...: token i of the tile, row r of the token
  int i = slot / nR, r = slot - i * nR;
  auto step = [&](int& ti, int& tr) {
    ti += step_t;
    tr += step_r;
    if (tr >= nR) {
      tr -= nR;
      ++ti;
    }
  };
  uint4 v[kBatch] = {};
  auto load = [&](int ti, int tr) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (ti < nt) {
        const int64_t t = t0 + ti;
        v[k] = *reinterpret_cast<const uint4*>(tr < nA ? A + t * a.A.ts + tr * a.A.hs : B + t * a.B.ts + (tr - nA) * a.B.hs);
      }
      step(ti, tr);
    }
  };
  load(i, r);

  if (normA && tid < kD) w_s[0][tid] = (float)reinterpret_cast<const T*>(a.A.w)[tid];
  if (normB && tid >= kD) w_s[1][tid - kD] = (float)reinterpret_cast<const T*>(a.B.w)[tid - kD];
  if (kPaged) {
    if (tid < kMaxTile) seq_s[tid] = -1;
    __syncthreads();
    for (int s = tid; s < a.b.num_seqs; s += kThreads) {
      const int q0 = a.b.q_start[s], q1 = a.b.q_start[s + 1];
      if (q0 >= t0 + nt || q1 <= t0) continue;
      const SeqView sv = seq_view(a.b, s);
      if (sv.n == 0) continue;
      for (int t = max(q0, t0); t < min(q1, t0 + nt); ++t) {
        seq_s[t - t0] = s;
        pos_s[t - t0] = sv.len - (q1 - t);
      }
    }
    __syncthreads();
    if (tid >= kThreads - nt) {   // not the first threads: they have angles to make
      const int t = tid - (kThreads - nt), s = seq_s[t];
      int64_t d = -1;
      if (s >= 0 && pos_s[t] >= 0) {
        const int pg = page_of(a.b, s, pos_s[t]);
        if (pg >= 0) d = ((int64_t)pg * a.b.heads * a.b.page_size + pos_s[t] % a.b.page_size) * kD;
      }
      dst_s[t] = d;
    }
  }
  if (rot) {
    const int h = a.r.rope_dim >> 1;
    for (int u = tid; u < nt * 64; u += kThreads) {
      const int t = u >> 6, f = u & 63;
      float c = 1.0f, s = 0.0f;
      int x, y;                 // the pair's features
      if (f < h) {
        const int pos = kPaged && !a.r.positions ? (seq_s[t] >= 0 ? pos_s[t] : 0) : a.r.positions[t0 + t];
        // parts of a turn, in float64 up to the last whole turn
        double turn = (double)pos * ((double)a.r.inv_freq[f] * 0.15915494309189533577);
        turn -= rint(turn);
        sincospif(2.0f * (float)turn, &s, &c);
        x = a.r.interleaved ? 2 * f : f;
        y = a.r.interleaved ? 2 * f + 1 : f + h;
      } else {                  // features that are not rotated
        x = 2 * f;
        y = 2 * f + 1;
      }
      float* row = trig + t * (2 * kD);
      row[x] = row[y] = c;
      row[kD + x] = -s;
      row[kD + y] = s;
    }
  }
  __syncthreads();

  // the 16 lanes of a row take part in its shuffles together
  const uint32_t mask = 0xffffu << (tid & 16);
  const int e0 = 8 * l, h8 = a.r.rope_dim >> 4;       // lanes of the first halves of half-split pairs
  const bool inside = e0 < a.r.rope_dim;
  const int partner = !inside ? l : l < h8 ? l + h8 : l - h8;
  for (;;) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i >= nt) break;
      const bool isA = r < nA;
      const int64_t t = t0 + i;
      uint4 out = v[k];
      if (!kPaged || isA) {     // values of the append go out as they are
        float x[8];
        Vec<T>::get(out, x);
        if (isA ? normA : normB) {
          float q = 0.0f, w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) q = fmaf(x[e], x[e], q);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) q += __shfl_xor_sync(mask, q, o, 16);
          const float f = 1.0f / sqrtf(q * (1.0f / kD) + a.r.eps);
          get8(&w_s[isA ? 0 : 1][e0], w);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * f * w[e];
        }
        if (rot) {
          float c[8], s[8], p[8];
          get8(trig + i * (2 * kD) + e0, c);
          get8(trig + i * (2 * kD) + kD + e0, s);
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = a.r.interleaved ? x[e ^ 1] : __shfl_sync(mask, x[e], partner, 16);
          if (inside) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(p[e], s[e], x[e] * c[e]);
          }
        }
        out = Vec<T>::put(x);
      }
      if (!kPaged || dst_s[i] >= 0) {
        T* dst = reinterpret_cast<T*>(isA ? a.Ao.p : a.Bo.p) + (kPaged ? dst_s[i] : t * (isA ? a.Ao.ts : a.Bo.ts)) + e0;
        *reinterpret_cast<uint4*>(dst + (isA ? r * a.Ao.hs : (r - nA) * a.Bo.hs)) = out;
      }
      step(i, r);
    }
    if (i >= nt) return;
    load(i, r);
  }
}

template <bool kPaged>
cudaError_t launch(jolt_dtype t, int tokens, RowsArgs a, int sms, cudaStream_t s) {
  if (tokens <= 0) return cudaSuccess;
  const int nR = a.A.heads + a.B.heads;
  // five rows a slot, but smaller tiles as long as the GPU is not full
  const int full = std::max(1, std::min(kMaxTile, kSlots * kBatch / nR));
  a.tokens = tokens;
  a.tile = std::max(1, std::min<int>(full, tokens / (2 * sms)));
  const int grid = (tokens + a.tile - 1) / a.tile, bytes = a.tile * 2 * kD * (int)sizeof(float);
  if (t == JOLT_BF16) k_rope_rows<__nv_bfloat16, kPaged><<<grid, kThreads, bytes, s>>>(a);
  else k_rope_rows<__half, kPaged><<<grid, kThreads, bytes, s>>>(a);
  note_launch();
  return cudaGetLastError();
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
