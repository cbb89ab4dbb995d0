// Rows of queries and keys normed and rotated by their position, and the append of keys and values
// to a paged cache. One row is the 128 features of one head of one token:
//     y = w * x / sqrt(mean(x^2) + eps)                        (left out without a weight),
//     (y_i, y_j) -> (y_i cos a - y_j sin a, y_j cos a + y_i sin a),  a = position * inv_freq[i],
// over the pairs j = i + rope_dim / 2 (half-split) or (2 i, 2 i + 1) (interleaved) of the first
// rope_dim features. All in float32 and rounded once; the angle is formed in float64 and reduced
// to a part of a turn there, since a float32 angle of position 10^5 is off by 10^-2 rad.
//
// Each row is read and written once, which bounds the kernel for long inputs (HBM); short inputs
// are bound by latency. One CTA takes a token, 16 lanes a row (16 bytes each): the token's sines
// are computed once (a thread each) and used by all its heads from registers, a CTA's threads keep
// kBatch rows each in flight, and the append's page lookup is one parallel pass over the batch's
// offsets instead of a search.
#include "../paged.h"

namespace jolt {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = kThreads / 16;   // rows at a time
constexpr int kBatch = 4;               // rows a slot keeps in flight

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
};

// One row's 8 features of this lane, normed (weight w8) and rotated (cosines c8, sines s8 of the
// lane's features, the sines negated on the first half of a half-split pair). Called by the 16 lanes
// of a row (mask), which share every condition but `inside`.
template <typename T>
__device__ __forceinline__ uint4 norm_rotate(uint32_t mask, const uint4& v, bool norm, const float (&w8)[8], float eps, bool rot,
                                             bool interleaved, const float (&c8)[8], const float (&s8)[8], int partner,
                                             bool inside) {
  float x[8];
  Vec<T>::get(v, x);
  if (norm) {
    float q = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(x[e], x[e], q);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) q += __shfl_xor_sync(mask, q, o, 16);
    const float f = 1.0f / sqrtf(q * (1.0f / kD) + eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = x[e] * f * w8[e];
  }
  if (rot) {
    if (interleaved) {
      if (inside) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float a = x[e], b = x[e + 1];
          x[e] = a * c8[e] - b * s8[e];
          x[e + 1] = b * c8[e] + a * s8[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(mask, x[e], partner, 16);
        if (inside) x[e] = fmaf(o, s8[e], x[e] * c8[e]);   // s8 carries the pair's sign
      }
    }
  }
  return Vec<T>::put(x);
}

template <typename T, bool kPaged>
__global__ void __launch_bounds__(kThreads) k_rope_rows(const RowsArgs a) {
  __shared__ __align__(16) float cs[64], sn[64];
  __shared__ int64_t dst_s;   // page row of the append, in elements from the pages' base; < 0: skip
  __shared__ int pos_s;
  const int tok = blockIdx.x, tid = threadIdx.x, slot = tid >> 4, l = tid & 15;
  const int nA = a.A.heads, nR = a.A.heads + a.B.heads;
  const T* Ap = reinterpret_cast<const T*>(a.A.p) + (int64_t)tok * a.A.ts + 8 * l;
  const T* Bp = a.B.p ? reinterpret_cast<const T*>(a.B.p) + (int64_t)tok * a.B.ts + 8 * l : nullptr;
  uint4 v[kBatch] = {};
  auto load = [&](int r0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * kSlots;
      if (r < nR) v[k] = *reinterpret_cast<const uint4*>(r < nA ? Ap + r * a.A.hs : Bp + (r - nA) * a.B.hs);
    }
  };
  load(slot);
  if (kPaged) {
    // the sequence that owns the token, its place in the cache and the page row it is written to
    if (tid == 0) dst_s = -1;
    __syncthreads();
    for (int s = tid; s < a.b.num_seqs; s += kThreads) {
      const int q0 = a.b.q_start[s], q1 = a.b.q_start[s + 1];
      if (tok < q0 || tok >= q1) continue;
      const SeqView sv = seq_view(a.b, s);
      const int pos = sv.len - (q1 - tok);
      if (sv.n == 0 || pos < 0) continue;
      const int pg = page_of(a.b, s, pos);
      pos_s = pos;
      if (pg >= 0) dst_s = ((int64_t)pg * a.b.heads * a.b.page_size + pos % a.b.page_size) * kD;
    }
    __syncthreads();
    if (dst_s < 0) return;
  }
  const bool rot = a.r.inv_freq != nullptr;
  const int h = a.r.rope_dim >> 1;
  if (rot) {
    if (tid < h) {
      const int pos = kPaged && !a.r.positions ? pos_s : a.r.positions[tok];
      // parts of a turn, in float64 up to the last whole turn
      double u = (double)pos * ((double)a.r.inv_freq[tid] * 0.15915494309189533577);
      u -= rint(u);
      float s, c;
      sincospif(2.0f * (float)u, &s, &c);
      cs[tid] = c;
      sn[tid] = s;
    }
    __syncthreads();
  }
  // this lane's cosines and (signed) sines, per feature
  float c8[8] = {}, s8[8] = {};
  const int e0 = 8 * l;
  const bool inside = e0 < a.r.rope_dim;
  int partner = l;
  if (rot && inside) {
    if (a.r.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c8[e] = cs[(e0 + e) >> 1];
        s8[e] = sn[(e0 + e) >> 1];
      }
    } else {
      const bool first = e0 < h;
      const int i0 = first ? e0 : e0 - h;
      partner = first ? l + (h >> 3) : l - (h >> 3);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c8[e] = cs[i0 + e];
        s8[e] = first ? -sn[i0 + e] : sn[i0 + e];
      }
    }
  }
  const bool normA = a.A.w != nullptr, normB = !kPaged && a.B.w != nullptr;
  float wA[8] = {}, wB[8] = {};
  if (normA) Vec<T>::get(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.A.w) + e0), wA);
  if (normB) Vec<T>::get(*reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.B.w) + e0), wB);
  T* Ao = reinterpret_cast<T*>(a.Ao.p) + (kPaged ? dst_s : (int64_t)tok * a.Ao.ts) + e0;
  T* Bo = reinterpret_cast<T*>(a.Bo.p) + (kPaged ? dst_s : (int64_t)tok * a.Bo.ts) + e0;
  // rows in whole rounds: all 16 lanes of a row take part in its shuffles
  const uint32_t mask = 0xffffu << (tid & 16);
  for (int r0 = slot; r0 - slot < nR; r0 += kSlots * kBatch) {
    if (r0 != slot) load(r0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int r = r0 + k * kSlots;
      if (r - slot >= nR) break;   // uniform over the CTA
      const bool isA = r < nA;
      uint4 y = v[k];
      if (!kPaged || isA) {   // values of the append go out as they are
        float w8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w8[e] = isA ? wA[e] : wB[e];
        y = norm_rotate<T>(mask, y, isA ? normA : normB, w8, a.r.eps, rot, a.r.interleaved, c8, s8, partner, inside);
      }
      if (r < nR) *reinterpret_cast<uint4*>(isA ? Ao + r * a.Ao.hs : Bo + (r - nA) * a.Bo.hs) = y;
    }
  }
}

template <bool kPaged>
cudaError_t launch(jolt_dtype t, int tokens, const RowsArgs& a, cudaStream_t s) {
  if (tokens <= 0) return cudaSuccess;
  if (t == JOLT_BF16) k_rope_rows<__nv_bfloat16, kPaged><<<tokens, kThreads, 0, s>>>(a);
  else k_rope_rows<__half, kPaged><<<tokens, kThreads, 0, s>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t norm_rope(jolt_dtype t, int tokens, const RowsIn& Q, const RowsOut& Qo, const RowsIn& K,
                      const RowsOut& Ko, const RopeArgs& r, cudaStream_t s) {
  RowsArgs a{};
  a.A = Q;
  a.B = K;
  a.Ao = Qo;
  a.Bo = Ko;
  a.r = r;
  return launch<false>(t, tokens, a, s);
}

cudaError_t paged_append(jolt_dtype t, const BatchView& b, const RowsIn& K, const RowsIn& V, void* K_pages,
                         void* V_pages, const RopeArgs& r, cudaStream_t s) {
  RowsArgs a{};
  a.A = K;
  a.B = V;
  a.Ao.p = K_pages;
  a.Bo.p = V_pages;
  a.Ao.hs = a.Bo.hs = (int64_t)b.page_size * kD;
  a.r = r;
  a.b = b;
  return launch<true>(t, b.total_q, a, s);
}

}  // namespace jolt
