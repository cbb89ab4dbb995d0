// Paged attention of few query rows: at most 32 rows of a sequence's chunk read one KV head (single
// tokens, a few drafted ones).
//
// Keys and values are read once and nothing else is large, so HBM bounds it; what costs is keeping
// enough bytes in flight. A CTA walks its share of the units (64 keys of one item), each of its four
// warps 16 of the keys, by itself: its own ring of TMA boxes (16 rows x 64 features, swizzled so that
// the matrix loads meet no bank conflicts; 16 keys never straddle a page), its own running maximum, sum
// and output in registers. Copies by the threads, 16 bytes each, took 680 of a unit's 2000 cycles.
// The products are m16n8k16 MMAs: with so few rows the tensor pipe idles either way, and warps that
// run apart need no barrier. Up to 8 rows are the columns of the MMAs and the keys their rows; 9 to 16 are
// padded to the 16 rows (that form for 8 rows too: 199 instead of 188 us for 64 ragged sequences). The
// weights enter the second product as a rounded part and a rounded remainder (two MMAs), so that only the
// output's rounding is left. Warps meet where an item ends or the share does. For 17 to 32 rows a
// warp has two blocks of 16, whose queries it reads from shared memory each time (their fragments would
// not fit the registers beside two outputs). A warp for each block on a common ring, with a barrier a
// unit, ran at half the speed.
// Measured: 64 sequences of up to 8192 keys (8 KV heads, 4 rows each, 1.14 GB) 184 us, 6.2 TB/s; one
// sequence of 131072 keys 89 us, 6.0 TB/s; one of 1024 keys 6.2 us in a graph, a chain of latencies.
#include <cooperative_groups.h>

#include <type_traits>

#include "paged_attention.cuh"

namespace jolt {
namespace {

using namespace pattn;

constexpr int kSlices = 4;                // slices of a unit's keys
constexpr int kKeys = 16;                 // keys of a slice
constexpr int kUnit = kKeys * kSlices;
constexpr int kTile = kKeys * kD * 2;     // bytes of a slice's keys (or values)
constexpr int kMinUnits = 1;
constexpr int kTeamCtas = 8;
constexpr int kThreads = 32 * kSlices;
// Weights are 2^kLift times as large as beside a maximum of 1: fp16 holds nothing below 2^-24, neither a weight nor
// the remainder of one, and the largest may be 2^15.
template <typename T>
constexpr float kLift = std::is_same_v<T, __half> ? 15.0f : 0.0f;
// What the weights are relative to beside the maximum m; rounded up, since with scores of 2^24 and more a last place
// is a whole unit, and no weight may pass 2^15 for it.
template <typename T>
__device__ __forceinline__ float base_of(float m) {
  return kLift<T> == 0.0f ? m : __fsub_ru(m, kLift<T>);
}
// kT: blocks of 16 query rows, 0 for up to 8 rows. CTAs per SM and stages of a ring: what registers and
// shared memory allow.
template <int kT>
constexpr int kCtas = kT <= 1 ? 3 : 2;
template <int kT>
constexpr int kStages = kT <= 1 ? 2 : 3;
template <int kT>
constexpr int kRowsOf = kT == 0 ? 8 : 16 * kT;
// Shared memory: the rings, the queries (kT = 2), a team's part.
template <int kT>
constexpr int kRing = kSlices * kStages<kT> * 2 * kTile;
template <int kT>
constexpr int kSmem = kRing<kT> + (kT > 1 ? 16 * kT * kD * 2 : 0);
template <int kT>
constexpr int kTeamSmem = kSmem<kT> + kRowsOf<kT> * kD * 4;

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(__nv_bfloat16, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(__half, float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two values rounded to the type, and what the rounding left, rounded.
__device__ __forceinline__ void split2(__nv_bfloat16, float x, float y, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  const float2 f = __bfloat1622float2(h);
  const __nv_bfloat162 l = __floats2bfloat162_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void split2(__half, float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x - f.x, y - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ int units_of(const SeqView& v) { return v.n == 0 ? 0 : max(1, (v.len + kUnit - 1) / kUnit); }

// A place on the line of units: block u of U of the item (s, h).
struct Cursor {
  int s, h, u, U;
  SeqView v;
};
__device__ __forceinline__ void advance(Cursor& c, const BatchView& b) {
  if (++c.u < c.U) return;
  c.u = 0;
  if (++c.h < b.heads) return;
  c.h = 0;
  do {   // ends: the caller only advances to units that exist
    ++c.s;
    if (c.s >= b.num_seqs) {
      c.U = 0;
      return;
    }
    c.v = seq_view(b, c.s);
    c.U = units_of(c.v);
  } while (c.U == 0);
}

// What one warp holds of an item, for blocks of 16 rows: queries as A fragments (read from shared memory
// each time for two blocks), outputs, running maxima (in units of log 2) and sums; lane: rows quad and
// quad + 8 of a block.
template <typename T, int kT>
struct Blocks16 {
  static constexpr int blocks = kT, per = 16, rows = 16 * kT;
  uint32_t q[8][4];
  float o[kT][16][4], m[kT][2], l[kT][2];
  int lim[kT][2];

  __device__ __forceinline__ void begin(const PagedAttnArgs& a, const SeqView& v, int h, uint8_t* qs, int tid) {
    const int g = a.g.d, lane = tid & 31, quad = lane >> 2, pair = lane & 3, R = v.n * g;
    const T* Q = reinterpret_cast<const T*>(a.Q) + (int64_t)v.q0 * a.q_ts + (int64_t)h * g * a.q_hs;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = 16 * t + quad + 8 * k;
        const int tok = a.g.quot(r);
        lim[t][k] = r < R ? (a.causal ? v.len - v.n + tok : v.len - 1) : -1;
        if (kT == 1) {
          const T* p = Q + (int64_t)tok * a.q_ts + (int64_t)(r - tok * g) * a.q_hs + 2 * pair;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            q[j][k] = r < R ? *reinterpret_cast<const uint32_t*>(p + 16 * j) : 0u;
            q[j][k + 2] = r < R ? *reinterpret_cast<const uint32_t*>(p + 16 * j + 8) : 0u;
          }
        }
        m[t][k] = -INFINITY;
        l[t][k] = 0.0f;
      }
    if (kT > 1) {   // no warp reads the queries before: the last item's end was a barrier
      for (int u = tid; u < rows * 16; u += kThreads) {
        const int r = u >> 4, c = u & 15, tok = a.g.quot(r);
        const uint4 x = r < R ? *reinterpret_cast<const uint4*>(Q + (int64_t)tok * a.q_ts + (int64_t)(r - tok * g) * a.q_hs + 8 * c)
                              : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(qs + r * (2 * kD) + ((c ^ (r & 7)) << 4)) = x;
      }
      __syncthreads();
    }
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][j][e] = 0.0f;
  }

  // A unit's 16 keys: scores of 16 rows x 16 keys, weights, weighted values.
  __device__ __forceinline__ void unit(uint32_t Ks, uint32_t Vs, uint32_t Qs, int key0, bool edge, float scale2, int lane) {
    const int pair = lane & 3;
      // scores of 16 rows x 16 keys: matrices (keys 0-7, 8-15) x (features 0-7, 8-15) of each k-step
      float s[kT][2][4] = {};
      const int mrow = (lane & 7) + ((lane >> 4) << 3), mcol = (lane >> 3) & 1, vrow = lane & 15, vcol = lane >> 4;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t k4[4];
        ldsm4(Ks + (j >> 2) * (kTile / 2) + mrow * 128 + (((2 * (j & 3) + mcol) ^ (mrow & 7)) << 4), k4);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          if (kT > 1) ldsm4(Qs + (16 * t + vrow) * (2 * kD) + (((2 * j + vcol) ^ (vrow & 7)) << 4), q[j]);
          mma(T(), s[t][0], q[j], k4[0], k4[1]);
          mma(T(), s[t][1], q[j], k4[2], k4[3]);
        }
      }
      // running softmax in units of log 2; lane: rows quad and quad + 8, keys 2 pair, + 1 of each block of 8
      uint32_t hi[kT][4], lo[kT][4];
#pragma unroll
      for (int t = 0; t < kT; ++t) {
        float mn[2] = {m[t][0], m[t][1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = s[t][n][e] * scale2;
            if (edge && key0 + 8 * n + 2 * pair + (e & 1) > lim[t][e >> 1]) x = -INFINITY;
            s[t][n][e] = x;
            mn[e >> 1] = fmaxf(mn[e >> 1], x);
          }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          mn[k] = fmaxf(mn[k], __shfl_xor_sync(0xffffffffu, mn[k], 1));
          mn[k] = fmaxf(mn[k], __shfl_xor_sync(0xffffffffu, mn[k], 2));
        }
        if (__any_sync(0xffffffffu, mn[0] > m[t][0] || mn[1] > m[t][1])) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float f = mn[k] == -INFINITY ? 1.0f : ex2(base_of<T>(m[t][k]) - base_of<T>(mn[k]));
            m[t][k] = mn[k];
            l[t][k] *= f;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              o[t][j][2 * k] *= f;
              o[t][j][2 * k + 1] *= f;
            }
          }
        }
        const float sub[2] = {m[t][0] == -INFINITY ? 0.0f : base_of<T>(m[t][0]), m[t][1] == -INFINITY ? 0.0f : base_of<T>(m[t][1])};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[t][n][e] = ex2(s[t][n][e] - sub[e >> 1]);
            l[t][e >> 1] += s[t][n][e];
          }
        split2(T(), s[t][0][0], s[t][0][1], hi[t][0], lo[t][0]);
        split2(T(), s[t][0][2], s[t][0][3], hi[t][1], lo[t][1]);
        split2(T(), s[t][1][0], s[t][1][1], hi[t][2], lo[t][2]);
        split2(T(), s[t][1][2], s[t][1][3], hi[t][3], lo[t][3]);
      }
      // weighted values: matrices (keys 0-7, 8-15) x (8 features), transposed
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t v4[4];
        ldsm4t(Vs + (j >> 2) * (kTile / 2) + vrow * 128 + (((2 * (j & 3) + vcol) ^ (vrow & 7)) << 4), v4);
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          mma(T(), o[t][2 * j], hi[t], v4[0], v4[1]);
          mma(T(), o[t][2 * j + 1], hi[t], v4[2], v4[3]);
        }
#pragma unroll
        for (int t = 0; t < kT; ++t) {
          mma(T(), o[t][2 * j], lo[t], v4[0], v4[1]);
          mma(T(), o[t][2 * j + 1], lo[t], v4[2], v4[3]);
        }
      }
  }

  __device__ __forceinline__ void sums(float2* ml, int lane) {
    const int quad = lane >> 2, pair = lane & 3;
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[t][k] = base_of<T>(m[t][k]);   // what sum and output are relative to
        l[t][k] += __shfl_xor_sync(0xffffffffu, l[t][k], 1);
        l[t][k] += __shfl_xor_sync(0xffffffffu, l[t][k], 2);
        if (pair == 0) ml[16 * t + quad + 8 * k] = make_float2(m[t][k], l[t][k]);
      }
  }
  // Block t's outputs relative to the maxima over all warps (ml), rows of 128 floats, 16-byte blocks
  // swizzled by the row.
  template <class ML>
  __device__ __forceinline__ void put(int t, float* so, const ML& ml, int lane) {
    const int quad = lane >> 2, pair = lane & 3;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int r = quad + 8 * k;
      float mx = ml[0][16 * t + r].x;
#pragma unroll
      for (int w = 1; w < kSlices; ++w) mx = fmaxf(mx, ml[w][16 * t + r].x);
      const float f = rescale(m[t][k], mx);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int blk = (2 * j + (pair >> 1)) ^ ((r & 7) << 1);
        *reinterpret_cast<float2*>(so + r * kD + 4 * blk + 2 * (pair & 1)) =
            make_float2(o[t][j][2 * k] * f, o[t][j][2 * k + 1] * f);
      }
    }
  }
};

__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The same for up to 8 rows, with the products turned: keys (and features) are the 16 rows of an MMA and
// the queries its 8 columns, so half the MMAs do. Lane: queries 2 pair and 2 pair + 1; of the scores
// keys quad and quad + 8, of the output features quad and quad + 8 of each 16.
template <typename T>
struct Block8 {
  static constexpr int blocks = 1, per = 8;
  uint32_t q[8][2];
  float o[8][4], m[2], l[2];
  int lim[2];

  __device__ __forceinline__ void begin(const PagedAttnArgs& a, const SeqView& v, int h, uint8_t*, int tid) {
    const int g = a.g.d, lane = tid & 31, quad = lane >> 2, pair = lane & 3, R = v.n * g, tok = a.g.quot(quad);
    const T* Q = reinterpret_cast<const T*>(a.Q) + (int64_t)v.q0 * a.q_ts + (int64_t)h * g * a.q_hs;
    const T* p = Q + (int64_t)tok * a.q_ts + (int64_t)(quad - tok * g) * a.q_hs + 2 * pair;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q[j][0] = quad < R ? *reinterpret_cast<const uint32_t*>(p + 16 * j) : 0u;
      q[j][1] = quad < R ? *reinterpret_cast<const uint32_t*>(p + 16 * j + 8) : 0u;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * pair + e;
      lim[e] = r < R ? (a.causal ? v.len - v.n + a.g.quot(r) : v.len - 1) : -1;
      m[e] = -INFINITY;
      l[e] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
  }

  __device__ __forceinline__ void unit(uint32_t Ks, uint32_t Vs, uint32_t, int key0, bool edge, float scale2, int lane) {
    const int quad = lane >> 2;
    const int arow = lane & 15, acol = lane >> 4, trow = (lane & 7) + ((lane >> 4) << 3), tcol = (lane >> 3) & 1;
    float sa[2][4] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t k4[4];
      ldsm4(Ks + (j >> 2) * (kTile / 2) + arow * 128 + (((2 * (j & 3) + acol) ^ (arow & 7)) << 4), k4);
      mma(T(), sa[j & 1], k4, q[j][0], q[j][1]);
    }
    float s[4], mn[2] = {m[0], m[1]};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float x = (sa[0][e] + sa[1][e]) * scale2;
      if (edge && key0 + quad + 8 * (e >> 1) > lim[e & 1]) x = -INFINITY;
      s[e] = x;
      mn[e & 1] = fmaxf(mn[e & 1], x);
    }
#pragma unroll
    for (int w = 4; w < 32; w <<= 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) mn[e] = fmaxf(mn[e], __shfl_xor_sync(0xffffffffu, mn[e], w));
    if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float f = mn[e] == -INFINITY ? 1.0f : ex2(base_of<T>(m[e]) - base_of<T>(mn[e]));
        m[e] = mn[e];
        l[e] *= f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][e] *= f;
          o[j][2 + e] *= f;
        }
      }
    }
    const float sub[2] = {m[0] == -INFINITY ? 0.0f : base_of<T>(m[0]), m[1] == -INFINITY ? 0.0f : base_of<T>(m[1])};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[e] = ex2(s[e] - sub[e & 1]);
      l[e & 1] += s[e];
    }
    uint32_t hi[2], lo[2];
    split2(T(), s[0], s[1], hi[0], lo[0]);
    split2(T(), s[2], s[3], hi[1], lo[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {   // keys x queries to queries x keys
      hi[k] = turn8x8(hi[k]);
      lo[k] = turn8x8(lo[k]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t v4[4];
      ldsm4t(Vs + (j >> 2) * (kTile / 2) + trow * 128 + (((2 * (j & 3) + tcol) ^ (trow & 7)) << 4), v4);
      mma(T(), o[j], v4, hi[0], hi[1]);
      mma(T(), o[j], v4, lo[0], lo[1]);
    }
  }

  __device__ __forceinline__ void sums(float2* ml, int lane) {
    const int quad = lane >> 2, pair = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[e] = base_of<T>(m[e]);   // what sum and output are relative to
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], w);
      if (quad == 0) ml[2 * pair + e] = make_float2(m[e], l[e]);
    }
  }
  template <class ML>
  __device__ __forceinline__ void put(int, float* so, const ML& ml, int lane) {
    const int quad = lane >> 2, pair = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 2 * pair + e;
      float mx = ml[0][r].x;
#pragma unroll
      for (int w = 1; w < kSlices; ++w) mx = fmaxf(mx, ml[w][r].x);
      const float f = rescale(m[e], mx);
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int d = 16 * j + 8 * k + quad;
          so[r * kD + 4 * ((d >> 2) ^ (r << 1)) + (d & 3)] = o[j][2 * k + e] * f;
        }
    }
  }
};

// The fills from .. to - 1 of a ring's stages, waited for once more; never in a run that ends well, so kept out of the
// kernel's registers.
__device__ __noinline__ void land(uint64_t* full, int stages, int from, int to) {
  for (int k = from; k < to; ++k) mbar_wait(&full[k % stages], (k / stages) & 1, 1u << 20);
}

// kTeam: instead of a share of the line a CTA takes an eighth of the item of its cluster, and the cluster's
// CTAs combine through one another's shared memory: one launch and no scratch.
template <typename T, int kT, bool kTeam>
__global__ void __launch_bounds__(kThreads, kCtas<kT>)
    k_attn_decode(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ Maps maps, const Workspace ws) {
  using Held = std::conditional_t<kT == 0, Block8<T>, Blocks16<T, kT == 0 ? 1 : kT>>;
  constexpr int kRows = kRowsOf<kT>, kDeep = kStages<kT>;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ __align__(8) uint64_t full_s[kSlices][kStages<kT>];
  __shared__ int valid_s[kSlices][kStages<kT>];      // rows of a stage that hold keys
  __shared__ int gave_up;
  __shared__ bool hid_s[kSlices];                    // whether the item's values hold what was hidden
  __shared__ float2 ml_s[kSlices][kRows];
  __shared__ float2 team_ml[kTeam ? kRows : 1];
  __shared__ int64_t scan_s[kSlices + 3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const BatchView& b = a.b;
  const int g = a.g.d;
  const float scale2 = a.scale * kLog2e;
  grid_release();
  if (tid < kSlices * kDeep) {
    mbar_init(&full_s[0][0] + tid, 1);
    (&valid_s[0][0])[tid] = kKeys;     // also of a stage that is never filled, when a wait has given up
  }
  if (tid == 0) {
    gave_up = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.K);
    prefetch_tensormap(&maps.V);
  }
  grid_wait();
  Start st{};
  Cursor lc;
  if (kTeam) {
    const int item = blockIdx.x / kTeamCtas, rank = blockIdx.x % kTeamCtas;
    lc.s = item / b.heads;
    lc.h = item % b.heads;
    lc.v = seq_view(b, lc.s);
    if (lc.v.n == 0) return;   // the whole cluster
    lc.U = units_of(lc.v);
    st.lo = (int64_t)rank * lc.U / kTeamCtas;
    st.hi = (int64_t)(rank + 1) * lc.U / kTeamCtas;
    lc.u = (int)st.lo;
  } else {
    st = find_start<kThreads>(
        b.num_seqs, [&](int s) { return s < b.num_seqs ? (int64_t)units_of(seq_view(b, s)) * b.heads : 0; }, kMinUnits, scan_s);
    if ((int)blockIdx.x >= st.G) {
      if (tid == 0) ws.list[blockIdx.x].s = -1;
      return;
    }
    lc.s = st.s;
    lc.v = seq_view(b, st.s);
    lc.U = units_of(lc.v);
    lc.h = (int)quot(st.lo - st.base, lc.U);
    lc.u = (int)(st.lo - st.base - (int64_t)lc.h * lc.U);
  }
  Cursor cc = lc;
  const int count = (int)(st.hi - st.lo);

  // ---- loads: a phase of the stage's barrier a unit, empty where the unit has no page
  __syncthreads();
  uint8_t* ring = sm + warp * (kDeep * 2 * kTile);
  const Waits wait{&gave_up, b.status};
  int pg_s = -1, pg_u0 = 0, pg = -1;     // this lane's page: that of unit pg_u0 + lane of sequence pg_s
  int issued = 0;
  auto issue = [&](int stage) {
    if (issued == count) return;
    if (lc.s != pg_s || lc.u < pg_u0 || lc.u >= pg_u0 + 32) {
      pg_s = lc.s;
      pg_u0 = lc.u;
      const int64_t key = (int64_t)(lc.u + lane) * kUnit + warp * kKeys;
      pg = key < lc.v.len ? page_of(b, lc.s, (int)key) : -1;
    }
    const int page = __shfl_sync(0xffffffffu, pg, lc.u - pg_u0);
    if (lane == 0) {
      const int key0 = lc.u * kUnit + warp * kKeys;
      uint64_t* bar = &full_s[warp][stage];
      valid_s[warp][stage] = page < 0 ? 0 : min(kKeys, lc.v.len - key0);
      if (page >= 0) {
        const int row = key0 - b.by_page.quot(key0) * b.page_size;
        uint8_t* dst = ring + stage * 2 * kTile;
        mbar_arrive_expect_tx(bar, 2 * kTile);
        tma_load_4d(dst, &maps.K, bar, 0, row, lc.h, page);
        tma_load_4d(dst + kTile / 2, &maps.K, bar, 64, row, lc.h, page);
        tma_load_4d(dst + kTile, &maps.V, bar, 0, row, lc.h, page);
        tma_load_4d(dst + kTile * 3 / 2, &maps.V, bar, 64, row, lc.h, page);
      } else {
        mbar_arrive(bar);
      }
    }
    ++issued;
    if (issued < count) advance(lc, b);
  };
#pragma unroll
  for (int i = 0; i < kDeep - 1; ++i) issue(i);

  Held held;
  bool fresh = true;         // the next unit begins an item (or this CTA's part of one)
  bool began = cc.u == 0;    // the current item began in this CTA's range
  Split split;
  split.s = -1;

  for (int i = 0; i < count; ++i) {
    const int stage = i % kDeep;
    // Where a wait gives up, the warp's copies in flight land (or are waited for as long again) and no stage is filled
    // after it: the result is void, and reported. The barriers of the items' ends need the warp all the same.
    if (!__all_sync(0xffffffffu, wait(&full_s[warp][stage], (i / kDeep) & 1))) {
      land(full_s[warp], kDeep, i, issued);
      issued = count;
    }
    issue((i + kDeep - 1) % kDeep);
    if (fresh) {
      fresh = false;
      if (lane == 0) hid_s[warp] = false;
      held.begin(a, cc.v, cc.h, sm + kRing<kT>, tid);
    }
    const uint32_t Ks = smem_u32(ring + stage * 2 * kTile), Vs = Ks + kTile;
    const int key0 = cc.u * kUnit + warp * kKeys;
    if (key0 < cc.v.len) {
      const int valid = valid_s[warp][stage];
      if (valid < kKeys) {
        // rows without keys are zeroed: values, since a weight of zero does not hide what lies in the page
        // (scores are masked), and all of a bad page
        for (int u = lane; u < 4 * 8 * (kKeys - valid); u += 32) {
          const int part = u & 3, c = (u >> 2) & 7, r = valid + (u >> 5);
          *reinterpret_cast<uint4*>(ring + stage * 2 * kTile + part * (kTile / 2) + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();   // before the stage's next copy
        __syncwarp();
      }
      const int seen = cc.v.len - cc.v.n;   // the last key that all rows see
      if (a.causal && key0 + valid - 1 > seen) {
        uint8_t* values = ring + stage * 2 * kTile + kTile;
        const int from = max(0, seen + 1 - key0);
        if (!finite<T, 1>(values, kTile / 2, from, valid, lane)) {
          hide<T>(values, kTile / 2, from, valid, lane);
          if (lane == 0) hid_s[warp] = true;
          fence_async_shared();
          __syncwarp();
        }
      }
      const bool edge = key0 + kKeys - 1 > (a.causal ? cc.v.len - cc.v.n : cc.v.len - 1) || cc.v.n * g < kRows;
      held.unit(Ks, Vs, smem_u32(sm + kRing<kT>), key0, edge, scale2, lane);
    }
    const bool ends = cc.u + 1 == cc.U;
    if (ends || i + 1 == count) {
      // join the four warps: maxima and sums first, then the outputs, a block of rows at a time, each warp's
      // in its own stage that was just read
      held.sums(ml_s[warp], lane);
      const int R = cc.v.n * g;
      const bool whole = ends && began;
      const int slot = began ? 1 : 0;
#pragma unroll
      for (int t = 0; t < Held::blocks; ++t) {
        __syncthreads();
        held.put(t, reinterpret_cast<float*>(ring + stage * 2 * kTile), ml_s, lane);
        __syncthreads();
        for (int rr = warp; rr < min(Held::per, R - Held::per * t); rr += kSlices) {
          const int r = Held::per * t + rr;
          const int tok = a.g.quot(r);
          const int64_t row = (int64_t)(cc.v.q0 + tok) * a.Hq + cc.h * g + r - tok * g;
          Prefix pre{};
          if (!kTeam && whole) pre = load_prefix(a, row, lane);
          float mx = -INFINITY, ls = 0.0f;
#pragma unroll
          for (int w = 0; w < kSlices; ++w) mx = fmaxf(mx, ml_s[w][r].x);
          float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kSlices; ++w) {
            const float2 p = ml_s[w][r];
            ls = fmaf(p.y, rescale(p.x, mx), ls);
            const float4 x = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(sm + (w * kDeep + stage) * 2 * kTile) + rr * kD + 4 * (lane ^ ((rr & 7) << 1)));
            y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
          }
          if (hid_s[0] | hid_s[1] | hid_s[2] | hid_s[3]) {
            const int seen = cc.v.len - cc.v.n;
            const uint32_t found = hidden16<T>(a, cc.s, cc.h, seen + 1, seen + tok, (4 * lane) & ~15) >> ((4 * lane) & 15);
            if (found & 1) y.x = NAN;
            if (found & 2) y.y = NAN;
            if (found & 4) y.z = NAN;
            if (found & 8) y.w = NAN;
          }
          if (kTeam) {
            *reinterpret_cast<float4*>(sm + kSmem<kT> + r * (4 * kD) + 16 * lane) = y;
            if (lane == 0) team_ml[r] = make_float2(mx, ls);
          } else if (whole) {
            finish_row<T>(a, row, lane, y, mx, ls, pre);
          } else {
            const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * ws.rows + r;
            *reinterpret_cast<float4*>(ws.o + at * kD + 4 * lane) = y;
            if (lane == 0) ws.ml[at] = make_float2(mx, ls);
          }
        }
      }
      if (began && !ends) {
        split.s = cc.s;
        split.h = cc.h;
        split.m = 0;
        split.slot = slot;
        split.q0 = cc.v.q0;
        split.rows = R;
        split.c_last = owner_of(st.lo + i + (cc.U - 1 - cc.u), st.each, st.more);
      }
      fence_async_shared();
      __syncthreads();   // the stages are written again, by copies
      fresh = began = true;
    }
    if (i + 1 < count) advance(cc, b);
  }
  if (!kTeam) {
    if (tid == 0) ws.list[blockIdx.x] = split;
    return;
  }
  // the cluster's parts: CTA k finishes the rows k, k + 8, ..., a warp each
  if (count == 0 && tid < kRows) team_ml[tid] = make_float2(-INFINITY, 0.0f);
  const cooperative_groups::cluster_group team = cooperative_groups::this_cluster();
  const int r = blockIdx.x % kTeamCtas + kTeamCtas * warp;
  const int tok = a.g.quot(r);
  const int64_t row = (int64_t)(cc.v.q0 + tok) * a.Hq + cc.h * g + r - tok * g;
  Prefix pre{};
  if (r < cc.v.n * g) pre = load_prefix(a, row, lane);
  team.sync();
  if (r < cc.v.n * g) {
    float2 p[kTeamCtas];
    float4 x[kTeamCtas], y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float mx = -INFINITY, ls = 0.0f;
#pragma unroll
    for (int c = 0; c < kTeamCtas; ++c) {
      p[c] = *team.map_shared_rank(&team_ml[r], c);
      x[c] = *reinterpret_cast<const float4*>(team.map_shared_rank(sm + kSmem<kT> + r * (4 * kD) + 16 * lane, c));
    }
#pragma unroll
    for (int c = 0; c < kTeamCtas; ++c) mx = fmaxf(mx, p[c].x);
#pragma unroll
    for (int c = 0; c < kTeamCtas; ++c) {
      if (p[c].y == 0.0f) continue;   // no keys, and perhaps no output written
      const float f = rescale(p[c].x, mx);
      ls = fmaf(p[c].y, f, ls);
      y.x = fmaf(x[c].x, f, y.x);
      y.y = fmaf(x[c].y, f, y.y);
      y.z = fmaf(x[c].z, f, y.z);
      y.w = fmaf(x[c].w, f, y.w);
    }
    finish_row<T>(a, row, lane, y, mx, ls, pre);
  }
  team.sync();   // no CTA leaves while another reads from it
}

template <typename T, int kT>
cudaError_t launch(const PagedAttnArgs& a, const AttnPlan& p, const Workspace& w, cudaStream_t s) {
  [[maybe_unused]] static SmemFlags allowed;
  static SmemFlags allowed_team;
  Maps maps;
  maps.K = a.maps[2];
  maps.V = a.maps[3];
  cudaError_t e;
  if (p.team) {
    e = allow_smem(k_attn_decode<T, kT, true>, kTeamSmem<kT>, a.device, allowed_team);
    if (e != cudaSuccess) return e;
    return launch_early(k_attn_decode<T, kT, true>, dim3(p.grid), dim3(kThreads), kTeamSmem<kT>, kTeamCtas, s, a, maps, w);
  }
  if constexpr (kT == 1) {   // 9 to 16 rows: clusters only
    return cudaErrorInvalidValue;
  } else {
    e = allow_smem(k_attn_decode<T, kT, false>, kSmem<kT>, a.device, allowed);
    if (e != cudaSuccess) return e;
    return launch_early(k_attn_decode<T, kT, false>, dim3(p.grid), dim3(kThreads), kSmem<kT>, 1, s, a, maps, w);
  }
}

}  // namespace

cudaError_t attn_decode(const PagedAttnArgs& a, const AttnPlan& p, const pattn::Workspace& w, cudaStream_t s) {
  const bool b = a.dtype == JOLT_BF16;
  if (p.rows == 8) return b ? launch<__nv_bfloat16, 0>(a, p, w, s) : launch<__half, 0>(a, p, w, s);
  if (p.rows == 16) return b ? launch<__nv_bfloat16, 1>(a, p, w, s) : launch<__half, 1>(a, p, w, s);
  return b ? launch<__nv_bfloat16, 2>(a, p, w, s) : launch<__half, 2>(a, p, w, s);
}

}  // namespace jolt
