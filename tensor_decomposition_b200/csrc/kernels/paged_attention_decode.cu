// Paged attention of few query rows: at most 16 rows of a sequence's chunk read one KV head (single
// tokens with up to 16 query heads a KV head, a few drafted tokens).
//
// Keys and values are read once and nothing else is large, so HBM bounds it; what costs is keeping
// enough bytes in flight. A CTA walks its share of the units (64 keys of one item), each of its four
// warps 16 of the keys, by itself: its own ring of asynchronous 16-byte copies (swizzled so that the
// matrix loads meet no bank conflicts; rows behind the sequence are filled with zeros), its own
// running maximum, sum and output (16 rows x 128 in registers). 16 keys never straddle a page. The
// products are m16n8k16 MMAs with the query rows padded to 16: with so few rows the tensor pipe idles
// either way, and warps that run apart need no barrier. The weights enter the second product as
// a rounded part and a rounded remainder (two MMAs), so that only the output's rounding is left.
// Warps meet where an item ends or the share does.
#include <cooperative_groups.h>

#include "paged_attention.cuh"

namespace jolt {
namespace {

using namespace pattn;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;                 // keys of a warp in a unit
constexpr int kUnit = kKeys * kWarps;
constexpr int kTile = kKeys * kD * 2;     // bytes of a warp's keys (or values)
constexpr int kStages = 3;
constexpr int kCtas = 2;                  // per SM
constexpr int kRows = 16;
constexpr int kMinUnits = 1;
constexpr int kSmem = kWarps * kStages * 2 * kTile;
constexpr int kTeamCtas = 8;
constexpr int kTeamSmem = kSmem + kRows * kD * 4;

__device__ __forceinline__ uint32_t smem_of(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

// kTeam: instead of a share of the line a CTA takes an eighth of the item of its cluster, and the cluster's
// CTAs combine through one another's shared memory: one launch and no scratch.
template <typename T, bool kTeam>
__global__ void __launch_bounds__(kThreads, kCtas) k_attn_decode(const PagedAttnArgs a, const Workspace ws) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ float2 ml_s[kWarps][kRows];
  __shared__ float2 team_ml[kTeam ? kRows : 1];
  __shared__ int64_t scan_s[kWarps + 3];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, pair = lane & 3;
  const BatchView& b = a.b;
  const int g = a.Hq / b.heads;
  const float scale2 = a.scale * kLog2e;
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
    grid_release();
    st = find_start<kThreads>(
        b.num_seqs, [&](int s) { return (int64_t)units_of(seq_view(b, s)) * b.heads; }, kMinUnits, scan_s);
    if ((int)blockIdx.x >= st.G) {
      if (tid == 0) ws.list[blockIdx.x].s = -1;
      return;
    }
    lc.s = st.s;
    lc.v = seq_view(b, st.s);
    lc.U = units_of(lc.v);
    lc.h = (int)((st.lo - st.base) / lc.U);
    lc.u = (int)((st.lo - st.base) % lc.U);
  }
  Cursor cc = lc;
  const int count = (int)(st.hi - st.lo);

  // ---- loads: one commit group a unit, empty ones behind the last
  uint8_t* ring = sm + warp * (kStages * 2 * kTile);
  const int c16 = lane & 15, r2 = lane >> 4;
  int pg_s = -1, pg_u0 = 0, pg = -1;     // this lane's page: that of unit pg_u0 + lane of sequence pg_s
  int issued = 0;
  auto issue = [&](int stage) {
    if (issued < count) {
      if (lc.s != pg_s || lc.u < pg_u0 || lc.u >= pg_u0 + 32) {
        pg_s = lc.s;
        pg_u0 = lc.u;
        const int64_t key = (int64_t)(lc.u + lane) * kUnit + warp * kKeys;
        pg = key < lc.v.len ? page_of(b, lc.s, (int)key) : -1;
      }
      const int key0 = lc.u * kUnit + warp * kKeys;
      const int page = __shfl_sync(0xffffffffu, pg, lc.u - pg_u0);
      const int valid = page < 0 ? 0 : lc.v.len - key0;   // rows that hold keys (may exceed 16)
      const int64_t off = (((int64_t)max(page, 0) * b.heads + lc.h) * b.page_size + (page < 0 ? 0 : key0 % b.page_size)) * kD;
      const T* K = reinterpret_cast<const T*>(a.K) + off + r2 * kD + 8 * c16;
      const T* V = reinterpret_cast<const T*>(a.V) + off + r2 * kD + 8 * c16;
      const uint32_t dst = smem_of(ring + stage * 2 * kTile);
#pragma unroll
      for (int i = 0; i < kKeys / 2; ++i) {
        const int r = 2 * i + r2;
        const uint32_t d = dst + r * (2 * kD) + ((c16 ^ (r & 7)) << 4);
        const uint32_t bytes = r < valid ? 16u : 0u;
        copy16(d, K + 2 * i * kD, bytes);
        copy16(d + kTile, V + 2 * i * kD, bytes);
      }
      ++issued;
      if (issued < count) advance(lc, b);
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  uint32_t q[8][4];
  float o[16][4], m[2], l[2];
  int lim[2];
  bool fresh = true;         // the next unit begins an item (or this CTA's part of one)
  bool began = cc.u == 0;    // the current item began in this CTA's range
  Split split;
  split.s = -1;

  for (int i = 0; i < count; ++i) {
    const int stage = i % kStages;
    copy_wait<kStages - 2>();
    __syncwarp();
    issue((i + kStages - 1) % kStages);
    if (fresh) {
      fresh = false;
      const int R = cc.v.n * g;
      const T* Q = reinterpret_cast<const T*>(a.Q);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = quad + 8 * k;
        const int tok = r / g;
        lim[k] = r < R ? (a.causal ? cc.v.len - cc.v.n + tok : cc.v.len - 1) : -1;
        const T* p = Q + (int64_t)(cc.v.q0 + tok) * a.q_ts + (int64_t)(cc.h * g + r % g) * a.q_hs + 2 * pair;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          q[j][k] = r < R ? *reinterpret_cast<const uint32_t*>(p + 16 * j) : 0u;
          q[j][k + 2] = r < R ? *reinterpret_cast<const uint32_t*>(p + 16 * j + 8) : 0u;
        }
        m[k] = -INFINITY;
        l[k] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    }
    const uint32_t Ks = smem_of(ring + stage * 2 * kTile), Vs = Ks + kTile;
    const int key0 = cc.u * kUnit + warp * kKeys;
    if (key0 < cc.v.len) {
      // scores of 16 rows x 16 keys: matrices (keys 0-7, 8-15) x (features 0-7, 8-15) of each k-step
      float s[2][4] = {};
      const int mrow = (lane & 7) + ((lane >> 4) << 3), mcol = (lane >> 3) & 1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t k4[4];
        ldsm4(Ks + mrow * (2 * kD) + (((2 * j + mcol) ^ (mrow & 7)) << 4), k4);
        mma(T(), s[0], q[j], k4[0], k4[1]);
        mma(T(), s[1], q[j], k4[2], k4[3]);
      }
      // running softmax in units of log 2; lane: rows quad and quad + 8, keys 2 pair, + 1 of each block of 8
      const bool edge = key0 + kKeys - 1 > (a.causal ? cc.v.len - cc.v.n : cc.v.len - 1) || cc.v.n * g < kRows;
      float mn[2] = {m[0], m[1]};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = s[n][e] * scale2;
          if (edge && key0 + 8 * n + 2 * pair + (e & 1) > lim[e >> 1]) x = -INFINITY;
          s[n][e] = x;
          mn[e >> 1] = fmaxf(mn[e >> 1], x);
        }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        mn[k] = fmaxf(mn[k], __shfl_xor_sync(0xffffffffu, mn[k], 1));
        mn[k] = fmaxf(mn[k], __shfl_xor_sync(0xffffffffu, mn[k], 2));
      }
      if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float f = mn[k] == -INFINITY ? 1.0f : ex2(m[k] - mn[k]);
          m[k] = mn[k];
          l[k] *= f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j][2 * k] *= f;
            o[j][2 * k + 1] *= f;
          }
        }
      }
      const float sub[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][e] = ex2(s[n][e] - sub[e >> 1]);
          l[e >> 1] += s[n][e];
        }
      uint32_t hi[4], lo[4];
      split2(T(), s[0][0], s[0][1], hi[0], lo[0]);
      split2(T(), s[0][2], s[0][3], hi[1], lo[1]);
      split2(T(), s[1][0], s[1][1], hi[2], lo[2]);
      split2(T(), s[1][2], s[1][3], hi[3], lo[3]);
      // weighted values: matrices (keys 0-7, 8-15) x (8 features), transposed
      const int vrow = lane & 15, vcol = lane >> 4;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t v4[4];
        ldsm4t(Vs + vrow * (2 * kD) + (((2 * j + vcol) ^ (vrow & 7)) << 4), v4);
        mma(T(), o[2 * j], hi, v4[0], v4[1]);
        mma(T(), o[2 * j + 1], hi, v4[2], v4[3]);
        mma(T(), o[2 * j], lo, v4[0], v4[1]);
        mma(T(), o[2 * j + 1], lo, v4[2], v4[3]);
      }
    }
    const bool ends = cc.u + 1 == cc.U;
    if (ends || i + 1 == count) {
      // join the four warps: maxima and sums first, then the outputs, each warp's in its own stage
      // that was just read (rows of 128 floats; 16-byte blocks swizzled by the row)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 1);
        l[k] += __shfl_xor_sync(0xffffffffu, l[k], 2);
        if (pair == 0) ml_s[warp][quad + 8 * k] = make_float2(m[k], l[k]);
      }
      __syncthreads();
      float* so = reinterpret_cast<float*>(ring + stage * 2 * kTile);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int r = quad + 8 * k;
        float mx = ml_s[0][r].x;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, ml_s[w][r].x);
        const float f = mx == -INFINITY ? 0.0f : ex2(m[k] - mx);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int blk = (2 * j + (pair >> 1)) ^ ((r & 7) << 1);
          *reinterpret_cast<float2*>(so + r * kD + 4 * blk + 2 * (pair & 1)) = make_float2(o[j][2 * k] * f, o[j][2 * k + 1] * f);
        }
      }
      __syncthreads();
      const int R = cc.v.n * g;
      const bool whole = ends && began;
      const int slot = began ? 1 : 0;
      for (int r = warp; r < R; r += kWarps) {
        float mx = -INFINITY, ls = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ml_s[w][r].x);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 p = ml_s[w][r];
          ls += mx == -INFINITY ? 0.0f : p.y * ex2(p.x - mx);
          const float4 x = *reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(sm + (w * kStages + stage) * 2 * kTile) + r * kD + 4 * (lane ^ ((r & 7) << 1)));
          y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
        }
        if (kTeam) {
          *reinterpret_cast<float4*>(sm + kSmem + r * (4 * kD) + 16 * lane) = y;
          if (lane == 0) team_ml[r] = make_float2(mx, ls);
        } else if (whole) {
          const int64_t row = (int64_t)(cc.v.q0 + r / g) * a.Hq + cc.h * g + r % g;
          finish_row<T>(a, row, lane, y, mx, ls);
        } else {
          const int64_t at = ((int64_t)blockIdx.x * 2 + slot) * ws.rows + r;
          *reinterpret_cast<float4*>(ws.o + at * kD + 4 * lane) = y;
          if (lane == 0) ws.ml[at] = make_float2(mx, ls);
        }
      }
      if (began && !ends) {
        split.s = cc.s;
        split.h = cc.h;
        split.m = 0;
        split.slot = slot;
        split.c_last = owner_of(st.lo + i + (cc.U - 1 - cc.u), st.W, st.G);
      }
      __syncthreads();   // the stages are written again
      fresh = began = true;
    }
    if (i + 1 < count) advance(cc, b);
  }
  if (!kTeam) {
    if (tid == 0) ws.list[blockIdx.x] = split;
    return;
  }
  // the cluster's parts: CTA k finishes the rows k and k + 8, a warp each
  if (count == 0 && tid < kRows) team_ml[tid] = make_float2(-INFINITY, 0.0f);
  const cooperative_groups::cluster_group team = cooperative_groups::this_cluster();
  team.sync();
  const int r = blockIdx.x % kTeamCtas + kTeamCtas * warp;
  if (r < cc.v.n * g) {
    float2 p[kTeamCtas];
    float4 x[kTeamCtas], y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float mx = -INFINITY, ls = 0.0f;
#pragma unroll
    for (int c = 0; c < kTeamCtas; ++c) {
      p[c] = *team.map_shared_rank(&team_ml[r], c);
      x[c] = *reinterpret_cast<const float4*>(team.map_shared_rank(sm + kSmem + r * (4 * kD) + 16 * lane, c));
    }
#pragma unroll
    for (int c = 0; c < kTeamCtas; ++c) mx = fmaxf(mx, p[c].x);
#pragma unroll
    for (int c = 0; c < kTeamCtas; ++c) {
      if (p[c].x == -INFINITY) continue;   // no keys, and perhaps no output written
      const float f = ex2(p[c].x - mx);
      ls = fmaf(p[c].y, f, ls);
      y.x = fmaf(x[c].x, f, y.x);
      y.y = fmaf(x[c].y, f, y.y);
      y.z = fmaf(x[c].z, f, y.z);
      y.w = fmaf(x[c].w, f, y.w);
    }
    finish_row<T>(a, (int64_t)(cc.v.q0 + r / g) * a.Hq + cc.h * g + r % g, lane, y, mx, ls);
  }
  team.sync();   // no CTA leaves while another reads from it
}

template <typename T>
cudaError_t launch(const PagedAttnArgs& a, const AttnPlan& p, const Workspace& w, cudaStream_t s) {
  static SmemFlags allowed, allowed_team;
  cudaError_t e;
  if (p.team) {
    e = allow_smem(k_attn_decode<T, true>, kTeamSmem, a.device, allowed_team);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kTeamSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kTeamCtas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, k_attn_decode<T, true>, a, w);
  } else {
    e = allow_smem(k_attn_decode<T, false>, kSmem, a.device, allowed);
    if (e != cudaSuccess) return e;
    k_attn_decode<T, false><<<p.grid, kThreads, kSmem, s>>>(a, w);
  }
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t attn_decode(const PagedAttnArgs& a, const AttnPlan& p, const Workspace& w, cudaStream_t s) {
  return a.dtype == JOLT_BF16 ? launch<__nv_bfloat16>(a, p, w, s) : launch<__half>(a, p, w, s);
}

}  // namespace jolt
