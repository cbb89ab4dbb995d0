// Shared device code of the paged attention kernels: how a batch's work is divided, the join with a
// prefix, and the workspace that carries an item's parts from one kernel to the next.
#pragma once

#include <algorithm>

#include "../paged.h"
#include "sm100.cuh"

namespace jolt {
namespace pattn {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x by the special function unit (2 units in the last place; exp2(-inf) = 0).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The work of a call is a line of units: the sequences in order, in each its items (the rows of one
// KV head that are attended together), in each item its blocks of keys. The CTAs take shares of one
// length of it, so that all end together whatever the sequences' lengths are. An item that falls
// into several CTAs leaves a part in each: its running maximum, sum and unscaled output, in slot 0 when
// the item began before the CTA's range and slot 1 otherwise. Where an item begins in a CTA and
// does not end there (one at most per CTA), the CTA lists it for the combining kernel.
struct Split {
  int32_t s, h, m;     // sequence, KV head, block of rows; s < 0: none
  int32_t c_last;      // CTA that holds its last unit (the first one is the list's index)
  int32_t slot;        // slot of its first part
  int32_t q0, rows;    // first token of the sequence's chunk; rows of the item
};
struct Workspace {
  float* o;            // [G][2][rows][128]
  float2* ml;          // [G][2][rows]: maximum (in units of log 2), sum
  Split* list;         // [G]
  int32_t rows;
};

// Quotient by a divisor that fits 32 bits; the long division only where the dividend does not.
__device__ __forceinline__ int64_t quot(int64_t a, uint32_t b) {
  return (uint64_t)a >> 32 ? a / b : (int64_t)((uint32_t)a / b);
}
// The shares: the first W % G CTAs have W / G + 1 units, the others W / G.
__device__ __forceinline__ int64_t share_begin(int c, int64_t each, int64_t more) { return c * each + min((int64_t)c, more); }
// CTA whose share holds unit u.
__device__ __forceinline__ int owner_of(int64_t u, int64_t each, int64_t more) {
  const int64_t longer = more * (each + 1);
  if (u < longer) return (int)(u / (each + 1));
  return (int)(more + (u - longer) / each);
}

struct Start {
  int64_t each, more;  // units of a share, shares that have one more
  int64_t lo, hi;      // this CTA's
  int64_t base, units; // the sequence that holds lo: its first unit, its number of them
  int32_t s, G;        // its index; CTAs that have work
};

template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sm, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) sm[warp] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const int64_t x = sm[w];
    before += w < warp ? x : 0;
    total += x;
  }
  __syncthreads();
  return v + before;   // inclusive
}

// This CTA's share of the line: work(s) is the units of sequence s, 0 behind the last; a CTA takes min_units at least.
// Called by all NT threads (NT a multiple of 32); sm: NT / 32 + 3 words of shared memory, free again on
// return and a barrier.
template <int NT, class F>
__device__ __forceinline__ Start find_start(int num_seqs, F work, int min_units, int64_t* sm) {
  int64_t &base_s = sm[NT / 32], &units_s = sm[NT / 32 + 1], &seq_s = sm[NT / 32 + 2];
  Start r{};
  const int tid = threadIdx.x;
  int64_t mine = work(tid), sum = mine;
  for (int s0 = NT; s0 < num_seqs; s0 += NT) sum += work(s0 + tid);
  int64_t total, base = 0;
  int64_t incl = block_scan<NT>(sum, sm, total);
  const int64_t most = quot(total + min_units - 1, min_units);
  r.G = (int)(most < (int64_t)gridDim.x ? most : (int64_t)gridDim.x);
  if ((int)blockIdx.x >= r.G) return r;
  r.each = quot(total, r.G);
  r.more = total - r.each * r.G;
  r.lo = share_begin(blockIdx.x, r.each, r.more);
  r.hi = share_begin(blockIdx.x + 1, r.each, r.more);
  if (num_seqs <= NT) {   // the scan just made is the one over sequences
    if (incl > r.lo && incl - mine <= r.lo) {
      base_s = incl - mine;
      units_s = mine;
      seq_s = tid;
    }
    __syncthreads();
  } else {
    for (int s0 = 0; s0 < num_seqs; s0 += NT) {
      const int64_t v = work(s0 + tid);
      incl = base + block_scan<NT>(v, sm, total);
      if (incl > r.lo && incl - v <= r.lo) {
        base_s = incl - v;
        units_s = v;
        seq_s = s0 + tid;
      }
      base += total;
      if (base > r.lo) break;   // uniform
    }
    __syncthreads();
  }
  r.base = base_s;
  r.units = units_s;
  r.s = (int)seq_s;
  return r;
}

// Four features of a row's prefix (lane i: 4 i ..) and its log-sum-exp, in units of log 2; -inf for none.
// Loaded apart from finish_row, so that the loads run while a row's parts are summed.
struct Prefix {
  float4 x;
  float lse;
};
// 1 / l and the log-sum-exp of a row of maximum m (units of log 2) and sum l; 0 and -inf without keys (l is
// 1 at least where there are any, or no number).
__device__ __forceinline__ float inverse_sum(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2; }
// What weights of maximum m are scaled by to be relative to mx >= m: 0 where there are none, as ex2(-inf) is. A
// row whose scores are no numbers has m = -inf and l = NaN, which 0 keeps.
__device__ __forceinline__ float rescale(float m, float mx) { return mx == -INFINITY ? 0.0f : ex2(m - mx); }

__device__ __forceinline__ Prefix load_prefix(const PagedAttnArgs& a, int64_t row, int lane) {
  Prefix p{make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY};
  if (a.pre_lse) {
    p.lse = a.pre_lse[row] * kLog2e;
    p.x = *reinterpret_cast<const float4*>(a.pre_out + row * kD + 4 * lane);
  }
  return p;
}

// Four output features of one row, from the unscaled sum o, maximum m (units of log 2) and sum l:
// joined with the prefix, scaled, rounded and stored; lane 0 stores the log-sum-exp.
template <typename T>
__device__ __forceinline__ void finish_row(const PagedAttnArgs& a, int64_t row, int lane, float4 o, float m, float l,
                                           const Prefix& p) {
  if (p.lse != -INFINITY) {
    const float mx = fmaxf(m, p.lse), f = rescale(m, mx), w = ex2(p.lse - mx);
    l = fmaf(l, f, w);
    o.x = fmaf(o.x, f, w * p.x.x);
    o.y = fmaf(o.y, f, w * p.x.y);
    o.z = fmaf(o.z, f, w * p.x.z);
    o.w = fmaf(o.w, f, w * p.x.w);
    m = mx;
  }
  const float inv = inverse_sum(l);
  T y[4] = {(T)(o.x * inv), (T)(o.y * inv), (T)(o.z * inv), (T)(o.w * inv)};
  *reinterpret_cast<uint2*>(reinterpret_cast<T*>(a.out) + row * kD + 4 * lane) = *reinterpret_cast<const uint2*>(y);
  if (a.lse && lane == 0) a.lse[row] = log_sum(m, l);
}

// Values that some rows of a block see and others do not (causal) may be no numbers, which a weight of zero
// does not hide in a matrix product. A warp looks for them in a tile in shared memory (two halves of 128-byte
// rows, `half` apart) and zeroes them there; the rows that see them look them up in the pages at the end
// (hidden16) and show NaN in their features. x 0 + sum is 0 until an x is no finite number.
__device__ __forceinline__ uint32_t times_0(__nv_bfloat16, uint32_t x, uint32_t sum) {
  const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), __floats2bfloat162_rn(0.0f, 0.0f),
                                   *reinterpret_cast<const __nv_bfloat162*>(&sum));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ uint32_t times_0(__half, uint32_t x, uint32_t sum) {
  const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&x), __floats2half2_rn(0.0f, 0.0f),
                            *reinterpret_cast<const __half2*>(&sum));
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ constexpr uint32_t exponent(__nv_bfloat16) { return 0x7f80; }
__device__ __forceinline__ constexpr uint32_t exponent(__half) { return 0x7c00; }
// Whether all is finite in rows ra .. rb - 1 of the tile.
template <typename T, int kAhead>
__device__ __forceinline__ bool finite(const uint8_t* tile, uint32_t half, int ra, int rb, int lane) {
  uint32_t sum[4] = {0, 0, 0, 0};
#pragma unroll kAhead
  for (int u = 2 * ra + (lane >> 3); u < 2 * rb; u += 4) {   // a half row each
    const uint4 v = *reinterpret_cast<const uint4*>(tile + (u & 1) * half + (u >> 1) * 128 + (lane & 7) * 16);
    sum[0] = times_0(T(), v.x, sum[0]);
    sum[1] = times_0(T(), v.y, sum[1]);
    sum[2] = times_0(T(), v.z, sum[2]);
    sum[3] = times_0(T(), v.w, sum[3]);
  }
  return !__any_sync(0xffffffffu, ((sum[0] | sum[1] | sum[2] | sum[3]) & 0x7fff7fffu) != 0);
}
// Zeroes in them what is not.
template <typename T>
__device__ __forceinline__ void hide(uint8_t* tile, uint32_t half, int ra, int rb, int lane) {
  const uint32_t e = exponent(T());
#pragma unroll 1
  for (int u = 64 * ra + lane; u < 64 * rb; u += 32) {   // two elements each
    uint32_t* w = reinterpret_cast<uint32_t*>(tile + ((u >> 5) & 1) * half + (u >> 6) * 128) + (u & 31);
    uint32_t x = *w;
    if ((x & e) == e) x &= 0xffff0000u;
    if (((x >> 16) & e) == e) x &= 0xffffu;
    *w = x;
  }
}
// Which of the features d0 .. d0 + 15 of the keys from .. to of a sequence are no finite numbers.
template <typename T>
__device__ __forceinline__ uint32_t hidden16(const PagedAttnArgs& a, int s, int h, int from, int to, int d0) {
  uint32_t found = 0;
#pragma unroll 1
  for (int key = max(from, 0); key <= to; ++key) {
    const int page = page_of(a.b, s, key);
    if (page < 0) continue;
    const uint16_t* v = reinterpret_cast<const uint16_t*>(a.V) +
                        (((int64_t)page * a.b.heads + h) * a.b.page_size + key - a.b.by_page.quot(key) * a.b.page_size) * kD + d0;
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if ((v[i] & exponent(T())) == exponent(T())) found |= 1u << i;
  }
  return found;
}

// Tensor maps of the pages.
struct Maps {
  CUtensorMap K, V;
};

// A bounded wait that also ends when another role of the CTA has given up. The clock is looked at
// only every 64 polls.
struct Waits {
  volatile int* gave_up;
  int32_t* status;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    const uint32_t a = smem_u32(bar);
    uint64_t t0 = 0;
    for (uint32_t it = 1;; ++it) {
      uint32_t done;
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done)
          : "r"(a), "r"(parity)
          : "memory");
      if (done) return true;
      if (*gave_up) return false;
      if ((it & 63) == 0) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (now - t0 > kWaitLimitNs) {
          *gave_up = 1;
          atomicOr(status, PST_TIMEOUT);
          return false;
        }
      }
    }
  }
};

}  // namespace pattn

// The two kernels.
cudaError_t attn_decode(const PagedAttnArgs& a, const AttnPlan& p, const pattn::Workspace& w, cudaStream_t s);
cudaError_t attn_chunk(const PagedAttnArgs& a, const AttnPlan& p, const pattn::Workspace& w, cudaStream_t s);

}  // namespace jolt
