// Paged attention of many query rows (chunks of a prompt, whole prompts): the rows of a chunk that
// read one KV head (token-major: row r is token r / g, query head h g + r % g) in blocks of 256.
//
// Two matrix products of 128 x 128 x 128 a tile of 128 keys and half block, and one exponential a
// score: at 4 exponentials a cycle and sub-partition both take about 1000 cycles, so the tensor
// pipe and the special function unit bound it alike. One persistent CTA an SM walks its share
// of the units (128 keys of one item). Its warps: two softmax groups of four, one for each half
// block (a thread a row; two threads a row, who have to agree on the maximum, took 3 to 4 % longer); one
// that issues the MMAs (tcgen05, 128 x 128 accumulators in Tensor
// Memory: scores and outputs of both halves fill its 512 columns); one that loads keys and values
// by TMA, a box of up to 128 rows of a page at a time, into a ring of five 32 KB stages; two that gather
// the query rows. While one half's scores are turned into weights, the tensor pipe works for the
// other. Weights overwrite their scores in Tensor Memory and are the second product's A operand
// from there, so only keys, values and queries pass through shared memory.
// The weights are rounded to the type of the values (the tensor pipe takes no wider ones; up to 128 rows
// what the rounding left follows as a second operand, kFew); their sum is not. A maximum that grows by less than 8 (in units of log 2; 6 in fp16) is not followed: weights up to 2^8
// are as exact, and most rescalings of the output fall away.
// Measured (32 query heads on 8): 2048 tokens over 32768 keys 0.97 PFLOP/s in a sustained run, where the
// card is at its power limit, up to 1.18 in a short one; a prompt of 8192 tokens 1.00; items of one or two
// tiles are bound by the chain of an item (queries, scores, weights, output), 10 us.
#include <type_traits>

#include "f32x2.cuh"
#include "paged_attention.cuh"
#include "sm100.cuh"

namespace jolt {
namespace {

using namespace pattn;
using namespace sm100;
using namespace f32x2;

constexpr int kHalf = 128;                   // rows of a half block, keys of a tile
constexpr int kBlockRows = 2 * kHalf;
constexpr int kStages = 5;
constexpr uint32_t kTileBytes = kHalf * kD * 2;
constexpr uint32_t kHalfTile = kTileBytes / 2;   // 128 rows x 64 features
constexpr int kSoftmaxWarps = 8;
constexpr int kThreads = 32 * (kSoftmaxWarps + 4);
constexpr int kRegsSoftmax = 200, kRegsOther = 104;   // 256 x 200 + 128 x 104 = 384 x 168
constexpr int kSmem = (2 + kStages) * kTileBytes;
constexpr int kItem = 3;                     // what an item costs besides its tiles, in tiles
// A maximum that grows by no more than kFollow (in units of log 2) is not followed, and weights are 2^kLift times as
// large as beside a maximum of 1: fp16 has nothing below 2^-24, and what lies so far below the largest counts where
// the keys are many, so there the largest weight is moved up to 2^15 and each is held to 2^-34 of it, whole down to
// 2^-23 (unmoved, all below 2^-25 was lost: keys 17.4 lower in the exponent). A prompt of 4096 tokens in fp16:
// 150.9 us, 149.1 with 8 and 2^7, 156.5 with 4 and 2^11.
template <typename T>
constexpr float kFollow = std::is_same_v<T, __half> ? 6.0f : 8.0f;
template <typename T>
constexpr float kLift = std::is_same_v<T, __half> ? 9.0f : 0.0f;
// What the weights are relative to beside the maximum m, and a score in units of log 2 as a maximum. Both are rounded
// up where there is a lift: with scores of 2^24 and more a last place is a whole unit, and no weight may pass 2^15 for it.
template <typename T>
__device__ __forceinline__ float base_of(float m) {
  return kLift<T> == 0.0f ? m : __fsub_ru(m, kLift<T>);
}
template <typename T>
__device__ __forceinline__ float top_of(float s, float scale2) {
  return kLift<T> == 0.0f ? s * scale2 : __fmul_ru(s, scale2);
}

struct Bars {
  uint64_t kv_full[kStages], kv_empty[kStages];
  uint64_t q_full[2], q_empty[2], s_full[2], p_lo[2], p_hi[2], o_full[2], o_empty[2];
  uint64_t tail, drain;
};

__device__ __forceinline__ int blocks_of(const SeqView& v, const Divisor& g) {
  return (v.n * (int)g.d + kBlockRows - 1) / kBlockRows;
}
// Keys that block m of the sequence's rows sees (none where it is not positive), and their tiles (one at least,
// so that empty rows are written).
__device__ __forceinline__ int seen_of(const SeqView& v, const Divisor& g, int m, bool causal) {
  return causal ? v.len + g.quot(min(v.n * (int)g.d, (m + 1) * kBlockRows) - 1) + 1 - v.n : v.len;
}
__device__ __forceinline__ int tiles_of(const SeqView& v, const Divisor& g, int m, bool causal) {
  return max(1, (seen_of(v, g, m, causal) + kHalf - 1) / kHalf);
}

// A part of an item: tiles t0 .. t1 - 1 of its T. On the line an item takes kItem units (its begin and
// end: queries in, output out) and one for each tile after them.
struct Piece {
  int s, h, m, M, t0, t1, T;
  int upto;         // keys that the block sees
  SeqView v;
  int left;         // units of the CTA's share behind the piece
};
// The piece of an item from its unit u on; false if the share ends before the item's first tile.
__device__ __forceinline__ bool enter(Piece& p, int u, const Divisor& g, bool causal) {
  p.upto = max(0, seen_of(p.v, g, p.m, causal));
  p.T = max(1, (p.upto + kHalf - 1) / kHalf);
  const int take = min(p.T + kItem - u, p.left);
  p.left -= take;
  p.t0 = max(u - kItem, 0);
  p.t1 = u + take - kItem;
  return p.t1 > p.t0;
}
// The next piece of the share; false behind the last.
__device__ __forceinline__ bool next(Piece& p, const BatchView& b, const Divisor& g, bool causal) {
  if (p.left <= 0) return false;
  if (++p.m == p.M) {
    p.m = 0;
    if (++p.h == b.heads) {
      p.h = 0;
      do {
        if (++p.s >= b.num_seqs) return false;
        p.v = seq_view(b, p.s);
        p.M = blocks_of(p.v, g);
      } while (p.M == 0);
    }
  }
  return enter(p, 0, g, causal);
}

// Barrier of the two warps, one of each half, that have the same rows when the halves share an item.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// Whether an item's rows fill one half only: the halves then take its tiles in turn, with the same
// queries, and their outputs are joined at the end.
__device__ __forceinline__ bool solo(const Piece& p, const Divisor& g) { return p.v.n * (int)g.d - p.m * kBlockRows <= kHalf; }

// A warp's common place moved on by its first lane.
__device__ __forceinline__ bool next_of_warp(Piece& p, const BatchView& b, const Divisor& g, bool causal, int lane) {
  __syncwarp();
  bool more = false;
  if (lane == 0) more = next(p, b, g, causal);
  more = __shfl_sync(0xffffffffu, more, 0);
  __syncwarp();
  return more;
}

__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(bdesc), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(__half, float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t wide2(__nv_bfloat16, uint32_t v) {
  return pair_of(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ uint64_t wide2(__half, uint32_t v) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v));
  return pair_of(f.x, f.y);
}
template <typename T>
__device__ __forceinline__ constexpr uint32_t idesc();
template <>
__device__ __forceinline__ constexpr uint32_t idesc<__nv_bfloat16>() {
  return idesc_bf16_f32(kHalf, kHalf);
}
template <>
__device__ __forceinline__ constexpr uint32_t idesc<__half>() {
  return idesc_f16_f32(kHalf, kHalf);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The weights 2^(s scale2 + sub) of a row, rounded to the type, written to Tensor Memory (tP); their
// sum goes to l unrounded. kRest: what the rounding left, rounded, behind them (kRestAt). The first half is
// announced while the second is made. (Making 1 or 2 of 8
// exponentials by a polynomial on the multiply-add units, to spare the special function unit, gave 0 and
// -8 % on a chunk of 2048 tokens over 32768 keys. Leaving out those of 32 keys that no row of the warp sees,
// by a branch, made items of one or two tiles 5 % faster and prompts 4 % slower.)
constexpr uint32_t kRestAt = kHalf / 2;      // columns
template <typename T, bool kRest>
__device__ __forceinline__ void weights(float (&s)[kHalf], float scale2, float sub, float& l, uint32_t tP,
                                        uint64_t* lo, uint64_t* hi, int lane) {
  const uint64_t sc = pair_of(scale2, scale2), sb = pair_of(sub, sub);
  uint64_t sum[2] = {pair_of(0.0f, 0.0f), pair_of(0.0f, 0.0f)};
#pragma unroll
  for (int c = 0; c < kHalf / 32; ++c) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint64_t x2 = fma2(pair_of(s[32 * c + 2 * i], s[32 * c + 2 * i + 1]), sc, sb);
      float x, y;
      unpair(x2, x, y);
      x = ex2(x);
      y = ex2(y);
      sum[i & 1] = add2(sum[i & 1], pair_of(x, y));
      w[i] = pack2(T(), x, y);
      if (kRest)   // in the place of the scores
        unpair(fma2(wide2(T(), w[i]), pair_of(-1.0f, -1.0f), pair_of(x, y)), s[32 * c + 2 * i], s[32 * c + 2 * i + 1]);
    }
    tmem_st16(tP + 16 * c, w);
    if (kRest) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = pack2(T(), s[32 * c + 2 * i], s[32 * c + 2 * i + 1]);
      tmem_st16(tP + kRestAt + 16 * c, w);
    }
    if (c & 1) {
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(c == 1 ? lo : hi);
    }
  }
  float x, y;
  unpair(add2(sum[0], sum[1]), x, y);
  l += x + y;
}

// Four lanes each hold four 16-byte blocks; afterwards block k of a lane is its own numbered block of
// the group's lane k.
__device__ __forceinline__ void transpose4(uint32_t (&y)[4][4], int lane) {
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k & d) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t give = up ? y[k][e] : y[k | d][e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, d);
        if (up) y[k][e] = got;
        else y[k | d][e] = got;
      }
    }
  }
}

// Sixteen columns of a row's output times f0, and with those of half 1 times f1.
__device__ __forceinline__ void output16(uint32_t t0, float f0, bool both, float f1, float (&v)[16]) {
  uint32_t o[16];
  tmem_ld16(t0, o);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(o[i]) * f0;
  if (both) {
    tmem_ld16(t0 + kHalf, o);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = fmaf(__uint_as_float(o[i]), f1, v[i]);
  }
}

// Rare, so kept out of the kernel's code: NaN where a row of the piece that sees the keys up to lim sees a value
// that is no finite number, in out (blocks of one feature) or a part (blocks of four).
template <typename T>
__device__ __noinline__ void show_values(const PagedAttnArgs& a, const Piece& p, int lim, T* out, float* part) {
  const Divisor& g = a.g;
  for (int d0 = 0; d0 < kD; d0 += 16) {
    const uint32_t found = hidden16<T>(a, p.s, p.h, p.v.len - p.v.n + g.quot(p.m * kBlockRows) + 1, lim, d0);
    for (int d = d0; d < d0 + 16; ++d) {
      if (!((found >> (d - d0)) & 1)) continue;
      if (out) out[d] = (T)NAN;
      else part[(d >> 2) * (4 * kBlockRows) + (d & 3)] = NAN;
    }
  }
}

// Where a wait gave up, copies and products in flight end before the CTA's memory and its Tensor Memory are given
// up; never in a run that ends well, so kept out of the kernel's code. Copies: those of the ring's last stages, and of
// a tile that was to be looked over.
__device__ __noinline__ void land(uint64_t* full, uint32_t kv, uint64_t* tail, uint32_t tails) {
  if (tails) mbar_wait(tail, (tails - 1) & 1, 1u << 20);
  const uint32_t n = min(kv, (uint32_t)kStages);
  for (uint32_t i = kv - n; i < kv; ++i) mbar_wait(&full[i % kStages], (i / kStages) & 1, 1u << 20);
}
__device__ __noinline__ void drain(uint64_t* bar) {
  umma_commit(bar);
  mbar_wait(bar, 0, 1u << 20);
}

// kFew: no item has more than half a block of rows. Their weights' remainders enter the second product too, as
// in the kernel for fewer rows, so that only the output is rounded: these calls wait for memory or an item's chain and not
// for the tensor pipe (16 sequences over up to 4096 keys: 42.8 us with them and 40.8 without for 2 to 5 drafted tokens, 65.6
// and 64.2 for 32). As a branch of one kernel it cost prompts 4 to 10 %, and items of whole blocks a third.
template <typename T, bool kFew>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_chunk(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ Maps maps, const Workspace ws, int box) {
  extern __shared__ __align__(1024) uint8_t sm[];   // what is static takes the rest, 3 KB
  __shared__ __align__(8) Bars bar;
  __shared__ uint32_t tmem_s;
  __shared__ int gave_up;
  __shared__ Piece first_s, piece_s[kSoftmaxWarps + 4];   // the share's begin, each warp's place on the line
  __shared__ bool any_s;
  __shared__ bool hid_s[8];                // whether a piece's values hold what was hidden: the last pieces'
  __shared__ float2 told_s[kHalf];         // what half 1 tells half 0
  __shared__ int64_t range_s[3];   // the end of this CTA's share, units of a share, shares with one more
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const BatchView& b = a.b;
  const Divisor& g = a.g;
  const bool causal = a.causal;
  grid_release();
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bar.kv_full[i], 1);
      mbar_init(&bar.kv_empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar.q_full[t], 32);
      mbar_init(&bar.q_empty[t], 1);
      mbar_init(&bar.s_full[t], 1);
      mbar_init(&bar.p_lo[t], kSoftmaxWarps / 2);
      mbar_init(&bar.p_hi[t], kSoftmaxWarps / 2);
      mbar_init(&bar.o_full[t], 1);
      mbar_init(&bar.o_empty[t], kSoftmaxWarps / 2);
    }
    mbar_init(&bar.tail, 1);
    mbar_init(&bar.drain, 1);
    gave_up = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.K);
    prefetch_tensormap(&maps.V);
  }
  if (warp == kSoftmaxWarps) {
    tmem_alloc(&tmem_s, 512);
    tmem_relinquish();
  }
  grid_wait();
  const Start st = find_start<kThreads>(
      b.num_seqs,
      [&](int s) {   // of a warp's 32 sequences at once, those of more than four blocks one by one
        SeqView v{0, 0, 0};
        if (s < b.num_seqs) v = seq_view(b, s);
        const int M = blocks_of(v, g);
        int64_t n = 0;
        if (M <= 4)
          for (int m = 0; m < M; ++m) n += tiles_of(v, g, m, causal) + kItem;
        for (uint32_t more = __ballot_sync(0xffffffffu, M > 4); more; more &= more - 1) {
          const int from = __ffs(more) - 1, blocks = __shfl_sync(0xffffffffu, M, from);
          const SeqView w{0, __shfl_sync(0xffffffffu, v.n, from), __shfl_sync(0xffffffffu, v.len, from)};
          int64_t sum = 0;
          for (int m = lane; m < blocks; m += 32) sum += tiles_of(w, g, m, causal) + kItem;
#pragma unroll
          for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (lane == from) n = sum;
        }
        return n * b.heads;
      },
      kItem + 2, reinterpret_cast<int64_t*>(told_s));
  if ((int)blockIdx.x >= st.G) {
    if (tid == 0) ws.list[blockIdx.x].s = -1;
    if (warp == kSoftmaxWarps) tmem_dealloc(tmem_s, 512);
    return;
  }
  if (warp == 0) {   // the share's first piece
    Piece p;
    p.s = st.s;
    p.v = seq_view(b, p.s);
    p.M = blocks_of(p.v, g);
    const int64_t per = quot(st.units, b.heads), from = st.lo - st.base;   // (a head's units fit 31 bits)
    p.h = (int)quot(from, (uint32_t)per);
    int at = (int)(from - p.h * per);
    for (p.m = 0; p.m < p.M; p.m += 32) {   // 32 blocks at a time
      const int n = p.m + lane < p.M ? tiles_of(p.v, g, p.m + lane, causal) + kItem : 0;
      int to = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += y;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, at < to);
      const int k = in ? __ffs(in) - 1 : 31;
      at -= __shfl_sync(0xffffffffu, in ? to - n : to, k);
      if (in) {
        p.m += k;
        break;
      }
    }
    if (lane == 0) {
      p.left = (int)(st.hi - st.lo);
      any_s = enter(p, at, g, causal);   // a share can lie in an item's first units only
      first_s = p;
      range_s[0] = st.hi;
      range_s[1] = st.each;
      range_s[2] = st.more;
      ws.list[blockIdx.x].s = -1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_s;
  if (lane < (int)(sizeof(Piece) / 4))
    reinterpret_cast<int32_t*>(&piece_s[warp])[lane] = reinterpret_cast<const int32_t*>(&first_s)[lane];
  __syncwarp();
  const Waits wait{&gave_up, b.status};
  uint8_t* Qs = sm;
  uint8_t* ring = sm + 2 * kTileBytes;

  if (!any_s) {
    // nothing to do: on to the end
  } else if (warp >= kSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kSoftmaxWarps) {
      // ---------------------------------------------------------------- MMA issue
      if (elect_one()) {
        Piece& p = piece_s[warp];
        constexpr uint32_t id_qk = idesc<T>(), id_pv = idesc<T>() | (1u << 16);   // V: MN-major
        uint32_t kv = 0, queries[2] = {0, 0}, outputs[2] = {0, 0}, tiles[2] = {0, 0};
        bool ok = true;
        auto full = [&](uint32_t i) { return wait(&bar.kv_full[i % kStages], (i / kStages) & 1); };
        auto qk = [&](int t, int q, uint32_t i) {   // scores of half t, from queries q and the stage
          const uint64_t A = desc_kmajor_sw128(smem_u32(Qs + q * kTileBytes));
          const uint64_t B = desc_kmajor_sw128(smem_u32(ring + (i % kStages) * kTileBytes));
#pragma unroll
          for (int k = 0; k < 8; ++k) {   // the address field counts 16 bytes
            const uint32_t off = ((k >> 2) * kHalfTile + (k & 3) * 32) >> 4;
            umma_bf16(tmem + t * kHalf, A + off, B + off, id_qk, k != 0);
          }
          umma_commit(&bar.s_full[t]);
        };
        auto pv = [&](int t, uint32_t i, bool first) {   // output of half t (+)= its weights times the stage
          if (!wait(&bar.p_lo[t], tiles[t] & 1)) return false;
          if (first && !wait(&bar.o_empty[t], (outputs[t]++ & 1) ^ 1)) return false;
          tc_fence_after();
          const uint64_t B = desc_mnmajor_sw128(smem_u32(ring + (i % kStages) * kTileBytes), kHalfTile, 1024);
#pragma unroll
          for (int k = 0; k < 8; ++k) {   // 16 keys a step: the first 64 are announced first
            if (k == 4) {
              if (!wait(&bar.p_hi[t], tiles[t] & 1)) return false;
              tc_fence_after();
            }
            umma_ts(tmem + (2 + t) * kHalf, tmem + t * kHalf + 8 * k, B + k * (2048 >> 4), id_pv, !first || k != 0);
            if (kFew) umma_ts(tmem + (2 + t) * kHalf, tmem + t * kHalf + kRestAt + 8 * k, B + k * (2048 >> 4), id_pv, 1);
          }
          ++tiles[t];
          return true;
        };
        auto query = [&](int t) {
          const bool in = wait(&bar.q_full[t], queries[t]++ & 1);
          tc_fence_after();
          return in;
        };
        do {
          const int nt = p.t1 - p.t0;
          if (kFew || solo(p, g)) {
            // the halves take the tiles in turn, each ahead of the other by its softmax
            const int lead = min(nt, 2);
            if (!(ok = query(0))) break;
            for (int j = 0; j < lead && (ok = full(kv)); ++j, ++kv) {
              tc_fence_after();
              qk(j, 0, kv);
              umma_commit(&bar.kv_empty[kv % kStages]);
            }
            if (ok && nt <= 2) umma_commit(&bar.q_empty[0]);
            for (int j = 0; j < nt && ok; ++j) {
              const int t = j & 1;
              if (!(ok = full(kv) && pv(t, kv, j < 2))) break;
              umma_commit(&bar.kv_empty[kv++ % kStages]);
              if (j + 2 < nt) {
                if (!(ok = full(kv))) break;
                tc_fence_after();
                qk(t, 0, kv);
                if (j + 3 == nt) umma_commit(&bar.q_empty[0]);
                umma_commit(&bar.kv_empty[kv++ % kStages]);
              } else {
                umma_commit(&bar.o_full[t]);
              }
            }
          } else {
            ok = full(kv);
            for (int t = 0; t < 2 && ok; ++t)
              if ((ok = query(t))) qk(t, t, kv);
            if (!ok) break;
            umma_commit(&bar.kv_empty[kv % kStages]);
            if (nt == 1)
              for (int t = 0; t < 2; ++t) umma_commit(&bar.q_empty[t]);
            for (int j = 0; j < nt && ok; ++j, kv += 2) {
              const uint32_t iv = kv + 1, ik = kv + 2;   // V of this tile, K of the next
              const bool more = j + 1 < nt;
              for (int t = 0; t < 2 && ok; ++t) {
                if (!(ok = (t || full(iv)) && pv(t, iv, j == 0))) break;
                if (more) {
                  if (!(ok = t || full(ik))) break;
                  tc_fence_after();
                  qk(t, t, ik);
                  if (j + 2 == nt) umma_commit(&bar.q_empty[t]);
                } else {
                  umma_commit(&bar.o_full[t]);
                }
              }
              if (!ok) break;
              umma_commit(&bar.kv_empty[iv % kStages]);
              if (more) umma_commit(&bar.kv_empty[ik % kStages]);
            }
          }
        } while (ok && next(p, b, g, causal));
        if (!ok) drain(&bar.drain);
      }
    } else if (warp == kSoftmaxWarps + 1) {
      // ---------------------------------------------------------------- keys and values
      Piece& p = piece_s[warp];
      uint32_t kv = 0, tails = 0, pieces = 0;
      const int box_log = 31 - __clz(box), per_log = 7 - box_log, per = 1 << per_log;   // boxes of a tile: one lane each
      // Pages are looked up for 32 boxes at once: lane i has that of box i % per of tile pg_j + i / per.
      const int tile_l = lane >> per_log, box_l = lane & (per - 1), ahead = 32 >> per_log;
      int pg = -1, pg_s = -1, pg_j = 0;
      bool ok = true;
      do {
        const int t0 = p.t0, nt = p.t1 - t0, len = p.v.len, upto = p.upto, h = p.h, seq = p.s;
        const bool alone = kFew || solo(p, g);
        const int seen = causal ? len - p.v.n + g.quot(p.m * kBlockRows) : len - 1;   // the last key that all rows see
        // (the ring holds the tiles of three pieces at most, and the softmax is at most two behind those)
        bool* hid = &hid_s[pieces++ & 7];
        if (lane == 0) *hid = false;
        for (int x = 0; x < 2 * nt && ok; ++x, ++kv) {
            // K0 V0 K1 V1 ..., or as the halves take them in turn K0 K1 V0 K2 V1 K3 ... V(nt - 2) V(nt - 1)
            int kind = x & 1, j = x >> 1;
            if (alone && x > 0 && nt > 1) {
              kind = x > 1 && ((x & 1) == 0 || x == 2 * nt - 1);
              j = x == 1 ? 1 : x == 2 * nt - 1 ? nt - 1 : (x & 1) ? (x + 1) >> 1 : (x - 2) >> 1;
            }
            j += t0;
            const int key = j * kHalf + lane * box;     // this lane's box
            if (seq != pg_s || j < pg_j || j >= pg_j + ahead) {
              pg_s = seq;
              pg_j = max(j - 1, 0);          // the halves' turns go back by one
              const int64_t k = (int64_t)(pg_j + tile_l) * kHalf + box_l * box;
              pg = k < len ? page_of(b, seq, (int)k) : -1;
            }
            const bool mine = lane < per && key < upto;
            int page = __shfl_sync(0xffffffffu, pg, ((j - pg_j) << per_log) + box_l);
            if (!mine) page = -1;
            const uint32_t good = __ballot_sync(0xffffffffu, page >= 0);
            const bool whole = __all_sync(0xffffffffu, !mine || page >= 0);
            const uint32_t s = kv % kStages;
            ok = __all_sync(0xffffffffu, wait(&bar.kv_empty[s], ((kv / kStages) & 1) ^ 1));
            if (!ok) break;
            // A tile that is looked over when it has landed, on a barrier of its own: values that no
            // row sees are zeroed, since a weight of zero does not hide what lies in the page (keys
            // are hidden by the mask on their scores), rows of a bad page for both, and values that not all
            // rows see where they are no numbers.
            const int here = upto - j * kHalf;
            const bool some = kind == 1 && j * kHalf + min(here, kHalf) - 1 > seen;
            const bool fix = !whole || (kind == 1 && here < kHalf) || some;
            uint64_t* fb = fix ? &bar.tail : &bar.kv_full[s];
            uint8_t* dst = ring + s * kTileBytes;
            if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)__popc(good) * box * kD * 2);
            __syncwarp();
            if (page >= 0) {
              const CUtensorMap* map = kind ? &maps.V : &maps.K;
              const int row = key - b.by_page.quot(key) * b.page_size;
              tma_load_4d(dst + lane * box * 128, map, fb, 0, row, h, page);
              tma_load_4d(dst + kHalfTile + lane * box * 128, map, fb, 64, row, h, page);
            }
            if (fix) {
              ok = __all_sync(0xffffffffu, wait(&bar.tail, tails & 1));
              ++tails;
              if (!ok) break;
              for (int r = (whole ? max(0, here) : 0) + (lane >> 3); r < kHalf; r += 4) {   // eight lanes a row
                if (((good >> (r >> box_log)) & 1) && r < here) continue;
                *reinterpret_cast<uint4*>(dst + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(dst + kHalfTile + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
              if (some) {
                const int from = max(0, seen + 1 - j * kHalf), to = min(kHalf, here);
                if (!finite<T, 2>(dst, kHalfTile, from, to, lane)) {
                  hide<T>(dst, kHalfTile, from, to, lane);
                  *hid = true;
                }
              }
              fence_async_shared();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.kv_full[s]);
            }
        }
      } while (ok && next_of_warp(p, b, g, causal, lane));
      if (!ok) land(bar.kv_full, kv, &bar.tail, tails);
    } else {
      // ---------------------------------------------------------------- queries: a warp a half block
      Piece& p = piece_s[warp];
      const int t = warp - kSoftmaxWarps - 2, c16 = lane & 15, r2 = lane >> 4;
      const int step_t = g.quot(2), step_h = 2 - step_t * g.d;       // from a row to the one two further
      uint32_t pieces = 0;
      bool ok = true;
      do {
        const int R = p.v.n * g.d, r0 = p.m * kBlockRows + t * kHalf;
        if (r0 >= R) continue;
        ok = __all_sync(0xffffffffu, wait(&bar.q_empty[t], (pieces & 1) ^ 1));
        if (!ok) break;
        ++pieces;
        int tok = g.quot(r0 + r2), hd = (r0 + r2) - tok * g.d;
        const T* Q = reinterpret_cast<const T*>(a.Q) + (int64_t)p.v.q0 * a.q_ts + (int64_t)p.h * g.d * a.q_hs + 8 * c16;
        const uint32_t dst = smem_u32(Qs + t * kTileBytes + (c16 >> 3) * kHalfTile);
        const int pairs = (min(kHalf, R - r0) + 1) / 2;   // what lies behind the last row does not matter
#pragma unroll 4
        for (int i = 0; i < pairs; ++i) {
          const int rr = 2 * i + r2;
          const bool in = r0 + rr < R;
          const T* src = in ? Q + (int64_t)tok * a.q_ts + (int64_t)hd * a.q_hs : Q;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + rr * 128 + (((c16 & 7) ^ (rr & 7)) << 4)),
                       "l"(src), "r"(in ? 16u : 0u)
                       : "memory");
          tok += step_t;
          hd += step_h;
          if (hd >= (int)g.d) {
            hd -= g.d;
            ++tok;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_async_shared();
        mbar_arrive(&bar.q_full[t]);
      } while (next_of_warp(p, b, g, causal, lane));
    }
  } else {
    // ------------------------------------------------------------------ softmax: a thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    Piece& p = piece_s[warp];
    const int t = warp >> 2, wq = warp & 3;     // half block, 32 of its rows
    const uint32_t tS = tmem + t * kHalf + ((uint32_t)(32 * wq) << 16), tO = tS + 2 * kHalf;
    const bool neg = a.scale < 0.0f;
    const float scale2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-30f);   // not 0: a masked score times 0 is no number
    uint32_t tiles = 0, outputs[2] = {0, 0}, pieces = 0;
    // A wait that gives up does not end this role: a pair's barriers need both of its warps, and the other
    // waits give up at once then. The result is reported as void.
    do {
      const bool alone = kFew || solo(p, g), began = p.t0 == 0, ends = p.t1 == p.T;
      const int R = p.v.n * g.d, r0 = p.m * kBlockRows + (alone ? 0 : t * kHalf);
      if (tid == 0 && began && !ends)   // the share's last piece
        ws.list[blockIdx.x] = Split{p.s, p.h, p.m, owner_of(range_s[0] + (p.T - p.t1) - 1, range_s[1], range_s[2]), 1,
                                    p.v.q0, min(kBlockRows, R - p.m * kBlockRows)};
      const int t1 = p.t1, every = alone ? 2 : 1, t0 = p.t0 + (alone ? t : 0);   // this half's tiles
      const bool rows = r0 + 32 * wq < R;         // whether the warp has any
      const int r = r0 + 32 * wq + lane;
      const int rc = min(r, R - 1), tok = g.quot(rc);
      const int lim = causal ? p.v.len - p.v.n + tok : p.v.len - 1;
      const int lim_warp = __shfl_sync(0xffffffffu, lim, 0);      // the least of the warp's rows
      float m = -INFINITY, l = 0.0f;
      for (int j = t0; j < t1; j += every) {
        wait(&bar.s_full[t], tiles & 1);
        __syncwarp();
        ++tiles;
        if (!rows) {   // whatever the weights are, no row that is stored comes of them
          if (lane == 0) {
            mbar_arrive(&bar.p_lo[t]);
            mbar_arrive(&bar.p_hi[t]);
          }
          continue;
        }
        tc_fence_after();
        float s[kHalf];
#pragma unroll
        for (int c = 0; c < kHalf / 32; ++c) tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
        tmem_ld_wait();
        if (neg) {
#pragma unroll
          for (int i = 0; i < kHalf; ++i) s[i] = -s[i];
        }
        if (j * kHalf + kHalf - 1 > lim_warp) {
          const int rel = lim - j * kHalf;
#pragma unroll
          for (int i = 0; i < kHalf; ++i) s[i] = i > rel ? -INFINITY : s[i];
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < kHalf - 4; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = max3(mx[k], s[i + 2 * k], s[i + 2 * k + 1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[kHalf - 4 + k]);
        const float mn = max3(m, top_of<T>(max3(mx[0], mx[1], mx[2]), scale2), top_of<T>(mx[3], scale2));
        if (j == t0) {
          m = mn;
        } else if (__any_sync(0xffffffffu, r < R && mn - m > kFollow<T>)) {   // lanes behind the rows hold anything
          const float f = mn == -INFINITY ? 1.0f : ex2(base_of<T>(m) - base_of<T>(mn));
          m = mn;
          l *= f;
          // the scores being complete, so is every earlier product: the output is at rest
#pragma unroll 1
          for (int c = 0; c < kHalf / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tO + 16 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st16(tO + 16 * c, o);
          }
        }
        const float sub = m == -INFINITY ? 0.0f : -base_of<T>(m);
        weights<T, kFew>(s, scale2, sub, l, tS, &bar.p_lo[t], &bar.p_hi[t], lane);
      }
      m = base_of<T>(m);   // what sum and output are relative to
      const int64_t row = (int64_t)(p.v.q0 + tok) * a.Hq + p.h * g.d + (rc - tok * g.d);
      if (a.pre_lse && r < R) {   // what the end needs of the prefix, while the last products are made
        prefetch_l2(a.pre_out + row * kD, kD * 4);
      }
      // the products are in
      const bool used[2] = {true, !alone || p.t1 - p.t0 > 1};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (used[k] && (k == t || alone)) {
          wait(&bar.o_full[k], outputs[k] & 1);
          __syncwarp();
        }
        if (used[k]) ++outputs[k];
      }
      tc_fence_after();
      const bool hid = *(volatile bool*)&hid_s[pieces++ & 7];
      float f0 = 1.0f, f1 = 0.0f;                 // weights of the two halves' outputs
      if (alone) {
        // half 1 tells half 0 its maximum and sum and is done; half 0 reads both outputs
        if (t == 1) told_s[32 * wq + lane] = make_float2(m, l);
        pair_sync(1 + wq);
        if (t == 0) {
          const float m1 = told_s[32 * wq + lane].x, l1 = told_s[32 * wq + lane].y, mn = fmaxf(m, m1);
          f0 = rescale(m, mn);
          f1 = rescale(m1, mn);
          l = l * f0 + l1 * f1;
          m = mn;
        }
        pair_sync(1 + wq);
        if (t == 1) continue;
      }
      const bool both = alone && used[1];
      if (began && ends) {
        float inv = 1.0f, w = 0.0f;
        if (a.pre_lse) {
          const float pl = a.pre_lse[row] * kLog2e, mn = fmaxf(m, pl);
          inv = rescale(m, mn);
          w = pl == -INFINITY ? 0.0f : ex2(pl - mn);   // one that is no number stays so, also without keys
          l = fmaf(l, inv, w);
          m = mn;
        }
        const float il = inverse_sum(l);
        f0 *= inv * il;
        f1 *= inv * il;
        w *= il;
        // Four lanes (four rows) exchange their 16-byte blocks, so that a store writes 64 bytes of a row
        const int64_t out_row = row * kD + 8 * (lane & 3);
        const uint32_t live = __ballot_sync(0xffffffffu, r < R);
#pragma unroll 1
        for (int c = 0; c < kD / 32; ++c) {
          uint32_t y[4][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v[16];
            output16(tO + 32 * c + 16 * h, f0, both, f1, v);
            if (a.pre_lse && w != 0.0f) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 x = reinterpret_cast<const float4*>(a.pre_out + row * kD + 32 * c + 16 * h)[i];
                v[4 * i] = fmaf(w, x.x, v[4 * i]);
                v[4 * i + 1] = fmaf(w, x.y, v[4 * i + 1]);
                v[4 * i + 2] = fmaf(w, x.z, v[4 * i + 2]);
                v[4 * i + 3] = fmaf(w, x.w, v[4 * i + 3]);
              }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) y[2 * h + (i >> 2)][i & 3] = pack2(T(), v[2 * i], v[2 * i + 1]);
          }
          transpose4(y, lane);   // y[k]: block (lane & 3) of the row of lane (lane & ~3) + k
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int from = (lane & ~3) + k;
            const int64_t at = __shfl_sync(0xffffffffu, out_row, from) + 32 * c + 8 * ((lane & 3) - k);
            if ((live >> from) & 1)
              *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + at) = make_uint4(y[k][0], y[k][1], y[k][2], y[k][3]);
          }
        }
        if (a.lse && r < R) a.lse[row] = log_sum(m, l);
        if (hid) {
          __syncwarp();   // other lanes stored the row
          if (r < R) show_values<T>(a, p, lim, reinterpret_cast<T*>(a.out) + row * kD, nullptr);
        }
      } else {
        // parts: blocks of four features, rows next to one another
        const int64_t slot = (int64_t)blockIdx.x * 2 + (began ? 1 : 0);
        const int row_in = r - p.m * kBlockRows;
        float4* dst = reinterpret_cast<float4*>(ws.o) + slot * 32 * kBlockRows + row_in;
#pragma unroll 1
        for (int c = 0; c < kD / 16; ++c) {
          float v[16];
          output16(tO + 16 * c, f0, both, f1, v);
          if (r < R) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[(4 * c + i) * kBlockRows] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        if (r < R) ws.ml[slot * kBlockRows + row_in] = make_float2(m, l);
        if (hid && r < R) show_values<T>(a, p, lim, nullptr, reinterpret_cast<float*>(dst));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar.o_empty[t]);
        if (both) mbar_arrive(&bar.o_empty[1]);   // for half 1, which went on
      }
    } while (next_of_warp(p, b, g, causal, lane));
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSoftmaxWarps) tmem_dealloc(tmem, 512);
}

template <typename T, bool kFew>
cudaError_t launch(const PagedAttnArgs& a, const AttnPlan& p, const Workspace& w, cudaStream_t s) {
  int box = kHalf;
  while (a.b.page_size % box) box /= 2;      // 16 at least
  Maps maps;
  maps.K = a.maps[0];
  maps.V = a.maps[1];
  static SmemFlags allowed;
  cudaError_t e = allow_smem(k_attn_chunk<T, kFew>, kSmem, a.device, allowed);
  if (e != cudaSuccess) return e;
  return launch_early(k_attn_chunk<T, kFew>, dim3(p.grid), dim3(kThreads), kSmem, 1, s, a, maps, w, box);
}

}  // namespace

cudaError_t attn_chunk(const PagedAttnArgs& a, const AttnPlan& p, const pattn::Workspace& w, cudaStream_t s) {
  const bool b = a.dtype == JOLT_BF16;
  if (p.most <= kHalf) return b ? launch<__nv_bfloat16, true>(a, p, w, s) : launch<__half, true>(a, p, w, s);
  return b ? launch<__nv_bfloat16, false>(a, p, w, s) : launch<__half, false>(a, p, w, s);
}

}  // namespace jolt
