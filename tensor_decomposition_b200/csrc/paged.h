// Internal declarations of the growing cache: the norm and rotation of query and key rows, the
// append to a paged cache and the attention of new tokens over it. Host side in paged_api.cpp,
// kernels in kernels/rope_rows.cu and kernels/paged_attention*.cu. Not part of the public C ABI.
#pragma once

#include <cuda.h>

#include <atomic>
#include <utility>

#include "jolt_internal.h"

namespace jolt {

// Bits of a page set's status word (OR-ed by kernels, read and cleared by jolt_pages_status).
enum : int32_t { PST_BAD_BATCH = 1, PST_BAD_PAGE = 2, PST_TIMEOUT = 4 };

// A divisor d that the host knows: the quotient of 0 <= n < 2^31 is floor(n m / 2^(31 + s)) with s = ceil(log2 d)
// and m = ceil(2^(31 + s) / d) < 2^32, which is n / d and less than 1 / d too much (Granlund and Montgomery's
// division by an invariant). The kernels divide on their way to the first copy, where a division costs 0.1 us.
struct Divisor {
  uint32_t d = 1, m = 1u << 31, s = 0;
#ifdef __CUDACC__
  __device__ __forceinline__ int quot(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> (31 + s)); }
#endif
};
inline Divisor divisor(uint32_t d) {
  Divisor r;
  r.d = d;
  while ((1u << r.s) < d && r.s < 31) ++r.s;
  r.m = (uint32_t)(((1ull << (31 + r.s)) + d - 1) / d);
  return r;
}

// One batch of sequences (device arrays; see jolt_batch in jolt.h) over one page set.
struct BatchView {
  int32_t num_seqs, total_q, max_q, max_pages;
  const int32_t* q_start;      // [num_seqs + 1]
  const int32_t* kv_len;       // [num_seqs]
  const int32_t* page_table;   // [num_seqs][max_pages]
  int32_t num_pages, heads, page_size;
  Divisor by_page;             // page_size
  int32_t* status;
};

// Tokens q0 .. q0 + n - 1 of the batch belong to the sequence, whose cache holds len tokens, the
// chunk's among them. n = 0 where there is nothing to do.
struct SeqView {
  int32_t q0, n, len;
};

// Sequence s with its bounds checked: one whose bounds do not fit the batch (offsets outside
// [0, total_q] or falling, more than max_q tokens, a length outside [0, max_pages * page_size])
// is flagged and gets n = 0, so that no kernel addresses anything by it.
__device__ __forceinline__ SeqView seq_view(const BatchView& b, int s) {
  const int q0 = b.q_start[s], q1 = b.q_start[s + 1], len = b.kv_len[s];
  SeqView v{q0, q1 - q0, len};
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= b.total_q && q1 - q0 <= b.max_q && len >= 0 &&
                  len <= (int64_t)b.max_pages * b.page_size;
  if (!ok) {
    atomicOr(b.status, PST_BAD_BATCH);
    v = SeqView{0, 0, 0};
  }
  return v;
}

// Page that holds token `pos` (0 <= pos < len) of sequence s, or -1 (flagged) when the table's
// entry is no page of the set.
__device__ __forceinline__ int page_of(const BatchView& b, int s, int pos) {
  const int p = b.page_table[(int64_t)s * b.max_pages + b.by_page.quot(pos)];
  if (p < 0 || p >= b.num_pages) {
    atomicOr(b.status, PST_BAD_PAGE);
    return -1;
  }
  return p;
}

// *out = *word; *word = 0, in one step.
cudaError_t take_status(int32_t* word, int32_t* out, cudaStream_t s);

// Allow a kernel its dynamic shared memory, once a device (`done`: the kernel's own flags).
struct SmemFlags {
  std::atomic<bool> on[64] = {};
};
template <class K>
inline cudaError_t allow_smem(K* kernel, int bytes, int device, SmemFlags& done) {
  if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
  if (done.on[device].load(std::memory_order_acquire)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.on[device].store(true, std::memory_order_release);
  return e;
}

// Launches that may be placed before the kernel ahead of them in the stream has ended, where that one allows
// it: the kernel itself waits for it (grid_wait) before it touches memory, and lets the one behind it be
// placed (grid_release) at its start. What goes before the wait, and the launch, overlaps.
template <class... P, class... A>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t s,
                                A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
  if (e != cudaSuccess) return e;
  note_launch();
  return cudaGetLastError();
}
#ifdef __CUDACC__
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

// Rows of 128 elements of a tensor [tokens][heads][128]; element strides.
struct RowsIn {
  const void* p = nullptr;
  int32_t ts = 0, hs = 0;
  int32_t heads = 0;
  const void* w = nullptr;     // norm weight [128], or null
};
struct RowsOut {
  void* p = nullptr;
  int32_t ts = 0, hs = 0;
};
struct RopeArgs {
  const int32_t* positions = nullptr;   // [tokens], or null (paged: the token's index in its cache)
  const float* inv_freq = nullptr;      // [rope_dim / 2], or null: no rotation
  int32_t rope_dim = 0, interleaved = 0;
  float eps = 0.0f;
};
// Queries (and keys) normed and rotated, out of place or in place.
cudaError_t norm_rope(jolt_dtype t, int tokens, const RowsIn& Q, const RowsOut& Qo, const RowsIn& K,
                      const RowsOut& Ko, const RopeArgs& r, int sms, cudaStream_t s);
// Keys (normed and rotated) and values written to the pages.
cudaError_t paged_append(jolt_dtype t, const BatchView& b, const RowsIn& K, const RowsIn& V, void* K_pages,
                         void* V_pages, const RopeArgs& r, int sms, cudaStream_t s);

struct PagedAttnArgs {
  BatchView b;
  jolt_dtype dtype;
  int32_t device;
  const CUtensorMap* maps;     // host: K and V with boxes of gcd(page_size, 128) rows, K and V with 16 rows
  const void* V;               // the value pages
  const void* Q;
  int64_t q_ts, q_hs;          // element strides of Q
  int32_t Hq;
  Divisor g;                   // query heads a KV head
  float scale;
  int32_t causal;
  const float *pre_out, *pre_lse;   // [total_q][Hq][128], [total_q][Hq], or null
  void* out;                        // [total_q][Hq][128] of dtype
  float* lse;                       // [total_q][Hq], or null
};
// How a call is run: which kernel, its CTAs, the rows of an item's block and the scratch it needs.
struct AttnPlan {
  int32_t decode = 0, team = 0, grid = 0, rows = 0, most = 0;   // most: rows an item can have
  size_t bytes = 0;
};
AttnPlan paged_attention_plan(const PagedAttnArgs& a, int sms);
cudaError_t paged_attention(const PagedAttnArgs& a, const AttnPlan& p, void* scratch, cudaStream_t s);

// Host services of jolt_api.cpp.
jolt_status host_fail(jolt_status st, const char* fmt, ...);
void host_clear_error();
cudaError_t host_pool_malloc(void** ptr, size_t bytes, cudaStream_t s);
cudaError_t host_dev_malloc(void** ptr, size_t bytes);
cudaError_t host_pool_ready();   // makes the current device's pool, so that captured calls find it
// Tracing of one phase on a stream: begin returns a token for end (null when tracing is off).
void* host_prof_begin(const char* name, cudaStream_t s);
void host_prof_end(void* token);

}  // namespace jolt
