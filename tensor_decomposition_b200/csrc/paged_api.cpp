// Host side of the growing cache (include/jolt.h): page sets, argument checks and launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <new>
#include <vector>

#include "paged.h"
#include "kernels/gemm_tc.h"

using namespace jolt;

struct jolt_pages_s {
  jolt_page_shape shape{};
  void *K = nullptr, *V = nullptr;
  int device = 0;
  int32_t* d_status = nullptr;
  CUtensorMap maps[4];   // K and V in boxes of gcd(page_size, 128) rows x 64 features, K and V of 16 rows
};

namespace {

// Status words of page sets: slabs of them per device, allocated once and handed out again, so that
// creating and destroying a set allocates and frees nothing (a destructor may run while another
// thread captures a graph, where freeing is an error).
constexpr int kSlab = 1024;
constexpr int kDevices = 64;
std::mutex g_slot_mu;
std::vector<int32_t*> g_free_slots[kDevices];

cudaError_t take_slot(int dev, int32_t** out) {
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> g(g_slot_mu);
  auto& fr = g_free_slots[dev];
  if (fr.empty()) {
    void* p = nullptr;
    const cudaError_t e = host_dev_malloc(&p, kSlab * sizeof(int32_t));
    if (e != cudaSuccess) return e;
    try {
      fr.reserve(fr.capacity() + kSlab);   // also what giving slots back needs
    } catch (...) {
      cudaFree(p);
      return cudaErrorMemoryAllocation;
    }
    for (int i = kSlab - 1; i >= 0; --i) fr.push_back(static_cast<int32_t*>(p) + i);
  }
  *out = fr.back();
  fr.pop_back();
  return cudaSuccess;
}
void give_slot(int dev, int32_t* p) {
  std::lock_guard<std::mutex> g(g_slot_mu);
  g_free_slots[dev].push_back(p);
}

cudaError_t sm_count(int dev, int* out) {
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  static std::atomic<int> n[kDevices];
  int v = n[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    const cudaError_t e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    n[dev].store(v, std::memory_order_relaxed);
  }
  *out = v;
  return cudaSuccess;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct ProfScope {
  ProfScope(const char* name, cudaStream_t s) : token(host_prof_begin(name, s)) {}
  ~ProfScope() {
    if (token) host_prof_end(token);
  }
  void* token;
};

jolt_status cuda_fail(const char* what, cudaError_t e) {
  return host_fail(e == cudaErrorMemoryAllocation ? JOLT_ERR_OOM : JOLT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Strides of a rows tensor: rows of 128 contiguous elements on 16-byte boundaries.
jolt_status check_rows(const char* what, const char* name, const void* p, int64_t ts, int64_t hs, int32_t heads) {
  if (heads <= 0) return host_fail(JOLT_ERR_INVALID_ARG, "%s: %s has no heads", what, name);
  if (!p) return host_fail(JOLT_ERR_INVALID_ARG, "%s: null %s", what, name);
  if (!aligned16(p) || ts % 8 || hs % 8)
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: %s rows must start on 16-byte boundaries (strides a multiple of 8)", what,
                     name);
  if (ts > INT32_MAX || ts < -INT32_MAX || hs > INT32_MAX || hs < -INT32_MAX)
    return host_fail(JOLT_ERR_UNSUPPORTED, "%s: strides of %s beyond 2^31 elements", what, name);
  return JOLT_OK;
}

// Whether rows of an output lie over one another, of 128 elements at ts t + hs h. Mostly one dimension lies within
// the other's stride; else each distance of heads is held against the nearest of tokens.
bool rows_overlap(int64_t ts, int64_t hs, int64_t tokens, int64_t heads) {
  ts = std::abs(ts);
  hs = std::abs(hs);
  if ((tokens > 1 && ts < kD) || (heads > 1 && hs < kD)) return true;
  if (tokens == 1 || heads == 1 || ts >= hs * (heads - 1) + kD || hs >= ts * (tokens - 1) + kD) return false;
  for (int64_t h = 1; h < heads; ++h) {
    const int64_t t = h * hs / ts, left = h * hs - t * ts;   // signs of the strides: the rows' set is the same mirrored
    if ((t < tokens && left < kD) || (t + 1 < tokens && ts - left < kD)) return true;
  }
  return false;
}

jolt_status check_rope(const char* what, const int32_t* positions, bool positions_needed, const float* inv_freq,
                       int32_t rope_dim) {
  if (!inv_freq) return JOLT_OK;
  if (positions_needed && !positions) return host_fail(JOLT_ERR_INVALID_ARG, "%s: inv_freq without positions", what);
  if (rope_dim <= 0 || rope_dim > kD || rope_dim % 16)
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: rope_dim %d is not a multiple of 16 in [16, %d]", what, rope_dim, kD);
  return JOLT_OK;
}

RowsIn rows_in(const void* p, int64_t ts, int64_t hs, int heads, const void* w) {
  RowsIn r;
  r.p = p;
  r.ts = (int32_t)ts;   // checked by check_rows
  r.hs = (int32_t)hs;
  r.heads = heads;
  r.w = w;
  return r;
}
RowsOut rows_out(void* p, int64_t ts, int64_t hs) {
  RowsOut r;
  r.p = p;
  r.ts = (int32_t)ts;
  r.hs = (int32_t)hs;
  return r;
}

jolt_status check_batch(const char* what, const jolt_pages_s* pg, const jolt_batch* b, const void* args) {
  if (!pg || !b || !args) return host_fail(JOLT_ERR_INVALID_ARG, "%s: null pages, batch or arguments", what);
  if (b->num_seqs < 0 || b->total_q < 0 || b->max_q < 0 || b->max_pages < 0)
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: negative batch size", what);
  if (b->num_seqs > 0 && (!b->q_start || !b->kv_len || (b->max_pages > 0 && !b->page_table)))
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: null q_start, kv_len or page_table", what);
  if ((int64_t)b->max_pages * pg->shape.page_size > INT32_MAX - 1024)
    return host_fail(JOLT_ERR_UNSUPPORTED, "%s: page tables of more than 2^31 tokens", what);
  if ((int64_t)b->num_seqs * pg->shape.heads > INT32_MAX)
    return host_fail(JOLT_ERR_UNSUPPORTED, "%s: more than 2^31 sequences times heads", what);
  return JOLT_OK;
}

jolt_status check_device(const char* what, const jolt_pages_s* pg) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(what, e);
  if (dev != pg->device)
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: the page set is on device %d, the current device is %d", what, pg->device,
                     dev);
  return JOLT_OK;
}

BatchView view_of(const jolt_pages_s* pg, const jolt_batch* b) {
  BatchView v{};
  v.num_seqs = b->num_seqs;
  v.total_q = b->total_q;
  v.max_q = b->max_q;
  v.max_pages = b->max_pages;
  v.q_start = b->q_start;
  v.kv_len = b->kv_len;
  v.page_table = b->page_table;
  v.num_pages = pg->shape.num_pages;
  v.heads = pg->shape.heads;
  v.page_size = pg->shape.page_size;
  v.by_page = divisor(v.page_size);
  v.status = pg->d_status;
  return v;
}

RopeArgs rope_of(float eps, const int32_t* positions, const float* inv_freq, int32_t rope_dim, int32_t interleaved) {
  RopeArgs r;
  r.positions = positions;
  r.inv_freq = inv_freq;
  r.rope_dim = inv_freq ? rope_dim : 0;
  r.interleaved = interleaved != 0;
  r.eps = eps;
  return r;
}

}  // namespace

extern "C" {

JOLT_API jolt_status jolt_pages_create(const jolt_page_shape* shape, void* K_pages, void* V_pages, void* cuda_stream,
                                       jolt_pages_t* out) {
  host_clear_error();
  if (!shape || !out) return host_fail(JOLT_ERR_INVALID_ARG, "jolt_pages_create: null shape or out");
  *out = nullptr;
  const jolt_page_shape& sh = *shape;
  if (sh.num_pages <= 0 || sh.heads <= 0 || sh.page_size <= 0)
    return host_fail(JOLT_ERR_INVALID_ARG, "jolt_pages_create: non-positive dimension");
  if (sh.head_dim != kD)
    return host_fail(JOLT_ERR_INVALID_ARG, "jolt_pages_create: head_dim %d unsupported (supported: 128)", sh.head_dim);
  if (sh.dtype != JOLT_BF16 && sh.dtype != JOLT_F16)
    return host_fail(JOLT_ERR_UNSUPPORTED, "jolt_pages_create: pages are bf16 or f16");
  if (sh.page_size % 16 || sh.page_size >= (1 << 24))   // a head's stride fits 32 bits
    return host_fail(JOLT_ERR_UNSUPPORTED, "jolt_pages_create: page_size %d is not a multiple of 16 below 2^24",
                     sh.page_size);
  if ((int64_t)sh.heads * sh.page_size * (2 * kD) >= (1ll << 40))
    return host_fail(JOLT_ERR_UNSUPPORTED, "jolt_pages_create: a page of 2^40 bytes or more");
  if (!K_pages || !V_pages) return host_fail(JOLT_ERR_INVALID_ARG, "jolt_pages_create: null pages");
  if (!aligned16(K_pages) || !aligned16(V_pages))
    return host_fail(JOLT_ERR_INVALID_ARG, "jolt_pages_create: pages must be 16-byte aligned");
  jolt_pages_s* p = new (std::nothrow) jolt_pages_s();
  if (!p) return host_fail(JOLT_ERR_OOM, "jolt_pages_create: host allocation");
  p->shape = sh;
  p->K = K_pages;
  p->V = V_pages;
  const uint64_t row = 2 * kD, P = (uint64_t)sh.page_size;
  const uint64_t dims[4] = {kD, P, (uint64_t)sh.heads, (uint64_t)sh.num_pages};
  const uint64_t strides[3] = {row, row * P, row * P * sh.heads};
  uint32_t box = 128;
  while (P % box) box /= 2;
  bool ok = true;
  for (int i = 0; i < 4; ++i)
    ok = ok && tc_map_bf16_box(&p->maps[i], i & 1 ? V_pages : K_pages, 4, dims, strides, i < 2 ? box : 16);
  if (!ok) {
    delete p;
    return host_fail(JOLT_ERR_CUDA, "jolt_pages_create: tensor map rejected");
  }
  cudaError_t e = cudaGetDevice(&p->device);
  if (e == cudaSuccess) e = host_pool_ready();
  if (e == cudaSuccess) e = take_slot(p->device, &p->d_status);
  if (e == cudaSuccess) e = cudaMemsetAsync(p->d_status, 0, sizeof(int32_t), (cudaStream_t)cuda_stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)cuda_stream);   // the set is used on any stream
  if (e != cudaSuccess) {
    if (p->d_status) give_slot(p->device, p->d_status);
    delete p;
    return cuda_fail("jolt_pages_create", e);
  }
  *out = p;
  return JOLT_OK;
}

JOLT_API void jolt_pages_destroy(jolt_pages_t p) {
  if (!p) return;
  give_slot(p->device, p->d_status);
  delete p;
}

JOLT_API jolt_status jolt_pages_status(jolt_pages_t p, void* cuda_stream) {
  host_clear_error();
  if (!p) return host_fail(JOLT_ERR_INVALID_ARG, "jolt_pages_status: null pages");
  if (jolt_status st = check_device("jolt_pages_status", p)) return st;
  cudaStream_t s = (cudaStream_t)cuda_stream;
  int32_t w = 0;
  void* got = nullptr;
  cudaError_t e = host_pool_malloc(&got, sizeof(w), s);
  if (e == cudaSuccess) {   // read and cleared in one: kernels on other streams may be reporting
    e = take_status(p->d_status, static_cast<int32_t*>(got), s);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&w, got, sizeof(w), cudaMemcpyDeviceToHost, s);
    const cudaError_t e2 = cudaFreeAsync(got, s);
    if (e == cudaSuccess) e = e2;
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail("jolt_pages_status", e);
  if (w) {
    const char* found[3] = {w & PST_TIMEOUT ? "a bounded device wait of paged attention gave up; " : "",
                            w & PST_BAD_BATCH ? "a sequence's q_start or kv_len does not fit its batch (the sequence was skipped); " : "",
                            w & PST_BAD_PAGE ? "a page table names a page outside the set (it was not followed); " : ""};
    char all[256];
    const int n = snprintf(all, sizeof(all), "%s%s%s", found[0], found[1], found[2]);
    all[n - 2] = 0;   // the last separator
    return host_fail(w & PST_TIMEOUT ? JOLT_ERR_TIMEOUT : JOLT_ERR_INVALID_ARG, "%s", all);
  }
  return JOLT_OK;
}

JOLT_API jolt_status jolt_qk_norm_rope(const jolt_norm_rope* args, void* cuda_stream) {
  const char* what = "jolt_qk_norm_rope";
  host_clear_error();
  if (!args) return host_fail(JOLT_ERR_INVALID_ARG, "%s: null arguments", what);
  const jolt_norm_rope& n = *args;
  if (n.dtype != JOLT_BF16 && n.dtype != JOLT_F16) return host_fail(JOLT_ERR_UNSUPPORTED, "%s: rows are bf16 or f16", what);
  if (n.tokens < 0 || n.k_heads < 0) return host_fail(JOLT_ERR_INVALID_ARG, "%s: negative size", what);
  if (n.tokens == 0) return JOLT_OK;
  jolt_status st = check_rows(what, "Q", n.Q, n.q_token_stride, n.q_head_stride, n.q_heads);
  if (st == JOLT_OK) st = check_rows(what, "Q_out", n.Q_out, n.qo_token_stride, n.qo_head_stride, n.q_heads);
  if (st == JOLT_OK && n.k_heads > 0) st = check_rows(what, "K", n.K, n.k_token_stride, n.k_head_stride, n.k_heads);
  if (st == JOLT_OK && n.k_heads > 0) st = check_rows(what, "K_out", n.K_out, n.ko_token_stride, n.ko_head_stride, n.k_heads);
  if (st == JOLT_OK) st = check_rope(what, n.positions, true, n.inv_freq, n.rope_dim);
  if (st != JOLT_OK) return st;
  if (((int64_t)n.q_heads + n.k_heads) * n.tokens > INT32_MAX)
    return host_fail(JOLT_ERR_UNSUPPORTED, "%s: more than 2^31 rows", what);
  if (rows_overlap(n.qo_token_stride, n.qo_head_stride, n.tokens, n.q_heads) ||
      (n.k_heads > 0 && rows_overlap(n.ko_token_stride, n.ko_head_stride, n.tokens, n.k_heads)))
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: rows of an output overlap", what);
  if (!aligned16(n.q_weight) || !aligned16(n.k_weight))
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: weights must be 16-byte aligned", what);
  RowsIn q = rows_in(n.Q, n.q_token_stride, n.q_head_stride, n.q_heads, n.q_weight), k;
  RowsOut qo = rows_out(n.Q_out, n.qo_token_stride, n.qo_head_stride), ko;
  if (n.k_heads > 0) {
    k = rows_in(n.K, n.k_token_stride, n.k_head_stride, n.k_heads, n.k_weight);
    ko = rows_out(n.K_out, n.ko_token_stride, n.ko_head_stride);
  }
  cudaStream_t s = (cudaStream_t)cuda_stream;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = sm_count(dev, &sms);
  if (e != cudaSuccess) return cuda_fail(what, e);
  ProfScope prof("qk_norm_rope", s);
  e = norm_rope(n.dtype, n.tokens, q, qo, k, ko, rope_of(n.eps, n.positions, n.inv_freq, n.rope_dim, n.interleaved), sms, s);
  return e == cudaSuccess ? JOLT_OK : cuda_fail(what, e);
}

JOLT_API jolt_status jolt_paged_append(jolt_pages_t pages, const jolt_batch* batch, const jolt_new_rows* rows,
                                       void* cuda_stream) {
  const char* what = "jolt_paged_append";
  host_clear_error();
  jolt_status st = check_batch(what, pages, batch, rows);
  if (st != JOLT_OK) return st;
  const jolt_new_rows& r = *rows;
  const int H = pages->shape.heads;
  if (batch->total_q == 0 || batch->num_seqs == 0) return JOLT_OK;
  st = check_rows(what, "K", r.K, r.k_token_stride, r.k_head_stride, H);
  if (st == JOLT_OK) st = check_rows(what, "V", r.V, r.v_token_stride, r.v_head_stride, H);
  if (st == JOLT_OK) st = check_rope(what, r.positions, false, r.inv_freq, r.rope_dim);
  if (st != JOLT_OK) return st;
  if (2 * (int64_t)H * batch->total_q > INT32_MAX) return host_fail(JOLT_ERR_UNSUPPORTED, "%s: more than 2^31 rows", what);
  if (!aligned16(r.k_weight)) return host_fail(JOLT_ERR_INVALID_ARG, "%s: the weight must be 16-byte aligned", what);
  st = check_device(what, pages);
  if (st != JOLT_OK) return st;
  cudaStream_t s = (cudaStream_t)cuda_stream;
  int sms = 0;
  cudaError_t e = sm_count(pages->device, &sms);
  if (e != cudaSuccess) return cuda_fail(what, e);
  ProfScope prof("paged_append", s);
  e = paged_append(pages->shape.dtype, view_of(pages, batch), rows_in(r.K, r.k_token_stride, r.k_head_stride, H, r.k_weight),
                   rows_in(r.V, r.v_token_stride, r.v_head_stride, H, nullptr), pages->K, pages->V,
                   rope_of(r.eps, r.positions, r.inv_freq, r.rope_dim, r.interleaved), sms, s);
  return e == cudaSuccess ? JOLT_OK : cuda_fail(what, e);
}

JOLT_API jolt_status jolt_paged_attention(jolt_pages_t pages, const jolt_batch* batch, const jolt_queries* queries,
                                          void* cuda_stream) {
  const char* what = "jolt_paged_attention";
  host_clear_error();
  jolt_status st = check_batch(what, pages, batch, queries);
  if (st != JOLT_OK) return st;
  const jolt_queries& q = *queries;
  if (q.q_heads <= 0 || q.q_heads % pages->shape.heads)
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: q_heads must be a positive multiple of the %d KV heads", what,
                     pages->shape.heads);
  if ((int64_t)batch->total_q * q.q_heads > INT32_MAX - 1024)
    return host_fail(JOLT_ERR_UNSUPPORTED, "%s: more than 2^31 query rows", what);
  if (!std::isfinite(q.scale)) return host_fail(JOLT_ERR_INVALID_ARG, "%s: the scale is no finite number", what);
  if (!q.prefix_out != !q.prefix_lse)
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: prefix_out and prefix_lse come together", what);
  if (batch->total_q == 0 || batch->num_seqs == 0) return JOLT_OK;
  st = check_rows(what, "Q", q.Q, q.q_token_stride, q.q_head_stride, q.q_heads);
  if (st != JOLT_OK) return st;
  if (!q.out) return host_fail(JOLT_ERR_INVALID_ARG, "%s: null out", what);
  if (!aligned16(q.out) || !aligned16(q.prefix_out))
    return host_fail(JOLT_ERR_INVALID_ARG, "%s: out and prefix_out must be 16-byte aligned", what);
  // a KV head's blocks of rows times tiles of keys are counted in 32 bits
  const int64_t tokens = (int64_t)batch->max_pages * pages->shape.page_size;
  const int64_t rows = (int64_t)std::min(batch->max_q, batch->total_q) * (q.q_heads / pages->shape.heads);
  if ((rows / 256 + 1) * (tokens / 128 + 4) > INT32_MAX)
    return host_fail(JOLT_ERR_UNSUPPORTED, "%s: chunks of %d tokens over page tables of %lld tokens", what,
                     (int)std::min(batch->max_q, batch->total_q), (long long)tokens);
  st = check_device(what, pages);
  if (st != JOLT_OK) return st;
  PagedAttnArgs a{};
  a.b = view_of(pages, batch);
  a.dtype = pages->shape.dtype;
  a.device = pages->device;
  a.maps = pages->maps;
  a.V = pages->V;
  a.Q = q.Q; a.q_ts = q.q_token_stride; a.q_hs = q.q_head_stride; a.Hq = q.q_heads;
  a.g = divisor(q.q_heads / pages->shape.heads);
  a.scale = q.scale; a.causal = q.causal != 0;
  a.pre_out = q.prefix_out; a.pre_lse = q.prefix_lse;
  a.out = q.out; a.lse = q.lse;
  cudaStream_t s = (cudaStream_t)cuda_stream;
  ProfScope prof("paged_attention", s);
  int sms = 0;
  cudaError_t e = sm_count(pages->device, &sms);
  if (e != cudaSuccess) return cuda_fail(what, e);
  const AttnPlan p = paged_attention_plan(a, sms);
  void* scratch = nullptr;
  if (p.bytes) e = host_pool_malloc(&scratch, p.bytes, s);
  if (e == cudaSuccess) {
    e = paged_attention(a, p, scratch, s);
    const cudaError_t e2 = scratch ? cudaFreeAsync(scratch, s) : cudaSuccess;
    if (e == cudaSuccess) e = e2;
  }
  return e == cudaSuccess ? JOLT_OK : cuda_fail(what, e);
}

}  // extern "C"
