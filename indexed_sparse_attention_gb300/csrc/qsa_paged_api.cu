// Host side of the entry points over paged K/V caches (include/qsa.h): argument
// checks, the choice of kernel, and the launches.  Nothing here allocates
// device memory or waits for the GPU.
#include <math.h>

#include <algorithm>

#include "qsa_host.cuh"
#include "qsa_paged.cuh"

using namespace qsa;

namespace {

int log2_of(int64_t x) {
  int s = 0;
  while (((int64_t)1 << s) < x) ++s;
  return s;
}

// A cache's shape and addresses for head_dim and dtype of cfg.
qsa_status check_cache(const qsa_paged_cache* c, const qsa_attn_config* cfg, const char* fn) {
  if (!c) return fail(QSA_ERR_INVALID_ARG, "%s: null cache", fn);
  if (cfg->n_kv_heads >= 1 << 16) return fail(QSA_ERR_UNSUPPORTED, "%s: %d KV heads", fn, cfg->n_kv_heads);
  if (!c->k || !c->v) return fail(QSA_ERR_INVALID_ARG, "%s: cache has a null K/V", fn);
  if (cfg->kv_dtype == QSA_Q8_0) return fail(QSA_ERR_UNSUPPORTED, "%s: Q8_0 caches are not paged", fn);
  if (c->n_pages < 1) return fail(QSA_ERR_INVALID_ARG, "%s: n_pages=%d", fn, c->n_pages);
  if (c->page_tokens < QSA_MIN_PAGE_TOKENS || c->page_tokens > QSA_MAX_PAGE_TOKENS ||
      (c->page_tokens & (c->page_tokens - 1)) != 0)
    return fail(QSA_ERR_UNSUPPORTED, "%s: page_tokens=%d (a power of two in %d..%d)", fn, c->page_tokens,
                QSA_MIN_PAGE_TOKENS, QSA_MAX_PAGE_TOKENS);
  const int64_t es = (int64_t)dtype_size(cfg->kv_dtype), most = (int64_t)1 << 38;   // a tensor map holds strides below 2^40 bytes
  if (c->tok_stride < cfg->head_dim || c->head_stride < cfg->head_dim || c->page_stride < cfg->head_dim ||
      c->tok_stride > most || c->head_stride > most || c->page_stride > most)
    return fail(QSA_ERR_INVALID_ARG, "%s: cache strides page=%lld head=%lld tok=%lld (each >= head_dim=%d)", fn,
                (long long)c->page_stride, (long long)c->head_stride, (long long)c->tok_stride, cfg->head_dim);
  if (!aligned16(c->k) || !aligned16(c->v) || (c->tok_stride * es) % 16 || (c->head_stride * es) % 16 ||
      (c->page_stride * es) % 16)
    return fail(QSA_ERR_MISALIGNED, "%s: cache K/V or strides not 16-byte aligned", fn);
  if (cfg->kv_dtype == QSA_FP8_E4M3) {
    if (!c->kv_scale) return fail(QSA_ERR_INVALID_ARG, "%s: fp8 cache has no scales", fn);
    if (reinterpret_cast<uintptr_t>(c->kv_scale) & 3u)
      return fail(QSA_ERR_MISALIGNED, "%s: scale records not 4-byte aligned", fn);
    if (c->scale_page_stride < 1 || c->scale_head_stride < 1 || c->scale_tok_stride < 1)
      return fail(QSA_ERR_INVALID_ARG, "%s: bad scale strides", fn);
  }
  return QSA_OK;
}

qsa_status check_batch(const qsa_paged_batch* b, const char* fn) {
  if (!b) return fail(QSA_ERR_INVALID_ARG, "%s: null batch", fn);
  if (b->n_seqs < 0 || b->n_rows < 0 || b->max_rows < 0)
    return fail(QSA_ERR_INVALID_ARG, "%s: n_seqs=%d, n_rows=%d, max_rows=%d", fn, b->n_seqs, b->n_rows, b->max_rows);
  if (b->n_rows > (1 << 24) - 256) return fail(QSA_ERR_UNSUPPORTED, "%s: too many rows", fn);   // entries below 2^28
  if (b->n_seqs == 0 || b->n_rows == 0) return QSA_OK;
  if (!b->table || !b->lens || !b->row_start) return fail(QSA_ERR_INVALID_ARG, "%s: batch has a null array", fn);
  if (b->table_ld < 1) return fail(QSA_ERR_INVALID_ARG, "%s: table_ld=%lld", fn, (long long)b->table_ld);
  return QSA_OK;
}

// Kernel of a call and how it divides the work.
struct Plan {
  bool tensor_cores;
  int mt;     // entries of an item
  int grid;   // runs
};

Plan plan_attn(const qsa_paged_batch* b, const qsa_attn_config* cfg) {
  Plan pl;
  pl.tensor_cores = cfg->kv_dtype != QSA_F32;
  if (pl.tensor_cores) {
    // Whole rows, as many as a sequence has, up to the 128 entries that are the
    // MMA's rows: what Q does not take of the shared memory is the ring's.
    const int group = cfg->n_q_heads / cfg->n_kv_heads;
    pl.mt = group * std::max(1, std::min(b->max_rows, 128 / group));
  } else {
    pl.mt = (int64_t)b->max_rows * (cfg->n_q_heads / cfg->n_kv_heads) <= 16 ? 16 : 32;
  }
  pl.grid = device_sm_count();   // a CTA takes an SM's shared memory or registers
  if (cfg->n_splits > 0) pl.grid = std::min(pl.grid, cfg->n_splits);
  return pl;
}

size_t up256(size_t b) { return (b + 255) / 256 * 256; }

// Workspace: the crossing items, then the parts' lse values, then their outputs.
size_t lse_offset(const Plan& pl) { return up256(sizeof(PagedPart) * (size_t)pl.grid); }
size_t out_offset(const Plan& pl) { return lse_offset(pl) + up256(sizeof(float) * 2 * (size_t)pl.grid * (size_t)pl.mt); }
size_t workspace_bytes_of(const Plan& pl, int head_dim) {
  return out_offset(pl) + sizeof(float) * 2 * (size_t)pl.grid * (size_t)pl.mt * (size_t)head_dim;
}

qsa_status check_config(const qsa_attn_config* cfg, const char* fn) {
  const qsa_status s = check_attn_config(cfg, fn);
  if (s != QSA_OK) return s;
  if (cfg->n_splits < 0) return fail(QSA_ERR_INVALID_ARG, "%s: n_splits=%d", fn, cfg->n_splits);
  return QSA_OK;
}

}  // namespace

QSA_API size_t qsa_paged_attn_workspace_size(const qsa_paged_batch* batch, const qsa_attn_config* cfg) {
  const char* fn = "qsa_paged_attn_workspace_size";
  if (check_config(cfg, fn) != QSA_OK || check_batch(batch, fn) != QSA_OK) return 0;
  if (cfg->kv_dtype == QSA_Q8_0) return 0;
  return workspace_bytes_of(plan_attn(batch, cfg), cfg->head_dim);
}

QSA_API qsa_status qsa_paged_attn(const qsa_paged_cache* cache, const qsa_paged_batch* batch,
                                  const qsa_attn_config* cfg, int32_t window, int32_t n_sinks, const void* q,
                                  void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const NvtxRange nvtx_range("qsa_paged_attn");
  const char* fn = "qsa_paged_attn";
  qsa_status s = check_config(cfg, fn);
  if (s != QSA_OK) return s;
  if ((s = check_cache(cache, cfg, fn)) != QSA_OK) return s;
  if ((s = check_batch(batch, fn)) != QSA_OK) return s;
  if (window < 0 || n_sinks < 0)
    return fail(QSA_ERR_INVALID_ARG, "%s: window=%d, n_sinks=%d", fn, window, n_sinks);
  if (batch->n_seqs == 0 || batch->n_rows == 0) return ok();
  if (!q || !out) return fail(QSA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (!aligned16(q) || !aligned16(out)) return fail(QSA_ERR_MISALIGNED, "%s: q/out not 16-byte aligned", fn);
  const Plan pl = plan_attn(batch, cfg);
  const size_t need = workspace_bytes_of(pl, cfg->head_dim);
  if (!workspace || workspace_bytes < need)
    return fail(QSA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                workspace ? workspace_bytes : (size_t)0);
  if (!aligned16(workspace)) return fail(QSA_ERR_MISALIGNED, "%s: workspace not aligned", fn);
  PagedParams p{};
  p.k = cache->k;
  p.v = cache->v;
  p.page_stride = cache->page_stride;
  p.head_stride = cache->head_stride;
  p.tok_stride = cache->tok_stride;
  p.kv_scale = static_cast<const uint8_t*>(cache->kv_scale);
  p.s_page_stride = cache->scale_page_stride;
  p.s_head_stride = cache->scale_head_stride;
  p.s_tok_stride = cache->scale_tok_stride;
  p.n_pages = cache->n_pages;
  p.page_shift = log2_of(cache->page_tokens);
  p.table = batch->table;
  p.table_ld = batch->table_ld;
  p.lens = batch->lens;
  p.row_start = batch->row_start;
  p.n_seqs = batch->n_seqs;
  p.n_rows = batch->n_rows;
  p.n_q_heads = cfg->n_q_heads;
  p.n_kv_heads = cfg->n_kv_heads;
  p.group = cfg->n_q_heads / cfg->n_kv_heads;
  p.group_magic = p.group == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + p.group - 1) / p.group);
  p.scale = cfg->scale > 0.f ? cfg->scale : 1.0f / sqrtf((float)cfg->head_dim);
  p.window = window < paged::kMaxLen ? window : 0;   // no sequence is longer
  p.n_sinks = n_sinks;
  p.q = q;
  p.out = out;
  p.lse = lse;
  p.out_dtype = cfg->out_dtype;
  p.mt = pl.mt;
  char* ws = static_cast<char*>(workspace);
  p.parts = reinterpret_cast<PagedPart*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + lse_offset(pl));
  p.part_o = reinterpret_cast<float*>(ws + out_offset(pl));
  cudaStream_t st = as_stream(stream);
  cudaError_t e = pl.tensor_cores ? launch_paged_tc(p, cfg->kv_dtype, cfg->head_dim, pl.grid, st)
                                  : launch_paged_f32(p, cfg->head_dim, pl.grid, st);
  if (e == cudaSuccess) e = launch_paged_merge(p, cfg->head_dim, pl.grid, st);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

QSA_API qsa_status qsa_paged_append(const qsa_paged_cache* cache, const qsa_paged_batch* batch,
                                    const qsa_attn_config* cfg, const void* k_new, const void* v_new,
                                    int64_t row_stride, int64_t head_stride, void* stream) {
  const NvtxRange nvtx_range("qsa_paged_append");
  const char* fn = "qsa_paged_append";
  qsa_status s = check_config(cfg, fn);
  if (s != QSA_OK) return s;
  if ((s = check_cache(cache, cfg, fn)) != QSA_OK) return s;
  if ((s = check_batch(batch, fn)) != QSA_OK) return s;
  if (batch->n_seqs == 0 || batch->n_rows == 0) return ok();
  const int64_t es = cfg->kv_dtype == QSA_F32 ? 4 : 2, most = (int64_t)1 << 40;
  if (!k_new || !v_new) return fail(QSA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (row_stride < 0 || head_stride < 0 || row_stride > most || head_stride > most)
    return fail(QSA_ERR_INVALID_ARG, "%s: row_stride=%lld, head_stride=%lld", fn, (long long)row_stride,
                (long long)head_stride);
  if (!aligned16(k_new) || !aligned16(v_new) || (row_stride * es) % 16 || (head_stride * es) % 16)
    return fail(QSA_ERR_MISALIGNED, "%s: k_new, v_new or their strides not 16-byte aligned", fn);
  PagedAppendParams p{};
  p.k = const_cast<void*>(cache->k);
  p.v = const_cast<void*>(cache->v);
  p.page_stride = cache->page_stride;
  p.head_stride = cache->head_stride;
  p.tok_stride = cache->tok_stride;
  p.kv_scale = const_cast<void*>(cache->kv_scale);
  p.s_page_stride = cache->scale_page_stride;
  p.s_head_stride = cache->scale_head_stride;
  p.s_tok_stride = cache->scale_tok_stride;
  p.n_pages = cache->n_pages;
  p.page_shift = log2_of(cache->page_tokens);
  p.table = batch->table;
  p.table_ld = batch->table_ld;
  p.lens = batch->lens;
  p.row_start = batch->row_start;
  p.n_seqs = batch->n_seqs;
  p.n_rows = batch->n_rows;
  p.n_kv_heads = cfg->n_kv_heads;
  p.head_dim = cfg->head_dim;
  p.k_new = k_new;
  p.v_new = v_new;
  p.row_stride = row_stride;
  p.new_head_stride = head_stride;
  const cudaError_t e = launch_paged_append(p, cfg->kv_dtype, as_stream(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

// ------------------------------------------------------------------ pages
namespace {

qsa_status check_pool(const qsa_page_pool* p, const char* fn) {
  if (!p) return fail(QSA_ERR_INVALID_ARG, "%s: null pool", fn);
  if (p->n_seqs < 1 || p->n_pages < 1 || p->table_ld < 1)
    return fail(QSA_ERR_INVALID_ARG, "%s: pool of %d places, %d pages, table_ld=%lld", fn, p->n_seqs, p->n_pages,
                (long long)p->table_ld);
  if (p->page_tokens < QSA_MIN_PAGE_TOKENS || p->page_tokens > QSA_MAX_PAGE_TOKENS ||
      (p->page_tokens & (p->page_tokens - 1)) != 0)
    return fail(QSA_ERR_UNSUPPORTED, "%s: page_tokens=%d (a power of two in %d..%d)", fn, p->page_tokens,
                QSA_MIN_PAGE_TOKENS, QSA_MAX_PAGE_TOKENS);
  if (p->n_pages > (1 << 24) || p->table_ld > (1 << 24))
    return fail(QSA_ERR_UNSUPPORTED, "%s: more than %d pages or table entries", fn, 1 << 24);
  if (!p->table || !p->lens || !p->refs) return fail(QSA_ERR_INVALID_ARG, "%s: pool has a null array", fn);
  return QSA_OK;
}

qsa_status check_requests(const int32_t* list, int32_t n, const char* fn) {
  if (n < 0) return fail(QSA_ERR_INVALID_ARG, "%s: n=%d", fn, n);
  if (n > QSA_MAX_PAGE_REQUESTS)
    return fail(QSA_ERR_UNSUPPORTED, "%s: %d requests (at most %d)", fn, n, QSA_MAX_PAGE_REQUESTS);
  if (n > 0 && !list) return fail(QSA_ERR_INVALID_ARG, "%s: null list", fn);
  return QSA_OK;
}

qsa_status check_caches(const qsa_page_pool* pool, const qsa_paged_cache* caches, int32_t n_caches,
                        const qsa_attn_config* cfg, const char* fn) {
  if (n_caches < 0 || n_caches > QSA_MAX_CACHES)
    return fail(QSA_ERR_UNSUPPORTED, "%s: %d caches (0..%d)", fn, n_caches, QSA_MAX_CACHES);
  if (n_caches == 0) return QSA_OK;
  if (!caches) return fail(QSA_ERR_INVALID_ARG, "%s: null caches", fn);
  qsa_status s = check_config(cfg, fn);
  if (s != QSA_OK) return s;
  for (int i = 0; i < n_caches; ++i) {
    if ((s = check_cache(caches + i, cfg, fn)) != QSA_OK) return s;
    // The copies count a page's 16-byte pieces, a batch of them ahead, in 32 bits.
    const int64_t bytes = (int64_t)caches[i].page_tokens * cfg->n_kv_heads * cfg->head_dim * (int64_t)dtype_size(cfg->kv_dtype);
    if (bytes / 16 > INT32_MAX - 4096)
      return fail(QSA_ERR_UNSUPPORTED, "%s: cache %d has pages of %lld bytes of K (below 32 GB)", fn, i, (long long)bytes);
    if (caches[i].page_tokens != (pool ? pool->page_tokens : caches[0].page_tokens))
      return fail(QSA_ERR_INVALID_ARG, "%s: cache %d has pages of another size", fn, i);
    if (pool && caches[i].n_pages < pool->n_pages)
      return fail(QSA_ERR_INVALID_ARG, "%s: cache %d has %d pages", fn, i, caches[i].n_pages);
  }
  return QSA_OK;
}

qsa_status check_workspace(const qsa_page_pool* pool, const void* ws, size_t bytes, const char* fn) {
  const size_t need = pages_workspace_bytes(*pool);
  if (!ws || bytes < need)
    return fail(QSA_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need, ws ? bytes : (size_t)0);
  if (!aligned16(ws)) return fail(QSA_ERR_MISALIGNED, "%s: workspace not aligned", fn);
  return QSA_OK;
}

// Caches [at, at + kPageCaches) of a call, as one launch takes them.
PageCaches caches_of(const qsa_paged_cache* caches, int n_caches, const qsa_attn_config* cfg, int at) {
  PageCaches out{};
  out.n = std::min(n_caches - at, kPageCaches);
  if (out.n <= 0) {
    out.n = 0;
    return out;
  }
  const int64_t es = (int64_t)dtype_size(cfg->kv_dtype);
  for (int i = 0; i < out.n; ++i) {
    const qsa_paged_cache& c = caches[at + i];
    out.c[i] = PageCache{const_cast<void*>(c.k),
                         const_cast<void*>(c.v),
                         cfg->kv_dtype == QSA_FP8_E4M3 ? const_cast<void*>(c.kv_scale) : nullptr,
                         c.page_stride * es,
                         c.head_stride * es,
                         c.tok_stride * es,
                         4 * c.scale_page_stride,
                         4 * c.scale_head_stride,
                         4 * c.scale_tok_stride};
  }
  out.n_pages = caches[0].n_pages;   // what all of the call's caches have
  for (int i = 1; i < n_caches; ++i) out.n_pages = std::min(out.n_pages, caches[i].n_pages);
  out.n_kv_heads = cfg->n_kv_heads;
  out.page_shift = log2_of(caches[at].page_tokens);
  out.row_shift = log2_of(cfg->head_dim * es / 16);
  return out;
}

}  // namespace

QSA_API size_t qsa_pages_workspace_size(const qsa_page_pool* pool) {
  return check_pool(pool, "qsa_pages_workspace_size") == QSA_OK ? pages_workspace_bytes(*pool) : 0;
}

static qsa_status extend(const qsa_page_pool* pool, const int32_t* seqs, const int32_t* n_new, int32_t n,
                         int32_t* step_lens, void* stream, const char* fn) {
  qsa_status s = check_pool(pool, fn);
  if (s != QSA_OK) return s;
  if ((s = check_requests(seqs, n, fn)) != QSA_OK) return s;
  if (n > 0 && !n_new) return fail(QSA_ERR_INVALID_ARG, "%s: null n_new", fn);
  if (n == 0 && !step_lens) return ok();
  const cudaError_t e = launch_pages_extend(*pool, seqs, n_new, n, step_lens, as_stream(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

QSA_API qsa_status qsa_pages_extend(const qsa_page_pool* pool, const int32_t* seqs, const int32_t* n_new, int32_t n,
                                    void* stream) {
  const NvtxRange nvtx_range("qsa_pages_extend");
  return extend(pool, seqs, n_new, n, nullptr, stream, "qsa_pages_extend");
}

QSA_API qsa_status qsa_pages_extend_step(const qsa_page_pool* pool, const int32_t* seqs, const int32_t* n_new,
                                         int32_t n, int32_t* step_lens, void* stream) {
  const NvtxRange nvtx_range("qsa_pages_extend_step");
  const char* fn = "qsa_pages_extend_step";
  if (!step_lens) return fail(QSA_ERR_INVALID_ARG, "%s: null step_lens", fn);
  return extend(pool, seqs, n_new, n, step_lens, stream, fn);
}

QSA_API qsa_status qsa_pages_fork(const qsa_page_pool* pool, const qsa_paged_cache* caches, int32_t n_caches,
                                  const qsa_attn_config* cfg, const int32_t* src, const int32_t* dst,
                                  const int32_t* keep, int32_t n, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  const NvtxRange nvtx_range("qsa_pages_fork");
  const char* fn = "qsa_pages_fork";
  qsa_status s = check_pool(pool, fn);
  if (s != QSA_OK) return s;
  if ((s = check_caches(pool, caches, n_caches, cfg, fn)) != QSA_OK) return s;
  if ((s = check_requests(src, n, fn)) != QSA_OK || (s = check_requests(dst, n, fn)) != QSA_OK) return s;
  if (n == 0) return ok();
  if ((s = check_workspace(pool, workspace, workspace_bytes, fn)) != QSA_OK) return s;
  cudaStream_t st = as_stream(stream);
  cudaError_t e = launch_pages_fork_plan(*pool, src, dst, keep, n, workspace, st);
  for (int at = 0; e == cudaSuccess && (at == 0 || at < n_caches); at += kPageCaches)
    e = launch_pages_fork(*pool, caches_of(caches, n_caches, cfg, at), at == 0, n, workspace, st);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

QSA_API qsa_status qsa_pages_free(const qsa_page_pool* pool, const int32_t* seqs, const int32_t* keep, int32_t n,
                                  void* stream) {
  const NvtxRange nvtx_range("qsa_pages_free");
  const char* fn = "qsa_pages_free";
  qsa_status s = check_pool(pool, fn);
  if (s != QSA_OK) return s;
  if ((s = check_requests(seqs, n, fn)) != QSA_OK) return s;
  if (n == 0) return ok();
  const cudaError_t e = launch_pages_free(*pool, seqs, keep, n, as_stream(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

QSA_API qsa_status qsa_pages_compact(const qsa_page_pool* pool, const qsa_paged_cache* caches, int32_t n_caches,
                                     const qsa_attn_config* cfg, int32_t* n_used, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const NvtxRange nvtx_range("qsa_pages_compact");
  const char* fn = "qsa_pages_compact";
  qsa_status s = check_pool(pool, fn);
  if (s != QSA_OK) return s;
  if ((s = check_caches(pool, caches, n_caches, cfg, fn)) != QSA_OK) return s;
  if ((s = check_workspace(pool, workspace, workspace_bytes, fn)) != QSA_OK) return s;
  cudaStream_t st = as_stream(stream);
  cudaError_t e = launch_pages_compact_plan(*pool, n_used, workspace, st);
  for (int at = 0; e == cudaSuccess && (at == 0 || at < n_caches); at += kPageCaches)
    e = launch_pages_compact(*pool, caches_of(caches, n_caches, cfg, at), at == 0, workspace, st);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}

QSA_API qsa_status qsa_pages_copy(const qsa_paged_cache* caches, int32_t n_caches, const qsa_attn_config* cfg,
                                  const int32_t* src, const int32_t* dst, int32_t n, void* stream) {
  const NvtxRange nvtx_range("qsa_pages_copy");
  const char* fn = "qsa_pages_copy";
  const qsa_status s = check_caches(nullptr, caches, n_caches, cfg, fn);
  if (s != QSA_OK) return s;
  if (n < 0) return fail(QSA_ERR_INVALID_ARG, "%s: n=%d", fn, n);
  if (n == 0 || n_caches == 0) return ok();
  if (!src || !dst) return fail(QSA_ERR_INVALID_ARG, "%s: null list", fn);
  cudaError_t e = cudaSuccess;
  for (int at = 0; e == cudaSuccess && at < n_caches; at += kPageCaches)
    e = launch_pages_copy(caches_of(caches, n_caches, cfg, at), src, dst, n, as_stream(stream));
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}
