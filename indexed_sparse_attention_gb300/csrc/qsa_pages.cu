// Keeping the pages of a paged cache on the device: extend, fork, free, compact
// and copy (include/qsa.h, qsa_page_pool).
//
// The bookkeeping of a call is small (a list of sequences, one count per page)
// and every step of it depends on the one before, so one CTA of 1,024 threads
// plans it: a thread takes the same number of consecutive pages, and one scan
// over the CTA gives each free (or used) page its rank, which is what "the
// lowest free page" needs.  Pages are copied by a second launch over the whole
// GPU, one CTA per (page, cache, K or V), 16 bytes per thread.
//
// What bounds it: freeing and forking 32 children over 12 caches (4.5 MB) is 12 us
// on the GPU, a chain of three launches and their dependent reads; compacting 642
// MB of pages 113 us, 84% of the measured copy bandwidth.
#include "qsa_paged.cuh"

namespace qsa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;

__device__ int g_unserved;   // requests that could not be served, page numbers outside a pool

// Sum of one value per thread over the CTA, and the exclusive prefix.  Values are
// 0 .. 2^24 (pages, or those of a table row), and sums of 2^29 and more need not be
// exact, only no smaller: 1,024 requests may want 2^34 pages together, of which none
// behind the pool's 2^24 exist.
constexpr int kManyPages = 1 << 29;
__device__ __forceinline__ int scan(int v, int* smem, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();
  if (lane == 31) smem[warp] = inc;
  __syncthreads();
  int w = smem[lane];   // kPlanThreads / 32 == 32 sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w = min(w + up, kManyPages);
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp ? before : 0) + inc - v;
}

__device__ __forceinline__ int pages_for(int64_t tokens, int page_tokens) {   // (a power of two)
  return (int)((tokens + page_tokens - 1) >> (__ffs(page_tokens) - 1));
}

// Tokens of place s, within what its table row holds.
__device__ __forceinline__ int place_len(const qsa_page_pool& pool, int s) {
  const int64_t most = pool.table_ld * pool.page_tokens;
  return (int)min((int64_t)max(__ldcg(pool.lens + s), 0), most);
}

// The pages that thread t looks at: [t * n, (t + 1) * n) of the pool's.
struct Slice {
  int lo, hi;
};
__device__ __forceinline__ Slice slice(int n_pages) {
  const int per = (n_pages + kPlanThreads - 1) / kPlanThreads;
  const int lo = min((int)threadIdx.x * per, n_pages);
  return Slice{lo, min(lo + per, n_pages)};
}

// Whether the place of this thread's list entry is in the pool and not listed
// before; list_s holds the n entries.  All threads call it.  A warp compares its
// 32 entries with each other by one match and with the warps' before, four at a
// time: a loop over the entries before, of a length of its own in each lane, was
// most of the time of a call with 32 requests (extending them 16.5 us, 3 this way;
// 64 of them with the step's lengths 3.5).
__device__ __forceinline__ bool valid_place(const int* list_s, int n, int n_seqs) {
  const int i = (int)threadIdx.x, lane = i & 31;
  const int s = i < n ? list_s[i] : -1;
  bool first = (__match_any_sync(0xffffffffu, s) & ((1u << lane) - 1u)) == 0u;
  if ((i & ~31) < n) {
#pragma unroll 1
    for (int j = 0; j < (i & ~31); j += 4) {
      const int4 e = *reinterpret_cast<const int4*>(list_s + j);
      first = first && e.x != s && e.y != s && e.z != s && e.w != s;
    }
  }
  return i < n && first && s >= 0 && s < n_seqs;
}

// Pages of one round of the plan: 8 consecutive ones a thread.
constexpr int kRound = 8 * kPlanThreads;

// Which of pages [first, first + 8) are free, as bits (none past the pool's end).
__device__ __forceinline__ uint32_t free_bits(const qsa_page_pool& pool, int first) {
  uint32_t bits = 0u;
  int r[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) r[k] = first + k < pool.n_pages ? __ldcg(pool.refs + first + k) : 1;
#pragma unroll
  for (int k = 0; k < 8; ++k) bits |= (r[k] == 0 ? 1u : 0u) << k;
  return bits;
}

// Gives request i (this thread's) its `need` new pages: the lowest free ones in
// list order.  Returns whether it is served; give(page, rank, n_free) is called
// for each page handed out, by any thread, with its rank over all requests, once
// off_s[0 .. n] holds every request's first rank.  n_free is the number of free
// pages as far as it matters (those behind the last one wanted are not counted).
template <typename Give>
__device__ __forceinline__ bool take_pages(const qsa_page_pool& pool, int n, int need, int* scan_s, int* off_s,
                                           Give give) {
  const int i = (int)threadIdx.x;
  // (The first round's pages are on their way while the needs are summed.)
  uint32_t bits = free_bits(pool, 8 * i);
  int wanted, n_free = 0, rank = 0;
  const int off = scan(need, scan_s, wanted);
  if (i < n) off_s[i] = off;
  if (i == 0) off_s[n] = wanted;
  int rounds = 0;
  for (int lo = 0; lo < pool.n_pages && n_free < wanted; lo += kRound, ++rounds) {
    if (rounds > 0) bits = free_bits(pool, lo + 8 * i);
    int found;
    rank = n_free + scan(__popc(bits), scan_s, found);   // (its barriers publish off_s)
    n_free += found;
  }
  const bool served = need == 0 || off + need <= n_free;
  const int many = rounds;
  int base = 0;
  for (int k = 0; k < many; ++k) {
    if (many > 1) {   // the ranks of the earlier rounds again
      int found;
      bits = free_bits(pool, k * kRound + 8 * i);
      rank = base + scan(__popc(bits), scan_s, found);
      base += found;
    }
    for (uint32_t b = bits; b && rank < wanted; b &= b - 1) give(k * kRound + 8 * i + __ffs(b) - 1, rank++, n_free);
  }
  return served;
}

// The request that rank r belongs to: the last one that starts at or before r
// and wants a page.
__device__ __forceinline__ int request_of(const int* off_s, int n, int r) {
  int lo = 0, hi = n;   // off_s[lo] <= r < off_s[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (off_s[mid] <= r) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ extend
__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const qsa_page_pool pool, const int32_t* seqs,
                                                              const int32_t* n_new, int n, int32_t* step_lens) {
  __shared__ __align__(16) int list_s[QSA_MAX_PAGE_REQUESTS], off_s[QSA_MAX_PAGE_REQUESTS + 1], have_s[QSA_MAX_PAGE_REQUESTS];
  __shared__ int scan_s[32];
  grid_dependency_sync();
  const int i = (int)threadIdx.x;
  if (i < n) list_s[i] = __ldcg(seqs + i);
  __syncthreads();
  int need = 0, len = 0, add = 0;
  bool valid = false;
  if (valid_place(list_s, n, pool.n_seqs)) {
    len = place_len(pool, list_s[i]);
    add = __ldcg(n_new + i);
    const int64_t after = (int64_t)len + add;
    valid = add >= 0 && after <= pool.table_ld * (int64_t)pool.page_tokens && after < INT32_MAX;
    if (valid) {
      have_s[i] = pages_for(len, pool.page_tokens);
      need = pages_for(after, pool.page_tokens) - have_s[i];
    }
  }
  const bool served = take_pages(pool, n, need, scan_s, off_s, [&](int page, int rank, int n_free) {
    const int q = request_of(off_s, n, rank);
    if (off_s[q + 1] > n_free) return;   // not enough for this request: nothing for it
    pool.table[list_s[q] * pool.table_ld + have_s[q] + (rank - off_s[q])] = page;
    pool.refs[page] = 1;
  });
  const bool ok = i >= n || (valid && served);
  if (i < n) {
    if (ok) pool.lens[list_s[i]] = len + add;
    else atomicAdd(&g_unserved, 1);
  }
  if (!step_lens) return;
  // The step's lengths: no tokens for a place with a request that was not served.
  __syncthreads();
  for (int s = i; s < pool.n_seqs; s += kPlanThreads) step_lens[s] = __ldcg(pool.lens + s);
  __syncthreads();
  if (!ok && (uint32_t)list_s[i] < (uint32_t)pool.n_seqs) step_lens[list_s[i]] = 0;
}

// ------------------------------------------------------------------ fork
struct ForkPlan {
  int32_t src, dst;
  int32_t len;    // tokens of the new sequence; -1: not served
  int32_t page;   // its last page's copy, -1: none
};

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const qsa_page_pool pool, const int32_t* src,
                                                                 const int32_t* dst, const int32_t* keep, int n,
                                                                 ForkPlan* plan) {
  __shared__ __align__(16) int list_s[QSA_MAX_PAGE_REQUESTS], off_s[QSA_MAX_PAGE_REQUESTS + 1], page_s[QSA_MAX_PAGE_REQUESTS];
  __shared__ int scan_s[32];
  grid_dependency_sync();
  const int i = (int)threadIdx.x;
  if (i < n) {
    list_s[i] = __ldcg(dst + i);
    page_s[i] = -1;
  }
  __syncthreads();
  int need = 0, len = 0, s = 0;
  bool valid = false;
  if (valid_place(list_s, n, pool.n_seqs)) {
    s = __ldcg(src + i);
    if (s >= 0 && s < pool.n_seqs && __ldcg(pool.lens + list_s[i]) == 0) {
      len = place_len(pool, s);
      const int k = keep ? __ldcg(keep + i) : len;
      valid = k >= 0;
      len = min(len, max(k, 0));
      need = valid && len % pool.page_tokens != 0;
    }
  }
  const bool served = take_pages(pool, n, need, scan_s, off_s, [&](int page, int rank, int n_free) {
    const int q = request_of(off_s, n, rank);
    if (off_s[q + 1] > n_free) return;
    page_s[q] = page;
    pool.refs[page] = 1;
  });
  __syncthreads();
  if (i < n) {
    const bool ok = valid && served;
    plan[i] = ForkPlan{s, list_s[i], ok ? len : -1, ok ? page_s[i] : -1};
    if (!ok) atomicAdd(&g_unserved, 1);
  }
}

// The 16-byte pieces [first, n) of a page's K or V, and its scale records, by
// this CTA; only the first `fill` tokens of the page.
__device__ __forceinline__ void copy_page(const PageCaches& cs, const PageCache& c, int which, int64_t src, int64_t dst,
                                          int fill) {
  const char* from = static_cast<const char*>(which ? c.v : c.k) + src * c.page_stride;
  char* to = static_cast<char*>(which ? c.v : c.k) + dst * c.page_stride;
  const int row = 1 << cs.row_shift;
  // Consecutive threads follow memory: the pieces of a row, then the shorter
  // of the two strides.
  const bool heads_inner = c.head_stride < c.tok_stride;
  const int rows = fill * cs.n_kv_heads, n = rows << cs.row_shift;
  auto offset = [&](int i) {
    const int r = i >> cs.row_shift, piece = i & (row - 1);
    const int h = heads_inner ? r % cs.n_kv_heads : r / fill;
    const int t = heads_inner ? r / cs.n_kv_heads : r - h * fill;
    return h * c.head_stride + t * c.tok_stride + piece * 16;
  };
  constexpr int kBatch = 8;   // loads of a thread in flight
  for (int i0 = (int)threadIdx.x; i0 < n; i0 += kCopyThreads * kBatch) {
    uint4 x[kBatch];
    int64_t at[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kCopyThreads;
      if (i < n) {
        at[k] = offset(i);
        x[k] = __ldcs(reinterpret_cast<const uint4*>(from + at[k]));
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k * kCopyThreads < n) __stcs(reinterpret_cast<uint4*>(to + at[k]), x[k]);
  }
  if (which == 0 && c.kv_scale) {
    const char* sf = static_cast<const char*>(c.kv_scale) + src * c.s_page_stride;
    char* st = static_cast<char*>(c.kv_scale) + dst * c.s_page_stride;
    for (int i = (int)threadIdx.x; i < rows * max(cs.record_pieces, 1); i += kCopyThreads) {
      const int r = cs.record_pieces > 1 ? i / cs.record_pieces : i;
      const int64_t o = (r / fill) * c.s_head_stride + (r % fill) * c.s_tok_stride;
      if (cs.record_pieces == 0) {
        *reinterpret_cast<uint32_t*>(st + o) = *reinterpret_cast<const uint32_t*>(sf + o);
      } else {
        const int64_t at = o + (i - r * cs.record_pieces) * 16;
        *reinterpret_cast<uint4*>(st + at) = *reinterpret_cast<const uint4*>(sf + at);
      }
    }
  }
}

// CTA (i, y): request i; y == 0 (with rows): its table row, counts and length;
// the others copy its last page in cache (y - rows) / 2, K or V.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const qsa_page_pool pool,
                                                            const __grid_constant__ PageCaches cs, int rows,
                                                            const ForkPlan* plan) {
  grid_dependency_sync();
  const ForkPlan f = plan[blockIdx.x];
  if (f.len < 0) return;
  const int full = f.len / pool.page_tokens;
  const int32_t* from = pool.table + f.src * pool.table_ld;
  if (rows && blockIdx.y == 0) {
    int32_t* to = pool.table + f.dst * pool.table_ld;
    constexpr int kBatch = 4;
    for (int j0 = (int)threadIdx.x; j0 < full; j0 += kBatch * kCopyThreads) {
      int32_t page[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) page[k] = j0 + k * kCopyThreads < full ? __ldcg(from + j0 + k * kCopyThreads) : -1;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (j0 + k * kCopyThreads < full) to[j0 + k * kCopyThreads] = page[k];
        if ((uint32_t)page[k] < (uint32_t)pool.n_pages) atomicAdd(pool.refs + page[k], 1);
      }
    }
    if (threadIdx.x == 0) {
      if (f.page >= 0) to[full] = f.page;
      pool.lens[f.dst] = f.len;
    }
    return;
  }
  const int y = (int)blockIdx.y - rows;
  const int32_t page = f.page >= 0 ? __ldcg(from + full) : -1;
  if ((uint32_t)page < (uint32_t)pool.n_pages) copy_page(cs, cs.c[y >> 1], y & 1, page, f.page, f.len % pool.page_tokens);
}

// ------------------------------------------------------------------ free
// The pages of sequence s behind its first `keep` tokens, by one group of
// threads (first thread t0 of n).
__device__ __forceinline__ void give_up(const qsa_page_pool& pool, int s, int keep, int len, int t0, int n) {
  int32_t* row = pool.table + s * pool.table_ld;
  const int last = pages_for(len, pool.page_tokens);
  constexpr int kBatch = 4;   // entries of a thread whose loads, then counts, are in flight together
  for (int j0 = pages_for(keep, pool.page_tokens) + t0; j0 < last; j0 += kBatch * n) {
    int32_t page[kBatch];
    int was[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) page[k] = j0 + k * n < last ? __ldcg(row + j0 + k * n) : -1;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (j0 + k * n < last) row[j0 + k * n] = -1;
      was[k] = (uint32_t)page[k] < (uint32_t)pool.n_pages ? atomicSub(pool.refs + page[k], 1) : 1;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (was[k] <= 0) {   // nobody used it: not this call's doing
        atomicAdd(pool.refs + page[k], 1);
        atomicAdd(&g_unserved, 1);
      }
  }
}

// Whole sequences: one CTA each.
__global__ void __launch_bounds__(kCopyThreads) free_kernel(const qsa_page_pool pool, const int32_t* seqs) {
  grid_dependency_sync();
  const int i = (int)blockIdx.x, s = __ldcg(seqs + i);
  int before = 0;
  for (int j = (int)threadIdx.x; j < i; j += kCopyThreads) before |= __ldcg(seqs + j) == s;
  const bool listed = __syncthreads_or(before);
  if (listed || s < 0 || s >= pool.n_seqs) {
    if (threadIdx.x == 0) atomicAdd(&g_unserved, 1);
    return;
  }
  const int len = place_len(pool, s);
  __syncthreads();
  give_up(pool, s, 0, len, (int)threadIdx.x, kCopyThreads);
  if (threadIdx.x == 0) pool.lens[s] = 0;
}

// Parts of sequences: one CTA, since a request that is not served depends on
// counts that the others of the call change.
__global__ void __launch_bounds__(kPlanThreads) cut_kernel(const qsa_page_pool pool, const int32_t* seqs,
                                                           const int32_t* keep, int n) {
  __shared__ __align__(16) int list_s[QSA_MAX_PAGE_REQUESTS], len_s[QSA_MAX_PAGE_REQUESTS], keep_s[QSA_MAX_PAGE_REQUESTS];
  grid_dependency_sync();
  const int i = (int)threadIdx.x;
  if (i < n) list_s[i] = __ldcg(seqs + i);
  __syncthreads();
  const bool listed = valid_place(list_s, n, pool.n_seqs);
  if (i < n) {
    int k = -1, len = 0;
    if (listed) {
      len = place_len(pool, list_s[i]);
      k = __ldcg(keep + i);
      if (k >= len && k >= 0) k = len;   // nothing to give up
      if (k > 0 && k < len && k % pool.page_tokens != 0) {
        const int32_t page = __ldcg(pool.table + list_s[i] * pool.table_ld + k / pool.page_tokens);
        if ((uint32_t)page < (uint32_t)pool.n_pages && __ldcg(pool.refs + page) > 1) k = -1;
      }
    }
    len_s[i] = len;
    keep_s[i] = k;
    if (k < 0) atomicAdd(&g_unserved, 1);
  }
  __syncthreads();
  for (int j = i / 32; j < n; j += kPlanThreads / 32) {
    const int k = keep_s[j], len = len_s[j];
    if (k < 0 || k >= len) continue;
    give_up(pool, list_s[j], k, len, i & 31, 32);
    if ((i & 31) == 0) pool.lens[list_s[j]] = k;
  }
}

// ------------------------------------------------------------------ compact
// Workspace: the number of moves, the first page number that moves away, then
// three arrays of n_pages: sources, destinations, and each source's destination.
struct CompactHead {
  int32_t moves, used, pad[2];
};
__device__ __forceinline__ int32_t* compact_list(void* ws, int n_pages, int which) {
  return reinterpret_cast<int32_t*>(static_cast<char*>(ws) + sizeof(CompactHead)) + (int64_t)which * n_pages;
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const qsa_page_pool pool, int32_t* n_used,
                                                                    void* ws) {
  __shared__ int scan_s[32], low_s;
  grid_dependency_sync();
  const Slice sl = slice(pool.n_pages);
  int mine = 0, used;
#pragma unroll 8
  for (int k = sl.lo; k < sl.hi; ++k) mine += __ldcg(pool.refs + k) > 0;
  const int before = scan(mine, scan_s, used);
  // Pages in use below page number `used`: the moves fill the holes there.
  int low = 0, total_low;
  for (int k = sl.lo; k < min(sl.hi, used); ++k) low += __ldcg(pool.refs + k) > 0;
  scan(low, scan_s, total_low);
  if (threadIdx.x == 0) low_s = total_low;
  __syncthreads();
  int32_t* src = compact_list(ws, pool.n_pages, 0);
  int32_t* dst = compact_list(ws, pool.n_pages, 1);
  int32_t* to = compact_list(ws, pool.n_pages, 2);
  int u = before;
  for (int k = sl.lo; k < sl.hi; ++k) {
    const bool in_use = __ldcg(pool.refs + k) > 0;
    if (k >= used && in_use) src[u - low_s] = k;
    if (k >= used && !in_use) to[k] = k;   // (a table that names a page nobody counts keeps it)
    if (k < used && !in_use) dst[k - u] = k;
    u += in_use;
  }
  __syncthreads();
  const int moves = used - low_s;
  for (int r = (int)threadIdx.x; r < moves; r += kPlanThreads) {
    const int a = src[r], b = dst[r];
    to[a] = b;
    pool.refs[b] = pool.refs[a];
    pool.refs[a] = 0;
  }
  if (threadIdx.x == 0) {
    *static_cast<CompactHead*>(ws) = CompactHead{moves, used, {0, 0}};
    if (n_used) *n_used = used;
  }
}

// Copies of (move, cache, K or V) in turn, and the table's entries (rows).
__global__ void __launch_bounds__(kCopyThreads) compact_kernel(const qsa_page_pool pool,
                                                               const __grid_constant__ PageCaches cs, int rows,
                                                               void* ws) {
  grid_dependency_sync();
  const CompactHead head = *static_cast<const CompactHead*>(ws);
  const int32_t* src = compact_list(ws, pool.n_pages, 0);
  const int32_t* dst = compact_list(ws, pool.n_pages, 1);
  const int32_t* to = compact_list(ws, pool.n_pages, 2);
  if (rows && head.moves > 0) {
    for (int s = (int)blockIdx.x; s < pool.n_seqs; s += (int)gridDim.x) {
      const int n = pages_for(place_len(pool, s), pool.page_tokens);
      int32_t* row = pool.table + s * pool.table_ld;
      for (int j = (int)threadIdx.x; j < n; j += kCopyThreads) {
        const int32_t page = row[j];
        if (page >= head.used && page < pool.n_pages) row[j] = __ldcg(to + page);
      }
    }
  }
  const int64_t jobs = (int64_t)head.moves * cs.n * 2;
  for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
    const int m = (int)(j / (cs.n * 2)), y = (int)(j % (cs.n * 2));
    copy_page(cs, cs.c[y >> 1], y & 1, __ldcg(src + m), __ldcg(dst + m), 1 << cs.page_shift);
  }
}

// ------------------------------------------------------------------ copy
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ PageCaches cs, const int32_t* src,
                                                            const int32_t* dst, int n) {
  grid_dependency_sync();
  const int64_t jobs = (int64_t)n * cs.n * 2;
  for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
    const int m = (int)(j / (cs.n * 2)), y = (int)(j % (cs.n * 2));
    const int a = __ldcg(src + m), b = __ldcg(dst + m);
    if ((uint32_t)a < (uint32_t)cs.n_pages && (uint32_t)b < (uint32_t)cs.n_pages && a != b)
      copy_page(cs, cs.c[y >> 1], y & 1, a, b, 1 << cs.page_shift);
    else if (threadIdx.x == 0 && y == 0 && a != b)
      atomicAdd(&g_unserved, 1);
  }
}

}  // namespace

size_t pages_workspace_bytes(const qsa_page_pool& pool) {
  const size_t compact = sizeof(CompactHead) + 3 * (size_t)pool.n_pages * sizeof(int32_t);
  const size_t fork = (size_t)QSA_MAX_PAGE_REQUESTS * sizeof(ForkPlan);
  return ((compact > fork ? compact : fork) + 255) / 256 * 256;
}

cudaError_t launch_pages_extend(const qsa_page_pool& pool, const int32_t* seqs, const int32_t* n_new, int n,
                                int32_t* step_lens, cudaStream_t st) {
  return launch_kernel(extend_kernel, dim3(1), dim3(kPlanThreads), 0, st, 0u, pool, seqs, n_new, n, step_lens);
}

cudaError_t launch_pages_fork_plan(const qsa_page_pool& pool, const int32_t* src, const int32_t* dst,
                                   const int32_t* keep, int n, void* ws, cudaStream_t st) {
  return launch_kernel(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 0u, pool, src, dst, keep, n,
                       static_cast<ForkPlan*>(ws));
}

cudaError_t launch_pages_fork(const qsa_page_pool& pool, const PageCaches& caches, bool rows, int n, const void* ws,
                              cudaStream_t st) {
  const unsigned y = (unsigned)(2 * caches.n + (rows ? 1 : 0));
  if (y == 0) return cudaSuccess;
  return launch_kernel(fork_kernel, dim3((unsigned)n, y), dim3(kCopyThreads), 0, st, 0u, pool, caches, rows ? 1 : 0,
                       static_cast<const ForkPlan*>(ws));
}

cudaError_t launch_pages_free(const qsa_page_pool& pool, const int32_t* seqs, const int32_t* keep, int n,
                              cudaStream_t st) {
  if (keep) return launch_kernel(cut_kernel, dim3(1), dim3(kPlanThreads), 0, st, 0u, pool, seqs, keep, n);
  return launch_kernel(free_kernel, dim3((unsigned)n), dim3(kCopyThreads), 0, st, 0u, pool, seqs);
}

cudaError_t launch_pages_compact_plan(const qsa_page_pool& pool, int32_t* n_used, void* ws, cudaStream_t st) {
  return launch_kernel(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 0u, pool, n_used, ws);
}

cudaError_t launch_pages_compact(const qsa_page_pool& pool, const PageCaches& caches, bool rows, void* ws,
                                 cudaStream_t st) {
  return launch_kernel(compact_kernel, dim3((unsigned)(8 * device_sm_count())), dim3(kCopyThreads), 0, st, 0u, pool,
                       caches, rows ? 1 : 0, ws);
}

cudaError_t launch_pages_copy(const PageCaches& caches, const int32_t* src, const int32_t* dst, int n,
                              cudaStream_t st) {
  const int64_t jobs = (int64_t)n * caches.n * 2, most = 8 * (int64_t)device_sm_count();
  return launch_kernel(copy_kernel, dim3((unsigned)(jobs < most ? jobs : most)), dim3(kCopyThreads), 0, st, 0u, caches,
                       src, dst, n);
}

int pages_unserved_take() { return take_counter(g_unserved); }

}  // namespace qsa
