// Shared by the kernels over a paged K/V cache: launch parameters, the
// division of a call's work over the CTAs, and the lookup of a page.
//
// Work items.  The query rows of a sequence (n of them, at positions
// len - n .. len - 1) and the G query heads of a KV head are one axis of
// f = row * G + head-in-group entries, cut into tiles of MT entries: an item is
// one (sequence, tile, KV head).  Its keys are the tokens that any row of the
// tile can see, in tiles of KT tokens aligned at token 0: the tiles of
// [0, n_sinks) and those of [p_first - window + 1, p_last] with a window, else
// all tiles up to p_last.  Every item has at least one tile, so a row that sees
// nothing is written too.
//
// Division.  The key tiles of all items, one after the other in the order
// (sequence, tile, KV head, key tile), are cut into one contiguous run of
// nearly equal length per CTA, whatever the lengths of the sequences: of N tiles,
// each of C CTAs takes N / C and the first N mod C one more.  An item inside one run is written
// to the output at once; the parts of an item that crosses runs go to the
// workspace (at most two per CTA: the item its run starts inside, and the item
// its run ends inside) and are joined by their log-sum-exp in a second launch.
// lens and row_start are read on the device, so a captured call follows them.
#pragma once

#include "qsa_internal.cuh"

namespace qsa {

struct PagedParams {
  const void* k;
  const void* v;
  int64_t page_stride, head_stride, tok_stride;   // elements
  const uint8_t* kv_scale;                        // fp8 state: (K, V) f16 pairs
  int64_t s_page_stride, s_head_stride, s_tok_stride;   // records of 4 bytes
  int32_t n_pages;
  int32_t page_shift;        // log2 of the tokens in a page
  const int32_t* table;      // [n_seqs, table_ld]
  int64_t table_ld;
  const int32_t* lens;       // [n_seqs]
  const int32_t* row_start;  // [n_seqs + 1]
  int32_t n_seqs;
  int32_t n_rows;            // rows of q and out
  int32_t n_q_heads, n_kv_heads, group;
  uint32_t group_magic;      // ceil(2^32 / group); group 1: not used
  float scale;
  int32_t window, n_sinks;   // window 0: every token up to the row's own
  const void* q;             // [n_rows, Hq, D]
  void* out;                 // [n_rows, Hq, D]
  float* lse;                // [n_rows, Hq] or null
  int32_t out_dtype;
  struct PagedPart* parts;   // [grid] items that start in a CTA and end in a later one
  float* part_lse;           // [2 grid, MT], base 2
  float* part_o;             // [2 grid, MT, D], normalised
  int32_t mt;                // entries of an item
};

// An item whose key tiles are spread over n_parts CTAs, from this entry's on.
struct alignas(16) PagedPart {
  int32_t n_parts;   // 0: no such item starts here
  int32_t row0;      // the sequence's first row
  int32_t f0;        // the item's first entry
  int32_t nf_head;   // its entries (at most 128), and 2^8 times the KV head
};

// Writing rows into their pages (qsa_paged_append.cu).
struct PagedAppendParams {
  void* k;
  void* v;
  int64_t page_stride, head_stride, tok_stride;         // elements
  void* kv_scale;
  int64_t s_page_stride, s_head_stride, s_tok_stride;   // records
  int32_t n_pages, page_shift;
  const int32_t* table;
  int64_t table_ld;
  const int32_t* lens;
  const int32_t* row_start;
  int32_t n_seqs, n_rows, n_kv_heads, head_dim;
  const void* k_new;
  const void* v_new;
  int64_t row_stride, new_head_stride;                  // elements
};
cudaError_t launch_paged_append(const PagedAppendParams& p, qsa_dtype kv_dtype, cudaStream_t st);
int paged_append_bad_pages_take();

// Keeping the pages of a pool (qsa_pages.cu).
constexpr int kPageCaches = 32;   // caches of one launch
struct PageCache {
  void* k;
  void* v;
  void* kv_scale;
  int64_t page_stride, head_stride, tok_stride;         // bytes
  int64_t s_page_stride, s_head_stride, s_tok_stride;   // bytes
};
struct PageCaches {
  PageCache c[kPageCaches];
  int32_t n;
  int32_t n_pages;           // that every cache of the call has
  int32_t n_kv_heads, page_shift;
  int32_t row_shift;         // log2 of the 16-byte pieces of a row
};
cudaError_t launch_pages_extend(const qsa_page_pool& pool, const int32_t* seqs, const int32_t* n_new, int n,
                                int32_t* step_lens, cudaStream_t st);
cudaError_t launch_pages_fork_plan(const qsa_page_pool& pool, const int32_t* src, const int32_t* dst,
                                   const int32_t* keep, int n, void* ws, cudaStream_t st);
cudaError_t launch_pages_fork(const qsa_page_pool& pool, const PageCaches& caches, bool rows, int n, const void* ws,
                              cudaStream_t st);
cudaError_t launch_pages_free(const qsa_page_pool& pool, const int32_t* seqs, const int32_t* keep, int n,
                              cudaStream_t st);
cudaError_t launch_pages_compact_plan(const qsa_page_pool& pool, int32_t* n_used, void* ws, cudaStream_t st);
cudaError_t launch_pages_compact(const qsa_page_pool& pool, const PageCaches& caches, bool rows, void* ws,
                                 cudaStream_t st);
cudaError_t launch_pages_copy(const PageCaches& caches, const int32_t* src, const int32_t* dst, int n, cudaStream_t st);
size_t pages_workspace_bytes(const qsa_page_pool& pool);
int pages_unserved_take();

// f32 caches (qsa_paged.cu).
cudaError_t launch_paged_f32(const PagedParams& p, int head_dim, int grid, cudaStream_t st);
// On the tensor cores (qsa_paged_tc.cu): bf16 and fp8 caches.
cudaError_t launch_paged_tc(const PagedParams& p, qsa_dtype kv_dtype, int head_dim, int grid, cudaStream_t st);
int paged_tc_bad_pages_take();
int paged_tc_wait_timeouts();
cudaError_t launch_paged_merge(const PagedParams& p, int head_dim, int runs, cudaStream_t st);
int paged_bad_pages_take();
int paged_f32_wait_timeouts();

namespace paged {

// Lengths above this are taken as this: positions and tiles then keep to 32 bits.
constexpr int32_t kMaxLen = INT32_MAX - (1 << 25);

// One sequence's rows and tokens, as the device arrays give them.
struct SeqRows {
  int32_t len, row0, n;
};
__device__ __forceinline__ SeqRows seq_rows(const PagedParams& p, int i) {
  SeqRows s;
  const int32_t a = __ldcg(p.row_start + i), b = __ldcg(p.row_start + i + 1);
  s.row0 = max(a, 0);
  s.n = max(min(b, p.n_rows) - s.row0, 0);   // rows past q's end are not there
  s.len = min(max(__ldcg(p.lens + i), 0), kMaxLen);
  return s;
}

// Row of entry f: f / group, for f below 2^28 (f * (magic * group - 2^32) is below
// 2^32 then, as group <= 16).  Divisions by a value that only the host knows are
// most of what finding a run and opening an item take.
__device__ __forceinline__ int row_of(const PagedParams& p, int f) {
  return p.group == 1 ? f : (int)__umulhi((uint32_t)f, p.group_magic);
}

template <int KT>
struct Tiles {
  int32_t count;      // key tiles of the item (at least 1)
  int32_t n_sink;     // the first n_sink of them start at token 0
  int32_t first;      // the others start at token first * KT
  __device__ __forceinline__ int32_t token(int x) const { return (x < n_sink ? x : first + x - n_sink) * KT; }
};

// The key tiles of entries [m MT, (m + 1) MT) of a sequence's rows.
template <int KT>
__device__ __forceinline__ Tiles<KT> item_tiles(const PagedParams& p, const SeqRows& s, int mt, int m) {
  const int j0 = row_of(p, m * mt), j1 = min(s.n - 1, row_of(p, (m + 1) * mt - 1));
  const int p0 = s.len - s.n + j0, p1 = s.len - s.n + j1;
  const int end = max(p1 + 1, 0);
  const int last = (end + KT - 1) / KT;
  Tiles<KT> t;
  t.n_sink = 0;
  t.first = 0;
  t.count = max(last, 1);
  if (p.window > 0) {
    const int lo = max(p0 - p.window + 1, 0) / KT;
    const int sink = (min(p.n_sinks, end) + KT - 1) / KT;
    if (sink < lo) {
      t.n_sink = sink;
      t.first = lo;
      t.count = max(sink + last - lo, 1);
    }
  }
  return t;
}
__device__ __forceinline__ int item_count(const PagedParams& p, const SeqRows& s, int mt) {
  const int f = s.n * p.group;
  if (f <= mt) return f > 0 ? 1 : 0;   // (no division where the call is short)
  return (f + mt - 1) / mt;
}

// a / b for a below 2^22, b above 0.
__device__ __forceinline__ uint32_t divide_small(uint32_t a, uint32_t b) {
  uint32_t q = (uint32_t)((float)a * __frcp_rn((float)b));   // off by one at most
  if (q * b > a) --q;
  else if ((q + 1) * b <= a) ++q;
  return q;
}

// Where a CTA's run starts: key tile x of item (seq, m, head); tile t0 of the
// call's `all`, which the first `ctas` CTAs share.
struct Start {
  int64_t n;           // tiles of the run
  int64_t t0, all;
  int32_t ctas;
  int32_t seq, m, head, x;
  SeqRows s;           // of seq
};

// Sum of one value per thread over the CTA, and the exclusive prefix (THREADS
// threads, all of them call; smem of THREADS / 32 values).
template <int THREADS>
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t* smem, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  __syncthreads();
  if (lane == 31) smem[warp] = inc;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += smem[w];
    total += smem[w];
  }
  return before + inc - v;
}

constexpr int kLongSeq = 8;   // items that one thread sums by itself

// Key tiles of sequence i0 + threadIdx.x over all its items and KV heads (all
// THREADS threads call; a sequence of many items is summed by the whole CTA).
template <int THREADS, int KT>
__device__ __forceinline__ int64_t seq_cost(const PagedParams& p, int mt, int i0, int64_t* scan_s) {
  const int i = i0 + (int)threadIdx.x;
  int items = 0;
  int64_t cost = 0;
  if (i < p.n_seqs) {
    const SeqRows s = seq_rows(p, i);
    items = item_count(p, s, mt);
    if (items <= kLongSeq)
      for (int m = 0; m < items; ++m) cost += item_tiles<KT>(p, s, mt, m).count;
  }
  for (int j = i0; j < min(i0 + THREADS, p.n_seqs); ++j) {
    if (!__syncthreads_or(i >= j && items > kLongSeq)) break;   // no long sequence is left
    const SeqRows sj = seq_rows(p, j);
    const int nj = item_count(p, sj, mt);
    if (nj <= kLongSeq) continue;
    int64_t mine = 0, sum;
    for (int m = (int)threadIdx.x; m < nj; m += THREADS) mine += item_tiles<KT>(p, sj, mt, m).count;
    cta_scan<THREADS>(mine, scan_s, sum);
    if (i == j) cost = sum;
  }
  return cost * p.n_kv_heads;
}

// Position r among the tiles of sequence i (as SeqRows s), as a run's start.
template <int KT>
__device__ __forceinline__ void place_in_seq(const PagedParams& p, int mt, int i, const SeqRows& s, int64_t r, Start& st) {
  int m = 0;
  Tiles<KT> t = item_tiles<KT>(p, s, mt, m);
  while (r >= (int64_t)t.count * p.n_kv_heads) {
    r -= (int64_t)t.count * p.n_kv_heads;
    t = item_tiles<KT>(p, s, mt, ++m);
  }
  st.seq = i;
  st.m = m;
  st.head = (int32_t)(r / t.count);
  st.x = (int32_t)(r - (int64_t)st.head * t.count);
  st.s = s;
}

// Key tiles of item m of a sequence, all KV heads (2^21 if they are more); 0
// behind its last item.
template <int KT>
__device__ __forceinline__ uint32_t item_cost(const PagedParams& p, int mt, const SeqRows& s, int items, int m) {
  const uint64_t all = (uint64_t)(uint32_t)item_tiles<KT>(p, s, mt, m).count * (uint32_t)p.n_kv_heads;
  return m < items ? (uint32_t)min(all, (uint64_t)1 << 21) : 0u;
}
__device__ __forceinline__ uint32_t warp_prefix(uint32_t v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  return v;
}

// find_run for at most 64 sequences: every warp finds the run by itself, two
// sequences a lane (a sequence of several items: one item a lane), with one round
// of loads and no barrier.  False (for all warps) where the call is larger.
template <int KT>
__device__ __forceinline__ bool find_run_small(const PagedParams& p, int mt, int cta, int n_ctas, Start& st) {
  if (p.n_seqs > 64) return false;
  const int lane = threadIdx.x & 31;
  const bool pairs = p.n_seqs > 32;   // lane's sequences: lane, or 2 lane and 2 lane + 1
  const int i0 = pairs ? 2 * lane : lane, i1 = i0 + 1;
  SeqRows mine[2] = {{0, 0, 0}, {0, 0, 0}};
  if (i0 < p.n_seqs) mine[0] = seq_rows(p, i0);
  if (pairs && i1 < p.n_seqs) mine[1] = seq_rows(p, i1);
  auto of = [&](int i) {   // sequence i
    const int k = pairs ? i & 1 : 0, from = pairs ? i >> 1 : i;
    SeqRows a{__shfl_sync(0xffffffffu, mine[0].len, from), __shfl_sync(0xffffffffu, mine[0].row0, from),
              __shfl_sync(0xffffffffu, mine[0].n, from)};
    const SeqRows b{__shfl_sync(0xffffffffu, mine[1].len, from), __shfl_sync(0xffffffffu, mine[1].row0, from),
                    __shfl_sync(0xffffffffu, mine[1].n, from)};
    return k ? b : a;
  };
  uint32_t cost[2] = {0u, 0u};
  uint32_t several[2] = {0u, 0u};   // sequences of more than one item
  bool large = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (k == 1 && !pairs) break;
    const int n = item_count(p, mine[k], mt);
    cost[k] = n == 1 ? item_cost<KT>(p, mt, mine[k], 1, 0) : 0u;
    large |= n > 4096 || cost[k] > (1u << 20);
    several[k] = __ballot_sync(0xffffffffu, n > 1 && !large);
  }
#pragma unroll 1
  while (several[0] | several[1]) {
    const int k = several[0] ? 0 : 1, from = __ffs(k == 0 ? several[0] : several[1]) - 1;
    if (k == 0) several[0] &= several[0] - 1;
    else several[1] &= several[1] - 1;
    const SeqRows s = of(pairs ? 2 * from + k : from);
    const int n = item_count(p, s, mt);
    uint32_t sum = 0;
#pragma unroll 1
    for (int m = lane; m < n; m += 32) {   // (at most 4,096 items of at most 2^13 tiles: 32 bits)
      const uint32_t c = item_cost<KT>(p, mt, s, n, m);
      large |= c > (1u << 13);
      sum += min(c, 1u << 13);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == from) {
      if (k == 0) cost[0] = sum;
      else cost[1] = sum;
      large |= sum > (1u << 20);
    }
  }
  if (__any_sync(0xffffffffu, large)) return false;
  const uint32_t inc = warp_prefix(cost[0] + cost[1], lane);
  const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);   // at most 2^26
  const uint32_t ctas = min((uint32_t)n_ctas, all);
  st = Start{0, 0, (int64_t)all, (int32_t)ctas, 0, 0, 0, 0, {0, 0, 0}};
  if ((uint32_t)cta >= ctas) return true;
  const uint32_t base = all == ctas ? 1u : all < (1u << 22) ? divide_small(all, ctas) : all / ctas, rem = all - base * ctas;
  const uint32_t t0 = base * (uint32_t)cta + min((uint32_t)cta, rem), tiles = base + ((uint32_t)cta < rem ? 1u : 0u);
  const int from = __ffs(__ballot_sync(0xffffffffu, inc > t0)) - 1;   // the first lane whose sequences end behind t0
  uint32_t r = t0 - __shfl_sync(0xffffffffu, inc - cost[0] - cost[1], from);
  const uint32_t first = __shfl_sync(0xffffffffu, cost[0], from);
  const bool second = r >= first;
  if (second) r -= first;
  const int i = pairs ? 2 * from + (second ? 1 : 0) : from;
  const SeqRows s = of(i);
  const int n = item_count(p, s, mt);
  int m = 0;
#pragma unroll 1
  for (int m0 = 0; n > 1; m0 += 32) {   // the first item that ends behind the rest
    const uint32_t c = item_cost<KT>(p, mt, s, n, m0 + lane);
    const uint32_t end = warp_prefix(c, lane);
    const uint32_t hit = __ballot_sync(0xffffffffu, end > r);
    if (hit || m0 + 32 >= n) {
      const int k = __ffs(hit) - 1;
      m = m0 + k;
      r -= __shfl_sync(0xffffffffu, end - c, k);
      break;
    }
    r -= __shfl_sync(0xffffffffu, end, 31);
  }
  const uint32_t count = (uint32_t)item_tiles<KT>(p, s, mt, m).count;
  st.n = tiles;
  st.t0 = t0;
  st.seq = i;
  st.m = m;
  st.head = (int32_t)(r < (1u << 22) ? divide_small(r, count) : r / count);
  st.x = (int32_t)(r - (uint32_t)st.head * count);
  st.s = s;
  return true;
}

// The first tile of CTA `cta`.
__device__ __forceinline__ int64_t run_start(int64_t all, int ctas, int cta) {
  const int64_t base = all / ctas;
  return base * cta + min((int64_t)cta, all - base * ctas);
}

// The run of CTA `cta` of at most `n_ctas` (all THREADS threads call; the
// result is the same for all).  Up to THREADS sequences take one pass; more
// take one for the number of tiles and one to find the run's start.
template <int THREADS, int KT>
__device__ Start find_run(const PagedParams& p, int mt, int cta, int n_ctas, int64_t* scan_s, Start* out_s) {
  Start small;
  if (find_run_small<KT>(p, mt, cta, n_ctas, small)) return small;
  int64_t all = 0, cost = 0, before = 0;
  for (int i0 = 0; i0 < p.n_seqs; i0 += THREADS) {
    int64_t total;
    cost = seq_cost<THREADS, KT>(p, mt, i0, scan_s);
    before = all + cta_scan<THREADS>(cost, scan_s, total);
    all += total;
  }
  const int ctas = (int)min((int64_t)n_ctas, all);   // every run holds a tile
  const int64_t t0 = cta < ctas ? run_start(all, ctas, cta) : 0, t1 = cta < ctas ? run_start(all, ctas, cta + 1) : 0;
  if (threadIdx.x == 0) *out_s = Start{0, 0, all, ctas, 0, 0, 0, 0, {0, 0, 0}};
  __syncthreads();
  if (t1 <= t0) return *out_s;
  int64_t base = 0;
  for (int i0 = 0; i0 < p.n_seqs; i0 += THREADS) {
    if (p.n_seqs > THREADS) {
      int64_t total;
      cost = seq_cost<THREADS, KT>(p, mt, i0, scan_s);
      before = base + cta_scan<THREADS>(cost, scan_s, total);
      base += total;
    }
    if (cost > 0 && t0 >= before && t0 < before + cost) {   // this thread's sequence holds the run's first tile
      Start st{t1 - t0, t0, all, ctas, 0, 0, 0, 0, {0, 0, 0}};
      const int i = i0 + (int)threadIdx.x;
      place_in_seq<KT>(p, mt, i, seq_rows(p, i), t0 - before, st);
      *out_s = st;
    }
  }
  __syncthreads();
  return *out_s;
}

// Steps through the items of a run; every role of a CTA keeps its own.
template <int KT>
struct Cursor {
  SeqRows s;
  Tiles<KT> tiles;
  int32_t seq, m, head, items;
  int32_t x, x1;       // this run's key tiles [x, x1) of the item
  int64_t left;        // tiles left, this item's included
  __device__ __forceinline__ void open(const PagedParams& p, int mt) {
    tiles = item_tiles<KT>(p, s, mt, m);
    x1 = (int32_t)min((int64_t)tiles.count, (int64_t)x + left);
  }
  __device__ __forceinline__ void begin(const PagedParams& p, int mt, const Start& st) {
    seq = st.seq;
    m = st.m;
    head = st.head;
    x = st.x;
    left = st.n;
    if (left <= 0) return;
    s = st.s;
    items = item_count(p, s, mt);
    open(p, mt);
  }
  // To the next item; false at the end of the run.
  __device__ __forceinline__ bool next(const PagedParams& p, int mt) {
    left -= x1 - x;
    if (left <= 0) return false;
    x = 0;
    if (++head == p.n_kv_heads) {
      head = 0;
      if (++m == items) {
        m = 0;
        do {
          s = seq_rows(p, ++seq);
          items = item_count(p, s, mt);
        } while (items == 0);
      }
    }
    open(p, mt);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return x == 0 && x1 == tiles.count; }
  // The workspace slot of this run's part of the item, of CTA `cta`.
  __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (x == 0 ? 1 : 0); }
};

// CTAs that the item at tile t_item of the call is spread over, from CTA `cta`
// (which holds its first tile) on.
template <int KT>
__device__ __forceinline__ int part_count(const Cursor<KT>& c, int64_t t_item, const Start& st, int cta) {
  const int64_t last = t_item + c.tiles.count - 1;
  // Runs of base + 1 tiles, then of base.
  int64_t e;
  if (st.all < INT32_MAX) {
    const uint32_t all = (uint32_t)st.all, b = all / (uint32_t)st.ctas, rem = all - b * (uint32_t)st.ctas, l = (uint32_t)last;
    e = l < rem * (b + 1) ? l / (b + 1) : rem + (l - rem * (b + 1)) / b;
  } else {
    const int64_t base = st.all / st.ctas;
    const int64_t rem = st.all - base * st.ctas;
    e = last < rem * (base + 1) ? last / (base + 1) : rem + (last - rem * (base + 1)) / base;
  }
  return (int)(e - cta) + 1;
}

// The item that crosses out of this run, for the joining launch: called by one
// thread with the run's last item (n_parts stays 0 where there is none).
template <int KT>
__device__ __forceinline__ void describe_part(const PagedParams& p, const Cursor<KT>& c, const Start& st, int cta) {
  PagedPart d{};
  if (st.n > 0 && c.x == 0 && c.x1 < c.tiles.count) {
    d.n_parts = part_count(c, st.t0 + st.n - (c.x1 - c.x), st, cta);
    d.row0 = c.s.row0;
    d.f0 = c.m * p.mt;
    d.nf_head = min(p.mt, c.s.n * p.group - d.f0) | c.head << 8;
  }
  p.parts[cta] = d;
}

// Token t of a sequence -> its page and the slot in it; false where the table
// has no such page (reported by qsa_check_device_status).
__device__ __forceinline__ bool page_of(const PagedParams& p, int seq, int t, int32_t& page) {
  const int64_t j = t >> p.page_shift;
  page = j < p.table_ld ? __ldcg(p.table + seq * p.table_ld + j) : -1;
  return (uint32_t)page < (uint32_t)p.n_pages;
}

// Whether the row at position pos sees token t.
__device__ __forceinline__ bool sees(const PagedParams& p, int pos, int t) {
  return t <= pos && (p.window == 0 || t > pos - p.window || t < p.n_sinks);
}

}  // namespace paged
}  // namespace qsa
