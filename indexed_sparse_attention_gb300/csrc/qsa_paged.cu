// Attention of a batch's newest rows over a paged K/V cache in f32, and the
// joining of an item's parts (see qsa_paged.cuh for the division of the work).
//
// For entry f = (row at position p, query head) of KV head g, with
// z_t = scale * q . k_t over the tokens t that the row sees:
//   m = max_t z_t,  l = sum_t exp(z_t - m),  out = sum_t exp(z_t - m) v_t / l,
//   lse = m + log l,
// in one pass over the key tiles with the running m and l of each entry (32-bit
// sums): a tile's new maximum m' rescales l and the output by exp(m - m').
#include <math.h>

#include "qsa_paged.cuh"
#include "qsa_tc.cuh"

namespace qsa {

namespace {

using namespace paged;
using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ int g_f32_timeouts;
__device__ int g_bad_pages;   // table entries outside [0, n_pages) among the tokens that a call read

// ------------------------------------------------------------------ f32 caches
// Products of f32 values on the tensor pipe, by tf32 halves: x = hi + lo with hi
// = x rounded to 11 significant bits and lo = x - hi rounded likewise, and
//   a b = hi_a hi_b + hi_a lo_b + lo_a hi_b  (+ lo_a lo_b, below 2^-22 |a b|, left out)
// with 32-bit accumulation: as exact as a 32-bit sum of rounded products.
//
// An item is 16 or 32 entries (one or two times the rows of m16n8k8), a key tile
// 32 tokens: warp w takes 16 entries (w / 4) and 8 tokens (w % 4) of it and keeps
// its own maximum, sum and output over its keys, so a tile needs no exchange; the
// four warps of an entry are joined like an item's parts at its end.
// Each row of K and V is one bulk copy, two tiles in flight.  Rows in shared memory
// are padded, Q's and K's by eight words and V's by four, which puts the eight
// rows and four column pairs (Q, K), or four row pairs and eight columns (V), of
// a fragment into different banks.
constexpr int kF32Threads = 256;
constexpr int kF32MT = 32;
constexpr int kF32KT = 32;

template <int D>
struct F32Layout {
  static constexpr int kRow = D + 8, kRowV = D + 4;        // words of a row of Q and K, and of V
  static constexpr int kK = kF32KT * kRow, kTile = kK + kF32KT * kRowV;   // words of K, and of K and V, of a tile
  static constexpr int kQ = 2 * kF32MT * kRow;             // hi, lo
  static constexpr size_t bytes = 4 * (size_t)(kQ + 2 * kTile);
  static_assert(8 * 16 * kRowV <= 2 * kTile, "the warps' outputs are joined in the tiles' place");
  static_assert((4 * kRow) % 16 == 0 && (4 * kRowV) % 16 == 0 && (4 * kQ) % 16 == 0, "rows on 16-byte boundaries");
};

// The halves of x.  Adding half a unit of the 11th significant bit to the pattern
// and clearing the 13 bits below rounds to nearest (halves away from zero); of lo
// the tensor pipe ignores those bits itself.  (In plain integer operations: the
// conversion instruction took most of the kernel's time.)
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) + 0x1000u;
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// bytes (a multiple of 16) from global to shared memory, counted by the barrier.
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
                   smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

template <int D>
__global__ void __launch_bounds__(kF32Threads) paged_f32_kernel(const PagedParams p) {
  using L = F32Layout<D>;
  constexpr int ROW = L::kRow, ROWV = L::kRowV, NT = D / 8;
  constexpr float kMoveMax = 8.f;   // as in the bf16 kernel: the maximum moves when a weight would pass 2^8
  extern __shared__ __align__(16) float fsm[];
  float* q_s = fsm;                 // hi [16][ROW], then lo
  float* kv_s = fsm + L::kQ;        // two tiles of [K 32][ROW], [V 32][ROWV]
  __shared__ int64_t scan_s[kF32Threads / 32];
  __shared__ Start start_s;
  __shared__ uint64_t full[2];
  __shared__ int abort_s;
  __shared__ uint8_t seen_s[2][4];  // tokens of a tile that some row sees and that have a page
  __shared__ float m_s[4][kF32MT], l_s[4][kF32MT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gr = lane >> 2, gc = lane & 3;   // a fragment's row group and column
  const int keys = warp & 3, rows16 = warp >> 2;
  if (tid == 0) {
    bar_init(&full[0], kF32Threads);
    bar_init(&full[1], kF32Threads);
    bar_init_fence();
    abort_s = 0;
  }
  __syncthreads();
  grid_dependency_sync();
  const Start st = find_run<kF32Threads, kF32KT>(p, p.mt, blockIdx.x, gridDim.x, scan_s, &start_s);
  Cursor<kF32KT> c;
  c.begin(p, p.mt, st);
  const float zscale = p.scale * kLog2e;
  if (st.n == 0 && tid == 0) p.parts[blockIdx.x] = PagedPart{};
  int tj = 0;   // tiles done: tile g of the run is in buffer g & 1, phase g >> 1
  for (bool more = st.n > 0; more;) {
    const int f0 = c.m * p.mt, nf = min(p.mt, c.s.n * p.group - f0);
    const int pos0 = c.s.len - c.s.n;
    const int first = pos0 + f0 / p.group, last = pos0 + (f0 + nf - 1) / p.group;
    // Entry f of the item -> its row and query head.
    auto entry = [&](int f) {
      const int r = (f0 + f) / p.group;
      return (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f0 + f - r * p.group);
    };
    const int T = c.x1 - c.x;
    // Thread i < 64 -> token i / 2 of a tile, its K or its V row.
    // Page of the thread's token: -1 where no row sees it, or it has no page.
    const int mine = tid >> 1, is_v = tid & 1;
    auto look_up = [&](int x) {
      if (tid >= 2 * kF32KT || x >= T) return -1;
      const int t = c.tiles.token(c.x + x) + mine;
      if (t > last || !(p.window == 0 || t > first - p.window || t < p.n_sinks)) return -1;
      int32_t page;
      if (page_of(p, c.seq, t, page)) return (int)page;
      if (!is_v) atomicAdd(&g_bad_pages, 1);
      return -1;
    };
    auto load = [&](int x, int page) {   // every thread arrives; a row that is not there becomes zeros
      const int b = (tj + x) & 1;
      if (tid < 2 * kF32KT) {
        float* dst = kv_s + b * L::kTile + (is_v ? L::kK + mine * ROWV : mine * ROW);
        const bool ok = page >= 0;
        if (ok) {
          const int64_t slot = (c.tiles.token(c.x + x) + mine) & ((1 << p.page_shift) - 1);
          const float* src = static_cast<const float*>(is_v ? p.v : p.k) + page * p.page_stride +
                             c.head * p.head_stride + slot * p.tok_stride;
          fence_async_smem();   // (zeros may have been stored there)
          bar_expect_tx(&full[b], 4 * D);
          bulk_copy(dst, src, 4 * D, &full[b]);
        } else {
          for (int i = 0; i < D / 4; ++i) reinterpret_cast<float4*>(dst)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          bar_arrive(&full[b]);
        }
        const uint32_t v = __ballot_sync(0xffffffffu, ok);   // two lanes a token, 16 tokens a warp
        uint32_t bits = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) bits |= ((v >> (2 * i)) & 1u) << i;
        if (lane == 0) seen_s[b][2 * warp] = (uint8_t)bits, seen_s[b][2 * warp + 1] = (uint8_t)(bits >> 8);
      } else {
        bar_arrive(&full[b]);
      }
    };
    fence_async_smem();   // (plain stores before the copies that follow)
    __syncthreads();      // the last item's joining is done with the tiles' place
    int page = look_up(0);
    load(0, page);
    page = look_up(1);
    // Q, eight 16-byte pieces of it a thread at a time.
    for (int i0 = tid; i0 < p.mt * (D / 4); i0 += 4 * kF32Threads) {
      float4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kF32Threads, f = i / (D / 4);
        x[k] = f < nf ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + entry(f) * D) + i % (D / 4))
                      : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * kF32Threads, f = i / (D / 4);
        if (f >= p.mt) continue;
        uint4 hi, lo;
        split_tf32(x[k].x, hi.x, lo.x);
        split_tf32(x[k].y, hi.y, lo.y);
        split_tf32(x[k].z, hi.z, lo.z);
        split_tf32(x[k].w, hi.w, lo.w);
        float* to = q_s + f * ROW + 4 * (i % (D / 4));
        *reinterpret_cast<uint4*>(to) = hi;
        *reinterpret_cast<uint4*>(to + kF32MT * ROW) = lo;
      }
    }
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // Rows gr and gr + 8 of the warp's 16 entries, and what they see.
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int pos[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) pos[h] = pos0 + (f0 + min(16 * rows16 + gr + 8 * h, nf - 1)) / p.group;
    for (int x = 0; x < T; ++x) {
      if (x + 1 < T) load(x + 1, page);
      page = look_up(x + 2);
      const int b = (tj + x) & 1;
      bar_wait(&full[b], (uint32_t)(((tj + x) >> 1) & 1), &g_f32_timeouts, &abort_s);
      if (x == 0) __syncthreads();   // Q is there
      const float* ks = kv_s + b * L::kTile + 8 * keys * ROW;   // the warp's 8 keys
      const float* vs = kv_s + b * L::kTile + L::kK + 8 * keys * ROWV;
      const uint32_t seen = seen_s[b][keys];
      const int t0 = c.tiles.token(c.x + x) + 8 * keys;
      if (seen != 0u && 16 * rows16 < nf) {
        // Logits of 16 entries x 8 keys: six sums (three products, even and odd
        // steps), so that the chains stay short.
        float z[6][4];
#pragma unroll
        for (int i = 0; i < 6; ++i) z[i][0] = z[i][1] = z[i][2] = z[i][3] = 0.f;
        // (A step's column gc is channel 2 gc, its column gc + 4 channel 2 gc + 1.)
        const float* qh = q_s + (16 * rows16 + gr) * ROW + 2 * gc;
        const float* ql = qh + kF32MT * ROW;
        const float* kk = ks + gr * ROW + 2 * gc;
        auto two = [](const float* x) { return *reinterpret_cast<const uint2*>(x); };
#pragma unroll 8
        for (int d = 0; d < D; d += 8) {
          const int e = (d >> 3) & 1;
          const uint2 h0 = two(qh + d), h1 = two(qh + 8 * ROW + d), l0 = two(ql + d), l1 = two(ql + 8 * ROW + d);
          const uint2 k = two(kk + d);
          const uint32_t ah[4] = {h0.x, h1.x, h0.y, h1.y}, al[4] = {l0.x, l1.x, l0.y, l1.y};
          uint32_t bh0, bl0, bh1, bl1;
          split_tf32(__uint_as_float(k.x), bh0, bl0);
          split_tf32(__uint_as_float(k.y), bh1, bl1);
          mma_tf32(z[3 * e], ah, bh0, bh1);
          mma_tf32(z[3 * e + 1], ah, bl0, bl1);
          mma_tf32(z[3 * e + 2], al, bh0, bh1);
        }
        // Entry (row gr + 8 h, key 2 gc + i) is s[2 h + i].
        float s[4], mx[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = i >> 1, key = 2 * gc + (i & 1);
          const float v = ((z[0][i] + z[3][i]) + ((z[1][i] + z[4][i]) + (z[2][i] + z[5][i]))) * zscale;
          s[i] = ((seen >> key) & 1u) && sees(p, pos[h], t0 + key) ? v : -INFINITY;
        }
        bool moves = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = quad_max(fmaxf(s[2 * h], s[2 * h + 1]));
          moves |= mx[h] > m[h] + kMoveMax || (m[h] == -INFINITY && mx[h] != -INFINITY);
        }
        if (__any_sync(0xffffffffu, moves)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[h], mx[h]);
            const float a = mn == -INFINITY ? 1.f : exp2f(m[h] - mn);
            m[h] = mn;
            l[h] *= a;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              o[i][2 * h] *= a;
              o[i][2 * h + 1] *= a;
            }
          }
        }
        // Weights, which are the A fragment of the output product as they lie: its
        // column gc is key 2 gc, its column gc + 4 key 2 gc + 1.
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = i >> 1;
          w[i] = m[h] == -INFINITY ? 0.f : exp2f(s[i] - m[h]);
          l[h] += w[i];
        }
        uint32_t ph[4], pl[4];
        split_tf32(w[0], ph[0], pl[0]);
        split_tf32(w[2], ph[1], pl[1]);
        split_tf32(w[1], ph[2], pl[2]);
        split_tf32(w[3], ph[3], pl[3]);
        const float* vv = vs + 2 * gc * ROWV + gr;
        constexpr int kAt = 4;   // channel blocks whose products are interleaved
#pragma unroll
        for (int i = 0; i < NT; i += kAt) {
          uint32_t bh[kAt][2], bl[kAt][2];
#pragma unroll
          for (int k = 0; k < kAt; ++k) {
            split_tf32(vv[8 * (i + k)], bh[k][0], bl[k][0]);
            split_tf32(vv[ROWV + 8 * (i + k)], bh[k][1], bl[k][1]);
          }
#pragma unroll
          for (int k = 0; k < kAt; ++k) mma_tf32(o[i + k], ph, bh[k][0], bh[k][1]);
#pragma unroll
          for (int k = 0; k < kAt; ++k) mma_tf32(o[i + k], ph, bl[k][0], bl[k][1]);
#pragma unroll
          for (int k = 0; k < kAt; ++k) mma_tf32(o[i + k], pl, bh[k][0], bh[k][1]);
        }
      }
      __syncthreads();   // the tile may be overwritten
    }
    tj += T;
    // The four warps' outputs, sums and maxima of each entry, joined in shared memory.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] = quad_sum(l[h]);
      if (gc == 0) {
        m_s[keys][16 * rows16 + gr + 8 * h] = m[h];
        l_s[keys][16 * rows16 + gr + 8 * h] = l[h];
      }
    }
    float* o_s = kv_s + warp * 16 * ROWV;   // warp 4 (f / 16) + keys: entry f
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2*>(o_s + (gr + 8 * h) * ROWV + 8 * i + 2 * gc) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
    __syncthreads();
    const bool whole = c.whole();
    const int64_t slot = whole ? 0 : (int64_t)c.slot(blockIdx.x) * p.mt;
    for (int f = warp; f < nf; f += kF32Threads / 32) {
      float M = -INFINITY, W = 0.f, e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) M = fmaxf(M, m_s[k][f]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e[k] = m_s[k][f] == -INFINITY ? 0.f : exp2f(m_s[k][f] - M);
        W = fmaf(e[k], l_s[k][f], W);
      }
      const float inv = W > 0.f ? 1.f / W : 0.f;
      const int64_t at = whole ? entry(f) : slot + f;
      for (int d = 4 * lane; d < D; d += 128) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 y = *reinterpret_cast<const float4*>(kv_s + ((4 * (f >> 4) + k) * 16 + (f & 15)) * ROWV + d);
          x.x = fmaf(e[k], y.x, x.x);
          x.y = fmaf(e[k], y.y, x.y);
          x.z = fmaf(e[k], y.z, x.z);
          x.w = fmaf(e[k], y.w, x.w);
        }
        x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        if (!whole || p.out_dtype == QSA_F32) {
          *reinterpret_cast<float4*>((whole ? static_cast<float*>(p.out) : p.part_o) + at * D + d) = x;
        } else {
          __nv_bfloat162* to = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at * D + d);
          to[0] = __floats2bfloat162_rn(x.x, x.y);
          to[1] = __floats2bfloat162_rn(x.z, x.w);
        }
      }
      if (lane == 0) {
        const float lse2 = W > 0.f ? M + log2f(W) : -INFINITY;
        if (!whole) p.part_lse[at] = lse2;
        else if (p.lse) p.lse[at] = lse2 * kLn2;
      }
    }
    const Cursor<kF32KT> done = c;
    more = c.next(p, p.mt);
    if (!more && tid == 0) describe_part(p, done, st, blockIdx.x);
  }
}

// ------------------------------------------------------------------ joining
// The items that cross runs, joined by their log-sum-exp.  An item's parts lie
// in the slots 2c + 1, 2(c + 1), 2(c + 2), ... of the run c it starts in.  A CTA
// takes units of eight warps' work from the list of all such items' entries:
// an entry of few parts is one warp's, one of many parts that of up to eight,
// which add up in shared memory in a fixed order.  (One CTA per entry of every
// run, most of them without work, took 50 us of a 2,048-row call's 255.)
constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = 32 * kJoinWarps;
constexpr int kMaxRuns = 1024;

__device__ __forceinline__ int join_warps(int n_parts) { return n_parts >= 24 ? 8 : n_parts >= 12 ? 4 : n_parts >= 6 ? 2 : 1; }

template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedParams p, int n_runs) {
  constexpr int CPL = D / 32;
  __shared__ float acc_s[kJoinWarps][D];
  __shared__ float m_s[kJoinWarps], w_s[kJoinWarps];
  __shared__ int off_s[kMaxRuns + 1];
  __shared__ int64_t scan_s[kJoinWarps];
  grid_dependency_sync();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t units = 0;
  for (int c0 = 0; c0 < n_runs; c0 += kJoinThreads) {
    int n = 0;
    if (c0 + tid < n_runs) {
      const int4 d = *reinterpret_cast<const int4*>(p.parts + c0 + tid);   // n_parts, row0, f0, nf
      if (d.x > 0) n = (d.w * join_warps(d.x) + kJoinWarps - 1) / kJoinWarps;
    }
    int64_t total;
    const int64_t before = units + cta_scan<kJoinThreads>(n, scan_s, total);
    if (c0 + tid < n_runs) off_s[c0 + tid] = (int)before;
    units += total;
  }
  if (tid == 0) off_s[n_runs] = (int)units;
  __syncthreads();
  for (int u = blockIdx.x; u < (int)units; u += gridDim.x) {
    int cta = 0, hi = n_runs;   // off_s[cta] <= u < off_s[hi]
    while (hi - cta > 1) {
      const int mid = (cta + hi) / 2;
      if (off_s[mid] <= u) cta = mid;
      else hi = mid;
    }
    const PagedPart d = p.parts[cta];
    const int w = join_warps(d.n_parts), sub = warp & (w - 1);
    const int f = (u - off_s[cta]) * (kJoinWarps / w) + warp / w;
    float m = -INFINITY, l = 0.f, acc[CPL];
#pragma unroll
    for (int i = 0; i < CPL; ++i) acc[i] = 0.f;
    constexpr int kBatch = 4;   // parts whose loads are in flight together
    for (int s0 = sub; s0 < d.n_parts && f < d.nf; s0 += w * kBatch) {
      float ls[kBatch];
      float4 v[kBatch][CPL / 4];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int s = s0 + k * w;
        const int64_t at = ((int64_t)2 * (cta + s) + (s == 0 ? 1 : 0)) * p.mt + f;
        ls[k] = s < d.n_parts ? p.part_lse[at] : -INFINITY;
#pragma unroll
        for (int i = 0; i < CPL / 4; ++i)
          v[k][i] = s < d.n_parts ? reinterpret_cast<const float4*>(p.part_o + at * D)[i * 32 + lane]
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mn = m;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) mn = fmaxf(mn, ls[k]);
      if (mn == -INFINITY) continue;
      const float a = exp2f(m - mn);
      l *= a;
#pragma unroll
      for (int i = 0; i < CPL; ++i) acc[i] *= a;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (ls[k] == -INFINITY) continue;
        const float e = exp2f(ls[k] - mn);
        l += e;
#pragma unroll
        for (int i = 0; i < CPL / 4; ++i) {
          acc[4 * i] = fmaf(e, v[k][i].x, acc[4 * i]);
          acc[4 * i + 1] = fmaf(e, v[k][i].y, acc[4 * i + 1]);
          acc[4 * i + 2] = fmaf(e, v[k][i].z, acc[4 * i + 2]);
          acc[4 * i + 3] = fmaf(e, v[k][i].w, acc[4 * i + 3]);
        }
      }
      m = mn;
    }
    if (w > 1) {   // the other warps' sums, each against the largest maximum
      __syncthreads();
#pragma unroll
      for (int i = 0; i < CPL / 4; ++i)
        reinterpret_cast<float4*>(acc_s[warp])[i * 32 + lane] =
            make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
      if (lane == 0) {
        m_s[warp] = m;
        w_s[warp] = l;
      }
      __syncthreads();
      if (sub == 0) {
        float M = m;
        for (int k = 1; k < w; ++k) M = fmaxf(M, m_s[warp + k]);
        const float own = m == -INFINITY ? 0.f : exp2f(m - M);
        l *= own;
#pragma unroll
        for (int i = 0; i < CPL; ++i) acc[i] *= own;
        for (int k = 1; k < w; ++k) {
          if (m_s[warp + k] == -INFINITY) continue;
          const float e = exp2f(m_s[warp + k] - M);
          l = fmaf(e, w_s[warp + k], l);
#pragma unroll
          for (int i = 0; i < CPL / 4; ++i) {
            const float4 x = reinterpret_cast<const float4*>(acc_s[warp + k])[i * 32 + lane];
            acc[4 * i] = fmaf(e, x.x, acc[4 * i]);
            acc[4 * i + 1] = fmaf(e, x.y, acc[4 * i + 1]);
            acc[4 * i + 2] = fmaf(e, x.z, acc[4 * i + 2]);
            acc[4 * i + 3] = fmaf(e, x.w, acc[4 * i + 3]);
          }
        }
        m = M;
      }
    }
    if (sub != 0 || f >= d.nf) continue;
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int r = (d.f0 + f) / p.group;
    const int64_t at = (int64_t)(d.row0 + r) * p.n_q_heads + d.head * p.group + (d.f0 + f - r * p.group);
#pragma unroll
    for (int i = 0; i < CPL / 4; ++i) {
      const float4 o = make_float4(acc[4 * i] * inv, acc[4 * i + 1] * inv, acc[4 * i + 2] * inv, acc[4 * i + 3] * inv);
      if (p.out_dtype == QSA_F32) {
        reinterpret_cast<float4*>(static_cast<float*>(p.out) + at * D)[i * 32 + lane] = o;
      } else {
        __nv_bfloat162* to = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at * D) + (i * 32 + lane) * 2;
        to[0] = __floats2bfloat162_rn(o.x, o.y);
        to[1] = __floats2bfloat162_rn(o.z, o.w);
      }
    }
    if (lane == 0 && p.lse) p.lse[at] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
}

template <int D>
cudaError_t launch_f32(const PagedParams& p, int grid, cudaStream_t st) {
  const size_t smem = F32Layout<D>::bytes;
  cudaError_t e = allow_dynamic_smem((const void*)paged_f32_kernel<D>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(paged_f32_kernel<D>, dim3((unsigned)grid), dim3(kF32Threads), smem, st, 0u, p);
}

}  // namespace

cudaError_t launch_paged_f32(const PagedParams& p, int head_dim, int grid, cudaStream_t st) {
  return head_dim == 256 ? launch_f32<256>(p, grid, st) : launch_f32<128>(p, grid, st);
}

cudaError_t launch_paged_merge(const PagedParams& p, int head_dim, int runs, cudaStream_t st) {
  if (runs < 2) return cudaSuccess;   // one run holds every item whole
  if (runs > kMaxRuns) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(4 * device_sm_count())), block(kJoinThreads);
  return head_dim == 256 ? launch_kernel(paged_join_kernel<256>, grid, block, 0, st, 0u, p, runs)
                         : launch_kernel(paged_join_kernel<128>, grid, block, 0, st, 0u, p, runs);
}

int paged_f32_wait_timeouts() {
  int v = 0;
  return cudaMemcpyFromSymbol(&v, g_f32_timeouts, sizeof(int)) == cudaSuccess ? v : -1;
}

int paged_bad_pages_take() { return take_counter(g_bad_pages); }

}  // namespace qsa
