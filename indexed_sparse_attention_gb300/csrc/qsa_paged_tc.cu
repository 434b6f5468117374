// Attention over a paged K/V cache on the 5th-generation tensor cores (bf16
// caches; see qsa_paged.cuh for the division of the work into runs of key
// tiles, and qsa_paged.cu for the formulas and the joining launch).
//
// An item's MT <= 128 entries (query row, head of the KV head's group) are the
// M rows of both products, 128 keys a tile:
//   S_j = Q K_j^T     tcgen05.mma, M = 128, N = 128, K = head_dim, Q and K from
//                     shared memory; two S buffers of 128 TMEM columns, so the
//                     next tile's logits are computed while this one's softmax runs;
//   P_j = exp(S_j - m), rounded to bf16, over S_j's own columns in TMEM;
//   O  += P_j V_j     M = 128, N = 64 channels a slab, K = 128 keys, P from TMEM and
//                     V from shared memory (MN-major), O in 128 or 256 TMEM columns.
// A thread owns one entry and half of the tile's keys, so row statistics need
// one exchange with the thread of the other half and no shuffles.  The running
// maximum m is only moved, and O rescaled, when a logit exceeds it by more than
// 2^8 in the weight: weights stay below 2^8, which the 32-bit sums and bf16's
// exponent hold as well as 1, and the quotient by l is the same.
//
// K and V come through TMA, 64 channels x 128 tokens (16 KB) a slab, one tensor
// copy for each page that a slab touches (pages of more than 128 tokens: one),
// into a ring of as many slabs as fit beside Q.  Copies of pages without visible
// tokens are aimed past the last page, which fills zeros without reading.
// Slots of V that belong to no visible token are cleared before the product, as
// 0 x NaN would reach O.  With fewer than 128 entries the rows behind Q's in the
// MMA read whatever lies there: rows of a product do not mix, and theirs are
// not read.
//
// Roles: warps 0-7 softmax and output (warp w: entries 32 (w % 4) .., keys 64
// (w / 4) ..; warps without entries idle), warp 8 copies K and V, warp 9
// issues the MMAs, warp 10 loads Q.  Every wait gives up after about two
// seconds (counted; the CTA then runs to its end).
#include <math.h>

#include <cudaTypedefs.h>

#include <mutex>

#include "qsa_paged.cuh"
#include "qsa_tc.cuh"

namespace qsa {

namespace {

using namespace paged;
using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKT = 128;                      // keys of a tile
constexpr int kSlab = kKT * 128;              // bytes of 64 channels of a tile
constexpr int kMaxSlabs = 14;
constexpr int kCopyWarp = 8, kMmaWarp = 9, kQWarp = 10;
constexpr int kThreads = 32 * 11;
constexpr uint32_t kTmemCols = 512, kOCol = 256;
constexpr int kSmemLimit = 227 * 1024;
constexpr float kMoveMax = 8.f;               // log2 of the weight at which the running maximum is moved

constexpr uint32_t kIdescS = idesc_bf16(128, kKT, false, false);
constexpr uint32_t kIdescO = idesc_bf16(128, 64, false, true);

__device__ int g_timeouts;
__device__ int g_bad_pages;

struct TcParams {
  CUtensorMap k, v;      // {D, page_tokens, Hkv, n_pages}, boxes of 64 channels x min(page_tokens, 128) tokens
  PagedParams p;
  int32_t n_slabs;
};

// Shared memory: this, then Q, then the ring (both on 1,024-byte boundaries).
// A wait by parity tells a phase from its neighbours only: the barriers that
// follow the tiles come in pairs, for even and odd tiles, so that a waiting
// thread knows the phase before the awaited one to be over (tile j's logits
// come after the product of tile j - 2).
struct Head {
  uint64_t full[kMaxSlabs], empty[kMaxSlabs];
  uint64_t s_full[2], p_full[2], pv_done[2], o_free, q_full, q_free, mma_done;
  int64_t scan[kThreads / 32];
  Start start;
  uint32_t tmem;
  int abort;
  uint32_t bad[8];              // 16-token pieces of a tile that have no page
  float stat[2][2][128];        // row maxima (and sums) of the two key halves
};
static_assert(sizeof(Head) <= 3072, "shared memory head");
constexpr int kHeadBytes = 3072;

__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::
          "r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

#define R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define S8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
// 64 consecutive columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, "
      "%38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, "
      "%60, %61, %62, %63}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24), R8(r, 32), R8(r, 40), R8(r, 48), R8(r, 56)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32u(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
      : "r"(taddr)
      : "memory");
}
// 32 consecutive columns, waited for.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};\n"
      "tcgen05.wait::st.sync.aligned;\n" ::S8(r, 0),
      S8(r, 8), S8(r, 16), S8(r, 24), "r"(taddr)
      : "memory");
}
#undef R8
#undef S8

// The rows of an item: entries, and the positions of its first and last row.
struct ItemRows {
  int f0, nf, pos0, first, last;   // pos0: position of the sequence's first row
};
template <int KT>
__device__ __forceinline__ ItemRows item_rows(const PagedParams& p, const Cursor<KT>& c) {
  ItemRows r;
  r.f0 = c.m * p.mt;
  r.nf = min(p.mt, c.s.n * p.group - r.f0);
  r.pos0 = c.s.len - c.s.n;
  r.first = r.pos0 + r.f0 / p.group;
  r.last = r.pos0 + (r.f0 + r.nf - 1) / p.group;
  return r;
}

// Place of tile j's K and V (T tiles in all) in an item's order of copies and
// products K0 K1 V0 K2 V1 ... V(T-1).
__device__ __forceinline__ int place_v(int j, int T) { return j < T - 1 ? 2 * j + 2 : 2 * T - 1; }

// A ring position: slab index and the parity of its use.
struct Ring {
  int slot = 0;
  uint32_t use = 0;
  __device__ __forceinline__ void step(int n) {
    if (++slot == n) {
      slot = 0;
      ++use;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_tc_kernel(const __grid_constant__ TcParams tp) {
  constexpr int NS = D / 64;   // slabs of a tile
  const PagedParams& p = tp.p;
  extern __shared__ __align__(1024) uint8_t raw[];
  Head& h = *reinterpret_cast<Head*>(raw);
  uint8_t* q_s = raw + kHeadBytes;
  const int q_slab = p.mt * 128, n_slabs = tp.n_slabs;
  uint8_t* ring = q_s + NS * q_slab;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quarters = (p.mt + 31) / 32, soft_threads = 64 * quarters;
  volatile int* abrt = &h.abort;

  if (tid == 0) {
    for (int i = 0; i < n_slabs; ++i) {
      bar_init(&h.full[i], 1);
      bar_init(&h.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&h.s_full[i], 1);
      bar_init(&h.p_full[i], soft_threads);
      bar_init(&h.pv_done[i], 1);
    }
    bar_init(&h.o_free, soft_threads);
    bar_init(&h.q_full, 1);
    bar_init(&h.q_free, 1);
    bar_init(&h.mma_done, 1);
    h.abort = 0;
    bar_init_fence();
  }
  if (warp == kMmaWarp) tmem_alloc(&h.tmem, kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = h.tmem;
  grid_dependency_wait();
  grid_dependency_release();
  const Start st = find_run<kThreads, kKT>(p, p.mt, blockIdx.x, gridDim.x, h.scan, &h.start);
  Cursor<kKT> c;
  c.begin(p, p.mt, st);

  if (st.n == 0) {
    if (tid == 0) p.parts[blockIdx.x] = PagedPart{};
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------ K and V
    const int box = min(1 << p.page_shift, kKT), n_box = kKT / box;
    Ring ring_at;
    int tj = 0;
    for (bool more = true; more; more = c.next(p, p.mt)) {
      const ItemRows ir = item_rows(p, c);
      const int T = c.x1 - c.x;
      // Lane b: the page of the tile's b-th box (n_pages: nothing to read, or no page).
      auto look_up = [&](int j, bool& missing) {
        missing = false;
        if (lane >= n_box) return p.n_pages;
        const int t = c.tiles.token(c.x + j) + lane * box;
        const int end = min(t + box - 1, ir.last);
        if (t > ir.last || !(p.window == 0 || end > ir.first - p.window || t < p.n_sinks)) return p.n_pages;
        int32_t page;
        if (page_of(p, c.seq, t, page)) return page;
        missing = true;
        return p.n_pages;
      };
      auto copy = [&](const CUtensorMap* map, int j, int page) {
        const int t = c.tiles.token(c.x + j) + lane * box;
        for (int s = 0; s < NS; ++s) {
          if (lane == 0) {
            if (ring_at.use > 0) bar_wait(&h.empty[ring_at.slot], (ring_at.use - 1) & 1, &g_timeouts, abrt);
            bar_expect_tx(&h.full[ring_at.slot], kSlab);
          }
          __syncwarp();
          if (lane < n_box)
            tma_4d(ring + ring_at.slot * kSlab + lane * box * 128, map, s * 64, t & ((1 << p.page_shift) - 1), c.head,
                   page, &h.full[ring_at.slot]);
          ring_at.step(n_slabs);
        }
      };
      bool missing;
      int now = look_up(0, missing), next = p.n_pages;
      for (int j = 0; j < T; ++j) {
        if (j == 0) {
          const uint32_t piece = missing ? ((1u << (box / 16)) - 1u) << (lane * (box / 16)) : 0u;
          const uint32_t bad = __reduce_or_sync(0xffffffffu, piece);
          if (missing) atomicAdd(&g_bad_pages, 1);
          if (lane == 0) h.bad[tj & 7] = bad;
          copy(&tp.k, 0, now);
        }
        if (j + 1 < T) {
          next = look_up(j + 1, missing);
          const uint32_t piece = missing ? ((1u << (box / 16)) - 1u) << (lane * (box / 16)) : 0u;
          const uint32_t bad = __reduce_or_sync(0xffffffffu, piece);
          if (missing) atomicAdd(&g_bad_pages, 1);
          if (lane == 0) h.bad[(tj + 1) & 7] = bad;
          copy(&tp.k, j + 1, next);
        }
        copy(&tp.v, j, now);
        now = next;
        ++tj;
      }
    }
    // Every copy has landed before the CTA ends (after a wait that gave up too).
    if (lane < n_slabs) {
      const uint32_t uses = ring_at.use + (lane < ring_at.slot ? 1u : 0u);
      if (uses > 0) bar_wait(&h.full[lane], (uses - 1) & 1, &g_timeouts);
    }
  } else if (warp == kQWarp) {
    // ------------------------------------------------------------ Q
    int it = 0;
    for (bool more = true; more; more = c.next(p, p.mt), ++it) {
      const ItemRows ir = item_rows(p, c);
      if (it > 0) bar_wait(&h.q_free, (uint32_t)((it - 1) & 1), &g_timeouts, abrt);
      constexpr int PER = D / 8;   // 16-byte pieces of an entry
      const int piece = lane % PER;
      for (int f = lane / PER; f < p.mt; f += 32 / PER) {
        const bool ok = f < ir.nf;
        const int row = (ir.f0 + f) / p.group;
        const int64_t at = ok ? (int64_t)(c.s.row0 + row) * p.n_q_heads + c.head * p.group + (ir.f0 + f - row * p.group) : 0;
        cp_async16(q_s + (piece >> 3) * q_slab + f * 128 + (((piece & 7) ^ (f & 7)) << 4),
                   static_cast<const __nv_bfloat16*>(p.q) + at * D + piece * 8, ok);
      }
      cp_async_wait_all();
      fence_async_smem();
      __syncwarp();
      if (lane == 0) bar_arrive(&h.q_full);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    if (lane == 0) {
      Ring at;
      int tj = 0, it = 0;
      for (bool more = true; more; more = c.next(p, p.mt), ++it) {
        const int T = c.x1 - c.x;
        auto logits = [&](int j) {   // S = Q K_j^T
          const uint32_t d = tmem + (uint32_t)((tj + j) & 1) * kKT;
          for (int s = 0; s < NS; ++s) {
            bar_wait(&h.full[at.slot], at.use & 1, &g_timeouts, abrt);
            fence_after();
            const uint8_t* k = ring + at.slot * kSlab;
#pragma unroll
            for (int x = 0; x < 4; ++x)
              mma_bf16(d, desc_sw128(q_s + s * q_slab + 32 * x, 16, 1024), desc_sw128(k + 32 * x, 16, 1024), kIdescS,
                       (s | x) != 0 ? 1u : 0u);
            commit(&h.empty[at.slot]);
            at.step(n_slabs);
          }
          commit(&h.s_full[(tj + j) & 1]);
          if (j == T - 1) commit(&h.q_free);
        };
        bar_wait(&h.q_full, (uint32_t)(it & 1), &g_timeouts, abrt);
        fence_after();
        logits(0);
        for (int j = 0; j < T; ++j) {
          if (j + 1 < T) logits(j + 1);
          const int buf = (tj + j) & 1;
          bar_wait(&h.p_full[buf], (uint32_t)(((tj + j) >> 1) & 1), &g_timeouts, abrt);
          if (j == 0 && it > 0) bar_wait(&h.o_free, (uint32_t)((it - 1) & 1), &g_timeouts, abrt);
          fence_after();
          for (int s = 0; s < NS; ++s) {
            bar_wait(&h.full[at.slot], at.use & 1, &g_timeouts, abrt);
            fence_after();
            const uint8_t* v = ring + at.slot * kSlab;
#pragma unroll
            for (int x = 0; x < kKT / 16; ++x)
              mma_bf16_ts(tmem + kOCol + (uint32_t)(s * 64), tmem + (uint32_t)(buf * kKT + 8 * x),
                          desc_sw128(v + x * 2048, kSlab, 1024), kIdescO, (j | x) != 0 ? 1u : 0u);
            commit(&h.empty[at.slot]);
            at.step(n_slabs);
          }
          commit(&h.pv_done[buf]);
        }
        tj += T;
      }
      commit(&h.mma_done);   // every MMA has completed before TMEM is released
      bar_wait(&h.mma_done, 0u, &g_timeouts);
    }
  } else if ((warp & 3) < quarters) {
    // ------------------------------------------------------------ softmax and output
    const int half = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    const int stid = (half * quarters + (warp & 3)) * 32 + lane;   // among the softmax threads
    const float zc = p.scale * kLog2e, move = fminf(kMoveMax / zc, 1e30f);
    int tj = 0, tiles_before = 0;   // tiles done; tiles of K and V before this item in the ring's order
    for (bool more = true; more;) {
      const ItemRows ir = item_rows(p, c);
      const int T = c.x1 - c.x;
      const bool mine = row < ir.nf;
      const int pos = ir.pos0 + (ir.f0 + min(row, ir.nf - 1)) / p.group;
      const int low = p.window > 0 ? pos - p.window + 1 : INT32_MIN;   // first token of the row's window
      const int dead = p.window > 0 ? ir.first - p.window : INT32_MIN;   // [n_sinks, dead]: no row's tokens
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < T; ++j, ++tj) {
        const int buf = tj & 1, t0 = c.tiles.token(c.x + j);
        uint32_t sr[64];
        bar_wait(&h.s_full[buf], (uint32_t)((tj >> 1) & 1), &g_timeouts, abrt);
        __syncwarp();
        fence_after();
        tmem_ld64(lanes + (uint32_t)(buf * kKT + half * 64), sr);
        const uint32_t bad = h.bad[tj & 7];
        const bool partly = bad != 0 || t0 + kKT - 1 > ir.first ||
                            (p.window > 0 && t0 <= ir.last - p.window && t0 + kKT > p.n_sinks);
        if (!mine) {
#pragma unroll
          for (int i = 0; i < 64; ++i) sr[i] = 0xff800000u;   // -infinity
        } else if (partly) {
          const int tb = t0 + half * 64;
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const int t = tb + i;
            const bool see = t <= pos && (t >= low || t < p.n_sinks) && !((bad >> (half * 4 + i / 16)) & 1u);
            sr[i] = see ? sr[i] : 0xff800000u;
          }
        }
        float mx = __uint_as_float(sr[0]);
#pragma unroll
        for (int i = 1; i < 64; ++i) mx = fmaxf(mx, __uint_as_float(sr[i]));
        h.stat[buf][half][row] = mx;
        named_sync(1, soft_threads);
        mx = fmaxf(mx, h.stat[buf][half ^ 1][row]);
        if (j == 0) {
          m = mx;
        } else {
          const bool moves = mx > m + move;   // (from -infinity too)
          if (__any_sync(0xffffffffu, moves)) {
            const float alpha = moves ? ex2((m - mx) * zc) : 1.f;
            if (moves) m = mx;
            l *= alpha;
            bar_wait(&h.pv_done[(tj - 1) & 1], (uint32_t)(((tj - 1) >> 1) & 1), &g_timeouts, abrt);
            fence_after();
            __syncwarp();
#pragma unroll 1
            for (int s = 0; s < D / 64; ++s) {   // this half's channels, 32 at a time
              uint32_t o[32];
              const uint32_t at = lanes + kOCol + (uint32_t)(half * (D / 2) + s * 32);
              tmem_ld32u(at, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(at, o);
            }
          }
        }
        // Weights: in bf16 for the product, their sum in 32 bits.
        const float shift = m == -INFINITY ? 0.f : -m * zc;
        uint32_t pr[32];
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float a = ex2(fmaf(__uint_as_float(sr[2 * i]), zc, shift));
          const float b = ex2(fmaf(__uint_as_float(sr[2 * i + 1]), zc, shift));
          s0 += a;
          s1 += b;
          pr[i] = pack_bf16(a, b);
        }
        l += s0 + s1;
        __syncwarp();
        tmem_st32(lanes + (uint32_t)(buf * kKT + half * 32), pr);
        fence_before();
        // Tokens that no row sees: their V may be anything, and P = 0 there.
        if (t0 + kKT - 1 > ir.last || (p.window > 0 && max(t0, p.n_sinks) <= min(dead, t0 + kKT - 1))) {
          const int v0 = (tiles_before + place_v(j, T)) * NS;
          for (int s = 0; s < NS; ++s) {
            const int slot = (v0 + s) % n_slabs;
            bar_wait(&h.full[slot], (uint32_t)(((v0 + s) / n_slabs) & 1), &g_timeouts, abrt);
            for (int tk = stid; tk < kKT; tk += soft_threads) {
              const int t = t0 + tk;
              if (t <= ir.last && (t > dead || t < p.n_sinks)) continue;
              uint4* v = reinterpret_cast<uint4*>(ring + slot * kSlab + tk * 128);
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          fence_async_smem();
        }
        bar_arrive(&h.p_full[buf]);
      }
      // The item's result, or this run's part of it.
      float* sums = h.stat[tj & 1][0];
      sums[half * 128 + row] = l;
      named_sync(1, soft_threads);
      l += sums[(half ^ 1) * 128 + row];
      named_sync(1, soft_threads);
      const float inv = l > 0.f ? 1.f / l : 0.f;
      const bool whole = c.whole();
      const int64_t part = (int64_t)c.slot(blockIdx.x) * p.mt + row;
      const int r = (ir.f0 + row) / p.group;
      const int64_t entry = (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (ir.f0 + row - r * p.group);
      bar_wait(&h.pv_done[(tj - 1) & 1], (uint32_t)(((tj - 1) >> 1) & 1), &g_timeouts, abrt);
      fence_after();
#pragma unroll 1
      for (int s = 0; s < D / 64; ++s) {
        uint32_t o[32];
        const int d = half * (D / 2) + s * 32;
        __syncwarp();
        tmem_ld32u(lanes + kOCol + (uint32_t)d, o);
        if (!mine) continue;
        if (!whole || p.out_dtype == QSA_F32) {
          float4* to = reinterpret_cast<float4*>((whole ? static_cast<float*>(p.out) + entry * D : p.part_o + part * D) + d);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[i] = make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
        } else {
          uint4* to = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + entry * D + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_bf16(__uint_as_float(o[8 * i + 2 * k]) * inv, __uint_as_float(o[8 * i + 2 * k + 1]) * inv);
            to[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      fence_before();
      bar_arrive(&h.o_free);
      if (mine && half == 0) {
        const float lse2 = l > 0.f ? fmaf(m, zc, log2f(l)) : -INFINITY;
        if (!whole) p.part_lse[part] = lse2;
        else if (p.lse) p.lse[entry] = lse2 * kLn2;
      }
      tiles_before += 2 * T;
      const Cursor<kKT> last = c;
      more = c.next(p, p.mt);
      if (!more && stid == 0) describe_part(p, last, st, blockIdx.x);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

bool encode_pages(CUtensorMap* map, const void* base, const PagedParams& p, int head_dim) {
  PFN_cuTensorMapEncodeTiled_v12000 f = encoder();
  if (!f) return false;
  const cuuint64_t page = (cuuint64_t)1 << p.page_shift;
  const cuuint64_t dims[4] = {(cuuint64_t)head_dim, page, (cuuint64_t)p.n_kv_heads, (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)p.tok_stride * 2, (cuuint64_t)p.head_stride * 2,
                                 (cuuint64_t)p.page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)(page < kKT ? page : kKT), 1, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_paged_tc(const PagedParams& p, int head_dim, int grid, cudaStream_t st) {
  TcParams tp{};
  tp.p = p;
  if (!encode_pages(&tp.k, p.k, p, head_dim) || !encode_pages(&tp.v, p.v, p, head_dim)) return cudaErrorInvalidValue;
  const int q_bytes = p.mt * head_dim * 2;
  const int slabs = (kSmemLimit - kHeadBytes - q_bytes) / kSlab;
  tp.n_slabs = slabs < kMaxSlabs ? slabs : kMaxSlabs;
  const size_t smem = (size_t)kHeadBytes + q_bytes + (size_t)tp.n_slabs * kSlab;
  const void* kernel = head_dim == 256 ? (const void*)paged_tc_kernel<256> : (const void*)paged_tc_kernel<128>;
  cudaError_t e = allow_dynamic_smem(kernel, kSmemLimit);
  if (e != cudaSuccess) return e;
  return head_dim == 256
             ? launch_kernel(paged_tc_kernel<256>, dim3((unsigned)grid), dim3(kThreads), smem, st, 0u, tp)
             : launch_kernel(paged_tc_kernel<128>, dim3((unsigned)grid), dim3(kThreads), smem, st, 0u, tp);
}

int paged_tc_bad_pages_take() { return take_counter(g_bad_pages); }

int paged_tc_wait_timeouts() {
  int v = 0;
  return cudaMemcpyFromSymbol(&v, g_timeouts, sizeof(int)) == cudaSuccess ? v : -1;
}

}  // namespace qsa
