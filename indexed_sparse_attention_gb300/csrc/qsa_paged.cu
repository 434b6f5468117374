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
// (A windowed batch of five sequences, 1 to 37 rows, head_dim 256: 56 us, of which
// the three tf32 products are 22 at the rate of mma.sync, and the start, the waits
// for the next call and the joining launch about 12; the rest is the splitting and the exchange of
// partial logits between two barriers a tile.)
//
// Products of f32 values on the tensor pipe, by tf32 halves: x = hi + lo with hi
// = x rounded to 11 significant bits and lo = x - hi cut off after as many, and
//   a b = hi_a hi_b + hi_a lo_b + lo_a hi_b  (+ lo_a lo_b, at most 2^-22 |a b|, left out).
// The tensor pipe cuts its 32-bit sums off instead of rounding them, so few are
// taken on one accumulator: a tile's sums are added to the running ones in plain
// 32-bit arithmetic.  (With the running ones as accumulators, outputs were 2.8e-6
// off 64 bits on a windowed batch where plain 32-bit sums are 1.5e-6 off.)
//
// An item is 16 or 32 entries (RT = one or two times the rows of m16n8k8), a key
// tile 32 tokens.  Warp w of eight takes the channels [w D / 8, (w + 1) D / 8) of
// both products: it holds its channels of Q in registers and reads
// each K and V value once, where a split by keys had every warp read all of Q
// (the shared memory's bandwidth was the bound then).  Per tile:
//   the warps' partial logits over their channels, to shared memory;
//   their sums, masks, maxima and weights, a thread four keys of one entry;
//   the output product of the weights with the warp's channels of V.
// Warp 8 copies: each row of K and V is one bulk copy.  Rows in shared memory are
// padded, K's by eight words and V's by four, which puts the eight rows and four
// column pairs (K), or four row pairs and eight columns (V), of a fragment into
// different banks.
constexpr int kF32Warps = 8;                       // without the copying one
constexpr int kF32Threads = 32 * (kF32Warps + 1);
constexpr int kF32KT = 32;
constexpr int kF32MaxStages = 4;

template <int D, int RT>
struct F32Layout {
  static constexpr int kRow = D + 8, kRowV = D + 4;        // words of a row of K, and of V
  static constexpr int kK = kF32KT * kRow, kTile = kK + kF32KT * kRowV;   // words of K, and of K and V, of a tile
  static constexpr int kStages = D == 256 ? 2 : 4;
  static constexpr int kSRow = kF32KT + 4, kPRow = kF32KT + 8;   // rows of partial logits, and of weights
  static constexpr int kS = kF32Warps * 16 * RT * kSRow, kP = 2 * 16 * RT * kPRow;
  static constexpr size_t bytes = 4 * (size_t)(kStages * kTile + kS + kP);
  static_assert((4 * kRow) % 16 == 0 && (4 * kRowV) % 16 == 0 && (4 * kK) % 16 == 0 && (4 * kTile) % 16 == 0 &&
                    (4 * kS) % 16 == 0, "rows on 16-byte boundaries");
};

// The halves of x.  Adding half a unit of the 11th significant bit to the pattern
// and clearing the 13 bits below rounds to nearest (halves away from zero); of lo
// the tensor pipe ignores those bits itself, at most 2^-22 |x|.  (In plain integer
// operations: the conversion instruction took most of the kernel's time.)  Patterns
// whose rounding would reach infinity, or past the NaNs the other sign, are taken as
// the largest one below: hi is always finite, and what is infinite or no number in x
// is so in lo, hence in two of the three products and never in opposite signs.  (The
// two minima cost 2 us of 54.  Rounding lo as well, which needs a third: 58 us, and
// the same error against 64 bits, 1.4e-7 in the root mean square of that batch.)
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = (min((uint32_t)min(__float_as_int(x), 0x7f7fefff), 0xff7fefffu) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(32 * kF32Warps) : "memory"); }

template <int D, int RT>
__global__ void __launch_bounds__(kF32Threads, 1) paged_f32_kernel(const PagedParams p) {
  using L = F32Layout<D, RT>;
  constexpr int ROW = L::kRow, ROWV = L::kRowV, ST = L::kStages;
  constexpr int C = D / kF32Warps;          // channels of a warp
  constexpr int KS = C / 8, NT = C / 8;     // steps of the logits' product, channel blocks of the output's
  constexpr float kMoveMax = 8.f;           // as in the bf16 kernel: the maximum moves when a weight would pass 2^8
  extern __shared__ __align__(16) float fsm[];
  float* kv_s = fsm;                        // stages of [K 32][ROW], [V 32][ROWV]
  float* s_s = kv_s + ST * L::kTile;        // [8 warps][16 RT entries][kSRow]
  float* p_s = s_s + L::kS;                 // weights: hi [16 RT][kPRow], then lo
  __shared__ int64_t scan_s[kF32Threads / 32];
  __shared__ Start start_s;
  __shared__ uint64_t full[ST], empty[ST];
  __shared__ int abort_s;
  __shared__ uint32_t seen_s[2 * kF32MaxStages];   // tokens of a tile that some row sees and that have a page
  __shared__ float a_s[16 * RT], l_s[16 * RT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      bar_init(&full[i], 32);
      bar_init(&empty[i], kF32Warps);
    }
    bar_init_fence();
    abort_s = 0;
  }
  __syncthreads();
  grid_dependency_sync();
  const Start st = find_run<kF32Threads, kF32KT>(p, p.mt, blockIdx.x, gridDim.x, scan_s, &start_s);
  Cursor<kF32KT> c;
  c.begin(p, p.mt, st);
  if (st.n == 0) {
    if (tid == 0) p.parts[blockIdx.x] = PagedPart{};
    return;
  }

  if (warp == kF32Warps) {
    // ------------------------------------------------------------ copies
    // Lane i: token i's rows; a row that is not there becomes zeros.
    int g = 0;
    bool live = true;
    for (bool more = true; more && live; more = c.next(p, p.mt)) {
      const int f0 = c.m * p.mt, nf = min(p.mt, c.s.n * p.group - f0), pos0 = c.s.len - c.s.n;
      const int first = pos0 + row_of(p, f0), last = pos0 + row_of(p, f0 + nf - 1);
      const int T = c.x1 - c.x;
      auto look_up = [&](int x) {   // page of the lane's token: -1 where no row sees it, or it has none
        const int t = c.tiles.token(c.x + x) + lane;
        if (x >= T || t > last || !(p.window == 0 || t > first - p.window || t < p.n_sinks)) return -1;
        int32_t page;
        if (page_of(p, c.seq, t, page)) return (int)page;
        atomicAdd(&g_bad_pages, 1);
        return -1;
      };
      int page = look_up(0);
      for (int x = 0; x < T; ++x, ++g) {
        const int next = look_up(x + 1);
        const int b = g % ST;
        live = g < ST || bar_wait(&empty[b], (uint32_t)((g / ST - 1) & 1), &g_f32_timeouts, &abort_s);
        live = __all_sync(0xffffffffu, live);
        if (!live) break;
        float* dst = kv_s + b * L::kTile;
        const bool ok = page >= 0;
        const uint32_t seen = __ballot_sync(0xffffffffu, ok);
        if (lane == 0) seen_s[g & (2 * kF32MaxStages - 1)] = seen;
        __syncwarp();
        if (ok) {
          const int64_t slot = (c.tiles.token(c.x + x) + lane) & ((1 << p.page_shift) - 1);
          const int64_t off = page * p.page_stride + c.head * p.head_stride + slot * p.tok_stride;
          fence_async_smem();   // (zeros may have been stored there)
          bar_expect_tx(&full[b], 8 * D);
          bulk_copy(dst + lane * ROW, static_cast<const float*>(p.k) + off, 4 * D, &full[b]);
          bulk_copy(dst + L::kK + lane * ROWV, static_cast<const float*>(p.v) + off, 4 * D, &full[b]);
        } else {
          for (int i = 0; i < D / 4; ++i) {
            reinterpret_cast<float4*>(dst + lane * ROW)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            reinterpret_cast<float4*>(dst + L::kK + lane * ROWV)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          bar_arrive(&full[b]);
        }
        page = next;
      }
    }
    // Every copy has landed before the CTA ends.
    for (int i = max(g - ST, 0); i < g; ++i) bar_wait(&full[i % ST], (uint32_t)((i / ST) & 1), &g_f32_timeouts);
    return;
  }

  // -------------------------------------------------------------- products
  const int gr = lane >> 2, gc = lane & 3;   // a fragment's row group and column
  const float zscale = p.scale * kLog2e;
  // The entry and four keys whose logits this thread sums (with RT = 1: half the threads).
  const int row = tid >> 3, key0 = 4 * (tid & 7);
  int g = 0;
  for (bool more = true; more;) {
    const int f0 = c.m * p.mt, nf = min(p.mt, c.s.n * p.group - f0);
    const int pos0 = c.s.len - c.s.n;
    const int first = pos0 + row_of(p, f0), last = pos0 + row_of(p, f0 + nf - 1);
    // Entry f of the item -> its row and query head.
    auto entry = [&](int f) {
      const int r = row_of(p, f0 + f);
      return (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f0 + f - r * p.group);
    };
    const int T = c.x1 - c.x;
    // The warp's channels of Q: a step's column gc is channel 2 gc, its column
    // gc + 4 channel 2 gc + 1.
    float q_r[RT][KS][4];   // (split where it is used: both halves would not fit the registers)
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = 16 * r + gr + 8 * h;
        const float* q = static_cast<const float*>(p.q) + (f < nf ? entry(f) : 0) * D + warp * C + 2 * gc;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const float2 x = f < nf ? __ldg(reinterpret_cast<const float2*>(q + 8 * k)) : make_float2(0.f, 0.f);
          q_r[r][k][h] = x.x;
          q_r[r][k][h + 2] = x.y;
        }
      }
    float o[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < NT; ++i) o[r][i][0] = o[r][i][1] = o[r][i][2] = o[r][i][3] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int pos = pos0 + row_of(p, f0 + min(row, nf - 1));
    for (int x = 0; x < T; ++x, ++g) {
      const int b = g % ST;
      bar_wait(&full[b], (uint32_t)((g / ST) & 1), &g_f32_timeouts, &abort_s);
      const float* ks = kv_s + b * L::kTile + gr * ROW + warp * C + 2 * gc;
      const float* vs = kv_s + b * L::kTile + L::kK + 2 * gc * ROWV + warp * C + gr;
      float* to = s_s + (warp * 16 * RT + gr) * L::kSRow + 2 * gc;
      {
        float z[RT][4][4];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int n = 0; n < 4; ++n) z[r][n][0] = z[r][n][1] = z[r][n][2] = z[r][n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t bh[4][2], bl[4][2];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float2 y = *reinterpret_cast<const float2*>(ks + 8 * n * ROW + 8 * k);
            split_tf32(y.x, bh[n][0], bl[n][0]);
            split_tf32(y.y, bh[n][1], bl[n][1]);
          }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            uint32_t qh[4], ql[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float q = q_r[r][k][i];
              asm volatile("" : "+f"(q));   // (else the halves are computed once and spilled)
              split_tf32(q, qh[i], ql[i]);
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) mma_tf32(z[r][n], qh, bl[n][0], bl[n][1]);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma_tf32(z[r][n], ql, bh[n][0], bh[n][1]);
#pragma unroll
            for (int n = 0; n < 4; ++n) mma_tf32(z[r][n], qh, bh[n][0], bh[n][1]);
          }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              *reinterpret_cast<float2*>(to + (16 * r + 8 * h) * L::kSRow + 8 * n) =
                  make_float2(z[r][n][2 * h], z[r][n][2 * h + 1]);
      }
      compute_sync();
      if (row < 16 * RT) {
        float4 y[kF32Warps];
#pragma unroll
        for (int w = 0; w < kF32Warps; ++w)
          y[w] = *reinterpret_cast<const float4*>(s_s + (w * 16 * RT + row) * L::kSRow + key0);
#pragma unroll
        for (int d = kF32Warps / 2; d > 0; d >>= 1)
#pragma unroll
          for (int w = 0; w < d; ++w)
            y[w] = make_float4(y[w].x + y[w + d].x, y[w].y + y[w + d].y, y[w].z + y[w + d].z, y[w].w + y[w + d].w);
        const uint32_t seen = seen_s[g & (2 * kF32MaxStages - 1)];
        const int t0 = c.tiles.token(c.x + x);
        float v[4] = {y[0].x * zscale, y[0].y * zscale, y[0].z * zscale, y[0].w * zscale};
        if (seen != 0xffffffffu || t0 + kF32KT - 1 > first || (p.window > 0 && t0 <= last - p.window)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((seen >> (key0 + i)) & 1u) || !sees(p, pos, t0 + key0 + i)) v[i] = -INFINITY;
        }
        float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = mx > m + kMoveMax || m == -INFINITY ? mx : m;
        const float a = mn == m ? 1.f : ex2(m - mn);
        const float shift = mn == -INFINITY ? 0.f : mn;
        m = mn;
        l *= a;
        if ((tid & 7) == 0) a_s[row] = a;
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w = ex2(v[i] - shift);
          l += w;
          split_tf32(w, hi[i], lo[i]);
        }
        *reinterpret_cast<uint4*>(p_s + row * L::kPRow + key0) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(p_s + (16 * RT + row) * L::kPRow + key0) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      compute_sync();
      // A step is eight keys: its column gc key 2 gc, its column gc + 4 key 2 gc + 1.
      float t[RT][NT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) t[r][n][0] = t[r][n][1] = t[r][n][2] = t[r][n][3] = 0.f;
#pragma unroll 2
      for (int k = 0; k < kF32KT / 8; ++k) {
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          split_tf32(vs[8 * k * ROWV + 8 * n], bh[n][0], bl[n][0]);
          split_tf32(vs[(8 * k + 1) * ROWV + 8 * n], bh[n][1], bl[n][1]);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          auto two = [&](int half, int f) {
            return *reinterpret_cast<const uint2*>(p_s + (16 * RT * half + 16 * r + f) * L::kPRow + 8 * k + 2 * gc);
          };
          const uint2 h0 = two(0, gr), h1 = two(0, gr + 8), l0 = two(1, gr), l1 = two(1, gr + 8);
          const uint32_t ph[4] = {h0.x, h1.x, h0.y, h1.y}, pl[4] = {l0.x, l1.x, l0.y, l1.y};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_tf32(t[r][n], ph, bl[n][0], bl[n][1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_tf32(t[r][n], pl, bh[n][0], bh[n][1]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_tf32(t[r][n], ph, bh[n][0], bh[n][1]);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float a0 = a_s[16 * r + gr], a1 = a_s[16 * r + gr + 8];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[r][n][i] = fmaf(o[r][n][i], i < 2 ? a0 : a1, t[r][n][i]);
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&empty[b]);
    }
    // The item's result, or this run's part of it.
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    const bool whole = c.whole();
    const int64_t slot = whole ? 0 : (int64_t)c.slot(blockIdx.x) * p.mt;
    if ((tid & 7) == 0 && row < nf) {
      l_s[row] = l == 0.f ? 0.f : 1.f / l;
      const float lse2 = l == 0.f ? -INFINITY : m + log2f(l);   // (a row of NaN keeps it)
      if (!whole) p.part_lse[slot + row] = lse2;
      else if (p.lse) p.lse[entry(row)] = lse2 * kLn2;
    }
    compute_sync();
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int f = 16 * r + gr + 8 * h;
        if (f >= nf) continue;
        const float inv = l_s[f];
        const int64_t at = (whole ? entry(f) : slot + f) * D + warp * C + 2 * gc;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const float x0 = o[r][i][2 * h] * inv, x1 = o[r][i][2 * h + 1] * inv;
          if (!whole || p.out_dtype == QSA_F32)
            *reinterpret_cast<float2*>((whole ? static_cast<float*>(p.out) : p.part_o) + at + 8 * i) = make_float2(x0, x1);
          else
            *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at + 8 * i) =
                __floats2bfloat162_rn(x0, x1);
        }
      }
    const Cursor<kF32KT> done = c;
    more = c.next(p, p.mt);
    if (!more && tid == 0) describe_part(p, done, st, blockIdx.x);
    compute_sync();   // l_s has been read
  }
}

// ------------------------------------------------------------------ joining
// The items that cross runs, joined by their log-sum-exp.  An item's parts lie
// in the slots 2c + 1, 2(c + 1), 2(c + 2), ... of the run c it starts in.  A CTA
// takes units of 16 warps' work from the list of all such items' entries and
// blocks of 128 channels: one of few parts is one warp's, one of many parts that
// of up to 16, which add up in shared memory in a fixed order.  The launch is a
// chain of latencies, so a warp has up to six parts in flight and 16 warps
// cover the parts of a call of one sequence at once.  (One CTA per entry of
// every run, most of them without work, took 50 us of a 2,048-row call's 255.)
constexpr int kJoinWarps = 16;
constexpr int kJoinThreads = 32 * kJoinWarps;
constexpr int kJoinBatch = 6;   // parts whose loads are in flight together
constexpr int kMaxRuns = 1024;

// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ int join_warps_log2(int n_parts) {
  return n_parts > 64 ? 4 : n_parts > 32 ? 3 : n_parts > 16 ? 2 : n_parts > 8 ? 1 : 0;
}
// Entries (and blocks) of an item of n_parts parts that a warp takes at a time.
template <bool MANY>
__device__ __forceinline__ int join_entries(int n_parts) {
  return !MANY || n_parts > 4 ? 1 : n_parts > 2 ? 2 : 4;
}
template <bool MANY>
__device__ __forceinline__ int join_units(int n_parts, int n) {   // of n entries and blocks
  const int per = kJoinWarps * join_entries<MANY>(n_parts);
  return ((n << join_warps_log2(n_parts)) + per - 1) / per;
}

// Writes four channels of a joined entry f of the item, by lane-wide position at_c.
template <int D>
__device__ __forceinline__ void join_write(const PagedParams& p, const PagedPart& d, int f, int at_c, bool first, float m,
                                           float l, float4 acc) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int r = row_of(p, d.f0 + f);
  const int64_t at = (int64_t)(d.row0 + r) * p.n_q_heads + (d.nf_head >> 8) * p.group + (d.f0 + f - r * p.group);
  const float4 o = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  if (p.out_dtype == QSA_F32) {
    reinterpret_cast<float4*>(static_cast<float*>(p.out) + at * D)[at_c] = o;
  } else {
    __nv_bfloat162* to = reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at * D) + at_c * 2;
    to[0] = __floats2bfloat162_rn(o.x, o.y);
    to[1] = __floats2bfloat162_rn(o.z, o.w);
  }
  if (first && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// E entries (and blocks) of at most P parts, from k0 on, by one warp: all their
// loads are in flight together.  (One entry at a time, a call of 2,048 rows over
// a window spent 14 us here, 8 dependent rounds a warp.)
template <int D, int P, int E>
__device__ __forceinline__ void join_few(const PagedParams& p, const PagedPart& d, int cta, int k0) {
  constexpr int CB = D / 128;
  const int lane = (int)threadIdx.x & 31, nf = d.nf_head & 255;
  float ls[E * P];
  float4 v[E * P];
#pragma unroll
  for (int i = 0; i < E * P; ++i) {
    const int k = k0 + i / P, f = k / CB, s = i % P;
    const bool there = f < nf && s < d.n_parts;
    const int at = (2 * (cta + s) + (s == 0 ? 1 : 0)) * p.mt + f;   // (at most 2^18, the float4 below 2^24)
    ls[i] = there ? p.part_lse[at] : -INFINITY;
    v[i] = there ? reinterpret_cast<const float4*>(p.part_o)[at * (D / 4) + k % CB * 32 + lane]
                 : make_float4(0.f, 0.f, 0.f, 0.f);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int k = k0 + e, f = k / CB;
    if (f >= nf) break;
    float m = ls[e * P];
#pragma unroll
    for (int s = 1; s < P; ++s) m = max_nan(m, ls[e * P + s]);
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < P; ++s) {
      const float w = ls[e * P + s] == -INFINITY ? 0.f : ex2(ls[e * P + s] - m);
      const float4 x = v[e * P + s];
      l += w;
      acc = make_float4(fmaf(w, x.x, acc.x), fmaf(w, x.y, acc.y), fmaf(w, x.z, acc.z), fmaf(w, x.w, acc.w));
    }
    join_write<D>(p, d, f, k % CB * 32 + lane, lane == 0 && k % CB == 0, m, l, acc);
  }
}

// MANY: calls whose items have many entries, of few parts each (chunks of rows).
template <int D, bool MANY>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedParams p, int n_runs) {
  constexpr int CB = D / 128;
  __shared__ float4 acc_s[kJoinWarps][32];
  __shared__ float m_s[kJoinWarps], l_s[kJoinWarps];
  __shared__ int off_s[kMaxRuns + 1], sums_s[kJoinWarps], first_s;
  grid_dependency_sync();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int units = 0;   // (an item has at most 128 entries)
  for (int c0 = 0; c0 < n_runs; c0 += kJoinThreads) {
    int n = 0;
    if (c0 + tid < n_runs) {
      const int4 d = *reinterpret_cast<const int4*>(p.parts + c0 + tid);
      if (d.x > 0) n = join_units<MANY>(d.x, (d.w & 255) * CB);
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += up;
    }
    if (c0 > 0) __syncthreads();
    if (lane == 31) sums_s[warp] = inc;
    __syncthreads();
    int before = units + inc - n;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const int x = sums_s[w];
      if (w < warp) before += x;
      units += x;
    }
    if (c0 + tid < n_runs) off_s[c0 + tid] = before;
    if ((int)blockIdx.x >= before && (int)blockIdx.x < before + n) first_s = c0 + tid;   // the run of this CTA's first unit
  }
  if (tid == 0) off_s[n_runs] = units;
  __syncthreads();
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    int cta = first_s;
    if (u != (int)blockIdx.x) {
      int hi = n_runs;   // off_s[cta] <= u < off_s[hi]
      cta = 0;
      while (hi - cta > 1) {
        const int mid = (cta + hi) / 2;
        if (off_s[mid] <= u) cta = mid;
        else hi = mid;
      }
    }
    const PagedPart d = p.parts[cta];
    const int nf = d.nf_head & 255, lw = join_warps_log2(d.n_parts), w = 1 << lw, sub = warp & (w - 1);
    if (MANY && d.n_parts <= 4) {
      const int k0 = ((u - off_s[cta]) * kJoinWarps + warp) * join_entries<MANY>(d.n_parts);
      if (d.n_parts <= 2) join_few<D, 2, 4>(p, d, cta, k0);
      else join_few<D, 4, 2>(p, d, cta, k0);
      continue;
    }
    const int k = ((u - off_s[cta]) * kJoinWarps + warp) >> lw, f = k / CB, at_c = k % CB * 32 + lane;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = sub; s0 < d.n_parts && f < nf; s0 += w * kJoinBatch) {
      float ls[kJoinBatch];
      float4 v[kJoinBatch];
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) {
        const int s = s0 + i * w;
        const int at = (2 * (cta + s) + (s == 0 ? 1 : 0)) * p.mt + f;
        ls[i] = s < d.n_parts ? p.part_lse[at] : -INFINITY;
        v[i] = s < d.n_parts ? reinterpret_cast<const float4*>(p.part_o)[at * (D / 4) + at_c]
                             : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float mn = m;
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) mn = max_nan(mn, ls[i]);
      if (mn == -INFINITY) continue;   // (parts without a visible token are all zeros)
      const float a = ex2(m - mn);
      l *= a;
      acc = make_float4(acc.x * a, acc.y * a, acc.z * a, acc.w * a);
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) {
        const float e = ex2(ls[i] - mn);
        l += e;
        acc = make_float4(fmaf(e, v[i].x, acc.x), fmaf(e, v[i].y, acc.y), fmaf(e, v[i].z, acc.z), fmaf(e, v[i].w, acc.w));
      }
      m = mn;
    }
    if (w > 1) {   // the other warps' sums, each against the largest maximum
      __syncthreads();
      acc_s[warp][lane] = acc;
      if (lane == 0) {
        m_s[warp] = m;
        l_s[warp] = l;
      }
      __syncthreads();
      if (sub == 0 && f < nf) {
        const float mi = lane < w ? m_s[warp + lane] : -INFINITY, li = lane < w ? l_s[warp + lane] : 0.f;
        m = mi;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float e = mi == -INFINITY ? 0.f : ex2(mi - m);
        l = e * li;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < w; ++i) {
          const float ei = __shfl_sync(0xffffffffu, e, i);
          const float4 x = acc_s[warp + i][lane];
          acc = make_float4(fmaf(ei, x.x, acc.x), fmaf(ei, x.y, acc.y), fmaf(ei, x.z, acc.z), fmaf(ei, x.w, acc.w));
        }
      }
    }
    if (sub == 0 && f < nf) join_write<D>(p, d, f, at_c, lane == 0 && k % CB == 0, m, l, acc);
  }
}

template <int D, int RT>
cudaError_t launch_f32(const PagedParams& p, int grid, cudaStream_t st) {
  const size_t smem = F32Layout<D, RT>::bytes;
  cudaError_t e = allow_dynamic_smem((const void*)paged_f32_kernel<D, RT>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(paged_f32_kernel<D, RT>, dim3((unsigned)grid), dim3(kF32Threads), smem, st, 0u, p);
}

}  // namespace

cudaError_t launch_paged_f32(const PagedParams& p, int head_dim, int grid, cudaStream_t st) {
  if (p.mt == 16) return head_dim == 256 ? launch_f32<256, 1>(p, grid, st) : launch_f32<128, 1>(p, grid, st);
  return head_dim == 256 ? launch_f32<256, 2>(p, grid, st) : launch_f32<128, 2>(p, grid, st);
}

cudaError_t launch_paged_merge(const PagedParams& p, int head_dim, int runs, cudaStream_t st) {
  if (runs < 2) return cudaSuccess;   // one run holds every item whole
  if (runs > kMaxRuns) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(2 * device_sm_count())), block(kJoinThreads);
  if (p.mt > 64)
    return head_dim == 256 ? launch_kernel(paged_join_kernel<256, true>, grid, block, 0, st, 0u, p, runs)
                           : launch_kernel(paged_join_kernel<128, true>, grid, block, 0, st, 0u, p, runs);
  return head_dim == 256 ? launch_kernel(paged_join_kernel<256, false>, grid, block, 0, st, 0u, p, runs)
                         : launch_kernel(paged_join_kernel<128, false>, grid, block, 0, st, 0u, p, runs);
}

int paged_f32_wait_timeouts() {
  int v = 0;
  return cudaMemcpyFromSymbol(&v, g_f32_timeouts, sizeof(int)) == cudaSuccess ? v : -1;
}

int paged_bad_pages_take() { return take_counter(g_bad_pages); }

}  // namespace qsa
