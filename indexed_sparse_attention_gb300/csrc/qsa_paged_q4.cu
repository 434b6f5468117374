// Attention over a paged K/V cache held in 4 bits (QSA_Q4_1: blocks of 32 channels,
// value = code * scale + minimum; see include/qsa.h for the layout, qsa_paged.cuh for
// the division of the work into runs of key tiles, and qsa_paged.cu for the joining
// launch).
//
// An item's 16 entries (query row, head of the KV head's group) are the M rows of
// mma.sync.m16n8k16 f16 products; a tile is 128 keys, 16 for each of eight warps.  A
// warp works through its keys by itself -- logits, softmax with statistics of its
// own, output -- so nothing is exchanged until an item ends, when the eight parts
// are joined through shared memory.
//
// Codes enter the products as they are: a nibble in bits 0-3 (4-7) of a half is the
// f16 subnormal code * 2^-24 (2^-20), exactly, so unpacking is masks only (5 for 8
// values) and no conversion.
//   logits   z_t = sum_g s_tg (sum_c q_c code_tc) + sum_g m_tg (sum_c q_c): the inner
//            sum is a product of two k-steps a block, 32-bit, scaled in 32 bits; the
//            second is one more product, of the block sums of q as two f16 halves
//            against the minima.  q times a power of two that brings its row's
//            largest magnitude to [2^8, 2^9) is exact in f16 from 2^-25 of that on
//            and off by at most 2^-33 of it below, so the logits are those of the
//            stored values.
//   output   sum_t w_t v_t = sum_t (w_t s_tg) code_tc + sum_t w_t m_tg: w_t and
//            f16(w_t s_tg) are f16 (two roundings of 2^-12 a weight); weights are kept
//            relative to a maximum so that 2^6 is the largest, lagging by up to 2^4,
//            and to scales above 2^5 (with |s| < 65504 nothing overflows), so that a
//            weight is exact to 2^-31 of the largest.
//
// K, V and their records come through TMA, 40 KB (head_dim 256) a tile, into a ring
// of as many tiles as fit; boxes of pages without visible tokens are aimed past the
// last page, which fills zeros without reading.  Every wait gives up after about two
// seconds (counted; nothing more is issued then, and the CTA runs to its end).
#include <cuda_fp16.h>
#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <mutex>

#include "qsa_paged.cuh"
#include "qsa_tc.cuh"

namespace qsa {

namespace {

using namespace paged;
using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKT = 128;                 // keys of a tile
constexpr int kWarps = 8;                // that compute
constexpr int kThreads = 32 * (kWarps + 4);   // three warpgroups: two that compute, one whose first warp copies
// Registers of a thread: 168 at launch (384 threads share 64,512), of which the
// copying warpgroup leaves 128 each to the others: 256 * 232 + 128 * 40 = 64,512.
constexpr int kRegsCompute = 232, kRegsCopy = 40;
constexpr int kMT = 16;                  // entries of an item
constexpr int kMaxSlots = 10;
constexpr int kSmemLimit = 227 * 1024;
constexpr float kTop = 3.f;              // log2 of the largest weight when the maximum is up to date
constexpr float kLag = 7.f;              // log2 of what a weight may pass it by
constexpr float kScaleTop = 5.f;         // log2 of the scales that this leaves room for

__device__ int g_timeouts;
__device__ int g_bad_pages;

struct Q4Params {
  CUtensorMap k, v, r;   // {bytes of a row or record, page_tokens, Hkv, n_pages}: boxes of min(page_tokens, 128) tokens
  PagedParams p;
  int32_t n_slots;
};

struct Head {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  int64_t scan[16];
  Start start;
  int abort;
  uint32_t bad[16];          // 16-token pieces of a tile that have no page
  float m[kWarps][kMT], l[kWarps][kMT];
};
constexpr int kHeadBytes = 2 * 1024;
static_assert(sizeof(Head) <= kHeadBytes, "shared memory head");

template <int D>
struct Layout {
  static constexpr int G = D / 32;                 // blocks of a row
  static constexpr int kRow = D / 2, kRecord = D / 4;
  static constexpr int kCodes = kKT * kRow, kSlot = 2 * kCodes + kKT * kRecord;
  // Joining: two blocks' channels of the 16 rows, rows 4 floats apart in banks.
  static constexpr int kPitch = 68, kJoin = kWarps * kMT * kPitch * 4;
  static constexpr bool kQShared = D == 256;       // Q's fragments in shared memory (registers are short)
  static constexpr int kQ = kQShared ? 2 * G * 512 : 0;
  static constexpr int kFixed = kHeadBytes + kQ + kJoin;
};

__device__ __forceinline__ bool wait_slow(uint64_t* b, uint32_t parity, int* abort) {
  return bar_wait(b, parity, &g_timeouts, abort);
}
__device__ __forceinline__ bool wait(uint64_t* b, uint32_t parity, int* abort) {
  return bar_try(b, parity) || wait_slow(b, parity, abort);
}
__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n" ::
          "r"(dst),
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
__device__ __forceinline__ uint4 lds128(const uint8_t* at) { return *reinterpret_cast<const uint4*>(at); }
__device__ __forceinline__ uint2 lds64(const uint8_t* at) { return *reinterpret_cast<const uint2*>(at); }
__device__ __forceinline__ uint32_t lds32(const uint8_t* at) { return *reinterpret_cast<const uint32_t*>(at); }
// c += a b, and c = a b.  (Not volatile: products of registers, which may be moved past
// each other.)
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// acc += f * d, two binary32 values at once.
__device__ __forceinline__ void fma2(float& a0, float& a1, float f0, float f1, float d0, float d1) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%0, %1};\n"
      " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(f0), "f"(f1), "f"(d0), "f"(d1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float low_half(uint32_t w) { return __low2float(*reinterpret_cast<const __half2*>(&w)); }

struct ItemRows {
  int f0, nf, pos0, first, last;
};
__device__ __forceinline__ ItemRows item_rows(const PagedParams& p, const Cursor<kKT>& c) {
  ItemRows r;
  r.f0 = c.m * kMT;
  r.nf = min(kMT, c.s.n * p.group - r.f0);
  r.pos0 = c.s.len - c.s.n;
  r.first = r.pos0 + row_of(p, r.f0);
  r.last = r.pos0 + row_of(p, r.f0 + r.nf - 1);
  return r;
}

// A row of 16 keys at tile column n of either half: the order that spreads the rows
// which one load of a warp touches over all banks (K: columns 2 i and 2 i + 1
// differ in the lowest bit; V and the records: columns 0, 2, 4, 6, and 1, 3, 5, 7,
// are two rows of each parity, two apart).
__device__ __forceinline__ int key_of(int n) { return n ^ ((n >> 1) & 1); }

// Byte offsets within a tile under TMA's swizzles: 16-byte chunk c of row r.
template <int BYTES>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  if constexpr (BYTES == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
  else if constexpr (BYTES == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  else return (uint32_t)(r * 32 + ((c ^ ((r >> 2) & 1)) << 4));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_q4_kernel(const __grid_constant__ Q4Params qp) {
  using L = Layout<D>;
  constexpr int G = L::G;
  const PagedParams& p = qp.p;
  extern __shared__ __align__(1024) uint8_t raw[];
  Head& h = *reinterpret_cast<Head*>(raw);
  uint8_t* const ring = raw + kHeadBytes;   // (1,024-byte boundaries: the head is 2 KB, slots are multiples)
  uint8_t* const q_s = ring + qp.n_slots * L::kSlot;
  float* const join_s = reinterpret_cast<float*>(raw + kHeadBytes + qp.n_slots * L::kSlot + L::kQ);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* abrt = &h.abort;
  if (tid == 0) {
    for (int i = 0; i < qp.n_slots; ++i) {
      bar_init(&h.full[i], 1);
      bar_init(&h.empty[i], kWarps);
    }
    h.abort = 0;
    bar_init_fence();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_dependency_release();
  const Start st = find_run<kThreads, kKT>(p, kMT, blockIdx.x, gridDim.x, h.scan, &h.start);
  Cursor<kKT> c;
  c.begin(p, kMT, st);
  if (st.n == 0) {
    if (tid == 0) p.parts[blockIdx.x] = PagedPart{};
    return;
  }
  int slot = 0;
  uint32_t use = 0;
  auto step = [&] {
    if (++slot == qp.n_slots) {
      slot = 0;
      ++use;
    }
  };

  if (warp >= kWarps) {
    // ------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsCopy));
    if (warp > kWarps) return;
    // A lane a box of tokens: its K, V and records.
    const int box = min(1 << p.page_shift, kKT), n_box = kKT / box, page_mask = (1 << p.page_shift) - 1;
    const bool copies = lane < n_box;
    int tj = 0;
    bool live = true;
    for (bool more = true; more && live; more = c.next(p, kMT)) {
      const ItemRows ir = item_rows(p, c);
      const int T = c.x1 - c.x;
      auto wanted = [&](int j) {
        const int t = c.tiles.token(c.x + j) + lane * box, end = min(t + box - 1, ir.last);
        return copies && t <= ir.last && (p.window == 0 || end > ir.first - p.window || t < p.n_sinks);
      };
      auto look_up = [&](int j) {
        const int64_t s = (int64_t)(c.tiles.token(c.x + j) + lane * box) >> p.page_shift;
        int32_t page = -1;
        if (wanted(j) && s < p.table_ld) page = __ldcg(p.table + c.seq * p.table_ld + s);
        return page;
      };
      int page = look_up(0), next = T > 1 ? look_up(1) : 0;
#pragma unroll 1
      for (int j = 0; j < T; ++j) {
        const int ahead = j + 2 < T ? look_up(j + 2) : 0;
        if (use > 0 && !wait(&h.empty[slot], (use - 1) & 1, abrt)) live = false;
        live = __all_sync(0xffffffffu, live);
        if (!live) break;
        const bool want = wanted(j), missing = want && (uint32_t)page >= (uint32_t)p.n_pages;
        if (!want || missing) page = p.n_pages;   // past the last page: zeros
        const uint32_t bad =
            __reduce_or_sync(0xffffffffu, missing ? ((1u << (box / 16)) - 1u) << (lane * (box / 16)) : 0u);
        if (missing) atomicAdd(&g_bad_pages, 1);
        if (lane == 0) {
          h.bad[(tj + j) & 15] = bad;
          bar_expect_tx(&h.full[slot], L::kSlot);
        }
        __syncwarp();
        if (copies) {
          const uint32_t to = smem_addr(ring) + slot * L::kSlot;
          const int token = c.tiles.token(c.x + j) & page_mask;
          tma_4d(to + lane * box * L::kRow, &qp.k, 0, token, c.head, page, &h.full[slot]);
          tma_4d(to + L::kCodes + lane * box * L::kRow, &qp.v, 0, token, c.head, page, &h.full[slot]);
          tma_4d(to + 2 * L::kCodes + lane * box * L::kRecord, &qp.r, 0, token, c.head, page, &h.full[slot]);
        }
        __syncwarp();
        step();
        page = next;
        next = ahead;
      }
      tj += T;
    }
    // Every copy has landed before the CTA ends.
    if (lane < qp.n_slots) {
      const uint32_t uses = use + (lane < slot ? 1u : 0u);
      if (uses > 0) bar_wait(&h.full[lane], (uses - 1) & 1, &g_timeouts);
    }
    return;
  }

  // -------------------------------------------------------------- products
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsCompute));
  const int n = lane >> 2, t = lane & 3;   // MMA row (and n + 8) and key column; k slot
  const int k0 = 16 * warp;                // the warp's keys of a tile
  int tj = 0;
  for (bool more = true; more;) {
    const ItemRows ir = item_rows(p, c);
    const int T = c.x1 - c.x;
    const int row_lo = min(n, ir.nf - 1), row_hi = min(n + 8, ir.nf - 1);
    const int pos_lo = ir.pos0 + row_of(p, ir.f0 + row_lo), pos_hi = ir.pos0 + row_of(p, ir.f0 + row_hi);
    // Q: row n (and n + 8), channels 32 g + 8 t .. + 7 of each block.
    uint32_t qf[L::kQShared ? 1 : 2 * G][4];
    uint32_t qm[4];                        // block sums: high halves in slots 0-7, low in 8-15
    float zc_lo, zc_hi;
    {
      uint4 x[2][G];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int f = ir.f0 + (i ? row_hi : row_lo), r = row_of(p, f);
        const int64_t entry = (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f - r * p.group);
        const bool mine = (i ? n + 8 : n) < ir.nf;
#pragma unroll
        for (int g = 0; g < G; ++g)
          x[i][g] = mine ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + entry * D + 32 * g) + t)
                         : make_uint4(0u, 0u, 0u, 0u);
      }
      float up[2], sums[2][G];
      bool odd[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t most = 0u;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t w[4] = {x[i][g].x, x[i][g].y, x[i][g].z, x[i][g].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) most = max(most, max((w[e] << 16) & 0x7fff0000u, w[e] & 0x7fff0000u));
        }
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // 2^(exponent - 8), at least 2^-100: a row of smaller values keeps fewer bits.
        const int e = max((int)(most >> 23) - 127 - 8, -100);
        odd[i] = most >= 0x7f800000u;      // infinity or NaN: the row's logits are NaN
        up[i] = odd[i] ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23);
        const float down = odd[i] ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
        // (Not 0, also where scale and power are both tiny: hidden logits are -infinity times it.)
        (i ? zc_hi : zc_lo) = fmaxf(p.scale * kLog2e * down, 1e-37f);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        uint32_t frag[2][4];               // k-steps 0 and 1
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w[4] = {x[i][g].x, x[i][g].y, x[i][g].z, x[i][g].w};
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[2 * e] = odd[i] ? __uint_as_float(0x7fffffffu) : bf16_lo(w[e]) * up[i];
            v[2 * e + 1] = odd[i] ? __uint_as_float(0x7fffffffu) : bf16_hi(w[e]) * up[i];
          }
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) s += v[e];
          s += __shfl_xor_sync(0xffffffffu, s, 1);
          s += __shfl_xor_sync(0xffffffffu, s, 2);
          sums[i][g] = s;
          // Slots 2 t, 2 t + 1 of a step hold channels j and 4 + j; the codes of even j are
          // 2^4 smaller.
#pragma unroll
          for (int x2 = 0; x2 < 2; ++x2) {
            frag[x2][i] = pack_f16(v[2 * x2] * 16.f, v[4 + 2 * x2] * 16.f);
            frag[x2][2 + i] = pack_f16(v[2 * x2 + 1], v[5 + 2 * x2]);
          }
        }
        if constexpr (L::kQShared) {
          if (g == warp) {
#pragma unroll
            for (int x2 = 0; x2 < 2; ++x2)
              *reinterpret_cast<uint4*>(q_s + (2 * g + x2) * 512 + lane * 16) =
                  make_uint4(frag[x2][0], frag[x2][1], frag[x2][2], frag[x2][3]);
          }
        } else {
#pragma unroll
          for (int x2 = 0; x2 < 2; ++x2)
#pragma unroll
            for (int e = 0; e < 4; ++e) qf[2 * g + x2][e] = frag[x2][e];
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float s0 = 0.f, s1 = 0.f;          // blocks 2 t and 2 t + 1
#pragma unroll
        for (int g = 0; g < G; g += 2)
          if (g == 2 * t) {
            s0 = sums[i][g];
            s1 = sums[i][g + 1];
          }
        const uint32_t hi = pack_f16(s0, s1);
        const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        qm[i] = hi;
        qm[2 + i] = pack_f16(s0 - back.x, s1 - back.y);
      }
      if constexpr (L::kQShared) named_sync(1, 32 * kWarps);
    }
    auto q_frag = [&](int i, uint32_t (&a)[4]) {
      if constexpr (L::kQShared) {
        const uint4 v = lds128(q_s + i * 512 + lane * 16);
        a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = qf[L::kQShared ? 0 : i][e];
      }
    };

    float o[G][4][4], om[4];
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[g][j][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) om[e] = 0.f;
    float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;   // l: of this thread's columns

#pragma unroll 1
    for (int j = 0; j < T; ++j) {
      const int t0 = c.tiles.token(c.x + j) + k0;
      wait(&h.full[slot], use & 1, abrt);
      __syncwarp();
      const bool gone = (h.bad[(tj + j) & 15] >> warp) & 1u;
      const bool any = !gone && t0 <= ir.last && (p.window == 0 || t0 + 15 > ir.first - p.window || t0 < p.n_sinks);
      if (any) {
        const uint8_t *const ks = ring + slot * L::kSlot, *const vs = ks + L::kCodes, *const rs = ks + 2 * L::kCodes;
        const bool edge = t0 + 15 > ir.first || (p.window > 0 && t0 <= ir.last - p.window && t0 + 16 > p.n_sinks);
        // ---- logits of two key columns of eight
        float z[2][4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int kr = k0 + 8 * hf + key_of(n);
          uint32_t wa[G / 2], wb[G / 2];   // units 2 t and 2 t + 1 of blocks (0, 1), (2, 3), ...
          if constexpr (D == 256) {
            const uint4 a = lds128(ks + swizzled<128>(kr, 2 * t)), b = lds128(ks + swizzled<128>(kr, 2 * t + 1));
            wa[0] = a.x, wa[1] = a.y, wa[2] = a.z, wa[3] = a.w;
            wb[0] = b.x, wb[1] = b.y, wb[2] = b.z, wb[3] = b.w;
          } else {
            const uint4 a = lds128(ks + swizzled<64>(kr, t));
            wa[0] = a.x, wa[1] = a.y, wb[0] = a.z, wb[1] = a.w;
          }
          // Scales of the thread's two key columns.
          uint32_t s0[G], s1[G];
#pragma unroll
          for (int i = 0; i < G / 4; ++i) {
            const uint4 a = lds128(rs + swizzled<L::kRecord>(k0 + 8 * hf + key_of(2 * t), i)),
                        b = lds128(rs + swizzled<L::kRecord>(k0 + 8 * hf + key_of(2 * t + 1), i));
            s0[4 * i] = a.x, s0[4 * i + 1] = a.y, s0[4 * i + 2] = a.z, s0[4 * i + 3] = a.w;
            s1[4 * i] = b.x, s1[4 * i + 1] = b.y, s1[4 * i + 2] = b.z, s1[4 * i + 3] = b.w;
          }
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t w = __byte_perm(wa[g / 2], wb[g / 2], g & 1 ? 0x7632 : 0x5410), w8 = w >> 8;
            float d[4];
            uint32_t a[4];
            q_frag(2 * g, a);
            mma_first(d, a, w & 0x000f000fu, w & 0x00f000f0u);
            q_frag(2 * g + 1, a);
            mma(d, a, w8 & 0x000f000fu, w8 & 0x00f000f0u);
            const float f0 = low_half(s0[g]), f1 = low_half(s1[g]);
            fma2(acc[0], acc[1], f0, f1, d[0], d[1]);
            fma2(acc[2], acc[3], f0, f1, d[2], d[3]);
          }
          // Minima of blocks 2 t, 2 t + 1 of key column n, against both halves of the sums.
          uint32_t mm = 0u;
          if (2 * t < G) {
            const uint2 two = lds64(rs + swizzled<L::kRecord>(kr, t >> 1) + 8 * (t & 1));
            mm = __byte_perm(two.x, two.y, 0x7632);
          }
          float d[4];
          mma_first(d, qm, mm, mm);
#pragma unroll
          for (int e = 0; e < 4; ++e) z[hf][e] = fmaf(acc[e], 0x1p20f, d[e]);
        }
        if (edge) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int tk = t0 + 8 * hf + key_of(2 * t + (e & 1));
              if (!sees(p, e < 2 ? pos_lo : pos_hi, tk)) z[hf][e] = -INFINITY;
            }
        }
        // ---- V's scales: pairs of the thread's keys (columns 2 t, 2 t + 1 of both halves)
        uint32_t sab[G], scd[G], mab = 0u, mcd = 0u;
        {
          uint32_t rec[4][G];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int kr = k0 + 8 * (i >> 1) + key_of(2 * t + (i & 1));
#pragma unroll
            for (int x = 0; x < G / 4; ++x) {
              const uint4 a = lds128(rs + swizzled<L::kRecord>(kr, G / 4 + x));
              rec[i][4 * x] = a.x, rec[i][4 * x + 1] = a.y, rec[i][4 * x + 2] = a.z, rec[i][4 * x + 3] = a.w;
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            sab[g] = __byte_perm(rec[0][g], rec[1][g], 0x5410);
            scd[g] = __byte_perm(rec[2][g], rec[3][g], 0x5410);
          }
          if (n < G) {   // minima of block n
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = lds32(rs + swizzled<L::kRecord>(k0 + 8 * (i >> 1) + key_of(2 * t + (i & 1)), G / 4 + (n >> 2)) + 4 * (n & 3));
            mab = __byte_perm(w[0], w[1], 0x7632);
            mcd = __byte_perm(w[2], w[3], 0x7632);
          }
          if (edge) {   // what no row sees may hold anything
            uint32_t keep[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tk = t0 + 8 * (i >> 1) + key_of(2 * t + (i & 1));
              if (tk <= ir.last && (p.window == 0 || tk > ir.first - p.window || tk < p.n_sinks))
                keep[i >> 1] |= i & 1 ? 0xffff0000u : 0xffffu;
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
              sab[g] &= keep[0];
              scd[g] &= keep[1];
            }
            mab &= keep[0];
            mcd &= keep[1];
          }
        }
        // Scales of 2^6 and more ask for smaller weights.
        float big = 0.f;
        {
          uint32_t any_s = 0u;
#pragma unroll
          for (int g = 0; g < G; ++g) any_s |= sab[g] | scd[g];
          if (__any_sync(0xffffffffu, (any_s & 0x40004000u) != 0u)) {
            uint32_t most = 0u;
#pragma unroll
            for (int g = 0; g < G; ++g)
              most = max(most, max(max(sab[g] & 0x7fffu, (sab[g] >> 16) & 0x7fffu), max(scd[g] & 0x7fffu, (scd[g] >> 16) & 0x7fffu)));
            most = __reduce_max_sync(0xffffffffu, most);
            // (|s| < 2^(exponent - 14))
            big = fmaxf((float)((int)(most >> 10) - 14) - kScaleTop, 0.f);
          }
        }
        // ---- the rows' maxima
        float x_lo = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1]));
        float x_hi = fmaxf(fmaxf(z[0][2], z[0][3]), fmaxf(z[1][2], z[1][3]));
        x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 1));
        x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 1));
        x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 2));
        x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 2));
        const float need_lo = fmaf(x_lo, zc_lo, big), need_hi = fmaf(x_hi, zc_hi, big);
        const bool move_lo = m_lo == -INFINITY ? need_lo > m_lo : need_lo > m_lo + kLag;
        const bool move_hi = m_hi == -INFINITY ? need_hi > m_hi : need_hi > m_hi + kLag;
        if (__any_sync(0xffffffffu, move_lo || move_hi)) {
          const float a_lo = move_lo ? ex2(m_lo - need_lo) : 1.f, a_hi = move_hi ? ex2(m_hi - need_hi) : 1.f;
          if (move_lo) m_lo = need_lo;
          if (move_hi) m_hi = need_hi;
          l_lo *= a_lo;
          l_hi *= a_hi;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              o[g][jj][0] *= a_lo;
              o[g][jj][1] *= a_lo;
              o[g][jj][2] *= a_hi;
              o[g][jj][3] *= a_hi;
            }
          om[0] *= a_lo;
          om[1] *= a_lo;
          om[2] *= a_hi;
          om[3] *= a_hi;
        }
        const float sh_lo = m_lo == -INFINITY ? 0.f : kTop - m_lo, sh_hi = m_hi == -INFINITY ? 0.f : kTop - m_hi;
        uint32_t pw[4];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float w0 = ex2(fmaf(z[hf][0], zc_lo, sh_lo)), w1 = ex2(fmaf(z[hf][1], zc_lo, sh_lo)),
                      w2 = ex2(fmaf(z[hf][2], zc_hi, sh_hi)), w3 = ex2(fmaf(z[hf][3], zc_hi, sh_hi));
          l_lo += w0 + w1;
          l_hi += w2 + w3;
          pw[2 * hf] = pack_f16(w0, w1);
          pw[2 * hf + 1] = pack_f16(w2, w3);
        }
        // ---- output
        mma(om, pw, mab, mcd);
        uint32_t vw[4][G / 2];   // the thread's four keys: unit n of blocks (0, 1), (2, 3), ...
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kr = k0 + 8 * (i >> 1) + key_of(2 * t + (i & 1));
          if constexpr (D == 256) {
            const uint4 a = lds128(vs + swizzled<128>(kr, n));
            vw[i][0] = a.x, vw[i][1] = a.y, vw[i][2] = a.z, vw[i][3] = a.w;
          } else {
            const uint2 a = lds64(vs + swizzled<64>(kr, n >> 1) + 8 * (n & 1));
            vw[i][0] = a.x, vw[i][1] = a.y;
          }
        }
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint32_t a[4] = {mul_f16(pw[0], sab[g]), mul_f16(pw[1], sab[g]), mul_f16(pw[2], scd[g]), mul_f16(pw[3], scd[g])};
          const uint32_t w0 = __byte_perm(vw[0][g / 2], vw[1][g / 2], g & 1 ? 0x7632 : 0x5410),
                         w1 = __byte_perm(vw[2][g / 2], vw[3][g / 2], g & 1 ? 0x7632 : 0x5410);
          const uint32_t u0 = w0 >> 8, u1 = w1 >> 8;
          mma(o[g][0], a, w0 & 0x000f000fu, w1 & 0x000f000fu);
          mma(o[g][1], a, w0 & 0x00f000f0u, w1 & 0x00f000f0u);
          mma(o[g][2], a, u0 & 0x000f000fu, u1 & 0x000f000fu);
          mma(o[g][3], a, u0 & 0x00f000f0u, u1 & 0x00f000f0u);
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&h.empty[slot]);
      step();
    }
    tj += T;

    // ---- the eight warps' parts of the item
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 1);
    l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 1);
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, 2);
    l_hi += __shfl_xor_sync(0xffffffffu, l_hi, 2);
    if (t == 0) {
      h.m[warp][n] = m_lo;
      h.m[warp][n + 8] = m_hi;
      h.l[warp][n] = l_lo;
      h.l[warp][n + 8] = l_hi;
    }
    named_sync(1, 32 * kWarps);
    float top_lo = -INFINITY, top_hi = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      top_lo = fmaxf(top_lo, h.m[w][n]);
      top_hi = fmaxf(top_hi, h.m[w][n + 8]);
    }
    const float f_lo = m_lo == -INFINITY ? 1.f : ex2(m_lo - top_lo), f_hi = m_hi == -INFINITY ? 1.f : ex2(m_hi - top_hi);
    // This thread's part of the joined rows: row jr, four channels from jc on, of two blocks a pass.
    const int jr = tid >> 4, jc = 4 * (tid & 15);
    float l = 0.f, top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, h.m[w][jr]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = h.m[w][jr];
      l += h.l[w][jr] * (mw == -INFINITY ? 1.f : ex2(mw - top));   // (no weights: 0, or NaN)
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const bool whole = c.whole();
    const int64_t part = (int64_t)c.slot(blockIdx.x) * kMT + jr;
    const int fr = ir.f0 + min(jr, ir.nf - 1), rr = row_of(p, fr);
    const int64_t entry = (int64_t)(c.s.row0 + rr) * p.n_q_heads + c.head * p.group + (fr - rr * p.group);
#pragma unroll
    for (int b = 0; b < G / 2; ++b) {
      if (b > 0) named_sync(1, 32 * kWarps);
      float* const mine = join_s + warp * (kMT * L::kPitch);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int g = 2 * b + x;
        // The block's minima's sums are column g: with the thread g / 2 of the row's four.
        const int from = (lane & ~3) | (g >> 1);
        const float mlo = __shfl_sync(0xffffffffu, om[g & 1], from), mhi = __shfl_sync(0xffffffffu, om[2 + (g & 1)], from);
        float v[2][8];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float s = jj & 1 ? 0x1p20f : 0x1p24f;
          v[0][jj] = fmaf(o[g][jj][0], s, mlo) * f_lo;
          v[0][4 + jj] = fmaf(o[g][jj][1], s, mlo) * f_lo;
          v[1][jj] = fmaf(o[g][jj][2], s, mhi) * f_hi;
          v[1][4 + jj] = fmaf(o[g][jj][3], s, mhi) * f_hi;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float4* to = reinterpret_cast<float4*>(mine + (n + 8 * i) * L::kPitch + 32 * x + 8 * t);
          to[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
          to[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
        }
      }
      named_sync(1, 32 * kWarps);
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(join_s + (w * kMT + jr) * L::kPitch + jc);
        sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
      }
      if (jr < ir.nf) {
        const int d = 64 * b + jc;
        sum = make_float4(sum.x * inv, sum.y * inv, sum.z * inv, sum.w * inv);
        if (!whole) {
          *reinterpret_cast<float4*>(p.part_o + part * D + d) = sum;
        } else if (p.out_dtype == QSA_F32) {
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + entry * D + d) = sum;
        } else {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + entry * D + d) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
        }
      }
    }
    if (jr < ir.nf && (tid & 15) == 0) {
      const float lse2 = l == 0.f ? -INFINITY : top - kTop + log2f(l);
      if (!whole) p.part_lse[part] = lse2;
      else if (p.lse) p.lse[entry] = lse2 * kLn2;
    }
    named_sync(1, 32 * kWarps);   // the statistics and Q are the next item's
    more = c.next(p, kMT);
    if (!more && tid == 0) describe_part(p, c, st, blockIdx.x);
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

// Rows of `bytes`, with strides in bytes.
bool encode_rows(CUtensorMap* map, const void* base, const PagedParams& p, int bytes, int64_t tok, int64_t head,
                 int64_t page_stride) {
  PFN_cuTensorMapEncodeTiled_v12000 f = encoder();
  if (!f) return false;
  const cuuint64_t page = (cuuint64_t)1 << p.page_shift;
  const cuuint64_t dims[4] = {(cuuint64_t)bytes, page, (cuuint64_t)p.n_kv_heads, (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)tok, (cuuint64_t)head, (cuuint64_t)page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)bytes, (cuuint32_t)(page < kKT ? page : kKT), 1, 1}, step[4] = {1, 1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE,
           bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const PagedParams& p, int grid, cudaStream_t st) {
  using L = Layout<D>;
  Q4Params qp{};
  qp.p = p;
  if (!encode_rows(&qp.k, p.k, p, L::kRow, p.tok_stride / 2, p.head_stride / 2, p.page_stride / 2) ||
      !encode_rows(&qp.v, p.v, p, L::kRow, p.tok_stride / 2, p.head_stride / 2, p.page_stride / 2) ||
      !encode_rows(&qp.r, p.kv_scale, p, L::kRecord, p.s_tok_stride * L::kRecord, p.s_head_stride * L::kRecord,
                   p.s_page_stride * L::kRecord))
    return cudaErrorInvalidValue;
  qp.n_slots = std::min((kSmemLimit - L::kFixed) / L::kSlot, kMaxSlots);
  const size_t smem = (size_t)L::kFixed + (size_t)qp.n_slots * L::kSlot;
  cudaError_t e = allow_dynamic_smem((const void*)paged_q4_kernel<D>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(paged_q4_kernel<D>, dim3((unsigned)grid), dim3(kThreads), smem, st, 0u, qp);
}

}  // namespace

cudaError_t launch_paged_q4(const PagedParams& p, int head_dim, int grid, cudaStream_t st) {
  return head_dim == 256 ? launch_d<256>(p, grid, st) : launch_d<128>(p, grid, st);
}

int paged_q4_bad_pages_take() { return take_counter(g_bad_pages); }

int paged_q4_wait_timeouts() {
  int v = 0;
  return cudaMemcpyFromSymbol(&v, g_timeouts, sizeof(int)) == cudaSuccess ? v : -1;
}

}  // namespace qsa
