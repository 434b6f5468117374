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
constexpr int kWarps = 12;               // that compute
constexpr int kThreads = 32 * (kWarps + 4);   // four warpgroups: three that compute, one whose first warp copies
// Registers of a thread: 128 at launch (512 threads share 65,536), of which the copying
// warpgroup leaves 96 to the others: 384 * 160 + 128 * 32 = 65,536.
constexpr int kRegsCompute = 160, kRegsCopy = 32;
constexpr int kMT = 16;                  // entries of an item
constexpr int kTeams = kWarps / 4, kMaxSlots = 5 * kTeams;
constexpr int kKT = 64;                  // keys of a tile: 16 for each of a team's four warps
constexpr int kSmemLimit = 227 * 1024;
constexpr float kTop = 3.f;              // log2 of the largest weight when the maximum is up to date
constexpr float kLag = 7.f;              // log2 of what a weight may pass it by
constexpr float kScaleTop = 5.f;         // log2 of the scales that this leaves room for

__device__ int g_timeouts;
__device__ int g_bad_pages;

struct Q4Params {
  CUtensorMap k, v, r;   // {bytes of a row or record, page_tokens, Hkv, n_pages}: boxes of min(page_tokens, 64) tokens
  PagedParams p;
};

struct Head {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  int64_t scan[kThreads / 32];
  Start start;
  int abort;
  uint32_t bad[kMaxSlots];   // 16-token pieces of the slot's tile that have no page
  float m[kWarps][kMT], l[kWarps][kMT];
};
constexpr int kHeadBytes = 4 * 1024;
static_assert(sizeof(Head) <= kHeadBytes, "shared memory head");

// Three teams of four warps take an item's tiles in turn, each with a ring of slots and a
// copying warp of its own: a slot's phases then follow each other for everyone who waits
// for one.  A warp computes the logits and weights of
// 16 keys, all channels; of head_dim 256, two warps exchange their weights and take half
// of the channels of all 32 keys each for the output (which is what 12 warps' registers
// hold).
template <int D>
struct Layout {
  static constexpr int kHalves = D / 128, kPairs = kWarps / kHalves;
  static constexpr int kRow = D / 2, kRecord = D / 4;
  static constexpr int kCodes = kKT * kRow, kSlot = 2 * kCodes + kKT * kRecord;
  static constexpr int kQ = 1024 * D / 32;         // Q's fragments, two k-steps a block
  // Joining: 32 channels of the 16 rows of each warp, rows 4 floats apart in banks (before
  // that, the weights' exchange).
  static constexpr int kPitch = 36, kJoin = kWarps * kMT * kPitch * 4;
  static constexpr int kFixed = kHeadBytes + kQ + kJoin;
  static constexpr int kFit = (kSmemLimit - kFixed) / (kTeams * kSlot);
  static constexpr int kTeamSlots = kFit < kMaxSlots / kTeams ? kFit : kMaxSlots / kTeams, kSlots = kTeams * kTeamSlots;
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
// (Not volatile: products of registers, which may be moved past each other.)
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {   // c = a b
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b, bool first) {   // 8 of k
  if (first)
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%7, %7, %7, %7};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(b), "f"(0.f));
  else
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b));
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

// The row of 16 keys at tile column n of either half: the order that spreads the rows
// which one load of a warp touches over all banks (K: columns 2 i and 2 i + 1 differ in
// the lowest bit; V and the records: columns 0, 2, 4, 6, and 1, 3, 5, 7, are two rows of
// each parity, two apart).
__device__ __forceinline__ int key_of(int n) { return n ^ ((n >> 1) & 1); }

// Where a tile's rows lie under TMA's swizzles: chunk c (16 bytes) of row r of codes or
// records.  Rows 8 on are 8 whole rows on, and chunks that differ by one bit are that bit
// of the offset apart, so a lane needs one offset for each of the rows it reads.
template <int BYTES>
__device__ __forceinline__ int swizzled(int r, int c) {
  if constexpr (BYTES == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else if constexpr (BYTES == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_q4_kernel(const __grid_constant__ Q4Params qp) {
  using L = Layout<D>;
  constexpr int G = D / 32, H = L::kHalves, KT = kKT;
  const PagedParams& p = qp.p;
  extern __shared__ __align__(1024) uint8_t raw[];
  Head& h = *reinterpret_cast<Head*>(raw);
  uint8_t* const ring = raw + kHeadBytes;   // (1,024-byte boundaries: the head is 4 KB, slots are multiples)
  uint8_t* const q_s = ring + L::kSlots * L::kSlot;
  float* const join_s = reinterpret_cast<float*>(q_s + L::kQ);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* abrt = &h.abort;
  if (tid == 0) {
    for (int i = 0; i < L::kSlots; ++i) {
      bar_init(&h.full[i], 1);
      bar_init(&h.empty[i], kWarps / kTeams);
    }
    h.abort = 0;
    bar_init_fence();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_dependency_release();
  const Start st = find_run<kThreads, KT>(p, kMT, blockIdx.x, gridDim.x, h.scan, &h.start);
  Cursor<KT> c;
  c.begin(p, kMT, st);
  if (tid == 0) h.start = st;   // for the end (this thread's): registers are short
  if (st.n == 0) {
    if (tid == 0) p.parts[blockIdx.x] = PagedPart{};
    return;
  }
  if (warp >= kWarps) {
    // ------------------------------------------------------------ copies
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kRegsCopy));
    // A warp for each team; a lane a box of tokens: its K, V and records.
    const int team = warp - kWarps;
    if (team >= kTeams) return;
    const int box = min(1 << p.page_shift, KT), n_box = KT / box, page_mask = (1 << p.page_shift) - 1;
    const bool copies = lane < n_box;
    int done = 0;   // the team's tiles
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
      int page = team < T ? look_up(team) : -1, next = team + kTeams < T ? look_up(team + kTeams) : -1;
#pragma unroll 1
      for (int j = team; j < T; j += kTeams, ++done) {
        const int ahead = j + 2 * kTeams < T ? look_up(j + 2 * kTeams) : -1;
        const int use = done / L::kTeamSlots, slot = team * L::kTeamSlots + done % L::kTeamSlots;
        if (use > 0 && !wait(&h.empty[slot], (uint32_t)(use - 1) & 1, abrt)) live = false;
        live = __all_sync(0xffffffffu, live);
        if (!live) break;
        const bool want = wanted(j), missing = want && (uint32_t)page >= (uint32_t)p.n_pages;
        if (!want || missing) page = p.n_pages;   // past the last page: zeros
        const uint32_t bad =
            __reduce_or_sync(0xffffffffu, missing ? ((1u << (box / 16)) - 1u) << (lane * (box / 16)) : 0u);
        if (missing) atomicAdd(&g_bad_pages, 1);
        if (lane == 0) {
          h.bad[slot] = bad;
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
        page = next;
        next = ahead;
      }
    }
    // Every copy has landed before the CTA ends: a lane a slot, the last tile that went there.
    if (lane < L::kTeamSlots && lane < done) {
      const int last = done - 1 - (done - 1 - lane) % L::kTeamSlots;
      bar_wait(&h.full[team * L::kTeamSlots + lane], (uint32_t)(last / L::kTeamSlots) & 1, &g_timeouts);
    }
    return;
  }

  // -------------------------------------------------------------- products
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRegsCompute));
  const int n = lane >> 2, t = lane & 3;   // MMA row (and n + 8) and key column; k slot
  const int team = warp >> 2, piece = warp & 3, half = H == 2 ? warp & 1 : 0;
  const int k0 = 16 * piece;               // the warp's keys of a tile
  // Weights on their way to the other warp of the pair (two buffers in turn), and what they
  // are relative to: 512 bytes and 16 numbers a warp.
  uint4* const pair_w = reinterpret_cast<uint4*>(join_s);
  float* const pair_r = reinterpret_cast<float*>(join_s) + 2 * kWarps * 128;
  const uint8_t* const my_q = q_s + lane * 16;
  // Offsets in a tile: K's codes of key column n; the records of key columns 2 t, 2 t + 1
  // and n; V's codes of key columns 2 t, 2 t + 1 (of the tile's first 16 keys).
  constexpr int kRow = L::kRow, kRec = L::kRecord, kRecords = 2 * L::kCodes;
  int at_k = swizzled<kRow>(k0 + key_of(n), D == 256 ? 2 * t : t);
  int at_r0 = kRecords + swizzled<kRec>(key_of(2 * t), 0), at_r1 = kRecords + swizzled<kRec>(key_of(2 * t + 1), 0);
  int at_m = kRecords + swizzled<kRec>(k0 + key_of(n), 0) + 8 * (t & 1);
  int at_v0 = L::kCodes + swizzled<kRow>(key_of(2 * t), D == 256 ? n : n >> 1) + 8 * (D == 256 ? half : n & 1);
  int at_v1 = L::kCodes + swizzled<kRow>(key_of(2 * t + 1), D == 256 ? n : n >> 1) + 8 * (D == 256 ? half : n & 1);
  const int to_v = (H + half) << 4;        // from K's part of a record to the warp's part of V's: these bits change
  // (Kept: the compiler would work them out again for every tile.)
  asm volatile("" : "+r"(at_k), "+r"(at_r0), "+r"(at_r1), "+r"(at_m), "+r"(at_v0), "+r"(at_v1));
  int done = 0;   // the team's tiles
  for (bool more = true; more;) {
    const ItemRows ir = item_rows(p, c);
    const int T = c.x1 - c.x;
    const int pos_lo = ir.pos0 + row_of(p, ir.f0 + min(n, ir.nf - 1)), pos_hi = ir.pos0 + row_of(p, ir.f0 + min(n + 8, ir.nf - 1));
    // Q: row n (and n + 8), channels 32 g + 8 t .. + 7 of each block.
    uint32_t qm[2][H];                     // sums of four blocks: high halves in slots 0-3, low in 4-7
    float zc_lo, zc_hi;
    {
      const uint4* from[2];
      float up[2];
      bool odd[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int f = ir.f0 + min(n + 8 * i, ir.nf - 1), r = row_of(p, f);
        const int64_t entry = (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f - r * p.group);
        from[i] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + entry * D) + t;
        uint32_t most = 0u;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const uint4 x = __ldg(from[i] + 4 * g);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) most = max(most, max((w[e] << 16) & 0x7fff0000u, w[e] & 0x7fff0000u));
        }
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
        most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
        // 2^(exponent - 8), at least 2^-100: a row of smaller values keeps fewer bits.
        const int e = max((int)(most >> 23) - 127 - 8, -100);
        odd[i] = most >= 0x7f800000u;      // infinity or NaN: the row's logits are NaN
        up[i] = __uint_as_float((uint32_t)(127 - e) << 23);
        const float down = odd[i] ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
        // (Not 0, also where scale and power are both tiny: hidden logits are -infinity times it.)
        (i ? zc_hi : zc_lo) = fmaxf(p.scale * kLog2e * down, 1e-37f);
      }
#pragma unroll
      for (int hh = 0; hh < H; ++hh) {
        float sums[2][2] = {{0.f, 0.f}, {0.f, 0.f}};   // of blocks 2 (t & 1) and the next
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t frag[2][4];             // k-steps 0 and 1
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 x = __ldg(from[i] + 4 * (4 * hh + b));
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
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
            if ((t & 1) == b >> 1) sums[i][b & 1] = s;
            // Slots 2 t, 2 t + 1 of a step hold channels j and 4 + j; the codes of even j are
            // 2^4 smaller.
#pragma unroll
            for (int x2 = 0; x2 < 2; ++x2) {
              frag[x2][i] = pack_f16(v[2 * x2] * 16.f, v[4 + 2 * x2] * 16.f);
              frag[x2][2 + i] = pack_f16(v[2 * x2 + 1], v[5 + 2 * x2]);
            }
          }
          if (warp == 4 * hh + b) {
#pragma unroll
            for (int x2 = 0; x2 < 2; ++x2)
              *reinterpret_cast<uint4*>(q_s + (2 * warp + x2) * 512 + lane * 16) =
                  make_uint4(frag[x2][0], frag[x2][1], frag[x2][2], frag[x2][3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t hi = pack_f16(sums[i][0], sums[i][1]);
          const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
          qm[i][hh] = t < 2 ? hi : pack_f16(sums[i][0] - back.x, sums[i][1] - back.y);
        }
      }
      named_sync(1, 32 * kWarps);
    }

    float o[4][4][4], om[4];
#pragma unroll
    for (int g = 0; g < 4; ++g)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[g][j][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) om[e] = 0.f;
    // What the output's weights are relative to (whole numbers; the same in both warps of a
    // pair), and the sums of this thread's columns.
    float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
    [[maybe_unused]] int turn = 0;   // of the exchange's two buffers: one barrier between writes to the same

#pragma unroll 1
    for (int j = team; j < T; j += kTeams, ++done) {
      const int slot = team * L::kTeamSlots + done % L::kTeamSlots, t0 = c.tiles.token(c.x + j);
      wait(&h.full[slot], (uint32_t)(done / L::kTeamSlots) & 1, abrt);
      __syncwarp();
      const uint32_t bad = h.bad[slot];
      auto seen = [&](int tk) { return tk <= ir.last && (p.window == 0 || tk > ir.first - p.window || tk < p.n_sinks); };
      // Tiles that every row sees whole are the rule.
      const bool edge = bad != 0u || t0 + KT - 1 > ir.first || (p.window > 0 && t0 <= ir.last - p.window && t0 + KT > p.n_sinks);
      bool mine = true, other = H == 2;
      if (edge) {
        auto some = [&](int pc) {   // a piece with keys that some row sees
          const int a = t0 + 16 * pc;
          return !((bad >> pc) & 1u) && a <= ir.last && (p.window == 0 || a + 15 > ir.first - p.window || a < p.n_sinks);
        };
        mine = some(piece);
        other = H == 2 && some(piece ^ 1);
      }
      if (mine || other) {   // (the same in both warps of a pair)
        const uint8_t* const at = ring + slot * L::kSlot;
        uint32_t pw[4] = {0u, 0u, 0u, 0u};
        float r_lo = m_lo, r_hi = m_hi, add_lo = 0.f, add_hi = 0.f;   // what pw is relative to, and its sums
        if (mine) {
          // ---- logits of two key columns of eight
          float z[2][4], acc[2][4];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[hf][e] = 0.f;
#pragma unroll
          for (int hh = 0; hh < H; ++hh) {
            uint32_t w[2][4];              // units 2 t and 2 t + 1 (halves) of a block
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              uint2 a, b;
              if constexpr (D == 256) {
                a = lds64(at + at_k + 8 * kRow * hf + 8 * hh);
                b = lds64(at + (at_k ^ 16) + 8 * kRow * hf + 8 * hh);
              } else {
                const uint4 both = lds128(at + at_k + 8 * kRow * hf);
                a = make_uint2(both.x, both.y), b = make_uint2(both.z, both.w);
              }
              w[hf][0] = __byte_perm(a.x, b.x, 0x5410), w[hf][1] = __byte_perm(a.x, b.x, 0x7632);
              w[hf][2] = __byte_perm(a.y, b.y, 0x5410), w[hf][3] = __byte_perm(a.y, b.y, 0x7632);
            }
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              // Scales of the thread's two key columns.
              const uint4 s0 = lds128(at + (at_r0 ^ (16 * hh)) + k0 * kRec + 8 * kRec * hf),
                          s1 = lds128(at + (at_r1 ^ (16 * hh)) + k0 * kRec + 8 * kRec * hf);
              const uint32_t r0[4] = {s0.x, s0.y, s0.z, s0.w}, r1[4] = {s1.x, s1.y, s1.z, s1.w};
              // Minima of two blocks of key column n, against the high or the low halves of the sums.
              const uint2 two = lds64(at + (at_m ^ (16 * hh)) + 8 * kRec * hf);
              mma8(z[hf], qm[0][hh], qm[1][hh], __byte_perm(two.x, two.y, 0x7632), hh == 0);
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const uint4 qa = lds128(my_q + (8 * hh + 2 * g) * 512), qb = lds128(my_q + (8 * hh + 2 * g + 1) * 512);
                const uint32_t a0[4] = {qa.x, qa.y, qa.z, qa.w}, a1[4] = {qb.x, qb.y, qb.z, qb.w};
                const uint32_t x = w[hf][g], x8 = x >> 8;
                float d[4];
                mma_first(d, a0, x & 0x000f000fu, x & 0x00f000f0u);
                mma(d, a1, x8 & 0x000f000fu, x8 & 0x00f000f0u);
                const float f0 = low_half(r0[g]), f1 = low_half(r1[g]);
                fma2(acc[hf][0], acc[hf][1], f0, f1, d[0], d[1]);
                fma2(acc[hf][2], acc[hf][3], f0, f1, d[2], d[3]);
              }
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int e = 0; e < 4; ++e) z[hf][e] = fmaf(acc[hf][e], 0x1p20f, z[hf][e]);
          if (edge) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tk = t0 + k0 + 8 * hf + key_of(2 * t + (e & 1));
                if (!sees(p, e < 2 ? pos_lo : pos_hi, tk)) z[hf][e] = -INFINITY;
              }
          }
          // V's scales of 2^5 and more ask for smaller weights: a lane looks at four blocks of a key.
          float big = 0.f;
          {
            const int kr = k0 + (H == 2 ? lane >> 1 : lane & 15);
            uint4 x = lds128(at + kRecords + swizzled<kRec>(kr, H + (H == 2 ? lane & 1 : 0)));
            if (edge && !seen(t0 + kr)) x = make_uint4(0u, 0u, 0u, 0u);
            if (__any_sync(0xffffffffu, ((x.x | x.y | x.z | x.w) & 0x4000u) != 0u)) {
              const uint32_t most = __reduce_max_sync(0xffffffffu, max(max(x.x & 0x7fffu, x.y & 0x7fffu), max(x.z & 0x7fffu, x.w & 0x7fffu)));
              // (|s| < 2^(exponent - 14))
              big = fmaxf((float)((int)(most >> 10) - 14) - kScaleTop, 0.f);
            }
          }
          // ---- the rows' maxima and weights
          float x_lo = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1]));
          float x_hi = fmaxf(fmaxf(z[0][2], z[0][3]), fmaxf(z[1][2], z[1][3]));
          x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 1));
          x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 1));
          x_lo = fmaxf(x_lo, __shfl_xor_sync(0xffffffffu, x_lo, 2));
          x_hi = fmaxf(x_hi, __shfl_xor_sync(0xffffffffu, x_hi, 2));
          const float need_lo = ceilf(fmaf(x_lo, zc_lo, big)), need_hi = ceilf(fmaf(x_hi, zc_hi, big));
          if (m_lo == -INFINITY || need_lo > m_lo + kLag) r_lo = fmaxf(need_lo, m_lo);
          if (m_hi == -INFINITY || need_hi > m_hi + kLag) r_hi = fmaxf(need_hi, m_hi);
          const float sh_lo = r_lo == -INFINITY ? 0.f : kTop - r_lo, sh_hi = r_hi == -INFINITY ? 0.f : kTop - r_hi;
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float w0 = ex2(fmaf(z[hf][0], zc_lo, sh_lo)), w1 = ex2(fmaf(z[hf][1], zc_lo, sh_lo)),
                        w2 = ex2(fmaf(z[hf][2], zc_hi, sh_hi)), w3 = ex2(fmaf(z[hf][3], zc_hi, sh_hi));
            add_lo += w0 + w1;
            add_hi += w2 + w3;
            pw[2 * hf] = pack_f16(w0, w1);
            pw[2 * hf + 1] = pack_f16(w2, w3);
          }
        }
        // ---- the pair's weights (the warp's own, then the other's), relative to the larger of two references
        uint32_t pv[H][4];
        float new_lo = r_lo, new_hi = r_hi;
        if constexpr (H == 2) {
          const int me = turn * kWarps + warp, you = me ^ 1;
          turn ^= 1;
          pair_w[me * 32 + lane] = make_uint4(pw[0], pw[1], pw[2], pw[3]);
          if (t == 0) {
            pair_r[me * 16 + n] = r_lo;
            pair_r[me * 16 + n + 8] = r_hi;
          }
          named_sync(2 + (warp >> 1), 64);
          const uint4 x = pair_w[you * 32 + lane];
          const float u_lo = pair_r[you * 16 + n], u_hi = pair_r[you * 16 + n + 8];
          const uint32_t y[4] = {x.x, x.y, x.z, x.w};
          new_lo = fmaxf(r_lo, u_lo);
          new_hi = fmaxf(r_hi, u_hi);
          // (Powers of two: exact, or below what f16 holds.)
          const float a_lo = r_lo == new_lo ? 1.f : ex2(r_lo - new_lo), a_hi = r_hi == new_hi ? 1.f : ex2(r_hi - new_hi),
                      b_lo = u_lo == new_lo ? 1.f : ex2(u_lo - new_lo), b_hi = u_hi == new_hi ? 1.f : ex2(u_hi - new_hi);
          if (__any_sync(0xffffffffu, r_lo != u_lo || r_hi != u_hi)) {
            add_lo *= a_lo;
            add_hi *= a_hi;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pv[0][e] = mul_f16(pw[e], pack_f16(e & 1 ? a_hi : a_lo, e & 1 ? a_hi : a_lo));
              pv[H - 1][e] = mul_f16(y[e], pack_f16(e & 1 ? b_hi : b_lo, e & 1 ? b_hi : b_lo));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pv[0][e] = pw[e];
              pv[H - 1][e] = y[e];
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) pv[0][e] = pw[e];
        }
        const bool move_lo = new_lo != m_lo, move_hi = new_hi != m_hi;   // (NaN: the weights are NaN anyway)
        if (__any_sync(0xffffffffu, move_lo || move_hi)) {
          const float a_lo = move_lo ? ex2(m_lo - new_lo) : 1.f, a_hi = move_hi ? ex2(m_hi - new_hi) : 1.f;
          m_lo = new_lo;
          m_hi = new_hi;
          l_lo *= a_lo;
          l_hi *= a_hi;
#pragma unroll
          for (int g = 0; g < 4; ++g)
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
        l_lo += add_lo;
        l_hi += add_hi;
        // ---- output: 16 keys at a time, the warp's 128 channels
#pragma unroll
        for (int s = 0; s < H; ++s) {
          if (!(s == 0 ? mine : other)) continue;
          const uint8_t* const mv = at + 16 * (s == 0 ? piece : piece ^ 1) * kRow;
          const uint8_t* const mr = at + 16 * (s == 0 ? piece : piece ^ 1) * kRec;
          uint32_t sab[4], scd[4], mab = 0u, mcd = 0u;   // scales, minima: pairs of the thread's keys
          {
            uint4 rec[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) rec[i] = lds128(mr + ((i & 1 ? at_r1 : at_r0) ^ to_v) + 8 * kRec * (i >> 1));
            sab[0] = __byte_perm(rec[0].x, rec[1].x, 0x5410), scd[0] = __byte_perm(rec[2].x, rec[3].x, 0x5410);
            sab[1] = __byte_perm(rec[0].y, rec[1].y, 0x5410), scd[1] = __byte_perm(rec[2].y, rec[3].y, 0x5410);
            sab[2] = __byte_perm(rec[0].z, rec[1].z, 0x5410), scd[2] = __byte_perm(rec[2].z, rec[3].z, 0x5410);
            sab[3] = __byte_perm(rec[0].w, rec[1].w, 0x5410), scd[3] = __byte_perm(rec[2].w, rec[3].w, 0x5410);
            if (n < 4) {   // minima of block n
              uint32_t x[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[i] = lds32(mr + ((i & 1 ? at_r1 : at_r0) ^ to_v) + 8 * kRec * (i >> 1) + 4 * n);
              mab = __byte_perm(x[0], x[1], 0x7632);
              mcd = __byte_perm(x[2], x[3], 0x7632);
            }
            if (edge) {   // what no row sees may hold anything
              uint32_t keep[2] = {0u, 0u};
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (seen(t0 + 16 * (s == 0 ? piece : piece ^ 1) + 8 * (i >> 1) + key_of(2 * t + (i & 1)))) keep[i >> 1] |= i & 1 ? 0xffff0000u : 0xffffu;
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                sab[g] &= keep[0];
                scd[g] &= keep[1];
              }
              mab &= keep[0];
              mcd &= keep[1];
            }
          }
          mma(om, pv[s], mab, mcd);
          uint2 vw[4];   // the thread's four keys: unit n of blocks (0, 1) and (2, 3)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            vw[i] = lds64(mv + (i & 1 ? at_v1 : at_v0) + 8 * kRow * (i >> 1));
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const uint32_t a[4] = {mul_f16(pv[s][0], sab[g]), mul_f16(pv[s][1], sab[g]), mul_f16(pv[s][2], scd[g]), mul_f16(pv[s][3], scd[g])};
            const uint32_t w0 = __byte_perm(g < 2 ? vw[0].x : vw[0].y, g < 2 ? vw[1].x : vw[1].y, g & 1 ? 0x7632 : 0x5410),
                           w1 = __byte_perm(g < 2 ? vw[2].x : vw[2].y, g < 2 ? vw[3].x : vw[3].y, g & 1 ? 0x7632 : 0x5410);
            const uint32_t u0 = w0 >> 8, u1 = w1 >> 8;
            mma(o[g][0], a, w0 & 0x000f000fu, w1 & 0x000f000fu);
            mma(o[g][1], a, w0 & 0x00f000f0u, w1 & 0x00f000f0u);
            mma(o[g][2], a, u0 & 0x000f000fu, u1 & 0x000f000fu);
            mma(o[g][3], a, u0 & 0x00f000f0u, u1 & 0x00f000f0u);
          }
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(&h.empty[slot]);
    }

    // ---- the warps' parts of the item
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
    for (int w = 0; w < L::kPairs; ++w) {
      top_lo = fmaxf(top_lo, h.m[H * w][n]);
      top_hi = fmaxf(top_hi, h.m[H * w][n + 8]);
    }
    const float f_lo = m_lo == -INFINITY ? 1.f : ex2(m_lo - top_lo), f_hi = m_hi == -INFINITY ? 1.f : ex2(m_hi - top_hi);
    // 128 H threads join: row jr, four channels from jc on of half jh, of a block a pass.
    const int jr = (tid >> 3) & 15, jc = 4 * (tid & 7), jh = tid >> 7;
    const bool joins = jh < H && jr < ir.nf;
    float l = 0.f, top = -INFINITY;
#pragma unroll
    for (int w = 0; w < L::kPairs; ++w) top = fmaxf(top, h.m[H * w][jr]);
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
    for (int g = 0; g < 4; ++g) {
      if (g > 0) named_sync(1, 32 * kWarps);
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
        float4* to = reinterpret_cast<float4*>(join_s + (warp * kMT + n + 8 * i) * L::kPitch + 8 * t);
        to[0] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
        to[1] = make_float4(v[i][4], v[i][5], v[i][6], v[i][7]);
      }
      named_sync(1, 32 * kWarps);
      if (joins) {
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < L::kPairs; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(join_s + ((H * w + jh) * kMT + jr) * L::kPitch + jc);
          sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
        }
        const int d = 128 * jh + 32 * g + jc;
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
    if (joins && jh == 0 && jc == 0) {
      const float lse2 = l == 0.f ? -INFINITY : top - kTop + log2f(l);
      if (!whole) p.part_lse[part] = lse2;
      else if (p.lse) p.lse[entry] = lse2 * kLn2;
    }
    named_sync(1, 32 * kWarps);   // the statistics, Q and the buffers are the next item's
    more = c.next(p, kMT);
    if (!more && tid == 0) describe_part(p, c, h.start, blockIdx.x);
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

// Rows of `bytes`, at most `most` tokens a copy, with strides in bytes.
bool encode_rows(CUtensorMap* map, const void* base, const PagedParams& p, int bytes, int most, int64_t tok,
                 int64_t head, int64_t page_stride) {
  PFN_cuTensorMapEncodeTiled_v12000 f = encoder();
  if (!f) return false;
  const cuuint64_t page = (cuuint64_t)1 << p.page_shift;
  const cuuint64_t dims[4] = {(cuuint64_t)bytes, page, (cuuint64_t)p.n_kv_heads, (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)tok, (cuuint64_t)head, (cuuint64_t)page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)bytes, (cuuint32_t)std::min<cuuint64_t>(page, (cuuint64_t)most), 1, 1}, step[4] = {1, 1, 1, 1};
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
  if (!encode_rows(&qp.k, p.k, p, L::kRow, kKT, p.tok_stride / 2, p.head_stride / 2, p.page_stride / 2) ||
      !encode_rows(&qp.v, p.v, p, L::kRow, kKT, p.tok_stride / 2, p.head_stride / 2, p.page_stride / 2) ||
      !encode_rows(&qp.r, p.kv_scale, p, L::kRecord, kKT, p.s_tok_stride * L::kRecord, p.s_head_stride * L::kRecord,
                   p.s_page_stride * L::kRecord))
    return cudaErrorInvalidValue;
  const size_t smem = (size_t)L::kFixed + (size_t)L::kSlots * L::kSlot;
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
