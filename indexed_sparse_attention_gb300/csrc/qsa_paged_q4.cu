// Attention of up to 16 query entries over a paged K/V cache held in 4 bits (QSA_Q4_1:
// blocks of 32 channels, value = code * scale + minimum; see include/qsa.h for the
// layout, qsa_paged.cuh for the division of the work into runs of key tiles, and
// qsa_paged.cu for the joining launch), on the 5th-generation tensor cores.
//
// An item's entries (query row, head of the KV head's group) are the 16 N columns of the
// products, and K and V the A operands, which warps bring from their codes into TMEM (128
// lanes) in registers: with entries as columns a product's time and its shared memory
// traffic stay small, and what is expanded never passes through shared memory.
//   logits   z_t = sum_g s_tg (sum_c q_c code_tc) + sum_g m_tg (sum_c q_c), lanes = a
//            tile's 128 keys.  A code is the E4M3 byte of code * 2^-9, subnormal or not:
//            masks only, eight codes in three instructions.  q times a power of two that
//            brings its row's largest magnitude to [2^11, 2^12) is the sum of an E5M2 code
//            and the E4M3 code of what that leaves: at most 16 of bf16's units, 4 bits, so
//            exact from 2^-13 of that largest on, off by at most 2^-10 (2^-21 of the
//            largest) below.  (Two E4M3 codes start at 2^8 and are exact from 2^-9 on only:
//            channels of 2^-13 were off by up to 1/16 of themselves.)  A block's
//            sum is a product of its own, kind::f8f6f4 with 32 of K, and the softmax, where a
//            thread owns a key, adds the blocks up times their scales in 32 bits.  The
//            minima are one more product, kind::f16, with 1/16 of the sums of q as two f16
//            halves (22 bits; a block of 2^12 is 2^17).
//   output   O^T += V^T P^T, lanes = 128 channels (twice for head_dim 256), kind::f16: V as
//            f16, code * scale + minimum rounded once.  A thread owns the four channels of a
//            code unit, of two keys a cell, in the fragment shape of tcgen05.st.
//            P^T = 2^(z - m) as f16 through shared memory, K-major like q.
// A row's maximum would be a reduction over lanes: instead the reference m of the weights
// stays until a logit passes it by 2^8 (one vote a tile), and only then the tile's maxima
// are reduced and O and the sums rescaled.  Weights are f16 with 2^7 at the reference, so
// 2^15 is the largest.  From a reference of 2^20 on, where units of a logit in binary32
// come near what f16 has room for, every tile is voted for, and the largest logit is taken
// off the others before they are multiplied: their differences keep all bits.
//
// Roles (16 warps): 0-7 expand codes (four warps a half of K's channels, and of V's keys),
// 8-11 softmax and output, 12 copies, 13 issues the logits' products, 14 the output's, 15
// writes Q.  K, V and their records come through TMA, 64 keys a slot; boxes of pages
// without visible tokens are aimed past the last page, which fills zeros without reading.  Every wait gives up after about two seconds (counted;
// nothing more is issued then, and the CTA runs to its end); its loop is out of line, as
// warps that wait in the middle of the roles' code take issue slots and instruction cache
// from those that expand (a ragged batch of 16 sequences took 146 us so, and 136 this way).
//
// What bounds it (us a call on one GB300, 24 query and 2 KV heads of 256): 16 sequences of
// 4k to 262k tokens 128, where HBM needs 77 and the copies alone take 95.  The rest is
// instructions, the expansion's and the softmax's side by side: with the softmax on two
// warpgroups of eight columns, which does more work, 136 -- then 118 without V's expansion,
// 125 without the softmax's arithmetic, 107 without both.  (Codes multiplied with mma.sync by
// 12 warps whose registers are full of output took 162; K expanded to f16 like V 151; 16
// expanding warps, at 64 registers, 163; 12, four of them for K, 140; one buffer of V's cells
// 145.)  One sequence of 65,536 tokens 28.5, of which 10 are the call's start, the joining launch
// and the first tiles' way through the roles.
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
constexpr int kHalfKeys = 64;            // of a slot, and of a half of V's product
constexpr int kCodeWarps = 8, kSoftWarp = 8, kCopyWarp = 12, kLogitWarp = 13, kOutWarp = 14;   // (15: Q)
constexpr int kThreads = 512;
constexpr int kEntries = 16;             // columns
constexpr int kMaxSlots = 20;
constexpr int kSmemLimit = 227 * 1024;
constexpr float kTop = 7.f;              // log2 of the weight at the reference
constexpr float kLag = 8.f;              // log2 of what a weight may pass it by
constexpr float kFar = 1048576.f;        // references from here on are taken off the logits
constexpr float kUnset = 3.402823466e38f; // shift of a column that has seen no logit: any finite one passes it
constexpr uint32_t kTmemCols = 512;
// TMEM columns: logits (16 a block, then the minima's), the minima, the output's two slabs, K's codes, two buffers
// of V's values.
constexpr uint32_t kSCol = 0, kMinCol = 144, kOCol = 160, kKCol = 192, kVCol = 256;

__device__ int g_timeouts;
__device__ int g_bad_pages;

struct Q4Params {
  CUtensorMap k, v, r;   // {bytes of a row or record, page_tokens, Hkv, n_pages}: boxes of min(page_tokens, 64) tokens
  PagedParams p;
  int32_t n_slots;
};

// A wait by parity tells a phase from its neighbours only: whoever waits for one has seen
// the phase before it, or caused it.
struct Head {
  uint64_t code_full[kMaxSlots], code_empty[kMaxSlots];
  uint64_t k_full, k_empty, s_full, s_empty;
  uint64_t v_full[2][2], v_empty[2][2];                    // halves of V's keys, of even and odd tiles
  uint64_t p_full[2], pv_done[2];                          // even and odd tiles
  uint64_t q_full, q_free, o_free, mma_done;
  uint64_t row_full[4];                                    // an item's q below
  int64_t scan[kThreads / 32];
  Start start;
  uint32_t tmem;
  int abort;
  uint8_t bad[16][2];              // 16-token pieces of a tile's halves that have no page (fewer tiles are under way)
  float q[4][kEntries];            // of an item's entries: the power of two that Q's row was divided by
  // Votes are about logit * x + y, and weights 2^(logit * x + y): the same but for references from kFar on.
  alignas(16) float2 vote[kEntries], column[kEntries];
  float ref[kEntries], factor[kEntries], inv[kEntries];
  alignas(16) float base[kEntries];   // the logit of such a reference, 0 else
  int far;                         // whether there is any
  int64_t to[kEntries];            // where the entry's outputs go, in elements
  int pos[kEntries];
  float mx[4][kEntries], sums[4][kEntries];
  alignas(16) uint4 scale[4][kKT];   // of K's blocks, of the last tiles
};
constexpr int kHeadBytes = 11 * 1024;
constexpr int kPBytes = 2 * kEntries * 128;   // a buffer of weights: slabs of 64 keys
static_assert(sizeof(Head) <= kHeadBytes, "shared memory head");

template <int D>
struct Slot {
  static constexpr int kRow = D / 2, kRecord = D / 4;
  static constexpr int kQSlab = kEntries * 128, kQ = (2 * (D / 128) + 1) * kQSlab;   // both codes of q, and its sums
  static constexpr int kCodes = kHalfKeys * kRow, kBytes = 2 * kCodes + kHalfKeys * kRecord;
};

__device__ __noinline__ bool wait_slow(uint64_t* b, uint32_t parity, int* abort) {
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
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 128;\n" ::: "memory"); }
// Whether any of the softmax's threads says so.
__device__ __forceinline__ bool soft_any(bool x) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(r)
               : "r"((uint32_t)x)
               : "memory");
  return r != 0;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two values to E4M3 or E5M2, the first in the low byte, and back.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e5m2x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e5m2x2(uint32_t two) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h2) : "h"((unsigned short)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h2));
}
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b) {   // (a & MASK) | b
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "n"(MASK), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t add_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// D[tmem] (+)= A[tmem] B[smem], f16.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// The same of 8-bit values, 32 of K.
__device__ __forceinline__ void mma_f8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Four consecutive columns of this thread's lane; tmem_st_wait before others read them.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};\n" ::"r"(a), "r"(b), "r"(c), "r"(d), "r"(taddr)
               : "memory");
}
// 16 lanes x 16 columns in two fragments of eight columns: of each, thread 4 i + j holds columns 2 j and
// 2 j + 1 of lane i, then of lane 8 + i.
__device__ __forceinline__ void tmem_st_fragments(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};\n" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr)
               : "memory");
}
// Eight consecutive columns of this thread's lane; the values are there after tmem_ld_wait of them.
__device__ __forceinline__ void tmem_ld8_start(uint32_t taddr, float* r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
               : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tmem_ld_done(float* r) {   // (uses of r stay behind the wait)
  asm volatile("" : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]));
}

// A reference from kFar on, or none yet, for a tile whose largest logit is top; the factor on what came before.  (Out
// of line: the first vote of an item waits for its instructions as they are.)
__device__ __noinline__ float far_reference(Head& h, int e, float top) {
  const float x = h.column[e].x, base = h.base[e], old = h.ref[e];
  if (base == 0.f ? top == -INFINITY : !((top - base) * x > kLag)) return 1.f;
  h.base[e] = top;
  h.ref[e] = top * x;
  h.vote[e].y = kUnset;
  h.column[e].y = kTop;
  h.far = 1;
  return old == -INFINITY ? 1.f : ex2(base == 0.f ? fmaf(-top, x, old) : (base - top) * x);
}

// v[0 .. 7] of every lane, reduced over the warp: lane x returns that of v[x / 4].
template <typename F>
__device__ __forceinline__ float reduce_columns(const float* from, int lane, F op) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = from[i];
#pragma unroll
  for (int n = 4; n >= 1; n >>= 1) {
    const bool up = (lane & (4 * n)) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = up ? v[n + i] : v[i], give = up ? v[i] : v[n + i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, 4 * n));
    }
  }
  v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
  return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// (a0, a1) += (f0, f1) (d0, d1).
__device__ __forceinline__ void fma2(float& a0, float& a1, float f0, float f1, float d0, float d1) {
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 z, {%0, %1};\n"
      " fma.rn.f32x2 z, x, y, z;\n mov.b64 {%0, %1}, z;\n}\n"
      : "+f"(a0), "+f"(a1)
      : "f"(f0), "f"(f1), "f"(d0), "f"(d1));
}

struct ItemRows {
  int f0, nf, pos0, first, last;
};
__device__ __forceinline__ ItemRows item_rows(const PagedParams& p, const Cursor<kKT>& c) {
  ItemRows r;
  r.f0 = c.m * p.mt;
  r.nf = min(p.mt, c.s.n * p.group - r.f0);
  r.pos0 = c.s.len - c.s.n;
  r.first = r.pos0 + row_of(p, r.f0);
  r.last = r.pos0 + row_of(p, r.f0 + r.nf - 1);
  return r;
}

// Where TMA's swizzles put chunk c (16 bytes) of row r of codes or records.
template <int BYTES>
__device__ __forceinline__ int swizzled(int r, int c) {
  if constexpr (BYTES == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else if constexpr (BYTES == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}
__device__ __forceinline__ uint4 lds128(const uint8_t* at) { return *reinterpret_cast<const uint4*>(at); }
__device__ __forceinline__ uint2 lds64(const uint8_t* at) { return *reinterpret_cast<const uint2*>(at); }
__device__ __forceinline__ uint32_t lds32(const uint8_t* at) { return *reinterpret_cast<const uint32_t*>(at); }

// Four codes of two units (nibbles j of both are the halves of word j) to values.  A code in
// bits 0-3 of a half is 1024 + code as the bits of an f16, in bits 4-7 with another
// exponent 64 + code; the difference is exact.
__device__ __forceinline__ void expand(uint32_t w, uint32_t scale, uint32_t minimum, uint32_t m1024, uint32_t m64,
                                       uint32_t (&v)[4]) {
  const uint32_t u = w >> 8;
  v[0] = fma_f16(add_f16(and_or<0x000f000fu>(w, m1024), 0xe400e400u), scale, minimum);
  v[1] = fma_f16(add_f16(and_or<0x00f000f0u>(w, m64), 0xd400d400u), scale, minimum);
  v[2] = fma_f16(add_f16(and_or<0x000f000fu>(u, m1024), 0xe400e400u), scale, minimum);
  v[3] = fma_f16(add_f16(and_or<0x00f000f0u>(u, m64), 0xd400d400u), scale, minimum);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_q4_kernel(const __grid_constant__ Q4Params qp) {
  using L = Slot<D>;
  constexpr int G = D / 32, NS = D / 128, N = kEntries;
  const PagedParams& p = qp.p;
  extern __shared__ __align__(1024) uint8_t raw[];
  Head& h = *reinterpret_cast<Head*>(raw);
  uint8_t* const q_s = raw + kHeadBytes;          // K-major: slabs of 128 channels of the first codes, of the second; sums
  uint8_t* const p_s = q_s + L::kQ;
  uint8_t* const ring = p_s + 2 * kPBytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int* abrt = &h.abort;
  if (tid == 0) {
    for (int i = 0; i < qp.n_slots; ++i) {
      bar_init(&h.code_full[i], 1);
      bar_init(&h.code_empty[i], kCodeWarps);     // four warps read its K, four its V
    }
    bar_init(&h.k_full, kCodeWarps);
    bar_init(&h.k_empty, 1);
    bar_init(&h.s_full, 1);
    bar_init(&h.s_empty, 4);
    for (int i = 0; i < 2; ++i) {
      bar_init(&h.p_full[i], 4);
      bar_init(&h.pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(&h.v_full[0][0] + i, 4);
      bar_init(&h.v_empty[0][0] + i, 1);
      bar_init(&h.row_full[i], 2);
    }
    bar_init(&h.q_full, 2);
    bar_init(&h.q_free, 1);
    bar_init(&h.o_free, 4);
    bar_init(&h.mma_done, 2);
    h.abort = 0;
    bar_init_fence();
  }
  if (warp == kLogitWarp) tmem_alloc(&h.tmem, kTmemCols);
  if (warp == kCopyWarp && lane < 3) prefetch_map(lane == 0 ? &qp.k : lane == 1 ? &qp.v : &qp.r);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = h.tmem;
  grid_dependency_wait();
  grid_dependency_release();
  const Start st = find_run<kThreads, kKT>(p, p.mt, blockIdx.x, gridDim.x, h.scan, &h.start);
  Cursor<kKT> c;
  c.begin(p, p.mt, st);
  if (tid == 32 * kSoftWarp) h.start = st;   // for the end (this thread's): registers are short
  if (st.n == 0) {
    if (tid == 0) p.parts[blockIdx.x] = PagedPart{};
  } else if (warp < kCodeWarps) {
    // ------------------------------------------------------------ codes to values
    const int part = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    uint32_t m1024 = 0x64006400u, m64 = 0x54005400u;   // kept in registers
    asm volatile("" : "+r"(m1024), "+r"(m64));
    // K: the thread's key is row kr of half kh; the warp's half of the channels is that of units n in [4 part, 4 part + 4).
    const int kh = quarter >> 1, kr = 32 * (quarter & 1) + lane;
    // V: units n of block g, or of blocks g and g + 1 (head_dim 256): of each 16 keys rows 2 j,
    // 2 j + 1, 2 j + 8 and 2 j + 9, whose codes lie in different banks.
    const int a8 = lane >> 2, j2 = 2 * (lane & 3), vn = 2 * quarter + (a8 >> 2), vg = (D == 256 ? 2 : 1) * (a8 & 3);
    int slot = 0;        // of the tile's first half; the second is the next
    uint32_t use = 0;
    int g = 0;           // tiles done
    for (bool more = true; more; more = c.next(p, p.mt)) {
      const ItemRows ir = item_rows(p, c);
      const int T = c.x1 - c.x;
#pragma unroll 1
      for (int j = 0; j < T; ++j, ++g) {
        int other = slot + 1;
        uint32_t other_use = use;
        if (other == qp.n_slots) other = 0, ++other_use;
        {
          const int sk = kh ? other : slot;
          wait(&h.code_full[sk], (kh ? other_use : use) & 1, abrt);
          __syncwarp();
          const uint8_t* const at = ring + sk * L::kBytes;
          uint32_t w[2 * G], pair[G / 2][2];   // four units n of G blocks; scales and minima of two blocks
#pragma unroll
          for (int i = 0; i < G / 2; ++i) {
            const uint4 x = lds128(at + swizzled<L::kRow>(kr, part * (G / 2) + i));
            w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
          }
#pragma unroll
          for (int i = 0; i < G / 4; ++i) {
            const uint4 x = lds128(at + 2 * L::kCodes + swizzled<L::kRecord>(kr, i));
            pair[2 * i][0] = __byte_perm(x.x, x.y, 0x5410), pair[2 * i][1] = __byte_perm(x.x, x.y, 0x7632);
            pair[2 * i + 1][0] = __byte_perm(x.z, x.w, 0x5410), pair[2 * i + 1][1] = __byte_perm(x.z, x.w, 0x7632);
          }
          __syncwarp();
          if (lane == 0) bar_arrive(&h.code_empty[sk]);
          if (g > 0) wait(&h.k_empty, (uint32_t)(g - 1) & 1, abrt);
          __syncwarp();
          fence_after();
          if (part == 0) {
            if constexpr (D == 256) h.scale[g & 3][32 * quarter + lane] = make_uint4(pair[0][0], pair[1][0], pair[G / 2 - 2][0], pair[G / 2 - 1][0]);
            else h.scale[g & 3][32 * quarter + lane] = make_uint4(pair[0][0], pair[1][0], 0u, 0u);
          }
          // The minima twice, for both halves of q's sums.
          const uint32_t at_min = lanes + kMinCol + 4u * part;
          if constexpr (D == 256) tmem_st4(at_min, pair[0][1], pair[1][1], pair[G / 2 - 2][1], pair[G / 2 - 1][1]);
          else if (part == 0) tmem_st4(at_min, pair[0][1], pair[1][1], pair[0][1], pair[1][1]);
          else tmem_st4(at_min, 0u, 0u, 0u, 0u);
          // Words i + G / 2 n of w are units n of blocks 2 i and 2 i + 1; cells of a block: of two units nibbles 0 and
          // 2, then 1 and 3.
#pragma unroll
          for (int i = 0; i < G / 2; ++i)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t x = __byte_perm(w[i], w[i + G / 2], b ? 0x7632 : 0x5410), y = __byte_perm(w[i + G], w[i + G + G / 2], b ? 0x7632 : 0x5410);
              tmem_st4(lanes + kKCol + (uint32_t)(8 * (2 * i + b) + 4 * part), x & 0x0f0f0f0fu, (x >> 4) & 0x0f0f0f0fu,
                       y & 0x0f0f0f0fu, (y >> 4) & 0x0f0f0f0fu);
            }
          tmem_st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&h.k_full);
        }
        const int sv = part ? other : slot, vb = g & 1;
        wait(&h.code_full[sv], (part ? other_use : use) & 1, abrt);
        __syncwarp();
        const uint8_t* const at = ring + sv * L::kBytes + L::kCodes;
        const uint8_t* const rec = at + L::kCodes;
        const int t0 = c.tiles.token(c.x + j) + kHalfKeys * part;
        // Tokens that no row sees become zeros: each of the four warps clears their records.
        if (t0 + kHalfKeys - 1 > ir.last || (p.window > 0 && t0 <= ir.first - p.window && t0 + kHalfKeys > p.n_sinks)) {
          uint8_t* const mine = ring + sv * L::kBytes + 2 * L::kCodes;
#pragma unroll 1
          for (int r = lane; r < kHalfKeys; r += 32) {
            const int t = t0 + r;
            if (t <= ir.last && (p.window == 0 || t > ir.first - p.window || t < p.n_sinks)) continue;
#pragma unroll
            for (int x = 0; x < NS; ++x)
              *reinterpret_cast<uint4*>(mine + swizzled<L::kRecord>(r, NS + x)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_async_smem();   // (copies will write there again)
          __syncwarp();
        }
#pragma unroll
        for (int i2 = 0; i2 < kHalfKeys / 32; ++i2) {
          uint32_t cell[NS][2][8];
#pragma unroll
          for (int i1 = 0; i1 < 2; ++i1) {
            uint32_t w[4], lo[4], hi[4];   // units; records of block g (and, head_dim 256, g + 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = 32 * i2 + 16 * i1 + j2 + (e & 1) + 8 * (e >> 1);
              if constexpr (D == 256) {
                w[e] = lds32(at + swizzled<L::kRow>(r, vn) + 2 * vg);
                const uint2 x = lds64(rec + swizzled<L::kRecord>(r, 2 + (vg >> 2)) + 4 * (vg & 3));
                lo[e] = x.x, hi[e] = x.y;
              } else {
                w[e] = *reinterpret_cast<const uint16_t*>(at + swizzled<L::kRow>(r, vn >> 1) + 8 * (vn & 1) + 2 * vg);
                lo[e] = lds32(rec + swizzled<L::kRecord>(r, 1) + 4 * vg);
                hi[e] = 0u;
              }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {   // keys 0, 1 and 2, 3: columns 2 j and 2 j + 1
#pragma unroll
              for (int b = 0; b < NS; ++b) {
                const uint32_t r0 = b ? hi[2 * k] : lo[2 * k], r1 = b ? hi[2 * k + 1] : lo[2 * k + 1];
                uint32_t v[4];
                expand(__byte_perm(w[2 * k], w[2 * k + 1], b ? 0x7632 : 0x5410), __byte_perm(r0, r1, 0x5410),
                       __byte_perm(r0, r1, 0x7632), m1024, m64, v);
                cell[b][0][4 * i1 + k] = v[0], cell[b][0][4 * i1 + 2 + k] = v[1];
                cell[b][1][4 * i1 + k] = v[2], cell[b][1][4 * i1 + 2 + k] = v[3];
              }
            }
          }
          if (i2 == kHalfKeys / 32 - 1) {
            __syncwarp();
            if (lane == 0) bar_arrive(&h.code_empty[sv]);
          }
          if (i2 == 0) {
            if (g >= 2) wait(&h.v_empty[part][vb], (uint32_t)((g - 2) >> 1) & 1, abrt);
            __syncwarp();
            fence_after();
          }
#pragma unroll
          for (int b = 0; b < NS; ++b)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              tmem_st_fragments(lanes + ((uint32_t)(16 * x) << 16) + kVCol + (uint32_t)(128 * vb + 64 * b + 32 * part + 16 * i2), cell[b][x]);
        }
        tmem_st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&h.v_full[part][vb]);
        slot = other + 1;
        use = other_use;
        if (slot == qp.n_slots) slot = 0, ++use;
      }
    }
  } else if (warp < kCopyWarp) {
    // ------------------------------------------------------------ softmax and output
    // A thread owns a key of a tile, and a channel of each slab of the output.
    const int quarter = warp & 3, me = tid & 127;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    // Where the key's weights lie: V's keys of each 16 are in the order of its fragments.
    const int key = 32 * (quarter & 1) + lane;
    const int at_k = (key & 48) | ((key & 6) << 1) | ((key & 8) >> 2) | (key & 1);
    const int to_p = (quarter >> 1) * (kPBytes / 2) + (((at_k >> 3) << 4) | ((at_k & 7) << 1));
    const int channel = (D == 256 ? 64 : 32) * (lane & 3) + 4 * (2 * quarter + ((lane >> 2) & 1)) + (lane >> 3);   // (and 32 further)
    int g = 0, it = 0;   // tiles and items done
    for (bool more = true; more;) {
      const ItemRows ir = item_rows(p, c);
      const int T = c.x1 - c.x;
      const bool whole = c.whole();
      const bool mine = me < ir.nf;   // the thread has a column's statistics, too
      wait(&h.row_full[it & 3], (uint32_t)(it >> 2) & 1, abrt);
      if (me < N) {
        const int e = me, f = ir.f0 + min(e, ir.nf - 1), r = row_of(p, f);
        // (The factor is not 0: hidden logits are -infinity times it.)
        h.vote[e] = h.column[e] = mine ? make_float2(fmaxf(h.q[it & 3][e] * (p.scale * kLog2e), 1e-37f), kUnset) : make_float2(0.f, -1000.f);
        h.ref[e] = -INFINITY;
        h.base[e] = 0.f;
        if (e == 0) h.far = 0;
        h.pos[e] = ir.pos0 + r;
        h.to[e] = (whole ? (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f - r * p.group)
                         : (int64_t)c.slot(blockIdx.x) * p.mt + e) * D;
      }
      soft_sync();
      // Eight columns' factors and shifts.
      float2 k[8];
      auto columns = [&](const float2* of) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 two = *reinterpret_cast<const float4*>(of + e);
          k[e] = make_float2(two.x, two.y), k[e + 1] = make_float2(two.z, two.w);
        }
      };
      float l[N];
#pragma unroll
      for (int e = 0; e < N; ++e) l[e] = 0.f;
#pragma unroll 1
      for (int j = 0; j < T; ++j, ++g) {
        const int buf = g & 1, t0 = c.tiles.token(c.x + j);
        wait(&h.s_full, (uint32_t)g & 1, abrt);
        __syncwarp();
        fence_after();
        // The blocks' sums times their scales (codes are times 2^-9), and the minima's part (sums are over 16):
        // three at a time in registers.
        const uint4 sc = h.scale[g & 3][32 * quarter + lane];
        const uint32_t bad = h.bad[g & 15][0] | (uint32_t)h.bad[g & 15][1] << 4;
        const uint32_t scales[4] = {sc.x, sc.y, sc.z, sc.w};
        float z[N];
#pragma unroll
        for (int e = 0; e < N; ++e) z[e] = 0.f;
        constexpr int kAtOnce = 3;
#pragma unroll
        for (int i0 = 0; i0 <= G; i0 += kAtOnce) {
          float part[kAtOnce][N];
#pragma unroll
          for (int i = 0; i < kAtOnce && i0 + i <= G; ++i)
#pragma unroll
            for (int x = 0; x < N; x += 8) tmem_ld8_start(lanes + kSCol + (uint32_t)(N * (i0 + i) + x), part[i] + x);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kAtOnce && i0 + i <= G; ++i)
#pragma unroll
            for (int x = 0; x < N; x += 8) tmem_ld_done(part[i] + x);
          if (i0 + kAtOnce > G) {
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(&h.s_empty);
          }
#pragma unroll
          for (int i = 0; i < kAtOnce && i0 + i <= G; ++i) {
            const int u = i0 + i;
            const float2 two = __half22float2(*reinterpret_cast<const __half2*>(&scales[u / 2 % 4]));
            const float f = u == G ? 16.f : 512.f * (u & 1 ? two.y : two.x);
#pragma unroll
            for (int e = 0; e < N; e += 2) fma2(z[e], z[e + 1], f, f, part[i][e], part[i][e + 1]);
          }
        }
        // Tiles that every row sees whole are the rule.
        if (bad != 0u || t0 + kKT - 1 > ir.first || (p.window > 0 && t0 <= ir.last - p.window && t0 + kKT > p.n_sinks)) {
          const int tk = t0 + 32 * quarter + lane;
          const bool gone = (bad >> (2 * quarter + (lane >> 4))) & 1u;
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (gone || !sees(p, h.pos[e], tk)) z[e] = -INFINITY;
        }
        // Whether a weight would be larger than the reference leaves room for.
        float most = -INFINITY;
#pragma unroll
        for (int x = 0; x < N; x += 8) {
          columns(h.vote + x);
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = fmaf(z[x + e], k[e].x, k[e].y);
#pragma unroll
          for (int n = 4; n >= 1; n >>= 1)
#pragma unroll
            for (int e = 0; e < n; ++e) y[e] = fmaxf(y[e], y[n + e]);
          most = fmaxf(most, y[0]);
        }
        if (soft_any(most > kTop + kLag)) {
#pragma unroll
          for (int x = 0; x < N; x += 8) {
            const float top = reduce_columns(z + x, lane, [](float a, float b) { return fmaxf(a, b); });
            if ((lane & 3) == 0) h.mx[quarter][x + (lane >> 2)] = top;
          }
          soft_sync();
          if (me < N) {
            const int e = me;   // (threads 0 to 15 have a column each)
            float factor = 1.f;
            if (mine) {
              const float top = fmaxf(fmaxf(h.mx[0][e], h.mx[1][e]), fmaxf(h.mx[2][e], h.mx[3][e]));
              const float old = h.ref[e], need = ceilf(top * h.column[e].x);
              const float now = top == -INFINITY ? old : old == -INFINITY || need > old + kLag ? need : old;
              if (fabsf(now) <= kFar) {
                if (old != -INFINITY && now != old) factor = ex2(old - now);
                h.ref[e] = now;
                h.base[e] = 0.f;
                h.vote[e].y = h.column[e].y = kTop - now;
              } else {
                factor = far_reference(h, e, top);
              }
            }
            h.factor[e] = factor;
          }
          soft_sync();
#pragma unroll
          for (int e = 0; e < N; ++e) l[e] *= h.factor[e];
          if (__builtin_expect(h.far != 0, 0)) {
#pragma unroll
            for (int e = 0; e < N; ++e) z[e] -= h.base[e];
          }
          if (j > 0) {   // the output as well
            wait(&h.pv_done[buf ^ 1], (uint32_t)((g - 1) >> 1) & 1, abrt);
            __syncwarp();
            fence_after();
#pragma unroll 1
            for (int x = 0; x < NS * N; x += 8) {
              const int b = x >= N ? 1 : 0, x0 = x - b * N;
              const uint32_t at = lanes + kOCol + (uint32_t)(N * b + x0);
              float o[8];
              uint32_t w[8];
              tmem_ld8_start(at, o);
              tmem_ld_wait();
              tmem_ld_done(o);
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(o[e] * h.factor[x0 + e]);
              tmem_st8(at, w);
            }
            tmem_st_wait();
          }
        }
        if (g >= 2) wait(&h.pv_done[buf], (uint32_t)((g - 2) >> 1) & 1, abrt);   // the buffer's weights have been used
        uint8_t* const to = p_s + buf * kPBytes;
        uint32_t w2[N / 2];
#pragma unroll
        for (int x = 0; x < N; x += 8) {   // (all before the stores, which the loads would wait behind)
          columns(h.column + x);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float a = ex2(fmaf(z[x + e], k[e].x, k[e].y)), b = ex2(fmaf(z[x + e + 1], k[e + 1].x, k[e + 1].y));
            l[x + e] += a;
            l[x + e + 1] += b;
            w2[(x + e) / 2] = pack_f16(a, b);
          }
        }
#pragma unroll
        for (int e = 0; e < N; ++e)
          *reinterpret_cast<uint16_t*>(to + (to_p ^ ((e & 7) << 4)) + e * 128) = (uint16_t)(e & 1 ? w2[e / 2] >> 16 : w2[e / 2]);
        fence_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&h.p_full[buf]);
      }
      // The item's result, or this run's part of it.
#pragma unroll
      for (int x = 0; x < N; x += 8) {
        const float sum = reduce_columns(l + x, lane, [](float a, float b) { return a + b; });
        if ((lane & 3) == 0) h.sums[quarter][x + (lane >> 2)] = sum;
      }
      soft_sync();
      if (mine) {
        const int e = me;
        const float sum = (h.sums[0][e] + h.sums[1][e]) + (h.sums[2][e] + h.sums[3][e]);
        h.inv[e] = sum == 0.f ? 0.f : 1.f / sum;   // (NaN stays)
        const float lse2 = sum == 0.f ? -INFINITY : h.ref[e] - kTop + log2f(sum);
        if (!whole) p.part_lse[h.to[e] / D] = lse2;
        else if (p.lse) p.lse[h.to[e] / D] = lse2 * kLn2;
      }
      soft_sync();
      wait(&h.pv_done[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1, abrt);
      __syncwarp();
      fence_after();
      const bool f32 = !whole || p.out_dtype == QSA_F32;
      float* const to32 = (whole ? static_cast<float*>(p.out) : p.part_o) + channel;
      __nv_bfloat16* const to16 = static_cast<__nv_bfloat16*>(p.out) + channel;
#pragma unroll 1
      for (int x = 0; x < ir.nf; x += 8) {
        float o[NS][8];
#pragma unroll
        for (int b = 0; b < NS; ++b) tmem_ld8_start(lanes + kOCol + (uint32_t)(N * b + x), o[b]);
        tmem_ld_wait();
#pragma unroll
        for (int b = 0; b < NS; ++b) tmem_ld_done(o[b]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (x + e >= ir.nf) break;
          const float inv = h.inv[x + e];
          const int64_t at = h.to[x + e];
#pragma unroll
          for (int b = 0; b < NS; ++b) {
            if (f32) to32[at + 32 * b] = o[b][e] * inv;
            else to16[at + 32 * b] = __float2bfloat16_rn(o[b][e] * inv);
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&h.o_free);
      soft_sync();   // the columns are the next item's
      ++it;
      more = c.next(p, p.mt);
      if (!more && tid == 32 * kSoftWarp) describe_part(p, c, h.start, blockIdx.x);   // (still at its last item)
    }
  } else if (warp == kCopyWarp) {
    // ------------------------------------------------------------ copies
    // A lane a box of tokens: its K, V and records.  The table's entries come a warp's lanes
    // at a time, the next ones while these are under way.
    const int box = min(1 << p.page_shift, kHalfKeys), n_box = kHalfKeys / box, page_mask = (1 << p.page_shift) - 1;
    const int per = 32 / n_box;   // slots of a look-up (4 boxes at most: 8 to 32)
    const int my_box = lane % n_box, my_slot = lane / n_box;
    int slot = 0, total = 0;
    uint32_t use = 0;
    int gt = 0;                   // tiles done
    bool live = true;
    for (bool more = true; more && live; more = c.next(p, p.mt)) {
      const ItemRows ir = item_rows(p, c);
      const int n = 2 * (c.x1 - c.x);   // slots
      auto token_of = [&](int i, int b) { return c.tiles.token(c.x + (i >> 1)) + kHalfKeys * (i & 1) + b * box; };
      auto wanted = [&](int t) {   // whether the box at token t holds a visible one
        return t <= ir.last && (p.window == 0 || t + box - 1 > ir.first - p.window || t < p.n_sinks);
      };
      // -2: not wanted.
      auto look_up = [&](int i) {
        if (i >= n) return -2;
        const int t = token_of(i, my_box);
        if (!wanted(t)) return -2;
        const int64_t s = (int64_t)t >> p.page_shift;
        return s < p.table_ld ? max(__ldcg(p.table + c.seq * p.table_ld + s), -1) : -1;
      };
      int pages = look_up(my_slot);
#pragma unroll 1
      for (int i0 = 0; i0 < n && live; i0 += per) {
        const int next = look_up(i0 + per + my_slot);
#pragma unroll 1
        for (int i = i0; i < min(i0 + per, n); ++i) {
          if (use > 0 && !wait(&h.code_empty[slot], (use - 1) & 1, abrt)) live = false;
          live = __all_sync(0xffffffffu, live);
          if (!live) break;
          const bool copies = lane < n_box;
          int page = __shfl_sync(0xffffffffu, pages, (i - i0) * n_box + my_box);
          const bool missing = copies && page != -2 && (uint32_t)page >= (uint32_t)p.n_pages;
          if ((uint32_t)page >= (uint32_t)p.n_pages) page = p.n_pages;   // past the last page: zeros
          const uint32_t bad = __reduce_or_sync(0xffffffffu, missing ? ((1u << (box / 16)) - 1u) << (lane * (box / 16)) : 0u);
          if (missing) atomicAdd(&g_bad_pages, 1);
          if (lane == 0) {
            h.bad[gt & 15][i & 1] = (uint8_t)bad;
            bar_expect_tx(&h.code_full[slot], L::kBytes);
          }
          __syncwarp();
          if (copies) {
            const uint32_t to = smem_addr(ring) + slot * L::kBytes;
            const int token = token_of(i, lane) & page_mask;
            tma_4d(to + lane * box * L::kRow, &qp.k, 0, token, c.head, page, &h.code_full[slot]);
            tma_4d(to + L::kCodes + lane * box * L::kRow, &qp.v, 0, token, c.head, page, &h.code_full[slot]);
            tma_4d(to + 2 * L::kCodes + lane * box * L::kRecord, &qp.r, 0, token, c.head, page, &h.code_full[slot]);
          }
          __syncwarp();
          gt += i & 1;
          ++total;
          if (++slot == qp.n_slots) slot = 0, ++use;
        }
        pages = next;
      }
    }
    // Every copy has landed before the CTA ends: a lane a slot, the last one that went there.
    if (lane < qp.n_slots && lane < total) {
      const int last = total - 1 - (total - 1 - lane) % qp.n_slots;
      bar_wait(&h.code_full[lane], (uint32_t)(last / qp.n_slots) & 1, &g_timeouts);
    }
  } else if (warp == kLogitWarp) {
    // ------------------------------------------------------------ logits
    // The whole warp walks through the tiles with values that are the same in all its
    // lanes, and one lane issues.
    const bool leader = elect_one();
    // 32-bit accumulators, both K-major, M = 128; E4M3 and f16 operands are both 0, E5M2 (B: bits 10-12) is 1.
    constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24), kIdescHi = kIdesc | (1u << 10);
    const uint64_t q_desc = desc_sw128(q_s, 16, 1024);
    constexpr uint32_t kSlab = L::kQSlab >> 4;
    int g = 0, it = 0;
    bool live = true;   // no wait of this CTA has given up: nothing is issued after one has
    for (bool more = true; more; more = __shfl_sync(0xffffffffu, (int)c.next(p, p.mt), 0) != 0, ++it) {
      const int T = __shfl_sync(0xffffffffu, c.x1 - c.x, 0);
      live = __all_sync(0xffffffffu, wait(&h.q_full, (uint32_t)it & 1, abrt) && live);
#pragma unroll 1
      for (int j = 0; j < T; ++j, ++g) {
        if (g > 0) live = __all_sync(0xffffffffu, wait(&h.s_empty, (uint32_t)(g - 1) & 1, abrt) && live);
        live = __all_sync(0xffffffffu, wait(&h.k_full, (uint32_t)g & 1, abrt) && live);
        fence_after();
        if (leader && live) {
#pragma unroll
          for (int x = 0; x < G; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y)   // both codes of q
              mma_f8_ts(tmem + kSCol + (uint32_t)(N * x), tmem + kKCol + 8u * x, q_desc + (uint32_t)(NS * y + (x >> 2)) * kSlab + 2 * (x & 3),
                        y ? kIdesc : kIdescHi, (uint32_t)y);
          mma_f16_ts(tmem + kSCol + (uint32_t)(N * G), tmem + kMinCol, q_desc + 2 * NS * kSlab, kIdesc, 0u);
          commit(&h.k_empty);
          commit(&h.s_full);
          if (j + 1 == T) commit(&h.q_free);
        }
        __syncwarp();
      }
    }
    if (leader) commit(&h.mma_done);   // every MMA has completed before TMEM is released
    __syncwarp();
    bar_wait(&h.mma_done, 0u, &g_timeouts);
  } else {
    // ------------------------------------------------------------ Q
    // An E5M2 and an E4M3 code of each value (see above) and the sums of its blocks, a row's 16
    // channels a lane, in the order of K's cells: of channels 8 i .. 8 i + 7 the bytes are
    // 0, 2, 4, 6, 1, 3, 5, 7.  (The first item's with the warp that has no output to issue yet.)
    constexpr int kLanes = D / 16, kRows = 32 / kLanes, kBatch = 8 / kRows;   // 16 rows of two warps
    const int chunk = lane % kLanes;
    auto queries = [&](int it, int first, int warps) {
      const ItemRows ir = item_rows(p, c);
      if (it > 0) wait(&h.q_free, (uint32_t)(it - 1) & 1, abrt);
      __syncwarp();
#pragma unroll 1
      for (int r0 = first * kRows + lane / kLanes; r0 < N; r0 += kBatch * warps * kRows) {
        uint4 a[kBatch], b[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int f = ir.f0 + min(r0 + x * warps * kRows, ir.nf - 1), r = row_of(p, f);
          const int64_t entry = (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f - r * p.group);
          const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + entry * D + 16 * chunk);
          a[x] = __ldg(from);
          b[x] = __ldg(from + 1);
        }
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int row = r0 + x * warps * kRows;
          const uint32_t w[8] = {a[x].x, a[x].y, a[x].z, a[x].w, b[x].x, b[x].y, b[x].z, b[x].w};
          uint32_t most = 0u;
#pragma unroll
          for (int e = 0; e < 8; ++e) most = max(most, max((w[e] << 16) & 0x7fff0000u, w[e] & 0x7fff0000u));
#pragma unroll
          for (int o = kLanes / 2; o >= 1; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
          // 2^(exponent - 11), at least 2^-100: a row of smaller values keeps fewer bits.
          const int e = max((int)(most >> 23) - 127 - 11, -100);
          const float up = row < ir.nf ? __uint_as_float((uint32_t)(127 - e) << 23) : 0.f;
          const bool odd = most >= 0x7f800000u;   // infinity or NaN: the row's logits are NaN
          uint32_t hi[4], lo[4];
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // bytes 4 i .. 4 i + 3: words 4 (i / 2) on, their low halves or their high ones
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t x2 = w[4 * (i >> 1) + k];
              v[k] = (i & 1 ? bf16_hi(x2) : bf16_lo(x2)) * up;
              sum += v[k];
            }
            const uint32_t c0 = to_e5m2x2(v[0], v[1]), c1 = to_e5m2x2(v[2], v[3]);
            const float2 d0 = from_e5m2x2(c0), d1 = from_e5m2x2(c1);
            hi[i] = c0 | c1 << 16;
            lo[i] = to_e4m3x2(v[0] - d0.x, v[1] - d0.y) | to_e4m3x2(v[2] - d1.x, v[3] - d1.y) << 16;
            if (odd) hi[i] = lo[i] = 0x7f7f7f7fu;   // NaN of both kinds
          }
          sum = 0.0625f * (sum + __shfl_xor_sync(0xffffffffu, sum, 1));
          const __half s_hi = __float2half_rn(odd ? __uint_as_float(0x7fffffffu) : sum), s_lo = __float2half_rn(sum - __half2float(s_hi));
          const int swap = row & 7;
          uint8_t* const to = q_s + row * 128;
          *reinterpret_cast<uint4*>(to + (chunk >> 3) * L::kQSlab + (((chunk & 7) ^ swap) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to + (NS + (chunk >> 3)) * L::kQSlab + (((chunk & 7) ^ swap) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          // Sums: the high halves of the blocks, their low ones, zeros (head_dim 128) up to 16.
          uint8_t* const to_sum = to + 2 * NS * L::kQSlab;
          const int block = chunk >> 1;
          if ((chunk & 1) == 0) {
            const int x0 = block, x1 = G + block;
            *reinterpret_cast<__half*>(to_sum + (((x0 >> 3) ^ swap) << 4) + 2 * (x0 & 7)) = s_hi;
            *reinterpret_cast<__half*>(to_sum + (((x1 >> 3) ^ swap) << 4) + 2 * (x1 & 7)) = s_lo;
          } else if (D == 128 && block == 0) {
            *reinterpret_cast<uint4*>(to_sum + ((1 ^ swap) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          if (chunk == 0) h.q[it & 3][row] = odd ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
        }
      }
      fence_async_smem();
      __syncwarp();
      for (int x = warps; x <= 2 && lane == 0; ++x) {   // (two arrivals)
        bar_arrive(&h.row_full[it & 3]);
        bar_arrive(&h.q_full);
      }
    };
    if (warp == kOutWarp) queries(0, 1, 2);
    else
      for (int it = 0, more = 1; more; more = c.next(p, p.mt), ++it) queries(it, 0, it == 0 ? 2 : 1);
    if (warp == kOutWarp) {
      // ---------------------------------------------------------- output
      const bool leader = elect_one();
      constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
      const uint64_t p_desc = desc_sw128(p_s, 16, 1024);
      int g = 0, it = 0;
      bool live = true;
      for (bool more = true; more; more = __shfl_sync(0xffffffffu, (int)c.next(p, p.mt), 0) != 0, ++it) {
        const int T = __shfl_sync(0xffffffffu, c.x1 - c.x, 0);
#pragma unroll 1
        for (int j = 0; j < T; ++j, ++g) {
          const int buf = g & 1, vb = g & 1;
          live = __all_sync(0xffffffffu, wait(&h.p_full[buf], (uint32_t)(g >> 1) & 1, abrt) && live);
          if (j == 0 && it > 0) live = __all_sync(0xffffffffu, wait(&h.o_free, (uint32_t)(it - 1) & 1, abrt) && live);
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            live = __all_sync(0xffffffffu, wait(&h.v_full[a][vb], (uint32_t)(g >> 1) & 1, abrt) && live);
            fence_after();
            if (leader && live) {
#pragma unroll
              for (int b = 0; b < NS; ++b)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  mma_f16_ts(tmem + kOCol + (uint32_t)(N * b), tmem + kVCol + 128u * vb + 64u * b + 32u * a + 8u * x,
                             p_desc + (uint32_t)(2 * buf + a) * (kPBytes >> 5) + 2 * x, kIdesc, (j | a | x) != 0 ? 1u : 0u);
              commit(&h.v_empty[a][vb]);
              if (a == 1) commit(&h.pv_done[buf]);
            }
            __syncwarp();
          }
        }
      }
      if (leader) commit(&h.mma_done);
      __syncwarp();
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == kLogitWarp) {
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
  using L = Slot<D>;
  Q4Params qp{};
  qp.p = p;
  if (!encode_rows(&qp.k, p.k, p, L::kRow, kHalfKeys, p.tok_stride / 2, p.head_stride / 2, p.page_stride / 2) ||
      !encode_rows(&qp.v, p.v, p, L::kRow, kHalfKeys, p.tok_stride / 2, p.head_stride / 2, p.page_stride / 2) ||
      !encode_rows(&qp.r, p.kv_scale, p, L::kRecord, kHalfKeys, p.s_tok_stride * L::kRecord, p.s_head_stride * L::kRecord,
                   p.s_page_stride * L::kRecord))
    return cudaErrorInvalidValue;
  constexpr int fixed = kHeadBytes + L::kQ + 2 * kPBytes;
  qp.n_slots = std::min((kSmemLimit - fixed) / L::kBytes, kMaxSlots);
  const size_t smem = (size_t)fixed + (size_t)qp.n_slots * L::kBytes;
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
