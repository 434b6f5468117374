// Attention over a paged K/V cache on the 5th-generation tensor cores: bf16 and
// fp8 caches, and 4-bit caches of calls of more than 16 entries (see qsa_paged.cuh for
// the division of the work into runs of key tiles, and qsa_paged.cu for the formulas and
// the joining launch).
//
// An item's MT <= 128 entries (query row, head of the KV head's group) are the
// M rows of both products, 128 keys a tile:
//   S_j = Q K_j^T     tcgen05.mma, M = 128, N = 128, K = head_dim; two S buffers of
//                     128 TMEM columns, so the next tile's logits are computed
//                     while this one's softmax runs; Q in TMEM (head_dim 128) or in
//                     shared memory (256), K in shared memory;
//   P_j = exp(S_j - m), rounded to bf16, over S_j's own columns in TMEM;
//   O  += P_j V_j     M = 128, N = 128 channels a slab, K = 128 keys, P from TMEM and
//                     V from shared memory (MN-major), O in 128 or 256 TMEM columns.
// Two groups of four softmax warps take 64 keys each of every tile; a thread owns
// one entry, so row statistics need one exchange with the thread of the other
// group and no shuffles, and its 64 logits stay in registers.  (Tiles of 128 keys
// in turn between the groups: the chain logits - weights - output of a tile, which
// two tiles in flight have to cover, was 3,300 cycles for head_dim 128; with that,
// 2,048 rows over 16k tokens took 303 us and this way 296, the ragged fp8 batch 181
// and 172.)
// The maximum m is only moved, and O rescaled, when a logit exceeds
// it by more than 2^8 in the weight: weights stay below 2^8, which the 32-bit sums
// and bf16's exponent hold as well as 1, and the quotient by l is the same.
//
// K and V come through TMA, 128 channels x 128 tokens (32 KB) a slab, one tensor
// copy for each page and 64 channels (pages of 128 tokens and more: one a slab),
// into rings of as many slabs as fit beside Q.  Copies of pages without visible
// tokens are aimed past the last page, which fills zeros without reading.
// Slots of V that belong to no visible token are cleared before the product, as
// 0 x NaN would reach O.  With fewer than 128 entries the rows behind Q's in the
// MMA read whatever lies there: rows of a product do not mix, and theirs are
// not read.
//
// fp8 caches: the logits' product takes K's codes as they are, against Q as the
// sum of two 8-bit codes a value, E5M2 and E4M3 (as many bytes, and as much time,
// as one bf16 product), and K's scales times the logit scale are applied to S by
// column; V's codes become bf16 in shared memory, and V's scales go with the
// weights, which are rounded once.  (That step, from K through bf16 as well, took a
// ragged batch of 16 sequences from 351 to 230 us; later ones to 172.)
//
// 4-bit caches: codes and records go through rings of their own, and eight warps write
// them to the slabs as f16, code * scale + minimum rounded once (f16 keeps 2^-11 of a
// value; rows that were bf16 have no two values in a block that differ by less than 2^-8
// of its largest, so that neither rounding makes one of two), in the order that two
// masks of a code word give (each 8 channels as 0, 4, 1, 5, 2, 6, 3, 7; Q in the same
// order, and the output put back); Q is f16 times a power of two of each row (its largest
// magnitude to [2^14, 2^15): exact from 2^-31 of that on, off by at most 2^-39 of it
// below), and weights are f16 with 2^7 at the maximum, so that 2^15 is the largest.  From a
// maximum of 2^20 on, where units of a logit in binary32 come near what f16 has room for,
// it is taken off the logits before they are multiplied.
//
// Roles: warps 0-7 softmax and output, warps 8 and 10 copy K and V, warp 9 issues
// the MMAs; bf16: warp 11 copies Q and clears V's ends; fp8: warps 12-15 write Q's
// codes and the scales and convert V, with those of warps 0-7 that have no
// entries; 4-bit: warps 12-19 write Q, K and V, and registers move from the copying warps
// to the softmax's.  Every wait gives up after about two seconds (counted; nothing more
// is issued then, and the CTA runs to its end).
//
// What bounds it (us a call on one GB300, floor at the measured 6,791 GB/s and
// 1,941 TFLOP/s): few rows, the K/V bytes -- 261,120 tokens x 4 rows 89 of 79; the
// call's start and the joining launch are what a 65,536-token row (32 of 20) and a
// windowed batch of 64 (49 of 33) add.  2,048 rows: over 16k tokens (head_dim 128)
// 292 of 199, the tensor pipe 67% busy at the power limit; over a
// 4,096-token window (256) 170 of 108, the shared memory's 128 bytes a cycle, which
// Q and K take whole in the logits' product (2,700 cycles a tile where the products
// alone take 2,048).  fp8: 170 of 115, shared memory too: the products, V's conversion
// and the scales pass over it 3,200 cycles a tile where HBM needs 2,800.  4-bit: 2,048
// rows over 16k tokens 402 of 199 (bf16: 292): expanding 256 values a thread and tile beside the
// softmax (without its arithmetic 300 to 312); 261,120 tokens x 4 rows 90 of 25, shared
// memory, over which Q, the expanded values twice and the codes pass 2,900 cycles a tile,
// and slabs for one tile only, so that expanding and products take turns (without the
// arithmetic 68).
#include <math.h>

#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "qsa_attn_common.cuh"
#include "qsa_paged.cuh"
#include "qsa_tc.cuh"

namespace qsa {

namespace {

using namespace paged;
using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKT = 128;                      // keys of a tile
constexpr int kHalf = kKT * 128;              // bytes of 64 channels of a tile
constexpr int kSlab = 2 * kHalf;              // bytes of 128 channels: what the ring holds
constexpr int kMaxSlabs = 6;                 // of K, and of V
constexpr int kKeyWarp = 8, kMmaWarp = 9, kValueWarp = 10, kQWarp = 11, kCodeWarp = 12, kCodeWarps = 4;
constexpr int kSoftWarps = 8;
// How the cache holds K and V.
constexpr int kBf16 = 0, kFp8 = 1, kQ4 = 2;
// 4-bit caches: four more warps expand codes, 20 in all, with 96 registers a thread at
// launch (61,440).  The copying and issuing warpgroup leaves what the softmax's two need:
// 256 * 136 + 128 * 48 + 256 * 80 = 61,440.
constexpr int kQ4CodeWarps = 8;
constexpr int kQ4SoftRegs = 136, kQ4CopyRegs = 48, kQ4CodeRegs = 80;
__host__ __device__ constexpr int code_warps_of(int kind) { return kind == kBf16 ? 0 : kind == kQ4 ? kQ4CodeWarps : kCodeWarps; }
__host__ __device__ constexpr int threads_of(int kind) { return 32 * (kind != kBf16 ? kCodeWarp + code_warps_of(kind) : kQWarp + 1); }
template <int REGS, bool MORE>
__device__ __forceinline__ void set_registers() {
  if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(REGS));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(REGS));
}
constexpr int kCodeSlab = kKT * 128;          // bytes of the codes of a slab (fp8 caches)
constexpr int kMaxCodeSlabs = 4;             // of V
// 4-bit caches: a slot of codes is the K, or the V, of 32 (head_dim 256, where Q and the
// operands leave 32 KB) or 128 tokens, with their block scales and minima.
template <int D>
struct Q4Slot {
  static constexpr int kTokens = D == 256 ? 32 : 128;
  static constexpr int kCodes = kTokens * D / 2, kBytes = kCodes + kTokens * D / 8;
};
constexpr int kMaxQ4Slots = 8;               // of K, and of V
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemLimit = 227 * 1024;
constexpr float kMoveMax = 8.f;               // log2 of the weight at which the running maximum is moved

constexpr uint32_t kIdescS = idesc_bf16(128, kKT, false, false);
constexpr uint32_t kIdescO = idesc_bf16(128, 128, false, true);
// kind::f8f6f4 with a 32-bit accumulator: A, Q's second or first codes, is E4M3 or
// E5M2 (bits 7-9 = 0 or 1), B, K's codes, E4M3 (bits 10-12 = 0), both K-major.
constexpr uint32_t kIdescLo8 = (1u << 4) | ((uint32_t)(kKT >> 3) << 17) | (8u << 24);
constexpr uint32_t kIdescHi8 = kIdescLo8 | (1u << 7);
// kind::f16 with f16 operands (bits 7-9 and 10-12 = 0 where bf16 has 1).
constexpr uint32_t kF16Operands = ~((1u << 7) | (1u << 10));
constexpr float kFar = 1048576.f;             // f16 weights: maxima from here on are taken off the logits first
constexpr float kF16Weights = 7.f;            // log2 of the weight at the running maximum, f16 weights: 2^15 is the largest

__device__ int g_timeouts;
__device__ int g_bad_pages;

struct TcParams {
  // {64 channels, page_tokens, D / 64, Hkv, n_pages}: boxes of 64 channels x min(page_tokens, 128)
  // tokens, of two channel blocks where the page has 128 tokens.
  CUtensorMap k, v;
  CUtensorMap r;         // 4-bit: the records
  CUtensorMap q;         // {D, Hq, n_rows}: boxes of 64 channels x a KV head's query heads x an item's rows
  PagedParams p;
  int32_t n_k, n_v;              // slabs in the rings of K (fp8 caches: of codes) and V
  int32_t n_code_v;              // fp8 caches: slabs of V's codes; 4-bit: slots of K's, and of V's
};

// bar_wait with everything behind its first try out of line: the loops of the
// roles stay small (they share the instruction caches).
__device__ __noinline__ bool wait_slow(uint64_t* b, uint32_t parity, int* abort) {
  return bar_wait(b, parity, &g_timeouts, abort);
}
// (With registers moved between warpgroups the compiler takes no calls.)
template <bool INLINE>
__device__ __forceinline__ bool wait_for(uint64_t* b, uint32_t parity, int* abort) {
  if (bar_try(b, parity)) return true;
  if constexpr (INLINE) return bar_wait(b, parity, &g_timeouts, abort);
  else return wait_slow(b, parity, abort);
}

// Shared memory: this, then Q, then the ring (both on 1,024-byte boundaries).
// A wait by parity tells a phase from its neighbours only, so a waiting thread
// has to know the phase before the awaited one to be over.  pv_done comes in a
// pair, for even and odd tiles: tile j's logits follow the output product of
// tile j - NB or later ones, NB = 2, so whoever has seen them may wait for the
// product of tile j - 1, and after that for tile j's.
struct Head {
  uint64_t full[2][kMaxSlabs], empty[2][kMaxSlabs];   // K, V
  uint64_t v_ready[kMaxSlabs];                        // bf16: V, without what no row sees
  uint64_t s_full[2], p_full[2], pv_done[2], o_free, q_full, q_free, q_used, mma_done;
  uint64_t code_full[kMaxCodeSlabs], code_empty[kMaxCodeSlabs], sc_full[8];   // fp8 caches: V's codes, scales
  int64_t scan[16];
  Start start;
  uint32_t tmem;
  int abort;
  uint32_t bad[16];             // 16-token pieces of a tile that have no page (fewer are under way)
  float mx[2][2][128];          // maxima of an even and an odd tile, by group
  float sums[2][128];           // the two groups' sums of weights
  uint4 odd_scale[8][2];        // fp8 caches: a tile's K scales that are negative, or no number (see put_scales)
};
constexpr int kHeadBytes = 4 * 1024;
// fp8 caches: scales of the tiles in flight, behind the head.
struct Scales {
  float k[8][kKT];   // times the logit scale and log2(e)
  float v[8][kKT];
  float q[4][128];   // of an item's rows of Q: the power of two that its codes were divided by
};
// 4-bit caches: Q's powers of two, and the rings of codes.
struct Q4Head {
  float q[4][128];
  uint64_t code_full[2][kMaxQ4Slots], code_empty[2][kMaxQ4Slots];   // K, V
};
constexpr int kQ4HeadBytes = 3 * 1024;
static_assert(sizeof(Head) <= kHeadBytes && (kHeadBytes + sizeof(Scales)) % 1024 == 0, "shared memory head");
static_assert(sizeof(Q4Head) <= kQ4HeadBytes && (kHeadBytes + kQ4HeadBytes) % 1024 == 0, "shared memory head");
__host__ __device__ constexpr int extra_bytes(int kind) {
  return kind == kFp8 ? (int)sizeof(Scales) : kind == kQ4 ? kQ4HeadBytes : 0;
}

__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[smem] B[smem] of 8-bit types, 32 of K.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// As mma_bf16_ts, of 8-bit types.
__device__ __forceinline__ void mma_f8_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 bytes of each of 128 rows from shared memory to 8 TMEM columns; products
// that the same thread issues later see them.
__device__ __forceinline__ void tmem_cp_rows(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.128x256b [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
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
// A box of a page's tokens: (token of the page, 64-channel block, KV head, page).
__device__ __forceinline__ void tma_5d(void* dst, const CUtensorMap* map, int token, int block, int head, int page,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], "
      "[%7];\n" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(token), "r"(block), "r"(head), "r"(page), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::
          "r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
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
// 32 bytes, as one store where the address allows it (a whole sector: a thread
// writes a row of its own), else as two.
__device__ __forceinline__ void st_global32(void* to, const uint32_t* x) {
  if ((reinterpret_cast<uintptr_t>(to) & 31u) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(to), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    static_cast<uint4*>(to)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    static_cast<uint4*>(to)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}
// Fetches a tensor map ahead of its first copy.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// One lane of a converged warp.
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
// a * b + c of two f16 values, rounded once.
__device__ __forceinline__ uint32_t fma_f16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// (a & mask) | b in one instruction: b from a register.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "n"(MASK), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t add_f16(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

#define R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define S8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
#define U8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), "+r"(a[i + 5]), "+r"(a[i + 6]), "+r"(a[i + 7])
// 32 consecutive columns of this thread's TMEM lane; the values are there after
// tmem_ld_wait of the same array.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : R8(r, 0), R8(r, 8), R8(r, 16), R8(r, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" : U8(r, 0), U8(r, 8), U8(r, 16), U8(r, 24) : : "memory");
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
// 16 consecutive columns; tmem_st_wait before others read them.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};\n" ::S8(r, 0),
      S8(r, 8), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// Two binary32 values in a register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
#undef U8
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
  r.first = r.pos0 + row_of(p, r.f0);
  r.last = r.pos0 + row_of(p, r.f0 + r.nf - 1);
  return r;
}

// Bits 0 .. n - 1 (n of any sign and size).
__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

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

template <int D, int KIND>
__global__ void __launch_bounds__(threads_of(KIND), 1) paged_tc_kernel(const __grid_constant__ TcParams tp) {
  constexpr bool F8 = KIND == kFp8, Q4 = KIND == kQ4, CODES = F8 || Q4;
  constexpr int kCodeWarps = code_warps_of(KIND);
  auto wait = [](uint64_t* b, uint32_t parity, int* abort) { return wait_for<Q4>(b, parity, abort); };
  constexpr int NS = D / 128;            // slabs of a tile
  constexpr int NB = 2;                  // buffers of logits in TMEM
  constexpr uint32_t kOCol = NB * kKT;   // O behind them
  // Behind O, for D = 128, Q: the product then reads only K from shared memory,
  // whose 128 bytes a cycle K and Q together take all of (a short decode 11.0 ->
  // 10.8 us; 2,048 rows over 16k tokens the same 318 at the power limit, and 8%
  // less where the operands were left zero).  For D = 256 TMEM is full.
  constexpr bool QT = D == 128;
  constexpr uint32_t kQCol = kOCol + D;
  static_assert(kQCol + (QT ? 64 : 0) <= kTmemCols, "TMEM columns");
  const PagedParams& p = tp.p;
  extern __shared__ __align__(1024) uint8_t raw[];
  Head& h = *reinterpret_cast<Head*>(raw);
  Scales& sc = *reinterpret_cast<Scales*>(raw + kHeadBytes);
  Q4Head& q4 = *reinterpret_cast<Q4Head*>(raw + kHeadBytes);
  uint8_t* q_s = raw + kHeadBytes + extra_bytes(KIND);
  const int q_slab = (p.mt * 128 + 1023) / 1024 * 1024;
  uint8_t* k_ring = q_s + 2 * NS * q_slab;
  constexpr int kKeySlab = F8 ? kCodeSlab : kSlab;   // (the products take K's codes as they are)
  uint8_t* v_ring = k_ring + tp.n_k * kKeySlab;
  uint8_t* v_codes = v_ring + tp.n_v * kSlab;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quarters = (p.mt + 31) / 32, soft_threads = 64 * quarters;
  // Warps that convert codes: their own, and (fp8) those of the softmax's eight without entries.
  const int code_warps = kCodeWarps + (Q4 ? 0 : kSoftWarps - 2 * quarters);
  int* abrt = &h.abort;

  if (tid == 0) {
    for (int kv = 0; kv < 2; ++kv) {
      for (int i = 0; i < kMaxSlabs; ++i) {
        bar_init(&h.full[kv][i], Q4 ? code_warps / 2 : F8 && kv == 1 ? code_warps : 1);
        bar_init(&h.empty[kv][i], 1);
      }
    }
    for (int i = 0; i < kMaxSlabs; ++i) bar_init(&h.v_ready[i], 1);
    for (int i = 0; F8 && i < kMaxCodeSlabs; ++i) {
      bar_init(&h.code_full[i], 1);
      bar_init(&h.code_empty[i], code_warps);
    }
    for (int i = 0; CODES && i < 8; ++i) bar_init(&h.sc_full[i], kCodeWarps);
    for (int i = 0; Q4 && i < 2 * kMaxQ4Slots; ++i) {
      bar_init(&q4.code_full[0][0] + i, 1);
      bar_init(&q4.code_empty[0][0] + i, code_warps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&h.s_full[i], 1);
      bar_init(&h.p_full[i], 2 * quarters);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&h.pv_done[i], 1);
    }
    bar_init(&h.o_free, 2 * quarters);
    bar_init(&h.q_full, CODES ? kCodeWarps : 1);
    bar_init(&h.q_free, 1);
    bar_init(&h.q_used, 1);
    bar_init(&h.mma_done, 1);
    h.abort = 0;
    bar_init_fence();
  }
  if (warp == kMmaWarp) tmem_alloc(&h.tmem, kTmemCols);
  if (warp == kQWarp && lane < (F8 ? 2 : 3)) prefetch_map(lane == 0 ? &tp.k : lane == 1 ? &tp.v : Q4 ? &tp.r : &tp.q);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = h.tmem;
  grid_dependency_wait();
  grid_dependency_release();
  const Start st = find_run<threads_of(KIND), kKT>(p, p.mt, blockIdx.x, gridDim.x, h.scan, &h.start);
  Cursor<kKT> c;
  c.begin(p, p.mt, st);
  if (tid == 0) h.start = st;   // for the end (this thread's): registers are short

  // (4-bit: the roles end by themselves, so that registers need not be the same again behind them.)
  if (st.n == 0) {
    if (tid == 0) p.parts[blockIdx.x] = PagedPart{};
  } else if (warp == kKeyWarp || warp == kValueWarp) {
    // ------------------------------------------------------------ K, or V
    // (bf16: into the ring of operands; fp8: codes into their own.)  One lane
    // issues, with values that all lanes agree on; see the products below.
    if constexpr (Q4) set_registers<kQ4CopyRegs, false>();
    const int kv = warp == kValueWarp ? 1 : 0;
    const CUtensorMap* map = kv ? &tp.v : &tp.k;
    constexpr int kSlotTokens = Q4 ? Q4Slot<D>::kTokens : kKT;   // 4-bit: slots of fewer tokens, all channels
    const int box = min(1 << p.page_shift, kSlotTokens), n_box = kKT / box, page_mask = (1 << p.page_shift) - 1;
    constexpr int kBytes = Q4 ? Q4Slot<D>::kBytes : F8 ? kCodeSlab : kSlab;
    // Copies of a slab (4-bit: of a tile); lane b's: box b % n_box, ...
    const int n_copies = Q4 ? 2 * n_box : F8 || n_box == 1 ? n_box : 2 * n_box;
    // ... channels 64 * half on (4-bit: codes, or records).
    const int my_box = lane % n_box, half = !F8 && (Q4 || n_box > 1) && lane >= n_box ? 1 : 0;
    const int my_slot = my_box * box / kSlotTokens;              // 4-bit: slot of the tile
    const int at_box = !Q4 ? my_box * box * 128 + half * kHalf
                           : half ? Q4Slot<D>::kCodes + (my_box * box - my_slot * kSlotTokens) * (D / 8)
                                  : (my_box * box - my_slot * kSlotTokens) * (D / 2);
    uint64_t* fulls = Q4 ? q4.code_full[kv] : F8 && kv ? h.code_full : h.full[kv];
    uint64_t* empties = Q4 ? q4.code_empty[kv] : F8 && kv ? h.code_empty : h.empty[kv];
    uint8_t* const to_ring = Q4 ? v_codes + kv * tp.n_code_v * Q4Slot<D>::kBytes : kv ? (F8 ? v_codes : v_ring) : k_ring;
    const int n_ring = Q4 ? tp.n_code_v : kv ? (F8 ? tp.n_code_v : tp.n_v) : tp.n_k;
    const bool leader = elect_one();
    Ring at;
    int tj = 0;
    bool live = true;   // no wait of this CTA has given up: nothing is issued after one has
    for (bool more = true; more && live; more = __shfl_sync(0xffffffffu, (int)c.next(p, p.mt), 0) != 0) {
      const ItemRows ir = item_rows(p, c);
      const int T = __shfl_sync(0xffffffffu, c.x1 - c.x, 0);
      auto wanted = [&](int j) {   // whether the lane's box of a tile holds a visible token
        const int t = c.tiles.token(c.x + j) + my_box * box, end = min(t + box - 1, ir.last);
        return lane < n_copies && t <= ir.last && (p.window == 0 || end > ir.first - p.window || t < p.n_sinks);
      };
      // The table's entry for it, not looked at before the tile's turn: that would
      // wait for the load.
      auto look_up = [&](int j) {
        const int64_t slot = (int64_t)(c.tiles.token(c.x + j) + my_box * box) >> p.page_shift;
        int32_t page = -1;
        if (wanted(j) && slot < p.table_ld) page = __ldcg(p.table + c.seq * p.table_ld + slot);
        return page;
      };
      // Pages are looked up two tiles ahead.
      int page = look_up(0), next = T > 1 ? look_up(1) : 0;
#pragma unroll 1
      for (int j = 0; j < T && live; ++j) {
        const int ahead = j + 2 < T ? look_up(j + 2) : 0;
        const bool want = wanted(j), missing = want && (uint32_t)page >= (uint32_t)p.n_pages;
        if (!want || missing) page = p.n_pages;   // copies of nothing go past the last page
        if (__any_sync(0xffffffffu, missing)) {
          const uint32_t bad =
              __reduce_or_sync(0xffffffffu, missing ? ((1u << (box / 16)) - 1u) << (my_box * (box / 16)) : 0u);
          if (missing && kv == 0 && half == 0) atomicAdd(&g_bad_pages, 1);
          if (leader && kv == 0) h.bad[(tj + j) & 15] = bad;   // 16-token pieces of the tile
        } else if (leader && kv == 0) {
          h.bad[(tj + j) & 15] = 0u;
        }
        const int slot_in_page = c.tiles.token(c.x + j) & page_mask;
        // (4-bit: a page of 128 tokens and more has several boxes of a tile.)
        [[maybe_unused]] const int page_offset = box > page_mask ? 0 : (my_box * box) & page_mask;
#pragma unroll 1
        for (int s = 0; s < (Q4 ? kKT / kSlotTokens : NS); ++s) {
          uint64_t* full = fulls + at.slot;
          uint8_t* dst = to_ring + at.slot * kBytes;
          if (at.use > 0 && !wait(empties + at.slot, (at.use - 1) & 1, abrt)) live = false;
          live = __all_sync(0xffffffffu, live);
          if (!live) break;
          if (leader) bar_expect_tx(full, kBytes);
          __syncwarp();
          // A lane a box: of 128 channels (fp8, or pages of 128 tokens), or of 64.
          if (lane < n_copies) {
            if constexpr (Q4) {
              if (my_slot == s) tma_4d(dst + at_box, half ? &tp.r : map, half ? kv * (D / 8) : 0, slot_in_page + page_offset, c.head, page, full);
            } else if constexpr (F8) tma_4d(dst + at_box, map, 128 * s, slot_in_page, c.head, page, full);
            else tma_5d(dst + at_box, map, slot_in_page, 2 * s + half, c.head, page, full);
          }
          __syncwarp();
          at.step(n_ring);
        }
        page = next;
        next = ahead;
      }
      tj += T;
    }
    // Every copy has landed before the CTA ends (after a wait that gave up too).
    if (lane < n_ring) {
      const uint32_t uses = at.use + (lane < at.slot ? 1u : 0u);
      if (uses > 0) bar_wait(fulls + lane, (uses - 1) & 1, &g_timeouts);
    }
    if constexpr (Q4) return;
  } else if (Q4 && warp >= kCodeWarp) {
    // ------------------------------------------------------------ 4-bit: Q, K, V
    if constexpr (Q4) set_registers<kQ4CodeRegs, false>();
    const int cw = warp - kCodeWarp;
    constexpr int G = D / 32, kSlotTokens = Q4Slot<D>::kTokens, kSlots = kKT / kSlotTokens;
    static_assert(kQ4CodeWarps == 8 && (kSlots == 1 || kSlots == 4), "four warps a tile of K, and of V");
    // Half of the warps expand K, the others V: each waits for its own ring only.
    const int kv = cw & 1;
    const int n_ring = kv ? tp.n_v : tp.n_k;
    uint8_t* const ring = kv ? v_ring : k_ring;
    const uint8_t* const codes = v_codes + kv * tp.n_code_v * Q4Slot<D>::kBytes;
    Ring in, out;
    int it = 0;
    for (bool more = true; more; more = c.next(p, p.mt), ++it) {
      const ItemRows ir = item_rows(p, c);
      const int T = c.x1 - c.x;
      // Q as f16: times a power of two that brings the row's largest magnitude to [2^14,
      // 2^15) a value of bf16's 8 bits is exact from 2^-31 of it on, and off by at most
      // 2^-39 of it below.  Of each 8 channels, j and 4 + j lie side by side, as K's do (see
      // below).  A warp a row, D / 32 channels a lane, four rows in flight.
      {
        if (it > 0) wait(&h.q_free, (uint32_t)((it - 1) & 1), abrt);
        constexpr int kCh = D / 32, kBatch = 4;
        const int at_c = lane * kCh;
        uint8_t* const to = q_s + (at_c >> 6) * q_slab;
#pragma unroll 1
        for (int r0 = cw; r0 < ir.nf; r0 += kBatch * kCodeWarps) {
          uint32_t x[kBatch][kCh / 2];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int f = ir.f0 + min(r0 + b * kCodeWarps, ir.nf - 1), r = row_of(p, f);
            const int64_t entry = (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f - r * p.group);
            const char* from = static_cast<const char*>(p.q) + (entry * D + at_c) * 2;
            if constexpr (kCh == 8) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(from));
              x[b][0] = v.x, x[b][1] = v.y, x[b][2] = v.z, x[b][3] = v.w;
            } else {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(from));
              x[b][0] = v.x, x[b][1] = v.y;
            }
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int row = r0 + b * kCodeWarps;
            uint32_t most = 0u;
#pragma unroll
            for (int i = 0; i < kCh / 2; ++i)
              most = max(most, max((x[b][i] << 16) & 0x7fff0000u, x[b][i] & 0x7fff0000u));
            most = __reduce_max_sync(0xffffffffu, most);
            // 2^(exponent - 14), at least 2^-100: a row of smaller values keeps fewer bits.
            const int e = max((int)(most >> 23) - 127 - 14, -100);
            const float up = __uint_as_float((uint32_t)(127 - e) << 23);
            const bool odd = most >= 0x7f800000u;   // infinity or NaN: the row's logits are NaN
            // Pairs of channels (j, 4 + j); of head_dim 128 the other half of the 8 is with the
            // lane beside this one, which takes j = 2 and 3 where this one takes 0 and 1.
            uint32_t lo4[2], hi4[2];   // channels 0 1, 2 3 and 4 5, 6 7
            if constexpr (kCh == 8) {
              lo4[0] = x[b][0], lo4[1] = x[b][1], hi4[0] = x[b][2], hi4[1] = x[b][3];
            } else {
              const uint32_t other = __shfl_xor_sync(0xffffffffu, lane & 1 ? x[b][0] : x[b][1], 1);
              lo4[0] = lane & 1 ? other : x[b][0], hi4[0] = lane & 1 ? x[b][1] : other;
            }
            uint32_t f16[kCh / 2];
#pragma unroll
            for (int i = 0; i < kCh / 4; ++i) {
              f16[2 * i] = odd ? 0x7fff7fffu : pack_f16(__uint_as_float(lo4[i] << 16) * up, __uint_as_float(hi4[i] << 16) * up);
              f16[2 * i + 1] = odd ? 0x7fff7fffu : pack_f16(__uint_as_float(lo4[i] & 0xffff0000u) * up, __uint_as_float(hi4[i] & 0xffff0000u) * up);
            }
            if (row < ir.nf) {
              const int byte = (at_c & 63) * 2;
              const int at = row * 128 + ((((byte >> 4) ^ (row & 7)) << 4) | (byte & 15));
              if constexpr (kCh == 8) *reinterpret_cast<uint4*>(to + at) = make_uint4(f16[0], f16[1], f16[2], f16[3]);
              else *reinterpret_cast<uint2*>(to + at) = make_uint2(f16[0], f16[1]);
              if (lane == 0) q4.q[it & 3][row] = odd ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&h.sc_full[it & 3]);
          bar_arrive(&h.q_full);
        }
      }
      // K's or V's codes of a tile to f16 in the layout the products read: value = code *
      // scale + minimum, rounded once.  V: tokens that no row sees become zeros.
      // Four lanes a token, each the units 2 i and 2 i + 1 (8 channels) of every block;
      // lanes next to each other take tokens that differ in bits 0 and 2, so that the
      // loads and the stores of eight lanes touch all 32 banks.  Of a block's 8 channels, j
      // and 4 + j (nibbles j of the two units) are one pair of halves and stay side by side.
      const int i = lane & 3, q8 = lane >> 2, in8 = q8 & 1 ? (q8 >> 1) ^ 5 : q8 >> 1;
      constexpr int kRow = D / 2, kRec = D / 8;   // bytes of a token
      uint32_t m1024 = 0x64006400u, m64 = 0x54005400u;   // kept in registers
      asm volatile("" : "+r"(m1024), "+r"(m64));
      const int from = in8 * kRow + (D == 256 ? (2 * i ^ in8) << 4 : (i ^ (in8 >> 1)) << 4);
      const int to = in8 * 128 + ((i ^ in8) << 4);
#pragma unroll 1
      for (int j = 0; j < T; ++j) {
        const int t0 = c.tiles.token(c.x + j);
        auto slot_of = [&](int t) { return min(max(t - t0, 0), kKT); };
        const int cut = slot_of(ir.last + 1);
        const int gap0 = p.window > 0 ? slot_of(p.n_sinks) : 0;
        const int gap1 = p.window > 0 ? slot_of(ir.first - p.window + 1) : 0;
        const bool some = kv == 1 && (cut < kKT || gap0 < gap1);
        // The warp's four blocks of eight tokens: one of each slot, or four of the one.  Codes
        // go to registers, as many as there are, before the slab they will fill is free.
        constexpr int kAhead = D == 256 ? 2 : 4;
#pragma unroll 1
        for (int b0 = 0; b0 < 4; b0 += kAhead) {
          uint4 w[kAhead][G / 4], rec[kAhead][G / 4];   // units 2 i and 2 i + 1; scales and minima
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const bool opens = kSlots == 4 || k == 0, closes = kSlots == 4 || k == kAhead - 1;
            const int block = (cw >> 1) + (kSlots == 4 ? 0 : 4 * k);
            if (opens) wait(&q4.code_full[kv][in.slot], in.use & 1, abrt);
            const uint8_t* const src = codes + in.slot * Q4Slot<D>::kBytes;
#pragma unroll
            for (int x = 0; x < G / 4; ++x) {
              w[k][x] = *reinterpret_cast<const uint4*>(src + (block * 8 * kRow + (from ^ (16 * x))));
              rec[k][x] = *reinterpret_cast<const uint4*>(src + Q4Slot<D>::kCodes + (block * 8 + in8) * kRec + 16 * x);
            }
            if (closes) {
              __syncwarp();
              if (lane == 0) bar_arrive(&q4.code_empty[kv][in.slot]);
              in.step(tp.n_code_v);
            }
          }
          if (b0 == 0) {
            Ring o = out;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
              if (o.use > 0) wait(&h.empty[kv][o.slot], (o.use - 1) & 1, abrt);
              o.step(n_ring);
            }
          }
          // (A tile of head_dim 256 takes both slabs of the ring, in order.)
          uint8_t* const slab = ring + out.slot * kSlab + to;
#pragma unroll
          for (int k = 0; k < kAhead; ++k) {
            const int R0 = kSlots == 4 ? (b0 + k) * kSlotTokens + (cw >> 1) * 8 : ((cw >> 1) + 4 * k) * 8, R = R0 + in8;
            const bool gone = some && (R >= cut || (R >= gap0 && R < gap1));
            uint8_t *const even = slab + R0 * 128, *const odd = even + ((to ^ 64) - to);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint32_t a4[4] = {w[k][0].x, w[k][0].y, w[k][0].z, w[k][0].w},
                             b4[4] = {w[k][G / 4 - 1].x, w[k][G / 4 - 1].y, w[k][G / 4 - 1].z, w[k][G / 4 - 1].w},
                             r4[4] = {rec[k][g / 4].x, rec[k][g / 4].y, rec[k][g / 4].z, rec[k][g / 4].w};
              // Unit 2 i of blocks (g, g + 1), and unit 2 i + 1: 16 bytes each, or one 16 bytes of both.
              const uint32_t ua = D == 256 ? a4[g / 2] : a4[(g / 2) & 1], ub = D == 256 ? b4[g / 2] : b4[2 + ((g / 2) & 1)];
              const uint32_t r1 = gone ? 0u : r4[g & 3];
              const uint32_t s2 = __byte_perm(r1, 0u, 0x1010), m2 = __byte_perm(r1, 0u, 0x3232);
              const uint32_t lo = __byte_perm(ua, ub, g & 1 ? 0x7632 : 0x5410), hi = lo >> 8;
              // Bits 0-3 of the halves are the units of 1024's mantissa, bits 4-7 those of 64's.
              *reinterpret_cast<uint4*>((g & 1 ? odd : even) + (g >> 2) * kSlab + ((g >> 1) & 1) * kHalf) =
                  make_uint4(fma_f16(add_f16(and_or<0x000f000fu>(lo, m1024), 0xe400e400u), s2, m2),
                             fma_f16(add_f16(and_or<0x00f000f0u>(lo, m64), 0xd400d400u), s2, m2),
                             fma_f16(add_f16(and_or<0x000f000fu>(hi, m1024), 0xe400e400u), s2, m2),
                             fma_f16(add_f16(and_or<0x00f000f0u>(hi, m64), 0xd400d400u), s2, m2));
            }
          }
        }
        fence_async_smem();
        __syncwarp();
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          if (lane == 0) bar_arrive(&h.full[kv][out.slot]);
          out.step(n_ring);
        }
      }
    }
    return;
  } else if (F8 && (warp >= kCodeWarp || (warp < kSoftWarps && (warp & 3) >= quarters))) {
    // ------------------------------------------------------------ fp8: Q, scales, V
    const int cw = warp >= kCodeWarp ? warp - kCodeWarp : kCodeWarps + (warp >> 2) * (4 - quarters) + (warp & 3) - quarters;
    const int ct = 32 * cw + lane;
    const bool own = cw < kCodeWarps;   // Q and the scales are these warps'
    const float zs = p.scale * kLog2e;
    Ring in, out;
    int tj = 0, it = 0;
    for (bool more = true; more; more = c.next(p, p.mt), ++it) {
      const ItemRows ir = item_rows(p, c);
      const int T = c.x1 - c.x;
      auto visible = [&](int t) {
        return t <= ir.last && (p.window == 0 || t > ir.first - p.window || t < p.n_sinks);
      };
      auto look_up = [&](int j) {   // the table's entry for the thread's token of tile j (not looked at), -1: none
        const int t = c.tiles.token(c.x + j) + ct;
        const int64_t slot = (int64_t)t >> p.page_shift;
        int32_t page = -1;
        if (own && j < T && visible(t) && slot < p.table_ld) page = __ldcg(p.table + c.seq * p.table_ld + slot);
        return page;
      };
      auto load = [&](int j, int page) {
        const int slot = (c.tiles.token(c.x + j) + ct) & ((1 << p.page_shift) - 1);
        uint32_t record = 0x00003c00u;   // K scale 1, V scale 0
        if ((uint32_t)page < (uint32_t)p.n_pages)
          record = __ldg(reinterpret_cast<const uint32_t*>(
              p.kv_scale + 4 * (page * p.s_page_stride + c.head * p.s_head_stride + slot * p.s_tok_stride)));
        return record;
      };
      int page = look_up(0);
      // Q as codes: with the row's largest magnitude brought to [2^11, 2^12) by a power
      // of two, a value v of [2^e, 2^(e + 1)) is the sum of its nearest E5M2 code (3
      // significant bits) and the nearest E4M3 code (4) of what that leaves, which is at
      // most 16 of bf16's units 2^(e - 7) and so exact where the unit is a step of E4M3:
      // 2^-9 or more, for e >= -2, values from 2^-13 of the row's largest on.  Smaller
      // ones are off by at most half of that step, 2^-21 of the largest.  (Two E4M3
      // codes, which have to start at 2^8, are exact from 2^-9 on only: with a channel
      // 1,000 times the others, logits were off by up to 1e-2.)  A warp a row, D / 32
      // channels a lane, four rows in flight.
      if (own) {
        if (it > 0) wait(&h.q_free, (uint32_t)((it - 1) & 1), abrt);
        constexpr int kCh = D / 32, kBatch = 4;
        const int at_x = (lane * kCh) & 127;   // channel within the slab of 128
        uint8_t* const hi_s = q_s + (lane * kCh >> 7) * q_slab;
        uint8_t* const lo_s = hi_s + NS * q_slab;
#pragma unroll 1
        for (int r0 = cw; r0 < ir.nf; r0 += kBatch * kCodeWarps) {
          uint32_t x[kBatch][kCh / 2];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int f = ir.f0 + min(r0 + b * kCodeWarps, ir.nf - 1), r = row_of(p, f);
            const int64_t entry = (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f - r * p.group);
            const char* from = static_cast<const char*>(p.q) + (entry * D + lane * kCh) * 2;
            if constexpr (kCh == 8) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(from));
              x[b][0] = v.x, x[b][1] = v.y, x[b][2] = v.z, x[b][3] = v.w;
            } else {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(from));
              x[b][0] = v.x, x[b][1] = v.y;
            }
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int row = r0 + b * kCodeWarps;
            uint32_t most = 0u;   // the largest magnitude's bits (ordered as the values are; NaN above all)
#pragma unroll
            for (int i = 0; i < kCh / 2; ++i)
              most = max(most, max((x[b][i] << 16) & 0x7fff0000u, x[b][i] & 0x7fff0000u));
            most = __reduce_max_sync(0xffffffffu, most);
            // 2^(exponent - 11), at least 2^-100: a row of smaller values keeps fewer bits.
            const int e = max((int)(most >> 23) - 127 - 11, -100);
            const float up = __uint_as_float((uint32_t)(127 - e) << 23);
            const bool odd = most >= 0x7f800000u;   // infinity or NaN: the row's logits are NaN
            uint32_t hi[kCh / 4], lo[kCh / 4];
#pragma unroll
            for (int i = 0; i < kCh / 4; ++i) {
              const float v0 = __uint_as_float(x[b][2 * i] << 16) * up, v1 = __uint_as_float(x[b][2 * i] & 0xffff0000u) * up,
                          v2 = __uint_as_float(x[b][2 * i + 1] << 16) * up,
                          v3 = __uint_as_float(x[b][2 * i + 1] & 0xffff0000u) * up;
              const uint32_t h01 = to_e5m2x2(v0, v1), h23 = to_e5m2x2(v2, v3);
              const float2 b01 = from_e5m2x2(h01), b23 = from_e5m2x2(h23);
              hi[i] = odd ? 0x7f7f7f7fu : h01 | h23 << 16;
              lo[i] = odd ? 0u : to_e4m3x2(v0 - b01.x, v1 - b01.y) | to_e4m3x2(v2 - b23.x, v3 - b23.y) << 16;
            }
            if (row < ir.nf) {
              const int at = row * 128 + ((((at_x >> 4) ^ (row & 7)) << 4) | (at_x & 15));
              if constexpr (kCh == 8) {
                *reinterpret_cast<uint2*>(hi_s + at) = make_uint2(hi[0], hi[1]);
                *reinterpret_cast<uint2*>(lo_s + at) = make_uint2(lo[0], lo[1]);
              } else {
                *reinterpret_cast<uint32_t*>(hi_s + at) = hi[0];
                *reinterpret_cast<uint32_t*>(lo_s + at) = lo[0];
              }
              if (lane == 0) sc.q[it & 3][row] = odd ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(&h.q_full);
      }
      uint32_t record = load(0, page);
      page = look_up(1);
      // A tile's scales; each thread has its token's page two tiles ahead and its
      // record one tile ahead.  The tile eight before it is done: what was converted
      // last is V of the tile NB before it, into a slot that the tile n_v / NS <= 5
      // further back had left.
      auto put_scales = [&](int j) {
        const __half2 both = *reinterpret_cast<const __half2*>(&record);
        // Logits are hidden by minus infinity before they are scaled, so the factors
        // are positive numbers: magnitudes, 1e-30 for zero.  Negative scales and NaN are
        // left to the softmax, as bits of a tile's 32 tokens: it changes the sign of
        // their logits, or makes them NaN, before it hides what a row does not see.
        const float f = __low2float(both) * zs;
        const uint32_t neg = __ballot_sync(0xffffffffu, f < 0.f), nan = __ballot_sync(0xffffffffu, f != f);
        sc.k[(tj + j) & 7][ct] = fabsf(f) > 0.f ? fabsf(f) : 1e-30f;
        sc.v[(tj + j) & 7][ct] = __high2float(both);
        if (lane == 0) reinterpret_cast<uint2*>(h.odd_scale[(tj + j) & 7])[cw] = make_uint2(neg, nan);
        __syncwarp();
        if (lane == 0) bar_arrive(&h.sc_full[(tj + j) & 7]);
        record = load(j + 1, page);
        page = look_up(j + 2);
      };
      // V's codes to bf16 in the layout the product reads;
      // exact.  Tokens that no row sees become zeros, whatever their codes.
      auto convert = [&](int j) {
        const int t0 = c.tiles.token(c.x + j);
        // Tokens [0, cut) of the tile less [gap0, gap1) are seen by some row.
        auto slot_of = [&](int t) { return min(max(t - t0, 0), kKT); };
        const int cut = slot_of(ir.last + 1);
        const int gap0 = p.window > 0 ? slot_of(p.n_sinks) : 0;
        const int gap1 = p.window > 0 ? slot_of(ir.first - p.window + 1) : 0;
        const bool some = cut < kKT || gap0 < gap1;
#pragma unroll 1
        for (int s = 0; s < NS; ++s) {
          wait(&h.code_full[in.slot], in.use & 1, abrt);
          if (out.use > 0) wait(&h.empty[1][out.slot], (out.use - 1) & 1, abrt);
          const uint8_t* src = v_codes + in.slot * kCodeSlab;
          uint8_t* dst = v_ring + out.slot * kSlab;
          // Eight threads a token, each 8 channels of one half of the slab and then of
          // the other, tokens next to each other in opposite order: the loads of a
          // warp and the stores of eight threads then touch all 32 banks.
          const int piece = ct & 7, odd = (ct >> 3) & 1;
#pragma unroll 4
          for (int tk = ct >> 3; tk < kKT; tk += 4 * code_warps) {
            uint2 x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const uint2*>(src + tk * 128 + (i ^ odd) * 64 + piece * 8);
            if (some && (tk >= cut || (tk >= gap0 && tk < gap1))) x[0] = x[1] = make_uint2(0u, 0u);
            uint8_t* row = dst + tk * 128 + ((piece ^ (tk & 7)) << 4);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              *reinterpret_cast<uint4*>(row + (i ^ odd) * kHalf) =
                  make_uint4(attn::e4m3x2_to_bf16x2(x[i].x & 0xffffu), attn::e4m3x2_to_bf16x2(x[i].x >> 16),
                             attn::e4m3x2_to_bf16x2(x[i].y & 0xffffu), attn::e4m3x2_to_bf16x2(x[i].y >> 16));
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(&h.full[1][out.slot]);
            bar_arrive(&h.code_empty[in.slot]);
          }
          in.step(tp.n_code_v);
          out.step(tp.n_v);
        }
      };
#pragma unroll 1
      for (int j = 0; j < T + NB - 1; ++j) {
        if (own && j < T) put_scales(j);
        if (j >= NB - 1) convert(j - (NB - 1));
      }
      tj += T;
    }
  } else if (!CODES && warp == kQWarp) {
    // ------------------------------------------------------------ Q, and V's ends
    // An item holds whole rows, so its entries are one box for each 64 channels.
    // The next item's are copied before the last tile's V is waited for.
    //
    // V's slabs pass through this warp on their way to the product: slots of tokens
    // that no row sees become zeros (P = 0 there, but 0 x NaN would reach O).  Boxes
    // without a visible token hold zeros already, so at most two boxes' parts of a
    // tile are left.  (Done by the softmax's warps before their weights, an item's
    // first and last tiles waited for V as well as for the logits: 5,000 cycles.)
    const bool leader = elect_one();
    const int rows = p.mt / p.group;
    const int box = min(1 << p.page_shift, kKT);
    bool live = true;
    auto load_q = [&](const Cursor<kKT>& i) {
      if (leader) {
        bar_expect_tx(&h.q_full, 2 * NS * p.mt * 128);
#pragma unroll 1
        for (int s = 0; s < 2 * NS; ++s)
          tma_3d(q_s + s * q_slab, &tp.q, 64 * s, i.head * p.group, i.s.row0 + i.m * rows, &h.q_full);
      }
      __syncwarp();
    };
    Cursor<kKT> ahead = c;
    Ring va;
    int it = 0, loads = 1;
    load_q(ahead);
    for (bool more = true; more && live; more = __shfl_sync(0xffffffffu, (int)c.next(p, p.mt), 0) != 0, ++it) {
      const ItemRows ir = item_rows(p, c);
      const int T = __shfl_sync(0xffffffffu, c.x1 - c.x, 0);
#pragma unroll 1
      for (int j = 0; j < T && live; ++j) {
        if (j == T - 1 && __shfl_sync(0xffffffffu, (int)ahead.next(p, p.mt), 0) != 0) {
          live = __all_sync(0xffffffffu, wait(&h.q_free, (uint32_t)(it & 1), abrt));
          if (!live) break;
          load_q(ahead);
          ++loads;
        }
        // Tokens [0, cut) of the tile less [gap0, gap1) are seen by some row.
        const int t0 = c.tiles.token(c.x + j);
        auto slot_of = [&](int t) { return min(max(t - t0, 0), kKT); };
        const int cut = slot_of(ir.last + 1), gap0 = p.window > 0 ? slot_of(p.n_sinks) : 0,
                  gap1 = p.window > 0 ? slot_of(ir.first - p.window + 1) : 0;
#pragma unroll 1
        for (int s = 0; s < NS; ++s) {
          live = __all_sync(0xffffffffu, wait(&h.full[1][va.slot], va.use & 1, abrt));
          if (!live) break;
          if (cut < kKT || gap0 < gap1) {
            uint8_t* const slab = v_ring + va.slot * kSlab;
            auto clear = [&](int from, int to) {
#pragma unroll 1
              for (int i = from * 8 + lane; i < to * 8; i += 32) {
                reinterpret_cast<uint4*>(slab)[i] = make_uint4(0u, 0u, 0u, 0u);
                reinterpret_cast<uint4*>(slab + kHalf)[i] = make_uint4(0u, 0u, 0u, 0u);
              }
            };
            clear(cut, (cut + box - 1) & -box);
            if (gap0 < gap1) {
              const int up = min((gap0 + box - 1) & -box, gap1);
              clear(gap0, up);
              clear(max(gap1 & -box, up), gap1);
            }
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) bar_arrive(&h.v_ready[va.slot]);
          va.step(tp.n_v);
        }
      }
    }
    bar_wait(&h.q_full, (uint32_t)((loads - 1) & 1), &g_timeouts);   // landed before the CTA ends
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    // The whole warp walks through the tiles with values that are the same in
    // all its lanes, and one lane issues: descriptors then stay in uniform
    // registers.  (One lane that walks alone has to move each of them over:
    // 115 cycles an MMA instead of the 32 and 64 that the products take.)
    if constexpr (Q4) set_registers<kQ4CopyRegs, false>();
    const bool leader = elect_one();
    const uint64_t q_desc = desc_sw128(q_s, 16, 1024), k_desc = desc_sw128(k_ring, 16, 1024),
                   v_desc = desc_sw128(v_ring, kHalf, 1024);
    const uint32_t q_step = (uint32_t)q_slab >> 4;
    uint64_t* const v_full = CODES ? h.full[1] : h.v_ready;   // (who passes bf16's V on has waited for the copies)
    constexpr uint32_t kOperands = Q4 ? kF16Operands : ~0u;
    Ring ka, va;
    int it = 0;
    int s_buf = 0, p_buf = 0, odd = 0;   // buffers of the next logits and the next weights; parity of the next output
    uint32_t p_phase = 0;                // bit b: the phase of p_full[b] to wait for
    bool live = true;                    // as above
    for (bool more = true; more; more = __shfl_sync(0xffffffffu, (int)c.next(p, p.mt), 0) != 0, ++it) {
      const int T = __shfl_sync(0xffffffffu, c.x1 - c.x, 0);
      auto logits = [&](bool last) {   // S = Q K^T of the next tile
        const uint32_t d = tmem + (uint32_t)(s_buf * kKT);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          live = wait(&h.full[0][ka.slot], ka.use & 1, abrt) && live;
          fence_after();
          if (leader && live) {
            const uint64_t k = k_desc + (uint32_t)(ka.slot * (kKeySlab >> 4)), q = q_desc + (F8 ? 1 : 2) * s * q_step;
#pragma unroll
            for (int x = 0; QT && x < 8; ++x) {
              if constexpr (F8) mma_f8_ts(d, tmem + kQCol + 8u * x, k + 2 * (x & 3), x < 4 ? kIdescHi8 : kIdescLo8, x != 0 ? 1u : 0u);
              else
                mma_bf16_ts(d, tmem + kQCol + 8u * x, k + (x >> 2) * (kHalf >> 4) + 2 * (x & 3), kIdescS & kOperands, x != 0 ? 1u : 0u);
            }
#pragma unroll
            for (int x = 0; !QT && F8 && x < 8; ++x)   // both codes of Q's values
              mma_f8(d, q + (x >> 2) * NS * q_step + 2 * (x & 3), k + 2 * (x & 3), x < 4 ? kIdescHi8 : kIdescLo8,
                     (s | x) != 0 ? 1u : 0u);
#pragma unroll
            for (int x = 0; !QT && !F8 && x < 8; ++x)
              mma_bf16(d, q + (x >> 2) * q_step + 2 * (x & 3), k + (x >> 2) * (kHalf >> 4) + 2 * (x & 3), kIdescS & kOperands,
                       (s | x) != 0 ? 1u : 0u);
            commit(&h.empty[0][ka.slot]);
            if (s == NS - 1) commit(&h.s_full[s_buf]);
            if (s == NS - 1 && last) commit(QT ? &h.q_used : &h.q_free);
          }
          __syncwarp();
          ka.step(tp.n_k);
        }
        s_buf = s_buf + 1 == NB ? 0 : s_buf + 1;
      };
      live = __all_sync(0xffffffffu, wait(&h.q_full, (uint32_t)(it & 1), abrt) && live);
      if constexpr (QT) {   // the item before has had its logits
        if (it > 0) live = __all_sync(0xffffffffu, wait(&h.q_used, (uint32_t)((it - 1) & 1), abrt) && live);
        fence_after();
        if (leader && live) {
#pragma unroll
          for (int x = 0; x < 8; ++x) tmem_cp_rows(tmem + kQCol + 8u * x, q_desc + (x >> 2) * q_step + 2 * (x & 3));
          commit(&h.q_free);
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int j = 0; j < min(NB, T); ++j) logits(j == T - 1);
      // Then an output product and the logits NB tiles ahead of it, which take the
      // buffer that its weights leave.
#pragma unroll 1
      for (int j = 0; j < T; ++j) {
        // (V is there first as a rule, so the weights are waited for last.)
        live = wait(v_full + va.slot, va.use & 1, abrt) && live;
        live = wait(&h.p_full[p_buf], (p_phase >> p_buf) & 1, abrt) && live;
        p_phase ^= 1u << p_buf;
        if (j == 0 && it > 0) wait(&h.o_free, (uint32_t)((it - 1) & 1), abrt);
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          if (s > 0) live = wait(v_full + va.slot, va.use & 1, abrt) && live;
          fence_after();
          if (leader && live) {
            const uint64_t v = v_desc + (uint32_t)(va.slot * (kSlab >> 4));
#pragma unroll
            for (int x = 0; x < 8; ++x)
              mma_bf16_ts(tmem + kOCol + (uint32_t)(s * 128), tmem + (uint32_t)(p_buf * kKT + 8 * x), v + 128 * x,
                          kIdescO & kOperands, (j | x) != 0 ? 1u : 0u);
            commit(&h.empty[1][va.slot]);
            if (s == NS - 1) commit(&h.pv_done[odd]);
          }
          __syncwarp();
          va.step(tp.n_v);
        }
        odd ^= 1;
        p_buf = p_buf + 1 == NB ? 0 : p_buf + 1;
        if (j + NB < T) logits(j + NB == T - 1);
      }
    }
    if (leader) commit(&h.mma_done);   // every MMA has completed before TMEM is released
    __syncwarp();
    bar_wait(&h.mma_done, 0u, &g_timeouts);
    if constexpr (Q4) {
      named_sync(15, 32 * (kSoftWarps + 1));   // the softmax's warps have read TMEM
      fence_after();
      tmem_dealloc(tmem, kTmemCols);
      return;
    }
  } else if (warp < kSoftWarps && (Q4 || (warp & 3) < quarters)) {
    // ------------------------------------------------------------ softmax and output
    // A thread owns one entry, and the keys [64 group, 64 group + 64) of each tile.
    if constexpr (Q4) set_registers<kQ4SoftRegs, true>();
    const int group = warp >> 2, row = 32 * (warp & 3) + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    // Logits to base 2; the scales of an fp8 cache's keys hold the factor already,
    // and what is left is the power of two that the row of Q was divided by.
    float zc = p.scale * kLog2e, move = fminf(kMoveMax / zc, 1e30f);
    int tj = 0;   // tiles done
    [[maybe_unused]] int it = 0;
    for (bool more = !Q4 || (warp & 3) < quarters; more;) {
      const ItemRows ir = item_rows(p, c);
      const int T = c.x1 - c.x;
      const bool mine = row < ir.nf;
      const int pos = ir.pos0 + row_of(p, ir.f0 + min(row, ir.nf - 1));
      const int low = p.window > 0 ? pos - p.window + 1 : 0;   // first token of the row's window
      // (Not known before a tile's scales are, which follow Q's.  Four items: a group
      // may be one behind the other, Q one ahead of both.)
      auto factor = [&] {
        zc = mine ? (Q4 ? q4.q : sc.q)[it & 3][row] : 1.f;
        if constexpr (Q4) zc = fmaxf(zc * (p.scale * kLog2e), 1e-37f);   // (not 0: hidden logits are -infinity times it)
        move = fminf(kMoveMax / zc, 1e30f);
      };
      if constexpr (Q4) {
        wait(&h.sc_full[it & 3], (uint32_t)((it >> 2) & 1), abrt);
        factor();
      }
      float m = -INFINITY, l = 0.f;   // the maximum that this thread's sum l is relative to
      // What a row does not see of keys [from, to) of a tile becomes -infinity, in
      // TMEM: the passes below stay short (with the masks unrolled into them they no
      // longer fit the instruction cache and take four times as long).
      auto hide = [&](int t0, uint32_t bad, uint32_t s_col, int from, int to, uint32_t(&x)[32], const uint4* odd_scale) {
        uint32_t odd = 0u;
        if constexpr (F8) {
          const uint4 o = odd_scale[from / 64];
          odd = o.x | o.y | o.z | o.w;
        }
        if (bad == 0 && odd == 0 && t0 + kKT - 1 <= ir.first &&
            !(p.window > 0 && t0 <= ir.last - p.window && t0 + kKT > p.n_sinks))
          return;
#pragma unroll 1
        for (int col = from; col < to; col += 32) {
          // Keys t .. t + 31: seen are those up to pos, from low on or among the first n_sinks.
          const int t = t0 + col;
          uint32_t see = below(pos + 1 - t) & (~below(low - t) | below(p.n_sinks - t));
          see &= ~((((bad >> (col / 16)) & 1u) * 0xffffu) | (((bad >> (col / 16 + 1)) & 1u) * 0xffff0000u));
          if (__all_sync(0xffffffffu, see == 0xffffffffu) && odd == 0) continue;
          tmem_ld32_start(s_col + (uint32_t)col, x);
          tmem_ld_wait(x);
          if (odd != 0) {   // (fp8)
            const uint2 o = reinterpret_cast<const uint2*>(odd_scale)[col / 32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              x[i] = o.y & (1u << i) ? 0x7fffffffu : o.x & (1u << i) ? x[i] ^ 0x80000000u : x[i];
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = see & (1u << i) ? x[i] : 0xff800000u;
          tmem_st32(s_col + (uint32_t)col, x);
        }
      };
      const int pair = 2 + (warp & 3), c0 = 64 * group;   // the barrier of the two warps of the same entries
#pragma unroll 1
      for (int j = 0; j < T; ++j) {
        const int g = tj + j, buf = g % NB, t0 = c.tiles.token(c.x + j);
        const uint32_t s_col = lanes + (uint32_t)(buf * kKT);
        wait(&h.s_full[buf], (uint32_t)((g / NB) & 1), abrt);
        __syncwarp();
        fence_after();
        uint32_t xa[32], xb[32];
        if constexpr (F8) {
          wait(&h.sc_full[g & 7], (uint32_t)((g >> 3) & 1), abrt);
          factor();
        }
        hide(t0, h.bad[g & 15], s_col, c0, c0 + 64, xa, h.odd_scale[g & 7]);
        tmem_ld32_start(s_col + (uint32_t)c0, xa);
        tmem_ld_wait(xa);
        tmem_ld32_start(s_col + (uint32_t)c0 + 32, xb);
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto take_max = [&](uint32_t(&x)[32], const float* ks) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float a[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) a[e] = __uint_as_float(x[i + e]);
            if constexpr (F8) {
              const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(ks + i);
              unpack2(mul2(pack2(a[0], a[1]), f.x), a[0], a[1]);
              unpack2(mul2(pack2(a[2], a[3]), f.y), a[2], a[3]);
            }
            m4[(i >> 2) & 3] = fmaxf(fmaxf(m4[(i >> 2) & 3], fmaxf(a[0], a[1])), fmaxf(a[2], a[3]));
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i + e] = __float_as_uint(a[e]);
          }
        };
        take_max(xa, F8 ? sc.k[g & 7] + c0 : nullptr);
        tmem_ld_wait(xb);
        take_max(xb, F8 ? sc.k[g & 7] + c0 + 32 : nullptr);
        float mx = mine ? fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) : -INFINITY;
        // (Also: both groups have read their logits, over which the weights go.)
        h.mx[g & 1][group][row] = mx;
        fence_before();
        named_sync(pair, 64);
        fence_after();
        mx = fmaxf(mx, h.mx[g & 1][group ^ 1][row]);
        // (f16: m + move may be off by more than there is room.)
        const bool moves = j == 0 ? mx != -INFINITY : Q4 ? mx - m > move : mx > m + move;
        if (__any_sync(0xffffffffu, moves)) {   // (the same in both warps)
          const float alpha = moves ? ex2((m - mx) * zc) : 1.f;
          if (moves) {
            l *= alpha;
            m = mx;
          }
          if (j > 0) {
            wait(&h.pv_done[(g - 1) & 1], (uint32_t)(((g - 1) >> 1) & 1), abrt);
            __syncwarp();
            fence_after();
#pragma unroll 1
            for (int s = 0; s < D / 64; ++s) {   // the group's half of the channels
              uint32_t o[32];
              const uint32_t at = lanes + kOCol + (uint32_t)(group * (D / 2) + 32 * s);
              tmem_ld32_start(at, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(at, o);
            }
            fence_before();
          }
        }
        float shift = m == -INFINITY ? 0.f : (Q4 ? kF16Weights : 0.f) - m * zc;
        if constexpr (Q4) {
          if (__builtin_expect(__any_sync(0xffffffffu, !(fabsf(shift) <= kFar)), 0)) {
            const float base = fabsf(shift) <= kFar ? 0.f : m;   // (a row's own: others keep their bits)
            shift = fabsf(shift) <= kFar ? shift : kF16Weights;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              xa[i] = __float_as_uint(__uint_as_float(xa[i]) - base);
              xb[i] = __float_as_uint(__uint_as_float(xb[i]) - base);
            }
          }
        }
        const uint64_t zc2 = pack2(zc, zc), shift2 = pack2(shift, shift);
        uint64_t sum2[2] = {0ull, 0ull};
        auto weigh = [&](uint32_t(&x)[32], const float* vs, uint32_t to) {
          uint32_t w[16];
          ulonglong2 vv = {0ull, 0ull};
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            if (F8 && !(i & 1)) vv = *reinterpret_cast<const ulonglong2*>(vs + 2 * i);
            unpack2(fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), zc2, shift2), a, b);
            a = ex2(a);
            b = ex2(b);
            const uint64_t e = pack2(a, b);
            sum2[i & 1] = add2(sum2[i & 1], e);
            if constexpr (F8) unpack2(mul2(e, i & 1 ? vv.y : vv.x), a, b);   // V's scale goes with the weight, rounded once
            w[i] = Q4 ? pack_f16(a, b) : pack_bf16(a, b);
          }
          tmem_st16(to, w);
        };
        __syncwarp();
        weigh(xa, F8 ? sc.v[g & 7] + c0 : nullptr, s_col + (uint32_t)(c0 / 2));
        weigh(xb, F8 ? sc.v[g & 7] + c0 + 32 : nullptr, s_col + (uint32_t)(c0 / 2 + 16));
        tmem_st_wait();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&h.p_full[buf]);
        float s0, s1;
        unpack2(add2(sum2[0], sum2[1]), s0, s1);
        l += s0 + s1;
      }
      tj += T;
      // The item's result, or this run's part of it: both groups' sums, relative
      // to the last maximum.
      named_sync(1, soft_threads);
      if constexpr (CODES) ++it;
      h.sums[group][row] = l;
      named_sync(1, soft_threads);
      l += h.sums[group ^ 1][row];
      const float inv = l == 0.f ? 0.f : 1.f / l;   // (NaN stays)
      const bool whole = c.whole();
      const int64_t part = (int64_t)c.slot(blockIdx.x) * p.mt + row;
      const int r = row_of(p, ir.f0 + row);
      const int64_t entry = (int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (ir.f0 + row - r * p.group);
      if (tj > 1) wait(&h.pv_done[tj & 1], (uint32_t)(((tj - 2) >> 1) & 1), abrt);
      wait(&h.pv_done[(tj - 1) & 1], (uint32_t)(((tj - 1) >> 1) & 1), abrt);
      __syncwarp();
      fence_after();
#pragma unroll 1
      for (int s = 0; s < D / 64; ++s) {
        uint32_t o[32];
        const int d = group * (D / 2) + s * 32;
        __syncwarp();
        tmem_ld32_start(lanes + kOCol + (uint32_t)d, o);
        tmem_ld_wait(o);
        if (!mine) continue;
        if constexpr (Q4) {   // columns 2 j and 2 j + 1 of 8 are channels j and 4 + j
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            const uint32_t x[8] = {o[e], o[e + 2], o[e + 4], o[e + 6], o[e + 1], o[e + 3], o[e + 5], o[e + 7]};
#pragma unroll
            for (int k = 0; k < 8; ++k) o[e + k] = x[k];
          }
        }
        if (!whole || p.out_dtype == QSA_F32) {
          float* to = (whole ? static_cast<float*>(p.out) + entry * D : p.part_o + part * D) + d;
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
#pragma unroll
          for (int i = 0; i < 4; ++i) st_global32(to + 8 * i, o + 8 * i);
        } else {
          __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.out) + entry * D + d;
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            w[i] = pack_bf16(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
#pragma unroll
          for (int i = 0; i < 2; ++i) st_global32(to + 16 * i, w + 8 * i);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) bar_arrive(&h.o_free);
      if (mine && group == 0) {
        const float lse2 = l == 0.f ? -INFINITY : fmaf(m, zc, log2f(l)) - (Q4 ? kF16Weights : 0.f);
        if (!whole) p.part_lse[part] = lse2;
        else if (p.lse) p.lse[entry] = lse2 * kLn2;
      }
      more = c.next(p, p.mt);
      if (!more && tid == 0) describe_part(p, c, h.start, blockIdx.x);   // (still at its last item)
    }
    if constexpr (Q4) {
      __syncwarp();
      fence_before();
      asm volatile("bar.arrive %0, %1;\n" ::"r"(15), "r"(32 * (kSoftWarps + 1)) : "memory");
      return;
    }
  } else if constexpr (Q4) {
    set_registers<kQ4CopyRegs, false>();   // the copying warpgroup's fourth warp
    return;
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

bool encode_pages(CUtensorMap* map, const void* base, const PagedParams& p, int head_dim, bool f8, bool swizzle) {
  PFN_cuTensorMapEncodeTiled_v12000 f = encoder();
  if (!f) return false;
  const cuuint64_t page = (cuuint64_t)1 << p.page_shift;
  const cuuint32_t tokens = (cuuint32_t)(page < kKT ? page : kKT);
  const cuuint32_t step[5] = {1, 1, 1, 1, 1};
  if (f8) {
    const cuuint64_t dims[4] = {(cuuint64_t)head_dim, page, (cuuint64_t)p.n_kv_heads, (cuuint64_t)p.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)p.tok_stride, (cuuint64_t)p.head_stride, (cuuint64_t)p.page_stride};
    const cuuint32_t box[4] = {128, tokens, 1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  const cuuint64_t dims[5] = {64, page, (cuuint64_t)head_dim / 64, (cuuint64_t)p.n_kv_heads, (cuuint64_t)p.n_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)p.tok_stride * 2, 128, (cuuint64_t)p.head_stride * 2,
                                 (cuuint64_t)p.page_stride * 2};
  const cuuint32_t box[5] = {64, tokens, page < kKT ? 1u : 2u, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_queries(CUtensorMap* map, const PagedParams& p, int head_dim) {
  PFN_cuTensorMapEncodeTiled_v12000 f = encoder();
  if (!f) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)head_dim, (cuuint64_t)p.n_q_heads, (cuuint64_t)p.n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)head_dim * 2, (cuuint64_t)head_dim * 2 * (cuuint64_t)p.n_q_heads};
  const cuuint32_t box[3] = {64, (cuuint32_t)p.group, (cuuint32_t)(p.mt / p.group)};
  const cuuint32_t step[3] = {1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows of `bytes` of a 4-bit cache's codes or records, in copies of `take` bytes and `tokens` tokens; strides in bytes.
bool encode_q4(CUtensorMap* map, const void* base, const PagedParams& p, int bytes, int take, int tokens, int64_t tok,
               int64_t head, int64_t page_stride, CUtensorMapSwizzle swizzle) {
  PFN_cuTensorMapEncodeTiled_v12000 f = encoder();
  if (!f) return false;
  const cuuint64_t page = (cuuint64_t)1 << p.page_shift;
  const cuuint64_t dims[4] = {(cuuint64_t)bytes, page, (cuuint64_t)p.n_kv_heads, (cuuint64_t)p.n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)tok, (cuuint64_t)head, (cuuint64_t)page_stride};
  const cuuint32_t box[4] = {(cuuint32_t)take, (cuuint32_t)std::min<cuuint64_t>(page, (cuuint64_t)tokens), 1, 1}, step[4] = {1, 1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, step,
           CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int KIND>
cudaError_t launch_d(const PagedParams& p, int grid, cudaStream_t st) {
  constexpr bool F8 = KIND == kFp8, Q4 = KIND == kQ4;
  TcParams tp{};
  tp.p = p;
  if constexpr (Q4) {
    constexpr int kTokens = Q4Slot<D>::kTokens, kRecord = D / 4;
    const CUtensorMapSwizzle sw = D == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!encode_q4(&tp.k, p.k, p, D / 2, D / 2, kTokens, p.tok_stride / 2, p.head_stride / 2, p.page_stride / 2, sw) ||
        !encode_q4(&tp.v, p.v, p, D / 2, D / 2, kTokens, p.tok_stride / 2, p.head_stride / 2, p.page_stride / 2, sw) ||
        !encode_q4(&tp.r, p.kv_scale, p, kRecord, kRecord / 2, kTokens, p.s_tok_stride * kRecord, p.s_head_stride * kRecord,
                   p.s_page_stride * kRecord, CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorInvalidValue;
  } else if (!encode_pages(&tp.k, p.k, p, D, F8, true) || !encode_pages(&tp.v, p.v, p, D, F8, !F8) ||
             (!F8 && !encode_queries(&tp.q, p, D))) {
    return cudaErrorInvalidValue;
  }
  const int q_slab = (p.mt * 128 + 1023) / 1024 * 1024;
  const int fixed = kHeadBytes + extra_bytes(KIND) + D / 64 * q_slab, room = kSmemLimit - fixed;
  if (F8) {   // operands of a whole tile of V, the rest for codes
    tp.n_v = 2;
    const int n = (room - tp.n_v * kSlab) / kCodeSlab;
    tp.n_code_v = std::min(n / 2, kMaxCodeSlabs);
    tp.n_k = std::min(n - tp.n_code_v, kMaxSlabs);
  } else if (Q4) {   // operands of a whole tile of K and V (two of head_dim 128), the rest for codes
    tp.n_k = tp.n_v = 2;
    tp.n_code_v = std::min((room - 4 * kSlab) / (2 * Q4Slot<D>::kBytes), kMaxQ4Slots);
  } else {
    const int n = room / kSlab;
    tp.n_k = std::min((n + 1) / 2, 3);
    tp.n_v = std::min(n / 2, 3);
  }
  const size_t smem = (size_t)fixed + (size_t)tp.n_k * (F8 ? kCodeSlab : kSlab) + (size_t)tp.n_v * kSlab +
                      (Q4 ? (size_t)tp.n_code_v * 2 * Q4Slot<D>::kBytes : (size_t)tp.n_code_v * kCodeSlab);
  cudaError_t e = allow_dynamic_smem((const void*)paged_tc_kernel<D, KIND>, kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_kernel(paged_tc_kernel<D, KIND>, dim3((unsigned)grid), dim3(threads_of(KIND)), smem, st, 0u, tp);
}

}  // namespace

cudaError_t launch_paged_tc(const PagedParams& p, qsa_dtype kv_dtype, int head_dim, int grid, cudaStream_t st) {
  if (kv_dtype == QSA_Q4_1) return head_dim == 256 ? launch_d<256, kQ4>(p, grid, st) : launch_d<128, kQ4>(p, grid, st);
  if (kv_dtype == QSA_FP8_E4M3) return head_dim == 256 ? launch_d<256, kFp8>(p, grid, st) : launch_d<128, kFp8>(p, grid, st);
  return head_dim == 256 ? launch_d<256, kBf16>(p, grid, st) : launch_d<128, kBf16>(p, grid, st);
}

int paged_tc_bad_pages_take() { return take_counter(g_bad_pages); }

int paged_tc_wait_timeouts() {
  int v = 0;
  return cudaMemcpyFromSymbol(&v, g_timeouts, sizeof(int)) == cudaSuccess ? v : -1;
}

}  // namespace qsa
