// A batch's rows into the pages of a cache with a rotation on the way, 4-bit
// caches, and rows back out of their pages (include/qsa.h,
// qsa_paged_append_rotate, qsa_paged_append of 4-bit caches, qsa_paged_read).
//
// Writing: one CTA a row, or up to four of a call of more rows than the GPU has places
// for.  Loads of Q, K and V are issued first, then a warp a row finds its sequence,
// position and page, and the (cos, sin) of its pairs go to shared memory once for all
// heads.  Rows that are stored as they are (f32, bf16) and Q go
// in jobs of the two 16-byte pieces that a rotation joins; a row that is quantized
// is a warp's, D / 32 channels a lane, its pairs exchanged by shuffles.  K is
// rounded to the rows' type before it is stored or quantized, so the cache holds
// what the rotation by itself and the append leave.
//
// 4 bits: blocks of 32 channels are 4 lanes (D = 256) or 8 (128): minimum and maximum
// by shuffles; the codes' order in the row (16-bit unit n * (D / 32) + g holds
// channels 32 g + 4 n .. + 3) gives each lane one 32-bit word of two units that two
// other lanes hold.
//
// On one GB300: 2,048 rows of Q, K and V of 256 into a 4-bit cache, and the rows read
// back, 22.9 us, where HBM needs 9 (dependent reads -- lengths and ranges, page -- before
// the first store, and 13 rows an SM in which to hide them); ragged prompts of 128 into an
// fp8 cache 27.3 of 14.3 (44 with a row a CTA; 20 were the sequences known); 65,536 rows of
// 256 back out of 4 bits 33.5 of 26 (52 with eight bytes of codes a lane); steps of a few
// rows 5.7 to 8.3, the host's call.
#include <cuda_fp16.h>

#include <algorithm>

#include "qsa_attn_common.cuh"
#include "qsa_paged.cuh"
#include "qsa_rope.cuh"

namespace qsa {

namespace {

using namespace paged;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 4;   // of a CTA that writes
__device__ int g_bad_pages;

// D / 32 consecutive values of a row of bf16 from lane * (D / 32) on.
template <int D>
__device__ __forceinline__ void load_lane(const __nv_bfloat16* src, uint32_t (&u)[D / 64]) {
  if constexpr (D == 256) {
    const uint4 w = *reinterpret_cast<const uint4*>(src);
    u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(src);
    u[0] = w.x, u[1] = w.y;
  }
}

// The rotation of a row that lies over a warp, rounded to bf16.
template <int D>
__device__ __forceinline__ void rotate_lane(uint32_t (&u)[D / 64], const qsa_rope& r, const float2* cs, int lane) {
  constexpr int PER = D / 32;
  const int c0 = lane * PER, half = r.rot_dim / 2;
  const bool turns = c0 < r.rot_dim, upper = c0 >= half;
  uint32_t y[D / 64];
  if (r.pairs) {
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      const float2 t = cs[rope::cs_at<2>(r.rot_dim, turns ? c0 / 2 + k : 0)];
      const float a = bf16_lo(u[k]), b = bf16_hi(u[k]);
      const __nv_bfloat162 w = __floats2bfloat162_rn(rope::low_of(a, b, t), rope::high_of(a, b, t));
      y[k] = *reinterpret_cast<const uint32_t*>(&w);
    }
  } else {
    // (rot_dim is a multiple of 16: half of it is whole lanes.)
    const int from = turns ? (upper ? lane - half / PER : lane + half / PER) : lane;
    const int i0 = turns ? c0 - (upper ? half : 0) : 0;
#pragma unroll
    for (int k = 0; k < D / 64; ++k) {
      const uint32_t other = __shfl_sync(0xffffffffu, u[k], from);
      const float2 t0 = cs[rope::cs_at<2>(r.rot_dim, i0 + 2 * k)], t1 = cs[rope::cs_at<2>(r.rot_dim, i0 + 2 * k + 1)];
      const float m0 = bf16_lo(u[k]), m1 = bf16_hi(u[k]), o0 = bf16_lo(other), o1 = bf16_hi(other);
      const __nv_bfloat162 w = upper ? __floats2bfloat162_rn(rope::high_of(o0, m0, t0), rope::high_of(o1, m1, t1))
                                     : __floats2bfloat162_rn(rope::low_of(m0, o0, t0), rope::low_of(m1, o1, t1));
      y[k] = *reinterpret_cast<const uint32_t*>(&w);
    }
  }
#pragma unroll
  for (int k = 0; k < D / 64; ++k) u[k] = turns ? y[k] : u[k];
}

// A row that lies over a warp, as E4M3 codes and a scale (as qsa_append_tokens).
template <int D>
__device__ __forceinline__ void store_fp8(const PagedAppendParams& p, const uint32_t (&u)[D / 64], int which, int64_t row,
                                          int64_t record, int lane) {
  constexpr int PER = D / 32;
  float x[PER];
#pragma unroll
  for (int k = 0; k < PER / 2; ++k) {
    x[2 * k] = bf16_lo(u[k]);
    x[2 * k + 1] = bf16_hi(u[k]);
  }
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < PER; ++k) amax = fmaxf(amax, fabsf(x[k]));
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const __half sh = __float2half_rn(__fdiv_rn(amax, 448.0f));
  const float sc = __half2float(sh);
  uint32_t c[PER / 2];
#pragma unroll
  for (int k = 0; k < PER / 2; ++k) c[k] = e4m3_codes(x[2 * k], x[2 * k + 1], sc);
  uint8_t* dst = static_cast<uint8_t*>(which ? p.v : p.k) + row + lane * PER;
  if constexpr (PER == 8)
    *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  else
    *reinterpret_cast<uint32_t*>(dst) = c[0] | (c[1] << 16);
  if (lane == 0) static_cast<__half*>(p.kv_scale)[2 * record + which] = sh;
}

// ... as 4-bit codes with a scale and a minimum for each 32 channels.
template <int D>
__device__ __forceinline__ void store_q4(const PagedAppendParams& p, const uint32_t (&u)[D / 64], int which, int64_t row,
                                         int64_t record, int lane) {
  constexpr int PER = D / 32, G = D / 32, LB = 32 / G;   // LB: lanes of a block
  float x[PER];
#pragma unroll
  for (int k = 0; k < PER / 2; ++k) {
    x[2 * k] = bf16_lo(u[k]);
    x[2 * k + 1] = bf16_hi(u[k]);
  }
  float lo = INFINITY, hi = -INFINITY;
  // What f16 does not hold (65,280 is the largest bf16 value that it does, and leaves the
  // rounding of scale and minimum room): infinities, NaN, larger values.
  bool odd = false;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    lo = fminf(lo, x[k]);
    hi = fmaxf(hi, x[k]);
    odd |= !(fabsf(x[k]) <= 65280.f);
  }
#pragma unroll
  for (int o = LB / 2; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  odd = ((__ballot_sync(0xffffffffu, odd) >> (lane / LB * LB)) & ((1u << LB) - 1u)) != 0u;
  const __half mh = odd ? __ushort_as_half((unsigned short)0) : __float2half_rn(lo);
  __half sh = __float2half_rn(__fdiv_rn(hi - lo, 15.0f));
  if (odd) sh = __ushort_as_half((unsigned short)0x7fff);
  const float m = __half2float(mh), s = __half2float(sh);
  uint32_t codes = 0u;   // 4 bits a channel
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    // (A scale that is 0 or NaN leaves code 0; so do differences that are not above 0, which
    // are not divided: every block has one that is 0, and a division of 0 takes ten times as
    // long.)
    const float d = x[k] - m;
    const float c = s > 0.f && d > 0.f ? fminf(rintf(__fdiv_rn(d > 0.f ? d : s, s)), 15.f) : 0.f;
    codes |= (uint32_t)c << (4 * k);
  }
  // 32-bit word w of the row: units 2 w and 2 w + 1, of blocks g and g + 1 and the same n.
  uint8_t* dst = static_cast<uint8_t*>(which ? p.v : p.k) + row;
  const int n = 2 * lane / G, g = (2 * lane) % G;
  if constexpr (D == 256) {   // lane 4 g + n / 2 holds units n (even: low half)
    const uint32_t a = __shfl_sync(0xffffffffu, codes, 4 * g + n / 2), b = __shfl_sync(0xffffffffu, codes, 4 * g + 4 + n / 2);
    reinterpret_cast<uint32_t*>(dst)[lane] = __byte_perm(a, b, n & 1 ? 0x7632 : 0x5410);
  } else {                    // lane 8 g + n holds unit n
    const uint32_t a = __shfl_sync(0xffffffffu, codes, (8 * g + n) & 31), b = __shfl_sync(0xffffffffu, codes, (8 * g + 8 + n) & 31);
    if (lane < 16) reinterpret_cast<uint32_t*>(dst)[lane] = __byte_perm(a, b, 0x5410);
  }
  if (lane % LB == 0) {
    const __half2 pair = __halves2half2(sh, mh);
    reinterpret_cast<__half2*>(static_cast<char*>(p.kv_scale) + record * (D / 4))[which * G + lane / LB] = pair;
  }
}

// The sequence of row r and its position, by one warp (-1: nobody's).  The first 32
// sequences' ranges and lengths are read at once; more are counted 256 at a time.
__device__ __forceinline__ int warp_sequence(const PagedAppendParams& a, int r, int lane, int& pos) {
  int first = 0, end = 0, len = 0;
  if (lane < a.n_seqs) {
    first = __ldcg(a.row_start + lane);
    end = __ldcg(a.row_start + lane + 1);
    len = __ldcg(a.lens + lane);
  }
  int seq = __popc(__ballot_sync(0xffffffffu, lane < a.n_seqs && end <= r));   // ranges that end at or before it
  if (seq < 32) {
    first = __shfl_sync(0xffffffffu, first, seq);
    end = __shfl_sync(0xffffffffu, end, seq);
    len = __shfl_sync(0xffffffffu, len, seq);
  } else {
    for (int i0 = 32; i0 < a.n_seqs; i0 += 256) {
      int mine = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + 32 * k + lane;
        mine += i < a.n_seqs && __ldcg(a.row_start + i + 1) <= r;
      }
      const int sum = __reduce_add_sync(0xffffffffu, mine);
      seq += sum;
      if (sum < 256) break;
    }
    if (seq < a.n_seqs) {
      first = __ldcg(a.row_start + seq);
      end = __ldcg(a.row_start + seq + 1);
      len = __ldcg(a.lens + seq);
    }
  }
  if (seq >= a.n_seqs || r < first) return -1;
  pos = max(len, 0) - (min(end, a.n_rows) - r);
  return seq;
}

// STATE: how the cache holds K and V.  D: head_dim.
template <int STATE, int D>
__global__ void __launch_bounds__(kThreads, 4) paged_rows_kernel(const __grid_constant__ PagedRowsParams p) {
  constexpr bool QUANT = STATE == QSA_FP8_E4M3 || STATE == QSA_Q4_1;
  constexpr int ES = STATE == QSA_F32 ? 4 : 2;          // of the rows
  constexpr int J = D * ES / 32;                        // jobs of a head
  const PagedAppendParams& a = p.a;
  __shared__ __align__(16) float2 cs[kMaxRows][QSA_MAX_ROPE_PAIRS];
  __shared__ int64_t page_s[kMaxRows];                  // -1: no page, -2: nobody's row
  __shared__ int pos_s[kMaxRows];
  grid_dependency_sync();
  const int tid = (int)threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = (int)blockIdx.x * p.rows, rows = min(p.rows, a.n_rows - r0);
  const int q_heads = p.q ? p.n_q_heads : 0;
  // A row is 256, 128 or 64 threads' (rows of a CTA are a power of two).  Its heads -- Q's,
  // then those of rows stored as they are, K's and V's -- are J jobs each, of which a
  // thread takes the same one of every `step`th head: its pieces and angles stay the same.
  const int row_shift = p.rows == 1 ? 8 : p.rows == 2 ? 7 : 6, per = 1 << row_shift;
  const int my = tid >> row_shift, t = tid & (per - 1);
  const int h0 = t / J, j = t % J, step = per / J;
  const int heads = my < rows ? q_heads + (QUANT ? 0 : 2 * a.n_kv_heads) : 0;
  const int64_t r = (int64_t)r0 + my;
  const rope::Job job = rope::job_of<ES>(p.rope.rot_dim, p.rope.pairs, j);
  const char* const q_row = static_cast<const char*>(p.q) + r * p.q_row_stride * ES;
  auto source = [&](int h) {
    if (h < q_heads) return q_row + h * p.q_head_stride * ES;
    const int hv = h - q_heads, v = hv >= a.n_kv_heads;
    return static_cast<const char*>(v ? a.v_new : a.k_new) + (r * a.row_stride + (v ? hv - a.n_kv_heads : hv) * a.new_head_stride) * ES;
  };
  constexpr int kAhead = 2;   // (3 spill)
  uint4 x0[kAhead], x1[kAhead];
  auto load = [&](int from) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int h = from + k * step;
      if (h >= heads) break;
      const uint4* const x = reinterpret_cast<const uint4*>(source(h));
      x0[k] = x[job.p0];
      x1[k] = x[job.p1];
    }
  };
  // Rows that are quantized, a warp each: unit w of the row is K or V of a head.
  const int units = QUANT && my < rows ? 2 * a.n_kv_heads : 0, unit0 = t >> 5, unit_step = per >> 5;
  uint32_t u[QUANT ? D / 64 : 1];
  auto load_row = [&](int w) {
    if constexpr (QUANT) {
      const int v = w >= a.n_kv_heads;
      load_lane<D>(static_cast<const __nv_bfloat16*>(v ? a.v_new : a.k_new) + r * a.row_stride +
                       (v ? w - a.n_kv_heads : w) * a.new_head_stride + lane * (D / 32),
                   u);
    }
  };
  if (unit0 < units) load_row(unit0);
  load(h0);
  // A warp a row: its sequence and position; its page arrives while the angles are computed.
  int64_t page = -2;
  int32_t id = 0;
  if (warp < rows) {
    int pos = 0;
    const int seq = warp_sequence(a, r0 + warp, lane, pos);
    if (seq >= 0) {
      const int64_t at = pos >> a.page_shift;
      page = pos >= 0 ? 0 : -1;
      id = pos >= 0 && at < a.table_ld ? __ldcg(a.table + seq * a.table_ld + at) : -1;
    }
    if (lane == 0) pos_s[warp] = pos;
  }
  __syncthreads();
  const int half = p.rope.rot_dim / 2;
  if (my < rows) {
    const int pos = pos_s[my];
    for (int k = t; k < half; k += per) cs[my][rope::cs_at<ES>(p.rope.rot_dim, k)] = rope::turn(p.rope, k, pos);
  }
  if (warp < rows && lane == 0) {
    if (page == 0) {
      page = (uint32_t)id < (uint32_t)a.n_pages ? id : -1;
      if (page < 0) atomicAdd(&g_bad_pages, 1);
    }
    page_s[warp] = page;
  }
  __syncthreads();
  if (my >= rows) return;
  page = page_s[my];
  if (page == -2) return;
  const int64_t slot = pos_s[my] & ((1 << a.page_shift) - 1);
  if (heads > 0) {
    char* const q_to = static_cast<char*>(p.q_out) + r * q_heads * (D * ES);
    const int64_t kv_to = (page * a.page_stride + slot * a.tok_stride) * ES;
    for (int from = h0; from < heads; from += kAhead * step) {
      if (from != h0) load(from);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int h = from + k * step;
        if (h >= heads) break;
        const int hv = h - q_heads, v = hv >= a.n_kv_heads;
        if (job.turns && hv < a.n_kv_heads) {
          float2 angle[16 / ES];
          rope::angles_of<ES>(p.rope.rot_dim, j, cs[my], angle);
          rope::rotate_job<ES>(x0[k], x1[k], p.rope.pairs, angle);
        }
        char* to = q_to + h * (D * ES);
        if (hv >= 0) {
          if (page < 0) break;
          to = static_cast<char*>(v ? a.v : a.k) + kv_to + (v ? hv - a.n_kv_heads : hv) * a.head_stride * ES;
        }
        reinterpret_cast<uint4*>(to)[job.p0] = x0[k];
        reinterpret_cast<uint4*>(to)[job.p1] = x1[k];
      }
    }
  }
  if constexpr (QUANT) {
    if (page < 0) return;
    const int64_t row = page * a.page_stride + slot * a.tok_stride, record = page * a.s_page_stride + slot * a.s_tok_stride;
    for (int w = unit0; w < units; w += unit_step) {
      if (w != unit0) load_row(w);
      const int v = w >= a.n_kv_heads, h = v ? w - a.n_kv_heads : w;
      if (!v && half > 0) rotate_lane<D>(u, p.rope, cs[my], lane);
      const int64_t at = row + h * a.head_stride, rec = record + h * a.s_head_stride;
      if constexpr (STATE == QSA_Q4_1) store_q4<D>(a, u, v, at / 2, rec, lane);
      else store_fp8<D>(a, u, v, at, rec, lane);
    }
  }
}

// ------------------------------------------------------------------ reading
// A warp takes rows_warp rows: lane i looks up row i's page, so their chains of
// dependent reads (range, length, table) run side by side; then K and V of their heads,
// 16 bytes of codes a lane (4-bit: 32 values, so that several rows are under way), or a
// row over the warp.
template <typename OUT>
__device__ __forceinline__ void put4(OUT* to, float a, float b, float c, float d) {
  if constexpr (sizeof(OUT) == 4) {
    *reinterpret_cast<float4*>(to) = make_float4(a, b, c, d);
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2*>(to) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

template <int STATE, int D, typename OUT>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(const __grid_constant__ PagedReadParams p) {
  const PagedAppendParams& a = p.a;
  grid_dependency_sync();
  const int lane = (int)threadIdx.x & 31;
  const int64_t r0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * p.rows_warp;
  // This lane's row.
  int64_t page = -1, slot = 0;
  const int64_t mine = r0 + lane;
  if (lane < p.rows_warp && mine < a.n_rows) {
    int lo = 0, hi = a.n_seqs;   // the sequences that end at or before it: found in [lo, hi]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(a.row_start + mid + 1) <= mine) lo = mid + 1;
      else hi = mid;
    }
    if (lo < a.n_seqs && mine >= __ldcg(a.row_start + lo)) {
      const int pos = max(__ldcg(a.lens + lo), 0) - (min(__ldcg(a.row_start + lo + 1), a.n_rows) - (int)mine);
      if (pos >= 0) {
        const int64_t j = pos >> a.page_shift;
        const int32_t id = j < a.table_ld ? __ldcg(a.table + lo * a.table_ld + j) : -1;
        slot = pos & ((1 << a.page_shift) - 1);
        if ((uint32_t)id < (uint32_t)a.n_pages) page = id;
        else atomicAdd(&g_bad_pages, 1);
      }
    }
  }
  // Units: K or V of a head of a row.  LU lanes share one, 32 / LU at a time.
  constexpr int LU = STATE == QSA_Q4_1 ? D / 32 : 32, UW = 32 / LU;
  const int n = (int)min((int64_t)p.rows_warp, a.n_rows - r0), each = 2 * a.n_kv_heads, all = n * each;
  const int sub = lane / LU, li = lane % LU;
  constexpr int kAhead = 2;   // units of a lane in flight
#pragma unroll 1
  for (int u0 = 0; u0 < all; u0 += kAhead * UW) {
    constexpr int ES = STATE == QSA_F32 ? 4 : STATE == QSA_BF16 ? 2 : 1;
    constexpr int NW = STATE == QSA_Q4_1 ? 1 + D / 128 : (D * ES / 32 + 15) / 16;   // 16-byte pieces of a lane
    uint4 w[kAhead][NW];
    float sc[kAhead];
    OUT* to[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int u = u0 + k * UW + sub, i = u / each, hv = u - i * each;
      const int64_t pg = __shfl_sync(0xffffffffu, page, i & 31), sl = __shfl_sync(0xffffffffu, slot, i & 31);
      to[k] = nullptr;
      if (u >= all || pg < 0) continue;
      const int which = hv >= a.n_kv_heads, h = which ? hv - a.n_kv_heads : hv;
      const int64_t at = pg * a.page_stride + h * a.head_stride + sl * a.tok_stride;
      const int64_t record = pg * a.s_page_stride + h * a.s_head_stride + sl * a.s_tok_stride;
      const char* from = static_cast<const char*>(which ? a.v : a.k);
      to[k] = static_cast<OUT*>(which ? p.v_out : p.k_out) + ((r0 + i) * a.n_kv_heads + h) * D;
      if constexpr (STATE == QSA_Q4_1) {
        w[k][0] = __ldcs(reinterpret_cast<const uint4*>(from + at / 2) + li);
        const uint4* rec = reinterpret_cast<const uint4*>(static_cast<const char*>(a.kv_scale) + record * (D / 4) + which * (D / 8));
#pragma unroll
        for (int x = 0; x < D / 128; ++x) w[k][1 + x] = __ldg(rec + x);
      } else if constexpr (D * ES / 32 >= 16) {
#pragma unroll
        for (int x = 0; x < NW; ++x) w[k][x] = __ldcs(reinterpret_cast<const uint4*>(from + at * ES) + 32 * x + lane);
      } else if constexpr (D * ES / 32 == 8) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(from + at * ES) + lane);
        w[k][0] = make_uint4(v.x, v.y, 0u, 0u);
      } else {
        w[k][0].x = __ldcs(reinterpret_cast<const uint32_t*>(from + at * ES) + lane);
      }
      if constexpr (STATE == QSA_FP8_E4M3) sc[k] = __half2float(__ldg(static_cast<const __half*>(a.kv_scale) + 2 * record + which));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (to[k] == nullptr) continue;
      if constexpr (STATE == QSA_Q4_1) {
        // The lane's 16 bytes: unit li of all eight blocks (D = 256), or units 2 li and 2 li + 1 of all four.
        constexpr int G = D / 32;
        const uint32_t c4[4] = {w[k][0].x, w[k][0].y, w[k][0].z, w[k][0].w};
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int g = x % G, unit = D == 256 ? li : 2 * li + x / G;
          const uint4 r4 = w[k][1 + g / 4];
          const uint32_t word = (g & 3) == 0 ? r4.x : (g & 3) == 1 ? r4.y : (g & 3) == 2 ? r4.z : r4.w;
          const __half2 sm = *reinterpret_cast<const __half2*>(&word);
          const float s = __low2float(sm), m = __high2float(sm);
          const uint32_t c = c4[x / 2] >> (16 * (x & 1));
          put4(to[k] + 32 * g + 4 * unit, fmaf((float)(c & 15u), s, m), fmaf((float)((c >> 4) & 15u), s, m),
               fmaf((float)((c >> 8) & 15u), s, m), fmaf((float)((c >> 12) & 15u), s, m));
        }
      } else if constexpr (STATE == QSA_F32) {
#pragma unroll
        for (int x = 0; x < NW; ++x)
          put4(to[k] + 128 * x + 4 * lane, __uint_as_float(w[k][x].x), __uint_as_float(w[k][x].y), __uint_as_float(w[k][x].z),
               __uint_as_float(w[k][x].w));
      } else if constexpr (STATE == QSA_BF16) {
        constexpr int PER = D / 32;
        put4(to[k] + PER * lane, bf16_lo(w[k][0].x), bf16_hi(w[k][0].x), bf16_lo(w[k][0].y), bf16_hi(w[k][0].y));
        if constexpr (PER == 8)
          put4(to[k] + PER * lane + 4, bf16_lo(w[k][0].z), bf16_hi(w[k][0].z), bf16_lo(w[k][0].w), bf16_hi(w[k][0].w));
      } else {
        constexpr int PER = D / 32;
#pragma unroll
        for (int x = 0; x < PER / 4; ++x) {
          const uint32_t v = x ? w[k][0].y : w[k][0].x;
          const uint32_t b0 = attn::e4m3x2_to_bf16x2(v & 0xffffu), b1 = attn::e4m3x2_to_bf16x2(v >> 16);
          put4(to[k] + PER * lane + 4 * x, bf16_lo(b0) * sc[k], bf16_hi(b0) * sc[k], bf16_lo(b1) * sc[k], bf16_hi(b1) * sc[k]);
        }
      }
    }
  }
}

template <int STATE>
cudaError_t launch_rows(PagedRowsParams p, cudaStream_t st) {
  // As many rows a CTA as leave eight CTAs for every SM.
  p.rows = 1;
  while (p.rows < kMaxRows && p.a.n_rows > 8 * device_sm_count() * p.rows) p.rows *= 2;
  const dim3 grid((unsigned)(((int64_t)p.a.n_rows + p.rows - 1) / p.rows)), block(kThreads);
  return p.a.head_dim == 256 ? launch_kernel(paged_rows_kernel<STATE, 256>, grid, block, 0, st, 0u, p)
                             : launch_kernel(paged_rows_kernel<STATE, 128>, grid, block, 0, st, 0u, p);
}

template <int STATE, typename OUT>
cudaError_t launch_read(const PagedReadParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)(((int64_t)p.a.n_rows + kWarps * p.rows_warp - 1) / (kWarps * p.rows_warp))), block(kThreads);
  return p.a.head_dim == 256 ? launch_kernel(paged_read_kernel<STATE, 256, OUT>, grid, block, 0, st, 0u, p)
                             : launch_kernel(paged_read_kernel<STATE, 128, OUT>, grid, block, 0, st, 0u, p);
}
template <int STATE>
cudaError_t launch_read_as(const PagedReadParams& p, qsa_dtype out, cudaStream_t st) {
  return out == QSA_F32 ? launch_read<STATE, float>(p, st) : launch_read<STATE, __nv_bfloat16>(p, st);
}

}  // namespace

cudaError_t launch_paged_rows(const PagedRowsParams& p, qsa_dtype kv_dtype, cudaStream_t st) {
  switch (kv_dtype) {
    case QSA_F32: return launch_rows<QSA_F32>(p, st);
    case QSA_BF16: return launch_rows<QSA_BF16>(p, st);
    case QSA_FP8_E4M3: return launch_rows<QSA_FP8_E4M3>(p, st);
    default: return launch_rows<QSA_Q4_1>(p, st);
  }
}

cudaError_t launch_paged_read(PagedReadParams p, qsa_dtype kv_dtype, qsa_dtype out_dtype, cudaStream_t st) {
  // As many rows a warp as leave a warp for every SM's place.
  const int64_t warps = (int64_t)device_sm_count() * 64;
  p.rows_warp = 1;
  while (p.rows_warp < 32 && p.a.n_rows > warps * p.rows_warp) p.rows_warp *= 2;
  switch (kv_dtype) {
    case QSA_F32: return launch_read_as<QSA_F32>(p, out_dtype, st);
    case QSA_BF16: return launch_read_as<QSA_BF16>(p, out_dtype, st);
    case QSA_FP8_E4M3: return launch_read_as<QSA_FP8_E4M3>(p, out_dtype, st);
    default: return launch_read_as<QSA_Q4_1>(p, out_dtype, st);
  }
}

int paged_rows_bad_pages_take() { return take_counter(g_bad_pages); }

}  // namespace qsa
