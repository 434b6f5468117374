// Writing a batch's new tokens into the pages of a paged K/V cache: the row of
// sequence i at position p goes to slot p mod page_tokens of page
// table[i][p / page_tokens] (include/qsa.h, qsa_paged_append).
//
// One CTA per row: its sequence is the number of ranges that end at or before
// it, counted by the whole CTA, and its K and V rows are read before that, so
// the two latencies overlap.  bf16 and f32 rows are copied 16 bytes per
// thread; for an fp8 cache a warp quantizes one (K or V, head) row with the
// arithmetic of qsa_append_tokens: scale = f16(f32(amax / 448)), code = the
// E4M3 value nearest to f32(x / scale), ties to even, saturated.
//
// What bounds it: for a step's rows latencies, a launch and three dependent reads
// (range, length, page): 147 rows of bf16 in 64 sequences take 2.0 us on the GPU (in
// a graph of 50 such calls).  2,048 rows for an fp8 cache (6.3 MB, 0.9 us at the
// measured bandwidth) take 6.5 us: each row's CTA looks for its sequence by itself,
// reads 16 bytes a thread and writes 8.  A call on its own is the host's 6 to 7 us.
#include <cuda_fp16.h>

#include "qsa_paged.cuh"

namespace qsa {

namespace {

constexpr int kThreads = 128;
__device__ int g_bad_pages;

// The sequence of row r and the row's position in it, for all threads of the
// CTA; -1 when no range holds the row.
__device__ __forceinline__ int row_sequence(const PagedAppendParams& p, int r, int& pos) {
  int seq = 0;
  for (int i0 = 0; i0 < p.n_seqs; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    const int n = __syncthreads_count(i < p.n_seqs && __ldcg(p.row_start + i + 1) <= r);
    seq += n;
    if (n < kThreads) break;
  }
  if (seq >= p.n_seqs || r < __ldcg(p.row_start + seq)) return -1;
  pos = max(__ldcg(p.lens + seq), 0) - (min(__ldcg(p.row_start + seq + 1), p.n_rows) - r);
  return seq;
}

// The row's page and slot; false when it has none.
__device__ __forceinline__ bool row_page(const PagedAppendParams& p, int seq, int pos, int64_t& page, int64_t& slot) {
  if (seq < 0 || pos < 0) return false;
  const int64_t j = pos >> p.page_shift;
  const int32_t id = j < p.table_ld ? __ldcg(p.table + seq * p.table_ld + j) : -1;
  if ((uint32_t)id >= (uint32_t)p.n_pages) {
    if (threadIdx.x == 0) atomicAdd(&g_bad_pages, 1);
    return false;
  }
  page = id;
  slot = pos & ((1 << p.page_shift) - 1);
  return true;
}

// ES: bytes of an element.
template <int ES>
__global__ void __launch_bounds__(kThreads) paged_copy_kernel(const PagedAppendParams p) {
  grid_dependency_sync();
  const int r = blockIdx.x;
  const int row_chunks = p.head_dim * ES / 16, all = 2 * p.n_kv_heads * row_chunks;
  // Piece i: K or V, head, 16-byte piece of the row.
  auto source = [&](int i) {
    const int c = i % row_chunks, hv = i / row_chunks;
    const int which = hv >= p.n_kv_heads, h = which ? hv - p.n_kv_heads : hv;
    const char* base = static_cast<const char*>(which ? p.v_new : p.k_new);
    return reinterpret_cast<const uint4*>(base + (r * p.row_stride + h * p.new_head_stride) * ES + c * 16);
  };
  constexpr int kAhead = 2;
  uint4 ahead[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = (int)threadIdx.x + j * kThreads;
    if (i < all) ahead[j] = *source(i);
  }
  int pos = 0;
  int64_t page, slot;
  if (!row_page(p, row_sequence(p, r, pos), pos, page, slot)) return;
  auto put = [&](int i, const uint4& x) {
    const int c = i % row_chunks, hv = i / row_chunks;
    const int which = hv >= p.n_kv_heads, h = which ? hv - p.n_kv_heads : hv;
    char* base = static_cast<char*>(which ? p.v : p.k);
    *reinterpret_cast<uint4*>(base + (page * p.page_stride + h * p.head_stride + slot * p.tok_stride) * ES + c * 16) = x;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = (int)threadIdx.x + j * kThreads;
    if (i < all) put(i, ahead[j]);
  }
  for (int i = (int)threadIdx.x + kAhead * kThreads; i < all; i += kThreads) put(i, *source(i));
}

template <int D>
__global__ void __launch_bounds__(kThreads) paged_quantize_kernel(const PagedAppendParams p) {
  constexpr int PER = D / 32;   // values of a lane
  grid_dependency_sync();
  const int r = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rows = 2 * p.n_kv_heads;
  auto load = [&](int hv, float (&x)[PER]) {
    const int which = hv >= p.n_kv_heads, h = which ? hv - p.n_kv_heads : hv;
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(which ? p.v_new : p.k_new) + r * p.row_stride +
                               h * p.new_head_stride + lane * PER;
    uint32_t u[PER / 2];
    if constexpr (PER == 8) {
      const uint4 w = *reinterpret_cast<const uint4*>(src);
      u[0] = w.x, u[1] = w.y, u[2] = w.z, u[3] = w.w;
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(src);
      u[0] = w.x, u[1] = w.y;
    }
#pragma unroll
    for (int k = 0; k < PER / 2; ++k) {
      x[2 * k] = bf16_lo(u[k]);
      x[2 * k + 1] = bf16_hi(u[k]);
    }
  };
  float x[PER];
  if (warp < rows) load(warp, x);
  int pos = 0;
  int64_t page, slot;
  if (!row_page(p, row_sequence(p, r, pos), pos, page, slot)) return;
  for (int hv = warp; hv < rows; hv += kThreads / 32) {
    if (hv != warp) load(hv, x);
    const int which = hv >= p.n_kv_heads, h = which ? hv - p.n_kv_heads : hv;
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
    uint8_t* dst = static_cast<uint8_t*>(which ? p.v : p.k) + page * p.page_stride + h * p.head_stride +
                   slot * p.tok_stride + lane * PER;
    if constexpr (PER == 8)
      *reinterpret_cast<uint2*>(dst) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    else
      *reinterpret_cast<uint32_t*>(dst) = c[0] | (c[1] << 16);
    if (lane == 0)
      static_cast<__half*>(p.kv_scale)[2 * (page * p.s_page_stride + h * p.s_head_stride + slot * p.s_tok_stride) +
                                       which] = sh;
  }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, qsa_dtype kv_dtype, cudaStream_t st) {
  const dim3 grid((unsigned)p.n_rows), block(kThreads);
  if (kv_dtype == QSA_FP8_E4M3)
    return p.head_dim == 256 ? launch_kernel(paged_quantize_kernel<256>, grid, block, 0, st, 0u, p)
                             : launch_kernel(paged_quantize_kernel<128>, grid, block, 0, st, 0u, p);
  return kv_dtype == QSA_F32 ? launch_kernel(paged_copy_kernel<4>, grid, block, 0, st, 0u, p)
                             : launch_kernel(paged_copy_kernel<2>, grid, block, 0, st, 0u, p);
}

int paged_append_bad_pages_take() { return take_counter(g_bad_pages); }

}  // namespace qsa
