// Attention of a batch's newest rows over a paged K/V cache: the CUDA-core
// kernel, and the joining of an item's parts (see qsa_paged.cuh for the
// division of the work).
//
// For entry f = (row at position p, query head) of KV head g, with
// z_t = scale * q . k_t over the tokens t that the row sees:
//   m = max_t z_t,  l = sum_t exp(z_t - m),  out = sum_t exp(z_t - m) v_t / l,
//   lse = m + log l,
// in one pass over the key tiles with the running m and l of each entry (32-bit
// sums): a tile's new maximum m' rescales l and the output by exp(m - m').
#include <math.h>

#include "qsa_attn_common.cuh"
#include "qsa_paged.cuh"

namespace qsa {

namespace {

using namespace paged;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ int g_bad_pages;   // table entries outside [0, n_pages) among the tokens that a call read

// ------------------------------------------------------------------ CUDA-core kernel
// 256 threads; an item is 16 entries, a key tile 32 tokens.  Thread -> channel
// d = tid % D of entries tid / D, tid / D + 256 / D, ...
constexpr int kSimtThreads = 256;
constexpr int kSimtMT = 16;
constexpr int kSimtKT = 32;

template <int D>
struct SimtLayout {
  static constexpr int kK = kSimtKT * (D + 1);   // rows padded by one word: threads of a warp read different banks
  static constexpr int kV = kSimtKT * D;
  static constexpr size_t floats = kSimtMT * D + kK + kV + kSimtMT * 33 + 3 * kSimtMT;
  static constexpr size_t bytes = floats * 4 + kSimtKT * 4;
};

// One element of the cache as a 32-bit value (fp8: without its scale).
template <int DT>
__device__ __forceinline__ float cache_value(const void* base, int64_t off) {
  if constexpr (DT == QSA_F32) return static_cast<const float*>(base)[off];
  if constexpr (DT == QSA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[off]);
  const uint32_t two = attn::e4m3x2_to_bf16x2(static_cast<const uint8_t*>(base)[off]);
  return bf16_lo(two);
}

template <int D, int DT>
__global__ void __launch_bounds__(kSimtThreads) paged_simt_kernel(const PagedParams p) {
  constexpr int HS = kSimtThreads / D, NE = kSimtMT / HS;
  extern __shared__ __align__(16) float fsm[];
  float* q_s = fsm;                                 // [16][D]
  float* k_s = q_s + kSimtMT * D;                   // [32][D + 1]
  float* v_s = k_s + SimtLayout<D>::kK;             // [32][D]
  float* z_s = v_s + SimtLayout<D>::kV;             // [16][33]
  float* m_s = z_s + kSimtMT * 33;
  float* l_s = m_s + kSimtMT;
  float* a_s = l_s + kSimtMT;
  int* ok_s = reinterpret_cast<int*>(a_s + kSimtMT);
  __shared__ int64_t scan_s[kSimtThreads / 32];
  __shared__ Start start_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dependency_sync();
  const Start st = find_run<kSimtThreads, kSimtKT>(p, p.mt, blockIdx.x, gridDim.x, scan_s, &start_s);
  Cursor<kSimtKT> c;
  c.begin(p, p.mt, st);
  const float zscale = p.scale * kLog2e;
  const int d = tid % D, hs = tid / D;
  for (bool more = st.n > 0; more;) {
    const int f0 = c.m * kSimtMT, nf = min(kSimtMT, c.s.n * p.group - f0);
    const int pos0 = c.s.len - c.s.n;
    // Entry f of the item -> its row and query head.
    auto entry = [&](int f) {
      const int r = (f0 + f) / p.group;
      return ((int64_t)(c.s.row0 + r) * p.n_q_heads + c.head * p.group + (f0 + f - r * p.group));
    };
    __syncthreads();
    for (int i = tid; i < nf * D; i += kSimtThreads) {
      const int64_t at = entry(i / D) * D + i % D;
      q_s[i] = DT == QSA_F32 ? static_cast<const float*>(p.q)[at]
                             : __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[at]);
    }
    if (tid < kSimtMT) {
      m_s[tid] = -INFINITY;
      l_s[tid] = 0.f;
    }
    float acc[NE];
#pragma unroll
    for (int j = 0; j < NE; ++j) acc[j] = 0.f;
    // Tokens that no row of the item sees are not read.
    const int pos_last = pos0 + (f0 + nf - 1) / p.group, pos_first = pos0 + f0 / p.group;
    for (int x = c.x; x < c.x1; ++x) {
      const int t0 = c.tiles.token(x);
      __syncthreads();
      for (int tk = warp; tk < kSimtKT; tk += kSimtThreads / 32) {
        const int t = t0 + tk;
        int32_t page = 0;
        bool ok = t <= pos_last && (p.window == 0 || t > pos_first - p.window || t < p.n_sinks);
        if (ok && !page_of(p, c.seq, t, page)) {
          if (lane == 0) atomicAdd(&g_bad_pages, 1);
          ok = false;
        }
        const int64_t slot = t & ((1 << p.page_shift) - 1);
        const int64_t off = page * p.page_stride + c.head * p.head_stride + slot * p.tok_stride;
        float ks = 1.f, vs = 1.f;
        if (DT == QSA_FP8_E4M3 && ok) {
          const __half2 s = *reinterpret_cast<const __half2*>(
              p.kv_scale + 4 * (page * p.s_page_stride + c.head * p.s_head_stride + slot * p.s_tok_stride));
          ks = __low2float(s);
          vs = __high2float(s);
        }
        for (int e = lane; e < D; e += 32) {
          k_s[tk * (D + 1) + e] = ok ? cache_value<DT>(p.k, off + e) * ks : 0.f;
          v_s[tk * D + e] = ok ? cache_value<DT>(p.v, off + e) * vs : 0.f;
        }
        if (lane == 0) ok_s[tk] = ok ? 1 : 0;
      }
      __syncthreads();
      for (int i = tid; i < nf * kSimtKT; i += kSimtThreads) {
        const int f = i / kSimtKT, tk = i % kSimtKT;
        float dot = 0.f;
        for (int e = 0; e < D; ++e) dot = fmaf(q_s[f * D + e], k_s[tk * (D + 1) + e], dot);
        z_s[f * 33 + tk] = ok_s[tk] && sees(p, pos0 + (f0 + f) / p.group, t0 + tk) ? dot * zscale : -INFINITY;
      }
      __syncthreads();
      for (int f = warp; f < nf; f += kSimtThreads / 32) {
        const float z = z_s[f * 33 + lane], mo = m_s[f];
        float mn = fmaxf(mo, z);
#pragma unroll
        for (int o = 16; o; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        const float pz = mn == -INFINITY ? 0.f : exp2f(z - mn);
        float sum = pz;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        z_s[f * 33 + lane] = pz;
        if (lane == 0) {
          const float alpha = mo == -INFINITY ? 0.f : exp2f(mo - mn);
          a_s[f] = alpha;
          m_s[f] = mn;
          l_s[f] = l_s[f] * alpha + sum;
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < NE; ++j) {
        const int f = hs + j * HS;
        if (f < nf) {
          float a = acc[j] * a_s[f];
          for (int tk = 0; tk < kSimtKT; ++tk) a = fmaf(z_s[f * 33 + tk], v_s[tk * D + d], a);
          acc[j] = a;
        }
      }
    }
    // The item's result, or this run's part of it.
    const bool whole = c.whole();
    const int64_t slot = whole ? 0 : (int64_t)c.slot(blockIdx.x) * p.mt;
#pragma unroll
    for (int j = 0; j < NE; ++j) {
      const int f = hs + j * HS;
      if (f >= nf) continue;
      const float l = l_s[f];
      const float o = l > 0.f ? acc[j] / l : 0.f;
      if (!whole) {
        p.part_o[(slot + f) * D + d] = o;
        if (d == 0) p.part_lse[slot + f] = l > 0.f ? m_s[f] + log2f(l) : -INFINITY;
        continue;
      }
      const int64_t at = entry(f);
      if (p.out_dtype == QSA_F32) static_cast<float*>(p.out)[at * D + d] = o;
      else static_cast<__nv_bfloat16*>(p.out)[at * D + d] = __float2bfloat16(o);
      if (d == 0 && p.lse) p.lse[at] = l > 0.f ? (m_s[f] + log2f(l)) * kLn2 : -INFINITY;
    }
    Cursor<kSimtKT> last = c;
    more = c.next(p, p.mt);
    if (!more && tid == 0) describe_part(p, last, st, blockIdx.x);
  }
  if (st.n == 0 && tid == 0) p.parts[blockIdx.x] = PagedPart{};
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

template <int D, int DT>
cudaError_t launch_simt(const PagedParams& p, int grid, cudaStream_t st) {
  const size_t smem = SimtLayout<D>::bytes;
  cudaError_t e = allow_dynamic_smem((const void*)paged_simt_kernel<D, DT>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(paged_simt_kernel<D, DT>, dim3((unsigned)grid), dim3(kSimtThreads), smem, st, 0u, p);
}

}  // namespace

cudaError_t launch_paged_simt(const PagedParams& p, qsa_dtype kv_dtype, int head_dim, int grid, cudaStream_t st) {
  if (kv_dtype == QSA_F32)
    return head_dim == 256 ? launch_simt<256, QSA_F32>(p, grid, st) : launch_simt<128, QSA_F32>(p, grid, st);
  if (kv_dtype == QSA_BF16)
    return head_dim == 256 ? launch_simt<256, QSA_BF16>(p, grid, st) : launch_simt<128, QSA_BF16>(p, grid, st);
  return head_dim == 256 ? launch_simt<256, QSA_FP8_E4M3>(p, grid, st) : launch_simt<128, QSA_FP8_E4M3>(p, grid, st);
}

cudaError_t launch_paged_merge(const PagedParams& p, int head_dim, int runs, cudaStream_t st) {
  if (runs < 2) return cudaSuccess;   // one run holds every item whole
  if (runs > kMaxRuns) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(4 * device_sm_count())), block(kJoinThreads);
  return head_dim == 256 ? launch_kernel(paged_join_kernel<256>, grid, block, 0, st, 0u, p, runs)
                         : launch_kernel(paged_join_kernel<128>, grid, block, 0, st, 0u, p, runs);
}

int paged_bad_pages_take() { return take_counter(g_bad_pages); }

}  // namespace qsa
