// Rotary positions (include/qsa.h): the host functions that make a rotation, and
// the rotation of rows by themselves.
//
// One CTA takes one row, or up to four of a call that has more rows than the GPU has
// places for CTAs: their (cos, sin) by pair go to shared memory once and serve all
// heads; a thread then takes jobs of two 16-byte pieces, the two that a rotation joins,
// so that nothing is exchanged, four of them in flight.  Each value is read and written
// once; the bound is HBM for a prompt's rows and the launch with a chain of three
// dependent steps (position, angles, rows) for a step's.  On one GB300 16,384 rows of 24
// heads of 256, in and out, take 64.6 us (6.2 TB/s of the 6.7 that a copy reaches; 76 with
// a row a CTA), a step's 64 rows the 6.2 us of the host's call.
#include <math.h>

#include <algorithm>

#include "qsa_host.cuh"
#include "qsa_rope.cuh"

namespace qsa {

namespace {

constexpr int kThreads = 256, kMaxRows = 4;

struct RotateParams {
  qsa_rope rope;
  const int32_t* positions;
  const void* x;
  void* y;
  int64_t x_row, x_head, y_row, y_head;   // bytes
  int32_t n_rows, rows;                   // rows: of a CTA
  int32_t jobs_head, jobs;                // jobs of a head, of a row
  uint32_t magic_head, magic_row;         // ceil(2^32 / jobs_head), ceil(2^32 / jobs); 1: not used
  int32_t in_place;
};

// a / b by its magic number (a < 2^25, b < 2^24: the product's error stays below 1).
__device__ __forceinline__ int divide(int a, int b, uint32_t magic) {
  if (b == 1) return a;
  int q = (int)__umulhi((uint32_t)a, magic);
  if (q * b > a) --q;
  return q;
}

template <int ES>
__global__ void __launch_bounds__(kThreads, 4) rotate_kernel(const __grid_constant__ RotateParams p) {
  __shared__ __align__(16) float2 cs[kMaxRows][QSA_MAX_ROPE_PAIRS];
  grid_dependency_sync();
  const int tid = (int)threadIdx.x;
  const int r0 = (int)blockIdx.x * p.rows, rows = min(p.rows, p.n_rows - r0), all = rows * p.jobs;
  constexpr int kAhead = 4;   // jobs of a thread in flight
  uint4 x0[kAhead], x1[kAhead];
  struct Place {
    int r, h, j;
  };
  auto place = [&](int i) {
    Place a;
    a.r = divide(i, p.jobs, p.magic_row);
    const int k = i - a.r * p.jobs;
    a.h = divide(k, p.jobs_head, p.magic_head);
    a.j = k - a.h * p.jobs_head;
    return a;
  };
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * kThreads;
      if (i >= all) continue;
      const Place a = place(i);
      const rope::Job b = rope::job_of<ES>(p.rope.rot_dim, p.rope.pairs, a.j);
      if (p.in_place && !b.turns) continue;
      const char* from = static_cast<const char*>(p.x) + (r0 + a.r) * p.x_row + a.h * p.x_head;
      x0[k] = __ldcs(reinterpret_cast<const uint4*>(from) + b.p0);
      x1[k] = __ldcs(reinterpret_cast<const uint4*>(from) + b.p1);
    }
  };
  load(tid);
  const int half = p.rope.rot_dim / 2;
  for (int i = tid; i < rows * half; i += kThreads) {
    const int r = i / half, k = i - r * half;
    cs[r][rope::cs_at<ES>(p.rope.rot_dim, k)] = rope::turn(p.rope, k, __ldg(p.positions + r0 + r));
  }
  __syncthreads();
  for (int i0 = tid; i0 < all; i0 += kAhead * kThreads) {
    if (i0 != tid) load(i0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * kThreads;
      if (i >= all) continue;
      const Place a = place(i);
      const rope::Job b = rope::job_of<ES>(p.rope.rot_dim, p.rope.pairs, a.j);
      if (p.in_place && !b.turns) continue;
      if (b.turns) {
        float2 angle[16 / ES];
        rope::angles_of<ES>(p.rope.rot_dim, a.j, cs[a.r], angle);
        rope::rotate_job<ES>(x0[k], x1[k], p.rope.pairs, angle);
      }
      char* to = static_cast<char*>(p.y) + (r0 + a.r) * p.y_row + a.h * p.y_head;
      __stcs(reinterpret_cast<uint4*>(to) + b.p0, x0[k]);
      __stcs(reinterpret_cast<uint4*>(to) + b.p1, x1[k]);
    }
  }
}

// w / (2 pi) modulo 1 to the nearest 2^-64, opposite for -w.  2 pi and the quotient are
// sums of two binary64 numbers each: an fma gives what the first quotient leaves.
uint64_t turns_of(double w) {
  const double two_pi = 6.283185307179586, rest_of_two_pi = 2.4492935982947064e-16, half = 4294967296.0;
  const double x = fabs(w), q = x / two_pi;
  const double left = fmod(fma(-q, rest_of_two_pi, fma(-q, two_pi, x)) / two_pi, 1.0);
  // Both fractions in halves of 32 bits; what lies below 2^-64 counts once, in the sum.
  const double f = (q - floor(q)) * half, g = left * half, high_f = floor(f), high_g = floor(g);
  const uint64_t t = ((uint64_t)((int64_t)high_f + (int64_t)high_g) << 32) +
                     (uint64_t)nearbyint((f - high_f) * half + (g - high_g) * half);
  return w < 0.0 ? 0 - t : t;
}

}  // namespace

qsa_status check_rope(const qsa_rope* rope, int head_dim, const char* fn) {
  if (!rope) return fail(QSA_ERR_INVALID_ARG, "%s: null rope", fn);
  if (rope->rot_dim < 16 || rope->rot_dim % 16 || rope->rot_dim > 2 * QSA_MAX_ROPE_PAIRS)
    return fail(QSA_ERR_UNSUPPORTED, "%s: rot_dim=%d (a multiple of 16, 16..%d)", fn, rope->rot_dim,
                2 * QSA_MAX_ROPE_PAIRS);
  if (rope->rot_dim > head_dim)
    return fail(QSA_ERR_INVALID_ARG, "%s: rot_dim=%d of heads of %d channels", fn, rope->rot_dim, head_dim);
  if (rope->pairs != 0 && rope->pairs != 1) return fail(QSA_ERR_INVALID_ARG, "%s: rope pairs=%d", fn, rope->pairs);
  if (!isfinite(rope->magnitude)) return fail(QSA_ERR_INVALID_ARG, "%s: rope magnitude not finite", fn);
  return QSA_OK;
}

}  // namespace qsa

using namespace qsa;

QSA_API qsa_status qsa_rope_frequencies(int32_t rot_dim, double base, qsa_rope_scaling scaling, double factor,
                                        double original_tokens, double fast, double slow, double* w,
                                        float* magnitude) {
  const char* fn = "qsa_rope_frequencies";
  if (!w || !magnitude) return fail(QSA_ERR_INVALID_ARG, "%s: null pointer", fn);
  if (rot_dim < 16 || rot_dim % 16 || rot_dim > 2 * QSA_MAX_ROPE_PAIRS)
    return fail(QSA_ERR_UNSUPPORTED, "%s: rot_dim=%d (a multiple of 16, 16..%d)", fn, rot_dim, 2 * QSA_MAX_ROPE_PAIRS);
  if (scaling < QSA_ROPE_PLAIN || scaling > QSA_ROPE_PARTS)
    return fail(QSA_ERR_UNSUPPORTED, "%s: unknown scaling %d", fn, (int)scaling);
  if (!(base >= 1.0) || !isfinite(base)) return fail(QSA_ERR_INVALID_ARG, "%s: base=%g", fn, base);
  if (scaling != QSA_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor)))
    return fail(QSA_ERR_INVALID_ARG, "%s: factor=%g", fn, factor);
  if (scaling == QSA_ROPE_PARTS && (!(original_tokens > 0.0) || !isfinite(original_tokens) || !(slow >= 0.0) ||
                                    !(fast > slow) || !isfinite(fast)))
    return fail(QSA_ERR_INVALID_ARG, "%s: original_tokens=%g, fast=%g, slow=%g", fn, original_tokens, fast, slow);
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double plain = pow(base, -2.0 * i / rot_dim);
    if (scaling == QSA_ROPE_PARTS) {
      const double g = std::min(1.0, std::max(0.0, (original_tokens * plain / two_pi - slow) / (fast - slow)));
      w[i] = (1.0 - g) * plain / factor + g * plain;
    } else {
      w[i] = scaling == QSA_ROPE_LINEAR ? plain / factor : plain;
    }
  }
  *magnitude = scaling == QSA_ROPE_PARTS ? (float)(0.1 * log(factor) + 1.0) : 1.f;
  return ok();
}

QSA_API qsa_status qsa_rope_init(qsa_rope* rope, int32_t rot_dim, int32_t pairs, const double* w, float magnitude) {
  const char* fn = "qsa_rope_init";
  if (!rope || !w) return fail(QSA_ERR_INVALID_ARG, "%s: null pointer", fn);
  qsa_rope r{};
  r.rot_dim = rot_dim;
  r.pairs = pairs;
  r.magnitude = magnitude;
  const qsa_status s = check_rope(&r, 2 * QSA_MAX_ROPE_PAIRS, fn);
  if (s != QSA_OK) return s;
  for (int i = 0; i < rot_dim / 2; ++i) {
    if (!isfinite(w[i])) return fail(QSA_ERR_INVALID_ARG, "%s: frequency %d is not finite", fn, i);
    r.turns[i] = turns_of(w[i]);
  }
  *rope = r;
  return ok();
}

QSA_API qsa_status qsa_rotate(const qsa_rope* rope, const int32_t* positions, int32_t n_rows, int32_t n_heads,
                              int32_t head_dim, qsa_dtype dtype, const void* x, int64_t x_row_stride,
                              int64_t x_head_stride, void* y, int64_t y_row_stride, int64_t y_head_stride,
                              void* stream) {
  const NvtxRange nvtx_range("qsa_rotate");
  const char* fn = "qsa_rotate";
  if (!valid_dtype(dtype)) return fail(QSA_ERR_UNSUPPORTED, "%s: unknown dtype", fn);
  if (head_dim < 16 || head_dim % 16 || head_dim > 1024)
    return fail(QSA_ERR_UNSUPPORTED, "%s: head_dim=%d (a multiple of 16, 16..1024)", fn, head_dim);
  const qsa_status s = check_rope(rope, head_dim, fn);
  if (s != QSA_OK) return s;
  if (n_rows < 0 || n_heads < 0) return fail(QSA_ERR_INVALID_ARG, "%s: n_rows=%d, n_heads=%d", fn, n_rows, n_heads);
  if (n_heads > 1 << 16) return fail(QSA_ERR_UNSUPPORTED, "%s: %d heads", fn, n_heads);
  if (n_rows == 0 || n_heads == 0) return ok();
  if (!positions || !x || !y) return fail(QSA_ERR_INVALID_ARG, "%s: null pointer", fn);
  const int64_t es = (int64_t)dtype_size(dtype), most = (int64_t)1 << 40;
  const bool in_place = x == y;
  for (const int64_t st : {x_row_stride, x_head_stride, y_row_stride, y_head_stride})
    if (st < 0 || st > most)
      return fail(QSA_ERR_INVALID_ARG, "%s: a stride of %lld elements", fn, (long long)st);
  // (Rows' offsets in bytes, and the sums below, then keep to 64 bits: heads are at most 2^16.)
  if (n_rows > 1 && std::max(x_row_stride, y_row_stride) > ((int64_t)1 << 58) / (n_rows - 1))
    return fail(QSA_ERR_INVALID_ARG, "%s: %d rows %lld elements apart pass 64 bits", fn, n_rows,
                (long long)std::max(x_row_stride, y_row_stride));
  if ((n_rows > 1 && y_row_stride < head_dim) || (n_heads > 1 && y_head_stride < head_dim) ||
      (n_rows > 1 && n_heads > 1 && y_row_stride < (n_heads - 1) * y_head_stride + head_dim &&
       y_head_stride < (n_rows - 1) * y_row_stride + head_dim))
    return fail(QSA_ERR_INVALID_ARG, "%s: y's rows or heads overlap (strides %lld, %lld)", fn, (long long)y_row_stride,
                (long long)y_head_stride);
  if (in_place && (x_row_stride != y_row_stride || x_head_stride != y_head_stride))
    return fail(QSA_ERR_INVALID_ARG, "%s: in place with other strides", fn);
  if (!aligned16(x) || !aligned16(y) || (x_row_stride * es) % 16 || (x_head_stride * es) % 16 ||
      (y_row_stride * es) % 16 || (y_head_stride * es) % 16)
    return fail(QSA_ERR_MISALIGNED, "%s: x, y or their strides not 16-byte aligned", fn);
  if (reinterpret_cast<uintptr_t>(positions) & 3u)
    return fail(QSA_ERR_MISALIGNED, "%s: positions not 4-byte aligned", fn);
  RotateParams p{};
  p.rope = *rope;
  p.positions = positions;
  p.x = x;
  p.y = y;
  p.x_row = x_row_stride * es;
  p.x_head = x_head_stride * es;
  p.y_row = y_row_stride * es;
  p.y_head = y_head_stride * es;
  p.n_rows = n_rows;
  p.jobs_head = (int32_t)(head_dim * es / 32);
  p.jobs = n_heads * p.jobs_head;
  auto magic = [](int n) { return n == 1 ? 0u : (uint32_t)((((uint64_t)1 << 32) + n - 1) / n); };
  p.magic_head = magic(p.jobs_head);
  p.magic_row = magic(p.jobs);
  p.in_place = in_place ? 1 : 0;
  // As many rows a CTA as leave eight CTAs for every SM, and no more than its threads have work for.
  p.rows = 1;
  while (p.rows < kMaxRows && n_rows > 8 * device_sm_count() * p.rows && p.rows * p.jobs < 4 * kThreads) p.rows *= 2;
  const dim3 grid((unsigned)(((int64_t)n_rows + p.rows - 1) / p.rows)), block(kThreads);
  const cudaError_t e = dtype == QSA_F32 ? launch_kernel(rotate_kernel<4>, grid, block, 0, as_stream(stream), 0u, p)
                                         : launch_kernel(rotate_kernel<2>, grid, block, 0, as_stream(stream), 0u, p);
  return e == cudaSuccess ? ok() : cuda_fail(e, fn);
}
