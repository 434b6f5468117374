// Rotary positions (include/qsa.h): the cosine and sine of a pair's angle, and
// the rotation of 16-byte pieces of a row.  Shared by qsa_rotate.cu (rows by
// themselves) and qsa_paged_rows.cu (rows on their way into a paged cache).
#pragma once

#include "qsa_internal.cuh"

namespace qsa {
namespace rope {

// (cos, sin) of pair i at position pos, times the magnitude.  The angle in turns is
// (pos * turns[i] mod 2^64) / 2^64: one integer product, exact for every position.  Its
// nearest quarter turn is taken off as an integer, and what is left, in [-1/8, 1/8] of a
// turn, becomes binary32 from all of its bits: an angle however small keeps 24 of them,
// and opposite positions have opposite angles.
__device__ __forceinline__ float2 turn(const qsa_rope& r, int i, int pos) {
  const uint64_t a = r.turns[i] * (uint64_t)(int64_t)pos;
  const uint32_t quarter = (uint32_t)((a + (1ull << 61)) >> 62);
  float s, c;
  sincospif(__ll2float_rn((int64_t)(a - ((uint64_t)quarter << 62))) * 0x1p-63f, &s, &c);
  if (quarter & 1u) {
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2u) {
    c = -c;
    s = -s;
  }
  return make_float2(c * r.magnitude, s * r.magnitude);
}

// The rotation of (a, b), in one order of operations everywhere: a row's bits do not
// depend on the call that rotates it.
__device__ __forceinline__ float low_of(float a, float b, float2 cs) { return fmaf(a, cs.x, -__fmul_rn(b, cs.y)); }
__device__ __forceinline__ float high_of(float a, float b, float2 cs) { return fmaf(b, cs.x, __fmul_rn(a, cs.y)); }

// Values of a 16-byte piece: 4 of f32 (ES = 4) or 8 of bf16 (ES = 2).
template <int ES>
__device__ __forceinline__ void open(const uint4& p, float (&v)[16 / ES]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (ES == 4) {
      v[i] = __uint_as_float(w[i]);
    } else {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}
template <int ES>
__device__ __forceinline__ uint4 close(const float (&v)[16 / ES]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (ES == 4) {
      w[i] = __float_as_uint(v[i]);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A head's row is cut into jobs of two pieces: those that a rotation joins (halves:
// piece j and the one rot_dim / 2 channels on; neighbours: pieces 2j and 2j + 1),
// then two pieces at a time of what is not rotated.
struct Job {
  int p0, p1;   // pieces
  bool turns;
};
template <int ES>
__device__ __forceinline__ Job job_of(int rot_dim, int pairs, int j) {
  constexpr int E = 16 / ES;
  const int n = rot_dim / (2 * E);   // jobs that rotate
  Job b;
  b.turns = j < n;
  b.p0 = b.turns && !pairs ? j : 2 * j;
  b.p1 = b.turns && !pairs ? j + n : 2 * j + 1;
  return b;
}
// A row's (cos, sin) in shared memory: of job j's pairs E j .. E j + E - 1, pair e is at e
// times the jobs plus j, so that a warp's loads (a job a lane) are consecutive.
template <int ES>
__device__ __forceinline__ int cs_at(int rot_dim, int pair) {
  constexpr int E = 16 / ES;
  return pair % E * (rot_dim / (2 * E)) + pair / E;
}
// Those of job j's pairs.
template <int ES>
__device__ __forceinline__ void angles_of(int rot_dim, int j, const float2* cs, float2 (&t)[16 / ES]) {
  constexpr int E = 16 / ES;
#pragma unroll
  for (int e = 0; e < E; ++e) t[e] = cs[e * (rot_dim / (2 * E)) + j];
}
// Rotates a job's pieces in place.
template <int ES>
__device__ __forceinline__ void rotate_job(uint4& x0, uint4& x1, int pairs, const float2 (&t)[16 / ES]) {
  constexpr int E = 16 / ES;
  float a[E], b[E], c[E], d[E];
  open<ES>(x0, a);
  open<ES>(x1, b);
  if (pairs) {
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      c[2 * e] = low_of(a[2 * e], a[2 * e + 1], t[e]);
      c[2 * e + 1] = high_of(a[2 * e], a[2 * e + 1], t[e]);
      d[2 * e] = low_of(b[2 * e], b[2 * e + 1], t[E / 2 + e]);
      d[2 * e + 1] = high_of(b[2 * e], b[2 * e + 1], t[E / 2 + e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      c[e] = low_of(a[e], b[e], t[e]);
      d[e] = high_of(a[e], b[e], t[e]);
    }
  }
  x0 = close<ES>(c);
  x1 = close<ES>(d);
}

}  // namespace rope
}  // namespace qsa
