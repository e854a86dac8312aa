// vocab_rows.cuh -- what the operators on rows of logits (top logits, beam selection, distillation) share:
// row loads, order-preserving keys, and sums of exponentials about a power of two.
//
// Sums of exponentials.  With c = log2(e) / T a row's terms are exp(z / T) = 2^(c z).  A partial sum is a
// pair (n, s) that stands for s * 2^n with n a whole number held in a float: a term is 2^(fma(z, c, -n)),
// rounded once before the exponential because n is exact, and two partial sums join by an exact scaling
// with a power of two.  (With the running maximum itself as the reference, c * max is rounded and that
// rounding, relative 2^-24 of the exponent, enters every rescaling.)  c is rounded to fp32 once;
// log_sum_exp adds back delta * max for the part delta that it lost, which leaves delta * E_q[max - z].
#pragma once

#include "common.cuh"

namespace domino {

// Sums take magnitudes above kBig for kBig, so that a masked value of the type's lowest, or an infinity, meets
// others in 64 bits with 2e-7 to spare at any temperature.  A row whose maximum lies within kPlain needs no
// clamp: what is below -kBig there has a term below 2^-700.
constexpr float kBig = 1e6f;
constexpr float kPlain = 5e5f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float big_clamp(float z) { return fminf(fmaxf(z, -kBig), kBig); }

// Whole-number reference for terms up to the maximum m > -infinity.
__device__ __forceinline__ float reference_of(float m, float c) { return ceilf(big_clamp(m) * c); }

// 2^(c z - n) for any z: NaN and -infinity have no mass.
__device__ __forceinline__ float term_guarded(float z, float c, float n) {
  return z > -INFINITY ? ex2(fmaf(big_clamp(z), c, -n)) : 0.f;
}

// Whether a row or part of a row with maximum m needs term_guarded throughout.
__device__ __forceinline__ bool is_extreme(float m) { return !(fabsf(m) <= kPlain); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A vector of barred tokens.
template <typename T> __device__ __forceinline__ uint4 barred_vec();
template <> __device__ __forceinline__ uint4 barred_vec<float>() {
  return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
}
template <> __device__ __forceinline__ uint4 barred_vec<bf16>() {
  return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
}

// The largest value of a vector (NaN aside); bf16 pairs go through one packed maximum.
__device__ __forceinline__ float vec_max(const uint4& q, float) {
  return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
}
__device__ __forceinline__ float vec_max(const uint4& q, bf16) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
  const float2 f = __bfloat1622float2(__hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3])));
  return fmaxf(f.x, f.y);
}

struct ExpSum {
  float n = -INFINITY, s = 0.f;
};

// Raises the reference of `a` to n (n >= a.n, n finite).
__device__ __forceinline__ void raise(ExpSum& a, float n) {
  a.s *= ex2(a.n - n);  // a.n = -infinity: 0
  a.n = n;
}

// Whether any value of the vectors is NaN, where none is above -infinity: -infinities alone add up to one.
template <typename T, int NV>
__device__ __forceinline__ bool barred_by_nan(const uint4 (&q)[NV]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float z[Vec<T>::N];
    widen(q[i], z);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) s += z[e];
  }
  return isnan(s);
}

// Adds the first `some` of the vectors, of maximum m (NaN aside), to a thread's sum; true where their terms need a
// guard: a magnitude beyond kPlain or a NaN, of which the maximum of a tile without another value says nothing.  The
// reference is raised only when a term would exceed 2^kSlack of it, so that it hardly ever is after the first vectors.
constexpr float kSlack = 40.f;
template <typename T, int NV>
__device__ __forceinline__ bool add_vectors(ExpSum& a, const uint4 (&q)[NV], int some, float m, float c) {
  if (!(m > -INFINITY)) return barred_by_nan<T>(q);
  if (fmaf(big_clamp(m), c, -a.n) > kSlack) raise(a, reference_of(m, c));
  float2 s = make_float2(0.f, 0.f);
  const float2 c2 = make_float2(c, c), n2 = make_float2(-a.n, -a.n);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (i >= some) break;
    float z[Vec<T>::N];
    widen(q[i], z);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; e += 2) {
      const float2 x = fma2(make_float2(z[e], z[e + 1]), c2, n2);
      s = add2(s, make_float2(ex2(x.x), ex2(x.y)));
    }
  }
  float t = s.x + s.y;
  const bool guard = is_extreme(m) || isnan(t);
  if (guard) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float z[Vec<T>::N];
      widen(q[i], z);
#pragma unroll
      for (int e = 0; e < Vec<T>::N; ++e) t += term_guarded(z[e], c, a.n);
    }
  }
  a.s += t;
  return guard;
}

// A thread's vectors of one tile: `at` is the thread's first, the others lie `threads` apart, and `left` vectors
// remain of the slice from the tile's first on (tid of them before the thread's).  Past the end: barred tokens.
template <typename T, int NV, bool KEEP>
__device__ __forceinline__ void load_tile(uint4 (&q)[NV], const uint4* at, int threads, int left) {
  auto get = [](const uint4* p) { return KEEP ? __ldcg(p) : __ldcs(p); };
  if (left >= NV * threads) {
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = get(at + i * threads);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = i * threads + (int)threadIdx.x < left ? get(at + i * threads) : barred_vec<T>();
  }
}

// The elements of q in the mask as barred tokens.
template <typename T>
__device__ __forceinline__ void bar_elements(uint4& q, uint32_t mask) {
  T* e = reinterpret_cast<T*>(&q);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i)
    if ((mask >> i) & 1u) e[i] = static_cast<T>(-INFINITY);
}
// The elements, as a mask, that lie from column V on of a vector at column v.
template <typename T>
__device__ __forceinline__ uint32_t beyond(int v, int V) {
  return v + Vec<T>::N <= V ? 0u : v >= V ? 0xffu : 0xffu << (V - v);
}

// Order-preserving map of a logit onto 32 bits: larger is larger, -0 equals +0; NaN and -infinity, which
// are never selected, are 0.
__device__ __forceinline__ uint32_t order_of(float z) {
  if (!(z > -INFINITY)) return 0u;
  uint32_t u = __float_as_uint(z);
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
// Selection key: a larger logit first, then the lower column.  Key 0 is none.
__device__ __forceinline__ uint64_t select_key(uint32_t order, int v) {
  return order ? (static_cast<uint64_t>(order) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(v)) : 0ull;
}

// log of sum * 2^n (natural), with the correction for c's rounding; m: the row's maximum.
constexpr double kLn2 = 0.693147180559945309417232;
constexpr double kLog2e = 1.44269504088896340735992;
__device__ __forceinline__ double log_sum_exp(double sum, double n, float m, float c, double inv_t) {
  if (!(sum > 0.0)) return -INFINITY;
  const double delta = kLog2e * inv_t - (double)c;
  return kLn2 * (log2(sum) + n + delta * (double)big_clamp(m));
}

}  // namespace domino
