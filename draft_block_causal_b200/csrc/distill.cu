// distill.cu -- distillation of rows of logits from a teacher's top logits: loss, and gradient.
//
// With x = z / T, L = log sum exp(x) over the row and L_rest the same over the tokens that are no entry, a
// row's loss is   w * (sum_k p_k (log p_k - x_k + L) + rho (log rho - L_rest + L))
// and its gradient   w / T * (P exp(x_v - L) - p_v)  at an entry's token,
//                    w / T * (P exp(L_rest - L) - rho) * exp(x_v - L_rest)  elsewhere.
// The row is summed without the entries' columns, about its own reference, and the at most 128 entries' terms
// are added in 64 bits: S_rest as S less the entries' terms would be lost for a student that puts all but 1e-7 of
// its mass on them.  log p_k is y_k less the entries' log-sum, so the entries need one exponential each.
//
// Loss and gradient in one call read a row once: a cluster of blocks holds it in registers (k_distill_row),
// the blocks exchange their sums through distributed shared memory, and each writes its slice's gradient.
// The entries take one warp of a block; block 0's also forms what the others need of them.  Rows that no
// cluster holds, the loss alone and the backward call go by k_distill_sum (a row's sums by a cluster, read
// once) and k_distill_grad (elementwise from the stats).
#include "cluster.cuh"
#include "launch.cuh"
#include "vocab_rows.cuh"
#include "vocab_rows.h"

namespace domino {

namespace {

constexpr int kMaxK = DOMINO_MAX_TOP;
constexpr int kMaxCluster = 16;

struct DistillArgs {
  domino_distill_t d;
  float c;        // log2(e) / T
  double inv_t;
  float* loss;
  float4* stats;  // two per row, see Stats
  const float* grad_loss;
  void* grad;
  int64_t grad_ld;
  int cluster;    // blocks per row (k_distill_grad: chunks)
  int32_t* status;
};

// What the gradient needs of a row.  An entry's token: all * exp(x - L) - scale * p, L = l_hi + l_lo and
// p = exp(y - lp), lp = lp_hi + lp_lo; others: rest * 2^(c z - n).  all = scale * P, scale = w / T; scale 0: no
// gradient.
struct Stats {
  float n, rest, l_hi, l_lo;
  float all, scale, lp_hi, lp_lo;
};
__device__ __forceinline__ void store_stats(float4* st, int r, const Stats& s) {
  if (!st) return;
  st[2 * (size_t)r] = make_float4(s.n, s.rest, s.l_hi, s.l_lo);
  st[2 * (size_t)r + 1] = make_float4(s.all, s.scale, s.lp_hi, s.lp_lo);
}
__device__ __forceinline__ Stats load_stats(const float4* st, int r) {
  const float4 a = st[2 * (size_t)r], b = st[2 * (size_t)r + 1];
  return Stats{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Block 0's findings on a row's entries, for every block of the cluster.
struct Top {
  double sum, psum, lp;  // sum * 2^ref: the distinct entries' terms of S; sum of p; log-sum of the entries' y
  double lead;           // sum of p (log p - x)
  float ref;
  int live, twice;       // whether the row counts; whether a token is given twice
};
// A block's sum over its columns that are no entry's.
struct Part {
  double s;
  float n, m;
};

// A row's entries, in the hands of one warp: lane l has entries l, l + 32, ...
struct Entries {
  int32_t id[kMaxK];  // -1: none
  double y[kMaxK];    // the teacher's logit over T, -infinity for one without mass
  double x[kMaxK];    // the student's, where it was asked for
  double p[kMaxK];
};

struct DistillShared {
  Part parts[kMaxCluster];
  Top top;
  double red_s[32];
  float red_n[32], red_m[32];
  Entries en;
};

__device__ __forceinline__ double warp_add(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Reads a row's entries; x for those with columns in [v0, v1).  One warp; ends with its barrier.
template <typename T>
__device__ __forceinline__ void load_entries(const DistillArgs& a, int r, const T* row, int v0, int v1, Entries& en,
                                             bool report) {
  const domino_distill_t& d = a.d;
  for (int k = threadIdx.x & 31; k < d.K; k += 32) {
    int id = __ldg(d.top_ids + (size_t)r * d.K + k);
    const float t = __ldg(d.top_logits + (size_t)r * d.K + k);
    if (id < 0 || id >= d.V) {
      if (id != -1 && report && a.status) set_status(a.status, DOMINO_STATUS_BAD_TOKEN);
      id = -1;
    }
    en.id[k] = id;
    en.y[k] = id >= 0 && t > -INFINITY ? (double)big_clamp(t) * a.inv_t : -INFINITY;
    double x = -INFINITY;
    if (id >= v0 && id < v1) {
      const float z = to_f32(row[id]);
      if (z > -INFINITY) x = (double)big_clamp(z) * a.inv_t;
    }
    en.x[k] = x;
  }
  __syncwarp();
}

// What block 0's entries' warp finds: sh.top.
__device__ __forceinline__ void find_top(const DistillArgs& a, int r, DistillShared& sh) {
  const domino_distill_t& d = a.d;
  const Entries& en = sh.en;
  const int lane = threadIdx.x & 31;
  Top t{};
  double m = -INFINITY, top = -INFINITY;
  for (int k = lane; k < d.K; k += 32) {
    m = fmax(m, en.y[k]);
    top = fmax(top, en.x[k]);
  }
  if (d.teacher_lse) {
    const float lse = d.teacher_lse[r];
    t.lp = lse;
    t.live = fabsf(lse) < INFINITY;
  } else {
    m = warp_max(m);
    double s = 0.0;
    for (int k = lane; k < d.K; k += 32)
      if (en.y[k] > -INFINITY) s += exp(en.y[k] - m);
    t.lp = m + log(warp_add(s));
    t.live = m > -INFINITY;
  }
  top = warp_max(top);
  const double ref = top > -INFINITY ? ceil(top * kLog2e) : 0.0;
  t.ref = (float)ref;
  bool twice = false;
  if (t.live) {
    for (int k = lane; k < d.K; k += 32) {
      const int id = en.id[k];
      if (id < 0) continue;
      bool first = true;
      for (int j = 0; j < k && first; ++j) first = en.id[j] != id;
      twice |= !first;
      if (first && en.x[k] > -INFINITY) t.sum += exp2(en.x[k] * kLog2e - ref);
      if (en.y[k] > -INFINITY) {
        const double p = exp(en.y[k] - t.lp);
        t.psum += p;
        if (p > 0.0) t.lead += p * (en.y[k] - t.lp - en.x[k]);
      }
    }
  }
  t.sum = warp_add(t.sum);
  t.psum = warp_add(t.psum);
  t.lead = warp_add(t.lead);
  t.twice = __any_sync(0xffffffffu, twice);
  if (!(t.psum > 0.0) && !isnan(t.psum)) t.live = 0;
  if (lane == 0) sh.top = t;
}

// 2^(difference of references): no power of two that a term could see is left out.
__device__ __forceinline__ double pow2(double e) { return e < -1000.0 ? 0.0 : e > 1000.0 ? INFINITY : ldexp(1.0, (int)e); }

// True S over the sum taken with c rounded to fp32: 2^(delta m).
__device__ __forceinline__ double rounding_of_c(float m, float c, double inv_t) {
  const double d = kLn2 * (kLog2e * inv_t - (double)c) * (double)big_clamp(m);
  return fabs(d) < 1e-5 ? 1.0 + d : exp(d);
}

// Loss and stats of a row: one thread of block 0.
__device__ __forceinline__ void finish_row(const DistillArgs& a, int r, float w, const Top& t, const Part& p) {
  const bool rest = p.s > 0.0;
  const double l_rest = log_sum_exp(p.s, p.n, p.m, a.c, a.inv_t);
  const double l_top = t.sum > 0.0 ? kLn2 * (log2(t.sum) + (double)t.ref) : -INFINITY;
  const double hi = fmax(l_rest, l_top), lo = fmin(l_rest, l_top);
  if (!t.live || !(hi > -INFINITY)) {
    a.loss[r] = 0.f;
    store_stats(a.stats, r, Stats{});
    return;
  }
  const double L = hi + log1p(exp(lo - hi));
  const double rho = a.d.teacher_lse && rest ? fmax(0.0, 1.0 - t.psum) : 0.0;
  const double loss = t.lead + t.psum * L + (rho > 0.0 ? rho * (log(rho) - l_rest + L) : 0.0);
  a.loss[r] = (float)((double)w * loss);
  if (a.stats) {
    const double scale = (double)w * a.inv_t, P = t.psum + rho;
    Stats st;
    st.n = p.n;
    st.rest = rest ? (float)(scale * (P * exp(l_rest - L) - rho) / p.s) : 0.f;
    st.l_hi = (float)L;
    st.l_lo = (float)(L - (double)st.l_hi);
    st.all = (float)(scale * P);
    st.scale = (float)scale;
    st.lp_hi = (float)t.lp;
    st.lp_lo = (float)(t.lp - (double)st.lp_hi);
    store_stats(a.stats, r, st);
  }
}

// The warps' sums (lane 0 of each holds its warp's) as the block's, in warp order; `warps` records.
__device__ __forceinline__ void give_warp(DistillShared& sh, const ExpSum& acc, float m) {
  float n = acc.n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  const double s = warp_add(n > -INFINITY ? (double)(acc.s * ex2(acc.n - n)) : 0.0);
  if ((threadIdx.x & 31) == 0) {
    sh.red_n[threadIdx.x >> 5] = n;
    sh.red_m[threadIdx.x >> 5] = m;
    sh.red_s[threadIdx.x >> 5] = s;
  }
}
__device__ __forceinline__ Part block_part(const DistillShared& sh, int warps) {
  Part p{0.0, -INFINITY, -INFINITY};
  for (int w = 0; w < warps; ++w) {
    p.n = fmaxf(p.n, sh.red_n[w]);
    p.m = fmaxf(p.m, sh.red_m[w]);
  }
  for (int w = 0; w < warps; ++w)
    if (sh.red_n[w] > -INFINITY) p.s += sh.red_s[w] * (double)ex2(sh.red_n[w] - p.n);
  return p;
}
// The blocks' parts as the row's.
__device__ __forceinline__ Part row_part(const DistillShared& sh, int cluster) {
  Part p{0.0, -INFINITY, -INFINITY};
  for (int c = 0; c < cluster; ++c) {
    p.n = fmaxf(p.n, sh.parts[c].n);
    p.m = fmaxf(p.m, sh.parts[c].m);
  }
  for (int c = 0; c < cluster; ++c)
    if (sh.parts[c].n > -INFINITY) p.s += sh.parts[c].s * (double)ex2(sh.parts[c].n - p.n);
  return p;
}
__device__ __forceinline__ void send_part(DistillShared& sh, uint32_t rank, uint32_t to, const Part& p) {
  const uint32_t at = cluster_address(&sh.parts[rank], to);
  cluster_store(at, p.s);
  cluster_store(at + 8, p.n, p.m);
}
// Block 0's top to another block.
__device__ __forceinline__ void send_top(DistillShared& sh, uint32_t to) {
  const uint32_t at = cluster_address(&sh.top, to);
  const Top& t = sh.top;
  cluster_store(at, t.sum);
  cluster_store(at + 8, t.psum);
  cluster_store(at + 16, t.lp);
  cluster_store(at + 24, t.lead);
  cluster_store(at + 32, __float_as_int(t.ref));
  cluster_store(at + 36, t.live);
  cluster_store(at + 40, t.twice);
}

// The columns that the entries' warp has set a bit for, of the vector `vec` of a slice, as a mask of its elements.
__device__ __forceinline__ uint32_t marked(const uint32_t* marks, int vec) {
  return (marks[vec >> 2] >> ((vec & 3) * 8)) & 0xffu;
}
// Clears the marks of `vecs` vectors and sets those of the entries in them; the entries' warp alone.
template <int N>
__device__ __forceinline__ void set_marks(uint32_t* marks, int first, int vecs, const Entries& en, int K) {
  for (int i = threadIdx.x & 31; i < (vecs + 3) / 4; i += 32) marks[i] = 0;
  __syncwarp();
  for (int k = threadIdx.x & 31; k < K; k += 32) {
    const int id = en.id[k], vec = id / N - first;
    if (id >= 0 && vec >= 0 && vec < vecs) atomicOr(&marks[vec >> 2], 1u << ((vec & 3) * 8 + id % N));
  }
}

// q's elements of the mask, or from column V on, as barred ones.
template <typename T>
__device__ __forceinline__ void bar(uint4& q, uint32_t mask) {
  T* e = reinterpret_cast<T*>(&q);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i)
    if ((mask >> i) & 1u) e[i] = static_cast<T>(-INFINITY);
}
template <typename T>
__device__ __forceinline__ uint32_t beyond(int v, int V) {  // mask of the vector at column v
  return v + Vec<T>::N <= V ? 0u : v >= V ? 0xffu : 0xffu << (V - v);
}
// Adds the first `vecs` of a thread's NV vectors, of maximum m > -infinity, to its sum; true where a value is NaN or
// the terms need a guard.
template <typename T, int NV>
__device__ __forceinline__ bool add_vectors(ExpSum& a, const uint4 (&q)[NV], int vecs, float m, float c) {
  const float n = fmaxf(a.n, reference_of(m, c));
  if (n > a.n) raise(a, n);
  float2 s = make_float2(0.f, 0.f);
  if (!is_extreme(m)) {
    const float2 c2 = make_float2(c, c), n2 = make_float2(-n, -n);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i >= vecs) break;
      float z[Vec<T>::N];
      widen(q[i], z);
#pragma unroll
      for (int e = 0; e < Vec<T>::N; e += 2) {
        const float2 x = fma2(make_float2(z[e], z[e + 1]), c2, n2);
        s = add2(s, make_float2(ex2(x.x), ex2(x.y)));
      }
    }
  }
  float t = s.x + s.y;
  const bool guard = is_extreme(m) || isnan(t);
  if (guard) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i >= vecs) break;
      float z[Vec<T>::N];
      widen(q[i], z);
#pragma unroll
      for (int e = 0; e < Vec<T>::N; ++e) t += term_guarded(z[e], c, n);
    }
  }
  a.s += t;
  return guard;
}

__device__ __forceinline__ void store_grad(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_grad(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// Writes one vector's gradient, coef * 2^(c z - n), without the columns from V on.
template <typename T, typename G>
__device__ __forceinline__ void write_vector(G* out, int v, int V, const uint4& q, float c, float n, float coef, bool guard) {
  constexpr int N = Vec<T>::N;
  float z[N];
  widen(q, z);
  if (!guard) {
    const float2 c2 = make_float2(c, c), n2 = make_float2(-n, -n), k2 = make_float2(coef, coef);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 x = fma2(make_float2(z[e], z[e + 1]), c2, n2);
      const float2 y = mul2(make_float2(ex2(x.x), ex2(x.y)), k2);
      z[e] = y.x;
      z[e + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = coef == 0.f ? 0.f : coef * term_guarded(z[e], c, n);
  }
  if (v + N <= V) {
    if constexpr (sizeof(G) == 4) {
#pragma unroll
      for (int e = 0; e < N; e += 4)
        __stcs(reinterpret_cast<float4*>(out + v + e), make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]));
    } else {
      __nv_bfloat162 h[N / 2];
#pragma unroll
      for (int e = 0; e < N; e += 2) h[e / 2] = __floats2bfloat162_rn(z[e], z[e + 1]);
      if constexpr (N == 8) __stcs(reinterpret_cast<uint4*>(out + v), *reinterpret_cast<uint4*>(h));
      else __stcs(reinterpret_cast<uint2*>(out + v), *reinterpret_cast<uint2*>(h));
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (v + e < V) store_grad(out + v + e, z[e]);
  }
}

// The entries' warp: f(entry, column, p) for the entries with columns in [v0, v1), once a token with the sum of its
// entries' p.
template <typename F>
__device__ __forceinline__ void each_own(int K, Entries& en, int v0, int v1, double lp, bool twice, F f) {
  const int lane = threadIdx.x & 31;
  if (twice) {
    for (int k = lane; k < K; k += 32) en.p[k] = en.y[k] > -INFINITY ? exp(en.y[k] - lp) : 0.0;
    __syncwarp();
  }
  for (int k = lane; k < K; k += 32) {
    const int id = en.id[k];
    if (id < v0 || id >= v1) continue;  // -1 too
    double p = 0.0;
    bool first = true;
    if (twice) {
      for (int j = 0; j < K; ++j)
        if (en.id[j] == id) {
          p += en.p[j];
          first &= j >= k;
        }
    } else if (en.y[k] > -INFINITY) {
      p = exp(en.y[k] - lp);
    }
    if (first) f(k, id, p);
  }
}

// Loss and gradient of one row a cluster, held in registers: kNV vectors of each of THREADS - 32 threads; the last
// warp has the entries.
//
// Bound by memory: V values read and V written a row.  One exponential for the sum and one for the gradient
// (16 a clock and SM) take half of the memory's time for bf16 in and out.
template <typename T, typename G, int THREADS, int NV>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_distill_row(DistillArgs a) {
  constexpr int N = Vec<T>::N, DATA = THREADS - 32, WARPS = DATA / 32;
  __shared__ DistillShared sh;
  __shared__ uint32_t marks[(DATA * NV + 3) / 4];
  pdl_wait();
  pdl_trigger();
  const domino_distill_t& d = a.d;
  const int cluster = a.cluster, r = blockIdx.x / cluster, tid = threadIdx.x;
  const uint32_t rank = blockIdx.x % cluster;
  const bool entries = tid >= DATA;
  const int all = (d.V + N - 1) / N, per = (all + cluster - 1) / cluster;
  const int first = min((int)rank * per, all), last = min(first + per, all);
  const int vecs = (last - first + DATA - 1) / DATA;  // <= NV
  G* out = static_cast<G*>(a.grad) + (size_t)r * a.grad_ld;
  const float w = d.row_weights ? d.row_weights[r] : 1.f;
  const T* row = static_cast<const T*>(d.logits) + (size_t)r * d.ld;
  uint4 q[NV];
  if (w == 0.f) {  // the whole cluster
    if (!entries) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int vec = first + i * DATA + tid;
        if (vec < last) write_vector<T>(out, vec * N, d.V, barred_vec<T>(), a.c, 0.f, 0.f, true);
      }
    } else if (rank == 0 && tid == DATA) {
      a.loss[r] = 0.f;
      store_stats(a.stats, r, Stats{});
    }
    return;
  }
  cluster_arrive();  // all blocks have started before one stores into another
  if (!entries) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vec = first + i * DATA + tid;
      q[i] = vec < last ? __ldcs(reinterpret_cast<const uint4*>(row) + vec) : barred_vec<T>();
    }
  } else {
    load_entries(a, r, row, rank == 0 ? 0 : first * N, rank == 0 ? d.V : last * N, sh.en, rank == 0);
    set_marks<N>(marks, first, last - first, sh.en, d.K);
  }
  __syncthreads();  // marks are set
  bool guard = false;
  if (!entries) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i >= vecs) break;
      const int vec = i * DATA + tid;
      if (first + vec < last) {
        const uint32_t mask = marked(marks, vec) | beyond<T>((first + vec) * N, d.V);
        if (mask) bar<T>(q[i], mask);
      }
      m = fmaxf(m, vec_max(q[i], T()));
    }
    ExpSum acc;
    if (m > -INFINITY) guard = add_vectors<T, NV>(acc, q, vecs, m, a.c);
    give_warp(sh, acc, m);
  } else if (rank == 0) {
    find_top(a, r, sh);
  }
  __syncthreads();
  cluster_wait();
  if (tid < cluster) send_part(sh, rank, tid, block_part(sh, WARPS));
  if (rank == 0 && tid > DATA && tid - DATA < cluster) send_top(sh, tid - DATA);
  cluster_arrive();
  cluster_wait();
  const Part part = row_part(sh, cluster);
  const Top& t = sh.top;
  const double scale = (double)w * a.inv_t;
  const double rest = part.s * rounding_of_c(part.m, a.c, a.inv_t);
  const double rho = d.teacher_lse && rest > 0.0 ? fmax(0.0, 1.0 - t.psum) : 0.0, P = t.psum + rho;
  const double gap = part.s > 0.0 ? (double)part.n - (double)t.ref : -2000.0;
  const bool live = t.live && (part.s > 0.0 || t.sum > 0.0);
  if (!entries) {
    // rest / (rest + top): what of S lies outside the entries
    const double outside = rest / (rest + t.sum * pow2(-gap));
    const float coef = live && part.s > 0.0 ? (float)(scale * (P * outside - rho) / part.s) : 0.f;
    guard |= coef == 0.f || is_extreme(part.m);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i >= vecs) break;
      const int vec = first + i * DATA + tid;
      if (vec < last) write_vector<T>(out, vec * N, d.V, q[i], a.c, part.n, coef, guard);
    }
  }
  __syncthreads();  // the entries' columns go over the others'
  if (entries) {
    if (live) {
      const double s = t.sum + (part.s > 0.0 ? rest * pow2(gap) : 0.0);
      each_own(d.K, sh.en, first * N, last * N, t.lp, t.twice, [&](int k, int v, double p) {
        const double q_v = sh.en.x[k] > -INFINITY ? exp2(sh.en.x[k] * kLog2e - (double)t.ref) / s : 0.0;
        store_grad(out + v, (float)(scale * (P * q_v - p)));
      });
    }
    if (rank == 0 && tid == DATA) finish_row(a, r, w, t, part);
  }
}

// A row's sums by a cluster that reads it once, for the loss and the stats.  The marks take a byte a vector of the
// slice.
constexpr int kSumThreads = 256;
constexpr int kSumVecs = 4;
constexpr int kSumSlice = 24576;  // vectors of a slice at most

template <typename T>
__global__ void __launch_bounds__(kSumThreads, 4) k_distill_sum(DistillArgs a) {
  constexpr int N = Vec<T>::N, DATA = kSumThreads - 32, WARPS = DATA / 32;
  __shared__ DistillShared sh;
  extern __shared__ uint32_t marks[];
  pdl_wait();
  pdl_trigger();
  const domino_distill_t& d = a.d;
  const int cluster = a.cluster, r = blockIdx.x / cluster, tid = threadIdx.x;
  const uint32_t rank = blockIdx.x % cluster;
  const bool entries = tid >= DATA;
  const int all = (d.V + N - 1) / N, per = (all + cluster - 1) / cluster;
  const int first = min((int)rank * per, all), last = min(first + per, all);
  const float w = d.row_weights ? d.row_weights[r] : 1.f;
  const T* row = static_cast<const T*>(d.logits) + (size_t)r * d.ld;
  if (w == 0.f) {  // the whole cluster
    if (rank == 0 && tid == 0) {
      a.loss[r] = 0.f;
      store_stats(a.stats, r, Stats{});
    }
    return;
  }
  cluster_arrive();
  constexpr int kTile = DATA * kSumVecs;
  auto load = [&](uint4(&q)[kSumVecs], int t0) {
#pragma unroll
    for (int i = 0; i < kSumVecs; ++i) {
      const int vec = t0 + i * DATA + tid;
      q[i] = vec < last ? __ldcs(reinterpret_cast<const uint4*>(row) + vec) : barred_vec<T>();
    }
  };
  uint4 next[kSumVecs];
  if (!entries) {
    load(next, first);
  } else {
    load_entries(a, r, row, 0, rank == 0 ? d.V : 0, sh.en, rank == 0);
    set_marks<N>(marks, first, last - first, sh.en, d.K);
  }
  __syncthreads();
  if (!entries) {
    ExpSum acc;
    float m = -INFINITY;
    for (int t0 = first; t0 < last; t0 += kTile) {
      uint4 q[kSumVecs];
#pragma unroll
      for (int i = 0; i < kSumVecs; ++i) q[i] = next[i];
      load(next, t0 + kTile);
      float tm = -INFINITY;
#pragma unroll
      for (int i = 0; i < kSumVecs; ++i) {
        const int vec = t0 + i * DATA + tid;
        if (vec < last) {
          const uint32_t mask = marked(marks, vec - first) | beyond<T>(vec * N, d.V);
          if (mask) bar<T>(q[i], mask);
        }
        tm = fmaxf(tm, vec_max(q[i], T()));
      }
      if (tm > -INFINITY) {
        m = fmaxf(m, tm);
        add_vectors<T, kSumVecs>(acc, q, kSumVecs, tm, a.c);
      }
    }
    give_warp(sh, acc, m);
  } else if (rank == 0) {
    find_top(a, r, sh);
  }
  __syncthreads();
  cluster_wait();
  if (tid == 0) send_part(sh, rank, 0, block_part(sh, WARPS));
  cluster_arrive();
  cluster_wait();
  if (rank == 0 && tid == DATA) finish_row(a, r, w, sh.top, row_part(sh, cluster));
}

// The gradient from a row's stats, a chunk of kGradVecs vectors a thread by each block.  The logits may be
// overwritten: a chunk's entries read theirs first.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 8;

template <typename T, typename G>
__global__ void __launch_bounds__(kGradThreads, 4) k_distill_grad(DistillArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Entries en;
  __shared__ float own[kMaxK];  // an entry's gradient, where it is this chunk's to write
  __shared__ int at[kMaxK];     // ... and its column, else -1
  pdl_wait();
  pdl_trigger();
  const domino_distill_t& d = a.d;
  const int r = blockIdx.x / a.cluster, chunk = blockIdx.x % a.cluster, tid = threadIdx.x;
  const int all = (d.V + N - 1) / N, first = chunk * kGradThreads * kGradVecs;
  const T* row = static_cast<const T*>(d.logits) + (size_t)r * d.ld;
  G* out = static_cast<G*>(a.grad) + (size_t)r * a.grad_ld;
  const Stats st = load_stats(a.stats, r);
  const float g = a.grad_loss ? a.grad_loss[r] : 1.f;
  const bool live = st.scale != 0.f && g != 0.f;
  uint4 q[kGradVecs];
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i) {
    const int vec = first + i * kGradThreads + tid;
    q[i] = live && vec < all ? __ldcs(reinterpret_cast<const uint4*>(row) + vec) : barred_vec<T>();
  }
  if (tid < 32 && live) {
    const int v0 = first * N, v1 = min(first + kGradThreads * kGradVecs, all) * N;
    load_entries(a, r, row, v0, v1, en, false);
    for (int k = tid; k < d.K; k += 32) at[k] = -1;
    const double lp = (double)st.lp_hi + (double)st.lp_lo, L = (double)st.l_hi + (double)st.l_lo;
    each_own(d.K, en, v0, v1, lp, true, [&](int k, int v, double p) {
      const double q_v = en.x[k] > -INFINITY ? exp(en.x[k] - L) : 0.0;
      own[k] = (float)((double)g * (q_v * (double)st.all - p * (double)st.scale));
      at[k] = v;
    });
  }
  __syncthreads();  // the entries' logits are read
  const float coef = live ? g * st.rest : 0.f;
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i) {
    const int vec = first + i * kGradThreads + tid;
    // the general form for NaN: this kernel has not summed the values
    if (vec < all) write_vector<T>(out, vec * N, d.V, q[i], a.c, st.n, coef, true);
  }
  __syncthreads();
  if (live && tid < d.K && at[tid] >= 0) store_grad(out + at[tid], own[tid]);
}

int vectors_of(const domino_distill_t& d) { return d.dtype == DOMINO_DTYPE_F32 ? (d.V + 3) / 4 : (d.V + 7) / 8; }

cudaError_t launch_sum(DistillArgs a, cudaStream_t st) {
  const int vecs = vectors_of(a.d);
  int cluster = 1;
  while (cluster < kMaxCluster && (vecs > cluster * kSumSlice || ((int64_t)a.d.rows * cluster < 4 * 148 &&
                                                                  vecs / (2 * cluster) >= 2 * kSumThreads)))
    cluster *= 2;
  a.cluster = cluster;
  const size_t smem = ((vecs + cluster - 1) / cluster + 3) / 4 * 4;
  auto kern = a.d.dtype == DOMINO_DTYPE_F32 ? k_distill_sum<float> : k_distill_sum<bf16>;
  return note_launch(launch_cluster(kern, cluster, dim3((unsigned)a.d.rows * (unsigned)cluster), dim3(kSumThreads), smem,
                                    st, a));
}

cudaError_t launch_grad(DistillArgs a, int grad_dtype, cudaStream_t st) {
  a.cluster = (vectors_of(a.d) + kGradThreads * kGradVecs - 1) / (kGradThreads * kGradVecs);
  const bool f = a.d.dtype == DOMINO_DTYPE_F32, g = grad_dtype == DOMINO_DTYPE_F32;
  auto kern = f ? (g ? k_distill_grad<float, float> : k_distill_grad<float, bf16>)
                : (g ? k_distill_grad<bf16, float> : k_distill_grad<bf16, bf16>);
  return note_launch(launch_pdl(kern, dim3((unsigned)a.d.rows * (unsigned)a.cluster), dim3(kGradThreads), 0, st, a));
}

template <typename T, typename G>
constexpr int row_threads() { return sizeof(T) == 4 ? 512 : 256; }
template <typename T, typename G>
constexpr int row_vecs() { return sizeof(T) == 4 ? 10 : 11; }

// Whether a cluster holds a row; the smallest cluster that does.
template <typename T, typename G>
cudaError_t launch_row_as(DistillArgs a, cudaStream_t st, bool* held) {
  constexpr int threads = row_threads<T, G>(), block = (threads - 32) * row_vecs<T, G>();
  const int vecs = vectors_of(a.d);
  int cluster = 1;
  while (cluster < kMaxCluster && vecs > cluster * block) cluster *= 2;
  *held = vecs <= cluster * block;
  if (!*held) return cudaSuccess;
  a.cluster = cluster;
  return note_launch(launch_cluster(k_distill_row<T, G, threads, row_vecs<T, G>()>, cluster,
                                    dim3((unsigned)a.d.rows * (unsigned)cluster), dim3(threads), 0, st, a));
}
cudaError_t launch_row(const DistillArgs& a, int grad_dtype, cudaStream_t st, bool* held) {
  const bool f = a.d.dtype == DOMINO_DTYPE_F32, g = grad_dtype == DOMINO_DTYPE_F32;
  return f ? (g ? launch_row_as<float, float>(a, st, held) : launch_row_as<float, bf16>(a, st, held))
           : (g ? launch_row_as<bf16, float>(a, st, held) : launch_row_as<bf16, bf16>(a, st, held));
}

int check_distill(const domino_distill_t* d) {
  if (!d || !rows_ok(d->rows, d->V, d->ld, d->dtype, d->logits)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (d->K < 1 || d->K > DOMINO_MAX_TOP || !temperature_ok(d->temperature)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (!d->top_ids || !d->top_logits) return DOMINO_ERR_INVALID_ARGUMENT;
  if (d->rows > DOMINO_MAX_ROWS) return DOMINO_ERR_UNSUPPORTED;
  return DOMINO_OK;
}

// Checks one output of n bytes against the inputs; `with_logits` false: the logits are checked elsewhere.
bool clear_of_inputs(const domino_distill_t& d, const void* p, size_t n, bool with_logits) {
  const size_t rows = (size_t)d.rows, e = rows * d.K * 4;
  return !(with_logits && overlap(p, n, d.logits, rows_span(d.rows, d.V, d.ld, d.dtype))) &&
         !overlap(p, n, d.top_ids, e) && !overlap(p, n, d.top_logits, e) && !overlap(p, n, d.teacher_lse, rows * 4) &&
         !overlap(p, n, d.row_weights, rows * 4);
}

int check_grad(const domino_distill_t& d, const void* grad, int64_t grad_ld, int grad_dtype) {
  if (!rows_ok(d.rows, d.V, grad_ld, grad_dtype, grad)) return DOMINO_ERR_INVALID_ARGUMENT;
  const bool in_place = grad == d.logits && grad_ld == d.ld && grad_dtype == d.dtype;
  return clear_of_inputs(d, grad, rows_span(d.rows, d.V, grad_ld, grad_dtype), !in_place) ? DOMINO_OK
                                                                                          : DOMINO_ERR_INVALID_ARGUMENT;
}

DistillArgs make_args(const domino_distill_t& d, int32_t* status) {
  DistillArgs a{};
  a.d = d;
  a.inv_t = 1.0 / (double)d.temperature;
  a.c = (float)(1.4426950408889634 * a.inv_t);
  a.status = status;
  return a;
}

}  // namespace

}  // namespace domino

using namespace domino;

extern "C" int domino_distill(const domino_distill_t* args, float* loss, float* stats, void* grad, int64_t grad_ld,
                              int32_t grad_dtype, int32_t* status_dev, domino_stream_t stream) {
  int rc = check_distill(args);
  if (rc != DOMINO_OK) return rc;
  if (!loss || (stats && (reinterpret_cast<uintptr_t>(stats) & 15u))) return DOMINO_ERR_INVALID_ARGUMENT;
  const size_t rows = (size_t)args->rows;
  if (!clear_of_inputs(*args, loss, rows * 4, true) || !clear_of_inputs(*args, stats, rows * 32, true) ||
      overlap(loss, rows * 4, stats, rows * 32))
    return DOMINO_ERR_INVALID_ARGUMENT;
  if (grad) {
    if ((rc = check_grad(*args, grad, grad_ld, grad_dtype)) != DOMINO_OK) return rc;
    const size_t n = rows_span(args->rows, args->V, grad_ld, grad_dtype);
    if (overlap(grad, n, loss, rows * 4) || overlap(grad, n, stats, rows * 32)) return DOMINO_ERR_INVALID_ARGUMENT;
    if (!stats) return DOMINO_ERR_INVALID_ARGUMENT;
  }
  DistillArgs a = make_args(*args, status_dev);
  a.loss = loss;
  a.stats = reinterpret_cast<float4*>(stats);
  a.grad = grad;
  a.grad_ld = grad_ld;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  bool held = false;
  cudaError_t e = cudaSuccess;
  if (grad) e = launch_row(a, grad_dtype, cs, &held);
  if (e == cudaSuccess && !held) {
    e = launch_sum(a, cs);
    if (e == cudaSuccess && grad) e = launch_grad(a, grad_dtype, cs);
  }
  return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}

extern "C" int domino_distill_backward(const domino_distill_t* args, const float* stats, const float* grad_loss,
                                       void* grad, int64_t grad_ld, int32_t grad_dtype, int32_t* status_dev,
                                       domino_stream_t stream) {
  int rc = check_distill(args);
  if (rc != DOMINO_OK) return rc;
  if (!stats || (reinterpret_cast<uintptr_t>(stats) & 15u)) return DOMINO_ERR_INVALID_ARGUMENT;
  if ((rc = check_grad(*args, grad, grad_ld, grad_dtype)) != DOMINO_OK) return rc;
  const size_t rows = (size_t)args->rows, n = rows_span(args->rows, args->V, grad_ld, grad_dtype);
  if (overlap(grad, n, stats, rows * 32) || overlap(grad, n, grad_loss, rows * 4)) return DOMINO_ERR_INVALID_ARGUMENT;
  DistillArgs a = make_args(*args, status_dev);
  a.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
  a.grad_loss = grad_loss;
  a.grad = grad;
  a.grad_ld = grad_ld;
  cudaError_t e = launch_grad(a, grad_dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}
