// distill.cu -- distillation of rows of logits from a teacher's top logits: loss, and gradient.
//
// With x = z / T, L = log sum exp(x) over the row and L_rest the same over the tokens that are no entry, a
// row's loss is   w * (sum_k p_k (log p_k - x_k + L) + rho (log rho - L_rest + L))
// and its gradient   w / T * (P exp(x_v - L) - p_v)  at an entry's token,
//                    w / T * (P exp(L_rest - L) - rho) * exp(x_v - L_rest)  elsewhere.
// The row is summed without the entries' columns, about its own reference, and the at most 128 entries' terms are
// formed and added in 64 bits: S_rest as S less the entries' terms would be lost for a student that puts all but
// 1e-7 of its mass on them, and so would rho, one less the sum of p, with masses in fp32 for such a teacher.  log
// p_k is y_k less the entries' log-sum, so the entries need one exponential each.
//
// A cluster of blocks takes a row (k_distill): each sums its slice, they exchange sums through distributed shared
// memory, and for the gradient each reads its slice again, out of L2, and writes.  A block deals with the entries
// whose columns it has, in a warp of their own.  The backward call is elementwise from the stats (k_distill_grad).
#include "cluster.cuh"
#include "launch.cuh"
#include "vocab_rows.cuh"
#include "vocab_rows.h"

#include <algorithm>
#include <type_traits>

namespace domino {

namespace {

constexpr int kMaxK = DOMINO_MAX_TOP;
constexpr int kMaxCluster = 16;
constexpr int kEach = kMaxK / 32;  // entries a lane of the entries' warp

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
  int in_work;    // rows in work at a time, about
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

// What a block of a cluster knows of a row: sums over its columns, references and maximum.
struct Record {
  double s;    // terms of the columns that are no entry's, times 2^-n
  double ts;   // terms of its entries' distinct tokens, times 2^-tn
  double z;    // sum of exp(y - my) over its entries
  double a;    // sum of exp(y - my) (y - x)
  float n, m, tn;
};

// The entries of a row whose columns a block has.
struct Own {
  int n;             // how many
  int live;          // the teacher's row counts
  int twice;         // a token may be among them twice
  double my;         // what y is taken from: teacher_lse, or the row's largest y
  int32_t id[kMaxK];
  double y[kMaxK];   // from sum_own on p = exp(y - my), all of the token's entries at its first, -1 at the others
};

// What one warp makes of them.
struct OwnSums {
  double e[kMaxK];   // 2^(log2(e) x - tn)
  float tn;
  double ts, z, a;   // as in Record
};

// A row's entries, k = 32 i + lane, as one warp reads them.
struct Teacher {
  int32_t id[kEach];
  float t[kEach], lse;
};
__device__ __forceinline__ void read_teacher(const domino_distill_t& d, int r, Teacher& in) {
  in.lse = d.teacher_lse ? d.teacher_lse[r] : 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int k = 32 * i + (threadIdx.x & 31);
    in.id[i] = -1;
    in.t[i] = -INFINITY;
    if (k < d.K) {
      in.id[i] = __ldg(d.top_ids + (size_t)r * d.K + k);
      in.t[i] = __ldg(d.top_logits + (size_t)r * d.K + k);
    }
  }
}

// Has a later row's entries brought into L2: under a full load of reads a miss takes 3000 cycles.
__device__ __forceinline__ void await_teacher(const domino_distill_t& d, int r) {
  for (int at = (threadIdx.x & 31) * 32; at < d.K + 31; at += 32 * 32) {
    const size_t k = (size_t)r * d.K + min(at, d.K - 1);
    asm volatile("prefetch.global.L2 [%0];" ::"l"(d.top_ids + k));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(d.top_logits + k));
  }
}

// One warp: those for the block with columns [v0, v1).  Ends with the warp's barrier.
__device__ __forceinline__ void find_own(const DistillArgs& a, Teacher& in, int v0, int v1, Own& own, bool report) {
  const domino_distill_t& d = a.d;
  const int lane = threadIdx.x & 31;
  int32_t(&id)[kEach] = in.id;
  const float(&t)[kEach] = in.t;
  const float lse = in.lse;
  float most = -INFINITY;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (32 * i >= d.K) break;
    if (id[i] < 0 || id[i] >= d.V) {
      if (id[i] != -1 && report && a.status) set_status(a.status, DOMINO_STATUS_BAD_TOKEN);
      id[i] = -1;
    } else {
      most = fmaxf(most, t[i]);
    }
    const bool mine = id[i] >= v0 && id[i] < v1;  // -1 is not
    const uint32_t all = __ballot_sync(0xffffffffu, mine);
    if (mine) {
      const int at = n + __popc(all & ((1u << lane) - 1));
      own.id[at] = id[i];
      own.y[at] = t[i] > -INFINITY ? (double)big_clamp(t[i]) * a.inv_t : -INFINITY;
    }
    n += __popc(all);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 0) {
    own.n = n;
    if (d.teacher_lse) {
      own.live = fabsf(lse) < INFINITY;
      own.my = own.live ? (double)lse : 0.0;
    } else {
      own.live = most > -INFINITY;
      own.my = own.live ? (double)big_clamp(most) * a.inv_t : 0.0;
    }
  }
  __syncwarp();
}

// 2^e of a whole number, in 64 bits: 0 below 2^-1022, infinity above 2^1023.  A difference of references is exact where
// it lies between, as they are whole numbers.
__device__ __forceinline__ double pow2(float e) {
  const int n = (int)fminf(fmaxf(e, -1023.f), 1024.f);
  return __hiloint2double((n + 1023) << 20, 0);
}

// One warp: the sums over a block's entries, from their logits in `row`.  In 64 bits: what a peaked teacher leaves to
// the other tokens, one less the masses' sum, has no more digits than they have.
template <typename T>
__device__ __forceinline__ void sum_own(const DistillArgs& a, Own& own, const T* row, OwnSums& sums) {
  const int lane = threadIdx.x & 31, n = own.n;
  float z[kEach], most = -INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (32 * i >= n) break;
    z[i] = 32 * i + lane < n ? to_f32(row[own.id[32 * i + lane]]) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (32 * i >= n) break;
    most = fmaxf(most, z[i]);  // NaN aside
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  // a whole number that a float holds, as it is handed on in one: above 2^24 not every one is, and the reference may
  // lie as far as 64 below the largest term's exponent (1e6 at T = 2^-10: 1.5e9), so that a term is 2^64 at most
  const double to2 = a.inv_t * kLog2e;
  const float tn = most > -INFINITY ? ceilf((float)((double)big_clamp(most) * to2)) : -INFINITY;
  double ts = 0.0, zs = 0.0, as = 0.0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (32 * i >= n) break;
    const int k = 32 * i + lane;
    if (k >= n) break;
    const double y = own.y[k], x = (double)big_clamp(z[i]);
    const double p = y > -INFINITY ? exp(y - own.my) : 0.0;
    const double e = z[i] > -INFINITY ? exp2(x * to2 - (double)tn) : 0.0;
    own.y[k] = p;
    sums.e[k] = e;
    if (!own.twice) ts += e;
    zs += p;
    if (p > 0.0) as += z[i] > -INFINITY ? p * (y - x * a.inv_t) : INFINITY;
  }
  __syncwarp();
  if (own.twice) {  // a token's masses go to its first entry, and its term counts once
    double all[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = 32 * i + lane;
      if (k >= n) break;
      all[i] = own.y[k];
      for (int j = 0; j < n; ++j) {
        if (own.id[j] != own.id[k] || j == k) continue;
        if (j < k) all[i] = -1.0;
        else if (all[i] >= 0.0) all[i] += own.y[j];
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int k = 32 * i + lane;
      if (k >= n) break;
      own.y[k] = all[i];
      if (all[i] >= 0.0) ts += sums.e[k];
    }
  }
  __syncwarp();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    ts += __shfl_xor_sync(0xffffffffu, ts, o);
    zs += __shfl_xor_sync(0xffffffffu, zs, o);
    as += __shfl_xor_sync(0xffffffffu, as, o);
  }
  if (lane == 0) {
    sums.tn = tn;
    sums.ts = ts;
    sums.z = zs;
    sums.a = as;
  }
  __syncwarp();
}

// True S over the sum taken with c rounded to fp32: 2^(delta m).
__device__ __forceinline__ double rounding_of_c(float m, float c, double inv_t) {
  const double d = kLn2 * (kLog2e * inv_t - (double)c) * (double)big_clamp(m);
  return fabs(d) < 1e-5 ? 1.0 + d : exp(d);
}

// The blocks' records but for `a` as the row's, in every lane of a warp.
__device__ __forceinline__ Record join_records(const Record* recs, int cluster) {
  Record t = recs[threadIdx.x & (cluster - 1)];  // a power of two, at most 16
  const float own_n = t.n, own_tn = t.tn;
  for (int o = cluster / 2; o > 0; o >>= 1) {
    t.n = fmaxf(t.n, __shfl_xor_sync(0xffffffffu, t.n, o));
    t.tn = fmaxf(t.tn, __shfl_xor_sync(0xffffffffu, t.tn, o));
    t.m = fmaxf(t.m, __shfl_xor_sync(0xffffffffu, t.m, o));
  }
  t.s = own_n > -INFINITY ? t.s * pow2(own_n - t.n) : 0.0;
  t.ts = own_tn > -INFINITY ? t.ts * pow2(own_tn - t.tn) : 0.0;
  for (int o = cluster / 2; o > 0; o >>= 1) {
    t.s += __shfl_xor_sync(0xffffffffu, t.s, o);
    t.ts += __shfl_xor_sync(0xffffffffu, t.ts, o);
    t.z += __shfl_xor_sync(0xffffffffu, t.z, o);
  }
  return t;
}
__device__ __forceinline__ double join_a(const Record* recs, int cluster) {
  double a = recs[threadIdx.x & (cluster - 1)].a;
  for (int o = cluster / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
  return a;
}

// What a row's loss, stats and gradient are made of.
struct Row {
  int live;
  float top;           // reference of the next two
  double total, rest;  // S and what of it lies outside the entries
  double scale;        // w / T
  double psum, rho;    // the teacher's mass on the entries and elsewhere, together P
};

__device__ __forceinline__ Row row_of(const DistillArgs& a, float w, int live, const Record& t) {
  Row o;
  o.live = live && (t.z > 0.0 || isnan(t.z)) && (t.s > 0.0 || t.ts > 0.0);
  o.top = t.ts > 0.0 ? (t.s > 0.0 ? fmaxf(t.n, t.tn) : t.tn) : t.n;
  o.rest = t.s > 0.0 ? t.s * rounding_of_c(t.m, a.c, a.inv_t) * pow2(t.n - o.top) : 0.0;
  o.total = o.rest + (t.ts > 0.0 ? t.ts * pow2(t.tn - o.top) : 0.0);
  o.scale = (double)w * a.inv_t;
  o.psum = a.d.teacher_lse ? t.z : 1.0;
  o.rho = a.d.teacher_lse && t.s > 0.0 ? fmax(0.0, 1.0 - o.psum) : 0.0;
  return o;
}

// The factor of 2^(c z - n) in the gradient of a column that is no entry's: scale (P tau - rho) / s.  In 64 bits, as
// rho is, up to its rounding: rho has no more digits than the masses that it is one less the sum of, and the
// difference is small for a student close to its teacher.
__device__ __forceinline__ float coef_of(const Record& t, const Row& o) {
  if (!o.live || !(t.s > 0.0)) return 0.f;
  return (float)(o.scale * ((o.psum + o.rho) * o.rest - o.rho * o.total) / (o.total * t.s));
}

// What the data warps' gradient needs of a row: coef * 2^(c z - n) at a column that is no entry's.
struct Write {
  float n, coef;
  int guard;
};

// Loss and stats of a row: one thread of block 0.
__device__ __forceinline__ void finish_row(const DistillArgs& a, int r, double my, const Record& t, const Row& o) {
  if (!o.live) {
    a.loss[r] = 0.f;
    store_stats(a.stats, r, Stats{});
    return;
  }
  const double L = kLn2 * (log2(o.total) + (double)o.top);
  const double lp = a.d.teacher_lse ? my : my + log(t.z), zn = a.d.teacher_lse ? 1.0 : t.z;
  double loss = t.a / zn - o.psum * lp + o.psum * L;
  if (o.rho > 0.0) {  // log tau = log(rest / total) unless that is too small
    const double tau = o.rest / o.total;
    loss += o.rho * (tau < 1e-300 ? log(o.rho) - log_sum_exp(t.s, t.n, t.m, a.c, a.inv_t) + L : log(o.rho / tau));
  }
  a.loss[r] = (float)(o.scale / a.inv_t * loss);
  if (a.stats) {
    Stats st;
    st.n = t.n;
    st.rest = coef_of(t, o);
    st.l_hi = (float)L;
    st.l_lo = (float)(L - (double)st.l_hi);
    st.all = (float)(o.scale * (o.psum + o.rho));
    st.scale = (float)o.scale;
    st.lp_hi = (float)lp;
    st.lp_lo = (float)(lp - (double)st.lp_hi);
    store_stats(a.stats, r, st);
  }
}

constexpr int kMaxWarps = 8;  // of data, at most
struct WarpSums {
  float s[kMaxWarps], n[kMaxWarps], m[kMaxWarps];
};
// A warp's sum, in fp32, and maximum; the warps' are joined by one of them in 64 bits.
__device__ __forceinline__ void give_warp(WarpSums& ws, const ExpSum& acc, float m) {
  float n = acc.n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  const float s = warp_sum(n > -INFINITY ? acc.s * ex2(acc.n - n) : 0.f);
  if ((threadIdx.x & 31) == 0) {
    ws.n[threadIdx.x >> 5] = n;
    ws.m[threadIdx.x >> 5] = m;
    ws.s[threadIdx.x >> 5] = s;
  }
}
// One warp: the block's record, in every lane.
__device__ __forceinline__ Record block_record(const WarpSums& ws, int warps, const OwnSums& own) {
  const int at = threadIdx.x % kMaxWarps;
  const float mine = at < warps ? ws.n[at] : -INFINITY;
  float n = mine, m = at < warps ? ws.m[at] : -INFINITY;
#pragma unroll
  for (int o = kMaxWarps / 2; o > 0; o >>= 1) {
    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  double s = mine > -INFINITY ? (double)ws.s[at] * pow2(mine - n) : 0.0;
#pragma unroll
  for (int o = kMaxWarps / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return Record{s, own.ts, own.z, own.a, n, m, own.tn};
}
__device__ __forceinline__ void send_record(Record* to_slot, uint32_t to, const Record& t) {
  const uint32_t at = cluster_address(to_slot, to);
  cluster_store(at, t.s);
  cluster_store(at + 8, t.ts);
  cluster_store(at + 16, t.z);
  cluster_store(at + 24, t.a);
  cluster_store(at + 32, t.n, t.m);
  cluster_store(at + 40, __float_as_int(t.tn));
}

// Marks: a word for each thread and tile, with a byte for each of its kVecs vectors there and a bit for each column
// of an entry.  The threads clear their own, then one warp sets its block's entries'.
constexpr int kThreads = 256;
constexpr int kPerSm = 4;         // blocks an SM
constexpr int kData = kThreads - 32;
static_assert(kData / 32 <= kMaxWarps, "a slot for each data warp");
constexpr int kVecs = 4;          // 16-byte vectors a thread and tile
constexpr int kTile = kData * kVecs;
constexpr int kSlice = 40960;     // vectors of a slice at most: a byte of marks each
template <int N>
__device__ __forceinline__ void set_marks(uint32_t* marks, int first, Own& own) {
  bool twice = false;
  for (int k = threadIdx.x & 31; k < own.n; k += 32) {
    const int vec = own.id[k] / N - first, tile = vec / kTile, at = vec % kTile;
    const uint32_t bit = 1u << (at / kData * 8 + own.id[k] % N);
    twice |= (atomicOr(&marks[tile * kData + at % kData], bit) & bit) != 0;
  }
  twice = __any_sync(0xffffffffu, twice);
  if ((threadIdx.x & 31) == 0) own.twice = twice;
  __syncwarp();
}

__device__ __forceinline__ void store_grad(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_grad(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// Writes one vector's gradient, coef * 2^(c z - n), the first `columns` of it.  CHECK: its values may be NaN without
// guard saying so.
template <typename T, bool CHECK = false, typename G>
__device__ __forceinline__ void write_vector(G* out, int columns, const uint4& q, float c, float n, float coef,
                                             bool guard) {
  constexpr int N = Vec<T>::N;
  float z[N];
  widen(q, z);
  if (!guard) {
    const float2 c2 = make_float2(c, c), n2 = make_float2(-n, -n), k2 = make_float2(coef, coef);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 x = fma2(make_float2(z[e], z[e + 1]), c2, n2);
      const float2 t = CHECK ? make_float2(fmaxf(ex2(x.x), 0.f), fmaxf(ex2(x.y), 0.f))
                             : make_float2(ex2(x.x), ex2(x.y));
      const float2 y = mul2(t, k2);
      z[e] = y.x;
      z[e + 1] = y.y;
    }
  } else {
    for (int e = 0; e < N; ++e) z[e] = coef == 0.f ? 0.f : coef * term_guarded(z[e], c, n);
  }
  if (columns >= N) {
    if constexpr (sizeof(G) == 4) {
#pragma unroll
      for (int e = 0; e < N; e += 4)
        __stcs(reinterpret_cast<float4*>(out + e), make_float4(z[e], z[e + 1], z[e + 2], z[e + 3]));
    } else {
      __nv_bfloat162 h[N / 2];
#pragma unroll
      for (int e = 0; e < N; e += 2) h[e / 2] = __floats2bfloat162_rn(z[e], z[e + 1]);
      if constexpr (N == 8) __stcs(reinterpret_cast<uint4*>(out), *reinterpret_cast<uint4*>(h));
      else __stcs(reinterpret_cast<uint2*>(out), *reinterpret_cast<uint2*>(h));
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < columns) store_grad(out + e, z[e]);
  }
}

// Named barriers of a block, for warps that go different ways (0 is __syncthreads): `n` threads arrive or wait.
template <int ID>
__device__ __forceinline__ void bar_arrive(int n) {
  asm volatile("bar.arrive %0, %1;" ::"n"(ID), "r"(n) : "memory");
}
template <int ID>
__device__ __forceinline__ void bar_wait(int n) {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "r"(n) : "memory");
}

// A thread's own vectors of a slice, tile after tile.  Ahead in registers, one tile; or, for the gradient, by
// asynchronous copies into its own places of shared memory, kStages - 1 tiles: no barrier is needed for either.
// (Loss and gradient of 1024 rows of 151936 bf16, when built: 136 us by registers, 127 by copies, 2 or 4 stages 130
// and 147; the loss alone of 512 rows fp32, whose larger slices' marks want the shared memory: 48 by registers and
// 57.)
constexpr int kStages = 3;
constexpr int kRing = kStages * kTile * 16;

struct Ahead {
  const uint4* at;
  uint4 next[kVecs];
  template <typename T>
  __device__ __forceinline__ void start(const uint4* slice, int vecs, char*) {
    at = slice + threadIdx.x;
    load_tile<T, kVecs, false>(next, at, kData, vecs);
  }
  // The next tile; `left` vectors of the slice remain from it on.
  template <typename T>
  __device__ __forceinline__ void take(uint4 (&q)[kVecs], int left) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) q[i] = next[i];
    at += kTile;
    load_tile<T, kVecs, false>(next, at, kData, left - kTile);
  }
};

struct Copies {
  const uint4* from;  // the thread's vector of the next tile to fetch
  uint4* ring;        // the thread's places: [kStages][kVecs], kData apart
  int left, put, get; // vectors of the slice from that tile on; places
  __device__ __forceinline__ void fetch() {
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
      if (i * kData + (int)threadIdx.x < left)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(ring + put * kTile + i * kData)),
                     "l"(from + i * kData)
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
    from += kTile;
    left -= kTile;
    put = put + 1 == kStages ? 0 : put + 1;
  }
  template <typename T>
  __device__ __forceinline__ void start(const uint4* slice, int vecs, char* shared) {
    ring = reinterpret_cast<uint4*>(shared) + threadIdx.x;
    from = slice + threadIdx.x;
    left = vecs;
    put = get = 0;
#pragma unroll
    for (int s = 0; s + 1 < kStages; ++s) fetch();
  }
  template <typename T>
  __device__ __forceinline__ void take(uint4 (&q)[kVecs], int now) {
    fetch();  // into the places read one tile ago
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
#pragma unroll
    for (int i = 0; i < kVecs; ++i) q[i] = ring[get * kTile + i * kData];
    if (now < kTile) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (i * kData + (int)threadIdx.x >= now) q[i] = barred_vec<T>();
    }
    get = get + 1 == kStages ? 0 : get + 1;
  }
};

// Loss, and gradient (G not void), of one row a cluster.  Data warps stream the slice, the next tiles on the way while
// one is worked on; one warp has the entries and the exchange.
//
// Bound by memory, then by the exponentials: V values are read once from DRAM and V written; one exponential for the
// sum and one for the gradient (16 a clock and SM) take two thirds of the memory's time for bf16 in and out, half of
// it for fp32.  The second read hits L2 while the rows in work take at most 48 MB, which the launch sees to with the
// cluster's size as far as 16 blocks a row will do (up to 340,000 fp32 or 680,000 bf16 a row; at 2^20 fp32 they are
// 155 MB, more than L2 holds): 1024 rows of 151936 bf16 read 275 MB of DRAM for the 272 MB that their live rows
// have.  Measured there: 117 us (584 MB, 5.0 TB/s; 128 when calls of it in a row bring the power limit's 1.77 GHz);
// holding a row in registers or in shared memory between its sum and its gradient took 231 and 346 us, for the work
// they leave to few threads; bringing the next rows into L2 meanwhile was no faster.  The entries and the row's
// factors in 64 bits take 1 of the 117 us.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads, kPerSm) k_distill(DistillArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr bool kGrad = !std::is_void<G>::value;
  __shared__ struct {
    Record recs[kMaxCluster];
    Own own;
    OwnSums sums;
    WarpSums warps;
    Write write;
  } sh;
  // the copies' places, then the marks; a place that does not start on 32 bytes costs (130 us for 116 with 16 off)
  extern __shared__ __align__(128) char dynamic[];
  uint32_t* const marks = reinterpret_cast<uint32_t*>(dynamic + (kGrad ? kRing : 0));
  pdl_wait();
  pdl_trigger();
  const domino_distill_t& d = a.d;
  const int cluster = a.cluster, r = blockIdx.x / cluster, tid = threadIdx.x;
  const uint32_t rank = blockIdx.x % cluster;
  const int all = (d.V + N - 1) / N, per = (all + cluster - 1) / cluster;
  const int first = min((int)rank * per, all), last = min(first + per, all);
  const float w = d.row_weights ? d.row_weights[r] : 1.f;
  Teacher in_row;
  if (tid >= kData) {  // on their way together with the weight
    read_teacher(d, r, in_row);
    if (rank == 0 && a.in_work < d.rows - r) await_teacher(d, r + a.in_work);
  } else {
    for (int i = 0; i < last - first; i += kTile) marks[i / kVecs + tid] = 0;
  }
  const T* row = static_cast<const T*>(d.logits) + (size_t)r * d.ld;
  using Out = typename std::conditional<kGrad, G, float>::type;
  Out* out = kGrad ? static_cast<Out*>(a.grad) + (size_t)r * a.grad_ld : nullptr;
  if (w == 0.f) {  // the whole cluster
    if constexpr (kGrad) {
      for (int vec = first + tid; vec < last; vec += kThreads)
        write_vector<T>(out + vec * N, d.V - vec * N, barred_vec<T>(), a.c, 0.f, 0.f, true);
    }
    if (rank == 0 && tid == 0) {
      a.loss[r] = 0.f;
      store_stats(a.stats, r, Stats{});
    }
    return;
  }
  cluster_arrive_relaxed();  // all blocks have started before one stores into another
  if (tid < kData) {
    bar_arrive<2>(kThreads);  // the marks are clear
    const uint4* const slice = reinterpret_cast<const uint4*>(row) + first;
    typename std::conditional<kGrad, Copies, Ahead>::type in;
    in.template start<T>(slice, last - first, dynamic);
    bar_wait<1>(kThreads);  // the marks are set
    const uint32_t* mark = marks + tid;
    ExpSum acc;
    float m = -INFINITY;
    bool guard = false;
    for (int left = last - first; left > 0; left -= kTile) {
      uint4 q[kVecs];
      in.template take<T>(q, left);
      const uint32_t mk = *mark;
      mark += kData;
      if (mk) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) bar_elements<T>(q[i], (mk >> (8 * i)) & 0xffu);
      }
      if (left <= kTile && d.V % N != 0) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) bar_elements<T>(q[i], beyond<T>((last - left + i * kData + tid) * N, d.V));
      }
      float tm = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) tm = fmaxf(tm, vec_max(q[i], T()));
      m = fmaxf(m, tm);
      guard |= add_vectors<T>(acc, q, (left + kData - 1) / kData, tm, a.c);
    }
    give_warp(sh.warps, acc, m);
    bar_arrive<2>(kThreads);  // sh.warps
    if (kGrad) in.template start<T>(slice, last - first, dynamic);
    cluster_wait();
    cluster_arrive_relaxed();
    if constexpr (kGrad) {
      bar_wait<1>(kThreads);  // sh.write
      const float n = sh.write.n, coef = sh.write.coef;
      guard |= sh.write.guard != 0;
      Out* to = out + (first + tid) * N;
      for (int left = last - first; left > 0; left -= kTile, to += kTile * N) {
        uint4 q[kVecs];
        in.template take<T>(q, left);
        if (left > kTile) {  // whole vectors
#pragma unroll
          for (int i = 0; i < kVecs; ++i) write_vector<T>(to + i * kData * N, N, q[i], a.c, n, coef, guard);
        } else {
#pragma unroll
          for (int i = 0; i < kVecs; ++i) {
            const int vec = last - left + i * kData + tid;
            if (vec < last) write_vector<T>(to + i * kData * N, d.V - vec * N, q[i], a.c, n, coef, guard);
          }
        }
      }
      bar_arrive<2>(kThreads);  // the entries' columns go over the others'
    }
    cluster_wait();
    return;
  }
  const int lane = tid & 31;
  find_own(a, in_row, first * N, last * N, sh.own, rank == 0);
  bar_wait<2>(kThreads);  // the marks are clear
  set_marks<N>(marks, first, sh.own);
  bar_wait<1>(kThreads);  // the marks are set
  sum_own(a, sh.own, row, sh.sums);
  bar_wait<2>(kThreads);  // sh.warps
  const Record rec = block_record(sh.warps, kData / 32, sh.sums);
  cluster_wait();
  if (lane < (kGrad ? cluster : 1)) send_record(&sh.recs[rank], lane, rec);
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  if (!kGrad && rank != 0) return;
  Record t = join_records(sh.recs, cluster);
  const Row o = row_of(a, w, sh.own.live, t);
  if constexpr (kGrad) {
    const float coef = coef_of(t, o);
    if (lane == 0) sh.write = Write{t.n, coef, coef == 0.f || is_extreme(t.m)};
    bar_wait<1>(kThreads);  // sh.write
  }
  if (rank == 0) {
    t.a = join_a(sh.recs, cluster);
    if (lane == 0) finish_row(a, r, sh.own.my, t, o);
  }
  if constexpr (kGrad) {
    // an entry's: scale * (P q - p)
    const double of_e = t.ts > 0.0 ? o.scale * (o.psum + o.rho) * pow2(sh.sums.tn - o.top) / o.total : 0.0;
    const double of_p = d.teacher_lse ? o.scale : o.scale / t.z;
    bar_wait<2>(kThreads);
    if (o.live)
      for (int k = lane; k < sh.own.n; k += 32)
        if (sh.own.y[k] >= 0.0) store_grad(out + sh.own.id[k], (float)(of_e * sh.sums.e[k] - of_p * sh.own.y[k]));
  }
}

// The gradient from a row's stats, a chunk of kGradVecs vectors a thread by each block, all loaded at once; the chunk's
// entries are found by one warp and taken by as many threads meanwhile.  The logits may be overwritten: the entries
// read theirs first.  Bound by memory: forward and backward of 360 rows of 50001 bf16 take 30 us of GPU time together
// for 104 MB, of which the two kernels' starts and the entries' chains of loads are a third.
constexpr int kGradThreads = 256;
static_assert(kGradThreads >= kMaxK, "a thread an entry");
constexpr int kGradVecs = 8;

template <typename T, typename G>
__global__ void __launch_bounds__(kGradThreads, 4) k_distill_grad(DistillArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Own own;
  __shared__ uint32_t bits[kGradThreads * kGradVecs * N / 32];  // the chunk's columns that are entries'
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
  float own_z = 0.f;
  int own_at = -1;  // the column of the thread's entry
  bool twice = false;
  if (live) {
    for (int i = tid; i < kGradThreads * kGradVecs * N / 32; i += kGradThreads) bits[i] = 0;
    if (tid < 32) {
      Teacher in;
      read_teacher(d, r, in);
      find_own(a, in, first * N, min(first + kGradThreads * kGradVecs, all) * N, own, false);
    }
    __syncthreads();
    bool again = false;
    if (tid < own.n) {
      own_at = own.id[tid];
      own_z = to_f32(row[own_at]);
      const int at = own_at - first * N;
      const uint32_t bit = 1u << (at & 31);
      again = (atomicOr(&bits[at >> 5], bit) & bit) != 0;
    }
    twice = __syncthreads_or(again);  // the entries' logits are read, too
  }
  const float coef = live ? g * st.rest : 0.f;
  const bool guard = coef == 0.f || is_extreme(st.n / a.c);
#pragma unroll
  for (int i = 0; i < kGradVecs; ++i) {
    const int vec = first + i * kGradThreads + tid;
    if (vec < all) write_vector<T, true>(out + vec * N, d.V - vec * N, q[i], a.c, st.n, coef, guard);
  }
  float own_grad = 0.f;
  if (own_at >= 0) {  // in 64 bits, as in k_distill, while the vectors are on their way
    const double lp = (double)st.lp_hi + (double)st.lp_lo, L = (double)st.l_hi + (double)st.l_lo;
    double p = own.y[tid] > -INFINITY ? exp(own.y[tid] - lp) : 0.0;
    const double q_v = own_z > -INFINITY ? exp((double)big_clamp(own_z) * a.inv_t - L) : 0.0;
    if (twice) {
      for (int j = 0; j < own.n; ++j)
        if (own.id[j] == own.id[tid] && j != tid) {
          if (own.y[j] > -INFINITY) p += exp(own.y[j] - lp);
          if (j < tid) own_at = -1;  // the token's first entry writes
        }
    }
    own_grad = (float)((double)g * (q_v * (double)st.all - p * (double)st.scale));
  }
  // a bad id of a row that is read, one without a gradient too: by the row's first block
  if (a.status && chunk == 0 && tid < d.K && g != 0.f && !(d.row_weights && d.row_weights[r] == 0.f)) {
    const int32_t id = __ldg(d.top_ids + (size_t)r * d.K + tid);
    if (id < -1 || id >= d.V) set_status(a.status, DOMINO_STATUS_BAD_TOKEN);
  }
  __syncthreads();
  if (own_at >= 0) store_grad(out + own_at, own_grad);
}

int vectors_of(const domino_distill_t& d) { return d.dtype == DOMINO_DTYPE_F32 ? (d.V + 3) / 4 : (d.V + 7) / 8; }

// Loss, and gradient where a.grad is set.
cudaError_t launch_distill(DistillArgs a, int grad_dtype, cudaStream_t st) {
  const int vecs = vectors_of(a.d);
  const int64_t blocks = kPerSm * 148;  // at a time
  const bool f = a.d.dtype == DOMINO_DTYPE_F32;
  int cluster = 1;
  // larger clusters: for slices that have their marks in shared memory; while all blocks can still run at once, so
  // that few rows use every SM; and to keep the rows in work in about 48 MB of L2
  while (cluster < kMaxCluster &&
         (vecs > cluster * kSlice || (2 * cluster * (int64_t)a.d.rows <= blocks && vecs / (2 * cluster) >= 2 * kData) ||
          (a.grad && std::min<int64_t>(a.d.rows, blocks / cluster) * vecs * 16 > (48 << 20) &&
           vecs / (2 * cluster) >= 2 * kData)))
    cluster *= 2;
  a.cluster = cluster;
  a.in_work = (int)(blocks / cluster);
  const int smem = (a.grad ? kRing : 0) + ((vecs + cluster - 1) / cluster + kTile - 1) / kTile * kTile;
  const bool g = grad_dtype == DOMINO_DTYPE_F32;
  auto kern = !a.grad ? (f ? k_distill<float, void> : k_distill<bf16, void>)
                      : f ? (g ? k_distill<float, float> : k_distill<float, bf16>)
                          : (g ? k_distill<bf16, float> : k_distill<bf16, bf16>);
  // the most that any call needs: host threads may be in here at once
  constexpr int most = kRing + (kSlice + kTile - 1) / kTile * kTile;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
  if (e != cudaSuccess) return e;
  return note_launch(launch_cluster(kern, cluster, dim3((unsigned)a.d.rows * (unsigned)cluster), dim3(kThreads), smem,
                                    st, a));
}

cudaError_t launch_grad(DistillArgs a, int grad_dtype, cudaStream_t st) {
  a.cluster = (vectors_of(a.d) + kGradThreads * kGradVecs - 1) / (kGradThreads * kGradVecs);
  const bool f = a.d.dtype == DOMINO_DTYPE_F32, g = grad_dtype == DOMINO_DTYPE_F32;
  auto kern = f ? (g ? k_distill_grad<float, float> : k_distill_grad<float, bf16>)
                : (g ? k_distill_grad<bf16, float> : k_distill_grad<bf16, bf16>);
  return note_launch(launch_pdl(kern, dim3((unsigned)a.d.rows * (unsigned)a.cluster), dim3(kGradThreads), 0, st, a));
}

int check_distill(const domino_distill_t* d) {
  if (!d || !rows_ok(d->rows, d->V, d->ld, d->dtype, d->logits)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (d->K < 1 || d->K > DOMINO_MAX_TOP || !temperature_ok(d->temperature)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (!d->top_ids || !d->top_logits) return DOMINO_ERR_INVALID_ARGUMENT;
  for (const void* q : {(const void*)d->top_ids, (const void*)d->top_logits, (const void*)d->teacher_lse,
                        (const void*)d->row_weights})
    if (!aligned4(q)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (d->rows > DOMINO_MAX_ROWS) return DOMINO_ERR_UNSUPPORTED;
  return DOMINO_OK;
}

// The checks of a call's outputs: alignment, and that no two of them, nor one and an input, share memory -- but
// for a gradient in the place of the logits.  grad_loss: another input, or null.
int check_outputs(const domino_distill_t& d, const float* loss, const float* stats, bool stats_out,
                  const float* grad_loss, const void* grad, int64_t grad_ld, int grad_dtype) {
  if (!aligned4(loss) || !aligned4(grad_loss) || (reinterpret_cast<uintptr_t>(stats) & 15u))
    return DOMINO_ERR_INVALID_ARGUMENT;
  if (grad && !rows_ok(d.rows, d.V, grad_ld, grad_dtype, grad)) return DOMINO_ERR_INVALID_ARGUMENT;
  const size_t rows = (size_t)d.rows, e = rows * d.K * 4, in_bytes = rows_span(d.rows, d.V, d.ld, d.dtype);
  const size_t grad_bytes = grad ? rows_span(d.rows, d.V, grad_ld, grad_dtype) : 0;
  const bool in_place = grad == d.logits && grad_ld == d.ld && grad_dtype == d.dtype;
  const Range ids{d.top_ids, e}, tops{d.top_logits, e}, lse{d.teacher_lse, rows * 4}, w{d.row_weights, rows * 4},
      given{stats_out ? nullptr : stats, rows * 32}, up{grad_loss, rows * 4};
  if (!disjoint({{loss, rows * 4}, {stats_out ? stats : nullptr, rows * 32}, {grad, grad_bytes}},
                {ids, tops, lse, w, given, up}) ||
      !disjoint({{loss, rows * 4}, {stats_out ? stats : nullptr, rows * 32}, {in_place ? nullptr : grad, grad_bytes}},
                {{d.logits, in_bytes}}))
    return DOMINO_ERR_INVALID_ARGUMENT;
  return DOMINO_OK;
}

DistillArgs make_args(const domino_distill_t& d, int32_t* status) {
  DistillArgs a{};
  a.d = d;
  a.inv_t = 1.0 / (double)d.temperature;
  a.c = (float)(kLog2e * a.inv_t);
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
  if (!loss || !aligned4(status_dev)) return DOMINO_ERR_INVALID_ARGUMENT;
  if ((rc = check_outputs(*args, loss, stats, true, nullptr, grad, grad_ld, grad_dtype)) != DOMINO_OK) return rc;
  DistillArgs a = make_args(*args, status_dev);
  a.loss = loss;
  a.stats = reinterpret_cast<float4*>(stats);
  a.grad = grad;
  a.grad_ld = grad_ld;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_distill(a, grad_dtype, cs);
  return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}

extern "C" int domino_distill_backward(const domino_distill_t* args, const float* stats, const float* grad_loss,
                                       void* grad, int64_t grad_ld, int32_t grad_dtype, int32_t* status_dev,
                                       domino_stream_t stream) {
  int rc = check_distill(args);
  if (rc != DOMINO_OK) return rc;
  if (!stats || !grad || !aligned4(status_dev)) return DOMINO_ERR_INVALID_ARGUMENT;
  if ((rc = check_outputs(*args, nullptr, stats, false, grad_loss, grad, grad_ld, grad_dtype)) != DOMINO_OK) return rc;
  DistillArgs a = make_args(*args, status_dev);
  a.stats = reinterpret_cast<float4*>(const_cast<float*>(stats));
  a.grad_loss = grad_loss;
  a.grad = grad;
  a.grad_ld = grad_ld;
  cudaError_t e = launch_grad(a, grad_dtype, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}
