// top_logits.cu -- the k largest logits of every row, in order, with the row's log-sum-exp.
//
// A row is read once, by a cluster of blocks that take contiguous slices of it.  A block walks its slice in
// tiles of kVecs 16-byte vectors a thread, held in registers: each thread takes its tile maximum and adds the
// tile's exponentials; then a threshold says which values can still be among the k largest, and those go to
// a list in shared memory.  The threshold comes from the thread maxima alone: a value that k threads' maxima
// reach has k values at or above it, so the k largest are at or above it too, and about as many values as
// threads are (a thread's second largest rarely is).  It is found by bisection over the order-preserving bits
// of the maxima, one __syncthreads_count a probe.  In later tiles, whose columns are higher, a value has to
// exceed the threshold.  Should one tile still bring more values than the list holds (all large values in one
// thread's columns, or a row of equal ones), the exact k are selected from the registers by bisection over
// value and column.  Each block ranks its list; block 0 receives the blocks' sorted lists and sums through
// distributed shared memory, and ranks a key by binary search in each.
#include "cluster.cuh"
#include "launch.cuh"
#include "vocab_rows.cuh"
#include "vocab_rows.h"

namespace domino {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 8;        // 16-byte vectors a thread and tile
constexpr int kList = 2048;     // candidates held; a tile adds about k + k * k / 1024
constexpr int kTidy = 1024;     // more than this are cut to the k largest before the next tile
constexpr int kMaxCluster = 16;
constexpr int kMaxK = DOMINO_MAX_TOP;

struct TopShared {
  uint64_t list[kList];
  uint64_t sorted[kMaxCluster][kMaxK];  // block 0: every block's k largest in order
  double sum[kMaxCluster];              // block 0: every block's sum ...
  float ref[kMaxCluster][2];            // ... its reference and maximum
  double red_s[kWarps];
  float red_n[kWarps], red_m[kWarps];
  uint32_t red_u[2][kWarps];
  int red_i[kWarps];
  int count;
};

template <typename T> __device__ __forceinline__ uint4 barred_vec();
template <> __device__ __forceinline__ uint4 barred_vec<float>() {
  return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
}
template <> __device__ __forceinline__ uint4 barred_vec<bf16>() {
  return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
}
// The vector at column v of a row of V with the columns from V on barred.
template <typename T>
__device__ __forceinline__ uint4 cut_vec(uint4 q, int v, int V) {
  T* e = reinterpret_cast<T*>(&q);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i)
    if (v + i >= V) e[i] = static_cast<T>(-INFINITY);
  return q;
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

// Adds a tile with maximum m > -infinity to the thread's sum; its first `vecs` vectors hold columns.
template <typename T>
__device__ __forceinline__ void add_tile(ExpSum& a, const uint4 (&q)[kVecs], int vecs, float m, float c) {
  const float n = fmaxf(a.n, reference_of(m, c));
  if (n > a.n) raise(a, n);
  float s0 = 0.f, s1 = 0.f;
  if (!is_extreme(m)) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if (i >= vecs) break;
      float z[Vec<T>::N];
      widen(q[i], z);
#pragma unroll
      for (int e = 0; e < Vec<T>::N; e += 2) {
        s0 += ex2(fmaf(z[e], c, -n));
        s1 += ex2(fmaf(z[e + 1], c, -n));
      }
    }
  }
  float s = s0 + s1;
  if (is_extreme(m) || isnan(s)) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float z[Vec<T>::N];
      widen(q[i], z);
#pragma unroll
      for (int e = 0; e < Vec<T>::N; ++e) s += term_guarded(z[e], c, n);
    }
  }
  a.s += s;
}

// Block 0's thread 0 gets sums over the block's threads.
__device__ __forceinline__ void join_threads(const ExpSum& a, float m, TopShared& sh, double* sum, float* ref, float* max) {
  float n = a.n, mm = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
    mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  }
  double s = n > -INFINITY ? (double)(a.s * ex2(a.n - n)) : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) {
    sh.red_n[threadIdx.x >> 5] = n;
    sh.red_m[threadIdx.x >> 5] = mm;
    sh.red_s[threadIdx.x >> 5] = s;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kWarps; ++w) {
    n = fmaxf(n, sh.red_n[w]);
    mm = fmaxf(mm, sh.red_m[w]);
  }
  s = 0.0;
  for (int w = 0; w < kWarps; ++w)
    if (sh.red_n[w] > -INFINITY) s += sh.red_s[w] * (double)ex2(sh.red_n[w] - n);
  *sum = s;
  *ref = n;
  *max = mm;
}

// The list's keys in order, cut to k: sh.list[0 .. min(k, n)).  All threads call it; returns the new count.
__device__ __forceinline__ int tidy(TopShared& sh, int n, int k, uint64_t* to) {
  constexpr int kEach = kList / kThreads;
  uint64_t key[kEach];
  int rank[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = threadIdx.x + i * kThreads;
    key[i] = 0;
    rank[i] = 0;
    if (at >= n) continue;
    key[i] = sh.list[at];
    for (int j = 0; j < n; ++j) rank[i] += sh.list[j] > key[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (key[i] != 0 && rank[i] < k) to[rank[i]] = key[i];
  const int left = min(n, k);
  if (threadIdx.x == 0) sh.count = left;
  __syncthreads();
  return left;
}

// A value that at least k of the threads' maxima reach, from their order bits `o` (at least k are not 0).
__device__ __forceinline__ uint32_t reached_by(uint32_t o, int k, TopShared& sh) {
  const uint32_t hi_w = __reduce_max_sync(0xffffffffu, o), lo_w = __reduce_min_sync(0xffffffffu, o);
  if ((threadIdx.x & 31) == 0) {
    sh.red_u[0][threadIdx.x >> 5] = lo_w;
    sh.red_u[1][threadIdx.x >> 5] = hi_w;
  }
  __syncthreads();
  uint32_t lo = sh.red_u[0][0], hi = sh.red_u[1][0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    lo = min(lo, sh.red_u[0][w]);
    hi = max(hi, sh.red_u[1][w]);
  }
  lo = max(lo, 1u);
  hi += 1;  // at least k reach lo, fewer than k reach hi
  const int enough = k + k / 4 + 8;
  while (hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int c = __syncthreads_count(o >= mid);
    if (c >= k) {
      lo = mid;
      if (c <= enough) break;
    } else {
      hi = mid;
    }
  }
  return lo;
}

// The least float above x < infinity.
__device__ __forceinline__ float nextafter_up(float x) { return order_value(order_of(x) ? order_of(x) + 1 : 0x00800000u); }

__device__ __forceinline__ int block_count(int n, TopShared& sh) {
  n = __reduce_add_sync(0xffffffffu, n);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.red_i[threadIdx.x >> 5] = n;
  __syncthreads();
  int c = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) c += sh.red_i[w];
  return c;
}

// The exact k of the `held` keys in the list and of the vectors [t0, t1) of a row, read again, into the list.
// Returns the least value kept.
template <typename T>
__device__ __noinline__ float select_exact(const T* row, int t0, int t1, int V, int held, int k, TopShared& sh) {
  constexpr int kEach = kList / kThreads;
  uint64_t own[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int at = threadIdx.x + i * kThreads;
    own[i] = at < held ? sh.list[at] : 0;
  }
  auto each = [&](auto f) {
    for (int vec = t0 + threadIdx.x; vec < t1; vec += kThreads) {
      const int v = vec * Vec<T>::N;
      for (int e = 0; e < Vec<T>::N; ++e)
        if (v + e < V) f(select_key(order_of(to_f32(row[v + e])), v + e));
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) f(own[i]);
  };
  uint64_t lo = 0;  // the largest key with at least k at or above it: keys are all different
  for (int bit = 63; bit >= 0; --bit) {
    const uint64_t probe = lo | (1ull << bit);
    int n = 0;
    each([&](uint64_t key) { n += key >= probe ? 1 : 0; });
    if (block_count(n, sh) >= k) lo = probe;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  each([&](uint64_t key) {
    if (key >= lo) sh.list[atomicAdd(&sh.count, 1)] = key;
  });
  __syncthreads();
  return order_value((uint32_t)(lo >> 32));
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) k_top_rows(TopRows a, int cluster) {
  constexpr int N = Vec<T>::N;
  __shared__ TopShared sh;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x / cluster, tid = threadIdx.x;
  const uint32_t rank = blockIdx.x % cluster;
  if ((a.scores && !(a.scores[r] > -INFINITY)) || (a.finished && a.finished[r])) return;  // the whole cluster
  if (tid == 0) sh.count = 0;
  if (cluster > 1) cluster_arrive();  // block 0 has started before another stores into it
  const T* row = static_cast<const T*>(a.logits) + (size_t)r * a.ld;
  const int all = (a.V + N - 1) / N, per = (all + cluster - 1) / cluster;
  const int first = min((int)rank * per, all), last = min(first + per, all);
  ExpSum acc;
  float m = -INFINITY, bar = -INFINITY;
  int held = 0;  // keys in the list
  for (int t0 = first; t0 < last; t0 += kThreads * kVecs) {
    const int vecs = min((last - t0 + kThreads - 1) / kThreads, kVecs);  // vectors of the tile's first thread
    uint4 q[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int vec = t0 + i * kThreads + tid;
      q[i] = vec < last ? __ldcs(reinterpret_cast<const uint4*>(row) + vec) : barred_vec<T>();
    }
    if (a.V % N != 0 && t0 + kThreads * kVecs >= all) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) q[i] = cut_vec<T>(q[i], (t0 + i * kThreads + tid) * N, a.V);
    }
    float vm[kVecs], tm = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      vm[i] = -INFINITY;
      if (i < vecs) vm[i] = fmaxf(vec_max(q[i], T()), -INFINITY);
      tm = fmaxf(tm, vm[i]);
    }
    if (tm > -INFINITY) {
      m = fmaxf(m, tm);
      add_tile<T>(acc, q, vecs, tm, a.c);
    }
    // the barrier also ends the previous tile's use of the list
    const int hot = __syncthreads_count(tm > bar);
    if (hot == 0) continue;
    bool equal_too = false;  // the bar is this tile's own
    if (hot >= a.k) {
      const float own = order_value(reached_by(order_of(tm), a.k, sh));
      equal_too = own > bar;
      bar = fmaxf(bar, own);
    }
    const float floor = equal_too ? bar : nextafter_up(bar);  // values from here on go to the list
    if (tm >= floor) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        if (vm[i] >= floor) {
          const int v = (t0 + i * kThreads + tid) * N;
          float z[N];
          widen(q[i], z);
#pragma unroll
          for (int e = 0; e < N; ++e)
            if (z[e] >= floor) {
              const int at = atomicAdd(&sh.count, 1);
              if (at < kList) sh.list[at] = select_key(order_of(z[e]), v + e);
            }
        }
      }
    }
    __syncthreads();
    const int n = sh.count;
    if (n > kList) {
      bar = select_exact(row, t0, min(t0 + kThreads * kVecs, last), a.V, held, a.k, sh);
      held = a.k;
    } else if (n > kTidy && t0 + kThreads * kVecs < last) {
      held = tidy(sh, n, a.k, sh.list);
      bar = fmaxf(bar, order_value((uint32_t)(sh.list[a.k - 1] >> 32)));
    } else {
      held = n;
    }
  }
  __syncthreads();
  const int found = tidy(sh, held, a.k, sh.sorted[0]);
  double sum = 0.0;
  float ref = -INFINITY, max = -INFINITY;
  join_threads(acc, m, sh, &sum, &ref, &max);
  float* const values = a.values + (size_t)r * a.k;
  int32_t* const ids = a.ids + (size_t)r * a.k;
  int have = found;
  if (cluster > 1) {
    cluster_wait();
    if (rank != 0) {
      const uint32_t to = cluster_address(sh.sorted[rank], 0);
      for (int i = tid; i < a.k; i += kThreads) cluster_store(to + 8 * i, i < found ? sh.sorted[0][i] : (uint64_t)0);
      if (tid == 0) {
        cluster_store(cluster_address(&sh.sum[rank], 0), sum);
        cluster_store(cluster_address(sh.ref[rank], 0), ref, max);
      }
    } else {
      for (int i = found + tid; i < a.k; i += kThreads) sh.sorted[0][i] = 0;
      if (tid == 0) {
        sh.sum[0] = sum;
        sh.ref[0][0] = ref;
        sh.ref[0][1] = max;
      }
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    have = 0;
    const int total = cluster * a.k;
    for (int i0 = 0; i0 < total; i0 += kThreads) {
      const int i = i0 + tid, c = i / a.k, p = i % a.k;
      const uint64_t key = i < total ? sh.sorted[c][p] : 0;
      if (key != 0) {
        int place = p;
        for (int o = 0; o < cluster && place < a.k; ++o) {
          if (o == c) continue;
          int lo = 0, hi = a.k;  // keys before lo are larger, from hi on are not
          while (lo < hi) {
            const int mid = (lo + hi) / 2;
            if (sh.sorted[o][mid] > key) lo = mid + 1;
            else hi = mid;
          }
          place += lo;
        }
        if (place < a.k) {
          values[place] = order_value((uint32_t)(key >> 32));
          ids[place] = key_index(key);
        }
      }
      have += __syncthreads_count(key != 0);
    }
    if (tid == 0) {
      for (int c = 1; c < cluster; ++c) {
        ref = fmaxf(ref, sh.ref[c][0]);
        max = fmaxf(max, sh.ref[c][1]);
      }
      sum = 0.0;
      for (int c = 0; c < cluster; ++c)
        if (sh.ref[c][0] > -INFINITY) sum += sh.sum[c] * (double)ex2(sh.ref[c][0] - ref);
    }
  } else {
    for (int i = tid; i < found; i += kThreads) {
      const uint64_t key = sh.sorted[0][i];
      values[i] = order_value((uint32_t)(key >> 32));
      ids[i] = key_index(key);
    }
  }
  for (int i = have + tid; i < a.k; i += kThreads) {
    values[i] = -INFINITY;
    ids[i] = -1;
  }
  if (tid == 0) {
    const double lse = log_sum_exp(sum, ref, max, a.c, a.inv_t);
    if (a.lse) a.lse[r] = (float)lse;
    if (a.lse64) a.lse64[r] = lse;
  }
}

}  // namespace

cudaError_t launch_top_rows(const TopRows& a, cudaStream_t st) {
  const bool f = a.dtype == DOMINO_DTYPE_F32;
  const int vecs = (a.V + (f ? 3 : 7)) / (f ? 4 : 8);
  // enough blocks for two on each of 148 SMs, none with less than a vector a thread
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)a.rows * cluster < 4 * 296 && vecs / (2 * cluster) >= kThreads) cluster *= 2;
  const dim3 grid((unsigned)a.rows * (unsigned)cluster);
  return note_launch(f ? launch_cluster(k_top_rows<float>, cluster, grid, dim3(kThreads), 0, st, a, cluster)
                       : launch_cluster(k_top_rows<bf16>, cluster, grid, dim3(kThreads), 0, st, a, cluster));
}

}  // namespace domino

using namespace domino;

extern "C" int domino_top_logits(int32_t rows, int32_t V, int64_t ld, int32_t dtype, const void* logits, int32_t k,
                                 float temperature, float* values, int32_t* ids, float* lse, domino_stream_t stream) {
  if (!rows_ok(rows, V, ld, dtype, logits) || !values || !ids) return DOMINO_ERR_INVALID_ARGUMENT;
  if (k < 1 || k > DOMINO_MAX_TOP || !temperature_ok(temperature)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (rows > DOMINO_MAX_ROWS) return DOMINO_ERR_UNSUPPORTED;
  const size_t in = rows_span(rows, V, ld, dtype), out = (size_t)rows * k * 4;
  if (overlap(logits, in, values, out) || overlap(logits, in, ids, out) || overlap(logits, in, lse, (size_t)rows * 4))
    return DOMINO_ERR_INVALID_ARGUMENT;
  TopRows a{};
  a.logits = logits;
  a.ld = ld;
  a.rows = rows;
  a.V = V;
  a.dtype = dtype;
  a.k = k;
  a.inv_t = 1.0 / (double)temperature;
  a.c = (float)(1.4426950408889634 * a.inv_t);
  a.values = values;
  a.ids = ids;
  a.lse = lse;
  return launch_top_rows(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}
