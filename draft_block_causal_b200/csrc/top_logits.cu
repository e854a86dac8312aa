// top_logits.cu -- the k largest logits of every row, in order, with the row's log-sum-exp.
//
// A row is read once, by a cluster of blocks that take contiguous slices of it.  A block walks its slice in
// tiles of kVecs 16-byte vectors a thread, the next tile's loads in flight while one is worked on: each thread
// takes its vectors' maxima, adds the tile's exponentials, and puts the values that reach a bar, and so can
// still be among the k largest, into a list in shared memory.  The bar comes from the threads' running maxima:
// a value that k threads' maxima reach has k values at or above it, and not many more than k, as a thread's
// second largest is rarely among them.  The least of the warps' j-th largest maxima, j = k / warps, is such a
// value, and takes one barrier (an exact k-th by bisection, one barrier a probe, took four times as long).  It
// is raised after 1, 3, 9, 27, ... tiles only, so that between them no thread waits for another; each such
// stretch adds about 2k values.  A value in a later tile, whose column is higher, has to exceed the bar.
// Should a stretch bring more than the list holds (ascending rows, many equal values), the exact k are selected
// from the stretch, read again, and the list.  At the end the list is cut by the bar and goes to block 0, with
// the sum, through distributed shared memory; block 0 cuts and ranks what it has got.
#include "cluster.cuh"
#include "launch.cuh"
#include "vocab_rows.cuh"
#include "vocab_rows.h"

#include <cfloat>

namespace domino {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;        // 16-byte vectors a thread and tile
constexpr int kList = 2048;     // candidates held
constexpr int kTidy = 1024;     // a list longer than this is cut by the bar before the next stretch
constexpr int kMaxCluster = 16;

// Keys a block of a cluster may hand to block 0: k or more, and kList of all blocks together.
__host__ __device__ constexpr int share_bits(int cluster) { return cluster > 8 ? 7 : 8; }

struct TopShared {
  alignas(16) uint64_t list[kList + 1];
  double sum[kMaxCluster];    // block 0: every block's sum ...
  float ref[kMaxCluster][2];  // ... its reference and maximum
  double red_s[kWarps];
  float red_n[kWarps], red_m[kWarps];
  uint32_t red_u[kWarps];
  int red_i[kWarps];
  int count;
  int handed[kMaxCluster];    // block 0: keys of every block
  uint32_t bars[kMaxCluster]; // block 0: every block's bar
};

// The least float of order o or more; the orders below -FLT_MAX's are no floats'.
__device__ __forceinline__ float floor_at(uint32_t o) { return order_value(max(o, 0x00800000u)); }

// The vector at column v of a row of V with the columns from V on barred.
template <typename T>
__device__ __forceinline__ uint4 cut_vec(uint4 q, int v, int V) {
  T* e = reinterpret_cast<T*>(&q);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i)
    if (v + i >= V) e[i] = static_cast<T>(-INFINITY);
  return q;
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

constexpr int kSlots = kList / kThreads;

// An order that at least k of the threads' orders o (0: none) reach.  `warps`: the warps to look at, all of whose
// lanes take part, warps * 32 >= k.  Where one has too few values the result is 0, which all reach.
__device__ __forceinline__ uint32_t reached_by(uint32_t o, int warps, int k, TopShared& sh) {
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t top = 0xffffffffu;
  if (wid < warps) {
    top = __reduce_max_sync(0xffffffffu, o);
    for (int j = (k + warps - 1) / warps; j > 1; --j) {
      if (lane == __ffs(__ballot_sync(0xffffffffu, o == top)) - 1) o = 0;  // one lane takes it out
      top = __reduce_max_sync(0xffffffffu, o);
    }
  }
  __syncthreads();  // an earlier result has been read
  if (lane == 0) sh.red_u[wid] = top;
  __syncthreads();
  uint32_t r = sh.red_u[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) r = min(r, sh.red_u[w]);
  return r;
}

__device__ __forceinline__ uint32_t order_bits(uint64_t key) { return (uint32_t)(key >> 32); }

// Cuts the list's n keys to those of order `bar` or more; returns how many.  Ends with a barrier.
__device__ __forceinline__ int cut_list(TopShared& sh, int n, uint32_t bar) {
  uint64_t key[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int at = threadIdx.x + i * kThreads;
    key[i] = at < n ? sh.list[at] : 0;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (key[i] != 0 && order_bits(key[i]) >= bar) sh.list[atomicAdd(&sh.count, 1)] = key[i];
  __syncthreads();
  return sh.count;
}

// f(key, rank) for each of the list's n keys below rank k.
template <typename F>
__device__ __forceinline__ void rank_list(TopShared& sh, int n, int k, F f) {
  if (threadIdx.x == 0) sh.list[n] = 0;  // pairs of keys are read at once
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const uint64_t own = sh.list[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; j += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(sh.list + j);
      rank += (two.x > own) + (two.y > own);
    }
    if (rank < k) f(own, rank);
  }
}

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
// Returns the order of the least value kept.
template <typename T>
__device__ __noinline__ uint32_t select_exact(const T* row, int t0, int t1, int V, int held, int k, TopShared& sh) {
  uint64_t own[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
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
    for (int i = 0; i < kSlots; ++i) f(own[i]);
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
  return (uint32_t)(lo >> 32);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_top_rows(TopRows a, int cluster) {
  constexpr int N = Vec<T>::N;
  __shared__ TopShared sh;
  extern __shared__ uint64_t handed[];  // block 0: [cluster][1 << share_bits(cluster)] keys
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
  constexpr int kTile = kThreads * kVecs;
  auto load = [&](uint4(&q)[kVecs], int t0) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int vec = t0 + i * kThreads + tid;
      q[i] = vec < last ? __ldcs(reinterpret_cast<const uint4*>(row) + vec) : barred_vec<T>();
    }
    if (a.V % N != 0 && t0 + kTile >= all) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) q[i] = cut_vec<T>(q[i], (t0 + i * kThreads + tid) * N, a.V);
    }
  };
  const int warps = min(last - first, kThreads) / 32;  // warps with a vector in every lane
  const bool can_bar = warps * 32 >= a.k;
  ExpSum acc;
  float m = -INFINITY;
  uint32_t bar = 0;        // an order that k values so far reach
  float floor = -FLT_MAX;  // values from here on go to the list
  uint4 next[kVecs];
  load(next, first);
  int held = 0, before = 0, from = first, stop = first + kTile, stretch = 2 * kTile;
  for (int t0 = first; t0 < last;) {
    for (; t0 < min(stop, last); t0 += kTile) {
      uint4 q[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) q[i] = next[i];
      load(next, t0 + kTile);
      float vm[kVecs], tm = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        vm[i] = fmaxf(vec_max(q[i], T()), -INFINITY);
        tm = fmaxf(tm, vm[i]);
      }
      m = fmaxf(m, tm);
      add_vectors<T>(acc, q, tm, a.c);
      if (bar == 0 && can_bar) {  // no bar yet: this tile's columns may be the lowest that reach it
        bar = reached_by(order_of(m), warps, a.k, sh);
        floor = floor_at(bar);
      }
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
    }
    __syncthreads();
    held = sh.count;
    if (held > kList) {
      bar = max(bar, select_exact(row, from, min(t0, last), a.V, before, a.k, sh));
      held = a.k;
    } else if (can_bar) {
      bar = max(bar, reached_by(order_of(m), warps, a.k, sh));
    }
    if (held > kTidy) held = cut_list(sh, held, bar);
    if (bar) floor = floor_at(bar + 1);
    before = held;
    from = t0;
    stop = t0 + stretch;
    stretch *= 3;
    __syncthreads();  // every thread has read the count before the next values come
  }
  double sum = 0.0;
  float ref = -INFINITY, most = -INFINITY;
  join_threads(acc, m, sh, &sum, &ref, &most);
  held = cut_list(sh, held, bar);
  if (cluster > 1) {
    const int bits = share_bits(cluster), share = 1 << bits;
    if (held > share) {  // many equal values at the bar: the k largest alone
      uint64_t own[kSlots];
      int at[kSlots];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) at[i] = kList;
      int i = 0;
      rank_list(sh, held, a.k, [&](uint64_t key, int rk) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (j == i) { own[j] = key; at[j] = rk; }
        ++i;
      });
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (at[j] < kList) sh.list[at[j]] = own[j];
      held = a.k;
      __syncthreads();
    }
    cluster_wait();
    const uint32_t to = cluster_address(handed + rank * share, 0);
    for (int i = tid; i < held; i += kThreads) cluster_store(to + 8 * i, sh.list[i]);
    if (tid == 0) {
      cluster_store(cluster_address(&sh.sum[rank], 0), sum);
      cluster_store(cluster_address(&sh.ref[rank], 0), ref, most);
      cluster_store(cluster_address(&sh.handed[rank], 0), held);
      cluster_store(cluster_address(&sh.bars[rank], 0), (int)bar);
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    // block 0: every block's keys that reach the highest of the blocks' bars, into its list
    if (tid == 0) sh.count = 0;
    bar = 0;
    for (int c = 0; c < cluster; ++c) bar = max(bar, sh.bars[c]);
    __syncthreads();
    for (int i = tid; i < cluster * share; i += kThreads)
      if ((i & (share - 1)) < sh.handed[i >> bits] && order_bits(handed[i]) >= bar) sh.list[atomicAdd(&sh.count, 1)] = handed[i];
    __syncthreads();
    held = sh.count;
    if (tid == 0) {
      for (int c = 1; c < cluster; ++c) {
        ref = fmaxf(ref, sh.ref[c][0]);
        most = fmaxf(most, sh.ref[c][1]);
      }
      sum = 0.0;
      for (int c = 0; c < cluster; ++c)
        if (sh.ref[c][0] > -INFINITY) sum += sh.sum[c] * (double)ex2(sh.ref[c][0] - ref);
    }
  }
  float* const values = a.values + (size_t)r * a.k;
  int32_t* const ids = a.ids + (size_t)r * a.k;
  rank_list(sh, held, a.k, [&](uint64_t key, int rk) {
    values[rk] = order_value(order_bits(key));
    ids[rk] = key_index(key);
  });
  for (int i = held + tid; i < a.k; i += kThreads) {
    values[i] = -INFINITY;
    ids[i] = -1;
  }
  if (tid == 0) {
    const double lse = log_sum_exp(sum, ref, most, a.c, a.inv_t);
    if (a.lse) a.lse[r] = (float)lse;
    if (a.lse64) a.lse64[r] = lse;
  }
}

}  // namespace

cudaError_t launch_top_rows(const TopRows& a, cudaStream_t st) {
  const bool f = a.dtype == DOMINO_DTYPE_F32;
  const int vecs = (a.V + (f ? 3 : 7)) / (f ? 4 : 8);
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)a.rows * cluster < 4 * 148 && vecs / (2 * cluster) >= 2 * kThreads) cluster *= 2;
  const dim3 grid((unsigned)a.rows * (unsigned)cluster);
  const size_t smem = cluster > 1 ? ((size_t)cluster << share_bits(cluster)) * sizeof(uint64_t) : 0;
  return note_launch(f ? launch_cluster(k_top_rows<float>, cluster, grid, dim3(kThreads), smem, st, a, cluster)
                       : launch_cluster(k_top_rows<bf16>, cluster, grid, dim3(kThreads), smem, st, a, cluster));
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
