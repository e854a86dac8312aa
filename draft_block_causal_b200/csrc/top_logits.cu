// top_logits.cu -- the k largest logits of every row, in order, with the row's log-sum-exp.
//
// A row is read once, by a cluster of blocks that take contiguous slices of it.  A block walks its slice in
// tiles of kVecs 16-byte vectors a thread, the next tile's loads in flight while one is worked on: each thread
// takes its vectors' maxima, adds the tile's exponentials, and notes the vectors whose maximum reaches a bar, so
// that they can hold one of the k largest.  The bar comes from the threads' running maxima: a value that k
// threads' maxima reach has k values at or above it, and not many more than k, as a thread's second largest is
// rarely among them.  It is raised after 1, 3, 9, 27, ... tiles only, so that between them no thread waits for
// another; each such stretch notes about 2k vectors.  A value in a later tile, whose column is higher, has to
// exceed the bar.  At the end the noted vectors whose maximum reaches the last bar are read again, by all threads
// alike, and their values that reach it become the list of candidates: taking them as they are met cost three
// times the instructions, since they come one lane at a time.  Should there be more than the notes or the list
// hold (ascending rows, many equal values), the exact k are selected digit by digit from the slice.  The lists go
// to block 0, with the sums, through distributed shared memory; block 0 cuts them and ranks what is left.
//
// Bound by memory: 512 rows of 151936 fp32 take 51 us for k = 8 (6.1 TB/s, 93% of the measured copy rate) and 58 us
// for k = 64, whose notes and ranking come after all blocks' reads; bf16 rows by the exponentials as well, one a
// value at 16 a clock and SM (1024 rows of 151936: 62 us, 5.0 TB/s).  One row of 151936 fp32 over 16 blocks: 9 us,
// all latency.
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
constexpr int kNotes = 2048;    // vectors noted
constexpr int kList = 2048;     // candidates held
constexpr int kDigits = 2048;   // values of an 11-bit digit, in the place of the notes
constexpr int kMaxCluster = 16;

// Keys a block of a cluster may hand to block 0: k or more, and kList of all blocks together.
__host__ __device__ constexpr int share_bits(int cluster) { return cluster > 8 ? 7 : 8; }

struct TopShared {
  alignas(16) uint64_t list[kList + 1];
  union {
    uint2 notes[kNotes];        // a vector, and the order of its maximum
    uint32_t digits[kDigits];
  };
  double sum[kMaxCluster];     // block 0: every block's sum ...
  float ref[kMaxCluster][2];   // ... its reference and maximum
  float red_s[kWarps], red_n[kWarps], red_m[kWarps];
  uint32_t red_u[kWarps];
  int count, noted;
  int handed[kMaxCluster];     // block 0: keys of every block
  uint32_t bars[kMaxCluster];  // block 0: every block's bar
};

// The least float of order o or more; the orders below -FLT_MAX's are no floats'.
__device__ __forceinline__ float floor_at(uint32_t o) { return order_value(max(o, 0x00800000u)); }

// Thread 0 gets the sum over the block's threads: in fp32 over a warp, then in 64 bits.
__device__ __forceinline__ void join_threads(const ExpSum& a, float m, TopShared& sh, double* sum, float* ref, float* max) {
  float n = a.n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, o));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  const float w = warp_sum(n > -INFINITY ? a.s * ex2(a.n - n) : 0.f);
  if ((threadIdx.x & 31) == 0) {
    sh.red_n[threadIdx.x >> 5] = n;
    sh.red_m[threadIdx.x >> 5] = m;
    sh.red_s[threadIdx.x >> 5] = w;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    n = fmaxf(n, sh.red_n[w]);
    m = fmaxf(m, sh.red_m[w]);
  }
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    if (sh.red_n[w] > -INFINITY) s += (double)sh.red_s[w] * (double)ex2(sh.red_n[w] - n);
  *sum = s;
  *ref = n;
  *max = m;
}

// An order that at least k of the threads' orders o (0: none) reach, and not many more.  `warps`: the warps to look
// at, all of whose lanes take part, warps * 32 >= k.  Where one has too few values the result may be 0, which all
// reach.  The least of the warps' j-th largest, j = k / warps, is reached by k; three probes by bisection between
// it and the greatest of them bring it near the k-th.
__device__ __forceinline__ uint32_t reached_by(uint32_t o, int warps, int k, TopShared& sh) {
  const int wid = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t own = wid < warps ? o : 0;
  uint32_t top = 0;
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
  uint32_t lo = sh.red_u[0], hi = lo;
  for (int w = 1; w < warps; ++w) {
    lo = min(lo, sh.red_u[w]);
    hi = max(hi, sh.red_u[w]);
  }
#pragma unroll 1
  for (int i = 0; i < 3 && hi - lo > 1; ++i) {
    const uint32_t mid = lo + (hi - lo) / 2;
    if (__syncthreads_count(own >= mid) >= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t order_bits(uint64_t key) { return (uint32_t)(key >> 32); }

// Cuts the list's n keys to those that reach an order which k of them reach, and returns how many are left.  Every
// thread looks at the largest of its share of the keys, one in kThreads.
constexpr int kSlots = kList / kThreads;
__device__ __forceinline__ int cut_list(TopShared& sh, int n, int k) {
  uint64_t key[kSlots];
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int at = threadIdx.x + i * kThreads;
    key[i] = at < n ? sh.list[at] : 0;
    o = max(o, order_bits(key[i]));
  }
  const uint32_t bar = reached_by(o, min(n, kThreads) / 32, k, sh);
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

// f(key) of every value of the vectors [first, last) of a row; whole warps call f together, with key 0 past the end.
template <typename T, typename F>
__device__ __forceinline__ void each_key(const T* row, int first, int last, int V, F f) {
  for (int v0 = first; v0 < last; v0 += kThreads) {
    const int vec = v0 + threadIdx.x;
    float z[Vec<T>::N];
    if (vec < last) widen(__ldcg(reinterpret_cast<const uint4*>(row) + vec), z);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) {
      const int v = vec * Vec<T>::N + e;
      f(vec < last && v < V ? select_key(order_of(z[e]), v) : (uint64_t)0);
    }
  }
}

// The exact k largest of the vectors [first, last) of a row, or all if they are fewer, into the list; returns how
// many.  The keys' bits (order, then column from the highest) are fixed 11 at a time from the top: the count of
// the keys with each value of the digit says which the k-th has.
template <typename T>
__device__ __noinline__ int select_exact(const T* row, int first, int last, int V, int k, TopShared& sh) {
  uint64_t fixed = 0;  // the k-th key's bits so far
  int want = k;        // its place among the keys that share them
  for (int shift = 53; shift >= -2; shift -= 11) {  // the last digit has 9 bits
    const int bits = shift < 0 ? 9 : 11, low = shift < 0 ? 0 : shift;
    __syncthreads();
    for (int i = threadIdx.x; i < kDigits; i += kThreads) sh.digits[i] = 0;
    __syncthreads();
    each_key(row, first, last, V, [&](uint64_t key) {
      const bool in = key != 0 && (low + bits == 64 || (key >> (low + bits)) == (fixed >> (low + bits)));
      const uint32_t digit = (uint32_t)(key >> low) & ((1u << bits) - 1);
      int same;  // whole warps of one value count once
      const uint32_t all = __ballot_sync(0xffffffffu, in);
      __match_all_sync(0xffffffffu, in ? digit : 0xffffffffu, &same);
      if (same) {
        if (all && (threadIdx.x & 31) == 0) atomicAdd(&sh.digits[digit], 32u);
      } else if (in) {
        atomicAdd(&sh.digits[digit], 1u);
      }
    });
    __syncthreads();
    if (threadIdx.x == 0) sh.noted = sh.count = 0;  // fewer than k keys: all stay
    // each thread has kMine digits, and the number of keys with a digit above them
    constexpr int kMine = kDigits / kThreads;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) sum += (int)sh.digits[threadIdx.x * kMine + i];
    int from_here = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_down_sync(0xffffffffu, from_here, o);
      if ((threadIdx.x & 31) + o < 32) from_here += t;
    }
    if ((threadIdx.x & 31) == 0) sh.red_u[threadIdx.x >> 5] = (uint32_t)from_here;
    __syncthreads();
    int above = from_here - sum;
    for (int w = (threadIdx.x >> 5) + 1; w < kWarps; ++w) above += (int)sh.red_u[w];
    if (above < want && want <= above + sum) {
      int i = kMine - 1;
      for (; above + (int)sh.digits[threadIdx.x * kMine + i] < want; --i) above += (int)sh.digits[threadIdx.x * kMine + i];
      sh.noted = threadIdx.x * kMine + i;
      sh.count = above;
    }
    __syncthreads();
    fixed |= (uint64_t)sh.noted << low;
    want -= sh.count;
  }
  __syncthreads();
  if (threadIdx.x == 0) sh.count = 0;
  __syncthreads();
  each_key(row, first, last, V, [&](uint64_t key) {
    if (key != 0 && key >= fixed) sh.list[atomicAdd(&sh.count, 1)] = key;
  });
  __syncthreads();
  return sh.count;
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
  if (tid == 0) sh.count = sh.noted = 0;
  if (cluster > 1) cluster_arrive();  // block 0 has started before another stores into it
  const T* row = static_cast<const T*>(a.logits) + (size_t)r * a.ld;
  const int all = (a.V + N - 1) / N, per = (all + cluster - 1) / cluster;
  const int first = min((int)rank * per, all), last = min(first + per, all);
  constexpr int kTile = kThreads * kVecs;
  const int warps = min(last - first, kThreads) / 32;  // warps with a vector in every lane
  const bool can_bar = warps * 32 >= a.k;
  ExpSum acc;
  float m = -INFINITY;
  uint32_t bar = 0;        // an order that k values so far reach
  float floor = -FLT_MAX;  // vectors with a value from here on are noted
  const uint4* at = reinterpret_cast<const uint4*>(row) + first + tid;
  uint4 next[kVecs];
  load_tile<T, kVecs, true>(next, at, kThreads, last - first);
  int stop = first + kTile, stretch = 2 * kTile;
  for (int t0 = first; t0 < last;) {
    for (; t0 < min(stop, last); t0 += kTile) {
      uint4 q[kVecs];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) q[i] = next[i];
      at += kTile;
      load_tile<T, kVecs, true>(next, at, kThreads, last - t0 - kTile);
      if (a.V % N != 0 && t0 + kTile >= all) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) bar_elements<T>(q[i], beyond<T>((t0 + i * kThreads + tid) * N, a.V));
      }
      float vm[kVecs], tm = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        vm[i] = vec_max(q[i], T());
        tm = fmaxf(tm, vm[i]);
      }
      m = fmaxf(m, tm);
      add_vectors<T>(acc, q, (last - t0 + kThreads - 1) / kThreads, tm, a.c);
      if (bar == 0 && can_bar) {  // no bar yet: this tile's columns may be the lowest that reach it
        bar = reached_by(order_of(m), warps, a.k, sh);
        floor = floor_at(bar);
      }
      if (tm >= floor) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
          if (vm[i] >= floor) {
            const int to = atomicAdd(&sh.noted, 1);
            if (to < kNotes) sh.notes[to] = make_uint2(t0 + i * kThreads + tid, order_of(vm[i]));
          }
      }
    }
    if (can_bar) {
      if (stretch > 2 * kTile) bar = max(bar, reached_by(order_of(m), warps, a.k, sh));
      if (bar) floor = floor_at(bar + 1);
    }
    stop = t0 + stretch;
    stretch *= 3;
  }
  __syncthreads();
  int held = sh.noted;
  bool exact = held > kNotes;
  if (!exact) {
    for (int i = tid; i < held; i += kThreads) {
      const uint2 note = sh.notes[i];
      if (note.y < bar) continue;
      const int vec = (int)note.x;
      float z[N];
      widen(__ldcg(reinterpret_cast<const uint4*>(row) + vec), z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t o = order_of(z[e]);
        if (o != 0 && o >= bar && vec * N + e < a.V) {
          const int to = atomicAdd(&sh.count, 1);
          if (to < kList) sh.list[to] = select_key(o, vec * N + e);
        }
      }
    }
    __syncthreads();
    held = sh.count;
    exact = held > kList;
  }
  if (exact) held = select_exact(row, first, last, a.V, a.k, sh);
  double sum = 0.0;
  float ref = -INFINITY, most = -INFINITY;
  join_threads(acc, m, sh, &sum, &ref, &most);
  if (cluster > 1) {
    const int bits = share_bits(cluster), share = 1 << bits;
    if (held > share) {  // the k largest alone
      uint64_t own[kSlots];
      int place[kSlots];
      int i = 0;
#pragma unroll
      for (int j = 0; j < kSlots; ++j) place[j] = kList;
      rank_list(sh, held, a.k, [&](uint64_t key, int rk) {
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (j == i) { own[j] = key; place[j] = rk; }
        ++i;
      });
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (place[j] < kList) sh.list[place[j]] = own[j];
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
    // ranking takes held * held comparisons: many blocks' bars are each far below the row's
    if (held > a.k + a.k / 2 + 32) held = cut_list(sh, held, a.k);
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
  // the largest cluster with which all blocks run at once, four an SM, and a thread has two vectors
  int cluster = 1;
  while (cluster < kMaxCluster && 2 * cluster * (int64_t)a.rows <= 4 * 148 && vecs / (2 * cluster) >= 2 * kThreads) cluster *= 2;
  const dim3 grid((unsigned)a.rows * (unsigned)cluster);
  const size_t smem = cluster > 1 ? ((size_t)cluster << share_bits(cluster)) * sizeof(uint64_t) : 0;
  auto kern = f ? k_top_rows<float> : k_top_rows<bf16>;
  // with the static part more than a block has by default; the same for all calls, of several host threads too
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kList * sizeof(uint64_t));
  if (e != cudaSuccess) return e;
  return note_launch(launch_cluster(kern, cluster, grid, dim3(kThreads), smem, st, a, cluster));
}

}  // namespace domino

using namespace domino;

extern "C" int domino_top_logits(int32_t rows, int32_t V, int64_t ld, int32_t dtype, const void* logits, int32_t k,
                                 float temperature, float* values, int32_t* ids, float* lse, domino_stream_t stream) {
  if (!rows_ok(rows, V, ld, dtype, logits) || !values || !ids) return DOMINO_ERR_INVALID_ARGUMENT;
  if (k < 1 || k > DOMINO_MAX_TOP || !temperature_ok(temperature)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (rows > DOMINO_MAX_ROWS) return DOMINO_ERR_UNSUPPORTED;
  if (!aligned4(values) || !aligned4(ids) || !aligned4(lse)) return DOMINO_ERR_INVALID_ARGUMENT;
  const size_t n = (size_t)rows * k * 4;
  if (!disjoint({{values, n}, {ids, n}, {lse, (size_t)rows * 4}}, {{logits, rows_span(rows, V, ld, dtype)}}))
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
