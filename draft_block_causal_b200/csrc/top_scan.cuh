// top_scan.cuh -- one read of a slice of a row of logits: its sum of exponentials and the candidates for its k
// largest.  The row scan of top_logits.cu and beam.cu.
//
// A block walks its slice in tiles of kVecs 16-byte vectors a thread, the next tile's loads in flight while one is
// worked on: each thread takes its vectors' maxima, adds the tile's exponentials, and notes the vectors whose maximum
// reaches a bar, so that they can hold one of the k largest.  The bar comes from the threads' running maxima: a value
// that k threads' maxima reach has k values at or above it, and not many more than k, as a thread's second largest is
// rarely among them.  It is raised after 1, 3, 9, 27, ... tiles only, so that between them no thread waits for
// another; each such stretch notes about 2k vectors.  A value in a later tile, whose column is higher, has to exceed
// the bar.  At the end the noted vectors whose maximum reaches the last bar are read again, by all threads alike, and
// their values that reach it become the list of candidates: taking them as they are met cost three times the
// instructions, since they come one lane at a time.  Should there be more than the notes or the list hold (ascending
// rows, many equal values), the exact k are selected digit by digit from the slice.
#pragma once

#include "cluster.cuh"
#include "vocab_rows.cuh"

#include <cfloat>

namespace domino {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kVecs = 4;        // 16-byte vectors a thread and tile
constexpr int kNotes = 2048;    // vectors noted
constexpr int kList = 2048;     // candidates held
constexpr int kDigits = 2048;   // values of an 11-bit digit, in the place of the notes
constexpr int kMaxCluster = 16;

// Keys that each of `givers` may hand to block 0 of a cluster: kList of all together.
__host__ __device__ constexpr int share_bits(int givers) { return givers > 16 ? 6 : givers > 8 ? 7 : 8; }

struct TopShared {
  alignas(16) uint64_t list[kList + 1];
  union {
    uint2 notes[kNotes];        // a vector, and the order of its maximum
    uint32_t digits[kDigits];
    uint16_t from[kList];       // beam selection: where a candidate was handed
  };
  float red_s[kWarps], red_n[kWarps], red_m[kWarps];
  uint32_t red_u[kWarps];
  int count, noted;
};

// What a block hands to block 0 beside its keys: its columns' sum of exponentials, maximum, bar and number of keys.
struct Given {
  double sum;
  float ref, most;
  int n, bar;
};
__device__ __forceinline__ void hand_over(const Given* to, uint32_t block, const Given& g) {
  const uint32_t at = cluster_address(to, block);
  cluster_store(at, g.sum);
  cluster_store(at + 8, g.ref, g.most);
  cluster_store(at + 16, g.n);
  cluster_store(at + 20, g.bar);
}
// Parts of a row's sum as one.
__device__ __forceinline__ Given join_given(const Given* parts, int n) {
  Given g = parts[0];
  for (int c = 1; c < n; ++c) {
    g.ref = fmaxf(g.ref, parts[c].ref);
    g.most = fmaxf(g.most, parts[c].most);
  }
  g.sum = 0.0;
  for (int c = 0; c < n; ++c)
    if (parts[c].ref > -INFINITY) g.sum += parts[c].sum * (double)ex2(parts[c].ref - g.ref);
  return g;
}

// The least float of order o or more; the orders below -FLT_MAX's are no floats'.
__device__ __forceinline__ float floor_at(uint32_t o) { return order_value(max(o, 0x00800000u)); }

// Thread 0 gets the sum over the block's threads: in fp32 over a warp, then in 64 bits.
__device__ __forceinline__ void join_threads(const ExpSum& a, float m, TopShared& sh, Given& g) {
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
  g.sum = s;
  g.ref = n;
  g.most = m;
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
// thread looks at the largest of its share of the keys, one in kThreads, from other places in each stretch of them:
// blocks hand over lists in order, and threads that had the same place in several would leave a low bar (of 16 times
// 128 keys for k = 128 it left 520 in place of 165, and the ranking took 23000 cycles).
constexpr int kSlots = kList / kThreads;
__device__ __forceinline__ int slot(int i) { return i * kThreads + (threadIdx.x + 37 * i) % kThreads; }
__device__ __forceinline__ int cut_list(TopShared& sh, int n, int k) {
  uint64_t key[kSlots];
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int at = slot(i);
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
      for (; above + (int)sh.digits[threadIdx.x * kMine + i] < want; --i)
        above += (int)sh.digits[threadIdx.x * kMine + i];
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

// The candidates for the k largest of the vectors [first, last) of a row of V, in the list, and how many; the
// thread's sum and maximum; and `bar`, an order that k of the values reach, or 0.  Every thread calls it, with
// sh.count and sh.noted set to 0 before a barrier.
template <typename T>
__device__ __forceinline__ int scan_slice(const T* row, int first, int last, int V, int k, float c, TopShared& sh,
                                          ExpSum& acc, float& m, uint32_t& bar) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x, all = (V + N - 1) / N;
  constexpr int kTile = kThreads * kVecs;
  const int warps = min(last - first, kThreads) / 32;  // warps with a vector in every lane
  const bool can_bar = warps * 32 >= k;
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
      if (V % N != 0 && t0 + kTile >= all) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) bar_elements<T>(q[i], beyond<T>((t0 + i * kThreads + tid) * N, V));
      }
      float vm[kVecs], tm = -INFINITY;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        vm[i] = vec_max(q[i], T());
        tm = fmaxf(tm, vm[i]);
      }
      m = fmaxf(m, tm);
      add_vectors<T>(acc, q, (last - t0 + kThreads - 1) / kThreads, tm, c);
      if (bar == 0 && can_bar) {  // no bar yet: this tile's columns may be the lowest that reach it
        bar = reached_by(order_of(m), warps, k, sh);
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
      // not for two tiles or less: their notes cost less than the barriers (4000 rows of 32000 bf16, k = 8: 75 us
      // for 81)
      if (stretch > 2 * kTile && (t0 >= last || last - t0 > 2 * kTile))
        bar = max(bar, reached_by(order_of(m), warps, k, sh));
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
        if (o != 0 && o >= bar && vec * N + e < V) {
          const int to = atomicAdd(&sh.count, 1);
          if (to < kList) sh.list[to] = select_key(o, vec * N + e);
        }
      }
    }
    __syncthreads();
    held = sh.count;
    exact = held > kList;
  }
  return exact ? select_exact(row, first, last, V, k, sh) : held;
}

// Cuts a list of n > most keys to its k largest, in order.
__device__ __forceinline__ int limit_list(TopShared& sh, int n, int most, int k) {
  if (n <= most) return n;
  uint64_t own[kSlots];
  int place[kSlots], i = 0;
#pragma unroll
  for (int j = 0; j < kSlots; ++j) place[j] = kList;
  rank_list(sh, n, k, [&](uint64_t key, int rk) {
#pragma unroll
    for (int j = 0; j < kSlots; ++j)
      if (j == i) { own[j] = key; place[j] = rk; }
    ++i;
  });
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSlots; ++j)
    if (place[j] < kList) sh.list[place[j]] = own[j];
  __syncthreads();
  return k;
}

}  // namespace domino
