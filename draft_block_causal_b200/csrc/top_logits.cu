// top_logits.cu -- the k largest logits of every row, in order, with the row's log-sum-exp.
//
// One block per row.  The first pass takes the maximum and the sum of exponentials; then the k-th largest
// value is found by bisection over the 32 bits of the order-preserving key, counting the row's values at or
// above each probe, and among values equal to it the k-th column by bisection over the columns.
#include "launch.cuh"
#include "vocab_rows.cuh"
#include "vocab_rows.h"

namespace domino {

namespace {

constexpr int kThreads = 512;

// One vector of a row, columns from V on as -infinity.
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int v, int V, float (&z)[Vec<T>::N]) {
  widen(__ldg(reinterpret_cast<const uint4*>(row + v)), z);
  if (v + Vec<T>::N > V) {
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e)
      if (v + e >= V) z[e] = -INFINITY;
  }
}

template <typename T, typename F>
__device__ __forceinline__ int count_row(const T* row, int V, int* red, F pred) {
  int n = 0;
  for (int v = threadIdx.x * Vec<T>::N; v < V; v += kThreads * Vec<T>::N) {
    float z[Vec<T>::N];
    load_vec(row, v, V, z);
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) n += pred(order_of(z[e]), v + e) ? 1 : 0;
  }
  return block_reduce(n, red, AddOp());
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_top_rows(TopRows a) {
  constexpr int N = Vec<T>::N;
  __shared__ float redf[kThreads / 32];
  __shared__ double redd[kThreads / 32];
  __shared__ int redi[kThreads / 32];
  __shared__ uint64_t keys[DOMINO_MAX_TOP];
  __shared__ int found;
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  if ((a.scores && !(a.scores[r] > -INFINITY)) || (a.finished && a.finished[r])) return;
  const T* row = static_cast<const T*>(a.logits) + (size_t)r * a.ld;
  float m = -INFINITY;
  for (int v = threadIdx.x * N; v < a.V; v += kThreads * N) {
    float z[N];
    load_vec(row, v, a.V, z);
#pragma unroll
    for (int e = 0; e < N; ++e) m = fmaxf(m, z[e]);
  }
  m = block_reduce(m, redf, MaxOp());
  const float n = m > -INFINITY ? reference_of(m, a.c) : 0.f;
  float s = 0.f;
  for (int v = threadIdx.x * N; v < a.V; v += kThreads * N) {
    float z[N];
    load_vec(row, v, a.V, z);
#pragma unroll
    for (int e = 0; e < N; ++e) s += term_guarded(z[e], a.c, n);
  }
  const double sum = block_reduce((double)s, redd, AddOp());
  if (threadIdx.x == 0) {
    const double lse = log_sum_exp(sum, n, m, a.c, a.inv_t);
    if (a.lse) a.lse[r] = (float)lse;
    if (a.lse64) a.lse64[r] = lse;
    found = 0;
  }
  const int have = count_row(row, a.V, redi, [](uint32_t o, int) { return o != 0; });
  const int k = min(a.k, have);
  uint32_t lo = 0;  // the largest value with at least k at or above it
  int last = a.V - 1;
  if (k > 0) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t probe = lo | (1u << bit);
      if (count_row(row, a.V, redi, [=](uint32_t o, int) { return o >= probe; }) >= k) lo = probe;
    }
    const int above = count_row(row, a.V, redi, [=](uint32_t o, int) { return o > lo; });
    int first = -1;  // fewer than k - above equal values up to here
    while (last - first > 1) {
      const int mid = first + (last - first) / 2;
      if (count_row(row, a.V, redi, [=](uint32_t o, int v) { return o == lo && v <= mid; }) >= k - above) last = mid;
      else first = mid;
    }
    for (int v = threadIdx.x * N; v < a.V; v += kThreads * N) {
      float z[N];
      load_vec(row, v, a.V, z);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t o = order_of(z[e]);
        if (o > lo || (o == lo && v + e <= last)) keys[atomicAdd(&found, 1)] = select_key(o, v + e);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.k; i += kThreads) {
    if (i < k) {
      const uint64_t key = keys[i];
      int rank = 0;
      for (int j = 0; j < k; ++j) rank += keys[j] > key;
      a.values[(size_t)r * a.k + rank] = order_value((uint32_t)(key >> 32));
      a.ids[(size_t)r * a.k + rank] = key_index(key);
    } else {
      a.values[(size_t)r * a.k + i] = -INFINITY;
      a.ids[(size_t)r * a.k + i] = -1;
    }
  }
}

}  // namespace

cudaError_t launch_top_rows(const TopRows& a, cudaStream_t st) {
  return note_launch(a.dtype == DOMINO_DTYPE_F32
                         ? launch_pdl(k_top_rows<float>, dim3((unsigned)a.rows), dim3(kThreads), 0, st, a)
                         : launch_pdl(k_top_rows<bf16>, dim3((unsigned)a.rows), dim3(kThreads), 0, st, a));
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
