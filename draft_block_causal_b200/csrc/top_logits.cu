// top_logits.cu -- the k largest logits of every row, in order, with the row's log-sum-exp.
//
// A row is read once, by a cluster of blocks that take contiguous slices of it (top_scan.cuh).  Their candidates go
// to block 0, with the sums, through distributed shared memory; block 0 cuts them and ranks what is left.
//
// Bound by memory: 512 rows of 151936 fp32 take 51 us for k = 8 (6.1 TB/s, 93% of the measured copy rate) and 59 us
// for k = 64, whose notes and ranking come after all blocks' reads; bf16 rows by the exponentials as well, one a
// value at 16 a clock and SM (1024 rows of 151936: 62 us, 5.0 TB/s).  One row of 151936 fp32 over 16 blocks: 9.6 us,
// all latency.
#include "launch.cuh"
#include "top_scan.cuh"
#include "vocab_rows.h"

namespace domino {

namespace {

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_top_rows(TopRows a, int cluster) {
  constexpr int N = Vec<T>::N;
  __shared__ TopShared sh;
  __shared__ Given given[kMaxCluster];  // block 0: every block's
  extern __shared__ uint64_t handed[];  // block 0: [cluster][1 << share_bits(cluster)] keys
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x / cluster, tid = threadIdx.x;
  const uint32_t rank = blockIdx.x % cluster;
  if ((a.scores && !(a.scores[r] > -INFINITY)) || (a.finished && a.finished[r])) return;  // the whole cluster
  if (tid == 0) sh.count = sh.noted = 0;
  if (cluster > 1) cluster_arrive_relaxed();  // block 0 has started before another stores into it
  const T* row = static_cast<const T*>(a.logits) + (size_t)r * a.ld;
  const int all = (a.V + N - 1) / N, per = (all + cluster - 1) / cluster;
  const int first = min((int)rank * per, all), last = min(first + per, all);
  ExpSum acc;
  float m = -INFINITY;
  uint32_t bar = 0;
  __syncthreads();
  int held = scan_slice(row, first, last, a.V, a.k, a.c, sh, acc, m, bar);
  Given g{0.0, -INFINITY, -INFINITY, 0, 0};
  join_threads(acc, m, sh, g);
  if (cluster > 1) {
    const int bits = share_bits(cluster), share = 1 << bits;
    held = limit_list(sh, held, share, a.k);
    g.n = held;
    g.bar = (int)bar;
    cluster_wait();
    const uint32_t to = cluster_address(handed + rank * share, 0);
    for (int i = tid; i < held; i += kThreads) cluster_store(to + 8 * i, sh.list[i]);
    if (tid == 0) hand_over(&given[rank], 0, g);
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;
    // block 0: every block's keys that reach the highest of the blocks' bars, into its list
    if (tid == 0) sh.count = 0;
    bar = 0;
    for (int c = 0; c < cluster; ++c) bar = max(bar, (uint32_t)given[c].bar);
    __syncthreads();
    for (int i = tid; i < cluster * share; i += kThreads)
      if ((i & (share - 1)) < given[i >> bits].n && order_bits(handed[i]) >= bar)
        sh.list[atomicAdd(&sh.count, 1)] = handed[i];
    __syncthreads();
    held = sh.count;
    // ranking takes held * held comparisons: many blocks' bars are each far below the row's
    if (held > a.k + a.k / 2 + 32) held = cut_list(sh, held, a.k);
    if (tid == 0) g = join_given(given, cluster);
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
    const double lse = log_sum_exp(g.sum, g.ref, g.most, a.c, a.inv_t);
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
  while (cluster < kMaxCluster && 2 * cluster * (int64_t)a.rows <= 4 * 148 && vecs / (2 * cluster) >= 2 * kThreads)
    cluster *= 2;
  const dim3 grid((unsigned)a.rows * (unsigned)cluster);
  const size_t smem = cluster > 1 ? ((size_t)cluster << share_bits(cluster)) * sizeof(uint64_t) : 0;
  auto kern = f ? k_top_rows<float> : k_top_rows<bf16>;
  // with the static part more than a block has by default; the same for all calls, of several host threads too
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kList * sizeof(uint64_t));
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
