// distill.cu -- distillation of rows of logits from a teacher's top logits: loss, and gradient.
//
// With x = z / T, L = log sum exp(x) over the row and L_rest the same over the tokens that are no entry, a
// row's loss is   w * (sum_k p_k (log p_k - x_k + L) + rho (log rho - L_rest + L))
// and its gradient   w / T * (P exp(x_v - L) - p_v)  at an entry's token,
//                    w / T * (P exp(L_rest - L) - rho) * exp(x_v - L_rest)  elsewhere.
// The row is summed without the entries' columns (one bit per column says which they are), about its own
// reference, and the at most 128 entries' terms are added in 64 bits: S_rest as S less the entries' terms
// would be lost for a student that puts all but 1e-7 of its mass on them.  k_distill_stats takes the sums
// and the loss, one block per row; k_distill_grad writes the gradient from them.
#include "launch.cuh"
#include "vocab_rows.cuh"
#include "vocab_rows.h"

namespace domino {

namespace {

constexpr int kThreads = 512;
constexpr int kMaxK = DOMINO_MAX_TOP;

struct DistillArgs {
  domino_distill_t d;
  float c;        // log2(e) / T
  double inv_t;
  float* loss;
  float4* stats;  // two per row, see Stats
  const float* grad_loss;
  void* grad;
  int64_t grad_ld;
  int chunks;     // blocks per row of k_distill_grad
  int32_t* status;
};

// What the gradient needs of a row.  An entry's token: all * exp(x - L) - scale * p, L = l_hi + l_lo; others:
// rest * 2^(c z - n).  all = scale * P, scale = w / T, both 0 where the gradient is 0.
struct Stats {
  float n, rest, l_hi, l_lo;
  float all, scale;
};
__device__ __forceinline__ void store_stats(float4* st, int r, const Stats& s) {
  if (!st) return;
  st[2 * (size_t)r] = make_float4(s.n, s.rest, s.l_hi, s.l_lo);
  st[2 * (size_t)r + 1] = make_float4(s.all, s.scale, 0.f, 0.f);
}
__device__ __forceinline__ Stats load_stats(const float4* st, int r) {
  const float4 a = st[2 * (size_t)r], b = st[2 * (size_t)r + 1];
  return Stats{a.x, a.y, a.z, a.w, b.x, b.y};
}

// A row's entries in shared memory: tokens (-1: none), probabilities.
struct Entries {
  int32_t id[kMaxK];
  double p[kMaxK];
};

// Loads row r's entries and forms p; returns the sum of p, 0 for a row to ignore.  Every thread calls it.
__device__ __forceinline__ double load_entries(const DistillArgs& a, int r, Entries& en, double* red, bool report) {
  const domino_distill_t& d = a.d;
  const int k = threadIdx.x;
  int id = -1;
  double y = -INFINITY;
  if (k < d.K) {
    id = d.top_ids[(size_t)r * d.K + k];
    const float t = d.top_logits[(size_t)r * d.K + k];
    if (id < -1 || id >= d.V) {
      if (report && a.status) set_status(a.status, DOMINO_STATUS_BAD_TOKEN);
      id = -1;
    }
    if (id >= 0 && t > -INFINITY) y = (double)big_clamp(t) * a.inv_t;
  }
  double p = 0.0;
  if (d.teacher_lse) {
    const float lse = d.teacher_lse[r];
    if (y > -INFINITY && fabsf(lse) < INFINITY) p = exp(y - (double)lse);
  } else {
    const double m = block_reduce(y, red, MaxOp());
    if (y > -INFINITY) p = exp(y - m);
    const double sum = block_reduce(p, red, AddOp());
    if (sum > 0.0) p /= sum;
  }
  if (k < d.K) {
    en.id[k] = id;
    en.p[k] = p;
  }
  return block_reduce(p, red, AddOp());  // its barriers publish en
}

template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int v, int V, float (&z)[Vec<T>::N]) {
  widen(*reinterpret_cast<const uint4*>(row + v), z);
  if (v + Vec<T>::N > V) {
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e)
      if (v + e >= V) z[e] = -INFINITY;
  }
}

__device__ __forceinline__ float term(float z, float c, float n, bool guard) {
  return guard || !(z > -INFINITY) ? term_guarded(z, c, n) : ex2(fmaf(z, c, -n));
}

// Entry k of a row is the first of its token's.
__device__ __forceinline__ bool first_of_token(const Entries& en, int k) {
  const int id = en.id[k];
  if (id < 0) return false;
  for (int j = 0; j < k; ++j)
    if (en.id[j] == id) return false;
  return true;
}

// Loss and stats of row r from the sum s * 2^n over the tokens that are no entry (maximum m).  Every thread calls it.
template <typename T>
__device__ __forceinline__ void finish_row(const DistillArgs& a, int r, float w, double psum, const Entries& en,
                                           const T* row, float m, float n, double s, double* red) {
  const domino_distill_t& d = a.d;
  const int k = threadIdx.x;
  double x = -INFINITY;
  if (k < d.K && en.id[k] >= 0) {
    const float z = to_f32(row[en.id[k]]);
    if (z > -INFINITY) x = (double)big_clamp(z) * a.inv_t;
  }
  const double l_rest = log_sum_exp(s, n, m, a.c, a.inv_t);
  const double top = fmax(block_reduce(x, red, MaxOp()), l_rest);  // the largest of what L joins
  const double joined = block_reduce(x > -INFINITY && first_of_token(en, k) ? exp(x - top) : 0.0, red, AddOp());
  const double L = top > -INFINITY ? top + log(joined + exp(l_rest - top)) : -INFINITY;
  const double pk = k < d.K ? en.p[k] : 0.0;
  const double term = block_reduce(pk > 0.0 ? pk * (log(pk) - (x - L)) : 0.0, red, AddOp());
  if (k != 0) return;
  if (!(L > -INFINITY)) {  // no student mass
    a.loss[r] = 0.f;
    store_stats(a.stats, r, Stats{});
    return;
  }
  const bool rest = l_rest > -INFINITY;
  const double rho = d.teacher_lse && rest ? fmax(0.0, 1.0 - psum) : 0.0;
  a.loss[r] = (float)((double)w * (term + (rho > 0.0 ? rho * (log(rho) - l_rest + L) : 0.0)));
  if (a.stats) {
    const double scale = (double)w * a.inv_t, P = psum + rho;
    Stats st{};
    st.n = n;
    st.rest = rest ? (float)(scale * (P * exp(l_rest - L) - rho) / s) : 0.f;
    st.l_hi = (float)L;
    st.l_lo = (float)(L - (double)st.l_hi);
    st.all = (float)(scale * P);
    st.scale = (float)scale;
    store_stats(a.stats, r, st);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_distill_stats(DistillArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ uint32_t marks[];  // one bit per column: an entry's token
  __shared__ Entries en;
  __shared__ float redf[kThreads / 32];
  __shared__ double redd[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const domino_distill_t& d = a.d;
  const int r = blockIdx.x, tid = threadIdx.x;
  const float w = d.row_weights ? d.row_weights[r] : 1.f;
  const double psum = w == 0.f ? 0.0 : load_entries(a, r, en, redd, true);
  if (!(psum > 0.0) && !isnan(psum)) {
    if (tid == 0) {
      a.loss[r] = 0.f;
      store_stats(a.stats, r, Stats{});
    }
    return;
  }
  const T* row = static_cast<const T*>(d.logits) + (size_t)r * d.ld;
  for (int i = tid; i < (d.V + 31) / 32; i += kThreads) marks[i] = 0;
  __syncthreads();
  if (tid < d.K && en.id[tid] >= 0) atomicOr(&marks[en.id[tid] >> 5], 1u << (en.id[tid] & 31));
  float m = -INFINITY;
  for (int v = tid * N; v < d.V; v += kThreads * N) {
    float z[N];
    load_vec(row, v, d.V, z);
    const uint32_t mk = marks[v >> 5] >> (v & 31);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!((mk >> e) & 1u)) m = fmaxf(m, z[e]);
  }
  m = block_reduce(m, redf, MaxOp());
  const float n = m > -INFINITY ? reference_of(m, a.c) : 0.f;
  const bool guard = is_extreme(m);
  float sum = 0.f;
  for (int v = tid * N; v < d.V; v += kThreads * N) {
    float z[N];
    load_vec(row, v, d.V, z);
    const uint32_t mk = marks[v >> 5] >> (v & 31);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!((mk >> e) & 1u)) sum += term(z[e], a.c, n, guard);
  }
  const double s_rest = block_reduce((double)sum, redd, AddOp());
  finish_row(a, r, w, psum, en, row, m, n, s_rest, redd);
}

__device__ __forceinline__ void store_grad(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_grad(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename T, typename G>
__global__ void __launch_bounds__(kThreads) k_distill_grad(DistillArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Entries en;
  __shared__ double redd[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const domino_distill_t& d = a.d;
  const int r = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks, tid = threadIdx.x;
  const int per = ((d.V + a.chunks - 1) / a.chunks + N - 1) / N * N;
  const int v0 = min(chunk * per, d.V), v1 = min(v0 + per, d.V);
  const T* row = static_cast<const T*>(d.logits) + (size_t)r * d.ld;
  G* out = static_cast<G*>(a.grad) + (size_t)r * a.grad_ld;
  const Stats st = load_stats(a.stats, r);
  const float g = a.grad_loss ? a.grad_loss[r] : 1.f;
  if (st.scale == 0.f || g == 0.f) {
    for (int v = v0 + tid; v < v1; v += kThreads) store_grad(out + v, 0.f);
    return;
  }
  load_entries(a, r, en, redd, false);
  const bool guard = is_extreme(st.n / a.c);
  // the entries' gradients of this chunk, before the logits may be overwritten
  float own = 0.f;
  int at = -1;
  if (tid < d.K && en.id[tid] >= v0 && en.id[tid] < v1 && first_of_token(en, tid)) {
    at = en.id[tid];
    double p = 0.0;
    for (int j = 0; j < d.K; ++j)
      if (en.id[j] == at) p += en.p[j];
    const float z = to_f32(row[at]);
    const double L = (double)st.l_hi + (double)st.l_lo;
    const double q = z > -INFINITY ? exp((double)big_clamp(z) * a.inv_t - L) : 0.0;
    own = (float)((double)g * (q * (double)st.all - p * (double)st.scale));
  }
  __syncthreads();
  const float coef = g * st.rest;
  for (int v = v0 + tid * N; v < v1; v += kThreads * N) {
    float z[N];
    load_vec(row, v, d.V, z);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (v + e < v1) store_grad(out + v + e, coef * term(z[e], a.c, st.n, guard));
  }
  __syncthreads();
  if (at >= 0) store_grad(out + at, own);
}

cudaError_t launch_stats(const DistillArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)(a.d.V + 31) / 32 * 4;
  const bool f = a.d.dtype == DOMINO_DTYPE_F32;
  auto kern = f ? k_distill_stats<float> : k_distill_stats<bf16>;
  if (smem > 32 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return note_launch(launch_pdl(kern, dim3((unsigned)a.d.rows), dim3(kThreads), smem, st, a));
}

cudaError_t launch_grad(DistillArgs a, int grad_dtype, cudaStream_t st) {
  a.chunks = (a.d.V + 16383) / 16384;
  const bool f = a.d.dtype == DOMINO_DTYPE_F32, g = grad_dtype == DOMINO_DTYPE_F32;
  auto kern = f ? (g ? k_distill_grad<float, float> : k_distill_grad<float, bf16>)
                : (g ? k_distill_grad<bf16, float> : k_distill_grad<bf16, bf16>);
  return note_launch(launch_pdl(kern, dim3((unsigned)a.d.rows * (unsigned)a.chunks), dim3(kThreads), 0, st, a));
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
  cudaError_t e = launch_stats(a, cs);
  if (e == cudaSuccess && grad) e = launch_grad(a, grad_dtype, cs);
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
