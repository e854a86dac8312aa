// beam.cu -- one step of beam search: the best continuations over a group's beams and the vocabulary, and
// the beams' states and histories reordered to follow their parents.
//
// Only a beam's W_out best tokens can be among the group's W_out best continuations.  For few logits a group is one
// cluster (k_beam_select): each beam's row goes to `parts` of its blocks (or two rows to each of 16, for more than
// 16 beams), which leave its candidates and its sum of exponentials (top_scan.cuh) with block 0; block 0 forms the
// scores and ranks them; all blocks copy the states.  For many, the row scan of top_logits.cu leaves the candidates
// in the workspace, and k_beam_merge ranks them: a group is read by more blocks than 16, and none waits for the
// ranking.  Scores are compared in 64 bits: two beams' candidates can lie closer together than one rounding of a
// score of tens to fp32 (2^-19).
//
// Bound by the read of the logits, and in small calls by the caller's thread: 32 groups of 8 beams of 151936 fp32
// take 38 us for 158 MB (65 in one kernel); one group of 4 such beams takes 17 us in one kernel and 13 in two, but a
// caller gets a step each 21 us with one launch and no workspace, and each 26 us with two.
#include "launch.cuh"
#include "top_scan.cuh"
#include "vocab_rows.h"

#include <algorithm>

namespace domino {

namespace {

constexpr int kMaxBeams = DOMINO_MAX_BEAMS;

// Order-preserving map of a score onto 64 bits.
__device__ __forceinline__ uint64_t score_order(double s) {
  const uint64_t u = (uint64_t)__double_as_longlong(s + 0.0);  // -0 becomes +0
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ double score_value(uint64_t o) {
  return __longlong_as_double((long long)((o >> 63) ? (o & ~(1ull << 63)) : ~o));
}

// Block 0's: the group's best continuations.
struct Chosen {
  int parent[kMaxBeams], token[kMaxBeams];
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_beam_select(domino_beam_t p, int cluster, int parts, float c) {
  constexpr int N = Vec<T>::N;
  __shared__ TopShared sh;
  __shared__ Given given[kMaxBeams];    // block 0: every row part's
  __shared__ double lse[kMaxBeams];
  __shared__ uint32_t bars[kMaxBeams];  // block 0: every beam's bar
  __shared__ Chosen chosen;
  extern __shared__ uint64_t handed[];  // block 0: [W_in * parts][1 << bits] keys
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x / cluster, tid = threadIdx.x;
  const uint32_t rank = blockIdx.x % cluster;
  const int givers = p.W_in * parts, bits = share_bits(givers), share = 1 << bits;
  const float* const scores = p.scores + (size_t)g * p.W_in;
  const uint8_t* const finished = p.finished ? p.finished + (size_t)g * p.W_in : nullptr;
  const int all = (p.V + N - 1) / N, per = (all + parts - 1) / parts;
  cluster_arrive_relaxed();  // block 0 has started before another stores into it
  bool waited = false;
  for (int at = rank; at < givers; at += cluster) {  // once, or twice for more than 16 beams
    const int w = at / parts, part = at % parts;
    Given own{0.0, -INFINITY, -INFINITY, 0, 0};
    if (scores[w] > -INFINITY && !(finished && finished[w])) {
      const T* row = static_cast<const T*>(p.logits) + ((size_t)g * p.W_in + w) * p.ld;
      const int first = min(part * per, all), last = min(first + per, all);
      ExpSum acc;
      float m = -INFINITY;
      uint32_t bar = 0;
      __syncthreads();  // the list is free
      if (tid == 0) sh.count = sh.noted = 0;
      __syncthreads();
      own.n = scan_slice(row, first, last, p.V, p.W_out, c, sh, acc, m, bar);
      join_threads(acc, m, sh, own);
      own.n = limit_list(sh, own.n, share, p.W_out);
      own.bar = (int)bar;
    }
    if (!waited) cluster_wait();
    waited = true;
    const uint32_t to = cluster_address(handed + (at << bits), 0);
    for (int i = tid; i < own.n; i += kThreads) cluster_store(to + 8 * i, sh.list[i]);
    if (tid == 0) hand_over(&given[at], 0, own);
  }
  cluster_arrive();
  cluster_wait();
  if (rank == 0) {
    if (tid == 0) sh.count = 0;
    if (tid < p.W_in) {
      const Given* row = given + tid * parts;
      const Given t = join_given(row, parts);
      lse[tid] = log_sum_exp(t.sum, t.ref, t.most, c, 1.0);
      uint32_t bar = 0;
      for (int i = 0; i < parts; ++i) bar = max(bar, (uint32_t)row[i].bar);
      bars[tid] = bar;
    }
    if (tid < kMaxBeams) {
      chosen.parent[tid] = -1;
      chosen.token[tid] = 0;
    }
    __syncthreads();
    // the candidates, by score, and where each was handed; a finished beam is one of its own
    for (int i = tid; i < givers << bits; i += kThreads) {
      const int at = i >> bits, w = at / parts;
      if ((i & (share - 1)) >= given[at].n) continue;
      const uint64_t key = handed[i];
      if (order_bits(key) < bars[w]) continue;
      const int to = atomicAdd(&sh.count, 1);
      sh.list[to] = score_order((double)scores[w] + ((double)big_clamp(order_value(order_bits(key))) - lse[w]));
      sh.from[to] = (uint16_t)i;
    }
    if (tid < p.W_in && finished && finished[tid] && scores[tid] > -INFINITY) {
      const int to = atomicAdd(&sh.count, 1);  // its blocks have handed nothing: there is room
      sh.list[to] = score_order((double)scores[tid]);
      sh.from[to] = (uint16_t)(0x8000 | tid);
    }
    __syncthreads();
    int n = sh.count;
    if (n > p.W_out + p.W_out / 2 + 32) {  // those that reach what W_out of them reach, by their high 32 bits
      uint64_t sc[kSlots];
      uint16_t at[kSlots];
      uint32_t o = 0;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int j = slot(i);
        sc[i] = j < n ? sh.list[j] : 0;
        at[i] = j < n ? sh.from[j] : 0;
        o = max(o, order_bits(sc[i]));
      }
      const uint32_t bar = reached_by(o, min(n, kThreads) / 32, p.W_out, sh);
      if (tid == 0) sh.count = 0;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (sc[i] != 0 && order_bits(sc[i]) >= bar) {
          const int to = atomicAdd(&sh.count, 1);
          sh.list[to] = sc[i];
          sh.from[to] = at[i];
        }
      __syncthreads();
      n = sh.count;
    }
    // score, then the lower beam, then the larger logit, then the lower token
    auto beam_of = [&](uint32_t at) { return at & 0x8000u ? (int)(at & 0x7fffu) : (int)(at >> bits) / parts; };
    for (int i = tid; i < n; i += kThreads) {
      const uint64_t sc = sh.list[i];
      const uint32_t at = sh.from[i];
      const int w = beam_of(at);
      int place = 0;
      for (int j = 0; j < n; ++j) {
        const uint64_t other = sh.list[j];
        if (other > sc) ++place;
        else if (other == sc && j != i) {
          const uint32_t oat = sh.from[j];
          const int ow = beam_of(oat);
          place += ow < w || (ow == w && handed[oat] > handed[at]);
        }
      }
      if (place < p.W_out) {
        const size_t to = (size_t)g * p.W_out + place;
        const int token = at & 0x8000u ? p.eos : key_index(handed[at]);
        chosen.parent[place] = w;
        chosen.token[place] = token;
        p.scores_out[to] = (float)score_value(sc);
        p.parents_out[to] = w;
        p.tokens_out[to] = token;
        if (p.finished_out) p.finished_out[to] = (finished && finished[w]) || token == p.eos;
      }
    }
    __syncthreads();
    if (tid < p.W_out && chosen.parent[tid] < 0) {  // fewer continuations than beams
      const size_t to = (size_t)g * p.W_out + tid;
      p.scores_out[to] = -INFINITY;
      p.parents_out[to] = 0;
      p.tokens_out[to] = 0;
      if (p.finished_out) p.finished_out[to] = 0;
      chosen.parent[tid] = 0;
    }
    __syncthreads();
    for (int i = tid; i < cluster * p.W_out; i += kThreads) {
      const int block = i / p.W_out, w = i % p.W_out;
      if (block == 0) continue;
      cluster_store(cluster_address(&chosen.parent[w], block), chosen.parent[w]);
      cluster_store(cluster_address(&chosen.token[w], block), chosen.token[w]);
    }
  }
  cluster_arrive();
  cluster_wait();
  if (p.states) {  // rows of Hs / 4 vectors, the group's as one run
    const int vecs = p.Hs / 4, run = p.W_out * vecs;
    const float4* from = reinterpret_cast<const float4*>(p.states) + (size_t)g * p.W_in * vecs;
    float4* to = reinterpret_cast<float4*>(p.states_out) + (size_t)g * run;
#pragma unroll 4
    for (int i = rank * kThreads + tid; i < run; i += cluster * kThreads) {
      const int w = i / vecs;
      to[i] = __ldcs(from + (size_t)chosen.parent[w] * vecs + (i - w * vecs));
    }
  }
  if (p.history) {
    const int run = p.W_out * p.hist_len;
    for (int i = rank * kThreads + tid; i < run; i += cluster * kThreads) {
      const int w = i / p.hist_len, at = i - w * p.hist_len;
      const size_t from = ((size_t)g * p.W_in + chosen.parent[w]) * p.hist_len;
      p.history_out[(size_t)g * run + i] = at == p.pos ? chosen.token[w] : p.history[from + at];
    }
  }
}

struct BeamArgs {
  domino_beam_t b;
  const float* values;   // [B * W_in][W_out] the rows' largest logits
  const int32_t* ids;
  const double* lse;     // [B * W_in]
};

// One group by `splits` blocks: each ranks the group's candidates, one a thread, and takes its share of the state rows
// to copy.  A candidate's rank is what lies before it in its own beam's list, which is in order, and in each other's,
// found by binary search: a chain of up to 155 reads, so that a thread has no second one (a step of two groups of 32
// beams of 100000 fp32 that go on to 32: 35 us with 1024 threads, 54 with 256 of four candidates).
template <int kMergeThreads>
__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(BeamArgs a, int splits) {
  __shared__ double score[kMergeThreads];  // W_in * W_out of them
  __shared__ int parent_s[kMaxBeams], token_s[kMaxBeams];
  const domino_beam_t& p = a.b;
  const int g = blockIdx.x / splits, split = blockIdx.x % splits, tid = threadIdx.x, n = p.W_in * p.W_out;
  // the states on their way to L2 while the row scan's last blocks run
  if (p.states) {
    const char* from = reinterpret_cast<const char*>(p.states + (size_t)g * p.W_in * p.Hs);
    const size_t bytes = (size_t)p.W_in * p.Hs * sizeof(float);
    for (size_t i = (size_t)(split * kMergeThreads + tid) * 128; i < bytes; i += (size_t)splits * kMergeThreads * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
  }
  pdl_wait();
  pdl_trigger();
  if (tid < p.W_out) { parent_s[tid] = -1; token_s[tid] = 0; }
  const int w = tid / p.W_out;
  double sc = -INFINITY;
  int token = 0;
  if (tid < n) {
    const size_t r = (size_t)g * p.W_in + w;
    const float cum = p.scores[r];
    const bool ended = p.finished && p.finished[r];
    const int k = tid - w * p.W_out;
    // a dead or finished beam's candidates were not written: read, and not used
    const float z = a.values[r * p.W_out + k];
    const int id = a.ids[r * p.W_out + k];
    const double lse = a.lse[r];
    if (cum > -INFINITY) {
      if (!ended && id >= 0) sc = (double)cum + ((double)big_clamp(z) - lse);
      if (ended && k == 0) sc = (double)cum;
    }
    token = ended ? p.eos : id;
    score[tid] = sc;
  }
  __syncthreads();
  if (sc > -INFINITY) {
    int rank = tid - w * p.W_out;
    for (int o = 0; o < p.W_in && rank < p.W_out; ++o) {
      if (o == w) continue;
      int lo = 0, hi = p.W_out;  // before lo they come first, from hi on they do not
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        const double other = score[o * p.W_out + mid];
        if (other > sc || (other == sc && o < w)) lo = mid + 1;
        else hi = mid;
      }
      rank += lo;
    }
    if (rank < p.W_out) {
      parent_s[rank] = w;
      token_s[rank] = token;
      if (split == 0) {
        const size_t at = (size_t)g * p.W_out + rank;
        p.scores_out[at] = (float)sc;
        p.parents_out[at] = w;
        p.tokens_out[at] = token;
        if (p.finished_out)
          p.finished_out[at] = (p.finished && p.finished[(size_t)g * p.W_in + w]) || token == p.eos;
      }
    }
  }
  __syncthreads();
  if (split == 0 && tid < p.W_out && parent_s[tid] < 0) {
    const size_t at = (size_t)g * p.W_out + tid;
    p.scores_out[at] = -INFINITY;
    p.parents_out[at] = 0;
    p.tokens_out[at] = 0;
    if (p.finished_out) p.finished_out[at] = 0;
  }
  if (p.states) {  // rows of Hs / 4 vectors, the group's as one run
    const int per = p.Hs / 4, all = p.W_out * per;
    const float4* from = reinterpret_cast<const float4*>(p.states) + (size_t)g * p.W_in * per;
    float4* to = reinterpret_cast<float4*>(p.states_out) + (size_t)g * all;
#pragma unroll 4
    for (int i = split * kMergeThreads + tid; i < all; i += splits * kMergeThreads) {
      const int w = i / per;
      to[i] = __ldcs(from + (size_t)max(parent_s[w], 0) * per + (i - w * per));
    }
  }
  if (p.history && split == splits - 1) {
    const int all = p.W_out * p.hist_len;
    for (int i = tid; i < all; i += kMergeThreads) {
      const int w = i / p.hist_len, at = i - w * p.hist_len;
      const size_t from = ((size_t)g * p.W_in + max(parent_s[w], 0)) * p.hist_len;
      p.history_out[(size_t)g * all + i] = at == p.pos ? token_s[w] : p.history[from + at];
    }
  }
}

inline size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

struct BeamLayout {
  size_t values, ids, lse, bytes;
};
BeamLayout beam_layout(int64_t B, int W_in, int W_out) {
  const size_t rows = (size_t)B * W_in;
  BeamLayout l{};
  l.values = 0;
  l.ids = al256(rows * W_out * sizeof(float));
  l.lse = l.ids + al256(rows * W_out * sizeof(int32_t));
  l.bytes = l.lse + al256(rows * sizeof(double));
  return l;
}

// A group's cluster in k_beam_select: the most parts a row with which all blocks run at once, four an SM, a cluster
// has room and a thread two vectors.  `fits`: whether k_beam_select takes the call, which it does where a step takes
// less than the 26 us that a caller's thread needs for the two kernels' launches and workspace: with up to 20 MB and
// 16384 vectors a block.  A step, in one kernel and in two: 1 x 4 beams of 151936 fp32 20 and 26 us, 64 x 1 of 151936
// bf16 24 and 27, 16 x 4 23 and 26; beyond, 1 x 13 of 151936 fp32 33 and 26, 32 x 8 of 32000 33 and 26.
struct BeamSplit {
  int parts, cluster;
  bool fits;
};
BeamSplit beam_split(int64_t rows, int W_in, int V, int dtype) {
  const int n = dtype == DOMINO_DTYPE_F32 ? 4 : 8, vecs = (V + n - 1) / n;
  BeamSplit s{1, 0, false};
  while (2 * s.parts * W_in <= kMaxCluster && 2 * s.parts * rows <= 4 * 148 && vecs / (2 * s.parts) >= 2 * kThreads)
    s.parts *= 2;
  s.cluster = std::min(W_in * s.parts, kMaxCluster);
  const int64_t block = (int64_t)((vecs + s.parts - 1) / s.parts) * ((W_in * s.parts + s.cluster - 1) / s.cluster);
  s.fits = rows * vecs <= (5 << 18) && block <= 16384;
  return s;
}

bool beams_ok(int32_t B, int32_t W_in, int32_t W_out) {
  return B >= 1 && W_in >= 1 && W_out >= 1 && W_in <= kMaxBeams && W_out <= kMaxBeams;
}

}  // namespace

}  // namespace domino

using namespace domino;

extern "C" size_t domino_beam_workspace_bytes(int32_t B, int32_t W_in, int32_t W_out, int32_t V, int32_t dtype) {
  if (!beams_ok(B, W_in, W_out) || V < 1 || V > DOMINO_MAX_V) return 0;
  if ((int64_t)B * std::max(W_in, W_out) > DOMINO_MAX_ROWS) return 0;
  if (beam_split((int64_t)B * W_in, W_in, V, dtype).fits) return 0;
  return beam_layout(B, W_in, W_out).bytes;
}

extern "C" int domino_beam_select(const domino_beam_t* beam, void* workspace, size_t workspace_bytes,
                                  domino_stream_t stream) {
  auto a16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  if (!beam) return DOMINO_ERR_INVALID_ARGUMENT;
  const domino_beam_t& p = *beam;
  if (!beams_ok(p.B, p.W_in, p.W_out)) return DOMINO_ERR_INVALID_ARGUMENT;
  const int64_t rows = (int64_t)p.B * p.W_in, outs = (int64_t)p.B * p.W_out;
  if (!rows_ok(rows, p.V, p.ld, p.dtype, p.logits)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (!p.scores || !p.scores_out || !p.parents_out || !p.tokens_out) return DOMINO_ERR_INVALID_ARGUMENT;
  for (const void* q : {(const void*)p.scores, (const void*)p.scores_out, (const void*)p.parents_out,
                        (const void*)p.tokens_out, (const void*)p.history, (const void*)p.history_out})
    if (!aligned4(q)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (p.eos < -1 || p.eos >= p.V || (p.finished && (p.eos < 0 || !p.finished_out)) || (p.finished_out && p.eos < 0))
    return DOMINO_ERR_INVALID_ARGUMENT;
  if (!p.states != !p.states_out || !p.history != !p.history_out) return DOMINO_ERR_INVALID_ARGUMENT;
  if (p.states && (p.Hs < 4 || p.Hs % 4 || !a16(p.states) || !a16(p.states_out))) return DOMINO_ERR_INVALID_ARGUMENT;
  if (p.history && (p.hist_len < 1 || p.pos < 0 || p.pos >= p.hist_len)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (rows > DOMINO_MAX_ROWS || outs > DOMINO_MAX_ROWS) return DOMINO_ERR_UNSUPPORTED;
  if ((p.states && p.Hs > (1 << 20)) || (p.history && p.hist_len > (1 << 20))) return DOMINO_ERR_UNSUPPORTED;
  const BeamSplit split = beam_split(rows, p.W_in, p.V, p.dtype);
  const bool one = split.fits;
  const BeamLayout lay = one ? BeamLayout{} : beam_layout(p.B, p.W_in, p.W_out);
  if (!one && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < lay.bytes))
    return DOMINO_ERR_WORKSPACE;
  // what is read while the outputs are written, by other blocks too, may not be an output
  const size_t outs4 = (size_t)outs * 4;
  if (!disjoint({{p.scores_out, outs4}, {p.parents_out, outs4}, {p.tokens_out, outs4}, {p.finished_out, (size_t)outs},
                 {p.states_out, outs4 * p.Hs}, {p.history_out, outs4 * p.hist_len}},
                {{p.logits, rows_span(rows, p.V, p.ld, p.dtype)}, {p.scores, (size_t)rows * 4},
                 {p.finished, (size_t)rows}, {p.states, (size_t)rows * p.Hs * 4},
                 {p.history, (size_t)rows * p.hist_len * 4}, {one ? nullptr : workspace, lay.bytes}}))
    return DOMINO_ERR_INVALID_ARGUMENT;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (!one) {
    char* ws = static_cast<char*>(workspace);
    TopRows t{};
    t.logits = p.logits;
    t.ld = p.ld;
    t.rows = (int)rows;
    t.V = p.V;
    t.dtype = p.dtype;
    t.k = p.W_out;
    t.inv_t = 1.0;
    t.c = 1.44269504f;
    t.scores = p.scores;
    t.finished = p.finished;
    t.values = reinterpret_cast<float*>(ws + lay.values);
    t.ids = reinterpret_cast<int32_t*>(ws + lay.ids);
    t.lse64 = reinterpret_cast<double*>(ws + lay.lse);
    const BeamArgs a{p, t.values, t.ids, t.lse64};
    // blocks a group: about 4 vectors of the states a thread
    const int threads = p.W_in * p.W_out <= 256 ? 256 : 1024;
    const int splits = p.states ? std::max(1, std::min(8, p.W_out * p.Hs / (16 * threads))) : 1;
    auto kern = threads == 256 ? k_beam_merge<256> : k_beam_merge<1024>;
    cudaError_t e = launch_top_rows(t, cs);
    if (e == cudaSuccess)
      e = note_launch(launch_pdl(kern, dim3((unsigned)(p.B * splits)), dim3(threads), 0, cs, a, splits));
    return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
  }
  const int parts = split.parts, cluster = split.cluster, givers = p.W_in * parts;
  const size_t smem = ((size_t)givers << share_bits(givers)) * sizeof(uint64_t);
  auto kern = p.dtype == DOMINO_DTYPE_F32 ? k_beam_select<float> : k_beam_select<bf16>;
  // with the static part more than a block has by default; the same for all calls, of several host threads too
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kList * sizeof(uint64_t));
  if (e == cudaSuccess)
    e = note_launch(launch_cluster(kern, cluster, dim3((unsigned)p.B * (unsigned)cluster), dim3(kThreads), smem,
                                   cs, p, cluster, parts, 1.44269504f));
  return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}
