// beam.cu -- one step of beam search: the best continuations over a group's beams and the vocabulary, and
// the beams' states and histories reordered to follow their parents.
//
// Only a beam's W_out best tokens can be among the group's W_out best continuations, so the row scan of
// top_logits.cu leaves W_in * W_out candidates a group (k_top_rows, one read of the logits), and k_beam_merge
// ranks them.  Scores are compared in 64 bits: two beams' candidates can lie closer together than one
// rounding of a score of tens to fp32 (2^-19).
//
// Bound by the read of the logits: 32 groups of 8 beams, fp32, take 38 us for 158 MB, the row scan 31 of them; the
// merge is a chain of three loads and a search in shared memory.
#include "launch.cuh"
#include "vocab_rows.cuh"
#include "vocab_rows.h"

#include <algorithm>

namespace domino {

namespace {

constexpr int kMergeThreads = 256;

struct BeamArgs {
  domino_beam_t b;
  const float* values;   // [B * W_in][W_out] the rows' largest logits
  const int32_t* ids;
  const double* lse;     // [B * W_in]
};

// One group by `splits` blocks: each ranks the group's candidates and takes its share of the state rows to copy.
// A candidate's rank is what lies before it in its own beam's list, which is in order, and in each other's, found
// by binary search.
__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(BeamArgs a, int splits) {
  __shared__ double score[DOMINO_MAX_BEAMS * DOMINO_MAX_BEAMS];
  __shared__ int parent_s[DOMINO_MAX_BEAMS], token_s[DOMINO_MAX_BEAMS];
  const domino_beam_t& p = a.b;
  const int g = blockIdx.x / splits, split = blockIdx.x % splits, tid = threadIdx.x, n = p.W_in * p.W_out;
  constexpr int kMine = DOMINO_MAX_BEAMS * DOMINO_MAX_BEAMS / kMergeThreads;
  int token[kMine];
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
#pragma unroll
  for (int c = 0; c < kMine; ++c) {
    const int i = tid + c * kMergeThreads;
    if (i >= n) break;
    const int w = i / p.W_out, k = i - w * p.W_out;
    const size_t r = (size_t)g * p.W_in + w;
    const float cum = p.scores[r];
    const bool ended = p.finished && p.finished[r];
    // a dead or finished beam's candidates were not written: read, and not used
    const float z = a.values[r * p.W_out + k];
    const int id = a.ids[r * p.W_out + k];
    const double lse = a.lse[r];
    double sc = -INFINITY;
    if (cum > -INFINITY) {
      if (!ended && id >= 0) sc = (double)cum + ((double)big_clamp(z) - lse);
      if (ended && k == 0) sc = (double)cum;
    }
    token[c] = ended ? p.eos : id;
    score[i] = sc;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kMine; ++c) {
    const int i = tid + c * kMergeThreads;
    if (i >= n) break;
    const double sc = score[i];
    if (!(sc > -INFINITY)) continue;
    const int w = i / p.W_out;
    int rank = i - w * p.W_out;
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
      token_s[rank] = token[c];
      if (split == 0) {
        const size_t at = (size_t)g * p.W_out + rank;
        p.scores_out[at] = (float)sc;
        p.parents_out[at] = w;
        p.tokens_out[at] = token[c];
        if (p.finished_out)
          p.finished_out[at] = (p.finished && p.finished[(size_t)g * p.W_in + w]) || token[c] == p.eos;
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

bool beams_ok(int32_t B, int32_t W_in, int32_t W_out) {
  return B >= 1 && W_in >= 1 && W_out >= 1 && W_in <= DOMINO_MAX_BEAMS && W_out <= DOMINO_MAX_BEAMS;
}

}  // namespace

}  // namespace domino

using namespace domino;

extern "C" size_t domino_beam_workspace_bytes(int32_t B, int32_t W_in, int32_t W_out) {
  if (!beams_ok(B, W_in, W_out) || (int64_t)B * std::max(W_in, W_out) > DOMINO_MAX_ROWS) return 0;
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
  const BeamLayout lay = beam_layout(p.B, p.W_in, p.W_out);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < lay.bytes)
    return DOMINO_ERR_WORKSPACE;
  // what is read while the outputs are written, by other blocks too, may not be an output
  const size_t outs4 = (size_t)outs * 4;
  if (!disjoint({{p.scores_out, outs4}, {p.parents_out, outs4}, {p.tokens_out, outs4}, {p.finished_out, (size_t)outs},
                 {p.states_out, outs4 * p.Hs}, {p.history_out, outs4 * p.hist_len}},
                {{p.logits, rows_span(rows, p.V, p.ld, p.dtype)}, {p.scores, (size_t)rows * 4}, {p.finished, (size_t)rows},
                 {p.states, (size_t)rows * p.Hs * 4}, {p.history, (size_t)rows * p.hist_len * 4}, {workspace, lay.bytes}}))
    return DOMINO_ERR_INVALID_ARGUMENT;
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
  BeamArgs a{};
  a.b = p;
  a.values = t.values;
  a.ids = t.ids;
  a.lse = t.lse64;
  // blocks a group: about 4 vectors of the states a thread
  const int splits = p.states ? std::max(1, std::min(8, p.W_out * p.Hs / (16 * kMergeThreads))) : 1;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_top_rows(t, cs);
  if (e == cudaSuccess)
    e = note_launch(launch_pdl(k_beam_merge, dim3((unsigned)(p.B * splits)), dim3(kMergeThreads), 0, cs, a, splits));
  return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}
