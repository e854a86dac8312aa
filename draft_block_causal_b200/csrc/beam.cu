// beam.cu -- one step of beam search: the best continuations over a group's beams and the vocabulary, and
// the beams' states and histories reordered to follow their parents.
//
// Only a beam's W_out best tokens can be among the group's W_out best continuations, so the row scan of
// top_logits.cu leaves W_in * W_out candidates a group (k_top_rows, one read of the logits), and k_beam_merge
// ranks them.  Scores are compared in 64 bits: two beams' candidates can lie closer together than one
// rounding of a score of tens to fp32 (2^-19).
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

__global__ void __launch_bounds__(kMergeThreads) k_beam_merge(BeamArgs a) {
  __shared__ double score[DOMINO_MAX_BEAMS * DOMINO_MAX_BEAMS];
  __shared__ int32_t token[DOMINO_MAX_BEAMS * DOMINO_MAX_BEAMS];
  __shared__ int parent_s[DOMINO_MAX_BEAMS], token_s[DOMINO_MAX_BEAMS];
  pdl_wait();
  pdl_trigger();
  const domino_beam_t& p = a.b;
  const int g = blockIdx.x, tid = threadIdx.x, n = p.W_in * p.W_out;
  for (int i = tid; i < n; i += kMergeThreads) {
    const int w = i / p.W_out, k = i % p.W_out;
    const size_t r = (size_t)g * p.W_in + w;
    const float cum = p.scores[r];
    double sc = -INFINITY;
    int id = 0;
    if (cum > -INFINITY) {
      if (p.finished && p.finished[r]) {
        if (k == 0) { sc = (double)cum; id = p.eos; }
      } else {
        const float z = a.values[r * p.W_out + k];
        id = a.ids[r * p.W_out + k];
        if (id >= 0) sc = (double)cum + ((double)big_clamp(z) - a.lse[r]);
      }
    }
    score[i] = sc;
    token[i] = id;
  }
  if (tid < p.W_out) { parent_s[tid] = -1; token_s[tid] = 0; }
  __syncthreads();
  for (int i = tid; i < n; i += kMergeThreads) {
    const double sc = score[i];
    if (!(sc > -INFINITY)) continue;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += score[j] > sc || (score[j] == sc && j < i);
    if (rank < p.W_out) {
      const size_t o = (size_t)g * p.W_out + rank;
      const int w = i / p.W_out;
      parent_s[rank] = w;
      token_s[rank] = token[i];
      p.scores_out[o] = (float)sc;
      p.parents_out[o] = w;
      p.tokens_out[o] = token[i];
      if (p.finished_out)
        p.finished_out[o] = (p.finished && p.finished[(size_t)g * p.W_in + w]) || token[i] == p.eos;
    }
  }
  __syncthreads();
  for (int w = tid; w < p.W_out; w += kMergeThreads)
    if (parent_s[w] < 0) {
      const size_t o = (size_t)g * p.W_out + w;
      p.scores_out[o] = -INFINITY;
      p.parents_out[o] = 0;
      p.tokens_out[o] = 0;
      if (p.finished_out) p.finished_out[o] = 0;
    }
  for (int w = 0; w < p.W_out; ++w) {
    const size_t from = (size_t)g * p.W_in + max(parent_s[w], 0), to = (size_t)g * p.W_out + w;
    if (p.states) {
      const float4* src = reinterpret_cast<const float4*>(p.states + from * p.Hs);
      float4* dst = reinterpret_cast<float4*>(p.states_out + to * p.Hs);
      for (int i = tid; i < p.Hs / 4; i += kMergeThreads) dst[i] = src[i];
    }
    if (p.history) {
      const int32_t* src = p.history + from * p.hist_len;
      int32_t* dst = p.history_out + to * p.hist_len;
      for (int i = tid; i < p.hist_len; i += kMergeThreads) dst[i] = i == p.pos ? token_s[w] : src[i];
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
  if (p.eos < -1 || p.eos >= p.V || (p.finished && (p.eos < 0 || !p.finished_out)) || (p.finished_out && p.eos < 0))
    return DOMINO_ERR_INVALID_ARGUMENT;
  if (!p.states != !p.states_out || !p.history != !p.history_out) return DOMINO_ERR_INVALID_ARGUMENT;
  if (p.states && (p.Hs < 4 || p.Hs % 4 || !a16(p.states) || !a16(p.states_out))) return DOMINO_ERR_INVALID_ARGUMENT;
  if (p.history && (p.hist_len < 1 || p.pos < 0 || p.pos >= p.hist_len)) return DOMINO_ERR_INVALID_ARGUMENT;
  if (rows > DOMINO_MAX_ROWS || outs > DOMINO_MAX_ROWS) return DOMINO_ERR_UNSUPPORTED;
  const BeamLayout lay = beam_layout(p.B, p.W_in, p.W_out);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < lay.bytes)
    return DOMINO_ERR_WORKSPACE;
  // what is read while the outputs are written, by other blocks too, may not be an output
  const struct { const void* p; size_t n; } in[] = {
      {p.logits, rows_span(rows, p.V, p.ld, p.dtype)}, {p.scores, (size_t)rows * 4}, {p.finished, (size_t)rows},
      {p.states, (size_t)rows * p.Hs * 4}, {p.history, (size_t)rows * p.hist_len * 4}, {workspace, lay.bytes}},
      out[] = {{p.scores_out, (size_t)outs * 4}, {p.parents_out, (size_t)outs * 4}, {p.tokens_out, (size_t)outs * 4},
               {p.finished_out, (size_t)outs}, {p.states_out, (size_t)outs * p.Hs * 4},
               {p.history_out, (size_t)outs * p.hist_len * 4}};
  for (const auto& o : out)
    for (const auto& i : in)
      if (overlap(o.p, o.n, i.p, i.n)) return DOMINO_ERR_INVALID_ARGUMENT;
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
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_top_rows(t, cs);
  if (e == cudaSuccess)
    e = note_launch(launch_pdl(k_beam_merge, dim3((unsigned)p.B), dim3(kMergeThreads), 0, cs, a));
  return e == cudaSuccess ? DOMINO_OK : DOMINO_ERR_CUDA;
}
