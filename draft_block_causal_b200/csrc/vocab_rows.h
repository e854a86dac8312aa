// vocab_rows.h -- host-side checks and the row scan's launch shared by the operators on rows of logits.
#pragma once

#include "internal.h"

namespace domino {

inline bool rows_ok(int64_t rows, int V, int64_t ld, int dtype, const void* p) {
  return rows >= 1 && V >= 1 && V <= DOMINO_MAX_V && ld >= V && ld % 8 == 0 && ld <= INT32_MAX &&
         (dtype == DOMINO_DTYPE_F32 || dtype == DOMINO_DTYPE_BF16) && p &&
         (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}
inline size_t dtype_bytes(int dtype) { return dtype == DOMINO_DTYPE_F32 ? 4 : 2; }
inline bool temperature_ok(float t) { return t >= 0.0009765625f && t <= 1024.f; }

// Bytes that rows of V values ld apart span.
inline size_t rows_span(int64_t rows, int V, int64_t ld, int dtype) {
  return ((size_t)(rows - 1) * ld + V) * dtype_bytes(dtype);
}
// Whether [a, a + na) and [b, b + nb) share a byte (null: no).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Outputs of a call against its inputs and against each other (null: not there).
struct Range {
  const void* p;
  size_t n;
};
template <int OUT, int IN>
bool disjoint(const Range (&out)[OUT], const Range (&in)[IN]) {
  for (int i = 0; i < OUT; ++i) {
    for (const Range& r : in)
      if (overlap(out[i].p, out[i].n, r.p, r.n)) return false;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return false;
  }
  return true;
}

// The k largest logits and the log-sum-exp of every row (top_logits.cu).  Row r is skipped, its outputs left
// alone, when scores (or null) has nothing above -infinity for it or finished (or null) is not 0.
struct TopRows {
  const void* logits;
  int64_t ld;
  int rows, V, dtype, k;
  float c;       // log2(e) / temperature
  double inv_t;
  const float* scores;
  const uint8_t* finished;
  float* values;
  int32_t* ids;
  float* lse;      // fp32 or
  double* lse64;   // double, either may be null
};
cudaError_t launch_top_rows(const TopRows& a, cudaStream_t st);

}  // namespace domino
