// Whether what a call over a list of tensors writes lies apart from everything else that it takes (host
// code, shared by ops_clip.hip and ops_adamw.hip).
#pragma once
#include <stdint.h>
#include <stdlib.h>

#include <algorithm>

#include "../../include/gemm.h"

namespace dg {

struct Span {
  uintptr_t begin, end;
  bool written;
};

// GEMM_OK where no span that is written overlaps another one.  at(i, s) puts entry i's spans into s, N at
// most and none of them empty, and returns how many there are.
template <int N, class At>
int spans_apart(int64_t count, At at) {
  // Most lists are cut from a few buffers, or allocated in order: a few runs of rising addresses that lie
  // apart as wholes (0.7 us for 153 tensors into others, 5 to sort them).
  constexpr int RUNS = 16;
  constexpr uintptr_t NEAR = 512;   // an allocator's rounding
  Span run[RUNS], s[N];
  int last[N] = {};   // the run that the spans of this place in an entry were in
  int runs = 0;
  bool simple = true;
  for (int64_t i = 0; i < count && simple; ++i)
    for (int k = at(i, s) - 1; k >= 0 && simple; --k) {
      const auto ends_before = [&](int r) { return s[k].begin - run[r].end < NEAR; };
      int to = last[k];   // a run that ends just before it
      if (to >= runs || !ends_before(to)) {
        to = 0;
        while (to < runs && !ends_before(to)) ++to;
      }
      if (to < runs)
        run[to].end = s[k].end;
      else if (runs < RUNS)
        run[runs++] = s[k];
      else
        simple = false;
      last[k] = to;
    }
  const auto before = [](const Span &a, const Span &b) { return a.begin < b.begin; };
  std::sort(run, run + runs, before);
  for (int r = 1; r < runs; ++r) simple = simple && run[r - 1].end <= run[r].begin;
  if (simple) return GEMM_OK;

  Span *const all = (Span *)malloc((size_t)count * N * sizeof(Span));
  if (!all) return GEMM_ERR_UNSUPPORTED;
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i)
    for (int k = at(i, s) - 1; k >= 0; --k) all[n++] = s[k];
  std::sort(all, all + n, before);
  uintptr_t read = 0, written = 0;   // where those so far end
  bool apart = true;
  for (int64_t i = 0; i < n; ++i) {
    apart = apart && all[i].begin >= written && !(all[i].written && all[i].begin < read);
    uintptr_t &end = all[i].written ? written : read;
    end = std::max(end, all[i].end);
  }
  free(all);
  return apart ? GEMM_OK : GEMM_ERR_INVALID_ARG;
}

}  // namespace dg
