// What a sequence has to read, as a list of blocks in stages: device code shared by the
// windowed / page-scaled decode and the kernel that joins its partials.
#pragma once

#include "span_decode.h"

namespace pa {
namespace span {

// The blocks that a sequence of `len` tokens has to read.
struct Span {
  int len, lo;        // lo: first token that the window of the first new token reaches
  int nblk;           // blocks in the list
  int ns, shift;      // list index v is block v + (v >= ns ? shift : 0)
  int nst;            // stages (at least one, so that empty sequences get their zero rows)
};

template <int TU>
__device__ __forceinline__ Span make_span(const SpanParams& p, int raw_len) {
  Span s;
  s.len = min(max(raw_len, 0), p.max_len);
  s.lo = max(0, s.len - p.q_len + 1 - p.window);
  const int nb = (s.len + TU - 1) / TU;
  const int wb = s.lo / TU;
  s.ns = (min(p.sinks, s.len) + TU - 1) / TU;
  s.shift = wb - s.ns;
  if (s.shift <= 0) s.ns = s.shift = 0;
  s.nblk = nb - s.shift;
  const int wph_log2 = 3 - p.hg_log2;
  s.nst = max(1, (s.nblk + (1 << wph_log2) - 1) >> wph_log2);
  return s;
}

// Stages of a CTA's share, rounded up (a 64-bit division takes a few hundred cycles).
__device__ __forceinline__ long long share_of(long long total, unsigned ctas) {
  return (total >> 31) == 0 ? static_cast<long long>((static_cast<unsigned>(total) + ctas - 1) / ctas)
                            : (total + ctas - 1) / ctas;
}

}  // namespace span
}  // namespace pa
