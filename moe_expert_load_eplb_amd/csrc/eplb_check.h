// Host-side checks that every entry point makes on its buffers.
#pragma once

#include "eplb.h"

namespace eplb {

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte (ends
// taken in 128 bits, so a range reaching past the address space still
// compares correctly).
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (a == nullptr || b == nullptr || na <= 0 || nb <= 0) return false;
  const unsigned __int128 x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (unsigned __int128)nb && y < x + (unsigned __int128)na;
}

// a * b * c bytes, saturated at 2^63 - 1 (a caller's window of W steps is
// not bounded above, so its byte count may not fit).
inline int64_t bytes_of(int64_t a, int64_t b, int64_t c) {
  int64_t ab = 0, abc = 0;
  if (__builtin_mul_overflow(a, b, &ab) || __builtin_mul_overflow(ab, c, &abc)) return INT64_MAX;
  return abc;
}

struct Range {
  const void* p;
  int64_t bytes;
};

// No output shares a byte with an input or another output (empty ranges and
// NULL pointers share nothing; the calls check NULLs themselves).
template <int NI, int NO>
inline int32_t check_disjoint(const Range (&in)[NI], const Range (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (const Range& c : in)
      if (overlap(out[i].p, out[i].bytes, c.p, c.bytes)) return EPLB_E_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return EPLB_E_ARG;
  }
  return EPLB_OK;
}

// A call with these input and output ranges: every pointer set, no output
// sharing a byte with an input or another output.
template <int NI, int NO>
inline int32_t check_buffers(const Range (&in)[NI], const Range (&out)[NO]) {
  for (const Range& a : in)
    if (a.p == nullptr) return EPLB_E_ARG;
  for (const Range& a : out)
    if (a.p == nullptr) return EPLB_E_ARG;
  return check_disjoint(in, out);
}

}  // namespace eplb
