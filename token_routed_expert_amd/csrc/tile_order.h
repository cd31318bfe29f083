// The order in which the XCDs take the tiles of a grouped product: plain
// integer functions, the same on the device and (for the tests) on the host.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define TRE_ORDER __host__ __device__ __forceinline__
#else
#define TRE_ORDER inline
#endif

namespace tre {

// Bijection on [0, n): block ids with the same value mod 8 (dispatched to the
// same XCD, each XCD with its own L2) get consecutive logical tile ids.
TRE_ORDER int xcd_remap(int i, int n) {
  const int x = i & 7, j = i >> 3;
  const int q = n >> 3, r = n & 7;
  return x * q + (x < r ? x : r) + j;
}

// The same in rounds of 8 C tiles: an XCD takes C consecutive ones of each
// round, so that tiles of unequal work spread over the XCDs; what is left after
// the last whole round is divided as above.
template <int C>
TRE_ORDER int xcd_remap_rounds(int i, int n) {
  const int whole = n / (8 * C) * (8 * C);
  if (i >= whole) return whole + xcd_remap(i - whole, n - whole);
  return i / (8 * C) * (8 * C) + (i & 7) * C + (i >> 3) % C;
}

// Whether some eighth of a list with the same number of tiles for each of E
// experts holds more than 5/4 of an eighth of the rows, offs [E + 1].  An eighth
// ends inside an expert where E is not a multiple of 8, and has that part of its
// rows: even rows are even for every E.
TRE_ORDER bool uneven_eighths(const int32_t* offs, int E) {
  int64_t most = 0, before = 0;  // in eighths of a row
  for (int x = 1; x <= 8; ++x) {
    const int e = (x * E) >> 3, part = (x * E) & 7;
    const int64_t upto = 8 * (int64_t)offs[e] + (part ? part * (int64_t)(offs[e + 1] - offs[e]) : 0);
    most = upto - before > most ? upto - before : most;
    before = upto;
  }
  return 4 * most > 5 * (int64_t)offs[E];
}

}  // namespace tre
