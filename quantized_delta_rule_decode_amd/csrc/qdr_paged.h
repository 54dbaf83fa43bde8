// qdr_paged.h -- what the kernels over the paged cache share.
#pragma once

#include "qdr_mfma.h"
#include "qdr_mixer.h"

namespace qdr {

// Tokens that a sequence's pages have room for.  (A page may stand at several
// places of a table, so a table can be longer than any cache; positions and
// blocks of keys, rounded up to whole pieces, are counted in 32 bits.)
__device__ __forceinline__ int room_of(const KvArgs &P) {
  return (int)min((long long)P.max_pages << P.page_shift, (long long)kMostContext);
}

// Counts and contexts out of order or range, found once a call by its first workgroup.
__device__ __forceinline__ void check_counts(const KvArgs &P) {
  const int room = room_of(P);
  for (int b = threadIdx.x; b < P.n; b += 256) {
    int first, len;
    if (!rows_of(P.cu, P.T, b, &first, &len) || (len > 0 && (P.context[b] < len || P.context[b] > room)))
      atomicOr(P.err, kErrLength);
  }
}

}  // namespace qdr
