// qdr_paged.h -- what the kernels over the paged cache share.
#pragma once

#include "qdr_mfma.h"
#include "qdr_mixer.h"

namespace qdr {

// Counts and contexts out of order or range, found once a call by its first workgroup.
__device__ __forceinline__ void check_counts(const KvArgs &P) {
  const long long room = (long long)P.max_pages << P.page_shift;
  for (int b = threadIdx.x; b < P.n; b += 256) {
    int first, len;
    if (!rows_of(P.cu, P.T, b, &first, &len) || (len > 0 && (P.context[b] < len || P.context[b] > room)))
      atomicOr(P.err, kErrLength);
  }
}

}  // namespace qdr
