// qdr_mfma.h -- device helpers of the matrix-core kernels: the 16x16x32
// bfloat16 product, its operand layout, and fp32 values as sums of bfloat16.
//
// v_mfma_f32_16x16x32_bf16, lane l = 16 g + i:
//   A (16 rows x 32): lane holds row i, eight values of the contraction;
//   B (32 x 16 columns): lane holds column i, the same eight;
//   C, D (16 x 16): lane holds column i, rows 4 g .. 4 g + 3.
// Which eight values of the contraction a lane group g stands for is free as
// long as A and B agree.  Everywhere here group g takes members 4 g .. 4 g + 3
// of the first and of the second 16: then the accumulators of two stacked
// 16x16 results ARE a B operand, lane for lane, and a product feeds the next
// without moving data between lanes.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qdr {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// in caller memory, which is only 4-byte aligned
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef u32x2 u32x2_a4 __attribute__((aligned(4)));

union Frag {
  bf16x8 v;
  u32x4 w;
  u32x2 h[2];
  uint32_t u[4];
};

__device__ __forceinline__ f32x4 mma(const Frag &a, const Frag &b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}

// Two fp32 values rounded to nearest-even bfloat16, the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 r = __builtin_convertvector((f32x2){a, b}, bf16x2);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a and b as sums of P bfloat16 values each, largest first: every part takes
// the next 8 bits of the significand, so three of them hold an fp32 value to
// its last bit (while the parts do not underflow).
template <int P>
__device__ __forceinline__ void parts(float a, float b, uint32_t *part) {
  part[0] = pack_bf16(a, b);
#pragma unroll
  for (int p = 1; p < P; ++p) {
    a -= lo_f32(part[p - 1]);
    b -= hi_f32(part[p - 1]);
    part[p] = pack_bf16(a, b);
  }
}

// Barrier of a workgroup whose waves exchange data through LDS only: waits for
// the LDS operations before it, not for loads and stores of global memory, so
// what was loaded ahead stays in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Index of the sequence that place `id` of a call belongs to, where sequence
// b has places first(b) = cu[b] / per + extra * b on: first() grows with b, and
// the last b with first(b) <= id is found 64 candidates at a time (a load for
// up to 64 sequences, two for up to 4096).  The whole wave calls it.
__device__ __forceinline__ int sequence_of(const int32_t *cu, int n, int per, int extra, int id) {
  const int lane = (int)(threadIdx.x & 63);
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 63) >> 6, at = lane * step;
    bool not_behind = false;
    if (at < len) {
      const int c = cu[lo + at];
      not_behind = (c >= 0 ? c / per : 0) + extra * (lo + at) <= id;
    }
    const int count = __popcll(__ballot(not_behind));
    if (count > 1) {
      lo += (count - 1) * step;
      len = min(step, len - (count - 1) * step);
    } else {
      len = min(step, len);
    }
    if (step == 1) break;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Rows [first, first + len) of sequence b; false where the counts are out of
// order or leave the arrays.
__device__ __forceinline__ bool rows_of(const int32_t *cu, int T, int b, int *first, int *len) {
  const int s = cu[b], e = cu[b + 1];
  *first = s;
  *len = e - s;
  return s >= 0 && e >= s && e <= T;
}

}  // namespace qdr
