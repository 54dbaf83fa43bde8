// qdr_rotary.hip -- rows turned by their positions.
// A workgroup takes some tokens of up to 128 heads, about 128 rows (token,
// head): the pairs' sines and cosines are made once a token, in LDS, while the
// rows are on their way, and each is used by every head.  Eight threads a row,
// two units of eight channels each (units_of).
// Bound by memory: 16385 tokens of 32 heads, bfloat16, 64 channels in pairs:
// 46.5 us for 268 MB (5.8 TB/s; a copy of 4 GiB reaches 5.4).  A thread's two
// units next to each other instead took 49.0, or 64 with stores past the caches
// (each filled half a line); as here without those stores and loads 50.8.  One
// token of 8 heads: 2.3 us of kernel, 6.5 a call.  fp32 stays in the caches (a
// store fills half of each 32 bytes): 105 us for the same rows, 537 MB (5.1 TB/s).
#include "qdr_rotary.h"

namespace qdr {

namespace {

constexpr int kD = 128, kPasses = 4;
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));

// Eight consecutive elements of a row.
template <bool BF16>
struct Eight;
template <>
struct Eight<true> {
  u32x4 w;
  __device__ __forceinline__ void load(const void *x, size_t at) { w = read_once((const uint16_t *)x + at); }
  __device__ __forceinline__ void store(void *y, size_t at) const { write_past((uint16_t *)y + at, w); }
  __device__ __forceinline__ void get(float *x) const { widen16(w, x); }
  __device__ __forceinline__ void set(const float *x) { w = narrow16(x); }
};
template <>
struct Eight<false> {
  f32x4 w[2];
  __device__ __forceinline__ void load(const void *x, size_t at) {
    w[0] = *(const f32x4_a4 *)((const float *)x + at);
    w[1] = *(const f32x4_a4 *)((const float *)x + at + 4);
  }
  __device__ __forceinline__ void store(void *y, size_t at) const {
    *(f32x4_a4 *)((float *)y + at) = w[0];
    *(f32x4_a4 *)((float *)y + at + 4) = w[1];
  }
  __device__ __forceinline__ void get(float *x) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = w[i >> 2][i & 3];
  }
  __device__ __forceinline__ void set(const float *x) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = x[i];
  }
};

template <bool BF16>
__global__ void __launch_bounds__(256) k_rotate(RotateArgs A) {
  __shared__ __attribute__((aligned(16))) CosSin table[32][kTableRow];
  const int tid = threadIdx.x, part = blockIdx.x % A.head_parts;
  const int t0 = (int)(blockIdx.x / A.head_parts) * A.tokens, h0 = part * A.part_heads;
  const int tokens = min(A.tokens, A.T - t0), heads = min(A.part_heads, A.heads - h0);
  const int rows = tokens * heads, pairs = A.rotary.channels >> 1;
  const Units u = units_of(A.rotary.channels, A.rotary.layout, tid & 7);
  bool ready = false;
  for (int base = 0; base < rows; base += 32 * kPasses) {
    Eight<BF16> a[kPasses], b[kPasses];
    int tok[kPasses], head[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = min(base + 32 * i + (tid >> 3), rows - 1);
      tok[i] = row / heads;
      head[i] = h0 + row - tok[i] * heads;
      const size_t at = (size_t)(t0 + tok[i]) * A.x_stride + (size_t)head[i] * kD;
      a[i].load(A.x, at + u.c0);
      b[i].load(A.x, at + u.c1);
    }
    if (!ready) {
      const int pair = tid & 63;
      const uint64_t f = pair < pairs ? A.rotary.turns[pair] : 0;
      for (int t = tid >> 6; t < tokens; t += 4) {
        CosSin w = cos_sin(f, A.positions[t0 + t]);
        w.c *= A.rotary.amplitude;
        w.s *= A.rotary.amplitude;
        table[t][pair] = w;
      }
      lds_barrier();
      ready = true;
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      if (base + 32 * i + (tid >> 3) >= rows) continue;
      if (u.turn0) {
        float x[16];
        a[i].get(x);
        b[i].get(x + 8);
        turn_units(u, table[tok[i]], x);
        a[i].set(x);
        if (u.turn1) b[i].set(x + 8);
      }
      const size_t at = (size_t)(t0 + tok[i]) * A.y_stride + (size_t)head[i] * kD;
      a[i].store(A.y, at + u.c0);
      b[i].store(A.y, at + u.c1);
    }
  }
}

}  // namespace

hipError_t launch_rotate(const RotateArgs &a, bool bf16, hipStream_t st) {
  const dim3 grid((uint32_t)((a.T + a.tokens - 1) / a.tokens) * (uint32_t)a.head_parts);
  if (bf16) hipLaunchKernelGGL(k_rotate<true>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_rotate<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace qdr
