// qdr_rotary.h -- sines and cosines of positions, and the turn of a pair.
//
// A pair's frequency is kept as turns a token in 64-bit fixed point, modulo
// one turn: position times it, in 64-bit wrap-around integers, is the angle
// modulo one turn with no rounding that grows with the position.  Its upper 32
// bits (2^-32 of a turn, 1.5e-9 radians) go through Taylor's series on an
// eighth of a turn to either side of the nearest quarter, whose first left-out
// terms are under 2^-28 there.
#pragma once

#include "qdr_cache.h"
#include "qdr_mfma.h"

namespace qdr {

struct CosSin {
  float c, s;
};

__device__ __forceinline__ CosSin cos_sin(uint64_t turns, int position) {
  const uint64_t a = turns * (uint64_t)(int64_t)position;
  const uint32_t t = (uint32_t)((a + 0x80000000u) >> 32);
  const uint32_t quarter = (t + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(t - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi / 2^32
  const float y = x * x;
  float s = __builtin_fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
  s = __builtin_fmaf(s, y, 8.3333333e-3f);
  s = __builtin_fmaf(s, y, -1.6666667e-1f);
  s = __builtin_fmaf(s * y, x, x);
  float c = __builtin_fmaf(y, -2.7557319e-7f, 2.4801587e-5f);
  c = __builtin_fmaf(c, y, -1.3888889e-3f);
  c = __builtin_fmaf(c, y, 4.1666667e-2f);
  c = __builtin_fmaf(c, y, -0.5f);
  c = __builtin_fmaf(c, y, 1.0f);
  const float u = (quarter & 1) ? s : c, v = (quarter & 1) ? c : s;
  CosSin r;
  r.c = (quarter == 1 || quarter == 2) ? -u : u;
  r.s = (quarter & 2) ? -v : v;
  return r;
}

// Turned pair.
__device__ __forceinline__ void turn(float a, float b, CosSin w, float *p, float *q) {
  *p = __builtin_fmaf(a, w.c, -(b * w.s));
  *q = __builtin_fmaf(a, w.s, b * w.c);
}

// The table of a workgroup's tokens: 64 pairs a token, and 16 bytes more so
// that the tokens of a wave begin on banks of their own.
constexpr int kTablePairs = 64, kTableRow = kTablePairs + 2;

// Pairs 8 u .. 8 u + 7 of a token of the table.
__device__ __forceinline__ void pairs_of(const CosSin *row, int u, CosSin *w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x4 y = *(const f32x4 *)&row[8 * u + 2 * i];
    w[2 * i] = {y[0], y[1]};
    w[2 * i + 1] = {y[2], y[3]};
  }
}

__device__ __forceinline__ void widen16(const u32x4 w, float *x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo_f32(w[i]);
    x[2 * i + 1] = hi_f32(w[i]);
  }
}
__device__ __forceinline__ u32x4 narrow16(const float *x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
  return w;
}

}  // namespace qdr
