// qdr_rotary.h -- sines and cosines of positions, and the turn of a pair.
//
// A pair's frequency is kept as turns a token in 64-bit fixed point, modulo
// one turn: position times it, in 64-bit wrap-around integers, is the angle
// modulo one turn, off by position times what the frequency was rounded by (2^-63
// of a turn at most up to a turn a token: 2^-32 at 2^31).  It is rounded to 32
// bits (2^-33 of a turn; 2^-31 in all, 2.9e-9 radians).  What is left of it to
// either side of the nearest quarter, an eighth of a turn at most, becomes fp32
// radians (2^-24 of itself twice, and the constant) and goes through Taylor's
// series, whose first left-out terms are under 2^-28 there: sine and cosine are
// off by 6 x 2^-24 at most, the product with the amplitude among it.
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

// Pairs 4 u .. 4 u + 3 of a token of the table.
__device__ __forceinline__ void pairs_of(const CosSin *row, int u, CosSin *w) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4 y = *(const f32x4 *)&row[4 * u + 2 * i];
    w[2 * i] = {y[0], y[1]};
    w[2 * i + 1] = {y[2], y[3]};
  }
}

// A row's 16 units of eight channels among eight threads, two each, whole pairs
// in both layouts and so that the threads' first units lie side by side, and
// their second ones: what they store fills its lines.
struct Units {
  int c0, c1;           // first channels
  int w0, w1;           // where the pairs' sines and cosines are, in fours
  bool turn0, turn1;
  bool half;
};
__device__ __forceinline__ Units units_of(int channels, int layout, int p) {
  const int n = channels >> 4;          // units of half the turned channels
  Units u;
  u.half = layout == 0;
  if (u.half) {
    u.turn0 = u.turn1 = p < n;
    u.c0 = 8 * (u.turn0 ? p : p + n);
    u.c1 = 8 * (u.turn0 ? p + n : p + 8);
    u.w0 = 2 * p;
    u.w1 = 2 * p + 1;
  } else {
    u.c0 = 8 * p;
    u.c1 = 64 + 8 * p;
    u.w0 = p;
    u.w1 = 8 + p;
    u.turn0 = u.c0 < channels;
    u.turn1 = u.c1 < channels;
  }
  return u;
}
// Both units' channels turned: x[0 .. 7] and x[8 .. 15].
__device__ __forceinline__ void turn_units(const Units &u, const CosSin *row, float *x) {
  CosSin w[8];
  pairs_of(row, u.w0, w);
  pairs_of(row, u.w1, w + 4);
  if (u.half) {
#pragma unroll
    for (int e = 0; e < 8; ++e) turn(x[e], x[8 + e], w[e], &x[e], &x[8 + e]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < 4 || u.turn1) turn(x[2 * e], x[2 * e + 1], w[e], &x[2 * e], &x[2 * e + 1]);
}

// Rows are read once and their results by a later launch, of more than the
// caches hold where it matters: both go past them.  Measured, with a copy that
// makes the rows before and qdr_kv_attend behind (us, plain / past the caches):
// 32 x 64 tokens of 32 heads 50.0 / 49.6, 32 x 256 141 / 141, 32 x 512 312 / 302.
__device__ __forceinline__ u32x4 read_once(const uint16_t *x) { return __builtin_nontemporal_load((const u32x4_a4 *)x); }
__device__ __forceinline__ void write_past(uint16_t *y, u32x4 w) { __builtin_nontemporal_store(w, (u32x4_a4 *)y); }

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
// widen16's inverse: channels that do not turn keep every bit (rounding would
// quiet a NaN).
__device__ __forceinline__ u32x4 unwiden16(const float *x) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(x[2 * i]) >> 16 | (__float_as_uint(x[2 * i + 1]) & 0xFFFF0000u);
  return w;
}

}  // namespace qdr
