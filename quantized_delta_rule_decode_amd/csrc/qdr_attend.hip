// qdr_attend.hip -- attention of new tokens over the paged cache: how a call's
// rows and keys are dealt to workgroups, and how the pieces of cut keys are
// joined.  What a workgroup computes is in qdr_attend_tiles.h.
#include "qdr_attend_tiles.h"

namespace qdr {

namespace {

template <bool FEW>
__device__ __forceinline__ bool tile_of(const AttendArgs &A, const AttendPlan &plan, int tile, int part, int kvh, Tile &t) {
  const KvArgs &P = A.kv;
  const int per = FEW ? plan.few_tokens : plan.many_tokens;
  if (FEW && tile < P.n) {
    // a sequence's first tile; in a call with both launches of the sequences
    // that have no other
    t.b = tile;
    if (!rows_of(P.cu, P.T, t.b, &t.first, &t.len) || t.len == 0 || (plan.many && t.len > per)) return false;
    t.token = 0;
  } else if (FEW) {
    // The other tiles, ceil(len / per) - 1 from place cu[b] / per on: behind the
    // first ones, so that in a call of single tokens no idle workgroup stands
    // between those that have work (which then miss a compute unit and wait for
    // a second turn: 64 requests of 8000 tokens, one head 46 us instead of 33).
    t.b = sequence_of(P.cu, P.n, per, 0, tile - P.n);
    if (!rows_of(P.cu, P.T, t.b, &t.first, &t.len)) return false;
    t.token = (tile - P.n - t.first / per + 1) * per;
    if (t.token < per || t.token >= t.len) return false;
  } else {
    t.b = sequence_of(P.cu, P.n, per, 1, tile);
    if (!rows_of(P.cu, P.T, t.b, &t.first, &t.len)) return false;
    t.token = (tile - (t.first / per + t.b)) * per;
    if (t.token < 0 || t.token >= t.len || (plan.few && t.len <= plan.few_tokens)) return false;
  }
  t.tokens = min(per, t.len - t.token);
  const int heads = FEW ? plan.few_heads : plan.many_heads;
  t.head = kvh * plan.group + part * heads;
  t.heads = min(heads, plan.group - part * heads);
  const int ctx = P.context[t.b];
  t.skipped = ctx < t.len || ctx > room_of(P);
  t.position = ctx - t.len + t.token;
  t.keys = t.skipped ? 0 : t.position + t.tokens;
  return true;
}

template <int KIND>
__global__ void __launch_bounds__(64 * kFewWaves, 2) k_attend_few(AttendArgs A, AttendPlan plan) {
  const KvArgs &P = A.kv;
  __shared__ FewShared<kFewWaves> sh;
  if (blockIdx.x == 0) check_counts(P);
  const int split = blockIdx.x % plan.few_splits;
  const int part = blockIdx.x / plan.few_splits % plan.few_parts;
  const int kvh = blockIdx.x / (plan.few_splits * plan.few_parts) % P.heads;
  const int tile = blockIdx.x / (plan.few_splits * plan.few_parts * P.heads);
  Tile t;
  if (!tile_of<true>(A, plan, tile, part, kvh, t)) return;
  const int blocks = (t.keys + kBlock - 1) / kBlock;
  const int each = piece_blocks(blocks, plan.few_splits, kFewLeast);
  const int lo = split * each, hi = min(lo + each, blocks);
  if (lo >= hi && split > 0) return;

  const int l = threadIdx.x & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  FewOut<kFewWaves> out;
  few_tile<KIND, kFewWaves, true>(A, t, threadIdx.x, kvh, lo, hi, sh, out);
  static_assert(kFewWaves == 8, "a wave to sixteen channels");
  const f32x4 y = out.o[0];
  if (plan.few_splits == 1) {
    if (out.row) {
      const float inv = out.sum > 0.0f || out.sum != out.sum ? 1.0f / out.sum : 0.0f;
      *(u32x2_a4 *)(A.o + out.at + 16 * w + 4 * g) = (u32x2){pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
    }
  } else {
    float *to = A.part + (size_t)blockIdx.x * (kFewRows * (kD + 2));
    *(f32x4 *)(to + (size_t)i16 * kD + 16 * w + 4 * g) = y;
    if (w == 0 && g == 0) {
      to[kFewRows * kD + i16] = out.m;
      to[kFewRows * kD + kFewRows + i16] = out.sum;
    }
  }
}

template <int KIND>
__global__ void __launch_bounds__(256, 2) k_attend_many(AttendArgs A, AttendPlan plan) {
  const KvArgs &P = A.kv;
  __shared__ ManyShared<KIND> sh[2];
  if (blockIdx.x == 0) check_counts(P);
  // heads change fastest (workgroups are dealt to the eight XCDs in turn, so
  // the tiles of one head share few L2s), and the tiles with most keys come first
  const int kvh = blockIdx.x % P.heads;
  const int part = blockIdx.x / P.heads % plan.many_parts;
  const int split = blockIdx.x / (P.heads * plan.many_parts) % plan.many_splits;
  const int tile = plan.many_tiles - 1 - (int)(blockIdx.x / (P.heads * plan.many_parts * plan.many_splits));
  Tile t;
  if (!tile_of<false>(A, plan, tile, part, kvh, t)) return;
  const int blocks = (t.keys + kBlock - 1) / kBlock;
  const int each = piece_blocks(blocks, plan.many_splits, kManyLeast);
  const int lo = split * each, hi = min(lo + each, blocks);
  if (lo >= hi && split > 0) return;

  const int l = threadIdx.x & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  ManyOut out;
  many_tile<KIND, false>(A, t, threadIdx.x, kvh, lo, hi, sh, out);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (plan.many_splits == 1) {
      if (!out.row[c]) continue;
      const float inv = out.sum[c] > 0.0f || out.sum[c] != out.sum[c] ? 1.0f / out.sum[c] : 0.0f;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const f32x4 y = out.o[c][d] * inv;
        *(u32x2_a4 *)(A.o + out.at[c] + 16 * d + 4 * g) = (u32x2){pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
      }
    } else {
      const size_t unit = (((size_t)tile * P.heads + kvh) * plan.many_parts + part) * plan.many_splits + split;
      float *to = A.part + plan.few_floats + unit * (kManyRows * (kD + 2));
      const int r = 32 * w + 16 * c + i16;
#pragma unroll
      for (int d = 0; d < 8; ++d) *(f32x4 *)(to + (size_t)r * kD + 16 * d + 4 * g) = out.o[c][d];
      if (g == 0) {
        to[kManyRows * kD + r] = out.m[c];
        to[kManyRows * kD + kManyRows + r] = out.sum[c];
      }
    }
  }
}

// Joins the pieces of the keys (64 at most): a wave takes OWN rows.  A lane has
// a piece's maximum and sum of each row; then half a wave takes four channels a
// lane of every other piece, sixteen loads on their way at once.  Eight rows a
// wave where there are few pieces of many rows, so that it finds its tile once
// (4 x 256 new tokens in two pieces 16 us, with one row 23; two of 961 in five
// 11.8 and 10.7, 20 in 64 26 and 8).
template <bool FEW, int OWN>
__global__ void __launch_bounds__(256) k_attend_join(AttendArgs A, AttendPlan plan) {
  constexpr int kRows = FEW ? kFewRows : kManyRows, kOwn = OWN, kLoads = OWN == 1 ? 8 : 2;
  const KvArgs &P = A.kv;
  const int parts = FEW ? plan.few_parts : plan.many_parts, splits = FEW ? plan.few_splits : plan.many_splits;
  const int l = threadIdx.x & 63, half = l >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int kGroups = kRows / (4 * kOwn);
  const int r0 = ((blockIdx.x % kGroups) * 4 + w) * kOwn, unit = blockIdx.x / kGroups;
  const int part = unit % parts, kvh = unit / parts % P.heads, tile = unit / (parts * P.heads);
  Tile t;
  if (!tile_of<FEW>(A, plan, tile, part, kvh, t) || r0 / t.heads >= t.tokens) return;
  const int blocks = (t.keys + kBlock - 1) / kBlock;
  const int each = piece_blocks(blocks, splits, FEW ? kFewLeast : kManyLeast);
  const int live = max((blocks + each - 1) / each, 1);
  constexpr size_t kStep = kRows * (kD + 2);
  const float *from = A.part + (FEW ? 0 : plan.few_floats) + (size_t)unit * splits * kStep;
  const float *stats = from + min(l, live - 1) * kStep + kRows * kD + r0;
  float f[kOwn], sum[kOwn], own[kOwn];
  f32x4 o[kOwn];
#pragma unroll
  for (int x = 0; x < kOwn; ++x) {
    own[x] = stats[x];
    sum[x] = stats[kRows + x];
  }
#pragma unroll
  for (int x = 0; x < kOwn; ++x) {
    const float m = wave_max(own[x]);
    f[x] = ex2(own[x] - (m == kNone ? 0.0f : m));
    sum[x] = l < live ? sum[x] * f[x] : 0.0f;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum[x] += __shfl_xor(sum[x], d);
    o[x] = (f32x4){0, 0, 0, 0};
  }
  for (int s0 = 0; s0 < live; s0 += 2 * kLoads) {
    f32x4 y[kOwn][kLoads];
#pragma unroll
    for (int x = 0; x < kOwn; ++x)
#pragma unroll
      for (int s = 0; s < kLoads; ++s)
        y[x][s] = *(const f32x4 *)(from + min(s0 + 2 * s + half, live - 1) * kStep + (size_t)(r0 + x) * kD + 4 * (l & 31));
#pragma unroll
    for (int x = 0; x < kOwn; ++x)
#pragma unroll
      for (int s = 0; s < kLoads; ++s) {
        const float fs = __shfl(f[x], s0 + 2 * s + half);
        if (s0 + 2 * s + half < live) o[x] += y[x][s] * fs;
      }
  }
#pragma unroll
  for (int x = 0; x < kOwn; ++x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[x][i] += __shfl_xor(o[x][i], 32);
    const int tok = (r0 + x) / t.heads, hd = (r0 + x) % t.heads;
    if (tok >= t.tokens || half) continue;
    const float inv = sum[x] > 0.0f || sum[x] != sum[x] ? 1.0f / sum[x] : 0.0f;
    const size_t at = ((size_t)(t.first + t.token + tok) * A.q_heads + t.head + hd) * kD;
    *(u32x2_a4 *)(A.o + at + 4 * l) = (u32x2){pack_bf16(o[x][0] * inv, o[x][1] * inv), pack_bf16(o[x][2] * inv, o[x][3] * inv)};
  }
}

}  // namespace

template <int KIND>
static hipError_t attend(const AttendArgs &a, const AttendPlan &p, hipStream_t st) {
  if (p.few) {
    const uint32_t units = (uint32_t)p.few_tiles * a.kv.heads * p.few_parts;
    hipLaunchKernelGGL(k_attend_few<KIND>, dim3(units * p.few_splits), dim3(64 * kFewWaves), 0, st, a, p);
    if (p.few_splits > 1) hipLaunchKernelGGL((k_attend_join<true, 1>), dim3(units * (kFewRows / 4)), dim3(256), 0, st, a, p);
  }
  if (p.many) {
    const uint32_t units = (uint32_t)p.many_tiles * a.kv.heads * p.many_parts;
    hipLaunchKernelGGL(k_attend_many<KIND>, dim3(units * p.many_splits), dim3(256), 0, st, a, p);
    if (p.many_splits > 4) hipLaunchKernelGGL((k_attend_join<false, 1>), dim3(units * (kManyRows / 4)), dim3(256), 0, st, a, p);
    else if (p.many_splits > 1) hipLaunchKernelGGL((k_attend_join<false, 8>), dim3(units * (kManyRows / 32)), dim3(256), 0, st, a, p);
  }
  return hipGetLastError();
}

hipError_t launch_attend(const AttendArgs &a, const AttendPlan &p, int kind, hipStream_t st) {
  return kind == 8 ? attend<8>(a, p, st) : attend<16>(a, p, st);
}

}  // namespace qdr
