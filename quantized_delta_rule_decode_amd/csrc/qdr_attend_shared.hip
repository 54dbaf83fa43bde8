// qdr_attend_shared.hip -- attention of new tokens over the paged cache where
// sequences share their first tokens: a group's rows go through the shared keys
// together, every sequence's rows through its own, in one launch; a second one
// joins what each row's passes left (qdr_cache.h).
#include "qdr_attend_tiles.h"
#include "qdr_cache.h"

namespace qdr {

namespace {

// Last i of 0 .. n - 1 with first(i) <= id, where first() does not fall; 64
// candidates at a time.  The whole wave calls it.
template <class F>
__device__ __forceinline__ int last_of(int n, int id, F first) {
  const int lane = (int)(threadIdx.x & 63);
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 63) >> 6, at = lane * step;
    const int count = __popcll(__ballot(at < len && first(lo + at) <= id));
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

// What a group's sequences share.
struct Share {
  bool bad;            // the group is skipped
  int tokens;          // shared ones
  int blocks;          // whole blocks of keys that its rows go through together; 0: each sequence by itself
  int begin;           // the group's first sequence
  int first, len;      // and its rows
};

__device__ __forceinline__ Share share_of(const SharedArgs &S, const SharedPlan &plan, int group) {
  const KvArgs &P = S.a.kv;
  Share r{true, 0, 0, 0, 0, 0};
  const int begin = S.group_cu[group], end = S.group_cu[group + 1];
  if (begin < 0 || end < begin || end > P.n) return r;
  r.begin = begin;
  r.tokens = S.shared[group];
  if (begin == end) {
    r.bad = false;
    return r;
  }
  const int room = room_of(P), c0 = P.cu[begin], c1 = P.cu[begin + 1], ce = P.cu[end], ctx = P.context[begin];
  r.bad = r.tokens < 0 || r.tokens > room || c0 < 0 || c1 < c0 || ce < c1 || ce > P.T || ctx > room || (long long)ctx - (c1 - c0) < r.tokens;
  r.first = c0;
  r.len = r.bad ? 0 : ce - c0;
  // sequences that fill tiles by themselves gain nothing, and would leave partial results
  const bool together = end - begin >= 2 && r.len < (long long)(end - begin) * plan.many_tokens;
  r.blocks = !r.bad && together ? r.tokens / kBlock : 0;
  return r;
}

__device__ __forceinline__ Share share_of_sequence(const SharedArgs &S, const SharedPlan &plan, int b) {
  Share none{false, 0, 0, 0, 0, 0};
  if (S.groups == 0) return none;
  const int group = last_of(S.groups, b, [&](int i) { return S.group_cu[i]; });
  if (b < S.group_cu[group] || b >= S.group_cu[group + 1]) return none;
  return share_of(S, plan, group);
}

// Counts, contexts and groups out of order or range, found once a call.
__device__ __forceinline__ void check_groups(const SharedArgs &S, const SharedPlan &plan) {
  const KvArgs &P = S.a.kv;
  check_counts(P);
  bool bad = false;
  for (int i = threadIdx.x; i < S.groups; i += 256) {
    const Share s = share_of(S, plan, i);
    bad = bad || s.bad;
    if (s.bad) continue;
    for (int b = S.group_cu[i] + 1; b < S.group_cu[i + 1]; ++b) {
      int first, len;
      if (rows_of(P.cu, P.T, b, &first, &len) && len > 0 && P.context[b] - len < s.tokens) bad = true;
    }
  }
  if (bad) atomicOr(P.err, kErrLength);
}

// Where a sequence's or group's many-row tiles begin.
__device__ __forceinline__ int many_place(const SharedArgs &S, const SharedPlan &plan, int first) {
  first = min(max(first, 0), S.a.kv.T);
  return first / plan.many_tokens + first / (plan.few_tokens + 1);
}

constexpr float kDone = -1.0f;     // in a row's first sum of its own: o is written

template <int KIND>
union Scratch {
  ManyShared<KIND> many[2];
  FewShared<kSharedWaves> few;
};

template <int KIND>
__global__ void __launch_bounds__(256, 2) k_attend_shared(SharedArgs S, SharedPlan plan) {
  __shared__ Scratch<KIND> sh;
  const AttendArgs &A = S.a;
  const KvArgs &P = A.kv;
  // whose tile, of what
  const int shared_many = plan.many_groups * plan.many_cuts * plan.many_parts * P.heads;
  const int shared_few = plan.few_groups * plan.few_cuts * plan.few_parts * P.heads;
  const int own_many = plan.many_tiles * plan.many_splits * plan.many_parts * P.heads;
  const int own_few = plan.few_tiles * plan.few_splits * plan.few_parts * P.heads;
  int x = blockIdx.x;
  bool prefix = true, few = false;
  if (x >= shared_many) {
    x -= shared_many;
    few = true;
    if (x >= shared_few) {
      x -= shared_few;
      prefix = few = false;
      if (x >= own_many) {
        x -= own_many;
        few = true;
        if (x >= own_few) {
          check_groups(S, plan);
          return;
        }
      }
    }
  }
  // heads change fastest: workgroups are dealt to the eight XCDs in turn, so the
  // tiles that read the same keys share few L2s
  const int kvh = x % P.heads;
  const int parts = few ? plan.few_parts : plan.many_parts, part = x / P.heads % parts;
  const int tiles = prefix ? (few ? plan.few_groups : plan.many_groups) : (few ? plan.few_tiles : plan.many_tiles);
  const int tile = x / (P.heads * parts) % tiles, split = x / (P.heads * parts) / tiles;
  const int splits = prefix ? (few ? plan.few_cuts : plan.many_cuts) : (few ? plan.few_splits : plan.many_splits);
  const int per = few ? plan.few_tokens : plan.many_tokens, most = few ? plan.few_heads : plan.many_heads;

  Tile t;
  int begin = 0, blocks;
  if (prefix) {
    const int group = few ? tile : last_of(plan.few_groups, tile, [&](int i) {
      const int b = S.group_cu[i];
      return b < 0 || b > P.n ? 0 : many_place(S, plan, P.cu[b]);
    });
    const Share s = share_of(S, plan, group);
    if (s.blocks == 0 || (s.len <= plan.few_tokens) != few) return;
    t.b = s.begin;
    t.first = s.first;
    t.len = s.len;
    t.token = few ? 0 : (tile - many_place(S, plan, s.first)) * per;
    if (t.token < 0 || t.token >= t.len) return;
    t.tokens = min(per, t.len - t.token);
    t.skipped = false;
    t.position = kMostContext;     // every row sees every key
    t.keys = s.blocks * kBlock;
    blocks = s.blocks;
  } else {
    t.b = few ? tile : last_of(P.n, tile, [&](int b) { return many_place(S, plan, P.cu[b]); });
    if (!rows_of(P.cu, P.T, t.b, &t.first, &t.len) || (t.len <= plan.few_tokens) != few) return;
    t.token = few ? 0 : (tile - many_place(S, plan, t.first)) * per;
    if (t.token < 0 || t.token >= t.len) return;
    t.tokens = min(per, t.len - t.token);
    const Share s = share_of_sequence(S, plan, t.b);
    const int ctx = P.context[t.b];
    t.skipped = s.bad || ctx < t.len || ctx > room_of(P) || ctx - t.len < s.tokens;
    t.position = ctx - t.len + t.token;
    t.keys = t.skipped ? 0 : t.position + t.tokens;
    begin = t.skipped ? 0 : s.blocks;
    blocks = (t.keys + kBlock - 1) / kBlock - begin;
  }
  t.head = kvh * plan.group + part * most;
  t.heads = min(most, plan.group - part * most);
  const int each = piece_blocks(blocks, splits, kSharedLeast);
  const int lo = begin + split * each, hi = min(lo + each, begin + blocks);
  const bool alone = !prefix && begin == 0 && each >= blocks;   // the rows' only pass
  if (alone && split > 0) return;

  // The rows' statistics also where a pass has no keys, and, by the last piece, in
  // the places that the other kind of tiles has more pieces for; where nothing is
  // shared, by the first piece, in those of shared keys.
  const int place = prefix ? split : plan.shared_places + split;
  const int end = split + 1 < splits ? place + 1 : prefix ? plan.shared_places : plan.places;
  const bool clears = !prefix && begin == 0 && split == 0;
  const int l = threadIdx.x & 63, g = l >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  auto note = [&](size_t at, float m, float sum) {
    float *to = S.stats + at / kD * plan.places * 2;
    if (alone) {
      to[2 * plan.shared_places + 1] = kDone;
      return;
    }
    *(f32x2 *)(to + 2 * place) = (f32x2){m, sum};
    for (int p = place + 1; p < end; ++p) *(f32x2 *)(to + 2 * p) = (f32x2){kNone, 0.0f};
    if (clears)
      for (int p = 0; p < plan.shared_places; ++p) *(f32x2 *)(to + 2 * p) = (f32x2){kNone, 0.0f};
  };
  // sixteen channels' four of a lane: 16 d + 4 g ..
  auto put = [&](size_t at, int d, f32x4 y, float sum) {
    if (alone) {
      const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
      *(u32x2_a4 *)(A.o + at + 16 * d + 4 * g) = (u32x2){pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
    } else if (lo < hi) {
      *(f32x4 *)(A.part + (at / kD * plan.places + place) * kD + 16 * d + 4 * g) = y;
    }
  };
  if (few) {
    FewOut<kSharedWaves> out;
    few_tile<KIND, kSharedWaves>(A, t, kvh, lo, hi, sh.few, out);
    if (!out.row) return;
#pragma unroll
    for (int y = 0; y < 8 / kSharedWaves; ++y) put(out.at, 8 / kSharedWaves * w + y, out.o[y], out.sum);
    if (w == 0 && g == 0) note(out.at, out.m, out.sum);
  } else {
    ManyOut out;
    many_tile<KIND>(A, t, kvh, lo, hi, sh.many, out);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (!out.row[c]) continue;
#pragma unroll
      for (int d = 0; d < 8; ++d) put(out.at[c], d, out.o[c][d], out.sum[c]);
      if (g == 0) note(out.at[c], out.m[c], out.sum[c]);
    }
  }
}

// Joins a row's passes (64 at most): a wave a row, a lane a pass's maximum and
// sum; then half a wave takes four channels a lane of every other pass that had
// keys, sixteen of them on their way at once.
__global__ void __launch_bounds__(256) k_join_shared(SharedArgs S, SharedPlan plan) {
  constexpr int kLoads = 8;
  const AttendArgs &A = S.a;
  const KvArgs &P = A.kv;
  const int l = threadIdx.x & 63, half = l >> 5;
  const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t token = row / A.q_heads;
  if (token < P.cu[0] || token >= P.cu[P.n] || token >= P.T) return;
  const f32x2 own = *(const f32x2 *)(S.stats + (row * plan.places + min(l, plan.places - 1)) * 2);
  if (__shfl(own[1], plan.shared_places) == kDone) return;
  const bool live = l < plan.places && !(own[0] == kNone && own[1] == 0.0f);
  const float top = wave_max(live ? own[0] : kNone);
  const float f = live ? ex2(own[0] - (top == kNone ? 0.0f : top)) : 0.0f;
  float sum = live ? own[1] * f : 0.0f;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  f32x4 o = (f32x4){0, 0, 0, 0};
  uint64_t left = __ballot(live);
  const float *from = A.part + row * plan.places * kD + 4 * (l & 31);
  while (left) {
    f32x4 y[kLoads];
    int at[kLoads];
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      // the next two passes, one a half; behind the last one the last again, without weight
      const int a = left ? __builtin_ctzll(left) : 0;
      const bool one = left != 0;
      left &= left - 1;
      const int b = left ? __builtin_ctzll(left) : a;
      const bool two = left != 0;
      left &= left - 1;
      at[x] = half ? (two ? b : -1) : (one ? a : -1);
      y[x] = *(const f32x4 *)(from + (size_t)(half ? b : a) * kD);
    }
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const float fs = __shfl(f, at[x] < 0 ? 0 : at[x]);
      if (at[x] >= 0) o += y[x] * fs;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] += __shfl_xor(o[i], 32);
  if (half) return;
  const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
  *(u32x2_a4 *)(A.o + row * kD + 4 * l) = (u32x2){pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
}

template <int KIND>
hipError_t attend_shared(const SharedArgs &s, const SharedPlan &p, hipStream_t st) {
  const int heads = s.a.kv.heads;
  const uint32_t groups = (uint32_t)((p.many_groups * p.many_cuts + p.many_tiles * p.many_splits) * p.many_parts * heads) +
                          (uint32_t)((p.few_groups * p.few_cuts + p.few_tiles * p.few_splits) * p.few_parts * heads);
  hipLaunchKernelGGL(k_attend_shared<KIND>, dim3(groups + 1), dim3(256), 0, st, s, p);
  const int64_t rows = (int64_t)s.a.kv.T * s.a.q_heads;
  hipLaunchKernelGGL(k_join_shared, dim3((uint32_t)((rows + 3) / 4)), dim3(256), 0, st, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_shared(const SharedArgs &s, const SharedPlan &p, int kind, hipStream_t st) {
  return kind == 8 ? attend_shared<8>(s, p, st) : attend_shared<16>(s, p, st);
}

}  // namespace qdr
