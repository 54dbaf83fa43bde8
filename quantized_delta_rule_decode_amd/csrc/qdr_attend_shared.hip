// qdr_attend_shared.hip -- attention of new tokens over the paged cache where
// sequences share their first tokens: a group's rows go through the shared keys
// together, every sequence's rows through its own, in one launch whose
// workgroups have equal parts of the groups' work or a sequence's tile; a second
// one joins what each row's passes left (qdr_cache.h).  With m, s and y a pass's
// maximum, sum of weights and unnormalised result: M = max m,
// o = sum 2^(m - M) y / sum 2^(m - M) s.
//
// 64 sequences with up to 700 tokens each behind 16384 shared ones, 32 and 8 heads,
// 8-bit: 62 to 65 us (every sequence by itself 233): 57 for the passes (17.7 GFLOP and
// 108 MB, 15 or 20 us at the card's rates), in which the vector units are
// busy half of the time and the matrix cores a fifth, the rest being the start of
// the line, a part's first blocks and results that leave at its end; 8 for the
// join of 27 MB of results, fp32 because each is one of many that are added.
// bfloat16 75 us for 208 MB over changing keys (55 and 8 where the caches hold them).
// 32 sequences of up to 20 new tokens behind 4 prefixes of up to 4100, 32 and 8
// heads: bfloat16 100 us for 27 GFLOP, 8-bit 105: passes 68 and 75, join 32.  Of up
// to 100: 264 and 329 us for 140 GFLOP (529 and 425 TFLOP/s), none of it together
// (share_of): every sequence's rows go through the prefix by themselves, as in
// qdr_kv_attend, in tiles that sequences of 50 to 100 tokens fill to about 85%, and
// an empty line and a join that finds every row done cost some 5 us.  Two sequences
// behind 300: 12 us, two launches' latency.
#include "qdr_attend_tiles.h"
#include "qdr_cache.h"

namespace qdr {

namespace {

constexpr int kCell = kD + 2;   // floats of a row's result: 128 sums, maximum, sum of weights
constexpr int kItems = 256;     // groups that a workgroup has at hand

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
  int begin, end;      // its sequences
  int first, len;      // its rows
};

// (The loads of a step do not wait for each other: what may be out of range is
// cut to it before, and looked at behind.)
__device__ __forceinline__ Share share_of(const SharedArgs &S, const SharedPlan &plan, int begin, int end, int tokens) {
  const KvArgs &P = S.a.kv;
  const bool order = begin >= 0 && end >= begin && end <= P.n;
  const int b0 = order ? min(begin, P.n - 1) : 0, b1 = order ? end : 0;
  const int c0 = P.cu[b0], c1 = P.cu[b0 + 1], ce = P.cu[b1], ctx = P.context[b0], room = room_of(P);
  const bool none = order && begin == end;
  Share r;
  r.tokens = tokens;
  r.begin = b0;
  r.end = b1;
  const bool counts = c0 >= 0 && c1 >= c0 && ce >= c1 && ce <= P.T;
  r.bad = !order || (!none && (tokens < 0 || tokens > room || !counts || ctx > room || (int64_t)ctx - (c1 - c0) < tokens));
  r.first = c0;
  r.len = r.bad || none ? 0 : ce - c0;
  // Sequences that fill tiles by themselves go so: dealt together their rows would
  // take fewer tiles (those of 33 tokens of four heads a key head half as many), but
  // leave partial results to join.  Measured (us a call, by themselves / together), 32
  // and 8 heads, bfloat16, then 8-bit, tokens of each sequence; 4 groups of 8 behind
  // 4100: 32 201 / 172, 240 / 181; 33 162 / 166, 202 / 179; 64 256 / 278, 315 / 286;
  // 100 314 / 379, 393 / 422; 250 634 / 919, 766 / 1039; 50 to 100 264 / 276, 329 / 298.
  // 8 behind 16384: 32 108 / 119, 125 / 128; 33 177 / 138, 219 / 156; 65 311 / 216,
  // 394 / 247; 100 319 / 305, 402 / 340; 250 585 / 633, 724 / 777.  So the rule holds
  // for long chunks, and loses just above a whole number of tiles and with 8 bits.
  const bool together = plan.ranges > 0 && r.end - r.begin >= 2 && r.len < (int64_t)(r.end - r.begin) * plan.many_tokens;
  r.blocks = r.len > 0 && together ? tokens / kBlock : 0;
  return r;
}

// The group of sequence b: the last i with group_cu[i] <= b.
template <class F>
__device__ __forceinline__ int group_of_sequence(int groups, int b, F group_cu) {
  int lo = 0, len = groups;
  while (len > 1) {
    const int half = len >> 1;
    const bool behind = group_cu(lo + half) <= b;
    lo = behind ? lo + half : lo;
    len = behind ? len - half : half;
  }
  return lo;
}

// Counts, contexts and groups out of order or range, found once a call.
__device__ __forceinline__ void check_groups(const SharedArgs &S, const SharedPlan &plan) {
  const KvArgs &P = S.a.kv;
  check_counts(P);
  bool bad = false;
  for (int i = threadIdx.x; i < S.groups; i += 256) bad = bad || share_of(S, plan, S.group_cu[i], S.group_cu[i + 1], S.shared[i]).bad;
  for (int b = threadIdx.x; b < P.n && S.groups > 0; b += 256) {
    const int group = group_of_sequence(S.groups, b, [&](int i) { return S.group_cu[i]; });
    int first, len;
    if (b >= S.group_cu[group] && b < S.group_cu[group + 1] && rows_of(P.cu, P.T, b, &first, &len) && len > 0 && P.context[b] - len < S.shared[group]) bad = true;
  }
  if (bad) atomicOr(P.err, kErrLength);
}

// The rows of a group and its shared keys, or of a sequence.
struct Item {
  double start;        // where a group's tiles begin in the line (a whole number)
  int tiles;           // 0: no rows
  int b;               // whose page table
  int first, len;      // rows
  int position;        // of row 0; kMostContext: every row sees every key
  int begin, blocks;   // blocks of keys: a sequence's own begin there; a group's
  int flags;
  int members;         // a group's sequences
};
constexpr int kFew = 1, kSkipped = 4, kPooled = 8;   // kPooled: its rows have shared keys too

// What a workgroup, a tile and each of its blocks cost, in 0.1 us, with the
// results they leave.  64 sequences behind 16384 tokens, 8-bit and bfloat16, and
// 8 x 8 of four new tokens behind 2048 (us a call): 60 and 60 63.2, 75.5, 52.8; 100
// and 60 61.3, 73.8, 52.2; 140 and 60 61.3, 64.0, 49.1; 140 and 100 61.8, 63.8, 48.1.
constexpr int kGroupCost = 140, kTileCost = 100, kLeastCost = 100;   // (the last: least of a part)
template <int KIND>
__device__ __forceinline__ double block_cost(int flags) { return flags & kFew ? (KIND == 8 ? 8.0 : 14.0) : 13.0; }
template <int KIND>
__device__ __forceinline__ double tile_cost(int flags, int blocks) { return kTileCost + blocks * block_cost<KIND>(flags); }
// What `blocks` of keys of a sequence of `len` tokens' own cost a key head.
template <int KIND>
__device__ __forceinline__ double own_cost(const SharedPlan &plan, double len, double blocks) {
  const bool few = len <= plan.few_tokens;
  return few ? plan.few_parts * blocks * (KIND == 8 ? 4.0 : 7.0) : ceil(len * plan.many_inverse) * plan.many_parts * blocks * block_cost<KIND>(0);
}

__device__ __forceinline__ Item item_of_group(const SharedArgs &S, const SharedPlan &plan, int i) {
  Item t{};
  if (i >= S.groups) return t;
  const Share share = share_of(S, plan, S.group_cu[i], S.group_cu[i + 1], S.shared[i]);
  t.b = share.begin;
  t.first = share.first;
  t.len = share.blocks ? share.len : 0;
  t.position = kMostContext;
  t.blocks = share.blocks;
  t.members = share.end - share.begin;
  const bool few = t.len <= plan.few_tokens;
  t.flags = few ? kFew : 0;
  t.tiles = t.len == 0 ? 0 : few ? plan.few_parts : (t.len + plan.many_tokens - 1) / plan.many_tokens * plan.many_parts;
  return t;
}

__device__ __forceinline__ Item item_of_sequence(const SharedArgs &S, const SharedPlan &plan, int b) {
  const KvArgs &P = S.a.kv;
  Item t{};
  const int s = P.cu[b], e = P.cu[b + 1], ctx = P.context[b];
  Share share{false, 0, 0, 0, 0, 0, 0};
  if (S.groups > 0) {
    const int group = last_of(S.groups, b, [&](int i) { return S.group_cu[i]; });
    const int g0 = S.group_cu[group], g1 = S.group_cu[group + 1];
    if (b >= g0 && b < g1) share = share_of(S, plan, g0, g1, S.shared[group]);
  }
  t.b = b;
  t.first = s;
  t.len = s >= 0 && e >= s && e <= P.T ? e - s : 0;
  const bool skipped = share.bad || ctx < t.len || ctx > room_of(P) || ctx - t.len < share.tokens;
  t.flags = (skipped ? kSkipped : share.blocks ? kPooled : 0) | (t.len <= plan.few_tokens ? kFew : 0);
  t.position = ctx - t.len;
  t.begin = skipped ? 0 : share.blocks;
  return t;
}

// A token's passes over keys: parts r0 .. r1 of the line (kPieces: pieces 0 .. r1
// of sequence r0's few rows or of many-row tile r0), and the row of its first head
// of the part in their tile.
struct Passes {
  int r0, r1, row;
  uint32_t flags;      // kFew, kPooled, kPieces; kDone: o is written; passes over own keys: the sequence above
};
constexpr int kDone = 16, kPieces = 128, kSequenceShift = 8;   // (n is under 2^24)

// The line of the groups' work, cut into ranges of `step` (rounded down to whole costs,
// the same everywhere).
struct Line {
  double total, own, step, inverse;   // own: the cost of sequences' own keys
  int ranges, range;       // of the workgroup
  double a, b;             // its part
};
// Parts of a line of length C, while the sequences' workgroups (A in all) have
// the other of M places: both end at once where (G + C / x) (M - x) = A with G a
// workgroup's cost, and no part is shorter than kLeastCost.
__device__ __forceinline__ int ranges_of(int most, double total, double own) {
  const double b = 0.5 * (own + total - (double)kGroupCost * most);
  const double x = (sqrt(b * b + (double)kGroupCost * most * total) - b) * (1.0 / kGroupCost);
  return (int)fmax(fmin(fmin((double)most, ceil(x)), ceil(total * (1.0 / kLeastCost))), 1.0);
}
__device__ __forceinline__ double range_begin(const Line &line, int r) { return r < line.ranges ? floor(r * line.step) : line.total; }
__device__ __forceinline__ int range_at(const Line &line, double x) {
  int r = min((int)(x * line.inverse), line.ranges - 1);
  if (range_begin(line, r) > x) --r;
  if (range_begin(line, r + 1) <= x) ++r;
  return min(max(r, 0), line.ranges - 1);
}

// One pass: a tile over blocks lo .. hi.
struct Job {
  Tile t;
  int lo, hi;
  int flags;               // of the item; kAlone: the rows' only pass; kCut: one of several over the tile
  size_t whole, cell;      // places in the workspace: results by row, and of the workgroup's cut tile
  Passes *info, passes;    // of the tile's first token, and what to write there (NULL: another workgroup does)
  int info_step;
};
constexpr int kAlone = 32, kCut = 64;

template <int KIND>
struct Scratch {
  union {
    ManyShared<KIND> many[2];
    FewShared<kSharedWaves> few;
  };
  Item items[kItems];
  double sums[4][2];
  int2 at;                 // item and tile where the part begins in it
  double base;             // where this chunk of items begins in the line
  SharedArgs args;
  SharedPlan plan;
  Line line;
  Job job;
};

// Sum of x over the threads before this one, of 256; *all and *all_y: of x and y
// over every thread.
__device__ __forceinline__ double sum_before(double x, double y, double (*lds)[2], double *all, double *all_y) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  double s = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double before = __shfl_up(s, d);
    if (lane >= d) s += before;
    y += __shfl_xor(y, d);
  }
  __syncthreads();
  if (lane == 63) {
    lds[w][0] = s;
    lds[w][1] = y;
  }
  __syncthreads();
  double before = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) before += i < w ? lds[i][0] : 0.0;
  *all = lds[0][0] + lds[1][0] + lds[2][0] + lds[3][0];
  *all_y = lds[0][1] + lds[1][1] + lds[2][1] + lds[3][1];
  return before + s - x;
}

__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Tile k of a group as the workgroup's next pass.
template <int KIND>
__device__ __forceinline__ void make_job(const SharedArgs &S, const SharedPlan &plan, const Line &line, const Item &it, int k, int kvh, Job &job) {
  const KvArgs &P = S.a.kv;
  const int flags = it.flags, blocks = it.blocks;
  const bool few = flags & kFew;
  const int parts = few ? plan.few_parts : plan.many_parts, per = few ? plan.few_tokens : plan.many_tokens, most = few ? plan.few_heads : plan.many_heads;
  const double each = tile_cost<KIND>(flags, blocks), from = it.start + k * each;
  const int r0 = from >= line.a ? line.range : range_at(line, from);
  const int r1 = from + each <= line.b ? line.range : range_at(line, from + each - 1);
  const double per_block = 1.0 / block_cost<KIND>(flags);
  auto cut = [&](double at) { return (int)fmin(fmax(ceil((at - from - kTileCost) * per_block), 0.0), (double)blocks); };
  const int tile = parts == 1 ? k : k / parts, part = k - tile * parts;
  Tile t;
  t.b = it.b;
  t.first = it.first;
  t.len = it.len;
  t.token = tile * per;
  t.tokens = min(per, it.len - t.token);
  t.head = kvh * plan.group + part * most;
  t.heads = min(most, plan.group - part * most);
  t.skipped = false;
  t.position = kMostContext;
  t.keys = blocks * kBlock;
  job.t = t;
  job.lo = r0 == line.range ? 0 : cut(line.a);
  job.hi = r1 == line.range ? blocks : cut(line.b);
  job.flags = flags | (r0 == r1 ? 0 : kCut);
  job.whole = 0;
  job.cell = plan.cut + (size_t)((line.range * P.heads + kvh) * 2 + (r0 == line.range)) * plan.slot_rows * kCell;
  // each token's passes are written down once
  Passes *info = (Passes *)(S.a.part + plan.info);
  job.info = kvh == 0 && line.range == r0 ? info + (size_t)(t.first + t.token) * plan.few_parts + part : nullptr;
  job.passes = {r0, r1, 0, (uint32_t)(flags & kFew)};
  job.info_step = plan.few_parts;
}

// Piece `split` of a sequence's tile from `token` on, whose number is `tile`;
// false: there is none.
__device__ __forceinline__ bool make_piece(const SharedArgs &S, const SharedPlan &plan, const Item &it, int tile, int token, int part, int split, int kvh, Job &job) {
  const KvArgs &P = S.a.kv;
  const bool few = it.flags & kFew;
  const int most = few ? plan.few_heads : plan.many_heads, splits = few ? plan.few_splits : plan.many_splits, parts = few ? plan.few_parts : plan.many_parts;
  Tile t;
  t.b = it.b;
  t.first = it.first;
  t.len = it.len;
  t.token = token;
  t.tokens = min(few ? plan.few_tokens : plan.many_tokens, it.len - token);
  t.head = kvh * plan.group + part * most;
  t.heads = min(most, plan.group - part * most);
  t.skipped = it.flags & kSkipped;
  t.position = it.position + token;
  t.keys = t.skipped ? 0 : t.position + t.tokens;
  const int blocks = (t.keys + kBlock - 1) / kBlock - it.begin;
  const int each = piece_blocks(blocks, splits, few ? kSharedLeast : kManyLeast), pieces = max((blocks + each - 1) / each, 1);
  if (split >= pieces) return false;
  const bool alone = pieces == 1 && !(it.flags & kPooled);
  job.t = t;
  job.lo = it.begin + split * each;
  job.hi = min(job.lo + each, it.begin + blocks);
  job.flags = it.flags | (alone ? kAlone : 0) | (pieces == 1 ? 0 : kCut);
  job.whole = plan.cut / 2;
  job.cell = (few ? plan.few_pieces : plan.many_pieces) + ((((size_t)tile * P.heads + kvh) * parts + part) * splits + split) * ((few ? kFewRows : kManyRows) * kCell);
  Passes *info = (Passes *)(S.a.part + plan.info) + (size_t)P.T * plan.few_parts;
  job.info = kvh == 0 && split == 0 ? info + (size_t)(t.first + token) * plan.few_parts + part : nullptr;
  const int kept = (it.flags & (kFew | kPooled)) | (alone ? kDone : 0) | (pieces == 1 ? 0 : kPieces);
  job.passes = {pieces == 1 ? 0 : tile, pieces - 1, 0, (uint32_t)kept | (uint32_t)it.b << kSequenceShift};
  job.info_step = plan.few_parts;
  return true;
}

// Where a pass leaves its rows, read from the job when its tile is done.
struct Results {
  uint16_t *o;
  float *part;         // by row, or by the tile's rows
  int flags;
  bool keys;
  __device__ __forceinline__ float *place(size_t at, int row) const { return part + (flags & kCut ? (size_t)row : at / kD) * kCell; }
  // channels c .. c + 3 of a row
  __device__ __forceinline__ void put(size_t at, int row, int c, f32x4 y, float sum) const {
    if (flags & kAlone) {
      const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
      *(u32x2_a4 *)(o + at + c) = (u32x2){pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
    } else if (keys) {
      float *to = place(at, row) + c;
      *(f32x2 *)to = (f32x2){y[0], y[1]};
      *(f32x2 *)(to + 2) = (f32x2){y[2], y[3]};
    }
  }
  __device__ __forceinline__ void note(size_t at, int row, float m, float sum) const {
    if (!(flags & kAlone)) *(f32x2 *)(place(at, row) + kD) = (f32x2){m, sum};
  }
};
__device__ __forceinline__ Results results_of(const AttendArgs &A, const Job &job) {
  asm volatile("" ::: "memory");       // not before the tile, which has no registers for it
  Results r;
  r.o = A.o;
  r.flags = scalar(job.flags);
  r.keys = scalar(job.lo) < scalar(job.hi);
  // (from the kernel's argument: the compiler knows that as global memory)
  const size_t at = r.flags & kCut ? job.cell : job.whole;
  r.part = A.part + ((size_t)(uint32_t)scalar((int)(at >> 32)) << 32 | (uint32_t)scalar((int)at));
  return r;
}

template <int KIND>
__device__ __forceinline__ void pass(const AttendArgs &A, int kvh, Scratch<KIND> &sh) {
  // (not known to be the same in every pass: what follows from it is made anew
  // instead of kept in registers that a pass has not got)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int l = tid & 63, g = l >> 4, w = scalar(tid >> 6);
  Tile t;
  t.b = scalar(sh.job.t.b);
  t.first = scalar(sh.job.t.first);
  t.token = scalar(sh.job.t.token);
  t.tokens = scalar(sh.job.t.tokens);
  t.head = scalar(sh.job.t.head);
  t.heads = scalar(sh.job.t.heads);
  t.position = scalar(sh.job.t.position);
  t.keys = scalar(sh.job.t.keys);
  const int lo = scalar(sh.job.lo), hi = scalar(sh.job.hi);
  if (sh.job.info && tid < t.tokens) {
    Passes p = sh.job.passes;
    p.row = tid * t.heads;
    sh.job.info[(size_t)tid * sh.job.info_step] = p;
  }
  if (scalar(sh.job.flags) & kFew) {
    FewOut<kSharedWaves> out;
    few_tile<KIND, kSharedWaves, KIND == 8>(A, t, tid, kvh, lo, hi, sh.few, out);
    const Results to = results_of(A, sh.job);
    if (!out.row) return;
#pragma unroll
    for (int y = 0; y < 8 / kSharedWaves; ++y) to.put(out.at, l & 15, 16 * (8 / kSharedWaves * w + y) + 4 * g, out.o[y], out.sum);
    if (w == 0 && g == 0) to.note(out.at, l & 15, out.m, out.sum);
  } else {
    ManyOut out;
    many_tile<KIND, true>(A, t, tid, kvh, lo, hi, sh.many, out);
    const Results to = results_of(A, sh.job);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (!out.row[c]) continue;
      const int row = 32 * w + 16 * c + (l & 15);
#pragma unroll
      for (int d = 0; d < 8; ++d) to.put(out.at[c], row, 16 * d + 4 * g, out.o[c][d], out.sum[c]);
      if (g == 0) to.note(out.at[c], row, out.m[c], out.sum[c]);
    }
  }
}

// Where a sequence's many-row tiles begin.
__device__ __forceinline__ int many_place(const SharedArgs &S, const SharedPlan &plan, int b, int first) {
  first = min(max(first, 0), S.a.kv.T);
  return first / plan.many_tokens + (plan.by_tokens ? first / (plan.few_tokens + 1) : b);
}

template <int KIND>
__global__ void __launch_bounds__(256, 2) k_attend_shared(SharedArgs S, SharedPlan plan) {
  __shared__ Scratch<KIND> sh;
  const int tid = threadIdx.x;
  // heads change fastest: workgroups are dealt to the eight XCDs in turn, so the
  // tiles that read the same keys share few L2s
  const int kvh = blockIdx.x % S.a.kv.heads;
  int place = blockIdx.x / S.a.kv.heads;
  if (place >= plan.ranges) {
    // sequences' own keys: few rows, then many, those with most keys first
    place -= plan.ranges;
    const bool few = place < S.a.kv.n * plan.few_parts * plan.few_splits;
    if (!few) place -= S.a.kv.n * plan.few_parts * plan.few_splits;
    const int parts = few ? plan.few_parts : plan.many_parts, splits = few ? plan.few_splits : plan.many_splits;
    const int part = place % parts, split = place / parts % splits;
    int tile = place / (parts * splits), b = tile, token = 0;
    if (!few) {
      tile = plan.many_tiles - 1 - tile;
      if (tile < 0) {      // one workgroup more
        check_groups(S, plan);
        return;
      }
      b = last_of(S.a.kv.n, tile, [&](int i) { return many_place(S, plan, i, S.a.kv.cu[i]); });
      token = tile - many_place(S, plan, b, S.a.kv.cu[b]);
    }
    const Item mine = item_of_sequence(S, plan, b);
    token *= few ? 1 : plan.many_tokens;
    if (mine.len == 0 || (mine.len <= plan.few_tokens) != few || token < 0 || token >= mine.len) return;
    Job job;
    if (!make_piece(S, plan, mine, tile, token, part, split, kvh, job)) return;
    if (tid == 0) sh.job = job;
  } else if (tid == 0) {
    // (a pass has no registers to spare: what deals out the work is at hand in LDS)
    sh.args = S;
    sh.plan = plan;
    sh.base = 0;
    sh.line.total = sh.line.own = 0;
  }
  __syncthreads();
  // Every workgroup of the line makes it by itself, 256 groups at a time: once
  // through for its length, and once (the only chunk is still at hand) for the
  // groups of its part.
  const bool line_part = (int)(blockIdx.x / S.a.kv.heads) < plan.ranges;
  const int chunks = line_part ? (S.groups + kItems - 1) / kItems : 1;
#pragma unroll 1
  for (int c = 0; c < 2 * chunks; ++c) {
    int x = 0, k = 0;
    double all = 0;
    bool here = true;
    if (line_part) {
      double own = 0, all_own = 0;
      if (c == 0)
        for (int b = tid; b < sh.args.a.kv.n; b += 256) {
          const KvArgs &P = sh.args.a.kv;
          const int len = min(max(P.cu[b + 1] - P.cu[b], 0), P.T), ctx = min(max(P.context[b], 0), room_of(P));
          own += len == 0 ? 0.0 : kGroupCost + own_cost<KIND>(sh.plan, len, ctx >> 5);
        }
      Item mine = item_of_group(sh.args, sh.plan, (c < chunks ? c : c - chunks) * kItems + tid);
      if (c < chunks && mine.tiles > 0) own -= mine.members * own_cost<KIND>(sh.plan, (double)mine.len / mine.members, mine.blocks);
      const double before = sum_before(mine.tiles * tile_cost<KIND>(mine.flags, mine.blocks), own, sh.sums, &all, &all_own);
      if (c < chunks) {
        if (tid == 0) {
          Line line = sh.line;
          line.total += all;
          line.own += all_own;
          if (c + 1 == chunks) {
            const int range = blockIdx.x / sh.args.a.kv.heads;
            line.ranges = ranges_of(sh.plan.ranges, line.total, line.own);
            line.step = line.total / line.ranges;
            line.inverse = line.ranges / line.total;
            line.range = range;
            line.a = range < line.ranges ? range_begin(line, range) : line.total;
            line.b = range < line.ranges ? range_begin(line, range + 1) : line.total;
          }
          sh.line = line;
        }
        __syncthreads();
        if (c + 1 < chunks) continue;
        if (sh.line.total == 0 || sh.line.a >= sh.line.b) return;
        if (chunks > 1) continue;
      }
      here = sh.base + all > sh.line.a;
      if (here) {
        // the first group that ends behind the part's beginning, and from there on
        const double into = sh.line.a - (sh.base + before), each = tile_cost<KIND>(mine.flags, mine.blocks);
        mine.start = sh.base + before;
        sh.items[tid] = mine;
        if (into >= 0 && into < mine.tiles * each) {
          k = (int)(into / each);
          if (k * each > into) --k;
          if ((k + 1) * each <= into) ++k;
          sh.at = make_int2(tid, k);
        } else if (tid == 0 && into < 0) {
          sh.at = make_int2(0, 0);
        }
        __syncthreads();
        x = sh.at.x;
        k = sh.at.y;
        x = scalar(x);
        k = scalar(k);
      }
    }
    while (here) {
      if (line_part) {
        if (x == kItems || sh.items[x].start >= sh.line.b) break;
        if (k >= scalar(sh.items[x].tiles)) {
          ++x;
          k = 0;
          continue;
        }
        if (sh.items[x].start + k * tile_cost<KIND>(sh.items[x].flags, sh.items[x].blocks) >= sh.line.b) break;
        if (tid == 0) make_job<KIND>(sh.args, sh.plan, sh.line, sh.items[x], k, kvh, sh.job);
        ++k;
        __syncthreads();
      }
      pass<KIND>(S.a, kvh, sh);
      if (!line_part) return;
      __syncthreads();
    }
    if (chunks == 1) return;
    __syncthreads();
    if (tid == 0) sh.base += all;
    __syncthreads();
    if (sh.base >= sh.line.b) return;
  }
}

// Joins the passes of OWN rows a wave, those over shared keys first: a lane has a
// pass's maximum and sum; then half a wave takes four channels a lane of every
// other pass, sixteen of them on their way at once.
template <int OWN>
__global__ void __launch_bounds__(256) k_join_shared(SharedArgs S, SharedPlan plan) {
  constexpr int kLoads = 8;
  const AttendArgs &A = S.a;
  const KvArgs &P = A.kv;
  const int l = threadIdx.x & 63, half = l >> 5;
  const int begin = P.cu[0], end = min(P.cu[P.n], P.T);
#pragma unroll 1
  for (int i = 0; i < OWN; ++i) {
    const int64_t row = ((int64_t)blockIdx.x * 4 + scalar((int)threadIdx.x >> 6)) * OWN + i;
    const int64_t token = row / A.q_heads;
    if (token >= P.T) continue;
    const int head = (int)(row - token * A.q_heads), kvh = head / plan.group, h = head - kvh * plan.group;
    const Passes *shared = (const Passes *)(A.part + plan.info) + token * plan.few_parts, *own = shared + (size_t)P.T * plan.few_parts;
    // (all that is read before the cells, at once)
    Passes o = own[0], first = shared[0], s{0, -1, 0, 0u};
    if (token < begin || token >= end) continue;
    if (o.flags & kDone && plan.few_parts == 1) {
      if (OWN > 1) i += min((int64_t)(OWN - 1 - i), (int64_t)A.q_heads - 1 - head);   // and the token's other rows are
      continue;
    }
    int part = 0;
    auto at_part = [&](const Passes *from, Passes &p) {
      const int heads = p.flags & kFew ? plan.few_heads : plan.many_heads;
      part = h / heads;
      if (part > 0) p = from[part];
      p.row += h - part * heads;
    };
    if (o.flags & kPooled) {
      s = first;
      at_part(shared, s);
    }
    at_part(own, o);
    if (o.flags & kDone) continue;
    // Counts out of order leave rows without passes, whose places hold what an
    // earlier call left: a row is written where its sequence has it in this one.
    const int b = (int)(o.flags >> kSequenceShift), at_b = min(b, P.n - 1), c0 = P.cu[at_b], c1 = P.cu[at_b + 1];
    const bool has = b < P.n && c0 >= 0 && c0 <= token && token < c1 && c1 <= P.T;
    const bool pieces = o.flags & kPieces;
    auto bad = [&](const Passes &p) { return p.r0 < 0 || p.r0 > p.r1 || p.r1 >= plan.ranges || p.row < 0 || p.row >= plan.slot_rows; };
    const bool own_few = o.flags & kFew;
    const int rows = own_few ? kFewRows : kManyRows, splits = own_few ? plan.few_splits : plan.many_splits, parts = own_few ? plan.few_parts : plan.many_parts;
    if (pieces ? o.r0 < 0 || o.r0 >= (own_few ? P.n : plan.many_tiles) || o.r1 < 0 || o.r1 >= splits || o.row < 0 || o.row >= rows : o.r0 != 0 || o.r1 != 0) continue;
    if (o.flags & kPooled && (plan.ranges == 0 || bad(s))) continue;
    if (!pieces && !(o.flags & kPooled)) continue;
    const int ns = s.r1 - s.r0 + 1, passes = ns + o.r1 + 1;
    const float *own_cell = pieces ? A.part + (own_few ? plan.few_pieces : plan.many_pieces) + ((((size_t)o.r0 * P.heads + kvh) * parts + part) * splits * rows + o.row) * kCell
                                   : A.part + plan.cut / 2 + row * kCell;
    auto cell = [&](int p) -> const float * {
      if (p >= ns) return own_cell + (size_t)(p - ns) * rows * kCell;
      const int r = s.r0 + p;
      return s.r0 == s.r1 ? A.part + row * kCell : A.part + plan.cut + ((size_t)((r * P.heads + kvh) * 2 + (r == s.r0)) * plan.slot_rows + s.row) * kCell;
    };
    float top = kNone, sum = 0.0f;
    f32x4 y = (f32x4){0, 0, 0, 0};
    for (int p0 = 0; p0 < passes; p0 += 64) {
      const f32x2 x = *(const f32x2 *)(cell(min(p0 + l, passes - 1)) + kD);
      const bool in = p0 + l < passes;
      const float top1 = fmaxf(top, wave_max(in ? x[0] : kNone));
      const float ref = top1 == kNone ? 0.0f : top1, fade = ex2(top - ref);
      top = top1;
      const float f = in ? ex2(x[0] - ref) : 0.0f;
      // (a pass without keys left no result to read)
      uint64_t left = __ballot(in && !(x[0] == kNone && x[1] == 0.0f));
      float add = in ? x[1] * f : 0.0f;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) add += __shfl_xor(add, d);
      sum = sum * fade + add;
      y *= fade;
      while (left) {
        f32x2 z[kLoads][2];
        int at[kLoads];
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          // the next two, one a half; behind the last one the first again, without weight
          const int one = left ? __builtin_ctzll(left) : -1;
          left &= left - 1;
          const int two = left ? __builtin_ctzll(left) : -1;
          left &= left - 1;
          at[j] = half ? two : one;
          const float *from = cell(p0 + max(at[j], 0)) + 4 * (l & 31);
          z[j][0] = *(const f32x2 *)from;
          z[j][1] = *(const f32x2 *)(from + 2);
        }
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
          const float fs = __shfl(f, max(at[j], 0));
          if (at[j] >= 0) y += (f32x4){z[j][0][0], z[j][0][1], z[j][1][0], z[j][1][1]} * fs;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += __shfl_xor(y[j], 32);
    if (half || !has) continue;
    const float inv = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    *(u32x2_a4 *)(A.o + row * kD + 4 * l) = (u32x2){pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
  }
}

template <int KIND>
hipError_t attend_shared(const SharedArgs &s, const SharedPlan &p, hipStream_t st) {
  const int places = p.ranges + s.a.kv.n * p.few_parts * p.few_splits + p.many_tiles * p.many_parts * p.many_splits;
  hipLaunchKernelGGL(k_attend_shared<KIND>, dim3((uint32_t)places * (uint32_t)s.a.kv.heads + 1), dim3(256), 0, st, s, p);
  if (p.ranges == 0 && p.few_splits == 1 && p.many_splits == 1) return hipGetLastError();   // nothing to join
  // eight rows a wave where there are many: most are done, or have few passes
  const int64_t rows = (int64_t)s.a.kv.T * s.a.q_heads;
  if (rows > 8192) hipLaunchKernelGGL(k_join_shared<8>, dim3((uint32_t)((rows + 31) / 32)), dim3(256), 0, st, s, p);
  else hipLaunchKernelGGL(k_join_shared<1>, dim3((uint32_t)((rows + 3) / 4)), dim3(256), 0, st, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attend_shared(const SharedArgs &s, const SharedPlan &p, int kind, hipStream_t st) {
  return kind == 8 ? attend_shared<8>(s, p, st) : attend_shared<16>(s, p, st);
}

}  // namespace qdr
