// qdr_attend.hip -- attention of new tokens over the paged cache:
//   o = sum_i p_i v_i / sum_i p_i,  p_i = 2^(s_i - m),  s_i = scale log2(e) q.k_i,
// one pass over the keys with the running maximum m and sum (online softmax).
// Everything is transposed: S^T = K Q^T has a query in each column, so a
// query's statistics are one value a lane, and the accumulators of S^T are the
// B operand of O^T = V^T P^T (qdr_mfma.h); the cache keeps K and V in the
// order of the A operands.  So nothing crosses lanes between the two products
// except the column maximum (two lane swaps).
// 8-bit caches: codes are exact in bfloat16, the key's scale multiplies its
// scores and the value's scale its weights, both in fp32.
#include "qdr_mfma.h"
#include "qdr_mixer.h"
#include "qdr_paged.h"

namespace qdr {

namespace {

constexpr int kD = 128;
constexpr float kNone = -INFINITY;

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// Largest of three as one instruction (fmaxf first quiets each operand with an
// instruction of its own); a NaN is passed over.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Largest over a column's four lanes (l ^ 16, l ^ 32): a swap of rows of 16, then
// of halves, gives every lane both sides without a trip through LDS.
__device__ __forceinline__ float column_max(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = max3(__uint_as_float(a[0]), __uint_as_float(a[1]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return max3(__uint_as_float(b[0]), __uint_as_float(b[1]), __uint_as_float(b[1]));
}

__device__ __forceinline__ float wave_max(float x) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) x = max3(x, __shfl_xor(x, d), x);
  return column_max(x);
}

// Eight codes as bfloat16 (exact).
__device__ __forceinline__ Frag widen(uint32_t a, uint32_t b) {
  Frag f;
  f.u[0] = pack_bf16((float)(int8_t)a, (float)(int8_t)(a >> 8));
  f.u[1] = pack_bf16((float)(int8_t)(a >> 16), (float)(int8_t)(a >> 24));
  f.u[2] = pack_bf16((float)(int8_t)b, (float)(int8_t)(b >> 8));
  f.u[3] = pack_bf16((float)(int8_t)(b >> 16), (float)(int8_t)(b >> 24));
  return f;
}

// A lane's eight values of one channel (tokens 4 g + {0..3, 16..19} of a
// block) with those from token `left` on cleared.
__device__ __forceinline__ u32x4 keep_tokens(u32x4 v, int g, int left) {
  Frag f;
  f.w = v;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const bool out = 4 * g + (e & 3) + 16 * (e >> 2) >= left;
    if (out) f.u[e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
  }
  return f.w;
}

// bfloat16 values that are not finite, in blocks where some rows of a tile do
// not see every token: 0 times them is not 0.  There they enter the product as
// 0, and where any was found they are added afterwards to the rows that see
// them (add_not_finite): infinities and NaN need no weight.
__device__ __forceinline__ bool is_finite16(uint32_t x) { return (x & 0x7F80u) != 0x7F80u; }
__device__ __forceinline__ u32x4 keep_finite(u32x4 v, bool *all) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = v[i];
    v[i] = (is_finite16(w) ? w & 0xFFFFu : 0u) | (is_finite16(w >> 16) ? w & 0xFFFF0000u : 0u);
    *all = *all && v[i] == w;
  }
  return v;
}

// The rows of a tile: `tokens` tokens from `token` on, times `heads` query
// heads from `head` on; row r is token r / heads, head r % heads.
struct Tile {
  int b, first, len;     // sequence and its rows
  int token, tokens;     // tokens of the tile, from the sequence's `token`
  int head, heads;       // query heads, from `head` of the whole call
  int position;          // of the tile's first token
  int keys;              // keys that the tile's last token sees
  bool skipped;          // its rows are 0
};

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

// Blocks of one piece of the keys: pieces are cut so that none is shorter
// than `least` blocks but the last.
__device__ __forceinline__ int piece_blocks(int blocks, int splits, int least) {
  return max((blocks + splits - 1) / splits, least);
}

// Page of a block of sequence b; asked for ahead of the block's own loads,
// which wait for it.
__device__ __forceinline__ int page_of(const KvArgs &P, int b, int block) {
  return P.pages[(size_t)b * P.max_pages + (block >> (P.page_shift - 5))];
}
// The block's memory; NULL on a bad page.
__device__ __forceinline__ const uint8_t *block_at(const KvArgs &P, int page, int kvh, int block, uint32_t bytes) {
  if (page < 0 || page >= P.num_pages) return nullptr;
  const int per = 1 << (P.page_shift - 5);
  return P.base + (((size_t)page * P.heads + kvh) * per + (block & (per - 1))) * bytes;
}

// Adds a bfloat16 block's values that are not finite to one column's eight
// results (lane (g, i): channels 16 d + 4 g .. of its row).
__device__ __forceinline__ void add_not_finite(const uint8_t *blk, int first_key, int limit, int g, f32x4 *o) {
#pragma unroll 1
  for (int x = 0; x < kBlock; ++x) {
    const int e = 4 * (x >> 4) + (x & 3), from = 16 * ((x >> 2) & 3) + 4 * g;
    const bool sees = first_key + x <= limit;
#pragma unroll
    for (int d = 0; d < 8; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t v = *(const uint16_t *)(blk + kKv16Half + (64 * d + from + r) * 16 + 2 * e);
        if (sees && !is_finite16(v)) o[d][r] += __uint_as_float(v << 16);
      }
  }
}

// ---- few rows: up to 16 (one token of up to 16 heads, a few tokens of fewer)
// Eight waves take every eighth block of 32 keys, each with its own running
// maximum, straight from memory into operands; they meet in LDS at the end.
// Bound by memory: 64 requests of 8192 cached tokens (ragged), 8 heads, 8-bit:
// 155 us for 0.85 GB, 5.5 TB/s.  A block is on its way while another is taken;
// one request of 777 keys: 9 us, the latency of page, block, and the exchange.
// Up to sixteen rows it beats the many-row loop at every length (one sequence's
// 4 new tokens and 777, 8192, 65536 cached: 10.5, 15.5, 48 us against 29, 26, 66).
template <int KIND>
struct FewIn {
  u32x4 k[KIND == 8 ? 4 : 8], v[KIND == 8 ? 4 : 8];
  f32x4 ks[2], vs[2];
  bool good;
};

template <int KIND>
__global__ void __launch_bounds__(64 * kFewWaves, 2) k_attend_few(AttendArgs A, AttendPlan plan) {
  const KvArgs &P = A.kv;
  __shared__ float sm[kFewWaves][16], sl[kFewWaves][16];
  __shared__ f32x4 so[kFewWaves][8][64];
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

  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // column i16 of the products: one (token, head) of the tile
  const int tok = i16 / t.heads, hd = i16 % t.heads;
  const bool row = tok < t.tokens;
  const size_t at = ((size_t)(t.first + t.token + (row ? tok : 0)) * A.q_heads + t.head + (row ? hd : 0)) * kD;
  const int limit = row ? t.position + tok : -1;   // last key that it sees
  Frag q[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    q[s].w = *(const u32x4_a4 *)(A.q + at + 64 * (s >> 1) + 16 * g + 8 * (s & 1));
    if (!row) q[s].w = (u32x4){0, 0, 0, 0};
  }
  f32x4 o[8];
#pragma unroll
  for (int d = 0; d < 8; ++d) o[d] = (f32x4){0, 0, 0, 0};
  float m = kNone, sum = 0.0f;
  bool finite = true;

  // A block's loads are always there: behind the wave's last it is the last
  // again (which the caches have), on a bad page some block, and its keys are
  // not looked at.
  const int last = lo + w < hi ? lo + w + (hi - 1 - lo - w) / kFewWaves * kFewWaves : hi - 1;
  int page = lo < hi ? page_of(P, t.b, min(lo + w, last)) : 0;
  auto load = [&](int block, FewIn<KIND> &in) {
    const uint8_t *blk = block_at(P, page, kvh, min(block, last), KIND == 8 ? kKv8Block : kKv16Block);
    page = page_of(P, t.b, min(block + kFewWaves, last));
    in.good = blk != nullptr;
    if (!blk) blk = P.base;
    constexpr int N = KIND == 8 ? 4 : 8;
#pragma unroll
    for (int i = 0; i < N; ++i) in.k[i] = *(const u32x4 *)(blk + (i * 64 + l) * 16);
#pragma unroll
    for (int i = 0; i < N; ++i) in.v[i] = *(const u32x4 *)(blk + N * 1024 + (i * 64 + l) * 16);
    if (KIND == 8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        in.ks[i] = *(const f32x4 *)(blk + kKv8Scale + 64 * i + 16 * g);
        in.vs[i] = *(const f32x4 *)(blk + kKv8Scale + 4 * kBlock + 64 * i + 16 * g);
      }
    }
  };
  auto take = [&](int block, FewIn<KIND> &in) {
    if (!in.good) {
      if (l == 0) atomicOr(P.err, kErrPage);
      return;
    }
    f32x4 s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) s[i] = (f32x4){0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Frag k;
        if (KIND == 8) {
          const u32x4 z = in.k[2 * i + (x >> 1)];
          k = (x & 1) ? widen(z[2], z[3]) : widen(z[0], z[1]);
        } else {
          k.w = in.k[(4 * i + x) & (KIND == 8 ? 3 : 7)];
        }
        s[i] = mma(k, q[x], s[i]);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (KIND == 8) s[i] *= in.ks[i];
      s[i] *= A.scale_log2;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (block * kBlock + 16 * i + 4 * g + r > limit) s[i][r] = kNone;
    }
    float top = max3(max3(s[0][0], s[0][1], s[0][2]), s[0][3], s[1][0]);
    top = max3(max3(top, s[1][1], s[1][2]), s[1][3], s[1][3]);
    top = column_max(top);
    if (__any(top > m)) {
      const float m1 = fmaxf(m, top);
      const float fade = ex2(m - (m1 == kNone ? 0.0f : m1));
      m = m1;
      sum *= fade;
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] *= fade;
    }
    const float ref = m == kNone ? 0.0f : m;        // no key seen yet: weights 2^(-inf) = 0
    f32x4 p[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        p[i][r] = ex2(s[i][r] - ref);
        sum += p[i][r];
        // a masked key's scale is not looked at
        if (KIND == 8) p[i][r] = s[i][r] == kNone ? 0.0f : p[i][r] * in.vs[i][r];
      }
    // two parts: the products are not what few rows wait for, and the weights'
    // rounding would be as large as the result's
    Frag pf[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t y[2];
      parts<2>(p[i >> 1][2 * (i & 1)], p[i >> 1][2 * (i & 1) + 1], y);
      pf[0].u[i] = y[0];
      pf[1].u[i] = y[1];
    }
    // values behind the last key of the tile may be anything: 0 times them is not 0
    const int left = t.keys - block * kBlock;
    if (KIND == 16 && left < kBlock)
#pragma unroll
      for (int d = 0; d < 8; ++d)
        in.v[d & (KIND == 8 ? 3 : 7)] = keep_tokens(in.v[d & (KIND == 8 ? 3 : 7)], g, left);
    if (KIND == 16 && (block + 1) * kBlock > t.position + 1)
#pragma unroll
      for (int d = 0; d < 8; ++d)
        in.v[d & (KIND == 8 ? 3 : 7)] = keep_finite(in.v[d & (KIND == 8 ? 3 : 7)], &finite);
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      Frag v;
      if (KIND == 8) {
        const u32x4 z = in.v[d >> 1];
        v = (d & 1) ? widen(z[2], z[3]) : widen(z[0], z[1]);
      } else {
        v.w = in.v[d & (KIND == 8 ? 3 : 7)];
      }
      o[d] = mma(v, pf[1], o[d]);
      o[d] = mma(v, pf[0], o[d]);
    }
  };

  if (lo < hi) {
    FewIn<KIND> even, odd;
    load(lo + w, even);
    for (int block = lo + w; block < hi; block += 2 * kFewWaves) {
      load(block + kFewWaves, odd);
      take(block, even);
      if (block + kFewWaves >= hi) break;
      load(block + 2 * kFewWaves, even);
      take(block + kFewWaves, odd);
    }
    if (KIND == 16 && __any(!finite))
      for (int block = lo + w; block < hi; block += kFewWaves) {
        if ((block + 1) * kBlock <= t.position + 1) continue;
        const uint8_t *blk = block_at(P, page_of(P, t.b, block), kvh, block, kKv16Block);
        if (blk) add_not_finite(blk, block * kBlock, limit, g, o);
      }
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (g == 0) {
    sm[w][i16] = m;
    sl[w][i16] = sum;
  }
  __syncthreads();
  float top = kNone;
#pragma unroll
  for (int x = 0; x < kFewWaves; ++x) top = fmaxf(top, sm[x][i16]);
  const float ref = top == kNone ? 0.0f : top;
  float total = 0.0f;
#pragma unroll
  for (int x = 0; x < kFewWaves; ++x) total = __builtin_fmaf(sl[x][i16], ex2(sm[x][i16] - ref), total);
  const float fade = ex2(m - ref);
#pragma unroll
  for (int d = 0; d < 8; ++d) so[w][d][l] = o[d] * fade;
  __syncthreads();
  // lane (g, i16) of wave w: channels 16 w + 4 g .. of column i16
  static_assert(kFewWaves == 8, "a wave to sixteen channels");
  f32x4 y = so[0][w][l];
#pragma unroll
  for (int x = 1; x < kFewWaves; ++x) y += so[x][w][l];
  if (plan.few_splits == 1) {
    if (row) {
      const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
      *(u32x2_a4 *)(A.o + at + 16 * w + 4 * g) = (u32x2){pack_bf16(y[0] * inv, y[1] * inv), pack_bf16(y[2] * inv, y[3] * inv)};
    }
  } else {
    float *to = A.part + (size_t)blockIdx.x * (kFewRows * (kD + 2));
    *(f32x4 *)(to + (size_t)i16 * kD + 16 * w + 4 * g) = y;
    if (w == 0 && g == 0) {
      to[kFewRows * kD + i16] = top;
      to[kFewRows * kD + kFewRows + i16] = total;
    }
  }
}

// ---- many rows: up to 128, 32 a wave; two blocks of keys at a time through
// LDS, two pairs of them in turn, the next pair on its way in registers.
// What the vector units do for a score is what counts beside the products:
// the scale rides on the subtraction of the maximum, masks are only looked at
// where a wave's rows end, and the maximum that the weights are taken from
// moves (and with it the accumulators) only when a score exceeds it by 2^8.
// The weights are rounded to bfloat16 once here, 2^-8 of each at most, which
// averages out over the keys (relative error of the result 0.0021, of which
// its own rounding is 0.0017); a second part would add half the products again.
// 4 sequences of 1024 new tokens, 8192 cached, 32 query and 8 key heads: 518 us
// for 357 GFLOP, 690 TFLOP/s.  For 64 keys and 32 rows a wave has 1024 cycles of
// products and about 1600 of vector instructions, 1000 of them exponentials;
// the matrix cores are busy 33% of the time and the vector units 39%, seldom
// together, and the operands take 3/4 of the LDS bandwidth.  Tried and slower:
// the next block's scores between the current one's exponentials (688 us),
// 64 rows a wave with one wave a SIMD (the accumulators leave the vector
// registers; 930 us), wave priorities around the products (596).
constexpr float kSlack = 8.0f;

template <int KIND>
struct ManyIn {
  u32x4 k[KIND == 8 ? 2 : 4], v[KIND == 8 ? 2 : 4];
  float scale;        // 8-bit: of the keys, then of the values
  int left[2];        // tokens of the two blocks that count (0: a bad page)
};

template <int KIND>
struct ManyShared {
  u32x4 k[2][8][64], v[2][8][64];    // [block of the pair]
  f32x4 scale[2][2][8];              // [block][keys, values]
};

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

  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  Frag q[2][4];
  f32x4 o[2][8];
  float m[2], sum[2];
  int limit[2];
  size_t at[2];
  bool row[2];
  // a negative scale: -q and its magnitude; none: q = 0, and 1 (a masked score is -inf)
  const uint32_t flip = A.scale_log2 < 0.0f ? 0x80008000u : 0u, keep = A.scale_log2 == 0.0f ? 0u : ~0u;
  const float scale = A.scale_log2 == 0.0f ? 1.0f : fabsf(A.scale_log2);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int r = 32 * w + 16 * c + i16;
    const int tok = r / t.heads, hd = r % t.heads;
    row[c] = tok < t.tokens;
    at[c] = ((size_t)(t.first + t.token + (row[c] ? tok : 0)) * A.q_heads + t.head + (row[c] ? hd : 0)) * kD;
    limit[c] = row[c] ? t.position + tok : -1;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      q[c][s].w = (*(const u32x4_a4 *)(A.q + at[c] + 64 * (s >> 1) + 16 * g + 8 * (s & 1)) & keep) ^ flip;
      if (!row[c]) q[c][s].w = (u32x4){0, 0, 0, 0};
    }
#pragma unroll
    for (int d = 0; d < 8; ++d) o[c][d] = (f32x4){0, 0, 0, 0};
    m[c] = kNone;
    sum[c] = 0.0f;
  }
  // keys that every row of the wave sees, and that any of them does
  const int first_tok = 32 * w / t.heads, last_tok = min((32 * w + 31) / t.heads, t.tokens - 1);
  const int all_see = t.position + first_tok + 1;
  const int some_see = first_tok < t.tokens ? t.position + last_tok + 1 : 0;

  int page[2] = {0, 0};
  if (lo < hi)
    for (int y = 0; y < 2; ++y) page[y] = page_of(P, t.b, min(lo + y, hi - 1));
  auto load = [&](int block, ManyIn<KIND> &in) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const uint8_t *blk = block_at(P, page[y], kvh, min(block + y, hi - 1), KIND == 8 ? kKv8Block : kKv16Block);
      page[y] = page_of(P, t.b, min(block + 2 + y, hi - 1));
      in.left[y] = block + y < hi && blk ? min(t.keys - (block + y) * kBlock, kBlock) : 0;
      if (!blk && block + y < hi && tid == 0) atomicOr(P.err, kErrPage);
      if (!blk) blk = P.base;
      if (KIND == 8) {
        in.k[y] = *(const u32x4 *)(blk + tid * 16);
        in.v[y] = *(const u32x4 *)(blk + kKv8Half + tid * 16);
        if (w == y) in.scale = *(const float *)(blk + kKv8Scale + 4 * l);
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          in.k[2 * y + (KIND == 8 ? 0 : x)] = *(const u32x4 *)(blk + (tid + 256 * x) * 16);
          in.v[2 * y + (KIND == 8 ? 0 : x)] = *(const u32x4 *)(blk + kKv16Half + (tid + 256 * x) * 16);
        }
      }
    }
  };
  bool finite = true;
  auto store = [&](int block, const ManyIn<KIND> &in, ManyShared<KIND> &to) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      if (KIND == 8) {
        to.k[y][2 * w][l] = widen(in.k[y][0], in.k[y][1]).w;
        to.k[y][2 * w + 1][l] = widen(in.k[y][2], in.k[y][3]).w;
        to.v[y][2 * w][l] = widen(in.v[y][0], in.v[y][1]).w;
        to.v[y][2 * w + 1][l] = widen(in.v[y][2], in.v[y][3]).w;
        if (w == y) ((float *)to.scale[y])[l] = in.scale;
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          to.k[y][4 * x + w][l] = in.k[2 * y + (KIND == 8 ? 0 : x)];
          u32x4 v = in.v[2 * y + (KIND == 8 ? 0 : x)];
          // values behind the last key may be anything: 0 times them is not 0
          if (in.left[y] < kBlock) v = keep_tokens(v, g, in.left[y]);
          if ((block + 2) * kBlock > t.position + 1) v = keep_finite(v, &finite);
          to.v[y][4 * x + w][l] = v;
        }
      }
    }
  };

  ManyIn<KIND> in;
  if (lo < hi) load(lo, in);
  for (int block = lo; block < hi; block += 2) {
    ManyShared<KIND> &now = sh[((block - lo) >> 1) & 1];
    store(block, in, now);
    const int left0 = in.left[0], left1 = in.left[1];
    lds_barrier();
    load(block + 2, in);        // always there: the waits stay exact
    if (block * kBlock >= some_see) continue;
    f32x4 s[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][i] = s[1][i] = (f32x4){0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Frag k;
        k.w = now.k[i >> 1][4 * (i & 1) + x][l];
        s[0][i] = mma(k, q[0][x], s[0][i]);
        s[1][i] = mma(k, q[1][x], s[1][i]);
      }
    if (KIND == 8)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 f = now.scale[i >> 1][0][4 * (i & 1) + g];
        s[0][i] *= f;
        s[1][i] *= f;
      }
    const bool masked = left0 < kBlock || left1 < kBlock || (block + 2) * kBlock > all_see;
    if (masked) {
      asm volatile("");   // a branch, not 64 selects in every pass
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = 16 * (i & 1) + 4 * g + r;
            if (key >= (i < 2 ? left0 : left1) || (block + (i >> 1)) * kBlock + key > limit[c]) s[c][i][r] = kNone;
          }
    }
    Frag pf[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float top = max3(s[c][0][0], s[c][0][1], s[c][0][2]), top1 = max3(s[c][2][0], s[c][2][1], s[c][2][2]);
      top = max3(top, s[c][0][3], s[c][1][0]);
      top1 = max3(top1, s[c][2][3], s[c][3][0]);
      top = max3(top, s[c][1][1], s[c][1][2]);
      top1 = max3(top1, s[c][3][1], s[c][3][2]);
      top = max3(max3(top, s[c][1][3], s[c][3][3]), top1, top1);
      top = column_max(top) * scale;
      if (__any(top > m[c] + kSlack)) {
        const float m1 = fmaxf(m[c], top);
        const float fade = ex2(m[c] - (m1 == kNone ? 0.0f : m1));
        m[c] = m1;
        sum[c] *= fade;
#pragma unroll
        for (int d = 0; d < 8; ++d) o[c][d] *= fade;
      }
      const float ref = m[c] == kNone ? 0.0f : m[c];
      float add[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x4 p;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          p[r] = ex2(__builtin_fmaf(s[c][i][r], scale, -ref));
          add[r & 1] += p[r];
        }
        if (KIND == 8) {
          const f32x4 f = now.scale[i >> 1][1][4 * (i & 1) + g];
          // a masked key's scale is not looked at
#pragma unroll
          for (int r = 0; r < 4; ++r) p[r] = masked && s[c][i][r] == kNone ? 0.0f : p[r] * f[r];
        }
        pf[c][i >> 1].u[2 * (i & 1)] = pack_bf16(p[0], p[1]);
        pf[c][i >> 1].u[2 * (i & 1) + 1] = pack_bf16(p[2], p[3]);
      }
      sum[c] += add[0] + add[1];
    }
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        Frag v;
        v.w = now.v[y][d][l];
        o[0][d] = mma(v, pf[0][y], o[0][d]);
        o[1][d] = mma(v, pf[1][y], o[1][d]);
      }
  }
  if (KIND == 16) {
    if (__syncthreads_or(!finite)) {
      for (int block = max(lo, (t.position + 1) / kBlock - 1); block < hi; ++block) {
        const uint8_t *blk = block_at(P, page_of(P, t.b, block), kvh, block, kKv16Block);
        // a pair of blocks before the rows' first position was not looked at
        if (!blk || (((block - lo) & ~1) + lo + 2) * kBlock <= t.position + 1) continue;
#pragma unroll
        for (int c = 0; c < 2; ++c) add_not_finite(blk, block * kBlock, limit[c], g, o[c]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    sum[c] += __shfl_xor(sum[c], 16);
    sum[c] += __shfl_xor(sum[c], 32);
    if (plan.many_splits == 1) {
      if (!row[c]) continue;
      const float inv = sum[c] > 0.0f || sum[c] != sum[c] ? 1.0f / sum[c] : 0.0f;
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const f32x4 y = o[c][d] * inv;
        *(u32x2_a4 *)(A.o + at[c] + 16 * d + 4 * g) = (u32x2){pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3])};
      }
    } else {
      const size_t unit = (((size_t)tile * P.heads + kvh) * plan.many_parts + part) * plan.many_splits + split;
      float *to = A.part + plan.few_floats + unit * (kManyRows * (kD + 2));
      const int r = 32 * w + 16 * c + i16;
#pragma unroll
      for (int d = 0; d < 8; ++d) *(f32x4 *)(to + (size_t)r * kD + 16 * d + 4 * g) = o[c][d];
      if (g == 0) {
        to[kManyRows * kD + r] = m[c];
        to[kManyRows * kD + kManyRows + r] = sum[c];
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
