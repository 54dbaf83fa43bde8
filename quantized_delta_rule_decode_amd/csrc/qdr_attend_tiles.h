// qdr_attend_tiles.h -- attention of one tile of rows over a run of blocks of keys:
//   o = sum_i p_i v_i / sum_i p_i,  p_i = 2^(s_i - m),  s_i = scale log2(e) q.k_i,
// one pass over the keys with the running maximum m and sum (online softmax).
// Everything is transposed: S^T = K Q^T has a query in each column, so a
// query's statistics are one value a lane, and the accumulators of S^T are the
// B operand of O^T = V^T P^T (qdr_mfma.h); the cache keeps K and V in the
// order of the A operands.  So nothing crosses lanes between the two products
// except the column maximum (two lane swaps).
// 8-bit caches: codes are exact in bfloat16, the key's scale multiplies its
// scores and the value's scale its weights, both in fp32.
#pragma once

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

// Blocks of one piece of the keys: pieces are cut so that none is shorter
// than `least` blocks but the last.
__device__ __forceinline__ int piece_blocks(int blocks, int splits, int least) {
  return max((blocks + splits - 1) / splits, least);
}

// Pages of a wave's blocks: block number i of it is first + i * step, and those
// behind `last` are the last again.  Lane x has the page of block x of 64, and of
// the 64 behind them, which are asked for 64 blocks ahead: a page number read by
// itself, block by block, would be waited for behind the keys and values that
// are on their way (they arrive in the order of the loads), and so would they.
struct PagesAhead {
  const int32_t *row;
  int first, step, last, shift;
  int now, next;
  __device__ __forceinline__ int fetch(int i) const {
    return row[min(first + (i + (int)(threadIdx.x & 63)) * step, last) >> shift];
  }
  __device__ __forceinline__ PagesAhead(const KvArgs &P, int b, int first_, int step_, int last_)
      : row(P.pages + (size_t)b * P.max_pages), first(first_), step(step_), last(last_), shift(P.page_shift - 5), now(0), next(0) {
    if (first > last) return;
    now = fetch(0);
    next = fetch(64);
  }
  // The page of block number i; called for 0, 1, 2 ... in turn.
  __device__ __forceinline__ int at(int i) {
    if (i > 0 && (i & 63) == 0) {
      now = next;
      next = fetch(i + 64);
    }
    return __builtin_amdgcn_readlane(now, i & 63);
  }
};
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
// The waves (eight in qdr_attend.hip, four in qdr_attend_shared.hip) take blocks
// of 32 keys in turn, each with its own running maximum, straight from memory into
// operands; they meet in LDS at the end.  Bound by memory with eight: 64 requests
// of up to 8192 cached tokens (ragged), 8 heads, 8-bit: 151 us for 0.81 GB, 5.4
// TB/s.  A block is on its way while another is taken; one request of 777 keys:
// 9 us, the latency of page, block, and the exchange.
// Up to sixteen rows it beats the many-row loop at every length (one sequence's
// 4 new tokens and 777, 8192, 65536 cached: 10.5, 15.5, 48 us against 29, 26, 66).
template <int KIND>
struct FewIn {
  u32x4 k[KIND == 8 ? 4 : 8], v[KIND == 8 ? 4 : 8];
  f32x4 ks[2], vs[2];
  bool good;
};

template <int WAVES>
struct FewShared {
  float m[WAVES][16], sum[WAVES][16];
  f32x4 o[WAVES][8][64];
};

// What a tile's pass over keys leaves: lane (g, i16) of wave w has column i16's
// maximum, sum of weights and, not divided by it, channels 16 d + 4 g .. for
// the 8 / WAVES values of d from 8 / WAVES w on.
template <int WAVES>
struct FewOut {
  f32x4 o[8 / WAVES];
  float m, sum;
  bool row;              // the column has a row, whose q and o are at `at`
  size_t at;
};

// Blocks lo .. hi of a tile's keys, by thread tid.  AHEAD: a wave's next block is
// on its way while it takes one (and has registers of its own).
template <int KIND, int WAVES, bool AHEAD>
__device__ __forceinline__ void few_tile(const AttendArgs &A, const Tile &t, int tid, int kvh, int lo, int hi, FewShared<WAVES> &sh, FewOut<WAVES> &out) {
  const KvArgs &P = A.kv;
  const int l = tid & 63, g = l >> 4, i16 = l & 15;
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
  const int last = lo + w < hi ? lo + w + (hi - 1 - lo - w) / WAVES * WAVES : hi - 1;
  PagesAhead pages(P, t.b, lo + w, WAVES, last);
  int taken = 0;
  auto load = [&](int block, FewIn<KIND> &in) {
    const uint8_t *blk = block_at(P, pages.at(taken++), kvh, min(block, last), KIND == 8 ? kKv8Block : kKv16Block);
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
    if (AHEAD) {
      FewIn<KIND> even, odd;
      load(lo + w, even);
      for (int block = lo + w; block < hi; block += 2 * WAVES) {
        load(block + WAVES, odd);
        take(block, even);
        if (block + WAVES >= hi) break;
        load(block + 2 * WAVES, even);
        take(block + WAVES, odd);
      }
    } else {
      FewIn<KIND> in;
      for (int block = lo + w; block < hi; block += WAVES) {
        load(block, in);
        take(block, in);
      }
    }
    if (KIND == 16 && __any(!finite))
      for (int block = lo + w; block < hi; block += WAVES) {
        if ((block + 1) * kBlock <= t.position + 1) continue;
        const uint8_t *blk = block_at(P, P.pages[(size_t)t.b * P.max_pages + (block >> (P.page_shift - 5))], kvh, block, kKv16Block);
        if (blk) add_not_finite(blk, block * kBlock, limit, g, o);
      }
  }
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (g == 0) {
    sh.m[w][i16] = m;
    sh.sum[w][i16] = sum;
  }
  __syncthreads();
  out.row = row;
  out.at = at;
  float top = kNone;
#pragma unroll
  for (int x = 0; x < WAVES; ++x) top = fmaxf(top, sh.m[x][i16]);
  const float ref = top == kNone ? 0.0f : top;
  float total = 0.0f;
#pragma unroll
  for (int x = 0; x < WAVES; ++x) total = __builtin_fmaf(sh.sum[x][i16], ex2(sh.m[x][i16] - ref), total);
  out.m = top;
  out.sum = total;
  const float fade = ex2(m - ref);
#pragma unroll
  for (int d = 0; d < 8; ++d) sh.o[w][d][l] = o[d] * fade;
  __syncthreads();
#pragma unroll
  for (int y = 0; y < 8 / WAVES; ++y) {
    out.o[y] = sh.o[0][8 / WAVES * w + y][l];
#pragma unroll
    for (int x = 1; x < WAVES; ++x) out.o[y] += sh.o[x][8 / WAVES * w + y][l];
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
// 4 sequences of 1024 new tokens, caches of up to 8192 with them (ragged), 32
// query and 8 key heads, calls queued back to back: bfloat16 470 us for 356
// GFLOP, 760 TFLOP/s, 8-bit 548; caches of 8192 each 562 and 656 for 515.  For 64
// keys and 32 rows a wave has 1024 cycles of products and about 1600 of vector
// instructions, 1000 of them exponentials; the matrix cores are busy 37% of the
// time and the vector units 44%, seldom together, and the operands take 3/4 of
// the LDS bandwidth.  Tried and slower, when the first took 560: the next block's
// scores between the current one's exponentials (688 us), 64 rows a wave with one
// wave a SIMD (the accumulators leave the vector registers; 930 us), wave
// priorities around the products (596).
constexpr float kSlack = 8.0f;

// 8 bits: a value's scale that is not finite (its vector had a NaN or an infinity)
// enters as 0, so that rows that do not see it need no select for every weight (three
// instructions, a seventh of the pass), and the rows that see it, all of whose
// channels it makes NaN, get that by their sum.  4 x 1024 new tokens, caches of 8192 each:
// 695 us with the selects, 670 so; two copies of the weights' code, one with them,
// 990 (spills).
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
  uint32_t odd[2];                   // [block] tokens whose values' scale is not finite, and 0 above
};

// What a tile's pass over keys leaves: lane (g, i16) of wave w has, of rows 32 w +
// 16 c + i16, the maximum, the sum of weights, and, not divided by it, channels 16 d + 4 g ...
struct ManyOut {
  f32x4 o[2][8];
  float m[2], sum[2];
  size_t at[2];          // of the row's q and o
  bool row[2];
};

// Blocks lo .. hi of a tile's keys, by thread tid.  STEPS: the operands are read
// four at a time, eight on their way while four are used, as they are written
// here.  Left to itself the compiler does nearly so where it has all registers,
// and where it has not reads each where it is used.  It matters little now (us,
// left to itself / in steps): 4 x 1024 new tokens as above 469 / 459, 8-bit 547 /
// 543; behind shared prefixes 32 sequences of 250 new tokens 627 / 627, 8-bit 766 /
// 753, of up to 100 262 / 263 and 335 / 329, of 20 123 / 121 and 129 / 128.
template <int KIND, bool STEPS>
__device__ __forceinline__ void many_tile(const AttendArgs &A, const Tile &t, int tid, int kvh, int lo, int hi, ManyShared<KIND> (&sh)[2], ManyOut &out) {
  const KvArgs &P = A.kv;
  const int l = tid & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  Frag q[2][4];
  auto &o = out.o;
  auto &m = out.m;
  auto &sum = out.sum;
  auto &at = out.at;
  auto &row = out.row;
  int limit[2];
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

  PagesAhead pages(P, t.b, lo, 1, hi - 1);
  auto load = [&](int block, ManyIn<KIND> &in) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const uint8_t *blk = block_at(P, pages.at(block + y - lo), kvh, min(block + y, hi - 1), KIND == 8 ? kKv8Block : kKv16Block);
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
        if (w == y) {
          const bool odd = l >= 32 && !(fabsf(in.scale) < INFINITY);
          const uint32_t tokens = (uint32_t)(__ballot(odd) >> 32);
          ((float *)to.scale[y])[l] = odd ? 0.0f : in.scale;
          if (l == 0) to.odd[y] = in.left[y] < kBlock ? tokens & ((1u << max(in.left[y], 0)) - 1u) : tokens;
        }
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
    const auto here = [] {
      if (STEPS) __builtin_amdgcn_sched_barrier(0);
    };
    // the 32 operands of K and V, four at a time
    Frag f[2][4];
    auto read = [&](int step) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[step & 1][i].w = step < 4 ? now.k[i >> 1][4 * (i & 1) + step][l] : now.v[(step - 4) >> 1][4 * (step & 1) + i][l];
      here();
    };
    f32x4 s[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[0][i] = s[1][i] = (f32x4){0, 0, 0, 0};
    here();
    read(0);
    read(1);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[0][i] = mma(f[x & 1][i], q[0][x], s[0][i]);
        s[1][i] = mma(f[x & 1][i], q[1][x], s[1][i]);
      }
      here();
      read(x + 2);
    }
    if (KIND == 8)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 by = now.scale[i >> 1][0][4 * (i & 1) + g];
        s[0][i] *= by;
        s[1][i] *= by;
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
    if (KIND == 8) {
      const uint32_t odd0 = __builtin_amdgcn_readfirstlane(now.odd[0]), odd1 = __builtin_amdgcn_readfirstlane(now.odd[1]);
      if (odd0 | odd1) {
        asm volatile("");
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if ((odd0 && block * kBlock + __builtin_ctz(odd0) <= limit[c]) || (odd1 && (block + 1) * kBlock + __builtin_ctz(odd1) <= limit[c]))
            sum[c] = __builtin_nanf("");
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
          const f32x4 by = now.scale[i >> 1][1][4 * (i & 1) + g];
          p *= by;
        }
        pf[c][i >> 1].u[2 * (i & 1)] = pack_bf16(p[0], p[1]);
        pf[c][i >> 1].u[2 * (i & 1) + 1] = pack_bf16(p[2], p[3]);
      }
      sum[c] += add[0] + add[1];
    }
    here();
#pragma unroll
    for (int x = 0; x < 4; ++x) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 4 * (x & 1) + i;
        o[0][d] = mma(f[x & 1][i], pf[0][x >> 1], o[0][d]);
        o[1][d] = mma(f[x & 1][i], pf[1][x >> 1], o[1][d]);
      }
      here();
      if (x < 2) read(x + 6);
    }
  }
  if (KIND == 16) {
    if (__syncthreads_or(!finite)) {
      for (int block = max(lo, (t.position + 1) / kBlock - 1); block < hi; ++block) {
        const uint8_t *blk = block_at(P, P.pages[(size_t)t.b * P.max_pages + (block >> (P.page_shift - 5))], kvh, block, kKv16Block);
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
  }
}

}  // namespace

}  // namespace qdr
