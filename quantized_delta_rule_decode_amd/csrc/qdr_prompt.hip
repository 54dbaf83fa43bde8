// qdr_prompt.hip -- the prompt form of the recurrences
//   S_t = a_t S_{t-1} + k_t u_t^T,  o_t = S_t^T q_t,
//   u_t = beta_t (v_t - a_t S_{t-1}^T k_t)  (DELTA)  or  u_t = v_t  (SUM)
// for ragged prompts, 64 tokens (a chunk) at a time.  With g_t the sum of
// log2 a over the chunk up to t and G_ts = 2^(g_t - g_s), a chunk that starts
// from S is
//   DELTA  (I + L) U = diag(beta) (V - diag(2^g) K S),  L_ts = beta_t G_ts k_t.k_s (t > s)
//   SUM    U = V
//   O  = diag(2^g) Q S + A U,   A_ts = G_ts q_t.k_s (t >= s)
//   S' = 2^g_63 S + K^T diag(2^(g_63 - g)) U
// so all of it is matrix products.  Launches:
//   k_prompt_slots    pools that hold no plain fp32 heads: which slots to unpack
//                     before and to pack after;
//   k_prompt_chunks   DELTA, every chunk at once: T = (I + L)^-1 diag(beta) and
//                     the decays, and which sequences are longest;
//   k_prompt_decays   SUM: the decays alone;
//   k_prompt_segment, k_prompt_join    SUM, long sequences: cut into segments;
//                     what each adds to a state, then the states they start from;
//   k_prompt_map, k_prompt_join_maps   the same for DELTA, where a segment's
//                     effect is a matrix and a sum;
//   k_prompt_chain    DELTA, few heads: the chunks in order, four workgroups a
//                     head that work on three chunks at once;
//   k_prompt_scan     the chunks of a sequence (segment) in order.
// Precision: q, k and v are bfloat16 and enter exactly.  Whatever is computed
// (S, U, T, A) enters a product as a sum of bfloat16 parts: three parts (24
// bits, an fp32 value) on the way to the state, two (16 bits) where only the
// bfloat16 readout follows; sums are fp32 in the matrix cores' accumulators.
// The decays are summed in fp64: differences of long sums lose nothing.
#include "qdr_mfma.h"
#include "qdr_mixer.h"

namespace qdr {

namespace {

// Where TIGHT: keeps the reads of later steps from being moved up across it.
// They would not fit the registers that four waves a SIMD leave (SUM); with
// two (DELTA) they hide the LDS behind the products.
template <bool TIGHT>
__device__ __forceinline__ void place() {
  if (TIGHT) __builtin_amdgcn_sched_barrier(0);
}

constexpr int kD = 128;
constexpr int kLd = 68;        // row stride of a 64 x 64 fp32 matrix in LDS
constexpr double kLogZero = -2000.0;   // for log2(0): 2^-2000 is 0, and sums of 64 of it stay finite

// First fragment of row tile w of a triangular matrix.
__device__ __forceinline__ int tri_frag(int w) { return w < 2 ? w : 2 * w - 2; }

// Workspace of one (chunk, head).
struct ChunkSpace {
  double *lg;      // [64] sums of log2 a over the chunk up to each token
  float *dec;      // [64] 2^lg, [64] 2^(lg_63 - lg)
  float *T;        // DELTA: fragments of T, [fragment][half][lane][4]
};
__device__ __forceinline__ ChunkSpace chunk_space(const PromptArgs &P, int place, int h) {
  float *ws = P.chunk_ws + ((size_t)place * P.H + h) * (P.beta ? kChunkFloats : kDecayFloats);
  return {(double *)ws, ws + 2 * kChunk, ws + kDecayFloats};
}

// x plus the value that DPP control CTRL brings to the rows of MASK.
template <int CTRL, int MASK>
__device__ __forceinline__ double add_from(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)b, CTRL, MASK, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(b >> 32), CTRL, MASK, 0xF, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sum of x over a wave's lanes up to each.
__device__ __forceinline__ double sum_up(double x) {
  x = add_from<0x111, 0xF>(x);   // from 1, 2, 4, 8 lanes below in the row of 16
  x = add_from<0x112, 0xF>(x);
  x = add_from<0x114, 0xF>(x);
  x = add_from<0x118, 0xF>(x);
  x = add_from<0x142, 0xA>(x);   // lane 15 of the row below, then lane 31
  return add_from<0x143, 0xC>(x);
}

// One wave: the decays of a chunk, a token to a lane.  A logarithm is rounded to
// fp32, which moves a decay 2^-g by a factor 1 + g 2^-24, less than rounding it;
// their sums are not rounded (fp64).
__device__ __forceinline__ double put_decays(const PromptArgs &P, size_t t0, int nt, int h, int l, const ChunkSpace &ws) {
  const float a = l < nt ? P.gate[(t0 + l) * P.H + h] : 1.0f;
  const double x = sum_up(a == 0.0f ? kLogZero : (double)log2f(a));
  const uint64_t last = __builtin_bit_cast(uint64_t, x);
  const double end = __builtin_bit_cast(double, (uint64_t)__builtin_amdgcn_readlane((uint32_t)(last >> 32), 63) << 32 |
                                                    (uint32_t)__builtin_amdgcn_readlane((uint32_t)last, 63));
  ws.lg[l] = x;
  ws.dec[l] = exp2f((float)x);
  ws.dec[kChunk + l] = exp2f((float)(end - x));
  return x;
}

// The chunk that place `place` of a head stands for; false: none, or one of a
// sequence that is skipped.
__device__ __forceinline__ bool chunk_at(const PromptArgs &P, int place, size_t *t0, int *nt) {
  const int b = sequence_of(P.cu, P.n, kChunk, 1, place);
  int first, len;
  if (!rows_of(P.cu, P.T, b, &first, &len)) return false;
  const int c = place - (first / kChunk + b), slot = P.slots[b];
  if (c < 0 || c >= (len + kChunk - 1) / kChunk || slot < 0 || slot >= P.num_slots) return false;
  *t0 = (size_t)first + (size_t)c * kChunk;
  *nt = min(kChunk, len - c * kChunk);
  return true;
}

__device__ __forceinline__ f32x4 mma4(const f32x4 a, const f32x4 b, f32x4 c) {   // 16x16x16 in fp32
#pragma unroll
  for (int r = 0; r < 4; ++r) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[r], b[r], c, 0, 0, 0);
  return c;
}

// Block column J of X = (I + L)^-1 from its diagonal blocks (already in X):
// X_iJ = -X_ii sum_{J <= m < i} L_im X_mJ.  A result's accumulators are the
// next product's B operand.
template <int J>
__device__ __forceinline__ void inverse_column(const float (*L)[kLd], float (*X)[kLd], int g, int i16) {
  f32x4 x[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) x[J][r] = X[16 * J + 4 * g + r][16 * J + i16];
#pragma unroll
  for (int i = J + 1; i < 4; ++i) {
    f32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int m = J; m < i; ++m) sum = mma4(*(const f32x4 *)&L[16 * i + i16][16 * m + 4 * g], x[m], sum);
    x[i] = mma4(*(const f32x4 *)&X[16 * i + i16][16 * i + 4 * g], -sum, (f32x4){0, 0, 0, 0});
  }
#pragma unroll
  for (int i = J + 1; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) X[16 * i + 4 * g + r][16 * J + i16] = x[i][r];
}

// SUM: a wave to a (chunk, head): 256 B in, 1 KiB out.  9 us for 12288 of them,
// 2 TB/s; the vector units half busy with logarithms and exponentials.
__global__ void __launch_bounds__(256) k_prompt_decays(PromptArgs P) {
  const int l = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int place = (int)(unit / P.H), h = (int)(unit % P.H);
  size_t t0;
  int nt;
  if (place >= P.chunks || !chunk_at(P, place, &t0, &nt)) return;
  put_decays(P, t0, nt, h, l, chunk_space(P, place, h));
}

// Sequences by falling length, so that the longest ones start first: the place
// of sequence b.
__device__ __forceinline__ void put_order(const PromptArgs &P, int b) {
  if (b >= P.n) return;
  auto length = [&](int i) { return (long long)P.cu[i + 1] - P.cu[i]; };
  const long long mine = length(b);
  int rank = 0;
  for (int i = 0; i < P.n; ++i) rank += length(i) > mine || (length(i) == mine && i < b);
  P.order[rank] = b;
}

// DELTA: T and the decays.  One workgroup per (chunk, head), and before them
// those that order the sequences; wave w makes
// rows 16 w .. 16 w + 15 of L, inverts the diagonal block w by substitution,
// then block column w of the inverse.  Everything fp32 but the exact products
// of k: the matrix cores' fp32 form for the blocks, whose rounding would be the
// whole chunk's.  16 KiB in and 13 KiB out: 24576 of them (32768 tokens, 48
// heads) 200 us, 4.1 TB/s of memory traffic, with the vector units busy 49% of
// the time.  All rows of k asked for before the first product: one latency, not
// one a tile (270 us).
__global__ void __launch_bounds__(256) k_prompt_chunks(PromptArgs P) {
  __shared__ __attribute__((aligned(16))) float L[kChunk][kLd], X[kChunk][kLd];
  __shared__ double lg[kChunk];
  __shared__ __attribute__((aligned(16))) float bt[kChunk];

  const int orders = P.order ? (P.n + 255) / 256 : 0;
  if ((int)blockIdx.x < orders) {
    put_order(P, blockIdx.x * 256 + threadIdx.x);
    return;
  }
  const int place = (blockIdx.x - orders) / P.H, h = (blockIdx.x - orders) % P.H;
  size_t t0;
  int nt;
  if (!chunk_at(P, place, &t0, &nt)) return;
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const ChunkSpace ws = chunk_space(P, place, h);
  const size_t row = (size_t)P.H * kD;

  // rows of k as operands: lane (g, i) holds channels 32 s + 8 g .. of token
  // 16 j + i, zero behind the sequence's end
  auto load = [&](int tile, Frag *f) {
    const int t = 16 * tile + i16;
    const uint16_t *src = P.k + (t0 + (t < nt ? t : 0)) * row + (size_t)h * kD + 8 * g;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      f[s].w = *(const u32x4_a4 *)(src + 32 * s);
      if (t >= nt) f[s].w = (u32x4){0, 0, 0, 0};
    }
  };
  // all asked for at once: one latency instead of one a tile
  Frag k[4], kj[4][4];
  load(w, k);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < w) load(j, kj[j]);
  if (w == 0) {
    lg[l] = put_decays(P, t0, nt, h, l, ws);
    bt[l] = l < nt ? P.beta[(t0 + l) * P.H + h] : 0.0f;
  }
  f32x4 kk[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) kk[j] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j > w) continue;
#pragma unroll
    for (int s = 0; s < 4; ++s) kk[j] = mma(k[s], j < w ? kj[j][s] : k[s], kk[j]);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (j > w) continue;
    const int col = 16 * j + i16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * g + r;
      L[t][col] = t > col ? bt[t] * (kk[j][r] * exp2f((float)(lg[t] - lg[col]))) : 0.0f;
    }
  }
  if ((w & 1) == 0) {   // the block above the diagonal that shares a fragment with it
#pragma unroll
    for (int r = 0; r < 4; ++r) X[16 * w + 4 * g + r][16 * (w + 1) + i16] = 0.0f;
  }
  // column j of the diagonal block in lane j
  if (l < 16) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = l == i ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < i; ++m) s = __builtin_fmaf(-L[16 * w + i][16 * w + m], x[m], s);
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) X[16 * w + i][16 * w + l] = x[i];
  }
  __syncthreads();
  if (w == 0) inverse_column<0>(L, X, g, i16);
  else if (w == 1) inverse_column<1>(L, X, g, i16);
  else if (w == 2) inverse_column<2>(L, X, g, i16);
  __syncthreads();
  for (int s = 0; s <= w >> 1; ++s) {
    float *f = ws.T + (size_t)(tri_frag(w) + s) * 512 + l * 4;
    *(f32x4 *)f = *(const f32x4 *)&X[16 * w + i16][32 * s + 4 * g] * *(const f32x4 *)&bt[32 * s + 4 * g];
    *(f32x4 *)(f + 256) = *(const f32x4 *)&X[16 * w + i16][32 * s + 16 + 4 * g] * *(const f32x4 *)&bt[32 * s + 16 + 4 * g];
  }
}

// Eight fp32 values as P bfloat16 operands.
template <int P>
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, Frag *f) {
  uint32_t p[4][P];
  parts<P>(a[0], a[1], p[0]);
  parts<P>(a[2], a[3], p[1]);
  parts<P>(b[0], b[1], p[2]);
  parts<P>(b[2], b[3], p[3]);
#pragma unroll
  for (int x = 0; x < P; ++x) f[x].w = (u32x4){p[0][x], p[1][x], p[2][x], p[3][x]};
}

// What a chunk shares with every column: left operands, 1 KiB each, values
// and decays.  Rows of q and k lie in pieces of 8 channels; piece c of row i
// of a tile is at 16 c + (i ^ x(c)), so that what LDS takes in one step lies on
// sixteen different 16-byte columns of its banks: four rows of four neighbouring
// pieces (a transposing read), and of 16-byte accesses lanes 0-3, 12-15, 20-23
// and 24-27, which are rows of two pieces (an operand) or pieces of two rows
// (coming in).  x(4 P + j) = 4 {0, 3, 1, 2}[j] + {0, 2, 3, 1}[P].
template <bool DELTA>
struct Stage {
  u32x4 Q[4][256], K[4][256];                 // [token tile]
  u32x4 A[kTriFrags][2][64];                  // two parts
  u32x4 T[DELTA ? kTriFrags : 1][3][64];      // three
  uint16_t V[kChunk][136];                    // then the readout
  double lg[kChunk];
  float dec[2 * kChunk];                      // decays from the chunk's start, then to its end
};
static_assert(sizeof(Stage<true>) <= 80 * 1024, "two workgroups share a compute unit's 160 KiB");

__device__ __forceinline__ int piece_at(int piece, int i) { return 16 * piece + (i ^ (int)(0x95D1B7F3A6E284C0ull >> (4 * piece) & 15)); }
// Operand of rows: lane (g, i) has channels 32 s + 8 g .. of row i of a tile.
__device__ __forceinline__ Frag rows_operand(const u32x4 *tile, int s, int l) {
  Frag f;
  f.w = tile[piece_at(4 * s + (l >> 4), l & 15)];
  return f;
}

struct ScanAt {
  int first, len, chunks, place0, h;
  size_t row;
};

// A thread's share of a chunk on its way in (READ: also what only the readout
// needs): pieces of 16 bytes of two rows, and of T.
template <bool DELTA, bool READ>
struct StageIn {
  u32x4 q[READ ? 2 : 1], k[2], v[2];
  f32x4 T[2];
  double lg;
  float dec;
};

// A uniform address and a 32-bit offset (the host keeps 64 rows under 2^32 bytes).
__device__ __forceinline__ const u32x4_a4 *piece_of(const uint16_t *base, uint32_t offset) {
  return (const u32x4_a4 *)((const uint8_t *)base + offset);
}

template <bool DELTA, bool READ>
__device__ __forceinline__ void fetch(const PromptArgs &P, const ScanAt &A, int c, int tid, StageIn<DELTA, READ> &in) {
  const int nt = min(kChunk, A.len - c * kChunk);
  const size_t base = ((size_t)A.first + (size_t)c * kChunk) * A.row + (size_t)A.h * kD;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = (tid >> 4) + 32 * x;
    const uint32_t at = (uint32_t)(t < nt ? t : 0) * (uint32_t)(2 * A.row) + 16 * (tid & 15);
    in.k[x] = *piece_of(P.k + base, at);
    in.v[x] = *piece_of(P.v + base, at);
    if (READ) in.q[READ ? x : 0] = *piece_of(P.q + base, at);
  }
  const ChunkSpace ws = chunk_space(P, A.place0 + c, A.h);
  if (DELTA) {   // 12 groups of 256 values
    in.T[0] = *(const f32x4 *)(ws.T + 4 * tid);
    in.T[1] = *(const f32x4 *)(ws.T + 4 * (tid < 256 ? tid + 512 : tid));
  }
  in.dec = ws.dec[tid & 127];
  if (READ) in.lg = ws.lg[tid & 63];
}

template <bool DELTA, bool READ>
__device__ __forceinline__ void put(const ScanAt &A, int c, int tid, const StageIn<DELTA, READ> &in, Stage<DELTA> &st) {
  const int nt = A.len - c * kChunk, piece = tid & 15;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = (tid >> 4) + 32 * x, at = piece_at(piece, t & 15);
    const bool out = t >= nt;   // nothing of the rows behind the end
    const u32x4 none = {0, 0, 0, 0};
    if (READ) st.Q[t >> 4][at] = out ? none : in.q[READ ? x : 0];
    st.K[t >> 4][at] = out ? none : in.k[x];
    *(u32x4 *)&st.V[t][8 * piece] = out ? none : in.v[x];
  }
  if (DELTA)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int group = (tid >> 6) + 8 * x, l = tid & 63;
      if (group >= 2 * kTriFrags) continue;
      uint32_t p[2][3];
      parts<3>(in.T[x][0], in.T[x][1], p[0]);
      parts<3>(in.T[x][2], in.T[x][3], p[1]);
#pragma unroll
      for (int y = 0; y < 3; ++y) ((Frag *)&st.T[DELTA ? group >> 1 : 0][y][l])->h[group & 1] = (u32x2){p[0][y], p[1][y]};
    }
  if (tid < 128) st.dec[tid] = in.dec;
  if (READ && tid >= 448) st.lg[tid - 448] = in.lg;
}

// Tile (t, j) of A, as the left operand that it becomes: computed transposed
// (rows are keys), its accumulators are half j & 1 of the operand's lanes.
__device__ __forceinline__ void put_tile(const u32x4 *K, const Frag *q, const double *lg, u32x4 (*A)[2][64], int t, int j, int l) {
  const int g = l >> 4, i16 = l & 15;
  f32x4 x = {0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) x = mma(rows_operand(K, s, l), q[s], x);
  const int query = 16 * t + i16, key = 16 * j + 4 * g;
  const double to = lg[query];
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = query >= key + r ? x[r] * __builtin_amdgcn_exp2f((float)(to - lg[key + r])) : 0.0f;
  uint32_t p[2][2];
  parts<2>(x[0], x[1], p[0]);
  parts<2>(x[2], x[3], p[1]);
#pragma unroll
  for (int y = 0; y < 2; ++y) ((Frag *)&A[tri_frag(t) + (j >> 1)][y][l])->h[j & 1] = (u32x2){p[0][y], p[1][y]};
}
// The ten tiles over eight waves; the halves above the diagonal are cleared
// once, before the first chunk.
template <bool DELTA>
__device__ __forceinline__ void put_A(Stage<DELTA> &st, int wave, int l) {
#pragma unroll 1
  for (int x = 0; x < (wave < 2 ? 2 : 1); ++x) {
    const int t = x ? wave : wave < 4 ? 3 : wave < 7 ? 2 : 1, j = x ? wave : wave < 4 ? wave : wave < 7 ? wave - 4 : 0;
    Frag q[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) q[s] = rows_operand(st.Q[t], s, l);
    put_tile(st.K[j], q, st.lg, st.A, t, j, l);
  }
}
__device__ __forceinline__ void clear_A(u32x4 (*A)[2][64], int tid) {
  if (tid < 256) ((Frag *)&A[tri_frag(tid < 128 ? 0 : 2) + (tid < 128 ? 0 : 1)][(tid >> 6) & 1][tid & 63])->h[1] = (u32x2){0, 0};
}

// The readout of a chunk, whole rows.
template <bool DELTA>
__device__ __forceinline__ void put_rows(const PromptArgs &P, const ScanAt &A, int c, int tid, const Stage<DELTA> &st) {
  const int nt = A.len - c * kChunk;
  const size_t base = ((size_t)A.first + (size_t)c * kChunk) * A.row + (size_t)A.h * kD;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int t = (tid >> 4) + 32 * x;
    if (t >= nt) continue;
    *(u32x4_a4 *)((uint8_t *)(P.o + base) + (uint32_t)t * (uint32_t)(2 * A.row) + 16 * (tid & 15)) = *(const u32x4 *)&st.V[t][8 * (tid & 15)];
  }
}

// Row 4 g + r of result 2 s + i of the state is channel state_row(2 s + i) + r:
// a lane's two results of a contraction step are the eight channels that one
// 16-byte piece of a row of q or k has.
__device__ __forceinline__ int state_row(int m, int g) { return 32 * (m >> 1) + 8 * g + 4 * (m & 1); }

typedef short s16x4 __attribute__((ext_vector_type(4)));

// Operand of K^T: rows (channels) of result m, tokens 32 s + {4 g.., 16 + 4 g..}.
// A transposing read gives lane i of a group of 16 the i-th of 16 columns of
// four rows; the group's lane 4 r + j points to columns 4 j .. of row r.
__device__ __forceinline__ Frag transposed(const u32x4 (*K)[256], int m, int s, int l) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const int g = l >> 4, r = (l >> 2) & 3, j = l & 3;
  Frag f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const u32x2 *piece = (const u32x2 *)&K[2 * s + half][piece_at(4 * (m >> 1) + j, 4 * g + r)] + (m & 1);
    f.h[half] = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)piece));
  }
  return f;
}

// S = 2^g_63 S + K^T diag(2^(g_63 - g)) U.
template <bool TIGHT>
__device__ __forceinline__ void update_state(const u32x4 (*K)[256], const float *dec, const f32x4 *u, f32x4 *S, int l) {
  const int g = l >> 4;
  const float all = dec[kChunk - 1];
#pragma unroll
  for (int m = 0; m < 8; ++m) S[m] *= all;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Frag d[3];
    split8<3>(u[2 * s] * *(const f32x4 *)&dec[kChunk + 32 * s + 4 * g], u[2 * s + 1] * *(const f32x4 *)&dec[kChunk + 32 * s + 16 + 4 * g], d);
#pragma unroll
    for (int half = 0; half < 8; half += 4) {
      Frag k[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) k[m] = transposed(K, half + m, s, l);
#pragma unroll
      for (int x = 2; x >= 0; --x)
#pragma unroll
        for (int m = 0; m < 4; ++m) S[half + m] = mma(k[m], d[x], S[half + m]);
      place<TIGHT>();
    }
  }
}

// U = T R.
__device__ __forceinline__ void solve(const u32x4 (*T)[3][64], const f32x4 *r, f32x4 *u, int l) {
#pragma unroll
  for (int t = 0; t < 4; ++t) u[t] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Frag R[3];
    split8<3>(r[2 * s], r[2 * s + 1], R);
#pragma unroll
    for (int x = 2; x >= 0; --x) {
      Frag a[4];
#pragma unroll
      for (int t = 2 * s; t < 4; ++t) a[t].w = T[tri_frag(t) + s][x][l];
#pragma unroll
      for (int y = 2 - x; y >= 0; --y)
#pragma unroll
        for (int t = 2 * s; t < 4; ++t) u[t] = mma(a[t], R[y], u[t]);
    }
  }
}

// One wave, sixteen columns, one chunk: DELTA 186 products of 16 cycles and
// 1030 vector instructions of 4, most of them the splitting into parts.  Products of S, R and U take their
// right operands from the accumulators of the product before: nothing but the
// shared left operands is read from LDS, and nothing waits for another wave.
// (Products of one accumulator never follow each other: four at a time.)
template <bool DELTA>
__device__ __forceinline__ void columns(int wave, int l, Stage<DELTA> &st, f32x4 *S) {
  const int g = l >> 4, col = 16 * wave + (l & 15);
  put_A<DELTA>(st, wave, l);
  f32x4 o[4], r[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) o[t] = r[t] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    Frag f[3];
    split8<DELTA ? 3 : 2>(S[2 * s], S[2 * s + 1], f);
    if (DELTA) {
      Frag k[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) k[t] = rows_operand(st.K[t], s, l);
#pragma unroll
      for (int x = 2; x >= 0; --x)
#pragma unroll
        for (int t = 0; t < 4; ++t) r[t] = mma(k[t], f[x], r[t]);
    }
    Frag q[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) q[t] = rows_operand(st.Q[t], s, l);
#pragma unroll
    for (int x = 1; x >= 0; --x)
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] = mma(q[t], f[x], o[t]);
    place<!DELTA>();
  }
  f32x4 u[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const f32x4 from = *(const f32x4 *)&st.dec[16 * t + 4 * g];
    o[t] *= from;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float v = __uint_as_float((uint32_t)st.V[16 * t + 4 * g + x][col] << 16);
      if (DELTA) r[t][x] = __builtin_fmaf(-from[x], r[t][x], v);
      else u[t][x] = v;
    }
  }
  if (DELTA) solve(st.T, r, u, l);
  lds_barrier();   // A is there, and every wave has its values
  // O += A U
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Frag U[2];
    split8<DELTA ? 2 : 1>(u[2 * s], u[2 * s + 1], U);   // SUM: V, exact in one
#pragma unroll
    for (int x = 1; x >= 0; --x) {
      Frag a[4];
#pragma unroll
      for (int t = 2 * s; t < 4; ++t) a[t].w = st.A[tri_frag(t) + s][x][l];
#pragma unroll
      for (int y = DELTA ? 1 - x : 0; y >= 0; --y)
#pragma unroll
        for (int t = 2 * s; t < 4; ++t) o[t] = mma(a[t], U[y], o[t]);
      place<!DELTA>();
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t y = pack_bf16(o[t][2 * x], o[t][2 * x + 1]);
      st.V[16 * t + 4 * g + 2 * x][col] = (uint16_t)y;
      st.V[16 * t + 4 * g + 2 * x + 1][col] = (uint16_t)(y >> 16);
    }
  update_state<!DELTA>(st.K, st.dec, u, S, l);
}

// Which chunks of which sequence a workgroup takes: a whole sequence, or a
// segment of P.segment chunks of one.
__device__ __forceinline__ bool scan_at(const PromptArgs &P, int place, int *b, int *from, int *to, int *segments, ScanAt &A) {
  const int per = P.segment * kChunk;
  *b = P.segment ? sequence_of(P.cu, P.n, per, 1, place) : P.order ? P.order[place] : place;
  if (!rows_of(P.cu, P.T, *b, &A.first, &A.len)) {
    if (threadIdx.x == 0) atomicOr(P.err, kErrLength);
    return false;
  }
  A.row = (size_t)P.H * kD;
  A.chunks = (A.len + kChunk - 1) / kChunk;
  A.place0 = A.first / kChunk + *b;
  *segments = P.segment ? max((A.chunks + P.segment - 1) / P.segment, 1) : 1;
  const int at = P.segment ? place - (A.first / per + *b) : 0;
  *from = at * P.segment;
  *to = P.segment ? min(*from + P.segment, A.chunks) : A.chunks;
  return at >= 0 && at < *segments;
}

// A segment's state in the workspace: a thread's eight results side by side
// with its neighbours'; before k_prompt_join what the segment adds to a state,
// and the decay over it (DELTA: what it makes of 0, and its map), then the state
// that it starts from.
__device__ __forceinline__ f32x4 *segment_ws(const PromptArgs &P, int place, int h, int tid) {
  return (f32x4 *)P.segment_ws + ((size_t)place * P.H + h) * (kD * kD / 4) + tid;
}
__device__ __forceinline__ float *segment_decay(const PromptArgs &P, int place, int h) {
  return P.map_ws + (size_t)place * P.H + h;
}

// The state of a (sequence, head) where it lives.
struct StateAt {
  f32x4 *blk;       // an uncompressed pool's block (four rows of a column together), or
  float *dense;
  __device__ __forceinline__ StateAt(const PromptArgs &P, int b, int slot, int h)
      : blk(P.pool ? (f32x4 *)(P.pool + (size_t)slot * P.slot_stride + (size_t)h * (kD * kD * 4)) : nullptr),
        dense(P.S + ((size_t)b * P.H + h) * kD * kD) {}
  __device__ __forceinline__ f32x4 get(int row, int col) const {
    if (blk) return blk[(row >> 2) * kD + col];
    const float *s = dense + row * kD + col;
    return (f32x4){s[0], s[kD], s[2 * kD], s[3 * kD]};
  }
  __device__ __forceinline__ void set(int row, int col, f32x4 x) const {
    if (blk) blk[(row >> 2) * kD + col] = x;
    else
      for (int r = 0; r < 4; ++r) dense[(row + r) * kD + col] = x[r];
  }
};

// The chunks in order, a wave to sixteen columns.  SUM: two workgroups a compute
// unit, one stages while the other computes (asking a chunk ahead was no faster,
// and the registers for it are not there).  DELTA: one, its rows on their way a
// chunk ahead.  What bounds it is issue: 32 sequences, 16411 tokens, 32 heads
// (DELTA) 286 us with the vector units busy 45% and the matrix cores 39% of the
// time, and little of both at once; 8 sequences, 16000 tokens, 48 heads (SUM)
// 282 us, 39% and 29%.  Tried for DELTA: workgroups of four waves and 64 columns,
// two a compute unit, stage everything twice (316 against 277 us, 16 heads in
// segments); waves of 32 columns need more registers than two a SIMD leave.
template <bool DELTA>
__global__ void __launch_bounds__(512, DELTA ? 2 : 4) k_prompt_scan(PromptArgs P) {
  __shared__ __attribute__((aligned(16))) Stage<DELTA> st;
  const int l = threadIdx.x & 63, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int place = blockIdx.x / P.H, col = 16 * wave + (l & 15);
  int b, from, to, segments;
  ScanAt A;
  A.h = blockIdx.x % P.H;
  if (!scan_at(P, place, &b, &from, &to, &segments, A)) return;
  const int slot = P.slots[b];
  if (slot < 0 || slot >= P.num_slots) {
    if (slot != -1 && threadIdx.x == 0) atomicOr(P.err, kErrSlot);
    const size_t first = (size_t)A.first + (size_t)from * kChunk, rows = min((to - from) * kChunk, A.len - from * kChunk);
    for (size_t i = threadIdx.x; i < rows * kD; i += 512) P.o[(first + i / kD) * A.row + (size_t)A.h * kD + i % kD] = 0;
    return;
  }
  const bool carried = P.carry != nullptr && P.carry[b] != 0;
  const StateAt state(P, b, slot, A.h);
  f32x4 S[8];
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    // (of a cut sequence the slot is written by another workgroup of this launch)
    if (segments > 1) S[m] = segment_ws(P, place, A.h, threadIdx.x)[m * 512];
    else if (carried) S[m] = state.get(state_row(m, g), col);
    else S[m] = (f32x4){0, 0, 0, 0};
  }
  clear_A(st.A, threadIdx.x);
  StageIn<DELTA, true> in;
  if (DELTA && from < to) fetch<DELTA, true>(P, A, from, threadIdx.x, in);
  for (int c = from; c < to; ++c) {
    if (!DELTA) fetch<DELTA, true>(P, A, c, threadIdx.x, in);
    if (c > from) {
      put_rows<DELTA>(P, A, c - 1, threadIdx.x, st);
      lds_barrier();
    }
    put<DELTA, true>(A, c, threadIdx.x, in, st);
    lds_barrier();
    if (DELTA) fetch<DELTA, true>(P, A, min(c + 1, to - 1), threadIdx.x, in);
    columns<DELTA>(wave, l, st, S);
    lds_barrier();
  }
  if (to > from) put_rows<DELTA>(P, A, to - 1, threadIdx.x, st);
  // the last segment has the sequence's state; a slot without rows stays as it is
  if (to < A.chunks || (carried && A.len == 0)) return;
#pragma unroll
  for (int m = 0; m < 8; ++m) state.set(state_row(m, g), col, S[m]);
}

// DELTA with few heads: what counts is how long one chunk takes, for they
// follow each other.  A workgroup takes 32 columns of one (sequence, head),
// and its waves work on three chunks at once.  Between two barriers at a
// chunk's ends there is one in its middle:
//   waves      before it                            after it
//   0, 1       U, the state (sixteen columns each)  U out, S out, the next K S
//   2, 3       A U of the chunk before, Q S         A
//   4 .. 7     the next chunk into LDS              A
// 32768 tokens, 48 heads: 1260 us, 5000 cycles a chunk, all of them waves 0 and
// 1: U 1300, the state 1850, its parts and the next K S 1500 (132 products of 16
// cycles and 430 vector instructions of 4); k_prompt_scan takes 14000.  With K S
// after the barrier 6000, with U split here 5100.  A raised priority of the two
// waves changes nothing.
struct ChainShared {
  struct Part {                       // chunk c in part c & 1
    u32x4 Q[4][256], K[4][256], T[kTriFrags][3][64];
    uint16_t V[kChunk][40];
    float dec[2 * kChunk];
    double lg[kChunk];
  } part[2];
  u32x4 A[kTriFrags][2][64];
  u32x4 S[2][4][2][64];               // [columns][contraction step][part]: the state before the chunk
  f32x4 U[2][4][64];
};
static_assert(sizeof(ChainShared) <= 160 * 1024, "one workgroup has a compute unit's LDS");

// Waves 0, 1: the state's parts for the readout (PUT), and K S of a chunk; one
// step's parts are made beside the products of the step before.
template <bool PUT, bool MULTIPLY>
__device__ __forceinline__ void chain_scores(const f32x4 *S, const u32x4 (*K)[256], u32x4 (*to)[2][64], f32x4 *r, int l) {
  if (MULTIPLY)
#pragma unroll
    for (int t = 0; t < 4; ++t) r[t] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    Frag f[3];
    split8<MULTIPLY ? 3 : 2>(S[2 * s], S[2 * s + 1], f);
    if (PUT)
#pragma unroll
      for (int x = 0; x < 2; ++x) to[s][x][l] = f[x].w;
    if (MULTIPLY) {
      Frag k[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) k[t] = rows_operand(K[t], s, l);
#pragma unroll
      for (int x = 2; x >= 0; --x)
#pragma unroll
        for (int t = 0; t < 4; ++t) r[t] = mma(k[t], f[x], r[t]);
    }
  }
}

// Waves 0, 1: chunk c, whose K S is in r, then the next one's.
__device__ __forceinline__ void chain_chunk(int c, bool more, int col, int l, ChainShared &sh, int group, f32x4 *r, f32x4 *S) {
  const int g = l >> 4;
  const ChainShared::Part &p = sh.part[c & 1];
  f32x4 u[4];
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const f32x4 from = *(const f32x4 *)&p.dec[16 * t + 4 * g];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      r[t][x] = __builtin_fmaf(-from[x], r[t][x], __uint_as_float((uint32_t)p.V[16 * t + 4 * g + x][col] << 16));
  }
  solve(p.T, r, u, l);
  update_state<false>(p.K, p.dec, u, S, l);
  lds_barrier();
#pragma unroll
  for (int t = 0; t < 4; ++t) sh.U[group][t][l] = u[t];
  if (more) chain_scores<true, true>(S, sh.part[(c + 1) & 1].K, sh.S[group], r, l);
}

// Waves 4 .. 7: a thread's share of a chunk on its way in.
struct HelpIn {
  u32x4 q[4], k[4], v;
  f32x4 T[3];
  double lg;
  float dec;
};

__device__ __forceinline__ void help_fetch(const PromptArgs &P, const ScanAt &A, int c, int col0, int tid, HelpIn &in) {
  const int nt = min(kChunk, A.len - c * kChunk);
  const size_t base = ((size_t)A.first + (size_t)c * kChunk) * A.row + (size_t)A.h * kD;
  auto offset = [&](int t) { return (uint32_t)(t < nt ? t : 0) * (uint32_t)(2 * A.row); };
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t at = offset((tid >> 4) + 16 * x) + 16 * (tid & 15);
    in.k[x] = *piece_of(P.k + base, at);
    in.q[x] = *piece_of(P.q + base, at);
  }
  in.v = *piece_of(P.v + base + col0, offset(tid >> 2) + 16 * (tid & 3));
  const ChunkSpace ws = chunk_space(P, A.place0 + c, A.h);
#pragma unroll
  for (int x = 0; x < 3; ++x) in.T[x] = *(const f32x4 *)(ws.T + 4 * (tid + 256 * x));
  in.lg = ws.lg[tid & 63];
  in.dec = ws.dec[tid & 127];
}

__device__ __forceinline__ void help_put(const ScanAt &A, int c, int tid, const HelpIn &in, ChainShared::Part &p) {
  const int nt = A.len - c * kChunk, piece = tid & 15, l = tid & 63, at = piece_at(piece, tid >> 4);
  const u32x4 none = {0, 0, 0, 0};   // nothing of the rows behind the end
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const bool out = (tid >> 4) + 16 * x >= nt;
    p.K[x][at] = out ? none : in.k[x];
    p.Q[x][at] = out ? none : in.q[x];
  }
  *(u32x4 *)&p.V[tid >> 2][8 * (tid & 3)] = tid >> 2 >= nt ? none : in.v;
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int group = (tid >> 6) + 4 * x;
    uint32_t y[2][3];
    parts<3>(in.T[x][0], in.T[x][1], y[0]);
    parts<3>(in.T[x][2], in.T[x][3], y[1]);
#pragma unroll
    for (int z = 0; z < 3; ++z) ((Frag *)&p.T[group >> 1][z][l])->h[group & 1] = (u32x2){y[0][z], y[1][z]};
  }
  if (tid < 64) p.lg[tid] = in.lg;
  else if (tid >= 128) p.dec[tid - 128] = in.dec;
}

// A's ten tiles over waves 2 .. 7: two in step to those beside no chain wave
// (they share their vector units with 2, 3, 6, 7), one to 4 and 5.
__device__ __forceinline__ void help_A(const ChainShared::Part &p, u32x4 (*A)[2][64], int wave, int l) {
  auto tile = [&](int i) {
    const int t = i < 4 ? 3 : i < 7 ? 2 : i < 9 ? 1 : 0, j = i < 4 ? i : i < 7 ? i - 4 : i < 9 ? i - 7 : 0;
    Frag q[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) q[s] = rows_operand(p.Q[t], s, l);
    put_tile(p.K[j], q, p.lg, A, t, j, l);
  };
  if (wave == 4 || wave == 5) {
    tile(wave + 4);
  } else {
    const int i = 2 * ((wave & 1) + (wave >> 2 << 1));
    tile(i);
    tile(i + 1);
  }
}

// Waves 2, 3.
__device__ __forceinline__ void read_state(int c, int l, const ChainShared &sh, int group, f32x4 *o) {
  const ChainShared::Part &p = sh.part[c & 1];
#pragma unroll
  for (int t = 0; t < 4; ++t) o[t] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    Frag q[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) q[t] = rows_operand(p.Q[t], s, l);
#pragma unroll
    for (int x = 1; x >= 0; --x) {
      Frag f;
      f.w = sh.S[group][s][x][l];
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] = mma(q[t], f, o[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) o[t] *= *(const f32x4 *)&p.dec[16 * t + 4 * (l >> 4)];
}

__device__ __forceinline__ void read_chunk(const PromptArgs &P, const ScanAt &A, int c, int col0, int l, const ChainShared &sh, int group, f32x4 *o) {
  const int g = l >> 4, i16 = l & 15, odd = l & 1, nt = A.len - c * kChunk;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Frag U[2];
    split8<2>(sh.U[group][2 * s][l], sh.U[group][2 * s + 1][l], U);
#pragma unroll
    for (int x = 1; x >= 0; --x)
#pragma unroll
      for (int y = 1 - x; y >= 0; --y)
#pragma unroll
        for (int t = 2 * s; t < 4; ++t) {
          Frag a;
          a.w = sh.A[tri_frag(t) + s][x][l];
          o[t] = mma(a, U[y], o[t]);
        }
  }
  // lanes of two neighbouring columns trade rows: two columns of a row a store
  const size_t base = ((size_t)A.first + (size_t)c * kChunk) * A.row + (size_t)A.h * kD + col0;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const uint32_t lo = pack_bf16(o[t][0], o[t][1]), hi = pack_bf16(o[t][2], o[t][3]);
    const uint32_t own = odd ? hi : lo, give = odd ? lo : hi;
    const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0xB1, 0xF, 0xF, true);   // lane ^ 1
    // rows 4 g + 2 odd, + 1 of columns i16 & 14, + 1
    const uint32_t x = odd ? got : own, y = odd ? own : got;
    const int at = 16 * t + 4 * g + 2 * odd;
    uint8_t *dst = (uint8_t *)(P.o + base) + (uint32_t)at * (uint32_t)(2 * A.row) + 2 * (i16 & 14);
    if (at < nt) *(uint32_t *)dst = __builtin_amdgcn_perm(y, x, 0x05040100u);
    if (at + 1 < nt) *(uint32_t *)(dst + 2 * A.row) = __builtin_amdgcn_perm(y, x, 0x07060302u);
  }
}

__global__ void __launch_bounds__(512, 2) k_prompt_chain(PromptArgs P) {
  __shared__ __attribute__((aligned(16))) ChainShared sh;
  // the four slices of a (sequence, head) go to one XCD (workgroups are dealt
  // to the eight in turn) and share its rows through one L2
  const int bh = blockIdx.x / 32 * 8 + blockIdx.x % 8, slice = blockIdx.x / 8 % 4;
  if (bh >= P.n * P.H) return;
  const int l = threadIdx.x & 63, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int b, from, to, segments;
  ScanAt A;
  A.h = bh % P.H;
  if (!scan_at(P, bh / P.H, &b, &from, &to, &segments, A)) return;
  const int slot = P.slots[b];
  if (slot < 0 || slot >= P.num_slots) {
    if (slot != -1 && threadIdx.x == 0) atomicOr(P.err, kErrSlot);
    for (size_t i = threadIdx.x; i < (size_t)A.len * 32; i += 512)
      P.o[((size_t)A.first + i / 32) * A.row + (size_t)A.h * kD + 32 * slice + i % 32] = 0;
    return;
  }
  const int chunks = A.chunks, group = wave & 1, col0 = 32 * slice + 16 * group;
  // Every wave passes 2 chunks + 1 barriers.  Loads are always there (the last
  // chunk asks for itself again): the waits count those behind the ones they need.
  if (wave >= 4) {
    if (chunks == 0) return;
    const int tid = threadIdx.x - 256;
    HelpIn in;
    help_fetch(P, A, 0, 32 * slice, tid, in);
    clear_A(sh.A, tid);
    help_put(A, 0, tid, in, sh.part[0]);
    help_fetch(P, A, min(1, chunks - 1), 32 * slice, tid, in);
    lds_barrier();
    for (int c = 0; c < chunks; ++c) {
      if (c + 1 < chunks) help_put(A, c + 1, tid, in, sh.part[(c + 1) & 1]);
      help_fetch(P, A, min(c + 2, chunks - 1), 32 * slice, tid, in);
      lds_barrier();
      help_A(sh.part[c & 1], sh.A, wave, l);
      lds_barrier();
    }
    return;
  }
  if (wave >= 2) {
    if (chunks == 0) return;
    f32x4 o[4];
    lds_barrier();
    for (int c = 0; c < chunks; ++c) {
      if (c > 0) read_chunk(P, A, c - 1, col0, l, sh, group, o);
      read_state(c, l, sh, group, o);
      lds_barrier();
      help_A(sh.part[c & 1], sh.A, wave, l);
      lds_barrier();
    }
    read_chunk(P, A, chunks - 1, col0, l, sh, group, o);
    return;
  }
  const bool carried = P.carry != nullptr && P.carry[b] != 0;
  const StateAt state(P, b, slot, A.h);
  const int col = col0 + (l & 15);
  f32x4 S[8];
#pragma unroll
  for (int m = 0; m < 8; ++m) S[m] = carried ? state.get(state_row(m, g), col) : (f32x4){0, 0, 0, 0};
  if (chunks > 0) {
    f32x4 r[4];
    chain_scores<true, false>(S, nullptr, sh.S[group], r, l);
    lds_barrier();
    chain_scores<false, true>(S, sh.part[0].K, nullptr, r, l);
    for (int c = 0; c < chunks; ++c) {
      chain_chunk(c, c + 1 < chunks, 16 * group + (l & 15), l, sh, group, r, S);
      lds_barrier();
    }
  }
  if (carried && A.len == 0) return;   // the slot stays as it is
#pragma unroll
  for (int m = 0; m < 8; ++m) state.set(state_row(m, g), col, S[m]);
}

// SUM: what a segment adds to the state it starts from, and the decay over it.
// 105 us of the 8 sequences above, bound as the scan is (44% and 36%).
__global__ void __launch_bounds__(512, 4) k_prompt_segment(PromptArgs P) {
  __shared__ __attribute__((aligned(16))) Stage<false> st;
  const int l = threadIdx.x & 63, g = l >> 4, i16 = l & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int place = blockIdx.x / P.H;
  int b, from, to, segments;
  ScanAt A;
  A.h = blockIdx.x % P.H;
  if (!scan_at(P, place, &b, &from, &to, &segments, A) || to >= A.chunks) return;
  f32x4 S[8];
#pragma unroll
  for (int m = 0; m < 8; ++m) S[m] = (f32x4){0, 0, 0, 0};
  float decay = 1.0f;
  StageIn<false, false> in;
  fetch<false, false>(P, A, from, threadIdx.x, in);
  for (int c = from; c < to; ++c) {
    put<false, false>(A, c, threadIdx.x, in, st);
    lds_barrier();
    fetch<false, false>(P, A, min(c + 1, to - 1), threadIdx.x, in);
    f32x4 u[4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        u[t][x] = __uint_as_float((uint32_t)st.V[16 * t + 4 * g + x][16 * wave + i16] << 16);
    update_state<true>(st.K, st.dec, u, S, l);
    decay *= st.dec[kChunk - 1];
    lds_barrier();
  }
#pragma unroll
  for (int m = 0; m < 8; ++m) segment_ws(P, place, A.h, threadIdx.x)[m * 512] = S[m];
  if (threadIdx.x == 0) *segment_decay(P, place, A.h) = decay;
}

// SUM: the states that the segments start from, a thread to one of its eight
// results: S_0, then S = decay S + what the segment adds.  11 us there, 17 us
// for one sequence of 33 segments: a memory latency each.
__global__ void __launch_bounds__(512) k_prompt_join(PromptArgs P) {
  const int m = blockIdx.x % 8, h = blockIdx.x / 8 % P.H, b = blockIdx.x / (8 * P.H);
  const int l = threadIdx.x & 63, per = P.segment * kChunk;
  int first, len;
  const int slot = P.slots[b];
  if (!rows_of(P.cu, P.T, b, &first, &len)) {   // no segment of k_prompt_scan may be this sequence's
    if (threadIdx.x == 0) atomicOr(P.err, kErrLength);
    return;
  }
  if (slot < 0 || slot >= P.num_slots) return;
  const int segments = (len + per - 1) / per, place = first / per + b;
  if (segments < 2) return;
  f32x4 S = {0, 0, 0, 0};
  if (P.carry != nullptr && P.carry[b] != 0) S = StateAt(P, b, slot, h).get(state_row(m, l >> 4), (threadIdx.x >> 6) * 16 + (l & 15));
  f32x4 next = segment_ws(P, place, h, threadIdx.x)[m * 512];
  for (int i = 0; i < segments; ++i) {
    const f32x4 add = next;
    const float decay = *segment_decay(P, place + i, h);   // (the last one's is not used)
    if (i + 1 < segments) next = segment_ws(P, place + i + 1, h, threadIdx.x)[m * 512];
    segment_ws(P, place + i, h, threadIdx.x)[m * 512] = S;
    S = S * decay + add;
  }
}

// DELTA: what a segment makes of the state S it starts from is P S + B.  A
// workgroup computes B (from S = 0; of a sequence's first segment the state
// that it ends in) or P (from S = 1 and without values), which goes out as the
// left operands of the join: [result][contraction step][part][lane].  5 us a
// chunk while there is a compute unit for every workgroup (4 heads in segments
// of 16 chunks: 82 us), 310 us for 32768 tokens and 16 heads; issue, as the scan.
__device__ __forceinline__ u32x4 *map_ws(const PromptArgs &P, int place, int h) {
  return (u32x4 *)P.map_ws + ((size_t)place * P.H + h) * (kMapFloats / 4);
}

__global__ void __launch_bounds__(512, 2) k_prompt_map(PromptArgs P) {
  __shared__ __attribute__((aligned(16))) union {
    Stage<true> st;
    float S[kD][kD + 4];
  } sh;
  const int l = threadIdx.x & 63, g = l >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int bh = blockIdx.x >> 1, place = bh / P.H, col = 16 * wave + (l & 15);
  const bool turn = blockIdx.x & 1;      // P
  int b, from, to, segments;
  ScanAt A;
  A.h = bh % P.H;
  if (!scan_at(P, place, &b, &from, &to, &segments, A) || to >= A.chunks || (turn && from == 0)) return;
  const int slot = P.slots[b];
  if (slot < 0 || slot >= P.num_slots) return;
  const bool carried = from == 0 && P.carry != nullptr && P.carry[b] != 0;
  const StateAt state(P, b, slot, A.h);
  f32x4 S[8];
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    S[m] = carried ? state.get(state_row(m, g), col) : (f32x4){0, 0, 0, 0};
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (turn && state_row(m, g) + r == col) S[m][r] = 1.0f;
  }
  StageIn<true, false> in;
  fetch<true, false>(P, A, from, threadIdx.x, in);
  for (int c = from; c < to; ++c) {
    put<true, false>(A, c, threadIdx.x, in, sh.st);
    lds_barrier();
    fetch<true, false>(P, A, min(c + 1, to - 1), threadIdx.x, in);
    f32x4 r[4], u[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) r[t] = (f32x4){0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      Frag f[3], k[4];
      split8<3>(S[2 * s], S[2 * s + 1], f);
#pragma unroll
      for (int t = 0; t < 4; ++t) k[t] = rows_operand(sh.st.K[t], s, l);
#pragma unroll
      for (int x = 2; x >= 0; --x)
#pragma unroll
        for (int t = 0; t < 4; ++t) r[t] = mma(k[t], f[x], r[t]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const f32x4 decay = *(const f32x4 *)&sh.st.dec[16 * t + 4 * g];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float v = turn ? 0.0f : __uint_as_float((uint32_t)sh.st.V[16 * t + 4 * g + x][col] << 16);
        r[t][x] = __builtin_fmaf(-decay[x], r[t][x], v);
      }
    }
    solve(sh.st.T, r, u, l);
    update_state<false>(sh.st.K, sh.st.dec, u, S, l);
    lds_barrier();
  }
  if (!turn) {
#pragma unroll
    for (int m = 0; m < 8; ++m) segment_ws(P, place, A.h, threadIdx.x)[m * 512] = S[m];
    return;
  }
#pragma unroll
  for (int m = 0; m < 8; ++m)
#pragma unroll
    for (int r = 0; r < 4; ++r) sh.S[state_row(m, g) + r][col] = S[m][r];
  lds_barrier();
  // row i of result m is channel state_row(m, i >> 2) + (i & 3)
  const int m = wave, i = l & 15, row = state_row(m, i >> 2) + (i & 3);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    Frag f[3];
    split8<3>(*(const f32x4 *)&sh.S[row][32 * s + 8 * g], *(const f32x4 *)&sh.S[row][32 * s + 8 * g + 4], f);
#pragma unroll
    for (int x = 0; x < 3; ++x) map_ws(P, place, A.h)[((m * 4 + s) * 3 + x) * 64 + l] = f[x].w;
  }
}

// DELTA: the states that the segments start from; the first one's is S_0, which
// takes the place of what the segment makes of it.  A
// workgroup takes sixteen columns of a (sequence, head); wave w makes results
// 2 w and 2 w + 1, which are what contraction step w needs of the next state,
// and has the next segment's operands on their way.  1.6 us a segment; one wave
// for all eight results, without operands ahead, took 5.5.
__global__ void __launch_bounds__(256, 1) k_prompt_join_maps(PromptArgs P) {
  __shared__ __attribute__((aligned(16))) u32x4 sf[2][4][3][64];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63;
  const int cols = blockIdx.x % 8, h = blockIdx.x / 8 % P.H, b = blockIdx.x / (8 * P.H);
  const int per = P.segment * kChunk;
  int first, len;
  const int slot = P.slots[b];
  if (!rows_of(P.cu, P.T, b, &first, &len)) {   // (as in k_prompt_join)
    if (threadIdx.x == 0) atomicOr(P.err, kErrLength);
    return;
  }
  if (slot < 0 || slot >= P.num_slots) return;
  const int segments = (len + per - 1) / per, place = first / per + b;
  if (segments < 2) return;
  struct In {
    u32x4 a[2][4][3];
    f32x4 add[2];
  };
  auto state = [&](int i) { return segment_ws(P, place + i, h, 64 * cols + l) + 2 * w * 512; };
  auto load = [&](int i, In &in) {   // (there is none of the last segment: that of the one before again)
    const u32x4 *map = map_ws(P, place + min(i, segments - 2), h) + l;
    const f32x4 *add = state(min(i, segments - 2));
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      in.add[y] = add[y * 512];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int x = 0; x < 3; ++x) in.a[y][s][x] = map[(((2 * w + y) * 4 + s) * 3 + x) * 64];
    }
  };
  f32x4 S[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) S[y] = state(0)[y * 512];
  const bool carried = P.carry != nullptr && P.carry[b] != 0;
  const StateAt start(P, b, slot, h);
#pragma unroll
  for (int y = 0; y < 2; ++y)
    state(0)[y * 512] = carried ? start.get(state_row(2 * w + y, l >> 4), 16 * cols + (l & 15)) : (f32x4){0, 0, 0, 0};
  auto step = [&](int i, In &in) {
#pragma unroll
    for (int y = 0; y < 2; ++y) state(i)[y * 512] = S[y];
    if (i + 1 == segments) return;
    Frag f[3];
    split8<3>(S[0], S[1], f);
#pragma unroll
    for (int x = 0; x < 3; ++x) sf[i & 1][w][x][l] = f[x].w;
    lds_barrier();
#pragma unroll
    for (int y = 0; y < 2; ++y) S[y] = in.add[y];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int z = 2; z >= 0; --z) {
        Frag f, a;
        f.w = sf[i & 1][s][z][l];
#pragma unroll
        for (int x = 2 - z; x >= 0; --x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            a.w = in.a[y][s][x];
            S[y] = mma(a, f, S[y]);
          }
      }
  };
  In odd, even;
  if (segments > 2) load(1, odd);
  for (int i = 1; i < segments; i += 2) {
    if (i + 1 < segments) load(i + 1, even);
    step(i, odd);
    if (i + 1 >= segments) break;
    if (i + 2 < segments) load(i + 2, odd);
    step(i + 1, even);
  }
}

// Slots whose states are unpacked before and packed after the scan.
__global__ void __launch_bounds__(256) k_prompt_slots(PromptArgs P) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= P.n) return;
  int first, len;
  const bool ok = rows_of(P.cu, P.T, b, &first, &len);
  const bool carried = P.carry != nullptr && P.carry[b] != 0;
  const int slot = P.slots[b];
  const bool in_pool = slot >= 0 && slot < P.num_slots;
  P.slots_in[b] = ok && carried && in_pool && len > 0 ? slot : -1;
  P.slots_out[b] = ok && in_pool && !(carried && len == 0) ? slot : -1;
}

}  // namespace

hipError_t launch_prompt_slots(const PromptArgs &a, hipStream_t st) {
  hipLaunchKernelGGL(k_prompt_slots, dim3((a.n + 255) / 256), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_prompt_chunks(const PromptArgs &a, bool delta, hipStream_t st) {
  if (delta) hipLaunchKernelGGL(k_prompt_chunks, dim3(a.chunks * a.H + (a.order ? (a.n + 255) / 256 : 0)), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_prompt_decays, dim3((uint32_t)(((int64_t)a.chunks * a.H + 3) / 4)), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_prompt_scan(const PromptArgs &a, bool delta, hipStream_t st) {
  if (delta) {
    if (a.segment) {
      hipLaunchKernelGGL(k_prompt_map, dim3(a.segments * a.H * 2), dim3(512), 0, st, a);
      hipLaunchKernelGGL(k_prompt_join_maps, dim3(a.n * a.H * 8), dim3(256), 0, st, a);
      hipLaunchKernelGGL(k_prompt_scan<true>, dim3(a.segments * a.H), dim3(512), 0, st, a);
      return hipGetLastError();
    }
    if (in_chains(a.n, a.H)) hipLaunchKernelGGL(k_prompt_chain, dim3((a.n * a.H + 7) / 8 * 32), dim3(512), 0, st, a);
    else hipLaunchKernelGGL(k_prompt_scan<true>, dim3(a.n * a.H), dim3(512), 0, st, a);
    return hipGetLastError();
  }
  if (a.segment) {
    hipLaunchKernelGGL(k_prompt_segment, dim3(a.segments * a.H), dim3(512), 0, st, a);
    hipLaunchKernelGGL(k_prompt_join, dim3(a.n * a.H * 8), dim3(512), 0, st, a);
  }
  hipLaunchKernelGGL(k_prompt_scan<false>, dim3((a.segment ? a.segments : a.n) * a.H), dim3(512), 0, st, a);
  return hipGetLastError();
}

}  // namespace qdr
