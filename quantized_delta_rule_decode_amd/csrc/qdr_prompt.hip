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
// so all of it is matrix products.  Two launches:
//   k_prompt_chunks  everything that does not depend on the state, every
//                    chunk at once: A, and for DELTA T = (I + L)^-1 diag(beta);
//   k_prompt_scan    the chunks in order; the columns of S, U and O do not
//                    mix, so a workgroup takes 16 NT columns of one (sequence,
//                    head) and keeps its part of S in registers throughout.
// Precision: q, k and v are bfloat16 and enter exactly.  Whatever is computed
// (S, U, T, A) enters a product as a sum of bfloat16 parts: three parts (24
// bits, an fp32 value) on the way to the state, two (16 bits) where only the
// bfloat16 readout follows; sums are fp32 in the matrix cores' accumulators.
// The decays are summed in fp64: differences of long sums lose nothing.
#include "qdr_mfma.h"
#include "qdr_mixer.h"

namespace qdr {

namespace {

constexpr int kD = 128;
constexpr int kLd = 68;        // row stride of a 64 x 64 fp32 matrix in LDS
constexpr double kLogZero = -2000.0;   // for log2(0): 2^-2000 is 0, and sums of 64 of it stay finite

// First fragment of row tile w of a triangular matrix.
__device__ __forceinline__ int tri_frag(int w) { return w < 2 ? w : 2 * w - 2; }

__device__ __forceinline__ float *chunk_ws(const PromptArgs &P, int place, int h) {
  return P.chunk_ws + ((size_t)place * P.H + h) * kChunkFloats;
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

// One workgroup per (chunk, head); wave w makes rows 16 w .. 16 w + 15.
template <bool DELTA>
__global__ void __launch_bounds__(256) k_prompt_chunks(PromptArgs P) {
  __shared__ __attribute__((aligned(16))) float mat[2][kChunk][kLd];   // L; A, then X
  __shared__ double lg[kChunk];
  __shared__ __attribute__((aligned(16))) float bt[kChunk];

  const int place = blockIdx.x / P.H, h = blockIdx.x % P.H;
  const int b = sequence_of(P.cu, P.n, kChunk, 1, place);
  int first, len;
  if (!rows_of(P.cu, P.T, b, &first, &len)) return;
  const int c = place - (first / kChunk + b);
  const int slot = P.slots[b];
  if (c < 0 || c * kChunk >= len || slot < 0 || slot >= P.num_slots) return;
  const int nt = min(kChunk, len - c * kChunk);
  const size_t t0 = (size_t)first + (size_t)c * kChunk;

  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  float *ws = chunk_ws(P, place, h);
  const size_t row = (size_t)P.H * kD;

  // rows of q and k as operands: lane (g, i) holds channels 32 s + 8 g .. of
  // token 16 j + i, zero behind the sequence's end
  auto load = [&](const uint16_t *x, int tile, Frag *f) {
    const int t = 16 * tile + i16;
    const uint16_t *src = x + (t0 + (t < nt ? t : 0)) * row + (size_t)h * kD + 8 * g;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      f[s].w = *(const u32x4_a4 *)(src + 32 * s);
      if (t >= nt) f[s].w = (u32x4){0, 0, 0, 0};
    }
  };
  Frag q[4], k[4];
  load(P.q, w, q);
  load(P.k, w, k);

  if (w == 0) {
    const float a = l < nt ? P.gate[(t0 + l) * P.H + h] : 1.0f;
    double x = a == 0.0f ? kLogZero : log2((double)a);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double y = __shfl_up(x, d);
      if (l >= d) x += y;
    }
    lg[l] = x;
    bt[l] = DELTA && l < nt ? P.beta[(t0 + l) * P.H + h] : 0.0f;
    const double end = __shfl(x, 63);
    ws[2 * kTriFloats + l] = exp2f((float)x);
    ws[2 * kTriFloats + kChunk + l] = exp2f((float)(end - x));
  }
  __syncthreads();

  for (int j = 0; j <= w; ++j) {
    Frag kj[4];
    load(P.k, j, kj);
    f32x4 qk = {0, 0, 0, 0}, kk = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      qk = mma(q[s], kj[s], qk);
      if (DELTA) kk = mma(k[s], kj[s], kk);
    }
    const int col = 16 * j + i16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * g + r;
      const float e = exp2f((float)(lg[t] - lg[col]));
      mat[1][t][col] = t >= col ? qk[r] * e : 0.0f;
      if (DELTA) mat[0][t][col] = t > col ? bt[t] * (kk[r] * e) : 0.0f;
    }
  }
  if ((w & 1) == 0) {   // the block above the diagonal that shares a fragment with it
#pragma unroll
    for (int r = 0; r < 4; ++r) mat[1][16 * w + 4 * g + r][16 * (w + 1) + i16] = 0.0f;
  }
  __syncthreads();

  auto store = [&](float *dst, bool scale) {
    for (int s = 0; s <= w >> 1; ++s) {
      f32x4 lo = *(const f32x4 *)&mat[1][16 * w + i16][32 * s + 4 * g];
      f32x4 hi = *(const f32x4 *)&mat[1][16 * w + i16][32 * s + 16 + 4 * g];
      if (scale) {
        lo *= *(const f32x4 *)&bt[32 * s + 4 * g];
        hi *= *(const f32x4 *)&bt[32 * s + 16 + 4 * g];
      }
      float *f = dst + (size_t)(tri_frag(w) + s) * 512 + l * 4;
      *(f32x4 *)f = lo;
      *(f32x4 *)(f + 256) = hi;
    }
  };
  store(ws, false);
  if (!DELTA) return;

  // diagonal block w: column j by forward substitution in lane j
  if (l < 16) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = l == i ? 1.0f : 0.0f;
#pragma unroll
      for (int m = 0; m < i; ++m) s = __builtin_fmaf(-mat[0][16 * w + i][16 * w + m], x[m], s);
      x[i] = s;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) mat[1][16 * w + i][16 * w + l] = x[i];
  }
  __syncthreads();
  if (w == 0) inverse_column<0>(mat[0], mat[1], g, i16);
  else if (w == 1) inverse_column<1>(mat[0], mat[1], g, i16);
  else if (w == 2) inverse_column<2>(mat[0], mat[1], g, i16);
  __syncthreads();
  store(ws + kTriFloats, true);
}

// Eight fp32 values as P bfloat16 operands.
template <int P>
__device__ __forceinline__ void split8(f32x4 a, f32x4 b, Frag *f) {
  uint32_t p[4][P];
  split<P>(a[0], a[1], p[0]);
  split<P>(a[2], a[3], p[1]);
  split<P>(b[0], b[1], p[2]);
  split<P>(b[2], b[3], p[3]);
#pragma unroll
  for (int x = 0; x < P; ++x) f[x].w = (u32x4){p[0][x], p[1][x], p[2][x], p[3][x]};
}
// Four values, each part to its place in a B operand of rows: part x at to + x * stride.
template <int P>
__device__ __forceinline__ void put4(f32x4 a, u32x4 *to, int stride, int half) {
  uint32_t p[2][P];
  split<P>(a[0], a[1], p[0]);
  split<P>(a[2], a[3], p[1]);
#pragma unroll
  for (int x = 0; x < P; ++x) ((Frag *)(to + x * stride))->h[half] = (u32x2){p[0][x], p[1][x]};
}

// What the scan's waves share of a chunk (operands, 1 KiB each).
template <bool DELTA, int NT>
struct ScanShared {
  u32x4 S[3][4][NT][64];                                    // S, three parts
  u32x4 R[DELTA ? 3 : 1][DELTA ? 2 : 1][NT][64];            // V - 2^g K S
  u32x4 U[DELTA ? 2 : 1][2][NT][64];                        // U
  u32x4 D[3][2][NT][64];                                    // 2^(g_63 - g) U
  uint16_t K[kD][72];                                       // K^T; a row's tokens in operand order
  uint16_t V[DELTA ? 16 * NT : 1][DELTA ? 68 : 8];          // V^T
};

// Where a (sequence, head) is.
struct ScanAt {
  int first, len, chunks, place0, h, col0;
  size_t row;
};

// Rows of a 64-row operand: tile w, channels 32 s + 8 g .. of row 16 w + i16.
__device__ __forceinline__ void load_rows(const uint16_t *x, const ScanAt &A, int c, int w, int l, Frag *f) {
  const int nt = min(kChunk, A.len - c * kChunk), t = 16 * w + (l & 15);
  const uint16_t *src = x + ((size_t)A.first + (size_t)c * kChunk + (t < nt ? t : 0)) * A.row + (size_t)A.h * kD + 8 * (l >> 4);
#pragma unroll
  for (int s = 0; s < 4; ++s) f[s].w = *(const u32x4_a4 *)(src + 32 * s);
}
__device__ __forceinline__ void clear_rows(const ScanAt &A, int c, int w, int l, Frag *f) {
  const int nt = A.len - c * kChunk;
  if (nt < kChunk && 16 * w + (l & 15) >= nt)
#pragma unroll
    for (int s = 0; s < 4; ++s) f[s].w = (u32x4){0, 0, 0, 0};
}
// Rows of tile w of a triangular matrix, [fragment][half]; a tile without a
// second fragment reads its first again.
__device__ __forceinline__ void load_tri(const float *m, int w, int l, f32x4 (*t)[2]) {
  const float *f = m + (size_t)tri_frag(w) * 512 + l * 4;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    t[s][0] = *(const f32x4 *)(f + (s > w >> 1 ? 0 : s) * 512);
    t[s][1] = *(const f32x4 *)(f + (s > w >> 1 ? 0 : s) * 512 + 256);
  }
}

// Waves 0 .. 3: the chain from state to state.  What they read of a chunk is
// asked for a whole chunk ahead.
template <bool DELTA, int NT>
struct ChainIn {
  Frag k[4];
  u32x2 v[NT];                // columns 4 (tid & 3) .. of tile n, row tid / 4
  f32x4 T[2][2];
  f32x4 from, to;             // DELTA: decays from the chunk's start, to its end (rows 4 g .. of tile w)
  float end;                  // SUM: to its end, of row tid / 4
  float all;                  // over the whole chunk
};

template <bool DELTA, int NT>
__device__ __forceinline__ void load_chain(const PromptArgs &P, const ScanAt &A, int c, int w, int tid, ChainIn<DELTA, NT> &in) {
  const int l = tid & 63, g = l >> 4, tv = tid >> 2, nt = min(kChunk, A.len - c * kChunk);
  load_rows(P.k, A, c, w, l, in.k);
  const uint16_t *v = P.v + ((size_t)A.first + (size_t)c * kChunk + (tv < nt ? tv : 0)) * A.row + (size_t)A.h * kD + A.col0 + 4 * (tid & 3);
#pragma unroll
  for (int n = 0; n < NT; ++n) in.v[n] = *(const u32x2_a4 *)(v + 16 * n);
  const float *ws = chunk_ws(P, A.place0 + c, A.h), *dec = ws + 2 * kTriFloats;
  if (DELTA) {
    load_tri(ws + kTriFloats, w, l, in.T);
    in.from = *(const f32x4 *)(dec + 16 * w + 4 * g);
    in.to = *(const f32x4 *)(dec + kChunk + 16 * w + 4 * g);
  } else {
    in.end = dec[kChunk + tv];
  }
  in.all = dec[kChunk - 1];
}

// K^T: lanes of two neighbouring tokens trade halves of each word.
__device__ __forceinline__ void put_k(const Frag *k, uint16_t (*K)[72], int w, int l) {
  const int g = l >> 4, i16 = l & 15, odd = l & 1;
  const int pos = 32 * (w >> 1) + 8 * (i16 >> 2) + 4 * (w & 1) + (i16 & 2);
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t own = k[s].u[x];
      const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)own, 0xB1, 0xF, 0xF, true);   // lane ^ 1
      const uint32_t word = odd ? __builtin_amdgcn_perm(own, other, 0x07060302u)
                                : __builtin_amdgcn_perm(other, own, 0x05040100u);
      *(uint32_t *)&K[32 * s + 8 * g + 2 * x + odd][pos] = word;
    }
}

// S as the B operand of contraction step w.
template <bool DELTA, int NT>
__device__ __forceinline__ void put_state(const f32x4 (*S)[NT], ScanShared<DELTA, NT> &sh, int w, int l) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    Frag f[3];
    split8<3>(S[0][n], S[1][n], f);
#pragma unroll
    for (int x = 0; x < 3; ++x) sh.S[x][w][n][l] = f[x].w;
  }
}

// S = 2^g_63 S + K^T D.
template <bool DELTA, int NT>
__device__ __forceinline__ void update_state(f32x4 (*S)[NT], float all, const ScanShared<DELTA, NT> &sh, int w, int l) {
  const int g = l >> 4, i16 = l & 15;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) S[i][n] *= all;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Frag a[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      a[i].w = *(const u32x4 *)&sh.K[32 * w + 8 * (i16 >> 2) + 4 * i + (i16 & 3)][32 * s + 8 * g];
#pragma unroll
    for (int x = 2; x >= 0; --x)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        Frag f;
        f.w = sh.D[x][s][n][l];
#pragma unroll
        for (int i = 0; i < 2; ++i) S[i][n] = mma(a[i], f, S[i][n]);
      }
  }
}

// DELTA's chain over one chunk; three barriers.
template <int NT>
__device__ __forceinline__ void chain_delta(const ScanAt &A, int c, int w, int tid, ChainIn<true, NT> &in, f32x4 (*S)[NT], ScanShared<true, NT> &sh) {
  const int l = tid & 63, g = l >> 4, i16 = l & 15, half = w & 1, step = w >> 1;
  clear_rows(A, c, w, l, in.k);
  if (A.len - c * kChunk <= tid >> 2)
#pragma unroll
    for (int n = 0; n < NT; ++n) in.v[n] = (u32x2){0, 0};
  put_state<true, NT>(S, sh, w, l);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x)
      sh.V[16 * n + 4 * (tid & 3) + x][tid >> 2] = (uint16_t)(in.v[n][x >> 1] >> (16 * (x & 1)));
  lds_barrier();
  f32x4 r[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) r[n] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int x = 2; x >= 0; --x)
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        Frag f;
        f.w = sh.S[x][s][n][l];
        r[n] = mma(in.k[s], f, r[n]);
      }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const u32x2 y = *(const u32x2 *)&sh.V[16 * n + i16][16 * w + 4 * g];
    const f32x4 v = {lo_f32(y[0]), hi_f32(y[0]), lo_f32(y[1]), hi_f32(y[1])};
#pragma unroll
    for (int x = 0; x < 4; ++x) r[n][x] = __builtin_fmaf(-in.from[x], r[n][x], v[x]);
    put4<3>(r[n], &sh.R[0][step][n][l], 2 * NT * 64, half);
  }
  Frag T[2][3];
#pragma unroll
  for (int s = 0; s < 2; ++s) split8<3>(in.T[s][0], in.T[s][1], T[s]);
  lds_barrier();
  // U = T R
  f32x4 u[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) u[n] = (f32x4){0, 0, 0, 0};
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > step) continue;
#pragma unroll
    for (int y = 2; y >= 0; --y)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        Frag f;
        f.w = sh.R[y][s][n][l];
#pragma unroll
        for (int x = 2 - y; x >= 0; --x) u[n] = mma(T[s][x], f, u[n]);
      }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    put4<3>(u[n] * in.to, &sh.D[0][step][n][l], 2 * NT * 64, half);
    put4<2>(u[n], &sh.U[0][step][n][l], 2 * NT * 64, half);
  }
  put_k(in.k, sh.K, w, l);
  lds_barrier();
  update_state<true, NT>(S, in.all, sh, w, l);
}

// SUM's: U = V is there from the start and exact in one part; one barrier,
// and the other half of the shared operands for the next chunk.
template <int NT>
__device__ __forceinline__ void chain_sum(const ScanAt &A, int c, int w, int tid, ChainIn<false, NT> &in, f32x4 (*S)[NT], ScanShared<false, NT> &sh) {
  const int l = tid & 63;
  clear_rows(A, c, w, l, in.k);
  const int t = tid >> 2, e = 4 * ((t >> 4) & 1) + (t & 3);
  const bool out = A.len - c * kChunk <= t;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t y = out ? 0 : in.v[n][x];
      uint32_t p[3];
      split<3>(lo_f32(y) * in.end, hi_f32(y) * in.end, p);
      const int lane = 16 * ((t >> 2) & 3) + 4 * (tid & 3) + 2 * x;
      uint16_t *u = (uint16_t *)&sh.U[0][t >> 5][n][lane] + e;
      u[0] = (uint16_t)y;
      u[8] = (uint16_t)(y >> 16);
#pragma unroll
      for (int z = 0; z < 3; ++z) {
        uint16_t *d = (uint16_t *)&sh.D[z][t >> 5][n][lane] + e;
        d[0] = (uint16_t)p[z];
        d[8] = (uint16_t)(p[z] >> 16);
      }
    }
  put_k(in.k, sh.K, w, l);
  put_state<false, NT>(S, sh, w, l);
  lds_barrier();
  update_state<false, NT>(S, in.all, sh, w, l);
}

// Waves 4 .. 7: the readout, rows of tile w.
struct ReadIn {
  Frag q[4];
  f32x4 A[2][2], from;
};

__device__ __forceinline__ void load_read(const PromptArgs &P, const ScanAt &A, int c, int w, int l, ReadIn &in) {
  load_rows(P.q, A, c, w, l, in.q);
  const float *ws = chunk_ws(P, A.place0 + c, A.h);
  load_tri(ws, w, l, in.A);
  in.from = *(const f32x4 *)(ws + 2 * kTriFloats + 16 * w + 4 * (l >> 4));
}

template <bool DELTA, int NT>
__device__ __forceinline__ void read_chunk(const PromptArgs &P, const ScanAt &A, int c, int w, int l, ReadIn &in, const ScanShared<DELTA, NT> &sh) {
  const int g = l >> 4, i16 = l & 15, step = w >> 1;
  f32x4 o[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) o[n] = (f32x4){0, 0, 0, 0};
  clear_rows(A, c, w, l, in.q);
  lds_barrier();
#pragma unroll
  for (int x = 1; x >= 0; --x)
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        Frag f;
        f.w = sh.S[x][s][n][l];
        o[n] = mma(in.q[s], f, o[n]);
      }
#pragma unroll
  for (int n = 0; n < NT; ++n) o[n] *= in.from;
  Frag a[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s) split8<2>(in.A[s][0], in.A[s][1], a[s]);
  if (DELTA) {
    lds_barrier();
    lds_barrier();
  }
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (s > step) continue;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      Frag f;
      if (DELTA) {
        f.w = sh.U[DELTA ? 1 : 0][s][n][l];
        o[n] = mma(a[s][0], f, o[n]);
      }
      f.w = sh.U[0][s][n][l];
      o[n] = mma(a[s][1], f, o[n]);
      o[n] = mma(a[s][0], f, o[n]);
    }
  }
  // lanes of two neighbouring columns trade rows: two columns of a row a store
  const int nt = min(kChunk, A.len - c * kChunk), odd = l & 1;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint32_t lo = pack_bf16(o[n][0], o[n][1]), hi = pack_bf16(o[n][2], o[n][3]);
    const uint32_t own = odd ? hi : lo, give = odd ? lo : hi;
    const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0xB1, 0xF, 0xF, true);
    // rows 4 g + 2 odd, + 1 of columns i16 & 14, + 1
    const uint32_t x = odd ? got : own, y = odd ? own : got;
    const uint32_t r0 = __builtin_amdgcn_perm(y, x, 0x05040100u), r1 = __builtin_amdgcn_perm(y, x, 0x07060302u);
    const int t = 16 * w + 4 * g + 2 * odd;
    uint16_t *dst = P.o + ((size_t)A.first + (size_t)c * kChunk + t) * A.row + (size_t)A.h * kD + A.col0 + 16 * n + (i16 & 14);
    if (t < nt) *(uint32_t *)dst = r0;
    if (t + 1 < nt) *(uint32_t *)(dst + A.row) = r1;
  }
}

// The chunks in order.  Four waves carry the state from chunk to chunk and
// four read it out beside them: the chain is what the time of a long prompt
// is made of, and everything that it does not need is off it.
template <bool DELTA, int NT>
__global__ void __launch_bounds__(512, 2) k_prompt_scan(PromptArgs P) {
  constexpr int kSlices = 8 / NT;
  __shared__ __attribute__((aligned(16))) ScanShared<DELTA, NT> shared[DELTA ? 1 : 2];

  // the slices of one (sequence, head) go to one XCD (workgroups are dealt to
  // the eight in turn): they share its q, k, A and T through one L2
  const int bh = (blockIdx.x / (8 * kSlices)) * 8 + blockIdx.x % 8;
  if (bh >= P.n * P.H) return;
  const int b = bh / P.H;
  const int tid = threadIdx.x & 255, l = tid & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool chain = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) == 0;

  ScanAt A;
  A.h = bh % P.H;
  A.col0 = (blockIdx.x / 8) % kSlices * 16 * NT;
  A.row = (size_t)P.H * kD;
  if (!rows_of(P.cu, P.T, b, &A.first, &A.len)) {
    if (threadIdx.x == 0) atomicOr(P.err, kErrLength);
    return;
  }
  const int slot = P.slots[b];
  if (slot < 0 || slot >= P.num_slots) {
    if (slot != -1 && threadIdx.x == 0) atomicOr(P.err, kErrSlot);
    for (size_t i = threadIdx.x; i < (size_t)A.len * (16 * NT); i += 512)
      P.o[((size_t)A.first + i / (16 * NT)) * A.row + (size_t)A.h * kD + A.col0 + i % (16 * NT)] = 0;
    return;
  }
  A.chunks = (A.len + kChunk - 1) / kChunk;
  A.place0 = A.first / kChunk + b;

  // A chunk's loads are always there (the last chunk asks for itself again):
  // waits count the loads issued behind the ones they need.
  if (!chain) {
    if (A.chunks == 0) return;
    ReadIn even, odd;
    load_read(P, A, 0, w, l, even);
    for (int c = 0; c < A.chunks; c += 2) {
      load_read(P, A, min(c + 1, A.chunks - 1), w, l, odd);
      read_chunk<DELTA, NT>(P, A, c, w, l, even, shared[0]);
      if (c + 1 >= A.chunks) break;
      load_read(P, A, min(c + 2, A.chunks - 1), w, l, even);
      read_chunk<DELTA, NT>(P, A, c + 1, w, l, odd, shared[DELTA ? 0 : 1]);
    }
    return;
  }

  // S: wave w holds rows 32 w .. 32 w + 31; row 4 g + r of result i is row
  // 32 w + 8 g + 4 i + r, so that a lane's two results are eight rows in a
  // row: the channels that one 16-byte load of q or k has
  const bool carried = P.carry != nullptr && P.carry[b] != 0;
  f32x4 S[2][NT];
  f32x4 *blk = P.pool ? (f32x4 *)(P.pool + (size_t)slot * P.slot_stride + (size_t)A.h * (kD * kD * 4)) : nullptr;
  float *dense = P.S + (size_t)bh * kD * kD;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = A.col0 + 16 * nt + i16;
      if (!carried) S[i][nt] = (f32x4){0, 0, 0, 0};
      else if (blk) S[i][nt] = blk[(8 * w + 2 * g + i) * kD + col];
      else
        for (int r = 0; r < 4; ++r) S[i][nt][r] = dense[(32 * w + 8 * g + 4 * i + r) * kD + col];
    }
  auto step = [&](int c, ChainIn<DELTA, NT> &in, ScanShared<DELTA, NT> &sh) {
    if constexpr (DELTA) chain_delta<NT>(A, c, w, tid, in, S, sh);
    else chain_sum<NT>(A, c, w, tid, in, S, sh);
  };
  if (A.chunks > 0) {
    ChainIn<DELTA, NT> even, odd;
    load_chain<DELTA, NT>(P, A, 0, w, tid, even);
    for (int c = 0; c < A.chunks; c += 2) {
      load_chain<DELTA, NT>(P, A, min(c + 1, A.chunks - 1), w, tid, odd);
      step(c, even, shared[0]);
      if (c + 1 >= A.chunks) break;
      load_chain<DELTA, NT>(P, A, min(c + 2, A.chunks - 1), w, tid, even);
      step(c + 1, odd, shared[DELTA ? 0 : 1]);
    }
  }

  if (carried && A.len == 0) return;   // the slot stays as it is
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = A.col0 + 16 * n + i16;
      if (blk) blk[(8 * w + 2 * g + i) * kD + col] = S[i][n];
      else
        for (int r = 0; r < 4; ++r) dense[(32 * w + 8 * g + 4 * i + r) * kD + col] = S[i][n][r];
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

template <bool DELTA, int NT>
hipError_t scan(const PromptArgs &a, hipStream_t st) {
  const int slices = 8 / NT, bh = (a.n * a.H + 7) / 8;
  hipLaunchKernelGGL((k_prompt_scan<DELTA, NT>), dim3(bh * 8 * slices), dim3(512), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prompt_slots(const PromptArgs &a, hipStream_t st) {
  hipLaunchKernelGGL(k_prompt_slots, dim3((a.n + 255) / 256), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_prompt_chunks(const PromptArgs &a, bool delta, hipStream_t st) {
  const dim3 grid(a.chunks * a.H);
  if (delta) hipLaunchKernelGGL(k_prompt_chunks<true>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_prompt_chunks<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_prompt_scan(const PromptArgs &a, bool delta, hipStream_t st) {
  const bool narrow = (int64_t)a.n * a.H * 8 <= 256;
  if (delta) return narrow ? scan<true, 1>(a, st) : scan<true, 2>(a, st);
  return narrow ? scan<false, 1>(a, st) : scan<false, 2>(a, st);
}

}  // namespace qdr
