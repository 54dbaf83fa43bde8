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
      float *f = dst + (size_t)(tri_frag(w) + s) * 512 + l * 8;
      *(f32x4 *)f = lo;
      *(f32x4 *)(f + 4) = hi;
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

// What a wave of the scan reads of one chunk, held a chunk ahead.
template <bool DELTA, int NT>
struct ChunkIn {
  Frag q[4], k[4];            // rows of tile w; channels 32 s + {4 g.., 16 + 4 g..}
  uint16_t v[NT][4];          // rows 4 g + r of tile w, the wave's columns
  f32x4 A[2][2], T[2][2];     // [fragment][half]
  f32x4 from, to;             // decays from the chunk's start, to its end
  float all;                  // over the whole chunk
};

template <bool DELTA, int NT>
__global__ void __launch_bounds__(256, 2) k_prompt_scan(PromptArgs P) {
  constexpr int kSlices = 8 / NT;
  __shared__ u32x4 sS[3][4][NT][64];                        // S as B operand, three parts
  __shared__ u32x4 sR[DELTA ? 3 : 1][DELTA ? 2 : 1][NT][64];   // V - 2^g K S
  __shared__ u32x4 sU[DELTA ? 2 : 1][2][NT][64];            // U
  __shared__ u32x4 sD[3][2][NT][64];                        // 2^(g_63 - g) U
  __shared__ __attribute__((aligned(16))) uint16_t sK[kD][72];   // K^T; a row's tokens in operand order

  // the slices of one (sequence, head) go to one XCD (workgroups are dealt to
  // the eight in turn): they share its q, k, A and T through one L2
  const int bh = (blockIdx.x / (8 * kSlices)) * 8 + blockIdx.x % 8;
  const int slice = (blockIdx.x / 8) % kSlices;
  if (bh >= P.n * P.H) return;
  const int b = bh / P.H, h = bh % P.H;
  const int tid = threadIdx.x, l = tid & 63, g = l >> 4, i16 = l & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col0 = slice * 16 * NT;
  const size_t row = (size_t)P.H * kD;

  int first, len;
  if (!rows_of(P.cu, P.T, b, &first, &len)) {
    if (tid == 0) atomicOr(P.err, kErrLength);
    return;
  }
  const int slot = P.slots[b];
  if (slot < 0 || slot >= P.num_slots) {
    if (slot != -1 && tid == 0) atomicOr(P.err, kErrSlot);
    for (size_t i = tid; i < (size_t)len * (16 * NT); i += 256)
      P.o[((size_t)first + i / (16 * NT)) * row + (size_t)h * kD + col0 + i % (16 * NT)] = 0;
    return;
  }
  const bool carried = P.carry != nullptr && P.carry[b] != 0;

  // S: wave w holds rows 32 w + 16 i + 4 g + r
  f32x4 S[2][NT];
  f32x4 *blk = P.pool ? (f32x4 *)(P.pool + (size_t)slot * P.slot_stride + (size_t)h * (kD * kD * 4)) : nullptr;
  float *dense = P.S + (size_t)bh * kD * kD;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = col0 + 16 * nt + i16;
      if (!carried) S[i][nt] = (f32x4){0, 0, 0, 0};
      else if (blk) S[i][nt] = blk[(8 * w + 4 * i + g) * kD + col];
      else
        for (int r = 0; r < 4; ++r) S[i][nt][r] = dense[(32 * w + 16 * i + 4 * g + r) * kD + col];
    }

  const int chunks = (len + kChunk - 1) / kChunk;
  const int place0 = first / kChunk + b;
  auto load = [&](int c, ChunkIn<DELTA, NT> &in) {
    const int nt = min(kChunk, len - c * kChunk);
    const size_t t0 = (size_t)first + (size_t)c * kChunk;
    const int t = 16 * w + i16;
    const size_t at = (t0 + (t < nt ? t : 0)) * row + (size_t)h * kD + 4 * g;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      in.q[s].h[0] = *(const u32x2_a4 *)(P.q + at + 32 * s);
      in.q[s].h[1] = *(const u32x2_a4 *)(P.q + at + 32 * s + 16);
      in.k[s].h[0] = *(const u32x2_a4 *)(P.k + at + 32 * s);
      in.k[s].h[1] = *(const u32x2_a4 *)(P.k + at + 32 * s + 16);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tv = 16 * w + 4 * g + r;
      const uint16_t *src = P.v + (t0 + (tv < nt ? tv : 0)) * row + (size_t)h * kD + col0 + i16;
#pragma unroll
      for (int n = 0; n < NT; ++n) in.v[n][r] = src[16 * n];
    }
    const float *ws = chunk_ws(P, place0 + c, h);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s > w >> 1) continue;
      const float *f = ws + (size_t)(tri_frag(w) + s) * 512 + l * 8;
      in.A[s][0] = *(const f32x4 *)f;
      in.A[s][1] = *(const f32x4 *)(f + 4);
      if (DELTA) {
        in.T[s][0] = *(const f32x4 *)(f + kTriFloats);
        in.T[s][1] = *(const f32x4 *)(f + kTriFloats + 4);
      }
    }
    const float *dec = ws + 2 * kTriFloats;
    in.from = *(const f32x4 *)(dec + 16 * w + 4 * g);
    in.to = *(const f32x4 *)(dec + kChunk + 16 * w + 4 * g);
    in.all = dec[kChunk - 1];
  };

  ChunkIn<DELTA, NT> in;
  if (chunks > 0) load(0, in);
  for (int c = 0; c < chunks; ++c) {
    const int nt = min(kChunk, len - c * kChunk);
    const size_t t0 = (size_t)first + (size_t)c * kChunk;
    {   // nothing of the rows behind the end
      const bool out = 16 * w + i16 >= nt;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        if (out) in.q[s].w = in.k[s].w = (u32x4){0, 0, 0, 0};
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (16 * w + 4 * g + r >= nt) in.v[n][r] = 0;
    }
    // S as the B operand of contraction step w
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      uint32_t p[4][3];
      split<3>(S[0][n][0], S[0][n][1], p[0]);
      split<3>(S[0][n][2], S[0][n][3], p[1]);
      split<3>(S[1][n][0], S[1][n][1], p[2]);
      split<3>(S[1][n][2], S[1][n][3], p[3]);
#pragma unroll
      for (int x = 0; x < 3; ++x) sS[x][w][n][l] = (u32x4){p[0][x], p[1][x], p[2][x], p[3][x]};
    }
    // K^T: lanes of two neighbouring tokens trade halves of each word
    {
      const int t = 16 * w + i16, odd = t & 1;
      const int pos = 32 * (w >> 1) + 8 * ((i16 >> 2)) + 4 * (w & 1) + (t & 2);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t own = in.k[s].u[x];
          const uint32_t other = (uint32_t)__builtin_amdgcn_mov_dpp((int)own, 0xB1, 0xF, 0xF, true);   // lane ^ 1
          const uint32_t word = odd ? __builtin_amdgcn_perm(own, other, 0x07060302u)
                                    : __builtin_amdgcn_perm(other, own, 0x05040100u);
          const int d = 32 * s + 16 * (x >> 1) + 4 * g + 2 * (x & 1) + odd;
          *(uint32_t *)&sK[d][pos] = word;
        }
    }
    float v[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[n][r] = __uint_as_float((uint32_t)in.v[n][r] << 16);
    const int half = w & 1, step = w >> 1;
    if (!DELTA) {   // U = V is known: exact in one part
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        ((Frag *)&sU[0][step][n][l])->h[half] = (u32x2){pack_bf16(v[n][0], v[n][1]), pack_bf16(v[n][2], v[n][3])};
        uint32_t p[2][3];
        split<3>(v[n][0] * in.to[0], v[n][1] * in.to[1], p[0]);
        split<3>(v[n][2] * in.to[2], v[n][3] * in.to[3], p[1]);
#pragma unroll
        for (int x = 0; x < 3; ++x) ((Frag *)&sD[x][step][n][l])->h[half] = (u32x2){p[0][x], p[1][x]};
      }
    }
    __syncthreads();

    // rows of tile w: Q S, and K S for DELTA
    f32x4 o[NT], r0[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n] = r0[n] = (f32x4){0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 2; x >= 0; --x) {
          Frag f;
          f.w = sS[x][s][n][l];
          if (DELTA) r0[n] = mma(in.k[s], f, r0[n]);
          if (x < 2) o[n] = mma(in.q[s], f, o[n]);
        }
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n] *= in.from;
    if (DELTA) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float r[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) r[x] = __builtin_fmaf(-in.from[x], r0[n][x], v[n][x]);
        uint32_t p[2][3];
        split<3>(r[0], r[1], p[0]);
        split<3>(r[2], r[3], p[1]);
#pragma unroll
        for (int x = 0; x < 3; ++x) ((Frag *)&sR[x][step][n][l])->h[half] = (u32x2){p[0][x], p[1][x]};
      }
      __syncthreads();
      // U = T R
      f32x4 u[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) u[n] = (f32x4){0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (s > step) continue;
        uint32_t p[4][3];
        split<3>(in.T[s][0][0], in.T[s][0][1], p[0]);
        split<3>(in.T[s][0][2], in.T[s][0][3], p[1]);
        split<3>(in.T[s][1][0], in.T[s][1][1], p[2]);
        split<3>(in.T[s][1][2], in.T[s][1][3], p[3]);
        Frag a[3];
#pragma unroll
        for (int x = 0; x < 3; ++x) a[x].w = (u32x4){p[0][x], p[1][x], p[2][x], p[3][x]};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int y = 2; y >= 0; --y) {
            Frag f;
            f.w = sR[y][s][n][l];
#pragma unroll
            for (int x = 2 - y; x >= 0; --x) u[n] = mma(a[x], f, u[n]);
          }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t p[2][3];
        split<2>(u[n][0], u[n][1], p[0]);
        split<2>(u[n][2], u[n][3], p[1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) ((Frag *)&sU[x][step][n][l])->h[half] = (u32x2){p[0][x], p[1][x]};
        u[n] *= in.to;
        split<3>(u[n][0], u[n][1], p[0]);
        split<3>(u[n][2], u[n][3], p[1]);
#pragma unroll
        for (int x = 0; x < 3; ++x) ((Frag *)&sD[x][step][n][l])->h[half] = (u32x2){p[0][x], p[1][x]};
      }
      __syncthreads();
    }
    // O += A U
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (s > step) continue;
      uint32_t p[4][2];
      split<2>(in.A[s][0][0], in.A[s][0][1], p[0]);
      split<2>(in.A[s][0][2], in.A[s][0][3], p[1]);
      split<2>(in.A[s][1][0], in.A[s][1][1], p[2]);
      split<2>(in.A[s][1][2], in.A[s][1][3], p[3]);
      Frag a[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) a[x].w = (u32x4){p[0][x], p[1][x], p[2][x], p[3][x]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        Frag f;
        if (DELTA) {
          f.w = sU[DELTA ? 1 : 0][s][n][l];
          o[n] = mma(a[0], f, o[n]);
        }
        f.w = sU[0][s][n][l];
        o[n] = mma(a[1], f, o[n]);
        o[n] = mma(a[0], f, o[n]);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * w + 4 * g + r;
      if (t < nt) {
        uint16_t *dst = P.o + (t0 + t) * row + (size_t)h * kD + col0 + i16;
#pragma unroll
        for (int n = 0; n < NT; ++n) dst[16 * n] = (uint16_t)pack_bf16(o[n][r], 0.0f);
      }
    }
    const float all = in.all;
    if (c + 1 < chunks) load(c + 1, in);
    // S = 2^g_63 S + K^T D
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) S[i][n] *= all;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        Frag a;
        a.w = *(const u32x4 *)&sK[32 * w + 16 * i + i16][32 * s + 8 * g];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 2; x >= 0; --x) {
            Frag f;
            f.w = sD[x][s][n][l];
            S[i][n] = mma(a, f, S[i][n]);
          }
      }
    // the next chunk writes sS, sK (and sU, sD for SUM) before its first
    // barrier: every wave has to be done with them
    __syncthreads();
  }

  if (carried && len == 0) return;   // the slot stays as it is
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = col0 + 16 * n + i16;
      if (blk) blk[(8 * w + 4 * i + g) * kD + col] = S[i][n];
      else
        for (int r = 0; r < 4; ++r) dense[(32 * w + 16 * i + 4 * g + r) * kD + col] = S[i][n][r];
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
  hipLaunchKernelGGL((k_prompt_scan<DELTA, NT>), dim3(bh * 8 * slices), dim3(256), 0, st, a);
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
  const bool narrow = (int64_t)a.n * a.H * 4 < 512;
  if (delta) return narrow ? scan<true, 1>(a, st) : scan<true, 2>(a, st);
  return narrow ? scan<false, 1>(a, st) : scan<false, 2>(a, st);
}

}  // namespace qdr
