// qdr_kv.hip -- quantising keys and values as they enter the paged cache, and
// reading them back.
// 8-bit: r = max |x| over the head's 128 channels (1 below 2^-126), z =
// nearest-even(127 x / r), scale r / 127.  x and r are bfloat16, so 127 x is
// exact in fp32 and the quotient is no nearer to a half-integer than 2^-9
// unless it is one.  Times 1/r it is right to a few units of 2^-23, and one
// step q + (127 x - q r) / r, whose difference is exact, returns a quotient
// that fp32 holds (a half-integer) exactly: the definition's code in every case.
// A workgroup takes one block (32 consecutive positions) of one (sequence,
// head), so that the values, which the cache keeps transposed, leave in whole
// 16-byte units wherever all their eight tokens are in the call; at a ragged
// end the bytes of other tokens are not touched.  512 B in and 264 (8-bit) or
// 512 B out a token and head.  16391 tokens of 8 heads, 8-bit: writing 21 us
// (4.9 TB/s; the vector units are busy 89% of the time with the quotients, which
// took 30 us as divisions and with bank conflicts in the transposition), reading
// 18 us (5.5 TB/s).  64 tokens: 6 and 4 us, latency.
#include "qdr_cache.h"
#include "qdr_mfma.h"
#include "qdr_paged.h"
#include "qdr_rotary.h"

namespace qdr {

namespace {

constexpr int kD = 128;

// The block a workgroup works on; lo .. hi are its positions that the call has.
struct Where {
  int lo, hi;            // 0 .. 32
  int pos;               // of its first token
  long long token0;      // row of position 0 of the block (rows lo .. hi exist)
  bool fits;             // false: the sequence is skipped
  uint8_t *blk;          // NULL: skipped, or a bad page
};

template <int KIND>
__device__ __forceinline__ bool locate(const KvArgs &P, int place, int h, Where &at) {
  if (blockIdx.x == 0) check_counts(P);
  // a sequence of len rows touches at most len/32 + 2 blocks
  const int b = sequence_of(P.cu, P.n, kBlock, 2, place);
  int first, len;
  const bool counts = rows_of(P.cu, P.T, b, &first, &len);
  const int i = place - ((counts ? first / kBlock : 0) + 2 * b);
  if (!counts || len == 0 || i < 0) return false;
  const int ctx = P.context[b];
  const bool fits = ctx >= len && ctx <= room_of(P);
  const int p0 = fits ? ctx - len : 0;            // position of row 0; rows stay in place where they are only cleared
  const int block = p0 / kBlock + i;
  const int pos = block * kBlock;
  at.lo = max(p0 - pos, 0);
  at.hi = min(p0 + len - pos, kBlock);
  if (at.lo >= at.hi) return false;
  at.pos = pos;
  at.token0 = (long long)first + pos - p0;
  at.fits = fits;
  at.blk = nullptr;
  if (!fits) return true;
  const int page = P.pages[(size_t)b * P.max_pages + (pos >> P.page_shift)];
  if (page < 0 || page >= P.num_pages) {
    if (threadIdx.x == 0) atomicOr(P.err, kErrPage);
    return true;
  }
  const int per = 1 << (P.page_shift - 5);
  at.blk = P.base + (((size_t)page * P.heads + h) * per + (block & (per - 1))) * (KIND == 8 ? kKv8Block : kKv16Block);
  return true;
}

// Place of token r (0..31) among the eight tokens of its lane group.
__device__ __forceinline__ int slot_of(int r) { return 4 * (r >> 4) + (r & 3); }
__device__ __forceinline__ int group_of(int r) { return (r >> 2) & 3; }

// Where a channel's tokens are in LDS: eight bytes more every 16 channels put
// the eight threads of a token (16 channels each) on banks of their own.
template <int E>
__device__ __forceinline__ int channel_at(int ch) { return ch * (kBlock * E + 8) + 8 * (ch >> 4); }
template <int E>
constexpr int kChannels = kD * (kBlock * E + 8) + 8 * (kD / 16);

__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Codes of 16 channels and the vector's scale.  |x| as integers order like
// the values, with infinity and NaN above them, so r is NaN for a vector that
// holds one, and the scale then is.
__device__ __forceinline__ u32x4 quantise(const u32x4 *x, float *scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = x[i >> 2][i & 3];
    m = max_u16(m, max_u16(w & 0x7FFFu, (w >> 16) & 0x7FFFu));
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) m = max_u16(m, (uint32_t)__shfl_xor((int)m, d));
  // infinity over 127 is infinity, and 0 times it NaN; but a code of 127 or
  // -127 would read back as infinity: make every such vector NaN
  float r = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __uint_as_float(m << 16);
  if (m < 0x0080u) r = 1.0f;
  *scale = __fdiv_rn(r, 127.0f);
  // 127 x has to stay finite, and what is left of it after q r exact
  const float by = r > 0x1p100f ? 0x1p-10f : r < 0x1p-60f ? 0x1p64f : 1.0f;
  r *= by;
  const float inv = __builtin_amdgcn_rcpf(r);
  u32x4 z;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w = x[(4 * i + j) >> 3][((4 * i + j) >> 1) & 3];
      const float y = (j & 1) ? hi_f32(w) : lo_f32(w);
      const float x127 = 127.0f * (y * by), q = x127 * inv;
      const float t = rintf(__builtin_fmaf(__builtin_fmaf(-q, r, x127), inv, q));
      word |= ((uint32_t)(int)(t == t ? t : 0.0f) & 0xFFu) << (8 * j);
    }
    z[i] = word;
  }
  return z;
}

// V of tokens lo .. hi of a block, channel by channel in LDS, to the cache.
template <int KIND>
__device__ __forceinline__ void store_values(const uint8_t *sv, uint8_t *blk, int lo, int hi) {
  constexpr int E = KIND / 8;
  uint8_t *dst = blk + (KIND == 8 ? kKv8Half : kKv16Half);
#pragma unroll
  for (int x = 0; x < E; ++x) {                     // 256 E units of 16 B
    const int unit = threadIdx.x + 256 * x, lane = unit & 63, gg = lane >> 4, m = lane & 15;
    // the tokens of lane group gg: 4 gg + {0..3, 16..19}
    const bool whole = lo <= 4 * gg && hi >= 20 + 4 * gg;
#pragma unroll
    for (int part = 0; part < (KIND == 8 ? 2 : 1); ++part) {
      const int ch = KIND == 8 ? 32 * (unit >> 6) + 16 * part + m : 16 * (unit >> 6) + m;
      const uint8_t *src = &sv[channel_at<E>(ch) + 8 * E * gg];
      uint8_t *to = dst + unit * 16 + 8 * part;
      if (whole) {
        *(u32x2 *)to = *(const u32x2 *)src;
        if (KIND == 16) *(u32x2 *)(to + 8) = *(const u32x2 *)(src + 8);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int t = 4 * gg + (e & 3) + 16 * (e >> 2);
          if (t < lo || t >= hi) continue;
          if (KIND == 8) to[e] = src[e];
          else ((uint16_t *)to)[e] = ((const uint16_t *)src)[e];
        }
      }
    }
  }
}

template <int KIND>
__global__ void __launch_bounds__(256) k_kv_write(KvArgs P) {
  constexpr int E = KIND / 8;                       // bytes of an element
  __shared__ __attribute__((aligned(16))) uint8_t sv[kChannels<E>];   // V, channel by channel
  Where at;
  const int h = blockIdx.x % P.heads;
  if (!locate<KIND>(P, blockIdx.x / P.heads, h, at) || !at.blk) return;
  const int tid = threadIdx.x, r = tid >> 3, seg = tid & 7;
  const bool in = r >= at.lo && r < at.hi;
  const size_t off = ((size_t)(at.token0 + (in ? r : at.lo)) * P.heads + h) * kD + 16 * seg;
  u32x4 k[2], v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    k[i] = *(const u32x4_a4 *)(P.k + off + 8 * i);
    v[i] = *(const u32x4_a4 *)(P.v + off + 8 * i);
  }
  const int tile = r >> 4, key = r & 15;
  const int half = seg >> 2, g = seg & 3;
  const int pos = 8 * group_of(r) + slot_of(r);     // token order within a channel
  if (KIND == 8) {
    float ks, vs;
    const u32x4 kz = quantise(k, &ks), vz = quantise(v, &vs);
    if (in) {
      *(u32x4 *)(at.blk + ((tile * 2 + half) * 64 + g * 16 + key) * 16) = kz;
      if (seg == 0) {
        *(float *)(at.blk + kKv8Scale + 4 * r) = ks;
        *(float *)(at.blk + kKv8Scale + 4 * kBlock + 4 * r) = vs;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) sv[channel_at<E>(16 * seg + i) + pos] = (uint8_t)(vz[i >> 2] >> (8 * (i & 3)));
    }
  } else if (in) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      *(u32x4 *)(at.blk + ((tile * 4 + half * 2 + p) * 64 + g * 16 + key) * 16) = k[p];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      *(uint16_t *)&sv[channel_at<E>(16 * seg + i) + 2 * pos] = (uint16_t)(v[i >> 3][(i >> 1) & 3] >> (16 * (i & 1)));
  }
  __syncthreads();
  store_values<KIND>(sv, at.blk, at.lo, at.hi);
}

// Codes of 16 fp32 channels and the vector's scale: nearest(127 x / r) with the
// quotient as a product, right to two units of 2^-23 (what is less sure than
// that is x itself, which two fp32 products made).
__device__ __forceinline__ u32x4 quantise(const float *x, float *scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t a = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    m = a > m ? a : m;
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) {
    const uint32_t a = (uint32_t)__shfl_xor((int)m, d);
    m = a > m ? a : m;
  }
  float r = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(m);
  if (m < 0x00800000u) r = 1.0f;
  *scale = __fdiv_rn(r, 127.0f);
  const float by = r < 0x1p-60f ? 0x1p64f : 1.0f;      // 127 / r has to stay finite
  const float inv = __fdiv_rn(127.0f, r * by);
  u32x4 z;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t word = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float t = rintf(x[4 * i + j] * by * inv);
      word |= ((uint32_t)(int)(t == t ? t : 0.0f) & 0xFFu) << (8 * j);
    }
    z[i] = word;
  }
  return z;
}

// The write with keys turned on the way, and the queries turned beside it.  A
// workgroup takes one block of one sequence and some key heads, or some query
// heads: the sines and cosines of its tokens are made once, in LDS, while the
// first rows are on their way.  A key row's thread has 16 channels in a row; what
// they are paired with in the half layout are 16 others of the same row, which
// it reads a second time (from the cache) rather than trade them between lanes.
// Queries go as in qdr_rotary.hip.  Bound by memory: 16391 tokens of 5 prompts, 32
// query and 8 key heads, bfloat16: 77 us for 403 MB (5.2 TB/s) when the queries
// stayed in the caches, with qdr_kv_read of it all 112.5 us a pass and 106.7 now.
// (8-bit, 472 MB: 101.5.)  64 single tokens: 8 us of kernel (bfloat16 7), the latency
// of counts, context, page and rows one after the other, and a token's values leave
// byte by byte.
template <int KIND>
__global__ void __launch_bounds__(256) k_kv_write_rotary(RotaryWriteArgs A) {
  constexpr int E = KIND / 8, kPasses = 4;
  __shared__ __attribute__((aligned(16))) uint8_t sv[2][kChannels<E>];
  __shared__ __attribute__((aligned(16))) CosSin table[kBlock][kTableRow];
  const KvArgs &P = A.kv;
  const int parts = A.kv_parts + A.query_parts, part = blockIdx.x % parts;
  const bool keys = part < A.kv_parts;
  Where at;
  if (!locate<KIND>(P, blockIdx.x / parts, 0, at) || (keys && !at.blk)) return;
  const int tid = threadIdx.x, pairs = A.rotary.channels >> 1;

  auto make_table = [&]() {
    const int pair = tid & 63;
    const uint64_t f = pair < pairs ? A.rotary.turns[pair] : 0;
    for (int r = at.lo + (tid >> 6); r < at.hi; r += 4) {
      CosSin w = cos_sin(f, at.pos + r);
      w.c *= A.rotary.amplitude;
      w.s *= A.rotary.amplitude;
      table[r][pair] = w;
    }
    lds_barrier();
  };

  if (!keys) {
    const int h0 = (part - A.kv_parts) * A.query_heads, heads = min(A.query_heads, A.q_heads - h0);
    const int rows = (at.hi - at.lo) * heads;
    const Units u = units_of(A.rotary.channels, A.rotary.layout, tid & 7);
    for (int base = 0; base < rows; base += 32 * kPasses) {
      u32x4 a[kPasses], b[kPasses];
      int tok[kPasses], head[kPasses];
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const int row = min(base + 32 * i + (tid >> 3), rows - 1);
        tok[i] = row / heads;
        head[i] = h0 + row - tok[i] * heads;
        tok[i] += at.lo;
        const size_t from = (size_t)(at.token0 + tok[i]) * A.q_stride + (size_t)head[i] * kD;
        a[i] = read_once(A.q + from + u.c0);
        b[i] = read_once(A.q + from + u.c1);
      }
      if (base == 0) make_table();
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (base + 32 * i + (tid >> 3) >= rows) continue;
        if (!at.fits) {
          a[i] = b[i] = (u32x4){0, 0, 0, 0};
        } else if (u.turn0) {
          float x[16];
          widen16(a[i], x);
          widen16(b[i], x + 8);
          turn_units(u, table[tok[i]], x);
          a[i] = narrow16(x);
          if (u.turn1) b[i] = narrow16(x + 8);
        }
        const size_t to = ((size_t)(at.token0 + tok[i]) * A.q_heads + head[i]) * kD;
        write_past(A.q_out + to + u.c0, a[i]);
        write_past(A.q_out + to + u.c1, b[i]);
      }
    }
    return;
  }

  const int h0 = part * A.kv_heads, h1 = min(h0 + A.kv_heads, P.heads);
  const int r = tid >> 3, seg = tid & 7, half = seg >> 2, g = seg & 3, tile = r >> 4, key = r & 15;
  const bool in = r >= at.lo && r < at.hi;
  const long long row = at.token0 + (in ? r : at.lo);
  const int pos = 8 * group_of(r) + slot_of(r);
  const size_t page_step = (size_t)(KIND == 8 ? kKv8Block : kKv16Block) << (P.page_shift - 5);   // of a head
  // the thread's two units of eight channels and, of the half layout, their partners'
  const bool apart = A.rotary.layout == 0;
  const int half_units = A.rotary.channels >> 4;
  int unit_pairs[2], partner[2];
  bool turns[2], second[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = 2 * seg + i;
    turns[i] = u < 2 * half_units;
    second[i] = u >= half_units;
    partner[i] = !turns[i] ? u : second[i] ? u - half_units : u + half_units;
    unit_pairs[i] = second[i] ? u - half_units : u;
  }
  u32x4 k[2], other[2], v[2];
  auto load = [&](int h) {
    const uint16_t *from = P.k + row * A.k_stride + (size_t)h * kD, *values = P.v + row * A.v_stride + (size_t)h * kD;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      k[i] = *(const u32x4_a4 *)(from + 16 * seg + 8 * i);
      v[i] = *(const u32x4_a4 *)(values + 16 * seg + 8 * i);
      if (apart) other[i] = *(const u32x4_a4 *)(from + 8 * partner[i]);
    }
  };
  load(h0);
  make_table();
  for (int h = h0; h < h1; ++h) {
    uint8_t *blk = at.blk + h * page_step, *to = sv[(h - h0) & 1];
    float x[16];
    widen16(k[0], x);
    widen16(k[1], x + 8);
    if (apart) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!turns[i]) continue;
        CosSin w[8];
        float y[8], unused;
        pairs_of(table[in ? r : at.lo], 2 * unit_pairs[i], w);
        pairs_of(table[in ? r : at.lo], 2 * unit_pairs[i] + 1, w + 4);
        widen16(other[i], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (second[i]) turn(y[e], x[8 * i + e], w[e], &unused, &x[8 * i + e]);
          else turn(x[8 * i + e], y[e], w[e], &x[8 * i + e], &unused);
        }
      }
    } else if (turns[0]) {   // (and with it turns[1])
      CosSin w[8];
      pairs_of(table[in ? r : at.lo], 2 * seg, w);
      pairs_of(table[in ? r : at.lo], 2 * seg + 1, w + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) turn(x[2 * e], x[2 * e + 1], w[e], &x[2 * e], &x[2 * e + 1]);
    }
    const u32x4 v0[2] = {v[0], v[1]};
    if (h + 1 < h1) load(h + 1);
    if (KIND == 8) {
      float ks, vs;
      const u32x4 kz = quantise(x, &ks), vz = quantise(v0, &vs);
      if (in) {
        *(u32x4 *)(blk + ((tile * 2 + half) * 64 + g * 16 + key) * 16) = kz;
        if (seg == 0) {
          *(float *)(blk + kKv8Scale + 4 * r) = ks;
          *(float *)(blk + kKv8Scale + 4 * kBlock + 4 * r) = vs;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) to[channel_at<E>(16 * seg + i) + pos] = (uint8_t)(vz[i >> 2] >> (8 * (i & 3)));
      }
    } else if (in) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
        *(u32x4 *)(blk + ((tile * 4 + half * 2 + p) * 64 + g * 16 + key) * 16) = turns[p] ? narrow16(x + 8 * p) : unwiden16(x + 8 * p);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *(uint16_t *)&to[channel_at<E>(16 * seg + i) + 2 * pos] = (uint16_t)(v0[i >> 3][(i >> 1) & 3] >> (16 * (i & 1)));
    }
    // two buffers in turn: a wave is a head behind another at most
    lds_barrier();
    store_values<KIND>(to, blk, at.lo, at.hi);
  }
}

__device__ __forceinline__ uint32_t two_codes(uint32_t w, int byte, float s) {
  return pack_bf16((float)(int8_t)(w >> (8 * byte)) * s, (float)(int8_t)(w >> (8 * byte + 8)) * s);
}

template <int KIND>
__global__ void __launch_bounds__(256) k_kv_read(KvArgs P) {
  constexpr int E = KIND / 8;
  __shared__ __attribute__((aligned(16))) uint8_t sv[kChannels<E>];
  Where at;
  const int h = blockIdx.x % P.heads;
  if (!locate<KIND>(P, blockIdx.x / P.heads, h, at)) return;
  const int tid = threadIdx.x, r = tid >> 3, seg = tid & 7;
  const bool in = r >= at.lo && r < at.hi;
  u32x4 k[2] = {}, v[2] = {};
  if (at.blk) {
    const uint8_t *src = at.blk + (KIND == 8 ? kKv8Half : kKv16Half);
#pragma unroll
    for (int x = 0; x < E; ++x) {
      const int unit = tid + 256 * x, lane = unit & 63, gg = lane >> 4, m = lane & 15;
      const u32x4 y = *(const u32x4 *)(src + unit * 16);
      if (KIND == 8) {
        *(u32x2 *)&sv[channel_at<E>(32 * (unit >> 6) + m) + 8 * gg] = (u32x2){y[0], y[1]};
        *(u32x2 *)&sv[channel_at<E>(32 * (unit >> 6) + 16 + m) + 8 * gg] = (u32x2){y[2], y[3]};
      } else {
        *(u32x2 *)&sv[channel_at<E>(16 * (unit >> 6) + m) + 16 * gg] = (u32x2){y[0], y[1]};
        *(u32x2 *)&sv[channel_at<E>(16 * (unit >> 6) + m) + 16 * gg + 8] = (u32x2){y[2], y[3]};
      }
    }
    const int tile = r >> 4, key = r & 15, half = seg >> 2, g = seg & 3;
    const int pos = 8 * group_of(r) + slot_of(r);
    if (KIND == 8) {
      const u32x4 z = *(const u32x4 *)(at.blk + ((tile * 2 + half) * 64 + g * 16 + key) * 16);
      const float ks = *(const float *)(at.blk + kKv8Scale + 4 * r);
      const float vs = *(const float *)(at.blk + kKv8Scale + 4 * kBlock + 4 * r);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        k[i >> 2][i & 3] = two_codes(z[i >> 1], 2 * (i & 1), ks);
        const float a = (float)(int8_t)sv[channel_at<E>(16 * seg + 2 * i) + pos] * vs;
        const float b = (float)(int8_t)sv[channel_at<E>(16 * seg + 2 * i + 1) + pos] * vs;
        v[i >> 2][i & 3] = pack_bf16(a, b);
      }
    } else {
#pragma unroll
      for (int p = 0; p < 2; ++p)
        k[p] = *(const u32x4 *)(at.blk + ((tile * 4 + half * 2 + p) * 64 + g * 16 + key) * 16);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i >> 2][i & 3] = (uint32_t)*(const uint16_t *)&sv[channel_at<E>(16 * seg + 2 * i) + 2 * pos] |
                           (uint32_t)*(const uint16_t *)&sv[channel_at<E>(16 * seg + 2 * i + 1) + 2 * pos] << 16;
    }
  }
  if (!in) return;
  const size_t off = ((size_t)(at.token0 + r) * P.heads + h) * kD + 16 * seg;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *(u32x4_a4 *)(P.k + off + 8 * i) = k[i];
    *(u32x4_a4 *)(P.v + off + 8 * i) = v[i];
  }
}

dim3 grid_of(const KvArgs &a) { return dim3((uint32_t)(a.T / kBlock + 2 * a.n) * (uint32_t)a.heads); }

}  // namespace

hipError_t launch_kv_write(const KvArgs &a, int kind, hipStream_t st) {
  if (kind == 8) hipLaunchKernelGGL(k_kv_write<8>, grid_of(a), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_kv_write<16>, grid_of(a), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvArgs &a, int kind, hipStream_t st) {
  if (kind == 8) hipLaunchKernelGGL(k_kv_read<8>, grid_of(a), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_kv_read<16>, grid_of(a), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_kv_write_rotary(const RotaryWriteArgs &a, int kind, hipStream_t st) {
  const dim3 grid((uint32_t)(a.kv.T / kBlock + 2 * a.kv.n) * (uint32_t)(a.kv_parts + a.query_parts));
  if (kind == 8) hipLaunchKernelGGL(k_kv_write_rotary<8>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_kv_write_rotary<16>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace qdr
