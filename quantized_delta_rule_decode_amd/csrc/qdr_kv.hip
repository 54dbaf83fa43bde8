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
#include "qdr_mfma.h"
#include "qdr_mixer.h"
#include "qdr_paged.h"

namespace qdr {

namespace {

constexpr int kD = 128;

// The block a workgroup works on; lo .. hi are its positions that the call has.
struct Where {
  int lo, hi;            // 0 .. 32
  long long token0;      // row of position 0 of the block (rows lo .. hi exist)
  uint8_t *blk;          // NULL: a bad page
};

template <int KIND>
__device__ __forceinline__ bool locate(const KvArgs &P, Where &at) {
  const int h = blockIdx.x % P.heads, place = blockIdx.x / P.heads;
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
  at.token0 = (long long)first + pos - p0;
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

template <int KIND>
__global__ void __launch_bounds__(256) k_kv_write(KvArgs P) {
  constexpr int E = KIND / 8;                       // bytes of an element
  __shared__ __attribute__((aligned(16))) uint8_t sv[kChannels<E>];   // V, channel by channel
  Where at;
  if (!locate<KIND>(P, at) || !at.blk) return;
  const int h = blockIdx.x % P.heads;
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
  uint8_t *dst = at.blk + (KIND == 8 ? kKv8Half : kKv16Half);
#pragma unroll
  for (int x = 0; x < E; ++x) {                     // 256 E units of 16 B
    const int unit = tid + 256 * x, lane = unit & 63, gg = lane >> 4, m = lane & 15;
    // the tokens of lane group gg: 4 gg + {0..3, 16..19}
    const bool whole = at.lo <= 4 * gg && at.hi >= 20 + 4 * gg;
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
          if (t < at.lo || t >= at.hi) continue;
          if (KIND == 8) to[e] = src[e];
          else ((uint16_t *)to)[e] = ((const uint16_t *)src)[e];
        }
      }
    }
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
  if (!locate<KIND>(P, at)) return;
  const int h = blockIdx.x % P.heads;
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

}  // namespace qdr
