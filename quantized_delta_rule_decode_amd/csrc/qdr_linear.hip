// qdr_linear.hip -- one token of linear attention with a decay per head, in
// place in an uncompressed pool:  S = a S + k v^T,  o = S^T q.
// 64 KiB read and written a (request, head) against 5 operations an element:
// bandwidth.  A workgroup takes 64 columns; a thread holds 32 rows of one
// column as eight 16-byte granules (an uncompressed block keeps four rows of
// a column together), so each wave instruction moves 1 KiB of consecutive
// bytes, all loads of a workgroup are issued before the first use, and only
// the four row groups' parts of o meet in LDS.  256 requests of 48 heads: 262 us
// for 1.62 GB, 6.2 TB/s in place (a copy between two buffers reaches 4.8 here);
// one request of 32 heads: 3.4 us, a launch.  Past the caches, since no state
// is read again in the same step.
#include "qdr_mfma.h"
#include "qdr_mixer.h"

namespace qdr {

namespace {

template <bool BF16>
__device__ __forceinline__ float in(const void *x, size_t i) {
  return BF16 ? __uint_as_float((uint32_t)((const uint16_t *)x)[i] << 16) : ((const float *)x)[i];
}

template <bool BF16>
__device__ __forceinline__ void out(void *x, size_t i, float y) {
  if (BF16) ((uint16_t *)x)[i] = (uint16_t)pack_bf16(y, 0.0f);
  else ((float *)x)[i] = y;
}

template <bool BF16>
__global__ void __launch_bounds__(256) k_linear_step(LinearArgs P) {
  __shared__ f32x4 kq[2][32];
  __shared__ float part[3][64];
  const int tid = threadIdx.x, col = 64 * (blockIdx.x & 1) + (tid & 63);
  const int rg = __builtin_amdgcn_readfirstlane(tid >> 6);
  const size_t bh = blockIdx.x >> 1;
  const int b = (int)(bh / P.H), h = (int)(bh % P.H);
  const int slot = P.slots[b];
  if (slot < 0 || slot >= P.num_slots) {
    if (slot != -1 && tid == 0) atomicOr(P.err, kErrSlot);
    if (rg == 0) out<BF16>(P.o, bh * 128 + col, 0.0f);
    return;
  }
  f32x4 *blk = (f32x4 *)(P.pool + (size_t)slot * P.slot_stride + (size_t)h * 65536) + rg * 8 * 128 + col;
  f32x4 S[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) S[i] = __builtin_nontemporal_load(blk + i * 128);
  const float v = in<BF16>(P.v, bh * 128 + col), a = P.gate[bh];
  ((float *)kq)[tid] = tid < 128 ? in<BF16>(P.k, bh * 128 + tid) : in<BF16>(P.q, bh * 128 + tid - 128);
  __syncthreads();
  float o = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const f32x4 k = kq[0][8 * rg + i], q = kq[1][8 * rg + i];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      S[i][r] = __builtin_fmaf(k[r], v, a * S[i][r]);
      o = __builtin_fmaf(q[r], S[i][r], o);
    }
    __builtin_nontemporal_store(S[i], blk + i * 128);
  }
  if (rg) part[rg - 1][tid & 63] = o;
  __syncthreads();
  if (rg == 0) out<BF16>(P.o, bh * 128 + col, ((o + part[0][tid]) + part[1][tid]) + part[2][tid]);
}

}  // namespace

hipError_t launch_linear_step(const LinearArgs &a, bool bf16, hipStream_t st) {
  const dim3 grid((uint32_t)a.B * (uint32_t)a.H * 2u);
  if (bf16) hipLaunchKernelGGL(k_linear_step<true>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(k_linear_step<false>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace qdr
