// qdr_pages.hip -- pages of the paged cache: copied, dealt out for the next
// step, and moved together; slots of a pool copied.
#include "qdr_cache.h"
#include "qdr_mfma.h"
#include "qdr_paged.h"

namespace qdr {

namespace {

constexpr uint64_t kPiece = 32768;   // bytes of a workgroup's pass

// `bytes` (a multiple of 16) from one place to another: pieces part, part +
// parts ... of 32 KiB, eight loads of 16 B a thread on their way at once.
__device__ __forceinline__ void copy_bytes(const uint8_t *from, uint8_t *to, uint64_t bytes, int part, int parts) {
  for (uint64_t at = (uint64_t)part * kPiece; at < bytes; at += (uint64_t)parts * kPiece) {
    const uint64_t end = min(at + kPiece, bytes);
    u32x4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t b = at + (threadIdx.x + 256 * i) * 16;
      if (b < end) x[i] = *(const u32x4 *)(from + b);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t b = at + (threadIdx.x + 256 * i) * 16;
      if (b < end) *(u32x4 *)(to + b) = x[i];
    }
  }
}

__global__ void __launch_bounds__(256) k_copy(CopyArgs A) {
  const int i = blockIdx.x / A.parts, part = blockIdx.x % A.parts;
  const int s = A.src[i], d = A.dst[i];
  if (part == 0 && threadIdx.x == 0) {
    if (s < -1 || s >= A.num_from) atomicOr(A.err_from, A.bit);
    if (d < -1 || d >= A.num_to) atomicOr(A.err_to, A.bit);
  }
  if (s < 0 || s >= A.num_from || d < 0 || d >= A.num_to) return;
  const uint8_t *from = A.from + (uint64_t)s * A.bytes;
  uint8_t *to = A.to + (uint64_t)d * A.bytes;
  if (from != to) copy_bytes(from, to, A.bytes, part, A.parts);
}

// Sum over the workgroup of 256; every thread gets it.
__device__ __forceinline__ int sum_all(int x, int *lds) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  return lds[0] + lds[1] + lds[2] + lds[3];
}
// Sum over the threads before this one, of 256; *total: over all.
__device__ __forceinline__ int sum_before(int x, int *lds, int *total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int s = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(s, d);
    if (lane >= d) s += y;
  }
  __syncthreads();
  if (lane == 63) lds[w] = s;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < 4; ++i) before += i < w ? lds[i] : 0;
  *total = lds[0] + lds[1] + lds[2] + lds[3];
  return before + s - x;
}

// The eight pages of a thread of a tile, as bits: which are free.
__device__ __forceinline__ uint32_t free_bits(const int32_t *refs, int num_pages, int tile) {
  const int64_t p0 = (int64_t)tile * kBookTile + 8 * threadIdx.x;
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (p0 + i < num_pages && refs[p0 + i] == 0) bits |= 1u << i;
  return bits;
}

// Free pages of a tile, and the counts that the next launch changes.
__global__ void __launch_bounds__(256) k_book(const int32_t *refs, int num_pages, int32_t *counts, int32_t *hold, int32_t *new_refs, int32_t *first) {
  __shared__ int lds[4];
  const int tile = blockIdx.x;
  const int total = sum_all(__popc(free_bits(refs, num_pages, tile)), lds);
  if (threadIdx.x == 0) counts[tile] = total;
  if (!hold) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t p = (int64_t)tile * kBookTile + 256 * i + threadIdx.x;
    if (p >= num_pages) break;
    const int32_t x = refs[p];
    hold[p] = x;
    new_refs[p] = x;
    first[p] = INT32_MAX;
  }
}

// Free pages before a tile.
__device__ __forceinline__ int free_before(const int32_t *counts, int tile, int *lds) {
  int x = 0;
  for (int i = threadIdx.x; i < tile; i += 256) x += counts[i];
  return sum_all(x, lds);
}

// ---- the next step's tables

// What row j of the new tables keeps.
struct Row {
  bool live;
  int parent;         // -1: none
  int kept, after;    // tokens
  int full, part;     // kept pages that are full, tokens of the one behind them
  int most;           // pages
};

__device__ __forceinline__ Row row_of(const AssignArgs &A, int j) {
  const KvArgs &P = A.kv;
  Row r;
  r.parent = A.parent[j];
  r.live = r.parent >= -1 && r.parent < P.n;
  const int room = room_of(P);
  const int have = r.live && r.parent >= 0 ? P.context[r.parent] : 0;
  const long long after = (long long)have + A.add[j];
  r.live = r.live && have >= 0 && have <= room && after >= 0 && after <= room;
  r.after = r.live ? (int)after : 0;
  r.kept = r.live ? min(have, r.after) : 0;
  r.full = r.kept >> P.page_shift;
  r.part = r.kept & ((1 << P.page_shift) - 1);
  r.most = (int)(((long long)r.after + (1 << P.page_shift) - 1) >> P.page_shift);
  return r;
}

__device__ __forceinline__ bool is_page(const KvArgs &P, int page) { return page >= 0 && page < P.num_pages; }

// Who holds which page: workgroups over the entries of old and new rows, then
// over the tiles of pages, which list the free ones.
__global__ void __launch_bounds__(256) k_assign_hold(AssignArgs A, int rows, int chunks) {
  const KvArgs &P = A.kv;
  __shared__ int lds[4];
  const int place = blockIdx.x;
  if (place >= rows * chunks) {
    const int tile = place - rows * chunks;
    const int before = free_before(A.counts, tile, lds);
    uint32_t bits = free_bits(A.refs, P.num_pages, tile);
    int total;
    int at = before + sum_before(__popc(bits), lds, &total);
    while (bits) {
      const int i = __ffs((int)bits) - 1;
      bits &= bits - 1;
      A.free[at++] = tile * kBookTile + 8 * (int)threadIdx.x + i;
    }
    return;
  }
  const int row = place / chunks, i = (place % chunks) * 256 + threadIdx.x;
  const bool inside = i < P.max_pages, old = row < P.n, made = row < A.m;
  Row r{};
  if (made) r = row_of(A, row);
  // a row that goes on holds what it held
  const int same = made && r.live && r.parent == row ? r.full : 0;
  if (old) {
    const int ctx = P.context[row], room = room_of(P);
    if (ctx < 0 || ctx > room) {
      if (i == 0) atomicOr(P.err, kErrLength);
    } else if (inside && i < (int)(((long long)ctx + (1 << P.page_shift) - 1) >> P.page_shift)) {
      const int page = P.pages[(size_t)row * P.max_pages + i];
      if (!is_page(P, page)) {
        atomicOr(P.err, kErrPage);
      } else if (i >= same) {
        atomicSub(&A.hold[page], 1);
        atomicSub(&A.new_refs[page], 1);
      }
    }
  }
  if (!made) return;
  if (!r.live && place % chunks == 0 && threadIdx.x == 0) atomicOr(P.err, kErrLength);
  if (!inside) return;
  int32_t *to = A.new_pages + (size_t)row * P.max_pages + i;
  if (i < r.full) {
    int page = P.pages[(size_t)r.parent * P.max_pages + i];
    if (!is_page(P, page)) {
      atomicOr(P.err, kErrPage);
      page = -1;
    } else if (i >= same) {
      atomicAdd(&A.hold[page], 1);
      atomicAdd(&A.new_refs[page], 1);
    }
    *to = page;
  } else if (i >= r.most) {
    *to = -1;
  } else if (i == r.full && r.part) {
    const int page = P.pages[(size_t)r.parent * P.max_pages + i];
    if (is_page(P, page)) atomicMin(&A.first[page], row);
  }
}

// The page behind a row's full ones, and whether it stays the row's; -1: none.
__device__ __forceinline__ int last_page(const AssignArgs &A, const Row &r, int j, bool *stays) {
  *stays = false;
  if (!r.part) return -1;
  const int page = A.kv.pages[(size_t)r.parent * A.kv.max_pages + r.full];
  if (!is_page(A.kv, page)) return -1;
  *stays = A.hold[page] == 0 && A.first[page] == j;
  return page;
}

// Where each row's free pages begin, by one workgroup.
__global__ void __launch_bounds__(1024) k_assign_rows(AssignArgs A, int tiles) {
  __shared__ long long lds[16];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  auto sum_of = [&](long long x, long long *before) {
    long long s = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long long y = __shfl_up(s, d);
      if (lane >= d) s += y;
    }
    __syncthreads();
    if (lane == 63) lds[w] = s;
    __syncthreads();
    long long b = 0, all = 0;
    for (int i = 0; i < 16; ++i) {
      b += i < w ? lds[i] : 0;
      all += lds[i];
    }
    *before = b + s - x;
    return all;
  };
  long long free = 0, unused;
  for (int i = tid; i < tiles; i += 1024) free += A.counts[i];
  free = sum_of(free, &unused);
  long long base = 0;
  for (int j0 = 0; j0 < A.m; j0 += 1024) {
    const int j = j0 + tid;
    int need = 0;
    if (j < A.m) {
      const Row r = row_of(A, j);
      bool stays;
      last_page(A, r, j, &stays);
      need = r.most - r.full - (stays ? 1 : 0);
    }
    long long before;
    const long long all = sum_of(need, &before);
    const long long at = base + before;
    if (j < A.m) {
      const bool fits = need == 0 || at + need <= free;
      if (!fits) atomicOr(A.kv.err, kErrFull);
      A.offset[j] = !fits ? -1 : need == 0 ? 0 : (int)at;
    }
    base += all;
  }
}

// A row's new pages and the copy of its last one's tokens: workgroup 0 of a row
// writes its entries, all copy.
__global__ void __launch_bounds__(256) k_assign_fill(AssignArgs A) {
  const KvArgs &P = A.kv;
  const int j = blockIdx.x / A.parts, part = blockIdx.x % A.parts;
  const Row r = row_of(A, j);
  const int offset = A.offset[j];
  bool stays;
  const int last = last_page(A, r, j, &stays);
  int32_t *row = A.new_pages + (size_t)j * P.max_pages;
  if (offset < 0) {   // too few free pages: an empty row
    if (part) return;
    for (int i = threadIdx.x; i < r.full; i += 256) {
      const int page = row[i];
      if (page >= 0) atomicSub(&A.new_refs[page], 1);
      row[i] = -1;
    }
    for (int i = r.full + threadIdx.x; i < r.most; i += 256) row[i] = -1;
    if (threadIdx.x == 0) A.new_context[j] = 0;
    return;
  }
  if (part == 0) {
    const int begin = r.full + (stays ? 1 : 0);
    for (int i = r.full + threadIdx.x; i < r.most; i += 256) {
      const int page = i < begin ? last : A.free[offset + i - begin];
      row[i] = page;
      A.new_refs[page] = 1;
    }
    if (threadIdx.x == 0) A.new_context[j] = r.after;
  }
  if (last < 0 || stays) return;
  const uint64_t block = A.kind == 8 ? kKv8Block : kKv16Block;
  const uint64_t bytes = (uint64_t)((r.part + kBlock - 1) / kBlock) * block, step = block << (P.page_shift - 5);
  const uint8_t *from = P.base + (uint64_t)last * P.heads * step;
  uint8_t *to = P.base + (uint64_t)A.free[offset] * P.heads * step;
  const uint64_t pieces = (bytes + kPiece - 1) / kPiece;
  for (uint64_t u = part; u < pieces * P.heads; u += A.parts) {
    const uint64_t at = u / pieces * step, piece = u % pieces * kPiece;
    copy_bytes(from + at + piece, to + at + piece, min(kPiece, bytes - piece), 0, 1);
  }
}

// ---- pages moved together

// Pages that stay, and the list of moves.
__global__ void __launch_bounds__(256) k_compact_list(CompactArgs A, int tiles) {
  __shared__ int lds[4];
  const int tile = blockIdx.x, tid = threadIdx.x;
  int before = free_before(A.counts, tile, lds);
  int after = 0;
  for (int i = tile + tid; i < tiles; i += 256) after += A.counts[i];
  const int free = before + sum_all(after, lds), live = A.num_pages - free;
  const int64_t p0 = (int64_t)tile * kBookTile + 8 * tid;
  const uint32_t bits = free_bits(A.refs, A.num_pages, tile);
  int total;
  int rank = before + sum_before(__popc(bits), lds, &total);   // free pages before p0
  // as many pages are used from `live` on as are free below it, and the k-th goes
  // to the k-th: src by the number of used pages before, dst of free ones
  if (live == A.num_pages && tile == 0 && tid == 0) A.moves[0] = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t p = p0 + i;
    if (p >= A.num_pages) break;
    const bool is_free = (bits >> i) & 1;
    if (p == live) {
      A.moves[0] = rank;
      A.moves[1] = live - rank;   // used pages below `live`
    }
    if (is_free) A.moved[p] = -1;
    if (p >= live) {
      A.new_refs[p] = 0;
      if (!is_free) A.src[p - rank] = (int)p;
    } else if (is_free) {
      A.dst[rank] = (int)p;
    } else {
      A.moved[p] = (int)p;
      A.new_refs[p] = A.refs[p];
    }
    rank += is_free;
  }
}

__global__ void __launch_bounds__(256) k_compact_move(CompactArgs A) {
  const int64_t moves = A.moves[0];
  for (int64_t x = blockIdx.x; x < moves * A.parts; x += gridDim.x) {
    const int k = (int)(x / A.parts), part = (int)(x % A.parts);
    const int s = A.src[A.moves[1] + k], d = A.dst[k];
    if (part == 0 && threadIdx.x == 0) {
      A.moved[s] = d;
      A.new_refs[d] = A.refs[s];
    }
    copy_bytes(A.base + (uint64_t)s * A.page_bytes, A.base + (uint64_t)d * A.page_bytes, A.page_bytes, part, A.parts);
  }
}

__global__ void __launch_bounds__(256) k_compact_tables(CompactArgs A) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= A.entries) return;
  const int page = A.pages[i];
  A.new_pages[i] = page >= 0 && page < A.num_pages ? A.moved[page] : -1;
}

}  // namespace

hipError_t launch_copy(const CopyArgs &a, hipStream_t st) {
  hipLaunchKernelGGL(k_copy, dim3((uint32_t)a.m * (uint32_t)a.parts), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_assign(const AssignArgs &a, hipStream_t st) {
  const int tiles = (int)book_tiles(a.kv.num_pages), rows = a.m > a.kv.n ? a.m : a.kv.n, chunks = (a.kv.max_pages + 255) / 256 + (a.kv.max_pages == 0);
  hipLaunchKernelGGL(k_book, dim3(tiles), dim3(256), 0, st, a.refs, a.kv.num_pages, a.counts, a.hold, a.new_refs, a.first);
  hipLaunchKernelGGL(k_assign_hold, dim3((uint32_t)rows * (uint32_t)chunks + (uint32_t)tiles), dim3(256), 0, st, a, rows, chunks);
  if (a.m > 0) {
    hipLaunchKernelGGL(k_assign_rows, dim3(1), dim3(1024), 0, st, a, tiles);
    hipLaunchKernelGGL(k_assign_fill, dim3((uint32_t)a.m * (uint32_t)a.parts), dim3(256), 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_compact(const CompactArgs &a, hipStream_t st) {
  const int tiles = (int)book_tiles(a.num_pages);
  hipLaunchKernelGGL(k_book, dim3(tiles), dim3(256), 0, st, a.refs, a.num_pages, a.counts, nullptr, nullptr, nullptr);
  hipLaunchKernelGGL(k_compact_list, dim3(tiles), dim3(256), 0, st, a, tiles);
  hipLaunchKernelGGL(k_compact_move, dim3(a.groups), dim3(256), 0, st, a);
  if (a.entries > 0) hipLaunchKernelGGL(k_compact_tables, dim3((uint32_t)((a.entries + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace qdr
