// qdr_pages.hip -- pages of the paged cache: copied, dealt out for the next
// step, and moved together; slots of a pool copied.
#include "qdr_cache.h"
#include "qdr_mfma.h"
#include "qdr_paged.h"

namespace qdr {

namespace {

constexpr uint64_t kPiece = 32768;   // bytes of a workgroup's pass
// Up to so many workgroups of rows count the pages before their own by
// themselves; more have a launch for it.  Measured per call (us, counted / with
// the launch), rows going on by a token and rows forked in eights: 64 rows of one
// workgroup 9.9 / 12.3 and 12.0 / 14.3, 256 10.6 / 13.4 and 13.2 / 15.5, 512 14.2 /
// 14.2 and 18.8 / 17.0; 128 rows of four workgroups 11.8 / 12.1 and 17.0 / 15.3.
constexpr int kCountedGroups = 256;
// And so many tiles of pages that each workgroup of a compaction counts: 1000
// pages 8.7 / 10.0, 4000 (two tiles) 13.9 / 14.6, 8000 20.0 / 19.3.
constexpr int kCountedTiles = 2;

// `bytes` (a multiple of 16) from one place to another: pieces part, part +
// parts ... of 32 KiB, eight loads of 16 B a thread on their way at once.  What
// is written goes past the caches (a page is larger than what they would keep of
// it, and the lines it would push out are the sources of the other pieces), and
// with ONCE what is read, too.  Measured per call over changing pages (us: plain,
// loads past the caches, stores, both): 1200 pages of 128 KiB copied 69.6, 65.6,
// 64.7, 63.0; 40 slots of 3 MiB 59.2, 54.2, 52.0, 49.7; 760 pages moved together 52.9,
// 47.0, 46.9, 45.1; 256 samples forked from 32 requests, whose last pages are read up
// to sixteen times, 27.1, 31.6, 24.2, 27.1.  Copies take both, for pairs that each have
// a source of their own; where sources repeat, which their callers may ask for, that
// costs: 16 states of 3 MiB to 128 slots 92, 140, 91, 143, 4 to 40 29, 35, 31, 38.
template <bool ONCE>
__device__ __forceinline__ void copy_bytes(const uint8_t *from, uint8_t *to, uint64_t bytes, int part, int parts) {
  for (uint64_t at = (uint64_t)part * kPiece; at < bytes; at += (uint64_t)parts * kPiece) {
    const uint64_t end = min(at + kPiece, bytes);
    u32x4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t b = at + (threadIdx.x + 256 * i) * 16;
      if (b < end) x[i] = ONCE ? __builtin_nontemporal_load((const u32x4 *)(from + b)) : *(const u32x4 *)(from + b);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t b = at + (threadIdx.x + 256 * i) * 16;
      if (b < end) __builtin_nontemporal_store(x[i], (u32x4 *)(to + b));
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
  if (from != to) copy_bytes<true>(from, to, A.bytes, part, A.parts);
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

// The eight pages of a thread of a tile, as bits: which are free.  (All eight
// loads at once; behind the last page it is read again.)
__device__ __forceinline__ uint32_t free_bits(const int32_t *refs, int num_pages, int tile, int32_t (&x)[8]) {
  const int64_t p0 = (int64_t)tile * kBookTile + 8 * threadIdx.x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = refs[min(p0 + i, (int64_t)num_pages - 1)];
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) bits |= x[i] == 0 && p0 + i < num_pages ? 1u << i : 0;
  return bits;
}

// Free pages of a tile, and the counts that the next launch changes.
__global__ void __launch_bounds__(256) k_book(const int32_t *refs, int num_pages, int32_t *counts, int32_t *hold, int32_t *new_refs, int32_t *first) {
  __shared__ int lds[4];
  const int tile = blockIdx.x;
  const int64_t p0 = (int64_t)tile * kBookTile + threadIdx.x;
  int32_t x[8];
  int free = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = refs[min(p0 + 256 * i, (int64_t)num_pages - 1)];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t p = p0 + 256 * i;
    if (p >= num_pages) break;
    free += x[i] == 0;
    if (!hold) continue;
    hold[p] = x[i];
    new_refs[p] = x[i];
    first[p] = INT32_MAX;
  }
  free = sum_all(free, lds);
  if (threadIdx.x == 0) counts[tile] = free;
}

// Free pages before a tile.
__device__ __forceinline__ int free_before(const int32_t *counts, int tile, int *lds) {
  int x = 0;
  for (int i = threadIdx.x; i < tile; i += 256) x += counts[i];
  return sum_all(x, lds);
}

// ---- the next step's tables
// Launches, each of which needs all of the one before: counts and free pages of
// tiles of pages (k_book); who holds which page, by atomics whose order does not
// matter, and the free pages in order (k_assign_hold); where each row's free pages
// begin, and entries and copies (k_assign_rows, k_assign_fill).  Bound by their
// latency, 3 to 4 us each: a step of 64 requests of up to 4000 tokens 13 us; by the
// copies where many rows fork: 256 from 32 requests 23.5 us for 38 MB.

// What row j of the new tables keeps.
struct Row {
  bool live;
  int parent;         // -1: none
  int kept, after;    // tokens
  int full, part;     // kept pages that are full, tokens of the one behind them
  int most;           // pages
};

__device__ __forceinline__ Row shape_of(const KvArgs &P, int after, int kept) {
  Row r;
  r.after = after;
  r.kept = kept;
  r.full = kept >> P.page_shift;
  r.part = kept & ((1 << P.page_shift) - 1);
  r.most = (int)(((long long)after + (1 << P.page_shift) - 1) >> P.page_shift);
  return r;
}

__device__ __forceinline__ Row row_of(const AssignArgs &A, int j) {
  const KvArgs &P = A.kv;
  Row r;
  r.parent = A.parent[j];
  r.live = r.parent >= -1 && r.parent < P.n;
  const int room = room_of(P);
  const int have = r.live && r.parent >= 0 ? P.context[r.parent] : 0;
  const long long after = (long long)have + A.add[j];
  r.live = r.live && have >= 0 && have <= room && after >= 0 && after <= room;
  const Row s = shape_of(P, r.live ? (int)after : 0, r.live ? min(have, (int)after) : 0);
  r.after = s.after;
  r.kept = s.kept;
  r.full = s.full;
  r.part = s.part;
  r.most = s.most;
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
    int32_t refs[8];
    uint32_t bits = free_bits(A.refs, P.num_pages, tile, refs);
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
  const int ctx = old ? P.context[row] : 0;
  const bool bad = ctx < 0 || ctx > room_of(P);
  const bool had = inside && old && !bad && i < (int)(((long long)ctx + (1 << P.page_shift) - 1) >> P.page_shift);
  const bool keeps = inside && made && (i < r.full || (i == r.full && r.part));
  const int before = had ? P.pages[(size_t)row * P.max_pages + i] : 0;
  const int after = keeps ? P.pages[(size_t)r.parent * P.max_pages + i] : 0;
  if ((bad && i == 0) || (made && !r.live && i == 0)) atomicOr(P.err, kErrLength);
  if (!is_page(P, before) || !is_page(P, after)) atomicOr(P.err, kErrPage);
  if (had && i >= same && is_page(P, before)) {
    atomicSub(&A.hold[before], 1);
    atomicSub(&A.new_refs[before], 1);
  }
  if (!made || !inside) return;
  int32_t *to = A.new_pages + (size_t)row * P.max_pages + i;
  if (i < r.full) {
    if (i >= same && is_page(P, after)) {
      atomicAdd(&A.hold[after], 1);
      atomicAdd(&A.new_refs[after], 1);
    }
    *to = is_page(P, after) ? after : -1;
  } else if (i >= r.most) {
    *to = -1;
  } else if (keeps && is_page(P, after)) {
    atomicMin(&A.first[after], row);
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

// Where each row's free pages begin, by one workgroup, and what else its
// workgroups of the next launch would have to look up one after the other.
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
    Row r{};
    int last = -1;
    bool stays = false;
    if (j < A.m) {
      r = row_of(A, j);
      last = last_page(A, r, j, &stays);
      need = r.most - r.full - (stays ? 1 : 0);
    }
    long long before;
    const long long all = sum_of(need, &before);
    const long long at = base + before;
    if (j < A.m) {
      const bool fits = need == 0 || at + need <= free;
      if (!fits) atomicOr(A.kv.err, kErrFull);
      int4 *job = (int4 *)A.offset + 2 * (size_t)j;
      job[0] = make_int4(!fits ? -1 : need == 0 ? 0 : (int)at, r.after, r.kept, last);
      job[1].x = stays;
    }
    base += all;
  }
}

// A row's new pages and the copy of its last one's tokens: workgroup 0 of a row
// writes its entries, all copy.  COUNT: each workgroup finds by itself where its
// row's free pages begin.
template <bool COUNT>
__global__ void __launch_bounds__(256) k_assign_fill(AssignArgs A, int tiles) {
  const KvArgs &P = A.kv;
  __shared__ Row own;
  __shared__ int own_last, own_stays;
  __shared__ long long sums[2][4];
  const int j = blockIdx.x / A.parts, part = blockIdx.x % A.parts, tid = threadIdx.x;
  Row r;
  bool stays;
  int last, offset;
  if (COUNT) {
    long long before = 0, free = 0;
    for (int i = tid; i < tiles; i += 256) free += A.counts[i];
    for (int i = tid; i <= j; i += 256) {   // its own among them: one chain of loads for all
      r = row_of(A, i);
      last = last_page(A, r, i, &stays);
      if (i < j) {
        before += r.most - r.full - (stays ? 1 : 0);
      } else {
        own = r;
        own_last = last;
        own_stays = stays;
      }
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      before += __shfl_xor(before, d);
      free += __shfl_xor(free, d);
    }
    if ((tid & 63) == 0) {
      sums[0][tid >> 6] = before;
      sums[1][tid >> 6] = free;
    }
    __syncthreads();
    before = sums[0][0] + sums[0][1] + sums[0][2] + sums[0][3];
    free = sums[1][0] + sums[1][1] + sums[1][2] + sums[1][3];
    r = own;
    last = own_last;
    stays = own_stays;
    const int need = r.most - r.full - (stays ? 1 : 0);
    offset = need == 0 ? 0 : before + need <= free ? (int)before : -1;
    if (offset < 0 && part == 0 && tid == 0) atomicOr(P.err, kErrFull);
  } else {
    const int4 *job = (const int4 *)A.offset + 2 * (size_t)j;
    const int4 x = job[0];
    offset = x.x;
    last = x.w;
    stays = job[1].x;
    r = shape_of(P, x.y, x.z);
  }
  int32_t *row = A.new_pages + (size_t)j * P.max_pages;
  if (offset < 0) {   // too few free pages: an empty row
    if (part) return;
#pragma unroll 1
    for (int i = threadIdx.x; i < r.full; i += 256) {
      const int page = row[i];
      if (page >= 0) atomicSub(&A.new_refs[page], 1);
      row[i] = -1;
    }
#pragma unroll 1
    for (int i = r.full + threadIdx.x; i < r.most; i += 256) row[i] = -1;
    if (threadIdx.x == 0) A.new_context[j] = 0;
    return;
  }
  if (part == 0) {
    const int begin = r.full + (stays ? 1 : 0);
#pragma unroll 1
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
#pragma unroll 1
  for (uint64_t u = part; u < pieces * P.heads; u += A.parts) {
    const uint64_t at = u / pieces * step, piece = u % pieces * kPiece;
    copy_bytes<false>(from + at + piece, to + at + piece, min(kPiece, bytes - piece), 0, 1);
  }
}

// ---- pages moved together
// Two launches (three beyond kCountedTiles): lists, 6 us, then moves, bound by
// memory: 760 pages of 128 KiB 42.7 us a call, 199 MB, 4.7 TB/s.

// Pages that stay, and the list of moves: as many pages are used from `live` on
// (the number of used ones) as are free below it, and the k-th goes to the k-th.
// A used page's place in the list is the number of used ones before it, a free
// page's that of free ones.  COUNT: each workgroup counts all tiles by itself.
template <bool COUNT>
__global__ void __launch_bounds__(256) k_compact_list(CompactArgs A, int tiles) {
  __shared__ int lds[4];
  const int tile = blockIdx.x, tid = threadIdx.x;
  const int64_t p0 = (int64_t)tile * kBookTile + 8 * tid;
  int32_t refs[8];
  const uint32_t bits = free_bits(A.refs, A.num_pages, tile, refs);
  int before = 0, after = 0;
  if (COUNT) {
    for (int i = 0; i < tiles; ++i) {
      int32_t unused[8];
      const int free = __popc(i == tile ? bits : free_bits(A.refs, A.num_pages, i, unused));
      before += i < tile ? free : 0;
      after += i < tile ? 0 : free;
    }
    before = sum_all(before, lds);
  } else {
    before = free_before(A.counts, tile, lds);
    for (int i = tile + tid; i < tiles; i += 256) after += A.counts[i];
  }
  const int free = before + sum_all(after, lds), live = A.num_pages - free;
  int total;
  int rank = before + sum_before(__popc(bits), lds, &total);   // free pages before p0
  if (tile == 0 && tid == 0) {
    A.moves[2] = live;
    if (live == A.num_pages) A.moves[0] = A.moves[1] = 0;
  }
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
      A.dst[p] = is_free ? -1 : (int)p - rank;   // dst has fewer than `live` entries
      if (!is_free) A.src[p - rank] = (int)p;
    } else if (is_free) {
      A.dst[rank] = (int)p;
    } else {
      A.moved[p] = (int)p;
      A.new_refs[p] = refs[i];
    }
    rank += is_free;
  }
}

// The moves, by the first workgroups, and the tables, which need no move's end.
__global__ void __launch_bounds__(256) k_compact_move(CompactArgs A) {
  if ((int)blockIdx.x >= A.groups) {
    const int64_t i = (int64_t)(blockIdx.x - A.groups) * 256 + threadIdx.x;
    if (i >= A.entries) return;
    int page = A.pages[i];
    if (page < 0 || page >= A.num_pages || A.refs[page] == 0) {
      page = -1;
    } else if (page >= A.moves[2]) {
      page = A.dst[A.dst[page] - A.moves[1]];
    }
    A.new_pages[i] = page;
    return;
  }
  const int64_t moves = A.moves[0];
#pragma unroll 1
  for (int64_t x = blockIdx.x; x < moves * A.parts; x += A.groups) {
    const int k = (int)(x / A.parts), part = (int)(x % A.parts);
    const int s = A.src[A.moves[1] + k], d = A.dst[k];
    if (part == 0 && threadIdx.x == 0) {
      A.moved[s] = d;
      A.new_refs[d] = A.refs[s];
    }
    copy_bytes<false>(A.base + (uint64_t)s * A.page_bytes, A.base + (uint64_t)d * A.page_bytes, A.page_bytes, part, A.parts);
  }
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
  if ((int64_t)a.m * a.parts > kCountedGroups) {
    hipLaunchKernelGGL(k_assign_rows, dim3(1), dim3(1024), 0, st, a, tiles);
    hipLaunchKernelGGL(k_assign_fill<false>, dim3((uint32_t)a.m * (uint32_t)a.parts), dim3(256), 0, st, a, tiles);
  } else if (a.m > 0) {
    hipLaunchKernelGGL(k_assign_fill<true>, dim3((uint32_t)a.m * (uint32_t)a.parts), dim3(256), 0, st, a, tiles);
  }
  return hipGetLastError();
}

hipError_t launch_compact(const CompactArgs &a, hipStream_t st) {
  const int tiles = (int)book_tiles(a.num_pages);
  if (tiles <= kCountedTiles) {
    hipLaunchKernelGGL(k_compact_list<true>, dim3(tiles), dim3(256), 0, st, a, tiles);
  } else {
    hipLaunchKernelGGL(k_book, dim3(tiles), dim3(256), 0, st, a.refs, a.num_pages, a.counts, nullptr, nullptr, nullptr);
    hipLaunchKernelGGL(k_compact_list<false>, dim3(tiles), dim3(256), 0, st, a, tiles);
  }
  hipLaunchKernelGGL(k_compact_move, dim3((uint32_t)a.groups + (uint32_t)((a.entries + 255) / 256)), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace qdr
