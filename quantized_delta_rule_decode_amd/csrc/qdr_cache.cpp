// qdr_cache.cpp -- host side of what is done around the paged cache
// (include/qdr_cache.h): argument checks, the rotation's handle, workspaces,
// and the launches.
#include "../../include/qdr_cache.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "qdr_cache.h"
#include "qdr_calls.h"
#include "qdr_host.h"

using namespace qdr::calls;

struct qdr_rotary {
  int device = 0;
  int32_t channels = 0, layout = 0;
  float amplitude = 1.0f;
  uint64_t *turns = nullptr;
};

namespace {

constexpr double kPi = 3.14159265358979323846;

size_t up(size_t x) { return (x + 255) / 256 * 256; }

qdr_status check_channels(int32_t channels) {
  if (channels < 16 || channels > QDR_DIM || channels % 16)
    return fail(QDR_E_INVAL, "channels must be a multiple of 16 from 16 to %d (got %d)", QDR_DIM, channels);
  return QDR_OK;
}

// Turns a token, modulo one turn, in units of 2^-64.
uint64_t turns_of(double freq) {
  long double t = (long double)freq / 6.28318530717958647692528676655900577L;
  t -= std::floor(t);                                   // [0, 1]
  t = std::ldexp(t, 63);                                // (2^64 itself would not fit)
  const uint64_t whole = (uint64_t)t;
  return 2 * whole + (uint64_t)(2 * (t - (long double)whole) + 0.5L);
}

qdr::RotaryView view_of(const qdr_rotary *r) { return {r->turns, r->channels, r->layout, r->amplitude}; }

constexpr int64_t kMostStride = (int64_t)1 << 30;
qdr_status check_stride(const char *name, int64_t stride, int64_t heads, bool bf16) {
  if (stride < heads * QDR_DIM || stride > kMostStride)
    return fail(QDR_E_INVAL, "%s must be from %lld to %lld elements (got %lld)", name, (long long)heads * QDR_DIM, (long long)kMostStride, (long long)stride);
  if (bf16 && stride % 2) return fail(QDR_E_INVAL, "%s must be even (got %lld)", name, (long long)stride);
  return QDR_OK;
}

qdr_status rotate(qdr_rotary *r, const int32_t *positions, int32_t T, int32_t heads, const void *x, int64_t x_stride,
                  void *y, int64_t y_stride, void *stream, bool bf16) {
  if (!r) return fail(QDR_E_INVAL, "rotary is NULL");
  QDR_TRY(check_counts(0, T));
  if (heads <= 0 || heads > kMostHeads) return fail(QDR_E_INVAL, "heads must be from 1 to %d (got %d)", kMostHeads, heads);
  QDR_TRY(check_stride("x_stride", x_stride, heads, bf16));
  QDR_TRY(check_stride("y_stride", y_stride, heads, bf16));
  if (T == 0) return qdr::set_ok();
  if (!positions || !x || !y) return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  if (!aligned4(x) || !aligned4(y)) return fail(QDR_E_INVAL, "tensors must be 4-byte aligned");
  QDR_TRY(check_device(r->device));
  qdr::RotateArgs a{};
  a.rotary = view_of(r);
  a.positions = positions;
  a.T = T;
  a.heads = heads;
  a.x = x;
  a.y = y;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  // about 128 rows a workgroup, the tokens that the table has room for at most
  a.part_heads = std::min(heads, 128);
  a.head_parts = (heads + a.part_heads - 1) / a.part_heads;
  a.tokens = std::max(1, std::min(32, 128 / heads));
  QDR_TRY(check_groups(((int64_t)T + a.tokens - 1) / a.tokens * a.head_parts));
  return launched(qdr::launch_rotate(a, bf16, static_cast<hipStream_t>(stream)));
}

uint64_t page_bytes(const qdr_kv *kv) {
  return (uint64_t)kv->desc.num_heads * (kv->desc.page_tokens / qdr::kBlock) * (kv->desc.kind == QDR_KV_INT8 ? qdr::kKv8Block : qdr::kKv16Block);
}

// Workgroups for one page or slot of so many bytes: 32 KiB each, 64 at most
// where they take several turns.
int32_t parts_of(uint64_t bytes) { return (int32_t)std::min<uint64_t>(64, (bytes + 32767) / 32768); }

qdr_status check_pages(const qdr_kv *kv) {
  if (kv->desc.num_pages > qdr::kMostBookPages)
    return fail(QDR_E_UNSUPPORTED, "page tables are kept for caches of at most %lld pages (got %d)", (long long)qdr::kMostBookPages, kv->desc.num_pages);
  return QDR_OK;
}

struct Span {
  const void *at;
  int64_t entries;
};
bool overlap(const Span &a, const Span &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.entries > 0 && b.entries > 0 && x < y + 4 * (uintptr_t)b.entries && y < x + 4 * (uintptr_t)a.entries;
}
qdr_status check_apart(const Span *in, int ins, const Span *out, int outs) {
  for (int o = 0; o < outs; ++o) {
    for (int i = 0; i < ins; ++i)
      if (overlap(in[i], out[o])) return fail(QDR_E_INVAL, "a new array overlaps an old one");
    for (int p = 0; p < o; ++p)
      if (overlap(out[p], out[o])) return fail(QDR_E_INVAL, "two new arrays overlap");
  }
  return QDR_OK;
}

// Parts of an assignment's workspace, in bytes.
struct AssignSpace {
  size_t pages, counts, rows;   // of [num_pages], [tiles] and [m][8]
  size_t total() const { return 3 * pages + counts + rows; }
};
AssignSpace assign_space(const qdr_kv *kv, int32_t m) {
  return {up((size_t)kv->desc.num_pages * 4), up((size_t)qdr::book_tiles(kv->desc.num_pages) * 4), up((size_t)m * 32)};
}
struct CompactSpace {
  size_t pages, counts, moves;
  size_t total() const { return 2 * pages + counts + moves; }
};
constexpr int kMoveGroups = 2048;   // workgroups of all moves: eight on each compute unit
CompactSpace compact_space(const qdr_kv *kv) {
  return {up((size_t)kv->desc.num_pages * 4), up((size_t)qdr::book_tiles(kv->desc.num_pages) * 4), 256};
}

qdr_status check_heads(const qdr_kv *kv, int32_t q_heads) {
  if (q_heads <= 0 || q_heads % kv->desc.num_heads)
    return fail(QDR_E_INVAL, "q_heads must be a positive multiple of the cache's %d heads (got %d)", kv->desc.num_heads, q_heads);
  return QDR_OK;
}

// The plan of a call, whether its launches can be counted, and its workspace.
qdr_status make_shared(const qdr_kv *kv, int32_t n, int32_t T, int32_t groups, int32_t q_heads, int32_t max_pages, qdr::SharedPlan *plan, size_t *bytes) {
  const int64_t heads = kv->desc.num_heads;
  QDR_TRY(check_groups(q_heads));
  QDR_TRY(check_groups(n));
  QDR_TRY(check_groups(groups));
  QDR_TRY(check_groups((int64_t)n * q_heads));
  *plan = qdr::plan_shared(n, T, groups, q_heads, kv->desc.num_heads, max_pages, kv->page_shift);
  QDR_TRY(check_groups(plan->many_tiles));
  const int64_t few = (int64_t)n * plan->few_parts * plan->few_splits, many = (int64_t)plan->many_tiles * plan->many_parts * plan->many_splits;
  QDR_TRY(check_groups(few));
  QDR_TRY(check_groups(many));
  QDR_TRY(check_groups((few + many + plan->ranges) * heads + 1));
  QDR_TRY(check_groups((int64_t)T * q_heads / 4));   // of the join: four rows a workgroup, the most that it takes
  *bytes = plan->floats * sizeof(float);
  return QDR_OK;
}

}  // namespace

namespace qdr {

SharedPlan plan_shared(int n, int T, int groups, int q_heads, int heads, int max_pages, int page_shift) {
  SharedPlan p{};
  p.group = q_heads / heads;
  p.few_heads = std::min(p.group, kFewRows);
  p.few_tokens = kFewRows / p.few_heads;
  p.few_parts = (p.group + p.few_heads - 1) / p.few_heads;
  p.many_heads = std::min(p.group, kManyRows);
  p.many_tokens = kManyRows / p.many_heads;
  p.many_inverse = 1.0f / p.many_tokens;
  p.many_parts = (p.group + p.many_heads - 1) / p.many_heads;
  // Sequences of more than few_tokens take ceil(len / many_tokens) many-row tiles,
  // from place cu / many_tokens + b on, or + cu / (few_tokens + 1) where that
  // makes fewer places: each finds as many as it needs before the next one's.
  const int64_t by_tokens = T / (p.few_tokens + 1) + 1;
  p.by_tokens = by_tokens < n;
  p.many_tiles = T > p.few_tokens ? (int)(T / p.many_tokens + std::min<int64_t>(by_tokens, n)) : 0;
  // Pieces of sequences' own keys: one workgroup of few rows a compute unit, two of
  // many, of kSharedLeast and kManyLeast blocks at least.  (Simpler than plan_attend,
  // which leaves few rows uncut up to 32 blocks and cuts longer pieces above 64
  // tiles: here they stand beside the line.)
  const int64_t blocks = (int64_t)max_pages << (page_shift - 5), each = ((int64_t)T + n - 1) / n;
  const int64_t few = (int64_t)n * heads * p.few_parts, many = (each + p.many_tokens - 1) / p.many_tokens * n * heads * p.many_parts;
  const auto cut = [&](int64_t units, int64_t places, int64_t least) {
    return (int)std::max<int64_t>(1, std::min<int64_t>({places / std::max<int64_t>(units, 1), (blocks + least - 1) / least, 32}));
  };
  p.few_splits = cut(few, 256, kSharedLeast);
  p.many_splits = p.many_tiles && blocks > 24 ? cut(many, 512, kManyLeast) : 1;
  // Groups' rows go through shared keys together where that can save reading
  // kLeastSaved blocks of a key head: the line and the join of its results cost
  // some 10 us.  What is saved is taken from the tables' width (only the device knows
  // the shared counts) and from n - groups, as if no group were empty and no sequence
  // in none.  Measured per call (us, together / each by itself), one group of 700
  // tokens a sequence, tables as wide as that takes, 8 key heads, 8-bit, then
  // bfloat16; behind 2048: 8 sequences (4760 blocks less) 25.1 / 18.7, 24.6 / 19.4;
  // 8192: 4 (6648) 23.5 / 22.1, 28.5 / 22.9; 8 (15512) 31.1 / 31.5, 35.6 / 30.0; 16384:
  // 2 (4264) 27.8 / 22.7, 38.5 / 23.4; 4 (12792) 28.6 / 30.4, 39.1 / 30.2; 1024: 32
  // (13144) 28.5 / 25.3, 31.9 / 30.9; 4096: 32 (36952) 31.5 / 48.9, 37.1 / 50.6; 2 key
  // heads, 4096: 32 (9238) 27.3 / 22.8, 27.3 / 25.3.  So with bfloat16 it comes somewhat
  // early, and with tables that are wider than need be it takes the first of each pair
  // where the second is the smaller.
  const bool together = groups && (int64_t)std::max(n - groups, 0) * heads * blocks >= kLeastSaved;
  // The line: two workgroups a compute unit, but no more than there can be work for,
  // every row a tile of as many blocks as the tables have.
  const int64_t wide = T > p.few_tokens ? (2 * (T / p.many_tokens) + groups) * (int64_t)p.many_parts : 0;
  p.ranges = !together ? 0 : (int)std::min<int64_t>(std::max(1, 512 / heads), ((int64_t)groups * p.few_parts + wide) * (2 + blocks / 4));
  p.slot_rows = T > p.few_tokens ? kManyRows : kFewRows;
  const size_t rows = (size_t)T * q_heads;
  p.cut = together ? 2 * rows * (QDR_DIM + 2) : 0;
  p.few_pieces = p.cut + (size_t)p.ranges * heads * 2 * p.slot_rows * (QDR_DIM + 2);
  p.many_pieces = p.few_pieces + (p.few_splits > 1 ? (size_t)few * p.few_splits * kFewRows * (QDR_DIM + 2) : 0);
  p.info = p.many_pieces + (p.many_splits > 1 ? (size_t)p.many_tiles * heads * p.many_parts * p.many_splits * kManyRows * (QDR_DIM + 2) : 0);
  p.floats = p.info + (size_t)T * p.few_parts * 2 * 4;
  return p;
}

}  // namespace qdr

extern "C" {

qdr_status qdr_rotary_frequencies(int32_t rule, int32_t channels, double base, double factor, double context,
                                  double low, double high, double *freq, double *amplitude) {
  if (rule < QDR_ROTARY_PLAIN || rule > QDR_ROTARY_INDEX) return fail(QDR_E_INVAL, "bad rule %d", rule);
  QDR_TRY(check_channels(channels));
  if (!freq || !amplitude) return fail(QDR_E_INVAL, "freq or amplitude is NULL");
  if (!(base > 1.0) || !std::isfinite(base)) return fail(QDR_E_INVAL, "base must be finite and > 1 (got %g)", base);
  if (rule != QDR_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return fail(QDR_E_INVAL, "factor must be finite and >= 1 (got %g)", factor);
  const bool blends = rule == QDR_ROTARY_TURNS || rule == QDR_ROTARY_INDEX;
  if (blends && (!(context > 0.0) || !std::isfinite(context))) return fail(QDR_E_INVAL, "context must be finite and > 0 (got %g)", context);
  if (blends && (!(low > 0.0) || !(high > low) || !std::isfinite(high))) return fail(QDR_E_INVAL, "low and high must be finite, 0 < low < high (got %g, %g)", low, high);
  const auto index_of = [&](double turns) { return channels * std::log(context / (2 * kPi * turns)) / (2 * std::log(base)); };
  const double a = rule == QDR_ROTARY_INDEX ? std::max(std::floor(index_of(high)), 0.0) : 0.0;
  const double b = rule == QDR_ROTARY_INDEX ? std::min(std::ceil(index_of(low)), channels - 1.0) : 0.0;
  for (int32_t i = 0; i < channels / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / channels);
    double keep = 1.0;
    if (rule == QDR_ROTARY_LINEAR) keep = 0.0;
    if (rule == QDR_ROTARY_TURNS) keep = (context * f / (2 * kPi) - low) / (high - low);
    if (rule == QDR_ROTARY_INDEX) keep = 1.0 - (i - a) / std::max(b - a, 0.001);
    keep = std::min(std::max(keep, 0.0), 1.0);
    freq[i] = rule == QDR_ROTARY_PLAIN ? f : keep * f + (1.0 - keep) * f / factor;
  }
  *amplitude = rule == QDR_ROTARY_INDEX ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return qdr::set_ok();
}

qdr_status qdr_rotary_create(const qdr_rotary_desc *desc, qdr_rotary **out) {
  if (!desc) return fail(QDR_E_INVAL, "desc is NULL");
  if (desc->d != QDR_DIM) return fail(QDR_E_UNSUPPORTED, "d must be %d (got %d)", QDR_DIM, desc->d);
  QDR_TRY(check_channels(desc->channels));
  if (desc->layout != QDR_ROTARY_HALF && desc->layout != QDR_ROTARY_PAIRS) return fail(QDR_E_INVAL, "bad layout %d", desc->layout);
  if (!desc->freq) return fail(QDR_E_INVAL, "freq is NULL");
  uint64_t turns[QDR_DIM / 2] = {};
  for (int32_t i = 0; i < desc->channels / 2; ++i) {
    if (!(std::fabs(desc->freq[i]) <= 1048576.0)) return fail(QDR_E_INVAL, "freq[%d] must be finite, of magnitude <= 2^20 (got %g)", i, desc->freq[i]);
    turns[i] = turns_of(desc->freq[i]);
  }
  if (!std::isfinite((float)desc->amplitude)) return fail(QDR_E_INVAL, "amplitude must be a finite fp32 (got %g)", desc->amplitude);
  if (!out) return fail(QDR_E_INVAL, "out is NULL");
  *out = nullptr;
  qdr_rotary *r = new (std::nothrow) qdr_rotary();
  if (!r) return fail(QDR_E_NOMEM, "host allocation failed");
  r->channels = desc->channels;
  r->layout = desc->layout;
  r->amplitude = (float)desc->amplitude;
  if (hipGetDevice(&r->device) != hipSuccess) {
    delete r;
    return fail(QDR_E_DEVICE, "no HIP device");
  }
  hipError_t e = hipMalloc(reinterpret_cast<void **>(&r->turns), sizeof turns);
  if (e != hipSuccess) r->turns = nullptr;
  if (e == hipSuccess) e = hipMemcpy(r->turns, turns, sizeof turns, hipMemcpyHostToDevice);
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) {
    (void)hipGetLastError();
    if (r->turns) (void)hipFree(r->turns);
    delete r;
    return fail(e == hipErrorOutOfMemory ? QDR_E_NOMEM : QDR_E_DEVICE, "rotary setup failed: %s", hipGetErrorString(e));
  }
  *out = r;
  return qdr::set_ok();
}

qdr_status qdr_rotary_destroy(qdr_rotary *r) {
  if (!r) return qdr::set_ok();
  const int own = r->device;
  int now = own;
  (void)hipGetDevice(&now);
  if (now != own) (void)hipSetDevice(own);
  (void)hipDeviceSynchronize();
  (void)hipFree(r->turns);
  delete r;
  if (now != own) (void)hipSetDevice(now);
  return qdr::set_ok();
}

qdr_status qdr_rotate(qdr_rotary *rotary, const int32_t *positions, int32_t T, int32_t heads, const float *x,
                      int64_t x_stride, float *y, int64_t y_stride, void *stream) {
  return rotate(rotary, positions, T, heads, x, x_stride, y, y_stride, stream, false);
}

qdr_status qdr_rotate_bf16(qdr_rotary *rotary, const int32_t *positions, int32_t T, int32_t heads, const uint16_t *x,
                           int64_t x_stride, uint16_t *y, int64_t y_stride, void *stream) {
  return rotate(rotary, positions, T, heads, x, x_stride, y, y_stride, stream, true);
}

qdr_status qdr_kv_write_rotary(qdr_kv *kv, qdr_rotary *rotary, const int32_t *pages, int32_t max_pages,
                               const int32_t *cu, const int32_t *context, int32_t n, int32_t T, const uint16_t *q,
                               int64_t q_stride, int32_t q_heads, uint16_t *q_out, const uint16_t *k,
                               int64_t k_stride, const uint16_t *v, int64_t v_stride, void *stream) {
  if (!rotary) return fail(QDR_E_INVAL, "rotary is NULL");
  QDR_TRY(check_kv_call(kv, pages, max_pages, cu, context, n, T, k, v));
  if (q_heads < 0 || q_heads > kMostHeads) return fail(QDR_E_INVAL, "q_heads must be from 0 to %d (got %d)", kMostHeads, q_heads);
  if (kv->desc.num_heads > kMostHeads) return fail(QDR_E_UNSUPPORTED, "a cache of at most %d heads (got %d)", kMostHeads, kv->desc.num_heads);
  QDR_TRY(check_stride("k_stride", k_stride, kv->desc.num_heads, true));
  QDR_TRY(check_stride("v_stride", v_stride, kv->desc.num_heads, true));
  if (q_heads) QDR_TRY(check_stride("q_stride", q_stride, q_heads, true));
  if (n == 0 || T == 0) return qdr::set_ok();
  if (q_heads && (!q || !q_out)) return fail(QDR_E_INVAL, "q or q_out is NULL");
  if (!aligned4(q) || !aligned4(q_out)) return fail(QDR_E_INVAL, "tensors must be 4-byte aligned");
  if (rotary->device != kv->device) return fail(QDR_E_INVAL, "rotary belongs to device %d, the cache to %d", rotary->device, kv->device);
  qdr::RotaryWriteArgs a{};
  a.kv = kv_args(kv, pages, max_pages, cu, context, n, T);
  a.kv.k = const_cast<uint16_t *>(k);
  a.kv.v = const_cast<uint16_t *>(v);
  a.rotary = view_of(rotary);
  a.q = q;
  a.q_out = q_out;
  a.q_heads = q_heads;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  // A block's table serves several heads, where whole blocks alone make enough
  // workgroups, and the other way round for queries, of which a single token has
  // few.  Measured per call (us), 32 and 8 heads, 8-bit; 1 and 4 key heads a
  // workgroup: 600 tokens of 5 prompts 10.6 and 13.9, 2000 18.0 and 16.7, 4100 27.7 and
  // 25.7, 16391 80 and 72 (bfloat16 83 and 81); 64 single tokens 9.8 and 12.6 (1024,
  // which this rule leaves at one, 77 and 50).  8 and 32 query heads: 256 single tokens
  // 25.2 and 21.3, 1024 95 and 77, 4096 251 and 174; 64 times 9 tokens 12.4 and 17.1;
  // 600 of 5 prompts 10.8 and 28.5, 16391 72 and 86.
  const bool prompts = T / qdr::kBlock >= 128;
  a.kv_heads = prompts ? 4 : 1;
  a.kv_parts = (kv->desc.num_heads + a.kv_heads - 1) / a.kv_heads;
  a.query_heads = T > 8 * (int64_t)n ? 8 : 32;
  a.query_parts = (q_heads + a.query_heads - 1) / a.query_heads;
  QDR_TRY(check_groups((T / qdr::kBlock + 2 * (int64_t)n) * (a.kv_parts + a.query_parts)));
  return launched(qdr::launch_kv_write_rotary(a, kv->desc.kind, static_cast<hipStream_t>(stream)));
}

qdr_status qdr_kv_copy(qdr_kv *from, const int32_t *src_pages, qdr_kv *to, const int32_t *dst_pages, int32_t m, void *stream) {
  if (!from || !to) return fail(QDR_E_INVAL, "from or to is NULL");
  QDR_TRY(check_counts(m, 0));
  if (from->desc.page_tokens != to->desc.page_tokens || from->desc.num_heads != to->desc.num_heads || from->desc.kind != to->desc.kind)
    return fail(QDR_E_INVAL, "the caches differ in page_tokens, num_heads or kind");
  if (from->device != to->device) return fail(QDR_E_INVAL, "the caches belong to devices %d and %d", from->device, to->device);
  if (m == 0) return qdr::set_ok();
  if (!src_pages || !dst_pages) return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  QDR_TRY(check_device(from->device));
  qdr::CopyArgs a{};
  a.from = from->base;
  a.to = to->base;
  a.bytes = page_bytes(from);
  a.src = src_pages;
  a.dst = dst_pages;
  a.m = m;
  a.num_from = from->desc.num_pages;
  a.num_to = to->desc.num_pages;
  a.parts = parts_of(a.bytes);
  a.err_from = from->d_err;
  a.err_to = to->d_err;
  a.bit = qdr::kErrPage;
  QDR_TRY(check_groups((int64_t)m * a.parts));
  return launched(qdr::launch_copy(a, static_cast<hipStream_t>(stream)));
}

qdr_status qdr_slot_copy(qdr_pool *pool, const int32_t *src_slots, const int32_t *dst_slots, int32_t m, void *stream) {
  if (!pool) return fail(QDR_E_INVAL, "pool is NULL");
  QDR_TRY(check_counts(m, 0));
  if (m == 0) return qdr::set_ok();
  if (!src_slots || !dst_slots) return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  const qdr::PoolView view = qdr::pool_view(pool);
  QDR_TRY(check_device(view.device));
  qdr::CopyArgs a{};
  a.from = view.base;
  a.to = view.base;
  a.bytes = view.slot_stride;
  a.src = src_slots;
  a.dst = dst_slots;
  a.m = m;
  a.num_from = a.num_to = view.num_slots;
  a.parts = parts_of(a.bytes);
  a.err_from = a.err_to = view.err;
  a.bit = qdr::kErrSlot;
  QDR_TRY(check_groups((int64_t)m * a.parts));
  hipStream_t st = static_cast<hipStream_t>(stream);
  hipError_t e = qdr::pool_after_writeback(pool, st);
  if (e == hipSuccess) e = qdr::launch_copy(a, st);
  return launched(e);
}

qdr_status qdr_kv_assign_workspace(const qdr_kv *kv, int32_t m, size_t *bytes) {
  if (!kv || !bytes) return fail(QDR_E_INVAL, "kv or bytes is NULL");
  QDR_TRY(check_counts(m, 0));
  QDR_TRY(check_pages(kv));
  *bytes = assign_space(kv, m).total();
  return qdr::set_ok();
}

qdr_status qdr_kv_assign(qdr_kv *kv, const int32_t *pages, const int32_t *context, int32_t n, int32_t max_pages,
                         const int32_t *parent, const int32_t *add, int32_t m, const int32_t *refs,
                         int32_t *new_pages, int32_t *new_context, int32_t *new_refs, void *workspace,
                         size_t workspace_bytes, void *stream) {
  if (!kv) return fail(QDR_E_INVAL, "kv is NULL");
  QDR_TRY(check_counts(n, m));
  QDR_TRY(check_pages(kv));
  if (max_pages < 0) return fail(QDR_E_INVAL, "max_pages must be >= 0 (got %d)", max_pages);
  if (!refs || !new_refs || (n > 0 && (!context || (max_pages > 0 && !pages))) ||
      (m > 0 && (!parent || !add || !new_context || (max_pages > 0 && !new_pages))))
    return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  QDR_TRY(check_device(kv->device));
  const int64_t total = kv->desc.num_pages, chunks = ((int64_t)max_pages + 255) / 256 + (max_pages == 0);
  const Span in[] = {{pages, (int64_t)n * max_pages}, {context, n}, {parent, m}, {add, m}, {refs, total}};
  const Span out[] = {{new_pages, (int64_t)m * max_pages}, {new_context, m}, {new_refs, total}};
  QDR_TRY(check_apart(in, 5, out, 3));
  const int32_t parts = parts_of(page_bytes(kv));
  QDR_TRY(check_groups(std::max<int64_t>(n, m)));   // (their products below fit 64 bits)
  QDR_TRY(check_groups(std::max<int64_t>(n, m) * chunks + qdr::book_tiles(total)));
  QDR_TRY(check_groups((int64_t)m * parts));
  const AssignSpace space = assign_space(kv, m);
  QDR_TRY(check_workspace(workspace, workspace_bytes, space.total()));
  char *ws = static_cast<char *>(workspace);
  qdr::AssignArgs a{};
  a.kv = kv_args(kv, pages, max_pages, nullptr, context, n, 0);
  a.kind = kv->desc.kind;
  a.parent = parent;
  a.add = add;
  a.refs = refs;
  a.m = m;
  a.new_pages = new_pages;
  a.new_context = new_context;
  a.new_refs = new_refs;
  a.hold = reinterpret_cast<int32_t *>(ws);
  a.first = reinterpret_cast<int32_t *>(ws + space.pages);
  a.free = reinterpret_cast<int32_t *>(ws + 2 * space.pages);
  a.counts = reinterpret_cast<int32_t *>(ws + 3 * space.pages);
  a.offset = reinterpret_cast<int32_t *>(ws + 3 * space.pages + space.counts);
  a.parts = parts;
  return launched(qdr::launch_assign(a, static_cast<hipStream_t>(stream)));
}

qdr_status qdr_kv_compact_workspace(const qdr_kv *kv, size_t *bytes) {
  if (!kv || !bytes) return fail(QDR_E_INVAL, "kv or bytes is NULL");
  QDR_TRY(check_pages(kv));
  *bytes = compact_space(kv).total();
  return qdr::set_ok();
}

qdr_status qdr_kv_compact(qdr_kv *kv, const int32_t *refs, const int32_t *pages, int32_t n, int32_t max_pages,
                          int32_t *moved, int32_t *new_refs, int32_t *new_pages, void *workspace,
                          size_t workspace_bytes, void *stream) {
  if (!kv) return fail(QDR_E_INVAL, "kv is NULL");
  QDR_TRY(check_counts(n, 0));
  QDR_TRY(check_pages(kv));
  if (max_pages < 0) return fail(QDR_E_INVAL, "max_pages must be >= 0 (got %d)", max_pages);
  const int64_t entries = (int64_t)n * max_pages, total = kv->desc.num_pages;
  if (!refs || !moved || !new_refs || (entries > 0 && (!pages || !new_pages))) return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  QDR_TRY(check_device(kv->device));
  const Span in[] = {{refs, total}, {pages, entries}}, out[] = {{moved, total}, {new_refs, total}, {new_pages, entries}};
  QDR_TRY(check_apart(in, 2, out, 3));
  QDR_TRY(check_groups(entries / 256 + 1 + kMoveGroups));
  const CompactSpace space = compact_space(kv);
  QDR_TRY(check_workspace(workspace, workspace_bytes, space.total()));
  char *ws = static_cast<char *>(workspace);
  qdr::CompactArgs a{};
  a.base = kv->base;
  a.page_bytes = page_bytes(kv);
  a.num_pages = kv->desc.num_pages;
  a.refs = refs;
  a.pages = pages;
  a.entries = entries;
  a.moved = moved;
  a.new_refs = new_refs;
  a.new_pages = new_pages;
  a.src = reinterpret_cast<int32_t *>(ws);
  a.dst = reinterpret_cast<int32_t *>(ws + space.pages);
  a.counts = reinterpret_cast<int32_t *>(ws + 2 * space.pages);
  a.moves = reinterpret_cast<int32_t *>(ws + 2 * space.pages + space.counts);
  a.parts = parts_of(a.page_bytes);
  a.groups = (int32_t)std::max<int64_t>(1, std::min<int64_t>(kMoveGroups, total / 2 * a.parts));
  return launched(qdr::launch_compact(a, static_cast<hipStream_t>(stream)));
}

qdr_status qdr_kv_attend_shared_workspace(const qdr_kv *kv, int32_t n, int32_t T, int32_t groups, int32_t q_heads,
                                          int32_t max_pages, size_t *bytes) {
  if (!kv || !bytes) return fail(QDR_E_INVAL, "kv or bytes is NULL");
  QDR_TRY(check_counts(n, T));
  QDR_TRY(check_counts(groups, 0));
  QDR_TRY(check_heads(kv, q_heads));
  if (max_pages < 0) return fail(QDR_E_INVAL, "max_pages must be >= 0 (got %d)", max_pages);
  *bytes = 0;
  if (n == 0 || T == 0) return qdr::set_ok();
  qdr::SharedPlan plan;
  QDR_TRY(make_shared(kv, n, T, groups, q_heads, max_pages, &plan, bytes));
  return qdr::set_ok();
}

qdr_status qdr_kv_attend_shared(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                                const int32_t *context, int32_t n, int32_t T, const int32_t *group_cu,
                                const int32_t *shared, int32_t groups, int32_t q_heads, const uint16_t *q,
                                float scale, uint16_t *o, void *workspace, size_t workspace_bytes, void *stream) {
  QDR_TRY(check_kv_call(kv, pages, max_pages, cu, context, n, T, q, o));
  QDR_TRY(check_counts(groups, 0));
  QDR_TRY(check_heads(kv, q_heads));
  if (!std::isfinite(scale)) return fail(QDR_E_INVAL, "scale must be finite");
  if (n == 0 || T == 0) return qdr::set_ok();
  if (groups > 0 && (!group_cu || !shared)) return fail(QDR_E_INVAL, "group_cu or shared is NULL");
  qdr::SharedPlan plan;
  size_t need = 0;
  QDR_TRY(make_shared(kv, n, T, groups, q_heads, max_pages, &plan, &need));
  QDR_TRY(check_workspace(workspace, workspace_bytes, need));
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return fail(QDR_E_INVAL, "scale is too large (%g)", (double)scale);
  qdr::SharedArgs s{};
  s.a.kv = kv_args(kv, pages, max_pages, cu, context, n, T);
  s.a.q = q;
  s.a.o = o;
  s.a.q_heads = q_heads;
  s.a.scale_log2 = scale_log2;
  s.a.part = static_cast<float *>(workspace);
  s.group_cu = group_cu;
  s.shared = shared;
  s.groups = groups;
  return launched(qdr::launch_attend_shared(s, plan, kv->desc.kind, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
