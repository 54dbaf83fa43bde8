// qdr_mixer.cpp -- host side of the token mixers (include/qdr_mixer.h):
// argument checks, workspaces, the paged cache's handle, and the launches.
#include "../../include/qdr_mixer.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "qdr_host.h"
#include "qdr_mixer.h"

namespace {

qdr_status fail(qdr_status st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return qdr::set_error(st, buf);
}

qdr_status launched(hipError_t e) {
  if (e != hipSuccess) return fail(QDR_E_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
  return qdr::set_ok();
}

// Counts of sequences and rows are kept where sums of them fit 32 bits, and
// launches under 2^32 threads.
constexpr int32_t kMostRows = 1 << 30;
constexpr int32_t kMostHeads = 1 << 17;             // 64 rows of a token array under 2^32 bytes
constexpr int64_t kMostGroups = (int64_t)1 << 24;   // of 256 threads

qdr_status check_counts(int32_t n, int32_t T) {
  if (n < 0 || T < 0) return fail(QDR_E_INVAL, "n and T must be >= 0 (got %d, %d)", n, T);
  if (n > kMostRows || T > kMostRows) return fail(QDR_E_INVAL, "n and T must be <= %d (got %d, %d)", kMostRows, n, T);
  return QDR_OK;
}

qdr_status check_groups(int64_t groups) {
  if (groups >= kMostGroups) return fail(QDR_E_INVAL, "the call is too large for one launch (%lld workgroups): cut it up", (long long)groups);
  return QDR_OK;
}

qdr_status check_device(int device) {
  int now = -1;
  if (hipGetDevice(&now) != hipSuccess) return fail(QDR_E_DEVICE, "no HIP device");
  if (now != device) return fail(QDR_E_INVAL, "the handle belongs to device %d, the current device is %d", device, now);
  return QDR_OK;
}

qdr_status check_workspace(const void *ws, size_t have, size_t need) {
  if (need == 0) return QDR_OK;
  if (!ws) return fail(QDR_E_INVAL, "workspace is NULL (%zu bytes are needed)", need);
  if (reinterpret_cast<uintptr_t>(ws) % 16) return fail(QDR_E_INVAL, "workspace must be 16-byte aligned");
  if (have < need) return fail(QDR_E_NOMEM, "workspace holds %zu bytes, the call needs %zu", have, need);
  return QDR_OK;
}

bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

#define QDR_TRY(x)                     \
  do {                                 \
    const qdr_status st_ = (x);        \
    if (st_ != QDR_OK) return st_;     \
  } while (0)

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Sequences cut into segments of so many chunks (0: not cut), and places of
// segments of one head.
struct Cut {
  int32_t chunks;
  int64_t places;
};

// SUM: segments of one length for all, as if the sequences were alike: as many
// as there are places for workgroups, two to each of 256 compute units (16385
// tokens of 16 heads in segments of 4, 8, 16, 32 chunks and uncut: 165, 139,
// 159, 263, 1396 us), that divide the mean length (eight sequences of 2000
// tokens, 48 heads, in 16, 24, 32 chunks: 345, 441, 302 us); of four chunks at
// least, and long ones of more, since they are joined one by one (32768 tokens
// of 4 heads in 4, 8, 16: 120, 105, 142 us).  Where the sequences alone fill
// the places, only one of twice the mean length is cut, which then does not run
// alone.
Cut cut_sum(int32_t heads, int32_t n, int32_t T) {
  const int64_t pairs = (int64_t)n * heads, places = 2 * 256;
  const int64_t mean = (T + (int64_t)n * qdr::kChunk - 1) / ((int64_t)n * qdr::kChunk);
  int64_t segment = qdr::kSegmentLeast;
  if (pairs > places) {
    while (segment < 2 * mean) segment *= 2;
  } else {
    const int64_t each = places / pairs;
    // (a last chunk that is nearly empty counts where it would be a segment by itself)
    segment = std::max(segment, each == 1 ? mean : (T / ((int64_t)n * qdr::kChunk) + each - 1) / each);
    while (8 * segment * segment < mean) ++segment;
  }
  if (segment * qdr::kChunk >= T) return {0, 0};
  return {(int32_t)segment, T / (segment * qdr::kChunk) + n};
}

// DELTA: a segment's map of states costs twice what its chunks cost, so it is
// calls of few heads that are cut, where most compute units would have nothing
// to do.  Whether and where follows from what the launches take, in 0.1 us: a
// chunk 51 in k_prompt_map and 70 in k_prompt_scan, one workgroup a compute
// unit at a time, 16 to join a segment, 40 a round of workgroups, 160 for the
// launches; 27 a chunk in k_prompt_chain.  Of a call of several sequences only
// the mean length is known: the longest is taken as twice that, and segments
// have to win by a fifth.  One sequence, chain against segments, us:
//   4 heads   16 chunks 57 / 67   64 chunks 189 / 91   512 chunks 1434 / 258
//   16 heads  32 chunks 105 / 88  64 chunks 199 / 135  512 chunks 1612 / 613
//   32 heads  32 chunks 108 / 125 64 chunks 213 / 192  256 chunks 854 / 595
//   48 heads  187 chunks 689 / 788   512 chunks 1780 / 1835
Cut cut_delta(int32_t heads, int32_t n, int32_t T) {
  const int64_t pairs = (int64_t)n * heads, chunks = T / qdr::kChunk, mean = (chunks + n - 1) / n;
  const int64_t longest = n == 1 ? mean : 2 * mean;
  if (!qdr::in_chains(n, heads)) return {0, 0};
  const auto rounds = [](int64_t groups) { return (groups + 255) / 256; };
  int64_t least = std::max(longest * 27, chunks * heads * 4 * 27 / 256), segment = 0;
  for (int64_t s = qdr::kSegmentLeast; s <= qdr::kSegmentMost; ++s) {
    const int64_t each = (mean + s - 1) / s;
    if (each < 2) break;
    const int64_t cost = rounds(pairs * (2 * each - 3)) * (51 * s + 40) + rounds(pairs * each) * (70 * s + 40) + (longest + s - 1) / s * 16 + 160;
    if ((n == 1 ? cost : cost * 5 / 4) < least) {
      least = n == 1 ? cost : cost * 5 / 4;
      segment = s;
    }
  }
  if (!segment) return {0, 0};
  return {(int32_t)segment, T / (segment * qdr::kChunk) + n};
}

// Parts of a prompt's workspace.  It is the same for both rules.
struct PromptSpace {
  int64_t places;                // chunk places of one head
  Cut sum, delta;
  bool ordered;
  size_t chunks, tables, states, parts;  // bytes
  size_t total() const { return chunks + tables + states + parts; }
};

PromptSpace prompt_space(const qdr::PoolView &v, int32_t n, int32_t T) {
  const size_t state = (size_t)v.num_heads * QDR_DIM * QDR_DIM * sizeof(float);
  PromptSpace s{};
  s.places = T / qdr::kChunk + (int64_t)n;
  s.chunks = up((size_t)s.places * v.num_heads * qdr::kChunkFloats * sizeof(float));
  s.ordered = n > 1 && n <= qdr::kMostOrdered;
  s.tables = up((size_t)n * ((v.all_fp32 ? 0 : 2) + (s.ordered ? 1 : 0)) * sizeof(int32_t));
  s.states = v.all_fp32 ? 0 : (size_t)n * state;
  s.sum = cut_sum(v.num_heads, n, T);
  s.delta = cut_delta(v.num_heads, n, T);
  s.parts = up(std::max((size_t)s.sum.places * (state + v.num_heads * sizeof(float)),
                        (size_t)s.delta.places * (state + v.num_heads * qdr::kMapFloats * sizeof(float))));
  return s;
}

// Whether a prompt's launches can be counted.
qdr_status check_prompt(const qdr::PoolView &v, const PromptSpace &s, int32_t n) {
  QDR_TRY(check_groups(s.places * v.num_heads + qdr::kMostOrdered / 256));
  // of 512 threads: segments, and to join them eight a head
  return check_groups((n + std::max(s.sum.places, s.delta.places)) * v.num_heads * 16);
}

}  // namespace

namespace qdr {

AttendPlan plan_attend(int n, int T, int q_heads, int heads, int max_pages, int page_shift) {
  AttendPlan p{};
  p.group = q_heads / heads;
  p.few_heads = p.group < kFewRows ? p.group : kFewRows;
  p.few_tokens = kFewRows / p.few_heads;
  p.few_parts = (p.group + p.few_heads - 1) / p.few_heads;
  p.many_heads = p.group < kManyRows ? p.group : kManyRows;
  p.many_tokens = kManyRows / p.many_heads;
  p.many_parts = (p.group + p.many_heads - 1) / p.many_heads;
  // T <= n: hardly a sequence has more than one token.  One sequence: its
  // length is T.  Else the two launches share the sequences out by length, also
  // where T says that most are long: a token among long chunks would walk its
  // whole context in one workgroup, and its weights would lose their second part
  // (32 query and 8 key heads, bfloat16: three tokens over 32768 keys beside a
  // prompt of 8192 711 us, in one launch 1714; 4 x 256 over 2048, where the
  // few-row launch finds nothing, 73 and 69).
  p.few = n > 1 || T <= p.few_tokens;
  p.many = T > n && !(n == 1 && T <= p.few_tokens);
  p.few_tiles = !p.few ? 0 : p.many ? n : T / p.few_tokens + n;
  p.many_tiles = p.many ? T / p.many_tokens + n : 0;
  const int64_t blocks = (int64_t)max_pages << (page_shift - 5);
  // Pieces: as many as the compute units have places for, which is one few-row
  // workgroup each or two many-row ones: more of them wait, and pay a start and
  // partial results for nothing (32 query and 8 key heads, 8192 cached tokens,
  // 8-bit: 8 requests in 4, 8, 16 pieces 32, 40, 52 us, one of 64 requests uncut
  // and in 2 193 and 210).  None where that costs more than it gives:
  //   few rows   up to 32 blocks (1 and 8 requests, bfloat16: 1024 tokens uncut
  //              10.5 and 11.5 us, cut 10.5 and 13.3; 2048 14.5 and 18.5, 10.7
  //              and 19.8); above 64 tiles pieces of 64 blocks (16 requests: 3000
  //              tokens uncut 33, in two 37; 8192, 8-bit, 65 and 53);
  //   many rows  up to 8 blocks, above 32 tiles up to 24 (20 new tokens: 512
  //              cached uncut 21.8 us, cut 15.8; three times 100: 512 26.8 and
  //              36.0, 1024 40.7 and 38.5).
  auto cut = [&](int64_t units, int64_t least, int places, int64_t uncut) {
    if (blocks <= uncut) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({places / std::max<int64_t>(units, 1), (blocks + least - 1) / least, 64}));
  };
  // tiles, as if the sequences were alike
  const int64_t each = (T + (int64_t)n - 1) / n;
  const int64_t few_units = (int64_t)(T <= n ? T : n) * heads * p.few_parts;
  const int64_t many_units = n * ((each + p.many_tokens - 1) / p.many_tokens) * heads * p.many_parts;
  p.few_splits = p.few ? cut(few_units, few_units > 64 ? 64 : kFewLeast, 256, 32) : 1;
  p.many_splits = p.many ? cut(many_units, kManyLeast, 512, many_units > 32 ? 24 : 8) : 1;
  p.few_floats = p.few_splits > 1 ? (size_t)p.few_tiles * heads * p.few_parts * p.few_splits * kFewRows * (QDR_DIM + 2) : 0;
  p.many_floats = p.many_splits > 1 ? (size_t)p.many_tiles * heads * p.many_parts * p.many_splits * kManyRows * (QDR_DIM + 2) : 0;
  return p;
}

}  // namespace qdr

struct qdr_kv {
  qdr_kv_desc desc{};
  int device = 0;
  int page_shift = 0;
  uint8_t *base = nullptr;
  bool owns_base = false;
  uint32_t *d_err = nullptr;
};

namespace {

qdr_status check_kv_desc(const qdr_kv_desc *d, size_t *bytes, int *shift) {
  if (!d) return fail(QDR_E_INVAL, "desc is NULL");
  if (d->num_pages <= 0) return fail(QDR_E_INVAL, "num_pages must be > 0 (got %d)", d->num_pages);
  if (d->num_heads <= 0) return fail(QDR_E_INVAL, "num_heads must be > 0 (got %d)", d->num_heads);
  if (d->d != QDR_DIM) return fail(QDR_E_UNSUPPORTED, "d must be %d (got %d)", QDR_DIM, d->d);
  if (d->kind != QDR_KV_INT8 && d->kind != QDR_KV_BF16) return fail(QDR_E_INVAL, "bad kind %d", d->kind);
  int s = 5;
  while (s <= 10 && (1 << s) != d->page_tokens) ++s;
  if (s > 10) return fail(QDR_E_INVAL, "page_tokens must be a power of two from 32 to 1024 (got %d)", d->page_tokens);
  const size_t block = d->kind == QDR_KV_INT8 ? qdr::kKv8Block : qdr::kKv16Block;
  const size_t page = (size_t)d->num_heads * (d->page_tokens / qdr::kBlock) * block;   // under 2^50
  if (page > (size_t)INT64_MAX / d->num_pages)
    return fail(QDR_E_INVAL, "%d pages of %zu bytes do not fit 64 bits", d->num_pages, page);
  *bytes = (size_t)d->num_pages * page;
  *shift = s;
  return QDR_OK;
}

void free_kv(qdr_kv *kv) {
  if (!kv) return;
  if (kv->owns_base && kv->base) (void)hipFree(kv->base);
  (void)hipFree(kv->d_err);
  delete kv;
}

qdr_status check_kv_call(const qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                         const int32_t *context, int32_t n, int32_t T, const void *x, const void *y) {
  if (!kv) return fail(QDR_E_INVAL, "kv is NULL");
  QDR_TRY(check_counts(n, T));
  if (max_pages < 0) return fail(QDR_E_INVAL, "max_pages must be >= 0 (got %d)", max_pages);
  if (n == 0 || T == 0) return QDR_OK;
  if (!cu || !context || (max_pages > 0 && !pages) || !x || !y) return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  if (!aligned4(x) || !aligned4(y)) return fail(QDR_E_INVAL, "tensors must be 4-byte aligned");
  return check_device(kv->device);
}

qdr::KvArgs kv_args(const qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                    const int32_t *context, int32_t n, int32_t T) {
  qdr::KvArgs a{};
  a.base = kv->base;
  a.num_pages = kv->desc.num_pages;
  a.page_shift = kv->page_shift;
  a.heads = kv->desc.num_heads;
  a.pages = pages;
  a.max_pages = max_pages;
  a.cu = cu;
  a.context = context;
  a.n = n;
  a.T = T;
  a.err = kv->d_err;
  return a;
}

}  // namespace

extern "C" {

qdr_status qdr_prompt_workspace(const qdr_pool *pool, int32_t n, int32_t T, size_t *bytes) {
  if (!pool || !bytes) return fail(QDR_E_INVAL, "pool or bytes is NULL");
  QDR_TRY(check_counts(n, T));
  *bytes = 0;
  if (n == 0) return qdr::set_ok();
  const qdr::PoolView view = qdr::pool_view(pool);
  if (view.num_heads > kMostHeads) return fail(QDR_E_UNSUPPORTED, "the prompt form takes at most %d heads (got %d)", kMostHeads, view.num_heads);
  const PromptSpace space = prompt_space(view, n, T);
  QDR_TRY(check_prompt(view, space, n));
  *bytes = space.total();
  return qdr::set_ok();
}

qdr_status qdr_prompt(qdr_pool *pool, int32_t rule, const int32_t *slots, const int32_t *carry, const int32_t *cu,
                      int32_t n, int32_t T, const uint16_t *q, const uint16_t *k, const uint16_t *v,
                      const float *beta, const float *gate, uint16_t *o, void *workspace, size_t workspace_bytes,
                      void *stream) {
  if (!pool) return fail(QDR_E_INVAL, "pool is NULL");
  if (rule != QDR_RULE_DELTA && rule != QDR_RULE_SUM) return fail(QDR_E_INVAL, "bad rule %d", rule);
  QDR_TRY(check_counts(n, T));
  if (n == 0) return qdr::set_ok();
  const bool delta = rule == QDR_RULE_DELTA;
  if (!slots || !cu || (T > 0 && (!q || !k || !v || !gate || !o || (delta && !beta))))
    return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  if (!aligned4(q) || !aligned4(k) || !aligned4(v) || !aligned4(o)) return fail(QDR_E_INVAL, "tensors must be 4-byte aligned");
  const qdr::PoolView view = qdr::pool_view(pool);
  if (view.gate != QDR_GATE_SCALAR) return fail(QDR_E_UNSUPPORTED, "the prompt form takes one gate a head (QDR_GATE_SCALAR)");
  if (view.num_heads > kMostHeads) return fail(QDR_E_UNSUPPORTED, "the prompt form takes at most %d heads (got %d)", kMostHeads, view.num_heads);
  QDR_TRY(check_device(view.device));
  const PromptSpace space = prompt_space(view, n, T);
  QDR_TRY(check_prompt(view, space, n));
  QDR_TRY(check_workspace(workspace, workspace_bytes, space.total()));
  hipStream_t st = static_cast<hipStream_t>(stream);
  QDR_TRY(qdr::pool_check_slots(pool, slots, n, st));

  uint8_t *ws = static_cast<uint8_t *>(workspace);
  qdr::PromptArgs a{};
  a.slots = slots;
  a.carry = carry;
  a.cu = cu;
  a.n = n;
  a.T = T;
  a.H = view.num_heads;
  a.num_slots = view.num_slots;
  a.chunks = (int32_t)space.places;
  a.q = q;
  a.k = k;
  a.v = v;
  a.beta = delta ? beta : nullptr;
  a.gate = gate;
  a.o = o;
  a.chunk_ws = reinterpret_cast<float *>(ws);
  a.err = view.err;
  int32_t *table = reinterpret_cast<int32_t *>(ws + space.chunks);
  if (view.all_fp32) {
    a.pool = view.base;
    a.slot_stride = view.slot_stride;
  } else {
    a.slots_in = table;
    a.slots_out = table + n;
    table += 2 * (size_t)n;
    a.S = reinterpret_cast<float *>(ws + space.chunks + space.tables);
  }
  const Cut cut = delta ? space.delta : space.sum;
  if (cut.chunks) {
    a.segment = cut.chunks;
    a.segments = (int32_t)cut.places;
    a.segment_ws = reinterpret_cast<float *>(ws + space.chunks + space.tables + space.states);
    a.map_ws = a.segment_ws + (size_t)cut.places * view.num_heads * QDR_DIM * QDR_DIM;
  } else if (delta && space.ordered && T > 0) {   // (without rows there is no launch that orders)
    a.order = table;
  }
  hipError_t e = qdr::pool_after_writeback(pool, st);
  if (e == hipSuccess && !a.pool) e = qdr::launch_prompt_slots(a, st);
  if (e != hipSuccess) return launched(e);
  if (!a.pool && carry) QDR_TRY(qdr::pool_unpack(pool, a.slots_in, n, a.S, st));
  if (T > 0) e = qdr::launch_prompt_chunks(a, delta, st);
  if (e == hipSuccess) e = qdr::launch_prompt_scan(a, delta, st);
  if (e != hipSuccess) return launched(e);
  if (!a.pool) return qdr::pool_pack(pool, a.slots_out, n, a.S, st);
  return qdr::set_ok();
}

static qdr_status linear_step(qdr_pool *pool, const int32_t *slots, int32_t B, const void *q, const void *k,
                              const void *v, const float *gate, void *o, void *stream, bool bf16) {
  if (!pool) return fail(QDR_E_INVAL, "pool is NULL");
  if (B < 0) return fail(QDR_E_INVAL, "B must be >= 0");
  if (B == 0) return qdr::set_ok();
  if (!slots || !q || !k || !v || !gate || !o) return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  const qdr::PoolView view = qdr::pool_view(pool);
  if (view.gate != QDR_GATE_SCALAR || !view.all_fp32)
    return fail(QDR_E_UNSUPPORTED, "the additive step needs an uncompressed pool (every head FP32) with QDR_GATE_SCALAR");
  QDR_TRY(check_device(view.device));
  QDR_TRY(check_groups((int64_t)B * view.num_heads * 2));
  hipStream_t st = static_cast<hipStream_t>(stream);
  QDR_TRY(qdr::pool_check_slots(pool, slots, B, st));
  qdr::LinearArgs a{};
  a.slots = slots;
  a.B = B;
  a.H = view.num_heads;
  a.num_slots = view.num_slots;
  a.q = q;
  a.k = k;
  a.v = v;
  a.gate = gate;
  a.o = o;
  a.pool = view.base;
  a.slot_stride = view.slot_stride;
  a.err = view.err;
  hipError_t e = qdr::pool_after_writeback(pool, st);
  if (e == hipSuccess) e = qdr::launch_linear_step(a, bf16, st);
  return launched(e);
}

qdr_status qdr_linear_step(qdr_pool *pool, const int32_t *slots, int32_t B, const float *q, const float *k,
                           const float *v, const float *gate, float *o, void *stream) {
  return linear_step(pool, slots, B, q, k, v, gate, o, stream, false);
}

qdr_status qdr_linear_step_bf16(qdr_pool *pool, const int32_t *slots, int32_t B, const uint16_t *q,
                                const uint16_t *k, const uint16_t *v, const float *gate, uint16_t *o, void *stream) {
  return linear_step(pool, slots, B, q, k, v, gate, o, stream, true);
}

qdr_status qdr_kv_bytes(const qdr_kv_desc *desc, size_t *bytes) {
  size_t need = 0;
  int shift = 0;
  QDR_TRY(check_kv_desc(desc, &need, &shift));
  if (!bytes) return fail(QDR_E_INVAL, "bytes is NULL");
  *bytes = need;
  return qdr::set_ok();
}

qdr_status qdr_kv_create(const qdr_kv_desc *desc, void *dev_mem, size_t dev_bytes, qdr_kv **out) {
  size_t need = 0;
  int shift = 0;
  QDR_TRY(check_kv_desc(desc, &need, &shift));
  if (!out) return fail(QDR_E_INVAL, "out is NULL");
  *out = nullptr;
  if (dev_mem && dev_bytes < need) return fail(QDR_E_NOMEM, "dev_mem holds %zu bytes, the cache needs %zu", dev_bytes, need);
  if (dev_mem && reinterpret_cast<uintptr_t>(dev_mem) % 256) return fail(QDR_E_INVAL, "dev_mem must be 256-byte aligned");
  qdr_kv *kv = new (std::nothrow) qdr_kv();
  if (!kv) return fail(QDR_E_NOMEM, "host allocation failed");
  kv->desc = *desc;
  kv->page_shift = shift;
  if (hipGetDevice(&kv->device) != hipSuccess) {
    free_kv(kv);
    return fail(QDR_E_DEVICE, "no HIP device");
  }
  if (dev_mem) {
    kv->base = static_cast<uint8_t *>(dev_mem);
  } else if (hipMalloc(reinterpret_cast<void **>(&kv->base), need) == hipSuccess) {
    kv->owns_base = true;
  } else {
    (void)hipGetLastError();
    kv->base = nullptr;
    free_kv(kv);
    return fail(QDR_E_NOMEM, "hipMalloc of %zu bytes failed", need);
  }
  hipError_t e = hipMalloc(reinterpret_cast<void **>(&kv->d_err), sizeof(uint32_t));
  if (e == hipSuccess) e = hipMemset(kv->d_err, 0, sizeof(uint32_t));
  if (e == hipSuccess) e = hipMemset(kv->base, 0, need);
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) {
    (void)hipGetLastError();
    free_kv(kv);
    return fail(e == hipErrorOutOfMemory ? QDR_E_NOMEM : QDR_E_DEVICE, "cache setup failed: %s", hipGetErrorString(e));
  }
  *out = kv;
  return qdr::set_ok();
}

qdr_status qdr_kv_destroy(qdr_kv *kv) {
  if (!kv) return qdr::set_ok();
  const int own = kv->device;
  int now = own;
  (void)hipGetDevice(&now);
  if (now != own) (void)hipSetDevice(own);
  (void)hipDeviceSynchronize();
  free_kv(kv);
  if (now != own) (void)hipSetDevice(now);
  return qdr::set_ok();
}

static qdr_status kv_move(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                          const int32_t *context, int32_t n, int32_t T, uint16_t *k, uint16_t *v, void *stream,
                          bool write) {
  QDR_TRY(check_kv_call(kv, pages, max_pages, cu, context, n, T, k, v));
  if (n == 0 || T == 0) return qdr::set_ok();
  QDR_TRY(check_groups((T / qdr::kBlock + 2 * (int64_t)n) * kv->desc.num_heads));
  qdr::KvArgs a = kv_args(kv, pages, max_pages, cu, context, n, T);
  a.k = k;
  a.v = v;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launched(write ? qdr::launch_kv_write(a, kv->desc.kind, st) : qdr::launch_kv_read(a, kv->desc.kind, st));
}

qdr_status qdr_kv_write(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                        const int32_t *context, int32_t n, int32_t T, const uint16_t *k, const uint16_t *v,
                        void *stream) {
  return kv_move(kv, pages, max_pages, cu, context, n, T, const_cast<uint16_t *>(k), const_cast<uint16_t *>(v), stream, true);
}

qdr_status qdr_kv_read(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                       const int32_t *context, int32_t n, int32_t T, uint16_t *k, uint16_t *v, void *stream) {
  return kv_move(kv, pages, max_pages, cu, context, n, T, k, v, stream, false);
}

static qdr_status check_heads(const qdr_kv *kv, int32_t q_heads) {
  if (q_heads <= 0 || q_heads % kv->desc.num_heads)
    return fail(QDR_E_INVAL, "q_heads must be a positive multiple of the cache's %d heads (got %d)", kv->desc.num_heads, q_heads);
  return QDR_OK;
}

// The plan of a call, and whether its launches and partial results can be counted.
static qdr_status make_plan(const qdr_kv *kv, int32_t n, int32_t T, int32_t q_heads, int32_t max_pages, qdr::AttendPlan *plan) {
  const int64_t heads = kv->desc.num_heads;
  // heads, sequences and with them tiles fit 32 bits; each is a part of the counts below
  QDR_TRY(check_groups(q_heads));
  QDR_TRY(check_groups(n));
  *plan = qdr::plan_attend(n, T, q_heads, kv->desc.num_heads, max_pages, kv->page_shift);
  const int64_t few = (int64_t)plan->few_tiles * heads * plan->few_parts, many = (int64_t)plan->many_tiles * heads * plan->many_parts;
  // of 512 threads a few-row tile and piece, and four workgroups to join its pieces
  QDR_TRY(check_groups(std::max(few * 2 * plan->few_splits, plan->few_splits > 1 ? few * 4 : 0)));
  return check_groups(many * std::max(plan->many_splits, plan->many_splits > 4 ? 32 : plan->many_splits > 1 ? 4 : 1));
}

qdr_status qdr_kv_attend_workspace(const qdr_kv *kv, int32_t n, int32_t T, int32_t q_heads, int32_t max_pages, size_t *bytes) {
  if (!kv || !bytes) return fail(QDR_E_INVAL, "kv or bytes is NULL");
  QDR_TRY(check_counts(n, T));
  QDR_TRY(check_heads(kv, q_heads));
  if (max_pages < 0) return fail(QDR_E_INVAL, "max_pages must be >= 0 (got %d)", max_pages);
  *bytes = 0;
  if (n == 0 || T == 0) return qdr::set_ok();
  qdr::AttendPlan plan;
  QDR_TRY(make_plan(kv, n, T, q_heads, max_pages, &plan));
  *bytes = (plan.few_floats + plan.many_floats) * sizeof(float);
  return qdr::set_ok();
}

qdr_status qdr_kv_attend(qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                         const int32_t *context, int32_t n, int32_t T, int32_t q_heads, const uint16_t *q,
                         float scale, uint16_t *o, void *workspace, size_t workspace_bytes, void *stream) {
  QDR_TRY(check_kv_call(kv, pages, max_pages, cu, context, n, T, q, o));
  QDR_TRY(check_heads(kv, q_heads));
  if (!std::isfinite(scale)) return fail(QDR_E_INVAL, "scale must be finite");
  if (n == 0 || T == 0) return qdr::set_ok();
  qdr::AttendPlan plan;
  QDR_TRY(make_plan(kv, n, T, q_heads, max_pages, &plan));
  QDR_TRY(check_workspace(workspace, workspace_bytes, (plan.few_floats + plan.many_floats) * sizeof(float)));
  const float scale_log2 = (float)((double)scale * 1.4426950408889634);
  if (!std::isfinite(scale_log2)) return fail(QDR_E_INVAL, "scale is too large (%g)", (double)scale);
  qdr::AttendArgs a{};
  a.kv = kv_args(kv, pages, max_pages, cu, context, n, T);
  a.q = q;
  a.o = o;
  a.q_heads = q_heads;
  a.scale_log2 = scale_log2;
  a.part = static_cast<float *>(workspace);
  return launched(qdr::launch_attend(a, plan, kv->desc.kind, static_cast<hipStream_t>(stream)));
}

qdr_status qdr_kv_poll_device_error(qdr_kv *kv, uint32_t *flags) {
  if (!kv || !flags) return fail(QDR_E_INVAL, "kv or flags is NULL");
  QDR_TRY(check_device(kv->device));
  hipError_t e = hipDeviceSynchronize();
  if (e == hipSuccess) e = hipMemcpy(flags, kv->d_err, sizeof(uint32_t), hipMemcpyDeviceToHost);
  if (e == hipSuccess) e = hipMemset(kv->d_err, 0, sizeof(uint32_t));
  if (e == hipSuccess) e = hipDeviceSynchronize();
  if (e != hipSuccess) return fail(QDR_E_DEVICE, "poll_device_error: %s", hipGetErrorString(e));
  return qdr::set_ok();
}

}  // extern "C"
