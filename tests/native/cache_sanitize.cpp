// cache_sanitize.cpp -- drives the host side of what is done around the paged
// cache (quantized_delta_rule_decode_amd/csrc/qdr_cache.cpp) without a device:
// every refusal of every entry point, workspaces, the rotation's constants, and
// how calls are cut up.  Built with g++ under AddressSanitizer / UBSan by
// tests/test_cache_abi.py; the HIP runtime, the pool and the kernel launches are
// replaced by the stubs below, which count what reaches them.
//
// Prints "ok <n>" (n = checks passed) and exits 0; a failed check exits 1.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

#include "../../include/qdr_cache.h"
#include "../../quantized_delta_rule_decode_amd/csrc/qdr_cache.h"
#include "../../quantized_delta_rule_decode_amd/csrc/qdr_calls.h"

static int device = 0, launches = 0;
static bool no_memory = false;
extern "C" {
hipError_t hipGetDevice(int *d) { *d = device; return hipSuccess; }
hipError_t hipSetDevice(int d) { device = d; return hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
const char *hipGetErrorString(hipError_t) { return "stub"; }
hipError_t hipMalloc(void **p, size_t n) {
  if (no_memory) return hipErrorOutOfMemory;
  *p = std::malloc(n);
  return hipSuccess;
}
hipError_t hipFree(void *p) { std::free(p); return hipSuccess; }
hipError_t hipMemcpy(void *d, const void *s, size_t n, hipMemcpyKind) { std::memcpy(d, s, n); return hipSuccess; }
hipError_t hipDeviceSynchronize(void) { return hipSuccess; }
}

static std::string message;
static qdr::PoolView view;
static qdr::RotateArgs rotated;
static qdr::RotaryWriteArgs written;
static qdr::CopyArgs copied;
static qdr::AssignArgs assigned;
static qdr::CompactArgs compacted;
static qdr::SharedArgs shared_args;
static qdr::SharedPlan shared_plan;
struct qdr_pool { int unused; };
namespace qdr {
PoolView pool_view(const qdr_pool *) { return view; }
qdr_status set_error(qdr_status st, const char *m) { message = m; return st; }
qdr_status set_ok() { message.clear(); return QDR_OK; }
hipError_t pool_after_writeback(qdr_pool *, hipStream_t) { return hipSuccess; }
hipError_t launch_rotate(const RotateArgs &a, bool, hipStream_t) { rotated = a; ++launches; return hipSuccess; }
hipError_t launch_kv_write_rotary(const RotaryWriteArgs &a, int, hipStream_t) { written = a; ++launches; return hipSuccess; }
hipError_t launch_copy(const CopyArgs &a, hipStream_t) { copied = a; ++launches; return hipSuccess; }
hipError_t launch_assign(const AssignArgs &a, hipStream_t) { assigned = a; ++launches; return hipSuccess; }
hipError_t launch_compact(const CompactArgs &a, hipStream_t) { compacted = a; ++launches; return hipSuccess; }
hipError_t launch_attend_shared(const SharedArgs &a, const SharedPlan &p, int, hipStream_t) {
  shared_args = a;
  shared_plan = p;
  ++launches;
  return hipSuccess;
}
}  // namespace qdr

static int checks = 0;
#define CHECK(x)                                                                                   \
  do {                                                                                             \
    if (!(x)) {                                                                                    \
      std::fprintf(stderr, "check failed at line %d: %s (%s)\n", __LINE__, #x, message.c_str());   \
      return 1;                                                                                    \
    }                                                                                              \
    ++checks;                                                                                      \
  } while (0)
// refused with `status`, a message, and nothing enqueued
#define REFUSED(x, status)                                                       \
  do {                                                                           \
    const int before_ = launches;                                                \
    message.clear();                                                             \
    CHECK((x) == (status) && launches == before_ && !message.empty());           \
  } while (0)

alignas(256) static char mem[1 << 16];
static uint16_t *x = (uint16_t *)mem, *odd = (uint16_t *)(mem + 2);
static float *f = (float *)mem;
static int32_t *i = (int32_t *)mem;

static int rotary() {
  double freq[64], amp = 0;
  CHECK(qdr_rotary_frequencies(QDR_ROTARY_PLAIN, 128, 10000, NAN, NAN, NAN, NAN, freq, &amp) == QDR_OK && amp == 1);
  CHECK(freq[0] == 1 && std::fabs(freq[32] - 0.01) < 1e-17);
  CHECK(qdr_rotary_frequencies(QDR_ROTARY_LINEAR, 16, 100, 4, 0, 0, 0, freq, &amp) == QDR_OK && freq[0] == 0.25);
  CHECK(qdr_rotary_frequencies(QDR_ROTARY_TURNS, 128, 10000, 8, 8192, 1, 4, freq, &amp) == QDR_OK && amp == 1);
  CHECK(freq[0] == 1 && std::fabs(freq[63] * 8 / std::pow(10000, -126. / 128) - 1) < 1e-14);
  CHECK(qdr_rotary_frequencies(QDR_ROTARY_INDEX, 128, 10000, 8, 8192, 1, 32, freq, &amp) == QDR_OK && std::fabs(amp - 1.2079441541679836) < 1e-15);
  CHECK(freq[0] == 1 && std::fabs(freq[63] * 8 / std::pow(10000, -126. / 128) - 1) < 1e-14);
  const double bad_base[] = {1, 0, -5, NAN, INFINITY}, bad_factor[] = {0.5, -1, NAN, INFINITY}, bad_context[] = {0, -1, NAN, INFINITY};
  for (double b : bad_base) REFUSED(qdr_rotary_frequencies(0, 64, b, 1, 1, 1, 2, freq, &amp), QDR_E_INVAL);
  for (double b : bad_factor) REFUSED(qdr_rotary_frequencies(1, 64, 10, b, 1, 1, 2, freq, &amp), QDR_E_INVAL);
  for (double b : bad_context) REFUSED(qdr_rotary_frequencies(2, 64, 10, 2, b, 1, 2, freq, &amp), QDR_E_INVAL);
  REFUSED(qdr_rotary_frequencies(2, 64, 10, 2, 9, 2, 2, freq, &amp), QDR_E_INVAL);
  REFUSED(qdr_rotary_frequencies(3, 64, 10, 2, 9, 0, 2, freq, &amp), QDR_E_INVAL);
  REFUSED(qdr_rotary_frequencies(3, 64, 10, 2, 9, 1, INFINITY, freq, &amp), QDR_E_INVAL);
  REFUSED(qdr_rotary_frequencies(4, 64, 10, 2, 9, 1, 2, freq, &amp), QDR_E_INVAL);
  REFUSED(qdr_rotary_frequencies(-1, 64, 10, 2, 9, 1, 2, freq, &amp), QDR_E_INVAL);
  REFUSED(qdr_rotary_frequencies(0, 64, 10, 2, 9, 1, 2, nullptr, &amp), QDR_E_INVAL);
  REFUSED(qdr_rotary_frequencies(0, 64, 10, 2, 9, 1, 2, freq, nullptr), QDR_E_INVAL);
  const int bad_channels[] = {0, -16, 8, 24, 144, 130};
  for (int c : bad_channels) REFUSED(qdr_rotary_frequencies(0, c, 10, 2, 9, 1, 2, freq, &amp), QDR_E_INVAL);

  // turns a token in units of 2^-64: 0, a half, 1 - 2^-40, -1/4, whole turns
  const double pi = 3.14159265358979323846;
  double turns[8] = {0, pi, -pi / 2, 2 * pi, 1048576, 1e-300, -1e-30, 2 * pi * 0.75};
  qdr_rotary_desc d{128, 16, QDR_ROTARY_PAIRS, turns, -2.5};
  qdr_rotary *r = nullptr;
  CHECK(qdr_rotary_create(&d, &r) == QDR_OK && r);
  qdr_rotary *const good = r;
  CHECK(qdr_rotate(r, i, 1, 1, f, 128, f, 128, nullptr) == QDR_OK && rotated.rotary.amplitude == -2.5f && rotated.rotary.channels == 16);
  const uint64_t *t = rotated.rotary.turns;
  const auto near = [](uint64_t a, uint64_t b, uint64_t by) { return a - b + by <= 2 * by; };
  CHECK(t[0] == 0 && near(t[1], 1ull << 63, 1 << 12) && near(t[2], 3ull << 62, 1 << 12) && near(t[3], 0, 1 << 12));
  // the fraction of 2^20 / (2 pi), in a 64-bit significand
  CHECK(near(t[4], 988884335487086749ull, 1ull << 18) && t[5] == 0 && near(t[6], 0, 1) && near(t[7], 3ull << 62, 1 << 12));
  for (int c : bad_channels) {
    d.channels = c;
    REFUSED(qdr_rotary_create(&d, &r), QDR_E_INVAL);
  }
  d.channels = 16;
  for (double b : {(double)NAN, (double)INFINITY, -1048577.0}) {
    turns[3] = b;
    REFUSED(qdr_rotary_create(&d, &r), QDR_E_INVAL);
  }
  turns[3] = 1;
  for (double b : {(double)NAN, (double)INFINITY, 1e39}) {
    d.amplitude = b;
    REFUSED(qdr_rotary_create(&d, &r), QDR_E_INVAL);
  }
  d.amplitude = 1;
  d.d = 64;
  REFUSED(qdr_rotary_create(&d, &r), QDR_E_UNSUPPORTED);
  d.d = 128;
  d.layout = 2;
  REFUSED(qdr_rotary_create(&d, &r), QDR_E_INVAL);
  d.layout = 0;
  REFUSED(qdr_rotary_create(&d, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotary_create(nullptr, &r), QDR_E_INVAL);
  d.freq = nullptr;
  REFUSED(qdr_rotary_create(&d, &r), QDR_E_INVAL);
  d.freq = turns;
  no_memory = true;
  REFUSED(qdr_rotary_create(&d, &r), QDR_E_NOMEM);
  no_memory = false;
  CHECK(r == nullptr);
  r = good;

  // rows of a workgroup
  struct { int T, heads, tokens, parts; } cuts[] = {{1, 1, 32, 1}, {5, 8, 16, 1}, {9, 32, 4, 1}, {9, 100, 1, 1}, {9, 129, 1, 2}, {9, 1 << 17, 1, 1024}};
  for (const auto &c : cuts) {
    CHECK(qdr_rotate(r, i, c.T, c.heads, f, c.heads * 128, f, c.heads * 128, nullptr) == QDR_OK);
    CHECK(rotated.tokens == c.tokens && rotated.head_parts == c.parts && rotated.head_parts * rotated.part_heads >= c.heads && rotated.tokens <= 32);
  }
  CHECK(qdr_rotate_bf16(r, i, 3, 2, x, 258, x, 256, nullptr) == QDR_OK && rotated.x_stride == 258);
  CHECK(qdr_rotate(r, i, 3, 2, f, 257, f, 256, nullptr) == QDR_OK);
  CHECK(qdr_rotate(r, nullptr, 0, 2, nullptr, 256, nullptr, 256, nullptr) == QDR_OK);
  REFUSED(qdr_rotate(nullptr, i, 3, 2, f, 256, f, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, -1, 2, f, 256, f, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, 3, 0, f, 256, f, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, 3, (1 << 17) + 1, f, 1 << 30, f, 1 << 30, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, 3, 2, f, 255, f, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, 3, 2, f, 256, f, -256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, 3, 2, f, 256, f, (1 << 30) + 1, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate_bf16(r, i, 3, 2, x, 257, x, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate_bf16(r, i, 3, 2, x, 256, x, 257, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate_bf16(r, i, 3, 2, odd, 256, x, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate_bf16(r, i, 3, 2, x, 256, odd, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, nullptr, 3, 2, f, 256, f, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, 3, 2, nullptr, 256, f, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, 3, 2, f, 256, nullptr, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_rotate(r, i, 1 << 30, 300, f, 300 * 128, f, 300 * 128, nullptr), QDR_E_INVAL);   // launch too large
  device = 1;
  REFUSED(qdr_rotate(r, i, 3, 2, f, 256, f, 256, nullptr), QDR_E_INVAL);
  device = 0;

  qdr_kv kv;
  kv.desc = {3, 64, 2, 128, QDR_KV_INT8};
  kv.page_shift = 6;
  kv.base = (uint8_t *)mem;
  auto write = [&](const uint16_t *q, int64_t qs, int heads, uint16_t *out, const uint16_t *k, int64_t ks, const uint16_t *v, int64_t vs, int n = 2, int T = 5) {
    return qdr_kv_write_rotary(&kv, r, i, 3, i, i, n, T, q, qs, heads, out, k, ks, v, vs, nullptr);
  };
  CHECK(write(x, 512, 4, x, x, 256, x, 300) == QDR_OK && written.kv_heads == 1 && written.kv_parts == 2 && written.query_parts == 1);
  CHECK(write(x, 40 * 128, 40, x, x, 256, x, 300, 1, 5000) == QDR_OK && written.kv_heads == 4 && written.kv_parts == 1 && written.query_parts == 5);
  CHECK(write(nullptr, 0, 0, nullptr, x, 256, x, 256) == QDR_OK && written.query_parts == 0);
  CHECK(write(x, 512, 4, x, nullptr, 256, nullptr, 300, 0, 5) == QDR_OK && write(x, 512, 4, x, nullptr, 256, nullptr, 300, 5, 0) == QDR_OK);
  REFUSED(qdr_kv_write_rotary(nullptr, r, i, 3, i, i, 2, 5, x, 512, 4, x, x, 256, x, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_write_rotary(&kv, nullptr, i, 3, i, i, 2, 5, x, 512, 4, x, x, 256, x, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_write_rotary(&kv, r, nullptr, 3, i, i, 2, 5, x, 512, 4, x, x, 256, x, 256, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_write_rotary(&kv, r, i, -1, i, i, 2, 5, x, 512, 4, x, x, 256, x, 256, nullptr), QDR_E_INVAL);
  REFUSED(write(x, 511, 4, x, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 510, 4, x, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 513, 4, x, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 512, 4, x, x, 254, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 512, 4, x, x, 256, x, 257), QDR_E_INVAL);
  REFUSED(write(x, 512, -1, x, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 1 << 30, (1 << 17) + 1, x, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(nullptr, 512, 4, x, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 512, 4, nullptr, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(odd, 512, 4, x, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 512, 4, odd, x, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 512, 4, x, odd, 256, x, 256), QDR_E_INVAL);
  REFUSED(write(x, 512, 4, x, x, 256, nullptr, 256), QDR_E_INVAL);
  REFUSED(write(x, 512, 4, x, x, 256, x, 256, 1 << 22, 5), QDR_E_INVAL);       // launch too large
  REFUSED(write(x, 512, 4, x, x, 256, x, 256, 1, 1 << 30), QDR_E_INVAL);
  kv.device = 1;
  REFUSED(write(x, 512, 4, x, x, 256, x, 256), QDR_E_INVAL);
  device = 1;
  REFUSED(write(x, 512, 4, x, x, 256, x, 256), QDR_E_INVAL);
  device = 0;
  CHECK(qdr_rotary_destroy(r) == QDR_OK && qdr_rotary_destroy(nullptr) == QDR_OK);
  return 0;
}

static int pages() {
  qdr_kv kv, other;
  kv.desc = {300, 64, 2, 128, QDR_KV_BF16};
  kv.page_shift = 6;
  kv.base = (uint8_t *)mem;
  other = kv;
  other.desc.num_pages = 7;
  CHECK(qdr_kv_copy(&kv, i, &other, i, 9, nullptr) == QDR_OK && copied.bytes == 2u * 2 * 16384 && copied.parts == 2 && copied.num_to == 7);
  CHECK(qdr_kv_copy(&kv, nullptr, &kv, nullptr, 0, nullptr) == QDR_OK);
  REFUSED(qdr_kv_copy(nullptr, i, &kv, i, 1, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_copy(&kv, i, nullptr, i, 1, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_copy(&kv, nullptr, &kv, i, 1, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_copy(&kv, i, &kv, nullptr, 1, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_copy(&kv, i, &kv, i, -1, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_copy(&kv, i, &kv, i, 1 << 23, nullptr), QDR_E_INVAL);         // launch too large
  other.desc.page_tokens = 32;
  REFUSED(qdr_kv_copy(&kv, i, &other, i, 1, nullptr), QDR_E_INVAL);
  other.desc = kv.desc;
  other.desc.kind = QDR_KV_INT8;
  REFUSED(qdr_kv_copy(&kv, i, &other, i, 1, nullptr), QDR_E_INVAL);
  other.desc = kv.desc;
  other.desc.num_heads = 1;
  REFUSED(qdr_kv_copy(&kv, i, &other, i, 1, nullptr), QDR_E_INVAL);
  other.desc = kv.desc;
  other.device = 1;
  REFUSED(qdr_kv_copy(&kv, i, &other, i, 1, nullptr), QDR_E_INVAL);
  device = 1;
  REFUSED(qdr_kv_copy(&kv, i, &kv, i, 1, nullptr), QDR_E_INVAL);
  device = 0;

  qdr_pool pool{};
  view = {};
  view.num_slots = 4;
  view.num_heads = 2;
  view.slot_stride = 66048;
  CHECK(qdr_slot_copy(&pool, i, i, 3, nullptr) == QDR_OK && copied.parts == 3 && copied.bytes == 66048 && copied.bit == QDR_DEVERR_SLOT);
  CHECK(qdr_slot_copy(&pool, nullptr, nullptr, 0, nullptr) == QDR_OK);
  REFUSED(qdr_slot_copy(nullptr, i, i, 3, nullptr), QDR_E_INVAL);
  REFUSED(qdr_slot_copy(&pool, nullptr, i, 3, nullptr), QDR_E_INVAL);
  REFUSED(qdr_slot_copy(&pool, i, nullptr, 3, nullptr), QDR_E_INVAL);
  REFUSED(qdr_slot_copy(&pool, i, i, -3, nullptr), QDR_E_INVAL);
  REFUSED(qdr_slot_copy(&pool, i, i, 1 << 23, nullptr), QDR_E_INVAL);
  device = 1;
  REFUSED(qdr_slot_copy(&pool, i, i, 3, nullptr), QDR_E_INVAL);
  device = 0;

  // arrays of their own: old tables of 3 x 5, new ones of 4 x 5
  static int32_t table[15], context[3], parent[4], add[4], refs[300], nt[20], nc[4], nr[300], moved[300];
  size_t need = 1;
  CHECK(qdr_kv_assign_workspace(&kv, 4, &need) == QDR_OK && need == 3 * 1280 + 256 + 256);
  CHECK(qdr_kv_assign_workspace(&kv, 0, &need) == QDR_OK && need == 3 * 1280 + 256);
  REFUSED(qdr_kv_assign_workspace(nullptr, 4, &need), QDR_E_INVAL);
  REFUSED(qdr_kv_assign_workspace(&kv, 4, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_assign_workspace(&kv, -1, &need), QDR_E_INVAL);
  CHECK(qdr_kv_assign_workspace(&kv, 4, &need) == QDR_OK);
  auto assign = [&](int32_t *t, int32_t *c, int n, int most, int32_t *p, int32_t *a, int m, int32_t *r, int32_t *nt_, int32_t *nc_, int32_t *nr_, void *ws = mem,
                    size_t bytes = sizeof mem) { return qdr_kv_assign(&kv, t, c, n, most, p, a, m, r, nt_, nc_, nr_, ws, bytes, nullptr); };
  CHECK(assign(table, context, 3, 5, parent, add, 4, refs, nt, nc, nr, mem, need) == QDR_OK && assigned.parts == 2);
  CHECK((char *)assigned.hold == mem && (char *)assigned.first == mem + 1280 && (char *)assigned.free == mem + 2560 && (char *)assigned.counts == mem + 3840 && (char *)assigned.offset == mem + 4096);
  CHECK(assign(nullptr, nullptr, 0, 5, parent, add, 4, refs, nt, nc, nr) == QDR_OK && assign(table, context, 3, 5, nullptr, nullptr, 0, refs, nullptr, nullptr, nr) == QDR_OK);
  CHECK(assign(nullptr, context, 3, 0, parent, add, 4, refs, nullptr, nc, nr) == QDR_OK);
  REFUSED(qdr_kv_assign(nullptr, table, context, 3, 5, parent, add, 4, refs, nt, nc, nr, mem, need, nullptr), QDR_E_INVAL);
  REFUSED(assign(nullptr, context, 3, 5, parent, add, 4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, nullptr, 3, 5, parent, add, 4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, nullptr, add, 4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, nullptr, 4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, nullptr, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nullptr, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, nullptr, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, nc, nullptr), QDR_E_INVAL);
  REFUSED(assign(table, context, -3, 5, parent, add, 4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, -5, parent, add, 4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, -4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, table, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, table + 14, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, context, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, nc, refs), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nr + 299, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, nc, nr, nullptr, need), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, nc, nr, mem + 4, need), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, nc, nr, mem, need - 1), QDR_E_NOMEM);
  const uintptr_t far = (uintptr_t)1 << 44;      // (sizes that are refused before anything is read)
  REFUSED(assign((int32_t *)far, (int32_t *)(2 * far), 1 << 24, 5, parent, add, 4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign((int32_t *)far, (int32_t *)(2 * far), 1 << 30, INT32_MAX, parent, add, 4, refs, nt, nc, nr), QDR_E_INVAL);
  REFUSED(assign(table, context, 3, 5, (int32_t *)far, (int32_t *)(2 * far), 1 << 23, refs, (int32_t *)(3 * far), (int32_t *)(4 * far), nr, (void *)(5 * far), (size_t)1 << 40), QDR_E_INVAL);
  device = 1;
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, nc, nr), QDR_E_INVAL);
  device = 0;

  CHECK(qdr_kv_compact_workspace(&kv, &need) == QDR_OK && need == 2 * 1280 + 512);
  REFUSED(qdr_kv_compact_workspace(nullptr, &need), QDR_E_INVAL);
  REFUSED(qdr_kv_compact_workspace(&kv, nullptr), QDR_E_INVAL);
  auto compact = [&](int32_t *r, int32_t *t, int n, int most, int32_t *mv, int32_t *nr_, int32_t *nt_, void *ws = mem, size_t bytes = sizeof mem) {
    return qdr_kv_compact(&kv, r, t, n, most, mv, nr_, nt_, ws, bytes, nullptr);
  };
  CHECK(compact(refs, table, 3, 5, moved, nr, nt, mem, need) == QDR_OK && compacted.groups == 300 && compacted.entries == 15);
  CHECK((char *)compacted.dst == mem + 1280 && (char *)compacted.counts == mem + 2560 && (char *)compacted.moves == mem + 2816);
  CHECK(compact(refs, nullptr, 0, 5, moved, nr, nullptr) == QDR_OK);
  REFUSED(qdr_kv_compact(nullptr, refs, table, 3, 5, moved, nr, nt, mem, need, nullptr), QDR_E_INVAL);
  REFUSED(compact(nullptr, table, 3, 5, moved, nr, nt), QDR_E_INVAL);
  REFUSED(compact(refs, nullptr, 3, 5, moved, nr, nt), QDR_E_INVAL);
  REFUSED(compact(refs, table, 3, 5, nullptr, nr, nt), QDR_E_INVAL);
  REFUSED(compact(refs, table, 3, 5, moved, nullptr, nt), QDR_E_INVAL);
  REFUSED(compact(refs, table, 3, 5, moved, nr, nullptr), QDR_E_INVAL);
  REFUSED(compact(refs, table, -3, 5, moved, nr, nt), QDR_E_INVAL);
  REFUSED(compact(refs, table, 3, -5, moved, nr, nt), QDR_E_INVAL);
  REFUSED(compact(refs, table, 3, 5, refs, nr, nt), QDR_E_INVAL);
  REFUSED(compact(refs, table, 3, 5, moved, moved, nt), QDR_E_INVAL);
  REFUSED(compact(refs, table, 3, 5, moved, nr, table), QDR_E_INVAL);
  REFUSED(compact(refs, table, 3, 5, moved, nr, nt, mem, need - 1), QDR_E_NOMEM);
  REFUSED(compact(refs, (int32_t *)far, 1 << 30, 1 << 10, moved, nr, (int32_t *)(8 * far)), QDR_E_INVAL);
  device = 1;
  REFUSED(compact(refs, table, 3, 5, moved, nr, nt), QDR_E_INVAL);
  device = 0;
  kv.desc.num_pages = (1 << 26) + 1;
  REFUSED(qdr_kv_assign_workspace(&kv, 4, &need), QDR_E_UNSUPPORTED);
  REFUSED(assign(table, context, 3, 5, parent, add, 4, refs, nt, nc, nr), QDR_E_UNSUPPORTED);
  REFUSED(qdr_kv_compact_workspace(&kv, &need), QDR_E_UNSUPPORTED);
  REFUSED(compact(refs, table, 3, 5, moved, nr, nt), QDR_E_UNSUPPORTED);
  return 0;
}

static int attend() {
  qdr_kv kv;
  kv.desc = {300, 64, 2, 128, QDR_KV_BF16};
  kv.page_shift = 6;
  kv.base = (uint8_t *)mem;
  size_t need = 1;
  auto call = [&](const int32_t *gcu, const int32_t *shared, int groups, int heads, const uint16_t *q, float scale, uint16_t *o, void *ws, size_t bytes, int n = 2, int T = 5,
                  int most = 9) { return qdr_kv_attend_shared(&kv, i, most, i, i, n, T, gcu, shared, groups, heads, q, scale, o, ws, bytes, nullptr); };
  // what the device's partial results take, whatever the counts
  const int ns[] = {1, 2, 7, 64, 500}, Ts[] = {1, 3, 17, 64, 900, 5000}, gs[] = {0, 1, 3, 64}, hs[] = {2, 8, 34, 400}, ms[] = {0, 1, 9, 300, 5000};
  static char space[1];
  for (int n : ns)
    for (int T : Ts)
      for (int g : gs)
        for (int h : hs)
          for (int m : ms) {
            CHECK(qdr_kv_attend_shared_workspace(&kv, n, T, g, h, m, &need) == QDR_OK);
            void *ws = (void *)((uintptr_t)space & ~(uintptr_t)15);
            CHECK(call(i, i, g, h, x, 1.0f, x, ws, need, n, T, m) == QDR_OK);
            const qdr::SharedPlan &p = shared_plan;
            const size_t rows = (size_t)T * h;
            const bool together = g > 0 && n > g && (int64_t)(n - g) * 2 * m * 2 >= qdr::kLeastSaved;
            CHECK((p.ranges >= 1) == together && p.ranges * 2 <= 512 && p.few_splits >= 1 && p.few_splits <= 32 && p.many_splits >= 1 && p.many_splits <= 32);
            CHECK(p.slot_rows == 128 || (p.slot_rows == 16 && T <= p.few_tokens));
            CHECK(p.cut == (together ? 2 * rows * 130 : 0) && p.few_pieces == p.cut + (size_t)p.ranges * 2 * 2 * p.slot_rows * 130 && p.floats == p.info + (size_t)T * p.few_parts * 8);
            CHECK(p.many_pieces == p.few_pieces + (p.few_splits > 1 ? (size_t)n * 2 * p.few_parts * p.few_splits * 16 * 130 : 0));
            CHECK(p.info == p.many_pieces + (p.many_splits > 1 ? (size_t)p.many_tiles * 2 * p.many_parts * p.many_splits * 128 * 130 : 0));
            CHECK((p.many_tiles > 0) == (T > p.few_tokens));
            CHECK(need == p.floats * 4 && p.info % 4 == 0 && shared_args.a.part == ws);
            CHECK(p.few_heads * p.few_parts >= p.group && p.many_heads * p.many_parts >= p.group && p.few_heads * p.few_tokens <= 16 && p.many_heads * p.many_tokens <= 128);
            CHECK(p.many_parts <= p.few_parts && p.many_tokens >= p.few_tokens);
          }
  CHECK(qdr_kv_attend_shared_workspace(&kv, 0, 5, 1, 2, 9, &need) == QDR_OK && need == 0);
  CHECK(call(nullptr, nullptr, 1, 2, x, 1.0f, x, nullptr, 0, 0, 5) == QDR_OK && call(nullptr, nullptr, 1, 2, x, 1.0f, x, nullptr, 0, 5, 0) == QDR_OK);
  CHECK(qdr_kv_attend_shared_workspace(&kv, 2, 5, 1, 4, 9, &need) == QDR_OK && need > 0);
  CHECK(call(i, i, 1, 4, x, 1.0f, x, mem, need) == QDR_OK && call(nullptr, nullptr, 0, 4, x, 1.0f, x, mem, need) == QDR_OK);
  REFUSED(qdr_kv_attend_shared_workspace(nullptr, 2, 5, 1, 4, 9, &need), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_shared_workspace(&kv, 2, 5, 1, 4, 9, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_shared_workspace(&kv, 2, 5, -1, 4, 9, &need), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_shared_workspace(&kv, 2, 5, 1, 4, -9, &need), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_shared_workspace(&kv, 2, 5, 1, 3, 9, &need), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_shared_workspace(&kv, 2, 1 << 27, 1, 2, 9, &need), QDR_E_INVAL);      // launch too large
  REFUSED(qdr_kv_attend_shared_workspace(&kv, 1 << 24, 5, 1, 2, 9, &need), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_shared_workspace(&kv, 2, 5, 1 << 24, 2, 9, &need), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_shared_workspace(&kv, 2, 5, 1, 1 << 25, 9, &need), QDR_E_INVAL);
  CHECK(qdr_kv_attend_shared_workspace(&kv, 2, 5, 1, 4, 9, &need) == QDR_OK);
  REFUSED(qdr_kv_attend_shared(nullptr, i, 9, i, i, 2, 5, i, i, 1, 4, x, 1.0f, x, mem, need, nullptr), QDR_E_INVAL);
  REFUSED(call(nullptr, i, 1, 4, x, 1.0f, x, mem, need), QDR_E_INVAL);
  REFUSED(call(i, nullptr, 1, 4, x, 1.0f, x, mem, need), QDR_E_INVAL);
  REFUSED(call(i, i, -1, 4, x, 1.0f, x, mem, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 3, x, 1.0f, x, mem, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 0, x, 1.0f, x, mem, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 4, nullptr, 1.0f, x, mem, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 4, x, 1.0f, odd, mem, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 4, x, NAN, x, mem, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 4, x, 3e38f, x, mem, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 4, x, 1.0f, x, nullptr, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 4, x, 1.0f, x, mem + 8, need), QDR_E_INVAL);
  REFUSED(call(i, i, 1, 4, x, 1.0f, x, mem, need - 1), QDR_E_NOMEM);
  device = 1;
  REFUSED(call(i, i, 1, 4, x, 1.0f, x, mem, need), QDR_E_INVAL);
  device = 0;
  return 0;
}

int main() {
  if (rotary() || pages() || attend()) return 1;
  std::printf("ok %d\n", checks);
  return 0;
}
