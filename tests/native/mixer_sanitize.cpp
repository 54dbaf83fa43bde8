// mixer_sanitize.cpp -- drives the host side of the token mixers
// (quantized_delta_rule_decode_amd/csrc/qdr_mixer.cpp) without a device: every
// refusal of every entry point, the workspace sizes, and how an attention
// call is cut up.  Built with g++ under AddressSanitizer / UBSan by
// tests/test_mixer_abi.py; the HIP runtime, the pool and the kernel launches
// are replaced by the stubs below, which count what reaches them.
//
// Prints "ok <n>" (n = checks passed) and exits 0; a failed check exits 1.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

#include "../../include/qdr_mixer.h"
#include "../../quantized_delta_rule_decode_amd/csrc/qdr_host.h"
#include "../../quantized_delta_rule_decode_amd/csrc/qdr_mixer.h"

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
hipError_t hipMemset(void *p, int v, size_t n) { std::memset(p, v, n); return hipSuccess; }
hipError_t hipMemcpy(void *d, const void *s, size_t n, hipMemcpyKind) { std::memcpy(d, s, n); return hipSuccess; }
hipError_t hipDeviceSynchronize(void) { return hipSuccess; }
}

static std::string message;
static qdr::PoolView view;
static qdr::AttendPlan last_plan;
static qdr::PromptArgs last_prompt;
struct qdr_pool { int unused; };
namespace qdr {
PoolView pool_view(const qdr_pool *) { return view; }
qdr_status set_error(qdr_status st, const char *m) { message = m; return st; }
qdr_status set_ok() { message.clear(); return QDR_OK; }
qdr_status pool_check_slots(const qdr_pool *, const int32_t *, int32_t, hipStream_t) { return QDR_OK; }
hipError_t pool_after_writeback(qdr_pool *, hipStream_t) { return hipSuccess; }
qdr_status pool_pack(qdr_pool *, const int32_t *, int32_t, const float *, hipStream_t) { ++launches; return QDR_OK; }
qdr_status pool_unpack(qdr_pool *, const int32_t *, int32_t, float *, hipStream_t) { ++launches; return QDR_OK; }
hipError_t launch_prompt_slots(const PromptArgs &, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_prompt_chunks(const PromptArgs &, bool, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_prompt_scan(const PromptArgs &a, bool, hipStream_t) {
  last_prompt = a;
  ++launches;
  return hipSuccess;
}
hipError_t launch_linear_step(const LinearArgs &, bool, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_kv_write(const KvArgs &, int, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_kv_read(const KvArgs &, int, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_attend(const AttendArgs &, const AttendPlan &p, int, hipStream_t) {
  last_plan = p;
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

static int prompts() {
  alignas(16) static char ws[1 << 16];
  uint16_t *x = (uint16_t *)ws, *odd = (uint16_t *)(ws + 2);
  float *f = (float *)ws;
  int32_t *i = (int32_t *)ws;
  qdr_pool pool{};
  view = {};
  view.num_slots = 4;
  view.num_heads = 2;
  view.all_fp32 = true;
  size_t need = 1;
  CHECK(qdr_prompt_workspace(&pool, 1, 64, &need) == QDR_OK && need == 2 * 2 * (6 * 512 + 256) * 4);
  CHECK(qdr_prompt_workspace(&pool, 0, 64, &need) == QDR_OK && need == 0);
  REFUSED(qdr_prompt_workspace(nullptr, 1, 1, &need), QDR_E_INVAL);
  REFUSED(qdr_prompt_workspace(&pool, 1, 1, nullptr), QDR_E_INVAL);
  REFUSED(qdr_prompt_workspace(&pool, -1, 1, &need), QDR_E_INVAL);
  REFUSED(qdr_prompt_workspace(&pool, 1, -1, &need), QDR_E_INVAL);
  REFUSED(qdr_prompt_workspace(&pool, 1 << 23, 5, &need), QDR_E_INVAL);      // launch too large
  REFUSED(qdr_prompt_workspace(&pool, 1, 1 << 30, &need), QDR_E_INVAL);
  view.num_heads = 1 << 20;
  REFUSED(qdr_prompt_workspace(&pool, 1, 5, &need), QDR_E_UNSUPPORTED);
  view.num_heads = 2;
  auto call = [&](int rule, const int32_t *slots, const int32_t *cu, int n, int T, const uint16_t *q, const float *beta,
                  const float *gate, uint16_t *o, void *w, size_t bytes) {
    return qdr_prompt(&pool, rule, slots, nullptr, cu, n, T, q, x, x, beta, gate, o, w, bytes, nullptr);
  };
  const size_t big = sizeof ws;
  CHECK(qdr_prompt_workspace(&pool, 1, 5, &need) == QDR_OK && need <= big);
  CHECK(call(QDR_RULE_DELTA, i, i, 1, 5, x, f, f, x, ws, need) == QDR_OK);
  CHECK(call(QDR_RULE_SUM, i, i, 1, 5, x, nullptr, f, x, ws, need) == QDR_OK);
  CHECK(call(QDR_RULE_SUM, nullptr, nullptr, 0, 5, x, nullptr, f, x, nullptr, 0) == QDR_OK);   // no sequences: nothing to do
  REFUSED(qdr_prompt(nullptr, 0, i, nullptr, i, 1, 5, x, x, x, f, f, x, ws, need, nullptr), QDR_E_INVAL);
  REFUSED(call(2, i, i, 1, 5, x, f, f, x, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_DELTA, i, i, 1, 5, x, nullptr, f, x, ws, need), QDR_E_INVAL);   // DELTA without beta
  REFUSED(call(QDR_RULE_SUM, nullptr, i, 1, 5, x, f, f, x, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, nullptr, 1, 5, x, f, f, x, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, nullptr, f, f, x, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, x, f, nullptr, x, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, -1, 5, x, f, f, x, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, 1, -5, x, f, f, x, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, odd, f, f, x, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, x, f, f, odd, ws, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, x, f, f, x, nullptr, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, x, f, f, x, ws + 4, need), QDR_E_INVAL);
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, x, f, f, x, ws, need - 1), QDR_E_NOMEM);
  REFUSED(call(QDR_RULE_SUM, i, i, 1 << 23, 5, x, f, f, x, ws, need), QDR_E_INVAL);      // launch too large
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 1 << 30, x, f, f, x, ws, need), QDR_E_INVAL);
  device = 1;
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, x, f, f, x, ws, need), QDR_E_INVAL);
  device = 0;
  view.gate = QDR_GATE_DIAG;
  REFUSED(call(QDR_RULE_SUM, i, i, 1, 5, x, f, f, x, ws, need), QDR_E_UNSUPPORTED);
  view.gate = QDR_GATE_SCALAR;

  // which calls are cut into segments, and that their parts fit the workspace
  struct { int rule, heads, n, T, segment; } cuts[] = {
      {QDR_RULE_DELTA, 2, 1, 1500, 0},   {QDR_RULE_DELTA, 2, 1, 2200, 4},  {QDR_RULE_DELTA, 4, 1, 32768, 8}, {QDR_RULE_DELTA, 32, 1, 32768, 64},
      {QDR_RULE_DELTA, 48, 1, 32768, 0}, {QDR_RULE_DELTA, 32, 1, 2048, 0}, {QDR_RULE_DELTA, 2, 3, 4000, 4},  {QDR_RULE_DELTA, 2, 5, 3000, 0},
      {QDR_RULE_SUM, 2, 1, 256, 0},      {QDR_RULE_SUM, 2, 1, 257, 4},     {QDR_RULE_SUM, 16, 1, 16385, 8},  {QDR_RULE_SUM, 17, 32, 32768, 32}};
  for (const auto &c : cuts) {
    view.num_heads = c.heads;
    CHECK(qdr_prompt_workspace(&pool, c.n, c.T, &need) == QDR_OK);
    char *space = (char *)std::aligned_alloc(256, (need + 255) / 256 * 256);
    CHECK(call(c.rule, i, i, c.n, c.T, x, f, f, x, space, need) == QDR_OK && last_prompt.segment == c.segment);
    const size_t cells = (size_t)last_prompt.segments * c.heads;
    if (c.segment) {
      CHECK(last_prompt.segments == c.T / (64 * c.segment) + c.n && (char *)(last_prompt.segment_ws + cells * 16384) == (char *)last_prompt.map_ws);
      CHECK((char *)(last_prompt.map_ws + cells * (c.rule == QDR_RULE_DELTA ? qdr::kMapFloats : 1)) <= space + need);
      CHECK((char *)last_prompt.segment_ws >= space + (size_t)last_prompt.chunks * c.heads * qdr::kDecayFloats * 4);
    }
    std::free(space);
  }
  view.num_heads = 2;
  CHECK(qdr_prompt_workspace(&pool, 1, 5, &need) == QDR_OK);

  // the step: uncompressed pools only
  CHECK(qdr_linear_step(&pool, i, 3, f, f, f, f, f, nullptr) == QDR_OK);
  CHECK(qdr_linear_step_bf16(&pool, i, 3, x, x, x, f, x, nullptr) == QDR_OK);
  CHECK(qdr_linear_step(&pool, nullptr, 0, f, f, f, f, f, nullptr) == QDR_OK);
  REFUSED(qdr_linear_step(nullptr, i, 3, f, f, f, f, f, nullptr), QDR_E_INVAL);
  REFUSED(qdr_linear_step(&pool, i, -1, f, f, f, f, f, nullptr), QDR_E_INVAL);
  REFUSED(qdr_linear_step(&pool, i, 3, f, f, nullptr, f, f, nullptr), QDR_E_INVAL);
  REFUSED(qdr_linear_step(&pool, i, 1 << 23, f, f, f, f, f, nullptr), QDR_E_INVAL);
  view.all_fp32 = false;
  REFUSED(qdr_linear_step(&pool, i, 3, f, f, f, f, f, nullptr), QDR_E_UNSUPPORTED);
  // a quantised pool's prompt needs room for its states too, and packs them
  size_t more = 0;
  CHECK(qdr_prompt_workspace(&pool, 1, 5, &more) == QDR_OK && more == need + 256 + 2 * 65536);
  view.all_fp32 = true;
  view.gate = QDR_GATE_DIAG;
  REFUSED(qdr_linear_step_bf16(&pool, i, 3, x, x, x, f, x, nullptr), QDR_E_UNSUPPORTED);
  return 0;
}

static int caches() {
  alignas(256) static char mem[1 << 16];
  uint16_t *x = (uint16_t *)mem, *odd = (uint16_t *)(mem + 2);
  int32_t *i = (int32_t *)mem;
  size_t n = 0;
  qdr_kv_desc d{3, 64, 2, 128, QDR_KV_INT8};
  CHECK(qdr_kv_bytes(&d, &n) == QDR_OK && n == 3u * 2 * 2 * (2 * 32 * 128 + 2 * 32 * 4));
  d.kind = QDR_KV_BF16;
  CHECK(qdr_kv_bytes(&d, &n) == QDR_OK && n == 3u * 2 * 2 * (2 * 32 * 128 * 2));
  REFUSED(qdr_kv_bytes(nullptr, &n), QDR_E_INVAL);
  REFUSED(qdr_kv_bytes(&d, nullptr), QDR_E_INVAL);
  const qdr_kv_desc bad[] = {{0, 64, 2, 128, 8}, {3, 16, 2, 128, 8}, {3, 48, 2, 128, 8}, {3, 2048, 2, 128, 8},
                             {3, 64, 0, 128, 8}, {3, 64, 2, 128, 4}, {3, 0, 2, 128, 8}, {3, -32, 2, 128, 8}};
  for (const qdr_kv_desc &b : bad) REFUSED(qdr_kv_bytes(&b, &n), QDR_E_INVAL);
  const qdr_kv_desc wide{3, 64, 2, 64, 8};
  REFUSED(qdr_kv_bytes(&wide, &n), QDR_E_UNSUPPORTED);
  qdr_kv *kv = nullptr;
  d.kind = QDR_KV_INT8;
  CHECK(qdr_kv_bytes(&d, &n) == QDR_OK);
  alignas(256) static char own[3 * 2 * 2 * 8448];
  REFUSED(qdr_kv_create(&d, own, n - 1, &kv), QDR_E_NOMEM);
  REFUSED(qdr_kv_create(&d, own + 16, n, &kv), QDR_E_INVAL);
  REFUSED(qdr_kv_create(&d, own, n, nullptr), QDR_E_INVAL);
  no_memory = true;
  REFUSED(qdr_kv_create(&d, nullptr, 0, &kv), QDR_E_NOMEM);
  REFUSED(qdr_kv_create(&d, own, n, &kv), QDR_E_NOMEM);
  no_memory = false;
  CHECK(kv == nullptr);
  CHECK(qdr_kv_create(&d, own, n, &kv) == QDR_OK && kv && qdr_kv_destroy(kv) == QDR_OK);
  CHECK(qdr_kv_destroy(nullptr) == QDR_OK);
  CHECK(qdr_kv_create(&d, nullptr, 0, &kv) == QDR_OK && kv);
  uint32_t flags = 9;
  CHECK(qdr_kv_poll_device_error(kv, &flags) == QDR_OK && flags == 0);
  REFUSED(qdr_kv_poll_device_error(kv, nullptr), QDR_E_INVAL);

  for (int write = 0; write < 2; ++write) {
    auto call = [&](qdr_kv *c, const int32_t *pages, int max, const int32_t *cu, const int32_t *ctx, int b, int T, uint16_t *k, uint16_t *v) {
      return write ? qdr_kv_write(c, pages, max, cu, ctx, b, T, k, v, nullptr) : qdr_kv_read(c, pages, max, cu, ctx, b, T, k, v, nullptr);
    };
    CHECK(call(kv, i, 2, i, i, 1, 5, x, x) == QDR_OK);
    const int before = launches;
    CHECK(call(kv, nullptr, 0, nullptr, nullptr, 0, 0, nullptr, nullptr) == QDR_OK && launches == before);
    REFUSED(call(nullptr, i, 2, i, i, 1, 5, x, x), QDR_E_INVAL);
    REFUSED(call(kv, nullptr, 2, i, i, 1, 5, x, x), QDR_E_INVAL);
    REFUSED(call(kv, i, -1, i, i, 1, 5, x, x), QDR_E_INVAL);
    REFUSED(call(kv, i, 2, nullptr, i, 1, 5, x, x), QDR_E_INVAL);
    REFUSED(call(kv, i, 2, i, nullptr, 1, 5, x, x), QDR_E_INVAL);
    REFUSED(call(kv, i, 2, i, i, -1, 5, x, x), QDR_E_INVAL);
    REFUSED(call(kv, i, 2, i, i, 1, -5, x, x), QDR_E_INVAL);
    REFUSED(call(kv, i, 2, i, i, 1, 5, nullptr, x), QDR_E_INVAL);
    REFUSED(call(kv, i, 2, i, i, 1, 5, x, odd), QDR_E_INVAL);
    REFUSED(call(kv, i, 2, i, i, 1 << 23, 5, x, x), QDR_E_INVAL);
    device = 1;
    REFUSED(call(kv, i, 2, i, i, 1, 5, x, x), QDR_E_INVAL);
    device = 0;
  }

  auto attend = [&](const int32_t *pages, int b, int T, int heads, uint16_t *q, float scale, void *ws, size_t bytes) {
    return qdr_kv_attend(kv, pages, 2, i, i, b, T, heads, q, scale, x, ws, bytes, nullptr);
  };
  CHECK(qdr_kv_attend_workspace(kv, 1, 5, 4, 2, &n) == QDR_OK && n <= sizeof mem);
  CHECK(attend(i, 1, 5, 4, x, 0.1f, mem, n) == QDR_OK);
  REFUSED(attend(nullptr, 1, 5, 4, x, 0.1f, mem, n), QDR_E_INVAL);
  REFUSED(attend(i, 1, 5, 3, x, 0.1f, mem, n), QDR_E_INVAL);      // not a multiple of the cache's heads
  REFUSED(attend(i, 1, 5, 0, x, 0.1f, mem, n), QDR_E_INVAL);
  REFUSED(attend(i, 1, 5, 4, odd, 0.1f, mem, n), QDR_E_INVAL);
  REFUSED(attend(i, 1, 5, 4, x, NAN, mem, n), QDR_E_INVAL);
  REFUSED(attend(i, 1, 5, 4, x, INFINITY, mem, n), QDR_E_INVAL);
  REFUSED(attend(i, 1, 5, 4, x, 3e38f, mem, n), QDR_E_INVAL);     // times log2(e): infinity
  REFUSED(attend(i, 1, 5, 4, x, -3e38f, mem, n), QDR_E_INVAL);
  CHECK(attend(i, 1, 5, 4, x, -2e38f, mem, n) == QDR_OK);
  REFUSED(attend(i, 1 << 22, 5, 4, x, 0.1f, mem, n), QDR_E_INVAL);
  size_t large = 0;
  CHECK(qdr_kv_attend_workspace(kv, 1, 64, 4, 4096, &large) == QDR_OK && large > 0);
  REFUSED(qdr_kv_attend(kv, i, 4096, i, i, 1, 64, 4, x, 0.1f, x, mem, large - 1, nullptr), QDR_E_NOMEM);
  REFUSED(qdr_kv_attend(kv, i, 4096, i, i, 1, 64, 4, x, 0.1f, x, nullptr, large, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_attend(kv, i, 4096, i, i, 1, 64, 4, x, 0.1f, x, mem + 8, large, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_workspace(kv, 1, 64, 4, -1, &n), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_workspace(kv, 1, 64, 4, 1, nullptr), QDR_E_INVAL);
  REFUSED(qdr_kv_attend_workspace(nullptr, 1, 64, 4, 1, &n), QDR_E_INVAL);
  device = 1;
  REFUSED(qdr_kv_poll_device_error(kv, &flags), QDR_E_INVAL);
  CHECK(qdr_kv_destroy(kv) == QDR_OK && device == 1);    // any device may be current
  device = 0;
  return 0;
}

// How calls are cut up: every row of every sequence has a tile of one launch,
// tiles stay inside their rows, and the pieces' results fit the workspace.
static int plans() {
  for (int heads : {1, 2, 8})
    for (int group : {1, 2, 3, 5, 7, 8, 16, 17, 40, 128, 200})
      for (int n : {1, 2, 33})
        for (int T : {1, 2, 7, 33, 500, 5000})
          for (int pages : {0, 1, 40, 1000000}) {
            const qdr::AttendPlan p = qdr::plan_attend(n, T, heads * group, heads, pages, 6);
            CHECK(p.group == group && (p.few || p.many));
            CHECK(p.few_heads * p.few_tokens <= qdr::kFewRows && p.few_tokens >= 1);
            CHECK(p.many_heads * p.many_tokens <= qdr::kManyRows && p.many_tokens >= 1);
            CHECK(p.few_parts * p.few_heads >= group && (p.few_parts - 1) * p.few_heads < group);
            CHECK(p.many_parts * p.many_heads >= group && (p.many_parts - 1) * p.many_heads < group);
            // one launch only: it takes every sequence; two: they share them out
            CHECK(p.few_tiles == (!p.few ? 0 : p.many ? n : T / p.few_tokens + n));
            CHECK((p.many ? p.many_tiles >= T / p.many_tokens + n : p.many_tiles == 0));
            CHECK(p.few_splits >= 1 && p.few_splits <= 64 && p.many_splits >= 1 && p.many_splits <= 64);
            const size_t few = (size_t)p.few_tiles * heads * p.few_parts * p.few_splits * 16 * 130;
            const size_t many = (size_t)p.many_tiles * heads * p.many_parts * p.many_splits * 128 * 130;
            CHECK(p.few_floats == (p.few_splits > 1 ? few : 0));
            CHECK(p.many_floats == (p.many_splits > 1 ? many : 0));
          }
  return 0;
}

int main() {
  if (prompts() || caches() || plans()) return 1;
  std::printf("ok %d\n", checks);
  return 0;
}
