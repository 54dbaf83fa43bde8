// mixer_plans.cpp -- what an attention call's plan promises to a single
// sequence whatever the others are, and which calls the counts of a launch
// refuse; with the stubs of mixer_sanitize.cpp.  Built and run by
// tests/test_mixer_plans.py.
//
// Prints "ok <n>" (n = checks passed) and exits 0; a failed check exits 1.
#define main other_main
#include "mixer_sanitize.cpp"
#undef main

// A sequence of few rows is taken by the few-row launch (its keys cut where
// there are places, its weights in two parts) also beside long ones.
static int few_rows_beside_long() {
  for (int heads : {1, 2, 8})
    for (int group : {1, 4, 16, 40})
      for (int n : {2, 4, 16, 64})
        for (int T : {n + 1, 1000, 8195, 1 << 16})
          for (int pages : {1, 32, 512}) {
            const qdr::AttendPlan p = qdr::plan_attend(n, T, heads * group, heads, pages, 6);
            CHECK(p.few && p.few_tiles >= n);
          }
  // three tokens over 32768 keys beside a prompt of 8192: their keys are cut
  const qdr::AttendPlan p = qdr::plan_attend(4, 8195, 32, 8, 512, 6);
  CHECK(p.many && p.few_splits == 8);
  return 0;
}

// A call is refused for the workgroups that it has, not for more than those.
static int sizes() {
  qdr_kv_desc d{4, 64, 8, 128, QDR_KV_BF16};
  qdr_kv *kv = nullptr;
  CHECK(qdr_kv_create(&d, nullptr, 0, &kv) == QDR_OK && kv);
  size_t need = 0;
  CHECK(qdr_kv_attend_workspace(kv, 1, 262144, 64, 4096, &need) == QDR_OK);
  CHECK(qdr_kv_attend_workspace(kv, 4096, 262144, 64, 1, &need) == QDR_OK && need == 0);
  CHECK(qdr_kv_attend_workspace(kv, 1, 1 << 22, 64, 1 << 16, &need) == QDR_OK && need == 0);
  // just under 2^24: tiles of sixteen tokens, eight heads; of a single token a few-row one
  CHECK(qdr_kv_attend_workspace(kv, 1, (1 << 25) - 32, 64, 1, &need) == QDR_OK);
  REFUSED(qdr_kv_attend_workspace(kv, 1, 1 << 25, 64, 1, &need), QDR_E_INVAL);
  CHECK(qdr_kv_attend_workspace(kv, (1 << 20) - 1, 1, 8, 1, &need) == QDR_OK);
  REFUSED(qdr_kv_attend_workspace(kv, 1 << 20, 1, 8, 1, &need), QDR_E_INVAL);
  // far over: nothing overflows on the way
  for (int n : {1, 2, 1 << 24, 1 << 30})
    for (int T : {1 << 28, 1 << 30})
      for (int q_heads : {8, 8 << 10, (1 << 24) - 8, (1 << 30), 0x7FFFFFF8})
        for (int pages : {0, 1, 0x7FFFFFFF}) REFUSED(qdr_kv_attend_workspace(kv, n, T, q_heads, pages, &need), QDR_E_INVAL);
  for (int q_heads : {(1 << 24), 0x7FFFFFF8}) REFUSED(qdr_kv_attend_workspace(kv, 1, 1, q_heads, 1, &need), QDR_E_INVAL);
  CHECK(qdr_kv_destroy(kv) == QDR_OK);
  return 0;
}

// A cache whose bytes do not fit 64 bits is refused, not made smaller.
static int large_caches() {
  size_t n = 0;
  const int32_t most = 0x7FFFFFFF;
  qdr_kv_desc d{most, 1024, 8, 128, QDR_KV_BF16};
  CHECK(qdr_kv_bytes(&d, &n) == QDR_OK && n == (size_t)most * 8 * 32 * 16384);
  alignas(256) static char own[1 << 16];
  for (int32_t heads : {1 << 20, 1 << 14, most}) {       // (2^31 - 1) 2^20 2^19 bytes: a small number modulo 2^64
    d.num_heads = heads;
    qdr_kv *kv = nullptr;
    REFUSED(qdr_kv_bytes(&d, &n), QDR_E_INVAL);
    REFUSED(qdr_kv_create(&d, own, sizeof own, &kv), QDR_E_INVAL);
    CHECK(kv == nullptr);
  }
  return 0;
}

int main() {
  if (few_rows_beside_long() || sizes() || large_caches()) return 1;
  std::printf("ok %d\n", checks);
  return 0;
}
