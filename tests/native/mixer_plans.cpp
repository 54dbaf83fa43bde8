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

int main() {
  if (few_rows_beside_long()) return 1;
  std::printf("ok %d\n", checks);
  return 0;
}
