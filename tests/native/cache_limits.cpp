// cache_limits.cpp -- the largest calls that are taken and the smallest that are
// refused for their size, over the stubs of cache_sanitize.cpp (built with g++ by
// tests/test_cache_limits.py).
#define main every_refusal
#include "cache_sanitize.cpp"
#undef main

static int rotations() {
  double freq[8] = {1, 1, 1, 1, 1, 1, 1, 1};
  qdr_rotary_desc d{128, 16, QDR_ROTARY_HALF, freq, 1};
  qdr_rotary *r = nullptr;
  CHECK(qdr_rotary_create(&d, &r) == QDR_OK);
  // 2^24 workgroups of so many tokens
  const struct { int heads; int64_t least; } at[] = {{1, 1 << 29}, {2, 1 << 29}, {4, 1 << 29}, {5, 25ll << 24}, {8, 1 << 28}, {32, 1 << 26}, {65, 1 << 24}, {128, 1 << 24}, {129, 1 << 23}, {1 << 17, 1 << 14}};
  for (const auto &x : at) {
    const int64_t stride = (int64_t)x.heads * 128;
    const int tokens = std::max(1, std::min(32, 128 / x.heads)), last = (int)(x.least - tokens);
    CHECK(qdr_rotate(r, i, last, x.heads, f, stride, f, stride, nullptr) == QDR_OK && rotated.T == last);
    CHECK(qdr_rotate_bf16(r, i, last, x.heads, ::x, stride, ::x, stride, nullptr) == QDR_OK);
    REFUSED(qdr_rotate(r, i, last + 1, x.heads, f, stride, f, stride, nullptr), QDR_E_INVAL);
    REFUSED(qdr_rotate_bf16(r, i, (int)x.least, x.heads, ::x, stride, ::x, stride, nullptr), QDR_E_INVAL);
  }
  return qdr_rotary_destroy(r) == QDR_OK ? 0 : 1;
}

static int shared() {
  qdr_kv kv;
  kv.desc = {300, 64, 2, 128, QDR_KV_BF16};
  kv.page_shift = 6;
  kv.base = (uint8_t *)mem;
  size_t need = 0;
  for (int heads : {2, 8, 64}) {
    const int most = (1 << 26) / heads - 1;
    CHECK(qdr_kv_attend_shared_workspace(&kv, 2, most, 1, heads, 9, &need) == QDR_OK);
    CHECK(qdr_kv_attend_shared(&kv, i, 9, i, i, 2, most, i, i, 1, heads, x, 1.0f, x, mem, need, nullptr) == QDR_OK);
    REFUSED(qdr_kv_attend_shared_workspace(&kv, 2, most + 1, 1, heads, 9, &need), QDR_E_INVAL);
  }
  return 0;
}

int main() {
  if (rotations() || shared()) return 1;
  std::printf("ok %d\n", checks);
  return 0;
}
