// qdr_calls.h -- what the host entry points over pools and caches share: their
// checks of arguments, their messages, and the cache's handle.
#pragma once

#include "../../include/qdr_mixer.h"

#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "qdr_host.h"
#include "qdr_mixer.h"

struct qdr_kv {
  qdr_kv_desc desc{};
  int device = 0;
  int page_shift = 0;
  uint8_t *base = nullptr;
  bool owns_base = false;
  uint32_t *d_err = nullptr;
};

namespace qdr {
namespace calls {

inline qdr_status fail(qdr_status st, const char *fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return qdr::set_error(st, buf);
}

inline qdr_status launched(hipError_t e) {
  if (e != hipSuccess) return fail(QDR_E_DEVICE, "kernel launch failed: %s", hipGetErrorString(e));
  return qdr::set_ok();
}

// Counts of sequences and rows are kept where sums of them fit 32 bits, and
// launches under 2^32 threads.
constexpr int32_t kMostRows = 1 << 30;
constexpr int32_t kMostHeads = 1 << 17;             // 64 rows of a token array under 2^32 bytes
constexpr int64_t kMostGroups = (int64_t)1 << 24;   // of 256 threads

inline qdr_status check_counts(int32_t n, int32_t T) {
  if (n < 0 || T < 0) return fail(QDR_E_INVAL, "n and T must be >= 0 (got %d, %d)", n, T);
  if (n > kMostRows || T > kMostRows) return fail(QDR_E_INVAL, "n and T must be <= %d (got %d, %d)", kMostRows, n, T);
  return QDR_OK;
}

inline qdr_status check_groups(int64_t groups) {
  if (groups >= kMostGroups) return fail(QDR_E_INVAL, "the call is too large for one launch (%lld workgroups): cut it up", (long long)groups);
  return QDR_OK;
}

inline qdr_status check_device(int device) {
  int now = -1;
  if (hipGetDevice(&now) != hipSuccess) return fail(QDR_E_DEVICE, "no HIP device");
  if (now != device) return fail(QDR_E_INVAL, "the handle belongs to device %d, the current device is %d", device, now);
  return QDR_OK;
}

inline qdr_status check_workspace(const void *ws, size_t have, size_t need) {
  if (need == 0) return QDR_OK;
  if (!ws) return fail(QDR_E_INVAL, "workspace is NULL (%zu bytes are needed)", need);
  if (reinterpret_cast<uintptr_t>(ws) % 16) return fail(QDR_E_INVAL, "workspace must be 16-byte aligned");
  if (have < need) return fail(QDR_E_NOMEM, "workspace holds %zu bytes, the call needs %zu", have, need);
  return QDR_OK;
}

inline bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

#define QDR_TRY(x)                     \
  do {                                 \
    const qdr_status st_ = (x);        \
    if (st_ != QDR_OK) return st_;     \
  } while (0)

inline qdr_status check_kv_call(const qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
                                const int32_t *context, int32_t n, int32_t T, const void *x, const void *y) {
  if (!kv) return fail(QDR_E_INVAL, "kv is NULL");
  QDR_TRY(check_counts(n, T));
  if (max_pages < 0) return fail(QDR_E_INVAL, "max_pages must be >= 0 (got %d)", max_pages);
  if (n == 0 || T == 0) return QDR_OK;
  if (!cu || !context || (max_pages > 0 && !pages) || !x || !y) return fail(QDR_E_INVAL, "a tensor pointer is NULL");
  if (!aligned4(x) || !aligned4(y)) return fail(QDR_E_INVAL, "tensors must be 4-byte aligned");
  return check_device(kv->device);
}

inline qdr::KvArgs kv_args(const qdr_kv *kv, const int32_t *pages, int32_t max_pages, const int32_t *cu,
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

}  // namespace calls
}  // namespace qdr
