// qdr_host.h -- what the host entry points outside qdr_runtime.cpp use of a
// pool: its fields, its launches and the calling thread's error message.
#pragma once

#include "../../include/qdr.h"
#include "qdr_internal.h"

namespace qdr {

struct PoolView {
  uint8_t *base;
  uint64_t slot_stride;
  int32_t num_slots, num_heads;
  int gate;
  int device;
  bool all_fp32;      // whole-head units, every head FP32: head h of a slot is the 64 KiB at h * 65536
  uint32_t *err;
};
PoolView pool_view(const qdr_pool *pool);

// Sets the thread's message and returns `st`; set_ok clears it.
qdr_status set_error(qdr_status st, const char *message);
qdr_status set_ok();

// The QDR_DEBUG=1 check of a slot table (padding allowed).
qdr_status pool_check_slots(const qdr_pool *pool, const int32_t *slots, int32_t n, hipStream_t st);
// Orders `st` after the pool's last two-stream write-back.
hipError_t pool_after_writeback(qdr_pool *pool, hipStream_t st);
// The pack / unpack launches without the host-side slot check.
qdr_status pool_pack(qdr_pool *pool, const int32_t *slots, int32_t n, const float *S, hipStream_t st);
qdr_status pool_unpack(qdr_pool *pool, const int32_t *slots, int32_t n, float *S, hipStream_t st);

}  // namespace qdr
