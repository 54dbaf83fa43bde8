// qdr_mixer.h -- arguments and launches of the token mixers (prompt form,
// additive step, key/value cache); the public ABI is include/qdr_mixer.h.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime.h>

namespace qdr {

constexpr uint32_t kErrSlot = 1u, kErrLength = 2u, kErrPage = 4u;   // QDR_DEVERR_*

// ---- prompt form (qdr_prompt.hip)
constexpr int kChunk = 64;                       // tokens taken at a time
// Fragments of a lower triangular 64 x 64 matrix: row tile w (16 rows) has
// w/2 + 1 of them, each 16 rows x 32 columns, 64 lanes x 8 fp32.
constexpr int kTriFrags = 6;
constexpr size_t kTriFloats = (size_t)kTriFrags * 512;
// Workspace of one (chunk, head): sums of the gates' logarithms (64 fp64), the
// decays from the chunk's start and to its end (64 fp32 each), and for DELTA
// one triangular matrix.
constexpr size_t kDecayFloats = 4 * kChunk, kChunkFloats = kDecayFloats + kTriFloats;
constexpr int kSegmentLeast = 4, kSegmentMost = 64;   // chunks of a segment (SUM: no most)
// Whether DELTA's chunks are taken by k_prompt_chain: four workgroups to a
// (sequence, head), a workgroup a compute unit, so few pairs.  4096 tokens of
// 128 and 160 heads 422 and 575 us, by k_prompt_scan 487 and 507.  Of several
// sequences the longest counts more than all together, and the chain is faster
// at one: 8192 tokens of 32 heads in six sequences of unlike lengths 232 us, the
// scan 399, of equal ones 224 and 190; in eight 240 and 230, 222 and 157.
inline bool in_chains(int64_t n, int64_t heads) { return n * heads <= (n == 1 ? 128 : 192); }
constexpr size_t kMapFloats = (size_t)8 * 4 * 3 * 64 * 4;   // a 128 x 128 left operand in three parts
// Sequences of a call that are put in order of length, which scans of unlike
// lengths gain from (the longest, started last, would run alone).  n^2
// comparisons beside the chunks' kernel; where there are thousands of sequences
// one of them is a small share of the whole.
constexpr int kMostOrdered = 1024;

struct PromptArgs {
  const int32_t *slots, *carry, *cu;
  int32_t n, T, H, num_slots;
  int32_t chunks;             // chunk places of a head: T/64 + n
  const uint16_t *q, *k, *v;
  const float *beta, *gate;   // beta: NULL for SUM
  uint16_t *o;
  float *chunk_ws;            // [chunks][H][kChunkFloats], SUM: [kDecayFloats]
  // where the states are: an uncompressed pool's blocks, or dense fp32
  uint8_t *pool;              // NULL: dense
  uint64_t slot_stride;
  float *S;                   // [n][H][128][128]
  int32_t *slots_in, *slots_out;   // dense: slots to unpack and to pack (-1: none)
  int32_t *order;             // DELTA: [n] sequences by falling length; NULL: as they come
  // a sequence is cut into segments of so many chunks that are taken side by
  // side (0: not cut); places of segments of a head, and their states
  int32_t segment, segments;
  float *segment_ws;          // [segments][H][128*128]
  float *map_ws;              // SUM: [segments][H] decays, DELTA: [segments][H][kMapFloats]
  uint32_t *err;
};
hipError_t launch_prompt_slots(const PromptArgs &, hipStream_t);
hipError_t launch_prompt_chunks(const PromptArgs &, bool delta, hipStream_t);
hipError_t launch_prompt_scan(const PromptArgs &, bool delta, hipStream_t);

// ---- additive step (qdr_linear.hip)
struct LinearArgs {
  const int32_t *slots;
  int32_t B, H, num_slots;
  const void *q, *k, *v;
  const float *gate;
  void *o;
  uint8_t *pool;
  uint64_t slot_stride;
  uint32_t *err;
};
hipError_t launch_linear_step(const LinearArgs &, bool bf16, hipStream_t);

// ---- key/value cache (qdr_kv.hip, qdr_attend.hip)
// A page holds, head after head, its tokens in blocks of 32.  A block is laid
// out in the order in which the attention's matrix instructions take it:
//   K   [16-token tile][.][lane (g, key)][16 B]: channels 64 h + 16 g ..: with
//       8-bit codes 16 of them (h = 0, 1), with bfloat16 8 (part 2 h + p holds
//       channels 64 h + 16 g + 8 p ..)
//   V   [16-channel tile][lane (g, channel)][8 tokens 4 g + {0..3, 16..19}];
//       8-bit codes keep the two tiles of a pair in one lane's 16 B
//   8-bit only: fp32 scales of the 32 keys, then of the 32 values.
constexpr int kBlock = 32;
constexpr int kMostContext = 1 << 30;
constexpr uint32_t kKv8Half = 4096, kKv8Scale = 2 * kKv8Half, kKv8Block = kKv8Scale + 2 * kBlock * 4;
constexpr uint32_t kKv16Half = 8192, kKv16Block = 2 * kKv16Half;

struct KvArgs {
  uint8_t *base;
  int32_t num_pages, page_shift, heads;   // page_shift: log2(page_tokens)
  const int32_t *pages;
  int32_t max_pages;
  const int32_t *cu, *context;
  int32_t n, T;
  uint16_t *k, *v;                // write: read only
  uint32_t *err;
};
hipError_t launch_kv_write(const KvArgs &, int kind, hipStream_t);
hipError_t launch_kv_read(const KvArgs &, int kind, hipStream_t);

// Rows (tokens x query heads of one key/value head) of the two kinds of
// tiles, waves of a few-row tile, and the fewest blocks of keys of a piece (one
// for each of the eight waves; two passes of the many-row loop).  Eight waves a
// few-row tile instead of four: 777 keys 10.0 -> 8.5 us, 64 requests of 8192
// 181 -> 175 us.
constexpr int kFewRows = 16, kManyRows = 128;
constexpr int kFewWaves = 8, kFewLeast = 8, kManyLeast = 4;

// How an attention call is cut up: rows of a tile, tiles, and pieces of the
// keys; decided on the host from the call's counts alone.
struct AttendPlan {
  int group;          // query heads a key/value head
  // few-row tiles: rows = tokens x heads <= 16
  bool few; int few_heads, few_tokens, few_parts, few_tiles, few_splits;
  // many-row tiles: up to 128 rows
  bool many; int many_heads, many_tokens, many_parts, many_tiles, many_splits;
  size_t few_floats, many_floats;   // partial results in the workspace
};
AttendPlan plan_attend(int n, int T, int q_heads, int heads, int max_pages, int page_shift);

struct AttendArgs {
  KvArgs kv;
  const uint16_t *q;
  uint16_t *o;
  int32_t q_heads;
  float scale_log2;      // scale * log2(e)
  float *part;           // partial results where the keys are cut
};
hipError_t launch_attend(const AttendArgs &, const AttendPlan &, int kind, hipStream_t);

}  // namespace qdr
