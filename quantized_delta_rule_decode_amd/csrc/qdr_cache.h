// qdr_cache.h -- arguments and launches of what is done around the paged cache
// (rotary positions, pages, attention behind shared prefixes); the public ABI is
// include/qdr_cache.h.
#pragma once

#include "qdr_mixer.h"

namespace qdr {

constexpr uint32_t kErrFull = 8u;   // QDR_DEVERR_FULL

// ---- rotary positions (qdr_rotary.hip)
struct RotaryView {
  const uint64_t *turns;   // [channels/2] turns a token, modulo 1, times 2^64
  int32_t channels, layout;
  float amplitude;
};
struct RotateArgs {
  RotaryView rotary;
  const int32_t *positions;
  int32_t T, heads;
  const void *x;
  void *y;
  int64_t x_stride, y_stride;
  int32_t tokens, head_parts, part_heads;   // of a workgroup
};
hipError_t launch_rotate(const RotateArgs &, bool bf16, hipStream_t);

struct RotaryWriteArgs {
  KvArgs kv;               // k and v are read only
  RotaryView rotary;
  const uint16_t *q;
  uint16_t *q_out;
  int32_t q_heads;
  int64_t q_stride, k_stride, v_stride;
  // heads of a workgroup, and workgroups of a block of tokens, for keys and queries
  int32_t kv_heads, kv_parts, query_heads, query_parts;
};
hipError_t launch_kv_write_rotary(const RotaryWriteArgs &, int kind, hipStream_t);

// ---- pages (qdr_pages.hip)
struct CopyArgs {
  const uint8_t *from;
  uint8_t *to;
  uint64_t bytes;                // of a page or slot, a multiple of 16
  const int32_t *src, *dst;
  int32_t m, num_from, num_to;
  int32_t parts;                 // workgroups of a pair
  uint32_t *err_from, *err_to;
  uint32_t bit;
};
hipError_t launch_copy(const CopyArgs &, hipStream_t);

constexpr int kBookTile = 2048;                     // pages of a workgroup
constexpr int64_t kMostBookPages = (int64_t)1 << 26;
inline int64_t book_tiles(int64_t num_pages) { return (num_pages + kBookTile - 1) / kBookTile; }

struct AssignArgs {
  KvArgs kv;                     // base, pages, context, n (old rows), max_pages, err
  int kind;
  const int32_t *parent, *add, *refs;
  int32_t m;
  int32_t *new_pages, *new_context, *new_refs;
  // workspace
  int32_t *hold;                 // [num_pages] who has a page besides rows that only begin to fill it
  int32_t *first;                // [num_pages] first row that keeps the page in part
  int32_t *free;                 // [num_pages] the free pages, lowest first
  int32_t *counts;               // [tiles] free pages of a tile of pages
  int32_t *offset;               // [m][8] the row's first place in `free` (-1: an empty row), its tokens, the kept
                                 // ones, the page behind its full ones (-1: none), and whether that one stays its own
  int32_t parts;                 // workgroups that copy a row's last page
};
hipError_t launch_assign(const AssignArgs &, hipStream_t);

struct CompactArgs {
  uint8_t *base;
  uint64_t page_bytes;
  int32_t num_pages;
  const int32_t *refs, *pages;
  int64_t entries;               // of the tables
  int32_t *moved, *new_refs, *new_pages;
  // workspace
  int32_t *counts;               // [tiles] free pages of a tile of pages
  int32_t *src, *dst;            // [num_pages] each: pages that move, by the used pages before them, and where to; dst[p] of a page that moves: its place in src
  int32_t *moves;                // [3] how many, where src begins, and the number of used pages
  int32_t parts, groups;         // workgroups of a move; of all moves
};
hipError_t launch_compact(const CompactArgs &, hipStream_t);

// ---- attention behind shared prefixes (qdr_attend_shared.hip)
// Rows (tokens x query heads of a key head) go through the keys in the two kinds
// of tiles of qdr_attend.  The rows of a group, which are consecutive, are dealt
// to tiles as if they were one sequence's and go through the shared keys; the
// rows of each sequence go through its own, a workgroup a tile or a piece of its
// keys, as there.
// The groups' tiles of a key head, with what their blocks cost, are laid end to
// end in a line that is cut into `ranges` equal parts, one a workgroup, which goes
// through the tiles, or pieces of tiles, of its part: groups of any sizes and
// prefixes fill the compute units.  A tile that was cut, or whose rows have
// shared keys too, leaves its rows' maximum, sum and unnormalised result in the
// workspace, and a last launch joins them.
constexpr int kSharedWaves = 4, kSharedLeast = 8;   // of a workgroup; fewest blocks of a piece of few rows
constexpr int kLeastSaved = 12288;                  // blocks of a key head
struct SharedPlan {
  int group;                                 // query heads a key head
  int few_heads, few_tokens, few_parts;
  int many_heads, many_tokens, many_parts;
  float many_inverse;                        // 1 / many_tokens
  int few_splits, many_splits;               // pieces of the keys of sequences' tiles
  int many_tiles;                            // places of many-row tiles of sequences
  bool by_tokens;                            // a sequence's place goes by the tokens before it, not by the sequences
  int ranges;                                // parts of the line, at most; 0: each sequence goes by itself
  int slot_rows;                             // rows of a piece of a cut tile of the line: 16 where no tile has more
  // places in the workspace, in floats: whole tiles' results by row, of shared
  // and own keys ([T * q_heads][130] each); the line's cut tiles' by workgroup
  // (two each: of its first tile and its last, [slot_rows][130]); few and many
  // rows' by piece ([16] and [128][130]); each token's passes
  size_t cut, few_pieces, many_pieces, info, floats;
};
SharedPlan plan_shared(int n, int T, int groups, int q_heads, int heads, int max_pages, int page_shift);

struct SharedArgs {
  AttendArgs a;          // part: the workspace
  const int32_t *group_cu, *shared;
  int32_t groups;
};
hipError_t launch_attend_shared(const SharedArgs &, const SharedPlan &, int kind, hipStream_t);

}  // namespace qdr
