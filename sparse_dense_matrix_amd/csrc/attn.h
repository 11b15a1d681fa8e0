// attn.h -- block-sparse attention: what the host calls (attn.cpp) and the
// kernels (attn_*.hip) share.
//
// Keys come in blocks of 64 (the pages of a cache).  A list names the blocks
// that a query block of q_block tokens reads for one key/value head; the rows
// of a query block are its tokens times the query heads that share the key
// head, token major: row r is token r / group, head r % group.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/spmm.h"

namespace sdm {

constexpr int32_t kAttnPage = 64;  // keys of a block
constexpr int32_t kAttnMaxScored = 32768;  // blocks the choice can score: their scores stand in LDS

// A tensor of heads on the device: byte strides of the sequence (or page),
// the token and the head; the head's elements are consecutive.
struct AttnView {
  char *p;
  int64_t sb, st, sh;
};

struct AttnArgs {
  AttnView q, k, v, o;
  AttnView g, dq, dk, dv;      // gradients (backward)
  float *lse;                  // [b][hq][nq]
  float *stats;                // [b * hq * nq + 1][2] workspace: rows' lse (base 2) and do . o; last: no row's
  const int32_t *lists;        // [b][hk][nqb][max_blocks], or null: every block
  const int32_t *table;        // [b][nkb] pages of the cache, or null
  const uint64_t *tree;        // [b][nq] rows of the drafted tokens' mask, or null
  const int32_t *lens, *starts;  // [b], or null: nk, 0
  int32_t b, nq, nk, hq, hk, group, q_block, nqb, nkb, max_blocks, pages;
  int32_t pack, list_nqb;      // lists that share a row tile (0: one), and lists of a head: q_block, nqb and
                               // rows are then those of `pack` query blocks
  int32_t rows;                // rows of a query block: min(q_block, nq) * group
  int32_t rtiles;              // row tiles of a query block
  int32_t nsplit, per_split;   // ranges of a list and entries of each
  int32_t entries;             // entries of a list: max_blocks, or nkb
  float scale;
  float *part_o;               // [nsplit][b * hq * nq][d] partial sums (nsplit > 1)
  float *part_ml;              // [nsplit][b * hq * nq][2] their maximum and sum
  // inverse lists (backward)
  int32_t *inv_ids;            // [b * hk][nqb * max_blocks] query blocks of each key block, key block major
  int32_t *inv_ptr;            // [b * hk][nkb][2] first entry and count of each key block
  int32_t *items;              // [b * hk][slots] key block (-1: none) and part of its inverse list, pairs
  int32_t *queue;              // [8] items taken of each queue of the dk, dv kernel
  int32_t chunk, slots;        // entries of an item; items of a head at most
  float *part_kv;              // [b * hk][slots][2][64][d] partial dk, dv of split key blocks
};

struct AttnPoolArgs {
  AttnView k;
  int8_t *pooled;              // [pages or b * nkb][hk][d]
  float *pooled_scale;         // [pages or b * nkb][hk]
  const int32_t *table, *lens, *first;
  int32_t b, nk, hk, nkb, pages, width;
};

struct AttnSelectArgs {
  AttnView q;
  const int8_t *pooled;
  const float *pooled_scale;
  int32_t *lists;
  const int32_t *table, *lens, *starts;
  int32_t b, nq, nk, hq, hk, group, q_block, nqb, nkb, max_blocks, pages, sink, local;
};

// ---- shared rules, for the kernels and the host's tests -------------------

// Length of sequence b, within what its tensors hold.
__host__ __device__ inline int32_t attn_len(const int32_t *lens, int32_t b, int32_t nk) {
  const int32_t n = lens ? lens[b] : nk;
  return n < 0 ? 0 : (n > nk ? nk : n);
}

// Position of sequence b's first query.  Positions below 0 or past the keys
// leave a query without keys, so what lies outside [-nq, nk] can be cut off.
__host__ __device__ inline int32_t attn_start(const int32_t *starts, int32_t b, int32_t nq, int32_t nk) {
  const int32_t s = starts ? starts[b] : 0;
  return s < -nq ? -nq : (s > nk ? nk : s);
}

// The page that block `id` of a sequence stands in: table[id], or -1 where
// the table names no page of the cache; without a table its own number.
__host__ __device__ inline int32_t attn_page(const int32_t *table_row, int32_t id, int32_t pages) {
  if (!table_row) return id;
  const int32_t p = table_row[id];
  return p >= 0 && p < pages ? p : -1;
}

// Whether a list's entry names a block with a key at or below last_key
// (last_key < len).
__host__ __device__ inline bool attn_names(int32_t id, int32_t last_key) {
  return id >= 0 && id <= last_key / kAttnPage && last_key >= 0;
}

// Row tile of the forward kernels and the rows of a workgroup.
struct AttnTile {
  int32_t row_waves, key_waves, key_tile, rows;
};
AttnTile attn_tile(int32_t rows, int32_t nqb);
// Lists that share a row tile of 32 rows (a power of two), for `lists` lists in
// all with `rows` rows and max_blocks entries each; 0: one list a tile.
int32_t attn_pack(int64_t lists, int32_t rows, int32_t max_blocks);
AttnArgs attn_packed(AttnArgs a, int32_t pack);
// Ranges a list is cut into, and entries of each, for `tiles` row tiles in
// all with tile_rows rows each; lists name about `entries` blocks at most, in
// max_entries places.
void attn_split(int64_t tiles, int32_t tile_rows, int32_t entries, int32_t max_entries, int32_t *nsplit,
                int32_t *per_split);
// Query blocks that one item of the dk, dv kernel takes, and items of a head,
// for nqb lists of a head with `entries` entries in all.
void attn_chunks(int64_t heads, int64_t entries, int32_t nqb, int32_t rows, int32_t nkb, int32_t *chunk, int32_t *slots);

hipError_t launch_attn_forward(const AttnArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_backward(const AttnArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_pool(const AttnPoolArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_select(const AttnSelectArgs &a, spmm_dtype_t t, int d, hipStream_t s);

}  // namespace sdm
