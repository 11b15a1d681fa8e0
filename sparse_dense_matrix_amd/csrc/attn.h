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

// Scales of a cache in 8 bits: [slots][hk][64], slot = page or b * nkb + block.
struct AttnScales {
  const float *k, *v;
};

// New tokens to a cache in 8 bits, or the cache back to tensors.
struct AttnCodesArgs {
  AttnView k, v;               // [b][nq or nk] tensors of 16 bits
  AttnView k8, v8;             // pages, or [b][nk]
  float *k_scale, *v_scale;    // [slots][hk][64]
  const int32_t *table, *lens, *starts;
  int32_t b, n, nk, hk, nkb, pages;  // n: tokens of a sequence in k and v
};

// Norm and rotation of queries and keys, and their gradients.
struct RopeArgs {
  AttnView x[2], y[2];         // queries, keys: inputs; outputs
  AttnView g[2], dx[2];        // gradients of the outputs and of the inputs (backward)
  const float *w[2];           // [d] weights of the norm, or null: no norm
  float *dw[2];                // [d] their gradients
  int32_t heads[2];
  const double *turns;         // [pairs] turns (of 2 pi) that one position makes
  const int32_t *axis;         // [pairs] axis whose positions turn the pair
  const int32_t *positions;    // [axes][b][n], or null: starts + t on every axis
  const int32_t *lens, *starts;
  float *part;                 // [grid][2][d] workspace: partial gradients of the weights (backward)
  int32_t b, n, pairs, axes, interleaved;
  int32_t grid;                // workgroups of the backward kernel at most
  float eps;
};

struct AttnPoolArgs {
  AttnView k;
  const float *k_scale;        // of a cache in 8 bits: [slots][hk][64]; null: k is 16 bits
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

// Where tokens go that stand from position `start` on, `n` of them, of which those
// in [0, len) count: in block w of the ones they can lie in, its keys [lo, hi)
// (none where lo >= hi).  Cut off to the block in 64 bits: a position at either
// end of 32 bits is further from a block than 32 bits reach.
struct AttnTaken {
  int32_t id, lo, hi;
};
__host__ __device__ inline AttnTaken attn_taken(int64_t start, int32_t n, int32_t len, uint32_t w) {
  const int64_t end = start + n < len ? start + n : len;
  const int64_t id = (start > 0 ? start : 0) / kAttnPage + w, lo = start - id * kAttnPage, hi = end - id * kAttnPage;
  const auto cut = [](int64_t x) { return static_cast<int32_t>(x < 0 ? 0 : (x > kAttnPage ? kAttnPage : x)); };
  return {static_cast<int32_t>(id), cut(lo), cut(hi)};
}

// Workgroups of 256 threads that a launch holds: work-items are counted in 32 bits.
constexpr int64_t kAttnMaxGroups = (int64_t(1) << 24) - 1;

// How the rows of a cache in 8 bits are written or read back: row by row, or by
// blocks (`width` of a sequence); and workgroups.
//
// Written row by row up to 32k rows, or sequences' parts of up to a block, which fill
// half of the two blocks that they may lie in: 32 sequences of 8 tokens of 8 heads of
// 128 take 3.5 us row by row, by blocks 6.1; 4096 tokens 8.0 and 8.1, 16k 22 and 18;
// 256 of 64 tokens 21 and 25, of 128 38 and 34.
struct AttnCodesLaunch {
  bool rows;
  int64_t width, groups;
};
inline AttnCodesLaunch attn_codes_launch(const AttnCodesArgs &a, int d, bool read) {
  const int64_t n = a.n, rows = static_cast<int64_t>(a.b) * n * a.hk, per = 256 / (d / 8);
  // the blocks that n tokens from any position on can lie in
  const int64_t reach = (n + kAttnPage - 2) / kAttnPage + 1, width = read || reach > a.nkb ? a.nkb : reach;
  const bool by_rows = !read && (rows <= 32768 || n <= kAttnPage);
  return {by_rows, width, by_rows ? (rows + per - 1) / per : static_cast<int64_t>(a.b) * width * a.hk};
}

// Tokens of a workgroup that turns rows.  Few heads: tokens enough that a group of
// lanes has rows of its own.  32k tokens of 12 and 4 heads of 64 take 26 us in
// sixteens, in fours 41; 6400 of 32 and 8 heads of 128 27 us in fours.
inline int32_t rope_tokens(int32_t heads) { return heads <= 16 ? 16 : 4; }

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
// The ranges' partial sums of launch_attn_forward and launch_attn_cache8.
hipError_t launch_attn_merge(const AttnArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_cache8(const AttnArgs &a, const AttnScales &x, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_write(const AttnCodesArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_read(const AttnCodesArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_rope(const RopeArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_rope_backward(const RopeArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_backward(const AttnArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_pool(const AttnPoolArgs &a, spmm_dtype_t t, int d, hipStream_t s);
hipError_t launch_attn_select(const AttnSelectArgs &a, spmm_dtype_t t, int d, hipStream_t s);

}  // namespace sdm
