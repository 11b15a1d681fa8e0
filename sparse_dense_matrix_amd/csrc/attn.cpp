// attn.cpp -- the attention calls of spmm.h: argument checks, workspace and
// launch dispatch.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <new>
#include <utility>

#include "attn.h"
#include "internal.h"

namespace sdm {
namespace {

constexpr int64_t kElem = 2;                      // bytes of bf16 and f16
constexpr int32_t kMaxEntries = 1 << 30;          // of a list
constexpr int64_t kMaxRowOffset = 0xffffff00ll;   // a sequence's last query byte in the backward kernels

spmm_status_t bad(const char *fn, const std::string &what) {
  return fail(SPMM_ERR_INVALID_ARG, std::string(fn) + ": " + what);
}

bool power_of_two(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

// Whether steps along the first k extents, each shorter than n[i] either way,
// lead from r elements to less than dim away from 0, with a step somewhere
// (`moved`: one was taken before).  Strides ascend, so that few steps of a
// longer one are in reach of the shorter ones: one where the extents nest.
// Strides that leave more than `tries` ways are taken to overlap.
bool meets(const int64_t *n, const int64_t *s, int k, int64_t r, bool moved, int64_t dim, int *tries) {
  if (k == 0) return moved && r > -dim && r < dim;
  const int64_t last = n[k - 1] - 1, step = s[k - 1];
  if (step == 0) return last > 0 || meets(n, s, k - 1, r, moved, dim, tries);
  int64_t reach = dim - 1;
  for (int i = 0; i < k - 1; ++i) reach += (n[i] - 1) * s[i];
  const auto floor_div = [](int64_t x, int64_t d) { return x / d - (x % d < 0); };
  const int64_t lo = std::max(-last, -floor_div(reach + r, step)), hi = std::min(last, floor_div(reach - r, step));
  for (int64_t d = lo; d <= hi; ++d)
    if (--*tries < 0 || meets(n, s, k - 1, r + d * step, moved || d != 0, dim, tries)) return true;
  return false;
}

// Whether two rows of dim elements at i * sb + j * st + l * sh share memory.
bool rows_overlap(int64_t outer, int64_t sb, int64_t tokens, int64_t st, int64_t heads, int64_t sh, int64_t dim) {
  int64_t n[3] = {outer, tokens, heads}, s[3] = {outer > 1 ? sb : 0, tokens > 1 ? st : 0, heads > 1 ? sh : 0};
  for (const auto &[i, j] : {std::pair{0, 1}, std::pair{1, 2}, std::pair{0, 1}})
    if (s[i] > s[j]) std::swap(s[i], s[j]), std::swap(n[i], n[j]);
  int tries = 1 << 16;
  return meets(n, s, 3, 0, false, dim, &tries);
}

// A tensor [batch][tokens][heads][dim] as the kernels take it.  `outer` is the
// number of sequences or pages.  Strides of an extent of one do not matter.
spmm_status_t view(const char *fn, const char *name, const spmm_attn_tensor_t *t, int64_t outer, int64_t tokens,
                   int64_t heads, int64_t dim, bool written, bool keys, AttnView *v) {
  *v = AttnView{nullptr, 0, 0, 0};
  if (!t) return bad(fn, std::string(name) + " is NULL");
  if (outer == 0 || tokens == 0) return SPMM_OK;  // holds nothing
  if (!t->data) return bad(fn, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(t->data) & 15u) return bad(fn, std::string(name) + " is not 16-byte aligned");
  const int64_t sb = outer > 1 ? t->stride_batch : 0, st = tokens > 1 ? t->stride_token : dim,
                sh = heads > 1 ? t->stride_head : 0;
  if (sb < 0 || st < 0 || sh < 0 || sb % 8 || st % 8 || sh % 8)
    return bad(fn, std::string(name) + ": strides must be multiples of 8 elements, none negative");
  const int64_t most = int64_t(1) << 60;
  if (sb > most / kElem / std::max<int64_t>(1, outer) || st > most / kElem / std::max<int64_t>(1, tokens) ||
      sh > most / kElem / std::max<int64_t>(1, heads))
    return bad(fn, std::string(name) + ": strides too large");
  if (written && rows_overlap(outer, sb, tokens, st, heads, sh, dim))
    return bad(fn, std::string(name) + " is written: its rows must not overlap");
  // the kernels bound a block's rows by their byte offset from its first one
  if (keys && (st < dim || st * kElem * kAttnPage >= (int64_t(1) << 31)))
    return fail(SPMM_ERR_UNSUPPORTED, std::string(fn) + ": " + name +
                                          ": the token stride must be at least dim and below 16 Mi elements");
  v->p = static_cast<char *>(t->data);
  v->sb = sb * kElem;
  v->st = st * kElem;
  v->sh = sh * kElem;
  return SPMM_OK;
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

spmm_status_t whole(const char *fn, const char *name, const void *p, uintptr_t to, bool needed) {
  if (!p && needed) return bad(fn, std::string(name) + " is NULL");
  if (!aligned(p, to)) return bad(fn, std::string(name) + " is not aligned to its elements");
  return SPMM_OK;
}

spmm_status_t attn_plan_of(const char *fn, spmm_plan_t p) {
  if (!p) return bad(fn, "plan is NULL");
  if (!p->attn) return bad(fn, "plan is not an attention plan");
  return SPMM_OK;
}

// number of pages, for a call with a table
spmm_status_t pages_of(const char *fn, const AttnArgs &a, const int32_t *table, int64_t pages, int64_t *outer) {
  *outer = a.b;
  if (!table) return SPMM_OK;
  if (pages < 0 || pages > INT32_MAX) return bad(fn, "pages must be 0 .. 2^31 - 1");
  *outer = pages;
  return SPMM_OK;
}

#define ATTN_TRY(call)                       \
  do {                                       \
    const spmm_status_t s_ = (call);         \
    if (s_ != SPMM_OK) return s_;            \
  } while (0)

spmm_status_t launched(hipError_t e) { return e == hipSuccess ? SPMM_OK : hip_fail(e, "kernel launch"); }

void attn_log(const spmm_plan_s *p) {
  const spmm_plan_info_t &i = p->info;
  const AttnArgs &a = p->attn_args;
  std::fprintf(stderr,
               "[spmm] spmm_plan_attn: format=attn device=%d m=%lld k=%lld n=%lld kernel=attn_forward%s "
               "rows=%d row_tiles=%d ranges=%d/%d chunk=%d tile=%dx%d grid=%lld device_bytes=%lld "
               "workspace_bytes=%lld\n",
               static_cast<int>(i.device), static_cast<long long>(i.m), static_cast<long long>(i.k),
               static_cast<long long>(i.n), p->attn_desc.backward ? "+attn_dq+attn_dkv" : "",
               static_cast<int>(a.rows), static_cast<int>(a.rtiles), static_cast<int>(p->attn_split_listed[0]),
               static_cast<int>(p->attn_split_all[0]), static_cast<int>(a.chunk), static_cast<int>(i.tile_m),
               static_cast<int>(i.tile_n), static_cast<long long>(i.grid), static_cast<long long>(i.device_bytes),
               static_cast<long long>(i.workspace_bytes));
  std::fflush(stderr);
}

}  // namespace

void attn_split(int64_t tiles, int32_t tile_rows, int32_t entries, int32_t max_entries, int32_t *nsplit,
                int32_t *per_split) {
  // 4096 workgroups to fill the chip and even out ragged lengths, but no more
  // than 48k rows of partial sums (24 drafted tokens over 16 sequences of up to
  // 8k: 4 ranges 113 us, 8 127 us, 16 146 us; 48 over 8 sequences: 2 121 us, 4 87
  // us, 8 104 us; over 105 shapes, 4 to 64 tokens of 1 to 32 sequences of up to
  // 4k, 8k and 20k, at most 1.05 times the best of caps from 12k up in 73 and 1.1
  // times in 91, at worst 1.44, where 32 sequences of 64 tokens stay whole), and
  // at least eight blocks a range (64 lists of 32 blocks: 108 us, with four
  // blocks 120 us), or four where that leaves CUs without work.
  tiles = std::max<int64_t>(1, tiles);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(4096 / tiles, 49152 / (tiles * tile_rows)));
  // What ranges gain: 0.35 us a block where four waves share up to 32 rows'
  // list, 0.7, 1.1 and 1.65 us with 64, 128 and 256 rows.  What they cost: a
  // merge 4 us, and a row's partial sums in each range 0.25 ns.  A prompt of 1024
  // tokens, 16 heads over 8, 16 blocks a query takes 24 us whole and 35 us in 3
  // ranges; 24 drafted tokens over two sequences of 1000 keys, 23 us whole and
  // 17 us in 4.
  const double block = tile_rows <= 32 ? 0.35 : (tile_rows <= 64 ? 0.7 : (tile_rows <= 128 ? 1.1 : 1.65));
  auto gain = [&](int64_t p) {
    const int64_t ranges = (max_entries + p - 1) / p;
    return static_cast<double>(entries - p) * block - 4.0 - static_cast<double>(ranges * tiles * tile_rows) * 0.25e-3;
  };
  int64_t per = std::max<int64_t>(1, max_entries);
  if (tile_rows <= 32) {
    int64_t p = std::max<int64_t>(4, (max_entries + want - 1) / want);
    if (p < 8 && tiles * ((int64_t{max_entries} + 7) / 8) >= 512) p = 8;
    if (entries > 16 && gain(p) > 0.0) per = p;
  } else {
    double best = 0.0;
    for (int64_t n = 2; n <= want; ++n) {
      const int64_t p = std::max<int64_t>(4, (max_entries + n - 1) / n);
      if (const double x = gain(p); x > best) best = x, per = p;
      if (p == 4) break;
    }
  }
  *nsplit = static_cast<int32_t>(std::max<int64_t>(1, (max_entries + per - 1) / per));
  *per_split = static_cast<int32_t>(per);
}

spmm_status_t attn_shape(const spmm_attn_desc_t &d, spmm_plan_s *p) {
  const char *fn = "spmm_plan_attn";
  if (d.batch < 0 || d.queries < 0 || d.keys < 0 || d.batch > INT32_MAX || d.queries > INT32_MAX - 256 ||
      d.keys > INT32_MAX - 256)
    return bad(fn, "batch, queries and keys must be 0 .. 2^31 - 257");
  if (d.heads_q < 1 || d.heads_kv < 1 || d.heads_q % d.heads_kv != 0)
    return bad(fn, "heads_q must be a multiple of heads_kv");
  if (d.q_block < 1 || d.max_blocks < 1 || d.sink_blocks < 0 || d.local_blocks < 1)
    return bad(fn, "q_block, max_blocks and local_blocks must be positive, sink_blocks not negative");
  if (!(d.scale >= 0.0f) || std::isinf(d.scale)) return bad(fn, "scale must be positive, or 0 for 1 / sqrt(dim)");
  if (d.backward != 0 && d.backward != 1) return bad(fn, "backward must be 0 or 1");
  if (d.dtype != SPMM_BF16 && d.dtype != SPMM_F16)
    return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: bf16 or f16 only");
  if (d.dim != 64 && d.dim != 128) return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: dim must be 64 or 128");
  if (!power_of_two(d.q_block) || d.q_block > 64)
    return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: q_block must be 1, 2, 4, .. 64");
  // positions and the last key of a row tile are counted in 32 bits
  if (d.queries + d.keys > INT32_MAX - 512)
    return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: queries + keys above 2^31 - 513");
  // the kernels step through lists by up to 256 entries in 32 bits
  if (d.max_blocks > kMaxEntries) return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: max_blocks above 2^30");
  if (d.heads_q > 65536) return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: more than 65536 query heads");

  p->attn = true;
  p->attn_desc = d;
  AttnArgs &a = p->attn_args;
  a = AttnArgs{};
  a.b = static_cast<int32_t>(d.batch);
  a.nq = static_cast<int32_t>(d.queries);
  a.nk = static_cast<int32_t>(d.keys);
  a.hq = d.heads_q;
  a.hk = d.heads_kv;
  a.group = d.heads_q / d.heads_kv;
  a.q_block = d.q_block;
  a.nqb = (a.nq + d.q_block - 1) / d.q_block;
  a.nkb = (a.nk + kAttnPage - 1) / kAttnPage;
  a.max_blocks = d.max_blocks;
  a.scale = d.scale > 0.0f ? d.scale : 1.0f / std::sqrt(static_cast<float>(d.dim));
  a.rows = std::min(a.q_block, std::max(a.nq, 1)) * a.group;
  const AttnTile t = attn_tile(a.rows, a.nqb);
  a.rtiles = (a.rows + t.rows - 1) / t.rows;
  const double tiles = static_cast<double>(a.b) * a.hk * a.nqb * a.rtiles;
  if (tiles > 0x7fffffff || static_cast<double>(a.b) * a.hk * a.nkb > 0x7fffffff ||
      static_cast<double>(a.b) * a.hq * a.nq > static_cast<double>(int64_t(1) << 40))
    return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: more workgroups than a launch holds");
  const int64_t n = static_cast<int64_t>(tiles);
  const int32_t rows = std::min(a.rows, t.rows);
  attn_split(n, rows, std::min(a.max_blocks, a.nkb), a.max_blocks, &p->attn_split_listed[0], &p->attn_split_listed[1]);
  attn_split(n, rows, a.nkb, a.nkb, &p->attn_split_all[0], &p->attn_split_all[1]);
  if (d.backward) {
    const int64_t entries = static_cast<int64_t>(a.nqb) * a.max_blocks;
    if (entries > INT32_MAX)
      return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: lists of a head hold more than 2^31 - 1 entries");
    attn_chunks(static_cast<int64_t>(a.b) * a.hk, entries, a.nqb, a.rows, a.nkb, &a.chunk, &a.slots);
    if (static_cast<double>(a.b) * a.hk * (static_cast<double>(a.nqb) * 2 * a.rtiles + a.nkb) > 0x7fffffff ||
        static_cast<double>(a.b) * a.hk * std::max<double>(a.slots, 16.0 * a.nkb) > 0x7fffffff)
      return fail(SPMM_ERR_UNSUPPORTED, "spmm_plan_attn: more workgroups than a launch holds");
  }
  p->info.format = SPMM_FORMAT_ATTN;
  p->info.m = d.batch * d.queries;
  p->info.k = d.keys;
  p->info.n = d.dim;
  p->info.tile_m = t.rows;
  p->info.tile_n = t.key_tile;
  p->info.grid = n * p->attn_split_listed[0];
  return SPMM_OK;
}

namespace {

spmm_status_t plan_attn(spmm_plan_s *p) {
  AttnArgs &a = p->attn_args;
  const spmm_attn_desc_t &d = p->attn_desc;
  const int64_t rows = static_cast<int64_t>(a.b) * a.hq * a.nq;
  int64_t ranges = std::max(p->attn_split_listed[0], p->attn_split_all[0]);
  if (ranges == 1) ranges = 0;
  void *ptr = nullptr;
  ATTN_TRY(plan_workspace(p, static_cast<size_t>(ranges * rows * d.dim * 4), &ptr));
  a.part_o = static_cast<float *>(ptr);
  ATTN_TRY(plan_workspace(p, static_cast<size_t>(ranges * rows * 8), &ptr));
  a.part_ml = static_cast<float *>(ptr);
  if (!d.backward) return SPMM_OK;
  const int64_t heads = static_cast<int64_t>(a.b) * a.hk;
  ATTN_TRY(plan_workspace(p, static_cast<size_t>((rows + 1) * 8), &ptr));
  a.stats = static_cast<float *>(ptr);
  ATTN_TRY(plan_workspace(p, static_cast<size_t>(heads * a.nqb * a.max_blocks * 4), &ptr));
  a.inv_ids = static_cast<int32_t *>(ptr);
  ATTN_TRY(plan_workspace(p, static_cast<size_t>(heads * a.nkb * 8), &ptr));
  a.inv_ptr = static_cast<int32_t *>(ptr);
  ATTN_TRY(plan_workspace(p, 8 * 4, &ptr));
  a.queue = static_cast<int32_t *>(ptr);
  ATTN_TRY(plan_workspace(p, static_cast<size_t>(heads * a.slots * 8), &ptr));
  a.items = static_cast<int32_t *>(ptr);
  if (a.slots > a.nkb) {
    ATTN_TRY(plan_workspace(p, static_cast<size_t>(heads * a.slots * 2 * kAttnPage * d.dim * 4), &ptr));
    a.part_kv = static_cast<float *>(ptr);
  }
  return SPMM_OK;
}

// q, k, v, o, lse and the lengths: what the forward calls share
spmm_status_t forward_args(const char *fn, spmm_plan_t p, const spmm_attn_tensor_t *q, const spmm_attn_tensor_t *k,
                           const spmm_attn_tensor_t *v, int64_t outer, int64_t tokens, const spmm_attn_tensor_t *o,
                           bool o_written, float *lse, const int32_t *lens, const int32_t *starts, AttnArgs *a) {
  const int64_t dim = p->attn_desc.dim;
  ATTN_TRY(view(fn, "q", q, a->b, a->nq, a->hq, dim, false, false, &a->q));
  ATTN_TRY(view(fn, "k", k, outer, tokens, a->hk, dim, false, true, &a->k));
  ATTN_TRY(view(fn, "v", v, outer, tokens, a->hk, dim, false, true, &a->v));
  ATTN_TRY(view(fn, "o", o, a->b, a->nq, a->hq, dim, o_written, false, &a->o));
  ATTN_TRY(whole(fn, "lse", lse, 4, static_cast<int64_t>(a->b) * a->nq > 0));
  ATTN_TRY(whole(fn, "lens", lens, 4, false));
  ATTN_TRY(whole(fn, "starts", starts, 4, false));
  a->lse = lse;
  a->lens = lens;
  a->starts = starts;
  return SPMM_OK;
}

}  // namespace
}  // namespace sdm

using namespace sdm;

extern "C" {

spmm_status_t spmm_plan_attn(const spmm_attn_desc_t *desc, int32_t device, spmm_plan_t *out) {
  alloc_hook_begin();
  if (!out) return fail(SPMM_ERR_INVALID_ARG, "spmm_plan_attn: out is NULL");
  *out = nullptr;
  if (!desc) return fail(SPMM_ERR_INVALID_ARG, "spmm_plan_attn: desc is NULL");
  return guarded([&]() -> spmm_status_t {
    if (alloc_hook_fail()) throw std::bad_alloc();
    auto *p = new spmm_plan_s();
    p->device = device;
    p->info.device = device;
    spmm_status_t s = SPMM_ERR_INTERNAL;
    try {
      s = attn_shape(*desc, p);
      if (s == SPMM_OK) {
        int ndev = 0;
        hipError_t e = hipGetDeviceCount(&ndev);
        if (e != hipSuccess) s = hip_fail(e, "hipGetDeviceCount");
        else if (device < 0 || device >= ndev) s = fail(SPMM_ERR_INVALID_ARG, "spmm_plan_attn: no such device");
      }
      if (s == SPMM_OK) {
        DeviceScope ds(device);
        s = ds.err != hipSuccess ? hip_fail(ds.err, "hipSetDevice") : plan_attn(p);
      }
    } catch (...) {
      free_plan(p);
      throw;
    }
    if (s != SPMM_OK) {
      free_plan(p);
      return s;
    }
    *out = p;
    if (plan_log_on()) attn_log(p);
    return SPMM_OK;
  });
}

spmm_status_t spmm_execute_attn_pool(spmm_plan_t p, const spmm_attn_tensor_t *k, int64_t pages, int8_t *pooled_dev,
                                     float *scale_dev, const int32_t *table, const int32_t *lens,
                                     const int32_t *first, hipStream_t stream) {
  const char *fn = "spmm_execute_attn_pool";
  return guarded([&]() -> spmm_status_t {
    ATTN_TRY(attn_plan_of(fn, p));
    const AttnArgs &a = p->attn_args;
    int64_t outer = 0;
    ATTN_TRY(pages_of(fn, a, table, pages, &outer));
    AttnPoolArgs x{};
    ATTN_TRY(view(fn, "k", k, outer, table ? kAttnPage : a.nk, a.hk, p->attn_desc.dim, false, true, &x.k));
    const bool some = outer > 0 && a.nkb > 0;
    ATTN_TRY(whole(fn, "pooled", pooled_dev, 16, some));
    ATTN_TRY(whole(fn, "pooled_scale", scale_dev, 4, some));
    ATTN_TRY(whole(fn, "table", table, 4, false));
    ATTN_TRY(whole(fn, "lens", lens, 4, false));
    ATTN_TRY(whole(fn, "first", first, 4, false));
    x.pooled = pooled_dev;
    x.pooled_scale = scale_dev;
    x.table = table;
    x.lens = lens;
    x.first = first;
    x.b = a.b;
    x.nk = a.nk;
    x.hk = a.hk;
    x.nkb = a.nkb;
    x.pages = static_cast<int32_t>(pages);
    // the blocks that nq tokens from `first` on can lie in
    x.width = first ? static_cast<int32_t>(std::min<int64_t>(a.nkb, (static_cast<int64_t>(a.nq) + kAttnPage - 2) / kAttnPage + 1)) : a.nkb;
    if (!some || a.b == 0) return SPMM_OK;
    DeviceScope ds(p->device);
    if (ds.err != hipSuccess) return hip_fail(ds.err, "hipSetDevice");
    return launched(launch_attn_pool(x, static_cast<spmm_dtype_t>(p->attn_desc.dtype), p->attn_desc.dim, stream));
  });
}

spmm_status_t spmm_execute_attn_select(spmm_plan_t p, const spmm_attn_tensor_t *q, const int8_t *pooled_dev,
                                       const float *scale_dev, int64_t pages, int32_t *lists_dev,
                                       const int32_t *table, const int32_t *lens, const int32_t *starts,
                                       hipStream_t stream) {
  const char *fn = "spmm_execute_attn_select";
  return guarded([&]() -> spmm_status_t {
    ATTN_TRY(attn_plan_of(fn, p));
    const AttnArgs &a = p->attn_args;
    int64_t outer = 0;
    ATTN_TRY(pages_of(fn, a, table, pages, &outer));
    AttnSelectArgs x{};
    ATTN_TRY(view(fn, "q", q, a.b, a.nq, a.hq, p->attn_desc.dim, false, false, &x.q));
    const bool some = static_cast<int64_t>(a.b) * a.nq > 0;
    ATTN_TRY(whole(fn, "pooled", pooled_dev, 16, some && outer > 0 && a.nkb > 0));
    ATTN_TRY(whole(fn, "pooled_scale", scale_dev, 4, some && outer > 0 && a.nkb > 0));
    ATTN_TRY(whole(fn, "lists", lists_dev, 4, some));
    ATTN_TRY(whole(fn, "table", table, 4, false));
    ATTN_TRY(whole(fn, "lens", lens, 4, false));
    ATTN_TRY(whole(fn, "starts", starts, 4, false));
    if (static_cast<int64_t>(p->attn_desc.sink_blocks) + p->attn_desc.local_blocks > a.max_blocks)
      return bad(fn, "sink_blocks + local_blocks must be at most max_blocks");
    if (a.nkb > kAttnMaxScored)
      return fail(SPMM_ERR_UNSUPPORTED, "spmm_execute_attn_select: more than 32768 blocks a sequence");
    x.pooled = pooled_dev;
    x.pooled_scale = scale_dev;
    x.lists = lists_dev;
    x.table = table;
    x.lens = lens;
    x.starts = starts;
    x.b = a.b;
    x.nq = a.nq;
    x.nk = a.nk;
    x.hq = a.hq;
    x.hk = a.hk;
    x.group = a.group;
    x.q_block = a.q_block;
    x.nqb = a.nqb;
    x.nkb = a.nkb;
    x.max_blocks = a.max_blocks;
    x.pages = static_cast<int32_t>(pages);
    x.sink = p->attn_desc.sink_blocks;
    x.local = p->attn_desc.local_blocks;
    if (!some) return SPMM_OK;
    DeviceScope ds(p->device);
    if (ds.err != hipSuccess) return hip_fail(ds.err, "hipSetDevice");
    return launched(launch_attn_select(x, static_cast<spmm_dtype_t>(p->attn_desc.dtype), p->attn_desc.dim, stream));
  });
}

spmm_status_t spmm_execute_attn(spmm_plan_t p, const spmm_attn_tensor_t *q, const spmm_attn_tensor_t *k,
                                const spmm_attn_tensor_t *v, const int32_t *lists_dev, const spmm_attn_tensor_t *o,
                                float *lse_dev, const int32_t *lens, const int32_t *starts, hipStream_t stream) {
  const char *fn = "spmm_execute_attn";
  return guarded([&]() -> spmm_status_t {
    ATTN_TRY(attn_plan_of(fn, p));
    AttnArgs a = p->attn_args;
    ATTN_TRY(forward_args(fn, p, q, k, v, a.b, a.nk, o, true, lse_dev, lens, starts, &a));
    const bool some = static_cast<int64_t>(a.b) * a.nq > 0;
    ATTN_TRY(whole(fn, "lists", lists_dev, 4, some));
    if (!some) return SPMM_OK;
    a.lists = lists_dev;
    a.entries = a.max_blocks;
    a.nsplit = p->attn_split_listed[0];
    a.per_split = p->attn_split_listed[1];
    DeviceScope ds(p->device);
    if (ds.err != hipSuccess) return hip_fail(ds.err, "hipSetDevice");
    return launched(launch_attn_forward(a, static_cast<spmm_dtype_t>(p->attn_desc.dtype), p->attn_desc.dim, stream));
  });
}

spmm_status_t spmm_execute_attn_backward(spmm_plan_t p, const spmm_attn_tensor_t *grad, const spmm_attn_tensor_t *q,
                                         const spmm_attn_tensor_t *k, const spmm_attn_tensor_t *v,
                                         const int32_t *lists_dev, const spmm_attn_tensor_t *o, const float *lse_dev,
                                         const spmm_attn_tensor_t *dq, const spmm_attn_tensor_t *dk,
                                         const spmm_attn_tensor_t *dv, const int32_t *lens, const int32_t *starts,
                                         hipStream_t stream) {
  const char *fn = "spmm_execute_attn_backward";
  return guarded([&]() -> spmm_status_t {
    ATTN_TRY(attn_plan_of(fn, p));
    if (!p->attn_desc.backward) return bad(fn, "the plan was made without backward");
    AttnArgs a = p->attn_args;
    const int64_t dim = p->attn_desc.dim;
    ATTN_TRY(forward_args(fn, p, q, k, v, a.b, a.nk, o, false, const_cast<float *>(lse_dev), lens, starts, &a));
    ATTN_TRY(view(fn, "grad", grad, a.b, a.nq, a.hq, dim, false, false, &a.g));
    ATTN_TRY(view(fn, "dq", dq, a.b, a.nq, a.hq, dim, true, false, &a.dq));
    ATTN_TRY(view(fn, "dk", dk, a.b, a.nk, a.hk, dim, true, false, &a.dk));
    ATTN_TRY(view(fn, "dv", dv, a.b, a.nk, a.hk, dim, true, false, &a.dv));
    ATTN_TRY(whole(fn, "lists", lists_dev, 4, static_cast<int64_t>(a.b) * a.nq > 0));
    for (const AttnView *x : {&a.q, &a.g})
      if (a.nq > 0 && (a.nq - 1) * x->st + (a.hq - 1) * x->sh + dim * kElem > kMaxRowOffset)
        return fail(SPMM_ERR_UNSUPPORTED, std::string(fn) + ": q or grad of a sequence spans 4 GiB or more");
    if (a.b == 0 || (a.nq == 0 && a.nk == 0)) return SPMM_OK;
    a.lists = lists_dev;
    a.entries = a.max_blocks;
    a.nsplit = 1;
    a.per_split = a.max_blocks;
    DeviceScope ds(p->device);
    if (ds.err != hipSuccess) return hip_fail(ds.err, "hipSetDevice");
    return launched(launch_attn_backward(a, static_cast<spmm_dtype_t>(p->attn_desc.dtype), p->attn_desc.dim, stream));
  });
}

spmm_status_t spmm_execute_attn_cache(spmm_plan_t p, const spmm_attn_tensor_t *q, const spmm_attn_tensor_t *k,
                                      const spmm_attn_tensor_t *v, int64_t pages, const spmm_attn_tensor_t *o,
                                      float *lse_dev, const int32_t *table, const int32_t *lists_dev,
                                      const uint64_t *tree, const int32_t *lens, const int32_t *starts,
                                      hipStream_t stream) {
  const char *fn = "spmm_execute_attn_cache";
  return guarded([&]() -> spmm_status_t {
    ATTN_TRY(attn_plan_of(fn, p));
    AttnArgs a = p->attn_args;
    int64_t outer = 0;
    ATTN_TRY(pages_of(fn, a, table, pages, &outer));
    ATTN_TRY(forward_args(fn, p, q, k, v, outer, table ? kAttnPage : a.nk, o, true, lse_dev, lens, starts, &a));
    ATTN_TRY(whole(fn, "table", table, 4, false));
    ATTN_TRY(whole(fn, "lists", lists_dev, 4, false));
    ATTN_TRY(whole(fn, "tree", tree, 8, false));
    if (tree && a.nq > 64) return fail(SPMM_ERR_UNSUPPORTED, std::string(fn) + ": a tree holds at most 64 tokens");
    if (static_cast<int64_t>(a.b) * a.nq == 0) return SPMM_OK;
    a.table = table;
    a.pages = static_cast<int32_t>(pages);
    a.lists = lists_dev;
    a.tree = tree;
    a.entries = lists_dev ? a.max_blocks : a.nkb;
    const int32_t *split = lists_dev ? p->attn_split_listed : p->attn_split_all;
    a.nsplit = split[0];
    a.per_split = split[1];
    DeviceScope ds(p->device);
    if (ds.err != hipSuccess) return hip_fail(ds.err, "hipSetDevice");
    return launched(launch_attn_forward(a, static_cast<spmm_dtype_t>(p->attn_desc.dtype), p->attn_desc.dim, stream));
  });
}

}  // extern "C"
