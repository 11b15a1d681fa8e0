// Host-side checks of the attention calls: the rules that the kernels share
// with the host, the plan's decisions, and the refusals of the execute calls
// on a plan without a device.  Input on stdin, one query per line:
//   plan <b nq nk hq hk d q_block blocks backward>  -> "<status> rows rtiles tile nsplit per_split chunk slots"
//   len <n nk>            -> length taken
//   start <s nq nk>       -> position taken
//   page <id pages p0 ..> -> page of block id of a table
//   names <id last_key>   -> 0 or 1
//   refuse <case>         -> "<status> <message>"
//   written <b nq hq sb st sh>  -> message for an output of these extents and strides (lse is missing too)
#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

#include "../sparse_dense_matrix_amd/csrc/internal.h"

namespace {

alignas(64) char memory[4096];  // never read: every call below is refused, or has nothing to do

spmm_attn_desc_t shape(int64_t b, int64_t nq, int64_t nk) {
  spmm_attn_desc_t d{};
  d.batch = b;
  d.queries = nq;
  d.keys = nk;
  d.heads_q = 4;
  d.heads_kv = 2;
  d.dim = 64;
  d.dtype = SPMM_BF16;
  d.q_block = 16;
  d.max_blocks = 4;
  d.sink_blocks = 1;
  d.local_blocks = 1;
  d.backward = 1;
  return d;
}

spmm_attn_tensor_t heads(int64_t tokens, int64_t n) {
  return {memory, tokens * n * 64, n * 64, 64};
}

spmm_status_t refuse(const std::string &what) {
  spmm_plan_s p;
  spmm_attn_desc_t d = shape(2, 32, 128);
  if (what == "select_short_list") d.sink_blocks = 4;
  if (what == "select_long") d.keys = 64 * 40000;
  if (what == "tree_long") d.queries = 65;
  if (what == "nothing") d = shape(0, 32, 128);
  if (what == "no_backward") d.backward = 0;
  const spmm_status_t s = sdm::attn_shape(d, &p);
  if (s != SPMM_OK) return s;
  const int64_t nq = d.queries;
  spmm_attn_tensor_t q = heads(nq, 4), o = q, g = q, dq = q, k = heads(d.keys, 2), v = k, dk = k, dv = k;
  float *f = reinterpret_cast<float *>(memory);
  int32_t *lists = reinterpret_cast<int32_t *>(memory);
  int8_t *pooled = reinterpret_cast<int8_t *>(memory);
  int64_t pages = 4;
  int32_t *table = nullptr;
  const uint64_t *tree = nullptr;
  const int32_t *lens = nullptr;
  if (what == "q_null") q.data = nullptr;
  if (what == "q_odd") q.data = memory + 2;
  if (what == "q_stride_odd") q.stride_token = 4 * 64 + 4;
  if (what == "q_stride_negative") q.stride_head = -64;
  if (what == "q_stride_huge") q.stride_batch = int64_t(1) << 61;
  if (what == "k_stride_short") k.stride_token = 56;
  if (what == "k_stride_wide") k.stride_token = int64_t(1) << 25;
  if (what == "o_overlaps") o.stride_token = 0;
  if (what == "o_heads_overlap") o.stride_head = 32;
  if (what == "lens_odd") lens = reinterpret_cast<int32_t *>(memory + 2);
  if (what == "lse_null") f = nullptr;
  if (what == "lists_null") lists = nullptr;
  if (what == "pages_negative" || what == "pages_huge") {
    table = reinterpret_cast<int32_t *>(memory);
    pages = what == "pages_huge" ? int64_t(1) << 31 : -1;
    return spmm_execute_attn_cache(&p, &q, &k, &v, pages, &o, f, table, nullptr, nullptr, lens, nullptr, nullptr);
  }
  if (what == "tree_long") {
    tree = reinterpret_cast<const uint64_t *>(memory);
    return spmm_execute_attn_cache(&p, &q, &k, &v, 0, &o, f, nullptr, nullptr, tree, lens, nullptr, nullptr);
  }
  if (what == "tree_odd") {
    tree = reinterpret_cast<const uint64_t *>(memory + 4);
    return spmm_execute_attn_cache(&p, &q, &k, &v, 0, &o, f, nullptr, nullptr, tree, lens, nullptr, nullptr);
  }
  if (what.rfind("select", 0) == 0) return spmm_execute_attn_select(&p, &q, pooled, f, 0, lists, nullptr, lens, nullptr, nullptr);
  if (what == "pool_odd") return spmm_execute_attn_pool(&p, &k, 0, pooled + 8, f, nullptr, lens, nullptr, nullptr);
  if (what == "q_null_tensor") return spmm_execute_attn(&p, nullptr, &k, &v, lists, &o, f, lens, nullptr, nullptr);
  if (what == "no_plan") return spmm_execute_attn(nullptr, &q, &k, &v, lists, &o, f, lens, nullptr, nullptr);
  if (what == "other_plan") {
    spmm_plan_s other;
    return spmm_execute_attn(&other, &q, &k, &v, lists, &o, f, lens, nullptr, nullptr);
  }
  if (what == "execute") return spmm_execute(&p, memory, 64, memory, 64, nullptr);
  if (what == "no_backward" || what.rfind("dq", 0) == 0 || what.rfind("dk", 0) == 0 || what == "g_wide") {
    if (what == "dq_null") dq.data = nullptr;
    if (what == "dk_broadcast") dk.stride_head = 0;
    if (what == "g_wide") g.stride_token = int64_t(1) << 30;
    return spmm_execute_attn_backward(&p, &g, &q, &k, &v, lists, &o, f, &dq, &dk, &dv, lens, nullptr, nullptr);
  }
  return spmm_execute_attn(&p, &q, &k, &v, lists, &o, f, lens, nullptr, nullptr);
}

}  // namespace

int main() {
  char what[64];
  while (std::scanf("%63s", what) == 1) {
    if (!std::strcmp(what, "plan")) {
      long long b, nq, nk;
      spmm_attn_desc_t d = shape(1, 1, 1);
      if (std::scanf("%lld %lld %lld %d %d %d %d %d %d", &b, &nq, &nk, &d.heads_q, &d.heads_kv, &d.dim, &d.q_block,
                     &d.max_blocks, &d.backward) != 9)
        return 2;
      d.batch = b;
      d.queries = nq;
      d.keys = nk;
      spmm_plan_s p;
      const spmm_status_t s = sdm::attn_shape(d, &p);
      const sdm::AttnArgs &a = p.attn_args;
      if (s == SPMM_OK)
        std::printf("%s %d %d %d %d %d %d %d\n", spmm_status_str(s), a.rows, a.rtiles, static_cast<int>(p.info.tile_m),
                    p.attn_split_listed[0], p.attn_split_listed[1], a.chunk, a.slots);
      else
        std::printf("%s\n", spmm_status_str(s));
    } else if (!std::strcmp(what, "len")) {
      int n, nk;
      if (std::scanf("%d %d", &n, &nk) != 2) return 2;
      std::printf("%d\n", sdm::attn_len(&n, 0, nk));
    } else if (!std::strcmp(what, "start")) {
      int s, nq, nk;
      if (std::scanf("%d %d %d", &s, &nq, &nk) != 3) return 2;
      std::printf("%d\n", sdm::attn_start(&s, 0, nq, nk));
    } else if (!std::strcmp(what, "page")) {
      int id, pages, n;
      if (std::scanf("%d %d %d", &id, &pages, &n) != 3 || n < 0) return 2;
      std::vector<int32_t> t(static_cast<size_t>(n));
      for (int32_t &x : t)
        if (std::scanf("%d", &x) != 1) return 2;
      std::printf("%d\n", sdm::attn_page(n ? t.data() : nullptr, id, pages));
    } else if (!std::strcmp(what, "names")) {
      int id, last;
      if (std::scanf("%d %d", &id, &last) != 2) return 2;
      std::printf("%d\n", sdm::attn_names(id, last) ? 1 : 0);
    } else if (!std::strcmp(what, "refuse")) {
      if (std::scanf("%63s", what) != 1) return 2;
      const spmm_status_t s = refuse(what);
      std::printf("%s %s\n", spmm_status_str(s), s == SPMM_OK ? "" : spmm_last_error());
    } else if (!std::strcmp(what, "written")) {
      long long b, nq, sb, st, sh;
      spmm_attn_desc_t d = shape(1, 1, 128);
      if (std::scanf("%lld %lld %d %lld %lld %lld", &b, &nq, &d.heads_q, &sb, &st, &sh) != 6) return 2;
      d.batch = b;
      d.queries = nq;
      d.heads_kv = 1;
      spmm_plan_s p;
      if (sdm::attn_shape(d, &p) != SPMM_OK) return 2;
      const spmm_attn_tensor_t q = heads(nq, d.heads_q), k = heads(128, 1), o = {memory, sb, st, sh};
      const spmm_status_t s = spmm_execute_attn(&p, &q, &k, &k, reinterpret_cast<int32_t *>(memory), &o, nullptr,
                                                nullptr, nullptr, nullptr);
      std::printf("%s\n", s == SPMM_OK ? "" : spmm_last_error());
    } else {
      return 2;
    }
    std::fflush(stdout);
  }
  return 0;
}
