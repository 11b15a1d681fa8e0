// Refusals of the calls around attention over a cache in 8 bits, on plans
// without a device.  Input on stdin: a case a line; output "<status> <message>".
#include <cmath>
#include <cstdio>
#include <cstring>
#include <string>

#include "../sparse_dense_matrix_amd/csrc/internal.h"

namespace {

alignas(64) char memory[4096];  // never read: every call below is refused, or has nothing to do

spmm_status_t cache_calls(const std::string &call, const std::string &what) {
  spmm_attn_desc_t d{};
  d.batch = what == "nothing" ? 0 : 2;
  d.queries = what == "tree_long" ? 65 : 32;
  d.keys = 128;
  d.heads_q = 4;
  d.heads_kv = 2;
  d.dim = 64;
  d.dtype = SPMM_BF16;
  d.q_block = 16;
  d.max_blocks = 4;
  d.sink_blocks = d.local_blocks = 1;
  if (what == "many_rows") {
    d.batch = 1 << 20;
    d.queries = d.keys = call == "read" ? 1 << 15 : 1 << 14;
    d.heads_q = d.heads_kv = call == "read" ? 2 : 4;
    d.q_block = 64;
  }
  if (what == "rows_launch") d.batch = 1 << 26, d.queries = 1, d.heads_q = d.heads_kv = 8;  // 2^24 times 32 rows
  if (what == "blocks_launch") d.batch = 1 << 20, d.queries = call == "read" ? 1 : 128, d.keys = 256, d.heads_q = d.heads_kv = 8;
  spmm_plan_s p;
  const spmm_status_t s = sdm::attn_shape(d, &p);
  if (s != SPMM_OK) return s;
  const int64_t hk = d.heads_kv;
  spmm_attn_tensor_t q = {memory, d.queries * d.heads_q * 64, d.heads_q * 64, 64}, o = q;
  spmm_attn_tensor_t k = {memory, d.queries * hk * 64, hk * 64, 64}, v = k;
  spmm_attn_tensor_t kf = {memory, d.keys * hk * 64, hk * 64, 64}, vf = kf;  // of the whole sequence
  spmm_attn_tensor_t k8 = {memory, d.keys * hk * 64, hk * 64, 64}, v8 = k8;
  float *ks = reinterpret_cast<float *>(memory), *vs = ks, *lse = ks;
  int8_t *pooled = reinterpret_cast<int8_t *>(memory);
  const int32_t *table = nullptr, *lens = nullptr, *starts = nullptr;
  const uint64_t *tree = nullptr;
  int64_t pages = 0;
  spmm_plan_t plan = &p;
  spmm_plan_s other;
  if (what == "no_plan") plan = nullptr;
  if (what == "other_plan") plan = &other;
  if (what == "k_null") k.data = kf.data = nullptr;
  if (what == "k_overlaps") kf.stride_head = 32;
  if (what == "k8_null") k8.data = nullptr;
  if (what == "k8_odd") k8.data = memory + 8;
  if (what == "k8_stride_odd") k8.stride_token = 2 * 64 + 8;
  if (what == "k8_stride_wide") k8.stride_token = int64_t(1) << 25;
  if (what == "k8_overlaps") k8.stride_head = 32;
  if (what == "v8_null") v8.data = nullptr;
  if (what == "ks_null") ks = nullptr;
  if (what == "ks_odd") ks = reinterpret_cast<float *>(memory + 2);
  if (what == "vs_null") vs = nullptr;
  if (what == "lens_odd") lens = reinterpret_cast<const int32_t *>(memory + 2);
  if (what == "starts_odd") starts = reinterpret_cast<const int32_t *>(memory + 2);
  if (what == "pooled_odd") pooled += 8;
  if (what == "tree_long") tree = reinterpret_cast<const uint64_t *>(memory);
  if (what == "pages_negative") {
    table = reinterpret_cast<const int32_t *>(memory);
    pages = -1;
  }
  if (what == "table_odd") {
    table = reinterpret_cast<const int32_t *>(memory + 1);
    pages = 4;
  }
  if (call == "write") return spmm_execute_attn_write(plan, &k, &v, &k8, &v8, ks, vs, pages, table, lens, starts, nullptr);
  if (call == "read") return spmm_execute_attn_read(plan, &k8, &v8, ks, vs, pages, &kf, &vf, table, lens, nullptr);
  if (call == "pool8") return spmm_execute_attn_pool8(plan, &k8, ks, pages, pooled, vs, table, lens, starts, nullptr);
  return spmm_execute_attn_cache8(plan, &q, &k8, &v8, ks, vs, pages, &o, lse, table, nullptr, tree, lens, starts, nullptr);
}

spmm_status_t rope_calls(bool back, const std::string &what) {
  double freqs[64];
  int32_t axis[64];
  for (int i = 0; i < 64; ++i) freqs[i] = 1.0, axis[i] = 0;
  spmm_rope_desc_t d{};
  d.batch = what == "nothing" ? 0 : 2;
  d.tokens = 16;
  d.heads_q = 4;
  d.heads_kv = 2;
  d.dim = 64;
  d.dtype = SPMM_BF16;
  d.pairs = 32;
  d.axes = 1;
  d.backward = what == "no_backward" ? 0 : 1;
  d.eps = 1e-6f;
  d.freqs = freqs;
  d.axis = axis;
  if (what == "batch") d.batch = -1;
  if (what == "tokens") d.tokens = int64_t(1) << 31;
  if (what == "too_many") d.batch = d.tokens = 1 << 16;
  if (what == "launch" || what == "launch_holds") d.batch = 4, d.tokens = (1 << 24) - (what == "launch" ? 0 : 1), d.heads_q = 15;
  if (what == "launch_few" || what == "launch_few_holds")
    d.batch = 16, d.tokens = (1 << 24) - (what == "launch_few" ? 0 : 1), d.heads_q = 14;
  if (what == "heads") d.heads_kv = 0;
  if (what == "heads_many") d.heads_q = 65537;
  if (what == "pairs") d.pairs = 40;
  if (what == "pairs_odd") d.pairs = 12;
  if (what == "axes") d.axes = 0;
  if (what == "axis") axis[3] = 1;
  if (what == "eps") d.eps = -1.0f;
  if (what == "eps_nan") d.eps = NAN;
  if (what == "freqs_null") d.freqs = nullptr;
  if (what == "freqs_nan") freqs[31] = NAN;
  if (what == "dim") d.dim = 96;
  if (what == "dtype") d.dtype = SPMM_F32;
  if (what == "interleaved") d.interleaved = 2;
  spmm_plan_s p;
  const spmm_status_t s = sdm::rope_shape(d, &p);
  if (s != SPMM_OK || what.compare(0, 6, "launch") == 0) return s;
  spmm_attn_tensor_t q = {memory, 16 * 256, 256, 64}, k = {memory, 16 * 128, 128, 64}, q2 = q, k2 = k, q3 = q, k3 = k;
  const float *qw = reinterpret_cast<const float *>(memory), *kw = qw;
  float *dqw = reinterpret_cast<float *>(memory), *dkw = dqw;
  const int32_t *positions = nullptr, *lens = nullptr;
  spmm_plan_t plan = &p;
  spmm_plan_s other;
  if (what == "no_plan") plan = nullptr;
  if (what == "other_plan") plan = &other;
  if (what == "execute") return spmm_execute(&p, memory, 64, memory, 64, nullptr);
  if (what == "sddmm") return spmm_execute_sddmm(&p, memory, 64, memory, 64, memory, nullptr);
  if (what == "attn") return spmm_execute_attn_read(&p, &k, &k, qw, qw, 0, &k, &k, nullptr, nullptr, nullptr);
  if (what == "q_null") q.data = nullptr;
  if (what == "q_stride") q.stride_token = 257;
  if (what == "k_odd") k.data = memory + 2;
  if (what == "out_null") q3.data = nullptr;
  if (what == "out_overlaps") k3.stride_head = 0;
  if (what == "weight_odd") qw = reinterpret_cast<const float *>(memory + 2);
  if (what == "positions_odd") positions = reinterpret_cast<const int32_t *>(memory + 2);
  if (what == "lens_odd") lens = reinterpret_cast<const int32_t *>(memory + 2);
  if (what == "dw_null") dkw = nullptr;
  if (what == "dw_without") qw = nullptr;
  if (what == "grad_null") q2.data = nullptr;
  if (back)
    return spmm_execute_attn_rope_backward(plan, &q2, &k2, &q, &k, qw, kw, &q3, &k3, dqw, dkw, positions, lens, nullptr, nullptr);
  return spmm_execute_attn_rope(plan, &q, &k, qw, kw, &q3, &k3, positions, lens, nullptr, nullptr);
}

}  // namespace

int main() {
  char call[64], what[64];
  while (std::scanf("%63s %63s", call, what) == 2) {
    const spmm_status_t s = !std::strcmp(call, "rope")            ? rope_calls(false, what)
                            : !std::strcmp(call, "rope_backward") ? rope_calls(true, what)
                                                                  : cache_calls(call, what);
    std::printf("%s %s\n", spmm_status_str(s), s == SPMM_OK ? "" : spmm_last_error());
    std::fflush(stdout);
  }
  return 0;
}
