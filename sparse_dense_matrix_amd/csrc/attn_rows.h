// attn_rows.h -- what the kernels of attention forward share: a workgroup's
// item, a lane's row, the range of a list, a row's softmax and its output.
#pragma once

#include "attn_dev.h"

namespace sdm {
namespace attn {

constexpr float kSlack = 8.0f;

// One workgroup's part of the work.  Heads run fastest: with 8 key heads each
// XCD keeps to one of them.
struct Item {
  int h, rt, split, qb, b;
};
__device__ __forceinline__ Item item_of(const AttnArgs &a) {
  int64_t i = blockIdx.x;
  Item r;
  r.h = i % a.hk;
  i /= a.hk;
  r.rt = i % a.rtiles;
  i /= a.rtiles;
  r.split = i % a.nsplit;
  i /= a.nsplit;
  r.qb = i % a.nqb;
  r.b = static_cast<int>(i / a.nqb);
  return r;
}

// A lane's row (lane % M) of a tile of tile_rows rows, and what the wave and
// the workgroup know of their rows together.
struct Row {
  int32_t len, start;
  int tok, head;
  bool real, live;     // of the tensor; with a position in [0, len)
  int32_t pos;
  int32_t last_key;    // the last key any row of the workgroup sees
  int32_t open;        // keys below it are seen by every live row of the wave
  uint64_t bits;       // tree mask
};
template <int M = 32>
__device__ __forceinline__ Row row_of(const AttnArgs &a, const Item &it, int tile_rows, int row0, int lane) {
  Row r;
  r.len = attn_len(a.lens, it.b, a.nk);
  r.start = attn_start(a.starts, it.b, a.nq, a.nk);
  const int row = it.rt * tile_rows + row0 + (lane & (M - 1));
  r.tok = it.qb * a.q_block + row / a.group;
  r.head = it.h * a.group + row % a.group;
  r.real = row < a.rows && r.tok < a.nq;
  r.pos = r.start + r.tok;
  r.live = r.real && r.pos >= 0 && r.pos < r.len;
  const int last_row = min(a.rows, (it.rt + 1) * tile_rows) - 1;
  const int last_tok = min(a.nq - 1, it.qb * a.q_block + last_row / a.group);
  r.last_key = min(r.len - 1, r.start + (a.tree ? 63 : last_tok));  // a tree's mask has 64 bits
  int32_t open = r.live ? (a.tree ? min(r.start, r.len) : r.pos + 1) : INT32_MAX;
#pragma unroll
  for (int m = 1; m < M; m *= 2) open = min(open, __shfl_xor(open, m));
  r.open = __builtin_amdgcn_readfirstlane(open);
  r.bits = a.tree && r.real ? a.tree[static_cast<int64_t>(it.b) * a.nq + r.tok] : 0;
  return r;
}

template <int D>
__device__ __forceinline__ void load_q(const AttnArgs &a, const Item &it, const Row &r, int lane, u32x4 *q) {
  const char *p = a.q.p + (r.real ? it.b * a.q.sb + r.tok * a.q.st + r.head * a.q.sh : 0) + 16 * (lane >> 5);
#pragma unroll
  for (int s = 0; s < D / 16; ++s) q[s] = *reinterpret_cast<const u32x4 *>(p + 32 * s);
}

// The entries [e0, e1) of the item's list that a range takes.
struct Range {
  const int32_t *list, *table_row;
  int32_t e0, e1;
};
__device__ __forceinline__ Range range_of(const AttnArgs &a, const Item &it, const Row &r) {
  Range x;
  x.list = a.lists ? a.lists + ((static_cast<int64_t>(it.b) * a.hk + it.h) * a.nqb + it.qb) * a.max_blocks : nullptr;
  x.table_row = a.table ? a.table + static_cast<int64_t>(it.b) * a.nkb : nullptr;
  x.e0 = it.split * a.per_split;
  x.e1 = min(a.entries, x.e0 + a.per_split);
  if (!x.list) x.e1 = min(x.e1, r.last_key < 0 ? 0 : r.last_key / kAttnPage + 1);
  return x;
}

// `kept` keys from key `first` of a block on (those that some row sees), as a
// buffer.  Rows past them read as zeros: what stands there may be anything, and
// a weight of zero does not make a NaN harmless.
template <int D>
__device__ __forceinline__ i32x4 keys_of(const AttnArgs &a, const AttnView &x, const Item &it, int id, int page,
                                         int32_t first, int32_t kept) {
  const char *p = x.p + it.h * x.sh;
  if (a.table)
    p += page * x.sb + first * x.st;
  else
    p += it.b * x.sb + (static_cast<int64_t>(id) * kAttnPage + first) * x.st;
  return buffer(p, kept > 0 ? static_cast<int32_t>((kept - 1) * x.st + D * 2) : 0);
}

// A row's softmax statistics, base 2; l is this lane's half of the keys.
struct Stats {
  float m = -INFINITY, l = 0.0f;
};

// The scores s of N * 32 keys from key0 on become weights, and o, m and l move
// with the maximum.
template <int D, int N>
__device__ __forceinline__ void softmax(const AttnArgs &a, const Row &r, int32_t key0, int lane, float c, f32x16 *s,
                                        Stats &st, f32x16 *o) {
  const int h2 = lane >> 5;
  if (key0 + 32 * N > r.open) {
    if (a.tree) {
      // the bits of the drafted tokens among the lane's keys, from its first on
      const int32_t before = r.start - (key0 + 4 * h2);  // keys of the text
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int32_t draft = 32 * n + 8 * (e >> 2) + (e & 3) - before;
          const uint64_t bit = draft < 64 ? r.bits >> (draft & 63) : 0;
          s[n][e] = (draft < 0 || (bit & 1)) && draft < r.len - r.start ? s[n][e] : -INFINITY;
        }
    } else {
      const int32_t last = min(r.pos, r.len - 1) - (key0 + 4 * h2);
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          s[n][e] = 32 * n + 8 * (e >> 2) + (e & 3) <= last ? s[n][e] : -INFINITY;
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, s[n][e]);
  top = max_halves(top) * c;
  if (__any(top > st.m + kSlack)) {
    const float next = fmaxf(st.m, top);
    const float f = next == -INFINITY ? 1.0f : exp2_(st.m - next);
    st.l *= f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[i][e] *= f;
    st.m = next;
  }
  const float from = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      s[n][e] = exp2_(__builtin_fmaf(s[n][e], c, -from));
      st.l += s[n][e];
    }
}

// The sums of key groups 1 .. KW - 1 (RW waves each), joined by the first in
// group order through LDS that nothing else uses by then.
template <int D, int RW, int KW>
__device__ __forceinline__ void join_groups(char *lds, int wave, int lane, Stats &st, f32x16 *o) {
  constexpr int kRowsF = D / 2;  // floats of o a lane holds
  float *buf = reinterpret_cast<float *>(lds);
  const int rw = wave % RW;
  barrier();
  if (wave >= RW) {
    float *p = buf + (wave - RW) * (kRowsF + 2) * 64 + lane;
#pragma unroll
    for (int i = 0; i < kRowsF; ++i) p[i * 64] = o[i / 16][i % 16];
    p[kRowsF * 64] = st.m;
    p[(kRowsF + 1) * 64] = st.l;
  }
  __syncthreads();
  if (wave >= RW) return;
#pragma unroll
  for (int g = 1; g < KW; ++g) {
    const float *p = buf + (g * RW + rw - RW) * (kRowsF + 2) * 64 + lane;
    const float m2 = p[kRowsF * 64], l2 = p[(kRowsF + 1) * 64];
    const float next = fmaxf(st.m, m2);
    const float f1 = st.m == -INFINITY ? 0.0f : exp2_(st.m - next);
    const float f2 = m2 == -INFINITY ? 0.0f : exp2_(m2 - next);
#pragma unroll
    for (int i = 0; i < kRowsF; ++i) o[i / 16][i % 16] = o[i / 16][i % 16] * f1 + p[i * 64] * f2;
    st.l = st.l * f1 + l2 * f2;
    st.m = next;
  }
}

// o and lse of a row, or its part of them where a list is cut into ranges.
template <class T, int D>
__device__ __forceinline__ void store(const AttnArgs &a, const Item &it, const Row &r, int lane, float m, float l,
                                      const f32x16 *o) {
  if (!r.real) return;
  const int h2 = lane >> 5;
  const int64_t rid = (static_cast<int64_t>(it.b) * a.hq + r.head) * a.nq + r.tok;
  if (a.nsplit > 1) {
    const int64_t at = it.split * (static_cast<int64_t>(a.b) * a.hq * a.nq) + rid;
    if (h2 == 0) {
      a.part_ml[2 * at] = m;
      a.part_ml[2 * at + 1] = l;
    }
    if (m == -INFINITY && l == 0.0f) return;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4 *>(a.part_o + at * D + 32 * i + 8 * g + 4 * h2) =
            f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]};
    return;
  }
  const bool none = l == 0.0f;
  const float inv = none ? 0.0f : 1.0f / l;
  char *op = a.o.p + it.b * a.o.sb + r.tok * a.o.st + r.head * a.o.sh;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      u32x2 w;
      w[0] = none ? 0 : pack2<T>(o[i][4 * g] * inv, o[i][4 * g + 1] * inv);
      w[1] = none ? 0 : pack2<T>(o[i][4 * g + 2] * inv, o[i][4 * g + 3] * inv);
      *reinterpret_cast<u32x2 *>(op + (32 * i + 8 * g + 4 * h2) * 2) = w;
    }
  if (h2 == 0) a.lse[rid] = none ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace attn
}  // namespace sdm
