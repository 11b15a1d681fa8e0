// attn_backward.hip -- gradients of attention over listed blocks.  With
// p_tj = exp(scale q_t . k_j - lse_t) over what query t sees, and
// delta_t = do_t . o_t = sum_j p_tj (do_t . v_j):
//   dv_j = sum_t p_tj do_t          ds_tj = p_tj (do_t . v_j - delta_t)
//   dq_t = scale sum_j ds_tj k_j    dk_j = scale sum_t ds_tj q_t
//
// Three launches.  attn_dq walks each query block's list as the forward does
// and keeps dq in registers; its first workgroups invert the lists (for each
// key block the query blocks that name it, ascending).  attn_dkv walks the
// inverse list of a key block and keeps dk and dv in registers.  A block that
// many lists name (the first of a sequence is in all of them) is cut into
// items of `chunk` query blocks, whose partial sums attn_dkv_merge adds in
// order: no atomics, so the same inputs give the same bits.
//
// p and ds are rounded to the element type for their products, at most half a
// step each; sums, statistics and delta stay in 32 bits.  ds may be far larger
// than the gradients it adds up to (heads of 128, unit normal inputs: 4 times
// dq), so in f16 a row's ds, or a key's, are rounded at a power of two that
// keeps the largest of them below 2^15 (Fit).
#include <algorithm>

#include "attn_dev.h"
#include "internal.h"

namespace sdm {
namespace attn {
namespace {

constexpr int kAhead = 4;               // operands read ahead of their product
constexpr int kShort = 128;             // queries of a short sequence
constexpr int kFewRows = 256;           // rows of a short inverse list: one query block of 64 with 4 heads to a key head
constexpr int kFew = 2;                 // blocks of a short list
constexpr int kFewBit = 1 << 30;        // of an item's part: few rows read the key block
constexpr int kMaxChunk = 1024;         // query blocks of an item
constexpr uint32_t kDeadRow = 0xffffff00u;  // offset past every buffer: a direct load gives zeros

// Sequence length, position of the first query, and last key that query block
// qb sees.
__device__ __forceinline__ int32_t last_key_of(const AttnArgs &a, int q_block, int qb, int32_t len, int32_t start) {
  return min(len - 1, start + min(a.nq - 1, qb * q_block + q_block - 1));
}

// x / d for d > 0, with inv = 0xffffffff / d: the product is at most one below
__device__ __forceinline__ uint32_t over(uint32_t x, uint32_t d, uint32_t inv) {
  const uint32_t r = __umulhi(x, inv);
  return x - r * d >= d ? r + 1 : r;
}

// Inverse list of key block kb of head bh, and its items.  Each wave reads a
// stretch of the head's lists twice: to count, then to write the query blocks
// behind those of the waves before it, so that they come out ascending.
__device__ void invert(const AttnArgs &a, int64_t which, char *lds) {
  const int kb = which % a.nkb;
  const int64_t bh = which / a.nkb;
  const int b = bh / a.hk;
  const int32_t len = attn_len(a.lens, b, a.nk), start = attn_start(a.starts, b, a.nq, a.nk);
  const int nqb = a.pack ? a.list_nqb : a.nqb, q_block = a.pack ? a.q_block / a.pack : a.q_block;  // of one list
  const int rows = a.pack ? a.rows / a.pack : a.rows;
  const uint32_t entries = static_cast<uint32_t>(nqb) * a.max_blocks;  // below 2^31
  const int32_t *lists = a.lists + bh * static_cast<int64_t>(entries);
  int *sums = reinterpret_cast<int *>(lds);  // [waves][2]
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 63, wave = tid >> 6, waves = nt >> 6;
  const uint32_t inv = 0xffffffffu / static_cast<uint32_t>(a.max_blocks);
  const uint32_t stretch = ((entries + nt - 1) / nt) * 64;
  const uint32_t e0 = min(entries, wave * stretch), e1 = min(entries, e0 + stretch);
  // the block that entry e names, or -1
  auto named = [&](uint32_t e) {
    const int32_t id = e < e1 ? lists[e] : -1;
    return id >= 0 && attn_names(id, last_key_of(a, q_block, over(e, a.max_blocks, inv), len, start)) ? id : -1;
  };

  int less = 0, same = 0;
#pragma unroll 4
  for (uint32_t e = e0; e < e1; e += 64) {
    const int32_t id = named(e + lane);
    less += id >= 0 && id < kb;
    same += id == kb;
  }
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    less += __shfl_xor(less, m);
    same += __shfl_xor(same, m);
  }
  if (lane == 0) {
    sums[2 * wave] = less;
    sums[2 * wave + 1] = same;
  }
  __syncthreads();
  const int mine = same;
  int before = 0;
  less = same = 0;
  for (int w = 0; w < waves; ++w) {
    if (w == wave) before = same;
    less += sums[2 * w];
    same += sums[2 * w + 1];
  }
  int32_t *ids = a.inv_ids + bh * static_cast<int64_t>(entries) + less + before;
  if (mine > 0) {
#pragma unroll 4
    for (uint32_t e = e0; e < e1; e += 64) {
      const bool here = named(e + lane) == kb;
      const uint64_t all = __ballot(here);
      const uint64_t below = (uint64_t(1) << lane) - 1;
      if (here) ids[__builtin_popcountll(all & below)] = static_cast<int32_t>(over(e + lane, a.max_blocks, inv));
      ids += __builtin_popcountll(all);
    }
  }
  // Items stand at kb + less / chunk on: that leaves room for max(1,
  // ceil(same / chunk)) of them before the next key block's.
  int32_t *items = a.items + bh * a.slots * 2;
  const int first = kb + less / a.chunk;
  const int next = kb + 1 == a.nkb ? a.slots : kb + 1 + (less + same) / a.chunk;
  const int n = max(1, (same + a.chunk - 1) / a.chunk);
  // few queries in the sequence, or few rows that may read the block
  const bool few = min(a.nq, len - start) - max(0, -start) <= kShort || static_cast<int64_t>(same) * rows <= kFewRows;
  for (int i = tid; i < next - first; i += nt) {
    items[2 * (first + i)] = i < n ? kb : -1;
    items[2 * (first + i) + 1] = few ? i | kFewBit : i;
  }
  if (tid == 0) {
    a.inv_ptr[2 * (bh * a.nkb + kb)] = less;
    a.inv_ptr[2 * (bh * a.nkb + kb) + 1] = same;
  }
}

// What workgroups below b * hk * nkb do: invert, and set what the dk, dv
// kernel starts from.
__device__ __forceinline__ void prepare(const AttnArgs &a, int64_t item, char *lds) {
  // the first items of the dk, dv kernel's queues are its workgroups' own
  if (item == 0 && threadIdx.x < 8) a.queue[threadIdx.x] = kCus / 8;
  // the statistics of a row that is not there
  if (item == 0 && threadIdx.x == 0)
    *reinterpret_cast<f32x2 *>(a.stats + 2 * static_cast<int64_t>(a.b) * a.hq * a.nq) = f32x2{INFINITY, 0.0f};
  invert(a, item, lds);
}

// The power of two at which dS enters its product where the type's range is
// narrow: it starts out high and falls, with the sums so far, when a value of
// the lane's row (or key) would pass 2^15.  A row's sums leave its wave at 2^0
// again.  A training step in f16 takes 2 to 7% longer for it (16k tokens, 32
// heads over 8, 1024 keys a query: 1.66 ms against 1.60).
template <class T, int D>
struct Fit {
  int x = 100;
  __device__ __forceinline__ void scale(f32x16 &ds, f32x16 *sum) {
    if constexpr (T::kNarrow) {
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(ds[e]));
      top = max_halves(top);
      const int n = __builtin_amdgcn_frexp_expf(top);  // top is in [2^(n - 1), 2^n)
      const bool past = top > 0.0f && n + x > 15;
      if (__any(past)) {
        const int to = past ? 13 - n : x;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) sum[i][e] = __builtin_ldexpf(sum[i][e], to - x);
        x = to;
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) ds[e] = __builtin_ldexpf(ds[e], x);
    }
  }
  __device__ __forceinline__ void back(f32x16 *sum) {
    if constexpr (T::kNarrow) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[i][e] = __builtin_ldexpf(sum[i][e], -x);
    }
  }
};

// A lane's row of a wave of the dq kernels.
template <class T, int D>
struct DqRow {
  int b, h, tok, head;
  bool real;
  int32_t last, last_key, open;  // last key the row sees; of the tile; below open every live row sees a key
  int64_t rid;
  float delta, lse2;
  u32x4 q[D / 16], g[D / 16];

  __device__ __forceinline__ DqRow(const AttnArgs &a, int b_, int h_, int qb, int rt, int tile_rows, int row0, int lane)
      : b(b_), h(h_) {
    const int h2 = lane >> 5;
    const int32_t len = attn_len(a.lens, b, a.nk), start = attn_start(a.starts, b, a.nq, a.nk);
    const int row = rt * tile_rows + row0 + (lane & 31);
    tok = qb * a.q_block + row / a.group;
    head = h * a.group + row % a.group;
    real = row < a.rows && tok < a.nq;
    const int32_t pos = start + tok;
    const bool live = real && pos >= 0 && pos < len;
    last = min(pos, len - 1);
    const int last_row = min(a.rows, (rt + 1) * tile_rows) - 1;
    const int last_tok = min(a.nq - 1, qb * a.q_block + last_row / a.group);
    last_key = min(len - 1, start + last_tok);
    open = live ? pos + 1 : INT32_MAX;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) open = min(open, __shfl_xor(open, m));
    open = __builtin_amdgcn_readfirstlane(open);
    rid = (static_cast<int64_t>(b) * a.hq + head) * a.nq + tok;
    const char *qp = a.q.p + (real ? b * a.q.sb + tok * a.q.st + head * a.q.sh : 0) + 16 * h2;
    const char *gp = a.g.p + (real ? b * a.g.sb + tok * a.g.st + head * a.g.sh : 0) + 16 * h2;
    const char *op = a.o.p + (real ? b * a.o.sb + tok * a.o.st + head * a.o.sh : 0) + 16 * h2;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      q[s] = *reinterpret_cast<const u32x4 *>(qp + 32 * s);
      g[s] = *reinterpret_cast<const u32x4 *>(gp + 32 * s);
    }
    delta = 0.0f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const u32x4 o = *reinterpret_cast<const u32x4 *>(op + 32 * s);
#pragma unroll
      for (int i = 0; i < 8; ++i) delta += elem<T>(g[s][i / 2], i & 1) * elem<T>(o[i / 2], i & 1);
    }
    delta = add_halves(delta);
    lse2 = INFINITY;  // a row that sees nothing: every weight 0
    if (live) {
      const float x = a.lse[rid];
      if (x != -INFINITY) lse2 = x * kLog2e;
    }
    if (lse2 == INFINITY) delta = 0.0f;
  }

  // Scores and do . v of 32 keys from key0 on become dS; sum is that of all dS.
  // The sum is what delta is off by: delta is sum_j p_j (do . v_j), and do . o
  // in its place carries the rounding of o.
  __device__ __forceinline__ void ds(f32x16 &s, f32x16 &dp, int32_t key0, float c, int lane, float &sum) const {
    if (key0 + 32 > open) {
      const int32_t most = last - (key0 + 4 * (lane >> 5));
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const bool sees = 8 * (e >> 2) + (e & 3) <= most;
        s[e] = sees ? s[e] : -INFINITY;
        dp[e] = sees ? dp[e] : 0.0f;  // what stands there may be no number
      }
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      s[e] = exp2_(__builtin_fmaf(s[e], c, -lse2)) * (dp[e] - delta);
      sum += s[e];
    }
  }

  // dq of the row, and its statistics for the dk, dv kernel, with delta
  // corrected once more.
  __device__ __forceinline__ void store(const AttnArgs &a, int lane, const f32x16 *dq, float sum) const {
    if (!real) return;
    const int h2 = lane >> 5;
    const bool none = lse2 == INFINITY;
    if (h2 == 0) *reinterpret_cast<f32x2 *>(a.stats + 2 * rid) = f32x2{lse2, none ? 0.0f : delta + sum};
    char *out = a.dq.p + b * a.dq.sb + tok * a.dq.st + head * a.dq.sh;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int g4 = 0; g4 < 4; ++g4) {
        u32x2 w;
        w[0] = none ? 0 : pack2<T>(dq[i][4 * g4] * a.scale, dq[i][4 * g4 + 1] * a.scale);
        w[1] = none ? 0 : pack2<T>(dq[i][4 * g4 + 2] * a.scale, dq[i][4 * g4 + 3] * a.scale);
        *reinterpret_cast<u32x2 *>(out + (32 * i + 8 * g4 + 4 * h2) * 2) = w;
      }
  }
};

// dq += K^T dS of 32 keys from row0 of the tile on.  dS goes in as two
// operands, what the first one's rounding leaves out in the second: its
// rounding alone puts dq off by more than dq's own rounding does (2.8e-3
// against 1.7e-3 of its norm for bf16), for a third more products.
template <class T, int D, class R>
__device__ __forceinline__ void add_dq(const f32x16 &s, R &ks, f32x16 *dq) {
  constexpr int kI = D / 32;
  u32x4 hi[2], lo[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) split8<T>(s, x, hi[x], lo[x]);
  ks.run([&](int i, u32x4 k) {
    dq[i % kI] = T::mma(k, hi[i / kI], dq[i % kI]);
    dq[i % kI] = T::mma(k, lo[i / kI], dq[i % kI]);
  });
}

// The sums of key groups 1 .. KW - 1 (RW waves each), added by the first in
// group order through LDS that nothing else uses by then.
template <int D, int RW, int KW>
__device__ __forceinline__ void join_dq(char *lds, int wave, int lane, f32x16 *dq, float &sum) {
  constexpr int kRowsF = D / 2;
  float *buf = reinterpret_cast<float *>(lds);
  barrier();
  if (wave >= RW) {
    float *p = buf + (wave - RW) * (kRowsF + 1) * 64 + lane;
#pragma unroll
    for (int i = 0; i < kRowsF; ++i) p[i * 64] = dq[i / 16][i % 16];
    p[kRowsF * 64] = sum;
  }
  __syncthreads();
  if (wave >= RW) return;
#pragma unroll
  for (int g = 1; g < KW; ++g) {
    const float *p = buf + (g * RW + wave - RW) * (kRowsF + 1) * 64 + lane;
#pragma unroll
    for (int i = 0; i < kRowsF; ++i) dq[i / 16][i % 16] += p[i * 64];
    sum += p[kRowsF * 64];
  }
}

// sum over the KW key groups of RW waves, for each row, in every wave.
template <int RW, int KW>
__device__ __forceinline__ float sum_groups(char *lds, int wave, int lane, float sum) {
  if constexpr (KW > 1) {
    float *buf = reinterpret_cast<float *>(lds);
    barrier();
    buf[wave * 64 + lane] = sum;
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int g = 0; g < KW; ++g) sum += buf[(g * RW + wave % RW) * 64 + lane];
    barrier();
  }
  return sum;
}

// Both dq kernels walk a list twice where it is short, whatever its neighbours
// in a shared tile are, the first time for delta (what it adds to dq is dropped: a branch around it costs registers).
// With few keys the error of do . o would be the larger part of dq's (14 keys
// in bf16: dq off by 2.9e-3 of its norm, 1.7e-3 with it corrected; past two
// blocks 2.1e-3, where another walk would cost half of the kernel's time).

// dq where a list has many rows.  Waves and tiles as in the forward kernel.
// 16k tokens, 32 heads over 8, 1024 keys a query: 550 us, 0.97 PFLOP/s with the
// second operand; a third of it is reading q, o and grad and writing dq.
template <class T, int D, int RW, int KW, int KT>
__global__ __launch_bounds__(64 * RW * KW, 2) void attn_dq(const AttnArgs a) {
  using L = Tile<D>;
  constexpr int kHalf = KT * L::kRowBytes;
  constexpr int kLoads = kHalf / 1024 / RW;
  static_assert(kLoads >= 1 && kLoads * RW * 1024 == kHalf, "loads of a stage");
  static_assert((KW - 1) * RW * (D / 2 + 1) * 256 <= KW * 4 * kHalf, "the groups' sums fit the stages");
  constexpr int kSubs = kAttnPage / KT;
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  int64_t item = blockIdx.x;
  const int64_t inverts = static_cast<int64_t>(a.b) * a.hk * a.nkb;
  if (item < inverts) {
    prepare(a, item, lds);
    return;
  }
  item -= inverts;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const int h = item % a.hk;
  item /= a.hk;
  const int rt = item % a.rtiles;
  item /= a.rtiles;
  const int qb = item % a.nqb;
  const int b = static_cast<int>(item / a.nqb);
  DqRow<T, D> row(a, b, h, qb, rt, 32 * RW, 32 * rw, lane);

  const uint32_t stage0 = lds_addr(lds) + kw * 4 * kHalf;
  const char *stage_p = lds + kw * 4 * kHalf;
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = L::load_row(rw * kLoads + i, lane), c = L::load_byte(rw * kLoads + i, lane);
    koff[i] = static_cast<uint32_t>(r * a.k.st + c);
    voff[i] = static_cast<uint32_t>(r * a.v.st + c);
  }
  f32x16 dq[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) dq[i] = zero16();
  Fit<T, D> fit;
  float sum = 0.0f;
  const float c = a.scale * kLog2e;
  const int32_t *list = a.lists + ((static_cast<int64_t>(b) * a.hk + h) * a.nqb + qb) * a.max_blocks;

#pragma unroll 1
  for (int walk = 0; walk < 2; ++walk) {
    int named = 0;
    for (int32_t e = 0; e < a.max_blocks; e += 64) {
      const Named blocks = named_blocks(list, nullptr, 0, e, a.max_blocks, row.last_key, lane);
      named += blocks.n;
      if (walk == 0 && named > kFew) break;
      const int tiles = blocks.n * kSubs;
      const int rounds = (tiles + KW - 1) / KW;
      auto issue = [&](int round) {
        const int t = round * KW + kw;
        const int id = __builtin_amdgcn_readlane(blocks.id, t < tiles ? t / kSubs : 0);
        const int64_t key = static_cast<int64_t>(id) * kAttnPage + (t % kSubs) * KT;
        const int32_t kept = t < tiles ? static_cast<int32_t>(min(static_cast<int64_t>(KT), row.last_key + 1 - key)) : 0;
        const i32x4 kbuf = buffer(a.k.p + b * a.k.sb + key * a.k.st + h * a.k.sh,
                                  kept > 0 ? static_cast<int32_t>((kept - 1) * a.k.st + D * 2) : 0);
        const i32x4 vbuf = buffer(a.v.p + b * a.v.sb + key * a.v.st + h * a.v.sh,
                                  kept > 0 ? static_cast<int32_t>((kept - 1) * a.v.st + D * 2) : 0);
        const uint32_t st = stage0 + (round & 1) * 2 * kHalf;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          load_lds16(__builtin_amdgcn_readfirstlane(st + (rw * kLoads + i) * 1024), kbuf, koff[i]);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          load_lds16(__builtin_amdgcn_readfirstlane(st + kHalf + (rw * kLoads + i) * 1024), vbuf, voff[i]);
      };
      if (rounds > 0) issue(0);
      for (int round = 0; round < rounds; ++round) {
        wait_vm<0>();
        barrier();
        if (round + 1 < rounds) issue(round + 1);
        const char *kt = stage_p + (round & 1) * 2 * kHalf, *vt = kt + kHalf;
        const int t = round * KW + kw;
        if (t >= tiles) continue;
        const int32_t key0 = __builtin_amdgcn_readlane(blocks.id, t / kSubs) * kAttnPage + (t % kSubs) * KT;
#pragma unroll
        for (int n = 0; n < KT / 32; ++n) {
          f32x16 s = zero16(), dp = zero16();
          auto kv = operands<D / 8, kAhead>([&](int i) { return L::operand(i % 2 ? vt : kt, 32 * n, i / 2, lane); });
          kv.begin();
          kv.run([&](int i, u32x4 x) {
            if (i % 2) dp = T::mma(x, row.g[i / 2], dp);
            else s = T::mma(x, row.q[i / 2], s);
          });
          constexpr int kI = D / 32;
          auto ks = operands<2 * kI, kAhead>([&](int i) { return L::operand_t(kt, 32 * n + 16 * (i / kI), i % kI, lane); });
          row.ds(s, dp, key0 + 32 * n, c, lane, sum);
          fit.scale(s, dq);
          ks.begin();
          add_dq<T, D>(s, ks, dq);
        }
      }
      barrier();
    }
    if (walk == 0) {
      if (named <= kFew) row.delta += sum_groups<RW, KW>(lds, wave, lane, add_halves(sum));
      sum = 0.0f;
      fit = Fit<T, D>();
#pragma unroll
      for (int i = 0; i < D / 32; ++i) dq[i] = zero16();
    }
  }
  fit.back(dq);
  sum = add_halves(sum);
  if constexpr (KW > 1) {
    join_dq<D, RW, KW>(lds, wave, lane, dq, sum);
    if (kw > 0) return;
  }
  row.store(a, lane, dq, sum);
}

// dq where a list has up to 32 rows: each wave streams tiles of 32 keys
// through LDS of its own, without barriers, V in one buffer and K in another:
// the next V loads during the scores and dS, the next K during do . v.  The
// four waves share a list, or with OWN have one each; with PACK the lists of
// neighbouring query blocks share a wave's 32 rows as in the forward kernel.
// 4k queries with a list each, 16 heads to a key head: 205 us (543 us with four
// waves, two stages and a barrier a list, 285 us without PACK).
template <class T, int D, bool OWN, bool PACK>
__global__ __launch_bounds__(256, 2) void attn_dq_stream(const AttnArgs a) {
  using L = Tile<D>;
  constexpr int KT = 32, kSubs = kAttnPage / KT;
  constexpr int kHalf = KT * L::kRowBytes;
  constexpr int kLoads = kHalf / 1024;
  constexpr int kX = D / 16, kI = D / 32;
  static_assert(!PACK || OWN, "packed lists are a wave's own");
  static_assert(3 * (D / 2 + 1) * 256 <= 8 * kHalf, "the waves' sums fit the tiles");
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  int64_t item = blockIdx.x;
  const int64_t inverts = static_cast<int64_t>(a.b) * a.hk * a.nkb;
  if (item < inverts) {
    prepare(a, item, lds);
    return;
  }
  item -= inverts;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = item % a.hk;
  item /= a.hk;
  if (OWN) item = item * 4 + wave;
  const int qb = item % a.nqb;
  const int64_t b64 = item / a.nqb;
  if (b64 >= a.b) return;
  const int b = static_cast<int>(b64);
  DqRow<T, D> row(a, b, h, qb, 0, 32, 0, lane);

  const char *kt = lds + wave * 2 * kHalf, *vt = kt + kHalf;
  const uint32_t lds_k = __builtin_amdgcn_readfirstlane(lds_addr(kt));
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = L::load_row(i, lane), c = L::load_byte(i, lane);
    koff[i] = static_cast<uint32_t>(r * a.k.st + c);
    voff[i] = static_cast<uint32_t>(r * a.v.st + c);
  }
  f32x16 dq[kI];
#pragma unroll
  for (int i = 0; i < kI; ++i) dq[i] = zero16();
  Fit<T, D> fit;
  float sum = 0.0f;
  const float c = a.scale * kLog2e;
  const int64_t head0 = (static_cast<int64_t>(b) * a.hk + h) * (PACK ? a.list_nqb : a.nqb);
  const int32_t *list = a.lists + (head0 + static_cast<int64_t>(qb) * (PACK ? a.pack : 1)) * a.max_blocks;
  const int lists = PACK ? min(a.pack, a.list_nqb - qb * a.pack) : 1;  // of the tile
  const int mine = PACK ? (lane & 31) / (a.rows / a.pack) : 0;         // the row's among them
  const int32_t entries = lists * a.max_blocks;
  constexpr int kStep = OWN ? 1 : 4;
  const int first = OWN ? 0 : wave;

  uint32_t brief = 0;  // the lists of up to kFew blocks
  if constexpr (PACK) {
    const int of = lane / a.max_blocks;  // the list that entry `lane` is of
    const int32_t len = attn_len(a.lens, b, a.nk), start = attn_start(a.starts, b, a.nq, a.nk);
    const int id = lane < entries ? list[lane] : -1;
    const uint64_t named =
        __ballot(attn_names(id, last_key_of(a, a.q_block / a.pack, qb * a.pack + of, len, start)));
    for (int l = 0; l < lists; ++l)
      if (__builtin_popcountll(named >> (l * a.max_blocks) & ((uint64_t(1) << a.max_blocks) - 1)) <= kFew)
        brief |= 1u << l;
  }

  // for delta of short lists; all lists together; then if need be one by one
#pragma unroll 1
  for (int pass = -2; pass < (PACK ? lists : 0); ++pass) {
    const uint32_t take = pass == -2 ? brief : (pass < 0 ? ~0u : 1u << pass);
    int named = 0;
    for (int32_t e = 0; e < entries; e += 64) {
      Shared blocks;
      if constexpr (PACK) {
        blocks = shared_blocks(list, entries, a.max_blocks, nullptr, 0, take, row.last_key, lane);
      } else {
        const Named n = named_blocks(list, nullptr, 0, e, entries, row.last_key, lane);
        blocks = Shared{n.id, n.page, 1, n.n};
      }
      named += blocks.n;
      if (!PACK && pass == -2 && named > kFew) break;
      const int tiles = blocks.n * kSubs;
      // past the last tile the loads are of no bytes, so that the waits below
      // always count the same loads
      auto issue = [&](int t, bool values) {
        const int id = __builtin_amdgcn_readlane(blocks.id, t < tiles ? t / kSubs : 0);
        const int64_t key = static_cast<int64_t>(id) * kAttnPage + (t % kSubs) * KT;
        const int32_t kept = t < tiles ? static_cast<int32_t>(min(static_cast<int64_t>(KT), row.last_key + 1 - key)) : 0;
        const AttnView &x = values ? a.v : a.k;
        const i32x4 buf = buffer(x.p + b * x.sb + key * x.st + h * x.sh,
                                 kept > 0 ? static_cast<int32_t>((kept - 1) * x.st + D * 2) : 0);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          load_lds16(lds_k + (values ? kHalf : 0) + i * 1024, buf, values ? voff[i] : koff[i]);
      };
      if (first < tiles) {
        issue(first, true);
        issue(first, false);
      }
      for (int t = first; t < tiles; t += kStep) {
        const int32_t key0 = __builtin_amdgcn_readlane(blocks.id, t / kSubs) * kAttnPage + (t % kSubs) * KT;
        f32x16 s = zero16(), dp = zero16();
        wait_vm<kLoads>();
        auto vs = operands<kX, kAhead>([&](int x) { return L::operand(vt, 0, x, lane); });
        vs.begin();
        vs.run([&](int x, u32x4 v) { dp = T::mma(v, row.g[x], dp); });
        wait_lds();
        issue(t + kStep, true);
        wait_vm<kLoads>();
        auto ks = operands<kX, kAhead>([&](int x) { return L::operand(kt, 0, x, lane); });
        ks.begin();
        ks.run([&](int x, u32x4 k) { s = T::mma(k, row.q[x], s); });
        auto ts = operands<2 * kI, kAhead>([&](int i) { return L::operand_t(kt, 16 * (i / kI), i % kI, lane); });
        if constexpr (PACK) {
          const int members = __builtin_amdgcn_readlane(blocks.members, t / kSubs);
          if (members != (1 << lists) - 1) {
            const bool in = members >> mine & 1;
#pragma unroll
            for (int e2 = 0; e2 < 16; ++e2) {
              s[e2] = in ? s[e2] : -INFINITY;
              dp[e2] = in ? dp[e2] : 0.0f;
            }
          }
        }
        row.ds(s, dp, key0, c, lane, sum);
        fit.scale(s, dq);
        ts.begin();
        add_dq<T, D>(s, ts, dq);
        wait_lds();
        issue(t + kStep, false);
      }
      wait_vm<0>();  // the loads of no bytes
    }
    if (pass == -2) {
      if (!PACK && named <= kFew) row.delta += sum_groups<1, OWN ? 1 : 4>(lds, wave, lane, add_halves(sum));
      if (PACK) row.delta += brief >> mine & 1 ? add_halves(sum) : 0.0f;
    } else {
      fit.back(dq);
      sum = add_halves(sum);
      if constexpr (!OWN) {
        join_dq<D, 1, 4>(lds, wave, lane, dq, sum);
        if (wave > 0) return;
      }
      if (!PACK || (take >> mine & 1)) row.store(a, lane, dq, sum);
      if constexpr (PACK) {
        if (pass < 0) {
          float x = 0.0f;  // NaN where anything is not finite
#pragma unroll
          for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) x = __builtin_fmaf(dq[i][e], 0.0f, x);
          if (!__any(row.lse2 != INFINITY && x != x)) return;
        }
      }
    }
    sum = 0.0f;
    fit = Fit<T, D>();
#pragma unroll
    for (int i = 0; i < kI; ++i) dq[i] = zero16();
  }
}

// The kernel's arguments, read again: what a loop's body needs of them would
// otherwise be kept in scalar registers throughout, more than there are.
__device__ __forceinline__ AttnArgs args_again() {
  typedef const __attribute__((address_space(4))) uint32_t *Words;
  Words p = (Words)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  struct {
    uint32_t w[sizeof(AttnArgs) / 4];
  } x;
#pragma unroll
  for (unsigned i = 0; i < sizeof(AttnArgs) / 4; ++i) x.w[i] = p[i];
  return __builtin_bit_cast(AttnArgs, x);
}

// An item of the dk, dv kernel: key block kb (-1: none) of key head h, and part
// `part` of the `same` entries of its inverse list, which stand from `less` on.
struct DkvItem {
  int b, h, slot, kb, part, less, same;
  bool few;
  int32_t len, start;

  __device__ __forceinline__ DkvItem(const AttnArgs &a, int64_t item) {
    const uint32_t at = static_cast<uint32_t>(item);  // below 2^31
    h = at % a.hk;
    slot = at / a.hk % a.slots;
    b = at / a.hk / a.slots;
    const int64_t bh = static_cast<int64_t>(b) * a.hk + h;
    kb = a.items[2 * (bh * a.slots + slot)];
    if (kb < 0) return;
    part = a.items[2 * (bh * a.slots + slot) + 1];
    few = part & kFewBit;
    part &= kFewBit - 1;
    less = a.inv_ptr[2 * (bh * a.nkb + kb)];
    same = a.inv_ptr[2 * (bh * a.nkb + kb) + 1];
    len = attn_len(a.lens, b, a.nk);
    start = attn_start(a.starts, b, a.nq, a.nk);
  }
};

// dk and dv of one item: 64 keys, up to `chunk` query blocks of the inverse
// list.  RG row groups of two waves; a wave owns 32 keys (K rows in registers
// as B operands, V rows in LDS) and 32 of the 32 RG rows staged at a time, so
// that S = Q K^T and dP = dO V^T come out with a key a lane, and P and dS feed
// dv^T += dO^T P and dk^T += Q^T dS from registers, with dO and Q read
// transposed from LDS.  dk and dv fill half of a wave's 256 registers, which
// is why V stays in LDS: with V in registers too the kernel spills (1502 us
// against 1022 us for 16k tokens, 32 heads over 8, 1024 keys a query).
// 64 keys and 512 registers a wave halve the LDS reads, but one wave a SIMD
// waits for each of them: 1218 us.  With operands read ahead and items from
// queues 650 to 670 us, 0.80 PFLOP/s: the matrix cores are busy for 37% of it,
// and the rows come from beyond L2 in half of all loads (each is read once for
// every key block that its list names), at 4.2 TB/s.
// FINE is for key blocks that few rows read: P and dS enter their products as
// two operands as dS does for dq, for a quarter more products.  With one operand
// dk and dv are off by 1.4 times their own rounding, averaged over a tensor, and
// single keys with few rows by up to 2.7 times; with two by their own rounding
// alone.  It goes by the sequence's own queries and the block's own list, so
// that a sequence's gradients are as exact next to a longer one.  Steps of 1000
// to 2000 tokens take 0 to 1% longer for it, 6% with a head to a key head and
// lists of 16 queries; with up to 1024 rows, 4 to 9%, for averages of 1.33 to
// 1.41.
template <class T, int D, int RG, bool FINE>
__device__ __forceinline__ void dkv_item(char *lds, int64_t at) {
  const AttnArgs a = args_again();
  const DkvItem it(a, at);
  using L = Tile<D>;
  constexpr int kRows = 32 * RG;
  constexpr int kHalf = kRows * L::kRowBytes;     // Q or dO of a stage
  constexpr int kLoads = kHalf / 1024 / (2 * RG);  // direct loads of each, of a wave
  static_assert(kLoads >= 1 && kLoads * 2 * RG * 1024 == kHalf, "loads of a stage");
  struct Rows {
    uint32_t qoff[kRows], goff[kRows];
  };
  struct Stats {
    float lse2[kRows], delta[kRows];
    int32_t lim[kRows];
    int32_t open[4];  // of 64 rows each, 1: every row sees the whole key block
  };
  Rows *rows = reinterpret_cast<Rows *>(lds + 4 * kHalf + kAttnPage * L::kRowBytes);  // [2]
  Stats *stats = reinterpret_cast<Stats *>(rows + 2);     // [4]
  int32_t *ids = reinterpret_cast<int32_t *>(stats + 4);  // [chunk]

  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));  // nothing of an item's is kept for the next
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kh = wave & 1, rg = wave >> 1;
  const int h2 = lane >> 5;
  const int h = it.h, b = it.b, kb = it.kb, same = it.same;
  const int32_t len = it.len, start = it.start;
  const int64_t bh = static_cast<int64_t>(b) * a.hk + h;
  const int count = min(a.chunk, same - it.part * a.chunk);
  {
    const int32_t *from = a.inv_ids + bh * a.nqb * a.max_blocks + it.less + it.part * a.chunk;
    for (int i = tid; i < count; i += 128 * RG) ids[i] = from[i];
  }
  const int32_t key = kb * kAttnPage + 32 * kh + (lane & 31);
  u32x4 kf[D / 16];
#pragma unroll
  for (int x = 0; x < D / 16; ++x) {
    kf[x] = u32x4{0, 0, 0, 0};
    if (key < len)
      kf[x] = *reinterpret_cast<const u32x4 *>(a.k.p + b * a.k.sb + key * a.k.st + h * a.k.sh + 32 * x + 16 * h2);
  }
  const char *vt = lds + 4 * kHalf;  // the block's V
  {
    constexpr int kVLoads = kAttnPage * L::kRowBytes / 1024 / (2 * RG);
    static_assert(kVLoads * 2 * RG * 1024 == kAttnPage * L::kRowBytes, "loads of V");
    const int32_t kept = min(kAttnPage, len - kb * kAttnPage);
    const i32x4 vbuf = buffer(a.v.p + b * a.v.sb + static_cast<int64_t>(kb) * kAttnPage * a.v.st + h * a.v.sh,
                              kept > 0 ? static_cast<int32_t>((kept - 1) * a.v.st + D * 2) : 0);
#pragma unroll
    for (int i = 0; i < kVLoads; ++i) {
      const int n = wave * kVLoads + i;
      load_lds16(__builtin_amdgcn_readfirstlane(lds_addr(vt) + n * 1024), vbuf,
                 static_cast<uint32_t>(L::load_row(n, lane) * a.v.st + L::load_byte(n, lane)));
    }
  }
  // the compiler does not see the waits in asm: here it waits for K itself,
  // and not again in each round, where that would wait for the round's loads
#pragma unroll
  for (int x = 0; x < D / 16; ++x) asm volatile("" : "+v"(kf[x]));
  wait_vm<0>();
  __syncthreads();

  const i32x4 qbuf = buffer(a.q.p + b * a.q.sb,
                            static_cast<int32_t>((a.nq - 1) * a.q.st + (a.hq - 1) * a.q.sh + D * 2));
  const i32x4 gbuf = buffer(a.g.p + b * a.g.sb,
                            static_cast<int32_t>((a.nq - 1) * a.g.st + (a.hq - 1) * a.g.sh + D * 2));
  const uint32_t total = static_cast<uint32_t>(count) * a.rows;
  const int rounds = static_cast<int>((total + kRows - 1) / kRows);
  const uint32_t per_list = 0xffffffffu / static_cast<uint32_t>(a.rows);
  const uint32_t per_token = 0xffffffffu / static_cast<uint32_t>(a.group);
  // Threads below kRows look after a row each, two rounds ahead: its offsets
  // for the direct loads, its limit, and its statistics on their way to LDS.
  // Rows that are not there, or stand before the key block, read zeros and see
  // no key: a weight of zero does not make a NaN in q or grad harmless.
  auto find = [&](int round) {
    const uint32_t flat = static_cast<uint32_t>(round) * kRows + tid;
    Stats &s = stats[round & 3];
    uint32_t qo = kDeadRow, go = kDeadRow;
    int32_t lim = -1;
    int64_t rid = static_cast<int64_t>(a.b) * a.hq * a.nq;
    if (flat < total) {
      const uint32_t e = over(flat, a.rows, per_list), row = flat - e * a.rows;
      const uint32_t t = over(row, a.group, per_token);
      const int tok = ids[e] * a.q_block + static_cast<int>(t);
      const int head = h * a.group + static_cast<int>(row - t * a.group);
      const int32_t pos = start + tok;
      if (tok < a.nq && pos >= kb * kAttnPage && pos < len) {
        rid = (static_cast<int64_t>(b) * a.hq + head) * a.nq + tok;
        lim = pos;
        qo = static_cast<uint32_t>(tok * a.q.st + head * a.q.sh);
        go = static_cast<uint32_t>(tok * a.g.st + head * a.g.sh);
      }
    }
    rows[round & 1].qoff[tid] = qo;
    rows[round & 1].goff[tid] = go;
    s.lim[tid] = lim;
    const bool all = __all(lim >= kb * kAttnPage + kAttnPage - 1);
    if (lane == 0) s.open[wave] = all;
    load_lds4(__builtin_amdgcn_readfirstlane(lds_addr(&s.lse2[64 * wave])), a.stats + 2 * rid);
    load_lds4(__builtin_amdgcn_readfirstlane(lds_addr(&s.delta[64 * wave])), a.stats + 2 * rid + 1);
  };
  const bool finder = wave < kRows / 64;
  auto issue = [&](int round) {
    const uint32_t st = lds_addr(lds) + (round & 1) * 2 * kHalf;
    const Rows &r = rows[round & 1];
    uint32_t qo[kLoads], go[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int n = wave * kLoads + i;
      qo[i] = r.qoff[L::load_row(n, lane)] + L::load_byte(n, lane);
      go[i] = r.goff[L::load_row(n, lane)] + L::load_byte(n, lane);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      load_lds16(__builtin_amdgcn_readfirstlane(st + (wave * kLoads + i) * 1024), qbuf, qo[i]);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      load_lds16(__builtin_amdgcn_readfirstlane(st + kHalf + (wave * kLoads + i) * 1024), gbuf, go[i]);
  };
  Fit<T, D> fit;
  f32x16 dk[D / 32], dv[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    dk[i] = zero16();
    dv[i] = zero16();
  }
  const float c = a.scale * kLog2e;
  if (rounds > 0) {
    if (finder) {
      find(0);
      find(1);
    }
    __syncthreads();
    issue(0);
  }
  for (int round = 0; round < rounds; ++round) {
    wait_vm<0>();
    barrier();
    if (round + 1 < rounds) issue(round + 1);
    if (round + 2 < rounds && finder) find(round + 2);
    const char *qt = lds + (round & 1) * 2 * kHalf, *gt = qt + kHalf;
    const Stats &st = stats[round & 3];
    f32x16 s = zero16(), dp = zero16();
    constexpr int AQ = 1;
    auto qs = operands<D / 16, AQ>([&](int x) { return L::operand(qt, 32 * rg, x, lane); });
    auto gs = operands<D / 16, AQ>([&](int x) { return L::operand(gt, 32 * rg, x, lane); });
    auto vs = operands<D / 16, AQ>([&](int x) { return L::operand(vt, 32 * kh, x, lane); });
    qs.begin();
    gs.begin();
    vs.begin();
#pragma unroll
    for (int x = 0; x < D / 16; ++x) {
      qs.next(x);
      gs.next(x);
      vs.next(x);
      pin();
      s = T::mma(qs.buf[x], kf[x], s);
      dp = T::mma(gs.buf[x], vs.buf[x], dp);
      pin();
    }
    constexpr int kI = D / 32;
    auto ts = operands<4 * kI, kAhead>([&](int i) {  // dO^T for P, then Q^T for dS
      return L::operand_t(i < 2 * kI ? gt : qt, 32 * rg + 16 * (i / kI % 2), i % kI, lane);
    });
    const bool masked = st.open[rg / 2] == 0;
    if (masked) {
#pragma unroll
      for (int g4 = 0; g4 < 4; ++g4) {
        const i32x4 m4 = *reinterpret_cast<const i32x4 *>(&st.lim[32 * rg + 8 * g4 + 4 * h2]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[4 * g4 + i] = key <= m4[i] ? s[4 * g4 + i] : -INFINITY;
          dp[4 * g4 + i] = key <= m4[i] ? dp[4 * g4 + i] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int g4 = 0; g4 < 4; ++g4) {
      const int r0 = 32 * rg + 8 * g4 + 4 * h2;
      const f32x4 l4 = *reinterpret_cast<const f32x4 *>(&st.lse2[r0]);
      const f32x4 d4 = *reinterpret_cast<const f32x4 *>(&st.delta[r0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[4 * g4 + i] = exp2_(__builtin_fmaf(s[4 * g4 + i], c, -l4[i]));
        dp[4 * g4 + i] = s[4 * g4 + i] * (dp[4 * g4 + i] - d4[i]);
      }
    }
    fit.scale(dp, dk);
    u32x4 w[4], low[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if constexpr (FINE) split8<T>(x < 2 ? s : dp, x % 2, w[x], low[x]);
      else w[x] = pack8<T>(x < 2 ? s : dp, x % 2);
    }
    ts.begin();
    ts.run([&](int i, u32x4 x) {
      f32x16 &to = i < 2 * kI ? dv[i % kI] : dk[i % kI];
      to = T::mma(x, w[i / kI], to);
      if constexpr (FINE) to = T::mma(x, low[i / kI], to);
    });
  }
  fit.back(dk);
  {
  const AttnArgs a = args_again();
  // the row groups' sums, each group adding a share of them in group order
  constexpr int kTiles = D / 32;
  float *buf = reinterpret_cast<float *>(lds);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    barrier();
    {
      float *p = buf + wave * kTiles * 16 * 64 + lane;
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) p[(i * 16 + e) * 64] = which ? dv[i][e] : dk[i][e];
    }
    __syncthreads();
    for (int i = rg; i < kTiles; i += RG) {
      const float *p = buf + (kh * kTiles + i) * 16 * 64 + lane;
      f32x16 sum;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float x = p[e * 64];
#pragma unroll
        for (int g = 1; g < RG; ++g) x += p[(2 * g * kTiles * 16 + e) * 64];
        sum[e] = x;
      }
      if (same > a.chunk) {
        float *out = a.part_kv + (bh * a.slots + it.slot) * 2 * kAttnPage * D + which * kAttnPage * D +
                     (32 * kh + (lane & 31)) * D + 32 * i + 4 * h2;
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4)
          *reinterpret_cast<f32x4 *>(out + 8 * g4) =
              f32x4{sum[4 * g4], sum[4 * g4 + 1], sum[4 * g4 + 2], sum[4 * g4 + 3]};
      } else if (key < a.nk) {
        const AttnView &o = which ? a.dv : a.dk;
        const float f = which ? 1.0f : a.scale;
        char *out = o.p + b * o.sb + key * o.st + h * o.sh + 64 * i + 8 * h2;
#pragma unroll
        for (int g4 = 0; g4 < 4; ++g4) {
          u32x2 w;
          w[0] = pack2<T>(sum[4 * g4] * f, sum[4 * g4 + 1] * f);
          w[1] = pack2<T>(sum[4 * g4 + 2] * f, sum[4 * g4 + 3] * f);
          *reinterpret_cast<u32x2 *>(out + 16 * g4) = w;
        }
      }
    }
  }
  }
}

// Each workgroup takes its own item, then further ones from queues: the
// dispatcher leaves a CU idle for a fifth of the time where a workgroup fills
// it and the items differ in length.  Queue x holds every eighth item, so that
// with 8 key heads XCD x keeps to one of them; a workgroup whose queue is empty
// goes on to the next one that is not.
template <class T, int D, int RG>
__global__ __launch_bounds__(128 * RG) void attn_dkv(const AttnArgs) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  __shared__ int32_t taken[2];  // queue, or -1: nothing is left; place in it
  int64_t item = blockIdx.x;
  for (;;) {
    int how = 0;
    {
      const AttnArgs a = args_again();
      if (item < static_cast<int64_t>(a.b) * a.slots * a.hk) {
        const DkvItem it(a, item);
        how = it.kb < 0 ? 0 : (it.few ? 1 : 2);
      }
    }
    if (how == 1) dkv_item<T, D, RG, true>(lds, item);
    if (how == 2) dkv_item<T, D, RG, false>(lds, item);
    const AttnArgs a = args_again();
    const int64_t items = static_cast<int64_t>(a.b) * a.slots * a.hk;
    if (items <= gridDim.x) return;
    __syncthreads();
    if (threadIdx.x < 64) {
      const int q = threadIdx.x & 7;
      const int64_t at = __hip_atomic_load(a.queue + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      const uint32_t some = __ballot(at * 8 + q < items) & 0xff, own = blockIdx.x & 7;
      const uint32_t first = some & (0xffu << own) ? some & (0xffu << own) : some;
      if (threadIdx.x == 0) {
        const int x = some ? __builtin_ctz(first) : -1;
        taken[0] = x;
        if (some) taken[1] = atomicAdd(a.queue + x, 1);
      }
    }
    __syncthreads();
    const int q = __builtin_amdgcn_readfirstlane(taken[0]);
    if (q < 0) return;
    item = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(taken[1])) * 8 + q;
  }
}

// dk and dv of the key blocks that were cut into items: their partial sums in
// order, four elements a thread.
template <class T, int D>
__global__ __launch_bounds__(256) void attn_dkv_merge(const AttnArgs a) {
  constexpr int kPer = 2 * kAttnPage * D / 4 / 256;  // workgroups of a key block
  const int64_t which = blockIdx.x / kPer;
  const int kb = which % a.nkb;
  const int64_t bh = which / a.nkb;
  const int less = a.inv_ptr[2 * which], same = a.inv_ptr[2 * which + 1];
  if (same <= a.chunk) return;
  const int n = (same + a.chunk - 1) / a.chunk;
  const int at = ((blockIdx.x % kPer) * 256 + threadIdx.x) * 4;  // in [2][64][D]
  const float *p = a.part_kv + (bh * a.slots + kb + less / a.chunk) * 2 * kAttnPage * D + at;
  f32x4 sum = *reinterpret_cast<const f32x4 *>(p);
  for (int i = 1; i < n; ++i) {
    const f32x4 x = *reinterpret_cast<const f32x4 *>(p + static_cast<int64_t>(i) * 2 * kAttnPage * D);
    for (int j = 0; j < 4; ++j) sum[j] += x[j];
  }
  const bool is_v = at >= kAttnPage * D;
  const int32_t key = kb * kAttnPage + (at / D) % kAttnPage;
  if (key >= a.nk) return;
  const AttnView &d = is_v ? a.dv : a.dk;
  const float f = is_v ? 1.0f : a.scale;
  u32x2 w;
  w[0] = pack2<T>(sum[0] * f, sum[1] * f);
  w[1] = pack2<T>(sum[2] * f, sum[3] * f);
  *reinterpret_cast<u32x2 *>(d.p + (bh / a.hk) * d.sb + key * d.st + (bh % a.hk) * d.sh + (at % D) * 2) = w;
}

template <class T, int D, int RW, int KW, int KT>
hipError_t run_dq(const AttnArgs &a, hipStream_t s) {
  constexpr size_t kLds = static_cast<size_t>(KW) * 4 * KT * D * 2;
  const int64_t grid = static_cast<int64_t>(a.b) * a.hk * (static_cast<int64_t>(a.nqb) * a.rtiles + a.nkb);
  if (grid == 0) return hipSuccess;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_dq<T, D, RW, KW, KT>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_dq<T, D, RW, KW, KT>), dim3(static_cast<unsigned>(grid)), dim3(64 * RW * KW), kLds, s, a);
  return hipGetLastError();
}

template <class T, int D, bool OWN, bool PACK>
hipError_t run_dq_stream(const AttnArgs &a, hipStream_t s) {
  constexpr size_t kLds = 4 * 2 * 32 * D * 2;
  const int64_t lists = static_cast<int64_t>(a.b) * a.nqb;
  const int64_t grid = static_cast<int64_t>(a.hk) * ((OWN ? (lists + 3) / 4 : lists) + static_cast<int64_t>(a.b) * a.nkb);
  if (grid == 0) return hipSuccess;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_dq_stream<T, D, OWN, PACK>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_dq_stream<T, D, OWN, PACK>), dim3(static_cast<unsigned>(grid)), dim3(256), kLds, s, a);
  return hipGetLastError();
}

template <class T, int D>
hipError_t run_dkv(const AttnArgs &a, hipStream_t s) {
  constexpr int kRG = 4;
  const size_t lds = 4 * 32 * kRG * D * 2 + kAttnPage * D * 2 + 2 * (2 * 32 * kRG * 4) + 4 * (3 * 32 * kRG * 4 + 16) +
                     static_cast<size_t>(a.chunk) * 4;
  const int64_t grid = static_cast<int64_t>(a.b) * a.hk * a.slots;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_dkv<T, D, kRG>), lds + (kMaxChunk - a.chunk) * 4);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_dkv<T, D, kRG>), dim3(static_cast<unsigned>(std::min<int64_t>(grid, kCus))), dim3(128 * kRG), lds, s, a);
  return hipGetLastError();
}

template <class T, int D>
hipError_t run_backward(const AttnArgs &a, hipStream_t s) {
  hipError_t e;
  switch (attn_tile(a.rows, a.nqb).row_waves) {
    // a wave a list where there are enough lists to fill the chip (8 waves a
    // CU) twice over
    case 1:
      if (const int64_t lists = static_cast<int64_t>(a.b) * a.hk * a.nqb; lists >= 4096) {
        const int32_t pack = a.nqb > 1 ? attn_pack(lists, a.rows, a.max_blocks) : 0;
        e = pack ? run_dq_stream<T, D, true, true>(attn_packed(a, pack), s) : run_dq_stream<T, D, true, false>(a, s);
      } else {
        e = run_dq_stream<T, D, false, false>(a, s);
      }
      break;
    case 2: e = run_dq<T, D, 2, 2, 32>(a, s); break;
    // two workgroups of four waves a CU rather than one of eight: one reads
    // its rows while the other multiplies (16k tokens: 605 us against 680)
    // Tiles of 64 rows whose keys two groups of waves share where that leaves at
    // most one workgroup a CU (1254 tokens, 8 heads over 2 of 64: 56 us the step
    // against 63; two a CU, 2048 tokens, 16 heads over 8: 140.5 against 139.6).
    default: {
      AttnArgs x = a;
      x.rtiles = (a.rows + 63) / 64;
      const bool small = static_cast<int64_t>(a.b) * a.hk * a.nqb * x.rtiles <= kCus;
      if (!small) x.rtiles = (a.rows + 127) / 128;
      e = small ? run_dq<T, D, 2, 2, 32>(x, s) : run_dq<T, D, 4, 1, 64>(x, s);
      break;
    }
  }
  if (e != hipSuccess || a.nkb == 0) return e;
  e = run_dkv<T, D>(a, s);
  if (e != hipSuccess || a.slots == a.nkb) return e;
  const int64_t merge = static_cast<int64_t>(a.b) * a.hk * a.nkb * (2 * kAttnPage * D / 4 / 256);
  if (merge > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((attn_dkv_merge<T, D>), dim3(static_cast<unsigned>(merge)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace attn

void attn_chunks(int64_t heads, int64_t entries, int32_t nqb, int32_t rows, int32_t nkb, int32_t *chunk, int32_t *slots) {
  // about 256 items more than one a key block: one a CU, taken from queues (a
  // step of 2048 tokens, 16 heads over 8: 117 us, with 512 140 us, with 128 135
  // us; of 16k tokens, 32 heads over 8: 1.53, 1.53 and 1.99 ms), but at least
  // 512 rows an item: its partial sums cost as much traffic as 128 rows' q and do
  const int64_t most = heads * entries / 256 + 1, least = (511 + rows) / rows;
  // (and at most 2^28, so that the kernel counts them in 32 bits)
  const int64_t cap = std::max<int64_t>(1, std::min<int64_t>(attn::kMaxChunk, (int64_t(1) << 28) / rows));
  int64_t c = std::min(cap, std::max(most, least));
  // no key block is cut, not even one that lists name more than once: without
  // partial sums there is no launch to merge them (4 us)
  if (nqb <= c && entries < cap) c = entries + 1;
  *chunk = static_cast<int32_t>(c);
  // items of key block kb start at kb + (entries before it) / chunk
  *slots = static_cast<int32_t>(nkb + entries / c);
}

hipError_t launch_attn_backward(const AttnArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16)
    return d == 64 ? attn::run_backward<attn::Bf16, 64>(a, s) : attn::run_backward<attn::Bf16, 128>(a, s);
  return d == 64 ? attn::run_backward<attn::F16, 64>(a, s) : attn::run_backward<attn::F16, 128>(a, s);
}

}  // namespace sdm
