// attn_forward.hip -- attention over listed blocks of keys, and over a cache:
//   o_t = sum_j p_tj v_j,   p_tj = exp(scale q_t . k_j - lse_t),
// over the keys j of the query block's list (or of every block) that query t
// sees: j < len and j <= start + t, or for drafted tokens the keys before
// them and those the tree mask names.
//
// One pass over the keys with a running maximum and sum.  A wave owns 32 rows
// (query tokens times the heads that share the key head) and computes the
// transposed scores S^T = K Q^T, so that a lane holds one row's scores: the
// softmax statistics are one number a lane, and P^T feeds O^T += V^T P^T from
// its registers, with V read transposed from LDS.  P is rounded to the element
// type for that product, at most half a step of each weight; sums, statistics
// and O stay in 32 bits.  The maximum is moved only when a score passes it by
// 8 (base 2): weights then reach 2^8 at most, the rounding is relative, and
// the rescale of O is left out of nearly every tile.
#include "attn_dev.h"
#include "internal.h"

namespace sdm {
namespace attn {
namespace {

constexpr float kSlack = 8.0f;

// RW waves share each staged tile of KT keys, 32 rows a wave; KW groups of
// them take the tiles in turn and join their sums at the end.
template <class T, int D, int RW, int KW, int KT>
__global__ __launch_bounds__(64 * RW * KW) void attn_forward(const AttnArgs a) {
  using L = Tile<D>;
  constexpr int kHalf = KT * L::kRowBytes;  // K or V of a stage
  constexpr int kLoads = kHalf / 1024 / RW;  // direct loads of K, and of V, of a wave
  static_assert(kLoads >= 1 && kLoads * RW * 1024 == kHalf, "loads of a stage");
  constexpr int kSubs = kAttnPage / KT;
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const int h2 = lane >> 5;

  // heads run fastest: with 8 key heads each XCD keeps to one of them
  int64_t item = blockIdx.x;
  const int h = item % a.hk;
  item /= a.hk;
  const int rt = item % a.rtiles;
  item /= a.rtiles;
  const int split = item % a.nsplit;
  item /= a.nsplit;
  const int qb = item % a.nqb;
  const int b = static_cast<int>(item / a.nqb);

  const int32_t len = attn_len(a.lens, b, a.nk);
  const int32_t start = attn_start(a.starts, b, a.nq, a.nk);

  // this lane's row
  const int row = rt * (32 * RW) + rw * 32 + (lane & 31);
  const int tok = qb * a.q_block + row / a.group;
  const int head = h * a.group + row % a.group;
  const bool real = row < a.rows && tok < a.nq;
  const int32_t pos = start + tok;
  const bool live = real && pos >= 0 && pos < len;
  // the last key any row of the workgroup sees
  const int last_row = min(a.rows, (rt + 1) * (32 * RW)) - 1;
  const int last_tok = min(a.nq - 1, qb * a.q_block + last_row / a.group);
  const int32_t last_key = a.tree ? len - 1 : min(len - 1, start + last_tok);
  // keys below `open` are seen by every live row of the wave
  int32_t open = live ? (a.tree ? min(start, len) : pos + 1) : INT32_MAX;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) open = min(open, __shfl_xor(open, m));
  open = __builtin_amdgcn_readfirstlane(open);
  const uint64_t bits = a.tree && real ? a.tree[static_cast<int64_t>(b) * a.nq + tok] : 0;

  u32x4 q[D / 16];
  {
    const int64_t at = real ? b * a.q.sb + tok * a.q.st + head * a.q.sh : 0;
    const char *p = a.q.p + at + 16 * h2;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) q[s] = *reinterpret_cast<const u32x4 *>(p + 32 * s);
  }

  const uint32_t stage0 = lds_addr(lds) + kw * 4 * kHalf;
  const char *stage_p = lds + kw * 4 * kHalf;
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = L::load_row(rw * kLoads + i, lane), c = L::load_byte(rw * kLoads + i, lane);
    koff[i] = static_cast<uint32_t>(r * a.k.st + c);
    voff[i] = static_cast<uint32_t>(r * a.v.st + c);
  }

  f32x16 o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = zero16();
  float m = -INFINITY, l = 0.0f;
  const float c = a.scale * kLog2e;

  const int32_t *list =
      a.lists ? a.lists + ((static_cast<int64_t>(b) * a.hk + h) * a.nqb + qb) * a.max_blocks : nullptr;
  const int32_t *table_row = a.table ? a.table + static_cast<int64_t>(b) * a.nkb : nullptr;
  int32_t e_end = min(a.entries, (split + 1) * a.per_split);
  if (!list) e_end = min(e_end, last_key < 0 ? 0 : last_key / kAttnPage + 1);

  for (int32_t e = split * a.per_split; e < e_end; e += 64) {
    const Named blocks = named_blocks(list, table_row, a.pages, e, e_end, last_key, lane);
    const int tiles = blocks.n * kSubs;
    // rounds are alike for all key groups where they meet at barriers
    const int rounds = (tiles - (RW > 1 ? 0 : kw) + KW - 1) / KW;
    auto issue = [&](int round) {
      const int t = round * KW + kw;
      const int at = t < tiles ? t / kSubs : 0;
      const int id = __builtin_amdgcn_readlane(blocks.id, at);
      const int page = __builtin_amdgcn_readlane(blocks.page, at);
      const int32_t first = (t % kSubs) * KT;  // key of the block the tile starts at
      const int32_t kept = t < tiles ? min(KT, len - id * kAttnPage - first) : 0;
      const char *kp, *vp;
      if (a.table) {
        kp = a.k.p + page * a.k.sb + first * a.k.st;
        vp = a.v.p + page * a.v.sb + first * a.v.st;
      } else {
        kp = a.k.p + b * a.k.sb + (static_cast<int64_t>(id) * kAttnPage + first) * a.k.st;
        vp = a.v.p + b * a.v.sb + (static_cast<int64_t>(id) * kAttnPage + first) * a.v.st;
      }
      // rows past the length are zeros: what stands there may be anything,
      // and a weight of zero does not make a NaN harmless
      const i32x4 kbuf = buffer(kp + h * a.k.sh, kept > 0 ? static_cast<int32_t>((kept - 1) * a.k.st + D * 2) : 0);
      const i32x4 vbuf = buffer(vp + h * a.v.sh, kept > 0 ? static_cast<int32_t>((kept - 1) * a.v.st + D * 2) : 0);
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
      if constexpr (RW > 1) barrier();
      else wait_lds();
      if (round + 1 < rounds) issue(round + 1);
      const char *kt = stage_p + (round & 1) * 2 * kHalf, *vt = kt + kHalf;
      const int t = round * KW + kw;
      if (t >= tiles) continue;
      const int32_t key0 = __builtin_amdgcn_readlane(blocks.id, t / kSubs) * kAttnPage + (t % kSubs) * KT;

      f32x16 s[KT / 32];
#pragma unroll
      for (int n = 0; n < KT / 32; ++n) {
        s[n] = zero16();
#pragma unroll
        for (int x = 0; x < D / 16; ++x) s[n] = T::mma(L::operand(kt, 32 * n, x, lane), q[x], s[n]);
      }
      if (key0 + KT > open) {
#pragma unroll
        for (int n = 0; n < KT / 32; ++n)
#pragma unroll
          for (int e2 = 0; e2 < 16; ++e2) {
            const int32_t key = key0 + 32 * n + 8 * (e2 >> 2) + 4 * h2 + (e2 & 3);
            bool sees;
            if (a.tree) {
              const int32_t draft = key - start;
              sees = key < len && (draft < 0 || (draft < 64 && ((bits >> (draft & 63)) & 1)));
            } else {
              sees = key <= pos && key < len;
            }
            s[n][e2] = sees ? s[n][e2] : -INFINITY;
          }
      }
      float top = s[0][0];
#pragma unroll
      for (int n = 0; n < KT / 32; ++n)
#pragma unroll
        for (int e2 = 0; e2 < 16; ++e2) top = fmaxf(top, s[n][e2]);
      top = max_halves(top) * c;
      if (__any(top > m + kSlack)) {
        const float next = fmaxf(m, top);
        const float f = next == -INFINITY ? 1.0f : exp2_(m - next);
        l *= f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int e2 = 0; e2 < 16; ++e2) o[i][e2] *= f;
        m = next;
      }
      const float from = m == -INFINITY ? 0.0f : m;
#pragma unroll
      for (int n = 0; n < KT / 32; ++n)
#pragma unroll
        for (int e2 = 0; e2 < 16; ++e2) {
          s[n][e2] = exp2_(__builtin_fmaf(s[n][e2], c, -from));
          l += s[n][e2];
        }
#pragma unroll
      for (int n = 0; n < KT / 32; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const u32x4 p = pack8<T>(s[n], x);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) o[i] = T::mma(L::operand_t(vt, 32 * n + 16 * x, i, lane), p, o[i]);
        }
    }
    // the next entries' first tiles go where the last ones may still be read
    if constexpr (RW > 1) barrier();
    else wait_lds();
  }

  l = add_halves(l);
  if (!live) {
    m = -INFINITY;
    l = 0.0f;
  }
  if constexpr (KW > 1) {
    // the key groups' sums, joined by the first of them in group order
    constexpr int kRowsF = D / 2;  // floats of o a lane holds
    float *buf = reinterpret_cast<float *>(lds);
    barrier();
    if (kw > 0) {
      float *p = buf + (wave - RW) * (kRowsF + 2) * 64 + lane;
#pragma unroll
      for (int i = 0; i < kRowsF; ++i) p[i * 64] = o[i / 16][i % 16];
      p[kRowsF * 64] = m;
      p[(kRowsF + 1) * 64] = l;
    }
    __syncthreads();
    if (kw > 0) return;
#pragma unroll
    for (int g = 1; g < KW; ++g) {
      const float *p = buf + (g * RW + rw - RW) * (kRowsF + 2) * 64 + lane;
      const float m2 = p[kRowsF * 64], l2 = p[(kRowsF + 1) * 64];
      const float next = fmaxf(m, m2);
      const float f1 = m == -INFINITY ? 0.0f : exp2_(m - next);
      const float f2 = m2 == -INFINITY ? 0.0f : exp2_(m2 - next);
#pragma unroll
      for (int i = 0; i < kRowsF; ++i) o[i / 16][i % 16] = o[i / 16][i % 16] * f1 + p[i * 64] * f2;
      l = l * f1 + l2 * f2;
      m = next;
    }
  }
  if (!real) return;
  const int64_t rid = (static_cast<int64_t>(b) * a.hq + head) * a.nq + tok;
  if (a.nsplit > 1) {
    const int64_t at = split * (static_cast<int64_t>(a.b) * a.hq * a.nq) + rid;
    if (h2 == 0) {
      a.part_ml[2 * at] = m;
      a.part_ml[2 * at + 1] = l;
    }
    if (m == -INFINITY && !(l != l)) return;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4 *>(a.part_o + at * D + 32 * i + 8 * g + 4 * h2) =
            f32x4{o[i][4 * g], o[i][4 * g + 1], o[i][4 * g + 2], o[i][4 * g + 3]};
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  char *op = a.o.p + b * a.o.sb + tok * a.o.st + head * a.o.sh;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const bool none = l == 0.0f;
      u32x2 w;
      w[0] = none ? 0 : pack2<T>(o[i][4 * g] * inv, o[i][4 * g + 1] * inv);
      w[1] = none ? 0 : pack2<T>(o[i][4 * g + 2] * inv, o[i][4 * g + 3] * inv);
      *reinterpret_cast<u32x2 *>(op + (32 * i + 8 * g + 4 * h2) * 2) = w;
    }
  if (h2 == 0) a.lse[rid] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// The sums m, l, o joined with others of the same row.
__device__ __forceinline__ void join(float &m, float &l, f32x4 &o, float m2, float l2, f32x4 o2) {
  if (m2 == -INFINITY && l2 == 0.0f) return;  // nothing was seen, and o2 not written
  const float next = fmaxf(m, m2);
  const float f1 = m == -INFINITY ? 0.0f : exp2_(m - next);
  const float f2 = m2 == -INFINITY ? 0.0f : exp2_(m2 - next);
  l = l * f1 + l2 * f2;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = o[i] * f1 + o2[i] * f2;
  m = next;
}

// The ranges' sums of a row.  `per_row` groups of D / 4 lanes (a power of
// two, up to the workgroup's) share a row: each joins its ranges, all loads
// in flight at once, and the first joins the groups in order.  Bound by
// latency: launch, one round of loads, one exchange through LDS.
template <class T, int D>
__global__ __launch_bounds__(256) void attn_merge(const AttnArgs a, int per_row) {
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
  __shared__ f32x4 so[kGroups][kLanes];
  __shared__ float sm[kGroups], sl[kGroups];
  const int64_t rows = static_cast<int64_t>(a.b) * a.hq * a.nq;
  const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, sub = group % per_row;
  const int64_t rid = static_cast<int64_t>(blockIdx.x) * (kGroups / per_row) + group / per_row;
  float m = -INFINITY, l = 0.0f;
  f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
  if (rid < rows) {
#pragma unroll 4
    for (int s = sub; s < a.nsplit; s += per_row) {
      const int64_t at = s * rows + rid;
      join(m, l, o, a.part_ml[2 * at], a.part_ml[2 * at + 1],
           *reinterpret_cast<const f32x4 *>(a.part_o + at * D + 4 * lane));
    }
  }
  so[group][lane] = o;
  if (lane == 0) {
    sm[group] = m;
    sl[group] = l;
  }
  __syncthreads();
  if (rid >= rows || sub > 0) return;
  for (int g = 1; g < per_row; ++g) join(m, l, o, sm[group + g], sl[group + g], so[group + g][lane]);
  const int tok = rid % a.nq;
  const int64_t bh = rid / a.nq;
  char *op = a.o.p + (bh / a.hq) * a.o.sb + tok * a.o.st + (bh % a.hq) * a.o.sh;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  u32x2 w;
  w[0] = pack2<T>(o[0] * inv, o[1] * inv);
  w[1] = pack2<T>(o[2] * inv, o[3] * inv);
  *reinterpret_cast<u32x2 *>(op + lane * 8) = w;
  if (lane == 0) a.lse[rid] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <class T, int D, int RW, int KW, int KT>
hipError_t run(const AttnArgs &a, hipStream_t s) {
  constexpr size_t kLds = static_cast<size_t>(KW) * 4 * KT * D * 2;
  const int64_t grid = static_cast<int64_t>(a.b) * a.hk * a.nqb * a.rtiles * a.nsplit;
  if (grid == 0) return hipSuccess;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_forward<T, D, RW, KW, KT>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_forward<T, D, RW, KW, KT>), dim3(static_cast<unsigned>(grid)), dim3(64 * RW * KW), kLds,
                     s, a);
  return hipGetLastError();
}

template <class T, int D>
hipError_t run_tile(const AttnArgs &a, hipStream_t s) {
  hipError_t e;
  switch (attn_tile(a.rows).row_waves) {
    case 1: e = run<T, D, 1, 4, 32>(a, s); break;
    case 2: e = run<T, D, 2, 2, 32>(a, s); break;
    case 4: e = run<T, D, 4, 1, 64>(a, s); break;
    default: e = run<T, D, 8, 1, 64>(a, s); break;
  }
  if (e != hipSuccess || a.nsplit == 1) return e;
  constexpr int kGroups = 256 / (D / 4);
  int per_row = 2;
  while (per_row < a.nsplit && per_row < kGroups) per_row *= 2;
  const int64_t rows = static_cast<int64_t>(a.b) * a.hq * a.nq;
  const int64_t grid = (rows * per_row + kGroups - 1) / kGroups;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((attn_merge<T, D>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a, per_row);
  return hipGetLastError();
}

}  // namespace
}  // namespace attn

AttnTile attn_tile(int32_t rows) {
  // one tile for all rows of a query block where that can be: rows in several
  // tiles stage the same keys again.  Past 256 rows the tile that pads least.
  int32_t best = 8;
  if (rows <= 256) {
    while (best > 1 && 32 * (best / 2) >= rows) best /= 2;
  } else if ((rows + 127) / 128 % 2 == 1) {
    best = 4;
  }
  AttnTile t;
  t.row_waves = best;
  t.key_waves = best == 1 ? 4 : (best == 2 ? 2 : 1);
  t.key_tile = best <= 2 ? 32 : 64;
  t.rows = 32 * best;
  return t;
}

hipError_t launch_attn_forward(const AttnArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16) return d == 64 ? attn::run_tile<attn::Bf16, 64>(a, s) : attn::run_tile<attn::Bf16, 128>(a, s);
  return d == 64 ? attn::run_tile<attn::F16, 64>(a, s) : attn::run_tile<attn::F16, 128>(a, s);
}

}  // namespace sdm
