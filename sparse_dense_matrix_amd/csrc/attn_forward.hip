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
#include "attn_rows.h"
#include "internal.h"

namespace sdm {
namespace attn {
namespace {

constexpr int kAhead = 2;  // operands read ahead of their product

// Many rows to a list: RW waves of 32 rows share each staged tile of KT keys;
// KW groups of them take the tiles in turn.  Two stages: the next tile loads
// while this one is multiplied.  32k tokens, 32 heads over 8, 2048 keys a
// query: 1.07 to 1.12 ms on different cards, 0.94 to 0.98 PFLOP/s, 77 to 80% of
// the rate of a large matrix product.
// Scores, softmax and the product with V follow one another in a wave, and ask
// for LDS, vector units and matrix cores for about half of the time each, so
// what counts is how many waves a SIMD holds: three (four waves of 32 rows a
// workgroup, 32 keys a tile, 168 registers) are 4% faster than two (eight
// waves, 64 keys, operands four ahead).  Two groups of waves half a tile apart
// (1.18 ms) or exponentials laid between products (1.15 ms) gain nothing.
template <class T, int D, int RW, int KW, int KT>
__global__ __launch_bounds__(64 * RW * KW, RW == 4 && KW == 1 ? 3 : 2) void attn_forward(const AttnArgs a) {
  using L = Tile<D>;
  constexpr int kHalf = KT * L::kRowBytes;  // K or V of a stage
  constexpr int kLoads = kHalf / 1024 / RW;  // direct loads of K, and of V, of a wave
  static_assert(kLoads >= 1 && kLoads * RW * 1024 == kHalf, "loads of a stage");
  constexpr int kSubs = kAttnPage / KT;
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const Item it = item_of(a);
  const Row row = row_of(a, it, 32 * RW, 32 * rw, lane);
  const Range range = range_of(a, it, row);
  u32x4 q[D / 16];
  load_q<D>(a, it, row, lane, q);

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
  Stats st;
  const float c = a.scale * kLog2e;

  for (int32_t e = range.e0; e < range.e1; e += 64) {
    const Named blocks = named_blocks(range.list, range.table_row, a.pages, e, range.e1, row.last_key, lane);
    const int tiles = blocks.n * kSubs;
    const int rounds = (tiles + KW - 1) / KW;
    auto issue = [&](int round) {
      const int t = round * KW + kw;
      const int at = t < tiles ? t / kSubs : 0;
      const int id = __builtin_amdgcn_readlane(blocks.id, at);
      const int page = __builtin_amdgcn_readlane(blocks.page, at);
      const int32_t first = (t % kSubs) * KT;
      const int32_t kept = t < tiles ? min(KT, row.last_key + 1 - id * kAttnPage - first) : 0;
      const i32x4 kbuf = keys_of<D>(a, a.k, it, id, page, first, kept);
      const i32x4 vbuf = keys_of<D>(a, a.v, it, id, page, first, kept);
      const uint32_t at_lds = stage0 + (round & 1) * 2 * kHalf;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        load_lds16(__builtin_amdgcn_readfirstlane(at_lds + (rw * kLoads + i) * 1024), kbuf, koff[i]);
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        load_lds16(__builtin_amdgcn_readfirstlane(at_lds + kHalf + (rw * kLoads + i) * 1024), vbuf, voff[i]);
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
      f32x16 s[KT / 32];
#pragma unroll
      for (int n = 0; n < KT / 32; ++n) s[n] = zero16();
      constexpr int kX = D / 16, kI = D / 32;
      auto ks = operands<KT / 32 * kX, kAhead>([&](int i) { return L::operand(kt, 32 * (i / kX), i % kX, lane); });
      ks.begin();
      ks.run([&](int i, u32x4 k) { s[i / kX] = T::mma(k, q[i % kX], s[i / kX]); });
      auto vs = operands<KT / 16 * kI, kAhead>([&](int i) { return L::operand_t(vt, 16 * (i / kI), i % kI, lane); });
      vs.begin();
      softmax<D, KT / 32>(a, row, key0, lane, c, s, st, o);
      u32x4 p[KT / 16];
#pragma unroll
      for (int x = 0; x < KT / 16; ++x) p[x] = pack8<T>(s[x / 2], x % 2);
      vs.run([&](int i, u32x4 v) { o[i % kI] = T::mma(v, p[i / kI], o[i % kI]); });
    }
    // the next entries' first tiles go where the last ones may still be read
    barrier();
  }

  st.l = add_halves(st.l);
  if (!row.live) st = Stats();
  if constexpr (KW > 1) {
    join_groups<D, RW, KW>(lds, wave, lane, st, o);
    if (kw > 0) return;
  }
  store<T, D>(a, it, row, lane, st.m, st.l, o);
}

// Up to 32 rows to a list: each wave streams tiles of 32 keys through LDS of
// its own, without barriers, K and V in one buffer each: the next K loads
// during the softmax and the product with V, the next V during the scores.
// Small buffers put 8 waves on a CU (registers allow no more), which covers
// each wave's waits.  KW waves share a list's tiles and join their sums; with
// KW = 1 a list is a wave's own.  Bound by reading the keys: one token for each
// of 32 sequences of up to 32k, 508 us, 5.4 TB/s.
//
// With PACK the lists of neighbouring query blocks share a wave's 32 rows: a
// block that several of them name is read once, and rows whose list does not
// name it have weights of zero there.  What each list alone would read and
// multiply (its tile has 32 rows, used or not) is never less.  8k queries with
// a list each, 16 heads to a key head: 485 us against 726 us.  A weight of
// zero does not make an infinite or NaN value harmless, so where a row comes
// out as neither finite the lists are gone through again one by one.
template <class T, int D, int KW, bool PACK>
__global__ __launch_bounds__(64 * KW, 2) void attn_stream(const AttnArgs a) {
  using L = Tile<D>;
  constexpr int KT = 32, kSubs = kAttnPage / KT;
  constexpr int kHalf = KT * L::kRowBytes;
  constexpr int kLoads = kHalf / 1024;
  static_assert(!PACK || KW == 1, "packed lists are a wave's own");
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Item it = item_of(a);
  const Row row = row_of(a, it, 32, 0, lane);
  Range range;
  int lists = 1, list = 0;  // lists of the tile; the row's among them
  if constexpr (PACK) {
    lists = min(a.pack, a.list_nqb - it.qb * a.pack);
    list = (lane & 31) / (a.rows / a.pack);
    range.list = a.lists + ((static_cast<int64_t>(it.b) * a.hk + it.h) * a.list_nqb + static_cast<int64_t>(it.qb) * a.pack) * a.max_blocks;
    range.table_row = a.table ? a.table + static_cast<int64_t>(it.b) * a.nkb : nullptr;
    range.e0 = 0;
    range.e1 = lists * a.max_blocks;  // at most 64
  } else {
    range = range_of(a, it, row);
  }
  u32x4 q[D / 16];
  load_q<D>(a, it, row, lane, q);

  const char *kt = lds + wave * 2 * kHalf, *vt = kt + kHalf;
  const uint32_t lds_k = __builtin_amdgcn_readfirstlane(lds_addr(kt));
  uint32_t koff[kLoads], voff[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int r = L::load_row(i, lane), c = L::load_byte(i, lane);
    koff[i] = static_cast<uint32_t>(r * a.k.st + c);
    voff[i] = static_cast<uint32_t>(r * a.v.st + c);
  }
  const float c = a.scale * kLog2e;

#pragma unroll 1
  for (int pass = -1; pass < (PACK ? lists : 0); ++pass) {  // all lists together, then if need be one by one
    const uint32_t take = pass < 0 ? ~0u : 1u << pass;
    f32x16 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = zero16();
    Stats st;
    for (int32_t e = range.e0; e < range.e1; e += 64) {
      Shared blocks;
      if constexpr (PACK) {
        blocks = shared_blocks(range.list, range.e1, a.max_blocks, range.table_row, a.pages, take, row.last_key, lane);
      } else {
        const Named b = named_blocks(range.list, range.table_row, a.pages, e, range.e1, row.last_key, lane);
        blocks = Shared{b.id, b.page, 1, b.n};
      }
      const int tiles = blocks.n * kSubs;
      // past the last tile the loads are of no bytes, so that the waits below
      // always count the same loads
      auto issue = [&](int t, bool values) {
        const int at = t < tiles ? t / kSubs : 0;
        const int id = __builtin_amdgcn_readlane(blocks.id, at);
        const int page = __builtin_amdgcn_readlane(blocks.page, at);
        const int32_t first = (t % kSubs) * KT;
        const int32_t kept = t < tiles ? min(KT, row.last_key + 1 - id * kAttnPage - first) : 0;
        const i32x4 buf = keys_of<D>(a, values ? a.v : a.k, it, id, page, first, kept);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          load_lds16(lds_k + (values ? kHalf : 0) + i * 1024, buf, values ? voff[i] : koff[i]);
      };
      if (wave < tiles) {
        issue(wave, false);
        issue(wave, true);
      }
      for (int t = wave; t < tiles; t += KW) {
        const int32_t key0 = __builtin_amdgcn_readlane(blocks.id, t / kSubs) * kAttnPage + (t % kSubs) * KT;
        wait_vm<kLoads>();
        f32x16 s = zero16();
        auto ks = operands<D / 16, D / 16>([&](int x) { return L::operand(kt, 0, x, lane); });
        ks.begin();
        ks.run([&](int x, u32x4 k) { s = T::mma(k, q[x], s); });
        wait_lds();
        issue(t + KW, false);
        if constexpr (PACK) {
          const int members = __builtin_amdgcn_readlane(blocks.members, t / kSubs);
          if (members != (1 << lists) - 1) {
            const bool in = members >> list & 1;
#pragma unroll
            for (int e2 = 0; e2 < 16; ++e2) s[e2] = in ? s[e2] : -INFINITY;
          }
        }
        softmax<D, 1>(a, row, key0, lane, c, &s, st, o);
        wait_vm<kLoads>();
        constexpr int kI = D / 32;
        auto vs = operands<2 * kI, kI>([&](int i) { return L::operand_t(vt, 16 * (i / kI), i % kI, lane); });
        vs.begin();
        const u32x4 p[2] = {pack8<T>(s, 0), pack8<T>(s, 1)};
        vs.run([&](int i, u32x4 v) { o[i % kI] = T::mma(v, p[i / kI], o[i % kI]); });
        wait_lds();
        issue(t + KW, true);
      }
      wait_vm<0>();  // the loads of no bytes
    }

    st.l = add_halves(st.l);
    if (!row.live) st = Stats();
    if constexpr (KW > 1) {
      join_groups<D, 1, KW>(lds, wave, lane, st, o);
      if (wave > 0) return;
    }
    if (!PACK || (take >> list & 1)) store<T, D>(a, it, row, lane, st.m, st.l, o);
    if constexpr (PACK) {
      if (pass < 0) {
        float x = 0.0f;  // NaN where anything is not finite
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) x = __builtin_fmaf(o[i][e], 0.0f, x);
        if (!__any(row.live && x != x)) return;
      }
    }
  }
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
// latency: launch, one round of loads, one exchange through LDS (5 us).  The
// last workgroup of a row tile could do this without a launch, but what other
// XCDs wrote has to come from beyond L2: one token over 4097 keys 15.3 us
// against 13.8 us, 24 drafted tokens 144 us against 113 us.
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

int64_t grid_of(const AttnArgs &a) {
  return static_cast<int64_t>(a.b) * a.hk * a.nqb * a.rtiles * a.nsplit;
}

template <class T, int D, int RW, int KW, int KT>
hipError_t run(const AttnArgs &a, hipStream_t s) {
  constexpr size_t kTiles = static_cast<size_t>(KW) * 4 * KT * D * 2;
  constexpr size_t kSums = static_cast<size_t>(KW - 1) * RW * (D / 2 + 2) * 256;
  constexpr size_t kLds = kTiles > kSums ? kTiles : kSums;
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_forward<T, D, RW, KW, KT>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_forward<T, D, RW, KW, KT>), dim3(static_cast<unsigned>(grid_of(a))), dim3(64 * RW * KW),
                     kLds, s, a);
  return hipGetLastError();
}

template <class T, int D, int KW, bool PACK>
hipError_t run_stream(const AttnArgs &a, hipStream_t s) {
  constexpr size_t kTiles = static_cast<size_t>(KW) * 2 * 32 * D * 2;
  constexpr size_t kSums = static_cast<size_t>(KW - 1) * (D / 2 + 2) * 256;
  constexpr size_t kLds = kTiles > kSums ? kTiles : kSums;
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_stream<T, D, KW, PACK>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_stream<T, D, KW, PACK>), dim3(static_cast<unsigned>(grid_of(a))), dim3(64 * KW), kLds, s, a);
  return hipGetLastError();
}

template <class T, int D>
hipError_t run_merge(const AttnArgs &a, hipStream_t s) {
  constexpr int kGroups = 256 / (D / 4);
  int per_row = 2;
  while (per_row < a.nsplit && per_row < kGroups) per_row *= 2;
  const int64_t rows = static_cast<int64_t>(a.b) * a.hq * a.nq;
  const int64_t grid = (rows * per_row + kGroups - 1) / kGroups;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL((attn_merge<T, D>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a, per_row);
  return hipGetLastError();
}

template <class T, int D>
hipError_t run_tile(const AttnArgs &a, hipStream_t s) {
  if (grid_of(a) == 0) return hipSuccess;
  if (grid_of(a) > 0x7fffffff) return hipErrorInvalidValue;
  hipError_t e;
  switch (attn_tile(a.rows, a.nqb).row_waves) {
    // a wave a list where there are enough lists to fill the chip (8 waves a
    // CU) twice over
    case 1:
      if (grid_of(a) >= 4096 && a.nsplit == 1) {
        const int32_t pack = a.lists && a.nqb > 1 ? attn_pack(grid_of(a), a.rows, a.max_blocks) : 0;
        e = pack ? run_stream<T, D, 1, true>(attn_packed(a, pack), s) : run_stream<T, D, 1, false>(a, s);
      } else {
        e = run_stream<T, D, 4, false>(a, s);
      }
      break;
    case 2: e = run<T, D, 2, 2, 32>(a, s); break;
    // up to a workgroup a CU, two groups of waves share its list (2048 tokens, 16
    // heads over 8, 16 blocks a query: 25.6 us against 31.0)
    case 4: e = grid_of(a) <= kCus ? run<T, D, 4, 2, 32>(a, s) : run<T, D, 4, 1, 32>(a, s); break;
    default: e = run<T, D, 8, 1, 64>(a, s); break;
  }
  return e != hipSuccess || a.nsplit == 1 ? e : run_merge<T, D>(a, s);
}

}  // namespace
}  // namespace attn

AttnTile attn_tile(int32_t rows, int32_t nqb) {
  // The smallest tile that holds all rows of a query block, up to 128, or 256
  // where it is a sequence's only one: rows in several tiles stage the same keys
  // again, which then come from memory and not from L2 (24 drafted tokens with 8
  // heads to a key head, 16 sequences of up to 8k: 172 us, in two tiles 226 us).
  int32_t best = nqb == 1 ? 8 : 4;
  while (best > 1 && 32 * (best / 2) >= rows) best /= 2;
  if (best == 8 && rows > 256 && (rows + 127) / 128 % 2 == 1) best = 4;  // which pads least
  AttnTile t;
  t.row_waves = best;
  t.key_waves = best == 1 ? 4 : (best == 2 ? 2 : 1);
  t.key_tile = best == 8 ? 64 : 32;
  t.rows = 32 * best;
  return t;
}

int32_t attn_pack(int64_t lists, int32_t rows, int32_t max_blocks) {
  // as many as fill a tile and a wave's lanes, while a wave is left for each
  // of the 8 places of a CU
  int32_t n = 1;
  while (n < 16 && 2 * n * rows <= 32 && 2 * n * max_blocks <= 64 && lists / (2 * n) >= 2048) n *= 2;
  return n > 1 ? n : 0;
}

AttnArgs attn_packed(AttnArgs a, int32_t pack) {
  a.pack = pack;
  a.list_nqb = a.nqb;
  a.rows *= pack;
  a.q_block *= pack;
  a.nqb = (a.nqb + pack - 1) / pack;
  return a;
}

hipError_t launch_attn_merge(const AttnArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16) return d == 64 ? attn::run_merge<attn::Bf16, 64>(a, s) : attn::run_merge<attn::Bf16, 128>(a, s);
  return d == 64 ? attn::run_merge<attn::F16, 64>(a, s) : attn::run_merge<attn::F16, 128>(a, s);
}

hipError_t launch_attn_forward(const AttnArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16) return d == 64 ? attn::run_tile<attn::Bf16, 64>(a, s) : attn::run_tile<attn::Bf16, 128>(a, s);
  return d == 64 ? attn::run_tile<attn::F16, 64>(a, s) : attn::run_tile<attn::F16, 128>(a, s);
}

}  // namespace sdm
