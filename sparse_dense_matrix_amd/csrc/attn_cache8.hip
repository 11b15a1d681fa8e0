// attn_cache8.hip -- attention over a cache in 8 bits: key j of a head stands
// as codes c_j with a scale ks_j, its value as codes d_j with vs_j, and
//   o_t = sum_j p_tj vs_j d_j,   p_tj = exp(scale ks_j (q_t . c_j) - lse_t),
// over the keys j that query t sees (attn_forward.hip has the same sums over a
// cache in 16 bits, and the form of the softmax).
//
// The codes are whole numbers up to 127, which bf16 and f16 hold exactly, so
// nothing is rounded on the way to the products: a score is the sum of q_t's
// elements times the codes in 32 bits, then times ks_j.  The value's scale goes
// to the weight: p_tj vs_j is two bf16 operands for the products with d_j, the
// weight and what its rounding left out, and so within 2^-16 of itself: a weight
// times a value's scale can pass f16's range both ways, bf16 reaches as far as 32
// bits.  The sum that divides is of p_tj itself.
#include "attn_rows.h"
#include "internal.h"

namespace sdm {
namespace attn {
namespace {

constexpr int kAhead = 2;  // operands read ahead of their product

// Four codes as a pair of operand words: converted to 32 bits each, where a
// whole number up to 127 leaves the lower half of the word zero (bf16), or
// packed exactly (f16).
template <class T>
__device__ __forceinline__ u32x2 widen4(unsigned u) {
  const float a = static_cast<float>(static_cast<int8_t>(u)), b = static_cast<float>(static_cast<int8_t>(u >> 8));
  const float c = static_cast<float>(static_cast<int8_t>(u >> 16)), d = static_cast<float>(static_cast<int8_t>(u >> 24));
  if constexpr (T::kNarrow) {
    return u32x2{__builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_pkrtz(a, b)),
                 __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_pkrtz(c, d))};
  } else {
    return u32x2{__builtin_amdgcn_perm(__builtin_bit_cast(unsigned, b), __builtin_bit_cast(unsigned, a), 0x07060302),
                 __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, d), __builtin_bit_cast(unsigned, c), 0x07060302)};
  }
}
template <class T>
__device__ __forceinline__ u32x4 widen8(unsigned lo, unsigned hi) {
  const u32x2 a = widen4<T>(lo), b = widen4<T>(hi);
  return u32x4{a[0], a[1], b[0], b[1]};
}

template <int M>
using Scores = float __attribute__((ext_vector_type(M / 2)));  // a lane's, of 32 keys

// Products for row tiles of M = 32 or 16 query rows.  Scores of 32 keys: a lane
// holds row lane % M and 32 M / 64 keys.  O^T: floats i of a lane come in
// groups of four consecutive elements of the head.
template <class T, int M>
struct Form;
template <class T>
struct Form<T, 32> {
  using Acc = f32x16;
  static constexpr int kAcc = 16, kGroups = 2;
  __device__ static __forceinline__ Acc zero() { return zero16(); }
  __device__ static __forceinline__ Acc mma(u32x4 a, u32x4 b, Acc c) { return T::mma(a, b, c); }
  // key of score e, from the lane's first one on
  __device__ static __forceinline__ constexpr int key(int e) { return 8 * (e >> 2) + (e & 3); }
  __device__ static __forceinline__ int first_key(int lane) { return 4 * (lane >> 5); }
  // first head element of float group j of O^T
  __device__ static __forceinline__ int dim(int j, int lane) { return 32 * (j >> 2) + 8 * (j & 3) + 4 * (lane >> 5); }
  __device__ static __forceinline__ float max_row(float x) { return max_halves(x); }
  __device__ static __forceinline__ float add_row(float x) { return add_halves(x); }
};
__device__ __forceinline__ Halves quarters(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const unsigned lo = r[0], hi = r[1];
  return {__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
template <class T>
struct Form<T, 16> {
  using Acc = f32x4;
  static constexpr int kAcc = 4, kGroups = 4;
  __device__ static __forceinline__ Acc zero() { return Acc{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ static __forceinline__ Acc mma(u32x4 a, u32x4 b, Acc c) {
    if constexpr (T::kNarrow)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  __device__ static __forceinline__ constexpr int key(int e) { return e; }
  __device__ static __forceinline__ int first_key(int lane) { return 8 * (lane >> 4); }
  __device__ static __forceinline__ int dim(int j, int lane) { return 16 * j + 4 * (lane >> 4); }
  __device__ static __forceinline__ float max_row(float x) {
    const Halves q = quarters(max_halves(x));
    return fmaxf(q.lo, q.hi);
  }
  __device__ static __forceinline__ float add_row(float x) {
    const Halves q = quarters(add_halves(x));
    return q.lo + q.hi;
  }
};

// One workgroup's part of the work: all key heads of a range after one another
// on one XCD.
__device__ __forceinline__ Item item8_of(const AttnArgs &a) {
  uint32_t item;
  Item r;
  r.h = head_of(blockIdx.x, gridDim.x / a.hk, a.hk, &item);
  r.rt = item % a.rtiles;
  item /= a.rtiles;
  r.split = item % a.nsplit;
  item /= a.nsplit;
  r.qb = item % a.nqb;
  r.b = item / a.nqb;
  return r;
}

// The entries that a range takes.  Where every block is read, a sequence's own
// blocks are dealt evenly to the ranges (four at least): cut by the longest
// sequence's, 32 sequences of 21.5k of up to 32k keys fill 2.6 rounds of
// workgroups and take 330 us, dealt evenly 4 shorter ones and 278 us.
__device__ __forceinline__ Range range8_of(const AttnArgs &a, const Item &it, const Row &r) {
  Range x = range_of(a, it, r);
  if (!x.list && a.nsplit > 1) {
    const int32_t blocks = r.last_key < 0 ? 0 : r.last_key / kAttnPage + 1;
    const int32_t per = min(a.per_split, max(4, (blocks + a.nsplit - 1) / a.nsplit));
    x.e0 = it.split * per;
    x.e1 = min(blocks, x.e0 + per);
  }
  return x;
}

// 32 staged rows of D codes in 16-byte pieces, piece c of row r at piece
// c ^ f(r).  Rows 2r and 2r + 1 (4r .. 4r + 3 at D = 64) share a 256-byte row
// of banks; f is such that 16 lanes that read one piece each of rows 0..15, or
// of every other 4 rows of 32 (the key operand with 16 query rows), and 32
// lanes that read two neighbouring pieces of 8 rows (the transposing reads)
// fall on different banks.
template <int D>
struct Codes {
  static constexpr int kPieces = D / 16;
  static constexpr int kRowsPerLoad = 64 / kPieces;
  static constexpr int kLoads = 32 / kRowsPerLoad;
  __device__ static __forceinline__ int f(int r) {
    if constexpr (D == 128) return ((r >> 1) & 4) | ((r & 2)) | (((r >> 2) ^ (r >> 4)) & 1);
    return ((r >> 2) & 2) | (((r >> 2) ^ (r >> 4)) & 1);
  }
  __device__ static __forceinline__ int load_row(int i, int lane) { return kRowsPerLoad * i + lane / kPieces; }
  __device__ static __forceinline__ int load_byte(int i, int lane) {
    return ((lane % kPieces) ^ f(load_row(i, lane))) * 16;
  }
  __device__ static __forceinline__ u32x4 piece(const char *t, int row, int p) {
    return *(const __attribute__((address_space(3))) u32x4 *)(lds_addr(t) + row * D + ((p ^ f(row)) << 4));
  }
  // element 16 p + lane % 16 of eight rows: this lane gives the address of row
  // `row` (its own among the eight) and half lane & 1 of the piece
  __device__ static __forceinline__ u32x2 column(const char *t, int row, int p, int lane) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2 *)(
                   lds_addr(t) + row * D + ((p ^ f(row)) << 4) + (lane & 1) * 8)));
  }
};

__device__ __forceinline__ void load_lds4(uint32_t lds, i32x4 buf, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(buf)
               : "memory", "m0");
}

// The kernels' first argument, read again: what only the end of a kernel needs
// would else stay in registers across its loop, with all that was loaded with it.
__device__ __forceinline__ const AttnArgs &again() {
  auto p = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnArgs *)p;
}

// Where a head's codes and scales stand: at base + block * step + key * row,
// `block` its page, or without a table its own number.
struct Source {
  const char *codes;
  const float *scales;
  int64_t step;
  int32_t row, scale_step;
};
__device__ __forceinline__ Source source_of(const AttnArgs &a, const AttnView &x, const float *scales, const Item &it) {
  Source s;
  s.codes = x.p + it.h * x.sh + (a.table ? 0 : it.b * x.sb);
  s.step = a.table ? x.sb : kAttnPage * x.st;
  s.row = static_cast<int32_t>(x.st);
  s.scales = scales + ((a.table ? 0 : static_cast<int64_t>(it.b) * a.nkb) * a.hk + it.h) * kAttnPage;
  s.scale_step = a.hk * kAttnPage;
  // in registers of their own: the compiler else keeps all arguments that were
  // loaded with them across the loop, and spills them
  asm("s_mov_b64 %0, %1" : "=&s"(s.step) : "s"(s.step));
  asm("s_mov_b32 %0, %1" : "=&s"(s.row) : "s"(s.row));
  return s;
}
__device__ __forceinline__ const char *codes_at(const Source &s, int block, int32_t first) {
  return s.codes + block * s.step + first * s.row;
}
__device__ __forceinline__ const float *scales_at(const Source &s, int block, int32_t first) {
  return s.scales + static_cast<int64_t>(block) * s.scale_step + first;
}

// Which of the 32 keys from `key` on a row sees.
__device__ __forceinline__ uint32_t seen_of(const AttnArgs &a, const Row &r, int32_t key) {
  if (!a.tree) {
    const int32_t last = min(r.pos, r.len - 1) - key;
    return last >= 31 ? ~0u : (last < 0 ? 0u : (2u << last) - 1);
  }
  const int32_t drafts = r.len - r.start, before = r.start - key;  // before: keys of the text
  const uint64_t bits = drafts >= 64 ? r.bits : (drafts <= 0 ? 0 : r.bits & ((uint64_t(1) << drafts) - 1));
  if (before >= 32) return ~0u;
  if (before > 0) return static_cast<uint32_t>(bits << before) | ((1u << before) - 1);
  return before > -64 ? static_cast<uint32_t>(bits >> -before) : 0u;
}

// The scores s of N * 32 keys from key0 on (each lane's, times ks already) become
// weights, and o, m and l move with the maximum.
template <class T, int D, int M, int N, class Acc>
__device__ __forceinline__ void softmax8(const AttnArgs &a, const Row &r, int32_t key0, int lane, float c, Scores<M> *s,
                                         Stats &st, Acc *o) {
  using F = Form<T, M>;
  constexpr int E = M / 2;
  if (key0 + 32 * N > r.open) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const uint32_t seen = seen_of(a, r, key0 + 32 * n + F::first_key(lane));
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t keep = static_cast<int32_t>(seen << (31 - F::key(e))) >> 31;  // a vector register, no mask of lanes
        s[n][e] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, static_cast<float>(s[n][e])) & keep) | (0xff800000u & ~keep));
      }
    }
  }
  float top = s[0][0];
#pragma unroll
  for (int e = 1; e < N * E; ++e) top = fmaxf(top, s[e / E][e % E]);
  top = F::max_row(top) * c;
  if (__any(top > st.m + kSlack)) {
    const float next = fmaxf(st.m, top);
    const float f = next == -INFINITY ? 1.0f : exp2_(st.m - next);
    st.l *= f;
#pragma unroll
    for (int i = 0; i < D * M / 64; ++i) o[i / F::kAcc][i % F::kAcc] *= f;
    st.m = next;
  }
  const float from = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
  for (int e = 0; e < N * E; ++e) {
    s[e / E][e % E] = exp2_(__builtin_fmaf(s[e / E][e % E], c, -from));
    st.l += s[e / E][e % E];
  }
}

// A buffer of `bytes` bytes from p: loads past its end give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t records(const void *p, int32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, bytes, 0x00020000);
}

// Two weights as words of the two operands of a product with codes.
__device__ __forceinline__ void weights2(float a, float b, unsigned &hi, unsigned &lo) {
  hi = pack2<Bf16>(a, b);
  lo = pack2<Bf16>(a - elem<Bf16>(hi, 0), b - elem<Bf16>(hi, 1));
}

// o and lse of a lane's row, or its part of them where a list is cut into ranges.
template <class T, int D, int M, class Acc>
__device__ __forceinline__ void store8(const AttnArgs &a, const Item &it, const Row &r, int lane, float m, float l,
                                       const Acc *o) {
  using F = Form<T, M>;
  if (!r.real) return;
  const int64_t rid = (static_cast<int64_t>(it.b) * a.hq + r.head) * a.nq + r.tok;
  const bool split = a.nsplit > 1, none = l == 0.0f;
  const int64_t at = it.split * (static_cast<int64_t>(a.b) * a.hq * a.nq) + rid;
  if (lane < M) {
    if (split) {
      a.part_ml[2 * at] = m;
      a.part_ml[2 * at + 1] = l;
    } else {
      a.lse[rid] = none ? -INFINITY : (m + log2f(l)) * kLn2;
    }
  }
  if (split && m == -INFINITY && none) return;
  const float inv = none ? 0.0f : 1.0f / l;
  char *op = a.o.p + it.b * a.o.sb + r.tok * a.o.st + r.head * a.o.sh;
#pragma unroll
  for (int j = 0; j < D * M / 256; ++j) {
    f32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = o[(4 * j + e) / F::kAcc][(4 * j + e) % F::kAcc];
    if (split) {
      *reinterpret_cast<f32x4 *>(a.part_o + at * D + F::dim(j, lane)) = x;
    } else {
      u32x2 w;
      w[0] = none ? 0 : pack2<T>(x[0] * inv, x[1] * inv);
      w[1] = none ? 0 : pack2<T>(x[2] * inv, x[3] * inv);
      *reinterpret_cast<u32x2 *>(op + F::dim(j, lane) * 2) = w;
    }
  }
}

// Up to 32 rows to a list: each wave streams tiles of 32 keys through LDS of
// its own, without barriers: the next codes and scales of keys load during the
// softmax and the product with the values, the next of values during the
// scores.  KW waves share a list's tiles and join their sums.  Bound by memory:
// 32 sequences of 21.5k of up to 32k keys, 8 key heads of 4: 263 us for 1.42 GB,
// 5.4 TB/s, and the join of the ranges 6.
template <class T, int D, int M, int KW>
__global__ __launch_bounds__(64 * KW, M == 16 ? 4 : 2) void attn_stream8(const AttnArgs a, const AttnScales scales) {
  using F = Form<T, M>;
  using V = Form<Bf16, M>;
  using L = Codes<D>;
  constexpr int kSubs = kAttnPage / 32;
  constexpr int kTile = 32 * D;
  constexpr int kE = 32 * M / 64;
  constexpr int kLoads = L::kLoads + 1;
  constexpr int kO = D * M / 64 / F::kAcc;
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Item it = item8_of(a);
  const Row row = row_of<M>(a, it, M, 0, lane);
  const Range range = range8_of(a, it, row);
  const Source ksrc = source_of(a, a.k, scales.k, it), vsrc = source_of(a, a.v, scales.v, it);
  const int g = lane / M;
  u32x4 q[D / 8 / F::kGroups];
  {
    const char *p = a.q.p + (row.real ? it.b * a.q.sb + row.tok * a.q.st + row.head * a.q.sh : 0) + 32 * g;
#pragma unroll
    for (int s = 0; s < D / 8 / F::kGroups; ++s)
      q[s] = *reinterpret_cast<const u32x4 *>(p + 32 * F::kGroups * (s / 2) + 16 * (s % 2));
  }

  const char *kt = lds + wave * kTile * 2, *vt = kt + kTile;
  const char *ks = lds + KW * kTile * 2 + wave * 512, *vs = ks + 256;
  const uint32_t lds_k = __builtin_amdgcn_readfirstlane(lds_addr(kt));
  const uint32_t lds_ks = __builtin_amdgcn_readfirstlane(lds_addr(ks));
  uint32_t koff[L::kLoads], voff[L::kLoads];
#pragma unroll
  for (int i = 0; i < L::kLoads; ++i) {
    const int r = L::load_row(i, lane), c = L::load_byte(i, lane);
    koff[i] = static_cast<uint32_t>(r * ksrc.row + c);
    voff[i] = static_cast<uint32_t>(r * vsrc.row + c);
  }
  // rows of the transposing reads: the eight keys whose weights a lane holds
  const int i8 = (lane >> 1) & 7;
  const int krow = M == 32 ? lane & 31 : 8 * ((lane & 15) >> 2) + (lane & 3);
  const float c = a.scale * kLog2e;

  typename F::Acc o[kO];
#pragma unroll
  for (int i = 0; i < kO; ++i) o[i] = F::zero();
  Stats st;
  for (int32_t e = range.e0; e < range.e1; e += 64) {
    const Named blocks = named_blocks(range.list, range.table_row, a.pages, e, range.e1, row.last_key, lane);
    const int tiles = blocks.n * kSubs;
    // past the last tile the loads are of no bytes, so that the waits below
    // always count the same loads
    auto issue = [&](int t, bool values) {
      const int at = t < tiles ? t / kSubs : 0;
      const int id = __builtin_amdgcn_readlane(blocks.id, at);
      const int page = __builtin_amdgcn_readlane(blocks.page, at);
      const int32_t first = (t % kSubs) * 32;
      const int32_t kept = t < tiles ? min(32, row.last_key + 1 - id * kAttnPage - first) : 0;
      const Source &x = values ? vsrc : ksrc;
      const i32x4 buf = buffer(codes_at(x, page, first), kept > 0 ? (kept - 1) * x.row + D : 0);
      const i32x4 sbuf = buffer(reinterpret_cast<const char *>(scales_at(x, page, first)), kept > 0 ? kept * 4 : 0);
#pragma unroll
      for (int i = 0; i < L::kLoads; ++i)
        load_lds16(lds_k + (values ? kTile : 0) + i * 1024, buf, values ? voff[i] : koff[i]);
      load_lds4(lds_ks + (values ? 256 : 0), sbuf, lane * 4);
    };
    if (wave < tiles) {
      issue(wave, false);
      issue(wave, true);
    }
    for (int t = wave; t < tiles; t += KW) {
      const int32_t key0 = __builtin_amdgcn_readlane(blocks.id, t / kSubs) * kAttnPage + (t % kSubs) * 32;
      wait_vm<kLoads>();
      Scores<M> s;
      float w[kE];
#pragma unroll
      for (int i = 0; i < kE / 4; ++i) {
        const f32x4 x = *reinterpret_cast<const f32x4 *>(ks + 4 * (F::first_key(lane) + F::key(4 * i)));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = x[j];
      }
      {
        typename F::Acc acc[32 / M];
#pragma unroll
        for (int n = 0; n < 32 / M; ++n) {
          acc[n] = F::zero();
#pragma unroll
          for (int p = 0; p < D / 16 / F::kGroups; ++p) {
            const u32x4 x = L::piece(kt, krow + 4 * n, F::kGroups * p + g);
            acc[n] = F::mma(widen8<T>(x[0], x[1]), q[2 * p], acc[n]);
            acc[n] = F::mma(widen8<T>(x[2], x[3]), q[2 * p + 1], acc[n]);
          }
        }
#pragma unroll
        for (int i = 0; i < kE; ++i) s[i] = acc[i / F::kAcc][i % F::kAcc] * w[i];
      }
      wait_lds();
      issue(t + KW, false);
      softmax8<T, D, M, 1>(a, row, key0, lane, c, &s, st, o);
      wait_vm<kLoads>();
#pragma unroll
      for (int i = 0; i < kE / 4; ++i) {
        const f32x4 x = *reinterpret_cast<const f32x4 *>(vs + 4 * (F::first_key(lane) + F::key(4 * i)));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = s[4 * i + j] * x[j];
      }
#pragma unroll
      for (int n = 0; n < kE / 8; ++n) {
        u32x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          unsigned x, y;
          weights2(w[8 * n + 2 * i], w[8 * n + 2 * i + 1], x, y);
          hi[i] = x;
          lo[i] = y;
        }
        const int vrow = M == 32 ? 16 * n + 4 * g + (i8 & 3) + 2 * (i8 & 4) : 8 * g + i8;
#pragma unroll
        for (int i = 0; i < kO; ++i) {
          const u32x2 x = L::column(vt, vrow, M == 32 ? 2 * i + ((lane >> 4) & 1) : i, lane);
          const u32x4 v = widen8<Bf16>(x[0], x[1]);
          o[i] = V::mma(v, hi, o[i]);
          o[i] = V::mma(v, lo, o[i]);
        }
      }
      wait_lds();
      issue(t + KW, true);
    }
    wait_vm<0>();  // the loads of no bytes
  }

  st.l = F::add_row(st.l);
  if (!row.live) st = Stats();
  if constexpr (KW > 1) {  // the waves' sums, joined by the first in order
    constexpr int kFloats = D * M / 64;
    float *buf = reinterpret_cast<float *>(lds);
    __syncthreads();
    if (wave > 0) {
      float *p = buf + (wave - 1) * (kFloats + 2) * 64 + lane;
#pragma unroll
      for (int i = 0; i < kFloats; ++i) p[i * 64] = o[i / F::kAcc][i % F::kAcc];
      p[kFloats * 64] = st.m;
      p[(kFloats + 1) * 64] = st.l;
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll 1
    for (int w2 = 1; w2 < KW; ++w2) {
      const float *p = buf + (w2 - 1) * (kFloats + 2) * 64 + lane;
      const float m2 = p[kFloats * 64], l2 = p[(kFloats + 1) * 64];
      const float next = fmaxf(st.m, m2);
      const float f1 = st.m == -INFINITY ? 0.0f : exp2_(st.m - next);
      const float f2 = m2 == -INFINITY ? 0.0f : exp2_(m2 - next);
#pragma unroll
      for (int i = 0; i < kFloats; ++i)
        o[i / F::kAcc][i % F::kAcc] = o[i / F::kAcc][i % F::kAcc] * f1 + p[i * 64] * f2;
      st.l = st.l * f1 + l2 * f2;
      st.m = next;
    }
  }
  store8<T, D, M>(again(), it, row, lane, st.m, st.l, o);
}

// More rows to a list: RW waves of 32 rows share each staged tile of KT keys,
// KW groups of them take the tiles in turn.  The codes are widened once, on
// their way through registers to LDS, which then holds the tiles that the 16-bit
// kernel stages (the values' as bf16); the next tile's codes load during this
// one's products.  A group's first wave brings the scales.
//
// Bound by matrix and vector instructions, which the two waves of a SIMD hardly
// overlap: a wave's 64 keys take 1536 cycles of the matrix unit, a third of them
// for the weights' second operand, and about 2200 of the softmax, of widening and
// of splitting weights.  24 drafted tokens of 32 heads over 16 sequences of up to
// 8k keys, the same inputs again and again: 105 us (bf16) and 107 us (f16); with
// one operand of the element type 85 and 88 us, which left outputs at 1.4 times
// their own rounding's error, and f16 without digits beside values 2^27 as large.
// 64 keys to a softmax have one maximum, one test and one barrier where 32 have two
// (a fifth less time).
template <class T, int D, int RW, int KW, int KT>
__global__ __launch_bounds__(64 * RW * KW, 2) void attn_forward8(const AttnArgs a, const AttnScales scales) {
  using L = Tile<D>;
  using F = Form<T, 32>;
  constexpr int kThreads = 64 * RW;
  constexpr int kHalf = KT * L::kRowBytes;
  constexpr int kPieces = D / 16;                      // 16-byte pieces of codes in a row
  constexpr int kFetch = 2 * KT * kPieces / kThreads;  // of K and V together, a thread's
  static_assert((kFetch == 1 || kFetch % 2 == 0) && kFetch * kThreads == 2 * KT * kPieces && KT * kPieces % 64 == 0,
                "pieces of a tile");
  constexpr int kSubs = kAttnPage / KT;
  constexpr int kScales = 2 * KT;  // floats of a stage: K's, V's
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rw = wave % RW, kw = wave / RW;
  const Item it = item8_of(a);
  const Row row = row_of(a, it, 32 * RW, 32 * rw, lane);
  const Range range = range8_of(a, it, row);
  const Source ksrc = source_of(a, a.k, scales.k, it), vsrc = source_of(a, a.v, scales.v, it);
  const bool some = __any(row.live);  // a wave without rows only stages
  u32x4 q[D / 16];
  load_q<D>(a, it, row, lane, q);

  char *tiles_at = lds + kw * 4 * kHalf;  // two stages of K and V
  float *scales_of = reinterpret_cast<float *>(lds + KW * 4 * kHalf) + kw * 2 * kScales;
  // a thread's pieces, those of K first: where they stand in the block, and in
  // the stage (the second half of the widened piece at ^ 16)
  auto of_values = [&](int i) { return kFetch > 1 ? i >= kFetch / 2 : 64 * rw >= KT * kPieces; };
  uint32_t from[kFetch], to[kFetch];
#pragma unroll
  for (int i = 0; i < kFetch; ++i) {
    const int at = 64 * rw + lane + i * kThreads;
    const bool values = of_values(i);
    const int r = at / kPieces % KT, p = at % kPieces;
    from[i] = static_cast<uint32_t>(r * (values ? vsrc.row : ksrc.row) + 16 * p);
    to[i] = (values ? kHalf : 0) + r * L::kRowBytes + (((2 * p) ^ L::f(r)) << 4);
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
    u32x4 codes[kFetch];
    float ks = 0.0f, vs = 0.0f;
    // rows past the last key that some row sees are zeros, as are their scales
    auto fetch = [&](int round) {
      const int t = round * KW + kw;
      const int at = t < tiles ? t / kSubs : 0;
      const int id = __builtin_amdgcn_readlane(blocks.id, at);
      const int page = __builtin_amdgcn_readlane(blocks.page, at);
      const int32_t first = (t % kSubs) * KT;
      const int32_t kept = t < tiles ? min(KT, row.last_key + 1 - id * kAttnPage - first) : 0;
      const auto kbuf = records(codes_at(ksrc, page, first), kept > 0 ? (kept - 1) * ksrc.row + D : 0);
      const auto vbuf = records(codes_at(vsrc, page, first), kept > 0 ? (kept - 1) * vsrc.row + D : 0);
#pragma unroll
      for (int i = 0; i < kFetch; ++i) {
        const bool values = of_values(i);
        codes[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(values ? vbuf : kbuf, from[i], 0, 0));
      }
      if (rw == 0) {
        const int bytes = kept > 0 ? kept * 4 : 0;
        ks = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(records(scales_at(ksrc, page, first), bytes), 4 * lane, 0, 0));
        vs = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(records(scales_at(vsrc, page, first), bytes), 4 * lane, 0, 0));
      }
    };
    auto stage = [&](int round) {
      char *dst = tiles_at + (round & 1) * 2 * kHalf;
#pragma unroll
      for (int i = 0; i < kFetch; ++i) {
        const bool values = of_values(i);
        const u32x4 x = codes[i];
        *reinterpret_cast<u32x4 *>(dst + to[i]) = values ? widen8<Bf16>(x[0], x[1]) : widen8<T>(x[0], x[1]);
        *reinterpret_cast<u32x4 *>(dst + (to[i] ^ 16)) = values ? widen8<Bf16>(x[2], x[3]) : widen8<T>(x[2], x[3]);
      }
      if (rw == 0) {
        float *x = scales_of + (round & 1) * kScales;
        if (lane < KT) {
          x[lane] = ks;
          x[KT + lane] = vs;
        }
      }
    };
    if (rounds > 0) {
      fetch(0);
      stage(0);
      fetch(1);
    }
    for (int round = 0; round < rounds; ++round) {
      barrier();
      const char *kt = tiles_at + (round & 1) * 2 * kHalf, *vt = kt + kHalf;
      const float *xs = scales_of + (round & 1) * kScales;
      if (round + 1 < rounds) {
        stage(round + 1);
        fetch(round + 2);
      }
      const int t = round * KW + kw;
      if (t >= tiles || !some) continue;
      const int32_t key0 = __builtin_amdgcn_readlane(blocks.id, t / kSubs) * kAttnPage + (t % kSubs) * KT;
      constexpr int kN = KT / 32, kI = D / 32;
      const float *x = xs + F::first_key(lane);
      Scores<32> s[kN];
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        f32x16 acc = zero16();
        auto kx = operands<D / 16, kAhead>([&](int i) { return L::operand(kt, 32 * n, i, lane); });
        kx.begin();
        kx.run([&](int i, u32x4 k) { acc = T::mma(k, q[i], acc); });
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 f = *reinterpret_cast<const f32x4 *>(x + 32 * n + 8 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[n][4 * i + j] = acc[4 * i + j] * f[j];
        }
      }
      auto vx = operands<2 * kN * kI, kAhead>([&](int i) { return L::operand_t(vt, 16 * (i / kI), i % kI, lane); });
      vx.begin();
      softmax8<T, D, 32, kN>(a, row, key0, lane, c, s, st, o);
      u32x4 hi[2 * kN], lo[2 * kN];
#pragma unroll
      for (int i = 0; i < 4 * kN; ++i) {
        const f32x4 f = *reinterpret_cast<const f32x4 *>(x + KT + 8 * i);
        const float *w = reinterpret_cast<const float *>(s) + 4 * i;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          unsigned h, l;
          weights2(w[2 * j] * f[2 * j], w[2 * j + 1] * f[2 * j + 1], h, l);
          hi[i / 2][2 * (i % 2) + j] = h;
          lo[i / 2][2 * (i % 2) + j] = l;
        }
      }
      vx.run([&](int i, u32x4 v) {
        o[i % kI] = Bf16::mma(v, hi[i / kI], o[i % kI]);
        o[i % kI] = Bf16::mma(v, lo[i / kI], o[i % kI]);
      });
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
  store8<T, D, 32>(again(), it, row, lane, st.m, st.l, o);
}

int64_t grid_of(const AttnArgs &a) {
  return static_cast<int64_t>(a.b) * a.hk * a.nqb * a.rtiles * a.nsplit;
}

template <class T, int D, int M, int KW>
hipError_t run_stream8(const AttnArgs &a, const AttnScales &x, hipStream_t s) {
  constexpr size_t kTiles = static_cast<size_t>(KW) * (64 * D + 512);
  constexpr size_t kSums = static_cast<size_t>(KW - 1) * (D * M / 64 + 2) * 256;
  constexpr size_t kLds = kTiles > kSums ? kTiles : kSums;
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_stream8<T, D, M, KW>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_stream8<T, D, M, KW>), dim3(static_cast<unsigned>(grid_of(a))), dim3(64 * KW), kLds, s, a, x);
  return hipGetLastError();
}

template <class T, int D, int RW, int KW, int KT>
hipError_t run_forward8(const AttnArgs &a, const AttnScales &x, hipStream_t s) {
  constexpr size_t kTiles = KW * (static_cast<size_t>(8) * KT * D + 16 * KT);
  constexpr size_t kSums = static_cast<size_t>(KW - 1) * RW * (D / 2 + 2) * 256;
  constexpr size_t kLds = kTiles > kSums ? kTiles : kSums;
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_forward8<T, D, RW, KW, KT>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_forward8<T, D, RW, KW, KT>), dim3(static_cast<unsigned>(grid_of(a))), dim3(64 * RW * KW), kLds, s,
                     a, x);
  return hipGetLastError();
}

template <class T, int D>
hipError_t run8(const AttnArgs &a, const AttnScales &x, spmm_dtype_t t, hipStream_t s) {
  if (grid_of(a) == 0) return hipSuccess;
  if (grid_of(a) > 0x7fffffff) return hipErrorInvalidValue;
  hipError_t e;
  switch (attn_tile(a.rows, a.nqb).row_waves) {
    // A wave a list where there are lists enough to fill the chip and a sequence's
    // queries read keys of each other's from L2; rows of 16 where they fit.  8 blocks
    // for every query, 8 key heads of 4: 2048 lists take 39 us, with four waves each 43,
    // 1024 28 and 26.5, 32k 333 and 401, with rows of 32 441.  One query each, from
    // memory: 300 sequences of 2k keys take 294 us with a wave a head, 245 with four.  32
    // sequences of 8k keys: rows of 16 119 us, of 32 147.
    case 1: {
      const bool alone = a.nqb > 1 && grid_of(a) >= 2048 && a.nsplit == 1;
      if (a.rows <= 16)
        e = alone ? run_stream8<T, D, 16, 1>(a, x, s) : run_stream8<T, D, 16, 4>(a, x, s);
      else
        e = alone ? run_stream8<T, D, 32, 1>(a, x, s) : run_stream8<T, D, 32, 4>(a, x, s);
      break;
    }
    // 2048 queries of 8 heads, 16 blocks for each 64: two groups of waves to a list
    // 31 us, one 49.  With four waves of rows a second group gains little or loses:
    // 26.4 us for 24 drafted tokens over 8k keys, 25.8 without; over 16 sequences 112
    // and 107; 2048 queries of 16 heads over lists 38 and 41.
    case 2: e = run_forward8<T, D, 2, 2, 32>(a, x, s); break;
    case 4: e = run_forward8<T, D, 4, 1, 64>(a, x, s); break;
    default: e = run_forward8<T, D, 8, 1, 64>(a, x, s); break;
  }
  return e != hipSuccess || a.nsplit == 1 ? e : launch_attn_merge(a, t, D, s);
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_cache8(const AttnArgs &a, const AttnScales &x, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16) return d == 64 ? attn::run8<attn::Bf16, 64>(a, x, t, s) : attn::run8<attn::Bf16, 128>(a, x, t, s);
  return d == 64 ? attn::run8<attn::F16, 64>(a, x, t, s) : attn::run8<attn::F16, 128>(a, x, t, s);
}

}  // namespace sdm
