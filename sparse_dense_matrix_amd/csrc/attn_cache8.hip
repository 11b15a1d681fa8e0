// attn_cache8.hip -- attention over a cache in 8 bits: key j of a head stands
// as codes c_j with a scale ks_j, its value as codes d_j with vs_j, and
//   o_t = sum_j p_tj vs_j d_j,   p_tj = exp(scale ks_j (q_t . c_j) - lse_t),
// over the keys j that query t sees (attn_forward.hip has the same sums over a
// cache in 16 bits, and the form of the softmax).
//
// The codes are whole numbers up to 127, which bf16 and f16 hold exactly, so
// nothing is rounded on the way to the products: a score is the sum of q_t's
// elements times the codes in 32 bits, then times ks_j.  The value's scale goes
// to the weight: p_tj vs_j is rounded to bf16 for the product with d_j, at most
// half a step of each weight.  For f16 outputs, whose step is eight times
// finer, it goes as two bf16 operands, the weight and what its rounding left
// out (2^-17 of it): a weight times a value's scale can pass f16's range both
// ways, bf16 reaches as far as 32 bits.  The sum that divides is of p_tj itself.
#include "attn_rows.h"
#include "internal.h"

namespace sdm {
namespace attn {
namespace {

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

// `kept` rows of codes from key `first` of a block on, and their scales, as buffers
// (zeros past them).
template <int D>
__device__ __forceinline__ i32x4 codes_of(const AttnArgs &a, const AttnView &x, const Item &it, int id, int page,
                                          int32_t first, int32_t kept) {
  const char *p = x.p + it.h * x.sh;
  if (a.table)
    p += page * x.sb + first * x.st;
  else
    p += it.b * x.sb + (static_cast<int64_t>(id) * kAttnPage + first) * x.st;
  return buffer(p, kept > 0 ? static_cast<int32_t>((kept - 1) * x.st + D) : 0);
}
__device__ __forceinline__ const float *scales_at(const AttnArgs &a, const float *x, const Item &it, int id, int page,
                                                  int32_t first) {
  const int64_t slot = a.table ? page : static_cast<int64_t>(it.b) * a.nkb + id;
  return x + (slot * a.hk + it.h) * kAttnPage + first;
}

// The scores s of 32 keys from key0 on (each lane's, times ks already) become
// weights, and o, m and l move with the maximum.
template <class T, int D, int M, int E, class Acc>
__device__ __forceinline__ void softmax8(const AttnArgs &a, const Row &r, int32_t key0, int lane, float c, float (&s)[E],
                                         Stats &st, Acc *o) {
  using F = Form<T, M>;
  if (key0 + 32 > r.open) {
    if (a.tree) {
      const int32_t before = r.start - (key0 + F::first_key(lane));  // keys of the text
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int32_t draft = F::key(e) - before;
        const uint64_t bit = draft < 64 ? r.bits >> (draft & 63) : 0;
        s[e] = (draft < 0 || (bit & 1)) && draft < r.len - r.start ? s[e] : -INFINITY;
      }
    } else {
      const int32_t last = min(r.pos, r.len - 1) - (key0 + F::first_key(lane));
#pragma unroll
      for (int e = 0; e < E; ++e) s[e] = F::key(e) <= last ? s[e] : -INFINITY;
    }
  }
  float top = s[0];
#pragma unroll
  for (int e = 1; e < E; ++e) top = fmaxf(top, s[e]);
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
  for (int e = 0; e < E; ++e) {
    s[e] = exp2_(__builtin_fmaf(s[e], c, -from));
    st.l += s[e];
  }
}

// Eight weights as the operand of a product with codes, and what their
// rounding left out (f16 outputs).
__device__ __forceinline__ void weights8(const float *w, u32x4 &hi, u32x4 *lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hi[i] = pack2<Bf16>(w[2 * i], w[2 * i + 1]);
    if (lo) (*lo)[i] = pack2<Bf16>(w[2 * i] - elem<Bf16>(hi[i], 0), w[2 * i + 1] - elem<Bf16>(hi[i], 1));
  }
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
// scores.  KW waves share a list's tiles and join their sums.
template <class T, int D, int M, int KW>
__global__ __launch_bounds__(64 * KW, M == 16 ? 4 : 3) void attn_stream8(const AttnArgs a, const AttnScales scales) {
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
  const Item it = item_of(a);
  const Row row = row_of<M>(a, it, M, 0, lane);
  const Range range = range_of(a, it, row);
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
    koff[i] = static_cast<uint32_t>(r * a.k.st + c);
    voff[i] = static_cast<uint32_t>(r * a.v.st + c);
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
      const i32x4 buf = codes_of<D>(a, values ? a.v : a.k, it, id, page, first, kept);
      const i32x4 sbuf = buffer(reinterpret_cast<const char *>(scales_at(a, values ? scales.v : scales.k, it, id, page, first)),
                                kept > 0 ? kept * 4 : 0);
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
      float s[kE], w[kE];
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
      softmax8<T, D, M>(a, row, key0, lane, c, s, st, o);
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
        weights8(w + 8 * n, hi, T::kNarrow ? &lo : nullptr);
        const int vrow = M == 32 ? 16 * n + 4 * g + (i8 & 3) + 2 * (i8 & 4) : 8 * g + i8;
#pragma unroll
        for (int i = 0; i < kO; ++i) {
          const u32x2 x = L::column(vt, vrow, M == 32 ? 2 * i + ((lane >> 4) & 1) : i, lane);
          const u32x4 v = widen8<Bf16>(x[0], x[1]);
          o[i] = V::mma(v, hi, o[i]);
          if constexpr (T::kNarrow) o[i] = V::mma(v, lo, o[i]);
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
#pragma unroll
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
  store8<T, D, M>(a, it, row, lane, st.m, st.l, o);
}

// More rows to a list: RW waves of 32 rows share each staged tile of KT keys.
// The codes are widened once, on their way to LDS, which then holds the tiles
// that the 16-bit kernel stages; the next tile's codes come in during the
// products of this one.
template <class T, int D, int RW, int KT>
__global__ __launch_bounds__(64 * RW, 2) void attn_forward8(const AttnArgs a, const AttnScales scales) {
  using L = Tile<D>;
  using F = Form<T, 32>;
  constexpr int kThreads = 64 * RW;
  constexpr int kHalf = KT * L::kRowBytes, kStage = 2 * kHalf + 2 * KT * 4;
  constexpr int kPieces = D / 16;                  // 16-byte pieces of codes in a row
  constexpr int kFetch = 2 * KT * kPieces / kThreads;  // of K and V together, a thread's
  static_assert(kFetch >= 1 && kFetch * kThreads == 2 * KT * kPieces, "pieces of a tile");
  static_assert(2 * KT <= kThreads, "scales of a tile");
  constexpr int kSubs = kAttnPage / KT, kE = KT / 2;
  extern __shared__ __attribute__((aligned(1024))) char lds[];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Item it = item_of(a);
  const Row row = row_of(a, it, 32 * RW, 32 * wave, lane);
  const Range range = range_of(a, it, row);
  u32x4 q[D / 16];
  load_q<D>(a, it, row, lane, q);

  f32x16 o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = zero16();
  Stats st;
  const float c = a.scale * kLog2e;

  for (int32_t e = range.e0; e < range.e1; e += 64) {
    const Named blocks = named_blocks(range.list, range.table_row, a.pages, e, range.e1, row.last_key, lane);
    const int tiles = blocks.n * kSubs;
    u32x4 codes[kFetch];
    float scale = 0.0f;
    // rows past the last key that some row sees count as zeros: what stands
    // there may be anything
    auto fetch = [&](int t) {
      if (t >= tiles) return;
      const int id = __builtin_amdgcn_readlane(blocks.id, t / kSubs);
      const int page = __builtin_amdgcn_readlane(blocks.page, t / kSubs);
      const int32_t first = (t % kSubs) * KT, kept = row.last_key + 1 - id * kAttnPage - first;
#pragma unroll
      for (int i = 0; i < kFetch; ++i) {
        const int at = tid + i * kThreads;
        const bool values = at >= KT * kPieces;
        const int r = at / kPieces % KT, p = at % kPieces;
        const AttnView &x = values ? a.v : a.k;
        const char *src = x.p + it.h * x.sh;
        src += a.table ? page * x.sb + (first + r) * x.st
                       : it.b * x.sb + (static_cast<int64_t>(id) * kAttnPage + first + r) * x.st;
        codes[i] = u32x4{0, 0, 0, 0};
        if (r < kept) codes[i] = *reinterpret_cast<const u32x4 *>(src + 16 * p);
      }
      if (tid < 2 * KT) {
        const int r = tid % KT;
        scale = r < kept ? scales_at(a, tid < KT ? scales.k : scales.v, it, id, page, first)[r] : 0.0f;
      }
    };
    auto stage = [&](int t) {
      if (t >= tiles) return;
      char *to = lds + (t & 1) * kStage;
#pragma unroll
      for (int i = 0; i < kFetch; ++i) {
        const int at = tid + i * kThreads;
        const bool values = at >= KT * kPieces;
        const int r = at / kPieces % KT, p = at % kPieces;
        char *dst = to + (values ? kHalf : 0) + r * L::kRowBytes;
        const u32x4 x = codes[i];
        const u32x4 lo = values ? widen8<Bf16>(x[0], x[1]) : widen8<T>(x[0], x[1]);
        const u32x4 hi = values ? widen8<Bf16>(x[2], x[3]) : widen8<T>(x[2], x[3]);
        *reinterpret_cast<u32x4 *>(dst + (((2 * p) ^ L::f(r)) << 4)) = lo;
        *reinterpret_cast<u32x4 *>(dst + (((2 * p + 1) ^ L::f(r)) << 4)) = hi;
      }
      if (tid < 2 * KT) reinterpret_cast<float *>(to + 2 * kHalf)[tid] = scale;
    };
    fetch(0);
    stage(0);
    fetch(1);
    for (int t = 0; t < tiles; ++t) {
      __syncthreads();
      stage(t + 1);
      fetch(t + 2);
      const char *kt = lds + (t & 1) * kStage, *vt = kt + kHalf;
      const float *ks = reinterpret_cast<const float *>(vt + kHalf), *vs = ks + KT;
      const int32_t key0 = __builtin_amdgcn_readlane(blocks.id, t / kSubs) * kAttnPage + (t % kSubs) * KT;
#pragma unroll
      for (int n = 0; n < KT / 32; ++n) {
        f32x16 acc = zero16();
#pragma unroll
        for (int x = 0; x < D / 16; ++x) acc = T::mma(L::operand(kt, 32 * n, x, lane), q[x], acc);
        float s[16], w[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 x = *reinterpret_cast<const f32x4 *>(ks + 32 * n + F::first_key(lane) + 8 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) s[4 * i + j] = acc[4 * i + j] * x[j];
        }
        softmax8<T, D, 32>(a, row, key0 + 32 * n, lane, c, s, st, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 x = *reinterpret_cast<const f32x4 *>(vs + 32 * n + F::first_key(lane) + 8 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[4 * i + j] = s[4 * i + j] * x[j];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4 hi, lo;
          weights8(w + 8 * h, hi, T::kNarrow ? &lo : nullptr);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const u32x4 v = L::operand_t(vt, 32 * n + 16 * h, i, lane);
            o[i] = Bf16::mma(v, hi, o[i]);
            if constexpr (T::kNarrow) o[i] = Bf16::mma(v, lo, o[i]);
          }
        }
      }
    }
    // the next entries' first tile goes where the last one may still be read
    __syncthreads();
  }

  st.l = add_halves(st.l);
  if (!row.live) st = Stats();
  store8<T, D, 32>(a, it, row, lane, st.m, st.l, o);
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

template <class T, int D, int RW, int KT>
hipError_t run_forward8(const AttnArgs &a, const AttnScales &x, hipStream_t s) {
  constexpr size_t kLds = 2 * (static_cast<size_t>(4) * KT * D + 8 * KT);
  hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_forward8<T, D, RW, KT>), kLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_forward8<T, D, RW, KT>), dim3(static_cast<unsigned>(grid_of(a))), dim3(64 * RW), kLds, s, a, x);
  return hipGetLastError();
}

template <class T, int D>
hipError_t run8(const AttnArgs &a, const AttnScales &x, spmm_dtype_t t, hipStream_t s) {
  if (grid_of(a) == 0) return hipSuccess;
  if (grid_of(a) > 0x7fffffff) return hipErrorInvalidValue;
  hipError_t e;
  switch (attn_tile(a.rows, a.nqb).row_waves) {
    // a wave a list where there are enough lists to fill the chip twice over
    case 1: {
      const bool alone = grid_of(a) >= 4096 && a.nsplit == 1;
      if (a.rows <= 16)
        e = alone ? run_stream8<T, D, 16, 1>(a, x, s) : run_stream8<T, D, 16, 4>(a, x, s);
      else
        e = alone ? run_stream8<T, D, 32, 1>(a, x, s) : run_stream8<T, D, 32, 4>(a, x, s);
      break;
    }
    case 2: e = run_forward8<T, D, 2, 32>(a, x, s); break;
    case 4: e = run_forward8<T, D, 4, 32>(a, x, s); break;
    default: e = run_forward8<T, D, 8, 64>(a, x, s); break;
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
