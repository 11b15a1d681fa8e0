// attn_dev.h -- device pieces the attention kernels share: element types,
// staged tiles and their swizzle, direct loads, lists.
//
// Every product is an MFMA 32x32x16 with the operands in the order that lets
// a result feed the next product from its own registers: lane l holds column
// l % 32, and its element e is row 8 (e / 4) + 4 (l / 32) + e % 4.  Where
// those rows are contracted next, the 8 elements 8s .. 8s+7 are the B operand
// of one MFMA if the A operand takes its contraction in the same order, rows
// 16s + 4h + 0..3 and 16s + 8 + 4h + 0..3 for half-wave h, which is what two
// transposing 8-byte reads of a staged tile give (operand_t below).
#pragma once

#include "attn.h"

// load_lds16 names m0 as clobbered on purpose (it sets m0 for the LDS-DMA
// instruction); clang warns about clobbering a reserved register.
#pragma clang diagnostic ignored "-Winline-asm"

namespace sdm {
namespace attn {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kCus = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Bf16 {
  using E = __bf16;
  static constexpr bool kNarrow = false;  // reaches as far as 32 bits
  __device__ static f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
};
struct F16 {
  using E = _Float16;
  static constexpr bool kNarrow = true;  // infinite from 65520 on
  __device__ static f32x16 mma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};

// two floats to the element type, round to nearest even, first in the low half
template <class T>
__device__ __forceinline__ unsigned pack2(float x, float y) {
  typedef typename T::E E2 __attribute__((ext_vector_type(2)));
  E2 v = {static_cast<typename T::E>(x), static_cast<typename T::E>(y)};
  return __builtin_bit_cast(unsigned, v);
}
// elements 8s .. 8s+7 of a result as an operand
template <class T>
__device__ __forceinline__ u32x4 pack8(const f32x16 &x, int s) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack2<T>(x[8 * s + 2 * i], x[8 * s + 2 * i + 1]);
  return r;
}
template <class T>
__device__ __forceinline__ float elem(unsigned v, int i) {
  typedef typename T::E E2 __attribute__((ext_vector_type(2)));
  return static_cast<float>(__builtin_bit_cast(E2, v)[i]);
}

// the same, and what the rounding left out as a second operand
template <class T>
__device__ __forceinline__ void split8(const f32x16 &x, int s, u32x4 &hi, u32x4 &lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = x[8 * s + 2 * i], b = x[8 * s + 2 * i + 1];
    hi[i] = pack2<T>(a, b);
    lo[i] = pack2<T>(a - elem<T>(hi[i], 0), b - elem<T>(hi[i], 1));
  }
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int e = 0; e < 16; ++e) z[e] = 0.0f;
  return z;
}

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// x of this lane and of lane ^ 32, combined.  The halves go through values of
// their own: a bit cast of a vector's element reads element 0.
struct Halves {
  float lo, hi;
};
__device__ __forceinline__ Halves halves(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned lo = r[0], hi = r[1];
  return {__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
__device__ __forceinline__ float max_halves(float x) {
  const Halves h = halves(x);
  return fmaxf(h.lo, h.hi);
}
__device__ __forceinline__ float add_halves(float x) {
  const Halves h = halves(x);
  return h.lo + h.hi;
}

// Workgroup i of n * heads as a head and one of n items.  Workgroups go to the
// XCDs in turn; each XCD takes all heads of an item one after another, so that
// what stands side by side of a token is read and written by one XCD at about one
// time.
__device__ __forceinline__ uint32_t head_of(uint32_t i, uint32_t n, uint32_t heads, uint32_t *item) {
  const uint32_t even = n / 8 * 8;  // items that go round all XCDs
  if (i < even * heads) {
    *item = i / (8 * heads) * 8 + i % 8;
    return i % (8 * heads) / 8;
  }
  i -= even * heads;
  *item = even + i % (n - even);
  return i / (n - even);
}

// Reductions over aligned groups of N = 8 or 16 lanes: neighbours, pairs, then
// the mirror images of 8 and 16 lanes, whose partners hold the other half.
template <int CTRL>
__device__ __forceinline__ unsigned dpp(unsigned x) {
  return static_cast<unsigned>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), CTRL, 0xf, 0xf, true));
}
template <int N, class F>
__device__ __forceinline__ unsigned over_lanes(unsigned x, F f) {
  static_assert(N == 8 || N == 16, "lanes of a row");
  x = f(x, dpp<0xb1>(x));   // lane ^ 1
  x = f(x, dpp<0x4e>(x));   // lane ^ 2
  x = f(x, dpp<0x141>(x));  // 7 - lane
  if constexpr (N == 16) x = f(x, dpp<0x140>(x));  // 15 - lane
  return x;
}
template <int N>
__device__ __forceinline__ float sum_lanes(float x) {
  return __builtin_bit_cast(float, over_lanes<N>(__builtin_bit_cast(unsigned, x), [](unsigned p, unsigned q) {
    return __builtin_bit_cast(unsigned, __builtin_bit_cast(float, p) + __builtin_bit_cast(float, q));
  }));
}

// s_waitcnt vmcnt(n), leaving the other counters alone
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

// Workgroup barrier after this wave's LDS reads have completed (so no read
// of a stage can still be in flight when another wave refills it), without
// waiting for the direct loads in flight (their waits are explicit).
__device__ __forceinline__ void barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The same for a stage that no other wave reads.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char *)(p)));
}

// A buffer of `bytes` bytes from base: direct loads past its end write zeros.
// A load must come five wait states after a vector instruction that wrote one
// of its scalar registers, as the reads of a first lane do.  The compiler does
// not see to that in front of asm.
__device__ __forceinline__ i32x4 buffer(const char *base, int32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const int lo = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(a)));
  const int hi = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(a >> 32) & 0xffffu));
  int size = __builtin_amdgcn_readfirstlane(bytes);
  asm("s_nop 4" : "+s"(size) : "s"(lo), "s"(hi));
  return i32x4{lo, hi, size, 0x00020000};
}

// Direct load of 16 bytes per lane: LDS[lds + 16 * lane] = buffer[voff].
// Inline asm, so the compiler neither waits on it (the kernels count vmcnt
// themselves) nor assumes later LDS reads depend on it.  The load must come one
// wait state after the write of M0 that gives its LDS address, which the
// compiler does not see to inside asm.
__device__ __forceinline__ void load_lds16(uint32_t lds, i32x4 buf, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(buf)
               : "memory", "m0");
}
// 4 bytes a lane: LDS[lds + 4 * lane] = *p.
__device__ __forceinline__ void load_lds4(uint32_t lds, const float *p) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory", "m0");
}

// A staged tile: rows of d elements in 16-byte pieces, piece c of row r at
// piece c ^ f(r).  One f serves both kinds of reads without bank conflicts:
// 16 consecutive rows at one piece land on 16 distinct pieces of the 256-byte
// bank row (f is a bijection of r % 16, with two rows to a bank row at d =
// 64), and so do 4 aligned rows at 4 aligned pieces (the transposing reads),
// because those rows differ in f's upper bits.
template <int D>
struct Tile {
  static constexpr int kRowBytes = D * 2;
  static constexpr int kPieces = kRowBytes / 16;
  static constexpr int kRowsPerLoad = 64 / kPieces;  // rows of a 1 KB direct load
  __device__ static __forceinline__ int f(int r) {
    return D == 128 ? (((r & 3) << 2) | ((r >> 2) & 3)) : ((((r >> 1) & 1) << 2) | ((r >> 2) & 3));
  }
  // the row and byte of a row that this lane fetches in 1 KB load i
  __device__ static __forceinline__ int load_row(int i, int lane) { return kRowsPerLoad * i + lane / kPieces; }
  __device__ static __forceinline__ int load_byte(int i, int lane) {
    return ((lane % kPieces) ^ f(load_row(i, lane))) * 16;
  }
  // A operand over the row: lane l gives row row0 + l % 32, elements
  // 16 step + 8 (l / 32) + 0..7.  row0 is a multiple of 32, t of 256 bytes.
  // The swizzle is an XOR, so steps differ by an XOR of the lane's address:
  // one register serves all of them.
  __device__ static __forceinline__ u32x4 operand(const char *t, int row0, int step, int lane) {
    const int r = lane & 31;
    const uint32_t at = lds_addr(t) + r * kRowBytes + (((lane >> 5) ^ f(r)) << 4);
    return *(const __attribute__((address_space(3))) u32x4 *)((at ^ (step << 5)) + row0 * kRowBytes);
  }
  // A operand of the tile's transpose: lane l gives element 32 dt + l % 32 of
  // rows row0 + 4 (l / 32) + 0..3 and row0 + 8 + 4 (l / 32) + 0..3.  row0 is
  // a multiple of 16.  f(r + 8) is f(r) ^ 2 for r < 8.
  __device__ static __forceinline__ u32x4 operand_t(const char *t, int row0, int dt, int lane) {
    const int r = ((lane >> 2) & 3) + 4 * (lane >> 5);
    const int piece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const uint32_t at = lds_addr(t) + r * kRowBytes + ((piece ^ f(r)) << 4) + (lane & 1) * 8;
    const u32x2 lo = tr((at ^ (dt << 6)) + row0 * kRowBytes);
    const u32x2 hi = tr((at ^ (dt << 6 | 32)) + (row0 + 8) * kRowBytes);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
  __device__ static __forceinline__ u32x2 tr(uint32_t at) {
    return __builtin_bit_cast(
        u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)(at)));
  }
};

// N products whose LDS operands are read AHEAD products before their use (left
// to itself the compiler reads each right before it and waits the latency out:
// a prompt of 32k tokens took 1177 us that way, 1101 us with reads ahead; only
// scalar and vector arithmetic may move across pin()).  begin() reads the
// first ones, which may stand before other work.
__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0x406); }
template <int N, int AHEAD, class R>
struct Operands {
  R read;
  u32x4 buf[N];
  __device__ __forceinline__ Operands(R r) : read(r) {}
  __device__ __forceinline__ void begin() {
#pragma unroll
    for (int i = 0; i < AHEAD && i < N; ++i) buf[i] = read(i);
    pin();
  }
  __device__ __forceinline__ void next(int i) {
    if (i + AHEAD < N) buf[i + AHEAD] = read(i + AHEAD);
  }
  template <class M>
  __device__ __forceinline__ void run(M mul) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      next(i);
      pin();
      mul(i, buf[i]);
      pin();
    }
  }
};
template <int N, int AHEAD, class R>
__device__ __forceinline__ Operands<N, AHEAD, R> operands(R read) {
  return Operands<N, AHEAD, R>(read);
}

// Up to 64 entries e0 .. e1 of a list, one a lane: the blocks they name with
// a key at or below last_key whose page exists, in order in the first n lanes.
struct Named {
  int id, page, n;
};
__device__ __forceinline__ Named named_blocks(const int32_t *list, const int32_t *table_row, int32_t pages,
                                              int32_t e0, int32_t e1, int32_t last_key, int lane) {
  const int32_t e = e0 + lane;
  int id = -1, page = -1;
  if (e < e1) id = list ? list[e] : e;
  if (attn_names(id, last_key)) page = attn_page(table_row, id, pages);
  const uint64_t ok = __ballot(page >= 0);
  const uint32_t lo = static_cast<uint32_t>(ok), hi = static_cast<uint32_t>(ok >> 32);
  const int before = __builtin_amdgcn_mbcnt_hi(hi, __builtin_amdgcn_mbcnt_lo(lo, 0));
  const int n = __builtin_popcountll(ok);
  const int to = page >= 0 ? before : n + lane - before;  // every lane has a place of its own
  Named r;
  r.id = __builtin_amdgcn_ds_permute(4 * to, id);
  r.page = __builtin_amdgcn_ds_permute(4 * to, page);
  r.n = __builtin_amdgcn_readfirstlane(n);
  return r;
}

// The blocks that consecutive lists of per_list entries name (those lists
// whose bit is set in `take`), each once, in the first n lanes; members has
// the bits of the lists that name it.  At most 64 entries in all, one a lane.
// A block that a list names twice stands twice.
struct Shared {
  int id, page, members, n;
};
__device__ __forceinline__ Shared shared_blocks(const int32_t *lists, int entries, int per_list,
                                                const int32_t *table_row, int32_t pages, uint32_t take,
                                                int32_t last_key, int lane) {
  int id = lane < entries ? lists[lane] : -1;
  const int list = lane / per_list;
  if (!attn_names(id, last_key) || !(take >> (list & 31) & 1)) id = -1;
  const int page = id >= 0 ? attn_page(table_row, id, pages) : -1;
  if (page < 0) id = -1;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const uint64_t one = per_list >= 64 ? ~uint64_t(0) : (uint64_t(1) << per_list) - 1;
  auto equal = [&](int key) {  // the lanes whose key is this lane's
    unsigned lo = 0, hi = 0;
    for (int l = 0; l < entries; ++l) {
      const uint64_t m = __ballot(key == __builtin_amdgcn_readlane(key, l));
      lo = lane == l ? static_cast<unsigned>(m) : lo;
      hi = lane == l ? static_cast<unsigned>(m >> 32) : hi;
    }
    return uint64_t(hi) << 32 | lo;
  };
  uint64_t same = equal(id);
  const int again = __builtin_popcountll(same & (one << (list * per_list & 63)) & below);
  if (__any(id >= 0 && again > 0)) same = equal(id * 64 + again);  // id < 2^25
  int members = 0;
  for (int l = 0; l * per_list < entries; ++l) members |= ((same & (one << (l * per_list))) != 0) << l;
  const bool leads = id >= 0 && (same & below) == 0;
  const uint64_t ok = __ballot(leads);
  const int before = __builtin_popcountll(ok & below), n = __builtin_popcountll(ok);
  const int to = leads ? before : n + lane - before;  // every lane has a place of its own
  Shared r;
  r.id = __builtin_amdgcn_ds_permute(4 * to, id);
  r.page = __builtin_amdgcn_ds_permute(4 * to, page);
  r.members = __builtin_amdgcn_ds_permute(4 * to, members);
  r.n = __builtin_amdgcn_readfirstlane(n);
  return r;
}

}  // namespace attn
}  // namespace sdm
