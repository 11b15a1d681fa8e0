// attn_codes.hip -- a cache in 8 bits, written and read back.  A row is one
// token's key or value of one head:
//   top = max_c |x_c|,  scale = top / 127,  code_c = round(127 x_c / top),
// and code_c * scale is what it stands for, within scale / 2 of x_c.
//
// The quotient is rounded as the number it is, ties to the even code: 127 x_c
// takes at most 18 bits, and a quotient of such numbers that is not half a
// whole number is further from one than a correctly rounded division is off.
#include "attn_dev.h"
#include "internal.h"

namespace sdm {
namespace attn {
namespace {

// A key's row of codes and its scale, block by block: `page` of a table, or without
// one the block's own number.
struct Place {
  int64_t k8, v8, scale;
};
__device__ __forceinline__ Place place_of(const AttnCodesArgs &a, int32_t b, int32_t h, int32_t page) {
  Place p;
  p.k8 = h * a.k8.sh + (a.table ? page * a.k8.sb : b * a.k8.sb + page * kAttnPage * a.k8.st);
  p.v8 = h * a.v8.sh + (a.table ? page * a.v8.sb : b * a.v8.sb + page * kAttnPage * a.v8.st);
  p.scale = ((a.table ? page : static_cast<int64_t>(b) * a.nkb + page) * a.hk + h) * kAttnPage;
  return p;
}
__device__ __forceinline__ int32_t page_of(const AttnCodesArgs &a, int32_t b, int32_t block) {
  return attn_page(a.table ? a.table + static_cast<int64_t>(b) * a.nkb : nullptr, block, a.pages);
}

// top / 127, correctly rounded: a quotient that is off by a step corrected by its
// remainder, which is exact (Markstein), where no result is subnormal.
__device__ __forceinline__ float scale_of(float top) {
  if (__any(top < 0x1p-100f)) return top / 127.0f;
  constexpr float kBy = 1.0f / 127.0f;
  const float q = top * kBy;
  return top < INFINITY ? __builtin_fmaf(__builtin_fmaf(-127.0f, q, top), kBy, q) : top;
}

// A lane's eight elements as codes, and the row's scale.  The largest magnitude
// is found among the bits, where a NaN is above infinity.
template <class T, int D>
__device__ __forceinline__ u32x2 encode(u32x4 v, float &scale) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 most = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, v[i] & 0x7fff7fffu));
  unsigned bits = max(static_cast<unsigned>(most[0]), static_cast<unsigned>(most[1]));
  bits = over_lanes<D / 8>(bits, [](unsigned p, unsigned q) { return max(p, q); });
  const float top = elem<T>(bits, 0);
  scale = scale_of(top);
  u32x2 r = {0, 0};
  if (!(top > 0.0f && top < INFINITY)) return r;
  // 1.5 2^23 added to the quotient leaves it rounded in the last byte.  Times a
  // reciprocal, taken 2^-21 too large, it is off by up to 127 2^-20, so that what
  // comes that near to a tie is divided: a wave in twelve, but for ties of top / 2,
  // which a row in three of 8-bit values has and which 63.5 and more rounds to their
  // even code, 64.  Where the reciprocal or 127 times it leaves the normal numbers,
  // all are divided.
  const float by = (127.0f + 127.0f * 0x1p-21f) * __builtin_amdgcn_rcpf(top);
  float x[8], t[8], far = top > 0x1p-100f && top < 0x1p120f ? 0.0f : 1.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = elem<T>(v[i / 2], i & 1);
    t[i] = __builtin_fmaf(x[i], by, 0x1.8p23f);
    const float off = __builtin_fmaf(x[i], by, -(t[i] - 0x1.8p23f));
    far = fmaxf(far, fabsf(2.0f * fabsf(x[i]) == top ? 0.0f : off));
  }
  if (__any(!(far <= 0.5f - 0x1p-13f))) {
    // both sides of the quotient 2^-8 times as large where 127 top passes 2^128
    const float f = !T::kNarrow && top >= 0x1p120f ? 0x1p-8f : 1.0f;
    const float num = 127.0f * f, den = top * f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = num * x[i] / den + 0x1.8p23f;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned *w = reinterpret_cast<const unsigned *>(t + 4 * i);
    r[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(w[3], w[2], 0x0c0c0400), __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0400),
                                 0x05040100);
  }
  return r;
}

// Few rows: D / 8 lanes take a token's key and value of a head each, heads
// fastest.  The rows load before it is known whether and where they go, which takes
// two loads after one another.  A token of 32 sequences, 8 heads of 128: 3.5 us, a
// launch of nothing 3.
template <class T, int D>
__global__ __launch_bounds__(256) void attn_write_rows(const AttnCodesArgs a) {
  constexpr uint32_t kRows = 256 / (D / 8);
  const uint32_t heads = a.hk, n = a.n;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  const int64_t token = base / heads;
  const uint32_t head = static_cast<uint32_t>(base % heads) + threadIdx.x / (D / 8);
  const uint32_t tt = static_cast<uint32_t>(token % n) + head / heads;
  const int32_t h = static_cast<int32_t>(head % heads), b = static_cast<int32_t>(token / n + tt / n);
  const int32_t t = static_cast<int32_t>(tt % n), lane = threadIdx.x % (D / 8);
  if (b >= a.b) return;
  const u32x4 k = *reinterpret_cast<const u32x4 *>(a.k.p + b * a.k.sb + t * a.k.st + h * a.k.sh + 16 * lane);
  const u32x4 v = *reinterpret_cast<const u32x4 *>(a.v.p + b * a.v.sb + t * a.v.st + h * a.v.sh + 16 * lane);
  const int64_t pos = static_cast<int64_t>(a.starts ? a.starts[b] : 0) + t;
  const int32_t len = attn_len(a.lens, b, a.nk);
  float ks, vs;
  const u32x2 kc = encode<T, D>(k, ks), vc = encode<T, D>(v, vs);
  if (pos < 0 || pos >= len) return;
  const int32_t page = page_of(a, b, static_cast<int32_t>(pos) / kAttnPage), at = static_cast<int32_t>(pos) % kAttnPage;
  if (page < 0) return;
  const Place p = place_of(a, b, h, page);
  *reinterpret_cast<u32x2 *>(a.k8.p + p.k8 + at * a.k8.st + 8 * lane) = kc;
  *reinterpret_cast<u32x2 *>(a.v8.p + p.v8 + at * a.v8.st + 8 * lane) = vc;
  if (lane == 0) a.k_scale[p.scale + at] = ks;
  if (lane == 1) a.v_scale[p.scale + at] = vs;
}

// More tokens: a workgroup takes a block of one head, so that where it stands is
// found once, in scalar registers, and its lines of scales are written by one
// workgroup.  16k tokens of 8 heads: token by token the addresses took more
// instructions than the codes (26 us).
template <class T, int D>
__global__ __launch_bounds__(256) void attn_write(const AttnCodesArgs a, uint32_t width) {
  constexpr int kRows = 256 / (D / 8), kU = kAttnPage / kRows;
  uint32_t item;
  const int32_t h = static_cast<int32_t>(head_of(blockIdx.x, gridDim.x / a.hk, a.hk, &item));
  const int32_t b = static_cast<int32_t>(item / width);
  const int64_t start = a.starts ? a.starts[b] : 0;
  const AttnTaken x = attn_taken(start, a.n, attn_len(a.lens, b, a.nk), item % width);
  if (x.lo >= x.hi) return;
  const int32_t page = page_of(a, b, x.id);
  const int lane = threadIdx.x % (D / 8), group = threadIdx.x / (D / 8);
  const int64_t t = static_cast<int64_t>(x.id) * kAttnPage - start;  // of the block's first key
  const char *kp = a.k.p + b * a.k.sb + h * a.k.sh + t * a.k.st, *vp = a.v.p + b * a.v.sb + h * a.v.sh + t * a.v.st;
  u32x4 k[kU], v[kU];
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int at = min(max(group + i * kRows, x.lo), x.hi - 1);
    k[i] = *reinterpret_cast<const u32x4 *>(kp + at * a.k.st + 16 * lane);
    v[i] = *reinterpret_cast<const u32x4 *>(vp + at * a.v.st + 16 * lane);
  }
  if (page < 0) return;
  const Place p = place_of(a, b, h, page);
  char *k8 = a.k8.p + p.k8, *v8 = a.v8.p + p.v8;
  float *ks = a.k_scale + p.scale, *vs = a.v_scale + p.scale;
  const int32_t kst = static_cast<int32_t>(a.k8.st), vst = static_cast<int32_t>(a.v8.st);
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int at = group + i * kRows;
    float kf, vf;
    const u32x2 kc = encode<T, D>(k[i], kf), vc = encode<T, D>(v[i], vf);
    if (at < x.lo || at >= x.hi) continue;
    *reinterpret_cast<u32x2 *>(k8 + static_cast<uint32_t>(at * kst + 8 * lane)) = kc;
    *reinterpret_cast<u32x2 *>(v8 + static_cast<uint32_t>(at * vst + 8 * lane)) = vc;
    if (lane == 0) ks[at] = kf;
    if (lane == 1) vs[at] = vf;
  }
}

template <class T>
__device__ __forceinline__ u32x4 decode(u32x2 c, float scale) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = pack2<T>(static_cast<float>(static_cast<int8_t>(c[i / 2] >> (16 * (i % 2)))) * scale,
                    static_cast<float>(static_cast<int8_t>(c[i / 2] >> (16 * (i % 2) + 8))) * scale);
  return r;
}

template <class T, int D>
__global__ __launch_bounds__(256) void attn_read(const AttnCodesArgs a, uint32_t width) {
  constexpr int kRows = 256 / (D / 8), kU = kAttnPage / kRows;
  uint32_t item;
  const int32_t h = static_cast<int32_t>(head_of(blockIdx.x, gridDim.x / a.hk, a.hk, &item));
  const int32_t b = static_cast<int32_t>(item / width);
  const AttnTaken x = attn_taken(0, a.n, attn_len(a.lens, b, a.nk), item % width);
  if (x.hi <= 0) return;
  const int32_t page = page_of(a, b, x.id);
  const int lane = threadIdx.x % (D / 8), group = threadIdx.x / (D / 8);
  u32x2 k[kU], v[kU];
  float kf[kU], vf[kU];
  if (page >= 0) {
    const Place p = place_of(a, b, h, page);
    const char *k8 = a.k8.p + p.k8, *v8 = a.v8.p + p.v8;
    const int32_t kst = static_cast<int32_t>(a.k8.st), vst = static_cast<int32_t>(a.v8.st);
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int at = min(group + i * kRows, x.hi - 1);
      k[i] = *reinterpret_cast<const u32x2 *>(k8 + static_cast<uint32_t>(at * kst + 8 * lane));
      v[i] = *reinterpret_cast<const u32x2 *>(v8 + static_cast<uint32_t>(at * vst + 8 * lane));
      kf[i] = a.k_scale[p.scale + at];
      vf[i] = a.v_scale[p.scale + at];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      k[i] = v[i] = u32x2{0, 0};
      kf[i] = vf[i] = 0.0f;
    }
  }
  const int64_t t = static_cast<int64_t>(x.id) * kAttnPage;
  char *kp = a.k.p + b * a.k.sb + h * a.k.sh + t * a.k.st, *vp = a.v.p + b * a.v.sb + h * a.v.sh + t * a.v.st;
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    const int at = group + i * kRows;
    if (at >= x.hi) break;
    *reinterpret_cast<u32x4 *>(kp + at * a.k.st + 16 * lane) = decode<T>(k[i], kf[i]);
    *reinterpret_cast<u32x4 *>(vp + at * a.v.st + 16 * lane) = decode<T>(v[i], vf[i]);
  }
}

template <class T, int D, bool READ>
hipError_t run_codes(const AttnCodesArgs &a, hipStream_t s) {
  const AttnCodesLaunch x = attn_codes_launch(a, D, READ);
  if (x.groups == 0) return hipSuccess;
  if (x.groups > kAttnMaxGroups) return hipErrorInvalidValue;
  const dim3 blocks(static_cast<unsigned>(x.groups));
  const uint32_t width = static_cast<uint32_t>(x.width);
  if (x.rows)
    hipLaunchKernelGGL((attn_write_rows<T, D>), blocks, dim3(256), 0, s, a);
  else if constexpr (READ)
    hipLaunchKernelGGL((attn_read<T, D>), blocks, dim3(256), 0, s, a, width);
  else
    hipLaunchKernelGGL((attn_write<T, D>), blocks, dim3(256), 0, s, a, width);
  return hipGetLastError();
}

template <bool READ>
hipError_t launch(const AttnCodesArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16) return d == 64 ? run_codes<Bf16, 64, READ>(a, s) : run_codes<Bf16, 128, READ>(a, s);
  return d == 64 ? run_codes<F16, 64, READ>(a, s) : run_codes<F16, 128, READ>(a, s);
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_write(const AttnCodesArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  return attn::launch<false>(a, t, d, s);
}
hipError_t launch_attn_read(const AttnCodesArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  return attn::launch<true>(a, t, d, s);
}

}  // namespace sdm
