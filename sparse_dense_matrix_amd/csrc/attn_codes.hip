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

// A workgroup's rows: D / 8 lanes a row, heads fastest, rows from `base` on.
struct CodeRow {
  int32_t b, t, h;
};
template <int D>
__device__ __forceinline__ CodeRow code_row(const AttnCodesArgs &a) {
  constexpr int kRows = 256 / (D / 8);
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  const int64_t token = base / a.hk;
  const uint32_t head = static_cast<uint32_t>(base % a.hk) + threadIdx.x / (D / 8);
  const uint32_t t = static_cast<uint32_t>(token % a.n) + head / static_cast<uint32_t>(a.hk);
  CodeRow r;
  r.h = static_cast<int32_t>(head % static_cast<uint32_t>(a.hk));
  r.b = static_cast<int32_t>(token / a.n + t / static_cast<uint32_t>(a.n));
  r.t = static_cast<int32_t>(t % static_cast<uint32_t>(a.n));
  return r;
}

// Slot of a sequence's key, and where its row of codes stands; slot < 0: nowhere.
struct Place {
  int64_t slot, k8, v8;
  int32_t at;
};
__device__ __forceinline__ Place place_of(const AttnCodesArgs &a, int32_t b, int32_t pos, int32_t h) {
  Place p;
  p.at = pos % kAttnPage;
  if (a.table) {
    p.slot = attn_page(a.table + static_cast<int64_t>(b) * a.nkb, pos / kAttnPage, a.pages);
    p.k8 = p.slot * a.k8.sb + p.at * a.k8.st;
    p.v8 = p.slot * a.v8.sb + p.at * a.v8.st;
  } else {
    p.slot = static_cast<int64_t>(b) * a.nkb + pos / kAttnPage;
    p.k8 = b * a.k8.sb + pos * a.k8.st;
    p.v8 = b * a.v8.sb + pos * a.v8.st;
  }
  p.k8 += h * a.k8.sh;
  p.v8 += h * a.v8.sh;
  return p;
}

// A lane's eight elements as codes, and the row's scale.  The largest magnitude
// is found among the bits, where a NaN is above infinity.
template <class T, int D>
__device__ __forceinline__ u32x2 encode(u32x4 v, float &scale) {
  float x[8];
  unsigned top_bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = elem<T>(v[i / 2], i & 1);
    top_bits = max(top_bits, __builtin_bit_cast(unsigned, x[i]) & 0x7fffffffu);
  }
  top_bits = over_lanes<D / 8>(top_bits, [](unsigned p, unsigned q) { return max(p, q); });
  const float top = __builtin_bit_cast(float, top_bits);
  scale = top / 127.0f;
  u32x2 r = {0, 0};
  if (top_bits == 0 || top_bits >= 0x7f800000u) return r;
  // both sides of the quotient 2^-8 times as large where 127 top passes 2^128
  const float f = !T::kNarrow && top >= 0x1p120f ? 0x1p-8f : 1.0f;
  const float num = 127.0f * f, den = top * f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int code = static_cast<int>(__builtin_rintf(num * x[i] / den));
    r[i / 4] |= static_cast<unsigned>(code & 0xff) << (8 * (i % 4));
  }
  return r;
}

// D / 8 lanes take a token's key and value of a head.
template <class T, int D>
__global__ __launch_bounds__(256) void attn_write(const AttnCodesArgs a) {
  const CodeRow r = code_row<D>(a);
  if (r.b >= a.b) return;
  const int64_t pos = static_cast<int64_t>(a.starts ? a.starts[r.b] : 0) + r.t;
  if (pos < 0 || pos >= attn_len(a.lens, r.b, a.nk)) return;
  const Place p = place_of(a, r.b, static_cast<int32_t>(pos), r.h);
  if (p.slot < 0) return;
  const int lane = threadIdx.x % (D / 8);
  const u32x4 k = *reinterpret_cast<const u32x4 *>(a.k.p + r.b * a.k.sb + r.t * a.k.st + r.h * a.k.sh + 16 * lane);
  const u32x4 v = *reinterpret_cast<const u32x4 *>(a.v.p + r.b * a.v.sb + r.t * a.v.st + r.h * a.v.sh + 16 * lane);
  float ks, vs;
  const u32x2 kc = encode<T, D>(k, ks), vc = encode<T, D>(v, vs);
  *reinterpret_cast<u32x2 *>(a.k8.p + p.k8 + 8 * lane) = kc;
  *reinterpret_cast<u32x2 *>(a.v8.p + p.v8 + 8 * lane) = vc;
  const int64_t at = (p.slot * a.hk + r.h) * kAttnPage + p.at;
  if (lane == 0) a.k_scale[at] = ks;
  if (lane == 1) a.v_scale[at] = vs;
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
__global__ __launch_bounds__(256) void attn_read(const AttnCodesArgs a) {
  const CodeRow r = code_row<D>(a);
  if (r.b >= a.b || r.t >= attn_len(a.lens, r.b, a.nk)) return;
  const Place p = place_of(a, r.b, r.t, r.h);
  const int lane = threadIdx.x % (D / 8);
  u32x2 kc = {0, 0}, vc = {0, 0};
  float ks = 0.0f, vs = 0.0f;
  if (p.slot >= 0) {
    kc = *reinterpret_cast<const u32x2 *>(a.k8.p + p.k8 + 8 * lane);
    vc = *reinterpret_cast<const u32x2 *>(a.v8.p + p.v8 + 8 * lane);
    const int64_t at = (p.slot * a.hk + r.h) * kAttnPage + p.at;
    ks = a.k_scale[at];
    vs = a.v_scale[at];
  }
  *reinterpret_cast<u32x4 *>(a.k.p + r.b * a.k.sb + r.t * a.k.st + r.h * a.k.sh + 16 * lane) = decode<T>(kc, ks);
  *reinterpret_cast<u32x4 *>(a.v.p + r.b * a.v.sb + r.t * a.v.st + r.h * a.v.sh + 16 * lane) = decode<T>(vc, vs);
}

template <class T, int D, bool READ>
hipError_t run_codes(const AttnCodesArgs &a, hipStream_t s) {
  constexpr int kRows = 256 / (D / 8);
  const int64_t rows = static_cast<int64_t>(a.b) * a.n * a.hk;
  const int64_t grid = (rows + kRows - 1) / kRows;
  if (grid == 0) return hipSuccess;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  if constexpr (READ)
    hipLaunchKernelGGL((attn_read<T, D>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((attn_write<T, D>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a);
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
