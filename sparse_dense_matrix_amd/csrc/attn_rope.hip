// attn_rope.hip -- what queries and keys go through before attention: the norm
// of each head, then the rotation of pairs of its channels by their position,
//   y_c = x_c r w_c,  r = (mean_c x_c^2 + eps)^(-1/2),
//   (o_u, o_v) = (y_u cos a - y_v sin a, y_u sin a + y_v cos a),
//   a = positions[axis of the pair] * freq of the pair,
// and the gradients, with g that of o:
//   (dy_u, dy_v) = (g_u cos a + g_v sin a, g_v cos a - g_u sin a),
//   dw_c = sum over rows of dy_c x_c r,
//   dx_c = r (dy_c w_c - x_c r^2 mean_c(dy_c w_c x_c)).
//
// An angle is taken in turns, in 64 bits: 2 pi, the frequency over it and the
// product with the position leave 3 2^-53 of the turns, and the fraction of a turn
// is rounded to 32 bits, 2^-26 of a turn (position 2^31 at one radian each: 2^-22.9
// of a turn in all; positions below 2^20: 2^-26).  Each token's angles are computed
// once for all heads, one a thread, and kept in LDS.  Everything else is in 32 bits,
// rounded once at the output.
#include "attn_dev.h"
#include "internal.h"

namespace sdm {
namespace attn {
namespace {

constexpr int kTile = 4;  // tokens of a workgroup of the backward kernel at a time

// TOK tokens from t0 of all sequences' tokens in one row: place and whether they
// count, and the angles of their pairs.
template <int D, int TOK>
struct RopeShared {
  float cosine[TOK][D / 2], sine[TOK][D / 2];
  float w[2][D];
  int32_t b[TOK], t[TOK], live[TOK];
};

template <int D, int TOK>
__device__ __forceinline__ void angles(const RopeArgs &a, RopeShared<D, TOK> &sh, uint32_t t0, uint32_t count) {
  const uint32_t pairs = max(a.pairs, 1), n = a.n;
  for (uint32_t i = threadIdx.x; i < count * pairs; i += 256) {
    const uint32_t tt = i / pairs, p = i % pairs;
    const uint32_t b = (t0 + tt) / n, t = (t0 + tt) % n;
    const int64_t at = static_cast<int64_t>(a.starts ? a.starts[b] : 0) + t;
    if (p == 0) {
      sh.b[tt] = static_cast<int32_t>(b);
      sh.t[tt] = static_cast<int32_t>(t);
      sh.live[tt] = !a.lens || (at >= 0 && at < a.lens[b]);
    }
    if (a.pairs > 0) {
      const double pos = static_cast<double>(
          a.positions ? a.positions[(static_cast<int64_t>(a.axis[p]) * a.b + b) * a.n + t] : at);
      const double turns = pos * a.turns[p];
      float s, c;
      sincospif(2.0f * static_cast<float>(turns - rint(turns)), &s, &c);
      sh.cosine[tt][p] = c;
      sh.sine[tt][p] = s;
    }
  }
}

template <int D, int TOK>
__device__ __forceinline__ void load_weights(const RopeArgs &a, RopeShared<D, TOK> &sh) {
  for (int i = threadIdx.x; i < 2 * D; i += 256) {
    const float *w = a.w[i / D];
    sh.w[i / D][i % D] = w ? w[i % D] : 1.0f;
  }
}

__device__ __forceinline__ char *row_at(const AttnView &v, int32_t b, int32_t t, int32_t h, int lane) {
  return v.p + b * v.sb + t * v.st + h * v.sh + 16 * lane;
}

// What a lane needs to turn its eight channels: where its angles and its
// partner's channels stand.
struct Turn {
  int first;    // of the lane's angles (8, or 4 where neighbours are pairs)
  int partner;  // lane of the row that holds the pairs' other channels
  bool turned, second;
};
template <int D>
__device__ __forceinline__ Turn turn_of(const RopeArgs &a, int lane) {
  Turn u;
  const int half = a.pairs / 8;  // lanes of the first channels
  if (a.interleaved) {
    u = {4 * lane, lane, 4 * lane < a.pairs, false};
  } else {
    u.second = lane >= half;
    u.turned = lane < 2 * half;
    u.first = 8 * (u.second ? lane - half : lane);
    u.partner = !u.turned ? lane : (u.second ? lane - half : lane + half);
  }
  if (!u.turned) u.first = 0;
  return u;
}

// A lane's cosines and sines of one token: of its first 4 pairs where neighbours
// are pairs, else of 8.
struct Angles {
  float c[8], s[8];
};
template <int D, int TOK>
__device__ __forceinline__ Angles angles_of(const RopeArgs &a, const RopeShared<D, TOK> &sh, int tt, const Turn &u) {
  Angles x;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool there = u.turned && (i < 4 || !a.interleaved);
    x.c[i] = there ? sh.cosine[tt][u.first + i] : 1.0f;
    x.s[i] = there ? sh.sine[tt][u.first + i] : 0.0f;
  }
  return x;
}

// x turned by its angles c and s (back: the other way), registers or LDS.  `other`
// are the pairs' other channels where the halves are paired.
__device__ __forceinline__ void rotate(const RopeArgs &a, const float *c, const float *s, const Turn &u, bool back,
                                       float *x, const float *other) {
  if (!u.turned) return;
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sn = back ? -s[i] : s[i], p = x[2 * i], q = x[2 * i + 1];
      x[2 * i] = p * c[i] - q * sn;
      x[2 * i + 1] = p * sn + q * c[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + other[i] * (u.second != back ? s[i] : -s[i]);
  }
}

// The partner lane's words.
template <int D>
__device__ __forceinline__ u32x4 from_partner(u32x4 v, const Turn &u) {
  const int from = 4 * ((threadIdx.x & 63 & ~(D / 8 - 1)) + u.partner);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = static_cast<unsigned>(__builtin_amdgcn_ds_bpermute(from, static_cast<int>(v[i])));
  return r;
}

// A lane's eight channels of a row, normed where there is a weight (w: of the
// lane's channels, w2: of its partner's) and turned.
template <class T, int D>
__device__ __forceinline__ u32x4 turned(const RopeArgs &a, u32x4 v, bool norm, const float *w, const float *w2,
                                        const Angles &turn, const Turn &u) {
  const u32x4 p = from_partner<D>(v, u);
  float x[8], y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = elem<T>(v[e / 2], e & 1);
    y[e] = elem<T>(p[e / 2], e & 1);
  }
  if (norm) {
    float sum = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(x[e], x[e], sum);
    const float r = rsqrtf(sum_lanes<D / 8>(sum) * (1.0f / D) + a.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = x[e] * r * w[e];
      y[e] = y[e] * r * w2[e];
    }
  }
  rotate(a, turn.c, turn.s, u, false, x, y);
  u32x4 out;
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = pack2<T>(x[2 * e], x[2 * e + 1]);
  return out;
}

// Few rows: D / 8 lanes take one each, all heads of a token after one another.
// Bound by its chain of loads and steps; the row loads before the angles are
// computed.  32 tokens of 32 and 8 heads of 128: 4.4 us, a launch of nothing 3.
template <class T, int D>
__global__ __launch_bounds__(256) void rope_rows(const RopeArgs a) {
  constexpr int kLanes = D / 8, kGroups = 256 / kLanes;
  __shared__ RopeShared<D, kGroups / 2 + 1> sh;  // two heads at least
  const uint32_t heads = a.heads[0] + a.heads[1], tokens = static_cast<uint32_t>(a.b) * a.n;
  const uint32_t r0 = blockIdx.x * kGroups, t0 = r0 / heads;  // few rows: below 2^32
  const uint32_t count = min((r0 + kGroups - 1) / heads + 1, tokens) - t0;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const uint32_t r = min(r0 + group, tokens * heads - 1), token = r / heads;
  const int32_t hh = r % heads, b = token / a.n, t = token % a.n;
  const bool key = hh >= a.heads[0];
  const int32_t h = key ? hh - a.heads[0] : hh;
  const u32x4 v = *reinterpret_cast<const u32x4 *>(row_at(key ? a.x[1] : a.x[0], b, t, h, lane));
  angles<D>(a, sh, t0, count);
  load_weights<D>(a, sh);
  __syncthreads();
  const int tt = token - t0;
  if (r0 + group >= tokens * heads || !sh.live[tt]) return;
  const Turn u = turn_of<D>(a, lane);
  const u32x4 out = turned<T, D>(a, v, a.w[key] != nullptr, sh.w[key] + 8 * lane, sh.w[key] + 8 * u.partner,
                                 angles_of<D>(a, sh, tt, u), u);
  *reinterpret_cast<u32x4 *>(row_at(key ? a.y[1] : a.y[0], b, t, h, lane)) = out;
}

// More rows: a token has 256 / (D / 8) / TOK groups of D / 8 lanes, which take its
// heads in turn, so that a lane keeps its token's angles and its channels'
// weights; the next rows load while rows are turned.  16k tokens of 32 and 8
// heads: 72 us, 4.7 TB/s (a row at a time with its heads counted out by divisions:
// 123 us).
template <class T, int D, int TOK>
__global__ __launch_bounds__(256) void rope_forward(const RopeArgs a) {
  constexpr int kLanes = D / 8, kGroups = 256 / kLanes, kOf = kGroups / TOK, kU = 4;
  __shared__ RopeShared<D, TOK> sh;
  const uint32_t tokens = static_cast<uint32_t>(a.b) * a.n, t0 = blockIdx.x * TOK;
  const uint32_t count = min(static_cast<uint32_t>(TOK), tokens - t0);
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int tt = group / kOf, sub = group % kOf;
  const uint32_t token = t0 + min(static_cast<uint32_t>(tt), count - 1);
  const int32_t b = token / a.n, t = token % a.n;
  angles<D>(a, sh, t0, count);
  load_weights<D>(a, sh);
  __syncthreads();
  if (tt >= static_cast<int>(count) || !sh.live[tt]) return;
  const Turn u = turn_of<D>(a, lane);
  const Angles turn = angles_of<D>(a, sh, tt, u);
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    const AttnView &from = a.x[side], &to = a.y[side];
    const int heads = a.heads[side];
    const bool norm = a.w[side] != nullptr;
    float w[8], w2[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w[e] = sh.w[side][8 * lane + e];
      w2[e] = sh.w[side][8 * u.partner + e];
    }
    u32x4 v[kU], next[kU];
    auto load = [&](int h0, u32x4 *to_regs) {
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (h0 + i * kOf < heads) to_regs[i] = *reinterpret_cast<const u32x4 *>(row_at(from, b, t, h0 + i * kOf, lane));
    };
    load(sub, v);
    for (int h0 = sub; h0 < heads; h0 += kU * kOf) {
      load(h0 + kU * kOf, next);
#pragma unroll
      for (int i = 0; i < kU; ++i) {
        const int h = h0 + i * kOf;
        if (h >= heads) break;
        *reinterpret_cast<u32x4 *>(row_at(to, b, t, h, lane)) = turned<T, D>(a, v[i], norm, w, w2, turn, u);
      }
#pragma unroll
      for (int i = 0; i < kU; ++i) v[i] = next[i];
    }
  }
}

// Workgroups take tiles in turn; each lane sums the weights' gradients of its
// channels over its rows, and the workgroup's sums go to the workspace.  16k tokens
// of 32 and 8 heads of 128: 108 us for 503 MB, 4.7 TB/s, bound by memory: tiles of
// 2 and 8 tokens and 4 rows in flight take as long.  Angles kept in registers, as
// forward, leave room for too few rows: 112 us.
template <class T, int D>
__global__ __launch_bounds__(256) void rope_backward(const RopeArgs a) {
  constexpr int kLanes = D / 8, kGroups = 256 / kLanes, kU = 2;
  __shared__ RopeShared<D, kTile> sh;
  __shared__ float sums[kGroups][D];
  const int64_t tokens = static_cast<int64_t>(a.b) * a.n;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const Turn u = turn_of<D>(a, lane);
  load_weights<D>(a, sh);
  float dw[2][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[0][e] = dw[1][e] = 0.0f;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTile; t0 < tokens; t0 += static_cast<int64_t>(gridDim.x) * kTile) {
    const int count = static_cast<int>(min(static_cast<int64_t>(kTile), tokens - t0));
    __syncthreads();
    angles<D>(a, sh, static_cast<uint32_t>(t0), count);
    __syncthreads();
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int heads = a.heads[side];
      const bool norm = a.w[side] != nullptr;
      for (int r0 = group; r0 < count * heads; r0 += kU * kGroups) {
        u32x4 gv[kU], xv[kU];
        int tt[kU], h[kU];
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          const int r = r0 + i * kGroups;
          tt[i] = min(r / heads, kTile - 1);
          h[i] = r < count * heads ? r % heads : -1;
          gv[i] = xv[i] = u32x4{0, 0, 0, 0};
          if (h[i] < 0 || !sh.live[tt[i]]) continue;
          gv[i] = *reinterpret_cast<const u32x4 *>(row_at(a.g[side], sh.b[tt[i]], sh.t[tt[i]], h[i], lane));
          if (norm) xv[i] = *reinterpret_cast<const u32x4 *>(row_at(a.x[side], sh.b[tt[i]], sh.t[tt[i]], h[i], lane));
        }
#pragma unroll
        for (int i = 0; i < kU; ++i) {
          if (h[i] < 0) continue;
          const u32x4 w = from_partner<D>(gv[i], u);
          float dy[8], other[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dy[e] = elem<T>(gv[i][e / 2], e & 1);
            other[e] = elem<T>(w[e / 2], e & 1);
          }
          rotate(a, sh.cosine[tt[i]] + u.first, sh.sine[tt[i]] + u.first, u, true, dy, other);
          if (norm) {
            float x[8], sum = 0.0f, dot = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x[e] = elem<T>(xv[i][e / 2], e & 1);
              sum = __builtin_fmaf(x[e], x[e], sum);
            }
            const float r = rsqrtf(sum_lanes<kLanes>(sum) * (1.0f / D) + a.eps);
            if (!sh.live[tt[i]]) {
#pragma unroll
              for (int e = 0; e < 8; ++e) dy[e] = 0.0f;
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                dw[side][e] = __builtin_fmaf(dy[e], x[e] * r, dw[side][e]);
                dy[e] *= sh.w[side][8 * lane + e];
                dot = __builtin_fmaf(dy[e], x[e], dot);
              }
              const float f = sum_lanes<kLanes>(dot) * (1.0f / D) * r * r;
#pragma unroll
              for (int e = 0; e < 8; ++e) dy[e] = r * (dy[e] - x[e] * f);
            }
          }
          u32x4 out;
#pragma unroll
          for (int e = 0; e < 4; ++e) out[e] = pack2<T>(dy[2 * e], dy[2 * e + 1]);
          *reinterpret_cast<u32x4 *>(row_at(a.dx[side], sh.b[tt[i]], sh.t[tt[i]], h[i], lane)) = out;
        }
      }
    }
  }
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    if (!a.dw[side]) continue;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[group][8 * lane + e] = dw[side][e];
    __syncthreads();
    if (threadIdx.x < D) {
      float x = 0.0f;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) x += sums[i][threadIdx.x];
      a.part[(static_cast<int64_t>(blockIdx.x) * 2 + side) * D + threadIdx.x] = x;
    }
  }
}

// The workgroups' sums, in their order: 32 rows of threads for 8 channels.
template <int D>
__global__ __launch_bounds__(256) void rope_weights(const RopeArgs a, int parts) {
  __shared__ float sums[32][8];
  const int c = threadIdx.x % 8, row = threadIdx.x / 8;
  const int at = blockIdx.x * 8 + c, side = at / D;
  float *to = a.dw[side];
  if (!to) return;
  float x = 0.0f;
#pragma unroll 8
  for (int i = row; i < parts; i += 32) x += a.part[static_cast<int64_t>(i) * 2 * D + at];
  sums[row][c] = x;
  __syncthreads();
  if (row > 0) return;
  for (int i = 1; i < 32; ++i) x += sums[i][c];
  to[at % D] = x;
}

template <class T, int D, int TOK>
hipError_t run_forward(const RopeArgs &a, int64_t tokens, hipStream_t s) {
  hipLaunchKernelGGL((rope_forward<T, D, TOK>), dim3(static_cast<unsigned>((tokens + TOK - 1) / TOK)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <class T, int D>
hipError_t run_forward(const RopeArgs &a, hipStream_t s) {
  constexpr int kGroups = 256 / (D / 8);
  const int64_t tokens = static_cast<int64_t>(a.b) * a.n, heads = a.heads[0] + a.heads[1];
  // A row a group of lanes up to eight workgroups a CU: 800 tokens of 32 and 8 heads
  // of 128 take 8.1 us, by tokens 9.2; 1600 tokens 12.7 and 10.8; 6400 39 and 27.
  const int64_t few = (tokens * heads + kGroups - 1) / kGroups;
  if (few <= 8 * kCus) {
    hipLaunchKernelGGL((rope_rows<T, D>), dim3(static_cast<unsigned>(few)), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  return rope_tokens(static_cast<int32_t>(heads)) == 16 ? run_forward<T, D, 16>(a, tokens, s) : run_forward<T, D, 4>(a, tokens, s);
}

template <class T, int D>
hipError_t run_backward(const RopeArgs &a, hipStream_t s) {
  const int64_t tiles = (static_cast<int64_t>(a.b) * a.n + kTile - 1) / kTile;
  const int grid = static_cast<int>(tiles < a.grid ? tiles : a.grid);
  if (grid > 0) {
    hipLaunchKernelGGL((rope_backward<T, D>), dim3(grid), dim3(256), 0, s, a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (!a.dw[0] && !a.dw[1]) return hipSuccess;
  hipLaunchKernelGGL((rope_weights<D>), dim3(2 * D / 8), dim3(256), 0, s, a, grid);
  return hipGetLastError();
}

}  // namespace
}  // namespace attn

hipError_t launch_rope(const RopeArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16) return d == 64 ? attn::run_forward<attn::Bf16, 64>(a, s) : attn::run_forward<attn::Bf16, 128>(a, s);
  return d == 64 ? attn::run_forward<attn::F16, 64>(a, s) : attn::run_forward<attn::F16, 128>(a, s);
}
hipError_t launch_rope_backward(const RopeArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16) return d == 64 ? attn::run_backward<attn::Bf16, 64>(a, s) : attn::run_backward<attn::Bf16, 128>(a, s);
  return d == 64 ? attn::run_backward<attn::F16, 64>(a, s) : attn::run_backward<attn::F16, 128>(a, s);
}

}  // namespace sdm
