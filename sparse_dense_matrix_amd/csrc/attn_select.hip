// attn_select.hip -- the choice of key blocks by a cheap score.
//   pool:    a block's keys are summed over its tokens and kept in 8 bits:
//            pooled = round(127 sum / max|sum|), scale = max|sum| / (127 kept)
//   select:  a query block's queries are summed over its tokens and the heads
//            that share the key head, Q, and rounded likewise; block j scores
//            (round(127 Q / max|Q|) . pooled_j) scale_j.  The `blocks` highest
//            stay, ties to the lower block; the first `sink` blocks and the
//            last `local` ones up to the queries' own always do.
//
// Sums run in 64 bits, so that the rounded values do not hang on the order of
// the sum (a 16-bit float's sum is then exact unless its values span more
// than 2^35), and the 8-bit products are whole numbers: the lists are the
// same on any path.  A sum that is not finite gives the values 0; a score
// that is not a number counts as the lowest.
#include <cmath>

#include "attn_dev.h"
#include "internal.h"

namespace sdm {
namespace attn {
namespace {

template <class T>
__device__ __forceinline__ void add8(double *sum, u32x4 v) {
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] += static_cast<double>(elem<T>(v[i / 2], i & 1));
}

// 8 sums as 8-bit values, given the largest of their row
__device__ __forceinline__ u32x2 round8(const double *sum, double top) {
  const bool fine = top > 0.0 && top < INFINITY;
  const double f = fine ? 127.0 / top : 0.0;
  u32x2 r = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int v = fine ? static_cast<int>(rint(sum[i] * f)) : 0;
    r[i / 4] |= static_cast<unsigned>(v & 0xff) << (8 * (i % 4));
  }
  return r;
}

// max that keeps a NaN
__device__ __forceinline__ double top_of(double x, double y) { return y > x || y != y ? y : x; }

// A wave pools one block of one head: 16 bytes a lane, rows over the other
// lanes.  Bound by reading the keys once: 32k tokens of 8 key heads 15.5 us,
// 4.3 TB/s.
template <class T, int D>
__global__ __launch_bounds__(256) void attn_pool(const AttnPoolArgs a) {
  constexpr int kPieces = D / 8, kStep = 64 / kPieces;
  const int lane = threadIdx.x & 63;
  int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = item % a.hk;
  item /= a.hk;
  const int w = item % a.width;
  const int64_t b = item / a.width;
  if (b >= a.b) return;
  const int32_t len = attn_len(a.lens, b, a.nk);
  int32_t first = a.first ? a.first[b] : 0;
  first = first < 0 ? 0 : first;
  const int64_t id = static_cast<int64_t>(first / kAttnPage) + w;
  if (id * kAttnPage >= len) return;
  const int32_t kept = static_cast<int32_t>(min(static_cast<int64_t>(kAttnPage), len - id * kAttnPage));
  int64_t slot;
  const char *p;
  if (a.table) {
    slot = attn_page(a.table + b * a.nkb, static_cast<int32_t>(id), a.pages);
    if (slot < 0) return;
    p = a.k.p + slot * a.k.sb;
  } else {
    slot = b * a.nkb + id;
    p = a.k.p + b * a.k.sb + id * kAttnPage * a.k.st;
  }
  p += h * a.k.sh + (lane % kPieces) * 16;
  double sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  constexpr int kRounds = kAttnPage / kStep;
  u32x4 v[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int r = i * kStep + lane / kPieces;
    v[i] = u32x4{0, 0, 0, 0};
    if (r < kept) v[i] = *reinterpret_cast<const u32x4 *>(p + r * a.k.st);
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i) add8<T>(sum, v[i]);
#pragma unroll
  for (int m = kPieces; m < 64; m *= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor(sum[i], m);
  double top = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = top_of(top, fabs(sum[i]));
#pragma unroll
  for (int m = 1; m < kPieces; m *= 2) top = top_of(top, __shfl_xor(top, m));
  const u32x2 q = round8(sum, top);
  const int64_t at = slot * a.hk + h;
  if (lane < kPieces) *reinterpret_cast<u32x2 *>(a.pooled + at * D + lane * 8) = q;
  if (lane == 0) a.pooled_scale[at] = top == 0.0 ? 0.0f : static_cast<float>(top / (127.0 * kept));
}

// The same from a cache in 8 bits, whose keys are code * scale: a product of 31
// bits, so that its sums in 64 bits are exact as long as the scales of a block
// are within 2^16 of one another.  W waves pool one block of one head, 8 bytes a
// lane; a lane ends with the sums of one or two channels.  Few blocks are bound by
// the latency of their chain, and four waves take each; many by vector instructions
// (each code becomes 32, then 64 bits, and a 64-bit sum: 6 of the 10.7 us that four
// prompts of up to 8k tokens take) and the loads.
template <int D, int W>
__global__ __launch_bounds__(256) void attn_pool8(const AttnPoolArgs a, uint32_t items) {
  constexpr int kLanes = D / 8, kStep = 64 / kLanes, kRows = 64 / W, kRounds = kRows / kStep;
  constexpr int kSteps = D == 128 ? 2 : 3, kKept = 8 >> kSteps;
  const int lane = threadIdx.x & 63;
  const int wave = W > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  uint32_t item = W > 1 ? blockIdx.x : blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (item >= items) return;
  const int h = item % static_cast<uint32_t>(a.hk);
  item /= static_cast<uint32_t>(a.hk);
  const int w = item % static_cast<uint32_t>(a.width);
  const int64_t b = item / static_cast<uint32_t>(a.width);
  const int32_t len = attn_len(a.lens, b, a.nk);
  int32_t first = a.first ? a.first[b] : 0;
  first = first < 0 ? 0 : first;
  const int64_t id = static_cast<int64_t>(first / kAttnPage) + w;
  if (id * kAttnPage >= len) return;
  const int32_t kept = static_cast<int32_t>(min(static_cast<int64_t>(kAttnPage), len - id * kAttnPage));
  int64_t slot;
  const char *p;
  if (a.table) {
    slot = attn_page(a.table + b * a.nkb, static_cast<int32_t>(id), a.pages);
    if (slot < 0) return;
    p = a.k.p + slot * a.k.sb;
  } else {
    slot = b * a.nkb + id;
    p = a.k.p + b * a.k.sb + id * kAttnPage * a.k.st;
  }
  const int64_t at = slot * a.hk + h;
  p += h * a.k.sh + (lane % kLanes) * 8;
  u32x2 v[kRounds];
  float x[kRounds];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int r = wave * kRows + i * kStep + lane / kLanes;
    v[i] = *reinterpret_cast<const u32x2 *>(p + min(r, kept - 1) * a.k.st);
    const float f = a.k_scale[at * kAttnPage + r];  // there for all 64 keys
    x[i] = r < kept ? f : 0.0f;
  }
  double sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const double f = x[i];
#pragma unroll
    for (int c = 0; c < 8; ++c)
      sum[c] = fma(static_cast<double>(static_cast<float>(static_cast<int8_t>(v[i][c / 4] >> (8 * (c % 4))))), f, sum[c]);
  }
  // over the lanes of the same channels: each step adds what the lane 32, 16, ..
  // away has of half the channels
  int channel = (lane % kLanes) * 8;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int m = 32 >> k, n = 4 >> k;  // distance; channels that stay
    const bool upper = lane & m;
    channel += upper ? n : 0;
#pragma unroll
    for (int c = 0; c < n; ++c) {
      const double mine = upper ? sum[c + n] : sum[c], other = upper ? sum[c] : sum[c + n];
      sum[c] = mine + __shfl_xor(other, m);
    }
  }
  if constexpr (W > 1) {
    __shared__ double part[W - 1][kKept][64];
    if (wave > 0)
#pragma unroll
      for (int c = 0; c < kKept; ++c) part[wave - 1][c][lane] = sum[c];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int c = 0; c < kKept; ++c)
#pragma unroll
      for (int i = 0; i < W - 1; ++i) sum[c] += part[i][c][lane];
  }
  double top = 0.0;
#pragma unroll
  for (int c = 0; c < kKept; ++c) top = top_of(top, fabs(sum[c]));
#pragma unroll
  for (int m = 1; m < 64; m *= 2) top = top_of(top, __shfl_xor(top, m));
  const bool fine = top > 0.0 && top < INFINITY;
  const double by = fine ? 127.0 / top : 0.0;
  int8_t *to = a.pooled + at * D + channel;
  unsigned code[kKept];
#pragma unroll
  for (int c = 0; c < kKept; ++c) code[c] = fine ? static_cast<int>(rint(sum[c] * by)) & 0xff : 0;
  if constexpr (kKept == 2)
    *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(code[0] | code[1] << 8);
  else
    *to = static_cast<int8_t>(code[0]);
  if (lane == 0) a.pooled_scale[at] = top == 0.0 ? 0.0f : static_cast<float>(top / (127.0 * kept));
}

// Scores as whole numbers in the same order; what is no number comes lowest.
__device__ __forceinline__ unsigned ordered(float x) {
  if (x != x) return 0;
  const unsigned u = __builtin_bit_cast(unsigned, x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 256;

// One workgroup a list.  The queries' sum is bound by reading them; the
// scores read the pooled keys of the visible blocks from L2.  The threshold
// (the blocks-th highest score) is found bit by bit by one wave with the
// scores in LDS, stopping as soon as the count fits.  32k tokens, 32 heads over
// 8: 60 us, 4.5 TB/s of queries (four rows of a lane in flight; with eight 69 us,
// as fewer lists fit on a CU); one token of 32 sequences 10.5 us, which is the
// chain of its loads and steps.  Loading the first pooled keys before the
// queries' sum takes 0.4 us off that, but costs the prompt 17 us: its registers
// leave half as many lists on a CU.
template <class T, int D>
__global__ __launch_bounds__(kSelThreads) void attn_select(const AttnSelectArgs a) {
  constexpr int kPieces = D / 8, kStep = kSelThreads / kPieces, kWaves = kSelThreads / 64;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  double *part = reinterpret_cast<double *>(lds);             // [waves][D]
  unsigned *q8 = reinterpret_cast<unsigned *>(part + kWaves * D);  // [D / 4]
  unsigned *keys = q8 + D / 4;                                // [nkb]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int64_t item = blockIdx.x;
  const int h = item % a.hk;
  item /= a.hk;
  const int qb = item % a.nqb;
  const int64_t b = item / a.nqb;
  const int32_t len = attn_len(a.lens, b, a.nk);
  const int32_t start = attn_start(a.starts, b, a.nq, a.nk);
  int32_t *out = a.lists + ((b * a.hk + h) * a.nqb + qb) * a.max_blocks;

  // live tokens of the query block: positions 0 .. len - 1
  const int t0 = max(qb * a.q_block, -start);
  const int t1 = min(min(a.nq, (qb + 1) * a.q_block), len - start);
  const int count = t1 > t0 ? (start + t1 - 1) / kAttnPage + 1 : 0;  // visible blocks
  if (count <= a.max_blocks) {  // all of them: no score is asked for
    for (int i = tid; i < a.max_blocks; i += kSelThreads) out[i] = i < count ? i : -1;
    return;
  }
  {
    double sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    const int rows = (t1 - t0) * a.group;
    const char *p = a.q.p + b * a.q.sb + static_cast<int64_t>(h) * a.group * a.q.sh + (tid % kPieces) * 16;
#pragma unroll 4
    for (int r = tid / kPieces; r < rows; r += kStep) {
      const int t = r / a.group;
      add8<T>(sum, *reinterpret_cast<const u32x4 *>(p + (t0 + t) * a.q.st + (r - t * a.group) * a.q.sh));
    }
#pragma unroll
    for (int m = kPieces; m < 64; m *= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += __shfl_xor(sum[i], m);
    if (lane < kPieces)
#pragma unroll
      for (int i = 0; i < 8; ++i) part[wave * D + lane * 8 + i] = sum[i];
    __syncthreads();
    if (tid < kPieces) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        double s = part[tid * 8 + i];
        for (int w = 1; w < kWaves; ++w) s += part[w * D + tid * 8 + i];
        sum[i] = s;
      }
      double top = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = top_of(top, fabs(sum[i]));
#pragma unroll
      for (int m = 1; m < kPieces; m *= 2) top = top_of(top, __shfl_xor(top, m));
      const u32x2 q = round8(sum, top);
      q8[2 * tid] = q[0];
      q8[2 * tid + 1] = q[1];
    }
    __syncthreads();
  }
  // scores: D / 16 lanes a block, 16 bytes each, kBatch blocks of a lane in
  // flight at once (page, then keys and scale)
  constexpr int kLanes = D / 16, kStride = kSelThreads / kLanes, kBatch = 4;
  const i32x4 mine = *reinterpret_cast<const i32x4 *>(q8 + 4 * (tid % kLanes));
  const int32_t *table_row = a.table ? a.table + b * a.nkb : nullptr;
  for (int j0 = 0; j0 < count; j0 += kBatch * kStride) {
    int64_t slot[kBatch];
    i32x4 v[kBatch];
    float scale[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i * kStride + tid / kLanes;
      slot[i] = j < count ? attn_page(table_row, j, a.pages) : -1;
      if (!table_row && slot[i] >= 0) slot[i] += b * a.nkb;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      v[i] = i32x4{0, 0, 0, 0};
      scale[i] = NAN;
      if (slot[i] >= 0) {
        v[i] = *reinterpret_cast<const i32x4 *>(a.pooled + (slot[i] * a.hk + h) * D + 16 * (tid % kLanes));
        scale[i] = a.pooled_scale[slot[i] * a.hk + h];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i * kStride + tid / kLanes;
      int dot = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) dot = __builtin_amdgcn_sdot4(v[i][w], mine[w], dot, false);
#pragma unroll
      for (int m = 1; m < kLanes; m *= 2) dot += __shfl_xor(dot, m);
      if (tid % kLanes == 0 && j < count) {
        // + 0 makes a score of -0 equal to one of 0
        unsigned k = ordered(static_cast<float>(dot) * scale[i] + 0.0f);
        if (j < a.sink || j >= count - a.local) k = 0xffffffffu;
        keys[j] = k;
      }
    }
  }
  __syncthreads();
  if (wave > 0) return;
  // the largest key that at least max_blocks scores reach; the first
  // kHeld * 64 scores in registers, what is past them read again each time
  constexpr int kHeld = 8;
  unsigned held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = i * 64 + lane < count ? keys[i * 64 + lane] : 0;
  auto reach = [&](unsigned want) {  // want > 0
    int n = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) n += __builtin_popcountll(__ballot(held[i] >= want));
    for (int j = kHeld * 64; j < count; j += 64)
      n += __builtin_popcountll(__ballot(j + lane < count && keys[j + lane] >= want));
    return n;
  };
  unsigned cut = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const unsigned want = cut | (1u << bit);
    const int n = reach(want);
    if (n >= a.max_blocks) cut = want;
    if (n == a.max_blocks) break;
  }
  // scores above the cut, and as many at the cut as still fit, lowest first
  const int above = cut == 0xffffffffu ? 0 : reach(cut + 1);
  int room = a.max_blocks - above, at = 0;
  for (int j0 = 0; j0 < count && at < a.max_blocks; j0 += 64) {
    const int j = j0 + lane;
    const unsigned k = j < count ? keys[j] : 0;
    const bool tie = j < count && k == cut;
    const uint64_t ties = __ballot(tie);
    const uint64_t below = (uint64_t(1) << lane) - 1;
    const bool take = j < count && (k > cut || (tie && __builtin_popcountll(ties & below) < room));
    const uint64_t taken = __ballot(take);
    if (take) out[at + __builtin_popcountll(taken & below)] = j;
    at += __builtin_popcountll(taken);
    room -= min(room, static_cast<int>(__builtin_popcountll(ties)));
  }
}

template <class T, int D>
hipError_t run_pool(const AttnPoolArgs &a, hipStream_t s) {
  const int64_t items = static_cast<int64_t>(a.b) * a.width * a.hk;
  if ((items + 3) / 4 > 0x7fffffff) return hipErrorInvalidValue;
  if (items == 0) return hipSuccess;
  if (a.k_scale) {
    if (items > 0x7fffffff) return hipErrorInvalidValue;
    // four waves a block up to two blocks a CU: 256 blocks take 3.9 us, with a wave
    // each 4.7; 512 4.7 both; 1024 6.4 and 4.9; 4096 16.2 and 10.4
    if (items <= 512)
      hipLaunchKernelGGL((attn_pool8<D, 4>), dim3(static_cast<unsigned>(items)), dim3(256), 0, s, a, items);
    else
      hipLaunchKernelGGL((attn_pool8<D, 1>), dim3(static_cast<unsigned>((items + 3) / 4)), dim3(256), 0, s, a, items);
  } else {
    hipLaunchKernelGGL((attn_pool<T, D>), dim3(static_cast<unsigned>((items + 3) / 4)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

template <class T, int D>
hipError_t run_select(const AttnSelectArgs &a, hipStream_t s) {
  const int64_t items = static_cast<int64_t>(a.b) * a.hk * a.nqb;
  if (items > 0x7fffffff) return hipErrorInvalidValue;
  if (items == 0) return hipSuccess;
  const size_t lds = kSelThreads / 64 * D * 8 + D + static_cast<size_t>(a.nkb) * 4;
  if (lds > 64 * 1024) {
    hipError_t e = allow_dynamic_lds(reinterpret_cast<const void *>(&attn_select<T, D>),
                                     kSelThreads / 64 * D * 8 + D + static_cast<size_t>(kAttnMaxScored) * 4);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((attn_select<T, D>), dim3(static_cast<unsigned>(items)), dim3(kSelThreads), lds, s, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace attn

hipError_t launch_attn_pool(const AttnPoolArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16) return d == 64 ? attn::run_pool<attn::Bf16, 64>(a, s) : attn::run_pool<attn::Bf16, 128>(a, s);
  return d == 64 ? attn::run_pool<attn::F16, 64>(a, s) : attn::run_pool<attn::F16, 128>(a, s);
}

hipError_t launch_attn_select(const AttnSelectArgs &a, spmm_dtype_t t, int d, hipStream_t s) {
  if (t == SPMM_BF16)
    return d == 64 ? attn::run_select<attn::Bf16, 64>(a, s) : attn::run_select<attn::Bf16, 128>(a, s);
  return d == 64 ? attn::run_select<attn::F16, 64>(a, s) : attn::run_select<attn::F16, 128>(a, s);
}

}  // namespace sdm
