// What the two matvec kernels share: the packed tile sizes, the arguments and the
// conversion of x.
#pragma once

#include "wd_block.cuh"

namespace wd {

constexpr int kTileRows = 16;   // rows of a packed tile: one MMA row tile
constexpr int kTileCols = 128;  // columns of a packed tile: 4 scale blocks
constexpr int kTileCodes = kTileRows * kTileCols / 2;    // 1024 bytes
constexpr int kTileScales = kTileRows * kTileCols / 32;  // 64 bytes

struct MvArgs {
  const uint8_t *codes, *scales;
  const uint16_t* x;
  void* y;
  int64_t ldx, ldy;
  int32_t B, y_type, N, K;
  int32_t tok0;   // first token of this launch
  int32_t chunk;  // stream kernel: column tiles of x staged at a time; all of them where that fits
  int32_t batch;  // stream kernel: row tiles of a CTA whose sums wait in shared memory
  int32_t per, more;  // row tiles of a CTA (or cluster), and how many have one more
};

// Columns that the tensor-memory kernel takes for `tokens` tokens (wd_fp4_tc.cu), and
// its launch: tokens tok0 .. B-1, in runs of 64 or fewer.
int tc_most_columns(int tokens);
moe_status launch_tc(MvArgs a, bool bf16, cudaStream_t st);

namespace {  // device code: one copy per translation unit

// Four rows of a token's y, rounded to its type.
__device__ __forceinline__ void store_rows(const MvArgs& a, int tok, int64_t row, const float4& v) {
  const int64_t at = (int64_t)tok * a.ldy + row;
  if (row + 4 <= a.N && a.y_type != WD_F32 && at % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7) == 0) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) =
        a.y_type == WD_BF16 ? make_uint2(pack2<true>(v.x, v.y), pack2<true>(v.z, v.w))
                            : make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
    return;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (row + j < a.N) store_elem(a.y, a.y_type, at + j, f[j]);
}

// ---- sums from the packed weights and x themselves, for the few that the kernels' own cannot hold

// The products of one row's block (codes word t of 4 at codes + 16 t) with 32 values of x, times 2^-8 so that
// none overflows.
template <bool BF16>
__device__ __forceinline__ float plain_block(const uint8_t* codes, const uint16_t* x) {
  float d = 0.0f;
#pragma unroll 1
  for (int t = 0; t < 4; ++t) {
    uint32_t h[4];
    e2m1x8_to_f16(__ldg(reinterpret_cast<const uint32_t*>(codes + 16 * t)), h);
    float f[8];
    unpack8<BF16>(ld_cached16(x + 8 * t), f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d = fmaf(half_lo(h[j]), f[2 * j] * 0.00390625f, d);
      d = fmaf(half_hi(h[j]), f[2 * j + 1] * 0.00390625f, d);
    }
  }
  return d;
}

// The sum of one row and token over the blocks of the column tiles [c0, c1), every `step`-th of them, whose
// scale code is at most `top` (NaN blocks are none such; 255: all). In 64 bits between blocks, so only the result
// can leave FP32's range.
template <bool BF16>
__device__ __forceinline__ float plain_sum(const MvArgs& a, int64_t row, int tok, int c0, int c1, int step, int top) {
  const int ct = (a.K + kTileCols - 1) / kTileCols, r = (int)(row % kTileRows);
  const uint16_t* x = a.x + (int64_t)tok * a.ldx;
  double sum = 0.0;
#pragma unroll 1
  for (int c = c0; c < c1; c += step) {
    const size_t tile = (size_t)(row / kTileRows) * ct + c;
    const uint32_t scales = __ldg(reinterpret_cast<const uint32_t*>(a.scales + tile * kTileScales + (r % 8) * 8 + r / 8 * 4));
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
      const int s = (scales >> (8 * b)) & 255, k = c * kTileCols + 32 * b;
      if (s > top || k >= a.K) continue;
      if (s == 255) return NAN;
      const float d = plain_block<BF16>(a.codes + tile * kTileCodes + r * 64 + b * 4, x + k);
      sum += (double)d * __longlong_as_double((long long)(s - 127 + 8 + 1023) << 52);
    }
  }
  return (float)sum;
}

__device__ __forceinline__ bool not_finite(const float4& v) {  // (or so large that their sum is not)
  return !(fabsf(v.x) + fabsf(v.y) + fabsf(v.z) + fabsf(v.w) < INFINITY);
}

// Takes the outputs of rows [row0, row1) and tokens [tok0, tok1) again that are not finite: FP32 may have
// overflowed on the way to a result that fits, or an infinity of x have met a 0 that stands for a small weight.
// All threads of the CTA, whose own outputs they are.
template <bool BF16>
__device__ __forceinline__ void take_again(const MvArgs& a, int64_t row0, int64_t row1, int tok0, int tok1) {
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  for (int tok = tok0; tok < tok1; ++tok) {
    bool nan = false;  // in x: then all of the token's outputs are NaN
    for (int k = threadIdx.x * 2; k < a.K; k += blockDim.x * 2) {
      const uint32_t two = __ldg(reinterpret_cast<const uint32_t*>(a.x + (int64_t)tok * a.ldx + k));
      nan |= (two & 0x7FFFu) > kInf || (two >> 16 & 0x7FFFu) > kInf;
    }
    if (__syncthreads_or(nan)) continue;
#pragma unroll 1
    for (int64_t row = row0 + threadIdx.x; row < row1 && row < a.N; row += blockDim.x) {
      const int64_t at = (int64_t)tok * a.ldy + row;
      const bool fine = a.y_type == WD_F32    ? (__ldcg(static_cast<const uint32_t*>(a.y) + at) & 0x7F800000u) != 0x7F800000u
                        : a.y_type == WD_BF16 ? (__ldcg(static_cast<const uint16_t*>(a.y) + at) & 0x7F80u) != 0x7F80u
                                              : (__ldcg(static_cast<const uint16_t*>(a.y) + at) & 0x7C00u) != 0x7C00u;
      if (!fine) store_elem(a.y, a.y_type, at, plain_sum<BF16>(a, row, tok, 0, (a.K + kTileCols - 1) / kTileCols, 1, 255));
    }
  }
}

// ---- x as f16 times a power of two per token. BF16: the largest finite magnitude
// comes into [2^14, 2^15), so values are exact down to 2^-31 of it and off by at most
// 2^-39 of it below. F16: the same where that scales up, else as it is: always exact.

// The largest finite magnitude, as an integer: 16-bit pairs, plus what takes infinities
// and NaN past the largest signed value, so that they lose against anything.
template <bool BF16>
constexpr uint32_t kPairs0 = BF16 ? 0x00800080u : 0x04000400u;

template <bool BF16>
__device__ __forceinline__ uint32_t largest_pairs(const uint4& v, uint32_t pair) {
  pair = __viaddmax_s16x2(v.x & 0x7FFF7FFFu, kPairs0<BF16>, pair);
  pair = __viaddmax_s16x2(v.y & 0x7FFF7FFFu, kPairs0<BF16>, pair);
  pair = __viaddmax_s16x2(v.z & 0x7FFF7FFFu, kPairs0<BF16>, pair);
  return __viaddmax_s16x2(v.w & 0x7FFF7FFFu, kPairs0<BF16>, pair);
}

template <bool BF16>
__device__ __forceinline__ uint32_t largest_of(uint32_t pair) {
  return max(pair & 0xFFFFu, pair >> 16) - (kPairs0<BF16> & 0xFFFFu);
}

// Of `count` pieces of 8 elements, `step` pieces apart.
template <bool BF16>
__device__ __forceinline__ uint32_t largest_finite16(const uint4* p, int count, int step) {
  uint32_t pair = kPairs0<BF16>;
#pragma unroll 4
  for (int i = 0; i < count; ++i) pair = largest_pairs<BF16>(p[i * step], pair);
  return largest_of<BF16>(pair);
}

// The exponent of the power of two for largest magnitude bits m.
template <bool BF16>
__device__ __forceinline__ int shift_of_16(uint32_t m) {
  const uint32_t mag = BF16 ? m << 16 : __float_as_uint(half_lo(m));
  return mag == 0 ? 0 : min(126, max(BF16 ? -126 : 0, 141 - (int)(mag >> 23)));
}

template <bool BF16>
__device__ __forceinline__ uint4 scaled_f16(const uint4& v, float up) {
  float f[8];
  unpack8<BF16>(v, f);
  return make_uint4(pack2<false>(f[0] * up, f[1] * up), pack2<false>(f[2] * up, f[3] * up),
                    pack2<false>(f[4] * up, f[5] * up), pack2<false>(f[6] * up, f[7] * up));
}

// Pieces of 8 elements times `up`, as f16, in place. Four are read before the first is
// written back: the compiler cannot know that a store hides no later load.
template <bool BF16>
__device__ __forceinline__ void scale_to_f16(uint4* p, int count, int step, float up) {
  constexpr int kAtOnce = 4;
#pragma unroll 1
  for (int i = 0; i < count; i += kAtOnce) {
    uint4 v[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (i + j < count) v[j] = p[(i + j) * step];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (i + j < count) p[(i + j) * step] = scaled_f16<BF16>(v[j], up);
  }
}

}  // namespace

}  // namespace wd
