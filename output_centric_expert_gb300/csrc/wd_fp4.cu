// Projections with 4-bit weights (MXFP4): the packers and the matrix-vector
// product.
#include "wd_block.cuh"

namespace wd {
namespace {

constexpr int kTileRows = 16;   // rows of a packed tile: one MMA row tile
constexpr int kTileCols = 128;  // columns of a packed tile: 4 scale blocks
constexpr int kTileCodes = kTileRows * kTileCols / 2;    // 1024 bytes
constexpr int kTileScales = kTileRows * kTileCols / 32;  // 64 bytes

__host__ __device__ inline int64_t row_tiles(int N) { return (N + kTileRows - 1) / kTileRows; }
__host__ __device__ inline int col_tiles(int K) { return (K + kTileCols - 1) / kTileCols; }

// ---------------------------------------------------------------- packers --
// One thread per 8 elements (one 4-byte word) of the padded matrix; the four
// threads of a block are neighbours.

struct WordAt {
  int64_t row;
  int k;       // first element
  size_t code, scale;  // byte offsets in the packed arrays
  bool inside;
};

__device__ __forceinline__ WordAt word_at(int64_t i, int N, int K) {
  const int words = col_tiles(K) * (kTileCols / 8);
  WordAt w;
  w.row = i / words;
  w.k = (int)(i - w.row * words) * 8;
  w.inside = w.row < N && w.k < K;
  const size_t tile = (size_t)(w.row / kTileRows) * col_tiles(K) + w.k / kTileCols;
  const int r = (int)(w.row % kTileRows), b = (w.k % kTileCols) / 32, t = (w.k % 32) / 8;
  w.code = tile * kTileCodes + r * 64 + t * 16 + b * 4;
  w.scale = tile * kTileScales + r * 4 + b;
  return w;
}

__global__ void __launch_bounds__(kThreads)
    fp4_pack_codes_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                          uint8_t* __restrict__ pc, uint8_t* __restrict__ ps, int N, int K,
                          int64_t total) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  const WordAt w = word_at(i, N, K);
  uint32_t v = 0, s = 0;
  if (w.inside) {
    const uint8_t* p = codes + ((size_t)w.row * K + w.k) / 2;
    v = p[0] | (uint32_t)p[1] << 8 | (uint32_t)p[2] << 16 | (uint32_t)p[3] << 24;
    s = scales[((size_t)w.row * K + w.k) / 32];
  }
  *reinterpret_cast<uint32_t*>(pc + w.code) = v;
  if (w.k % 32 == 0) ps[w.scale] = (uint8_t)s;
}

__global__ void __launch_bounds__(kThreads)
    fp4_pack_weights_kernel(const void* __restrict__ src, int32_t type, int64_t ldw,
                            uint8_t* __restrict__ pc, uint8_t* __restrict__ ps, int N, int K,
                            int64_t total) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;  // total % 32 == 0: whole warps
  if (i >= total) return;
  const WordAt w = word_at(i, N, K);
  float f[8];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f[j] = w.inside ? load_elem(src, type, w.row * ldw + w.k + j) : 0.0f;
    m = max(m, magnitude(f[j]));
  }
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  const uint32_t s = fp4_scale_code(__uint_as_float(m));
  const float u = fp4_unscale(s);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = s == 255u ? 0.0f : f[j] * u;
  *reinterpret_cast<uint32_t*>(pc + w.code) = e2m1x8(f);
  if (w.k % 32 == 0) ps[w.scale] = (uint8_t)s;
}

// ----------------------------------------------------------------- matvec --
// One CTA per row tile of 16 and per NT * 8 tokens; its 8 warps share the
// columns out tile by tile and add their sums through shared memory.
//   mma.sync m16n8k16, f16 x f16 -> FP32: rows are output rows, columns are
//   tokens. A block's 32 products are summed by two MMAs, times its scale
//   added to the FP32 accumulator.
// x is staged in shared memory as f16 times a power of two per token (the
// largest finite magnitude of the staged columns in [2^14, 2^15)).

constexpr int kStageCols = 4096;  // columns of x staged at a time
constexpr int kStageRow = 2 * kStageCols + 64;  // bytes; 16 banks apart: conflict-free reads

template <int NT, bool BF16>
__global__ void __launch_bounds__(kThreads)
    fp4_matvec_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      const uint16_t* __restrict__ x, int64_t ldx, int B, void* __restrict__ y,
                      int32_t y_type, int64_t ldy, int N, int K) {
  extern __shared__ uint4 dyn4[];
  uint8_t* xs = reinterpret_cast<uint8_t*>(dyn4);
  __shared__ float s_back[NT * 8];
  __shared__ float s_sum[kWarpsPerCta][kTileRows][NT * 8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int64_t tile_row = blockIdx.x;
  const int tok0 = blockIdx.y * NT * 8;
  const int ct = col_tiles(K);
  const uint8_t* crow = codes + (size_t)tile_row * ct * kTileCodes;
  const uint8_t* srow = scales + (size_t)tile_row * ct * kTileScales;

  float total[NT][4] = {};
  for (int c0 = 0; c0 < ct; c0 += kStageCols / kTileCols) {
    const int c1 = min(ct, c0 + kStageCols / kTileCols);
    __syncthreads();
    for (int r = warp; r < NT * 8; r += kWarpsPerCta) {  // a warp stages whole tokens
      const int k0 = c0 * kTileCols, k1 = min(K, c1 * kTileCols), kp = c1 * kTileCols;
      const bool real = tok0 + r < B;
      const uint16_t* row = x + (real ? (int64_t)(tok0 + r) * ldx : 0);
      float m = 0.0f;
      for (int k = k0 + lane * 8; real && k < k1; k += 256) {
        float f[8];
        unpack8<BF16>(ld_cached16(row + k), f);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (fabsf(f[j]) < INFINITY) m = fmaxf(m, fabsf(f[j]));
      }
      m = warp_max(m);
      const int sigma = pow2_shift_for(m);
      const float up = exp2i(sigma);
      for (int k = k0 + lane * 8; k < kp; k += 256) {
        float f[8] = {};
        if (real && k < k1) unpack8<BF16>(ld_cached16(row + k), f);
        uint4 o;
        o.x = pack2<false>(f[0] * up, f[1] * up);
        o.y = pack2<false>(f[2] * up, f[3] * up);
        o.z = pack2<false>(f[4] * up, f[5] * up);
        o.w = pack2<false>(f[6] * up, f[7] * up);
        *reinterpret_cast<uint4*>(xs + (size_t)r * kStageRow + (k - k0) * 2) = o;
      }
      if (lane == 0) s_back[r] = exp2i(-sigma);
    }
    __syncthreads();
    float acc[NT][4] = {};
    for (int c = c0 + warp; c < c1; c += kWarpsPerCta) {
      const uint4 lo = ld_cached16(crow + (size_t)c * kTileCodes + g * 64 + t * 16);
      const uint4 hi = ld_cached16(crow + (size_t)c * kTileCodes + (g + 8) * 64 + t * 16);
      const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
      float sl[4], sh[4];
      e8m0x4_to_f32(__ldg(reinterpret_cast<const uint32_t*>(srow + (size_t)c * kTileScales) + g), sl);
      e8m0x4_to_f32(__ldg(reinterpret_cast<const uint32_t*>(srow + (size_t)c * kTileScales) + g + 8), sh);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t al[4], ah[4];
        e2m1x8_to_f16(wl[b], al);
        e2m1x8_to_f16(wh[b], ah);
        const uint32_t a0[4] = {al[0], ah[0], al[1], ah[1]}, a1[4] = {al[2], ah[2], al[3], ah[3]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = *reinterpret_cast<const uint4*>(
              xs + (size_t)(n * 8 + g) * kStageRow + ((c - c0) * kTileCols + 32 * b + 8 * t) * 2);
          const float zero[4] = {};
          float d[4];
          mma_16816(d, a0, v.x, v.y, zero);
          mma_16816(d, a1, v.z, v.w, d);
          acc[n][0] = fmaf(sl[b], d[0], acc[n][0]);
          acc[n][1] = fmaf(sl[b], d[1], acc[n][1]);
          acc[n][2] = fmaf(sh[b], d[2], acc[n][2]);
          acc[n][3] = fmaf(sh[b], d[3], acc[n][3]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float b0 = s_back[n * 8 + 2 * t], b1 = s_back[n * 8 + 2 * t + 1];
      total[n][0] = fmaf(acc[n][0], b0, total[n][0]);
      total[n][1] = fmaf(acc[n][1], b1, total[n][1]);
      total[n][2] = fmaf(acc[n][2], b0, total[n][2]);
      total[n][3] = fmaf(acc[n][3], b1, total[n][3]);
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    s_sum[warp][g][n * 8 + 2 * t] = total[n][0];
    s_sum[warp][g][n * 8 + 2 * t + 1] = total[n][1];
    s_sum[warp][g + 8][n * 8 + 2 * t] = total[n][2];
    s_sum[warp][g + 8][n * 8 + 2 * t + 1] = total[n][3];
  }
  __syncthreads();
  for (int i = tid; i < kTileRows * NT * 8; i += kThreads) {
    const int r = i % kTileRows, n = i / kTileRows;
    float s = s_sum[0][r][n];
#pragma unroll
    for (int w = 1; w < kWarpsPerCta; ++w) s += s_sum[w][r][n];
    const int64_t row = tile_row * kTileRows + r;
    if (row < N && tok0 + n < B) store_elem(y, y_type, (int64_t)(tok0 + n) * ldy + row, s);
  }
}

moe_status check_fp4(const wd_fp4_shape* s, const uint8_t* pc, const uint8_t* ps) {
  if (!s || !pc || !ps) return refuse(MOE_ERR_NULL, "wd_fp4: shape, codes and scales are required");
  if (s->N < 1 || s->K < 32 || s->K % 32 || s->K > 65536)
    return refuse(MOE_ERR_SHAPE, "wd_fp4: need N >= 1, K % 32 == 0 and 32 <= K <= 65536");
  if (!aligned(pc, 32) || !aligned(ps, 32))
    return refuse(MOE_ERR_ALIGN, "wd_fp4: packed codes and scales need 32 bytes");
  return MOE_OK;
}

int64_t padded_words(const wd_fp4_shape* s) {
  return row_tiles(s->N) * kTileRows * col_tiles(s->K) * (kTileCols / 8);
}

template <int NT, bool BF16>
moe_status launch_matvec(const wd_fp4_shape* s, const uint8_t* pc, const uint8_t* ps,
                         const uint16_t* x, int64_t ldx, int B, void* y, int32_t y_type,
                         int64_t ldy, cudaStream_t st) {
  auto k = fp4_matvec_kernel<NT, BF16>;
  const size_t smem = (size_t)NT * 8 * kStageRow;
  moe_status rc = allow_smem(k, smem);
  if (rc != MOE_OK) return rc;
  const dim3 grid((unsigned)row_tiles(s->N), (unsigned)((B + NT * 8 - 1) / (NT * 8)));
  k<<<grid, kThreads, smem, st>>>(pc, ps, x, ldx, B, y, y_type, ldy, s->N, s->K);
  return launched("wd_fp4_matvec launch");
}

}  // namespace
}  // namespace wd

extern "C" size_t wd_fp4_packed_bytes(const wd_fp4_shape* s, int which) {
  using namespace wd;
  if (!s || s->N < 1 || s->K < 32 || s->K % 32 || s->K > 65536) return 0;
  const size_t tiles = (size_t)row_tiles(s->N) * col_tiles(s->K);
  return which == WD_FP4_CODES ? tiles * kTileCodes : which == WD_FP4_SCALES ? tiles * kTileScales : 0;
}

extern "C" moe_status wd_fp4_pack_codes(const wd_fp4_shape* s, const uint8_t* codes,
                                        const uint8_t* scales, uint8_t* pc, uint8_t* ps,
                                        void* stream) {
  using namespace wd;
  moe_status rc = check_fp4(s, pc, ps);
  if (rc != MOE_OK) return rc;
  if (!codes || !scales) return refuse(MOE_ERR_NULL, "wd_fp4_pack_codes: codes and scales are required");
  const int64_t total = padded_words(s);
  fp4_pack_codes_kernel<<<(unsigned)((total + kThreads - 1) / kThreads), kThreads, 0,
                          (cudaStream_t)stream>>>(codes, scales, pc, ps, s->N, s->K, total);
  return launched("wd_fp4_pack_codes launch");
}

extern "C" moe_status wd_fp4_pack_weights(const wd_fp4_shape* s, const void* w, int32_t w_type,
                                          int64_t ldw, uint8_t* pc, uint8_t* ps, void* stream) {
  using namespace wd;
  moe_status rc = check_fp4(s, pc, ps);
  if (rc != MOE_OK) return rc;
  if (!w) return refuse(MOE_ERR_NULL, "wd_fp4_pack_weights: w is required");
  if (!valid_type(w_type)) return refuse(MOE_ERR_UNSUPPORTED, "wd_fp4_pack_weights: unknown type");
  if (ldw < s->K) return refuse(MOE_ERR_SHAPE, "wd_fp4_pack_weights: ldw is shorter than a row");
  if (!aligned(w, type_bytes(w_type))) return refuse(MOE_ERR_ALIGN, "wd_fp4_pack_weights: w is misaligned");
  const int64_t total = padded_words(s);
  fp4_pack_weights_kernel<<<(unsigned)((total + kThreads - 1) / kThreads), kThreads, 0,
                            (cudaStream_t)stream>>>(w, w_type, ldw, pc, ps, s->N, s->K, total);
  return launched("wd_fp4_pack_weights launch");
}

extern "C" moe_status wd_fp4_matvec(const wd_fp4_shape* s, const uint8_t* pc, const uint8_t* ps,
                                    const void* x, int32_t x_type, int64_t ldx, int32_t B,
                                    void* y, int32_t y_type, int64_t ldy, void* stream) {
  using namespace wd;
  moe_status rc = check_fp4(s, pc, ps);
  if (rc != MOE_OK) return rc;
  if (B < 0) return refuse(MOE_ERR_SHAPE, "wd_fp4_matvec: need B >= 0");
  if (B == 0) return MOE_OK;
  if (!x || !y) return refuse(MOE_ERR_NULL, "wd_fp4_matvec: x and y are required");
  if (!half_type(x_type) || !valid_type(y_type))
    return refuse(MOE_ERR_UNSUPPORTED, "wd_fp4_matvec: x is BF16 or F16, y is F32, BF16 or F16");
  if (ldx < s->K || ldy < s->N || (B + 7) / 8 > 65535)
    return refuse(MOE_ERR_SHAPE, "wd_fp4_matvec: ldx or ldy is shorter than a row, or B is too large");
  if (!aligned(x, 16) || ldx % 8 || !aligned(y, type_bytes(y_type)))
    return refuse(MOE_ERR_ALIGN, "wd_fp4_matvec: x needs 16 bytes and ldx % 8 == 0, y its type's size");
  const uint16_t* x16 = static_cast<const uint16_t*>(x);
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf16 = x_type == WD_BF16;
  if (B <= 8)
    return bf16 ? launch_matvec<1, true>(s, pc, ps, x16, ldx, B, y, y_type, ldy, st)
                : launch_matvec<1, false>(s, pc, ps, x16, ldx, B, y, y_type, ldy, st);
  return bf16 ? launch_matvec<2, true>(s, pc, ps, x16, ldx, B, y, y_type, ldy, st)
              : launch_matvec<2, false>(s, pc, ps, x16, ldx, B, y, y_type, ldy, st);
}
