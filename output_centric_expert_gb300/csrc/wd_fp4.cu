// Projections with 4-bit weights (MXFP4): the packers and the matrix-vector
// product.
#include "wd_fp4.h"

#include "wd_block.cuh"

namespace wd {
namespace {

__host__ __device__ inline int64_t row_tiles(int N) { return (N - 1) / kTileRows + 1; }  // (N + 15 may pass 2^31)
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
  w.scale = tile * kTileScales + (r % 8) * 8 + (r / 8) * 4 + b;
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
// A CTA of 16 warps per SM takes a contiguous run of row tiles; their (row tile,
// column tile) pairs, which lie one after another in memory, are shared out evenly
// among its warps, so each warp streams one dense run of codes through registers.
//   mma.sync m16n8k16, f16 x f16 -> FP32: rows are output rows, columns are
//   tokens. A block's 32 products are summed by two MMAs, times its scale
//   added to the FP32 accumulator. x times 2^14 and more beside weights past 2^96 can
//   overflow it where the result does not: a sum that is not finite is taken again
//   from x itself.
// x is staged once per CTA in shared memory, as f16 times a power of two per
// token and in the order of the B
// fragment: [column tile][block][lane][16 bytes]. Row tiles that warps share are
// joined in shared memory in column order, so results do not depend on timing.
//   Bound by the codes' bytes where the matrix is large: 8 tokens of 129283 x 2048
// (145 MB) take 29.2 us, 5.0 TB/s, 73 % of a copy. 16 warps and 4 column tiles ahead of
// each: 12, 20 and 24 warps took 6, 4 and 13 % longer, 3 and 5 column tiles 1 and 2 %.
// Small products are latency: one token of 4096 x 2048 4.7 us, of which 2.5 are the
// launch and 1 is the trip for x.

constexpr int kMvWarps = 16, kMvThreads = kMvWarps * 32;
constexpr int kMvTokens = 8;  // of a launch: the columns of an MMA
constexpr int kAhead = 4;  // column tiles in flight per warp
constexpr size_t kStaticSmem = 512;  // more than the kernel's static shared memory

// Stage `toks` tokens' columns [128 c0, 128 c1) (zero from K on) as f16 fragments;
// s_max[n] becomes the bits of the token's largest finite magnitude (16 bits). Copied
// as they are to their places, then converted there by the thread that copied them;
// its pieces are all of one token. Short loops instead of unrolled registers: a
// small product spends its time fetching code. All threads of the CTA; ends behind a
// barrier.
template <bool BF16>
__device__ __forceinline__ void stage_x(const MvArgs& a, int c0, int c1, int toks, uint4* xs, uint32_t* s_max) {
  const int k0 = c0 * kTileCols, quads = (c1 - c0) * 4;  // blocks of 32 columns: 4 pieces of 8
  const int real = (min(a.K, c1 * kTileCols) - k0) / 8;
  const int share = toks > 4 ? 3 : toks > 2 ? 2 : toks > 1 ? 1 : 0;  // 1 << share tokens, the last may be zero
  const int q = threadIdx.x & 3, tok = (threadIdx.x >> 2) & ((1 << share) - 1);
  const int first = threadIdx.x >> (2 + share), step = kMvThreads >> (2 + share);
  const uint16_t* x = a.x + (int64_t)(a.tok0 + (tok < toks ? tok : 0)) * a.ldx + k0 + q * 8;
  uint4* own = xs + first * 32 + tok * 4 + q;  // and 32 * step units on
  for (int b = first; b < quads; b += step) {
    const int bytes = tok < toks && b * 4 + q < real ? 16 : 0;  // 0: zeros, the source is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(xs + b * 32 + tok * 4 + q)),
                 "l"(x + (bytes ? b * 32 : 0)), "r"(bytes)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (threadIdx.x < 8) s_max[threadIdx.x] = 0;
  __syncthreads();
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  const int mine = (quads - first + step - 1) / step;
  uint32_t m = largest_finite16<BF16>(own, mine, 32 * step);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  for (int o = 16; o >= 4 << share; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) < 4u << share && q == 0) atomicMax(s_max + tok, m);
  __syncthreads();
  scale_to_f16<BF16>(own, mine, 32 * step, exp2i(shift_of_16<BF16>(s_max[tok])));
  __syncthreads();
}

// kChunked: x is staged a.chunk column tiles at a time, the sums of a batch of row tiles
// wait in shared memory. Else all of x is staged once and a warp's run is one dense
// stretch of memory; its row tiles' sums wait too (kWait), or a row tile that the run has
// all of is written as it ends (kDirect: more code for each, and no burst of writes behind
// the loads).
enum Mode { kWait, kDirect, kChunked };
template <bool BF16, Mode MODE>
__global__ void __launch_bounds__(kMvThreads, 1) fp4_matvec_kernel(const MvArgs a) {
  constexpr bool CHUNKED = MODE == kChunked;
  extern __shared__ uint4 dyn4[];
  __shared__ uint32_t s_max[kMvTokens];
  constexpr int kSums = kTileRows * kMvTokens;  // of a row tile: [token][row]
  // parts of row tiles that warps share: [warp][0: begun before, 1: begun here]
  float(*s_part)[2][kSums] = reinterpret_cast<float(*)[2][kSums]>(dyn4);
  float(*s_sum)[kSums] = reinterpret_cast<float(*)[kSums]>(dyn4 + kMvWarps * 2 * kSums / 4);  // [batch]
  float(*s_held)[kSums] = s_sum + a.batch;  // CHUNKED: sums of the chunks before
  uint4* xs = dyn4 + (kMvWarps * 2 + a.batch * (CHUNKED ? 2 : 1)) * (kSums / 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int toks = min(kMvTokens, a.B - a.tok0);
  const int b0 = blockIdx.x;  // row tiles [r0, r1)
  const int r0 = b0 * a.per + min(b0, a.more), r1 = r0 + a.per + (b0 < a.more ? 1 : 0);
  const int ct = col_tiles(a.K);

  struct Tile {
    uint4 lo, hi;
    uint2 sc;
  };
  bool staged = false, again = false;  // again: an output is not finite
  for (int q0 = r0; q0 < r1; q0 += a.batch) {
    const int nq = min(a.batch, r1 - q0);
    for (int c0 = 0; c0 < ct; c0 += CHUNKED ? a.chunk : ct) {
      const int kt = CHUNKED ? min(a.chunk, ct - c0) : ct, units = nq * kt;
      const int u0 = units * warp / kMvWarps, u1 = units * (warp + 1) / kMvWarps;
      const int t0 = u0 / kt;
      int k = u0 - t0 * kt;  // column tile at hand
      const size_t at = (size_t)(q0 + t0) * ct + c0 + k;
      const uint8_t* lc = a.codes + at * kTileCodes + lane * 16;  // of the next tile to load
      const uint8_t* ls = a.scales + at * kTileScales + g * 8;
      int left = CHUNKED ? kt - k : 0;  // column tiles up to the chunk's end
      Tile buf[kAhead];
      auto load = [&](Tile& b) {
        b.lo = ld_codes16(lc);
        b.hi = ld_codes16(lc + 512);
        b.sc = ld_scales8(ls);
        lc += kTileCodes;
        ls += kTileScales;
        if (CHUNKED && --left == 0) {
          left = kt;
          lc += (size_t)(ct - kt) * kTileCodes;
          ls += (size_t)(ct - kt) * kTileScales;
        }
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (u0 + i < u1) load(buf[i]);
      if (!staged) stage_x<BF16>(a, c0, c0 + kt, toks, xs, s_max);
      staged = !CHUNKED;

      float acc[4] = {};
      const uint4* xk = xs + (size_t)k * 4 * 32 + lane;
      // where the sums of the tile at hand go: a slot if it began in another warp's run
      const int sum_at = 2 * t * kTileRows + g;
      float* whole = s_sum[t0] + sum_at;
      float* to = k == 0 ? whole : s_part[warp][0] + sum_at;
      auto finish = [&](float* p) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          p[(c & 1) * kTileRows + 8 * (c >> 1)] = acc[c];
          acc[c] = 0.0f;
        }
      };
      int q = q0 + t0;  // kDirect: the row tile at hand, and what tokens 2t and 2t + 1 are multiplied by
      float back[2];
      if (MODE == kDirect)
#pragma unroll
        for (int c = 0; c < 2; ++c) back[c] = exp2i(-shift_of_16<BF16>(s_max[2 * t + c]));
      auto write = [&]() {  // 32 bytes of a token and more from 8 lanes
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int64_t row = (int64_t)q * kTileRows + g + 8 * (c >> 1);
          const int tok = 2 * t + (c & 1);
          const float v = acc[c] * back[c & 1];
          if (tok < toks && row < a.N) {
            store_elem(a.y, a.y_type, (int64_t)(a.tok0 + tok) * a.ldy + row, v);
            again |= !(fabsf(v) < INFINITY);
          }
          acc[c] = 0.0f;
        }
      };
      auto use = [&](const Tile& b) {
        const uint32_t wl[4] = {b.lo.x, b.lo.y, b.lo.z, b.lo.w}, wh[4] = {b.hi.x, b.hi.y, b.hi.z, b.hi.w};
        float sl[4], sh[4];
        e8m0x4_to_f32(b.sc.x, sl);
        e8m0x4_to_f32(b.sc.y, sh);
#pragma unroll
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t al[4], ah[4];
          e2m1x8_to_f16(wl[blk], al);
          e2m1x8_to_f16(wh[blk], ah);
          const uint32_t a0[4] = {al[0], ah[0], al[1], ah[1]}, a1[4] = {al[2], ah[2], al[3], ah[3]};
          // columns without a token hold whatever is there: they reach no other column
          const uint4 v = xk[blk * 32];
          float d[4];
          mma_new(d, a0, v.x, v.y);
          mma_add(d, a1, v.z, v.w);
          acc[0] = fmaf(sl[blk], d[0], acc[0]);
          acc[1] = fmaf(sl[blk], d[1], acc[1]);
          acc[2] = fmaf(sh[blk], d[2], acc[2]);
          acc[3] = fmaf(sh[blk], d[3], acc[3]);
        }
        xk += 4 * 32;
        if (++k == kt) {
          if (MODE == kDirect && to == whole)
            write();
          else
            finish(to);
          ++q;
          k = 0;
          xk = xs + lane;
          whole += kSums;
          to = whole;
        }
      };
      int u = u0;
      for (; u + 2 * kAhead <= u1; u += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          use(buf[i]);
          load(buf[i]);
        }
      }
#pragma unroll 1
      for (; u < u1; u += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          if (u + i < u1) use(buf[i]);
          if (u + i + kAhead < u1) load(buf[i]);
        }
      }
      if (k > 0 && u0 < u1) finish(to == whole ? s_part[warp][1] + sum_at : to);
      __syncthreads();
      const bool last = !CHUNKED || c0 + kt >= ct;
      const int starts = lane < kMvWarps ? units * lane / kMvWarps : 0x7FFFFFFF;  // of the warps' runs
      for (int q = warp; q < nq; q += kMvWarps) {  // a warp per row tile
        // the warps that have its first and last column tile; a lane has 4 rows of a token
        const int w0 = __popc(__ballot_sync(0xFFFFFFFFu, starts <= q * kt)) - 1;
        const int w1 = __popc(__ballot_sync(0xFFFFFFFFu, starts < (q + 1) * kt)) - 1;
        if (MODE == kDirect && w0 == w1) continue;
        const int o = lane * 4, tok = o / kTileRows;
        float4 v = *reinterpret_cast<const float4*>(w0 == w1 ? s_sum[q] + o : s_part[w0][1] + o);
        for (int w = w0 + 1; w <= w1; ++w) {
          if (units * w / kMvWarps == units * (w + 1) / kMvWarps) continue;  // an empty run
          const float4 p = *reinterpret_cast<const float4*>(s_part[w][0] + o);
          v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
        }
        const float back = exp2i(-shift_of_16<BF16>(s_max[tok]));
        v.x *= back, v.y *= back, v.z *= back, v.w *= back;
        if (CHUNKED) {
          float4* held = reinterpret_cast<float4*>(s_held[q] + o);
          if (c0 > 0) v.x += held->x, v.y += held->y, v.z += held->z, v.w += held->w;
          if (!last) *held = v;
        }
        if (last && tok < toks) {
          store_rows(a, a.tok0 + tok, (int64_t)(q0 + q) * kTileRows + o % kTileRows, v);
          again |= not_finite(v);
        }
      }
      __syncthreads();  // the sums, and x where it comes in chunks, are written again
    }
  }
  if (__syncthreads_or(again))
    take_again<BF16>(a, (int64_t)r0 * kTileRows, (int64_t)r1 * kTileRows, a.tok0, a.tok0 + toks);
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

template <bool BF16>
moe_status launch_matvec(MvArgs a, cudaStream_t st) {
  static SmemOnce once[3];
  Mode mode = kWait;
  constexpr size_t kTileX = (size_t)4 * 32 * 16;  // x of a column tile
  constexpr size_t kTileSum = (size_t)kTileRows * kMvTokens * 4;
  constexpr size_t kRoom = kMaxDynSmem - kStaticSmem - kMvWarps * 2 * kTileSum;
  const int ct = col_tiles(a.K);
  const int64_t tiles = row_tiles(a.N);
  const int sms = sm_count();
  const unsigned grid = (unsigned)(tiles < sms ? tiles : sms);
  a.per = (int)(tiles / grid);
  a.more = (int)(tiles - (int64_t)a.per * grid);
  const int64_t per = (tiles + grid - 1) / grid;
  size_t smem;
  if (ct * kTileX + 8 * kTileSum <= kRoom) {  // all of x, and the sums of as many row tiles as fit
    const int64_t fit = (int64_t)((kRoom - ct * kTileX) / kTileSum);
    a.chunk = ct;
    a.batch = (int)(per < fit ? per : fit);
    // us for 8 tokens: 129283 x 2048 (54 row tiles a CTA) 28.9 written as they end, 30.5 waiting;
    // 65536 x 4096 (27) 30.0 and 30.7; 9216 x 4096 (4) 10.5 and 10.4; 2048 x 2048 (1) 5.9 and 5.6 (when both were measured)
    if (per >= kMvWarps) mode = kDirect;
    smem = ct * kTileX + a.batch * kTileSum;
  } else {  // columns in chunks of 128 KB of x
    mode = kChunked;
    a.chunk = 64;
    a.batch = (int)(per < 32 ? per : 32);
    smem = a.chunk * kTileX + 2 * a.batch * kTileSum;
  }
  smem += kMvWarps * 2 * kTileSum;
  auto k = mode == kWait ? fp4_matvec_kernel<BF16, kWait> : mode == kDirect ? fp4_matvec_kernel<BF16, kDirect>
                                                                            : fp4_matvec_kernel<BF16, kChunked>;
  moe_status rc = once[mode].allow(k, kMaxDynSmem - kStaticSmem);
  if (rc != MOE_OK) return rc;
  for (int64_t tok = 0; tok < a.B; tok += kMvTokens) {
    a.tok0 = (int)tok;
    k<<<grid, kMvThreads, smem, st>>>(a);
    if ((rc = launched("wd_fp4_matvec launch")) != MOE_OK) return rc;
  }
  return MOE_OK;
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
  if (ldx < s->K || ldy < s->N)
    return refuse(MOE_ERR_SHAPE, "wd_fp4_matvec: ldx or ldy is shorter than a row");
  if (!aligned(x, 16) || ldx % 8 || !aligned(y, type_bytes(y_type)))
    return refuse(MOE_ERR_ALIGN, "wd_fp4_matvec: x needs 16 bytes and ldx % 8 == 0, y its type's size");
  const MvArgs a = {pc, ps, static_cast<const uint16_t*>(x), y, ldx, ldy, B, y_type, s->N, s->K, 0, 0, 0};
  cudaStream_t st = (cudaStream_t)stream;
  // Up to 8 tokens (and where rows are too long for the other kernel's shared memory) the stream kernel:
  // it reads the weights once per 8 tokens. us for 8 and 9 tokens: 10.3 and 18.0 against 11.9 and 10.8 for
  // 9216 x 4096, 5.4 and 9.7 against 7.3 and 6.9 for 2048 x 2048, 30 and 59 against 50 and 42 for 65536 x 4096
  // (when the other kernel had no test for quiet blocks, 1 to 5 % of it).
  if (B > 8 && s->K <= tc_most_columns(B)) return launch_tc(a, x_type == WD_BF16, st);
  return x_type == WD_BF16 ? launch_matvec<true>(a, st) : launch_matvec<false>(a, st);
}
