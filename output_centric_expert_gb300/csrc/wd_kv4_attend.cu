// wd_kv4_attend: attention of one query token per sequence over the paged
// 4-bit cache.
//
// Mathematics. With z_j = scale q.k_j in units of log 2, one pass keeps the
// running maximum m, l = sum 2^(z_j - m) and acc = sum 2^(z_j - m) v_j; partial
// results join as l = sum l_i 2^(m_i - m), acc likewise, out = acc / l.
//   S = K q: mma.sync m16n8k16, rows are 16 keys, columns 8 query heads that
//   share the KV head. E2M1 codes decode exactly to f16; q is f16 times a power of
//   two per head (largest magnitude in [2^14, 2^15), exact for BF16 and F16
//   values down to 2^-32 of it). A block's 32 products are summed by two MMAs
//   and added to the FP32 logit times the key's E8M0 scale.
//   out = V^T p: rows are dims, k is the keys. A V scale belongs to (key, block):
//   it multiplies the probabilities, which are f16 here (11 bits, 2^6 p): the
//   power of two 2^(s - M + 9), with M the running maximum of the block's scale
//   codes, is exact in f16. A key whose scale is below 2^-23 of the block's
//   largest adds nothing (its part is below FP32's own rounding of the sum's
//   largest term).
//
// Work. All (sequence, KV head, head tile) rows are cut into tiles of 256 keys;
// CTA c of G takes the c-th contiguous share of all tiles, found from the
// lengths on the device, so ragged batches and single long sequences load the
// SMs evenly and the host needs no lengths. In a tile each of the 8 warps takes
// 32 keys by itself, streamed through its own cp.async ring. The warps' sums join
// in shared memory. A row that several CTAs share is joined by the last of them
// to finish (a counter per first CTA; the sums are taken in CTA order, so the
// result does not depend on which one it is), without waiting.
#include "wd_block.cuh"
#include "wd_kv4.cuh"

namespace wd {
namespace {

constexpr int kWarpKeys = 32;                          // keys per warp and iteration
constexpr int kTileKeys = kWarpsPerCta * kWarpKeys;  // keys per CTA tile
constexpr int kSub = 16;                               // keys of one MMA tile; a page holds whole ones
constexpr unsigned kAll = 0xFFFFFFFFu;

struct AttendArgs {
  const uint8_t *kc, *ks, *vc, *vs;
  const uint16_t* q;
  const int32_t *table, *lens;
  uint16_t* out;
  float* lse;
  float* parts;       // [2 * grid][heads of a tile * (D + 2)]
  uint32_t* arrived;  // [grid]
  int32_t* err;
  int64_t ldq, ldo;
  int32_t S, max_blocks, pages, page_shift, heads, group, head_tiles, window;
  float scale_log2;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool real) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  const int n = real ? 16 : 0;  // 0: zeros, the source is not read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float over_g_max(float v) {
#pragma unroll
  for (int m = 4; m <= 16; m <<= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, m));
  return v;
}
__device__ __forceinline__ float over_g_sum(float v) {
#pragma unroll
  for (int m = 4; m <= 16; m <<= 1) v += __shfl_xor_sync(kAll, v, m);
  return v;
}

// Sizes of one ring stage: 32 keys of K and V codes and scales, each part the
// image of two 16-key runs of the cache.
template <int D>
struct Stage {
  static constexpr int kCodes = kSub * D / 2, kScales = kSub * D / 32;  // bytes of 16 keys
  static constexpr int kK = 0, kV = 2 * kCodes, kKs = 4 * kCodes, kVs = kKs + 2 * kScales;
  static constexpr int kBytes = kVs + 2 * kScales;
};

// One warp's running state over the keys it has seen, for NT * 8 heads: column c
// of head tile n is head n * 8 + c; a lane holds columns 2t and 2t + 1.
template <int D, int NT>
struct State {
  float m[NT][2], l[NT][2];
  float acc[NT][D / 16][4];  // rows of MMA tile 2b + h: dims 32b + 4g + 2h (first), + 1
  uint32_t top[(D + 127) / 128 * 2];  // running maximum of the V scale codes, byte pairs (b, b) like v_scales
};

template <int D, int NT>
__device__ __forceinline__ void clear(State<D, NT>& s) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    s.m[n][0] = s.m[n][1] = -INFINITY;
    s.l[n][0] = s.l[n][1] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) s.acc[n][i][c] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < (D + 127) / 128 * 2; ++i) s.top[i] = 0;
}

// The keys of an iteration: [kb, kb + 32), of which [lo, hi) count.
struct Keys {
  int64_t kb, lo, hi;
  bool page_ok[2];
};

template <int D, int NT>
__device__ __forceinline__ void attend_keys(uint8_t* st, const uint32_t (&q)[NT][D / 32][4],
                                            const float (&qs)[NT][2], const Keys& keys,
                                            State<D, NT>& s) {
  using L = Stage<D>;
  constexpr int NB = D / 32;          // scale blocks
  constexpr int NWORD = (NB + 1) / 2;  // 4-byte words of a key's V codes; V scale words of a pair
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool edge = keys.kb < keys.lo || keys.kb + kWarpKeys > keys.hi || !keys.page_ok[0] ||
                    !keys.page_ok[1];
  bool off[2][2] = {};  // [16-key run][row g or g + 8]: masked
  if (edge) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int64_t j = keys.kb + u * kSub + r * 8 + g;
        off[u][r] = j < keys.lo || j >= keys.hi || !keys.page_ok[u];
      }
    // what a masked key's V scales hold must not count
    {
      const int64_t j = keys.kb + lane;
      if (j < keys.lo || j >= keys.hi || !keys.page_ok[lane >> 4]) {
        uint8_t* p = st + L::kVs + (lane >> 4) * L::kScales;
#pragma unroll
        for (int b = 0; b < NB; ++b) p[v_scale<D>(lane & 15, b)] = 0;
      }
    }
    __syncwarp();
  }

  // ---- logits
  float z[2][NT][4];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int n = 0; n < NT; ++n) z[u][n][0] = z[u][n][1] = z[u][n][2] = z[u][n][3] = 0.0f;
    const uint8_t* kp = st + L::kK + u * L::kCodes;
    const uint8_t* sp = st + L::kKs + u * L::kScales;
#pragma unroll
    for (int b0 = 0; b0 < NB; b0 += 4) {
      constexpr int W = NB < 4 ? NB : 4;
      uint32_t wl[4], wh[4], scl = 0, sch = 0;
      if constexpr (W == 4) {
        const uint4 a = *reinterpret_cast<const uint4*>(kp + k_word<D>(g, t, b0));
        const uint4 c = *reinterpret_cast<const uint4*>(kp + k_word<D>(g + 8, t, b0));
        wl[0] = a.x, wl[1] = a.y, wl[2] = a.z, wl[3] = a.w;
        wh[0] = c.x, wh[1] = c.y, wh[2] = c.z, wh[3] = c.w;
        scl = *reinterpret_cast<const uint32_t*>(sp + g * NB + b0);
        sch = *reinterpret_cast<const uint32_t*>(sp + (g + 8) * NB + b0);
      } else {
        const uint2 a = *reinterpret_cast<const uint2*>(kp + k_word<D>(g, t, b0));
        const uint2 c = *reinterpret_cast<const uint2*>(kp + k_word<D>(g + 8, t, b0));
        wl[0] = a.x, wl[1] = a.y, wh[0] = c.x, wh[1] = c.y;
        wl[2] = wl[3] = wh[2] = wh[3] = 0;
        scl = *reinterpret_cast<const uint16_t*>(sp + g * NB + b0);
        sch = *reinterpret_cast<const uint16_t*>(sp + (g + 8) * NB + b0);
      }
      float sl[4], sh[4];
      e8m0x4_to_f32(scl, sl);
      e8m0x4_to_f32(sch, sh);
#pragma unroll
      for (int i = 0; i < W; ++i) {
        uint32_t al[4], ah[4];
        e2m1x8_to_f16(wl[i], al);
        e2m1x8_to_f16(wh[i], ah);
        const uint32_t a0[4] = {al[0], ah[0], al[1], ah[1]}, a1[4] = {al[2], ah[2], al[3], ah[3]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float zero[4] = {};
          float d[4];
          mma_16816(d, a0, q[n][b0 + i][0], q[n][b0 + i][1], zero);
          mma_16816(d, a1, q[n][b0 + i][2], q[n][b0 + i][3], d);
          z[u][n][0] = fmaf(sl[i], d[0], z[u][n][0]);
          z[u][n][1] = fmaf(sl[i], d[1], z[u][n][1]);
          z[u][n][2] = fmaf(sh[i], d[2], z[u][n][2]);
          z[u][n][3] = fmaf(sh[i], d[3], z[u][n][3]);
        }
      }
    }
  }

  // ---- running maximum, probabilities (times 2^6)
  uint32_t p[2][NT][2];  // f16x2 as the B fragment of out = V^T p
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float mx[2] = {s.m[n][0], s.m[n][1]};
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float v = z[u][n][c] * qs[n][c & 1];
        if (edge && off[u][c >> 1]) v = -INFINITY;
        z[u][n][c] = v;
        mx[c & 1] = fmaxf(mx[c & 1], v);
      }
    mx[0] = over_g_max(mx[0]);
    mx[1] = over_g_max(mx[1]);
    const float b0 = mx[0] == -INFINITY ? 0.0f : mx[0], b1 = mx[1] == -INFINITY ? 0.0f : mx[1];
    if (__any_sync(kAll, mx[0] > s.m[n][0] || mx[1] > s.m[n][1])) {
      const float f0 = exp2_fast(s.m[n][0] - b0), f1 = exp2_fast(s.m[n][1] - b1);
      s.l[n][0] *= f0;
      s.l[n][1] *= f1;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        s.acc[n][i][0] *= f0;
        s.acc[n][i][1] *= f1;
        s.acc[n][i][2] *= f0;
        s.acc[n][i][3] *= f1;
      }
      s.m[n][0] = mx[0];
      s.m[n][1] = mx[1];
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const float e0 = exp2_fast(z[u][n][0] - b0 + 6.0f), e1 = exp2_fast(z[u][n][1] - b1 + 6.0f);
      const float e2 = exp2_fast(z[u][n][2] - b0 + 6.0f), e3 = exp2_fast(z[u][n][3] - b1 + 6.0f);
      s.l[n][0] += e0 + e2;
      s.l[n][1] += e1 + e3;
      p[u][n][0] = transpose8x8(pack2<false>(e0, e1));
      p[u][n][1] = transpose8x8(pack2<false>(e2, e3));
    }
  }

  // ---- running maximum of the V scales: a warp's 16 pairs x NWORD words
  bool poison = false;  // a NaN block among the keys
  {
    constexpr int kWords = 16 * NWORD;  // of both runs, contiguous
    bool above = false;
#pragma unroll
    for (int i = lane, r = 0; r < (kWords + 31) / 32; i += 32, ++r) {
      if (i < kWords) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(st + L::kVs + i * 4);
        const uint32_t have = NWORD == 1 ? s.top[0]
                              : NWORD == 2 ? ((i & 1) ? s.top[1] : s.top[0])
                                           : ((i & 3) == 0   ? s.top[0]
                                              : (i & 3) == 1 ? s.top[1]
                                              : (i & 3) == 2 ? s.top[2]
                                                             : s.top[3]);
        above |= __vmaxu4(w, have) != have;
      }
    }
    if (__any_sync(kAll, above)) {
      uint32_t best[NB] = {};
#pragma unroll
      for (int i = lane, r = 0; r < (kWords + 31) / 32; i += 32, ++r) {
        if (i < kWords) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(st + L::kVs + i * 4);
          const uint32_t c[4] = {w & 255u, (w >> 8) & 255u, (w >> 16) & 255u, w >> 24};
          uint32_t lo = 0, hi = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (c[k] == 255u)
              poison = true;
            else if (k < 2)
              lo = max(lo, c[k]);
            else
              hi = max(hi, c[k]);
          }
#pragma unroll
          for (int b = 0; b < NB; b += 2)
            if (i % NWORD == b / 2) {
              best[b] = max(best[b], lo);
              best[b + 1] = max(best[b + 1], hi);
            }
        }
      }
      poison = __any_sync(kAll, poison);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t have = (s.top[b / 2] >> (16 * (b & 1))) & 255u;
        const uint32_t now = max(have, __reduce_max_sync(kAll, best[b]));
        if (now > have) {
          const float f = exp2i(max(-126, (int)have - (int)now));
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              s.acc[n][2 * b][c] *= f;
              s.acc[n][2 * b + 1][c] *= f;
            }
          const uint32_t two = now | now << 8;
          s.top[b / 2] = (b & 1) ? (s.top[b / 2] & 0x0000FFFFu) | two << 16
                                 : (s.top[b / 2] & 0xFFFF0000u) | two;
        }
      }
    }
  }

  // ---- out += V^T p
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* vp = st + L::kV + u * L::kCodes;
    const uint8_t* sp = st + L::kVs + u * L::kScales;
#pragma unroll
    for (int j = 0; j < NWORD; ++j) {
      uint32_t even[2][4], odd[2][4], mult[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // pairs t and t + 4: k rows 2t, 2t + 1 and 8 more
        const uint8_t* row = vp + (t + 4 * h) * D + g * (D / 8) + j * 4;
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(row);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(row + D / 16);
        e2m1x8_to_f16((w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u), even[h]);
        e2m1x8_to_f16(((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u), odd[h]);
        const uint32_t sc = *reinterpret_cast<const uint32_t*>(sp + (t + 4 * h) * (D / 16) + j * 4);
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // block 2j + k
          const uint32_t two = __byte_perm(sc, 0, k ? 0x4342 : 0x4140);  // codes of the two keys
          const int bias = 24 - (int)((s.top[j] >> (16 * k)) & 255u);
          const uint32_t add = ((uint32_t)bias & 0xFFFFu) | (uint32_t)bias << 16;
          uint32_t e = __viaddmax_s16x2_relu(two, add, 0u) << 10;
          if (poison) {
            if ((two & 0xFFFFu) == 255u) e = (e & 0xFFFF0000u) | 0x7E00u;
            if ((two >> 16) == 255u) e = (e & 0x0000FFFFu) | 0x7E000000u;
          }
          mult[h][k] = e;
        }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t a0[4] = {even[0][2 * k], odd[0][2 * k], even[1][2 * k], odd[1][2 * k]};
        const uint32_t a1[4] = {even[0][2 * k + 1], odd[0][2 * k + 1], even[1][2 * k + 1],
                                odd[1][2 * k + 1]};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t p0 = hmul2(p[u][n][0], mult[0][k]), p1 = hmul2(p[u][n][1], mult[1][k]);
          mma_16816(s.acc[n][2 * (2 * j + k)], a0, p0, p1, s.acc[n][2 * (2 * j + k)]);
          mma_16816(s.acc[n][2 * (2 * j + k) + 1], a1, p0, p1, s.acc[n][2 * (2 * j + k) + 1]);
        }
      }
    }
  }
}

// Start copying the 32 keys from kb of (sequence, head) into a ring stage.
template <int D>
__device__ __forceinline__ void fetch(uint8_t* st, const AttendArgs& a, int head, int64_t kb,
                                      const int (&page)[2]) {
  using L = Stage<D>;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const bool real = page[u] >= 0;
    const int64_t key = kb + u * kSub;
    const size_t at = ((((size_t)(real ? page[u] : 0) * a.heads) + head) << a.page_shift) +
                      (size_t)(real ? (key & ((1 << a.page_shift) - 1)) : 0);
#pragma unroll
    for (int i = 0; i < L::kCodes / 512; ++i) {
      const int o = (lane + 32 * i) * 16;
      cp_async16(st + L::kK + u * L::kCodes + o, a.kc + at * (D / 2) + o, real);
      cp_async16(st + L::kV + u * L::kCodes + o, a.vc + at * (D / 2) + o, real);
    }
    if (lane < L::kScales / 16)
      cp_async16(st + L::kKs + u * L::kScales + lane * 16, a.ks + at * (D / 32) + lane * 16, real);
    else if (lane >= 16 && lane < 16 + L::kScales / 16)
      cp_async16(st + L::kVs + u * L::kScales + (lane - 16) * 16,
                 a.vs + at * (D / 32) + (lane - 16) * 16, real);
  }
}

// The pages of the two 16-key runs from kb (-1: outside the counted keys or invalid).
__device__ __forceinline__ void pages_of(const AttendArgs& a, int seq, int64_t kb, int64_t lo,
                                         int64_t hi, int (&page)[2]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t key = kb + u * kSub;
    page[u] = -1;
    if (key < hi && key + kSub > lo) {
      const int id = __ldg(a.table + (int64_t)seq * a.max_blocks + (key >> a.page_shift));
      if (id >= 0 && id < a.pages)
        page[u] = id;
      else
        flag_invalid(a.err);
    }
  }
}

// The keys that count for sequence s and its number of tiles.
__device__ __forceinline__ int tiles_of(const AttendArgs& a, int s, int64_t& lo, int64_t& hi) {
  const int64_t len = __ldg(a.lens + s), most = (int64_t)a.max_blocks << a.page_shift;
  hi = len < 0 ? 0 : len > most ? most : len;
  lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
  return (int)((hi - (lo & ~(int64_t)(kSub - 1)) + kTileKeys - 1) / kTileKeys);
}

template <int D, int NT, int STAGES, bool BF16>
__global__ void __launch_bounds__(kThreads)
    kv4_attend_kernel(const AttendArgs a) {
  using L = Stage<D>;
  constexpr int NH = NT * 8;              // heads of a tile
  constexpr int kPart = NH * (D + 2);     // floats of a partial result: acc [NH][D], m [NH], l [NH]
  extern __shared__ uint4 dyn4[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(dyn4);
  __shared__ int64_t s_scan[kWarpsPerCta];
  __shared__ int64_t s_total, s_base;
  __shared__ int s_seq;
  __shared__ float s_m[kWarpsPerCta][NH], s_l[kWarpsPerCta][NH], s_w[kWarpsPerCta][NH];
  __shared__ float s_sum[NH], s_max[NH];
  __shared__ bool s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rows = a.heads * a.head_tiles;  // of a sequence
  int64_t lo, hi;

  // ---- this CTA's share of all tiles
  {
    int64_t sum = 0;
    for (int s = tid; s < a.S; s += kThreads) {
      const int n = tiles_of(a, s, lo, hi);
      if (blockIdx.x == 0 && (__ldg(a.lens + s) < 0 ||
                              __ldg(a.lens + s) > ((int64_t)a.max_blocks << a.page_shift)))
        flag_invalid(a.err);
      sum += (int64_t)n * rows;
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(kAll, sum, m);
    if (lane == 0) s_scan[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      int64_t all = 0;
      for (int w = 0; w < kWarpsPerCta; ++w) all += s_scan[w];
      s_total = all;
    }
    __syncthreads();
  }
  const int64_t total = s_total;
  const int64_t G = total < gridDim.x ? total : gridDim.x;
  // sequences without keys: their outputs are zeros
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    if (tiles_of(a, s, lo, hi) != 0) continue;
    const int heads = a.heads * a.group;
    for (int i = tid; i < heads * D; i += kThreads) a.out[(int64_t)s * a.ldo + i] = 0;
    for (int i = tid; a.lse && i < heads; i += kThreads) a.lse[(int64_t)s * heads + i] = -INFINITY;
  }
  if ((int64_t)blockIdx.x >= G) return;
  const int64_t begin = total * blockIdx.x / G, end = total * (blockIdx.x + 1) / G;
  {
    int64_t base = 0;
    for (int s0 = 0; s0 < a.S; s0 += kThreads) {
      const int s = s0 + tid;
      const int64_t mine = s < a.S ? (int64_t)tiles_of(a, s, lo, hi) * rows : 0;
      int64_t inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(kAll, inc, d);
        if (lane >= d) inc += o;
      }
      __syncthreads();
      if (lane == 31) s_scan[warp] = inc;
      __syncthreads();
      int64_t before = base, chunk = 0;
      for (int w = 0; w < kWarpsPerCta; ++w) {
        if (w < warp) before += s_scan[w];
        chunk += s_scan[w];
      }
      const int64_t start = before + inc - mine;
      if (begin >= start && begin < start + mine) {
        s_seq = s;
        s_base = start;
      }
      base += chunk;
      if (base > begin) break;
    }
    __syncthreads();
  }
  int seq = s_seq;
  int64_t base = s_base;
  int n_tiles = tiles_of(a, seq, lo, hi);
  uint8_t* ring = smem + (size_t)warp * STAGES * L::kBytes;

  for (int64_t pos = begin; pos < end;) {
    while (pos >= base + (int64_t)n_tiles * rows) {
      base += (int64_t)n_tiles * rows;
      n_tiles = tiles_of(a, ++seq, lo, hi);
    }
    const int row = (int)((pos - base) / n_tiles), first = (int)((pos - base) - (int64_t)row * n_tiles);
    const int last = (int)min((int64_t)n_tiles, first + (end - pos));  // tiles [first, last) of the row
    const int head = row / a.head_tiles, h0 = (row % a.head_tiles) * NH;
    const int nh = min(NH, a.group - h0);  // real heads of the tile
    const int64_t k0 = lo & ~(int64_t)(kSub - 1);

    // ---- queries: f16 times a power of two per head
    uint32_t q[NT][D / 32][4];
    float qs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const bool real = n * 8 + g < nh;
      const uint16_t* qp = a.q + (int64_t)seq * a.ldq + ((int64_t)head * a.group + h0 + (real ? n * 8 + g : 0)) * D;
      float m = 0.0f;
      uint4 raw[D / 32];
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        raw[b] = real ? ld_cached16(qp + 32 * b + 8 * t) : make_uint4(0, 0, 0, 0);
        float f[8];
        unpack8<BF16>(raw[b], f);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (fabsf(f[j]) < INFINITY) m = fmaxf(m, fabsf(f[j]));
      }
      m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
      m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
      const int sigma = pow2_shift_for(m);
      const float up = exp2i(sigma), back = exp2i(-sigma) * a.scale_log2;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        float f[8];
        unpack8<BF16>(raw[b], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[n][b][j] = pack2<false>(f[2 * j] * up, f[2 * j + 1] * up);
      }
      qs[n][0] = __shfl_sync(kAll, back, 8 * t);  // head 2t: lane g = 2t
      qs[n][1] = __shfl_sync(kAll, back, 8 * t + 4);
    }

    // ---- the warp's keys of tiles [first, last)
    State<D, NT> st;
    clear(st);
    const int iters = last - first;
    const int64_t kw = k0 + (int64_t)first * kTileKeys + warp * kWarpKeys;  // of iteration 0
    int page[STAGES][2];  // pages of the stages in flight
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      page[i][0] = page[i][1] = -1;
      if (i < iters) {
        pages_of(a, seq, kw + (int64_t)i * kTileKeys, lo, hi, page[i]);
        fetch<D>(ring + i * L::kBytes, a, head, kw + (int64_t)i * kTileKeys, page[i]);
      }
      cp_async_commit();
    }
    int next[2] = {-1, -1};  // pages of the next stage to fetch
    if (STAGES - 1 < iters) pages_of(a, seq, kw + (int64_t)(STAGES - 1) * kTileKeys, lo, hi, next);
    for (int i0 = 0; i0 < iters; i0 += STAGES) {
#pragma unroll
      for (int k = 0; k < STAGES; ++k) {
        const int i = i0 + k;
        if (i >= iters) break;
        cp_async_wait<STAGES - 2>();
        __syncwarp();
        constexpr int kAhead = STAGES - 1;
        const int into = (k + kAhead) % STAGES;
        page[into][0] = next[0];
        page[into][1] = next[1];
        if (i + kAhead < iters)
          fetch<D>(ring + into * L::kBytes, a, head, kw + (int64_t)(i + kAhead) * kTileKeys, next);
        cp_async_commit();
        next[0] = next[1] = -1;
        if (i + STAGES < iters) pages_of(a, seq, kw + (int64_t)(i + STAGES) * kTileKeys, lo, hi, next);
        const Keys keys = {kw + (int64_t)i * kTileKeys, lo, hi, {page[k][0] >= 0, page[k][1] >= 0}};
        if (keys.kb < hi && keys.kb + kWarpKeys > lo) attend_keys<D, NT>(ring + k * L::kBytes, q, qs, keys, st);
        __syncwarp();
      }
    }
    cp_async_wait<0>();

    // ---- join the warps
    __syncthreads();  // every ring is idle: its memory holds the sums now
    float* sums = reinterpret_cast<float*>(smem);  // [warp][NH][D]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float l0 = over_g_sum(st.l[n][0]), l1 = over_g_sum(st.l[n][1]);
      if (g == 0) {
        s_m[warp][n * 8 + 2 * t] = st.m[n][0];
        s_m[warp][n * 8 + 2 * t + 1] = st.m[n][1];
        s_l[warp][n * 8 + 2 * t] = l0;
        s_l[warp][n * 8 + 2 * t + 1] = l1;
      }
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        // the accumulators hold 2^6 p times 2^(9 - top) of the scale
        const float f = e8m0_to_f32((st.top[b / 2] >> (16 * (b & 1))) & 255u) * 0.001953125f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
          *reinterpret_cast<float4*>(sums + (size_t)(warp * NH + n * 8 + 2 * t + c) * D + 32 * b + 4 * g) =
              make_float4(st.acc[n][2 * b][c] * f, st.acc[n][2 * b][2 + c] * f,
                          st.acc[n][2 * b + 1][c] * f, st.acc[n][2 * b + 1][2 + c] * f);
      }
    }
    __syncthreads();
    if (tid < NH) {
      float m = s_m[0][tid];
#pragma unroll
      for (int w = 1; w < kWarpsPerCta; ++w) m = fmaxf(m, s_m[w][tid]);
      const float b = m == -INFINITY ? 0.0f : m;
      float l = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarpsPerCta; ++w) {
        const float f = exp2_fast(s_m[w][tid] - b);
        s_w[w][tid] = f;
        l = fmaf(s_l[w][tid], f, l);
      }
      s_max[tid] = m;
      s_sum[tid] = l;
    }
    __syncthreads();
    const bool whole = first == 0 && last == n_tiles;
    const int64_t row0 = base + (int64_t)row * n_tiles;
    const int64_t c0 = whole ? 0 : ((row0 + 1) * G - 1) / total;
    float* part = a.parts + ((size_t)blockIdx.x * 2 + ((int64_t)blockIdx.x == c0 ? 1 : 0)) * kPart;
    const int heads = a.heads * a.group;
    uint16_t* orow = a.out + (int64_t)seq * a.ldo + ((int64_t)head * a.group + h0) * D;
    float* lrow = a.lse ? a.lse + (int64_t)seq * heads + head * a.group + h0 : nullptr;
    for (int i = tid * 2; i < nh * D; i += kThreads * 2) {
      const int h = i / D;
      float v0 = 0.0f, v1 = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarpsPerCta; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(sums + (size_t)w * NH * D + i);
        v0 = fmaf(v.x, s_w[w][h], v0);
        v1 = fmaf(v.y, s_w[w][h], v1);
      }
      if (whole)
        *reinterpret_cast<uint32_t*>(orow + i) = pack2<BF16>(v0 / s_sum[h], v1 / s_sum[h]);
      else
        *reinterpret_cast<float2*>(part + i) = make_float2(v0, v1);
    }
    if (tid < nh) {
      if (whole) {
        if (lrow) lrow[tid] = (s_max[tid] + log2f(s_sum[tid]) - 6.0f) * 0.6931471805599453f;
      } else {
        part[NH * D + tid] = s_max[tid];
        part[NH * D + NH + tid] = s_sum[tid];
      }
    }
    if (!whole) {
      // ---- the last CTA of the row joins its parts, in CTA order
      const int64_t c1 = ((row0 + n_tiles) * G - 1) / total;
      const int parts = (int)(c1 - c0) + 1;
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(a.arrived + c0, 1u) == (uint32_t)parts - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        if (tid == 0) a.arrived[c0] = 0;
        const float* p0 = a.parts + ((size_t)c0 * 2 + 1) * kPart;        // of the first CTA
        const float* p1 = a.parts + (size_t)(c0 + 1) * 2 * kPart;        // of the others, 2 * kPart apart
        auto at = [&](int i) { return i == 0 ? p0 : p1 + (size_t)(i - 1) * 2 * kPart; };
        if (tid < nh) {
          float m = -INFINITY, l = 0.0f;
          for (int i = 0; i < parts; ++i) m = fmaxf(m, __ldcg(at(i) + NH * D + tid));
          const float b = m == -INFINITY ? 0.0f : m;
          for (int i = 0; i < parts; ++i)
            l = fmaf(__ldcg(at(i) + NH * D + NH + tid), exp2_fast(__ldcg(at(i) + NH * D + tid) - b), l);
          s_max[tid] = b;
          s_sum[tid] = l;
          if (lrow) lrow[tid] = (b + log2f(l) - 6.0f) * 0.6931471805599453f;
        }
        __syncthreads();
        for (int i = tid * 4; i < nh * D; i += kThreads * 4) {
          const int h = i / D;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
          for (int k = 0; k < parts; ++k) {
            const float f = exp2_fast(__ldcg(at(k) + NH * D + h) - s_max[h]);
            const float4 o = __ldcg(reinterpret_cast<const float4*>(at(k) + i));
            v.x = fmaf(o.x, f, v.x);
            v.y = fmaf(o.y, f, v.y);
            v.z = fmaf(o.z, f, v.z);
            v.w = fmaf(o.w, f, v.w);
          }
          const float inv = 1.0f / s_sum[h];
          uint2 o;
          o.x = pack2<BF16>(v.x * inv, v.y * inv);
          o.y = pack2<BF16>(v.z * inv, v.w * inv);
          *reinterpret_cast<uint2*>(orow + i) = o;
        }
      }
    }
    __syncthreads();  // the sums and the ring share their memory
    pos += last - first;
  }
}

// Heads of a tile: 8, or 16 where the group has more and the accumulators fit.
int tile_heads(const wd_kv4_cache* c, int group) { return group > 8 && c->dim < 256 ? 16 : 8; }
int head_tiles(const wd_kv4_cache* c, int group) {
  const int n = tile_heads(c, group);
  return (group + n - 1) / n;
}

template <int D, int NT, int STAGES, bool BF16>
moe_status launch(const AttendArgs& a, unsigned grid, cudaStream_t st) {
  auto k = kv4_attend_kernel<D, NT, STAGES, BF16>;
  const size_t ring = (size_t)kWarpsPerCta * STAGES * Stage<D>::kBytes;
  const size_t sums = (size_t)kWarpsPerCta * NT * 8 * D * 4;
  const size_t smem = ring > sums ? ring : sums;
  moe_status rc = allow_smem(k, smem);
  if (rc != MOE_OK) return rc;
  k<<<grid, kThreads, smem, st>>>(a);
  return launched("wd_kv4_attend launch");
}

constexpr int kCtasPerSm = 1;

size_t part_floats(const wd_kv4_cache* c, int group) {
  return (size_t)tile_heads(c, group) * (c->dim + 2);
}

}  // namespace
}  // namespace wd

extern "C" size_t wd_kv4_attend_workspace(const wd_kv4_cache* c, int32_t S, int32_t q_heads) {
  using namespace wd;
  if (!c || wd_kv4_cache_bytes(c, WD_KV4_CODES) == 0 || S < 0 || q_heads < 1 || q_heads % c->heads)
    return 0;
  const size_t grid = (size_t)sm_count() * kCtasPerSm;
  return (grid * 4 + 15) / 16 * 16 + grid * 2 * part_floats(c, q_heads / c->heads) * 4;
}

extern "C" moe_status wd_kv4_attend(const wd_kv4_cache* c, const void* q, int32_t type,
                                    int64_t ldq, int32_t S, int32_t q_heads,
                                    const int32_t* table, int32_t max_blocks,
                                    const int32_t* lens, float scale, int32_t window, void* out,
                                    int64_t ldo, float* lse, void* workspace,
                                    size_t workspace_bytes, int32_t* err, void* stream) {
  using namespace wd;
  moe_status rc = check_kv4(c);
  if (rc != MOE_OK) return rc;
  if (S < 0 || q_heads < 1 || q_heads % c->heads || max_blocks < 1 || window < 0)
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend: need S >= 0, q_heads a multiple of heads, max_blocks >= 1, window >= 0");
  if (!half_type(type)) return refuse(MOE_ERR_UNSUPPORTED, "wd_kv4_attend: q and out are BF16 or F16");
  if (ldq < (int64_t)q_heads * c->dim || ldo < (int64_t)q_heads * c->dim)
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend: ldq or ldo is shorter than a token");
  if (S == 0) return MOE_OK;
  if (!q || !table || !lens || !out || !workspace)
    return refuse(MOE_ERR_NULL, "wd_kv4_attend: q, block_table, seq_lens, out and workspace are required");
  if (!aligned(q, 16) || ldq % 8 || !aligned(out, 16) || ldo % 8 || !aligned(table, 4) ||
      !aligned(lens, 4) || !aligned(lse, 4) || !aligned(workspace, 16) || !aligned(err, 4))
    return refuse(MOE_ERR_ALIGN, "wd_kv4_attend: q, out and workspace need 16 bytes, strides % 8 == 0, the others 4");
  if (workspace_bytes < wd_kv4_attend_workspace(c, S, q_heads))
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend: workspace is smaller than wd_kv4_attend_workspace");
  const int group = q_heads / c->heads;
  const unsigned grid = (unsigned)(sm_count() * kCtasPerSm);
  AttendArgs a = {};
  a.kc = c->k_codes, a.ks = c->k_scales, a.vc = c->v_codes, a.vs = c->v_scales;
  a.q = static_cast<const uint16_t*>(q);
  a.table = table, a.lens = lens, a.out = static_cast<uint16_t*>(out), a.lse = lse;
  a.arrived = static_cast<uint32_t*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ((size_t)grid * 4 + 15) / 16 * 16);
  a.err = err, a.ldq = ldq, a.ldo = ldo, a.S = S, a.max_blocks = max_blocks, a.pages = c->pages;
  a.page_shift = kv4_page_shift(c->page_size), a.heads = c->heads, a.group = group;
  a.head_tiles = head_tiles(c, group), a.window = window;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf16 = type == WD_BF16, wide = tile_heads(c, group) == 16;
  if (c->dim == 64) {
    if (wide) return bf16 ? launch<64, 2, 4, true>(a, grid, st) : launch<64, 2, 4, false>(a, grid, st);
    return bf16 ? launch<64, 1, 4, true>(a, grid, st) : launch<64, 1, 4, false>(a, grid, st);
  }
  if (c->dim == 128) {
    if (wide) return bf16 ? launch<128, 2, 4, true>(a, grid, st) : launch<128, 2, 4, false>(a, grid, st);
    return bf16 ? launch<128, 1, 4, true>(a, grid, st) : launch<128, 1, 4, false>(a, grid, st);
  }
  return bf16 ? launch<256, 1, 3, true>(a, grid, st) : launch<256, 1, 3, false>(a, grid, st);
}
