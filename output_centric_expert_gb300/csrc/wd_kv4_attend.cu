// wd_kv4_attend: attention of one query token per sequence over the paged
// 4-bit cache.
//
// Mathematics. With z_j = scale q.k_j in units of log 2, one pass keeps the
// running maximum m, l = sum 2^(z_j - m) and acc = sum 2^(z_j - m) v_j; partial
// results join as l = sum l_i 2^(m_i - m), acc likewise, out = acc / l.
//   S = K q: mma.sync m16n8k16, rows are 16 keys, columns 8 query heads that
//   share the KV head. E2M1 codes decode exactly to f16; q is f16 times a power of
//   two per head: the largest magnitude in [2^14, 2^15) is exact for BF16 values down
//   to 2^-31 of it; F16 is never scaled down and always exact. A block's 32 products are summed by two MMAs
//   and added to the FP32 logit times the key's E8M0 scale.
//   out = V^T p: rows are dims, k is the keys. A V scale belongs to (key, block):
//   it multiplies the probabilities, as the power of two 2^(s - M + kLift) with M the
//   running maximum of the block's scale codes. A weight p 2^(s - M) is two BF16 terms,
//   the second what the rounding of the first left: 16 bits, and FP32's range of
//   exponents. So it is off by 2^-17 of itself whatever the other keys hold, and the row
//   sum l (of the unrounded p) matches the weights. (f16 weights, one term of 11 bits with
//   5 of exponent, took 27.9 and 50.3 us where these take 31.5 and 61.0, but outputs were
//   off by 2^-12 of their terms, and keys with small p or small scales beside a large one
//   were lost.)
//
// Work. All (sequence, KV head, head tile) rows are cut into tiles of 32 keys per
// warp; CTA c of G takes the c-th contiguous share of all tiles, found from the
// lengths on the device, so ragged batches and single long sequences load the
// SMs evenly and the host needs no lengths. In a tile each warp takes 32 keys by
// itself, streamed through its own cp.async ring, which runs ahead into the CTA's
// next row. The warps' sums join in shared memory. A row that several CTAs share
// leaves their parts in the workspace; a second, dependent launch joins them in CTA
// order. (Joining in the last CTA to finish, by a counter, took 11 us of 42 for 76
// parts of one row: one SM reads them all.)
//
// Bound. 64 sequences of up to 8192 keys with 16 heads per KV head (119 MB): 61.0 us,
// 2.0 TB/s; one of 131071 with 8 heads (71 MB): 31.5 us, 2.3 TB/s. Decoding, scaling and
// the softmax are about 1140 instructions per warp and 32 keys for 16 heads (96 of them
// MMAs), issued in 45 % of the cycles: registers leave 12 to 16 warps per SM, too few to
// hide every dependency. The first 6 us are a chain of trips to memory: lengths, block
// table, keys.
#include "wd_block.cuh"
#include "wd_kv4.cuh"

namespace wd {
namespace {

constexpr int kWarpKeys = 32;  // keys per warp and iteration
constexpr int kSub = 16;       // keys of one MMA tile; a page holds whole ones
constexpr unsigned kAll = 0xFFFFFFFFu;

constexpr float kSlack = 4.0f;  // how far (in log 2) a probability may be above its reference
constexpr int kLift = 122;      // a weight is p 2^(s - M + 122): up to 2^126, which BF16 holds

// What a row costs beside its tiles (queries staged, sums joined), in tiles: CTAs share
// both out. 1, 2, 3: 45.0, 43.6, 44.9 us for 64 sequences up to 4096 with 8 heads, 17.1,
// 16.1, 16.1 for 16 up to 16384 of dim 64; 53.3, 52.0, 52.1 for 64 up to 8192 with 16 heads
// (with weights of one term).
constexpr int kRowUnits = 2;
// Units of a CTA at least, on average, unless it has a row to itself: joining is cheap
// (one sequence of 8192: 13.1 us with 4, 12.4 with 2).
constexpr int kMinUnits = 2;

// The split row that goes on from this CTA into the next, parts 0 where there is none:
// a row with parts in the CTAs c .. c + parts - 1 is in all their entries but the last.
struct __align__(16) Split {
  int32_t parts, index, seq, head;  // index: this CTA's among them; head: the row's first query head
};

struct AttendArgs {
  const uint8_t *kc, *ks, *vc, *vs;
  const uint16_t* q;
  const int32_t *table, *lens;
  uint16_t* out;
  float* lse;
  float* parts;       // [2 * grid][heads of a tile * (D + 2)]
  Split* split;       // [grid]
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
// 16 bytes, and 16 more elsewhere, where `here`; without a branch.
__device__ __forceinline__ void copy16_if(bool here, uint32_t to, const uint8_t* from) {
  asm volatile(
      "{.reg .pred p;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(to),
      "l"(from), "r"((uint32_t)here)
      : "memory");
}
__device__ __forceinline__ void copy16_if(bool here, uint32_t to, const uint8_t* from, uint32_t to2, const uint8_t* from2) {
  asm volatile(
      "{.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "@p cp.async.cg.shared.global [%0], [%1], 16;\n\t"
      "@p cp.async.cg.shared.global [%2], [%3], 16;\n\t}" ::"r"(to),
      "l"(from), "r"(to2), "l"(from2), "r"((uint32_t)here)
      : "memory");
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
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));  // below 2^-126: 0
  return r;
}

__device__ __forceinline__ uint32_t mul2_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// d += a * b with BF16 operands.
__device__ __forceinline__ void mma_add_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight E2M1 codes -> BF16 pairs times 2^-126, e[j] the codes of byte j (low nibble in the low half): E2M1's
// exponent and mantissa are the lowest bits of BF16's exponent and the highest of its mantissa, and its 0.5
// becomes the subnormal 2^-127, which the MMA takes as it is. A selector from 8 on repeats a byte's top bit,
// here the code's sign, which so comes to the half's top.
__device__ __forceinline__ void e2m1x8_to_bf16(uint32_t w, uint32_t (&e)[4]) {
  const uint32_t up = w << 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t two;  // the codes in bits 7 .. 4 of the halves, their signs in 15 .. 8
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(two) : "r"(up), "r"(w), "r"(0xC480 + 0x1111 * j));
    e[j] = two << 2 & 0x81C081C0u;
  }
}

// 1 / l; 0 where no key of the row has a page, whose sums are 0 then.
__device__ __forceinline__ float over(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }

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
  float m[NT][2], l[NT][2];  // reference of K q (before the scale), sum of p
  float acc[NT][D / 16][4];  // rows of MMA tile 2b + h: dims 32b + 4g + 2h (first), + 1
  uint32_t top[D / 64];      // running maximum of the V scale codes, bytes (b, b, b + 1, b + 1) as in v_scales
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
  for (int i = 0; i < D / 64; ++i) s.top[i] = 0;
}

// Bytes of shared memory, 4, 8 or 16 at a time.
template <int WORDS>
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&w)[WORDS]) {
  if constexpr (WORDS == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}

// The scale codes of one key's blocks -> FP32 scales.
template <int NB>
__device__ __forceinline__ void key_scales(const uint8_t* p, float (&f)[NB]) {
  if constexpr (NB == 2) {
    const uint32_t w = *reinterpret_cast<const uint16_t*>(p);
    e8m0x2_to_f32(w & 255u, w >> 8, f[0], f[1]);
  } else {
#pragma unroll
    for (int i = 0; i < NB; i += 4) {
      float four[4];
      e8m0x4_to_f32(*reinterpret_cast<const uint32_t*>(p + i), four);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[i + k] = four[k];
    }
  }
}

// The V scale codes' maxima with a stage's (rare: kept out of the loop's code).
template <int NWORD>
struct Tops {
  uint32_t w[NWORD];
  uint32_t nan;  // bit b: a NaN block b is among the keys
};
template <int D>
__device__ __noinline__ Tops<D / 64> raised_tops(const uint8_t* vs, Tops<D / 64> top) {
  constexpr int NB = D / 32, NWORD = D / 64, kWords = 16 * NWORD;
  const int lane = threadIdx.x & 31;
  uint32_t best[NB] = {}, nan = 0;
#pragma unroll
  for (int r = 0; r < (kWords + 31) / 32; ++r) {
    const int i = lane + 32 * r;
    if (i >= kWords) break;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(vs + i * 4);
    uint32_t both[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t c = (w >> (8 * k)) & 255u;
      if (c == 255u)
        nan |= 1u << (2 * (i % NWORD) + (k >> 1));
      else
        both[k >> 1] = max(both[k >> 1], c);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (i % NWORD == b / 2) best[b] = max(best[b], both[b & 1]);
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint32_t now = max((top.w[b / 2] >> (16 * (b & 1))) & 255u, __reduce_max_sync(kAll, best[b]));
    const uint32_t two = now | now << 8;
    top.w[b / 2] = (b & 1) ? (top.w[b / 2] & 0x0000FFFFu) | two << 16 : (top.w[b / 2] & 0xFFFF0000u) | two;
  }
  top.nan = __reduce_or_sync(kAll, nan);
  return top;
}

// One iteration: 32 keys of a ring stage. qf: the queries' B fragments in shared
// memory, [NT][D / 32][32 lanes][16 bytes]; qs: what turns K q into log 2 units;
// on: bit (u * 16 + k) tells whether key k of run u counts.
template <int D, int NT>
__device__ __forceinline__ void attend_keys(uint8_t* st, const uint8_t* qf, const float (&qs)[NT][2],
                                            uint32_t on, State<D, NT>& s) {
  using L = Stage<D>;
  constexpr int NB = D / 32;     // scale blocks
  constexpr int NWORD = D / 64;  // 4-byte words of a pair's V scales
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (on != kAll) {  // what a masked key's V scales hold must not count
    if (!((on >> lane) & 1u)) {
      uint8_t* p = st + L::kVs + (lane >> 4) * L::kScales;
#pragma unroll
      for (int b = 0; b < NB; ++b) p[v_scale<D>(lane & 15, b)] = 0;
    }
    __syncwarp();
  }

  // ---- K q
  float z[2][NT][4];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* kp = st + L::kK + u * L::kCodes + lane * (D / 8);
    const uint8_t* sp = st + L::kKs + u * L::kScales + g * NB;
    uint32_t wl[NB], wh[NB];
    lds(kp, wl);
    lds(kp + L::kCodes / 2, wh);
    float sl[NB], sh[NB];
    key_scales<NB>(sp, sl);
    key_scales<NB>(sp + 8 * NB, sh);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t al[4], ah[4];
      e2m1x8_to_f16(wl[b], al);
      e2m1x8_to_f16(wh[b], ah);
      const uint32_t a0[4] = {al[0], ah[0], al[1], ah[1]}, a1[4] = {al[2], ah[2], al[3], ah[3]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t q[4];
        lds(qf + ((n * NB + b) * 32 + lane) * 16, q);
        float d[4];
        mma_new(d, a0, q[0], q[1]);
        mma_add(d, a1, q[2], q[3]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float sc = c < 2 ? sl[b] : sh[b];
          z[u][n][c] = b == 0 ? sc * d[c] : fmaf(sc, d[c], z[u][n][c]);
        }
      }
    }
  }
  if (on != kAll) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!((on >> (u * 16 + (c >> 1) * 8 + g)) & 1u)) z[u][n][c] = -INFINITY;
  }

  // ---- reference maximum, probabilities
  // The reference follows the maximum only when that is kSlack above it (in log 2
  // units), so the sums are seldom rescaled; p then stays below 2^4.
  uint32_t p[2][NT][2][2];  // BF16 pairs as the B fragment of out = V^T p; and what their rounding left
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float mx[2];
#pragma unroll
    for (int c = 0; c < 2; ++c)
      mx[c] = fmaxf(fmaxf(z[0][n][c], z[0][n][c + 2]), fmaxf(z[1][n][c], z[1][n][c + 2]));
    // (from -inf to -inf the difference is NaN, which is not above)
    if (__any_sync(kAll, (mx[0] - s.m[n][0]) * qs[n][0] > kSlack || (mx[1] - s.m[n][1]) * qs[n][1] > kSlack)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float to = fmaxf(s.m[n][c], over_g_max(mx[c]));
        // from -inf the sums are 0: any finite factor will do
        const float f = s.m[n][c] == -INFINITY ? 0.0f : exp2_fast((s.m[n][c] - to) * qs[n][c]);
        s.m[n][c] = to;
        s.l[n][c] *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          s.acc[n][i][c] *= f;
          s.acc[n][i][c + 2] *= f;
        }
      }
    }
    // the reference is taken off before the scale: exact near the maximum however large the logits are
    const float base[2] = {s.m[n][0] == -INFINITY ? 0.0f : s.m[n][0], s.m[n][1] == -INFINITY ? 0.0f : s.m[n][1]};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float e[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) e[c] = exp2_fast((z[u][n][c] - base[c & 1]) * qs[n][c & 1]);
      s.l[n][0] += e[0] + e[2];
      s.l[n][1] += e[1] + e[3];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t first = pack2<true>(e[2 * h], e[2 * h + 1]);
        p[u][n][h][0] = transpose8x8(first);
        p[u][n][h][1] = transpose8x8(pack2<true>(e[2 * h] - bf16_lo(first), e[2 * h + 1] - bf16_hi(first)));
      }
    }
  }

  // ---- V scales above the running maximum? (the 16 pairs' words lie together)
  {
    constexpr int kWords = 16 * NWORD;
    bool above = false;
#pragma unroll
    for (int r = 0; r < (kWords + 31) / 32; ++r) {
      const int i = lane + 32 * r;
      if (kWords >= 32 || i < kWords) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(st + L::kVs + i * 4);
        uint32_t have = s.top[0];
#pragma unroll
        for (int k = 1; k < NWORD; ++k)
          if (lane % NWORD == k) have = s.top[k];
        above |= __vmaxu4(w, have) != have;
      }
    }
    if (__any_sync(kAll, above)) {
      Tops<NWORD> top;
#pragma unroll
      for (int k = 0; k < NWORD; ++k) top.w[k] = s.top[k];
      top = raised_tops<D>(st + L::kVs, top);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int have = (s.top[b / 2] >> (16 * (b & 1))) & 255u, now = (top.w[b / 2] >> (16 * (b & 1))) & 255u;
        // a key with a NaN block makes that block's sums NaN, whatever its probability
        const float f = (top.nan >> b) & 1u ? NAN : exp2i(max(-126, have - now)) * exp2i(max(-126, min(0, have - now + 126)));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s.acc[n][2 * b][c] *= f;
            s.acc[n][2 * b + 1][c] *= f;
          }
      }
#pragma unroll
      for (int k = 0; k < NWORD; ++k) s.top[k] = top.w[k];
    }
  }

  // ---- out += V^T p
  uint32_t up[NB];  // the exponent field of 2^(kLift - top) in both halves
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint32_t d = kLift + 127u - ((s.top[b / 2] >> (16 * (b & 1))) & 255u);
    up[b] = __byte_perm(d, d, 0x1010);
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    uint32_t v[2][NB], sc[2][NWORD];  // pairs t and t + 4: k rows 2t, 2t + 1 and 8 more
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lds(st + L::kV + u * L::kCodes + (t + 4 * h) * D + g * (D / 8), v[h]);
      lds(st + L::kVs + u * L::kScales + (t + 4 * h) * (D / 16), sc[h]);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t e[2][4], mult[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        e2m1x8_to_bf16(v[h][b], e[h]);  // e[h][i]: element i of both keys
        const uint32_t two = __byte_perm(sc[h][b / 2], 0, b & 1 ? 0x4342 : 0x4140);  // codes of the two keys
        // 2^(s - top + kLift) as BF16, 0 where that is below its range
        mult[h] = __viaddmax_s16x2_relu(two, up[b], 0u) << 7;
      }
      const uint32_t a0[4] = {e[0][0], e[0][1], e[1][0], e[1][1]}, a1[4] = {e[0][2], e[0][3], e[1][2], e[1][3]};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t p0 = mul2_bf16(p[u][n][0][k], mult[0]), p1 = mul2_bf16(p[u][n][1][k], mult[1]);
          mma_add_bf16(s.acc[n][2 * b], a0, p0, p1);
          mma_add_bf16(s.acc[n][2 * b + 1], a1, p0, p1);
        }
    }
  }
}

// Start copying the 16-key runs run[0], run[1] of the cache (-1: none) into a ring stage. sc: this
// lane's scales of run 0 (lanes below n K's, the next n V's), sc_to their place in a stage.
template <int D>
__device__ __forceinline__ void fetch(uint8_t* st, const AttendArgs& a, const int (&run)[2], const uint8_t* sc,
                                      uint32_t sc_to) {
  using L = Stage<D>;
  constexpr int n = L::kScales / 16;
  const int lane = threadIdx.x & 31;
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(st);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint64_t at = (uint64_t)(uint32_t)run[u] * L::kCodes + lane * 16;
#pragma unroll
    for (int i = 0; i < L::kCodes / 512; ++i) {
      const uint32_t piece = to + u * L::kCodes + 512 * i + lane * 16;
      copy16_if(run[u] >= 0, piece + L::kK, a.kc + at + 512 * i, piece + L::kV, a.vc + at + 512 * i);
    }
    copy16_if(run[u] >= 0 && lane < 2 * n, to + sc_to + u * L::kScales, sc + (uint64_t)(uint32_t)run[u] * L::kScales);
  }
}

// The keys that count for sequence s, and its number of tiles of TILE keys.
template <int TILE>
__device__ __forceinline__ int tiles_of(const AttendArgs& a, int s, uint32_t& lo, uint32_t& hi) {
  const int64_t len = __ldg(a.lens + s), most = (int64_t)a.max_blocks << a.page_shift;
  hi = (uint32_t)(len < 0 ? 0 : len > most ? most : len);
  lo = a.window > 0 && hi > (uint32_t)a.window ? hi - a.window : 0u;
  return (int)((hi - (lo & ~(uint32_t)(kWarpKeys - 1)) + TILE - 1) / TILE);
}

// A segment: the tiles of one row that fall to a CTA.
struct Segment {
  int seq, head, nh, iters;  // head: its first query head
  uint32_t kw, lo, hi;       // the first tile's first key, the keys that count
  int begins, ends;          // whether it has the row's first and last tile
};

template <int D, int NT, int W, int STAGES, int CTAS, bool BF16>
__global__ void __launch_bounds__(W * 32, CTAS) kv4_attend_kernel(const AttendArgs a) {
  using L = Stage<D>;
  constexpr int TILE = W * kWarpKeys, THREADS = W * 32;
  constexpr int NB = D / 32;
  constexpr int NH = NT * 8;           // heads of a tile
  constexpr int kPart = NH * (D + 2);  // floats of a partial result: acc [NH][D], m [NH], l [NH]
  static_assert(8 * D * 4 <= L::kBytes, "a warp's sums of 8 heads fit the stage they came from");
  extern __shared__ uint4 dyn4[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(dyn4);
  __shared__ uint4 s_raw[2][NH * D / 8];  // two segments' queries as they are in memory
  __shared__ uint4 s_q[NT * NB * 32];
  __shared__ float s_qs[NH];
  __shared__ Segment s_seg[W][2];  // every warp keeps its own
  __shared__ int s_scan[W];
  __shared__ int s_base, s_seq;
  __shared__ float s_m[W][NH], s_l[W][NH];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rows = a.heads * a.head_tiles;  // of a sequence

  if (tid == 0) a.split[blockIdx.x].parts = 0;  // until a split row turns out to go on from here
  launch_dependents();
  // ---- this CTA's share of all units: an inclusive scan over the sequences
  uint32_t lo, hi;
  const int chunks = (a.S + THREADS - 1) / THREADS;
  int with_keys = 0;  // sequences
  auto units_of = [&](int s, int& tiles, uint32_t& first, uint32_t& end) {
    tiles = tiles_of<TILE>(a, s, first, end);
    return tiles ? (tiles + kRowUnits) * rows : 0;
  };
  auto scan = [&](int chunk, int before, int& inc, int& mine) {  // returns the units up to the chunk's end
    const int s = chunk * THREADS + tid;
    mine = 0;
    if (s < a.S) {
      int tiles;
      mine = units_of(s, tiles, lo, hi);
      if (blockIdx.x == 0 && (uint32_t)__ldg(a.lens + s) != hi) flag_invalid(a.err);
    }
    inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(kAll, inc, d);
      if (lane >= d) inc += o;
    }
    if (chunks > 1) __syncthreads();  // s_scan may still be read
    if (lane == 31) s_scan[warp] = inc;
    with_keys += __syncthreads_count(mine > 0);
    int end = before;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w == warp) inc += end;
      end += s_scan[w];
    }
    return end;
  };
  int inc, mine, total = 0;
  for (int k = 0; k < chunks; ++k) total = scan(k, total, inc, mine);
  // sequences without keys: their outputs are zeros
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    if (tiles_of<TILE>(a, s, lo, hi) != 0) continue;
    const int heads = a.heads * a.group;
    for (int i = tid; i < heads * D; i += THREADS) a.out[(int64_t)s * a.ldo + i] = 0;
    for (int i = tid; a.lse && i < heads; i += THREADS) a.lse[(int64_t)s * heads + i] = -INFINITY;
  }
  // CTA c of G has units [c q + min(c, r), ...) with total = G q + r
  const int G = min((int)gridDim.x, max(with_keys * rows, total / kMinUnits));
  if ((int)blockIdx.x >= G) return;
  const int gq = total / G, gr = total - G * gq;
  const int begin = (int)blockIdx.x * gq + min((int)blockIdx.x, gr);
  const int end = begin + gq + ((int)blockIdx.x < gr ? 1 : 0);
  for (int k = 0, before = 0; k < chunks; ++k) {
    if (chunks > 1) before = scan(k, before, inc, mine);
    if (begin >= inc - mine && begin < inc) {
      s_seq = k * THREADS + tid;
      s_base = inc - mine;
    }
  }
  __syncthreads();

  // ---- the fetching side: runs up to STAGES - 1 iterations ahead, also into the
  // next segment. All warps go through the same segments and iterations.
  uint8_t* ring = smem + (size_t)warp * STAGES * L::kBytes;
  int f_seq = s_seq, f_base = s_base, f_tiles, f_unit = begin;
  int f_units = units_of(f_seq, f_tiles, lo, hi);  // lo, hi: of f_seq from here on
  int f_segs = 0, f_i = 0, f_iters = 0, f_head = 0, f_stage = 0;
  uint32_t f_key = 0;  // the warp's first key of the segment
  // 16-key runs, counted through the cache ([page][head][run of the page]), -1 without a page:
  // lane l has run (l & 1) of iteration (l >> 1) of 16
  int held = -1;
  uint32_t ok = 0;     // two bits per iteration in flight, the oldest lowest: runs with a page
  int lead = 0;        // iterations in flight
  const int run_shift = a.page_shift - 4;
  constexpr int kScaleLanes = L::kScales / 16;
  const uint8_t* sc_from = lane < kScaleLanes ? a.ks + lane * 16 : a.vs + (lane - kScaleLanes) * 16;
  const uint32_t sc_to = lane < kScaleLanes ? L::kKs + lane * 16 : L::kVs + (lane - kScaleLanes) * 16;
  auto next_segment = [&]() {
    while (f_unit < end) {
      while (f_unit >= f_base + f_units) {
        f_base += f_units;
        f_units = units_of(++f_seq, f_tiles, lo, hi);
      }
      const int per = f_tiles + kRowUnits, row = (f_unit - f_base) / per, row0 = f_base + row * per;
      const int first = max(0, f_unit - row0 - kRowUnits), stop = min(per, end - row0);
      const int last = max(0, stop - kRowUnits);
      f_unit = row0 + stop;
      if (last == first) continue;  // only the row's own units
      const int kv = row / a.head_tiles, h0 = (row - kv * a.head_tiles) * NH, nh = min(NH, a.group - h0);
      f_i = 0, f_iters = last - first, f_head = kv;
      const uint32_t kw = (lo & ~(uint32_t)(kWarpKeys - 1)) + (uint32_t)first * TILE;
      f_key = kw + warp * kWarpKeys;
      const int slot = f_segs & 1;
      if (lane == 0)
        s_seg[warp][slot] = {f_seq, kv * a.group + h0, nh, f_iters, kw, lo, hi, first == 0, last == f_tiles};
      if (tid == 0 && last != f_tiles) {
        auto cta_of = [&](int u) { return u < gr * (gq + 1) ? u / (gq + 1) : gr + (u - gr * (gq + 1)) / gq; };
        const int c0 = first == 0 ? (int)blockIdx.x : cta_of(row0 + kRowUnits), c1 = cta_of(row0 + per - 1);
        a.split[blockIdx.x] = {c1 - c0 + 1, (int)blockIdx.x - c0, f_seq, kv * a.group + h0};
      }
      for (int i = tid; i < NH * D / 8; i += THREADS) {
        const bool real = i / (D / 8) < nh;
        cp_async16(&s_raw[slot][i],
                   a.q + (int64_t)f_seq * a.ldq + (int64_t)(kv * a.group + h0) * D + (real ? i * 8 : 0), real);
      }
      ++f_segs;
      return true;
    }
    return false;
  };
  auto fill = [&](int segs) {  // segs: segments that the computing side has finished
#pragma unroll 1
    while (lead < STAGES - 1) {
      if (f_i == f_iters && (f_segs - segs >= 2 || !next_segment())) break;
      if ((f_i & 15) == 0) {
        const uint32_t key = f_key + (uint32_t)(f_i + (lane >> 1)) * TILE + (lane & 1) * kSub;
        held = -1;
        if (f_i + (lane >> 1) < f_iters && key < hi && key + kSub > lo) {
          const int page = __ldg(a.table + (int64_t)f_seq * a.max_blocks + (key >> a.page_shift));
          if (page < 0 || page >= a.pages)
            flag_invalid(a.err);
          else
            held = ((page * a.heads + f_head) << run_shift) + (int)((key >> 4) & ((1u << run_shift) - 1u));
        }
      }
      int run[2];
      run[0] = __shfl_sync(kAll, held, (f_i & 15) * 2);
      run[1] = __shfl_sync(kAll, held, (f_i & 15) * 2 + 1);
      ok |= ((run[0] >= 0 ? 1u : 0u) | (run[1] >= 0 ? 2u : 0u)) << (2 * lead);
      fetch<D>(ring + f_stage * L::kBytes, a, run, sc_from, sc_to);
      cp_async_commit();
      f_stage = f_stage + 1 == STAGES ? 0 : f_stage + 1;
      ++lead;
      ++f_i;
    }
  };
  auto await = [&]() {  // the oldest iteration in flight
    if (lead == STAGES - 1)
      cp_async_wait<STAGES - 2>();
    else
      cp_async_wait<0>();
    __syncwarp();
  };

  int stage = 0;
#pragma unroll 1
  for (int seg = 0;; ++seg) {
    fill(seg);
    if (lead == 0) break;
    await();
    const Segment& sg = s_seg[warp][seg & 1];
    // ---- queries: f16 times a power of two per head, the scale's sign among it
    __syncthreads();  // every thread's piece of the queries is here, and s_q is free
    for (int n = warp; n < NT; n += W) {
      float m = 0.0f;
      const uint4* raw = s_raw[seg & 1] + (n * 8 + g) * (D / 8) + t;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float f[8];
        unpack8<BF16>(raw[4 * b], f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (fabsf(f[k]) < INFINITY) m = fmaxf(m, fabsf(f[k]));
      }
      m = fmaxf(m, __shfl_xor_sync(kAll, m, 1));
      m = fmaxf(m, __shfl_xor_sync(kAll, m, 2));
      const int sigma = BF16 ? pow2_shift_for(m) : max(0, pow2_shift_for(m));
      const float up = copysignf(exp2i(sigma), a.scale_log2);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float f[8];
        unpack8<BF16>(raw[4 * b], f);
        s_q[(n * NB + b) * 32 + lane] =
            make_uint4(pack2<false>(f[0] * up, f[1] * up), pack2<false>(f[2] * up, f[3] * up),
                       pack2<false>(f[4] * up, f[5] * up), pack2<false>(f[6] * up, f[7] * up));
      }
      const float back = exp2i(-sigma) * fabsf(a.scale_log2);
      if (t == 0) s_qs[n * 8 + g] = back == 0.0f ? 1.17549435e-38f : back;  // masked: -inf times it stays -inf
    }
    __syncthreads();
    float qs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      qs[n][0] = s_qs[n * 8 + 2 * t];
      qs[n][1] = s_qs[n * 8 + 2 * t + 1];
    }
    State<D, NT> st;
    clear(st);

    const int iters = sg.iters;
#pragma unroll 1
    for (int i = 0; i < iters; ++i) {
      if (i > 0) {
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        fill(seg);
        await();
      }
      const uint32_t kb = sg.kw + (uint32_t)i * TILE + warp * kWarpKeys;
      uint32_t on = ((ok & 1u) ? 0x0000FFFFu : 0u) | ((ok & 2u) ? 0xFFFF0000u : 0u);
      ok >>= 2;
      --lead;
      if (on) {
        if (kb < sg.lo) on &= kAll << (sg.lo - kb);  // less than 32: a run counts
        if (kb + kWarpKeys > sg.hi) on &= kAll >> (kb + kWarpKeys - sg.hi);
        attend_keys<D, NT>(ring + stage * L::kBytes, reinterpret_cast<const uint8_t*>(s_q), qs, on, st);
      }
      __syncwarp();
    }

    // ---- join the warps: 8 heads at a time through the stages just used
    const bool whole = sg.begins && sg.ends;
    // a row that goes on in another CTA's share: its first part goes to slot 1, the others to slot 0
    float* part = a.parts + ((size_t)blockIdx.x * 2 + (sg.begins ? 1 : 0)) * kPart;
    uint16_t* orow = a.out + (int64_t)sg.seq * a.ldo + (int64_t)sg.head * D;
    float* lrow = a.lse ? a.lse + (int64_t)sg.seq * a.heads * a.group + sg.head : nullptr;
    // every warp's weights against the CTA's maximum first: then its sums only add
    if (g == 0)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          s_m[warp][n * 8 + 2 * t + c] = st.m[n][c] == -INFINITY ? -INFINITY : st.m[n][c] * qs[n][c];
    __syncthreads();
    auto top_of = [&](int h) {
      float m = s_m[0][h];
#pragma unroll
      for (int w = 1; w < W; ++w) m = fmaxf(m, s_m[w][h]);
      return m;
    };
    auto sum_of = [&](int h) {
      float l = s_l[0][h];
#pragma unroll
      for (int w = 1; w < W; ++w) l += s_l[w][h];
      return l;
    };
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float* mine_sums = reinterpret_cast<float*>(ring + stage * L::kBytes);  // [8][D]
      float f[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = n * 8 + 2 * t + c;
        const float m = top_of(h);
        f[c] = exp2_fast(s_m[warp][h] - (m == -INFINITY ? 0.0f : m));
        const float l = over_g_sum(st.l[n][c]) * f[c];
        if (g == 0) s_l[warp][h] = l;
        f[c] *= exp2i(126 - kLift);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        // the accumulators hold E2M1 times 2^-126 and p times 2^(kLift - top) of the scale
        const float scale = e8m0_to_f32((st.top[b / 2] >> (16 * (b & 1))) & 255u);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float up = scale * f[c];
          *reinterpret_cast<float4*>(mine_sums + (2 * t + c) * D + 32 * b + 4 * g) =
              make_float4(st.acc[n][2 * b][c] * up, st.acc[n][2 * b][2 + c] * up,
                          st.acc[n][2 * b + 1][c] * up, st.acc[n][2 * b + 1][2 + c] * up);
        }
      }
      __syncthreads();
      for (int i = tid * 4; i < 8 * D; i += THREADS * 4) {
        const int h = n * 8 + i / D;
        if (h >= sg.nh) break;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 o = *reinterpret_cast<const float4*>(smem + (size_t)(w * STAGES + stage) * L::kBytes + i * 4);
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        if (whole) {
          const float l = sum_of(h), inv = over(l);
          *reinterpret_cast<uint2*>(orow + n * 8 * D + i) =
              make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
          if (lrow && i % D == 0) {
            const float m = top_of(h);
            lrow[h] = ((m == -INFINITY ? 0.0f : m) + log2f(l)) * 0.6931471805599453f;
          }
        } else {
          *reinterpret_cast<float4*>(part + n * 8 * D + i) = v;
          if (i % D == 0) {
            part[NH * D + h] = top_of(h);
            part[NH * D + NH + h] = sum_of(h);
          }
        }
      }
      __syncthreads();  // the stages are free again
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

// Joins the parts of the rows that several CTAs share. A row with P parts has P - 1
// CTAs here (each attending CTA's entry names at most one row), which share out its
// sums, so a CTA reads about one part's size whatever P is: many rows of two parts and
// one row of many take one wave. A sum of P parts is taken by as many threads as there
// are: 1 for two parts of 2048 sums, 64 for 76 parts of 1024. (A CTA per 256 sums of
// each row, threads sized for many parts: 2432 CTAs in 8 waves for 64 sequences.)
// A dependent launch.
constexpr int kJoin = 256;
template <int D, int NT, bool BF16>
__global__ void __launch_bounds__(kJoin) kv4_join_kernel(const AttendArgs a) {
  constexpr int NH = NT * 8, kPart = NH * (D + 2);
  __shared__ float4 s_v[kJoin];
  __shared__ float s_m[kJoin], s_l[kJoin];
  const int tid = threadIdx.x;
  wait_prerequisite();
  const Split sp = a.split[blockIdx.x];
  if (sp.parts == 0) return;
  const int c0 = (int)blockIdx.x - sp.index, shares = sp.parts - 1;
  const int all = min(NH, a.group - sp.head % a.group) * (D / 4);  // groups of 4 sums of the row
  const int i0 = all * sp.index / shares, i1 = all * (sp.index + 1) / shares;
  if (i0 == i1) return;
  const int log = i1 - i0 >= kJoin ? 8 : 32 - __clz(i1 - i0 - 1);  // threads side by side: 1 << log
  const int side = tid >> log, sides = kJoin >> log;                 // and at one group of sums
  const float* p0 = a.parts + ((size_t)c0 * 2 + 1) * kPart;  // of the first CTA
  const float* p1 = a.parts + (size_t)(c0 + 1) * 2 * kPart;  // of the others, 2 * kPart apart
  auto at = [&](int k) { return k == 0 ? p0 : p1 + (size_t)(k - 1) * 2 * kPart; };
  for (int first = i0; first < i1; first += kJoin) {
    const int i = first + (tid & ((1 << log) - 1)), h = i * 4 / D;
    float m = -INFINITY, l = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto add = [&](float pm, float pl, const float4& o) {
      const float to = fmaxf(m, pm), b = to == -INFINITY ? 0.0f : to;
      const float f = exp2_fast(m - b), g = exp2_fast(pm - b);
      m = to;
      l = fmaf(pl, g, l * f);
      v.x = fmaf(o.x, g, v.x * f);
      v.y = fmaf(o.y, g, v.y * f);
      v.z = fmaf(o.z, g, v.z * f);
      v.w = fmaf(o.w, g, v.w * f);
    };
    if (i < i1) {
      constexpr int kFlight = 4;  // parts in flight per thread
      for (int k0 = side; k0 < sp.parts; k0 += kFlight * sides) {
        float4 o[kFlight];
        float pm[kFlight], pl[kFlight];
#pragma unroll
        for (int k = 0; k < kFlight; ++k)
          if (k0 + k * sides < sp.parts) {
            const float* part = at(k0 + k * sides);
            o[k] = __ldcg(reinterpret_cast<const float4*>(part) + i);
            pm[k] = __ldcg(part + NH * D + h);
            pl[k] = __ldcg(part + NH * D + NH + h);
          }
#pragma unroll
        for (int k = 0; k < kFlight; ++k)
          if (k0 + k * sides < sp.parts) add(pm[k], pl[k], o[k]);
      }
    }
    for (int n = kJoin / 2; n >= 1 << log; n >>= 1) {  // halves: the upper threads' sums to the lower
      if (tid >= n && tid < 2 * n) s_v[tid] = v, s_m[tid] = m, s_l[tid] = l;
      __syncthreads();
      if (tid < n) add(s_m[tid + n], s_l[tid + n], s_v[tid + n]);
    }
    if (side != 0 || i >= i1) continue;
    const float inv = over(l);
    uint16_t* orow = a.out + (int64_t)sp.seq * a.ldo + (int64_t)sp.head * D;
    *reinterpret_cast<uint2*>(orow + i * 4) =
        make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
    if (a.lse && i * 4 % D == 0)
      a.lse[(int64_t)sp.seq * a.heads * a.group + sp.head + h] =
          ((m == -INFINITY ? 0.0f : m) + log2f(l)) * 0.6931471805599453f;
  }
}

// Heads of a tile: 8, or 16 where the group has more and the accumulators fit.
int tile_heads(const wd_kv4_cache* c, int group) { return group > 8 && c->dim < 256 ? 16 : 8; }
int head_tiles(const wd_kv4_cache* c, int group) {
  const int n = tile_heads(c, group);
  return (group + n - 1) / n;
}

constexpr int kCtasPerSm = 2;  // the workspace has room for as many

// Warps of a CTA.
constexpr int warps_of(int dim, bool wide) { return dim == 256 ? 4 : dim == 128 && wide ? 6 : 8; }

// The launch for the capacity of the sequences' rows, which the host knows, whatever their lengths are.
struct Plan {
  int64_t row_tiles;  // tiles of a row at most
  unsigned grid;      // CTAs, no more than tiles; 0: more tiles than the kernel counts
};
Plan plan_of(const wd_kv4_cache* c, int32_t S, int group, int32_t max_blocks, int32_t window) {
  const int64_t keys = (int64_t)max_blocks * c->page_size;
  const int64_t seen = (int64_t)window + 2 * kWarpKeys;  // (in 64 bits: a window may be INT32_MAX)
  const int64_t most = window > 0 && seen < keys ? seen : keys;
  const int tile = warps_of(c->dim, tile_heads(c, group) == 16) * kWarpKeys;
  const int64_t row_tiles = (most + tile - 1) / tile;
  const int64_t rows = (int64_t)S * c->heads * head_tiles(c, group);
  if (rows > 0x7FFFFFFF / (row_tiles + kRowUnits)) return {row_tiles, 0};
  const int64_t tiles = row_tiles * rows, fill = (int64_t)sm_count() * kCtasPerSm;
  return {row_tiles, (unsigned)(tiles < fill ? tiles : fill)};
}

template <int D, int NT, int W, int STAGES, int CTAS>
moe_status launch(const AttendArgs& a, const Plan& plan, bool bf16, cudaStream_t st) {
  static_assert(CTAS == kCtasPerSm && W == warps_of(D, NT == 2), "the plan's");
  auto k = bf16 ? kv4_attend_kernel<D, NT, W, STAGES, CTAS, true> : kv4_attend_kernel<D, NT, W, STAGES, CTAS, false>;
  const size_t ring = (size_t)W * STAGES * Stage<D>::kBytes;
  static SmemOnce once[2];
  moe_status rc = once[bf16].allow(k, ring);
  if (rc != MOE_OK) return rc;
  k<<<plan.grid, W * 32, ring, st>>>(a);
  rc = launched("wd_kv4_attend launch");
  if (rc != MOE_OK || plan.row_tiles == 1) return rc;  // a row of one tile is never split
  cudaLaunchAttribute dependent = {};
  dependent.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  dependent.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.grid);
  cfg.blockDim = dim3(kJoin);
  cfg.stream = st;
  cfg.attrs = &dependent;
  cfg.numAttrs = 1;
  const cudaError_t e =
      bf16 ? cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT, true>, a) : cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT, false>, a);
  if (e != cudaSuccess) {
    set_error("wd_kv4_attend join launch", e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

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
  return grid * sizeof(Split) + grid * 2 * part_floats(c, q_heads / c->heads) * 4;
}

extern "C" int32_t wd_kv4_attend_ctas(const wd_kv4_cache* c, int32_t S, int32_t q_heads, int32_t max_blocks,
                                      int32_t window) {
  using namespace wd;
  if (wd_kv4_attend_workspace(c, S, q_heads) == 0 || max_blocks < 1 || window < 0) return 0;
  return (int32_t)plan_of(c, S, q_heads / c->heads, max_blocks, window).grid;
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
  if ((int64_t)c->pages * c->heads * (c->page_size / kSub) > 0x7FFFFFFF)  // 1 TB of codes
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend: the cache has too many pages");
  const int group = q_heads / c->heads;
  const Plan plan = plan_of(c, S, group, max_blocks, window);
  if (plan.grid == 0) return refuse(MOE_ERR_SHAPE, "wd_kv4_attend: block_table's capacity is too large");
  const unsigned grid = (unsigned)(sm_count() * kCtasPerSm);
  AttendArgs a = {};
  a.kc = c->k_codes, a.ks = c->k_scales, a.vc = c->v_codes, a.vs = c->v_scales;
  a.q = static_cast<const uint16_t*>(q);
  a.table = table, a.lens = lens, a.out = static_cast<uint16_t*>(out), a.lse = lse;
  a.split = static_cast<Split*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + (size_t)grid * sizeof(Split));
  a.err = err, a.ldq = ldq, a.ldo = ldo, a.S = S, a.max_blocks = max_blocks, a.pages = c->pages;
  a.page_shift = kv4_page_shift(c->page_size), a.heads = c->heads, a.group = group;
  a.head_tiles = head_tiles(c, group), a.window = window;
  a.scale_log2 = scale * 1.4426950408889634f;
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf16 = type == WD_BF16, wide = tile_heads(c, group) == 16;
  // <dim, head tiles, warps, ring stages, CTAs per SM>. 16 heads of dim 128 take 168 registers: 2 x 6
  // warps 63.8 us, 1 x 12 warps 67.3 (their barriers hold each other up); a fourth ring stage leaves room
  // for one CTA only, 74 us against 52. Dim 256: 2 x 4 warps 52.8 us, 1 x 8 warps 54.0. (All with
  // weights of one term.)
  if (c->dim == 64) return wide ? launch<64, 2, 8, 4, 2>(a, plan, bf16, st) : launch<64, 1, 8, 4, 2>(a, plan, bf16, st);
  if (c->dim == 128) return wide ? launch<128, 2, 6, 3, 2>(a, plan, bf16, st) : launch<128, 1, 8, 3, 2>(a, plan, bf16, st);
  return launch<256, 1, 4, 2, 2>(a, plan, bf16, st);
}
