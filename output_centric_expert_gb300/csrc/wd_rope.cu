// Rotary positions: wd_rope turns the heads of a tensor, wd_kv4_rope_append turns the
// queries and keys of new tokens and puts keys and values into the 4-bit cache.
//
// Mathematics. Pair i of a head is turned by the angle pos * f_i. A frequency is kept as
// turns per position in units of 2^-64, so the product with a position in 64-bit
// integers is the angle less its whole turns, exactly: no position is too far. What is
// left after the nearest quarter turn, at most an eighth either way, becomes FP32 (off by 1.3 * 2^-24 at
// most: conversion, product with 2 pi, its rounding) and goes through the Taylor series of sine and cosine.
//
// What the cache holds is the nearest MXFP4 to the exact turned key. FP32 gives it to
// within kDoubt of the largest input of a piece of eight elements and of their partners: codes are
// taken at both ends of that interval, and where they differ (in one block of 2000) the element is computed
// again in 64 bits. So the codes do not depend on the order of FP32 operations. A turn by nothing is exact and leaves
// no doubt: its results are the inputs, which in BF16 often lie on a border, as do elements that do not turn. So the
// doubt is a piece's own, not its block's: 10056 tokens with heads of 128, 80 of them turned and the rest zeros, 58 us for
// 245; heads of 64 with 16 turned 30 for 59.
//
// Work. A CTA has a run of tokens and some of their heads. It computes the angles' sines
// and cosines once for all its heads into shared memory (planes of 16 bytes, so that
// neighbouring pieces are neighbouring words).
//
// Measured (GB300). wd_rope, 7001 tokens with 20 heads of 256 in FP16, a quarter turned: 22.4 us
// for 143 MB in a graph on one set of inputs, which L2 holds in part; 24.4 in one wave of CTAs that wait for their
// tables before they read, 31 with two items of a thread in flight, in 63 registers. A few
// tokens: 2.1 us, a launch. wd_kv4_rope_append, 10056 tokens with 32 query and 8 KV heads of
// 128: 53 us for 216 MB; 64 tokens with 64 and 4: 4.6 us. The first is bound by the
// instructions that a key takes (30 us with no queries, issue slots 63 % busy) and by the
// queries' memory traffic, which overlap only in part. Left to the compiler the kernel took 83
// registers, two CTAs of an SM, and 82 us; at 64 and four of them, with 72 bytes of a thread spilled and 100 to 108 read back, 59, and 56 with two items
// of a thread's queries in flight. Three items, five CTAs (62), halves of the queries' slices
// (62): slower. Runs short enough for three waves, with what a CTA reads asked into L2
// while it finds its tokens' places: 54; for one wave 60.
#include <algorithm>
#include <cmath>

#include "wd_kv4_tokens.cuh"

namespace wd {
namespace {

constexpr float kDoubt = 9.5367431640625e-7f;  // 2^-20: 12 of FP32's 2^-24 and some more (test_rope_gpu derives them)

// cos and sin of pos * turns / 2^64 turns.
__device__ __forceinline__ float2 cos_sin(uint64_t turns, int64_t pos) {
  const uint64_t a = turns * (uint64_t)pos;
  const uint32_t quarter = (uint32_t)((a + (1ull << 61)) >> 62);
  const int64_t rest = (int64_t)(a - ((uint64_t)quarter << 62));  // within 2^61
  const float x = (float)(int32_t)(rest >> 32) * 1.46291807926715968e-9f;  // 2 pi / 2^32
  const float y = x * x;
  float s = fmaf(x * y, fmaf(y, fmaf(y, fmaf(y, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), x);
  if (x == 0.0f && rest != 0) s = 1.17549435e-38f;  // so that 0 says that the angle is whole quarter turns
  const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
  const float u = quarter & 1 ? s : c, v = quarter & 1 ? c : s;
  return make_float2((quarter + 1) & 2 ? -u : u, quarter & 2 ? -v : v);
}

// The table of a CTA's tokens, [token][4 planes][rot / 16 groups] of 16 bytes: planes 0, 1 hold the cosines of a group of
// eight pairs, 2, 3 the sines. Positions of -1 are left out. All threads, a barrier behind it.
struct RopeArgs {
  const uint64_t* turns;
  double magnitude;
  int32_t rot, pairs;  // pairs: rot / 2
  int32_t neighbours;
  int32_t unit;  // the magnitude is 1 or -1, not merely in FP32
};

template <typename F>
__device__ __forceinline__ void make_table(const RopeArgs& r, int tokens, float* table, F position) {
  const float mag = (float)r.magnitude;
  const int step_j = blockDim.x / r.pairs, step_i = blockDim.x - step_j * r.pairs;
  int j = threadIdx.x / r.pairs, i = threadIdx.x - j * r.pairs;
  while (j < tokens) {
    int64_t pos;
    if (position(j, pos)) {
      const float2 cs = cos_sin(__ldg(r.turns + i), pos);
      float* to = table + (size_t)j * r.rot + ((i & 7) >> 2) * (r.rot / 4) + (i >> 3) * 4 + (i & 3);
      to[0] = cs.x * mag;
      to[r.rot / 2] = cs.y * mag;
    }
    i += step_i;
    j += step_j;
    if (i >= r.pairs) i -= r.pairs, ++j;
  }
  __syncthreads();
}

// Asks for bytes, a multiple of 16, to be in L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// Eight cosines and sines of a group.
__device__ __forceinline__ void group_of(const float* table, int rot, int g, float (&c)[8], float (&s)[8]) {
  const float4* t = reinterpret_cast<const float4*>(table);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 a = t[h * (rot / 16) + g], b = t[(2 + h) * (rot / 16) + g];
    c[4 * h] = a.x, c[4 * h + 1] = a.y, c[4 * h + 2] = a.z, c[4 * h + 3] = a.w;
    s[4 * h] = b.x, s[4 * h + 1] = b.y, s[4 * h + 2] = b.z, s[4 * h + 3] = b.w;
  }
}

// A piece of eight elements as it lies in memory.
template <int TYPE>
struct Piece {
  uint4 w[TYPE == WD_F32 ? 2 : 1];
};
template <int TYPE>
__device__ __forceinline__ Piece<TYPE> load_piece(const void* p) {  // (may be written by this kernel later)
  Piece<TYPE> v;
#pragma unroll
  for (int i = 0; i < (TYPE == WD_F32 ? 2 : 1); ++i) v.w[i] = reinterpret_cast<const uint4*>(p)[i];
  return v;
}
template <int TYPE>
__device__ __forceinline__ void store_piece(void* p, const Piece<TYPE>& v) {
#pragma unroll
  for (int i = 0; i < (TYPE == WD_F32 ? 2 : 1); ++i) reinterpret_cast<uint4*>(p)[i] = v.w[i];
}
template <int TYPE>
__device__ __forceinline__ void floats_of(const Piece<TYPE>& v, float (&f)[8]) {
  if constexpr (TYPE == WD_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[4 * i] = __uint_as_float(v.w[i].x), f[4 * i + 1] = __uint_as_float(v.w[i].y);
      f[4 * i + 2] = __uint_as_float(v.w[i].z), f[4 * i + 3] = __uint_as_float(v.w[i].w);
    }
  } else {
    unpack8<TYPE == WD_BF16>(v.w[0], f);
  }
}
template <int TYPE>
__device__ __forceinline__ Piece<TYPE> piece_of(const float (&f)[8]) {
  Piece<TYPE> v;
  if constexpr (TYPE == WD_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      v.w[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
  } else {
    constexpr bool B = TYPE == WD_BF16;
    v.w[0] = make_uint4(pack2<B>(f[0], f[1]), pack2<B>(f[2], f[3]), pack2<B>(f[4], f[5]), pack2<B>(f[6], f[7]));
  }
  return v;
}

// Item w of a head: two pieces, both read before either is written, so that out may be x.
// The first rot / 16 turn (the pieces w and w + rot / 16, or 2w and 2w + 1), the rest are copied where `copies`.
template <int TYPE>
struct TurnItem {
  static constexpr int kPieceBytes = TYPE == WD_F32 ? 32 : 16;
  Piece<TYPE> a, b;
  const float* table;  // null: copied
  char* to;            // null: nothing to do
  int w, q;            // q: of the second piece, 0: none

  __device__ __forceinline__ void none() { to = nullptr; }
  __device__ __forceinline__ void load(const RopeArgs& r, const float* row, const void* head, void* out, int item, int pieces,
                                       bool copies) {
    const int groups = r.rot / 16;
    const bool turns = item < groups;
    to = nullptr;
    if (!turns && !copies) return;
    int p = 2 * item;
    w = item, q = 2 * item + 1;
    if (turns && !r.neighbours) p = item, q = item + groups;
    const char* from = static_cast<const char*>(head);
    table = turns ? row : nullptr;
    to = static_cast<char*>(out) + p * kPieceBytes;
    a = load_piece<TYPE>(from + p * kPieceBytes);
    b = a;
    if (q < pieces) b = load_piece<TYPE>(from + q * kPieceBytes);
    q = q < pieces ? q - p : 0;
  }
  __device__ __forceinline__ void finish(const RopeArgs& r) {
    if (!to) return;
    if (table) {
      float x[8], y[8], c[8], s[8];
      floats_of<TYPE>(a, x);
      floats_of<TYPE>(b, y);
      group_of(table, r.rot, w, c, s);
      if (r.neighbours) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = x[2 * i], o = x[2 * i + 1], e2 = y[2 * i], o2 = y[2 * i + 1];
          x[2 * i] = fmaf(e, c[i], -(o * s[i])), x[2 * i + 1] = fmaf(o, c[i], e * s[i]);
          y[2 * i] = fmaf(e2, c[4 + i], -(o2 * s[4 + i])), y[2 * i + 1] = fmaf(o2, c[4 + i], e2 * s[4 + i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u = x[i], v = y[i];
          x[i] = fmaf(u, c[i], -(v * s[i])), y[i] = fmaf(v, c[i], u * s[i]);
        }
      }
      a = piece_of<TYPE>(x);
      b = piece_of<TYPE>(y);
    }
    store_piece<TYPE>(to, a);
    if (q) store_piece<TYPE>(to + q * kPieceBytes, b);
  }
};

// ------------------------------------------------------------------ wd_rope --

struct TurnArgs {
  RopeArgs r;
  const char* x;
  char* out;
  const int32_t* positions;
  int64_t ldx, ldo;  // bytes
  int32_t T, head_bytes, pieces;
  int32_t per, heads, items, chunk;  // tokens of a CTA, heads in all, items of a head, of a token in a CTA
  bool copies, ahead;  // ahead: whole heads are asked into L2
};

template <int TYPE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const TurnArgs a) {
  extern __shared__ float4 dyn4[];
  float* table = reinterpret_cast<float*>(dyn4);
  const int tok0 = blockIdx.x * a.per, tokens = min(a.per, a.T - tok0);
  const int w0 = blockIdx.y * a.chunk, end = min(a.chunk, a.heads * a.items - w0);
  if (a.ahead && threadIdx.x < tokens) {  // what this CTA reads comes to L2 while it computes its table
    const int h0 = w0 / a.items, h1 = (w0 + end - 1) / a.items;
    prefetch_l2(a.x + (int64_t)(tok0 + threadIdx.x) * a.ldx + (int64_t)h0 * a.head_bytes, (h1 - h0 + 1) * a.head_bytes);
  }
  make_table(a.r, tokens, table, [&](int j, int64_t& pos) {
    pos = __ldg(a.positions + tok0 + j);
    return true;
  });
  for (Walk walk(a.chunk); walk.j < tokens; walk.next()) {
    if (walk.w >= end) continue;
    const int head = (w0 + walk.w) / a.items, w = w0 + walk.w - head * a.items;
    const int64_t tok = tok0 + walk.j;
    TurnItem<TYPE> item;
    item.load(a.r, table + walk.j * a.r.rot, a.x + tok * a.ldx + (int64_t)head * a.head_bytes,
              a.out + tok * a.ldo + (int64_t)head * a.head_bytes, w, a.pieces, a.copies);
    item.finish(a.r);
  }
}

// ------------------------------------------------------- wd_kv4_rope_append --

struct RopeAppendArgs {
  RopeArgs r;
  TokenArgs t;
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  uint8_t *kc, *ks, *vc, *vs;
  int64_t ldq, ldqo;
  int32_t slices, kv_slices;      // of a run of tokens, one CTA each and next to each other; behind kv_slices the queries'
  int32_t q_heads, q_chunk;       // items of a token in a CTA
  bool copies;
};

// The exact turned element e of a head of k, in 64 bits.
template <bool BF16>
__device__ double exact_element(const RopeArgs& r, const uint16_t* head, int e, int64_t pos) {
  const double x = load_elem(head, BF16 ? WD_BF16 : WD_F16, e);
  if (e >= r.rot) return x;
  const int half = r.rot / 2;
  const int other = r.neighbours ? e ^ 1 : e < half ? e + half : e - half;
  const bool second = r.neighbours ? e & 1 : e >= half;
  const int i = r.neighbours ? e >> 1 : second ? other : e;
  const double y = load_elem(head, BF16 ? WD_BF16 : WD_F16, other);
  double s, c;
  sincospi((double)(int64_t)(r.turns[i] * (uint64_t)pos) * 0x1p-63, &s, &c);
  return r.magnitude * (second ? x * c + y * s : x * c - y * s);
}

__device__ __forceinline__ uint32_t nearest_e2m1(double v) {
  const double m = fabs(v);
  return (uint32_t)((m > 0.25) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)) |
         (signbit(v) ? 8u : 0u);
}

__device__ __forceinline__ double unscale64(uint32_t s) { return __longlong_as_double((long long)(1023 + 127 - (int)s) << 52); }

// The codes of a piece again, for the nibbles that `unsure` has set.
template <bool BF16>
__device__ __noinline__ uint32_t settle_codes(const RopeArgs& r, const uint16_t* head, int w, int64_t pos, uint32_t scale,
                                              uint32_t codes, uint32_t unsure) {
#pragma unroll 1
  for (int j = 0; j < 8; ++j)
    if (unsure >> (4 * j) & 15u) {
      const uint32_t c = nearest_e2m1(exact_element<BF16>(r, head, 8 * w + j, pos) * unscale64(scale));
      codes = (codes & ~(15u << (4 * j))) | c << (4 * j);
    }
  return codes;
}

// The scale of a block again (the four threads of `quad`).
template <bool BF16>
__device__ __noinline__ uint32_t settle_scale(const RopeArgs& r, const uint16_t* head, int w, int64_t pos, unsigned quad) {
  double m = 0.0;
#pragma unroll 1
  for (int j = 0; j < 8; ++j) m = fmax(m, fabs(exact_element<BF16>(r, head, 8 * w + j, pos)));
  m = fmax(m, __shfl_xor_sync(quad, m, 1));
  m = fmax(m, __shfl_xor_sync(quad, m, 2));
  const int e = (int)(__double_as_longlong(m) >> 52) - 1023 - 2 + 127;
  return (uint32_t)(m == 0.0 ? 0 : max(0, min(254, e)));
}

// The largest magnitude of a piece, as FP32 bits (NaN and infinities: infinity).
template <bool BF16>
__device__ __forceinline__ uint32_t piece_top(const uint4& raw) {
  const uint32_t two = __vmaxu2(__vmaxu2(raw.x & 0x7FFF7FFFu, raw.y & 0x7FFF7FFFu),
                                __vmaxu2(raw.z & 0x7FFF7FFFu, raw.w & 0x7FFF7FFFu));
  const uint32_t m = max(two & 0xFFFFu, two >> 16);
  return magnitude(BF16 ? __uint_as_float(m << 16) : half_lo(m));
}

constexpr int kAppendResident = 4;  // CTAs of an SM, in 64 registers

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, kAppendResident) kv4_rope_append_kernel(const RopeAppendArgs a) {
  extern __shared__ float4 dyn4[];
  float* table = reinterpret_cast<float*>(dyn4);
  __shared__ Pair s_pair[kMostPer];
  __shared__ int64_t s_pos[kMostPer];
  const TokenArgs& t = a.t;
  const RopeArgs& r = a.r;
  const int run = blockIdx.x / a.slices, slice = blockIdx.x - run * a.slices;
  const int tok0 = run * t.per, tid = threadIdx.x;
  const bool queries = slice >= a.kv_slices;
  // What this CTA reads comes to L2 while it finds its tokens' places, unless its run is short, as in a step: then a projection has
  // just written it, and it is there. 64 tokens with 64 + 4 heads 4.6 us so and 4.8 with it (5.5 and 5.0 from DRAM), 256 with 32 + 8 heads
  // 5.6 and 5.8 (6.2 and 5.8); 4800 tokens 31.4 without and 29.7 with it (32.5 and 31.1).
  if (t.per > 4 && tid < t.per && tok0 + tid < t.T) {
    const int64_t tok = tok0 + tid;
    if (queries) {
      const int w0 = (slice - a.kv_slices) * a.q_chunk, end = min(a.q_chunk, a.q_heads * (D / 16) - w0);
      prefetch_l2(a.q + tok * a.ldq + w0 * 16, end * 32);
    } else {
      prefetch_l2(a.k + tok * t.ldk + slice * t.chunk * 8, t.chunk * 16);
      prefetch_l2(a.v + tok * t.ldv + slice * t.chunk * 8, t.chunk * 16);
    }
  }
  const int pairs = find_pairs(t, tok0, s_pair, s_pos);
  // one token more for the keys: a pair may end behind the run
  make_table(r, t.per + (queries ? 0 : 1), table, [&](int j, int64_t& pos) {
    pos = j < t.per ? s_pos[j] : s_pos[j - 1] + (s_pos[j - 1] >= 0);
    return pos >= 0;
  });
  if (queries) {
    constexpr int kPerHead = D / 16, kItems = 2;  // kItems: of a thread, in flight
    const int w0 = (slice - a.kv_slices) * a.q_chunk, end = min(a.q_chunk, a.q_heads * kPerHead - w0);
    for (Walk walk(a.q_chunk); walk.j < t.per;) {
      TurnItem<BF16 ? WD_BF16 : WD_F16> item[kItems];
#pragma unroll
      for (int n = 0; n < kItems; ++n, walk.next()) {
        item[n].none();
        if (walk.j >= t.per || walk.w >= end || s_pos[walk.j] < 0) continue;
        const int w = w0 + walk.w;
        const int64_t tok = tok0 + walk.j, head = (int64_t)(w / kPerHead) * D;
        item[n].load(r, table + walk.j * r.rot, a.q + tok * a.ldq + head, a.q_out + tok * a.ldqo + head, w % kPerHead, D / 8,
                     a.copies);
      }
#pragma unroll
      for (int n = 0; n < kItems; ++n) item[n].finish(r);
    }
    return;
  }
  const unsigned quad = 0xFu << (tid & 28);
  auto plain = [&](const uint4& raw, uint32_t& scale) {  // of V
    uint32_t m = piece_top<BF16>(raw);
    m = max(m, __shfl_xor_sync(quad, m, 1));
    m = max(m, __shfl_xor_sync(quad, m, 2));
    float f[8];
    unpack8<BF16>(raw, f);
    scale = fp4_scale_code(__uint_as_float(m));
    const float u = fp4_unscale(scale);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= u;
    return e2m1x8(f);
  };
  const int groups = r.rot / 16;
  // w: the piece of the head; j: the token in the run
  auto turned = [&](const uint4& raw, const uint4& raw2, int w, int j, int64_t tok, int head, uint32_t& scale) {
    float f[8];
    unpack8<BF16>(raw, f);
    uint32_t in = 0;  // the largest of what is turned
    uint32_t sines = 0;  // 0 where the turn changes signs at most
    if (w < 2 * groups) {
      in = piece_top<BF16>(raw);
      const float* row = table + j * r.rot;
      if (r.neighbours) {
        const float4 c = reinterpret_cast<const float4*>(row)[(w & 1) * groups + (w >> 1)];
        const float4 s = reinterpret_cast<const float4*>(row)[(2 + (w & 1)) * groups + (w >> 1)];
        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) sines |= __float_as_uint(sn[i]) << 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = f[2 * i], o = f[2 * i + 1];
          f[2 * i] = fmaf(e, cs[i], -(o * sn[i])), f[2 * i + 1] = fmaf(o, cs[i], e * sn[i]);
        }
      } else {
        in = max(in, piece_top<BF16>(raw2));
        float y[8], c[8], s[8];
        unpack8<BF16>(raw2, y);
        group_of(row, r.rot, w < groups ? w : w - groups, c, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) sines |= __float_as_uint(s[i]) << 1;
        const uint32_t flip = w < groups ? 0x80000000u : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = fmaf(f[i], c[i], __uint_as_float(__float_as_uint(y[i] * s[i]) ^ flip));
      }
    }
    if (sines == 0 && r.unit) in = 0;  // f is exact
    // The doubt is this piece's own: one that turns by nothing, or not at all, has none in a block that turns.
    const float own = __uint_as_float(in) * (kDoubt * fabsf((float)r.magnitude));
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, magnitude(f[i]));
    uint32_t lo = m == 0x7F800000u ? m : __float_as_uint(fmaxf(__uint_as_float(m) - own, 0.0f));
    uint32_t hi = __float_as_uint(__uint_as_float(m) + own);
    lo = max(lo, __shfl_xor_sync(quad, lo, 1));
    lo = max(lo, __shfl_xor_sync(quad, lo, 2));
    hi = max(hi, __shfl_xor_sync(quad, hi, 1));
    hi = max(hi, __shfl_xor_sync(quad, hi, 2));
    scale = fp4_scale_code(__uint_as_float(lo));
    if (scale == 255u) return 0u;
    const uint16_t* row = a.k + tok * t.ldk + (int64_t)head * D;
    auto pos = [&]() { return j < t.per ? s_pos[j] : s_pos[j - 1] + 1; };
    if (fp4_scale_code(__uint_as_float(hi)) != scale) scale = settle_scale<BF16>(r, row, w, pos(), quad);
    const float u = fp4_unscale(scale), d = -own * u;  // (-0 leaves zeros their signs)
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = fmaf(f[i], u, -d), f[i] = fmaf(f[i], u, d);
    const uint32_t codes = e2m1x8(f), other = own == 0.0f ? codes : e2m1x8(g);
    return codes == other ? codes : settle_codes<BF16>(r, row, w, pos(), scale, codes, codes ^ other);
  };
  const int kv0 = slice * t.chunk;
  for (Walk walk(t.chunk); walk.j < pairs; walk.next()) {
    const int hw = kv0 + walk.w;
    const Pair p = s_pair[walk.j];  // the four threads of a block have the same
    const int head = hw / (D / 8), w = hw % (D / 8), b = w >> 2, q4 = w & 3;
    const int64_t tok = tok0 + p.j;
    const uint16_t *kp = a.k + tok * t.ldk + hw * 8, *vp = a.v + tok * t.ldv + hw * 8;
    const int apart = r.neighbours || w >= 2 * groups ? 0 : w < groups ? 8 * groups : -8 * groups;  // to the partners' piece
    const uint4 raw_v = ld_cached16(vp), raw_k = ld_cached16(kp), raw_k2 = ld_cached16(kp + apart);
    uint4 next_v, next_k, next_k2;
    if (p.both) next_v = ld_cached16(vp + t.ldv), next_k = ld_cached16(kp + t.ldk), next_k2 = ld_cached16(kp + t.ldk + apart);
    const size_t at = ((size_t)p.page * t.heads + head) << t.page_shift;  // in tokens
    uint32_t sv, sk, v0 = plain(raw_v, sv), v1 = 0, sv1 = 0;
    uint8_t* kto = a.kc + at * (D / 2) + k_word<D>(p.slot, q4, b);
    uint8_t* ksto = a.ks + at * (D / 32) + p.slot * (D / 32) + b;
    *reinterpret_cast<uint32_t*>(kto) = turned(raw_k, raw_k2, w, p.j, tok, head, sk);
    if (q4 == 0) *ksto = (uint8_t)sk;
    if (p.both) {
      v1 = plain(next_v, sv1);
      *reinterpret_cast<uint32_t*>(kto + D / 2) = turned(next_k, next_k2, w, p.j + 1, tok + 1, head, sk);
      if (q4 == 0) ksto[D / 32] = (uint8_t)sk;
    }
    // V as in wd_kv4_append: a key alone replaces its own nibbles
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t* to = reinterpret_cast<uint32_t*>(a.vc + at * (D / 2) + v_word<D>(p.slot >> 1, 2 * q4 + h, b));
      const uint32_t x = spread4(v0 >> (16 * h));
      if (p.both) {
        *to = x | spread4(v1 >> (16 * h)) << 4;
      } else {
        const int up = (p.slot & 1) * 4;
        atomicAnd(to, ~(0x0F0F0F0Fu << up));
        atomicOr(to, x << up);
      }
    }
    if (q4 == 0) {
      uint8_t* to = a.vs + at * (D / 32) + v_scale<D>(p.slot, b);
      if (p.both)
        *reinterpret_cast<uint16_t*>(to) = (uint16_t)(sv | sv1 << 8);
      else
        *to = (uint8_t)sv;
    }
  }
}

// ------------------------------------------------------------------ launches --

moe_status check_rotation(const wd_rotation* r, int32_t dim) {
  if (!r) return refuse(MOE_ERR_NULL, "wd_rope: a rotation is required");
  if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > dim)
    return refuse(MOE_ERR_SHAPE, "wd_rope: rot_dim is a multiple of 16, from 16 to the head's elements");
  const double m = std::fabs(r->magnitude);
  if (!(m <= 65536.0 && (m == 0.0 || m >= 0x1p-100)))  // (below, FP32 has it with fewer bits, or as 0)
    return refuse(MOE_ERR_UNSUPPORTED, "wd_rope: the magnitude is 0, or from 2^-100 to 65536");
  if (!r->turns) return refuse(MOE_ERR_NULL, "wd_rope: turns are required");
  if (!aligned(r->turns, 8)) return refuse(MOE_ERR_ALIGN, "wd_rope: turns need 8 bytes");
  return MOE_OK;
}

RopeArgs rope_args(const wd_rotation* r) {
  return {r->turns, r->magnitude, r->rot_dim, r->rot_dim / 2, r->neighbours ? 1 : 0, std::fabs(r->magnitude) == 1.0};
}

// Tokens of a CTA: T tokens in `slices` slices, each run's table at most kTable bytes, in a multiple of `waves_of` waves.
constexpr int kTable = 16 * 1024;
int tokens_of_a_cta(int64_t T, int slices, int rot, int resident, int least, int waves_of) {
  const int64_t slots = (int64_t)sm_count() * resident, most = std::max(least, std::min(kMostPer - 1, kTable / (rot * 4)));
  const int64_t waves = (T * slices + slots * most * waves_of - 1) / (slots * most * waves_of) * waves_of;
  const int64_t even = (T * slices + slots * waves - 1) / (slots * waves);
  return (int)std::max((int64_t)least, std::min(most, even));
}

template <int TYPE>
moe_status turn(const TurnArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((a.T + (int64_t)a.per - 1) / a.per), (unsigned)((a.heads * a.items + a.chunk - 1) / a.chunk));
  rope_kernel<TYPE><<<grid, kThreads, (size_t)a.per * a.r.rot * 4, st>>>(a);
  return launched("wd_rope launch");
}

template <int D>
moe_status rope_append(const RopeAppendArgs& a, bool bf16, unsigned grid, cudaStream_t st) {
  const size_t table = (size_t)(a.t.per + 1) * a.r.rot * 4;
  if (bf16)
    kv4_rope_append_kernel<D, true><<<grid, kThreads, table, st>>>(a);
  else
    kv4_rope_append_kernel<D, false><<<grid, kThreads, table, st>>>(a);
  return launched("wd_kv4_rope_append launch");
}

}  // namespace
}  // namespace wd

extern "C" moe_status wd_rope_turns(int32_t n, const double* freqs, uint64_t* turns) {
  using namespace wd;
  if (n < 0) return refuse(MOE_ERR_SHAPE, "wd_rope_turns: need n >= 0");
  if (n && (!freqs || !turns)) return refuse(MOE_ERR_NULL, "wd_rope_turns: freqs and turns are required");
  for (int32_t i = 0; i < n; ++i)
    if (!(std::fabs(freqs[i]) <= 65536.0))
      return refuse(MOE_ERR_UNSUPPORTED, "wd_rope_turns: a frequency is at most 65536 radians per position");
  // 1 / (2 pi) as a sum of two doubles; the product's whole turns do not matter
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  for (int32_t i = 0; i < n; ++i) {
    const double f = std::fabs(freqs[i]), p = f * hi, rest = std::fma(f, hi, -p) + f * lo;
    const double part = p - std::floor(p);  // exact
    const double first = std::floor(part * 0x1p32), second = (part * 0x1p32 - first) * 0x1p32 + rest * 0x1p64;
    const uint64_t t = ((uint64_t)first << 32) + (uint64_t)(int64_t)std::nearbyint(second);
    turns[i] = freqs[i] < 0 ? 0 - t : t;
  }
  return MOE_OK;
}

extern "C" moe_status wd_rope(const wd_rotation* r, const void* x, int32_t type, int64_t ldx, int32_t T, int32_t heads,
                              int32_t dim, const int32_t* positions, void* out, int64_t ldo, void* stream) {
  using namespace wd;
  if (T < 0 || heads < 0 || dim < 16 || dim % 8 || dim > 1024)
    return refuse(MOE_ERR_SHAPE, "wd_rope: need T, heads >= 0 and dim a multiple of 8 from 16 to 1024");
  moe_status rc = check_rotation(r, dim);
  if (rc != MOE_OK) return rc;
  if (!valid_type(type)) return refuse(MOE_ERR_UNSUPPORTED, "wd_rope: x and out are F32, BF16 or F16");
  const int64_t row = (int64_t)heads * dim;
  if (row > 1 << 20) return refuse(MOE_ERR_SHAPE, "wd_rope: a token has at most 2^20 elements");
  if (ldx < row || ldo < row || (x == out && ldx != ldo))
    return refuse(MOE_ERR_SHAPE, "wd_rope: ldx or ldo is shorter than a token, or they differ in place");
  if (T == 0 || heads == 0) return MOE_OK;
  if (!x || !positions || !out) return refuse(MOE_ERR_NULL, "wd_rope: x, positions and out are required");
  const int vec = type == WD_F32 ? 4 : 8;
  if (!aligned(x, 16) || !aligned(out, 16) || ldx % vec || ldo % vec || !aligned(positions, 4))
    return refuse(MOE_ERR_ALIGN, "wd_rope: x and out need 16 bytes, as do their strides, positions 4");
  TurnArgs a = {};
  a.r = rope_args(r);
  a.x = static_cast<const char*>(x), a.out = static_cast<char*>(out), a.positions = positions;
  a.ldx = ldx * type_bytes(type), a.ldo = ldo * type_bytes(type);
  a.T = T, a.head_bytes = dim * type_bytes(type), a.pieces = dim / 8, a.heads = heads;
  a.copies = x != out;
  a.items = a.copies ? (a.pieces + 1) / 2 : a.r.rot / 16;
  const int all = heads * a.items, slices = (all + kThreads - 1) / kThreads;
  a.chunk = (all + slices - 1) / slices;
  a.per = tokens_of_a_cta(T, slices, a.r.rot, 6, 1, 4);
  // In place only the turned elements are read: of a third of a head or less they wait rather than bring the rest along. With and
  // without, 7001 tokens with 20 heads of 256 in place, 64 turned: 14.2 and 10.3 us; 128 turned: 17.6 and 19.2; 5000 with 33 heads of
  // 80, 32 turned: 8.8 and 10.6; 10000 with 40 heads of 128, 32 turned: 20.9 and 16.5, 64 turned 24.0 and 21.3.
  a.ahead = a.per > 1 && (a.copies || 3 * a.r.rot > dim);
  cudaStream_t st = (cudaStream_t)stream;
  return type == WD_F32 ? turn<WD_F32>(a, st) : type == WD_BF16 ? turn<WD_BF16>(a, st) : turn<WD_F16>(a, st);
}

extern "C" moe_status wd_kv4_rope_append(const wd_kv4_cache* c, const wd_rotation* r, const void* q, int64_t ldq,
                                         int32_t q_heads, void* q_out, int64_t ldqo, const void* k, const void* v, int32_t type,
                                         int64_t ldk, int64_t ldv, int32_t T, const int32_t* table, int32_t max_blocks,
                                         const int32_t* lens, const int32_t* cu, int32_t S, int32_t* err, void* stream) {
  using namespace wd;
  moe_status rc = check_tokens(c, k, v, type, ldk, ldv, T, table, max_blocks, lens, cu, S, err, false);
  if (rc != MOE_OK) return rc;
  rc = check_rotation(r, c->dim);
  if (rc != MOE_OK) return rc;
  const int64_t row = (int64_t)q_heads * c->dim;
  if (q_heads < 0 || row > 1 << 20 || (q_heads && (ldq < row || ldqo < row || (q == q_out && ldq != ldqo))))
    return refuse(MOE_ERR_SHAPE, "wd_kv4_rope_append: need q_heads >= 0, up to 2^20 elements, ldq and ldqo of a token "
                                 "at least, and the same in place");
  if (T == 0 || S == 0) return MOE_OK;
  if (q_heads && (!q || !q_out)) return refuse(MOE_ERR_NULL, "wd_kv4_rope_append: q and q_out are required");
  if (q_heads && (!aligned(q, 16) || !aligned(q_out, 16) || ldq % 8 || ldqo % 8))
    return refuse(MOE_ERR_ALIGN, "wd_kv4_rope_append: q and q_out need 16 bytes and strides % 8 == 0");
  RopeAppendArgs a = {};
  a.r = rope_args(r);
  a.t = token_args(c, ldk, ldv, T, table, max_blocks, lens, cu, S, err);
  a.q = static_cast<const uint16_t*>(q), a.q_out = static_cast<uint16_t*>(q_out), a.ldq = ldq, a.ldqo = ldqo;
  a.k = static_cast<const uint16_t*>(k), a.v = static_cast<const uint16_t*>(v);
  a.kc = c->k_codes, a.ks = c->k_scales, a.vc = c->v_codes, a.vs = c->v_scales;
  a.copies = q != q_out;
  a.kv_slices = c->heads * (c->dim / 8) / a.t.chunk;
  // A slice of the queries: up to 256 items of 16 elements.
  const int items = q_heads * (c->dim / 16), q_slices = (items + kThreads - 1) / kThreads;
  a.q_heads = q_heads;
  a.q_chunk = q_slices ? (items + q_slices - 1) / q_slices : 1;
  a.slices = a.kv_slices + q_slices;
  a.t.per = tokens_of_a_cta(T, a.slices, a.r.rot, kAppendResident, 2, 3);
  const int64_t ctas = (T + (int64_t)a.t.per - 1) / a.t.per * a.slices;
  if (ctas > INT32_MAX) return refuse(MOE_ERR_SHAPE, "wd_kv4_rope_append: too many tokens times heads");
  const unsigned grid = (unsigned)ctas;
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf16 = type == WD_BF16;
  return c->dim == 64    ? rope_append<64>(a, bf16, grid, st)
         : c->dim == 128 ? rope_append<128>(a, bf16, grid, st)
                         : rope_append<256>(a, bf16, grid, st);
}
