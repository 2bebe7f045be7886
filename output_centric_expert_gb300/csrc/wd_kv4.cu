// The KV cache held in 4 bits (MXFP4): appending tokens and reading them back.
#include "wd_block.cuh"
#include "wd_kv4.cuh"

namespace wd {
namespace {

// ------------------------------------------------------- append and gather --
// A CTA takes `per` tokens in a row and up to 128 of their 8-element pieces. Its first
// threads find the tokens' places (sequence by bisection in cu_new, page, slot) once
// for all, and a thread takes a piece of two tokens that share bytes of V: no exchange
// between threads (through shared memory and a barrier: 27.4 us for the prompts below).
// The four threads of a 32-element block are neighbours: its largest magnitude takes
// two shuffles. Both kernels are bound by integer instructions (conversions,
// packing, addresses), so magnitudes are compared as 16-bit pairs and a thread steps
// through its pieces without divisions. Prompts of 9.7k tokens, 8 heads of dim 128, into
// the cache and back (100 MB): 23.5 us, 4.3 TB/s, half of it places, first loads and the
// two launches; 262k tokens of 4 heads into it 98 us, DRAM 70 %, ALU 64 %. One token each
// of 64 sequences: 3.6 us a launch.

struct TokenArgs {
  const int32_t *table, *lens, *cu;
  int32_t* err;
  int64_t ldk, ldv;
  int32_t T, S, max_blocks;
  int32_t pages, page_shift, heads;
  int32_t per, chunk;  // tokens of a CTA, pieces of a token in a CTA
};

// The place of a new token; `before`, `behind`: the tokens next to it are new ones of
// its sequence too. page -1: ignored (behind cu[S]) or left out (flagged).
struct Place {
  int32_t page, slot;
  bool before, behind;
};
// A new token with an even slot and the next one where that is new too (`both`), or one
// with an odd slot whose neighbour is none of its sequence's new ones: what shares bytes of V. j: the first's.
struct Pair {
  int32_t page, slot, j;
  bool both;
};
constexpr int kMostPer = 64;
constexpr int kResident = 5;  // CTAs of an SM: a pair's four loads in flight take 48 registers

__device__ __forceinline__ Place place_of(const TokenArgs& a, int tok, bool here) {
  Place p = {-1, 0, false, false};
  int s = tok, first = tok, end = tok + 1;
  if (!here || tok >= a.T) return p;
  if (a.cu) {
    if (tok >= __ldg(a.cu + a.S) || tok < __ldg(a.cu)) return p;
    int lo = 0, hi = a.S - 1;  // the last s with cu[s] <= tok
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.cu + mid) <= tok)
        lo = mid;
      else
        hi = mid - 1;
    }
    s = lo;
    first = __ldg(a.cu + s);
    end = min(__ldg(a.cu + s + 1), a.T);
  }
  p.before = tok > first;
  p.behind = tok + 1 < end;
  const int len = __ldg(a.lens + s);
  const int64_t pos = (int64_t)len + (tok - first);
  const int64_t block = pos >> a.page_shift;
  if (len >= 0 && block < a.max_blocks) p.page = __ldg(a.table + (int64_t)s * a.max_blocks + block);
  p.slot = (int)(pos & ((1 << a.page_shift) - 1));
  if (p.page < 0 || p.page >= a.pages) {
    p.page = -1;
    flag_invalid(a.err);
  }
  return p;
}

// The pairs that begin in a CTA's tokens, in order; returns their number. All threads.
__device__ __forceinline__ int find_pairs(const TokenArgs& a, int tok0, Pair* s_pair) {
  __shared__ uint32_t s_first[kMostPer / 32];
  const int tid = threadIdx.x;
  Place p;
  uint32_t first = 0;
  if (tid < kMostPer) {  // whole warps
    p = place_of(a, tok0 + tid, tid < a.per);
    first = __ballot_sync(0xFFFFFFFFu, p.page >= 0 && !((p.slot & 1) && p.before));
    if ((tid & 31) == 0) s_first[tid >> 5] = first;
  }
  __syncthreads();
  int pairs = 0;
#pragma unroll
  for (int n = 0; n < kMostPer / 32; ++n) pairs += __popc(s_first[n]);
  if (tid < kMostPer && (first >> (tid & 31)) & 1u) {
    int at = __popc(first & ((1u << (tid & 31)) - 1u));
#pragma unroll
    for (int n = 0; n < kMostPer / 32; ++n) at += n < tid >> 5 ? __popc(s_first[n]) : 0;
    s_pair[at] = {p.page, p.slot, tid, !(p.slot & 1) && p.behind};
  }
  __syncthreads();
  return pairs;
}

// The (pair, piece) of a thread's i-th item, i = threadIdx.x, + kThreads, ...
struct Walk {
  int i, j, w;
  const int chunk, dj, dw;
  __device__ explicit Walk(int c)
      : i(threadIdx.x), j(threadIdx.x / c), w(threadIdx.x - threadIdx.x / c * c), chunk(c), dj(kThreads / c),
        dw(kThreads - kThreads / c * c) {}
  __device__ void next() {
    i += kThreads;
    j += dj;
    w += dw;
    if (w >= chunk) {
      w -= chunk;
      ++j;
    }
  }
};

// Four E2M1 codes (the low 16 bits) to the low nibbles of four bytes.
__device__ __forceinline__ uint32_t spread4(uint32_t x) {
  const uint32_t t = __byte_perm(x, 0, 0x4140);  // byte 0 and byte 1 to the halves
  return (t & 0x000F000Fu) | ((t << 4) & 0x0F000F00u);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, kResident)
    kv4_append_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                      uint8_t* __restrict__ kc, uint8_t* __restrict__ ks, uint8_t* __restrict__ vc,
                      uint8_t* __restrict__ vs, const TokenArgs a) {
  __shared__ Pair s_pair[kMostPer];
  const int tok0 = blockIdx.x * a.per, w0 = blockIdx.y * a.chunk, tid = threadIdx.x;
  const int pairs = find_pairs(a, tok0, s_pair);
  // the scale code of a piece's block, and its codes
  const unsigned quad = 0xFu << (tid & 28);
  auto quantise = [&](const uint4& raw, uint32_t& scale) {
    // magnitudes as 16-bit integers, two to a word (NaN above infinity above the rest)
    const uint32_t two = __vmaxu2(__vmaxu2(raw.x & 0x7FFF7FFFu, raw.y & 0x7FFF7FFFu),
                                  __vmaxu2(raw.z & 0x7FFF7FFFu, raw.w & 0x7FFF7FFFu));
    uint32_t m = max(two & 0xFFFFu, two >> 16);
    m = max(m, __shfl_xor_sync(quad, m, 1));
    m = max(m, __shfl_xor_sync(quad, m, 2));
    float f[8];
    unpack8<BF16>(raw, f);
    scale = fp4_scale_code(BF16 ? __uint_as_float(m << 16) : half_lo(m));
    const float u = fp4_unscale(scale);  // (the codes of a NaN block, whose u is 0, do not matter)
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] *= u;
    return e2m1x8(f);
  };
  for (Walk walk(a.chunk); walk.j < pairs; walk.next()) {
    const int w = w0 + walk.w;
    const Pair p = s_pair[walk.j];  // the four threads of a block have the same
    const int head = w / (D / 8), b = w % (D / 8) >> 2, t = w & 3;
    const int64_t tok = tok0 + p.j;
    const uint16_t *kp = k + tok * a.ldk + w * 8, *vp = v + tok * a.ldv + w * 8;
    const uint4 raw_v = ld_cached16(vp), raw_k = ld_cached16(kp);
    uint4 next_v, next_k;
    if (p.both) next_v = ld_cached16(vp + a.ldv), next_k = ld_cached16(kp + a.ldk);
    const size_t at = ((size_t)p.page * a.heads + head) << a.page_shift;  // in tokens
    uint32_t sv, sk, v0 = quantise(raw_v, sv), v1 = 0, sv1 = 0;
    uint8_t* kto = kc + at * (D / 2) + k_word<D>(p.slot, t, b);
    uint8_t* ksto = ks + at * (D / 32) + p.slot * (D / 32) + b;
    *reinterpret_cast<uint32_t*>(kto) = quantise(raw_k, sk);
    if (t == 0) *ksto = (uint8_t)sk;
    if (p.both) {
      v1 = quantise(next_v, sv1);
      *reinterpret_cast<uint32_t*>(kto + D / 2) = quantise(next_k, sk);
      if (t == 0) ksto[D / 32] = (uint8_t)sk;
    }
    // V: a byte holds an element of an even key and the next. A key alone replaces its own nibbles, and the
    // neighbour's stay as they are: another entry of the call may write those meanwhile, so each of the two
    // steps is one operation of memory. (They touch different bits, so their order does not matter.)
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // elements 4h .. 4h + 3: g = 2t + h
      uint32_t* to = reinterpret_cast<uint32_t*>(vc + at * (D / 2) + v_word<D>(p.slot >> 1, 2 * t + h, b));
      const uint32_t x = spread4(v0 >> (16 * h));
      if (p.both) {
        *to = x | spread4(v1 >> (16 * h)) << 4;
      } else {
        const int up = (p.slot & 1) * 4;
        atomicAnd(to, ~(0x0F0F0F0Fu << up));
        atomicOr(to, x << up);
      }
    }
    if (t == 0) {
      uint8_t* to = vs + at * (D / 32) + v_scale<D>(p.slot, b);
      if (p.both)
        *reinterpret_cast<uint16_t*>(to) = (uint16_t)(sv | sv1 << 8);
      else
        *to = (uint8_t)sv;
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t i, const uint32_t (&h)[4], float s) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = half_lo(h[j]) * s;
    f[2 * j + 1] = half_hi(h[j]) * s;
  }
  if (TYPE == WD_F32) {
    float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + i);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    uint4 o;
    o.x = pack2<TYPE == WD_BF16>(f[0], f[1]);
    o.y = pack2<TYPE == WD_BF16>(f[2], f[3]);
    o.z = pack2<TYPE == WD_BF16>(f[4], f[5]);
    o.w = pack2<TYPE == WD_BF16>(f[6], f[7]);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + i) = o;
  }
}

template <int D, int TYPE>
__global__ void __launch_bounds__(kThreads)
    kv4_gather_kernel(void* __restrict__ k, void* __restrict__ v, const uint8_t* __restrict__ kc,
                      const uint8_t* __restrict__ ks, const uint8_t* __restrict__ vc,
                      const uint8_t* __restrict__ vs, const TokenArgs a) {
  __shared__ Pair s_pair[kMostPer];
  const int tok0 = blockIdx.x * a.per, w0 = blockIdx.y * a.chunk;
  const int pairs = find_pairs(a, tok0, s_pair);
  for (Walk walk(a.chunk); walk.j < pairs; walk.next()) {
    const int w = w0 + walk.w;
    const Pair p = s_pair[walk.j];
    const int head = w / (D / 8), b = w % (D / 8) >> 2, t = w & 3, odd = p.slot & 1;
    const int64_t tok = tok0 + p.j;
    const size_t at = ((size_t)p.page * a.heads + head) << a.page_shift;
    const uint8_t* kfrom = kc + at * (D / 2) + k_word<D>(p.slot, t, b);
    const uint8_t* ksfrom = ks + at * (D / 32) + p.slot * (D / 32) + b;
    const uint8_t* vsfrom = vs + at * (D / 32) + v_scale<D>(p.slot, b);
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(kfrom), sk = *ksfrom, sv = *vsfrom;
    uint32_t vw[2], kw1 = 0, sk1 = 0, sv1 = 0;
#pragma unroll
    for (int n = 0; n < 2; ++n)
      vw[n] = *reinterpret_cast<const uint32_t*>(vc + at * (D / 2) + v_word<D>(p.slot >> 1, 2 * t + n, b));
    if (p.both) kw1 = *reinterpret_cast<const uint32_t*>(kfrom + D / 2), sk1 = ksfrom[D / 32], sv1 = vsfrom[1];
    uint32_t h[4], pair[2][4];  // pair: the even key's element and the odd key's
    const int64_t k_to = tok * a.ldk + w * 8, v_to = tok * a.ldv + w * 8;
    e2m1x8_to_f16(kw, h);
    store8<TYPE>(k, k_to, h, e8m0_to_f32(sk));
#pragma unroll
    for (int n = 0; n < 2; ++n) e2m1x8_to_f16(vw[n], pair[n]);
    auto pick = [&](int key) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
        h[n] = __byte_perm(pair[n >> 1][2 * (n & 1)], pair[n >> 1][2 * (n & 1) + 1], key ? 0x7632 : 0x5410);
    };
    pick(odd);
    store8<TYPE>(v, v_to, h, e8m0_to_f32(sv));
    if (p.both) {
      pick(1);
      store8<TYPE>(v, v_to + a.ldv, h, e8m0_to_f32(sv1));
      e2m1x8_to_f16(kw1, h);
      store8<TYPE>(k, k_to + a.ldk, h, e8m0_to_f32(sk1));
    }
  }
}

moe_status check_tokens(const wd_kv4_cache* c, const void* k, const void* v, int32_t type,
                        int64_t ldk, int64_t ldv, int32_t T, const int32_t* table,
                        int32_t max_blocks, const int32_t* lens, const int32_t* cu, int32_t S,
                        const int32_t* err, bool f32_ok) {
  moe_status rc = check_kv4(c);
  if (rc != MOE_OK) return rc;
  if (T < 0 || S < 0 || max_blocks < 1 || (!cu && T != S))
    return refuse(MOE_ERR_SHAPE, "wd_kv4: need T, S >= 0, max_blocks >= 1, and T == S without cu_new");
  if (!half_type(type) && !(f32_ok && type == WD_F32))
    return refuse(MOE_ERR_UNSUPPORTED, "wd_kv4: k and v are BF16 or F16 (gather: F32 too)");
  const int64_t row = (int64_t)c->heads * c->dim;
  if (ldk < row || ldv < row) return refuse(MOE_ERR_SHAPE, "wd_kv4: ldk or ldv is shorter than a token");
  if (T == 0 || S == 0) return MOE_OK;
  if (!k || !v || !table || !lens)
    return refuse(MOE_ERR_NULL, "wd_kv4: k, v, block_table and seq_lens are required");
  if (!aligned(k, 16) || !aligned(v, 16) || ldk % 8 || ldv % 8 || !aligned(table, 4) ||
      !aligned(lens, 4) || !aligned(cu, 4) || !aligned(err, 4))
    return refuse(MOE_ERR_ALIGN, "wd_kv4: k and v need 16 bytes and strides % 8 == 0, the int32 arrays 4");
  if ((int64_t)T * row / 8 > 0x7FFFFFFFll * kThreads)
    return refuse(MOE_ERR_SHAPE, "wd_kv4: too many tokens for one call");
  return MOE_OK;
}

TokenArgs token_args(const wd_kv4_cache* c, int64_t ldk, int64_t ldv, int32_t T,
                     const int32_t* table, int32_t max_blocks, const int32_t* lens,
                     const int32_t* cu, int32_t S, int32_t* err) {
  const int piece = c->dim / 8, words = c->heads * piece;  // 8-element pieces of a head, of a token
  int h = 128 / piece < c->heads ? 128 / piece : c->heads;  // heads of a CTA
  while (c->heads % h) --h;
  const int chunk = h * piece;
  // tokens of a CTA: up to 8 pieces a thread, in whole waves of resident CTAs. (Powers of two up to 4
  // pieces: 15.6 us instead of 13.1 for 16 prompts of up to 2000, 8 heads of dim 64, with one token
  // a thread; 12.1 now.)
  const int64_t runs = (int64_t)T * (words / chunk), slots = (int64_t)sm_count() * kResident;
  const int most = 8 * kThreads / chunk < kMostPer ? 8 * kThreads / chunk : kMostPer;
  const int64_t waves = (runs + slots * most - 1) / (slots * most);
  const int64_t even = (runs + slots * waves - 1) / (slots * waves);
  const int per = even < 2 ? 2 : (int)even;
  return {table, lens, cu, err, ldk, ldv, T, S, max_blocks, c->pages, kv4_page_shift(c->page_size),
          c->heads, per, chunk};
}

// The grid: runs of tokens, and pieces of a token in chunks of whole heads.
dim3 token_grid(const TokenArgs& a, int words) {
  return dim3((unsigned)((a.T + a.per - 1) / a.per), (unsigned)(words / a.chunk));
}

template <int D>
moe_status append(const wd_kv4_cache* c, const void* k, const void* v, int32_t type,
                  const TokenArgs& a, cudaStream_t st) {
  const dim3 grid = token_grid(a, a.heads * (D / 8));
  const uint16_t *k16 = static_cast<const uint16_t*>(k), *v16 = static_cast<const uint16_t*>(v);
  if (type == WD_BF16)
    kv4_append_kernel<D, true><<<grid, kThreads, 0, st>>>(k16, v16, c->k_codes, c->k_scales,
                                                             c->v_codes, c->v_scales, a);
  else
    kv4_append_kernel<D, false><<<grid, kThreads, 0, st>>>(k16, v16, c->k_codes, c->k_scales,
                                                              c->v_codes, c->v_scales, a);
  return launched("wd_kv4_append launch");
}

template <int D>
moe_status gather(const wd_kv4_cache* c, void* k, void* v, int32_t type, const TokenArgs& a,
                  cudaStream_t st) {
  const dim3 grid = token_grid(a, a.heads * (D / 8));
  auto run = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, st>>>(k, v, c->k_codes, c->k_scales, c->v_codes, c->v_scales, a);
  };
  if (type == WD_F32)
    run(kv4_gather_kernel<D, WD_F32>);
  else if (type == WD_BF16)
    run(kv4_gather_kernel<D, WD_BF16>);
  else
    run(kv4_gather_kernel<D, WD_F16>);
  return launched("wd_kv4_gather launch");
}

}  // namespace

int kv4_page_shift(int page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

moe_status check_kv4(const wd_kv4_cache* c) {
  if (!c) return refuse(MOE_ERR_NULL, "wd_kv4: cache is required");
  if (wd_kv4_cache_bytes(c, WD_KV4_CODES) == 0)
    return refuse(MOE_ERR_SHAPE, "wd_kv4: need pages >= 1, page_size 16, 32, 64, 128 or 256, heads >= 1 "
                                 "and dim 64, 128 or 256");
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales)
    return refuse(MOE_ERR_NULL, "wd_kv4: the cache's four arrays are required");
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
      !aligned(c->v_scales, 16))
    return refuse(MOE_ERR_ALIGN, "wd_kv4: the cache's arrays need 16 bytes");
  return MOE_OK;
}

}  // namespace wd

extern "C" size_t wd_kv4_cache_bytes(const wd_kv4_cache* c, int which) {
  if (!c || c->pages < 1 || c->heads < 1 || c->heads > 65535) return 0;
  if (c->dim != 64 && c->dim != 128 && c->dim != 256) return 0;
  const int p = c->page_size;
  if (p != 16 && p != 32 && p != 64 && p != 128 && p != 256) return 0;
  const size_t tokens = (size_t)c->pages * c->heads * p;
  return which == WD_KV4_CODES    ? tokens * (c->dim / 2)
         : which == WD_KV4_SCALES ? tokens * (c->dim / 32)
                                  : 0;
}

extern "C" moe_status wd_kv4_append(const wd_kv4_cache* c, const void* k, const void* v,
                                    int32_t type, int64_t ldk, int64_t ldv, int32_t T,
                                    const int32_t* table, int32_t max_blocks,
                                    const int32_t* lens, const int32_t* cu, int32_t S,
                                    int32_t* err, void* stream) {
  using namespace wd;
  moe_status rc = check_tokens(c, k, v, type, ldk, ldv, T, table, max_blocks, lens, cu, S, err, false);
  if (rc != MOE_OK || T == 0 || S == 0) return rc;
  const TokenArgs a = token_args(c, ldk, ldv, T, table, max_blocks, lens, cu, S, err);
  cudaStream_t st = (cudaStream_t)stream;
  return c->dim == 64    ? append<64>(c, k, v, type, a, st)
         : c->dim == 128 ? append<128>(c, k, v, type, a, st)
                         : append<256>(c, k, v, type, a, st);
}

extern "C" moe_status wd_kv4_gather(const wd_kv4_cache* c, void* k, void* v, int32_t type,
                                    int64_t ldk, int64_t ldv, int32_t T, const int32_t* table,
                                    int32_t max_blocks, const int32_t* lens, const int32_t* cu,
                                    int32_t S, int32_t* err, void* stream) {
  using namespace wd;
  moe_status rc = check_tokens(c, k, v, type, ldk, ldv, T, table, max_blocks, lens, cu, S, err, true);
  if (rc != MOE_OK || T == 0 || S == 0) return rc;
  const TokenArgs a = token_args(c, ldk, ldv, T, table, max_blocks, lens, cu, S, err);
  cudaStream_t st = (cudaStream_t)stream;
  return c->dim == 64    ? gather<64>(c, k, v, type, a, st)
         : c->dim == 128 ? gather<128>(c, k, v, type, a, st)
                         : gather<256>(c, k, v, type, a, st);
}
