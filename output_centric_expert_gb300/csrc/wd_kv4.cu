// The KV cache held in 4 bits (MXFP4): appending tokens and reading them back.
#include "wd_block.cuh"
#include "wd_kv4.cuh"

namespace wd {
namespace {

// ------------------------------------------------------- append and gather --
// A CTA takes `per` tokens in a row and up to 128 of their 8-element pieces. Its first
// threads find the tokens' places (sequence by bisection in cu_new, page, slot) once
// for all. The four threads of a 32-element block are neighbours: its largest magnitude
// takes two shuffles. Both kernels are bound by integer instructions (conversions,
// packing, addresses), so magnitudes are compared as 16-bit pairs and a thread steps
// through its pieces without divisions. Prompts of 9.7k tokens, 8 heads of dim 128, into
// the cache and back (100 MB): 27.4 us, 3.7 TB/s; ALU 55 % busy, DRAM 27 %, 68 % of the
// issue slots in larger batches. One token each of 64 sequences: 3.7 us a launch.

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
constexpr int kMostPer = 64;
constexpr int kResident = 6;  // CTAs of an SM: both loads of a thread in flight take 39 registers

__device__ __forceinline__ Place place_of(const TokenArgs& a, int tok, bool flag) {
  Place p = {-1, 0, false, false};
  int s = tok, first = tok, end = tok + 1;
  if (tok >= a.T) return p;
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
    if (flag) flag_invalid(a.err);
  }
  return p;
}

// The (token, piece) of a thread's i-th item, i = threadIdx.x, + kThreads, ...
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
  __shared__ Place s_place[kMostPer + 1];
  extern __shared__ uint32_t s_code[];  // V's codes: [per + 1 tokens][chunk]; scale codes behind
  uint8_t* s_scale = reinterpret_cast<uint8_t*>(s_code + (a.per + 1) * a.chunk);
  const int tok0 = blockIdx.x * a.per, w0 = blockIdx.y * a.chunk, tid = threadIdx.x;
  if (tid <= a.per) s_place[tid] = place_of(a, tok0 + tid, tid < a.per);
  __syncthreads();
  // the scale code of a piece's block, and its codes
  auto quantise = [&](const uint4& raw, unsigned quad, uint32_t& scale) {
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
  const unsigned quad = 0xFu << (tid & 28);
  // the token behind the last may share bytes with it
  for (Walk walk(a.chunk); walk.j <= a.per; walk.next()) {
    const int i = walk.i, j = walk.j, w = w0 + walk.w;
    const Place p = s_place[j];
    if (p.page < 0) continue;  // the four threads of a block alike
    const int head = w / (D / 8), b = w % (D / 8) >> 2, t = w & 3;
    const int64_t tok = tok0 + j;
    const uint4 raw_v = ld_cached16(v + tok * a.ldv + w * 8);
    uint4 raw_k;
    if (j < a.per) raw_k = ld_cached16(k + tok * a.ldk + w * 8);
    uint32_t sv;
    s_code[i] = quantise(raw_v, quad, sv);
    if (t == 0) s_scale[i >> 2] = (uint8_t)sv;
    if (j == a.per) continue;
    uint32_t sk;
    const uint32_t code = quantise(raw_k, quad, sk);
    const size_t at = ((size_t)p.page * a.heads + head) << a.page_shift;  // in tokens
    *reinterpret_cast<uint32_t*>(kc + at * (D / 2) + k_word<D>(p.slot, t, b)) = code;
    if (t == 0) ks[at * (D / 32) + p.slot * (D / 32) + b] = (uint8_t)sk;
  }
  __syncthreads();
  // V: a byte holds an element of an even key and the next, so one thread writes both:
  // the even key's where both are new
  for (Walk walk(a.chunk); walk.j < a.per; walk.next()) {
    const int i = walk.i, j = walk.j, w = w0 + walk.w;
    const Place p = s_place[j];
    const bool odd = p.slot & 1;
    if (p.page < 0 || (odd && p.before)) continue;
    const int head = w / (D / 8), b = w % (D / 8) >> 2, t = w & 3;
    const size_t at = ((size_t)p.page * a.heads + head) << a.page_shift;
    const bool both = !odd && p.behind;
    const uint32_t even = odd ? 0u : s_code[i], next = odd ? s_code[i] : both ? s_code[i + a.chunk] : 0u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // elements 4h .. 4h + 3: g = 2t + h
      uint32_t* to = reinterpret_cast<uint32_t*>(vc + at * (D / 2) + v_word<D>(p.slot >> 1, 2 * t + h, b));
      const uint32_t x = spread4(even >> (16 * h)) | spread4(next >> (16 * h)) << 4;
      *to = odd ? (*to & 0x0F0F0F0Fu) | x : x;  // an odd key alone joins the key before
    }
    if (t == 0) {
      uint8_t* to = vs + at * (D / 32) + v_scale<D>(p.slot, b);
      if (both)
        *reinterpret_cast<uint16_t*>(to) = (uint16_t)(s_scale[i >> 2] | s_scale[(i + a.chunk) >> 2] << 8);
      else
        *to = s_scale[i >> 2];
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
  __shared__ Place s_place[kMostPer];
  const int tok0 = blockIdx.x * a.per, w0 = blockIdx.y * a.chunk, tid = threadIdx.x;
  if (tid < a.per) s_place[tid] = place_of(a, tok0 + tid, true);
  __syncthreads();
  for (Walk walk(a.chunk); walk.j < a.per; walk.next()) {
    const int j = walk.j, w = w0 + walk.w;
    const Place p = s_place[j];
    if (p.page < 0) continue;
    const int head = w / (D / 8), b = w % (D / 8) >> 2, t = w & 3, slot = p.slot;
    const int64_t tok = tok0 + j;
    const size_t at = ((size_t)p.page * a.heads + head) << a.page_shift;
    uint32_t h[4], pair[2][4];
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(kc + at * (D / 2) + k_word<D>(slot, t, b));
    uint32_t vw[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
      vw[n] = *reinterpret_cast<const uint32_t*>(vc + at * (D / 2) + v_word<D>(slot >> 1, 2 * t + n, b));
    const uint32_t sk = ks[at * (D / 32) + slot * (D / 32) + b], sv = vs[at * (D / 32) + v_scale<D>(slot, b)];
    e2m1x8_to_f16(kw, h);
    store8<TYPE>(k, tok * a.ldk + w * 8, h, e8m0_to_f32(sk));
    const uint32_t pick = slot & 1 ? 0x7632 : 0x5410;  // the halves of an odd or an even key
#pragma unroll
    for (int n = 0; n < 2; ++n) e2m1x8_to_f16(vw[n], pair[n]);
#pragma unroll
    for (int n = 0; n < 4; ++n) h[n] = __byte_perm(pair[n >> 1][2 * (n & 1)], pair[n >> 1][2 * (n & 1) + 1], pick);
    store8<TYPE>(v, tok * a.ldv + w * 8, h, e8m0_to_f32(sv));
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
  // pieces: 15.6 us instead of 13.1 for 16 prompts of up to 2000, 8 heads of dim 64.)
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
  const size_t smem = (size_t)(a.per + 1) * a.chunk * 4 + (size_t)(a.per + 1) * a.chunk / 4;
  const uint16_t *k16 = static_cast<const uint16_t*>(k), *v16 = static_cast<const uint16_t*>(v);
  if (type == WD_BF16)
    kv4_append_kernel<D, true><<<grid, kThreads, smem, st>>>(k16, v16, c->k_codes, c->k_scales,
                                                             c->v_codes, c->v_scales, a);
  else
    kv4_append_kernel<D, false><<<grid, kThreads, smem, st>>>(k16, v16, c->k_codes, c->k_scales,
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
