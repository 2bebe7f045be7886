// The KV cache held in 4 bits (MXFP4): appending tokens and reading them back.
#include "wd_block.cuh"
#include "wd_kv4.cuh"

namespace wd {
namespace {

// ------------------------------------------------------- append and gather --
// One thread per 8 elements of one (token, head) of K and of V; the four
// threads of a 32-element block are neighbours, so a block's largest magnitude
// takes two shuffles. The sequence of a token is found by bisection in cu_new.

struct TokenArgs {
  const int32_t *table, *lens, *cu;
  int32_t* err;
  int64_t ldk, ldv;
  int32_t T, S, max_blocks;
  int32_t pages, page_shift, heads;
};

// The place of new token `tok`: page and slot in the page, and whether the tokens
// before and behind it are new ones of its sequence too. False for a token that is
// ignored (behind cu[S]) or left out (flagged).
struct Place {
  int page, slot;
  bool before, behind;
};
__device__ __forceinline__ bool place_of(const TokenArgs& a, int tok, Place& p) {
  int s = tok, first = tok, end = tok + 1;
  if (a.cu) {
    if (tok >= __ldg(a.cu + a.S) || tok < __ldg(a.cu)) return false;
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
  p.page = -1;
  if (len >= 0 && block < a.max_blocks) p.page = __ldg(a.table + (int64_t)s * a.max_blocks + block);
  p.slot = (int)(pos & ((1 << a.page_shift) - 1));
  if (p.page < 0 || p.page >= a.pages) {
    flag_invalid(a.err);
    return false;
  }
  return true;
}

template <int D>
__device__ __forceinline__ void item_of(int64_t i, int heads, int& tok, int& head, int& b, int& t) {
  const int w = (int)(i % (D / 8));
  const int64_t th = i / (D / 8);
  head = (int)(th % heads);
  tok = (int)(th / heads);
  b = w >> 2;
  t = w & 3;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const uint16_t* __restrict__ k, const uint16_t* __restrict__ v,
                      uint8_t* __restrict__ kc, uint8_t* __restrict__ ks, uint8_t* __restrict__ vc,
                      uint8_t* __restrict__ vs, const TokenArgs a, int64_t total) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;  // total % (D / 8) == 0: the four threads of a block leave together
  int tok, head, b, t;
  item_of<D>(i, a.heads, tok, head, b, t);
  const unsigned quad = 0xFu << (threadIdx.x & 28);
  Place p;
  if (!place_of(a, tok, p)) return;  // the same answer for the whole block
  const int e = head * D + 32 * b + 8 * t;
  const size_t at = ((size_t)p.page * a.heads + head) << a.page_shift;  // in tokens
  // scale code of a block, and its elements times 2^-scale (0 in a NaN block)
  auto scaled = [&](const uint16_t* src, float (&f)[8]) {
    unpack8<BF16>(ld_cached16(src + e), f);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, magnitude(f[j]));
    m = max(m, __shfl_xor_sync(quad, m, 1));
    m = max(m, __shfl_xor_sync(quad, m, 2));
    const uint32_t s = fp4_scale_code(__uint_as_float(m));
    const float u = fp4_unscale(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = s == 255u ? 0.0f : f[j] * u;
    return s;
  };
  float f[8];
  const uint32_t sk = scaled(k + tok * a.ldk, f);
  *reinterpret_cast<uint32_t*>(kc + at * (D / 2) + k_word<D>(p.slot, t, b)) = e2m1x8(f);
  if (t == 0) ks[at * (D / 32) + p.slot * (D / 32) + b] = (uint8_t)sk;

  // V: a byte holds an element of an even key and the next, so one thread writes both:
  // the even key's where both are new
  const bool odd = p.slot & 1;
  if (odd && p.before) return;
  float pair[2][8];
  const uint32_t sv = scaled(v + tok * a.ldv, f);
  uint32_t next = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    pair[0][j] = odd ? 0.0f : f[j];
    pair[1][j] = odd ? f[j] : 0.0f;
  }
  if (!odd && p.behind) next = scaled(v + (int64_t)(tok + 1) * a.ldv, pair[1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // elements 4h .. 4h + 3: g = 2t + h
    const float both[8] = {pair[0][4 * h],     pair[1][4 * h],     pair[0][4 * h + 1], pair[1][4 * h + 1],
                           pair[0][4 * h + 2], pair[1][4 * h + 2], pair[0][4 * h + 3], pair[1][4 * h + 3]};
    uint32_t* to = reinterpret_cast<uint32_t*>(vc + at * (D / 2) + v_word<D>(p.slot >> 1, 2 * t + h, b));
    const uint32_t w = e2m1x8(both);
    *to = odd ? (*to & 0x0F0F0F0Fu) | (w & 0xF0F0F0F0u) : w;  // an odd key alone joins the key before
  }
  if (t == 0) {
    uint8_t* to = vs + at * (D / 32) + v_scale<D>(p.slot, b);
    if (!odd && p.behind)
      *reinterpret_cast<uint16_t*>(to) = (uint16_t)(sv | next << 8);
    else
      *to = (uint8_t)sv;
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
                      const uint8_t* __restrict__ vs, const TokenArgs a, int64_t total) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= total) return;
  int tok, head, b, t;
  item_of<D>(i, a.heads, tok, head, b, t);
  Place p;
  if (!place_of(a, tok, p)) return;
  const int slot = p.slot;
  const size_t at = ((size_t)p.page * a.heads + head) << a.page_shift;
  const int e = head * D + 32 * b + 8 * t;
  uint32_t h[4];
  e2m1x8_to_f16(*reinterpret_cast<const uint32_t*>(kc + at * (D / 2) + k_word<D>(slot, t, b)), h);
  store8<TYPE>(k, tok * a.ldk + e, h, e8m0_to_f32(ks[at * (D / 32) + slot * (D / 32) + b]));
  uint32_t pair[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    e2m1x8_to_f16(*reinterpret_cast<const uint32_t*>(vc + at * (D / 2) + v_word<D>(slot >> 1, 2 * t + i, b)), pair[i]);
  const uint32_t pick = slot & 1 ? 0x7632 : 0x5410;  // the halves of an odd or an even key
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __byte_perm(pair[i >> 1][2 * (i & 1)], pair[i >> 1][2 * (i & 1) + 1], pick);
  store8<TYPE>(v, tok * a.ldv + e, h, e8m0_to_f32(vs[at * (D / 32) + v_scale<D>(slot, b)]));
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
  return {table, lens, cu, err, ldk, ldv, T, S, max_blocks, c->pages, kv4_page_shift(c->page_size),
          c->heads};
}

template <int D>
moe_status append(const wd_kv4_cache* c, const void* k, const void* v, int32_t type,
                  const TokenArgs& a, cudaStream_t st) {
  const int64_t total = (int64_t)a.T * a.heads * (D / 8);
  const unsigned grid = (unsigned)((total + kThreads - 1) / kThreads);
  const uint16_t *k16 = static_cast<const uint16_t*>(k), *v16 = static_cast<const uint16_t*>(v);
  if (type == WD_BF16)
    kv4_append_kernel<D, true><<<grid, kThreads, 0, st>>>(k16, v16, c->k_codes, c->k_scales,
                                                          c->v_codes, c->v_scales, a, total);
  else
    kv4_append_kernel<D, false><<<grid, kThreads, 0, st>>>(k16, v16, c->k_codes, c->k_scales,
                                                           c->v_codes, c->v_scales, a, total);
  return launched("wd_kv4_append launch");
}

template <int D>
moe_status gather(const wd_kv4_cache* c, void* k, void* v, int32_t type, const TokenArgs& a,
                  cudaStream_t st) {
  const int64_t total = (int64_t)a.T * a.heads * (D / 8);
  const unsigned grid = (unsigned)((total + kThreads - 1) / kThreads);
  auto run = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, st>>>(k, v, c->k_codes, c->k_scales, c->v_codes, c->v_scales, a,
                                      total);
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
