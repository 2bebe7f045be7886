// wd_kv4_attend_chunk: attention of several new tokens per sequence over the paged
// 4-bit cache, which holds them already.
//
// A warp takes one (token, query head): 32 keys at a time, a key per lane for its logit,
// then the dims over the lanes for the sum of values, with the running maximum and sum of
// the softmax between.
#include "wd_block.cuh"
#include "wd_kv4.cuh"

namespace wd {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

struct ChunkArgs {
  const uint8_t *kc, *ks, *vc, *vs;
  const uint16_t* q;
  const int32_t *table, *lens, *cu;
  uint16_t* out;
  float* lse;
  int32_t* err;
  int64_t ldq, ldo;
  int32_t T, S, max_blocks, pages, page_shift, heads, group, window;
  float scale;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_chunk_kernel(const ChunkArgs a) {
  __shared__ float s_q[kWarpsPerCta][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q_heads = a.heads * a.group;
  const int64_t row = (int64_t)blockIdx.x * kWarpsPerCta + warp;
  const int tok = (int)(row / q_heads), h = (int)(row % q_heads), kv = h / a.group;
  if (tok >= a.T) return;
  int s = tok, first = tok;
  if (a.cu) {
    if (tok >= __ldg(a.cu + a.S) || tok < __ldg(a.cu)) return;
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.cu + mid) <= tok)
        lo = mid;
      else
        hi = mid - 1;
    }
    s = lo;
    first = __ldg(a.cu + s);
  }
  const int len = __ldg(a.lens + s);
  const int64_t room = (int64_t)a.max_blocks << a.page_shift;
  int64_t end = len < 0 ? 0 : (int64_t)len + (tok - first) + 1;
  const int64_t begin = a.window && len >= 0 ? max((int64_t)0, end - a.window) : 0;
  if (len < 0 || end > room) {
    flag_invalid(a.err);
    end = min(end, room);
  }
  const uint16_t* q = a.q + (int64_t)tok * a.ldq + (int64_t)h * D;
  for (int i = lane; i < D; i += 32) s_q[warp][i] = load_elem(q, BF16 ? WD_BF16 : WD_F16, i);
  __syncwarp();
  float m = -INFINITY, l = 0.0f, acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.0f;
  const int mask = (1 << a.page_shift) - 1;
  for (int64_t k0 = begin; k0 < end; k0 += 32) {
    const int64_t key = k0 + lane;
    int page = -1;
    if (key < end) {
      page = __ldg(a.table + (int64_t)s * a.max_blocks + (key >> a.page_shift));
      if (page < 0 || page >= a.pages) flag_invalid(a.err), page = -1;
    }
    const int slot = (int)(key & mask);
    const int64_t at = page < 0 ? 0 : ((int64_t)page * a.heads + kv) << a.page_shift;
    float z = -INFINITY;
    if (page >= 0) {
      z = 0.0f;
      for (int b = 0; b < D / 32; ++b) {
        float part = 0.0f;
        for (int t = 0; t < 4; ++t) {
          uint32_t hx[4];
          e2m1x8_to_f16(__ldg(reinterpret_cast<const uint32_t*>(a.kc + at * (D / 2) + k_word<D>(slot, t, b))), hx);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            part = fmaf(half_lo(hx[j]), s_q[warp][32 * b + 8 * t + 2 * j], part);
            part = fmaf(half_hi(hx[j]), s_q[warp][32 * b + 8 * t + 2 * j + 1], part);
          }
        }
        z = fmaf(part, e8m0_to_f32(a.ks[at * (D / 32) + slot * (D / 32) + b]), z);
      }
      z *= a.scale;
    }
    float top = z;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const float to = fmaxf(m, top), base = to == -INFINITY ? 0.0f : to;
    const float f = expf(m - base), p = page >= 0 ? expf(z - base) : 0.0f;
    m = to;
    l *= f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= f;
    for (int j = 0; j < 32; ++j) {
      const float pj = __shfl_sync(kAll, p, j);
      const int page_j = __shfl_sync(kAll, page, j), slot_j = __shfl_sync(kAll, slot, j);
      const int64_t at_j = __shfl_sync(kAll, at, j);
      if (page_j < 0) continue;
      l += pj;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {  // element lane of block i: byte lane % 4 of word g = lane / 4
        const uint8_t c = a.vc[at_j * (D / 2) + v_word<D>(slot_j >> 1, lane >> 2, i) + (lane & 3)];
        uint32_t hx[4];
        e2m1x8_to_f16(slot_j & 1 ? c >> 4 : c & 15, hx);
        acc[i] = fmaf(pj * e8m0_to_f32(a.vs[at_j * (D / 32) + v_scale<D>(slot_j, i)]), half_lo(hx[0]), acc[i]);
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    store_elem(a.out, BF16 ? WD_BF16 : WD_F16, (int64_t)tok * a.ldo + (int64_t)h * D + 32 * i + lane, acc[i] * inv);
  if (a.lse && lane == 0) a.lse[(int64_t)tok * q_heads + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

}  // namespace
}  // namespace wd

extern "C" size_t wd_kv4_attend_chunk_workspace(const wd_kv4_cache* c, int32_t T, int32_t q_heads) {
  using namespace wd;
  if (!c || wd_kv4_cache_bytes(c, WD_KV4_CODES) == 0 || T < 0 || q_heads < 1 || q_heads % c->heads) return 0;
  return 16;
}

extern "C" moe_status wd_kv4_attend_chunk(const wd_kv4_cache* c, const void* q, int32_t type, int64_t ldq, int32_t T,
                                          int32_t q_heads, const int32_t* table, int32_t max_blocks, const int32_t* lens,
                                          const int32_t* cu, int32_t S, float scale, int32_t window, void* out, int64_t ldo,
                                          float* lse, void* workspace, size_t workspace_bytes, int32_t* err, void* stream) {
  using namespace wd;
  moe_status rc = check_kv4(c);
  if (rc != MOE_OK) return rc;
  if (T < 0 || S < 0 || q_heads < 1 || q_heads % c->heads || max_blocks < 1 || window < 0 || (!cu && T != S))
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend_chunk: need T, S >= 0, q_heads a multiple of heads, max_blocks >= 1, "
                                 "window >= 0, and T == S without cu_new");
  if (!half_type(type)) return refuse(MOE_ERR_UNSUPPORTED, "wd_kv4_attend_chunk: q and out are BF16 or F16");
  if (ldq < (int64_t)q_heads * c->dim || ldo < (int64_t)q_heads * c->dim)
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend_chunk: ldq or ldo is shorter than a token");
  if (T == 0 || S == 0) return MOE_OK;
  if (!q || !table || !lens || !out || !workspace)
    return refuse(MOE_ERR_NULL, "wd_kv4_attend_chunk: q, block_table, seq_lens, out and workspace are required");
  if (!aligned(q, 16) || ldq % 8 || !aligned(out, 16) || ldo % 8 || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(cu, 4) || !aligned(lse, 4) || !aligned(workspace, 16) || !aligned(err, 4))
    return refuse(MOE_ERR_ALIGN, "wd_kv4_attend_chunk: q, out and workspace need 16 bytes, strides % 8 == 0, the others 4");
  if (workspace_bytes < wd_kv4_attend_chunk_workspace(c, T, q_heads))
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend_chunk: workspace is smaller than wd_kv4_attend_chunk_workspace");
  constexpr int64_t kMost = 0x7FFFFFFF - 0xFFFF;
  if ((int64_t)max_blocks * c->page_size >= kMost || (int64_t)T * q_heads >= kMost)
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend_chunk: block_table's capacity, or T * q_heads, is too large");
  ChunkArgs a = {};
  a.kc = c->k_codes, a.ks = c->k_scales, a.vc = c->v_codes, a.vs = c->v_scales;
  a.q = static_cast<const uint16_t*>(q), a.out = static_cast<uint16_t*>(out), a.lse = lse, a.err = err;
  a.table = table, a.lens = lens, a.cu = cu;
  a.ldq = ldq, a.ldo = ldo, a.T = T, a.S = S, a.max_blocks = max_blocks, a.pages = c->pages;
  a.page_shift = kv4_page_shift(c->page_size), a.heads = c->heads, a.group = q_heads / c->heads, a.window = window;
  a.scale = scale;
  cudaStream_t st = (cudaStream_t)stream;
  const unsigned grid = (unsigned)(((int64_t)T * q_heads + kWarpsPerCta - 1) / kWarpsPerCta);
  auto run = [&](auto kernel) { kernel<<<grid, kThreads, 0, st>>>(a); };
  const bool bf16 = type == WD_BF16;
  if (c->dim == 64)
    bf16 ? run(kv4_chunk_kernel<64, true>) : run(kv4_chunk_kernel<64, false>);
  else if (c->dim == 128)
    bf16 ? run(kv4_chunk_kernel<128, true>) : run(kv4_chunk_kernel<128, false>);
  else
    bf16 ? run(kv4_chunk_kernel<256, true>) : run(kv4_chunk_kernel<256, false>);
  return launched("wd_kv4_attend_chunk launch");
}
