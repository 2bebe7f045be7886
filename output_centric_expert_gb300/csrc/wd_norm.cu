// wd_block_norm: one CTA per token, the row in registers between its passes.
#include "wd_block.cuh"

namespace wd {
namespace {

constexpr int kNormMaxH = 8192;
constexpr int kNormPer = kNormMaxH / kThreads;  // channels per thread at most

struct NormArgs {
  const void *res, *y, *w_post, *w_pre, *gate;
  void *res_out, *out;
  int64_t ldr, ldy, gate_ld, ldro, ldo;
  int32_t H, res_type, y_type, w_type, out_type, gate_step;
  float res_scale, eps;
};

// Sum over the CTA, the same in every thread.
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int i = 1; i < kWarpsPerCta; ++i) s += red[i];
  return s;
}

__global__ void __launch_bounds__(kThreads) block_norm_kernel(const NormArgs a) {
  __shared__ float red[kWarpsPerCta];
  const int64_t tok = blockIdx.x;
  float r[kNormPer], n[kNormPer];
#pragma unroll
  for (int i = 0; i < kNormPer; ++i) {
    const int c = threadIdx.x + i * kThreads;
    r[i] = c < a.H ? a.res_scale * load_elem(a.res, a.res_type, tok * a.ldr + c) : 0.0f;
    n[i] = c < a.H && a.y ? load_elem(a.y, a.y_type, tok * a.ldy + c) : 0.0f;
  }
  if (a.y) {
    float inv = 1.0f;
    if (a.w_post) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < kNormPer; ++i) s = fmaf(n[i], n[i], s);
      inv = rsqrtf(cta_sum(s, red) / (float)a.H + a.eps);
    }
#pragma unroll
    for (int i = 0; i < kNormPer; ++i) {
      const int c = threadIdx.x + i * kThreads;
      if (c >= a.H) continue;
      float v = n[i];
      if (a.w_post) v = v * inv * load_elem(a.w_post, a.w_type, c);
      if (a.gate) v *= load_elem(a.gate, a.w_type, tok * a.gate_ld + (int64_t)c * a.gate_step);
      r[i] += v;
    }
  }
  if (a.res_out) {
#pragma unroll
    for (int i = 0; i < kNormPer; ++i) {
      const int c = threadIdx.x + i * kThreads;
      if (c < a.H) store_elem(a.res_out, a.res_type, tok * a.ldro + c, r[i]);
    }
  }
  if (a.out) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormPer; ++i) s = fmaf(r[i], r[i], s);
    const float inv = rsqrtf(cta_sum(s, red) / (float)a.H + a.eps);
#pragma unroll
    for (int i = 0; i < kNormPer; ++i) {
      const int c = threadIdx.x + i * kThreads;
      if (c < a.H)
        store_elem(a.out, a.out_type, tok * a.ldo + c, r[i] * inv * load_elem(a.w_pre, a.w_type, c));
    }
  }
}

}  // namespace
}  // namespace wd

extern "C" moe_status wd_block_norm(int32_t T, int32_t H, const void* res, int32_t res_type,
                                    int64_t ldr, const void* y, int32_t y_type, int64_t ldy,
                                    const void* w_post, const void* w_pre, const void* gate,
                                    int32_t w_type, int64_t gate_ld, int32_t gate_step,
                                    float res_scale, float eps, void* res_out, int64_t ldro,
                                    void* out, int32_t out_type, int64_t ldo, void* stream) {
  using namespace wd;
  if (T < 0 || H < 1 || H > kNormMaxH)
    return refuse(MOE_ERR_SHAPE, "wd_block_norm: need T >= 0 and 1 <= H <= 8192");
  if (!valid_type(res_type) || !valid_type(y_type) || !valid_type(w_type) || !valid_type(out_type))
    return refuse(MOE_ERR_UNSUPPORTED, "wd_block_norm: types are F32, BF16 or F16");
  if (ldr < H || (y && ldy < H) || (res_out && ldro < H) || (out && ldo < H) || gate_ld < 0 ||
      gate_step < 0 || gate_step > 1)
    return refuse(MOE_ERR_SHAPE, "wd_block_norm: a stride is shorter than a row, or gate_step is not 0 or 1");
  if (T == 0) return MOE_OK;
  if (!res || (!w_pre != !out) || (!res_out && !out) || (!y && (w_post || gate)))
    return refuse(MOE_ERR_NULL, "wd_block_norm: needs res, out with w_pre, an output, and y for w_post and gate");
  if (!aligned(res, type_bytes(res_type)) || !aligned(y, type_bytes(y_type)) ||
      !aligned(w_post, type_bytes(w_type)) || !aligned(w_pre, type_bytes(w_type)) ||
      !aligned(gate, type_bytes(w_type)) || !aligned(res_out, type_bytes(res_type)) ||
      !aligned(out, type_bytes(out_type)))
    return refuse(MOE_ERR_ALIGN, "wd_block_norm: a pointer is not aligned to its type");
  const NormArgs a = {res, y, w_post, w_pre, gate, res_out, out, ldr, ldy, gate_ld, ldro, ldo,
                      H, res_type, y_type, w_type, out_type, gate_step, res_scale, eps};
  block_norm_kernel<<<(unsigned)T, kThreads, 0, (cudaStream_t)stream>>>(a);
  return launched("wd_block_norm launch");
}
