// Device code and host helpers shared by the operators around the MoE layer
// (wd_fp4.cu, wd_kv4.cu, wd_norm.cu): element types, the MXFP4 quantiser and
// the E2M1 decode.
#pragma once

#include <atomic>

#include "warp_decode_block.h"
#include "wd_device.cuh"

namespace wd {

inline bool valid_type(int32_t t) { return t == WD_F32 || t == WD_BF16 || t == WD_F16; }
inline bool half_type(int32_t t) { return t == WD_BF16 || t == WD_F16; }
inline int type_bytes(int32_t t) { return t == WD_F32 ? 4 : 2; }

inline moe_status refuse(moe_status rc, const char* why) {
  set_error_msg(why);
  return rc;
}

inline moe_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return MOE_OK;
  set_error(what, e);
  return MOE_ERR_CUDA;
}

// allow_smem once per device for a kernel's largest size (a call of the runtime takes as
// long as a small kernel): one of these per kernel, static beside its launch.
struct SmemOnce {
  std::atomic<uint64_t> done{0};  // a bit per device
  template <typename K>
  moe_status allow(K kernel, size_t most) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return allow_smem(kernel, most);
    const uint64_t bit = 1ull << dev;
    if (done.load(std::memory_order_acquire) & bit) return MOE_OK;
    const moe_status rc = allow_smem(kernel, most);
    if (rc == MOE_OK) done.fetch_or(bit, std::memory_order_release);
    return rc;
  }
};

namespace {  // device code: one copy per translation unit

__device__ __forceinline__ float half_lo(uint32_t v) {
  return __half2float(__ushort_as_half((unsigned short)(v & 0xFFFFu)));
}
__device__ __forceinline__ float half_hi(uint32_t v) {
  return __half2float(__ushort_as_half((unsigned short)(v >> 16)));
}

// Eight 16-bit elements (BF16, or F16) -> FP32.
template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = BF16 ? bf16_lo(w[i]) : half_lo(w[i]);
    f[2 * i + 1] = BF16 ? bf16_hi(w[i]) : half_hi(w[i]);
  }
}

// Two FP32 values rounded to a pair of BF16 or F16, a in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float load_elem(const void* p, int32_t type, int64_t i) {
  if (type == WD_F32) return __ldg(reinterpret_cast<const float*>(p) + i);
  const uint16_t h = __ldg(reinterpret_cast<const uint16_t*>(p) + i);
  return type == WD_BF16 ? __uint_as_float((uint32_t)h << 16) : __half2float(__ushort_as_half(h));
}

__device__ __forceinline__ void store_elem(void* p, int32_t type, int64_t i, float v) {
  if (type == WD_F32)
    reinterpret_cast<float*>(p)[i] = v;
  else if (type == WD_BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}

// ------------------------------------------------------------------ MXFP4 --

// The E8M0 code of a block whose largest magnitude is m (NaN and infinities
// count as infinity): the exponent of m less E2M1's own 2, clamped.
__device__ __forceinline__ uint32_t fp4_scale_code(float m) {
  const uint32_t bits = __float_as_uint(m);
  if (bits >= 0x7F800000u) return 255u;
  if (bits < 0x00800000u) return 0u;  // 0 and subnormals: below 2^-126
  const int e = (int)(bits >> 23) - 2;  // biased exponent of m / 4
  return (uint32_t)(e < 0 ? 0 : e);
}

// 2^(127 - s): what an element of a block with scale code s is multiplied by
// before rounding (exact; s = 254 never comes from an FP32 value).
__device__ __forceinline__ float fp4_unscale(uint32_t s) {
  return s >= 254u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// |v| with NaN counted as infinity, as bits (ordered as unsigned integers).
__device__ __forceinline__ uint32_t magnitude(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b > 0x7F800000u ? 0x7F800000u : b;
}

// Eight scaled values -> eight E2M1 codes (ties to even, saturating), element i
// in bits 4i .. 4i+3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Eight E2M1 codes -> four f16x2 words, exact: h[j] = elements 2j (low), 2j + 1.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// m16n8k16, f16 operands, FP32 sums:
// d += a * b, and d = a * b: operands in place, so no register is copied around the MMA.
__device__ __forceinline__ void mma_add(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

}  // namespace
}  // namespace wd
