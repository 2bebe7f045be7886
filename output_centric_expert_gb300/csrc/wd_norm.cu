// wd_block_norm: the norms, gate and residual between two blocks.
//
// The row stays in registers between its two sums: 8 channels per thread, so a
// row is one warp (H <= 256) or one CTA of H / 8 threads, up to 1024. DRAM traffic
// is each input read and each output written once. CTAs stay resident and walk
// the rows: the weights (and a gate that all tokens share) are read once per CTA
// into registers instead of once per row from L2, and the next row's loads are
// in flight while this one is summed.
// Loads of different arrays must not wait for one another (a token's latency is
// one trip to memory, not four): they are issued as raw words under a branch on
// the type, and converted after.
//   Bound by DRAM for many rows: 8192 tokens of 4096 BF16 channels (268 MB) 42.9 us,
// 6.3 TB/s, 92 % of a copy (47.4 with a division in each sum's use); one token 2.7 us, a
// launch and one trip to memory. A width of 7167 goes channel by channel: 33 tokens 4.8
// us, most of it that trip and two sums; 4000 tokens 88 us, 2.6 TB/s: instructions, of
// one row per SM at a time. (Rows ahead through shared memory at their own alignment, or
// in registers: 2 to 5 % less for it, 8 to 20 % more for narrower ones.)
#include <type_traits>

#include "wd_block.cuh"

namespace wd {
namespace {

constexpr int kNormMaxH = 8192;
constexpr int kNormPer = 8;  // channels per thread
constexpr size_t kStaticSmem = 512;  // more than the kernels' static shared memory

struct NormArgs {
  const void *res, *y, *w_post, *w_pre, *gate;
  void *res_out, *out;
  int64_t ldr, ldy, gate_ld, ldro, ldo;
  int32_t T, H, res_type, y_type, w_type, out_type, gate_step;
  float res_scale, eps;
};

// A thread's 8 channels of a row: VEC: 8 * i .. 8 * i + 7 as one or two 16-byte
// words; else i + k * n for n threads in the row.
struct Raw {
  uint32_t w[8];
};

// Whether a thread's k-th channel on the element path is inside the row, which has more
// than 4 N channels where N is the least that holds it.
template <int N>
__device__ __forceinline__ bool has(int i, int k, int H) {
  return (N >= 64 && k < 4) || i + k * N < H;
}

// N: threads of the row, a constant on the element path so that strides are immediates.
template <bool VEC, int N>
__device__ __forceinline__ void load_raw(const void* p, int32_t type, int64_t row, int i, int H,
                                         Raw& r) {
  if (VEC) {
    if (i * 8 < H) {
      const char* a = static_cast<const char*>(p) + (row + i * 8) * (type == WD_F32 ? 4 : 2);
      asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                   : "l"(a));
      if (type == WD_F32)
        asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                     : "l"(a + 16));
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) r.w[k] = 0;
    }
  } else if (type == WD_F32) {
    const uint32_t* a = static_cast<const uint32_t*>(p) + row + i;
#pragma unroll
    for (int k = 0; k < 8; ++k) r.w[k] = has<N>(i, k, H) ? a[k * N] : 0u;
  } else {
    const uint16_t* a = static_cast<const uint16_t*>(p) + row + i;
#pragma unroll
    for (int k = 0; k < 8; ++k) r.w[k] = has<N>(i, k, H) ? a[k * N] : 0u;
  }
}

template <bool VEC>
__device__ __forceinline__ void convert(const Raw& r, int32_t type, float (&f)[8]) {
  if (type == WD_F32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(r.w[k]);
  } else if (type == WD_BF16) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      f[k] = !VEC ? __uint_as_float(r.w[k] << 16) : (k & 1) ? bf16_hi(r.w[k / 2]) : bf16_lo(r.w[k / 2]);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      f[k] = !VEC ? half_lo(r.w[k]) : (k & 1) ? half_hi(r.w[k / 2]) : half_lo(r.w[k / 2]);
  }
}

template <bool VEC, int N>
__device__ __forceinline__ void store_row(void* p, int32_t type, int64_t row, int i, int H,
                                          const float (&f)[8]) {
  if (VEC) {
    if (i * 8 >= H) return;
    char* a = static_cast<char*>(p) + (row + i * 8) * (type == WD_F32 ? 4 : 2);
    if (type == WD_F32) {
      reinterpret_cast<float4*>(a)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(a)[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else if (type == WD_BF16) {
      *reinterpret_cast<uint4*>(a) = make_uint4(pack2<true>(f[0], f[1]), pack2<true>(f[2], f[3]),
                                                pack2<true>(f[4], f[5]), pack2<true>(f[6], f[7]));
    } else {
      *reinterpret_cast<uint4*>(a) = make_uint4(pack2<false>(f[0], f[1]), pack2<false>(f[2], f[3]),
                                                pack2<false>(f[4], f[5]), pack2<false>(f[6], f[7]));
    }
  } else if (type == WD_F32) {
    float* a = static_cast<float*>(p) + row + i;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (has<N>(i, k, H)) a[k * N] = f[k];
  } else {
    uint16_t* a = static_cast<uint16_t*>(p) + row + i;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (has<N>(i, k, H))
        a[k * N] = (uint16_t)(type == WD_BF16 ? pack2<true>(f[k], 0.0f) : pack2<false>(f[k], 0.0f));
  }
}

// Sum over the row's threads, the same in each: a warp's butterfly, then the
// warps' sums through shared memory (two slots in turn: one barrier per sum).
template <bool WARP>
__device__ __forceinline__ float row_sum(const float (&f)[8], float (*red)[32], int& slot) {
  float v = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) v = fmaf(f[k], f[k], v);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  if (WARP) return v;
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) red[slot][threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? red[slot][lane] : 0.0f;
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  slot ^= 1;
  return v;
}

__device__ __forceinline__ void copy16(uint32_t to, const char* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Rows in flight of the vector path: 1024 threads times these are 128 to 192 KB
// of an SM's shared memory.
__host__ __device__ constexpr int row_depth(int rt, int yt) { return rt == WD_F32 || yt == WD_F32 ? 3 : 4; }
__host__ __device__ constexpr int elem_bytes(int type) { return type == WD_F32 ? 4 : 2; }

// RT, YT: the types of res and y (-1: looked up at run time, on the element path
// of odd widths and strides).
// ROWS: the gate has a value per token and channel.
// N: threads of a row on the element path; 32: a warp per row, else a CTA per row.
// The vector path copies its rows ahead with cp.async; a thread reads only what it
// has copied itself, so the copies need no barrier.
template <int RT, int YT, bool VEC, bool ROWS, int N>
__global__ void __launch_bounds__(N == 32 ? kThreads : VEC ? 1024 : N, N == 32 ? 1024 / kThreads : VEC ? 1 : 1024 / N)
    block_norm_kernel(const NormArgs a) {
  constexpr bool WARP = N == 32;
  constexpr int DEPTH = VEC ? row_depth(RT, YT) : 1;
  constexpr int RB = VEC ? elem_bytes(RT) / 2 : 0, YB = VEC ? elem_bytes(YT) / 2 : 0;  // 16-byte words
  extern __shared__ uint4 dyn4[];
  __shared__ float red[2][32];
  const int i = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int per = WARP ? blockDim.x >> 5 : 1;       // rows of a CTA at a time
  const uint32_t step = gridDim.x * per, T = a.T;  // (unsigned: the last row and a step may pass 2^31)
  uint32_t tok = blockIdx.x * per + (WARP ? threadIdx.x >> 5 : 0);
  int slot = 0;
  const int rt = RT >= 0 ? RT : a.res_type, yt = YT >= 0 ? YT : a.y_type;
  const bool own_gate = a.gate && a.gate_ld != 0;  // a gate row or value per token
  const bool inside = VEC && i * 8 < a.H;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(dyn4) + threadIdx.x * 16;
  const uint32_t word = blockDim.x * 16;  // between a thread's 16-byte words

  auto ahead = [&](int64_t t, int stage) {
    if (inside && t < a.T) {
      const char* r = static_cast<const char*>(a.res) + (t * a.ldr + i * 8) * (RB * 2);
      const char* y = static_cast<const char*>(a.y) + (t * a.ldy + i * 8) * (YB * 2);
#pragma unroll
      for (int w = 0; w < RB; ++w) copy16(ring + (stage * (RB + YB) + w) * word, r + 16 * w);
      if (a.y)
#pragma unroll
        for (int w = 0; w < YB; ++w) copy16(ring + (stage * (RB + YB) + RB + w) * word, y + 16 * w);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (VEC)
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d) ahead(tok + (int64_t)d * step, d);

  float post[8], pre[8];
  {
    Raw wp, wq, sg;
    if (a.w_post) load_raw<VEC, N>(a.w_post, a.w_type, 0, i, a.H, wp);
    if (a.w_pre) load_raw<VEC, N>(a.w_pre, a.w_type, 0, i, a.H, wq);
    if (a.gate && !own_gate && a.gate_step) load_raw<VEC, N>(a.gate, a.w_type, 0, i, a.H, sg);
    if (a.w_pre) convert<VEC>(wq, a.w_type, pre);
    if (a.w_post) {
      convert<VEC>(wp, a.w_type, post);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) post[k] = 1.0f;
    }
    if (a.gate && !own_gate) {  // a gate that all tokens share belongs to the weights
      float g[8];
      if (a.gate_step) {
        convert<VEC>(sg, a.w_type, g);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = load_elem(a.gate, a.w_type, 0);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) post[k] *= g[k];
    }
  }

  const float per_channel = 1.0f / (float)a.H;
  for (int stage = 0; tok < T; tok += step, stage = stage + 1 == DEPTH ? 0 : stage + 1) {
    float y[8], r[8];
    Raw rg;
    float g1 = 1.0f;
    if (ROWS)
      load_raw<VEC, N>(a.gate, a.w_type, tok * a.gate_ld, i, a.H, rg);
    else if (own_gate)
      g1 = load_elem(a.gate, a.w_type, tok * a.gate_ld);
    {
      Raw rr = {}, ry = {};
      if (VEC) {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH >= 2 ? DEPTH - 2 : 0) : "memory");
        const uint4* own = dyn4 + threadIdx.x + (size_t)stage * (RB + YB) * blockDim.x;
        auto take = [&](Raw& raw, int first, int words) {
#pragma unroll
          for (int w = 0; w < 2; ++w)
            if (w < words) {
              const uint4 v = own[(size_t)(first + w) * blockDim.x];
              raw.w[4 * w] = v.x, raw.w[4 * w + 1] = v.y, raw.w[4 * w + 2] = v.z, raw.w[4 * w + 3] = v.w;
            }
        };
        if (inside) {
          take(rr, 0, RB);
          if (a.y) take(ry, RB, YB);
        }
        ahead(tok + (int64_t)(DEPTH - 1) * step, stage == 0 ? DEPTH - 1 : stage - 1);
      } else {
        load_raw<VEC, N>(a.res, rt, tok * a.ldr, i, a.H, rr);
        if (a.y) load_raw<VEC, N>(a.y, yt, tok * a.ldy, i, a.H, ry);
      }
      convert<VEC>(rr, rt, r);
      if (a.y) convert<VEC>(ry, yt, y);
    }
    if (a.y) {
      float inv = g1;
      if (a.w_post) inv *= rsqrtf(row_sum<WARP>(y, red, slot) * per_channel + a.eps);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= post[k];
      if (ROWS) {
        float g[8];
        convert<VEC>(rg, a.w_type, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] *= g[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] = fmaf(y[k], inv, r[k] * a.res_scale);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] *= a.res_scale;
    }
    if (a.res_out) store_row<VEC, N>(a.res_out, rt, tok * a.ldro, i, a.H, r);
    if (a.out) {
      const float inv = rsqrtf(row_sum<WARP>(r, red, slot) * per_channel + a.eps);
#pragma unroll
      for (int k = 0; k < 8; ++k) r[k] = r[k] * inv * pre[k];
      store_row<VEC, N>(a.out, a.out_type, tok * a.ldo, i, a.H, r);
    }
  }
  if (VEC) asm volatile("cp.async.wait_all;" ::: "memory");
}

// Whether a row of this array can be read 8 channels at a time.
bool vector_rows(const void* p, int32_t type, int64_t ld) {
  return !p || (aligned(p, 16) && ld * type_bytes(type) % 16 == 0);
}

template <int RT, int YT, bool VEC, int N>
moe_status launch_norm(const NormArgs& a, cudaStream_t st) {
  const bool rows_gate = a.gate && a.gate_ld != 0 && a.gate_step != 0;
  auto k = rows_gate ? block_norm_kernel<RT, YT, VEC, true, N> : block_norm_kernel<RT, YT, VEC, false, N>;
  const int rows = N == 32 ? kWarpsPerCta : 1;
  const int threads = N == 32 ? kThreads : VEC ? ((a.H + 7) / 8 + 31) / 32 * 32 : N;
  const size_t smem = VEC ? (size_t)threads * row_depth(RT, YT) * 8 * (elem_bytes(RT) + elem_bytes(YT)) : 0;
  static SmemOnce once[2];
  const moe_status rc = VEC ? once[rows_gate].allow(k, kMaxDynSmem - kStaticSmem) : MOE_OK;
  if (rc != MOE_OK) return rc;
  // resident CTAs: 64 registers a thread at most, so 1024 threads fill an SM
  const int64_t most = (int64_t)sm_count() * (1024 / threads);
  const int64_t want = ((int64_t)a.T + rows - 1) / rows;
  k<<<(unsigned)(want < most ? want : most), threads, smem, st>>>(a);
  return launched("wd_block_norm launch");
}

template <int N>
moe_status launch_vector(const NormArgs& a, cudaStream_t st) {
  auto with_y = [&](auto rt) {
    constexpr int R = decltype(rt)::value;
    return a.y_type == WD_F32    ? launch_norm<R, WD_F32, true, N>(a, st)
           : a.y_type == WD_BF16 ? launch_norm<R, WD_BF16, true, N>(a, st)
                                 : launch_norm<R, WD_F16, true, N>(a, st);
  };
  return a.res_type == WD_F32    ? with_y(std::integral_constant<int, WD_F32>())
         : a.res_type == WD_BF16 ? with_y(std::integral_constant<int, WD_BF16>())
                                 : with_y(std::integral_constant<int, WD_F16>());
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
  const NormArgs a = {res, y, w_post, w_pre, gate, res_out, out, ldr, ldy, gate_ld, ldro, ldo, T, H,
                      res_type, y_type, w_type, out_type, gate_step, res_scale, eps};
  // vectors need every row (and the weights) on a 16-byte boundary; a width that
  // is no multiple of 8, or any odd stride, goes one channel at a time
  const bool vec = H % 8 == 0 && vector_rows(res, res_type, ldr) && vector_rows(y, y_type, ldy) &&
                   vector_rows(res_out, res_type, ldro) && vector_rows(out, out_type, ldo) &&
                   vector_rows(w_post, w_type, 0) && vector_rows(w_pre, w_type, 0) &&
                   (gate_step == 0 || vector_rows(gate, w_type, gate_ld));
  cudaStream_t st = (cudaStream_t)stream;
  if (vec) return H <= 32 * kNormPer ? launch_vector<32>(a, st) : launch_vector<1024>(a, st);
  // As few threads as hold the row: more rows of an SM overlap, each waiting for its loads and sums. 8000
  // rows of 511, 1001, 4095 channels: 10.5, 19.9, 70.8 us; with 256 threads for up to 2048 and 1024 above
  // three times, 1.7 times and twice that.
  return H <= 32 * kNormPer    ? launch_norm<-1, -1, false, 32>(a, st)
         : H <= 64 * kNormPer  ? launch_norm<-1, -1, false, 64>(a, st)
         : H <= 128 * kNormPer ? launch_norm<-1, -1, false, 128>(a, st)
         : H <= 256 * kNormPer ? launch_norm<-1, -1, false, 256>(a, st)
         : H <= 512 * kNormPer ? launch_norm<-1, -1, false, 512>(a, st)
                               : launch_norm<-1, -1, false, 1024>(a, st);
}
