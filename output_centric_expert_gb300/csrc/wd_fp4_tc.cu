// wd_fp4_matvec for more than 8 tokens: the fifth-generation tensor cores, with the
// weights decoded into tensor memory.
//
//   tcgen05.mma kind::f16, M = 128 output rows, N = 16, 32 or 64 tokens, K = 16:
//   A is the decoded weights in tensor memory, B the tokens in shared memory, D the
//   FP32 sums in tensor memory. (mma.sync takes 2 cycles of an SM for 16 x 8 x 16, an
//   eighth of this rate: 64 tokens of a 9216 x 4096 matrix spent 14 us in it.)
//
// Scales. The sums run over all of a CTA's columns inside the tensor core, so a
// block's scale has to be in A: the decoded value times 2^(s - top + 12), with top the
// largest scale code of the row among the CTA's columns. Exact in f16 for blocks
// down to 2^-26 of the row's largest scale; smaller ones add nothing (less than FP32
// rounding of the row's largest products). The row's 2^top comes back at the end.
//
// Work. A cluster of CTAs shares a run of 128-row tiles, each CTA with its share of the
// columns, so that it stages and converts only that share of x (64 tokens of 1024
// columns are 128 KB). In a CTA each of two warpgroups takes a row tile: a thread
// decodes a row, 128 columns at a time, stores them to tensor memory, and one thread
// issues the eight MMAs while all decode the next columns. The CTAs add their sums
// in column order through distributed shared memory.
#include <cooperative_groups.h>

#include <mutex>

#include "wd_block.cuh"
#include "wd_fp4.h"

namespace wd {
namespace {

namespace cg = cooperative_groups;

constexpr int kTcThreads = 256, kGroups = 2;  // warpgroups
constexpr int kTcRows = 128;
constexpr int kTcAhead = 3;         // column tiles of codes in flight per row
constexpr int kTmemCols = 256;      // per warpgroup: 64 for A, up to 64 for D
constexpr int kStageX = 128 * 1024; // bytes of x per CTA at most
constexpr uint32_t kWaitLimit = 1u << 22;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[64], int o) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]),
      "r"(r[o + 7]), "r"(r[o + 8]), "r"(r[o + 9]), "r"(r[o + 10]), "r"(r[o + 11]), "r"(r[o + 12]),
      "r"(r[o + 13]), "r"(r[o + 14]), "r"(r[o + 15]), "r"(r[o + 16]), "r"(r[o + 17]), "r"(r[o + 18]),
      "r"(r[o + 19]), "r"(r[o + 20]), "r"(r[o + 21]), "r"(r[o + 22]), "r"(r[o + 23]), "r"(r[o + 24]),
      "r"(r[o + 25]), "r"(r[o + 26]), "r"(r[o + 27]), "r"(r[o + 28]), "r"(r[o + 29]), "r"(r[o + 30]),
      "r"(r[o + 31])
      : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// D (+)= A B: A in tensor memory, B by its shared-memory descriptor.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// Wait for the phase of an mbarrier, with a limit; false when it runs out.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity) {
  uint32_t done = 0;
  for (uint32_t i = 0; i < kWaitLimit && !done; ++i)
    asm volatile(
        "{.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
  return done != 0;
}

__device__ __forceinline__ void group_sync(int group) {
  asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory");
}

// Magnitude bits of eight 16-bit elements' largest finite one (BF16 or F16).
template <bool BF16>
__device__ __forceinline__ uint32_t largest16(const uint4& v, uint32_t m) {
  constexpr uint32_t kInf = BF16 ? 0x7F80u : 0x7C00u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    m = max(m, lo < kInf ? lo : 0u);
    m = max(m, hi < kInf ? hi : 0u);
  }
  return m;
}

// The exponent of a token's power of two: its magnitude bits m come into [2^14, 2^15).
template <bool BF16>
__device__ __forceinline__ int token_shift(uint32_t m) {
  const uint32_t mag = BF16 ? m << 16 : __float_as_uint(half_lo(m));
  return mag == 0 ? 0 : min(126, max(-126, 141 - (int)(mag >> 23)));
}

// x of `toks` tokens (zero up to n), columns [128 c0, 128 c1) (zero from K on), as f16
// times a power of two per token, K-major without a swizzle: 16-byte unit (k / 8) n +
// token. Copied as it is, then converted in place. s_max: magnitude bits per token.
template <bool BF16>
__device__ __forceinline__ void stage(const MvArgs& a, int c0, int c1, int toks, int n, uint4* xs, uint32_t* s_max) {
  const int k0 = c0 * kTileCols, k8 = (c1 - c0) * (kTileCols / 8), real = (min(a.K, c1 * kTileCols) - k0) / 8;
  const uint16_t* x = a.x + (int64_t)a.tok0 * a.ldx + k0;
  // 2 units of 16 tokens per warp and step: whole sectors, two-way bank conflicts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, blocks = n >> 4;
  for (int i = warp; i < blocks * (k8 / 2); i += kTcThreads / 32) {
    const int tok = (i % blocks) * 16 + (lane >> 1), u = (i / blocks) * 2 + (lane & 1);
    const bool ok = tok < toks && u < real;
    const uint16_t* p = x + (ok ? (int64_t)tok * a.ldx + u * 8 : 0);
    const int bytes = ok ? 16 : 0;  // 0: zeros, the source is not read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(xs + u * n + tok)), "l"(p), "r"(bytes)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  if (threadIdx.x < n) s_max[threadIdx.x] = 0;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  const int tok = threadIdx.x & (n - 1);  // of every unit that this thread converts
  uint32_t m = 0;
#pragma unroll 4
  for (int i = threadIdx.x; i < k8 * n; i += kTcThreads) m = largest16<BF16>(xs[i], m);
  if (m) atomicMax(s_max + tok, m);
  __syncthreads();
  float f[8];
  const float up = exp2i(token_shift<BF16>(s_max[tok]));
#pragma unroll 4
  for (int i = threadIdx.x; i < k8 * n; i += kTcThreads) {
    unpack8<BF16>(xs[i], f);
    xs[i] = make_uint4(pack2<false>(f[0] * up, f[1] * up), pack2<false>(f[2] * up, f[3] * up),
                       pack2<false>(f[4] * up, f[5] * up), pack2<false>(f[6] * up, f[7] * up));
  }
  // the tensor core reads through the asynchronous proxy
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <bool BF16>
__global__ void __launch_bounds__(kTcThreads, 1) fp4_tc_kernel(const MvArgs a, int n) {
  extern __shared__ uint4 dyn4[];
  __shared__ uint32_t s_max[64], s_tmem;
  __shared__ __align__(8) uint64_t s_bar[kGroups];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), size = cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, group = tid >> 7, gt = tid & 127;
  const int toks = min(n, a.B - a.tok0);
  const int ct = (a.K + kTileCols - 1) / kTileCols, c0 = ct * rank / size, kt = ct * (rank + 1) / size - c0;
  const int mt = (a.N + kTcRows - 1) / kTcRows, tiles = (a.N + kTileRows - 1) / kTileRows;
  const int set = blockIdx.x / size, sets = gridDim.x / size;
  const int per = mt / sets, more = mt - per * sets;
  const int q0 = set * per + min(set, more), q1 = q0 + per + (set < more ? 1 : 0);
  float* sums = reinterpret_cast<float*>(dyn4);  // [group][token][128 rows]
  uint4* xs = dyn4 + kGroups * n * kTcRows / 4;

  if (warp == 0)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                 "n"(kTmemCols)
                 : "memory");
  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&s_bar[i])) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  struct Tile {
    Codes32 a, b;  // a row's 64 bytes of a column tile
    uint32_t sc;
  };
  Tile buf[kTcAhead];
  const uint8_t *lc, *ls;
  bool inside;
  auto point = [&](int q) {  // at this thread's row of tile q
    const int row = q * kTcRows + gt, rt = row / kTileRows;
    inside = q < q1 && rt < tiles;
    const size_t at = inside ? (size_t)rt * ct + c0 : 0;
    lc = a.codes + at * kTileCodes + (row % kTileRows) * 64;
    ls = a.scales + at * kTileScales + (row % 8) * 8 + (row % kTileRows) / 8 * 4;
  };
  auto load = [&](Tile& t, int k) {
    if (inside) {
      t.a = ld_codes32(lc + (size_t)k * kTileCodes);
      t.b = ld_codes32(lc + (size_t)k * kTileCodes + 32);
      t.sc = __ldg(reinterpret_cast<const uint32_t*>(ls + (size_t)k * kTileScales));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) t.a.w[i] = t.b.w[i] = 0;
      t.sc = 0;
    }
  };
  point(q0 + group);
#pragma unroll
  for (int i = 0; i < kTcAhead; ++i)
    if (i < kt) load(buf[i], i);

  stage<BF16>(a, c0, c0 + kt, toks, n, xs, s_max);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem + group * (kTmemCols / kGroups);     // A here, D 64 columns on
  const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21);        // this warp's 32 lanes
  const uint32_t bar = smem_addr(&s_bar[group]);
  // kind::f16: D FP32, A and B f16, both K-major, N / 8 at bit 17, M / 16 at bit 24
  const uint32_t idesc = (1u << 4) | ((uint32_t)(n / 8) << 17) | ((uint32_t)(kTcRows / 16) << 24);
  // B: core matrices of 8 tokens x 16 bytes; 16 n bytes to the next 8 columns, 128 to the next 8 tokens
  const uint64_t bdesc = ((uint64_t)(smem_addr(xs) >> 4) & 0x3FFFu) | ((uint64_t)n << 16) | ((uint64_t)8 << 32) |
                         ((uint64_t)1 << 46);
  uint32_t phase = 0;
  bool ok = true;

  for (int q = q0; q < q1; q += kGroups) {
    if (q + group < q1) {
      // the row's largest scale code (NaN blocks apart)
      uint32_t top = 0;
      if (inside) {
#pragma unroll 8
        for (int k = 0; k < kt; ++k) {
          const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(ls + (size_t)k * kTileScales));
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t s = (w >> (8 * b)) & 255u;
            top = max(top, s == 255u ? 0u : s);
          }
        }
      }
      for (int k0 = 0; k0 < kt; k0 += kTcAhead) {
#pragma unroll
        for (int i = 0; i < kTcAhead; ++i) {
          const int k = k0 + i;
          if (k >= kt) break;
          // ---- decode: MMA step j covers columns 16j ..: block j / 2, quarters 2 (j & 1) and + 1
          uint32_t v[64], mul[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t s = (buf[i].sc >> (8 * b)) & 255u;
            const int e = max(0, (int)s - (int)top + 27);
            mul[b] = s == 255u ? 0x7E007E00u : (uint32_t)e * 0x04000400u;
          }
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              uint32_t h[4];
              e2m1x8_to_f16(t < 2 ? buf[i].a.w[t * 4 + b] : buf[i].b.w[(t - 2) * 4 + b], h);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[c]),
                                          *reinterpret_cast<const __half2*>(&mul[b]));
                v[b * 16 + t * 4 + c] = *reinterpret_cast<const uint32_t*>(&p);
              }
            }
          if (k + kTcAhead < kt) load(buf[i], k + kTcAhead);
          if (k > 0) {  // the MMAs of the column tile before have read A
            ok = ok && wait_phase(bar, phase);
            phase ^= 1;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          }
          tmem_store32(mine, v, 0);
          tmem_store32(mine + 32, v, 32);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          group_sync(group);
          if (gt == 0) {
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint64_t b = bdesc + (uint64_t)(k * 16 * n);  // 16 units of 8 columns, n * 16 bytes each
#pragma unroll
            for (int j = 0; j < 8; ++j) tc_mma(tmem + 64, tmem + j * 8, b + (uint64_t)(j * 2 * n), idesc, k + j > 0);
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                         : "memory");
          }
        }
      }
      // the next row tile's first codes, while this one's sums are taken
      point(q + kGroups + group);
#pragma unroll
      for (int i = 0; i < kTcAhead; ++i)
        if (i < kt) load(buf[i], i);
      ok = ok && wait_phase(bar, phase);
      phase ^= 1;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      float* to = sums + group * n * kTcRows + gt;
#pragma unroll 1
      for (int c = 0; c < n; c += 16) {
        uint32_t d[16];
        tmem_load16(mine + 64 + c, d);
#pragma unroll
        for (int j = 0; j < 16; ++j)
          // D holds 2^(12 - (top - 127)) times the token's power of two (one step: either
          // factor alone may leave FP32's range); a wait that ran out: no sum to trust
          to[(c + j) * kTcRows] =
              ok ? ldexpf(__uint_as_float(d[j]), (int)top - 139 - token_shift<BF16>(s_max[c + j])) : NAN;
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    cluster.sync();
    // ---- add the CTAs' sums: this CTA's share of the tokens, 4 rows a thread
    const int t0 = toks * rank / size, t1 = toks * (rank + 1) / size;
    const int here = min(kGroups, q1 - q) * (t1 - t0) * (kTcRows / 4);
    for (int i = tid; i < here; i += kTcThreads) {
      const int r = i % (kTcRows / 4) * 4, tt = i / (kTcRows / 4), tok = t0 + tt % (t1 - t0), g = tt / (t1 - t0);
      float* src = sums + (g * n + tok) * kTcRows + r;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int o = 0; o < size; ++o) {
        const float4 w = *reinterpret_cast<const float4*>(cluster.map_shared_rank(src, o));
        v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
      }
      const int64_t row = (int64_t)(q + g) * kTcRows + r, at = (int64_t)(a.tok0 + tok) * a.ldy + row;
      const float f[4] = {v.x, v.y, v.z, v.w};
      if (row + 4 <= a.N && a.y_type != WD_F32 && at % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7) == 0) {
        const uint2 o = a.y_type == WD_BF16 ? make_uint2(pack2<true>(v.x, v.y), pack2<true>(v.z, v.w))
                                            : make_uint2(pack2<false>(v.x, v.y), pack2<false>(v.z, v.w));
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) = o;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (row + j < a.N) store_elem(a.y, a.y_type, at + j, f[j]);
      }
    }
    cluster.sync();  // the sums are written again, or their CTA leaves
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 0) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "n"(kTmemCols));
  }
}

// The most clusters of `size` CTAs of this kernel that the device holds at a time
// (looked up once per device and kernel).
template <typename K>
int resident_clusters(K k, int size, size_t smem) {
  static std::mutex mu;
  static int cached[64][4] = {};  // [device][log2 size]
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  int l = 0;
  while ((1 << l) < size) ++l;
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev][l] == 0) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, k, &cfg) != cudaSuccess || c < 1) {
      (void)cudaGetLastError();
      c = sm_count() / size > 0 ? sm_count() / size : 1;
    }
    cached[dev][l] = c;
  }
  return cached[dev][l];
}

constexpr int kMaxCluster = 8;
int tokens_up(int tokens) { return tokens > 32 ? 64 : tokens > 16 ? 32 : 16; }
int stage_tiles(int n) { return kStageX / (n * 2 * kTileCols); }  // column tiles of x in a CTA

template <bool BF16>
moe_status launch(MvArgs a, cudaStream_t st) {
  auto k = fp4_tc_kernel<BF16>;
  const int ct = (a.K + kTileCols - 1) / kTileCols, mt = (a.N + kTcRows - 1) / kTcRows;
  int n = tokens_up(a.B - a.tok0);
  while (n > 16 && ct > kMaxCluster * stage_tiles(n)) n /= 2;
  // CTAs per cluster: as many as x needs, and more while there are fewer row tiles than
  // warpgroups and every CTA keeps 4 column tiles
  int size = 1;
  while (size < kMaxCluster && ((ct + size - 1) / size > stage_tiles(n) ||
                                (mt * size < sm_count() * kGroups && ct >= 8 * size)))
    size *= 2;
  const size_t room = kStageX + (size_t)kGroups * 64 * kTcRows * 4;
  moe_status rc = allow_smem(k, room);
  if (rc != MOE_OK) return rc;
  const int most = resident_clusters(k, size, room), want = (mt + kGroups - 1) / kGroups;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((want < most ? want : most) * size));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = (size_t)((ct + size - 1) / size) * n * 2 * kTileCols + (size_t)kGroups * n * kTcRows * 4;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  for (; a.tok0 < a.B; a.tok0 += n) {
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k, a, n);
    if (e != cudaSuccess) {
      set_error("wd_fp4_matvec launch", e);
      return MOE_ERR_CUDA;
    }
  }
  return MOE_OK;
}

}  // namespace

int tc_most_columns(int) { return kMaxCluster * stage_tiles(16) * kTileCols; }

moe_status launch_tc(MvArgs a, bool bf16, cudaStream_t st) { return bf16 ? launch<true>(a, st) : launch<false>(a, st); }

}  // namespace wd
