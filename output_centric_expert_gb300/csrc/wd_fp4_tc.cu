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
// down to 2^-26 of the row's largest scale. Smaller ones are 0 there; where one has a
// code other than 0, which no ordinary matrix has, its products are added at the end,
// block by block. The row's 2^top comes back at the end.
//
// Work. A cluster of CTAs shares a run of 128-row tiles, each CTA with its share of the
// columns, so that it stages and converts only that share of x (64 tokens of 1024
// columns are 128 KB). In a CTA two warpgroups take a row tile, every other column tile
// each: a thread decodes 128 columns of a row, stores them to tensor memory, and one
// thread issues the eight MMAs while all decode the next columns. (One warpgroup per
// row tile left the decode waiting on its own latency: two warps per scheduler.) A
// pair's sums are added on their way out of tensor memory; the CTAs' go to the one that
// writes their tokens, through distributed shared memory, and are added there in order.
//
// Bound. 64 tokens of 9216 x 4096 (20 MB, 4.8 GFLOP): 15.3 us, of which 2.5 are the
// launch, 4.7 x (1.7 for its trip from L2 to all SMs, the rest largest magnitudes and
// conversion), 4.1 the loop (about 330 instructions per warp and column tile of 128,
// 64 of them conversions at half rate), 3.4 the sums. Tensor cores are busy 14 % of it,
// DRAM 20 %. Large matrices are held by the loop: 16 tokens of 65536 x 4096 43.3 us,
// 3.3 TB/s; 64 tokens 79 us (42.1 and 77 without the test for blocks that A has as 0).
#include <cooperative_groups.h>

#include <mutex>

#include "wd_block.cuh"
#include "wd_fp4.h"

namespace wd {
namespace {

namespace cg = cooperative_groups;

constexpr int kTcThreads = 512, kGroups = 4;  // warpgroups
constexpr int kRowTiles = 2;        // row tiles of a CTA at a time, two warpgroups on each
constexpr int kTcRows = 128;
constexpr int kTcAhead = 2;         // column tiles of codes in flight per thread
constexpr int kTmemCols = 512;      // per warpgroup: 64 for A, up to 64 for D
constexpr int kMaxCluster = 8;      // CTAs, a power of two as every size here
constexpr int kStageX = 128 * 1024; // bytes of x per CTA at most
constexpr uint32_t kWaitLimit = 1u << 22;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
      "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
      "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}

// Eight columns from `at` and, where `both`, from `at2`.
__device__ __forceinline__ void tmem_load8(uint32_t at, uint32_t at2, bool both, uint32_t (&r)[8], uint32_t (&q)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at));
  if (both)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7])
                 : "r"(at2));
  // the registers are operands, so that no use of them moves above
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(q[0]), "+r"(q[1]), "+r"(q[2]), "+r"(q[3]), "+r"(q[4]), "+r"(q[5]), "+r"(q[6]), "+r"(q[7])::"memory");
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

// The two warpgroups of a row tile.
__device__ __forceinline__ void pair_sync(int side) {
  asm volatile("bar.sync %0, 256;" ::"r"(side + 1 + kGroups) : "memory");
}

// x of `toks` tokens (zero up to n), columns [128 c0, 128 c1) (zero from K on), as f16
// times a power of two per token, K-major in the 128-byte swizzle: [64 columns][token]
// [128 bytes], 16-byte unit u of a row at u ^ (token & 7). 8 lanes have a token's 128
// bytes (whole lines, no bank conflicts) and keep them in registers from the load to the
// converted store. s_max: magnitude bits per token. 1 << nlog = n.
// `meanwhile` runs while they are loaded.
template <bool BF16, typename F>
__device__ __forceinline__ void stage(const MvArgs& a, int c0, int c1, int toks, int nlog, uint4* xs, uint32_t* s_max,
                                      F meanwhile) {
  constexpr int kStep = kTcThreads / 8, kMost = kStageX / 16 / kTcThreads;
  const int u = threadIdx.x & 7, first = threadIdx.x >> 3;
  const int rows = (c1 - c0) * 2 << nlog;  // 128-byte rows, row = 64-column run * n + token
  const int tok = first & ((1 << nlog) - 1);  // with 64 rows a step, every row of this thread is of one token
  const int k0 = c0 * kTileCols + (first >> nlog) * 64 + u * 8, dk = kStep >> nlog << 6;
  const uint16_t* x = a.x + (int64_t)(a.tok0 + tok) * a.ldx + k0;
  const int mine = tok < toks ? (min(a.K, c1 * kTileCols) - k0 + dk - 1) / dk : 0;  // pieces that are there
  // in fours that small products skip: they spend their time fetching code
  constexpr int kFour = 4;
  uint4 v[kMost];
#pragma unroll
  for (int f = 0; f < kMost; f += kFour)
    if (f * kStep < rows)
#pragma unroll
      for (int i = f; i < f + kFour; ++i)
        v[i] = i < mine ? __ldg(reinterpret_cast<const uint4*>(x + i * dk)) : make_uint4(0, 0, 0, 0);
  if (threadIdx.x < 1 << nlog) s_max[threadIdx.x] = 0;
  meanwhile();
  __syncthreads();
  uint32_t pair = kPairs0<BF16>;
#pragma unroll
  for (int f = 0; f < kMost; f += kFour)
    if (f * kStep < rows)
#pragma unroll
      for (int i = f; i < f + kFour; ++i) pair = largest_pairs<BF16>(v[i], pair);
  uint32_t m = largest_of<BF16>(pair);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (u == 0) atomicMax(s_max + tok, m);
  __syncthreads();
  const float up = exp2i(shift_of_16<BF16>(s_max[tok]));
  uint4* to = xs + first * 8 + (u ^ (tok & 7));
#pragma unroll
  for (int f = 0; f < kMost; f += kFour)
    if (f * kStep < rows)
#pragma unroll
      for (int i = f; i < f + kFour; ++i)
        if (first + i * kStep < rows) to[i * kStep * 8] = scaled_f16<BF16>(v[i], up);
  // the tensor core reads through the asynchronous proxy
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <bool BF16>
__global__ void __launch_bounds__(kTcThreads, 1) fp4_tc_kernel(const MvArgs a, int n) {
  extern __shared__ uint4 dyn4[];
  __shared__ uint32_t s_max[64], s_tmem, s_failed, s_again;  // s_again: an output is not finite
  __shared__ __align__(16) float s_back[64];  // 1 / the tokens' powers of two
  __shared__ __align__(8) uint64_t s_bar[kGroups];
  __shared__ uint16_t s_top[kGroups][kTcRows];  // and bit 8: the row has blocks that A has as 0 although they are not
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), size = cluster.num_blocks();
  const int tid = threadIdx.x, warp = tid >> 5, group = tid >> 7, gt = tid & 127;
  const int side = group >> 1, half = group & 1;  // row tile of the CTA, and which column tiles of it
  const int toks = min(n, a.B - a.tok0);
  const int log = 31 - __clz(size), nlog = 31 - __clz(n);
  const int ct = (a.K + kTileCols - 1) / kTileCols, c0 = (ct * rank) >> log, kt = ((ct * (rank + 1)) >> log) - c0;
  const int tiles = (a.N - 1) / kTileRows + 1;
  const int set = blockIdx.x >> log;  // a cluster's row tiles [q0, q1)
  const int q0 = set * a.per + min(set, a.more), q1 = q0 + a.per + (set < a.more ? 1 : 0);
  uint4* xs = dyn4 + (1024 - (smem_addr(dyn4) & 1023)) % 1024 / 16;  // the swizzle counts from 1024-byte boundaries
  const int own = n >> log;  // tokens whose sums this CTA writes, rank * own on
  float* sums = reinterpret_cast<float*>(xs + ((ct + size - 1) >> log) * 16 * n);  // [row tile][CTA][token][128 rows]

  if (size > 1) cluster.barrier_arrive();  // waited for before the first sums go to another CTA
  struct Tile {
    Codes32 a, b;  // a row's 64 bytes of a column tile
    uint32_t sc;
  };
  Tile buf[kTcAhead];
  const uint8_t *lc, *ls;
  const int my_kt = (kt - half + 1) / 2;  // column tiles half, half + 2, ...
  auto point = [&](int q) {  // at this thread's row of tile q; behind the last row: any row, y has none
    const int row = q * kTcRows + gt, rt = row / kTileRows;
    const size_t at = (size_t)(rt < tiles ? rt : 0) * ct + c0 + half;
    lc = a.codes + at * kTileCodes + (row % kTileRows) * 64;
    ls = a.scales + at * kTileScales + (row % 8) * 8 + (row % kTileRows) / 8 * 4;
  };
  auto load = [&](Tile& t, int k) {
    t.a = ld_codes32(lc + (size_t)k * 2 * kTileCodes);
    t.b = ld_codes32(lc + (size_t)k * 2 * kTileCodes + 32);
    t.sc = __ldg(reinterpret_cast<const uint32_t*>(ls + (size_t)k * 2 * kTileScales));
  };
  // The row's largest scale here, NaN blocks apart: their 255 + 0x7F01 is negative in 16 bits.
  auto largest_scale = [&]() {
    uint32_t top = 0x7F017F01u;
#pragma unroll 8
    for (int k = 0; k < my_kt; ++k) {
      const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(ls + (size_t)k * 2 * kTileScales));
      top = __viaddmax_s16x2(w & 0x00FF00FFu, 0x7F017F01u, top);
      top = __viaddmax_s16x2((w >> 8) & 0x00FF00FFu, 0x7F017F01u, top);
    }
    return max(top & 0xFFFFu, top >> 16) - 0x7F01u;
  };
  // The next round's weights to L2, 16 rows a lane. Clusters wait for one another between rounds:
  // 64 tokens of 65536 x 4096 83.4 -> 77.8 us. (A CTA alone has its row tiles out of step, and so
  // much ahead only disturbs the loads at hand: 16 tokens 42.8 -> 49 us.)
  auto prefetch = [&](int q) {
    const int rt = q * (kTcRows / kTileRows) + (tid & 31);
    if (warp == 1 && (tid & 31) < kRowTiles * kTcRows / kTileRows && rt < tiles && rt < q1 * (kTcRows / kTileRows)) {
      const size_t at = (size_t)rt * ct + c0;
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.codes + at * kTileCodes), "r"(kt * kTileCodes)
                   : "memory");
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.scales + at * kTileScales), "r"(kt * kTileScales)
                   : "memory");
    }
  };
  point(q0 + side);
#pragma unroll
  for (int i = 0; i < kTcAhead; ++i)
    if (i < my_kt) load(buf[i], i);
  stage<BF16>(a, c0, c0 + kt, toks, nlog, xs, s_max, [&]() {
    if (warp == 0)
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                   "n"(kTmemCols)
                   : "memory");
    if (tid == 0) {
      s_failed = s_again = 0;
#pragma unroll
      for (int i = 0; i < kGroups; ++i)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(&s_bar[i])) : "memory");
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
  });
  if (tid < n) s_back[tid] = exp2i(-shift_of_16<BF16>(s_max[tid]));
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = s_tmem + group * (kTmemCols / kGroups);     // A here, D 64 columns on
  const uint32_t mine = tmem + ((uint32_t)(warp & 3) << 21);        // this warp's 32 lanes
  const uint32_t bar = smem_addr(&s_bar[group]);
  // kind::f16: D FP32, A and B f16, both K-major, N / 8 at bit 17, M / 16 at bit 24
  const uint32_t idesc = (1u << 4) | ((uint32_t)(n / 8) << 17) | ((uint32_t)(kTcRows / 16) << 24);
  // B: K-major, 128-byte swizzle; 1024 bytes from 8 tokens to the next 8
  const uint64_t bdesc = ((uint64_t)(smem_addr(xs) >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)64 << 32) |
                         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
  uint32_t phase = 0, next_top = largest_scale();
  bool ok = true;

  for (int q = q0; q < q1; q += kRowTiles) {
    if (size > 1 && q + kRowTiles < q1) prefetch(q + kRowTiles);
    if (q + side < q1) {
      const uint32_t top = next_top;
      uint32_t low = 0;
      for (int k0 = 0; k0 < my_kt; k0 += kTcAhead) {
#pragma unroll
        for (int i = 0; i < kTcAhead; ++i) {
          const int k = k0 + i;
          if (k >= my_kt) break;
          // 2^(s - top + 12) in both halves of mul[b], 0 below 2^-14; a NaN block's is above 2^12
          uint32_t mul[4];
          {
            const uint32_t less = ((27u - top) & 0xFFFFu) * 0x10001u;
            const uint32_t e02 = __viaddmax_s16x2(buf[i].sc & 0x00FF00FFu, less, 0u);
            const uint32_t e13 = __viaddmax_s16x2((buf[i].sc >> 8) & 0x00FF00FFu, less, 0u);
            mul[0] = __byte_perm(e02 << 10, 0, 0x1010), mul[2] = __byte_perm(e02 << 10, 0, 0x3232);
            mul[1] = __byte_perm(e13 << 10, 0, 0x1010), mul[3] = __byte_perm(e13 << 10, 0, 0x3232);
            if ((__vmaxs2(e02, e13) + 0x7FE47FE4u) & 0x80008000u)  // the row's sum is NaN
              mul[0] = mul[1] = mul[2] = mul[3] = 0x7E007E00u;
            if (((__vminu2(e02, e13) + 0x7FFF7FFFu) & 0x80008000u) != 0x80008000u) {  // a multiplier is 0
#pragma unroll
              for (int b = 0; b < 4; ++b)
                if (mul[b] == 0) low |= buf[i].a.w[b] | buf[i].a.w[4 + b] | buf[i].b.w[b] | buf[i].b.w[4 + b];
            }
          }
          // ---- decode and store two blocks at a time; column k / 2 of A holds the elements k, k + 1
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            uint32_t v[32];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                uint32_t h[4];
                e2m1x8_to_f16(t < 2 ? buf[i].a.w[t * 4 + 2 * o + b] : buf[i].b.w[(t - 2) * 4 + 2 * o + b], h);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[c]),
                                            *reinterpret_cast<const __half2*>(&mul[2 * o + b]));
                  v[b * 16 + t * 4 + c] = *reinterpret_cast<const uint32_t*>(&p);
                }
              }
            if (o == 0 && k > 0) {  // the MMAs of the column tile before have read A
              ok = ok && wait_phase(bar, phase);
              phase ^= 1;
              asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            }
            tmem_store32(mine + 32 * o, v);
          }
          if (k + kTcAhead < my_kt) load(buf[i], k + kTcAhead);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
          group_sync(group);
          if (gt == 32 * group) {  // a different scheduler's warp in each group
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const uint64_t b = bdesc + (uint64_t)((2 * k + half) * 16 * n);  // two runs of 64 columns, 8 n units each
#pragma unroll
            for (int j = 0; j < 8; ++j)  // 32 bytes on in a row, or in the second run
              tc_mma(tmem + 64, tmem + j * 8, b + (uint64_t)(j / 4 * 8 * n + j % 4 * 2), idesc, k + j > 0);
            asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                         : "memory");
          }
        }
      }
      // the next row tile's first codes, while this one's sums are taken
      if (q + kRowTiles + side < q1) {
        point(q + kRowTiles + side);
#pragma unroll
        for (int i = 0; i < kTcAhead; ++i)
          if (i < my_kt) load(buf[i], i);
        next_top = largest_scale();
      }
      if (my_kt > 0) {
        ok = ok && wait_phase(bar, phase);
        phase ^= 1;
      }
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      s_top[group][gt] = (uint16_t)(top | ((low & 0x77777777u) != 0 ? 256 : 0));
      if (!ok) s_failed = 1;
      pair_sync(side);  // both halves' sums are there
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    }
    if (size > 1) cluster.barrier_wait();  // the owners have read the sums before
    if (q + side < q1) {
      // D holds the sum times 2^(12 - (top - 127)) and the token's power of two. Taken off
      // one after the other where neither step can leave FP32's range, else in one.
      // Either half adds both halves' sums of its half of the tokens.
      const uint32_t half0 = s_top[side * 2][gt], half1 = s_top[side * 2 + 1][gt];
      const uint32_t t0 = half0 & 255u, t1 = kt > 1 ? half1 & 255u : t0;
      const bool plain = __all_sync(0xFFFFFFFFu, min(t0, t1) >= 64u && max(t0, t1) <= 190u);
      const float fail = s_failed ? NAN : 1.0f;  // a wait that ran out: no sum to trust
      const float back0 = plain ? exp2i((int)t0 - 139) * fail : fail, back1 = plain ? exp2i((int)t1 - 139) * fail : fail;
      const uint32_t d0 = s_tmem + side * 2 * (kTmemCols / kGroups) + ((uint32_t)(warp & 3) << 21) + 64;
      const int64_t row = (int64_t)(q + side) * kTcRows + gt;
      const bool low = row < a.N && ((half0 | half1) & 256u);
      const bool any_low = __any_sync(0xFFFFFFFFu, low);
      const uint32_t slot = smem_addr(sums + ((side << log) + rank) * own * kTcRows + gt);
      uint32_t place = 0;
#pragma unroll 1
      for (int c = half * (n / 2); c < (half + 1) * (n / 2); c += 8) {
        uint32_t d[8], e[8] = {};
        tmem_load8(d0 + c, d0 + kTmemCols / kGroups + c, kt > 1, d, e);
        const float4 b0 = *reinterpret_cast<const float4*>(s_back + c), b1 = *reinterpret_cast<const float4*>(s_back + c + 4);
        const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          o[j] = (__uint_as_float(d[j]) * back0 + __uint_as_float(e[j]) * back1) * b[j];
        if (!plain) {
#pragma unroll 1
          for (int j = 0; j < 8; ++j) {
            float v = 0.0f, w = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (j == k) v = __uint_as_float(d[k]) * back0, w = __uint_as_float(e[k]) * back1;
            const int shift = shift_of_16<BF16>(s_max[c + j]);
            v = ldexpf(v, (int)t0 - 139 - shift) + ldexpf(w, (int)t1 - 139 - shift);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (j == k) o[k] = v;
          }
        }
        if (any_low) {
#pragma unroll 1
          for (int j = 0; low && j < 8 && c + j < toks; ++j) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (j == k) v = o[k];
#pragma unroll 1
            for (int part = 0; part < 2; ++part)  // either half's column tiles
              v += plain_sum<BF16>(a, row, a.tok0 + c + j, c0 + part, c0 + kt, 2, (int)(part ? t1 : t0) - 27);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (j == k) o[k] = v;
          }
          __syncwarp();
        }
        if (size == 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j < toks && row < a.N) store_elem(a.y, a.y_type, (int64_t)(a.tok0 + c + j) * a.ldy + row, o[j]);
          float all = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) all += fabsf(o[j]);
          if (!(all < INFINITY)) s_again = 1;
        } else {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {  // own >= 2
            if (j == 0 || own < 8)  // the owner's place for token c + j
              asm("mapa.shared::cluster.u32 %0, %1, %2;"
                  : "=r"(place)
                  : "r"(slot + ((c + j) & (own - 1)) * (kTcRows * 4)), "r"((c + j) >> (nlog - log)));
            const uint32_t to = own < 8 ? place : place + j * kTcRows * 4;
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(o[j]) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + kTcRows * 4), "f"(o[j + 1]) : "memory");
          }
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      if (size == 1) pair_sync(side);  // the next row tile's MMAs write D again
    }
    if (size > 1) {
      cluster.sync();
      // ---- add the CTAs' sums of this one's tokens, 4 rows a thread
      const int here = q + side < q1 ? min(own, toks - rank * own) * (kTcRows / 4) : 0;
      for (int i = tid & (kTcThreads / kRowTiles - 1); i < here; i += kTcThreads / kRowTiles) {
        const int r = i % (kTcRows / 4) * 4, tok = i / (kTcRows / 4);
        const float* src = sums + ((side << log) * own + tok) * kTcRows + r;
        float4 v = *reinterpret_cast<const float4*>(src);
        for (int o = 1; o < size; ++o) {
          const float4 w = *reinterpret_cast<const float4*>(src + o * own * kTcRows);
          v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
        }
        store_rows(a, a.tok0 + rank * own + tok, (int64_t)(q + side) * kTcRows + r, v);
        if (not_finite(v)) s_again = 1;
      }
      if (q + kRowTiles < q1) cluster.barrier_arrive();
    }
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 0) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "n"(kTmemCols));
  }
  if (s_again) {
    const int first = size == 1 ? 0 : rank * own, end = size == 1 ? toks : min(toks, first + own);
    take_again<BF16>(a, (int64_t)q0 * kTcRows, (int64_t)q1 * kTcRows, a.tok0 + first, a.tok0 + end);
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

int tokens_up(int tokens) { return tokens > 32 ? 64 : tokens > 16 ? 32 : 16; }
int stage_tiles(int n) { return kStageX / (n * 2 * kTileCols); }  // column tiles of x in a CTA

template <bool BF16>
moe_status launch(MvArgs a, cudaStream_t st) {
  auto k = fp4_tc_kernel<BF16>;
  const int ct = (a.K + kTileCols - 1) / kTileCols, mt = (a.N - 1) / kTcRows + 1;
  int n = tokens_up(a.B - a.tok0);
  while (n > 16 && ct > kMaxCluster * stage_tiles(n)) n /= 2;
  const size_t room = kStageX + (size_t)kRowTiles * 64 * kTcRows * 4 + 1024;
  static SmemOnce once;
  const moe_status rc = once.allow(k, room);
  if (rc != MOE_OK) return rc;
  // CTAs per cluster: as many as x needs, and more while all row tiles still have a
  // place at once and every CTA keeps 2 column tiles. 16 tokens of 9216 x 4096 (36 pairs
  // of row tiles): 21.6 us alone, 14.1, 10.9 and, where only 15 clusters fit, 16.3 us
  // for 2, 4 and 8 CTAs; 65536 x 4096: 42.3, 52.0, 62.8, 90.4.
  const int want = (mt + kRowTiles - 1) / kRowTiles;
  int size = 1;
  while (size < kMaxCluster && (ct + size - 1) / size > stage_tiles(n)) size *= 2;
  while (size < kMaxCluster && ct >= 4 * size && want <= resident_clusters(k, 2 * size, room)) size *= 2;
  const int most = resident_clusters(k, size, room);
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  const int sets = want < most ? want : most;
  a.per = mt / sets;
  a.more = mt - a.per * sets;
  cfg.gridDim = dim3((unsigned)(sets * size));
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = (size_t)((ct + size - 1) / size) * n * 2 * kTileCols + (size_t)kRowTiles * n * kTcRows * 4 + 1024;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  for (int64_t tok = a.tok0; tok < a.B; tok += n) {
    a.tok0 = (int)tok;
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
