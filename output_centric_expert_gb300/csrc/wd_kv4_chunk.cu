// wd_kv4_attend_chunk: attention of several new tokens per sequence over the paged
// 4-bit cache, which holds them already.
//
// Mathematics. Rows are (token, query head) pairs that share a KV head. With z = scale q.k
// in units of log 2, one pass over the keys keeps m, l = sum 2^(z_j - m) and acc = sum
// 2^(z_j - m) v_j; partial results join as l = sum l_i 2^(m_i - m), acc likewise. m follows
// the row's maximum only when that is more than 2^kSlack above it, so acc is hardly ever
// rescaled.
//   S = Q K^T: tcgen05.mma kind::f16, 128 rows, f16 operands. Queries are f16 times a power of
//   two per row, as in wd_kv4_attend. Keys are E2M1 times 2^(s - 127 + 4), which f16 holds
//   exactly for scale codes s from 109 to 136 (and zero blocks); keys with others get a power of
//   two of their own, by which their column of S is multiplied.
//   acc += P V: BF16 operands. V is decoded to BF16, which holds every E2M1 code times every E8M0
//   scale up to 6 * 2^125 exactly. P is two BF16 terms, the second what the cut of the first
//   left: 16 bits down to 2^-118, where BF16 begins to lack the second term's, and none below 2^-126.
//
// Work. A CTA has kQ tiles of 128 rows against tiles of kKeys keys. Its warps:
//   4 per row tile   softmax: a thread has a row. S comes from tensor memory, P goes back in
//                    its place (16 columns of first terms, 16 of second for 32 keys); the
//                    queries, copied into shared memory as f16
//   8 per row tile   decode: codes and scales come by bulk copies, 8 or 16 keys to a warp, and
//                    go to shared memory as operands (K-major and dim-major, 128-byte swizzle);
//                    with two row tiles half of these warps have the keys, half the values
//   4                issue the MMAs: for each row tile one the products with keys, one those
//                    with values
// The keys of a tile are in the softmax 64 at a time, in two buffers per row tile: while one is
// exponentiated the other's scores are computed, and while one row tile is in its softmax the
// tensor cores have the other's products. An item of up to 128 rows gives its even key tiles to
// the first row tile and its odd ones to the second, which join at the end.
// All (sequence, row block, KV head) items are cut into units of one key tile; CTA c of G
// takes the c-th contiguous share of all units, found from the lengths on the device. An
// item that several CTAs share leaves its parts in the workspace, and a dependent launch
// joins them in CTA order.
//
// Barriers. A wait names a phase by its parity, so a reader must not fall two phases behind. All readers but one kind wait
// for every phase: one warp for queries, filled slots, probabilities and raw codes, the four softmax warps of a row tile
// for scores, eight decode warps for freed slots. o_done, the sums of a buffer, is read by the warp that issues the
// products with keys, at every phase, and by the row tile's four softmax warps, which skip some. They are safe
// because a buffer's next sums need its next probabilities, which these same warps give: one phase at most
// is open when they wait. Every wait for an mbarrier has a limit, after which the warp goes on and the results are NaN;
// the two named barriers of the softmax warps have none, and all of these warps always reach them.
//
// Measured (GB300). 2048 tokens behind 30011 keys, 28 query heads of 128 on 4 KV heads: 938
// us, 971 TFLOP/s of the two products, or 1457 of the three that are issued, 79 % of a library
// BF16 GEMM; 8192 tokens with 64 query heads, causal: 1251 us; heads of 256, 24 prompts of up
// to 1500 with a window of 1000: 210 us. Of the first's 942 (as a call) it takes 817 without the arithmetic of decoding, 888
// without the second term of P, 950 without exponentials, 734 without all three; 7 tokens behind 131000 keys 123, 92,
// 119, 126 and 88; heads of 256 213, 175, 203, 215 and 154. So exponentials cost nothing, decoding an eighth to a
// quarter, and what is left is presumably the chain of a piece (scores out of tensor memory, their
// largest, probabilities back in, sums), which a row tile's pieces go through one after the other. 72 registers at launch spill
// 64 to 84 bytes of a thread, 128 with heads of 256 72. Tried: one warp per group for all MMAs, 2 % slower;
// the same eight warps decoding K, then V, 12 %; an item counted as two tiles 18 % for the second
// case, as six 2 %; V as f16, K-major, 24 % (more code: the warps of all roles share the
// instruction caches, which miss in 13 % of their requests).
#include <cmath>

#include "wd_block.cuh"
#include "wd_fp4.h"
#include "wd_kv4.cuh"

namespace wd {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kSlack = 8.0f;
constexpr int kRows = 128;       // of a row tile
constexpr int kPiece = 64;       // keys that are in the softmax at a time
constexpr int kItemUnits = 4;    // what an item costs beside its key tiles, in tiles
constexpr int kMinUnits = 3;     // of a CTA, on average, unless it has an item to itself
constexpr uint32_t kWaitLimit = 1u << 20;  // tries of a wait for an mbarrier
constexpr int kSeqChunk = 512;   // sequences whose units are in shared memory at a time
constexpr int kDecodeWarps = 8;
constexpr int kMeta = 8;         // key tiles whose page masks and bad blocks are kept

// The split item that goes on from this CTA into the next, parts 0 where there is none: an item with parts in the
// CTAs c .. c + parts - 1 is in all their entries but the last.
struct __align__(16) Split {
  int32_t parts, index;   // index: this CTA's among them
  int32_t seq, head;      // KV head
  int32_t row0, rows;     // of the sequence's flat rows (token * group + query head of the group)
  int32_t pad[2];
};

struct ChunkArgs {
  const uint8_t *kc, *ks, *vc, *vs;
  const uint16_t* q;
  const int32_t *table, *lens, *cu;
  uint16_t* out;
  float* lse;
  float* parts;  // [2 * grid][part_rows * (D + 2)]
  Split* split;  // [grid]
  int32_t* err;
  int64_t ldq, ldo;
  int32_t T, S, max_blocks, pages, page_shift, heads, group, window, room;  // room: keys of a row of the table
  int32_t part_rows;
  float scale_log2;
  uint32_t group_mul, group_shift;  // n / group = n * mul >> 32 >> shift for n below 2^31
};

template <int D_, int KEYS, int Q>
struct Config {
  static constexpr int D = D_, kKeys = KEYS, kQ = Q;
  static constexpr int kSlots = 2;  // of K, and of V
  static constexpr int kItemRows = Q * kRows;
  static constexpr int kSoftWarps = 4 * Q, kDecoders = kDecodeWarps * Q, kThreadsAll = (kSoftWarps + kDecoders + 4) * 32;
  static constexpr int kWarpKeys = KEYS / kDecodeWarps;  // keys of a decode warp in a tile: 8 or 16, inside a run of 16
  static constexpr int kQBytes = kRows * D * 2;          // of a row tile
  static constexpr int kTile = KEYS * D * 2;             // of K or V
  static constexpr int kCodes = kWarpKeys * D / 2, kScales = kWarpKeys * D / 32;  // bytes of a decode warp's keys, K or V
  static constexpr int kRaw = 2 * (kCodes + kScales);    // codes of K, of V, scales of K, of V
  static constexpr int kSmem = 1024 + Q * kQBytes + 2 * kSlots * kTile + kDecodeWarps * kRaw;
  static constexpr int kPieces = KEYS / kPiece;          // of a tile
  static constexpr int kCols = Q * (2 * kPiece + D);     // two pieces' S and the sums of each row tile
  static constexpr int kTmem = kCols <= 256 ? 256 : 512;
  // registers of a thread: setmaxnreg shares out what the launch has
  static constexpr int kSoftRegs = 136, kDecodeRegs = 48, kMmaRegs = 40;
  static constexpr int kRegs = 32 * (kSoftWarps * kSoftRegs + kDecoders * kDecodeRegs + 4 * kMmaRegs);
  static_assert(kCols <= 512 && kSmem <= 221 * 1024, "fits an SM");
};

// ------------------------------------------------------------------ PTX --

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

#define WD_R32(r)                                                                                                       \
  "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),           \
      "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),            \
      "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),           \
      "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])

// 32 columns of this warp's lanes; the registers are not valid before tmem_wait.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : WD_R32(r)::"memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 columns, waited for.
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (+)= A B: both by shared-memory descriptors (the low words; the high ones are constants), or A in tensor memory.
template <uint32_t A_HI, uint32_t B_HI, uint32_t IDESC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, bool add) {
  asm volatile(
      "{.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %4};\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %6, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"((uint32_t)add), "n"(A_HI), "n"(B_HI), "n"(IDESC)
      : "memory");
}
template <uint32_t B_HI, uint32_t IDESC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, bool add) {
  asm volatile(
      "{.reg .pred p;\n\t.reg .b64 y;\n\t"
      "mov.b64 y, {%2, %4};\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %5, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"((uint32_t)add), "n"(B_HI), "n"(IDESC)
      : "memory");
}
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile(
      "{.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// The barrier completes when every MMA issued so far by this thread has.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Wait for the phase of an mbarrier, with a limit; false when it runs out.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = kWaitLimit; i; --i) {
    uint32_t done;
    asm volatile(
        "{.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t to, const void* from, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to), "l"(from),
               "r"(bytes), "r"(bar)
               : "memory");
}
// All threads of the softmax warps (no limit: none of them leaves its loop before the others).
__device__ __forceinline__ void soft_sync(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two FP32 operations in one instruction.
__device__ __forceinline__ uint64_t pair_of(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void split_pair(uint64_t v, uint32_t& a, uint32_t& b) { asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));  // below 2^-126: 0
  return r;
}
__device__ __forceinline__ uint32_t mul2_bf16(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r =
      __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// -------------------------------------------------------------- the items --

// The token of a flat row.
__device__ __forceinline__ int token_of(const ChunkArgs& a, int row) {
  return a.group_mul ? (int)(__umulhi((uint32_t)row, a.group_mul) >> a.group_shift) : row >> a.group_shift;
}

// A sequence's new rows.
struct Seq {
  int32_t first, tokens, len;  // first row of q, new tokens, keys before them
};
__device__ __forceinline__ Seq seq_of(const ChunkArgs& a, int s) {
  Seq q = {s, 1, __ldg(a.lens + s)};
  if (a.cu) {
    const int c0 = max(0, __ldg(a.cu + s)), c1 = min(a.T, __ldg(a.cu + s + 1));
    q.first = c0;
    q.tokens = max(0, c1 - c0);
  }
  return q;
}
// The keys [lo, hi) that a token sees.
__device__ __forceinline__ int keys_end(const ChunkArgs& a, const Seq& q, int token) {
  return q.len < 0 ? 0 : (int)min((int64_t)a.room, (int64_t)q.len + token + 1);
}
__device__ __forceinline__ int keys_begin(const ChunkArgs& a, const Seq& q, int token) {
  return q.len < 0 || a.window == 0 ? 0 : (int)min((int64_t)a.room, max((int64_t)0, (int64_t)q.len + token + 1 - a.window));
}
// The keys that the rows of block b see, as tiles from kt0 on.
template <typename C>
__device__ __forceinline__ int block_tiles(const ChunkArgs& a, const Seq& q, int b, int& kt0) {
  const int rows = q.tokens * a.group;
  const int lo = keys_begin(a, q, token_of(a, b * C::kItemRows));
  const int hi = keys_end(a, q, token_of(a, min((b + 1) * C::kItemRows, rows) - 1));
  kt0 = lo / C::kKeys;
  return hi > lo ? (hi + C::kKeys - 1) / C::kKeys - kt0 : 0;
}
template <typename C>
__device__ __forceinline__ int blocks_of(const ChunkArgs& a, const Seq& q) {
  return (q.tokens * a.group + C::kItemRows - 1) / C::kItemRows;
}
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// A sequence's units (a warp).
template <typename C>
__device__ __forceinline__ int64_t seq_units(const ChunkArgs& a, int s) {
  const Seq q = seq_of(a, s);
  const int blocks = blocks_of<C>(a, q);
  int64_t u = 0;
  for (int b = threadIdx.x & 31; b < blocks; b += 32) {
    int kt0;
    u += block_tiles<C>(a, q, b, kt0) + kItemUnits;
  }
  return warp_sum(u) * a.heads;
}

// Where a CTA's share begins, and the shares.
struct Share {
  int64_t begin, end, total;
  int32_t ctas, seq, block, head, off;  // off: units of the first item that are not this CTA's
};
__device__ __forceinline__ int64_t share_begin(int64_t total, int ctas, int c) {
  const int64_t q = total / ctas, r = total % ctas;
  return q * c + min((int64_t)c, r);
}
__device__ __forceinline__ int cta_of(int64_t total, int ctas, int64_t unit) {
  const int64_t q = total / ctas, r = total % ctas;
  return (int)(unit < r * (q + 1) ? unit / (q + 1) : r + (unit - r * (q + 1)) / q);
}

// An item, or the part of it that is this CTA's.
struct Item {
  Seq q;
  int32_t seq, head, row0, rows;   // rows: of this block
  int32_t tile, tiles, pieces;     // its key tiles, and their pieces of 64 keys up to the last that is seen
  bool begins, ends;               // with the item's first tile, its last
  int64_t unit0;                   // the item's first unit of all
  int32_t all;                     // units of the whole item
};

// A walk through a CTA's items. Every warp has its own, between items in shared memory: it would take the registers of the
// loops over tiles.
template <typename C>
struct Items {
  int64_t unit, end;
  int s, b, h, off, blocks, n, kt0;  // blocks: -1 before the sequence's are known
  bool opened;                       // the block's tiles are known
  Seq q;
  __device__ __forceinline__ void start(const Share& sh) {
    unit = sh.begin, end = sh.end, s = sh.seq, b = sh.block, h = sh.head, off = sh.off, blocks = -1, opened = false;
  }
  __device__ __forceinline__ bool next(const ChunkArgs& a, Item& it) {
    while (unit < end) {
      while (!opened) {
        if (b == blocks) ++s, b = 0, blocks = -1;  // (units are left, so there is another sequence with rows)
        if (blocks < 0) q = seq_of(a, s), blocks = blocks_of<C>(a, q);
        if (b < blocks) n = block_tiles<C>(a, q, b, kt0), opened = true;
      }
      const int per = n + kItemUnits, take = (int)min((int64_t)(per - off), end - unit);
      const int first = max(0, off - kItemUnits), last = max(0, off + take - kItemUnits);
      const bool head_of_it = off == 0;
      it.q = q, it.seq = s, it.head = h, it.row0 = b * C::kItemRows;
      it.rows = min(C::kItemRows, q.tokens * a.group - it.row0);
      it.tile = kt0 + first, it.tiles = last - first;
      const int seen = keys_end(a, q, token_of(a, it.row0 + it.rows - 1)) - it.tile * C::kKeys;
      it.pieces = min(it.tiles * C::kPieces, (seen + kPiece - 1) / kPiece);
      it.begins = first == 0, it.ends = last == n;
      it.unit0 = unit - off, it.all = per;
      unit += take;
      off += take;
      if (off == per) {
        off = 0;
        if (++h == a.heads) {
          h = 0, ++b, opened = false;
        }
      }
      if (it.tiles > 0 || (head_of_it && it.begins && it.ends)) return true;
    }
    return false;
  }
};

// Finds this CTA's share. All threads; s_units: kSeqChunk values, s_warp: one per warp.
template <typename C>
__device__ void find_share(const ChunkArgs& a, int64_t* s_units, int64_t* s_warp, Share* s_share) {
  constexpr int kWarps = C::kThreadsAll / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t mine = 0;
  for (int s = warp; s < a.S; s += kWarps) {
    const int64_t u = seq_units<C>(a, s);
    if (s < kSeqChunk && lane == 0) s_units[s] = u;
    mine += u;
  }
  if (lane == 0) s_warp[warp] = mine;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += s_warp[w];
  const int64_t want = (total + kMinUnits - 1) / kMinUnits;
  const int ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, want));
  const int c = blockIdx.x;
  const int64_t begin = c < ctas ? share_begin(total, ctas, c) : total, end = c < ctas ? share_begin(total, ctas, c + 1) : total;
  if (tid == 0) *s_share = {begin, end, total, ctas, 0, 0, 0, 0};
  int64_t base = 0;  // units before the chunk
  for (int s0 = 0; s0 < a.S && begin < end; s0 += kSeqChunk) {
    if (s0) {
      __syncthreads();
      for (int s = s0 + warp; s < min(a.S, s0 + kSeqChunk); s += kWarps) {
        const int64_t u = seq_units<C>(a, s);
        if (lane == 0) s_units[s - s0] = u;
      }
    }
    __syncthreads();
    if (warp == 0) {
      for (int i = 0; i < kSeqChunk && s0 + i < a.S; i += 32) {
        const int64_t u = s0 + i + lane < a.S ? s_units[i + lane] : 0;
        int64_t inc = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(kAll, inc, o);
          if (lane >= o) inc += v;
        }
        const bool here = begin >= base + inc - u && begin < base + inc;
        const unsigned who = __ballot_sync(kAll, here);
        if (who) {  // the sequence: now the block and the head
          const int l = __ffs(who) - 1, s = s0 + i + l;
          int64_t rest = begin - (base + __shfl_sync(kAll, inc - u, l));
          const Seq q = seq_of(a, s);
          const int blocks = blocks_of<C>(a, q);
          for (int b0 = 0; b0 < blocks; b0 += 32) {
            int kt0;
            const int64_t per = b0 + lane < blocks ? block_tiles<C>(a, q, b0 + lane, kt0) + kItemUnits : 0;
            int64_t sum = per * a.heads;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int64_t v = __shfl_up_sync(kAll, sum, o);
              if (lane >= o) sum += v;
            }
            const int64_t before = sum - per * a.heads;
            if (rest >= before && rest < sum) {
              s_share->seq = s, s_share->block = b0 + lane;
              s_share->head = (int)((rest - before) / per), s_share->off = (int)((rest - before) % per);
            }
            const int64_t all = __shfl_sync(kAll, sum, 31);
            if (rest < all) break;
            rest -= all;
          }
        }
        base += __shfl_sync(kAll, inc, 31);
        if (base > begin) break;
      }
      if (lane == 0) s_warp[0] = base;
    }
    __syncthreads();
    base = s_warp[0];
    if (base > begin) break;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- decode --

// The multipliers of a block with scale code s for e2m1 pairs times 2^-126: both together are 2^(s - 1).
__device__ __forceinline__ uint32_t first_factor(uint32_t s) { return (min(s, 128u) + 126u) * 0x800080u; }
__device__ __forceinline__ uint32_t second_factor(uint32_t s) { return s <= 128u ? 0x3F803F80u : (s - 1u) * 0x800080u; }

constexpr int kLow = 108, kHigh = 136;  // scale codes of K in (kLow, kHigh] are the f16 exponents 1 .. 28
constexpr float kUnit = 0.0625f;        // a key is its f16 values times this: 2^(kLow + 1 - 127) = 2^-14 * 2^-4

// The codes in two bytes of (w << 4, w) that `sel` names (each byte, then it with its top bit repeated) as BF16
// times 2^-126: E2M1's exponent and mantissa are the lowest bits of BF16's exponent and the highest of its
// mantissa; its 0.5 becomes the subnormal 2^-127.
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t up, uint32_t w, uint32_t sel) {
  uint32_t two;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(two) : "r"(up), "r"(w), "r"(sel));
  return two << 2 & 0x81C081C0u;
}

template <int WORDS>
__device__ __forceinline__ void read_words(const uint8_t* p, uint32_t (&w)[WORDS]) {  // shared memory
  if constexpr (WORDS == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (WORDS == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}

// A decode warp has an eighth of a tile's keys, whose codes lie in `raw` as in the cache. Of 8 keys at a time a lane has
// one key, l & 7, and the words t = l >> 3 ^ key >> 1 of all blocks; of 8 pairs of keys (4 where a warp has no more, and
// half of the blocks) one pair and the words of g = 2u, 2u + 1. With that t the 8 lanes that read or write 16 bytes
// together meet all banks, in the cache's order on one side and the 128-byte swizzle on the other.

__device__ __forceinline__ uint32_t mul2_f16(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A key whose scale codes f16 does not take as they are: its blocks relative to its largest scale, and the power of two
// that its column of S is multiplied by. A block 2^-36 below that is 0. Where all scale codes are 0, which is a key of zeros as a
// rule, the result is negative if this lane's codes are zeros.
template <typename C>
__device__ __noinline__ float wide_key(uint8_t* row, const uint8_t* codes, const uint8_t* scales, int t, int k) {
  constexpr int NB = C::D / 32;
  int top = 0;
#pragma unroll 1
  for (int b = 0; b < NB; ++b) top = max(top, (int)scales[b]);
  if (top == 0) {
    uint32_t any = 0;
#pragma unroll 1
    for (int b = 0; b < NB; ++b) any |= *reinterpret_cast<const uint32_t*>(codes + 4 * b);
    if (!(any & 0x77777777u)) return -ldexpf(1.0f, -127 - 12 + 4);
  }
#pragma unroll 1
  for (int b = 0; b < NB; ++b) {
    const uint32_t f = __half_as_ushort(__float2half_rn(exp2i(max(-126, (int)scales[b] - top + 12)))) * 0x10001u;
    uint32_t e[4];
    e2m1x8_to_f16(*reinterpret_cast<const uint32_t*>(codes + 4 * b), e);
    *reinterpret_cast<uint4*>(row + (b >> 1) * (C::kKeys * 128) + ((((b & 1) * 4 + t) ^ k) << 4)) =
        make_uint4(mul2_f16(e[0], f), mul2_f16(e[1], f), mul2_f16(e[2], f), mul2_f16(e[3], f));
  }
  return top == 255 ? NAN : ldexpf(1.0f, top - 127 - 12 + 4);
}

// K as it is in the tile: [D / 64][keys][128 bytes], 16-byte unit u of a row at u ^ (row & 7), f16. here: the keys have
// a page. factors: of the tile's columns of S. Returns whether any of this warp's is not 1.
template <typename C>
__device__ __forceinline__ bool decode_k(uint8_t* tile, const uint8_t* raw, bool here, int warp, float* factors) {
  constexpr int D = C::D, NB = D / 32;
  const int lane = threadIdx.x & 31, k = lane & 7, t = (lane >> 3) ^ (k >> 1);
  bool wide = false;
#pragma unroll
  for (int i = 0; i < C::kWarpKeys / 8; ++i) {
    const int key = 8 * i + k;
    uint32_t w[NB], sc[(NB + 3) / 4];
    read_words<NB>(raw + key * (D / 2) + t * (D / 8), w);
    const uint8_t* scales = raw + 2 * C::kCodes + key * NB;
    if constexpr (NB == 2)
      sc[0] = *reinterpret_cast<const uint16_t*>(scales);
    else
      read_words<NB / 4>(scales, sc);
    uint8_t* row = tile + (warp * C::kWarpKeys + key) * 128;
    uint32_t least = 0xFFFFFFFFu, most = 0;  // of codes less one (so that 0 is none), and of codes, in pairs
#pragma unroll
    for (int j = 0; j < (NB + 3) / 4; ++j) {
      // exponents of f16 in pairs of blocks (0, 2), (1, 3); 0 for what is below
      const uint32_t even = sc[j] & 0x00FF00FFu, odd = sc[j] >> 8 & 0x00FF00FFu;
      least = __viaddmin_u16x2(even, 0xFFFFFFFFu, least);
      least = __viaddmin_u16x2(odd, 0xFFFFFFFFu, least);
      most = __vmaxu2(__vmaxu2(even, odd), most);
      constexpr uint32_t kLess = (uint32_t)(0x10000 - kLow) * 0x10001u;
      const uint32_t e02 = here ? __viaddmax_s16x2(even, kLess, 0u) << 10 : 0u, e13 = here ? __viaddmax_s16x2(odd, kLess, 0u) << 10 : 0u;
#pragma unroll
      for (int b = 0; b < 4 && 4 * j + b < NB; ++b) {
        const uint32_t f = __byte_perm(b & 1 ? e13 : e02, 0, b & 2 ? 0x3232 : 0x1010);
        uint32_t e[4];
        e2m1x8_to_f16(w[4 * j + b], e);
        *reinterpret_cast<uint4*>(row + ((4 * j + b) >> 1) * (C::kKeys * 128) + ((((b & 1) * 4 + t) ^ k) << 4)) =
            make_uint4(mul2_f16(e[0], f), mul2_f16(e[1], f), mul2_f16(e[2], f), mul2_f16(e[3], f));
      }
    }
    const bool mine = here && (min(least & 0xFFFFu, least >> 16) < kLow || max(most & 0xFFFFu, most >> 16) > kHigh || most == 0);
    float f = 1.0f;
    if (mine) f = wide_key<C>(row, raw + key * (D / 2) + t * (D / 8), scales, t, k);
    if (lane < 8) factors[warp * C::kWarpKeys + 8 * i + k] = fabsf(f);
    wide |= mine && !(f < 0.0f);
  }
  return __any_sync(kAll, wide);
}

// V as it is in the tile: [D / 64][keys][128 bytes] too. Blocks of NaN, or past BF16's range, become 0 and are noted in
// `bad` (a byte per key, a bit per block); returns whether there are any.
template <typename C>
__device__ __forceinline__ bool decode_v(uint8_t* tile, const uint8_t* raw, bool here, uint8_t* bad, int warp) {
  constexpr int D = C::D, NB = D / 32, PAIRS = C::kWarpKeys / 2, NBL = NB * PAIRS / 8;  // NBL: blocks of a lane
  const int lane = threadIdx.x & 31, p = lane % PAIRS;
  const int u = (lane / PAIRS & 3) ^ (PAIRS == 8 ? p >> 1 : p), half = PAIRS == 8 ? 0 : lane >> 4;
  const uint8_t *codes = raw + C::kCodes + p * D + u * (D / 4) + half * 16;
  const uint8_t* scales = raw + 2 * C::kCodes + C::kScales + p * (D / 16) + half * 8;
  uint32_t w[2 * NBL], sc[NBL / 2];
  uint32_t first[NBL], next[NBL];
  read_words<NBL>(codes, first);
  read_words<NBL>(codes + D / 8, next);
#pragma unroll
  for (int b = 0; b < NBL; ++b) w[b] = first[b], w[NBL + b] = next[b];
  read_words<NBL / 2>(scales, sc);
  const int row0 = warp * C::kWarpKeys + 2 * p;
  uint32_t big = 0, mask = 0;
#pragma unroll
  for (int j = 0; j < NBL / 2; ++j) big |= __vmaxu4(sc[j], 0x80808080u) ^ 0x80808080u;
  const bool plain = !big || !here;
  if (!plain) {
#pragma unroll
    for (int b = 0; b < NBL; ++b)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (((sc[b / 2] >> (16 * (b & 1) + 8 * k)) & 255u) >= 253u) mask |= 1u << (8 * k + half * NBL + b);
  }
  if (PAIRS != 8) mask |= __shfl_xor_sync(kAll, mask, 16);
  if (lane < PAIRS) *reinterpret_cast<uint16_t*>(bad + row0) = (uint16_t)mask;
#pragma unroll 1
  for (int n = 0; n < 2; ++n) {
    const int key = PAIRS == 8 ? n ^ (p >> 2) : n, row = row0 + key;  // (8 pairs: half of the lanes store the odd key first)
    const uint32_t sel = key ? 0xD5C4u : 0x9180u;                     // the bytes 0, 1 of w or of w << 4
    uint8_t* at = tile + row * 128;
#pragma unroll
    for (int b = 0; b < NBL; ++b) {
      const uint32_t s = (sc[b / 2] >> (16 * (b & 1) + 8 * key)) & 255u;
      const uint32_t f = plain ? (here ? (s + 126u) * 0x800080u : 0u) : s >= 253u ? 0u : first_factor(s);
      uint32_t e[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t x = w[j * NBL + b], up = x << 4;
        e[2 * j] = mul2_bf16(e2m1_pair(up, x, sel), f);
        e[2 * j + 1] = mul2_bf16(e2m1_pair(up, x, sel + 0x2222u), f);
      }
      if (!plain) {
        const uint32_t g = s >= 253u ? 0u : second_factor(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = mul2_bf16(e[j], g);
      }
      const int block = half * NBL + b;
      *reinterpret_cast<uint4*>(at + (block >> 1) * (C::kKeys * 128) + ((((block & 1) * 4 + u) ^ (row & 7)) << 4)) =
          make_uint4(e[0], e[1], e[2], e[3]);
    }
  }
  return mask != 0;
}

// ---------------------------------------------------------------- kernel --

template <typename C>
struct Shared {  // beside the operands
  // (their readers, and why none falls behind: in the file's first comment)
  uint64_t q_full[C::kQ], q_twin, k_full[C::kSlots][C::kQ], v_full[C::kSlots][C::kQ], k_free[C::kSlots][C::kQ], v_free[C::kSlots][C::kQ];
  uint64_t s_full[C::kQ][2], p_full[C::kQ][2], o_done[C::kQ][2], raw_full[2][kDecodeWarps], drained[C::kQ];  // (raw: K, V)
  int64_t units[kSeqChunk], warp[C::kThreadsAll / 32];
  Items<C> items[C::kThreadsAll / 32];
  Share share;
  uint32_t tmem, failed;
  uint32_t bad_tile[kMeta];                        // number + 1 of the last tile in this place with bad blocks of V
  __align__(8) uint8_t valid[kMeta][kDecodeWarps];  // a decode warp's keys: 1 with a page, 3 with factors besides
  __align__(16) float factors[kMeta][C::kKeys];     // of the columns of S
  float back[2][C::kItemRows];                      // 1 / the power of two of a row's queries, for two items in turn
  __align__(4) uint8_t bad[kMeta][C::kKeys];       // blocks of V that are NaN
  float twin_m[kRows], twin_l[kRows];              // a second row tile's, where both have the same rows
  uint32_t twin_nan[kRows];
};

template <typename C, bool BF16>
__global__ void __launch_bounds__(C::kThreadsAll, 1) kv4_chunk_kernel(const ChunkArgs a) {
  constexpr int D = C::D, KEYS = C::kKeys, SLOTS = C::kSlots;
  extern __shared__ uint4 dyn4[];
  __shared__ Shared<C> sh;
  uint8_t* base = reinterpret_cast<uint8_t*>(dyn4) + (1024 - (smem_addr(dyn4) & 1023)) % 1024;
  uint8_t* const s_q = base;                                    // [row tile][D / 64][128][128 bytes]
  uint8_t* const s_k = s_q + C::kQ * C::kQBytes;    // [slot][tile]
  uint8_t* const s_v = s_k + SLOTS * C::kTile;
  uint8_t* const s_raw = s_v + SLOTS * C::kTile;                // [decode warp]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "n"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 32) {
    for (int i = 0; i < SLOTS; ++i) {
      for (int j = 0; j < C::kQ; ++j) {
        bar_init(smem_addr(&sh.k_full[i][j]), kDecodeWarps), bar_init(smem_addr(&sh.v_full[i][j]), kDecodeWarps);
        bar_init(smem_addr(&sh.k_free[i][j]), 1), bar_init(smem_addr(&sh.v_free[i][j]), 1);
      }
    }
    for (int i = 0; i < kMeta; ++i) sh.bad_tile[i] = 0;
    bar_init(smem_addr(&sh.q_twin), 4);
    for (int i = 0; i < C::kQ; ++i) {
      bar_init(smem_addr(&sh.q_full[i]), 4), bar_init(smem_addr(&sh.drained[i]), 2);
      for (int j = 0; j < 2; ++j) bar_init(smem_addr(&sh.s_full[i][j]), 1), bar_init(smem_addr(&sh.p_full[i][j]), 4), bar_init(smem_addr(&sh.o_done[i][j]), 1);
    }
    for (int i = 0; i < 2 * kDecodeWarps; ++i) bar_init(smem_addr(&sh.raw_full[0][0]) + 8 * i, 1);
    sh.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_before();
  find_share<C>(a, sh.units, sh.warp, &sh.share);  // (ends with a barrier)
  tc_after();
  const uint32_t tmem = sh.tmem;  // S of the row tiles, then their sums
  const Share share = sh.share;
  if (lane == 0) sh.items[warp].start(share);
  __syncwarp();
  auto next_item = [&](Item& item) {
    Items<C> items = sh.items[warp];
    __syncwarp();
    const bool more = items.next(a, item);
    if (lane == 0) sh.items[warp] = items;
    __syncwarp();
    return more;
  };
  Item it;
  bool ok = true;
  uint32_t tile = 0;  // key tiles so far

  if (warp < C::kSoftWarps) {
    // ---------------------------------------------------------- softmax --
    if constexpr (C::kQ == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftRegs));
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = tmem + lanes + t * 2 * kPiece, o_at = tmem + lanes + C::kQ * 2 * kPiece + t * D;
    const uint32_t s_full = smem_addr(&sh.s_full[t][0]), p_full = smem_addr(&sh.p_full[t][0]), o_done = smem_addr(&sh.o_done[t][0]);
    uint32_t s_phase = 0, number = 0;  // a bit per buffer; items with tiles
    uint32_t taken = 0;                // a bit per buffer: whether its pieces so far are an odd number
    // The sums of every piece given so far in a buffer. (s_full of a buffer's next piece says that the one before is done,
    // so at most one phase is open.)
    auto summed = [&](int buffer) { ok = ok && bar_wait(o_done + 8 * buffer, ~(taken >> buffer) & 1u); };
    if (tid == 0) a.split[blockIdx.x] = Split{};
    // The queries of an item, f16 times a power of two per row, the scale's sign among it: this warp's 32 rows, D / 8 lanes to
    // a row, kBatch loads in flight.
    constexpr int kUnits = D / 8, kRowsAtOnce = 32 / kUnits, kBatch = 8;
    // The rows of a group: a twin's are the first group's; a second group of twins has none to bring.
    auto has_twins = [&](const Item& n) { return C::kQ == 2 && n.rows <= kRows; };
    auto bring = [&](const Item& n, uint32_t count) {
      if (n.tiles == 0 || (t == 1 && has_twins(n))) return;
      const int u = lane % kUnits, mine = (warp & 3) * 32 + lane / kUnits, first = has_twins(n) ? 0 : t * kRows;
      float* back = sh.back[count & 1] + first;
      uint8_t* const to = s_q + (first / kRows) * C::kQBytes + (u >> 3) * (kRows * 128);
      const uint16_t* q = a.q + (int64_t)n.q.first * a.ldq + (int64_t)n.head * a.group * D + u * 8;
      int token = token_of(a, n.row0 + first + mine), head = n.row0 + first + mine - token * a.group;
#pragma unroll 1
      for (int row0 = mine; row0 - mine < 32; row0 += kBatch * kRowsAtOnce) {
        uint4 query[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          query[k] = make_uint4(0, 0, 0, 0);
          if (first + row0 + k * kRowsAtOnce < n.rows) query[k] = ld_cached16(q + (int64_t)token * a.ldq + head * D);
          head += kRowsAtOnce;
          while (head >= a.group) head -= a.group, ++token;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int row = row0 + k * kRowsAtOnce;
          uint32_t top = largest_of<BF16>(largest_pairs<BF16>(query[k], kPairs0<BF16>));
#pragma unroll
          for (int o = 1; o < kUnits; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
          const int sigma = shift_of_16<BF16>(top);
          *reinterpret_cast<uint4*>(to + row * 128 + (((u & 7) ^ (row & 7)) << 4)) =
              scaled_f16<BF16>(query[k], copysignf(exp2i(sigma), a.scale_log2));
          if (u == 0) back[row] = exp2i(-sigma);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&sh.q_full[t]));
      if (lane == 0 && has_twins(n) && n.pieces > C::kPieces) bar_arrive(smem_addr(&sh.q_twin));
    };
    Item coming;
    bool more_items = next_item(coming);
    if (more_items) bring(coming, 0);
    while (more_items) {
      it = coming;
      if (tid == 0) {
        if (!it.ends) {  // goes on in the next CTA
          const int c0 = it.begins ? (int)blockIdx.x : cta_of(share.total, share.ctas, it.unit0 + kItemUnits);
          const int c1 = cta_of(share.total, share.ctas, it.unit0 + it.all - 1);
          a.split[blockIdx.x] = {c1 - c0 + 1, (int)blockIdx.x - c0, it.seq, it.head, it.row0, it.rows, {0, 0}};
        }
        if (it.q.len < 0 || (int64_t)it.q.len + it.q.tokens > a.room) flag_invalid(a.err);
      }
      // Few rows: both groups of warps have them, and every other key tile.
      const bool twin = has_twins(it);
      const int above = twin ? 0 : t * kRows;  // rows of the item before this group's
      const int rows = it.rows - above;
      const bool mine = r < rows, busy = (warp & 3) * 32 < rows;
      const int flat = it.row0 + above + (mine ? r : 0), token = token_of(a, flat);
      const int lo = keys_begin(a, it.q, token), hi = keys_end(a, it.q, token);
      // keys that all rows of the group see
      const int all_lo = keys_begin(a, it.q, token_of(a, it.row0 + above + min(rows, kRows) - 1));
      const int all_hi = keys_end(a, it.q, token_of(a, it.row0 + above));
      float m = -INFINITY, l = 0.0f, raw = 0.0f, scale = 0.0f;  // m = raw * scale, rounded
      uint32_t nan = 0;
      const uint32_t tile0 = tile;
      // Tile i from `tile` on, whose sums have begun, so that its values are there: NaN blocks of keys that this row sees.
      auto check = [&](int i) {
        const uint32_t at = tile + i;
        const int k0 = (it.tile + i + (int)(tile - tile0)) * KEYS;
        if (*reinterpret_cast<volatile uint32_t*>(&sh.bad_tile[at % kMeta]) == at + 1)
          for (int key = max(0, lo - k0); key < min(KEYS, hi - k0); ++key) nan |= sh.bad[at % kMeta][key];
      };
      int before = -1;  // the tile before
      for (int n = twin ? t * C::kPieces : 0; n < it.pieces;) {
        const int i = n / C::kPieces, in = n % C::kPieces, buffer = n & 1;
        const uint32_t at = (tile + i) % kMeta;
        ok = ok && bar_wait(s_full + 8 * buffer, s_phase >> buffer & 1u);
        s_phase ^= 1u << buffer;
        __syncwarp();
        tc_after();
        const int k0 = (it.tile + i) * KEYS + in * kPiece;
        if (in == 0) {
          if (before >= 0) {
            check(before);
          } else {  // (the queries are there)
            scale = fabsf(a.scale_log2) * sh.back[number & 1][above + r] * kUnit;
            if (scale == 0.0f) scale = 1.40129846e-45f;  // masked: -inf times it stays -inf; 2^127 times it is nothing
          }
          before = i;
        }
        const uint32_t s_in = s_at + buffer * kPiece, p_bar = p_full + 8 * buffer;
        if (busy) {
          uint32_t x[2][32];
          tmem_load32(s_in, x[0]);
          tmem_load32(s_in + 32, x[1]);
          // a decode warp's byte: a run of 16 keys (two warps to a run where they have 8 keys)
          uint32_t valid4 = *reinterpret_cast<const uint32_t*>(&sh.valid[at][C::kPieces == 2 ? 4 * in : 0]), more = valid4;
          if (C::kPieces == 1) more = *reinterpret_cast<const uint32_t*>(&sh.valid[at][4]);
          const bool whole = k0 >= all_lo && k0 + kPiece <= all_hi && valid4 == 0x01010101u && more == 0x01010101u;
          tmem_wait(x[0]);
          asm volatile("" : WD_R32(x[1]));
          if (!whole) {
            const bool wide = ((valid4 | more) & 0x02020202u) != 0;
            uint32_t valid = ((valid4 & 0x01010101u) * 0x01020408u) >> 24 & 15u;
            if (C::kPieces == 1) {
              valid |= ((more & 0x01010101u) * 0x01020408u) >> 20 & 0xF0u;
              valid = (valid & 1u) | (valid >> 1 & 2u) | (valid >> 2 & 4u) | (valid >> 3 & 8u);
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // the row's keys among these 32
              const int b = max(0, min(32, lo - k0 - 32 * c)), e = max(0, min(32, hi - k0 - 32 * c));
              uint32_t v = (e >= 32 ? kAll : (1u << e) - 1u) & ~(b >= 32 ? kAll : (1u << b) - 1u);
              if (!(valid >> (2 * c) & 1u)) v &= 0xFFFF0000u;
              if (!(valid >> (2 * c) & 2u)) v &= 0x0000FFFFu;
              if (wide) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const float4 f4 = *reinterpret_cast<const float4*>(&sh.factors[at][in * kPiece + 32 * c + j]);
                  x[c][j] = __float_as_uint(__uint_as_float(x[c][j]) * f4.x);
                  x[c][j + 1] = __float_as_uint(__uint_as_float(x[c][j + 1]) * f4.y);
                  x[c][j + 2] = __float_as_uint(__uint_as_float(x[c][j + 2]) * f4.z);
                  x[c][j + 3] = __float_as_uint(__uint_as_float(x[c][j + 3]) * f4.w);
                }
              }
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(v >> j & 1u)) x[c][j] = 0xFF800000u;
            }
          }
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; j += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tops[k] = max3(tops[k], __uint_as_float(x[c][j + 2 * k]), __uint_as_float(x[c][j + 2 * k + 1]));
          const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])), to = top * scale;
          bool moved = false;
          float f = 1.0f;
          if (m == -INFINITY) {
            if (top != -INFINITY) m = to, raw = top;
          } else if (to > m + kSlack) {
            f = exp2_fast((raw - top) * scale);
            m = to, raw = top;
            l *= f;
            moved = mine;  // (rows that are not there hold anything)
          }
          // s scale - m in one step is off by the rounding of m: too much for logits this loud
          const bool loud = mine && fabsf(m) > 1048576.0f && m != -INFINITY;
          float less = m == -INFINITY ? 0.0f : -m;
          if (__any_sync(kAll, moved || loud)) {
            if (__any_sync(kAll, moved)) {  // (not at the item's first piece: m is -inf)
              // the sums of the piece before have to be there
              summed(buffer ^ 1);
              __syncwarp();
              tc_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tmem_load16(o_at + c, o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_store16(o_at + c, o);
              }
            }
            if (__any_sync(kAll, loud)) {
              less = 0.0f;
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) x[c][j] = __float_as_uint(__uint_as_float(x[c][j]) - raw);
            }
          }
          const uint64_t scale2 = pair_of(__float_as_uint(scale), __float_as_uint(scale));
          const uint64_t less2 = pair_of(__float_as_uint(less), __float_as_uint(less));
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              uint32_t u0, u1;
              float r0, r1;
              split_pair(fma2(pair_of(x[c][j], x[c][j + 1]), scale2, less2), u0, u1);
              u0 = __float_as_uint(exp2_fast(__uint_as_float(u0)));
              u1 = __float_as_uint(exp2_fast(__uint_as_float(u1)));
              sums[(j / 2) & 1] = add2(sums[(j / 2) & 1], pair_of(u0, u1));
              p[j / 2] = __byte_perm(u0, u1, 0x7632);
              // what the cut leaves: p - hi
              asm("{.reg .b16 a, b, m;\n\t"
                  "mov.b32 {a, b}, %2;\n\t"
                  "mov.b16 m, 0xBF80;\n\t"
                  "fma.rn.f32.bf16 %0, a, m, %3;\n\t"
                  "fma.rn.f32.bf16 %1, b, m, %4;\n\t}"
                  : "=f"(r0), "=f"(r1)
                  : "r"(p[j / 2]), "f"(__uint_as_float(u0)), "f"(__uint_as_float(u1)));
              p[16 + j / 2] = pack2<true>(r0, r1);
            }
            tmem_store32(s_in + 32 * c, p);
          }
          uint32_t a0, a1, b0, b1;
          split_pair(sums[0], a0, a1);
          split_pair(sums[1], b0, b1);
          l += (__uint_as_float(a0) + __uint_as_float(a1)) + (__uint_as_float(b0) + __uint_as_float(b1));
          tmem_stored();
        }
        tc_before();
        __syncwarp();
        if (lane == 0) bar_arrive(p_bar);
        taken ^= 1u << buffer;
        ++n;
        if (twin && n % C::kPieces == 0) n += C::kPieces;
      }
      tile += it.tiles;
      if (it.tiles) ++number;
      more_items = next_item(coming);
      if (before >= 0) {
        summed(0), summed(1);
        check(before - it.tiles);
      }
      __syncwarp();
      tc_after();
      if (!ok) sh.failed = 1;
      if (*(volatile uint32_t*)&sh.failed) l = NAN;  // a wait that ran out, of any role: no sums to trust
      if (twin) {
        if (t == 1) sh.twin_m[r] = m, sh.twin_l[r] = l, sh.twin_nan[r] = nan;
        tc_before();
        soft_sync(1);
        tc_after();
      }
      // (every product with this item's queries is done)
      if (more_items) bring(coming, number);
      if (twin && t == 1) {
        soft_sync(2);
        continue;
      }
      const bool final = it.begins && it.ends;
      float f0 = 1.0f, f1 = 0.0f;
      const bool second = twin && it.pieces > C::kPieces;  // the other group has sums of these rows
      if (second) {
        const float om = sh.twin_m[r], to = fmaxf(m, om), less = to == -INFINITY ? 0.0f : to;
        f0 = exp2_fast(m - less), f1 = exp2_fast(om - less);
        l = fmaf(sh.twin_l[r], f1, l * f0);
        m = to;
        nan |= sh.twin_nan[r];
      }
      if (busy) {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        const int64_t row = it.q.first + token;
        const int q_head = it.head * a.group + flat - token * a.group;
        float* part = a.parts + ((size_t)blockIdx.x * 2 + (it.begins ? 1 : 0)) * a.part_rows * (D + 2);
        const float w0 = final ? f0 * inv : f0, w1 = final ? f1 * inv : f1;
        auto put = [&](int c, uint32_t(&o)[32]) {  // 32 columns
          if (nan >> (c / 32) & 1u) {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0x7FC00000u;
          }
          if (mine && final) {
            uint4* to = reinterpret_cast<uint4*>(a.out + row * a.ldo + (int64_t)q_head * D + c);
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) h[k] = pack2<BF16>(__uint_as_float(o[j + 2 * k]), __uint_as_float(o[j + 2 * k + 1]));
              to[j / 8] = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else if (mine) {
            uint4* to = reinterpret_cast<uint4*>(part + (size_t)(above + r) * D + c);
#pragma unroll
            for (int j = 0; j < 32; j += 4) to[j / 4] = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < D; c += second ? 32 : 64) {
          uint32_t o[2][32];
          if (it.tiles) {
            tmem_load32(o_at + c, o[0]);
            tmem_load32(second ? o_at + D + c : o_at + c + 32, o[1]);
            tmem_wait(o[0]);
            asm volatile("" : WD_R32(o[1]));
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[0][j] = o[1][j] = 0;
          }
          if (second) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[0][j] = __float_as_uint(fmaf(__uint_as_float(o[1][j]), w1, __uint_as_float(o[0][j]) * w0));
            put(c, o[0]);
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
              for (int j = 0; j < 32; ++j) o[k][j] = __float_as_uint(__uint_as_float(o[k][j]) * w0);
              put(c + 32 * k, o[k]);
            }
          }
        }
        if (mine && final && a.lse)
          a.lse[row * (a.heads * a.group) + q_head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        if (mine && !final) {
          part[(size_t)a.part_rows * D + above + r] = m;
          part[(size_t)a.part_rows * (D + 1) + above + r] = l;
        }
      }
      tc_before();  // the next item's sums go where these were
      if (twin) soft_sync(2);
    }
  } else if (warp < C::kSoftWarps + C::kDecoders) {
    // ----------------------------------------------------------- decode --
    if constexpr (C::kQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kDecodeRegs));
    // Eight warps for K and eight for V; in one row tile's form (D 256) the same eight for both.
    const int w = (warp - C::kSoftWarps) % kDecodeWarps;
    const bool does_k = warp - C::kSoftWarps < kDecodeWarps, does_v = C::kQ == 1 || !does_k;
    const uint32_t raw_k = smem_addr(&sh.raw_full[0][w]), raw_v = smem_addr(&sh.raw_full[1][w]);
    const uint8_t* raw = s_raw + w * C::kRaw;
    uint32_t pending_k = 0, phases_k = 0, pending_own = 0, phases_own = 0;
    uint32_t &pending_v = C::kQ == 2 ? pending_k : pending_own, &phases_v = C::kQ == 2 ? phases_k : phases_own;
    while (next_item(it)) {
      if (!it.tiles) continue;
      const int end = keys_end(a, it.q, token_of(a, it.row0 + it.rows - 1)), begin = keys_begin(a, it.q, token_of(a, it.row0));
      int held = -1;
      // This warp's place in 32 tiles from tile i on: lane has tile i + lane. In runs of 16 keys, -1 without a page.
      auto look_up = [&](int i) {
        const int key = (it.tile + i + lane) * KEYS + w * C::kWarpKeys, run = key & ~15;
        held = -1;
        if (i + lane < it.tiles && run < end && run + 16 > begin) {
          const int page = __ldg(a.table + (int64_t)it.seq * a.max_blocks + (key >> a.page_shift));
          if (page < 0 || page >= a.pages)
            flag_invalid(a.err);
          else
            held = ((page * a.heads + it.head) << (a.page_shift - 4)) + ((key & ((1 << a.page_shift) - 1)) >> 4);
        }
      };
      auto run_of = [&](int i) { return __shfl_sync(kAll, held, i & 31); };
      // The codes and scales of a run, of K (part 0) or V; run -1: nothing.
      constexpr int kPerRun = 16 / C::kWarpKeys;
      auto send = [&](int run, int part, const uint8_t* codes, const uint8_t* scales, uint32_t bar) {
        if (lane == 0) {
          bar_expect(bar, run < 0 ? 0 : C::kCodes + C::kScales);
          if (run >= 0) {
            const int64_t id = (int64_t)run * kPerRun + w % kPerRun;
            bulk_copy(smem_addr(raw) + part * C::kCodes, codes + id * C::kCodes, C::kCodes, bar);
            bulk_copy(smem_addr(raw) + 2 * C::kCodes + part * C::kScales, scales + id * C::kScales, C::kScales, bar);
          }
        }
      };
      look_up(0);
      if constexpr (C::kQ == 1) {  // the queries, which the softmax warps will want soon, to L2 (two row tiles' form lost 1 % by it)
        const int row = w * 32 + lane;
        if (row < it.rows) {
          const int token = token_of(a, it.row0 + row), head = it.head * a.group + it.row0 + row - token * a.group;
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.q + ((int64_t)it.q.first + token) * a.ldq + (int64_t)head * D),
                       "n"(D * 2)
                       : "memory");
        }
      }
      int run_k = run_of(0), run_v = run_k;  // (without keys to decode, run_k is the next tile's)
      if (does_k) send(run_k, 0, a.kc, a.ks, raw_k);
      if (does_v) send(run_v, 1, a.vc, a.vs, raw_v);
      auto filled = [&](uint64_t(&bars)[C::kQ], uint32_t users) {  // what this warp wrote is for the tensor cores
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane < C::kQ && users >> lane & 1u) bar_arrive(smem_addr(&bars[lane]));
      };
      for (int i = 0; i < it.tiles; ++i, ++tile) {
        const uint32_t slot = tile % SLOTS;
        const bool more = i + 1 < it.tiles;
        // a bit per slot and group: who still reads what was there, and the phase of its barrier
        const uint32_t users = C::kQ == 1 ? 1u : it.rows <= kRows ? 1u << (i & 1) : 3u;
        auto await_free = [&](uint64_t(&bars)[SLOTS][C::kQ], uint32_t& pending, uint32_t& phases) {
#pragma unroll
          for (int t = 0; t < C::kQ; ++t) {
            const uint32_t bit = 1u << (slot * 2 + t);
            if (pending & bit) {
              ok = ok && bar_wait(smem_addr(&bars[slot][t]), (phases & bit) != 0);
              phases ^= bit;
            }
          }
          pending = (pending & ~(3u << (slot * 2))) | users << (slot * 2);
          if (!ok) sh.failed = 1;
        };
        if (does_k) {
          ok = bar_wait(raw_k, tile & 1) && ok;  // (whatever was before: the copies have to end)
          await_free(sh.k_free, pending_k, phases_k);
          __syncwarp();
          const bool wide = decode_k<C>(s_k + slot * C::kTile, raw, run_k >= 0, w, sh.factors[tile % kMeta]);
          if (lane == 0) sh.valid[tile % kMeta][w] = (run_k >= 0 ? 1 : 0) | (wide ? 2 : 0);
          filled(sh.k_full[slot], users);  // (every lane has read the codes)
          if (more) {
            if (((i + 1) & 31) == 0) look_up(i + 1);
            run_k = run_of(i + 1);
            send(run_k, 0, a.kc, a.ks, raw_k);
          }
        }
        if (does_v) {
          if (!does_k && more) {
            if (((i + 1) & 31) == 0) look_up(i + 1);
            run_k = run_of(i + 1);
          }
          ok = bar_wait(raw_v, tile & 1) && ok;
          await_free(sh.v_free, pending_v, phases_v);
          __syncwarp();
          if (decode_v<C>(s_v + slot * C::kTile, raw, run_v >= 0, sh.bad[tile % kMeta], w)) sh.bad_tile[tile % kMeta] = tile + 1;
          filled(sh.v_full[slot], users);
          run_v = run_k;
          if (more) send(run_v, 1, a.vc, a.vs, raw_v);
        }
      }
    }
  } else {
    // -------------------------------------------------------------- MMA --
    if constexpr (C::kQ == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kMmaRegs));
    // For each group of softmax warps a warp issues the products with keys, and one those with values: fewer spent longer on
    // issuing and on their barriers than the tensor cores on computing.
    const int t = (warp & 3) % C::kQ;
    const bool sums = (warp & 3) >= C::kQ;
    if ((warp & 3) < 2 * C::kQ) {
      // FP32 sums, f16 operands (bits 7, 10: BF16); N / 8 at bit 17, M / 16 at bit 24; bit 16: B is dim-major
      constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(kRows / 16) << 24);
      constexpr uint32_t kIdescS = kIdesc | ((uint32_t)(kPiece / 8) << 17);
      constexpr uint32_t kIdescO = kIdesc | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(D / 8) << 17);
      // Descriptors, high words: 128-byte swizzle, 1024 bytes from 8 rows (keys) to the next. Low words: the address; K-major
      // 1, dim-major the bytes from 64 dims to the next, a tile's keys.
      constexpr uint32_t kDescHigh = 64u | 1u << 14 | 2u << 29;
      constexpr uint32_t kDescLow = 1u << 16, kLowV = (uint32_t)(KEYS * 128 / 16) << 16;
      const uint32_t q_at = kDescLow + (smem_addr(s_q) >> 4), k_at = kDescLow + (smem_addr(s_k) >> 4), v_at = kLowV + (smem_addr(s_v) >> 4);
      const uint32_t s_at = tmem + t * 2 * kPiece, o_at = tmem + C::kQ * 2 * kPiece + t * D;
      // Piece `in` of the tile in `slot`: S, and the sums.
      auto product = [&](int row_tile, uint32_t slot, int in, int buffer, bool last) {
        const uint32_t s = __shfl_sync(kAll, s_at + buffer * kPiece, 0), q = __shfl_sync(kAll, q_at + row_tile * (C::kQBytes / 16), 0),
                       k = __shfl_sync(kAll, k_at + slot * (C::kTile / 16) + in * (kPiece * 128 / 16), 0);
        if (elected()) {
#pragma unroll
          for (int j = 0; j < D / 16; ++j)
            mma_ss<kDescHigh, kDescHigh, kIdescS>(s, q + (uint32_t)(j / 4) * (kRows * 128 / 16) + (j % 4) * 2,
                                                  k + (uint32_t)(j / 4) * (KEYS * 128 / 16) + (j % 4) * 2, j > 0);
          tc_commit(smem_addr(&sh.s_full[t][buffer]));
          if (last) tc_commit(smem_addr(&sh.k_free[slot][t]));
        }
        __syncwarp();
      };
      auto values = [&](uint32_t slot, int in, int buffer, bool first, bool last) {
        const uint32_t o = __shfl_sync(kAll, o_at, 0), p = __shfl_sync(kAll, s_at + buffer * kPiece, 0),
                       v = __shfl_sync(kAll, v_at + slot * (C::kTile / 16) + in * (kPiece * 128 / 16), 0);
        if (elected()) {
#pragma unroll
          for (int j = 0; j < kPiece / 16; ++j)
#pragma unroll
            for (int term = 0; term < 2; ++term)
              mma_ts<kDescHigh, kIdescO>(o, p + (j / 2) * 32 + term * 16 + (j % 2) * 8, v + j * 128, j + term > 0 || !first);
          tc_commit(smem_addr(&sh.o_done[t][buffer]));
          if (last) tc_commit(smem_addr(&sh.v_free[slot][t]));
        }
        __syncwarp();
      };
      uint32_t phase = 0;                 // of p_full or o_done, a bit per buffer
      uint32_t slot_phase = 0;            // of k_full or v_full, a bit per slot
      uint32_t q_phase = 0;               // of q_full, and of q_twin
      while (next_item(it)) {
        if (!it.tiles) continue;
        const int np = it.pieces;
        const bool twin = C::kQ == 2 && it.rows <= kRows;
        // This group's pieces: all, or those of every other tile.
        const int full = np / (2 * C::kPieces) * C::kPieces, rest = np - 2 * full;
        const int count = !twin ? np : full + (t == 0 ? min(rest, C::kPieces) : max(0, rest - C::kPieces));
        if (!sums && count) {
          const int which = twin && t == 1 ? 1 : 0;
          ok = ok && bar_wait(smem_addr(which ? &sh.q_twin : &sh.q_full[t]), q_phase >> which & 1u);
          q_phase ^= 1u << which;
        }
        // The product of a piece waits for the sums of the piece two before, which had the same columns (at the item's end for
        // the last two, whose columns are the next item's).
        const int steps = sums ? count : count + 2;
#pragma unroll 1
        for (int n = 0; n < steps; ++n) {
          const int buffer = n & 1, i = twin ? (n / C::kPieces * 2 + t) * C::kPieces + n % C::kPieces : n, in = i % C::kPieces;
          const uint32_t slot = (tile + i / C::kPieces) % SLOTS;
          const bool last = in == C::kPieces - 1 || i == np - 1;
          if (in == 0 && n < count) {
            ok = ok && bar_wait(smem_addr(sums ? &sh.v_full[slot][t] : &sh.k_full[slot][t]), slot_phase >> slot & 1u);
            slot_phase ^= 1u << slot;
          }
          if (sums || n >= 2) {
            ok = ok && bar_wait(smem_addr(sums ? &sh.p_full[t][buffer] : &sh.o_done[t][buffer]), phase >> buffer & 1u);
            phase ^= 1u << buffer;
          }
          if (!ok) sh.failed = 1;
          __syncwarp();
          tc_after();
          if (sums)
            values(slot, in, buffer, n == 0, last);
          else if (n < count)
            product(twin ? 0 : t, slot, in, buffer, last);
        }
        tile += it.tiles;
      }
      if (elected()) tc_commit(smem_addr(&sh.drained[t]));
      __syncwarp();
      ok = ok && bar_wait(smem_addr(&sh.drained[t]), 0);
      if (!ok) sh.failed = 1;
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 0) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kTmem));
  }
}

// Joins the parts of the items that several CTAs share: an item with P parts has P - 1 CTAs here (each attending CTA's
// entry names at most one item), which share out its rows. A dependent launch. What it takes is its chain of trips to
// memory, so a CTA asks for all maxima at once, then every thread for four words of sums per part, and where its rows are few
// its threads share out the parts too. (A warp per row, one after the other: 54 us where the rows are 256; this 18, and 11 with
// 1024 threads.)
constexpr int kMostItemRows = 256;
constexpr int kJoinThreads = 1024;
constexpr int kMostWeights = 1024;  // parts of an item times a CTA's rows of it: P (256 / (P - 1) + 1), at most 514

template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) kv4_chunk_join_kernel(const ChunkArgs a) {
  __shared__ float s_m[kMostWeights], s_l[kMostWeights], s_inv[kMostItemRows];
  __shared__ float4 s_sum[kJoinThreads];
  constexpr int kWords = D / 4, kAtOnce = 4;
  const int tid = threadIdx.x;
  wait_prerequisite();
  const Split sp = a.split[blockIdx.x];
  if (sp.parts == 0) return;
  const int c0 = (int)blockIdx.x - sp.index, shares = sp.parts - 1, parts = sp.parts;
  const int r0 = (int)((int64_t)sp.rows * sp.index / shares), n = (int)((int64_t)sp.rows * (sp.index + 1) / shares) - r0;
  if (n == 0) return;
  const size_t size = (size_t)a.part_rows * (D + 2);
  auto part_of = [&](int k) { return a.parts + ((size_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * size; };
  for (int i = tid; i < parts * n; i += kJoinThreads) {
    const int k = i / n, r = i - k * n;
    const float* p = part_of(k) + (size_t)a.part_rows * D + r0 + r;
    s_m[i] = __ldcg(p);
    s_l[i] = __ldcg(p + a.part_rows);
  }
  const Seq q = seq_of(a, sp.seq);
  __syncthreads();
  // What each part weighs.
  if (tid < n) {
    float top = -INFINITY, l = 0.0f;
#pragma unroll 8
    for (int k = 0; k < parts; ++k) top = fmaxf(top, s_m[k * n + tid]);
    const float less = top == -INFINITY ? 0.0f : top;
#pragma unroll 8
    for (int k = 0; k < parts; ++k) {
      const float f = exp2_fast(s_m[k * n + tid] - less);
      l = fmaf(s_l[k * n + tid], f, l);
      s_m[k * n + tid] = f;
    }
    s_inv[tid] = l == 0.0f ? 0.0f : 1.0f / l;
    const int flat = sp.row0 + r0 + tid, token = token_of(a, flat), head = sp.head * a.group + flat - token * a.group;
    if (a.lse)
      a.lse[((int64_t)q.first + token) * (a.heads * a.group) + head] = l == 0.0f ? -INFINITY : (less + log2f(l)) * 0.6931471805599453f;
  }
  __syncthreads();
  auto put = [&](int word, const float4& v) {
    const int r = word / kWords, flat = sp.row0 + r0 + r, token = token_of(a, flat), head = sp.head * a.group + flat - token * a.group;
    const float inv = s_inv[r];
    *reinterpret_cast<uint2*>(a.out + ((int64_t)q.first + token) * a.ldo + (int64_t)head * D + word % kWords * 4) =
        make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
  };
  auto add = [&](float4& v, const float4& x, float f) {
    v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y), v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
  };
  const int words = n * kWords;
  auto word_of = [&](int k, int word) { return __ldcg(reinterpret_cast<const float4*>(part_of(k) + (size_t)r0 * D) + word); };
  if (words * 2 <= kJoinThreads) {
    const int teams = kJoinThreads / words, team = tid / words, word = tid - team * words;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (team < teams) {
#pragma unroll 4
      for (int k = team; k < parts; k += teams) add(v, word_of(k, word), s_m[k * n + word / kWords]);
    }
    s_sum[tid] = v;
    __syncthreads();
    if (team == 0) {
      for (int i = 1; i < teams; ++i) add(v, s_sum[i * words + word], 1.0f);
      put(word, v);
    }
    return;
  }
  for (int base = tid; base < words; base += kJoinThreads * kAtOnce) {
    float4 v[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int k = 0; k < parts; ++k) {
      float4 x[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (base + i * kJoinThreads < words) x[i] = word_of(k, base + i * kJoinThreads);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (base + i * kJoinThreads < words) add(v[i], x[i], s_m[k * n + (base + i * kJoinThreads) / kWords]);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (base + i * kJoinThreads < words) put(base + i * kJoinThreads, v[i]);
  }
}

// ---------------------------------------------------------------- launch --

// Rows of a part, whose sums are 16-byte words.
int64_t part_rows_of(int64_t T, int group) { return T * group < kMostItemRows ? (T * group + 3) / 4 * 4 : kMostItemRows; }

template <typename C, bool BF16>
moe_status launch(ChunkArgs a, cudaStream_t st) {
  auto k = kv4_chunk_kernel<C, BF16>;
  static SmemOnce once;
  moe_status rc = once.allow(k, C::kSmem);
  if (rc != MOE_OK) return rc;
  if (C::kQ == 2) {  // what setmaxnreg shares out has to be there, or its increase would wait for ever
    static const int regs = [&] {
      cudaFuncAttributes attr = {};
      return cudaFuncGetAttributes(&attr, k) == cudaSuccess ? attr.numRegs : 0;
    }();
    if (regs * C::kThreadsAll < C::kRegs) return refuse(MOE_ERR_UNSUPPORTED, "wd_kv4_attend_chunk: built with too few registers");
  }
  // items at most, and units of one at most
  const int64_t items = ((int64_t)a.T * a.group / C::kItemRows + a.S) * a.heads;
  const int64_t seen = (int64_t)a.window + C::kItemRows + 2 * C::kKeys;
  const int64_t most = a.window > 0 && seen < a.room ? seen : a.room, units = (most + C::kKeys - 1) / C::kKeys;
  const int64_t fill = (int64_t)sm_count();  // a CTA has an SM's shared memory
  const unsigned grid = (unsigned)(items < fill && items * (units + kItemUnits) < fill ? items * (units + kItemUnits) : fill);
  k<<<grid, C::kThreadsAll, C::kSmem, st>>>(a);
  rc = launched("wd_kv4_attend_chunk launch");
  if (rc != MOE_OK) return rc;
  if (a.room <= C::kKeys) return MOE_OK;  // items of one key tile, which are in one CTA: nothing to join (12.0 us to 10.9)
  cudaLaunchAttribute dependent = {};
  dependent.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  dependent.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cfg.attrs = &dependent;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_chunk_join_kernel<C::D, BF16>, a);
  if (e != cudaSuccess) {
    set_error("wd_kv4_attend_chunk join launch", e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace wd

extern "C" size_t wd_kv4_attend_chunk_workspace(const wd_kv4_cache* c, int32_t T, int32_t q_heads) {
  using namespace wd;
  if (!c || wd_kv4_cache_bytes(c, WD_KV4_CODES) == 0 || T < 0 || q_heads < 1 || q_heads % c->heads) return 0;
  const int64_t rows = part_rows_of(T, q_heads / c->heads), grid = (int64_t)sm_count();
  return (size_t)(grid * sizeof(Split) + grid * 2 * rows * (c->dim + 2) * 4);
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
  if ((int64_t)c->pages * c->heads * (c->page_size / 16) > 0x7FFFFFFF)  // 1 TB of codes
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend_chunk: the cache has too many pages");
  if (q_heads > 65536) return refuse(MOE_ERR_SHAPE, "wd_kv4_attend_chunk: a token has at most 65536 heads");
  constexpr int64_t kMost = 0x7FFFFFFF - 0xFFFF;
  if ((int64_t)max_blocks * c->page_size >= kMost || (int64_t)T * q_heads >= kMost || S >= kMost)
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend_chunk: block_table's capacity, T * q_heads, or S is too large");
  ChunkArgs a = {};
  a.kc = c->k_codes, a.ks = c->k_scales, a.vc = c->v_codes, a.vs = c->v_scales;
  a.q = static_cast<const uint16_t*>(q), a.out = static_cast<uint16_t*>(out), a.lse = lse, a.err = err;
  a.table = table, a.lens = lens, a.cu = cu;
  a.ldq = ldq, a.ldo = ldo, a.T = T, a.S = S, a.max_blocks = max_blocks, a.pages = c->pages;
  a.page_shift = kv4_page_shift(c->page_size), a.heads = c->heads, a.group = q_heads / c->heads, a.window = window;
  a.room = max_blocks * c->page_size;
  a.scale_log2 = scale * 1.4426950408889634f;
  // round up 2^(32 + shift) / group: exact for numerators below 2^31 (Granlund and Montgomery)
  while ((1u << a.group_shift) < (unsigned)a.group) ++a.group_shift;
  if ((1u << a.group_shift) != (unsigned)a.group) {
    --a.group_shift;
    a.group_mul = (uint32_t)(((1ull << (32 + a.group_shift)) + a.group - 1) / a.group);
  }
  const int64_t grid = (int64_t)sm_count();
  a.split = static_cast<Split*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + grid * sizeof(Split));
  a.part_rows = (int32_t)part_rows_of(T, a.group);
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf16 = type == WD_BF16;
  // <dim, keys of a tile, row tiles>
  if (c->dim == 64) return bf16 ? launch<Config<64, 128, 2>, true>(a, st) : launch<Config<64, 128, 2>, false>(a, st);
  if (c->dim == 128) return bf16 ? launch<Config<128, 128, 2>, true>(a, st) : launch<Config<128, 128, 2>, false>(a, st);
  return bf16 ? launch<Config<256, 64, 1>, true>(a, st) : launch<Config<256, 64, 1>, false>(a, st);
}
