// wd_kv4_attend_chunk: attention of several new tokens per sequence over the paged
// 4-bit cache, which holds them already.
//
// Mathematics. Rows are (token, query head) pairs that share a KV head. With z = scale q.k
// in units of log 2, one pass over the keys keeps m, l = sum 2^(z_j - m) and acc = sum
// 2^(z_j - m) v_j; partial results join as l = sum l_i 2^(m_i - m), acc likewise. m follows
// the row's maximum only when that is more than 2^kSlack above it, so acc is hardly ever
// rescaled.
//   S = Q K^T and acc += P V: tcgen05.mma kind::f16 with BF16 operands, 128 rows. K and V are
//   decoded to BF16, which holds every E2M1 code times every E8M0 scale up to 6 * 2^125
//   exactly; so are queries (F16: as two BF16 terms). P is two BF16 terms, the second what
//   the cut of the first left: 16 bits, and FP32's range of exponents, as in wd_kv4_attend.
//
// Work. A CTA has kQ tiles of 128 rows against tiles of kKeys keys. Its warps:
//   4 per row tile   softmax: a thread has a row. S comes from tensor memory, P goes back in
//                    its place (16 columns of first terms, 16 of second for 32 keys)
//   4                decode: K and V codes from global memory through registers into shared
//                    memory (K-major and dim-major, 128-byte swizzle); the queries
//   1                issues the MMAs
// While one row tile is in its softmax the tensor cores have the other's products.
// All (sequence, row block, KV head) items are cut into units of one key tile; CTA c of G
// takes the c-th contiguous share of all units, found from the lengths on the device. An
// item that several CTAs share leaves its parts in the workspace, and a dependent launch
// joins them in CTA order.
#include <cmath>

#include "wd_block.cuh"
#include "wd_kv4.cuh"

namespace wd {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr float kSlack = 8.0f;
constexpr int kRows = 128;       // of a row tile
constexpr int kItemUnits = 2;    // what an item costs beside its key tiles, in tiles
constexpr int kMinUnits = 3;     // of a CTA, on average, unless it has an item to itself
constexpr uint32_t kWaitLimit = 1u << 20;
constexpr int kSeqChunk = 512;   // sequences whose units are in shared memory at a time
constexpr int kMeta = 4;         // key tiles whose page masks are kept

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
  float scale_log2;  // positive
  uint32_t flip;     // what a pair of queries is xored with: the scale's sign
  uint32_t keep;     // and then masked: 0 for a scale of 0
};

template <int D_, int KEYS, int Q, int TERMS, int NK_, int NV_, int CTAS>
struct Config {
  static constexpr int D = D_, kKeys = KEYS, kQ = Q, kTerms = TERMS, kNK = NK_, kNV = NV_, kCtas = CTAS;
  static constexpr int kItemRows = Q * kRows;
  static constexpr int kSoftWarps = 4 * Q, kThreadsAll = (4 * Q + 5) * 32;
  static constexpr int kQBytes = kRows * D * 2;        // of a term of a row tile
  static constexpr int kTile = KEYS * D * 2;           // of K or V
  static constexpr int kSmem = 1024 + Q * TERMS * kQBytes + (NK_ + NV_) * kTile;
  static constexpr int kCols = Q * (KEYS + D);
  static constexpr int kTmem = kCols <= 256 ? 256 : 512;
  static_assert(kCols <= 512 && kTmem * CTAS <= 512 && kSmem * CTAS <= 226 * 1024, "fits an SM");
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
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// D (+)= A B: both by shared-memory descriptors, or A in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
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
  const int lo = keys_begin(a, q, b * C::kItemRows / a.group);
  const int hi = keys_end(a, q, (min((b + 1) * C::kItemRows, rows) - 1) / a.group);
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
  int32_t tile, tiles;             // its key tiles
  bool begins, ends;               // with the item's first tile, its last
  int64_t unit0;                   // the item's first unit of all
  int32_t all;                     // units of the whole item
};

// A walk through a CTA's items. Every role has its own.
template <typename C>
struct Items {
  const ChunkArgs& a;
  int64_t unit, end;
  int s, b, h, off, blocks, n, kt0;
  Seq q;
  __device__ Items(const ChunkArgs& args, const Share& sh)
      : a(args), unit(sh.begin), end(sh.end), s(sh.seq), b(sh.block), h(sh.head), off(sh.off) {
    if (unit < end) open_seq(), open_block();
  }
  __device__ __forceinline__ void open_seq() {
    q = seq_of(a, s);
    blocks = blocks_of<C>(a, q);
  }
  __device__ __forceinline__ void open_block() {
    n = block_tiles<C>(a, q, b, kt0);
  }
  __device__ __forceinline__ bool next(Item& it) {
    while (unit < end) {
      while (b == blocks) {  // (units are left, so there is another sequence with rows)
        ++s, b = 0;
        open_seq();
        if (blocks) open_block();
      }
      const int per = n + kItemUnits, take = (int)min((int64_t)(per - off), end - unit);
      const int first = max(0, off - kItemUnits), last = max(0, off + take - kItemUnits);
      const bool head_of_it = off == 0;
      it.q = q, it.seq = s, it.head = h, it.row0 = b * C::kItemRows;
      it.rows = min(C::kItemRows, q.tokens * a.group - it.row0);
      it.tile = kt0 + first, it.tiles = last - first;
      it.begins = first == 0, it.ends = last == n;
      it.unit0 = unit - off, it.all = per;
      unit += take;
      off += take;
      if (off == per) {
        off = 0;
        if (++h == a.heads) {
          h = 0, ++b;
          if (b < blocks) open_block();
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

// The codes in two bytes of (w << 4, w) that `sel` names (each byte, then it with its top bit repeated) as BF16
// times 2^-126: E2M1's exponent and mantissa are the lowest bits of BF16's exponent and the highest of its
// mantissa; its 0.5 becomes the subnormal 2^-127.
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t up, uint32_t w, uint32_t sel) {
  uint32_t two;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(two) : "r"(up), "r"(w), "r"(sel));
  return two << 2 & 0x81C081C0u;
}

template <int WORDS>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[WORDS], int at = 0) {
  if constexpr (WORDS == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + 4 * i));
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
}

// A decode warp has a quarter of a tile's keys. K: lane (l & 7, t = l >> 3) has of 8 keys at a time the words (t, all
// blocks); V: of 8 pairs of keys at a time those of g = 2u, 2u + 1, u = l >> 3. So the 8 lanes that store together
// have 8 rows of 128 bytes, and the swizzle spreads them over all banks.
template <typename C>
struct KRegs {
  static constexpr int NB = C::D / 32, kSteps = C::kKeys / 32;
  uint32_t w[kSteps][NB], s[kSteps][(NB + 3) / 4];
};
template <typename C>
struct VRegs {
  static constexpr int NB = C::D / 32, kSteps = C::kKeys / 64;
  uint32_t w[kSteps][2 * NB], s[kSteps][NB / 2];
};

// run(i): the 16-key run i of this warp, -1 where it has no page.
template <typename C, typename F>
__device__ __forceinline__ void load_k(const ChunkArgs& a, KRegs<C>& r, F run) {
  constexpr int D = C::D, NB = KRegs<C>::NB;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < KRegs<C>::kSteps; ++i) {
    const int id = run(i / 2);
#pragma unroll
    for (int j = 0; j < NB; ++j) r.w[i][j] = 0;
#pragma unroll
    for (int j = 0; j < (NB + 3) / 4; ++j) r.s[i][j] = 0;
    if (id >= 0) {
      const int64_t key = (int64_t)id * 16 + (i & 1) * 8 + (lane & 7);
      load_words<NB>(a.kc + key * (D / 2) + (lane >> 3) * (D / 8), r.w[i]);
      if constexpr (NB == 2)
        r.s[i][0] = __ldg(reinterpret_cast<const uint16_t*>(a.ks + key * 2));
      else if constexpr (NB == 4)
        r.s[i][0] = __ldg(reinterpret_cast<const uint32_t*>(a.ks + key * 4));
      else
        load_words<2>(a.ks + key * 8, r.s[i]);
    }
  }
}
template <typename C, typename F>
__device__ __forceinline__ void load_v(const ChunkArgs& a, VRegs<C>& r, F run) {
  constexpr int D = C::D, NB = VRegs<C>::NB;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < VRegs<C>::kSteps; ++i) {
    const int id = run(i);
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) r.w[i][j] = 0;
#pragma unroll
    for (int j = 0; j < NB / 2; ++j) r.s[i][j] = 0;
    if (id >= 0) {
      const int64_t pair = (int64_t)id * 8 + (lane & 7);
      load_words<2 * NB>(a.vc + pair * D + (lane >> 3) * (D / 4), r.w[i]);
      if constexpr (NB == 2)
        r.s[i][0] = __ldg(reinterpret_cast<const uint32_t*>(a.vs + pair * 4));
      else
        load_words<NB / 2>(a.vs + pair * (D / 16), r.s[i]);
    }
  }
}

// Decoded K into its tile: [D / 64][keys][128 bytes], 16-byte unit u of a row at u ^ (row & 7).
template <typename C>
__device__ __forceinline__ void store_k(uint8_t* tile, const KRegs<C>& r) {
  constexpr int NB = KRegs<C>::NB;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, t = lane >> 3;
  const int row0 = warp * (C::kKeys / 4) + (lane & 7);
#pragma unroll
  for (int i = 0; i < KRegs<C>::kSteps; ++i) {
    uint8_t* row = tile + (row0 + 8 * i) * 128;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint32_t s = (r.s[i][b / 4] >> (8 * (b & 3))) & 255u, w = r.w[i][b], up = w << 4;
      const uint32_t f = s == 255u ? 0x7FC07FC0u : first_factor(s);
      uint32_t e[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) e[j] = mul2_bf16(e2m1_pair(up, w, 0xC480 + 0x1111 * j), f);
      if (s > 128u) {
        const uint32_t g = second_factor(s);
#pragma unroll
        for (int j = 0; j < 4; ++j) e[j] = mul2_bf16(e[j], g);
      }
      *reinterpret_cast<uint4*>(row + (b >> 1) * (C::kKeys * 128) + ((((b & 1) * 4 + t) ^ (lane & 7)) << 4)) =
          make_uint4(e[0], e[1], e[2], e[3]);
    }
  }
}

// Decoded V into its tile: [D / 64][keys][128 bytes] too. Blocks of NaN, or past BF16's range, become 0 and are noted in
// `bad` (a byte per key, a bit per block); returns whether there are any.
template <typename C>
__device__ __forceinline__ bool store_v(uint8_t* tile, const VRegs<C>& r, uint8_t* bad) {
  constexpr int NB = VRegs<C>::NB;
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3, u = lane >> 3;
  const int odd = (lane >> 2) & 1;  // which key of the pair this lane stores first
  bool any = false;
#pragma unroll
  for (int i = 0; i < VRegs<C>::kSteps; ++i) {
    const int row0 = warp * (C::kKeys / 4) + 16 * i + 2 * (lane & 7);
    uint32_t big = 0, mask[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < NB / 2; ++j) big |= __vmaxu4(r.s[i][j], 0xFCFCFCFCu) ^ 0xFCFCFCFCu;
    if (big) {
      any = true;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (((r.s[i][b / 2] >> (16 * (b & 1) + 8 * k)) & 255u) >= 253u) mask[k] |= 1u << b;
    }
    if (u == 0) *reinterpret_cast<uint16_t*>(bad + row0) = (uint16_t)(mask[0] | mask[1] << 8);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int key = k ^ odd, row = row0 + key;
      const uint32_t sel = key ? 0xD5C4u : 0x9180u;  // the bytes j, j + 1 of w or of w << 4
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t s = (r.s[i][b / 2] >> (16 * (b & 1) + 8 * key)) & 255u;
        const uint32_t f = s >= 253u ? 0u : first_factor(s);
        uint32_t e[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t w = r.w[i][j * NB + b], up = w << 4;
          e[2 * j] = mul2_bf16(e2m1_pair(up, w, sel), f);
          e[2 * j + 1] = mul2_bf16(e2m1_pair(up, w, sel + 0x2222u), f);
        }
        if (s > 128u) {
          const uint32_t g = s >= 253u ? 0u : second_factor(s);
#pragma unroll
          for (int j = 0; j < 4; ++j) e[j] = mul2_bf16(e[j], g);
        }
        *reinterpret_cast<uint4*>(tile + (b >> 1) * (C::kKeys * 128) + row * 128 + ((((b & 1) * 4 + u) ^ (row & 7)) << 4)) =
            make_uint4(e[0], e[1], e[2], e[3]);
      }
    }
  }
  return any;
}

// ---------------------------------------------------------------- kernel --

template <typename C>
struct Shared {  // beside the operands
  uint64_t q_full, q_free, k_full[C::kNK], k_free[C::kNK], v_full[C::kNV], v_free[C::kNV];
  uint64_t s_full[C::kQ], p_full[C::kQ], o_done[C::kQ], drained;
  int64_t units[kSeqChunk], warp[C::kThreadsAll / 32];
  Share share;
  uint32_t tmem, failed;
  uint32_t bad_tile[C::kNV];                       // number + 1 of the last tile in the slot with bad blocks of V
  __align__(4) uint8_t valid[kMeta][4];            // runs with a page, by decode warp
  __align__(4) uint8_t bad[C::kNV][C::kKeys];      // blocks of V that are NaN
};

template <typename C, bool BF16>
__global__ void __launch_bounds__(C::kThreadsAll, C::kCtas) kv4_chunk_kernel(const ChunkArgs a) {
  constexpr int D = C::D, KEYS = C::kKeys;
  extern __shared__ uint4 dyn4[];
  __shared__ Shared<C> sh;
  uint8_t* base = reinterpret_cast<uint8_t*>(dyn4) + (1024 - (smem_addr(dyn4) & 1023)) % 1024;
  uint8_t* const s_q = base;                                    // [row tile][term][D / 64][128][128 bytes]
  uint8_t* const s_k = s_q + C::kQ * C::kTerms * C::kQBytes;    // [slot][tile]
  uint8_t* const s_v = s_k + C::kNK * C::kTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem)), "n"(C::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 32) {
    bar_init(smem_addr(&sh.q_full), 128);
    bar_init(smem_addr(&sh.q_free), 1);
    for (int i = 0; i < C::kNK; ++i) bar_init(smem_addr(&sh.k_full[i]), 128), bar_init(smem_addr(&sh.k_free[i]), 1);
    for (int i = 0; i < C::kNV; ++i) {
      bar_init(smem_addr(&sh.v_full[i]), 128), bar_init(smem_addr(&sh.v_free[i]), 1);
      sh.bad_tile[i] = 0;
    }
    for (int i = 0; i < C::kQ; ++i) {
      bar_init(smem_addr(&sh.s_full[i]), 1), bar_init(smem_addr(&sh.p_full[i]), 128);
      bar_init(smem_addr(&sh.o_done[i]), 1);
    }
    bar_init(smem_addr(&sh.drained), 1);
    sh.failed = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_before();
  find_share<C>(a, sh.units, sh.warp, &sh.share);  // (ends with a barrier)
  tc_after();
  const uint32_t tmem = sh.tmem;  // S of the row tiles, then their sums
  const Share share = sh.share;
  Items<C> items(a, share);
  Item it;
  bool ok = true;
  uint32_t tile = 0;  // key tiles so far

  if (warp < C::kSoftWarps) {
    // ---------------------------------------------------------- softmax --
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t s_at = tmem + lanes + t * KEYS, o_at = tmem + lanes + C::kQ * KEYS + t * D;
    const uint32_t s_full = smem_addr(&sh.s_full[t]), p_full = smem_addr(&sh.p_full[t]), o_done = smem_addr(&sh.o_done[t]);
    uint32_t s_phase = 0, o_phase = 0;
    if (tid == 0) a.split[blockIdx.x] = Split{};
    while (items.next(it)) {
      if (tid == 0) {
        if (!(it.begins && it.ends) && !it.ends) {  // goes on in the next CTA
          const int c0 = it.begins ? (int)blockIdx.x : cta_of(share.total, share.ctas, it.unit0 + kItemUnits);
          const int c1 = cta_of(share.total, share.ctas, it.unit0 + it.all - 1);
          a.split[blockIdx.x] = {c1 - c0 + 1, (int)blockIdx.x - c0, it.seq, it.head, it.row0, it.rows, {0, 0}};
        }
        if (it.q.len < 0 || (int64_t)it.q.len + it.q.tokens > a.room) flag_invalid(a.err);
      }
      const int rows = it.rows - t * kRows;  // of this row tile, and of the warp below
      if (rows <= 0) {
        tile += it.tiles;
        continue;
      }
      const bool mine = r < rows, busy = (warp & 3) * 32 < rows;
      const int flat = it.row0 + t * kRows + (mine ? r : 0), token = flat / a.group;
      const int lo = keys_begin(a, it.q, token), hi = keys_end(a, it.q, token);
      // keys that all rows of the tile see
      const int all_lo = keys_begin(a, it.q, (it.row0 + t * kRows + min(rows, kRows) - 1) / a.group);
      const int all_hi = keys_end(a, it.q, (it.row0 + t * kRows) / a.group);
      float m = -INFINITY, l = 0.0f, raw = 0.0f;  // m = raw * scale, rounded
      uint32_t nan = 0;
      for (int i = 0; i < it.tiles; ++i, ++tile) {
        ok = ok && bar_wait(s_full, s_phase);
        s_phase ^= 1;
        __syncwarp();
        tc_after();
        const int k0 = (it.tile + i) * KEYS;
        if (busy) {
          const uint32_t valid4 = *reinterpret_cast<const uint32_t*>(sh.valid[tile % kMeta]);
          constexpr int kRuns = KEYS / 64;  // 16-key runs of a decode warp
          uint32_t valid = 0;
#pragma unroll
          for (int w = 0; w < 4; ++w) valid |= ((valid4 >> (8 * w)) & ((1u << kRuns) - 1u)) << (w * kRuns);
          const bool whole = k0 >= all_lo && k0 + KEYS <= all_hi && valid == (1u << (KEYS / 16)) - 1u;
          // the row's keys among 32 from column c on
          auto seen = [&](int c) {
            const int b = max(0, min(32, lo - k0 - c)), e = max(0, min(32, hi - k0 - c));
            uint32_t v = (e >= 32 ? kAll : (1u << e) - 1u) & ~(b >= 32 ? kAll : (1u << b) - 1u);
            if (!(valid >> (c / 16) & 1u)) v &= 0xFFFF0000u;
            if (!(valid >> (c / 16) & 2u)) v &= 0x0000FFFFu;
            return v;
          };
          float top = -INFINITY;
          uint32_t x[2][32];
#pragma unroll
          for (int c = 0; c < KEYS; c += 64) {
            tmem_load32(s_at + c, x[0]);
            tmem_load32(s_at + c + 32, x[1]);
            tmem_wait(x[0]);
            asm volatile("" : WD_R32(x[1]));
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (!whole) {
                const uint32_t v = seen(c + 32 * half);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!(v >> j & 1u)) x[half][j] = 0xFF800000u;
              }
              float p0 = -INFINITY, p1 = -INFINITY;
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                p0 = fmaxf(p0, __uint_as_float(x[half][j]));
                p1 = fmaxf(p1, __uint_as_float(x[half][j + 1]));
              }
              top = fmaxf(top, fmaxf(p0, p1));
            }
          }
          const float to = top * a.scale_log2;
          bool moved = false;
          float f = 1.0f;
          if (m == -INFINITY) {
            if (top != -INFINITY) m = to, raw = top;
          } else if (to > m + kSlack) {
            f = exp2_fast((raw - top) * a.scale_log2);
            m = to, raw = top;
            l *= f;
            moved = i > 0 && mine;  // (rows that are not there hold anything)
          }
          if (__any_sync(kAll, moved)) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              tmem_load32(o_at + c, x[0]);
              tmem_wait(x[0]);
#pragma unroll
              for (int j = 0; j < 32; ++j) x[0][j] = __float_as_uint(__uint_as_float(x[0][j]) * f);
              tmem_store32(o_at + c, x[0]);
            }
          }
          // s scale - m in one step is off by the rounding of m: too much for logits this loud
          const bool loud = __any_sync(kAll, mine && fabsf(m) > 1048576.0f && m != -INFINITY);
          const float less = m == -INFINITY || loud ? 0.0f : -m;
          float sum0 = 0.0f, sum1 = 0.0f;
          tmem_load32(s_at, x[0]);
#pragma unroll
          for (int c = 0; c < KEYS; c += 32) {
            uint32_t(&now)[32] = x[(c / 32) & 1];
            tmem_wait(now);
            if (c + 32 < KEYS) tmem_load32(s_at + c + 32, x[(c / 32 + 1) & 1]);
            if (!whole) {
              const uint32_t v = seen(c);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!(v >> j & 1u)) now[j] = 0xFF800000u;
            }
            if (loud) {
#pragma unroll
              for (int j = 0; j < 32; ++j) now[j] = __float_as_uint(__uint_as_float(now[j]) - raw);
            }
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float p0 = exp2_fast(fmaf(__uint_as_float(now[j]), a.scale_log2, less));
              const float p1 = exp2_fast(fmaf(__uint_as_float(now[j + 1]), a.scale_log2, less));
              sum0 += p0;
              sum1 += p1;
              const uint32_t u0 = __float_as_uint(p0), u1 = __float_as_uint(p1);
              p[j / 2] = __byte_perm(u0, u1, 0x7632);
              p[16 + j / 2] = pack2<true>(p0 - __uint_as_float(u0 & 0xFFFF0000u), p1 - __uint_as_float(u1 & 0xFFFF0000u));
            }
            tmem_store32(s_at + c, p);
          }
          l += sum0 + sum1;
          tmem_stored();
        }
        const uint32_t slot = tile % C::kNV;
        ok = ok && bar_wait(smem_addr(&sh.v_full[slot]), (tile / C::kNV) & 1);
        if (*reinterpret_cast<volatile uint32_t*>(&sh.bad_tile[slot]) == tile + 1)
          for (int key = max(0, lo - k0); key < min(KEYS, hi - k0); ++key) nan |= sh.bad[slot][key];
        tc_before();
        bar_arrive(p_full);
      }
      if (it.tiles) {
        ok = ok && bar_wait(o_done, o_phase);
        o_phase ^= 1;
      }
      __syncwarp();
      tc_after();
      if (!ok) sh.failed = 1, l = NAN;
      const bool final = it.begins && it.ends;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      const int64_t row = it.q.first + token;
      const int q_head = it.head * a.group + flat % a.group;
      float* part = a.parts + ((size_t)blockIdx.x * 2 + (it.begins ? 1 : 0)) * a.part_rows * (D + 2);
      if (busy) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t x[32];
          if (it.tiles) {
            tmem_load32(o_at + c, x);
            tmem_wait(x);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = 0;
          }
          if (nan >> (c / 32) & 1u) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = 0x7FC00000u;
          }
          if (mine && final) {
            uint4* to = reinterpret_cast<uint4*>(a.out + row * a.ldo + (int64_t)q_head * D + c);
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                o[k] = pack2<BF16>(__uint_as_float(x[j + 2 * k]) * inv, __uint_as_float(x[j + 2 * k + 1]) * inv);
              to[j / 8] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          } else if (mine) {
            uint4* to = reinterpret_cast<uint4*>(part + (size_t)(t * kRows + r) * D + c);
#pragma unroll
            for (int j = 0; j < 32; j += 4) to[j / 4] = make_uint4(x[j], x[j + 1], x[j + 2], x[j + 3]);
          }
          __syncwarp();
        }
        if (mine && final && a.lse)
          a.lse[row * (a.heads * a.group) + q_head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        if (mine && !final) {
          part[(size_t)a.part_rows * D + t * kRows + r] = m;
          part[(size_t)a.part_rows * (D + 1) + t * kRows + r] = l;
        }
        tc_before();  // the next item's sums go where these were
      }
    }
  } else if (warp < C::kSoftWarps + 4) {
    // ----------------------------------------------------------- decode --
    const int w = warp - C::kSoftWarps, dt = tid - C::kSoftWarps * 32;
    constexpr int kRuns = KEYS / 64, kAhead = 32 / kRuns;  // runs of this warp in a tile, tiles whose pages a warp holds
    uint32_t number = 0;  // items with tiles
    while (items.next(it)) {
      if (!it.tiles) continue;
      const int end = keys_end(a, it.q, (it.row0 + it.rows - 1) / a.group), begin = keys_begin(a, it.q, it.row0 / a.group);
      int held = -1;
      auto pages = [&](int i) {  // lane: run lane % kRuns of tile i + lane / kRuns
        const int j = i + lane / kRuns, key = (it.tile + j) * KEYS + w * (KEYS / 4) + (lane % kRuns) * 16;
        held = -1;
        if (j < it.tiles && key < end && key + 16 > begin) {
          const int page = __ldg(a.table + (int64_t)it.seq * a.max_blocks + (key >> a.page_shift));
          if (page < 0 || page >= a.pages)
            flag_invalid(a.err);
          else
            held = ((page * a.heads + it.head) << (a.page_shift - 4)) + ((key & ((1 << a.page_shift) - 1)) >> 4);
        }
      };
      pages(0);
      KRegs<C> kr;
      VRegs<C> vr;
      auto run_of = [&](int i) {
        return [&, i](int n) { return __shfl_sync(kAll, held, (i % kAhead) * kRuns + n); };
      };
      load_k<C>(a, kr, run_of(0));
      load_v<C>(a, vr, run_of(0));
      uint32_t on = __ballot_sync(kAll, held >= 0);  // runs with a page, of the tiles in `held`
      if (number) ok = ok && bar_wait(smem_addr(&sh.q_free), (number - 1) & 1);
      ++number;
      // the queries: as they are (BF16), or as two terms (F16), times the scale's sign
      constexpr int kUnits = D / 8;
#pragma unroll 4
      for (int n = dt; n < it.rows * kUnits; n += 128) {
        const int row = n / kUnits, u = n % kUnits, flat = it.row0 + row, token = flat / a.group;
        uint4 v = ld_cached16(a.q + (int64_t)(it.q.first + token) * a.ldq + (int64_t)(it.head * a.group + flat - token * a.group) * D + u * 8);
        v.x = (v.x ^ a.flip) & a.keep, v.y = (v.y ^ a.flip) & a.keep, v.z = (v.z ^ a.flip) & a.keep, v.w = (v.w ^ a.flip) & a.keep;
        uint8_t* to = s_q + (row / kRows) * C::kTerms * C::kQBytes + (u >> 3) * (kRows * 128) + (row % kRows) * 128 + (((u & 7) ^ (row & 7)) << 4);
        if constexpr (BF16) {
          *reinterpret_cast<uint4*>(to) = v;
        } else {
          float f[8];
          unpack8<false>(v, f);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            hi[k] = pack2<true>(f[2 * k], f[2 * k + 1]);
            lo[k] = pack2<true>(f[2 * k] - bf16_lo(hi[k]), f[2 * k + 1] - bf16_hi(hi[k]));
          }
          *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(to + C::kQBytes) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      bar_arrive(smem_addr(&sh.q_full));
      for (int i = 0; i < it.tiles; ++i, ++tile) {
        const uint32_t ks = tile % C::kNK, kn = tile / C::kNK, vs = tile % C::kNV, vn = tile / C::kNV;
        if (kn) ok = ok && bar_wait(smem_addr(&sh.k_free[ks]), (kn - 1) & 1);
        store_k<C>(s_k + ks * C::kTile, kr);
        if (lane == 0) sh.valid[tile % kMeta][w] = (uint8_t)((on >> ((i % kAhead) * kRuns)) & ((1u << kRuns) - 1u));
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        bar_arrive(smem_addr(&sh.k_full[ks]));
        const bool more = i + 1 < it.tiles;
        if (more && (i + 1) % kAhead == 0) {
          pages(i + 1);
          on = __ballot_sync(kAll, held >= 0);
        }
        if (more) load_k<C>(a, kr, run_of(i + 1));
        if (vn) ok = ok && bar_wait(smem_addr(&sh.v_free[vs]), (vn - 1) & 1);
        if (store_v<C>(s_v + vs * C::kTile, vr, sh.bad[vs])) sh.bad_tile[vs] = tile + 1;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        bar_arrive(smem_addr(&sh.v_full[vs]));
        if (more) load_v<C>(a, vr, run_of(i + 1));
      }
    }
  } else if (lane == 0) {  // (the others wait at the end)
    // -------------------------------------------------------------- MMA --
    // BF16 operands, FP32 sums; N / 8 at bit 17, M / 16 at bit 24; bit 16: B is dim-major
    constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kRows / 16) << 24);
    constexpr uint32_t kIdescS = kIdesc | ((uint32_t)(KEYS / 8) << 17), kIdescO = kIdesc | (1u << 16) | ((uint32_t)(D / 8) << 17);
    // K-major, 128-byte swizzle, 1024 bytes from 8 rows to the next
    constexpr uint64_t kDesc = ((uint64_t)1 << 16) | ((uint64_t)64 << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
    // dim-major: from 64 dims to the next a tile's keys, 1024 bytes from 8 keys to the next
    constexpr uint64_t kDescV = ((uint64_t)(KEYS * 128 / 16) << 16) | ((uint64_t)64 << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
    const uint32_t q_at = smem_addr(s_q) >> 4, k_at = smem_addr(s_k) >> 4, v_at = smem_addr(s_v) >> 4;
    auto product = [&](int t, uint32_t slot) {  // S of row tile t
#pragma unroll
      for (int term = 0; term < C::kTerms; ++term)
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const uint32_t in = (j % 4) * 2;
          mma_ss(tmem + t * KEYS,
                 kDesc | (q_at + (uint32_t)((t * C::kTerms + term) * C::kQBytes + (j / 4) * kRows * 128) / 16 + in),
                 kDesc | (k_at + (slot * C::kTile + (uint32_t)(j / 4) * KEYS * 128) / 16 + in), kIdescS, term + j > 0);
        }
    };
    auto values = [&](int t, uint32_t slot, bool first) {  // its sums
#pragma unroll
      for (int j = 0; j < KEYS / 16; ++j)
#pragma unroll
        for (int term = 0; term < 2; ++term)
          mma_ts(tmem + C::kQ * KEYS + t * D, tmem + t * KEYS + (j / 2) * 32 + term * 16 + (j % 2) * 8,
                 kDescV | (v_at + (slot * C::kTile + (uint32_t)j * 2048) / 16), kIdescO, !first || j + term > 0);
    };
    uint32_t number = 0, p_phase[C::kQ] = {};
    while (items.next(it)) {
      if (!it.tiles) continue;
      ok = ok && bar_wait(smem_addr(&sh.q_full), number & 1);
      ++number;
      ok = ok && bar_wait(smem_addr(&sh.k_full[tile % C::kNK]), (tile / C::kNK) & 1);
      tc_after();
#pragma unroll
      for (int t = 0; t < C::kQ; ++t)
        if (it.rows > t * kRows) {
          product(t, tile % C::kNK);
          tc_commit(smem_addr(&sh.s_full[t]));
        }
      tc_commit(smem_addr(&sh.k_free[tile % C::kNK]));
      if (it.tiles == 1) tc_commit(smem_addr(&sh.q_free));
      for (int i = 0; i < it.tiles; ++i, ++tile) {
        const bool more = i + 1 < it.tiles;
        const uint32_t vs = tile % C::kNV, ks = (tile + 1) % C::kNK;
        ok = ok && bar_wait(smem_addr(&sh.v_full[vs]), (tile / C::kNV) & 1);
        if (more) ok = ok && bar_wait(smem_addr(&sh.k_full[ks]), ((tile + 1) / C::kNK) & 1);
#pragma unroll
        for (int t = 0; t < C::kQ; ++t)
          if (it.rows > t * kRows) {
            ok = ok && bar_wait(smem_addr(&sh.p_full[t]), p_phase[t]);
            p_phase[t] ^= 1;
            tc_after();
            values(t, vs, i == 0);
            if (more) {
              product(t, ks);
              tc_commit(smem_addr(&sh.s_full[t]));
            } else {
              tc_commit(smem_addr(&sh.o_done[t]));
            }
          }
        tc_commit(smem_addr(&sh.v_free[vs]));
        if (more) tc_commit(smem_addr(&sh.k_free[ks]));
        if (i + 2 == it.tiles) tc_commit(smem_addr(&sh.q_free));
      }
    }
    tc_commit(smem_addr(&sh.drained));
    ok = ok && bar_wait(smem_addr(&sh.drained), 0);
    if (!ok) sh.failed = 1;
  }
  __syncwarp();
  __syncthreads();
  if (warp == 0) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(C::kTmem));
  }
}

// Joins the parts of the items that several CTAs share: an item with P parts has P - 1 CTAs here (each attending CTA's
// entry names at most one item), which share out its rows; a warp takes a row. A dependent launch.
template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) kv4_chunk_join_kernel(const ChunkArgs a) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_prerequisite();
  const Split sp = a.split[blockIdx.x];
  if (sp.parts == 0) return;
  const int c0 = (int)blockIdx.x - sp.index, shares = sp.parts - 1;
  const size_t size = (size_t)a.part_rows * (D + 2);
  const Seq q = seq_of(a, sp.seq);
  auto part_of = [&](int k) { return a.parts + ((size_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * size; };
  constexpr int V = D / 32;
  for (int r = (int)((int64_t)sp.rows * sp.index / shares) + warp; r < (int)((int64_t)sp.rows * (sp.index + 1) / shares);
       r += kWarpsPerCta) {
    float top = -INFINITY;
    for (int k = lane; k < sp.parts; k += 32) top = fmaxf(top, __ldcg(part_of(k) + (size_t)a.part_rows * D + r));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
    const float less = top == -INFINITY ? 0.0f : top;
    float l = 0.0f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll 4
    for (int k = 0; k < sp.parts; ++k) {
      const float* p = part_of(k);
      const float f = exp2_fast(__ldcg(p + (size_t)a.part_rows * D + r) - less);
      l = fmaf(__ldcg(p + (size_t)a.part_rows * (D + 1) + r), f, l);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(__ldcg(p + (size_t)r * D + lane + 32 * i), f, acc[i]);
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int flat = sp.row0 + r, token = flat / a.group, head = sp.head * a.group + flat - token * a.group;
    const int64_t row = q.first + token;
#pragma unroll
    for (int i = 0; i < V; ++i)
      store_elem(a.out, BF16 ? WD_BF16 : WD_F16, row * a.ldo + (int64_t)head * D + lane + 32 * i, acc[i] * inv);
    if (a.lse && lane == 0) a.lse[row * (a.heads * a.group) + head] = l == 0.0f ? -INFINITY : (less + log2f(l)) * 0.6931471805599453f;
  }
}

// ---------------------------------------------------------------- launch --

constexpr int kMostCtas = 2;      // per SM
constexpr int kMostItemRows = 256;

// Rows of a part, whose sums are 16-byte words.
int64_t part_rows_of(int64_t T, int group) { return T * group < kMostItemRows ? (T * group + 3) / 4 * 4 : kMostItemRows; }

template <typename C, bool BF16>
moe_status launch(ChunkArgs a, cudaStream_t st) {
  auto k = kv4_chunk_kernel<C, BF16>;
  static SmemOnce once;
  moe_status rc = once.allow(k, C::kSmem);
  if (rc != MOE_OK) return rc;
  // items at most, and units of one at most
  const int64_t items = ((int64_t)a.T * a.group / C::kItemRows + a.S) * a.heads;
  const int64_t seen = (int64_t)a.window + C::kItemRows + 2 * C::kKeys;
  const int64_t most = a.window > 0 && seen < a.room ? seen : a.room, units = (most + C::kKeys - 1) / C::kKeys;
  const int64_t fill = (int64_t)sm_count() * C::kCtas;
  const unsigned grid = (unsigned)(items < fill && items * (units + kItemUnits) < fill ? items * (units + kItemUnits) : fill);
  k<<<grid, C::kThreadsAll, C::kSmem, st>>>(a);
  rc = launched("wd_kv4_attend_chunk launch");
  if (rc != MOE_OK) return rc;
  cudaLaunchAttribute dependent = {};
  dependent.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  dependent.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
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
  const int64_t rows = part_rows_of(T, q_heads / c->heads), grid = (int64_t)sm_count() * kMostCtas;
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
  constexpr int64_t kMost = 0x7FFFFFFF - 0xFFFF;
  if ((int64_t)max_blocks * c->page_size >= kMost || (int64_t)T * q_heads >= kMost)
    return refuse(MOE_ERR_SHAPE, "wd_kv4_attend_chunk: block_table's capacity, or T * q_heads, is too large");
  ChunkArgs a = {};
  a.kc = c->k_codes, a.ks = c->k_scales, a.vc = c->v_codes, a.vs = c->v_scales;
  a.q = static_cast<const uint16_t*>(q), a.out = static_cast<uint16_t*>(out), a.lse = lse, a.err = err;
  a.table = table, a.lens = lens, a.cu = cu;
  a.ldq = ldq, a.ldo = ldo, a.T = T, a.S = S, a.max_blocks = max_blocks, a.pages = c->pages;
  a.page_shift = kv4_page_shift(c->page_size), a.heads = c->heads, a.group = q_heads / c->heads, a.window = window;
  a.room = max_blocks * c->page_size;
  const float z = scale * 1.4426950408889634f;
  a.scale_log2 = z == 0.0f ? 1.0f : std::fabs(z);
  a.flip = std::signbit(z) ? 0x80008000u : 0u;
  a.keep = z == 0.0f ? 0u : ~0u;
  const int64_t grid = (int64_t)sm_count() * kMostCtas;
  a.split = static_cast<Split*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + grid * sizeof(Split));
  a.part_rows = (int32_t)part_rows_of(T, a.group);
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf16 = type == WD_BF16;
  // <dim, keys of a tile, row tiles, terms of a query, slots of K, of V, CTAs per SM>
  const bool deep = (int64_t)T * a.group > (int64_t)S * kRows;  // more than one row tile per sequence
  if (c->dim == 64) {
    if (deep) return bf16 ? launch<Config<64, 128, 2, 1, 2, 2, 1>, true>(a, st) : launch<Config<64, 128, 2, 2, 2, 2, 1>, false>(a, st);
    return bf16 ? launch<Config<64, 128, 1, 1, 2, 2, 2>, true>(a, st) : launch<Config<64, 128, 1, 2, 2, 2, 2>, false>(a, st);
  }
  if (c->dim == 128) {
    if (deep) return bf16 ? launch<Config<128, 128, 2, 1, 2, 2, 1>, true>(a, st) : launch<Config<128, 128, 2, 2, 1, 1, 1>, false>(a, st);
    return bf16 ? launch<Config<128, 128, 1, 1, 1, 1, 2>, true>(a, st) : launch<Config<128, 64, 1, 2, 1, 1, 2>, false>(a, st);
  }
  return bf16 ? launch<Config<256, 64, 1, 1, 2, 2, 1>, true>(a, st) : launch<Config<256, 64, 1, 2, 1, 1, 1>, false>(a, st);
}
