// Where new tokens go in the paged 4-bit cache: shared by the kernels that write and
// read whole tokens (wd_kv4.cu, wd_rope.cu).
#pragma once

#include "wd_block.cuh"
#include "wd_kv4.cuh"

namespace wd {

struct TokenArgs {
  const int32_t *table, *lens, *cu;
  int32_t* err;
  int64_t ldk, ldv;
  int32_t T, S, max_blocks;
  int32_t pages, page_shift, heads;
  int32_t per, chunk;  // tokens of a CTA, pieces of a token in a CTA
};

constexpr int32_t kMostTokens = 0x7FFFFFFF - 0xFFFF;  // tokens, or sequences, of a call are fewer: a run behind the last fits 32 bits
// The arguments' checks, and the work of a CTA.
moe_status check_tokens(const wd_kv4_cache* c, const void* k, const void* v, int32_t type, int64_t ldk, int64_t ldv,
                        int32_t T, const int32_t* table, int32_t max_blocks, const int32_t* lens, const int32_t* cu,
                        int32_t S, const int32_t* err, bool f32_ok);
TokenArgs token_args(const wd_kv4_cache* c, int64_t ldk, int64_t ldv, int32_t T, const int32_t* table,
                     int32_t max_blocks, const int32_t* lens, const int32_t* cu, int32_t S, int32_t* err);

namespace {  // device code: one copy per translation unit

// The place of a new token; `before`, `behind`: the tokens next to it are new ones of
// its sequence too. page -1: ignored (behind cu[S]) or left out (flagged). pos: its position,
// -1 where it is ignored or its sequence's length is negative.
struct Place {
  int32_t page, slot;
  bool before, behind;
  int64_t pos;
};
// A new token with an even slot and the next one where that is new too (`both`), or one
// with an odd slot whose neighbour is none of its sequence's new ones: what shares bytes of V. j: the first's.
struct Pair {
  int32_t page, slot, j;
  bool both;
};
constexpr int kMostPer = 64;
constexpr int kResident = 5;  // CTAs of an SM: a pair's four loads in flight take 48 registers

__device__ __forceinline__ Place place_of(const TokenArgs& a, int tok, bool here) {
  Place p = {-1, 0, false, false, -1};
  int s = tok, first = tok, end = tok + 1;
  if (!here || tok >= a.T) return p;
  if (a.cu) {
    if (tok >= __ldg(a.cu + a.S) || tok < __ldg(a.cu)) return p;
    int lo = 0, hi = a.S - 1;  // the last s with cu[s] <= tok
    while (lo < hi) {
      const int mid = lo + ((hi - lo + 1) >> 1);
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
  if (len >= 0) p.pos = pos;
  if (len >= 0 && block < a.max_blocks) p.page = __ldg(a.table + (int64_t)s * a.max_blocks + block);
  p.slot = (int)(pos & ((1 << a.page_shift) - 1));
  if (p.page < 0 || p.page >= a.pages) {
    p.page = -1;
    flag_invalid(a.err);
  }
  return p;
}

// The pairs that begin in a CTA's tokens, in order; returns their number. All threads. s_pos: the
// tokens' positions, where they are asked for.
__device__ __forceinline__ int find_pairs(const TokenArgs& a, int tok0, Pair* s_pair, int64_t* s_pos = nullptr) {
  __shared__ uint32_t s_first[kMostPer / 32];
  const int tid = threadIdx.x;
  Place p;
  uint32_t first = 0;
  if (tid < kMostPer) {  // whole warps
    p = place_of(a, tok0 + tid, tid < a.per);
    if (s_pos) s_pos[tid] = p.pos;
    first = __ballot_sync(0xFFFFFFFFu, p.page >= 0 && !((p.slot & 1) && p.before));
    if ((tid & 31) == 0) s_first[tid >> 5] = first;
  }
  __syncthreads();
  int pairs = 0;
#pragma unroll
  for (int n = 0; n < kMostPer / 32; ++n) pairs += __popc(s_first[n]);
  if (tid < kMostPer && (first >> (tid & 31)) & 1u) {
    int at = __popc(first & ((1u << (tid & 31)) - 1u));
#pragma unroll
    for (int n = 0; n < kMostPer / 32; ++n) at += n < tid >> 5 ? __popc(s_first[n]) : 0;
    s_pair[at] = {p.page, p.slot, tid, !(p.slot & 1) && p.behind};
  }
  __syncthreads();
  return pairs;
}

// The (pair, piece) of a thread's i-th item, i = threadIdx.x, + kThreads, ...
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

}  // namespace
}  // namespace wd
