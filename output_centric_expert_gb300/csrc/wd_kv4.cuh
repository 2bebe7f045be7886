// The layout of the 4-bit KV cache, shared by its writers (wd_kv4.cu) and the
// attention that reads it (wd_kv4_attend.cu).
//
// Both layouts are the mma.sync m16n8k16 A fragment's: a lane's bytes of a key
// are contiguous, and a warp's are a dense run.
//   K is the operand of S = K q (rows are keys): lane (g, t) reads of key g the
//   elements 32b + 8t .. + 7 of every block b.
//   V is the operand of out = V^T p (rows are dims, k is keys): lane (g, t) reads
//   of the keys 2t, 2t + 1 the elements 32b + 4g .. + 3 of every block b. A register of
//   the fragment holds one element of both keys, so a byte does too: the low nibble is
//   the even key's, and one conversion decodes the pair (with the keys in bytes of
//   their own, exchanging nibbles was a tenth of the attention's integer work).
#pragma once

#include "warp_decode_block.h"

namespace wd {

moe_status check_kv4(const wd_kv4_cache* c);
int kv4_page_shift(int page_size);

namespace {

// Byte offsets from the start of a (page, head).
template <int D>
__device__ __forceinline__ int k_word(int slot, int t, int b) {
  return slot * (D / 2) + t * (D / 8) + b * 4;
}
template <int D>
__device__ __forceinline__ int v_word(int pair, int g, int b) {
  return pair * D + g * (D / 8) + b * 4;
}
template <int D>
__device__ __forceinline__ int v_scale(int slot, int b) {
  return (slot >> 1) * (D / 16) + b * 2 + (slot & 1);
}

}  // namespace
}  // namespace wd
