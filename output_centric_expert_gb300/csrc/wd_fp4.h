// What the two matvec kernels share: the packed tile sizes and the arguments.
#pragma once

#include "warp_decode_block.h"

namespace wd {

constexpr int kTileRows = 16;   // rows of a packed tile: one MMA row tile
constexpr int kTileCols = 128;  // columns of a packed tile: 4 scale blocks
constexpr int kTileCodes = kTileRows * kTileCols / 2;    // 1024 bytes
constexpr int kTileScales = kTileRows * kTileCols / 32;  // 64 bytes

struct MvArgs {
  const uint8_t *codes, *scales;
  const uint16_t* x;
  void* y;
  int64_t ldx, ldy;
  int32_t B, y_type, N, K;
  int32_t tok0;   // first token of this launch
  int32_t chunk;  // stream kernel: column tiles of x staged at a time; all of them where that fits
  int32_t batch;  // stream kernel: row tiles of a CTA whose sums wait in shared memory
};

// Columns that the tensor-memory kernel takes for `tokens` tokens (wd_fp4_tc.cu), and
// its launch: tokens tok0 .. B-1, in runs of 64 or fewer.
int tc_most_columns(int tokens);
moe_status launch_tc(MvArgs a, bool bf16, cudaStream_t st);

}  // namespace wd
