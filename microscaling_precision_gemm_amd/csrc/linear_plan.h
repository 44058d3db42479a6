// linear_plan.h -- which kernel of linear.hip takes a product of M tokens and N
// columns.  Plain C++: the tests read the rule from here too.
#pragma once
#include <stdint.h>

namespace mxk {

// operands straight to registers; tiles whose K the waves share out; tiles through a
// common ring (128 x 128 and 256 x 256)
enum class LinearKernel { kDirect, kSplit32x32, kSplit32x64, kSplit64x32, kSplit64x64, kTile128, kTile256 };

inline LinearKernel linear_kernel(int64_t M, int64_t N) {
  auto tiles = [&](int64_t bm, int64_t bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  // One token, and few over few columns: operands straight to registers (1 x 8192
  // x 4096 4-bit 7.8 us, through LDS 9.2; 16 x 4096 x 14336 8-bit 25 and 34).
  // Lanes of one row read X in pieces of 16 bytes there, which for more columns
  // costs more than LDS does (16 x 28672 x 4096 4-bit 40 us, through LDS 24).
  if (M <= 4 || (M <= 16 && N <= 4096)) return LinearKernel::kDirect;
  // Up to two rounds of 256 tiles of 64 x 64, and 64 tokens in any case, share K out
  // among the waves: larger tiles leave CUs idle (256 x 4096 x 4096 4-bit 15 us, 128
  // x 128 tiles 33; 384 x 4096 x 4096 27 and 36), and beyond that they take less time
  // (600 x 4096 x 4096 39 and 36; 4096 x 520 x 2080 34 and 29).  Among those the
  // smallest tile that fills no more than one round: more CUs share the weights (32
  // x 7168 x 2048 with 32 x 32 7.2 us, with 32 x 64 8.3; 128 x 4096 x 4096 with 64 x
  // 32 11.4, with 64 x 64 13.8; 48 x 4096 x 14336 8-bit with 64 x 32 44.6, with 32 x
  // 32 and twice the waves 31.9), but a second round costs more (32 x 10000 x 4096
  // with 32 x 32 18.3 us, with 32 x 64 13.1; 48 x 9000 x 4096 8-bit with 64 x 32
  // 28.5, with 64 x 64 22.1).
  if (M <= 32) return tiles(32, 32) <= 256 ? LinearKernel::kSplit32x32 : LinearKernel::kSplit32x64;
  if (M <= 64 || tiles(64, 64) <= 512) {
    if (tiles(32, 32) <= 256) return LinearKernel::kSplit32x32;
    return tiles(64, 32) <= 256 ? LinearKernel::kSplit64x32 : LinearKernel::kSplit64x64;
  }
  // A round of 256 tiles of 256 x 256 takes the card 1 / 0.61 times as long as one
  // of 512 tiles of 128 x 128, which is half the work (2048 x 4096 x 4096 77 us in
  // half a round of the large, 66 in one of the small; 4096 x 7168 x 2048 115 in
  // two, 147 in four).
  const int64_t large = (tiles(256, 256) + 255) / 256, small = (tiles(128, 128) + 511) / 512;
  return 100 * large <= 61 * small ? LinearKernel::kTile256 : LinearKernel::kTile128;
}

}  // namespace mxk
