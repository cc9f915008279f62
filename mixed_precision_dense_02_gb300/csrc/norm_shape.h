// The launch of the norm's gradient for rows of `vectors` 16-byte vectors:
// plain host code, by itself so that it can be checked over all widths.
#pragma once

#include <stdint.h>

namespace mmagb {

struct NormBackShape {
  int vpt;      // vectors per thread: 1, 2, 4 (0: the kernel for wide rows)
  int threads;  // per block
  int per_sm;   // blocks that run at once on an SM; the grid is that many
  int stages;   // rows in the ring, at least two
};

constexpr int64_t kNormBackMostVectors = 2048;

// As many blocks per SM as fit: three of up to 320 threads, two of up to 512
// (64 registers a thread with one or two vectors), one with four vectors (up
// to 128 registers).  The ring takes the block's share of the SM's 228 KB, up
// to four rows of h, dy and (three tensors) the residual's gradient.
// Measured, BF16 with it: 8192 x 8192 94 us, by the kernel for wide rows 411;
// 8192 x 6000 68 us, with blocks for three per SM where two run at once 90;
// 4096 x 16384 102 us, with three blocks in turn on an SM 125.
constexpr NormBackShape norm_back_shape(int64_t vectors, int tensors) {
  if (vectors < 1 || vectors > kNormBackMostVectors) return NormBackShape{0, 1024, 1, 0};
  const int vpt = vectors <= 512 ? 1 : vectors <= 1024 ? 2 : 4;
  const int threads = int((vectors + vpt - 1) / vpt + 31) / 32 * 32;
  const int per_sm = vpt == 4 ? 1 : threads <= 320 ? 3 : 2;
  const int64_t room = (per_sm == 3 ? 73 : per_sm == 2 ? 110 : 220) * 1024;
  const int64_t rows = room / (vectors * 16 * tensors);
  return NormBackShape{vpt, threads, per_sm, int(rows < 4 ? rows : 4)};
}

}  // namespace mmagb
