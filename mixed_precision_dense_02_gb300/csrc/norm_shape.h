// The launches of the norm's gradient and of the layer norm for rows of `vectors` 16-byte vectors:
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

// The layer norm's rings: rows of x and (two tensors) the residual, or of h, dy and
// (three) the residual's gradient.  Four vectors per thread, fewer in narrow rows;
// the blocks of an SM share its registers (80 or, of the wide ones and the
// gradient's, 128 a thread) and 220 KB, a KB of them beside each ring.
struct NormRingShape {
  int vpt;  // 0: the kernel for wide rows
  int threads, per_sm, stages;
};

constexpr NormRingShape norm_ring(int64_t vectors, int tensors, int vpt, int most_threads,
                                  int most_blocks) {
  const int threads = int((vectors + vpt - 1) / vpt + 31) / 32 * 32;
  const int64_t row = vectors * 16 * tensors;
  int per_sm = most_threads / threads < most_blocks ? most_threads / threads : most_blocks;
  while (per_sm > 1 && (220 / per_sm - 2) * 1024 / row < 2) --per_sm;
  const int64_t rows = (220 / per_sm - 2) * 1024 / row;
  return NormRingShape{vpt, threads, per_sm, int(rows < 4 ? rows : 4)};
}

constexpr NormRingShape layernorm_shape(int64_t vectors, int tensors) {
  if (vectors < 1 || vectors > kNormBackMostVectors) return NormRingShape{0, 0, 0, 0};
  const int vpt = vectors >= 128 ? 4 : vectors >= 64 ? 2 : 1;
  return norm_ring(vectors, tensors, vpt, 512, 16);
}

constexpr NormRingShape layernorm_back_shape(int64_t vectors, int tensors) {
  if (vectors < 1 || vectors > kNormBackMostVectors) return NormRingShape{0, 0, 0, 0};
  const int vpt = vectors > 256 ? 4 : vectors > 64 ? 2 : 1;
  return norm_ring(vectors, tensors, vpt, vpt == 4 ? 512 : vpt == 2 ? 768 : 1024, 8);
}

// Blocks of the layer norm's gradient, each with a share of dw and db: eight per
// SM with narrow rows, else three.
constexpr int64_t layernorm_most_parts(int64_t n) { return n <= 2048 ? 1216 : 456; }

}  // namespace mmagb
