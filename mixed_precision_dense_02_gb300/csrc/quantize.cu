// Quantisation to 8-bit floating point (E4M3 or E5M2) with a scale for each
// block of 128 values of a row, or of 128 x 128 values, as it is or
// transposed:
//     s_b = max(max|x| over block b / format's largest value, 2^-126)
//     q = x / s_b, rounded to nearest
// (q is x times the reciprocal of s_b, one rounding more than the quotient;
// the same when s_b is a power of two).
//
// The transposed form serves products that reduce over what is the row index
// here: the weight's transpose for an input gradient, an activation's or
// gradient's transpose for a weight gradient, because 8-bit operands of the
// tensor core are read along the reduction.  Its row blocks run along the
// output's rows, that is, down the input's columns.
//
// Bound by memory: x is read once, q written once.
#include <algorithm>

#include "f8_common.cuh"

namespace mmagb {
namespace {

// Blocks of 1 x 128, not transposed: a group of lanes per block of columns,
// four rows at a time.  The divisions that make a scale and its reciprocal
// are done for the four rows at once, each by another lane of the group (for
// every lane by itself they were a third of all instructions: 16384 x 2048
// BF16 took 37 us).
constexpr int kRowsAtOnce = 4;

template <class T, bool E5M2, bool TAIL>
__global__ void __launch_bounds__(256)
    quantize_rows_kernel(const QuantProblem p) {
  constexpr int E = Vec<T>::kN;
  constexpr int kLanes = kScaleBlock / E;
  const int lane = threadIdx.x & 31;
  const int64_t v = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  const bool live = v * E < p.N;
  const int64_t b = v / kLanes;
  for (int64_t row0 = int64_t(blockIdx.y) * kRowsAtOnce; row0 < p.M;
       row0 += int64_t(gridDim.y) * kRowsAtOnce) {
    float x[kRowsAtOnce][E], m[kRowsAtOnce];
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
      const int64_t row = row0 + i < p.M ? row0 + i : p.M - 1;
      load_row<T, TAIL>(static_cast<const T*>(p.X) + row * p.ldx, v, p.N, x[i]);
    }
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
      m[i] = 0.f;
#pragma unroll
      for (int j = 0; j < E; ++j) m[i] = abs_max(m[i], x[i][j]);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1)
        m[i] = abs_max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
    }
    const int mine = lane & (kRowsAtOnce - 1);
    const float mm = mine & 2 ? (mine & 1 ? m[3] : m[2]) : (mine & 1 ? m[1] : m[0]);
    const float s = block_scale<E5M2>(abs_bits(mm), p.pow2);
    const float inv = __fdiv_rn(1.f, s);
    if (b * kScaleBlock < p.N && lane % kLanes < kRowsAtOnce && row0 + mine < p.M)
      p.S[(row0 + mine) * p.s_row + b * p.s_blk] = s;
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
      const float f = __shfl_sync(0xffffffffu, inv, (lane & ~(kLanes - 1)) + i);
      if (live && row0 + i < p.M)
        store_f8<E5M2, E, TAIL>(static_cast<uint8_t*>(p.Q) + (row0 + i) * p.ldq, v,
                                p.N, x[i], f);
    }
  }
}

// One 128 x 128 tile per block, held in registers: a thread has RPT
// consecutive rows of one vector of E columns.  SQUARE: one scale for the
// tile, else (transposed only) one per column.  The transposed bytes go
// through shared memory, RPT of one column at a time.
template <class T, bool E5M2, bool SQUARE, bool TRANS>
__global__ void __launch_bounds__(256)
    quantize_tile_kernel(const QuantProblem p, int64_t tiles_n) {
  constexpr int E = Vec<T>::kN;
  constexpr int VEC = kScaleBlock / E;  // vectors per tile row
  constexpr int TR = 256 / VEC;         // rows of threads
  constexpr int RPT = kScaleBlock / TR;
  constexpr int PITCH = 144;
  __shared__ uint32_t red[SQUARE ? 8 : TR * kScaleBlock];
  __shared__ float inv_of[SQUARE ? 1 : kScaleBlock];
  __shared__ __align__(16) uint8_t turned[TRANS ? kScaleBlock * PITCH : 16];
  const int64_t tm = blockIdx.x / tiles_n, tn = blockIdx.x - tm * tiles_n;
  const int64_t m0 = tm * kScaleBlock, n0 = tn * kScaleBlock;
  const int c = threadIdx.x % VEC, tr = threadIdx.x / VEC;
  const int64_t v = n0 / E + c;
  float x[RPT][E];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int64_t row = m0 + tr * RPT + i;
    if (row < p.M)
      load_row(static_cast<const T*>(p.X) + row * p.ldx, v, p.N, x[i]);
    else
      for (int j = 0; j < E; ++j) x[i][j] = 0.f;
  }
  float inv[SQUARE ? 1 : E];
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) m = max(m, abs_bits(x[i][j]));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
    for (int w = 0; w < 8; ++w) m = max(m, red[w]);
    const float s = block_scale<E5M2>(m, p.pow2);
    inv[0] = __fdiv_rn(1.f, s);
    if (threadIdx.x == 0)
      p.S[(TRANS ? tn : tm) * p.s_row + (TRANS ? tm : tn) * p.s_blk] = s;
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < RPT; ++i) m = max(m, abs_bits(x[i][j]));
      red[tr * kScaleBlock + c * E + j] = m;
    }
    __syncthreads();
    if (threadIdx.x < kScaleBlock) {
      uint32_t m = 0;
      for (int t = 0; t < TR; ++t) m = max(m, red[t * kScaleBlock + threadIdx.x]);
      const float s = block_scale<E5M2>(m, p.pow2);
      inv_of[threadIdx.x] = __fdiv_rn(1.f, s);
      if (n0 + threadIdx.x < p.N)
        p.S[(n0 + threadIdx.x) * p.s_row + tm * p.s_blk] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) inv[j] = inv_of[c * E + j];
  }
  if constexpr (!TRANS) {
    if (v * E < p.N)
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int64_t row = m0 + tr * RPT + i;
        if (row < p.M)
          store_f8<E5M2>(static_cast<uint8_t*>(p.Q) + row * p.ldq, v, p.N, x[i],
                         inv[0]);
      }
  } else {
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float f = inv[SQUARE ? 0 : j];
      uint32_t w[RPT / 4];
#pragma unroll
      for (int i = 0; i < RPT / 4; ++i)
        w[i] = to_f8x2<E5M2>(x[4 * i][j] * f, x[4 * i + 1][j] * f) |
               (to_f8x2<E5M2>(x[4 * i + 2][j] * f, x[4 * i + 3][j] * f) << 16);
      uint8_t* dst = turned + (c * E + j) * PITCH + tr * RPT;
      if constexpr (RPT == 8)
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    // 16-byte chunks of the output's rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = threadIdx.x + 256 * i;
      const int n = k >> 3, m = (k & 7) * 16;
      if (n0 + n >= p.N || m0 + m >= p.M) continue;
      const uint8_t* src = turned + n * PITCH + m;
      uint8_t* dst = static_cast<uint8_t*>(p.Q) + (n0 + n) * p.ldq + m0 + m;
      if (m0 + m + 16 <= p.M) {
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
      } else {
        for (int b = 0; m0 + m + b < p.M; ++b) dst[b] = src[b];
      }
    }
  }
}

template <class T, bool E5M2>
mma_status_t quantize(const Ctx& ctx, const QuantProblem& p) {
  const int64_t tiles_n = (p.N + kScaleBlock - 1) / kScaleBlock;
  const int64_t tiles = (p.M + kScaleBlock - 1) / kScaleBlock * tiles_n;
  if (p.block_rows == 1 && !p.transpose) {
    constexpr int E = Vec<T>::kN;
    const int64_t vectors = tiles_n * (kScaleBlock / E);  // whole blocks
    const int threads = int(std::min<int64_t>(256, (vectors + 31) / 32 * 32));
    const dim3 grid(unsigned((vectors + threads - 1) / threads),
                    unsigned(std::min<int64_t>(65535, (p.M + kRowsAtOnce - 1) / kRowsAtOnce)));
    if (p.N % E)
      quantize_rows_kernel<T, E5M2, true><<<grid, threads, 0, ctx.stream>>>(p);
    else
      quantize_rows_kernel<T, E5M2, false><<<grid, threads, 0, ctx.stream>>>(p);
  } else {
    if (tiles > INT32_MAX) return MMA_ERR_UNSUPPORTED;
    const unsigned grid = unsigned(tiles);
    if (!p.transpose)
      quantize_tile_kernel<T, E5M2, true, false><<<grid, 256, 0, ctx.stream>>>(p, tiles_n);
    else if (p.block_rows == 128)
      quantize_tile_kernel<T, E5M2, true, true><<<grid, 256, 0, ctx.stream>>>(p, tiles_n);
    else
      quantize_tile_kernel<T, E5M2, false, true><<<grid, 256, 0, ctx.stream>>>(p, tiles_n);
  }
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

template <class T>
mma_status_t by_format(const Ctx& ctx, const QuantProblem& p) {
  return p.e5m2 ? quantize<T, true>(ctx, p) : quantize<T, false>(ctx, p);
}

}  // namespace

mma_status_t launch_quantize_f8(const Ctx& ctx, const QuantProblem& p) {
  switch (p.type) {
    case MMA_BF16: return by_format<__nv_bfloat16>(ctx, p);
    case MMA_F16: return by_format<__half>(ctx, p);
    default: return by_format<float>(ctx, p);
  }
}

}  // namespace mmagb
