// What the root-mean-square norm and the layer norm share: sums over a block,
// weights, the outputs of a row and the columns' sums of the gradients.
#pragma once

#include "f8_common.cuh"
#include "ptx.cuh"

namespace mmagb {
namespace {

// Sum of two values over the block, the same in every thread.  `buf` holds
// 64 floats; calls in turn use different buffers, so one barrier is enough.
// VOTE: *any becomes whether any thread's is set.
template <bool VOTE = false>
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* buf,
                                             bool* any = nullptr) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) {
    if constexpr (VOTE) *any = __any_sync(0xffffffffu, *any);
    return make_float2(a, b);
  }
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
  if constexpr (VOTE)
    *any = __syncthreads_or(*any);
  else
    __syncthreads();
  // every thread adds the warps' sums in their order (independent reads; a
  // second tree of shuffles took longer)
  a = 0.f;
  b = 0.f;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    a += buf[w].x;
    b += buf[w].y;
  }
  return make_float2(a, b);
}

// The weights of vector v: of the input's type or FP32.
template <class T>
__device__ __forceinline__ void load_weight(const void* W, bool w32, int64_t v,
                                            int64_t n, float (&f)[Vec<T>::kN]) {
  constexpr int E = Vec<T>::kN;
  if (!w32) {
    load_row(static_cast<const T*>(W), v, n, f);
  } else {
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
      float t[4];
      load_row(static_cast<const float*>(W), v * (E / 4) + j, n, t);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[4 * j + i] = t[i];
    }
  }
}

// The bias, or zeros where there is none.
template <class T>
__device__ __forceinline__ void load_bias(const void* B, bool w32, int64_t v,
                                          int64_t n, float (&f)[Vec<T>::kN]) {
  if (B) {
    load_weight<T>(B, w32, v, n, f);
  } else {
#pragma unroll
    for (int j = 0; j < Vec<T>::kN; ++j) f[j] = 0.f;
  }
}

// Row `row` of the outputs: h times rstd, weight and bias, in the input's type,
// in 8 bits or both, and (PUT_H) h itself.
// `weights` gives those and the bias of the thread's vector i.
template <class T, int VPT, bool TAIL, bool CENTRE, bool PUT_H, class F>
__device__ __forceinline__ void norm_out(const NormProblem& p, int64_t row,
                                         float (&h)[VPT][Vec<T>::kN], float rstd,
                                         F&& weights) {
  constexpr int E = Vec<T>::kN;
  constexpr int kLanes = kScaleBlock / E;  // lanes that share a block
  const int64_t n = p.N;
  // y replaces h; m: the largest magnitude of each vector's scale block
  float m[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int64_t v = threadIdx.x + i * blockDim.x;
    const bool live = v * E < n;
    if (PUT_H && p.H && live)
      store_row<T, TAIL>(static_cast<T*>(p.H) + row * p.ldh, v, n, h[i]);
    float w[E], b[E];
    weights(i, v, w, b);
    m[i] = 0.f;
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      float2 y = __fmul2_rn(make_float2(h[i][j], h[i][j + 1]), make_float2(rstd, rstd));
      if constexpr (CENTRE)
        y = __ffma2_rn(y, make_float2(w[j], w[j + 1]), make_float2(b[j], b[j + 1]));
      else
        y = __fmul2_rn(y, make_float2(w[j], w[j + 1]));
      // columns past the end (rstd may be infinite or NaN) do not count
      h[i][j] = TAIL && v * E + j >= n ? 0.f : y.x;
      h[i][j + 1] = TAIL && v * E + j + 1 >= n ? 0.f : y.y;
      m[i] = abs_max(m[i], h[i][j], h[i][j + 1]);
    }
    if (!live) m[i] = 0.f;
    if (p.Y && live)
      store_row<T, TAIL>(static_cast<T*>(p.Y) + row * p.ldy, v, n, h[i]);
  }
  if (p.Q) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1)
        m[i] = abs_max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
    // the thread's VPT scales and their reciprocals, each made by another
    // lane of the block's group
    const int mine = threadIdx.x % kLanes % 4;
    float mm = m[0];
#pragma unroll
    for (int i = 1; i < VPT; ++i) mm = mine == i ? m[i] : mm;
    const float s = block_scale<false>(mm, p.pow2);
    const Divisor by(s);
    const int lane0 = threadIdx.x & 31 & ~(kLanes - 1);
    if (threadIdx.x % kLanes < VPT) {
      const int64_t b = (threadIdx.x + int64_t(mine) * blockDim.x) / kLanes;
      if (b * kScaleBlock < n) p.S[row * p.s_row + b * p.s_blk] = s;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t v = threadIdx.x + i * blockDim.x;
      const Divisor d = by.from(lane0 + i);
      if (v * E < n)
        store_f8<false, E, TAIL>(static_cast<uint8_t*>(p.Q) + row * p.ldq, v, n,
                                 h[i], d);
    }
  }
}

// out[c] = sum of part[g][c] over g, of n columns (those from n1 on to out1): 32
// columns per block, 32 rows of
// threads that each add up every 32nd part, two loads at once (more got in
// each other's way: backward pass of 8190 x 5000 62.7 us, four 63.7, sixteen
// 69.9).  Starts beside the end of the kernel that makes the parts.
__global__ void __launch_bounds__(1024)
    sum_parts_kernel(const float* __restrict__ part, int parts, int64_t n,
                     float* __restrict__ out, int64_t n1, float* __restrict__ out1) {
  __shared__ float t[32][33];
  const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.f;
  grid_dependency_wait();
  for (int from = threadIdx.y; from < parts; from += 2 * 32) {
    float v[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int g = from + i * 32;
      v[i] = g < parts && col < n ? part[g * n + col] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) s += v[i];
  }
  t[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = t[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && c < n) {
    if (c < n1)
      out[c] = s;
    else
      out1[c - n1] = s;
  }
}

// Adds up `grid` rows of n columns, beside the end of the kernel that makes them.
inline mma_status_t sum_parts(const Ctx& ctx, const float* part, int grid, int64_t n,
                              float* out, int64_t n1, float* out1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((n + 31) / 32), 1, 1);
  cfg.blockDim = dim3(32, 32, 1);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, sum_parts_kernel, part, grid, n, out, n1, out1);
  const cudaError_t last = cudaGetLastError();
  return e == cudaSuccess && last == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

}  // namespace
}  // namespace mmagb
