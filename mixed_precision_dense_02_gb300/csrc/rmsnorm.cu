// Root-mean-square norm with the residual's addition and an 8-bit output
// with a scale for each block of 128 columns, and its gradient.
//
// Forward, a row of x, residual r and weight w, all sums in FP32:
//     h = x + r
//     y = h * w / sqrt(mean(h^2) + eps)
//     s_b = max(max|y| over block b / 448, 2^-126),  q = y / s_b in E4M3
// h leaves rounded to the input's type; y is formed from the unrounded sum.
// q is y times the reciprocal of s_b, one rounding more than the quotient;
// with s_b a power of two the two are the same.
//
// Backward, with g = dy * w and the rounded h that the forward stored:
//     dx = g / rms - h * mean(g h) / rms^3 + dr,   dw = sum over rows dy h / rms
// (dx is the gradient of x and of the residual alike; dr the gradient that
// reaches h from elsewhere).
//
// Both are bound by memory: each input is read once and each output written
// once, a row is held in registers between its two uses.  Rows wider than
// the registers hold are read twice (the second time from L2).
#include "f8_common.cuh"

namespace mmagb {
namespace {

// Sum of two values over the block, the same in every thread.  `buf` holds
// 64 floats; calls in turn use different buffers, so one barrier is enough.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* buf) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return make_float2(a, b);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const float2 v = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
  a = v.x;
  b = v.y;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
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

// One row per block; VPT 16-byte vectors per thread are kept in registers
// (VPT = 0: none, the row is read again).
template <class T, int VPT>
__global__ void __launch_bounds__(1024)
    rmsnorm_kernel(const NormProblem p, bool w32) {
  constexpr int E = Vec<T>::kN;
  constexpr int kLanes = kScaleBlock / E;  // lanes that share a block
  __shared__ float2 red[32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.X) + row * p.ldx;
  const T* r = p.R ? static_cast<const T*>(p.R) + row * p.ldr : nullptr;
  T* hrow = p.H ? static_cast<T*>(p.H) + row * p.ldh : nullptr;
  T* yrow = p.Y ? static_cast<T*>(p.Y) + row * p.ldy : nullptr;
  uint8_t* qrow = p.Q ? static_cast<uint8_t*>(p.Q) + row * p.ldq : nullptr;
  auto load = [&](int64_t v, float (&h)[E]) {
    load_row(x, v, p.N, h);
    if (r) {
      float t[E];
      load_row(r, v, p.N, t);
#pragma unroll
      for (int j = 0; j < E; ++j) h[j] += t[j];
    }
  };
  auto emit = [&](int64_t v, const float (&h)[E], float rstd) {
    float y[E];
    load_weight<T>(p.W, w32, v, p.N, y);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      y[j] = h[j] * rstd * y[j];
      // columns past the end (rstd may be infinite or NaN) do not count
      if (v * E + j >= p.N) y[j] = 0.f;
      m = max(m, abs_bits(y[j]));
    }
    const bool live = v * E < p.N;
    if (yrow && live) store_row(yrow, v, p.N, y);
    if (!qrow) return;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
      m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float s = block_scale<false>(m, p.pow2);
    if (!live) return;
    store_f8<false>(qrow, v, p.N, y, __fdiv_rn(1.f, s));
    if (threadIdx.x % kLanes == 0)
      p.S[row * p.s_row + (v * E / kScaleBlock) * p.s_blk] = s;
  };
  const int64_t vectors = (p.N + E - 1) / E;
  float h[VPT > 0 ? VPT : 1][E];
  float ss = 0.f;
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) load(threadIdx.x + i * blockDim.x, h[i]);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) ss = fmaf(h[i][j], h[i][j], ss);
  } else {
    for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
      load(v, h[0]);
#pragma unroll
      for (int j = 0; j < E; ++j) ss = fmaf(h[0][j], h[0][j], ss);
    }
  }
  ss = block_sum2(ss, 0.f, red).x;
  const float rstd = __frsqrt_rn(ss / float(p.N) + p.eps);
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int64_t v = threadIdx.x + i * blockDim.x;
      if (hrow && v * E < p.N) store_row(hrow, v, p.N, h[i]);
      emit(v, h[i], rstd);
    }
  } else {
    // whole warps take part in the block maxima: round up to the block
    for (int64_t v = threadIdx.x; v < (vectors + 31) / 32 * 32; v += blockDim.x) {
      load(v, h[0]);
      if (hrow && v * E < p.N) store_row(hrow, v, p.N, h[0]);
      emit(v, h[0], rstd);
    }
  }
}

// Rows b, b + gridDim.x, ... per block.  The block's share of dw stays in
// registers and goes to row b of `part` at the end (VPT = 0: it is added up
// there); the shares are added in a fixed order by sum_parts_kernel, so the
// result does not change from run to run.
template <class T, int VPT>
__global__ void __launch_bounds__(1024)
    rmsnorm_backward_kernel(const NormBackProblem p, bool w32,
                            float* __restrict__ part) {
  constexpr int E = Vec<T>::kN;
  constexpr int V = VPT > 0 ? VPT : 1;
  __shared__ float2 red[2][32];
  float dw[V][E], w[V][E];
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      load_weight<T>(p.W, w32, threadIdx.x + i * blockDim.x, p.N, w[i]);
#pragma unroll
      for (int j = 0; j < E; ++j) dw[i][j] = 0.f;
    }
  }
  const int64_t vectors = (p.N + E - 1) / E;
  float* mine = part + int64_t(blockIdx.x) * p.N;
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, flip ^= 1) {
    const T* dyr = static_cast<const T*>(p.DY) + row * p.lddy;
    const T* hr = static_cast<const T*>(p.H) + row * p.ldh;
    const T* rr = p.R ? static_cast<const T*>(p.R) + row * p.ldr : nullptr;
    T* dxr = static_cast<T*>(p.DX) + row * p.lddx;
    float dy[V][E], h[V][E];
    float ss = 0.f, gh = 0.f;
    auto sums = [&](int i) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        ss = fmaf(h[i][j], h[i][j], ss);
        gh = fmaf(dy[i][j] * w[i][j], h[i][j], gh);
      }
    };
    if constexpr (VPT > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        load_row(hr, threadIdx.x + i * blockDim.x, p.N, h[i]);
        load_row(dyr, threadIdx.x + i * blockDim.x, p.N, dy[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sums(i);
    } else {
      for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
        load_row(hr, v, p.N, h[0]);
        load_row(dyr, v, p.N, dy[0]);
        load_weight<T>(p.W, w32, v, p.N, w[0]);
        sums(0);
      }
    }
    const float2 s = block_sum2(ss, gh, red[flip]);
    const float rstd = __frsqrt_rn(s.x / float(p.N) + p.eps);
    const float c = rstd * rstd * (s.y / float(p.N));
    auto emit = [&](int i, int64_t v) {
      if (v * E >= p.N) return;
      float o[E], r[E];
      if (rr) load_row(rr, v, p.N, r);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        o[j] = rstd * (dy[i][j] * w[i][j] - h[i][j] * c);
        if (rr) o[j] += r[j];
      }
      store_row(dxr, v, p.N, o);
    };
    if constexpr (VPT > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        emit(i, threadIdx.x + i * blockDim.x);
#pragma unroll
        for (int j = 0; j < E; ++j) dw[i][j] = fmaf(dy[i][j] * rstd, h[i][j], dw[i][j]);
      }
    } else {
      for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
        load_row(hr, v, p.N, h[0]);
        load_row(dyr, v, p.N, dy[0]);
        load_weight<T>(p.W, w32, v, p.N, w[0]);
        emit(0, v);
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const int64_t n = v * E + j;
          if (n < p.N)
            mine[n] = fmaf(dy[0][j] * rstd, h[0][j],
                           row == blockIdx.x ? 0.f : mine[n]);
        }
      }
    }
  }
  if constexpr (VPT > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const int64_t n = (threadIdx.x + int64_t(i) * blockDim.x) * E + j;
        if (n < p.N) mine[n] = dw[i][j];
      }
  }
}

// out[n] = sum of part[g][n] over g: 32 columns per block, 32 rows of
// threads that each add up every 32nd part.
__global__ void __launch_bounds__(1024)
    sum_parts_kernel(const float* __restrict__ part, int parts, int64_t n,
                     float* __restrict__ out) {
  __shared__ float t[32][33];
  const int64_t col = int64_t(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.f;
  if (col < n) {
#pragma unroll 4
    for (int g = threadIdx.y; g < parts; g += 32) s += part[g * n + col];
  }
  t[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = t[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  const int64_t c = int64_t(blockIdx.x) * 32 + threadIdx.y;
  if (threadIdx.x == 0 && c < n) out[c] = s;
}

int backward_blocks(int num_sms, int64_t M) {
  const int64_t most = int64_t(num_sms) * 2;
  return int(M < most ? M : most);
}

// Vectors per thread and threads per block for rows of `vectors` vectors.
void shape(int64_t vectors, int* vpt, int* threads) {
  *vpt = vectors <= 512 ? 1 : vectors <= 1024 ? 2 : vectors <= 4096 ? 4 : 0;
  const int64_t per = *vpt ? (vectors + *vpt - 1) / *vpt : 1024;
  *threads = int((per + 31) / 32 * 32);
}

template <class T>
mma_status_t forward(const Ctx& ctx, const NormProblem& p, bool w32) {
  int vpt, threads;
  shape((p.N + Vec<T>::kN - 1) / Vec<T>::kN, &vpt, &threads);
  const unsigned grid = unsigned(p.M);
  switch (vpt) {
    case 1: rmsnorm_kernel<T, 1><<<grid, threads, 0, ctx.stream>>>(p, w32); break;
    case 2: rmsnorm_kernel<T, 2><<<grid, threads, 0, ctx.stream>>>(p, w32); break;
    case 4: rmsnorm_kernel<T, 4><<<grid, threads, 0, ctx.stream>>>(p, w32); break;
    default: rmsnorm_kernel<T, 0><<<grid, threads, 0, ctx.stream>>>(p, w32);
  }
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

template <class T>
mma_status_t backward(const Ctx& ctx, const NormBackProblem& p, bool w32,
                      float* part) {
  int vpt, threads;
  shape((p.N + Vec<T>::kN - 1) / Vec<T>::kN, &vpt, &threads);
  const int grid = backward_blocks(ctx.num_sms, p.M);
  if (grid > 0) switch (vpt) {
    case 1: rmsnorm_backward_kernel<T, 1><<<grid, threads, 0, ctx.stream>>>(p, w32, part); break;
    case 2: rmsnorm_backward_kernel<T, 2><<<grid, threads, 0, ctx.stream>>>(p, w32, part); break;
    case 4: rmsnorm_backward_kernel<T, 4><<<grid, threads, 0, ctx.stream>>>(p, w32, part); break;
    default: rmsnorm_backward_kernel<T, 0><<<grid, threads, 0, ctx.stream>>>(p, w32, part);
  }
  sum_parts_kernel<<<unsigned((p.N + 31) / 32), dim3(32, 32), 0, ctx.stream>>>(
      part, grid, p.N, p.DW);
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

}  // namespace

mma_status_t launch_rmsnorm(const Ctx& ctx, const NormProblem& p) {
  const bool w32 = p.w_type == MMA_F32;
  switch (p.type) {
    case MMA_BF16: return forward<__nv_bfloat16>(ctx, p, w32);
    case MMA_F16: return forward<__half>(ctx, p, w32);
    default: return forward<float>(ctx, p, false);
  }
}

size_t rmsnorm_backward_workspace_bytes(int num_sms, int64_t M, int64_t N) {
  return size_t(backward_blocks(num_sms, M)) * size_t(N) * 4;
}

mma_status_t launch_rmsnorm_backward(const Ctx& ctx, const NormBackProblem& p,
                                     void* workspace) {
  const bool w32 = p.w_type == MMA_F32;
  float* part = static_cast<float*>(workspace);
  switch (p.type) {
    case MMA_BF16: return backward<__nv_bfloat16>(ctx, p, w32, part);
    case MMA_F16: return backward<__half>(ctx, p, w32, part);
    default: return backward<float>(ctx, p, false, part);
  }
}

}  // namespace mmagb
