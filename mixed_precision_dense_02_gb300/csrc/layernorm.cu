// Layer norm with the residual's addition, in the input's type or in 8 bits with a
// scale for each block of 128 columns, and its gradient.
//
// Forward, a row of x, residual r, weight w and bias b, all sums in FP32:
//     h = x + r,   c = h - mean(h),   y = c / sqrt(mean(c^2) + eps) * w + b
// Backward, with g = dy * w, g' = g - mean(g) and the rounded h of the forward:
//     dx = g' / std - c * mean(g' c) / std^3 + dr
//     dw = sum over rows dy c / std,   db = sum over rows dy
//
// Sums about a pivot.  With the row's mean as a first sum and the distances to it
// as a second, every row waits for two exchanges.  One is enough for the sums of d
// and d^2, d being the distances to any number k: mean = k + mean(d), var =
// mean(d^2) - mean(d)^2.  That loses as many bits of the variance as mean(d)^2 is
// larger than it, so k is the mean of 32 samples of the row, and a row whose
// mean(d)^2 is more than its variance all the same, so that more than a bit is lost, or
// whose sums leave FP32 (the decision is the same in every thread) has its sums taken
// again about the mean itself: a pivot of 32 numbers of one distribution is that far once
// in 10^8 rows.  Likewise mean(g' c) = mean(g d) - mean(g) mean(d).
//
// Forward and gradient are bound by HBM: 8192 x 8192 BF16 with residual to 8 bits 94 us
// (5.0 TB/s; with two exchanges 105), gradient of 8190 x 5000 with the residual's 78
// (4.2 TB/s; 97), of which the shares of dw and db cost some 10; one row of 4096 2.9.
#include <algorithm>
#include <type_traits>

#include "norm_common.cuh"
#include "norm_shape.h"

namespace mmagb {
namespace {

// Sums of four values over the block, the same in every thread, and the vote of
// block_sum2.  The four are shared out among the lanes while they are added up:
// six shuffles in place of twenty.
__device__ __forceinline__ float4 block_sum4(float a, float b, float c, float d, float4* buf,
                                             bool* any) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const bool up = lane & 16, odd = lane & 8;
  float x = up ? c : a, y = up ? d : b;
  x += __shfl_xor_sync(0xffffffffu, up ? a : c, 16);
  y += __shfl_xor_sync(0xffffffffu, up ? b : d, 16);
  float z = odd ? y : x;
  z += __shfl_xor_sync(0xffffffffu, odd ? x : y, 8);
#pragma unroll
  for (int k = 4; k > 0; k >>= 1) z += __shfl_xor_sync(0xffffffffu, z, k);
  if ((lane & 7) == 0) reinterpret_cast<float*>(buf + (threadIdx.x >> 5))[lane >> 3] = z;
  *any = __syncthreads_or(*any);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    const float4 t = buf[w];
    s = make_float4(s.x + t.x, s.y + t.y, s.z + t.z, s.w + t.w);
  }
  return s;
}

// The element of a row of n at which this lane samples it: spread over the row
// and over the banks of shared memory (multiples of n / 32 alone meet in one bank:
// 8192 x 4096 BF16 83 us, so 68).
__device__ __forceinline__ int sample_of(int n) {
  const int lane = threadIdx.x & 31, q = n >> 5;
  return q > 0 ? lane * q + 2 * lane % q : lane * n >> 5;
}

// The mean of the row's samples, the same in every thread of the block.
template <class T>
__device__ __forceinline__ float row_pivot(const uint8_t* h, const uint8_t* r, int at) {
  float k = float(reinterpret_cast<const T*>(h)[at]);
  if (r) k += float(reinterpret_cast<const T*>(r)[at]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) k += __shfl_xor_sync(0xffffffffu, k, d);
  return k * (1.f / 32.f);
}

// Whether sums about a pivot that is `off` from the mean lose more than one bit of the
// variance `var`, or leave FP32 (then it is infinite or NaN).
__device__ __forceinline__ bool pivot_is_far(float off, float var) {
  return !(off * off <= var && var < INFINITY);
}

__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// 1 / sqrt(var + eps); rounding may take equal values' variance below zero, and
// NaN stays.
__device__ __forceinline__ float over_std(float var, float eps) {
  return __frsqrt_rn((var < 0.f ? 0.f : var) + eps);
}

// A row per block and a vector per thread: the shortest way for few rows.
template <class T, bool TAIL>
__global__ void __launch_bounds__(1024)
    layernorm_row_kernel(const NormProblem p, bool w32) {
  constexpr int E = Vec<T>::kN;
  __shared__ float2 red[2][32];
  const int64_t row = blockIdx.x, v = threadIdx.x, n = p.N;
  const bool live = v * E < n;
  float h[1][E], t[E];
  const uint4 xr = load_raw(static_cast<const T*>(p.X) + row * p.ldx, v, n);
  const uint4 rr = p.R ? load_raw(static_cast<const T*>(p.R) + row * p.ldr, v, n)
                       : make_uint4(0, 0, 0, 0);
  // (on their way beside the row)
  float w[E], b[E];
  load_weight<T>(p.W, w32, v, n, w);
  load_bias<T>(p.B, w32, v, n, b);
  Vec<T>::unpack(xr, h[0]);
  Vec<T>::unpack(rr, t);
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) h[0][j] += t[j];
  if constexpr (TAIL) clear_tail<T>(v, n, h[0]);
  if (p.H && live) store_row<T, TAIL>(static_cast<T*>(p.H) + row * p.ldh, v, n, h[0]);
#pragma unroll
  for (int j = 0; j < E; ++j) s += h[0][j];
  const float mean = block_sum2(s, 0.f, red[0]).x / float(n);
  s = 0.f;
#pragma unroll
  for (int j = 0; j < E; ++j) {
    // (vectors past the row hold zeros)
    h[0][j] = v * E + (TAIL ? j : 0) < n ? h[0][j] - mean : 0.f;
    s = fmaf(h[0][j], h[0][j], s);
  }
  const float rstd = over_std(block_sum2(s, 0.f, red[1]).x / float(n), p.eps);
  norm_out<T, 1, TAIL, true, false>(p, row, h, rstd,
                                    [&](int, int64_t, float (&wo)[E], float (&bo)[E]) {
#pragma unroll
                                      for (int j = 0; j < E; ++j) {
                                        wo[j] = w[j];
                                        bo[j] = b[j];
                                      }
                                    });
}

// Many rows: rows b, b + gridDim.x, ... per block, through a ring of `stages` rows
// of x and r in shared memory that bulk copies fill ahead.  A thread has VPT
// vectors, because the exchange costs it some 150 instructions whatever it holds
// (8192 x 8192 to 8 bits: with one vector 124 us and four fifths of all issue
// slots taken).  Four take 128 registers, of BF16 with some 32 bytes a thread spilled.
template <class T, int VPT, bool TAIL>
__global__ void __launch_bounds__(512, 1)
    layernorm_kernel(const NormProblem p, bool w32, int stages, int row_bytes,
                     unsigned* status) {
  constexpr int E = Vec<T>::kN;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[3][32];
  __shared__ uint64_t full[4];
  __shared__ int abort_flag;
  const int n = int(p.N);
  const int stage_bytes = (p.R ? 2 : 1) * row_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  auto fetch = [&](int64_t row, int s) {
    if (row >= p.M) return;
    uint8_t* dst = ring + s * stage_bytes;
    mbar_arrive_expect_tx(&full[s], uint32_t(stage_bytes));
    bulk_load(dst, static_cast<const T*>(p.X) + row * p.ldx, row_bytes, &full[s]);
    if (p.R)
      bulk_load(dst + row_bytes, static_cast<const T*>(p.R) + row * p.ldr, row_bytes,
                &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages; ++s) fetch(blockIdx.x + int64_t(s) * gridDim.x, s);
  // The thread's weights and bias, packed (FP32 ones are read again for every row,
  // from L2, because the ring leaves little L1: so 8192 x 4096 BF16 took 58 us).
  uint4 wr[VPT], br[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    wr[i] = br[i] = make_uint4(0, 0, 0, 0);
    if (!w32) wr[i] = load_raw(static_cast<const T*>(p.W), v, n);
    if (!w32 && p.B) br[i] = load_raw(static_cast<const T*>(p.B), v, n);
  }
  const int sample = sample_of(n);
  const float over_n = 1.f / float(n);
  int s = 0, flip = 0;
  uint32_t phase = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, flip ^= 1) {
    const uint8_t* xs = ring + s * stage_bytes;
    const uint8_t* rs = p.R ? xs + row_bytes : nullptr;
    // (a failed wait ends the block behind the sums' barrier)
    bool failed = !mbar_wait(&full[s], phase, &abort_flag, status);
    const float k = row_pivot<T>(xs, rs, sample);
    float h[VPT][E];  // distances to the pivot, zeros past the row
    float2 sd = both(0.f), ss = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      const bool live = v * E < n;
      if (live) {
        Vec<T>::unpack(*(reinterpret_cast<const uint4*>(xs) + v), h[i]);
        if (rs) {
          float t[E];
          Vec<T>::unpack(*(reinterpret_cast<const uint4*>(rs) + v), t);
#pragma unroll
          for (int j = 0; j < E; ++j) h[i][j] += t[j];
        }
        if (p.H && !failed)
          store_row<T, TAIL>(static_cast<T*>(p.H) + row * p.ldh, v, n, h[i]);
      }
#pragma unroll
      for (int j = 0; j < E; j += 2) {
        float2 d = __fadd2_rn(make_float2(h[i][j], h[i][j + 1]), both(-k));
        if (!live || (TAIL && v * E + j >= n)) d.x = 0.f;
        if (!live || (TAIL && v * E + j + 1 >= n)) d.y = 0.f;
        sd = __fadd2_rn(sd, d);
        ss = __ffma2_rn(d, d, ss);
        h[i][j] = d.x;
        h[i][j + 1] = d.y;
      }
    }
    const float2 sum = block_sum2<true>(sd.x + sd.y, ss.x + ss.y, red[flip], &failed);
    if (failed) {
      // the loads of this row and of those ahead
      if (threadIdx.x == 0)
        for (int i = 0; i < stages && row + i * int64_t(gridDim.x) < p.M; ++i)
          mbar_drain(&full[(s + i) % stages], phase ^ uint32_t(s + i >= stages), status);
      return;
    }
    if (blockDim.x == 32) __syncwarp();
    // every thread has read the row: its stage takes the one `stages` rows on
    if (threadIdx.x == 0) fetch(row + int64_t(stages) * gridDim.x, s);
    const float off = sum.x * over_n;
    float var = sum.y * over_n - off * off;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int j = 0; j < E; ++j) h[i][j] -= off;
    if (pivot_is_far(off, var)) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (int(threadIdx.x + i * blockDim.x) * E + j < n) a = fmaf(h[i][j], h[i][j], a);
      var = block_sum2(a, 0.f, red[2]).x * over_n;
    }
    norm_out<T, VPT, TAIL, true, false>(
        p, row, h, over_std(var, p.eps), [&](int i, int64_t v, float (&w)[E], float (&b)[E]) {
          if (w32) {
            load_weight<T>(p.W, true, v, n, w);
            load_bias<T>(p.B, true, v, n, b);
          } else {
            Vec<T>::unpack(wr[i], w);
            Vec<T>::unpack(br[i], b);
          }
        });
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
}

constexpr int64_t kRowBytes = 212 * 1024;  // shared memory for one row

// Rows too wide for that: one row per block, which a block keeps in shared memory (h in
// FP32; 2048 x 32768 BF16 with residual 211 us, 224 without) or, `cached` false, reads
// three times.  A thread reads what it has written.
template <class T>
__global__ void __launch_bounds__(1024)
    layernorm_wide_kernel(const NormProblem p, bool w32, bool cached) {
  constexpr int E = Vec<T>::kN;
  constexpr int kLanes = kScaleBlock / E;
  extern __shared__ __align__(16) float kept[];
  __shared__ float2 red[2][32];
  const int64_t row = blockIdx.x, n = p.N;
  const T* x = static_cast<const T*>(p.X) + row * p.ldx;
  const T* r = p.R ? static_cast<const T*>(p.R) + row * p.ldr : nullptr;
  float h[E];
  auto load = [&](int64_t v) {
    load_row(x, v, n, h);
    if (r) {
      float t[E];
      load_row(r, v, n, t);
#pragma unroll
      for (int j = 0; j < E; ++j) h[j] += t[j];
    }
  };
  auto again = [&](int64_t v) {
    if (!cached) return load(v);
#pragma unroll
    for (int j = 0; j < E; j += 4)
      *reinterpret_cast<float4*>(h + j) = *reinterpret_cast<const float4*>(kept + v * E + j);
  };
  const int64_t vectors = (n + E - 1) / E;
  float s = 0.f;
#pragma unroll 2
  for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
    load(v);
    if (cached) {
#pragma unroll
      for (int j = 0; j < E; j += 4)
        *reinterpret_cast<float4*>(kept + v * E + j) = *reinterpret_cast<const float4*>(h + j);
    }
#pragma unroll
    for (int j = 0; j < E; ++j) s += h[j];
  }
  const float mean = block_sum2(s, 0.f, red[0]).x / float(n);
  s = 0.f;
  for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
    again(v);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float c = v * E + j < n ? h[j] - mean : 0.f;
      s = fmaf(c, c, s);
    }
  }
  const float rstd = over_std(block_sum2(s, 0.f, red[1]).x / float(n), p.eps);
  // whole warps take part in the block maxima: round up to the block
  for (int64_t v = threadIdx.x; v < (vectors + 31) / 32 * 32; v += blockDim.x) {
    const bool live = v < vectors;
    if (live) again(v);
    if (p.H && live) store_row(static_cast<T*>(p.H) + row * p.ldh, v, n, h);
    float y[E], b[E];
    load_weight<T>(p.W, w32, v, n, y);
    load_bias<T>(p.B, w32, v, n, b);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      y[j] = v * E + j < n ? fmaf((h[j] - mean) * rstd, y[j], b[j]) : 0.f;
      m = abs_max(m, y[j]);
    }
    if (p.Y && live) store_row(static_cast<T*>(p.Y) + row * p.ldy, v, n, y);
    if (!p.Q) continue;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
      m = abs_max(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float sc = block_scale<false>(m, p.pow2);
    if (!live) continue;
    store_f8<false>(static_cast<uint8_t*>(p.Q) + row * p.ldq, v, n, y, Divisor(sc));
    if (threadIdx.x % kLanes == 0)
      p.S[row * p.s_row + (v * E / kScaleBlock) * p.s_blk] = sc;
  }
}

// The gradient: rows b, b + gridDim.x, ... per block through a ring of `stages`
// rows of h, dy and r; each thread reads its VPT vectors twice, for the sums and
// for the output, so that only its shares of dw and db stay in registers.  They go
// to row b of `part` at the end (n of dw, n of db), and the shares are added in a
// fixed order.
template <class T, int VPT, int MAXT, int MINB, bool TAIL>
__global__ void __launch_bounds__(MAXT, MINB)
    layernorm_backward_kernel(const NormBackProblem p, bool w32, int stages,
                              int row_bytes, float* __restrict__ part,
                              unsigned* status) {
  constexpr int E = Vec<T>::kN;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float4 red[2][16];
  __shared__ float2 far_red[32];
  __shared__ uint64_t full[4];
  __shared__ int abort_flag;
  const int n = int(p.N), vectors = (n + E - 1) / E;
  const int stage_bytes = (p.R ? 3 : 2) * row_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  auto fetch = [&](int64_t row, int s) {
    if (row >= p.M) return;
    uint8_t* dst = ring + s * stage_bytes;
    mbar_arrive_expect_tx(&full[s], uint32_t(stage_bytes));
    bulk_load(dst, static_cast<const T*>(p.H) + row * p.ldh, row_bytes, &full[s]);
    bulk_load(dst + row_bytes, static_cast<const T*>(p.DY) + row * p.lddy, row_bytes,
              &full[s]);
    if (p.R)
      bulk_load(dst + 2 * row_bytes, static_cast<const T*>(p.R) + row * p.ldr, row_bytes,
                &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages; ++s) fetch(blockIdx.x + int64_t(s) * gridDim.x, s);
  float2 dw[VPT][E / 2], db[VPT][E / 2];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < E / 2; ++j) dw[i][j] = db[i][j] = both(0.f);
  // vector v of a row in the ring
  auto load = [&](const uint8_t* row, int v, float2 (&f)[E / 2]) {
    float t[E];
    Vec<T>::unpack(*(reinterpret_cast<const uint4*>(row) + v), t);
    if constexpr (TAIL) clear_tail<T>(v, n, t);
#pragma unroll
    for (int j = 0; j < E / 2; ++j) f[j] = make_float2(t[2 * j], t[2 * j + 1]);
  };
  // the weights: packed in registers, or (FP32) read again
  uint4 wr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    wr[i] = w32 ? make_uint4(0, 0, 0, 0)
                : load_raw(static_cast<const T*>(p.W), threadIdx.x + i * blockDim.x, n);
  auto weight = [&](int i, int v, float2 (&f)[E / 2]) {
    float t[E];
    if (w32) {
      load_weight<T>(p.W, true, v, n, t);
    } else {
      Vec<T>::unpack(wr[i], t);
      if constexpr (TAIL) clear_tail<T>(v, n, t);
    }
#pragma unroll
    for (int j = 0; j < E / 2; ++j) f[j] = make_float2(t[2 * j], t[2 * j + 1]);
  };
  // distances to a, zeros past the row
  auto minus = [&](float2 h, float a, int at) {
    float2 d = __fadd2_rn(h, both(-a));
    if (TAIL && at >= n) d.x = 0.f;
    if (TAIL && at + 1 >= n) d.y = 0.f;
    return d;
  };
  const int sample = sample_of(n);
  const float over_n = 1.f / float(n);
  int s = 0, flip = 0;
  uint32_t phase = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const uint8_t* hs = ring + s * stage_bytes;
    const uint8_t* ds = hs + row_bytes;
    const uint8_t* rs = ds + row_bytes;
    // (a failed wait ends the block behind the sums' barrier)
    bool failed = !mbar_wait(&full[s], phase, &abort_flag, status);
    const float k = row_pivot<T>(hs, nullptr, sample);
    float2 sd = both(0.f), ss = both(0.f), sg = both(0.f), gd = both(0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= vectors) continue;
      float2 h[E / 2], dy[E / 2], w[E / 2];
      load(hs, v, h);
      load(ds, v, dy);
      weight(i, v, w);
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        const float2 d = minus(h[j], k, v * E + 2 * j), g = __fmul2_rn(dy[j], w[j]);
        sd = __fadd2_rn(sd, d);
        ss = __ffma2_rn(d, d, ss);
        sg = __fadd2_rn(sg, g);
        gd = __ffma2_rn(g, d, gd);
      }
    }
    const float4 sum = block_sum4(sd.x + sd.y, ss.x + ss.y, sg.x + sg.y, gd.x + gd.y,
                                  red[flip], &failed);
    if (failed) {
      // the loads of this row and of those ahead (all but the one that would be
      // fetched below)
      const int ahead = row == blockIdx.x ? stages : stages - 1;
      if (threadIdx.x == 0)
        for (int i = 0; i < ahead && row + i * int64_t(gridDim.x) < p.M; ++i)
          mbar_drain(&full[(s + i) % stages], phase ^ uint32_t(s + i >= stages), status);
      return;
    }
    // Every thread is past the row before: its stage takes the row that is
    // `stages` rows after it.
    if (threadIdx.x == 0 && row != blockIdx.x)
      fetch(row + int64_t(stages - 1) * gridDim.x, s == 0 ? stages - 1 : s - 1);
    const float off = sum.x * over_n, mean = k + off, mean_g = sum.z * over_n;
    float var = sum.y * over_n - off * off;
    float cov = sum.w * over_n - off * mean_g;  // mean(g' c)
    if (pivot_is_far(off, var)) {
      float2 a = both(0.f), b = both(0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= vectors) continue;
        float2 h[E / 2], dy[E / 2], w[E / 2];
        load(hs, v, h);
        load(ds, v, dy);
        weight(i, v, w);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const float2 c = minus(h[j], mean, v * E + 2 * j);
          a = __ffma2_rn(c, c, a);
          b = __ffma2_rn(__ffma2_rn(dy[j], w[j], both(-mean_g)), c, b);
        }
      }
      const float2 again = block_sum2(a.x + a.y, b.x + b.y, far_red);
      var = again.x * over_n;
      cov = again.y * over_n;
    }
    const float rstd = over_std(var, p.eps);
    // (rstd^3 by itself leaves the range of FP32 at deviations of 2^42 and 2^-42)
    const float2 f = both(-cov * rstd * rstd * rstd), r1 = both(rstd);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= vectors) continue;
      float2 h[E / 2], dy[E / 2], w[E / 2];
      float o[E];
      load(hs, v, h);
      load(ds, v, dy);
      weight(i, v, w);
#pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        const float2 c = __fadd2_rn(h[j], both(-mean));
        dw[i][j] = __ffma2_rn(__fmul2_rn(dy[j], r1), c, dw[i][j]);
        db[i][j] = __fadd2_rn(db[i][j], dy[j]);
        const float2 t = __ffma2_rn(__ffma2_rn(dy[j], w[j], both(-mean_g)), r1,
                                    __fmul2_rn(f, c));
        o[2 * j] = t.x;
        o[2 * j + 1] = t.y;
      }
      if (p.R) {
        load(rs, v, h);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          o[2 * j] += h[j].x;
          o[2 * j + 1] += h[j].y;
        }
      }
      store_row<T, TAIL>(static_cast<T*>(p.DX) + row * p.lddx, v, n, o);
    }
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
    flip ^= 1;
  }
  grid_dependents_start();
  float* mine = part + int64_t(blockIdx.x) * n * 2;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int at = int(threadIdx.x + i * blockDim.x) * E;
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (at + j < n) {
        mine[at + j] = j & 1 ? dw[i][j / 2].y : dw[i][j / 2].x;
        mine[n + at + j] = j & 1 ? db[i][j / 2].y : db[i][j / 2].x;
      }
  }
}

// Rows too wide for that, in two kernels.  First what dx and dw take from a whole row:
// its mean, 1 / std, mean(g) and -mean(g' c) / std^3.  A block keeps the row (h and dy)
// in shared memory or, `cached` false, reads it twice.  (2048 x 32768 BF16: 233 us for
// both; a block per row that adds to its share of dw and db in memory took 708.)
template <class T>
__global__ void __launch_bounds__(1024)
    layernorm_stats_kernel(const NormBackProblem p, bool w32, bool cached,
                           float* __restrict__ stats) {
  constexpr int E = Vec<T>::kN;
  extern __shared__ __align__(16) uint4 kept_rows[];
  __shared__ float2 red[2][32];
  const int64_t n = p.N, vectors = (n + E - 1) / E;
  float dy[E], h[E], w[E];
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    auto load = [&](int64_t v, bool first) {
      uint4 hv, dv;
      if (first || !cached) {
        hv = load_raw(static_cast<const T*>(p.H) + row * p.ldh, v, n);
        dv = load_raw(static_cast<const T*>(p.DY) + row * p.lddy, v, n);
      } else {
        hv = kept_rows[v];
        dv = kept_rows[vectors + v];
      }
      if (first && cached) {  // (read again by this thread alone)
        kept_rows[v] = hv;
        kept_rows[vectors + v] = dv;
      }
      Vec<T>::unpack(hv, h);
      Vec<T>::unpack(dv, dy);
      clear_tail<T>(v, n, h);
      clear_tail<T>(v, n, dy);
      load_weight<T>(p.W, w32, v, n, w);
    };
    float a = 0.f, b = 0.f;
#pragma unroll 2
    for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
      load(v, true);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        a += h[j];
        b = fmaf(dy[j], w[j], b);
      }
    }
    float2 s = block_sum2(a, b, red[0]);
    const float mean = s.x / float(n), mean_g = s.y / float(n);
    a = b = 0.f;
#pragma unroll 2
    for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
      load(v, false);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float c = v * E + j < n ? h[j] - mean : 0.f;
        a = fmaf(c, c, a);
        b = fmaf(fmaf(dy[j], w[j], -mean_g), c, b);
      }
    }
    s = block_sum2(a, b, red[1]);
    if (threadIdx.x == 0) {
      const float rstd = over_std(s.x / float(n), p.eps);
      stats[4 * row] = mean;
      stats[4 * row + 1] = rstd;
      stats[4 * row + 2] = mean_g;
      stats[4 * row + 3] = -(s.y / float(n)) * rstd * rstd * rstd;
    }
  }
}

// Then dx and shares of dw and db: a vector of columns per thread, rows [b * per, ...)
// for row b of part, four on their way at a time.  dx is stored where dy or r was read.
template <class T>
__global__ void __launch_bounds__(128)
    layernorm_columns_kernel(const NormBackProblem p, bool w32,
                             const float* __restrict__ stats, int64_t per,
                             float* __restrict__ part) {
  constexpr int E = Vec<T>::kN;
  constexpr int U = 4;
  const int64_t v = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, n = p.N;
  const int64_t from = blockIdx.y * per, to = min(from + per, p.M);
  if (v * E >= n) return;
  float w[E], dw[E], db[E];
  load_weight<T>(p.W, w32, v, n, w);
#pragma unroll
  for (int j = 0; j < E; ++j) dw[j] = db[j] = 0.f;
  for (int64_t base = from; base < to; base += U) {
    uint4 hv[U], dv[U], rv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = base + u;
      if (row >= to) break;
      hv[u] = load_raw(static_cast<const T*>(p.H) + row * p.ldh, v, n);
      dv[u] = load_raw(static_cast<const T*>(p.DY) + row * p.lddy, v, n);
      if (p.R) rv[u] = load_raw(static_cast<const T*>(p.R) + row * p.ldr, v, n);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = base + u;
      if (row >= to) break;
      float h[E], dy[E], r[E];
      Vec<T>::unpack(hv[u], h);
      Vec<T>::unpack(dv[u], dy);
#pragma unroll
      for (int j = 0; j < E; ++j) r[j] = 0.f;
      if (p.R) Vec<T>::unpack(rv[u], r);
      const float mean = stats[4 * row], rstd = stats[4 * row + 1];
      const float mean_g = stats[4 * row + 2], f = stats[4 * row + 3];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float c = h[j] - mean;
        dw[j] = fmaf(dy[j] * rstd, c, dw[j]);
        db[j] += dy[j];
        r[j] += fmaf(fmaf(dy[j], w[j], -mean_g), rstd, f * c);
      }
      store_row(static_cast<T*>(p.DX) + row * p.lddx, v, n, r);
    }
  }
  float* const mine = part + blockIdx.y * 2 * n;
#pragma unroll
  for (int j = 0; j < E; ++j)
    if (v * E + j < n) {
      mine[v * E + j] = dw[j];
      mine[n + v * E + j] = db[j];
    }
}

// Launches a kernel with a ring in up to 220 KB of shared memory.
template <class K, class... Args>
bool launch_ring(const Ctx& ctx, PerContext<bool>& attr, K kernel, int64_t grid, int threads,
                 int64_t smem, Args... args) {
  bool ok = false;
  if (!attr.get(ctx, &ok, [&](bool* v) {
        *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  220 * 1024) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return false;
  kernel<<<unsigned(grid), threads, size_t(smem), ctx.stream>>>(args...);
  return true;
}

template <class T>
mma_status_t forward(const Ctx& ctx, const NormProblem& p, bool w32) {
  constexpr int E = Vec<T>::kN;
  const int64_t vectors = (p.N + E - 1) / E;
  const int tensors = p.R ? 2 : 1;
  const NormRingShape shape = layernorm_shape(vectors, tensors);
  bool ok = true;
  if (p.M <= ctx.num_sms && vectors <= 1024) {
    const int threads = int(vectors + 31) / 32 * 32;
    if (p.N % E)
      layernorm_row_kernel<T, true><<<unsigned(p.M), threads, 0, ctx.stream>>>(p, w32);
    else
      layernorm_row_kernel<T, false><<<unsigned(p.M), threads, 0, ctx.stream>>>(p, w32);
  } else if (shape.vpt) {
    auto run = [&](auto kernel, PerContext<bool>& attr) {
      ok = launch_ring(ctx, attr, kernel,
                       std::min<int64_t>(p.M, int64_t(ctx.num_sms) * shape.per_sm),
                       shape.threads, shape.stages * tensors * vectors * 16, p, w32,
                       shape.stages, int(vectors * 16), ctx.status);
    };
    static PerContext<bool> a1, a2, a4, t1, t2, t4;
    if (p.N % E) {
      if (shape.vpt == 1) run(layernorm_kernel<T, 1, true>, t1);
      else if (shape.vpt == 2) run(layernorm_kernel<T, 2, true>, t2);
      else run(layernorm_kernel<T, 4, true>, t4);
    } else {
      if (shape.vpt == 1) run(layernorm_kernel<T, 1, false>, a1);
      else if (shape.vpt == 2) run(layernorm_kernel<T, 2, false>, a2);
      else run(layernorm_kernel<T, 4, false>, a4);
    }
  } else {
    static PerContext<bool> wide;
    const int64_t row = vectors * E * 4;
    const bool cached = row <= kRowBytes;
    ok = launch_ring(ctx, wide, layernorm_wide_kernel<T>, p.M, 1024, cached ? row : 0, p, w32,
                     cached);
  }
  return cudaGetLastError() == cudaSuccess && ok ? MMA_OK : MMA_ERR_LAUNCH;
}

template <class T>
mma_status_t backward(const Ctx& ctx, const NormBackProblem& p, bool w32, float* part) {
  constexpr int E = Vec<T>::kN;
  const int64_t vectors = (p.N + E - 1) / E;
  const int tensors = p.R ? 3 : 2;
  const NormRingShape shape = layernorm_back_shape(vectors, tensors);
  const int64_t most = std::min(p.M, layernorm_most_parts(p.N));
  int64_t grid = std::min(most, int64_t(shape.per_sm) * ctx.num_sms);  // rows of part
  bool ok = true;
  if (grid > 0 && shape.vpt) {
    auto run = [&](auto kernel, PerContext<bool>& attr) {
      ok = launch_ring(ctx, attr, kernel, grid, shape.threads,
                       shape.stages * tensors * vectors * 16, p, w32, shape.stages,
                       int(vectors * 16), part, ctx.status);
    };
    static PerContext<bool> a1, a2, a4, t1, t2, t4;
    if (p.N % E) {
      if (shape.vpt == 1) run(layernorm_backward_kernel<T, 1, 128, 8, true>, t1);
      else if (shape.vpt == 2) run(layernorm_backward_kernel<T, 2, 384, 2, true>, t2);
      else run(layernorm_backward_kernel<T, 4, 512, 1, true>, t4);
    } else {
      if (shape.vpt == 1) run(layernorm_backward_kernel<T, 1, 128, 8, false>, a1);
      else if (shape.vpt == 2) run(layernorm_backward_kernel<T, 2, 384, 2, false>, a2);
      else run(layernorm_backward_kernel<T, 4, 512, 1, false>, a4);
    }
  } else if (p.M > 0) {
    static PerContext<bool> wide;
    float* const stats = part + most * 2 * p.N;
    const bool cached = vectors * 32 <= kRowBytes;
    ok = launch_ring(ctx, wide, layernorm_stats_kernel<T>,
                     std::min<int64_t>(p.M, ctx.num_sms * (cached ? 1 : 2)), 1024,
                     cached ? vectors * 32 : 0, p, w32, cached, stats);
    if (!ok) return MMA_ERR_LAUNCH;
    // as many blocks of rows as give every SM some sixteen of columns
    const int64_t columns = (vectors + 127) / 128;
    const int64_t want = std::max<int64_t>(1, 16 * ctx.num_sms / columns);
    const int64_t per = (p.M + std::min(most, want) - 1) / std::min(most, want);
    grid = (p.M + per - 1) / per;
    layernorm_columns_kernel<T>
        <<<dim3(unsigned(columns), unsigned(grid)), 128, 0, ctx.stream>>>(p, w32, stats, per,
                                                                          part);
  }
  if (!ok || cudaPeekAtLastError() != cudaSuccess) return MMA_ERR_LAUNCH;
  return sum_parts(ctx, part, int(grid), 2 * p.N, p.DW, p.N, p.DB);
}

}  // namespace

int64_t layernorm_backward_workspace_bytes(int64_t M, int64_t N) {
  // (behind the shares four floats per row, where rows may be too wide for the ring)
  return std::min(M, layernorm_most_parts(N)) * N * 8 +
         (N > 4 * kNormBackMostVectors ? 16 * M : 0);
}

mma_status_t launch_layernorm(const Ctx& ctx, const NormProblem& p) {
  const bool w32 = p.w_type == MMA_F32;
  switch (p.type) {
    case MMA_BF16: return forward<__nv_bfloat16>(ctx, p, w32);
    case MMA_F16: return forward<__half>(ctx, p, w32);
    default: return forward<float>(ctx, p, false);
  }
}

mma_status_t launch_layernorm_backward(const Ctx& ctx, const NormBackProblem& p,
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
