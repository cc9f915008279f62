// Root-mean-square norm with the residual's addition and an 8-bit output
// with a scale for each block of 128 columns, and its gradient.
//
// Forward, a row of x, residual r and weight w, all sums in FP32:
//     h = x + r
//     y = h * w / sqrt(mean(h^2) + eps)
//     s_b = max(max|y| over block b / 448, 2^-126),  q = y / s_b in E4M3
// h leaves rounded to the input's type; y is formed from the unrounded sum.
// q is the FP32 quotient y / s_b, rounded to nearest.
//
// Backward, with g = dy * w and the rounded h that the forward stored:
//     dx = g / rms - h * mean(g h) / rms^3 + dr,   dw = sum over rows dy h / rms
// (dx is the gradient of x and of the residual alike; dr the gradient that
// reaches h from elsewhere).
//
// Both are bound by memory: each input is read once and each output written
// once, a row is held on chip between its two uses.  BF16, 8192 x 8192:
// forward 77 us, 6.1 TB/s; one row of 4096 2.5 us, all latency.  Backward, 8190
// x 5000 BF16: 64 us, 5.1 TB/s, some 6 us of them for the shares of dw (456
// rows written, read and added up by a second kernel); 8192 x 8192 94 us.
// Rows of more than 2048 vectors are read twice: forward 2048 x 32768 BF16 183
// us of 69 (floor), 4096 x 16384 FP32 266 of 129; backward 2048 x 32768 387 of
// 79, where the share of dw also goes through memory for every row.
#include <algorithm>
#include <type_traits>

#include "norm_common.cuh"
#include "norm_shape.h"

namespace mmagb {
namespace {

// Rows b, b + gridDim.x, ... per block, a row at a time: VPT 16-byte vectors
// per thread stay in registers between the sum of squares and the output,
// and the next row's loads are issued before this row's sum is exchanged.
template <class T, int VPT, int MAXT, bool TAIL>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1)
    rmsnorm_kernel(const NormProblem p, bool w32) {
  constexpr int E = Vec<T>::kN;
  __shared__ float2 red[2][32];
  const T* const X = static_cast<const T*>(p.X);
  const T* const R = static_cast<const T*>(p.R);
  const int64_t n = p.N;
  uint4 xr[VPT], rr[VPT];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      xr[i] = load_raw(X + row * p.ldx, threadIdx.x + i * blockDim.x, n);
    if (R) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        rr[i] = load_raw(R + row * p.ldr, threadIdx.x + i * blockDim.x, n);
    }
  };
  fetch(blockIdx.x);
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, flip ^= 1) {
    float h[VPT][E];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      Vec<T>::unpack(xr[i], h[i]);
      if (R) {
        float t[E];
        Vec<T>::unpack(rr[i], t);
#pragma unroll
        for (int j = 0; j < E; ++j) h[i][j] += t[j];
      }
      if constexpr (TAIL) clear_tail<T>(threadIdx.x + i * blockDim.x, n, h[i]);
#pragma unroll
      for (int j = 0; j < E; ++j) ss = fmaf(h[i][j], h[i][j], ss);
    }
    if (row + gridDim.x < p.M) fetch(row + gridDim.x);
    ss = block_sum2(ss, 0.f, red[flip]).x;
    const float rstd = __frsqrt_rn(ss / float(n) + p.eps);
    norm_out<T, VPT, TAIL, false, true>(
        p, row, h, rstd, [&](int, int64_t v, float (&w)[E], float (&)[E]) {
          load_weight<T>(p.W, w32, v, n, w);
        });
  }
}

// Rows wider than the registers hold: one row per block, read twice.
template <class T>
__global__ void __launch_bounds__(1024)
    rmsnorm_wide_kernel(const NormProblem p, bool w32) {
  constexpr int E = Vec<T>::kN;
  constexpr int kLanes = kScaleBlock / E;
  __shared__ float2 red[32];
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
  const int64_t vectors = (n + E - 1) / E;
  float ss = 0.f;
  for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
    load(v);
#pragma unroll
    for (int j = 0; j < E; ++j) ss = fmaf(h[j], h[j], ss);
  }
  ss = block_sum2(ss, 0.f, red).x;
  const float rstd = __frsqrt_rn(ss / float(n) + p.eps);
  // whole warps take part in the block maxima: round up to the block
  for (int64_t v = threadIdx.x; v < (vectors + 31) / 32 * 32; v += blockDim.x) {
    load(v);
    const bool live = v < vectors;
    if (p.H && live) store_row(static_cast<T*>(p.H) + row * p.ldh, v, n, h);
    float y[E];
    load_weight<T>(p.W, w32, v, n, y);
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      y[j] = v * E + j < n ? h[j] * rstd * y[j] : 0.f;
      m = abs_max(m, y[j]);
    }
    if (p.Y && live) store_row(static_cast<T*>(p.Y) + row * p.ldy, v, n, y);
    if (!p.Q) continue;
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1)
      m = abs_max(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float s = block_scale<false>(m, p.pow2);
    if (!live) continue;
    store_f8<false>(static_cast<uint8_t*>(p.Q) + row * p.ldq, v, n, y,
                    Divisor(s));
    if (threadIdx.x % kLanes == 0)
      p.S[row * p.s_row + (v * E / kScaleBlock) * p.s_blk] = s;
  }
}

// Rows b, b + gridDim.x, ... per block, through a ring of `stages` rows of
// h, dy and r in shared memory that bulk copies fill ahead; each thread
// reads its VPT vectors twice, for the sums and for the output, so that only
// its share of dw stays in registers.  That goes to row b of `part` at the
// end; the shares are added in a fixed order by sum_parts_kernel, so the
// result does not change from run to run.
template <class T, int VPT, bool TAIL>
__global__ void __launch_bounds__(512, VPT <= 2 ? 2 : 1)
    rmsnorm_backward_kernel(const NormBackProblem p, bool w32, int stages,
                            int row_bytes, float* __restrict__ part,
                            unsigned* status, const WaitHook hook) {
  constexpr int E = Vec<T>::kN;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float2 red[2][32];
  __shared__ uint64_t full[4];
  __shared__ int abort_flag;
  const int n = int(p.N), vectors = (n + E - 1) / E;
  const int tensors = p.R ? 3 : 2;
  const int stage_bytes = tensors * row_bytes;
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  auto fetch = [&](int64_t row, int s) {
    if (row >= p.M || hook.withhold) return;
    uint8_t* dst = ring + s * stage_bytes;
    mbar_arrive_expect_tx(&full[s], uint32_t(stage_bytes));
    bulk_load(dst, static_cast<const T*>(p.H) + row * p.ldh, row_bytes, &full[s]);
    bulk_load(dst + row_bytes, static_cast<const T*>(p.DY) + row * p.lddy,
              row_bytes, &full[s]);
    if (p.R)
      bulk_load(dst + 2 * row_bytes, static_cast<const T*>(p.R) + row * p.ldr,
                row_bytes, &full[s]);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < stages; ++s)
      fetch(blockIdx.x + int64_t(s) * gridDim.x, s);
  float dw[VPT][E];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < E; ++j) dw[i][j] = 0.f;
  // vector v of a row in the ring
  auto load = [&](const uint8_t* row, int v, float (&f)[E]) {
    Vec<T>::unpack(*(reinterpret_cast<const uint4*>(row) + v), f);
    if constexpr (TAIL) clear_tail<T>(v, n, f);
  };
  // the weights: packed in registers, or (FP32) read again
  uint4 wr[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    wr[i] = w32 ? make_uint4(0, 0, 0, 0)
                : load_raw(static_cast<const T*>(p.W), threadIdx.x + i * blockDim.x, n);
  auto weight = [&](int i, int v, float (&f)[E]) {
    if (w32) {
      load_weight<T>(p.W, true, v, n, f);
    } else {
      Vec<T>::unpack(wr[i], f);
      if constexpr (TAIL) clear_tail<T>(v, n, f);
    }
  };
  int s = 0, flip = 0;
  uint32_t phase = 0;
  const float over_n = 1.f / float(n);
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
    const uint8_t* hs = ring + s * stage_bytes;
    const uint8_t* ds = hs + row_bytes;
    const uint8_t* rs = ds + row_bytes;
    // A failed wait ends the block behind the sums' barrier, before anything is
    // stored or fetched.  (8190 x 5000 BF16 64 us; with threads that remember it
    // and go on without storing 70.)
    bool failed = !mbar_wait(&full[s], phase, &abort_flag, status, hook.limit_ns);
    float ss = 0.f, gh = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= vectors) continue;
      float h[E], dy[E], w[E];
      load(hs, v, h);
      load(ds, v, dy);
      weight(i, v, w);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        ss = fmaf(h[j], h[j], ss);
        gh = fmaf(dy[j] * w[j], h[j], gh);
      }
    }
    const float2 sum = block_sum2<true>(ss, gh, red[flip], &failed);
    if (failed) {
      // the loads of this row and of those ahead (all but the one that would be
      // fetched below)
      const int ahead = row == blockIdx.x ? stages : stages - 1;
      if (threadIdx.x == 0)
        for (int k = 0; k < ahead && row + k * int64_t(gridDim.x) < p.M; ++k)
          mbar_drain(&full[(s + k) % stages], phase ^ uint32_t(s + k >= stages), status,
                     hook.limit_ns);
      return;
    }
    if (blockDim.x == 32) __syncwarp();
    // Every thread is past the row before: its stage takes the row that is
    // `stages` rows after it.
    if (threadIdx.x == 0 && row != blockIdx.x)
      fetch(row + int64_t(stages - 1) * gridDim.x, s == 0 ? stages - 1 : s - 1);
    const float rstd = __frsqrt_rn(sum.x * over_n + p.eps);
    // (rstd^3 by itself leaves the range of FP32 at rms of 2^42 and 2^-42)
    const float c = -(sum.y * over_n) * rstd * rstd * rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v >= vectors) continue;
      float h[E], dy[E], w[E], o[E];
      load(hs, v, h);
      load(ds, v, dy);
      weight(i, v, w);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float d = dy[j] * rstd;
        dw[i][j] = fmaf(d, h[j], dw[i][j]);
        o[j] = fmaf(d, w[j], c * h[j]);
      }
      if (p.R) {
        float r[E];
        load(rs, v, r);
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] += r[j];
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
  float* mine = part + int64_t(blockIdx.x) * n;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int64_t at = int64_t(threadIdx.x + i * blockDim.x) * E;
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (at + j < n) mine[at + j] = dw[i][j];
  }
}

// Rows too wide for that: read twice, dw added up in `part`.
template <class T>
__global__ void __launch_bounds__(1024)
    rmsnorm_backward_wide_kernel(const NormBackProblem p, bool w32,
                                 float* __restrict__ part) {
  constexpr int E = Vec<T>::kN;
  __shared__ float2 red[2][32];
  const int64_t n = p.N, vectors = (n + E - 1) / E;
  float* mine = part + int64_t(blockIdx.x) * n;
  float dy[E], h[E], w[E];
  int flip = 0;
  for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, flip ^= 1) {
    auto load = [&](int64_t v) {
      load_row(static_cast<const T*>(p.H) + row * p.ldh, v, n, h);
      load_row(static_cast<const T*>(p.DY) + row * p.lddy, v, n, dy);
      load_weight<T>(p.W, w32, v, n, w);
    };
    float ss = 0.f, gh = 0.f;
    for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
      load(v);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        ss = fmaf(h[j], h[j], ss);
        gh = fmaf(dy[j] * w[j], h[j], gh);
      }
    }
    const float2 s = block_sum2(ss, gh, red[flip]);
    const float rstd = __frsqrt_rn(s.x / float(n) + p.eps);
    const float c = s.y / float(n) * rstd * rstd * rstd;
    for (int64_t v = threadIdx.x; v < vectors; v += blockDim.x) {
      load(v);
      float o[E], r[E];
      if (p.R) load_row(static_cast<const T*>(p.R) + row * p.ldr, v, n, r);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float d = dy[j] * rstd;
        o[j] = fmaf(d, w[j], -c * h[j]) + (p.R ? r[j] : 0.f);
        const int64_t at = v * E + j;
        if (at < n)
          mine[at] = fmaf(d, h[j], row == blockIdx.x ? 0.f : mine[at]);
      }
      store_row(static_cast<T*>(p.DX) + row * p.lddx, v, n, o);
    }
  }
}

constexpr int kMostParts = 456;  // blocks of the backward pass, three per SM at most

// Calls f(VPT, MAXT, threads) for rows of `vectors` vectors: up to 256
// threads with up to 4 vectors each, so that several rows are under way per
// SM, wider rows up to 512 threads.  False: too wide.
template <class F>
bool with_shape(int64_t vectors, F&& f) {
  auto threads = [&](int vpt) { return int((vectors + vpt - 1) / vpt + 31) / 32 * 32; };
  using std::integral_constant;
#define MMA_SHAPE(V, T) \
  f(integral_constant<int, V>{}, integral_constant<int, T>{}, threads(V)), true
  if (vectors <= 256) return MMA_SHAPE(1, 256);
  if (vectors <= 512) return MMA_SHAPE(2, 256);
  if (vectors <= 768) return MMA_SHAPE(3, 256);
  if (vectors <= 1024) return MMA_SHAPE(4, 256);
  if (vectors <= 2048) return MMA_SHAPE(4, 512);
#undef MMA_SHAPE
  return false;
}

template <class T>
mma_status_t forward(const Ctx& ctx, const NormProblem& p, bool w32) {
  constexpr int E = Vec<T>::kN;
  const int64_t vectors = (p.N + E - 1) / E;
  auto launch = [&](auto vpt, auto maxt, int threads) {
    constexpr int V = decltype(vpt)::value, B = decltype(maxt)::value;
    // as many blocks as run at once, each taking rows in turn
    const int64_t most = int64_t(ctx.num_sms) * (768 / threads + (threads > 768));
    const unsigned grid = unsigned(std::min(p.M, most));
    if (p.N % E)
      rmsnorm_kernel<T, V, B, true><<<grid, threads, 0, ctx.stream>>>(p, w32);
    else
      rmsnorm_kernel<T, V, B, false><<<grid, threads, 0, ctx.stream>>>(p, w32);
  };
  bool fits = true;
  if (p.M <= ctx.num_sms && vectors <= 1024)
    // one row per SM at most: the whole row at once
    launch(std::integral_constant<int, 1>{}, std::integral_constant<int, 1024>{},
           int(vectors + 31) / 32 * 32);
  else
    fits = with_shape(vectors, launch);
  if (!fits)
    rmsnorm_wide_kernel<T><<<unsigned(p.M), 1024, 0, ctx.stream>>>(p, w32);
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

template <class T>
mma_status_t backward(const Ctx& ctx, const NormBackProblem& p, bool w32,
                      float* part, WaitHook hook = WaitHook{kWaitLimitNs, 0}) {
  constexpr int E = Vec<T>::kN;
  const int64_t vectors = (p.N + E - 1) / E;
  const int tensors = p.R ? 3 : 2;
  const NormBackShape shape = norm_back_shape(vectors, tensors);
  const int vpt = shape.vpt;
  const int at_once = (vpt ? shape.per_sm : 3) * ctx.num_sms;
  const int grid = int(std::min<int64_t>(p.M, std::min(kMostParts, at_once)));
  if (grid > 0 && vpt) {
    auto run = [&](auto kernel, PerContext<bool>& attr) {
      bool ok = false;
      if (!attr.get(ctx, &ok, [&](bool* v) {
            *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      220 * 1024) == cudaSuccess;
            if (!*v) cudaGetLastError();
            return *v;
          }))
        return false;
      kernel<<<grid, shape.threads, size_t(shape.stages) * tensors * vectors * 16,
               ctx.stream>>>(p, w32, shape.stages, int(vectors * 16), part, ctx.status,
                             hook);
      return true;
    };
    static PerContext<bool> a1, a2, a4;
    static PerContext<bool> t1, t2, t4;
    const bool ok =
        p.N % E ? vpt == 1   ? run(rmsnorm_backward_kernel<T, 1, true>, t1)
                  : vpt == 2 ? run(rmsnorm_backward_kernel<T, 2, true>, t2)
                             : run(rmsnorm_backward_kernel<T, 4, true>, t4)
        : vpt == 1 ? run(rmsnorm_backward_kernel<T, 1, false>, a1)
        : vpt == 2 ? run(rmsnorm_backward_kernel<T, 2, false>, a2)
                   : run(rmsnorm_backward_kernel<T, 4, false>, a4);
    if (!ok) return MMA_ERR_LAUNCH;
  } else if (grid > 0) {
    rmsnorm_backward_wide_kernel<T><<<grid, 1024, 0, ctx.stream>>>(p, w32, part);
  }
  return sum_parts(ctx, part, grid, p.N, p.DW, p.N, nullptr);
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

mma_status_t launch_rmsnorm_abort_selftest(const Ctx& ctx, int64_t limit_ns, const void* X,
                                           void* DX, float* DW, void* workspace) {
  const NormBackProblem p = {MMA_BF16, MMA_BF16, 1024, 1024, X, 1024, X, 1024, X, 1e-6f,
                             nullptr, 0, DX, 1024, DW, nullptr};
  return backward<__nv_bfloat16>(ctx, p, false, static_cast<float*>(workspace),
                                 WaitHook{static_cast<unsigned long long>(limit_ns), 1});
}

int64_t rmsnorm_backward_workspace_bytes(int64_t M, int64_t N) {
  return std::min<int64_t>(M, kMostParts) * N * 4;
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
