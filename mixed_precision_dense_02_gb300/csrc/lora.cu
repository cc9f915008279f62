// Low-rank adapters of many requests beside a shared product.  Rows are sorted by
// request, request i has rows [offsets[i], offsets[i + 1]) and an adapter (A, B):
//
//     s = scale * x A          `rank` sums per row        (lora_shrink_kernel)
//     d = x W + s B + c                                   (gemm_grouped.cu)
//
// and, from the gradient dy of d with u = scale * dy B^T (the same kernels on the
// transposed matrices), the adapters' own gradients over all their rows:
//
//     dA = sum of u^T x,   dB = sum of dy^T s             (lora_wgrad_kernel)
//
// A and B have one of two layouts, as W: K-major (A rank x K, B N x rank) or
// row-major (A K x rank, B rank x N).
//
// Pieces.  Both kernels cut the rows into blocks and at the requests' ends.  Piece
// (block i, request j) has the number i + j: as the rows go on, one of the two goes
// up from piece to piece, so the numbers are all different, and a number's request
// is the last j whose first block + j is not above it.  The rows before the first
// and after the last request count as requests without an adapter.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace mmagb {
namespace {

constexpr int kThreads = 256;

// The requests' bounds in shared memory: bound[0] = 0, then the offsets, within
// [0, T] and none below the one before it, then T; requests + 3 values.
__device__ __forceinline__ void load_bounds(int* bound, const int* offsets, int requests,
                                            int T, int* scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
  for (int base = 0; base <= requests; base += kThreads) {
    const int i = base + threadIdx.x;
    int v = i <= requests ? min(max(__ldg(offsets + i), 0), T) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v = max(v, o);
    }
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v = max(v, scan[w]);
    v = max(v, before);
    if (i <= requests) bound[i + 1] = v;
    for (int w = 0; w < kThreads / 32; ++w) before = max(before, scan[w]);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    bound[0] = 0;
    bound[requests + 2] = T;
  }
  __syncthreads();
}

// Piece `u` of blocks of `per` rows: its request (counted from the one before the
// first) and rows; none: from == to.
struct Piece {
  int request, from, to;
};

__device__ __forceinline__ Piece piece_of(const int* bound, int requests, int per, int u) {
  int n = 0;
  for (int base = 0; base < requests + 2; base += kThreads) {
    const int j = base + threadIdx.x;
    n += __syncthreads_count(j < requests + 2 && bound[j] / per + j <= u);
  }
  const int j = n - 1;  // (request 0 starts in block 0)
  const int64_t from = max(int64_t(u - j) * per, int64_t(bound[j]));
  const int to = int(min(int64_t(u - j + 1) * per, int64_t(bound[j + 1])));
  return Piece{j, int(min(from, int64_t(to))), to};
}

// The adapter of a request counted from the one before the first, or -1.
__device__ __forceinline__ int adapter_of(int j, int requests, const int* adapters, int total) {
  if (j < 1 || j > requests) return -1;
  const int a = adapters ? __ldg(adapters + j - 1) : j - 1;
  return a >= 0 && a < total ? a : -1;
}

// Byte offset of 16-byte chunk c of a row of ROW_BYTES, so that eight rows' chunks
// c are in different banks.
template <int ROW_BYTES>
__device__ __forceinline__ int swizzled(int row, int c) {
  constexpr int kChunks = ROW_BYTES / 16;
  const int line = ROW_BYTES >= 128 ? row : row * ROW_BYTES / 128;
  return row * ROW_BYTES + ((c ^ (line & (kChunks < 8 ? kChunks - 1 : 7))) << 4);
}

template <bool BF16>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  const uint32_t b[2] = {b0, b1};
  if constexpr (BF16)
    mma_bf16_16816(d, a, b);
  else
    mma_f16_16816(d, a, b);
}

// 16 bits of v; v becomes what they leave of it.
template <bool BF16>
__device__ __forceinline__ uint16_t take_half(float& v) {
  if constexpr (BF16) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    v -= __bfloat162float(h);
    return __bfloat16_as_ushort(h);
  } else {
    const __half h = __float2half_rn(v);
    v -= __half2float(h);
    return __half_as_ushort(h);
  }
}

// Copy 16 bytes of which the first `left` elements of two bytes are in the row.
__device__ __forceinline__ void copy_chunk(uint32_t dst, const uint16_t* src, int left,
                                           const void* any) {
  const int n = min(max(left, 0), 8) * 2;
  cp_async_16_zfill(dst, n ? static_cast<const void*>(src) : any, n);
}

// ------------------------------------------------------------- a row's sums

// Piece blockIdx.x of blocks of BM rows; the CTAs of a cluster (blockIdx.y) share
// the k range, and so do the warps that have the same 16 rows.  Stages of KS k's by
// cp.async; sums past the rank, rows past the piece and k's past K are zeros.
template <int BM, int RP>
struct Shrink {
  static constexpr int MW = BM / 16, KW = 8 / MW;  // warps along rows, along k
  static constexpr int KS = KW * 32;
  static constexpr int X_BYTES = BM * KS * 2, A_BYTES = RP * KS * 2;
  static constexpr int STAGE = X_BYTES + A_BYTES;
  static constexpr int STAGES = 4 * STAGE <= 200 * 1024 ? 4 : 3;
  static constexpr int SMEM = STAGES * STAGE;  // (the sums: 512 * RP bytes of them)
};

template <bool BF16, bool ROW, int BM, int RP>
__global__ void __launch_bounds__(kThreads)
    lora_shrink_kernel(const LoraProblem g, const LoraLow low) {
  using L = Shrink<BM, RP>;
  constexpr int KS = L::KS;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int bound[MMA_MAX_GROUPS + 3], scan[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependents_start();
  load_bounds(bound, g.offsets, int(g.requests), int(g.rows), scan);
  const Piece piece = piece_of(bound, int(g.requests), BM, blockIdx.x);
  const int who =
      adapter_of(piece.request, int(g.requests), g.adapters, int(g.adapters_total));
  const int rows = piece.to - piece.from, rank = int(g.rank);
  // (the same in all CTAs of the cluster, so that all of them return)
  if (rows <= 0) return;
  const int part = blockIdx.y, parts = gridDim.y;
  auto put = [&](int row, int n, float v) {
    const int64_t t = piece.from + row;
    if (n >= rank) v = 0.f;
    if (n < low.ld32) low.f32[t * low.ld32 + n] = v;
    if (n < low.ld16) {
      uint16_t* d = static_cast<uint16_t*>(low.f16) + t * low.ld16 + n;
      for (int i = 0; i < low.parts; ++i) d[i * g.rows * low.ld16] = take_half<BF16>(v);
    }
  };
  if (who < 0) {
    for (int i = part * kThreads + threadIdx.x; i < rows * RP; i += parts * kThreads)
      put(i / RP, i % RP, 0.f);
    return;
  }
  const uint16_t* const X = static_cast<const uint16_t*>(g.X) + piece.from * g.ldx;
  const uint16_t* const A = static_cast<const uint16_t*>(g.A) + who * g.stride_a;
  const int K = int(g.K);
  const int all = (K + KS - 1) / KS;
  const int first = int(int64_t(all) * part / parts), last = int(int64_t(all) * (part + 1) / parts);
  const uint32_t base = smem_u32(smem);
  auto load = [&](int step) {
    const int k0 = step * KS;
    const uint32_t xs = base + (step - first) % L::STAGES * L::STAGE, as = xs + L::X_BYTES;
#pragma unroll
    for (int i = threadIdx.x; i < BM * KS / 8; i += kThreads) {
      const int row = i / (KS / 8), c = i % (KS / 8), k = k0 + c * 8;
      copy_chunk(xs + swizzled<KS * 2>(row, c), X + row * g.ldx + k, row < rows ? K - k : 0,
                 g.X);
    }
#pragma unroll
    for (int i = threadIdx.x; i < RP * KS / 8; i += kThreads) {
      if constexpr (!ROW) {
        const int n = i / (KS / 8), c = i % (KS / 8), k = k0 + c * 8;
        copy_chunk(as + swizzled<KS * 2>(n, c), A + n * g.lda + k, n < rank ? K - k : 0, g.X);
      } else {
        const int row = i / (RP / 8), c = i % (RP / 8), k = k0 + row;
        copy_chunk(as + swizzled<RP * 2>(row, c), A + k * g.lda + c * 8,
                   k < K ? rank - c * 8 : 0, g.X);
      }
    }
  };
  float acc[RP / 8][4];
#pragma unroll
  for (int n = 0; n < RP / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
#pragma unroll
  for (int s = 0; s < L::STAGES - 1; ++s) {
    if (first + s < last) load(first + s);
    cp_async_commit();
  }
  const int mw = warp % L::MW, kw = warp / L::MW;
  for (int step = first; step < last; ++step) {
    cp_async_wait<L::STAGES - 2>();
    __syncthreads();  // this stage has landed, and the one before has been read
    if (step + L::STAGES - 1 < last) load(step + L::STAGES - 1);
    cp_async_commit();
    const uint32_t xs = base + (step - first) % L::STAGES * L::STAGE, as = xs + L::X_BYTES;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int k = kw * 32 + kk * 16;
      uint32_t a[4];
      ldmatrix_x4(a, xs + swizzled<KS * 2>(mw * 16 + (lane & 15), k / 8 + (lane >> 4)));
#pragma unroll
      for (int n = 0; n < RP / 16; ++n) {
        uint32_t b[4];
        const int m = lane >> 3, at = lane & 7;
        if constexpr (!ROW)
          ldmatrix_x4(b, as + swizzled<KS * 2>(n * 16 + (m >> 1) * 8 + at, k / 8 + (m & 1)));
        else
          ldmatrix_x4_trans(b, as + swizzled<RP * 2>(k + (m & 1) * 8 + at, n * 2 + (m >> 1)));
        mma16<BF16>(acc[2 * n], a, b[0], b[1]);
        mma16<BF16>(acc[2 * n + 1], a, b[2], b[3]);
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();
  // the warps' sums, then the CTAs', each in order
  float* sums = reinterpret_cast<float*>(smem);  // [KW][BM][RP]
#pragma unroll
  for (int n = 0; n < RP / 8; ++n) {
    float* d = sums + (kw * BM + mw * 16 + (lane >> 2)) * RP + n * 8 + 2 * (lane & 3);
    d[0] = acc[n][0];
    d[1] = acc[n][1];
    d[8 * RP] = acc[n][2];
    d[8 * RP + 1] = acc[n][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < BM * RP; i += kThreads) {
    float v = sums[i];
#pragma unroll
    for (int w = 1; w < L::KW; ++w) v += sums[w * BM * RP + i];
    sums[i] = v;  // (read by this thread alone)
  }
  const float scale = g.scales ? __ldg(g.scales + who) : 1.f;
  if (parts > 1) cluster_sync();
  else __syncthreads();
  const int share = BM * RP / parts;
  for (int i = part * share + threadIdx.x; i < (part + 1) * share; i += kThreads) {
    float v = 0.f;
    if (parts > 1) {
      for (int r = 0; r < parts; ++r)
        v += ld_shared_cluster_f32(mapa_shared(smem_u32(sums + i), r));
    } else {
      v = sums[i];
    }
    if (i / RP < rows) put(i / RP, i % RP, v * scale);
  }
  if (parts > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

template <bool BF16, bool ROW, int BM, int RP>
mma_status_t shrink(const Ctx& ctx, const LoraProblem& g, const LoraLow& low) {
  using L = Shrink<BM, RP>;
  auto kernel = lora_shrink_kernel<BF16, ROW, BM, RP>;
  static PerContext<bool> attr;
  bool ok = false;
  if (!attr.get(ctx, &ok, [&](bool* v) {
        *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  L::SMEM) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return MMA_ERR_LAUNCH;
  const int64_t pieces = (g.rows + BM - 1) / BM + g.requests + 1;
  const int64_t steps = (g.K + L::KS - 1) / L::KS;
  // as many CTAs per piece as fill the SMs twice, each with four stages at least
  int parts = 1;
  while (parts < 8 && pieces * parts * 2 <= 2 * ctx.num_sms && steps >= parts * 8) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(pieces), unsigned(parts), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = L::SMEM;
  cfg.stream = ctx.stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 1;
  at.val.clusterDim.y = unsigned(parts);
  at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, g, low);
  const cudaError_t after = cudaGetLastError();
  return e == cudaSuccess && after == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

// Calls f for the rank rounded up to 16, 32, 64 or 128.
template <class F>
mma_status_t by_rank(int64_t rank, F&& f) {
  if (rank <= 16) return f(std::integral_constant<int, 16>{});
  if (rank <= 32) return f(std::integral_constant<int, 32>{});
  if (rank <= 64) return f(std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 128>{});
}

// ----------------------------------------------- what the sums add, few rows

// extra[row][p] = sum over n of s[row][n] B[n][p], FP32, a lane per p: of every row
// (EVERY: pieces of eight rows, zeros where there is no adapter) or of the requests
// of fewer than kLoraRows rows.  Bound by B's bytes and latency.  The grid is small
// enough to be on the SMs at once with its neighbours, so that the shared product
// after it starts before it ends.
template <bool BF16, bool ROW, bool EVERY>
__global__ void __launch_bounds__(kThreads)
    lora_expand_kernel(const LoraProblem g, const LoraLow low, int units) {
  constexpr int kCols = 4;  // p per thread at a time, their loads together
  __shared__ int bound[MMA_MAX_GROUPS + 3], scan[kThreads / 32];
  grid_dependents_start();
  const int requests = int(g.requests), rank = int(g.rank), N = int(g.N);
  load_bounds(bound, g.offsets, requests, int(g.rows), scan);
  bool ready = false;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    Piece piece;
    if constexpr (EVERY) {
      piece = piece_of(bound, requests, 8, u);
    } else {
      piece = Piece{u + 1, bound[u + 1], bound[u + 2]};
      if (piece.to - piece.from >= kLoraRows) continue;
    }
    if (piece.to <= piece.from) continue;
    const int who = adapter_of(piece.request, requests, g.adapters, int(g.adapters_total));
    if (!EVERY && who < 0) continue;
    const uint16_t* const B = static_cast<const uint16_t*>(g.B) + (who < 0 ? 0 : who * g.stride_b);
    // (the offsets and B are older than the kernel before this one, the sums are not)
    if (!ready) grid_dependency_wait();
    ready = true;
    for (int p0 = blockIdx.y * kThreads * kCols; p0 < N; p0 += gridDim.y * kThreads * kCols) {
      for (int t = piece.from; t < piece.to; ++t) {
        const float* s = low.f32 + int64_t(t) * low.ld32;
        float v[kCols];
#pragma unroll
        for (int x = 0; x < kCols; ++x) v[x] = 0.f;
#pragma unroll 1
        for (int k = 0; k < rank && who >= 0; k += 8) {
          uint4 w[kCols];
          const int left = rank - k;
#pragma unroll
          for (int x = 0; x < kCols; ++x) {
            const int p = p0 + x * kThreads + threadIdx.x;
            w[x] = make_uint4(0, 0, 0, 0);
            if (p >= N) continue;
            if constexpr (ROW) {
              uint32_t f[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) f[y] = y < left ? B[(k + y) * g.ldb + p] : 0u;
              w[x] = make_uint4(f[0] | f[1] << 16, f[2] | f[3] << 16, f[4] | f[5] << 16,
                                f[6] | f[7] << 16);
            } else {
              w[x] = __ldg(reinterpret_cast<const uint4*>(B + p * g.ldb + k));
            }
          }
          const float4 s0 = *reinterpret_cast<const float4*>(s + k);
          const float4 s1 = *reinterpret_cast<const float4*>(s + k + 4);
          const float2 f[4] = {make_float2(s0.x, s0.y), make_float2(s0.z, s0.w),
                               make_float2(s1.x, s1.y), make_float2(s1.z, s1.w)};
#pragma unroll
          for (int x = 0; x < kCols; ++x) {
            uint32_t q[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              // (what stands behind a row's rank numbers is none of them)
              if (!ROW && left < 2 * y + 2) q[y] = left <= 2 * y ? 0u : q[y] & 0xFFFFu;
              float2 b;
              if constexpr (BF16)
                b = make_float2(__uint_as_float(q[y] << 16), __uint_as_float(q[y] & 0xFFFF0000u));
              else
                b = __half22float2(*reinterpret_cast<const __half2*>(&q[y]));
              v[x] = fmaf(f[y].x, b.x, v[x]);
              v[x] = fmaf(f[y].y, b.y, v[x]);
            }
          }
        }
        const int64_t row =
            EVERY ? t : int64_t(u) * (kLoraRows - 1) + t - piece.from;
#pragma unroll
        for (int x = 0; x < kCols; ++x) {
          const int p = p0 + x * kThreads + threadIdx.x;
          if (p < N) low.extra[row * N + p] = v[x];
        }
      }
    }
  }
  // (a kernel after this one may count on the one before being done)
  if (!ready) grid_dependency_wait();
}

template <bool BF16, bool ROW>
mma_status_t expand(const Ctx& ctx, const LoraProblem& g, const LoraLow& low) {
  const bool every = g.rows <= kLoraEveryRow;
  const int64_t units = every ? (g.rows + 7) / 8 + g.requests + 1 : g.requests;
  const int64_t columns = (g.N + kThreads * 4 - 1) / (kThreads * 4);
  const int64_t most = ctx.num_sms * 2;
  const int64_t x = std::min(units, most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(x), unsigned(std::max<int64_t>(1, std::min(columns, most / x))), 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, every ? lora_expand_kernel<BF16, ROW, true>
                                     : lora_expand_kernel<BF16, ROW, false>,
                         g, low, int(units));
  const cudaError_t after = cudaGetLastError();
  return e == cudaSuccess && after == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

// ------------------------------------------------- the adapters' own gradients

// One side of the gradient: features of M (T x F) times the rows' sums.
struct Side {
  const uint16_t* m;
  int64_t ldm;
  int F;
  const float* low;  // T x rank, FP32
  int64_t ldl;
  void* out;  // per adapter: `by_rank` rank x F, else F x rank
  int64_t ldo, slice;
  bool by_rank;
};

struct WgradArgs {
  Side side[2];  // the gradients of B (M = dy, s) and of A (M = x, u)
  int tiles0;    // tiles of 128 features of the first side
  int T, rank, requests, total, per;
  const int *offsets, *adapters;
  int d_type, parts;
  bool accumulate;
  float* part;  // [pieces][rank][features of both sides]
};

constexpr int kTile = 128;      // features per CTA, 16 per warp
constexpr int kStageRows = 64;  // rows per stage

template <int RP>
struct Wgrad {
  static constexpr int M_BYTES = kStageRows * kTile * 2, L_BYTES = kStageRows * RP * 4;
  static constexpr int STAGE = M_BYTES + L_BYTES;
  static constexpr int HALF_BYTES = kStageRows * RP * 2;  // the sums in 16 bits, a part
  static constexpr int STAGES = RP <= 64 ? 4 : 3;
  static constexpr int SMEM = STAGES * STAGE + 3 * HALF_BYTES;
};

// Piece blockIdx.x's share of 128 features: G[f][n] = sum over its rows M[t][f] *
// low[t][n] on the tensor cores, FP32.  The sums come in FP32 and are taken as a sum
// of `parts` numbers of 16 bits (see lora_parts).
template <bool BF16, int RP>
__global__ void __launch_bounds__(kThreads)
    lora_wgrad_kernel(const WgradArgs a) {
  using L = Wgrad<RP>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int bound[MMA_MAX_GROUPS + 3], scan[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  load_bounds(bound, a.offsets, a.requests, a.T, scan);
  const Piece piece = piece_of(bound, a.requests, a.per, blockIdx.x);
  const int rows = piece.to - piece.from;
  if (rows <= 0 || adapter_of(piece.request, a.requests, a.adapters, a.total) < 0) return;
  const bool second = int(blockIdx.y) >= a.tiles0;
  const Side& side = a.side[second];
  const int f0 = (int(blockIdx.y) - (second ? a.tiles0 : 0)) * kTile;
  const uint16_t* const M = side.m + piece.from * side.ldm + f0;
  const float* const S = side.low + piece.from * side.ldl;
  const int F = side.F - f0, rank = a.rank;
  // 16 bytes of a row of sums at a time
  const bool wide = side.ldl % 4 == 0 && (reinterpret_cast<uintptr_t>(side.low) & 15) == 0;
  const uint32_t base = smem_u32(smem), half = base + L::STAGES * L::STAGE;
  const int steps = (rows + kStageRows - 1) / kStageRows;
  auto load = [&](int step) {
    const uint32_t ms = base + step % L::STAGES * L::STAGE, ls = ms + L::M_BYTES;
#pragma unroll
    for (int i = threadIdx.x; i < kStageRows * kTile / 8; i += kThreads) {
      const int row = i / (kTile / 8), c = i % (kTile / 8), t = step * kStageRows + row;
      copy_chunk(ms + swizzled<kTile * 2>(row, c), M + t * side.ldm + c * 8,
                 t < rows ? F - c * 8 : 0, side.m);
    }
#pragma unroll
    for (int i = threadIdx.x; i < kStageRows * RP / 4; i += kThreads) {
      const int row = i / (RP / 4), c = i % (RP / 4), t = step * kStageRows + row;
      const int n = t < rows ? min(max(rank - c * 4, 0), 4) : 0;
      const float* src = S + t * side.ldl + c * 4;
      if (wide) {
        cp_async_16_zfill(ls + i * 16, n ? src : side.low, n * 4);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          cp_async_4_zfill(ls + i * 16 + j * 4, j < n ? src + j : side.low, j < n ? 4 : 0);
      }
    }
  };
  float acc[RP / 8][4];
#pragma unroll
  for (int n = 0; n < RP / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
#pragma unroll
  for (int s = 0; s < L::STAGES - 1; ++s) {
    if (s < steps) load(s);
    cp_async_commit();
  }
  for (int step = 0; step < steps; ++step) {
    cp_async_wait<L::STAGES - 2>();
    __syncthreads();  // this stage has landed, and the one before has been read
    if (step + L::STAGES - 1 < steps) load(step + L::STAGES - 1);
    cp_async_commit();
    const uint32_t ms = base + step % L::STAGES * L::STAGE;
    const float* ls = reinterpret_cast<const float*>(smem + step % L::STAGES * L::STAGE +
                                                     L::M_BYTES);
    for (int i = threadIdx.x; i < kStageRows * RP / 8; i += kThreads) {
      const int row = i / (RP / 8), c = i % (RP / 8);
      float v[8];
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(ls + i * 8);
      *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(ls + i * 8 + 4);
      uint8_t* d = smem + L::STAGES * L::STAGE + swizzled<RP * 2>(row, c);
      for (int part = 0; part < a.parts; ++part, d += L::HALF_BYTES) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t h0 = take_half<BF16>(v[2 * j]), h1 = take_half<BF16>(v[2 * j + 1]);
          w[j] = h0 | h1 << 16;
        }
        *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStageRows; k += 16) {
      const int m = lane >> 3, at = lane & 7;
      uint32_t f[4];
      ldmatrix_x4_trans(f, ms + swizzled<kTile * 2>(k + (m >> 1) * 8 + at, warp * 2 + (m & 1)));
#pragma unroll
      for (int n = 0; n < RP / 16; ++n) {
        uint32_t b[4];
        const int where = swizzled<RP * 2>(k + (m & 1) * 8 + at, n * 2 + (m >> 1));
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          if (part >= a.parts) continue;
          ldmatrix_x4_trans(b, half + part * L::HALF_BYTES + where);
          mma16<BF16>(acc[2 * n], f, b[0], b[1]);
          mma16<BF16>(acc[2 * n + 1], f, b[2], b[3]);
        }
      }
    }
  }
  cp_async_wait<0>();
  // rows of features per sum, through shared memory
  __syncthreads();
  float* t = reinterpret_cast<float*>(smem);  // [RP][kTile + 4]
#pragma unroll
  for (int n = 0; n < RP / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      t[(n * 8 + 2 * (lane & 3) + (j & 1)) * (kTile + 4) + warp * 16 + (lane >> 2) +
        (j >> 1) * 8] = acc[n][j];
  __syncthreads();
  const int64_t features = a.side[0].F + a.side[1].F;
  float* out = a.part + int64_t(blockIdx.x) * rank * features + (second ? a.side[0].F : 0) + f0;
  for (int i = threadIdx.x; i < rank * kTile; i += kThreads)
    if (i % kTile < F) out[i / kTile * features + i % kTile] = t[i / kTile * (kTile + 4) + i % kTile];
}

__device__ __forceinline__ float load_out(const void* p, int64_t i, int type) {
  if (type == MMA_F32) return static_cast<const float*>(p)[i];
  if (type == MMA_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void store_out(void* p, int64_t i, int type, float v) {
  if (type == MMA_F32)
    static_cast<float*>(p)[i] = v;
  else if (type == MMA_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Adapter blockIdx.y: its pieces' shares added in order, for 256 features of each
// of the rank's sums in turn.
__global__ void __launch_bounds__(kThreads)
    lora_wgrad_sum_kernel(const WgradArgs a) {
  __shared__ int bound[MMA_MAX_GROUPS + 3], scan[kThreads / 32], list[MMA_MAX_GROUPS], found;
  load_bounds(bound, a.offsets, a.requests, a.T, scan);
  if (threadIdx.x < 32) {
    int n = 0;
    for (int base = 0; base < a.requests; base += 32) {
      const int i = base + threadIdx.x;
      const bool mine = i < a.requests && (a.adapters ? a.adapters[i] : i) == int(blockIdx.y) &&
                        bound[i + 2] > bound[i + 1];
      const unsigned which = __ballot_sync(0xffffffffu, mine);
      if (mine) list[n + __popc(which & ((1u << threadIdx.x) - 1))] = i;
      n += __popc(which);
    }
    if (threadIdx.x == 0) found = n;
  }
  __syncthreads();
  const int features = a.side[0].F + a.side[1].F;
  const int at = blockIdx.x * kThreads + threadIdx.x;
  if (at >= features) return;
  const bool second = at >= a.side[0].F;
  const Side& side = a.side[second];
  const int f = at - (second ? a.side[0].F : 0);
  const int64_t out = int64_t(blockIdx.y) * side.slice;
  for (int n = blockIdx.z; n < a.rank; n += gridDim.z) {
    float v = 0.f;
    for (int i = 0; i < found; ++i) {
      const int j = list[i] + 1;
      const int first = bound[j] / a.per, last = (bound[j + 1] - 1) / a.per;
      for (int b = first; b <= last; ++b)
        v += a.part[(int64_t(b + j) * a.rank + n) * features + at];
    }
    const int64_t o = out + (side.by_rank ? n * side.ldo + f : f * side.ldo + n);
    if (a.accumulate) {
      if (found == 0) continue;
      v += load_out(side.out, o, a.d_type);
    }
    store_out(side.out, o, a.d_type, v);
  }
}

// Rows per block: some four pieces of work per SM (of 152, so that the workspace
// needs no device), 256 rows at least, in whole stages.
int rows_per_piece(int64_t T, int64_t N, int64_t K) {
  const int64_t tiles = (N + kTile - 1) / kTile + (K + kTile - 1) / kTile;
  const int64_t per = T * tiles / (4 * 152);
  return int(std::min<int64_t>(std::max<int64_t>((per + 63) / 64 * 64, 256), 1 << 20));
}

template <bool BF16, int RP>
mma_status_t wgrad(const Ctx& ctx, const WgradArgs& a, int tiles, int64_t pieces) {
  using L = Wgrad<RP>;
  auto kernel = lora_wgrad_kernel<BF16, RP>;
  static PerContext<bool> attr;
  bool ok = false;
  if (!attr.get(ctx, &ok, [&](bool* v) {
        *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  L::SMEM) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return MMA_ERR_LAUNCH;
  static_assert(RP * (kTile + 4) * 4 <= L::SMEM, "the sums' transposition");
  ctx.mark_start();
  if (a.T > 0)
    kernel<<<dim3(unsigned(pieces), unsigned(tiles)), kThreads, L::SMEM, ctx.stream>>>(a);
  ctx.mark_stop();
  const int64_t features = int64_t(a.side[0].F) + a.side[1].F;
  lora_wgrad_sum_kernel<<<dim3(unsigned((features + kThreads - 1) / kThreads), unsigned(a.total),
                               unsigned(std::min(a.rank, 8))),
                          kThreads, 0, ctx.stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

}  // namespace

mma_status_t launch_lora_shrink(const Ctx& ctx, const LoraProblem& g, const LoraLow& low) {
  return by_rank(g.rank, [&](auto r) {
    constexpr int RP = decltype(r)::value;
    auto go = [&](auto bf16, auto row) {
      constexpr bool B = decltype(bf16)::value, R = decltype(row)::value;
      // (few rows: the k range over all eight warps)
      return g.rows <= 256 ? shrink<B, R, 16, RP>(ctx, g, low)
                           : shrink<B, R, 64, RP>(ctx, g, low);
    };
    if (g.bf16)
      return g.row_major ? go(std::true_type{}, std::true_type{})
                         : go(std::true_type{}, std::false_type{});
    return g.row_major ? go(std::false_type{}, std::true_type{})
                       : go(std::false_type{}, std::false_type{});
  });
}

mma_status_t launch_lora_expand(const Ctx& ctx, const LoraProblem& g, const LoraLow& low) {
  if (g.bf16)
    return g.row_major ? expand<true, true>(ctx, g, low) : expand<true, false>(ctx, g, low);
  return g.row_major ? expand<false, true>(ctx, g, low) : expand<false, false>(ctx, g, low);
}

int64_t lora_wgrad_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t rank,
                                   int64_t requests) {
  const int64_t per = rows_per_piece(T, N, K);
  return T == 0 ? 0 : ((T + per - 1) / per + requests + 1) * rank * (N + K) * 4;
}

mma_status_t launch_lora_wgrad(const Ctx& ctx, const LoraWgradProblem& g, float* workspace) {
  WgradArgs a = {};
  a.side[0] = {static_cast<const uint16_t*>(g.DY), g.lddy, int(g.N), g.S, g.lds,
               g.DB, g.lddb, g.stride_db, false};
  a.side[1] = {static_cast<const uint16_t*>(g.X), g.ldx, int(g.K), g.U, g.ldu,
               g.DA, g.ldda, g.stride_da, true};
  a.tiles0 = int((g.N + kTile - 1) / kTile);
  a.T = int(g.rows);
  a.rank = int(g.rank);
  a.requests = int(g.requests);
  a.total = int(g.adapters_total);
  a.per = rows_per_piece(g.rows, g.N, g.K);
  a.offsets = g.offsets;
  a.adapters = g.adapters;
  a.d_type = g.d_type;
  a.parts = lora_parts(g.bf16, g.d_type);
  a.accumulate = g.accumulate;
  a.part = workspace;
  const int tiles = a.tiles0 + int((g.K + kTile - 1) / kTile);
  const int64_t pieces = (g.rows + a.per - 1) / a.per + g.requests + 1;
  return by_rank(g.rank, [&](auto r) {
    constexpr int RP = decltype(r)::value;
    return g.bf16 ? wgrad<true, RP>(ctx, a, tiles, pieces)
                  : wgrad<false, RP>(ctx, a, tiles, pieces);
  });
}

}  // namespace mmagb
