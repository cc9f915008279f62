// Quantisation to 8-bit floating point (E4M3 or E5M2) with a scale for each
// block of 128 values of a row, or of 128 x 128 values, as it is or
// transposed:
//     s_b = max(max|x| over block b / format's largest value, 2^-126)
//     q = x / s_b, the FP32 quotient rounded to nearest
//
// The transposed form serves products that reduce over what is the row index
// here: the weight's transpose for an input gradient, an activation's or
// gradient's transpose for a weight gradient, because 8-bit operands of the
// tensor core are read along the reduction.  Its row blocks run along the
// output's rows, that is, down the input's columns.
//
// Bound by memory: x is read once, q written once.  16384 x 2048 BF16 by rows:
// 19.5 us, 5.2 TB/s; 4000 x 8192 FP32 by squares, transposed: 29.4 us,
// 5.6 TB/s; 8192 x 8192 BF16 by squares 33.8 us, by rows transposed 34.7.
#include <algorithm>

#include <cudaTypedefs.h>

#include "f8_common.cuh"
#include "ptx.cuh"

namespace mmagb {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm_tc.cu

namespace {

// Blocks of 1 x 128, not transposed: a group of lanes per block of columns,
// four rows at a time.  The scales and their reciprocals are made for the four
// rows at once, each by another lane of the group (by every lane for itself:
// 16384 x 2048 BF16 20.5 us, so 19.6).
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
      for (int j = 0; j < E; j += 2) m[i] = abs_max(m[i], x[i][j], x[i][j + 1]);
#pragma unroll
      for (int d = kLanes / 2; d > 0; d >>= 1)
        m[i] = abs_max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
    }
    const int mine = lane & (kRowsAtOnce - 1);
    const float mm = mine & 2 ? (mine & 1 ? m[3] : m[2]) : (mine & 1 ? m[1] : m[0]);
    const float s = block_scale<E5M2>(mm, p.pow2);
    const Divisor by(s);
    if (b * kScaleBlock < p.N && lane % kLanes < kRowsAtOnce && row0 + mine < p.M)
      p.S[(row0 + mine) * p.s_row + b * p.s_blk] = s;
#pragma unroll
    for (int i = 0; i < kRowsAtOnce; ++i) {
      const Divisor d = by.from((lane & ~(kLanes - 1)) + i);
      if (live && row0 + i < p.M)
        store_f8<E5M2, E, TAIL>(static_cast<uint8_t*>(p.Q) + (row0 + i) * p.ldq, v,
                                p.N, x[i], d);
    }
  }
}

// 128 x 128 tiles in turn per block, the next two on their way by TMA while
// one is worked on (one tile per block, loaded by its threads, left memory
// idle in between: 4000 x 8192 FP32 took 60 us).  A thread has RPT = 8
// consecutive rows of one vector of E columns.  SQUARE: one scale for the
// tile, else (transposed only) one per column.  The transposed bytes go
// through shared memory, eight of one column at a time; a row's 8-byte pieces
// are permuted by the column's vector so that neither side has bank
// conflicts.
template <class T>
struct Tile {
  static constexpr int E = Vec<T>::kN;
  static constexpr int VEC = kScaleBlock / E;   // vectors per tile row
  static constexpr int RPT = 8;
  static constexpr int THREADS = VEC * kScaleBlock / RPT;
  static constexpr int BYTES = kScaleBlock * kScaleBlock * int(sizeof(T));
  static constexpr int STAGES = 2;
  static constexpr int SMEM = STAGES * BYTES + kScaleBlock * kScaleBlock + 128;
  static constexpr int PER_SM = sizeof(T) == 4 ? 1 : 2;
};

template <class T, bool E5M2, bool SQUARE, bool TRANS>
__global__ void __launch_bounds__(Tile<T>::THREADS, Tile<T>::PER_SM)
    quantize_tile_kernel(const __grid_constant__ CUtensorMap map,
                         const QuantProblem p, int64_t tiles_n, int64_t tiles,
                         unsigned* status, const WaitHook hook) {
  using L = Tile<T>;
  constexpr int E = L::E, VEC = L::VEC, RPT = L::RPT;
  constexpr int TR = kScaleBlock / RPT;  // rows of threads
  constexpr int WARPS = L::THREADS / 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint8_t* turned = smem + L::STAGES * L::BYTES;
  __shared__ float red[SQUARE ? 2 * WARPS : TR * kScaleBlock];
  __shared__ float scale_of[SQUARE ? 1 : kScaleBlock];
  __shared__ uint64_t full[L::STAGES];
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::STAGES; ++s) mbar_init(&full[s], 1);
    abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  __syncthreads();
  auto fetch = [&](int64_t t, int s) {
    if (t >= tiles || hook.withhold) return;
    mbar_arrive_expect_tx(&full[s], L::BYTES);
    tma_load_3d(&map, &full[s], smem + s * L::BYTES,
                int(t % tiles_n) * kScaleBlock, int(t / tiles_n) * kScaleBlock, 0);
  };
  if (threadIdx.x == 0)
    for (int s = 0; s < L::STAGES; ++s)
      fetch(blockIdx.x + int64_t(s) * gridDim.x, s);
  const int c = threadIdx.x % VEC, tr = threadIdx.x / VEC;
  int s = 0, flip = 0;
  uint32_t phase = 0;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, flip ^= 1) {
    const int64_t tm = t / tiles_n, tn = t - tm * tiles_n;
    const int64_t m0 = tm * kScaleBlock, n0 = tn * kScaleBlock;
    // A failed wait ends the block behind the next barrier, before anything is
    // stored or fetched.
    const bool failed = !mbar_wait(&full[s], phase, &abort_flag, status, hook.limit_ns);
    // thread 0 lets this tile's and the next ones' loads land
    auto drain = [&] {
      if (threadIdx.x == 0)
        for (int k = 0; k < L::STAGES && t + k * int64_t(gridDim.x) < tiles; ++k)
          mbar_drain(&full[(s + k) % L::STAGES], phase ^ uint32_t(s + k >= L::STAGES), status,
                     hook.limit_ns);
    };
    float x[RPT][E];
    const uint4* src = reinterpret_cast<const uint4*>(smem + s * L::BYTES);
#pragma unroll
    for (int i = 0; i < RPT; ++i) Vec<T>::unpack(src[(tr * RPT + i) * VEC + c], x[i]);
    float scale[SQUARE ? 1 : E];
    if constexpr (SQUARE) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < E; j += 2) m = abs_max(m, x[i][j], x[i][j + 1]);
      const uint32_t w = __reduce_max_sync(0xffffffffu, abs_bits(m));
      if ((threadIdx.x & 31) == 0) red[flip * WARPS + (threadIdx.x >> 5)] = __uint_as_float(w);
      if (__syncthreads_or(failed)) return drain();
      m = 0.f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) m = abs_max(m, red[flip * WARPS + k]);
      const float sc = block_scale<E5M2>(m, p.pow2);
      scale[0] = sc;
      if (threadIdx.x == 0)
        p.S[(TRANS ? tn : tm) * p.s_row + (TRANS ? tm : tn) * p.s_blk] = sc;
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; i += 2) m = abs_max(m, x[i][j], x[i + 1][j]);
        red[tr * kScaleBlock + j * VEC + c] = m;  // j-major: no conflicts
      }
      if (__syncthreads_or(failed)) return drain();
      if (threadIdx.x < kScaleBlock) {
        const int col = (threadIdx.x % VEC) * E + threadIdx.x / VEC;
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < TR; ++k) m = abs_max(m, red[k * kScaleBlock + threadIdx.x]);
        const float sc = block_scale<E5M2>(m, p.pow2);
        scale_of[threadIdx.x] = sc;
        if (n0 + col < p.N) p.S[(n0 + col) * p.s_row + tm * p.s_blk] = sc;
      }
    }
    // every thread has taken its part of the stage
    if (threadIdx.x == 0) fetch(t + int64_t(L::STAGES) * gridDim.x, s);
    if (++s == L::STAGES) {
      s = 0;
      phase ^= 1u;
    }
    if constexpr (!SQUARE) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < E; ++j) scale[j] = scale_of[j * VEC + c];
    }
    if constexpr (!TRANS) {
      const int64_t v = n0 / E + c;
      const Divisor d(scale[0]);
      if (v * E < p.N)
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const int64_t row = m0 + tr * RPT + i;
          if (row < p.M)
            store_f8<E5M2>(static_cast<uint8_t*>(p.Q) + row * p.ldq, v, p.N, x[i],
                           d);
        }
    } else {
      if constexpr (SQUARE) {
        // (here, where the registers of a pair are side by side: 4000 x 8192
        // FP32 29.6 us, below 30.0; with a divisor per column 8192 x 8192 BF16
        // 34.8 us, below 33.7)
        const Divisor d(scale[0]);
#pragma unroll
        for (int i = 0; i < RPT; ++i)
#pragma unroll
          for (int j = 0; j < E; j += 2) {
            const float2 v = d(x[i][j], x[i][j + 1]);
            x[i][j] = v.x;
            x[i][j + 1] = v.y;
          }
      }
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const Divisor d(scale[SQUARE ? 0 : j]);
        auto pair = [&](int i) {
          return to_f8x2<E5M2>(SQUARE ? make_float2(x[i][j], x[i + 1][j])
                                      : d(x[i][j], x[i + 1][j]));
        };
        const uint32_t w[2] = {pair(0) | (pair(2) << 16), pair(4) | (pair(6) << 16)};
        *reinterpret_cast<uint2*>(turned + (c * E + j) * kScaleBlock +
                                  ((tr ^ (c & 15)) << 3)) = make_uint2(w[0], w[1]);
      }
      __syncthreads();
      // 16-byte chunks of the output's rows
#pragma unroll
      for (int i = 0; i < kScaleBlock * 8 / L::THREADS; ++i) {
        const int k = threadIdx.x + L::THREADS * i;
        const int n = k >> 3, ch = k & 7, sw = (n / E) & 15;
        if (n0 + n >= p.N || m0 + ch * 16 >= p.M) continue;
        uint4 v = *reinterpret_cast<const uint4*>(turned + n * kScaleBlock +
                                                  ((ch ^ (sw >> 1)) << 4));
        if (sw & 1) v = make_uint4(v.z, v.w, v.x, v.y);
        uint8_t* dst = static_cast<uint8_t*>(p.Q) + (n0 + n) * p.ldq + m0 + ch * 16;
        if (m0 + ch * 16 + 16 <= p.M) {
          *reinterpret_cast<uint4*>(dst) = v;
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int b = 0; b < 15; ++b)
            if (m0 + ch * 16 + b < p.M) dst[b] = uint8_t(w[b >> 2] >> (8 * (b & 3)));
        }
      }
    }
  }
}

template <class T, bool E5M2, bool SQUARE, bool TRANS>
mma_status_t run_tiles(const Ctx& ctx, const QuantProblem& p,
                       WaitHook hook = WaitHook{kWaitLimitNs, 0}) {
  using L = Tile<T>;
  const int64_t tiles_n = (p.N + kScaleBlock - 1) / kScaleBlock;
  const int64_t tiles = (p.M + kScaleBlock - 1) / kScaleBlock * tiles_n;
  auto enc = encode_fn();
  if (!enc) return MMA_ERR_LAUNCH;
  CUtensorMap map;
  cuuint64_t dims[3] = {cuuint64_t(p.N), cuuint64_t(p.M), 1};
  cuuint64_t strides[2] = {cuuint64_t(p.ldx) * sizeof(T), cuuint64_t(p.ldx) * sizeof(T)};
  cuuint32_t box[3] = {kScaleBlock, kScaleBlock, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  if (enc(&map, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
          3, const_cast<void*>(p.X), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return MMA_ERR_LAUNCH;
  auto kern = quantize_tile_kernel<T, E5M2, SQUARE, TRANS>;
  static PerContext<bool> attr;
  bool ok = false;
  if (!attr.get(ctx, &ok, [&](bool* v) {
        *v = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  L::SMEM) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return MMA_ERR_LAUNCH;
  const unsigned grid =
      unsigned(std::min<int64_t>(tiles, int64_t(ctx.num_sms) * L::PER_SM));
  kern<<<grid, L::THREADS, L::SMEM, ctx.stream>>>(map, p, tiles_n, tiles, ctx.status,
                                                hook);
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

template <class T, bool E5M2>
mma_status_t quantize(const Ctx& ctx, const QuantProblem& p) {
  const int64_t tiles_n = (p.N + kScaleBlock - 1) / kScaleBlock;
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
    return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
  }
  if (!p.transpose) return run_tiles<T, E5M2, true, false>(ctx, p);
  if (p.block_rows == 128) return run_tiles<T, E5M2, true, true>(ctx, p);
  return run_tiles<T, E5M2, false, true>(ctx, p);
}

template <class T>
mma_status_t by_format(const Ctx& ctx, const QuantProblem& p) {
  return p.e5m2 ? quantize<T, true>(ctx, p) : quantize<T, false>(ctx, p);
}

}  // namespace

mma_status_t launch_quantize_abort_selftest(const Ctx& ctx, int64_t limit_ns, int transpose,
                                            const void* X, void* Q, float* S) {
  const QuantProblem p = {MMA_BF16, false, transpose != 0, false, transpose ? 1 : 128,
                          1024, 1024, X, 1024, Q, 1024, S, 8, 1};
  const WaitHook hook = {static_cast<unsigned long long>(limit_ns), 1};
  return transpose ? run_tiles<__nv_bfloat16, false, false, true>(ctx, p, hook)
                   : run_tiles<__nv_bfloat16, false, true, false>(ctx, p, hook);
}

mma_status_t launch_quantize_f8(const Ctx& ctx, const QuantProblem& p) {
  switch (p.type) {
    case MMA_BF16: return by_format<__nv_bfloat16>(ctx, p);
    case MMA_F16: return by_format<__half>(ctx, p);
    default: return by_format<float>(ctx, p);
  }
}

}  // namespace mmagb
