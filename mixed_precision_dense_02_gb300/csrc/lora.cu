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
//
// One token, 8192 x 4096, rank 16: 17.5 us, the shared product alone 16; 64 requests'
// tokens 25.5, the product 23 (bound by latency: the sums, their exchange, s B); 8192 rows
// of 6 prompts, 8192 x 4096, rank 64: 337, the product 300 (the tensor pipe); the
// gradients of that batch's adapters, rank 16, FP32: 56 with its sums (3.7 TB/s).  These are
// device times in a graph; a call by itself takes 23 us at least, the host's time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace mmagb {
namespace {

constexpr int kThreads = 256;

// The requests, in shared memory.
struct Requests {
  // 0, then the offsets, within [0, T] and none below the one before it, then T
  int bound[MMA_MAX_GROUPS + 3];
  int who[MMA_MAX_GROUPS];  // their adapters, or -1
  int scan[kThreads / 32 + 1];
};

__device__ __forceinline__ void load_requests(Requests& r, const int* offsets,
                                              const int* adapters, int total, int requests,
                                              int T) {
  int *bound = r.bound, *scan = r.scan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
  for (int base = 0; base <= requests; base += blockDim.x) {
    const int i = base + threadIdx.x;
    int v = i <= requests ? min(max(__ldg(offsets + i), 0), T) : 0;
    if (i < requests) {
      const int a = adapters ? __ldg(adapters + i) : i;
      r.who[i] = a < total ? a : -1;
    }
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
    for (int w = 0; w < int(blockDim.x) / 32; ++w) before = max(before, scan[w]);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    bound[0] = 0;
    bound[requests + 2] = T;
  }
  __syncthreads();
}

// A piece: its request (counted from the one before the first) and rows; none: from == to.
struct Piece {
  int request, from, to;
};

// The adapter of a request counted from the one before the first, or -1.
__device__ __forceinline__ int adapter_of(const Requests& r, int j, int requests) {
  return j < 1 || j > requests ? -1 : max(r.who[j - 1], -1);
}

// Piece `u` of blocks of `per` rows (a power of two), of any number of requests: each thread
// has kAtOnce of them, and only the piece's own is kept.
struct OnePiece {
  int scan[kThreads / 32 + 1];
  int request, first, next, who;  // `next`: the request's end; who: its adapter, or -1
};

constexpr int kAtOnce = 4;

__device__ __forceinline__ Piece find_piece(OnePiece& o, const int* offsets,
                                            const int* adapters, int total, int requests,
                                            int T, int per, int u) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (threadIdx.x == 0) o.request = -1;
  int before = 0;
  // element j is the bound behind request j - 1, which is the last one there is for u
  // if its own first piece is not above u and that of request j is
  for (int base = 1; base <= requests + 2; base += blockDim.x * kAtOnce) {
    int v[kAtOnce], who[kAtOnce], most = 0;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int j = base + threadIdx.x * kAtOnce + i;
      v[i] = j <= requests + 1 ? min(max(__ldg(offsets + j - 1), 0), T) : T;
      who[i] = j < 2 || j > requests + 1 ? -1 : adapters ? __ldg(adapters + j - 2) : j - 2;
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) most = v[i] = max(v[i], most);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, most, d);
      if (lane >= d) most = max(most, up);
    }
    if (lane == 31) o.scan[warp] = most;
    int last = __shfl_up_sync(0xffffffffu, most, 1);
    last = max(lane > 0 ? last : 0, before);
    __syncthreads();
    for (int w = 0; w < warps; ++w) {
      if (w < warp) last = max(last, o.scan[w]);
      before = max(before, o.scan[w]);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int j = base + threadIdx.x * kAtOnce + i, end = max(last, v[i]);
      if (j <= requests + 2 && last / per + j - 1 <= u &&
          (j == requests + 2 || end / per + j > u)) {
        o.request = j - 1;
        o.first = last;
        o.next = end;
        o.who = who[i] < total ? max(who[i], -1) : -1;
      }
      last = end;
    }
    __syncthreads();
    if (o.request >= 0) break;
  }
  const int j = o.request;
  const int64_t from = max(int64_t(u - j) * per, int64_t(o.first));
  const int to = int(min(int64_t(u - j + 1) * per, int64_t(o.next)));
  return Piece{j, int(min(from, int64_t(to))), to};
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

// 16 bits of v; v becomes what they leave of it, nothing of NaN and infinities.
template <bool BF16>
__device__ __forceinline__ uint16_t take_half(float& v) {
  uint16_t bits;
  float f;
  if constexpr (BF16) {
    __nv_bfloat16 h = __float2bfloat16_rn(v);
    f = __bfloat162float(h);
    if (fabsf(f) == INFINITY && fabsf(v) < INFINITY) {  // (rounded up from a number)
      h = __ushort_as_bfloat16(v < 0.f ? 0xFF7F : 0x7F7F);
      f = __bfloat162float(h);
    }
    bits = __bfloat16_as_ushort(h);
  } else {
    const __half h = __float2half_rn(v);
    f = __half2float(h);
    bits = __half_as_ushort(h);
  }
  v = fabsf(f) < INFINITY ? v - f : 0.f;
  return bits;
}

// What the threads of a block share to wait for loads.
struct Ring {
  uint64_t full[4], empty[4];
  uint64_t cleared;  // (the gradient's last stage)
  int abort_flag;
};

__device__ __forceinline__ void ring_init(Ring& r, int stages) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&r.full[s], 1);
      mbar_init(&r.empty[s], kThreads / 32);
    }
    mbar_init(&r.cleared, kThreads / 32);
    r.abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
}

// Stages of loads for a block's eight warps.  load(step, shared memory, barrier)
// issues a stage of `bytes`; use(step, stage) is what a warp does with it.  PRODUCER: a
// ninth warp issues them.  Else thread 0 does, the first ones before the loop, later
// ones when every warp has left the stage: for blocks beside which another kernel's is
// to fit (two of nine warps and the shared product's twelve need more registers than an
// SM has).  8192 x 4096 and 8192 rows, rank 16, the gradients: 50 us with a ninth warp,
// 62 without.  Returns, to every thread, whether all waits were met; no load is on its
// way any more.
template <bool PRODUCER, int STAGES, int STAGE, class Load, class Use>
__device__ __forceinline__ bool ring_run(Ring& r, uint8_t* smem, int steps, int bytes,
                                         unsigned* status, Load&& load, Use&& use) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  int issued = 0;
  auto issue = [&] {
    const int s = issued % STAGES;
    mbar_arrive_expect_tx(&r.full[s], uint32_t(bytes));
    load(issued, smem + s * STAGE, &r.full[s]);
    ++issued;
  };
  auto parity = [](int step) { return uint32_t(step / STAGES) & 1u; };
  const bool issuer = threadIdx.x == (PRODUCER ? kThreads : 0);
  if (issuer)
    while (issued < steps && issued < STAGES) issue();
  if (PRODUCER && threadIdx.x >= kThreads) {
    if (issuer)
      while (issued < steps && ok) {
        const int before = issued - STAGES;
        ok = mbar_wait(&r.empty[before % STAGES], parity(before), &r.abort_flag, status);
        if (ok) issue();
      }
  } else {
    __syncwarp();
    for (int step = 0; step < steps; ++step) {
      const int s = step % STAGES;
      ok = mbar_wait(&r.full[s], parity(step), &r.abort_flag, status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      use(step, smem + s * STAGE);
      __syncwarp();
      mbar_arrive_if(&r.empty[s], lane == 0);
      if constexpr (!PRODUCER) {
        if (issuer && issued < steps) {
          ok = mbar_wait(&r.empty[s], parity(step), &r.abort_flag, status);
          if (ok) issue();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
    }
  }
  if (issuer)
    for (int i = max(issued - STAGES, 0); i < issued; ++i)
      mbar_drain(&r.full[i % STAGES], parity(i), status);
  __syncwarp();
  return !__syncthreads_or(!ok || r.abort_flag);
}

// ------------------------------------------------------------- a row's sums

// Piece blockIdx.x of blocks of BM rows; the CTAs of a cluster (blockIdx.y) share
// the k range, and so do the warps that have the same 16 rows.  Boxes of 64 k's by
// TMA into a ring (cp.async's addresses were half of all instructions: 8192 x 4096,
// rank 64, 33 us).  Rows of X past the piece are other requests' and their sums are
// dropped; sums past the rank and k's past K are zeros.
//
// A few rows' share of the result, s B, is made here as well: of every row up to
// kLoraEveryRow or with more requests than the product lists (lora_every), else of the
// requests of fewer than kLoraRows.  Every CTA of the
// cluster adds all of the piece's sums up, and a thread has one of 256 columns of B, which
// come through a ring of their own (2100 rows, 60 of them single tokens, 4096 x 4096, rank
// 32: 72 us with the product, 76 with plain loads of B; the kernel itself some 23).
// BM 16: two stages and 64 registers a thread.  With EVERY (up to kLoraEveryRow rows)
// two CTAs then leave an SM room for one of the shared product's, which runs beside
// them.
template <int BM, int RP, bool EVERY>
struct Shrink {
  static constexpr int MW = BM / 16, KW = 8 / MW;  // warps along rows, along k
  static constexpr int KS = BM == 16 ? 256 : 128;  // k's per stage
  static constexpr int X_BYTES = BM * KS * 2, A_BYTES = RP * KS * 2;
  static constexpr int STAGE = X_BYTES + A_BYTES;
  static constexpr int STAGES = BM == 16 ? 2 : 4 * STAGE <= 100 * 1024 ? 4 : 3;
  static constexpr bool PRODUCER = BM != 16;
  static constexpr int THREADS = kThreads + (PRODUCER ? 32 : 0);
  static constexpr int BLOCKS = BM == 16 && RP <= 32 ? 4 : 2;
  static constexpr int SMEM = STAGES * STAGE + 1024;  // (the sums: 512 * RP bytes)
  // columns of B behind the piece's own and its cluster's sums
  static constexpr int B_BYTES = kThreads * RP * 2, B_AT = 2 * BM * RP * 4;
  static constexpr int B_ROOM = (STAGES * STAGE - B_AT) / B_BYTES;
  static constexpr int B_STAGES = B_ROOM < 4 ? B_ROOM : 4;
  static_assert(B_STAGES >= 1 && B_AT % 1024 == 0);
};

constexpr int kMostParts = 8;       // CTAs that share a piece's k range
constexpr int kSmallBlocks = 4096;  // rows up to which blocks have 16

// The swizzle of rows of `bytes` (the same that swizzled() computes).
constexpr CUtensorMapSwizzle swizzle_of(int bytes) {
  return bytes == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
         : bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                       : CU_TENSOR_MAP_SWIZZLE_128B;
}

// `many` rows of extra, up to R: their sums `s` (RP apart, zeros past the rank; the
// room behind the last is read too) times a column of B, this thread's in `stage`.
template <bool BF16, int R, int RP>
__device__ __forceinline__ void expand(const uint8_t* stage, const float* s, int many,
                                       float* out, int N) {
  constexpr int RB = RP < 64 ? RP : 64;
  float2 v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < RP; k += 8) {
    const uint4 w = *reinterpret_cast<const uint4*>(
        stage + k / RB * kThreads * RB * 2 + swizzled<RB * 2>(threadIdx.x, k % RB / 8));
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float2 b;
      if constexpr (BF16)
        b = make_float2(__uint_as_float(q[y] << 16), __uint_as_float(q[y] & 0xFFFF0000u));
      else
        b = __half22float2(*reinterpret_cast<const __half2*>(&q[y]));
#pragma unroll
      for (int r = 0; r < R; ++r)
        v[r] = __ffma2_rn(*reinterpret_cast<const float2*>(s + r * RP + k + 2 * y), b, v[r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (r < many) out[int64_t(r) * N] = v[r].x + v[r].y;
}

// The same of a row-major B, kCols columns per thread from p0 on, kThreads apart, whose
// loads go together.
constexpr int kCols = 4;

template <bool BF16, int R, int RP>
__device__ __forceinline__ void expand_rows(const LoraProblem& g, const uint16_t* B,
                                            const float* s, int many, int p0, float* out) {
  const int rank = int(g.rank), N = int(g.N);
  float2 v[R][kCols];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int x = 0; x < kCols; ++x) v[r][x] = make_float2(0.f, 0.f);
  const int p1 = p0 + threadIdx.x;
#pragma unroll 2
  for (int k = 0; k < rank; k += 8) {
    const int left = rank - k;
#pragma unroll
    for (int x = 0; x < kCols; ++x) {
      const int p = min(p1 + x * kThreads, N - 1);
      uint32_t f[8];
#pragma unroll
      for (int y = 0; y < 8; ++y) f[y] = y < left ? B[(k + y) * g.ldb + p] : 0u;
#pragma unroll
      for (int y = 0; y < 8; y += 2) {
        const uint32_t q = f[y] | f[y + 1] << 16;
        float2 b;
        if constexpr (BF16)
          b = make_float2(__uint_as_float(q << 16), __uint_as_float(q & 0xFFFF0000u));
        else
          b = __half22float2(*reinterpret_cast<const __half2*>(&q));
#pragma unroll
        for (int r = 0; r < R; ++r)
          v[r][x] = __ffma2_rn(*reinterpret_cast<const float2*>(s + r * RP + k + y), b, v[r][x]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int x = 0; x < kCols; ++x)
      if (r < many && p1 + x * kThreads < N)
        out[int64_t(r) * N + p1 + x * kThreads] = v[r][x].x + v[r][x].y;
}

template <bool BF16, bool ROW, int BM, int RP, bool EVERY>
__global__ void __launch_bounds__(Shrink<BM, RP, EVERY>::THREADS, Shrink<BM, RP, EVERY>::BLOCKS)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap tmX,
                       const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB, const LoraProblem g,
                       const LoraLow low, unsigned* status) {
  using L = Shrink<BM, RP, EVERY>;
  constexpr int KS = L::KS, KB = KS / 64;
  constexpr int RB = RP < 64 ? RP : 64;  // (ROW) sums per box of A, else of B
  constexpr int kRows = L::BLOCKS == 4 ? 1 : 2;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ OnePiece one;
  __shared__ Ring ring, columns;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ring_init(ring, L::STAGES);
  ring_init(columns, L::B_STAGES);
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  // The kernel after this one reads what is older than this one without waiting: it
  // may start when that is there.
  grid_dependency_wait();
  grid_dependents_start();
  const int requests = int(g.requests);
  const Piece piece = find_piece(one, g.offsets, g.adapters, int(g.adapters_total), requests,
                                 int(g.rows), BM, blockIdx.x);
  const int who = one.who;
  const int rows = piece.to - piece.from, rank = int(g.rank), N = int(g.N);
  // (the same in all CTAs of the cluster, so that all of them return)
  if (rows <= 0) return;
  const int part = blockIdx.y, parts = gridDim.y;
  const int first_of = one.first;
  // (without k there is nothing to add, and B need not exist)
  const bool every = EVERY || lora_every(g.rows, requests);
  const bool add = g.K > 0 && (every || one.next - first_of < kLoraRows);
  auto extra_row = [&](int row) {
    const int64_t t = piece.from + row;
    return low.extra +
           (lora_own_places(g.rows, requests)
                ? t
                : int64_t(piece.request - 1) * (kLoraRows - 1) + t - first_of) * N;
  };
  auto put = [&](int row, int n, float v) {
    if (n < low.ld32) low.f32[(int64_t(piece.from) + row) * low.ld32 + n] = v;
  };
  if (who < 0) {
    for (int i = part * L::THREADS + threadIdx.x; i < rows * RP; i += parts * L::THREADS)
      put(i / RP, i % RP, 0.f);
    if (every)
      for (int r = 0; r < rows; ++r)
        for (int p = part * L::THREADS + threadIdx.x; p < N; p += parts * L::THREADS)
          extra_row(r)[p] = 0.f;
    return;
  }
  const float scale = g.scales ? __ldg(g.scales + who) : 1.f;
  const uint16_t* const B = static_cast<const uint16_t*>(g.B) + who * g.stride_b;
  if (add && g.ldb <= (ROW ? int64_t(1) << 40 : 2 * rank + 8)) {
    // this CTA's part of B on its way to L2 while the sums are made
    for (int p0 = part * kThreads * kCols; p0 < N; p0 += parts * kThreads * kCols) {
      const int cols = min(kThreads * kCols, N - p0);
      const int lines = ROW ? (cols + 63) / 64 : int((cols * g.ldb + 63) / 64);
      for (int i = threadIdx.x; i < (ROW ? lines * rank : lines); i += L::THREADS)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            ROW ? B + i / lines * g.ldb + p0 + min(i % lines * 64, cols - 1)
                : B + p0 * g.ldb + min(int64_t(i) * 64, (cols - 1) * g.ldb)));
    }
  }
  const int K = int(g.K);
  const int all = (K + KS - 1) / KS;
  const int first = int(int64_t(all) * part / parts);
  const int steps = int(int64_t(all) * (part + 1) / parts) - first;
  float acc[RP / 8][4];
#pragma unroll
  for (int n = 0; n < RP / 8; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
  const int mw = warp % L::MW, kw = warp / L::MW;
  const bool ok = ring_run<L::PRODUCER, L::STAGES, L::STAGE>(
      ring, smem, steps, L::STAGE, status,
      [&](int step, uint8_t* xs, uint64_t* bar) {
        const int k = (first + step) * KS;
        uint8_t* as = xs + L::X_BYTES;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          tma_load_3d(&tmX, bar, xs + b * BM * 128, k + b * 64, piece.from, 0);
          if constexpr (!ROW) tma_load_3d(&tmA, bar, as + b * RP * 128, k + b * 64, 0, who);
        }
        if constexpr (ROW)
          for (int b = 0; b < RP / RB; ++b)
            tma_load_3d(&tmA, bar, as + b * KS * RB * 2, b * RB, k, who);
      },
      [&](int, const uint8_t* stage) {
        const uint32_t xs = smem_u32(stage), as = xs + L::X_BYTES;
        const int m = lane >> 3, at = lane & 7;
        // (the tensor cores' FP32 sums drop low bits: they run over a warp's k's of a stage,
        // 32 or 64, and are added to others to nearest)
        constexpr int kAt = RP == 128 ? 2 : RP / 16;
#pragma unroll
        for (int n0 = 0; n0 < RP / 16; n0 += kAt) {
          float sum[2 * kAt][4] = {};
#pragma unroll
          for (int kk = 0; kk < KS / L::KW / 16; ++kk) {
            const int k = kw * (KS / L::KW) + kk * 16, box = k / 64, in = k % 64;
            uint32_t a[4];
            ldmatrix_x4(a, xs + box * BM * 128 +
                               swizzled<128>(mw * 16 + (lane & 15), in / 8 + (lane >> 4)));
#pragma unroll
            for (int x = 0; x < kAt; ++x) {
              const int n = n0 + x;
              uint32_t b[4];
              if constexpr (!ROW)
                ldmatrix_x4(b, as + box * RP * 128 +
                                   swizzled<128>(n * 16 + (m >> 1) * 8 + at, in / 8 + (m & 1)));
              else
                ldmatrix_x4_trans(b, as + n * 16 / RB * KS * RB * 2 +
                                         swizzled<RB * 2>(k + (m & 1) * 8 + at,
                                                          n * 2 % (RB / 8) + (m >> 1)));
              mma16<BF16>(sum[2 * x], a, b[0], b[1]);
              mma16<BF16>(sum[2 * x + 1], a, b[2], b[3]);
            }
          }
#pragma unroll
          for (int x = 0; x < 2 * kAt; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[2 * n0 + x][j] += sum[x][j];
        }
      });
  // the warps' sums, then the CTAs', each in order
  float* sums = reinterpret_cast<float*>(smem);  // [KW][BM][RP]
#pragma unroll
  for (int n = 0; n < RP / 8; ++n) {
    if (L::PRODUCER && warp == kThreads / 32) break;
    float* d = sums + (kw * BM + mw * 16 + (lane >> 2)) * RP + n * 8 + 2 * (lane & 3);
    d[0] = acc[n][0];
    d[1] = acc[n][1];
    d[8 * RP] = acc[n][2];
    d[8 * RP + 1] = acc[n][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < rows * RP; i += L::THREADS) {
    float v = sums[i];
#pragma unroll
    for (int w = 1; w < L::KW; ++w) v += sums[w * BM * RP + i];
    sums[i] = v;  // (read by this thread alone)
  }
  fence_proxy_async_smem();  // (the columns of B land where other sums were)
  if (parts > 1) cluster_sync();
  else __syncthreads();
  float* mine = sums + BM * RP;  // all CTAs' (the room of a warp's sums, done with)
  const int share_rows = (rows + parts - 1) / parts, share = share_rows * RP;
  for (int i = add ? threadIdx.x : part * share + threadIdx.x;
       i < (add ? rows * RP : min((part + 1) * share, rows * RP)); i += L::THREADS) {
    float v = 0.f;
    if (parts > 1) {
      float w[kMostParts];  // (their loads together)
#pragma unroll
      for (int r = 0; r < kMostParts; ++r)
        w[r] = r < parts ? ld_shared_cluster_f32(mapa_shared(smem_u32(sums + i), r)) : 0.f;
#pragma unroll
      for (int r = 0; r < kMostParts; ++r) v += w[r];
    } else {
      v = sums[i];
    }
    v = i % RP < rank ? v * scale : 0.f;
    mine[i] = v;
    if (ok && i / share == part) put(i / RP, i % RP, v);
  }
  if (parts > 1) cluster_sync();  // no CTA leaves while another reads its sums
  else __syncthreads();
  if (!ok) return;
  // The rows' sums in 16 bits, a warp for each; FP16 ones scaled by a power of two of
  // the row's own, whose exponent stands behind the first of them.
  if (!EVERY && low.parts > 0) {
    for (int row = part * share_rows + warp; row < min((part + 1) * share_rows, rows);
         row += L::THREADS / 32) {
      float v[(RP + 31) / 32], m = 0.f;
#pragma unroll
      for (int x = 0; x < (RP + 31) / 32; ++x) {
        v[x] = x * 32 + lane < rank ? mine[row * RP + x * 32 + lane] : 0.f;
        const float size = fabsf(v[x]);
        m = fmaxf(m, size < INFINITY ? size : 0.f);
      }
      uint16_t* d = static_cast<uint16_t*>(low.f16) + (int64_t(piece.from) + row) * low.ld16;
      float up = 1.f;
      if constexpr (!BF16) {
        const int exponent =
            up_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m))));
        up = up_of(exponent);
        if (lane == 0) d[rank] = uint16_t(exponent);
      }
#pragma unroll
      for (int x = 0; x < (RP + 31) / 32; ++x) {
        if (x * 32 + lane >= rank) break;
        float left = v[x] * up;
        for (int i = 0; i < low.parts; ++i)
          d[i * g.rows * low.ld16 + x * 32 + lane] = take_half<BF16>(left);
      }
    }
  }
  if (!add || N == 0) return;
  if constexpr (ROW) {
    if (L::PRODUCER && warp == kThreads / 32) return;
    for (int p0 = part * kThreads * kCols; p0 < N; p0 += parts * kThreads * kCols)
      for (int r0 = 0; r0 < rows; r0 += kRows)
        expand_rows<BF16, kRows, RP>(g, B, mine + r0 * RP, min(rows - r0, kRows), p0,
                                     extra_row(r0));
  } else {
    const int blocks = ((N + kThreads - 1) / kThreads - part + parts - 1) / parts;
    ring_run<L::PRODUCER, L::B_STAGES, L::B_BYTES>(
        columns, smem + L::B_AT, blocks, L::B_BYTES, status,
        [&](int step, uint8_t* bs, uint64_t* bar) {
          const int p = (part + step * parts) * kThreads;
#pragma unroll
          for (int b = 0; b < RP / RB; ++b)
            tma_load_3d(&tmB, bar, bs + b * kThreads * RB * 2, b * RB, p, who);
        },
        [&](int step, const uint8_t* stage) {
          const int p = (part + step * parts) * kThreads + threadIdx.x;
          if (p >= N) return;
          if (rows == 1) return expand<BF16, 1, RP>(stage, mine, 1, extra_row(0) + p, N);
          for (int r = 0; r < rows; r += 4)
            expand<BF16, 4, RP>(stage, mine + r * RP, rows - r, extra_row(r) + p, N);
        });
  }
}

template <bool BF16, bool ROW, int BM, int RP, bool EVERY>
mma_status_t shrink(const Ctx& ctx, const LoraProblem& g, const LoraLow& low) {
  using L = Shrink<BM, RP, EVERY>;
  constexpr int RB = RP < 64 ? RP : 64;
  auto kernel = lora_shrink_kernel<BF16, ROW, BM, RP, EVERY>;
  static PerContext<bool> attr;
  bool ok = false;
  if (!attr.get(ctx, &ok, [&](bool* v) {
        // (all of an SM's memory as shared memory: the shared product's CTAs cannot
        // start beside these on an SM that is divided otherwise)
        *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  L::SMEM) == cudaSuccess &&
             cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                  cudaSharedmemCarveoutMaxShared) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return MMA_ERR_LAUNCH;
  // (without adapters or k there is nothing to load, but the maps have to be valid:
  // over the sums, which are 16-byte aligned and eight numbers at least)
  const bool any = g.K > 0 && g.adapters_total > 0;
  const int64_t slices = any ? g.adapters_total : 1;
  const int64_t slice = slices > 1 ? g.stride_a : any ? g.lda : 8;
  const void* const a = any ? g.A : low.f32;
  CUtensorMap tx, ta, tb;
  if (!make_map(&tx, any ? g.X : low.f32, 2, any ? g.K : 8, any ? g.rows : 1,
                any ? g.ldx : 8, 1, any ? g.ldx : 8, 64, BM) ||
      !(ROW ? make_map(&ta, a, 2, any ? g.rank : 8, any ? g.K : 1, any ? g.lda : 8,
                       slices, slice, RB, L::KS, swizzle_of(RB * 2))
            : make_map(&ta, a, 2, any ? g.K : 8, any ? g.rank : 1, any ? g.lda : 8,
                       slices, slice, 64, RP)))
    return MMA_ERR_LAUNCH;
  tb = ta;
  if (!ROW && any && g.N > 0 &&
      !make_map(&tb, g.B, 2, g.rank, g.N, g.ldb, g.adapters_total,
                g.adapters_total > 1 ? g.stride_b : g.ldb, RB, kThreads, swizzle_of(RB * 2)))
    return MMA_ERR_LAUNCH;
  const int64_t pieces = (g.rows + BM - 1) / BM + g.requests + 1;
  const int64_t steps = (g.K + L::KS - 1) / L::KS;
  // As many CTAs per piece as there is room for at once (with few rows twice per SM,
  // beside the shared product; of rank 32 three, though four fit: 200 single tokens, 4096 x
  // 4096, 43 us, 46), each with two stages at least.
  const int per_sm = EVERY ? 2 : std::min(BM == 16 ? 4 : 2, 224 * 1024 / (L::SMEM + 10 * 1024));
  int parts = 1;
  while (parts < kMostParts && pieces * parts * 2 <= int64_t(per_sm) * ctx.num_sms && steps >= parts * 4)
    parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(pieces), unsigned(parts), 1);
  cfg.blockDim = dim3(L::THREADS, 1, 1);
  cfg.dynamicSmemBytes = L::SMEM;
  cfg.stream = ctx.stream;
  cudaLaunchAttribute at[2] = {};
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = unsigned(parts);
  at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tx, ta, tb, g, low, ctx.status);
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

// ------------------------------------------------- the adapters' own gradients

// One side of the gradient: features of M (T x F) times the rows' sums.
struct Side {
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
  int d_type, parts, ld16;
  bool accumulate;
  const int* from;   // gathered rows: the row at each place; else null
  float* part;       // [pieces - 2][rank][features of both sides]
  uint16_t* halves;  // [2][parts][T][ld16]
  float* down;       // (FP16) [2][chunks][RP]: what a chunk's sums are scaled back by
  int chunks;
  unsigned* status;
};

struct WgradMaps {
  CUtensorMap m[2], low[2];
};

constexpr int kTile = 128;      // features per CTA, 16 per warp
constexpr int kStageRows = 64;  // rows per stage

template <int RP>
struct Wgrad {
  static constexpr int RB = RP < 64 ? RP : 64;  // sums per box
  static constexpr int M_BYTES = kStageRows * kTile * 2;
  static constexpr int PART = kStageRows * RP * 2;  // one part of the sums
  // (a KB behind them for the sums' scales)
  static constexpr int stage(int parts) { return M_BYTES + parts * PART + 1024; }
  // two CTAs per SM if that leaves them two stages each
  static constexpr int per_sm(int parts) { return 2 * stage(parts) <= 102 * 1024 ? 2 : 1; }
  static constexpr int stages(int parts) {
    const int n = (per_sm(parts) == 2 ? 102 : 210) * 1024 / stage(parts);
    return n < 4 ? n : 4;
  }
  static constexpr int smem(int parts) { return stages(parts) * stage(parts) + 1024; }
  static_assert(stages(3) >= 2 && smem(3) <= 216 * 1024, "the ring");
};

// Gathered rows: many small requests of few adapters would make a piece each, with a
// share of the gradient as large as an adapter (1000 single tokens, 8192 + 8192
// features, rank 128: 8 GB).  Instead the rows are copied in the order of their
// adapters, which then are the requests.
struct Gather {
  int T, requests, total;
  const int *offsets, *adapters;
  int* bound;   // [requests + 1]: the offsets, clamped and in order
  int* first;   // [requests]: the place of a request's first row, or -1
  int* starts;  // [total + 1]: the adapters' rows
  int* from;    // [T]: the row at each place
  const uint16_t* in[2];  // dy, x
  int64_t ld[2], ld_out[2];
  int F[2];
  uint16_t* out[2];
};

// One block.  The adapters' rows are counted by 32 warps, each with consecutive
// requests; a request's place is behind those of its adapter's in earlier warps and in
// its own before it.
__global__ void __launch_bounds__(1024) lora_order_kernel(const Gather g) {
  extern __shared__ int count[];  // [32][total]
  __shared__ int scan[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int before = 0;
  for (int base = 0; base <= g.requests; base += 1024) {
    const int i = base + threadIdx.x;
    int v = i <= g.requests ? min(max(__ldg(g.offsets + i), 0), g.T) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v = max(v, o);
    }
    if (lane == 31) scan[warp] = v;
    __syncthreads();
    v = max(v, before);
    for (int w = 0; w < 32; ++w) {
      if (w < warp) v = max(v, scan[w]);
      before = max(before, scan[w]);
    }
    if (i <= g.requests) g.bound[i] = v;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 32 * g.total; i += 1024) count[i] = 0;
  __syncthreads();
  const int per = (g.requests + 1023) / 1024 * 32;  // requests of a warp
  const int from = min(warp * per, g.requests), to = min(from + per, g.requests);
  int* const mine = count + warp * g.total;
  auto request = [&](int i, int* rows) {
    int who = -1;
    *rows = 0;
    if (i < to) {
      who = g.adapters ? __ldg(g.adapters + i) : i;
      who = who < g.total ? max(who, -1) : -1;
      *rows = g.bound[i + 1] - g.bound[i];
    }
    return who;
  };
  for (int i = from + lane; i < to; i += 32) {
    int rows;
    const int who = request(i, &rows);
    if (who >= 0) atomicAdd(mine + who, rows);
  }
  __syncthreads();
  int sum = 0;  // of adapter threadIdx.x, in place of each warp's those before it
  if (int(threadIdx.x) < g.total)
    for (int w = 0; w < 32; ++w) {
      const int n = count[w * g.total + threadIdx.x];
      count[w * g.total + threadIdx.x] = sum;
      sum += n;
    }
  int s = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) scan[warp] = s;
  __syncthreads();
  for (int w = 0; w < warp; ++w) s += scan[w];
  if (int(threadIdx.x) < g.total) {
    g.starts[threadIdx.x] = s - sum;
    if (int(threadIdx.x) == g.total - 1) g.starts[g.total] = s;
    for (int w = 0; w < 32; ++w) count[w * g.total + threadIdx.x] += s - sum;
  }
  __syncthreads();
  for (int base = from; base < to; base += 32) {
    const int i = base + lane;
    int rows, earlier = 0;
    const int who = request(i, &rows);
    bool last = true;
    for (int d = 0; d < 32; ++d) {
      const int n = __shfl_sync(0xffffffffu, rows, d);
      const int w = __shfl_sync(0xffffffffu, who, d);
      if (w == who && d < lane) earlier += n;
      if (w == who && d > lane) last = false;
    }
    const int at = who >= 0 ? mine[who] + earlier : -1;
    __syncwarp();
    if (who >= 0 && last) mine[who] = at + rows;
    __syncwarp();
    if (i < to) g.first[i] = at;
  }
}

// Each row to its place.
__global__ void __launch_bounds__(256) lora_gather_kernel(const Gather g) {
  for (int t = blockIdx.x; t < g.T; t += gridDim.x) {
    int lo = 0, hi = g.requests;  // the last request that starts by row t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (g.bound[mid] <= t) lo = mid; else hi = mid;
    }
    int place = -1;
    if (t >= g.bound[lo] && t < g.bound[lo + 1] && g.first[lo] >= 0)
      place = g.first[lo] + t - g.bound[lo];
    if (place < 0) continue;
    if (threadIdx.x == 0) g.from[place] = t;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4* in = reinterpret_cast<const uint4*>(g.in[i] + t * g.ld[i]);
      uint4* out = reinterpret_cast<uint4*>(g.out[i] + place * g.ld_out[i]);
#pragma unroll 4
      for (int v = threadIdx.x; v < (g.F[i] + 7) / 8; v += 256) out[v] = __ldg(in + v);
    }
  }
}

// Both sides' sums in parts of 16 bits: BF16, whose range is FP32's.
template <int RP>
__device__ __forceinline__ void split_rows(const WgradArgs& a, const Side& side, uint16_t* out) {
  const int64_t all = int64_t(a.T) * a.ld16;
  constexpr int kWidth = RP < 32 ? RP : 32;  // lanes for a row
  constexpr int kRows = kThreads / kWidth;
  // (the places of gathered rows end with the last adapter's)
  const int last = a.from ? __ldg(a.offsets + a.requests) : a.T;
  for (int64_t place = int64_t(blockIdx.x) * kRows + threadIdx.x / kWidth; place < last;
       place += int64_t(gridDim.x) * kRows) {
    const int64_t row = a.from ? a.from[place] : place;
    for (int n = threadIdx.x % kWidth; n < a.ld16; n += kWidth) {
      float v = n < a.rank ? side.low[row * side.ldl + n] : 0.f;
      for (int part = 0; part < a.parts; ++part)
        out[part * all + place * a.ld16 + n] = take_half<true>(v);
    }
  }
}

// FP16, with the sums' scales.  A block has a chunk, which is a stage of the kernel below:
// 64 rows of a piece, counted from its first, and numbered by that row's block of 64 and
// the piece's request (their sum, as the pieces).  Each column of it has a power of two
// of its own, so that what stands beside small sums, other requests' or other columns',
// does not take their bits: two numbers leave 2^-22 of a sum, and 2^-38 of the largest
// of its column in the chunk.
template <int RP>
__device__ __forceinline__ void split_chunk(const WgradArgs& a, const Side& side, uint16_t* out) {
  constexpr int kGroups = kThreads / RP, kEach = kStageRows / kGroups;
  __shared__ OnePiece one;
  __shared__ float most[kThreads];
  const int request = find_piece(one, a.offsets, a.adapters, a.total, a.requests, a.T,
                                 kStageRows, blockIdx.x).request;
  // (a piece that starts with its request, or with a block of `per` rows)
  const int64_t block = int64_t(blockIdx.x - request) * kStageRows;
  const int64_t piece = block / a.per * a.per;
  const int64_t from = block + (one.first > piece ? one.first % kStageRows : 0);
  const int to = int(min(min(from + kStageRows, piece + a.per), int64_t(one.next)));
  if (one.who < 0 || from >= to) return;
  const int n = threadIdx.x % RP, first = int(from) + threadIdx.x / RP;
  float v[kEach], m = 0.f;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int place = first + i * kGroups;
    v[i] = 0.f;
    if (place < to && n < a.rank)
      v[i] = side.low[int64_t(a.from ? a.from[place] : place) * side.ldl + n];
    const float size = fabsf(v[i]);
    m = fmaxf(m, size < INFINITY ? size : 0.f);
  }
  most[threadIdx.x] = m;
  __syncthreads();
#pragma unroll
  for (int g = 0; g < kGroups; ++g) m = fmaxf(m, most[g * RP + n]);
  const int exponent = up_exponent(m);
  const float up = up_of(exponent);
  if (threadIdx.x < RP)
    a.down[(int64_t(blockIdx.y) * a.chunks + blockIdx.x) * RP + n] = down_of(exponent);
  if (n >= a.ld16) return;
  const int64_t all = int64_t(a.T) * a.ld16;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int place = first + i * kGroups;
    if (place >= to) break;
    float left = v[i] * up;
    for (int part = 0; part < a.parts; ++part)
      out[part * all + int64_t(place) * a.ld16 + n] = take_half<false>(left);
  }
}

template <bool BF16, int RP>
__global__ void __launch_bounds__(kThreads)
    lora_halves_kernel(const WgradArgs a) {
  grid_dependents_start();
  const Side& side = a.side[blockIdx.y];
  if (side.F == 0) return;
  uint16_t* const out = a.halves + int64_t(blockIdx.y) * a.parts * a.T * a.ld16;
  if constexpr (BF16)
    split_rows<RP>(a, side, out);
  else
    split_chunk<RP>(a, side, out);
}

// A piece's share of 128 features: G[f][n] = sum over its rows M[t][f] * low[t][n] on
// the tensor cores, FP32.  As many CTAs as run at once take the shares in turn, the
// features of a piece side by side, through one ring of rows and sums that runs on from
// share to share (a CTA for each share: 51 us of 8192 x (8192 + 4096), rank 16, so 44).
// The tensor cores' FP32 sums drop low bits on the way, so that they run over a stage's
// rows, 64 of a request at most, and are added to others to nearest, scaled back (8192
// rows: 3.9e-6 off without, so 4e-7).
// What stands in a share's last stage behind the piece is another request's and becomes
// zeros in both (in one alone, an infinity in the other would leave NaN).
template <bool BF16, int RP, int PARTS>
__global__ void __launch_bounds__(kThreads + 32)
    lora_wgrad_kernel(const __grid_constant__ WgradMaps maps, const WgradArgs a, int pieces,
                      int tiles) {
  using L = Wgrad<RP>;
  constexpr int RB = L::RB;
  constexpr int stages = L::stages(PARTS), stage_bytes = L::stage(PARTS);
  extern __shared__ uint8_t raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ Requests req;
  __shared__ Ring ring;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependents_start();
  ring_init(ring, stages);
  load_requests(req, a.offsets, a.adapters, a.total, a.requests, a.T);
  grid_dependency_wait();  // (the halves)
  struct Share {
    int from, to, request, second, f0;
  };
  // share i, the shares of a piece in a row; without rows or an adapter: from == to
  auto share_of = [&](int i) {
    const int u = i / tiles, tile = i - u * tiles;
    int j = 0;
    for (int hi = a.requests + 2; hi - j > 1;) {
      const int mid = (j + hi) >> 1;
      if (req.bound[mid] / a.per + mid <= u) j = mid; else hi = mid;
    }
    const int64_t from = max(int64_t(u - j) * a.per, int64_t(req.bound[j]));
    const int to = int(min(int64_t(u - j + 1) * a.per, int64_t(req.bound[j + 1])));
    const bool none = adapter_of(req, j, a.requests) < 0 || from >= to;
    const int second = tile >= a.tiles0;
    return Share{none ? to : int(from), to, j, second,
                 (tile - (second ? a.tiles0 : 0)) * kTile};
  };
  const int shares = pieces * tiles;
  bool ok = true;
  int s = 0;
  uint32_t phase = 0;
  auto next = [&] {
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  };
  if (warp == kThreads / 32) {
    if (lane == 0) {
      int issued = 0;
      for (int i = blockIdx.x; i < shares && ok; i += gridDim.x) {
        const Share w = share_of(i);
        for (int t = w.from; t < w.to; t += kStageRows) {
          ok = mbar_wait(&ring.empty[s], phase ^ 1u, &ring.abort_flag, a.status);
          if (!ok) break;
          uint8_t* ms = smem + s * stage_bytes;
          uint64_t* bar = &ring.full[s];
          mbar_arrive_expect_tx(
              bar, uint32_t(L::M_BYTES + PARTS * L::PART + (BF16 ? 0 : RP * 4)));
#pragma unroll
          for (int b = 0; b < kTile / 64; ++b)
            tma_load_3d(&maps.m[w.second], bar, ms + b * kStageRows * 128, w.f0 + b * 64, t, 0);
          for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int b = 0; b < RP / RB; ++b)
              tma_load_3d(&maps.low[w.second], bar,
                          ms + L::M_BYTES + part * L::PART + b * kStageRows * RB * 2, b * RB,
                          t, part);
          if constexpr (!BF16)
            bulk_load(ms + L::M_BYTES + PARTS * L::PART,
                      a.down + (int64_t(w.second) * a.chunks + t / kStageRows + w.request) * RP,
                      RP * 4, bar);
          ++issued;
          next();
        }
      }
      // (the stages from s on are those of the round before)
      for (int c = 0; c < stages; ++c)
        if (c < s || issued >= stages)
          mbar_drain(&ring.full[c], c < s ? phase : phase ^ 1u, a.status);
    }
    return;
  }
  const int64_t features = int64_t(a.side[0].F) + a.side[1].F;
  // This lane's addresses of the first rows' blocks (16 rows on the swizzle is the
  // same).
  const int m = lane >> 3, at = lane & 7;
  const uint32_t f_at = warp / 4 * kStageRows * 128 +
                        swizzled<128>((m >> 1) * 8 + at, warp % 4 * 2 + (m & 1));
  uint32_t low_at[RB / 16];
#pragma unroll
  for (int n = 0; n < RB / 16; ++n)
    low_at[n] = swizzled<RB * 2>((m & 1) * 8 + at, n * 2 + (m >> 1));
  uint32_t cleared = 0;
  for (int i = blockIdx.x; i < shares && ok; i += gridDim.x) {
    const Share w = share_of(i);
    if (w.from >= w.to) continue;
    float acc[RP / 8][4];
#pragma unroll
    for (int n = 0; n < RP / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
    for (int t = w.from; t < w.to; t += kStageRows, next()) {
      uint8_t* stage = smem + s * stage_bytes;
      ok = mbar_wait(&ring.full[s], phase, &ring.abort_flag, a.status);
      const int valid = w.to - t;
      if (valid < kStageRows) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        for (int b = 0; b < kTile / 64; ++b)
          for (int x = valid * 8 + threadIdx.x; x < kStageRows * 8; x += kThreads)
            *reinterpret_cast<uint4*>(stage + b * kStageRows * 128 + x * 16) = zero;
        for (int b = 0; b < PARTS * RP / RB; ++b)
          for (int x = valid * (RB / 8) + threadIdx.x; x < kStageRows * (RB / 8); x += kThreads)
            *reinterpret_cast<uint4*>(stage + L::M_BYTES + b * kStageRows * RB * 2 + x * 16) =
                zero;
        // (the loads that follow into this stage come after these writes)
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_if(&ring.cleared, lane == 0);
        ok = mbar_wait(&ring.cleared, cleared, &ring.abort_flag, a.status) && ok;
        cleared ^= 1u;
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t ms = smem_u32(stage) + f_at;
      const uint32_t ls = smem_u32(stage) + L::M_BYTES;
      [[maybe_unused]] const float* const down =
          reinterpret_cast<const float*>(stage + L::M_BYTES + PARTS * L::PART);
      // (64 of the rank's sums at a time: eight products that do not wait for one another,
      // in registers that leave room for two blocks per SM)
      constexpr int kAt = RP < 64 ? RP / 16 : 4;
#pragma unroll
      for (int n0 = 0; n0 < RP / 16; n0 += kAt) {
        float sum[2 * kAt][4] = {};
#pragma unroll
        for (int k = 0; k < kStageRows; k += 16) {
          uint32_t f[4];
          ldmatrix_x4_trans(f, ms + k * 128);
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int x = 0; x < kAt; ++x) {
              const int n = n0 + x;
              uint32_t b[4];
              ldmatrix_x4_trans(b, ls + part * L::PART + n * 16 / RB * kStageRows * RB * 2 +
                                       k * RB * 2 + low_at[n * 16 % RB / 16]);
              mma16<BF16>(sum[2 * x], f, b[0], b[1]);
              mma16<BF16>(sum[2 * x + 1], f, b[2], b[3]);
            }
        }
#pragma unroll
        for (int x = 0; x < 2 * kAt; ++x) {
          float* const d = acc[2 * n0 + x];
          float2 scale = make_float2(1.f, 1.f);
          if constexpr (!BF16)
            scale = *reinterpret_cast<const float2*>(down + n0 * 16 + x * 8 + 2 * (lane & 3));
#pragma unroll
          for (int j = 0; j < 4; ++j)
            d[j] = BF16 ? d[j] + sum[x][j] : fmaf(sum[x][j], j & 1 ? scale.y : scale.x, d[j]);
        }
      }
      __syncwarp();
      mbar_arrive_if(&ring.empty[s], lane == 0);
    }
    if (!ok) break;
    // (eight lanes: 32 consecutive bytes of four of the sums' rows)
    float* out = a.part + int64_t(i / tiles - 1) * a.rank * features +
                 (w.second ? a.side[0].F : 0) + w.f0;
    const int F = a.side[w.second].F - w.f0;
#pragma unroll
    for (int n = 0; n < RP / 8; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = n * 8 + 2 * (lane & 3) + (j & 1);
        const int f = warp * 16 + (lane >> 2) + (j >> 1) * 8;
        if (row < a.rank && f < F) out[row * features + f] = acc[n][j];
      }
  }
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

// Adapter blockIdx.y: its pieces' shares of 256 features added in order, a lane per
// feature and kSums of the rank's sums at a time, whose loads go together (64 features
// to a block, four sums to a thread: 8192 features of rank 64 62 us, so 20).
constexpr int kSums = 8;
// (at most 2^31 rows in blocks of 2^20 and 1024 requests; rows_per_piece)
constexpr int kMostPieces = 2048 + MMA_MAX_GROUPS + 2;

__global__ void __launch_bounds__(kThreads)
    lora_wgrad_sum_kernel(const WgradArgs a) {
  __shared__ Requests req;
  __shared__ int list[kMostPieces], found;  // its pieces
  // (older than the kernel before)
  load_requests(req, a.offsets, a.adapters, a.total, a.requests, a.T);
  const int* bound = req.bound;
  if (threadIdx.x < 32) {
    int n = 0;
    for (int base = 0; base < a.requests; base += 32) {
      const int i = base + threadIdx.x;
      const bool mine = i < a.requests && req.who[i] == int(blockIdx.y) &&
                        bound[i + 2] > bound[i + 1];
      for (unsigned left = __ballot_sync(0xffffffffu, mine); left; left &= left - 1) {
        const int j = base + __ffs(left);  // counted from the one before the first
        const int first = bound[j] / a.per, last = (bound[j + 1] - 1) / a.per;
        for (int b = first + threadIdx.x; b <= last; b += 32) list[n + b - first] = b + j;
        n += last - first + 1;
      }
    }
    if (threadIdx.x == 0) found = n;
  }
  __syncthreads();
  // (also where there is nothing to add: what follows this kernel may count on the ends
  // of those before it)
  grid_dependency_wait();
  if (a.accumulate && found == 0) return;
  const int tiles0 = (a.side[0].F + kThreads - 1) / kThreads;
  const bool second = int(blockIdx.x) >= tiles0;
  const Side& side = a.side[second];
  const int64_t features = int64_t(a.side[0].F) + a.side[1].F;
  const int f = (int(blockIdx.x) - (second ? tiles0 : 0)) * kThreads + threadIdx.x;
  if (f >= side.F) return;
  const int n0 = blockIdx.z * kSums, many = min(a.rank - n0, kSums);
  const float* const part = a.part + (second ? a.side[0].F : 0) + f + n0 * features;
  float v[kSums] = {};
#pragma unroll 2
  for (int i = 0; i < found; ++i) {
    const float* p = part + int64_t(list[i] - 1) * a.rank * features;
    float w[kSums];
#pragma unroll
    for (int x = 0; x < kSums; ++x) w[x] = x < many ? p[x * features] : 0.f;
#pragma unroll
    for (int x = 0; x < kSums; ++x) v[x] += w[x];
  }
  const int64_t o = int64_t(blockIdx.y) * side.slice +
                    (side.by_rank ? n0 * side.ldo + f : f * side.ldo + n0);
  const int64_t step = side.by_rank ? side.ldo : 1;
  if (a.accumulate) {
#pragma unroll
    for (int x = 0; x < kSums; ++x)
      if (x < many) v[x] += load_out(side.out, o + x * step, a.d_type);
  }
  const int eb = a.d_type == MMA_F32 ? 4 : 2;
  uint8_t* const d = static_cast<uint8_t*>(side.out) + o * eb;
  if (!side.by_rank && many == kSums && (reinterpret_cast<uintptr_t>(d) & 15) == 0) {
    // a row's eight numbers
    if (a.d_type == MMA_F32) {
      reinterpret_cast<float4*>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint16_t h[8];
#pragma unroll
      for (int x = 0; x < kSums; ++x) store_out(h, x, a.d_type, v[x]);
      *reinterpret_cast<uint4*>(d) = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16,
                                                h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    return;
  }
#pragma unroll
  for (int x = 0; x < kSums; ++x)
    if (x < many) store_out(side.out, o + x * step, a.d_type, v[x]);
}

// Rows per block, in whole stages: some three shares per SM (of 152, so that the
// workspace needs no device), but 16 for each of the rank's sums and 256 at least, so
// that the shares' FP32 sums are a fraction of the rows they are made of.
int rows_per_piece(int64_t T, int64_t N, int64_t K, int64_t rank) {
  const int64_t tiles = (N + kTile - 1) / kTile + (K + kTile - 1) / kTile;
  const int64_t per = std::max<int64_t>(T * tiles / (3 * 152), std::max<int64_t>(16 * rank, 256));
  return int(std::min<int64_t>((per + 63) / 64 * 64, 1 << 20));
}

template <class K, class... Args>
cudaError_t launch_after(const Ctx& ctx, K kernel, dim3 grid, int threads, int smem,
                         const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <bool BF16, int RP, int PARTS>
mma_status_t wgrad(const Ctx& ctx, const LoraWgradProblem& g, const WgradArgs& a) {
  using L = Wgrad<RP>;
  auto kernel = lora_wgrad_kernel<BF16, RP, PARTS>;
  static PerContext<bool> attr;
  bool ok = false;
  if (!attr.get(ctx, &ok, [&](bool* v) {
        *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  L::smem(PARTS)) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return MMA_ERR_LAUNCH;
  cudaError_t e = cudaSuccess;
  if (a.T > 0) {
    WgradMaps maps;
    const int64_t all = int64_t(a.T) * a.ld16;
    for (int i = 0; i < 2; ++i) {
      const bool there = a.side[i].F > 0;  // (else the maps are never used)
      const void* m = !there ? a.halves : i ? g.X : g.DY;
      const int64_t ld = !there ? 8 : i ? g.ldx : g.lddy;
      if (!make_map(&maps.m[i], m, 2, there ? a.side[i].F : 8, there ? a.T : 1, ld, 1, ld, 64,
                    kStageRows) ||
          !make_map(&maps.low[i], a.halves + i * a.parts * all, 2, a.rank, a.T, a.ld16, a.parts,
                    a.parts > 1 ? all : a.ld16, L::RB, kStageRows, swizzle_of(L::RB * 2)))
        return MMA_ERR_LAUNCH;
    }
    const int64_t blocks =
        BF16 ? std::min<int64_t>((all + kThreads - 1) / kThreads, ctx.num_sms * 8) : a.chunks;
    lora_halves_kernel<BF16, RP><<<dim3(unsigned(blocks), 2), kThreads, 0, ctx.stream>>>(a);
    const int64_t pieces = (g.rows + a.per - 1) / a.per + g.requests + 1;
    const int64_t tiles = a.tiles0 + (g.K + kTile - 1) / kTile;
    if (pieces * tiles > INT32_MAX / 2) return MMA_ERR_UNSUPPORTED;
    const int64_t at_once = int64_t(ctx.num_sms) * L::per_sm(PARTS);
    ctx.mark_start();
    e = launch_after(ctx, kernel, dim3(unsigned(std::min(pieces * tiles, at_once))),
                     kThreads + 32, L::smem(PARTS), maps, a, int(pieces), int(tiles));
    ctx.mark_stop();
  }
  const int64_t sums = (g.N + kThreads - 1) / kThreads + (g.K + kThreads - 1) / kThreads;
  if (e == cudaSuccess)
    e = launch_after(ctx, lora_wgrad_sum_kernel,
                     dim3(unsigned(sums), unsigned(a.total),
                          unsigned((a.rank + kSums - 1) / kSums)),
                     kThreads, 0, a);
  const cudaError_t after = cudaGetLastError();
  return e == cudaSuccess && after == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

}  // namespace

mma_status_t launch_lora_shrink(const Ctx& ctx, const LoraProblem& g, const LoraLow& low) {
  return by_rank(g.rank, [&](auto r) {
    constexpr int RP = decltype(r)::value;
    auto go = [&](auto bf16, auto row) {
      constexpr bool B = decltype(bf16)::value, R = decltype(row)::value;
      // (few rows: the k range over all eight warps)
      return g.rows <= kLoraEveryRow ? shrink<B, R, 16, RP, true>(ctx, g, low)
             : g.rows <= kSmallBlocks ? shrink<B, R, 16, RP, false>(ctx, g, low)
                                      : shrink<B, R, 64, RP, false>(ctx, g, low);
    };
    if (g.bf16)
      return g.row_major ? go(std::true_type{}, std::true_type{})
                         : go(std::true_type{}, std::false_type{});
    return g.row_major ? go(std::false_type{}, std::true_type{})
                       : go(std::false_type{}, std::false_type{});
  });
}

namespace {

int64_t round16(int64_t n) { return (n + 15) / 16 * 16; }

// More requests than a kernel lists, or shares of small requests that take more than
// the rows' copies (8 bytes per sum and feature, 8 per row and feature).
bool gathers(int64_t T, int64_t rank, int64_t requests, int64_t total) {
  return total <= MMA_MAX_GROUPS &&
         (requests > MMA_MAX_GROUPS || (requests - total) * rank > T);
}

int64_t gather_ints(int64_t T, int64_t requests, int64_t total) {
  return round16((2 * requests + total + 2 + T) * 4);
}

// Where the shares, the sums' parts and their scales lie.  A piece's number is its block
// and its request, counted from the one before the first: number 0 and the last are of no
// request, so that two shares less are stored than there are pieces.  They are counted in
// `bytes` all the same, and make room for the scales and, with a 16-bit result, for the
// sums' second numbers where those fit.
struct WgradSpace {
  int64_t pieces, chunks, halves, down, bytes;
};

WgradSpace wgrad_space(bool bf16, int d_type, int64_t T, int64_t N, int64_t K, int64_t rank,
                       int64_t requests) {
  const int64_t per = rows_per_piece(T, N, K, rank), share = rank * (N + K) * 4;
  const int64_t number = 2 * T * ((rank + 7) / 8 * 8) * 2;
  const int64_t sums = number * lora_parts(bf16, d_type);
  const int64_t room = rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : 128;
  WgradSpace s;
  s.pieces = (T + per - 1) / per + requests + 1;
  s.chunks = (T + kStageRows - 1) / kStageRows + requests + 1;
  s.halves = round16(std::max<int64_t>(s.pieces - 2, 0) * share);  // (T 0: no pieces)
  s.down = s.halves + round16(sums);
  s.bytes = std::max(round16(s.pieces * share) + (d_type == MMA_F32 ? sums : number),
                     s.down + (bf16 ? 0 : 2 * s.chunks * room * 4));
  return s;
}

// The rows in the order of their adapters.
mma_status_t gather(const Ctx& ctx, LoraWgradProblem& p, WgradArgs& a, uint8_t*& room) {
  Gather g = {};
  g.T = int(p.rows);
  g.requests = int(p.requests);
  g.total = int(p.adapters_total);
  g.offsets = p.offsets;
  g.adapters = p.adapters;
  g.bound = reinterpret_cast<int*>(room);
  g.first = g.bound + g.requests + 1;
  g.starts = g.first + g.requests;
  g.from = g.starts + g.total + 1;
  room += gather_ints(p.rows, p.requests, p.adapters_total);
  const void* const in[2] = {p.DY, p.X};
  const int64_t ld[2] = {p.lddy, p.ldx}, features[2] = {p.N, p.K};
  for (int i = 0; i < 2; ++i) {
    g.in[i] = static_cast<const uint16_t*>(in[i]);
    g.ld[i] = ld[i];
    g.F[i] = int(features[i]);
    g.ld_out[i] = (features[i] + 7) / 8 * 8;
    g.out[i] = reinterpret_cast<uint16_t*>(room);
    room += round16(p.rows * g.ld_out[i] * 2);
  }
  static PerContext<bool> attr;
  bool ok = false;
  if (!attr.get(ctx, &ok, [&](bool* v) {
        *v = cudaFuncSetAttribute(lora_order_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  32 * MMA_MAX_GROUPS * 4) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return MMA_ERR_LAUNCH;
  lora_order_kernel<<<1, 1024, size_t(32 * g.total * 4), ctx.stream>>>(g);
  lora_gather_kernel<<<unsigned(std::min<int64_t>(p.rows, ctx.num_sms * 8)), 256, 0,
                       ctx.stream>>>(g);
  a.from = g.from;
  p.DY = g.out[0];
  p.X = g.out[1];
  p.lddy = g.ld_out[0];
  p.ldx = g.ld_out[1];
  p.offsets = g.starts;
  p.adapters = nullptr;
  p.requests = p.adapters_total;
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

}  // namespace

int64_t lora_wgrad_workspace_bytes(bool bf16, int d_type, int64_t T, int64_t N, int64_t K,
                                   int64_t rank, int64_t requests, int64_t total) {
  if (T == 0) return 0;
  if (gathers(T, rank, requests, total))
    return gather_ints(T, requests, total) + round16(T * ((N + 7) / 8 * 8) * 2) +
           round16(T * ((K + 7) / 8 * 8) * 2) +
           lora_wgrad_workspace_bytes(bf16, d_type, T, N, K, rank, total, total);
  return wgrad_space(bf16, d_type, T, N, K, rank, requests).bytes;
}

mma_status_t launch_lora_wgrad(const Ctx& ctx, const LoraWgradProblem& p, void* workspace) {
  WgradArgs a = {};
  LoraWgradProblem g = p;
  uint8_t* room = static_cast<uint8_t*>(workspace);
  if (p.rows > 0 && gathers(p.rows, p.rank, p.requests, p.adapters_total)) {
    const mma_status_t st = gather(ctx, g, a, room);
    if (st != MMA_OK) return st;
  } else if (p.requests > MMA_MAX_GROUPS) {
    if (p.rows > 0) return MMA_ERR_UNSUPPORTED;
    g.requests = 0;  // (no rows, so none with an adapter)
  }
  a.side[0] = {int(g.N), g.S, g.lds, g.DB, g.lddb, g.stride_db, false};
  a.side[1] = {int(g.K), g.U, g.ldu, g.DA, g.ldda, g.stride_da, true};
  a.tiles0 = int((g.N + kTile - 1) / kTile);
  a.T = int(g.rows);
  a.rank = int(g.rank);
  a.requests = int(g.requests);
  a.total = int(g.adapters_total);
  a.per = rows_per_piece(g.rows, g.N, g.K, g.rank);
  a.offsets = g.offsets;
  a.adapters = g.adapters;
  a.d_type = g.d_type;
  a.parts = lora_parts(g.bf16, g.d_type);
  a.ld16 = (a.rank + 7) / 8 * 8;
  a.accumulate = g.accumulate;
  const WgradSpace space = wgrad_space(g.bf16, g.d_type, g.rows, g.N, g.K, g.rank, g.requests);
  a.part = reinterpret_cast<float*>(room);
  a.halves = reinterpret_cast<uint16_t*>(room + space.halves);
  a.down = reinterpret_cast<float*>(room + space.down);
  a.chunks = int(space.chunks);
  a.status = ctx.status;
  return by_rank(g.rank, [&](auto r) {
    constexpr int RP = decltype(r)::value;
    if (!g.bf16) return wgrad<false, RP, 2>(ctx, g, a);
    return a.parts == 2 ? wgrad<true, RP, 2>(ctx, g, a) : wgrad<true, RP, 3>(ctx, g, a);
  });
}

}  // namespace mmagb
