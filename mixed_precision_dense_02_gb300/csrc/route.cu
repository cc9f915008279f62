// The router of a layer of experts: each token's best k of its logits, their
// weights, the tokens sorted by expert, a balance loss; and its gradient.
//
// A token with logits x: p = softmax(x) in FP32, and its choices are the k largest
// x, of equal ones the lowest index.  Choice j weighs p_j over the sum of the
// chosen p (normalize), or p_j.  An expert with x = -inf is never chosen, and a
// masked token chooses nothing (expert -1, weight 0).  With the n tokens that are
// not masked, counts c_e and share_e = sum over them of p_e / n:
//     loss = E * sum over e of (c_e / (n k)) * share_e
// Its gradient takes the counts as given: with a_e = dloss E c_e / (n^2 k),
//     dx_e = p_e (a_e - sum p a) + (e chosen) w_e (dw_e - sum over chosen w dw)
// or, without normalize, p_e (a_e + dw_e - sum p (a + dw)).
//
// A warp has a token, lane l its experts l, l + 32, ... (any alignment of a row,
// 128 bytes per load).
//
// Sorting is by counting, without atomics whose order would show.  A block sets,
// for each expert, a bit for each of 64 tokens: an expert's tokens before a given
// one are the bits below it.  Blocks of consecutive tokens count, a second kernel
// adds the counts up over the blocks, a third puts every choice in its place.  Of
// few tokens one block does all of it: one launch for generated tokens.
//
// 16384 tokens, 256 experts, 8 each, FP32: 25.5 us, of which the choices take some 15,
// bound by instructions (600 per token; the logits' 17 MB are read at 0.9 TB/s), the
// other two kernels the rest by their launches and latencies.  Gradient 12 us (3 TB/s).
// A lane's share of more than 512 experts does not fit its registers: 144 to 168 bytes a
// thread are spilled, in one block 600 to 660 (from 257 experts 140 to 170).
#include <algorithm>
#include <type_traits>

#include "f8_common.cuh"
#include "ptx.cuh"

namespace mmagb {
namespace {

constexpr int kBatch = 64;        // tokens whose bits are set at a time
constexpr int kMostBlocks = 304;  // of the first kernel
// Least tokens of one, a warp for each (64 experts, 257 tokens: 9.4 us, with 64 13.2).
constexpr int kLeast = 16;
constexpr int kOneBlock = 96;  // most tokens that one block takes alone
// One block or three kernels, device time: 64 experts, 6 each, 32 tokens 5.6 and 8.4 us,
// 64 7.4 and 8.4, 80 9.2 and 8.8, 96 9.5 and 9.1, where a whole call still takes less with
// one launch and no workspace (96 tokens 22.8 us, 97 30.8); 256 experts, 8 each, 32 tokens
// 8.2 and 9.6, 128 19.7 and 11.0; 1024, 32 tokens 22 and 14.9.
constexpr bool one_block(int64_t T, int64_t E) { return T <= kOneBlock && T * E <= 8192; }

struct Choices {
  int tokens, experts, k, per_block, blocks;
  int64_t ldx;
  const void* x;
  const uint8_t* mask;
  bool normalize;
  float* weights;
  int *chosen, *order, *place, *offsets, *live;
  float *share, *loss;
  int* counts;    // [blocks][experts + 2]: choices of each expert, none, tokens
  float* shares;  // [blocks][experts]: sums of p
  int* totals;    // [experts + 2]
};

// FP32 in the order of its bits as an unsigned integer (0: no number).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (uint32_t(int(u) >> 31) | 0x80000000u);
}
constexpr uint32_t kMinusInf = 0x007FFFFFu;
__device__ __forceinline__ float unordered(uint32_t q) {
  return __uint_as_float(q & 0x80000000u ? q ^ 0x80000000u : ~q);
}

// (+ 0: one zero, one NaN, which is above infinity)
__device__ __forceinline__ float logit(float v) { return v + 0.f; }
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// exp(d) for d <= 0 (or NaN), zero where it is below 2^-126: the special function by
// itself, without the scaling that subnormal results take.  d log2(e) in two numbers,
// h + l, because the rounding of one grows with d: 2^h 2^l, 2^l = 1 + l ln 2.
__device__ __forceinline__ float exp_of(float d) {
  d = d < -200.f ? -200.f : d;  // (infinite distances would leave a NaN in l)
  const float h = d * 1.4426950408889634f;
  // (the second constant: what is left of log2(e) beyond FP32, 1.92596e-8)
  const float l = fmaf(d, 1.92596299e-8f, fmaf(d, 1.4426950408889634f, -h));
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(h));
  return fmaf(r, l * 0.69314718056f, r);
}

template <class T, int V>
__device__ __forceinline__ void load_logits(const T* row, int experts, float (&x)[V]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < V; ++c)
    x[c] = c * 32 + lane < experts ? logit(to_float(row[c * 32 + lane])) : -INFINITY;
}

// The k largest of the warp's x, the best first: lane j gets the j-th one's expert,
// or -1 where there is none that is above -inf.
//
// A number's upper 22 bits and, below them, the expert counted from the top: the
// maximum over the warp is one instruction, and of equal ones the lowest index
// wins.  Of 16-bit logits these are all the bits.  FP32 ones that agree in them are
// told apart by `exact_choices`, which is asked if a choice and the next one do.  A
// lane keeps its three largest, and looks through all of its own again when those
// are gone.
template <int V>
__device__ __forceinline__ int exact_choices(const float (&x)[V], int experts, int k) {
  const int lane = threadIdx.x & 31;
  int id = -1;
  uint32_t gone = 0;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint32_t m = 0;
    int c1 = 0;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const uint32_t q =
          c * 32 + lane < experts && !((gone >> c) & 1) ? ordered(x[c]) : 0u;
      if (q > m) {
        m = q;
        c1 = c;
      }
    }
    const uint32_t best = __reduce_max_sync(0xffffffffu, m);
    if (best <= kMinusInf) break;
    const int e = __reduce_min_sync(0xffffffffu, m == best ? c1 * 32 + lane : INT32_MAX);
    if (lane == j) id = e;
    if (lane == (e & 31)) gone |= 1u << c1;
  }
  return id;
}

template <bool WIDE, int V>
__device__ __forceinline__ int choices(const float (&x)[V], int experts, int k) {
  const int lane = threadIdx.x & 31;
  uint32_t q[V], m1 = 0, m2 = 0, m3 = 0;
  auto add = [&](uint32_t v) {
    const uint32_t a = min(m1, v), b = min(m2, a);
    m1 = max(m1, v);
    m2 = max(m2, a);
    m3 = max(m3, b);
  };
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const int e = c * 32 + lane;
    q[c] = e < experts ? (ordered(x[c]) & ~1023u) | uint32_t(1023 - e) : 0u;
    add(q[c]);
  }
  [[maybe_unused]] int left = experts > lane ? (experts - lane + 31) / 32 : 0;
  uint32_t mine = 0, after = 0;
#pragma unroll 1
  for (int j = 0; j <= k; ++j) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, m1);
    if (best <= kMinusInf) break;
    if (j == k) {
      after = best;
      break;
    }
    if (lane == j) mine = best;
    if (m1 == best) {
      m1 = m2;
      m2 = m3;
      m3 = 0;
      --left;
    }
    if constexpr (V > 3) {
      if (__any_sync(0xffffffffu, m1 == 0 && left > 0)) {
        // what this lane has left is below what it has given
        if (m1 == 0) {
#pragma unroll
          for (int c = 0; c < V; ++c) add(q[c] < best ? q[c] : 0u);
        }
      }
    }
  }
  if constexpr (WIDE) {
    uint32_t next = __shfl_down_sync(0xffffffffu, mine, 1);
    if (lane >= k - 1) next = after;
    if (__any_sync(0xffffffffu, mine != 0 && next != 0 && ((mine ^ next) >> 10) == 0))
      return exact_choices<V>(x, experts, k);
  }
  return mine ? 1023 - int(mine & 1023u) : -1;
}

// Exclusive sums of the block's values, one per thread, in `sums` (32 ints).
__device__ __forceinline__ int block_scan(int v, int* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += o;
  }
  if (lane == 31) sums[warp] = s;
  __syncthreads();
  if (warp == 0) {
    const int warps = int(blockDim.x + 31) / 32;
    int t = lane < warps ? sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += o;
    }
    __syncwarp();
    sums[lane] = t;
  }
  __syncthreads();
  return s - v + (warp > 0 ? sums[warp - 1] : 0);
}

// E times the sum of count times share, over the block; in thread 0.
__device__ __forceinline__ float balance(const int* counts, const float* share, int experts,
                                         int k, int live, float* buf) {
  float s = 0.f;
#pragma unroll 1
  for (int e = threadIdx.x; e < experts; e += blockDim.x)
    s = fmaf(float(counts[e]), share[e], s);
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.f;
#pragma unroll 4
  for (int w = 0; w < int(blockDim.x) / 32; ++w) s += buf[w];
  return live > 0 ? s * float(experts) / (float(live) * float(k)) : 0.f;
}

// Tokens [b * per_block, ...) of block b.  ONE: all tokens, and the rest of the
// work too.
template <class T, int V, bool ONE>
__global__ void __launch_bounds__(ONE ? 1024 : 512)
    route_kernel(const Choices a) {
  extern __shared__ __align__(16) uint8_t room[];
  __shared__ int warp_live[32], scan[32];
  __shared__ float fsum[32];
  const int E = a.experts, k = a.k, warps = blockDim.x >> 5;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // an expert's tokens of the batch; behind them those without a choice j
  uint2* bits = reinterpret_cast<uint2*>(room);
  int* count = reinterpret_cast<int*>(bits + E + k);  // E experts, none
  float* psum = reinterpret_cast<float*>(count + E + 1);       // [warps][E]
  uint16_t* ids = reinterpret_cast<uint16_t*>(psum + warps * E);  // E: none
  uint16_t* ranks = ids + (ONE ? kOneBlock : kBatch) * k;         // (ONE)
#pragma unroll 1
  for (int e = threadIdx.x; e < E + k; e += blockDim.x) bits[e] = make_uint2(0, 0);
#pragma unroll 1
  for (int e = threadIdx.x; e <= E; e += blockDim.x) count[e] = 0;
  if constexpr (!ONE) grid_dependents_start();
  const int first = ONE ? 0 : blockIdx.x * a.per_block;
  const int last = min(first + a.per_block, a.tokens);
  const T* X = static_cast<const T*>(a.x);
  float acc[V];
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.f;
  int live = 0;
  float x[V];
  bool on = true;  // (the next token's, as x)
  auto fetch = [&](int t) {
    load_logits<T, V>(X + t * a.ldx, E, x);
    if (a.mask) on = __ldg(a.mask + t) != 0;
  };
  if (first + warp < last) fetch(first + warp);
  __syncthreads();
  for (int t0 = first; t0 < last; t0 += kBatch) {
    uint16_t* const id0 = ids + (ONE ? t0 * k : 0);
#pragma unroll 1
    for (int i = warp; i < kBatch && t0 + i < last; i += warps) {
      const int t = t0 + i;
      float y[V];
#pragma unroll
      for (int c = 0; c < V; ++c) y[c] = x[c];
      // the warp's next token, in this batch or the one after
      const int next = i + warps < kBatch ? t + warps : t0 + kBatch + warp;
      const bool live_one = on;
      if (next < last) fetch(next);
      int id = -1;      // lane j: choice j
      float top = 0.f;  // its logit
      uint32_t most_key = 0;
#pragma unroll
      for (int c = 0; c < V; ++c) most_key = max(most_key, ordered(y[c]));
      most_key = __reduce_max_sync(0xffffffffu, most_key);
      const bool some = live_one && most_key > kMinusInf;
      const float most = unordered(most_key);
      if (some) {
        id = choices<sizeof(T) == 4, V>(y, E, k);
        if (id >= 0) top = logit(to_float(X[t * a.ldx + id]));
      }
      live += live_one;
      float sum = 0.f;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        y[c] = some ? exp_of(y[c] - most) : 0.f;
        sum += y[c];
      }
      sum = warp_sum(sum);
      const float over = some ? __fdividef(1.f, sum) : 0.f;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] = fmaf(y[c], over, acc[c]);
      float w = id >= 0 ? exp_of(top - most) : 0.f;
      if (a.normalize) {
        // (a NaN among the logits is in every weight)
        const float chosen = warp_sum(w);
        w = id < 0 ? 0.f : sum == sum ? __fdividef(w, chosen) : sum;
      } else {
        w = id < 0 ? 0.f : w * over;
      }
      if (lane < k) {
        a.weights[int64_t(t) * k + lane] = w;
        a.chosen[int64_t(t) * k + lane] = id;
        id0[i * k + lane] = uint16_t(id < 0 ? E : id);
        uint2* b = bits + (id < 0 ? E + lane : id);
        atomicOr(i < 32 ? &b->x : &b->y, 1u << (i & 31));
      }
    }
    __syncthreads();
    const int here = min(kBatch, last - t0) * k;
#pragma unroll 1
    for (int c = threadIdx.x; c < here; c += blockDim.x) {
      const int i = c / k, j = c - i * k, id = id0[c];
      const uint2 below = i < 32 ? make_uint2((1u << i) - 1, 0u)
                                 : make_uint2(0xffffffffu, (1u << (i & 31)) - 1);
      auto before = [&](int b) {
        return __popc(bits[b].x & below.x) + __popc(bits[b].y & below.y);
      };
      int rank = count[id];
      if (id < E) {
        rank += before(id);
      } else {
        // choices without an expert: of earlier tokens, and this one's earlier
#pragma unroll 1
        for (int q = 0; q < k; ++q) {
          rank += before(E + q);
          if (q < j) rank += ((i < 32 ? bits[E + q].x : bits[E + q].y) >> (i & 31)) & 1;
        }
      }
      if constexpr (ONE)
        ranks[t0 * k + c] = uint16_t(rank);
      else
        a.place[int64_t(t0) * k + c] = rank;
    }
    __syncthreads();
#pragma unroll 1
    for (int e = threadIdx.x; e <= E; e += blockDim.x) {
      int n = 0;
#pragma unroll 1
      for (int b = e; b < (e < E ? e + 1 : E + k); ++b) {
        n += __popc(bits[b].x) + __popc(bits[b].y);
        bits[b] = make_uint2(0, 0);
      }
      count[e] += n;
    }
    __syncthreads();
  }
#pragma unroll
  for (int c = 0; c < V; ++c)
    if (c * 32 + lane < E) psum[warp * E + c * 32 + lane] = acc[c];
  if (lane == 0) warp_live[warp] = live;
  __syncthreads();
  live = 0;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) live += warp_live[w];
#pragma unroll 1
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    float s = 0.f;
#pragma unroll 4
    for (int w = 0; w < warps; ++w) s += psum[w * E + e];
    if constexpr (ONE) {
      psum[e] = live > 0 ? s / float(live) : 0.f;  // (this thread's own column)
      a.share[e] = psum[e];
    } else {
      a.shares[int64_t(blockIdx.x) * E + e] = s;
    }
  }
  if constexpr (!ONE) {
    int* out = a.counts + int64_t(blockIdx.x) * (E + 2);
#pragma unroll 1
    for (int e = threadIdx.x; e <= E; e += blockDim.x) out[e] = count[e];
    if (threadIdx.x == 0) out[E + 1] = live;
  } else {
    __syncthreads();
    const float loss = balance(count, psum, E, k, live, fsum);
    const int mine = int(threadIdx.x) < E ? count[threadIdx.x] : 0;
    const int at = block_scan(mine, scan);
    // (every thread is past its reads of the counts)
    if (int(threadIdx.x) < E) {
      count[threadIdx.x] = at;
      a.offsets[threadIdx.x] = at;
      if (int(threadIdx.x) == E - 1) {
        a.offsets[E] = at + mine;
        count[E] = at + mine;
      }
    }
    if (threadIdx.x == 0) {
      *a.loss = loss;
      *a.live = live;
    }
    __syncthreads();
#pragma unroll 1
    for (int c = threadIdx.x; c < a.tokens * k; c += blockDim.x) {
      const int at = count[ids[c]] + ranks[c];
      a.place[c] = at;
      a.order[at] = c;
    }
  }
}

// For each of 32 columns of the counts, the sums over the blocks before; the
// totals; the shares.  A thread has up to ten consecutive blocks of a column, which
// stay in registers between the two readings; the sums of the threads of a column
// are added up by a warp.
__global__ void __launch_bounds__(1024) route_scan_kernel(const Choices a) {
  constexpr int kRows = (kMostBlocks + 31) / 32;
  __shared__ int part[32][33], live_of[32];
  __shared__ float fpart[32][33];
  const int columns = a.experts + 2, x = threadIdx.x, y = threadIdx.y;
  const int e = blockIdx.x * 32 + x;
  grid_dependency_wait();
  grid_dependents_start();
  int n[kRows], sum = 0;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = y * kRows + i;
    n[i] = r < a.blocks && e <= a.experts ? a.counts[r * columns + e] : 0;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = y * kRows + i;
    if (r < a.blocks && e < a.experts) s += a.shares[r * a.experts + e];
    sum += n[i];
  }
  part[y][x] = sum;
  fpart[y][x] = s;
  // tokens that take part, over all blocks (column E + 1 stays as it is)
  const int thread = y * 32 + x;
  int live = thread < a.blocks ? a.counts[thread * columns + a.experts + 1] : 0;
  live = __reduce_add_sync(0xffffffffu, live);
  if (x == 0) live_of[y] = live;
  __syncthreads();
  live = __reduce_add_sync(0xffffffffu, live_of[x]);
  // column y of this block's 32, thread rows along the lanes
  const int col = blockIdx.x * 32 + y;
  const int mine = part[x][y];
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, before, d);
    if (x >= d) before += o;
  }
  if (x == 31 && col <= a.experts) a.totals[col] = before;
  const float share = warp_sum(fpart[x][y]);
  if (x == 0 && col < a.experts) a.share[col] = live > 0 ? share / float(live) : 0.f;
  part[x][y] = before - mine;
  if (blockIdx.x == 0 && thread == 0) *a.live = live;
  __syncthreads();
  int at = part[y][x];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = y * kRows + i;
    if (r < a.blocks && e <= a.experts) a.counts[r * columns + e] = at;
    at += n[i];
  }
}

// Every choice's place.
__global__ void __launch_bounds__(1024) route_place_kernel(const Choices a) {
  __shared__ int offset[kMaxGroups + 1];
  __shared__ int scan[32];
  __shared__ float fsum[32];
  grid_dependency_wait();
  const int E = a.experts;
  const int mine = int(threadIdx.x) < E ? a.totals[threadIdx.x] : 0;
  const int at = block_scan(mine, scan);
  if (int(threadIdx.x) < E) {
    offset[threadIdx.x] = at;
    if (int(threadIdx.x) == E - 1) offset[E] = at + mine;
  }
  __syncthreads();
  if (blockIdx.x == 0) {
#pragma unroll 1
    for (int e = threadIdx.x; e <= E; e += blockDim.x) a.offsets[e] = offset[e];
    const float loss = balance(a.totals, a.share, E, a.k, *a.live, fsum);
    if (threadIdx.x == 0) *a.loss = loss;
  }
  // (a block of the first kernel after the other: its counts are one row)
#pragma unroll 1
  for (int b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    const int per = a.per_block * a.k, from = b * per, to = min(from + per, a.tokens * a.k);
    const int* before = a.counts + int64_t(b) * (E + 2);
#pragma unroll 1
    for (int c = from + threadIdx.x; c < to; c += blockDim.x) {
      const int id = a.chosen[c], e = id < 0 ? E : id;
      const int p = offset[e] + before[e] + a.place[c];
      a.place[c] = p;
      a.order[p] = c;
    }
  }
}

// The gradient of the logits, a warp per token.
template <class T, int V>
__global__ void __launch_bounds__(256)
    route_backward_kernel(const RouteBackProblem p) {
  extern __shared__ float slabs[];  // per warp, by expert: what its choice adds
  const int E = int(p.E), k = int(p.k), lane = threadIdx.x & 31;
  float* const slab = slabs + (threadIdx.x >> 5) * E;
  float a[V];
#pragma unroll
  for (int c = 0; c < V; ++c) a[c] = 0.f;
  if (p.dloss) {
    const float n = float(max(*p.tokens, 1));
    const float f = *p.dloss * float(E) / n / n / float(k);
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int e = c * 32 + lane;
      if (e < E) a[c] = f * float(p.offsets[e + 1] - p.offsets[e]);
    }
  }
#pragma unroll 1
  for (int e = lane; e < E; e += 32) slab[e] = 0.f;
  __syncwarp();
  const int warps = gridDim.x * (blockDim.x >> 5);
  for (int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); t < int(p.T); t += warps) {
    T* const out = static_cast<T*>(p.dx) + t * p.lddx;
    const bool on = p.mask == nullptr || p.mask[t] != 0;
    float x[V];
    load_logits<T, V>(static_cast<const T*>(p.x) + t * p.ldx, E, x);
    int id = -1;
    float g = 0.f;
    if (p.dweights && on && lane < k) {
      id = p.chosen[int64_t(t) * k + lane];
      if (id >= E) id = -1;
      if (id >= 0) g = p.dweights[int64_t(t) * k + lane];
    }
    if (p.dweights && p.normalize) {
      const float w = id >= 0 ? p.weights[int64_t(t) * k + lane] : 0.f;
      const float mean = warp_sum(w * g);
      g = w * (g - mean);
    }
    if (id >= 0) slab[id] = g;
    // (as the forward kernel: a NaN is the largest, and makes the whole row NaN)
    uint32_t most_key = 0;
#pragma unroll
    for (int c = 0; c < V; ++c) most_key = max(most_key, ordered(x[c]));
    most_key = __reduce_max_sync(0xffffffffu, most_key);
    const bool some = on && most_key > kMinusInf;
    const float most = unordered(most_key);
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      x[c] = some ? exp_of(x[c] - most) : 0.f;
      sum += x[c];
    }
    sum = warp_sum(sum);
    const float over = some ? __fdividef(1.f, sum) : 0.f;
    __syncwarp();
    float dot = 0.f, add[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int e = c * 32 + lane;
      add[c] = p.dweights && e < E ? slab[e] : 0.f;
      x[c] *= over;
      dot = fmaf(x[c], p.normalize ? a[c] : a[c] + add[c], dot);
    }
    dot = warp_sum(dot);
    __syncwarp();
    if (id >= 0) slab[id] = 0.f;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const int e = c * 32 + lane;
      const float d = p.normalize ? fmaf(x[c], a[c] - dot, add[c])
                                  : x[c] * (a[c] + add[c] - dot);
      if (e < E) out[e] = Vec<T>::round(some ? d : 0.f);
    }
    __syncwarp();
  }
}

template <class F>
cudaError_t launch(const Ctx& ctx, F kernel, dim3 grid, dim3 block, size_t smem, bool after,
                   const Choices& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

struct Split {
  int per_block, blocks;
};

Split split_of(int64_t T) {
  const int64_t per = std::max<int64_t>(kLeast, (T + kMostBlocks - 1) / kMostBlocks);
  return Split{int(per), int(std::max<int64_t>(1, (T + per - 1) / per))};
}

template <class T, int V>
mma_status_t route(const Ctx& ctx, const Choices& a) {
  const bool one = one_block(a.tokens, a.experts);
  const int warps = one ? 32 : 16;
  const size_t smem = size_t(a.experts + a.k) * 8 + size_t(a.experts + 1) * 4 +
                      size_t(warps) * a.experts * 4 +
                      size_t(one ? 2 * kOneBlock : kBatch) * a.k * 2;
  auto kernel = one ? route_kernel<T, V, true> : route_kernel<T, V, false>;
  static PerContext<bool> attr[2];
  bool ok = false;
  if (!attr[one].get(ctx, &ok, [&](bool* v) {
        *v = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  200 * 1024) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return MMA_ERR_LAUNCH;
  cudaError_t e = launch(ctx, kernel, dim3(one ? 1 : a.blocks), dim3(warps * 32), smem, false, a);
  if (!one) {
    if (e == cudaSuccess)
      e = launch(ctx, route_scan_kernel, dim3((a.experts + 2 + 31) / 32), dim3(32, 32), 0, true, a);
    if (e == cudaSuccess)
      e = launch(ctx, route_place_kernel, dim3(a.blocks), dim3(1024), 0, true, a);
  }
  const cudaError_t last = cudaGetLastError();
  return e == cudaSuccess && last == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

template <class T, int V>
mma_status_t route_back(const Ctx& ctx, const RouteBackProblem& p) {
  // (a warp's share of the counts is some hundred instructions, so several tokens)
  const int64_t blocks = std::min<int64_t>((p.T + 7) / 8, int64_t(ctx.num_sms) * 4);
  route_backward_kernel<T, V><<<unsigned(blocks), 256, size_t(8) * p.E * 4, ctx.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

// Calls f for the registers that a lane's share of the experts takes.
template <class F>
mma_status_t by_width(int64_t experts, F&& f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>{});
  if (experts <= 64) return f(std::integral_constant<int, 2>{});
  if (experts <= 128) return f(std::integral_constant<int, 4>{});
  if (experts <= 256) return f(std::integral_constant<int, 8>{});
  if (experts <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace

int64_t route_workspace_bytes(int64_t T, int64_t E) {
  return one_block(T, E) ? 0 : (int64_t(split_of(T).blocks) * (2 * E + 2) + E + 2) * 4;
}

mma_status_t launch_route(const Ctx& ctx, const RouteProblem& p, void* workspace) {
  Choices a = {};
  const Split s = split_of(p.T);
  a.tokens = int(p.T);
  a.experts = int(p.E);
  a.k = int(p.k);
  a.per_block = one_block(p.T, p.E) ? kOneBlock : s.per_block;
  a.blocks = s.blocks;
  a.ldx = p.ldx;
  a.x = p.x;
  a.mask = p.mask;
  a.normalize = p.normalize;
  a.weights = p.weights;
  a.chosen = p.chosen;
  a.order = p.order;
  a.place = p.place;
  a.offsets = p.offsets;
  a.live = p.tokens;
  a.share = p.share;
  a.loss = p.loss;
  a.counts = static_cast<int*>(workspace);
  a.totals = a.counts + int64_t(s.blocks) * (p.E + 2);
  a.shares = reinterpret_cast<float*>(a.totals + p.E + 2);
  return by_width(p.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    return p.type == MMA_F32    ? route<float, V>(ctx, a)
           : p.type == MMA_BF16 ? route<__nv_bfloat16, V>(ctx, a)
                                : route<__half, V>(ctx, a);
  });
}

mma_status_t launch_route_backward(const Ctx& ctx, const RouteBackProblem& p) {
  return by_width(p.E, [&](auto v) {
    constexpr int V = decltype(v)::value;
    return p.type == MMA_F32    ? route_back<float, V>(ctx, p)
           : p.type == MMA_BF16 ? route_back<__nv_bfloat16, V>(ctx, p)
                                : route_back<__half, V>(ctx, p);
  });
}

}  // namespace mmagb
