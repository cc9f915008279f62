// Products with scaled 8-bit operands and products grouped by expert, on
// the tcgen05 tensor cores.  One kernel carries all of them:
//
//     D[q][p] or D[p][q] = C + sum_k P[p][k] * Q[q][k]
//
// with P the operand on the tensor core's M side (128 rows per CTA) and Q
// the one on its N side:
//
//   call                          P (rows p)       Q (rows q)       k
//   grouped forward               B_e (N x K)      A (token x K)    K
//   grouped, row-major B          B_e (K x N)^T    A (token x K)    K
//   grouped weight gradient       X (token x K)^T  dY (token x N)^T tokens
//   8-bit, few rows or scales     B_e (N x K)      A (token x K)    K
//     of single rows of B
//   8-bit, many rows (ROWS)       A (token x K)    B_e (N x K)      K
//
// In all but the last D's rows leave the kernel as runs of consecutive p,
// one per lane, and the ragged dimension of a group (its tokens) is the N
// side, whose extent is chosen per tile in steps of 16 (32 with CTA pairs):
// a group of 300 tokens costs 320 rows of tensor work, not 384 or 512.  With
// ROWS a lane holds one token, so that both scales of an 8-bit block product
// are one number per lane.
//
// Arithmetic.  The tensor core's FP32 sums drop low bits on the way (a
// relative error that grows with the length of the sum: 1.2e-7 at 128 terms
// and 4.2e-6 at 4096, measured against 64 bits), so K is cut into chunks;
// each chunk's sum is added to FP32 registers, rounded to nearest.  With
// 8-bit operands a chunk is one block of 128 and the addition multiplies by
// the product of the block's two scales: acc += (sp * sq) * t.
//
// Roles: warp 0 loads operand boxes by TMA into a ring of stages of 128
// bytes of k, warp 1 issues the MMAs into two accumulators in tensor memory,
// eight warps add the chunks up in registers and store D.  CL = 2: a pair of
// CTAs shares one MMA of 256 rows of P, each staging its own 128 rows and
// half of Q, so that a stage brings 32 KB per SM instead of 48; every SM
// streaming from L2 gets about 69 bytes per clock, and the stage's MMAs take
// 512 clocks.
//
// Few tiles (a token or a few through one matrix): a cluster of up to six
// CTAs shares a tile's k range (SPLIT); the sums meet in the shared memory of
// its first CTA, which adds them in order of rank.
//
// Measured, operands rotating through more than L2, and what bounds it.  First
// in a graph of a few calls, then under a load of half a second and more, when
// the power limit has lowered the clock:
//   8-bit 8192 x 8192 x 4096, square scales, BF16 D: 207-212 us, 222-234
//     (2350 to 2660 TFLOP/s).  The additions: a chunk's loads of tensor memory
//     and FMAs keep an epilogue warp some 830 clocks, its MMAs take 530.
//   8-bit 2048 x 4096 x 8200, row scales, FP32 C and D: 99 us, 99 (1384
//     TFLOP/s).  The same with a multiplication more per element, and 128 tiles
//     are two waves of 76 pairs, the second two thirds full.
//   32 experts of 4096 x 2048, 16384 tokens, BF16: forward 184-192 us, 212-220;
//     input gradient 182-220, 210-221 (1250 to 1510 TFLOP/s).  The tensor pipe
//     at a power-capped clock; groups rounded to 32 rows are 3 % more work, and
//     tiles of some 205 of the 256 columns read P more often.
//   The same weight gradient: FP32 307-350 us, 315-327; BF16 242-248, 254-262.
//     Writes of D: 1.07 GB, which take 186 us when there is nothing to add up.
//   The same forward in 8 bits: 157 us, 165-169 (1640 TFLOP/s).  The additions.
//   64 experts of 2048 x 4096, 96 tokens, 8-bit: 63 us, 5.9 TB/s.  HBM.
//   One token, 8192 x 4096, 8-bit: 10.0 us, 3.4 TB/s.  Some 2 us each for the
//     first loads' latency and for the join of a cluster's sums.
// All with the scales of one k block side by side.  Scales with a row's side by
// side (a gather of rows makes them so) are 32 lines per copy: 221-225 us, the
// row scales 139, one token 10.0-10.8, the experts' the same.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace mmagb {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm_tc.cu

bool make_map(CUtensorMap* map, const void* base, int elem, int64_t inner,
              int64_t outer, int64_t ld, int64_t count, int64_t slice,
              int box_inner, int box_outer,
              CUtensorMapSwizzle swizzle) {
  auto enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {cuuint64_t(inner), cuuint64_t(outer), cuuint64_t(count)};
  cuuint64_t strides[2] = {cuuint64_t(ld) * elem, cuuint64_t(slice) * elem};
  cuuint32_t box[3] = {cuuint32_t(box_inner), cuuint32_t(box_outer), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  // 16-bit elements are moved as bit patterns; zero fill is the same for all
  return enc(map,
             elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                       : CU_TENSOR_MAP_DATA_TYPE_UINT16,
             3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

constexpr int kP = 128;  // rows of P per CTA
constexpr int kEpiWarps = 8;
// One warpgroup for the loads and MMAs (two of its warps idle), two for the
// epilogue.  384 threads start with 168 registers each; with 128 sums per
// lane the epilogue takes 224 and leaves the first warpgroup 56
// (56 + 2 * 224 = 3 * 168): at 168 the sums spill, and a spill is an L2
// round trip because shared memory leaves no L1 (8-bit 8192 x 8192 x 4096:
// 1290 us with the spills).
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr int kLaunchRegs = 168, kLoadRegs = 56, kEpiRegs = 224;
static_assert(kLoadRegs + 2 * kEpiRegs <= 3 * kLaunchRegs, "registers");
constexpr int kBand = 16;  // q tiles of a band of the raster

// What a launch computes (see the table above).  Group e's tokens are
// [row[e], row[e + 1]) of `offsets` (one group of rows_total without
// offsets): rows of Q, rows of P with ROWS, the k range for the weight
// gradient.  The sides that no group cuts have p_size and q_size rows.
struct GroupedArgs {
  int p_size, q_size, k_size, groups, rows_total;
  const int* offsets;
  uint32_t idesc;  // without the N field
  int kb_per_chunk;
  int part_cols;  // SPLIT: most columns of a tile in use
  int d_type;  // MMA_F32, MMA_F16 or MMA_BF16
  // ROWS: four elements of a row of D (and C) can move at once; D is 16-bit,
  // there is no C and eight can
  int vec4, vec8;
  int d_tma;  // ROWS: D may be stored through tmD
  const void* C;
  int64_t ldc, c_group;
  void* D;
  int64_t ldd, d_group;
  // 8-bit operands.  The scale of row p for k block b: sp[e * sp_group +
  // (p >> p_shift) * sp_row + b * sp_blk]; likewise of row q.
  const float* sp;
  int64_t sp_group, sp_row, sp_blk;
  int p_shift;
  const float* sq;
  int64_t sq_group, sq_row, sq_blk;
  int q_shift;
  int withhold;  // (self-test) issue no loads
  unsigned* status;
  // LORA: what the adapters add in FP32, rows of p_size.  kEveryRow: of every row of
  // Q.  kRequests: `offsets` are those of `groups` requests, which cut nothing.
  // Request i's rows have the adapter adapters[i] (NULL: i; outside [0,
  // adapters_total): none), whose `rank` sums per row are, in `parts` parts of 16
  // bits, behind tmD, and whose second matrix is behind tmZ.rows[0]; `extra` has
  // those of requests of fewer than kLoraRows rows (places: lora_own_places).
  // `up`: the exponents of the rows' scales, ld_up apart (FP16), or null.
  const float* extra;
  const int* adapters;
  int adapters_total, rank, parts;
  const uint16_t* up;
  int ld_up;
};

template <bool KIND8, bool ROWS, bool SPLIT, int CL, int BN, int STAGES>
struct Layout {
  static constexpr int P_BYTES = kP * 128;
  static constexpr int Q_BYTES = BN / CL * 128;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  // 8-bit: a ring of the chunks' scales, G chunks per slot; a chunk's are
  // 128 of P, then those of Q (ROWS: of the two halves of the columns)
  // (a change of slots costs an epilogue warp some 300 clocks: 8192 x 8192 x
  // 4096 with two chunks per slot 247 us, with four 228, with eight 220)
  static constexpr int G = BN <= 64 ? 4 : 8;
  static constexpr int SLOTS = KIND8 ? 2 : 0;
  static constexpr int CHUNK_FLOATS = kP + (ROWS ? 4 : BN);
  static constexpr int SLOT_FLOATS = G * CHUNK_FLOATS;
  static constexpr int SCALE_OFFSET = STAGES * STAGE_BYTES;
  // per epilogue warp: a ring of blocks of D, 32 rows x 64 bytes (ROWS)
  static constexpr int BLOCKS = ROWS ? 4 : 0;
  static constexpr int WARP_BYTES = BLOCKS * 2048;
  static constexpr int WARP_OFFSET =
      (SCALE_OFFSET + SLOTS * SLOT_FLOATS * 4 + 1023) / 1024 * 1024;
  static constexpr int BAR_OFFSET = WARP_OFFSET + kEpiWarps * WARP_BYTES;
  // Accumulators in tensor memory: as many as fit (with 32 and 64 columns
  // 256 of the 512, for two CTAs per SM).  A chunk's way through the MMAs, the
  // epilogue and back takes some 1000 clocks whatever its size.
  static constexpr int ACCS = BN == 32 ? 8 : BN == 64 ? 4 : 512 / BN;
  // Parts of an accumulator that are handed over by themselves (8-bit,
  // 256 columns: its two halves, each to the four warps that add it), so
  // that a half's MMAs wait for half the epilogue.
  static constexpr int HV = KIND8 && BN == 256 ? 2 : 1;
  static constexpr int NUM_BARS =
      4 * STAGES + 1 + 2 * ACCS * HV + 2 * SLOTS + (SPLIT ? kEpiWarps : 0);
  static constexpr int GROUP_OFFSET = BAR_OFFSET + NUM_BARS * 8 + 24;
  static constexpr int round16(int v) { return (v + 15) & ~15; }
  // SPLIT: sums of the other ranks, 128 rows of P times the columns in use
  static constexpr int part_offset(int groups, int lists = 2) {
    return round16(GROUP_OFFSET + lists * (groups + 1) * 4);
  }
  static constexpr int alloc(int groups, int split, int part_cols, int lists = 2) {
    // (1024: alignment of the base)
    return part_offset(groups, lists) + (split - 1) * part_cols * kP * 4 + 1024;
  }
  static constexpr uint32_t TMEM_COLS = ACCS * BN;
};

// Maps of boxes of 1, 2, 4 and 8 rows (the weight gradient's zeros).
struct ZeroMaps {
  CUtensorMap rows[4];
};

// One tile of work.
struct Tile {
  int e;       // group
  int p0, p1;  // rows of P: first of the tile, end of the group's or operand's
  int q0, q1;  // rows of Q
  int nt;      // MMA N: q1 - q0 rounded up
  int k0, k1;  // k range
};

__device__ __forceinline__ float load_c(const void* c, int64_t i, int t) {
  if (t == MMA_F32) return static_cast<const float*>(c)[i];
  if (t == MMA_BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(c)[i]);
  return __half2float(static_cast<const __half*>(c)[i]);
}

__device__ __forceinline__ void store_d(void* d, int64_t i, int t, float v) {
  if (t == MMA_F32)
    static_cast<float*>(d)[i] = v;
  else if (t == MMA_BF16)
    static_cast<__nv_bfloat16*>(d)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(d)[i] = __float2half_rn(v);
}

// Two FP32 values rounded to 16 bits, lo in the low half.
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float4 load_c4(const void* c, int64_t i, int t) {
  if (t == MMA_F32)
    return *reinterpret_cast<const float4*>(static_cast<const float*>(c) + i);
  const uint2 w =
      *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(c) + i);
  float2 lo, hi;
  if (t == MMA_BF16) {
    lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.x));
    hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.y));
  } else {
    lo = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
    hi = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
  }
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

__device__ __forceinline__ void store_d4(void* d, int64_t i, int t, float4 v) {
  if (t == MMA_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(d) + i) = v;
    return;
  }
  const bool bf16 = t == MMA_BF16;
  const uint2 w = make_uint2(pack16(v.x, v.y, bf16), pack16(v.z, v.w, bf16));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(d) + i) = w;
}

// Row and column of sum s of a lane that holds pairs (PAIRS), counted from
// its first of each.
__device__ constexpr int pairs_row(int s) { return ((s >> 4) & 1) * 16 + ((s >> 1) & 1) * 8; }
__device__ constexpr int pairs_q(int s) { return (s >> 5) * 32 + ((s >> 2) & 3) * 8 + (s & 1); }

// LORA: what the adapters of requests add to a product's rows.  kEveryRow: FP32
// rows that another kernel has made.  kRequests: products of the tensor core's, a
// request at a time, with an accumulator of its own of which only the request's
// columns are added, so that an adapter's infinities stay with it; requests of fewer
// than kLoraRows rows as with kEveryRow.  (Both wait for the kernels before only
// where they read what those make, so that the shared product runs beside them: a CTA's
// first tile up to its sums.  From there on a bounded wait could last as long as those
// kernels, for accumulators whose sums wait for them, and every role waits for their end
// first.)
enum Lora { kNoLora, kEveryRow, kRequests };

// KIND8: 8-bit operands with scales, else 16-bit.  P_MN, Q_MN: the operand
// is stored with its row index contiguous (16-bit only).  RAGK: the groups
// cut the k range (the weight gradient).  ROWS: D[p][q], the groups cut P.
// SPLIT: the CTAs of a cluster share the k range (CL = 1, K-major).  LORA: one
// group (16-bit, neither RAGK nor ROWS).
template <bool KIND8, bool P_MN, bool Q_MN, bool RAGK, bool ROWS, bool SPLIT, int CL,
          int BN, int STAGES, Lora LORA>
__global__ void __launch_bounds__(kThreads,
                                  SPLIT && (BN == 32 || (LORA && BN == 64)) ? 2 : 1)
    gemm_grouped_kernel(const __grid_constant__ CUtensorMap tmP,
                        const __grid_constant__ CUtensorMap tmQ,
                        const __grid_constant__ CUtensorMap tmD,
                        const __grid_constant__ ZeroMaps tmZ,
                        const __grid_constant__ GroupedArgs a) {
  using L = Layout<KIND8, ROWS, SPLIT, CL, BN, STAGES>;
  constexpr int KE = KIND8 ? 128 : 64;  // k elements per stage
  constexpr int PT = kP * CL;           // rows of P per tile
  constexpr int QS = 16 * CL;           // granularity of the MMA's N
  constexpr int HALF = BN / 2;          // most columns of an epilogue warp
  constexpr int HV = L::HV;
  constexpr int QPART = BN / CL / HV;   // rows of Q per box
  // (with 80 registers, so that two CTAs fit an SM, 32 sums leave room for 16 more)
  constexpr int CB = HALF < 32 || (LORA && SPLIT && BN == 64) ? 16 : 32;
  constexpr int NB = HALF / CB;
  constexpr bool kSplitRegs = HALF == 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFFSET);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + L::ACCS * L::HV;
  uint64_t* done = tempty + L::ACCS * L::HV;
  uint64_t* cut_in = done + 1;         // RAGK: a cut block has landed here
  uint64_t* cut_ok = cut_in + STAGES;  // and its zeros are in place (leader)
  uint64_t* sfull = cut_ok + STAGES;
  uint64_t* sempty = sfull + L::SLOTS;
  // SPLIT, one per epilogue warp: the other ranks' sums are here (rank 0)
  uint64_t* part_full = sempty + L::SLOTS;
  uint32_t* tmem_slot =
      reinterpret_cast<uint32_t*>(part_full + (SPLIT ? kEpiWarps : 0));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* grow = reinterpret_cast<int*>(smem + L::GROUP_OFFSET);  // groups + 1
  int* gunit = grow + a.groups + 1;                            // groups + 1
  [[maybe_unused]] int* glist = gunit + a.groups + 1;          // (kRequests) groups + 1

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = CL > 1 ? int(cluster_ctarank()) : 0;
  const int krank = SPLIT ? int(cluster_ctarank()) : 0;
  const int ksplit = SPLIT ? int(cluster_size()) : 1;
  const int p_tiles = (a.p_size + PT - 1) / PT;  // ROWS: of no meaning
  const int q_tiles = (a.q_size + BN - 1) / BN;  // RAGK, ROWS
  // tiles of a group with `rows` rows
  auto units_of = [&](int rows) {
    return RAGK ? q_tiles * p_tiles
           : ROWS ? ((rows + PT - 1) / PT) * q_tiles
                  : ((rows + BN - 1) / BN) * p_tiles;
  };

  if (threadIdx.x == 32) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&cut_in[s], 1);
      mbar_init(&cut_ok[s], 1);
    }
    for (int s = 0; s < L::SLOTS; ++s) {
      mbar_init(&sfull[s], 32);
      mbar_init(&sempty[s], kEpiWarps);
    }
    for (int i = 0; i < L::ACCS * L::HV; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], CL * kEpiWarps / L::HV);
    }
    mbar_init(done, 1);
    if constexpr (SPLIT)
      for (int i = 0; i < kEpiWarps; ++i) mbar_init(&part_full[i], 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    if constexpr (CL == 1) {
      tmem_alloc(tmem_slot, L::TMEM_COLS);
      tmem_relinquish();
    } else {
      tmem_alloc_pair(tmem_slot, L::TMEM_COLS);
      tmem_relinquish_pair();
    }
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  // All of this overlaps the end of the kernel before this one, which every
  // role waits for before its first global access.
  if (warp == 0) {
    if constexpr (LORA == kRequests) {
      // the requests' bounds, in the place of the groups' units adapters (behind them
      // whether there are small requests), and which are done as products (behind
      // them their number).  Lone threads that went through all requests of a tile
      // took 100 clocks for each: 2100 rows, 63 requests without adapters 57 us.
      int row = min(max(__ldg(a.offsets), 0), a.rows_total), listed = 0;
      bool small = false;
      if (lane == 0) grow[0] = row;
      for (int base = 0; base < a.groups; base += 32) {
        const int i = base + lane;
        int hi = i < a.groups ? min(max(__ldg(a.offsets + i + 1), 0), a.rows_total) : 0;
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, hi, d);
          if (lane >= d) hi = max(hi, o);
        }
        hi = max(hi, row);
        int lo = __shfl_up_sync(0xffffffffu, hi, 1);
        if (lane == 0) lo = row;
        int who = -1;
        if (i < a.groups) {
          who = a.adapters ? __ldg(a.adapters + i) : i;
          if (who >= a.adapters_total) who = -1;
          grow[i + 1] = hi;
          gunit[i] = who;
        }
        const bool product = who >= 0 && hi - lo >= kLoraRows;
        const unsigned all = __ballot_sync(0xffffffffu, product);
        if (product) glist[listed + __popc(all & ((1u << lane) - 1u))] = i;
        listed += __popc(all);
        small = small || (who >= 0 && hi > lo && !product);
        row = __shfl_sync(0xffffffffu, hi, 31);
      }
      small = __any_sync(0xffffffffu, small);
      if (lane == 0) {
        gunit[a.groups] = small;
        glist[a.groups] = listed;
      }
    } else if (!a.offsets) {
      if (lane == 0) {
        grow[0] = 0;
        grow[1] = a.rows_total;
        gunit[0] = 0;
        gunit[1] = units_of(a.rows_total);
      }
    } else {
      // Row and unit ranges of the groups.  Offsets are clamped to
      // [0, rows_total] and made non-decreasing, so that no value of theirs
      // leads outside the operands.
      grid_dependency_wait();
      auto at = [&](int i) {
        return min(max(__ldg(a.offsets + i), 0), a.rows_total);
      };
      int row = at(0), unit = 0;
      if (lane == 0) {
        grow[0] = row;
        gunit[0] = 0;
      }
      for (int base = 0; base < a.groups; base += 32) {
        const int i = base + lane;
        int hi = i < a.groups ? at(i + 1) : 0;
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, hi, d);
          if (lane >= d) hi = max(hi, o);
        }
        hi = max(hi, row);
        int lo = __shfl_up_sync(0xffffffffu, hi, 1);
        if (lane == 0) lo = row;
        int n = i < a.groups ? units_of(hi - lo) : 0;
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, n, d);
          if (lane >= d) n += o;
        }
        if (i < a.groups) {
          grow[i + 1] = hi;
          gunit[i + 1] = unit + n;
        }
        row = __shfl_sync(0xffffffffu, hi, 31);
        unit += __shfl_sync(0xffffffffu, n, 31);
      }
    }
  }
  tc_fence_before();
  if constexpr (CL > 1 || SPLIT)
    cluster_sync();  // the others' barriers exist before anything targets them
  __syncthreads();
  tc_fence_after();
  grid_dependents_start();
  const uint32_t tmem_base = *tmem_slot;
  const int units = LORA == kRequests ? units_of(a.rows_total) : gunit[a.groups];
  const int first_unit = blockIdx.x / (CL * ksplit);
  const int unit_step = gridDim.x / (CL * ksplit);

  [[maybe_unused]] int split_k0 = 0, split_k1 = a.k_size;
  if (SPLIT && ksplit > 1) {
    // (at most 2^24 blocks of k times 6)
    const int blocks = (a.k_size + KE - 1) / KE;
    split_k0 = blocks * krank / ksplit * KE;
    split_k1 = min(blocks * (krank + 1) / ksplit * KE, a.k_size);
  }

  // Unit u: its group by bisection; within the group bands of kBand q tiles,
  // q fastest, so that what runs at one time shares few panels (with p
  // fastest a group's few q tiles read its P panels at different times:
  // grouped forward 181 us, so 176).
  auto decode = [&](int u) {
    int lo = 0, hi = LORA == kRequests ? 1 : a.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (gunit[mid] <= u) lo = mid; else hi = mid;
    }
    Tile t;
    t.e = lo;
    const int r = LORA == kRequests ? u : u - gunit[lo];
    const int g0 = LORA == kRequests ? 0 : grow[lo];
    const int g1 = LORA == kRequests ? a.rows_total : grow[lo + 1];
    const int np = ROWS ? (g1 - g0 + PT - 1) / PT : p_tiles;
    const int nq = RAGK || ROWS ? q_tiles : (g1 - g0 + BN - 1) / BN;
    // (divisions cost a lone thread some hundred clocks each)
    int pi = r, qi = 0;
    if (nq > 1) {
      const int band = nq > kBand ? r / (kBand * np) : 0;
      const int bq = min(nq - band * kBand, kBand);
      const int in = r - band * kBand * np;
      pi = in / bq;
      qi = band * kBand + in - pi * bq;
    }
    if constexpr (ROWS) {
      t.p0 = g0 + pi * PT;
      t.p1 = g1;
      t.q0 = qi * BN;
      t.q1 = min(t.q0 + BN, a.q_size);
    } else {
      t.p0 = pi * PT;
      t.p1 = a.p_size;
      // the rows are shared out evenly between the q tiles
      const int first = RAGK ? 0 : g0;
      const int rows = RAGK ? a.q_size : g1 - g0;
      const int share = nq > 1 ? (rows + nq - 1) / nq : rows;
      const int step = (share + QS - 1) / QS * QS;
      t.q0 = first + min(qi * step, rows);
      t.q1 = first + min(qi * step + step, rows);
    }
    t.nt = max((t.q1 - t.q0 + QS - 1) / QS * QS, QS);
    t.k0 = RAGK ? g0 : 0;
    t.k1 = RAGK ? g1 : a.k_size;
    if constexpr (SPLIT) {
      t.k0 = split_k0;
      t.k1 = split_k1;
    }
    return t;
  };

  // (kRequests) f(request, its first row, one past its last) for the requests done as
  // products that have rows in the tile.
  [[maybe_unused]] auto each_product = [&](const Tile& t, auto&& f) {
    const int n = glist[a.groups];
    int lo = 0, hi = n;  // the last that starts by the tile's start
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (grow[glist[mid]] <= t.q0) lo = mid; else hi = mid;
    }
    for (; lo < n; ++lo) {
      const int i = glist[lo];
      const int from = max(grow[i], t.q0), to = min(grow[i + 1], t.q1);
      if (from >= t.q1) break;
      if (to > from) f(i, from, to);
    }
  };
  [[maybe_unused]] const int lora_blocks = LORA == kRequests ? (a.rank + 63) / 64 : 0;

  if (warp < 4) {
  if constexpr (kSplitRegs) registers_give<kLoadRegs>();
  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      uint32_t cut_fills = 0;  // parity of the cut fills of each stage
      bool ok = !a.withhold;
      // the leader CTA's full barriers, which count both CTAs' bytes
      const uint32_t full_lead =
          CL > 1 ? mapa_shared(smem_u32(&full[0]), 0) : 0u;
      if constexpr (!LORA) grid_dependency_wait();
      for (int u = first_unit; u < units && ok; u += unit_step) {
        if (LORA && u != first_unit) grid_dependency_wait();
        const Tile t = decode(u);
        const int py = t.p0 + rank * kP;
        const int qy = t.q0 + rank * (t.nt / CL);
        for (int k = t.k0; k < t.k1; k += KE) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          uint8_t* sp = smem + stage * L::STAGE_BYTES;
          uint8_t* sq = sp + L::P_BYTES;
          // A pair's loads complete on the leader's barrier.  Those of a
          // block that a group ends in, inside a step of 16 (cut), complete
          // on a barrier of each CTA's own, where rows are cleared first.
          const bool cut = RAGK && t.k1 - k < KE && ((t.k1 - k) & 15);
          [[maybe_unused]] uint32_t bar = full_lead + uint32_t(stage) * 8u;
          if (cut) {
            if (rank == 0) mbar_arrive(&full[stage]);
            mbar_arrive_expect_tx(&cut_in[stage], L::STAGE_BYTES);
            if (CL > 1) bar = mapa_shared(smem_u32(&cut_in[stage]), rank);
            cut_fills ^= 1u << stage;
          } else if (rank == 0) {
            mbar_arrive_expect_tx(&full[stage], CL * L::STAGE_BYTES);
          }
          auto load = [&](const CUtensorMap* m, uint8_t* dst, int x, int y, int z) {
            if constexpr (CL > 1)
              tma_load_3d_pair(m, bar, dst, x, y, z);
            else
              tma_load_3d(m, cut ? &cut_in[stage] : &full[stage], dst, x, y, z);
          };
          const int zp = RAGK || ROWS ? 0 : t.e;
          const int zq = ROWS ? t.e : 0;
          if constexpr (P_MN) {
            for (int i = 0; i < kP / 64; ++i) load(&tmP, sp + i * 8192, py + 64 * i, k, zp);
          } else {
            load(&tmP, sp, k, py, zp);
          }
          if constexpr (Q_MN) {
            for (int i = 0; i < BN / CL / 64; ++i)
              load(&tmQ, sq + i * 8192, qy + 64 * i, k, zq);
          } else {
            // (each half's columns from the two CTAs of a pair in equal parts)
#pragma unroll
            for (int v = 0; v < HV; ++v) {
              const int nv = min(max(t.nt - v * HALF, 0), BN / HV);
              load(&tmQ, sq + v * QPART * 128, k, t.q0 + v * HALF + rank * (nv / CL), zq);
            }
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if constexpr (LORA == kRequests) {
          grid_dependency_wait();
          each_product(t, [&](int i, int, int) {
            for (int b = 0; b < lora_blocks * a.parts && ok; ++b) {
              if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.status)) {
                ok = false;
                return;
              }
              const int part = b / lora_blocks, k = (b - part * lora_blocks) * 64;
              uint8_t* sp = smem + stage * L::STAGE_BYTES;
              uint8_t* sq = sp + L::P_BYTES;
              if (rank == 0) mbar_arrive_expect_tx(&full[stage], CL * L::STAGE_BYTES);
              auto load = [&](const CUtensorMap* m, uint8_t* dst, int x, int y, int z) {
                if constexpr (CL > 1)
                  tma_load_3d_pair(m, full_lead + uint32_t(stage) * 8u, dst, x, y, z);
                else
                  tma_load_3d(m, &full[stage], dst, x, y, z);
              };
              if constexpr (P_MN) {
                for (int j = 0; j < kP / 64; ++j)
                  load(&tmZ.rows[0], sp + j * 8192, py + 64 * j, k, gunit[i]);
              } else {
                load(&tmZ.rows[0], sp, k, py, gunit[i]);
              }
              load(&tmD, sq, k, qy, part);
              ++issued;
              if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
              }
            }
          });
        }
      }
      for (int s = 0; s < STAGES; ++s) {
        const uint32_t fills = issued / STAGES + (uint32_t(s) < issued % STAGES);
        if (!fills) continue;
        // after an abort, let the loads in flight land before the CTA exits
        if (!ok && rank == 0) mbar_drain(&full[s], (fills - 1) & 1u, a.status);
        if (!ok && RAGK) mbar_drain(&cut_in[s], ~(cut_fills >> s) & 1u, a.status);
        // with a pair, the last release of each stage is the leader's
        // commit; wait until it has arrived on this CTA
        if (CL > 1) mbar_drain(&empty[s], (fills - 1) & 1u, a.status);
      }
    }
    __syncwarp();
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------ MMA issuer
    // One thread.  Issuing waits for room in the tensor pipe, so the next
    // stage's barrier is looked at before the last MMA of a stage is issued.
    if (elect_one()) {
      // (touches no memory, but its bounded waits are not to run while the
      // kernel before does)
      if constexpr (!LORA) grid_dependency_wait();
      int stage = 0;
      uint32_t phase = 0, acc_phase = 0;
      [[maybe_unused]] uint32_t cut_phase = 0;  // one bit per stage
      int acc = 0;
      bool ok = true, ready = false;
      const uint32_t s0 = smem_u32(smem);
      const uint64_t dp0 = P_MN ? sw128_mnmajor_desc(s0) : sw128_kmajor_desc(s0);
      const uint64_t dq0 = Q_MN ? sw128_mnmajor_desc(s0 + L::P_BYTES)
                                : sw128_kmajor_desc(s0 + L::P_BYTES);
      // 32 bytes of a row (K-major) or 16 rows (MN-major) per step
      constexpr uint32_t kStepP = P_MN ? 128 : 2;
      constexpr uint32_t kStepQ = Q_MN ? 128 : 2;
      for (int u = first_unit; u < units && ok; u += unit_step) {
        if (LORA && u != first_unit) grid_dependency_wait();
        const Tile t = decode(u);
        const uint32_t idesc = a.idesc | (uint32_t(t.nt >> 3) << 17);
        int left = t.k1 - t.k0;  // k still to be issued
        while (left > 0 && ok) {
          if constexpr (HV == 2) {
            // one block of k per chunk, in halves of the columns
            if (!ready) ok = mbar_wait(&full[stage], phase, abort_flag, a.status);
            if (!ok) break;
            const uint64_t dp = dp0 + uint32_t(stage * (L::STAGE_BYTES >> 4));
            const uint64_t dq = dq0 + uint32_t(stage * (L::STAGE_BYTES >> 4));
            uint64_t* const done_with = &empty[stage];
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              ok = mbar_wait(&tempty[acc * 2 + v], acc_phase ^ 1u, abort_flag, a.status);
              if (!ok) break;
              tc_fence_after();
              const int nv = min(max(t.nt - v * HALF, 0), HALF);
              const uint32_t id = a.idesc | (uint32_t(nv >> 3) << 17);
              const uint32_t d_tmem = tmem_base + uint32_t(acc * BN + v * HALF);
#pragma unroll
              for (int s = 0; s < 4; ++s) {
                if (v == 1 && s == 3) ready = mbar_test(&full[stage], phase);
                if (nv > 0)
                  umma_f8<CL>(d_tmem, dp + s * kStepP,
                              dq + uint32_t(v * QPART * 8) + s * kStepQ, id, s > 0);
              }
              if (v == 1) umma_commit_pair(done_with, 3u);
              umma_commit_pair(&tfull[acc * 2 + v], 3u);
            }
            if (!ok) break;
            left -= KE;
          } else {
          ok = mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + uint32_t(acc * BN);
          uint32_t accum = 0;
          for (int i = a.kb_per_chunk; i > 0 && left > 0; --i) {
            if (!ready) ok = mbar_wait(&full[stage], phase, abort_flag, a.status);
            int steps = 4;
            if constexpr (RAGK) {
              if (ok && left < KE) {
                steps = (left + 15) >> 4;
                if (left & 15) {
                  ok = mbar_wait(&cut_ok[stage], (cut_phase >> stage) & 1u, abort_flag,
                                 a.status);
                  cut_phase ^= 1u << stage;
                }
              }
            }
            if (!ok) break;
            tc_fence_after();
            // (the start address is the low bits of a descriptor)
            const uint64_t dp = dp0 + uint32_t(stage * (L::STAGE_BYTES >> 4));
            const uint64_t dq = dq0 + uint32_t(stage * (L::STAGE_BYTES >> 4));
            uint64_t* const done_with = &empty[stage];
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              if (s == 3) ready = mbar_test(&full[stage], phase);
              if (RAGK && s >= steps) continue;
              if constexpr (KIND8)
                umma_f8<CL>(d_tmem, dp + s * kStepP, dq + s * kStepQ, idesc, accum);
              else if constexpr (CL == 1)
                umma_f16(d_tmem, dp + s * kStepP, dq + s * kStepQ, idesc, accum);
              else
                umma_f16_pair(d_tmem, dp + s * kStepP, dq + s * kStepQ, idesc, accum);
              accum = 1;
            }
            if constexpr (CL == 1)
              umma_commit(done_with);
            else
              umma_commit_pair(done_with, 3u);
            left -= KE;
          }
          if (!ok) break;
          if constexpr (CL == 1)
            umma_commit(&tfull[acc]);
          else
            umma_commit_pair(&tfull[acc], 3u);
          }
          if (++acc == L::ACCS) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
        if constexpr (LORA == kRequests) {
          grid_dependency_wait();
          each_product(t, [&](int, int, int) {
            if (!ok) return;
            ok = mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag, a.status);
            if (!ok) return;
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + uint32_t(acc * BN);
            uint32_t accum = 0;
            for (int b = 0; b < lora_blocks * a.parts; ++b) {
              if (!ready) ok = mbar_wait(&full[stage], phase, abort_flag, a.status);
              if (!ok) return;
              ready = false;
              tc_fence_after();
              const uint64_t dp = dp0 + uint32_t(stage * (L::STAGE_BYTES >> 4));
              const uint64_t dq = dq0 + uint32_t(stage * (L::STAGE_BYTES >> 4));
              // (past the rank both operands are zeros)
              const int steps = min((a.rank - b % lora_blocks * 64 + 15) / 16, 4);
              for (int s = 0; s < steps; ++s) {
                if constexpr (CL == 1)
                  umma_f16(d_tmem, dp + s * kStepP, dq + s * kStepQ, idesc, accum);
                else
                  umma_f16_pair(d_tmem, dp + s * kStepP, dq + s * kStepQ, idesc, accum);
                accum = 1;
              }
              if constexpr (CL == 1)
                umma_commit(&empty[stage]);
              else
                umma_commit_pair(&empty[stage], 3u);
              if (++stage == STAGES) {
                stage = 0;
                phase ^= 1u;
              }
            }
            if constexpr (CL == 1)
              umma_commit(&tfull[acc]);
            else
              umma_commit_pair(&tfull[acc], 3u);
            if (++acc == L::ACCS) {
              acc = 0;
              acc_phase ^= 1u;
            }
          });
        }
      }
      // Every MMA issued above completes before tensor memory is released.
      if constexpr (CL == 1)
        umma_commit(done);
      else
        umma_commit_pair(done, 1u);
      mbar_drain(done, 0, a.status);
    }
    __syncwarp();
  } else if (RAGK && warp == 2) {
    // ------------------------------------------------ cut blocks
    // A group that ends inside a step of 16: the step's other rows are the
    // next group's and become zeros in both operands (in one alone, an
    // infinity in the other would leave NaN).  The zeros are TMA loads of
    // rows beyond a tensor's end (8, 4, 2 or 1 rows of a 64-wide box), issued
    // when the block has landed; both CTAs' complete on the leader's barrier.
    // (Zeros written by the warps had to be released to the other CTA, which
    // took some 1200 clocks per tile: 32 groups of 500 tokens 317 us, of 512
    // tokens 276.)
    int stage = 0;
    uint32_t cut_phase = 0;  // one bit per stage
    bool ok = true;
    grid_dependency_wait();  // (as the MMA issuer)
    const uint32_t cut_lead = mapa_shared(smem_u32(&cut_ok[0]), CL > 1 ? 0 : cluster_ctarank());
    for (int u = first_unit; u < units; u += unit_step) {
      const Tile t = decode(u);
      const int blocks = (t.k1 - t.k0 + KE - 1) / KE;
      const int left = (t.k1 - t.k0) - (blocks - 1) * KE;
      if (blocks > 0 && left < KE && (left & 15)) {
        constexpr int kBoxes = (kP + BN / CL) / 64;
        const int s = (stage + blocks - 1) % STAGES;
        const int n = 16 - (left & 15);  // rows to clear
        ok = mbar_wait(&cut_in[s], (cut_phase >> s) & 1u, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        cut_phase ^= 1u << s;
        if (rank == 0 && lane == 0)
          mbar_arrive_expect_tx(&cut_ok[s], uint32_t(CL * kBoxes * n * 128));
        __syncwarp();
        // lane: which power of two of n, which box
        const int e = lane / kBoxes;
        if (e < 4 && ((n >> e) & 1)) {
          const int row = left + (n & ((1 << e) - 1));
          uint8_t* dst = smem + s * L::STAGE_BYTES + lane % kBoxes * 8192 + row * 128;
          if constexpr (CL > 1)
            tma_load_3d_pair(&tmZ.rows[e], cut_lead + uint32_t(s) * 8u, dst, 0,
                             a.rows_total, 0);
          else
            tma_load_3d(&tmZ.rows[e], &cut_ok[s], dst, 0, a.rows_total, 0);
        }
        __syncwarp();
      }
      stage = (stage + blocks) % STAGES;
    }
    // after an abort, let the zeros in flight land
    if (rank == 0 && lane == 0 && *abort_flag)
      for (int s = 0; s < STAGES; ++s)
        mbar_drain(&cut_ok[s], ~(cut_phase >> s) & 1u, a.status);
    __syncwarp();
  } else if (KIND8 && warp == 3) {
    // ------------------------------------------------ scales
    // Those of each chunk (one k block) by cp.async into a ring, zero beyond
    // the operands; every lane's copies count as one arrival.
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    const float* ring = reinterpret_cast<const float*>(smem + L::SCALE_OFFSET);
    grid_dependency_wait();
    for (int u = first_unit; u < units && ok; u += unit_step) {
      const Tile t = decode(u);
      constexpr int NP = kP / 32, NQ = ROWS ? 1 : BN / 32;
      // 32 rows per copy; with one scale per 128 rows all of P has one
      const int p0 = t.p0 + rank * kP + lane;
      const int q0 = ROWS ? t.q0 + lane * 128 : t.q0 + lane;
      const float* src_p = a.sp + (ROWS ? 0 : t.e * a.sp_group) +
                           (int64_t(p0) >> a.p_shift) * a.sp_row + (t.k0 / KE) * a.sp_blk;
      const float* src_q = a.sq + (ROWS ? t.e * a.sq_group : 0) +
                           (int64_t(q0) >> a.q_shift) * a.sq_row + (t.k0 / KE) * a.sq_blk;
      const int64_t step_p = a.p_shift ? 0 : 32 * a.sp_row, step_q = 32 * a.sq_row;
      const int chunks = (t.k1 - t.k0 + KE - 1) / KE;
      for (int ch = 0; ch < chunks; ch += L::G) {
        ok = mbar_wait(&sempty[slot], phase ^ 1u, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        uint32_t dst = smem_u32(ring + slot * L::SLOT_FLOATS);
        for (int g = 0; g < L::G && ch + g < chunks; ++g, dst += L::CHUNK_FLOATS * 4) {
          // (beyond the operand nothing is read, and zero is written)
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const bool in = p0 + i * 32 < t.p1;
            cp_async_4_zfill(dst + (i * 32 + lane) * 4, in ? src_p + i * step_p : a.sp, in * 4);
          }
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            const bool in = q0 + i * 32 < t.q1;
            if (!ROWS || lane < 2)
              cp_async_4_zfill(dst + (kP + i * 32 + lane) * 4,
                               in ? src_q + i * step_q : a.sq, in * 4);
          }
          src_p += a.sp_blk;
          src_q += a.sq_blk;
        }
        cp_async_mbar_arrive(&sfull[slot]);
        if (++slot == L::SLOTS) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    cp_async_commit();
    cp_async_wait<0>();  // none is in flight when the CTA ends
  }
  } else {
    // ------------------------------------------------ epilogue warps
    // A warp owns 32 rows of P (its tensor-memory lane quarter) and, of the
    // columns, its half (ROWS, halves) or every other block of CB.
    if constexpr (kSplitRegs) registers_take<kEpiRegs>();
    const int ew = warp - 4;
    const int quarter = warp & 3;
    const int h = ew >> 2;
    // PAIRS: a lane has two columns out of eight of four rows, so that it
    // needs a quarter of the columns' scales, and in pairs (2048 x 4096 x 8200
    // with C: one row per lane and all scales as broadcasts out of shared
    // memory 127 us, pairs 104, with packed arithmetic 96).
    constexpr bool PAIRS = KIND8 && !ROWS && BN == 256;
    [[maybe_unused]] const int pair_q = h * HALF + 2 * (lane & 3);
    auto column = [&](int i) {
      return ROWS || HV == 2 ? h * HALF + i * CB : (2 * i + h) * CB;
    };
    [[maybe_unused]] float* wbuf =
        reinterpret_cast<float*>(smem + L::WARP_OFFSET + ew * L::WARP_BYTES);
    [[maybe_unused]] const float* ring =
        reinterpret_cast<const float*>(smem + L::SCALE_OFFSET);
    [[maybe_unused]] uint32_t fills = 0;  // slots taken so far
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    // the issuing CTA's barriers that hand the accumulators back
    const uint32_t tempty_lead =
        mapa_shared(smem_u32(&tempty[0]), CL > 1 ? 0 : cluster_ctarank());
    [[maybe_unused]] int block = 0;  // of the ring of blocks of D
    if constexpr (!LORA) grid_dependency_wait();
    [[maybe_unused]] const int part_at =
        L::part_offset(a.groups) + (quarter * 32 + lane) * 4;
    for (int u = first_unit; u < units && ok; u += unit_step) {
      __syncwarp();
      if (LORA && u != first_unit) grid_dependency_wait();
      const Tile t = decode(u);
      const int pw = t.p0 + rank * kP + quarter * 32;
      const int p = pw + lane;
      float sum[HALF];
      if constexpr (PAIRS) {
        // (as below)
        const int left = t.q1 - t.q0 - pair_q;
        const int64_t ci = int64_t(t.q0 + pair_q) * a.ldc + pw + (lane >> 2);
        auto start = [&](auto read) {
#pragma unroll
          for (int s = 0; s < HALF; ++s) {
            const int q = pairs_q(s), r = pairs_row(s);
            sum[s] = a.C && q < left && pw + (lane >> 2) + r < t.p1
                         ? read(ci + q * a.ldc + r)
                         : 0.f;
          }
        };
        if (a.d_type == MMA_F32)
          start([&](int64_t i) { return static_cast<const float*>(a.C)[i]; });
        else
          start([&](int64_t i) { return load_c(a.C, i, a.d_type); });
      } else if (!ROWS && a.C && krank == 0 && p < t.p1) {
        // The sums start from C, all of whose loads are under way at once
        // (and land while the first chunks are computed).
        const int64_t ci = (RAGK ? t.e * a.c_group : 0) + int64_t(t.q0) * a.ldc + p;
        auto start = [&](auto read) {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            int64_t at = ci + column(i) * a.ldc;
            const int left = t.q1 - t.q0 - column(i);
#pragma unroll
            for (int j = 0; j < CB; ++j, at += a.ldc)
              sum[i * CB + j] = j < left ? read(at) : 0.f;
          }
        };
        if (a.d_type == MMA_F32)
          start([&](int64_t i) { return static_cast<const float*>(a.C)[i]; });
        else
          start([&](int64_t i) { return load_c(a.C, i, a.d_type); });
      } else {
#pragma unroll
        for (int j = 0; j < HALF; ++j) sum[j] = 0.f;
      }
      __syncwarp();
      const int num_kb = (t.k1 - t.k0 + KE - 1) / KE;
      const int chunks = (num_kb + a.kb_per_chunk - 1) / a.kb_per_chunk;
      // Wait for a chunk's sums in tensor memory, add them (through `add`,
      // for each block of columns) and return the accumulator as soon as its
      // last block is in registers.  Scalar additions (but for PAIRS) and one
      // block in flight: packed ones and a second block spill sums (8192 x
      // 8192 x 4096 with square scales 209 us, packed 235, 16 columns at a time
      // with the next ones on their way 235).  Of a tile of 256
      // columns all are added, those beyond nt to sums that are not stored:
      // asking cost more (8-bit with row scales 139 us, without 119).
      auto take = [&](auto&& add) {
        const int ah = HV == 2 ? acc * 2 + h : acc;
        mbar_wait_lean(&tfull[ah], acc_phase, abort_flag, a.status);
        tc_fence_after();
        const uint32_t taddr =
            tmem_base + uint32_t(acc * BN) + (uint32_t(quarter * 32) << 16);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const bool in = BN == 256 || column(i) < t.nt;
          uint32_t r[CB];
          if (in) {
            if constexpr (PAIRS) {
              tmem_ld_16x256b_x4(taddr + column(i), r);
              tmem_ld_16x256b_x4(taddr + column(i) + (16u << 16), r + 16);
            } else if constexpr (CB == 32) {
              tmem_ld_32x32b_x32(taddr + column(i), r);
            } else {
              tmem_ld_32x32b_x16(taddr + column(i), r);
            }
            tmem_ld_wait();
          }
          if (i + 1 == NB) {
            tc_fence_before();
            __syncwarp();
            mbar_arrive_remote_if(tempty_lead + uint32_t(ah) * 8u, lane == 0);
          }
          if (in) add(i, r);
        }
        acc = (acc + 1) % L::ACCS;
        acc_phase ^= acc == 0;
      };
      if constexpr (!KIND8) {
        for (int ch = 0; ch < chunks; ++ch)
          take([&](int i, const uint32_t (&r)[CB]) {
#pragma unroll
            for (int j = 0; j < CB; ++j) sum[i * CB + j] += __uint_as_float(r[j]);
          });
        if constexpr (LORA == kRequests) {
          grid_dependency_wait();
          // (lane l has the scales of column l of each block)
          static_assert(LORA != kRequests || CB == 32);
          float down[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int64_t q = min(t.q0 + column(b) + lane, a.rows_total - 1);
            down[b] = a.up ? down_of(a.up[q * a.ld_up]) : 1.f;
          }
          each_product(t, [&](int, int from, int to) {
            // (what other rows' sums with this adapter are does not matter)
            take([&](int b, const uint32_t (&r)[CB]) {
              const int first = t.q0 + column(b) - from;
#pragma unroll
              for (int j = 0; j < CB; ++j) {
                const float d = __shfl_sync(0xffffffffu, down[b], j);
                if (unsigned(first + j) < unsigned(to - from))
                  sum[b * CB + j] = fmaf(__uint_as_float(r[j]), d, sum[b * CB + j]);
              }
            });
          });
          // The rows of small requests: lane l has the place in `extra` of column l
          // of each block, or -1.  (One row after the other, each added to the sum
          // that a comparison picks, was 128 comparisons a row: 2100 rows, 60 of them
          // small, 123 us where 83 were taken in all.)
          int slot[NB], lo[NB];
          bool some = false;
          if (gunit[a.groups]) {
#pragma unroll
            for (int b = 0; b < NB; ++b) lo[b] = 0;
            // (the blocks' bisections side by side)
            for (int step = 512; step > 0; step >>= 1) {
              if (step >= a.groups) continue;
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                const int mid = lo[b] + step;
                if (mid < a.groups && grow[mid] <= t.q0 + column(b) + lane) lo[b] = mid;
              }
            }
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            slot[b] = -1;
            if (!gunit[a.groups]) continue;
            const int q = t.q0 + column(b) + lane, i = lo[b];
            if (lane < CB && q < t.q1 && q >= grow[i] && q < grow[i + 1] && gunit[i] >= 0 &&
                grow[i + 1] - grow[i] < kLoraRows)
              slot[b] = lora_own_places(a.rows_total, a.groups)
                            ? q
                            : i * (kLoraRows - 1) + q - grow[i];
            some = some || slot[b] >= 0;
          }
          if (__any_sync(0xffffffffu, some)) {
            const float* e = a.extra + min(p, t.p1 - 1);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const unsigned which = __ballot_sync(0xffffffffu, slot[b] >= 0);
#pragma unroll
              for (int j = 0; j < CB; j += 8) {
                if (!((which >> j) & 255u)) continue;
                float v[8];  // (their loads together)
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  const int r = __shfl_sync(0xffffffffu, slot[b], j + x);
                  v[x] = r >= 0 ? e[int64_t(r) * a.p_size] : 0.f;
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) sum[b * CB + j + x] += v[x];
              }
            }
          }
        }
      } else {
        static_assert(L::SLOTS == 2);
#pragma unroll 1
        for (int left = chunks; left > 0; left -= L::G, ++fills) {
          mbar_wait_lean(&sfull[fills & 1], (fills >> 1) & 1, abort_flag, a.status);
          const float* sc = ring + (fills & 1) * L::SLOT_FLOATS;
#pragma unroll 1
          for (int g = min(L::G, left); g > 0; --g) {
            [[maybe_unused]] float sp, spr[4];
            if constexpr (PAIRS) {
#pragma unroll
              for (int x = 0; x < 4; ++x) spr[x] = sc[quarter * 32 + (lane >> 2) + 8 * x];
            } else {
              sp = ROWS ? sc[quarter * 32 + lane] * sc[kP + h] : sc[quarter * 32 + lane];
            }
            take([&](int i, const uint32_t (&r)[CB]) {
              if constexpr (PAIRS) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const float2 v =
                      *reinterpret_cast<const float2*>(sc + kP + pair_q + i * 32 + x * 8);
#pragma unroll
                  for (int y = 0; y < 8; y += 2) {
                    const int j = (y >> 2) * 16 + x * 4 + (y & 3);
                    const float sp1 = spr[pairs_row(j) / 8];
                    float* const s = sum + i * CB + j;
                    const float2 d = __ffma2_rn(
                        __fmul2_rn(v, make_float2(sp1, sp1)),
                        make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                        make_float2(s[0], s[1]));
                    s[0] = d.x;
                    s[1] = d.y;
                  }
                }
              } else if constexpr (ROWS) {
#pragma unroll
                for (int j = 0; j < CB; ++j)
                  sum[i * CB + j] = fmaf(sp, __uint_as_float(r[j]), sum[i * CB + j]);
              } else {
#pragma unroll
                for (int j = 0; j < CB; j += 4) {
                  const float4 v =
                      *reinterpret_cast<const float4*>(sc + kP + column(i) + j);
                  float* const s = sum + i * CB + j;
                  s[0] = fmaf(v.x * sp, __uint_as_float(r[j]), s[0]);
                  s[1] = fmaf(v.y * sp, __uint_as_float(r[j + 1]), s[1]);
                  s[2] = fmaf(v.z * sp, __uint_as_float(r[j + 2]), s[2]);
                  s[3] = fmaf(v.w * sp, __uint_as_float(r[j + 3]), s[3]);
                }
              }
            });
            sc += L::CHUNK_FLOATS;
          }
          __syncwarp();
          mbar_arrive_if(&sempty[fills & 1], lane == 0);
        }
      }
      ok = !__any_sync(0xffffffffu, *abort_flag != 0);
      // (SPLIT, lane 0 of rank 0) await this warp's columns of the other ranks'
      [[maybe_unused]] auto expect_parts = [&] {
        int mine = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) mine += min(max(t.q1 - t.q0 - column(i), 0), CB);
        mbar_arrive_expect_tx(&part_full[ew], uint32_t((ksplit - 1) * mine * 128));
      };
      if (!ok) {
        // after an abort, let the sums that other ranks still send land
        if (SPLIT && ksplit > 1 && krank == 0 && lane == 0) {
          expect_parts();
          mbar_drain(&part_full[ew], 0, a.status);
        }
        break;
      }
      if constexpr (SPLIT) {
        if (ksplit > 1) {
          // Only the columns that hold rows of D travel, as stores that
          // complete on rank 0's barrier: no release, no arrival.  (The launch
          // has a cluster for every tile there can be, so that a cluster takes
          // one at most and the room for the sums is used once.)
          const int cols = t.q1 - t.q0;
          if (krank > 0) {
            const uint32_t dst = mapa_shared(
                smem_u32(smem + part_at + (krank - 1) * a.part_cols * kP * 4), 0);
            const uint32_t bar = mapa_shared(smem_u32(&part_full[ew]), 0);
#pragma unroll
            for (int j = 0; j < HALF; ++j)
              if (const int c = column(j / CB) + j % CB; c < cols)
                st_async_f32(dst + c * kP * 4, sum[j], bar);
            continue;
          }
          if (lane == 0) expect_parts();
          const bool got =
              mbar_wait_cluster(&part_full[ew], 0, abort_flag, a.status);
          if (!__all_sync(0xffffffffu, got)) {
            if (lane == 0) mbar_drain(&part_full[ew], 0, a.status);
            break;
          }
          for (int r = 1; r < ksplit; ++r) {
            const float* src = reinterpret_cast<const float*>(
                smem + part_at + (r - 1) * a.part_cols * kP * 4);
#pragma unroll
            for (int j = 0; j < HALF; ++j)
              if (const int c = column(j / CB) + j % CB; c < cols) sum[j] += src[c * kP];
          }
        }
      }
      if constexpr (ROWS) {
        if (a.d_tma && pw + 32 <= t.p1) {
          // Blocks of 64 bytes of the warp's rows leave by TMA, which has the
          // whole next tile's time to move them (stored by the warps they
          // held up the MMAs: 8192 x 8192 x 4096 257 us, so 228).
          const bool wide = a.d_type == MMA_F32, bf16 = a.d_type == MMA_BF16;
          auto send = [&](int c, const uint4 (&w)[4], int cols) {
            const int q = t.q0 + h * HALF + c * cols;
            if (q >= t.q1) return;
            uint8_t* buf = reinterpret_cast<uint8_t*>(wbuf) + block * 2048;
            if (++block == L::BLOCKS) block = 0;
            if (lane == 0) bulk_wait_group_read<L::BLOCKS - 1>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(buf + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = w[j];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&tmD, buf, q, pw, 0);
              bulk_commit_group();
            }
          };
          if (wide) {
#pragma unroll
            for (int c = 0; c < HALF / 16; ++c) {
              uint4 w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float* const s = sum + c * 16 + 4 * j;
                w[j] = make_uint4(__float_as_uint(s[0]), __float_as_uint(s[1]),
                                  __float_as_uint(s[2]), __float_as_uint(s[3]));
              }
              send(c, w, 16);
            }
          } else {
#pragma unroll
            for (int c = 0; c < HALF / 32; ++c) {
              uint4 w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float* const s = sum + c * 32 + 8 * j;
                w[j] = make_uint4(pack16(s[0], s[1], bf16), pack16(s[2], s[3], bf16),
                                  pack16(s[4], s[5], bf16), pack16(s[6], s[7], bf16));
              }
              send(c, w, 32);
            }
          }
          continue;
        }
        // by the warp, through the ring's first block
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
        block = 0;
        if (a.vec8) {
          // 16-bit D without C: 32 columns at a time, rounded, through
          // shared memory, so that four lanes store 64 bytes of a row and a
          // warp eight rows
          const bool bf16 = a.d_type == MMA_BF16;
#pragma unroll
          for (int c = 0; c < HALF / 32; ++c) {
            const int q = t.q0 + h * HALF + c * 32;
            if (q >= t.q1) continue;
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = pack16(sum[c * 32 + j * 8 + 2 * x], sum[c * 32 + j * 8 + 2 * x + 1], bf16);
              *reinterpret_cast<uint4*>(wbuf + lane * 16 +
                                        ((j ^ ((lane >> 1) & 3)) << 2)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
            const int j = lane & 3;
            const int col = q + 8 * j;
            uint16_t* d = static_cast<uint16_t*>(a.D) + int64_t(pw) * a.ldd + col;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = i * 8 + (lane >> 2);
              const uint4 v = *reinterpret_cast<const uint4*>(
                  wbuf + r * 16 + ((j ^ ((r >> 1) & 3)) << 2));
              if (pw + r >= t.p1 || col >= t.q1) continue;
              if (col + 8 <= t.q1) {
                *reinterpret_cast<uint4*>(d + r * a.ldd) = v;
              } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int x = 0; x < 7; ++x)
                  if (col + x < t.q1)
                    d[r * a.ldd + x] = uint16_t(w[x >> 1] >> (16 * (x & 1)));
              }
            }
          }
          continue;
        }
        // 16 columns at a time through shared memory, so that four lanes
        // store one row's 16 columns and a warp eight rows
#pragma unroll
        for (int c = 0; c < HALF / 16; ++c) {
          const int q = t.q0 + h * HALF + c * 16;
          if (q >= t.q1) continue;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float* const s = sum + c * 16 + 4 * j;
            *reinterpret_cast<float4*>(wbuf + lane * 16 +
                                       ((j ^ ((lane >> 1) & 3)) << 2)) =
                make_float4(s[0], s[1], s[2], s[3]);
          }
          __syncwarp();
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int r = i * 8 + (lane >> 2), j = lane & 3;
            float4 v = *reinterpret_cast<const float4*>(
                wbuf + r * 16 + ((j ^ ((r >> 1) & 3)) << 2));
            const int col = q + 4 * j;
            if (pw + r >= t.p1 || col >= t.q1) continue;
            const int64_t di = int64_t(pw + r) * a.ldd + col;
            const int64_t ci = int64_t(pw + r) * a.ldc + col;
            if (a.vec4 && col + 4 <= t.q1) {
              if (a.C) {
                const float4 w = load_c4(a.C, ci, a.d_type);
                v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
              }
              store_d4(a.D, di, a.d_type, v);
            } else {
#pragma unroll 1
              for (int x = 0; x < 4 && col + x < t.q1; ++x) {
                const float f = x == 0 ? v.x : x == 1 ? v.y : x == 2 ? v.z : v.w;
                store_d(a.D, di + x, a.d_type,
                        f + (a.C ? load_c(a.C, ci + x, a.d_type) : 0.f));
              }
            }
          }
        }
      } else if constexpr (PAIRS) {
        // (each store instruction: 8 consecutive p of 4 rows of D)
        const int left = t.q1 - t.q0 - pair_q;
        const int rows = t.p1 - pw - (lane >> 2);
        const int64_t di = int64_t(t.q0 + pair_q) * a.ldd + pw + (lane >> 2);
        if (a.d_type == MMA_F32) {
          float* d = static_cast<float*>(a.D) + di;
#pragma unroll
          for (int s = 0; s < HALF; ++s)
            if (pairs_q(s) < left && pairs_row(s) < rows)
              d[pairs_q(s) * a.ldd + pairs_row(s)] = sum[s];
        } else {
          uint16_t* d = static_cast<uint16_t*>(a.D) + di;
          const bool bf16 = a.d_type == MMA_BF16;
#pragma unroll
          for (int s = 0; s < HALF; ++s)
            if (pairs_q(s) < left && pairs_row(s) < rows)
              d[pairs_q(s) * a.ldd + pairs_row(s)] = uint16_t(pack16(sum[s], 0.f, bf16));
        }
      } else {
        if constexpr (LORA) grid_dependency_wait();
        if (p >= t.p1) continue;
        if constexpr (LORA == kEveryRow) {
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const float* e = a.extra + int64_t(t.q0 + column(i)) * a.p_size + p;
            const int left = t.q1 - t.q0 - column(i);
            float v[CB];
#pragma unroll
            for (int j = 0; j < CB; ++j) v[j] = j < left ? e[int64_t(j) * a.p_size] : 0.f;
#pragma unroll
            for (int j = 0; j < CB; ++j) sum[i * CB + j] += v[j];
          }
        }
        const int64_t group = RAGK ? t.e : 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int q = t.q0 + column(i);
          if (q >= t.q1) continue;
          int64_t di = group * a.d_group + int64_t(q) * a.ldd + p;
          const int left = t.q1 - q;
          if (a.d_type == MMA_F32) {
            float* d = static_cast<float*>(a.D) + di;
#pragma unroll
            for (int j = 0; j < CB; ++j, d += a.ldd)
              if (j < left) *d = sum[i * CB + j];
          } else {
            uint16_t* d = static_cast<uint16_t*>(a.D) + di;
            const bool bf16 = a.d_type == MMA_BF16;
#pragma unroll
            for (int j = 0; j < CB; ++j, d += a.ldd)
              if (j < left) *d = uint16_t(pack16(sum[i * CB + j], 0.f, bf16));
          }
        }
      }
    }
  }
  if (ROWS && warp >= 4 && lane == 0) bulk_wait_group<0>();  // D is written
  tc_fence_before();
  if (CL > 1 || ksplit > 1)
    cluster_sync();  // no CTA leaves while another may still signal it
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if constexpr (CL == 1)
      tmem_dealloc(tmem_base, L::TMEM_COLS);
    else
      tmem_dealloc_pair(tmem_base, L::TMEM_COLS);
  }
}

// ----------------------------------------------------------------- host

// An operand: K-major (rows of k) or MN-major (k rows), `rows` of them in a
// slice, `slices` slices.
struct Operand {
  const void* p;
  int64_t ld, rows, slices, slice;
};

// The operands of a product with adapters: their second matrices, by row of P or
// (MN-major) by sum, and the rows' sums in 16 bits.
struct LoraMaps {
  Operand up, low;
};

template <bool KIND8, bool P_MN, bool Q_MN, bool RAGK, bool ROWS, bool SPLIT, int CL,
          int BN, int STAGES, Lora LORA = kNoLora>
mma_status_t run(const Ctx& ctx, const Operand& P, const Operand& Q,
                 const GroupedArgs& args, const LoraMaps* lora = nullptr) {
  using L = Layout<KIND8, ROWS, SPLIT, CL, BN, STAGES>;
  constexpr int EB = KIND8 ? 1 : 2;
  constexpr int KE = KIND8 ? 128 : 64;
  constexpr int PT = kP * CL;
  const int64_t p_tiles = (args.p_size + PT - 1) / PT;
  const int64_t q_tiles = (args.q_size + BN - 1) / BN;
  // an upper bound of the units, whatever the offsets: a group with n rows
  // has at most n tiles' rows of them, and full tiles besides one
  auto tiles_of = [&](int64_t rows, int64_t per) {
    return args.offsets && LORA != kRequests
               ? std::min<int64_t>(rows, rows / per + args.groups)
               : (rows + per - 1) / per;
  };
  const int64_t most = RAGK   ? args.groups * q_tiles * p_tiles
                       : ROWS ? tiles_of(args.rows_total, PT) * q_tiles
                              : tiles_of(args.rows_total, BN) * p_tiles;
  // rows and k are ints on the device, a tile past the end included
  constexpr int kMost = INT32_MAX - 1024;
  if (most > int64_t(INT32_MAX) / 2 || args.p_size > kMost || args.q_size > kMost ||
      args.k_size > kMost || args.rows_total > kMost)
    return MMA_ERR_UNSUPPORTED;
  auto map_of = [&](CUtensorMap* m, const Operand& o, bool mn, int64_t len, int box) {
    // no k at all (D = C): the kernel loads nothing but wants a valid map
    if (args.k_size == 0)
      return make_map(m, reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(args.D) &
                                                 ~uintptr_t(15)),
                      EB, 64, 1, 64, 1, 64, 64, 1);
    const int64_t slice = o.slices > 1 ? o.slice : o.ld;  // unused when 1
    return mn ? make_map(m, o.p, EB, len, o.rows, o.ld, o.slices, slice, 64, 64)
              : make_map(m, o.p, EB, args.k_size, o.rows, o.ld, o.slices, slice, KE, box);
  };
  CUtensorMap tp, tq, td;
  ZeroMaps tz;
  if (!map_of(&tp, P, P_MN, args.p_size, kP) || !map_of(&tq, Q, Q_MN, args.q_size, BN / CL / L::HV))
    return MMA_ERR_LAUNCH;
  GroupedArgs a = args;
  td = tp;
  if constexpr (LORA == kRequests) {
    const Operand &u = lora->up, &l = lora->low;
    if (!(P_MN ? make_map(&tz.rows[0], u.p, EB, args.p_size, args.rank, u.ld, u.slices,
                          u.slices > 1 ? u.slice : u.ld, 64, 64)
               : make_map(&tz.rows[0], u.p, EB, args.rank, u.rows, u.ld, u.slices,
                          u.slices > 1 ? u.slice : u.ld, KE, kP)) ||
        !make_map(&td, l.p, EB, args.rank, l.rows, l.ld, l.slices, l.slice, KE, BN / CL))
      return MMA_ERR_LAUNCH;
  }
  for (int e = LORA == kRequests ? 1 : 0; e < 4; ++e) {
    tz.rows[e] = tp;  // (read beyond their end only)
    if (RAGK && args.k_size > 0 &&
        !make_map(&tz.rows[e], P.p, EB, args.p_size, P.rows, P.ld, 1, P.ld, 64, 1 << e,
                  CU_TENSOR_MAP_SWIZZLE_NONE))
      return MMA_ERR_LAUNCH;
  }
  if constexpr (ROWS) {
    // D by TMA: without C, 16-byte rows, and a width that is a multiple of
    // 16 bytes (a box clipped inside a 16-byte chunk writes the chunk whole)
    const int db = args.d_type == MMA_F32 ? 4 : 2;
    if (args.C == nullptr && (reinterpret_cast<uintptr_t>(args.D) & 15) == 0 &&
        args.ldd * db % 16 == 0 && int64_t(args.q_size) * db % 16 == 0) {
      if (!make_cd_map(&td, args.D, args.q_size, args.rows_total, args.ldd,
                       db == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32
                               : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                       db))
        return MMA_ERR_LAUNCH;
      a.d_tma = 1;
    }
  }
  auto kern =
      gemm_grouped_kernel<KIND8, P_MN, Q_MN, RAGK, ROWS, SPLIT, CL, BN, STAGES, LORA>;
  constexpr int kLists = LORA == kRequests ? 3 : 2;
  constexpr int kMostSplit = !SPLIT ? 1 : BN == 32 ? 6 : BN == 64 ? 4 : 2;
  static_assert(L::alloc(kMaxGroups, kMostSplit, BN, kLists) <= 232448, "shared memory per CTA");
  // SPLIT: as many CTAs per tile as leave every tile's cluster room at once
  // (two CTAs per SM if their shared memory fits twice), each with four k
  // blocks at least.  One row, 8192 x 4096: 64 tiles, 14.7 us without.
  int split = 1;
  if constexpr (SPLIT) {
    const int64_t blocks = (int64_t(a.k_size) + KE - 1) / KE;
    a.part_cols = a.offsets ? BN : std::min(BN, a.rows_total);
    for (int s = kMostSplit; s > 1 && split == 1; --s) {
      const int64_t slots =
          ctx.num_sms * (2 * (L::alloc(a.groups, s, a.part_cols) + 1024) <= 233472 ? 2 : 1);
      if (most * s <= slots && blocks >= 4 * s) split = s;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads, 1, 1);
  // One CTA per SM when there is no more than one for each: were there room
  // for two, the next call's CTAs would come in pairs beside this one's and
  // leave SMs idle (16 rows, 8192 x 4096: 10.4 us, else 11.9).
  int smem = L::alloc(a.groups, split, a.part_cols, kLists);
  if (SPLIT && most * split <= ctx.num_sms) smem = std::max(smem, 118 * 1024);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = ctx.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // CTAs (or pairs) that run at once, with few groups and without a split;
  // once per context and instantiation
  static PerContext<int> resident;
  int at_once = 0;
  if (!resident.get(ctx, &at_once, [&](int* v) {
        bool ok = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       L::alloc(kMaxGroups, kMostSplit, BN, kLists)) == cudaSuccess;
        // the split of the registers counts on the launch's
        cudaFuncAttributes fa = {};
        ok = ok && cudaFuncGetAttributes(&fa, kern) == cudaSuccess &&
             (BN < 256 || fa.numRegs == kLaunchRegs);
        cudaLaunchConfig_t probe = cfg;
        probe.numAttrs = 1;
        probe.dynamicSmemBytes = size_t(L::alloc(64, 1, 0));
        probe.gridDim = dim3(unsigned(CL * (ctx.num_sms / CL)), 1, 1);
        ok = ok && cudaOccupancyMaxActiveClusters(v, kern, &probe) == cudaSuccess && *v > 0;
        if (!ok) cudaGetLastError();
        return ok;
      }))
    return MMA_ERR_LAUNCH;
  const int64_t clusters = split > 1 ? most : std::min<int64_t>(most, at_once);
  attr[0].val.clusterDim.x = unsigned(CL * split);
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(unsigned(clusters * CL * split), 1, 1);
  ctx.mark_start();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tp, tq, td, tz, a);
  ctx.mark_stop();
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

// Whether `n` consecutive elements at multiples of n in a row can move at once.
bool elements_aligned(const void* p, int64_t ld, int bytes, int n) {
  return (reinterpret_cast<uintptr_t>(p) & uintptr_t(n * bytes - 1)) == 0 && ld % n == 0;
}

// Few rows per group (`per`), column-major B: tiles of 32, 64 or 128 columns.
// With fewer of them than SMs a cluster shares each one's k range; else one
// CTA per SM with a deep ring streams them (64 experts of 2048 x 4096 with 96
// tokens: 62 us, two CTAs per SM with half the ring 66).  8192 x 4096 8-bit,
// 32 rows: 32 columns 10.4 us, 64 11.0, 128 11.3; 64 rows: 64 columns 12.5 us,
// 128 12.7; 128 rows: 128 columns 16.0 us, pairs with 256 17.9.  32 experts of
// 4096 x 2048 by 64 rows, 16-bit, streamed: 64 columns 94.7 us, 128 87.9.
template <bool KIND8, Lora LORA = kNoLora>
mma_status_t few_rows(const Ctx& ctx, const Operand& B, const Operand& A,
                      const GroupedArgs& a, int64_t per) {
  const int64_t tiles = (a.p_size + kP - 1) / kP *
                        (a.offsets ? std::min<int64_t>(a.rows_total, a.groups) : 1);
  const bool split = tiles < ctx.num_sms;
  if (per <= 32)
    return split ? run<KIND8, false, false, false, false, true, 1, 32, 4, LORA>(ctx, B, A, a)
                 : run<KIND8, false, false, false, false, false, 1, 32, 8, LORA>(ctx, B, A, a);
  if (per <= 64 && split)
    return run<KIND8, false, false, false, false, true, 1, 64, 4, LORA>(ctx, B, A, a);
  return split ? run<KIND8, false, false, false, false, true, 1, 128, 4, LORA>(ctx, B, A, a)
               : run<KIND8, false, false, false, false, false, 1, 128, 6, LORA>(ctx, B, A, a);
}

}  // namespace

mma_status_t launch_gemm_f8(const Ctx& ctx, const F8Problem& f) {
  GroupedArgs a = {};
  a.k_size = int(f.K);
  a.groups = int(f.groups);
  a.rows_total = int(f.rows);
  a.offsets = f.offsets;
  a.kb_per_chunk = 1;
  a.d_type = f.d_type;
  a.C = f.C;
  a.ldc = f.ldc;
  a.D = f.D;
  a.ldd = f.ldd;
  a.status = ctx.status;
  a.withhold = f.withhold;
  const Operand A = {f.A, f.lda, f.rows, 1, 0};
  const Operand B = {f.B, f.ldb, f.N, f.groups, f.stride_b};
  const int shift = f.sb_rows == 128 ? 7 : 0;
  const int64_t per = (f.rows + f.groups - 1) / f.groups;
  // Few tiles, on single CTAs of 128 x 128: those that one wave takes if B has
  // a scale for each row (512 x 4096 x 4096: 19.6 us, on pairs 28.8; 512 x 8192
  // x 4096, two waves: 35.7, on pairs 29.7), and with square scales, where
  // pairs take half the time, if two CTAs can share each one's long k range
  // (512 x 1024 x 16384: 38 us, on pairs 53; 1024 x 1024 x 4096: 16.1 and
  // 16.7; 512 x 1024 x 1024: 8.8 and 7.3; 512 x 4096 x 4096: 20.5 and 17.2).
  const int64_t tiles = (f.N + kP - 1) / kP *
                        (f.offsets ? f.rows / kP + f.groups : (f.rows + kP - 1) / kP);
  const bool few = per <= 128 || (shift == 7 ? 2 * tiles <= ctx.num_sms && f.K >= 4096
                                             : tiles <= ctx.num_sms);
  // Many rows: a lane per row of A.  That needs one scale of B for the
  // columns of a lane's half tile; a tile holds 256 rows of one group.
  if (shift == 7 && !few) {
    const int db = f.d_type == MMA_F32 ? 4 : 2;
    a.p_size = int(f.rows);
    a.q_size = int(f.N);
    a.vec4 = elements_aligned(f.D, f.ldd, db, 4) &&
             (f.C == nullptr || elements_aligned(f.C, f.ldc, db, 4));
    a.vec8 = db == 2 && f.C == nullptr && elements_aligned(f.D, f.ldd, db, 8);
    a.idesc = idesc_f32(f.a_e5m2, f.b_e5m2, false, false, 2 * kP);
    a.sp = f.SA;
    a.sp_row = f.sa_row;
    a.sp_blk = f.sa_blk;
    a.sq = f.SB;
    a.sq_group = f.sb_group;
    a.sq_row = f.sb_row;
    a.sq_blk = f.sb_blk;
    a.q_shift = 7;
    return run<true, false, false, false, true, false, 2, 256, 4>(ctx, A, B, a);
  }
  a.p_size = int(f.N);
  a.q_size = int(f.rows);
  a.sp = f.SB;
  a.sp_group = f.sb_group;
  a.sp_row = f.sb_row;
  a.sp_blk = f.sb_blk;
  a.p_shift = shift;
  a.sq = f.SA;
  a.sq_row = f.sa_row;
  a.sq_blk = f.sa_blk;
  if (!few) {
    a.idesc = idesc_f32(f.b_e5m2, f.a_e5m2, false, false, 2 * kP);
    return run<true, false, false, false, false, false, 2, 256, 6>(ctx, B, A, a);
  }
  a.idesc = idesc_f32(f.b_e5m2, f.a_e5m2, false, false, kP);
  return few_rows<true>(ctx, B, A, a, per);
}

mma_status_t launch_gemm_grouped(const Ctx& ctx, const GroupedProblem& g) {
  GroupedArgs a = {};
  a.p_size = int(g.N);
  a.q_size = int(g.rows);
  a.k_size = int(g.K);
  a.groups = int(g.groups);
  a.rows_total = int(g.rows);
  a.offsets = g.offsets;
  // (a 16-bit result's own rounding is 500 times what 512 terms lose)
  a.kb_per_chunk = g.d_type == MMA_F32 ? 4 : 8;
  a.d_type = g.d_type;
  a.C = g.C;
  a.ldc = g.ldc;
  a.D = g.D;
  a.ldd = g.ldd;
  a.status = ctx.status;
  const int64_t per = (g.rows + g.groups - 1) / g.groups;
  const Operand A = {g.A, g.lda, g.rows, 1, 0};
  const Operand B = {g.B, g.ldb, g.b_row_major ? g.K : g.N, g.groups, g.stride_b};
  // (32 experts of 4096 x 2048: by 128 rows 92 us, on pairs 95; by 160 rows
  // 120 us, on pairs 97; with row-major B 88 and 91, 119 and 93)
  const bool pair = per > 128;
  a.idesc = idesc_f32(g.bf16, g.bf16, g.b_row_major, false, pair ? 2 * kP : kP);
  if (g.b_row_major) {
    if (pair) return run<false, true, false, false, false, false, 2, 256, 6>(ctx, B, A, a);
    return run<false, true, false, false, false, false, 1, 128, 6>(ctx, B, A, a);
  }
  if (pair) return run<false, false, false, false, false, false, 2, 256, 6>(ctx, B, A, a);
  return few_rows<false>(ctx, B, A, a, per);
}

mma_status_t launch_gemm_lora(const Ctx& ctx, const LoraProblem& g, const LoraLow* low) {
  GroupedArgs a = {};
  a.p_size = int(g.N);
  a.q_size = int(g.rows);
  a.k_size = int(g.K);
  a.rows_total = int(g.rows);
  a.kb_per_chunk = g.d_type == MMA_F32 ? 4 : 8;  // (as launch_gemm_grouped)
  a.d_type = g.d_type;
  a.C = g.C;
  a.ldc = g.ldc;
  a.D = g.D;
  a.ldd = g.ldd;
  a.status = ctx.status;
  const Operand X = {g.X, g.ldx, g.rows, 1, 0};
  const Operand W = {g.W, g.ldw, g.row_major ? g.K : g.N, 1, 0};
  // (with more requests than fit beside a pair's tiles every row is added)
  const bool every = low && lora_every(g.rows, g.requests);
  const bool pair = g.rows > kLoraEveryRow && !every;
  a.idesc = idesc_f32(g.bf16, g.bf16, g.row_major, false, pair ? 2 * kP : kP);
  a.groups = 1;
  if (!low) {
    if (g.row_major) {
      if (pair) return run<false, true, false, false, false, false, 2, 256, 6>(ctx, W, X, a);
      return run<false, true, false, false, false, false, 1, 128, 6>(ctx, W, X, a);
    }
    if (pair) return run<false, false, false, false, false, false, 2, 256, 6>(ctx, W, X, a);
    return few_rows<false>(ctx, W, X, a, g.rows);
  }
  a.extra = low->extra;
  if (!pair) {
    if (g.row_major)
      return run<false, true, false, false, false, false, 1, 128, 6, kEveryRow>(ctx, W, X, a);
    if (g.rows > kLoraEveryRow)
      return run<false, false, false, false, false, false, 1, 128, 6, kEveryRow>(ctx, W, X, a);
    return few_rows<false, kEveryRow>(ctx, W, X, a, g.rows);
  }
  a.groups = int(g.requests);
  a.offsets = g.offsets;
  a.adapters = g.adapters;
  a.adapters_total = int(g.adapters_total);
  a.rank = int(g.rank);
  a.parts = low->parts;
  a.up = g.bf16 ? nullptr : static_cast<const uint16_t*>(low->f16) + g.rank;
  a.ld_up = low->ld16;
  const LoraMaps m = {{g.B, g.ldb, g.N, g.adapters_total, g.stride_b},
                      {low->f16, low->ld16, g.rows, low->parts, int64_t(low->ld16) * g.rows}};
  if (g.row_major)
    return run<false, true, false, false, false, false, 2, 256, 6, kRequests>(ctx, W, X, a, &m);
  return run<false, false, false, false, false, false, 2, 256, 6, kRequests>(ctx, W, X, a, &m);
}

mma_status_t launch_gemm_grouped_wgrad(const Ctx& ctx, const WgradProblem& g) {
  GroupedArgs a = {};
  a.p_size = int(g.K);
  a.q_size = int(g.N);
  a.k_size = int(g.rows);
  a.groups = int(g.groups);
  a.rows_total = int(g.rows);
  a.offsets = g.offsets;
  // (a 16-bit result's own rounding is 500 times what 512 terms lose)
  a.kb_per_chunk = g.d_type == MMA_F32 ? 4 : 8;
  a.d_type = g.d_type;
  a.C = g.C;
  a.ldc = g.ldc;
  a.c_group = g.stride_c;
  a.D = g.D;
  a.ldd = g.ldd;
  a.d_group = g.stride_d;
  a.status = ctx.status;
  a.withhold = g.withhold;
  a.idesc = idesc_f32(g.bf16, g.bf16, true, true, 2 * kP);
  const Operand X = {g.X, g.ldx, g.rows, 1, 0};
  const Operand DY = {g.DY, g.lddy, g.rows, 1, 0};
  return run<false, true, true, true, false, false, 2, 256, 6>(ctx, X, DY, a);
}

mma_status_t launch_products_abort_selftest(const Ctx& ctx, int kind, const void* X, void* D,
                                            float* S) {
  if (kind == 2) {
    WgradProblem g = {};
    g.bf16 = true;
    g.d_type = MMA_BF16;
    g.groups = 1;
    g.rows = g.N = g.K = 1024;
    g.DY = g.X = X;
    g.lddy = g.ldx = g.ldd = 1024;
    g.offsets = reinterpret_cast<const int*>(S);
    g.D = D;
    g.withhold = 1;
    return launch_gemm_grouped_wgrad(ctx, g);
  }
  F8Problem f = {};
  f.d_type = MMA_BF16;
  f.groups = 1;
  f.rows = kind == 0 ? 1 : 1024;
  f.N = f.K = 1024;
  f.A = f.B = X;
  f.lda = f.ldb = f.ldd = 1024;
  f.SA = f.SB = S;
  f.sa_row = f.sb_row = 1;
  f.sa_blk = f.sb_blk = 1024;
  f.sb_rows = 128;
  f.D = D;
  f.withhold = 1;
  return launch_gemm_f8(ctx, f);
}

}  // namespace mmagb
