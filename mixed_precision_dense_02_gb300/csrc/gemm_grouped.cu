// Products with scaled 8-bit operands and products grouped by expert, on
// the tcgen05 tensor cores.  One kernel carries all of them:
//
//     D_e[q][p] = C_e[q][p] + sum_k Q_e[q][k] * P_e[p][k]
//
// with P the operand whose 128 rows fill the tensor core's M side and whose
// index p is the contiguous one of D, and Q the operand on the N side:
//
//   call                      P (rows p)        Q (rows q)       k
//   8-bit product             B (N x K)         A (M x K)        K
//   grouped forward           B_e (N x K)       A (token x K)    K
//   grouped, row-major B      B_e (K x N)^T     A (token x K)    K
//   grouped weight gradient   X (token x K)^T   dY (token x N)^T tokens of e
//
// so D's rows leave the kernel as runs of consecutive p, one per lane, and
// the ragged dimension of a group (its tokens) is the N side, whose extent
// is chosen per tile in steps of 16: a group of 300 tokens costs 304 rows of
// tensor work, not 384.
//
// Arithmetic.  The tensor core's FP32 sums drop low bits on the way (a
// relative error that grows with the length of the sum, 1.2e-7 at 128 terms
// and 4.2e-6 at 4096, measured against 64 bits), so K is cut into chunks;
// each chunk's sum is added to FP32 registers, rounded to nearest.  With
// 8-bit operands a chunk is one block of 128 and the addition multiplies by
// the block's two scales: acc += (sp * sq) * t.
//
// Roles, as in the dense kernel: warp 0 loads operand boxes by TMA into a
// ring of stages of 128 bytes of k, warp 1 issues the MMAs into two
// accumulators in tensor memory, eight warps add the chunks up in registers
// and store D.
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace mmagb {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn();  // gemm_tc.cu

namespace {

constexpr int kP = 128;  // rows of P per CTA
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;

// What a launch computes (see the table above).  Group e's rows of Q are
// [row[e], row[e + 1]) of `offsets` (one group of q_size rows without
// offsets); for the weight gradient those are its k range and every group
// has q_size rows of Q.
struct GroupedArgs {
  int p_size, q_size, k_size, groups, rows_total;
  const int* offsets;
  uint32_t idesc;  // without the N field
  int kb_per_chunk;
  int d_type;  // MMA_F32, MMA_F16 or MMA_BF16
  const void* C;
  int64_t ldc, c_group;
  void* D;
  int64_t ldd, d_group;
  // 8-bit operands: the scale of row p (or of the 128 rows around it, with
  // p_shift = 7) of group e for k block b at sp[e * sp_group +
  // (p >> p_shift) * sp_row + b * sp_blk]; of row q at sq[q * sq_row + b * sq_blk]
  const float* sp;
  int64_t sp_group, sp_row, sp_blk;
  int p_shift;
  const float* sq;
  int64_t sq_row, sq_blk;
  unsigned* status;
};

template <int BN, int STAGES>
struct Layout {
  static constexpr int P_BYTES = kP * 128;
  static constexpr int Q_BYTES = BN * 128;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr int SCALE_OFFSET = STAGES * STAGE_BYTES;
  // q scales of the warp's columns, two buffers per warp
  static constexpr int SCALE_BYTES = kEpiWarps * 2 * (BN / 2) * 4;
  static constexpr int BAR_OFFSET = SCALE_OFFSET + SCALE_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int GROUP_OFFSET = BAR_OFFSET + NUM_BARS * 8 + 24;
  static int alloc(int groups) {
    return GROUP_OFFSET + 2 * (groups + 1) * 4 + 1024;  // base alignment
  }
  static constexpr uint32_t TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
};

// One tile of work.
struct Tile {
  int e;         // group
  int p0;        // first row of P
  int q0, q1;    // rows of Q (rows of D)
  int nt;        // MMA N: q1 - q0 rounded up to 16
  int k0, k1;    // k range
};

__device__ __forceinline__ float load_c(const void* c, int64_t i, int t) {
  if (t == MMA_F32) return static_cast<const float*>(c)[i];
  if (t == MMA_BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(c)[i]);
  return __half2float(static_cast<const __half*>(c)[i]);
}

// Drain without giving up on the abort flag.
__device__ __forceinline__ void wait_drain(uint64_t* bar, uint32_t parity,
                                           unsigned* status) {
  const uint32_t a = smem_u32(bar);
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(a, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, kStatusTimeout);
      return;
    }
  }
}

// KIND8: 8-bit operands with scales, else 16-bit.  P_MN, Q_MN: the operand
// is stored with its row index contiguous (16-bit only).  RAGK: the groups
// cut the k range (the weight gradient).
template <bool KIND8, bool P_MN, bool Q_MN, bool RAGK, int BN, int STAGES>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_grouped_kernel(const __grid_constant__ CUtensorMap tmP,
                        const __grid_constant__ CUtensorMap tmQ,
                        const __grid_constant__ GroupedArgs a) {
  using L = Layout<BN, STAGES>;
  constexpr int KE = KIND8 ? 128 : 64;  // k elements per stage
  constexpr int HALF = BN / 2;          // most columns of an epilogue warp
  constexpr int CB = HALF < 32 ? HALF : 32;
  constexpr int NB = HALF / CB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFFSET);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* grow = reinterpret_cast<int*>(smem + L::GROUP_OFFSET);  // groups + 1
  int* gunit = grow + a.groups + 1;                            // groups + 1

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int p_tiles = (a.p_size + kP - 1) / kP;
  const int q_tiles = (a.q_size + BN - 1) / BN;  // RAGK: per group

  if (threadIdx.x == 32) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tmP);
      tma_prefetch_desc(&tmQ);
    }
    // Row and unit ranges of the groups.  Offsets are clamped to
    // [0, rows_total] and made non-decreasing, so that no value of theirs
    // leads outside the operands.
    auto at = [&](int i) {
      if (!a.offsets) return i == 0 ? 0 : a.rows_total;
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
      int n = RAGK ? q_tiles * p_tiles : ((hi - lo + BN - 1) / BN) * p_tiles;
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
  if (warp == 1) {
    tmem_alloc(tmem_slot, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int units = gunit[a.groups];

  // Unit u: its group by bisection, then p tiles fastest.
  auto decode = [&](int u) {
    int lo = 0, hi = a.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (gunit[mid] <= u) lo = mid; else hi = mid;
    }
    Tile t;
    t.e = lo;
    const int r = u - gunit[lo];
    const int first = RAGK ? 0 : grow[lo];
    const int rows = RAGK ? a.q_size : grow[lo + 1] - first;
    const int tiles = (rows + BN - 1) / BN;
    // the group's rows are shared out evenly, in steps of 16
    const int step = ((rows + tiles - 1) / tiles + 15) & ~15;
    const int qi = r / p_tiles;
    t.p0 = (r - qi * p_tiles) * kP;
    t.q0 = first + qi * step;
    t.q1 = min(t.q0 + step, first + rows);
    t.nt = (t.q1 - t.q0 + 15) & ~15;
    t.k0 = RAGK ? grow[lo] : 0;
    t.k1 = RAGK ? grow[lo + 1] : a.k_size;
    return t;
  };

  if (warp == 0) {
    // ------------------------------------------------ TMA producer
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        const Tile t = decode(u);
        for (int k = t.k0; k < t.k1; k += KE) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          uint8_t* sp = smem + stage * L::STAGE_BYTES;
          uint8_t* sq = sp + L::P_BYTES;
          mbar_arrive_expect_tx(&full[stage], L::STAGE_BYTES);
          if constexpr (P_MN) {
            for (int i = 0; i < kP / 64; ++i)
              tma_load_3d(&tmP, &full[stage], sp + i * 8192, t.p0 + 64 * i, k,
                          RAGK ? 0 : t.e);
          } else {
            tma_load_3d(&tmP, &full[stage], sp, k, t.p0, t.e);
          }
          if constexpr (Q_MN) {
            for (int i = 0; i < BN / 64; ++i)
              tma_load_3d(&tmQ, &full[stage], sq + i * 8192, t.q0 + 64 * i, k, 0);
          } else {
            tma_load_3d(&tmQ, &full[stage], sq, k, t.q0, 0);
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // after an abort, let the loads in flight land before the CTA exits
      if (!ok)
        for (int s = 0; s < STAGES; ++s) {
          const uint32_t fills = issued / STAGES + (uint32_t(s) < issued % STAGES);
          if (fills) wait_drain(&full[s], (fills - 1) & 1u, a.status);
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    // (the whole warp walks the stages; lane 0 issues)
    int stage = 0;
    uint32_t phase = 0, acc_phase = 0;
    int acc = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const Tile t = decode(u);
      const uint32_t idesc = a.idesc | (uint32_t(t.nt >> 3) << 17);
      int in_chunk = 0;
      for (int k = t.k0; k < t.k1; k += KE) {
        const uint32_t d_tmem = tmem_base + uint32_t(acc * BN);
        if (in_chunk == 0) {
          ok = mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag, a.status);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          tc_fence_after();
        }
        ok = mbar_wait(&full[stage], phase, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        uint8_t* sp = smem + stage * L::STAGE_BYTES;
        const int left = t.k1 - k;
        int steps = 4;
        if constexpr (RAGK) {
          // The group ends inside this block: its last step of 16 holds
          // rows of the next group, which become zeros in both operands
          // (in one of them alone, an infinity in the other would leave
          // NaN).
          if (left < KE) {
            steps = (left + 15) >> 4;
            const int zrows = steps * 16 - left;
            const int units16 = zrows * 8;
            for (int i = lane; i < (kP / 64 + BN / 64) * units16; i += 32) {
              const int box = i / units16, r = i - box * units16;
              uint8_t* dst = box < kP / 64 ? sp + box * 8192
                                           : sp + L::P_BYTES + (box - kP / 64) * 8192;
              *reinterpret_cast<uint4*>(dst + left * 128 + r * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        tc_fence_after();
        const bool last = in_chunk + 1 == a.kb_per_chunk || left <= KE;
        if (lane == 0) {
          const uint32_t sa = smem_u32(sp);
          const uint64_t dp = P_MN ? sw128_mnmajor_desc(sa) : sw128_kmajor_desc(sa);
          const uint64_t dq = Q_MN ? sw128_mnmajor_desc(sa + L::P_BYTES)
                                   : sw128_kmajor_desc(sa + L::P_BYTES);
          // 32 bytes of a row (K-major) or 16 rows (MN-major) per step
          constexpr uint64_t kStepP = P_MN ? 128 : 2;
          constexpr uint64_t kStepQ = Q_MN ? 128 : 2;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if (RAGK && s >= steps) break;
            const uint32_t accum = (in_chunk != 0 || s != 0) ? 1u : 0u;
            if constexpr (KIND8)
              umma_f8<1>(d_tmem, dp + s * kStepP, dq + s * kStepQ, idesc, accum);
            else
              umma_f16(d_tmem, dp + s * kStepP, dq + s * kStepQ, idesc, accum);
          }
          umma_commit(&empty[stage]);
          if (last) umma_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (last) {
          in_chunk = 0;
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        } else {
          ++in_chunk;
        }
      }
    }
    // Every MMA issued above completes before tensor memory is released.
    if (lane == 0) {
      umma_commit(done);
      wait_drain(done, 0, a.status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue warps
    // A warp owns 32 rows of P (its tensor-memory lane quarter) and every
    // other block of CB columns.
    const int ew = warp - 2;
    const int quarter = warp & 3;
    const int h = ew >> 2;
    float* sqs = reinterpret_cast<float*>(smem + L::SCALE_OFFSET) + ew * 2 * HALF;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const Tile t = decode(u);
      const int p = t.p0 + quarter * 32 + lane;
      uint64_t sum[HALF / 2];
#pragma unroll
      for (int j = 0; j < HALF / 2; ++j) sum[j] = 0ull;
      const int num_kb = (t.k1 - t.k0 + KE - 1) / KE;
      const int chunks = (num_kb + a.kb_per_chunk - 1) / a.kb_per_chunk;
      // 8-bit: the scales of chunk ch (one k block): this lane's row of P
      // and one column per block of columns
      [[maybe_unused]] float spv = 0.f, sqv[NB];
      [[maybe_unused]] auto load_scales = [&](int ch) {
        spv = 0.f;
        if (p < a.p_size)
          spv = __ldg(a.sp + t.e * a.sp_group + (p >> a.p_shift) * a.sp_row +
                      ch * a.sp_blk);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int q = t.q0 + (2 * i + h) * CB + lane;
          sqv[i] = 0.f;
          if (lane < CB && q < t.q1) sqv[i] = __ldg(a.sq + q * a.sq_row + ch * a.sq_blk);
        }
      };
      if constexpr (KIND8)
        if (chunks > 0) load_scales(0);
      for (int ch = 0; ch < chunks; ++ch) {
        [[maybe_unused]] float* buf = sqs + (ch & 1) * HALF;
        [[maybe_unused]] uint64_t sp2 = 0;
        if constexpr (KIND8) {
          if (lane < CB) {
#pragma unroll
            for (int i = 0; i < NB; ++i) buf[i * CB + lane] = sqv[i];
          }
          sp2 = pack_f32x2(__float_as_uint(spv), __float_as_uint(spv));
          __syncwarp();
          if (ch + 1 < chunks) load_scales(ch + 1);
        }
        ok = mbar_wait(&tfull[acc], acc_phase, abort_flag, a.status);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr =
            tmem_base + uint32_t(acc * BN) + (uint32_t(quarter * 32) << 16);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int col = (2 * i + h) * CB;
          if (col >= t.nt) continue;
          uint32_t r[CB];
          if constexpr (CB == 32)
            tmem_ld_32x32b_x32(taddr + col, r);
          else
            tmem_ld_32x32b_x16(taddr + col, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < CB; j += 4) {
            uint64_t& s0 = sum[(i * CB + j) / 2];
            uint64_t& s1 = sum[(i * CB + j) / 2 + 1];
            const uint64_t t0 = pack_f32x2(r[j], r[j + 1]);
            const uint64_t t1 = pack_f32x2(r[j + 2], r[j + 3]);
            if constexpr (KIND8) {
              const ulonglong2 v =
                  *reinterpret_cast<const ulonglong2*>(buf + i * CB + j);
              s0 = fma_f32x2(mul_f32x2(v.x, sp2), t0, s0);
              s1 = fma_f32x2(mul_f32x2(v.y, sp2), t1, s1);
            } else {
              s0 = add_f32x2(s0, t0);
              s1 = add_f32x2(s1, t1);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      if (!ok) break;
      if (p >= a.p_size) continue;
      const int64_t group = RAGK ? t.e : 0;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int q = t.q0 + (2 * i + h) * CB;
        if (q >= t.q1) continue;
        float v[CB];
#pragma unroll
        for (int j = 0; j < CB; j += 2)
          unpack_f32x2(sum[(i * CB + j) / 2], v[j], v[j + 1]);
        if (a.C) {
          const int64_t ci = group * a.c_group + int64_t(q) * a.ldc + p;
#pragma unroll
          for (int j = 0; j < CB; ++j)
            if (q + j < t.q1) v[j] += load_c(a.C, ci + j * a.ldc, a.d_type);
        }
        const int64_t di = group * a.d_group + int64_t(q) * a.ldd + p;
        if (a.d_type == MMA_F32) {
          float* d = static_cast<float*>(a.D) + di;
#pragma unroll
          for (int j = 0; j < CB; ++j)
            if (q + j < t.q1) d[j * a.ldd] = v[j];
        } else if (a.d_type == MMA_BF16) {
          __nv_bfloat16* d = static_cast<__nv_bfloat16*>(a.D) + di;
#pragma unroll
          for (int j = 0; j < CB; ++j)
            if (q + j < t.q1) d[j * a.ldd] = __float2bfloat16_rn(v[j]);
        } else {
          __half* d = static_cast<__half*>(a.D) + di;
#pragma unroll
          for (int j = 0; j < CB; ++j)
            if (q + j < t.q1) d[j * a.ldd] = __float2half_rn(v[j]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, L::TMEM_COLS);
}

// ----------------------------------------------------------------- host

// A 3-D map over 1- or 2-byte elements with 128-byte swizzle: `inner`
// contiguous elements, `outer` rows `ld` elements apart, `count` slices
// `slice` elements apart; box box_inner x box_outer x 1.
bool make_map(CUtensorMap* map, const void* base, int elem, int64_t inner,
              int64_t outer, int64_t ld, int64_t count, int64_t slice,
              int box_inner, int box_outer) {
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
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operands {
  const void* P;
  int64_t ldp, p_slice;  // p_slice: elements between the groups' P
  const void* Q;
  int64_t ldq;
  int64_t p_rows_total, q_rows_total;  // extents of the maps' rows
};

template <bool KIND8, bool P_MN, bool Q_MN, bool RAGK, int BN, int STAGES>
mma_status_t run(const Ctx& ctx, const Operands& o, const GroupedArgs& a) {
  using L = Layout<BN, STAGES>;
  constexpr int EB = KIND8 ? 1 : 2;
  constexpr int KE = KIND8 ? 128 : 64;
  const int64_t p_tiles = (a.p_size + kP - 1) / kP;
  const int64_t most =
      RAGK ? int64_t(a.groups) * ((a.q_size + BN - 1) / BN) * p_tiles
           : (int64_t(a.rows_total) / BN + (a.offsets ? a.groups : 1)) * p_tiles;
  if (most > int64_t(INT32_MAX) / 2) return MMA_ERR_UNSUPPORTED;
  CUtensorMap tp, tq;
  bool ok_p, ok_q;
  if (a.k_size == 0) {
    // Nothing to load (D = C): the kernel still wants two valid maps.
    void* any = reinterpret_cast<void*>(reinterpret_cast<uintptr_t>(a.D) & ~uintptr_t(15));
    ok_p = make_map(&tp, any, EB, 64, 1, 64, 1, 64, 64, 1);
    tq = tp;
    ok_q = ok_p;
  } else {
    const int64_t slices = RAGK ? 1 : a.groups;
    const int64_t slice = slices > 1 ? o.p_slice : o.ldp;  // unused when 1
    ok_p = P_MN ? make_map(&tp, o.P, EB, a.p_size, o.p_rows_total, o.ldp, slices,
                           slice, 64, 64)
                : make_map(&tp, o.P, EB, a.k_size, o.p_rows_total, o.ldp, slices,
                           slice, KE, kP);
    ok_q = Q_MN ? make_map(&tq, o.Q, EB, a.q_size, o.q_rows_total, o.ldq, 1,
                           o.ldq, 64, 64)
                : make_map(&tq, o.Q, EB, a.k_size, o.q_rows_total, o.ldq, 1,
                           o.ldq, KE, BN);
  }
  if (!ok_p || !ok_q) return MMA_ERR_LAUNCH;
  auto kern = gemm_grouped_kernel<KIND8, P_MN, Q_MN, RAGK, BN, STAGES>;
  static_assert(L::GROUP_OFFSET + 2 * (kMaxGroups + 1) * 4 + 1024 <= 232448,
                "shared memory per CTA");
  static PerContext<bool> attr;
  bool ok = false;
  if (!attr.get(ctx, &ok, [&](bool* v) {
        *v = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  L::alloc(kMaxGroups)) == cudaSuccess;
        if (!*v) cudaGetLastError();
        return *v;
      }))
    return MMA_ERR_LAUNCH;
  const int grid = int(most < ctx.num_sms ? most : ctx.num_sms);
  ctx.mark_start();
  kern<<<grid, kThreads, L::alloc(a.groups), ctx.stream>>>(tp, tq, a);
  ctx.mark_stop();
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

}  // namespace

mma_status_t launch_gemm_f8(const Ctx& ctx, const F8Problem& f) {
  GroupedArgs a = {};
  a.p_size = int(f.N);
  a.q_size = int(f.rows);
  a.k_size = int(f.K);
  a.groups = int(f.groups);
  a.rows_total = int(f.rows);
  a.offsets = f.offsets;
  a.idesc = idesc_f32(f.b_e5m2, f.a_e5m2, false, false, kP);
  a.kb_per_chunk = 1;
  a.d_type = f.d_type;
  a.C = f.C;
  a.ldc = f.ldc;
  a.D = f.D;
  a.ldd = f.ldd;
  a.sp = f.SB;
  a.sp_group = f.sb_group;
  a.sp_row = f.sb_row;
  a.sp_blk = f.sb_blk;
  a.p_shift = f.sb_rows == 128 ? 7 : 0;
  a.sq = f.SA;
  a.sq_row = f.sa_row;
  a.sq_blk = f.sa_blk;
  a.status = ctx.status;
  const Operands o = {f.B, f.ldb, f.stride_b, f.A, f.lda, f.N, f.rows};
  const int64_t per = (f.rows + f.groups - 1) / f.groups;
  if (per <= 32) return run<true, false, false, false, 32, 8>(ctx, o, a);
  if (per <= 128) return run<true, false, false, false, 128, 6>(ctx, o, a);
  return run<true, false, false, false, 256, 4>(ctx, o, a);
}

mma_status_t launch_gemm_grouped(const Ctx& ctx, const GroupedProblem& g) {
  GroupedArgs a = {};
  a.p_size = int(g.N);
  a.q_size = int(g.rows);
  a.k_size = int(g.K);
  a.groups = int(g.groups);
  a.rows_total = int(g.rows);
  a.offsets = g.offsets;
  a.kb_per_chunk = 4;
  a.d_type = g.d_type;
  a.C = g.C;
  a.ldc = g.ldc;
  a.D = g.D;
  a.ldd = g.ldd;
  a.status = ctx.status;
  a.idesc = idesc_f32(g.bf16, g.bf16, g.b_row_major, false, kP);
  const int64_t per = (g.rows + g.groups - 1) / g.groups;
  const Operands o = {g.B, g.ldb, g.stride_b, g.A, g.lda,
                      g.b_row_major ? g.K : g.N, g.rows};
  if (g.b_row_major) {
    if (per <= 128) return run<false, true, false, false, 128, 6>(ctx, o, a);
    return run<false, true, false, false, 256, 4>(ctx, o, a);
  }
  if (per <= 32) return run<false, false, false, false, 32, 8>(ctx, o, a);
  if (per <= 128) return run<false, false, false, false, 128, 6>(ctx, o, a);
  return run<false, false, false, false, 256, 4>(ctx, o, a);
}

mma_status_t launch_gemm_grouped_wgrad(const Ctx& ctx, const WgradProblem& g) {
  GroupedArgs a = {};
  a.p_size = int(g.K);
  a.q_size = int(g.N);
  a.k_size = int(g.rows);
  a.groups = int(g.groups);
  a.rows_total = int(g.rows);
  a.offsets = g.offsets;
  a.kb_per_chunk = 4;
  a.d_type = g.d_type;
  a.C = g.C;
  a.ldc = g.ldc;
  a.c_group = g.stride_c;
  a.D = g.D;
  a.ldd = g.ldd;
  a.d_group = g.stride_d;
  a.status = ctx.status;
  a.idesc = idesc_f32(g.bf16, g.bf16, true, true, kP);
  const Operands o = {g.X, g.ldx, 0, g.DY, g.lddy, g.rows, g.rows};
  return run<false, true, true, true, 256, 4>(ctx, o, a);
}

}  // namespace mmagb
