// C ABI of the library (declared in include/mma_gb300.h): argument
// validation, per-device set-up and dispatch to the kernels.  Nothing here
// computes any part of D = A * B + C; every arithmetic step runs on the GPU.
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "kernels.h"

namespace mmagb {

// Device-side status word: bounded pipeline waits OR their error bits in.
__device__ unsigned g_mma_status;

namespace {

struct DeviceInfo {
  bool ready = false;
  bool usable = false;
  int num_sms = 0;
  unsigned* status = nullptr;
  uint64_t gen = 0;  // context the fields above were set up in
};

DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mu;

// Profiling ring: while active, each call records one event pair around its
// dominant kernel.  Events are created once and reused.
constexpr int kProfMax = 4096;
struct Profile {
  bool active = false;
  int device = -1;
  int count = 0;
  cudaEvent_t ev[2 * kProfMax] = {};
  bool created = false;
  uint64_t gen = 0;  // context the events belong to
};
Profile g_prof;
std::mutex g_prof_mu;

// INT8 scratch: one buffer per device for the BF16 copies of A and B,
// allocated on the first INT8 call that needs it and grown (never shrunk)
// when a larger problem arrives; kept until the process exits.  An event
// records the last call that used it, and a call on another stream waits
// for that event first, so concurrent calls never share it in flight.
struct Workspace {
  void* ptr = nullptr;
  size_t bytes = 0;
  cudaEvent_t done = nullptr;
  uint64_t gen = 0;  // context the buffer and event belong to
};
Workspace g_ws[kMaxDevices];
std::mutex g_ws_mu;

// Stream-K hand-off flags: one small buffer per device (zeroed when
// allocated) and the sequence number of the last stream-K call; calls use
// the flags in the order the scratch buffer's event imposes on them.
struct StreamKFlags {
  unsigned* ptr = nullptr;
  size_t count = 0;
  unsigned seq = 0;
  uint64_t gen = 0;
};
StreamKFlags g_skf[kMaxDevices];

// Identifier of the calling thread's current CUDA context plus one (0 when
// no context is current yet).  Without the driver's context-id call every
// context reads as 1, and state is then set up once per device.
uint64_t current_context_gen() {
  static PFN_cuCtxGetCurrent_v4000 get_cur = nullptr;
  static PFN_cuCtxGetId_v12000 get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_cur = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
    p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
    cudaGetLastError();
  });
  if (!get_cur || !get_id) return 1;
  CUcontext c = nullptr;
  unsigned long long id = 0;
  if (get_cur(&c) != CUDA_SUCCESS || c == nullptr) return 0;
  if (get_id(c, &id) != CUDA_SUCCESS) return 1;
  return uint64_t(id) + 1;
}

// Per-device set-up, once per context, with that device current: SM count,
// the architecture check and the device address of the status word.  A
// replaced context (cudaDeviceReset) is set up again.
const DeviceInfo* device_info(int* dev_out) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return nullptr;
  }
  *dev_out = dev;
  uint64_t gen = current_context_gen();
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready || (gen != 0 && gen != d.gen)) {
    d = DeviceInfo{};
    d.ready = true;
    int major = 0, minor = 0, sms = 0;
    void* p = nullptr;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor,
                               dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor,
                               dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) ==
            cudaSuccess &&
        major == 10 && minor == 3 &&
        cudaGetSymbolAddress(&p, g_mma_status) == cudaSuccess) {
      d.usable = true;
      d.num_sms = sms;
      d.status = static_cast<unsigned*>(p);
    } else {
      cudaGetLastError();
    }
    // the symbol lookup made the device's primary context current
    if (gen == 0) gen = current_context_gen();
    d.gen = gen != 0 ? gen : 1;
  }
  return d.usable ? &d : nullptr;
}

Ctx make_ctx(void* stream, int dev, const DeviceInfo* info) {
  return Ctx{static_cast<cudaStream_t>(stream), dev, info->num_sms,
             info->status, info->gen};
}

bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

bool ld_ok(int64_t ld, int64_t elem) { return ((ld * elem) & 15) == 0; }

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

__global__ void copy_c_kernel(const uint8_t* __restrict__ C, int64_t ldc_b,
                              uint8_t* __restrict__ D, int64_t ldd_b,
                              int64_t M, int64_t N, int elem) {
  const int64_t total = M * N;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t r = i / N, c = i % N;
    if (elem == 8) {
      const uint64_t v =
          C ? *reinterpret_cast<const uint64_t*>(C + r * ldc_b + c * 8) : 0ull;
      *reinterpret_cast<uint64_t*>(D + r * ldd_b + c * 8) = v;
    } else if (elem == 2) {
      const uint16_t v =
          C ? *reinterpret_cast<const uint16_t*>(C + r * ldc_b + c * 2) : 0u;
      *reinterpret_cast<uint16_t*>(D + r * ldd_b + c * 2) = v;
    } else {
      const uint32_t v =
          C ? *reinterpret_cast<const uint32_t*>(C + r * ldc_b + c * 4) : 0u;
      *reinterpret_cast<uint32_t*>(D + r * ldd_b + c * 4) = v;
    }
  }
}

}  // namespace

bool current_ctx(void* stream, Ctx* out) {
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return false;
  *out = make_ctx(stream, dev, info);
  return true;
}

void attach_profile(Ctx& ctx) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  if (!g_prof.active || g_prof.device != ctx.device || g_prof.gen != ctx.gen ||
      g_prof.count >= kProfMax)
    return;
  ctx.prof_start = g_prof.ev[2 * g_prof.count];
  ctx.prof_stop = g_prof.ev[2 * g_prof.count + 1];
  ++g_prof.count;
}

mma_status_t launch_copy_c(const Ctx& ctx, int64_t M, int64_t N,
                           int elem_bytes, const void* C, int64_t ldc, void* D,
                           int64_t ldd) {
  int64_t blocks = (M * N + 255) / 256;
  if (blocks > int64_t(ctx.num_sms) * 16) blocks = int64_t(ctx.num_sms) * 16;
  copy_c_kernel<<<int(blocks), 256, 0, ctx.stream>>>(
      static_cast<const uint8_t*>(C), ldc * elem_bytes,
      static_cast<uint8_t*>(D), ldd * elem_bytes, M, N, elem_bytes);
  return cudaGetLastError() == cudaSuccess ? MMA_OK : MMA_ERR_LAUNCH;
}

}  // namespace mmagb

using namespace mmagb;

namespace {

// Problems at least this large (M*N*K) take the tcgen05 exact-INT8 path;
// smaller ones stay on the IMMA kernel, which needs no scratch.
constexpr double kI8TensorCoreMinWork = 16777216.0;  // 2^24

// Run `enqueue(workspace)` with at least `need` bytes of the device's
// scratch buffer, growing it if needed, ordered after the buffer's previous
// user (an event) and marking this stream as its new user.
template <class F>
mma_status_t with_workspace(const Ctx& ctx, size_t need, F&& enqueue) {
  std::lock_guard<std::mutex> lk(g_ws_mu);
  Workspace& w = g_ws[ctx.device];
  if (w.gen != ctx.gen) {
    // set up in a context that has since been replaced: its buffer and
    // event went with it
    w = Workspace{};
    w.gen = ctx.gen;
  }
  if (!w.done &&
      cudaEventCreateWithFlags(&w.done, cudaEventDisableTiming) != cudaSuccess) {
    cudaGetLastError();
    w.done = nullptr;
    return MMA_ERR_LAUNCH;
  }
  if (w.bytes < need) {
    if (w.ptr) {
      if (cudaEventSynchronize(w.done) != cudaSuccess) return MMA_ERR_LAUNCH;
      cudaFree(w.ptr);
      w.ptr = nullptr;
      w.bytes = 0;
    }
    const size_t grain = size_t(64) << 20;
    const size_t bytes = (need + grain - 1) / grain * grain;
    if (cudaMalloc(&w.ptr, bytes) != cudaSuccess) {
      cudaGetLastError();
      w.ptr = nullptr;
      return MMA_ERR_NO_MEMORY;
    }
    w.bytes = bytes;
  }
  if (cudaStreamWaitEvent(ctx.stream, w.done, 0) != cudaSuccess)
    return MMA_ERR_LAUNCH;
  const mma_status_t st = enqueue(w.ptr);
  if (cudaEventRecord(w.done, ctx.stream) != cudaSuccess) return MMA_ERR_LAUNCH;
  return st;
}

}  // namespace

namespace {

// Enqueue a stream-K GEMM: partial sums in the scratch buffer, hand-off
// flags with a fresh sequence number.  Runs under the scratch buffer's lock
// (inside with_workspace), which also orders the flags' users.
mma_status_t enqueue_stream_k(const Ctx& ctx, bool bf16, int64_t M, int64_t N,
                              int64_t K, const void* A, int64_t lda,
                              const void* B, int64_t ldb, const void* C,
                              int64_t ldc, void* D, int64_t ldd, void* ws) {
  StreamKFlags& f = g_skf[ctx.device];
  if (f.gen != ctx.gen) f = StreamKFlags{};  // set up in a replaced context
  const size_t need = gemm_sk_flag_count(ctx.num_sms);
  if (f.ptr == nullptr || f.count < need) {
    if (f.ptr) cudaFree(f.ptr);
    f = StreamKFlags{};
    void* p = nullptr;
    if (cudaMalloc(&p, need * sizeof(unsigned)) != cudaSuccess) {
      cudaGetLastError();
      return MMA_ERR_NO_MEMORY;
    }
    if (cudaMemset(p, 0, need * sizeof(unsigned)) != cudaSuccess) {
      cudaFree(p);
      cudaGetLastError();
      return MMA_ERR_LAUNCH;
    }
    f.ptr = static_cast<unsigned*>(p);
    f.count = need;
    f.gen = ctx.gen;
  }
  // nonzero and different from every value still in the flags; after 2^32
  // calls the flags are cleared again before the numbers repeat
  if (++f.seq == 0) {
    if (cudaMemsetAsync(f.ptr, 0, f.count * sizeof(unsigned), ctx.stream) !=
        cudaSuccess)
      return MMA_ERR_LAUNCH;
    f.seq = 1;
  }
  return launch_gemm_sk(ctx, bf16, M, N, K, A, lda, B, ldb,
                        static_cast<const float*>(C), ldc,
                        static_cast<float*>(D), ldd, static_cast<float*>(ws),
                        f.ptr, f.seq);
}

// Element sizes of a supported (dtype_in, dtype_acc) pair, or false.
bool pair_sizes(int in, int acc, int64_t* in_b, int64_t* acc_b) {
  if ((in == MMA_F16 || in == MMA_BF16) && acc == MMA_F32) {
    *in_b = 2;
    *acc_b = 4;
    return true;
  }
  if ((in == MMA_F16 || in == MMA_BF16) && acc == in) {  // 16-bit accumulate
    *in_b = 2;
    *acc_b = 2;
    return true;
  }
  if (in == MMA_I8 && acc == MMA_I32) {
    *in_b = 1;
    *acc_b = 4;
    return true;
  }
  if (in == MMA_F64 && acc == MMA_F64) {
    *in_b = 8;
    *acc_b = 8;
    return true;
  }
  return false;
}

}  // namespace

namespace {

// Argument checks shared by the dense entry points (element sizes eb of A
// and B, ea of C and D).  Returns MMA_OK when the call should go ahead.
mma_status_t check_dense_args(int64_t eb, int64_t ea, int layout_b, int64_t M,
                              int64_t N, int64_t K, const void* A, int64_t lda,
                              const void* B, int64_t ldb, const void* C,
                              int64_t ldc, const void* D, int64_t ldd) {
  if (layout_b != MMA_COL_MAJOR && layout_b != MMA_ROW_MAJOR)
    return MMA_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return MMA_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return MMA_OK;
  const bool b_row = layout_b == MMA_ROW_MAJOR;
  if (D == nullptr || ldd < N) return MMA_ERR_INVALID_ARG;
  if (C != nullptr && ldc < N) return MMA_ERR_INVALID_ARG;
  if (C != nullptr && C == D && ldc != ldd) return MMA_ERR_INVALID_ARG;
  if (K > 0) {
    if (A == nullptr || B == nullptr) return MMA_ERR_INVALID_ARG;
    if (lda < K || ldb < (b_row ? N : K)) return MMA_ERR_INVALID_ARG;
    if (!aligned16(A) || !aligned16(B) || !ld_ok(lda, eb) || !ld_ok(ldb, eb))
      return MMA_ERR_MISALIGNED;
  }
  if (!aligned16(D) || !ld_ok(ldd, ea)) return MMA_ERR_MISALIGNED;
  if (C != nullptr && (!aligned16(C) || !ld_ok(ldc, ea)))
    return MMA_ERR_MISALIGNED;
  return MMA_OK;
}

}  // namespace

extern "C" mma_status_t mma_gemm_ex(int dtype_in, int dtype_acc, int64_t M,
                                    int64_t N, int64_t K, const void* A,
                                    int64_t lda, const void* B, int64_t ldb,
                                    int layout_b, const void* C, int64_t ldc,
                                    void* D, int64_t ldd, void* stream) {
  int64_t eb = 0, ea = 0;
  if (!pair_sizes(dtype_in, dtype_acc, &eb, &ea)) return MMA_ERR_UNSUPPORTED;
  const mma_status_t chk = check_dense_args(eb, ea, layout_b, M, N, K, A, lda,
                                            B, ldb, C, ldc, D, ldd);
  if (chk != MMA_OK || M == 0 || N == 0) return chk;
  const bool b_row = layout_b == MMA_ROW_MAJOR;
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  attach_profile(ctx);

  if (K == 0) return launch_copy_c(ctx, M, N, int(ea), C, ldc, D, ldd);
  switch (dtype_in) {
    case MMA_F16:
    case MMA_BF16: {
      const bool bf16 = dtype_in == MMA_BF16;
      const bool out16 = dtype_acc != MMA_F32;
      // fewer output tiles than SMs: K split across every SM (stream-K)
      if (!b_row && !out16 && gemm_sk_fits(ctx.num_sms, M, N, K))
        return with_workspace(ctx, gemm_sk_workspace_bytes(ctx.num_sms),
                              [&](void* ws) {
                                return enqueue_stream_k(ctx, bf16, M, N, K, A,
                                                        lda, B, ldb, C, ldc, D,
                                                        ldd, ws);
                              });
      if (!b_row)
        return launch_gemm_tc_f16(ctx, bf16, out16, M, N, K, A, lda, B, ldb, C,
                                  ldc, D, ldd);
      return with_workspace(ctx, gemm_tc_rowb_workspace_bytes(N, K),
                            [&](void* ws) {
                              return launch_gemm_tc_f16_rowb(
                                  ctx, bf16, out16, M, N, K, A, lda, B, ldb, C,
                                  ldc, D, ldd, ws);
                            });
    }
    case MMA_I8: {
      const int8_t* A8 = static_cast<const int8_t*>(A);
      const int8_t* B8 = static_cast<const int8_t*>(B);
      const int32_t* Ci = static_cast<const int32_t*>(C);
      int32_t* Di = static_cast<int32_t*>(D);
      // Large problems, and every row-major B, take the tensor-pipe path.
      if (b_row || double(M) * double(N) * double(K) >= kI8TensorCoreMinWork)
        return with_workspace(ctx, gemm_i8_tc_workspace_bytes(M, N, K),
                              [&](void* ws) {
                                return launch_gemm_i8_tc(
                                    ctx, M, N, K, A8, lda, B8, ldb, Ci, ldc,
                                    Di, ldd, ws, b_row, true, true, false);
                              });
      return launch_gemm_i8_imma(ctx, M, N, K, A8, lda, B8, ldb, Ci, ldc, Di,
                                 ldd);
    }
    case MMA_F64:
      return launch_gemm_f64(ctx, M, N, K, static_cast<const double*>(A), lda,
                             static_cast<const double*>(B), ldb, b_row,
                             static_cast<const double*>(C), ldc,
                             static_cast<double*>(D), ldd);
    default:
      return MMA_ERR_UNSUPPORTED;
  }
}

extern "C" mma_status_t mma_gemm_i8_ex(int64_t M, int64_t N, int64_t K,
                                       const void* A, int64_t lda, int a_neg,
                                       const void* B, int64_t ldb, int b_neg,
                                       int layout_b, const void* C,
                                       int64_t ldc, void* D, int64_t ldd,
                                       int clamp, void* stream) {
  const bool a_signed = a_neg != 0, b_signed = b_neg != 0;
  // signed x signed without saturation is the plain INT8 product
  if (a_signed && b_signed && clamp == 0)
    return mma_gemm_ex(MMA_I8, MMA_I32, M, N, K, A, lda, B, ldb, layout_b, C,
                       ldc, D, ldd, stream);
  const mma_status_t chk = check_dense_args(1, 4, layout_b, M, N, K, A, lda,
                                            B, ldb, C, ldc, D, ldd);
  if (chk != MMA_OK || M == 0 || N == 0) return chk;
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  attach_profile(ctx);
  if (K == 0) {
    // D = C: a 32-bit C is in range, so saturation changes nothing
    return launch_copy_c(ctx, M, N, 4, C, ldc, D, ldd);
  }
  const bool b_row = layout_b == MMA_ROW_MAJOR;
  return with_workspace(
      ctx, gemm_i8_tc_workspace_bytes(M, N, K), [&](void* ws) {
        return launch_gemm_i8_tc(ctx, M, N, K, static_cast<const int8_t*>(A),
                                 lda, static_cast<const int8_t*>(B), ldb,
                                 static_cast<const int32_t*>(C), ldc,
                                 static_cast<int32_t*>(D), ldd, ws, b_row,
                                 a_signed, b_signed, clamp != 0);
      });
}

extern "C" mma_status_t mma_gemm(int dtype_in, int dtype_acc, int64_t M,
                                 int64_t N, int64_t K, const void* A,
                                 int64_t lda, const void* B, int64_t ldb,
                                 const void* C, int64_t ldc, void* D,
                                 int64_t ldd, void* stream) {
  return mma_gemm_ex(dtype_in, dtype_acc, M, N, K, A, lda, B, ldb,
                     MMA_COL_MAJOR, C, ldc, D, ldd, stream);
}

extern "C" mma_status_t mma_gemm_batched_ex(
    int dtype_in, int dtype_acc, int64_t M, int64_t N, int64_t K,
    const void* A, int64_t lda, const void* B, int64_t ldb, const void* C,
    int64_t ldc, void* D, int64_t ldd, int64_t batch, int a_broadcast_group,
    int a_broadcast_id, int b_lane_group_pattern, void* stream) {
  int64_t eb = 0, ea = 0;
  if (!pair_sizes(dtype_in, dtype_acc, &eb, &ea)) return MMA_ERR_UNSUPPORTED;
  const int G = a_broadcast_group;
  const int blgp = b_lane_group_pattern;
  if (G != 1 && G != 2 && G != 4 && G != 8 && G != 16)
    return MMA_ERR_INVALID_ARG;
  if (a_broadcast_id < 0 || a_broadcast_id >= G) return MMA_ERR_INVALID_ARG;
  if (blgp < 0 || blgp > 7) return MMA_ERR_INVALID_ARG;
  if (batch < 0 || batch % G != 0) return MMA_ERR_INVALID_ARG;
  if (blgp != 0 && batch % 4 != 0) return MMA_ERR_INVALID_ARG;
  if (batch > int64_t(INT32_MAX)) return MMA_ERR_UNSUPPORTED;
  if (M < 0 || N < 0 || K < 0) return MMA_ERR_INVALID_ARG;
  if (batch == 0) return MMA_OK;
  // each tile is checked as a single column-major-B problem
  const mma_status_t chk = check_dense_args(eb, ea, MMA_COL_MAJOR, M, N, K, A,
                                            lda, B, ldb, C, ldc, D, ldd);
  if (chk != MMA_OK || batch == 0 || M == 0 || N == 0) return chk;
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  attach_profile(ctx);
  // K == 0: D = C tile by tile; the tiles are contiguous, so batch * M rows
  if (K == 0) return launch_copy_c(ctx, batch * M, N, int(ea), C, ldc, D, ldd);
  const int abid = a_broadcast_id;
  switch (dtype_in) {
    case MMA_F16:
    case MMA_BF16: {
      const bool bf16 = dtype_in == MMA_BF16;
      const bool out16 = dtype_acc != MMA_F32;
      // 16 x 16 x 16 FP32-accumulate tiles stored densely: the HBM-streaming
      // kernel; every other shape: the tcgen05 kernel over 3-D tensor maps
      if (!out16 && M == 16 && N == 16 && K == 16 && lda == 16 && ldb == 16 &&
          ldd == 16 && (C == nullptr || ldc == 16))
        return launch_batched16(ctx, bf16, batch, G, abid, blgp, A, B,
                                static_cast<const float*>(C),
                                static_cast<float*>(D));
      // mid-size dense blocks in multiples of 64: CTA-cooperative tiles
      if (batched_tile_fits(M, N, K, lda, ldb, ldc, ldd, C != nullptr))
        return launch_batched_tile(ctx, bf16, out16, M, N, K, A, B, C, D,
                                   batch, G, abid, blgp);
      // small and mid-size dense blocks: warp-level MMAs streaming from HBM
      if (batched_mma_fits(M, N, K, lda, ldb, ldc, ldd, C != nullptr, false))
        return launch_batched_mma(ctx, bf16, out16, M, N, K, A, B, C, D, batch,
                                  G, abid, blgp);
      return launch_gemm_tc_batched(ctx, bf16, out16, M, N, K, A, lda, B, ldb,
                                    C, ldc, D, ldd, batch, G, abid, blgp);
    }
    case MMA_I8:
      // small and mid-size dense blocks: integer warp-level MMAs, exact
      if (batched_mma_fits(M, N, K, lda, ldb, ldc, ldd, C != nullptr, true))
        return launch_batched_i8_mma(ctx, M, N, K, A, B, C, D, batch, G, abid,
                                     blgp);
      return with_workspace(
          ctx, gemm_i8_tc_batched_workspace_bytes(M, N, K, batch),
          [&](void* ws) {
            return launch_gemm_i8_tc_batched(
                ctx, M, N, K, static_cast<const int8_t*>(A), lda,
                static_cast<const int8_t*>(B), ldb,
                static_cast<const int32_t*>(C), ldc, static_cast<int32_t*>(D),
                ldd, batch, G, abid, blgp, ws);
          });
    case MMA_F64:
      return launch_gemm_f64_batched(ctx, M, N, K,
                                     static_cast<const double*>(A), lda,
                                     static_cast<const double*>(B), ldb,
                                     static_cast<const double*>(C), ldc,
                                     static_cast<double*>(D), ldd, batch, G,
                                     abid, blgp);
    default:
      return MMA_ERR_UNSUPPORTED;
  }
}

extern "C" mma_status_t mma_gemm_batched(int dtype_in, int dtype_acc,
                                         int64_t M, int64_t N, int64_t K,
                                         const void* A, int64_t lda,
                                         const void* B, int64_t ldb,
                                         const void* C, int64_t ldc, void* D,
                                         int64_t ldd, int64_t batch,
                                         int a_broadcast_group,
                                         int a_broadcast_id, void* stream) {
  return mma_gemm_batched_ex(dtype_in, dtype_acc, M, N, K, A, lda, B, ldb, C,
                             ldc, D, ldd, batch, a_broadcast_group,
                             a_broadcast_id, 0, stream);
}

extern "C" mma_status_t mma_device_status(void* stream) {
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess)
    return MMA_ERR_LAUNCH;
  unsigned v = 0;
  if (cudaMemcpyFromSymbol(&v, g_mma_status, sizeof(v)) != cudaSuccess)
    return MMA_ERR_LAUNCH;
  if (v != 0) {
    const unsigned zero = 0;
    if (cudaMemcpyToSymbol(g_mma_status, &zero, sizeof(zero)) != cudaSuccess)
      return MMA_ERR_LAUNCH;
    return MMA_ERR_TIMEOUT;
  }
  return MMA_OK;
}

extern "C" mma_status_t mma_profile_begin(void) {
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  std::lock_guard<std::mutex> lk(g_prof_mu);
  if (g_prof.created && g_prof.device != dev) return MMA_ERR_INVALID_ARG;
  if (g_prof.created && g_prof.gen != info->gen) {
    // the events belonged to a context that has since been replaced
    g_prof.created = false;
  }
  if (!g_prof.created) {
    for (int i = 0; i < 2 * kProfMax; ++i) {
      if (cudaEventCreate(&g_prof.ev[i]) != cudaSuccess) {
        for (int j = 0; j < i; ++j) cudaEventDestroy(g_prof.ev[j]);
        cudaGetLastError();
        return MMA_ERR_LAUNCH;
      }
    }
    g_prof.created = true;
    g_prof.device = dev;
    g_prof.gen = info->gen;
  }
  g_prof.active = true;
  g_prof.count = 0;
  return MMA_OK;
}

extern "C" mma_status_t mma_profile_end(float* ms, int max_count,
                                        int* count) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  if (!g_prof.active) return MMA_ERR_INVALID_ARG;
  g_prof.active = false;
  const int n = g_prof.count < max_count ? g_prof.count : max_count;
  if (count) *count = g_prof.count;
  for (int i = 0; i < n; ++i) {
    if (cudaEventSynchronize(g_prof.ev[2 * i + 1]) != cudaSuccess ||
        cudaEventElapsedTime(&ms[i], g_prof.ev[2 * i], g_prof.ev[2 * i + 1]) !=
            cudaSuccess) {
      cudaGetLastError();
      return MMA_ERR_LAUNCH;
    }
  }
  return MMA_OK;
}

extern "C" const char* mma_status_string(int status) {
  switch (status) {
    case MMA_OK: return "MMA_OK";
    case MMA_ERR_INVALID_ARG: return "MMA_ERR_INVALID_ARG";
    case MMA_ERR_UNSUPPORTED: return "MMA_ERR_UNSUPPORTED";
    case MMA_ERR_MISALIGNED: return "MMA_ERR_MISALIGNED";
    case MMA_ERR_LAUNCH: return "MMA_ERR_LAUNCH";
    case MMA_ERR_TIMEOUT: return "MMA_ERR_TIMEOUT";
    case MMA_ERR_NO_DEVICE: return "MMA_ERR_NO_DEVICE";
    case MMA_ERR_NO_MEMORY: return "MMA_ERR_NO_MEMORY";
    default: return "MMA_ERR_UNKNOWN";
  }
}

extern "C" int mma_version(void) { return 200; }

// ---------------------------- 8-bit operands and products grouped by expert

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool dim_ok(int64_t d) { return d >= 0 && d <= kMaxDim; }

// Element size of a 16- or 32-bit floating-point type, or 0.
int64_t float_bytes(int type) {
  return type == MMA_F32 ? 4 : type == MMA_F16 || type == MMA_BF16 ? 2 : 0;
}

bool is_f8(int type) { return type == MMA_F8E4M3 || type == MMA_F8E5M2; }

// An input of `rows` rows of `len` elements: 16-byte rows.
mma_status_t check_in(const void* p, int64_t ld, int64_t len, int64_t eb) {
  if (p == nullptr || ld < len) return MMA_ERR_INVALID_ARG;
  return aligned16(p) && ld_ok(ld, eb) ? MMA_OK : MMA_ERR_MISALIGNED;
}

// An output (or C): rows of `len` elements, aligned to one element.
mma_status_t check_out(const void* p, int64_t ld, int64_t len, int64_t eb) {
  if (p == nullptr || ld < len) return MMA_ERR_INVALID_ARG;
  return (reinterpret_cast<uintptr_t>(p) & uintptr_t(eb - 1)) == 0
             ? MMA_OK
             : MMA_ERR_MISALIGNED;
}

mma_status_t check_scales(const float* s, int64_t row, int64_t blk) {
  if (s == nullptr || row < 0 || blk < 0) return MMA_ERR_INVALID_ARG;
  return aligned4(s) ? MMA_OK : MMA_ERR_MISALIGNED;
}

// D of a product, and C, which may be NULL or D itself.
mma_status_t check_cd(const void* C, int64_t ldc, const void* D, int64_t ldd,
                      int64_t len, int64_t eb) {
  mma_status_t st = check_out(D, ldd, len, eb);
  if (st != MMA_OK || C == nullptr) return st;
  if (C == D && ldc != ldd) return MMA_ERR_INVALID_ARG;
  return check_out(C, ldc, len, eb);
}

// Slices of `rows` rows of `len` elements, `stride` elements apart.
bool slices_ok(int64_t groups, int64_t stride, int64_t rows, int64_t ld,
               int64_t len) {
  return groups <= 1 || stride >= (rows - 1) * ld + len;
}

#define MMA_CHECK(expr)                       \
  do {                                        \
    const mma_status_t st_ = (expr);          \
    if (st_ != MMA_OK) return st_;            \
  } while (0)

mma_status_t gemm_f8(int type_a, int type_b, int type_d, int64_t groups,
                     int64_t M, int64_t N, int64_t K, const void* A,
                     int64_t lda, const float* SA, int64_t sa_row,
                     int64_t sa_blk, const void* B, int64_t ldb,
                     int64_t stride_b, const float* SB, int sb_rows,
                     int64_t sb_group, int64_t sb_row, int64_t sb_blk,
                     bool grouped, const int32_t* offsets, const void* C,
                     int64_t ldc, void* D, int64_t ldd, void* stream) {
  const int64_t eb = float_bytes(type_d);
  if (!is_f8(type_a) || !is_f8(type_b) || eb == 0) return MMA_ERR_UNSUPPORTED;
  if (!dim_ok(M) || !dim_ok(N) || !dim_ok(K) || groups < 0)
    return MMA_ERR_INVALID_ARG;
  if (sb_rows != 1 && sb_rows != 128) return MMA_ERR_INVALID_ARG;
  if (groups > kMaxGroups) return MMA_ERR_UNSUPPORTED;
  if (groups == 0 || M == 0 || N == 0) return MMA_OK;
  if (grouped && offsets == nullptr) return MMA_ERR_INVALID_ARG;
  if (grouped && !aligned4(offsets)) return MMA_ERR_MISALIGNED;
  MMA_CHECK(check_cd(C, ldc, D, ldd, N, eb));
  if (K > 0) {
    if (sb_group < 0 || !slices_ok(groups, stride_b, N, ldb, K))
      return MMA_ERR_INVALID_ARG;
    MMA_CHECK(check_scales(SA, sa_row, sa_blk));
    MMA_CHECK(check_scales(SB, sb_row, sb_blk));
    MMA_CHECK(check_in(A, lda, K, 1));
    MMA_CHECK(check_in(B, ldb, K, 1));
    if (groups > 1 && !ld_ok(stride_b, 1)) return MMA_ERR_MISALIGNED;
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  attach_profile(ctx);
  F8Problem f = {};
  f.a_e5m2 = type_a == MMA_F8E5M2;
  f.b_e5m2 = type_b == MMA_F8E5M2;
  f.d_type = type_d;
  f.groups = groups;
  f.rows = M;
  f.N = N;
  f.K = K;
  f.A = A;
  f.lda = lda;
  f.SA = SA;
  f.sa_row = sa_row;
  f.sa_blk = sa_blk;
  f.B = B;
  f.ldb = ldb;
  f.stride_b = stride_b;
  f.SB = SB;
  f.sb_rows = sb_rows;
  f.sb_group = sb_group;
  f.sb_row = sb_row;
  f.sb_blk = sb_blk;
  f.offsets = offsets;
  f.C = C;
  f.ldc = ldc;
  f.D = D;
  f.ldd = ldd;
  return launch_gemm_f8(ctx, f);
}

}  // namespace

extern "C" mma_status_t mma_gemm_f8(
    int type_a, int type_b, int type_d, int64_t M, int64_t N, int64_t K,
    const void* A, int64_t lda, const float* SA, int64_t sa_row,
    int64_t sa_blk, const void* B, int64_t ldb, const float* SB, int sb_rows,
    int64_t sb_row, int64_t sb_blk, const void* C, int64_t ldc, void* D,
    int64_t ldd, void* stream) {
  return gemm_f8(type_a, type_b, type_d, 1, M, N, K, A, lda, SA, sa_row, sa_blk,
                 B, ldb, 0, SB, sb_rows, 0, sb_row, sb_blk, false, nullptr, C,
                 ldc, D, ldd, stream);
}

extern "C" mma_status_t mma_gemm_grouped_f8(
    int type_a, int type_b, int type_d, int64_t groups, int64_t T, int64_t N,
    int64_t K, const void* A, int64_t lda, const float* SA, int64_t sa_row,
    int64_t sa_blk, const void* B, int64_t ldb, int64_t stride_b,
    const float* SB, int sb_rows, int64_t sb_group, int64_t sb_row,
    int64_t sb_blk, const int32_t* offsets, const void* C, int64_t ldc, void* D,
    int64_t ldd, void* stream) {
  return gemm_f8(type_a, type_b, type_d, groups, T, N, K, A, lda, SA, sa_row,
                 sa_blk, B, ldb, stride_b, SB, sb_rows, sb_group, sb_row, sb_blk,
                 true, offsets, C, ldc, D, ldd, stream);
}

extern "C" mma_status_t mma_gemm_grouped(
    int type_in, int type_d, int64_t groups, int64_t T, int64_t N, int64_t K,
    const void* A, int64_t lda, const void* B, int64_t ldb, int64_t stride_b,
    int layout_b, const int32_t* offsets, const void* C, int64_t ldc, void* D,
    int64_t ldd, void* stream) {
  if ((type_in != MMA_F16 && type_in != MMA_BF16) ||
      (type_d != type_in && type_d != MMA_F32))
    return MMA_ERR_UNSUPPORTED;
  if (layout_b != MMA_COL_MAJOR && layout_b != MMA_ROW_MAJOR)
    return MMA_ERR_INVALID_ARG;
  if (!dim_ok(T) || !dim_ok(N) || !dim_ok(K) || groups < 0)
    return MMA_ERR_INVALID_ARG;
  if (groups > kMaxGroups) return MMA_ERR_UNSUPPORTED;
  if (groups == 0 || T == 0 || N == 0) return MMA_OK;
  const bool row = layout_b == MMA_ROW_MAJOR;
  if (offsets == nullptr) return MMA_ERR_INVALID_ARG;
  if (!aligned4(offsets)) return MMA_ERR_MISALIGNED;
  MMA_CHECK(check_cd(C, ldc, D, ldd, N, float_bytes(type_d)));
  if (K > 0) {
    if (!slices_ok(groups, stride_b, row ? K : N, ldb, row ? N : K))
      return MMA_ERR_INVALID_ARG;
    MMA_CHECK(check_in(A, lda, K, 2));
    MMA_CHECK(check_in(B, ldb, row ? N : K, 2));
    if (groups > 1 && !ld_ok(stride_b, 2)) return MMA_ERR_MISALIGNED;
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  attach_profile(ctx);
  GroupedProblem g = {};
  g.bf16 = type_in == MMA_BF16;
  g.b_row_major = row;
  g.d_type = type_d;
  g.groups = groups;
  g.rows = T;
  g.N = N;
  g.K = K;
  g.A = A;
  g.lda = lda;
  g.B = B;
  g.ldb = ldb;
  g.stride_b = stride_b;
  g.offsets = offsets;
  g.C = C;
  g.ldc = ldc;
  g.D = D;
  g.ldd = ldd;
  return launch_gemm_grouped(ctx, g);
}

extern "C" mma_status_t mma_gemm_grouped_wgrad(
    int type_in, int type_d, int64_t groups, int64_t T, int64_t N, int64_t K,
    const void* DY, int64_t lddy, const void* X, int64_t ldx,
    const int32_t* offsets, const void* C, int64_t ldc, int64_t stride_c,
    void* D, int64_t ldd, int64_t stride_d, void* stream) {
  if ((type_in != MMA_F16 && type_in != MMA_BF16) ||
      (type_d != type_in && type_d != MMA_F32))
    return MMA_ERR_UNSUPPORTED;
  if (!dim_ok(T) || !dim_ok(N) || !dim_ok(K) || groups < 0)
    return MMA_ERR_INVALID_ARG;
  if (groups > kMaxGroups) return MMA_ERR_UNSUPPORTED;
  if (groups == 0 || N == 0 || K == 0) return MMA_OK;
  if (offsets == nullptr) return MMA_ERR_INVALID_ARG;
  if (!aligned4(offsets)) return MMA_ERR_MISALIGNED;
  MMA_CHECK(check_cd(C, ldc, D, ldd, K, float_bytes(type_d)));
  if (!slices_ok(groups, stride_d, N, ldd, K) ||
      (C != nullptr && !slices_ok(groups, stride_c, N, ldc, K)) ||
      (C != nullptr && C == D && groups > 1 && stride_c != stride_d))
    return MMA_ERR_INVALID_ARG;
  if (T > 0) {
    MMA_CHECK(check_in(DY, lddy, N, 2));
    MMA_CHECK(check_in(X, ldx, K, 2));
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  attach_profile(ctx);
  WgradProblem g = {};
  g.bf16 = type_in == MMA_BF16;
  g.d_type = type_d;
  g.groups = groups;
  g.rows = T;
  g.N = N;
  g.K = K;
  g.DY = DY;
  g.lddy = lddy;
  g.X = X;
  g.ldx = ldx;
  g.offsets = offsets;
  g.C = C;
  g.ldc = ldc;
  g.stride_c = stride_c;
  g.D = D;
  g.ldd = ldd;
  g.stride_d = stride_d;
  return launch_gemm_grouped_wgrad(ctx, g);
}

namespace {

// Both norms (B and DB: the layer norm's bias and its gradient).
mma_status_t norm(bool centre, const NormProblem& p, void* stream) {
  const int64_t eb = float_bytes(p.type);
  if (eb == 0 || (p.w_type != p.type && p.w_type != MMA_F32)) return MMA_ERR_UNSUPPORTED;
  if (!dim_ok(p.M) || !dim_ok(p.N) || !(p.eps >= 0.f)) return MMA_ERR_INVALID_ARG;
  if (p.M == 0 || p.N == 0) return MMA_OK;
  if (p.Y == nullptr && p.Q == nullptr) return MMA_ERR_INVALID_ARG;
  if ((p.H != nullptr && p.H == p.X && p.ldh != p.ldx) ||
      (p.H != nullptr && p.H == p.R && p.ldh != p.ldr))
    return MMA_ERR_INVALID_ARG;
  MMA_CHECK(check_in(p.X, p.ldx, p.N, eb));
  if (p.R) MMA_CHECK(check_in(p.R, p.ldr, p.N, eb));
  MMA_CHECK(check_in(p.W, p.N, p.N, 16));
  if (p.B) MMA_CHECK(check_in(p.B, p.N, p.N, 16));
  if (p.H) MMA_CHECK(check_in(p.H, p.ldh, p.N, eb));
  if (p.Y) MMA_CHECK(check_in(p.Y, p.ldy, p.N, eb));
  if (p.Q) {
    MMA_CHECK(check_scales(p.S, p.s_row, p.s_blk));
    MMA_CHECK(check_in(p.Q, p.ldq, p.N, 1));
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  return centre ? launch_layernorm(ctx, p) : launch_rmsnorm(ctx, p);
}

mma_status_t norm_backward(bool centre, const NormBackProblem& p, void* workspace,
                           int64_t workspace_bytes, void* stream) {
  const int64_t eb = float_bytes(p.type);
  if (eb == 0 || (p.w_type != p.type && p.w_type != MMA_F32)) return MMA_ERR_UNSUPPORTED;
  if (!dim_ok(p.M) || !dim_ok(p.N) || !(p.eps >= 0.f)) return MMA_ERR_INVALID_ARG;
  if (p.N == 0) return MMA_OK;
  if (p.DW == nullptr || (centre && p.DB == nullptr)) return MMA_ERR_INVALID_ARG;
  if (!aligned4(p.DW) || !aligned4(p.DB)) return MMA_ERR_MISALIGNED;
  const int64_t need = centre ? layernorm_backward_workspace_bytes(p.M, p.N)
                              : rmsnorm_backward_workspace_bytes(p.M, p.N);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return MMA_ERR_INVALID_ARG;
  if (need > 0 && !aligned4(workspace)) return MMA_ERR_MISALIGNED;
  if (p.M > 0) {
    if ((p.DX == p.DY && p.lddx != p.lddy) ||
        (p.R != nullptr && p.DX == p.R && p.lddx != p.ldr))
      return MMA_ERR_INVALID_ARG;
    MMA_CHECK(check_in(p.DY, p.lddy, p.N, eb));
    MMA_CHECK(check_in(p.H, p.ldh, p.N, eb));
    MMA_CHECK(check_in(p.W, p.N, p.N, 16));
    if (p.R) MMA_CHECK(check_in(p.R, p.ldr, p.N, eb));
    MMA_CHECK(check_in(p.DX, p.lddx, p.N, eb));
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  return centre ? launch_layernorm_backward(ctx, p, workspace)
                : launch_rmsnorm_backward(ctx, p, workspace);
}

}  // namespace

extern "C" mma_status_t mma_rmsnorm_f8(
    int type, int w_type, int64_t M, int64_t N, const void* X, int64_t ldx,
    const void* R, int64_t ldr, const void* W, float eps, int pow2, void* H,
    int64_t ldh, void* Y, int64_t ldy, void* Q, int64_t ldq, float* S,
    int64_t s_row, int64_t s_blk, void* stream) {
  return norm(false, NormProblem{type, w_type, M, N, X, ldx, R, ldr, W, eps, pow2 != 0,
                                 H, ldh, Y, ldy, Q, ldq, S, s_row, s_blk}, stream);
}

extern "C" mma_status_t mma_layernorm(
    int type, int w_type, int64_t M, int64_t N, const void* X, int64_t ldx,
    const void* R, int64_t ldr, const void* W, const void* B, float eps, int pow2,
    void* H, int64_t ldh, void* Y, int64_t ldy, void* Q, int64_t ldq, float* S,
    int64_t s_row, int64_t s_blk, void* stream) {
  return norm(true, NormProblem{type, w_type, M, N, X, ldx, R, ldr, W, eps, pow2 != 0,
                                H, ldh, Y, ldy, Q, ldq, S, s_row, s_blk, B}, stream);
}

extern "C" int64_t mma_rmsnorm_backward_workspace(int64_t M, int64_t N) {
  return dim_ok(M) && dim_ok(N) ? rmsnorm_backward_workspace_bytes(M, N) : 0;
}

extern "C" int64_t mma_layernorm_backward_workspace(int64_t M, int64_t N) {
  return dim_ok(M) && dim_ok(N) ? layernorm_backward_workspace_bytes(M, N) : 0;
}

extern "C" mma_status_t mma_rmsnorm_backward(
    int type, int w_type, int64_t M, int64_t N, const void* DY, int64_t lddy,
    const void* H, int64_t ldh, const void* W, float eps, const void* R,
    int64_t ldr, void* DX, int64_t lddx, float* DW, void* workspace,
    int64_t workspace_bytes, void* stream) {
  return norm_backward(false, NormBackProblem{type, w_type, M, N, DY, lddy, H, ldh, W, eps,
                                              R, ldr, DX, lddx, DW, nullptr},
                       workspace, workspace_bytes, stream);
}

extern "C" mma_status_t mma_layernorm_backward(
    int type, int w_type, int64_t M, int64_t N, const void* DY, int64_t lddy,
    const void* H, int64_t ldh, const void* W, float eps, const void* R,
    int64_t ldr, void* DX, int64_t lddx, float* DW, float* DB, void* workspace,
    int64_t workspace_bytes, void* stream) {
  return norm_backward(true, NormBackProblem{type, w_type, M, N, DY, lddy, H, ldh, W, eps,
                                             R, ldr, DX, lddx, DW, DB},
                       workspace, workspace_bytes, stream);
}

extern "C" mma_status_t mma_quantize_f8(
    int type, int f8_type, int64_t M, int64_t N, int block_rows, int transpose,
    int pow2, const void* X, int64_t ldx, void* Q, int64_t ldq, float* S,
    int64_t s_row, int64_t s_blk, void* stream) {
  const int64_t eb = float_bytes(type);
  if (eb == 0 || !is_f8(f8_type)) return MMA_ERR_UNSUPPORTED;
  if (!dim_ok(M) || !dim_ok(N) || (block_rows != 1 && block_rows != 128))
    return MMA_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return MMA_OK;
  MMA_CHECK(check_in(X, ldx, N, eb));
  MMA_CHECK(check_in(Q, ldq, transpose ? M : N, 1));
  MMA_CHECK(check_scales(S, s_row, s_blk));
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  return launch_quantize_f8(ctx, QuantProblem{type, f8_type == MMA_F8E5M2,
                                              transpose != 0, pow2 != 0,
                                              block_rows, M, N, X, ldx, Q, ldq,
                                              S, s_row, s_blk});
}

// ------------------------------------------------- router of a layer of experts

namespace {

// What both directions ask of the sizes; choices are counted in ints, those of
// the last block's rounding among them.
mma_status_t check_route(int type, int64_t T, int64_t E, int64_t k) {
  if (float_bytes(type) == 0) return MMA_ERR_UNSUPPORTED;
  if (!dim_ok(T) || E < 1 || k < 1 || k > E) return MMA_ERR_INVALID_ARG;
  if (E > kMaxGroups || k > MMA_MAX_CHOICES || T * k > (int64_t(1) << 30))
    return MMA_ERR_UNSUPPORTED;
  return MMA_OK;
}

mma_status_t check_words(const void* p) {
  return p == nullptr ? MMA_ERR_INVALID_ARG : aligned4(p) ? MMA_OK : MMA_ERR_MISALIGNED;
}

}  // namespace

extern "C" int64_t mma_route_workspace(int64_t T, int64_t E) {
  return dim_ok(T) && E >= 1 && E <= kMaxGroups ? route_workspace_bytes(T, E) : 0;
}

extern "C" mma_status_t mma_route(int type, int64_t T, int64_t E, int64_t k,
                                  const void* X, int64_t ldx, const uint8_t* mask,
                                  int normalize, float* weights, int32_t* experts,
                                  int32_t* order, int32_t* place, int32_t* offsets,
                                  float* share, float* loss, int32_t* tokens,
                                  void* workspace, int64_t workspace_bytes,
                                  void* stream) {
  MMA_CHECK(check_route(type, T, E, k));
  for (const void* q : {static_cast<const void*>(offsets), static_cast<const void*>(share),
                        static_cast<const void*>(loss), static_cast<const void*>(tokens)})
    MMA_CHECK(check_words(q));
  if (T > 0) {
    MMA_CHECK(check_out(X, ldx, E, float_bytes(type)));
    for (const void* q : {static_cast<const void*>(weights), static_cast<const void*>(experts),
                          static_cast<const void*>(order), static_cast<const void*>(place)})
      MMA_CHECK(check_words(q));
  }
  const int64_t need = route_workspace_bytes(T, E);
  if (need > 0) {
    MMA_CHECK(check_words(workspace));
    if (workspace_bytes < need) return MMA_ERR_INVALID_ARG;
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  return launch_route(ctx, RouteProblem{type, T, E, k, X, ldx, mask, normalize != 0, weights,
                                        experts, order, place, offsets, share, loss, tokens},
                      workspace);
}

extern "C" mma_status_t mma_route_backward(
    int type, int64_t T, int64_t E, int64_t k, const void* X, int64_t ldx,
    const uint8_t* mask, int normalize, const float* weights, const int32_t* experts,
    const int32_t* offsets, const int32_t* tokens, const float* DW, const float* DLOSS,
    void* DX, int64_t lddx, void* stream) {
  MMA_CHECK(check_route(type, T, E, k));
  if (T == 0) return MMA_OK;
  const int64_t eb = float_bytes(type);
  MMA_CHECK(check_out(X, ldx, E, eb));
  MMA_CHECK(check_out(DX, lddx, E, eb));
  if (DX == X && lddx != ldx) return MMA_ERR_INVALID_ARG;
  if (DW) {
    MMA_CHECK(check_words(DW));
    MMA_CHECK(check_words(experts));
    if (normalize) MMA_CHECK(check_words(weights));
  }
  if (DLOSS) {
    MMA_CHECK(check_words(DLOSS));
    MMA_CHECK(check_words(offsets));
    MMA_CHECK(check_words(tokens));
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  return launch_route_backward(
      ctx, RouteBackProblem{type, T, E, k, X, ldx, mask, normalize != 0, weights, experts,
                            offsets, tokens, DW, DLOSS, DX, lddx});
}

// ------------------------------------------------------------ low-rank adapters

namespace {

mma_status_t check_lora(int type_in, int type_d, int64_t T, int64_t N, int64_t K,
                        int64_t rank, int64_t requests, const int32_t* offsets,
                        int64_t adapters_total) {
  if ((type_in != MMA_F16 && type_in != MMA_BF16) ||
      (type_d != type_in && type_d != MMA_F32))
    return MMA_ERR_UNSUPPORTED;
  if (!dim_ok(T) || !dim_ok(N) || !dim_ok(K) || rank < 0 || requests < 0 ||
      adapters_total < 0)
    return MMA_ERR_INVALID_ARG;
  // (the kernels' counters go on by up to 8192 past an end)
  constexpr int64_t kMost = INT32_MAX - 65535;
  if (rank > MMA_MAX_RANK || requests > MMA_MAX_REQUESTS || adapters_total > 65535 ||
      T > kMost || N > kMost || K > kMost)
    return MMA_ERR_UNSUPPORTED;
  return rank > 0 && T > 0 ? check_words(offsets) : MMA_OK;
}

// The rows' sums: FP32, rows of at least `rank`.
mma_status_t check_sums(const float* s, int64_t ld, int64_t rank) {
  if (s == nullptr || ld < rank) return MMA_ERR_INVALID_ARG;
  return aligned4(s) ? MMA_OK : MMA_ERR_MISALIGNED;
}

// The workspace: the adapters' rows, then the sums in 16 bits.
struct LoraSpace {
  int64_t extra, halves;
};

LoraSpace lora_space(int type_in, int type_d, int64_t T, int64_t N, int64_t rank,
                     int64_t requests) {
  const bool every = lora_every(T, requests);
  const int64_t rows = lora_own_places(T, requests) ? T : requests * (kLoraRows - 1);
  const int64_t parts = every ? 0 : lora_parts(type_in == MMA_BF16, type_d);
  return LoraSpace{(rows * N * 4 + 15) / 16 * 16,
                   parts * T * lora_ld16(type_in == MMA_BF16, rank) * 2};
}

}  // namespace

extern "C" int64_t mma_gemm_lora_workspace(int type_in, int type_d, int64_t T, int64_t N,
                                           int64_t rank, int64_t requests) {
  if (!dim_ok(T) || !dim_ok(N) || rank < 1 || rank > MMA_MAX_RANK || requests < 0 ||
      requests > MMA_MAX_REQUESTS)
    return 0;
  const LoraSpace s = lora_space(type_in, type_d, T, N, rank, requests);
  return s.extra + s.halves;
}

extern "C" mma_status_t mma_gemm_lora(
    int type_in, int type_d, int64_t T, int64_t N, int64_t K, int64_t rank, const void* X,
    int64_t ldx, const void* W, int64_t ldw, const void* A, int64_t lda, int64_t stride_a,
    const void* B, int64_t ldb, int64_t stride_b, int layout, int64_t requests,
    const int32_t* offsets, const int32_t* adapters, int64_t adapters_total,
    const float* scales, const void* C, int64_t ldc, void* D, int64_t ldd, float* S,
    int64_t lds, void* workspace, int64_t workspace_bytes, void* stream) {
  MMA_CHECK(check_lora(type_in, type_d, T, N, K, rank, requests, offsets, adapters_total));
  if (layout != MMA_COL_MAJOR && layout != MMA_ROW_MAJOR) return MMA_ERR_INVALID_ARG;
  if (T == 0) return MMA_OK;
  const bool row = layout == MMA_ROW_MAJOR;
  if (N > 0) MMA_CHECK(check_cd(C, ldc, D, ldd, N, float_bytes(type_d)));
  if (K > 0) {
    MMA_CHECK(check_in(X, ldx, K, 2));
    if (N > 0) MMA_CHECK(check_in(W, ldw, row ? N : K, 2));
  }
  if (rank > 0) {
    MMA_CHECK(check_sums(S, lds, rank));
    if (!aligned16(S) || lds % 8 != 0 || lds > INT32_MAX) return MMA_ERR_MISALIGNED;
    if (adapters) MMA_CHECK(check_words(adapters));
    if (scales) MMA_CHECK(check_words(scales));
    const int64_t need = mma_gemm_lora_workspace(type_in, type_d, T, N, rank, requests);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need))
      return MMA_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return MMA_ERR_MISALIGNED;
    if (adapters_total > 0 && K > 0) {
      MMA_CHECK(check_in(A, lda, row ? rank : K, 2));
      if (!slices_ok(adapters_total, stride_a, row ? K : rank, lda, row ? rank : K))
        return MMA_ERR_INVALID_ARG;
      if (adapters_total > 1 && !ld_ok(stride_a, 2)) return MMA_ERR_MISALIGNED;
      if (N > 0) {
        MMA_CHECK(check_in(B, ldb, row ? N : rank, 2));
        if (!slices_ok(adapters_total, stride_b, row ? rank : N, ldb, row ? N : rank))
          return MMA_ERR_INVALID_ARG;
        if (adapters_total > 1 && !ld_ok(stride_b, 2)) return MMA_ERR_MISALIGNED;
      }
    }
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  attach_profile(ctx);
  LoraProblem g = {};
  g.bf16 = type_in == MMA_BF16;
  g.row_major = row;
  g.d_type = type_d;
  g.rows = T;
  g.N = N;
  g.K = K;
  g.rank = rank;
  g.requests = requests;
  g.adapters_total = adapters_total;
  g.X = X;
  g.ldx = ldx;
  g.W = W;
  g.ldw = ldw;
  g.A = A;
  g.lda = lda;
  g.stride_a = stride_a;
  g.B = B;
  g.ldb = ldb;
  g.stride_b = stride_b;
  g.offsets = offsets;
  g.adapters = adapters;
  g.scales = scales;
  g.C = C;
  g.ldc = ldc;
  g.D = D;
  g.ldd = ldd;
  const LoraSpace space = lora_space(type_in, type_d, T, N, rank, requests);
  const int parts = lora_every(T, requests) ? 0 : lora_parts(g.bf16, type_d);
  LoraLow low = {S, static_cast<uint8_t*>(workspace) + space.extra,
                 static_cast<float*>(workspace), int(lds), int(lora_ld16(g.bf16, rank)),
                 parts};
  if (rank > 0) MMA_CHECK(launch_lora_shrink(ctx, g, low));
  if (N == 0) return MMA_OK;
  // without them there is nothing to add
  const bool plain = rank == 0 || requests == 0 || adapters_total == 0 || K == 0;
  return launch_gemm_lora(ctx, g, plain ? nullptr : &low);
}

extern "C" int64_t mma_gemm_lora_wgrad_workspace(int type_in, int type_d, int64_t T,
                                                 int64_t N, int64_t K, int64_t rank,
                                                 int64_t requests,
                                                 int64_t adapters_total) {
  if (!dim_ok(T) || !dim_ok(N) || !dim_ok(K) || rank < 1 || rank > MMA_MAX_RANK ||
      requests < 0 || requests > MMA_MAX_REQUESTS || adapters_total < 0)
    return 0;
  return lora_wgrad_workspace_bytes(type_in == MMA_BF16, type_d, T, N, K, rank, requests,
                                    adapters_total);
}

extern "C" mma_status_t mma_gemm_lora_wgrad(
    int type_in, int type_d, int64_t T, int64_t N, int64_t K, int64_t rank, const void* DY,
    int64_t lddy, const void* X, int64_t ldx, const float* S, int64_t lds, const float* U,
    int64_t ldu, int64_t requests, const int32_t* offsets, const int32_t* adapters,
    int64_t adapters_total, void* DA, int64_t ldda, int64_t stride_da, void* DB,
    int64_t lddb, int64_t stride_db, int accumulate, void* workspace,
    int64_t workspace_bytes, void* stream) {
  MMA_CHECK(check_lora(type_in, type_d, T, N, K, rank, requests, offsets, adapters_total));
  if ((N + 127) / 128 + (K + 127) / 128 > 65535) return MMA_ERR_UNSUPPORTED;
  if (requests > kMaxGroups && adapters_total > kMaxGroups) return MMA_ERR_UNSUPPORTED;
  if (rank == 0 || adapters_total == 0 || N + K == 0) return MMA_OK;
  MMA_CHECK(check_words(offsets));
  if (adapters) MMA_CHECK(check_words(adapters));
  const int64_t eb = float_bytes(type_d);
  if (K > 0) {
    MMA_CHECK(check_out(DA, ldda, K, eb));
    if (!slices_ok(adapters_total, stride_da, rank, ldda, K)) return MMA_ERR_INVALID_ARG;
  }
  if (N > 0) {
    MMA_CHECK(check_out(DB, lddb, rank, eb));
    if (!slices_ok(adapters_total, stride_db, N, lddb, rank)) return MMA_ERR_INVALID_ARG;
  }
  if (T > 0) {
    if (N > 0) MMA_CHECK(check_in(DY, lddy, N, 2));
    if (K > 0) MMA_CHECK(check_in(X, ldx, K, 2));
    if (N > 0) MMA_CHECK(check_sums(S, lds, rank));
    if (K > 0) MMA_CHECK(check_sums(U, ldu, rank));
    if (workspace == nullptr) return MMA_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return MMA_ERR_MISALIGNED;
    if (workspace_bytes <
        mma_gemm_lora_wgrad_workspace(type_in, type_d, T, N, K, rank, requests,
                                      adapters_total))
      return MMA_ERR_INVALID_ARG;
  }
  int dev = -1;
  const DeviceInfo* info = device_info(&dev);
  if (!info) return MMA_ERR_NO_DEVICE;
  Ctx ctx = make_ctx(stream, dev, info);
  attach_profile(ctx);
  LoraWgradProblem g = {};
  g.bf16 = type_in == MMA_BF16;
  g.d_type = type_d;
  g.rows = T;
  g.N = N;
  g.K = K;
  g.rank = rank;
  g.requests = requests;
  g.adapters_total = adapters_total;
  g.DY = DY;
  g.lddy = lddy;
  g.X = X;
  g.ldx = ldx;
  g.S = S;
  g.lds = lds;
  g.U = U;
  g.ldu = ldu;
  g.offsets = offsets;
  g.adapters = adapters;
  g.DA = DA;
  g.ldda = ldda;
  g.stride_da = stride_da;
  g.DB = DB;
  g.lddb = lddb;
  g.stride_db = stride_db;
  g.accumulate = accumulate != 0;
  return launch_lora_wgrad(ctx, g, workspace);
}
