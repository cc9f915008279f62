/*
 * mma_gb300.h -- C ABI of the GB300 (sm_103a) dense multiply-accumulate
 * library  D = A * B + C.
 *
 * Operation (page "CDNA2 dense MFMA builtins", section "Naming convention"):
 * one matrix instruction adds the contribution of an M x K panel of A and a
 * K x N panel of B to an M x N output tile, and the caller loops over K to
 * accumulate the full product.  Each call here performs that whole K loop:
 *
 *     D[i][j] = C[i][j] + sum_{k < K} A[i][k] * B[k][j]
 *
 * with the input/accumulator pairs of the pages' builtin lists ("CDNA2 dense
 * MFMA builtins", section "Builtin reference"; "RDNA3 dense WMMA builtins",
 * section "Builtin reference", which defines every builtin's result as
 * srcA x srcB + srcC):
 *
 *     dtype_in  dtype_acc   A, B element     C, D element
 *     MMA_F16   MMA_F32     IEEE binary16    float
 *     MMA_BF16  MMA_F32     bfloat16 bits    float
 *     MMA_F16   MMA_F16     IEEE binary16    IEEE binary16  (16-bit accumulate)
 *     MMA_BF16  MMA_BF16    bfloat16 bits    bfloat16 bits  (16-bit accumulate)
 *     MMA_I8    MMA_I32     signed int8      int32_t  (exact; wraps mod 2^32)
 *     MMA_F64   MMA_F64     double           double
 *
 * The 16-bit-accumulate pairs ("RDNA3 dense WMMA builtins", section
 * "Builtin reference", FP16/BF16-accumulate builtins) accumulate in FP32
 * inside and round A*B + C once to the 16-bit format (nearest, ties to
 * even); the builtins round their 16-bit accumulator after every K step.
 *
 * Any other pair returns MMA_ERR_UNSUPPORTED.
 *
 * Layouts (elements, not bytes; "RDNA3 dense WMMA builtins", section
 * "Using WMMA builtins as a compute policy": A rows and B columns are read
 * K-contiguous, the output is written row-major):
 *   A  M x K row-major:     A[i][k] at A[i*lda + k],  lda >= K
 *   B  column-major:        B[k][j] at B[j*ldb + k],  ldb >= K   (mma_gemm)
 *      or row-major:        B[k][j] at B[k*ldb + j],  ldb >= N   (mma_gemm_ex)
 *   C, D  M x N row-major:  C[i][j] at C[i*ldc + j],  ldc, ldd >= N
 *
 * Pointers and ownership: A, B, C and D are device pointers owned by the
 * caller; the library keeps no reference to them after the call returns.
 * C may be NULL (read as zero).  C may equal D (in place) only when
 * ldc == ldd; any other overlap between D and an input is undefined.
 *
 * Device memory owned by the library: some paths first rewrite an operand
 * into a scratch buffer -- INT8 products with M*N*K >= 2^24 (and every INT8
 * product with row-major B, and every mma_gemm_i8_ex product other than
 * signed x signed without clamp) widen A and B to BF16 for the tensor pipe,
 * (M + N) * roundup(K, 8) * 2 bytes, plus (M + N) * 8 bytes of correction
 * terms; batched INT8 products widen every tile, batch * (M + N) *
 * roundup(K, 8) * 2 bytes; FP16/BF16 products with row-major B transpose
 * B, N * roundup(K, 8) * 2 bytes; FP16/BF16 -> FP32 products with
 * column-major B, fewer than half as many 128 x 128 output tiles as SMs
 * and deep enough K (at least eight 64-deep K steps per tile, and either at
 * most a quarter as many tiles as SMs or at least 128 steps) split K over
 * the SMs and meet in it, SMs * 128 KiB, plus a hand-off flag buffer of
 * SMs * 32 bytes allocated (and zeroed) once per device.  That buffer is allocated once
 * per device by the first such call, grown (cudaMalloc, after the previous
 * user finishes) only when a larger problem arrives, and kept until the
 * process exits; calls on different streams are ordered on it by an event.
 * Failure to grow it returns MMA_ERR_NO_MEMORY.  No other call allocates.
 *
 * Alignment: every non-NULL base pointer must be 16-byte aligned and every
 * leading dimension times the element size must be a multiple of 16 bytes
 * (the tensor-memory-access engine's rule); otherwise MMA_ERR_MISALIGNED.
 * M, N and K themselves are arbitrary (>= 0): ragged edges are handled
 * inside the kernels.  M == 0 or N == 0 is a no-op; K == 0 gives D = C.
 *
 * Streams and errors: `stream` is a cudaStream_t (NULL = the legacy default
 * stream).  Work is enqueued on it and the call returns without
 * synchronising.  Argument errors are detected before anything is launched
 * and reported by the return value; a failed launch returns MMA_ERR_LAUNCH.
 * No C++ exception crosses this interface.  Every pipeline wait inside the
 * kernels is bounded; a wait that runs out records MMA_ERR_TIMEOUT in a
 * device-side status word that mma_device_status() reads back.  Calls on
 * different streams may run concurrently; the library holds no per-call
 * state.
 */
#ifndef MMA_GB300_H
#define MMA_GB300_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MMA_F16 = 1,
  MMA_BF16 = 2,
  MMA_I8 = 3,
  MMA_F64 = 4,
  MMA_F32 = 5,
  MMA_I32 = 6,
  MMA_F8E4M3 = 7, /* 8-bit floating point, 448 the largest value */
  MMA_F8E5M2 = 8  /* 8-bit floating point, 57344 the largest finite value */
} mma_dtype_t;

typedef enum { MMA_COL_MAJOR = 0, MMA_ROW_MAJOR = 1 } mma_layout_t;

typedef enum {
  MMA_OK = 0,
  MMA_ERR_INVALID_ARG = 1, /* negative size, short leading dimension, NULL
                              operand, bad broadcast group/id            */
  MMA_ERR_UNSUPPORTED = 2, /* dtype pair or batched shape not provided    */
  MMA_ERR_MISALIGNED = 3,  /* pointer or leading dimension not 16 B       */
  MMA_ERR_LAUNCH = 4,      /* CUDA reported an error at launch            */
  MMA_ERR_TIMEOUT = 5,     /* a bounded in-kernel wait ran out            */
  MMA_ERR_NO_DEVICE = 6,   /* no usable sm_103 device is current          */
  MMA_ERR_NO_MEMORY = 7    /* the scratch buffer could not be grown       */
} mma_status_t;

/*
 * mma_gemm -- D = A * B + C with column-major B.
 *
 * Passage: "CDNA2 dense MFMA builtins", sections "Naming convention" (the
 * K-loop contract) and "Builtin reference" (FP16/BF16 -> FP32, INT8 ->
 * INT32, FP64 -> FP64 with round-to-nearest-even); "RDNA3 dense WMMA
 * builtins", section "Builtin reference" (srcA x srcB + srcC; signed int8).
 *
 * dtype_in, dtype_acc : one of the pairs in the table above.
 * M, N, K             : problem size, each >= 0.
 * A, lda              : M x K row-major input, lda >= K.
 * B, ldb              : K x N column-major input (stored as N rows of K
 *                       contiguous elements), ldb >= K.
 * C, ldc              : M x N row-major addend of type dtype_acc, or NULL.
 * D, ldd              : M x N row-major output of type dtype_acc.
 * stream              : cudaStream_t to enqueue on.
 * Returns MMA_OK or an error code; see the header comment for each case.
 */
mma_status_t mma_gemm(int dtype_in, int dtype_acc, int64_t M, int64_t N,
                      int64_t K, const void *A, int64_t lda, const void *B,
                      int64_t ldb, const void *C, int64_t ldc, void *D,
                      int64_t ldd, void *stream);

/*
 * mma_gemm_ex -- as mma_gemm, with the layout of B chosen by `layout_b`:
 * MMA_COL_MAJOR (same as mma_gemm) or MMA_ROW_MAJOR (B[k][j] at
 * B[k*ldb + j], ldb >= N).  Same passages as mma_gemm; the row-major form
 * is the plain storage of a K x N matrix.
 */
mma_status_t mma_gemm_ex(int dtype_in, int dtype_acc, int64_t M, int64_t N,
                         int64_t K, const void *A, int64_t lda, const void *B,
                         int64_t ldb, int layout_b, const void *C, int64_t ldc,
                         void *D, int64_t ldd, void *stream);

/*
 * mma_gemm_i8_ex -- 8-bit integer D = A * B + C with INT32 C and D, each of
 * A and B signed or unsigned, and optional saturation.
 *
 * Passage: "RDNA3 dense WMMA builtins", sections "INT32-accumulate
 * builtins" (integer inputs signed or unsigned, chosen per operand by
 * a_neg and b_neg) and "INT8 and UINT8 inputs" (the iu8 builtin:
 * srcA x srcB + srcC, and `clamp`: saturate the output on overflow).
 *
 * a_neg, b_neg : nonzero -- A (B) holds int8 values in [-128, 127];
 *                zero    -- uint8 values in [0, 255].
 * clamp        : zero    -- D is the exact value modulo 2^32 (wrapping, as
 *                           mma_gemm's INT8 product);
 *                nonzero -- D is the exact value of A*B + C, saturated once
 *                           to [INT32_MIN, INT32_MAX].
 * Other arguments, layouts, alignment rules and status codes are those of
 * mma_gemm_ex with dtype_in = MMA_I8, dtype_acc = MMA_I32 (A, B: 1-byte
 * elements; layout_b MMA_COL_MAJOR or MMA_ROW_MAJOR).  Signed x signed
 * without clamp is exactly mma_gemm_ex; every other combination runs on the
 * tensor pipe and grows the library's scratch buffer like it
 * ((M + N) * roundup(K, 8) * 2 bytes; MMA_ERR_NO_MEMORY if it cannot).
 */
mma_status_t mma_gemm_i8_ex(int64_t M, int64_t N, int64_t K, const void *A,
                            int64_t lda, int a_neg, const void *B, int64_t ldb,
                            int b_neg, int layout_b, const void *C,
                            int64_t ldc, void *D, int64_t ldd, int clamp,
                            void *stream);

/*
 * mma_gemm_batched -- `batch` independent M x N x K products with A-block
 * broadcast:
 *
 *     for b in [0, batch):  D_b = A_{src(b)} * B_b + C_b,
 *                           src(b) = (b / G) * G + a_broadcast_id
 *
 * Passage: "Common MFMA parameters", section "Shared parameters" (cbsz:
 * one chosen input block of A is broadcast to the 2^cbsz - 1 neighbouring
 * blocks of its group; abid: which block of each group is the source;
 * worked example cbsz = 2, abid = 1: block 1's A goes to blocks 0, 2, 3 and
 * block 5's to 4, 6, 7), and "CDNA2 dense MFMA builtins", section
 * "Accumulator layout" (one instruction computes several independent
 * blocks, each with its own A, B, C and D).  Here a batch entry plays the
 * role of a block and G = a_broadcast_group = 2^cbsz.
 *
 * Storage: tiles are contiguous, tile b of A at A + b*M*lda, of B at
 * B + b*N*ldb (column-major tiles), of C and D at b*M*ldc and b*M*ldd
 * (elements).  A holds `batch` tiles; only tile src(b) is read for entry b.
 * B, C and D are never broadcast here (see mma_gemm_batched_ex for B).
 * Pairs: the four of mma_gemm plus 16-bit accumulate; any M, N, K >= 0;
 * leading dimensions and alignment as for mma_gemm (each tile is one
 * mma_gemm problem).  The kernel follows the block shape (dense tiles,
 * leading dimensions equal to the tile's row length):
 *   - 16 x 16 x 16 FP16/BF16 -> FP32: an HBM-streaming kernel;
 *   - FP16/BF16 with M, N, K multiples of 64 and M*N*K <= 2^20: a
 *     CTA-cooperative kernel (64 x 64 tiles, operands staged once in shared
 *     memory);
 *   - FP16/BF16 with M, N, K multiples of 16 and M*N*K <= 96*96*64, and
 *     INT8 with M, N, K multiples of 16 and M*N*K <= 128^3: warp-level
 *     streaming kernels;
 *   - everything else: the tensor-memory GEMM over per-entry tensor maps
 *     (INT8: through BF16 copies of every tile in the library's scratch
 *     buffer, grown like mma_gemm's); FP64: DMMA tiles.
 * The choice changes speed only: FP16/BF16 results agree within the
 * accumulation tolerance (the routes sum in different orders), and INT8
 * results are bit-identical across routes.
 * Constraints: a_broadcast_group in {1, 2, 4, 8, 16}; 0 <= a_broadcast_id
 * < a_broadcast_group; batch % a_broadcast_group == 0 (else
 * MMA_ERR_INVALID_ARG); batch < 2^31 (else MMA_ERR_UNSUPPORTED).
 */
mma_status_t mma_gemm_batched(int dtype_in, int dtype_acc, int64_t M,
                              int64_t N, int64_t K, const void *A, int64_t lda,
                              const void *B, int64_t ldb, const void *C,
                              int64_t ldc, void *D, int64_t ldd, int64_t batch,
                              int a_broadcast_group, int a_broadcast_id,
                              void *stream);

/*
 * mma_gemm_batched_ex -- mma_gemm_batched with a B-group pattern as well:
 *
 *     D_b = A_{src(b)} * B_{bsrc(b)} + C_b,
 *     bsrc(b) = (b / 4) * 4 + P[b_lane_group_pattern][b % 4]
 *
 * Passage: "Common MFMA parameters", section "Dense MFMA parameters"
 * (blgp: a constrained swizzle of B between the lanes of the 64-lane
 * operand).  Read at matrix level: consecutive groups of four batch entries
 * play the four 16-lane quarters, and P[p][q] is the quarter whose B the
 * entry at quarter q reads:
 *   p = 0  q            (no swizzling)
 *   p = 1  q & 1        (lanes 0-31 broadcast into lanes 32-63)
 *   p = 2  2 + (q & 1)  (lanes 32-63 broadcast into lanes 0-31)
 *   p = 3  (q + 1) % 4  (all lanes rotated down by 16)
 *   p = 4..7  p - 4     (one quarter broadcast into the other three)
 * b_lane_group_pattern in 0..7, and batch % 4 == 0 when it is nonzero (else
 * MMA_ERR_INVALID_ARG).  Everything else is as for mma_gemm_batched, which
 * is this call with b_lane_group_pattern = 0.
 */
mma_status_t mma_gemm_batched_ex(int dtype_in, int dtype_acc, int64_t M,
                                 int64_t N, int64_t K, const void *A,
                                 int64_t lda, const void *B, int64_t ldb,
                                 const void *C, int64_t ldc, void *D,
                                 int64_t ldd, int64_t batch,
                                 int a_broadcast_group, int a_broadcast_id,
                                 int b_lane_group_pattern, void *stream);

/*
 * mma_device_status -- synchronise `stream`, then read and clear the
 * library's device-side status word on the current device.  Returns MMA_OK
 * when no in-kernel wait has run out since the last call, MMA_ERR_TIMEOUT
 * otherwise, or MMA_ERR_LAUNCH if the synchronisation itself failed.
 * (The pages check errors after every launch: "RDNA3 dense WMMA builtins",
 * section "Instantiating the kernel"; this is the matching device-side
 * check.)
 */
mma_status_t mma_device_status(void *stream);

/*
 * mma_selftest_wait_timeout -- exercise the failure-detection path of the
 * kernels without faulting or hanging the GPU.  The pages have no
 * counterpart; it backs mma_device_status's contract with a test.
 *
 * Every pipeline wait inside the kernels is bounded: when one runs out, the
 * kernel records MMA_ERR_TIMEOUT in the device status word, drains and
 * returns.  This call enqueues on `stream` one tiny kernel that performs
 * that same bounded wait on a barrier that nothing ever signals, with the
 * limit `limit_ns` (1000 .. 10^10 nanoseconds), so the wait runs out after
 * about limit_ns and the kernel returns.  A following mma_device_status
 * (stream) then returns MMA_ERR_TIMEOUT once and clears the word; the
 * context stays usable.  Returns MMA_ERR_INVALID_ARG for a limit out of
 * range, MMA_ERR_NO_DEVICE without a device, else MMA_OK.
 */
mma_status_t mma_selftest_wait_timeout(int64_t limit_ns, void *stream);

/*
 * mma_selftest_gemm_abort -- exercise the tcgen05 GEMM kernel's own abort
 * path without faulting or hanging the GPU.  The pages have no counterpart;
 * it backs the bounded-wait contract of the GEMM kernels with a test.
 *
 * Enqueues on `stream` the BF16 -> FP32 GEMM kernel for a 256 x 256 x 256
 * product on single CTAs (cluster = 1) or on a CTA pair sharing one MMA
 * (cluster = 2), with its operand producer told to issue no loads and every
 * pipeline wait limited to limit_ns (10^6 .. 10^10 ns).  The MMA issuer's
 * first stage wait therefore runs out with nothing in flight; the kernel
 * raises its abort flag, records MMA_ERR_TIMEOUT in the device status word,
 * drains, frees its tensor memory and exits, so the context stays usable.
 * A and B (256 x 256 BF16) and D (256 x 256 FP32) are caller device
 * buffers, 16-byte aligned; nothing reads or writes them.  Returns
 * MMA_ERR_INVALID_ARG (bad cluster, limit or NULL buffer),
 * MMA_ERR_MISALIGNED, MMA_ERR_NO_DEVICE or the launch status; a following
 * mma_device_status(stream) returns MMA_ERR_TIMEOUT once.
 */
mma_status_t mma_selftest_gemm_abort(int cluster, int64_t limit_ns,
                                     const void *A, const void *B, void *D,
                                     void *stream);

/*
 * mma_selftest_f8_abort -- the same for the kernels of the 8-bit and grouped
 * calls.  X and Q are buffers of 1024 x 1024 BF16, S one of 8192 floats:
 *
 *   kernel 0, 1 : mma_quantize_f8 of X, blocks of 128 x 128 as is, blocks of 1 x
 *                 128 of the transpose
 *   kernel 2    : mma_rmsnorm_backward, X as DY, H and W; Q is DX, S is DW;
 *                 workspace: 456 * 1024 floats
 *   kernel 3, 4 : mma_gemm_f8 of X's first 1 or 1024 rows by its first 1024 (of
 *                 1024 bytes each), k split over a cluster or on CTA pairs
 *   kernel 5    : mma_gemm_grouped_wgrad, X as DY and X, S as the offsets
 *
 * No loads are issued.  Waits end after limit_ns (10^6 .. 10^10 ns; kernels 3 to
 * 5: after their own limit of two seconds), every block stops, drains and
 * returns, and Q is not written, nor is S (but kernel 2 adds up the untouched
 * workspace there).  Buffers are 16-byte aligned device memory of the caller;
 * workspace may be NULL but for kernel 2.  Returns as mma_selftest_gemm_abort.
 */
mma_status_t mma_selftest_f8_abort(int kernel, int64_t limit_ns, const void *X,
                                   void *Q, float *S, void *workspace,
                                   void *stream);

/*
 * mma_peak_probe -- enqueue one issue-rate probe of a compute pipe on every
 * SM of the current device and report the operations it performs.
 *
 * Passage: "CDNA2 dense MFMA builtins", section "Instruction throughput":
 * peak throughput = operations per instruction / cycles per instruction x
 * clock.  The probe measures that rate instead of deriving it: every SM
 * issues `iterations` rounds of independent back-to-back instructions of
 * one kind on register or shared-memory operands (no DRAM traffic), so
 * *ops_per_launch (written before the launch) divided by the launch's
 * duration (CUDA events around the call, on `stream`) is the pipe's rate
 * at the clock the launch ran at.  Kinds:
 *   MMA_PEAK_TC_F16  tcgen05.mma kind::f16, BF16 in, FP32 accumulate
 *                    (M = 128, N = 256, K = 16; the FP16/BF16 and exact
 *                    INT8 GEMMs' pipe); iterations <= 2^21
 *   MMA_PEAK_DMMA    mma.sync m8n8k4 FP64 (the FP64 GEMM's instruction)
 *   MMA_PEAK_IMMA    mma.sync m16n8k32 int8 -> int32 (small INT8 products)
 *   MMA_PEAK_DFMA    scalar FP64 fused multiply-add
 * One operation is one multiply or one add (a multiply-add counts 2).
 * Returns MMA_ERR_INVALID_ARG for an unknown kind, iterations < 1 or above
 * the kind's limit (2^40 for the warp-level kinds), or a NULL
 * ops_per_launch; MMA_ERR_NO_DEVICE without a device; else the launch
 * status.  Recorded by mma_profile_begin like the GEMM calls.
 */
typedef enum {
  MMA_PEAK_TC_F16 = 1,
  MMA_PEAK_DMMA = 2,
  MMA_PEAK_IMMA = 3,
  MMA_PEAK_DFMA = 4
} mma_peak_kind_t;
mma_status_t mma_peak_probe(int kind, int64_t iterations,
                            double *ops_per_launch, void *stream);

/*
 * mma_profile_begin / mma_profile_end -- per-launch timing of the dominant
 * kernel (the contraction kernel of each mma_gemm* call), for measuring it
 * against its roofline.  The pages time each kernel launch after warm-up
 * runs ("RDNA3 dense WMMA builtins", section "Instantiating the kernel");
 * this is the device-side counterpart.
 *
 * mma_profile_begin: start recording, on the current device, one CUDA event
 * pair on the caller's stream immediately around the dominant kernel of
 * each subsequent call (at most 4096 calls; later calls are not recorded).
 * The event pool is created on the first begin (never per call).  Returns
 * MMA_ERR_NO_DEVICE without a device, MMA_ERR_INVALID_ARG if the pool
 * belongs to another device.
 *
 * mma_profile_end: stop recording, wait for the recorded events, write the
 * durations in milliseconds of the first min(count, max_count) recorded
 * launches to ms[] (host array owned by the caller) and the number recorded
 * to *count.  Returns MMA_ERR_INVALID_ARG if profiling was not active.
 * Not thread-safe with concurrent calls on other threads.
 */
mma_status_t mma_profile_begin(void);
mma_status_t mma_profile_end(float *ms, int max_count, int *count);

/*
 * mma_gemm_i8_noalloc -- the exact INT8 -> INT32 product of mma_gemm
 * (column-major B, same layouts, alignment, C handling and status codes),
 * computed on the tensor pipe without allocating any device memory.
 *
 * The pages have no counterpart: this entry point exists for callers that
 * cannot let a library allocate device memory.  mma_gemm grows a scratch
 * buffer with cudaMalloc for large INT8 problems; a program whose pool
 * allocator has already reserved the memory it may use, or a service that
 * forbids allocation after start-up (cudaMalloc/cudaFree can block and
 * synchronise the device), calls this instead.  Its scratch is a fixed
 * array of MMA_NOALLOC_SCRATCH_BYTES in the library's device image, held by
 * every GPU that loads the library until the process exits.
 *
 * Limit: (M + N) * roundup(K, 8) * 2 bytes must fit in
 * MMA_NOALLOC_SCRATCH_BYTES (for example M = N = K = 4096); larger problems
 * return MMA_ERR_UNSUPPORTED and launch nothing.
 * Set-up: the first call on each device, made with that device current,
 * looks up the array's device address (cudaGetSymbolAddress) and caches it
 * for the device's current context (after cudaDeviceReset the next call
 * looks it up again); make that first call before any stream capture
 * begins.  Status codes and profiling (mma_profile_begin) as for mma_gemm.
 * Sharing: all calls on a device use the same array and leave their data in
 * it (nothing there needs to start at zero); calls whose work overlaps on
 * the GPU race on it, so order calls issued on different streams.
 */
#define MMA_NOALLOC_SCRATCH_BYTES (64u << 20)
mma_status_t mma_gemm_i8_noalloc(int64_t M, int64_t N, int64_t K,
                                 const void *A, int64_t lda, const void *B,
                                 int64_t ldb, const void *C, int64_t ldc,
                                 void *D, int64_t ldd, void *stream);

/*
 * ------------------------------------------------------------------------
 * 8-bit floating-point operands with scales, and products grouped by expert
 * ------------------------------------------------------------------------
 *
 * An 8-bit operand is a matrix q of E4M3 or E5M2 values and FP32 scales: the
 * value of element (i, k) is q[i][k] * S(i / r, k / 128), with r = 1 (a scale
 * for each block of 128 along a row) or r = 128 (square blocks).  S(i, b) is
 * at S[i * s_row + b * s_blk]; both strides are given in elements and are
 * >= 0, the scales are 4-byte aligned.  s_row = 1 (the scales of one k block
 * for all rows side by side) is the order that is read fastest.
 *
 * Unlike the calls above, the products ask of their outputs (and of C) no
 * more than the alignment of one element; inputs keep the rule of 16-byte
 * rows, except that scales and offsets need 4 bytes.  Rows, columns and k of
 * a product are at most 2^31 - 1025 (more: MMA_ERR_UNSUPPORTED).  None of
 * these calls allocates memory or waits for the device; all can be captured
 * in a graph.  The products start while the kernel before them on the stream
 * ends and wait for it before they touch memory (programmatic launch).
 */

/*
 * mma_rmsnorm_f8 -- root-mean-square norm of the rows of X + R, in 8 bits.
 *
 *     h = x + r,   y = h * w / sqrt(mean(h^2) + eps)     (FP32 throughout)
 *     s = max(max |y| over 128 columns / 448, 2^-126),   q = y / s  (E4M3)
 *
 * The quotient is formed in FP32, then in 8 bits, each to nearest, ties to
 * even.
 *
 * type   : MMA_F16, MMA_BF16 or MMA_F32, of X, R, H and Y.
 * w_type : of W (N elements): `type` or MMA_F32.
 * R      : M x N residual, or NULL (then h = x).
 * pow2   : nonzero -- s is rounded up to a power of two.
 * H      : M x N, the sum rounded to `type` (the next layer's residual), or
 *          NULL.  May be X or R itself, with the same leading dimension.
 * Y      : M x N, y rounded to `type`, or NULL.
 * Q, S   : M x N E4M3 values and their scales (1 x 128 blocks), or both
 *          NULL.  One of Y and Q is required.  Q's rows start on 16-byte
 *          boundaries, as the products read them.
 * A NaN or infinity in a row makes its row NaN; one that w brings into a
 * block makes that block's scale NaN or infinite and its values NaN or zero.
 */
mma_status_t mma_rmsnorm_f8(int type, int w_type, int64_t M, int64_t N,
                            const void *X, int64_t ldx, const void *R,
                            int64_t ldr, const void *W, float eps, int pow2,
                            void *H, int64_t ldh, void *Y, int64_t ldy,
                            void *Q, int64_t ldq, float *S, int64_t s_row,
                            int64_t s_blk, void *stream);

/*
 * mma_rmsnorm_backward -- gradient of the norm, from the stored sum H:
 *
 *     g = dy * w,  DX = g / rms - h * mean(g h) / rms^3 + R
 *     DW[j] = sum over rows of dy * h / rms               (FP32)
 *
 * R is the gradient that reaches H from elsewhere, or NULL; DX is the
 * gradient of X and of the forward's residual alike, and may be DY or R.
 * DW is summed in a fixed order (the same bits from run to run), through
 * `workspace`: device memory of the caller, 4-byte aligned, of at least
 * mma_rmsnorm_backward_workspace(M, N) bytes (at most 456 * N * 4), which
 * the call's work on `stream` uses and nothing else may meanwhile.  Types as
 * in mma_rmsnorm_f8.  M == 0 gives DW = 0.
 */
int64_t mma_rmsnorm_backward_workspace(int64_t M, int64_t N);
mma_status_t mma_rmsnorm_backward(int type, int w_type, int64_t M, int64_t N,
                                  const void *DY, int64_t lddy, const void *H,
                                  int64_t ldh, const void *W, float eps,
                                  const void *R, int64_t ldr, void *DX,
                                  int64_t lddx, float *DW, void *workspace,
                                  int64_t workspace_bytes, void *stream);

/*
 * mma_layernorm -- layer norm of the rows of X + R, in `type`, in 8 bits or both.
 *
 *     h = x + r,   c = h - mean(h),   y = c / sqrt(mean(c^2) + eps) * w + b
 *
 * in FP32 throughout; H, Y, Q and S and all other arguments as in mma_rmsnorm_f8.
 * B is the bias, N elements of w_type, or NULL.  The variance is taken from the distances
 * to the mean, or to a number whose distance to the mean is at most a deviation (the mean
 * of some of the row's elements), so that a row far from zero keeps its own.  A variance
 * beyond FP32 is infinite and y the bias.  A NaN or infinity in a row makes its row NaN.
 */
mma_status_t mma_layernorm(int type, int w_type, int64_t M, int64_t N,
                           const void *X, int64_t ldx, const void *R,
                           int64_t ldr, const void *W, const void *B, float eps,
                           int pow2, void *H, int64_t ldh, void *Y, int64_t ldy,
                           void *Q, int64_t ldq, float *S, int64_t s_row,
                           int64_t s_blk, void *stream);

/*
 * mma_layernorm_backward -- gradient of the layer norm, from the stored sum H:
 *
 *     g = dy * w,  g' = g - mean(g),  DX = g' / std - c * mean(g' c) / std^3 + R
 *     DW[j] = sum over rows of dy * c / std,   DB[j] = sum over rows of dy
 *
 * DW and DB in FP32, summed in a fixed order through `workspace` of at least
 * mma_layernorm_backward_workspace(M, N) bytes (at most 912 * N * 4, with N <= 2048
 * 2432 * N * 4, with N > 8192 16 * M more).  All else as in mma_rmsnorm_backward.
 */
int64_t mma_layernorm_backward_workspace(int64_t M, int64_t N);
mma_status_t mma_layernorm_backward(int type, int w_type, int64_t M, int64_t N,
                                    const void *DY, int64_t lddy, const void *H,
                                    int64_t ldh, const void *W, float eps,
                                    const void *R, int64_t ldr, void *DX,
                                    int64_t lddx, float *DW, float *DB,
                                    void *workspace, int64_t workspace_bytes,
                                    void *stream);

/*
 * mma_quantize_f8 -- X (M x N; MMA_F16, MMA_BF16 or MMA_F32) as 8-bit values
 * of type f8_type with scales:
 *
 *     s = max(max |x| over the block / format's largest value, 2^-126)
 *     q = x / s, in FP32 and then in 8 bits, each to nearest, ties to even
 *
 * block_rows : 1 or 128 (the blocks are block_rows x 128).
 * transpose  : nonzero -- Q is N x M, the transpose; its blocks of 128 run
 *              along its rows, that is, down X's columns.
 * pow2       : nonzero -- s is rounded up to a power of two.
 * Q's rows start on 16-byte boundaries.  A block with a NaN has a NaN
 * scale, one with an infinity an infinite scale.
 */
mma_status_t mma_quantize_f8(int type, int f8_type, int64_t M, int64_t N,
                             int block_rows, int transpose, int pow2,
                             const void *X, int64_t ldx, void *Q, int64_t ldq,
                             float *S, int64_t s_row, int64_t s_blk,
                             void *stream);

/*
 * mma_gemm_f8 -- D = A * B + C for 8-bit operands with scales, B
 * column-major: with a = q * s of A and b of B,
 *
 *     D[i][j] = C[i][j] + sum_b SA(i, b) SB(j / sb_rows, b)
 *                             * sum_{k in block b} qa[i][k] qb[j][k]
 *
 * type_a, type_b : MMA_F8E4M3 or MMA_F8E5M2, each.
 * type_d         : MMA_F32, MMA_BF16 or MMA_F16, of C and D.
 * A, SA          : M x K, scales of 1 x 128 blocks.
 * B, SB          : N x K, scales of sb_rows x 128 blocks, sb_rows 1 or 128.
 * C              : M x N or NULL; may be D with the same leading dimension.
 * Block products are summed in the tensor core's FP32, scaled by the FP32
 * product of the two scales and added in FP32; D is rounded once.  SA * SB
 * must be in FP32's range: a block for which it is below 2^-126 loses bits and
 * below 2^-150 all of its share, also where the share itself (up to 2^25 for
 * E4M3, 2^39 for E5M2, times that) would be in range.  The
 * gradients are the same call on quantised gradients and transposes (see
 * mma_quantize_f8); sb_rows = 1 serves the weight's.
 */
mma_status_t mma_gemm_f8(int type_a, int type_b, int type_d, int64_t M,
                         int64_t N, int64_t K, const void *A, int64_t lda,
                         const float *SA, int64_t sa_row, int64_t sa_blk,
                         const void *B, int64_t ldb, const float *SB,
                         int sb_rows, int64_t sb_row, int64_t sb_blk,
                         const void *C, int64_t ldc, void *D, int64_t ldd,
                         void *stream);

/*
 * mma_gemm_grouped -- products grouped by expert: the T rows of A are sorted
 * by group, group e is rows [offsets[e], offsets[e + 1]), and
 *
 *     D[i] = A[i] * B_e + C[i]     for the rows i of each group e.
 *
 * type_in  : MMA_F16 or MMA_BF16 (A, B); type_d : that or MMA_F32 (C, D).
 * groups   : 0 .. MMA_MAX_GROUPS (more: MMA_ERR_UNSUPPORTED).
 * offsets  : groups + 1 int32 values in DEVICE memory, read when the kernel
 *            runs; non-decreasing, within [0, T].  Values outside are
 *            clamped and decreasing ones raised to the one before; rows of
 *            no group are not written.  Groups may be empty.
 * B        : B_e at B + e * stride_b elements, column-major (N x K stored)
 *            or row-major (K x N stored; the input gradient of the
 *            column-major product with N and K exchanged).
 * C        : T x N or NULL; may be D with the same leading dimension.
 * Sums are FP32 (chunks of 256 terms from the tensor core, 512 for a 16-bit
 * result, added to nearest).
 */
#define MMA_MAX_GROUPS 1024
mma_status_t mma_gemm_grouped(int type_in, int type_d, int64_t groups,
                              int64_t T, int64_t N, int64_t K, const void *A,
                              int64_t lda, const void *B, int64_t ldb,
                              int64_t stride_b, int layout_b,
                              const int32_t *offsets, const void *C,
                              int64_t ldc, void *D, int64_t ldd, void *stream);

/*
 * mma_gemm_grouped_wgrad -- the weight gradient of mma_gemm_grouped:
 *
 *     D_e = DY_e^T * X_e + C_e     (N x K, over the rows of group e)
 *
 * DY is T x N, X is T x K; D_e is at D + e * stride_d, C_e at
 * C + e * stride_c (C may be D with the same strides: accumulation).  An
 * empty group gives D_e = C_e, or zeros.  Other arguments as above.
 */
mma_status_t mma_gemm_grouped_wgrad(int type_in, int type_d, int64_t groups,
                                    int64_t T, int64_t N, int64_t K,
                                    const void *DY, int64_t lddy,
                                    const void *X, int64_t ldx,
                                    const int32_t *offsets, const void *C,
                                    int64_t ldc, int64_t stride_c, void *D,
                                    int64_t ldd, int64_t stride_d,
                                    void *stream);

/*
 * mma_gemm_grouped_f8 -- mma_gemm_grouped with column-major 8-bit B and the
 * operands and scales of mma_gemm_f8; the scales of B_e start at
 * SB + e * sb_group.
 */
mma_status_t mma_gemm_grouped_f8(int type_a, int type_b, int type_d,
                                 int64_t groups, int64_t T, int64_t N,
                                 int64_t K, const void *A, int64_t lda,
                                 const float *SA, int64_t sa_row,
                                 int64_t sa_blk, const void *B, int64_t ldb,
                                 int64_t stride_b, const float *SB,
                                 int sb_rows, int64_t sb_group, int64_t sb_row,
                                 int64_t sb_blk, const int32_t *offsets,
                                 const void *C, int64_t ldc, void *D,
                                 int64_t ldd, void *stream);

/*
 * mma_route -- the router of a layer of experts.  Of each of T tokens' E logits
 * the k largest (of equal ones the lowest index) are its choices:
 *
 *     p = softmax(x) in FP32,  weights[t][j] = p of choice j, with `normalize`
 *     over the sum of the token's chosen p
 *     experts[t][j]  its expert, the best first
 *     offsets[e]     choices of the experts before e (E + 1 of them): the row
 *                    ranges of mma_gemm_grouped
 *     order[i]       the choice (t * k + j) at place i when the choices are
 *                    sorted by expert, within an expert by token
 *     place[t][j]    the place of that choice: order's inverse
 *     share[e]       mean of p_e over the tokens
 *     loss           E * sum over e of share[e] * (choices of e) / (tokens * k)
 *
 * type     : MMA_F16, MMA_BF16 or MMA_F32, of X (T x E, rows ldx apart, aligned to
 *            one element); E at most MMA_MAX_GROUPS, k at most MMA_MAX_CHOICES,
 *            T * k at most 2^30 (more: MMA_ERR_UNSUPPORTED).
 * mask     : T bytes or NULL; a token with 0 takes no part in anything.
 * tokens   : one int32, how many tokens take part.
 * An expert whose logit is -inf is not chosen.  Where no expert is left, and for a
 * masked token, experts is -1 and the weight 0; such choices stand behind
 * offsets[E] in `order`, so that it is a permutation whatever the mask.  Without
 * tokens share and loss are 0.  A NaN or +inf in a token's logits makes its
 * weights, share and loss NaN, its choices being experts all the same.
 * All outputs are contiguous device memory, the same bits from run to run.
 * workspace: device memory, 4-byte aligned, of mma_route_workspace(T, E) bytes (0
 * for up to 96 tokens and 8192 logits), which the call's work on `stream` uses and
 * nothing else may meanwhile.
 */
#define MMA_MAX_CHOICES 32
int64_t mma_route_workspace(int64_t T, int64_t E);
mma_status_t mma_route(int type, int64_t T, int64_t E, int64_t k, const void *X,
                       int64_t ldx, const uint8_t *mask, int normalize,
                       float *weights, int32_t *experts, int32_t *order,
                       int32_t *place, int32_t *offsets, float *share,
                       float *loss, int32_t *tokens, void *workspace,
                       int64_t workspace_bytes, void *stream);

/*
 * mma_route_backward -- gradient of the logits from DW (T x k, of the weights) and
 * DLOSS (one value in device memory, of the loss), either of which may be NULL:
 *
 *     a_e = DLOSS * E * (choices of e) / (tokens^2 * k)
 *     DX = p (a - sum p a), and at the chosen  w (DW - sum over chosen w DW)
 *
 * (without normalize p (a + DW - sum p (a + DW)), DW standing at the chosen), the
 * choices and their numbers being taken as given.  weights, experts, offsets and
 * tokens are mma_route's; those of NULL gradients may be NULL.  DX (T x E of X's
 * type) may be X; a masked token's row is 0.
 */
mma_status_t mma_route_backward(int type, int64_t T, int64_t E, int64_t k,
                                const void *X, int64_t ldx, const uint8_t *mask,
                                int normalize, const float *weights,
                                const int32_t *experts, const int32_t *offsets,
                                const int32_t *tokens, const float *DW,
                                const float *DLOSS, void *DX, int64_t lddx,
                                void *stream);

/*
 * mma_gemm_lora -- a product shared by many requests, each with a low-rank adapter
 * beside it.  The T rows of X are sorted by request, request i has the rows
 * [offsets[i], offsets[i + 1]) and the adapter a = adapters[i]:
 *
 *     S = scales[a] * X A_a             (T x rank, FP32)
 *     D = X W + C + S B_a               for the rows of request i
 *
 * type_in : MMA_F16 or MMA_BF16 (X, W, A, B); type_d : that or MMA_F32 (C, D).
 * layout  : MMA_COL_MAJOR -- W is stored N x K, A_a rank x K, B_a N x rank;
 *           MMA_ROW_MAJOR -- W K x N, A_a K x rank, B_a rank x N: the gradient of
 *           the other layout's X, with N and K exchanged and its B as A, its A as
 *           B (S is then what mma_gemm_lora_wgrad calls U).
 * A, B    : adapter a's matrices at A + a * stride_a and B + a * stride_b
 *           elements, adapters_total of them (at most 65535), of one rank, at most
 *           MMA_MAX_RANK (a smaller one is padded with zeros).
 * T, N, K : at most 2^31 - 65536 (more: MMA_ERR_UNSUPPORTED).
 * requests: 0 .. MMA_MAX_REQUESTS; offsets: as mma_gemm_grouped's, but no row is left
 *           out: rows of no request have no adapter.
 * adapters: int32 in device memory, or NULL (request i has adapter i).  Outside [0,
 *           adapters_total): none.  Requests may share an adapter.
 * scales  : one float per adapter, in device memory, or NULL (1).
 * C       : T x N or NULL; may be D with the same leading dimension.
 * S       : T x lds, 16-byte aligned, lds a multiple of 8; written whole (zeros
 *           where there is no adapter), columns from rank to the next eighth one
 *           included.
 * workspace: 16-byte aligned device memory of mma_gemm_lora_workspace(type_in,
 *           type_d, T, N, rank, requests) bytes, which the call's work on `stream`
 *           uses and nothing else may meanwhile.
 * With up to 128 rows or more than MMA_MAX_GROUPS requests, and for requests of fewer
 * than 8 rows, the product with B takes S as it is.  For the others S is rounded to a sum
 * of two numbers of type_in (BF16 and an FP32 D: three); FP16 ones are scaled
 * by a power of two for each row, whatever their size, and keep what is above 2^-38 of
 * the row's largest.  A NaN or infinity in one adapter or row stays with the rows of that
 * adapter, or that row, which may have either there.
 */
#define MMA_MAX_RANK 128
#define MMA_MAX_REQUESTS 65536
int64_t mma_gemm_lora_workspace(int type_in, int type_d, int64_t T, int64_t N,
                                int64_t rank, int64_t requests);
mma_status_t mma_gemm_lora(int type_in, int type_d, int64_t T, int64_t N,
                           int64_t K, int64_t rank, const void *X, int64_t ldx,
                           const void *W, int64_t ldw, const void *A,
                           int64_t lda, int64_t stride_a, const void *B,
                           int64_t ldb, int64_t stride_b, int layout,
                           int64_t requests, const int32_t *offsets,
                           const int32_t *adapters, int64_t adapters_total,
                           const float *scales, const void *C, int64_t ldc,
                           void *D, int64_t ldd, float *S, int64_t lds,
                           void *workspace, int64_t workspace_bytes,
                           void *stream);

/*
 * mma_gemm_lora_wgrad -- the gradients of the adapters of mma_gemm_lora, over the
 * rows t of all requests with adapter a:
 *
 *     DA_a = sum U_t^T X_t   (rank x K),     DB_a = sum DY_t^T S_t   (N x rank)
 *
 * with S of the forward call (T x lds) and U of the call for the input's gradient
 * (T x ldu), both FP32, any lds and ldu, scales included.
 * type_d  : of DA and DB, type_in or MMA_F32.  S and U are taken as sums of two
 *           numbers of type_in (BF16 and an FP32 result: three).  They may be of any
 *           size: FP16 ones are scaled by a power of two for each column of at most 64
 *           rows of a request, and keep what is above 2^-38 of its largest.
 *           An infinity in DY, X, S or U makes infinities or NaN of its adapter's sums
 *           that it is in.
 * accumulate : nonzero -- added to DA and DB; else an adapter without rows gets
 *           zeros.
 * Sums are FP32, in a fixed order, through `workspace`: 16-byte aligned device
 * memory of mma_gemm_lora_wgrad_workspace(type_in, type_d, T, N, K, rank, requests,
 * adapters_total) bytes.  Not both more than MMA_MAX_GROUPS requests and adapters
 * (MMA_ERR_UNSUPPORTED).  Other arguments as above.
 */
int64_t mma_gemm_lora_wgrad_workspace(int type_in, int type_d, int64_t T,
                                      int64_t N, int64_t K, int64_t rank,
                                      int64_t requests, int64_t adapters_total);
mma_status_t mma_gemm_lora_wgrad(int type_in, int type_d, int64_t T, int64_t N,
                                 int64_t K, int64_t rank, const void *DY,
                                 int64_t lddy, const void *X, int64_t ldx,
                                 const float *S, int64_t lds, const float *U,
                                 int64_t ldu, int64_t requests,
                                 const int32_t *offsets,
                                 const int32_t *adapters,
                                 int64_t adapters_total, void *DA, int64_t ldda,
                                 int64_t stride_da, void *DB, int64_t lddb,
                                 int64_t stride_db, int accumulate,
                                 void *workspace, int64_t workspace_bytes,
                                 void *stream);

/* Human-readable name of a status code (static string, never NULL). */
const char *mma_status_string(int status);

/* Library ABI version: major * 10000 + minor * 100 + patch. */
int mma_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MMA_GB300_H */
