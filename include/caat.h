/*
 * caat.h - C ABI of the B200 (sm_100a) library for the partially synchronized
 * row-parallel linear layer of CAAT-Net.
 *
 * Source of every operation: "Tensor-Parallelism with Partially Synchronized Activations"
 * (Lamprecht, Karnieli, Hanani, Giladi, Soudry; arXiv 2506.19645).
 *
 *   - P tensor-parallel ranks are emulated side by side in one GPU's memory, as the paper's
 *     "logical devices" (§3.2): the partial channel-reduce becomes an on-chip sum.
 *   - Partial products: Zt_m = X_m W_m^T over rank m's K/P slice (§3.1 Eq. 4-5, App. A.2
 *     Eq. 21-22; W_m is the row-parallel block B~_m, stored transposed).
 *   - Partial channel-reduce (App. A.2 Eq. 22; §3.1 Eq. 8): for the shared channels
 *     c in S, |S| = floor(H p), every rank gets sum_m Zt_m[:, c]; the private channels keep
 *     the rank's own Zt_m[:, c], optionally times private_scale (§4 Eq. 14-15: sqrt(P)).
 *   - Residual add and norm (§4 Eq. 9, App. B Eq. 25): h_m = Z_m + R_m, then RMSNorm per
 *     rank and token, out_m = h_m / sqrt(mean_c h_m^2 + eps) * gamma (gamma shared by the
 *     ranks, since norm parameters are synchronized, §4).
 *   - MLP block (§3.1 Eq. 6 with sigma = SwiGLU): Y_m = silu(X_m A_gate,m^T) * (X_m A_up,m^T),
 *     then the layer above with X := Y.
 *   - Backward of the layer (§4 Eq. 10-13): the norm derivative per rank, then the reduction
 *     over ranks of the shared channels' gradients, then the gradients of the partial products.
 *   - Speed-up model of partial synchronization (App. C Eq. 31-35), host only.
 *
 * Conventions for every call below
 *   - bf16 tensors are raw bfloat16 bit patterns (caat_bf16), row-major, last dim contiguous.
 *   - Device pointers are owned by the caller, must be 16-byte aligned and stay valid until
 *     the work queued on `stream` has finished.  The library never allocates device memory
 *     and never synchronizes the stream in a forward call.
 *   - Every forward call validates all arguments on the host first; an invalid call queues
 *     no work and returns an error code.  No call throws across the ABI.
 *   - Work is queued asynchronously on `stream` (a cudaStream_t; NULL = legacy default).
 *   - Device-side waits are bounded: a wait that runs out (2 s; the environment variable
 *     CAAT_TIMEOUT_MS overrides) records CAAT_ERR_TIMEOUT in a device status word, which
 *     caat_get_device_status() reads.
 */
#ifndef CAAT_H_
#define CAAT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(CAAT_BUILD) && defined(__GNUC__)
#define CAAT_API __attribute__((visibility("default")))
#else
#define CAAT_API
#endif

typedef uint16_t caat_bf16;                   /* bfloat16 bit pattern */
typedef struct CUstream_st* caat_stream_t;    /* identical to cudaStream_t */
typedef struct caat_timing caat_timing;       /* opaque per-kernel event recorder */

typedef enum caat_status {
  CAAT_OK = 0,
  CAAT_ERR_INVALID_ARG = 1,   /* a pointer, size or value is invalid (nothing queued) */
  CAAT_ERR_UNSUPPORTED = 2,   /* valid, but outside what the kernels handle (alignment,
                                 divisibility, limits) or no sm_100 device */
  CAAT_ERR_CUDA = 3,          /* a CUDA runtime call failed */
  CAAT_ERR_TIMEOUT = 4,       /* a bounded device-side wait ran out (read from the device) */
  CAAT_ERR_WORKSPACE = 5      /* workspace NULL, misaligned or smaller than required */
} caat_status;

/* Limits of this build. */
#define CAAT_MAX_H 65536      /* hidden size H */
#define CAAT_MAX_P 64         /* emulated tensor-parallel ranks */
#define CAAT_DECODE_MAX_T 64  /* 1 <= T <= this (with P <= 16, H <= 8192) uses the decode
                                 (weight-streaming) path */

/* Workspace variants for caat_workspace_size(). */
#define CAAT_VARIANT_ROWPAR 0 /* caat_rowpar_forward[_ex]; K = FFN dim */
#define CAAT_VARIANT_MLP 1    /* caat_mlp_forward[_ex]; K = F */
#define CAAT_VARIANT_ROWPAR_HOST 2 /* caat_rowpar_forward_host; K = FFN dim */
#define CAAT_VARIANT_ROWPAR_BWD 4  /* caat_rowpar_backward; K = FFN dim */

/* Flags of caat_rowpar_args.flags / caat_mlp_args.flags. */
#define CAAT_FLAG_FORCE_GEMM_PATH 0x1u   /* use the tensor-core GEMM path even for small T */
#define CAAT_FLAG_FORCE_DECODE_PATH 0x2u /* use the weight-streaming path even for large T */
#define CAAT_FLAG_FUSED_NORM 0x8u        /* run the RMSNorm inside the GEMM kernel (normalizer
                                            warps fed by row-block completion counters) instead
                                            of as a separate row kernel after it */
#define CAAT_FLAG_ORDER_ROWBLOCK 0x10u   /* schedule the GEMM tiles row block by row block
                                            (default: shared-channel tiles first, then the
                                            private tiles rank by rank) */
#define CAAT_FLAG_OVERLAP_NORM 0x20u     /* T >= 4096: run the GEMM in 2048-token launches and the
                                            row norm of each launch's tokens on a library-owned
                                            side stream, overlapping the next launch */
#define CAAT_FLAG_ORDER_GROUPED 0x40u    /* schedule the GEMM tiles in groups of row blocks
                                            (shared tiles of the group, then its private tiles
                                            rank by rank); the fused norm always does */
#define CAAT_FLAG_SINGLE_CTA 0x4u        /* use the single-CTA GEMM kernel (128-token tiles)
                                            instead of the CTA-pair kernel (256-token tiles) */
#define CAAT_FLAG_W_PERMUTED 0x80u       /* W is the channel-permuted weight written by
                                            caat_permute_weights for this (sync_idx, p):
                                            the GEMM sees a contiguous sync set (no column
                                            block mixes shared and private channels) and the
                                            norm kernel restores the original channel order.
                                            Outputs stay in the original order.  Needs a
                                            buffer for Z' (h_out if given and distinct from
                                            residual, else out, which must then not alias
                                            residual); not with CAAT_FLAG_FUSED_NORM; the
                                            GEMM path needs H <= 4096. */
#define CAAT_FLAG_NORM_BESIDE_GEMM 0x200u /* CTA-pair GEMM path, H <= 4096, separate norm: start the
                                            row norm while the GEMM runs, on SMs the GEMM leaves
                                            free; it normalizes each 128-token block of a rank as
                                            soon as the GEMM has stored all of it (the GEMM counts
                                            its finished tiles per block in the workspace).  Needs
                                            the workspace caat_workspace_size reports; same bits
                                            as the default (norm after the GEMM) */
#define CAAT_FLAG_TEST_STALL 0x100u      /* test hook: the GEMM kernel's MMA warp never signals
                                            its accumulator, so every consumer wait runs out
                                            and the call reports CAAT_ERR_TIMEOUT through
                                            caat_get_device_status().  Nothing faults. */

/*
 * caat_rowpar_forward - the partially synchronized row-parallel layer, residual add and
 * per-rank RMSNorm (App. A.2 Eq. 22, §4 Eq. 9).
 *
 *   X         device, bf16 [P, T, K/P]   rank m's input slice X_m
 *   W         device, bf16 [P, H, K/P]   rank m's weight block (B~_m transposed, K contiguous)
 *   residual  device, bf16 [P, T, H]     per-rank residual R_m (App. B)
 *   gamma     device, bf16 [H]           RMSNorm weight, shared by the ranks
 *   sync_idx  HOST, int32, NULL or floor(H p) strictly increasing channels in [0, H).
 *             NULL selects the first floor(H p) channels (§3).  Read before return.
 *   P, p      ranks (1..CAAT_MAX_P) and sync factor p in [0, 1]; n_s = floor(H p) in double.
 *   out       device, bf16 [P, T, H]     normalized output; may alias `residual`.
 *   T, K, H   tokens (>= 0), FFN dim (K % P == 0, (K/P) % 8 == 0), hidden (H % 8 == 0).
 *   workspace device scratch, 256-byte aligned; contents need not be initialized and are
 *             clobbered.  caat_workspace_size(T, K, H, P, CAAT_VARIANT_ROWPAR) bytes enable
 *             every path: the fused norm's row-block counters and per-row partial sums of
 *             squares (about 64 ceil(H/256) P T bytes), the completion flags that give
 *             column blocks mixing shared and private channels the TMA epilogue (T/8
 *             ceil(H/256) bytes), the decode path's fp32 partials (4 P T H bytes, T <= 64),
 *             and the cross-rank sums of the shared channels stored once for all ranks
 *             (4 T n_s bytes; H <= 4096, S the first n_s channels, n_s % 8 == 0; each rank's
 *             residual is then added by the norm kernel).  The separate-norm GEMM path runs
 *             with 256 bytes (mixed column blocks then take the register epilogue and every
 *             shared tile stores h for all P ranks); a smaller workspace than a call needs
 *             gives CAAT_ERR_WORKSPACE.
 * eps = 1e-5 and private_scale = 1 (use caat_rowpar_forward_ex for other values).
 * Returns CAAT_OK once the work is queued.
 */
CAAT_API caat_status caat_rowpar_forward(const caat_bf16* X, const caat_bf16* W, const caat_bf16* residual,
                                const caat_bf16* gamma, const int32_t* sync_idx, int P, double p,
                                caat_bf16* out, int64_t T, int64_t K, int64_t H,
                                void* workspace, size_t ws_bytes, caat_stream_t stream);

/* Extended arguments of the row-parallel layer (same meaning as above, plus): */
typedef struct caat_rowpar_args {
  const caat_bf16* X;
  const caat_bf16* W;
  const caat_bf16* residual;
  const caat_bf16* gamma;
  const int32_t* sync_idx;     /* host */
  caat_bf16* out;
  caat_bf16* h_out;            /* optional (NULL): device bf16 [P, T, H] receives the pre-norm
                                  residual stream h = Z + R; may alias `residual` */
  void* workspace;
  size_t ws_bytes;
  caat_stream_t stream;
  caat_timing* timing;         /* optional (NULL): records CUDA events around each kernel */
  int64_t T, K, H;
  double p;
  float eps;                   /* RMSNorm epsilon, >= 0, inside the square root */
  float private_scale;         /* multiplies private channels before the residual add */
  int32_t P;
  uint32_t flags;              /* CAAT_FLAG_* */
} caat_rowpar_args;

CAAT_API caat_status caat_rowpar_forward_ex(const caat_rowpar_args* args);

/*
 * caat_rowpar_forward_host - the same layer for callers whose tensors live in HOST memory.
 * args->X, W, residual, gamma, out (and h_out if not NULL) are host pointers (pinned memory
 * for asynchronous copies; pageable memory also works, with synchronous staging).
 * args->workspace is a device buffer of caat_workspace_size(T, K, H, P,
 * CAAT_VARIANT_ROWPAR_HOST) bytes that receives device copies of the inputs and outputs.
 * The call is pipelined over chunks of 1024 tokens, the last ones halving down to 256 (token
 * rows are independent; a small last chunk keeps the final copy back short): W and gamma
 * are copied once, then each chunk's X and residual rows are copied in, its kernels run on
 * args->stream and its out (and h_out) rows are copied back, on two library-owned copy
 * streams (created on the first call on a device) so that both copy directions overlap the
 * kernels.  All of it is ordered after the work already queued on args->stream, and
 * args->stream waits for the last copy back: the call is complete when args->stream reaches
 * that point, and the host buffers must stay valid until then.
 */
CAAT_API caat_status caat_rowpar_forward_host(const caat_rowpar_args* args);

/*
 * caat_rowpar_forward_noalloc - the same layer for callers that cannot allocate device memory
 * at all: code running where cudaMalloc is unavailable or forbidden (a host process whose
 * allocator is owned by someone else, an embedding that may not grow its memory footprint,
 * a hot loop that must never enter the allocator).  No counterpart in the paper: it is a
 * deployment convenience of this library.
 *
 * Arguments as caat_rowpar_forward_ex, except that args->workspace and args->ws_bytes are
 * ignored.  The scratch the kernels need lives in a fixed device array inside the library,
 * CAAT_NOALLOC_SCRATCH_BYTES bytes per GPU, held by every GPU that loads the library until the
 * process exits.  It holds whatever workspace the path the call takes uses, when that fits:
 * the GEMM kernel's work-unit counter (always), the row-block counters and job list of the
 * norm that runs beside the GEMM (8 bytes per 128 tokens per rank), the completion flags of
 * column blocks that mix shared and private channels (T/8 ceil(H/256) bytes), the shared
 * channels' cross-rank sums (4 T n_s bytes), the fused norm's counters and partials, and the
 * decode path's fp32 partials (4 P T H bytes).
 *   - A fused norm (CAAT_FLAG_FUSED_NORM) whose partials do not fit runs as the separate norm;
 *     a decode-sized call whose partials do not fit takes the GEMM path; the optional parts
 *     (job list, flags, shared sums) are simply not used when they do not fit.  A call that still needs
 *     more than the array (a forced decode path that does not fit) returns
 *     CAAT_ERR_WORKSPACE and queues nothing.
 *   - Calls no cudaMalloc, cudaFree or other allocating routine.
 *   - The first call on a device looks up the array's device address (once per device and
 *     context, with that device current); make that first call before any stream capture.
 *   - Every call shares the one array and clears the part that must start at zero; calls
 *     whose work overlaps on the GPU (other streams, other host threads) race on it and must
 *     be serialized by the caller.
 */
#define CAAT_NOALLOC_SCRATCH_BYTES 1048576
CAAT_API caat_status caat_rowpar_forward_noalloc(const caat_rowpar_args* args);

/*
 * Plans: the graph-capture-friendly form of caat_rowpar_forward_ex for calls repeated on the
 * same buffers (a decode loop, a layer in a captured step).  caat_plan_create validates the
 * arguments and builds the sync mask once, binding every pointer, size and option of `args`
 * (which is copied; sync_idx is read before return); caat_plan_execute then only queues the
 * kernels on `stream` (it allocates nothing and never synchronizes, so it can be captured in
 * a CUDA graph once the device's first call has been made outside capture).  The buffers
 * must stay valid for the plan's lifetime.  A plan is host memory owned by the caller
 * through the handle; executing one plan on two streams at once races on its workspace.
 * No counterpart in the paper.
 */
typedef struct caat_plan caat_plan;
CAAT_API caat_status caat_plan_create(const caat_rowpar_args* args, caat_plan** plan_out);
CAAT_API caat_status caat_plan_execute(const caat_plan* plan, caat_stream_t stream);
CAAT_API caat_status caat_plan_destroy(caat_plan* plan);

/*
 * caat_mlp_forward - the MLP block per rank: column-parallel FC1 with SwiGLU (§3.1 Eq. 6),
 * then the partially synchronized FC2 (App. A.2 Eq. 22), residual add and RMSNorm (Eq. 9).
 *
 *   X         device, bf16 [P, T, H]        per-rank block input X_m
 *   A         device, bf16 [P, 2F/P, H]     rank m's FC1 rows: F/P gate rows, then F/P up rows
 *   W2        device, bf16 [P, H, F/P]      rank m's FC2 block
 *   residual, gamma, sync_idx, P, p, out    as for caat_rowpar_forward
 *   T, H, F   F % P == 0, (F/P) % 8 == 0, H % 8 == 0
 *   workspace caat_workspace_size(T, F, H, P, CAAT_VARIANT_MLP) bytes (holds Y [P,T,F/P]).
 */
CAAT_API caat_status caat_mlp_forward(const caat_bf16* X, const caat_bf16* A, const caat_bf16* W2,
                             const caat_bf16* residual, const caat_bf16* gamma,
                             const int32_t* sync_idx, int P, double p, caat_bf16* out,
                             int64_t T, int64_t H, int64_t F,
                             void* workspace, size_t ws_bytes, caat_stream_t stream);

typedef struct caat_mlp_args {
  const caat_bf16* X;
  const caat_bf16* A;
  const caat_bf16* W2;
  const caat_bf16* residual;
  const caat_bf16* gamma;
  const int32_t* sync_idx;     /* host */
  caat_bf16* out;
  caat_bf16* h_out;            /* optional pre-norm residual stream, as in caat_rowpar_args */
  void* workspace;
  size_t ws_bytes;
  caat_stream_t stream;
  caat_timing* timing;
  int64_t T, H, F;
  double p;
  float eps;
  float private_scale;
  int32_t P;
  uint32_t flags;
} caat_mlp_args;

CAAT_API caat_status caat_mlp_forward_ex(const caat_mlp_args* args);

/*
 * caat_rowpar_backward - gradients of the row-parallel layer (forward: caat_rowpar_forward)
 * for training, §4 Eq. 10-13 and Fig. 2b: the RMSNorm derivative per rank first, THEN the
 * reduction over ranks of the shared channels' gradients (fp32 accumulation, §4 "32 bit
 * gradient accumulation"), the private scale on the private channels, then the partial
 * products' gradients dX_m = dZt_m W_m and dW_m = dZt_m^T X_m (tcgen05 GEMMs); the shared
 * RMSNorm weight's gradient is summed over ranks and tokens (§4 Eq. 12-13).
 *
 *   X, W, gamma, sync_idx, p, P, T, K, H, eps, private_scale  as in the forward call
 *   h        device bf16 [P, T, H]: the pre-norm stream of the forward (its h_out)
 *   dout     device bf16 [P, T, H]: dL/d(out)
 *   dX       device bf16 [P, T, K/P]   (out)
 *   dW       device bf16 [P, H, K/P]   (out)
 *   dR       device bf16 [P, T, H] or NULL: dL/d(residual) = dL/dh  (out)
 *   dgamma   device fp32 [H]            (out)
 *   workspace caat_workspace_size(T, K, H, P, CAAT_VARIANT_ROWPAR_BWD) bytes, 256-byte aligned:
 *            dZt, per-CTA dgamma partials, and room for transposed copies of W, dZt and X,
 *            which only calls with T <= 128 or H <= 128 use (larger calls read the three
 *            tensors in place, MN-major).
 * Requires P <= 16 and H <= 8192.  Outputs must not overlap the inputs.  Asynchronous.
 */
typedef struct caat_rowpar_bwd_args {
  const caat_bf16* X;
  const caat_bf16* W;
  const caat_bf16* h;
  const caat_bf16* gamma;
  const caat_bf16* dout;
  const int32_t* sync_idx;     /* host */
  caat_bf16* dX;
  caat_bf16* dW;
  caat_bf16* dR;
  float* dgamma;
  void* workspace;
  size_t ws_bytes;
  caat_stream_t stream;
  caat_timing* timing;         /* optional: events around each of the backward's kernels */
  int64_t T, K, H;
  double p;
  float eps;
  float private_scale;
  int32_t P;
  uint32_t flags;              /* 0, or CAAT_BWD_FLAG_TRANSPOSED_OPERANDS */
} caat_rowpar_bwd_args;

/* Test hook: run the gradient GEMMs on transposed K-major copies of W, dZt and X (the path of
 * calls with T <= 128 or H <= 128) at any size.  The results equal the default path's bit for
 * bit: same MMA steps on the same values, only the operands' layout in memory differs. */
#define CAAT_BWD_FLAG_TRANSPOSED_OPERANDS 0x1u

CAAT_API caat_status caat_rowpar_backward(const caat_rowpar_bwd_args* args);

/*
 * The layer over real devices, one tensor-parallel rank per GPU (App. A.2 Eq. 22; §3: only the
 * first floor(h p) channels are synchronized; App. D: the exchange moves p times the bytes of
 * a full all-reduce).  Each rank r runs, on its own GPU:
 *   1. caat_rowpar_tp_local: its partial product X_r W_r^T (tcgen05 GEMM); the shared channels
 *      c < n_s = floor(H p) are written to zs as fp32 partials, the private channels are
 *      finished into h (private_scale * partial + residual, bf16);
 *   2. the caller's collective: zs summed over the ranks in place (e.g. an NCCL all-reduce,
 *      sum, fp32, of T * n_s elements); every rank then holds the same sums (Eq. 22);
 *   3. caat_rowpar_tp_finish: h[:, c] = bf16(zs[:, c] + residual[:, c]) for c < n_s (so h is the
 *      complete pre-norm residual stream), then out = RMSNorm(h) * gamma (§4 Eq. 9).
 * S is the first n_s channels (the paper's definition); n_s % 8 == 0 and H <= 4096 are
 * required (CAAT_ERR_UNSUPPORTED otherwise).  The single-device entry points above emulate the
 * same layer with the exchange folded into the tensor-core accumulation.
 *
 *   X         device bf16 [T, K_r]   this rank's input slice (local)
 *   W         device bf16 [H, K_r]   this rank's weight block (local)
 *   residual  device bf16 [T, H]     this rank's residual (local, finish)
 *   gamma     device bf16 [H]        RMSNorm weight (finish)
 *   zs        device fp32 [T, n_s]   local: out (this rank's partial); finish: in (the sum over
 *                                    ranks); NULL allowed when n_s == 0
 *   h         device bf16 [T, H]     local: out (private channels); finish: in/out (complete h)
 *   out       device bf16 [T, H]     finish: out; may alias h
 *   workspace local: 256 device bytes, 256-byte aligned (finish: unused)
 * Both calls are asynchronous on `stream`.  Outputs must not overlap other inputs.
 */
typedef struct caat_tp_args {
  const caat_bf16* X;
  const caat_bf16* W;
  const caat_bf16* residual;
  const caat_bf16* gamma;
  float* zs;
  caat_bf16* h;
  caat_bf16* out;
  void* workspace;
  size_t ws_bytes;
  caat_stream_t stream;
  caat_timing* timing;
  int64_t T, K_r, H;
  double p;
  float eps;
  float private_scale;
  uint32_t flags;              /* 0 */
} caat_tp_args;

CAAT_API caat_status caat_rowpar_tp_local(const caat_tp_args* args);
CAAT_API caat_status caat_rowpar_tp_finish(const caat_tp_args* args);

/*
 * The same layer with the exchange done by the library over peer memory (NVLink), no
 * collective library involved (App. A.2 Eq. 22; §3; §4: fp32 sum of the shared channels; App. D:
 * only the n_s shared channels cross devices).  Owner q of the world ranks owns the shared
 * columns [q w, (q + 1) w), w = n_s / world.  Per call, in this order on every rank:
 *   1. caat_rowpar_tp_local_push: the local GEMM (as caat_rowpar_tp_local) whose epilogue
 *      stores this rank's fp32 partial of every shared column straight into its owner's receive
 *      buffer (recv[q][rank][t][c - q w]); the launch's last CTA then raises
 *      flags[q][0 * world + rank] = epoch on every rank q.  args->zs is not used.
 *   2. caat_rowpar_tp_reduce: waits (bounded) until flags[rank][0 * world + r] = epoch for every
 *      r, sums the world partials of its columns in rank order (fp32), writes the sum into
 *      gather[g][t][rank w + j] of every rank g, and raises flags[g][1 * world + rank] = epoch.
 *   3. caat_rowpar_tp_finish_wait: waits until flags[rank][1 * world + q] = epoch for every q,
 *      then finishes as caat_rowpar_tp_finish with zs = gather[rank].
 * A rank's own entries are its local buffers; the others are the peers' buffers mapped into
 * this process (CUDA IPC), all on GPUs with peer access.  The caller allocates, per rank:
 * recv [world][T][w] fp32, gather [T][n_s] fp32, flags [2][world] uint32 zeroed once, and
 * reuses them across calls with an epoch that grows by one per call (0 is never used).  The
 * three calls of one rank go on one stream in order; then no buffer is overwritten while it is
 * still read: a rank's next push follows its finish, which waited for every owner's reduce, and
 * an owner's next reduce waits for every rank's next push.  A wait that runs out (a rank that
 * never arrives) sets
 * the device status word (caat_get_device_status: CAAT_ERR_TIMEOUT) and the kernel returns;
 * after an error nothing is signalled, so the other ranks' waits run out too.
 * Requirements: world = 1..8, rank < world, n_s = floor(H p) a multiple of 32 world, the
 * caat_rowpar_tp_local requirements, all pointers 16-byte aligned.
 */
#define CAAT_TP_MAX_WORLD 8
typedef struct caat_tp_peers {
  int32_t world;
  int32_t rank;
  uint32_t epoch;
  float* recv[CAAT_TP_MAX_WORLD];
  float* gather[CAAT_TP_MAX_WORLD];
  uint32_t* flags[CAAT_TP_MAX_WORLD];
} caat_tp_peers;

CAAT_API caat_status caat_rowpar_tp_local_push(const caat_tp_args* args, const caat_tp_peers* peers);
CAAT_API caat_status caat_rowpar_tp_reduce(const caat_tp_args* args, const caat_tp_peers* peers);
CAAT_API caat_status caat_rowpar_tp_finish_wait(const caat_tp_args* args, const caat_tp_peers* peers);

/*
 * caat_permute_weights - reorders the output channels (rows) of W for a sync set: with
 * perm(i) = the i-th shared channel for i < n_s and the (i - n_s)-th private channel
 * otherwise (both ascending), W_out[m, i, :] = W[m, perm(i), :] for every rank m.  The
 * layer's result does not depend on the order of the output channels (Eq. 22 sums each
 * shared channel over the ranks, whatever its index), so a forward call given W_out and
 * CAAT_FLAG_W_PERMUTED computes the same layer with the shared channels contiguous, which
 * keeps every 256-channel tile of the GEMM pure when S is an arbitrary list.  Done once per
 * weight (static weights: at load time).  No counterpart in the paper.
 *
 *   W, W_out  device, bf16 [P, H, K/P], 16-byte aligned, must not overlap.
 *   sync_idx, p, P, H, K  as for caat_rowpar_forward (same validation).
 * Asynchronous on `stream`; returns CAAT_OK once the copy kernel is queued.
 */
CAAT_API caat_status caat_permute_weights(const caat_bf16* W, caat_bf16* W_out, const int32_t* sync_idx, double p,
                                          int P, int64_t H, int64_t K, caat_stream_t stream);

/*
 * caat_speedup_model - the paper's speed-up model of partial synchronization (App. C,
 * Eq. 31-35), host only.  Per device and transformer layer (forward): G = (24 s h^2 +
 * 4 s^2 h) / r GEMM operations and P(p) = 2 s h p exchanged activations; with C the ratio of
 * compute to communication capacity in operations per exchanged activation, T(p) = G + C P(p),
 *   speedup = (T(1) - T(p)) / T(1) = (1 - p) / (1 + (12 h + 2 s) / (C r)),
 *   p*      = min((12 h + 2 s) / (C r), 1)   (C P(p*) = G: the exchange just fits under the compute).
 * h hidden size, s tokens, r tensor-parallel ranks, p in [0, 1], C > 0; outputs may be NULL.
 */
CAAT_API caat_status caat_speedup_model(double h, double s, double r, double p, double C, double* speedup_out,
                                        double* p_star_out);

/*
 * The attention block in front of the row-parallel output projection (§3.1 Eq. 6 and App. A
 * Eq. 18-19, 23-24: rank m computes the heads it owns from its own input; their outputs, side by
 * side, are the X_m [T, K/P] of caat_rowpar_forward with K / P = heads_q * dh).  The paper fixes
 * neither the positions nor the attention kernel; the four operators below are the usual ones of a
 * decoder, for P ranks side by side like every call of this library:
 *
 *   caat_rope          rotary positions of q and k, or of q with k and v appended to a cache
 *   caat_attn_forward  causal attention over packed prompts, heads_q / heads_k queries per key head
 *   caat_attn_backward its gradients
 *   caat_attn_decode   one token per sequence against a cache
 *
 * Strides: *_stride_rank and *_stride_token count elements between ranks and tokens, so that q, k
 * and v may be views of one fused projection [P, T, (heads_q + 2 heads_k) dh]; within a token the
 * heads are dh apart and a head is contiguous.  Both 0: a contiguous [P, T, heads, dh].  Strides are
 * multiples of 8 elements.
 */

/* Frequency scalings of caat_rope_frequencies for contexts longer than the trained one. */
#define CAAT_ROPE_SCALING_NONE 0
#define CAAT_ROPE_SCALING_LINEAR 1 /* position interpolation: f_j / factor */
#define CAAT_ROPE_SCALING_NTK 2    /* theta raised by factor^(rot / (rot - 2)): the slowest pair is
                                      slowed by `factor`, the fastest keeps its speed */
#define CAAT_ROPE_SCALING_YARN 3   /* per pair between f_j / factor (fewer than 1 turn over the
                                      trained length) and f_j (more than 32 turns), linear in the
                                      number of turns; vectors scaled by 0.1 ln(factor) + 1 */

/*
 * caat_rope_frequencies - host only: the rotation per position (radians) of the rot / 2 pairs,
 * f_j = theta^(-2 j / rot), scaled as above, and the factor on the rotated vectors.
 *   rot      rotated elements of a head, even, 2..256 (4.. for NTK)
 *   theta    > 1;  factor >= 1 and trained_length > 0 (YARN) are ignored where they play no part
 *   inv_freq host, rot / 2 doubles (out);  mscale_out may be NULL
 */
CAAT_API caat_status caat_rope_frequencies(int rot, double theta, int scaling, double factor, double trained_length,
                                           double* inv_freq, float* mscale_out);

#define CAAT_ROPE_FLAG_INTERLEAVED 0x1u /* pairs (2 j, 2 j + 1); default: (j, j + rot / 2) */
#define CAAT_ROPE_FLAG_BACKWARD 0x2u    /* rotate by the negative angle: the gradient of the call
                                           (mscale multiplies there too) */

/*
 * caat_rope - rotary positions.  With t = position * inv_freq[j] (evaluated in double, so far
 * positions keep their angle), pair (a, b) of every head becomes
 *   (mscale (a cos t - b sin t), mscale (b cos t + a sin t)),
 * in fp32, rounded once; elements rot..dh-1 of a head are copied.
 *
 *   q, k       device bf16 [P, T, heads_q | heads_k, dh], strided as above; heads_q or heads_k may
 *              be 0 (the pointer is then ignored)
 *   q_out      device bf16 [P, T, heads_q, dh] contiguous, or q itself (in place, q's strides)
 *   slots      NULL: k_out is [P, T, heads_k, dh] contiguous or k itself.
 *              Else device int64 [T]: token t's rotated k goes to row slots[t] of k_out
 *              [P, cache_rows, heads_k, dh] and its v, unchanged, to the same row of v_out; slot -1
 *              skips the token's k and v (padding).  Any other slot outside [0, cache_rows) is
 *              skipped too and reported by caat_get_device_status as CAAT_ERR_INVALID_ARG.  Two
 *              tokens must not share a slot (which of them a row then holds is unspecified).
 *              Rows without a token keep their contents.
 *   v, v_out   only with slots
 *   positions  device int32 [T], shared by the ranks; NULL: 0..T-1
 *   inv_freq   HOST, rot / 2 doubles, finite; read before return
 *   rot        0 < rot <= dh; rot % 16 == 0 (interleaved: rot % 8 == 0)
 *   dh         dh % 8 == 0, dh <= 256
 * Outputs that are not in place must not overlap the inputs; a tensor turned in place must not share
 * elements with another one, nor with itself between ranks (slices of one projection do not); from one of
 * other strides it must lie apart.  Pointers 16-byte aligned, positions 4, slots 8.
 */
typedef struct caat_rope_args {
  const caat_bf16* q;
  const caat_bf16* k;
  const caat_bf16* v;
  caat_bf16* q_out;
  caat_bf16* k_out;
  caat_bf16* v_out;
  const int32_t* positions;
  const int64_t* slots;
  const double* inv_freq;      /* host */
  caat_stream_t stream;
  caat_timing* timing;
  int64_t T, cache_rows;
  int64_t q_stride_rank, q_stride_token;
  int64_t k_stride_rank, k_stride_token;
  int64_t v_stride_rank, v_stride_token;
  int32_t P, heads_q, heads_k, dh, rot;
  float mscale;
  uint32_t flags;              /* CAAT_ROPE_FLAG_* */
} caat_rope_args;

CAAT_API caat_status caat_rope(const caat_rope_args* args);

/*
 * caat_attn_forward - causal attention over packed sequences, on every rank.  Sequence s owns the
 * queries [cu_q[s], cu_q[s+1]) and the keys [cu_k[s], cu_k[s+1]); its last query sees its last key,
 * so query i of n sees the first i + 1 + (m - n) of m keys (m > n: a cached prefix; m < n: the first
 * queries see none).  Query head h reads key head h / (heads_q / heads_k).
 *   S = scale q k^T over the visible keys, out = softmax(S) v, lse = log(sum exp S)
 * with S, the softmax and the sums in fp32; the probabilities are rounded to bf16 for the product
 * with v.  A row that sees no key gives out = 0 and lse = -inf.  Rows of out and lse behind the last
 * sequence are not written.  Values of k and v outside a sequence's keys never reach its rows.
 *
 *   q          device bf16 [P, Tq, heads_q, dh], strided
 *   k, v       device bf16 [P, Tk, heads_k, dh], strided
 *   out        device bf16 [P, Tq, heads_q * dh] contiguous; must not overlap the inputs
 *   lse        device fp32 [P, heads_q, Tq], or NULL
 *   cu_q, cu_k HOST int32 [n_seq + 1], non-decreasing, from >= 0 up to <= Tq | Tk; cu_k NULL: cu_q.
 *              Read before return.  A sequence has at most 2^25 queries and keys.
 *   dh         dh % 8 == 0, dh <= 128;  heads_q % heads_k == 0;  scale > 0, finite
 *   workspace  caat_attn_workspace_size(..., CAAT_VARIANT_ATTN) bytes, 256-byte aligned; NULL when
 *              that is 0.  Clobbered; two calls that may overlap on the GPU need one each.
 * Capturable in a CUDA graph (which then holds the offsets of the captured call).
 */
typedef struct caat_attn_args {
  const caat_bf16* q;
  const caat_bf16* k;
  const caat_bf16* v;
  caat_bf16* out;
  float* lse;
  const int32_t* cu_q;         /* host */
  const int32_t* cu_k;         /* host, or NULL */
  void* workspace;
  size_t ws_bytes;
  caat_stream_t stream;
  caat_timing* timing;
  int64_t Tq, Tk;
  int64_t q_stride_rank, q_stride_token;
  int64_t k_stride_rank, k_stride_token;
  int64_t v_stride_rank, v_stride_token;
  int32_t n_seq, P, heads_q, heads_k, dh;
  float scale;
  uint32_t flags;              /* 0 */
} caat_attn_args;

CAAT_API caat_status caat_attn_forward(const caat_attn_args* args);

/*
 * caat_attn_backward - gradients of caat_attn_forward.  With P the probabilities (recomputed from lse),
 * D = rowsum(dout * out):
 *   dv = P^T dout,  dS = scale P (dout v^T - D),  dq = dS k,  dk = dS^T q
 * (of the first queries of a sequence, which see 128 keys at most, D is the sum of P (dout v^T) instead: the
 * same without the rounding of out),
 * sums in fp32 (over the queries of every head that shares a key head, too, in a fixed order: results
 * do not change from run to run); P and dS are rounded to bf16 as operands of the products.
 *
 *   q, k, v, cu_q, cu_k, scale, sizes  as in the forward
 *   out, lse    the forward's results;  dout  device bf16 [P, Tq, heads_q * dh]
 *   dq [P, Tq, heads_q, dh], dk, dv [P, Tk, heads_k, dh]  device bf16, contiguous (out).  Keys that no
 *               query sees get zeros; rows outside every sequence are not written.
 *   workspace   caat_attn_workspace_size(..., CAAT_VARIANT_ATTN_BWD) bytes, 256-byte aligned; as above
 * Outputs must not overlap the inputs or each other.  Values that are not finite make the gradients of
 * their own sequence unspecified; they never reach another sequence's.  Capturable as the forward.
 */
typedef struct caat_attn_bwd_args {
  const caat_bf16* q;
  const caat_bf16* k;
  const caat_bf16* v;
  const caat_bf16* out;
  const float* lse;
  const caat_bf16* dout;
  caat_bf16* dq;
  caat_bf16* dk;
  caat_bf16* dv;
  const int32_t* cu_q;         /* host */
  const int32_t* cu_k;         /* host, or NULL */
  void* workspace;
  size_t ws_bytes;
  caat_stream_t stream;
  caat_timing* timing;
  int64_t Tq, Tk;
  int64_t q_stride_rank, q_stride_token;
  int64_t k_stride_rank, k_stride_token;
  int64_t v_stride_rank, v_stride_token;
  int32_t n_seq, P, heads_q, heads_k, dh;
  float scale;
  uint32_t flags;              /* 0 */
} caat_attn_bwd_args;

CAAT_API caat_status caat_attn_backward(const caat_attn_bwd_args* args);

/*
 * caat_attn_decode - attention of one new token per sequence over its cache, on every rank:
 * out[b] = softmax(scale q[b] K[b, :n]^T) V[b, :n], n = lens[b] (the new token's own key included, as
 * caat_rope appended it).  out is the X of caat_rowpar_forward for T = B tokens.
 *   q                device bf16 [P, B, heads_q, dh], strided (q_stride_token between sequences)
 *   k_cache, v_cache device bf16 [P, B, capacity, heads_k, dh] contiguous
 *   lens             DEVICE int32 [B] (it grows from step to step of a captured graph).  0 gives
 *                    out = 0; a length outside [0, capacity] does too, and is reported by
 *                    caat_get_device_status as CAAT_ERR_INVALID_ARG.  Cache rows from lens[b] on are
 *                    never used, whatever they hold.
 *   out              device bf16 [P, B, heads_q * dh] contiguous; must not overlap the inputs
 *   workspace        caat_attn_workspace_size(B, capacity, ..., CAAT_VARIANT_ATTN_DECODE) bytes, 256-byte
 *                    aligned, NULL when that is 0; two calls that may overlap on the GPU need one each.  It is
 *                    0 where a cluster of CTAs takes each segment (sequence, rank, key head, 16 query heads), and
 *                    is not for capacities above 16384, for few segments (fewer than 148 CTAs) of long capacity,
 *                    and for more than 592 CTAs with less than 1 MiB of K and V each
 *   B                at most 4096
 *   dh, heads, scale as in caat_attn_forward
 * Deterministic; capturable.
 */
typedef struct caat_attn_decode_args {
  const caat_bf16* q;
  const caat_bf16* k_cache;
  const caat_bf16* v_cache;
  const int32_t* lens;
  caat_bf16* out;
  void* workspace;
  size_t ws_bytes;
  caat_stream_t stream;
  caat_timing* timing;
  int64_t B, capacity;
  int64_t q_stride_rank, q_stride_token;
  int32_t P, heads_q, heads_k, dh;
  float scale;
  uint32_t flags;              /* 0 */
} caat_attn_decode_args;

CAAT_API caat_status caat_attn_decode(const caat_attn_decode_args* args);

/* Workspace variants of caat_attn_workspace_size. */
#define CAAT_VARIANT_ATTN 0
#define CAAT_VARIANT_ATTN_BWD 1
#define CAAT_VARIANT_ATTN_DECODE 2

/* Bytes of device workspace an attention call of this shape needs (SIZE_MAX for invalid sizes).
 * CAAT_VARIANT_ATTN and _BWD: Tq, Tk, n_seq as in the call; CAAT_VARIANT_ATTN_DECODE: Tq = B,
 * Tk = capacity, n_seq is not used. */
CAAT_API size_t caat_attn_workspace_size(int64_t Tq, int64_t Tk, int n_seq, int P, int heads_q, int heads_k, int dh,
                                         int variant);

/* Bytes of device workspace a forward call of this shape needs (0 for invalid shapes is
 * never returned: invalid shapes give SIZE_MAX).  variant: CAAT_VARIANT_*; for the MLP
 * variant K is F. */
CAAT_API size_t caat_workspace_size(int64_t T, int64_t K, int64_t H, int P, int variant);

/*
 * caat_sync_mask - host-only sync-set bookkeeping (App. A.2 Eq. 22; §3): n_s = floor(H p)
 * in double, S = first n_s channels (sync_idx NULL) or the given list, validated exactly as
 * the forward calls validate it.  mask_out (host, H bytes, may be NULL) receives 1 for
 * shared and 0 for private channels; n_sync_out (may be NULL) receives n_s.  No GPU needed.
 */
CAAT_API caat_status caat_sync_mask(int64_t H, double p, const int32_t* sync_idx, uint8_t* mask_out,
                           int64_t* n_sync_out);

/* Synchronizes `stream`, returns the device status word recorded by bounded waits since the
 * last call (0 = none; low byte = caat_status, upper bits = where) and clears it. */
CAAT_API caat_status caat_get_device_status(caat_stream_t stream, int32_t* status_out);

/* Event recorder for per-kernel device timing (outside the hot path: create once).
 * Each forward call given a recorder appends one record: events before the first kernel and
 * after each kernel it launches.  caat_timing_read synchronizes on the last event and
 * returns, for record i and kernel j, ms[i * max_kernels + j]. */
CAAT_API caat_status caat_timing_create(int capacity, caat_timing** out);
CAAT_API caat_status caat_timing_destroy(caat_timing* t);
CAAT_API caat_status caat_timing_reset(caat_timing* t);
CAAT_API caat_status caat_timing_read(caat_timing* t, float* ms, int max_records, int max_kernels,
                             int* n_records, int* n_kernels);

CAAT_API const char* caat_status_string(caat_status s);
CAAT_API const char* caat_version(void);

#ifdef __cplusplus
}
#endif
#endif /* CAAT_H_ */
