/*
 * moe_ragged_bf16.h - C ABI of the deterministic ragged BF16 grouped GEMM for
 * Mixture-of-Experts expert projections, built for AMD MI355X (gfx950).
 *
 * Operations (Cake ragged BF16 grouped GEMM API page, docs.flashinfer.ai,
 * introduction and operations table), for every expert e with rows
 * s_e = offs[e-1] (0 for e == 0) up to t_e = offs[e]:
 *
 *   fwd    Y [s_e:t_e] = X[s_e:t_e] @ W[e]^T        Y  [M, N]    bf16
 *   dgrad  dX[s_e:t_e] = G[s_e:t_e] @ W[e]          dX [M, K]    bf16
 *   wgrad  dW[e]       = G[s_e:t_e]^T @ X[s_e:t_e]  dW [E, N, K] bf16 or fp32
 *
 * with all operands bf16, products summed in fp32 in one fixed order (no atomics),
 * so every output is bitwise identical from run to run on one device with one
 * build.  An expert with no rows gets an exactly-zero (+0.0) dW.  wgrad can
 * instead accumulate into dW (a Megatron-style main_grad), bitwise equal to
 * adding this library's own overwrite dW in dW's dtype (flashinfer PR #8924,
 * "Design and numerics"): fp32, dW[e] = RN32(dW[e] + G_e^T X_e), one IEEE fp32
 * add of the finished product per element; bf16, the bf16 overwrite result is
 * added in bf16: RNE_bf16(RN32(dW[e] + RNE_bf16(G_e^T X_e))).
 *
 * Common conventions of every entry point below:
 *
 *  - Pointers.  Every tensor pointer is a DEVICE pointer on the current HIP
 *    device.  Tensors are dense and row-major: X [m_rows, k], W [E, n, k],
 *    G and Y [m_rows, n], dX [m_rows, k], dW [E, n, k] (k is the unit-stride
 *    dimension of X, W, dX and dW; n of G and Y).  Every tensor pointer must be
 *    16-byte aligned, except offs, which needs 4-byte alignment.  Pointers to
 *    tensors with a row dimension (X, G, Y, dX) may be NULL when m_rows == 0;
 *    all others must be non-NULL.
 *  - Groups.  offs holds num_groups int32 cumulative END offsets, on the device;
 *    the host never reads it.  A caller holding m_indptr[E + 1] (leading zero)
 *    passes m_indptr + 1.  Offsets must be non-decreasing and within
 *    [0, m_rows].  An array that breaks this still accesses no memory out of
 *    bounds: the kernels use end[e] = max over e' <= e of
 *    min(max(offs[e'], 0), m_rows), so it gives the results of that sanitised
 *    array.  Rows at or past end[E-1] belong to no group: fwd and dgrad leave those output rows
 *    untouched and wgrad ignores them.
 *  - Shapes.  1 <= num_groups <= 1024, m_rows >= 0, n >= 8 with n % 8 == 0,
 *    k >= 8 with k % 8 == 0.  (The API page states n % 256 == 0 and k % 64 == 0
 *    for its stable forward entry; here both only need multiples of 8, i.e.
 *    rows of whole 16-byte chunks, the unit of every load and store: the last
 *    256-wide output tile along n or k may be partial, and a reduction over k
 *    (fwd) or n (dgrad) that is not a multiple of 32 ends in a partial stage
 *    whose missing columns load as zeros.)
 *  - Ownership.  The caller owns every buffer.  The library allocates and frees
 *    no device memory, never synchronises the stream or the device, keeps no
 *    pointer after returning and reads no device memory on the host.  Inputs and
 *    outputs must stay alive until the stream has passed the enqueued work.
 *  - Streams.  All work is enqueued on `stream` (a hipStream_t; NULL is the null
 *    stream), in order.  Calls are thread-safe; the only global state is a
 *    per-device property cache filled once.
 *  - Errors.  Every entry returns an mdg_status.  On a validation error nothing
 *    is enqueued and no output is touched.  No exception or abort crosses the
 *    ABI.  A failed kernel launch returns MDG_EHIP.
 */
#ifndef MOE_RAGGED_BF16_H
#define MOE_RAGGED_BF16_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Entry points are the library's only exported symbols (it is built with
   hidden visibility by default). */
#if defined(__GNUC__) || defined(__clang__)
#define MDG_API __attribute__((visibility("default")))
#else
#define MDG_API
#endif

#define MDG_ABI_VERSION 6

typedef enum {
  MDG_OK = 0,
  MDG_EINVAL = 1,        /* null pointer, negative size, misaligned pointer, bad enum */
  MDG_EUNSUPPORTED = 2,  /* shape outside the supported set, or device is not gfx950 */
  MDG_EOVERLAP = 3,      /* an output shares a byte with an input, offs or the workspace */
  MDG_EWORKSPACE = 4,    /* workspace missing or smaller than required */
  MDG_EHIP = 5,          /* the HIP runtime reported an error when enqueueing */
  MDG_ENOMEM = 6         /* host memory for a prepared launch could not be allocated */
} mdg_status;

/* MDG_E4M3: 8-bit floating point (4 exponent and 3 mantissa bits, no infinities), taken where it is named. */
typedef enum { MDG_BF16 = 0, MDG_FP32 = 1, MDG_E4M3 = 2 } mdg_dtype;

/* Version of this ABI (MDG_ABI_VERSION of the header the library was built with). */
MDG_API int grouped_det_gemm_abi_version(void);

/* Static, NUL-terminated description of a status code (never NULL; an unknown
   code gives "unknown status"). */
MDG_API const char* grouped_det_gemm_status_string(int status);

/*
 * Bytes of device workspace grouped_det_gemm_fwd (resp. _dgrad) needs for these
 * sizes: a small plan table plus fp32 partial tiles of the tail split described
 * below (at most 8 KiB + 64 MiB).  It depends on the sizes only (never on offs or
 * the device).  Returns 0 for invalid sizes.
 */
MDG_API size_t grouped_det_gemm_fwd_workspace_bytes(int64_t m_rows, int64_t n, int64_t k,
                                                    int32_t num_groups);
MDG_API size_t grouped_det_gemm_dgrad_workspace_bytes(int64_t m_rows, int64_t n, int64_t k,
                                                      int32_t num_groups);

/*
 * fwd: Y[s_e:t_e] = X[s_e:t_e] @ W[e]^T  (API page, operations table, "fwd").
 *   x  [m_rows, k] bf16, read.        w [num_groups, n, k] bf16, read.
 *   offs [num_groups] int32, read.    y [m_rows, n] bf16, written (rows of groups only).
 *   workspace: device buffer of at least grouped_det_gemm_fwd_workspace_bytes()
 *      bytes, 256-byte aligned, owned by the caller, contents on entry ignored;
 *      must not overlap any other argument.  Two calls that share a workspace must
 *      be ordered on one stream.
 * Work is scheduled as 256 x 256 output tiles (units).  When the number of units
 * U leaves a remainder T = U mod 256 that would occupy only part of the GPU in
 * the last round, each of those last T units is cut into S consecutive ranges
 * of its reduction (S <= 8, a function of U and the sizes only); each range is
 * summed in fp32 in the one fixed order and a second kernel adds the S partial
 * tiles in range order before rounding to bf16.  Every output is therefore
 * still a fixed function of the inputs: bitwise identical from run to run.
 * m_rows == 0 enqueues nothing.  y must not overlap x, w, offs or the workspace.
 */
MDG_API mdg_status grouped_det_gemm_fwd(const void* x, const void* w, const int32_t* offs, void* y,
                                        int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                        void* workspace, size_t workspace_bytes, void* stream);

/*
 * fwd for callers that cannot allocate device memory at all (code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation): the
 * arguments and results of grouped_det_gemm_fwd, bit for bit, without a
 * workspace argument.  Its scratch (the tail plan and the fp32 partial tiles
 * of the tail split) is a static device array of the library, 64 MiB + 8 KiB,
 * the largest workspace any fwd call needs, so every size grouped_det_gemm_fwd
 * accepts is accepted (a size needing more would get MDG_EWORKSPACE).  Each
 * device the library runs on holds its own copy from the library's loading on
 * that device until the process ends; its address is looked up once per
 * device, at the first call.  No call allocates or frees memory, synchronises
 * or copies; only kernels are enqueued on `stream`.
 * Every call on one device shares that device's array, and nothing in it needs
 * to start cleared: each call writes the plan and partial tiles before reading
 * them, in stream order.  Calls that may overlap on one device (on different
 * streams, or from different threads without ordering) RACE on the array and
 * give undefined results: order them on one stream.
 * m_rows == 0 enqueues nothing.  y must not overlap x, w or offs.
 */
MDG_API mdg_status grouped_det_gemm_fwd_noalloc(const void* x, const void* w, const int32_t* offs, void* y,
                                                int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                                void* stream);

/*
 * dgrad: dX[s_e:t_e] = G[s_e:t_e] @ W[e], W read in place (API page, operations
 * table, "dgrad").
 *   g  [m_rows, n] bf16, read.        w [num_groups, n, k] bf16, read.
 *   offs [num_groups] int32, read.    dx [m_rows, k] bf16, written (rows of groups only).
 *   workspace: as for fwd, of at least grouped_det_gemm_dgrad_workspace_bytes()
 *      bytes; the same tail split applies (the reduction here runs over n).
 * m_rows == 0 enqueues nothing.  dx must not overlap g, w, offs or the workspace.
 */
MDG_API mdg_status grouped_det_gemm_dgrad(const void* g, const void* w, const int32_t* offs, void* dx,
                                          int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace grouped_det_gemm_wgrad needs for these sizes: a small
 * work table plus fp32 partial tiles of the fixed-order row split.  It depends
 * on the sizes only (never on offs or the device), so the host can allocate it
 * without a sync.  Returns 0 for invalid sizes.
 */
MDG_API size_t grouped_det_gemm_wgrad_workspace_bytes(int64_t m_rows, int64_t n, int64_t k,
                                                      int32_t num_groups);

/*
 * wgrad: dW[e] = G[s_e:t_e]^T @ X[s_e:t_e]  (API page, operations table, "wgrad";
 * accumulate from flashinfer PR #8924, "Deterministic weight-gradient
 * accumulation" and "Design and numerics").
 *   g [m_rows, n] bf16, read.   x [m_rows, k] bf16, read.   offs [num_groups] int32, read.
 *   dw [num_groups, n, k] of dw_dtype (MDG_BF16 or MDG_FP32):
 *      accumulate == 0: written; an expert with no rows gets +0.0 everywhere.
 *      accumulate != 0: read and written as dw = RN32(dw + dW_e) (MDG_FP32) or
 *        dw = RNE_bf16(RN32(dw + RNE_bf16(dW_e))) (MDG_BF16: both bf16 values
 *        widen exactly, one fp32 add, one rounding).  The add is done for empty
 *        experts too, so -0.0 becomes +0.0 as an add of the zero dW would make
 *        it.  m_rows == 0 then enqueues nothing and leaves dw unchanged.
 *   workspace: device buffer of at least grouped_det_gemm_wgrad_workspace_bytes()
 *      bytes, 256-byte aligned, owned by the caller, contents on entry ignored;
 *      must not overlap any other argument.  Two calls that share a workspace must
 *      be ordered on one stream.
 * The rows of each expert are split into fixed-size consecutive chunks whose
 * size depends only on (m_rows, n, k, num_groups); chunk partials are summed in
 * chunk order by a second kernel on the same stream.  dw must not overlap g, x,
 * offs or the workspace.
 */
MDG_API mdg_status grouped_det_gemm_wgrad(const void* g, const void* x, const int32_t* offs, void* dw,
                                          int dw_dtype, int accumulate,
                                          int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rows per chunk of the wgrad row split for these sizes (a pure function of the
 * sizes; exposed so tests can build cases with and without a split).
 * Returns 0 for invalid sizes.
 */
MDG_API int64_t grouped_det_gemm_wgrad_chunk_rows(int64_t m_rows, int64_t n, int64_t k,
                                                  int32_t num_groups);

/*
 * Zero fill of the rows that belong to no group: out[r, :] = 0 for
 * end <= r < m_rows (Cake ragged BF16 grouped GEMM API page,
 * introduction: groups are consecutive row ranges ending at offs[E-1]; the row
 * padding case of flashinfer PR #8924, "Tests").  fwd and dgrad leave those
 * rows untouched; an autograd wrapper uses this to give them a defined value
 * (zero: they depend on no input) without the host reading offs.
 *   out [m_rows, row_bytes] bytes, row-major, 16-byte aligned; row_bytes a
 *     positive multiple of 16 (at most 2^24).  Written only in the rows named.
 *   offs [num_groups] int32 on the device.  end is the last group end the
 *     GEMM entry points use: the maximum of the offsets clamped to [0, m_rows],
 *     i.e. offs[num_groups-1] for a valid array.  An m_indptr caller passes
 *     m_indptr + 1.
 * m_rows == 0 enqueues nothing.  out must not overlap offs.
 */
MDG_API mdg_status grouped_det_gemm_zero_pad_rows(void* out, const int32_t* offs, int64_t m_rows, int64_t row_bytes,
                                                  int32_t num_groups, void* stream);

/*
 * Prepared launches (Cake ragged BF16 grouped GEMM API page, "Prepared
 * launches": prepare once, launch many times with no allocation and no host
 * synchronisation, capturable into a graph, still valid after new offsets or
 * values are written into the bound buffers).
 *
 * grouped_det_gemm_prepare_{fwd,dgrad,wgrad} take exactly the arguments of the
 * one-shot entry of the same operation (without the stream), run all of its
 * checks and return the same status; on MDG_OK, *launch receives a new
 * host-side object holding the bound pointers and the computed kernel
 * parameters (on any error *launch is set to NULL).  It belongs to the caller,
 * who releases it with grouped_det_gemm_launch_free.  The bound buffers are
 * not copied or owned: they must stay allocated while the launch may be
 * enqueued and until the stream has passed the enqueued work.
 *
 * grouped_det_gemm_launch enqueues the prepared kernels on `stream` (they run
 * exactly as the one-shot entry's would, reading offs and the data on the
 * device at that time): no validation beyond a NULL check and that the current
 * HIP device is the one current at preparation (else MDG_EINVAL), no
 * allocation, no synchronisation and no memset or copy, so it may be called
 * while the stream is being captured into a HIP graph.  Every launch (and
 * every replay of a graph holding one) computes again; an accumulating wgrad
 * adds again.  Launches that share a workspace or an output must be ordered on
 * one stream.  A prepared launch may be used from several threads.
 */
typedef struct mdg_launch mdg_launch;

typedef struct {
  int32_t op;               /* 0 fwd, 1 dgrad, 2 wgrad */
  int32_t device;           /* HIP device of the preparation */
  int32_t kernels;          /* kernels one launch enqueues (0: nothing to do) */
  int32_t gemm_grid;        /* workgroups of the GEMM kernel's persistent grid */
  int32_t dw_dtype;         /* wgrad: MDG_BF16 or MDG_FP32 */
  int32_t accumulate;       /* wgrad: 1 if the launch adds into dw */
  int32_t chunk_rows;       /* wgrad: rows per chunk of the fixed-order row split */
  int32_t tail_slots;       /* fwd/dgrad: fp32 partial tiles available to the tail split */
  int64_t workspace_bytes;  /* workspace bytes the launch uses */
} mdg_launch_info;

MDG_API mdg_status grouped_det_gemm_prepare_fwd(const void* x, const void* w, const int32_t* offs, void* y,
                                                int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                                void* workspace, size_t workspace_bytes, mdg_launch** launch);
MDG_API mdg_status grouped_det_gemm_prepare_dgrad(const void* g, const void* w, const int32_t* offs, void* dx,
                                                  int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                                  void* workspace, size_t workspace_bytes, mdg_launch** launch);
MDG_API mdg_status grouped_det_gemm_prepare_wgrad(const void* g, const void* x, const int32_t* offs, void* dw,
                                                  int dw_dtype, int accumulate,
                                                  int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                                  void* workspace, size_t workspace_bytes, mdg_launch** launch);
MDG_API mdg_status grouped_det_gemm_launch(const mdg_launch* launch, void* stream);
/* Describes a prepared launch (MDG_EINVAL for NULL arguments). */
MDG_API mdg_status grouped_det_gemm_launch_info(const mdg_launch* launch, mdg_launch_info* info);
/* Releases a prepared launch (NULL is ignored).  Work already enqueued is unaffected. */
MDG_API void grouped_det_gemm_launch_free(mdg_launch* launch);

/*
 * ---------------------------------------------------------------------------
 * Around the expert products: routing, the plan, rows in and out
 * ---------------------------------------------------------------------------
 * These make what the products above read (offs, packed rows) and take their
 * outputs back to tokens.  The conventions above hold, with these additions:
 * tokens >= 0, 1 <= experts <= 1024, 1 <= top_k <= 32, tokens * top_k at most
 * 4,000,000; a "slot" is a (token, choice) pair, number token * top_k + choice;
 * dtype is MDG_BF16 or MDG_FP32 and names the type of the large tensors.  Sums
 * are in fp32 (probability sums, dot products, rows) or integers, in one fixed
 * order, without floating-point atomics.  Outputs must not overlap inputs, the
 * workspace or each other.
 *
 * moe_route_fwd: softmax top-k routing with counts and the balance loss.
 *   logits [tokens, experts] of dtype (aligned to its element), read.
 *   token_mask [tokens] bytes or NULL, read: a token whose byte is 0 is not routed.
 *   An expert is available to a token that is kept and whose logit is not -inf.
 *   idx [tokens, top_k] int32, written: the available experts with the largest
 *     logits, largest first, ties to the lower expert (NaN counts as largest);
 *     -1 in the slots for which no expert is left.
 *   weight [tokens, top_k] fp32, written: normalize != 0: the softmax over the
 *     chosen experts; else their entries in the softmax over the available
 *     ones; 0 in slots without an expert.
 *   counts [experts] int32, written: slots that chose the expert.
 *   loss [1] fp32, written: E / (top_k R^2) sum_e counts_e S_e, where R is the
 *     number of tokens with an available expert and S_e the sum over tokens of
 *     the expert's softmax probability; 0 when R == 0.
 *   balance [experts] fp32, written: E counts_e / (top_k R^2), the derivative
 *     of loss by S_e (counts are constants), for moe_route_bwd.
 *   workspace: at least moe_route_fwd_workspace_bytes() bytes (may be 0, then
 *     NULL will do), 256-byte aligned, contents on entry ignored.
 *   top_k <= experts.  tokens == 0 writes counts, loss and balance (zeros).
 * A NaN or +inf logit makes its row's weights, and with them loss, NaN.
 */
MDG_API size_t moe_route_fwd_workspace_bytes(int64_t tokens, int32_t experts);
MDG_API mdg_status moe_route_fwd(const void* logits, int dtype, const uint8_t* token_mask, float* weight,
                                 int32_t* idx, int32_t* counts, float* loss, float* balance, int64_t tokens,
                                 int32_t experts, int32_t top_k, int normalize, void* workspace,
                                 size_t workspace_bytes, void* stream);

/*
 * moe_route_bwd: the gradient of moe_route_fwd's weight and loss by the logits.
 *   logits, weight, idx, balance, normalize: as moe_route_fwd took and left them, read.
 *   dweight [tokens, top_k] fp32 or NULL (zeros); dloss [1] fp32 on the device or NULL (zero), read.
 *   dlogits [tokens, experts] of dtype, written (zeros for a token whose first slot has no expert).
 * tokens == 0 enqueues nothing.
 */
MDG_API mdg_status moe_route_bwd(const void* logits, int dtype, const float* weight, const int32_t* idx,
                                 const float* balance, const float* dweight, const float* dloss, void* dlogits,
                                 int64_t tokens, int32_t experts, int32_t top_k, int normalize, void* stream);

/*
 * moe_plan: where each slot's row goes, the rows sorted by expert and, within
 * an expert, by slot.
 *   idx [tokens, top_k] int32, read (an entry outside [0, experts) has no row).
 *   offs [experts] int32, written: cumulative end offsets, as the grouped products read them.
 *   dest [tokens, top_k] int32, written: the slot's row, -1 for a slot without one.
 *   workspace: at least moe_plan_workspace_bytes() bytes (may be 0), 256-byte aligned.
 */
MDG_API size_t moe_plan_workspace_bytes(int64_t tokens, int32_t top_k, int32_t experts);
MDG_API mdg_status moe_plan(const int32_t* idx, int32_t* offs, int32_t* dest, int64_t tokens, int32_t top_k,
                            int32_t experts, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rows by a plan.  A row has `hidden` elements of dtype, whole 16-byte pieces
 * (hidden * element size a multiple of 16, hidden <= 2^20); packed rows are
 * [tokens * top_k, hidden].  A dest outside [0, tokens * top_k) is a slot
 * without a row.  tokens == 0 enqueues nothing.
 *
 *   moe_dispatch_fwd  rows[dest[t, j]] = x[t]; rows from offs[experts - 1] on: zeros
 *   moe_dispatch_bwd  dx[t] = sum_j drows[dest[t, j]]
 *   moe_combine_fwd   out[t] = sum_j weight[t, j] y[dest[t, j]]
 *   moe_combine_bwd   dy[dest[t, j]] = weight[t, j] dout[t]; rows from offs[experts - 1] on: zeros;
 *                     dweight[t, j] = <dout[t], y[dest[t, j]]> (0 for a slot without a row)
 *
 * Sums over j run in fp32 in the order of j and are rounded to dtype once.
 */
MDG_API mdg_status moe_dispatch_fwd(const void* x, const int32_t* dest, const int32_t* offs, void* rows,
                                    int64_t tokens, int32_t top_k, int32_t experts, int64_t hidden, int dtype,
                                    void* stream);
MDG_API mdg_status moe_dispatch_bwd(const void* drows, const int32_t* dest, void* dx, int64_t tokens, int32_t top_k,
                                    int64_t hidden, int dtype, void* stream);
MDG_API mdg_status moe_combine_fwd(const void* y, const float* weight, const int32_t* dest, void* out, int64_t tokens,
                                   int32_t top_k, int64_t hidden, int dtype, void* stream);
MDG_API mdg_status moe_combine_bwd(const void* dout, const void* y, const float* weight, const int32_t* dest,
                                   const int32_t* offs, void* dy, float* dweight, int64_t tokens, int32_t top_k,
                                   int32_t experts, int64_t hidden, int dtype, void* stream);

/*
 * ---------------------------------------------------------------------------
 * The grouped product in 8 bits
 * ---------------------------------------------------------------------------
 * Values are e4m3 with one scale for each block of 128: of a row of x, 128
 * consecutive values along k; of a weight, 128 x 128 values.  A scale is a power
 * of two 2^(code - 127), one byte (e8m0; 255 is NaN): the smallest with which
 * the block's largest magnitude is at most 448, e4m3's largest value, and not
 * below 2^-127; a value is rounded once, q = RNE(x / scale).  A block that holds
 * a NaN or an infinity has scale NaN and q NaN throughout.  Blocks at the end
 * of a row (k not a multiple of 128) hold what there is.
 *
 * Rows of 8-bit values (of q, and of q_t) lie at a pitch of their length rounded
 * up to 16 bytes, with zeros behind the values.
 *
 * Sizes: m_rows as above; n % 8 == 0; k % 8 == 0; n, k <= 2^20, n * k (each rounded
 * up to 16) < 2^31.
 *
 * grouped_fp8_quantize_rows: x [m_rows, k] of dtype (MDG_BF16 or MDG_FP32), read.
 *   q [m_rows, k], written.  scale, written: 32-bit words of four consecutive
 *   blocks of a row, word [block / 4][row], 4-byte aligned, ceil(ceil(k / 128) / 4)
 *   * m_rows words (codes past the last block are 0).
 *   m_rows == 0 enqueues nothing.
 * grouped_fp8_quantize_weight: w [num_groups, n, k] of dtype, read.
 *   q [num_groups, n, k] and scale [num_groups, ceil(n / 128), ceil(k / 128)], written.
 *   q_t [num_groups, k, n] and scale_t [num_groups, ceil(k / 128), ceil(n / 128)],
 *   written, or both NULL: the same values and scales transposed (a 128 x 128
 *   block transposes into one), with which the product below computes dgrad.
 * grouped_fp8_gemm_fwd: Y[s_e:t_e] = X[s_e:t_e] @ W[e]^T with X and W the values
 *   the 8-bit operands stand for, summed as below, bf16 y [m_rows, n], written
 *   (rows of groups only).
 *   x_dtype MDG_E4M3: x and x_scale as grouped_fp8_quantize_rows wrote them;
 *   else x [m_rows, k] of x_dtype and x_scale NULL: quantised by the call into the
 *   workspace.  w, w_scale: as grouped_fp8_quantize_weight wrote q and scale (or,
 *   with n and k exchanged, q_t and scale_t: dX = G @ W[e]).
 *   workspace: at least grouped_fp8_gemm_fwd_workspace_bytes() bytes (0 for
 *   MDG_E4M3), 256-byte aligned.  m_rows == 0 enqueues nothing.
 *
 * Sums.  The matrix unit takes 8 consecutive values along k (8 i .. 8 i + 7) at a
 * time: their products are aligned to the largest 2^E among them, E the sum of the
 * two values' exponents (a subnormal's is -6; products with a zero are left out of
 * it), and each is cut toward zero to a multiple of 2^(E - 13).  So a product
 * smaller than that is lost beside a large one of its 8, also where other products
 * cancel the large one.  The sums of 8, times the two scales, are added in fp32,
 * and the result is rounded to bf16 once.  Before that rounding it differs from
 * the exact sum by at most
 *   7 * 2^-13 * (sum over the groups of 8 of 2^E times the scales)
 *   + (k + 8) * 2^-24 * (sum of the products' magnitudes),
 * which is more than a sum in fp32 throughout would allow.  (On operands drawn
 * from a normal distribution about one bf16 output in 50 differs from that of fp32
 * sums.)
 * Order.  Without atomics; the same for all rows and columns of a call, whatever
 * the other rows hold and however offs cuts them, so a call repeats bit for bit.
 * With few rows (a function of m_rows, n, num_groups and the device's number of
 * CUs) k is dealt to four partial sums in pieces of 512, which are added at the
 * end; otherwise, and for k <= 512 in any case, it is summed from 0 on.  So with k > 512
 * the same row can get different bits in calls of different sizes (a decode step
 * and a prompt, or with more experts), within the bound above: results are not
 * invariant under batching.
 */
MDG_API mdg_status grouped_fp8_quantize_rows(const void* x, int dtype, void* q, void* scale, int64_t m_rows,
                                             int64_t k, void* stream);
MDG_API mdg_status grouped_fp8_quantize_weight(const void* w, int dtype, void* q, void* scale, void* q_t,
                                               void* scale_t, int32_t num_groups, int64_t n, int64_t k,
                                               void* stream);
MDG_API size_t grouped_fp8_gemm_fwd_workspace_bytes(int64_t m_rows, int64_t n, int64_t k, int32_t num_groups,
                                                    int x_dtype);
MDG_API mdg_status grouped_fp8_gemm_fwd(const void* x, int x_dtype, const void* x_scale, const void* w,
                                        const void* w_scale, const int32_t* offs, void* y, int64_t m_rows,
                                        int64_t n, int64_t k, int32_t num_groups, void* workspace,
                                        size_t workspace_bytes, void* stream);

/*
 * The experts' gated feed-forward.  For every expert e with rows s_e:t_e (offs as above):
 *
 *   fwd    a = X W_gate[e]^T, b = X W_up[e]^T, h = act(a) b
 *   dgrad  dh = dY W_down[e], da = dh b act'(a), db = dh act(a)
 *
 * with act(a) = a s(q(a)), s the logistic function: MDG_SILU, q(a) = a; MDG_GELU_TANH,
 * q(a) = 2 sqrt(2 / pi) (a + 0.044715 a^3), the tanh form of GELU.
 *
 *   x        [m_rows, k] bf16, read.
 *   w        [num_groups, 2 f, k] bf16, read: rows 0 .. f-1 of an expert are W_gate, rows
 *            f .. 2f-1 W_up.
 *   h        [m_rows, f] bf16, written: act(a) b from the fp32 sums a and b, rounded once.
 *   gate_up  fwd: [m_rows, 2 f] bf16, written: a and b rounded (what grouped_det_gemm_fwd
 *            gives for x and w), which the gradient needs; NULL: not kept, with the same h.
 *            dgrad: the same, read; a and b are those bf16 values.
 *   dy       [m_rows, n] bf16, read: the gradient of y = h W_down^T.
 *   w_down   [num_groups, n, f] bf16, read.
 *   dgate_up [m_rows, 2 f] bf16, written: da and db from the fp32 dh, rounded once.  The
 *            rest of the block's backward pass is the products': dx = dgrad(dgate_up, w),
 *            dw = wgrad(dgate_up, x), dw_down = wgrad(dy, h).
 *
 * k, f and n are multiples of 8, 2 f <= 2^20, 2 f k and 2 f n < 2^31; 1 <= num_groups <= 1024; m_rows
 * up to 4,000,000.
 * Rows at or past the last group's end are left as they are, and malformed offs are read
 * as for the products.  s is off by at most 2^-23 (|q| + 3) of its value, which bf16's
 * rounding hides, and 0 below 2^-126.  A value of a or b that is not finite reaches its own h, da and db only;
 * act(-inf), and act' at either infinity, are NaN.
 * workspace: at least grouped_gated_gemm_{fwd,dgrad}_workspace_bytes() bytes (a function of
 * the sizes and, as the kernels are chosen by it, the current device's number of compute
 * units; 0 for invalid sizes), 256-byte aligned, used until the stream has passed the
 * call.  The sums' order is fixed by the sizes and offs: a call repeats bit for bit, and
 * the same row can get different bits in calls of other sizes.  m_rows == 0 enqueues nothing.
 */
typedef enum { MDG_SILU = 0, MDG_GELU_TANH = 1 } mdg_activation;

MDG_API size_t grouped_gated_gemm_fwd_workspace_bytes(int64_t m_rows, int64_t f, int64_t k, int32_t num_groups);
MDG_API mdg_status grouped_gated_gemm_fwd(const void* x, const void* w, const int32_t* offs, void* h, void* gate_up,
                                          int activation, int64_t m_rows, int64_t f, int64_t k, int32_t num_groups,
                                          void* workspace, size_t workspace_bytes, void* stream);
MDG_API size_t grouped_gated_gemm_dgrad_workspace_bytes(int64_t m_rows, int64_t n, int64_t f, int32_t num_groups);
MDG_API mdg_status grouped_gated_gemm_dgrad(const void* dy, const void* w_down, const void* gate_up,
                                            const int32_t* offs, void* dgate_up, int activation, int64_t m_rows,
                                            int64_t n, int64_t f, int32_t num_groups, void* workspace,
                                            size_t workspace_bytes, void* stream);

/*
 * The norms before and after a block, with the block's gate and the scaled residual.  For
 * token t, with rms(v) = sqrt(sum v^2 / hidden + eps):
 *
 *   z = y, or with post_weight y / rms(y) * post_weight
 *   out = residual + scale gate[t] z                 (gate NULL: ones), rounded to dtype
 *   normed = out / rms(out) * weight                 of out as rounded, with weight
 *
 *   residual, y, out, normed  [tokens, hidden] of dtype (MDG_BF16 or MDG_FP32).  y NULL: only the norm of
 *                         the residual; post_weight, gate and out are NULL and weight is not.
 *   weight, post_weight   [hidden] of weight_dtype, or NULL.
 *   gate                  [tokens] fp32.
 *   rstd, post_rstd       [tokens] fp32, written with weight / post_weight (else NULL): 1 / rms(out), 1 / rms(y).
 *
 * block_norm_bwd: the gradients for dout and dnormed (either may be NULL: zeros; not both),
 * with out, rstd and post_rstd as the forward gave them (out: the residual where there was no y):
 *   dresidual, dy         [tokens, hidden] of dtype, rounded once from fp32.
 *   dweight, dpost_weight [hidden] of weight_dtype: sums over the tokens in fp32, rounded once.
 *   dgate                 [tokens] fp32.
 * Each may be NULL (not wanted).  out and rstd may be NULL without dnormed, y without post_weight and gate.
 * workspace: block_norm_bwd_workspace_bytes() bytes, 256-byte aligned, where dweight or
 * dpost_weight is wanted.  tokens == 0: both are zeros, nothing else is enqueued.
 *
 * hidden is a multiple of 8 up to 16384; tokens up to 4,000,000.  Rows, weights and their gradients are 16-byte
 * aligned.  Sums are in fp32 in an order fixed by the sizes; a row whose squares overflow
 * fp32 is divided by infinity.
 */
MDG_API mdg_status block_norm_fwd(const void* residual, const void* y, const void* weight, const void* post_weight,
                                  const float* gate, void* out, void* normed, float* rstd, float* post_rstd,
                                  int64_t tokens, int64_t hidden, int dtype, int weight_dtype, float scale, float eps,
                                  void* stream);
MDG_API size_t block_norm_bwd_workspace_bytes(int64_t tokens, int64_t hidden);
MDG_API mdg_status block_norm_bwd(const void* dout, const void* dnormed, const void* out, const void* y,
                                  const void* weight, const void* post_weight, const float* gate, const float* rstd,
                                  const float* post_rstd, void* dresidual, void* dy, void* dweight, void* dpost_weight,
                                  float* dgate, int64_t tokens, int64_t hidden, int dtype, int weight_dtype,
                                  float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The norm of many gradients, sqrt(sum of g^2), and the gradients clipped by it.
 *
 *   gradients   `count` (up to 65536) tensors, in HOST memory, read before the call returns: data (read) and
 *               out (written by grad_clip; out == data: in place) of `elements` values of dtype MDG_BF16 or
 *               MDG_FP32 on the device, aligned to their type.  Pointers of empty tensors may be NULL.
 *               Up to 2^36 values each, and fewer than 2^31 - 1024 pieces of 32 KiB in all.
 *   norm        one fp32 value on the device, written: the norm, squares and sums in 64 bits.
 *   norm_in     grad_clip: one fp32 value on the device to clip by; NULL: the gradients' norm, which
 *               norm receives (norm is NULL otherwise).
 *
 * grad_clip: out = g * min(1, max_norm / (norm + 1e-6)), the factor rounded to fp32 and the
 * product once to the type; max_norm >= 0.  A norm that is not finite counts as a factor of
 * 1; with that factor a copy keeps every bit, and in place nothing is written.  Outputs share no
 * memory with each other or with another tensor's data.
 * workspace: grad_norm_workspace_bytes(count) bytes, 256-byte aligned (none with norm_in).
 */
typedef struct {
  const void* data;
  void* out;
  int64_t elements;
  int32_t dtype;
  int32_t reserved;
} mdg_gradient;

MDG_API size_t grad_norm_workspace_bytes(int64_t count);
MDG_API mdg_status grad_norm(const mdg_gradient* gradients, int64_t count, float* norm, void* workspace,
                             size_t workspace_bytes, void* stream);
MDG_API mdg_status grad_clip(const mdg_gradient* gradients, int64_t count, float max_norm, const float* norm_in,
                             float* norm, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_RAGGED_BF16_H */
