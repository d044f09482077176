/*
 * shardgemm -- the sharded GEMMs of 1-D tensor parallelism and SUMMA's 2-D
 * block accumulation, with every shard of a layer held on one MI355X GPU.
 *
 * Sources (page title, then the section the entry point follows):
 *  [MLX]   "MLX 张量并行（Tensor Parallelism）实战指南：用 AllToShardedLinear 与
 *          ShardedToAllLinear 实现 Llama 多设备推理"
 *  [HSYM]  "Sharded Matrices and How to Multiply Them 精华笔记"
 *  [SUMMA] "ColossalAI 2D 张量并行：基于 SUMMA 的二维模型切分原理与实现"
 *  [EAI]   "拆解EnergonAI的张量并行实现：Linear1D与词表并行的2个关键技巧"
 *
 * Conventions shared by every entry point
 *  - Weights use the (out, in) row-major layout and a linear layer computes
 *    y = x W^T ([MLX] 2.1 and 2.2).  Activations are row-major (tokens, features).
 *  - P shards are emulated on the current HIP device: the shard copies of a
 *    layer live in one allocation, shard r at offset r.
 *  - Pointers named x, y, X, A, Y, workspace are device pointers owned by the
 *    caller.  Layer weights passed to the constructors may be host or device
 *    memory; they are read, never modified ([MLX] 3.1: the source layer is
 *    only read).
 *  - `stream` is a hipStream_t (NULL = the default stream).  Work is enqueued
 *    asynchronously; results are ready after the stream synchronises.
 *  - Validation happens on the host before any device work and returns a
 *    status; sg_last_error() then describes the failure (thread-local).
 *    A device fault surfaces at the next synchronisation of the stream.
 *  - B == 0 tokens is a successful no-op.
 *  - Results are bitwise identical run to run (fixed reduction order).
 *  - Accumulation is fp32; the output dtype is the caller's choice.
 */
#ifndef SHARDGEMM_H
#define SHARDGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SG_OK = 0,
    SG_ERR_INVALID_ARG = 1,   /* null pointer, negative size, bad dtype or epilogue */
    SG_ERR_BAD_MODE = 2,      /* sharding is neither all-to-sharded nor sharded-to-all */
    SG_ERR_NOT_DIVISIBLE = 3, /* a dimension does not split evenly */
    SG_ERR_UNSUPPORTED = 4,   /* valid request this library does not implement */
    SG_ERR_WORKSPACE = 5,     /* workspace missing or too small */
    SG_ERR_OOM = 6,           /* device allocation failed */
    SG_ERR_HIP = 7            /* a HIP runtime call failed */
} sg_status;

typedef enum { SG_ALL_TO_SHARDED = 0, SG_SHARDED_TO_ALL = 1 } sg_mode;
typedef enum { SG_F32 = 0, SG_BF16 = 1, SG_F16 = 2 } sg_dtype;
typedef enum { SG_EPI_NONE = 0, SG_EPI_SWIGLU = 1 } sg_epilogue;
/* activation layouts across ranks ([HSYM] Cases 1-3) */
typedef enum { SG_IN_FULL = 0, SG_IN_SHARDED = 1 } sg_in_layout;   /* (B, in) | (P, B, in/P) */
typedef enum { SG_OUT_FULL = 0, SG_OUT_SHARDED = 1 } sg_out_layout; /* (B, n) | (P, B, n/P) */

typedef struct sg_layer sg_layer; /* opaque, owned by the library */

/* Shard a dense linear layer over P ranks ([MLX] 3.1 shard_linear; slicing
 * rule of [MLX] 3.2).
 *   weight   (out_dims, in_dims) of `dtype`, row-major.
 *   bias     (out_dims) of `dtype`, or NULL.
 *   mode     SG_ALL_TO_SHARDED: rank r keeps out_dims/P weight rows and the
 *            matching bias entries ([MLX] 2.1).  SG_SHARDED_TO_ALL: rank r keeps
 *            in_dims/P weight columns; the whole bias is added once after the
 *            cross-rank sum ([MLX] 2.2).  Anything else: SG_ERR_BAD_MODE.
 *   segments the split dimension is first cut into `segments` equal segments
 *            (a fused weight such as [Wq; Wk; Wv]); rank r keeps its part of
 *            every segment, in segment order ([MLX] 3.2).
 *   P        number of ranks (P >= 1; P == 1 is the unsharded layer).
 * Errors: SG_ERR_NOT_DIVISIBLE when the split dimension is not divisible by
 * segments, or dim/segments not by P ([MLX] 2.1 and 6: a layer whose output
 * width does not split evenly over the devices is rejected; the message
 * names the size and the device count).  *out receives the new layer. */
sg_status sg_shard_linear(const void* weight, sg_dtype dtype, int64_t out_dims, int64_t in_dims,
                          const void* bias, int mode, int segments, int P, void* stream,
                          sg_layer** out);

/* Shard a 4-bit affine quantized linear layer ([MLX] 2.3, 6: group_size 64,
 * bits 4, mode affine).  Stored format: w[o,k] = scale[o,g] * q[o,k] + bias[o,g]
 * with g = k / group_size; eight 4-bit codes per uint32 along k, element k in
 * bits [4 (k mod 8), 4 (k mod 8) + 4).
 *   wq       (out_dims, in_dims/8) uint32.
 *   scales   (out_dims, in_dims/group_size) fp16 bit patterns.
 *   qbiases  (out_dims, in_dims/group_size) fp16 bit patterns.
 *   act      activation dtype of the layer (SG_BF16 or SG_F16).
 *   bias     (out_dims) of `act`, or NULL (the layer bias, as for sg_shard_linear).
 * Only group_size 64 and bits 4 are implemented (else SG_ERR_UNSUPPORTED).
 * Up to 32 tokens run on the streaming kernels, more on a matrix-core tile
 * kernel (both when out_dims % 32 == 0 and the rank's in_dims % 256 == 0, the
 * fragment-major code layout); other shapes take the generic kernel.
 * Sharded-to-all needs (in_dims/segments/P) % group_size == 0 so that no
 * quantization group straddles two ranks (SG_ERR_NOT_DIVISIBLE). */
sg_status sg_shard_quantized_linear(const uint32_t* wq, const uint16_t* scales,
                                    const uint16_t* qbiases, int64_t out_dims, int64_t in_dims,
                                    int group_size, int bits, sg_dtype act, const void* bias,
                                    int mode, int segments, int P, void* stream, sg_layer** out);

/* Shard an MX FP8 layer ([MLX] 2.3: the non-affine quantization mode
 * "mxfp8"; [MLX] 4: such a layer has no quantization biases).  Format read as
 * the OCP Microscaling one: w[o,k] = 2^(scales[o, k/32] - 127) * e4m3(codes[o,k]),
 * codes FP8 E4M3 (sign, 4 exponent bits with bias 7, 3 mantissa bits, 0x7F /
 * 0xFF NaN), scales E8M0 (255 NaN), one per block of 32 inputs of a row.
 *   codes    (out_dims, in_dims) uint8.   scales (out_dims, in_dims/32) uint8.
 *   act      activation dtype: SG_BF16 only (else SG_ERR_UNSUPPORTED).
 *   bias     (out_dims) bf16, or NULL (the layer bias, as for sg_shard_linear).
 * SG_ERR_NOT_DIVISIBLE when in_dims % 32, or for sharded-to-all when a scale
 * block would straddle two ranks ((in_dims/segments/P) % 32).  Up to 16 tokens
 * run on the streaming kernel (codes converted to bf16 in registers) when the
 * shards tile into 16-row blocks and in/P (sharded-to-all) or in is a multiple
 * of 128; more tokens on the matrix-core tile kernels (codes converted to bf16
 * after the LDS or as they are staged; 17 to 32 tokens stay on the streaming
 * kernel for shards that the few-token tiles do not take); other calls take
 * the generic kernel.  sg_layer_copy_shard returns
 * codes (what 0) and scales (what 2); sg_layer_info reports quantized = 2. */
sg_status sg_shard_mxfp8_linear(const uint8_t* codes, const uint8_t* scales, int64_t out_dims,
                                int64_t in_dims, sg_dtype act, const void* bias, int mode, int segments,
                                int P, void* stream, sg_layer** out);

/* All-to-sharded forward ([MLX] 2.1; [HSYM] Case 1: no communication).
 *   x        (B, in_dims) of the layer's dtype, replicated to every rank.
 *   y        gather == 0: (P, B, n_out/P), rank r's output at offset r
 *            (the output stays sharded); gather == 1: (B, n_out) with rank r
 *            in columns [r n_out/P, (r+1) n_out/P) -- the rank-order all-gather
 *            of the vocabulary-parallel head ([EAI], LM head).
 *   epilogue SG_EPI_NONE: n_out = out_dims, y = x W_r^T (+ b_r).
 *            SG_EPI_SWIGLU: the layer must be all-to-sharded with segments == 2
 *            holding [W_gate; W_up]; n_out = out_dims/2 and
 *            y_r = silu(x Wg_r^T) * (x Wu_r^T), silu(z) = z / (1 + e^-z), computed
 *            in fp32 and rounded once ([MLX] 5.2-5.3: the elementwise product
 *            keeps the sharding).  Bias is not allowed with SWIGLU.
 *   y_dtype  SG_F32, SG_BF16 or SG_F16. */
sg_status sg_all_to_sharded(const sg_layer* layer, const void* x, int64_t B, void* y, int gather,
                            int epilogue, sg_dtype y_dtype, void* stream);

/* All-to-sharded forward with explicit activation layouts ([HSYM] Cases 1 and 2).
 *   in_layout  SG_IN_FULL: x (B, in_dims), replicated to every rank (Case 1).
 *              SG_IN_SHARDED: x (P, B, in_dims/P), slice r holding columns
 *              [r in/P, (r+1) in/P) of the activation; every rank all-gathers it
 *              before its matmul (Case 2), which here is the K loop walking the P
 *              slices in order.  SG_ERR_UNSUPPORTED for fragment-stored dense
 *              weights when (in_dims/P) % 32 != 0, for 4-bit layers when
 *              (in_dims/P) is not a multiple of 256 (fragment-stored codes) or
 *              64 (row-major codes), and for MX FP8 layers when it is not a
 *              multiple of 128 (fragment-stored codes) or 32 (row-major codes);
 *              SG_ERR_NOT_DIVISIBLE when P does not divide in_dims.
 *   out_layout SG_OUT_SHARDED: y (P, B, n_out/P) (gather = 0 of sg_all_to_sharded);
 *              SG_OUT_FULL: y (B, n_out), the rank-order all-gather (gather = 1).
 * Everything else as sg_all_to_sharded. */
sg_status sg_all_to_sharded_ex(const sg_layer* layer, const void* x, int in_layout, int64_t B, void* y,
                               int out_layout, int epilogue, sg_dtype y_dtype, void* stream);

/* Sharded-to-all forward ([MLX] 2.2; [HSYM] Case 3 with AllReduce).
 *   x_partial (P, B, in_dims/P) of the layer's dtype; slice r is rank r's
 *            input (columns r of the full activation under the layer's
 *            segments rule).
 *   y        (B, out_dims) of y_dtype: sum over r = 0..P-1 of
 *            x_partial[r] W_r^T, then + bias once.
 *   workspace device scratch of at least sg_sharded_to_all_workspace(layer, B)
 *            bytes, 16-byte aligned (NULL allowed when that is 0); no
 *            initial contents are needed, and the same workspace serves later
 *            calls of any shape.  Calls that share a workspace must not run
 *            concurrently. */
sg_status sg_sharded_to_all(const sg_layer* layer, const void* x_partial, int64_t B, void* y,
                            sg_dtype y_dtype, void* workspace, size_t ws_bytes, void* stream);

/* Sharded-to-all forward with an explicit output layout ([HSYM] Case 3).
 *   out_layout SG_OUT_FULL: y (B, out_dims), the all-reduce (= sg_sharded_to_all).
 *              SG_OUT_SHARDED: y (P, B, out_dims/P), the reduce-scatter: slice r
 *              holds columns [r out/P, (r+1) out/P) of the same rank-order sum
 *              (+ bias once); SG_ERR_NOT_DIVISIBLE when P does not divide out_dims.
 * Everything else, the workspace included, as sg_sharded_to_all. */
sg_status sg_sharded_to_all_ex(const sg_layer* layer, const void* x_partial, int64_t B, void* y,
                               int out_layout, sg_dtype y_dtype, void* workspace, size_t ws_bytes,
                               void* stream);

/* Gated MLP forward, the chain of [MLX] 5.2-5.3: h_r = silu(x W_gate,r^T) *
 * (x W_up,r^T) on every rank (all-to-sharded with the SwiGLU epilogue), then
 * y = sum over r = 0..P-1 of h_r W_down,r^T (+ the down bias once), with the
 * sharded h kept in the workspace instead of a caller array.  Results are
 * bitwise those of sg_all_to_sharded(gate_up, ..., SG_EPI_SWIGLU, act dtype)
 * followed by sg_sharded_to_all(down, ...).
 *   gate_up  all-to-sharded layer, segments = 2 ([W_gate; W_up]), no bias.
 *   down     sharded-to-all layer over the same P, in_dims = gate_up's
 *            out_dims / 2, the same activation dtype.
 *   x        (B, in_dims) of that dtype; y (B, out_dims of down) of y_dtype.
 *   workspace device memory of at least sg_mlp_workspace(...) bytes, 16-byte
 *            aligned, no initial contents needed: the down layer's
 *            sg_sharded_to_all workspace first, then h (when both layers
 *            run on a streaming kernel and B >= 8, stored fragment-major in
 *            the down kernel's operand order so that it reads each 16-token
 *            operand fragment as one contiguous 1 KB).  The same workspace serves later calls of any B
 *            it is large enough for; calls sharing it must not run concurrently.
 * Errors: SG_ERR_INVALID_ARG for layers that do not form such a pair (the
 * message says which rule fails), SG_ERR_WORKSPACE for a missing, small or
 * misaligned workspace; B = 0 is a no-op. */
sg_status sg_mlp(const sg_layer* gate_up, const sg_layer* down, const void* x, int64_t B, void* y,
                 sg_dtype y_dtype, void* workspace, size_t ws_bytes, void* stream);

/* Bytes of workspace sg_mlp needs for B tokens (0 for layers that do not form
 * a gate|up, down pair or B <= 0). */
size_t sg_mlp_workspace(const sg_layer* gate_up, const sg_layer* down, int64_t B);

/* sg_mlp for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * kernels and bitwise the same results as sg_mlp, with the workspace taken
 * from a fixed scratch array of SG_MLP_STATIC_SCRATCH_BYTES (16 MiB) that the
 * library holds on every device it runs on until the process ends.  The
 * caller passes x and y as for sg_mlp; nothing is allocated or freed.
 * Errors: as sg_mlp, and SG_ERR_WORKSPACE when sg_mlp_workspace(gate_up,
 * down, B) exceeds the scratch (on 4096 x 14336 decode-MLP layers over 8
 * ranks the scratch holds every token count up to 64, bf16, MX FP8 and 4-bit
 * layers alike: beyond, the down layer's rank split needs more).
 * All calls on one device share its scratch, so calls that overlap on one
 * GPU (other streams or threads) race: the caller serialises them. */
#define SG_MLP_STATIC_SCRATCH_BYTES (16u << 20)
sg_status sg_mlp_static(const sg_layer* gate_up, const sg_layer* down, const void* x, int64_t B, void* y,
                        sg_dtype y_dtype, void* stream);

/* Backward of an all-to-sharded layer: the vector-Jacobian product of [MLX]
 * 2.1 with its sum_gradients wrapper.  The input x is shared by every rank,
 * so its gradient is the all_sum of the rank gradients, summed here on chip in
 * rank order:
 *   dx (B, in_dims) of dx_dtype = sum over r = 0..P-1 of dy[r] W_r;
 *   dw (P, out_dims/P, in_dims) of dw_dtype, dw[r] = dy[r]^T x, laid out like
 *      rank r's shard (the rows sg_layer_copy_shard returns, segments rule).
 *   x  (B, in_dims) of the layer's dtype (needed for dw only; may be NULL
 *      otherwise); dy (P, B, out_dims/P) of the layer's dtype, the layout of
 *      the forward's sharded output.
 *   workspace device scratch of at least sg_layer_backward_workspace(layer, B)
 *      bytes, 16-byte aligned, or NULL.  dw runs on the matrix cores: up to
 *      128 tokens reading dy and x in place (no workspace), beyond that over
 *      x and dy transposed into the workspace (tokens padded to a multiple of
 *      32), or on the vector units when no workspace is given.  No
 *      initialisation needed; calls that share a workspace must not overlap.
 *      SG_ERR_WORKSPACE when a needed workspace is given too small or
 *      misaligned.
 * dx runs on the forward kernels over a transposed copy of the rank shards
 * that the layer builds on the first backward call that reads it (16-bit
 * layers whose out_dims/P is a multiple of 32 and in_dims of 16; the same
 * bytes as the weights again, held until sg_layer_free; that first call
 * allocates and synchronises the stream).  Backward calls on one layer must not
 * run concurrently with its first one.
 * dx or dw may be NULL (not both).  Dense layers only (SG_ERR_UNSUPPORTED for
 * 4-bit and MX FP8 layers); no bias gradient.  fp32 accumulation; the rank sum
 * is deterministic.  B = 0 is a no-op. */
sg_status sg_all_to_sharded_backward(const sg_layer* layer, const void* x, const void* dy, int64_t B, void* dx,
                                     sg_dtype dx_dtype, void* dw, sg_dtype dw_dtype, void* workspace,
                                     size_t ws_bytes, void* stream);

/* Backward of a sharded-to-all layer ([MLX] 2.2): every rank receives the
 * full gradient dy (B, out_dims) of the summed output, so
 *   dx_partial (P, B, in_dims/P) of dx_dtype, slice r = dy W_r (stays sharded,
 *      no reduction);
 *   dw (P, out_dims, in_dims/P) of dw_dtype, dw[r] = dy^T x_partial[r].
 *   x_partial (P, B, in_dims/P) of the layer's dtype (for dw only).
 * The transposed shard copy needs out_dims % 32 == 0 and (in_dims/P) % 16 == 0.
 * Everything else, the workspace included, as sg_all_to_sharded_backward. */
sg_status sg_sharded_to_all_backward(const sg_layer* layer, const void* x_partial, const void* dy, int64_t B,
                                     void* dx_partial, sg_dtype dx_dtype, void* dw, sg_dtype dw_dtype,
                                     void* workspace, size_t ws_bytes, void* stream);

/* Bytes of workspace the matrix-core weight gradient of either backward needs
 * for B tokens ((out_dims + in_dims) x B rounded up to 32, 16-bit); 0 when it
 * needs none (at most 128 tokens), when the layer's gradients run on the
 * vector units only (fp32, quantized, or shapes whose transposes do not
 * tile), or on bad input. */
size_t sg_layer_backward_workspace(const sg_layer* layer, int64_t B);

/* SUMMA backward ([SUMMA] Matmul_ABT_2D and Matmul_ATB_2D, the gradients of
 * Y = X A): with the inner dimension of each product cut into the q SUMMA step
 * blocks, summed in step order t = 0..q-1,
 *   dX (M, K) fp32 = dY A^T   (dX_ik = sum_t dY_it A_kt^T),
 *   dA (K, N) fp32 = X^T dY   (dA_kj = sum_t X_tk^T dY_tj).
 *   X (M, K), A (K, N), dY (M, N): row-major, of dtype.  dX or dA may be NULL
 *   (not both); each output is overwritten.
 *   workspace device scratch of at least sg_summa_backward_workspace(...)
 *   bytes, 16-byte aligned, or NULL: with it dA runs on the matrix cores over
 *   X^T and the transposed step blocks of dY written into it; without it on
 *   the vector units.  dX always runs on the matrix cores (16-bit dtypes).
 * Errors as sg_summa_matmul (q must divide M, K and N); SG_ERR_WORKSPACE for a
 * workspace below the size the query gives. */
sg_status sg_summa_backward(const void* X, const void* A, const void* dY, sg_dtype dtype, int64_t M, int64_t K,
                            int64_t N, int q, float* dX, float* dA, void* workspace, size_t ws_bytes, void* stream);

/* Bytes of workspace sg_summa_backward's matrix-core dA needs ((K + N) M
 * 16-bit elements): 0 unless dtype is 16-bit, (M/q) % 32 == 0, N % 16 == 0 and
 * K % 8 == 0. */
size_t sg_summa_backward_workspace(sg_dtype dtype, int64_t M, int64_t K, int64_t N, int q);

/* Bytes of workspace sg_sharded_to_all needs for B tokens (0 on bad input, and
 * when the call runs without one).  Non-zero when the output alone gives too
 * few tiles to fill the chip (dense 16-bit and MX FP8 layers beyond 16 tokens,
 * 4-bit layers beyond 32): groups of ranks are then workgroups of their own, their
 * partial tiles stored in the workspace and summed in rank order by a second
 * kernel. */
size_t sg_sharded_to_all_workspace(const sg_layer* layer, int64_t B);

/* SUMMA on a q x q grid ([SUMMA], SUMMA section, equations (1), (2)).
 *   X (M, K) and A (K, N) row-major of `dtype` (SG_BF16 or SG_F16); Y (M, N)
 *   fp32.  Both operands are cut into q x q blocks; for t = 0 .. q-1 every
 *   block performs Y_ij += X_it A_tj.
 *   accumulate 0: Y = X A; 1: Y += X A.
 *   fused      0: q launches, step t adds its block products into Y in place
 *              (the step structure of the derivation); 1: one launch that keeps
 *              each block's accumulator in registers across the q steps.
 *   workspace  device scratch of at least sg_summa_workspace(dtype, K, N, q)
 *              bytes, or NULL.  With it, each call first writes A_t^T for every
 *              t into the workspace in the fragment-major layout the matrix-core
 *              kernels read (as for a linear layer's weights); without it they
 *              read A in place, more slowly.  Contents need no initialisation;
 *              calls that share a workspace must not run concurrently.
 * Errors: SG_ERR_NOT_DIVISIBLE when q does not divide M, K and N or q < 1
 * (P = q x q processors); SG_ERR_WORKSPACE when workspace is not NULL and
 * ws_bytes is below the required size. */
sg_status sg_summa_matmul(const void* X, const void* A, sg_dtype dtype, int64_t M, int64_t K,
                          int64_t N, int q, float* Y, int accumulate, int fused, void* workspace,
                          size_t ws_bytes, void* stream);

/* Bytes of workspace sg_summa_matmul can use for these sizes: K N element
 * sizes for SG_BF16 / SG_F16 when N % 16 == 0 and (K / q) % 32 == 0, else 0
 * (the call then reads A in place whatever workspace it is given). */
size_t sg_summa_workspace(sg_dtype dtype, int64_t K, int64_t N, int q);

/* Layer description (any output pointer may be NULL); quantized: 0 dense,
 * 1 4-bit affine, 2 MX FP8. */
sg_status sg_layer_info(const sg_layer* layer, int64_t* out_dims, int64_t* in_dims, int* mode,
                        int* segments, int* P, sg_dtype* dtype, int* quantized);

/* Copy rank r's stored shard of one layer tensor into dst (device or host).
 *   what 0: weight (dense: (rows_r, cols_r) of dtype; quantized: packed uint32)
 *        1: bias (all-to-sharded: out_dims/P entries; sharded-to-all: the full bias)
 *        2: quantization scales, 3: quantization biases.
 * Synchronous with respect to `stream`; dst_bytes must be at least the size. */
sg_status sg_layer_copy_shard(const sg_layer* layer, int r, int what, void* dst, size_t dst_bytes,
                              void* stream);

/* Release a layer and its device memory (NULL is ignored). */
void sg_layer_free(sg_layer* layer);

/* ---------------------------------------------------------------------------
 * Mixture of experts.  A token goes through k of E experts, each a gated MLP
 * whose layers are sharded over P ranks like any other layer here.  The
 * router chooses (sg_moe_route) and groups the (token, choice) slots by
 * expert; the grouped products (sg_experts_*) run every expert's rows in one
 * launch; sg_moe_combine adds a token's results.  sg_moe_mlp is the chain.
 *
 * Grouped rows.  R rows, sorted by expert: rows offsets[e] .. offsets[e + 1] - 1
 * are expert e's (offsets: E + 1 int32 on the device, not decreasing, NULL
 * only when E == 1: every row is its).  Rows from offsets[E] on belong to no
 * expert: they are not read, and outputs of theirs stay as they were.  What
 * the index arrays hold is not checked on the host; contents outside their
 * range never lead outside the caller's arrays.
 * ------------------------------------------------------------------------- */
typedef struct sg_experts sg_experts; /* opaque, owned by the library */

/* Shard E dense linear layers over P ranks, each by the rules of
 * sg_shard_linear (mode, segments, P); no bias.
 *   weight (E, out_dims, in_dims) of dtype SG_BF16 or SG_F16, host or device
 *   memory.  At most 1024 experts, dimensions of 2^24, 4 GiB an expert and 64
 *   GiB a layer; calls take activation slices (one rank's rows) below 4 GiB
 *   (else SG_ERR_UNSUPPORTED). */
sg_status sg_shard_experts(const void* weight, sg_dtype dtype, int64_t E, int64_t out_dims, int64_t in_dims, int mode,
                           int segments, int P, void* stream, sg_experts** out);

/* The same from MXFP4 weights (sg_quantize_mxfp4's format along the inputs):
 *   codes (E, out_dims, in_dims / 2), scales (E, out_dims, in_dims / 32) uint8.
 * in_dims % 32 == 0 and, sharded-to-all, (in_dims / segments / P) % 32 == 0
 * (SG_ERR_NOT_DIVISIBLE).  E == 1 is a plain MXFP4 layer.  Activations are
 * bf16, the codes turned into bf16 exactly (unless scale times code leaves
 * bf16's range), or MXFP4 themselves (a_scales below). */
sg_status sg_shard_mxfp4_experts(const uint8_t* codes, const uint8_t* scales, int64_t E, int64_t out_dims,
                                 int64_t in_dims, int mode, int segments, int P, void* stream, sg_experts** out);

/* New weights (E, out_dims, in_dims) into a bf16 or fp16 layer, on the stream;
 * nothing is allocated when they are in device memory. */
sg_status sg_experts_update(sg_experts* layer, const void* weight, void* stream);

/* Layer description (any output pointer may be NULL). */
sg_status sg_experts_info(const sg_experts* layer, int64_t* E, int64_t* out_dims, int64_t* in_dims, int* mode,
                          int* segments, int* P, sg_dtype* dtype, int* mxfp4);
void sg_experts_free(sg_experts* layer); /* NULL is ignored */

/* Grouped all-to-sharded product: y_r[m] = x[row(m)] W_{e(m), r}^T.
 *   x        (T, in_dims) of the layer's dtype (bf16 for MXFP4 layers), row
 *            stride ldx elements.
 *   a_scales NULL, or (MXFP4 layers) the scales of MXFP4 activations: x is
 *            then codes (T, in_dims / 2), a_scales (T, in_dims / 32), packed.
 *   rows     NULL: row(m) = m; or (R) int32: row(m) = rows[m] / k (a plan's
 *            slots).  A row outside 0 .. T - 1 reads zeros.
 *   y        (P, R, n / P): n = out_dims, or with SG_EPI_SWIGLU (segments == 2,
 *            [W_gate; W_up]) out_dims / 2 and silu(gate) * up, rounded once. */
sg_status sg_experts_all_to_sharded(const sg_experts* layer, const void* x, const uint8_t* a_scales, int64_t T,
                                    int64_t ldx, const int32_t* offsets, const int32_t* rows, int k, int64_t R,
                                    void* y, int epilogue, sg_dtype y_dtype, void* stream);

/* Grouped sharded-to-all product: y[m] = sum over r of h_r[m] W_{e(m), r}^T in
 * rank order.  h (P, R, in_dims / P) of the layer's dtype, or MXFP4 codes
 * (P, R, in_dims / P / 2) with h_scales (P, R, in_dims / P / 32); y (R, out_dims). */
sg_status sg_experts_sharded_to_all(const sg_experts* layer, const void* h, const uint8_t* h_scales,
                                    const int32_t* offsets, int64_t R, void* y, sg_dtype y_dtype, void* stream);

/* Gradients of the two (bf16 and fp16 layers).
 *   all-to-sharded: dy (P, R, out_dims / P) -> dx (R, in_dims), one row for
 *     every grouped row (a token's are added by sg_moe_combine without
 *     weights), summed over the ranks; dw (E, P, out_dims / P, in_dims), x and
 *     rows as in the forward call (needed for dw only).
 *   sharded-to-all: dy (R, out_dims) -> dh (P, R, in_dims / P);
 *     dw (E, P, out_dims, in_dims / P).
 * dw of an expert without rows is zero.  dx or dw may be NULL (not both). */
sg_status sg_experts_all_to_sharded_backward(const sg_experts* layer, const void* x, int64_t T, int64_t ldx,
                                             const void* dy, const int32_t* offsets, const int32_t* rows, int k,
                                             int64_t R, void* dx, sg_dtype dx_dtype, void* dw, sg_dtype dw_dtype,
                                             void* stream);
sg_status sg_experts_sharded_to_all_backward(const sg_experts* layer, const void* h, const void* dy,
                                             const int32_t* offsets, int64_t R, void* dh, sg_dtype dh_dtype, void* dw,
                                             sg_dtype dw_dtype, void* stream);

/* SwiGLU on its own, on rank-local rows [gate; up] (what an all-to-sharded
 * layer with segments = 2 gives without the epilogue): gu (rows, 2 f) ->
 * h (rows, f) = silu(gate) * up; dh (rows, f) -> dgu (rows, 2 f).  One dtype, in
 * which dgu is stored: one rounding of 16-bit gradients ahead of the layer's own. */
sg_status sg_swiglu(const void* gu, sg_dtype dtype, int64_t rows, int64_t f, void* h, void* stream);
sg_status sg_swiglu_backward(const void* gu, const void* dh, sg_dtype dtype, int64_t rows, int64_t f, void* dgu,
                             void* stream);

/* Router.  For every token the k experts of the largest logits, in falling
 * order, ties to the lowest expert; a logit of -inf (or NaN) closes the expert
 * to the token, and a token with fewer than k open experts has dropped slots.
 *   logits   (T, E) of dtype, row stride ld; E <= 1024, k <= 16, T <= 2^25.
 *   weights  (T, k) fp32: the softmax over the token's open experts, with
 *            normalize over its chosen ones; 0 for a dropped slot.
 *   experts  (T, k) int32, -1 for a dropped slot.
 * and the plan, slot s = t k + j:
 *   offsets  (E + 1): the grouped rows of each expert.
 *   rows     (T k): the slot of each grouped row, in slot order for each
 *            expert; -1 behind the last.
 *   slots    (T, k): the grouped row of each slot, -1 if dropped.
 *   workspace sg_moe_route_workspace(T, E, k) bytes (0 for few slots), no
 *            initial contents; calls that share it must not overlap. */
sg_status sg_moe_route(const void* logits, int64_t ld, sg_dtype dtype, int64_t T, int E, int k, int normalize,
                       float* weights, int32_t* experts, int32_t* offsets, int32_t* rows, int32_t* slots,
                       void* workspace, size_t ws_bytes, void* stream);
size_t sg_moe_route_workspace(int64_t T, int E, int k);

/* Its gradient: dweights (T, k) fp32 -> dlogits (T, E) of dtype, packed; 0 for
 * closed experts.  weights and experts as sg_moe_route gave them; logits may
 * be NULL with normalize. */
sg_status sg_moe_route_backward(const void* logits, int64_t ld, sg_dtype dtype, int64_t T, int E, int k, int normalize,
                                const float* weights, const int32_t* experts, const float* dweights, void* dlogits,
                                void* stream);

/* out[t] (T, D) = sum over j of weights[t][j] * y[slots[t][j]], in choice order,
 * fp32, rounded once.  y (R, D); weights NULL: 1; slots outside 0 .. R - 1 are
 * left out; k <= 16. */
sg_status sg_moe_combine(const void* y, sg_dtype y_dtype, int64_t R, const int32_t* slots, const float* weights,
                         int64_t T, int k, int64_t D, void* out, sg_dtype out_dtype, void* stream);

/* Its gradient, dout, y and dy of one dtype: dy (R, D), dy[slots[t][j]] =
 * weights[t][j] * dout[t], rows of no slot left as they were; dweights (T, k)
 * fp32 = <dout[t], y[slots[t][j]]>, 0 for a slot left out.  Either may be NULL
 * (not both).  A row may stand in slots once. */
sg_status sg_moe_combine_backward(const void* dout, const void* y, sg_dtype dtype, int64_t R, const int32_t* slots,
                                  const float* weights, int64_t T, int k, int64_t D, void* dy, float* dweights,
                                  void* stream);

/* The gated MLP over experts: y[t] = sum over t's slots of weight times
 * down_e(silu(x[t] W_gate,e^T) * (x[t] W_up,e^T)).  h is stored in the layers'
 * dtype (fp16: infinite beyond 65504), the down layer's rows in fp32; bitwise the chain of
 * sg_experts_all_to_sharded (SWIGLU), sg_experts_sharded_to_all (fp32 y) and
 * sg_moe_combine.
 *   gate_up all-to-sharded with segments = 2, down sharded-to-all with
 *   segments = 1, of one E, P and dtype (an MXFP4 layer's is bf16: the pair may
 *   be of MXFP4, of bf16, or of one each).
 *   x (T, in_dims), row stride ldx; weights, offsets, rows, slots: a plan of
 *   T tokens and k choices; y (T, out_dims of down).
 *   workspace sg_moe_mlp_workspace(...) bytes, 16-byte aligned, no initial
 *   contents; calls that share it must not overlap. */
sg_status sg_moe_mlp(const sg_experts* gate_up, const sg_experts* down, const void* x, int64_t T, int64_t ldx,
                     const float* weights, const int32_t* offsets, const int32_t* rows, const int32_t* slots, int k,
                     void* y, sg_dtype y_dtype, void* workspace, size_t ws_bytes, void* stream);
size_t sg_moe_mlp_workspace(const sg_experts* gate_up, const sg_experts* down, int64_t T, int k);

/* MXFP4 (OCP Microscaling): blocks of 32 values share one E8M0 scale byte s,
 * each value an E2M1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign bit), worth
 * code * 2^(s - 127).  Quantisation: s - 127 = floor(log2 max|x|) - 2, within
 * -127 .. 127 (a block of zeros: -127); codes round to nearest even, above 6
 * to 6; a block holding an infinity or a NaN: s = 255 (NaN), codes 0.
 *   x (rows, cols) of dtype, row stride ldx; cols % 32 == 0.
 *   codes (rows, cols / 2), value 2i of a row in the low half of byte i;
 *   scales (rows, cols / 32). */
sg_status sg_quantize_mxfp4(const void* x, sg_dtype dtype, int64_t rows, int64_t cols, int64_t ldx, uint8_t* codes,
                            uint8_t* scales, void* stream);
/* The values it stands for, rounded to dtype (exact in fp32 below 2^128); x packed. */
sg_status sg_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* x,
                              sg_dtype dtype, void* stream);

/* Profiling: arm two hipEvent_t (created with timing enabled; either may be
 * NULL) for the next kernel this thread launches through the library, which
 * records start_event when that kernel begins and stop_event when it ends
 * (hipExtLaunchKernel), so hipEventElapsedTime gives its execution time
 * without launch overhead.  One-shot: disarmed by that launch.  For entry
 * points that launch several kernels, the first one is timed. */
sg_status sg_time_next_launch(void* start_event, void* stop_event);

/* Message describing the last failure on this thread ("" if none). */
const char* sg_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* SHARDGEMM_H */
