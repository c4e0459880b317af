/*
 * sharded_linear.h -- C ABI of one tensor-parallel rank's linear step on gfx950 (MI355X).
 *
 * The step (llm-infra-atlas, "01 · ColumnParallelLinear / RowParallelLinear and the core
 * autograd", section 4): forward Y = X.W^T, input gradient dX = dY.W, and the weight gradient
 * fused into gradient accumulation, main_grad += dY^T.X in fp32, where main_grad is a view of a
 * flat grad_data buffer and W a view of a matching param_data buffer (llm-infra-atlas,
 * "05 · grad/param buffer", sections 4-5).  Collectives are not part of this library.
 *
 * Conventions shared by every entry point
 *   - Matrices are row-major and dense: the leading dimension is the last extent.
 *       X, dX : [T, in]     W : [out, in]     Y, dY : [T, out]     main_grad : [out, in]
 *     T = tokens (sequence x micro-batch rows flattened), in/out = the shard's features.
 *   - bf16 tensors are passed as raw 16-bit storage; main_grad and grad_data are fp32.
 *   - Device pointers must be 16-byte aligned; in and out must be multiples of 8 (32 for the
 *     MXFP8 entry points); T may be any value >= 0.  A zero extent is a no-op.
 *   - Every call is asynchronous on `stream` (a hipStream_t; NULL is the null stream) and
 *     performs no synchronisation, no allocation and no free.  The caller owns all memory.
 *   - Arguments are validated on the host before any HIP call; on error nothing is launched.
 *   - Return value: SL_OK (0) or a negative SL_E* status; sl_status_str() names it.
 *   - Results of the GEMMs are deterministic: the same inputs give the same bits.
 *   - Tile and split choices, and so the sizes the *_workspace_bytes queries return, are the
 *     library's own unless forced through sl_set_tuning(); the library reads no environment
 *     variables.  Keep the knobs unchanged between a query and the calls whose workspace it
 *     sizes; a call that finds its workspace too small returns SL_EWORKSPACE and launches
 *     nothing.
 */
#ifndef SHARDED_LINEAR_H
#define SHARDED_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  SL_OK = 0,
  SL_EINVAL = -1,      /* null pointer with a nonzero extent, negative extent, bad option      */
  SL_EALIGN = -2,      /* device pointer not 16-byte aligned                                   */
  SL_ESHAPE = -3,      /* in/out not a multiple of 8 (32 for MXFP8), or an extent >= 2^31       */
  SL_EWORKSPACE = -4,  /* workspace missing or smaller than sl_wgrad_workspace_bytes()          */
  SL_EHIP = -5,        /* the HIP runtime reported an error at launch                          */
  SL_ECAPACITY = -6    /* an output array given to sl_layout_build is too small                */
};

/* Name of a status code (static storage). */
const char* sl_status_str(int status);

/* ---------------------------------------------------------------------------------------------
 * Tuning knobs, for measurement and tests (not needed for correct use).  sl_set_tuning forces
 * one choice for every later call and workspace query of this process; value -1 restores the
 * built-in choice.  The previous value is stored in *previous when it is not NULL.  Ranges:
 *   SL_TUNE_FWD_CONFIG                bf16 tile configuration 0..25 of the forward (25: 256x192
 *                                     tiles, which only the forward has)
 *   SL_TUNE_{DGRAD,WGRAD}_CONFIG      bf16 tile configuration 0..24 of that product
 *   SL_TUNE_SPLITK                    split count 1..64 of the bf16 weight gradient
 *   SL_TUNE_F8_CONFIG                 block-scaled configuration 0..2, for the weight gradient as
 *                                     well, of the products of two MXFP8 operands (0: 256x256, 1:
 *                                     128x128, 2: 256x128) and of two MXFP4 operands (0: 256x256, 1:
 *                                     128x128, 2: 128x128 staged four deep): one value, set for both
 * An unknown knob or a value out of range returns SL_EINVAL and changes nothing.  The knobs are
 * process-wide atomics: safe to set from any thread, but a call that overlaps a change may see
 * either value, so change them only while no call is being planned.
 * ------------------------------------------------------------------------------------------- */
enum {
  SL_TUNE_FWD_CONFIG = 0,
  SL_TUNE_DGRAD_CONFIG = 1,
  SL_TUNE_WGRAD_CONFIG = 2,
  SL_TUNE_SPLITK = 3,
  SL_TUNE_F8_CONFIG = 4,
  SL_TUNE_COUNT = 5
};
int sl_set_tuning(int32_t knob, int32_t value, int32_t* previous);

/* ---------------------------------------------------------------------------------------------
 * Buffer layout (host only; llm-infra-atlas "05 · grad/param buffer", sections 4.1-4.3 and 5).
 *
 * Places n parameters, numel[] given in model definition order, into one flat buffer:
 *   - in reverse definition order (backprop order), so offset 0 holds the last parameter;
 *   - each parameter start rounded up to a multiple of param_align elements (64 under the
 *     distributed optimizer; the page notes the unit is elements, not bytes);
 *   - a bucket is closed right after the parameter whose end makes (end - bucket_start) reach
 *     bucket_size elements; bucket_size <= 0 puts everything in one bucket;
 *   - each bucket end is rounded up to a multiple of `divisor` (lcm(dp,128), or
 *     lcm(dp,128,65536) with the high-bus-bandwidth option, see sl_bucket_divisor), and the next
 *     bucket starts there.
 * Outputs (caller-owned host arrays): start/end/bucket_id per parameter (definition order);
 * per bucket: offset, padded numel and unpadded numel (param end - bucket start), up to
 * bucket_cap entries; *n_buckets and *total_numel.  If bucket_cap is too small the call
 * returns SL_ECAPACITY and sets *n_buckets to the number needed.  A zero-size parameter is
 * allowed; n = 0 gives total_numel 0 and no buckets.
 * ------------------------------------------------------------------------------------------- */
int sl_layout_build(int32_t n, const int64_t* numel, int64_t param_align, int64_t bucket_size,
                    int64_t divisor, int64_t* start, int64_t* end, int32_t* bucket_id,
                    int32_t bucket_cap, int64_t* bucket_offset, int64_t* bucket_numel,
                    int64_t* bucket_numel_unpadded, int32_t* n_buckets, int64_t* total_numel);

/* Default bucket size in elements, max(40,000,000, 1,000,000 * dp) (same page, section 4.3). */
int64_t sl_default_bucket_size(int64_t dp);

/* Bucket-end divisor lcm(dp, 128), or lcm(dp, 128, 65536) when high_busbw != 0 (section 4.2).
 * Returns 0 for dp <= 0. */
int64_t sl_bucket_divisor(int64_t dp, int32_t high_busbw);

/* ---------------------------------------------------------------------------------------------
 * Gradient-buffer zeroing (same page, section 6.6: grad_data is zeroed once per iteration and
 * never freed).  Writes 0.0f to grad_data[0, numel).  A fill kernel, so it is safe to record in
 * a captured HIP graph.  Also used to prepare a wgrad workspace before its first use.
 * ------------------------------------------------------------------------------------------- */
int sl_grad_buffer_zero(void* stream, float* grad_data, int64_t numel);

/* ---------------------------------------------------------------------------------------------
 * Forward GEMM: Y[T,out] = X[T,in] . W[out,in]^T, bf16 inputs, fp32 accumulation, one
 * round-to-nearest-even to bf16 (atlas page "01", section 4.1).  For a row-parallel weight Y is
 * the partial sum that the following all-reduce would add up.
 * ------------------------------------------------------------------------------------------- */
int sl_linear_fwd(void* stream, const void* X, const void* W, void* Y,
                  int64_t T, int64_t in, int64_t out);

/* ---------------------------------------------------------------------------------------------
 * Input-gradient GEMM: dX[T,in] = dY[T,out] . W[out,in], bf16 in/out, fp32 accumulation
 * (atlas page "01", section 4.2, the dgrad).
 * ------------------------------------------------------------------------------------------- */
int sl_linear_dgrad(void* stream, const void* dY, const void* W, void* dX,
                    int64_t T, int64_t in, int64_t out);

/* ---------------------------------------------------------------------------------------------
 * Weight gradient fused into accumulation: main_grad[out,in] += dY[T,out]^T . X[T,in] in fp32
 * (atlas page "01", section 4.2, gradient_accumulation_fusion).  The micro-batch gradient is
 * never rounded and never stored on its own; main_grad is read and written only inside its
 * [out, in] extent, so neighbouring views and padding of grad_data are untouched.
 *
 * workspace: device memory of at least sl_wgrad_workspace_bytes(T, in, out) bytes (0 when the
 * shape needs no split-K; workspace may then be NULL).  It holds fp32 split-K partial planes
 * [splits][out][in], written and then read within the call; its initial contents do not
 * matter.  A split call launches a second, reducing kernel on the same stream.  Calls that may
 * run concurrently must use distinct workspaces.
 * ------------------------------------------------------------------------------------------- */
size_t sl_wgrad_workspace_bytes(int64_t T, int64_t in, int64_t out);
int sl_linear_wgrad_accum(void* stream, const void* X, const void* dY, float* main_grad,
                          int64_t T, int64_t in, int64_t out,
                          void* workspace, size_t workspace_bytes);

/* ---------------------------------------------------------------------------------------------
 * The weight gradient for callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, and harnesses that forbid hipMalloc.  Same operation, arguments
 * (other than the workspace), results and kernels as sl_linear_wgrad_accum; the split-K partial
 * planes go into a library-owned device array of SL_NOALLOC_SCRATCH_BYTES (64 MiB) that each GPU
 * holds from module load until the process ends.  The call allocates and frees nothing.
 *   - A shape whose plan needs more than that (sl_wgrad_workspace_bytes(T, in, out) >
 *     SL_NOALLOC_SCRATCH_BYTES) returns SL_EWORKSPACE and launches nothing.
 *   - `stream` must belong to the current device (SL_EINVAL otherwise): the array is the current
 *     device's, resolved at the first call on that device.
 *   - Every call on one GPU shares that GPU's array, and its partial planes are written and read
 *     within the call (nothing needs clearing between calls).  Calls that overlap on one GPU --
 *     on different streams, or from different host threads -- race on the array: serialise them.
 * ------------------------------------------------------------------------------------------- */
#define SL_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
int sl_linear_wgrad_accum_noalloc(void* stream, const void* X, const void* dY, float* main_grad,
                                  int64_t T, int64_t in, int64_t out);

/* ---------------------------------------------------------------------------------------------
 * MXFP8 operand variants (NVIDIA Megatron-Core guide "Generalized Tensor Parallelism",
 * section 1.3: E4M3 elements with one E8M0 scale per 32 elements).  A quantised matrix M[r, c]
 * is passed as codes Mq[r, c] (uint8, E4M3FN) and scales Ms[r, c/32] (uint8, E8M0), and stands
 * for deq(q, s) = E4M3(q) * 2^(s - 127).  Blocks run along `in` for both X and W.
 *   fwd:   Y  = deq(Xq).deq(Wq)^T           (bf16 out; block-scaled fp8 MFMA when 128 | in and
 *                                            the scale pointers are 4-byte aligned)
 *   dgrad: dX = dY.deq(Wq)                  (dY, dX bf16)
 *   wgrad: main_grad += dY^T.deq(Xq)        (dY bf16, main_grad fp32)
 * Every dequantised element must be representable in bf16 (an E4M3 value times a power of two
 * whose result is a normal bf16); it then enters the GEMMs exactly.  in must be a multiple of
 * 32.  Code pointers must be 16-byte aligned; scale pointers have no alignment requirement.
 *
 * dgrad and wgrad take a device workspace of at least sl_mxfp8_workspace_bytes(T, in, out)
 * bytes: the MXFP8 operand is dequantised into its front (bf16), the rest serves the bf16
 * weight-gradient split-K planes.  Its initial contents do not matter; calls that may run
 * concurrently must use distinct workspaces.
 * ------------------------------------------------------------------------------------------- */
size_t sl_mxfp8_workspace_bytes(int64_t T, int64_t in, int64_t out);
int sl_linear_fwd_mxfp8(void* stream, const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                        const uint8_t* Ws, void* Y, int64_t T, int64_t in, int64_t out);
int sl_linear_dgrad_mxfp8w(void* stream, const void* dY, const uint8_t* Wq, const uint8_t* Ws,
                           void* dX, int64_t T, int64_t in, int64_t out,
                           void* workspace, size_t workspace_bytes);
int sl_linear_wgrad_accum_mxfp8x(void* stream, const uint8_t* Xq, const uint8_t* Xs,
                                 const void* dY, float* main_grad, int64_t T, int64_t in,
                                 int64_t out, void* workspace, size_t workspace_bytes);

/* sl_mxfp8_dequantize: out[r, c] (bf16) = deq(q, s)[r, c] = E4M3(q[r, c]) * 2^(s[r, c/32] - 127)
 * for q[rows, cols] codes and s[rows, cols/32] scales (section 1.3 block of 32 above).  Exact under
 * the representability rule above (results that are not normal bf16 values are unspecified).
 * cols % 32 == 0 (SL_ESHAPE); q and out 16-byte aligned (SL_EALIGN); the caller owns all buffers.
 * This is the expansion sl_linear_dgrad_mxfp8w and sl_linear_wgrad_accum_mxfp8x perform into
 * their workspace; sl_linear_dgrad on its output gives the same dX bit for bit.
 */
int sl_mxfp8_dequantize(void* stream, const uint8_t* q, const uint8_t* s, void* out, int64_t rows,
                        int64_t cols);

/* ---------------------------------------------------------------------------------------------
 * All-MXFP8 step: the backward GEMMs in MXFP8 as well (NVIDIA Megatron-Core guide "Generalized
 * Tensor Parallelism", section 1.3: in the MXFP8 recipe each GEMM reads E4M3 elements with one
 * E8M0 scale per 32 elements along its own contraction axis; the weight gradient still
 * accumulates into fp32 main_grad, section 3.1).  A tensor read along both axes is quantised
 * twice: rowwise (blocks along the last axis) and columnwise (blocks down the columns, stored
 * transposed so that the consuming GEMM reads k contiguously).
 *   fwd:   sl_linear_fwd_mxfp8 with X, W rowwise                      (above)
 *   dgrad: dX[T,in]         = deq(dYq)[T,out] . deq(WqT)[in,out]^T    dY rowwise, W columnwise
 *   wgrad: main_grad[out,in] += deq(dYqT)[out,T] . deq(XqT)[in,T]^T   dY and X columnwise
 *
 * sl_mxfp8_quantize: x[rows, cols] bf16 (row-major, 16-byte aligned) into rowwise codes
 * q_rows[rows, cols] + scales s_rows[rows, cols/32] and/or columnwise codes q_cols[cols, rows] +
 * scales s_cols[cols, rows/32]; a NULL pair is skipped (each code pointer must come with its
 * scale pointer: SL_EINVAL otherwise).  The rowwise copy needs cols % 32 == 0, the columnwise
 * copy rows % 32 == 0 and cols % 8 == 0 (SL_ESHAPE).  The rule is the OCP MX v1.0 conversion (the pages fix only
 * the block and per-block scaling): per block X = clamp(floor(log2 amax) - 8, -127, 127),
 * scale byte X + 127, codes = E4M3 round-to-nearest-even of x / 2^X saturating at +-448 with
 * the sign kept; an all-zero block stores scale 0 and zero codes.  Inputs must be finite
 * (non-finite elements give unspecified codes).  Code pointers 16-byte aligned.
 *
 * sl_linear_dgrad_mxfp8 / sl_linear_wgrad_accum_mxfp8: the contraction extent (out for dgrad,
 * T for wgrad) must be a multiple of 128, in/out multiples of 8 (SL_ESHAPE); code pointers
 * 16-byte aligned, scale pointers 4-byte aligned (SL_EALIGN).  The weight gradient takes a
 * device workspace of at least sl_mxfp8_wgrad_workspace_bytes(T, in, out) bytes (fp32 split-K
 * planes [splits][out][in]; 0 when the shape needs no split, workspace may then be NULL); its
 * initial contents do not matter, a split call launches a second, reducing kernel on the same
 * stream, and concurrent calls need distinct workspaces.  main_grad is read and written only
 * inside its [out, in] extent.
 * ------------------------------------------------------------------------------------------- */
int sl_mxfp8_quantize(void* stream, const void* x, int64_t rows, int64_t cols, uint8_t* q_rows,
                      uint8_t* s_rows, uint8_t* q_cols, uint8_t* s_cols);
int sl_linear_dgrad_mxfp8(void* stream, const uint8_t* dYq, const uint8_t* dYs, const uint8_t* WqT,
                          const uint8_t* WsT, void* dX, int64_t T, int64_t in, int64_t out);
size_t sl_mxfp8_wgrad_workspace_bytes(int64_t T, int64_t in, int64_t out);
int sl_linear_wgrad_accum_mxfp8(void* stream, const uint8_t* dYqT, const uint8_t* dYsT,
                                const uint8_t* XqT, const uint8_t* XsT, float* main_grad,
                                int64_t T, int64_t in, int64_t out, void* workspace,
                                size_t workspace_bytes);

/* ---- NVFP4 weights -------------------------------------------------------------------------
 * NVIDIA Megatron-Core guide "Generalized Tensor Parallelism", section 1.3 (native NVFP4 param):
 * the weight shard W[out, in] is kept as NVFP4 -- packed 4-bit E2M1 codes, one E4M3 scale per
 * 16 elements along in, and one fp32 per-tensor scale t (set when the optimizer writes the
 * shard) -- and activations and gradients stay bf16:
 *   deq(W)[o][i] = E2M1(code[o][i]) * E4M3(scale[o][i/16]) * t
 *   forward: Y  = X . deq(W)^T          dgrad: dX = dY . deq(W)
 * (the weight gradient does not read W: sl_linear_wgrad_accum applies unchanged).
 *
 * sl_nvfp4_materialize: Wq[rows, cols/2] packed codes (element 2j of a row in the low nibble of
 * byte j) and Ws[rows, cols/16] E4M3 scale bytes into Wm[rows, cols] bf16 holding
 * E2M1(code) * E4M3(scale) -- exact, since every such product is a bf16 value; t is NOT applied.
 * cols % 16 == 0 (the NVFP4 alignment pad; SL_ESHAPE otherwise); Wq and Wm 16-byte aligned
 * (SL_EALIGN); the caller owns all three buffers.  A NaN scale byte (S.1111.111) gives NaN
 * weights.  Wm may be materialised once per optimizer step and reused; materialising it right
 * before each product measured faster on the 8-micro-batch MLP step, since the GEMM then reads a
 * copy that is still in the caches.
 *
 * sl_linear_fwd_nvfp4w / sl_linear_dgrad_nvfp4w: as sl_linear_fwd / sl_linear_dgrad with W = Wm
 * from sl_nvfp4_materialize and w_scale = t: the fp32 accumulators are multiplied by w_scale
 * before the bf16 rounding of Y or dX.  in % 16 == 0 (SL_ESHAPE); w_scale must be finite
 * (SL_EINVAL); the other rules are those of the bf16 entry points.
 * ------------------------------------------------------------------------------------------- */
int sl_nvfp4_materialize(void* stream, const uint8_t* Wq, const uint8_t* Ws, void* Wm, int64_t rows,
                         int64_t cols);
int sl_linear_fwd_nvfp4w(void* stream, const void* X, const void* Wm, float w_scale, void* Y,
                         int64_t T, int64_t in, int64_t out);
int sl_linear_dgrad_nvfp4w(void* stream, const void* dY, const void* Wm, float w_scale, void* dX,
                           int64_t T, int64_t in, int64_t out);

/* ---- MXFP4 -----------------------------------------------------------------------------------
 * Microscaled 4-bit floats (OCP MX v1.0): E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
 * negatives) with one E8M0 scale per 32 elements along the axis that the product contracts.  A
 * quantised matrix M[r, k] (k a multiple of 32) is passed as packed codes Mq[r, k/2] (uint8, element
 * 2j of a row in the low nibble of byte j) and scales Ms[r, k/32] (uint8), and stands for
 *   deq(q, s) = E2M1(q) * 2^(s - 127),  NaN where s = 255.
 * All code pointers must be 16-byte aligned; scale pointers have no alignment requirement (rows of
 * scales are read in whole aligned 4-byte words, so up to 3 bytes beside the array, in the same
 * word as one of its bytes, are read and not used).
 *
 * sl_mxfp4_quantize: x[rows, cols] bf16 (cols % 8 == 0, 16-byte aligned) into rowwise codes
 * q_rows[rows, Cp/2] + scales s_rows[rows, Cp/32] and/or columnwise ones, stored transposed,
 * q_cols[cols, Rp/2] + s_cols[cols, Rp/32], where Cp and Rp are cols and rows rounded up to 32: the
 * last block of a row or column is padded with zeros.  2^24 tiles of 128 x 128 or more are
 * SL_ESHAPE.  A NULL pair is skipped (a code pointer without its scale pointer, or the reverse, is
 * SL_EINVAL).  With v = x / 2^X for the block's shared exponent X (scale byte X + 127):
 *   SL_ROUND_NEAREST     X = clamp(floor(log2 amax) - 2, -127, 127); code = E2M1 of v, round half to
 *                        even, saturating at 6 (the OCP MX conversion)
 *   SL_ROUND_STOCHASTIC  X = the least exponent >= -127 with amax <= 6 * 2^X, so that nothing
 *                        saturates; with s the step of E2M1 at |v| (0.5 below 2, 1 below 4, else 2),
 *                        |code| = s * floor((floor(|v| / s * 2^16) + r) / 2^16).  r is the element's
 *                        16-bit draw: element i of x (row-major) takes half word i % 8 (low halves
 *                        first) of Philox4x32-7 at counter i / 8 with the 64-bit key
 *                        seed + (seed_offset ? *seed_offset : 0) (mod 2^64).  Both copies use the same
 *                        draws; the same key gives the same codes.
 * seed_offset is a device pointer (8-byte aligned) or NULL, read when the kernel runs, so that a
 * captured graph can be replayed with other draws; both are ignored by SL_ROUND_NEAREST.  A block of
 * zeros has scale 0 and codes 0; a block with an infinity or a NaN has scale 255 and codes 0.
 *
 * sl_mxfp4_dequantize: out[rows, cols] (bf16) = deq(q, s); cols % 32 == 0.  Exact; 4 and 6 at scale
 * 253 and every nonzero element from 2 up at scale 254 pass bf16's range and become infinite.
 *
 * Products (fp32 accumulation; bf16 results are rounded once):
 *   fwd:   Y[T,out]           = deq(Xq)[T,in] . deq(Wq)[out,in]^T      in % 32 == 0
 *   dgrad: dX[T,in]           = deq(dYq)[T,out] . deq(WqT)[in,out]^T   out % 32 == 0
 *   wgrad: main_grad[out,in] += deq(dYqT)[out,T] . deq(XqT)[in,T]^T    T % 32 == 0, fp32, in place
 * (the contracted extent is the padded one that sl_mxfp4_quantize writes; the others follow the
 * conventions above; in, out or a contracted extent above 2^23 is SL_ESHAPE).  Each
 * takes a device workspace of at least its query's bytes (16-byte aligned; fp32 split-K planes; 0 when the shape
 * needs no split, workspace may then be NULL): its initial contents do not matter, and calls that may
 * run concurrently need distinct workspaces.  main_grad is read and written only inside [out, in].
 *
 * bf16 activations with MXFP4 weights blocked along in (in % 32 == 0), for serving and for frozen
 * weights; every dequantised weight must be a finite bf16 value or a NaN:
 *   fwd:   Y[T,out] = X[T,in] . deq(Wq)[out,in]^T        dgrad: dX[T,in] = dY[T,out] . deq(Wq)
 * Their workspaces follow the same rules: split-K planes, or for many tokens a bf16 copy of the weight.
 * Up to 16 tokens only the last of these products (dgrad through Wq) may need one.
 * The SL_TUNE_F8_CONFIG knob forces the tiles of the products of two MXFP4 operands too (0: 256x256,
 * 1: 128x128, 2: 128x128 staged four deep), from one token on; it is read by the queries as by the calls.
 * --------------------------------------------------------------------------------------------- */
enum { SL_ROUND_NEAREST = 0, SL_ROUND_STOCHASTIC = 1 };
int sl_mxfp4_quantize(void* stream, const void* x, int64_t rows, int64_t cols, uint8_t* q_rows,
                      uint8_t* s_rows, uint8_t* q_cols, uint8_t* s_cols, int32_t rounding,
                      uint64_t seed, const uint64_t* seed_offset);
int sl_mxfp4_dequantize(void* stream, const uint8_t* q, const uint8_t* s, void* out, int64_t rows,
                        int64_t cols);
size_t sl_mxfp4_fwd_workspace_bytes(int64_t T, int64_t in, int64_t out);
int sl_linear_fwd_mxfp4(void* stream, const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                        const uint8_t* Ws, void* Y, int64_t T, int64_t in, int64_t out,
                        void* workspace, size_t workspace_bytes);
size_t sl_mxfp4_dgrad_workspace_bytes(int64_t T, int64_t in, int64_t out);
int sl_linear_dgrad_mxfp4(void* stream, const uint8_t* dYq, const uint8_t* dYs, const uint8_t* WqT,
                          const uint8_t* WsT, void* dX, int64_t T, int64_t in, int64_t out,
                          void* workspace, size_t workspace_bytes);
size_t sl_mxfp4_wgrad_workspace_bytes(int64_t T, int64_t in, int64_t out);
int sl_linear_wgrad_accum_mxfp4(void* stream, const uint8_t* dYqT, const uint8_t* dYsT,
                                const uint8_t* XqT, const uint8_t* XsT, float* main_grad, int64_t T,
                                int64_t in, int64_t out, void* workspace, size_t workspace_bytes);
size_t sl_mxfp4w_fwd_workspace_bytes(int64_t T, int64_t in, int64_t out);
int sl_linear_fwd_mxfp4w(void* stream, const void* X, const uint8_t* Wq, const uint8_t* Ws, void* Y,
                         int64_t T, int64_t in, int64_t out, void* workspace, size_t workspace_bytes);
size_t sl_mxfp4w_dgrad_workspace_bytes(int64_t T, int64_t in, int64_t out);
int sl_linear_dgrad_mxfp4w(void* stream, const void* dY, const uint8_t* Wq, const uint8_t* Ws,
                           void* dX, int64_t T, int64_t in, int64_t out, void* workspace,
                           size_t workspace_bytes);

/* ---- Vocabulary-parallel embedding -----------------------------------------------------------
 * The table shard W[V, H] (bf16, a param_data view) holds the ids vocab_start .. vocab_start + V - 1;
 * an id outside them is another rank's (any value: it is never used as an index).
 *   fwd:   Y[t]          = bf16(scale * W[ids[t] - vocab_start]), zeros for another rank's id, so that the
 *                          ranks' results add up, as a row-parallel forward's do
 *   wgrad: main_grad[v] += scale * sum of dY[t] over the t with ids[t] - vocab_start = v, fp32, in place;
 *                          rows that no token names are not touched
 * ids[T] are int32 or int64 (ids_bytes 4 or 8, aligned to that).  H % 8 == 0; V up to 2^24; the gradient
 * takes up to 2^26 tokens, T * H up to 2^37 and H up to 2^23 (SL_ESHAPE).  vocab_start >= 0 and scale finite
 * (SL_EINVAL).  The gradient's sums are fp32 in an order that depends on the ids alone: the same call gives
 * the same bits.  It takes a workspace of its query's bytes (0 for few tokens, workspace may then be NULL; 16-byte
 * aligned; initial contents do not matter; calls that may run concurrently need distinct ones) and makes up to three
 * launches.
 * --------------------------------------------------------------------------------------------- */
int sl_embedding_fwd(void* stream, const void* ids, int32_t ids_bytes, const void* W, void* Y, int64_t T,
                     int64_t V, int64_t H, int64_t vocab_start, float scale);
size_t sl_embedding_wgrad_workspace_bytes(int64_t T, int64_t V, int64_t H);
int sl_embedding_wgrad_accum(void* stream, const void* ids, int32_t ids_bytes, const void* dY, float* main_grad,
                             int64_t T, int64_t V, int64_t H, int64_t vocab_start, float scale,
                             void* workspace, size_t workspace_bytes);

/* ---- Root-mean-square norm ---------------------------------------------------------------------
 * Rows x[T, H] (bf16), an optional residual[T, H] (bf16) and the weight w[H] (bf16):
 *   h = bf16(x + residual) (x itself without one)    rstd[t] = (mean(h[t]^2) + eps)^-1/2 (fp32)
 *   y = h * rstd * w
 * sl_rmsnorm_fwd writes y in bf16.  sl_rmsnorm_fwd_mxfp8 writes it in MXFP8 by the rule of
 * sl_mxfp8_quantize, from the product of h, w and rstd in two floats as if it were exact (to 2^-100; below, from its fp32 rounding): rowwise codes q_rows[T, H] +
 * s_rows[T, H/32] (H % 32 == 0) and/or columnwise ones, stored transposed, q_cols[H, T] + s_cols[H, T/32]
 * (T % 32 == 0); a NULL pair is skipped.  A block with an infinity or a NaN has scale 255 (NaN) and codes 0.
 * Both write h (only with a residual; else h may be NULL) and rstd, which the gradient reads; with q_cols rstd has 2 T
 * elements, the second T for what the rounding of the first left:
 *   sl_rmsnorm_bwd: g = w * dY;  dX = rstd * (g - h * rstd^2 * mean(g * h)) + dresidual;
 *                   w_grad[H] += sum over t of dY * h * rstd (fp32, in place, fixed order); w_grad NULL
 *                   (with any workspace) leaves it out
 * dX is the gradient of x and of the residual alike; dresidual (bf16, may be NULL) is the gradient that reaches
 * h by other ways, and may be dX itself.  Sums and means are fp32.  H % 8 == 0 and H <= 16384 (SL_ESHAPE); eps >= 0 and finite
 * (SL_EINVAL); w_grad and rstd 4-byte aligned.  The gradient takes a workspace of its query's bytes, as above.
 * --------------------------------------------------------------------------------------------- */
int sl_rmsnorm_fwd(void* stream, const void* x, const void* residual, const void* w, float eps, void* y, void* h,
                   float* rstd, int64_t T, int64_t H);
int sl_rmsnorm_fwd_mxfp8(void* stream, const void* x, const void* residual, const void* w, float eps,
                         uint8_t* q_rows, uint8_t* s_rows, uint8_t* q_cols, uint8_t* s_cols, void* h,
                         float* rstd, int64_t T, int64_t H);
size_t sl_rmsnorm_bwd_workspace_bytes(int64_t T, int64_t H);
int sl_rmsnorm_bwd(void* stream, const void* dY, const void* h, const void* w, const float* rstd,
                   const void* dresidual, void* dX, float* w_grad, int64_t T, int64_t H, void* workspace,
                   size_t workspace_bytes);

/* ---- Orthogonalised updates ---------------------------------------------------------------------
 * L matrices [rows, cols] of one shape, any extents (not bound to multiples of 8).  With U a matrix as
 * [m, n], m <= n (a tall one is transposed on the way in and out):
 *   X = U / |U|_F (zeros stay zeros);   `steps` times:  A = X.X^T,  X <- a X + (b A + c A.A).X
 * coeffs is a host array of a, b, c for each step.  Products run in fp16 at one fixed scale with fp32 sums; the
 * host checks that the coefficients keep singular values that start in [0, 1] below 3, a I + b A + c A.A
 * below 15 and c A.X below 60 (SL_EINVAL otherwise), which keeps every element in fp16's range.  A gradient with an infinity or a NaN gives
 * NaN.
 *
 * sl_orthogonalize: O[L, rows, cols] (bf16) = X for U = G[L, rows, cols] (fp32 or bf16: g_bytes 4 or 2).
 * sl_muon_step: one optimiser step of L weights.  W, G, M and master are host arrays of L device pointers, read
 * during the call: bf16 weights, fp32 gradients (main_grad views), fp32 momenta, and fp32 master weights (master NULL:
 * none).  A matrix of W, M or master overlaps no other of the call's.
 *   M <- momentum * M + G;   U = nesterov ? G + momentum * M : M
 *   W <- (1 - lr * weight_decay) * W - lr * scale * X   (of the master where there is one, which is then rounded to W)
 * lr, momentum, weight_decay and scale must be finite, steps 0 .. 64 (SL_EINVAL); L <= 65535 and a padded matrix under
 * 2 GiB in fp16 (SL_ESHAPE).  Matrices are 16-byte aligned, or as slices of a 16-byte aligned
 * batch are: to their elements' bytes where cols % 4 != 0, bf16 ones of odd rows to 8 bytes where cols % 8 == 4.  Both take a workspace of the query's bytes, as above.
 * sl_orthogonalize_tiles (host only, for measurement and tests): how the three products of a step, X.X^T, A.A and P.X, are
 * taken apart, tiles[12] = for each the number of 256x256 tiles, of 128x128 tiles, of the latter with split sums, and of
 * their parts (1: none are split); zeros where the steps go to the kernels for few rows.
 * --------------------------------------------------------------------------------------------- */
size_t sl_orthogonalize_workspace_bytes(int64_t L, int64_t rows, int64_t cols);
int sl_orthogonalize_tiles(int64_t L, int64_t rows, int64_t cols, int64_t* tiles);
int sl_orthogonalize(void* stream, const void* G, int32_t g_bytes, void* O, int64_t L, int64_t rows, int64_t cols,
                     int32_t steps, const float* coeffs, void* workspace, size_t workspace_bytes);
int sl_muon_step(void* stream, void* const* W, float* const* master, const float* const* G, float* const* M,
                 int64_t L, int64_t rows, int64_t cols, float lr, float momentum, int32_t nesterov,
                 float weight_decay, float scale, int32_t steps, const float* coeffs, void* workspace,
                 size_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* SHARDED_LINEAR_H */
