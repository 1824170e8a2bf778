/*
 * fp8q.h -- C ABI of libfp8q.so: the FP8 (OCP E4M3) quantize-and-consume path on
 * AMD MI355X (gfx950).
 *
 * Conventions for every call
 *   - Device buffers are plain device pointers owned by the caller; the library never
 *     keeps them past the call (the calibrator keeps only its own staging copies).
 *   - bf16 data is passed as its 16-bit pattern (uint16_t), E4M3 codes as uint8_t, scales
 *     as IEEE binary32.  E4M3 is the OCP "FN" encoding: bias 7, no infinities,
 *     S.1111.111 = NaN, largest finite 448.  Encoding is round-to-nearest-even after one
 *     IEEE binary32 division by the scale, saturating to +-448 (never NaN); the sign is
 *     kept, so a negative value that rounds to zero is 0x80.
 *   - Work is enqueued on `stream` (0 = the null stream) and returns without waiting.
 *     No call allocates or synchronizes, except the calibrator as documented.
 *   - Arguments are validated on the host before anything is enqueued; a bad argument
 *     returns a negative FP8Q_E* code and enqueues nothing.  0 means success.  No C++
 *     exception crosses this boundary.
 *
 * Sources (the pages this path comes from, cited by page title and the item on it):
 *   [actq]    spark_model/layers/ops/fp8_act_quant.rs
 *   [decode]  spark_model/layers/ops/dispatch_proj_decode.rs
 *   [staging] spark_model/layers/fp8_calibration/staging.rs
 *   [calib]   metrale_model_layers/layers/fp8_calibration.rs
 *   [resid]   fp8_residency.rs (weight loader page), fp8_twin_bytes
 */
#ifndef FP8Q_H
#define FP8Q_H

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------------- status codes */
#define FP8Q_OK 0
#define FP8Q_EINVAL (-1) /* a size, stride or scale outside the contract */
#define FP8Q_ENULL (-2)  /* a required pointer is NULL */
#define FP8Q_EALIGN (-3) /* a pointer or stride breaks the documented alignment */
#define FP8Q_ELAUNCH (-4) /* the kernel launch was rejected by the HIP runtime */
#define FP8Q_EHIP (-5)   /* another HIP runtime call failed (alloc, copy, sync) */
#define FP8Q_ESTATE (-6) /* calibrator used against its contract (e.g. new device) */

/* Human-readable text for a status code (static storage). */
const char* fp8q_strerror(int status);
/* Library version, major*10000 + minor*100 + patch. */
int fp8q_version(void);
/* Measurement hook: the next kernel this host thread enqueues through the library records
 * `start` as it begins executing and `stop` as it completes (hipExtLaunchKernelGGL), so
 * the events' elapsed time is that kernel's own duration.  Either may be NULL.  Every
 * entry point below enqueues exactly one kernel per call, except calls that enqueue
 * nothing (zero sizes, errors), the calibrator, attn_prefill, fp8_attn_decode and
 * fp8_attn_chunk (whose first kernel is the timed one).  Always returns FP8Q_OK. */
int fp8q_time_next_launch(hipEvent_t start, hipEvent_t stop);

/* Measurement references (not steps of the path): kernels that the path's timings are read
 * against, launched through the same hook.  fp8q_reference_empty enqueues one empty
 * 256-thread block (what a launch costs before any work).  fp8q_reference_stream reads
 * src_bytes (a multiple of 16) from src (non-temporal 16-byte loads) and writes
 * src_bytes / 2 to dst -- the 2:1 read/write mix of the group quantizer and the KV write,
 * with no arithmetic -- over a grid of 4 blocks per CU.  src 16-byte and dst 8-byte aligned device memory.
 * fp8q_reference_lds_stream moves total_bytes from src into LDS the way the prefill GEMM
 * moves its operand tiles (16-byte buffer_load ... lds, 64 KB slices, one 512-thread
 * workgroup per CU, one slice landing while the next is issued, a barrier per slice) and
 * nothing else; slice s reads src bytes [(s * 65536) % span_bytes, + 65536).  span_bytes
 * and total_bytes are multiples of 65536, 65536 <= span_bytes <= 0x7FFF0000; src holds
 * span_bytes of device memory, 16-byte aligned.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int fp8q_reference_empty(hipStream_t stream);
int fp8q_reference_stream(const void* src, void* dst, int64_t src_bytes, hipStream_t stream);
int fp8q_reference_lds_stream(const void* src, int64_t span_bytes, int64_t total_bytes,
                              hipStream_t stream);

/* ------------------------------------------------ per-token 1x128 group quant
 * [actq] module doc: one FP32 scale per 128-wide K-group of one token row;
 * [decode] decode_w8a8_quant_act: the activation is quantized once and shared by every
 * projection that reads it, scales in token-major [m, k/128] order.
 *
 * For every row r < m and group g < k/128:
 *   amax = max_j |x[r, 128g + j]|            (exact)
 *   s    = max(amax, 1e-10f) / 448.0f        (binary32, correctly rounded)
 *   scales[r * (k/128) + g] = s
 *   q[r, 128g + j] = E4M3(x[r, 128g + j] / s)
 *
 *   x       device, bf16 [m, k] row-major, 16-byte aligned
 *   q       device, uint8 [m, k] row-major, 16-byte aligned
 *   scales  device, fp32 [m, k/128] row-major, 4-byte aligned
 *   m       rows, 0 <= m (0 is a no-op); m * k < 2^62
 *   k       columns, k > 0 and k % 128 == 0 (the pages' grid is k/128 groups)
 * Errors: FP8Q_EINVAL (k, m), FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int fp8_group_quant(const uint16_t* x, uint8_t* q, float* scales, int64_t m, int32_t k,
                    hipStream_t stream);

/* ------------------- RMS norm with the residual's addition, to 1x128 groups
 * The step before a projection ([decode] decode_w8a8_quant_act quantizes a normed activation), in
 * one pass.  For every row r < m, in binary32:
 *   h[j] = bf16_rne(x[r, j] + residual[r, j])   (residual NULL: x[r, j]); residual_out[r, j] = h[j]
 *   y[j] = h[j] * weight[j] / sqrt(mean_j(h[j]^2) + eps)
 *   per group of 128: scale and codes of y as fp8_group_quant makes them; norm_out[r, j] =
 *   bf16_rne(y[j])
 * y is not rounded to bf16 before it is quantized: codes and scales are those of the binary32 row,
 * not of norm_out.  Rows are read once (twice beyond 32768 columns).
 *   x, residual, residual_out, norm_out   device bf16 rows at their strides (elements, multiples of
 *           8, at most 2^40), 16-byte aligned; residual_out goes with residual and may be it or x;
 *           norm_out (for the W8A16 tier) may be NULL
 *   weight  device bf16 [k], 16-byte aligned, or NULL (ones)
 *   q       device uint8 [m, k], 16-byte aligned;  scales  device fp32 [m, k/128]
 *   k > 0 and k % 128 == 0; m >= 0 (0 is a no-op), m * (k/128) < 2^31; 0 <= eps <= 1
 * The squares' sum must stay within binary32.  A NaN makes its row NaN codes; so does a row of
 * zeros with eps = 0.  An infinity (of h: also a sum that rounds to one) makes its own value NaN
 * and the others of its row 0.  Other outputs must not overlap inputs.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int fp8_rms_norm_group_quant(const uint16_t* x, const uint16_t* residual, const uint16_t* weight,
                             float eps, uint16_t* residual_out, uint16_t* norm_out, uint8_t* q,
                             float* scales, int64_t m, int32_t k, int64_t x_stride,
                             int64_t residual_stride, int64_t residual_out_stride,
                             int64_t norm_out_stride, hipStream_t stream);

/* --------------------------------- SiLU of the gate times up, to 1x128 groups
 * The step between the gate and up projections and the down projection, in one pass.  For every
 * row r < m, in binary32:
 *   y[j] = gate[r, j] / (1 + exp(-gate[r, j])) * up[r, j]
 *   per group of 128: scale and codes of y as fp8_group_quant makes them; out[r, j] =
 *   bf16_rne(y[j]).  y is not rounded to bf16 before it is quantized.
 *   gate, up, out   device bf16 rows at their strides (elements, multiples of 8, at most 2^40;
 *           gate and up may be column halves of one buffer), 16-byte aligned; out may be NULL
 *   q       device uint8 [m, k], 16-byte aligned;  scales  device fp32 [m, k/128]
 *   k > 0 and k % 128 == 0; m >= 0 (0 is a no-op), m * (k/128) < 2^31
 * The products must stay within binary32; y is off by (2 |gate| + 8) 2^-24 of itself, and may be 0
 * where the gate's factor 1 / (1 + exp(-gate)) is below 2^-125.  Outputs must not overlap inputs.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int fp8_silu_mul_group_quant(const uint16_t* gate, const uint16_t* up, uint16_t* out, uint8_t* q,
                             float* scales, int64_t m, int32_t k, int64_t gate_stride,
                             int64_t up_stride, int64_t out_stride, hipStream_t stream);

/* ---------------------------------------------- 128x128 weight block quant
 * [decode] module doc, NUMERICS: E4M3 weights carry one FP32 scale per 128x128 block;
 * [resid] fp8_twin_bytes: the grid has ceil(n/128) * ceil(k/128) fp32 entries.
 * The same formula as fp8_group_quant over each 128x128 block (edge blocks clipped):
 *   ws[nb * ceil(k/128) + kb] = max(amax_block, 1e-10f) / 448.0f
 *   wq[i, j] = E4M3(w[i, j] / ws[i/128, j/128])
 *   w   device, bf16 [n, k] row-major; wq device, uint8 [n, k]; ws device, fp32 grid
 *   n, k > 0.  A preparation utility (weights arrive pre-quantized on the pages).
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_ELAUNCH. */
int fp8_block_quant(const uint16_t* w, uint8_t* wq, float* ws, int32_t n, int32_t k,
                    hipStream_t stream);

/* -------------------------------------------- element-wise binary32 -> E4M3
 * The encoder every kernel above uses, exposed on its own: q[i] = E4M3(x[i]) for finite
 * x, round-to-nearest-even, saturating to +-448 (no scale).
 *   x device fp32 [n], q device uint8 [n], n >= 0.  Errors: FP8Q_EINVAL, FP8Q_ENULL,
 *   FP8Q_ELAUNCH. */
int fp8_e4m3_encode(const float* x, uint8_t* q, int64_t n, hipStream_t stream);

/* ----------------------------------------------- block-scaled W8A8 decode GEMM
 * [decode] decode_w8a8_gemm and module doc NUMERICS: out = act_fp8 @ weight^T with the
 * per-token 1x128 activation scales and the 128x128 weight block scales folded in an
 * FP32 epilogue; DecodeW8a8Plan / decode_w8a8_selected: n % 128 == 0, k % 128 == 0,
 * ldc >= n; DECODE_W8A8_ROWS: the decode band is up to 16 rows; strided_out_extent_elems:
 * a call touches (rows - 1) * ldc + n elements of `out`.
 *
 *   out[r, c] = bf16_rne( sum_g a_scale[r, g] * w_scale[c/128, g]
 *                                * sum_{j<128} dec(a_q[r, 128g+j]) * dec(w_q[c, 128g+j]) )
 * with FP32 products and accumulation.  Only rows 0..m-1 are written: exactly the
 * (m - 1) * ldc + n elements starting at `out`, columns n..ldc-1 of each row untouched.
 *
 *   a_q      device, uint8 [m, k] row-major (E4M3 codes), 16-byte aligned
 *   a_scale  device, fp32 [m, k/128] token-major (fp8_group_quant's own order)
 *   w_q      device, uint8 [n, k] row-major (K contiguous), 16-byte aligned
 *   w_scale  device, fp32 [n/128, k/128]; block (nb, kb) at nb * (k/128) + kb
 *   out      device, bf16 [m, ldc] row-major, 2-byte aligned
 *   1 <= m <= 16; n > 0, n % 128 == 0; k > 0, k % 128 == 0, k <= 131072; ldc >= n.
 * Codes 0x7F/0xFF (NaN) in a_q or w_q propagate NaN into the affected outputs.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int w8a8_block_gemm(const uint8_t* a_q, const float* a_scale, const uint8_t* w_q,
                    const float* w_scale, uint16_t* out, int32_t m, int32_t n, int32_t k,
                    int32_t ldc, hipStream_t stream);

/* ------------------------------------ block-scaled W8A8 decode GEMM, K split
 * [decode] module doc, WHY table: a decode projection is a stream over its weight, and the
 * pages' own library splits K (a split-K pass plus a reduce) when an output alone cannot
 * keep the machine busy.  Computes exactly what w8a8_block_gemm specifies (same operands,
 * layouts, rows written and errors), but when the shape has too few 16-column output
 * strips to give every CU a full share, K is split over `parts` sets of workgroups: each
 * writes its part's FP32 16x16 tile sums to the workspace, and the workgroup that completes
 * a strip adds the parts in a fixed order (p = 0, 1, ...), so the result is deterministic
 * (it may differ from w8a8_block_gemm's in the last bits: another FP32 summation order).
 * Shapes that do not benefit run w8a8_block_gemm's kernel and touch no workspace; K a
 * multiple of 1024 never splits (w8a8_block_gemm's staged form is faster there).
 *
 * w8a8_block_gemm_workspace_size: *bytes = the workspace this shape needs on the current
 *   device (0: no split).  Errors: FP8Q_ENULL, FP8Q_EINVAL (shape as w8a8_block_gemm).
 * w8a8_block_gemm_ws:
 *   workspace        device memory of workspace_bytes >= the size above, 256-byte aligned,
 *                    owned by the caller; its counts (the first ceil(n/16 * 4 / 256) * 256
 *                    bytes) must be zero before the first call that uses it (e.g. zero-filled
 *                    at allocation); every call leaves them zero again, so later calls need
 *                    no clearing.  Calls sharing a workspace must not overlap in time (calls
 *                    on one stream never do).  NULL / 0 is fine when the size is 0.
 * Errors: as w8a8_block_gemm, and FP8Q_ENULL (no workspace where one is needed),
 * FP8Q_EINVAL (workspace_bytes too small), FP8Q_EALIGN (workspace not 256-byte aligned). */
int w8a8_block_gemm_workspace_size(int32_t m, int32_t n, int32_t k, uint64_t* bytes);
int w8a8_block_gemm_ws(const uint8_t* a_q, const float* a_scale, const uint8_t* w_q,
                       const float* w_scale, uint16_t* out, int32_t m, int32_t n, int32_t k,
                       int32_t ldc, void* workspace, uint64_t workspace_bytes,
                       hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph capture, serving
 * loops that forbid allocation): w8a8_block_gemm_ws without the workspace argument.  Same
 * arguments as w8a8_block_gemm and exactly w8a8_block_gemm_ws's result (the same split and
 * summation order), with the split's counts and part tiles in a static device array of
 * 4 KiB + 1 MiB that the library holds on every GPU it runs on until the process ends.
 * Allocates nothing.  The first call on a device looks the array's address up and enqueues
 * a fill that zeroes its counts on `stream`; every call leaves them zero.  All calls on one
 * GPU share the array: calls that overlap in time on one GPU (e.g. on two streams) race;
 * calls on one stream never overlap.  A shape whose split needs more than the array (more
 * than 1024 strips, or strips x parts above 1024) is refused with FP8Q_EINVAL before
 * anything is enqueued; shapes that run unsplit use no scratch.
 * Errors: as w8a8_block_gemm, and FP8Q_EHIP (the array's address could not be looked up). */
int w8a8_block_gemm_noalloc(const uint8_t* a_q, const float* a_scale, const uint8_t* w_q,
                            const float* w_scale, uint16_t* out, int32_t m, int32_t n,
                            int32_t k, int32_t ldc, hipStream_t stream);

/* ------------------------------------------------ W8A8 GEMM at prefill widths
 * [resid] DenseFp8Inputs::w8a8_kernels (the W8A8 prefill arm: per-token group quant, then
 * a block-scaled FP8 GEMM); [actq] module doc (a 4593-token prefill).  The arithmetic and
 * operand layouts are w8a8_block_gemm's; only the row range differs: any m >= 1.  Tiled
 * 256 x 256 (one workgroup per CU) once there are at least half as many such tiles as CUs,
 * else 128 x 128 (two per CU); both tilings give bit-identical results.
 *   out[r, c] = bf16_rne( sum_g a_scale[r, g] * w_scale[c/128, g]
 *                                * sum_{j<128} dec(a_q[r, 128g+j]) * dec(w_q[c, 128g+j]) )
 * FP32 products and accumulation, one scaled FMA per group.  Only rows 0..m-1 are written
 * ((m - 1) * ldc + n elements).
 *   a_q, a_scale, w_q, w_scale, out  as w8a8_block_gemm
 *   m >= 1; n % 128 == 0; k % 128 == 0, 128 * k < 2^31; ldc >= n (16-byte row stores when
 *   ldc % 8 == 0 and out is 16-byte aligned, element stores otherwise).
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int w8a8_block_gemm_prefill(const uint8_t* a_q, const float* a_scale, const uint8_t* w_q,
                            const float* w_scale, uint16_t* out, int32_t m, int32_t n,
                            int32_t k, int32_t ldc, hipStream_t stream);

/* ---------------------------------------------- grouped W8A8 decode GEMM
 * [decode] decode_w8a8_quant_act: several projections that read the same activation
 * (attention Q/K/V, a layer's projections) share one quantization; DecodeW8a8Plan::strided:
 * outputs may be written at their own row pitch.  One launch computes, for each
 * projection p < count, exactly what w8a8_block_gemm(a_q, a_scale, projs[p].w_q,
 * projs[p].w_scale, projs[p].out, m, projs[p].n, k, projs[p].ldc) computes (same
 * arithmetic, same bits).  `projs` is host memory read during the call; 1 <= count <= 8;
 * every projection obeys w8a8_block_gemm's rules.  Errors as w8a8_block_gemm. */
typedef struct fp8q_gemm_proj {
  const uint8_t* w_q;    /* device, uint8 [n, k] */
  const float* w_scale;  /* device, fp32 [n/128, k/128] */
  uint16_t* out;         /* device, bf16 [m, ldc] */
  int32_t n;
  int32_t ldc;
} fp8q_gemm_proj;

int w8a8_block_gemm_grouped(const uint8_t* a_q, const float* a_scale,
                            const fp8q_gemm_proj* projs, int32_t count, int32_t m, int32_t k,
                            hipStream_t stream);

/* ------------------------------------- group quant fused into the grouped GEMM
 * [actq] module doc and [decode] decode_w8a8_quant_act + decode_w8a8_gemm, in one launch:
 * the activation is quantized per 1x128 group (exactly fp8_group_quant's arithmetic, so
 * the codes and scales are bit-identical to it) inside the GEMM, each wave quantizing the
 * K-slice it multiplies, then every projection is computed as w8a8_block_gemm_grouped
 * would from those codes (same bits).
 *   a        device, bf16 [m, k] row-major, 16-byte aligned
 *   a_q, a_scale  optional outputs (both NULL or both set): the codes [m, k] and scales
 *            [m, k/128] as fp8_group_quant writes them (16- / 4-byte aligned); required
 *            when k > 8192, where the quantizer and the GEMM run as two launches through
 *            them (FP8Q_ENULL if missing)
 *   projs, count  as w8a8_block_gemm_grouped;  1 <= m <= 16;  k % 128 == 0, k <= 131072
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int fp8_quant_w8a8_gemm_grouped(const uint16_t* a, uint8_t* a_q, float* a_scale,
                                const fp8q_gemm_proj* projs, int32_t count, int32_t m,
                                int32_t k, hipStream_t stream);

/* --------------------------------------------- W8A16 decode tier (1..4 rows)
 * [decode] module doc NUMERICS (the W8A16 arithmetic: bf16 activation times E4M3 weight
 * with the same 128x128 FP32 block scales) and DECODE_W8A8_ROWS (up to four rows stay on
 * this tier).  The activation is not quantized:
 *   out[r, c] = bf16_rne( sum_g w_scale[c/128, g] * sum_{j<128} a[r, 128g+j] * dec(w_q[c, 128g+j]) )
 * with exact products and FP32 accumulation (the group's partial, then times its scale).
 * A row's result does not depend on m (the same row gives the same bits at m = 1..4).
 * Only rows 0..m-1 are written ((m - 1) * ldc + n elements).
 *   a        device, bf16 [m, k] row-major, 16-byte aligned
 *   w_q, w_scale, out, n, ldc  as w8a8_block_gemm
 *   1 <= m <= 4; n % 128 == 0; k > 0, k % 128 == 0, k <= 131072; ldc >= n.
 *   (k <= 8192 runs a persistent kernel that keeps the activation in registers; longer k
 *   a per-strip kernel that reads it from L2.  Both sum in a fixed order per k.)
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int w8a16_block_gemv(const uint16_t* a, const uint8_t* w_q, const float* w_scale,
                     uint16_t* out, int32_t m, int32_t n, int32_t k, int32_t ldc,
                     hipStream_t stream);

/* Several projections of one bf16 activation in one launch (as w8a8_block_gemm_grouped):
 * each projs[p] gets exactly what w8a16_block_gemv computes for it. 1 <= count <= 8. */
int w8a16_block_gemv_grouped(const uint16_t* a, const fp8q_gemm_proj* projs, int32_t count,
                             int32_t m, int32_t k, hipStream_t stream);

/* --------------------------------------------------------- paged FP8 KV write
 * [staging] Fp8KvWriteTarget and replay_and_release (the write's arguments: strides in
 * elements, pool stride = block_size * heads * head_dim); [staging] module doc: one scale
 * per tensor, later writes of a slot replace earlier ones.
 *
 * For each token t < num_tokens with 0 <= slot < num_blocks * block_size (slot =
 * slot_mapping[t]; other slots are skipped -- negative ones are padding):
 *   b = slot / block_size, o = slot % block_size, for all h < H, d < D:
 *   k_cache[b * cache_stride + (o * H + h) * D + d] = E4M3(k[t * key_stride + h*D + d] / k_scale)
 *   v_cache[... same index ...]                       = E4M3(v[t * value_stride + h*D + d] / v_scale)
 * Slots must be distinct within one call (two tokens on one slot race).
 *
 *   k, v            device bf16 rows of key_stride / value_stride elements
 *   k_cache,v_cache device uint8 pools of num_blocks * cache_stride bytes each
 *   slot_mapping    device int64 [num_tokens]
 *   num_tokens >= 0 (0 is a no-op); num_kv_heads, head_dim, block_size, num_blocks > 0;
 *   key_stride, value_stride >= H*D; cache_stride >= block_size*H*D;
 *   k_scale, v_scale in [2^-64, 2^64] (dequantization multipliers).
 * The vector path needs 16-byte aligned k/v/pools and H*D, strides, cache_stride all
 * multiples of 8; anything else takes an element-wise path with the same results.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_ELAUNCH. */
int fp8_kv_write(const uint16_t* k, const uint16_t* v, uint8_t* k_cache, uint8_t* v_cache,
                 const int64_t* slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                 int32_t head_dim, int32_t block_size, int64_t num_blocks, float k_scale,
                 float v_scale, int32_t key_stride, int32_t value_stride,
                 int64_t cache_stride, hipStream_t stream);

/* [calib] Fp8KvCalibration::observe + [staging] module doc, in one pass: inside the
 * calibration window every batch is both measured (absmax) and written (at the provisional
 * scale).  Exactly fp8_kv_write(...) followed by fp8_kv_amax over the same batch's rows:
 *   amax2[0] = max(amax2[0], max |k[t * key_stride + i]|), amax2[1] likewise for v, over
 *   every t < num_tokens and i < H*D (padding tokens included: the batch's data, as the
 *   pages' absmax), with the pools written as fp8_kv_write writes them.
 * One kernel when H*D is a multiple of 16 up to 512 and the rows are 16-byte aligned; else
 * the absmax pass and the write run back to back.  amax2: device fp32[2], 4-byte aligned.
 * Errors as fp8_kv_write, and FP8Q_ENULL for a NULL amax2. */
int fp8_kv_write_amax(const uint16_t* k, const uint16_t* v, uint8_t* k_cache,
                      uint8_t* v_cache, const int64_t* slot_mapping, int32_t num_tokens,
                      int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                      int64_t num_blocks, float k_scale, float v_scale, int32_t key_stride,
                      int32_t value_stride, int64_t cache_stride, float* amax2,
                      hipStream_t stream);

/* ------------------------------------------------------ paged FP8 KV read (dequant)
 * [staging] module doc: every token of a sequence's history is read back at the one
 * per-tensor scale the layer holds (which is why early tokens written at the provisional
 * scale must be rewritten at the frozen one); the write above defines the pool layout.
 *
 * For each token t < num_tokens with 0 <= slot < num_blocks * block_size (slot =
 * slot_mapping[t]; output rows of other tokens are left untouched):
 *   b = slot / block_size, o = slot % block_size, for all h < H, d < D:
 *   k_out[t * out_key_stride + h*D + d] =
 *       bf16_rne(fp32(E4M3 value of k_cache[b * cache_stride + (o * H + h) * D + d]) * k_scale)
 *   v_out[... same ...] likewise with v_cache and v_scale
 * The product is one binary32 multiplication (round to nearest even), then rounded to
 * bf16 to nearest even; the NaN codes 0x7F / 0xFF read as the quiet NaN 0x7FC0.
 *
 *   k_cache, v_cache   device uint8 pools of num_blocks * cache_stride bytes each
 *   slot_mapping       device int64 [num_tokens]
 *   k_out, v_out       device bf16 rows of out_key_stride / out_value_stride elements
 *   num_tokens >= 0 (0 is a no-op); num_kv_heads, head_dim, block_size, num_blocks > 0;
 *   out strides >= H*D; cache_stride >= block_size*H*D; scales in [2^-64, 2^64].
 * The vector path needs H*D, the output strides and cache_stride multiples of 8, 8-byte
 * aligned pools and 16-byte aligned outputs; anything else takes an element-wise path
 * with the same results.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int fp8_kv_read(const uint8_t* k_cache, const uint8_t* v_cache, const int64_t* slot_mapping,
                int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                int64_t num_blocks, float k_scale, float v_scale, uint16_t* k_out,
                uint16_t* v_out, int32_t out_key_stride, int32_t out_value_stride,
                int64_t cache_stride, hipStream_t stream);

/* ------------------------------------------------------------- KV absolute max
 * [calib] Fp8KvCalibration::absmax: max |K| and max |V| of a batch, max-accumulated into
 * a device float[2] that the caller zeroes once (so a window's running max can stay on
 * the device).
 *   amax2[0] = max(amax2[0], max_i |k[i]|), amax2[1] = max(amax2[1], max_i |v[i]|)
 *   k, v device bf16 [n_elems] packed; amax2 device fp32[2], 4-byte aligned, >= +0.0
 *   n_elems >= 0.  Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_ELAUNCH. */
int fp8_kv_amax(const uint16_t* k, const uint16_t* v, int64_t n_elems, float* amax2,
                hipStream_t stream);

/* -------------------------------- head norms, rotary positions and the paged write
 * The step between the QKV projection and attention.  For every token t < num_tokens with
 * 0 <= positions[t] < num_positions (other tokens are padding: nothing of theirs is written)
 * and every query and key head row x of D = head_dim values, in binary32:
 *   n[i] = x[i] * w[i] / sqrt(mean(x^2) + eps)   (w: q_weight / k_weight; NULL: n = x)
 *   pairs (a, b) = (i, i + R/2), or (2i, 2i + 1) when interleaved, i < R/2, R = rot_dim, with
 *   c = cos_sin[positions[t]][i], s = cos_sin[positions[t]][R/2 + i]:
 *     y[a] = n[a] * c - n[b] * s,  y[b] = n[b] * c + n[a] * s;   y[i] = n[i] for i >= R
 *   q_out / k_out = bf16_rne(y)
 * fp8_qk_norm_rope_kv_write also writes the caches as fp8_kv_write(k_out, v, ...) would (the
 * same bytes: the codes are made of the rounded bf16 keys, so that a calibration window's replay
 * of staged rows leaves what the live write leaves); a token whose slot is outside the pool gets
 * its q_out (and k_out) and no cache write.  Where tokens of one call share a slot, each of its
 * bytes is one of theirs, of which is not defined.
 *   q, k, v        device bf16 rows of H*D values at q_stride / key_stride / value_stride
 *                  (views of one projection's output are fine)
 *   q_weight, k_weight  device bf16 [D] or NULL;  0 <= eps <= 1
 *   positions      device int64 [num_tokens];  cos_sin  device fp32 [num_positions, rot_dim]:
 *                  the cosines, then the sines of each position (any base, any scaling for long
 *                  contexts).  Both may be NULL when rot_dim is 0.
 *   q_out, k_out   device bf16 rows at their strides; each may be its input (same address and
 *                  stride), other overlaps are not allowed; k_out may be NULL in the writing form
 *   0 <= num_tokens; heads > 0; 0 < head_dim <= 65536; 0 <= rot_dim <= head_dim, even;
 *   strides >= H*D, at most 2^30; the cache arguments as fp8_kv_write.
 * The vector path needs head_dim in {32, 64, 128, 256, 512}, rot_dim % 16 == 0 (% 8 interleaved),
 * strides % 8 == 0 and 16-byte aligned rows, weights and table (pools 8-byte aligned,
 * cache_stride % 8 == 0); anything else takes an element-wise path with the same formula.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int qk_norm_rope(const uint16_t* q, const uint16_t* k, const uint16_t* q_weight,
                 const uint16_t* k_weight, float eps, const int64_t* positions,
                 const float* cos_sin, int64_t num_positions, int32_t rot_dim,
                 int32_t interleaved, int32_t num_tokens, int32_t num_q_heads,
                 int32_t num_kv_heads, int32_t head_dim, int64_t q_stride, int64_t key_stride,
                 uint16_t* q_out, uint16_t* k_out, int64_t q_out_stride, int64_t k_out_stride,
                 hipStream_t stream);
int fp8_qk_norm_rope_kv_write(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                              const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                              const int64_t* positions, const float* cos_sin,
                              int64_t num_positions, int32_t rot_dim, int32_t interleaved,
                              uint8_t* k_cache, uint8_t* v_cache, const int64_t* slot_mapping,
                              int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t block_size, int64_t num_blocks,
                              float k_scale, float v_scale, int64_t q_stride,
                              int64_t key_stride, int64_t value_stride, int64_t cache_stride,
                              uint16_t* q_out, uint16_t* k_out, int64_t q_out_stride,
                              int64_t k_out_stride, hipStream_t stream);

/* ------------------------------------------------ attention over whole prompts
 * Packed sequences: sequence s has the query rows cu_seqlens_q[s] .. cu_seqlens_q[s + 1] - 1
 * and the key / value rows cu_seqlens_k[s] .. cu_seqlens_k[s + 1] - 1 (Lq and Lk of them; Lk > Lq
 * for a chunk of a prompt behind its history).  Query head h reads KV head h / (Hq / Hkv).
 * Query i sees the keys j < Lk, with `causal` those with j <= i + Lk - Lq (the last query sees
 * every key):
 *   s[i][j] = softmax_scale * q[i] . k[j]
 *   out[i]  = bf16_rne( sum_j exp(s[i][j]) v[j] / sum_j exp(s[i][j]) )
 *   lse[i]  = log sum_j exp(s[i][j])
 * A query that sees no key gets zeros and lse = -infinity.  What a query does not see does not
 * reach it, infinities and NaN included.  An infinity or a NaN in a value row reaches the outputs of
 * all queries that see it, however small its weight (infinities of both signs: NaN).  FP32 products,
 * sums and statistics; out's weights are rounded to bf16, in its numerator and its denominator alike.
 *   q, k, v   device bf16 rows at q_stride / key_stride / value_stride elements, 16-byte aligned
 *   out       device bf16 rows at out_stride; rows outside every sequence are left untouched
 *   lse       device fp32 [total_q, num_q_heads], or NULL
 *   cu_seqlens_q, cu_seqlens_k  device int32 [num_seqs + 1], ascending from 0 to at most total_q /
 *             total_k (the rows of q and of k); entries are clamped to that range
 *   head_dim in {64, 128, 256}; num_q_heads a multiple of num_kv_heads; strides multiples of 8,
 *   at most 2^23; num_seqs <= 65536; total_q, total_k <= 2^30; 0 < softmax_scale <= 2^64.
 *   workspace   device memory of workspace_bytes >= attn_prefill_workspace_size's, 256-byte
 *               aligned, of any content (nothing is kept in it from call to call); calls that
 *               share one must not overlap in time; NULL is fine where the size is 0.  At most
 *               256 MiB: a few binary32 rows for each query row and head
 * Few queries over long keys are split along the keys: then two kernels are enqueued, the second
 * joining the parts in order, and a workspace is needed (results do not depend on the order in
 * which workgroups run).  attn_prefill_workspace_size: for the current device.
 * The scores, and 2^8 times a row's sum of |v|, must stay within binary32.  Outputs must not
 * overlap inputs.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int attn_prefill_workspace_size(int32_t num_seqs, int32_t total_q, int32_t total_k,
                                int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                uint64_t* bytes);
int attn_prefill(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                 const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, uint16_t* out,
                 float* lse, int32_t num_seqs, int32_t total_q, int32_t total_k,
                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                 float softmax_scale, int32_t causal, int64_t q_stride, int64_t key_stride,
                 int64_t value_stride, int64_t out_stride, void* workspace,
                 uint64_t workspace_bytes, hipStream_t stream);

/* ------------------------------- single-token attention over the paged E4M3 cache
 * [staging] module doc: paged attention reads a sequence's whole history at the one scale the
 * layer holds; fp8_kv_write defines the pool layout.  Sequence s has one query token and
 * len = context_lens[s] cached positions (its own token's among them, written before the call);
 * position p lies in block block_tables[s * table_stride + p / block_size] at offset
 * p % block_size.  With K, V the E4M3 values there, of KV head h / (Hq / Hkv):
 *   s[p] = softmax_scale * k_scale * q[s][h] . K[p]
 *   out[s][h] = bf16_rne( v_scale * sum_p exp(s[p]) V[p] / sum_p exp(s[p]) )
 *   lse[s][h] = log sum_p exp(s[p])
 * len is clamped to [0, max_blocks * block_size]; positions in a block outside [0, num_blocks)
 * do not count; a sequence without positions gets zeros and lse = -infinity.  FP32 products,
 * sums and statistics; out's weights are rounded to bf16, in its numerator and its denominator
 * alike.  What lies in the pools behind a sequence's end does not reach it, NaN codes included.
 * Results do not depend on the order in which workgroups run.
 *   q, out      device bf16 rows at q_stride / out_stride elements, 16-byte aligned
 *   k_cache, v_cache  device uint8 pools of num_blocks * cache_stride bytes, 16-byte aligned
 *   block_tables      device int32 [num_seqs, table_stride], the first max_blocks of each row used
 *   context_lens      device int32 [num_seqs];  lse  device fp32 [num_seqs, num_q_heads] or NULL
 *   workspace   device memory of workspace_bytes >= fp8_attn_decode_workspace_size's, 256-byte
 *               aligned, of any content (nothing is kept in it from call to call); calls that
 *               share one must not overlap in time
 *   head_dim in {64, 128, 256}; num_q_heads a multiple of num_kv_heads; block_size > 0;
 *   num_seqs <= 65536; max_blocks * block_size <= 2^30 and num_seqs * (max_blocks * block_size / 32 + 1) <= 2^30;
 *   cache_stride >= block_size*H*D, a multiple of 16; q / out
 *   strides multiples of 8; k_scale, v_scale in [2^-64, 2^64]; 0 < softmax_scale <= 2^32.
 * The scores must stay within binary32.  Outputs must not overlap inputs.
 * Enqueues two kernels where max_blocks * block_size > 1024, whatever the lengths (the second joins
 * the parts of histories that were cut), else one: a table no wider than the longest history needs
 * is the faster one for short histories.
 * fp8_attn_decode_workspace_size: for the current device.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int fp8_attn_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                   int32_t head_dim, uint64_t* bytes);
int fp8_attn_decode(const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                    const int32_t* block_tables, const int32_t* context_lens, uint16_t* out,
                    float* lse, int32_t num_seqs, int32_t max_blocks, int64_t table_stride,
                    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                    int32_t block_size, int64_t num_blocks, float k_scale, float v_scale,
                    float softmax_scale, int64_t q_stride, int64_t out_stride,
                    int64_t cache_stride, void* workspace, uint64_t workspace_bytes,
                    hipStream_t stream);

/* ------------------------- attention of chunks of new tokens over the paged E4M3 cache
 * [staging] module doc, as for fp8_attn_decode, for any number of new tokens a sequence: a chunk
 * of a prompt, drafted tokens to verify, single steps, all in one batch.  Sequence s has the query
 * rows cu_seqlens_q[s] .. cu_seqlens_q[s + 1] - 1 (Lq of them) and len = context_lens[s] cached
 * positions, the new tokens' own among them as the last ones, written before the call; position p
 * lies where fp8_attn_decode's does.  Query i sees the positions p < len, with `causal` those with
 * p <= i + len - Lq (the last query sees every position).  With K, V the E4M3 values of KV head
 * h / (Hq / Hkv):
 *   s[i][p] = softmax_scale * k_scale * q[i][h] . K[p]
 *   out[i][h] = bf16_rne( v_scale * sum_p exp(s[i][p]) V[p] / sum_p exp(s[i][p]) )
 *   lse[i][h] = log sum_p exp(s[i][p])
 * len is clamped to [0, max_blocks * block_size]; positions in a block outside [0, num_blocks)
 * do not count; a query that sees no position gets zeros and lse = -infinity.  FP32 products, sums
 * and statistics; out's weights are rounded to bf16, in its numerator and its denominator alike.
 * What a query does not see does not reach it, NaN codes included; a NaN code of a value reaches
 * that output of every query that sees it, however small its weight.  Results do not depend on the
 * order in which workgroups run.
 *   q, out      device bf16 rows at q_stride / out_stride elements, 16-byte aligned; rows of out
 *               outside every sequence are left untouched
 *   k_cache, v_cache  device uint8 pools of num_blocks * cache_stride bytes, 16-byte aligned
 *   block_tables      device int32 [num_seqs, table_stride], the first max_blocks of each row used
 *   context_lens      device int32 [num_seqs]
 *   cu_seqlens_q      device int32 [num_seqs + 1], ascending from 0 to at most total_q (q's rows);
 *                     entries are clamped to that range
 *   lse         device fp32 [total_q, num_q_heads] or NULL
 *   workspace   device memory of workspace_bytes >= fp8_attn_chunk_workspace_size's, 256-byte
 *               aligned, of any content (nothing is kept in it from call to call); calls that
 *               share one must not overlap in time; NULL is fine where the size is 0
 *   head_dim in {64, 128, 256}; num_q_heads a multiple of num_kv_heads; total_q * num_q_heads <=
 *   2^30; block_size > 0; num_seqs <= 65536; max_blocks * block_size <= 2^30; cache_stride >=
 *   block_size*H*D, a multiple of 16, below 2^32; q / out strides multiples of 8, up to 2^30;
 *   k_scale, v_scale in [2^-64, 2^64]; 0 < softmax_scale <= 2^32.
 * The scores must stay within binary32.  Outputs must not overlap inputs.
 * Where the batch is too small to fill the GPU by its queries alone, histories are cut into parts:
 * then a workspace is needed and two kernels are enqueued, the second joining the parts in order
 * (batches of more than 256 sequences are never cut, nor those whose tables have room for at most
 * 256 positions, though the workspace is checked: a table no wider than needed is the faster one for
 * short histories).  In a batch that is not cut the call takes as long as one workgroup needs for the
 * longest history (3.3 ms for 100000 positions of 128-wide heads): where one is far longer than the
 * others, and the batch is of more than 256 sequences or holds thousands of new tokens, give that
 * sequence a call of its own, single steps to fp8_attn_decode.
 * Every workgroup reads all lengths: the time grows with the square of the number of sequences from
 * some thousands on (8192 steps of 1 to 64 positions: 1.7 ms).
 * fp8_attn_chunk_workspace_size: for the current device.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EALIGN, FP8Q_ELAUNCH. */
int fp8_attn_chunk_workspace_size(int32_t num_seqs, int32_t total_q, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t head_dim, uint64_t* bytes);
int fp8_attn_chunk(const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                   const int32_t* block_tables, const int32_t* context_lens,
                   const int32_t* cu_seqlens_q, uint16_t* out, float* lse, int32_t num_seqs,
                   int32_t total_q, int32_t max_blocks, int64_t table_stride,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                   int32_t block_size, int64_t num_blocks, float k_scale, float v_scale,
                   float softmax_scale, int32_t causal, int64_t q_stride, int64_t out_stride,
                   int64_t cache_stride, void* workspace, uint64_t workspace_bytes,
                   hipStream_t stream);

/* ----------------------------------------------- online KV scale calibrator
 * [calib] module doc, PROVISIONAL_SCALE, Fp8KvCalibration::{new, observe, scales};
 * [staging] module doc ("The fix, and its tradeoff"), KvStaging::{stage,
 * replay_and_release, release}, MAX_STAGED_TOKENS.
 *
 * One attention layer's per-tensor K/V scale calibration.  Inside the window each
 * observed batch's |K|/|V| maximum folds into a running maximum kept on the device, and
 * the batch (bf16 rows + slots) is copied into packed staging; the caller then writes
 * it at the provisional scale.  The observe whose token count reaches the window freezes
 * scale = (max(amax, 1e-10) * headroom) / 448 for K and V over every observed token
 * including its own batch, replays the staged batches at the frozen scales into the
 * target pools (one write of every staged token whose slot no later staged token writes,
 * which leaves the bytes an in-order replay leaves), and releases the staging in stream
 * order; the caller then writes that batch at the frozen scales.  Later observes do
 * nothing.  A batch whose heads x head_dim differ from the first staged batch, or that
 * would overflow the window's staging, is not staged (it keeps the provisional scale).
 * The window is clamped to 4096 tokens and headroom to >= 1.
 * Call order per batch: fp8q_kv_calib_observe, then fp8q_kv_calib_scales, then the
 * caller's fp8_kv_write of that batch, all on one stream.  Not capturable in a HIP graph
 * (the freeze reads the running maximum back to the host). */
typedef struct fp8q_kv_calib fp8q_kv_calib;

/* Where the replay writes (the live write's own pools and geometry). */
typedef struct fp8q_kv_target {
  uint8_t* k_pool;
  uint8_t* v_pool;
  const int64_t* slot_mapping; /* this batch's slots, int64 [num_tokens] */
  int32_t block_size;
  int32_t key_stride;          /* row stride of the observed K, elements */
  int32_t value_stride;        /* row stride of the observed V, elements */
  int32_t reserved;
  int64_t cache_stride;        /* elements per block = block_size * H * D or more */
  int64_t num_blocks;          /* blocks in each pool */
} fp8q_kv_target;

typedef struct fp8q_kv_calib_info {
  int32_t window_tokens;    /* after the 4096 clamp */
  int32_t requested_tokens; /* as passed to create */
  int32_t frozen;
  int32_t staged_batches;
  int64_t tokens_seen;
  int64_t staged_tokens;
  int64_t unstaged_tokens;  /* tokens of declined batches */
  int64_t replayed_tokens;  /* tokens rewritten at the freeze */
  float k_scale;            /* provisional until frozen */
  float v_scale;
  float k_amax;             /* running maxima read at the freeze (0 before) */
  float v_amax;
  float headroom;           /* after the >= 1 clamp */
  float provisional_scale;
} fp8q_kv_calib_info;

/* What observe would do with a batch, without doing it. */
#define FP8Q_CALIB_STAGE 0
#define FP8Q_CALIB_DECLINE 1
#define FP8Q_CALIB_FREEZE 2
#define FP8Q_CALIB_FROZEN 3

/* The device work of a calibrator, as a table of callbacks ([staging] and [calib] take a
 * GPU backend object for the same purpose).  The calibrator's bookkeeping (window, stage,
 * decline, freeze formula and range check, replay order, counters) only calls these; it
 * never touches device memory itself, so a table backed by host memory runs the whole
 * state machine on a CPU.  fp8q_kv_calib_create uses the library's own HIP table.
 * Every callback returns FP8Q_OK or a negative FP8Q_E* status, which observe returns.
 *   device      the current device (observe refuses a device other than the first one)
 *   alloc       *out = `bytes` of device memory, usable by work enqueued on `stream` after
 *               this call (HIP: hipMallocAsync)
 *   release     free what alloc returned: in stream order after the work enqueued on
 *               `stream` when at_destroy == 0; when at_destroy != 0 (from
 *               fp8q_kv_calib_destroy, stream unused) only once all device work is done
 *   zero        bytes of p = 0, stream-ordered
 *   amax_rows   amax2[0] = max(amax2[0], max|k|), amax2[1] likewise for v, over `rows` rows of
 *               `elems` bf16 at key/value strides (elements), stream-ordered
 *   copy2d      `rows` rows of row_bytes bytes from src (rows src_pitch bytes apart) to dst,
 *               packed, stream-ordered
 *   read        bytes from device src to host dst once the work enqueued on `stream` is done
 *               (blocks the caller)
 *   replay      write n staged packed rows (`elems` bf16 each, K and V) to the target's pools
 *               at (k_scale, v_scale) as fp8_kv_write would write them one after another in
 *               staging order (a slot staged twice keeps its later row); scratch_slots is
 *               int64 [n] of device scratch the callback may use; stream-ordered
 *   stage       optional (NULL: amax_rows, then copy2d of the K rows, V rows and slots): the
 *               same in one call -- amax_rows over the batch, its rows copied packed to
 *               dst_k / dst_v (row t at t * elems) and its `rows` slots to dst_slots */
typedef struct fp8q_kv_calib_ops {
  void* ctx;
  int (*device)(void* ctx, int32_t* dev);
  int (*alloc)(void* ctx, uint64_t bytes, void** out, hipStream_t stream);
  int (*release)(void* ctx, void* p, hipStream_t stream, int32_t at_destroy);
  int (*zero)(void* ctx, void* p, uint64_t bytes, hipStream_t stream);
  int (*amax_rows)(void* ctx, const uint16_t* k, const uint16_t* v, int64_t rows,
                   int64_t elems, int64_t key_stride, int64_t value_stride, float* amax2,
                   hipStream_t stream);
  int (*copy2d)(void* ctx, void* dst, const void* src, int64_t src_pitch, int64_t row_bytes,
                int64_t rows, hipStream_t stream);
  int (*read)(void* ctx, void* host_dst, const void* src, uint64_t bytes, hipStream_t stream);
  int (*replay)(void* ctx, const uint16_t* k, const uint16_t* v, const int64_t* slots,
                int64_t* scratch_slots, int32_t n, int32_t elems, const fp8q_kv_target* target,
                float k_scale, float v_scale, hipStream_t stream);
  int (*stage)(void* ctx, const uint16_t* k, const uint16_t* v, const int64_t* slots,
               int64_t rows, int64_t elems, int64_t key_stride, int64_t value_stride,
               uint16_t* dst_k, uint16_t* dst_v, int64_t* dst_slots, float* amax2,
               hipStream_t stream);
} fp8q_kv_calib_ops;

/* window_tokens > 0 (window 0 means no calibrator: FP8Q_EINVAL); headroom finite and
 * <= 2^64 (values below 1 are raised to 1); provisional_scale in [2^-64, 2^64] (the
 * pages use 2.0).  Allocates host state only; device buffers are allocated on the first
 * observe, on the device current then.  *out receives the handle.
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EHIP (host allocation). */
int fp8q_kv_calib_create(int32_t window_tokens, float headroom, float provisional_scale,
                         fp8q_kv_calib** out);
/* As fp8q_kv_calib_create, with the device work going through `ops` (copied; every
 * callback but stage must be set; the table's ctx must outlive the calibrator). */
int fp8q_kv_calib_create_with_ops(int32_t window_tokens, float headroom,
                                  float provisional_scale, const fp8q_kv_calib_ops* ops,
                                  fp8q_kv_calib** out);
/* Fold one batch in (see above).  k, v: device bf16 [num_tokens] rows at the target's
 * key/value strides.  Enqueues work on `stream`; blocks only at the freeze, to read the
 * 8-byte running maximum back (through 64 bytes of page-locked host memory that the first
 * freeze of the process allocates and every later one reuses; concurrent freezes take
 * turns).  The first staged batch allocates the staging in one piece
 * (window * H * D * 2 * 2 + window * 16 bytes, stream-ordered); the freeze releases it in
 * stream order.  With the library's HIP table an in-window observe is one kernel (absmax
 * and staging copy in one pass).
 * A frozen scale outside [2^-64, 2^64] (the write's scale range) fails the freezing
 * observe with FP8Q_EINVAL and leaves the calibrator as it was (the batch's absmax may
 * already be folded into the running maximum; folding the same batch again changes
 * nothing).
 * Errors: FP8Q_EINVAL, FP8Q_ENULL, FP8Q_EHIP, FP8Q_ELAUNCH, FP8Q_ESTATE. */
int fp8q_kv_calib_observe(fp8q_kv_calib* c, const uint16_t* k, const uint16_t* v,
                          int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                          const fp8q_kv_target* target, hipStream_t stream);
/* Pure query: FP8Q_CALIB_* for a batch of num_tokens x elems_per_token, or < 0. */
int fp8q_kv_calib_decide(const fp8q_kv_calib* c, int32_t num_tokens,
                         int32_t elems_per_token);
/* The scales the caller writes with now (provisional until the freeze). */
int fp8q_kv_calib_scales(const fp8q_kv_calib* c, float* k_scale, float* v_scale);
/* Snapshot of the calibrator's counters, scales and running maxima. */
int fp8q_kv_calib_state(const fp8q_kv_calib* c, fp8q_kv_calib_info* info);
/* Frees staging and device state (after all device work is done). NULL ok. */
void fp8q_kv_calib_destroy(fp8q_kv_calib* c);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_H */
