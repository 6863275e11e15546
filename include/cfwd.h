/*
 * cfwd.h -- forward 2-D convolution for CNN inference on one AMD Instinct
 * MI355X (gfx950).  Plain C ABI: no C++ types, no exceptions, no torch types.
 *
 * What is computed (every entry point that writes y):
 *   The forward convolution of CNN inference as the naive loop nest of the
 *   blog post "卷积总结" (convolution summary), section "最原始的卷积实现",
 *   defines it -- a cross-correlation, output[k, oh, ow] = sum over c, r, s of
 *   w[k, c, r, s] * x[c, oh*stride + r*dil - pad, ow*stride + s*dil - pad],
 *   with a batch loop, symmetric zero padding, stride, dilation and groups
 *   (output channel k reads input channels of group k / (K/G) only), and
 *   OH = floor((H + 2*pad_h - dil_h*(R-1) - 1) / stride_h) + 1 (OW likewise).
 *
 * Algorithms (MegEngine inference article, sections "Im2col+MatMul",
 * "Winograd" and "Fast-Run"; Momenta talk "Paper Reading | 讓深度學習更高效運行
 * 的兩個視角", section "優化2：Depthwise卷積" for the depthwise / 1x1 layers):
 *   IMPLICIT_GEMM   im2col x matmul without materialising im2col: input patches
 *                   are staged in LDS and multiplied on the matrix cores.  Its
 *                   last config(s) are the NHWC kernel, the only ones that take
 *                   NHWC problems (and they take nothing else): both operands
 *                   are staged by plain 16-byte copies, the channels of a
 *                   pixel being contiguous.
 *   WINOGRAD_F2X2_3X3 / WINOGRAD_F6X6_3X3
 *                   F(m x m, 3 x 3) minimal filtering for 3x3, stride 1,
 *                   dilation 1, groups 1; float dtypes, and int8 for
 *                   F(2x2) config 0 (below).  bf16 runs its
 *                   transformed operands in fp16 (11 significant bits); to
 *                   keep them in fp16's range, input and filter are scaled by
 *                   powers of two that bring each one's largest magnitude
 *                   (found on the device: the input's on every call, the
 *                   filter's when it is prepared) into [2^7, 2^8), and the
 *                   output is scaled back -- exactly, so any finite
 *                   magnitudes work.  Values below 2^-22 of their tensor's
 *                   largest magnitude become fp16 subnormals and lose
 *                   precision; the Fast-Run accuracy gate sees that on the
 *                   caller's data.
 *                   int8 F(2x2) (MegEngine Beta release article, section
 *                   "业界领先的原生 ARM 推理性能": int8 Winograd with float as
 *                   the intermediate format, no narrowing of the weights):
 *                   B^T d B (multiples of 1/4, |.| <= 512) and G g G^T
 *                   (integers, |.| <= 1152) are fp16 operands, exactly; the
 *                   channel sums and the output transform are fp32, then
 *                   rounded to the nearest integer and requantised as below.
 *                   Exact while every fp32 partial sum stays below 2^22 in
 *                   magnitude; beyond that an output can be 1 away from the
 *                   exact one.  Runs when named explicitly; a Fast-Run
 *                   candidate only after cfwd_fastrun_allow_inexact_int8(1).
 *   DIRECT          direct summation; the depthwise (G = C = K) path.
 *   POINTWISE       1x1 convolution as a low-K matrix product.
 *   AUTO            resolved per problem: a Fast-Run map entry if one exists,
 *                   else (or a search with CFWD_FASTRUN_MODE=search) a fixed
 *                   preference: depthwise -> DIRECT, 1x1 -> POINTWISE, else
 *                   IMPLICIT_GEMM.  Winograd is never chosen without timing.
 *
 * Tensors (all device memory, owned by the caller, 16-byte aligned, dense):
 *   x  activations  NCHW  [N][C][H][W]
 *                   NCHWX [N][ceil(C/x)][H][W][x], x = 4 or 8 (MegEngine
 *                   inference article, section "NCHWX"); channels past C are
 *                   ignored on input.
 *                   NHWC  [N][H][W][C] (channels contiguous; fp32 / bf16, groups
 *                   1, C a multiple of 4 (fp32) or 8 (bf16); runs on the NHWC
 *                   implicit GEMM configs, see IMPLICIT_GEMM).
 *   w  weights      KCRS  [K][C/G][R][S] in every layout, activation dtype.
 *   y  output       same layout and dtype as x, with K channels; in NCHWX the
 *                   channels past K are written as 0.
 *   requant_scale   int8 only: fp32 [K] on the device; the int32 accumulator
 *                   becomes int8 as clamp(rne(fp32(acc) * scale[k]), -127, 127)
 *                   (round to nearest even, symmetric clamp, zero point 0).
 * Dtypes: fp32 (fp32 accumulate), bf16 (fp32 accumulate, output rounded to
 * nearest even), int8 (int32 accumulate, requantised output).
 *
 * Streams: `stream` is a hipStream_t passed as void* (NULL = the default
 * stream).  Calls that only enqueue work return without waiting.
 *
 * Environment (read once per process):
 *   CFWD_FASTRUN_MODE  readonly (default): AUTO takes the Fast-Run map entry,
 *                      else the fixed preference; off: AUTO ignores the map;
 *                      search: a map miss of cfwd_conv2d_fwd with a workspace
 *                      of cfwd_fastrun_workspace_size bytes runs the selection.
 *   CFWD_FASTRUN_CACHE a map file merged into the map before the first AUTO
 *                      resolution; in search mode rewritten after each
 *                      selection.
 *   CFWD_LOG           0 silent (default); 1 every failure's reason on stderr;
 *                      2 also each AUTO resolution and how it was made; 3 also
 *                      the algorithm of every convolution call.
 *
 * Errors: every call returns a cfwd_status; on failure nothing has been
 * enqueued and cfwd_last_error() (per thread) describes why.  Validation
 * failures never touch y.  No call allocates device memory.
 */
#ifndef CFWD_H
#define CFWD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CFWD_OK = 0,
    CFWD_ERR_INVALID_ARG = 1,  /* bad descriptor, NULL or misaligned pointer */
    CFWD_ERR_UNSUPPORTED = 2,  /* valid problem this algorithm cannot run   */
    CFWD_ERR_WORKSPACE = 3,    /* workspace / prepared buffer too small      */
    CFWD_ERR_NO_CANDIDATE = 4, /* Fast-Run found no candidate passing its gate */
    CFWD_ERR_HIP = 5,          /* a HIP runtime call failed (message kept)   */
    CFWD_ERR_CACHE_IO = 6      /* Fast-Run map file could not be written    */
} cfwd_status;

typedef enum { CFWD_LAYOUT_NCHW = 0, CFWD_LAYOUT_NCHWX = 1, CFWD_LAYOUT_NHWC = 2 } cfwd_layout;

/* MXFP4: only where the section on 4-bit floating point names it. */
typedef enum { CFWD_F32 = 0, CFWD_BF16 = 1, CFWD_I8 = 2, CFWD_MXFP4 = 3 } cfwd_dtype;

typedef enum {
    CFWD_ALGO_AUTO = 0,
    CFWD_ALGO_IMPLICIT_GEMM = 1,
    CFWD_ALGO_WINOGRAD_F2X2_3X3 = 2,
    CFWD_ALGO_WINOGRAD_F6X6_3X3 = 3,
    CFWD_ALGO_DIRECT = 4,
    CFWD_ALGO_POINTWISE = 5
} cfwd_algo_kind;

/* One convolution problem.  pad_* >= 0; every other integer >= 1;
 * C and K divisible by groups; x is 4 or 8 when layout is NCHWX (ignored for
 * NCHW).  Each of x and y must hold fewer than 2^31 elements per image. */
typedef struct {
    int n, c, h, w, k, r, s;
    int stride_h, stride_w, pad_h, pad_w, dil_h, dil_w, groups;
    cfwd_layout layout;
    int x;
    cfwd_dtype dtype;
} cfwd_conv_desc;

/* An algorithm choice: family, tile configuration within the family
 * (-1 = the family's default for the problem), and the median time Fast-Run
 * measured for it in milliseconds (0 when not measured). */
typedef struct {
    cfwd_algo_kind kind;
    int config_id;
    float median_ms;
} cfwd_algo;

/* Activation of the fused epilogue.  Convolutions take NONE and RELU; the
 * MXFP4 product also v / (1 + e^-v) and 0.5 v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))). */
typedef enum { CFWD_ACT_NONE = 0, CFWD_ACT_RELU = 1, CFWD_ACT_SILU = 2, CFWD_ACT_GELU = 3 } cfwd_activation;

/* Fused epilogue of cfwd_conv2d_fwd_ex: what a ResNet block applies after
 * its convolution, folded into the convolution's own output pass (Momenta
 * talk "Paper Reading | 讓深度學習更高效運行的兩個視角", section "Graph層面":
 * conv, bias and ReLU computed as one operation, the output written once).
 *   bias      device [K]: fp32 for fp32 / bf16 problems, int32 for int8;
 *             NULL = none.  4-byte aligned.
 *   residual  device tensor of y's shape, layout and dtype (the skip
 *             connection); NULL = none.  16-byte aligned, must not overlap y.
 *   act       CFWD_ACT_NONE or CFWD_ACT_RELU.
 * fp32 / bf16: y = act(conv + bias[k] + residual), in fp32, then one
 *   conversion to the output dtype (bf16: round to nearest even).
 * int8: y = clamp(rne(fp32(acc + bias[k]) * scale[k] + fp32(residual)), lo, 127)
 *   with the bias added to the int32 accumulator (acc + bias must stay in
 *   int32), one fp32 multiply, one fp32 add, ties to even, lo = 0 under ReLU
 *   and -127 otherwise (the residual is taken to be in y's quantised scale). */
typedef struct {
    const void *bias;
    const void *residual;
    cfwd_activation act;
} cfwd_epilogue;

/* Library version string, e.g. "cfwd 0.1.0 gfx950". */
const char *cfwd_version(void);

/* OH, OW of the problem (the floor formula above).  INVALID_ARG if the
 * descriptor is invalid or the window does not fit. */
cfwd_status cfwd_output_dims(const cfwd_conv_desc *desc, int *oh, int *ow);

/* Resolve `algo` (AUTO, or a family with config_id -1) to the concrete
 * (kind, config_id) conv2d_fwd would run.  UNSUPPORTED if the family cannot
 * run this problem. */
cfwd_status cfwd_resolve_algo(const cfwd_conv_desc *desc, cfwd_algo algo, cfwd_algo *resolved);

/* Every (kind, config_id) that can run the problem, in Fast-Run's fixed
 * candidate order (IMPLICIT_GEMM < POINTWISE < DIRECT < WINOGRAD_F2 <
 * WINOGRAD_F6, then config id).  Writes at most `cap` entries to out (out may
 * be NULL when cap is 0) and the total count to *count. */
cfwd_status cfwd_list_candidates(const cfwd_conv_desc *desc, cfwd_algo *out, int cap, int *count);

/* Bytes of the prepared (re-laid-out or transformed) filter the algorithm
 * reads; 0 means it reads the KCRS weights directly. */
cfwd_status cfwd_filter_size(const cfwd_conv_desc *desc, cfwd_algo algo, size_t *bytes);

/* Build the prepared filter of `algo` from KCRS weights into w_prepared
 * (`bytes` >= cfwd_filter_size).  Enqueued on `stream`.  Winograd: the
 * G g G^T filter transform (MegEngine inference article, section "Winograd",
 * step one); implicit GEMM: the weight tile order its matrix-core loop reads
 * (the pack step the article's "融合 PACK" section folds away on the
 * activation side). */
cfwd_status cfwd_prepare_filter(const cfwd_conv_desc *desc, cfwd_algo algo, const void *w_kcrs,
                                void *w_prepared, size_t bytes, void *stream);

/* Workspace bytes conv2d_fwd needs for `algo` when it is given no prepared
 * filter: the prepared filter (built into the workspace first), rounded up to
 * 256 bytes, plus the algorithm's scratch.  0 when none. */
cfwd_status cfwd_workspace_size(const cfwd_conv_desc *desc, cfwd_algo algo, size_t *bytes);

/* Workspace bytes conv2d_fwd needs for `algo` when it is given a prepared
 * filter: the algorithm's scratch only (Winograd: the transformed input
 * tiles B^T d B, alpha^2 x ceil(C / chunk) x tiles x 64 bytes, and for bf16
 * 8 KiB for the input's largest magnitude; implicit GEMM split
 * reductions: their int32 partial tiles).  0 when none. */
cfwd_status cfwd_scratch_size(const cfwd_conv_desc *desc, cfwd_algo algo, size_t *bytes);

/* y = conv(x, w).  w_kcrs is required.  w_prepared may be NULL; when it is
 * not, it must hold cfwd_prepare_filter's output for the same descriptor and
 * resolved algorithm, and the filter is not re-prepared.  requant_scale is
 * required for int8 and must be NULL otherwise.  Enqueued on `stream`. */
cfwd_status cfwd_conv2d_fwd(const cfwd_conv_desc *desc, cfwd_algo algo, const void *x,
                            const void *w_kcrs, const void *w_prepared,
                            const float *requant_scale, void *y, void *workspace,
                            size_t ws_bytes, void *stream);

/* cfwd_conv2d_fwd with a fused epilogue (see cfwd_epilogue; NULL = none,
 * which is exactly cfwd_conv2d_fwd).  Every algorithm and config applies it
 * in its own output pass, so AUTO dispatch from the Fast-Run map works
 * unchanged (the map is chosen on the convolution alone; a
 * CFWD_FASTRUN_MODE=search miss with an epilogue falls back to the fixed
 * preference instead of searching).  INVALID_ARG for an unknown activation,
 * a misaligned bias or residual, or a residual overlapping y. */
cfwd_status cfwd_conv2d_fwd_ex(const cfwd_conv_desc *desc, cfwd_algo algo, const void *x,
                               const void *w_kcrs, const void *w_prepared,
                               const float *requant_scale, const cfwd_epilogue *epilogue, void *y,
                               void *workspace, size_t ws_bytes, void *stream);

/* Scratch capacity of cfwd_conv2d_fwd_noalloc, per device (64 MiB). */
#define CFWD_NOALLOC_SCRATCH_BYTES (64u << 20)

/* Allocation-free variant of cfwd_conv2d_fwd, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  Same arguments and result as
 * cfwd_conv2d_fwd without the workspace: what that call takes from the
 * workspace (the prepared filter when w_prepared is NULL, plus the
 * algorithm's scratch -- split-reduction partial tiles, Winograd transformed
 * input) lives instead in a library-owned device array of
 * CFWD_NOALLOC_SCRATCH_BYTES, one per device, held until the process ends.
 * Returns CFWD_ERR_WORKSPACE, enqueuing nothing, when the resolved algorithm
 * needs more than that (cfwd_scratch_size / cfwd_workspace_size tell in
 * advance).  AUTO resolves from the Fast-Run map or the fixed preference,
 * never by a search.  Every call on one device shares that device's array:
 * calls that overlap on one GPU (other streams, other host threads) race on
 * it; calls in one stream are ordered.  No kernel needs the array zeroed --
 * each overwrites what it reads -- so the previous call's contents are
 * harmless.  Allocates nothing, frees nothing. */
cfwd_status cfwd_conv2d_fwd_noalloc(const cfwd_conv_desc *desc, cfwd_algo algo, const void *x,
                                    const void *w_kcrs, const void *w_prepared,
                                    const float *requant_scale, void *y, void *stream);

/* Fast-Run selection phase (MegEngine inference article, section "Fast-Run"):
 * time every candidate of cfwd_list_candidates on this device with these
 * buffers (median of 7 runs after 2 warm-ups; before each run the Infinity
 * Cache and L2 are flushed by overwriting a 512 MiB region of the workspace
 * unless x and y together already exceed that, so candidates are timed from
 * HBM), reject any whose output fails the accuracy gate against the generic
 * DIRECT kernel's result on the same data (for NHWC, run on x converted to
 * NCHW and converted back; bit-identical for int8, except
 * int8 Winograd F(2x2): no output more than 1 away;
 * normalised error <= 1e-5 fp32 except Winograd F(6x6), 1e-3 fp32 F(6x6),
 * 1e-2 bf16; NaN or infinity fails), keep the fastest (times within 1% count
 * as equal and the earlier candidate wins), record it in the map and return
 * it in *best.  Synchronises `stream`; overwrites y.  workspace must hold
 * cfwd_fastrun_workspace_size bytes. */
cfwd_status cfwd_fastrun_select(const cfwd_conv_desc *desc, const void *x, const void *w_kcrs,
                                const float *requant_scale, void *y, void *workspace,
                                size_t ws_bytes, void *stream, cfwd_algo *best);

/* Workspace for cfwd_fastrun_select: the largest candidate workspace, the
 * reference output and error normaliser, and the cache-flush region. */
cfwd_status cfwd_fastrun_workspace_size(const cfwd_conv_desc *desc, size_t *bytes);

/* Fast-Run execution-phase map (host memory, process-wide, thread-safe).
 * lookup: CFWD_OK and *algo when the problem has an entry on this device,
 * UNSUPPORTED otherwise.  load: merge a map file (one record per line); a
 * missing, corrupt or other-device file is ignored with CFWD_OK.
 * save: write the whole map (CACHE_IO on failure).  clear: empty it. */
cfwd_status cfwd_fastrun_lookup(const cfwd_conv_desc *desc, cfwd_algo *algo);
cfwd_status cfwd_fastrun_load(const char *path);
cfwd_status cfwd_fastrun_save(const char *path);
cfwd_status cfwd_fastrun_clear(void);

/* Copy an activation tensor of n x c x h x w elements of `dtype` from one
 * layout to another (NCHW, NHWC, NCHWX with x = src_x / dst_x = 4 or 8; the
 * x arguments are ignored for the others).  NCHWX destinations get their
 * channels past c written as 0; NCHWX sources' are not read.  For networks
 * whose layers prefer different layouts (MegEngine CPU-inference article,
 * section "结论": a network-wide mixed choice of layouts).  src and dst
 * (device, element-aligned) must not overlap.  Enqueued on `stream`. */
cfwd_status cfwd_convert_layout(int n, int c, int h, int w, cfwd_dtype dtype, cfwd_layout src_layout,
                                int src_x, const void *src, cfwd_layout dst_layout, int dst_x, void *dst,
                                void *stream);

/* 4-bit weights (MegEngine CPU-inference article, section "结论": lower-bit
 * quantisation after int8).  gfx950's matrix cores have no int4 operands, so
 * 4-bit weights are stored packed and widened once, when loaded, to the int8
 * KCRS tensor every int8 call takes; results are then the int8 path's, bit
 * for bit.  out_int8[i] = signed value i of `packed`: byte i / 2, low nibble
 * for even i, high nibble for odd i, two's complement (-8 .. 7).  packed
 * holds (count + 1) / 2 bytes and must be 16-byte aligned, out_int8 count
 * bytes, 16-byte aligned, not overlapping packed.  Enqueued on `stream`. */
cfwd_status cfwd_unpack_int4(const void *packed, void *out_int8, long long count, void *stream);

/* Whether int8 candidates whose results are not always bit-identical to the
 * integer ones (int8 Winograd F(2x2), see WINOGRAD_F2X2_3X3 above) take part
 * in cfwd_list_candidates and cfwd_fastrun_select: 0 (the default) = no,
 * nonzero = yes.  Process-wide; an algorithm named explicitly runs either
 * way, and a Fast-Run map entry chosen while they were allowed stays in use. */
cfwd_status cfwd_fastrun_allow_inexact_int8(int allow);

/* The host-side part of Fast-Run's choice, for callers that time candidates
 * themselves (and for testing the rule without a GPU): cands[n] in Fast-Run
 * order, times[n * reps] row-major in ms, gate_ok[n] nonzero when the
 * candidate passed the accuracy gate.  *chosen = index of the candidate with
 * the smallest median time, where a later candidate wins only if its median is
 * more than 1% below the current best's; -1 if none passed. */
cfwd_status cfwd_fastrun_choose(const cfwd_algo *cands, const float *times, int n, int reps,
                                const int *gate_ok, int *chosen);

/* ---- Fused bottleneck block.
 * The ResNet bottleneck (Momenta talk "Paper Reading | 讓深度學習更高效運行的兩個
 * 視角", section "優化1：Bottleneck") as one operation, with the spatial tiling
 * of its section "Operator的粒度": each workgroup computes a band of output
 * rows and keeps the two 64-channel intermediates on chip, so x is read and y
 * written once, with no intermediate tensor in memory.
 *   t1 = act1(conv1x1(x, w1) + b1)            C -> mid
 *   t2 = act2(conv3x3(t1, w2, pad 1) + b2)    mid -> mid
 *   y  = act3(conv1x1(t2, w3) + b3 + residual) mid -> K
 * all stride 1, cross-correlation as above, act = ReLU where asked.
 * t1 and t2 are rounded to bf16 (what three separate bf16 layers store);
 * each stage accumulates in fp32 and applies its epilogue in fp32 before its
 * single rounding.  Supported: bf16, NCHW, mid = 64, C and K multiples of
 * 32, W a multiple of 8 and at most 64, any N and H. */
typedef struct {
    int n, c, h, w; /* x: [N][C][H][W] */
    int mid;        /* channels of the two inner convolutions */
    int k;          /* channels of y: [N][K][H][W] */
    cfwd_dtype dtype;
} cfwd_bottleneck_desc;

/* Per-stage epilogue: fp32 biases b1 [mid], b2 [mid], b3 [K] (NULL = none,
 * 4-byte aligned); residual: bf16 of y's shape added before act3 (NULL =
 * none, 16-byte aligned, must not overlap y); relu1..3 nonzero = ReLU. */
typedef struct {
    const void *b1, *b2, *b3;
    const void *residual;
    int relu1, relu2, relu3;
} cfwd_bottleneck_epilogue;

/* CFWD_OK when the fused kernel runs this block, UNSUPPORTED (reason in
 * cfwd_last_error) when not, INVALID_ARG for a NULL descriptor. */
cfwd_status cfwd_bottleneck_check(const cfwd_bottleneck_desc *desc);

/* Bytes of the prepared 3x3 weights (9 x mid x mid bf16, tap-major). */
cfwd_status cfwd_bottleneck_filter_size(const cfwd_bottleneck_desc *desc, size_t *bytes);

/* Prepare w2 (KCRS [mid][mid][3][3], bf16, device) into w2_prepared
 * (>= cfwd_bottleneck_filter_size bytes, 16-byte aligned).  Enqueued on
 * `stream`. */
cfwd_status cfwd_bottleneck_prepare(const cfwd_bottleneck_desc *desc, const void *w2, void *w2_prepared,
                                    size_t bytes, void *stream);

/* y = the block of x.  w1 KCRS [mid][C][1][1], w3 KCRS [K][mid][1][1] (bf16,
 * device, as given), w2_prepared from cfwd_bottleneck_prepare; epilogue may
 * be NULL (no bias, no residual, no ReLU).  x, w1, w2_prepared, w3, y
 * 16-byte aligned; y must not overlap x or the residual.  Allocates
 * nothing; enqueued on `stream`. */
cfwd_status cfwd_bottleneck_fwd(const cfwd_bottleneck_desc *desc, const void *x, const void *w1,
                                const void *w2_prepared, const void *w3,
                                const cfwd_bottleneck_epilogue *epilogue, void *y, void *stream);

/* ---- Microscaled 4-bit floating point (MXFP4) and the feed-forward block.
 * For the parts of a network that are products over channels: 1x1
 * convolutions of NHWC activations, fully connected layers, the feed-forward
 * halves of transformer layers.  gfx950's matrix cores take MXFP4 operands.
 *
 * Format: 32 consecutive values of a row ("block") share a scale.
 *   codes   uint8 [rows][16 * KB], KB = ceil(k / 32): two values a byte, the
 *           even one in the low four bits; bit 3 of a value is its sign, bits
 *           0..2 name 0, 0.5, 1, 1.5, 2, 3, 4, 6 (E2M1).  Values past k are 0.
 *   scales  uint8 [rows][KB rounded up to a multiple of 4]: 2^(byte - 127),
 *           255 = NaN; the bytes past KB are written as 127 and do not count when read.
 * Quantisation of a block: with E the biased fp32 exponent of its largest
 * magnitude, byte = max(E - 2, 0), or 255 if the block holds a NaN or an
 * infinity (its codes are then 0); each value / scale is rounded to the
 * nearest E2M1 value, a tie to the even code, saturating at 6, sign kept.
 *
 * codes must be 16-byte aligned, scales 4-byte; x and y in fp32 / bf16
 * need only their element's alignment, bias and weights 4 bytes.  rows (m)
 * may be 0: nothing is done; rows <= 2^38, rows times x_stride <= 2^60,
 * 1 <= k <= 2^22, 1 <= n <= 2^22.  Every call is enqueued on `stream`,
 * allocates nothing and gives the same bits each time. */

/* Bytes of the codes and of the scales of `rows` rows of k values. */
cfwd_status cfwd_mx_size(long long rows, int k, size_t *code_bytes, size_t *scale_bytes);

/* x [rows][k] (fp32 / bf16, row pitch x_stride >= k elements) -> codes, scales. */
cfwd_status cfwd_mx_quantize(long long rows, int k, cfwd_dtype dtype, const void *x, long long x_stride,
                             void *codes, void *scales, void *stream);

/* The values that codes and scales stand for -> y [rows][k] (fp32 / bf16, both exact). */
cfwd_status cfwd_mx_dequantize(long long rows, int k, cfwd_dtype dtype, const void *codes, const void *scales,
                               void *y, void *stream);

/* y [m][n] = act(x w^T + bias): x [m][k], w MXFP4 [n][k]. */
typedef struct {
    long long m;
    int n, k;
    cfwd_dtype x_dtype; /* MXFP4, or fp32 / bf16: x is quantised by the call, to the same codes as cfwd_mx_quantize's */
    cfwd_dtype y_dtype; /* fp32, bf16 (round to nearest even) or MXFP4 (quantised from the fp32 result) */
    long long x_stride; /* row pitch of an fp32 / bf16 x in elements, >= k; ignored for MXFP4 */
    cfwd_activation act;
} cfwd_mx_matmul_desc;

/* Workspace bytes of cfwd_mx_matmul (the quantised x, partial sums of a split reduction); 0 when none. */
cfwd_status cfwd_mx_matmul_workspace_size(const cfwd_mx_matmul_desc *desc, size_t *bytes);

/* The product: exact products, fp32 sums, bias and activation in fp32, one
 * rounding to y.  x_scales and y_scales belong to an MXFP4 x / y and are NULL
 * otherwise.  bias: fp32 [n] or NULL.  y and y_scales must not overlap an
 * input; workspace 256-byte aligned. */
cfwd_status cfwd_mx_matmul(const cfwd_mx_matmul_desc *desc, const void *x, const void *x_scales, const void *w,
                           const void *w_scales, const float *bias, void *y, void *y_scales, void *workspace,
                           size_t ws_bytes, void *stream);

/* Norms before and after a block, with its gate and the residual scale:
 *   s = residual_scale * r + gate * post(b)      h = pre(s)
 * b: the block's output, r: the residual stream, s: the new residual stream,
 * h: the next block's input, all [rows][c].  A norm of v over its row is
 *   RMS    v / sqrt(mean(v^2) + eps) * weight + bias
 *   LAYER  (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) * weight + bias
 *   NONE   v
 * All in fp32; s and h are rounded once, h from the unrounded s. */
typedef enum { CFWD_NORM_NONE = 0, CFWD_NORM_RMS = 1, CFWD_NORM_LAYER = 2 } cfwd_norm_kind;

typedef struct {
    long long rows;
    int c;
    long long rows_per_gate;  /* row i takes row i / rows_per_gate of gate; 0: one row of gate for all */
    float residual_scale, eps;
    cfwd_norm_kind post, pre;
    cfwd_dtype dtype;         /* of b and gate: fp32 or bf16 */
    cfwd_dtype stream_dtype;  /* of r and s: fp32, or bf16 where dtype is bf16 or b and gate are NULL */
    cfwd_dtype out_dtype;     /* of h: dtype, or MXFP4 */
} cfwd_gated_norm_desc;

/* residual may be NULL (it then contributes 0), or b (its norm then counts as 0
 * whatever eps is, so that post(b) is post_bias), gate NULL (1), s or h NULL
 * (not wanted); weights and biases are fp32 [c] or NULL (1 and 0).
 * gate: [ceil(rows / rows_per_gate)][c].  h_scales: with an MXFP4 h only.  s
 * may be residual itself, or b itself where both have one type; apart from that no output
 * may overlap an input or the other output.  1 <= c <= 2^22, eps >= 0. */
cfwd_status cfwd_gated_norm(const cfwd_gated_norm_desc *desc, const void *b, const void *residual, const void *gate,
                            const float *post_weight, const float *post_bias, const float *pre_weight,
                            const float *pre_bias, void *s, void *h, void *h_scales, void *stream);

/* ---- Attention: rotary positions, a paged cache in MXFP4, attention over the
 * cache and over packed prompts.  With the products and norms above, the other half of a
 * transformer layer; image and video networks with attention over patches use
 * the same calls.
 *
 * A tensor of heads is [tokens][heads][dim] with dense dims; its token and head
 * strides (in elements) are the caller's, so that queries, keys and values may
 * be parts of one projection's output.  Outputs of attention and of the cache
 * are dense.  Integers that live on the device (positions, slots, pages,
 * lengths, starts) are read by the kernels: values out of range never lead a
 * memory access out of its buffer, and what they mean instead stands at each call.
 * Nothing here allocates device memory, waits, or uses atomics: the same
 * inputs give the same bits.  tokens or sequences may be 0: nothing is done. */

/* Rotary positions.  Pair i of a head, (a, b), becomes
 *   (a cos t - b sin t, a sin t + b cos t),   t = position[axis_i] * frequency_i,
 * a and b being values i and i + pairs (or, adjacent, 2 i and 2 i + 1) of the
 * head; values from 2 * pairs on stay as they are.  One table entry for each pair:
 *   turns  frequency / (2 pi), the part of a whole turn that one position makes, as a
 *          fraction of 2^64: the product with a position then wraps round at whole turns by
 *          itself, and the angle is exact to 2^-32 of a turn however far the position is
 *   axis   which of a token's positions counts; outside 0 .. axes - 1: none, the pair stays as it is
 * (cfwd_rope_turns gives turns from a frequency.)  sin and cos are taken to 2^-23. */
typedef struct {
    uint64_t turns;
    int32_t axis;
    int32_t reserved; /* 0 */
} cfwd_rope_pair;

typedef struct {
    long long tokens;
    int q_heads, k_heads, head_dim; /* k_heads may be 0 */
    int pairs, axes;                /* 2 * pairs <= head_dim */
    int adjacent;
    int wide_positions; /* positions are int64 [tokens][axes] instead of int32 */
    cfwd_dtype dtype;   /* fp32 or bf16 */
    long long q_stride, q_head_stride, k_stride, k_head_stride; /* of the inputs, in elements */
    long long q_out_stride, q_out_head_stride, k_out_stride, k_out_head_stride;
} cfwd_rope_desc;

/* round(2^64 frequency / (2 pi)) mod 2^64 for a frequency in radians a position. */
uint64_t cfwd_rope_turns(double frequency);

/* q, k -> q_out, k_out, which may be the inputs themselves (same pointer and
 * strides) and overlap nothing else.  table: device [pairs], 16-byte aligned.
 * Tensors need only their element's alignment.  Enqueued on `stream`. */
cfwd_status cfwd_rope(const cfwd_rope_desc *desc, const void *q, const void *k, const void *positions,
                      const cfwd_rope_pair *table, void *q_out, void *k_out, void *stream);

/* The paged cache: keys, and values, as MXFP4 rows [pages][heads][page_size]
 * of head_dim values (codes and scales as above).  A token's place is its slot,
 * page * page_size + offset; a sequence's tokens 0, 1, .. lie in the pages that its row of the
 * page table [sequences][table_pitch] names, page_size in each. */
typedef struct {
    int pages, page_size, kv_heads, head_dim;
    void *k_codes, *k_scales, *v_codes, *v_scales; /* codes 16-byte aligned, scales 4-byte */
} cfwd_mx_cache;

/* Quantises k and v [tokens][kv_heads][head_dim] (fp32 / bf16; strides for both) into the
 * slots int32 (or wide: int64) [tokens], to the same codes as cfwd_mx_quantize.  A token whose slot is not in
 * 0 .. pages * page_size - 1 is left out (a padded batch has -1 there).  Slots that are given must
 * differ from each other: what a slot given twice then holds is not defined. */
typedef struct {
    long long tokens;
    cfwd_dtype dtype;
    int wide_slots;
    long long k_stride, k_head_stride, v_stride, v_head_stride;
} cfwd_mx_cache_write_desc;

cfwd_status cfwd_mx_cache_write(const cfwd_mx_cache_write_desc *desc, const cfwd_mx_cache *cache, const void *k,
                                const void *v, const void *slots, void *stream);

/* The first tokens of every sequence back as values (exact in both types):
 * row t of k and v [tokens][kv_heads][head_dim] is token t - starts[i] of the sequence i with
 * starts[i] <= t < starts[i + 1] (starts: int32 [sequences + 1], from 0, never falling).
 * Rows behind the last sequence, and rows whose page is not in 0 .. pages - 1 or not in the table, are not written. */
typedef struct {
    long long tokens;
    int sequences, table_pitch;
    cfwd_dtype dtype;
} cfwd_mx_cache_read_desc;

cfwd_status cfwd_mx_cache_read(const cfwd_mx_cache_read_desc *desc, const cfwd_mx_cache *cache, const int32_t *page_table,
                               const int32_t *starts, void *k, void *v, void *stream);

/* Attention of each sequence's newest tokens over its cache:
 *   o = softmax(scale * q K^T) V
 * q [sequences][tokens][q_heads][head_dim] and o are bf16; query head h reads head h / (q_heads / kv_heads)
 * of the cache.  lengths: int32 [sequences], tokens in the cache, the new ones
 * among them: query i sees the first length - tokens + 1 + i of them.  Lengths
 * are taken as 0 below 0 and as table_pitch * page_size above it; tokens on pages outside 0 .. pages - 1 are not
 * seen; a query that sees nothing gives 0.  head_dim: a multiple of 32 up to
 * 256; page_size: a multiple of 16; tokens <= 1024; q_heads a multiple of kv_heads; q 16-byte aligned with strides
 * that are multiples of 8 elements.
 * Queries meet the cache's codes in two parts of 8 bits: exactly, but for values under 2^-13 of the largest of their 128,
 * which are within 2^-21 of it.  Products are exact and summed in fp32, as are the softmax's sums; its weights are rounded
 * to bf16 before the product with V.  A NaN in a key that a query sees makes that query's output NaN, one in a value its
 * column; the others keep their bits.
 * CFWD_ERR_UNSUPPORTED for other types and sizes, pages of 2^31 bytes of codes or more, and page tables that stand for 2^31
 * or more pairs of 128 tokens and 16 queries. */
typedef struct {
    int sequences, tokens, q_heads, table_pitch;
    float scale; /* > 0 */
    cfwd_dtype dtype;
    long long q_seq_stride, q_stride, q_head_stride;
} cfwd_mx_cache_attention_desc;

cfwd_status cfwd_mx_cache_attention_workspace_size(const cfwd_mx_cache_attention_desc *desc, const cfwd_mx_cache *cache,
                                                   size_t *bytes);

/* workspace: 256-byte aligned, needs no initial contents. */
cfwd_status cfwd_mx_cache_attention(const cfwd_mx_cache_attention_desc *desc, const cfwd_mx_cache *cache, const void *q,
                                    const int32_t *page_table, const int32_t *lengths, void *o, void *workspace,
                                    size_t ws_bytes, void *stream);

/* Attention over packed prompts: o = softmax(scale * q k^T) v for each sequence
 * i, whose queries are rows q_starts[i] .. q_starts[i + 1] - 1 of q [q_tokens][q_heads][head_dim] and
 * whose keys and values are rows k_starts[i] .. k_starts[i + 1] - 1 of k, v [k_tokens][kv_heads][head_dim]
 * (starts: int32 [sequences + 1], never falling; taken as the nearest number in 0 .. tokens).
 * causal: the last query sees every key, the one before it one fewer, and so
 * on; a query that sees no key gives 0.  Rows of o behind the last sequence are
 * not written.  bf16; head_dim a multiple of 8 up to 256; q_heads a multiple of kv_heads; tensors 16-byte aligned, strides
 * multiples of 8 elements, k and v strides from head_dim to 2^24 (CFWD_ERR_UNSUPPORTED for others).  Products are exact and
 * summed in fp32, as are the softmax's sums; its weights are rounded to bf16 before the product with v.  They are taken
 * relative to a number that the scores pass by at most a factor of 2^12, here as over the cache: values up to 2^90 or so
 * leave the sums in fp32's range. */
typedef struct {
    long long q_tokens, k_tokens;
    int sequences, q_heads, kv_heads, head_dim;
    int causal;
    float scale; /* > 0 */
    cfwd_dtype dtype;
    long long q_stride, q_head_stride, k_stride, k_head_stride, v_stride, v_head_stride;
} cfwd_attention_desc;

cfwd_status cfwd_attention_workspace_size(const cfwd_attention_desc *desc, size_t *bytes);

cfwd_status cfwd_attention(const cfwd_attention_desc *desc, const void *q, const void *k, const void *v,
                           const int32_t *q_starts, const int32_t *k_starts, void *o, void *workspace, size_t ws_bytes,
                           void *stream);

/* Static description of a status code. */
const char *cfwd_status_string(cfwd_status status);

/* Detail of this thread's most recent failure ("" if none). */
const char *cfwd_last_error(void);

/* Name of an algorithm, e.g. "implicit_gemm/3". */
const char *cfwd_algo_name(cfwd_algo algo);

#ifdef __cplusplus
}
#endif

#endif /* CFWD_H */
