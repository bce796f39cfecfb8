/*
 * conv_wgrad.h -- C ABI of the MI355X (gfx950) convolution weight-gradient library.
 *
 * Operation (the weight gradient of a 2-D convolution, "weight.grad" of
 * nn.Conv2d in rocm-libraries PR #11188 "fix silent zero wgrad", section
 * Motivation; for a 1x1 filter it equals dY^T X on the [N*H*W, .] matrices,
 * the "F.linear on the reshaped tensor" equivalence of the same section):
 *
 *   dW[k, r, s, c] = sum_{n, ho, wo} dY[n, ho, wo, k]
 *                    * X[n, ho*stride + r*dilation - pad, wo*stride + s*dilation - pad, g(k)*Cg + c]
 *
 *   Cg = C / groups, Kg = K / groups, g(k) = k / Kg; X is zero outside the
 *   H x W image (the same pad on all four sides; stride and dilation are the
 *   same on both axes); Ho = (H + 2*pad - dilation*(R-1) - 1) / stride + 1,
 *   Wo likewise.
 *
 * Layouts (dense, row-major, no strides):
 *   x  : [N][H][W][C]    element type desc->dtype
 *   dy : [N][Ho][Wo][K]  element type desc->dtype
 *   dw : [K][R][S][Cg]   fp32, always (fp32 accumulation for every dtype)
 *
 * Execution: the reduction over N*Ho*Wo is cut into ks_count slices
 * ("split-K", the two-stage scheme of rocm-libraries PR #14393 "split-K
 * forward implicit-GEMM convolution on gfx1250", section "Two-stage split-K").
 * With ks_count > 1 every stage-1 workgroup writes its fp32 partial tile into
 * slab `slice` of the workspace exactly once, and a second kernel folds the
 * slabs in one fixed order that depends only on ks_count (16 consecutive
 * parts of the slab range, each summed in ascending slab order, then the part
 * sums in ascending part order; beyond 256 slabs, runs of 32 slabs are folded
 * first the same way); with ks_count == 1 stage 1 writes dw directly.  Results are therefore bit-identical from run to run for a fixed
 * split degree, and the workspace needs no clearing.  Tensor base addresses
 * and image offsets are 64-bit, so tensors larger than 4 GB are handled in
 * one launch (the failure mode of rocm-libraries PR #11188, sections
 * Motivation and Technical Details, where a truncating split computation let
 * one dispatch address more than ~4 GB and silently return zeros).
 *
 * Errors are returned, never hidden: validation is synchronous and happens
 * before anything is enqueued; on any error nothing is enqueued and dw is not
 * touched.  There is no fallback path.
 */
#ifndef CONV_WGRAD_H_
#define CONV_WGRAD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of x and dy.  dw is always fp32. */
typedef enum conv_wgrad_dtype {
  CONV_WGRAD_F32 = 0,
  CONV_WGRAD_BF16 = 1,
  CONV_WGRAD_F16 = 2
} conv_wgrad_dtype_t;

/*
 * Problem descriptor.  All fields are read; the struct is copied, never kept.
 *   N, C, H, W : input batch, channels, height, width (each >= 1)
 *   K, R, S    : output channels, filter height, filter width (each >= 1)
 *   pad >= 0, stride >= 1, dilation >= 1 (same value for both spatial axes)
 *   groups >= 1, dividing both C and K
 *   dtype      : conv_wgrad_dtype_t of x and dy
 *   split_k    : -1 = choose the number of reduction slices automatically;
 *                n >= 1 = pin it.  The pinned degree is honoured except that
 *                no slice may be empty: with U reduction units the plan uses
 *                ceil(U / ceil(U / n')) slices with n' = min(n, 65536)
 *                (never more than n).  Any other
 *                value (0, < -1) is CONV_WGRAD_ERR_BAD_SPLIT, as in the
 *                split-K validators of rocm-libraries PR #14393 (section
 *                "Review follow-ups": split_k <= 0 is rejected).
 */
typedef struct conv_wgrad_desc {
  int64_t N, C, H, W, K, R, S;
  int64_t pad, stride, dilation, groups;
  int32_t dtype;
  int32_t split_k;
} conv_wgrad_desc_t;

typedef enum conv_wgrad_status {
  CONV_WGRAD_OK = 0,
  CONV_WGRAD_ERR_NULL_ARG = 1,     /* desc, x, dy, dw or a needed workspace is NULL */
  CONV_WGRAD_ERR_BAD_SHAPE = 2,    /* a dimension < 1, pad < 0, stride/dilation < 1,
                                      C or K not divisible by groups, Ho or Wo < 1,
                                      or a size that overflows int64 */
  CONV_WGRAD_ERR_BAD_DTYPE = 3,    /* dtype is not a conv_wgrad_dtype_t */
  CONV_WGRAD_ERR_BAD_SPLIT = 4,    /* split_k is 0 or < -1 */
  CONV_WGRAD_ERR_UNSUPPORTED = 5,  /* valid, but outside the library's documented
                                      limits (see conv_wgrad_get_plan) */
  CONV_WGRAD_ERR_MISALIGNED = 6,   /* x, dy, dw or workspace not 16-byte aligned */
  CONV_WGRAD_ERR_WORKSPACE = 7,    /* conv_wgrad_ex: ws_bytes smaller than required */
  CONV_WGRAD_ERR_HIP = 8           /* the HIP runtime reported an error at launch */
} conv_wgrad_status_t;

/* Which stage-1 kernel family a plan uses. */
typedef enum conv_wgrad_path {
  CONV_WGRAD_PATH_DENSE = 0,   /* implicit GEMM per group on MFMA */
  CONV_WGRAD_PATH_DIRECT = 1   /* direct per-group kernel for small groups (depthwise, <= 8 ch/group) */
} conv_wgrad_path_t;

/*
 * The execution plan the library derives from a descriptor (pure host
 * integer arithmetic; no GPU needed).  Exposed for tests and diagnostics.
 */
typedef struct conv_wgrad_plan {
  int32_t path;            /* conv_wgrad_path_t */
  int32_t variant;         /* kernel variant within the path (diagnostic) */
  int64_t Ho, Wo;          /* output extents */
  int64_t L;               /* reduction length N*Ho*Wo */
  int64_t E;               /* dW elements K*R*S*Cg */
  int64_t unit_rows;       /* reduction rows per unit (a unit is the smallest slice grain) */
  int64_t units;           /* reduction units: ceil(L / unit_rows) or per-path equivalent */
  int64_t units_per_slice; /* ceil(units / requested degree); depthwise with 2..256 slices: the
                              longest slice (slices there are balanced by the X rows each stages) */
  int32_t ks_count;        /* slices >= 1, none empty: ceil(units / units_per_slice), except for
                              balanced depthwise slices, whose count is the uniform one's */
  int32_t needs_reduce;    /* 1 iff ks_count > 1: the only condition for launching stage 2 */
  int64_t tiles;           /* output tiles per slice */
  int64_t grid;            /* stage-1 workgroups = tiles * ks_count */
  int64_t slab_stride;     /* fp32 elements between workspace slabs (multiple of 64) */
  uint64_t ws_bytes;       /* workspace bytes: ks_count * slab_stride * 4, or 0 */
  uint64_t x_bytes, dy_bytes, dw_bytes;  /* tensor sizes in bytes */
  int64_t windows_4g;      /* ceil(max(x_bytes, dy_bytes) / 2^32): 4-GiB address windows the
                              tensors span (diagnostic; one launch covers them all) */
} conv_wgrad_plan_t;

/*
 * Human-readable name of a status code (static storage; never NULL; "unknown
 * status" for a value outside the enum).  Every failure is reported as one of
 * these codes rather than as a silently wrong dW: a weight gradient that came
 * back all zeros with no error is the failure rocm-libraries PR #11188
 * ("fix silent zero wgrad", section Motivation) fixed.
 */
const char* conv_wgrad_status_string(conv_wgrad_status_t status);

/*
 * Workspace bytes conv_wgrad and conv_wgrad_bias need for desc: ks_count fp32
 * slabs (each holding one slice's partial dW, then its partial db), or 0 when
 * the plan has one slice.  The workspace is the split-K slab buffer of
 * rocm-libraries PR #14393 (section "Two-stage split-K": every workgroup stores
 * an fp32 partial tile into its slab; section "ABI, AOT and runtime": the
 * split-K form takes a workspace argument).
 *   desc  : read only
 *   bytes : host pointer, written on success only
 * Pure host function (no HIP call).  Errors: NULL_ARG (desc or bytes NULL),
 * BAD_SHAPE / BAD_DTYPE / BAD_SPLIT as for conv_wgrad, UNSUPPORTED.
 */
conv_wgrad_status_t conv_wgrad_workspace_size(const conv_wgrad_desc_t* desc, size_t* bytes);

/*
 * Fill *plan with the plan for desc: the stage-1 kernel, the reduction units,
 * the split degree (split_k = -1 resolves it automatically, n >= 1 pins it, as
 * in rocm-libraries PR #14393, section "Auto-deduced degree (split_k = -1)";
 * the slices come from exact integer ceiling divisions, the form whose
 * truncating variant under-counted the batch split in rocm-libraries
 * PR #11188, section Technical Details), the grid and the workspace size.
 *   desc : read only;  plan : host pointer, written on success only
 * Pure host function (no HIP call); the same validation and errors as
 * conv_wgrad (NULL_ARG for a NULL desc or plan).
 */
conv_wgrad_status_t conv_wgrad_get_plan(const conv_wgrad_desc_t* desc, conv_wgrad_plan_t* plan);

/*
 * Enqueue the weight gradient on `stream` (a hipStream_t; NULL = the null
 * stream of the current device) and return without synchronising.
 *   x, dy     : device pointers, layouts above, 16-byte aligned
 *   dw        : device pointer, fp32 [K][R][S][Cg], 16-byte aligned; overwritten
 *               (every element written exactly once; no accumulate)
 *   workspace : device pointer of at least conv_wgrad_workspace_size bytes,
 *               16-byte aligned; may be NULL when that size is 0.  Its content on
 *               entry is irrelevant.  The caller owns every buffer; the library
 *               never allocates or frees device memory.
 * Buffers must not overlap.  Concurrent calls on different streams need
 * different workspaces.
 */
conv_wgrad_status_t conv_wgrad(const conv_wgrad_desc_t* desc, const void* x, const void* dy,
                               float* dw, void* workspace, void* stream);

/* As conv_wgrad, also checking that ws_bytes covers the workspace the plan needs
 * (CONV_WGRAD_ERR_WORKSPACE otherwise). */
conv_wgrad_status_t conv_wgrad_ex(const conv_wgrad_desc_t* desc, const void* x, const void* dy,
                                  float* dw, void* workspace, size_t ws_bytes, void* stream);

/*
 * Profiling variant of conv_wgrad: identical work on `stream`, and the caller's
 * HIP events (hipEvent_t, created by the caller; either may be NULL) take the
 * start and end timestamps of the stage-1 kernel's own dispatch (the stage-1
 * launch goes through hipExtLaunchKernel with them), so the caller can time
 * that kernel alone, without the launch gaps around it; the slab reduce, when
 * launched, is not included.  The events are only recorded, never
 * synchronised or destroyed.
 */
conv_wgrad_status_t conv_wgrad_timed(const conv_wgrad_desc_t* desc, const void* x, const void* dy,
                                     float* dw, void* workspace, size_t ws_bytes, void* stream,
                                     void* stage1_begin, void* stage1_end);

/*
 * Weight gradient and bias gradient in one pass over dy.  The bias gradient of
 * a convolution is the sum of the output gradient over every output pixel
 * (rocm-libraries PR #11188, section Motivation, checks bias.grad beside
 * weight.grad of nn.Conv2d):
 *   db[k] = sum over n, ho, wo of dy[n][ho][wo][k]
 *   db        : device pointer, fp32 [K], 16-byte aligned; overwritten
 * The stage-1 kernels add up the dy values they already stage, per slice;
 * db is folded with the slabs in the same fixed order as dw (fp32 adds), so
 * the result is bit-identical from run to run at a fixed split, and dw is
 * bit-identical to what conv_wgrad_ex writes for the same desc.  The other
 * arguments, the workspace size and the errors are those of conv_wgrad_ex
 * (NULL_ARG also for a NULL db, MISALIGNED for a misaligned one).
 */
conv_wgrad_status_t conv_wgrad_bias(const conv_wgrad_desc_t* desc, const void* x, const void* dy,
                                    float* dw, float* db, void* workspace, size_t ws_bytes,
                                    void* stream);

/* Profiling variant of conv_wgrad_bias, with stage-1 events as in conv_wgrad_timed. */
conv_wgrad_status_t conv_wgrad_bias_timed(const conv_wgrad_desc_t* desc, const void* x,
                                          const void* dy, float* dw, float* db, void* workspace,
                                          size_t ws_bytes, void* stream, void* stage1_begin,
                                          void* stage1_end);

/*
 * Extended problem descriptor: per-axis geometry, an arithmetic mode for fp32
 * inputs and the width fold.  conv_wgrad_desc_t is this with equal axes,
 * math = CONV_WGRAD_MATH_EXACT and fold_width = -1.
 *
 * Per-axis geometry (the column padding pad_w beside the row padding of
 * rocm-libraries PR #14393's embedded depthwise-dgrad PR #14386, section
 * "Per-axis padding"; stride and dilation the same way):
 *   dW[k, r, s, c] = sum_{n, ho, wo} dY[n, ho, wo, k]
 *       * X[n, ho*stride_h + r*dil_h - pad_h, wo*stride_w + s*dil_w - pad_w, g(k)*Cg + c]
 *   Ho = (H + 2*pad_h - dil_h*(R-1) - 1) / stride_h + 1,
 *   Wo = (W + 2*pad_w - dil_w*(S-1) - 1) / stride_w + 1.
 *   pad_h, pad_w >= 0; stride_h, stride_w, dil_h, dil_w >= 1 (BAD_SHAPE otherwise).
 *
 * math (fp32 inputs; ignored for bf16 / fp16, which always use their own MFMA):
 *   CONV_WGRAD_MATH_EXACT  (0): fp32 products on f32 MFMA (the default).
 *   CONV_WGRAD_MATH_BF16X3 (1): BF16x3 emulation, the form the pages give for
 *       fp32 ("TF32") matrix work on gfx950 (rocm-libraries PR #14393,
 *       timeline, the TF32 entry: native XF32 on gfx942, BF16x3 on gfx950):
 *       each fp32 value v = hi + lo with hi = bf16(v), lo = bf16(v - hi), and
 *       a*b ~ a_hi*b_hi + a_hi*b_lo + a_lo*b_hi on bf16 MFMA with fp32
 *       accumulation.  Each product carries a relative error of at most about
 *       3 * 2^-16 (the dropped a_lo*b_lo term and the two splits' residuals),
 *       so the normalised error is bounded by ~4.6e-5 in the worst case and is
 *       ~1e-7 for inputs of random sign.  It is a permission, never a silent
 *       downgrade of other shapes: the plan uses it only where a BF16x3 kernel
 *       covers the shape (plan variant CONV_WGRAD_VARIANT_DENSE_BF16X3 or
 *       CONV_WGRAD_VARIANT_DENSE_BF16X3_TAPS) and the exact fp32 path
 *       elsewhere.  Any other value is BAD_DTYPE.
 * fold_width (rocm-libraries PR #14393, commit bodies, the fold_width
 * paragraph: f adjacent W positions folded into the channels when f divides
 * the filter width, the W stride, the input width and the W padding; the
 * identity holds in every direction, so it is a view of the same tensors):
 *   -1: fold by the largest such f when the shape gains from it (input
 *       channels per group not a multiple of 4, a multiple after folding);
 *    0 or 1: never fold;  f >= 2: fold by f (BAD_SHAPE if f does not divide
 *       S, stride_w, W and pad_w, or if dil_w != 1 or groups != 1).
 *   Folding changes only the kernel and the summation order, never the
 *   layouts: X [N][H][W][C] is read as [N][H][W/f][f*C], dY is unchanged, and
 *   dW [K][R][S][Cg] is written as [K][R][S/f][f*Cg] -- the same bytes.
 */
typedef struct conv_wgrad_desc2 {
  int64_t N, C, H, W, K, R, S;
  int64_t pad_h, pad_w, stride_h, stride_w, dil_h, dil_w;
  int64_t groups;
  int32_t dtype;       /* conv_wgrad_dtype_t of x and dy */
  int32_t split_k;     /* as in conv_wgrad_desc_t */
  int32_t math;        /* CONV_WGRAD_MATH_* */
  int32_t fold_width;  /* -1 auto, 0 / 1 off, f >= 2 fold by f */
} conv_wgrad_desc2_t;

#define CONV_WGRAD_MATH_EXACT 0
#define CONV_WGRAD_MATH_BF16X3 1

/* conv_wgrad_plan_t::variant of the BF16x3 dense kernels: the row kernel
 * (one filter row per tile) and the all-taps kernel (3 x 3 filters, output
 * rows of at most 61 pixels). */
#define CONV_WGRAD_VARIANT_DENSE_BF16X3 4
#define CONV_WGRAD_VARIANT_DENSE_BF16X3_TAPS 6

/* The plan of an extended descriptor: the base plan (of the problem the kernels
 * run, i.e. after a width fold) and what was applied. */
typedef struct conv_wgrad_plan2 {
  conv_wgrad_plan_t base;
  int32_t math;        /* CONV_WGRAD_MATH_* the kernels use */
  int32_t fold_width;  /* applied fold (1 = none) */
} conv_wgrad_plan2_t;

/*
 * conv_wgrad_workspace_size for an extended descriptor: the workspace bytes
 * conv_wgrad2 needs (0 when the plan has one slice).  Pure host function;
 * errors: NULL_ARG (desc or bytes NULL), BAD_SHAPE, BAD_DTYPE (also a math
 * value outside CONV_WGRAD_MATH_*), BAD_SPLIT, UNSUPPORTED.
 */
conv_wgrad_status_t conv_wgrad2_workspace_size(const conv_wgrad_desc2_t* desc, size_t* bytes);

/* conv_wgrad_get_plan for an extended descriptor (same validation and errors). */
conv_wgrad_status_t conv_wgrad2_get_plan(const conv_wgrad_desc2_t* desc, conv_wgrad_plan2_t* plan);

/*
 * The weight gradient (and, when db is not NULL, the bias gradient db[k] =
 * sum of dy over n, ho, wo) for an extended descriptor, enqueued on `stream`.
 * Layouts, ownership, workspace rules (at least conv_wgrad2_workspace_size
 * bytes, WORKSPACE otherwise; NULL allowed when that is 0), alignment,
 * determinism at a fixed split and errors are those of conv_wgrad_bias; dw
 * and db are overwritten.
 */
conv_wgrad_status_t conv_wgrad2(const conv_wgrad_desc2_t* desc, const void* x, const void* dy,
                                float* dw, float* db, void* workspace, size_t ws_bytes, void* stream);

/* Profiling variant of conv_wgrad2, with stage-1 events as in conv_wgrad_timed. */
conv_wgrad_status_t conv_wgrad2_timed(const conv_wgrad_desc2_t* desc, const void* x, const void* dy,
                                      float* dw, float* db, void* workspace, size_t ws_bytes,
                                      void* stream, void* stage1_begin, void* stage1_end);

/* Profiling variant of conv_wgrad2 that times the whole call on the GPU: the
 * caller's events (hipEvent_t, either may be NULL) take the start timestamp of
 * the call's first kernel (stage 1) and the end timestamp of its last kernel
 * (the slab fold, or stage 1 with one slice), through hipExtLaunchKernel, so
 * hipEventElapsedTime gives stage 1 + fold + the gap between them without any
 * marker of its own.  Only recorded, never synchronised or destroyed. */
conv_wgrad_status_t conv_wgrad2_call_timed(const conv_wgrad_desc2_t* desc, const void* x, const void* dy,
                                           float* dw, float* db, void* workspace, size_t ws_bytes,
                                           void* stream, void* call_begin, void* call_end);

/*
 * Forward convolution and data gradient on the same implicit-GEMM, split-K
 * slab and fold machinery (rocm-libraries PR #14393 "split-K forward
 * implicit-GEMM convolution on gfx1250": sections Summary, "Two-stage
 * split-K" -- every workgroup stores an fp32 partial tile into its slab, a
 * second kernel folds the slabs, no workspace clearing, deterministic -- and
 * "Auto-deduced degree (split_k = -1)", whose policy is refitted here for 256
 * CUs: split only a grid under 4 workgroups per CU (1024) over a reduction at
 * least 512 deep, by the smallest power of two that brings the grid to 8
 * workgroups per CU (2048), at most 32, with at least two 32-entry reduction
 * tiles per slice).
 *
 *   forward: y[n][ho][wo][k] = sum_{r,s,c} x[n][ho*stride_h + r*dil_h - pad_h]
 *                                            [wo*stride_w + s*dil_w - pad_w][g(k)*Cg + c]
 *                                          * w[k][r][s][c]
 *   dgrad:   dx[n][h][w][g*Cg + c] = sum over k of group g and r, s with
 *              ho*stride_h = h + pad_h - r*dil_h, wo*stride_w = w + pad_w - s*dil_w
 *              (exactly, 0 <= ho < Ho, 0 <= wo < Wo) of dy[n][ho][wo][k] * w[k][r][s][c]
 *
 * The descriptor is conv_wgrad_desc2_t (per-axis geometry, groups, dtype,
 * split_k, fold_width; math is read as in conv_wgrad2 and only the exact path
 * exists for these directions).  Layouts: x [N][H][W][C] and dy [N][Ho][Wo][K]
 * and the filter w [K][R][S][Cg] in desc->dtype; y [N][Ho][Wo][K] and dx
 * [N][H][W][C] are fp32 (fp32 accumulation for every dtype), overwritten.
 * Workspace, alignment (16 bytes), ownership, determinism at a fixed split and
 * errors are those of conv_wgrad_ex; the workspace holds ks_count slabs of the
 * whole output.
 */
#define CONV_DIRECTION_WGRAD 0
#define CONV_DIRECTION_FWD 1
#define CONV_DIRECTION_DGRAD 2

/* Plan of a direction (CONV_DIRECTION_*; WGRAD gives conv_wgrad2_get_plan's).
 * For FWD / DGRAD: base.L is the output pixel count, base.E the output
 * elements, base.unit_rows 32 reduction entries, base.variant 20 / 21.
 * Unknown direction: BAD_DTYPE.  Pure host function. */
conv_wgrad_status_t conv_igemm_get_plan(const conv_wgrad_desc2_t* desc, int32_t direction,
                                        conv_wgrad_plan2_t* plan);

/* Workspace bytes of conv_fwd (direction FWD) or conv_dgrad (DGRAD). */
conv_wgrad_status_t conv_igemm_workspace_size(const conv_wgrad_desc2_t* desc, int32_t direction,
                                              size_t* bytes);

/* Forward convolution: y (fp32) from x and w, enqueued on stream. */
conv_wgrad_status_t conv_fwd(const conv_wgrad_desc2_t* desc, const void* x, const void* w, float* y,
                             void* workspace, size_t ws_bytes, void* stream);

/* Data gradient: dx (fp32) from dy and w, enqueued on stream. */
conv_wgrad_status_t conv_dgrad(const conv_wgrad_desc2_t* desc, const void* dy, const void* w, float* dx,
                               void* workspace, size_t ws_bytes, void* stream);

/* Profiling variant of conv_fwd (direction FWD: src = x, out = y) and
 * conv_dgrad (DGRAD: src = dy, out = dx) that times the whole call on the
 * GPU as conv_wgrad2_call_timed does: call_begin takes the start timestamp of
 * the implicit GEMM's dispatch, call_end the end timestamp of the call's last
 * kernel (either may be NULL; only recorded).  Another direction: BAD_DTYPE. */
conv_wgrad_status_t conv_igemm_call_timed(const conv_wgrad_desc2_t* desc, int32_t direction,
                                          const void* src, const void* w, float* out, void* workspace,
                                          size_t ws_bytes, void* stream, void* call_begin,
                                          void* call_end);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): conv_wgrad_bias
 * without the workspace argument.  The slabs live in a library-owned device
 * array of CONV_WGRAD_NOALLOC_SCRATCH_BYTES (64 MiB) per GPU, held until the
 * process ends; its device address is looked up (hipGetSymbolAddress) on the
 * first call on each device, with that device current.  No call allocates or
 * frees memory (no hipMalloc / hipFree, no allocating library routine).
 *   db : NULL for the weight gradient only (dw then equals conv_wgrad's), or
 *        an fp32 [K] buffer for the bias gradient as in conv_wgrad_bias
 * The other arguments, the results and the errors are those of conv_wgrad_bias,
 * plus CONV_WGRAD_ERR_WORKSPACE when conv_wgrad_workspace_size(desc) exceeds
 * CONV_WGRAD_NOALLOC_SCRATCH_BYTES (pin a smaller split_k to fit) and
 * CONV_WGRAD_ERR_HIP when the address lookup fails; errors are returned
 * before anything is enqueued.  The current device must be the stream's.
 * Every call on one GPU shares that GPU's array (nothing in it needs clearing:
 * each slab element is written before the fold reads it), so calls that
 * overlap in time on one GPU (other streams, other host threads) race.
 */
#define CONV_WGRAD_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
conv_wgrad_status_t conv_wgrad_noalloc(const conv_wgrad_desc_t* desc, const void* x, const void* dy,
                                       float* dw, float* db, void* stream);

/* ------------------------------------------------------------------------------------------------------------------
 * Sequence operators: the root-mean-square norm and the layer norm, the short causal (depthwise) convolution over tokens,
 * the selective state space scan and the gated delta rule, which together with two matrix products make a layer of a
 * sequence model.  Tokens are rows, channels the contiguous axis; element types as above (desc dtype), arithmetic and
 * every sum in fp32.
 *
 * Execution is as for the convolutions: validation is synchronous and comes before anything is enqueued, the kernels
 * go to `stream`, nothing is allocated, and results are bit-identical from run to run.  The one thing validation
 * cannot see is the content of device arrays: any offsets and slots are memory-safe (see seq_tokens_t).
 */

/* A tensor of rows: element (b, t, c) is at ptr + b * batch + t * row + c, strides in elements, >= 0 (0: the same row
 * for all).  Element alignment suffices. */
typedef struct seq_view {
  void* ptr;
  int64_t batch, row;
} seq_view_t;

/*
 * How rows make up sequences.
 *   offsets NULL : `sequences` sequences of `rows` tokens each; sequence s is batch index s.
 *   offsets      : device int32 [sequences + 1], offsets[0] = 0, not decreasing: sequence s is rows offsets[s] ..
 *                  offsets[s + 1] - 1 of `rows` in all (batch index 0).  Rows from offsets[sequences] on are padding:
 *                  their outputs are zero.  Offsets that break these rules give outputs without meaning, in bounds.
 *   slots        : device int32 [sequences] or NULL (s itself): where sequence s has its state in a pool of `pool`
 *                  states.  A slot outside [0, pool) stands for no state: it reads as zeros and is not written.
 *                  Two sequences with one slot race on it.
 */
typedef struct seq_tokens {
  int64_t sequences, rows;
  const int32_t* offsets;
  const int32_t* slots;
  int64_t pool;
} seq_tokens_t;

/*
 * y = h r w,  h = x + residual rounded to the element type,  r = 1 / sqrt(mean(h^2) + eps), per row.
 *   x, residual : rows x channels (residual NULL: h = x); row strides in elements
 *   w           : fp32 [channels]
 *   y, h, rstd  : dense outputs; h may be NULL (not needed), rstd fp32 [rows] or NULL.
 * 1 <= channels <= 16384, rows >= 0.
 */
typedef struct seq_norm_args {
  int64_t rows, channels;
  int32_t dtype;
  int32_t group;          /* seq_rms_norm_e4m3: channels per scale (0: the row; 32, 64, 128, 256) */
  float eps;
  int32_t reserved;
  const void* x;
  int64_t x_row;
  const void* residual;
  int64_t residual_row;
  const float* w;
  void* y;                /* seq_rms_norm_e4m3: 8-bit [rows][channels] */
  void* h;
  float* rstd;
  float* scale;           /* seq_rms_norm_e4m3: [rows][ceil(channels / group)] */
} seq_norm_args_t;

conv_wgrad_status_t seq_rms_norm(const seq_norm_args_t* args, void* stream);

/* The norm with an 8-bit output (OCP e4m3, largest value 448): per group of channels scale = max|h r w| / 448 (1 where
 * that is zero) and y = e4m3(h r w / scale), rounded to nearest even.  A scale below fp32's normal range has few bits,
 * so that the quotient can pass 448: it is held to that. */
conv_wgrad_status_t seq_rms_norm_e4m3(const seq_norm_args_t* args, void* stream);

/*
 * Gradients of seq_rms_norm:  dx = r (dy w - h r^2 mean(dy w h)) + dh  (also the residual's gradient) and
 * dw = sum over rows of dy h r.  h and rstd are the forward's (h = x without a residual).
 *   dh : gradient that reaches h by another way, or NULL
 *   workspace : 16-byte aligned, seq_rms_norm_grad_workspace bytes
 */
typedef struct seq_norm_grad_args {
  int64_t rows, channels;
  int32_t dtype;
  int32_t reserved;
  const void* dy;
  int64_t dy_row;
  const void* h;
  int64_t h_row;
  const void* dh;
  int64_t dh_row;
  const float* w;
  const float* rstd;
  void* dx;               /* [rows][channels] */
  float* dw;              /* [channels] */
} seq_norm_grad_args_t;

conv_wgrad_status_t seq_rms_norm_grad_workspace(const seq_norm_grad_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_rms_norm_grad(const seq_norm_grad_args_t* args, void* workspace, size_t ws_bytes, void* stream);

/*
 * Layer norm:  y = (h - m) r w + b,  h = x + residual rounded to the element type,  m = mean(h),
 * r = 1 / sqrt(mean((h - m)^2) + eps), per row.
 *   x, residual : rows x channels (residual NULL: h = x); row strides in elements
 *   w, b        : fp32 [channels]; b may be NULL (zeros)
 *   y, h        : dense outputs; h may be NULL (not needed)
 *   mean, rstd  : fp32 [rows] or NULL: m and r, which the gradient reads
 * 1 <= channels <= 16384, rows >= 0.
 */
typedef struct seq_layer_norm_args {
  int64_t rows, channels;
  int32_t dtype;
  float eps;
  const void* x;
  int64_t x_row;
  const void* residual;
  int64_t residual_row;
  const float* w;
  const float* b;
  void* y;
  void* h;
  float* mean;
  float* rstd;
} seq_layer_norm_args_t;

conv_wgrad_status_t seq_layer_norm(const seq_layer_norm_args_t* args, void* stream);

/*
 * Gradients of seq_layer_norm, with n = (h - m) r and g = dy w:
 *   dx = r (g - mean(g) - n mean(g n)) + dh  (also the residual's gradient),  dw = sum over rows of dy n,
 *   db = sum over rows of dy (NULL: not needed).  h, mean and rstd are the forward's (h = x without a residual).
 *   dh : gradient that reaches h by another way, or NULL
 *   workspace : 16-byte aligned, seq_layer_norm_grad_workspace bytes
 */
typedef struct seq_layer_norm_grad_args {
  int64_t rows, channels;
  int32_t dtype;
  int32_t reserved;
  const void* dy;
  int64_t dy_row;
  const void* h;
  int64_t h_row;
  const void* dh;
  int64_t dh_row;
  const float* w;
  const float* mean;
  const float* rstd;
  void* dx;               /* [rows][channels] */
  float* dw;              /* [channels] */
  float* db;              /* [channels] */
} seq_layer_norm_grad_args_t;

conv_wgrad_status_t seq_layer_norm_grad_workspace(const seq_layer_norm_grad_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_layer_norm_grad(const seq_layer_norm_grad_args_t* args, void* workspace, size_t ws_bytes,
                                        void* stream);

/*
 * Short causal convolution, one filter of `width` taps per channel:
 *   p[t, d] = bias[d] + sum_k w[d, k] x[t - (width - 1) + k, d],   y = p  or, with silu, p / (1 + e^-p).
 * Before a sequence's first token x is its state: [pool][width - 1][channels], the last width - 1 inputs, oldest first
 * (NULL: zeros).  state_out receives the window after the last token (NULL: not needed); it is `state` itself or does
 * not overlap it.  State strides are elements between two states of a pool.
 * 2 <= width <= 4; w fp32 [channels][width], bias fp32 [channels] or NULL.
 */
typedef struct seq_conv_args {
  seq_tokens_t tokens;
  int64_t channels;
  int32_t width, dtype, silu, reserved;
  seq_view_t x;
  const float* w;
  const float* bias;
  const void* state;
  int64_t state_stride;
  void* state_out;
  int64_t state_out_stride;
  seq_view_t y;
} seq_conv_args_t;

conv_wgrad_status_t seq_causal_conv(const seq_conv_args_t* args, void* stream);

/* The same for one token of each sequence (tokens.offsets NULL, tokens.rows 1); the window of a slot is read and
 * written by the same lane, so state_out may be state. */
conv_wgrad_status_t seq_causal_conv_step(const seq_conv_args_t* args, void* stream);

/* Gradients: dx, dw, dbias (NULL: not needed) and dstate (dense [sequences][width - 1][channels], NULL: not needed)
 * from dy and dstate_out (the same shape; gradient of the outgoing windows, NULL: zero).  fwd.state holds the windows as
 * they were before the forward: a caller whose forward wrote state_out over them keeps a copy.  fwd.y, fwd.state_out
 * and their strides are not read. */
typedef struct seq_conv_grad_args {
  seq_conv_args_t fwd;
  seq_view_t dy;
  const void* dstate_out;
  seq_view_t dx;
  float* dw;
  float* dbias;
  void* dstate;
} seq_conv_grad_args_t;

conv_wgrad_status_t seq_causal_conv_grad_workspace(const seq_conv_grad_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_causal_conv_grad(const seq_conv_grad_args_t* args, void* workspace, size_t ws_bytes,
                                         void* stream);

/*
 * Selective state space scan.  Per sequence, channel d and state n, with g = d / (channels / groups):
 *   D[t, d] = delta[t, d] + delta_bias[d], with softplus: log(1 + e^that)
 *   h[t, d, n] = e^(D A[d, n]) h[t - 1, d, n] + D u[t, d] B[t, g, n]
 *   y[t, d] = (sum_n h[t, d, n] C[t, g, n] + skip[d] u[t, d]) * (z / (1 + e^-z), z = z[t, d])
 * A fp32 [channels][states]; skip, delta_bias fp32 [channels] or NULL; z.ptr NULL: no gate.  B and C: element
 * (b, t, g, n) at ptr + b * batch + t * row + g * group_stride + n.
 * state, state_out: fp32 [pool][channels][states] (stride elements apart), NULL: zeros / not needed; they may be the
 * same.  save: NULL, or what seq_selective_scan_grad needs, seq_selective_scan_save bytes.
 * longest: no sequence is longer (<= 0: not known); a hint for the split of long sequences, results do not depend on
 * its being right.  1 <= states <= 32.
 */
typedef struct seq_scan_args {
  seq_tokens_t tokens;
  int64_t channels, groups;
  int32_t states, dtype, softplus, reserved;
  int64_t longest;
  seq_view_t u, delta, z, B, C;
  int64_t B_group, C_group;
  const float* A;
  const float* skip;
  const float* delta_bias;
  const float* state;
  int64_t state_stride;
  float* state_out;
  int64_t state_out_stride;
  float* save;
  seq_view_t y;
} seq_scan_args_t;

conv_wgrad_status_t seq_selective_scan_save(const seq_scan_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_selective_scan_workspace(const seq_scan_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_selective_scan(const seq_scan_args_t* args, void* workspace, size_t ws_bytes, void* stream);

/* The same for one token of each sequence (tokens.offsets NULL, tokens.rows 1). */
conv_wgrad_status_t seq_selective_scan_step(const seq_scan_args_t* args, void* stream);

/* Gradients, from dy, dstate_out (dense fp32 [sequences][channels][states], gradient of the final states, NULL: zero)
 * and fwd.save as the forward filled it.  Outputs dense: du, ddelta, dz (NULL without a gate) rows x channels, dB and
 * dC rows x groups x states, dA, dskip and ddelta_bias fp32 (the last two may be NULL), dstate fp32 [sequences]
 * [channels][states] or NULL.  Row strides stay below 2^26 elements.  fwd.y, fwd.state and fwd.state_out are not read. */
typedef struct seq_scan_grad_args {
  seq_scan_args_t fwd;
  seq_view_t dy;
  const float* dstate_out;
  void* du;
  void* ddelta;
  void* dz;
  void* dB;
  void* dC;
  float* dA;
  float* dskip;
  float* ddelta_bias;
  float* dstate;
} seq_scan_grad_args_t;

conv_wgrad_status_t seq_selective_scan_grad_workspace(const seq_scan_grad_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_selective_scan_grad(const seq_scan_grad_args_t* args, void* workspace, size_t ws_bytes,
                                            void* stream);

/*
 * Gated delta rule.  Per sequence and head h, with a state S [key_dim][value_dim] and the queries and keys of head
 * h / (heads / key_heads):
 *   a = e^g[t, h],   S[t] = a S[t - 1] + beta[t, h] k[t] (v[t, h] - (a S[t - 1])^T k[t])^T,   o[t, h] = scale S[t]^T q[t]
 * q, k: element (b, t, h, d) at ptr + b * batch + t * row + h * q_head + d; v likewise; o likewise with value_dim
 * elements between heads.  g, beta: fp32, element (b, t, h) at ptr + b * batch + t * row + h.  g is a logarithm, as a rule
 * <= 0 (-inf forgets); keys are as a rule of unit length (with beta |k|^2 > 2 the recurrence itself grows).
 * state, state_out: fp32 [pool][heads][key_dim][value_dim] (stride elements apart), NULL: zeros / not needed; they may be
 * the same and do not overlap otherwise, nor do outputs and inputs.  save: NULL, or what seq_gated_delta_grad needs,
 * seq_gated_delta_save bytes, 16-byte aligned.
 * 1 <= key_dim <= 256, 1 <= value_dim <= 1024, heads a multiple of key_heads and at most 65536.
 * States, products and sums keep 32-bit accuracy for every element type; where g > 0, of what a chunk of 64 tokens would grow
 * to by its g alone (a growth that beta k k^T takes back in every direction, as with key_dim 1, leaves e^(sum of g) 2^-24 of
 * it).  What an infinite or NaN element reaches: of q its
 * own token's output; of v its column of the head's outputs from its token on, and of the state; of k, beta and g (-inf is
 * none, it forgets) all of the head's outputs from its token on, and the state; of the state its column of all the
 * sequence's outputs.  As a chunk of 64 tokens of a sequence is one system, those of v, k, beta and g may reach the up to
 * 63 tokens before theirs in the chunk as well.  In a gradient each, and those of dout, may reach all tokens of the sequence
 * and head (dq and dk of the key head).  Other sequences and heads are not touched.
 */
typedef struct seq_delta_args {
  seq_tokens_t tokens;
  int64_t heads, key_heads;
  int32_t key_dim, value_dim;
  int32_t dtype;
  float scale;
  seq_view_t q, k, v;
  int64_t q_head, k_head, v_head;
  seq_view_t g, beta;
  const float* state;
  int64_t state_stride;
  float* state_out;
  int64_t state_out_stride;
  float* save;
  seq_view_t o;
} seq_delta_args_t;

conv_wgrad_status_t seq_gated_delta_save(const seq_delta_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_gated_delta_workspace(const seq_delta_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_gated_delta(const seq_delta_args_t* args, void* workspace, size_t ws_bytes, void* stream);

/* The same for one token of each sequence (tokens.offsets NULL, tokens.rows 1); save is not written. */
conv_wgrad_status_t seq_gated_delta_step(const seq_delta_args_t* args, void* stream);

/* Gradients, from dout (strided as v, dout_head elements between heads), dstate_out (dense fp32 [sequences][heads]
 * [key_dim][value_dim], gradient of the final states, NULL: zero) and fwd.save as the forward filled it.  Outputs dense:
 * dq, dk rows x key_heads x key_dim, dv rows x heads x value_dim, dg and dbeta fp32 rows x heads, dstate fp32 [sequences]
 * [heads][key_dim][value_dim] or NULL.  fwd.o, fwd.state and fwd.state_out are not read. */
typedef struct seq_delta_grad_args {
  seq_delta_args_t fwd;
  seq_view_t dout;
  int64_t dout_head;
  const float* dstate_out;
  void* dq;
  void* dk;
  void* dv;
  float* dg;
  float* dbeta;
  float* dstate;
} seq_delta_grad_args_t;

conv_wgrad_status_t seq_gated_delta_grad_workspace(const seq_delta_grad_args_t* args, size_t* bytes);
conv_wgrad_status_t seq_gated_delta_grad(const seq_delta_grad_args_t* args, void* workspace, size_t ws_bytes,
                                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONV_WGRAD_H_ */
