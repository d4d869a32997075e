/*
 * adamw_matrix.h -- C ABI of the matrix operators of a training step, on the
 * tensor cores: orthogonalising matrices by Newton-Schulz products, the Muon
 * step built on it, and products grouped by expert with their gradients.
 *
 * Conventions, as in adamw_losses.h: every entry point is asynchronous on the
 * given stream of the current device unless stated, returns one of the
 * ADAMW_* status codes, and launches nothing when it returns an error that its
 * arguments caused.  Buffers belong to the caller and are not kept.  Pointers
 * are not looked up by the calls without a plan: they must be dereferenceable
 * by the current device.  Two calls may run at the same time when they share
 * no output and no workspace.  Whether two arguments overlap goes by their outer
 * ends.
 *
 * Values: products are summed in fp32 and rounded once, to nearest even, when
 * they are stored (what orthogonalisation keeps between its products is said
 * there).
 */
#ifndef ADAMW_MATRIX_H
#define ADAMW_MATRIX_H

#include "adamw_losses.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A batch of matrices: element (b, r, c) is at b * batch_stride + r *
 * row_stride + c of `data`, in elements; a row's elements are consecutive.
 * Strides are not negative; of what is read they may be 0 (one matrix for all of
 * a batch); of what is written no two elements share a place (matrices one after the
 * other, or their rows by turns).  Sizes up to what each call says, offsets 64-bit. */
typedef struct {
    void* data;
    int64_t batch;
    int64_t rows;
    int64_t cols;
    int64_t batch_stride;
    int64_t row_stride;
    int32_t dtype; /* ADAMW_DTYPE_* */
    int32_t pad_;
} adamw_matrices_t;

/* The Newton-Schulz iteration. */
typedef struct {
    int32_t steps;             /* 1 to 32                                        */
    int32_t n_coefficients;    /* 1 to 32: step k takes row min(k, n - 1)        */
    const float* coefficients; /* host, [n_coefficients][3]: a, b, c             */
    float eps;                 /* > 0                                            */
} adamw_ortho_t;

/* dst = the orthogonalised src, matrix by matrix:
 *     X <- src / max(|src|_F, eps)
 *     steps times:  G = X X^T,  X <- a X + (b G + c G G) X
 * (G = X^T X and the products from the right where rows > cols, which is the
 * same polynomial of smaller matrices).  With the coefficients of the Muon
 * optimizer (3.4445, -4.775, 2.0315) five steps bring every singular value
 * above 2e-3 of the norm to between 0.68 and 1.21.
 * Precision: G and b G + c G G are rounded to fp16 (2^12 times their values),
 * X is kept as a sum of two fp16 numbers, of which the products take the
 * first (both, and two of b G + c G G, where the smaller side is at most 128; all of
 * them, and two of G, where it is at most 32).
 * What is rounded away of a product's operand cannot reach directions of small
 * singular values, where each step multiplies errors by a; what is kept of X
 * itself could, and has 22 bits, but where the steps left multiply errors by 16 or
 * less (then 11).  After five steps of the usual coefficients, results are off the
 * iteration in exact arithmetic, before their rounding to dst's type and in the 2-norm,
 * by 9e-5 at most for smaller sides of up to 32; by 5e-4 to 1.5e-3 above (2.5e-3 where
 * seven eighths of the singular values are 0), 3.3e-3 at most of 205000 matrices of sides of 33 to
 * 2048 (random, scaled rows, low rank, singular values over four decades, sparse,
 * heavy-tailed).  That holds for five steps and fewer: these coefficients contract
 * nothing, and each step beyond multiplies errors by up to 1.8 (512 x 512: 1.3e-3 after
 * five, 3e-3 after eight, 2e-2 after 32).
 * Coefficients are the caller's: entries of X, G or b G + c G G above 16 overflow.
 * A zero matrix gives zeros; one with an inf or NaN gives NaN throughout.
 * src: bf16, fp16 or fp32; dst: any of the three, the same batch, rows and
 *   cols, matrices and rows not overlapping.  It may be src itself (the same
 *   data, type and strides) but must not overlap it otherwise.
 * workspace: adamw_orthogonalize_workspace(batch, rows, cols) bytes of device
 *   memory, 256-byte aligned, contents undefined before and after.
 * Errors: INVALID_ARG, MISALIGNED (workspace, or data not aligned to its
 * element), TOO_LARGE (rows or cols above 2^20, more than 2^40 elements or
 * 2^20 matrices), CUDA. */
int adamw_orthogonalize(const adamw_matrices_t* src, const adamw_matrices_t* dst,
                        const adamw_ortho_t* ortho, void* workspace, adamw_stream_t stream);
/* Bytes of workspace, 0 for sizes that the call refuses (and for no elements). */
int64_t adamw_orthogonalize_workspace(int64_t batch, int64_t rows, int64_t cols);

/* A parameter of a Muon plan: `batch` matrices of rows x cols, contiguous, in
 * each of four buffers. */
typedef struct {
    void* param;      /* bf16, written                    */
    const void* grad; /* bf16, read                       */
    void* momentum;   /* fp32 or bf16, read and written   */
    float* master;    /* fp32, read and written           */
    int64_t batch;
    int64_t rows;
    int64_t cols;
} adamw_muon_tensor_t;

/* How the update is scaled. */
#define ADAMW_MUON_SPECTRAL 0 /* sqrt(max(1, rows / cols))   */
#define ADAMW_MUON_RMS 1      /* 0.2 sqrt(max(rows, cols)): the size of an AdamW update */

typedef struct {
    adamw_ortho_t ortho;
    int32_t nesterov;       /* 0 or 1                             */
    int32_t scale;          /* ADAMW_MUON_*                       */
    int32_t momentum_dtype; /* ADAMW_DTYPE_FP32 or _BF16          */
} adamw_muon_options_t;

/* Read by the step on the device. */
typedef struct {
    float lr;
    float momentum;
    float weight_decay;
    float pad_;
} adamw_muon_hparams_t;

typedef struct adamw_muon_plan* adamw_muon_plan_t;

/* Builds a plan over a list of parameters on the current device: checks the
 * list, uploads its table and allocates the workspace (about 6 bytes an
 * element, at most about 2 GB at a time).  Synchronous.  Used from one host
 * thread at a time; steps of one plan must not overlap on the GPU.
 * Errors: INVALID_ARG (NULLs, negative sizes, bad options, buffers of the list
 * that overlap), MISALIGNED, NOT_ACCESSIBLE, TOO_LARGE, CUDA. */
int adamw_muon_plan_create(const adamw_muon_tensor_t* host_table, int32_t n,
                           const adamw_muon_options_t* options, adamw_muon_plan_t* out);

/* One step:
 *     M <- M + (1 - momentum) (G - M)
 *     U  = nesterov ? G + momentum (M - G) : M        (before M is rounded)
 *     W <- W (1 - lr weight_decay) - lr scale orthogonalize(U)
 *     param = W rounded
 * hparams: device adamw_muon_hparams_t, 16-byte aligned, so that a captured
 *   step takes other values later.
 * nonfinite: device int32: 1 when a gradient or momentum of the list is inf or
 *   NaN (or their norm beyond fp64); then nothing else is written.  2 added when a
 *   kernel's bounded wait ran out (adamw_matrix_status says so too): momenta,
 *   masters and parameters are then undefined.  0 otherwise.
 * No host synchronisation; sums run in a fixed order.
 * Errors: INVALID_ARG, MISALIGNED, CUDA. */
int adamw_muon_step(adamw_muon_plan_t plan, const adamw_muon_hparams_t* hparams,
                    int32_t* nonfinite, adamw_stream_t stream);

/* Releases the plan's device memory (synchronises its device first).  NULL is
 * accepted. */
int adamw_muon_plan_destroy(adamw_muon_plan_t plan);

/* Products grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 of x belong
 * to expert e, whose matrix is w[e].
 *     y[r] = w[e] x[r]        (w: experts x (y's cols) x (x's cols))
 *     y[r] = w[e]^T x[r]      (transposed: experts x (x's cols) x (y's cols))
 * The second, on the gradient of y and with w as it is, is the gradient of x.
 * x: one matrix (batch 1), bf16 or fp16.  w: the same type, batch = experts.
 * y: one matrix of x's rows, bf16, fp16 or fp32.  Rows of no expert (before
 *   offsets[0], from offsets[experts] on) are zeros in y whatever x holds.
 * offsets: device int64 [experts + 1], ascending within [0, rows].  Offsets
 *   outside that range are taken to its ends, one below its predecessor to the
 *   predecessor.
 * y must not overlap x or w.  Up to ADAMW_EXPERT_STREAM_ROWS rows, with transposed = 0
 *   and y of fewer than 2^24 columns, the weights are streamed once, at any alignment, and
 *   no workspace is needed, whatever adamw_expert_workspace says.
 * workspace: adamw_expert_workspace(x, w) bytes of device memory, 256-byte
 *   aligned; 0 where data are 16-byte aligned, rows do not overlap and strides are
 *   multiples of 8 (others are copied there first).
 * Errors: INVALID_ARG, MISALIGNED, TOO_LARGE (more than 1024 experts, rows or
 * cols above 2^30), CUDA. */
#define ADAMW_EXPERT_STREAM_ROWS 16
int adamw_expert_rows(const adamw_matrices_t* x, const adamw_matrices_t* w, int32_t transposed,
                      const int64_t* offsets, const adamw_matrices_t* y, void* workspace,
                      adamw_stream_t stream);

/* The gradient of w:
 *     dw[e] = sum over rows r of expert e of dy[r] x[r]^T     (accumulate: added)
 * dy, x: one matrix each (batch 1) of the same rows and type, bf16 or fp16.
 * dw: batch = experts, dy's cols x x's cols (or, exchanged, the caller
 *   exchanges dy and x); bf16, fp16 or fp32.  An expert without rows gets
 *   zeros (nothing with accumulate).  Sums run in a fixed order.
 * workspace: adamw_expert_workspace(dy, x) bytes.
 * Errors: as above. */
int adamw_expert_outer(const adamw_matrices_t* dy, const adamw_matrices_t* x,
                       const int64_t* offsets, const adamw_matrices_t* dw, int32_t accumulate,
                       void* workspace, adamw_stream_t stream);
int64_t adamw_expert_workspace(const adamw_matrices_t* a, const adamw_matrices_t* b);

/* Both gradients of y[r] = w[e] x[r] (w[e]^T x[r] where transposed) in one call:
 *   dx: as adamw_expert_rows makes it of dy with the other `transposed`, or NULL
 *   dw: as adamw_expert_outer makes it of dy and x (dw_transposed: of x and dy,
 *       experts x (x's cols) x (dy's cols)), or NULL
 * Each is what its own call gives. workspace: adamw_expert_backward_workspace
 * bytes. dx overlaps none of the others, nor does dw. Errors: as above. */
int adamw_expert_backward(const adamw_matrices_t* dy, const adamw_matrices_t* x, const adamw_matrices_t* w,
                          int32_t transposed, const int64_t* offsets, const adamw_matrices_t* dx,
                          const adamw_matrices_t* dw, int32_t dw_transposed, int32_t accumulate, void* workspace,
                          adamw_stream_t stream);
int64_t adamw_expert_backward_workspace(const adamw_matrices_t* dy, const adamw_matrices_t* x, const adamw_matrices_t* w);

/* Reads and clears the current device's status word of these operators: 1 when
 * a kernel's bounded wait ran out (its results are then undefined).
 * Synchronises the device. */
int adamw_matrix_status(int32_t* out);

/* For tests: while on, the kernels of adamw_orthogonalize and adamw_muon_step
 * that this process launches report a wait that ran out, though none did. */
void adamw_matrix_test_expire(int32_t on);

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_MATRIX_H */
