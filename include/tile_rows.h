/*
 * tile_rows.h -- C ABI of the fused FP32 row-normalisation library for
 * NVIDIA GB300 (sm_103a).
 *
 * Four operations, each applied independently to every row of a row-major
 * FP32 matrix [rows][width] (row i starts at element i*width):
 *
 *   residual LayerNorm  y = (c - mean(c)) / sqrt(var(c) + eps),  c = x + r
 *   LayerNorm           y = (x - mean(x)) / sqrt(var(x) + eps)
 *   RMSNorm             y = x / sqrt(mean(x^2) + eps)
 *   softmax             y = exp(x - max(x)) / sum(exp(x - max(x)))
 *
 * var is the centred, biased variance (divided by width); there are no
 * affine weights.  The definitions follow the notes "Residual LayerNorm
 * shared-Tile materialization search" (section "Structural finding": the
 * residual LayerNorm expression, eps = 1e-5 inside the square root) and
 * "Immutable input reuse in Metal reductions" (softmax, RMSNorm and
 * LayerNorm rows; each input element read once and kept in worker-private
 * stripes across the reduction phases).  Several rows may be packed into one
 * CTA as cooperating programs, as in "Cooperating-program packing",
 * section "Implementation boundary".
 *
 * Common contract of the four compute entry points
 * ------------------------------------------------
 *  - Pointers are DEVICE pointers (or managed/host-mapped memory the device
 *    can read), FP32, 4-byte aligned.  16-byte alignment is not required:
 *    rows whose start is not 16-byte aligned take a scalar head and tail.
 *  - The caller owns every buffer.  The library allocates nothing, writes
 *    exactly rows*width elements of `out` and nothing else, and never writes
 *    `in` or `residual`.
 *  - `out` must not overlap `in` or `residual` (the caller guarantees
 *    no aliasing; an overlap that the library can see from the address
 *    ranges is rejected with TILE_ERR_ALIAS).  `in` and `residual` may
 *    overlap each other.
 *  - Work is enqueued on `stream` (0 = the legacy default stream); the call
 *    returns without synchronising.  Results are bitwise reproducible for a
 *    given (op, rows, width, pointer alignment) on the same GPU.
 *  - rows == 0 is a no-op returning TILE_OK.  1 <= width <= tile_max_width().
 *  - Return value: TILE_OK (0) or a negative TILE_ERR_* code; on error
 *    nothing is launched, except TILE_ERR_CUDA, which reports the launch
 *    error returned by the CUDA runtime.
 */
#ifndef TILE_ROWS_H
#define TILE_ROWS_H

#include <stddef.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define TILE_OK               0
#define TILE_ERR_NULL        -1  /* a required pointer is NULL (rows > 0)       */
#define TILE_ERR_SHAPE       -2  /* rows < 0, width < 1 or width > max width   */
#define TILE_ERR_ALIAS       -3  /* out overlaps in or residual               */
#define TILE_ERR_EPS         -4  /* eps negative or not finite (normalisers)  */
#define TILE_ERR_CUDA        -5  /* the CUDA runtime reported a launch error  */
#define TILE_ERR_OP          -6  /* unknown operation code                    */
#define TILE_ERR_ALIGN       -7  /* a pointer is not 4-byte aligned           */
#define TILE_ERR_PLAN        -8  /* an explicit plan is not one of the built  */
#define TILE_ERR_DEVICE      -9  /* a kernel recorded an error on the device  */
#define TILE_ERR_WORKSPACE  -10  /* device workspace too small for one row    */
#define TILE_ERR_DTYPE      -11  /* unknown element type code                 */

/* ---- element types of row data (tile_row_args_t, tile_*_ex) ------------ */
#define TILE_DTYPE_F32  0   /* IEEE binary32                                  */
#define TILE_DTYPE_BF16 1   /* bfloat16: the high 16 bits of a binary32       */
#define TILE_DTYPE_F16  2   /* IEEE binary16                                  */

/* ---- operation codes (tile_describe_plan, tile_run_plan_*) ------------- */
#define TILE_OP_RESIDUAL_LAYERNORM 0
#define TILE_OP_LAYERNORM          1
#define TILE_OP_RMSNORM            2
#define TILE_OP_SOFTMAX            3
#define TILE_OP_ROW_SUM            4
#define TILE_OP_ROW_MINMAX         5
#define TILE_OP_LAYERNORM_AFFINE   6
#define TILE_OP_RMSNORM_WEIGHTED   7

/* ---- launch paths ------------------------------------------------------ */
#define TILE_PATH_CTA      0  /* P programs x S warps per CTA, one row each  */
#define TILE_PATH_CLUSTER  1  /* one row split over a cluster of C CTAs,     */
                              /* partials exchanged through DSMEM            */
#define TILE_PATH_STAGED   2  /* persistent CTAs; whole rows copied into a   */
                              /* ring of shared-memory stages by the bulk-   */
                              /* copy engine (mbarrier completion), several  */
                              /* rows in flight per CTA; 16-byte aligned     */
                              /* rows of whole vectors; normalisers, softmax */
#define TILE_PATH_ROWS     3  /* one CTA normalises R rows, each thread      */
                              /* owning the same columns of all R (one       */
                              /* reduction round and one gamma/beta load     */
                              /* serve R rows); 16-byte aligned rows of      */
                              /* whole vectors; normalisers, softmax;        */
                              /* programs_per_cta reports R                  */

/*
 * A launch plan: how rows map onto the GPU.  Worker w of program p in a CTA
 * owns the row elements e = (chunk * W * C + rank * W + w) * V + v of its
 * row (chunk < K, v < V; rank = CTA rank in the cluster), keeps them in
 * registers across every reduction phase, and reduces with warp shuffles,
 * then P*S shared partials, then (C > 1) the C CTA partials of the cluster.
 */
typedef struct tile_plan {
    int op;                 /* TILE_OP_*                                      */
    int rows, width;        /* the shape the plan was made for                */
    int id;                 /* index in the built plan table                  */
    int path;               /* TILE_PATH_*                                    */
    int vec;                /* elements per access: a 16-byte vector (4 FP32  */
                            /* or 8 BF16/FP16, + scalar head/tail), or 1      */
    int warps_per_program;  /* S                                              */
    int programs_per_cta;   /* P                                              */
    int chunks;             /* K: V-vectors per worker                        */
    int cluster;            /* C: CTAs per row (1 = no cluster)               */
    int threads;            /* T = 32 * S * P                                 */
    int workers;            /* W = 32 * S                                     */
    int stripe_floats;      /* K * vec FP32 registers of row data per thread  */
    int max_width;          /* widest row this plan covers                    */
    int smem_bytes;         /* static shared memory per CTA                   */
    int barriers_per_row;   /* CTA or cluster barriers on a row's path        */
    long long grid;         /* CTAs launched for `rows` (0 for staged plans:  */
                            /* persistent, min(rows, SMs x resident CTAs))    */
    int dtype;              /* TILE_DTYPE_* the plan was described for        */
} tile_plan_t;

/* ---- compute entry points --------------------------------------------- */

/* Residual LayerNorm, no affine: c = in + residual, then LayerNorm of c.
 * "Residual LayerNorm shared-Tile materialization search", "Structural
 * finding".  in, residual, out: [rows][width] FP32 on the device. */
int tile_residual_layernorm_f32(const float *in, const float *residual, float *out,
                                int rows, int width, float eps, cudaStream_t stream);

/* LayerNorm, no affine.  "Cooperating-program packing", "Validation"
 * (no-affine LayerNorm); "Immutable input reuse in Metal reductions". */
int tile_layernorm_f32(const float *in, float *out, int rows, int width, float eps,
                       cudaStream_t stream);

/* RMSNorm, no weight: y = x / sqrt(mean(x^2) + eps).  Named in "Immutable
 * input reuse in Metal reductions" (fixed-width results table). */
int tile_rmsnorm_f32(const float *in, float *out, int rows, int width, float eps,
                     cudaStream_t stream);

/* softmax over each row with the row maximum subtracted first (the max
 * collective of "Cooperating-program packing", "Implementation boundary").
 * `eps` is accepted for a uniform signature and ignored. */
int tile_softmax_f32(const float *in, float *out, int rows, int width, float eps,
                     cudaStream_t stream);

/* ---- more row operations ---------------------------------------------- */

/* Affine LayerNorm: y = LayerNorm(in [+ residual]) * gamma + beta.  The
 * pages list affine LayerNorm (tolerance atol 1e-5) in "Cooperating-program
 * packing", "Predeclared comparison and measurement"; the formula is the
 * LayerNorm above followed by the per-column scale and shift.  residual and
 * beta may be NULL; gamma, beta: [width] FP32 device vectors (read through
 * the read-only cache; any 4-byte alignment).  Same contract otherwise. */
int tile_layernorm_affine_f32(const float *in, const float *residual, const float *gamma,
                              const float *beta, float *out, int rows, int width, float eps,
                              cudaStream_t stream);

/* Weighted RMSNorm: y = in / sqrt(mean(in^2) + eps) * gamma, gamma [width]. */
int tile_rmsnorm_weighted_f32(const float *in, const float *gamma, float *out, int rows,
                              int width, float eps, cudaStream_t stream);

/* Row sums: sums[i] = sum_j in[i][j], sums: [rows] FP32 on the device.  The
 * "sum" operator of "Cooperating-program packing", "Validation".  Each
 * thread and every reduction level keeps a compensated (TwoSum) pair, so the
 * result is close to the correctly rounded sum even when terms cancel. */
int tile_row_sum_f32(const float *in, float *sums, int rows, int width, cudaStream_t stream);

/* Paired row min/max in one pass: mins[i] = min_j in[i][j], maxs[i] =
 * max_j in[i][j] (exact).  The "paired min/max" operator of
 * "Cooperating-program packing", "Validation".  Inputs must not be NaN. */
int tile_row_minmax_f32(const float *in, float *mins, float *maxs, int rows, int width,
                        cudaStream_t stream);

/* Operands of a row operation for tile_run_plan_args_f32.  Unused pointers
 * are ignored (set them NULL). */
typedef struct tile_row_args {
    const void *in;         /* [rows][width] of `dtype`                         */
    const void *residual;   /* residual LayerNorm; optional for affine LN       */
    const float *gamma;     /* affine LN / weighted RMSNorm: [width] FP32       */
    const float *beta;      /* affine LN: [width] FP32 or NULL                  */
    void *out;              /* [rows][width] of `dtype`, or [rows] FP32 sums /  */
                            /* minima                                            */
    float *out2;            /* [rows] FP32 maxima (TILE_OP_ROW_MINMAX)          */
    int rows, width;
    float eps;              /* normalisers only                                  */
    int dtype;              /* TILE_DTYPE_F32, TILE_DTYPE_BF16 or TILE_DTYPE_F16 */
} tile_row_args_t;

/* Any row operation with the built plan `plan_id` forced (plan sweeps,
 * per-plan tests).  Errors as tile_run_plan_f32. */
int tile_run_plan_args_f32(int op, int plan_id, const tile_row_args_t *args, cudaStream_t stream);

/* ---- BF16 rows ----------------------------------------------------------
 * The row operations on BF16 data (2 bytes per element; the pages cover FP32
 * only and name low precision as not covered, "Residual LayerNorm
 * shared-Tile materialization search", "Exact command").  Each element is
 * widened exactly to FP32, every reduction and map runs in FP32 as for the
 * FP32 entry points (except that the row statistics multiply by 1/width
 * and take rsqrtf, at most 2 ulp, where the FP32 rows divide and take a
 * correctly rounded 1/sqrt: a few FP32 ulp, far inside half a BF16 ulp),
 * and outputs are rounded to nearest-even BF16.  gamma,
 * beta and the row outputs of sum and min/max stay FP32.  Pointers to BF16
 * data must be 2-byte aligned; 16-byte vectors (8 elements) are used when
 * in, residual and out share a 16-byte phase.  Everything else is the
 * contract of the FP32 entry point of the same name. */
int tile_residual_layernorm_bf16(const void *in, const void *residual, void *out, int rows,
                                 int width, float eps, cudaStream_t stream);
int tile_layernorm_bf16(const void *in, void *out, int rows, int width, float eps,
                        cudaStream_t stream);
int tile_rmsnorm_bf16(const void *in, void *out, int rows, int width, float eps,
                      cudaStream_t stream);
int tile_softmax_bf16(const void *in, void *out, int rows, int width, float eps,
                      cudaStream_t stream);
int tile_layernorm_affine_bf16(const void *in, const void *residual, const float *gamma,
                               const float *beta, void *out, int rows, int width, float eps,
                               cudaStream_t stream);
int tile_rmsnorm_weighted_bf16(const void *in, const float *gamma, void *out, int rows,
                               int width, float eps, cudaStream_t stream);
int tile_row_sum_bf16(const void *in, float *sums, int rows, int width, cudaStream_t stream);
int tile_row_minmax_bf16(const void *in, float *mins, float *maxs, int rows, int width,
                         cudaStream_t stream);

/* ---- FP16 rows ----------------------------------------------------------
 * The same row operations on IEEE binary16 data (the "FP16 I/O" of low
 * precision the pages name as not covered, same section as above): each
 * element is widened exactly to FP32, every reduction and map runs in FP32
 * (row statistics as for BF16 rows), outputs are rounded to nearest-even
 * binary16 (an output beyond 65504
 * becomes +-inf, as a binary16 rounding does; normalised rows stay far below
 * it).  Layout, alignment, vectors, plans and errors as the BF16 entry
 * points; gamma, beta and the row outputs of sum and min/max stay FP32. */
int tile_residual_layernorm_f16(const void *in, const void *residual, void *out, int rows,
                                int width, float eps, cudaStream_t stream);
int tile_layernorm_f16(const void *in, void *out, int rows, int width, float eps,
                       cudaStream_t stream);
int tile_rmsnorm_f16(const void *in, void *out, int rows, int width, float eps,
                     cudaStream_t stream);
int tile_softmax_f16(const void *in, void *out, int rows, int width, float eps,
                     cudaStream_t stream);
int tile_layernorm_affine_f16(const void *in, const void *residual, const float *gamma,
                              const float *beta, void *out, int rows, int width, float eps,
                              cudaStream_t stream);
int tile_rmsnorm_weighted_f16(const void *in, const float *gamma, void *out, int rows,
                              int width, float eps, cudaStream_t stream);
int tile_row_sum_f16(const void *in, float *sums, int rows, int width, cudaStream_t stream);
int tile_row_minmax_f16(const void *in, float *mins, float *maxs, int rows, int width,
                        cudaStream_t stream);

/* ---- backward passes ---------------------------------------------------
 * Input gradients of LayerNorm, RMSNorm and softmax, FP32.  The pages do
 * not cover backward normalisation ("Residual LayerNorm shared-Tile
 * materialization search", last paragraph); these are the chain rule of the
 * forward maps above:
 *   LayerNorm  dx = rstd (g - mean(g) - xhat mean(g xhat)),  xhat = (x - mean) rstd
 *   RMSNorm    dx = rstd (g - xhat mean(g xhat)),            xhat = x rstd
 *   softmax    dx = y (dy - sum(dy y))
 * with g = dy * gamma (gamma = 1 when NULL).  `in` is the forward input
 * (x, or x + residual for residual LayerNorm); the statistics are recomputed
 * from it exactly as the forward kernels compute them.  Each row of in and
 * dy is read once into registers, dx written once.  If row_stats is not
 * NULL, (mean, rstd) of every row is written to row_stats[2*i], [2*i+1]
 * (mean 0 for RMSNorm) for tile_norm_param_grad_f32.  dx and row_stats must
 * not overlap any input.  Other rules as the forward entry points. */
int tile_layernorm_backward_f32(const float *in, const float *gamma, const float *dy, float *dx,
                                float *row_stats, int rows, int width, float eps,
                                cudaStream_t stream);
int tile_rmsnorm_backward_f32(const float *in, const float *gamma, const float *dy, float *dx,
                              float *row_stats, int rows, int width, float eps,
                              cudaStream_t stream);
/* y: the forward softmax output. */
int tile_softmax_backward_f32(const float *y, const float *dy, float *dx, int rows, int width,
                              cudaStream_t stream);

/* A backward call with the built plan `plan_id` forced (op: TILE_OP_LAYERNORM,
 * TILE_OP_RMSNORM or TILE_OP_SOFTMAX).  TILE_ERR_PLAN if the plan is not built
 * for backward (two stripes of at most 32 floats), cannot cover the width, or
 * needs co-aligned pointers. */
int tile_run_backward_plan_f32(int op, int plan_id, const float *in, const float *gamma,
                               const float *dy, float *dx, float *row_stats, int rows, int width,
                               float eps, cudaStream_t stream);

/* Parameter gradients, summed over rows:
 *   dgamma[j] = sum_i dy[i][j] (in[i][j] - mean_i) rstd_i,  dbeta[j] = sum_i dy[i][j]
 * from the row statistics a backward call wrote (RMSNorm: mean 0, pass
 * dbeta = NULL).  Deterministic: rows are split into fixed blocks whose
 * column partials (compensated sums) go to the caller's device `workspace`
 * of at least tile_norm_param_grad_workspace_bytes(rows, width) bytes,
 * then are summed in block order.  rows == 0 writes zeros. */
size_t tile_norm_param_grad_workspace_bytes(int rows, int width);
int tile_norm_param_grad_f32(const float *in, const float *dy, const float *row_stats,
                             float *dgamma, float *dbeta, int rows, int width, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/* The backward passes with BF16 or FP16 in / y, dy and dx (2 bytes per
 * element, 2-byte aligned): every element is widened exactly to FP32, the
 * statistics, sums and maps run in FP32 as above (row statistics as for the
 * 2-byte forward rows), and dx is rounded to
 * nearest-even of its type.  gamma, row_stats, dgamma, dbeta and the
 * workspace stay FP32; tile_norm_param_grad_* uses the same workspace size.
 * 16-byte vectors (8 elements) are used when in, dy and dx share a 16-byte
 * phase.  Everything else is the contract of the FP32 entry point. */
int tile_layernorm_backward_bf16(const void *in, const float *gamma, const void *dy, void *dx,
                                 float *row_stats, int rows, int width, float eps,
                                 cudaStream_t stream);
int tile_rmsnorm_backward_bf16(const void *in, const float *gamma, const void *dy, void *dx,
                               float *row_stats, int rows, int width, float eps,
                               cudaStream_t stream);
int tile_softmax_backward_bf16(const void *y, const void *dy, void *dx, int rows, int width,
                               cudaStream_t stream);
int tile_norm_param_grad_bf16(const void *in, const void *dy, const float *row_stats,
                              float *dgamma, float *dbeta, int rows, int width, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream);
int tile_layernorm_backward_f16(const void *in, const float *gamma, const void *dy, void *dx,
                                float *row_stats, int rows, int width, float eps,
                                cudaStream_t stream);
int tile_rmsnorm_backward_f16(const void *in, const float *gamma, const void *dy, void *dx,
                              float *row_stats, int rows, int width, float eps,
                              cudaStream_t stream);
int tile_softmax_backward_f16(const void *y, const void *dy, void *dx, int rows, int width,
                              cudaStream_t stream);
int tile_norm_param_grad_f16(const void *in, const void *dy, const float *row_stats,
                             float *dgamma, float *dbeta, int rows, int width, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/* tile_run_backward_plan_f32 for an element type (TILE_DTYPE_*; in, dy, dx
 * of that type).  For BF16 / FP16, plans whose stripes would pass 32 floats
 * (K above 4 with 16-byte vectors) return TILE_ERR_PLAN; an unknown type
 * TILE_ERR_DTYPE. */
int tile_run_backward_plan_ex(int op, int plan_id, int dtype, const void *in, const float *gamma,
                              const void *dy, void *dx, float *row_stats, int rows, int width,
                              float eps, cudaStream_t stream);

/* The plan the backward entry points launch for (op, dtype, rows, width)
 * with 16-byte co-aligned in, dy and dx (op: TILE_OP_LAYERNORM,
 * TILE_OP_RMSNORM or TILE_OP_SOFTMAX; the choice depends on the width, not
 * on the rows).  Host only; touches no GPU.  Returns TILE_OK, TILE_ERR_OP,
 * TILE_ERR_DTYPE, TILE_ERR_SHAPE or TILE_ERR_NULL; `plan` is written on
 * success only. */
int tile_describe_backward_plan(int op, int dtype, int rows, int width, tile_plan_t *plan);

/* ---- block norm ---------------------------------------------------------
 * The norms around one block of a residual network, fused with the block's
 * gate and the scaled residual sum.  For every row, with
 * norm(v; gamma) = v / sqrt(mean(v^2) + eps) * gamma (RMSNorm):
 *
 *   n      = norm(in; gamma_post)          with TILE_NORM_POST, else n = in
 *   hidden = residual_scale * residual + gate * n
 *   out    = norm(hidden; gamma_pre)       with TILE_NORM_PRE
 *
 * in: the block's output; residual: the residual stream the block read;
 * hidden: the residual stream after it; out: the next block's input.  (The
 * notes this library follows have no counterpart.)  out is computed from the
 * unrounded hidden row and rounded once; hidden is rounded once.
 *
 * Rows are [rows][width] of `dtype`, contiguous; gammas [width] FP32, NULL
 * for ones; gate [ceil(rows / rows_per_gate)][width] FP32, NULL for ones:
 * row i takes gate row i / rows_per_gate (rows_per_gate >= rows: one learned
 * gate per channel; the tokens of a sequence: a gate per sequence; 1: a
 * gate per element).  rows_per_gate is ignored without a gate.  Any
 * alignment of the element type works; rows whose pointers are all 16-byte
 * aligned and whose width is a multiple of 16 bytes take vector accesses.
 * No output may overlap an input or another output.  Everything is FP32
 * inside, and results are bitwise reproducible for a given (shape, dtype,
 * alignment) on the same GPU.  Captured into CUDA graphs as any launch. */
#define TILE_NORM_POST 1   /* norm after the block                           */
#define TILE_NORM_PRE  2   /* norm before the next block                     */

typedef struct tile_block_norm_args {
    const void *in;            /* [rows][width]                              */
    const void *residual;      /* [rows][width]                              */
    const float *gamma_post;   /* TILE_NORM_POST: [width] or NULL            */
    const float *gate;         /* [ceil(rows / rows_per_gate)][width] or NULL */
    const float *gamma_pre;    /* TILE_NORM_PRE: [width] or NULL             */
    void *hidden;              /* [rows][width], written                     */
    void *out;                 /* TILE_NORM_PRE: [rows][width], written      */
    int rows, width;           /* 1 <= width <= tile_max_width()             */
    int rows_per_gate;         /* >= 1 with a gate                           */
    int norms;                 /* TILE_NORM_POST | TILE_NORM_PRE, at least one */
    float residual_scale;      /* finite                                     */
    float eps;
    int dtype;                 /* TILE_DTYPE_*                               */
} tile_block_norm_args_t;

/* Errors as the row entry points; TILE_ERR_OP for norms that are not a
 * non-empty set of the two bits; TILE_ERR_SHAPE also for rows_per_gate < 1
 * with a gate; TILE_ERR_EPS also for a residual_scale that is not finite. */
int tile_block_norm(const tile_block_norm_args_t *args, cudaStream_t stream);

/* Gradients of a block norm.  dhidden, dout: the gradients of hidden and
 * out; dhidden may be NULL (no use of hidden but out), dout is read with
 * TILE_NORM_PRE only.  in is the forward `in`, hidden the forward's rounded
 * `hidden`, whose statistics are taken again from it.  Writes
 *
 *   din, dresidual          [rows][width] of dtype
 *   dgamma_post, dgamma_pre [width] FP32 (NULL: not wanted)
 *   dgate                   the gate's shape, FP32 (NULL: not wanted)
 *
 * Column sums are FP32 partial sums of contiguous row ranges in the caller's
 * device `workspace` (16-byte aligned), joined in a fixed order; no atomics.
 * `in` may be NULL without TILE_NORM_POST and gate; `hidden` and dout may
 * be NULL without TILE_NORM_PRE.  rows == 0 writes zero parameter
 * gradients.  A row's sums (of in^2, hidden^2 and gate gamma_post in hidden)
 * have to lie within FP32's range, as the forward's two do.  dgamma_post
 * needs TILE_NORM_POST, dgamma_pre TILE_NORM_PRE, dgate a gate (TILE_ERR_OP).
 * Calls that overlap in time need workspaces
 * of their own. */
typedef struct tile_block_norm_backward_args {
    const void *in, *hidden, *dhidden, *dout;
    const float *gamma_post, *gate, *gamma_pre;
    void *din, *dresidual;
    float *dgamma_post, *dgate, *dgamma_pre;
    int rows, width, rows_per_gate, norms;
    float residual_scale, eps;
    int dtype;
} tile_block_norm_backward_args_t;

/* Workspace: 16 width bytes for each program of a call, as many as run at once
 * (at most 40 MiB in all) and no more than rows; but for widths that are not
 * multiples of 8 at least 8 for each gate row, up to 1024 (2432 where width
 * <= 1024).  The first function has enough for any number of gate rows, the
 * second for this one (0: no gate), which is what a call checks. */
size_t tile_block_norm_backward_workspace_bytes(int rows, int width);
size_t tile_block_norm_backward_gated_workspace_bytes(int rows, int width, int gate_rows);
int tile_block_norm_backward(const tile_block_norm_backward_args_t *args, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream);

/* ---- linear cross entropy --------------------------------------------------
 * The loss at the end of a language model: a linear head over a vocabulary
 * and the softmax cross entropy of its logits, without keeping them.  For
 * every row i of `in` ([rows][width]), with the logits
 * l_v = sum_h in[i][h] weight[v][h], v < vocab:
 *
 *   lse[i]  = log(sum_v exp(l_v))
 *   loss[i] = lse[i] - l_target[i]
 *
 * Both FP32 [rows]; a row whose target is ignore_index gets loss = lse = 0.
 * The loss is log(1 + sum over the other entries of exp(l_v - l_target)) with
 * the target's logit as an FP32 sum, so it is never negative and small losses
 * keep their digits.  The other logits are sums of the tensor cores, in parts of
 * at most 4096 columns, which cut off low bits as they add: of random rows
 * about 2^-26 of a part for each 16 columns, which is put back; of products of
 * one sign up to 2^-23 of it (2e-5 of the logit at 4096 columns and beyond);
 * of sums that fit 24 bits, such as rows of few columns, nothing: there the
 * logit comes out up to 2^-18 of itself (3.8e-6) too large.
 * dtype: TILE_DTYPE_BF16 or TILE_DTYPE_F16 of in and weight ([vocab][width]);
 * the products of 16-bit elements are exact, and every sum is FP32.  (FP32
 * operands are refused with TILE_ERR_DTYPE: the tensor cores would round
 * them.)  target: [rows] 64-bit integers on the device.  A target that is
 * neither ignore_index nor in [0, vocab) gives that row a NaN loss, an lse
 * of 0, and sets the device status word (tile_check_device_status).
 *
 * `workspace`: device memory of the caller, 256-byte aligned, at least
 * tile_linear_cross_entropy_workspace_bytes(rows, width, vocab) bytes: four
 * numbers per row and tile of 192 to 256 vocabulary entries, for long calls
 * a copy of in (the rows that count), and, for widths that are not multiples
 * of 8, of weight, in rows of whole 128 bytes.  Calls that
 * overlap in time need workspaces of their own.  in and weight: 16-byte
 * aligned where width is a multiple of 8, else 2-byte (TILE_ERR_ALIGN).
 * Other rules and errors as the row entry points (TILE_ERR_SHAPE also for
 * vocab < 1, and rows or vocab above 2^30; rows == 0 is a no-op).  The call
 * may be captured into a CUDA graph. */
size_t tile_linear_cross_entropy_workspace_bytes(int rows, int width, int vocab);
int tile_linear_cross_entropy(int dtype, const void *in, const void *weight,
                              const long long *target, float *loss, float *lse, int rows,
                              int width, int vocab, long long ignore_index, void *workspace,
                              size_t workspace_bytes, cudaStream_t stream);

/* Its gradients: with g[i][v] = (exp(l_v - lse[i]) - [v = target[i]]) dloss[i],
 *
 *   din = g weight ([rows][width]),   dweight = g^T in ([vocab][width])
 *
 * of dtype, either may be NULL.  lse: the forward's.  dloss: [rows] FP32,
 * the gradient of each row's loss (1 / rows of a mean).  Rows whose target is
 * ignore_index or whose dloss is 0 get din = 0 and take no part in dweight,
 * whatever they hold; so do rows with a target out of range, which set the
 * device status word.
 *
 * g is made in pieces of the vocabulary (at most about 512 MiB of the
 * workspace, or 4096 columns; an FP32 din and a copy of in come to that) and
 * held in 16 bits for one piece: dtype
 * values of (p - onehot) dloss / max |dloss| rounded once, FP16 ones of 2^15
 * times that.  Sums are FP32, din and dweight rounded once.  No
 * atomics: results are bitwise reproducible.  rows == 0 writes a zero
 * dweight. */
size_t tile_linear_cross_entropy_backward_workspace_bytes(int rows, int width, int vocab);
int tile_linear_cross_entropy_backward(int dtype, const void *in, const void *weight,
                                       const long long *target, const float *lse,
                                       const float *dloss, void *din, void *dweight, int rows,
                                       int width, int vocab, long long ignore_index,
                                       void *workspace, size_t workspace_bytes,
                                       cudaStream_t stream);

/* ---- embedding ------------------------------------------------------------
 * The lookup at the start of a language model and its gradient; the weight is
 * often the linear head's too, whose gradient
 * tile_linear_cross_entropy_backward leaves.  (The notes this library follows
 * have no counterpart.)  For every row i,
 *
 *   out[i] = scale * weight[tokens[i]]
 *
 * out [rows][width] and weight [vocab][width] of `dtype`, contiguous; tokens
 * [rows] 64-bit integers on the device.  The product is FP32, rounded once.  A
 * token equal to ignore_index gives a row of zeros (whatever vocabulary entry
 * that might be); another one outside [0, vocab) a row of NaN, and sets the
 * device status word (tile_check_device_status).  Any alignment of the element
 * type works; 16-byte aligned rows of whole 16-byte vectors are the fastest.
 * rows == 0 is a no-op; rows up to 2^24, vocab up to 2^30 (TILE_ERR_SHAPE).
 * TILE_ERR_EPS for a scale that is not finite; other rules and errors as the
 * row entry points. */
int tile_embedding(int dtype, const long long *tokens, const void *weight, void *out, int rows,
                   int width, int vocab, float scale, long long ignore_index,
                   cudaStream_t stream);

/* Its gradient: dweight[v] = scale * (sum of dout[i] over the rows with
 * tokens[i] = v), of the whole [vocab][width] matrix (zero where v does not
 * occur), or, with accumulate != 0, that added to what dweight holds, rounded
 * once; rows of dweight whose token does not occur are then neither read nor
 * written.  dweight is of `dtype` or FP32 (TILE_ERR_DTYPE).  Rows whose token is
 * ignore_index or out of range (the status word) take no part, whatever they
 * hold.  Sums are FP32, over the positions in order in parts that depend on
 * the tokens alone: no atomics on values, results are bitwise reproducible.
 *
 * `workspace`: device memory of the caller, 256-byte aligned, at least
 * tile_embedding_backward_workspace_bytes(rows, width, vocab) bytes (0 for few
 * rows): the positions sorted by token, and partial sums of tokens that occur
 * often (64 MiB at most).  Calls that overlap in time need workspaces of their
 * own.  The sort's counts grow with the square of the rows: 2^20 rows of 64 BF16
 * columns take 0.2 ms, 2^24 3.6.  rows == 0 writes a zero
 * dweight, or nothing where it accumulates.  May be captured into a CUDA
 * graph. */
size_t tile_embedding_backward_workspace_bytes(int rows, int width, int vocab);
int tile_embedding_backward(int dtype, int dweight_dtype, const long long *tokens,
                            const void *dout, void *dweight, int rows, int width, int vocab,
                            float scale, long long ignore_index, int accumulate, void *workspace,
                            size_t workspace_bytes, cudaStream_t stream);

/* ---- policy loss ------------------------------------------------------------
 * The clipped loss that a policy is trained with on sampled sequences, with a
 * term that holds it near a reference, from the negative log probabilities
 * that tile_linear_cross_entropy returns as `loss`.  (The notes this library
 * follows have no counterpart.)  For every token, with r = exp(old_nll - nll)
 * and q = nll - ref_nll,
 *
 *   l = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *       + kl_coef (exp(q) - q - 1)
 *
 * where A is the token's advantage, or its sequence's with
 * TILE_POLICY_SEQUENCE_ADVANTAGE.  Writes
 *
 *   stats    [4] FP32: the mean of l, of its first term, of exp(q) - q - 1 and
 *            of whether the clip holds r A back
 *   weights  [sequences] FP32: the weight of each token of a sequence in the
 *            means, which the gradient takes
 *
 * The means are over all tokens that count, or, with
 * TILE_POLICY_SEQUENCE_MEAN, over the sequences with such tokens of the means
 * over them.  Where nothing counts, all are 0.
 *
 * Sequences lie one behind the other: sequence s is the rows from offsets[s] up
 * to offsets[s + 1] ([sequences + 1] 64-bit integers on the device that do not
 * fall; sequences may be empty).  Rows before the first and behind the last
 * one do not count, nor do rows whose target is ignore_index; what they hold
 * is not used.  Offsets that fall or leave [0, rows] set the device
 * status word and make stats NaN.  offsets NULL: one sequence of all rows
 * (sequences 1).  target NULL: every row counts.  ref_nll NULL: no such term
 * (kl_coef 0).  kl_coef 0 with a ref_nll: stats[2] alone looks at it, loss and
 * gradient are those without one.
 *
 * nll, old_nll, ref_nll [rows], advantage [rows] or [sequences]: FP32.  Whether r
 * is held back is decided from old_nll - nll as if it had not been rounded; r A
 * equal to its bound is not.  An advantage of 0 gives a first term of 0.
 * exp(q) - q - 1 is good to 14 roundings of 2^-24 of itself up to |q| = 3, however
 * small q is.  Sums are FP32 over 512 rows and compensated beyond, bitwise
 * reproducible; one CTA joins the sequences (16384 of 1048576 tokens: 58 us with
 * TILE_POLICY_SEQUENCE_MEAN, 19 without; 512: 14.6 and 9.8).  `workspace`: 16-byte
 * aligned device memory of the caller; calls that overlap in time need workspaces
 * of their own.  rows == 0 writes zeros.
 * TILE_ERR_EPS for clip_low outside [0, 1], a negative or NaN clip_high or a
 * kl_coef that is not finite; TILE_ERR_SHAPE for rows or sequences above 2^30,
 * sequences < 1, or other than 1 without offsets; TILE_ERR_OP for unknown flags;
 * other rules and errors as the row entry points.  May be captured into a CUDA
 * graph. */
#define TILE_POLICY_SEQUENCE_ADVANTAGE 1   /* advantage is [sequences]            */
#define TILE_POLICY_SEQUENCE_MEAN      2   /* the mean of the sequences' means    */

typedef struct tile_policy_loss_args {
    const float *nll, *old_nll;   /* [rows]                                       */
    const float *ref_nll;         /* [rows] or NULL                               */
    const float *advantage;       /* [rows], or [sequences]                       */
    const long long *target;      /* [rows] or NULL                               */
    const long long *offsets;     /* [sequences + 1] or NULL                      */
    long long ignore_index;
    int rows, sequences;
    int flags;                    /* TILE_POLICY_*                                */
    float clip_low, clip_high, kl_coef;
} tile_policy_loss_args_t;

size_t tile_policy_loss_workspace_bytes(int rows, int sequences);
int tile_policy_loss(const tile_policy_loss_args_t *args, float *stats, float *weights,
                     void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Its gradient for the forward's `weights` and the gradient dloss ([1] FP32 on
 * the device; NULL for 1) of stats[0]: dnll [rows] FP32,
 *
 *   dnll = dloss weight (r A, or 0 where the clip holds it back,
 *                        + kl_coef (exp(q) - 1))
 *
 * and 0 for rows that do not count: the dloss of
 * tile_linear_cross_entropy_backward.  args as the forward's
 * (TILE_POLICY_SEQUENCE_MEAN is in the weights and plays no part).  rows == 0
 * is a no-op. */
int tile_policy_loss_backward(const tile_policy_loss_args_t *args, const float *weights,
                              const float *dloss, float *dnll, cudaStream_t stream);

/* ---- gradient norm and AdamW step ---------------------------------------------
 * Over many tensors at once, in one launch for up to 1024 (norm) or 384 (step)
 * of them.  (The notes this library follows have no counterpart.)
 *
 * tile_grad_norm writes out [2] FP32:
 *
 *   out[0] = norm = scale * sqrt(sum over all tensors of g^2)
 *   out[1] = factor = scale * min(1, max_norm / norm)
 *
 * scale: what the gradients are to be multiplied by (the inverse of a loss
 * scale), finite and above 0; max_norm above 0, INFINITY for no clip
 * (TILE_ERR_EPS).  factor is NaN where the norm is not finite.  Squares are FP32
 * (magnitudes above 1.8e19 come out infinite, far below 1e-19 as nothing), sums
 * compensated FP32 and FP64: bitwise reproducible.  Tensors are contiguous and
 * of any size, 0 included, `data` aligned to the element; none: a norm of 0.
 * `workspace`: 16-byte aligned, tile_grad_norm_workspace_bytes(count) bytes;
 * calls that overlap in time need workspaces of their own. */
typedef struct tile_tensor {
    const void *data;
    long long n;               /* elements                                        */
    int dtype;                 /* TILE_DTYPE_*                                    */
} tile_tensor_t;

size_t tile_grad_norm_workspace_bytes(int count);
int tile_grad_norm(const tile_tensor_t *tensors, int count, float scale, float max_norm,
                   float *out, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* One AdamW step of every tensor, in place.  With g = factor * grad and the
 * step t,
 *
 *   exp_avg    = beta1 exp_avg + (1 - beta1) g
 *   exp_avg_sq = beta2 exp_avg_sq + (1 - beta2) g^2
 *   param      = (1 - lr weight_decay) param - lr / (1 - beta1^t) exp_avg
 *                / (sqrt(exp_avg_sq / (1 - beta2^t)) + eps)
 *   copy       = param rounded to copy_dtype, where wanted
 *
 * factor: [1] FP32 on the device (tile_grad_norm's out + 1), NULL for 1; where
 * it is not finite, nothing is changed.  step (>= 1) and lr may lie on the
 * device instead, so that a captured step can be replayed with others: NULL
 * takes the number given (a step below 1 on the device counts as 1).
 *
 * param is FP32 (an update is often less than half a 16-bit step of it); the 16-bit
 * weights that a model runs on are the copy.  TILE_STATE_F32: both states
 * [n] FP32.  TILE_STATE_E4M3: [n] bytes of e4m3 and FP32 scales
 * [ceil(n / 256)], a power of two for each 256 elements: exp_avg = code * scale,
 * exp_avg_sq = (code * scale)^2.  These are rounded up with the
 * probability of what is cut off (16 bits of SplitMix64's finalizer of seed,
 * step, the tensor's place in the list and the element): to nearest, exp_avg_sq
 * could not move by less than 6 %.  The same call gives the same bits.  A zero
 * state is zero codes with any finite scale.  A state of 256 elements one of which
 * is not finite becomes NaN.
 *
 * Everything else is FP32; exp_avg and exp_avg_sq are rounded after each product
 * and sum.  Pointers: aligned to their element; the 16-byte grid is the fastest,
 * and with FP32 states so are tensors that are off it by the same elements.  No
 * written range may overlap another range of the call (TILE_ERR_ALIAS): a tensor
 * is listed once.  n >= 0, no limit on count.  TILE_ERR_EPS for betas outside
 * [0, 1), eps that is not finite or below 2^-126 (one above 2^126 leaves decay
 * alone), an lr or weight_decay that is not finite; TILE_ERR_SHAPE for n < 0,
 * count < 0, step < 1; TILE_ERR_DTYPE for unknown types (copy_dtype: BF16 or F16);
 * other rules and errors as the row entry points.  May be captured into a CUDA
 * graph, which then holds the pointers. */
#define TILE_STATE_F32  0
#define TILE_STATE_E4M3 1

typedef struct tile_adamw_tensor {
    float *param;
    const void *grad;
    void *exp_avg, *exp_avg_sq;
    float *exp_avg_scale, *exp_avg_sq_scale;   /* TILE_STATE_E4M3                 */
    void *copy;                                /* or NULL                         */
    long long n;
    float weight_decay;
    int grad_dtype;                            /* TILE_DTYPE_*                    */
    int copy_dtype;                            /* with a copy                     */
} tile_adamw_tensor_t;

typedef struct tile_adamw_config {
    double lr, beta1, beta2, eps;
    long long step;
    const float *lr_device;          /* [1] or NULL                               */
    const long long *step_device;    /* [1] or NULL                               */
    const float *factor;             /* [1] or NULL                               */
    unsigned long long seed;         /* TILE_STATE_E4M3                           */
    int state;                       /* TILE_STATE_*                              */
} tile_adamw_config_t;

int tile_adamw(const tile_adamw_tensor_t *tensors, int count, const tile_adamw_config_t *config,
               cudaStream_t stream);

/* ---- pointwise value/derivative pairs ---------------------------------- */

/* value[k] = sigmoid(in[k]) and derivative[k] = sigmoid'(in[k]) for k < n,
 * one read and two writes per element in one kernel ("Multi-output
 * pointwise fusion: evidence and limits", "Measurement definitions and
 * population").  Device buffers of n floats, 4-byte aligned; the outputs
 * must not overlap the input or each other.  n == 0 is a no-op. */
int tile_sigmoid_pair_f32(const float *in, float *value, float *derivative, long long n,
                          cudaStream_t stream);

/* The same for tanh-approximate GELU, g(x) = x/2 (1 + tanh(sqrt(2/pi)
 * (x + 0.044715 x^3))), and its derivative. */
int tile_gelu_tanh_pair_f32(const float *in, float *value, float *derivative, long long n,
                            cudaStream_t stream);

/* ---- end to end on host buffers ---------------------------------------- */
/* The notes time single calls in two phases, GPU time and end to end with
 * the host's part included ("Immutable input reuse in Metal reductions",
 * "Fixed-width GPU and dispatch results"); on a GPU whose inputs start in
 * host memory the end-to-end phase also moves the rows across the host
 * link, which these entry points pipeline.  The notes have no interface of
 * this kind: its arguments and schedule are this library's own. */

/* Run `op` on HOST buffers h_in[, h_residual] -> h_out ([rows][width] FP32
 * each).  Rows stream through the caller's device workspace `d_work`
 * (`work_bytes` bytes, 256-byte aligned) in chunks of about rows/16 rows (at
 * least 1 MiB of a tensor, at most what fits twice in the workspace), held in
 * a ring of 2 to 4 workspace buffers (as many as fit): the host->device copy
 * of one chunk, the kernel on an earlier chunk and the device->host copy of
 * one before that overlap on three streams (the caller's
 * `stream` runs the kernels; two internal non-blocking streams per device,
 * created on first use, run the copies).  Host buffers should be pinned
 * (cudaHostAlloc / cudaHostRegister) for the copies to overlap; pageable
 * memory gives the same results more slowly.  When h_out is pinned the
 * kernels store the results straight into it through its device address
 * (NVLink-C2C on Grace systems) and no device->host copies are made.  When
 * h_in, h_residual and h_out are all pinned and device-addressable, there is
 * no pipeline: one launch of the selected kernel reads and writes the host
 * buffers directly (d_work is then not touched).  Ownership: the caller owns all
 * buffers and must keep them alive and untouched until `stream` has passed
 * this call (the call returns once everything is enqueued; `stream` is
 * ordered after the last copy or the kernel).  Results meet the same tolerance
 * as the device entry points, and are bitwise equal to those of a device
 * call on the whole matrix when width is a multiple of 4: every chunk runs
 * the whole matrix's plan (chunks start 256-byte aligned in the workspace,
 * so row start phases can differ from the full matrix otherwise).  `h_residual` is read only by
 * TILE_OP_RESIDUAL_LAYERNORM.  Errors: as the compute entry points, plus
 * TILE_ERR_NULL for a NULL d_work, TILE_ERR_ALIGN for a misaligned d_work and
 * TILE_ERR_WORKSPACE when not even one row fits twice.  Calls from several
 * host threads on one device are serialised inside the library. */
int tile_run_host_f32(int op, const float *h_in, const float *h_residual, float *h_out,
                      int rows, int width, float eps, void *d_work, size_t work_bytes,
                      cudaStream_t stream);

/* Workspace bytes tile_run_host_f32 needs to move `chunk_rows` rows per
 * chunk (0 for invalid arguments).  Host only. */
size_t tile_host_workspace_bytes(int op, int width, int chunk_rows);

/* The schedule tile_run_host_f32 uses for these arguments: rows per full
 * chunk (the first and the last chunk are a quarter of that when a quarter
 * still holds 1 MiB of an input and there are more than two chunks; the
 * last may otherwise be shorter) and the number of workspace buffers in the
 * ring.  `direct_output` != 0 describes a call whose h_out is pinned and
 * device-addressable (results stored straight into it), 0 one whose results
 * are copied out.  Host only: no CUDA call.  Returns TILE_OK, TILE_ERR_OP,
 * TILE_ERR_SHAPE (rows < 1 or width outside 1..tile_max_width()),
 * TILE_ERR_NULL for a NULL output pointer, or TILE_ERR_WORKSPACE as
 * tile_run_host_f32 would. */
int tile_host_schedule(int op, int rows, int width, size_t work_bytes, int direct_output,
                       int *chunk_rows, int *slots);

/* Size of the library's own device staging area used by
 * tile_run_host_static_f32: 64 MiB, held by every GPU that loads the library
 * until the process exits. */
#define TILE_STATIC_STAGING_BYTES (64u << 20)

/* tile_run_host_f32 for callers that cannot allocate device memory.  (The
 * notes this library follows have no counterpart of this call.)
 *
 * Some callers cannot call cudaMalloc where they run: code that runs after
 * an application has fixed its device memory budget, plugin code inside a
 * framework that owns the device allocator, or latency-critical code where a
 * device allocation (which can synchronise the device) is not allowed.  This
 * call allocates nothing: rows are staged through a static device array of
 * TILE_STATIC_STAGING_BYTES inside the library instead of a caller
 * workspace (pinned, device-addressable buffers are processed in place, as
 * by tile_run_host_f32).  Arguments, results, errors and ownership are those of
 * tile_run_host_f32 without d_work/work_bytes.
 *
 * Limits: any number of rows (they stream through the area in chunks);
 * 1 <= width <= tile_max_width() (one row of every tensor, 3 x 4 x 131072
 * bytes at most, fits the area twice).  A width beyond that maximum returns
 * TILE_ERR_SHAPE, and TILE_ERR_WORKSPACE would report a row that cannot fit.
 *
 * Set-up: the first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, which may load the library's device code) and
 * creates one event; make that first call before any stream capture.
 *
 * Sharing: every call on a device uses the same array, and the array keeps
 * the last call's contents (nothing in it needs to start at zero: each
 * chunk is copied in before the kernel reads it).  Calls that overlapped on
 * the GPU would race on the array, so the library orders each call's work
 * on the GPU after the previous call's end (an event), whatever stream it
 * was given; calls on different streams therefore run one after another.
 * A call that fails part-way (TILE_ERR_CUDA after some chunks were
 * enqueued) still marks its end after everything it enqueued, so the next
 * call waits for that work too.  Argument errors are returned before any
 * CUDA call. */
int tile_run_host_static_f32(int op, const float *h_in, const float *h_residual, float *h_out,
                             int rows, int width, float eps, cudaStream_t stream);

/* ---- plans and diagnostics -------------------------------------------- */

/* The plan the library would launch for (op, rows, width) with 16-byte
 * co-aligned pointers (the common case).  Host only; touches no GPU.
 * Returns TILE_OK, TILE_ERR_OP or TILE_ERR_SHAPE.  `plan` is written on
 * success only. */
int tile_describe_plan(int op, int rows, int width, tile_plan_t *plan);

/* tile_describe_plan for an element type (TILE_DTYPE_*); TILE_ERR_DTYPE for
 * an unknown one.  For large problems (rows * width above 2^22) the answer
 * may be a plan that needs rows of whole 16-byte vectors -- a
 * shared-memory-staged plan (path TILE_PATH_STAGED) or an R-rows-per-CTA
 * plan (TILE_PATH_ROWS) -- which a call takes only when every pointer is
 * 16-byte aligned and width is a multiple of the vector (4 FP32, 8 BF16 /
 * FP16 elements); other calls of that shape take the register plan of the
 * same width.  For TILE_OP_LAYERNORM_AFFINE the answer is that of a call
 * without a residual (a call with a residual has its own measured table). */
int tile_describe_plan_ex(int op, int dtype, int rows, int width, tile_plan_t *plan);

/* Number of plans built into the library, and plan `id` of that table
 * described for (op, rows, width).  Returns TILE_ERR_PLAN for a bad id and
 * TILE_ERR_SHAPE if the plan cannot cover `width`.  Host only. */
int tile_plan_count(void);
int tile_plan_info(int id, int op, int rows, int width, tile_plan_t *plan);

/* tile_plan_info for an element type; TILE_ERR_PLAN also when plan `id` is
 * not built for that type (BF16 / FP16 plans whose stripe would pass 64 floats), or
 * is a shared-memory-staged plan and `op` a row reduction (sum, min/max),
 * which only the register plans implement. */
int tile_plan_info_ex(int id, int op, int dtype, int rows, int width, tile_plan_t *plan);

/* Test hook for failure detection without a GPU fault (the notes have no
 * counterpart: their runner has no error path to test).  After `skip` more
 * launch attempts that proceed normally, the next `count` kernel launch
 * attempts of the library's entry points fail on the host with the CUDA
 * error `cuda_error` (a nonzero cudaError_t value) instead of launching:
 * the entry point returns TILE_ERR_CUDA and tile_last_cuda_error() on that
 * thread gives `cuda_error`.  Argument errors are still reported first.
 * Nothing reaches the GPU for an injected failure; work the same call
 * enqueued before it (copies and kernels of earlier chunks of
 * tile_run_host_f32 / tile_run_host_static_f32) stays enqueued, and the
 * caller's stream stays ordered after it.  count = 0 disarms.  Process-wide,
 * thread-safe, host only.  Returns TILE_OK, or TILE_ERR_SHAPE for a negative
 * skip or count, or a zero error with count > 0. */
int tile_inject_launch_failure(int cuda_error, int skip, int count);

/* Test hook for the whole-vector kernels (the notes have no counterpart).
 * 2-byte rows that are 16-byte aligned and hold whole 16-byte vectors run
 * a form of the row kernel (and, on the S = 4, P = 1, K = 4 shape, of the
 * LayerNorm backward kernel) without a scalar head and tail; its results
 * are bitwise those of the general form, where a head and tail of no
 * elements add exact +0 terms (which can change only the sign of a zero
 * result, after a partial sum of exactly -0).  With `on` nonzero every
 * later launch takes the general form instead, so a test can compare the
 * two on the same rows; 0 restores the default.  Process-wide, host only;
 * returns TILE_OK. */
int tile_test_force_general_kernels(int on);

/* Test hook for the bounded waits of the shared-memory-staged kernel (the
 * notes have no counterpart: their kernels have no copy engine to wait on).
 * Runs the staged plan `plan_id` (path TILE_PATH_STAGED) of `op` on `args`
 * as tile_run_plan_args_f32 would, except that no CTA issues the bulk copy
 * of its first row and every barrier wait gives up after `spin_limit` polls
 * (0 counts as 1).  The first wait of every CTA therefore runs out: the
 * kernel sets its wait-timeout bit in the device status word, stops
 * waiting and copying, waits (bounded) for the copies it did issue, and
 * returns with its outputs invalid.  tile_check_device_status then returns
 * TILE_ERR_DEVICE and clears the word.  Nothing is left in flight (the
 * withheld copy is never issued).  No other entry point withholds a copy;
 * library calls wait up to 2^20 polls.  Errors as tile_run_plan_args_f32;
 * TILE_ERR_PLAN also for a plan that is not staged. */
int tile_test_staged_wait_timeout(int op, int plan_id, const tile_row_args_t *args,
                                  unsigned int spin_limit, cudaStream_t stream);

/* The same for the block norm's gradients and the linear cross entropy
 * (forward): the call, with the first row of the first program, or the first
 * tiles of the first CTA pair, never copied, and waits of 16 ms instead of 2 s.
 * BF16 rows of whole 16-byte vectors in CTAs of up to 256 threads (widths up to
 * 5120, and above 16384 up to 32768), and BF16 rows of up to 4096 columns, are
 * built for it; TILE_ERR_PLAN for others.  Else arguments and errors of
 * tile_block_norm_backward and tile_linear_cross_entropy. */
int tile_test_block_norm_backward_wait_timeout(const tile_block_norm_backward_args_t *args,
                                               void *workspace, size_t workspace_bytes,
                                               cudaStream_t stream);
int tile_test_linear_cross_entropy_wait_timeout(int dtype, const void *in, const void *weight,
                                                const long long *target, float *loss, float *lse,
                                                int rows, int width, int vocab,
                                                long long ignore_index, void *workspace,
                                                size_t workspace_bytes, cudaStream_t stream);

/* Run `op` (one of the first four op codes) with the built plan `plan_id`
 * instead of the selector's choice (used by the measured plan sweep and by
 * tests that check every plan; tile_run_plan_args_f32 covers every op).
 * Same contract as the compute entry points; `residual` is used only by
 * TILE_OP_RESIDUAL_LAYERNORM.  Returns TILE_ERR_PLAN if the plan does not
 * exist, cannot cover `width`, or needs 16-byte co-alignment (V = 4) that
 * the pointers do not have. */
int tile_run_plan_f32(int op, int plan_id, const float *in, const float *residual,
                      float *out, int rows, int width, float eps, cudaStream_t stream);

/* Widest row any built plan covers. */
int tile_max_width(void);

/* The cudaError_t value behind the last TILE_ERR_CUDA returned on this host
 * thread (0 if none). */
int tile_last_cuda_error(void);

/* A static, human-readable description of a status code. */
const char *tile_status_string(int status);

/* Synchronise `stream`, then read and clear the device error word that
 * kernels set instead of trapping.  Returns TILE_OK, TILE_ERR_DEVICE (a
 * kernel recorded an error since the last check) or TILE_ERR_CUDA. */
int tile_check_device_status(cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TILE_ROWS_H */
