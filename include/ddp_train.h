/*
 * ddp_train.h -- C ABI of the operators around the gradient sync of
 * ddp_ring.h, on the same MI355X (gfx950): what makes the gradients where the
 * sync reads them (a linear layer and its gradients), and what reads them
 * after it (the global gradient norm, clipping, an AdamW step).
 *
 * In the step of "DDP 与 Ring All-Reduce" (blog.vllbc.top), section 05, the
 * layer is step 2 (backward produces the gradients, whose hooks mark them
 * ready) and the optimizer is what step 5 hands the reduced gradients to. The
 * operators themselves are written from the formulas given with each.
 *
 * Conventions: those of ddp_ring.h (status codes, ddp_last_error, device
 * pointers checked against their allocations before anything is launched,
 * host arrays of device pointers, work enqueued on `stream` without waiting,
 * DDP_FP32 / DDP_BF16). In addition:
 *   - All sums are held in fp32 or wider; a bf16 result is rounded once, to
 *     nearest, ties to even.
 *   - Results do not depend on the order in which blocks run: no floating
 *     point atomics are used, so a call repeated on the same inputs gives the
 *     same bits.
 *   - Every call except the create and free functions can be captured in a
 *     graph.
 */
#ifndef DDP_TRAIN_H
#define DDP_TRAIN_H

#include <stdint.h>

#include "ddp_ring.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- gradient norm, clipping
 * A ddp_grads is a set of gradient tensors (one rank's, or any others on one
 * device) whose places stay the same from step to step, as those of a
 * gradient arena (ddp_plan_grad_arena) do.
 *
 * ddp_grads_create: grads[n] are device pointers (host array, copied), each
 *   aligned to its element size and numels[i] >= 0 contiguous elements of
 *   `dtype`, pairwise disjoint; an empty tensor's pointer may be NULL. n >= 0.
 *   The set belongs to the current device: a table of 16 bytes per 8192
 *   elements (one entry at least per tensor that is not empty) and 17 KiB of scratch are
 *   allocated there. The tensors must stay allocated while the set exists.
 *   Calls on one set share its scratch: they must be ordered (one stream, or
 *   streams that wait for each other). Creating a set asks the runtime about every
 *   tensor, allocates and copies, and waits for it: some 100 us, which is more than the
 *   calls of a step on a small set take. A set is made once, not every step; the same
 *   goes for ddp_adamw_create. */
typedef struct ddp_grads ddp_grads;
int ddp_grads_create(void* const* grads, const int64_t* numels, int32_t n, int32_t dtype, ddp_grads** out);

/* Releases a set (NULL is accepted); no work that uses it, and no ddp_adamw
 * made from it, may be left. */
void ddp_grads_free(ddp_grads* grads);

/* ddp_grads_norm: *norm_dev (a device float, overwritten, in none of the tensors) receives
 *   DDP_NORM_L2:  sqrt(sum g^2) over every element of every tensor;
 *   DDP_NORM_MAX: max |g|.
 * The squares are summed in fp64, so no finite fp32 gradient overflows or
 * vanishes on the way. A NaN element makes the norm NaN, an infinite one (without NaN)
 * infinite; an empty set's norm is 0. One launch. */
#define DDP_NORM_L2 0
#define DDP_NORM_MAX 1
int ddp_grads_norm(ddp_grads* grads, int32_t kind, float* norm_dev, void* stream);

/* ddp_grads_clip: into = rnd(g * f), f = min(1, max_norm / (*norm_dev + 1e-6)),
 * element by element. `into` is a set of the same element counts (of either
 * dtype), none of whose tensors overlaps one of `grads`, or NULL to scale
 * `grads` in place, where a factor of 1 leaves the gradients untouched. *norm_dev is
 * read when the launch runs: the value of ddp_grads_norm on the same stream, or one
 * combined from several sets' by the caller; it lies in none of the tensors that
 * are written. A NaN norm gives NaN gradients;
 * an infinite one gives f = 0 (NaN if max_norm is infinite too). max_norm >= 0
 * (infinity: never clip a finite norm). */
int ddp_grads_clip(const ddp_grads* grads, const ddp_grads* into, float max_norm, const float* norm_dev,
                   void* stream);

/* ---------------------------------------------------------------- AdamW
 * ddp_adamw_create: an optimizer over the set's tensors. For tensor i of n
 *   (the set's n), params[i], exp_avg[i] and exp_avg_sq[i] are fp32 device
 *   arrays of the gradient's element count; params_bf16 (NULL for none) gives
 *   bf16 arrays that receive the rounded new weights; decay (NULL: all 1)
 *   holds 1 for tensors that weight decay applies to, else 0. *step_dev is a
 *   device int64, the number of steps done (0 at first). Everything but the
 *   gradients is written, so none of it may overlap anything else. The pointers
 *   are copied into a device table; the set must outlive the optimizer. */
typedef struct ddp_adamw ddp_adamw;
int ddp_adamw_create(const ddp_grads* grads, void* const* params, void* const* exp_avg, void* const* exp_avg_sq,
                     void* const* params_bf16, const uint8_t* decay, int64_t* step_dev, ddp_adamw** out);

/* Releases an optimizer (NULL is accepted); no work that uses it may be left. */
void ddp_adamw_free(ddp_adamw* opt);

/* ddp_adamw_step: one AdamW step, in one launch up to 2.1e9 elements. With t = *step_dev + 1 and
 * f = 1 if norm_dev is NULL, else min(1, max_norm / (*norm_dev + 1e-6)):
 *   g = f * grad
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + (1 - beta2) g^2
 *   p = (1 - lr * weight_decay [if the tensor decays]) p
 *       - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps)
 *   params_bf16 = rnd(p); *step_dev = t.
 * The gradients are left as they are: clipping costs no pass of its own. If
 * norm_dev is given and *norm_dev is not finite, the step is skipped: nothing
 * is written. lr, eps, weight_decay and max_norm >= 0; beta1 and beta2 in
 * [0, 1). max_norm is not looked at without norm_dev, which lies in nothing
 * that the step writes. Calls on one optimizer
 * must be ordered. */
int ddp_adamw_step(ddp_adamw* opt, double lr, double beta1, double beta2, double eps, double weight_decay,
                   double max_norm, const float* norm_dev, void* stream);

/* ---------------------------------------------------------------- linear layer
 * Matrices are row-major: element (i, j) of a matrix with leading dimension
 * ld lies at i * ld + j; ld >= its number of columns and, with more than one
 * row, ld <= 2^22. Pointers are aligned to
 * the element; no other alignment is needed. Matrices that must not overlap
 * share no element; column blocks of one buffer do not. M, N, K >= 0: M rows (tokens),
 * K input and N output features; weights are w[N][K].
 * `dtype` is the type of x, w, bias, residual, y, z, dz, dx and add. Products
 * are summed in fp32: bf16 on the bf16 matrix instructions, fp32 on the fp32
 * ones.
 * Activations and their slopes:
 *   DDP_ACT_NONE       z
 *   DDP_ACT_RELU       max(z, 0), slope 0 at 0
 *   DDP_ACT_GELU       z/2 (1 + erf(z / sqrt 2))
 *   DDP_ACT_GELU_TANH  z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3)))
 *   DDP_ACT_SILU       z / (1 + exp(-z))
 * With fp32 data a value is off by a few 2^-24 of itself (for negative z, where
 * the exponential rules, times the exponent: gelu z^2 / 2, gelu_tanh 0.07 |z|^3).
 * With bf16 data faster forms are used, whose errors hide behind the result's
 * rounding: exponentials are off by 2^-24 times their argument, and gelu by 1.5e-7
 * |z| at most, which is 2e-3 of it at z = -5 and more below, where it is under 2e-6.
 * Workspace: with few output tiles the long sum is cut into parts, which need
 * scratch on the device: ddp_linear_workspace gives the bytes (0 if none) for
 * a direction and shape on the current device. A call with less (NULL, 0) is refused. The
 * contents need not be kept between calls; calls that may overlap need their own. 16-byte aligned. */
#define DDP_ACT_NONE 0
#define DDP_ACT_RELU 1
#define DDP_ACT_GELU 2
#define DDP_ACT_GELU_TANH 3
#define DDP_ACT_SILU 4

#define DDP_LINEAR_FORWARD 0
#define DDP_LINEAR_BACKWARD_INPUT 1
#define DDP_LINEAR_BACKWARD_WEIGHT 2
int ddp_linear_workspace(int32_t direction, int64_t M, int64_t N, int64_t K, int32_t dtype, int64_t* bytes);

/* ddp_linear_tiling: how a product of these sizes is cut, for whoever wants to
 * understand its time or to test a form: *tile is the side of its square tiles
 * (0: a few rows, without tiles), *parts the number of parts of the sum.
 * direct = 1: every operand's rows begin on 16 bytes and hold whole 16-byte
 * chunks; 0: any other alignment. */
int ddp_linear_tiling(int32_t direction, int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t direct, int32_t* tile,
                      int32_t* parts);

/* y = act(x w^T + bias) + residual; z (NULL: not kept) receives
 * rnd(x w^T + bias), which the backward pass takes. bias[N] and
 * residual may be NULL. The activation is applied to the unrounded sum.
 * y and z must not overlap the inputs, except that y may be the residual. */
int ddp_linear_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                       const void* residual, int64_t ldr, void* y, int64_t ldy, void* z, int64_t ldz,
                       int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t act,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* dx = (dz w) * act'(z) + add: the gradient of the layer's input, carried on
 * through the activation of the layer before it, whose kept z[M][K] is given
 * (NULL: no activation, `act` must be DDP_ACT_NONE), and joined with `add`
 * (NULL: none), the gradient that reaches the same place along a residual. dz
 * is the gradient of this layer's z, [M][N]. dx must not overlap the inputs,
 * except that it may be `add`. */
int ddp_linear_backward_input(const void* dz, int64_t lddz, const void* w, int64_t ldw, const void* z, int64_t ldz,
                              const void* add, int64_t ldadd, void* dx, int64_t lddx,
                              int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t act,
                              void* workspace, int64_t workspace_bytes, void* stream);

/* dw = dz^T x and db = sum of dz's rows (NULL: not wanted), of grad_dtype:
 * `dtype`, or fp32 gradients of bf16 data. accumulate = 0 overwrites; 1 adds
 * to what is there (one rounding of old + new), as over the micro-batches of
 * a step. dw[N][K] and db[N] may lie in a gradient arena, where the sync
 * reduces them in place. With M = 0 the sums are zero. */
int ddp_linear_backward_weight(const void* dz, int64_t lddz, const void* x, int64_t ldx, void* dw, int64_t lddw,
                               void* db, int64_t M, int64_t N, int64_t K, int32_t dtype, int32_t grad_dtype,
                               int32_t accumulate, void* workspace, int64_t workspace_bytes, void* stream);

/* dz = dy * act'(z), element by element over [M][N]: the gradient of a
 * layer's z where that of its output comes from something other than
 * ddp_linear_backward_input. dz may be dy. */
int ddp_act_backward(const void* dy, int64_t lddy, const void* z, int64_t ldz, void* dz, int64_t lddz,
                     int64_t M, int64_t N, int32_t dtype, int32_t act, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* DDP_TRAIN_H */
