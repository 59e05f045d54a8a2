/*
 * lmhead.h -- C ABI of the MI355X (gfx950) LM-head logits library.
 *
 *   logits[m, v] = alpha * (hidden[m, :] . W[v, :]) + bias[v]
 *
 * bf16 inputs, fp32 accumulation, fp32 or bf16 output; an NVFP4 weight-only
 * (W4A16) variant with bf16 output. Every output row depends only on its own
 * hidden row, the weight, alpha, bias and the output type: never on how many
 * rows are in the call, where the row sits in it, or which entry point (bf16
 * weight at any M) produced it. Each logit is summed over K in one fixed
 * order, starting at a point that depends on H and on the column's index v
 * within the call (in groups of 10240 columns) and wrapping around; so a call
 * on a row sub-range W + v0*H of the vocabulary (one GPU's shard) gives the
 * full call's columns bit for bit when v0 is a multiple of
 * 10240 * (H / 256) / gcd(5, H / 256) (any v0 when H % 256 != 0 or
 * H == 256: every column then starts at 0), and agrees with them within the
 * fp32 accumulation tolerance otherwise.
 *
 * Where the operation is defined (page title, then section):
 *  - bf16 x bf16 products accumulated at fp32 with fp32 logits and no fp32
 *    copy of the weight: sglang PR 32370 digest "FP32 LM head skips the FP32
 *    cast" (motivation; implementation breakdown; key source excerpt of
 *    _compute_lm_head), and vLLM PR 49120 "Honor fp32 head_dtype in Inkling
 *    muP logits (target + MTP draft)", section Purpose.
 *  - alpha = 1/mup folded into the projection's epilogue, equal bit for bit
 *    to the projection followed by a separate multiply: vLLM PR 49120,
 *    sections Purpose and "muP is folded into the fp32 GEMM (not a bypass)".
 *  - the embedding bias added to the logits: sglang digest, _compute_lm_head
 *    excerpt (embedding_bias argument).
 *  - the NVFP4 head with 16-bit activations and bf16 logits, whose rows do
 *    not depend on the row count, run in calls of at most 64 rows: metrale
 *    "lm_head_nvfp4_rows.rs" source page, module documentation and the row
 *    loop of lm_head_nvfp4_rows_run.
 *  - "launch nothing and report that the fast path does not cover the case",
 *    leaving the caller to fall back: the same metrale page (the Ok(false)
 *    return of lm_head_nvfp4_rows_run) and vLLM PR 49120, section Purpose
 *    (fallback cases the fused op does not cover).
 *
 * Conventions shared by every entry point:
 *  - Every tensor pointer is a DEVICE pointer to memory the caller owns and
 *    keeps alive until the enqueued work has finished. The library never
 *    allocates, frees or synchronises; it only enqueues kernels on `stream`.
 *  - All tensors are dense and row-major: hidden [M, H], W [V, H] (the
 *    nn.Linear layout, used transposed), logits [M, V].
 *  - `stream` is a hipStream_t passed as void*; NULL means the default stream.
 *  - `out` must not overlap any input.
 *  - Work is checked on the host before anything is launched; on any non-OK
 *    status nothing was launched. Faults inside a kernel surface at the
 *    caller's next synchronisation, as for any HIP work.
 *  - The library keeps no state between calls apart from HIP's own
 *    once-per-process code-object load; calls from several threads are safe.
 */
#ifndef LMHEAD_H
#define LMHEAD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  LMHEAD_F32 = 0,   /* fp32, 4 bytes per element */
  LMHEAD_BF16 = 1,  /* bf16, 2 bytes per element (logits: rounded to nearest even) */
  LMHEAD_F16 = 2    /* IEEE fp16, 2 bytes per element (logits: rounded to nearest even) */
} lmhead_dtype;

typedef enum {
  LMHEAD_OK = 0,           /* work enqueued on `stream`, or M == 0 and nothing to do */
  LMHEAD_NOT_HANDLED = 1,  /* well-formed, outside the shape or dtype contract: nothing
                              launched, the caller falls back */
  LMHEAD_ERR_INVALID = -1, /* NULL pointer with M > 0, M < 0, H <= 0, V <= 0, unknown dtype
                              or path, sizes beyond the documented maxima */
  LMHEAD_ERR_ALIGN = -2,   /* a base pointer below its required alignment */
  LMHEAD_ERR_DEVICE = -3   /* HIP reported an error when the kernel was launched */
} lmhead_status;

typedef enum {
  LMHEAD_PATH_NONE = -1,   /* outside the contract: NOT_HANDLED */
  LMHEAD_PATH_AUTO = -2,   /* let the library choose (the normal use) */
  LMHEAD_PATH_SKINNY = 0,  /* weight-streaming split-V kernel, chosen for M <= 64 */
  LMHEAD_PATH_TILED = 1,   /* LDS-tiled MFMA GEMM, chosen for M > 64 */
  LMHEAD_PATH_NVFP4 = 2    /* NVFP4 W4A16 kernel */
} lmhead_path;

/* Shape contract (both entry points):
 *   M >= 0, H >= 32 and H % 32 == 0, V >= 1,
 *   M <= LMHEAD_MAX_M, H <= LMHEAD_MAX_H, V <= LMHEAD_MAX_V.
 * (The kernels address one work-group's block of output rows, and one wave's
 * slice of weight rows, with 32-bit byte offsets; the maxima keep every such
 * block below 1 GiB. V <= 2^20 covers every vocabulary in use.)
 * Alignment: hidden, W, w_e2m1 and out 16-byte aligned; bias 4-byte aligned;
 * w_scale 2-byte aligned. (torch allocations are 256-byte aligned; a row
 * sub-range W + v0*H stays 16-byte aligned because H % 32 == 0.) */
#define LMHEAD_MAX_M ((int64_t)1 << 24)
#define LMHEAD_MAX_H ((int64_t)1 << 16)
#define LMHEAD_MAX_V ((int64_t)1 << 20)

/* The projection with a bf16 weight.
 *   hidden    bf16 [M, H]                       (device, read)
 *   W         bf16 [V, H]                       (device, read)
 *   alpha     fp32 scale applied to the fp32 accumulator: t = fl32(alpha * acc)
 *   bias      fp32 [V] or NULL                  (device, read): t = fl32(t + bias[v]),
 *             a separate rounding, never fused with the multiply
 *   out_dtype LMHEAD_F32 or LMHEAD_BF16
 *   out       [M, V] of out_dtype               (device, written; every element)
 * Returns LMHEAD_OK, LMHEAD_NOT_HANDLED (H % 32 != 0) or an error. */
lmhead_status lmhead_logits(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V,
                            float alpha, const float *bias, lmhead_dtype out_dtype, void *out,
                            void *stream);

/* As lmhead_logits, with the kernel chosen by the caller: LMHEAD_PATH_AUTO,
 * LMHEAD_PATH_SKINNY (any M; the chunked skinny kernel walks 64-row blocks)
 * or LMHEAD_PATH_TILED (any M). Both kernels run the same K-step chain, so
 * their results are bit-identical; this entry point exists to show that. */
lmhead_status lmhead_logits_path(const void *hidden, int64_t M, int64_t H, const void *W,
                                 int64_t V, float alpha, const float *bias,
                                 lmhead_dtype out_dtype, void *out, void *stream, int path);

/* The projection with 16-bit inputs of either kind: hidden and W both bf16,
 * or both IEEE fp16 (sglang PR 32370 digest, implementation breakdown and the
 * key source excerpt: the fp32-output fast path takes bf16 or fp16 inputs of
 * one dtype and falls back otherwise). fp16 inputs run the fp16 MFMA of the
 * same shape through the same K-step chain and epilogue, so everything said
 * of lmhead_logits holds with fp16 in place of bf16.
 *   in_dtype   LMHEAD_BF16 or LMHEAD_F16: the type of hidden and of W
 *   out_dtype  LMHEAD_F32, or in_dtype (logits rounded to nearest even)
 *   path       as in lmhead_logits_path
 * Returns LMHEAD_NOT_HANDLED for any other (in_dtype, out_dtype) pair, for
 * instance fp32 inputs (nothing launched; the caller falls back), else as
 * lmhead_logits. lmhead_logits(...) is lmhead_logits_ex(..., LMHEAD_BF16,
 * out_dtype, out, stream, LMHEAD_PATH_AUTO). */
lmhead_status lmhead_logits_ex(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V,
                               float alpha, const float *bias, lmhead_dtype in_dtype,
                               lmhead_dtype out_dtype, void *out, void *stream, int path);

/* The projection with a row-reduction epilogue: for every row m, over the
 * fp32 logits t[m, v] the call computes (the epilogue values of
 * lmhead_logits_ex, before any rounding to a 16-bit out_dtype):
 *   row_max[m]    = max over v of t[m, v]
 *   row_argmax[m] = the lowest v with t[m, v] == row_max[m]
 *   row_sumexp[m] = sum over v of exp(t[m, v] - row_max[m])   (>= 1)
 * Logits of -inf (a masked vocabulary entry, through a -inf bias) are
 * allowed and contribute exp(-inf) = 0; a row whose logits are all -inf gets
 * row_max -inf, row_argmax its lowest column and row_sumexp 0. +inf and NaN
 * logits are outside the contract.
 * so that the row's log-sum-exp is row_max + log(row_sumexp) and
 * softmax(t)[m, v] = exp(t[m, v] - row_max[m]) / row_sumexp[m]. These feed
 * the target and draft heads' acceptance distributions (vLLM PR 49120,
 * section Purpose) and greedy selection whose ties keep the lowest index, as
 * a stable descending sort does (tokenspeed PR 720, summary and review
 * thread). They are computed inside the GEMM's epilogue, so the [M, V] logits
 * need not be written at all.
 *   hidden, W, alpha, bias, in_dtype, out_dtype, path   as in lmhead_logits_ex
 *   out         [M, V] of out_dtype, or NULL: the logits are then not written
 *   row_max     fp32 [M]                          (device, written)
 *   row_argmax  int32 [M]                         (device, written)
 *   row_sumexp  fp32 [M]                          (device, written)
 *   workspace   device memory of at least lmhead_rowreduce_workspace_bytes(M, V)
 *               bytes, 16-byte aligned; the call overwrites it (it holds one
 *               16-byte partial per row and 16-column block) and it must not be
 *               in use by other work until this call's work has finished
 * row_max and row_argmax are exact: the maximum and the lowest argmax of the
 * fp32 logits lmhead_logits_ex writes (a zero maximum present with both signs
 * may be returned as either zero). row_sumexp is accumulated at fp32 in a
 * fixed order that depends only on V, each exponential taken as
 * 2^(x log2 e). All three are the same, bit for bit, whatever the row count
 * of the call and the path.
 * Returns as lmhead_logits_ex; LMHEAD_ERR_INVALID also for a NULL row output
 * or workspace, or a workspace smaller than required (M > 0); LMHEAD_ERR_ALIGN
 * for a misaligned workspace or row output (4-byte). */
lmhead_status lmhead_logits_rowreduce(const void *hidden, int64_t M, int64_t H, const void *W,
                                      int64_t V, float alpha, const float *bias,
                                      lmhead_dtype in_dtype, lmhead_dtype out_dtype, void *out,
                                      float *row_max, int32_t *row_argmax, float *row_sumexp,
                                      void *workspace, size_t workspace_bytes, void *stream,
                                      int path);

/* Host-only: bytes of workspace lmhead_logits_rowreduce needs for (M, V):
 * 16 * M * ceil(V / 16); 0 when M or V is outside the shape contract. */
size_t lmhead_rowreduce_workspace_bytes(int64_t M, int64_t V);

/* Bytes of the partials buffer the library holds for
 * lmhead_logits_rowreduce_noalloc, per GPU it runs on (32 MiB). */
#define LMHEAD_NOALLOC_SCRATCH_BYTES ((int64_t)32 << 20)

/* lmhead_logits_rowreduce for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, hosts that forbid
 * allocation. It takes no workspace: the partials go to a buffer of
 * LMHEAD_NOALLOC_SCRATCH_BYTES that the library keeps in a file-scope device
 * array, one per GPU, held until the process ends. The call allocates and
 * frees nothing (no hipMalloc, no allocating library routine); the caller
 * still passes the inputs and outputs. Arguments, results and bits are those
 * of lmhead_logits_rowreduce with the same arguments.
 * Limit: lmhead_rowreduce_workspace_bytes(M, V) <= LMHEAD_NOALLOC_SCRATCH_BYTES
 * (16 M ceil(V / 16) bytes: M <= 220 rows at V = 151936), else
 * LMHEAD_ERR_INVALID with nothing launched.
 * Every call on one GPU shares that GPU's buffer: calls whose work overlaps in
 * time on one GPU (other streams, other host threads) race on it and must be
 * ordered by the caller. The buffer's device address is looked up on the
 * first call on each device (LMHEAD_ERR_DEVICE if that fails). */
lmhead_status lmhead_logits_rowreduce_noalloc(const void *hidden, int64_t M, int64_t H,
                                              const void *W, int64_t V, float alpha,
                                              const float *bias, lmhead_dtype in_dtype,
                                              lmhead_dtype out_dtype, void *out, float *row_max,
                                              int32_t *row_argmax, float *row_sumexp,
                                              void *stream, int path);

/* The NVFP4 W4A16 head (bf16 logits).
 *   hidden       bf16 [M, H]                    (device, read)
 *   w_e2m1       uint8 [V, H/2]: two OCP E2M1 codes per byte, element 2i in the
 *                low nibble and 2i+1 in the high nibble (device, read)
 *   w_scale      uint8 [V, H/16]: one OCP E4M3 scale per 16 consecutive
 *                elements of a weight row (device, read)
 *   global_scale fp32 per-tensor scale g
 *   alpha, bias  as in lmhead_logits; the epilogue multiplies the accumulator
 *                by s = fl32(global_scale * alpha), then adds the bias
 *   out          bf16 [M, V]                    (device, written)
 * The weight w[v, k] = e2m1 * e4m3 is exact in bf16 and runs through the same
 * K-step chain as lmhead_logits: lmhead_logits_nvfp4 equals lmhead_logits on
 * the dequantised weight with alpha' = s, bit for bit. */
lmhead_status lmhead_logits_nvfp4(const void *hidden, int64_t M, int64_t H,
                                  const uint8_t *w_e2m1, const uint8_t *w_scale,
                                  float global_scale, int64_t V, float alpha, const float *bias,
                                  void *out, void *stream);

/* BF16 -> NVFP4 quantisation of a head: the weight lmhead_logits_nvfp4 reads,
 * made from a bf16 weight in two passes -- the tensor's absolute maximum, then
 * block quantisation -- as the metrale page "layers/mtp_head/new_bf16_moe.rs"
 * requantises BF16 weights to NVFP4 at load with an absmax kernel and an NVFP4
 * kernel (quantize_to_nvfp4, new_nvfp4_draft_moe). Every step is a binary32
 * operation (division correctly rounded):
 *   g = amax / 2688 (6 * 448; 1 when that is 0), amax = max |W|
 *   per 16 consecutive elements of a row: s = bmax / (6 g) rounded to E4M3
 *     (nearest even, at most 448); d = e4m3(s) * g
 *   per element: code = sign bit of W | E2M1(|W| / d) (nearest even,
 *     at most 6; magnitude 0 when d == 0)
 *   W             bf16 [V, H], finite               (device, read)
 *   w_e2m1        uint8 [V, H/2], layout as in lmhead_logits_nvfp4 (device, written)
 *   w_scale       uint8 [V, H/16]                   (device, written)
 *   global_scale  one fp32, g                       (device, written)
 *   workspace     at least lmhead_quantize_nvfp4_workspace_bytes() bytes of
 *                 device memory, 4-byte aligned, overwritten by the call
 * Shape contract as for the projection with M = 1 (H % 32 != 0:
 * LMHEAD_NOT_HANDLED). Alignment: W 16, w_e2m1 4, global_scale 4 bytes.
 * The result is deterministic (maxima are exact, the per-element steps fixed). */
lmhead_status lmhead_quantize_nvfp4(const void *W, int64_t V, int64_t H, uint8_t *w_e2m1,
                                    uint8_t *w_scale, float *global_scale, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* Host-only: bytes of workspace lmhead_quantize_nvfp4 needs (a constant). */
size_t lmhead_quantize_nvfp4_workspace_bytes(void);

/* ---------------------------------------------------------------------------
 * Training the head: softmax cross entropy over the vocabulary without the
 * logits in memory, and its gradients.
 *   t[m, v] = alpha * (hidden[m, :] . W[v, :]) + bias[v]   (as lmhead_logits_ex, fp32)
 *   lse[m]  = log sum_v exp(t[m, v]);  loss[m] = lse[m] - t[m, target[m]]
 * (the loss is made from the row's largest t, not from lse as rounded).
 * A row is left out when its target equals ignore_index or is no column of
 * the call (target < 0 or >= V): its loss is 0 and carries no gradient; its
 * lse is written all the same. t = -inf (a masked column, through a -inf
 * bias) has probability 0: a target there has loss +inf, and a row of
 * only -inf has lse -inf. The type's lowest value is a number: it masks a column
 * just as well, and a target there has the finite loss lse - t. The
 * probabilities of the backward pass are exp(t - lse) of lse as rounded to fp32:
 * off by 2^-24 |lse|, relatively, so good for |lse| up to thousands, and no
 * probabilities any more past 2^24 (a row masked in every column by the lowest
 * value). +inf and NaN logits give NaN (and a hidden row that
 * is not finite makes grad_W so, even where the row is left out: it enters the
 * product with 0).
 * ------------------------------------------------------------------------- */
typedef enum {
  LMHEAD_INDEX32 = 0, /* int32 targets or token ids */
  LMHEAD_INDEX64 = 1  /* int64 */
} lmhead_index;

/* loss and lse.
 *   hidden [M, H], W [V, H]  both bf16 or both fp16 (in_dtype)  (device, read)
 *   bias        fp32 [V] or NULL                                (device, read)
 *   target      [M] of target_type                              (device, read)
 *   loss, lse   fp32 [M]                                        (device, written)
 *   workspace   at least lmhead_xent_forward_workspace_bytes(M, V) bytes, 16-byte
 *               aligned, overwritten; not in use by other work until this call's
 *               work has finished
 * A row's results depend on that row, W, alpha and bias only, not on the call's
 * other rows, and do not change from run to run. Returns as lmhead_logits_ex
 * (LMHEAD_NOT_HANDLED for fp32 inputs or H % 32 != 0). */
lmhead_status lmhead_xent_forward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V,
                                  float alpha, const float *bias, lmhead_dtype in_dtype,
                                  const void *target, lmhead_index target_type,
                                  int64_t ignore_index, float *loss, float *lse, void *workspace,
                                  size_t workspace_bytes, void *stream);

/* Host-only: bytes of workspace lmhead_xent_forward needs (0 outside the shape contract). */
size_t lmhead_xent_forward_workspace_bytes(int64_t M, int64_t V);

/* Gradients of sum_m grad_loss[m] loss[m] + grad_lse[m] lse[m]. With
 *   G[m, v] = (grad_loss[m] + grad_lse[m]) exp(t[m, v] - lse[m]) - grad_loss[m] [v = target[m]]
 * (grad_loss taken as 0 in rows left out):
 *   grad_hidden = alpha G W, grad_W = alpha G^T hidden, grad_bias = sum over rows of G.
 *   hidden .. ignore_index   as given to lmhead_xent_forward
 *   lse         fp32 [M], as lmhead_xent_forward wrote it       (device, read)
 *   grad_loss   fp32 [M]                                        (device, read)
 *   grad_lse    fp32 [M], or NULL for zeros                     (device, read)
 *   grad_hidden [M, H] of in_dtype, or NULL (not wanted)        (device, written)
 *   grad_W      [V, H] of in_dtype, or NULL                     (device, written, every row)
 *   grad_bias   fp32 [V], or NULL                               (device, written)
 *   workspace   at least lmhead_xent_backward_workspace_bytes(M, H, V, grad_bias != NULL)
 *               bytes, 256-byte aligned, overwritten; as above
 * Sums are fp32 in a fixed order; G enters the two products rounded to the
 * inputs' type. It is rounded after scaling by one factor for the whole call,
 * made from the largest finite upstream gradient of its rows: unlike the forward
 * pass's results, the last bits of a row's grad_hidden depend on the other rows'
 * upstream gradients, and with fp16 the entries of G below 2^-28 of the largest
 * lose digits, those below 2^-39 vanish. With M = 0, grad_W and grad_bias are
 * zero. */
lmhead_status lmhead_xent_backward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V,
                                   float alpha, const float *bias, lmhead_dtype in_dtype,
                                   const void *target, lmhead_index target_type,
                                   int64_t ignore_index, const float *lse, const float *grad_loss,
                                   const float *grad_lse, void *grad_hidden, void *grad_W,
                                   float *grad_bias, void *workspace, size_t workspace_bytes,
                                   void *stream);

/* Host-only: bytes of workspace lmhead_xent_backward needs: one piece of G (at
 * most 256 MiB, or 2 * 8192 * M bytes where that is more), the fp32 [M, H] sum of
 * grad_hidden, once per split of the vocabulary (up to 64 where M H is small; the
 * same whether grad_hidden is wanted or not), and little else. 0 outside the
 * shape contract or when M == 0. */
size_t lmhead_xent_backward_workspace_bytes(int64_t M, int64_t H, int64_t V, int grad_bias);

/* The K largest logits of each row, their columns, and the row's log-sum-exp at a
 * temperature: what a token is sampled from, and what lmhead_distill_forward takes of a
 * teacher.
 *   values[m, k], ids[m, k]  the k-th of row m's logits in descending order, and its
 *               column; equal logits (zeros of both signs too) by ascending column, NaN
 *               before all others. values are the logits' own bits.
 *   lse[m]      log sum_v exp(logits[m, v] / temperature): -inf for a row of only -inf, NaN
 *               for one with +inf or NaN; infinite else only where the largest logit /
 *               temperature is past fp32's range
 *   logits      [M, V] of dtype, rows row_stride elements apart (row_stride >= V), any
 *               alignment of an element                          (device, read)
 *   values      [M, K] of dtype; ids int32 [M, K]; lse fp32 [M]  (device, written)
 *   workspace   at least lmhead_logits_topk_workspace_bytes(M, V, K) bytes, 16-byte aligned,
 *               overwritten; as above (NULL where that is 0)
 *   1 <= K <= V, K <= LMHEAD_MAX_TOPK; temperature > 0
 * A row's results depend on that row alone but for lse's last bits, whose order of sums
 * depends on M, V and K; they do not change from run to run. Returns LMHEAD_OK or an error. */
#define LMHEAD_MAX_TOPK ((int64_t)1024)
lmhead_status lmhead_logits_topk(const void *logits, int64_t M, int64_t V, int64_t row_stride, lmhead_dtype dtype, int64_t K,
                                 float temperature, void *values, int32_t *ids, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Host-only: bytes of workspace lmhead_logits_topk needs (0 outside the contract, and
 * where it needs none). */
size_t lmhead_logits_topk_workspace_bytes(int64_t M, int64_t V, int64_t K);

/* ---------------------------------------------------------------------------
 * Further losses of the head's logits, which need not be whole in memory:
 *   t[m, v] = (alpha * (hidden[m, :] . W[v, :]) + bias[v]) / temperature,
 *   lse[m] = log sum_v exp(t[m, v]),  log q[m, v] = t[m, v] - lse[m]
 * (alpha / temperature and bias[v] / temperature are taken at fp32 each).
 * A forward call makes the rows' losses and, where `state` is given, leaves
 * there what lmhead_loss_backward needs; that call may be made more than once on
 * one state, and the state belongs to the call's hidden, W and bias.
 *   temperature > 0
 *   state       at least lmhead_loss_state_bytes(M, H, V, K, keep_logits) bytes,
 *               256-byte aligned (device, written), or NULL when no backward pass
 *               follows
 *   keep_logits 0, or 1: the forward call leaves every t it works on in the state (fp32,
 *               4 M V bytes and the ends of tiles; room for all rows), and the backward
 *               call reads them instead of making them again, which is one of its three
 *               products. The gradients are the same, bit for bit; grad_bias up to the
 *               order of its fp32 sums. The backward call is given what the forward call was
 *   workspace   at least lmhead_loss_forward_workspace_bytes(M, H, V, K, state != NULL)
 *               bytes, 256-byte aligned, overwritten; not in use by other work
 *               until this call's work has finished
 * K is the teacher's logits per row for lmhead_distill_forward and 0 for the others. What
 * is said of lmhead_xent_forward about -inf, the lowest value, +inf and NaN
 * holds, as does its independence of the call's other rows (preference: of the
 * other pairs). What stands in the hidden rows that are left out reaches no result, not
 * grad_W either. Returns as lmhead_xent_forward.
 * ------------------------------------------------------------------------- */

/* The divergence from a teacher's top logits. A row's entries k are those whose
 * id is a column of the call and whose logit is not -inf; the others are absent.
 *   p_k = exp(teacher_logits[m, k] / temperature - n),
 *   n = teacher_lse[m], or (NULL) the log-sum-exp over the row's entries
 *   loss[m] = sum_k p_k (log p_k - log q[m, id_k])
 * With teacher_lse, the log-sum-exp of the teacher's logits / temperature over its
 * whole vocabulary, the entries' mass P = sum p_k is below 1 and what lies
 * outside them is left out of the sum. A row without entries has loss 0 and no
 * gradient. An id that a row has twice counts twice.
 *   teacher_ids     [M, K] of ids_type                          (device, read)
 *   teacher_logits  [M, K] of logits_dtype, any order           (device, read)
 *   teacher_lse     fp32 [M] or NULL                            (device, read)
 *   loss            fp32 [M]                                    (device, written)
 *   1 <= K <= LMHEAD_MAX_TEACHER */
#define LMHEAD_MAX_TEACHER ((int64_t)1024)
lmhead_status lmhead_distill_forward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                                     const float *bias, lmhead_dtype in_dtype, float temperature,
                                     const void *teacher_ids, lmhead_index ids_type, const void *teacher_logits,
                                     lmhead_dtype logits_dtype, int64_t K, const float *teacher_lse, float *loss,
                                     void *state, size_t state_bytes, int keep_logits, void *workspace, size_t workspace_bytes,
                                     void *stream);

/* The clipped policy loss with a KL term of the tokens target[m]:
 *   logp[m] = log q[m, target[m]],  r = exp(logp - old_logp) (NULL: 1),
 *   d = ref_logp - logp,
 *   loss[m] = -min(r A, min(max(r, 1 - clip_low), 1 + clip_high) A) + kl_coef (exp(d) - d - 1)
 * with A = advantage[m]; the first term is 0 where A is 0, the second where ref_logp
 * is NULL or kl_coef is 0. Its derivative by logp is -r A where the minimum is r A
 * (ties included) and 0 elsewhere, and kl_coef (1 - exp(d)); NaN where the first term
 * is. Rows whose target is
 * ignore_index or no column of the call have loss and logp 0 and no gradient.
 *   target     [M] of target_type; advantage, old_logp, ref_logp fp32 [M]  (device, read)
 *   loss, logp fp32 [M]                                                    (device, written) */
lmhead_status lmhead_policy_forward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                                    const float *bias, lmhead_dtype in_dtype, float temperature, const void *target,
                                    lmhead_index target_type, int64_t ignore_index, const float *advantage,
                                    const float *old_logp, const float *ref_logp, float clip_low, float clip_high,
                                    float kl_coef, float *loss, float *logp, void *state, size_t state_bytes, int keep_logits,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* The logistic loss of preferred pairs. Sequence s is rows starts[s] ..
 * starts[s + 1] - 1 (ascending, within [0, M]; rows in none of them are left out);
 * sequence i is the preferred one of pair i, sequence pairs + i the other.
 *   logp[s] = sum of log q[m, target[m]] over the sequence's rows that are not left
 *             out (as above), or (average != 0) their mean; 0 without any
 *   z = beta ((logp[i] - ref_logp[i]) - (logp[pairs + i] - ref_logp[pairs + i])) - margin
 *   loss[i] = -(1 - label_smoothing) log sigma(z) - label_smoothing log sigma(-z)
 * with ref_logp taken as 0 where NULL; sums and z are fp64.
 *   starts      [2 pairs + 1] of starts_type                    (device, read)
 *   ref_logp    fp32 [2 pairs] or NULL                          (device, read)
 *   loss, logp  fp32 [pairs], [2 pairs]                         (device, written)
 *   0 <= label_smoothing <= 1 */
lmhead_status lmhead_preference_forward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                                        const float *bias, lmhead_dtype in_dtype, float temperature, const void *target,
                                        lmhead_index target_type, int64_t ignore_index, const void *starts,
                                        lmhead_index starts_type, int64_t pairs, const float *ref_logp, float beta,
                                        float margin, float label_smoothing, int average, float *loss, float *logp,
                                        void *state, size_t state_bytes, int keep_logits, void *workspace, size_t workspace_bytes,
                                        void *stream);

/* Gradients of sum_m grad_loss[m] loss[m] (preference: over the pairs) of one of the
 * three calls above, whose state is given and whose other arguments are the same
 * (K: 0 but for lmhead_distill_forward). hidden's values are not read again: the state
 * has the rows that are worked on.
 *   grad_loss   fp32 [M], or [pairs]; NULL: zeros               (device, read)
 *   grad_hidden, grad_W, grad_bias, workspace   as in lmhead_xent_backward, with
 *               lmhead_loss_backward_workspace_bytes(M, H, V, K, keep_logits, grad_bias != NULL)
 *               bytes
 * Rounded and scaled as there, but that in bf16 a target's entry of the logits' gradient, the
 * row's largest by far, is not rounded: grad_hidden's row takes it in fp32, and grad_W's row
 * of the token, rounded once, takes its tokens' entries in fp32 and is rounded again. */
lmhead_status lmhead_loss_backward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                                   const float *bias, lmhead_dtype in_dtype, float temperature, int64_t K,
                                   const float *grad_loss, const void *state, size_t state_bytes, int keep_logits, void *grad_hidden,
                                   void *grad_W, float *grad_bias, void *workspace, size_t workspace_bytes,
                                   void *stream);

/* Host-only: bytes of the state and of the workspaces (0 outside the shape contract or when M == 0). */
size_t lmhead_loss_state_bytes(int64_t M, int64_t H, int64_t V, int64_t K, int keep_logits);
size_t lmhead_loss_forward_workspace_bytes(int64_t M, int64_t H, int64_t V, int64_t K, int with_state);
size_t lmhead_loss_backward_workspace_bytes(int64_t M, int64_t H, int64_t V, int64_t K, int keep_logits,
                                            int grad_bias);

/* The embedding lookup out[m, :] = scale * W[ids[m], :], the product taken at
 * fp32 and rounded once. An id outside [0, V) gives a row of zeros (so a
 * vocabulary shard takes ids - v0 and the shards' results add up).
 *   ids  [M] of ids_type                     (device, read)
 *   W    [V, H] bf16 or fp16 (dtype)         (device, read)
 *   out  [M, H] of dtype                     (device, written)
 * Alignment: W and out 16 bytes. Returns as lmhead_logits_ex. */
lmhead_status lmhead_embed(const void *ids, lmhead_index ids_type, int64_t M, const void *W, int64_t V,
                           int64_t H, lmhead_dtype dtype, float scale, void *out, void *stream);

/* Its gradient: s[v, :] = scale * sum over {m : ids[m] == v} of grad_out[m, :],
 * summed at fp32 in an order that depends on ids only (the same bits every
 * run). Ids outside [0, V) and ids equal to padding_index (pass a value
 * outside [0, V) for none) have no gradient.
 *   grad_out    [M, H] bf16 or fp16 (dtype)   (device, read)
 *   accumulate  0: grad_W = s, every row written; else grad_W += s (one fp32
 *               addition and one rounding; rows without an id are not touched):
 *               the gradient of a head tied to the embedding is
 *               lmhead_xent_backward's with this added
 *   grad_W      [V, H] of dtype               (device, written, or read and written)
 *   workspace   at least lmhead_embed_backward_workspace_bytes(M, H) bytes,
 *               256-byte aligned, overwritten; not in use by other work until
 *               this call's work has finished */
lmhead_status lmhead_embed_backward(const void *ids, lmhead_index ids_type, int64_t M, const void *grad_out,
                                    int64_t V, int64_t H, lmhead_dtype dtype, float scale,
                                    int64_t padding_index, int accumulate, void *grad_W, void *workspace,
                                    size_t workspace_bytes, void *stream);

/* Host-only: bytes of workspace lmhead_embed_backward needs (0 outside the shape contract). */
size_t lmhead_embed_backward_workspace_bytes(int64_t M, int64_t H);

/* Rows to int8: scales[r] = max |x[r, :]| / 127 (1 where that is 0),
 * codes[r, k] = x[r, k] / scales[r] rounded to nearest even, in [-127, 127];
 * binary32 operations, the division correctly rounded. Tokens (one scale per
 * token) and weights (one per vocabulary row) alike.
 *   x       [rows, H] bf16 or fp16 (dtype), finite   (device, read)
 *   codes   int8 [rows, H]                           (device, written)
 *   scales  fp32 [rows]                              (device, written)
 * Alignment: x and codes 16 bytes. Shapes as for the projection with M = rows. */
lmhead_status lmhead_quantize_int8(const void *x, int64_t rows, int64_t H, lmhead_dtype dtype, int8_t *codes,
                                   float *scales, void *stream);

/* The int8 head: t = fl32(fl32(float(sum_k hidden[m, k] W[v, k]) * hidden_scale[m]) * w_scale[v]),
 * then alpha and bias as in lmhead_logits. The integer sum is exact, so a
 * row's logits depend on nothing but the row, whatever M.
 *   hidden int8 [M, H], hidden_scale fp32 [M]   (device, read)
 *   W      int8 [V, H], w_scale fp32 [V]        (device, read)
 *   out_dtype  LMHEAD_F32, LMHEAD_BF16 or LMHEAD_F16 (rounded to nearest even)
 *   out    [M, V] of out_dtype                  (device, written)
 * Alignment: hidden, W and out 16 bytes. */
lmhead_status lmhead_logits_int8(const int8_t *hidden, const float *hidden_scale, int64_t M, int64_t H,
                                 const int8_t *W, const float *w_scale, int64_t V, float alpha,
                                 const float *bias, lmhead_dtype out_dtype, void *out, void *stream);

/* Host-only shape predicate (no device access): 1 when (M, H, V) is inside the
 * shape contract of the bf16 (nvfp4 = 0) or NVFP4 (nvfp4 = 1) entry point,
 * else 0. Like the shape check the metrale page's install step runs before
 * enabling its row-tile head. */
int lmhead_shape_ok(int64_t M, int64_t H, int64_t V, int nvfp4);

/* Host-only: the lmhead_path the AUTO choice takes for this shape, or
 * LMHEAD_PATH_NONE when the shape is outside the contract. The tests use it
 * to assert which kernel a call takes, as the sglang PR 32370 digest's test
 * changes (test coverage of test_fp32_lm_head.py: the probe_mm interceptor
 * asserts which torch operation, input dtype and out_dtype a call used, and a
 * fallback case checks the explicit-fp32 path) check the path as well as the
 * values. */
int lmhead_path_for(int64_t M, int64_t H, int64_t V, int nvfp4);

/* Static, human-readable name of a status code. */
const char *lmhead_status_string(int status);

/* Library version string, "major.minor.patch". */
const char *lmhead_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LMHEAD_H */
