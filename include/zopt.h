/*
 * zopt.h -- one data-parallel rank's optimizer step under ZeRO-style
 * sharding, on AMD Instinct MI355X (gfx950).
 *
 * libzopt holds two optimizers that a ZeRO-sharded trainer runs on each rank
 * after its gradients are in place:
 *
 *  - zopt_adamw_shard_step: AdamW over the rank's flat, bucket-padded fp32
 *    master shard, in one pass that reads the bf16 gradient, updates the fp32
 *    master and both fp32 moments, and writes the bf16 compute weights;
 *  - zopt_muon_step: Muon on whole 2-D matrices the rank owns (momentum with
 *    Nesterov look-ahead, Newton-Schulz orthogonalisation on bf16 matrix
 *    cores, a decayed and scaled update of the fp32 master), and
 *    zopt_muon_step_groups, the same on several shapes in one call, with
 *    zopt_muon_step_groups_guarded adding the Newton-Schulz health checks,
 *    and zopt_muon_graph_* capturing a call once for replay each step;
 *  - zopt_round_bf16: the fp32 -> bf16 round-to-nearest-even write-back on
 *    its own;
 *  - zopt_grad_sq_norm, zopt_grad_clip_stats and zopt_adamw_shard_step_clipped:
 *    the gradient norm of the shard, the clip statistics, and the AdamW step
 *    taking its gradient scale from them in device memory;
 *
 * and the operators that produce its gradients where memory is shortest:
 * zopt_linear_xent (a vocabulary projection's loss and gradients; the caller
 * holds no logits), zopt_glu_forward / zopt_glu_backward (the gated feed-forward) and
 * zopt_act8_* (activation checkpoints in 8 bits); zopt_qk_norm_rope (norms and
 * rotation of queries and keys) and zopt_moe_* (routing to experts and the
 * experts' gated feed-forward), forward and backward.
 *
 * Conventions common to every call
 * --------------------------------
 *  - Every buffer is device memory owned by the caller.  The library
 *    allocates no device memory at run time and keeps no state between calls,
 *    with five exceptions: a captured Muon graph is a handle the caller owns;
 *    zopt_set_ns_workgroup_limit is a process-wide setting that every later
 *    call in the process uses (one thread's setting changes the launch plan,
 *    never the results, of another's calls); zopt_set_ns_form is another,
 *    which selects how Newton-Schulz is computed (and so changes results
 *    within bf16 rounding, and the workspace size); zopt_grad_sq_norm_noalloc
 *    uses a 16 KiB array per GPU that the library holds for the life of the
 *    process; and a grouped Muon call whose Newton-Schulz launches are short
 *    (see zopt_muon_step_groups) uses a second stream per GPU, with two
 *    events, that the library creates at the first such call and holds for
 *    the life of the process.  Every other call is reentrant.
 *  - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream) and
 *    the call returns without synchronising.  All launch parameters travel
 *    as kernel arguments, so back-to-back calls need no host sync.
 *  - Arguments are checked before anything is enqueued.  On any status other
 *    than ZOPT_OK nothing has been enqueued and no buffer has been touched,
 *    except ZOPT_ERR_DEVICE, which reports a failed launch.
 *  - NaN and Inf in the data are not reported; they propagate as IEEE
 *    arithmetic dictates.
 *  - Buffers must not overlap.  No alignment is required; bases aligned to
 *    16 bytes take the 128-bit vector path.
 *  - bf16 is the upper half of an IEEE binary32, carried as uint16_t.
 *  - Rounding to bf16 is round-to-nearest, ties to even, with no flush of
 *    subnormals; a value beyond the largest finite bf16 becomes infinity and
 *    a NaN becomes 0x7FC0 -- what a cast of an fp32 tensor to bf16 yields
 *    [DEG zero.py, ZeroMaster docstring and gather_params: the updated shard
 *    is rounded to bf16, bitwise the unsharded trainer's copy of the master
 *    into the bf16 weights].
 *  - Per-step scalars derived from the hyperparameters are formed in double
 *    on the host and rounded once to binary32; the optimizers' elementwise
 *    arithmetic is binary32 with no fused multiply-adds, in the order stated
 *    below.
 */
#ifndef ZOPT_H
#define ZOPT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ZOPT_OK = 0,
    ZOPT_ERR_NULL = 1,      /* a required pointer is NULL                       */
    ZOPT_ERR_SIZE = 2,      /* a size, count, rank or shard length is invalid   */
    ZOPT_ERR_HYPER = 3,     /* a hyperparameter is out of its domain            */
    ZOPT_ERR_WORKSPACE = 4, /* workspace too small or not 256-byte aligned      */
    ZOPT_ERR_DEVICE = 5     /* the HIP runtime reported a launch failure        */
} zopt_status;

/* A static, human-readable name of a status code. */
const char *zopt_status_string(zopt_status status);

/*
 * zopt_adamw_shard_step -- one AdamW step over rank `rank`'s shard.
 *
 * Layout [DEG zero.py: ZeroMaster module docstring, ZeroMaster.__init__,
 * reduce_scatter, gather_params].  The trainable parameters lie end to end in
 * a flat vector of N elements.  The bucket length is lowered to a multiple of
 * `world` (never below `world`): B = max(world, bucket - bucket % world).
 * Buckets [s, e) tile [0, N); bucket b has padded length
 * L_b = ceil((e - s) / world) * world and is cut into `world` equal pieces
 * of p_b = L_b / world elements.  Rank r owns piece r of every bucket; its
 * shard is those pieces concatenated, so shard_len = sum_b p_b.  Shard
 * element j of bucket b (shard offset o_b = sum of earlier pieces) is flat
 * element f = s_b + r * p_b + (j - o_b); it is padding when f >= e_b.
 *
 * Per shard element, in this order [dmuon PR #16, commit "foreach AdamW":
 * decoupled weight decay, then the moments, then the bias-corrected addcdiv,
 * bias corrections being per-step scalars of the post-increment step;
 * BluScript trainer source, optimizer-precision note: the decay is a
 * (1 - lr*wd) multiply on fp32 masters and moments; DeepSpeed PR #9021,
 * commits "bf16 gradients of fp32 params" (the bf16 gradient is promoted in
 * registers) and "grad_scale" (multiplied as each element is loaded, after
 * the promotion)]:
 *
 *   g  = fp32(grad[f]) * grad_scale          (g = 0 on padding)
 *   p  = p * decay
 *   m  = beta1 * m + omb1 * g
 *   v  = beta2 * v + (omb2 * g) * g
 *   p  = p - step_size * (m / (sqrt(v) / bc2_sqrt + eps))
 *   weight[f] = bf16(p)                      (real elements only)
 *
 * with t = step and, in double rounded once to binary32,
 *   step_size = lr / (1 - beta1^t),  bc2_sqrt = sqrt(1 - beta2^t),
 *   decay = 1 - lr * weight_decay,   omb1 = 1 - beta1,  omb2 = 1 - beta2.
 * The gradient here is this rank's contribution as it stands: the sum over
 * ranks (a reduce-scatter) is not part of this call; an average over ranks
 * is grad_scale = 1/world.
 *
 * Arguments
 *   master, exp_avg, exp_avg_sq  fp32 [shard_len], device, read and written.
 *                                Padding positions are stepped with g = 0.
 *   grad      bf16 [N] flat gradient, device, read only at this rank's real
 *             elements.
 *   weight    bf16 [N] flat compute weights, device, written only at this
 *             rank's real elements; NULL skips the write-back.
 *   N, bucket, world, rank, shard_len   the layout above; shard_len must equal
 *             the value it derives from (N, bucket, world).
 *   lr, beta1, beta2, eps, weight_decay, step, grad_scale   as above; step
 *             is 1 on the first update (already incremented by the caller).
 *   stream    hipStream_t or NULL.
 *
 * Errors: ZOPT_ERR_NULL (master, exp_avg, exp_avg_sq or grad NULL);
 * ZOPT_ERR_SIZE (N < 1, bucket < 1, world < 1, rank outside [0, world),
 * shard_len wrong); ZOPT_ERR_HYPER (lr < 0 or not finite, beta outside
 * [0, 1), eps <= 0 or not finite, weight_decay < 0 or not finite, step < 1,
 * grad_scale not finite); ZOPT_ERR_DEVICE.
 */
zopt_status zopt_adamw_shard_step(float *master, float *exp_avg, float *exp_avg_sq,
                                  const uint16_t *grad, uint16_t *weight,
                                  int64_t N, int64_t bucket, int32_t world,
                                  int32_t rank, int64_t shard_len,
                                  float lr, float beta1, float beta2, float eps,
                                  float weight_decay, int64_t step, float grad_scale,
                                  void *stream);

/*
 * Gradient clipping without a host round trip.  A ZeRO rank clips on the
 * norm of the whole summed gradient: each rank squares and sums its own real
 * gradient elements, the ranks' sums are added (an all-reduce, not part of
 * this library), and the clip coefficient derived from the total scales the
 * gradient as the AdamW step loads it [DEG zero.py: ZeroMaster.grad_sq_norm;
 * BluScript trainer source, cross-group global clipping block: coefficient
 * min(1, clip / (norm + 1e-6)), and the Muon path does not apply it; DeepSpeed
 * PR #9021, commit "grad_scale": the factor is multiplied in as each gradient
 * element is loaded].  The statistics stay in device memory as binary32
 * scalars, so nothing waits for the host [dmuon PR #16, commit "device-tensor
 * stats": total_norm / clip_coef / clipped / found_inf as device scalars,
 * finiteness judged on the norm, so an infinite norm reports found_inf and
 * not clipped].  A clipped step is three calls on one stream:
 *
 *   zopt_grad_sq_norm(grad, ..., sq, ws, &ws_bytes, s);     per rank
 *   (all-reduce sq over ranks, or pass the per-rank sums to the next call)
 *   zopt_grad_clip_stats(sq, 1, max_norm, inv_scale, stats, s);
 *   zopt_adamw_shard_step_clipped(..., stats, skip_nonfinite, s);
 */

/* Layout of the clip statistics: ZOPT_CLIP_STATS binary32 values. */
enum {
    ZOPT_CLIP_TOTAL_NORM = 0, /* fp32(sqrt(sum of squares) * inv_scale)            */
    ZOPT_CLIP_COEF = 1,       /* min(1, max_norm / (total_norm + 1e-6)), binary32   */
    ZOPT_CLIP_CLIPPED = 2,    /* 1 if !found_inf and clip_coef < 1, else 0          */
    ZOPT_CLIP_FOUND_INF = 3,  /* 1 if total_norm is not finite, else 0              */
    ZOPT_CLIP_GRAD_SCALE = 4, /* inv_scale * clip_coef: the AdamW gradient factor   */
    ZOPT_CLIP_STATS = 5
};

/*
 * zopt_grad_sq_norm -- *sq = the sum of the squares of rank `rank`'s real
 * gradient elements (the layout of zopt_adamw_shard_step; padding and other
 * ranks' positions are not read).  Each square is exact in double and the sum
 * is double, in an order fixed by shard_len alone: the result is the same on
 * every run.
 *
 * Arguments
 *   grad      bf16 [N] flat gradient, device, read.
 *   N, bucket, world, rank, shard_len   as for zopt_adamw_shard_step.
 *   sq        one double, device, written.
 *   workspace device scratch, 256-byte aligned, of at least the size the
 *             NULL-workspace query writes to *workspace_bytes (at most 16 KiB);
 *             with workspace == NULL the call only writes that size.
 *   stream    hipStream_t or NULL.
 *
 * Errors: ZOPT_ERR_NULL (workspace_bytes NULL; grad or sq NULL with a
 * workspace); ZOPT_ERR_SIZE (the layout arguments as for
 * zopt_adamw_shard_step); ZOPT_ERR_WORKSPACE; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_grad_sq_norm(const uint16_t *grad, int64_t N, int64_t bucket, int32_t world,
                              int32_t rank, int64_t shard_len, double *sq, void *workspace,
                              size_t *workspace_bytes, void *stream);

/*
 * zopt_grad_sq_norm_noalloc -- zopt_grad_sq_norm for callers that cannot
 * allocate device memory (code under stream capture, tight training loops,
 * harnesses that forbid allocation): the same sum, bit for bit, with the
 * partial sums kept in a scratch array inside the library instead of a
 * caller's workspace.  The array is 16 KiB per GPU (2048 doubles, the most
 * partials any shard length needs), allocated when the library is loaded and
 * held until the process ends; the call itself allocates nothing.  Every
 * call on one GPU uses that GPU's one array, so calls that may overlap on a
 * GPU (different streams, or different host threads without ordering) race
 * and must not be issued; calls in one stream are ordered and safe.  The
 * array needs no clearing: each call writes every partial it reads.
 *
 * Arguments as zopt_grad_sq_norm, without workspace and workspace_bytes.
 *
 * Errors: ZOPT_ERR_NULL (grad or sq NULL); ZOPT_ERR_SIZE (the layout
 * arguments as for zopt_adamw_shard_step); ZOPT_ERR_WORKSPACE (the partials
 * would exceed the array -- no valid layout does); ZOPT_ERR_DEVICE (the
 * array's address could not be found on the current device, or a launch
 * failed).
 */
zopt_status zopt_grad_sq_norm_noalloc(const uint16_t *grad, int64_t N, int64_t bucket,
                                      int32_t world, int32_t rank, int64_t shard_len,
                                      double *sq, void *stream);

/*
 * zopt_grad_clip_stats -- the clip statistics (layout above) from `count`
 * sums of squares, added in index order in double:
 *   total_norm = fp32(sqrt(sum) * inv_scale)
 *   clip_coef  = min(1, max_norm / (total_norm + 1e-6f)), binary32; an
 *                infinite norm gives 0, a NaN norm gives NaN
 *   clipped    = !found_inf && clip_coef < 1,  found_inf = !isfinite(total_norm)
 *   grad_scale = inv_scale * clip_coef
 *
 * Arguments
 *   sq         `count` doubles, device, read (per-rank sums, or one total).
 *   count      1 .. 65536.
 *   max_norm   > 0 (+inf reports the norm without clipping).
 *   inv_scale  finite, > 0: the gradients are a loss scale times the true
 *              ones; 1 = none.
 *   stats      ZOPT_CLIP_STATS floats, device, written.
 *   stream     hipStream_t or NULL.
 *
 * Errors: ZOPT_ERR_NULL; ZOPT_ERR_SIZE (count); ZOPT_ERR_HYPER (max_norm,
 * inv_scale); ZOPT_ERR_DEVICE.
 */
zopt_status zopt_grad_clip_stats(const double *sq, int32_t count, float max_norm,
                                 float inv_scale, float *stats, void *stream);

/*
 * zopt_adamw_shard_step_clipped -- zopt_adamw_shard_step with grad_scale
 * read from device memory when the kernel runs: grad_scale =
 * clip_stats[ZOPT_CLIP_GRAD_SCALE].  With skip_nonfinite = 1 a step whose
 * clip_stats[ZOPT_CLIP_FOUND_INF] is non-zero writes nothing (master, moments
 * and weights keep their values); the step count is the caller's, who may
 * read found_inf later and not count that step.  Every other argument,
 * and the arithmetic, as zopt_adamw_shard_step: given the same grad_scale
 * value the two calls give the same bits.
 *
 * Errors: those of zopt_adamw_shard_step; ZOPT_ERR_NULL also for clip_stats
 * NULL; ZOPT_ERR_HYPER also for skip_nonfinite not 0/1.
 */
zopt_status zopt_adamw_shard_step_clipped(float *master, float *exp_avg, float *exp_avg_sq,
                                          const uint16_t *grad, uint16_t *weight, int64_t N,
                                          int64_t bucket, int32_t world, int32_t rank,
                                          int64_t shard_len, float lr, float beta1, float beta2,
                                          float eps, float weight_decay, int64_t step,
                                          const float *clip_stats, int32_t skip_nonfinite,
                                          void *stream);

/*
 * zopt_shard_len -- the shard length every rank holds for a flat vector of N
 * elements in buckets of `bucket` over `world` ranks (the layout above:
 * sum over buckets of ceil(len_b / world)).  Host-only; enqueues nothing.
 * Returns -1 if N < 1, bucket < 1 or world < 1.
 */
int64_t zopt_shard_len(int64_t N, int64_t bucket, int32_t world);

/*
 * zopt_muon_step -- one Muon step on `batch` matrices of one stored shape
 * [rows, cols] (row-major, PyTorch's [out, in]), each owned whole by this
 * rank [BluScript trainer source, ShardedMuon comment block: Newton-Schulz is
 * a whole-matrix operator, so Muon shards by whole parameter, the owner
 * holding the matrix's fp32 master and momentum; dmuon PR #16, commit "NS
 * CUDA-graph replay": Newton-Schulz runs on a small stable set of shapes,
 * lr / wd / momentum stay in the pre- and post-steps around it].
 *
 * Per matrix, in this order:
 *   1. Momentum [BluScript trainer source, Muon config block: momentum 0.95,
 *      Nesterov; the buffer is an exponential moving average]:
 *        g = fp32(grad);  M = mu * M + omm * g;
 *        U = omm * g + mu * M  (nesterov)   or   U = M   (otherwise)
 *      with mu = momentum_beta and omm = fp32(1 - mu) formed in double.
 *   2. Pre-scale: X0 = s U, s = 1 / (||U||_F + ns_eps), ||U||_F^2 a
 *      fixed-order (run-to-run deterministic) fp64 sum of the exact squares
 *      and s formed in double; X0 is taken transposed when rows > cols, so X
 *      is m x n with m = min(rows, cols).  With ns_steps = 0,
 *      X0 = bf16(U * s) (the product in double) is the result.  Otherwise,
 *      when 2^-60 <= ||U||_F^2 <= 2^100, X0 is never stored: the first
 *      iteration reads bf16(U) and applies s in fp32 to its products (s^2 to
 *      X X^T, s to B X), which in that range can neither overflow nor lose
 *      precision to underflow; outside it (huge or tiny gradients, Inf, NaN)
 *      X0 = bf16(U * s) is written first and the iteration reads that.
 *   3. ns_steps Newton-Schulz iterations [BluScript trainer source, ShardedMuon
 *      comment block: X <- aX + (bXX' + c(XX')^2)X]:
 *        A = X X^T;  B = b A + c A A;  X = a X + B X
 *      on bf16 matrix cores with fp32 accumulation; A, B and X are rounded to
 *      bf16 after each product; only the upper triangle of the symmetric A
 *      and B is computed and mirrored.  Where the long side is at least twice
 *      the short one (n >= 2 m), m <= 4096 and the group is large enough for
 *      the flops saved to pay for two more launches (batch m^2 (n - m) >=
 *      2^29; a rule on the group alone) the same polynomial map runs in
 *      segments of
 *      up to three steps on the m x m Gram matrix: with A_j = X_j X_j^T and
 *      P_j = a I + b A_j + c A_j^2, X_{j+1} = P_j X_j gives A_{j+1} =
 *      P_j^2 A_j and X_L = (P_{L-1} ... P_0) X_0, so a segment forms X X^T
 *      once and multiplies X by one m x m matrix; every other product is of
 *      two commuting symmetric m x m matrices (upper triangle computed), and
 *      the chain of them is held in fp16 where the coefficients allow
 *      (zopt_set_ns_form), with the final m x m factor rounded to bf16.  Five
 *      steps are segments of 3 and 2: 6 m^2 n + 14 m^3 flops against
 *      15 m^2 n + 5 m^3.  Each segment restarts from its X, which keeps the
 *      bf16 rounding of the m x m chain from compounding.  The two forms
 *      agree to within bf16 rounding, not bit for bit; zopt_set_ns_form
 *      selects plain iterations for every matrix.  Every symmetric m x m
 *      matrix is held as a bf16 off-diagonal part and an fp32 diagonal.
 *   4. Post-step [BluScript trainer source, Muon config block (weight decay
 *      pinned to AdamW's) and the note beside the MuonAdjustLr choice]:
 *        P = P * decay - step_lr * fp32(O),  weight = bf16(P)
 *      with O the result of step 3 in the stored orientation and, in double
 *      rounded once to binary32, decay = 1 - lr * weight_decay and
 *      step_lr = lr * scale, scale = 0.2 * sqrt(max(rows, cols)) when
 *      adjust_lr = 1 (the update's entry RMS matches AdamW's 0.2) or
 *      sqrt(max(1, rows / cols)) when adjust_lr = 0 (the original convention).
 *
 * Arguments
 *   batch        1 .. 64 matrices.
 *   rows, cols   the stored shape, >= 1, rows * cols < 2^31 and
 *                max(rows, cols) <= 2^21 (2,097,152: the kernels address a
 *                row panel of the padded matrix with 32-bit byte offsets).
 *   master, momentum   host arrays of `batch` device pointers, fp32
 *                [rows * cols] each, read and written.
 *   grad         host array of `batch` device pointers, bf16 [rows * cols].
 *   weight       host array of `batch` device pointers, bf16 [rows * cols],
 *                written; NULL skips the write-back (if non-NULL, every entry
 *                must be non-NULL).
 *   lr, momentum_beta, nesterov (0/1), weight_decay, ns_steps (0 .. 100),
 *   ns_a, ns_b, ns_c, ns_eps, adjust_lr (0/1)   as above.
 *   workspace    device scratch, 256-byte aligned, of at least the size the
 *                NULL-workspace query returns.  With workspace == NULL the call
 *                only writes that size to *workspace_bytes and returns ZOPT_OK.
 *                Otherwise *workspace_bytes is the size provided.  The
 *                workspace's contents need no initialisation; after the call,
 *                zopt_muon_output_view locates the step-3 result in it.
 *   stream       hipStream_t or NULL.
 *
 * Errors: ZOPT_ERR_NULL (a pointer array or one of its entries NULL,
 * workspace_bytes NULL); ZOPT_ERR_SIZE (batch, rows, cols out of range);
 * ZOPT_ERR_HYPER (lr or weight_decay < 0 or not finite, momentum_beta outside
 * [0, 1), nesterov or adjust_lr not 0/1, ns_steps outside [0, 100], a
 * coefficient not finite, ns_eps < 0 or not finite); ZOPT_ERR_WORKSPACE;
 * ZOPT_ERR_DEVICE.
 */
zopt_status zopt_muon_step(int32_t batch, int64_t rows, int64_t cols,
                           float *const *master, float *const *momentum,
                           const uint16_t *const *grad, uint16_t *const *weight,
                           float lr, float momentum_beta, int32_t nesterov,
                           float weight_decay, int32_t ns_steps,
                           float ns_a, float ns_b, float ns_c, float ns_eps,
                           int32_t adjust_lr, void *workspace, size_t *workspace_bytes,
                           void *stream);

/*
 * zopt_muon_output_view -- where the orthogonalised update O of matrix
 * `index` lies in a workspace that zopt_muon_step(batch, rows, cols, ...,
 * ns_steps, ...) has filled: bf16 O[r][c] (stored orientation, [rows, cols])
 * is at (*out)[r * (*row_stride) + c].  Host-only; enqueues nothing.  The view
 * is valid until the workspace is reused, and assumes the Newton-Schulz form
 * (zopt_set_ns_form) in effect when the workspace was filled: the form decides
 * which buffer holds the result.  Errors: ZOPT_ERR_NULL,
 * ZOPT_ERR_SIZE (batch, rows, cols or index out of range), ZOPT_ERR_HYPER
 * (ns_steps out of range).
 */
zopt_status zopt_muon_output_view(int32_t batch, int64_t rows, int64_t cols,
                                  int32_t ns_steps, const void *workspace,
                                  int32_t index, const uint16_t **out,
                                  int64_t *row_stride);

/*
 * zopt_muon_step_groups -- zopt_muon_step on `ngroups` groups of matrices in
 * one call.  A rank's Muon parameters fall into a few stored shapes, and
 * launch count is what limits a per-shape loop of small steps [dmuon PR #16,
 * commit "NS CUDA-graph replay": one rank steps tens of Muon matrices of a
 * small, stable set of shapes, and the launches issued per step dominated its
 * host time].  Here every Newton-Schulz product of every group whose short
 * side selects the same output tile is one launch, so small groups share the
 * GPU instead of running one after another.  Each matrix gets exactly the
 * arithmetic zopt_muon_step gives it; the call equals ngroups separate
 * zopt_muon_step calls, except that the groups' Newton-Schulz products
 * interleave in time.
 *
 * Short launches on two streams: when the groups on 256 x 256 output tiles
 * give the X X^T launch fewer than two rounds of workgroups (2 x 256 on a
 * 256-CU GPU), each product's launch would leave much of the GPU idle in its
 * last round.  The groups then run on `stream` and on a second stream of the
 * library's.  In a call that mixes the two forms of step 3, the groups of one
 * form and output tile stay on one stream (they share its launches), these
 * classes placed by Newton-Schulz work (largest first, each to the stream
 * with less); in a call of one form the groups are placed so one by one.  The
 * side estimated to take longer runs on `stream`.  Each group's momentum
 * pass, iterations and (with no health pass) post-step run on its side's
 * stream: the second stream waits (an event) for everything enqueued on
 * `stream` before the call and for the momentum passes of `stream`'s groups,
 * and `stream` waits for the second stream's last launch (another event)
 * before the health pass, or at the end of the call, so the call is ordered
 * on `stream` as any other.  The results are the same bit for bit.  The
 * second stream is
 * created at the first such call on the GPU that is not under stream capture
 * (a call under capture before that runs on one stream) and by
 * zopt_muon_graph_create before its capture; calls from several host threads
 * enqueue this part one at a time (a lock), and their work on the second
 * stream runs in that order.  Measured on the 1B rank-0 share (12 matrices,
 * four groups): 2.81 -> 2.58 ms per five-step call with the division by
 * class (3.49 -> 3.05 ms when two streams first replaced one).
 *
 * Arguments
 *   ngroups      1 .. 16.
 *   batch, rows, cols   host arrays of `ngroups` entries; group g has
 *                batch[g] (1 .. 64) matrices of stored shape
 *                [rows[g], cols[g]] with the limits of zopt_muon_step.
 *   master, momentum, grad, weight   host arrays of sum(batch) device
 *                pointers, group 0's matrices first, then group 1's, ...;
 *                weight may be NULL (no write-back for any group).
 *   lr ... stream      as for zopt_muon_step, shared by all groups.
 *   workspace    as for zopt_muon_step; the NULL-workspace query returns the
 *                size for all groups together (the sum of the per-group sizes).
 *
 * Errors: those of zopt_muon_step; ZOPT_ERR_NULL also if batch, rows or cols
 * is NULL, ZOPT_ERR_SIZE if ngroups is out of range.
 */
zopt_status zopt_muon_step_groups(int32_t ngroups, const int32_t *batch, const int64_t *rows,
                                  const int64_t *cols, float *const *master,
                                  float *const *momentum, const uint16_t *const *grad,
                                  uint16_t *const *weight, float lr, float momentum_beta,
                                  int32_t nesterov, float weight_decay, int32_t ns_steps,
                                  float ns_a, float ns_b, float ns_c, float ns_eps,
                                  int32_t adjust_lr, void *workspace, size_t *workspace_bytes,
                                  void *stream);

/*
 * zopt_muon_step_groups_guarded -- zopt_muon_step_groups with the Newton-Schulz
 * health checks [BluScript trainer source, per-step report: nsratio, the
 * worst ||update||_F / sqrt(min(rows, cols)) among the applied updates (about
 * 1 when healthy), and nsrej, the updates the divergence guard refused because
 * an element exceeded 1000 in magnitude; dmuon PR #16, commit "device-tensor
 * stats": diagnostics stay device scalars, read back on the caller's
 * schedule].  After step 3, per matrix i of the call (in call order), from its
 * bf16 result O:
 *   ratio_i    = ||O||_F / sqrt(min(rows, cols)), the squares summed exactly
 *                in double in a fixed order, formed in double, rounded once
 *   absmax_i   = max |O_jk| (NaN if an element is NaN)
 *   rejected_i = !(absmax_i <= ns_guard)
 * A rejected matrix is not updated: step 4 leaves its master and weight as
 * they were (its momentum has taken step 1).  The other matrices get exactly
 * what zopt_muon_step_groups gives them.
 *
 * Arguments: those of zopt_muon_step_groups, and
 *   ns_guard   > 0; 1000 is the pages' value; +inf only reports.
 *   ns_health  device floats, written: [0] the number of matrices rejected,
 *              [1] the worst ratio among those not rejected (0 if none), then
 *              [2 + 3i .. 4 + 3i] = ratio_i, absmax_i, rejected_i (0 / 1) for
 *              each of the sum(batch) matrices.
 *
 * Errors: those of zopt_muon_step_groups; with a workspace, ZOPT_ERR_NULL also
 * for ns_health NULL and ZOPT_ERR_HYPER for ns_guard not > 0.
 */
zopt_status zopt_muon_step_groups_guarded(int32_t ngroups, const int32_t *batch,
                                          const int64_t *rows, const int64_t *cols,
                                          float *const *master, float *const *momentum,
                                          const uint16_t *const *grad, uint16_t *const *weight,
                                          float lr, float momentum_beta, int32_t nesterov,
                                          float weight_decay, int32_t ns_steps, float ns_a,
                                          float ns_b, float ns_c, float ns_eps, int32_t adjust_lr,
                                          float ns_guard, float *ns_health, void *workspace,
                                          size_t *workspace_bytes, void *stream);

/*
 * Captured Muon calls.  One Muon call is tens of kernel launches; issued one
 * by one per step they cost host time that a graph replay does not [dmuon PR
 * #16, commit "NS CUDA-graph replay": the launches of a Newton-Schulz call
 * captured once per shape and replayed, cutting the host cost of a call from
 * milliseconds to tens of microseconds; lr / wd / momentum are kept out of
 * the captured part so a schedule needs no re-capture].  Here the whole call
 * (pre-step, Newton-Schulz, optional health pass, post-step) is one hipGraph,
 * and lr, momentum_beta and weight_decay live in device memory, read by the
 * kernels each time the graph runs: a caller changes them with an ordinary
 * device write (a copy or a fill on the stream) before a launch.
 *
 *   scalars  device float[3] = {lr, momentum_beta, weight_decay}.  Read when
 *            the kernels run; the library cannot check these values (they
 *            should satisfy zopt_muon_step's limits).  Every derived scalar
 *            (1 - mu, 1 - lr*wd, lr*scale) is formed in double on the device
 *            exactly as the host forms it, so a replay gives the bits a
 *            zopt_muon_step_groups(_guarded) call with the same values gives.
 *
 * zopt_muon_graph_create captures one call with the arguments of
 * zopt_muon_step_groups_guarded (ns_health NULL: no health pass, ns_guard
 * ignored) -- the buffers, shapes, workspace and fixed hyperparameters are
 * baked in and must stay valid while the graph is used -- and returns a
 * handle.  Capture runs on a stream of its own and enqueues nothing (a call
 * split over two streams is captured with its fork and join).
 * workspace_bytes is the size provided (the query of zopt_muon_step_groups
 * gives the size needed).  Errors: ZOPT_ERR_NULL (graph, workspace, scalars
 * or a buffer pointer NULL); ZOPT_ERR_SIZE; ZOPT_ERR_HYPER (nesterov,
 * ns_steps, a coefficient, ns_eps, adjust_lr, or ns_guard with ns_health);
 * ZOPT_ERR_WORKSPACE; ZOPT_ERR_DEVICE (capture or instantiation failed).
 *
 * zopt_muon_graph_launch enqueues one replay on `stream` (hipStream_t or
 * NULL).  Replays on one workspace must not overlap (one stream, or ordered).
 *
 * zopt_muon_graph_destroy frees the handle (NULL is a no-op); no replay may
 * still be pending (synchronise the stream first).  The handle is host
 * memory owned by the caller until then; the library holds no other state.
 */
typedef struct zopt_muon_graph zopt_muon_graph;

zopt_status zopt_muon_graph_create(int32_t ngroups, const int32_t *batch, const int64_t *rows,
                                   const int64_t *cols, float *const *master,
                                   float *const *momentum, const uint16_t *const *grad,
                                   uint16_t *const *weight, const float *scalars,
                                   int32_t nesterov, int32_t ns_steps, float ns_a, float ns_b,
                                   float ns_c, float ns_eps, int32_t adjust_lr, float ns_guard,
                                   float *ns_health, void *workspace, size_t workspace_bytes,
                                   zopt_muon_graph **graph);
zopt_status zopt_muon_graph_launch(const zopt_muon_graph *graph, void *stream);
zopt_status zopt_muon_graph_destroy(zopt_muon_graph *graph);

/*
 * zopt_muon_groups_output_view -- zopt_muon_output_view for matrix `index` of
 * group `group` of a workspace that zopt_muon_step_groups(ngroups, batch,
 * rows, cols, ..., ns_steps, ...) has filled.  Host-only.  Errors as
 * zopt_muon_output_view; ZOPT_ERR_SIZE also for `group` out of range.
 */
zopt_status zopt_muon_groups_output_view(int32_t ngroups, const int32_t *batch,
                                         const int64_t *rows, const int64_t *cols,
                                         int32_t ns_steps, const void *workspace, int32_t group,
                                         int32_t index, const uint16_t **out,
                                         int64_t *row_stride);

/*
 * zopt_round_bf16 -- dst[i] = bf16(src[i]) for i in [0, n), round to
 * nearest even as above [DEG zero.py, gather_params: the updated fp32 shard
 * cast to the bf16 compute dtype].
 *   src  fp32 [n], device, read.   dst  bf16 [n], device, written.
 *   n    >= 0; n = 0 enqueues nothing.
 * Errors: ZOPT_ERR_NULL (src or dst NULL with n > 0); ZOPT_ERR_SIZE (n < 0);
 * ZOPT_ERR_DEVICE.
 */
zopt_status zopt_round_bf16(const float *src, uint16_t *dst, int64_t n, void *stream);

/*
 * zopt_set_ns_workgroup_limit -- caps the workgroups that the Newton-Schulz
 * X' = a X + B X launches keep resident.  Those launches are persistent: one
 * round of workgroups walks all the tiles, each starting its next tile's
 * loads while it finishes the current one.  n = 0 restores the default, one
 * full round of the device (one 256 x 256-tile workgroup per compute unit);
 * n > 0 caps it at max(8, n rounded down to a multiple of 8), which leaves
 * compute units free for work running beside the optimizer (collectives on
 * another stream, say) at a cost in Newton-Schulz time.  Process-wide; it
 * applies to calls enqueued, and graphs captured, after it.  Results do not
 * depend on it: every tile is computed the same way by whichever workgroup.
 * Errors: ZOPT_ERR_SIZE (n < 0).
 */
zopt_status zopt_set_ns_workgroup_limit(int32_t n);

/*
 * zopt_set_ns_form -- the Newton-Schulz form of later calls:
 *   0 (the default) runs the groups that zopt_muon_step's step 3 names
 *     (n >= 2 m, m <= 4096, batch m^2 (n - m) >= 2^29) in segments on the
 *     Gram matrix,
 *     holding a segment's m x m chain in fp16 (3 more mantissa bits than
 *     bf16, the same matrix-core rate) when the coefficients keep every
 *     matrix of the chain below 2^13 in magnitude (checked on the scalar
 *     map over singular values in [0, 1.05]; true for the usual quintic and
 *     cubic coefficients), else in bf16; plain iterations hold A in fp16
 *     under the same condition for m <= 4096 (fp16's subnormal range
 *     begins near the off-diagonal entries of larger matrices' A), in bf16
 *     otherwise;
 *   1 runs plain iterations for every matrix;
 *   2 is form 0 with the chain always in bf16 (for comparison: less
 *     accurate than both others on some inputs).
 * Process-wide; it applies to workspace queries, calls and graph captures
 * made after it.  Forms 0 and 2 need more workspace for those shapes (three
 * more m x m 16-bit matrices and fp32 diagonals per matrix), so a workspace
 * sized under form 1 fails their size check (ZOPT_ERR_WORKSPACE).
 * Errors: ZOPT_ERR_HYPER (form not 0, 1 or 2).
 */
zopt_status zopt_set_ns_form(int32_t form);

/*
 * Gradients of a large vocabulary and of the gated feed-forward block, and
 * activation checkpoints in 8 bits: the operators that produce what the calls
 * above step, where a training rank's memory goes -- the logits, the
 * pre-activations and the activations kept between forward and backward.
 * Their gradients are bf16 and may be written straight into a flat gradient
 * vector (any element offset), such as zopt_adamw_shard_step and
 * zopt_muon_step read.
 *
 * Matrices are row-major; a row stride counts elements between rows (>= the
 * row's length, <= 2^31).  Widths (D, V, F, N, cols) are 1 .. 2^21, rows T
 * 0 .. 2^30.  Products run on bf16 matrix cores with fp32 accumulation; every
 * result is the same on every run.  An operand whose row length, row stride
 * or base is not a multiple of 8 elements (16 bytes) is copied into the
 * workspace first; nothing else depends on alignment but speed.
 *
 * workspace: device scratch, 256-byte aligned, of at least the size that the
 * call with workspace == NULL writes to *workspace_bytes.  That size depends
 * on the sizes, strides, the alignment of the operands and which optional
 * pointers are NULL, so query with the arguments of the call.  Where it is 0
 * the workspace is not touched: any non-NULL, aligned value will do.
 */

/*
 * zopt_linear_xent -- softmax cross entropy of a vocabulary projection, with
 * its gradients, from x and w (the caller forms and holds no logits):
 *   z_tv  = sum_d x_td w_vd                         (fp32, never stored)
 *   row_t = log sum_v exp(z_tv) - z_t,target        (0 for ignored rows)
 *   loss  = s sum_t row_t,   s = 1, or 1 / (rows not ignored) with mean = 1
 *                            (0 where every row is ignored)
 *   P_tv  = softmax(z_t)_v - [v = target_t]         (0 for ignored rows)
 *   dx    = s grad_scale P w,   dw = s grad_scale P^T x
 * With a gradient the workspace holds an exponential for every logit of a
 * piece of rows, in 16 bits (fp16, relative to the largest of 64 neighbouring
 * logits): as much as the piece's logits in bf16 would take, at most 2 GiB, so
 * that each of the call's three products is computed once.  The loss alone
 * keeps none.  P is rounded to bf16 for the last two products; the error of dx
 * and dw is about 1.2 times that of one rounding to bf16.  No row's loss is
 * negative.
 *
 * Arguments
 *   x       bf16 [T, D], row stride ldx.     w   bf16 [V, D], row stride ldw.
 *   target  int64 [T], device.  Rows whose target is ignore_index take no
 *           part: whatever x holds there reaches neither loss nor dw.  Any
 *           other target outside [0, V) makes its row's loss NaN, and with it
 *           loss, dw and that row of dx; no memory is read at it.
 *   mean    0 or 1.          grad_scale   finite.
 *   loss    one float, device, written.
 *   row_loss  float [T], device, written; NULL: not wanted.
 *   dx      bf16 [T, D], row stride lddx; NULL: not wanted.
 *   dw      bf16 [V, D], row stride lddw; NULL: not wanted.  With neither,
 *           only the loss is computed.  T = 0 writes loss 0 and dw zero.
 *
 * Errors: ZOPT_ERR_NULL (workspace_bytes; with a workspace w, loss, or with
 * T > 0 x or target); ZOPT_ERR_SIZE (T, D, V or a stride out of range);
 * ZOPT_ERR_HYPER (mean, grad_scale); ZOPT_ERR_WORKSPACE; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_linear_xent(int64_t T, int64_t D, int64_t V, const uint16_t *x, int64_t ldx,
                             const uint16_t *w, int64_t ldw, const int64_t *target,
                             int64_t ignore_index, int32_t mean, float grad_scale, float *loss,
                             float *row_loss, uint16_t *dx, int64_t lddx, uint16_t *dw,
                             int64_t lddw, void *workspace, size_t *workspace_bytes,
                             void *stream);

/*
 * 8-bit activation checkpoints.  A bf16 matrix [rows, cols] is kept as
 *   q      e4m3 (OCP, 4 exponent and 3 mantissa bits) [rows, cols], and
 *   scale  one byte b per 32 neighbouring columns of a row, [rows, ceil(cols / 32)]:
 * an element is q * 2^(b - 127).  b is the smallest that brings the block's
 * largest magnitude to at most 448 (e4m3's largest), but at least 3; values
 * are divided by the power of two (exact) and rounded to nearest even, so an
 * element is off by at most 2^-4 of itself, or 2^-10 2^(b - 127).  (With
 * b = 247 values are held to 240 2^120, so that a finite one stays a finite
 * bf16.)  A block with a NaN or an infinity gets b = 255 and reads back as NaN.
 *
 * zopt_act8_pack writes q and scale from x; zopt_act8_unpack writes x from
 * them (exact: every value is a bf16).  rows = 0 enqueues nothing.
 * Errors: ZOPT_ERR_NULL; ZOPT_ERR_SIZE; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_act8_pack(int64_t rows, int64_t cols, const uint16_t *x, int64_t ldx, uint8_t *q,
                           uint8_t *scale, void *stream);
zopt_status zopt_act8_unpack(int64_t rows, int64_t cols, const uint8_t *q, const uint8_t *scale,
                             uint16_t *x, int64_t ldx, void *stream);

/*
 * zopt_act8_wgrad -- the weight gradient of a linear layer y = x w^T whose
 * input was kept as an 8-bit checkpoint: dw [N, D] = dy^T x, with
 *   dy        bf16 [T, N], row stride lddy;
 *   q, scale  the checkpoint of x [T, D];
 *   dw        bf16 [N, D], row stride lddw, written (zero for T = 0).
 * Errors: ZOPT_ERR_NULL; ZOPT_ERR_SIZE; ZOPT_ERR_WORKSPACE; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_act8_wgrad(int64_t T, int64_t N, int64_t D, const uint16_t *dy, int64_t lddy,
                            const uint8_t *q, const uint8_t *scale, uint16_t *dw, int64_t lddw,
                            void *workspace, size_t *workspace_bytes, void *stream);

/* Activations of the gated feed-forward block. */
enum {
    ZOPT_ACT_SILU = 0, /* g / (1 + exp(-g))                                      */
    ZOPT_ACT_GELU = 1  /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2      */
};

/*
 * zopt_glu_forward -- the gated feed-forward's first half in one kernel:
 *   g = x w_gate^T,  u = x w_up^T  (fp32),   h = act(g) u
 *   x               bf16 [T, D], row stride ldx.
 *   w_gate, w_up    bf16 [F, D], both with row stride ldw (two halves of one
 *                   fused [2 F, D] weight, or two matrices).
 *   act             ZOPT_ACT_*.
 *   h               bf16 [T, F], row stride ldh, written.
 *   g8, g_scale, u8, u_scale   where g and u go as 8-bit checkpoints
 *                   ([T, F] each, from their fp32 values), for
 *                   zopt_glu_backward; all four or none (NULL).
 * T = 0 enqueues nothing.
 * Errors: ZOPT_ERR_NULL (also some but not all of the checkpoint);
 * ZOPT_ERR_SIZE; ZOPT_ERR_HYPER (act); ZOPT_ERR_WORKSPACE; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_glu_forward(int64_t T, int64_t D, int64_t F, const uint16_t *x, int64_t ldx,
                             const uint16_t *w_gate, const uint16_t *w_up, int64_t ldw,
                             int32_t act, uint16_t *h, int64_t ldh, uint8_t *g8,
                             uint8_t *g_scale, uint8_t *u8, uint8_t *u_scale, void *workspace,
                             size_t *workspace_bytes, void *stream);

/*
 * zopt_glu_backward -- gradients of zopt_glu_forward from dh:
 *   du = dh act(g),  dg = dh u act'(g)             (rounded to bf16)
 *   dx = dg w_gate + du w_up,  dw_gate = dg^T x,  dw_up = du^T x
 *   dh        bf16 [T, F], row stride lddh.
 *   x, ldx    the forward's input, or x8, x_scale: its 8-bit checkpoint
 *             (then x is not read and the gradients are those of the values
 *             the checkpoint stands for).
 *   g8, g_scale, u8, u_scale   the forward's checkpoint of g and u; all NULL:
 *             g and u are computed again from x.
 *   h         bf16 [T, F], row stride ldh, written with act(g) u (for the
 *             weight gradient of the projection after it); NULL: not wanted.
 *   dx        bf16 [T, D], row stride lddx;  dw_gate, dw_up  bf16 [F, D], row
 *             stride lddw; written (T = 0: the weight gradients zero).
 * Other arguments and errors as zopt_glu_forward.
 */
zopt_status zopt_glu_backward(int64_t T, int64_t D, int64_t F, const uint16_t *dh, int64_t lddh,
                              const uint16_t *x, int64_t ldx, const uint8_t *x8,
                              const uint8_t *x_scale, const uint16_t *w_gate,
                              const uint16_t *w_up, int64_t ldw, int32_t act, const uint8_t *g8,
                              const uint8_t *g_scale, const uint8_t *u8, const uint8_t *u_scale,
                              uint16_t *h, int64_t ldh, uint16_t *dx, int64_t lddx,
                              uint16_t *dw_gate, uint16_t *dw_up, int64_t lddw, void *workspace,
                              size_t *workspace_bytes, void *stream);

/*
 * A decoder layer's other operators: norms and rotation of queries and keys,
 * and a feed-forward of experts.  The conventions of the gradient operators
 * above hold, but for what is said here.
 */

/* Which elements of a head turn together. */
enum {
    ZOPT_ROPE_HALF = 0, /* i and i + rot / 2, i < rot / 2 */
    ZOPT_ROPE_PAIRS = 1 /* 2 i and 2 i + 1                */
};

/*
 * zopt_rope_table -- the cosines and sines of the angles
 *   angle(p, i) = p base^(-2 i / rot),   p < positions, i < rot / 2
 * formed in 64 bits: table, float [positions, rot / 2, 2], written.  A program
 * makes it once; any other table of that layout (scaled angles, say) will do.
 * positions 0 .. 2^30 (0 enqueues nothing); rot even, 2 .. 512; base > 0.
 * Errors: ZOPT_ERR_SIZE; ZOPT_ERR_HYPER (base); ZOPT_ERR_NULL; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_rope_table(int64_t positions, int32_t rot, double base, float *table,
                            void *stream);

/*
 * zopt_qk_norm_rope -- the norm of every head of the queries and keys, and the
 * rotation of its first `rot` elements to its token's position, in one pass:
 *   n = x / sqrt(mean(x^2) + eps),   y = n w
 *   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)
 * for each pair (a, b) of ZOPT_ROPE_*, (c, s) its angle's cosine and sine.
 *   T         tokens, 0 .. 2^30 (0 enqueues nothing).
 *   heads_q, heads_k   1 .. 65536 and 0 .. 65536 heads of `width` elements,
 *             1 .. 512; 0: no keys, and k, yk are not looked at.
 *   rot       even, 0 .. width; 0: the norm alone.
 *   q, k      bf16 [T, heads, width]; *_token and *_head are the strides
 *             between tokens and between heads, 0 .. 2^40, so that both may be
 *             views of one projection [T, (heads_q + 2 heads_k) width], or lie
 *             head by head.
 *   table     float [positions, rot / 2, 2].
 *   position  int64 [T], device; NULL: token t has position t.  A row with a
 *             negative position takes no part: its output is zero.  One with a
 *             position that the table does not hold is NaN.
 *   w_q, w_k  bf16 [width], one for all heads of a kind; NULL: 1.
 *   eps       finite, >= 0.     style   ZOPT_ROPE_*.
 *   yq, yk    bf16 [T, heads, width], written; their heads may not overlap.
 *             yq may be q, with the same strides, and yk k.
 * Norms and sums are held in fp32 (a row whose squares pass its range, or vanish
 * in it beside an eps as small, is multiplied by a power of two first); the only
 * rounding to bf16 is the output's.
 * Errors: ZOPT_ERR_NULL; ZOPT_ERR_SIZE (sizes, strides); ZOPT_ERR_HYPER (eps,
 * style); ZOPT_ERR_DEVICE.
 */
zopt_status zopt_qk_norm_rope(int64_t T, int32_t heads_q, int32_t heads_k, int32_t width,
                              int32_t rot, const uint16_t *q, int64_t q_token, int64_t q_head,
                              const uint16_t *k, int64_t k_token, int64_t k_head,
                              const float *table, int64_t positions, const int64_t *position,
                              const uint16_t *w_q, const uint16_t *w_k, float eps,
                              int32_t style, uint16_t *yq, int64_t yq_token, int64_t yq_head,
                              uint16_t *yk, int64_t yk_token, int64_t yk_head, void *stream);

/*
 * zopt_qk_norm_rope_backward -- its gradients, from those of yq and yk and from
 * the forward's inputs:
 *   g = dy turned back,   dw = sum over tokens and heads of g n
 *   dx = (g w - n mean(g w n)) / sqrt(mean(x^2) + eps)
 *   dyq, dyk  bf16 [T, heads, width].    dq, dk   the same, written; dq may be
 *             dyq or q with the same strides, dk dyk or k.
 *   dw_q, dw_k  bf16 [width], written (zero for T = 0); NULL: not wanted.
 * Rows without a position get zero gradients and no share of dw.
 * Errors: as zopt_qk_norm_rope, dw_k without keys being ZOPT_ERR_NULL;
 * ZOPT_ERR_WORKSPACE.
 */
zopt_status zopt_qk_norm_rope_backward(
    int64_t T, int32_t heads_q, int32_t heads_k, int32_t width, int32_t rot, const uint16_t *dyq,
    int64_t dyq_token, int64_t dyq_head, const uint16_t *dyk, int64_t dyk_token,
    int64_t dyk_head, const uint16_t *q, int64_t q_token, int64_t q_head, const uint16_t *k,
    int64_t k_token, int64_t k_head, const float *table, int64_t positions,
    const int64_t *position, const uint16_t *w_q, const uint16_t *w_k, float eps, int32_t style,
    uint16_t *dq, int64_t dq_token, int64_t dq_head, uint16_t *dk, int64_t dk_token,
    int64_t dk_head, uint16_t *dw_q, uint16_t *dw_k, void *workspace, size_t *workspace_bytes,
    void *stream);

/* What a router's logits are made into. */
enum {
    ZOPT_SCORE_SOFTMAX = 0, /* softmax over the experts   */
    ZOPT_SCORE_SIGMOID = 1  /* the logistic of each logit */
};

/*
 * zopt_moe_route -- from a router's logits to each token's experts and weights,
 * and to the order in which the experts read the tokens.
 *   s = score(logits);  an expert ranks by s + bias (by its logit, which ranks
 *   the same, without a bias and groups), of equal ones the lower first
 *   with groups > 1 the experts lie in `groups` equal ranges, a range ranks by
 *   the sum of its two best, and only the best `top_groups` are chosen from
 *   weight = scale s, or (renormalise) scale s / (sum of s over the chosen);
 *   the bias has no part in it
 * An expert whose logit or bias is -inf is not there: where fewer than `top`
 * are, a token's last experts are -1 with weight 0 (a row of -inf: all of them),
 * and the token takes no part in the products there.  A NaN ranks behind every
 * number and before what is not there; so does a range with one among its two best.
 * Ranks and sums are settled in 64 bits (sums of unlike terms that only their
 * rounding there tells apart come in either order).
 *   T         tokens, 0 .. 2^30, with T top <= 2^30.
 *   experts   1 .. 1024.      top   1 .. min(experts, 32).
 *   logits    fp32 (bf16 = 0) or bf16 (1) [T, experts], row stride ld.
 *   score     ZOPT_SCORE_*.   bias   float [experts], or NULL.
 *   groups    1 .. 64, a divisor of experts; top_groups 1 .. groups, with at
 *             least `top` experts in them.
 *   renormalise   0 or 1.     scale   finite.
 *   chosen, weights   int32 and float [T, top], written, the best first.
 *   offsets   int32 [experts + 1], written: a slot is one of a token's `top`,
 *             number t top + j; the slots of expert e are order[offsets[e]] ..
 *             order[offsets[e + 1] - 1], in order.
 *   order     int32 [T top], written; -1 from offsets[experts] on.
 *   place     int32 [T, top], written: where a slot is in order, or -1.
 * Errors: ZOPT_ERR_NULL; ZOPT_ERR_SIZE; ZOPT_ERR_HYPER (bf16, score,
 * renormalise, scale); ZOPT_ERR_WORKSPACE; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_moe_route(int64_t T, int32_t experts, int32_t top, const void *logits,
                           int64_t ld, int32_t bf16, int32_t score, const float *bias,
                           int32_t groups, int32_t top_groups, int32_t renormalise, float scale,
                           int32_t *chosen, float *weights, int32_t *offsets, int32_t *order,
                           int32_t *place, void *workspace, size_t *workspace_bytes,
                           void *stream);

/*
 * zopt_moe_plan -- offsets, order and place of zopt_moe_route for experts that
 * the caller chose: chosen, int32 [T, top], any number outside [0, experts)
 * standing for none, the same expert more than once in a row counting as often.
 * Other arguments and errors as there, but top may be more than experts.
 */
zopt_status zopt_moe_plan(int64_t T, int32_t experts, int32_t top, const int32_t *chosen,
                          int32_t *offsets, int32_t *order, int32_t *place, void *workspace,
                          size_t *workspace_bytes, void *stream);

/*
 * zopt_moe_route_backward -- the gradient of the logits from that of the
 * weights, dweights float [T, top] (entries of slots without an expert are not
 * looked at).  logits, ld, bf16, score, renormalise and scale as the forward
 * had them, chosen as it wrote them; dlogits, in the logits' type, row stride
 * lddl, written whole.  Choice and bias have no gradient.
 * Errors: ZOPT_ERR_NULL; ZOPT_ERR_SIZE; ZOPT_ERR_HYPER; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_moe_route_backward(int64_t T, int32_t experts, int32_t top,
                                    const float *dweights, const void *logits, int64_t ld,
                                    int32_t bf16, int32_t score, int32_t renormalise,
                                    float scale, const int32_t *chosen, void *dlogits,
                                    int64_t lddl, void *stream);

/*
 * zopt_moe_forward -- the experts' gated feed-forward:
 *   h_s = act(x_t w_gate[e]^T) (x_t w_up[e]^T)      for slot s of token t, expert e
 *   y_t = sum over t's slots of weight_s (h_s w_down[e]^T)
 *   x             bf16 [T, D], row stride ldx.  Rows of tokens without an expert
 *                 are not read; their y is zero.
 *   w_gate, w_up  bf16 [experts, F, D], both with row stride ldw and w_expert
 *                 elements between experts (which do not overlap).
 *   w_down        bf16 [experts, D, F], ldd and wd_expert.
 *   act           ZOPT_ACT_*.
 *   weights       float [T, top];  offsets, order, place   as zopt_moe_route or
 *                 zopt_moe_plan wrote them for T, experts and top <= 32.
 *                 (Others give wrong sums, but no access outside the buffers.)
 *   y             bf16 [T, D], row stride ldy, written.
 * The sizes of the experts' shares stay on the device: nothing waits for them.
 * Sums are fp32; h is rounded to bf16 between the products, as a dense layer's is,
 * and a slot's row of y, before the sum over the token's slots, to 11 bits (fp16
 * with a power of two for 64 neighbours), as y to bf16 in the end.
 * Errors: ZOPT_ERR_NULL; ZOPT_ERR_SIZE; ZOPT_ERR_HYPER (act);
 * ZOPT_ERR_WORKSPACE; ZOPT_ERR_DEVICE.
 */
zopt_status zopt_moe_forward(int64_t T, int64_t D, int64_t F, int32_t experts, int32_t top,
                             const uint16_t *x, int64_t ldx, const uint16_t *w_gate,
                             const uint16_t *w_up, int64_t ldw, int64_t w_expert,
                             const uint16_t *w_down, int64_t ldd, int64_t wd_expert, int32_t act,
                             const float *weights, const int32_t *offsets, const int32_t *order,
                             const int32_t *place, uint16_t *y, int64_t ldy, void *workspace,
                             size_t *workspace_bytes, void *stream);

/*
 * zopt_moe_backward -- gradients of zopt_moe_forward from dy, bf16 [T, D], row
 * stride lddy; g, u and h are computed again from x:
 *   dx            bf16 [T, D], row stride lddx (zero for tokens without an expert).
 *   dw_gate, dw_up   bf16 [experts, F, D], row stride lddw, dw_expert elements
 *                 between experts;  dw_down   bf16 [experts, D, F], lddd and
 *                 dwd_expert; zero for experts without a token.
 *   dweights      float [T, top], 0 for slots without an expert.
 * All are written.  A row of x and of dy whose token has no expert reaches
 * none of them.  dg, du and weight h are rounded to bf16 between the products, a
 * slot's row of dx to 11 bits as one of y; dy w_down, and with it dweights, is kept
 * in fp32.
 * Other arguments and errors as zopt_moe_forward.
 */
zopt_status zopt_moe_backward(int64_t T, int64_t D, int64_t F, int32_t experts, int32_t top,
                              const uint16_t *dy, int64_t lddy, const uint16_t *x, int64_t ldx,
                              const uint16_t *w_gate, const uint16_t *w_up, int64_t ldw,
                              int64_t w_expert, const uint16_t *w_down, int64_t ldd,
                              int64_t wd_expert, int32_t act, const float *weights,
                              const int32_t *offsets, const int32_t *order,
                              const int32_t *place, uint16_t *dx, int64_t lddx,
                              uint16_t *dw_gate, uint16_t *dw_up, int64_t lddw,
                              int64_t dw_expert, uint16_t *dw_down, int64_t lddd,
                              int64_t dwd_expert, float *dweights, void *workspace,
                              size_t *workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZOPT_H */
