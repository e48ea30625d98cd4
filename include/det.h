/*
 * det.h -- reproducible floating-point add-reductions on AMD Instinct MI355X (gfx950).
 *
 * Three operations whose result bits depend only on (op, flags, dtype, input): never on the
 * grid, occupancy, CU count, stream, run or device.  Every addition is one IEEE-754
 * round-to-nearest-even addition in the input dtype (no contraction, subnormals kept); the
 * association order is fixed by the problem size alone:
 *
 *  PW(v)   adjacent-pair tree: pad v with -0.0 to a power of two, then replace the list by
 *          v0+v1, v2+v3, ... until one value remains (course page "Floating point and
 *          reproducibility", section "Fix the order of every addition": a fixed bracket over
 *          pairs instead of an atomic tail).
 *
 * Conventions for every entry point:
 *  - Data pointers are DEVICE pointers owned by the caller.  Any element-aligned address is
 *    accepted (tensor views); alignment never changes the bits.  A data pointer that is not
 *    aligned to its element size is rejected with DET_ERROR_INVALID_VALUE.
 *  - The library never allocates and never synchronises.  Scratch memory is a caller-provided
 *    device workspace of at least *_workspace_size(...) bytes, 256-byte aligned (else
 *    DET_ERROR_WORKSPACE; torch's and hipMalloc's allocations are); its contents
 *    on entry do not matter and are undefined on return.  Calls that overlap in time must not
 *    share a workspace.
 *  - All work is enqueued on `stream` (a hipStream_t; NULL = the default stream) and the call
 *    returns without waiting for it.
 *  - Host-checkable problems return a status and enqueue nothing.  Data-dependent conditions
 *    never fail: out-of-range scatter indices are skipped and counted.
 *  - Sizes: 0 <= n <= DET_MAX_N (2^31 - 1), as scatter record slots are signed 32-bit
 *    (Warp "Deterministic Execution", section "Limitations", large launches).
 *  - No C++ exception crosses this interface.
 *
 * The language-model operators further down (norms, relative position bias, token log
 * probabilities, embedding, gated recurrence, linear cross entropy) keep these conventions; their
 * arithmetic and the order of their sums are stated there.
 */
#ifndef DET_H
#define DET_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* DET_I32 is accepted by det_scan only (Warp "Deterministic Execution", section "Pattern 2:
 * Slot Allocation": the count-scan-write workflow's prefix scan over int32 slot counts); its
 * sums wrap modulo 2^32 as two's complement, which no association order can change. */
/* DET_F16, DET_BF16: storage types of the language-model operators only (they compute in f32).
 * DET_E4M3 (8-bit floats: 4 exponent and 3 mantissa bits, largest 448, no infinity): the output
 * type of det_rms_norm only.  DET_I64 (and DET_I32): token ids of det_embedding. */
typedef enum {
    DET_F32 = 0,
    DET_F64 = 1,
    DET_I32 = 2,
    DET_F16 = 3,
    DET_BF16 = 4,
    DET_E4M3 = 5,
    DET_I64 = 6
} det_dtype;

typedef enum {
    DET_SUCCESS = 0,
    DET_ERROR_INVALID_VALUE = 1, /* bad argument (negative size, NULL pointer, bad flags...) */
    DET_ERROR_UNSUPPORTED = 2,   /* unknown dtype */
    DET_ERROR_TOO_LARGE = 3,     /* n or a derived size beyond DET_MAX_N */
    DET_ERROR_WORKSPACE = 4,     /* ws NULL, not 256-byte aligned, or smaller than the
                                    matching *_workspace_size */
    DET_ERROR_LAUNCH = 5         /* the HIP runtime refused a launch */
} det_status;

#define DET_MAX_N 2147483647LL

/* det_scan flags (inclusive and forward when 0) */
#define DET_SCAN_EXCLUSIVE 1u
#define DET_SCAN_REVERSE 2u

/* ------------------------------------------------------------------ sum */

/* Bytes of workspace det_sum needs for n elements (0 when the arguments are invalid). */
size_t det_sum_workspace_size(int64_t n, det_dtype dtype);

/* *out = PW(x[0..n)) for n >= 1, +0.0 for n == 0.
 * x:   device, n elements of dtype (read only).
 * out: device, one element of dtype (written).
 * The fixed tree replaces the atomic tail of a block-partials reduction (course page
 * "Floating point and reproducibility", sections "Twenty answers, none of them wrong" and
 * "Fix the order of every addition").  Any aligned power-of-two chunk of x is a subtree of
 * PW, so the kernels may split x into chunks of any power-of-two size without moving a bit.
 * ws: device, at least det_sum_workspace_size(n, dtype) bytes, 256-byte aligned, any initial
 * contents; the call leaves it holding partial values.  Sums of 2 to 1024 chunks of 2^14
 * elements (up to 2^24 elements) finish in one launch: the grid's last workgroup waits for
 * the chunk values tagged for the call, a wait bounded at 2 seconds of the GPU's 100 MHz
 * clock after which *out receives a NaN instead of the sum (a failure of the GPU's forward
 * progress, not of the data).  Calls that share a workspace must be ordered on one stream. */
det_status det_sum(const void* x, int64_t n, det_dtype dtype, void* out, void* ws,
                   size_t ws_bytes, void* stream);

/* det_sum for callers that cannot allocate device memory (code under HIP graph capture that
 * must not call hipMalloc, tight serving loops, harnesses that forbid allocation): no
 * workspace argument and no allocation; the result bits are det_sum's.
 * x, out, n, dtype, stream and the errors are det_sum's (n up to DET_MAX_N, beyond it
 * DET_ERROR_TOO_LARGE); DET_ERROR_LAUNCH if the runtime cannot give the array's address.
 * The partial sums live in a static device array of DET_SUM_NOALLOC_SCRATCH_BYTES bytes, one
 * per GPU the library runs on, loaded with the library's code and held until the process
 * ends; that size covers every n up to DET_MAX_N in f32 and f64.  Every call on one GPU uses
 * that GPU's single array, which keeps the last call's partials: calls that overlap in time
 * on one GPU (different streams or host threads without ordering) race and give unspecified
 * results.  Calls ordered on one stream are safe. */
#define DET_SUM_NOALLOC_SCRATCH_BYTES (1048576 + 16384 + 256)
det_status det_sum_noalloc(const void* x, int64_t n, det_dtype dtype, void* out, void* stream);

/* ------------------------------------------------------------------ scan */

/* Bytes of workspace det_scan needs. */
size_t det_scan_workspace_size(int64_t n, det_dtype dtype, unsigned flags, int64_t num_segments);

/* Prefix sum with look-back through fixed anchor intervals (drjit-core pull request "Make
 * CUDA floating-point prefix sums deterministic", sections "Root cause" and
 * "Implementation"; inclusive/exclusive, forward/reverse, full/segmented per "Validation").
 *
 * Order (constants from det_spec_constants: V = 32 elements per lane, W = 64 lanes per wave,
 * 4 waves per tile, T = 8192 elements per tile, A = 256 tiles per anchor interval, A2 = 256
 * intervals per super-interval):
 *   lane-serial prefix s over each lane's run of V elements; Kogge-Stone over the lane totals
 *   inside each wave (p = lane-exclusive prefix); Kogge-Stone over the 4 wave totals
 *   (P = wave-exclusive prefix; the last value is the tile total Agg_j); for tile j in anchor
 *   interval q of super-interval Q: W_j = PW(Agg_{qA..j-1}); interval totals
 *   G_q = PW(all Agg of q); WG = PW(G_{Q*A2..q-1}); super-interval carries CC_0 = -0.0,
 *   CC_{Q+1} = CC_Q + PW(all G of Q); y = ((((CC_Q + WG) + W_j) + P) + p) + s.  Only fixed
 *   anchors publish totals and carries, so the bits do not depend on which predecessors a tile
 *   saw as finished.
 *
 * dtype DET_I32: int32 elements, sums wrapping modulo 2^32 (the same dataflow; every order
 *         gives the same integers), the exclusive scan's first value 0.
 * x, y:   device, n elements of dtype.  Inclusive scans may run in place (y == x); exclusive
 *         scans must not overlap x and y (DET_ERROR_INVALID_VALUE if the ranges overlap).
 * flags:  DET_SCAN_EXCLUSIVE (y[0] = +0.0, y[i] = inclusive[i-1]) and/or DET_SCAN_REVERSE
 *         (scan of the flipped array, flipped back).
 * seg_offsets: NULL for one segment, else device int64 [num_segments + 1] with
 *         0 = o_0 <= o_1 <= ... <= o_S = n (precondition, not checked on the device).  Each
 *         segment restarts the scan: the head-flag operator (f1|f2, f2 ? b : a + b) runs
 *         through the same order; exclusive scans write +0.0 at every segment head (for
 *         reverse: at every segment's last element).  num_segments >= 1 when n > 0. */
det_status det_scan(const void* x, void* y, int64_t n, det_dtype dtype, unsigned flags,
                    const int64_t* seg_offsets, int64_t num_segments, void* ws, size_t ws_bytes,
                    void* stream);

/* Health word of the last det_scan run in workspace ws, for callers that want to verify it.
 * A scan of more than one anchor interval (more than 256 * 8192 elements) waits on status words
 * that earlier tiles publish.  Each such wait is bounded: after 2 seconds of the GPU's constant
 * 100 MHz clock it gives up, sets this word and leaves y unspecified while det_scan has already
 * returned DET_SUCCESS.  Any failure of the kernel's forward progress (a broken offsets
 * precondition, a hardware fault, a scheduler that never runs a workgroup holding a claimed
 * tile) ends that way, never in a hang; a silent wrong result is possible only if a status
 * word arrives corrupted yet tagged ready.  Shorter and empty scans never wait and leave the
 * word at 0.
 * Enqueues on `stream` a copy of the word into *out (device int32: 0 = every wait ended
 * normally, 1 = some wait gave up); returns without waiting.  ws: the workspace the scan used
 * (device); out: device int32 (written).  DET_ERROR_INVALID_VALUE for NULL. */
det_status det_scan_error(const void* ws, int32_t* out, void* stream);

/* ------------------------------------------------------------------ scatter-add */

/* Bytes of workspace det_scatter_add needs. */
size_t det_scatter_add_workspace_size(int64_t n, int64_t num_out, int64_t row_len,
                                      det_dtype dtype);

/* Keyed scatter-add along axis 0, the reproducible form of atomic_add(out, index[i],
 * values[i]) (Warp "Deterministic Execution", sections "Pattern 1: Accumulation" and
 * "Writing Manual Deterministic Code") and, for row_len > 1, of the row-indexed tile
 * accumulate (Warp reference "warp.tile_atomic_add_indexed").
 *
 * For destination r and column c: M = [values[i*row_len + c] for ascending i with
 * index[i] == r]; if M is non-empty, out[r*row_len + c] = out[r*row_len + c] + PW(M), else
 * out is left untouched.
 *
 * values:  device, [n * row_len] of dtype, row-major (read only; must not alias out).
 * index:   device int32 [n].  Entries outside [0, num_out) are skipped, never an error.
 * out:     device, [num_out * row_len] of dtype, updated in place.
 * prev:    NULL, or device [n * row_len]: for every valid i, the destination row as it was
 *          before this call (rows of skipped i are not written).
 * n_skipped: NULL, or device int64: set (not accumulated) to the number of skipped i.
 * row_len: >= 1. */
det_status det_scatter_add(const void* values, const int32_t* index, int64_t n, int64_t row_len,
                           det_dtype dtype, void* out, int64_t num_out, void* prev,
                           int64_t* n_skipped, void* ws, size_t ws_bytes, void* stream);

/* Keyed scatter-subtract, the reproducible form of atomic_sub(out, index[i], values[i]): the
 * values are negated and then added in the order of det_scatter_add (Warp "Deterministic
 * Execution", section "Pattern 1: Accumulation", its table of atomics).  So for destination r
 * and column c, out = out + PW(-M) with every element of M negated on its own; this is not
 * out - PW(M) where a destination's contributions cancel to zero (the zero's sign differs).
 * Arguments, workspace (det_scatter_add_workspace_size), ownership and errors as for
 * det_scatter_add; prev receives the destination rows before the call. */
det_status det_scatter_sub(const void* values, const int32_t* index, int64_t n, int64_t row_len,
                           det_dtype dtype, void* out, int64_t num_out, void* prev,
                           int64_t* n_skipped, void* ws, size_t ws_bytes, void* stream);

/* Bytes of workspace det_scatter_add_running needs (0 when the arguments are invalid). */
size_t det_scatter_add_running_workspace_size(int64_t n, int64_t num_out, int64_t row_len,
                                              det_dtype dtype);

/* det_scatter_add whose prev is the running value: what a loop of atomic adds in ascending
 * source index would hand back to each source, with the sum of the earlier contributions
 * formed in a fixed order.  The Warp reference "warp.tile_atomic_add_indexed" returns the
 * destination rows as they were before the accumulate and leaves them unspecified under
 * repeated indices; this entry point fixes them.
 *
 * Order: lay the members of every destination (ascending source index, as in
 * det_scatter_add) end to end in destination order, one segment per destination, and take
 * E = the forward exclusive segmented det_scan of each column of that array.  The member at
 * position g of that array, source row i, destination r, gets
 *   prev[i*row_len + c] = out[r*row_len + c]          at r's first position,
 *   prev[i*row_len + c] = out[r*row_len + c] + E[g]   elsewhere
 * (out as before the call).  out receives exactly what det_scatter_add gives it.
 *
 * values, index, out, n_skipped, row_len: as for det_scatter_add.
 * prev:    device [n * row_len] of dtype, required when n > 0 (rows of skipped i are not
 *          written); must not overlap values or out (DET_ERROR_INVALID_VALUE).
 * row_len: 1 .. 65535 * 32 (DET_ERROR_TOO_LARGE beyond).
 * Workspace: det_scatter_add_running_workspace_size bytes, about 2 * n * row_len elements
 * more than det_scatter_add's (f32 with row_len 1 and more than 2^21 members, whose values
 * travel through the sort beside their source indices and whose prev goes out through windows
 * of the source index: about 7 * n 4-byte words more).  The columns are scanned in one launch
 * when each fits one anchor interval of tiles, else one scan per column. */
det_status det_scatter_add_running(const void* values, const int32_t* index, int64_t n,
                                   int64_t row_len, det_dtype dtype, void* out, int64_t num_out,
                                   void* prev, int64_t* n_skipped, void* ws, size_t ws_bytes,
                                   void* stream);

/* ------------------------------------------------------------------ language-model operators
 *
 * Norms, relative position bias, token log probabilities, embedding, gated recurrence and linear
 * cross entropy, forward and backward.  dtype is
 * DET_F32, DET_F16 or DET_BF16 (else DET_ERROR_UNSUPPORTED): the type of every tensor not
 * declared float, int32 or int64 below.  Everything between loading and the one rounding on
 * storing is f32 (the bias table's gradient f64, of 16-bit types but for sums over 8 rows).  Every
 * sum's order is fixed by the arguments that its comment names, never by the launch, so the bits
 * depend on the arguments alone; the results of a row depend on that row alone, not on the rows
 * beside it or (but for the linear cross entropy) their number.
 * Strides count elements; the innermost dimension is contiguous.  No wait inside any kernel
 * depends on another workgroup. */

/* Root-mean-square norm of rows, with the residual's addition before and 8-bit codes behind:
 *   h = x + residual (x where residual is NULL; used unrounded)
 *   rstd = 1 / sqrt(sum(h^2) / d + eps);  y = (h * rstd) * weight
 *   y_dtype DET_E4M3: for every group of neighbouring elements of a row, m = max(|y|, 2^-100),
 *   code = round(y * (448 / m)), scale = m / 448.
 * Order of the row's sum: fixed by (d, dtype).
 * x, residual:  [rows] rows of d elements, x_stride and residual_stride apart (>= d when
 *               rows > 1).  residual may be NULL.
 * weight:       [d].
 * h:            [rows * d], x + residual rounded to dtype; NULL if and only if residual is.
 *               h may be x or residual itself where that is contiguous (written in place).
 * y:            [rows * d] of y_dtype, which is dtype or DET_E4M3.
 * group:        for codes 32, 64 or 128 elements (a row's last group may be shorter), or 0 for
 *               one scale a row; 0 otherwise.
 * scales:       float [rows * ceil(d / group)] (group 0: [rows]) for codes, else NULL.
 * rstd:         NULL, or float [rows] for the backward pass.
 * d >= 1 when rows > 0; eps >= 0 and finite.  rows * d up to 2^62. */
det_status det_rms_norm(const void* x, int64_t x_stride, const void* residual,
                        int64_t residual_stride, const void* weight, int64_t rows, int64_t d,
                        det_dtype dtype, double eps, void* h, void* y, det_dtype y_dtype,
                        int64_t group, float* scales, float* rstd, void* stream);

/* Bytes of workspace det_rms_norm_backward needs (0 when the arguments are invalid). */
size_t det_rms_norm_backward_workspace_size(int64_t rows, int64_t d, det_dtype dtype);

/* Gradients of det_rms_norm's y in dtype: with xhat = h * rstd,
 *   dx = rstd * (dy weight - xhat * sum(dy weight xhat) / d) (+ dh)
 *   dweight = sum over the rows of dy * xhat
 * dx is also the gradient of the residual.
 * dy, h:    [rows] rows of d elements, dy_stride and h_stride apart; h as det_rms_norm wrote it
 *           (x itself where there was no residual).
 * rstd:     float [rows], as det_rms_norm wrote it.
 * dh:       NULL, or the gradient that reaches h from elsewhere, dh_stride apart.
 * dx:       [rows * d]; may be dy, h or dh itself where that is contiguous and d <= 16384.
 * dweight:  [d], written (zero for no rows).
 * Order: a row's sum fixed by (d, dtype); dweight's by (rows, d, dtype): strips of rows in
 * ascending order; the strips of 1 to 4 neighbours in theirs; of these sums 256 chains (k, k + 256,
 * ...), which a halving tree joins. */
det_status det_rms_norm_backward(const void* dy, int64_t dy_stride, const void* h,
                                 int64_t h_stride, const void* weight, const float* rstd,
                                 const void* dh, int64_t dh_stride, int64_t rows, int64_t d,
                                 det_dtype dtype, void* dx, void* dweight, void* ws,
                                 size_t ws_bytes, void* stream);

/* det_relative_bias flags */
#define DET_BIAS_BIDIRECTIONAL 1u /* own buckets for keys after the query */
#define DET_BIAS_CAUSAL 2u        /* keys after the query are masked */
#define DET_BIAS_MAX_BUCKETS 256

/* A learned relative position bias by buckets, alone or added to attention scores:
 *   out[b, h, i, j] = (scores[b, h, i, j] +) table[bucket(j - i - offset_b), h], and -inf
 * where the masks leave nothing: j > i + offset_b when DET_BIAS_CAUSAL, and j or i + offset_b at
 * or past lengths[b].  A masked place is -inf whatever its score holds.
 * bucket(r): a side has n = num_buckets buckets (half of them, rounded down, when
 * DET_BIAS_BIDIRECTIONAL; r > 0 then takes the second half, else r > 0 counts as distance 0).
 * Distances a below n/2 (rounded down) have a bucket each; beyond, bucket n/2 + floor((n - n/2)
 * log(a / (n/2)) / log(max_distance / (n/2))), at most n - 1.  The borders are computed in whole
 * numbers: a distance on a border lies above it.
 * table:     [num_buckets * heads], a row for each bucket.
 * q_offset:  position of query 0 among the keys; q_offsets: NULL, or int32 [batch], one for each
 *            sequence in its place.
 * lengths:   NULL, or int32 [batch]; values above q or k mean no padding, below 1 that every
 *            place is masked.
 * scores:    NULL, or [batch, heads, q, k] with strides (stride_b, stride_h, stride_q, 1); a
 *            stride may be 0.
 * out:       [batch * heads * q * k].  May be scores itself where that is contiguous.
 * 2 <= n <= 128 per side, n/2 < max_distance < 2^31, 1 <= heads < 65536,
 * |q_offset| < 2^40.  Nothing is summed but the score and its bias. */
det_status det_relative_bias(const void* table, int64_t num_buckets, int64_t heads,
                             int64_t max_distance, unsigned flags, int64_t batch, int64_t q,
                             int64_t k, int64_t q_offset, const int32_t* q_offsets,
                             const int32_t* lengths, const void* scores, int64_t stride_b,
                             int64_t stride_h, int64_t stride_q, det_dtype dtype, void* out,
                             void* stream);

/* Bytes of workspace det_relative_bias_backward needs (0 when the arguments are invalid). */
size_t det_relative_bias_backward_workspace_size(int64_t batch, int64_t heads, int64_t q,
                                                 int64_t k, int64_t num_buckets, det_dtype dtype);

/* The table's gradient: dtable[c, h] = sum of dout[b, h, i, j] over the unmasked places with
 * bucket c.  dout at masked places is not used, whatever it holds.
 * dout:     [batch, heads, q, k] with strides (stride_b, stride_h, stride_q, 1).
 * dtable:   [num_buckets * heads], written.
 * dscores:  NULL, or [batch * heads * q * k]: dout with zeros at the masked places (the gradient
 *           of the scores).  May be dout itself where that is contiguous.
 * The other arguments as for det_relative_bias.
 * Order, fixed by (batch, heads, q, k, dtype) and, where a bucket's diagonals begin and end, by
 * (num_buckets, max_distance, direction, offsets): 8 rows of a diagonal in row order (in float for
 * 16-bit types), a strip's blocks of 8 rows; the diagonals of a bucket inside a tile (512 of them,
 * 256 of f32): runs of up to 16 in ascending order, longer ones by lanes of a vector each and the
 * adjacent-lanes tree; four neighbouring tiles; of these sums, sequence by sequence, 64 chains (g, g
 * + 64, ...), which a halving tree joins.  All but the 8 rows in f64. */
det_status det_relative_bias_backward(const void* dout, int64_t stride_b, int64_t stride_h,
                                      int64_t stride_q, int64_t num_buckets, int64_t heads,
                                      int64_t max_distance, unsigned flags, int64_t batch,
                                      int64_t q, int64_t k, int64_t q_offset,
                                      const int32_t* q_offsets, const int32_t* lengths,
                                      det_dtype dtype, void* dtable, void* dscores, void* ws,
                                      size_t ws_bytes, void* stream);

#define DET_LOGPROB_MAX_TOP 64
#define DET_LOGPROB_MAX_TOP_VOCAB 1048576

/* Log probabilities of given tokens: with z = scale * logits, per row
 *   lse = log(sum exp z);  logp = z[target] - lse;  entropy = -sum p log p, p = exp(z - lse)
 *   top_logp, top_ids: the `top` largest logits, descending, ties to the lower index (both zeros
 *   alike, a NaN like -inf).
 * logits:    [rows] rows of vocab elements, row_stride apart (>= vocab when rows > 1).
 * targets:   int64 [rows]; one outside [0, vocab) is not scored: its logp is 0.
 *            entropy and lse are written for every row, scored or not.
 * logp, entropy, lse:  float [rows].
 * top:       0 .. min(vocab, DET_LOGPROB_MAX_TOP); above 0, vocab is at most
 *            DET_LOGPROB_MAX_TOP_VOCAB (DET_ERROR_TOO_LARGE).
 * top_logp, top_ids:  float and int64 [rows * top], NULL when top is 0.
 * A row of -inf alone has lse -inf, entropy 0, logp -inf; a result past float's range is infinite
 * (lse of a row of the lowest floats with a scale above 1).  vocab >= 1 when rows > 0; scale > 0
 * and finite.  Order of a row's sums: fixed by (vocab, dtype). */
det_status det_token_logprobs(const void* logits, int64_t row_stride, const int64_t* targets,
                              int64_t rows, int64_t vocab, det_dtype dtype, double scale,
                              float* logp, float* entropy, float* lse, int64_t top,
                              float* top_logp, int64_t* top_ids, void* stream);

/* Gradient of det_token_logprobs for the logits:
 *   dlogits = scale * (dlogp * (hit - p) - dentropy * p * (log p + entropy))
 * where hit is 1 at the target; a target outside [0, vocab) takes no dlogp.
 * lse, entropy:  float [rows], as det_token_logprobs wrote them for these logits and scale.  A
 *                float lse has few digits of log(sum) where it is large (none in a row of the
 *                type's lowest values): a row with |lse| > 256 takes log p from its logits again,
 *                in an order fixed by (vocab, dtype).
 * dlogp:         float [rows].
 * dentropy:      NULL (then entropy may be NULL too), or float [rows].
 * dlogits:       [rows] rows of vocab elements, dlogits_stride apart; may be logits itself (with
 *                its stride).  A row of -inf alone has gradient 0. */
det_status det_token_logprobs_backward(const void* logits, int64_t row_stride,
                                       const int64_t* targets, const float* lse,
                                       const float* dlogp, const float* entropy,
                                       const float* dentropy, int64_t rows, int64_t vocab,
                                       det_dtype dtype, double scale, void* dlogits,
                                       int64_t dlogits_stride, void* stream);

/* Layer norm of rows, with the residual's addition before:
 *   h = x + residual (x where residual is NULL; used unrounded)
 *   mean = sum(h) / d;  rstd = 1 / sqrt(sum((h - mean)^2) / d + eps)
 *   y = ((h - mean) * rstd) * weight + bias
 * The arguments as for det_rms_norm; bias: NULL, or [d]; mean, rstd: NULL, or float [rows] for the
 * backward pass.  Order of a row's sums: fixed by (d, dtype). */
det_status det_layer_norm(const void* x, int64_t x_stride, const void* residual,
                          int64_t residual_stride, const void* weight, const void* bias,
                          int64_t rows, int64_t d, det_dtype dtype, double eps, void* h, void* y,
                          float* mean, float* rstd, void* stream);

/* Bytes of workspace det_layer_norm_backward needs (0 when the arguments are invalid). */
size_t det_layer_norm_backward_workspace_size(int64_t rows, int64_t d, det_dtype dtype);

/* Gradients of det_layer_norm's y in dtype: with xhat = (h - mean) * rstd, g = dy weight,
 *   dx = rstd * (g - sum(g) / d - xhat * sum(g xhat) / d) (+ dh)
 *   dweight = sum over the rows of dy * xhat;  dbias = sum over the rows of dy
 * dbias: NULL, or [d].  The other arguments, where dx may lie, and the order of the sums as for
 * det_rms_norm_backward. */
det_status det_layer_norm_backward(const void* dy, int64_t dy_stride, const void* h,
                                   int64_t h_stride, const void* weight, const float* mean,
                                   const float* rstd, const void* dh, int64_t dh_stride,
                                   int64_t rows, int64_t d, det_dtype dtype, void* dx,
                                   void* dweight, void* dbias, void* ws, size_t ws_bytes,
                                   void* stream);

/* Rows of a table by token ids: out[i] = scale * table[tokens[i]]; a token outside [0, vocab) (such
 * as -1 for padding) has a row of zeros.
 * table:   [vocab] rows of d elements, table_stride apart (>= d when vocab > 1).
 * tokens:  [n] of token_type, DET_I32 or DET_I64 (else DET_ERROR_UNSUPPORTED).
 * out:     [n * d].  scale: finite. */
det_status det_embedding(const void* table, int64_t table_stride, const void* tokens,
                         det_dtype token_type, int64_t n, int64_t vocab, int64_t d,
                         det_dtype dtype, double scale, void* out, void* stream);

/* Bytes of workspace det_embedding_backward needs (0 when the arguments are invalid). */
size_t det_embedding_backward_workspace_size(int64_t n, int64_t vocab, int64_t d, det_dtype dtype);

/* The table's gradient: dtable[v] = scale * sum of dout[i] over the i with tokens[i] = v, zeros
 * where there is none; tokens outside [0, vocab) add to nothing.
 * dout:    [n] rows of d elements, dout_stride apart.
 * dtable:  [vocab * d], written whole.
 * Order: ascending i; blocks of 64 from a token's first position on in float, the blocks of a token
 * that has several in double.  A row's bits depend on the positions of its own token alone.
 * n <= DET_MAX_N, vocab < DET_MAX_N. */
det_status det_embedding_backward(const void* dout, int64_t dout_stride, const void* tokens,
                                  det_dtype token_type, int64_t n, int64_t vocab, int64_t d,
                                  det_dtype dtype, double scale, void* dtable, void* ws,
                                  size_t ws_bytes, void* stream);

/* det_gated_scan flags */
#define DET_GATE_SIGMOID 1u /* gates pass through a sigmoid and mix the input in */
#define DET_SCAN_MAX_CHANNELS 4194303

/* Bytes of workspace det_gated_scan needs (0 when the arguments are invalid). */
size_t det_gated_scan_workspace_size(int64_t batch, int64_t steps, int64_t d, det_dtype dtype);

/* The gated linear recurrence of every channel of every sequence:
 *   h[t] = a[t] h[t-1] + b[t],  h[-1] = state0
 * with a = gate, b = x, or with DET_GATE_SIGMOID a = 1 / (1 + e^-gate), b = (1 - a) x.
 * gate, x, h: [batch * steps * d], channels innermost.  In f32 between the loads and h's rounding.
 * state0:     NULL (zeros), or float [batch * d].
 * state:      float [batch * d]: h behind each sequence's last step, unrounded.  May be state0 itself
 *             where steps <= 8.
 * lengths:    NULL, or int32 [batch]: steps at or past a sequence's length keep the state, and their
 *             h is 0; gate and x there are not used, whatever they hold.  Values above steps mean
 *             steps, below 0 none.
 * Without DET_GATE_SIGMOID gates are taken to have |gate| <= 1: products of up to 128 neighbouring
 * gates are formed, and where one overflows h may be infinite or NaN.  A gate that is NaN, or infinite
 * beside a state of 0, makes h NaN from its step on, as the recurrence has it.
 * steps >= 1 when batch * d > 0; d <= DET_SCAN_MAX_CHANNELS, batch * d <= DET_MAX_N.
 * Order: fixed by the step's position alone (spans of 8 steps, chunks of 16 spans), so a sequence's
 * bits depend neither on the other channels nor on the steps that follow. */
det_status det_gated_scan(const void* gate, const void* x, const float* state0,
                          const int32_t* lengths, unsigned flags, int64_t batch, int64_t steps,
                          int64_t d, det_dtype dtype, void* h, float* state, void* ws,
                          size_t ws_bytes, void* stream);

/* Bytes of workspace det_gated_scan_backward needs (0 when the arguments are invalid). */
size_t det_gated_scan_backward_workspace_size(int64_t batch, int64_t steps, int64_t d,
                                              det_dtype dtype);

/* Gradients of det_gated_scan, from the last step on:
 *   G[t] = dh[t] + E[t+1],  E[t] = a[t] G[t],  E behind a sequence's last step = dstate
 *   dx = G, dgate = G h[t-1];  with DET_GATE_SIGMOID dx = (1 - a) G, dgate = a (h[t-1] - x) dx
 * dh, h:    [batch * steps * d]; h as det_gated_scan wrote it.  dh past a length is not used.
 * state0:   as handed to det_gated_scan.  dstate: NULL (zeros), or float [batch * d].
 * dgate, dx: [batch * steps * d], 0 past a length.
 * dstate0:  NULL, or float [batch * d]: E[0], the gradient of state0.
 * Order: fixed by the step's position and the number of steps. */
det_status det_gated_scan_backward(const void* dh, const void* gate, const void* x, const void* h,
                                   const float* state0, const float* dstate,
                                   const int32_t* lengths, unsigned flags, int64_t batch,
                                   int64_t steps, int64_t d, det_dtype dtype, void* dgate,
                                   void* dx, float* dstate0, void* ws, size_t ws_bytes,
                                   void* stream);

/* Bytes of workspace det_linear_cross_entropy needs (0 when the arguments are invalid): 8 for a row and
 * tile of 64 to 256 entries, 4 for a row. */
size_t det_linear_cross_entropy_workspace_size(int64_t rows, int64_t vocab, int64_t d,
                                               det_dtype dtype);

/* Cross entropy behind an output projection, without its logits in memory:
 *   z = scale * x weight^T;  lse = log(sum exp z);  loss = lse - z[target]
 * x:        [rows] rows of d elements, x_stride apart.
 * weight:   [vocab] rows of d elements, weight_stride apart.
 * targets:  int64 [rows]; one outside [0, vocab) is not scored: its loss is 0.  lse is written for
 *           every row.
 * loss, lse: float [rows].
 * The products are of dtype's matrix instructions with f32 sums: a logit is off by at most (d + 8) 2^-23
 * of the sum of its products' magnitudes, as each addition rounds.  f32 goes through them in three parts of 8
 * bits each: each product is off by up to 2^-22 of itself besides, to either side, and an infinite factor
 * may give NaN.  rows <= 2^20, 1 <= d <= 2^20, vocab >= 1; scale > 0 and finite.
 * Order: fixed by (rows, vocab, d, dtype). */
det_status det_linear_cross_entropy(const void* x, int64_t x_stride, const void* weight,
                                    int64_t weight_stride, const int64_t* targets, int64_t rows,
                                    int64_t vocab, int64_t d, det_dtype dtype, double scale,
                                    float* loss, float* lse, void* ws, size_t ws_bytes,
                                    void* stream);

/* Bytes of workspace det_linear_cross_entropy_backward needs (0 when the arguments are invalid).  With
 * P = min(vocab, max(4096, min(65536, 2^26 / rows))) entries a piece and s bytes an element:
 *   D by rows, and in 16-bit types by columns:     rows P s each
 *   x by columns:                                  rows d s
 *   weight by columns, 16 bits above 64 rows:      P d s
 *   dx's sums:                                     4 rows d, or up to 2^26 where workgroups share a sum
 * and up to 64 more rows, entries or columns of each.  Above 16384 rows D grows with them. */
size_t det_linear_cross_entropy_backward_workspace_size(int64_t rows, int64_t vocab, int64_t d,
                                                        det_dtype dtype);

/* Gradients of det_linear_cross_entropy's loss, the logits made again piece by piece:
 *   D = exp(z - lse) - hit;  dx = scale * dloss * (D weight);  dweight = scale * (dloss D)^T x
 * D is rounded to dtype once (f32: and x times dloss once, for dweight).  A row that is not scored has dx 0 and adds nothing to dweight,
 * whatever it holds.  exp(z - lse) is off by about |lse| 2^-24 relative to it.
 * lse:      float [rows], as det_linear_cross_entropy wrote it for these x, weight and scale.
 * dloss:    float [rows].
 * dx:       [rows * d].  dweight: [vocab * d].
 * vocab, d >= 1; no rows: dweight is 0.  Order: fixed as for det_linear_cross_entropy. */
det_status det_linear_cross_entropy_backward(const void* x, int64_t x_stride, const void* weight,
                                             int64_t weight_stride, const int64_t* targets,
                                             const float* lse, const float* dloss, int64_t rows,
                                             int64_t vocab, int64_t d, det_dtype dtype,
                                             double scale, void* dx, void* dweight, void* ws,
                                             size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ introspection */

/* Version of the association order; results of one version never change. */
int det_spec_version(void);

/* Scan constants of this version: elements per lane, lanes per tile, tiles per anchor
 * interval, anchor intervals per super-interval (any pointer may be NULL). */
void det_spec_constants(int64_t* V, int64_t* L, int64_t* A, int64_t* A2);

/* Static string naming a status code. */
const char* det_status_string(det_status s);

/* ------------------------------------------------------------------ test hooks */

/* Not part of the stable interface.  Overrides how the work is spread over the GPU, for the
 * tests that show the bits depend on neither the block count nor the occupancy:
 *   grid_wgs > 0 sets the number of workgroups of the sum kernel and of the look-back scan
 *     kernel, also beyond the number that fit on the GPU at once (workgroups that start late
 *     claim their tiles when they start); 0 = the default;
 *   extra_lds_bytes in [0, 65536] adds that much dynamic LDS to every workgroup of the sum,
 *     look-back scan and radix-sort kernels, which lowers how many fit per compute unit.
 * Process-wide; DET_ERROR_INVALID_VALUE when out of range. */
det_status det_debug_set_launch(int grid_wgs, int extra_lds_bytes);

/* Not part of the stable interface.  chunk_log2 in [14, 24] sets the elements per partial of
 * the sum's first level (0 = default, 14).  Process-wide; DET_ERROR_INVALID_VALUE when out of
 * range. */
det_status det_debug_set_sum_chunk(int chunk_log2);

/* Not part of the stable interface.  The launch shape the library last used: the grid of the
 * sum kernel's first level, the grid of the look-back scan kernel and the scan workgroups the
 * runtime reported resident per compute unit for that launch (with its extra LDS).  Any
 * pointer may be NULL; values are 0 before the first such launch. */
void det_debug_last_launch(int64_t* sum_grid, int64_t* scan_grid, int64_t* scan_per_cu);

/* Not part of the stable interface.  Seeded pauses in the look-back scan: with max_us > 0,
 * the publishing thread of one status publication in four (tile totals, interval totals,
 * super-interval carries) first pauses for a time in [0, max_us] microseconds chosen by a
 * hash of seed, tile and publication kind, so successors find predecessors' status words
 * ready or not at different moments (drjit-core pull request "Make CUDA floating-point prefix
 * sums deterministic", section "Root cause": results must not depend on the states a tile
 * observes).  max_us in [0, 1000], 0 = off.  Process-wide; DET_ERROR_INVALID_VALUE when out
 * of range. */
det_status det_debug_set_scan_delay(unsigned seed, int max_us);

/* Not part of the stable interface.  Replaces the scan's anchor constants (tiles per anchor
 * interval A, intervals per super-interval A2; each in [1, 256], 0 = the spec's 256) so tests
 * can exercise many intervals and super-interval carries at small n against the oracle run
 * with the same constants.  Results then follow that variant's order, not SPEC v1.
 * Process-wide; DET_ERROR_INVALID_VALUE when out of range. */
det_status det_debug_set_scan_anchors(int A, int A2);

/* Not part of the stable interface.  Kernel timing for benchmarks: while enabled, every kernel
 * the library enqueues is bracketed by two HIP events recorded on the call's stream.
 * enable = 1 drops earlier records and starts recording, 0 drops them and stops; anything else
 * is DET_ERROR_INVALID_VALUE.  Recording adds an event pair per launch. */
det_status det_debug_kernel_timing(int enable);

/* Not part of the stable interface.  Waits for every recorded event pair, then writes one line
 * per kernel name, "name launches total_ms average_ms", into buf (at most len bytes including
 * the terminating NUL; buf may be NULL).  The records stay until det_debug_kernel_timing is
 * called again.  Launches whose events failed are counted in a last line starting with '#'.
 * Returns the bytes the full report needs, NUL included. */
size_t det_debug_kernel_report(char* buf, size_t len);

#ifdef __cplusplus
}
#endif

#endif /* DET_H */
