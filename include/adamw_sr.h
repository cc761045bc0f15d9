/*
 * adamw_sr.h -- C ABI of the fused AdamW step with stochastic-rounding bf16
 * write-back, for AMD Instinct MI355X (gfx950).
 *
 * The operation (pages cited by title and section):
 *   - "adamw-sr" (kernels hub page), intro, Usage, Method, Correctness:
 *     a decoupled-weight-decay Adam step with float32 moment states, f32 or
 *     bf16 parameters and gradients, bf16 parameters written back by
 *     unbiased stochastic rounding with no fp32 master copy; the random bits
 *     come from a counter-based Philox whose key is the pair (seed, step)
 *     and whose counter is derived from the element's position in the whole
 *     parameter set, so a tensor updated in one piece or in shards (each
 *     shard passing the position of its first element) gets the same bits;
 *   - "Add stochastic rounding and philox RNG helpers" (FlyDSL pull request),
 *     Primitives: philox_4x32(counter, key) -> four 32-bit words, and
 *     stochastic rounding f32 -> bf16 by adding 16 random bits to the 16
 *     dropped mantissa bits and truncating; discussion: stochastic rounding
 *     as a rounding mode of the narrowing conversion.
 *
 * Conventions shared by every entry point:
 *   - All device pointers are HIP device (or managed) memory owned by the
 *     caller; the library allocates no device memory and keeps no generator
 *     state (the generator is counter-based).
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream of
 *     the current device). The current device must be the stream's device.
 *     Work is enqueued asynchronously; no call synchronizes the host. A
 *     device-side fault surfaces at the caller's next synchronization.
 *   - Every call returns an asr_status. On a non-zero status nothing was
 *     enqueued (argument errors are found before any launch) unless the
 *     status is ASR_EHIP, and asr_last_error() describes the problem.
 *   - Element counts are int64_t; global positions are uint64_t and wrap
 *     modulo 2**64.
 *
 * Random-bit contract (the "stream"), used by asr_adamw_step and
 * asr_cvt_f32_bf16_sr: element i of a tensor whose first element sits at
 * global position base_index has position p = base_index + i (64-bit).
 * Its 16 random bits are the low 16 bits of word (p & 3) of
 * Philox4x32-10(counter = (lo32(p >> 2), hi32(p >> 2), 0, 0),
 *              key     = (seed, step)).
 * Philox4x32-10 is the published generator of Salmon et al. (SC 2011):
 * multipliers 0xD2511F53 (word 0) and 0xCD9E8D57 (word 2), key bumps
 * 0x9E3779B9 and 0xBB67AE85, 10 rounds.
 *
 * Rounding rules (bit patterns u of f32, results are bf16 patterns):
 *   SR: NaN -> (u >> 16) | 0x0040 (stays NaN, sign and top payload kept);
 *       otherwise (u + r16) >> 16 in 32-bit arithmetic.
 *   RN: NaN as above; otherwise round to nearest, ties to even.
 */
#ifndef ADAMW_SR_H
#define ADAMW_SR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum asr_status {
  ASR_OK = 0,
  ASR_EINVAL = 1,     /* an argument value is out of its documented range      */
  ASR_EDTYPE = 2,     /* a dtype code is neither ASR_F32 nor ASR_BF16          */
  ASR_EALIGN = 3,     /* a pointer is not aligned to its element size          */
  ASR_EWORKSPACE = 4, /* workspace NULL, smaller than required, or misaligned  */
  ASR_EHIP = 5        /* the HIP runtime reported an error (see last_error)    */
} asr_status;

enum { ASR_F32 = 0, ASR_BF16 = 1 };
enum { ASR_ROUND_SR = 0, ASR_ROUND_RN = 1 };

/* One tensor of the optimizer's list, flattened and contiguous. */
typedef struct asr_tensor {
  void* param;          /* numel elements of param_dtype, updated in place   */
  const void* grad;     /* numel elements of grad_dtype, read only           */
  float* exp_avg;       /* numel f32: first moment m, updated in place       */
  float* exp_avg_sq;    /* numel f32: second moment v, updated in place      */
  int64_t numel;        /* >= 0; a tensor with numel 0 is skipped            */
  uint64_t base_index;  /* global position of element 0 (random-bit stream)  */
  int32_t param_dtype;  /* ASR_F32 | ASR_BF16                                */
  int32_t grad_dtype;   /* ASR_F32 | ASR_BF16                                */
} asr_tensor;

/* Bytes of device workspace asr_adamw_step needs for this list (0 when
 * n_tensors <= 0 or tensors is NULL). Only the count of tensors and their
 * numel matter, so the size stays valid across steps of a fixed list. The
 * workspace holds the list's metadata and a table of one 32-bit entry per
 * 1,024-element slot (under 0.4% of the bf16 parameter bytes). A step whose
 * launches each cover at most 48 tensors (any list of at most 48 tensors)
 * passes the metadata in its kernel arguments and leaves the workspace
 * untouched; the workspace is still required. */
size_t asr_adamw_workspace_bytes(const asr_tensor* tensors, int32_t n_tensors);

/*
 * One AdamW step over a list of tensors, in one pass over memory.
 * ("adamw-sr" page: intro, Usage, Method, Correctness.)
 *
 * For every element, in binary32, each operation rounded to nearest even
 * and never fused into a multiply-add:
 *     m   = b1*m + omb1*g
 *     v   = b2*v + omb2*(g*g)
 *     p   = p*decay - step_size * (m / (sqrt(v)*inv_bc2_sqrt + eps32))
 * where g and p are the gradient and parameter upcast exactly to f32, and the
 * constants are formed once per call in binary64 (bc1 = 1 - beta1**step,
 * bc2 = 1 - beta2**step by binary powering) and rounded to binary32:
 *     decay = 1 - lr*weight_decay, b1 = beta1, omb1 = 1 - beta1, b2 = beta2,
 *     omb2 = 1 - beta2, step_size = lr/bc1, inv_bc2_sqrt = 1/sqrt(bc2),
 *     eps32 = eps    (asr_adamw_host_scalars returns them).
 * m and v are stored as f32. An f32 parameter is stored as computed; a bf16
 * parameter is rounded by SR (rounding = ASR_ROUND_SR; key (seed, step),
 * position base_index + i) or by RN (ASR_ROUND_RN).
 *
 * tensors      host array of n_tensors descriptors (read during the call only);
 *              the param, grad, exp_avg and exp_avg_sq buffers of all tensors
 *              must be pairwise disjoint (not checked here; the Python
 *              binding checks).
 * lr           >= 0, finite.       beta1, beta2   in [0, 1).
 * eps          >= 0, finite.       weight_decay   >= 0, finite.
 * step         1-based step count t, in [1, 2**32 - 1]; used for the bias
 *              corrections and as key word 1.
 * seed         key word 0.
 * workspace    device buffer of at least asr_adamw_workspace_bytes(tensors,
 *              n_tensors) bytes, 16-byte aligned, owned by the caller. Its
 *              contents are overwritten (stream-ordered); it must not be used
 *              by other work that runs concurrently with this step.
 * Errors: ASR_EINVAL (n_tensors < 0, NULL tensors with n_tensors > 0,
 * numel < 0, a NULL buffer in a non-empty tensor, hyperparameter or step out
 * of range, rounding code unknown, more than 2**32 slots of 1,024 elements
 * of one dtype pair), ASR_EDTYPE, ASR_EALIGN (param/grad not aligned to 2 or 4 bytes as
 * their dtype needs, m/v not 4-byte aligned), ASR_EWORKSPACE, ASR_EHIP.
 * Layout of the work: each tensor is walked in runs of 4 consecutive
 * elements, one run per GPU lane, shifted by s elements (0 <= s < 4) so
 * that every whole run starts on a vector-aligned address of all four
 * buffers (16 bytes for f32, 8 for bf16) -- a tensor cut out of aligned
 * buffers at any element offset has such a shift. Whole runs move with
 * vector accesses; the cut runs at either end, and every run of a tensor
 * whose buffers are misaligned against each other (no such shift), move
 * element by element. The results are the same either way.
 */
int asr_adamw_step(const asr_tensor* tensors, int32_t n_tensors,
                   double lr, double beta1, double beta2, double eps,
                   double weight_decay, int64_t step, uint32_t seed,
                   int32_t rounding, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * asr_adamw_step without a workspace argument, for callers that cannot
 * allocate device memory: code being captured into a HIP graph, tight
 * serving loops, harnesses that forbid hipMalloc. The call allocates
 * nothing (no hipMalloc, hipFree or allocating library routine): its
 * kernels use a static device array of 4 MiB ("scratch", one copy per GPU,
 * held until the process ends) in place of the workspace, found on the
 * first call on each device with that device current. Results are those
 * of asr_adamw_step bit for bit (the same kernels).
 * Limit: the list's metadata (60 bytes per tensor plus a few hundred) plus
 * a 4-byte slot-table entry per 1,024 elements of the tensors that are not
 * in a size class must fit in 4 MiB (a Llama-3-8B list needs about 18 KiB);
 * a larger list is rejected with ASR_EWORKSPACE before anything is
 * enqueued. Nothing in the scratch needs to start at zero: each call
 * writes all it reads. All calls on one GPU share its scratch, so calls
 * that may overlap on one GPU (other streams, other threads, several
 * replays of graphs in flight at once) race: order them on one stream.
 * Other arguments and errors as for asr_adamw_step.
 */
int asr_adamw_step_noalloc(const asr_tensor* tensors, int32_t n_tensors,
                           double lr, double beta1, double beta2, double eps,
                           double weight_decay, int64_t step, uint32_t seed,
                           int32_t rounding, void* stream);

/*
 * The eight binary32 constants asr_adamw_step uses for these
 * hyperparameters, in this order: decay, b1, omb1, b2, omb2, step_size,
 * inv_bc2_sqrt, eps32 (see asr_adamw_step). Host only; touches no device.
 * out: host array of 8 floats. Errors: ASR_EINVAL as for asr_adamw_step.
 */
int asr_adamw_host_scalars(double lr, double beta1, double beta2, double eps,
                           double weight_decay, int64_t step, float* out);

/*
 * Philox4x32-10 words of n_counters consecutive counters.
 * ("Add stochastic rounding and philox RNG helpers", Primitives.)
 * Call k (0 <= k < n_counters) uses counter
 *   (lo32(c), hi32(c), lo32(counter_upper), hi32(counter_upper)),
 *   c = counter_base + k (mod 2**64),
 * and key (seed, step); its words 0..3 go to out[4k .. 4k+3].
 * With counter_upper = 0 these are the calls of the random-bit stream.
 * out: device buffer of 4*n_counters uint32, 4-byte aligned.
 * Errors: ASR_EINVAL (n_counters < 0, out NULL with n_counters > 0),
 * ASR_EALIGN, ASR_EHIP.
 */
int asr_philox_4x32_fill(uint32_t* out, int64_t n_counters,
                         uint64_t counter_base, uint64_t counter_upper,
                         uint32_t seed, uint32_t step, void* stream);

/*
 * Stochastic-rounding conversion f32 -> bf16 of n elements.
 * ("Add stochastic rounding and philox RNG helpers", Primitives and
 * discussion: SR as a rounding mode of the conversion.)
 * out[i] = SR(in[i], r16(base_index + i)) with key (seed, step).
 * in: device, n f32, 4-byte aligned; out: device, n bf16 patterns, 2-byte
 * aligned; in and out must not overlap.
 * Errors: ASR_EINVAL (n < 0, NULL buffer with n > 0), ASR_EALIGN, ASR_EHIP.
 */
int asr_cvt_f32_bf16_sr(const float* in, uint16_t* out, int64_t n,
                        uint32_t seed, uint32_t step, uint64_t base_index,
                        void* stream);

/*
 * Round-to-nearest-even conversion f32 -> bf16 (the comparison mode; the
 * FlyDSL page's Consumer section keeps "rn" as the default rounding).
 * Same buffers and errors as asr_cvt_f32_bf16_sr.
 */
int asr_cvt_f32_bf16_rn(const float* in, uint16_t* out, int64_t n,
                        void* stream);

/*
 * Stochastic rounding f32 -> bf16 with the random bits supplied by the
 * caller: out[i] = SR(x[i], r16[i]) under the rule at the top of this file.
 * ("Add stochastic rounding and philox RNG helpers", Primitives: the
 * rounding primitive takes its random bits as an input.) The same device
 * rounding as asr_adamw_step and asr_cvt_f32_bf16_sr, so it is the hook
 * that checks the rounding apart from the generator.
 * x: device, n f32; r16: device, n uint16 random values; out: device, n bf16
 * patterns. Natural alignment. Errors: ASR_EINVAL, ASR_EALIGN, ASR_EHIP.
 */
int asr_sr_bf16_given_bits(const float* x, const uint16_t* r16, uint16_t* out,
                           int64_t n, void* stream);

/*
 * bf16 GEMM with a stochastic-rounding (or round-to-nearest) epilogue.
 * ("Add stochastic rounding and philox RNG helpers", Consumer section: the f32
 * accumulator of a bf16 GEMM is converted to bf16 by SR keyed per output
 * element from a seed, RN being the other rounding; Tests: SR within
 * tolerance of RN, seed-dependent, reproducible.)
 *
 *   C[m][n] = round( sum_k A[m][k] * B[n][k] )     0 <= m < M, 0 <= n < N
 *
 * i.e. C = A * B^T with A (M x K) and B (N x K) both row-major, K
 * contiguous (the layout of x and W in a linear layer y = x W^T). The sum
 * is accumulated in f32 on the matrix cores in an order of the library's
 * choosing (fixed for given M, N, K, so results are reproducible).
 * rounding ASR_ROUND_SR: element (m, n) is rounded with the 16 random bits
 * of stream position base_index + m*N + n under key (seed, step) -- the
 * stream and rule of asr_cvt_f32_bf16_sr, so C equals that conversion of
 * the f32 result bit for bit, and a block of rows [r0, r1) computed alone
 * with base_index + r0*N reproduces those rows of the whole product.
 * rounding ASR_ROUND_RN: round to nearest even (seed, step, base_index
 * unused).
 *
 * a: device bf16 patterns, row m at a + m*lda; b: device, row n at
 * b + n*ldb; c: device bf16 patterns, row m at c + m*ldc; c_f32: NULL, or
 * a device f32 buffer with the same row stride ldc that receives the
 * unrounded f32 result. No output may overlap an input.
 * Requirements: 0 <= M, N, K < 2**31; K, lda, ldb multiples of 8;
 * K <= lda < 2**22, K <= ldb < 2**22, ldc >= N; a and b 16-byte aligned; c and c_f32 aligned to
 * their element size; base_index + M*N <= 2**64. M or N = 0 writes
 * nothing; K = 0 writes zeros.
 * Errors: ASR_EINVAL (sizes, strides, rounding, NULL), ASR_EALIGN,
 * ASR_EHIP (launch failure). Runs on `stream`; does not synchronize.
 */
int asr_gemm_bf16(const uint16_t* a, int64_t lda, const uint16_t* b,
                  int64_t ldb, uint16_t* c, int64_t ldc, float* c_f32,
                  int64_t m, int64_t n, int64_t k, int32_t rounding,
                  uint32_t seed, uint32_t step, uint64_t base_index,
                  void* stream);

/*
 * 8-bit codes of a matrix with one scale a group, the operands of
 * asr_gemm_i8. x is rows x cols, row i at x + i*ldx. A group is a row of x
 * (transpose = 0) or a column of x (transpose = 1: q is then the transposed
 * matrix, cols x rows, so that a group's codes are contiguous either way).
 * For a group with largest magnitude amax:
 *   scale = f32(amax / 127),
 *   q = sign(x) * min(127, Q(|x| / scale)), of the exact quotient:
 *   ASR_ROUND_RN: to nearest, ties to even;
 *   ASR_ROUND_SR: floor(|x| / scale + r16 * 2**-16), r16 being the 16 bits of
 *   stream position base_index + i*cols + j under key (seed, step) for x's
 *   element (i, j), in both forms (rounding to either neighbour with
 *   probabilities that make the code unbiased up to 2**-17 of a step).
 * A group with an Inf or NaN gets scale NaN and codes 0; one whose scale
 * would be below 2**-126 (all zeros, or all tiny) scale 0 and codes 0.
 * Group g's codes start at q + g*ldq; they are followed by zeros up to the
 * next multiple of 16.
 * dtype: of x, ASR_F32 or ASR_BF16. scale: device, one f32 a group.
 * Requirements: 0 <= rows, cols < 2**31; ldx >= cols; ldq a multiple of 16, at
 * least the group's length; q 16-byte aligned; x and scale aligned to their
 * elements (x's rows starting on 16-byte addresses take the vector path);
 * fewer than 2**24 workgroups: of one row (four, up to 2048 columns), or in
 * the transposed form of one tile of 128 rows x 64 columns (and rows at most
 * 2**31 - 64); base_index + rows*cols <= 2**64; no buffer overlaps another. workspace: asr_quantize_i8_workspace_bytes
 * bytes of device memory, 16-byte aligned (0 bytes, NULL allowed, unless
 * transpose), as for asr_adamw_step.
 * Errors: ASR_EINVAL, ASR_EDTYPE, ASR_EALIGN, ASR_EWORKSPACE, ASR_EHIP. Runs
 * on `stream`; does not synchronize.
 */
size_t asr_quantize_i8_workspace_bytes(int64_t rows, int64_t cols, int32_t transpose);
int asr_quantize_i8(const void* x, int32_t dtype, int64_t ldx, int64_t rows,
                    int64_t cols, int32_t transpose, int8_t* q, int64_t ldq,
                    float* scale, int32_t rounding, uint32_t seed,
                    uint32_t step, uint64_t base_index, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * 8-bit integer GEMM with a scale for each row of both operands (for each
 * token and each output channel of a linear layer y = x W^T):
 *
 *   C[m][n] = round((f32(sum_k A[m][k] * B[n][k]) * scale_a[m]) * scale_b[n])
 *
 * A (M x K) and B (N x K) are int8, row-major, K contiguous; the sum is exact
 * (32-bit integers; any int8 values, -128 included), its conversion to f32
 * and the two products are rounded to nearest, and C is rounded to bf16 by
 * SR (position base_index + m*N + n under key (seed, step)) or RN, as
 * asr_gemm_bf16 rounds. c_f32: NULL, or a device f32 buffer with row stride
 * ldc that receives the value before that rounding.
 * Bytes past a row's K codes are never used, whatever they hold.
 * Requirements: 0 <= M, N < 2**31; 0 <= K < 2**17; lda, ldb multiples of 16,
 * at least K and below 2**23; ldc >= N; a and b 16-byte aligned; scales, c and c_f32
 * aligned to their element size; at most 2**23 - 256 tiles of 256 x 256;
 * base_index + M*N <= 2**64; no output overlaps an input. M or N = 0 writes
 * nothing; K = 0 writes products of 0.
 * Errors: ASR_EINVAL, ASR_EALIGN, ASR_EHIP. Runs on `stream`; does not
 * synchronize.
 */
int asr_gemm_i8(const int8_t* a, int64_t lda, const int8_t* b, int64_t ldb,
                const float* scale_a, const float* scale_b, uint16_t* c,
                int64_t ldc, float* c_f32, int64_t m, int64_t n, int64_t k,
                int32_t rounding, uint32_t seed, uint32_t step,
                uint64_t base_index, void* stream);

/*
 * A linear layer's three products in 8-bit integers, from bf16 matrices:
 *   forward:   y  = x w^T     x (tokens x k), w (n x k), y (tokens x n)
 *   backward:  dx = dy w      (NULL dx: not wanted; w is then not read)
 *              dw = dy^T x    (NULL dw: not wanted; x is then not read)
 * Each is asr_gemm_i8 (rounded to nearest) of the codes asr_quantize_i8 gives:
 * of the rows of x and w; of the rows of dy and the columns of w; of the
 * columns of dy and x. x and w are rounded to nearest, dy by `rounding`:
 * ASR_ROUND_SR (key (seed, step), element (t, j) at base_index + t*n + j, the
 * same bits in both products) or ASR_ROUND_RN. Results are those of the
 * separate calls bit for bit; what one matrix's two forms share is read and
 * drawn once.
 * Requirements: 0 <= tokens, n, k < 2**17; row strides (in elements) at least
 * the rows' lengths; matrices aligned to 2 bytes (rows starting on 16-byte
 * addresses take the vector paths); base_index + tokens*n <= 2**64; no output
 * overlaps an input. workspace: asr_linear_i8_workspace_bytes(tokens, n, k,
 * backward) bytes of device memory, 256-byte aligned, overwritten in stream
 * order (the codes: about one byte an element of every matrix read).
 * Errors: ASR_EINVAL, ASR_EALIGN, ASR_EWORKSPACE, ASR_EHIP. Run on `stream`;
 * do not synchronize.
 */
size_t asr_linear_i8_workspace_bytes(int64_t tokens, int64_t n, int64_t k,
                                     int32_t backward);
int asr_linear_i8_forward(const uint16_t* x, int64_t ldx, const uint16_t* w,
                          int64_t ldw, uint16_t* y, int64_t ldy,
                          int64_t tokens, int64_t n, int64_t k,
                          void* workspace, size_t workspace_bytes,
                          void* stream);
int asr_linear_i8_backward(const uint16_t* x, int64_t ldx, const uint16_t* w,
                           int64_t ldw, const uint16_t* dy, int64_t lddy,
                           uint16_t* dx, int64_t lddx, uint16_t* dw,
                           int64_t lddw, int64_t tokens, int64_t n, int64_t k,
                           int32_t rounding, uint32_t seed, uint32_t step,
                           uint64_t base_index, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * The same layer with x kept in 8 bits between the two calls. The forward
 * call also writes x's row codes and scales, those of its product
 * (asr_quantize_i8 of x's rows, to nearest): q (tokens rows ldq bytes apart) and
 * scale (tokens). The backward call takes them in x's place. With X the codes and s the scales,
 *   dw[n][k] = sum_t dy[t][n] s[t] X[t][k]:
 * the token's scale goes into the gradient, z = f32(dy[t][n] * s[t]), and
 * dw = asr_gemm_i8 of the codes of z's columns (by `rounding`, with dy's own
 * positions) and X turned round, with the scales of z and 1. x is rounded
 * once, in the forward product; dx is the same as above. A token with an Inf
 * or NaN in x makes all of dw NaN.
 * Requirements: as above; ldq a multiple of 16, at least k up to a multiple of
 * 16 and below 2**23; q 16-byte aligned, scale 4-byte aligned; n > 0 in the
 * forward call. workspace: of asr_linear_i8_workspace_bytes(1, n, k, 0) bytes in
 * the forward call (x's codes need no room there), in the backward call as above.
 */
int asr_linear_i8_forward_saved(const uint16_t* x, int64_t ldx,
                                const uint16_t* w, int64_t ldw, uint16_t* y,
                                int64_t ldy, int8_t* q, int64_t ldq,
                                float* scale, int64_t tokens, int64_t n,
                                int64_t k, void* workspace,
                                size_t workspace_bytes, void* stream);
int asr_linear_i8_backward_saved(const int8_t* q, int64_t ldq,
                                 const float* scale, const uint16_t* w,
                                 int64_t ldw, const uint16_t* dy, int64_t lddy,
                                 uint16_t* dx, int64_t lddx, uint16_t* dw,
                                 int64_t lddw, int64_t tokens, int64_t n,
                                 int64_t k, int32_t rounding, uint32_t seed,
                                 uint32_t step, uint64_t base_index,
                                 void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * Activations in 8 bits, with one scale for every 128 consecutive columns of a
 * row (the last block of a row has the rest). Codes and scale of a block are
 * those asr_quantize_i8 gives a row of the block's elements (x's element (i, j)
 * at stream position base_index + i*cols + j); what they stand for is f32(q *
 * scale), which asr_unpack_i8 writes, to nearest if x is bf16. x: rows x cols of
 * dtype, row i at x + i*ldx; q: row i at q + i*ldq, followed by zeros up to the
 * next multiple of 16; scale: rows x ceil(cols / 128) f32, contiguous.
 * Requirements: 0 <= rows < 2**31, 0 <= cols < 2**31 - 4096; ldx >= cols; ldq a
 * multiple of 16 that holds the columns up to a multiple of 16; q 16-byte
 * aligned, x and scale aligned to their elements; fewer than 2**31 pieces of 2048
 * elements (16 rows of 128 columns, to one row of 2048 where rows are that long);
 * base_index + rows*cols <= 2**64; no buffer overlaps another.
 * Errors: ASR_EINVAL, ASR_EDTYPE, ASR_EALIGN, ASR_EHIP. Run on `stream`; do not
 * synchronize.
 */
int asr_pack_i8(const void* x, int32_t dtype, int64_t ldx, int64_t rows,
                int64_t cols, int8_t* q, int64_t ldq, float* scale,
                int32_t rounding, uint32_t seed, uint32_t step,
                uint64_t base_index, void* stream);
int asr_unpack_i8(const int8_t* q, int64_t ldq, const float* scale,
                  int64_t rows, int64_t cols, void* x, int32_t dtype,
                  int64_t ldx, void* stream);

/*
 * Layer norm of rows of `cols` elements:
 *   mean = sum x / cols, rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps),
 *   xh = (x - mean) * rstd,  y = xh * weight + bias,
 * and its gradients, with g = dy * weight:
 *   dx = rstd * (g - sum g / cols - xh * sum (g xh) / cols),
 *   dweight = sum over rows of dy * xh,  dbias = sum over rows of dy.
 * mean and rstd are formed in 64 bits, the rest in 32; the sums over rows take an order
 * that depends on the sizes only, in several levels, so that rounding them costs at most
 * (342 + 3 sqrt(rows / 256 + rows cols / 2**22)) 2**-24 of the sums of the magnitudes.
 * x - mean and rstd have to fit binary32. weight, bias: cols elements of param_dtype,
 * NULL: 1 and 0. stat: NULL, or rows x 4 f32 that the backward call takes.
 * q, scale: NULL, or they receive asr_pack_i8's codes (to nearest) of xh,
 * computed in 64 bits; the backward call then takes them, with x NULL, and uses what
 * they stand for. dx, dweight, dbias: NULL where not wanted; dweight and dbias
 * of param_dtype, not accumulated into.
 * y and dx have contiguous rows and x's dtype, as dy. An Inf or NaN in a row makes
 * its y and dx NaN.
 * Requirements: 0 <= rows < 2**24, 0 <= cols <= 2**24; row strides at least
 * cols; ldq, q and scale as for asr_pack_i8; eps >= 0, finite; stat 16-byte
 * aligned, the rest aligned to its elements; no output overlaps an input, but
 * y may be x (with its row stride cols) unless x is kept for the backward call.
 * workspace (with dweight or dbias):
 * asr_layer_norm_backward_workspace_bytes(rows, cols) bytes of device memory,
 * 16-byte aligned. Errors: ASR_EINVAL, ASR_EDTYPE, ASR_EALIGN, ASR_EWORKSPACE,
 * ASR_EHIP. Run on `stream`; do not synchronize.
 */
int asr_layer_norm_forward(const void* x, int32_t dtype, int64_t ldx,
                           int64_t rows, int64_t cols, const void* weight,
                           const void* bias, int32_t param_dtype, double eps,
                           void* y, float* stat, int8_t* q, int64_t ldq,
                           float* scale, void* stream);
size_t asr_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols);
int asr_layer_norm_backward(const void* dy, int64_t ld_dy, const void* x,
                            int64_t ldx, const int8_t* q, int64_t ldq,
                            const float* scale, const float* stat,
                            int32_t dtype, int64_t rows, int64_t cols,
                            const void* weight, int32_t param_dtype, void* dx,
                            void* dweight, void* dbias, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * The gated activation of an MLP, sig(g) = 1 / (1 + exp(-g)):
 *   y = g sig(g) u,   dup = dy g sig(g),
 *   dgate = dy u sig(g) (1 + g (1 - sig(g))).
 * All matrices rows x cols of dtype with row strides of their own, so that
 * gate and up may be the halves of one matrix, as may their gradients. q_gate,
 * s_gate, q_up, s_up: NULL, or they receive asr_pack_i8's codes (to nearest) of
 * gate and up, both with row stride ldq; the backward call takes either gate and
 * up or these, and then uses what they stand for.
 * Requirements: sizes, codes and alignment as for asr_pack_i8; row strides at least
 * cols; no output overlaps an input, but in the forward call y may be gate or
 * up, and in the backward call dgate may be dy, gate or up, and dup another of them (with the same
 * stride). A sig(g) below 2**-126 may be taken as 0. Errors: ASR_EINVAL, ASR_EDTYPE,
 * ASR_EALIGN, ASR_EHIP. Run on `stream`; do not synchronize.
 */
int asr_silu_mul_forward(const void* gate, int64_t ld_gate, const void* up,
                         int64_t ld_up, int32_t dtype, int64_t rows,
                         int64_t cols, void* y, int64_t ld_y, int8_t* q_gate,
                         float* s_gate, int8_t* q_up, float* s_up, int64_t ldq,
                         void* stream);
int asr_silu_mul_backward(const void* dy, int64_t ld_dy, const void* gate,
                          int64_t ld_gate, const void* up, int64_t ld_up,
                          const int8_t* q_gate, const float* s_gate,
                          const int8_t* q_up, const float* s_up, int64_t ldq,
                          int32_t dtype, int64_t rows, int64_t cols,
                          void* dgate, int64_t ld_dgate, void* dup,
                          int64_t ld_dup, void* stream);

/*
 * Embedding: y[t] = f32(table[ids[t]]) * f32(scale), rounded to nearest, and
 * the table's gradient dtable[v] = (sum of dy[t], ids[t] = v) * f32(scale),
 * summed in f32 in an order that ids fixes (equal calls give equal bits; for m tokens of
 * an id off by at most (min(m, 518 + 3 sqrt(n / 512)) + 2) 2**-24 of the sum of the
 * magnitudes) and rounded once; rows of ids without a token are 0, and dtable is written whole.
 * ids: n ids on the device, 64-bit (ids_64 = 1) or 32-bit integers. An id outside
 * [0, vocab) gives a row of NaN and no gradient; padding_idx (-1: none) an
 * ordinary row and no gradient. table: vocab rows, ld elements apart; y and
 * dtable contiguous; dy's rows ld_dy elements apart; all of dtype.
 * Requirements: 0 <= n, vocab < 2**31; 0 <= dim <= 2**24; a gradient of
 * fewer than 2**24 workgroups' work (2048 columns, or rows side by side with 128
 * columns each at least: 64 GB of bf16 rows of whole 2048 columns);
 * row strides at least dim; pointers aligned to their elements; scale finite
 * in binary32; no output overlaps an input. workspace:
 * asr_embedding_backward_workspace_bytes(n, vocab, dim) bytes of device
 * memory, 256-byte aligned (0 bytes, NULL allowed, for n = 0 and for up to 1024
 * tokens of a small table). Errors:
 * ASR_EINVAL, ASR_EDTYPE, ASR_EALIGN, ASR_EWORKSPACE, ASR_EHIP. Run on
 * `stream`; do not synchronize.
 */
int asr_embedding_forward(const void* ids, int32_t ids_64, int64_t n,
                          const void* table, int32_t dtype, int64_t ld,
                          int64_t vocab, int64_t dim, double scale, void* y,
                          void* stream);
size_t asr_embedding_backward_workspace_bytes(int64_t n, int64_t vocab,
                                              int64_t dim);
int asr_embedding_backward(const void* ids, int32_t ids_64, int64_t n,
                           const void* dy, int64_t ld_dy, int32_t dtype,
                           int64_t vocab, int64_t dim, double scale,
                           int64_t padding_idx, void* dtable, void* workspace,
                           size_t workspace_bytes, void* stream);

/*
 * Orthogonalisation of n matrices of one shape by Newton-Schulz products:
 *
 *   X = G / (|G|_F + eps), its short side first;
 *   steps times:  A = X X^T,  X <- a X + (b A + c A A) X;
 *   out = bf16(X), in G's orientation, rounded to nearest even.
 *
 * With (a, b, c) = (3.4445, -4.775, 2.0315) and 5 steps, singular values from
 * about 1/100 of |G|_F up come out between about 0.7 and 1.2 (the update of
 * the Muon optimizer). The products run on the matrix cores with f16 operands
 * and f32 sums, X itself held as two f16 numbers. After these 5 steps the result is
 * off the exact one (relative, Frobenius norm; rounding it to bf16 adds its own
 * 1.7e-3) by up to
 *   3e-3    entries of varied size (Gaussian, uniform, of any rank), short side 64
 *           or more;
 *   4e-3    the same, short side 16 to 63;
 *   1.8e-2  where the roundings are few or alike and do not average: short sides
 *           below 16, entries of one magnitude (ones, signs), orthogonal rows, a
 *           single entry. (One singular value alone: 4.5e-2 at the very worst.)
 * A G with |G|_F below 1e-5 eps falls under f16's range as X: O, itself below 5e-3
 * then, is off by up to 4.1e-5 in all. The norm is summed in 64 bits. A G of
 * zeros gives zeros (with eps > 0); an Inf or NaN in G makes all
 * of its result NaN.
 *
 * g, out: host arrays of n device pointers (read during the call only), each
 * to rows x cols contiguous elements, of g_dtype (ASR_F32 or ASR_BF16) and of
 * bf16. out[k] may be g[k] itself (bf16); otherwise no buffer overlaps another.
 * Requirements: 0 <= rows, cols <= 2**20; 1 <= steps <= 64; eps >= 0; the coefficients
 * must keep singular values in [0, 1] below 1.4 over the steps, and
 * |b x^2 + c x^4| below 3.75 there. workspace:
 * asr_newton_schulz_workspace_bytes(n, rows, cols) bytes of device memory,
 * 256-byte aligned, overwritten in stream order: calls that may overlap need
 * a workspace each. (About 8 bytes an element and 4 a squared short side, both
 * sides counted up to the next multiple of 64, for
 * at most 32 matrices at a time, and of large ones about 4 GiB; none for matrices
 * that one workgroup holds, such as 128 x 128 or 64 x 512.)
 * Errors: ASR_EINVAL, ASR_EDTYPE, ASR_EALIGN, ASR_EWORKSPACE, ASR_EHIP. Runs
 * on `stream`; does not synchronize; nothing is allocated.
 */
size_t asr_newton_schulz_workspace_bytes(int32_t n, int64_t rows, int64_t cols);
int asr_newton_schulz(const void* const* g, uint16_t* const* out, int32_t n,
                      int64_t rows, int64_t cols, int32_t g_dtype,
                      int32_t steps, double a, double b, double c, double eps,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * One Muon step over n matrices, of any shapes and of one type. For each, in binary32,
 * every operation rounded on its own:
 *   m <- momentum*m + g,   u = nesterov ? g + momentum*m : m,
 *   O = the orthogonalisation of u as above (before its rounding to bf16),
 *   p <- p*decay - eta*O,  decay = f32(1 - lr*weight_decay),
 *                          eta = f32(lr*lr_factor).
 * A bf16 parameter is rounded by SR (element (i, j) at position base_index +
 * i*cols + j under key (seed, step)) or RN, an f32 one stored as computed (O
 * keeps the accuracy above). lr_factor: the adjustment to the shape, for
 * example sqrt(max(1, rows / cols)), or 0.2 sqrt(max(rows, cols)).
 * lr, weight_decay, lr_factor >= 0; 0 <= momentum < 1; step in [1, 2**32 - 1].
 * tensors: host array, read during the call only; buffers pairwise disjoint.
 * workspace: asr_muon_workspace_bytes(tensors, n) bytes (only the shapes
 * matter), as for asr_newton_schulz; other arguments and errors as there.
 */
typedef struct asr_muon_tensor {
  void* param;          /* rows*cols elements of param_dtype, updated in place */
  const void* grad;     /* rows*cols elements of grad_dtype, read only         */
  float* momentum;      /* rows*cols f32, updated in place                     */
  int64_t rows, cols;   /* in [0, 2**20]; an empty matrix is skipped           */
  uint64_t base_index;  /* global position of element 0 (random-bit stream)    */
  double lr_factor;     /* finite, >= 0                                        */
} asr_muon_tensor;
size_t asr_muon_workspace_bytes(const asr_muon_tensor* tensors, int32_t n);
int asr_muon_step(const asr_muon_tensor* tensors, int32_t n,
                  int32_t param_dtype, int32_t grad_dtype, double lr,
                  double momentum, int32_t nesterov, double weight_decay,
                  int32_t ns_steps, double ns_a, double ns_b, double ns_c,
                  double eps, int64_t step, uint32_t seed, int32_t rounding,
                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Random numbers on the library's stream, beyond rounding.
 * ("Add stochastic rounding and philox RNG helpers", discussion: the
 * counter-based generator as a general facility for dropout and
 * initialisation; "adamw-sr", Method: keyed by (seed, step), indexed by the
 * global position of the element.)
 * Position p = base_index + i takes 32-bit word W = word p & 3 of the
 * Philox4x32-10 call with counter (lo32(p >> 2), hi32(p >> 2), 0, 0) and key
 * (seed, step) -- the stream asr_philox_4x32_fill writes. All arithmetic is
 * binary32 without contraction; an ASR_BF16 output is the round-to-nearest-
 * even of the binary32 value. A tensor split into pieces that each pass
 * their own base_index reproduces the whole bit for bit.
 *
 * asr_random_uniform: out[i] = f32(low) + f32(high - low) * U,
 *   U = (W >> 8) * 2**-24 in [0, 1). low, high and high - low finite in
 *   binary32.
 * asr_random_normal: Box-Muller on position pairs (2q, 2q + 1):
 *   u1 = ((W(2q) >> 8) + 1) * 2**-24, u2 = (W(2q + 1) >> 8) * 2**-24,
 *   r = sqrt(-2 ln u1); z(2q) = r cos(2 pi u2), z(2q + 1) = r sin(2 pi u2);
 *   out[i] = f32(mean) + f32(std) * z. ln is 2 ln 2 * |log2|, and log2,
 *   sin and cos are gfx950's transcendental instructions (v_log_f32,
 *   v_sin_f32, v_cos_f32), whose error over every input they can receive
 *   here is measured by asr_box_muller_given_words; values are reproducible
 *   on this library but not bit-identical to other implementations.
 *   mean and std finite in binary32, std >= 0.
 * asr_dropout: drop probability p in [0, 1). Element i is dropped when
 *   W < floor(p * 2**32); y[i] = x[i] * (dropped ? 0 : f32(1 / (1 - p))), one
 *   binary32 multiply (a dropped Inf or NaN gives NaN, a dropped negative
 *   value -0). mask: NULL, or n bytes receiving 1 for kept, 0 for dropped.
 *   x and y may be the same buffer (in place).
 *
 * out, x, y: device, n elements of dtype (ASR_F32 or ASR_BF16), aligned to
 * the element size (16-byte f32 / 8-byte bf16 alignment takes the vector
 * path). Errors: ASR_EDTYPE, ASR_EINVAL (sizes, parameters, NULL),
 * ASR_EALIGN, ASR_EHIP. Run on `stream`; do not synchronize.
 */
int asr_random_uniform(void* out, int32_t dtype, int64_t n, double low,
                       double high, uint32_t seed, uint32_t step,
                       uint64_t base_index, void* stream);
int asr_random_normal(void* out, int32_t dtype, int64_t n, double mean,
                      double std, uint32_t seed, uint32_t step,
                      uint64_t base_index, void* stream);
int asr_dropout(const void* x, void* y, uint8_t* mask, int32_t dtype,
                int64_t n, double p, uint32_t seed, uint32_t step,
                uint64_t base_index, void* stream);

/*
 * Measurement support: copies `bytes` bytes from src to dst with a kernel
 * built like the AdamW step (one slot of 16 KiB per workgroup, 128-bit loads
 * and stores, the step's residency cap; one address window per XCD). The benchmark
 * quotes the step's bandwidth against this copy's as well as against the
 * HBM peak. src, dst: device, 16-byte aligned, not overlapping; bytes a
 * multiple of 16. Errors: ASR_EINVAL, ASR_EALIGN, ASR_EHIP.
 */
int asr_stream_copy(void* dst, const void* src, int64_t bytes, void* stream);

/*
 * Measurement support: what HBM gives a plain stream under the launch
 * structure of asr_stream_copy (16 KiB slot per workgroup, 128-bit
 * accesses, XCD windows, residency cap). The benchmark reports these
 * beside the AdamW step as the memory ceiling it is measured against.
 *   ASR_PROBE_READ   reads `bytes` bytes of src. Fill src with equal 16-byte
 *                    words (e.g. all bytes alike): the kernel then writes
 *                    nothing; dst is a 16-byte sink that it could write
 *                    otherwise.
 *   ASR_PROBE_WRITE  writes `bytes` bytes of dst (src unused, may be NULL).
 *   ASR_PROBE_COPY   asr_stream_copy(dst, src, bytes).
 * Buffers device, 16-byte aligned; bytes a multiple of 16.
 * Errors: ASR_EINVAL (kind, bytes < 0, NULL), ASR_EALIGN, ASR_EHIP.
 */
enum { ASR_PROBE_READ = 0, ASR_PROBE_WRITE = 1, ASR_PROBE_COPY = 2 };
int asr_hbm_probe(int32_t kind, void* dst, const void* src, int64_t bytes,
                  void* stream);

/*
 * Measurement support: the memory traffic of asr_adamw_step over this list
 * without its arithmetic -- the same launch plan, slots, runs, vector and
 * element accesses, windows and residency cap, reading param, grad,
 * exp_avg and exp_avg_sq and writing param, exp_avg and exp_avg_sq of
 * every element, with param := param XOR grad (for a bf16 param, the high
 * halves of the upcast values) and the moments written back as read. It
 * DESTROYS the parameters; it is a bandwidth probe of the step's access
 * pattern (four streams read, three written), not an optimizer.
 * Arguments, workspace and errors as for asr_adamw_step.
 */
int asr_adamw_stream_probe(const asr_tensor* tensors, int32_t n_tensors,
                           void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * Test support: the Box-Muller pair of asr_random_normal from given words:
 * zc[i], zs[i] = r cos(2 pi u2), r sin(2 pi u2) with u1, u2 from
 * w_even[i], w_odd[i] as above -- the same device function, so its error
 * can be measured over every possible input. All buffers: device, n
 * 4-byte elements. Errors: ASR_EINVAL, ASR_EALIGN, ASR_EHIP.
 */
int asr_box_muller_given_words(const uint32_t* w_even, const uint32_t* w_odd,
                               float* zc, float* zs, int64_t n, void* stream);

/*
 * Test support: the binary32 square root and division exactly as the AdamW
 * kernel evaluates them: sqrt_out[i] = sqrt(a[i]), div_out[i] = a[i] / b[i],
 * both correctly rounded (to nearest even, subnormals kept).
 * All buffers: device, n floats, 4-byte aligned.
 * Errors: ASR_EINVAL, ASR_EALIGN, ASR_EHIP.
 */
int asr_f32_sqrt_div(const float* a, const float* b, float* sqrt_out,
                     float* div_out, int64_t n, void* stream);

/* Text for the last non-OK status returned on this thread ("" if none). The
 * pointer stays valid until the next library call on this thread. */
const char* asr_last_error(void);

/* ABI version of this header and library (major * 100 + minor). */
int asr_abi_version(void);

#define ASR_ABI_VERSION 109

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_SR_H */
