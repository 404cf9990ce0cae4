/*
 * pq.h -- C ABI of libpq, the gfx950 (MI355X) implementation of the ParetoQ
 * quantized linear layer: per-row fake-quantization of fp32 shadow weights at
 * 1 / 1.58 / 2 / 3 / 4 bits, its straight-through backward with the learned
 * per-row scale's gradient, 2-bit (and 4-bit) export packing, and the
 * packed-weight x bf16-activation GEMM used at deployment.
 *
 * Sources (web pages, cited by title and section):
 *   [Note]     "ParetoQ, the strongest low-bit QAT I could find" -- sections
 *              "QAT versus PTQ", "Finding 3", "The 2-bit recipe, in full",
 *              "Paper vs. code".
 *   [Rebuttal] "ParetoQ: Improving Scaling Laws in Extremely Low-bit LLM
 *              Quantization" -- authors' replies, part on why SEQ beats LSQ.
 *   [News]     "Meta's ParetoQ compares five bit widths and puts the accuracy
 *              cliff at 1 bit" -- speed and storage paragraphs.
 *   [Abstract] "ParetoQ: Scaling Laws in Extremely Low-bit LLM Quantization".
 *
 * Conventions shared by every entry point
 *   Memory     Every array argument is a DEVICE pointer owned by the caller;
 *              the library keeps no pointer after the call returns and never
 *              allocates or frees device memory: the GEMM's scratch (split-K
 *              partial sums) is a caller-owned
 *              workspace sized by pq_gemm_workspace_bytes.  The one
 *              exception is pq_gemm_noalloc, whose scratch is a fixed array
 *              inside the library (see there).  Arrays are row-major and
 *              contiguous
 *              (leading dimension = cols), except the exported codes of
 *              pq_pack_w2 / pq_pack_w4 (the export byte order below).  Weight matrices are [out, in]:
 *              a "row" is one output channel, the unit the scale alpha
 *              belongs to ([Note] "Paper vs. code": one learned scale per
 *              row, shape (rows, 1)).
 *   Streams    `stream` is a hipStream_t (NULL = the null stream).  Calls only
 *              enqueue work on it and return, without waiting on the host;
 *              results are ready when the stream is.  Apart from
 *              pq_gemm_noalloc's scratch the library holds no global mutable
 *              state, so calls from several host threads are safe, and every
 *              call can be captured into a HIP graph (including its first
 *              call).
 *   bf16       bf16 arrays are passed as void* and hold IEEE bfloat16 bit
 *              patterns; every cast to bf16 rounds to nearest-even.
 *   Errors     Arguments are checked on the host before anything is enqueued:
 *              a NULL required pointer -> PQ_ERR_NULL; rows, cols, M, N or K
 *              negative, cols not a positive multiple of 8, K not a
 *              positive multiple of 64 or above 2^24, or N above 2^24 ->
 *              PQ_ERR_SHAPE; an
 *              unknown mode,
 *              flag or dtype -> PQ_ERR_MODE; an array pointer not 16-byte
 *              aligned -> PQ_ERR_ALIGN; a bad descriptor table or grad_scale
 *              -> PQ_ERR_ARG.  A failed launch -> PQ_ERR_HIP.  On any error
 *              nothing is enqueued.  Zero rows (or M = 0 / N = 0) is valid
 *              and enqueues nothing; the array pointers of such an empty
 *              matrix are not checked or used.
 *   Inputs     Weights, scales and gradients must be finite (not checked;
 *              outputs are unspecified otherwise).  A scale alpha <= 1e-5 is
 *              used as 1e-5 in the arithmetic (and stored unchanged), so an
 *              all-zero row gives finite outputs.
 */
#ifndef PQ_H_
#define PQ_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pq_status {
    PQ_OK = 0,
    PQ_ERR_NULL = 1,
    PQ_ERR_SHAPE = 2,
    PQ_ERR_MODE = 3,
    PQ_ERR_ALIGN = 4,
    PQ_ERR_UNSUPPORTED = 5,
    PQ_ERR_HIP = 6,
    PQ_ERR_ARG = 7
} pq_status;

/* Bit widths of the unified framework ([Abstract]: 1, 1.58, 2, 3, 4 bits).
 * SEQ at 1.58 and 2 bits, LSQ at 3 and 4 bits ([Note] "Paper vs. code",
 * dispatch row); the two LSQ grids the pages set against SEQ at 2 and 1.58
 * bits ([Rebuttal], part on why SEQ beats LSQ) are the ablation modes 5 and
 * 6.  Level sets, in units of alpha:
 *   PQ_W1_BINARY         {-1, +1}            sign(w), sign(0) = +1
 *   PQ_W158_SEQ_TERNARY  {-2/3, 0, +2/3}     ([Note] "Finding 3"; bins of
 *                                             [Rebuttal], 1.58-bit bullet)
 *   PQ_W2_SEQ            {-3/4,-1/4,1/4,3/4} ([Note] "Finding 3" and the SEQ
 *                                             formula row of "Paper vs. code")
 *   PQ_W3_LSQ            {-4 .. 3}           ([Note] "Finding 3": integer grid)
 *   PQ_W4_LSQ            {-8 .. 7}
 *   PQ_W2_LSQ            {-2, -1, 0, 1}      ([Rebuttal], 2-bit bullet)
 *   PQ_W158_LSQ          {-1, 0, 1}          (weights scaled to [-1, 1];
 *                                             [Rebuttal], 1.58-bit bullet)
 * LSQ clips x to [Qn, Qp] (the set's ends) and rounds half-to-even.
 * Stored codes: 1 bit for binary (0 -> -1, 1 -> +1); 2 bits for ternary and
 * 2-bit SEQ (code = step + 1 resp. step + 2, so ternary never stores 3; the
 * [News] storage paragraph notes ternary is commonly held in 2-bit integers);
 * a 4-bit nibble for 3- and 4-bit LSQ (code = step + 2^(b-1)); 2 bits for
 * the ablation grids (code = step - Qn).  Codes are a bit stream
 * per row, first element in the lowest bits of the first byte. */
typedef enum pq_mode {
    PQ_W1_BINARY = 0,
    PQ_W158_SEQ_TERNARY = 1,
    PQ_W2_SEQ = 2,
    PQ_W3_LSQ = 3,
    PQ_W4_LSQ = 4,
    PQ_W2_LSQ = 5,
    PQ_W158_LSQ = 6
} pq_mode;

/* pq_quantize_fwd flag: compute alpha from the row first and store it
 * ([Note] "The 2-bit recipe" table and the scale-init row of "Paper vs.
 * code": alpha = max|w| for SEQ and ternary, max|w| / Qp for LSQ with
 * Qp = 2^(b-1)-1, i.e. 3, 7, and 1 for both ablation grids;
 * mean|w| for 1 bit, summed in binary64). */
#define PQ_INIT_ALPHA 1u

/* pq_quantize_fwd flag: write `codes` in the export byte order of
 * pq_pack_w2 (pq_packed_bytes(mode, rows, cols) bytes, padding zeroed)
 * instead of row-major, so that the next GEMM can read them directly (the
 * training forward through pq_gemm_f32a, with no bf16 weights written or
 * read).  Deployable widths only (else PQ_ERR_MODE); codes must then be
 * non-NULL. */
#define PQ_CODES_EXPORT 2u

/* Upstream-gradient dtypes for pq_quantize_bwd. */
#define PQ_G_F32 0
#define PQ_G_BF16 1

/* Bytes per row of the code array of `mode` for `cols` weights
 * (cols * code_bits / 8), or -1 for a bad mode / cols. */
int64_t pq_code_row_bytes(int mode, int64_t cols);

/* Default alpha-gradient scale 1/sqrt(n * Qp) with n = rows * cols and
 * Qp = 1, 1, 1, 3, 7 for 1, 1.58, 2, 3, 4 bits ([Note] "Paper vs. code",
 * LSQ-gradient row: LSQ's 1/sqrt(n * Qp)).  Returns 0 for a bad argument. */
double pq_default_grad_scale(int mode, int64_t rows, int64_t cols);

/* Human-readable name of a status code (static string). */
const char *pq_status_str(pq_status s);

/* Library version string (static). */
const char *pq_version(void);

/*
 * pq_quantize_fwd -- forward fake-quantization of one weight matrix.
 * Every training step re-quantizes the fp32 shadow weights ([Note] "QAT
 * versus PTQ"); per weight w of row i, with a = max(alpha[i], 1e-5):
 *   x = w / a (IEEE division), clipped to [-0.99, 0.99] for SEQ / ternary
 *   ([Note] "Paper vs. code", first bullet) or to [Qn, Qp] for LSQ, rounded
 *   half-to-even onto the mode's grid; q = a * level; Wq = bf16(q), the cast
 *   to the activation dtype ([Note] "Paper vs. code", last bullet).
 *
 *   mode      pq_mode
 *   rows,cols W is [rows, cols] fp32; cols a positive multiple of 8
 *   W         in   [rows, cols] fp32 shadow weights
 *   alpha     in   [rows] fp32 per-row scale; with PQ_INIT_ALPHA it is OUT:
 *                  written with the row statistic, then used
 *   flags     0, PQ_INIT_ALPHA and/or PQ_CODES_EXPORT
 *   Wq_bf16   out  [rows, cols] bf16 fake-quantized weights, or NULL
 *   Wq_f32    out  [rows, cols] the same values before the bf16 cast, or NULL
 *   codes     out  [rows, pq_code_row_bytes(mode, cols)] packed codes, or NULL
 *   stream    hipStream_t
 */
pq_status pq_quantize_fwd(int mode, int64_t rows, int64_t cols, const float *W,
                          float *alpha, unsigned flags, void *Wq_bf16, float *Wq_f32,
                          uint8_t *codes, void *stream);

/*
 * pq_quantize_bwd -- straight-through backward of pq_quantize_fwd.
 * Per weight (same a and x as the forward, bit for bit):
 *   inside = x within the clip range, bounds included ([-0.99, 0.99] SEQ and
 *            ternary, [Qn, Qp] LSQ, [-1, 1] binary);
 *   dW     = G inside, exactly +0 outside -- the rounding is treated as the
 *            identity inside the range and the clamp is flat outside ([Note]
 *            "QAT versus PTQ" and the gradient paragraph of "The 2-bit
 *            recipe, in full");
 *   dalpha = grad_scale * sum_j s_j * G_j per row, with s = level - x inside
 *            and s = the boundary level outside (clipped weights still feed
 *            the scale), accumulated in binary64 and rounded once ([Note]
 *            "Paper vs. code", LSQ-gradient row).
 *   The boundary level is +-0.75 at 2-bit SEQ, +-fl32(2/3) for ternary (the
 *   level of the clipped value), Qn or Qp for the LSQ grids.  For 1 bit,
 *   sign(w) plays the part of the rounding, so the same rule reads
 *   s = sign(w) - x inside |x| <= 1 and s = sign(w) outside (sign(+-0) = +1).
 *   The pages name no binary gradient; this uniform reading is the library's
 *   own, and an alternative (s = sign(w) everywhere, the derivative of
 *   q = alpha * sign(w)) would change dalpha on every binary row.  The
 *   ternary outside value and the default grad_scale carry readings the
 *   pages do not pin either.
 *
 *   W, alpha   in   as in the forward (alpha is the value the forward used)
 *   G          in   [rows, cols] dL/dWq, fp32 (PQ_G_F32) or bf16 (PQ_G_BF16)
 *   g_dtype    PQ_G_F32 or PQ_G_BF16
 *   grad_scale the alpha-gradient scale; pass pq_default_grad_scale(...)
 *              for LSQ's 1/sqrt(n*Qp); must be finite
 *   dW         out  [rows, cols] fp32, or NULL; may alias G when g_dtype is
 *                   PQ_G_F32 (each element is read before it is written)
 *   dalpha     out  [rows] fp32
 *   mask_bits  out  [rows, cols/8] the `inside` bit per weight, first weight
 *                   in the lowest bit, or NULL
 */
pq_status pq_quantize_bwd(int mode, int64_t rows, int64_t cols, const float *W,
                          const float *alpha, const void *G, int g_dtype,
                          double grad_scale, float *dW, float *dalpha,
                          uint8_t *mask_bits, void *stream);

/*
 * Export byte order.  The exported codes are the forward's code rows
 * (pq_quantize_fwd `codes`: rb = cols * b / 8 bytes per row, eight 1-bit,
 * four 2-bit or two 4-bit codes per byte, first code lowest), reordered for
 * the deployment GEMM, which reads 16 rows x 64 bytes as one MFMA operand
 * ([News] speed paragraph: the 2-bit kernel consumes packed weights; the
 * pages fix four codes per byte and a bf16 scale per row, not a byte order):
 * 1. 2-bit codes only: each 4-byte word of a row (16 codes k0 .. k15, code
 *    ki in bits 2i .. 2i+1 of the little-endian word; the row zero-padded to
 *    whole words, rbw = rb rounded up to 4) is rewritten so that its byte j
 *    holds k(2j) in bits 0-1, k(8+2j) in bits 2-3, k(2j+1) in bits 4-5 and
 *    k(9+2j) in bits 6-7: masked with 0x33333333 the word's nibbles are
 *    codes k0 .. k7 in order (low nibble of each byte first), and shifted
 *    right by 2 and masked, k8 .. k15.  1- and 4-bit rows keep their bytes
 *    (rbw = rb).
 * 2. With Np = rows rounded up to a multiple of 16 and G = ceil(rb / 64):
 *    byte c of row n (c < rbw, n < rows) is stored at
 *      (c / 64) * Np * 64 + (n / 16) * 1024 + (n % 16) * 64 + c % 64,
 *    i.e. group-major runs of 64 bytes of every row, each 16-row tile 1 KB
 *    ordered [row][64 bytes].  Every other byte (rows rows .. Np - 1,
 *    bytes rbw .. 64 G - 1 of a row) is written as 0.  Total size
 *    G * Np * 64 bytes = pq_packed_bytes(mode, rows, cols).
 */
int64_t pq_packed_bytes(int mode, int64_t rows, int64_t cols);

/* Widths with a deployment format ("deployable" below): PQ_W1_BINARY in a
 * 1-bit container (eight codes per byte), PQ_W158_SEQ_TERNARY, PQ_W2_SEQ,
 * PQ_W2_LSQ and PQ_W158_LSQ in a 2-bit container, PQ_W3_LSQ and PQ_W4_LSQ
 * in a 4-bit one
 * (ternary is commonly held in 2-bit integers, [News] storage paragraph).
 * pq_packed_bytes returns -1 for a bad mode. */

/*
 * pq_pack_w2 -- export a 2-bit SEQ layer for deployment: the forward's codes
 * (the bytes of pq_quantize_fwd(PQ_W2_SEQ, ...) codes, bit for bit) in the
 * export byte order, and the scale rounded to bf16.  Memory savings exist
 * only after export ([Note] "Paper vs. code", last bullet); the deployed
 * GEMM consumes this format ([News] speed paragraph).
 *   W          in   [rows, cols] fp32, cols a positive multiple of 8
 *   alpha      in   [rows] fp32
 *   packed     out  pq_packed_bytes(PQ_W2_SEQ, rows, cols) bytes, export
 *                   byte order (above); every byte is written
 *   alpha_bf16 out  [rows] bf16
 */
pq_status pq_pack_w2(int64_t rows, int64_t cols, const float *W, const float *alpha,
                     uint8_t *packed, void *alpha_bf16, void *stream);

/* pq_pack -- the export of any deployable width (the same contract as
 * pq_pack_w2, with the width's code container); an other mode ->
 * PQ_ERR_MODE.  pq_pack_w2 is pq_pack(PQ_W2_SEQ, ...), pq_pack_w4
 * pq_pack(PQ_W4_LSQ, ...). */
pq_status pq_pack(int mode, int64_t rows, int64_t cols, const float *W, const float *alpha,
                  uint8_t *packed, void *alpha_bf16, void *stream);

/* pq_pack_w4 -- the 4-bit LSQ counterpart of pq_pack_w2 (two codes per byte,
 * low nibble first; pq_packed_bytes(PQ_W4_LSQ, rows, cols) bytes in the
 * export byte order), feeding pq_w4a16_gemm, the 4-bit comparison point of
 * the [News] speed paragraph. */
pq_status pq_pack_w4(int64_t rows, int64_t cols, const float *W, const float *alpha,
                     uint8_t *packed, void *alpha_bf16, void *stream);

/*
 * pq_gemm_workspace_bytes -- device workspace, in bytes, that the GEMM entry
 * points below need for this width and shape: 0 when the kernels chosen for
 * the shape use none, -1 for an unknown mode or a shape they reject.  The
 * kernel choice is a fixed function of (mode, M, N, K), so the value is the
 * same for every call with these arguments:
 *   M <= 16 (weight streaming): none;
 *   larger M with 64 x 256 (or 64 x 192) output tiles: when there are too
 *     few tiles to fill the chip, K is split over blocks, each split writes
 *     fp32 partial sums [splits, M, N] and a second kernel adds them in
 *     split order -- splits * M * N * 4 bytes; otherwise none;
 *   large M at 2-bit widths (K >= 2048; M >= 1024, or M >= 512 when N gives
 *     at least 512 tiles of 64 x 256): none (the kernel sums the activation
 *     rows for the level offset itself);
 *   short K at 2-bit widths (K <= 704, M >= 1024; the codes of a column
 *     tile stay in LDS): none.
 */
int64_t pq_gemm_workspace_bytes(int mode, int64_t M, int64_t N, int64_t K);

/*
 * pq_w2a16_gemm -- deployment GEMM with packed 2-bit SEQ weights and bf16
 * activations ([News] speed paragraph: 2-bit-weight kernel against FP16 and
 * 4-bit weights at a 16384 x 16384 weight; the layer has no bias, [Note]
 * "Paper vs. code"):
 *   Y[m, n] = bf16( alpha_bf16[n] * sum_k X[m, k] * level(code[n, k]) )
 * with level(c) = (c - 1.5) / 2, fp32 accumulation.
 *   M, N, K    X is [M, K]; K a positive multiple of 64 (so every packed
 *              row is a whole number of 16-byte pieces) and at most 2^24,
 *              0 <= N <= 2^24 (the kernels address up to 64 activation rows
 *              or one 64-byte group of all weight rows with 32-bit offsets);
 *              M >= 0
 *   X          in   [M, K] bf16 activations
 *   packed     in   pq_packed_bytes(PQ_W2_SEQ, N, K) bytes from pq_pack_w2
 *                   (export byte order; the padding bytes are never used)
 *   alpha_bf16 in   [N] bf16
 *   Y          out  [M, N] bf16
 *   workspace  scratch device memory of at least
 *              pq_gemm_workspace_bytes(PQ_W2_SEQ, M, N, K) bytes, 16-byte
 *              aligned, owned by the caller; its contents on entry do not
 *              matter and on return are unspecified.  May be NULL when that
 *              size is 0.  Two calls in flight at once (on different
 *              streams) need different workspaces.
 *   workspace_bytes  the size of `workspace` (>= 0)
 * Errors as above, and: workspace needed but NULL -> PQ_ERR_NULL; not
 * 16-byte aligned -> PQ_ERR_ALIGN; workspace_bytes too small or negative ->
 * PQ_ERR_ARG.
 * Caches: with M <= 16 the weight codes are read as non-temporal (streaming)
 * loads, so that they neither displace other data nor force dirty lines out
 * of the last-level cache; a later call on the same weight should not count
 * on finding them cached.  Larger M reads them with ordinary loads.
 */
pq_status pq_w2a16_gemm(int64_t M, int64_t N, int64_t K, const void *X,
                        const uint8_t *packed, const void *alpha_bf16, void *Y,
                        void *workspace, int64_t workspace_bytes, void *stream);

/* pq_w4a16_gemm -- the same GEMM on pq_pack_w4 weights
 * (pq_packed_bytes(PQ_W4_LSQ, N, K) bytes), level(c) = c - 8. */
pq_status pq_w4a16_gemm(int64_t M, int64_t N, int64_t K, const void *X,
                        const uint8_t *packed, const void *alpha_bf16, void *Y,
                        void *workspace, int64_t workspace_bytes, void *stream);

/* pq_gemm -- the same GEMM for any deployable width, on pq_pack(mode, ...)
 * weights, with the width's levels ([Note] "Finding 3"): ternary
 * (c - 1) * fl32(2/3), 2-bit SEQ (c - 1.5) / 2, 3-bit LSQ c - 4, 4-bit LSQ
 * c - 8, and the ablation grids c - 2 (2-bit LSQ) and c - 1 (1.58-bit LSQ);
 * an other mode -> PQ_ERR_MODE.  These are the widths whose accuracy
 * and storage the pages compare ([News] speed and storage paragraphs).
 * Workspace as pq_w2a16_gemm, sized by pq_gemm_workspace_bytes(mode, ...). */
pq_status pq_gemm(int mode, int64_t M, int64_t N, int64_t K, const void *X,
                  const uint8_t *packed, const void *alpha_bf16, void *Y,
                  void *workspace, int64_t workspace_bytes, void *stream);

/* pq_gemm_f32a -- pq_gemm with the binary32 scale of training (alpha [N]
 * fp32, as pq_quantize_fwd keeps it) instead of the exported bf16 one: the
 * QAT forward's linear layer computed from the codes, Y = bf16(alpha[n] *
 * sum_k X[m,k] * level(code[n,k])), with the codes written by
 * pq_quantize_fwd(..., PQ_CODES_EXPORT, ...).  It reads 1/8 or 1/4 of the
 * bytes of the fake-quantized bf16 weights and never materialises them; the
 * forward's own Wq = bf16(alpha * level) rounds each weight to bf16 first,
 * so the two differ by that rounding (relative 2^-9 per weight).  Errors
 * and workspace as pq_gemm; alpha NULL -> PQ_ERR_NULL. */
pq_status pq_gemm_f32a(int mode, int64_t M, int64_t N, int64_t K, const void *X,
                       const uint8_t *packed, const float *alpha, void *Y,
                       void *workspace, int64_t workspace_bytes, void *stream);

/*
 * pq_gemm_noalloc -- pq_gemm for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, kernels and results as pq_gemm, without the
 * workspace: the scratch the kernels need (split-K partial sums;
 * pq_gemm_workspace_bytes of the shape) is a fixed array of
 * PQ_NOALLOC_SCRATCH_BYTES bytes inside the library, one per GPU, looked up
 * on the first call made on that GPU and held until the process ends.  The
 * call allocates nothing and never waits on the host.
 *   A shape whose scratch need exceeds PQ_NOALLOC_SCRATCH_BYTES ->
 *   PQ_ERR_UNSUPPORTED, with nothing enqueued (use pq_gemm with a workspace).
 *   Other errors as pq_gemm.
 * Every call on one GPU shares that GPU's array, which keeps the last call's
 * contents (no part of it needs to start at zero): calls that overlap on one
 * GPU (on different streams, or from different host threads) race on it and
 * must be serialised by the caller.
 */
#define PQ_NOALLOC_SCRATCH_BYTES (((int64_t)32) << 20)
pq_status pq_gemm_noalloc(int mode, int64_t M, int64_t N, int64_t K, const void *X,
                          const uint8_t *packed, const void *alpha_bf16, void *Y, void *stream);

/*
 * Grouped launches: one kernel launch over a whole stack of matrices (for
 * example every projection of every layer of a model), since a training step
 * re-quantizes all of them with the same mode.
 *
 * pq_mat describes one matrix.  The caller fills an array of them twice --
 * in host memory (checked and used for launch sizing) and an identical copy
 * in device memory (read by the kernels); the two must hold the same values.
 * Unused fields may be NULL.  Any count >= 0 is accepted (large stacks are
 * split over several launches internally).
 */
typedef struct pq_mat {
    const float *W;       /* [rows, cols] fp32                             */
    float *alpha;         /* [rows] fp32 (in; out with PQ_INIT_ALPHA)      */
    void *wq_bf16;        /* fwd out [rows, cols] bf16, or NULL            */
    float *wq_f32;        /* fwd out [rows, cols] fp32, or NULL            */
    uint8_t *codes;       /* fwd out codes, or NULL                        */
    const void *G;        /* bwd in [rows, cols] (dtype per call)          */
    float *dW;            /* bwd out [rows, cols] fp32, or NULL            */
    float *dalpha;        /* bwd out [rows] fp32                           */
    uint8_t *mask_bits;   /* bwd out [rows, cols/8], or NULL               */
    double grad_scale;    /* bwd alpha-gradient scale for this matrix      */
    int64_t rows;
    int64_t cols;         /* positive multiple of 8                        */
    void *alpha_bf16;     /* export out [rows] bf16 (pq_pack_grouped)      */
} pq_mat;

/* Forward over `count` matrices; per matrix exactly pq_quantize_fwd.
 * descs_host / descs_dev: identical pq_mat[count] in host / device memory. */
pq_status pq_quantize_fwd_grouped(int mode, int count, const pq_mat *descs_host,
                                  const pq_mat *descs_dev, unsigned flags, void *stream);

/* Backward over `count` matrices; per matrix exactly pq_quantize_bwd with
 * that entry's grad_scale. */
pq_status pq_quantize_bwd_grouped(int mode, int count, const pq_mat *descs_host,
                                  const pq_mat *descs_dev, int g_dtype, void *stream);

/* Export over `count` matrices in one launch; per matrix exactly
 * pq_pack(mode, rows, cols, W, alpha, codes, alpha_bf16): `codes` receives
 * pq_packed_bytes(mode, rows, cols) bytes in the export byte order and
 * `alpha_bf16` the [rows] bf16 scales (the export of a whole model, [Note]
 * "Paper vs. code", last bullet: savings exist only after export). */
pq_status pq_pack_grouped(int mode, int count, const pq_mat *descs_host,
                          const pq_mat *descs_dev, void *stream);

/*
 * Fused QAT step: the straight-through backward of the current forward,
 * AdamW on W and alpha, and the next forward's fake-quantization, in one
 * pass over each row.  The recipe trains the shadow weights and the per-row
 * scale with AdamW at weight decay 0 and a cosine-decayed learning rate
 * ([Note] "The 2-bit recipe, in full", optimizer and learning-rate rows);
 * the pages give no update formula, so this is AdamW as published, with
 * decoupled weight decay, computed in binary32 in this order, one rounding
 * per operation (g = dW for W, g = dalpha for alpha):
 *   m'  = b1 * m + (1 - b1) * g
 *   v'  = b2 * v + ((1 - b2) * g) * g
 *   den = sqrt(v') / sqrt(1 - b2^t) + eps
 *   p'  = p * (1 - lr * wd) - (lr / (1 - b1^t)) * m' / den
 * where b1, 1 - b1, b2, 1 - b2, sqrt(1 - b2^t), eps, 1 - lr * wd and
 * lr / (1 - b1^t) are computed in binary64 on the host and rounded once to
 * binary32.  dW and dalpha are exactly pq_quantize_bwd's (from W, alpha and
 * G before the update); the outputs Wq / codes are exactly
 * pq_quantize_fwd's for the updated W and alpha.
 */
typedef struct pq_adamw {
    double lr;            /* this step's learning rate (the schedule is the caller's) */
    double beta1, beta2;  /* in [0, 1) */
    double eps;           /* > 0 */
    double weight_decay;  /* >= 0 (the recipe uses 0) */
    int64_t step;         /* t >= 1, for the bias corrections */
} pq_adamw;

/* One matrix of a fused step (grouped launches, as pq_mat). */
typedef struct pq_step_mat {
    float *W;             /* in/out [rows, cols] fp32 shadow weights        */
    float *alpha;         /* in/out [rows] fp32 scale                       */
    const void *G;        /* in [rows, cols] dL/dWq (dtype per call)        */
    float *mW;            /* in/out [rows, cols] first moment of W          */
    float *vW;            /* in/out [rows, cols] second moment of W         */
    float *m_alpha;       /* in/out [rows] first moment of alpha            */
    float *v_alpha;       /* in/out [rows] second moment of alpha           */
    void *wq_bf16;        /* out [rows, cols] next forward's bf16, or NULL  */
    uint8_t *codes;       /* out [rows, pq_code_row_bytes] codes, or NULL   */
    float *dalpha;        /* out [rows] this step's alpha gradient, or NULL */
    double grad_scale;    /* the alpha-gradient scale, as pq_quantize_bwd   */
    int64_t rows;
    int64_t cols;         /* positive multiple of 8                         */
} pq_step_mat;

/*
 * pq_qat_step -- the fused step on one matrix.  W, alpha and the four moment
 * arrays are updated in place; G is read only.  Wq_bf16, codes and dalpha
 * are optional outputs (NULL skips them).  hp is a host pointer read during
 * the call.  Errors as the other entry points; hp NULL -> PQ_ERR_NULL; a
 * hyper-parameter out of its range (or a non-finite one), or a non-finite
 * grad_scale -> PQ_ERR_ARG.  Weights, moments and gradients must be finite.
 */
pq_status pq_qat_step(int mode, int64_t rows, int64_t cols, float *W, float *alpha,
                      const void *G, int g_dtype, double grad_scale, float *mW, float *vW,
                      float *m_alpha, float *v_alpha, const pq_adamw *hp, void *Wq_bf16,
                      uint8_t *codes, float *dalpha, void *stream);

/* The fused step over `count` matrices in one launch; per matrix exactly
 * pq_qat_step.  descs_host / descs_dev: identical pq_step_mat[count] in host
 * / device memory; every entry must use the same set of optional outputs. */
pq_status pq_qat_step_grouped(int mode, int count, const pq_step_mat *descs_host,
                              const pq_step_mat *descs_dev, int g_dtype, const pq_adamw *hp,
                              void *stream);

/*
 * Diagnostics.  How the weights of each row spread over the levels -- the
 * level occupancy behind the SEQ-vs-LSQ argument ([Rebuttal], part on why
 * SEQ beats LSQ; [Note] "Finding 3" level sets) -- and how far training
 * moved the shadow weights from a reference ([Note] "QAT versus PTQ": QAT
 * compensates for the quantizer rather than reconstructing the weights).
 *
 * pq_num_levels -- levels of a mode (2, 3, 4, 8, 16 for 1, 1.58, 2, 3, 4
 * bits; 4 and 3 for the 2- and 1.58-bit LSQ grids), -1 for a bad mode.
 *
 * pq_level_stats -- from the forward's row-major codes ([rows,
 * pq_code_row_bytes(mode, cols)]): counts [rows, pq_num_levels(mode)] u32,
 * counts[i, c] = weights of row i stored with code c (code c is level c,
 * lowest first), and optionally entropy [rows] f64, -sum_c p_c log2 p_c with
 * p_c = counts[i, c] / cols (binary64; 0 for a row on one level).  Reads
 * 1/8 .. 1/2 byte per weight.
 *
 * pq_quantize_fwd_stats -- the forward of pq_quantize_fwd (alpha given, no
 * init) with the level statistics of pq_level_stats taken in the same pass,
 * from the codes as they are made: codes [rows, pq_code_row_bytes] are
 * written (required), Wq_bf16 [rows, cols] optionally (NULL: not written),
 * counts [rows, pq_num_levels(mode)] u32 (required) and entropy [rows] f64
 * (optional) as pq_level_stats defines them.  All pointers 16-byte aligned.
 * Errors as pq_quantize_fwd; codes or counts NULL -> PQ_ERR_NULL.
 *
 * pq_weight_movement -- sq_diff[i] = sum_j (W[i,j] - W0[i,j])^2 and
 * sq_ref[i] = sum_j W0[i,j]^2 per row, each difference and square in
 * binary64, summed in a fixed order (run-to-run identical); the relative
 * movement of a matrix is sqrt(sum sq_diff / sum sq_ref).  W, W0 fp32
 * [rows, cols] (16-byte aligned), outputs f64 [rows].
 */
int pq_num_levels(int mode);
pq_status pq_level_stats(int mode, int64_t rows, int64_t cols, const uint8_t *codes,
                         uint32_t *counts, double *entropy, void *stream);
pq_status pq_quantize_fwd_stats(int mode, int64_t rows, int64_t cols, const float *W,
                                const float *alpha, void *Wq_bf16, uint8_t *codes,
                                uint32_t *counts, double *entropy, void *stream);
pq_status pq_weight_movement(int64_t rows, int64_t cols, const float *W, const float *W0,
                             double *sq_diff, double *sq_ref, void *stream);

/*
 * Serving: rotary positions, a key-value cache held in 16, 8 or 4 bits, and
 * attention of one new token over it -- what a decode step needs between the
 * packed-weight GEMMs.  The conventions at the top of this file hold, with
 * these additions: activations may be strided (strides in elements, the last
 * dimension contiguous); a NULL stream is the null stream; sizes of zero
 * enqueue nothing; a NaN that is copied stays one, but a signalling one of a
 * 16-bit type becomes quiet.
 */

/* Element types of activations (PQ_G_F32 and PQ_G_BF16 have the same values). */
#define PQ_F32 0
#define PQ_BF16 1
#define PQ_F16 2

/* Pairs of a head's first `rot` channels that are rotated together:
 * PQ_ROPE_HALF (c, c + rot / 2); PQ_ROPE_INTERLEAVED (2c, 2c + 1). */
#define PQ_ROPE_HALF 0
#define PQ_ROPE_INTERLEAVED 1

/* How pq_rope_table scales the angles for contexts longer than the trained
 * one.  With f_c = base^(-2c / rot) and s = factor:
 *   PQ_ROPE_PLAIN   f_c
 *   PQ_ROPE_LINEAR  f_c / s
 *   PQ_ROPE_NTK     base replaced by base * s^(rot / (rot - 2)); rot > 2
 *   PQ_ROPE_YARN    f_c ((1 - g) / s + g), g = 1 - clamp((c - lo) / (hi - lo), 0, 1)
 *                   with lo, hi the (rounded outwards, clamped to [0, rot - 1])
 *                   pair indices that make `beta_fast` and `beta_slow` turns in
 *                   `trained` positions; cos and sin are also multiplied by
 *                   0.1 ln s + 1
 *   PQ_ROPE_BANDS   wavelength w = 2 pi / f_c: f_c / s where w > trained / beta_slow,
 *                   f_c where w < trained / beta_fast, in between
 *                   f_c ((1 - g) / s + g), g = (trained / w - beta_slow) / (beta_fast - beta_slow)
 */
#define PQ_ROPE_PLAIN 0
#define PQ_ROPE_LINEAR 1
#define PQ_ROPE_NTK 2
#define PQ_ROPE_YARN 3
#define PQ_ROPE_BANDS 4

typedef struct pq_rope_scaling {
    int32_t kind;         /* PQ_ROPE_PLAIN ..                               */
    int32_t reserved;     /* 0                                              */
    double factor;        /* s >= 1                                         */
    double trained;       /* YARN, BANDS: trained context length, > 0       */
    double beta_fast;     /* YARN: 32; BANDS: 4 (> beta_slow)               */
    double beta_slow;     /* YARN, BANDS: 1 (> 0)                           */
} pq_rope_scaling;

/* pq_rope_table -- the (cos, sin) rows of positions 0 .. max_pos - 1, made
 * once per model: table [max_pos, rot / 2, 2] fp32, each value rounded once
 * from binary64.
 *   rot      even, 2 .. 1024;  max_pos 0 .. 2^31 - 1, at most 2^33 - 512
 *            values in all;  base > 1
 *   scaling  host pointer read during the call, or NULL for PQ_ROPE_PLAIN
 * An unknown kind -> PQ_ERR_MODE; base or a scaling value out of range (or
 * not finite) -> PQ_ERR_ARG. */
pq_status pq_rope_table(int64_t max_pos, int64_t rot, double base, const pq_rope_scaling *scaling,
                        float *table, void *stream);

/* pq_rope -- rotary positions of x [tokens, heads, dim]: each pair (x1, x2)
 * of the first `rot` channels becomes
 *   y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin
 * in fp32 (one rounding an operation), rounded once to the type; the other
 * channels are copied.  `inverse` != 0 takes -sin: the transposed rotation,
 * which is the gradient of the forward call.
 *   dtype      PQ_F32, PQ_BF16 or PQ_F16, of x and y
 *   tokens     at most 2^26 - 4;  heads at most 2^30
 *   dim        1 .. 1024;  rot even, 0 .. dim
 *   strides    elements between tokens and between heads, any value
 *   positions  in [tokens] int32.  A negative one (padding) leaves the row as
 *              it is; one past the table gives NaN in the rotated channels
 *   table      in [max_pos, rot / 2, 2] of pq_rope_table (or any cos, sin)
 *   y          out; y == x with equal strides works in place, any other
 *              overlap is not allowed
 * Only the element alignment of x and y is required (else PQ_ERR_ALIGN). */
pq_status pq_rope(int dtype, int64_t tokens, int64_t heads, int64_t dim, int64_t rot, int layout, int inverse,
                  const void *x, int64_t x_token_stride, int64_t x_head_stride, const int32_t *positions,
                  const float *table, int64_t max_pos, void *y, int64_t y_token_stride, int64_t y_head_stride,
                  void *stream);

/* Formats of a key-value cache.  PQ_KV_16: the values themselves (bf16 or
 * f16).  PQ_KV_8, PQ_KV_4: a row (the `dim` channels of one token and head, K
 * and V apart) is held as unsigned codes n in 0 .. Q (Q = 255, 15) and one
 * pair of bf16, a scale s and a zero z:  x^ = z + s n  with
 *   z = bf16(min x),  s = max(bf16((max x - min x) fl32(1 / Q)), 2^-60),
 *   n = clamp(rint((x - z) r), 0, Q),  r = fl32(1 / s),
 * fp32 throughout, one rounding an operation, rint to even.  A row that holds
 * a NaN is stored with a NaN zero and reads back as NaN; so does a row whose
 * range is not finite.  Rows of zero bytes, which nothing was written to, are
 * rows of zeros; pairs from elsewhere may hold any s and z. */
#define PQ_KV_16 0
#define PQ_KV_8 1
#define PQ_KV_4 2

/* A paged cache: page p, head h, token t of the page at
 *   k + p * page_stride + h * head_stride + t * token_stride  (bytes)
 * so that head-major and token-major pages, and K and V in one array, are
 * all described by strides.  A row is pq_kv_row_bytes(format, dim) contiguous
 * bytes; 4-bit rows hold channel 2i in the low half of byte i. */
typedef struct pq_kv_cache {
    void *k, *v;              /* 16-byte aligned                            */
    void *k_param, *v_param;  /* PQ_KV_8, PQ_KV_4: bf16 pairs (s, z),
                                 [num_pages, heads, page_size, 2]; 16 bit: NULL */
    int64_t num_pages;
    int64_t page_stride, head_stride, token_stride;   /* bytes, >= 0, multiples of 8 */
    int32_t format;           /* PQ_KV_16, PQ_KV_8, PQ_KV_4                 */
    int32_t dtype;            /* PQ_KV_16: PQ_BF16 or PQ_F16                */
    int32_t page_size;        /* tokens: a power of two, 16 .. 32768        */
    int32_t heads;            /* 1 .. 65535                                 */
    int32_t dim;              /* a multiple of 16, 16 .. 256                */
    int32_t reserved;         /* 0                                          */
} pq_kv_cache;

/* Bytes of a row (2, 1 or 1/2 per channel), -1 for a bad format or dim. */
int64_t pq_kv_row_bytes(int format, int64_t dim);

/*
 * pq_kv_append -- write new tokens' keys and values into the cache, rotating
 * the keys (and the queries) on the way.
 *   cache      host pointer read during the call
 *   dtype      of k, v, q and q_out: PQ_F32, PQ_BF16 or PQ_F16
 *   tokens     at most 2^26 - 4;  q_heads at most 65535
 *   k, v       in [tokens, heads, dim], strides in elements
 *   slots      in [tokens] int64: page * page_size + offset.  A slot below 0
 *              or past the cache is skipped: padding has to use one, since
 *              the tokens of a call are written side by side.  Where two have
 *              the same slot, its rows may mix them (the codes of one with the
 *              scale of the other)
 *   table      (with positions, max_pos, rot, layout, as pq_rope) rotates k
 *              in fp32 before it is stored, so that it is rounded once; NULL
 *              stores k as it is
 *   q, q_out   [tokens, q_heads, dim]: rotated into q_out in the same launch
 *              (q_out == q in place); NULL with q_heads 0 for none; a q
 *              without a table -> PQ_ERR_ARG
 * k, v, q and q_out 16-byte aligned, their strides multiples of 8 elements.
 */
pq_status pq_kv_append(const pq_kv_cache *cache, int dtype, int64_t tokens, const void *k, int64_t k_token_stride,
                       int64_t k_head_stride, const void *v, int64_t v_token_stride, int64_t v_head_stride,
                       const int64_t *slots, const int32_t *positions, const float *table, int64_t max_pos,
                       int64_t rot, int layout, const void *q, int64_t q_heads, int64_t q_token_stride,
                       int64_t q_head_stride, void *q_out, int64_t qo_token_stride, int64_t qo_head_stride,
                       void *stream);

/*
 * pq_kv_load -- read tokens back into dense arrays.  Output row i, with
 * cu[b] <= i < cu[b + 1], is token starts[b] + i - cu[b] of sequence b, whose
 * page j is block_table[b * table_stride + j].
 *   dtype        of k_out and v_out (x^ in fp32, rounded once)
 *   starts       in [batch] int32, or NULL for 0
 *   cu           in [batch + 1] int32, not decreasing, cu[0] = 0
 *   tokens       rows of k_out and v_out (cu[batch], known to the caller), at
 *                most 2^28 - 16
 *   max_pages    columns of block_table.  A token past them, a page id outside
 *                the cache and rows past cu[batch] read as 0
 *   k_out, v_out out [tokens, heads, dim], 16-byte aligned, strides (in
 *                elements) multiples of 8
 */
pq_status pq_kv_load(const pq_kv_cache *cache, int dtype, int64_t batch, int64_t tokens, const int32_t *block_table,
                     int64_t table_stride, int64_t max_pages, const int32_t *starts, const int32_t *cu, void *k_out,
                     int64_t ko_token_stride, int64_t ko_head_stride, void *v_out, int64_t vo_token_stride,
                     int64_t vo_head_stride, void *stream);

/*
 * pq_attn_decode -- attention of one new token per sequence over the cache:
 *   x_t = scale * q . k^_t,   t in [max(0, len - window), len)
 *   out = sum_t softmax(x)_t v^_t,   lse = ln sum_t exp x_t
 * with sums, maximum and weights in fp32; query head h reads cache head
 * h / (q_heads / heads).  The matrix unit takes the weights in 16-bit pieces:
 * all 24 bits over a bf16 cache, the upper 22 over the others.  A score of
 * -inf has weight 0.  An infinite value of an attended token makes its channel
 * of out infinite; two of opposite signs give NaN, and so may one in an f16
 * cache whose weight is below 2^-30 of the largest.
 *   q, out       [batch, q_heads, dim] of q_dtype (PQ_BF16 or PQ_F16; the
 *                cache's dtype if that is PQ_KV_16), 16-byte aligned, strides
 *                (elements) multiples of 8
 *   q_heads      a positive multiple of cache->heads, at most 65535
 *   block_table  in [batch, max_pages] int32 with rows table_stride apart.
 *                Only the entries of attended tokens are used; a page id
 *                outside the cache hides its tokens
 *   lens         in [batch] int32: tokens in the cache, the new one among
 *                them, clamped to [0, max_pages * page_size] (at most 2^30).  Nothing to
 *                attend to gives out = 0 and lse = -inf; what lies in the
 *                cache past len or before the window is never used, NaN and
 *                infinities included
 *   window       attended tokens, 0 for all of them
 *   max_len      an upper bound of lens that sizes the launch; longer ones
 *                count as max_len (0: max_pages * page_size)
 *   lse          out [batch, q_heads] fp32, or NULL
 *   workspace    device memory of pq_attn_decode_workspace_bytes(cache,
 *                batch, q_heads) bytes, 16-byte aligned; its contents on
 *                entry do not matter.  Calls that overlap, on different
 *                streams, need different workspaces
 * For fixed arguments the result is the same in every run (max_len and the
 * other sequences of a batch decide where a sequence is split, and with it
 * the order of its sums).
 */
int64_t pq_attn_decode_workspace_bytes(const pq_kv_cache *cache, int64_t batch, int64_t q_heads);
pq_status pq_attn_decode(const pq_kv_cache *cache, int q_dtype, int64_t batch, int64_t q_heads, const void *q,
                         int64_t q_batch_stride, int64_t q_head_stride, const int32_t *block_table,
                         int64_t table_stride, int64_t max_pages, const int32_t *lens, double scale, int64_t window,
                         int64_t max_len, void *out, int64_t out_batch_stride, int64_t out_head_stride, float *lse,
                         void *workspace, int64_t workspace_bytes, void *stream);

/*
 * Around the packed product: normalisation, rows in 8 bits, the product of
 * 8-bit activations with its epilogue, and distillation.  The conventions of
 * the serving operators above hold (strides in elements, the last dimension
 * contiguous, sizes of zero enqueue nothing); matrices need the alignment of
 * their elements only, unless said otherwise, and scales, statistics and
 * losses are fp32.  An output may be the same array as an input where that is
 * said (same address, same stride); any other overlap is not allowed, and an
 * output of more than one row whose stride is less than a row (in size: it may
 * be negative) is PQ_ERR_SHAPE.  Inputs may have any stride, 0 too, unless said
 * otherwise.  For fixed arguments every result is the same in every run.
 *
 * Rows in 8 bits: row m of a matrix y is held as int8 codes q in -127 .. 127
 * and one fp32 scale, standing for y^ = scale[m] q:
 *   scale = max(max_j |y_j| fl32(1/127), 2^-60),   q_j = rint(y_j / scale)
 * in fp32 (the quotient as a product with the reciprocal), rint to even.  A
 * row y that holds a NaN or an infinity has a NaN scale, and so no values.
 */

/* pq_rmsnorm -- root-mean-square norm, with the residual's addition and an
 * output in 8 bits on request:
 *   h = x + residual (rounded to the type; x itself without a residual)
 *   y = (h rstd) weight,   rstd = (mean_j h_j^2 + eps)^(-1/2)
 * in fp32 (a row whose squares add up to 2^128 and more has rstd 0); this y is
 * rounded to the type, or given in 8 bits as above.
 *   dtype      of x, residual, sum and y: PQ_F32, PQ_BF16 or PQ_F16
 *   rows       at most 2^31 - 1;  cols 1 .. 32768
 *   residual   in [rows, cols], or NULL;  sum out h, required with it (NULL
 *              without); sum may be x or residual
 *   weight     in [cols] of w_dtype (as dtype)
 *   eps        > 0
 *   y          out [rows, cols], or NULL; may be x (then not also sum's)
 *   q, scale   out [rows, cols] int8 and [rows]: the row in 8 bits, instead of
 *              y (exactly one of y and q; else PQ_ERR_ARG)
 *   rstd       out [rows], or NULL: what pq_rmsnorm_bwd takes */
pq_status pq_rmsnorm(int dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride, const void *residual,
                     int64_t r_stride, void *sum, int64_t s_stride, const void *weight, int w_dtype, double eps,
                     void *y, int64_t y_stride, int8_t *q, int64_t q_stride, float *scale, float *rstd, void *stream);

/* pq_rmsnorm_bwd -- its gradient, from h (x, or sum where there was a residual):
 *   n = h rstd,   g = dy weight
 *   dx = rstd (g - n mean_j(g_j n_j)) + dsum      (x's and the residual's alike)
 *   dweight_j = sum over the rows of dy_j n_j
 *   dtype      of h, dy, dsum and dx
 *   dsum       in: the gradient that reaches h from elsewhere, or NULL
 *   dx         out; may be dy or dsum
 *   dweight    out [cols] fp32, or NULL
 *   workspace  device memory of pq_rmsnorm_bwd_workspace_bytes(rows, cols)
 *              bytes, 16-byte aligned, for dweight (NULL without it); its
 *              contents on entry do not matter.  Calls that overlap need
 *              different ones */
int64_t pq_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t cols);
pq_status pq_rmsnorm_bwd(int dtype, int64_t rows, int64_t cols, const void *h, int64_t h_stride, const void *weight,
                         int w_dtype, const float *rstd, const void *dy, int64_t dy_stride, const void *dsum,
                         int64_t ds_stride, void *dx, int64_t dx_stride, float *dweight, void *workspace,
                         int64_t workspace_bytes, void *stream);

/* pq_quantize_rows -- x [rows, cols] (cols 1 .. 65536) in 8 bits as above. */
pq_status pq_quantize_rows(int dtype, int64_t rows, int64_t cols, const void *x, int64_t x_stride, int8_t *q,
                           int64_t q_stride, float *scale, void *stream);

/* Activations of the product's epilogue: none, max(v, 0), v / (1 + e^-v),
 * v (1 + erf(v / sqrt 2)) / 2, and the latter's tanh form
 * v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2.  In fp32, where they are
 * small too: an activation that makes v smaller by e^-u has a relative error of
 * at most 2^-24 (12 + 9 u). */
#define PQ_ACT_NONE 0
#define PQ_ACT_RELU 1
#define PQ_ACT_SILU 2
#define PQ_ACT_GELU 3
#define PQ_ACT_GELU_TANH 4

/* What the epilogue does with `other`: adds it (a residual) or multiplies by
 * it (the other half of a gated layer). */
#define PQ_COMBINE_ADD 0
#define PQ_COMBINE_MUL 1

typedef struct pq_epilogue {
    const void *bias;     /* [N] of bias_dtype, or NULL                     */
    const void *other;    /* [M, N] of y's dtype, or NULL                   */
    int64_t other_stride; /* elements between its rows                      */
    int32_t bias_dtype;   /* PQ_F32, PQ_BF16, PQ_F16                        */
    int32_t activation;   /* PQ_ACT_..                                      */
    int32_t combine;      /* PQ_COMBINE_.. (0 is right without `other`)     */
    int32_t reserved;     /* 0                                              */
} pq_epilogue;

/*
 * pq_gemm_a8 -- the packed product on activations in 8 bits:
 *   v[m, n] = x_scale[m] alpha[n] sum_k X[m, k] level(code[n, k]) + bias[n]
 *   Y[m, n] = act(v) (+ or *) other[m, n]
 * with pq_gemm's weights and levels.  The levels of every width are whole
 * numbers times a power of two (ternary: times fl32(2/3)), so the sum over k
 * is an integer sum on the matrix unit and exact; what follows is fp32,
 * rounded once to y's type.
 *   mode       a deployable width
 *   M, N       0 .. 2^24, up to 2^24 - 1 tiles of 128 x 256 (else
 *              PQ_ERR_SHAPE);  K a positive multiple of 64, at most 2^17 - 64
 *              (the sums then fit 32 bits)
 *   X          in [M, K] int8 codes, 16-byte aligned, x_stride a multiple of 16,
 *              K .. 2^23
 *   x_scale    in [M]
 *   packed     in pq_packed_bytes(mode, N, K) bytes in the export byte order
 *   alpha      in [N] of alpha_dtype: PQ_BF16 (the exported scale) or PQ_F32
 *   epilogue   host pointer read during the call, or NULL for none
 *   Y          out [M, N] of y_dtype: PQ_F32, PQ_BF16 or PQ_F16; may be
 *              epilogue->other (with the same stride)
 *   workspace  device memory of pq_gemm_a8_workspace_bytes(mode, M, N, K)
 *              bytes, 16-byte aligned (NULL where that is 0); its contents on
 *              entry do not matter.  Calls that overlap need different ones
 * Caches: with M <= 32 the codes may be read with the streaming hint, as in
 * pq_gemm's weight streaming; larger M reads them with ordinary loads.
 */
int64_t pq_gemm_a8_workspace_bytes(int mode, int64_t M, int64_t N, int64_t K);
pq_status pq_gemm_a8(int mode, int64_t M, int64_t N, int64_t K, const int8_t *X, int64_t x_stride,
                     const float *x_scale, const uint8_t *packed, const void *alpha, int alpha_dtype,
                     const pq_epilogue *epilogue, int y_dtype, void *Y, int64_t y_stride, void *workspace,
                     int64_t workspace_bytes, void *stream);

/*
 * pq_distill -- distillation from a teacher's top logits.  Row r's teacher
 * gives logits top[r, j] at words index[r, j], j < k; with temperature T
 *   p_j = softmax_j(top[r, j] / T) over the entries with an index in
 *         [0, vocab) (others do not count)
 *   q = softmax_i(logits[r, i] / T) over all words
 *   loss[r] = row_weight[r] T^2 sum_j p_j (ln p_j - ln q_index[j])
 *   dlogits[r, i] = grad_scale row_weight[r] T (q_i - P_i)
 *   P_i = the sum of the p_j with index[r, j] = i, 0 for other words
 * i.e. the gradient of grad_scale * sum_r loss[r], computed while the row is
 * at hand.  Where every word is named once the loss is the divergence of q from
 * p.  A word that is named again counts entry by entry in the loss, which is
 * then lower than the divergence from P by T^2 (sum_i P_i ln P_i -
 * sum_j p_j ln p_j), a number that does not depend on the logits (and may
 * make the loss negative); the gradient is that of both.  A row of weight 0, or without an entry that counts and is above
 * -inf, has loss 0 and gradient 0, whatever its logits hold (and stats (0, 1));
 * an entry of p_j = 0 adds nothing to the loss.
 * A logit of -inf has q_i = 0; NaN, +inf and rows of nothing but -inf give NaN.
 *   dtype       of logits and dlogits
 *   rows        at most 2^31 - 1;  vocab 1 .. 2^30;  k 1 .. 1024
 *   index       in [rows, k] int32, top in [rows, k] of top_dtype
 *   temperature > 0
 *   row_weight  in [rows], or NULL for 1
 *   loss        out [rows], or NULL
 *   stats       out [rows, 2]: (max_i logits_i, sum_i exp((logits_i - max) / T)),
 *               what pq_distill_bwd takes, or NULL
 *   dlogits     out [rows, vocab], or NULL; may be logits
 * At least one of loss, stats and dlogits is wanted.  Sums are fp32, the loss
 * of a row is put together in binary64 and rounded once.
 */
pq_status pq_distill(int dtype, int64_t rows, int64_t vocab, const void *logits, int64_t l_stride, int64_t k,
                     const int32_t *index, const void *top, int top_dtype, double temperature,
                     const float *row_weight, float *loss, float *stats, double grad_scale, void *dlogits,
                     int64_t d_stride, void *stream);

/* pq_distill_bwd -- the gradient by itself, for losses that are weighed later:
 * dlogits[r, i] = dloss[r] row_weight[r] T (q_i - P_i), from the stats of
 * pq_distill on the same logits.  dlogits may be logits. */
pq_status pq_distill_bwd(int dtype, int64_t rows, int64_t vocab, const void *logits, int64_t l_stride, int64_t k,
                         const int32_t *index, const void *top, int top_dtype, double temperature,
                         const float *row_weight, const float *stats, const float *dloss, void *dlogits,
                         int64_t d_stride, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PQ_H_ */
