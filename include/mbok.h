/*
 * mbok.h -- C ABI of the Multi-Boolean-kernel (MBOK) linear layer for AMD
 * Instinct MI355X (gfx950).
 *
 * The operation is the linear-layer product of a weight matrix stored as K
 * Boolean kernels with group scales:
 *
 *     W_hat = sum_{k=1..K} alpha_k (.) B_k,   B_k in {-1,+1}^{m x n},
 *     y     = W_hat . x      (decode, one token)
 *     Y     = X . W_hat^T    (several tokens)
 *
 * Sources (page title, then the section on that page):
 *   [RN]  "Highly Efficient and Effective LLMs with Multi-Boolean
 *         Architectures", Paper-Notes reading note (zhaoyang97.github.io),
 *         sections 关键设计 (key design: multi-kernel Boolean parameters,
 *         closed-form scale fit, group-wise scales), 消融实验 (ablation table:
 *         group size 128 is the usual choice), 训练策略 (initialisation by SVD or
 *         greedy search) and 局限与展望 (activations stay full precision).
 *   [GS]  the same paper's gist.science summaries (Italian, Dutch, Spanish),
 *         sections "Architetture Multi-Kernel" / "Successive SVID" /
 *         "Extracción Sucesiva": successive kernels are fitted to the residual
 *         of the previous ones.
 *
 * Conventions shared by every call
 * ---------------------------------
 *  - m = output features (rows of W), n = input features (columns of W).
 *    W is row-major [m, n]; x has n entries; y has m entries; X is row-major
 *    [T, ldx >= n]; Y is row-major [T, ldy >= m].
 *  - Scales: one alpha per (kernel k, output row i, group g) where group g is
 *    the 128 consecutive input columns 128g .. 128g+127 ([RN] group-wise scales,
 *    group size 128).  n must be a multiple of 128.
 *  - Sign encoding: bit 1 <-> +1, bit 0 <-> -1 ([GS] Dutch summary,
 *    Methodologie 1: a Boolean weight is -1/+1, equivalently FALSE/TRUE; here
 *    TRUE is bit 1 and means +1).  sign(0) and sign(-0.0) are +1.
 *  - All data pointers are DEVICE memory owned by the caller.  The library
 *    allocates nothing and every call only enqueues work on `stream` (a
 *    hipStream_t; NULL = the default stream) and returns without
 *    synchronising.  The one piece of global state is the static scratch of
 *    mbok_gemvt_noalloc (a fixed device array, its address cached per device).
 *  - Every argument check runs on the host before anything is enqueued, so an
 *    error return means nothing was launched and no output was touched.
 *    MBOK_ERR_HIP is returned when a launch itself fails (hipGetLastError).
 *  - Results are deterministic: the same inputs give the same output bits
 *    (fixed reduction order; no atomics but mbok_distill's, which set bits in
 *    LDS and so come out the same in any order).
 *
 * Packed layout MBOK_LAYOUT_L64 (what mbok_pack writes and mbok_gemv /
 * mbok_gemm read)
 * -------------------------------------------------------------------------
 *  m_pad = m rounded up to a multiple of 64, G = n / 128.
 *  The buffer has two regions:
 *
 *  1. sign bits, K * m_pad * n / 8 bytes, starting at byte 0.  It is a
 *     sequence of 16-byte chunks; chunk c holds the 128 signs of one
 *     (row i, group g, kernel k) with
 *         c = ((rb * G + g) * K + k) * 64 + r,   rb = i / 64,  r = i % 64.
 *     A chunk is four little-endian uint32 words; word w (0..3) covers
 *     columns 128g + 32w .. 128g + 32w + 31, and
 *         bit (8e + q) of word w  <->  column 128g + 32w + 4q + e
 *     for e in 0..3, q in 0..7.  Equivalently: byte 4w + e of the chunk,
 *     bit q, is column 128g + 32w + 4q + e.  So each 4-bit nibble of a word
 *     holds 4 columns spaced 4 apart (one signed-sum lookup in the decode
 *     kernel), and the 4 bits of 4 consecutive columns 4q..4q+3 sit at the
 *     same position q of the word's 4 bytes (one byte-select in the prefill
 *     unpack).  Rows m .. m_pad-1 are all-zero bits.
 *
 *  2. scales, starting at byte K * m_pad * n / 8 (a multiple of 1024):
 *     K * m_pad * G values of the descriptor's alpha dtype (fp32 or IEEE
 *     fp16), value index ((rb * G + g) * K + k) * 64 + r, i.e. in the same
 *     order as the chunks.  Scales of padding rows are 0.
 *
 *  So one (row block, group) holds K consecutive 1 KB sign planes of 64 rows,
 *  and 64 consecutive scales per plane: a wavefront of 64 lanes, one lane per
 *  row, reads one plane with one 16-byte load per lane (1 KB contiguous).
 */
#ifndef MBOK_H
#define MBOK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MBOK_GROUP 128      /* input columns per scale group */
#define MBOK_ROW_BLOCK 64   /* rows per packed row block */
#define MBOK_MAX_K 4        /* kernels per layer accepted by the library */
#define MBOK_MAX_T 65536    /* tokens per mbok_gemm call */

/* Status codes.  0 is success; errors are negative. */
enum {
  MBOK_OK = 0,
  MBOK_ERR_INVALID_ARG = -1, /* NULL pointer, unknown enum, bad leading dim */
  MBOK_ERR_SHAPE = -2,       /* m < 1, n < 128, n % 128 != 0, T out of range */
  MBOK_ERR_DTYPE = -3,       /* dtype not accepted by this call */
  MBOK_ERR_ALIGN = -4,       /* pointer or leading dimension misaligned */
  MBOK_ERR_HIP = -5,         /* the HIP runtime rejected a launch */
  MBOK_ERR_UNSUPPORTED = -6, /* K or group outside what the library runs */
  MBOK_ERR_INFEASIBLE = -7,  /* no kernel allocation fits the bit budget */
  MBOK_ERR_SCRATCH = -8      /* more scratch needed than the static scratch holds */
};

/* Element types.  MBOK_E4M3 (8-bit float, 4 exponent and 3 mantissa bits,
 * largest value 448) is taken by mbok_adamw's states alone. */
enum { MBOK_F32 = 0, MBOK_F16 = 1, MBOK_BF16 = 2, MBOK_E4M3 = 3 };

/* Packed layouts. */
enum { MBOK_LAYOUT_L64 = 1 };

/* Shape of one MBOK layer.  Fill it with mbok_desc_init. */
typedef struct mbok_desc {
  int32_t m;           /* output features, >= 1 */
  int32_t n;           /* input features, a positive multiple of 128 */
  int32_t K;           /* Boolean kernels, 1 .. MBOK_MAX_K */
  int32_t group;       /* always MBOK_GROUP */
  int32_t alpha_dtype; /* MBOK_F32 or MBOK_F16 */
  int32_t layout;      /* always MBOK_LAYOUT_L64 */
} mbok_desc;

/*
 * Describes one layer of K Boolean kernels with group-wise scales ([RN]
 * 关键设计: a weight matrix is the sum of K Boolean kernels, each with its own
 * scales, one scale per group of input columns; [RN] 消融实验: groups of 128).
 * Fills *d after checking the shape: 1 <= m <= 2^24, 128 <= n <= 2^20 with
 * n % 128 == 0, 1 <= K <= MBOK_MAX_K, alpha_dtype in {MBOK_F32, MBOK_F16}.
 * Host only.  Returns MBOK_OK, MBOK_ERR_INVALID_ARG (d NULL),
 * MBOK_ERR_SHAPE, MBOK_ERR_UNSUPPORTED (K) or MBOK_ERR_DTYPE.
 */
int mbok_desc_init(mbok_desc* d, int32_t m, int32_t n, int32_t K,
                   int32_t alpha_dtype);

/* Bytes of the packed buffer (both regions of MBOK_LAYOUT_L64).  Host only;
 * returns 0 for a NULL or invalid descriptor. */
size_t mbok_packed_bytes(const mbok_desc* d);

/* Bytes of the natural-order scale array alpha[K][m][n/128] that
 * mbok_residual_binarize writes and mbok_pack reads.  Host only; 0 for a NULL
 * or invalid descriptor. */
size_t mbok_alpha_bytes(const mbok_desc* d);

/*
 * Greedy residual binarization: the data-free extraction of the K kernels
 * from a floating-point weight ([RN] 训练策略: initialisation by greedy
 * search; [GS] successive kernels fitted to the residual; [RN] 关键设计: for
 * fixed signs the least-squares scale has a closed form).  Per (row, group),
 * in float64:
 *     R_0 = W
 *     for k = 1..K:
 *         B_k   = sign(R_{k-1})                  (0 and -0.0 map to +1)
 *         a     = mean over the group of |R_{k-1}|   (the LS-optimal scale)
 *         alpha = a rounded to nearest-even in the alpha dtype
 *         R_k   = R_{k-1} - alpha * B_k          (uses the rounded alpha)
 *
 *  W      device, fp32, row-major [m, ldw], ldw >= n (elements).
 *  signs  device, int8 [K][m][n] row-major, written with +1 / -1.
 *  alpha  device, [K][m][n/128] of d->alpha_dtype (natural order).
 *  flag   device int32 or NULL.  If W holds a NaN or an Inf the call stores 1
 *         there (it never stores 0: the caller clears it beforehand) and the
 *         outputs for the affected groups are unspecified.
 * Errors: INVALID_ARG (NULL, ldw < n), SHAPE/DTYPE/UNSUPPORTED from d,
 * ALIGN (W, signs or alpha not 16-byte aligned, ldw % 4 != 0), HIP.
 */
int mbok_residual_binarize(const mbok_desc* d, const float* W, int64_t ldw,
                           int8_t* signs, void* alpha, int32_t* flag,
                           void* stream);

/* Largest `rounds` accepted by mbok_refit. */
#define MBOK_MAX_REFIT_ROUNDS 64

/*
 * Alternating least-squares refit of K Boolean kernels and their scales for
 * the weight W they approximate ([RN] 关键设计, efficient scale optimisation:
 * with the Boolean matrices fixed the scales have a closed-form least-squares
 * solution, and signs and scales are optimised in turn).  Usually run on the
 * output of mbok_residual_binarize, before mbok_pack.  Per (row i, group g),
 * with w the 128 weights of the group and b_k its signs:
 *     repeat `rounds` times: scale step, sign step; then one scale step
 *     scale step: alpha = exact solution of (B^T B) alpha = B^T w, rounded
 *                 once to nearest-even in the alpha dtype; when the integer
 *                 K x K matrix B^T B is singular the scales are kept
 *     sign step:  each weight takes the signs of its nearest level
 *                 sum_k alpha_k b_k (float64 levels summed in k order and
 *                 float64 distances; a tie goes to the larger level, then to
 *                 the larger pattern index sum_k [b_k = +1] 2^k)
 * rounds = 0 only re-solves the scales.  With K = 1 nothing changes (the
 * least-squares scale of sign(w) is mean |w|).  Scales may come out
 * negative.
 *  W       device, fp32, row-major [m, ldw], ldw >= n (elements); read only.
 *  signs   device, int8 [K][m][n], read and overwritten in place with +1 /
 *          -1; an entry >= 0 is read as +1.
 *  alpha   device, [K][m][n/128] of d->alpha_dtype (natural order), read
 *          and overwritten in place.
 *  rounds  0 .. MBOK_MAX_REFIT_ROUNDS.
 * The scale step is exact (one rounding of the rational solution) whenever,
 * within each group, the nonzero weights' magnitudes lie within a factor 2^48
 * of one another; otherwise the solution is accurate to about 2^-100 before
 * its rounding.  NaN or Inf weights give unspecified outputs for their
 * groups (mbok_residual_binarize reports them).
 * Errors: INVALID_ARG (NULL, ldw < n, rounds out of range),
 * SHAPE/DTYPE/UNSUPPORTED from d, ALIGN (W, signs or alpha not 16-byte
 * aligned, ldw % 4 != 0), HIP.
 */
int mbok_refit(const mbok_desc* d, const float* W, int64_t ldw, int8_t* signs,
               void* alpha, int32_t rounds, void* stream);

/*
 * Residual energy of the greedy decomposition (the chain of
 * mbok_residual_binarize with d->K kernels) after k = 0..K kernels: the
 * residual approximation error that the kernel allocation weighs ([GS]
 * Italian summary, section "D. Allocazione Automatica dei Kernel").
 *     row_energy[k * m + i] = float64 nearest to sum_j R_k[i, j]^2
 *     layer_energy[k]       = float64 nearest to sum_i row_energy[k * m + i]
 * with R_0 = W and R_k the float64 residual after k kernels (the scales
 * rounded to d->alpha_dtype exactly as mbok_residual_binarize rounds them).
 * Because the greedy chain does not depend on how many kernels follow,
 * layer_energy[K'] is the error of the K'-kernel decomposition for every
 * K' <= K.  The sums are exact pair sums before their one rounding when a
 * row's squared residuals (and the layer's row energies) lie within a factor
 * of about 2^90 (2^48) of one another.
 *  W             device, fp32, row-major [m, ldw], ldw >= n; read only.
 *  row_energy    device, float64 [K + 1][m]; overwritten.
 *  layer_energy  device, float64 [K + 1]; overwritten.
 * Errors: INVALID_ARG (NULL, ldw < n), SHAPE/DTYPE/UNSUPPORTED from d, ALIGN
 * (W 16 bytes, ldw % 4, energies 8 bytes), HIP.
 */
int mbok_residual_energy(const mbok_desc* d, const float* W, int64_t ldw,
                         double* row_energy, double* layer_energy, void* stream);

/*
 * Number of kernels for each of L weights under a bit budget ([GS] Italian
 * summary, section "D. Allocazione Automatica dei Kernel": kernels per
 * weight chosen for an average bit budget from residual error and weight
 * size; the importance term needs data and is left out, so every weight
 * counts the same).  Host only, no GPU work.  Chooses K_l in 1..kmax with
 *     sum_l K_l * sizes[l] <= budget
 * minimising the exact sum of errors[l * kmax + K_l - 1]; among equal
 * errors the fewest bits, then the first K vector in lexicographic order.
 * The answer is exact (dynamic programming over exact error sums).
 *  L       number of weights, >= 1.
 *  sizes   host int64 [L], entries per weight (bits per kernel), each >= 1.
 *  errors  host float64 [L][kmax], errors[l * kmax + K - 1] = residual energy
 *          of weight l with K kernels (e.g. layer_energy[K] of
 *          mbok_residual_energy); finite and >= 0.
 *  kmax    1 .. MBOK_MAX_K.
 *  budget  total kernel-bits, e.g. floor(average kernels * sum of sizes).
 *  K_out   host int32 [L], written on success only.
 * Errors: INVALID_ARG (NULL, L < 1, kmax, sizes < 1, errors negative or not
 * finite, budget < 0), INFEASIBLE (sum of sizes > budget), UNSUPPORTED (more
 * than 2^22 partial allocations would be compared).
 */
int mbok_allocate_kernels(int32_t L, const int64_t* sizes, const double* errors,
                          int32_t kmax, int64_t budget, int32_t* K_out);

/* Largest number of power-iteration rounds accepted by mbok_svid_decompose. */
#define MBOK_MAX_SVID_ITERS 1000

/* Bytes of the workspace mbok_svid_decompose needs (float64 iterates and
 * partial sums).  Host only; 0 for a NULL or invalid descriptor. */
size_t mbok_svid_workspace_bytes(const mbok_desc* d);

/*
 * Successive sign-value-independent decomposition (SVID), the scale variant
 * of the [GS] summaries ("Riformulazione Booleana e SVID", "Successive
 * SVID", "Descomposición SVID"): W ~ sum_k B_k (.) (s_out^k s_in^k^T), where
 * for k = 1..K, with R_0 = W:
 *     B_k          = sign(R_{k-1})            (0 and -0.0 give +1)
 *     sigma, u, v  = the top singular triple of |R_{k-1}|, by `iters` rounds
 *                    of float64 power iteration from v = 1/sqrt(n)
 *     s_out^k      = sqrt(sigma) u, s_in^k = sqrt(sigma) v, each rounded once
 *                    to nearest-even in d->alpha_dtype
 *     R_k          = R_{k-1} - B_k (.) (s_out^k s_in^k^T)  (float64, with the
 *                    rounded vectors)
 * The residual is recomputed from W on every pass (never stored).  Power
 * iteration reaches the SVD's vectors when the ratio of the two largest
 * singular values of |R| is well below 1 (about 0.03 for trained-like
 * weights, so 16-32 rounds give float64 accuracy).  Sums run in a fixed
 * order: results are bit-reproducible.
 *  W          device, fp32, row-major [m, ldw], ldw >= n; read only.
 *  signs      device, int8 [K][m][n]; written with +1 / -1.
 *  s_out      device, [K][m] of d->alpha_dtype; written.
 *  s_in       device, [K][n] of d->alpha_dtype; written.
 *  iters      1 .. MBOK_MAX_SVID_ITERS.
 *  workspace  device, mbok_svid_workspace_bytes(d) bytes, 256-byte aligned;
 *             needs no initialisation; calls that may overlap need distinct
 *             workspaces.
 * Errors: INVALID_ARG (NULL, ldw < n, iters), SHAPE/DTYPE/UNSUPPORTED from
 * d, ALIGN (W and signs 16 bytes, ldw % 4, vectors 4 bytes, workspace 256
 * bytes), HIP.
 */
int mbok_svid_decompose(const mbok_desc* d, const float* W, int64_t ldw,
                        int8_t* signs, void* s_out, void* s_in, int32_t iters,
                        void* workspace, void* stream);

/*
 * Packs SVID kernels into MBOK_LAYOUT_L64: the sign bits as mbok_pack writes
 * them, and s_out^k[i] in the scale slot of every group of row i, kernel k.
 * (s_in is passed to mbok_svid_gemv separately.)
 *  signs   device int8 [K][m][n];  s_out  device [K][m] of d->alpha_dtype;
 *  packed  device, mbok_packed_bytes(d) bytes, fully overwritten.
 * Errors: INVALID_ARG, SHAPE/DTYPE/UNSUPPORTED, ALIGN (signs and packed 16
 * bytes, s_out 4 bytes), HIP.
 */
int mbok_svid_pack(const mbok_desc* d, const int8_t* signs, const void* s_out,
                   void* packed, void* stream);

/* Bytes of the workspace mbok_svid_gemv uses: 0 (the argument is kept for a
 * form that stages activations).  Host only. */
size_t mbok_svid_gemv_workspace_bytes(const mbok_desc* d);

/*
 * Decode product of the SVID representation ([GS] summaries: the product is
 * the Boolean one with x scaled per kernel and the output scaled per row):
 *     y[i] = sum_k s_out^k[i] * sum_j b_k[i, j] * s_in^k[j] * x[j]
 * s_in^k (.) x is formed in fp32 (exact for fp16 scales and bf16 x) and
 * split into four fp8 parts with one power-of-two scale per 32 columns, 4
 * bits each, so the matrix cores see 16 significant bits of each 32-column
 * word's largest value (MBOK_SVID_VARIANT=skinny: bf16 hi + lo parts, about
 * 2^-17 relative per value); the +-1 contractions accumulate in fp32 and
 * s_out applies in fp32.  Within 1e-5 of sum_k |s_out^k[i]| sum_j |s_in^k[j]
 * x[j]| on the workloads; a non-finite product s_in^k[j] x[j] makes every
 * output NaN.  Results are bit-reproducible.
 *  packed     device, the buffer of mbok_svid_pack.
 *  s_in       device [K][n] of d->alpha_dtype, 16-byte aligned.
 *  x          device, n values of x_dtype (MBOK_BF16 or MBOK_F32), 16-byte
 *             aligned.
 *  y          device fp32 [m]; overwritten.
 *  workspace  device pointer or NULL; unused (checked for 256-byte alignment
 *             when given).
 * Errors: INVALID_ARG (NULL), SHAPE/UNSUPPORTED from d, DTYPE (x_dtype),
 * ALIGN (packed, s_in, x 16 bytes, y 4 bytes, workspace 256 bytes), HIP.
 */
int mbok_svid_gemv(const mbok_desc* d, const void* packed, const void* s_in,
                   const void* x, int32_t x_dtype, float* y, void* workspace,
                   void* stream);

/*
 * Packs Boolean kernels and their scales into MBOK_LAYOUT_L64 (see the top
 * of this header): the storage form of the multi-kernel Boolean parameters
 * ([RN] 关键设计: K sign matrices and their group scales; [GS] Dutch
 * summary, Methodologie 1: a Boolean weight is -1/+1, i.e. FALSE/TRUE, so one
 * bit holds it).
 * Any +-1 signs are accepted, e.g. those of a finetuned model ([GS] Dutch
 * summary, Methodologie 3: the kernels are finetuned in the Boolean domain);
 * an entry >= 0 packs as bit 1 (+1) and < 0 as bit 0 (-1).
 *  signs   device int8 [K][m][n].
 *  alpha   device [K][m][n/128] of d->alpha_dtype.
 *  packed  device, mbok_packed_bytes(d) bytes; fully overwritten, padding
 *          included.
 * Errors: INVALID_ARG, SHAPE/DTYPE/UNSUPPORTED, ALIGN (16 bytes), HIP.
 */
int mbok_pack(const mbok_desc* d, const int8_t* signs, const void* alpha,
              void* packed, void* stream);

/*
 * Bytes of the workspace mbok_gemv uses for this shape: 0 when the call needs
 * none, which is the case for every shape with the default kernel (the
 * column-split kernel, selected for comparison with the environment variable
 * MBOK_GEMV_VARIANT=split, is the one that uses it).  Host only; 0 for a NULL
 * or invalid descriptor.
 */
size_t mbok_gemv_workspace_bytes(const mbok_desc* d);

/*
 * Decode product for one token ([RN] 关键设计: Wx splits into K Boolean
 * matrix-vector products, so each weight multiply becomes an add or a
 * subtract of an activation; [RN] 局限与展望: activations stay full
 * precision):
 *     y[i] = sum_k sum_g alpha_k[i,g] * sum_{j in group g} b_k[i,j] * x[j]
 * with fp32 accumulation.
 *  packed    device, MBOK_LAYOUT_L64 buffer of this descriptor.
 *  x         device, n values of x_dtype (MBOK_BF16 or MBOK_F32).
 *  y         device fp32 [m]; overwritten (not accumulated).
 *  workspace device, mbok_gemv_workspace_bytes(d) bytes, 256-byte aligned,
 *            or NULL (always allowed; ignored when the size is 0).  When used
 *            it receives the partial sums of column slices, which a second
 *            small kernel on the same stream adds in a fixed order; its
 *            contents need no initialisation and are meaningless after the
 *            call, and calls that may run at the same time (other streams)
 *            need distinct workspaces.
 * The default kernels keep one workgroup per compute unit and stream 16-row
 * tiles.  For bf16 x the products run on the matrix cores when a row holds at
 * least 8192 sign bits (K n >= 8192), the layer at least 2^25 (K m n), or
 * K = 4: signs as fp4 values (one of two per sign, a known offset removed per
 * group), each activation as an exact pair of fp8 parts with one power-of-two
 * scale per 32 columns, alpha applied per (row, group, kernel) in fp32.
 * Otherwise (and for fp32 x) signed-sum tables of x are built once and the
 * sign nibbles index them.
 * Non-finite x: with the table kernels a NaN or infinity propagates through
 * the fp32 sums; with the matrix-core kernel any NaN or infinite activation
 * makes every output NaN.
 * Errors: INVALID_ARG, SHAPE/UNSUPPORTED, DTYPE (x_dtype), ALIGN (packed and
 * x 16-byte aligned, y 4-byte aligned, workspace 256-byte aligned), HIP.
 */
int mbok_gemv(const mbok_desc* d, const void* packed, const void* x,
              int32_t x_dtype, float* y, void* workspace, void* stream);

/*
 * Bytes of the workspace mbok_gemvt uses for this shape (the partial column
 * sums of its row slices), 0 when it needs none.  Host only; 0 for a NULL or
 * invalid descriptor.
 */
size_t mbok_gemvt_workspace_bytes(const mbok_desc* d);

/*
 * Transposed decode product for one gradient vector, the activation gradient
 * of the layer (the [GS] summaries' Boolean-domain training propagates
 * gradients through the Boolean weights; [RN] 关键设计: the product splits
 * into K Boolean products):
 *     dx[j] = sum_i sum_k alpha_k[i, j/128] * b_k[i, j] * g[i]
 * Each term alpha_k[i, .] * g[i] is formed in fp32; the sums are fp32.
 *  packed    device, MBOK_LAYOUT_L64 buffer of this descriptor (the same
 *            buffer mbok_gemv reads).
 *  g         device, m values of g_dtype (MBOK_BF16 or MBOK_F32).
 *  dx        device fp32 [n]; overwritten (not accumulated).
 *  workspace device, mbok_gemvt_workspace_bytes(d) bytes, 256-byte aligned,
 *            or NULL.  With NULL one workgroup per column group walks all
 *            rows (correct, slower); with the workspace the rows are split
 *            into slices whose partial sums a second kernel adds in a fixed
 *            order.  Its contents need no initialisation; calls that may run
 *            at the same time need distinct workspaces.
 * Errors: INVALID_ARG (NULL), SHAPE/UNSUPPORTED from d, DTYPE (g_dtype),
 * ALIGN (packed 16 bytes, g and dx 4 bytes, workspace 256 bytes), HIP.
 */
int mbok_gemvt(const mbok_desc* d, const void* packed, const void* g,
               int32_t g_dtype, float* dx, void* workspace, void* stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): mbok_gemvt
 * with its workspace replaced by the library's static scratch, a file-scope
 * device array of mbok_gemvt_scratch_bytes() = 512 KiB per device, held until
 * the process ends.  Same kernels, same slicing and the same output bits as
 * mbok_gemvt with a workspace.  The call allocates nothing: on its first call
 * on a device it looks up that device's address of the array
 * (hipGetSymbolAddress, with the caller's current device) and caches it.
 *  packed, g, g_dtype, dx, stream: as for mbok_gemvt.
 * Every call on one GPU shares that GPU's scratch: calls that may overlap in
 * time on the same GPU (different streams, different host threads) race and
 * must be serialised by the caller.  The scratch needs no initialisation
 * (every partial sum is written before it is read).
 * Errors: as mbok_gemvt; SCRATCH when the shape needs more than the static
 * scratch (no shape the descriptor accepts does); HIP when the device or the
 * array's address cannot be queried, or a launch fails.
 */
size_t mbok_gemvt_scratch_bytes(void);
int mbok_gemvt_noalloc(const mbok_desc* d, const void* packed, const void* g,
                       int32_t g_dtype, float* dx, void* stream);

/*
 * The same product for T tokens ([RN] 关键设计: the layer's product is the sum
 * of its K Boolean products, scaled per group; [RN] 局限与展望: activations
 * stay full precision):  Y[t, i] = sum_j W_hat[i, j] * X[t, j].
 * T = 1 runs the decode kernel of mbok_gemv (without a workspace).  T = 2,
 * and T = 3..6 on layers of at least 2^26 sign bits (K m n), run matrix-core
 * forms of that kernel for several tokens (signs as fp4 operands, each bf16
 * activation as two exact fp8 parts with one power-of-two scale per 32
 * columns, alpha applied per group in fp32: within ~1e-6 of the bound
 * sum_j |W_hat_ij| |X_tj| on Gaussian activations; bit-exact for small
 * integer activations and power-of-two scales).  The other T <= 16 run the
 * weight-streaming few-token kernel (exact fp32 scaling of +-1 products).  A
 * non-finite activation of token t makes row t of Y NaN on the matrix-core
 * paths (IEEE propagation elsewhere).  T > 16 is the prefill GEMM: each tile of W_hat is formed
 * as sum_k alpha_k * b_k in fp32, rounded to bf16 (nearest-even) in LDS, and
 * contracted with the bf16 X tile on the matrix cores with fp32 accumulation.
 *  X        device bf16 [T, ldx], ldx >= n, ldx % 8 == 0.
 *  Y        device fp32 [T, ldy], ldy >= m; overwritten.
 *  T        1 .. MBOK_MAX_T.
 * Errors: INVALID_ARG (NULL, ldx < n, ldy < m), SHAPE (T), DTYPE (x_dtype
 * other than MBOK_BF16), ALIGN (packed/X 16 bytes, ldx % 8, Y 4 bytes), HIP.
 */
int mbok_gemm(const mbok_desc* d, const void* packed, const void* X,
              int32_t x_dtype, int64_t T, int64_t ldx, float* Y, int64_t ldy,
              void* stream);

/*
 * mbok_gemm with the prefill weights carried to 16 significant bits ([RN]
 * 关键设计: W_hat x is the sum of the K scaled Boolean products, each weight
 * exactly sum_k alpha_k b_k; carrying that value to the matrix cores needs
 * more than bf16's 8 significant bits).  Same arguments, checks, errors and
 * output layout as mbok_gemm; T = 1 runs the same kernel as mbok_gemm, and
 * T = 2..16 always the weight-streaming few-token kernel (its products are
 * fp32-exact per scale).  For T > 16
 * each level v = sum_k +-alpha_k is formed in fp32 and split as
 * v = hi + lo with hi = bf16(v) and lo = bf16(v - hi), so |v - hi - lo| <=
 * 2^-16 |v|.  Two products run on `stream`: Y = X . HI^T, then Y += X . LO^T
 * (two launches, about twice the time and one extra read of Y).  Per output,
 * |Y - Y_exact| stays far below 1e-3 * sum_j |W_hat_ij| |X_tj| for any X
 * (2^-16 from the weights plus fp32 accumulation), where mbok_gemm's
 * one-term bf16 levels allow up to 2^-8 per weight.  The result is exactly
 * the fp64 product when every level has at most 16 significant bits (power-
 * of-two scales within 15 binades of each other) and the activations and sums
 * are small integers.
 */
int mbok_gemm_precise(const mbok_desc* d, const void* packed, const void* X,
                      int32_t x_dtype, int64_t T, int64_t ldx, float* Y,
                      int64_t ldy, void* stream);

/* ------------------------------------------------------------------------
 * Fine-tuning a Boolean-kernel model against a teacher, and the gated
 * feed-forward block ([GS] Dutch summary, Methodologie 3, and the Spanish
 * summary's training section: the kernels are finetuned by distillation from
 * the full-precision model, gradients flowing through the Boolean weights;
 * [RN] 训练策略: the last kernel and the scales are tuned).
 * ------------------------------------------------------------------------ */

/*
 * Transposed product for T gradient rows, the activation gradient of a layer
 * (mbok_gemvt is the one-row form with fp32 terms):
 *     dX[t, j] = sum_i dY[t, i] * W_hat[i, j]
 * Each tile of W_hat is formed as sum_k alpha_k b_k in fp32, rounded to bf16
 * (nearest-even) and contracted with dY on the matrix cores with fp32
 * accumulation; dX is the sum rounded once to bf16 (the gradient of bf16
 * activations, and what the layer below takes as its dY).  Row sums run in a
 * fixed order: results are bit-reproducible for a given workspace choice.
 *  packed    device, MBOK_LAYOUT_L64 buffer of this descriptor.
 *  dY        device bf16 [T, lddy], lddy >= m, 2-byte aligned (16-byte
 *            aligned rows, lddy % 8 == 0, run faster).
 *  T         1 .. MBOK_MAX_T.
 *  dX        device bf16 [T, lddx], lddx >= n, lddx % 8 == 0; overwritten.
 *            Must not overlap dY.
 *  workspace device, mbok_gemmt_workspace_bytes(d, T) bytes, 256-byte
 *            aligned, or NULL.  With it the rows of W_hat are split into
 *            slices when the output alone gives too few tiles, and a second
 *            kernel adds the slices' partial sums in a fixed order; with NULL
 *            every tile walks all rows (correct, slower for few tokens).  Its
 *            contents need no initialisation; calls that may run at the same
 *            time need distinct workspaces.
 * A non-finite dY element makes its whole row of dX NaN or infinite.
 * Errors: INVALID_ARG (NULL, lddy < m, lddx < n), SHAPE (T), ALIGN (packed
 * and dX 16 bytes, lddx % 8, dY 2 bytes, workspace 256 bytes), HIP, and the
 * descriptor's.
 */
int mbok_gemmt(const mbok_desc* d, const void* packed, const void* dY, int64_t T,
               int64_t lddy, void* dX, int64_t lddx, void* workspace, void* stream);

/*
 * mbok_gemmt with each W_hat value carried as two bf16 terms (hi = bf16(v), lo
 * = bf16(v - hi), off by at most 2^-16 |v|), as mbok_gemm_precise is to
 * mbok_gemm: twice the matrix work.  Same arguments, workspace and errors.
 */
int mbok_gemmt_precise(const mbok_desc* d, const void* packed, const void* dY, int64_t T,
                       int64_t lddy, void* dX, int64_t lddx, void* workspace, void* stream);

/* Bytes of the workspace mbok_gemmt uses for this layer and T rows (0 when it
 * needs none).  Host only; 0 for a NULL or invalid descriptor or T. */
size_t mbok_gemmt_workspace_bytes(const mbok_desc* d, int64_t T);

/*
 * Gradient of the scales ([RN] 关键设计: W_hat = sum_k alpha_k (.) B_k, so a
 * scale's derivative is the weight gradient contracted with its signs):
 *     dalpha_k[i, g] = sum_{j in group g} b_k[i, j] * sum_t dY[t, i] X[t, j]
 * The m x n weight gradient is formed tile by tile on the matrix cores (exact
 * bf16 products, fp32 sums), contracted with the signs in fp32 and never
 * stored.
 *  packed     device, the layer's buffer (its signs are read, not its scales).
 *  dY         device bf16 [T, lddy], lddy >= m, 2-byte aligned (16-byte
 *             aligned rows, lddy % 8 == 0, run faster).
 *  X          device bf16 [T, ldx], ldx >= n, ldx % 8 == 0, 16-byte aligned.
 *             Leading dimensions below 2^26.
 *  T          1 .. MBOK_MAX_T.
 *  dalpha     device fp32 [K][m][n/128] (the order of mbok_pack's alpha).
 *  accumulate 0 overwrites dalpha; otherwise the result is added to it
 *             (gradient accumulation over several calls).
 *  workspace  device, mbok_scale_grad_workspace_bytes(d, T) bytes, 256-byte
 *             aligned, or NULL.  With it the tokens are split into slices when
 *             the layer alone gives too few tiles; the partial sums are added
 *             in a fixed order.  As for mbok_gemmt.
 * A non-finite value of dY or X reaches every scale it contributes to.
 * Errors: INVALID_ARG (NULL, lddy < m, ldx < n), SHAPE (T), ALIGN (packed and
 * X 16 bytes, ldx % 8, dY 2 bytes, dalpha 4 bytes, workspace 256 bytes), HIP,
 * and the descriptor's.
 */
int mbok_scale_grad(const mbok_desc* d, const void* packed, const void* dY, int64_t T,
                    int64_t lddy, const void* X, int64_t ldx, float* dalpha,
                    int32_t accumulate, void* workspace, void* stream);

/* Bytes of the workspace mbok_scale_grad uses (0 when it needs none).  Host
 * only; 0 for a NULL or invalid descriptor or T. */
size_t mbok_scale_grad_workspace_bytes(const mbok_desc* d, int64_t T);

/* Activations of the gated block and (with MBOK_ACT_NONE) of mbok_linear. */
enum {
  MBOK_ACT_SILU = 0, /* x / (1 + exp(-x)) */
  MBOK_ACT_GELU = 1, /* x (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))) / 2 */
  MBOK_ACT_NONE = 2  /* x; mbok_linear and its backward only */
};

/*
 * Gated feed-forward block H = act(X Wg^T) (.) (X Wu^T) with both projections
 * as Boolean kernels.  The two projections have one shape `d` (m outputs, n
 * inputs, K kernels each) and are kept as ONE layer in MBOK_LAYOUT_L64, the
 * stacked layer, of 16 ceil(m / 8) rows in which every 16-row tile holds 8
 * gate rows and then the same 8 up rows:
 *     stacked row 16 u + r     = gate row 8 u + r      (r = 0..7)
 *     stacked row 16 u + 8 + r = up   row 8 u + r
 * Rows past m are zero (bits and scales).  So both values of an output meet in
 * one tile and every call here takes one pass over one buffer.  The stacked
 * layer is an ordinary one: mbok_gemm, mbok_gemmt and mbok_scale_grad take it
 * with the descriptor that mbok_gated_stack fills.
 */

/* Fills *stacked with the descriptor of the stacked layer of two projections
 * of shape *d (the pointers may be equal).  Host only.  Errors: the
 * descriptor's, INVALID_ARG (NULL), SHAPE (more than 2^24 stacked rows). */
int mbok_gated_stack(const mbok_desc* d, mbok_desc* stacked);

/*
 * Packs the two projections into the stacked layer.
 *  signs_gate, signs_up  device int8 [K][m][n], as for mbok_pack.
 *  alpha_gate, alpha_up  device [K][m][n/128] of d->alpha_dtype.
 *  packed                device, mbok_packed_bytes of the stacked descriptor;
 *                        fully overwritten, padding included.
 * Errors: INVALID_ARG (NULL), ALIGN (16 bytes), HIP, mbok_gated_stack's.
 */
int mbok_gated_pack(const mbok_desc* d, const int8_t* signs_gate, const void* alpha_gate,
                    const int8_t* signs_up, const void* alpha_up, void* packed,
                    void* stream);

/*
 * H[t, i] = act(g) * u with g = sum_j Wg[i, j] X[t, j], u = sum_j Wu[i, j]
 * X[t, j].  One kernel: both products in fp32 as mbok_gemm computes them for
 * T rows of the stacked layer, activation and product in fp32, one rounding
 * to bf16.
 *  packed  device, the buffer of mbok_gated_pack.
 *  X       device bf16 [T, ldx], ldx >= n, ldx % 8 == 0, 16-byte aligned.
 *  T       1 .. MBOK_MAX_T.
 *  act     MBOK_ACT_SILU or MBOK_ACT_GELU.
 *  H       device bf16 [T, ldh], ldh >= m, 2-byte aligned; overwritten.
 *  pre     device bf16 [T, ldpre] or NULL; ldpre >= 16 ceil(m / 8): g and u,
 *          each rounded once to bf16, in the stacked order (padding columns
 *          are written as 0), for mbok_gated_backward.  16-byte aligned,
 *          ldpre % 8 == 0.
 * Weights: exact per scale (see mbok_gemm) for T <= 16, levels rounded to bf16
 * for larger T.  H and pre must not overlap X or each other.
 * For T <= 16 a non-finite activation of a token makes its H (and pre) NaN on
 * the matrix-core paths; larger T follow IEEE arithmetic.
 * Errors: INVALID_ARG (NULL, act, leading dimensions; ldx >= 2^23 for T > 16),
 * SHAPE (T; a stacked layer of 2^32 or more sign words for T > 16), DTYPE
 * (x_dtype other than MBOK_BF16), ALIGN, HIP, mbok_gated_stack's.
 */
int mbok_gated(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
               int64_t T, int64_t ldx, int32_t act, void* H, int64_t ldh, void* pre,
               int64_t ldpre, void* stream);

/*
 * mbok_gated with each weight carried as two bf16 terms for T > 16 (see
 * mbok_gemmt_precise), so that no token count rounds the weights; for T <= 16
 * the same kernels.  Same arguments and errors.
 */
int mbok_gated_precise(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                       int64_t T, int64_t ldx, int32_t act, void* H, int64_t ldh, void* pre,
                       int64_t ldpre, void* stream);

/*
 * Backward of the gated block.  With g, u from pre and s = dH:
 *     dg = s u act'(g),  du = s act(g)      (fp32, rounded once to bf16)
 *     dX = dg Wg + du Wu                    (mbok_gemmt of the stacked layer)
 *  pre   device bf16 [T, ldpre], as mbok_gated wrote it (padding columns are
 *        not read).
 *  dH    device bf16 [T, lddh], lddh >= m, 2-byte aligned.
 *  dpre  device bf16 [T, lddpre]; overwritten with dg and du in the stacked
 *        order, padding columns 0: the dY of mbok_scale_grad on the stacked
 *        layer.  May be pre itself (same leading dimension).
 *  dX    device bf16 [T, lddx] or NULL (then only dpre is computed).
 *  workspace  device, mbok_gemmt_workspace_bytes(stacked, T) bytes or NULL,
 *        as for mbok_gemmt.
 * Errors: INVALID_ARG (NULL, act, leading dimensions), SHAPE (T; T ceil(m / 8)
 * of 2^32 or more), ALIGN (packed, pre, dpre, dX 16 bytes, ldpre, lddpre, lddx % 8, dH 2 bytes,
 * workspace 256 bytes), HIP, mbok_gated_stack's.
 */
int mbok_gated_backward(const mbok_desc* d, const void* packed, const void* pre,
                        int64_t ldpre, const void* dH, int64_t lddh, int64_t T, int32_t act,
                        void* dpre, int64_t lddpre, void* dX, int64_t lddx, void* workspace,
                        void* stream);

/*
 * mbok_gated_backward with dX by mbok_gemmt_precise (dpre is the same: rounded
 * once to bf16).  Same arguments, workspace and errors.
 */
int mbok_gated_backward_precise(const mbok_desc* d, const void* packed, const void* pre,
                                int64_t ldpre, const void* dH, int64_t lddh, int64_t T,
                                int32_t act, void* dpre, int64_t lddpre, void* dX, int64_t lddx,
                                void* workspace, void* stream);

/*
 * One layer with what follows it in a block:
 *     z[t, i] = sum_j W_hat[i, j] X[t, j] + bias[i]
 *     Y[t, i] = residual[t, i] + act(z[t, i])
 * The product as mbok_gated computes its own for T rows (exact per scale for T
 * <= 16 and, on small layers, for more; levels rounded to bf16 otherwise), then
 * bias, activation and residual in fp32 and one rounding to Y's type.
 *  packed    device, MBOK_LAYOUT_L64 buffer of this descriptor.
 *  X         device bf16 [T, ldx], ldx >= n, ldx % 8 == 0, 16-byte aligned.
 *  T         1 .. MBOK_MAX_T.
 *  bias      device [m] of bias_dtype (MBOK_F32, MBOK_F16 or MBOK_BF16), or NULL.
 *  act       MBOK_ACT_NONE, MBOK_ACT_SILU or MBOK_ACT_GELU.
 *  residual  device [T, ldr] of y_dtype, ldr >= m, or NULL.  May be Y itself
 *            (same leading dimension): the residual stream updated in place.
 *  Y         device [T, ldy] of y_dtype (MBOK_BF16 or MBOK_F32), ldy >= m;
 *            overwritten.
 *  pre       device bf16 [T, ldpre], ldpre >= m, or NULL: z rounded once, for
 *            mbok_linear_backward.
 * residual, Y and pre rows start at any element (16-byte aligned rows run
 * faster).  Y and pre must not overlap X or each other, and the residual no other
 * way than by being Y.  Non-finite activations
 * as for mbok_gated.
 * Errors: INVALID_ARG (NULL, act, leading dimensions, residual = Y with another
 * one; ldx >= 2^23 for T > 16), SHAPE (T; a layer of 2^32 or more sign words for
 * T > 16), DTYPE (x_dtype other
 * than MBOK_BF16, y_dtype, bias_dtype), ALIGN (packed and X 16 bytes, ldx % 8,
 * the others to their element), HIP, and the descriptor's.
 */
int mbok_linear(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                int64_t T, int64_t ldx, const void* bias, int32_t bias_dtype, int32_t act,
                const void* residual, int64_t ldr, void* Y, int32_t y_dtype, int64_t ldy,
                void* pre, int64_t ldpre, void* stream);

/* mbok_linear with each weight carried as two bf16 terms for T > 16 (see
 * mbok_gated_precise).  Same arguments and errors. */
int mbok_linear_precise(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                        int64_t T, int64_t ldx, const void* bias, int32_t bias_dtype,
                        int32_t act, const void* residual, int64_t ldr, void* Y,
                        int32_t y_dtype, int64_t ldy, void* pre, int64_t ldpre, void* stream);

/*
 * Backward of mbok_linear (the residual's gradient is dY itself):
 *     dpre = dY act'(pre)          (fp32, rounded once to bf16)
 *     dbias[i] = sum_t dpre[t, i]  (fp32, of the values before that rounding)
 *     dX = dpre W_hat              (mbok_gemmt)
 *  dY    device bf16 [T, lddy], lddy >= m.
 *  pre   device bf16 [T, ldpre], as mbok_linear wrote it.
 *  dpre  device bf16 [T, lddpre]; overwritten: the dY of mbok_scale_grad.  May be
 *        pre or dY itself (same leading dimension).
 *        With MBOK_ACT_NONE pre and dpre are NULL: dY is dpre.
 *  dbias device fp32 [m] or NULL; accumulate 0 overwrites it, otherwise the sums
 *        are added to it (as for mbok_scale_grad).
 *  dX    device bf16 [T, lddx], lddx >= n, lddx % 8 == 0, 16-byte aligned, or
 *        NULL.  Must not overlap dY or dpre.
 *  workspace  device, mbok_linear_backward_workspace_bytes(d, T) bytes, 256-byte
 *        aligned, or NULL, as for mbok_gemmt: with it the rows are split into
 *        slices for dbias too, whose sums are added in a fixed order.
 * Errors: INVALID_ARG (NULL, act, leading dimensions; nothing asked for: no
 * activation, dbias and dX NULL), SHAPE (T), ALIGN (packed and dX 16 bytes,
 * lddx % 8, dY, pre, dpre 2 bytes, dbias 4, workspace 256 bytes), HIP, and the
 * descriptor's.
 */
int mbok_linear_backward(const mbok_desc* d, const void* packed, const void* pre, int64_t ldpre,
                         const void* dY, int64_t lddy, int64_t T, int32_t act, void* dpre,
                         int64_t lddpre, float* dbias, int32_t accumulate, void* dX,
                         int64_t lddx, void* workspace, void* stream);

/* mbok_linear_backward with dX by mbok_gemmt_precise, of the same dpre, rounded to
 * bf16.  Same arguments, workspace and errors. */
int mbok_linear_backward_precise(const mbok_desc* d, const void* packed, const void* pre,
                                 int64_t ldpre, const void* dY, int64_t lddy, int64_t T,
                                 int32_t act, void* dpre, int64_t lddpre, float* dbias,
                                 int32_t accumulate, void* dX, int64_t lddx, void* workspace,
                                 void* stream);

/* Bytes of the workspace mbok_linear_backward uses for this layer and T rows (0
 * when it needs none).  Host only; 0 for a NULL or invalid descriptor or T. */
size_t mbok_linear_backward_workspace_bytes(const mbok_desc* d, int64_t T);

/* Largest number of listed teacher entries and largest vocabulary of
 * mbok_distill, its most rows, and floats of statistics per row. */
#define MBOK_MAX_TOP 1024
#define MBOK_MAX_VOCAB (1 << 19)
#define MBOK_MAX_DISTILL_ROWS (1 << 23)
#define MBOK_DISTILL_STATS 8

/* Shape of one distillation loss.  Fill it with mbok_distill_desc_init. */
typedef struct mbok_distill_desc {
  int32_t vocab;     /* V, 1 .. MBOK_MAX_VOCAB */
  int32_t top;       /* listed entries per row, 1 .. MBOK_MAX_TOP */
  float temperature; /* tau, finite and at least 2^-126 */
} mbok_distill_desc;

/* Host only.  Errors: INVALID_ARG (NULL, temperature), SHAPE (vocab, top). */
int mbok_distill_desc_init(mbok_distill_desc* d, int32_t vocab, int32_t top,
                           float temperature);

/*
 * Distillation from a teacher's top logits ([GS] summaries' training
 * sections: knowledge distillation on the logits of the full-precision
 * model, of which a corpus keeps the `top` largest per row).  Per row, with
 * q = softmax(z / tau) over the vocabulary and the listed entries (v_j, l_j):
 *   t_lse NULL:  p_j = exp(l_j / tau) / sum of the listed exp(l / tau)
 *                loss = w tau^2 sum_j p_j (log p_j - log q_{v_j})
 *                dz_v = w tau (q_v - sum_{j: v_j = v} p_j)
 *   t_lse given: p_j = exp(l_j / tau - t_lse) (the teacher's own
 *                probabilities); what is not listed is one more class of
 *                mass p_r = max(0, 1 - sum_j p_j), q_r = sum of the other q_v:
 *                loss += w tau^2 p_r log(p_r / q_r)
 *                (no such class when every token is listed or q_r is 0)
 *                dz_v = w tau (s q_v - sum_{j: v_j = v} p_j), for unlisted v
 *                w tau q_v (s - p_r / q_r), with s = sum_j p_j plus the p_r
 *                that was used: 1, more where an index is listed twice or
 *                t_lse is too small for p_r to make up, less without the class
 * An entry whose index is negative or >= V is not there (rows with fewer
 * entries); an index listed twice counts twice.  A row whose listed entries
 * carry no teacher weight (none there, or all l = -inf) has, without t_lse,
 * loss 0 and gradient 0.  A row of weight 0 is not read: loss 0, gradient 0.
 * A p_j of 0 contributes nothing; q_{v_j} = 0 with p_j > 0 gives +inf; NaN
 * or +inf among a row's logits or its listed teacher logits, and rows of only
 * -inf, give NaN (the loss and the row's gradient).
 * Row maxima, sums and logarithms are at least fp32 (the sums of a row and
 * the loss in float64 at the end).  Gradient terms below 2^-90 w tau may be
 * written as 0.
 *  Z        device [T, ldz] of z_dtype (MBOK_F32, MBOK_F16, MBOK_BF16).
 *  T        1 .. MBOK_MAX_DISTILL_ROWS.
 *  t_logits device [T, ldt] of t_dtype (any of the three), l.
 *  t_index  device int32 [T, ldt], v; ldt >= top for both.
 *  t_lse    device fp32 [T] or NULL: log sum exp(teacher logits / tau).
 *  weight   device fp32 [T] or NULL (all 1): w.
 *  loss     device fp32 [T]; overwritten.
 *  stats    device fp32 [T][MBOK_DISTILL_STATS] or NULL; overwritten: what
 *           mbok_distill_backward needs of this pass.  16-byte aligned.
 *  dZ       device [T, lddz] of dz_dtype (z_dtype or MBOK_BF16), or NULL for
 *           the loss alone: the gradient of sum_t loss[t], in the same pass
 *           over Z.  May be Z itself (same dtype and leading dimension).
 * Errors: INVALID_ARG (NULL, leading dimensions), SHAPE (T, the descriptor's),
 * DTYPE, ALIGN (Z, dZ and t_logits to their element, t_index, t_lse, weight and
 * loss 4 bytes, stats 16 bytes), HIP.
 */
int mbok_distill(const mbok_distill_desc* d, const void* Z, int32_t z_dtype, int64_t T,
                 int64_t ldz, const void* t_logits, int32_t t_dtype, const int32_t* t_index,
                 int64_t ldt, const float* t_lse, const float* weight, float* loss,
                 float* stats, void* dZ, int32_t dz_dtype, int64_t lddz, void* stream);

/*
 * The gradient alone, after mbok_distill with stats on the same inputs:
 * dZ[t, v] = dloss[t] * d loss[t] / d Z[t, v].
 *  dloss  device fp32 [T], the gradient arriving at the loss.
 * A row whose weight or dloss is 0 is written as 0.  Everything else as for
 * mbok_distill (dZ may be Z itself).
 */
int mbok_distill_backward(const mbok_distill_desc* d, const void* Z, int32_t z_dtype,
                          int64_t T, int64_t ldz, const void* t_logits, int32_t t_dtype,
                          const int32_t* t_index, int64_t ldt, const float* t_lse,
                          const float* weight, const float* stats, const float* dloss,
                          void* dZ, int32_t dz_dtype, int64_t lddz, void* stream);

/* ------------------------------------------------------------------------
 * Log-probabilities of a batch's tokens and two losses on them: what follows
 * distillation when a model is tuned on answers and their value.
 * ------------------------------------------------------------------------ */

/* Floats of statistics per row of mbok_logp and mbok_policy, and the most pairs
 * of one mbok_preference call. */
#define MBOK_LOGP_STATS 4
#define MBOK_MAX_PAIRS (1 << 23)

/* Rows of logits and the temperature that divides them.  Fill it with
 * mbok_logp_desc_init. */
typedef struct mbok_logp_desc {
  int32_t vocab;     /* V, 1 .. MBOK_MAX_VOCAB */
  float temperature; /* tau, finite and at least 2^-126 */
} mbok_logp_desc;

/* Host only.  Errors: INVALID_ARG (NULL, temperature), SHAPE (vocab). */
int mbok_logp_desc_init(mbok_logp_desc* d, int32_t vocab, float temperature);

/*
 * logp[t] = z_a / tau - log sum_v exp(z_v / tau) of row t's token a = label[t].
 * A row whose label is negative or >= V has no token: it is not read, logp 0.
 * A NaN or +inf among a row's logits, and a row of only -inf, give NaN; z_a =
 * -inf beside finite logits gives -inf.  Row sums are float64 at the end.
 *  Z      device [T, ldz] of z_dtype (MBOK_F32, MBOK_F16, MBOK_BF16).
 *  T      1 .. MBOK_MAX_DISTILL_ROWS.
 *  label  device int32 [T].
 *  logp   device fp32 [T]; overwritten.
 *  stats  device fp32 [T][MBOK_LOGP_STATS] or NULL; overwritten: what
 *         mbok_logp_backward needs of this pass.  16-byte aligned.
 * Errors: INVALID_ARG (NULL, ldz), SHAPE (T, the descriptor's), DTYPE, ALIGN (Z to
 * its element, label and logp 4 bytes, stats 16 bytes), HIP.
 */
int mbok_logp(const mbok_logp_desc* d, const void* Z, int32_t z_dtype, int64_t T, int64_t ldz,
              const int32_t* label, float* logp, float* stats, void* stream);

/*
 * The logits' gradient of sum_t dlogp[t] logp[t]:
 *     dZ[t, v] = dlogp[t] / tau ([v = a] - q_v),  q = softmax(z / tau),
 * after mbok_logp (or mbok_policy) with stats on the same Z, label and descriptor
 * values.  Rows without a token and rows whose dlogp is 0 are written as 0.
 * Terms below 2^-126 dlogp / tau of the largest may be written as 0.
 *  dlogp  device fp32 [T].
 *  dZ     device [T, lddz] of dz_dtype (z_dtype or MBOK_BF16); overwritten.  May
 *         be Z itself (same dtype and leading dimension).
 * Errors: as mbok_logp; INVALID_ARG (lddz), ALIGN (dZ to its element).
 */
int mbok_logp_backward(const mbok_logp_desc* d, const void* Z, int32_t z_dtype, int64_t T,
                       int64_t ldz, const int32_t* label, const float* stats,
                       const float* dlogp, void* dZ, int32_t dz_dtype, int64_t lddz,
                       void* stream);

/* Shape and constants of one clipped policy loss.  Fill it with
 * mbok_policy_desc_init. */
typedef struct mbok_policy_desc {
  int32_t vocab;     /* V, 1 .. MBOK_MAX_VOCAB */
  float temperature; /* tau, finite and at least 2^-126 */
  float clip_low;    /* the ratio is clipped to 1 - clip_low (0 .. 1) ... */
  float clip_high;   /* ... and 1 + clip_high (0 or more; may be infinite) */
  float kl;          /* beta, weight of the KL term, finite, 0 or more */
} mbok_policy_desc;

/* Host only.  Errors: INVALID_ARG (NULL, a constant out of its range or NaN),
 * SHAPE (vocab). */
int mbok_policy_desc_init(mbok_policy_desc* d, int32_t vocab, float temperature,
                          float clip_low, float clip_high, float kl);

/*
 * Clipped policy loss with a KL term, per token, and the logits' gradient in the
 * same pass.  With logp as mbok_logp's and r = exp(logp - old_logp):
 *     loss[t] = w ( -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
 *                   + beta (exp(x) - x - 1) ),   x = ref_logp - logp
 *     dlogp[t] = w ( -(r A, or 0 where the clipped side is the smaller)
 *                    + beta (1 - exp(x)) )
 *     dZ[t, v] = dlogp[t] / tau ([v = a] - q_v)
 * r = 1 + clip_high and r = 1 - clip_low count as not clipped.  An advantage of 0
 * gains nothing at any ratio.  A row without a token has loss, logp and gradient
 * 0; a row of weight 0 has loss and gradient 0 and is read only where logp or
 * stats are asked for.  Non-finite logits as for mbok_logp: a row whose logp is NaN
 * has loss, dlogp and all of dZ NaN.  A token at -inf beside a finite ref_logp has
 * loss +inf, dlogp -inf and a row of dZ that is not finite; at -inf in both, NaN.
 *  Z, z_dtype, T, ldz, label, logp (or NULL), stats (or NULL): as for mbok_logp.
 *  advantage  device fp32 [T], A.
 *  old_logp   device fp32 [T] or NULL: the log-probabilities when the tokens were
 *             sampled; NULL takes the present ones (r = 1, its slope kept; NaN where
 *             logp is NaN).
 *  ref_logp   device fp32 [T] or NULL: a reference model's.  NULL, or beta 0: no KL
 *             term, whatever it holds.
 *  weight     device fp32 [T] or NULL (all 1): w.
 *  loss       device fp32 [T]; overwritten.
 *  dlogp      device fp32 [T] or NULL; overwritten: with stats, what
 *             mbok_logp_backward takes for the gradient alone later.
 *  dZ         device [T, lddz] of dz_dtype, or NULL, as for mbok_logp_backward:
 *             the gradient of sum_t loss[t].
 * Errors: INVALID_ARG (NULL, leading dimensions), SHAPE (T, the descriptor's),
 * DTYPE, ALIGN (Z and dZ to their element, stats 16 bytes, the others 4), HIP.
 */
int mbok_policy(const mbok_policy_desc* d, const void* Z, int32_t z_dtype, int64_t T,
                int64_t ldz, const int32_t* label, const float* advantage,
                const float* old_logp, const float* ref_logp, const float* weight, float* loss,
                float* logp, float* stats, float* dlogp, void* dZ, int32_t dz_dtype,
                int64_t lddz, void* stream);

/* Constants of one preference loss.  Fill it with mbok_preference_desc_init. */
typedef struct mbok_preference_desc {
  float beta;      /* finite, above 0 */
  float smoothing; /* share of pairs taken to be the wrong way round, 0 .. 0.5 */
  float margin;    /* what h has to exceed, finite */
  int32_t mean;    /* 0: sums over a sequence's tokens; else their means */
  int32_t vocab;   /* labels outside 0 .. vocab - 1 are no tokens */
} mbok_preference_desc;

/* Host only.  Errors: INVALID_ARG (NULL, a constant out of its range or NaN),
 * SHAPE (vocab not in 1 .. MBOK_MAX_VOCAB). */
int mbok_preference_desc_init(mbok_preference_desc* d, float beta, float smoothing,
                              float margin, int32_t mean, int32_t vocab);

/*
 * Loss of paired log ratios.  Sequence 2p is pair p's chosen one, 2p + 1 its
 * rejected one; sequence s is rows offsets[s] .. offsets[s + 1] - 1.  With S_s the
 * sum (mean) of logp - ref_logp over the sequence's rows that hold a token:
 *     h = beta (S_2p - S_2p+1) - margin
 *     loss[p] = w ((1 - smoothing) log(1 + exp(-h)) + smoothing log(1 + exp(h)))
 *     dlogp[t] = +-w beta (smoothing sig(h) - (1 - smoothing) sig(-h)) (/ tokens)
 * with + for rows of the chosen sequence and - for the rejected one's; rows
 * without a token get 0.  A sequence without tokens has S = 0.  Sums are float64.
 * dlogp goes to mbok_logp_backward; its rows outside every sequence are left as
 * they were.
 *  offsets  device int32 [2 pairs + 1], not decreasing, within 0 .. T (values
 *           outside are cut to that range, a decreasing one is read as the largest
 *           before it: no two sequences share a row).
 *  pairs    1 .. MBOK_MAX_PAIRS.
 *  logp     device fp32 [T], of mbok_logp.
 *  ref_logp device fp32 [T] or NULL (all 0): the reference model's.
 *  label    device int32 [T] or NULL (every row holds a token), as for mbok_logp with
 *           the descriptor's vocab: the logits' own, or rows that mbok_logp finds no
 *           token in (labels of V or more) count.
 *  T        1 .. MBOK_MAX_DISTILL_ROWS.
 *  weight   device fp32 [pairs] or NULL (all 1): w.  A pair of weight 0 has loss
 *           and dlogp 0.
 *  loss     device fp32 [pairs]; overwritten.
 *  dlogp    device fp32 [T] or NULL.
 * Errors: INVALID_ARG (NULL, the descriptor's constants), SHAPE (T, pairs, the
 * descriptor's), ALIGN (4 bytes each), HIP.
 */
int mbok_preference(const mbok_preference_desc* d, const int32_t* offsets, int64_t pairs,
                    const float* logp, const float* ref_logp, const int32_t* label, int64_t T,
                    const float* weight, float* loss, float* dlogp, void* stream);

/* ------------------------------------------------------------------------
 * The optimizer step ([RN] 训练策略: the scales are tuned).
 * ------------------------------------------------------------------------ */

/* Values of an 8-bit state that share a scale, and limits of one plan. */
#define MBOK_ADAMW_BLOCK 256
#define MBOK_MAX_ADAMW_TENSORS 65536
#define MBOK_MAX_ADAMW_VALUES ((int64_t)1 << 32)

/*
 * One tensor of a step.  All pointers are device memory.
 *  param        fp32 [count], updated: the master values.
 *  grad         [count] of grad_dtype (MBOK_F32, MBOK_F16, MBOK_BF16).
 *  state_dtype  MBOK_F32: m and v fp32 [count], the moments; m_scale, v_scale NULL.
 *               MBOK_E4M3: m and v are codes [count], m_scale and v_scale fp32
 *               [ceil(count / MBOK_ADAMW_BLOCK)]: the first moment is m m_scale
 *               and the SQUARE ROOT of the second v v_scale of the value's
 *               block.  Zeros are the states before the first step, either way.
 *  layer        NULL: out is NULL or a flat copy of the new values [count] of
 *               out_dtype (MBOK_F32, MBOK_F16, MBOK_BF16).  Else the descriptor of
 *               a layer (read by mbok_adamw_plan_init alone): param are its
 *               scales in mbok_pack's order [K][m][n/128], count = K m n/128, and
 *               out is its packed buffer, in which the step writes the scales, in
 *               the layer's alpha_dtype (rounded once; no signs and no padding
 *               are touched).  out_dtype is not read then.
 *  weight_decay wd, finite, 0 or more.
 */
typedef struct mbok_adamw_tensor {
  float* param;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  void* out;
  const mbok_desc* layer;
  int64_t count;
  double weight_decay;
  int32_t grad_dtype, state_dtype, out_dtype;
} mbok_adamw_tensor;

/* What mbok_adamw needs of a set of tensors beside the table. */
typedef struct mbok_adamw_plan {
  int64_t table_bytes;
  int32_t tensors, parts, lds_bytes;
} mbok_adamw_plan;

/* Bytes of the table of n tensors; 0 if mbok_adamw_plan_init would refuse them.
 * Host only. */
size_t mbok_adamw_table_bytes(const mbok_adamw_tensor* tensors, int32_t n);

/*
 * Fills *plan and the table of n tensors (1 .. MBOK_MAX_ADAMW_TENSORS), in HOST
 * memory of mbok_adamw_table_bytes(tensors, n) bytes; the caller copies it to the
 * device.  Host only.  Errors: INVALID_ARG (NULL; a pointer missing or, of
 * scales, given without 8-bit states; weight_decay; count < 1; two written
 * ranges, of one tensor or of two, that overlap, or one written that is another's
 * gradient), SHAPE (n; more than MBOK_MAX_ADAMW_VALUES values; count is not the
 * layer's), DTYPE, ALIGN (each pointer to its element, out of a layer 16 bytes),
 * SCRATCH (no host memory for the check), and the layer descriptor's.
 */
int mbok_adamw_plan_init(mbok_adamw_plan* plan, const mbok_adamw_tensor* tensors, int32_t n,
                         void* table);

/* Constants of one step. */
typedef struct mbok_adamw_step {
  double lr, beta1, beta2, eps; /* finite; beta in [0, 1), eps at least 2^-126 */
  int64_t step;                 /* t, 1 for the first, below 2^53 */
  float grad_scale;             /* c: gradients are multiplied by it */
  uint32_t seed;                /* of the stochastic rounding of 8-bit states */
} mbok_adamw_step;

/*
 * One step of AdamW on every tensor of a plan, in one kernel:
 *     g' = c g,  m = beta1 m + (1 - beta1) g',  v = beta2 v + (1 - beta2) g'^2
 *     p = p (1 - lr wd) - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32; the same inputs give the same bits.  8-bit states are rounded
 * stochastically to e4m3 with a power-of-two scale per block that puts its
 * largest magnitude in [128, 256); the random bits are a hash of seed, t, the
 * tensor's place in the plan and the value's.  A value that is not finite makes
 * its block's scale NaN.  A root of the second moment of 2^-74 or more is not 0 after
 * a step with beta2 of 1/2 or more (the square of a smaller one is 0 in fp32, as it is
 * with fp32 states).  Scales are at least 2^-87.
 *  table  device, the plan's table, 16-byte aligned; it and the tensors are read when
 *         the step runs, so a captured step needs them as long as its graph lives.
 *  live   device fp32 [4] or NULL: lr, grad_scale, t (a whole number from 1, below 2^24)
 *         and a flag, read when the step runs (so that a captured step follows
 *         them) instead of the constants of `step`; a flag other than 0 (an
 *         overflow was found) or t below 1 or NaN (a buffer not filled yet) skips the
 *         step: nothing is written.
 * Errors: INVALID_ARG (NULL, constants out of range, a plan that is none), ALIGN
 * (table 16 bytes, live 4), HIP.
 */
int mbok_adamw(const mbok_adamw_plan* plan, const void* table, const mbok_adamw_step* step,
               const float* live, void* stream);

/* Static description of a status code ("unknown status" for others). */
const char* mbok_status_str(int status);

/* Library version, e.g. "mbok 0.1.0 gfx950". */
const char* mbok_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MBOK_H */
