/*
 * hsl.h — C ABI of libhsl: weight matrices compressed as W ≈ S + U Vᵀ
 * ("hierarchical sparse + low-rank"), split and applied on one B200 (sm_100a).
 *
 * Source of the operations (cited by page title and section):
 *   [HSS]    "Hierarchical Sparse + Low-Rank Compression of LLMs"
 *            (LLMの階層的スパース+低ランク圧縮)
 *            - §Two-stage hierarchical sparse + low-rank compression:
 *              W ≈ S + U Vᵀ, U ∈ R^{m×r}, V ∈ R^{n×r}; Stage 1 keeps the
 *              largest-magnitude weights in a sparse matrix (COO/CSR), the
 *              rest is the dense residual; Stage 2 factors the residual.
 *            - §Implementation and operational patterns: the layer holds
 *              (S, U, V) and computes the forward as a sparse product plus
 *              two small dense products without forming W.
 *            - §Implementation and operational patterns (from theory to
 *              production), mixed precision: 16-bit factors and narrow
 *              sparse indices.
 *   [HASSLE] HASSLE-free article (aibr.jp/archives/82335), §3: N:M
 *            structured sparsity as the GPU-friendly form of S.
 *   [SQZ]    SqueezeLLM article (aibr.jp/archives/208940), §1: single-batch
 *            decoding is bound by reading the weights from memory.
 *
 * Conventions (all entry points):
 *   - Shapes: W and Ŵ are m×n (m output features, n input features),
 *     row-major.  X is [batch][n], Y is [batch][m], row-major, and each row
 *     satisfies y = Ŵ x = S x + U (Vᵀ x).  (The page writes the same product
 *     in row-vector form, output = input @ (S + U Vᵀ); this is its transpose.)
 *   - Data pointers are DEVICE pointers owned by the caller, unless an entry
 *     point says otherwise.  The handle owns only its own copies (canonical
 *     and packed S, U, V) and workspace, allocated by the call that first
 *     needs them and released by hsl_destroy.
 *   - Every call taking a stream is asynchronous and stream-ordered on it.
 *     A stream is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Host-side argument checks return immediately; launch errors
 *     come back as HSL_ERR_CUDA.  Errors found on the device (NaN in W, a
 *     bounded wait that ran out) are recorded in the handle and returned by
 *     hsl_check.  Nothing aborts and no C++ exception crosses the ABI.
 *   - A handle is not thread-safe and keeps per-call workspace: use one
 *     handle per stream, and do not overlap calls on one handle across
 *     streams.
 *   - hsl_check reports a CSR column index outside [0, n) found while packing
 *     an imported S as HSL_ERR_INVALID_ARG (the entry is dropped).
 *   - Calls that allocate (the first split/set/pack/apply of a handle, or a
 *     split with a larger k than before) must not be made under stream
 *     capture; repeat calls with the same sizes allocate nothing.
 */
#ifndef HSL_H_
#define HSL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct hsl_handle_s* hsl_handle;
typedef void* hsl_stream; /* cudaStream_t */

typedef enum {
  HSL_OK = 0,
  HSL_ERR_INVALID_ARG = 1, /* a NULL/out-of-range argument, host-side check */
  HSL_ERR_UNSUPPORTED = 2, /* a valid request the library does not handle   */
  HSL_ERR_NOT_READY = 3,   /* e.g. hsl_apply before hsl_pack                */
  HSL_ERR_OOM = 4,         /* a device allocation failed                    */
  HSL_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed          */
  HSL_ERR_NAN_INPUT = 6,   /* W held a NaN (device-detected, via hsl_check) */
  HSL_ERR_TIMEOUT = 7      /* a bounded device wait gave up (via hsl_check) */
} hsl_status;

typedef enum { HSL_FMT_CSR = 0, HSL_FMT_NM24 = 1 } hsl_format;
typedef enum { HSL_F32 = 0, HSL_BF16 = 1 } hsl_dtype;

/* Create a layer handle for an m×n matrix with rank-r factors.
 *   fmt:   HSL_FMT_CSR (unstructured top-k S) or HSL_FMT_NM24 (2:4 S;
 *          needs n % 4 == 0).
 *   dtype: storage and arithmetic type of S values, U, V, X and Y
 *          (HSL_F32 or HSL_BF16); products accumulate in fp32.
 * Limits: 1 ≤ m, n; m·n < 2^31; 0 ≤ r ≤ 256.
 * Allocates nothing on the device; *out owns what later calls allocate.
 * [HSS] §Two-stage compression (the (S, U, V) triple), §Implementation. */
hsl_status hsl_create(int64_t m, int64_t n, int32_t r, hsl_format fmt,
                      hsl_dtype dtype, hsl_handle* out);

/* Release the handle and all device memory it owns.  Waits for the device
 * (cudaDeviceSynchronize on the handle's device) before freeing.  NULL is
 * a no-op.  The handle is the layer object of [HSS] §Implementation and
 * operational patterns, which holds (S, U, V) in place of the dense weight;
 * this ends its life. */
hsl_status hsl_destroy(hsl_handle h);

/* Stage 1: split W into S (kept in the handle) and the residual.
 *   W:        device, m×n row-major, element type w_dtype.
 *   frac:     CSR handles keep k = floor(frac·m·n) entries (frac ≤ 0 → 0,
 *             frac ≥ 1 → m·n), chosen by |w| descending with ties to the
 *             lower linear index i·n + j (exact radix select on the
 *             magnitude bits).  NM24 handles need frac == 0.5 and keep,
 *             in every group of 4 consecutive inputs of a row, the 2
 *             largest |w| (ties to the lower in-group index).
 *   residual: device, m×n of w_dtype, or NULL; receives W with the kept
 *             positions set to +0.0, bit-exact elsewhere.
 * S values are stored in the handle dtype (f32 → bf16 rounds to nearest
 * even; bf16 → f32 is exact).  A NaN in W is reported by hsl_check as
 * HSL_ERR_NAN_INPUT (the outputs are then meaningless but in bounds).
 * Invalidates any earlier hsl_pack.
 * [HSS] §Two-stage compression, Stage 1; [HASSLE] §3 for 2:4. */
hsl_status hsl_split_topk(hsl_handle h, const void* W, hsl_dtype w_dtype,
                          double frac, void* residual, hsl_stream s);

/* Top-k split that allocates no device memory.  The source pages have no
 * counterpart of this entry point: it exists for callers that may not call
 * cudaMalloc — code inside a serving runtime or plugin host that owns all
 * device memory and hands out pre-planned buffers, code that must not risk the
 * device-wide synchronisation of cudaMalloc/cudaFree, or callers without a
 * handle to keep workspace alive.  It computes exactly what hsl_split_topk
 * computes on a CSR handle (same kernels, bit-identical results), with every
 * input and output owned by the caller and no handle:
 *   W:        device, m×n row-major, element type w_dtype.
 *   frac:     k = floor(frac·m·n) kept (frac ≤ 0 → 0, frac ≥ 1 → m·n).
 *   row_ptr:  device int32[m+1];  col: device int32[k];  val: device, k values
 *             of val_dtype (f32 → bf16 rounds to nearest even).  col/val may
 *             be NULL when k == 0.
 *   residual: device m×n of w_dtype, or NULL.
 *   status:   device uint32, required (NULL → HSL_ERR_INVALID_ARG): it is the
 *             only channel for device-detected errors.  Cleared, then OR-ed
 *             with 1 for a NaN in W and 2 for a device wait that gave up.
 * Scratch: one fixed static device array of about 2.2 MB per GPU (held until
 * the process exits).  Limits: m ≤ 65536, n ≤ 2^31 − 1 and m·n < 2^31, else
 * HSL_ERR_UNSUPPORTED.  The first call on a device looks the array up with
 * that device current (make it before any stream capture).  All calls share
 * the array, so calls that can overlap on the GPU race: serialise them on one
 * stream.  Asynchronous on s, like the other entry points.
 * What it computes: [HSS] §Two-stage compression, Stage 1 (as hsl_split_topk). */
hsl_status hsl_split_topk_noalloc(const void* W, int64_t m, int64_t n, hsl_dtype w_dtype,
                                  double frac, int32_t* row_ptr, int32_t* col, void* val,
                                  hsl_dtype val_dtype, void* residual, uint32_t* status,
                                  hsl_stream s);

/* Number of stored sparse values (k for CSR, m·n/2 for NM24; 0 before any
 * split/set).  Host-only, no synchronisation (k is known on the host).
 * [HSS] §Two-stage compression, worked example: the count of kept weights
 * (52,428 for 5 % of a 1024×1024 matrix) that enters the parameter total. */
hsl_status hsl_get_nnz(hsl_handle h, int64_t* nnz);

/* Export the canonical S (stream-ordered device→device copies).
 * [HSS] §Two-stage compression, Stage 1: the kept weights are stored as a
 * sparse matrix in COO/CSR form; [HASSLE] §3 for the N:M form.
 *   CSR:  row_ptr[m+1] int32, col[nnz] int32 (ascending in each row),
 *         val[nnz] of the handle dtype; nm_idx unused (may be NULL).
 *   NM24: val[m][n/2] (the two kept values of each group, ascending column),
 *         nm_idx[m][n/4] uint8 = i0 | i1 << 2 with in-group indices
 *         i0 < i1; row_ptr/col unused (may be NULL). */
hsl_status hsl_get_sparse(hsl_handle h, int32_t* row_ptr, int32_t* col,
                          void* val, uint8_t* nm_idx, hsl_stream s);

/* Import a canonical CSR S (same layout as hsl_get_sparse), e.g. from a
 * checkpoint ([HSS] §Two-stage compression, Stage 1: S in COO/CSR form).  Columns must be < n; the handle trusts row_ptr to be
 * monotone with row_ptr[0] = 0 and row_ptr[m] = nnz.  CSR handles only.
 * Invalidates any earlier hsl_pack. */
hsl_status hsl_set_sparse_csr(hsl_handle h, int64_t nnz, const int32_t* row_ptr,
                              const int32_t* col, const void* val, hsl_stream s);

/* Import a canonical 2:4 S (layout as hsl_get_sparse; [HASSLE] §3, N:M
 * structured sparsity).  NM24 handles only.
 * Invalidates any earlier hsl_pack. */
hsl_status hsl_set_sparse_nm24(hsl_handle h, const void* val, const uint8_t* nm_idx,
                               hsl_stream s);

/* Build the device layouts hsl_apply streams: S repacked (CSR: rows padded
 * to 8 values with 16-bit column indices, [HSS] §Implementation (mixed
 * precision: narrow indices; the width is chosen by hsl_set_index_bits);
 * NM24: metadata interleaved per warp lane),
 * and copies of U [m][r] and V [n][r] (row-major, handle dtype, device).
 * Needs S (split or set) first, else HSL_ERR_NOT_READY. */
hsl_status hsl_pack(hsl_handle h, const void* U, const void* V, hsl_stream s);

/* Column-index width of the packed CSR S, used from the next hsl_pack on:
 *   16 — 16-bit columns (needs n < 65535); the default when n < 65535;
 *   32 — 32-bit columns (any n); the default when n ≥ 65535;
 *    8 — one delta byte per entry (column minus the previous entry's) plus a
 *        16-bit column base per 8-entry vector: 1.25 bytes per entry against
 *        2, so 3.25 instead of 4 streamed bytes per bf16 entry at decode.
 *        A gap of more than 255 columns inside a row takes filler entries
 *        (value 0, one per 255 columns); needs n < 65535 and each row's
 *        columns in ascending order (else hsl_pack returns HSL_ERR_UNSUPPORTED);
 *    0 — back to the default.
 * Large batches on the tensor cores use 16-bit columns; with another width
 * they run on the decode kernel.  CSR handles only; invalidates hsl_pack.
 * [HSS] §Implementation and operational patterns (from theory to production),
 * mixed precision: sparse indices as INT32 or in narrower integers (INT16,
 * INT8) to cut the memory of S further. */
hsl_status hsl_set_index_bits(hsl_handle h, int32_t bits);

/* Y = X Ŵᵀ, i.e. y = S x + U (Vᵀ x) for each of the batch rows of X.
 *   X: [batch][n], Y: [batch][m], handle dtype, row-major.  X and Y may be
 *   device pointers, or host pointers (pinned or pageable), in which case
 *   the call stages them through handle-owned device buffers with
 *   cudaMemcpyAsync on s (pinned Y: synchronise s before reading it).
 *   batch = 0 is a no-op.  Needs hsl_pack first, else HSL_ERR_NOT_READY.
 * [HSS] §Implementation and operational patterns, the forward
 * decomposition; [SQZ] §1 for why decode batches stream the weights. */
hsl_status hsl_apply(hsl_handle h, const void* X, void* Y, int64_t batch, hsl_stream s);

/* A group applies `count` independent layers in one pass (e.g. every
 * projection of a model at decode): one launch per kernel stage covers all of
 * them, with the rows of all layers split into CTA ranges of equal streamed
 * bytes.  All members must be packed and share format, dtype and device.
 * The group refers to the members' packed buffers: re-splitting, re-setting,
 * re-packing or destroying a member invalidates it (hsl_group_apply then
 * returns HSL_ERR_NOT_READY for a re-split member; create the group again).
 * Creating a group uploads its plan on s and synchronises s once.
 * [HSS] §Implementation and operational patterns (operating patterns): layers
 * are compressed and deployed one by one across a model's attention and MLP
 * projections; a group applies such a set of layers together. */
typedef struct hsl_group_s* hsl_group;
hsl_status hsl_group_create(const hsl_handle* hs, int32_t count, hsl_group* out, hsl_stream s);

/* Y[i] = apply(member i, X[i]) for every member; X[i] is [batch][n_i] and
 * Y[i] is [batch][m_i], device pointers.  The pointer tables are host
 * arrays; they are uploaded to the device only when they change.
 * Each member's product is the forward decomposition of hsl_apply ([HSS]
 * §Implementation and operational patterns; [SQZ] §1). */
hsl_status hsl_group_apply(hsl_group g, const void* const* X, void* const* Y, int64_t batch,
                           hsl_stream s);

/* Release the group (synchronises its device first).  NULL is a no-op.
 * [HSS] §Implementation and operational patterns (the layers held for the
 * forward pass), as hsl_group_create. */
hsl_status hsl_group_destroy(hsl_group g);

/* Stage 2 on the GPU: the rank-r factors of the residual R (device, m×n of
 * r_dtype; e.g. the residual hsl_split_topk wrote) as its truncated SVD with
 * √σ on each side, R ≈ U Vᵀ, U = U_r √Σ_r, V = V_r √Σ_r, computed by the
 * randomized range finder (Halko–Martinsson–Tropp) with the caller's Gaussian
 * test matrix:
 *   omega:       device fp32 [n][k], r ≤ k ≤ min(m, n, 512) (k − r is the
 *                oversampling);
 *   power_iters: q ≥ 0 subspace iterations (Y ← R Rᵀ Q, then Q = orth(Y));
 *   U [m][r], V [n][r]: device, handle dtype (pass them to hsl_pack);
 *   sigma [r]: device fp32, σ_1 ≥ … ≥ σ_r (0 where R has no such direction).
 * The tall products run on the tensor cores with fp32 operands split into
 * three bf16 terms (fp32-accurate); orthonormalisation and the small SVD use
 * fp64 Gram matrices and a Jacobi eigensolver.  Uses the handle's m, n, r and
 * dtype; allocates its workspace for the call (about 2·m·n·2 bytes for bf16
 * R) and synchronises s before freeing it.  r = 0 is a no-op.
 * [HSS] §Two-stage compression, Stage 2 (the residual factored into two
 * m×r / n×r matrices), and the implementation flow (low-rank factorisation,
 * O(n³)). */
hsl_status hsl_factor(hsl_handle h, const void* R, hsl_dtype r_dtype, const float* omega, int32_t k,
                      int32_t power_iters, void* U, void* V, float* sigma, hsl_stream s);

/* ---- Permutation for concentration ------------------------------------------
 * [HSS] §Permutation and hierarchical alignment: reorder the rows and columns
 * of W (reverse Cuthill–McKee) so that its large entries gather near the
 * diagonal, measure the gain with the concentration ratio
 *   ρ = Σ_{diagonal blocks} |W_ij| / Σ |W_ij|,
 * and keep the order so the layer is applied in the original order. */

/* ρ of W (device, m×n row-major, dtype): the diagonal blocks are the top-left
 * and bottom-right blocks of the 2×2 partition split at row ⌊m/2⌋ and column
 * ⌊n/2⌋; an all-zero W gives 0, a NaN in W gives NaN.  Sums in fp64 in a fixed
 * order (deterministic).  Writes *rho (host) and synchronises s.  Allocates a
 * small workspace for the call and frees it.
 * [HSS] §Permutation and hierarchical alignment (the ρ equation). */
hsl_status hsl_concentration(const void* W, int64_t m, int64_t n, hsl_dtype dtype, double* rho,
                             hsl_stream s);

/* Reverse Cuthill–McKee order of an m×n sparse pattern given as a HOST CSR
 * (row_ptr[m+1] from 0, col[row_ptr[m]] in [0, n)).  The graph is the
 * bipartite row–column graph (an edge per stored entry); start each component
 * at the unvisited vertex of least degree (ties: rows before columns, lower
 * index first), visit breadth first taking neighbours by increasing degree
 * (same ties), reverse the whole order.  row_order[k] / col_order[k] (host,
 * m and n int32) receive the original row / column placed k-th.  Runs on the
 * host (a one-off graph step); HSL_ERR_INVALID_ARG for a bad pattern.
 * [HSS] §Permutation and hierarchical alignment (reverse Cuthill–McKee). */
hsl_status hsl_rcm_order(int64_t m, int64_t n, const int32_t* row_ptr, const int32_t* col,
                         int32_t* row_order, int32_t* col_order);

/* out[k][l] = W[row_order[k]][col_order[l]] (device arrays; bit copies).  The
 * orders are copied to the host and checked to be permutations first
 * (HSL_ERR_INVALID_ARG otherwise), which synchronises s.
 * [HSS] §Permutation and hierarchical alignment (W permuted before the split). */
hsl_status hsl_permute(const void* W, int64_t m, int64_t n, hsl_dtype dtype,
                       const int32_t* row_order, const int32_t* col_order, void* out,
                       hsl_stream s);

/* Declare that the handle holds the permuted layer W' = W[row_order][:, col_order]
 * (split, set and packed from W'), so that hsl_apply returns the original
 * layer's output: x' = x[col_order], y' = Ŵ' x', y[row_order[k]] = y'[k].
 * Device arrays, copied into the handle after a host-side permutation check
 * (synchronises s).  NULL for both clears it.  Groups do not take permuted
 * layers.  [HSS] §Permutation and hierarchical alignment (outputs in the
 * original order). */
hsl_status hsl_set_permutation(hsl_handle h, const int32_t* row_order, const int32_t* col_order,
                               hsl_stream s);

/* ---- Microscaled blocks: 4-bit weights and 8-bit activations ------------------
 * 32 consecutive values of a row share one power of two.  A matrix in blocks
 * is plain device memory of the caller's, in this layout:
 *   scales  [rows][scale_pitch] bytes e (ue8m0): the block's power of two is
 *           2^(e − 127); e = 255: the block stands for NaN.  scale_pitch is
 *           ceil(cols/32) rounded up to a multiple of 16; padding bytes are 0.
 *   codes   [rows][code_pitch] bytes, whole blocks per row, padding codes 0:
 *     HSL_MX_E2M1  code_pitch = 16·ceil(cols/32).  4-bit floats; bit 3 is the
 *                  sign, codes 0..7 stand for 0, 0.5, 1, 1.5, 2, 3, 4, 6;
 *                  element 2i of a row is the low half of byte i.
 *     HSL_MX_INT8  code_pitch = 32·ceil(cols/32).  Integers in −127..127 that
 *                  stand for q/64.
 * Both arrays must be 16-byte aligned.  These are the element and scale types
 * of the OCP Microscaling Formats specification v1.0 (MXFP4, MXINT8).
 *
 * What they serve: [SQZ] §2–4, Dense-and-Sparse: W = D + S with a low-bit dense
 * D and the outliers in a sparse S, multiplied in parallel; here D (e2m1) joins
 * the layer's S and U Vᵀ through the `add` argument of the products.  [HSS]
 * §Implementation and operational patterns, backward pass: the gradients of the
 * factors, taken from activations kept in 8 bits.
 *
 * The calls own nothing and keep nothing between calls.  Those that need
 * scratch memory take it from the caller: hsl_mx_workspace gives the bytes for
 * the sizes of a call (16-byte aligned; contents need not survive the call, and
 * calls that may overlap need one each).  The device of the pointers and the
 * stream must be current.  All are asynchronous on s, allocate nothing and can
 * be captured.  X, Y and the other plain matrices start on a whole element.
 * Outputs and scratch may not overlap each other or an input (but `add` may be
 * the output itself).  Rows, columns and batches are at most 2^30. */
typedef enum { HSL_MX_E2M1 = 0, HSL_MX_INT8 = 1 } hsl_mx_elem;
typedef struct {
  const void* codes;
  const void* scales;
  int64_t rows, cols;
  hsl_mx_elem elem;
} hsl_mx;
typedef enum {
  HSL_MX_OP_APPLY = 0,
  HSL_MX_OP_APPLY_T = 1,
  HSL_MX_OP_MATMUL = 2,
  HSL_MX_OP_FACTOR_GRAD = 3
} hsl_mx_op;

/* Row pitches in bytes of a matrix with `cols` columns.  Host-only.
 * [HSS] §Implementation and operational patterns, mixed precision (the storage
 * format of a compressed weight). */
hsl_status hsl_mx_pitch(int64_t cols, hsl_mx_elem elem, int64_t* code_pitch, int64_t* scale_pitch);

/* Scratch bytes of a product: batch (rows of X, dY, A or of the checkpoint),
 * m×n of D (or B rows × cols, or U rows × V rows), r of the factors.
 * Host-only.  [HSS] §Implementation and operational patterns (the forward and
 * backward products whose scratch this is). */
hsl_status hsl_mx_workspace(hsl_mx_op op, int64_t batch, int64_t m, int64_t n, int64_t r,
                            hsl_dtype dtype, size_t* bytes);

/* Quantise X (device, rows×cols row-major) into blocks along its rows:
 *   s = 2^(floor(log2 max|x|) − emax), emax = 2 (e2m1) or 0 (int8), exponent
 *       clamped to −127..127;   q = x/s rounded to nearest even, saturating.
 * Every code is determined by this (division by s is exact).  A block of zeros
 * gets e = 0 and codes that stand for 0 (in e2m1 −0 keeps its sign bit); a block with a NaN or an infinity e = 255 and zero
 * codes.  rows = 0 is a no-op.
 * [SQZ] §2–4 (the low-bit dense part); the rule is that of the OCP
 * specification, §6.3. */
hsl_status hsl_mx_quantize(const void* X, hsl_dtype dtype, int64_t rows, int64_t cols,
                           hsl_mx_elem elem, void* codes, void* scales, hsl_stream s);

/* X[rows][cols] = the values the blocks stand for (exact in both dtypes; a
 * value past the dtype's range becomes infinite).  [SQZ] §2–4, as
 * hsl_mx_quantize. */
hsl_status hsl_mx_dequantize(const hsl_mx* q, void* X, hsl_dtype dtype, hsl_stream s);

/* Y = X Dᵀ (+ add): y[t][i] = add[t][i] + Σ_j x[t][j] d[i][j], D m×n in e2m1 blocks,
 * X [batch][n], Y and add [batch][m] of dtype (add may be NULL, or Y itself);
 * products and sums in fp32, one rounding at the end.  batch = 0 is a no-op.
 * [SQZ] §2–4: the dense term of (D + S) x; [SQZ] §1 for why it is bound by the
 * bytes of D at small batches. */
hsl_status hsl_mx4_apply(const hsl_mx* D, const void* X, const void* add, void* Y, int64_t batch,
                         hsl_dtype dtype, void* ws, size_t ws_bytes, hsl_stream s);

/* dX = dY D (+ add): the gradient of hsl_mx4_apply's input; dY [batch][m], dX and
 * add [batch][n] (add may be NULL, or dX itself).
 * [HSS] §Implementation and operational patterns, backward pass. */
hsl_status hsl_mx4_apply_t(const hsl_mx* D, const void* dY, const void* add, void* dX, int64_t batch,
                           hsl_dtype dtype, void* ws, size_t ws_bytes, hsl_stream s);

/* Y = A Bᵀ (+ add), both in e2m1 blocks with the same number of columns; Y and add
 * [A.rows][B.rows] of dtype (add may be NULL, or Y itself), sums in fp32.
 * [SQZ] §2–4, as hsl_mx4_apply, with the activations in 4 bits as well. */
hsl_status hsl_mx4_matmul(const hsl_mx* A, const hsl_mx* B, const void* add, void* Y, hsl_dtype dtype,
                          void* ws, size_t ws_bytes, hsl_stream s);

/* Backward pass of x → U (Vᵀ x) from a checkpoint of its input in int8 blocks:
 *   Z = X V, G = dY U;  dU = dYᵀ Z, dV = Xᵀ G, dX = G Vᵀ (+ add)
 * X [T][n] blocks (T = X.rows; T = 0 writes zeros to dU and dV), dY [T][m],
 * U and dU [m][r], V and dV [n][r], dX and add [T][n] of dtype; dX may be NULL
 * (then add must be), add may be NULL or dX itself.  1 ≤ r ≤ 256.  Sums are fp32,
 * and so are Z and G (bf16: below 2^−109 to the nearest multiple of about 2^−133).
 * With an infinity in dY, U or V, what is infinite by the formulas may come out as a
 * NaN (and nothing else is touched).
 * [HSS] §Implementation and operational patterns, backward pass (the gradients
 * of U and V, as derived from the forward decomposition). */
hsl_status hsl_mx8_factor_grad(const hsl_mx* X, const void* dY, int64_t m, const void* U,
                               const void* V, int32_t r, const void* add, void* dU, void* dV, void* dX,
                               hsl_dtype dtype, void* ws, size_t ws_bytes, hsl_stream s);

/* Synchronise s and return, then clear, the device-side error of the microscaled
 * operators on the current device: HSL_ERR_TIMEOUT if a bounded device wait of
 * any of them gave up (its output is then incomplete), HSL_OK if none did.  The
 * calls have no handle, so that the error is the device's: the first check after
 * it has it, on whatever stream or thread.  No report is lost.
 * [HSS] §Risks and mitigations, risk 1, as hsl_check. */
hsl_status hsl_mx_check(hsl_stream s);

/* Synchronise s and return, then clear, the device-side error of the handle
 * (HSL_ERR_NAN_INPUT, HSL_ERR_TIMEOUT) — HSL_OK if none.
 * [HSS] §Risks and mitigations, risk 1: keep the uncompressed weights as a
 * fallback for a compressed layer that misbehaves; this call is the detection
 * half of that, as a status. */
hsl_status hsl_check(hsl_handle h, hsl_stream s);

/* Static text for a status code (the statuses of hsl_check and of the
 * host-side checks; [HSS] §Risks and mitigations, risk 1, the same
 * detection-and-fallback passage). */
const char* hsl_status_str(hsl_status st);

/* Detail of the last failing call on this thread ("" if none).
 * [HSS] §Risks and mitigations, risk 1 (detection of a misbehaving layer),
 * as hsl_status_str. */
const char* hsl_last_message(void);

/* Number of kernels libhsl has launched in this process (all devices).
 * [HSS] §Implementation and operational patterns (actionable suggestions):
 * profile the compressed layers on the target hardware; this count lets a
 * profile tell the library's own kernels from everything else. */
uint64_t hsl_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* HSL_H_ */
