/*
 * qmm.h -- C ABI of libqmm: affine group-quantized small-M matmul for
 * AMD Instinct MI355X (gfx950).
 *
 * The operation is y[M,N] = x[M,K] . dequant(Wq[N,K])^T, the transposed
 * quantized matmul of a speculative-decoding verify step (M = 4..6 rows for
 * 3..5 draft tokens) and of batched decode (M up to 64):
 *   - "How the NAX Verify Kernel Path Improves Decode Performance in MTPLX",
 *     sections "Architectural Differences" (verify shapes M = 4-6) and
 *     "Implementation and Configuration" (operands x, w_q, scales, biases;
 *     y has shape (M, N));
 *   - MLX issue #4720 "[BUG] qmm_splitk is chosen over qmm_nax on M5 ...",
 *     "To Reproduce" (quantize(w, group_size, bits) -> (wq, scales, biases);
 *     quantized_matmul(x, wq, scales, biases, transpose=True, ...)).
 * Supported formats follow "What Are NAX Verify Kernels and When Is the
 * Turbo Profile Activated in MTPLX?", "Supported Data Formats and
 * Quantization Schemes": 4-, 6- or 8-bit affine codes, group sizes 32, 64,
 * 128, fp16 or bf16 activations.
 *
 * Data layout (all arrays dense, row-major, caller-owned device memory):
 *   w       [N, K]            dtype dt (weights before quantization)
 *   wq      [N, K*bits/32]    uint32; each row is a little-endian bitstream
 *                             with code k at bits [bits*k, bits*k+bits):
 *                             4-bit = 8 codes per word, low nibble first;
 *                             8-bit = 4 codes per word; 6-bit = 4 codes per
 *                             24 bits (16 codes per 3 words)
 *   scales  [N, K/gs]         dtype dt
 *   biases  [N, K/gs]         dtype dt
 *   x       [M, K]            dtype dt
 *   y       [M, N]            dtype dt
 * Dequantized weight: w_hat = s*q + b.  Accumulation is fp32; y is rounded
 * once to dt (nearest-even).
 *
 * Quantizer (no formula is printed on the pages; this is the min/max affine
 * reading): per group, lo = min, hi = max,
 *   s = fp32 (hi - lo) / (2^bits - 1), stored in dt rounded toward +inf;
 *   b = lo;  q = clamp(rint_half_even(fp32 (w - b) / s), 0, 2^bits - 1),
 *   and q = 0 when s == 0 (constant group).
 *
 * Conventions shared by every entry point:
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream).
 *     No entry point synchronizes, allocates memory or keeps a pointer
 *     after it returns; the caller keeps buffers alive until the stream has
 *     passed the call (scratch, where a variant needs it, is a
 *     caller-provided workspace).  Entry points are thread-safe.
 *   - Arguments are validated before any HIP call.  Return values:
 *       QMM_OK               success (also for empty problems: M == 0 or
 *                            N == 0 launch nothing and may pass NULL)
 *       QMM_ERR_INVALID_ARG  negative size, or NULL pointer for a non-empty
 *                            array
 *       QMM_ERR_UNSUPPORTED  dt not fp16/bf16, bits not 4/6/8, group size
 *                            not 32/64/128, K < 64 or K % 64 != 0,
 *                            K % group_size != 0, M > 64, unknown kernel id
 *       QMM_ERR_MISALIGNED   an array base pointer not 16-byte aligned
 *       QMM_ERR_HIP          the launch failed (asynchronous faults surface
 *                            at the caller's next synchronization)
 *   - Inputs must be finite; inputs to the quantizer must have a finite
 *     fp32 group range.  Output arrays must not alias input arrays.
 */
#ifndef QMM_H
#define QMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum qmm_dtype { QMM_F16 = 0, QMM_BF16 = 1 };

enum qmm_status {
    QMM_OK = 0,
    QMM_ERR_INVALID_ARG = -1,
    QMM_ERR_UNSUPPORTED = -2,
    QMM_ERR_MISALIGNED = -3,
    QMM_ERR_HIP = -4
};

/* Kernel variants for qmm_small_m_forced / qmm_select_kernel. */
enum qmm_kernel {
    QMM_KERNEL_VALU = 0,      /* split-free, VALU dot products, cross-lane K reduction */
    QMM_KERNEL_MFMA_REG = 1,  /* split-free, MFMA with in-register weight fragments (16-row blocks above 16 rows) */
    QMM_KERNEL_MFMA_PASS = 2, /* split-free, MFMA, K walked in passes of 16 k-blocks, any K, M <= 64 */
    QMM_KERNEL_MFMA_TILE16 = 3, /* split-free, MFMA, 16-column tiles, activations shared through LDS, M <= 64 */
    QMM_KERNEL_MFMA_TILE64 = 4, /* as TILE16 with 64-column tiles (wide N) */
    QMM_KERNEL_MFMA_DQLDS = 5,  /* split-free, MFMA, weights dequantized into LDS (64-column tiles, M <= 64,
                                   N a multiple of 64, K a multiple of 256) */
    QMM_KERNEL_COUNT = 6
};

/*
 * Quantize W [N, K] (dtype dt) into wq / scales / biases with the rule
 * above.  Bit-exact: the same inputs always give the same words, scales
 * and biases.
 */
int qmm_quantize(int dt, int bits, int group_size, int64_t N, int64_t K,
                 const void* w, uint32_t* wq, void* scales, void* biases,
                 void* stream);

/*
 * Dequantize into w_out [N, K] (dtype dt): w_out = RNE_dt(fp32(s*q + b)).
 * s*q is exact in fp32, so this is one fp32 rounding then one rounding to
 * dt.  Bit-exact.
 */
int qmm_dequantize(int dt, int bits, int group_size, int64_t N, int64_t K,
                   const uint32_t* wq, const void* scales, const void* biases,
                   void* w_out, void* stream);

/*
 * y [M, N] = x [M, K] . dequant(wq, scales, biases)^T with fp32
 * accumulation and one rounding to dt.  1 <= M <= 64 (M == 0 is an empty
 * no-op).  The kernel variant is chosen by qmm_select_kernel.
 * Deterministic: identical inputs give bit-identical outputs.
 */
int qmm_small_m(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K,
                const void* x, const uint32_t* wq, const void* scales,
                const void* biases, void* y, void* stream);

/*
 * Batched form: `batch` independent products, each with its own weights,
 *   y[b] [M, N] = x[b] [M, K] . dequant(wq[b], scales[b], biases[b])^T,
 * over dense arrays x [batch, M, K], wq [batch, N, K*bits/32],
 * scales / biases [batch, N, K/gs], y [batch, M, N] (entry b at b times one
 * entry's size).  MLX issue #4720, "Describe the bug", confines its dispatch
 * story to transposed, non-batched calls; this is the batched case of the
 * same product.  The variant is the one qmm_small_m picks for (M, N, K);
 * the register-resident variant runs every entry in one launch (entries
 * share its resident workgroups), the others launch once per entry.  Each
 * entry's result is bit-identical to qmm_small_m on that entry.
 * batch < 0 -> QMM_ERR_INVALID_ARG; batch == 0 (or M == 0 or N == 0) ->
 * QMM_OK with nothing launched (NULL allowed); with batch > 1 every entry's
 * arrays must start 16-byte aligned (M*K*2, N*K*bits/8, N*(K/gs)*2 and
 * M*N*2 bytes multiples of 16), else QMM_ERR_MISALIGNED.  Otherwise as
 * qmm_small_m.
 */
int qmm_small_m_batched(int dt, int bits, int group_size, int64_t batch, int64_t M, int64_t N, int64_t K,
                        const void* x, const uint32_t* wq, const void* scales, const void* biases,
                        void* y, void* stream);

/*
 * Non-transposed weights: y [M, N] = x [M, K] . dequant(wq, scales, biases),
 * with W stored [K, N] and quantized along N -- the other orientation of the
 * call in MLX issue #4720, "Describe the bug" (transposed weights there):
 *   wq      [K, N*bits/32]  row k = the packed codes of W[k, :] (same
 *                           bitstream as a transposed row)
 *   scales  [K, N/gs]       one scale and bias per gs consecutive columns
 *   biases  [K, N/gs]
 * (what qmm_quantize produces from a [K, N] matrix).  fp32 accumulation and
 * one rounding to dt; deterministic.  N obeys the rules K obeys in
 * qmm_small_m (N >= 64, N % 64 == 0, N % gs == 0); K must be a positive
 * multiple of 32; 1 <= M <= 64 (M == 0: QMM_OK, nothing launched).
 * Otherwise as qmm_small_m.
 */
int qmm_small_m_nt(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K,
                   const void* x, const uint32_t* wq, const void* scales,
                   const void* biases, void* y, void* stream);

/*
 * Non-transposed weights with K split across workgroups: as qmm_small_m_nt,
 * with column-block workgroups each taking one slice of K and leaving fp32
 * partial outputs ([split][M][N]) in a caller-provided workspace; a second
 * kernel adds them in slice order and rounds once (deterministic).  4/8-bit
 * codes with N >= 4096: 256-column blocks on the fewest slices of whole
 * 16 KiB chunks dividing K that give 224..512 workgroups (at most 32 slices;
 * unsplit from 256 blocks); otherwise 128-column blocks on at most 16 slices
 * for about 256 workgroups.
 * Where the plan does not split (wide N, short K) the workspace may be NULL
 * and the call is exactly qmm_small_m_nt.
 * qmm_small_m_nt_workspace_bytes: bytes of workspace the call needs (0: no
 * split), or a negative status.  Pure host logic.
 * qmm_small_m_nt_ws: workspace is caller-owned device memory of
 * workspace_bytes >= that, 16-byte aligned, not aliasing the other arrays;
 * too small or NULL when needed -> QMM_ERR_INVALID_ARG, misaligned ->
 * QMM_ERR_MISALIGNED.  Two calls in flight need two workspaces.
 */
int64_t qmm_small_m_nt_workspace_bytes(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K);
int qmm_small_m_nt_ws(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K,
                      const void* x, const uint32_t* wq, const void* scales, const void* biases,
                      void* y, void* workspace, int64_t workspace_bytes, void* stream);

/* As qmm_small_m with the variant forced (measurement and tests): the
 * counterpart of timing qmm_nax forced against the stock dispatch in MLX
 * issue #4720, "Expected behavior".
 * QMM_ERR_UNSUPPORTED if the variant cannot run this shape
 * (QMM_KERNEL_MFMA_REG needs K <= 4096; for M = 17..64 it runs on 16-row
 * blocks and needs K to fill 16 wavefronts with whole k-blocks (above 1024
 * for 4-bit codes, above 512 for 6/8-bit) and N either to give more 4-bit
 * 16-column tiles than its row-block slots or at most one tile per resident
 * workgroup -- qmm_kernel_supported says which shapes; the TILE variants
 * need K to be a multiple of 128 for 4-bit codes, of 64 for 6- and 8-bit). */
int qmm_small_m_forced(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K,
                       const void* x, const uint32_t* wq, const void* scales,
                       const void* biases, void* y, void* stream, int kernel_id);

/*
 * K split across workgroups, for the shapes with few column tiles per CU
 * (the batched-decode down projection: N = 4096, K = 14336).  A split-free
 * kernel makes every CU read the whole activation matrix (M*K*2 bytes) for
 * its columns; with K split S ways a CU reads 1/S of it.  The partial
 * outputs (fp32, [S][M][N]) go to a caller-provided workspace and a second
 * kernel adds them in split order and rounds once, so results stay
 * deterministic.  This splits K the way MLX issue #4720 ("Describe the bug")
 * describes qmm_splitk; there it is the slow path on Apple parts, here it is
 * taken only where it measured faster.
 *
 * qmm_small_m_workspace_bytes: bytes qmm_small_m_ws needs for this problem
 * (0: it runs split-free, exactly as qmm_small_m), or a negative status.
 * Pure host logic.
 *
 * qmm_small_m_ws: as qmm_small_m, with `workspace` caller-owned device
 * memory of `workspace_bytes` >= qmm_small_m_workspace_bytes(...) bytes,
 * 16-byte aligned (may be NULL when that is 0).  The workspace is
 * overwritten by the call and must not alias x, wq, scales, biases or y;
 * two calls in flight at once need two workspaces.  Too small or NULL when
 * needed -> QMM_ERR_INVALID_ARG; misaligned -> QMM_ERR_MISALIGNED.  Nothing
 * is allocated.
 *
 * qmm_small_m_split_forced: the same with the variant and split forced
 * (measurement and tests).  split >= 1.  split > 1 with a TILE variant is
 * reduced to the largest count that gives every split part of K; with
 * QMM_KERNEL_MFMA_REG (4-bit; above 16 rows on 16-row blocks) K must be
 * exactly `split` slices of a depth that variant covers split-free
 * (K/split in {2048, 4096} with group sizes whose scale rows split evenly),
 * with more 16-column tiles than 256 / (split x row blocks), else
 * QMM_ERR_UNSUPPORTED -- that is how it runs K it cannot take whole.  The
 * workspace must hold that many [M][N] fp32 outputs.
 *
 * qmm_split_plan: the variant and split qmm_small_m_ws uses.  Pure host
 * logic.
 */
int64_t qmm_small_m_workspace_bytes(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K);
int qmm_small_m_ws(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K,
                   const void* x, const uint32_t* wq, const void* scales,
                   const void* biases, void* y, void* workspace, int64_t workspace_bytes, void* stream);
int qmm_small_m_split_forced(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K,
                             const void* x, const uint32_t* wq, const void* scales,
                             const void* biases, void* y, void* workspace, int64_t workspace_bytes,
                             void* stream, int kernel_id, int split);
int qmm_split_plan(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K,
                   int* kernel_id, int* split);

/*
 * For callers that cannot allocate device memory (code under HIP stream or
 * graph capture, serving loops and harnesses that forbid hipMalloc):
 * exactly qmm_small_m_ws -- the same plan, kernels and results -- with the
 * workspace in a library-owned static device array of
 * QMM_NOALLOC_SCRATCH_BYTES per GPU instead of a caller buffer.  Nothing is
 * allocated by the call (the array is part of the loaded library; each GPU
 * the library runs on holds its own copy until the process ends; its
 * address is looked up once per device, at the first call on it).
 *   - A problem whose planned workspace (qmm_small_m_workspace_bytes)
 *     exceeds QMM_NOALLOC_SCRATCH_BYTES -> QMM_ERR_UNSUPPORTED, checked
 *     before any HIP call; use qmm_small_m_ws with a caller buffer there.
 *   - Every call on one GPU shares that GPU's array, which keeps the last
 *     call's partial sums: calls that overlap on one GPU (two streams, two
 *     threads) race and must be ordered by the caller.  Sequential calls
 *     need no clearing (each split overwrites the partials it reads).
 * Otherwise as qmm_small_m.
 */
#define QMM_NOALLOC_SCRATCH_BYTES (8 * 1024 * 1024)
int qmm_small_m_noalloc(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K,
                        const void* x, const uint32_t* wq, const void* scales,
                        const void* biases, void* y, void* stream);

/* The variant qmm_small_m runs for this problem (a qmm_kernel value), or a
 * negative status if the problem is not supported.  Pure host logic.  The
 * selection is a table of measured crossovers over (dt, bits, group size, M,
 * N, K): MLX issue #4720 shows a dispatch keyed on M and N (its qmv cutoff
 * and split_k rule, "Describe the bug") misrouting shapes whose crossover
 * lies elsewhere ("Expected behavior": near M = 6-8 on 4096-class shapes). */
int qmm_select_kernel(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K);

/* 1 if variant `kernel_id` can run this problem, 0 if it cannot, or a
 * negative status if the problem itself is invalid or unsupported.  Pure
 * host logic. */
int qmm_kernel_supported(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K, int kernel_id);

/* uint32 words per packed row: K*bits/32 (-1 for unsupported bits or a K
 * that does not fill whole words). */
int64_t qmm_packed_words(int bits, int64_t K);

/* Hex digest (SHA-256, first 16 digits) of the source files this library
 * was built from, or "unknown" for a build that did not record it; callers
 * compare it with the sources they ship to detect a stale binary. */
const char* qmm_build_digest(void);

/* Static description of a status code. */
const char* qmm_strerror(int status);

/* Static name of a kernel variant ("?" if unknown). */
const char* qmm_kernel_name(int kernel_id);

/*
 * Measurement helpers (not part of the matmul path).
 *
 * qmm_probe_stream_read: read `bytes` (a multiple of 16) from device memory
 * `src` with coalesced 16-byte nontemporal loads and discard the data, in
 * one of two shapes: `shape` 0, a grid-stride loop over `grid` workgroups of
 * 256 threads (0 = 2048), four loads in flight per thread; `shape` 1, each
 * wavefront reading whole 8 KiB chunks (8 loads of 1 KiB in flight) in
 * `grid` workgroups of 1024 threads (0 = 512).  Never more workgroups than
 * the data needs; another shape -> QMM_ERR_INVALID_ARG.
 * `sink` is caller-owned device memory of at least 256 uint32 that the
 * kernel may write (practically never does).  It is the streaming-read
 * ceiling a matmul streaming the same bytes can approach.
 *
 * qmm_probe_copy: copy `bytes` (a multiple of 16) from `src` to `dst`
 * (device memory, not overlapping).  It reads and writes exactly `bytes`
 * each, so hardware byte counters taken on it give their scale.
 *
 * Both: 16-byte aligned pointers (QMM_ERR_MISALIGNED otherwise), negative
 * sizes -> QMM_ERR_INVALID_ARG, other sizes -> QMM_ERR_UNSUPPORTED, 0 bytes
 * -> QMM_OK with nothing launched; asynchronous on `stream` like the rest.
 */
int qmm_probe_stream_read(const void* src, int64_t bytes, uint32_t* sink, int grid, int shape, void* stream);
int qmm_probe_copy(const void* src, void* dst, int64_t bytes, void* stream);

/*
 * qmm_probe_small_m_loop: `passes` times over `count` weight sets, one
 * qmm_small_m call each (x, y and the formats shared), issued back to back
 * from this C loop on `stream`: the stream-launched rate of the matmul with
 * no interpreter between the calls.  `wq`, `scales`, `biases` are HOST
 * arrays of `count` device pointers (caller-owned, read during the call
 * only).  Stops at the first call that fails and returns its status;
 * count < 0, passes < 0 or a NULL pointer array -> QMM_ERR_INVALID_ARG;
 * count or passes 0 -> QMM_OK with nothing launched.
 */
int qmm_probe_small_m_loop(int dt, int bits, int group_size, int64_t M, int64_t N, int64_t K, const void* x,
                           const uint32_t* const* wq, const void* const* scales, const void* const* biases, void* y,
                           int count, int passes, void* stream);

/* ---------------------------------------------------------------------------
 * Paged K/V cache held in 4 bits, and attention over it.
 *
 * What a decoder keeps next to the products above: the keys and values of
 * the tokens so far, quantized with qmm_quantize's rule at 4 bits (one scale
 * and one bias of dtype dt per token, kv head and group of group_size
 * consecutive values), in pages of page_size tokens.
 *
 * The pool is one dense array [layers][pages][kv_heads] of records, one
 * record of page_size * (head_dim + 8 * head_dim / group_size) bytes per page
 * of one layer and head.  With PS = page_size, D = head_dim, G = D / gs, a
 * record holds in this order (words are uint32):
 *   K codes  [PS][4][D/32] words        word (t, j, s): values d = 32 s + 8 j
 *            + e of token t, value e in bits 4e..4e+3 (a row's 16-byte pieces
 *            are the matrix-core operand of one lane)
 *   V codes  [PS/4][16][2][D/64] words  word (u, i, p, c): token 4u + 2p in
 *            the low half, 4u + 2p + 1 in the high half, each with the values
 *            d = 64 c + 16 n + i in bits 4n..4n+3, n = 0..3
 *   K s, b   [PS/4][G][2][4] values     (u, g): the scales of tokens
 *            4u..4u+3, then their biases
 *   V s, b   the same
 *
 * Sequences: `tables` [seqs][table_width] (int32, dense) names the pages of
 * each sequence in order, entries not in use negative; `lens` [seqs] (int32)
 * is its length in tokens.  Position t of sequence b lies in slot
 * t % PS of page tables[b][t / PS].  `refs` [pages] (int32) counts the
 * sequences that hold each page (0: free).  Tables, lengths and counts live
 * in device memory and are read when the kernels run, so that steps can be
 * captured in a graph.
 *
 * New tokens of a call: `rows` in all, dense over the sequences.  With
 * starts == NULL every sequence has max_new of them (rows = seqs * max_new);
 * else starts [seqs + 1] (int32, device) are the first rows of the
 * sequences, at most max_new each.  lens counts them in: row i of sequence b
 * with n new tokens is position lens[b] - n + i.
 *
 * A row of a table has room for at most 2^30 tokens (table_width * page_size;
 * QMM_ERR_UNSUPPORTED otherwise).
 *
 * Every page id, length, start and sequence number read from device memory
 * is checked against the sizes given here before it becomes an address: a
 * position whose table entry names no page of the pool, or that lies outside
 * the table, is skipped by qmm_kv_append, reads as zeros from qmm_kv_read and
 * is not attended to.
 * ------------------------------------------------------------------------- */
typedef struct qmm_kv_cache {
    int32_t dt;          /* qmm_dtype of scales, biases, q, k, v and outputs */
    int32_t group_size;  /* 32, 64 or 128, at most head_dim */
    int32_t head_dim;    /* 64, 128 or 256 */
    int32_t kv_heads;    /* 1..65535 */
    int32_t page_size;   /* 32, 64, 128 or 256 tokens */
    int32_t layers;      /* 1..65535 */
    int64_t pages;       /* 0..2^30 */
    void* pool;          /* 16-byte aligned device memory */
} qmm_kv_cache;

/* Bytes of one record, or a negative status for an unsupported geometry
 * (pool is not looked at).  A pool takes layers * pages * kv_heads records. */
int64_t qmm_kv_record_bytes(const qmm_kv_cache* cache);

/*
 * Quantize the new tokens' keys and values into `layer` of the cache.
 * k, v: dt, element (row, head, d) at row * stride_row + head * stride_head
 * + d; base 16-byte aligned, strides (in elements, >= 0) multiples of 8.
 * Bit-exact: the codes, scales and biases are qmm_quantize's; but a group that
 * holds a NaN gets a NaN scale and bias, and reads back as NaN.  Other tokens'
 * slots of the same pages are not touched.
 */
int qmm_kv_append(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                  const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts,
                  const void* k, int64_t k_stride_row, int64_t k_stride_head,
                  const void* v, int64_t v_stride_row, int64_t v_stride_head, void* stream);

/*
 * Dequantize the new tokens' (the last n of each sequence) keys and values
 * out of `layer`: k, v [rows][kv_heads][head_dim] (dense), RNE_dt(s*q + b) as
 * qmm_dequantize.  The whole of a sequence: all its tokens as new ones.
 */
int qmm_kv_read(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts,
                void* k, void* v, void* stream);

/*
 * Attention of the new tokens over `layer` of the cache (which already holds
 * them): out [rows][heads][head_dim] (dt, dense) and, unless NULL, lse
 * [rows][heads] (fp32, natural logarithm of the sum of exponentials).
 *   - heads is a multiple of kv_heads; heads h*heads/kv_heads .. share kv
 *     head h.  1 <= max_new <= 64.
 *   - q as k in qmm_kv_append, of values below 2^105 in size.  Scores are
 *     scale * q . k_hat.
 *   - A row sees every token before its sequence's new ones, and of these
 *     the ones up to itself; with mask (int64 [rows], device) instead the
 *     new tokens j whose bit j is set in the row's word (a draft tree: the
 *     row's own token and its ancestors).
 *   - A row that sees nothing gives zeros and lse = -infinity; one whose scores
 *     are NaN gives NaN for both.
 *   - What a row does not see has no part in it, infinite or NaN as it may be;
 *     infinite or NaN values that it sees reach their group of the output.
 * fp32 accumulation, softmax and sums; k_hat and v_hat are not rounded.  For
 * the second product the probabilities times the scale of their value are
 * rounded to fp16, either dt, in units of their own row and group (11 bits
 * down to 2^-10 of the largest, 2^-21 of it below); for what the biases and
 * 7.5 times the scales add, the probabilities are rounded to dt, and the sum
 * of the rounded ones divides it; one rounding to dt at the end.
 * Deterministic.  Values of V may be of any size; where their scales leave
 * 2^-9..2^4 a call takes about twice as long.
 *
 * max_len: no sequence is longer (1..table_width * page_size); it bounds how
 * many parts the sequences are cut into.  Longer ones are still attended to
 * in whole.
 * workspace: device memory of at least qmm_kv_attend_workspace_bytes(...)
 * bytes, 16-byte aligned (may be NULL when that is 0), not aliasing the
 * other arrays.  Its first QMM_KV_ATTEND_ZEROED_BYTES bytes must be zero
 * before the first call that uses it; every call leaves them zero (calls of
 * any sizes may follow each other on one workspace).  Two calls in flight
 * need two.  Fewer sequences or tokens can need more; no call needs more
 * than QMM_KV_ATTEND_ZEROED_BYTES + 32768 * (head_dim + 4) bytes.
 * heads < 1, or not a multiple of kv_heads, max_new > 64 ->
 * QMM_ERR_UNSUPPORTED.
 */
#define QMM_KV_ATTEND_ZEROED_BYTES 65536
int64_t qmm_kv_attend_workspace_bytes(const qmm_kv_cache* cache, int64_t seqs, int64_t max_new, int64_t rows,
                                      int64_t heads, int64_t max_len);
int qmm_kv_attend(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                  const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts,
                  const void* q, int64_t q_stride_row, int64_t q_stride_head, int64_t heads, float scale,
                  const int64_t* mask, void* out, float* lse, int64_t max_len,
                  void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Attention with a window and sinks: as qmm_kv_attend, but of the tokens that
 * a row would see there, in order of their positions, it sees the last
 * `window` (1 or more) and besides those at positions below `sinks` (0 or
 * more).  A row of a draft tree thus has its own token, its ancestors and as
 * many tokens before the new ones as fill the window.  Tokens count whether
 * or not a page holds them.  Reads the pages of those tokens and no others
 * (with a mask: of the tokens that a row whose word is 0 would see as well,
 * though none may be such a row): table entries of pages that no row sees may
 * be negative.
 * The workspace is qmm_kv_attend's, at least
 * qmm_kv_attend_window_workspace_bytes(...) bytes (the same bound and
 * QMM_KV_ATTEND_ZEROED_BYTES hold; one workspace may serve both calls in
 * turn).  window < 1 or sinks < 0 -> QMM_ERR_INVALID_ARG.
 */
int64_t qmm_kv_attend_window_workspace_bytes(const qmm_kv_cache* cache, int64_t seqs, int64_t max_new, int64_t rows,
                                             int64_t heads, int64_t max_len, int64_t window, int64_t sinks);
int qmm_kv_attend_window(const qmm_kv_cache* cache, int layer, int64_t seqs, int64_t max_new, int64_t rows,
                         const int32_t* tables, int64_t table_width, const int32_t* lens, const int32_t* starts,
                         const void* q, int64_t q_stride_row, int64_t q_stride_head, int64_t heads, float scale,
                         const int64_t* mask, int64_t window, int64_t sinks, void* out, float* lse, int64_t max_len,
                         void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Pages.  All layers move together; ids out of range are skipped.
 *
 * qmm_kv_copy_pages: page dst[i] <- page src[i] for i < n (device int32
 * arrays).  No page may be both a source and a destination, or twice a
 * destination.
 *
 * The next ones keep the bookkeeping.  A sequence holds the pages its row
 * names; `lens` may be cut back by the caller (rejected drafts) as long as
 * no token of a page shared with a fork is written again.
 *
 * qmm_kv_reserve: room for add[s] more tokens of every sequence s < seqs
 * (device int32): missing pages are taken, lens[s] += add[s], ok[s] = 1.
 * A sequence whose pages are not there (or whose row is too short, or
 * add[s] < 0) keeps what it has, ok[s] = 0.
 *
 * qmm_kv_fork: sequence dst[i] becomes a copy of sequence src[i], i < n: it
 * shares the whole pages (refs + 1) and gets a page of its own with a copy
 * of a partly filled last one, in every layer.  dst[i] must hold nothing; no
 * dst may be a src or named twice.  ok[i] = 1, or 0 (and an empty dst) where
 * no page is left or src[i] is not a sound sequence.
 *
 * Both take the free pages lowest first and serve the requests in order: one
 * gets its pages if the free ones suffice for it and all before it.
 *
 * qmm_kv_free: every page that the named sequences hold is given up
 * (refs - 1), their rows are cleared to -1 and their lengths to 0.
 *
 * qmm_kv_compact: the live pages (refs > 0; L of them) move into ids
 * 0..L-1: those at or above L, in order, into the free ones below L, in
 * order.  tables_out and refs_out get tables and refs rewritten for that
 * (they may be tables and refs themselves), live_out[0] = L.  The contents of
 * pages at or above L stay.
 *
 * workspace: qmm_kv_pages_workspace_bytes(cache, n) bytes of device memory,
 * 16-byte aligned, for reserve (n = seqs), fork (n) and compact (n = 0).
 */
int64_t qmm_kv_pages_workspace_bytes(const qmm_kv_cache* cache, int64_t n);
int qmm_kv_copy_pages(const qmm_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t n, void* stream);
int qmm_kv_reserve(const qmm_kv_cache* cache, int64_t seqs, int32_t* tables, int64_t table_width, int32_t* lens,
                   int32_t* refs, const int32_t* add, int32_t* ok, void* workspace, int64_t workspace_bytes,
                   void* stream);
int qmm_kv_fork(const qmm_kv_cache* cache, int64_t seqs, int32_t* tables, int64_t table_width, int32_t* lens,
                int32_t* refs, const int32_t* src, const int32_t* dst, int64_t n, int32_t* ok, void* workspace,
                int64_t workspace_bytes, void* stream);
int qmm_kv_free(const qmm_kv_cache* cache, int64_t seqs, int32_t* tables, int64_t table_width, int32_t* lens,
                int32_t* refs, const int32_t* which, int64_t n, void* stream);
int qmm_kv_compact(const qmm_kv_cache* cache, int64_t seqs, const int32_t* tables, int64_t table_width,
                   const int32_t* refs, int32_t* tables_out, int32_t* refs_out, int32_t* live_out, void* workspace,
                   int64_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * What lies between the products and the cache in a decoder's step: the gated
 * block, rotary positions, log probabilities.  Arrays and types as above
 * unless said; every call may be captured in a graph.
 * ------------------------------------------------------------------------- */

/*
 * Gated block: h [M, F] = act(x . Wg^T) * (x . Wu^T) with W = [Wg; Wu]
 * (dequantized) of wq [2F, K*bits/32], scales, biases [2F, K/gs]: the gate's
 * rows first, as one qmm_quantize of both leaves them.  Both products,
 * accumulated in fp32, go through the activation in fp32; h is rounded once.
 * K obeys qmm_small_m's rules, up to 2^24, F is any; 1 <= M <= 64.  Deterministic.
 * Statuses as qmm_small_m (M == 0 or F == 0: QMM_OK, nothing launched); an
 * unknown act -> QMM_ERR_UNSUPPORTED.
 */
enum qmm_act {
    QMM_ACT_SILU = 0,
    QMM_ACT_GELU = 1,       /* a Phi(a), by the error function */
    QMM_ACT_GELU_TANH = 2,  /* its form by tanh */
    QMM_ACT_RELU = 3        /* slope 0 at 0 */
};
int qmm_gated(int dt, int bits, int group_size, int act, int64_t M, int64_t F, int64_t K, const void* x,
              const uint32_t* wq, const void* scales, const void* biases, void* h, void* stream);

/*
 * Its gradient for given (constant) weights: with g, u the two products, formed
 * again, and grad [M, F] that of h,
 *   grad_gate_up [M, 2F] = [grad * u * act'(g), grad * act(g)]
 *   grad_x [M, K]        = grad_gate_up . W
 * grad_gate_up is rounded once to dt; grad_x is formed from its fp32 values,
 * kept to 16 bits, and rounded once.  F a multiple of 16 (QMM_ERR_UNSUPPORTED
 * otherwise); with F == 0 grad_x is zero and the only array looked at (M == 0:
 * QMM_OK, nothing launched).
 * workspace: device memory of at least qmm_gated_backward_workspace_bytes(...)
 * bytes (a negative status for what is not supported), 16-byte aligned, not
 * aliasing the other arrays; two calls in flight need two.
 */
int64_t qmm_gated_backward_workspace_bytes(int dt, int bits, int group_size, int64_t M, int64_t F, int64_t K);
int qmm_gated_backward(int dt, int bits, int group_size, int act, int64_t M, int64_t F, int64_t K, const void* x,
                       const uint32_t* wq, const void* scales, const void* biases, const void* grad,
                       void* grad_gate_up, void* grad_x, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Rotary positions: out = x [rows][heads][head_dim] with the pairs p <
 * rotary_dim / 2 of every head of row r turned by positions[axis(p)][r] *
 * freq[p]:
 *   (a, b) -> (scale * (a cos - b sin), scale * (b cos + a sin)),
 * by minus the angle with inverse != 0 (which is the gradient's map); values
 * behind rotary_dim stay as they are.  A pair is (p, p + rotary_dim / 2)
 * with QMM_PAIRS_HALVES, (2p, 2p + 1) with QMM_PAIRS_ADJACENT.
 *   - axes 1..4; sections (host, [axes]; may be NULL with one axis) are the
 *     numbers of consecutive pairs of each axis, rotary_dim / 2 together.
 *   - positions: int32, or int64 with positions_64 != 0, [axes][rows], the
 *     axes position_stride elements apart; any values (angles are formed in
 *     fp64, to 2^-51 of themselves).  freq: fp32 [rotary_dim / 2], radians.
 *   - head_dim a multiple of 8 up to 1024, rotary_dim a multiple of 16 up to
 *     head_dim (QMM_ERR_UNSUPPORTED otherwise).
 *   - x, out: element (row, head, d) at row * stride_row + head * stride_head
 *     + d; bases 16-byte aligned, strides (elements, >= 0) multiples of 8.
 *     out may be x with the same strides; no two places of out may overlap
 *     (QMM_ERR_INVALID_ARG).
 */
enum qmm_pairs { QMM_PAIRS_HALVES = 0, QMM_PAIRS_ADJACENT = 1 };
int qmm_rotary(int dt, int64_t rows, int64_t heads, int64_t head_dim, int64_t rotary_dim, int pairs, int inverse,
               float scale, const void* x, int64_t x_stride_row, int64_t x_stride_head, const void* positions,
               int positions_64, int64_t position_stride, int axes, const int32_t* sections, const float* freq,
               void* out, int64_t out_stride_row, int64_t out_stride_head, void* stream);

/*
 * Log probabilities of rows of logits [rows][vocab] (dt; row r at r * stride
 * elements, stride >= 0, any alignment of 2 bytes), z = scale * logit, scale
 * finite and above 0 (QMM_ERR_INVALID_ARG otherwise), 2^-100 to 2^100
 * (QMM_ERR_UNSUPPORTED otherwise):
 *   lse [rows]                 ln sum_v exp z_v
 *   entropy [rows]             -sum_v p_v ln p_v (nats), p_v = exp(z_v - lse)
 *   token_logprobs [rows][given]  z_t - lse of tokens [rows][given] (int32, or
 *                              int64 with tokens_64 != 0); 0 where t lies
 *                              outside 0..vocab-1 (padding)
 *   top_logprobs, top_ids [rows][top]  the `top` likeliest, likeliest first,
 *                              of equal logits the lowest id
 * all fp32, ids int64.  given 0..64 and top 0..min(64, vocab)
 * (QMM_ERR_UNSUPPORTED otherwise; arrays of none may be NULL).
 * Logits may be -infinity (barred): probability 0, log probability -infinity.
 * A row of nothing else has lse and log probabilities -infinity and entropy
 * 0.  A row with NaN or +infinity has NaN for all and ids of -1.  |z| of
 * finite logits is to stay below 2^127.
 * Deterministic.
 * workspace: QMM_LOG_PROBS_WORKSPACE_BYTES of device memory, 16-byte aligned,
 * whose first QMM_LOG_PROBS_ZEROED_BYTES are zero before the first call that
 * uses it; every call leaves them zero (calls of any sizes may follow each
 * other on one workspace, two in flight need two).  It may be NULL where
 * qmm_log_probs_needs_workspace(rows, vocab) is 0 (1: needed, or a negative
 * status).
 */
#define QMM_LOG_PROBS_MOST_TOP 64
#define QMM_LOG_PROBS_ZEROED_BYTES 65536
#define QMM_LOG_PROBS_WORKSPACE_BYTES (65536 + 1024 * 66 * 8)
int qmm_log_probs_needs_workspace(int64_t rows, int64_t vocab);
int qmm_log_probs(int dt, int64_t rows, int64_t vocab, float scale, const void* logits, int64_t stride,
                  const void* tokens, int tokens_64, int64_t given, int64_t top, float* lse, float* entropy,
                  float* token_logprobs, float* top_logprobs, int64_t* top_ids, void* workspace,
                  int64_t workspace_bytes, void* stream);

/*
 * Its gradient, with lse and entropy as qmm_log_probs left them: of
 *   sum grad_tokens * token_logprobs + grad_entropy * entropy + grad_lse * lse
 * for the logits, out [rows][vocab] (dt, rounded once; row r at r * out_stride
 * elements, out_stride >= vocab).  Each of the three may be NULL (entropy too
 * without grad_entropy).  A token named twice counts twice; padding has no
 * part.  Rows whose lse is -infinity get zeros.  out may be logits with the
 * same stride.  Probabilities are exp(z_v - lse), so that they share the fp32
 * rounding of z and lse: within 2^-23 (|z_v| + |lse|) of themselves.
 */
int qmm_log_probs_backward(int dt, int64_t rows, int64_t vocab, float scale, const void* logits, int64_t stride,
                           const void* tokens, int tokens_64, int64_t given, const float* lse, const float* entropy,
                           const float* grad_tokens, const float* grad_entropy, const float* grad_lse, void* out,
                           int64_t out_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
