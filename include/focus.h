/*
 * focus.h -- C ABI of libfocus.so, the B200 (sm_100a) implementation of the
 * Focus-dLLM sparse denoising-step attention.
 *
 * Source of the operations: "Focus-dLLM: Accelerating Long-Context Diffusion LLM
 * Inference via Confidence-Guided Context Focusing" (summary page of arXiv
 * 2602.02159), section "方法步骤详情" (method steps) steps (1)-(5), and section
 * "核心方法" (core method). At a block-entry step the whole sequence runs dense
 * attention; at every other step:
 *   (1) PCGI picks the top-k still-[MASK] positions by the previous step's
 *       confidence, k = floor(rho * n(t))                     -> focus_select_queries
 *   (2) each is widened to a window of size w -> I_active     -> focus_select_queries
 *   (3) the first layers run full attention; the attention distribution of the
 *       sink layer picks the attention sinks                   -> focus_dense_attention,
 *                                                                focus_sink_identify
 *   (4) prompt blocks are represented by their mean key, scored against the
 *       active queries, and the top-C kept                     -> focus_block_means,
 *                                                                focus_block_select
 *   (5) the active queries attend over I_p = sinks U kept blocks U current block
 *                                                              -> focus_sparse_attention
 *
 * Conventions shared by every call:
 *   - Every pointer is a DEVICE pointer unless stated otherwise. The caller owns all
 *     memory (tensors and workspace); the library allocates nothing.
 *   - bf16 tensors are passed as `focus_bf16` (raw IEEE bfloat16 bits).
 *   - Layouts are dense row-major: K, V [B, Hkv, L, d]; Q [B, Hq, qcap, d];
 *     query head hq uses KV head hq / (Hq / Hkv).
 *   - `stream` is a cudaStream_t (NULL = legacy default stream). Every call only
 *     enqueues work on it and never synchronises the host; counts (n_focus,
 *     n_active) stay on the device.
 *   - Every call returns a focus_status. Arguments are validated before any launch;
 *     an invalid call launches nothing and returns FOCUS_ERR_INVALID_ARG (or
 *     FOCUS_ERR_UNSUPPORTED / FOCUS_ERR_CAPACITY) with a message in
 *     focus_last_error(). A failed launch returns FOCUS_ERR_CUDA.
 *   - Index outputs are sorted ascending; unused tail slots hold -1.
 *   - Every top-k orders by (score descending, index ascending): ties go to the
 *     lower index and -0.0 equals +0.0. Scores must be finite.
 *   - A kernel wait that runs out (2 s) records a code in the device error word
 *     (read it with focus_device_error) and the kernel returns early; outputs of
 *     that call are then undefined.
 */
#ifndef FOCUS_H_
#define FOCUS_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(FOCUS_BUILD) && defined(__GNUC__)
#define FOCUS_API __attribute__((visibility("default")))
#else
#define FOCUS_API
#endif

typedef uint16_t focus_bf16;

typedef enum {
  FOCUS_OK = 0,
  FOCUS_ERR_INVALID_ARG = -1,
  FOCUS_ERR_UNSUPPORTED = -2,
  FOCUS_ERR_CUDA = -3,
  FOCUS_ERR_CAPACITY = -4,
  FOCUS_ERR_DEVICE_CHECK = -5
} focus_status;

/* Human-readable name of a status code. Never NULL. */
FOCUS_API const char* focus_status_string(int status);

/* Message of the last failing call on this host thread ("" if none). Never NULL. */
FOCUS_API const char* focus_last_error(void);

/* Number of kernels this library has launched in this process (all threads). */
FOCUS_API uint64_t focus_launch_count(void);

/* Synchronises the current device, copies the device error word to *code_out (0 = no
 * error) and clears it. Returns FOCUS_ERR_DEVICE_CHECK if the word was set. */
FOCUS_API int focus_device_error(int* code_out);

/*
 * (1)+(2) PCGI and window expansion -- method steps (1) and (2).
 * conf_prev [B, G] fp32, G = g1 - g0: c_{t-1} of position g0 + j at conf_prev[b, j].
 * mask [B, L] uint8, nonzero = still [MASK]. Candidates: masked positions of the current
 * block [g0, g1). k = min(floor(rho * n_t), #candidates); I_focus = the top-k candidates
 * by conf. Each p in I_focus becomes [p - w/2, p - w/2 + w - 1] clipped to [g0, g1);
 * I_active = the sorted union.
 * Outputs: i_focus [B, kcap], n_focus [B], i_active [B, acap], n_active [B] (int32).
 * Requires 0 <= g0 < g1 <= L, G <= 1024, n_t >= 0, rho >= 0, w >= 1,
 * kcap >= min(floor(rho*n_t), G), acap >= min(G, kcap * w) (else FOCUS_ERR_CAPACITY).
 */
FOCUS_API int focus_select_queries(const float* conf_prev, const uint8_t* mask, int B, int L, int g0, int g1, int n_t,
                         float rho, int w, int32_t* i_focus, int32_t* n_focus, int kcap, int32_t* i_active,
                         int32_t* n_active, int acap, void* stream);

/*
 * Gathers rows of a stack of head-major matrices by per-batch row lists (the queries of
 * the active positions). X [n_mat, B, H, L, d] -> X_rows [n_mat, B, H, cap, d] with
 * X_rows[m, b, h, i] = X[m, b, h, rows[b, i]] for i < n_rows[b], zero otherwise.
 * rows [B, cap] and n_rows [B] int32 (device). Row indices outside [0, L) are written
 * as zero rows and flagged in the device error word (code 5).
 */
FOCUS_API int focus_gather_rows(const focus_bf16* X, const int32_t* rows, const int32_t* n_rows, int n_mat, int B, int H,
                      int L, int d, int cap, focus_bf16* X_rows, void* stream);

/*
 * Approximate-KV-cache refresh (Focus-dLLM summary page, "近似KV缓存" / approximate KV
 * cache: a token of the refresh set U(t) takes its recomputed key and value, every other
 * token keeps its cached one). The inverse of focus_gather_rows: for every matrix m,
 * X[m, b, h, rows[b, i]] = X_rows[m, b, h, i] for i < n_rows[b]; all other rows of X are
 * left unchanged. X [n_mat, B, H, L, d] (the K or V cache of n_mat layers, updated in
 * place), X_rows [n_mat, B, H, cap, d], rows [B, cap] and n_rows [B] int32 (device), e.g.
 * I_active (or I_focus) from focus_select_queries. Row lists must not repeat a row (the
 * selection outputs are ascending and unique). Indices outside [0, L) are skipped and
 * flagged in the device error word (code 5). d a multiple of 8; X and X_rows 16-byte
 * aligned. The pages have no fused form of this step; it runs as one scatter launch.
 */
FOCUS_API int focus_scatter_rows(focus_bf16* X, const int32_t* rows, const int32_t* n_rows, int n_mat, int B, int H,
                                 int L, int d, int cap, const focus_bf16* X_rows, void* stream);

/*
 * (4a) Block representative keys -- method steps (4): the prompt [0, P) is cut into
 * nb = ceil(P / bs) contiguous blocks; kbar[b, h, j] = mean of K[b, h, j*bs : min(P,(j+1)*bs)].
 * K [B, Hkv, L, d] bf16 -> kbar [B, Hkv, nb, d] fp32. Requires 1 <= P <= L, bs >= 1,
 * d in {64, 128}, K 16-byte aligned.
 */
FOCUS_API int focus_block_means(const focus_bf16* K, int B, int Hkv, int L, int d, int P, int bs, float* kbar,
                      void* stream);

/*
 * (4b) Block relevance and top-C -- method steps (4).
 * R[b, h, j] = mean over the n_active[b] active queries and the Hq/Hkv query heads of
 * KV group h of q . kbar[b, h, j] / sqrt(d) (0 when n_active[b] == 0).
 * blocks[b, h, :] = the top-min(C, nb) blocks, ascending, -1 tail.
 * Q_active [B, Hq, acap, d] bf16; n_active [B]; kbar [B, Hkv, nb, d] fp32;
 * scores_opt: NULL or [B, Hkv, nb] fp32 receiving R. Requires nb <= 49152, C >= 1,
 * d in {64, 128}.
 */
FOCUS_API int focus_block_select(const focus_bf16* Q_active, const int32_t* n_active, const float* kbar, int B, int Hq,
                       int Hkv, int d, int acap, int nb, int C, int32_t* blocks, float* scores_opt,
                       void* stream);

/*
 * (3) Dense bidirectional attention -- method steps (3) and the block-entry full refresh.
 * For query i < n_q[b] (all qcap rows when n_q == NULL) of head hq:
 *   O[b, hq, i] = softmax_j(scale * q_i . k_j) V over all L keys (fp32 accumulation).
 * Rows i >= n_q[b] of O are written as zero.
 * colsum_opt: NULL, or [B, Hkv, L] fp32 receiving the sink importance
 *   colsum[b, h, j] = sum over the group's query heads and the valid queries of p_ij
 *   (requires (Hq/Hkv) * qcap <= 256).
 * ws/ws_bytes: device workspace of at least focus_dense_workspace_bytes(...) bytes,
 *   256-byte aligned (may be NULL when that size is 0).
 * Requires d in {64, 128}, Hq % Hkv == 0, L >= 8, Q/K/V/O 16-byte aligned.
 */
FOCUS_API int focus_dense_attention(const focus_bf16* Q, const int32_t* n_q, const focus_bf16* K, const focus_bf16* V,
                          int B, int Hq, int Hkv, int L, int d, int qcap, float scale, focus_bf16* O,
                          float* colsum_opt, void* ws, size_t ws_bytes, void* stream);

FOCUS_API size_t focus_dense_workspace_bytes(int B, int Hq, int Hkv, int L, int d, int qcap, int want_colsum);

/*
 * Block entry in one call -- "半自回归重遮蔽策略" (semi-AR remasking: at block entry the whole
 * sequence runs dense attention) and method steps (4) (a prompt block is represented by the
 * mean of its keys, computed once per generation block): O = dense attention of all L
 * queries of Q [B, Hq, L, d] over all L keys (as focus_dense_attention with n_q = NULL,
 * qcap = L) and kbar [B, Hkv, nb, d] fp32 = the block means of the prompt [0, P) in blocks of
 * bs (as focus_block_means). Where the many-row kernel serves the shape (d = 128, enough
 * 256-row blocks to fill the GPU) and bs divides 128, the block means are summed from the K
 * tiles the attention streams anyway: one launch, no second read of K. Otherwise the two
 * calls run in sequence; ws/ws_bytes then serve the dense attention (size them with
 * focus_dense_workspace_bytes(B, Hq, Hkv, L, d, L, 0)). Requires 1 <= P <= L, bs >= 1,
 * kbar 16-byte aligned and the conditions of focus_dense_attention.
 */
FOCUS_API int focus_full_refresh(const focus_bf16* Q, const focus_bf16* K, const focus_bf16* V, int B, int Hq,
                                 int Hkv, int L, int d, float scale, focus_bf16* O, int P, int bs, float* kbar,
                                 void* ws, size_t ws_bytes, void* stream);

/*
 * (3) The sink layer in one call -- method steps (3) and core method: dense attention of the
 * active queries (as focus_dense_attention), the sink importance colsum [B, Hkv, L] (as its
 * colsum_opt) and the sinks [B, Hkv, S] = top-min(S, L) columns of colsum per KV head,
 * ascending, -1 tail (as focus_sink_identify). Where the few-query kernel serves the shape
 * (d = 128, (Hq/Hkv) * qcap <= 64) the attention and the column sums run in one launch:
 * after the cluster merge the kernel re-reads the K tiles, most recently read first, for
 * the column sums. The same launch also selects the sinks within the cluster when
 * S <= 512, S <= L and (CTAs per KV head) x S <= 2048; otherwise the top-S runs as a
 * second launch. Other shapes run the calls in sequence. colsum and sinks are both written in every case. Requires 1 <= S <= 4096
 * and the conditions of focus_dense_attention with column sums; ws/ws_bytes as there.
 */
FOCUS_API int focus_dense_attention_sinks(const focus_bf16* Q, const int32_t* n_q, const focus_bf16* K,
                                          const focus_bf16* V, int B, int Hq, int Hkv, int L, int d, int qcap,
                                          float scale, focus_bf16* O, float* colsum, int S, int32_t* sinks, void* ws,
                                          size_t ws_bytes, void* stream);

/*
 * (3) Sink identification -- core method / method steps (3): the attention distribution
 * of the sink layer, aggregated over the active queries, picks the S sinks per KV head,
 * reused by every deeper sparse layer. sinks[b, h, :] = top-min(S, L) of colsum[b, h, :],
 * ascending, -1 tail. colsum [B, Hkv, L] fp32 -> sinks [B, Hkv, S] int32. Requires
 * 1 <= S <= 4096.
 */
FOCUS_API int focus_sink_identify(const float* colsum, int B, int Hkv, int L, int S, int32_t* sinks, void* stream);

/*
 * (5) Sparse attention -- method steps (5): for each active query (i < n_active[b]) of
 * head hq (KV head h): O_active[b, hq, i] = softmax over I_p of scale * q . k, applied to V,
 * with I_p = sinks[b, h, :] U (blocks [j*bs, min(P, (j+1)*bs)) for j in blocks[b, h, :])
 * U [g0, g1) taken as a SET (a key named twice counts once). Negative entries of
 * sinks/blocks are ignored; entries must otherwise lie in [0, L) and [0, nb). Rows
 * i >= n_active[b] of O_active are written as zero.
 * ws/ws_bytes: at least focus_sparse_workspace_bytes(...) bytes, 256-byte aligned.
 * Requires d in {64, 128}, L >= 8, 0 <= P <= g0 < g1 <= L, bs >= 1, 0 <= S <= 1024,
 * 1 <= C <= 1024, blocks sorted ascending among their valid entries.
 */
FOCUS_API int focus_sparse_attention(const focus_bf16* Q_active, const int32_t* n_active, const focus_bf16* K,
                           const focus_bf16* V, const int32_t* sinks, int S, const int32_t* blocks, int C, int bs,
                           int P, int g0, int g1, int B, int Hq, int Hkv, int L, int d, int acap, float scale,
                           focus_bf16* O_active, void* ws, size_t ws_bytes, void* stream);

/*
 * (4b)+(5) Block relevance, top-C and sparse attention of one layer in a single launch --
 * method steps (4) and (5). Same results as focus_block_select (kept blocks written to
 * blocks [B, Hkv, C], -1 tail) followed by focus_sparse_attention on them. kbar
 * [B, Hkv, nb, d] fp32 with nb = ceil(P / bs). Shapes outside the fused kernel's range
 * (d != 128, more than 256 query rows per KV head, nb > 4096, C > 512 or S > 512) run the
 * two calls in sequence; ws/ws_bytes then serve focus_sparse_attention (size them with
 * focus_sparse_workspace_bytes).
 */
FOCUS_API int focus_sparse_attention_fused(const focus_bf16* Q_active, const int32_t* n_active, const focus_bf16* K,
                                           const focus_bf16* V, const float* kbar, int nb, int C,
                                           const int32_t* sinks, int S, int bs, int P, int g0, int g1, int B, int Hq,
                                           int Hkv, int L, int d, int acap, float scale, int32_t* blocks,
                                           focus_bf16* O_active, void* ws, size_t ws_bytes, void* stream);

FOCUS_API size_t focus_sparse_workspace_bytes(int B, int Hq, int Hkv, int L, int d, int acap, int S, int C, int bs, int P,
                                    int g0, int g1);

/*
 * Allocation-free variant of focus_sparse_attention. The paper has no counterpart: this
 * entry point exists for callers that cannot call cudaMalloc, e.g. code that runs while a
 * stream is being captured in a mode that forbids allocation, plugin hosts whose enqueue
 * path must not allocate, or servers that reserve all device memory up front. It takes the
 * same arguments minus the workspace and computes the same result.
 *
 * Scratch: the split-KV partials live in one library-owned device array of
 * FOCUS_NOALLOC_SCRATCH_BYTES bytes (a static __device__ array: every GPU that loads the
 * library holds it until the process exits). A call whose partials would need more
 * (focus_sparse_workspace_bytes(...) > FOCUS_NOALLOC_SCRATCH_BYTES) returns
 * FOCUS_ERR_CAPACITY and launches nothing. The call allocates nothing.
 * The first call on a device looks the array's device address up (cudaGetSymbolAddress,
 * with that device current) and caches it per device ordinal; make that first call before
 * any stream capture. The cached address is only valid for the device context it was
 * taken in: after a cudaDeviceReset (or any other teardown of the primary context) it is
 * stale, and this entry point must not be called again in that process.
 * All calls share the array and it keeps the previous call's contents; every element a
 * call reads is written earlier by the same call, so nothing has to be cleared (a split
 * whose kernel gave up on a timed-out wait marks its partial empty). Calls that overlap
 * on the GPU (e.g. on two streams without ordering) race on the array. After a call that
 * leaves the device error word set (focus_device_error), its output is undefined.
 */
#define FOCUS_NOALLOC_SCRATCH_BYTES ((size_t)8 << 20)

FOCUS_API int focus_sparse_attention_noalloc(const focus_bf16* Q_active, const int32_t* n_active,
                                             const focus_bf16* K, const focus_bf16* V, const int32_t* sinks, int S,
                                             const int32_t* blocks, int C, int bs, int P, int g0, int g1, int B,
                                             int Hq, int Hkv, int L, int d, int acap, float scale,
                                             focus_bf16* O_active, void* stream);

/*
 * ---------------------------------------------------------------- 8-bit paged cache
 * The approximate KV cache (Focus-dLLM summary page, "近似KV缓存") held in 8 bits, in pages of
 * `page` positions that sequences can share. The pages describe a cache of the model's own
 * type only; this form halves the bytes that an attention over it reads.
 *
 * Codes k, v [n_mat, n_pages, Hkv, page, d] (n_mat layers) with one fp32 scale for each
 * layer, page and head, k_scale, v_scale [n_mat, n_pages, Hkv]: an element stands for
 * code * scale. format FOCUS_CACHE_E4M3 (e4m3 floats, top = 448) or FOCUS_CACHE_INT8
 * (two's complement, top = 127). A page's scale is s = max|x| / top over the rows written to
 * it, a code the nearest (ties to even) to x / s, both divisions rounded in fp32; s = 0 (a
 * page of zeros) gives codes 0. Values must be finite: a NaN or an infinity makes the scale
 * of its page and head NaN or infinite, and what reads that page NaN.
 * The attention's products of codes are scaled in fp32: keys below 2^106 and values below 2^64 in
 * magnitude stay finite on the way, and scores may be of any finite size. Of int8, a row of
 * queries whose largest is below 1e-30 counts as a row of zeros.
 *
 * table [B, table_cols] int32 (device): page table[b, j] holds the positions
 * [j * page, (j + 1) * page) of sequence b. Entries that a call needs must lie in
 * [0, n_pages); a position whose entry does not is skipped (not written; not attended;
 * loaded as zeros) and flagged in the device error word (code 5), as are positions behind
 * table_cols * page. A page that a call writes must be named once among the sequences of
 * that call (focus_pages_own gives a sequence its own copies of shared pages).
 *
 * Requires d in {64, 128}, page in {16, 32, 64, 128}, Hkv >= 1, n_pages * Hkv < 2^31,
 * k, v 16-byte aligned, scales 4-byte aligned. The struct lives on the host and is read
 * during the call only; a layer's cache is the struct with its four pointers moved to that
 * layer and n_mat = 1.
 */
typedef enum { FOCUS_CACHE_E4M3 = 0, FOCUS_CACHE_INT8 = 1 } focus_cache_format;

typedef struct {
  void* k;          /* codes [n_mat, n_pages, Hkv, page, d] */
  void* v;
  float* k_scale;   /* [n_mat, n_pages, Hkv] */
  float* v_scale;
  int n_mat, n_pages, Hkv, page, d;
  int format;       /* focus_cache_format */
} focus_cache;

/*
 * Block entry: the keys and values of positions [0, lens[b]) go into the cache, their pages'
 * scales are set anew. K, V [n_mat, B, Hkv, L, d] bf16; lens [B] int32 (device, clamped to
 * [0, L]) or NULL for L. Positions behind lens[b] keep their codes (in the last page, under
 * that page's new scale). One pass: every element is read once and every code written once.
 * Requires n_mat * B <= 65535.
 */
FOCUS_API int focus_cache_store(const focus_bf16* K, const focus_bf16* V, int B, int L, const int32_t* lens,
                                const int32_t* table, int table_cols, const focus_cache* cache, void* stream);

/*
 * The refresh of single rows (as focus_scatter_rows): position rows[b, i] of sequence b takes
 * K_rows[m, b, h, i], V_rows[m, b, h, i] for i < n_rows[b]; K_rows, V_rows
 * [n_mat, B, Hkv, cap, d] bf16, rows [B, cap], n_rows [B] int32 (device), in any order; of a
 * position listed twice the later row stays. lens [B] int32 (device): positions the sequence
 * held before the call. The scale of a page that held any only grows: s' = max(s, max|new| /
 * top); when it does, its other held rows are coded again, the nearest code to
 * (code * s) / s' (product and quotient rounded in fp32). A page that starts at or behind
 * lens[b] held nothing: s' = max|new| / top. Other positions behind lens[b] keep their codes.
 * Negative rows are flagged like positions behind the table. Requires 1 <= cap <= 4096 and
 * n_mat * B * Hkv <= 65535.
 */
FOCUS_API int focus_cache_scatter_rows(const focus_bf16* K_rows, const focus_bf16* V_rows, const int32_t* rows,
                                       const int32_t* n_rows, int B, int cap, const int32_t* lens,
                                       const int32_t* table, int table_cols, const focus_cache* cache, void* stream);

/*
 * Positions [start, min(start + L, lens[b])) of the cache as bf16: K[m, b, h, i] = code * scale
 * of position start + i, rounded once; K, V [n_mat, B, Hkv, L, d]. Rows behind lens[b] are left
 * as they were. start >= 0; lens as in focus_cache_store, but not clamped to L. Requires
 * n_mat * B <= 65535.
 */
FOCUS_API int focus_cache_load(const focus_cache* cache, const int32_t* table, int table_cols, const int32_t* lens,
                               int B, int start, int L, focus_bf16* K, focus_bf16* V, void* stream);

/*
 * (3) Dense attention from the cache (as focus_dense_attention): for i < n_q[b] (all qcap rows
 * when n_q == NULL) of query head hq, O[b, hq, i] = softmax over positions j < lens[b] of
 * scale * q_i . k_j, applied to V, with k_j, v_j the values that the codes stand for. Rows
 * i >= n_q[b], and every row of a sequence with lens[b] <= 0, are written as zero. Q, O
 * [B, Hq, qcap, d] bf16; cache of one layer (n_mat = 1); lens [B] int32 (device).
 * ws/ws_bytes: at least focus_cache_workspace_bytes(...) bytes, 256-byte aligned; two calls
 * that may overlap on the GPU need a workspace each. Requires Hq % Hkv == 0, qcap >= 1,
 * table_cols * page <= 2^31 - 2^18.
 */
FOCUS_API int focus_cache_attention(const focus_bf16* Q, const int32_t* n_q, const focus_cache* cache,
                                    const int32_t* table, int table_cols, const int32_t* lens, int B, int Hq,
                                    int qcap, float scale, focus_bf16* O, void* ws, size_t ws_bytes, void* stream);

/*
 * (5) Sparse attention from the cache (as focus_sparse_attention, each sequence with a prompt
 * length of its own): the key set of (b, h) is sinks[b, h, :] U (blocks [j * page,
 * min(P[b], (j + 1) * page)) for j in blocks[b, h, :]) U [g0[b], g0[b] + G), taken as a SET.
 * P, g0 [B] int32 (device), 0 <= P[b] <= g0[b]; sinks [B, Hkv, S] (NULL when S = 0) and
 * blocks [B, Hkv, C] int32 (device), negative entries ignored, repeated entries counted once,
 * in any order. Requires G >= 1, 0 <= S <= 1024, 1 <= C <= 1024; the rest as above.
 */
FOCUS_API int focus_cache_sparse_attention(const focus_bf16* Q_active, const int32_t* n_active,
                                           const focus_cache* cache, const int32_t* table, int table_cols,
                                           const int32_t* P, const int32_t* g0, int G, const int32_t* sinks, int S,
                                           const int32_t* blocks, int C, int B, int Hq, int qcap, float scale,
                                           focus_bf16* O_active, void* ws, size_t ws_bytes, void* stream);

FOCUS_API size_t focus_cache_workspace_bytes(int B, int Hq, int Hkv, int d, int qcap);

/*
 * Pages of the cache. refs [n_pages]: table entries that name the page, 0 = free;
 * table [n_seq, table_cols]: -1 behind held[s]; held [n_seq]: pages of sequence s (all int32,
 * device). Every call runs on the device without a host round trip (it can be captured);
 * calls on the same pages must be ordered (one stream, or events). Free pages are taken in
 * ascending order, for the listed sequences in the order of the list, so results do not
 * depend on timing. status [1] int32 (device): 0, or the number of pages (or pairs) that are
 * missing; a call that is short of any changes nothing else. Lists hold n <= 1024 entries
 * (n = 0 does nothing). List entries that name no sequence, and table entries that name no
 * page, are skipped and flagged in the device error word (code 5).
 */
typedef struct {
  int32_t* refs;
  int32_t* table;
  int32_t* held;
  int n_pages, n_seq, table_cols;
} focus_pages;

/* Sequences seqs[i] grow to want[i] pages (shorter wants change nothing; a want above
 * table_cols is skipped and flagged). */
FOCUS_API int focus_pages_reserve(const focus_pages* pages, const int32_t* seqs, const int32_t* want, int n,
                                  int32_t* status, void* stream);

/* Sequence dst[i], which holds nothing (else skipped and flagged), shares the first
 * min(keep[i], held) pages of src[i]; in the order of the list. Nothing is copied. */
FOCUS_API int focus_pages_fork(const focus_pages* pages, const int32_t* src, const int32_t* dst, const int32_t* keep,
                               int n, void* stream);

/* Copy on write: pages first[i] <= j < last[i] of sequence seqs[i] that others share are
 * replaced by free pages; pairs[r] = (shared page, own page), r < n_pairs[0], is what
 * focus_pages_copy has to copy. Of a page that every one of its sequences is listed with,
 * the last in the list keeps it. pairs [pair_cap, 2], n_pairs [1]. A call that is short sets
 * n_pairs to 0 and leaves what it has tried in pairs. Requires n * table_cols < 2^31 - 1024. */
FOCUS_API int focus_pages_own(const focus_pages* pages, const int32_t* seqs, const int32_t* first,
                              const int32_t* last, int n, int32_t* pairs, int pair_cap, int32_t* n_pairs,
                              int32_t* status, void* stream);

/* Sequences seqs[i] give up their pages behind the first keep[i] (0: all of them). */
FOCUS_API int focus_pages_release(const focus_pages* pages, const int32_t* seqs, const int32_t* keep, int n,
                                  void* stream);

/* The n live pages move to [0, n): the live pages at or behind n, ascending, into the free
 * ones before n, ascending. pairs [pair_cap, 2] and n_pairs [1] are what focus_pages_copy has
 * to copy; remap [n_pages] = each page's new index, -1 for free ones. refs and the first held
 * entries of the tables follow. pair_cap >= n_pages / 2 (else FOCUS_ERR_CAPACITY). */
FOCUS_API int focus_pages_compact(const focus_pages* pages, int32_t* pairs, int pair_cap, int32_t* n_pairs,
                                  int32_t* remap, void* stream);

/* Codes and scales of page pairs[r, 0] to page pairs[r, 1], r < min(n_pairs[0], pair_cap), in
 * all n_mat layers. No page may be both source and target, or target twice. Pairs outside
 * [0, n_pages) are skipped and flagged. A call of 2^31 pieces of 16 KB, or nearly as many, is
 * refused (FOCUS_ERR_UNSUPPORTED). */
FOCUS_API int focus_pages_copy(const focus_cache* cache, const int32_t* pairs, const int32_t* n_pairs, int pair_cap,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FOCUS_H_ */
