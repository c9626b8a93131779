/*
 * dv.h -- C ABI of the GB300 (sm_103a) contextually sparse decode library
 * (libdv.so).
 *
 * The library computes one decode step of Deja Vu's contextual sparsity:
 * a low-rank predictor picks input-dependent attention heads and MLP
 * neurons, and fused gather-and-multiply kernels compute only those.
 *
 * Pages that define the operations (cited per entry point):
 *   [blog]  "用Deja Vu来提高 LLM 的推理速度" (m.haoling.cc/wenzhang/678872),
 *           §2 稀疏性预测 (sparsity prediction), §3.1 并行化稀疏性预测
 *           (parallel / look-ahead prediction), §3.2 Kernel Fusion,
 *           §3.3 Memory coalescing.
 *   [notes] Deja Vu reading notes (pages.squarehuang.top/paper/DejaVu):
 *           "Sparsified MLP", "Sparsified Attention", "Deja Vu Framework"
 *           (sparsity operators for MLP / attention, KV repair,
 *           "Reducing Overhead with Asynchronous Execution").
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer argument that names a tensor is DEVICE memory owned by
 *    the caller; the library never allocates, frees or keeps a pointer after
 *    the call returns.  Host-side descriptor structs (dv_kv, dv_predictor)
 *    are read during the call only.
 *  - Every compute call is asynchronous on the given stream and can be
 *    captured into a CUDA graph.  The host never reads device data (counts
 *    stay on the device); only dv_check() synchronises.
 *  - Weights, token embeddings and the KV cache share one storage type
 *    `dt` (DV_F32, DV_F16 or DV_BF16); accumulation is fp32.  Outputs of
 *    the sparse blocks are fp32.
 *  - Tensor pointers must be 16-byte aligned and row lengths (d, r, d_h)
 *    multiples of 8 elements (4 for DV_F32); otherwise DV_ERR_INVALID_ARG.
 *  - Index lists are int32, ascending, with their element count held in
 *    device memory; a list has room for `cap` entries per batch row.
 *  - Scratch space: each call takes a caller-owned device workspace of at
 *    least the size its *_workspace_size() query reports.  A workspace must
 *    be zero-filled once (dv_workspace_init) before its first use; the
 *    library leaves it reusable, also after a device wait has timed out
 *    (DV_ERR_TIMEOUT): a late arrival still brings the workspace's counters
 *    back to zero.  A workspace that was never zero-filled reports
 *    DV_ERR_TIMEOUT or DV_ERR_WORKSPACE from dv_check; zero-fill it
 *    (dv_workspace_init) before the next call.  Calls that may run
 *    concurrently (e.g. the look-ahead predictor on a side stream) need
 *    distinct workspaces.
 *  - Errors found on the host (bad arguments) are returned at once and
 *    nothing is launched.  Errors found on the device (an index outside
 *    [0, N), a count above cap, a position outside the cache) never trap:
 *    the offending element is skipped and a code is recorded in the
 *    workspace's error word, which dv_check() returns and clears.
 *
 * Storage layouts (row-major; "rows" are contiguous):
 *    y      [B][d]              token input(s) of a block
 *    P1t    [r][d]              predictor layer 1, row j = column j of P1
 *    P2t    [N][r]              predictor layer 2, row u = column u of P2
 *    W1n    [N][d]              row j = column j of W^1 (neuron j's input)
 *    W2n    [N][d]              row j = column j of W^2 (neuron j's output)
 *    Wqkv   [h][3][d_h][d]      [i][m][t] = column t of W_i^m, m = Q, K, V
 *    Wo     [h][d_h][d]         W_i^O
 *    K, V   [B][h][n_max][d_h]  KV cache, X [B][n_max][d], valid [B][h][n_max]
 */
#ifndef DV_H_
#define DV_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dv_status {
  DV_OK = 0,
  DV_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misalignment, cap < k;
                              device: a row that dv_sample cannot draw from  */
  DV_ERR_DTYPE = 2,        /* unsupported storage / output type            */
  DV_ERR_WORKSPACE = 3,    /* workspace missing or smaller than required   */
  DV_ERR_CUDA = 4,         /* a CUDA call failed: see dv_last_cuda_error() */
  DV_ERR_INDEX_RANGE = 5,  /* device: an index outside [0, N) was skipped  */
  DV_ERR_TIMEOUT = 6,      /* device: a bounded wait gave up               */
  DV_ERR_UNSUPPORTED = 7,  /* shape outside what the kernels support       */
  DV_ERR_CAPACITY = 8,     /* device: a list was longer than cap; truncated */
  DV_ERR_POSITION = 9      /* device: a position outside [0, n_max)        */
} dv_status;

typedef enum dv_dtype { DV_F32 = 0, DV_F16 = 1, DV_BF16 = 2 } dv_dtype;

typedef enum dv_select {
  DV_TOPK = 0,       /* the k units with the largest score; ties -> lower index */
  DV_THRESHOLD = 1   /* every unit with score s > t (strict)                    */
} dv_select;

/* One sparsity predictor ([blog] §2: a two-layer MLP with one sigmoid per
 * head / neuron).  Used by dv_predict and dv_lookahead. */
typedef struct dv_predictor {
  const void* P1t;     /* [r][d], storage type                               */
  const void* P2t;     /* [N][r], storage type                               */
  int r;               /* predictor rank (hidden width)                      */
  int N;               /* units scored: h (heads) or 4d (neurons)            */
  dv_select mode;
  int k;               /* DV_TOPK: units kept per row, 0 <= k <= min(N, cap) */
  float t;             /* DV_THRESHOLD: keep s > t                           */
  int32_t* idx;        /* out [B][cap]: selected units, ascending            */
  int cap;             /* room per row in idx                                */
  int32_t* count;      /* out [B]: entries written per row                   */
  float* scores;       /* out [B][N] fp32 sigmoid scores, or NULL            */
} dv_predictor;

/* Per-layer KV cache of a batch of sequences ([notes] "Sparsity operator
 * for Attention": the cache holds K/V of heads that were computed and the
 * token embedding X of every position, so skipped heads can be repaired). */
typedef struct dv_kv {
  void* K;          /* [B][h][n_max][d_h], storage type                      */
  void* V;          /* [B][h][n_max][d_h], storage type                      */
  void* X;          /* [B][n_max][d], storage type: attention input per pos  */
  uint8_t* valid;   /* [B][h][n_max]: 1 where K/V of (head, pos) are present */
  int n_max;        /* positions per sequence                                */
} dv_kv;

/* A matrix [N][d] in 4 bits with group scales (the pages have no counterpart:
 * their weights are 16 bits wide): w[n][t] = (code[n][t] - 8) scale[n][t / group].
 * A row is ceil(d / 128) blocks of 64 bytes.  The 32-bit word k of a block,
 * g = k / 2 and s = k % 2, holds the codes of the elements 64 s + 8 g + e,
 * e = 0..7, at bit 4 (e / 2) + 16 (e % 2).  What a block holds behind d does not
 * matter (dv_q4_quantize writes 8). */
typedef struct dv_q4 {
  const void* q;      /* [N][64 ceil(d / 128)] bytes                          */
  const void* scale;  /* [N][ceil(d / group)], storage type                   */
  int group;          /* elements that share a scale: 64 or 128               */
} dv_q4;

/* ---------------------------------------------------------------- utility */

const char* dv_status_str(dv_status s);
/* The cudaError_t (as int) of the last failing CUDA call in this thread. */
int dv_last_cuda_error(void);
/* Library version, e.g. 100 for 0.1.0. */
int dv_version(void);
/* Number of kernels the library has enqueued in this process so far,
 * launches captured into a CUDA graph included (a diagnostic: the difference
 * across the calls of one step is that step's kernel count).  No
 * counterpart in the pages. */
long long dv_kernel_launches(void);

/* Zero-fill a workspace (once, before its first use). */
dv_status dv_workspace_init(void* ws, size_t ws_bytes, cudaStream_t stream);

/* Synchronise `stream`, then read and clear the workspace's device error
 * word.  Returns DV_OK or the first device-detected error code recorded
 * since the last check; *info (if not NULL) receives the offending value
 * (an index, a count or a position). */
dv_status dv_check(void* ws, cudaStream_t stream, int* info);

/* ------------------------------------------------------------- predictor */

/* Workspace bytes for dv_predict / dv_lookahead with up to `n_preds`
 * predictors of rank <= r_max scoring <= N_max units, batch B. */
dv_status dv_predict_workspace_size(int B, int n_preds, int r_max, int N_max,
                                    size_t* bytes);

/* Sparsity prediction ([blog] §2; [notes] "Sparsity operator for MLP" and
 * "... for Attention"): for each predictor p and batch row b
 *     h = ReLU(y_b P1),  z = h P2,  s = sigmoid(z)   (fp32 throughout)
 * then top-k or threshold selection into p.idx[b][...] (ascending) and
 * p.count[b].  Top-k ranks by s, ties to the lower index.  1 <= n_preds <= 2;
 * both predictors read the same y [B][d] and run in fused launches.
 * Limits: B <= 32, d <= 16384, r <= 4096, N <= 53248 (the selection stages
 * one row's scores in shared memory). */
dv_status dv_predict(const void* y, int B, int d, dv_dtype dt,
                     const dv_predictor* preds, int n_preds,
                     void* ws, size_t ws_bytes, cudaStream_t stream);

/* Asynchronous look-ahead prediction ([blog] §3.1; [notes] "Reducing
 * Overhead with Asynchronous Execution"): layer l+1's predictors run on
 * `side` from layer l's attention input y.  `side` first waits for
 * `input_ready` (if not NULL), then runs dv_predict, then records `done`
 * (if not NULL), which the main stream waits on before layer l+1. */
dv_status dv_lookahead(const void* y, int B, int d, dv_dtype dt,
                       const dv_predictor* preds, int n_preds,
                       void* ws, size_t ws_bytes,
                       cudaEvent_t input_ready, cudaStream_t side,
                       cudaEvent_t done);

/* Sparsity prediction without a caller workspace.  The pages have no
 * counterpart to this entry point: it exists for callers that cannot
 * allocate device memory -- for example a plugin inside a serving engine
 * that owns every device allocation, or a latency-critical loop where a
 * cudaMalloc (which can synchronise the device) is not allowed.
 *
 * Computes exactly what dv_predict computes, with the same arguments minus
 * the workspace.  Its scratch lives in a fixed array inside the library
 * (about 1.1 MB; every GPU that loads the library holds one until the
 * process exits).  Limits: B <= 4, r <= 1024 and N <= 32768 per predictor;
 * larger shapes are rejected with DV_ERR_WORKSPACE before anything runs.
 * Nothing is allocated or freed: no cudaMalloc, no cudaFree.
 *  - The first call on a device looks up the array's device address (with
 *    that device current); make that first call before any stream capture.
 *  - Every call, on any stream, shares the one array and overwrites what the
 *    previous call left there: calls whose work overlaps on the GPU race and
 *    give wrong results.  Serialise them (one stream, or events).
 *  - Device-side conditions are not reported: a threshold list longer than
 *    cap is truncated to cap entries as in dv_predict, with no error word to
 *    read back. */
dv_status dv_predict_static(const void* y, int B, int d, dv_dtype dt,
                            const dv_predictor* preds, int n_preds,
                            cudaStream_t stream);

/* ------------------------------------------------------------ sparse MLP */

dv_status dv_sparse_mlp_workspace_size(int B, int d, int N, int cap,
                                       size_t* bytes);

/* Sparsified MLP ([notes] "Sparsified MLP"; fused gather [blog] §3.2):
 *     out_b (+)= sum_{j in S_b} ReLU(y_b . W1n[j]) * W2n[j]
 * computed in one pass over the selected rows of W1n and W2n (no weight
 * sub-matrix is materialised).  S_b = idx[b][0 .. count[b]).  For B > 1 the
 * rows of the batch union are read once and each row b uses its own S_b.
 * out [B][d] fp32: overwritten (accumulate = 0) or added to (accumulate = 1,
 * e.g. a residual stream).  Below 8 rows every output element has one
 * writer and a fixed summation order, so results repeat bit for bit; the
 * tensor-core path (2+ rows of a 16-bit type) adds partial sums with fp32
 * atomics, so there the last bits of out may differ between runs.
 * Limits: B <= 32, d <= 16384 (8192 for DV_F32), N <= 65536. */
dv_status dv_sparse_mlp(const void* y, int B, int d, int N,
                        const void* W1n, const void* W2n,
                        const int32_t* idx, int cap, const int32_t* count,
                        dv_dtype dt, float* out, int accumulate,
                        void* ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------------ matrices in 4 bits */

/* Quantise W [N][d] (dt, row lengths as everywhere) in groups of `group` (64 or
 * 128) elements of a row, the last of a row as long as is left:
 *     scale = max |w| / 7, rounded to the storage type,
 *     code  = 8 + round-to-even(w / scale), kept within 0..15
 * (8 where the scale is 0).  A group with a NaN or an infinity gets a NaN as its
 * scale and codes 8: its products are NaNs.  q and scale as in dv_q4; values
 * [N][d] (storage type), unless NULL: what the codes stand for, rounded once.
 * Limits: N <= 16777216, d <= 32768; other groups return DV_ERR_UNSUPPORTED. */
dv_status dv_q4_quantize(const void* W, int N, int d, dv_dtype dt, int group,
                         void* q, void* scale, void* values,
                         cudaStream_t stream);

/* Workspace bytes of dv_q4_matvec. */
dv_status dv_q4_matvec_workspace_size(int B, int d, int N, size_t* bytes);

/* Products of B vectors with every row of a 4-bit matrix (an output head, a
 * projection):
 *     out[b][n] (+)= sum_t w[n][t] y[b][t],
 * y [B][d] in the storage type of the scales, out [B][N] fp32, see
 * dv_sparse_mlp for `accumulate`.  Codes and scales enter as they are.  For one
 * vector, and for two of up to 22528 elements, y enters in fixed point, 30 bits
 * below the largest magnitude of each group of elements (a scale times that magnitude
 * is taken in fp32: below 2^-120 it loses bits, above 2^127 a product may be a NaN),
 * else as it is; sums are fp32 and results repeat bit for bit.  A NaN or an infinity in y makes the products of that
 * vector NaN or infinite and no other's.  Like dv_layernorm's, its first
 * kernel may be started before the kernel ahead of the call has ended and waits
 * for it before it reads or writes anything.
 * Device errors: DV_ERR_TIMEOUT (see dv_set_wait_limit_ns; two and more vectors).
 * Limits: B <= 32, N <= 16777216, d <= 32768. */
dv_status dv_q4_matvec(const void* y, int B, int d, int N, const dv_q4* W,
                       dv_dtype dt, float* out, int accumulate,
                       void* ws, size_t ws_bytes, cudaStream_t stream);

dv_status dv_q4_sparse_mlp_workspace_size(int B, int d, int N, int cap,
                                          size_t* bytes);

/* dv_sparse_mlp with both matrices in 4 bits (their groups may differ):
 *     out_b (+)= sum_{j in S_b} ReLU(y_b . W1[j]) W2[j],
 * arguments as there.  An entry that a list holds twice counts once (for B = 1:
 * if the two are neighbours, as in the ascending lists of dv_predict), and a
 * neuron whose activation is 0 adds nothing, whatever its row of W2 holds.  The
 * first product is dv_q4_matvec's.  The activations are fp32; times their rows'
 * scales, rounded once, they enter the second product as they are for three and
 * more vectors, and for one and two in fixed point, 30 bits below the largest of
 * a share of the list.  Every output has one writer and a fixed order of
 * summation: results repeat bit for bit.
 * Its workspace is not one of dv_sparse_mlp (which keeps counters there).
 * dv_set_launch_overlap as for dv_sparse_mlp.
 * Device errors: DV_ERR_INDEX_RANGE (an entry outside [0, N) is skipped),
 * DV_ERR_CAPACITY (a count above cap is cut off), DV_ERR_TIMEOUT as for
 * dv_q4_matvec.
 * Limits: B <= 32, N <= 65536, d <= 32768. */
dv_status dv_q4_sparse_mlp(const void* y, int B, int d, int N, const dv_q4* W1,
                           const dv_q4* W2, const int32_t* idx, int cap,
                           const int32_t* count, dv_dtype dt, float* out,
                           int accumulate, void* ws, size_t ws_bytes,
                           cudaStream_t stream);

/* ------------------------------------------------------------- attention */

dv_status dv_sparse_attn_workspace_size(int B, int d, int h, int d_h, int cap,
                                        int n_max, size_t* bytes);

/* Sparsified attention for the token at position pos[b] of each sequence
 * ([notes] "Sparsified Attention" and "Sparsity operator for Attention"):
 *   1. append: X[b][pos] = y_b; for i in S_b: K/V[b][i][pos] = y_b W_i^{K,V}
 *      rounded to the storage type; valid[b][i][pos] = (i in S_b);
 *   2. KV repair: for i in S_b and every j < pos with valid[b][i][j] = 0,
 *      K/V[b][i][j] = X[b][j] W_i^{K,V}, then valid = 1;
 *   3. H_i = softmax(scale * q_i K_i^T) V_i over positions 0..pos, with
 *      q_i = y_b W_i^Q (fp32);
 *   4. out_b (+)= sum_{i in S_b} H_i W_i^O.
 * S_b = head_idx[b][0 .. head_count[b]); pos [B] is device memory.
 * scale multiplies the logits (1/sqrt(d_h) for the usual convention; the
 * page's formula prints none).  out [B][d] fp32, see dv_sparse_mlp for
 * `accumulate`.  Limits: B <= 32, d_h in {64, 128}, h <= 1024,
 * n_max <= 65536 (a multiple of 16), and one projection row of at most
 * 40 KB (d <= 20480 for 16-bit types, 10240 for DV_F32); other head
 * dimensions and rows return DV_ERR_UNSUPPORTED. */
dv_status dv_sparse_attn(const void* y, int B, int d, int h, int d_h,
                         const void* Wqkv, const void* Wo, const dv_kv* kv,
                         const int32_t* pos, const int32_t* head_idx, int cap,
                         const int32_t* head_count, float scale, dv_dtype dt,
                         float* out, int accumulate,
                         void* ws, size_t ws_bytes, cudaStream_t stream);

/* KV repair alone ([notes] "Sparsity operator for Attention"): for every
 * selected head i of sequence b and every j < pos[b] with valid = 0,
 * recompute K/V[b][i][j] from X[b][j] and set valid = 1.  With every head
 * selected and valid all 0 this is a dense prefill of positions 0..pos-1.
 * 0 <= pos[b] <= n_max (else DV_ERR_POSITION, the row is left as it is): a
 * full cache can be repaired.  Uses the dv_sparse_attn workspace. */
dv_status dv_kv_repair(const dv_kv* kv, int B, int d, int h, int d_h,
                       const void* Wqkv, const int32_t* pos,
                       const int32_t* head_idx, int cap,
                       const int32_t* head_count, dv_dtype dt,
                       void* ws, size_t ws_bytes, cudaStream_t stream);

/* ------------------------------------------------- true-sparsity labels */

/* Workspace bytes for dv_label_neurons (sequence of T tokens, N neurons)
 * and dv_label_heads (h heads of d_h); one workspace serves both. */
dv_status dv_label_workspace_size(int T, int d, int N, int h, int d_h,
                                  size_t* bytes);

/* Neuron labels ([blog] §1 Contextual Sparsity: MLP neurons whose outputs
 * over the input sequence have a large L2 norm, read neuron by neuron):
 *     norms[j] = sqrt( sum_t ReLU(X[t] . W1n[j])^2 ),  j < N,
 * for a sequence X [T][d] (e.g. a prompt's MLP inputs).  The product runs
 * on the tensor cores: 16-bit storage only (DV_F32 -> DV_ERR_DTYPE);
 * d a multiple of 8; fp32 accumulation; per-tile sums added in a fixed
 * order.  norms [N] fp32, device. */
dv_status dv_label_neurons(const void* X, int T, int d, int N, const void* W1n,
                           dv_dtype dt, float* norms, void* ws, size_t ws_bytes,
                           cudaStream_t stream);

/* Head labels ([blog] §1: attention heads whose output matrix over the
 * sequence has a large L2 norm, taken before the output projection):
 *     norms[i] = || H_i ||_F,  H_i[t] = softmax(scale q_t K_i[0..t]^T) V_i[0..t]
 * (causal: token t attends to tokens 0..t), q_t = X[t] W_i^Q in fp32 and
 * K/V = X W_i^{K,V} rounded to the storage type as a KV cache holds them.
 * 16-bit storage only; d_h in {64, 128}; norms [h] fp32, device. */
dv_status dv_label_heads(const void* X, int T, int d, int h, int d_h,
                         const void* Wqkv, float scale, dv_dtype dt,
                         float* norms, void* ws, size_t ws_bytes,
                         cudaStream_t stream);

/* Selection over rows of non-negative, finite fp32 scores [B][N] (e.g. the
 * label norms; [blog] §2: a threshold on the norm gives the labels): top-k
 * (ties to the lower index) or score > t, ascending, into idx [B][cap] with
 * count [B]; the same selection as dv_predict's.  N <= 53248.  ws: at
 * least 256 bytes, zero-filled once (its error word: a threshold list
 * longer than cap is truncated and reported as DV_ERR_CAPACITY). */
dv_status dv_select_scores(const float* scores, int B, int N, dv_select mode,
                           int k, float t, int32_t* idx, int cap,
                           int32_t* count, void* ws, size_t ws_bytes,
                           cudaStream_t stream);

/* ------------------------------------------- several candidates per sequence */

/* Workspace bytes of dv_tree_attn for trees of up to T nodes. */
dv_status dv_tree_attn_workspace_size(int B, int T, int h, int group, int d_h,
                                      size_t* bytes);

/* Attention of a drafted token tree over the KV cache: the queries of T
 * drafted tokens (nodes) per sequence against the committed positions and the
 * nodes' own K/V, in one pass over the cache (the pages have no counterpart:
 * a step there has one token).  The nodes of sequence b occupy the cache
 * positions pos[b] .. pos[b] + nodes[b] - 1; write their embeddings into X
 * there, clear their valid flags and let dv_kv_repair (with pos + nodes)
 * compute their K/V together with whatever the selected heads had skipped:
 * the valid flags themselves are not read here.
 *     out[b][t][i g + e] = sum_j p_j V[b][i][j] / sum_j p_j,
 *     p_j = exp(scale q[b][t][i g + e] . K[b][i][j]),   g = group, e < g,
 * over j < pos[b] and j = pos[b] + u for the nodes u that t sees.
 *  q, out [B][T][h g][d_h], storage type: g query heads share a K/V head
 *     (g = 1: one each, as in dv_sparse_attn).  out must not overlap q.
 *  nodes [B], or NULL: T nodes in every tree (0 <= nodes[b] <= T).
 *  mask: bytes, [T][T] for every sequence (mask_batched = 0) or [B][T][T]
 *     (1); node t sees node u where mask[t][u] != 0.  NULL: u <= t, a linear
 *     draft or a chunk of a prompt.  K/V of a node that a row does not see do
 *     not reach that row, whatever they hold.
 *  scale > 0, scale log2(e) finite.
 *  head_idx [B][cap] with head_count [B]: the K/V heads of each sequence's
 *     tree, as in dv_sparse_attn, each at most once; both NULL: all h heads.
 * Every row of out is written: those of other heads, of nodes behind
 * nodes[b], and of nodes that see nothing are 0.  Maximum, sum and numerator
 * are held in fp32; for 16-bit storage the weights p_j enter the product with V
 * as the sum of two values of the storage type (2^-17 relative for DV_BF16,
 * 2^-22, or 2^-31 of the row's largest weight, for DV_F16).  Results repeat bit
 * for bit.
 * Device errors: DV_ERR_POSITION (nodes[b] > 0, and pos[b] < 0 or
 * pos[b] + nodes[b] > n_max: the sequence's rows are 0), DV_ERR_INDEX_RANGE
 * (head skipped: its rows are 0), DV_ERR_CAPACITY (count above cap, or nodes
 * above T: cut off).
 * Limits: B <= 512, T <= 1024, h <= 1024, group <= 64, d_h in {64, 128}
 * (others DV_ERR_UNSUPPORTED), n_max <= 1048576, a multiple of 16, and
 * B heads (T group / 16) (n_max / 64) below 2^32 (else DV_ERR_UNSUPPORTED). */
dv_status dv_tree_attn(const void* q, int B, int T, int h, int group, int d_h,
                       const dv_kv* kv, const int32_t* pos,
                       const int32_t* nodes, const uint8_t* mask,
                       int mask_batched, const int32_t* head_idx, int cap,
                       const int32_t* head_count, float scale, dv_dtype dt,
                       void* out, void* ws, size_t ws_bytes,
                       cudaStream_t stream);

/* Keep the accepted nodes of a drafted tree: in each of the n_kv caches (a
 * decoder's layers) the rows of positions pos[b] + idx[b][k] move to
 * pos[b] + k, k < count[b], in place -- K and V where the valid flag is set,
 * X and the flags always.  idx [B][cap] is strictly ascending in every row
 * (a path of the tree in the order of its nodes).  Nothing else changes: the
 * flags behind the kept rows stay (they are cleared when the next tree's
 * rows are written).  new_pos [B] = pos + count, unless NULL; it may be pos.
 * Device errors: DV_ERR_INDEX_RANGE (a list that is negative or does not
 * ascend) and DV_ERR_POSITION (a position outside the cache): nothing moves
 * in that sequence, new_pos = pos; DV_ERR_CAPACITY: count cut off at cap.
 * All caches have the same shape and n_max.  ws: at least 256 bytes,
 * zero-filled once.  Limits: n_kv <= 1024, B <= 65535, h <= 1024. */
dv_status dv_kv_compact(const dv_kv* kv, int n_kv, int B, int d, int h, int d_h,
                        const int32_t* pos, const int32_t* idx, int cap,
                        const int32_t* count, dv_dtype dt, int32_t* new_pos,
                        void* ws, size_t ws_bytes, cudaStream_t stream);

/* Let beam w of each sequence continue beam parent[s][w]: in each of the n_kv
 * caches, whose rows are s * width + w, positions start[s] .. pos - 1 of row w
 * become those of row parent[s][w], all beams at once and in place, pos being
 * that of the parent's row (pos [n_seq][width]: positions held).  K and V
 * move where the parent's valid flag is set, X and the flags always; a beam
 * that continues itself is left alone, and so are positions below start (a
 * prompt that the beams share; NULL: 0) and behind.  pos itself is not
 * changed: where a sequence's beams differ in length, gather it by parent.
 * Device errors: DV_ERR_INDEX_RANGE (a parent outside [0, width): that beam is
 * left alone) and DV_ERR_POSITION (a parent whose pos is outside [0, n_max]: the
 * beams that continue it are left alone).
 * ws: at least 256 bytes, zero-filled once.  Limits: n_kv <= 1024,
 * n_seq <= 1023, width <= 32, h <= 1024. */
dv_status dv_kv_reorder(const dv_kv* kv, int n_kv, int n_seq, int width, int d,
                        int h, int d_h, const int32_t* pos,
                        const int32_t* start, const int32_t* parent,
                        dv_dtype dt, void* ws, size_t ws_bytes,
                        cudaStream_t stream);

/* Workspace bytes of dv_beam_select. */
dv_status dv_beam_select_workspace_size(int n_seq, int width, int V, int K,
                                        size_t* bytes);

/* The K best continuations of each sequence over its beams and the vocabulary:
 *     score(w, v) = cum[s][w] + logits[s][w][v] - log sum_u exp(logits[s][w][u]),
 * by score descending, ties to the lower w V + v; into score (fp32), token and
 * beam (the w it continues), each [n_seq][K].  K = width gives the next beams
 * and their parents for dv_kv_reorder; a larger K leaves a choice.
 *  logits [n_seq][width] rows of V, row_stride elements apart; any alignment.
 *  done [n_seq][width], or NULL: a beam whose byte is not 0 has ended: it
 *     offers end_token at score cum[s][w] and every other token at -inf.
 * Beams that have not ended: a row whose log-sum-exp is not finite (a NaN, a
 * +inf, or nothing above -inf) and a row whose cum is not finite offer every
 * token at -inf.  A beam's candidates are in the order of its logits, those of
 * different beams are compared in double precision.  A row's log-sum-exp is
 * taken over fp32 exponentials, summed with compensation by each thread of a
 * part of the row, in fp32 over a part's threads and in double over parts:
 * 4e-7 off at most in rows that were tried, 177 x 2^-24 in any row, whatever V.
 * Results repeat bit for bit.
 * Limits: n_seq * width <= 65535, width <= 32, V <= 4194304, 1 <= K <= 64 and
 * K <= width V. */
dv_status dv_beam_select(const void* logits, int n_seq, int width, int V,
                         long long row_stride, dv_dtype dt, const float* cum,
                         const uint8_t* done, int end_token, int K,
                         float* score, int32_t* token, int32_t* beam,
                         void* ws, size_t ws_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------- sampling */

/* Workspace bytes of dv_sample. */
dv_status dv_sample_workspace_size(int B, int V, size_t* bytes);

/* One token of each row, drawn with the caller's random number (the pages have
 * no counterpart: they end with the logits).  For row b, x = logits[b],
 *     w_i = exp((x_i - max x) / T),
 * and the tokens in the order of x descending, of equal ones the lower index
 * first, kept are
 *   the first top_k (all if top_k <= 0);
 *   of those, the ones before which less than top_p of their mass lies: the
 *     smallest set that holds top_p of it (the first token always; all if
 *     top_p >= 1);
 *   of those, the ones with w_i >= min_p (min_p above 1 counts as 1).
 * token[b] is the lowest kept i for which the kept w up to and with i add up to
 * more than u of the sum of all kept w; prob[b], unless NULL, is w_i over that
 * sum.  T = 0: the best token, prob 1; otherwise 1e-30 <= T <= 1e30.
 *  logits: B rows of V, row_stride elements apart; any alignment.  -inf tokens
 *     are never drawn.
 *  u [B] in [0, 1) (below counts as 0, above as just below 1); temperature,
 *     top_p, min_p [B] fp32, top_k [B] int32, each or NULL: 1, 1, 0, 0.
 * Weights are held to 2^-29 of themselves and 2^-40 (1 being the best token's;
 * below 2^-40 they count as none) and added without rounding: a sum over n
 * tokens is off by 2^-29 of itself and n 2^-40 at most (4.8e-7 of the best
 * token's weight for 524288 of them; each is as likely to be up as down).  The
 * token is the one of the formulas in exact arithmetic unless a border lies
 * that near: a token's weight to min_p, a sum to its share top_p or u of
 * another.  Results repeat bit for bit, whatever else is in the batch.
 * A row without a distribution (a NaN or +inf, or nothing above -inf, among its
 * logits; another temperature; a NaN as u, top_p or min_p)
 * gets token -1 and prob 0 and is reported as DV_ERR_INVALID_ARG with b; other
 * rows are not affected.
 * ws: dv_sample_workspace_size bytes (the error word), zero-filled once.
 * Limits: B <= 65535, V <= 524288. */
dv_status dv_sample(const void* logits, int B, int V, long long row_stride,
                    dv_dtype dt, const float* u, const float* temperature,
                    const int32_t* top_k, const float* top_p, const float* min_p,
                    int32_t* token, float* prob, void* ws, size_t ws_bytes,
                    cudaStream_t stream);

/* ---------------------------------------------------- decoder-step helpers */

/* y_b = LayerNorm(x_b) without affine terms (eps given), rounded to the
 * storage type: the pre-LN input of each sparse block (the pages do not state
 * the normalisation; this is the plain pre-LN reading).  x [B][d] fp32,
 * 16-byte aligned, d a multiple of 4 and at most 16384; y [B][d] 8-byte
 * aligned.  Other shapes return DV_ERR_INVALID_ARG. */
dv_status dv_layernorm(const float* x, int B, int d, float eps,
                       void* y, dv_dtype dt, cudaStream_t stream);

/* Launch policy (no counterpart in the pages; it changes timing, never
 * results).  Inside every entry point the later kernels start during the
 * earlier ones and read only data those do not write.  At level 0 (the
 * default) the first kernel of each call waits for everything before it
 * (those of dv_layernorm, dv_tree_attn, dv_beam_select, dv_q4_matvec and
 * dv_sample may be started earlier, at either level, and wait before they read
 * or write anything).
 * At level 1, for batch 1, the first kernel of dv_sparse_attn, dv_sparse_mlp and
 * dv_q4_sparse_mlp may also start while the kernel before the call is still
 * running, and reads before waiting for it: the head / neuron lists and
 * counts, pos, the valid flags and the weights.  Enable it only when the
 * kernel issued just before each such call (on the same stream) writes none
 * of those -- true when that kernel is the dv_layernorm producing the call's
 * y, as in a pre-LN decoder -- and neither does the kernel before that
 * layernorm, which lets its consumer start at once (in a pre-LN decoder it
 * is the previous block's dv_sparse_attn or dv_sparse_mlp).  dv_tree_attn,
 * too, lets the call after it start while both its kernels run; they write
 * nothing but its out and its workspace.  Process-wide; returns the previous
 * level. */
int dv_set_launch_overlap(int level);

/* Bound of every device-side wait (no counterpart in the pages): the
 * one-launch MLP's wait for its up-projection CTAs, the tensor-core paths'
 * pipeline waits (those of dv_tree_attn, and of dv_q4_matvec and
 * dv_q4_sparse_mlp for two and more vectors, among them) and the waits for
 * copies of the streaming MLP, dv_beam_select and dv_sample give up after `ns`
 * nanoseconds of the GPU's global timer, record DV_ERR_TIMEOUT in the
 * workspace (read it with dv_check)
 * and unwind; the kernel still waits for its own tensor-core and copy work in
 * flight before it exits.  ns <= 0 restores the default of one second.
 * Read at launch (a captured graph keeps the value it was captured with);
 * process-wide; returns the previous bound. */
long long dv_set_wait_limit_ns(long long ns);

/* pos[b] = pos[b] + 1, or `lo` when that reaches `hi` (decode loop). */
dv_status dv_positions_advance(int32_t* pos, int B, int lo, int hi,
                               cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DV_H_ */
