/*
 * gt_attn.h -- C ABI of libgt: topology-biased graph attention on one GB300.
 *
 * The operation (MegaGraph, "Towards Efficient Training of Large-Scale Graph
 * Transformers with Automated Hybrid Parallelism"):
 *   - abstract: a Graph Transformer layer carries, besides the attention score
 *     matrix, a topology-aware bias matrix of the same N x N shape per head;
 *   - Fig. 4: attention is computed KV block by KV block, and the bias columns
 *     that go with each incoming KV block are sliced on the fly.
 * The bias is the Graphormer spatial encoding over clipped shortest-path
 * distances:  b[h][i][j] = T[h][ spd[i][j] ],  spd[i][j] = min(dist(i,j), D) for
 * reachable pairs and D+1 otherwise, so T has nb = D+2 columns.  Per head h:
 *   s_ij = scale * <q_i, k_j> + b[h][i][j],   o_i = sum_j softmax_j(s_i) v_j,
 *   lse_i = log sum_j exp(s_ij)  (natural log),
 * and the backward pass returns dq, dk, dv and dT[h][c] = sum over pairs with
 * spd[i][j] = c of dS_ij, where dS_ij = p_ij (<dO_i, v_j> - <dO_i, o_i>).
 * Neither the N x N scores nor the N x N x H bias is ever stored.
 *
 * Conventions for every call below
 *   - Pointers named as device buffers must be device memory of the current
 *     CUDA device.  The caller owns and allocates every buffer, including the
 *     workspace; the library allocates no device memory and keeps no state
 *     between calls apart from one device status word per device (see
 *     gt_check_device_status) and the launch statistics at the end of this
 *     header.  Every kernel runs on the caller's stream.
 *   - The library caches per-device addresses (the status word; the scratch
 *     array of gt_bias_attn_bwd_noalloc).  Do not reset a device
 *     (cudaDeviceReset) while the library is loaded in the process: the cached
 *     addresses would outlive the context they belong to.
 *   - Layouts are dense row-major: q, k, v, o, dO, dq, dk, dv are [n][h][d]
 *     (node, head, channel); lse is [h][n] fp32; T and dT are [h][nb] fp32;
 *     spd is int8 [n][ld_spd] (row i holds the bucket codes of pairs (i, *)).
 *   - `dtype` selects the element type of q, k, v, o, dO, dq, dk, dv:
 *     GT_F32 (exact fp32 arithmetic) or GT_BF16 (bf16 storage, tensor-core
 *     products with fp32 accumulation, fp32 softmax statistics).
 *   - All calls are asynchronous on `stream` (a cudaStream_t, NULL = legacy
 *     default stream).  They check their arguments on the host before any
 *     launch and return a negative gt_status without launching if a check
 *     fails.  GT_OK means the work was enqueued.  Within a call, a kernel may
 *     be scheduled while the one before it finishes (programmatic dependent
 *     launch); each such kernel waits for its predecessor before reading that
 *     one's output and before it completes, so what the caller's later work
 *     on the stream sees is the same as with plain stream order.
 *   - Bucket codes are read as unsigned bytes; codes >= nb select a zero bias
 *     in the forward and are dropped from dT (they never occur in the output of
 *     gt_spd_build).
 */
#ifndef GT_ATTN_H
#define GT_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GT_OK = 0,
    GT_ERR_INVALID_ARG = -1,  /* NULL, size, alignment or layout check failed */
    GT_ERR_UNSUPPORTED = -2,  /* shape valid but not handled by this library */
    GT_ERR_CUDA = -3,         /* a CUDA runtime call or launch failed */
    GT_ERR_TIMEOUT = -4,      /* a kernel gave up a bounded wait (see below) */
    GT_ERR_WORKSPACE = -5     /* workspace NULL or smaller than the size query */
} gt_status;

typedef enum { GT_F32 = 0, GT_BF16 = 1 } gt_dtype;

/* Largest clip distance: codes 0..D+1 must fit a signed byte. */
#define GT_MAX_D 126

/*
 * Bytes of device workspace gt_spd_build needs for this graph size on the
 * current device.
 */
size_t gt_spd_workspace_size(int32_t n, int64_t nnz, int32_t D);

/*
 * gt_spd_build: clipped shortest-path bucket matrix of an undirected graph
 * (the topology the bias of the MegaGraph abstract is built from).
 *   indptr  device int64[n+1], indices device int32[nnz]: CSR adjacency with
 *           both directions of every edge stored (self-loops and repeated
 *           entries are harmless).
 *   n >= 1, 1 <= D <= GT_MAX_D.
 *   spd     device int8 [n][ld_spd], written for columns 0..n-1 of every row:
 *           spd[i][j] = min(dist(i,j), D) if j is reachable from i, D+1 if not,
 *           0 on the diagonal.  ld_spd >= n and ld_spd % 16 == 0; spd 16-byte
 *           aligned.  Columns n..ld_spd-1 are not written.
 *   workspace/ws_bytes: device scratch of at least gt_spd_workspace_size().
 * Errors: GT_ERR_INVALID_ARG for NULL pointers, n < 1, nnz < 0, D out of range,
 * bad ld_spd or alignment; GT_ERR_WORKSPACE for a short workspace.
 */
int gt_spd_build(const int64_t* indptr, const int32_t* indices, int32_t n, int64_t nnz,
                 int32_t D, int8_t* spd, int64_t ld_spd,
                 void* workspace, size_t ws_bytes, void* stream);

/*
 * Search algorithms of gt_spd_build.  All give the same codes; they differ in
 * where the per-vertex state lives, which bounds the graph size they take:
 *   GT_SPD_SCAN32    32 sources per batch, every per-vertex word in shared
 *                    memory (12 bytes per vertex), n up to ~18.8K on a GB300.
 *   GT_SPD_SCAN16    16 sources per batch, two vertices per word (6 bytes per
 *                    vertex), n up to ~37K.
 *   GT_SPD_QUEUE32   32 sources per batch, frontier queues in global memory,
 *                    pushes into shared memory (4 bytes per vertex), n up to ~58K.
 *   GT_SPD_GLOBAL64  64 sources per batch, all state in global memory: any n.
 *   GT_SPD_AUTO      what gt_spd_build uses: a scan search that runs two CTAs
 *                    per SM when its state fits twice in an SM's shared memory
 *                    and the batches outnumber the SMs (SCAN32 if it does so,
 *                    else SCAN16 when 32-source batches would fill the SMs
 *                    anyway), otherwise the first of these that fits.
 * The scan searches run one CTA of 1024 threads per SM, or two of 512 under the
 * condition above.
 */
enum { GT_SPD_AUTO = 0, GT_SPD_SCAN32 = 1, GT_SPD_SCAN16 = 2, GT_SPD_QUEUE32 = 3, GT_SPD_GLOBAL64 = 4 };

/*
 * Workspace bytes of gt_spd_build_algo for this algorithm, or 0 when the
 * algorithm cannot take n vertices on the current device (or the arguments are
 * out of range).
 */
size_t gt_spd_workspace_size_algo(int32_t algo, int32_t n, int64_t nnz, int32_t D);

/*
 * gt_spd_build with an explicit search algorithm (same arguments and result).
 * Errors as gt_spd_build, plus GT_ERR_INVALID_ARG for an unknown algo and
 * GT_ERR_UNSUPPORTED when the algorithm cannot take n vertices on this device.
 */
int gt_spd_build_algo(int32_t algo, const int64_t* indptr, const int32_t* indices, int32_t n,
                      int64_t nnz, int32_t D, int8_t* spd, int64_t ld_spd,
                      void* workspace, size_t ws_bytes, void* stream);

/*
 * The uniform KV block gt_bias_attn_fwd uses for these arguments (0 = none;
 * -1 for invalid arguments): an explicit kv_block (< n) is used as given.  With
 * kv_block = 0 no uniform split is made; the bf16 tensor-core path instead
 * deals its (query tile, head half, KV block) work out in equal contiguous
 * shares to a whole number of waves of two CTAs per SM, whenever one CTA per
 * tile and head half would leave part of the last wave idle.  A share covers
 * the end of one tile's KV range and the start of the next; rows whose range
 * more than one CTA covered are merged exactly through their lse (the same
 * merge as for KV blocks, Fig. 4), the others are written directly.
 */
int32_t gt_bias_attn_fwd_kv_block(int32_t dtype, int32_t n, int32_t h, int32_t d, int32_t kv_block);

/*
 * CTAs of that balanced tensor-core forward for these arguments on the current
 * device (-1 for invalid arguments): 0 when the forward runs one CTA per 128-row
 * tile and head half (an explicit kv_block, another dtype or shape, or a grid
 * whose waves are full already).  A balanced forward launches one merge kernel
 * after the attention kernel.
 */
int32_t gt_bias_attn_fwd_ctas(int32_t dtype, int32_t n, int32_t h, int32_t d, int32_t kv_block);

/*
 * How many CTAs share each dq task (a 128-row query tile and a head half) of
 * the bf16 tensor-core backward for these sizes on the current device (1 = none;
 * -1 for invalid arguments).  The dq tasks that do not fill a whole wave of two
 * CTAs per SM (all of them on a graph too small to fill one) are split along
 * their KV blocks, k ways with k in 2..8 chosen so that the last waves fill the
 * SMs.  The dk/dv groups (a 128-row KV tile and a head half) past the last full
 * wave of one CTA per SM are split along their query tiles the same way; fewer
 * groups than SMs run instead as equal shares of all (group, query tile) steps,
 * one CTA per SM.  Split or shared work sums in fp32 (workspace included in
 * gt_bias_attn_workspace_size; a workspace too small for the sums runs
 * unsplit).
 */
int32_t gt_bias_attn_bwd_split(int32_t dtype, int32_t n, int32_t h, int32_t d, int32_t nb);

/*
 * Kernel launches of one gt_bias_attn_fwd call (*fwd, with this kv_block) and of
 * one gt_bias_attn_bwd call (*bwd, with these nb buckets) on the current device,
 * given a workspace of gt_bias_attn_workspace_size bytes; memsets are not
 * counted.  A split of the tasks past the last full wave (see
 * gt_bias_attn_bwd_split) adds the split tasks' own launch when whole tasks
 * fill waves before them; the backward's last launch converts every split's
 * fp32 sums and the bucket sums at once.  Returns GT_OK, or
 * GT_ERR_INVALID_ARG for invalid arguments or NULL outputs.
 */
int gt_bias_attn_launches(int32_t dtype, int32_t n, int32_t h, int32_t d, int32_t nb, int32_t kv_block,
                          int32_t* fwd, int32_t* bwd);

/*
 * Bytes of device workspace needed by gt_bias_attn_fwd (with this kv_block)
 * and by gt_bias_attn_bwd for these sizes; one buffer of this size serves both.
 */
size_t gt_bias_attn_workspace_size(int32_t dtype, int32_t n, int32_t h, int32_t d,
                                   int32_t kv_block);

/*
 * gt_bias_attn_fwd: o = softmax(scale * q k^T + T[h][spd]) v per head, plus lse.
 *   q, k, v  device [n][h][d] of `dtype`, 16-byte aligned.
 *   spd      device int8 [n][ld_spd] bucket codes (ld_spd >= n, % 16 == 0,
 *            16-byte aligned).
 *   T        device fp32 [h][nb], nb <= 128.
 *   scale    multiplies q.k before the bias is added (1/sqrt(d) is usual).
 *   kv_block 0: every Q tile streams all n KV columns (in at most a few
 *            balanced pieces: see gt_bias_attn_fwd_kv_block).
 *            > 0 (a multiple of 128): the columns are cut into blocks of
 *            kv_block (the KV blocks of Fig. 4); each block yields a partial
 *            (o, lse) and the partials are merged exactly through their lse.
 *   o        device [n][h][d] of `dtype` (output); lse device fp32 [h][n].
 *   workspace/ws_bytes: at least gt_bias_attn_workspace_size(...).
 * Supported: n >= 1, 1 <= h <= 16, 1 <= d <= 64.  GT_BF16 with h = 8 and
 * d in {8, 16} runs on the tensor cores; other shapes run on a CUDA-core kernel.
 */
int gt_bias_attn_fwd(int32_t dtype, int32_t n, int32_t h, int32_t d,
                     const void* q, const void* k, const void* v,
                     const int8_t* spd, int64_t ld_spd, const float* T, int32_t nb,
                     float scale, int32_t kv_block,
                     void* o, float* lse, void* workspace, size_t ws_bytes, void* stream);

/*
 * The forward over one range of KV columns, and the exact merge of such
 * partials: Fig. 4's ring step on one GPU.  A caller that holds KV blocks
 * [a_0, a_1), [a_1, a_2), ... in turn (a ring across GPUs, or blocks streamed
 * from host memory) computes each block's partial with gt_bias_attn_fwd_partial
 * and combines them with gt_bias_attn_merge; the result equals
 * gt_bias_attn_fwd over all columns up to rounding.
 *
 * gt_bias_attn_fwd_partial: every query row attends only to KV columns
 * [kv_begin, kv_end), with the bias columns of that range.
 *   q, k, v, spd, ld_spd, T, nb, scale: as for gt_bias_attn_fwd (k and v hold
 *            all n rows; only the range's rows are read).
 *   kv_begin a multiple of 128, 0 <= kv_begin < kv_end <= n.
 *   o_part   device fp32 [n][h][d] (output, 16-byte aligned): the output
 *            normalised over the range's columns.
 *   lse_part device fp32 [h][n] (output): log of the range's softmax
 *            denominator (natural log, scores include the bias).
 * Needs no workspace.  Errors as for gt_bias_attn_fwd, plus GT_ERR_INVALID_ARG
 * for a bad range.
 *
 * gt_bias_attn_merge: o = sum_p exp(lse_p - lse) o_p with lse = log sum_p
 * exp(lse_p), per (node, head).
 *   o_parts  device fp32 [nparts][n][h][d]; lse_parts device fp32 [nparts][h][n].
 *   o        device [n][h][d] of `dtype` (output); lse device fp32 [h][n].
 * Errors: GT_ERR_INVALID_ARG for NULL pointers, n, h, d or nparts < 1;
 * GT_ERR_UNSUPPORTED for h > 16 or d > 64.
 */
int gt_bias_attn_fwd_partial(int32_t dtype, int32_t n, int32_t h, int32_t d,
                             const void* q, const void* k, const void* v,
                             const int8_t* spd, int64_t ld_spd, const float* T, int32_t nb,
                             float scale, int32_t kv_begin, int32_t kv_end,
                             float* o_part, float* lse_part, void* stream);
int gt_bias_attn_merge(int32_t dtype, int32_t n, int32_t h, int32_t d, int32_t nparts,
                       const float* o_parts, const float* lse_parts, void* o, float* lse,
                       void* stream);

/*
 * gt_bias_attn_bwd: gradients of sum(o * dO) with respect to q, k, v and T.
 *   o, lse   the forward's outputs for the same inputs.
 *   dO       device [n][h][d] of `dtype`, the upstream gradient.
 *   dq, dk, dv device [n][h][d] of `dtype` (outputs, overwritten).
 *   dT       device fp32 [h][nb] (output, overwritten).
 * Other arguments and the supported shapes are as for gt_bias_attn_fwd.
 */
int gt_bias_attn_bwd(int32_t dtype, int32_t n, int32_t h, int32_t d,
                     const void* q, const void* k, const void* v, const void* o,
                     const void* dO, const float* lse,
                     const int8_t* spd, int64_t ld_spd, const float* T, int32_t nb,
                     float scale, void* dq, void* dk, void* dv, float* dT,
                     void* workspace, size_t ws_bytes, void* stream);

/*
 * gt_bias_attn_bwd_noalloc: gt_bias_attn_bwd for callers that cannot allocate.
 * The paper has no counterpart; this is a library convenience.
 *
 * Some callers cannot call cudaMalloc or any allocator (a host framework that
 * owns all device memory, a real-time or embedded host that forbids allocation
 * after start-up, a plain C host with no caching allocator).  This variant takes
 * no workspace: it runs the same backward pass with its scratch in an array of
 * GT_NOALLOC_SCRATCH_BYTES compiled into the library, which every GPU that loads
 * the library holds until the process exits.  Inputs and outputs are passed and
 * owned by the caller exactly as for gt_bias_attn_bwd, and the results match it.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, once per device, with that device current); make
 *     that first call before any stream capture.  No call allocates or frees
 *     device memory.
 *   - Every call shares the one array and leaves its contents behind (the pass
 *     clears what must start at zero).  Calls whose GPU work overlaps, on
 *     different streams or host threads of one device, race on the array and
 *     corrupt each other's results: serialise them.
 *   - Returns GT_ERR_WORKSPACE, with nothing launched, when the backward run
 *     without its split (the split's fp32 sums are left out when they do not
 *     fit) needs more than GT_NOALLOC_SCRATCH_BYTES.  That scratch is, in bytes,
 *     with 256-byte alignment of each part: 4 h n (D) + 1024 (dT sums)
 *     + 64 * ((n + 3) / 4 * 4) (per-node lse and D rows) + 256 n (the bf16 lse / D
 *     operand of the dk/dv products) + 64; with H = 8 about 352 bytes per node,
 *     so N up to about 11,900 nodes.  gt_bias_attn_workspace_size may report
 *     more than this for small graphs (it includes the split's sums); such calls
 *     still succeed, unsplit.
 */
#define GT_NOALLOC_SCRATCH_BYTES (4u << 20)
int gt_bias_attn_bwd_noalloc(int32_t dtype, int32_t n, int32_t h, int32_t d,
                             const void* q, const void* k, const void* v, const void* o,
                             const void* dO, const float* lse,
                             const int8_t* spd, int64_t ld_spd, const float* T, int32_t nb,
                             float scale, void* dq, void* dk, void* dv, float* dT, void* stream);

/*
 * The GT encoder layer around the biased attention (MegaGraph, Fig. 8: 8 heads,
 * hidden and FFN width 64).  The pages give the widths, not the order of the
 * steps; this is the pre-LayerNorm (Graphormer) encoder layer:
 *
 *   u = LN1(x); [q|k|v] = u W_qkv + b_qkv; o = biased attention(q, k, v);
 *   hh = x + o W_o + b_o; z = LN2(hh); y = hh + GELU(z W_1 + b_1) W_2 + b_2
 *
 * with LN(v) = gain (v - mean v) / sqrt(var v + 1e-5) + shift over the 64
 * features of a node, GELU(a) = a Phi(a) (Phi the normal CDF), the attention
 * scale 1/sqrt(8), and q, k, v split into heads as [n][8][8] (feature = head * 8
 * + channel).  Supported: h = 8, d = 8, f = 64 (else GT_ERR_UNSUPPORTED); the
 * attention runs in bf16 on the tensor cores, and so do the layer's products:
 * tf32 (fp32 storage) for the projections and the FFN, bf16 for the products
 * over node rows that form the weight gradients, fp32 accumulation in both.
 *
 * All weights are device fp32, row-major: ln*_g / ln*_b [64]; w_qkv [64][192]
 * (columns q | k | v); b_qkv [192]; w_o [64][64]; b_o [64]; w_1 [64][64] (in x
 * out); b_1 [64]; w_2 [64][64]; b_2 [64]; the four matrices 16-byte aligned,
 * and so every node-row array (x, y, dy, dx, q, k, v, o): the layer kernels move
 * whole rows with bulk copies.
 * gt_layer_grads has the same shapes and receives dL/d(weight) (overwritten).
 */
typedef struct {
    const float *ln1_g, *ln1_b, *w_qkv, *b_qkv, *w_o, *b_o, *ln2_g, *ln2_b, *w_1, *b_1, *w_2, *b_2;
} gt_layer_weights;

typedef struct {
    float *ln1_g, *ln1_b, *w_qkv, *b_qkv, *w_o, *b_o, *ln2_g, *ln2_b, *w_1, *b_1, *w_2, *b_2;
} gt_layer_grads;

/* Workspace bytes of gt_layer_fwd and gt_layer_bwd (one buffer serves both);
 * 0 for unsupported sizes. */
size_t gt_layer_workspace_size(int32_t n, int32_t h, int32_t d, int32_t f);

/*
 * gt_layer_fwd: y (device fp32 [n][64]) from x (device fp32 [n][64]).  Also
 * writes what the backward needs: q, k, v, o (device bf16 [n][8][8]) and lse
 * (fp32 [8][n]).  spd, ld_spd, T, nb as for gt_bias_attn_fwd.
 * Errors: GT_ERR_UNSUPPORTED for other sizes, GT_ERR_INVALID_ARG for NULL
 * pointers (any weight included) or unaligned matrices, the attention's own
 * checks, GT_ERR_WORKSPACE.
 */
int gt_layer_fwd(int32_t n, int32_t h, int32_t d, int32_t f, const float* x, const gt_layer_weights* w,
                 const int8_t* spd, int64_t ld_spd, const float* T, int32_t nb,
                 void* q, void* k, void* v, void* o, float* lse, float* y,
                 void* workspace, size_t ws_bytes, void* stream);

/*
 * gt_layer_bwd: given dy = dL/dy (device fp32 [n][64]) and the forward's x, q,
 * k, v, o, lse: dx (device fp32 [n][64], overwritten), every weight gradient
 * (overwritten) and dT (fp32 [8][nb], overwritten).  Errors as gt_layer_fwd.
 */
int gt_layer_bwd(int32_t n, int32_t h, int32_t d, int32_t f, const float* x, const gt_layer_weights* w,
                 const int8_t* spd, int64_t ld_spd, const float* T, int32_t nb,
                 const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const float* dy, float* dx, const gt_layer_grads* g, float* dT,
                 void* workspace, size_t ws_bytes, void* stream);

/*
 * LayerNorm and linear layers at any width: what surrounds the biased attention
 * in an encoder layer whose widths gt_layer_fwd does not take (the attention
 * itself takes h <= 16 heads of d <= 64 channels).  The pre-LayerNorm layer above is
 *   u = gt_layer_norm_fwd(x);  q, k, v = gt_linear_fwd(u, W_q | W_k | W_v);
 *   o = gt_bias_attn_fwd(q, k, v);  hh = gt_linear_fwd(o, W_o, r = x);
 *   z = gt_layer_norm_fwd(hh);  g = gt_linear_fwd(z, W_1, act = GELU);
 *   y = gt_linear_fwd(g, W_2, r = hh)
 * with a row per node.  Every matrix is row-major with a leading dimension in
 * elements (ld >= columns), so slices of wider matrices serve; any alignment of
 * its element type is accepted, and rows whose base and stride are multiples of
 * 16 bytes move faster.  Statistics and sums are fp32.  Results do not change
 * from run to run.  Outputs must not overlap each other or any input, except
 * where a call says so.  A workspace is 16-byte aligned (GT_ERR_WORKSPACE if not);
 * its contents matter during a call only, and calls that may run at the same time
 * need workspaces of their own.
 *
 * gt_layer_norm_fwd: per row, over its c features,
 *   mean = sum_j x_j / c, rstd = 1 / sqrt(sum_j (x_j - mean)^2 / c + eps),
 *   y_j = gain_j (x_j - mean) rstd + shift_j
 *   xtype, ytype  element types (gt_dtype) of x and of y, any pair.
 *   x  device [n][ldx], y device [n][ldy]; gain, shift device fp32 [c]; mean,
 *   rstd device fp32 [n] (outputs: the backward takes them).
 * Errors: GT_ERR_INVALID_ARG for a NULL pointer, an unknown type, n < 1, c < 1, a
 * leading dimension below c, or an eps that is not finite and positive;
 * GT_ERR_UNSUPPORTED for c > 16384.
 *
 * gt_layer_norm_bwd: given dy = dL/dy, with xh = (x - mean) rstd and d = gain dy,
 *   dx = rstd (d - sum_j d_j / c - xh sum_j d_j xh_j / c) + dres
 *   dgain = sum over rows of dy xh,  dshift = sum over rows of dy
 *   dy has y's type; dx (output) and dres (NULL: none; the gradient that reaches x
 *   around the norm) have x's type, and may be one buffer; dgain, dshift device
 *   fp32 [c] (outputs, overwritten).  workspace: at least
 *   gt_layer_norm_workspace_size(n, c) bytes (0 for sizes not supported).
 * Errors as the forward's, plus GT_ERR_WORKSPACE.
 */
int gt_layer_norm_fwd(int32_t xtype, int32_t ytype, int32_t n, int32_t c, const void* x, int64_t ldx,
                      const float* gain, const float* shift, float eps, void* y, int64_t ldy,
                      float* mean, float* rstd, void* stream);
size_t gt_layer_norm_workspace_size(int32_t n, int32_t c);
int gt_layer_norm_bwd(int32_t xtype, int32_t ytype, int32_t n, int32_t c, const void* dy, int64_t lddy,
                      const void* x, int64_t ldx, const float* gain, const float* mean, const float* rstd,
                      const void* dres, int64_t ldr, void* dx, int64_t lddx, float* dgain, float* dshift,
                      void* workspace, size_t ws_bytes, void* stream);

/*
 * Activations of the linear layer: none, or GELU(a) = a Phi(a) (Phi the normal CDF), in fp32:
 * 1.2e-7 off for |a| <= 2, 6e-5 of itself down to a = -13; infinity for infinity, NaN for minus
 * infinity (its product with 0).
 */
typedef enum { GT_ACT_NONE = 0, GT_ACT_GELU = 1 } gt_act;

/*
 * gt_linear_fwd: a = x W + b, y = act(a) + r.
 *   dtype  type of x, W and pre: GT_BF16 (bf16 products, fp32 sums) or GT_F32
 *          (products of three-part bf16 splits, fp32 sums: fp32 accuracy for inputs
 *          above 2^-100 in magnitude, smaller ones lose low bits; a non-finite input, or
 *          a product past the range of fp32, makes the sums it enters non-finite, NaN
 *          where exact arithmetic may give an infinity).
 *   ytype  type of y and r: GT_F32, or GT_BF16 with dtype GT_BF16.
 *   x  device [m][ldx >= k]; W device [k][ldw >= n] (in x out); b device fp32 [n] or
 *   NULL; r device [m][ldr >= n] or NULL (it may be y itself).
 *   y  device [m][ldy >= n] (output); pre device [m][ldpre >= n] or NULL (output): a,
 *   rounded to dtype, which the backward of a GELU layer takes.
 *   workspace: at least gt_linear_fwd_workspace_size bytes (may be NULL where that
 *   is 0).  `aligned`: non-zero when the bases and row strides of all the call's
 *   matrices are multiples of 16 bytes; else the size includes the copies of x and W
 *   and the fp32 result ([m][n]) that such rows may need.
 * Supported: 1 <= m <= 2^24, 1 <= k, n <= 65536.
 * Errors: GT_ERR_INVALID_ARG for a NULL x, W or y, an unknown type or activation, m,
 * k or n < 1, or a leading dimension below its row; GT_ERR_UNSUPPORTED for larger
 * sizes or a bf16 y of fp32 products; GT_ERR_WORKSPACE.
 *
 * gt_linear_bwd: given dy = dL/dy (type ytype), with da = dy act'(pre),
 *   dx = da W^T + add,  dW = x^T da,  db = sum over rows of da
 *   (the gradient with respect to r is dy itself).  Any of dx, dw, db may be NULL: it
 *   is not computed, and what only it reads (W for dx, x for dw) may be NULL too.
 *   pre    the forward's pre with GT_ACT_GELU; NULL with GT_ACT_NONE.
 *   add    device [m][ldadd >= k] of dtype or NULL (it may be dx itself): a gradient
 *          that reaches x another way.
 *   dx     device [m][lddx >= k] of dtype; dw device [k][lddw >= n] of dtype; db device
 *          fp32 [n] (outputs, overwritten).
 *   With dtype GT_BF16 da is rounded to bf16 for the two products, from fp32 dy too (db is
 *   summed before that rounding); with GT_F32 (operands converted by the caller) it is not.
 *   workspace: at least gt_linear_bwd_workspace_size bytes (may be NULL where that is 0;
 *   `aligned` as above; else with copies of dy, x and W and fp32 results, [m][k] and [k][n]).
 * Errors as the forward's, plus GT_ERR_INVALID_ARG when dx, dw and db are all NULL,
 * pre and act disagree, or add comes without dx.
 */
size_t gt_linear_fwd_workspace_size(int32_t dtype, int32_t m, int32_t k, int32_t n, int32_t aligned);
int gt_linear_fwd(int32_t dtype, int32_t ytype, int32_t m, int32_t k, int32_t n, const void* x, int64_t ldx,
                  const void* w, int64_t ldw, const float* b, int32_t act, const void* r, int64_t ldr,
                  void* y, int64_t ldy, void* pre, int64_t ldpre, void* workspace, size_t ws_bytes,
                  void* stream);
size_t gt_linear_bwd_workspace_size(int32_t dtype, int32_t ytype, int32_t m, int32_t k, int32_t n, int32_t act,
                                    int32_t aligned);
int gt_linear_bwd(int32_t dtype, int32_t ytype, int32_t m, int32_t k, int32_t n, const void* dy, int64_t lddy,
                  const void* x, int64_t ldx, const void* w, int64_t ldw, const void* pre, int64_t ldpre,
                  int32_t act, const void* add, int64_t ldadd, void* dx, int64_t lddx, void* dw, int64_t lddw,
                  float* db, void* workspace, size_t ws_bytes, void* stream);

/*
 * Cross attention: queries of one side over the keys and values of another, of any lengths (a
 * readout of a graph by a few learned queries, a decoder over the states of the nodes).  Per query
 * i of head j, over the keys of its own sequence that are not hidden,
 *   s = scale <q_i, k>,  o = softmax(s) v,  lse = log sum exp s  (natural log)
 * and backward, with p = exp(s - lse) and D = <dO_i, o_i>,
 *   dS = p (<dO_i, v> - D),  dq = scale sum dS k,  dk = scale sum dS q,  dv = sum p dO_i.
 *   dtype   GT_BF16 (bf16 storage, tensor-core products with fp32 sums, fp32 softmax statistics;
 *           p and dS are rounded to bf16 for the products they enter) or GT_F32 (fp32 throughout).
 *   q, o, dO, dq  device [nq][h][d]; k, v, dk, dv device [nk][hk][d]; query head j reads key head
 *           j / (h / hk), whose gradients are the sums over its query heads.  Channels are
 *           contiguous; ld* is the stride of a row and hd* that of a head, in elements, so slices
 *           of a fused projection serve as they are.  Any alignment of the type is accepted; bf16
 *           inputs whose base and strides are multiples of 16 bytes are read in place, others are
 *           copied to the workspace.
 *   lse     device fp32 [h][nq].
 *   batch   sequences, packed one after another: sequence b is rows q_off[b] .. q_off[b + 1] - 1
 *           of the queries and kv_off[b] .. kv_off[b + 1] - 1 of the keys.  q_off, kv_off: device
 *           int32 [batch + 1], not falling, within [0, nq] and [0, nk] (values outside are cut
 *           to that; what falling ones give is not specified), or both NULL with batch = 1: all
 *           rows.  A sequence may have no rows on either side.  Rows in front of the first sequence
 *           and behind the last are not read into any result, and left as they were in outputs.
 *   key_mask  device uint8 [nk] or NULL: keys with 0 are seen by no query (their dk and dv are 0,
 *           and nothing of theirs, infinities and NaN included, reaches any result).
 *   A query that sees no key has o = 0, lse = -infinity and dq = 0.
 *   scale   above 0, and finite times log2 e (up to 2.35e38).
 *   workspace  at least gt_cross_attn_workspace_size bytes (`backward`: non-zero for the
 *           backward; `aligned`: non-zero when all bf16 inputs are read in place), 16-byte aligned; may
 *           be NULL where that is 0.
 * Outputs must not overlap each other or any input.  Results do not change from run to run.
 * Errors: GT_ERR_INVALID_ARG for a NULL pointer, an unknown type, a size below 1, h % hk != 0, a
 * negative stride, one of q_off and kv_off without the other, batch > 1 without them, or a bad scale;
 * GT_ERR_UNSUPPORTED for d > 128, h > 1024, h / hk > 64, batch > 2^20, nq or nk > 2^30;
 * GT_ERR_WORKSPACE.
 */
size_t gt_cross_attn_workspace_size(int32_t dtype, int32_t nq, int32_t nk, int32_t h, int32_t hk, int32_t d,
                                    int32_t batch, int32_t backward, int32_t aligned);
int gt_cross_attn_fwd(int32_t dtype, int32_t nq, int32_t nk, int32_t h, int32_t hk, int32_t d, int32_t batch,
                      const void* q, int64_t ldq, int64_t hdq, const void* k, int64_t ldk, int64_t hdk,
                      const void* v, int64_t ldv, int64_t hdv, const int32_t* q_off, const int32_t* kv_off,
                      const uint8_t* key_mask, float scale, void* o, int64_t ldo, int64_t hdo, float* lse,
                      void* workspace, size_t ws_bytes, void* stream);
int gt_cross_attn_bwd(int32_t dtype, int32_t nq, int32_t nk, int32_t h, int32_t hk, int32_t d, int32_t batch,
                      const void* q, int64_t ldq, int64_t hdq, const void* k, int64_t ldk, int64_t hdk,
                      const void* v, int64_t ldv, int64_t hdv, const void* o, int64_t ldo, int64_t hdo,
                      const void* dO, int64_t lddo, int64_t hddo, const float* lse, const int32_t* q_off,
                      const int32_t* kv_off, const uint8_t* key_mask, float scale, void* dq, int64_t lddq,
                      int64_t hddq, void* dk, int64_t lddk, int64_t hddk, void* dv, int64_t lddv, int64_t hddv,
                      void* workspace, size_t ws_bytes, void* stream);

/*
 * Which channels of a head make a pair of the rotation: i and i + rot / 2, or 2 i and 2 i + 1.
 */
typedef enum { GT_ROT_HALVES = 0, GT_ROT_PAIRS = 1 } gt_rot;

/*
 * gt_qk_norm_fwd: the norm of every head of the queries and of the keys, and the rotation of their
 * channels by position, in one pass (before gt_bias_attn_fwd or gt_cross_attn_fwd):
 *   r = 1 / sqrt(sum_c x_c^2 / d + eps),  y = R (gain x r)      (for x and eps over the whole range of fp32)
 * where R turns pair i < rot / 2 of the first rot channels, (a, b) to (a cos - b sin, a sin + b cos),
 * by the angle pos * freq[i] (radians; to fp32 accuracy for any int32 position while |freq| < 2^24),
 * and leaves the channels past rot.
 *   xtype, ytype  element types of q and k, and of yq and yk: any pair.
 *   freq    device fp32 [rot / 2]; NULL with rot = 0: the norm alone.  rot even, 0 <= rot <= d.
 *   q, yq   device [nq][h][d], k, yk device [nk][hk][d], channels contiguous, strides of rows (ld*)
 *           and heads (hd*) in elements, any alignment; k NULL: the queries alone.  An output may
 *           be its own input (same type, address and strides).
 *   gain_q, gain_k  device fp32 [d].
 *   pos_q, pos_k    device int32 [nq], [nk]; NULL: the row's index.
 * Errors: GT_ERR_INVALID_ARG for a NULL pointer, an unknown type or pairing, a size below 1, a bad
 * rot, freq with rot = 0 or rot without freq, a negative stride, or an eps that is not finite and
 * positive; GT_ERR_UNSUPPORTED for d > 256, h or hk > 1024.
 *
 * gt_qk_norm_bwd: from dy = dL/dy (y's type), with g = R^T dy and w = gain g,
 *   dx = r (w - x r^2 sum_c w_c x_c / d),  dgain = sum over rows and heads of g x r
 *   dq, dk have x's type (either may be its own dy where the types are one), dgain_q, dgain_k are
 *   device fp32 [d] (outputs, overwritten).  Nothing of the forward is needed but its inputs.
 *   workspace  at least gt_qk_norm_workspace_size(d) bytes (0 for a d that is not supported).
 * Errors as the forward's, plus GT_ERR_WORKSPACE.  Results do not change from run to run.
 */
int gt_qk_norm_fwd(int32_t xtype, int32_t ytype, int32_t d, float eps, const float* freq, int32_t rot, int32_t pairs,
                   int32_t nq, int32_t h, const void* q, int64_t ldq, int64_t hdq, const float* gain_q,
                   const int32_t* pos_q, void* yq, int64_t ldyq, int64_t hdyq, int32_t nk, int32_t hk,
                   const void* k, int64_t ldk, int64_t hdk, const float* gain_k, const int32_t* pos_k, void* yk,
                   int64_t ldyk, int64_t hdyk, void* stream);
size_t gt_qk_norm_workspace_size(int32_t d);
int gt_qk_norm_bwd(int32_t xtype, int32_t ytype, int32_t d, float eps, const float* freq, int32_t rot, int32_t pairs,
                   int32_t nq, int32_t h, const void* dyq, int64_t lddyq, int64_t hddyq, const void* q, int64_t ldq,
                   int64_t hdq, const float* gain_q, const int32_t* pos_q, void* dq, int64_t lddq, int64_t hddq,
                   float* dgain_q, int32_t nk, int32_t hk, const void* dyk, int64_t lddyk, int64_t hddyk,
                   const void* k, int64_t ldk, int64_t hdk, const float* gain_k, const int32_t* pos_k, void* dk,
                   int64_t lddk, int64_t hddk, float* dgain_k, void* workspace, size_t ws_bytes, void* stream);

/*
 * gt_grad_clip: the norm of all gradients of a step together, and each of them scaled so that it
 * does not exceed max_norm:
 *   norm = sqrt(sum over all tensors of g^2),  out = g (norm <= max_norm ? 1 : max_norm / norm)
 * over the whole range of fp32 (squares that leave it are summed in fp64, and a quotient below 2^-126 multiplies in fp64;
 * a norm past the range is stored as infinity, and the gradients are scaled by what it is).
 *   list    host array of `count` tensors, read during the call only.  g: device, numel elements
 *           in a row, of gtype; out: device, of otype (output: it may be g itself with the same
 *           type; NULL: the tensor only counts).  numel may be 0.  No output may overlap another
 *           or another tensor's g.
 *   max_norm  0 or more; infinity only measures (out is g in otype).  A sum of squares that is
 *           not finite scales by max_norm / norm all the same: 0 for infinity, NaN for NaN.
 *   norm    device fp32 [1] (output).
 *   workspace  at least gt_grad_clip_workspace_size(count) bytes, 16-byte aligned.
 * Errors: GT_ERR_INVALID_ARG for a NULL list, norm or g, count < 1, an unknown type, out = g of
 * another type, or a max_norm that is negative or NaN; GT_ERR_UNSUPPORTED for numel > 2^40 or more
 * than 2^40 elements in 256 consecutive tensors; GT_ERR_WORKSPACE.  Results do not change from run to run.
 */
typedef struct {
    const void* g;
    void* out;
    int64_t numel;
    int32_t gtype, otype;
} gt_grad;
size_t gt_grad_clip_workspace_size(int32_t count);
int gt_grad_clip(const gt_grad* list, int32_t count, float max_norm, float* norm, void* workspace, size_t ws_bytes,
                 void* stream);

/* Static English text for a gt_status value. */
const char* gt_status_string(int status);

/*
 * Synchronises `stream`, then reports GT_ERR_TIMEOUT if any kernel of this
 * library gave up a bounded wait since the last check (kernels never spin
 * without a limit; on giving up they record it in a device status word and
 * return), GT_ERR_CUDA if the stream reports an error, else GT_OK.  The status
 * word is cleared by the call.
 */
int gt_check_device_status(void* stream);

/*
 * Self-test of the bounded waits (no counterpart in the method): launches one
 * CTA on `stream` whose wait on a barrier that nothing arrives at gives up after
 * limit_ns nanoseconds of wall time, exactly as a kernel's wait would; the next
 * gt_check_device_status then reports GT_ERR_TIMEOUT and the context stays
 * usable.  1e6 <= limit_ns <= 1e9, else GT_ERR_INVALID_ARG.
 */
int gt_selftest_wait_timeout(int64_t limit_ns, void* stream);

/*
 * Launch statistics (a measurement aid; no counterpart in the method).
 *
 * The library counts, per kernel name, every kernel it launches.  With timing
 * on, each launch is also bracketed by two CUDA events recorded on the
 * launching stream (events come from a pool the library creates on demand and
 * keeps), so the sum of (end - start) per name is the device time of that
 * kernel's launches, queueing behind earlier work on the stream excluded.
 * Timing adds two event records per launch; leave it off while timing whole
 * steps.  The table is process-wide and guarded by a mutex; with timing on,
 * use one CUDA device per process.
 *
 *   gt_kernel_stats_reset(timing)  clears the table (waiting for events still
 *       pending) and sets timing on (non-zero) or off.  Returns GT_OK or
 *       GT_ERR_CUDA.
 *   gt_kernel_stats_read(out, cap, count)  waits for the recorded events, sets
 *       *count to the number of distinct kernel names seen since the reset and
 *       fills min(cap, *count) entries of out (host memory, caller-owned) in
 *       first-launch order; total_ms is -1 when timing is off.  Returns
 *       GT_ERR_INVALID_ARG for count == NULL, cap < 0 or out == NULL with
 *       cap > 0, GT_ERR_CUDA if an event query fails, else GT_OK.
 */
typedef struct {
    char name[40];      /* NUL-terminated kernel name, e.g. "bwd_dq" */
    int64_t launches;   /* launches since the last reset */
    double total_ms;    /* summed device time of those launches (timing on) */
} gt_kernel_stat;

int gt_kernel_stats_reset(int32_t timing);
int gt_kernel_stats_read(gt_kernel_stat* out, int32_t cap, int32_t* count);

#ifdef __cplusplus
}
#endif
#endif /* GT_ATTN_H */
