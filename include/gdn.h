/* gdn.h - C ABI of the GB300 GDN speculative tree-verify library.
 *
 * One speculative round of a hybrid model's Gated DeltaNet (GDN) layer, for a
 * batch of sequences whose draft tokens form trees:
 *
 *   gdn_conv_tree_step  depthwise causal conv (4 taps) + SiLU over each token
 *                       tree, reading the conv history through a slot map;
 *                       also emits each node's conv commit window.
 *   gdn_tree_verify     gated delta rule over each tree with the gates and the
 *                       q/k L2 norm computed in the kernel; reads the
 *                       recurrent state read-only from its slot and emits the
 *                       attention output and one replay row per node and head.
 *   gdn_chain_verify    the same verify for batches of chains (node i's parent
 *                       is node i - 1), in chunked form.
 *   gdn_commit          once acceptance is known, advances the persistent conv
 *                       and recurrent state of every sequence by its accepted
 *                       root-to-node path, on the device, as one transaction.
 *
 * and what stands around it in a hybrid model's round: the full-attention
 * layers (gdn_rope_append, gdn_paged_attention, gdn_kv_commit), the same over a
 * cache held in 4 bits (gdn_kvq_append, gdn_paged_attention_kvq, gdn_kvq_commit),
 * the way from logits to probabilities (gdn_logits_probs, gdn_token_commit) and
 * the decision on the drafted tokens (gdn_tree_accept).
 *
 * Sources (page title, section):
 *   lucebox PR #707 "perf(qwen35): fuse the DFlash2 concurrent verify Gated
 *     DeltaNet route" - Optimizations: ssm_conv_tree_step, the read-only
 *     mapped recurrence, gate preparation inside the recurrence; Validation:
 *     persistent state unchanged by verify.
 *   lucebox PR #659 "perf(qwen38): various DFlash2 optimizations concurrency
 *     C1-C5" - Summary item 3 (replay rows of width 257 at state size 128);
 *     test list (padded/permuted slots, transaction preflight); review note on
 *     running the commit on the compute stream.
 *   TensorSharp PR #175 "Feature/support dflash2" - committing the accepted
 *     prefix on the device instead of restore + re-forward; state kept in its
 *     own buffer, read and written as separate in/out.
 *   lucebox PR #625 "qwen35: DSpark speculative decoding" - raw gates
 *     sigmoid(beta) and softplus(alpha + dt_bias) * A applied in the kernel;
 *     one L2 norm over q|k; q/k heads broadcast to the value heads.
 *   llama-cpp-bonsai "llama-cpp-bonsai-gdn-conv.patch" - conv input column
 *     order (history then tokens) and tap/accumulation order.
 *   Yang, Kautz & Hatamizadeh, "Gated Delta Networks" (ICLR 2025) - the
 *     recurrence S_t = a_t S_{t-1} (I - b_t k_t k_t^T) + b_t v_t k_t^T.
 *
 * Conventions shared by every call
 * --------------------------------
 * Memory.  Every pointer argument except `dims` is CUDA device memory on the
 *   current device, owned by the caller (e.g. a torch tensor's data_ptr).  The
 *   library allocates no device memory and keeps no state between calls
 *   (the TMA descriptor of the state pool is encoded on the host per call).
 *   Float tensors are fp32, index tensors int32, all row-major and dense
 *   unless a stride is given.  Pointers to float tensors must be 16-byte
 *   aligned; strides given in floats must be multiples of 4.
 * Shapes.  S = n_seqs, N = n_nodes (all sequences), P = n_slots, d = d_k = d_v
 *   in {16, 32, 64, 128}, H_v a multiple of H_k, G = H_v / H_k, d_conv = 4,
 *   C = 2 H_k d + H_v d conv channels in the order q (H_k d) | k (H_k d) |
 *   v (H_v d).  Sequence s owns nodes node_off[s] .. node_off[s+1]-1
 *   (node_off[0] = 0, node_off[S] = N); N_s = node_off[s+1] - node_off[s]
 *   <= max_seq_nodes <= 64.  parents[n] is the parent's index local to the
 *   sequence, or -1 for a root (which starts from the slot's state and conv
 *   history); a parent precedes its child.  Value head h reads q/k head
 *   floor(h / G).
 * Streams.  All work is enqueued on `stream` (a cudaStream_t; NULL = the
 *   legacy default stream) and is asynchronous.  verify -> acceptance (by
 *   gdn_tree_accept or by the host) -> commit must be ordered by the caller's
 *   stream; gdn_tree_accept does not release its dependents early, so the
 *   commits may follow it directly.  The
 *   library's kernels use programmatic dependent launch: each may start
 *   while the previous kernel on the stream finishes, and waits for it to
 *   complete before touching any buffer the library writes.  They may read
 *   the pure inputs (parents, node_off, slot_map, accepted, win_ref) before
 *   that wait, so a caller that produces those in a kernel on the same stream
 *   must not let that kernel trigger its dependents early
 *   (cudaTriggerProgrammaticLaunchCompletion / griddepcontrol.launch_dependents
 *   before its writes); a plain launch, or a copy, is always safe.
 * Access.  gdn_conv_tree_step and gdn_tree_verify never write the state pools
 *   (`conv_hist`, `ssm`).  Only gdn_commit writes them.  No float atomics:
 *   results are bit-for-bit reproducible run to run.
 * Errors.  The return value is a host-side status: GDN_OK or a negative
 *   GDN_ERR_* (nothing was enqueued).  Errors that need the index data are
 *   found on the device and written to `*status` (a device int32 the caller
 *   zeroes; the first error wins).  After a device error the outputs of that
 *   call are unspecified; gdn_commit writes nothing at all (it checks every
 *   sequence before the first write, and also refuses to run when `*status`
 *   is already non-zero on entry, e.g. after a failed verify).  Kernels never
 *   trap; every wait in a kernel is bounded and reports GDN_DEV_TIMEOUT.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int32_t n_seqs;         /* S                                                 */
    int32_t n_nodes;        /* N, tree nodes over all sequences                  */
    int32_t n_slots;        /* P, slots in the conv-history and state pools      */
    int32_t h_k;            /* q/k heads                                         */
    int32_t h_v;            /* value heads (multiple of h_k)                     */
    int32_t d_k;            /* key width   (= d_v, in {16, 32, 64, 128})         */
    int32_t d_v;            /* value width                                       */
    int32_t d_conv;         /* conv taps, must be 4                              */
    int32_t max_seq_nodes;  /* bound on any N_s, 1..64; selects the kernel       */
} gdn_dims;

/* host-side return codes */
enum {
    GDN_OK = 0,
    GDN_ERR_NULL = -1,         /* a required pointer is NULL                      */
    GDN_ERR_DIMS = -2,         /* inconsistent or unsupported dims                */
    GDN_ERR_STRIDE = -3,       /* a stride is smaller than its row or not % 4     */
    GDN_ERR_ALIGN = -4,        /* a float pointer is not 16-byte aligned          */
    GDN_ERR_ALIAS = -5,        /* an output overlaps an input or another output  */
    GDN_ERR_LAUNCH = -6,       /* the CUDA launch failed (cudaGetLastError)       */
    GDN_ERR_TMA = -7,          /* the TMA descriptor of the state pool failed     */
    GDN_ERR_ARG = -8           /* an argument outside its allowed values          */
};

/* device-side codes written to *status */
enum {
    GDN_DEV_BAD_NODE_OFF = 1,  /* node_off not 0..N non-decreasing, or N_s > max  */
    GDN_DEV_BAD_PARENT = 2,    /* parents[n] outside [-1, local index)            */
    GDN_DEV_BAD_SLOT = 3,      /* slot_map[s] outside [0, P)                      */
    GDN_DEV_DUP_SLOT = 4,      /* two committing sequences share a slot           */
    GDN_DEV_BAD_ACCEPTED = 5,  /* accepted[s] outside [-1, N_s)                   */
    GDN_DEV_TIMEOUT = 6,       /* a bounded wait in a kernel ran out              */
    GDN_DEV_BAD_WINDOW = 7,    /* a window reference outside [-3, N) (compact)    */
    GDN_DEV_BAD_PAGE = 8,      /* a page index outside [0, n_pages)               */
    GDN_DEV_BAD_LEN = 9,       /* ctx_len[s] < 0, or the new tokens pass the table */
    GDN_DEV_BAD_AXIS = 10,     /* axis[i] outside [0, n_axes) (rope)              */
    GDN_DEV_BAD_TOKEN = 11,    /* a token outside [0, vocab), or (bias) out of order */
    GDN_DEV_BAD_BIAS = 12,     /* bias_off not 0 <= .. <= n_bias, non-decreasing  */
    GDN_DEV_BAD_MASK = 13      /* mask_row[n] outside [-1, n_masks)               */
};

/* Conv tree step (lucebox PR #707, Optimizations: fused convolution
 * preparation; conv arithmetic as in llama-cpp-bonsai-gdn-conv.patch).
 * For node t of sequence s, let P_t be the column sequence
 *     h_0, h_1, h_2, x(root), ..., x(parent of t), x(t)
 * with h = conv_hist[slot_map[s]] (h_2 newest).  Then
 *     xc[t][c]     = SiLU( sum_{j=0..3} P_t[-4 + j][c] * conv_w[c][j] )
 * summed in tap order j = 0 (oldest) .. 3 (= x(t)), no bias, and
 *     win[t][j][c] = P_t[-3 + j][c]           j = 0..2 (oldest first)
 * the raw columns that become the slot's history if t is accepted.
 *   x         [N][x_stride] in, first C floats of each row used
 *   conv_w    [C][4]        in
 *   conv_hist [P][3][C]     in (read-only here)
 *   parents   [N], node_off [S+1], slot_map [S]   in
 *   xc        [N][C]        out
 *   win       [N][3][C]     out
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_PARENT, GDN_DEV_BAD_SLOT. */
int gdn_conv_tree_step(const gdn_dims *dims, const float *x, int64_t x_stride,
                       const float *conv_w, const float *conv_hist,
                       const int32_t *parents, const int32_t *node_off,
                       const int32_t *slot_map, float *xc, float *win,
                       int32_t *status, void *stream);

/* Tree verify (lucebox PR #707, Optimizations: read-only mapped recurrence and
 * gate preparation inside the recurrence; lucebox PR #659, Summary item 3).
 * For node t (topological order) and value head h, with k-head j = h / G:
 *     q = xc[t][j d ..], k = xc[t][H_k d + j d ..], v = xc[t][2 H_k d + h d ..]
 *     q^ = q / sqrt(|q|^2 + 1e-6),  k^ likewise
 *     beta = sigmoid(ba[t][h]),  decay = exp(softplus(ba[t][H_v + h] + dt_bias[h]) * A[h])
 *     S'   = decay * S_parent         (S_parent of a root = ssm[slot_map[s]][h])
 *     u    = beta * (v - S' k^)
 *     S_t  = S' + u k^T               (= decay S_p (I - beta k^ k^T) + beta v k^T)
 *     o[t][h] = q_scale * S_t q^
 *     replay[t][h] = k^ (d) | u (d) | decay (1)
 * S is [d_v][d_k] (row = value index).  ssm is only read.  softplus(x) = x
 * above 20.
 *   xc       [N][C] in (dense)         ba [N][ba_stride] in (b | a; stride >= 2 H_v)
 *   dt_bias  [H_v], A [H_v]  in        ssm [P][H_v][d][d] in (read-only)
 *   o        [N][H_v][d]  out
 *   replay   [N][H_v][replay_stride] out; replay_stride >= 2d + 1 and % 4 == 0
 *            (gdn_replay_row_floats gives the smallest); floats past 2d + 1
 *            in a row are not written
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_PARENT, GDN_DEV_BAD_SLOT,
 * GDN_DEV_TIMEOUT. */
int gdn_tree_verify(const gdn_dims *dims, const float *xc, const float *ba,
                    int64_t ba_stride, const float *dt_bias, const float *A,
                    const float *ssm, float q_scale, const int32_t *parents,
                    const int32_t *node_off, const int32_t *slot_map, float *o,
                    float *replay, int64_t replay_stride, int32_t *status,
                    void *stream);

/* Chain verify (lucebox PR #707, Scope and fallback: dense chains keep a path
 * of their own; TensorSharp PR #175, change 1: a run of tokens goes through a
 * chunked GDN kernel).  The same operation, arguments, outputs and replay rows
 * as gdn_tree_verify, for batches in which every sequence's nodes form a chain
 * (parents[node_off[s] + i] = i - 1), d = 128 only.  It evaluates the chain in
 * chunks of 16 nodes and carries the state on chip between them, so long
 * chains (up to max_seq_nodes = 64) cost little more per node than short ones.
 * The replay rows feed gdn_commit / gdn_commit_compact unchanged.
 * Host errors: as gdn_tree_verify, and GDN_ERR_DIMS when d != 128.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_SLOT, GDN_DEV_BAD_PARENT
 * (a sequence that is not a chain; its outputs are not written),
 * GDN_DEV_TIMEOUT. */
int gdn_chain_verify(const gdn_dims *dims, const float *xc, const float *ba,
                     int64_t ba_stride, const float *dt_bias, const float *A,
                     const float *ssm, float q_scale, const int32_t *parents,
                     const int32_t *node_off, const int32_t *slot_map, float *o,
                     float *replay, int64_t replay_stride, int32_t *status,
                     void *stream);

/* Replay-log commit (lucebox PR #707, Summary; TensorSharp PR #175 on-device
 * commit; lucebox PR #659 transaction preflight and stream ordering).
 * accepted[s] in {-1} U [0, N_s): -1 commits nothing for s.  Otherwise the
 * path root .. accepted[s] is found by walking parents, and for every head h
 *     S <- decay_j S + u_j k^_j^T     for j along the path, root first
 * on ssm[slot_map[s]][h] (k^, u, decay from the replay rows), and
 *     conv_hist[slot_map[s]] <- win[accepted[s]].
 * A preflight checks node_off, accepted, the parent walk and that no two
 * committing sequences share a slot; if any check fails (or *status is
 * already non-zero) nothing is written.
 *   accepted [S] in; parents, node_off, slot_map in; replay, win in (as
 *   produced by verify and conv for this round); ssm, conv_hist in/out.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_ACCEPTED,
 * GDN_DEV_BAD_PARENT, GDN_DEV_BAD_SLOT, GDN_DEV_DUP_SLOT. */
int gdn_commit(const gdn_dims *dims, const int32_t *accepted, const int32_t *parents,
               const int32_t *node_off, const int32_t *slot_map, const float *replay,
               int64_t replay_stride, const float *win, float *ssm, float *conv_hist,
               int32_t *status, void *stream);

/* Compact commit windows (lucebox PR #707, Optimizations: the conv tree step
 * also produces the commit window; a window is three columns of the node's
 * column sequence, so it can be named instead of copied).
 * gdn_conv_tree_step_compact computes xc exactly as gdn_conv_tree_step but,
 * instead of the window rows, writes for every node t
 *     win_ref[t][j], j = 0..2 (oldest first)
 * naming column j of t's commit window: a global node index n >= 0 (the
 * window column is x row n) or -1 - k for column h_k of the slot's history.
 * gdn_commit_compact then performs gdn_commit with the accepted node's window
 * gathered through win_ref from x and from the slot's history as it stands
 * before the commit; the caller keeps x (and its stride) unchanged from the
 * conv call to the commit.  This saves the 3 C floats per node that
 * gdn_conv_tree_step writes and the commit reads.
 *   win_ref  [N][3] int32 out (conv) / in (commit); x, x_stride as for conv.
 * Device errors: as the non-compact calls, plus GDN_DEV_BAD_WINDOW (commit:
 * a reference of an accepted node outside [-3, N); nothing is written). */
int gdn_conv_tree_step_compact(const gdn_dims *dims, const float *x, int64_t x_stride,
                               const float *conv_w, const float *conv_hist,
                               const int32_t *parents, const int32_t *node_off,
                               const int32_t *slot_map, float *xc, int32_t *win_ref,
                               int32_t *status, void *stream);

int gdn_commit_compact(const gdn_dims *dims, const int32_t *accepted, const int32_t *parents,
                       const int32_t *node_off, const int32_t *slot_map, const float *replay,
                       int64_t replay_stride, const float *x, int64_t x_stride,
                       const int32_t *win_ref, float *ssm, float *conv_hist, int32_t *status,
                       void *stream);

/* Gated RMS norm, the output stage after the recurrence (TensorSharp PR #175,
 * the Qwen 3.5 / Qwen4Exp GDN block: gated delta net -> gated norm; the output
 * gate is a SiLU, gate_mode 0, or a sigmoid, gate_mode 1).  For node t, value
 * head h and i < d:
 *     y[t][h][i] = o[t][h][i] / sqrt(mean_i(o[t][h][.]^2) + eps) * norm_w[i]
 *                  * gate(z[t][h d + i])
 *   o       [N][H_v][d] in (e.g. gdn_tree_verify's output)
 *   z       [N][z_stride] in, z_stride >= H_v d and % 4 == 0
 *   norm_w  [d] in (one weight vector shared by the heads)
 *   eps     >= 0 (eps = 0 with an all-zero head gives NaN)
 *   y       [N][H_v][d] out (must not overlap the inputs)
 * Host errors: GDN_ERR_ARG for gate_mode outside {0, 1} or eps < 0 / not
 * finite.  No device errors. */
int gdn_gated_rmsnorm(const gdn_dims *dims, const float *o, const float *z, int64_t z_stride,
                      const float *norm_w, float eps, int gate_mode, float *y, void *stream);

/* Plain decode step (TensorSharp PR #175: a step without speculation commits
 * its post-window state at once, the caller's "slot -1"; lucebox PR #625:
 * ggml_ssm_conv_step with in-place history write-back and the raw-gate gated
 * delta net in place).  One token per sequence: dims->n_nodes must equal
 * dims->n_seqs and token s belongs to sequence s.  For each s, with
 * h = conv_hist[slot_map[s]] and the column sequence P = [h_0, h_1, h_2, x_s]:
 *     xc[s][c] = SiLU(sum_{j=0..3} P[j][c] conv_w[c][j]);   h <- [h_1, h_2, x_s]
 * and for every value head h with the gates and normalised q/k of
 * gdn_tree_verify:
 *     S <- decay S;  u = beta (v - S k^);  S <- S + u k^T;  o[s][h] = q_scale S q^
 * on ssm[slot_map[s]][h] in place.  This is gdn_conv_tree_step +
 * gdn_tree_verify + gdn_commit on one-node trees with every node accepted,
 * without the windows and replay rows.
 *   x [S][x_stride] in; conv_w in; conv_hist, ssm in/out; ba [S][ba_stride] in;
 *   dt_bias, A in; slot_map [S] in; xc [S][C] out; o [S][H_v][d] out.
 * Device errors: GDN_DEV_BAD_SLOT, GDN_DEV_DUP_SLOT (two sequences in one
 * slot); on any error (or a non-zero *status on entry) nothing is written. */
int gdn_decode_step(const gdn_dims *dims, const float *x, int64_t x_stride, const float *conv_w,
                    float *conv_hist, const float *ba, int64_t ba_stride, const float *dt_bias,
                    const float *A, float *ssm, float q_scale, const int32_t *slot_map, float *xc,
                    float *o, int32_t *status, void *stream);

/* Attention layers of the round
 * -----------------------------
 * A hybrid model runs full-attention layers between its GDN layers.  Their keys
 * and values live in a paged cache: pools of n_pages pages of page_size tokens,
 * and a page table that names, for each sequence, the page of each run of
 * page_size positions.  Position x of sequence s is token x % page_size of page
 * page_table[s][x / page_size].  Sequence s has ctx_len[s] cached positions; the
 * new token i of this call (tokens node_off[s] .. node_off[s + 1] - 1 of the
 * batch, as for the trees above) takes position ctx_len[s] + i.
 *   gdn_rope_append      writes the new tokens' keys and values there
 *   gdn_paged_attention  reads them together with the context
 *   gdn_kv_commit        once acceptance is known, moves the accepted path's
 *                        keys and values to positions ctx_len[s] + 0, 1, ...
 * Positions from ctx_len[s] on are written: their pages belong to s alone.  Pages
 * that hold only earlier positions may be in any number of sequences' tables.
 * 16-bit tensors hold bf16 or fp16 (dims->dtype).  Both pools have the same
 * strides, in elements, so a cache of [page][token][head][d], of
 * [page][head][token][d] or one that interleaves keys and values all work. */
enum { GDN_BF16 = 0, GDN_FP16 = 1, GDN_FP32 = 2 };  /* FP32: gdn_logits_probs only */

typedef struct {
    int32_t n_seqs;          /* S                                                   */
    int32_t n_tokens;        /* N, new tokens over all sequences                    */
    int32_t max_seq_tokens;  /* bound on any sequence's new tokens                  */
    int32_t h_q;             /* query heads (multiple of h_kv, h_q / h_kv <= 128)   */
    int32_t h_kv;            /* key/value heads                                     */
    int32_t d_head;          /* head width, in {64, 128, 256}                       */
    int32_t dtype;           /* GDN_BF16 or GDN_FP16                                */
    int32_t n_pages;         /* pages in each pool                                  */
    int32_t page_size;       /* tokens of a page: a power of two, 8..1024           */
    int32_t table_width;     /* page-table entries of a sequence                    */
    int64_t page_stride;     /* elements between pages (multiples of 8, as are ...) */
    int64_t token_stride;    /* ... between the tokens of a page                    */
    int64_t head_stride;     /* ... between the heads of a token                    */
} gdn_attn_dims;

/* q/k RMS norm, rotary positions, and the append to the cache.  For token n and
 * each head x of q (h_q of them) and k (h_kv):
 *     y = x                                             without a norm weight
 *     y = x / sqrt(mean(x^2) + eps) * w                 with one (q_norm_w, k_norm_w)
 *     phi_i = pos[n][axis[i]] * inv_freq[i]             i = 0 .. rot_dim / 2 - 1
 *     (z_a, z_b) = (y_a cos phi_i - y_b sin phi_i, y_b cos phi_i + y_a sin phi_i)
 * with (a, b) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) when `interleaved`; the
 * d_head - rot_dim other elements keep y.  q rows go to q_out, k rows and the
 * plain v rows to the pools.  A token has n_axes positions (time, height, width
 * of an image's patches, say); `axis` gives each frequency its axis, so sections
 * and interleaved layouts are both a table.  For any int32 position an angle is
 * off by |pos| (inv_freq + 1) 2^-64 + 2^-26 + 2^-32 turns at most: inv_freq / 2 pi is
 * held to 2^-64, the product modulo a turn is exact and is cut to 32 bits and rounded
 * to fp32.
 *   q [N][q_stride], k [N][k_stride], v [N][v_stride]   in, 16-bit, strides in
 *            elements, multiples of 8
 *   q_norm_w, k_norm_w  [d_head] fp32, or NULL
 *   pos      [N][n_axes] int32;  inv_freq [rot_dim / 2] fp64
 *   axis     [rot_dim / 2] int32, or NULL (axis 0);  n_axes 1..4
 *   rot_dim  a multiple of 16, 0 .. d_head (0: no rotation)
 *   q_out    [N][q_out_stride] out; may be q itself with the same stride.  q, k, v
 *            and q_out may be columns of one buffer, with its row as their stride
 * Host errors: GDN_ERR_ARG for eps, n_axes, rot_dim or interleaved.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_LEN, GDN_DEV_BAD_PAGE (the
 * token's k and v are not written), GDN_DEV_BAD_AXIS. */
int gdn_rope_append(const gdn_attn_dims *dims, const void *q, int64_t q_stride, const void *k,
                    int64_t k_stride, const void *v, int64_t v_stride, const float *q_norm_w,
                    const float *k_norm_w, float eps, const int32_t *pos, int n_axes,
                    const double *inv_freq, const int32_t *axis, int rot_dim, int interleaved,
                    const int32_t *node_off, const int32_t *ctx_len, const int32_t *page_table,
                    void *q_out, int64_t q_out_stride, void *k_pool, void *v_pool, int32_t *status,
                    void *stream);

/* Attention of the new tokens over the paged cache.  New token i of sequence s,
 * query head h, key/value head h / (h_q / h_kv):
 *     o[n][h] = sum_x p_x v_x,   p = softmax over the positions it sees of
 *               scale * q[n][h] . k_x
 * It sees the positions below ctx_len[s], itself, and of the other new tokens
 * those before it (parents NULL: a prompt's chunk, a chain, one token) or its
 * ancestors (parents as for the trees, max_seq_tokens <= 64).  What it does not
 * see has no influence, whatever it holds: NaN and infinities in the rest of a
 * page or in other branches stay there.
 *   q [N][q_stride] in (16-byte aligned rows);  o [N][h_q * d_head] out
 *   k_pool, v_pool, page_table, ctx_len, node_off, parents  in
 *   scale    finite, > 0
 *   workspace  at least gdn_attention_workspace_bytes(dims) bytes, 16-byte
 *            aligned, contents irrelevant before and after the call
 * Host errors: GDN_ERR_ARG for scale or a workspace too small.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_PARENT, GDN_DEV_BAD_LEN,
 * GDN_DEV_BAD_PAGE, GDN_DEV_TIMEOUT. */
int gdn_paged_attention(const gdn_attn_dims *dims, const void *q, int64_t q_stride,
                        const void *k_pool, const void *v_pool, const int32_t *page_table,
                        const int32_t *ctx_len, const int32_t *node_off, const int32_t *parents,
                        float scale, void *o, void *workspace, int64_t workspace_bytes,
                        int32_t *status, void *stream);

/* Workspace of gdn_paged_attention on the current device, in bytes (0 for dims
 * that the call refuses).  It does not depend on the lengths. */
size_t gdn_attention_workspace_bytes(const gdn_attn_dims *dims);

/* Commit of the accepted path in the cache, the attention layers' part of
 * gdn_commit, for n_layers layers at once (pool of layer l at k_pool +
 * l * layer_stride elements, one page table for all).  With p_0 < p_1 < ... the
 * path root .. accepted[s] (m nodes), for every layer and head
 *     position ctx_len[s] + j  <-  position ctx_len[s] + p_j        j = 0 .. m - 1
 * in k_pool and v_pool, and new_len[s] = ctx_len[s] + m.  accepted[s] = -1 moves
 * nothing (m = 0).  As for gdn_commit, a preflight checks every sequence first;
 * if a check fails, or *status is already non-zero, nothing is written.  With
 * n_layers = 0, as with n_seqs = 0, nothing is enqueued and new_len is not written.
 *   max_seq_tokens <= 64; h_q is not used (give h_kv)
 *   accepted [S], parents [N], node_off, ctx_len, page_table in; new_len [S] out
 *            (must not overlap ctx_len); layer_stride a multiple of 8
 *            and, for several layers, one that keeps their rows apart: whole pools
 *            one after the other, or layers between the pages, tokens or heads
 * Host errors: GDN_ERR_STRIDE also for layers that share rows.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_ACCEPTED,
 * GDN_DEV_BAD_PARENT, GDN_DEV_BAD_LEN, GDN_DEV_BAD_PAGE. */
int gdn_kv_commit(const gdn_attn_dims *dims, int n_layers, int64_t layer_stride,
                  const int32_t *accepted, const int32_t *parents, const int32_t *node_off,
                  const int32_t *ctx_len, const int32_t *page_table, void *k_pool, void *v_pool,
                  int32_t *new_len, int32_t *status, void *stream);

/* Attention layers over a cache held in 4 bits
 * --------------------------------------------
 * The same paged cache with 4-bit values: 4.5 bits an element instead of 16, so as
 * many sequences and positions more in the same memory, and as many fewer bytes for a
 * step that reads a long context.  The 16 elements 16 b .. 16 b + 15 of a key (or
 * value) row of a head share a scale:
 *     s    = e4m3(max |x| / (6 unit))             at most 448
 *     code = e2m1(x / (s unit))                   at most 6; 0 where s = 0
 *     x   ~= code * s * unit
 * both to nearest, a tie to the even code, of the exact quotients.  unit is a power
 * of two of the caller's choice for all of a layer's keys (k_unit) and one for its
 * values (v_unit), the same in every call on a cache: 1 serves elements of 2^-5 to
 * 2^11, and below 2^-10 unit a block loses precision, above 2688 unit it saturates.
 * 16 elements of which one is not finite get the scale NaN: all 16 read as NaN.
 * Every stored row is a function of that row alone, so a token that was verified in
 * a tree and one that was decoded by itself leave the same cache.
 *   A block (page, head) of gdn_kvq_block_bytes(dims) bytes is page_size rows of
 * d_head / 2 bytes of codes (element 2 i in the low half of byte i), then page_size
 * rows of d_head / 16 scales.  dims are those of the 16-bit cache with the strides in
 * BYTES, multiples of 16: page_stride and head_stride lie between blocks and are at
 * least a block each; token_stride is not used.  dims->dtype is that of the 16-bit
 * rows and of q and o.  k and v rows come from anywhere; gdn_rope_append turns keys
 * into such rows when its pool is one of [N][h_kv * d_head] rows: n_seqs = 1,
 * node_off = {0, N}, ctx_len = {0}, page_table = {0, 1, 2, ..}. */

/* Bytes of a block (0 for dims that the calls refuse). */
size_t gdn_kvq_block_bytes(const gdn_attn_dims *dims);

/* Quantises the new tokens' rows into the cache, token i of sequence s at position
 * ctx_len[s] + i.
 *   k [N][k_stride], v [N][v_stride]   in, 16-bit, strides in elements, multiples of 8
 *   k_unit, v_unit   powers of two, 2^-24 .. 2^24
 *   node_off, ctx_len, page_table      in;  k_pool, v_pool  in/out
 * Host errors: GDN_ERR_ARG for a unit.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_LEN, GDN_DEV_BAD_PAGE (the
 * token's rows are not written). */
int gdn_kvq_append(const gdn_attn_dims *dims, const void *k, int64_t k_stride, const void *v,
                   int64_t v_stride, float k_unit, float v_unit, const int32_t *node_off,
                   const int32_t *ctx_len, const int32_t *page_table, void *k_pool, void *v_pool,
                   int32_t *status, void *stream);

/* The other way: what the cache holds at positions start[s] + i, for token i of
 * sequence s and n_layers layers at once (pool of layer l at k_pool + l *
 * layer_stride BYTES), as 16-bit rows, rounded to dims->dtype (in range of it nothing
 * is lost: a stored value has 6 significant bits).
 *   k, v [n_layers][N][row_stride] out, row_stride in elements, a multiple of 8
 * Host errors and device errors as gdn_kvq_append (the token's rows of k and v are
 * then not written), and GDN_ERR_ARG for n_layers. */
int gdn_kvq_read(const gdn_attn_dims *dims, int n_layers, int64_t layer_stride, const void *k_pool,
                 const void *v_pool, float k_unit, float v_unit, const int32_t *node_off,
                 const int32_t *start, const int32_t *page_table, void *k, void *v,
                 int64_t row_stride, int32_t *status, void *stream);

/* gdn_paged_attention over the 4-bit cache: the same formula, arguments, masks and
 * errors, with keys and values as the cache holds them.  The products run in fp16
 * with fp32 sums, in which codes times scales are exact; for bf16 a q row is first
 * scaled by a power of two, 2^100 at most, so that its largest element, from 2^-86 on,
 * is in [2^14, 2^15) (what is then below 2^-25 is lost, and put back afterwards is the
 * factor).
 *   dims->max_seq_tokens chooses the kernel: up to 16 query rows a key/value head (8
 * for d_head 256), that is h_q / h_kv times the bound, take one made for few rows.  A
 * larger bound than a batch needs costs time: 64 single tokens of 16/2 heads of 256
 * over up to 16,384 positions take 79 us with a bound of 1 and 145 with 16, and beside
 * a chunk of 512 tokens 267 in one call, 78 and 143 in two.
 *   workspace  at least gdn_attention_kvq_workspace_bytes(dims) bytes
 * Host errors: also GDN_ERR_ARG for a unit, and for scale * k_unit from 1e38 on. */
int gdn_paged_attention_kvq(const gdn_attn_dims *dims, const void *q, int64_t q_stride,
                            const void *k_pool, const void *v_pool, float k_unit, float v_unit,
                            const int32_t *page_table, const int32_t *ctx_len,
                            const int32_t *node_off, const int32_t *parents, float scale, void *o,
                            void *workspace, int64_t workspace_bytes, int32_t *status, void *stream);

size_t gdn_attention_kvq_workspace_bytes(const gdn_attn_dims *dims);

/* gdn_kv_commit for the 4-bit cache: codes and scales of the accepted path move as
 * they are.  layer_stride in BYTES, a multiple of 16, one that keeps the layers'
 * blocks apart; otherwise its arguments, checks and errors. */
int gdn_kvq_commit(const gdn_attn_dims *dims, int n_layers, int64_t layer_stride,
                   const int32_t *accepted, const int32_t *parents, const int32_t *node_off,
                   const int32_t *ctx_len, const int32_t *page_table, void *k_pool, void *v_pool,
                   int32_t *new_len, int32_t *status, void *stream);

/* From logits to the probabilities that gdn_tree_accept takes (the target's p, and
 * a draft's q), for every node of the trees.  logits[n] is the model's row after
 * node n, so what has been produced before it is the sequence's history and the
 * tokens on the path root .. n, n's own included.  For row n of sequence s and
 * token y, with c(y) the times y was produced (history's count and the path's,
 * 32767 at most) and `seen` for c(y) > 0 or y in the prompt:
 *     x = logits[n][y]
 *     x = x > 0 ? x * (1 / repetition[s]) : x * repetition[s]      where seen
 *     x = x - frequency[s] * c(y);  x = x - presence[s] where c(y) > 0
 *     x = x + bias(y)
 *     x = -infinity                                  where the mask forbids y
 *     p[n][y] = exp((x - max) / temperature[s]) / sum               temperature > 0
 *     p[n][y] = 1 for the largest x (the lowest y among equals), else 0   otherwise
 * in fp32, each step rounded on its own.  A finite logit stays finite through the
 * penalties (at fp32's largest).  A row in which every x is -infinity becomes all
 * zeros, one with a NaN that the mask lets through all NaN.  What the mask forbids
 * has no influence, whatever it holds.
 *   dims     n_seqs, n_nodes, n_slots, max_seq_nodes
 *   vocab    1 .. 2^28
 *   dtype    of logits: GDN_BF16, GDN_FP16 or GDN_FP32
 *   logits   [N][logits_stride] in, stride in elements, a multiple of 8 and at least
 *            vocab rounded up to one; what a row holds past vocab is not used
 *   tokens [N], parents [N], node_off [S+1] in (node 0's token is read here); the
 *            tokens are read only where a penalty array is given
 *   history  [n_slots][history_stride] in, or NULL (nothing produced): bits 0..14 how
 *            often the token was produced, bit 15 that it is in the prompt; sequence
 *            s has row slot_map[s].  Stride as for logits.  slot_map is used only here
 *   repetition, frequency, presence, temperature   [S] in, or NULL (1, 0, 0, 1).
 *            Without the first three neither tokens nor history is read
 *   bias_off [S+1], bias_token, bias_value [n_bias]  in, or all NULL: sequence s has
 *            entries bias_off[s] .. bias_off[s+1] - 1, tokens in ascending order
 *   mask     [n_masks][mask_stride] words in, or NULL: bit y % 32 of word y / 32 set
 *            where y is allowed;  mask_row [N]: node n's row, -1 for none; NULL: n
 *   p        [N][p_stride] out, stride a multiple of 4 and at least vocab rounded up
 *            to one; what a row holds past vocab is left as it was
 * Host errors: GDN_ERR_ARG for vocab, dtype, n_bias or n_masks.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_PARENT, GDN_DEV_BAD_SLOT,
 * GDN_DEV_BAD_TOKEN (a token of the path, or a bias's), GDN_DEV_BAD_BIAS,
 * GDN_DEV_BAD_MASK; the row is then not written. */
int gdn_logits_probs(const gdn_dims *dims, int vocab, int dtype, const void *logits,
                     int64_t logits_stride, const int32_t *tokens, const int32_t *parents,
                     const int32_t *node_off, const int32_t *slot_map, const uint16_t *history,
                     int64_t history_stride, const float *repetition, const float *frequency,
                     const float *presence, const float *temperature, const int32_t *bias_off,
                     const int32_t *bias_token, const float *bias_value, int n_bias,
                     const uint32_t *mask, int64_t mask_stride, const int32_t *mask_row,
                     int n_masks, float *p, int64_t p_stride, int32_t *status, void *stream);

/* The round's commit of the token history: the tokens of the path root ..
 * accepted[s] (of all of a sequence's tokens, whatever their number, where accepted is
 * NULL) are counted once each in history[slot_map[s]], or with prompt = 1 marked as
 * the prompt's.  A count stops at 32767.  As for gdn_commit, a preflight checks every
 * sequence first; if a check fails, or *status is already non-zero, nothing is
 * written.  A new sequence's row is zeroed by the caller.
 *   accepted [S] or NULL, parents [N] (not read without accepted), tokens [N],
 *            node_off, slot_map in; history as above in/out
 *   dims     as above; with accepted NULL max_seq_nodes is no bound
 * Host errors: GDN_ERR_ARG for vocab or prompt.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_ACCEPTED, GDN_DEV_BAD_PARENT,
 * GDN_DEV_BAD_SLOT, GDN_DEV_DUP_SLOT, GDN_DEV_BAD_TOKEN. */
int gdn_token_commit(const gdn_dims *dims, int vocab, const int32_t *tokens,
                     const int32_t *accepted, const int32_t *parents, const int32_t *node_off,
                     const int32_t *slot_map, int prompt, uint16_t *history,
                     int64_t history_stride, int32_t *status, void *stream);

/* Acceptance of drafted trees on the device (lucebox PR #707 leaves it to the
 * host between verify and commit).  Node 0 of a sequence is its last sampled
 * token, always accepted; the other nodes are drafted, tokens[n] each, children
 * tried in the order of their index.  p[n] is the target's distribution after
 * node n, q[n] the one the draft drew n's children from.  At node t, with
 * c = 0, W = Z = 1 at first, child x with uniform u[x] and token y is
 *     accepted   if u[x] q[t][y] W < max(p[t][y] - c q[t][y], 0) Z
 * and the walk goes on at x; otherwise, in this order,
 *     c <- c + W / Z,  Z <- max(Z - q[t][y], 0),  y is taken out,
 *     W <- sum over the vocabulary of max(p[t] - c q[t], 0)
 * so that max(p - c q, 0) / W is the residual distribution of rejection
 * sampling without replacement (Z = 0, a draft with nothing left: no further
 * child is tried).  When no child is left the next token is drawn
 * from that residual (from p[t] itself when its sum is 0): the first y whose
 * cumulative sum passes u_next[s] times the total.  The tokens that come out are
 * distributed as the target's.  W, Z and the sums are good to 2^-48 of a
 * distribution's mass, and with them c to about 2^-48 (1 + W / Z) / Z a rejection.
 *   replacement  0: as above.  1: the draft draws children independently (Z
 *            stays 1 and nothing is taken out)
 *   q        NULL: the children are proposed outright (q[t][y] = 1 for them;
 *            the residual is p without the rejected tokens, W <- W - p[t][y])
 *   dims     n_seqs, n_nodes, max_seq_nodes (the GDN layers' dims as they are)
 *   p [N][p_stride], q [N][q_stride]   fp32 rows of `vocab` probabilities; strides
 *            multiples of 4 and at least vocab rounded up to one (a dense row of
 *            50003 takes 50004); what a row holds past vocab is not used
 *   tokens [N] (node 0's is not read), parents, node_off, u [N], u_next [S]  in
 *   accepted [S]   deepest accepted node (-1 for a sequence without nodes): the
 *                  argument of gdn_commit and gdn_kv_commit
 *   next_token [S] the token that follows it (-1 for a sequence without nodes)
 *   n_accepted [S] nodes of the accepted path, node 0 included
 * Rows that are not distributions give tokens in [0, vocab) of no meaning.
 * Host errors: GDN_ERR_ARG for vocab or replacement.
 * Device errors: GDN_DEV_BAD_NODE_OFF, GDN_DEV_BAD_PARENT (not before its
 * child, or a root other than node 0), GDN_DEV_BAD_TOKEN; the sequence's
 * outputs are then -1, -1 and 0. */
int gdn_tree_accept(const gdn_dims *dims, int vocab, const float *p, int64_t p_stride,
                    const float *q, int64_t q_stride, int replacement, const int32_t *tokens,
                    const int32_t *parents, const int32_t *node_off, const float *u,
                    const float *u_next, int32_t *accepted, int32_t *next_token,
                    int32_t *n_accepted, int32_t *status, void *stream);

/* Test hook for the device timeout path.  The next call that runs a
 * tensor-core verify kernel (gdn_tree_verify with d = 128 and
 * max_seq_nodes <= 16, or gdn_chain_verify) makes one role of its first CTA
 * wait on a barrier that nothing ever completes, for wait_ns (capped at the
 * library's 2 s wait limit); the wait runs out, every role of that CTA drains
 * its copies and tensor-core work and leaves (the chain kernel's other roles
 * each wait out their own limit first, so that call takes about 2 s), and the
 * call reports GDN_DEV_TIMEOUT in *status (its outputs are then unspecified).
 * The hook is consumed by that one call; calls that run another kernel leave
 * it pending.  The paper has no counterpart; it exists so that the bounded-wait
 * path can be tested without a GPU fault. */
void gdn_test_stall_next_verify(uint64_t wait_ns);

/* The same for gdn_paged_attention: the next call that launches makes one role
 * of its first CTA wait for wait_ns (capped at 2 s) on a barrier that nothing
 * ever completes, then give up; the CTA's other roles wait out their own limits
 * (about 2 s), drain and leave, and the call reports GDN_DEV_TIMEOUT.
 * gdn_paged_attention_kvq takes it in the same way.
 *   role  0 softmax and results, 1 copies, 2 scores, 3 values' products,
 *         4 cleaning of values (with the 4-bit cache its conversion; where a call
 *         of that has 16 query rows a key/value head at most, 8 for d = 256, 1 is
 *         one of the copying warps and the others are working warps); any other is ignored */
void gdn_test_stall_next_attention(uint64_t wait_ns, int role);

/* Name of a host or device status code ("GDN_OK", "GDN_DEV_DUP_SLOT", ...);
 * "unknown" for any other value.  Never NULL. */
const char *gdn_status_str(int code);

/* Smallest replay_stride for widths d_k, d_v: d_k + d_v + 1 rounded up to a
 * multiple of 4 floats (260 at d = 128).  0 for unsupported widths. */
size_t gdn_replay_row_floats(int d_k, int d_v);

#ifdef __cplusplus
}
#endif
#endif /* GDN_H */
