/*
 * treeverify — target-side verification of an EAGLE draft-token tree on one
 * NVIDIA GB300 (sm_103a).  C ABI.
 *
 * One decode step of speculative decoding, as the pages on EAGLE describe it:
 * the draft head proposes a tree of candidate tokens, and the target model
 * verifies every root-to-leaf path in ONE forward pass under a tree-shaped
 * attention mask ("vLLM-TreeEagle", section 核心组件 / TreeAttentionLayer and
 * 技术创新点 / 1. Tree Attention并行验证), keeps the longest verified path and
 * truncates at the first rejection ("P-EAGLE in vLLM", 技术原理和实现方式,
 * steps 3-4), and then moves the kept entries of the KV cache into place
 * ("EAGLE code principles", KV缓存优化: KVCache.copy with index_select /
 * narrow / copy_).  The four calls below are those steps, in order:
 *
 *   tree_mask_build        parent array -> ancestor bitmask, depth
 *   tree_verify_attention  tree-masked, split-KV, paged GQA attention
 *   tree_accept            greedy argmax or rejection-sampling acceptance
 *   kv_compact             gather-then-scatter of the accepted K/V rows
 *
 * Beside them: growing the tree (draft_tree_expand), writing its K/V rows
 * (tree_kv_append), the prompts and plainly decoded tokens of the same cache
 * (chunk_kv_append, chunk_attention), and what the model's rows go through before
 * acceptance reads them (tree_logits_process, token_counts_update).  The same cache in
 * 8 bits, for prompts, decoded tokens and trees alike (chunk_kv_append_q8,
 * chunk_attention_q8, kv_compact_q8), and the sampling of rows (logits_sample).
 *
 * Conventions shared by all calls
 * -------------------------------
 * - Tree: N nodes (1 <= N <= 64).  Node 0 is the root: the last token the
 *   target already emitted, parent -1.  Nodes are in topological order:
 *   0 <= parents[i] < i for i >= 1.  Node i's K/V rows were written into the
 *   paged cache at logical position prefix_len + i before attention runs; its
 *   rotary position is prefix_len + depth(i) (applied by the caller).
 * - Paged KV cache: [num_blocks][Hkv][block_size][d] elements, row-major.
 *   Logical position t of sequence b lives in block block_table[b][t / bs],
 *   row t % bs.  block_table is [B][max_blocks_per_seq] int32.
 * - All pointer arguments are DEVICE pointers owned by the caller, unless a
 *   parameter says otherwise.  The library never allocates device memory:
 *   calls that need scratch take a caller-provided workspace whose size is
 *   given by the matching *_workspace() query.
 * - Every call is asynchronous on `stream` (NULL = the legacy default
 *   stream) and never synchronises with the host.
 * - The return value reports argument/shape errors (checked on the host
 *   before anything is launched: nothing is launched when it is not TV_OK)
 *   and launch failures (TV_ERR_CUDA).  Data-dependent errors are written to
 *   the per-sequence device array `status[B]` (TV_OK or an error code), and
 *   the affected sequence's outputs take a documented, defined value.  No
 *   kernel traps, asserts or waits without bound: a wait that runs out
 *   (about one second) records TV_ERR_TIMEOUT in status.
 * - Calls that overlap on the GPU must not share a workspace.
 */
#ifndef TREEVERIFY_H
#define TREEVERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
/* Identical to cudaStream_t. */
typedef struct CUstream_st* tv_stream_t;

typedef enum {
    TV_OK = 0,
    TV_ERR_INVALID_ARG = 1,  /* host: null pointer, bad size or shape            */
    TV_ERR_BAD_TREE = 2,     /* device: parent array violates the conventions     */
    TV_ERR_OUT_OF_RANGE = 3, /* device: block id, position, token id or length    */
    TV_ERR_UNSUPPORTED = 4,  /* host: shape/dtype not built                       */
    TV_ERR_CUDA = 5,         /* host: a CUDA runtime call or launch failed        */
    TV_ERR_TIMEOUT = 6,      /* device: a bounded wait ran out                    */
    TV_ERR_BAD_VALUES = 7,   /* device: an all-NaN logit row or a zero-mass
                                distribution where a token must be chosen         */
    TV_ERR_WORKSPACE = 8     /* host: workspace missing or too small; device
                                (draft_tree_expand): no state from the previous
                                layer in the workspace                          */
} tv_status;

typedef enum { TV_F32 = 0, TV_BF16 = 1 } tv_dtype;
typedef enum {
    TV_ACCEPT_GREEDY = 0,
    TV_ACCEPT_STOCHASTIC = 1,
    TV_ACCEPT_GREEDY_MASKED = 2
} tv_accept_mode;

/* Static description of a status code.  Never NULL. */
const char* tv_status_string(int status);

/* ABI version of this header (incremented on any signature change). */
int tv_abi_version(void);

/* ------------------------------------------------------------------------
 * Node counts ("P-EAGLE in vLLM", practice 5: shapes are kept fixed so that
 * CUDA graphs stay valid while the drafts change).  tree_mask_build,
 * tree_verify_attention(_noalloc), tree_accept and tree_kv_append take
 * node_counts: a device int32 [B] array, or NULL for trees of N nodes.  With
 * it, sequence b's tree is its first node_counts[b] nodes (node_counts[b] in
 * [1, N]; the other slots are absent and may hold anything): absent nodes get
 * no mask bits and depth -1, no attention output row (their rows of `out` are
 * not written) and are never attended (the keys are positions
 * 0 .. P_b + node_counts[b] - 1), are never accepted (a chain of
 * node_counts[b] nodes has node_counts[b] - 1 drafts, and the draw indices
 * that the rules below write as N read node_counts[b]), and are not
 * appended.  A count outside [1, N] gives the sequence TV_ERR_OUT_OF_RANGE
 * with that call's error outputs.  The values are read on the device, so one
 * captured graph serves every count vector.
 * ------------------------------------------------------------------------ */

/* ------------------------------------------------------------------------
 * tree_mask_build — "vLLM-TreeEagle", 核心组件 / 1. TreeAttentionLayer: the
 * tree attention mask is built dynamically for an arbitrary path structure.
 *
 *   mask[b][i]  bit j set  <=>  node j is node i or one of its ancestors
 *   depth[b][i] number of edges from the root to node i
 *
 * parents: int32 [B][N]; mask: uint64 [B][N]; depth: int32 [B][N] or NULL;
 * status: int32 [B].  A sequence whose parent array breaks the conventions
 * gets status TV_ERR_BAD_TREE, mask 0 and depth -1 for every node.
 * Host errors: B < 0, N outside [1, 64], a NULL required pointer.
 * ------------------------------------------------------------------------ */
tv_status tree_mask_build(const int32_t* parents, int B, int N, const int32_t* node_counts,
                          uint64_t* mask, int32_t* depth, int32_t* status, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * tree_verify_attention — "vLLM-TreeEagle", 技术创新点 / 1. Tree Attention
 * 并行验证 (one forward pass verifies all candidate paths under the tree
 * mask) and "P-EAGLE in vLLM", 技术原理和实现方式 step 3.
 *
 * For node i of sequence b and query head h (kv head g = h / (Hq / Hkv)):
 *   keys   K = { logical positions 0 .. P_b-1 } U { P_b + a : bit a of mask[b][i], a < N }
 *   O[b][i][h] = sum_{t in K} softmax_t(scale * q . k_t) v_t
 * with P_b = prefix_lens[b]; mask bits >= N are ignored; a node with no
 * visible key gets a zero output.
 *
 * q: [B][N][Hq][d] and out: [B][N][Hq][d], same dtype as the caches.
 * dt = TV_BF16: bfloat16 inputs/outputs, float32 accumulation and softmax;
 *   requires d in {64, 128} and block_size a multiple of 16.
 * dt = TV_F32: float32 throughout; requires d <= 256 and d % 32 == 0.
 * scale <= 0 selects 1/sqrt(d).
 * mask: uint64 [B][N] (from tree_mask_build).  status: int32 [B]; a sequence
 * with P_b < 0, P_b + N > max_blocks_per_seq * block_size, or a block id
 * outside [0, num_blocks) among the blocks covering positions 0..P_b+N-1 gets
 * TV_ERR_OUT_OF_RANGE and zero outputs.  Positions beyond P_b + N - 1 in the
 * last block are never read into the result (they may hold anything, NaN
 * included).
 * workspace: device scratch of tree_verify_attention_workspace() bytes,
 * 256-byte aligned.  Its leading bytes are scheduler counters and
 * per-(sequence, kv head, row tile) arrival counters that must be zero
 * before the first call (zero the whole buffer once); every call that
 * completes leaves them at zero again.  The rest holds split-KV partial
 * results (per row: softmax max and sum, normalised output) of the
 * balanced schedule, which gives every SM the same number of key tiles.
 * A smaller workspace of at least 256 bytes is accepted and selects a
 * schedule without partial results in global memory (groups of sequences
 * handed to clusters of SMs); below 256 bytes the call returns
 * TV_ERR_WORKSPACE.
 * ------------------------------------------------------------------------ */
size_t tree_verify_attention_workspace(int B, int N, int Hq, int Hkv, int d,
                                       int max_blocks_per_seq, int block_size, tv_dtype dt);

/* Kernels one tree_verify_attention call with these sizes and this workspace
 * size launches on the current device (launch accounting: the balanced
 * schedule adds a merge kernel); 0 when B = 0, -1 for arguments the call
 * rejects before launching. */
int tree_verify_attention_kernels(int B, int N, int Hq, int Hkv, int d, int max_blocks_per_seq,
                                  int block_size, tv_dtype dt, size_t workspace_bytes);

tv_status tree_verify_attention(const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_table, int max_blocks_per_seq,
                                const int32_t* prefix_lens, const uint64_t* mask, int B, int N,
                                const int32_t* node_counts, int Hq, int Hkv, int d,
                                int block_size, int num_blocks,
                                tv_dtype dt, float scale, void* out, int32_t* status,
                                void* workspace, size_t workspace_bytes, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * tree_accept — "P-EAGLE in vLLM", 技术原理和实现方式 step 4 (accept the
 * verified drafts, truncate at the first rejection) and "vLLM EAGLE in
 * practice", 无损性保障 (greedy speculation reproduces greedy decoding;
 * rejection sampling reproduces the target distribution).
 *
 * Row i of `target` ([B][N][V] float32) is the target model's output for the
 * token that FOLLOWS node i: logits for TV_ACCEPT_GREEDY, probabilities for
 * TV_ACCEPT_STOCHASTIC.  draft_tokens: int32 [B][N] (entry 0 unused).
 *
 * TV_ACCEPT_GREEDY: node c >= 1 matches iff draft_tokens[c] equals the argmax
 *   of row parents[c] (lowest index on ties; NaN never wins).  Accepted nodes
 *   are those whose whole root path matches; the chosen node is the deepest
 *   accepted node (ties: smallest id).  The bonus token is the argmax of the
 *   chosen node's row.  draft_probs is ignored (may be NULL).
 * TV_ACCEPT_GREEDY_MASKED: the same for rows in which -infinity marks tokens that
 *   are not allowed (tree_logits_process): it never wins either, so a row without
 *   anything above it is like a row of NaNs.  It has no argmax, no child matches
 *   it, and chosen it gives TV_ERR_BAD_VALUES.
 * TV_ACCEPT_STOCHASTIC: draft_probs [B][N][V] row k is the draft
 *   distribution node k's token was drawn from.  On a chain (parents[i] =
 *   i - 1):
 *   For k = 1..N-1, with (w0, w1, w2, w3) = Philox4x32-10(counter = (k, b,
 *   offset_lo, offset_hi), key = (seed_lo, seed_hi)) and u = w0 >> 8:
 *   accept x_k iff u * draft_probs[k][x_k] < target[k-1][x_k] * 2^24 (exact).
 *   At the first rejection the emitted token is drawn from the residual
 *   max(0, target[k-1] - draft_probs[k]) (one float32 subtraction per entry),
 *   or from target[k-1] if the residual has zero mass; after N-1 acceptances
 *   it is drawn from target[N-1] with the draw for k = N.  A draw from
 *   weights r uses integer weights floor(min(r,1) * 2^40) (0 for NaN or
 *   r <= 0), their exact sum S, T = floor(w1 * S / 2^32), and returns the
 *   smallest index whose inclusive prefix sum exceeds T.
 *   On a branching tree (this rule is the library's: the pages fix only that
 *   the result follows the target distribution) the children of the current
 *   node cur are tried in node order.  The first is tested as above against
 *   target[cur].  After a rejection the target is the residual, kept as the
 *   integer weights w (sum S): after the first rejected child c, w_t =
 *   weight(target[cur][t] - draft_probs[c][t]); after each further rejected
 *   child c', w_t -= min(w_t, floor(weight(draft_probs[c'][t]) * S / 2^40))
 *   with S before the update.  A later child c' (token x) is accepted iff
 *   u * weight(draft_probs[c'][x]) * S < w_x * 2^64.  An accepted child
 *   becomes cur.  When every child is rejected the token is drawn from w
 *   (from target[cur] if S = 0, and then no later child is tried) with w1
 *   of the last rejected child's draw; when cur is a leaf the bonus token is
 *   drawn from target[cur] with w1 of the draw for k = N (leaf N-1) or
 *   k = N + cur.  On a chain both descriptions agree.  A tree is walked by
 *   one thread-block cluster per sequence, launched after the chain kernel
 *   on the same stream (so a stochastic call launches two kernels when
 *   N > 2).
 *
 * Outputs: accept_len int32 [B] = depth of the chosen node (number of
 * accepted drafts); path int32 [B][max_path] = node ids root..chosen, then
 * -1; out_tokens int32 [B][max_path] = the accepted drafts' tokens followed
 * by the bonus/correction token, then -1.  status int32 [B].  On a data
 * error (TV_ERR_BAD_TREE, TV_ERR_OUT_OF_RANGE for a token outside [0, V) or
 * a path longer than max_path, TV_ERR_BAD_VALUES) the sequence gets accept_len 0, path
 * [0, -1, ...] and out_tokens all -1.
 * workspace: at least tree_accept_workspace() bytes (0 means none is needed
 * and NULL is allowed).  Greedy acceptance on small batches reads every row
 * once in parallel, cut into chunks, and keeps per-chunk and per-row argmax
 * results plus per-row and per-sequence arrival counters there; stochastic
 * acceptance keeps per-chunk weight sums and a per-sequence arrival counter.
 * The counters must be zero before the first call (zero the whole buffer
 * once) and every completed call leaves them at zero; calls sharing one
 * workspace must not run concurrently.
 * Host errors: N outside [1, 64], V outside [1, 2^24], max_path < 1;
 * TV_ERR_WORKSPACE when the workspace is missing or too small.
 * ------------------------------------------------------------------------ */
size_t tree_accept_workspace(tv_accept_mode mode, int B, int N, int V);

tv_status tree_accept(tv_accept_mode mode, const int32_t* parents, const int32_t* draft_tokens,
                      const float* target, const float* draft_probs, int B, int N,
                      const int32_t* node_counts, int V,
                      uint64_t seed, uint64_t offset, int32_t* accept_len, int32_t* path,
                      int32_t* out_tokens, int max_path, int32_t* status, void* workspace,
                      size_t workspace_bytes, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * tree_kv_append — "EAGLE code principles", KV缓存优化: KVCache.cat appends
 * the new tokens' K/V after the prefix.  The step before
 * tree_verify_attention ("write then attend"): node i of sequence b sits at
 * logical position t = P_b + i (physical slot block_table[b][t / block_size]
 * * block_size + t % block_size).
 *
 * k_new, v_new: [B][N][Hkv][d] (dt elements), the tree's keys and values.
 * For every node and kv head the value row, and the key row when
 * rope_theta <= 0, is copied to the node's slot of v_cache / k_cache
 * ([num_blocks][Hkv][block_size][d]).  With rope_theta > 0 the key is first
 * rotated by its tree position P_b + depth[b][i] (depth int32 [B][N], e.g.
 * from tree_mask_build): rotate-half pairs (j, j + d/2), j < d/2, angle
 * pos * rope_theta^(-2j/d):
 *   k'_j = k_j cos - k_{j+d/2} sin,  k'_{j+d/2} = k_{j+d/2} cos + k_j sin,
 * every product and sum in double, rounded to float32, then to dt.
 * status int32 [B]: TV_ERR_OUT_OF_RANGE for P_b < 0, a position
 * P_b .. P_b+N-1 without a valid block, or (rotation only) a depth outside
 * [0, N); such a sequence's cache is left unchanged.
 * Host errors: N outside [1, 64], d odd, d * element size not a multiple of
 * 16 bytes (TV_ERR_UNSUPPORTED), a NULL depth with rope_theta > 0, NaN
 * rope_theta, pointers not 16-byte aligned.
 * ------------------------------------------------------------------------ */
tv_status tree_kv_append(const void* k_new, const void* v_new, const int32_t* depth, int B, int N,
                         const int32_t* node_counts, int Hkv, int d, float rope_theta,
                         void* k_cache, void* v_cache,
                         const int32_t* block_table, int max_blocks_per_seq,
                         const int32_t* prefix_lens, int block_size, int num_blocks, tv_dtype dt,
                         int32_t* status, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * kv_compact — "EAGLE code principles", KV缓存优化: KVCache.copy(indices,
 * prev_length) selects the kept rows (index_select), locates the
 * destination (narrow at prev_length) and copies them there; "P-EAGLE in
 * vLLM", 技术难点: roll back on rejection, append on acceptance.
 *
 * For every layer l < num_layers (caches at k_cache/v_cache + l *
 * layer_stride elements), every kv head and both caches: first read the rows
 * at logical positions P_b + path[b][j], j = 0..accept_len[b], then write them
 * to positions P_b + j (gather-then-scatter, so a destination may be the
 * source of another row).  new_lens[b] = P_b + accept_len[b] + 1.
 * src_slots / dst_slots (int64 [B][max_path], nullable) receive the physical
 * slots block * block_size + row, padded with -1.
 * A sequence with P_b < 0, accept_len outside [0, max_path), a negative path
 * entry, or a position not covered by a valid block gets TV_ERR_OUT_OF_RANGE,
 * new_lens = P_b, slots -1 and no cache change.  Positions P_b .. P_b+N-1
 * must map to blocks that no other sequence writes in the same call.
 * dt selects the element size (TV_BF16: 2 bytes, TV_F32: 4 bytes);
 * d * element size must be a multiple of 16 bytes.
 * ------------------------------------------------------------------------ */
tv_status kv_compact(void* k_cache, void* v_cache, int num_layers, int64_t layer_stride,
                     const int32_t* block_table, int max_blocks_per_seq,
                     const int32_t* prefix_lens, const int32_t* path, const int32_t* accept_len,
                     int max_path, int B, int Hkv, int d, int block_size, int num_blocks,
                     tv_dtype dt, int32_t* new_lens, int64_t* src_slots, int64_t* dst_slots,
                     int32_t* status, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * draft_tree_expand — "vLLM-TreeEagle", 核心组件 / 3. EnhancedEagleProposer
 * (candidates generated over several levels, paths pruned) and "EAGLE code
 * principles", 树结构缓冲 (likely paths precomputed, high-probability paths
 * kept, low-probability branches cut).  The step before verification: the
 * draft tree is grown one layer per call from the draft model's logits (the
 * draft model runs between calls, on the frontier each call returns).
 *
 * logits: fp32 [B][F][V]; F = 1 at layer 0 (the row after the root, whose
 * token is root_tokens[b]), F = topk at later layers (row f follows frontier
 * entry f of the previous call).  Each row's topk largest logits (ties: lowest
 * token id) become children, scored score(parent) + logit - logsumexp(row) in
 * fp32 (the root scores 0).  Nodes are numbered in creation order: row-major,
 * then rank.  The next frontier is the topk best new nodes by (score
 * descending, creation id ascending): front_tokens int32 [B][topk] (their
 * tokens, best first) and front_src int32 [B][topk] (the row each came from);
 * both nullable.  The call for the last layer (layer == layers - 1) also
 * writes the tree: the root and the N - 1 best of all created nodes, same
 * order, labelled breadth-first from the root with each node's children in
 * creation order (so 0 <= parents[i] < i, the order tree_mask_build and
 * tree_accept expect): parents int32 [B][N] (-1 at the root), tokens int32
 * [B][N] (tokens[b][0] = root token), scores fp32 [B][N] (nullable).
 * status int32 [B], written by every call: TV_ERR_OUT_OF_RANGE for a root
 * token outside [0, V) (layer 0), TV_ERR_BAD_VALUES for a NaN or +inf logit
 * or a row without a finite one, TV_ERR_WORKSPACE when the workspace does not
 * hold the sequence's state after layer - 1.  An error sticks for the later
 * layers of the tree; the sequence's frontier outputs become -1, its tree
 * parents and tokens -1 and its scores -inf.
 * workspace: draft_tree_workspace() bytes, 16-byte aligned.  It holds
 * per-sequence arrival counters that must be zero before the first call (zero
 * the whole buffer once; every completed call leaves them at zero), the tree
 * state carried from layer to layer, and per-chunk partial results.  The
 * calls of one tree go in order layer 0, 1, ..., layers - 1 on one workspace;
 * calls sharing a workspace must not run concurrently.
 * Host errors: TV_ERR_INVALID_ARG for topk outside [1, 16] or above V, V
 * outside [1, 2^30], layers < 1, layer outside [0, layers), N outside [1, 64]
 * or above the number of created nodes 1 + topk + (layers - 1) * topk^2, a
 * NULL logits or status, a NULL root_tokens at layer 0, a NULL parents or
 * tokens at the last layer; TV_ERR_UNSUPPORTED for more than 2048 created
 * nodes; TV_ERR_WORKSPACE for a missing, misaligned or small workspace.
 * draft_tree_workspace returns 0 for unsupported sizes.
 * ------------------------------------------------------------------------ */
size_t draft_tree_workspace(int B, int topk, int layers);

tv_status draft_tree_expand(const float* logits, const int32_t* root_tokens, int B, int V,
                            int topk, int layer, int layers, int N, int32_t* front_tokens,
                            int32_t* front_src, int32_t* parents, int32_t* tokens, float* scores,
                            int32_t* status, void* workspace, size_t workspace_bytes,
                            tv_stream_t stream);

/* ------------------------------------------------------------------------
 * tree_verify_attention_noalloc — no counterpart on the pages describing the
 * method; an addition of this library for callers that cannot allocate.
 *
 * Some callers cannot provide device scratch memory: an engine that reserved
 * all of HBM for its own pools up front and does not allocate while decoding,
 * or a plugin host that gives its plugins no allocator.  This call computes
 * exactly what tree_verify_attention computes (same arguments, minus the
 * workspace) but takes its scratch from a fixed array inside the library,
 * and picks the schedule a tree_verify_attention call would pick with a
 * workspace of exactly tree_verify_attention_workspace(...) bytes, so the
 * two give bit-identical outputs.  The array is
 * TV_NOALLOC_SCRATCH_BYTES of device memory that every GPU loading the
 * library holds until the process exits.  It never calls cudaMalloc,
 * cudaFree or any allocating routine.
 *
 * - Sizes whose workspace (tree_verify_attention_workspace) exceeds
 *   TV_NOALLOC_SCRATCH_BYTES are rejected with TV_ERR_WORKSPACE before
 *   anything is launched.
 * - The first call on a device looks up the array's device address (with
 *   that device current) and caches it; make that first call before any
 *   stream capture begins.
 * - All calls share the one array, and it keeps the previous call's
 *   contents: each call first clears (cudaMemsetAsync on `stream`) the part
 *   that must start at zero.  Calls that overlap on the GPU (different
 *   streams, or concurrent host threads) race on the array and must not be
 *   issued.
 * ------------------------------------------------------------------------ */
#define TV_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

size_t tree_verify_attention_noalloc_capacity(void);

tv_status tree_verify_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_table, int max_blocks_per_seq,
                                        const int32_t* prefix_lens, const uint64_t* mask, int B,
                                        int N, const int32_t* node_counts, int Hq, int Hkv, int d,
                                        int block_size,
                                        int num_blocks, tv_dtype dt, float scale, void* out,
                                        int32_t* status, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * Chunks of new tokens.  chunk_kv_append and chunk_attention take a ragged
 * batch: T rows (tokens) laid end to end, sequence b owning rows q_start[b] ..
 * q_start[b+1] - 1 (q_start: device int32 [B + 1], non-decreasing, within
 * [0, T]; n_b = q_start[b+1] - q_start[b] may be 0).  Row q_start[b] + i is the
 * token at logical position P_b + i, P_b = prefix_lens[b].  Rows before
 * q_start[0] or from q_start[B] on belong to no sequence: they are neither read
 * into a result nor written.  If q_start breaks these rules every sequence gets
 * TV_ERR_OUT_OF_RANGE and nothing else is written.  P_b + n_b is at most
 * 2^31 - 1024.  A prompt is one chunk or several, plain decoding is n_b = 1, and
 * both may share a batch.
 * ------------------------------------------------------------------------ */

/* Rotary positions.  A table holds, for each of dim / 2 pairs of columns, the
 * pair's turns per position as a 64-bit fraction of a turn: position times that
 * integer, modulo 2^64, is the angle modulo one turn without rounding, however
 * far the position.  It is plain host data (no pointers) that
 * rope_table_init fills; calls copy it, so it may be freed or changed after
 * they return.
 *
 *   f_j = theta^(-2 j / dim) radians per position, j < dim / 2, then by scaling
 *   TV_ROPE_NONE    f_j
 *   TV_ROPE_LINEAR  f_j / factor
 *   TV_ROPE_BANDS   with n_j = original_len f_j / (2 pi) turns over the original
 *                   context and k = clamp((n_j - low) / (high - low), 0, 1):
 *                   f_j (k + (1 - k) / factor)            (low 1, high 4)
 *   TV_ROPE_RAMP    with e(n) = dim ln(original_len / (2 pi n)) / (2 ln theta),
 *                   a = max(0, floor(e(high))), z = min(dim - 1, ceil(e(low))),
 *                   s = clamp((j - a) / max(z - a, 0.001), 0, 1):
 *                   f_j (1 - s) + f_j / factor s          (low 1, high 32)
 * low, high <= 0 select the values in parentheses.  amplitude multiplies cos
 * and sin; <= 0 selects 0.1 ln(factor) + 1 for TV_ROPE_RAMP and 1 otherwise.
 * interleaved: pairs are columns (2j, 2j + 1); otherwise (j, j + dim / 2).
 * Columns from dim on are not rotated. */
typedef enum {
    TV_ROPE_NONE = 0,
    TV_ROPE_LINEAR = 1,
    TV_ROPE_BANDS = 2,
    TV_ROPE_RAMP = 3
} tv_rope_scaling;

#define TV_ROPE_MAX_DIM 256

typedef struct {
    int32_t dim;          /* rotated columns, even, <= TV_ROPE_MAX_DIM */
    int32_t interleaved;  /* 0 or 1 */
    float amplitude;
    float amplitude_rest; /* what the rounding of amplitude leaves (or 0) */
    uint64_t turn[TV_ROPE_MAX_DIM / 2];
} tv_rope_table;

/* Host only.  TV_ERR_INVALID_ARG: NULL table, dim odd or outside [2,
 * TV_ROPE_MAX_DIM], theta not finite or <= 1, an unknown scaling, and with a
 * scaling factor not finite or < 1, or (bands, ramp) original_len not finite or
 * < 1, or high <= low. */
tv_status rope_table_init(tv_rope_table* table, int dim, int interleaved, double theta,
                          tv_rope_scaling scaling, double factor, double original_len, double low,
                          double high, double amplitude);

/* ------------------------------------------------------------------------
 * chunk_kv_append — "EAGLE code principles", KV缓存优化: KVCache.cat, for a
 * chunk of tokens of any length.  The step before chunk_attention (or, with
 * positions P_b + depth, before tree_verify_attention: the call that rotates a
 * tree's queries).
 *
 * q [T][Hq][d], k and v [T][Hkv][d] (dt elements; heads contiguous, rows
 * q_stride / k_stride / v_stride elements apart, so all three may be views of
 * one fused projection).  For every row of a sequence: the value row, and the
 * rotated key row, go to the slot of logical position P_b + i; the rotated
 * query row goes to q_out (rows q_out_stride apart; q_out may be q with the
 * same stride: each element is read by the thread that writes it).  q and
 * q_out NULL: keys and values only.  rope NULL: nothing is rotated.
 * The rotary position of a row is P_b + i, or positions[row] (device int32 [T])
 * if positions is not NULL.  A pair (x, y) with angle a becomes
 * (x cos a - y sin a, y cos a + x sin a) times amplitude: the angle's fraction
 * of a turn exact to 64 bits, cos, sin, products and sums in float32, one
 * rounding to dt.
 * status int32 [B]: TV_ERR_OUT_OF_RANGE for P_b < 0, a position P_b .. P_b + n_b
 * - 1 without a valid block, or a negative position; that sequence's cache
 * slots and q_out rows are left unchanged.  Two sequences must not append to
 * the same slot.
 * Host errors: TV_ERR_INVALID_ARG for sizes, NULL or (16 bytes) misaligned
 * pointers, strides smaller than a row, rope->dim above d; TV_ERR_UNSUPPORTED for d
 * or a stride that is no multiple of 16 bytes, or rope->dim no multiple of 32
 * bytes.
 * ------------------------------------------------------------------------ */
tv_status chunk_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const int32_t* positions, int T,
                          const int32_t* q_start, const int32_t* prefix_lens, int B, int Hq,
                          int Hkv, int d, const tv_rope_table* rope, void* q_out,
                          int64_t q_out_stride, void* k_cache, void* v_cache,
                          const int32_t* block_table, int max_blocks_per_seq, int block_size,
                          int num_blocks, tv_dtype dt, int32_t* status, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * chunk_attention — the target model's attention for what tree_verify_attention
 * does not cover: prompts in chunks, and plain decoding (n_b = 1), over the
 * same paged cache ("vLLM-TreeEagle", 核心组件: PagedAttention underneath).
 *
 * For row q_start[b] + i (position p = P_b + i) and query head h (kv head g = h
 * / (Hq / Hkv)):
 *   keys  K = { t : max(0, p - window + 1) <= t <= p }   (window <= 0: 0 <= t <= p)
 *   s_t = scale * q . k_t, and with softcap > 0  s_t = softcap * tanh(s_t / softcap)
 *   out[row][h] = sum_{t in K} softmax_t(s) v_t
 * (NaN for a row whose every score is -infinity).
 * The chunk's own keys and values are in the cache already (chunk_kv_append).
 * q [T][Hq][d] and out [T][Hq][d], dt elements, heads contiguous, rows
 * q_stride / out_stride elements apart.  out must not overlap q.
 * dt = TV_BF16: float32 accumulation and softmax; d in {64, 128}, block_size a
 * multiple of 16.  dt = TV_F32: float32 throughout; d <= 256, d % 32 == 0.
 * scale <= 0 selects 1/sqrt(d).
 * status int32 [B]: TV_ERR_OUT_OF_RANGE (and zero rows of out) for P_b < 0, P_b +
 * n_b > max_blocks_per_seq * block_size, or a block id outside [0, num_blocks)
 * among the blocks that hold a key of K for some row of the sequence (blocks
 * wholly before the first row's window may have been given back: their table
 * entries are not read).  TV_ERR_TIMEOUT: a wait ran out in work on the sequence, or on another
 * beside it; its rows of out are not all written.
 * Cache rows that no row of the sequence attends to are never read into a
 * result.  Where a key is outside K for one row and inside for another, its
 * contents reach only the rows that attend to it, infinities and NaN included.
 * workspace: chunk_attention_workspace() bytes, 16-byte aligned, any contents;
 * partial results of rows whose keys are split over several SMs.  Missing or
 * smaller: TV_ERR_WORKSPACE.
 * Other host errors: TV_ERR_INVALID_ARG for sizes, NULL or (16 bytes) misaligned
 * pointers, strides smaller than a row, a softcap that is NaN or infinite;
 * TV_ERR_UNSUPPORTED for other head or block sizes, a stride that is no multiple
 * of 16 bytes, or a bfloat16 cache of 2^31 rows (blocks x heads x block size).
 * ------------------------------------------------------------------------ */
size_t chunk_attention_workspace(int T, int B, int Hq, int Hkv, int d, tv_dtype dt);

tv_status chunk_attention(const void* q, int64_t q_stride, const void* k_cache,
                          const void* v_cache, const int32_t* block_table,
                          int max_blocks_per_seq, const int32_t* q_start,
                          const int32_t* prefix_lens, int T, int B, int Hq, int Hkv, int d,
                          int block_size, int num_blocks, tv_dtype dt, float scale, float softcap,
                          int window, void* out, int64_t out_stride, int32_t* status,
                          void* workspace, size_t workspace_bytes, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * 8-bit caches.  k_cache and v_cache hold e4m3 codes (sign, four bits of exponent with
 * bias 7, three of mantissa; subnormals; no infinities, 0x7f and 0xff are NaN), laid
 * out like the other caches: [num_blocks][Hkv][block_size][d] bytes.  Each block of
 * each kv head has a scale, k_scale and v_scale float32 [num_blocks][Hkv], and a code
 * stands for code * scale.  Scales are powers of two from 2^-100 on, as
 * chunk_kv_append_q8 writes them (of any other number the exponent alone counts, and
 * smaller ones may count as 2^-100), so that what a code stands for is a bfloat16
 * number exactly (but for 256 times 2^120: numbers from 1.9375 2^127 on are rounded to 2^128,
 * and attention may take that for the largest bfloat16 number), and a code moves to a larger
 * scale without rounding until it falls below the smallest normal code (2^-6).  block_size is a multiple of 16; d is 64 or
 * 128; queries, new keys and values and outputs are bfloat16.  Half the bytes of the
 * stream that bounds decoding and verification, for a relative error of 2^-4 an
 * element.
 *
 * A block's codes mean nothing until chunk_kv_append_q8 has written to it; beyond a
 * sequence's last position they may hold anything, and so may a block's scales until
 * its first position has been appended.
 * ------------------------------------------------------------------------ */

/* ------------------------------------------------------------------------
 * chunk_kv_append_q8 — chunk_kv_append into an 8-bit cache: new keys and values
 * rotated, then quantised; queries rotated.  q, k, v, q_out, strides, positions and
 * rope as there, all of them bfloat16; keys and values are rounded once, from
 * float32 to codes.
 *
 * Per block, kv head and cache that new rows fall into, with m their largest finite
 * absolute value (of keys after the rotation):
 *   scale = the smallest power of two, at least 2^-100, with m <= 448 scale; but at
 *           least the block's present scale if it holds positions before P_b
 *   new codes      = e4m3(value / scale), to the nearest, ties to even; infinities
 *                    and NaN become NaN
 *   earlier codes  (positions before P_b) = e4m3(code * present scale / scale)
 * So a block that is appended to from its first position on starts anew, and the
 * scale of one that is filled step by step only grows; rows of rejected drafts that
 * a later call overwrites leave at most a larger scale behind.
 * status int32 [B], refused sequences and host errors: as chunk_kv_append, for d 64
 * or 128 and block sizes that are multiples of 16 (others: TV_ERR_UNSUPPORTED); NULL
 * scales: TV_ERR_INVALID_ARG.  Two sequences must not append to the same block.
 * ------------------------------------------------------------------------ */
tv_status chunk_kv_append_q8(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, const int32_t* positions, int T,
                             const int32_t* q_start, const int32_t* prefix_lens, int B, int Hq,
                             int Hkv, int d, const tv_rope_table* rope, void* q_out,
                             int64_t q_out_stride, void* k_cache, void* v_cache, float* k_scale,
                             float* v_scale, const int32_t* block_table, int max_blocks_per_seq,
                             int block_size, int num_blocks, int32_t* status,
                             tv_stream_t stream);

/* ------------------------------------------------------------------------
 * chunk_attention_q8 — chunk_attention over an 8-bit cache, for every kind of new
 * token: prompts in chunks, single tokens and chains of drafts (the rows of a
 * sequence are causal), and trees (mask).
 *
 * For row q_start[b] + i (position p = P_b + i) and query head h:
 *   keys  K = { t : t <= p and (window <= 0 or t > p - window or t < sinks) }
 *   with mask: K = { t : t < P_b } U { P_b + a : bit a of mask[row], a <= i }
 *   s_t and out as in chunk_attention, k_t and v_t what the codes stand for.
 * sinks: the first tokens that stay visible behind a window, 0 .. 64; without a
 * window they are visible anyway.  mask: uint64 [T] (row i of a sequence is node i
 * of its tree, as tree_mask_build writes them for trees of n_b nodes) or NULL; with
 * it n_b is at most 64, and there is no window.
 * A row without a key is zero; one whose every score is -infinity is NaN.
 * Float32 accumulation and softmax.  Besides their order, what is rounded: the weights,
 * to bfloat16 or (few rows per sequence: those below 2^-27 of a row's largest weight x
 * scale of V by 2^-38 of that) float16; with d = 128, elements of a query row below 2^-10 of
 * its largest, to steps of 2^-17 of that.
 * Sums beyond float32 are infinite, or NaN: q . k_t, and (unless there are few rows per
 * sequence) 2^8 times the sum of weights up to 1 times values.
 * status int32 [B]: as chunk_attention (with sinks, the blocks of the first sinks
 * positions are needed too), and TV_ERR_OUT_OF_RANGE for more than 64 rows with a
 * mask.  Cache contents outside K reach no row, NaN included.
 * One of two kernels serves a whole call, chosen by the average of rows per sequence (T / B
 * times Hq / Hkv: up to 24, or more): a long chunk among many decoding sequences is better
 * given a call of its own (512 rows after 16,000 keys and 128 single rows after 512-8,192, 32/8
 * heads of 128: 910 us together, 146 and 214 apart).
 * workspace: chunk_attention_q8_workspace() bytes, 16-byte aligned, any contents.
 * Host errors: as chunk_attention; TV_ERR_INVALID_ARG for sinks outside [0, 64], mask
 * with a window, NULL scales; TV_ERR_UNSUPPORTED for d other than 64 and 128, a block
 * size that is no multiple of 16, more than 128 query heads per kv head.
 * ------------------------------------------------------------------------ */
#define TV_MAX_SINKS 64

size_t chunk_attention_q8_workspace(int T, int B, int Hq, int Hkv, int d);

tv_status chunk_attention_q8(const void* q, int64_t q_stride, const void* k_cache,
                             const void* v_cache, const float* k_scale, const float* v_scale,
                             const int32_t* block_table, int max_blocks_per_seq,
                             const int32_t* q_start, const int32_t* prefix_lens,
                             const uint64_t* mask, int T, int B, int Hq, int Hkv, int d,
                             int block_size, int num_blocks, float scale, float softcap,
                             int window, int sinks, void* out, int64_t out_stride,
                             int32_t* status, void* workspace, size_t workspace_bytes,
                             tv_stream_t stream);

/* ------------------------------------------------------------------------
 * kv_compact_q8 — kv_compact on 8-bit caches (the steps around it as there; on a
 * chain the accepted rows lie where they belong already, and no call is needed).
 *
 * For every layer l (caches layer_stride bytes apart, scales scale_layer_stride
 * numbers apart), kv head and cache: what the rows at positions P_b + path[b][j] stand
 * for goes to positions P_b + j, gather-then-scatter.  The scale of a block that holds
 * destinations becomes the largest of the scales of the blocks that its rows come
 * from (its own among them where a row stays) and, where it holds positions before
 * P_b, of its own; codes whose scale grows, those before P_b too, are rounded again.
 * new_lens, src_slots, dst_slots, status and host errors: as kv_compact, for d 64 or 128
 * (others: TV_ERR_UNSUPPORTED) and block sizes that are multiples of 16; NULL scales:
 * TV_ERR_INVALID_ARG.  accept_len is below 64.
 * ------------------------------------------------------------------------ */
tv_status kv_compact_q8(void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                        int num_layers, int64_t layer_stride, int64_t scale_layer_stride,
                        const int32_t* block_table, int max_blocks_per_seq,
                        const int32_t* prefix_lens, const int32_t* path,
                        const int32_t* accept_len, int max_path, int B, int Hkv, int d,
                        int block_size, int num_blocks, int32_t* new_lens, int64_t* src_slots,
                        int64_t* dst_slots, int32_t* status, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * token_counts_update — the history that tree_logits_process reads: counts
 * int32 [B][V], bit 31 of a word set when the token occurs in the prompt, the
 * low 31 bits the number of times it was emitted.
 *
 * tokens: with starts (device int32 [B + 1], non-decreasing, within [0, total])
 * sequence b's tokens are tokens[starts[b]] .. tokens[starts[b+1] - 1]; with
 * starts NULL they are row b of [B][total / B] (as tree_accept's out_tokens).
 * Entries of -1 are skipped.  clear: the row is zeroed first.  prompt: the
 * tokens set bit 31, otherwise each adds 1 (integer atomics: the order does not
 * matter).
 * status int32 [B]: TV_ERR_OUT_OF_RANGE for a token outside [-1, V) or a bad
 * starts array; that sequence's row is left unchanged.
 * Host errors: B < 0, V outside [1, 2^24], total < 0, starts NULL and total no
 * multiple of B, NULL pointers (tokens may be NULL when total is 0).
 * ------------------------------------------------------------------------ */
tv_status token_counts_update(int32_t* counts, const int32_t* tokens, const int32_t* starts,
                              int total, int B, int V, int clear, int prompt, int32_t* status,
                              tv_stream_t stream);

/* ------------------------------------------------------------------------
 * tree_logits_process — the step between the target model and tree_accept: the
 * model's row for every node of a tree becomes the logits (TV_ACCEPT_GREEDY_MASKED)
 * or the probabilities (TV_ACCEPT_STOCHASTIC) that tree_accept reads.
 *
 * logits: [B][N][V], float32 or bfloat16 (dt); out float32 [B][N][V] (may be
 * logits itself when dt is TV_F32).  For row i of sequence b and token x:
 *   z = logits[b][i][x] + bias[b][x]
 *   n = occurrences of x among the emitted tokens: the low 31 bits of
 *       counts[b][x], plus the nodes c >= 1 with bit c of mask[b][i] set and
 *       draft_tokens[b][c] == x (the node's own path; the root is the last token
 *       that counts already holds)
 *   if n > 0 or bit 31 of counts[b][x]:  z = z > 0 ? z / repetition[b] : z * repetition[b]
 *   z = z - frequency[b] * n - (n > 0 ? presence[b] : 0)
 *   z = z / temperature[b]
 *   bit (x % 32) of grammar[b][i][x / 32] clear:  z = -infinity
 *   probs == 0: out = z;  else out = softmax over x of z (0 for a masked token;
 *   a row without an allowed token above -infinity is all zeros; a NaN or +infinity
 *   among the allowed z makes the row NaN).
 * Every product and sum in float32; the divisions by repetition and temperature are
 * products with their float32 reciprocals.  bias [B][V] float32, counts int32 [B][V],
 * grammar uint32 [B][N][ceil(V / 32)], repetition / frequency / presence /
 * temperature float32 [B], mask uint64 [B][N] with draft_tokens int32 [B][N]: each
 * may be NULL (no bias; no history; every token allowed; 1, 0, 0, 1; no path).
 * The penalties need counts.  node_counts as above: rows of absent nodes are not
 * written.
 * status int32 [B]: TV_ERR_OUT_OF_RANGE for a node count outside [1, N] or (with
 * mask) a token of nodes 1 .. n_b - 1 outside [0, V); TV_ERR_BAD_VALUES for a
 * repetition or temperature not finite, <= 0 or below 2^-126, a frequency or
 * presence not finite.  That sequence's rows (all N when the count is bad) are -infinity
 * (probs == 0) or zero; so are those not finished when a wait runs out
 * (TV_ERR_TIMEOUT).  Acceptance takes such rows, and those of a grammar that
 * allows nothing, for what they are in the modes TV_ACCEPT_GREEDY_MASKED and
 * TV_ACCEPT_STOCHASTIC: no token is emitted, and its status is TV_ERR_BAD_VALUES.
 * Host errors: N outside [1, 64], V outside [1, 2^24], NULL logits, out or
 * status, mask without draft_tokens or the reverse, a penalty without counts.
 * ------------------------------------------------------------------------ */
tv_status tree_logits_process(const void* logits, tv_dtype dt, int B, int N, int V,
                              const int32_t* node_counts, const uint64_t* mask,
                              const int32_t* draft_tokens, const int32_t* counts,
                              const float* bias, const uint32_t* grammar,
                              const float* repetition, const float* frequency,
                              const float* presence, const float* temperature, int probs,
                              float* out, int32_t* status, tv_stream_t stream);

/* ------------------------------------------------------------------------
 * logits_sample — sampling, for the rows that no draft covers (the first token behind
 * a prompt, plain decoding), and the filtered distributions of a tree's rows as the
 * target of tree_accept (TV_ACCEPT_STOCHASTIC; a draft model's rows likewise).
 *
 * logits: [B][N][V], float32 or bfloat16 (dt), -infinity for what is not allowed
 * (tree_logits_process without probs).  Per row, with the parameters of its sequence,
 * the entries ordered by (logit descending, index ascending):
 *   temperature 0: the first entry is kept, with probability 1; otherwise
 *   w_x = exp((logit_x - the largest) / temperature), and kept are
 *   1. the first top_k entries (all for top_k <= 0 or >= V),
 *   2. of these the entry e when the w of those before it sum to less than top_p times
 *      the w of all of these (so the first one always; all for top_p = 1),
 *   3. of these the entries with w >= min_p (0: all).
 *   probs[b][i][x] = w_x / (the sum W of the kept ones), 0 for the others
 *   tokens[b][i] = the smallest x with w_0 + .. + w_x (kept ones) > uniform[b][i] * W
 * The w of 1 and 2 and the sums are in fixed point, steps of 2^-42, each w off by at
 * most 2^-38 of itself and half a step (one below 2^-13, in the sum over a whole row that
 * top_p is taken of where top_k does not limit it, by 2^-18 of itself and 2^-39): cuts and
 * tokens differ from the exact ones only where a sum comes that near to its border.  probs are float32, off by at most 2^-20
 * of themselves and of the exponent's rounding, 2^-23 (logit - largest) / temperature.
 * temperature, top_p, min_p float32 [B], top_k int32 [B]: each may be NULL (1; 1; 0; all).
 * uniform float32 [B][N], in [0, 1): the random numbers are the caller's.  probs float32
 * [B][N][V] or NULL (not logits).  node_counts as above: rows of absent nodes are not
 * written, nor are their tokens and statuses.
 * status int32 [B][N], per row: TV_ERR_OUT_OF_RANGE for a node count outside [1, N];
 * TV_ERR_BAD_VALUES for a temperature that is not finite, negative, or positive below
 * 2^-126, a top_p outside (0, 1], a min_p outside [0, 1], a uniform outside [0, 1), and
 * for a row with NaN or +infinity, or with nothing above -infinity.  Such a row has
 * token -1 and probs 0.
 * Host errors: TV_ERR_INVALID_ARG for N outside [1, 64], V outside [1, 2^24], B < 0, NULL
 * logits, uniform, tokens or status; TV_ERR_UNSUPPORTED for V above 786,432 (a row is
 * held in the shared memory of 16 SMs).
 * ------------------------------------------------------------------------ */
tv_status logits_sample(const void* logits, tv_dtype dt, int B, int N, int V,
                        const int32_t* node_counts, const float* uniform,
                        const float* temperature, const int32_t* top_k, const float* top_p,
                        const float* min_p, int32_t* tokens, float* probs, int32_t* status,
                        tv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TREEVERIFY_H */
