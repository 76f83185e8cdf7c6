/*
 * spectree.h -- C ABI of the GB300 (sm_103a) tree speculative verification
 * library (libspectree.so).
 *
 * One verification pass of tree-based speculative inference: the target model
 * checks a whole token tree in one forward pass, with every tree node attending
 * to the committed prefix plus its own ancestors, then a verifier picks the
 * accepted root path (greedy, or stochastic with the min(1, p/q) accept rule
 * and the norm(max(p - q, 0)) residual), and the KV cache keeps only that path.
 * Sources, by page title and section:
 *   "SpecInfer Guide: Tree-Based Speculative LLM Serving": "Mathematical
 *     Formulation of the Token Tree", "Tree-Based Parallel Decoding &
 *     Topology-Aware Causal Masking", "Depth-First Flattening and KV Cache
 *     Reuse", "Exact Output Verification: Greedy and Stochastic Sampling",
 *     "Integration with Continuous Batching", "PagedKV Allocation with
 *     Zero-Copy Pruning".
 *   "Inference Optimization Techniques: Speed and Efficiency": the accept rule
 *     and residual of the "Misconception" section, "Traced Example".
 *   Around the pass: "Token Tree Construction: Expansion vs. Merge" (SpecInfer
 *     guide) for the tree builders, and "Hardware-aware dynamic speculative
 *     decoding" (Cohere) for the goodput table and the <tokens, K> graph keys.
 *
 * Conventions shared by every call
 *   - Every pointer argument is DEVICE memory owned by the caller, except where
 *     a call says otherwise.  The library never allocates, frees or
 *     synchronises; each call enqueues kernels on `stream` (a cudaStream_t,
 *     NULL = the legacy default stream) and returns.
 *   - A batch holds B requests.  Request b owns tree nodes
 *     [tree_off[b], tree_off[b+1]) of every per-node array (ragged packing).
 *     Inside a request nodes are numbered 0..n_b-1 (local index); node 0 is
 *     the root, the last verified token, and parent[t] is the LOCAL index of
 *     the parent (-1 for the root).  Parents come before children:
 *     0 <= parent[i] < i.  n_b <= n_max <= 1024.
 *   - Calls on prompts and packed rows (spec_prompt_attention,
 *     spec_token_logprobs, and spec_kv_append when it appends a prompt's rows)
 *     use the same ragged packing with seq_off in the place of tree_off; their
 *     requests have no limit of 1024 rows.
 *   - mask rows have W = ceil(n_max / 64) 64-bit words.
 *   - The return value reports errors visible on the host (bad scalar
 *     arguments, NULL pointers, unsupported sizes, launch failures); on such
 *     an error nothing is launched.  Errors that depend on device data are
 *     or-ed into the caller's int32 status[B] as SPEC_DEV_* bits; no kernel
 *     traps or asserts.
 *   - Paged KV cache: k_cache and v_cache are [num_blocks][Hkv][block_size][D]
 *     elements of `dtype`; slot s of request b lives in block
 *     block_table[b * max_blocks + s / block_size], row s % block_size.  Slots
 *     [0, prefix_len[b]) hold the committed prefix and slots
 *     prefix_len[b] + v hold tree node v (already written by the caller).
 */
#ifndef SPECTREE_H
#define SPECTREE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t spec_status;

/* Host-visible status codes (return values). */
#define SPEC_OK 0
#define SPEC_ERR_INVALID_ARG 1 /* NULL pointer, negative size, Hq not a multiple of Hkv, ... */
#define SPEC_ERR_UNSUPPORTED 2 /* D not 64/128, n_max > 1024, V > 131072, block_size not a power of two in [8, 65536] */
#define SPEC_ERR_CUDA 3        /* a CUDA launch or attribute call failed */
#define SPEC_ERR_WORKSPACE 4   /* workspace smaller than the matching *_workspace_size() */

/* Per-request device status bits, or-ed into status[b]. */
#define SPEC_DEV_BAD_TREE 1   /* parent[0] != -1, parent[i] outside [0, i), n_b < 0 or n_b > n_max */
#define SPEC_DEV_BAD_TOKEN 2  /* a node token outside [0, V) */
#define SPEC_DEV_CAPACITY 4   /* prefix_len < 0, prefix_len > max_prefix, or prefix_len + n_b beyond the block table */
#define SPEC_DEV_TIMEOUT 8    /* a bounded device wait expired (the kernel returned early) */
#define SPEC_DEV_BAD_BLOCK 16 /* a block-table entry outside [0, num_blocks) */
#define SPEC_DEV_BAD_PATH 32  /* a commit path that is not strictly increasing from node 0 */
#define SPEC_DEV_BAD_TEMP 64  /* stochastic verify: an inverse temperature that is not finite and positive */
#define SPEC_DEV_BAD_ROW 128 /* page calls: a block-table row out of range, named twice, or not empty where it must be */
#define SPEC_DEV_BAD_POSITION 256 /* spec_rope_append: a position outside [0, 2^24), or a pair's axis outside [0, axes) */

typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1 } spec_dtype;

/* spec_tree_attention flags */
/* SPEC_ATTN_AUTO: the tcgen05 tensor-core path for every bf16 call (a KV group
 * with fewer than 128 query rows runs in a zero-padded 128-row tile: the path
 * is bound by the K/V stream, and on GB300 the padded tile streams K/V at
 * 5.3 TB/s for 36-row groups where the CUDA-core kernel reaches 0.22 TB/s);
 * the CUDA-core path for fp32. */
#define SPEC_ATTN_AUTO 0u
#define SPEC_ATTN_CUDA_CORE 1u  /* force the CUDA-core path */
#define SPEC_ATTN_TCGEN05 2u    /* force the tcgen05 path (bf16 only) */

/* Library version, (major << 16) | minor. */
int spec_version(void);

/* Human-readable name of a return code (SPEC_OK, SPEC_ERR_*). */
const char* spec_status_string(spec_status s);

/* Human-readable name of one device status bit (SPEC_DEV_*); "unknown status
 * bit" for anything else (0, several bits, or an undefined bit). */
const char* spec_dev_status_string(int32_t bit);

/*
 * Topology mask build.  "SpecInfer Guide", "The Topology-Aware 2D Causal Mask":
 * M[u][v] = 0 if v is u or an ancestor of u, else -inf; here packed as bits.
 *   parent   int32 [T]     local parent index per node (-1 at the root)
 *   tree_off int32 [B+1]   request offsets into the node arrays
 *   mask     uint64 [T][W] out: bit v of word v/64 of row u set iff v is u or an ancestor of u
 *   depth    int32 [T]     out: number of ancestors of the node (root 0)
 *   status   int32 [B]     out: WRITTEN (not or-ed): 0, or SPEC_DEV_BAD_TREE; this call
 *                          starts a verification pass.  A bad request gets all-zero mask
 *                          rows and depth -1.
 */
spec_status spec_tree_mask_build(const int32_t* parent, const int32_t* tree_off, int B, int n_max,
                                 uint64_t* mask, int32_t* depth, int32_t* status, void* stream);

/* Bytes of workspace spec_tree_attention needs for this shape (T = tree_off[B],
 * max_prefix = the largest prefix_len the call may see). */
size_t spec_attention_workspace_size(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D);

/*
 * Tree attention.  "SpecInfer Guide", "Generalizing Attention to Tree
 * Topologies" and "Depth-First Flattening and KV Cache Reuse": for request b,
 * node u and query head h, out = sum_k softmax_k(scale * q . K_k) V_k over the
 * keys k in slots [0, prefix_len[b]) (the committed prefix) and slots
 * prefix_len[b] + v for every v with mask bit v of row u set (the node and
 * its ancestors).  Query head h reads kv-head h / (Hq / Hkv).  fp32
 * accumulation; bf16 inputs give bf16 output.
 *   q        [T][Hq][D] dtype   queries (positions already applied; RoPE position = prefix + depth)
 *   k_cache, v_cache            paged cache, see the conventions above
 *   block_table int32 [B][max_blocks]
 *   prefix_len  int32 [B]       committed prefix length per request (<= max_prefix)
 *   mask        from spec_tree_mask_build
 *   out      [T][Hq][D] dtype   out
 *   workspace   device scratch of spec_attention_workspace_size() bytes
 *   status   int32 [B]          in/out: or-ed with SPEC_DEV_CAPACITY / SPEC_DEV_BAD_BLOCK.
 *                               A flagged request's output rows are unspecified (the
 *                               CUDA-core path skips requests whose status is non-zero on
 *                               entry; the tcgen05 path computes them).
 *   flags       SPEC_ATTN_*
 * The tcgen05 kernel is launched as a programmatic dependent of the previous
 * kernel in the stream: its set-up and K/V loads may overlap that kernel (the
 * mask build allows this at its start), and it reads the mask and the status
 * word, writes the status word, and loads any key tile that reaches the
 * tree's own slots (prefix_len[b] and on) only after waiting for that kernel
 * to finish; the grid does not complete before that kernel.  The tree K/V
 * rows may therefore be written by the kernel right before this call
 * (spec_kv_append).  A kernel that allows programmatic dependents and sits
 * right before this call must not write q, the prefix slots of the caches,
 * block_table, prefix_len or tree_off; kernels that do not allow it (the
 * usual case) are waited for in full, as with any launch.
 */
spec_status spec_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                                const int32_t* block_table, int max_blocks, int block_size, int num_blocks,
                                const int32_t* prefix_len, const int32_t* tree_off, const uint64_t* mask,
                                int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D,
                                spec_dtype dtype, float scale, void* out,
                                void* workspace, size_t workspace_bytes, int32_t* status,
                                uint32_t flags, void* stream);

/*
 * spec_tree_attention without a workspace argument (the pages have no
 * counterpart of this call).  Some callers cannot allocate device memory where
 * they run attention: a host framework that passes the library only the
 * tensors it owns, or a serving loop whose graphs are captured once and must
 * not pay cudaMalloc's device-wide synchronisation per shape.  When the plan
 * splits a long key range over several CTAs (long prefixes, few requests), the
 * splits' partial outputs need scratch; this call keeps it in one fixed
 * file-scope device array of SPEC_ATTN_NOALLOC_BYTES, which every GPU that
 * loads the library holds until the process exits.  It calls no allocator.
 *   Limit: the plan's scratch for this shape, dtype and flags (at most
 *   spec_attention_workspace_size()) must fit in SPEC_ATTN_NOALLOC_BYTES;
 *   otherwise SPEC_ERR_UNSUPPORTED and nothing is launched.
 *   Set-up: the first call on each device looks up the array's device address
 *   with that device current; make that first call before any stream capture.
 *   The address is cached per device together with the current context: after
 *   a reset of the device's primary context (cudaDeviceReset) the next call
 *   looks it up again, so that call too belongs before any capture.  A failed
 *   lookup returns SPEC_ERR_CUDA and leaves no pending runtime error.
 *   Sharing: every call uses the same array, which keeps the last call's
 *   contents.  Nothing in it must start at zero (a call writes every partial
 *   it reads back), but calls whose kernels overlap on the GPU race: serialise
 *   them (one stream per device).
 *   Other arguments, outputs and statuses as in spec_tree_attention.
 */
#define SPEC_ATTN_NOALLOC_BYTES (16u << 20)
spec_status spec_tree_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_table, int max_blocks, int block_size, int num_blocks,
                                        const int32_t* prefix_len, const int32_t* tree_off, const uint64_t* mask,
                                        int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D,
                                        spec_dtype dtype, float scale, void* out, int32_t* status, uint32_t flags,
                                        void* stream);

/* Bytes of workspace the verifiers take (a small constant: the walk keeps no
 * state in global memory; the argument stays so that callers need not change
 * when a variant needs scratch). */
size_t spec_verify_workspace_size(int B, int n_max, int V);

/*
 * Greedy token-tree verification.  "SpecInfer Guide", "Greedy Verification
 * Algorithm": starting at the root, descend into the child whose token equals
 * argmax of the current node's target logits; when none matches, emit that
 * argmax and stop.  p_logits[t] is the target's next-token logits after node
 * t's sequence, so child c is tested against argmax(p_logits[parent c]).
 * The accepted node f is the deepest node whose whole root path follows the
 * argmax chain (ties between equally deep nodes: lowest node index; with
 * distinct sibling tokens this is the walk above).  argmax ties go to the
 * lowest token id.  Logits must be finite.  One thread-block cluster per
 * request walks the tree level by level; only rows of nodes on matching
 * paths are read.
 *   p_logits   float [T][V]
 *   tokens     int32 [T]       draft token of each node (the root's is not used for matching)
 *   parent, tree_off           as for spec_tree_mask_build
 *   path       int32 [B][n_max] out: accepted nodes root first (local indices), then -1
 *   accept_len int32 [B]       out: number of accepted nodes including the root
 *   emitted    int32 [B][n_max] out: tokens of path[1..] then the correction / bonus token, then -1
 *   n_emitted  int32 [B]       out: = accept_len
 *   workspace  device memory of at least spec_verify_workspace_size() bytes (not read or written)
 *   status     int32 [B]       in/out: a request whose incoming status is non-zero is skipped;
 *                              otherwise or-ed with SPEC_DEV_BAD_TREE (invalid parent array or
 *                              n_b outside [0, n_max]) and SPEC_DEV_BAD_TOKEN; a request whose
 *                              status is non-zero after the call has accept_len = n_emitted = 0
 *                              and -1 rows.
 * Both verifiers are launched as programmatic dependents of the previous
 * kernel in the stream (tree attention lets them launch once its CTAs have
 * issued their last MMA): their prologue (input checks, the root row's
 * copy) may overlap that kernel, and they read the status word only after
 * waiting for it to finish.  A kernel that allows programmatic dependents and
 * sits right before a verify call must therefore not write p_logits,
 * q_probs, tokens, parent, tree_off, uniforms or inv_temperature; kernels
 * that do not allow it are waited for in full.
 */
spec_status spec_tree_verify_greedy(const float* p_logits, const int32_t* tokens, const int32_t* parent,
                                    const int32_t* tree_off, int B, int n_max, int V,
                                    int32_t* path, int32_t* accept_len, int32_t* emitted, int32_t* n_emitted,
                                    void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * Stochastic token-tree verification (multi-step speculative sampling over a
 * tree).  "SpecInfer Guide", "Stochastic Verification Algorithm" with the
 * rule of "Inference Optimization Techniques" ("Misconception" section):
 * a draft token x is accepted with probability min(1, p(x)/q(x)); after a
 * rejection the target becomes norm(max(p - q, 0)).  The children of a node
 * are tried in increasing node index, each against the residual left by the
 * siblings rejected before it; the first accepted child becomes the current
 * node.  When every child is rejected, a token is sampled from the last
 * residual; at a leaf, the bonus token is sampled from p.  The emitted tokens
 * follow the target distribution when each node's children were drawn
 * i.i.d. from q_probs of that node (SPEC_Q_PER_PARENT), or each child
 * independently from its own row (SPEC_Q_PER_CHILD: "Merge-Based Tree
 * Construction", siblings proposed by different draft models; child c is
 * tested against, and on rejection subtracted as, row c).  Sampling at
 * temperature T > 0 ("Stochastic Verification Algorithm"): the target is
 * softmax(p_logits / T), given as the inverse temperature tau = 1/T per
 * request; q_probs are the draft's probabilities as drawn (its own
 * temperature already applied).
 * Arithmetic (fixed so that every decision is reproducible bit for bit):
 * p = softmax(tau * p_logits) with e = E(fp32(fp32(l - max l) * tau)), E
 * the library's own fp32 exp (x <= 0: Cody-Waite reduction, degree-7 Taylor
 * polynomial), normalisers as exact fixed-point sums of trunc(v * 2^46);
 * accept iff u * q(t) <= r(t) with u = (word0 >> 8) * 2^-24; terminal
 * sample = smallest x whose fixed-point prefix sum exceeds
 * floor(word1 * S / 2^32).
 *   q_probs          float [T][V]  SPEC_Q_PER_PARENT: row u is the draft distribution the
 *                                  children of u were drawn from; SPEC_Q_PER_CHILD: row c is
 *                                  the distribution node c was drawn from (row 0 unused)
 *   uniforms         uint32 [T][2] raw random words: [t][0] acceptance word of node t,
 *                                  [t][1] sampling word used if the walk stops at node t
 *   inv_temperature  float [B]     tau of each request, or NULL for tau = 1 (device memory).
 *                                  A tau that is not finite and positive sets
 *                                  SPEC_DEV_BAD_TEMP; the request is skipped.
 *   q_layout         SPEC_Q_PER_PARENT or SPEC_Q_PER_CHILD (else SPEC_ERR_INVALID_ARG)
 *   other arguments as in spec_tree_verify_greedy.  One cluster per request
 *   follows the walk: a node's target row is read when the walk reaches it,
 *   a draft row when a child is rejected against it.
 */
#define SPEC_Q_PER_PARENT 0
#define SPEC_Q_PER_CHILD 1
spec_status spec_tree_verify_stochastic(const float* p_logits, const float* q_probs, const int32_t* tokens,
                                        const int32_t* parent, const int32_t* tree_off, const uint32_t* uniforms,
                                        const float* inv_temperature, int q_layout, int B, int n_max, int V,
                                        int32_t* path, int32_t* accept_len, int32_t* emitted, int32_t* n_emitted,
                                        void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * Tree K/V append.  "SpecInfer Guide", "Depth-First Flattening and KV Cache
 * Reuse", step 1 of the verification pass: every tree token appends the key
 * and value the target model computed for it to the active cache, in the
 * tree's node order, right after the committed prefix.  Row h of node u of
 * request b, k_new[tree_off[b] + u][h][0..D-1] (likewise v_new), is written
 * to slot prefix_len[b] + u of kv-head h through the block table; no other
 * slot changes.  This is how the tree K/V reach the slots that
 * spec_tree_attention reads.
 *   k_new, v_new  [T][Hkv][D] dtype, T = tree_off[B]; 16-byte aligned, as are the caches
 *                 (else SPEC_ERR_INVALID_ARG).  A prompt's rows are appended the same way
 *                 (tree_off = its packing, n_max = its longest request, of any length)
 *   k_cache, v_cache, block_table, max_blocks, block_size, num_blocks  as for attention
 *   prefix_len, tree_off  int32 [B], [B+1]
 *   status   int32 [B] in/out, or-ed with SPEC_DEV_BAD_TREE (n_b outside [0, n_max]),
 *            SPEC_DEV_CAPACITY (prefix_len < 0, or prefix_len + n_b beyond the block table)
 *            or SPEC_DEV_BAD_BLOCK (an id outside [0, num_blocks) among the pages of slots
 *            [prefix_len, prefix_len + n_b)); such a request is left untouched.  The
 *            incoming status is not read: an upstream failure does not stop the append.
 * Launched as a programmatic dependent of the previous kernel (the mask build
 * allows it at its start), it waits for that kernel's results before it reads
 * anything: k_new, v_new, the table, the lengths and the packing may come from
 * the kernel right before this call.  One launch, grid (B, parts).
 */
spec_status spec_kv_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                           const int32_t* block_table, int max_blocks, int block_size, int num_blocks,
                           const int32_t* prefix_len, const int32_t* tree_off, int B, int n_max, int Hkv, int D,
                           spec_dtype dtype, int32_t* status, void* stream);

/*
 * KV commit / rollback.  "SpecInfer Guide", "Depth-First Flattening and KV
 * Cache Reuse" and "PagedKV Allocation with Zero-Copy Pruning": only the
 * accepted path stays.  In place, for every kv-head: slot prefix_len[b] + i
 * receives the old slot prefix_len[b] + path[b][i], i < accept_len[b] (rows
 * already in place are not copied); new_len[b] = prefix_len[b] + accept_len[b].
 * Requests with a non-zero status on entry, or accept_len 0, are untouched
 * (new_len = prefix_len).  A path that is not strictly increasing from 0 or
 * leaves the block table sets SPEC_DEV_BAD_PATH; a bad block id sets
 * SPEC_DEV_BAD_BLOCK; such requests are untouched.
 *   path        int32 [B][path_stride]  accepted local node indices, root first
 *   accept_len  int32 [B]
 *   new_len     int32 [B] out
 *   status      int32 [B] in/out (or-ed)
 */
spec_status spec_kv_commit(void* k_cache, void* v_cache, const int32_t* block_table, int max_blocks,
                           int block_size, int num_blocks, const int32_t* prefix_len, const int32_t* path,
                           int path_stride, const int32_t* accept_len, int B, int Hkv, int D, spec_dtype dtype,
                           int32_t* new_len, int32_t* status, void* stream);

/*
 * Multi-layer KV commit and page release.  "SpecInfer Guide", "PagedKV
 * Allocation with Zero-Copy Pruning": after verification the accepted path is
 * compacted in every layer's cache (each layer exactly as spec_kv_commit
 * does, in one launch), then the tree's pages lying wholly past the new length
 * go back to the free pool in one metadata update.  The tree of request b
 * fills slots [prefix_len[b], prefix_len[b] + n_b); its pages
 * ceil(new_len / block_size) .. ceil((prefix_len + n_b) / block_size) - 1 are
 * released: their block-table entries become -1 and their ids are appended to
 * free_pool after *free_count, in request order then page order, and
 * *free_count grows by their number.  The entries are taken as the table
 * holds them (call once per pass: a second call over the same tree would
 * append the -1 entries the first left).  Requests with a non-zero status after
 * the commit keep every page.  When the pool cannot take every page of the
 * call (*free_count + released > free_cap), none is released and each request
 * that had pages to release gets SPEC_DEV_CAPACITY.
 *   k_caches, v_caches  device arrays of `layers` device pointers, each a paged
 *                       cache [num_blocks][Hkv][block_size][D] of dtype
 *   block_table int32 [B][max_blocks]  in/out (released entries become -1)
 *   tree_off    int32 [B+1]  tree sizes (as for the mask build)
 *   free_pool   int32 [free_cap], free_count int32 [1]: device memory, in/out;
 *               both NULL: commit only, no release
 *   other arguments as in spec_kv_commit.  Two kernels: the commit (grid
 *   B x Hkv x Z, each CTA moving the rows of every Z-th cache, Z chosen to
 *   fill the GPU about once), then the release (one CTA).
 */
spec_status spec_kv_commit_layers(void* const* k_caches, void* const* v_caches, int layers,
                                  int32_t* block_table, int max_blocks, int block_size, int num_blocks,
                                  const int32_t* prefix_len, const int32_t* tree_off, const int32_t* path,
                                  int path_stride, const int32_t* accept_len, int B, int Hkv, int D,
                                  spec_dtype dtype, int32_t* new_len, int32_t* free_pool, int free_cap,
                                  int32_t* free_count, int32_t* status, void* stream);

/*
 * Philox4x32-10 random words for one verification round (Salmon et al.,
 * "Parallel random numbers: as easy as 1, 2, 3", SC'11): node u (local index)
 * of request b uses counter (u, b, round, 0) and key (seed low 32 bits, seed
 * high 32 bits); out[t][0] = output word 0, out[t][1] = output word 1.
 *   tree_off int32 [B+1]; out uint32 [T][2]; n_max bounds n_b (larger requests are skipped).
 */
spec_status spec_philox_uniforms(uint64_t seed, uint32_t round, const int32_t* tree_off, int B, int n_max,
                                 uint32_t* out, void* stream);

/*
 * Token-tree construction ("SpecInfer Guide", "Token Tree Construction:
 * Expansion vs. Merge").  The trees come out in the layout the calls above
 * take (parent before child, packed by tree_off).
 *
 * spec_tree_init: request b's tree occupies n_total slots from b * n_total;
 * node 0 gets parent -1 and token root_tok[b] (the last verified token), and
 * tree_off[b] = b * n_total for b = 0..B (tree_off may be NULL).
 *   root_tok int32 [B]; tree_off int32 [B+1] out; parent, tokens int32 [B * n_total] out.
 *   n_total in [1, 1024].
 *
 * spec_tree_expand_level: one level of "Method A: Expansion-Based Tree
 * Construction": every frontier node gets its top-k tokens as children.
 * Every request has the same shape; its F frontier nodes are level_start ..
 * level_start + F - 1 and their children are appended after them, frontier
 * node by frontier node, each node's k children in rank order: child r of
 * frontier node i is node level_start + F + i * k + r, with parent
 * level_start + i.  Rank order: larger score first, equal scores by lower
 * token id, NaN after every number, -0 equal to +0.  A whole schedule
 * <k_1, ..., k_m> is spec_tree_init, then one call per level (level_start
 * 0, 1, 1 + k_1, ...), with the draft model's rows for the new frontier in
 * between.
 *   scores   float [B * F][V]  row b * F + i: draft scores (logits or probabilities)
 *                              of frontier node i of request b
 *   parent, tokens  int32 [B * n_total]  in/out: the level's children are written
 *   k in [0, 32], k <= V; level_start + F + F * k <= n_total <= 1024, else an error
 *   code and nothing is launched.
 *
 * spec_tree_merge: "Method B: Merge-Based Tree Construction": request b's
 * M candidate sequences (one per draft model: sequence s is
 * seqs[b][s][0 .. lens[b][s]-1]) are united into one tree in which every
 * prefix of every sequence is one node and no two nodes share a token path.
 * Node 0 is the root (root_tok[b]); the others are numbered in
 * first-appearance order (sequences in order, each from its first token).
 * The output is packed: tree_off is written (tree_off[0] = 0), request b's
 * nodes are tree_off[b] .. tree_off[b+1]-1.
 *   seqs     int32 [B][M][m]   candidate tokens (entries past a length are ignored)
 *   lens     int32 [B][M]      sequence lengths in [0, m]
 *   tree_off int32 [B+1] out
 *   parent, tokens int32 [B * (1 + M * m)] out (capacity; tree_off[B] entries written)
 *   src      int32 [same]  out: s * m + j of the prefix that created each node, -1 for roots
 *   node_of  int32 [B][M][m] out: the node (request-local index) of prefix (s, j), -1 past
 *                              the length; with it per-child draft rows can be gathered
 *   status   int32 [B]     out: WRITTEN (a merge starts a pass): 0, SPEC_DEV_BAD_TREE (a
 *                              length outside [0, m]) and/or SPEC_DEV_BAD_TOKEN (a token or
 *                              root token outside [0, V)); such a request gets only its root.
 *   M * m <= 1023 and M <= 1023.  Three launches (counts, offsets, nodes).
 */
spec_status spec_tree_init(const int32_t* root_tok, int B, int n_total, int32_t* tree_off, int32_t* parent,
                           int32_t* tokens, void* stream);
spec_status spec_tree_expand_level(const float* scores, int B, int F, int V, int k, int level_start, int n_total,
                                   int32_t* parent, int32_t* tokens, void* stream);
spec_status spec_tree_merge(const int32_t* seqs, const int32_t* lens, const int32_t* root_tok, int B, int M, int m,
                            int V, int32_t* tree_off, int32_t* parent, int32_t* tokens, int32_t* src,
                            int32_t* node_of, int32_t* status, void* stream);

/*
 * Prompt attention (the pages have no counterpart: they start from a committed
 * prefix; this call fills the prefix's hidden states).  Causal attention of
 * whole prompts, or of the next chunk of prompts, over the paged cache:
 * request b's new tokens are rows [seq_off[b], seq_off[b+1]) of q and out; row
 * i of them is the token at slot s = prefix_len[b] + i and sees slots 0 .. s:
 * out = sum_{k <= s} softmax_k(scale * q . K_k) V_k.  Query head h reads
 * kv-head h / (Hq / Hkv).  One token per request (n_b = 1) is the plain decode
 * step.  The rows' own K/V must be in the cache (spec_kv_append before this
 * call on the stream).  fp32 accumulation and softmax.  bf16 inputs give bf16
 * output, and each softmax weight is rounded to bf16 (by at most 2^-8 of it)
 * before it meets V; the weights are normalised by the sum of the rounded
 * ones.  Values of V may have any magnitude in fp32, and 0 or 2^-60 to 2^80 in
 * bf16 (weights reach 2^30 there before they are normalised).
 *   q        [T][Hq][D] dtype, T >= seq_off[B]; 16-byte aligned, as are out and the caches
 *            (else SPEC_ERR_INVALID_ARG)
 *   k_cache, v_cache, block_table, max_blocks, block_size, num_blocks  paged cache, see
 *            the conventions above.  Slots [0, prefix_len[b] + n_b) hold finite values; what
 *            lies in the pages behind them is never used.
 *   prefix_len int32 [B]    slots already filled before row 0 (0: a fresh prompt; <= max_prefix)
 *   seq_off  int32 [B+1]    packing; n_b may be 0
 *   n_max    the largest n_b the call may see (n_max * (Hq / Hkv) < 2^30; T * Hq < 2^31)
 *   scale    finite and not negative (else SPEC_ERR_INVALID_ARG)
 *   out      [T][Hq][D] dtype out; rows outside every request are not written
 *   workspace  16-byte aligned device scratch, used when the keys of few rows are split over
 *            the GPU.  spec_prompt_workspace_size() is what the call of these sizes wants
 *            (smaller batches often want more: fewer rows, more splits).  Any buffer of 256
 *            bytes or more will do: where it is too small for that the keys are split less
 *            and the call takes longer (else SPEC_ERR_WORKSPACE)
 *   status   int32 [B] in/out: a request that comes in non-zero is skipped, its rows left as
 *            they were.  Or-ed with SPEC_DEV_BAD_TREE (n_b outside [0, n_max], or rows outside
 *            [0, T)), SPEC_DEV_CAPACITY (prefix_len outside [0, max_prefix], or
 *            prefix_len + n_b beyond the block table): such a request is skipped too;
 *            (a seq_off that decreases flags a request whose n_b is negative; rows that two
 *            requests then both own are unspecified);
 *            SPEC_DEV_BAD_BLOCK (a block id outside [0, num_blocks)) and SPEC_DEV_TIMEOUT: its
 *            output rows are unspecified.
 */
size_t spec_prompt_workspace_size(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D);
spec_status spec_prompt_attention(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_table, int max_blocks, int block_size, int num_blocks,
                                  const int32_t* prefix_len, const int32_t* seq_off, int B, int T, int n_max,
                                  int max_prefix, int Hq, int Hkv, int D, spec_dtype dtype, float scale, void* out,
                                  void* workspace, size_t workspace_bytes, int32_t* status, void* stream);

/*
 * Log probabilities of given tokens, with the entropy of their distribution,
 * their rank and the top alternatives (what a server answers with beside the
 * tokens; the pages have no counterpart).  For a row of logits x and an
 * inverse temperature tau, p = softmax(tau * x):
 *   logprob = log p(token);  entropy = -sum_i p_i log p_i (nats; 0 log 0 = 0);
 *   rank = number of tokens that come before the given one, and top_tokens the
 *   first k, in the order of spec_tree_expand_level: larger logit first, equal
 *   logits by lower id, NaN after every number, -0 equal to +0;
 *   top_logprobs = their log p.
 * Logits of -inf have probability 0.  A row with a NaN, a +inf or nothing
 * above -inf has no distribution: its logprob, entropy and top_logprobs are
 * NaN, its rank and top_tokens as ordered above.
 *
 * spec_token_logprobs: packed rows; row t of logits is scored for tokens[t].
 * spec_path_logprobs: the tokens a verification emitted: entry (b, i),
 *   i < accept_len[b], scores emitted[b][i] with the row of node path[b][i]
 *   (logits row tree_off[b] + path[b][i]).  path, accept_len and emitted are
 *   the verifier's outputs; a request that failed there has accept_len 0.
 *
 *   logits   [T][V] of dtype, aligned to its element; V <= 131072
 *   tokens   int32 [T]; -1: no token given (logprob NaN, rank -1; the rest is computed)
 *   seq_off / tree_off int32 [B+1]
 *   inv_temperature float [B] (device) or NULL for tau = 1
 *   k        alternatives per entry, 0 <= k <= min(32, V)
 *   logprob, entropy float, rank int32: [T], or [B][n_max] for the path call; entropy and rank
 *            may be NULL
 *   top_tokens int32, top_logprobs float: [T][k], or [B][n_max][k]; either may be NULL
 *   status   int32 [B] or-ed (the incoming word is not read): SPEC_DEV_BAD_TOKEN (a token
 *            outside [0, V)), SPEC_DEV_BAD_TEMP (tau not in [1e-30, inf)), SPEC_DEV_BAD_PATH
 *            (accept_len above n_max, a path node outside the request's tree, or rows outside
 *            [0, T)); only the entries concerned are affected.  SPEC_DEV_TIMEOUT: entries may
 *            be unspecified
 * Entries without a result (i >= accept_len[b], rows outside every request,
 * flagged entries) get NaN, rank -1 and top_tokens -1.  One launch.
 */
spec_status spec_token_logprobs(const void* logits, spec_dtype dtype, const int32_t* tokens, const int32_t* seq_off,
                                const float* inv_temperature, int B, int T, int V, int k, float* logprob,
                                float* entropy, int32_t* rank, int32_t* top_tokens, float* top_logprobs,
                                int32_t* status, void* stream);
spec_status spec_path_logprobs(const void* p_logits, spec_dtype dtype, const int32_t* tree_off, const int32_t* path,
                               const int32_t* accept_len, const int32_t* emitted, const float* inv_temperature,
                               int B, int T, int n_max, int V, int k, float* logprob, float* entropy, int32_t* rank,
                               int32_t* top_tokens, float* top_logprobs, int32_t* status, void* stream);

/*
 * Page calls ("SpecInfer Guide", "PagedKV Allocation with Zero-Copy Pruning":
 * pages are handed out and taken back by metadata alone; sharing between rows
 * and compaction have no counterpart there).  A page is held by every row of
 * the block table that names it, free when it is among free_pool's first
 * *free_count entries, and otherwise the caller's own; the table is the only
 * record, so these calls and spec_kv_commit_layers' release need no counters.
 * Pages are taken from the pool's end.  Table entries below 0 mean "no page".
 * Slots are written (spec_kv_append, the commits) in pages that one row alone
 * names: a row that was cut back to a length inside a shared page
 * (spec_pages_free) goes on in an empty row forked from it, which gets a copy
 * of that page.  The release of spec_kv_commit_layers likewise returns the
 * pages behind a tree's new length without looking for them in other rows.
 *
 * spec_pages_fork: fork i makes row dst[i] hold the first len[i] slots of row
 *   src[i], with pages for room[i] further slots.  Full pages are shared; the
 *   slots of a partial last page are copied, in every layer, to a fresh page;
 *   the pages for room are fresh.  src[i] = -1 with len[i] = 0 is an empty
 *   row.  src[i] == dst[i] extends a row in place: its missing pages up to
 *   len[i] + room[i] slots are filled in (nothing is shared or copied).
 *   Fresh pages are taken in the order of i, then of the page.  When the pool
 *   has fewer pages than the call's sound forks need, none that needs a page
 *   is done and each of those gets SPEC_DEV_CAPACITY.
 *   status int32 [N] WRITTEN per fork: 0; SPEC_DEV_BAD_ROW (src outside
 *   [-1, B), dst outside [0, B), len or room < 0, src = -1 with len > 0, a row
 *   that is dst twice, a src that another fork has as dst, or a dst row with
 *   pages where new ones go); SPEC_DEV_CAPACITY (also len + room beyond the
 *   table); SPEC_DEV_BAD_BLOCK (a source page, or a pool entry about to be
 *   taken, outside [0, num_blocks)).  A flagged fork changes nothing.
 *
 * spec_pages_free: row rows[i] keeps its first keep_len[i] slots (keep_len
 *   NULL: none): its entries from page ceil(keep_len / block_size) on become
 *   -1, and the pages among them that no row names any more are appended to
 *   the pool in the order of i, then of the page, each once.  When the pool
 *   cannot take them all, nothing is done and each sound row that had a page to
 *   drop gets SPEC_DEV_CAPACITY, whoever else names that page.
 *   status int32 [N] WRITTEN per row: 0, SPEC_DEV_BAD_ROW (outside [0, B),
 *   named twice, keep_len < 0), SPEC_DEV_BAD_BLOCK (a dropped entry of
 *   num_blocks or more) or SPEC_DEV_CAPACITY; a flagged row is left as it was.
 *
 * spec_pages_compact: moves held pages to the lowest ids.  Among the pages
 *   that are held or free, in increasing id, the first n (n = held pages)
 *   become the held ones: the i-th free page among them receives the i-th held
 *   page beyond them, in every layer.  The table is renumbered, the pool lists
 *   the remaining pages by decreasing id (so that the lowest is taken first;
 *   *free_count is unchanged), and page_map tells callers who keep ids
 *   elsewhere.  The caller's own pages stay.
 *   page_map int32 [num_blocks] out: new id of each page; moved int32 [1] out
 *   status int32 [1] WRITTEN: 0, or SPEC_DEV_BAD_BLOCK (an id out of range in
 *   the table or the pool, a page twice in the pool, or both held and in the
 *   pool, or a *free_count outside [0, free_cap]): nothing is changed then.
 *
 *   k_caches, v_caches  device arrays of `layers` device pointers, as in spec_kv_commit_layers,
 *            each cache 16-byte aligned; layers = 0 (pointers NULL): metadata only
 *   block_table int32 [B][max_blocks] in/out; B * max_blocks and N * max_blocks <= 2^30
 *   free_pool int32 [free_cap], free_count int32 [1]: device memory, in/out
 *   workspace  16-byte aligned device scratch of spec_pages_workspace_size() bytes (N of the
 *            call; 0 for compact)
 */
size_t spec_pages_workspace_size(int B, int max_blocks, int num_blocks, int N);
spec_status spec_pages_fork(void* const* k_caches, void* const* v_caches, int layers, int32_t* block_table, int B,
                            int max_blocks, int block_size, int num_blocks, const int32_t* src, const int32_t* dst,
                            const int32_t* len, const int32_t* room, int N, int Hkv, int D, spec_dtype dtype,
                            int32_t* free_pool, int free_cap, int32_t* free_count, void* workspace,
                            size_t workspace_bytes, int32_t* status, void* stream);
spec_status spec_pages_free(int32_t* block_table, int B, int max_blocks, int block_size, int num_blocks,
                            const int32_t* rows, const int32_t* keep_len, int N, int32_t* free_pool, int free_cap,
                            int32_t* free_count, void* workspace, size_t workspace_bytes, int32_t* status,
                            void* stream);
spec_status spec_pages_compact(void* const* k_caches, void* const* v_caches, int layers, int32_t* block_table, int B,
                               int max_blocks, int block_size, int num_blocks, int Hkv, int D, spec_dtype dtype,
                               int32_t* free_pool, int free_cap, int32_t* free_count, int32_t* page_map,
                               int32_t* moved, void* workspace, size_t workspace_bytes, int32_t* status,
                               void* stream);

/*
 * Head norms, rotary positions and the append in one pass (the pages take
 * queries and cache rows as given; this call makes them from a projection's
 * output).  Row t of qkv holds Hq query, Hkv key and Hkv value heads of D
 * elements.  Query and key heads are normalised, x w / sqrt(mean(x^2) + eps),
 * then the first rot_dim elements of a head are turned by pairs:
 *   (x, y) -> (x cos a - y sin a, y cos a + x sin a),  a = position * inv_freq[i]
 * for pair i < rot_dim / 2: elements i and i + rot_dim / 2 (SPEC_ROPE_HALVES) or
 * 2 i and 2 i + 1 (SPEC_ROPE_NEIGHBOURS).  Queries go to q_out, keys and values
 * to slot prefix_len[b] + u of row u of request b, as spec_kv_append puts them.
 * fp32 arithmetic, the angle in 64 bits; results are rounded once to dtype,
 * values are copied bit for bit.
 * Positions are not slots: a request that lost slots (spec_kv_evict) goes on at
 * the positions of its text.  Row u of request b has position
 *   pos_base[b] + (pos ? pos[axis * T + tree_off[b] + u] : u)
 * on each of `axes` axes (time, height and width of an image, say).  A tree's
 * nodes: pos = the depth of spec_tree_mask_build, axes = 1.
 *   qkv      [T] rows of dtype, row_stride elements apart (>= (Hq + 2 Hkv) D), 16-byte
 *            aligned, as are row_stride in bytes, q_out, the caches and the norms' weights
 *   q_norm, k_norm  [D] dtype, either may be NULL: those heads are not normalised; eps >= 0
 *   inv_freq float [rot_dim / 2], finite (radians per position); NULL with rot_dim = 0
 *   axis     int32 [rot_dim / 2]: the axis of each pair; NULL: axis 0 (axes = 1)
 *   rot_dim  even, 0 <= rot_dim <= D (0: no rotation, no position is read)
 *   pos_base int32 [B] or NULL for prefix_len;  pos int32 [axes][T] or NULL (axes = 1)
 *   axes     1 to 4
 *   q_out    [T][Hq][D] dtype out, apart from qkv; rows outside every request are not written
 *   k_cache, v_cache, block_table, max_blocks, block_size, num_blocks, prefix_len, tree_off,
 *   n_max    as for spec_kv_append (packed prompts have no limit of 1024 rows).  The rows of
 *            requests behind a tree_off that decreases are unspecified
 *   status   int32 [B] in/out, not read, or-ed with SPEC_DEV_BAD_TREE (n_b outside [0, n_max],
 *            or rows outside [0, T)), SPEC_DEV_CAPACITY or SPEC_DEV_BAD_BLOCK as for
 *            spec_kv_append: such a request is left untouched.  SPEC_DEV_BAD_POSITION: the
 *            rows with such a position are left untouched
 * Launched as a programmatic dependent of the previous kernel; it waits for that
 * kernel's results before it reads anything.  One launch.
 */
#define SPEC_ROPE_HALVES 0
#define SPEC_ROPE_NEIGHBOURS 1
spec_status spec_rope_append(const void* qkv, long long row_stride, const void* q_norm, const void* k_norm, float eps,
                             const float* inv_freq, const int32_t* axis, int rot_dim, int pairing,
                             const int32_t* pos_base, const int32_t* pos, int axes, void* q_out, void* k_cache,
                             void* v_cache, const int32_t* block_table, int max_blocks, int block_size, int num_blocks,
                             const int32_t* prefix_len, const int32_t* tree_off, int B, int T, int n_max, int Hq,
                             int Hkv, int D, spec_dtype dtype, int32_t* status, void* stream);

/*
 * Attention weight gathered by cached slots (no counterpart on the pages): how
 * much the attention of a layer looked at every slot, per kv-head, the measure
 * that spec_kv_evict keeps slots by.  For slot s of request b and kv-head h
 *   weight[b][h][s] = decay * before[b][h][s] + sum softmax_s(scale * q . K)
 * over the query heads of the group and the counted rows, each row over the
 * slots it sees.  Slots of the request's own new rows (s >= prefix_len[b]) have
 * no `before`.  The rows are those of spec_prompt_attention: row i of request b
 * is the token at slot prefix_len[b] + i and sees slots 0 .. prefix_len[b] + i;
 * or, with `path` and `accept_len`, the accepted path of a verification AFTER its
 * commit: token i < accept_len[b] has its queries in row tree_off[b] + path[b][i]
 * of q and its key in slot prefix_len[b] + i (seq_off = tree_off, prefix_len as
 * before the commit).  Sums, maxima and weights are fp32; each slot's weight is
 * summed in a fixed order.
 *   q        [T][Hq][D] dtype, as the attention call had it; 16-byte aligned, as is k_cache
 *   k_cache, block_table, max_blocks, block_size, num_blocks, prefix_len, seq_off, B, T, n_max,
 *   max_prefix  as for spec_prompt_attention (slots [0, prefix_len[b] + rows) hold finite keys;
 *            what lies in the pages behind them is never used)
 *   path     int32 [B][path_stride] and accept_len int32 [B], or both NULL: every row
 *   window   > 0: only the last `window` rows of a request count; 0: all
 *   scale, decay  finite and not negative (else SPEC_ERR_INVALID_ARG)
 *   before   float [B][Hkv][weight_stride], or NULL for zeros;  weight  the same shape, out;
 *            they may be one buffer.  Only slots [0, prefix_len[b] + rows) are read and
 *            written.  A request without rows has its weights decayed
 *   workspace  16-byte aligned device scratch of spec_weight_workspace_size() bytes, which are
 *            enough for every batch of no larger sizes too, whatever its window and type; calls
 *            that may run at once need one each
 *   status   int32 [B] in/out: a request that comes in non-zero is left as it was.  Or-ed with
 *            SPEC_DEV_BAD_TREE, SPEC_DEV_CAPACITY (also prefix_len + rows beyond
 *            weight_stride), SPEC_DEV_BAD_PATH (accept_len outside [0, min(path_stride, n_b)],
 *            or a counted path node outside the tree): left as it was;
 *            SPEC_DEV_BAD_BLOCK and SPEC_DEV_TIMEOUT: its weights are unspecified
 */
size_t spec_weight_workspace_size(int B, int T, int n_max, int max_prefix, int Hq, int Hkv, int D);
spec_status spec_attention_weight(const void* q, const void* k_cache, const int32_t* block_table, int max_blocks,
                                  int block_size, int num_blocks, const int32_t* prefix_len, const int32_t* seq_off,
                                  const int32_t* path, int path_stride, const int32_t* accept_len, int window, int B,
                                  int T, int n_max, int max_prefix, int Hq, int Hkv, int D, spec_dtype dtype,
                                  float scale, float decay, const float* before, float* weight,
                                  long long weight_stride, void* workspace, size_t workspace_bytes, int32_t* status,
                                  void* stream);

/*
 * Eviction by weight (no counterpart on the pages): eviction i copies what row
 * src[i] of the block table keeps of its len[i] slots to row dst[i], in every
 * layer.  Each layer and kv-head keeps kept = min(keep[i], len[i]) slots: the
 * first min(first, kept), the last min(last, kept - first), and, of the slots
 * between, those of the largest weight (equal weights by lower slot, NaN after
 * every number, -0 equal to +0).  They keep their order: the j-th kept slot
 * becomes slot j of dst[i], K, V and weight.  Keys keep the positions they were
 * rotated by.  Row src[i] stays as it was: shared pages may be evicted from;
 * spec_pages_free gives the row's pages back.
 *   k_caches, v_caches, layers  as in spec_pages_fork (layers >= 1)
 *   block_table int32 [B][max_blocks], read: dst rows have pages of their own for kept slots
 *            (spec_pages_fork of an empty row with room), which no source row names
 *   src, dst, len int32 [N];  keep int32 [N] or NULL for keep_max in every row
 *   keep_max the most slots a row may keep
 *   weight   float [layers][B][Hkv][weight_stride] by table row, in/out, or NULL: all equal
 *            (first and last alone then say what stays, as in a sliding window)
 *   slots    int32 [layers][N][Hkv][keep_max] out: the kept slots of src[i], increasing, then -1
 *   new_len  int32 [N] out: kept, the length of row dst[i] (0 for a flagged one)
 *   status   int32 [N] WRITTEN: 0; SPEC_DEV_BAD_ROW (src or dst outside [0, B), src = dst, a dst
 *            named twice or a src of the call, len < 0, keep outside [0, keep_max]);
 *            SPEC_DEV_CAPACITY (len beyond the table, weight_stride or 2^30);
 *            SPEC_DEV_BAD_BLOCK (a page of either row outside [0, num_blocks)).  A flagged
 *            eviction copies nothing
 * No workspace.  One launch where the CTAs that select also copy (layers * N * Hkv of two
 * or more per SM, or little to copy), else two.
 */
spec_status spec_kv_evict(void* const* k_caches, void* const* v_caches, int layers, const int32_t* block_table, int B,
                          int max_blocks, int block_size, int num_blocks, const int32_t* src, const int32_t* dst,
                          const int32_t* len, const int32_t* keep, int N, int keep_max, int first, int last,
                          float* weight, long long weight_stride, int Hkv, int D, spec_dtype dtype, int32_t* slots,
                          int32_t* new_len, int32_t* status, void* stream);

/*
 * Dynamic draft length ("Hardware-aware dynamic speculative decoding",
 * "Dynamic speculative decoding" and "Compatibility with full CUDA Graph"):
 * the scheduler picks, per step, the number of draft tokens K of highest
 * goodput = AL / ITL (acceptance length over inter-token latency) for the
 * current batch size, from a table profiled offline and refreshed with live
 * statistics, and replays the full CUDA graph captured for <tokens, K>.
 * HOST functions: every pointer is host memory; nothing is launched.
 *
 * spec_dsd_optimal_k: al, itl double [n_bs][n_k] (measured AL and ITL for the
 *   draft lengths k_values[0..n_k-1] at each profiled batch size); a cell
 *   counts when both are finite and itl > 0.  k_opt int32 [n_bs] out: the K
 *   of the largest goodput in each row, the earliest column on ties; -1 when
 *   no cell of the row counts.
 * spec_dsd_select_k: bs_table int32 [n] strictly ascending (else
 *   SPEC_ERR_INVALID_ARG), k_table int32 [n]; *k_out = the entry of the
 *   largest bs_table[i] <= bs, or k_table[0] when bs < bs_table[0].
 * spec_dsd_update: folds one live measurement into cell (bs_index, k_index):
 *   x <- x + weight * (sample - x), weight in (0, 1]; a cell that is not
 *   finite (unmeasured) takes the sample.  Samples must be finite.
 * spec_dsd_graph_keys: every <tokens, K> with 1 <= tokens <= max_tokens and
 *   1 <= K <= max_k such that tokens is divisible by K + 1 (every request of
 *   the batch is then a decode request with K drafts), ordered by tokens
 *   then K.  *count = their number; the first min(cap, count) are stored.
 */
spec_status spec_dsd_optimal_k(const double* al, const double* itl, int n_bs, int n_k, const int32_t* k_values,
                               int32_t* k_opt);
spec_status spec_dsd_select_k(const int32_t* bs_table, const int32_t* k_table, int n, int bs, int32_t* k_out);
spec_status spec_dsd_update(double* al, double* itl, int n_bs, int n_k, int bs_index, int k_index, double al_sample,
                            double itl_sample, double weight);
spec_status spec_dsd_graph_keys(int max_tokens, int max_k, int32_t* tokens_out, int32_t* k_out, int cap,
                                int32_t* count);

/*
 * Diagnostic of the bounded device waits (no counterpart on the pages): one
 * small kernel waits on a barrier that nothing ever completes, with a limit of
 * `polls` polls (1 .. 2^20), the same wait the tensor-core attention roles use
 * with a limit of 2^25; on expiry it or-s SPEC_DEV_TIMEOUT into status[0] and
 * returns, leaving the context usable.
 */
spec_status spec_selftest_bounded_wait(int32_t* status, uint32_t polls, void* stream);

/*
 * Diagnostics of the stochastic verifier's arithmetic contract (no
 * counterpart on the pages).  They run the very device functions the
 * verifier uses (the exp E, the fixed-point weight FX and its two
 * accumulators, the residual step) over arrays, so that a test can compare
 * them bit for bit with an independent implementation of the contract
 * described at spec_tree_verify_stochastic.  Device pointers, asynchronous on
 * `stream`; SPEC_ERR_INVALID_ARG for a negative n, a bad segment or no output.
 *
 * spec_selftest_exp: x_i is the fp32 whose bit pattern is first_bits + i
 *   (modulo 2^32), i < n.  exp_scalar[i] = E(x_i) by the scalar routine;
 *   exp_pair[i] = E(x_i) by the two-lane routine, entries 2k and 2k+1 forming
 *   one pair.  Either output may be NULL.
 * spec_selftest_fx: v float [n] (the contract's domain is [0, 2)).
 *   fx_out[i] = trunc(v[i] * 2^46); for each of the n / seg segments of seg
 *   consecutive entries (1 <= seg <= 510, n a multiple of seg), seg_scalar[s]
 *   = the fixed-point sum of the segment by the scalar accumulator and
 *   seg_pair[s] = the same by the two-lane accumulator (seg even).  Any
 *   output may be NULL (not all three).
 * spec_selftest_resid: one residual step max(d / Z - q, 0) of the contract
 *   per entry i < n, with Z = Zp[i / 2] (Zp holds ceil(n / 2) normalisers;
 *   entries 2k and 2k+1 share one, as in the verifier's paired passes):
 *   r_div by IEEE division, r_markstein by the scalar Markstein sequence the
 *   residual passes use (y = RN(1/Z)), r_pair by its two-lane form.  Any
 *   output may be NULL (not all three).
 */
spec_status spec_selftest_exp(uint32_t first_bits, long long n, float* exp_scalar, float* exp_pair, void* stream);
spec_status spec_selftest_fx(const float* v, long long n, int seg, uint64_t* fx_out, uint64_t* seg_scalar,
                             uint64_t* seg_pair, void* stream);
spec_status spec_selftest_resid(const float* d, const float* q, const float* Zp, long long n, float* r_div,
                                float* r_markstein, float* r_pair, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECTREE_H */
