/*
 * tv.h -- C ABI of libtv: GB300 (sm_103a) tree-verify MLA-absorb attention for DDTree
 * speculative decoding.
 *
 * The operations come from three web pages about a native DDTree engine:
 *   [RoPE]   "Precision as Correctness: The Float64 RoPE Decision in a Custom CUDA
 *             Inference Engine"
 *   [VERIFY] "The Precision Imperative: Validating Numerical Accuracy in a Custom CUDA
 *             Attention Kernel"
 *   [GOLDEN] "The Golden Reference: A Pivotal Moment in Building a Native DDTree
 *             Inference Engine"
 *
 * One verify step of a draft tree with q_len = Q nodes (node 0 is the root) over a
 * sequence whose cache already holds prefix_len = P tokens is:
 *   1. tv_build_visibility: parent array -> ancestor-or-self bitsets and depths;
 *   2. tv_rope_neox: NeoX RoPE at position P + depth on the queries' rope part, and on the
 *      draft tokens' k_pe rows, which it writes into cache slots P + node;
 *   3. tv_verify_attn: for every (sequence, node, head), softmax attention in latent
 *      space over the P prefix keys plus the node's ancestor-or-self tree keys, returning
 *      the softmax-weighted sum of latent rows and the log-sum-exp of the scores.
 *
 * Conventions (every entry point):
 *   - Tensor pointers are DEVICE pointers owned by the caller, unless stated otherwise.
 *     The library allocates no device memory; scratch is a caller-provided workspace.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy default stream).
 *     The return value reports synchronous argument checks and launch errors only.
 *   - Calls make no synchronising CUDA call, so they can be captured into a CUDA graph on
 *     a capturing stream.  The first call in a process (or on a new device) does one-time
 *     set-up (occupancy query, driver entry points); make it outside a capture.  A graph
 *     keeps the call's arguments, sizes and workspace as they were when it was captured.
 *   - Data-dependent errors found on the device (an invalid parent array, a prefix that
 *     does not fit the cache geometry, a device wait that ran out) are stored as a
 *     negative tv_status into *status, a caller-owned device int32.  The library never
 *     clears it: set it to TV_OK before the first call and read it when convenient.
 *     `status` may be NULL, in which case such errors are dropped silently.
 *   - On a non-OK return, tv_last_error() (thread-local) describes the failure.
 *   - Element strides are in ELEMENTS, not bytes.
 */
#ifndef TV_H_
#define TV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  TV_OK = 0,
  TV_ERR_INVALID_ARG = -1,  /* a pointer, size or stride is invalid */
  TV_ERR_INVALID_TREE = -2, /* parent[0] != -1 or parent[i] outside [0, i) */
  TV_ERR_UNSUPPORTED = -3,  /* valid but outside what the library implements (Q > 64 ...) */
  TV_ERR_CUDA = -4,         /* a CUDA runtime/driver call failed (see tv_last_error) */
  TV_ERR_TIMEOUT = -5,      /* a bounded device-side wait gave up (device status only) */
  TV_ERR_WORKSPACE = -6,    /* workspace missing or smaller than the size query asked for */
  TV_ERR_BOUNDS = -7,       /* prefix_len[b] + Q exceeds the cache geometry (device) */
  TV_ERR_NO_PAGES = -8      /* too few free pages in the pool (device status only) */
} tv_status;

typedef enum { TV_F32 = 0, TV_BF16 = 1 } tv_dtype;

/* Kernel family for tv_verify_attn.  AUTO picks by shape and dtype; the others force one
 * family (used by tests to check both) and fail with TV_ERR_UNSUPPORTED when it cannot
 * run the request. */
typedef enum { TV_PATH_AUTO = 0, TV_PATH_SIMT = 1, TV_PATH_TCGEN05 = 2 } tv_path;

/* How the tensor-core path reads a paged cache.  AUTO (and TV_PAGED_STEP_MAPS) builds two
 * tensor maps per 128-key step that read the two 64-token pages of the step in place;
 * TV_PAGED_GATHER first copies the pages into a contiguous key view in the workspace
 * (needs B * (max_prefix_len + Q rounded up to 128) < 2^31 rows, else the maps are used).
 * Ignored by the CUDA-core path and by contiguous caches. */
typedef enum { TV_PAGED_AUTO = 0, TV_PAGED_STEP_MAPS = 1, TV_PAGED_GATHER = 2 } tv_paged_view;

/* Which keys a query row sees (tv_attn_args.mask_mode).  [GOLDEN] §"Principled
 * Abstraction": one forward_tokens call serves tree verification, autoregressive decoding
 * (one query, every key) and prefill (causal masking).
 *   TV_MASK_TREE   : node i sees the P prefix keys and its ancestor-or-self tree keys
 *                    (anc bitsets from tv_build_visibility; Q <= 64);
 *   TV_MASK_CAUSAL : query token i (at logical key P + i) sees keys 0 .. P + i: prefill of
 *                    Q tokens after a cache of P (P = 0: no prior cache); anc is not read
 *                    and may be NULL; Q is limited only by B*Q*H < 2^31. */
typedef enum { TV_MASK_TREE = 0, TV_MASK_CAUSAL = 1 } tv_mask_mode;

/*
 * Geometry of the latent KV cache.  Logical key j (0 <= j < prefix_len[b] + Q) of
 * sequence b lives in cache row
 *     page_table[b*max_pages + j/page_size]*page_size + j%page_size   (paged), or
 *     b*kv_stride_b + j                                                (page_table NULL).
 * The draft-tree token of node i occupies logical key prefix_len[b] + i.  ([GOLDEN]
 * §"Recursive Refinement of the Decode Loop Design" works out the cache slots of the root
 * and draft tokens without printing a formula; the reading taken here is that the tree
 * tokens follow the prefix in node order.)  Paged caches need page_size == 64 on the
 * tensor-core path.
 */
typedef struct {
  const int32_t* page_table; /* device [B, max_pages] int32, or NULL for contiguous */
  int32_t page_size;         /* tokens per page (paged layout) */
  int32_t max_pages;         /* row stride of page_table, pages per sequence at most */
  int64_t kv_stride_b;       /* contiguous layout: cache rows per sequence */
  int64_t num_rows;          /* rows in the c_kv / k_pe arrays; bounds the tensor-core
                                path's TMA reads (0 = unknown: that path is not used) */
} tv_cache_layout;

/*
 * tv_build_visibility -- ancestor-or-self bitsets of a draft tree.
 *
 * [VERIFY] §Context: the verify kernel applies a visibility mask that decides which tree
 * tokens each query may attend to; [GOLDEN] §"Principled Abstraction": the step is M query
 * tokens against the cache under an [M, kv_len] mask.  Each node sees its ancestors and
 * itself.
 *
 * parent     : device [B, Q] int32, topologically ordered: parent[b*Q] == -1 and
 *              0 <= parent[b*Q+i] < i for i > 0.
 * anc        : device [B, Q] uint64 out; bit k of anc[b*Q+i] is set iff node k is node i or
 *              one of its ancestors.
 * depth      : device [B, Q] int32 out; parent steps from node i to the root.
 * dense_mask : device [B, Q, Q] uint8 out, nullable; dense_mask[(b*Q+i)*Q+k] = bit k of
 *              anc[b*Q+i].
 * status     : see the conventions above.  A sequence with an invalid parent array gets
 *              anc = 0, depth = -1 (and an all-zero mask row) and TV_ERR_INVALID_TREE.
 * Returns TV_ERR_UNSUPPORTED for Q > 64 (one 64-bit word per node), TV_ERR_INVALID_ARG
 * for B < 0, Q < 1 or a NULL parent/anc/depth with B > 0.
 */
int tv_build_visibility(const int32_t* parent, int B, int Q, uint64_t* anc, int32_t* depth,
                        uint8_t* dense_mask, int32_t* status, void* stream);

/*
 * tv_rope_neox -- NeoX (rotate-half) rotary embedding with a float64 angle.
 *
 * [RoPE] §"The Message" and §"What Input Knowledge Is Required" (item 1): split the rope
 * vector in half and rotate each pair (k, k + d_rope/2) by cos/sin of the angle;
 * §"The Float64 Decision": the angle and the trigonometry run in double precision and the
 * result is converted to float32 at the end.  Here the rotation itself is also done in
 * double, so the float32 result carries one rounding; bf16 output rounds that float32
 * value to nearest-even once more.
 *
 * For every (b, i, h), with pos = prefix_len[b] + depth[b*Q+i] and, for k < d_rope/2,
 * inv_k = 1 / base^(2k/d_rope), a = pos * inv_k:
 *     out[k]          = in[k] cos a - in[k + d/2] sin a
 *     out[k + d/2]    = in[k + d/2] cos a + in[k] sin a
 *
 * in  : element (b, i, h, r) at in[(b*Q+i)*in_stride_row + h*in_stride_head + r].
 * out : element (b, i, h, r) at out[row*out_stride_row + h*out_stride_head + r] where
 *       row = b*Q+i when out_cache is NULL, else the cache row of logical key
 *       prefix_len[b] + i under *out_cache (host struct; the draft tokens' k_pe rows are
 *       rotated straight into their cache slots).  in == out with equal strides is
 *       allowed (in place).
 * in_dt / out_dt : TV_F32 or TV_BF16 each.
 * prefix_len [B], depth [B, Q]: device int32 (depth from tv_build_visibility; a negative
 *       depth -- an invalid tree -- leaves that row untouched).  depth may be NULL: then
 *       row i is at position prefix_len[b] + i (a chain of tokens, as in prefill).  With out_cache, rows whose
 *       slot lies outside the geometry (negative prefix_len, a page index >= max_pages, a
 *       negative page-table entry, or a slot >= kv_stride_b) are skipped.
 * Returns TV_ERR_INVALID_ARG for odd or non-positive d_rope, n_heads < 1, or strides
 * that make rows overlap.
 */
int tv_rope_neox(const void* in, tv_dtype in_dt, int64_t in_stride_row,
                 int64_t in_stride_head, void* out, tv_dtype out_dt, int64_t out_stride_row,
                 int64_t out_stride_head, const tv_cache_layout* out_cache, int B, int Q,
                 int n_heads, int d_rope, const int32_t* prefix_len, const int32_t* depth,
                 double base, void* stream);

/*
 * Arguments of tv_verify_attn (absorbed-MLA tree-verify attention).
 *
 * [VERIFY] §"Input Knowledge Required" and [GOLDEN] §"The Absorb Form of MLA": the key
 * projection is folded into the query, so the score of query row (b, i, h) against key j
 * is taken in latent space:
 *     s_j = scale * ( q_latent[b,i,h,:] . c_kv[j,:]  +  q_pe[b,i,h,:] . k_pe[j,:] )
 * over the visible keys V = { j < P_b } U { P_b + k : bit k of anc[b*Q+i] }, and
 *     out[b,i,h,:] = sum_{j in V} softmax(s)_j * c_kv[j,:],   lse[b,i,h] = ln sum exp(s_j).
 * With mask_mode = TV_MASK_CAUSAL the visible set is V = { j <= P_b + i } instead (prefill;
 * Q > 64 allowed, anc unused).
 */
typedef struct {
  uint32_t struct_size;     /* sizeof(tv_attn_args): ABI check */
  int32_t B, H, Q;          /* batch, heads, q_len (tree nodes, 1..64) */
  int32_t d_latent, d_rope; /* d_latent % 8 == 0, d_rope % 8 == 0 (vector loads) */
  float scale;              /* softmax scale */
  tv_dtype q_dt, kv_dt;     /* (F32, F32) or (BF16, BF16) */
  const void* q_latent;     /* [B, Q, H, d_latent] contiguous */
  const void* q_pe;         /* [B, Q, H, d_rope] contiguous, RoPE already applied */
  const void* c_kv;         /* cache rows, row r at c_kv + r*ckv_row_stride (16 B aligned) */
  const void* k_pe;         /* cache rows, row r at k_pe + r*kpe_row_stride (16 B aligned) */
  int64_t ckv_row_stride, kpe_row_stride; /* elements; rows 16-byte aligned */
  tv_cache_layout cache;    /* where key j of sequence b lives */
  const int32_t* prefix_len; /* device [B] int32, 0 <= prefix_len[b] <= max_prefix_len */
  int32_t max_prefix_len;   /* host-side bound on prefix_len, sizes the launch */
  const uint64_t* anc;      /* device [B, Q] from tv_build_visibility */
  float* out;               /* device [B, Q, H, d_latent] float32 out */
  float* lse;               /* device [B, Q, H] float32 out (natural log) */
  int32_t* status;          /* device int32, nullable (see conventions) */
  int32_t path;             /* tv_path; TV_PATH_AUTO normally */
  int32_t num_splits;       /* 0 = automatic; else cut every KV sweep into this many
                               pieces (tensor cores: each 128-row tile's sweep) */
  int32_t paged_view;       /* tv_paged_view; TV_PAGED_AUTO normally */
  int32_t mask_mode;        /* tv_mask_mode; TV_MASK_TREE for tree verification */
  int32_t overlap_prev;     /* 0 normally.  1: the call that queued the stream's last work before
                               this one (one with nothing to do, such as a copy of an empty
                               list, queues none) writes none of prefix_len and the page table
                               (as for tv_verify_prologue, which writes q_pe, cache rows, anc);
                               the tensor-core path's preparation kernel (work schedule,
                               per-step tensor maps) may then run while that call finishes.
                               Calls before that one may write them (tv_pages_reserve, say,
                               with tv_pages_copy between): this library's calls let it start
                               only once the call before them has ended.  The attention itself
                               still starts only after all of it. */
} tv_attn_args;

/* Bytes of workspace tv_verify_attn needs for these arguments (0 if none).  The size
 * depends on B, H, Q, d_latent, max_prefix_len, whether the cache is paged, the path,
 * num_splits and paged_view only (the tensor-core path of a paged cache keeps two tensor
 * maps per 128-key step there, or with TV_PAGED_GATHER a contiguous copy of the keys). */
size_t tv_verify_attn_workspace_size(const tv_attn_args* a);

/* The kernel family TV_PATH_AUTO resolves to for these arguments, or a negative
 * tv_status if the arguments are invalid. */
int tv_verify_attn_path(const tv_attn_args* a);

/* How many kernels one tv_verify_attn call with these arguments enqueues (for launch
 * accounting; the CUDA-core path: attention + split combine; the tensor-core path: work
 * preparation + key gather (TV_PAGED_GATHER only) + attention + the merge of split tiles
 * unless num_splits == 1), or a negative tv_status if the arguments are invalid. */
int tv_verify_attn_launches(const tv_attn_args* a);

/*
 * tv_verify_attn -- run the attention.  workspace: device memory of at least
 * tv_verify_attn_workspace_size(a) bytes, 256-byte aligned (NULL allowed when the size
 * is 0); it is scratch and may be reused once the call's work on `stream` is done.
 * Rows of a sequence whose prefix_len is negative or does not fit the cache geometry get
 * out = 0, lse = -inf and TV_ERR_BOUNDS in *status.  Page-table entries of the pages that
 * hold keys 0 .. prefix_len[b]+Q-1 must name valid cache pages (they are not checked).
 */
int tv_verify_attn(const tv_attn_args* a, void* workspace, size_t ws_bytes, void* stream);

/*
 * tv_verify_attn_noalloc -- tv_verify_attn for callers that cannot allocate device memory.
 *
 * The pages describe nothing like this; it exists for callers that cannot give the library
 * a workspace: a plugin inside a host program that owns all device memory and offers no
 * allocator, a serving loop that must not call cudaMalloc/cudaFree because they can
 * synchronise the device, or a caller whose device memory budget is fixed in advance.
 *
 * It runs the CUDA-core attention kernel (TV_PATH_AUTO or TV_PATH_SIMT; TV_PATH_TCGEN05
 * is rejected) and keeps the split-KV partial results in a fixed array of
 * TV_NOALLOC_SCRATCH_BYTES bytes that the library reserves in device memory on every GPU
 * that loads it, held until the process exits.  It never allocates.  The caller still
 * passes every input and output through `a`.
 *   - The first call on a device looks up the array's address on that device (a
 *     cudaGetSymbolAddress), whatever the request; so does the first call after the
 *     device's CUDA context changed (cudaDeviceReset, or another context made current),
 *     since the array then lives in a newly loaded module.  Make such a first call before
 *     any stream capture.
 *   - A request whose scratch need exceeds TV_NOALLOC_SCRATCH_BYTES returns
 *     TV_ERR_WORKSPACE with an explanation in tv_last_error().  The need is what
 *     tv_verify_attn_workspace_size(a) reports for the same arguments with
 *     a->path = TV_PATH_SIMT (with TV_PATH_AUTO on a tensor-core shape that query reports
 *     the tensor-core path's size instead).
 *   - All calls share the one array and it keeps the last call's contents (nothing in it
 *     needs to start at zero).  Calls whose kernels can overlap on the GPU -- unordered
 *     streams, several host threads -- race on it; the caller must serialise them.
 * Results equal tv_verify_attn's on the CUDA-core path.
 */
#define TV_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
int tv_verify_attn_noalloc(const tv_attn_args* a, void* stream);

/* Size in bytes of the fixed scratch array behind tv_verify_attn_noalloc. */
size_t tv_noalloc_scratch_bytes(void);

/*
 * tv_verify_prologue -- the steps before tv_verify_attn in one launch.
 *
 * [RoPE] §"The Thinking Process": cos/sin are computed once and reused; [RoPE] §"The
 * Broader Context: A Full Native Engine from Scratch": the engine manages the KV cache;
 * [VERIFY] §Context: the visibility mask.  Same results, bit for bit, as
 *     tv_build_visibility(parent -> anc, depth)
 *     tv_rope_neox(q_pe_in -> q_pe_out, position prefix_len + depth)
 *     tv_rope_neox(kpe_tree -> k_pe cache slots prefix_len + i)
 * plus the copy of the draft tokens' latent rows ckv_tree[b,i,:] into c_kv cache slot
 * prefix_len[b] + i, with each node's cos/sin computed once for all of them.
 */
typedef struct {
  uint32_t struct_size;      /* sizeof(tv_prologue_args): ABI check */
  int32_t B, Q, H;           /* Q <= 64 (tree) */
  int32_t d_latent, d_rope;  /* d_rope % 8 == 0, d_rope <= 512, H * d_rope <= 8192;
                                d_latent % 8 == 0 */
  const int32_t* parent;     /* device [B, Q] draft tree */
  const int32_t* prefix_len; /* device [B] */
  const void* q_pe_in;       /* device [B, Q, H, d_rope] contiguous, q_dt */
  void* q_pe_out;            /* same shape and type; may equal q_pe_in */
  tv_dtype q_dt;
  const void* kpe_tree;      /* device [B, Q, d_rope] un-rotated draft keys, kv_dt */
  const void* ckv_tree;      /* device [B, Q, d_latent] draft latent rows, kv_dt; nullable */
  void* c_kv;                /* cache arrays (kv_dt), rows 16-byte aligned */
  void* k_pe;
  tv_dtype kv_dt;
  int64_t ckv_row_stride, kpe_row_stride; /* elements */
  tv_cache_layout cache;     /* slots outside it (or beyond num_rows when set) are skipped */
  uint64_t* anc;             /* device [B, Q] out */
  int32_t* depth;            /* device [B, Q] out */
  double rope_base;
  int32_t* status;           /* device int32, nullable: TV_ERR_INVALID_TREE for a bad tree
                                (that sequence's rows are left alone) */
} tv_prologue_args;

int tv_verify_prologue(const tv_prologue_args* a, void* stream);

/*
 * tv_build_tree -- best-first draft-tree construction under a node budget.
 *
 * [VERIFY] §"The Context: What Led to This Moment": the engine's GPU best-first tree
 * builder replaces a per-request CPU heapq implementation.  The pages give no formula; the
 * reading taken here: the drafter proposes, for each depth d = 1..L after the root, K
 * candidate tokens with log-probabilities sorted in descending order (one list per depth,
 * shared by every path).  A node is a path of candidate ranks (r_1..r_d) with token
 * cand_tokens[b,d-1,r_d] and score lp[b,0,r_1] + ... + lp[b,d-1,r_d] (float32, added in
 * depth order).  The tree is the root plus the `budget` best nodes taken best first --
 * larger score, then smaller depth, then lexicographically smaller rank path -- numbered
 * in the order taken (node 0 is the root), so parent[i] < i.
 *
 * logprobs    : device [B, L, K] float32, finite, descending over K (a sequence whose
 *               lists are not sorted gets TV_ERR_INVALID_ARG in *status).
 * cand_tokens : device [B, L, K] int32.
 * root_token  : device [B] int32, nullable (node 0's token; -1 when NULL).
 * parent, tokens : device [B, budget+1] int32 out, the tree as tv_build_visibility and
 *               tv_tree_accept take it.  depth [B, budget+1] int32 and score [B, budget+1]
 *               float32 are optional outputs (nullable).
 * Returns TV_ERR_UNSUPPORTED unless L <= 16, K <= 16, budget <= 63 (the verify kernels'
 * q_len <= 64), TV_ERR_INVALID_ARG for a budget above the number of possible nodes.
 */
int tv_build_tree(const float* logprobs, const int32_t* cand_tokens, const int32_t* root_token,
                  int B, int L, int K, int budget, int32_t* parent, int32_t* tokens,
                  int32_t* depth, float* score, int32_t* status, void* stream);

/*
 * tv_tree_accept -- greedy acceptance of a verified draft tree.
 *
 * [RoPE] §"The Broader Context: A Full Native Engine from Scratch" names a greedy
 * tree-accept kernel in the DDTree decode loop, whose greedy output must equal greedy
 * autoregressive decoding token for token; [GOLDEN] §"Context: The Quest for a
 * Hyper-Optimized Inference Stack" lists it among the engine's three custom kernels.  The
 * pages give no formula; the reading taken here:
 *   target[b,i] = argmax_v logits[b,i,v]  (the target model's next token after node i;
 *                 ties go to the smallest token id; logits must be finite),
 *   walk from the root: the next accepted node is the child c of the current node with
 *   tokens[b,c] == target[b,current] (the smallest such c), until there is none; the
 *   bonus token is target[b,last accepted node].
 *
 * logits     : device [B, Q, vocab] (row (b,i) at logits + (b*Q+i)*logits_row_stride
 *              elements), F32 or BF16 (rows at 16-byte boundaries stream fastest).
 * parent     : device [B, Q] int32 draft tree (as for tv_build_visibility).
 * tokens     : device [B, Q] int32 draft token of every node (node 0's entry, the root
 *              token, is not read).
 * target     : device [B, Q] int32 out, nullable: the argmax of every node's logits.
 * accept_len : device [B] int32 out: accepted draft nodes A (0 .. Q-1).
 * path       : device [B, Q] int32 out: 0 (the root), then the accepted nodes in depth
 *              order, then -1.
 * new_tokens : device [B, Q] int32 out: the accepted draft tokens, then the bonus token,
 *              then -1 (A + 1 tokens emitted by the step).
 * status     : see the conventions.  A sequence with an invalid parent array gets A = 0,
 *              path = [0, -1, ...], new_tokens all -1 and TV_ERR_INVALID_TREE.
 * workspace  : device memory of tv_tree_accept_workspace_size(B, Q, vocab) bytes, 256-byte
 *              aligned (the per-chunk argmax keys); scratch, reusable after the call.
 * Returns TV_ERR_UNSUPPORTED for Q > 64, TV_ERR_INVALID_ARG for bad sizes or pointers,
 * TV_ERR_WORKSPACE for a missing, misaligned or short workspace.
 */
size_t tv_tree_accept_workspace_size(int B, int Q, int64_t vocab);
int tv_tree_accept(const void* logits, tv_dtype logits_dt, int64_t vocab,
                   int64_t logits_row_stride, const int32_t* parent, const int32_t* tokens,
                   int B, int Q, int32_t* target, int32_t* accept_len, int32_t* path,
                   int32_t* new_tokens, int32_t* status, void* workspace, size_t ws_bytes,
                   void* stream);

/*
 * tv_compact_kv -- post-verify compaction of the latent KV cache.
 *
 * [RoPE] §"The Broader Context: A Full Native Engine from Scratch": the engine keeps a KV
 * cache with post-verify compaction.  Reading taken here: node i's row sits at logical key
 * prefix_len[b] + i; after acceptance the node at depth d (path[b, d], from tv_tree_accept)
 * moves to logical key prefix_len[b] + d, for d = 1 .. accept_len[b] (the root stays), so
 * that the accepted tokens follow the prefix contiguously.  Both the c_kv row and the k_pe
 * row move; the k_pe row was rotated at position prefix_len + depth, which is its new key
 * index, so it moves unchanged.  new_prefix_len[b] = prefix_len[b] + 1 + accept_len[b].
 *
 * c_kv, k_pe : device cache arrays (rows of d_latent / d_rope elements at the given row
 *              strides, in elements); row sizes, strides and pointers must be multiples of
 *              16 bytes.  Updated in place.
 * cache      : host struct, the cache geometry (page table or contiguous) with num_rows > 0.
 * prefix_len [B], path [B, Q], accept_len [B]: device int32 (path and accept_len as written
 *              by tv_tree_accept).  new_prefix_len [B]: device int32 out (may alias
 *              prefix_len only if the caller does not need the old value).
 * status     : a sequence whose path or keys fall outside the geometry is left unmoved,
 *              keeps new_prefix_len = prefix_len and gets TV_ERR_BOUNDS.
 */
int tv_compact_kv(void* c_kv, void* k_pe, tv_dtype kv_dt, int64_t ckv_row_stride,
                  int64_t kpe_row_stride, int d_latent, int d_rope,
                  const tv_cache_layout* cache, const int32_t* prefix_len, const int32_t* path,
                  const int32_t* accept_len, int B, int Q, int32_t* new_prefix_len,
                  int32_t* status, void* stream);

/*
 * tv_tree_sample -- sampled acceptance of a verified draft tree.
 *
 * The counterpart of tv_tree_accept for a target that is sampled from: every emitted token
 * is distributed as the target's own p = softmax(logits[b,n] / T_b) at its node n, whatever
 * the drafter proposed.  The random numbers are inputs.  From the root, the children of the
 * current node are tested in index order with their own uniform numbers; with unnormalised
 * weights w = p and W = sum w:
 *   draft_probs NULL (candidates chosen without chance, as by tv_build_tree):
 *       child c is accepted iff  uniforms[b,c] * W < w[x_c]; else w[x_c] = 0.
 *   draft_probs given (the children of a node are a draw without replacement from the
 *   drafter's distribution g there, in index order; G = 1 at first):
 *       child c is accepted iff  uniforms[b,c] * g[x_c] * W < w[x_c] * G; else
 *       w = max(w - g * W/G, 0), G = G - g[x_c], g[x_c] = 0; no child is tested any more
 *       once G <= 0, and if no weight is left after a rejection the child is accepted
 *       after all (w and g are then equal but for rounding).  If the target gives that child
 *       no weight at all, the bonus token is drawn from what was left before its rejection
 *       instead.
 * With no child accepted (any more) the walk ends and the bonus token is the smallest v
 * with w[0] + .. + w[v] > uniforms[b,0] * W.  T_b = 0 is greedy: w is 1 at the largest
 * logit (the smallest index among equals) and 0 elsewhere, and draft_probs are not read; the
 * result then equals tv_tree_accept's (on rows that either call takes: see status).  A T_b > 0
 * below 1.5e-30 or above 1.4e30 counts as that.
 *
 * Weights are integers in units of 2^-44 of the row's largest and their sums are exact, so
 * results do not depend on how a row is split.  A weight is off by at most 2^-37 of itself and
 * half a unit.  Results equal those of the rule in 64-bit arithmetic unless a uniform number
 * falls as near to a boundary as these move it.  The sums of a draw move by about 2^-37 of the
 * row's (by 2^-27 if 2^18 half units all went one way), which is a larger share of what
 * rejections have left; a test's sides move by the share that a half unit is of the child's
 * weight; and what rejections leave counts as nothing once it is below half a unit everywhere.
 */
typedef enum { TV_DRAFT_BY_DEPTH = 0, TV_DRAFT_BY_NODE = 1 } tv_draft_mode;

typedef struct {
  uint32_t struct_size;      /* sizeof(tv_sample_args): ABI check */
  int32_t B, Q;              /* sequences, tree nodes (1..64) */
  int64_t vocab;             /* 1 .. 2^18 */
  const void* logits;        /* device [B, Q, vocab], row (b,i) at logits +
                                (b*Q+i)*logits_row_stride elements.  -inf masks a token. */
  tv_dtype logits_dt;        /* F32 or BF16 */
  int64_t logits_row_stride; /* >= vocab */
  const float* temperature;  /* device [B], >= 0; nullable (1 for every sequence) */
  const int32_t* parent;     /* device [B, Q] draft tree */
  const int32_t* tokens;     /* device [B, Q] draft tokens (entry 0 is not read; a token
                                outside [0, vocab) is never accepted and not tested) */
  const float* uniforms;     /* device [B, Q] in [0, 1) (clamped into it; a NaN counts as 0):
                                entry i > 0 tests node i, entry 0 draws the bonus token */
  const float* draft_probs;  /* device [B, draft_rows, vocab] float32, rows that sum to 1;
                                nullable */
  int64_t draft_row_stride;  /* elements between rows, >= vocab (a sequence's rows follow
                                the previous one's) */
  int32_t draft_rows;        /* rows per sequence */
  int32_t draft_mode;        /* tv_draft_mode: the children of node n were drawn from row
                                depth(n) (TV_DRAFT_BY_DEPTH) or n (TV_DRAFT_BY_NODE) */
  int32_t* accept_len;       /* device [B] out, as tv_tree_accept */
  int32_t* path;             /* device [B, Q] out, as tv_tree_accept */
  int32_t* new_tokens;       /* device [B, Q] out, as tv_tree_accept */
  int32_t* status;           /* device int32, nullable.  TV_ERR_INVALID_TREE: invalid parent
                                array (A = 0, path [0, -1, ..], new_tokens all -1).
                                TV_ERR_INVALID_ARG: a negative or NaN temperature (same
                                outputs), or a visited row with a NaN, a +inf or nothing
                                but -inf (the walk ends there without a bonus token: -1).
                                TV_ERR_BOUNDS: depth(n) >= draft_rows at a visited node
                                with children and T_b > 0 (they are not tested). */
} tv_sample_args;

/* Returns TV_ERR_UNSUPPORTED for Q > 64 or vocab > 2^18, TV_ERR_INVALID_ARG for bad sizes,
 * strides, modes or pointers (draft_rows < Q with TV_DRAFT_BY_NODE, and outputs that share
 * memory with inputs or each other, among them). */
int tv_tree_sample(const tv_sample_args* a, void* stream);

/*
 * Pages of a cache: a pool that is kept on the device.
 *
 * Rows are the scheduler's sequence slots.  Row r holds the pages page_table[r, 0 ..
 * n_pages[r]-1]; entries behind them are -1.  refcount[p] counts the table entries that
 * name page p; 0 means free.  The same page numbers serve every layer's c_kv and k_pe
 * arrays.  An empty pool has n_pages = 0, refcount = 0 and page_table = -1.  Calls on one
 * pool that are not ordered by a stream race.  Every per-row argument has one entry for
 * each of the `rows` slots, so that no row can be named twice.
 */
typedef struct {
  int32_t* page_table; /* device [rows, max_pages] */
  int32_t* n_pages;    /* device [rows] */
  int32_t* refcount;   /* device [num_pages] */
  int32_t rows;        /* 1 .. 4096 */
  int32_t max_pages;   /* pages per row at most */
  int32_t num_pages;   /* pages in the pool, < 2^24 */
  int32_t page_size;   /* tokens per page */
} tv_page_pool;

/*
 * tv_pages_reserve -- give rows the pages of the keys they are about to write.
 *
 * Row r, holding length[r] keys, is to hold new_length[r]: it gets pages up to
 * ceil(new_length / page_size), and the pages that keys length .. new_length-1 fall into
 * become its own.  A shared one (refcount > 1) is replaced by a fresh page, unless every
 * holder writes it in this call and r is the lowest of them, which keeps it.  If such a
 * page already holds keys of the row (length % page_size of them), copies[r] says what to
 * copy.  Fresh pages are dealt in order of (row, page index): the i-th takes the i-th
 * lowest free page.  Rows with new_length[r] <= length[r] are left alone.
 *
 * length, new_length : device [rows] int32.
 * copies : device [rows, 3] int32 out: {source page, new page, keys to copy}, or {-1, -1,
 *          0}; the list tv_pages_copy takes (run it for every layer before the keys are
 *          written).
 * status : TV_ERR_NO_PAGES: too few free pages; TV_ERR_BOUNDS: a row needs more than
 *          max_pages, has length > n_pages * page_size or length < 0, or its table names a
 *          page outside the pool.  In both cases nothing is changed (copies: all {-1, -1, 0}).
 * workspace : device memory of tv_pages_workspace_size(pool) bytes, 256-byte aligned.
 */
size_t tv_pages_workspace_size(const tv_page_pool* pool);
int tv_pages_reserve(const tv_page_pool* pool, const int32_t* length, const int32_t* new_length,
                     int32_t* copies, int32_t* status, void* workspace, size_t ws_bytes,
                     void* stream);

/*
 * tv_pages_fork -- rows that share another row's first keys.
 *
 * fork_from : device [rows] int32: the row to fork from, or -1 for rows left alone.
 * length    : device [rows] int32: row r shares the first ceil(length[r] / page_size)
 *             pages of row fork_from[r].  No key is copied; tv_pages_reserve does that for
 *             the one page that is written again.
 * status    : TV_ERR_BOUNDS (that row is left alone): the row holds pages already, its
 *             source is not a row, is itself forked into by this call, or has fewer pages.
 */
int tv_pages_fork(const tv_page_pool* pool, const int32_t* fork_from, const int32_t* length,
                  int32_t* status, void* stream);

/*
 * tv_pages_release -- drop the pages behind a row's first keys.
 *
 * keep   : device [rows] int32: the row keeps its first ceil(keep[r] / page_size) pages (0:
 *          none); a negative entry, or one that covers every page, leaves the row alone.
 *          A page that no row names any more is free.
 * status : TV_ERR_BOUNDS: a dropped entry named no page of the pool, or a free one (the
 *          entry is dropped, no count changes).
 */
int tv_pages_release(const tv_page_pool* pool, const int32_t* keep, int32_t* status, void* stream);

/*
 * tv_pages_compact -- move the pages in use to the front of the pool.
 *
 * With U pages in use, the k-th page in use at U or above (in ascending order) moves to the
 * k-th free page below U; tables and counts are rewritten, and pages U .. num_pages-1 are
 * free afterwards.
 *
 * moves   : device [num_pages, 3] int32 out: {from, to, page_size}, n_moves entries (the
 *           rest is left as it was); the list tv_pages_copy takes.  No page is both a
 *           source and a target.
 * n_moves : device int32 out.
 * status  : TV_ERR_BOUNDS: a table entry below n_pages names no page of the pool (it is left
 *           as it is).
 * workspace : as for tv_pages_reserve.
 */
int tv_pages_compact(const tv_page_pool* pool, int32_t* moves, int32_t* n_moves, int32_t* status,
                     void* workspace, size_t ws_bytes, void* stream);

/*
 * tv_pages_copy -- copy pages of the cache arrays as a list says.
 *
 * Entry {s, d, n} copies rows s*page_size .. s*page_size+n-1 to rows d*page_size .. of
 * c_kv and of k_pe (nullable when d_rope is 0) in each of n_layers layers.  Entries with a negative source
 * or n = 0 are skipped, and so are those whose pages lie outside num_rows rows or whose n
 * exceeds page_size (TV_ERR_BOUNDS).  No page may be both a source and a target, nor a
 * target twice.
 *
 * c_kv, k_pe : rows of d_latent / d_rope elements at the given row strides, layers at the
 *              given layer strides (elements; ignored for one layer).  Row sizes, strides
 *              and pointers are multiples of 16 bytes.
 * list       : device [n_list, 3] int32.  count: device int32, nullable: only the first
 *              *count entries (at most n_list).
 */
int tv_pages_copy(void* c_kv, void* k_pe, tv_dtype kv_dt, int64_t ckv_row_stride,
                  int64_t kpe_row_stride, int d_latent, int d_rope, int n_layers,
                  int64_t ckv_layer_stride, int64_t kpe_layer_stride, int page_size,
                  int64_t num_rows, const int32_t* list, const int32_t* count, int n_list,
                  int32_t* status, void* stream);

/*
 * tv_prefill_attn -- causal latent attention of prompts in its expanded form.
 *
 * With W_uk[h], W_uv[h] the rows 0 .. d_nope-1 and d_nope .. of w_kv[h], key j of a
 * sequence is k_j = W_uk[h] c_kv_j for head h, with the rope part k_pe_j that all heads
 * share, and its value v_j = W_uv[h] c_kv_j.  Query i of sequence b, at logical key
 * prefix_len[b] + i, takes
 *     s_j = scale * ( q_nope[i,h] . k_j + q_pe[i,h] . k_pe_j ),   0 <= j <= prefix_len[b] + i
 *     out[i,h] = sum_j softmax(s)_j v_j.
 * This is the attention that tv_verify_attn with TV_MASK_CAUSAL computes in the latent
 * space (q_latent = q_nope W_uk, and W_uv applied to its output) at 640 instead of 2176
 * flop per (query, key, head), plus 2 * d_latent * (d_nope + d_v) flop per key and head for
 * the expansion; it is the cheaper form from about 170 queries on, tv_verify_attn for
 * fewer (a draft tree, single tokens).
 *
 * The sequences' queries are packed: sequence b has rows q_start[b] .. q_start[b+1]-1 of
 * q_nope, q_pe and out.  Its keys 0 .. prefix_len[b] + q_len - 1 are all in the cache (the
 * prompt's own rows included).  For the tensor cores expanded keys are rounded to bf16,
 * expanded values and the softmax weights to fp16 (so a value's magnitude must stay within
 * 65504: a larger one is clamped and reported; a weight is off by at most 2^-11 of itself or
 * 2^-32 of its row's largest, whichever is more); sums and statistics are 32-bit.  The inputs
 * must be finite.  A score that is NaN makes the rows that see it NaN and no others; an expanded
 * value that is NaN is reported.
 */
typedef struct {
  uint32_t struct_size;      /* sizeof(tv_prefill_args): ABI check */
  int32_t B, H, T;           /* sequences, heads, rows of q_nope, q_pe and out */
  int32_t d_latent;          /* a multiple of 64 */
  int32_t d_nope, d_rope, d_v; /* 128, 64, 128 */
  float scale;               /* > 0 */
  tv_dtype dt;               /* TV_BF16 */
  const void* q_nope;        /* device [T, H, d_nope] contiguous */
  const void* q_pe;          /* device [T, H, d_rope] contiguous, RoPE applied */
  const void* w_kv;          /* device [H, d_nope + d_v, d_latent] contiguous */
  const void* c_kv;          /* cache rows, as tv_attn_args */
  const void* k_pe;          /* cache rows, RoPE applied */
  int64_t ckv_row_stride, kpe_row_stride;
  tv_cache_layout cache;     /* 64-token pages, or contiguous; num_rows > 0, < 2^31 */
  const int32_t* q_start;    /* device [B + 1], ascending, 0 .. T */
  const int32_t* prefix_len; /* device [B] */
  int32_t max_q_len;         /* host bounds: queries of one sequence, */
  int32_t max_kv_len;        /* prefix_len + queries of one sequence, */
  int64_t total_kv;          /* and that summed over the sequences with queries */
  void* out;                 /* device [T, H, d_v] bf16 out, 32-byte aligned.  Rows of no
                                sequence are left as they were. */
  int32_t* status;           /* device int32, nullable.  TV_ERR_BOUNDS: a sequence outside
                                the bounds above, with a negative prefix_len, or whose
                                q_start is negative, above its end or below an earlier one
                                (its rows are left as they were), or a page of
                                it outside the cache (that page reads as zeros), or an expanded
                                value past 65504 or NaN. */
} tv_prefill_args;

/* Bytes of workspace (the expanded keys and values: about 512 * H + 128 bytes per key, and up
 * to 20 MB for small batches); depends on B, H, T and total_kv, and on the device.  0 for invalid arguments. */
size_t tv_prefill_attn_workspace_size(const tv_prefill_args* a);

/* workspace: device memory of at least that size, 256-byte aligned; scratch. */
int tv_prefill_attn(const tv_prefill_args* a, void* workspace, size_t ws_bytes, void* stream);

/*
 * Rotary positions: which elements make a pair, and how its angle depends on the position.
 *
 * Pair k < rot_dim/2 of a rotated part x is (x[k], x[k + rot_dim/2]) with TV_ROPE_HALF (as
 * tv_rope_neox), (x[2k], x[2k+1]) with TV_ROPE_INTERLEAVED.  It turns by pos * f_k, and cos and
 * sin are multiplied by the magnitude.  With e_k = base^(-2k/rot_dim) and c the original
 * context:
 *   TV_ROPE_PLAIN       f_k = e_k
 *   TV_ROPE_LINEAR      f_k = e_k / factor
 *   TV_ROPE_NTK         f_k = base'^(-2k/rot_dim), base' = base * factor^(rot_dim/(rot_dim-2))
 *   TV_ROPE_YARN        f_k = e_k (1 - r_k) + e_k/factor * r_k, r_k rising from 0 to 1 between
 *                       the pairs floor(d(high)) and ceil(d(low)), d(n) = rot_dim
 *                       ln(c / (2 pi n)) / (2 ln base) being the pair that turns n times over
 *                       c positions (the two are kept within 0 .. rot_dim-1, and 0.001 apart)
 *   TV_ROPE_WAVELENGTH  the same with 1 - r_k = (n_k - low) / (high - low), cut off at 0 and 1,
 *                       where n_k = c e_k / (2 pi) is how often pair k turns over c positions
 */
typedef enum { TV_ROPE_HALF = 0, TV_ROPE_INTERLEAVED = 1 } tv_rope_layout;
typedef enum {
  TV_ROPE_PLAIN = 0,
  TV_ROPE_LINEAR = 1,
  TV_ROPE_NTK = 2,
  TV_ROPE_YARN = 3,
  TV_ROPE_WAVELENGTH = 4
} tv_rope_kind;

typedef struct {
  double base;               /* > 1 */
  int32_t kind;              /* tv_rope_kind */
  double factor;             /* >= 1: how far the context is stretched (PLAIN: not read) */
  double original_context;   /* > 0 (YARN, WAVELENGTH) */
  double low, high;          /* turns, 0 < low < high (YARN, WAVELENGTH) */
  double magnitude;          /* factor on cos and sin; 0: 0.1 ln(factor) + 1 for YARN, else 1 */
} tv_rope_scaling;

/* The f_k of rot_dim/2 pairs and the magnitude (host memory), as the calls below take them.
 * TV_ERR_INVALID_ARG for a bad scaling or a rot_dim that is odd, below 2 or above 512. */
int tv_rope_frequencies(const tv_rope_scaling* scaling, int rot_dim, double* frequencies,
                        double* magnitude);

/*
 * tv_rope -- rotate a part of every head at given positions.
 *
 * Head h of token t is x = in + t*in_stride_token + h*in_stride_head, d_head elements of which
 * [rot_offset, rot_offset + rot_dim) are rotated: pair (a, b) at angle t_k becomes
 *     a cos t_k - b sin t_k,   b cos t_k + a sin t_k;
 * the other elements are copied.  `inverse` turns by -t_k (the gradient of the forward turn; or
 * a way back to un-rotated keys, at magnitude 1).  The angle runs in double.  float32 results
 * are within one unit of the last place of the formula in double, and equal tv_rope_neox's where
 * that can express them; bf16 results are rounded once from a value within 2^-20 (|a| + |b|)
 * times the magnitude, so that one in some thousands has another last bit than tv_rope_neox and
 * tv_verify_prologue store, which round the correctly rounded float32 value.
 */
typedef struct {
  uint32_t struct_size;      /* sizeof(tv_rope_args): ABI check */
  int32_t T, n_heads;        /* tokens, heads */
  int32_t d_head;            /* elements of a head, at most 65536 */
  int32_t rot_offset, rot_dim; /* rot_dim even, 2 .. 512 */
  int32_t layout;            /* tv_rope_layout */
  int32_t inverse;           /* 0 or 1 */
  tv_dtype dt;               /* F32 or BF16, of in and out */
  const void* in;
  void* out;                 /* in itself (with the same strides), or memory apart from it: its
                                vectors may lie between in's where the strides are the same, or
                                where a period of one stride holds both side by side */
  int64_t in_stride_token, in_stride_head, out_stride_token, out_stride_head; /* elements */
  const int32_t* positions;  /* device [T] */
  tv_rope_scaling scaling;
} tv_rope_args;

int tv_rope(const tv_rope_args* a, void* stream);

/*
 * tv_norm_rope -- norms of queries and keys, rotation, and the append to the cache, in one pass.
 *
 * The tokens are packed as for tv_prefill_attn: sequence b has tokens q_start[b] ..
 * q_start[b+1]-1, the i-th of them at key prefix_len[b] + i and at position prefix_len[b] + i,
 * or prefix_len[b] + depth[t] for a draft tree.  With N(x; w) = x / sqrt(mean(x^2) + eps) * w,
 * or x where w is NULL, and R the rotation of the first rot_dim elements:
 *     q[t,h] = (q_nope, q_pe):  N(q[t,h]; q_weight), its last d_rope elements through R
 *     kv[t] = (latent, rope):   c_kv row = N(latent; kv_weight),  k_pe row = R N(rope; k_weight)
 * Sums, products and the rotation are 32-bit (the angle in double), rounded once: the sum of a
 * vector's squares, and its mean with eps, have to lie within a float's normal range (elements up
 * to 10^16 do).  A bf16 rotation is tv_rope's, not to the last bit tv_verify_prologue's.  q_nope and
 * q_pe are what tv_prefill_attn takes; with d_nope = 0 only q_pe is written, for queries that
 * were taken into the latent space.
 */
typedef struct {
  uint32_t struct_size;      /* sizeof(tv_norm_rope_args): ABI check */
  int32_t B, T, H;           /* sequences, packed tokens, query heads */
  int32_t d_nope, d_rope, d_latent; /* d_nope >= 0; together at most 65536 */
  int32_t rot_dim;           /* even, 2 .. min(d_rope, 512) */
  int32_t layout;            /* tv_rope_layout */
  tv_dtype dt;               /* F32 or BF16, of every tensor */
  float eps;                 /* >= 0 */
  const void* q;             /* device, [t, h] at q + t*q_stride_token + h*q_stride_head; NULL:
                                no queries (nor their outputs) */
  int64_t q_stride_token, q_stride_head;
  const void* kv;            /* device, [t] at kv + t*kv_stride_token; NULL: no keys (the cache is
                                not read) */
  int64_t kv_stride_token;
  const void* q_weight;      /* device [d_nope + d_rope], nullable */
  const void* kv_weight;     /* device [d_latent], nullable */
  const void* k_weight;      /* device [d_rope], nullable */
  const int32_t* q_start;    /* device [B + 1], ascending */
  const int32_t* prefix_len; /* device [B] */
  const int32_t* depth;      /* device [T], nullable; a negative one leaves its token alone */
  void* q_nope;              /* device [T, H, d_nope] contiguous out */
  void* q_pe;                /* device [T, H, d_rope] contiguous out */
  void* c_kv;                /* cache arrays, rows of d_latent and d_rope elements; they may be */
  void* k_pe;                /* slices of one, whose rows do not meet */
  int64_t ckv_row_stride, kpe_row_stride;
  tv_cache_layout cache;     /* any page size; num_rows > 0 */
  tv_rope_scaling scaling;
  int32_t* status;           /* device int32, nullable.  TV_ERR_BOUNDS: a negative prefix_len
                                (its tokens are left alone), or a key outside the cache (its rows
                                are not written).  Tokens of no sequence are left as they were. */
} tv_norm_rope_args;

int tv_norm_rope(const tv_norm_rope_args* a, void* stream);

/*
 * tv_shared_attn -- attention of sequences that share a long prefix.
 *
 * tv_verify_attn for a batch in which neighbouring sequences hold the same first keys, as rows
 * forked from one prompt do (tv_pages_fork): group g is the sequences group_start[g] ..
 * group_start[g+1]-1, and their keys 0 .. shared_len[g]-1 are the same.  The scores of those keys
 * are taken for the rows of all of a group's sequences together, from the pages of its first
 * one, and joined with every sequence's own keys by their softmax sums, where that takes fewer
 * 128-row tiles.  Every row's result is that of the attention over all of its keys:
 *     s_j = scale * ( q_latent . c_kv_j + q_pe . k_pe_j ),  out = sum_j softmax(s)_j c_kv_j,
 *     lse = ln sum_j exp(s_j)
 * over the prefix keys j < prefix_len[b], shared or not, and of the Q own ones the
 * ancestors-or-self in anc, or with anc NULL the row's token and those before it.  A row that
 * sees no key gets out = 0 and lse = -inf.
 *
 * Softmax weights are rounded to bf16 for the tensor cores (2^-8 of themselves at most), sums and
 * statistics are 32-bit.  The keys 0 .. prefix_len[b]+Q-1 must be finite for rows that do not
 * see them, too; what lies behind them in the cache may be anything.
 */
typedef struct {
  uint32_t struct_size;      /* sizeof(tv_shared_args): ABI check */
  int32_t B, H, Q;           /* sequences, heads, queries of a sequence (1 .. 64) */
  int32_t d_latent, d_rope;  /* 512, 64 */
  float scale;               /* > 0 */
  tv_dtype dt;               /* TV_BF16: queries and cache */
  tv_dtype out_dt;           /* F32 or BF16 */
  const void* q_latent;      /* device [B, Q, H, d_latent] contiguous */
  const void* q_pe;          /* device [B, Q, H, d_rope] contiguous, RoPE applied */
  const void* c_kv;          /* cache rows, as tv_attn_args */
  const void* k_pe;
  int64_t ckv_row_stride, kpe_row_stride;
  tv_cache_layout cache;     /* 64-token pages, or contiguous; num_rows > 0, < 2^31 - 64 */
  const int32_t* prefix_len; /* device [B] */
  int32_t max_prefix_len;    /* host bound on prefix_len */
  int32_t G;                 /* groups, 0 .. B (0: nothing is shared) */
  const int32_t* group_start; /* device [G + 1]: 0 = first, ascending, B = last */
  const int32_t* shared_len; /* device [G], 0 .. the group's smallest prefix_len */
  const uint64_t* anc;       /* device [B, Q] from tv_build_visibility, nullable */
  void* out;                 /* device [B, Q, H, d_latent] out, 32-byte aligned */
  float* lse;                /* device [B, Q, H] out, nullable */
  int32_t* status;           /* device int32, nullable.  TV_ERR_BOUNDS: a sequence whose
                                prefix_len is negative, above the bound or past the cache (its
                                rows get out = 0, lse = -inf); groups that are not as above (they
                                are not shared: every sequence reads its own pages); a page
                                outside the cache (it reads as zeros). */
} tv_shared_args;

/* Bytes of workspace (partial results: 2 KB for each row of the batch, twice, and about 20 MB);
 * depends on B, H, Q, G and the device.  0 for invalid arguments. */
size_t tv_shared_attn_workspace_size(const tv_shared_args* a);

/* workspace: device memory of at least that size, 256-byte aligned; scratch. */
int tv_shared_attn(const tv_shared_args* a, void* workspace, size_t ws_bytes, void* stream);

/*
 * tv_token_sample -- the next token of each row, from given uniform numbers.
 *
 * For a row with temperature T > 0, let w_v = exp((x_v - max x) / T) and order the tokens by
 * falling logit, equal ones by index.  Kept is the longest beginning of that order in which
 * every token passes each filter that is on (the first one always does):
 *     top_k k > 0    it is among the first k;
 *     top_p p < 1    the tokens before it weigh less than p times those that top_k keeps;
 *     min_p m > 0    w_v >= m (an m below 2^-44 counts as that).
 * The token is the smallest kept v whose kept weights up to v sum to more than uniforms[b] times
 * the sum of all of them.  T = 0 is greedy: the largest logit, the smallest index among equals;
 * the filters are not read.  A T > 0 below 1.5e-30 or above 1.4e30 counts as that.
 *
 * Weights are integers in units of 2^-44 of the largest, off by at most 5/8 of a unit and 2^-36 of
 * themselves (2^-46 |max x| / T where that is more), and their sums are exact: results equal those
 * of the rule in 64-bit arithmetic unless a sum or a weight falls as near to a border as these move
 * it, and do not depend on how a row is split.
 */
typedef struct {
  uint32_t struct_size;      /* sizeof(tv_token_args): ABI check */
  int32_t B;                 /* rows */
  int64_t vocab;             /* 1 .. 2^18 */
  const void* logits;        /* device, row b at logits + b*logits_row_stride elements; -inf masks
                                a token: it is never kept */
  tv_dtype logits_dt;        /* F32 or BF16 */
  int64_t logits_row_stride; /* >= vocab */
  const float* temperature;  /* device [B], nullable (1 for every row) */
  const int32_t* top_k;      /* device [B], nullable; <= 0: off */
  const float* top_p;        /* device [B], nullable; >= 1: off; <= 0: only the first token */
  const float* min_p;        /* device [B], nullable; <= 0: off; above 1: as 1 */
  const float* uniforms;     /* device [B] in [0, 1) (clamped into it; a NaN counts as 0) */
  int32_t* tokens;           /* device [B] out */
  int32_t* kept;             /* device [B] out, nullable: how many tokens are kept */
  int32_t* status;           /* device int32, nullable.  TV_ERR_INVALID_ARG: a negative or NaN
                                temperature, a NaN top_p or min_p where the row samples, or a row
                                with a NaN, a +inf or nothing but -inf (token -1, kept 0). */
} tv_token_args;

int tv_token_sample(const tv_token_args* a, void* stream);

/* Text for a tv_status code (static storage). */
const char* tv_status_string(int code);

/* Description of the last failure on this host thread ("" if none). */
const char* tv_last_error(void);

/* Library version as major*10000 + minor*100 + patch. */
int tv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TV_H_ */
