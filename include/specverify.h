/*
 * specverify.h -- C ABI of libspecverify, the GB300 (sm_103a) implementation
 * of the speculative-sampling verification step.
 *
 * The operation (sources cited by page title and section):
 *   [L17] CMU 15-779 Lecture 17 notes, "Speculative Decoding": sec. 2.2
 *         (greedy verification), 2.3 (speculative sampling: accept x ~ q
 *         with probability min(1, p(x)/q(x)), otherwise resample from
 *         norm(max(0, p - q))), 2.4 (Algorithm 1: gamma drafts, one target
 *         pass over gamma+1 positions, stop at the first rejection, bonus
 *         token from p_{gamma+1}), 4.3-4.5 (token trees in depth-first
 *         order, VerifyGreedy, multi-step speculative sampling).
 *   [S14] "Speculative decoding" tutorial (llminference s14): verify(
 *         draft_tokens, q_probs, p_probs, rng) returns the accepted drafts
 *         plus one token; the engine truncates the KV cache by
 *         K - accepted drafts.
 *   [N02] "LLM speculative decoding study notes 02": sec. 3 (r_i ~ U[0,1]),
 *         4 (algorithm), 5.4 (p and q use the same decoding strategy:
 *         temperature, top-k), 10 (greedy), 11.3 (deterministic RNG per
 *         request; drafts of different lengths padded to one K).
 *   [DVP] "Speculative decoding: draft, verify and payoff", II.2 (the
 *         round, KV rollback to the rejected position).
 *
 * Co-residency: the streaming engine's CTAs wait on one another's results
 * (bounded waits), so it is launched cooperatively: every CTA of its grid
 * (one per SM of the device) is resident at once, or the launch fails with
 * SV_ECORESIDENT.  A caller that confines the library to part of the GPU
 * (green contexts, MPS active-thread limits) gets that status rather than
 * timeouts.  The tree walk and the row-statistics kernel wait only inside
 * a thread-block cluster, which the hardware schedules as a unit; the
 * top-k pass waits only within a CTA.
 *
 * Conventions for every entry point:
 *   - All array arguments are DEVICE pointers owned by the caller; the
 *     library allocates nothing and keeps no state between calls except what
 *     lives in the caller's workspace.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).  The returned status covers host-side argument
 *     checks and launch errors only; errors found while the kernel reads the
 *     data are recorded in the workspace and read with sv_get_error().
 *   - A workspace must be zeroed once with sv_workspace_init() before its
 *     first use.  Every call leaves each word it wrote zeroed again (the
 *     role that reads a word last clears it), whatever the sizes, so one
 *     workspace (large enough for each call) serves chain and tree calls of
 *     any shape in sequence; after a device error it must be
 *     re-initialised.  One workspace serves one call at a time: calls that
 *     may overlap on the GPU need separate workspaces.
 *   - Status codes are never negative.
 */
#ifndef SPECVERIFY_H
#define SPECVERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* sv_stream_t; /* identical to cudaStream_t */

typedef enum {
  SV_OK = 0,
  SV_EINVAL = 1,      /* bad argument (null pointer, size out of range ...) */
  SV_ECUDA = 2,       /* a CUDA runtime call failed (launch, memcpy ...) */
  SV_ETIMEOUT = 3,    /* a bounded device wait expired (see sv_get_error) */
  SV_EDATA = 4,       /* the data broke a precondition (see sv_get_error) */
  SV_EWORKSPACE = 5,  /* workspace null, too small or misaligned */
  SV_EUNSUPPORTED = 6, /* no sm_103a device / kernel image for this device */
  SV_ECORESIDENT = 7   /* the grid cannot be resident at once (fewer SMs free
                          than the device has: a green context, MPS limits) */
} sv_status;

/* Logits are SV_BF16 or SV_FP32; the key/value cache calls take SV_FP16 too
   (each call says which). */
typedef enum { SV_BF16 = 0, SV_FP32 = 1, SV_FP16 = 2 } sv_dtype;

typedef enum {
  /* SpecInfer multi-step speculative sampling: child c is tested against
     the draft row q_row[c] as given ([L17] sec. 4.5).  Lossless when the
     children were drawn i.i.d. from their draft rows. */
  SV_TREE_MSS = 0,
  /* MSS for children drawn WITHOUT replacement ([L17] sec. 4.5, the
     precondition of the proof, and sec. 10 exercise 7, the fix): the j-th
     child tried at a node is tested, and the residual formed, against
     q_j = q_row[c] with the tokens of the siblings tried before it removed
     and renormalised; a q_j with no mass left is zero everywhere. */
  SV_TREE_MSS_NOREPLACE = 1,
  /* Naive sampling ([L17] sec. 4.5), the baseline MSS improves on: at the
     current node draw x from p_node by inverse CDF with u_accept[node];
     move to the first child whose token is x, else emit x.  Draft rows are
     not read (draft_logits may be NULL) and u_sample is unused. */
  SV_TREE_NAIVE = 2
} sv_tree_mode;

/* Device error flags, OR-ed into the workspace error word. */
#define SV_DERR_TOKEN 0x01     /* a draft / node token outside [0, V) */
#define SV_DERR_NONFINITE 0x02 /* NaN or +inf in a logit row the step reads */
#define SV_DERR_MASS 0x04      /* a distribution with no mass (all -inf) */
#define SV_DERR_TREE 0x08      /* parent / q_row / depth breaks the format */
#define SV_DERR_TIMEOUT 0x10   /* a bounded wait on a bulk copy expired */
#define SV_DERR_ARG 0x20       /* num_drafts, temperature or top_k invalid */
#define SV_DERR_CHECK 0x40     /* an internal bounds or alignment check failed (debug
                                  builds, -DSV_CHECKS, only): a library bug, never the
                                  data; the access it guarded was skipped */
#define SV_DERR_PAGE 0x80      /* a page id outside [0, num_pages) in a page table entry
                                  that the call needs */

/* Limits of this implementation. */
#define SV_MAX_K 32        /* drafts per chain */
#define SV_MAX_B 1024      /* requests per call */
#define SV_MAX_V (1 << 20) /* vocabulary entries */
#define SV_MAX_TOPK 64     /* top-k filter size */
#define SV_MAX_TREE_NODES 64 /* nodes per tree (N) and draft rows (M) */
#define SV_MAX_TREE_B 1024  /* requests per tree call */
#define SV_MAX_KV_T 65536   /* tokens a request adds to the cache in one call */
#define SV_MAX_KV_HEADS 256 /* key/value heads, and query heads */
#define SV_MAX_ROTATE_D 256 /* channels of a head that sv_rotate takes */
#define SV_MAX_GIVEN 1024   /* tokens asked of one row of logits */

/*
 * Chain verification, one request per b ([L17] sec. 2.4 Algorithm 1).
 *
 * For request b with nd = num_drafts[b] (or K), temperature t = temperature[b]
 * and top-k k = top_k[b] (0 or >= V: no filter):
 *   p_i = softmax(target row i / t) and q_i = softmax(draft row i / t), both
 *   restricted to their own top-k set (k largest, ties to the lower id);
 *   for i = 0..nd-1: accept x_i iff u_i * q_i(x_i) < p_i(x_i); stop at the
 *   first rejection n and emit one token drawn from norm(max(0, p_n - q_n))
 *   by inverse CDF over ascending token id with u_K; if all nd are accepted,
 *   emit the bonus token drawn from p_nd with u_K.
 *   t == 0 (greedy): accept x_i iff x_i == argmax target row i (lowest id on
 *   ties); emit argmax of target row n.  Draft rows and uniforms are unused.
 *
 * Layout: row i of request b starts at element (b*(K+1) + i) *
 * target_row_stride of target_logits (row_stride >= V), likewise draft rows
 * at (b*K + i) * draft_row_stride.  Rows whose byte address and stride are
 * multiples of 16 (bf16: V a multiple of 8) take the bulk-copy path; others
 * a slower direct path.
 *
 * With a top_k array and max_top_k > 0 the call launches two kernels on the
 * stream: a pass that reduces every filtered row to its top-k (logit, id)
 * list and (max, sum of exp) in the workspace, then the verification kernel,
 * which reads no filtered row itself and finalizes filtered requests from
 * those lists.  Otherwise one kernel.
 */
typedef struct {
  int32_t B, K, V;
  sv_dtype dtype;
  const void* target_logits;   /* [B][K+1][row_stride] */
  int64_t target_row_stride;   /* elements between consecutive rows */
  const void* draft_logits;    /* [B][K][row_stride]; may be NULL when every
                                  request is greedy */
  int64_t draft_row_stride;
  const int32_t* draft_tokens; /* [B][K] */
  const int32_t* num_drafts;   /* [B] in [0, K], or NULL (= K) */
  const float* temperature;    /* [B]; 0 = greedy; < 0 or NaN -> SV_DERR_ARG */
  const int32_t* top_k;        /* [B] or NULL; 0 or >= V = no filter; a
                                  filter keeps the top_k largest logits of p
                                  and of q (ties: lower id first) and must be
                                  <= max_top_k (else SV_DERR_ARG) */
  int32_t max_top_k;           /* host-known bound on top_k (0 = none);
                                  sizes the workspace's top-k lists */
  const float* uniforms;       /* [B][K+1] in [0,1): [0..K-1] accept tests,
                                  [K] the residual / bonus draw */
  int32_t* out_tokens;         /* [B][K+1]: accepted drafts then the emitted
                                  token, -1 padded */
  int32_t* out_len;            /* [B] = accept_len + 1 (0 on a data error) */
  int32_t* accept_len;         /* [B] = accepted drafts = KV truncation
                                  index ([S14] "step": n_rejected = K - it) */
  float* p_at_draft;           /* optional [B][K]: p_i(x_i), NaN unused */
  float* q_at_draft;           /* optional [B][K]: q_i(x_i), NaN unused */
} sv_chain_args;

/*
 * Token-tree verification ([L17] sec. 4.4 VerifyGreedy, 4.5 MSS).
 *
 * Request b holds a tree of n = num_nodes[b] nodes in depth-first order:
 * node 0 is the root (the last verified token; its token is ignored) and
 * 0 <= parent[c] < c for c >= 1.  Target row c is the target distribution
 * after the path root..c; draft row q_row[c] is the draft distribution that
 * proposed node c (siblings may share it).  Starting at the root: children
 * of the current node are tried in ascending index order against the
 * residual r (initially p_node): accept c iff u_accept[c] * q(x_c) < r(x_c)
 * and move to c; on rejection r <- norm(max(0, r - q)).  All rejected: emit
 * a draw from r with u_sample; a node without children: emit a draw from
 * p_node.  Greedy (t == 0): move to the first child whose token is argmax
 * p_node, else emit that argmax.
 *
 * Layout: target row c of request b at (b*N + c) * target_row_stride,
 * draft row m at (b*M + m) * draft_row_stride.
 *
 * Each request is walked by one thread-block cluster that reads only the
 * rows on its path (the target rows of the nodes it stands on, the draft
 * rows its children are tested against, and the next step's rows ahead of
 * time); rows too long for the cluster's shared memory (bf16 V above about
 * 160 K) take a slower engine that reduces every row first.
 */
typedef struct {
  int32_t B, N, M, V, max_depth;
  sv_dtype dtype;
  sv_tree_mode mode;
  const void* target_logits;   /* [B][N][row_stride] */
  int64_t target_row_stride;
  const void* draft_logits;    /* [B][M][row_stride] */
  int64_t draft_row_stride;
  const int32_t* node_tokens;  /* [B][N] */
  const int32_t* parent;       /* [B][N] */
  const int32_t* q_row;        /* [B][N] in [0, M) for c >= 1 */
  const int32_t* num_nodes;    /* [B] in [1, N], or NULL (= N) */
  const float* temperature;    /* [B] */
  const int32_t* top_k;        /* [B] or NULL */
  int32_t max_top_k;
  const float* u_accept;       /* [B][N] */
  const float* u_sample;       /* [B] */
  int32_t* out_tokens;         /* [B][max_depth+1], -1 padded */
  int32_t* out_len;            /* [B] */
  int32_t* accept_len;         /* [B] accepted nodes */
  int32_t* accepted_nodes;     /* [B][max_depth]: node ids along the accepted
                                  path (the KV entries to keep), -1 padded */
} sv_tree_args;

/* Workspace bytes a chain / tree call needs (0 on invalid sizes). */
size_t sv_chain_workspace_bytes(int32_t B, int32_t K, int32_t V, sv_dtype dtype,
                                int32_t max_top_k);
size_t sv_tree_workspace_bytes(int32_t B, int32_t N, int32_t M, int32_t V,
                               sv_dtype dtype, int32_t max_top_k);

/* Zero a workspace (cudaMemsetAsync on `stream`). */
sv_status sv_workspace_init(void* workspace, size_t ws_bytes, sv_stream_t stream);

/* The id of the capture that `stream` is part of, 0 outside captures: for
   callers that keep a workspace for each graph (a workspace that a graph
   uses must live as long as the graph, and be no other call's while the
   graph may run). */
sv_status sv_stream_capture_id(sv_stream_t stream, uint64_t* id);

/* Enqueue one chain / tree verification on `stream`.  The workspace must be
   256-byte aligned and at least the size the matching *_workspace_bytes
   call returns. */
sv_status sv_verify_chain(const sv_chain_args* args, void* workspace,
                          size_t ws_bytes, sv_stream_t stream);
sv_status sv_verify_tree(const sv_tree_args* args, void* workspace,
                         size_t ws_bytes, sv_stream_t stream);

/*
 * Tree-attention mask and depth position ids ([L17] sec. 4.3, tree
 * attention: the tree is laid out depth first; a node attends to the
 * verified prefix, its ancestors and itself; a node's position is its
 * depth; sec. 10 exercise 5).  The step that comes before the tree is
 * verified: the target model's forward pass over the tree uses them.
 *
 * Request b holds n = num_nodes[b] nodes (NULL: N) in depth-first order
 * with parent[b][0] == -1 and 0 <= parent[b][i] < i.  Outputs, row i of
 * request b:
 *   mask[(b*N + i)*words + j/32] bit j%32 is set iff node j is node i or
 *   one of its ancestors (j < N; words beyond the second are zero);
 *   depth[b*N + i] = edges from the root (the position offset after the
 *   verified prefix).
 * Rows i >= n are zero with depth -1.  A malformed tree records
 * SV_DERR_TREE (n outside [1, N]: SV_DERR_ARG) and all its rows are zero
 * with depth -1.  Only the workspace's error word is used: any workspace of
 * at least SV_MIN_WORKSPACE_BYTES (zeroed by sv_workspace_init) will do.
 */
#define SV_MIN_WORKSPACE_BYTES 8192u

typedef struct {
  int32_t B, N;               /* B <= SV_MAX_TREE_B, 1 <= N <= SV_MAX_TREE_NODES */
  int32_t words;              /* 32-bit words per mask row, >= (N + 31) / 32 */
  const int32_t* parent;      /* [B][N] */
  const int32_t* num_nodes;   /* [B] in [1, N], or NULL (= N) */
  uint32_t* mask;             /* [B][N][words] */
  int32_t* depth;             /* [B][N] */
} sv_tree_mask_args;

sv_status sv_tree_mask(const sv_tree_mask_args* args, void* workspace, size_t ws_bytes,
                       sv_stream_t stream);

/*
 * Per-position acceptance statistics of a chain round ([L17] sec. 2.3,
 * Thm 3.5: the draft at position i is accepted with probability
 * alpha_i = sum_x min(p_i(x), q_i(x)) = 1 - TV(p_i, q_i); [N02] sec. 7:
 * E[N] = (1 - a^(K+1)) / (1 - a) when every alpha_i = a).  The inputs an
 * adaptive draft length or an on/off switch for speculation would use.
 *
 * Reads the target, draft, num_drafts, temperature, top_k and max_top_k
 * fields of a chain call's arguments (B, K, V, dtype and strides as there;
 * tokens, uniforms and the outputs are not used and may be NULL).  Outputs:
 *   alpha [B][K]: alpha_i for i < num_drafts[b], NaN beyond.  Greedy
 *     requests (t == 0) have one-hot p and q: alpha_i = 1 iff argmax p_i ==
 *     argmax q_i (lowest id on ties), else 0.  With a top-k filter p_i and
 *     q_i are each restricted to their own top-k set ([N02] sec. 5.4), so
 *     alpha_i sums min(p_i, q_i) over the tokens both sets hold.
 *   expected [B]: sum_{j=0..nd} prod_{i<j} alpha_i, the expected number of
 *     tokens the round emits under these rates.
 * With a top_k array and max_top_k > 0 the call first runs the chain's
 * top-k pass (the same lists sv_verify_chain builds) and needs a workspace
 * of sv_chain_workspace_bytes(B, K, V, dtype, max_top_k) bytes; a filter
 * above max_top_k, or any filter when max_top_k is 0, is reported as
 * SV_DERR_ARG, like a bad num_drafts or temperature.  NaN or +inf logits
 * give SV_DERR_NONFINITE, a row without mass SV_DERR_MASS.  The failing
 * request gets NaN.  Without top-k lists the workspace only needs its
 * header and per-request counters (any sv_chain_workspace_bytes size); what
 * the call uses is left zeroed.
 */
sv_status sv_row_stats(const sv_chain_args* args, float* alpha, float* expected,
                       void* workspace, size_t ws_bytes, sv_stream_t stream);

/* ---- Key/value cache in 8 bits (no counterpart on the pages beyond the
 * truncation index: [S14] "step", [DVP] II.2, [L17] sec. 4.3) ----
 *
 * The target model's forward pass over a round reads the keys and values of
 * every earlier token; accept_len and accepted_nodes say which of the
 * round's own tokens stay.  These calls hold that cache, write a round's
 * tokens into it, attend to it, and read tokens back.
 *
 * Layout.  The cache is paged: page p holds page_size tokens of every
 * key/value head, k and v apart, as e4m3 codes (1 sign, 4 exponent, 3
 * mantissa bits; largest value 448, no infinity) in blocks [page_size][D]:
 *   code of token i, channel d, head h of page p:
 *     k[p * page_stride + h * head_stride + i * D + d]
 * and one scale for each page and head, again k and v apart:
 *     value = code * k_scale[p * Hkv + h].
 * A scale is a power of two, 2^e with -48 <= e <= 48: the largest value of
 * a page and head decides e (below), so codes lose no more than e4m3's own
 * rounding, and changing a page's scale moves codes by whole exponents.  A
 * stored scale that is none of these records SV_DERR_ARG in a call that uses
 * it; it counts as the power of two of its exponent bits, clamped.
 * Token position i of request b lives in page page_table[b * slots + i /
 * page_size]; entries a call does not need are not read and may hold
 * anything.  Several requests may name one page as long as no call writes
 * into it.
 */
typedef struct {
  int32_t num_pages, page_size;  /* page_size: 16, 32, 64 or 128 */
  int32_t Hkv, D;                /* D: 64 or 128 */
  void *k, *v;                   /* codes, 16-byte aligned */
  int64_t page_stride;           /* bytes between pages, a multiple of 16 */
  int64_t head_stride;           /* bytes between heads, a multiple of 16, >= page_size * D */
  float *k_scale, *v_scale;      /* [num_pages][Hkv] */
  const int32_t* page_table;     /* [B][slots] */
  int32_t slots;
} sv_kv_cache;

/*
 * Write the keys and values of a round's tokens: token t < n = num_new[b]
 * of request b goes to position kv_len[b] + t.
 *
 * For every page and head that gets tokens, k and v apart:
 *   a = the largest finite |x| of the new tokens in the page,
 *   e = the smallest integer with a <= 448 * 2^e, kept within [-48, 48]
 *       (-48 when a == 0);
 *   if the page holds tokens below kv_len[b], which stay, e is raised to
 *   the page's present e where that is larger; where it is smaller the
 *   codes of the tokens that stay are rounded again at the new scale;
 *   code = x / 2^e to the nearest e4m3 value, ties to even, saturated at
 *   448 (so +-inf becomes +-448 * 2^e); NaN stays NaN.
 * A page without tokens that stay starts anew: tokens of an earlier round
 * that were rejected leave no trace in its scale.  Codes past the last
 * token written are not touched.
 *
 * NaN or inf in the new values records SV_DERR_NONFINITE; kv_len < 0,
 * num_new outside [0, T] or tokens past slots * page_size record
 * SV_DERR_ARG and the request is not written; a page id outside
 * [0, num_pages) records SV_DERR_PAGE and that page is not written.  Only
 * the workspace's error word is used (SV_MIN_WORKSPACE_BYTES).
 */
typedef struct {
  sv_kv_cache cache;
  int32_t B, T;              /* 0 <= B <= SV_MAX_B, 1 <= T <= SV_MAX_KV_T */
  sv_dtype dtype;            /* SV_BF16, SV_FP16 or SV_FP32 */
  const void* k_new;         /* [B][T][Hkv][D], D contiguous */
  const void* v_new;
  int64_t k_batch_stride, k_token_stride, k_head_stride; /* elements */
  int64_t v_batch_stride, v_token_stride, v_head_stride;
  const int32_t* kv_len;     /* [B] tokens the request holds before the call */
  const int32_t* num_new;    /* [B] in [0, T], or NULL (= T) */
} sv_kv_write_args;

sv_status sv_kv_write(const sv_kv_write_args* args, void* workspace, size_t ws_bytes,
                      sv_stream_t stream);

/*
 * Read tokens back: row t < n = num[b] of request b is the value (code *
 * scale, rounded to dtype) at position start[b] + (rows ? rows[b][t] : t);
 * rows t >= n are zero.  With start = kv_len and rows = the accepted nodes
 * of a tree this is the accepted path; written again at kv_len + 1 it
 * becomes contiguous (read and write give back the same codes unless a
 * page's scale drops values below its smallest step).
 *
 * num outside [0, T] records SV_DERR_ARG (all rows zero), a position
 * outside [0, slots * page_size) SV_DERR_ARG and a page id outside
 * [0, num_pages) SV_DERR_PAGE (that row is zero).
 */
typedef struct {
  sv_kv_cache cache;
  int32_t B, T;
  sv_dtype dtype;            /* of k_out and v_out: SV_BF16, SV_FP16 or SV_FP32 */
  void *k_out, *v_out;       /* [B][T][Hkv][D], D contiguous */
  int64_t out_batch_stride, out_token_stride, out_head_stride; /* elements, of both */
  const int32_t* start;      /* [B], or NULL (= 0) */
  const int32_t* num;        /* [B] in [0, T], or NULL (= T) */
  const int32_t* rows;       /* [B][T], or NULL (row t is token t) */
} sv_kv_read_args;

sv_status sv_kv_read(const sv_kv_read_args* args, void* workspace, size_t ws_bytes,
                     sv_stream_t stream);

/*
 * Attention of a round's queries over the cache, after sv_kv_write put the
 * round's own keys and values there.  Query token t < n = num_new[b] of
 * request b, query head j (key/value head j / (Hq / Hkv)):
 *   x_i = scale * sum_d q[d] * key_i[d]         over the positions i it sees,
 *   out = sum_i exp(x_i) value_i / sum_i exp(x_i),
 *   lse = log sum_i exp(x_i).
 * It sees every position i < kv_len[b] and, of the round's own tokens
 * (position kv_len[b] + s, s < n): s <= t when mask is NULL (a chain of
 * drafts, or a chunk of a prompt), else those whose bit s of mask row t is
 * set (sv_tree_mask's rows: a node's ancestors and itself; T <= 64).  A row
 * that sees nothing, and every row t >= n, is 0 with lse = -inf.  What a
 * row does not see does not reach it, NaN and stale codes included.
 * Products and sums are taken in 32 bits.  What enters the products in 16:
 *   - fp16 queries as they are; bf16 queries exactly too, but for channels
 *     below 2^-31 of the row's largest, which are off by up to 2^-39 of it;
 *   - the weights exp(x_i - max) as halves: rounded to 11 bits or, where that
 *     is coarser, off by up to 2^-19 of the largest weight among the 128
 *     positions (a multiple of 128 on) around position i, and by no more than
 *     2^-28 of the row's largest (in blocks more than 2^30 below it the second
 *     may be the only bound).  Weights count with their page's v_scale here.
 *     The sum in the denominator has them unrounded.
 *
 * kv_len < 0, num_new outside [0, T] or a length past slots * page_size
 * records SV_DERR_ARG (all rows of the request as if n were 0); a page id
 * outside [0, num_pages) records SV_DERR_PAGE and no row sees that page.
 * SV_EINVAL also for slots * page_size > 2^30 and for
 * B * Hkv * ceil(T * Hq / Hkv / 16) * ceil(slots * page_size / 64) >= 2^31.
 */
typedef struct {
  sv_kv_cache cache;
  int32_t B, T, Hq;          /* Hq: a multiple of Hkv, <= SV_MAX_KV_HEADS */
  sv_dtype dtype;            /* of q and out: SV_BF16 or SV_FP16 */
  const void* q;             /* [B][T][Hq][D], D contiguous */
  int64_t q_batch_stride, q_token_stride, q_head_stride; /* elements */
  void* out;                 /* [B][T][Hq][D] contiguous; apart from q and the cache */
  float* lse;                /* optional [B][T][Hq] */
  const int32_t* kv_len;     /* [B] tokens before the round */
  const int32_t* num_new;    /* [B] in [0, T], or NULL (= T) */
  const uint32_t* mask;      /* [B][T][words], or NULL (causal) */
  int32_t words;             /* 32-bit words of a mask row, >= (T + 31) / 32 */
  float scale;
} sv_kv_attention_args;

/* Workspace bytes an attention call needs (0 on invalid sizes). */
size_t sv_kv_attention_workspace_bytes(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t D);

sv_status sv_kv_attention(const sv_kv_attention_args* args, void* workspace, size_t ws_bytes,
                          sv_stream_t stream);

/* ---- Norms and positions of queries and keys (no counterpart on the pages:
 * what a target model does between its projections and its attention) ----
 *
 * A head's vector x of D channels becomes
 *   y_i = x_i / sqrt(mean_j x_j^2 + eps) * w_i            (if it has a norm),
 * and pair c (0 <= c < dim / 2) of its first dim channels turns by the
 * angle of the token's position p:
 *   a = 2 pi * frac(p * freq[c] / 2^64),
 *   (u, v) -> scale * (u cos a - v sin a, v cos a + u sin a),
 * where (u, v) are channels (c, c + dim / 2) of y or, interleaved,
 * (2c, 2c + 1).  Channels dim .. D are y's.  Everything is computed in 32 bits
 * (the fraction of the turn exactly, as whole numbers) and rounded once.
 *
 * freq holds turns a position as 64-bit fractions: a frequency of f radians a
 * position is round(f / (2 pi) * 2^64).  However frequencies were stretched for
 * long contexts, they and scale carry it.
 */
typedef struct {
  int32_t dim;             /* channels that turn: a multiple of 16, 0 .. D (0: none) */
  int32_t interleaved;     /* pairs (2c, 2c + 1) instead of (c, c + dim / 2) */
  float scale;             /* factor of the channels that turn, finite (1: none) */
  const uint64_t* freq;    /* [dim / 2], 16-byte aligned; may be NULL when dim is 0 */
} sv_rope;

typedef struct {
  const void* weight;      /* [D], or NULL (ones) */
  sv_dtype weight_dtype;   /* SV_BF16, SV_FP16 or SV_FP32 */
  float eps;               /* 1e-30 or more; 0: no norm (weight must be NULL) */
} sv_head_norm;

/* Heads of one kind, in and out: element (b, t, h, i) at b * batch_stride + t *
   token_stride + h * head_stride + i.  No two elements of out share a place
   (SV_EINVAL for a stride of 0 along more than one), and none one with other
   inputs or results of the call (SV_EINVAL where heads of the first token do). */
typedef struct {
  const void* x;
  void* out;               /* x itself (the same strides and type) or apart from it */
  int32_t heads;           /* 0: none (the other fields are not read) */
  sv_dtype out_dtype;      /* SV_BF16, SV_FP16 or SV_FP32 */
  int64_t batch_stride, token_stride, head_stride; /* of x, in elements */
  int64_t out_batch_stride, out_token_stride, out_head_stride;
  sv_head_norm norm;
} sv_heads;

/*
 * Norm and rotate queries and keys.  Token t < n = num[b] of request b has
 * position start[b] + (offset ? offset[b][t] : t); offsets are, for a token
 * tree, sv_tree_mask's depths.  Rows t >= n of out become zero.
 *
 * num outside [0, T] records SV_DERR_ARG (all rows of the request become
 * zero).  Positions may be any sum of two 32-bit integers.  Only the
 * workspace's error word is used.
 */
typedef struct {
  int32_t B, T, D;           /* 0 <= B <= SV_MAX_B, 1 <= T <= SV_MAX_KV_T; D: a
                                multiple of 16, 16 .. SV_MAX_ROTATE_D */
  sv_dtype dtype;            /* of x: SV_BF16, SV_FP16 or SV_FP32 */
  sv_heads q, k;
  const int32_t* start;      /* [B], or NULL (= 0) */
  const int32_t* num;        /* [B] in [0, T], or NULL (= T) */
  const int32_t* offset;     /* [B][T], or NULL (= t) */
  sv_rope rope;
} sv_rotate_args;

sv_status sv_rotate(const sv_rotate_args* args, void* workspace, size_t ws_bytes,
                    sv_stream_t stream);

/*
 * A round's tokens on their way to sv_kv_attention, in one launch: keys are
 * normed, rotated and, with the values, written into the cache as sv_kv_write
 * would write them (positions, scales, codes, errors: see there; the scales
 * are those of the rotated keys, which are not rounded in between); queries
 * are normed and rotated as by sv_rotate.  A token's position is kv_len[b] +
 * (offset ? offset[b][t] : t); its place in the cache is kv_len[b] + t.
 */
typedef struct {
  sv_kv_cache cache;
  int32_t B, T;              /* 0 <= B <= SV_MAX_B, 1 <= T <= SV_MAX_KV_T */
  sv_dtype dtype;            /* of q, k_new, v_new: SV_BF16, SV_FP16 or SV_FP32 */
  sv_heads q;                /* heads 0: no queries */
  const void* k_new;         /* [B][T][Hkv][D], D contiguous */
  const void* v_new;
  int64_t k_batch_stride, k_token_stride, k_head_stride; /* elements */
  int64_t v_batch_stride, v_token_stride, v_head_stride;
  sv_head_norm k_norm;
  const int32_t* kv_len;     /* [B] tokens the request holds before the call */
  const int32_t* num_new;    /* [B] in [0, T], or NULL (= T) */
  const int32_t* offset;     /* [B][T], or NULL (= t) */
  sv_rope rope;
} sv_kv_append_args;

sv_status sv_kv_append(const sv_kv_append_args* args, void* workspace, size_t ws_bytes,
                       sv_stream_t stream);

/*
 * Log probabilities of given tokens, entropies and likeliest tokens of rows of
 * logits ([N02] sec. 5: temperature softmax), without the probabilities
 * themselves: what a server reports beside the tokens that sv_verify_chain or
 * sv_verify_tree emitted, and what scores a prompt.
 *
 * Output row r < n = num_rows[b] of request b is row i = rows ? rows[b][r] : r
 * of its logits (for a tree: 0, then the accepted nodes).  With x the row, t =
 * temperature[b] (0 and NULL: 1; below 2^-126: 2^-126) and ln p_j = x_j / t -
 * ln sum_k exp(x_k / t):
 *   logprob[b][r][m] = ln p of tokens[b][r][m], -inf where that passes the range of
 *     fp32; NaN where the token is -1;
 *   entropy[b][r]    = - sum_j p_j ln p_j (logits of -inf add nothing);
 *   top_token[b][r][], top_logprob[b][r][]: the `top` largest logits, the lower
 *     token first among equal ones; -1 and -inf where fewer than `top` tokens
 *     have a logit above -inf.
 * Rows r >= n: NaN, and -1 for top_token.  Sums are taken in 32 bits.
 *
 * A row with NaN or +inf records SV_DERR_NONFINITE, one with only -inf
 * SV_DERR_MASS, a row index outside [0, N), num_rows outside [0, R] or a
 * temperature that is negative, infinite or NaN SV_DERR_ARG: these rows (for
 * num_rows and temperature, all of the request) are as rows r >= n.  A token
 * outside [-1, V) records SV_DERR_TOKEN and its logprob is NaN.  Only the
 * workspace's error word is used.
 */
typedef struct {
  int32_t B, N, R, M, V;      /* 0 <= B <= SV_MAX_B; N rows of logits and R of output a
                                 request, 1 .. 65536; 0 <= M <= SV_MAX_GIVEN */
  sv_dtype dtype;             /* SV_BF16 or SV_FP32 */
  const void* logits;         /* [B][N][V], V contiguous */
  int64_t batch_stride, row_stride; /* elements, >= 0 */
  const int32_t* tokens;      /* [B][R][M]; may be NULL when M is 0 */
  const int32_t* num_rows;    /* [B] in [0, R], or NULL (= R) */
  const int32_t* rows;        /* [B][R], or NULL (row r; then R <= N) */
  const float* temperature;   /* [B], or NULL */
  int32_t top;                /* 0 .. SV_MAX_TOPK */
  float* logprob;             /* [B][R][M]; may be NULL when M is 0 */
  float* entropy;             /* [B][R], or NULL */
  int32_t* top_token;         /* [B][R][top]; may be NULL when top is 0 */
  float* top_logprob;         /* [B][R][top]; may be NULL when top is 0 */
} sv_token_logprobs_args;

sv_status sv_token_logprobs(const sv_token_logprobs_args* args, void* workspace, size_t ws_bytes,
                            sv_stream_t stream);

/* Synchronise `stream`, read and clear the workspace error word.
   *device_flags receives the SV_DERR_* bits (may be NULL).  Returns SV_OK,
   SV_EDATA, SV_ETIMEOUT (when the timeout bit is set) or SV_ECUDA. */
sv_status sv_get_error(void* workspace, sv_stream_t stream, int32_t* device_flags);

/* Self-test of the bounded device wait: one CTA waits on an mbarrier that
   nothing arrives at, with a limit of limit_ns nanoseconds, then reports
   through the workspace error word.  Synchronises `stream`.  Returns
   SV_ETIMEOUT when the wait expired as it must. */
sv_status sv_selftest_wait_timeout(void* workspace, size_t ws_bytes,
                                   int64_t limit_ns, sv_stream_t stream);

/* ---- Allocation-free chain entry point (no counterpart on the pages) ----
 *
 * For callers that cannot hand the library a workspace buffer: a host
 * program with no device allocator of its own at the call site, or a call
 * site where allocating device memory is not allowed or could block.  The
 * scratch these calls use is one file-scope device array per device,
 * SV_NOALLOC_SCRATCH_BYTES long, reserved when the library's module loads;
 * the calls themselves allocate nothing.
 *
 *   - Every call looks up the array's address on the current device
 *     (cudaGetSymbolAddress).  The first call in a context (after a device
 *     reset too) zeroes it on `stream` (cudaMemsetAsync), ahead of the
 *     kernel; make that first call before any stream capture that should
 *     contain only the verification.
 *   - A call whose sv_chain_workspace_bytes(...) exceeds
 *     SV_NOALLOC_SCRATCH_BYTES is rejected with SV_EWORKSPACE before any
 *     device work; use sv_verify_chain with a caller workspace instead.
 *   - The counters at the start of the scratch must be zero when a call
 *     starts; every call leaves them zero.  sv_noalloc_get_error re-zeroes
 *     the scratch (on `stream`) after reporting a device error.
 *   - All calls on one device share the one scratch: calls that may overlap
 *     on the GPU (e.g. on different streams without ordering) race and give
 *     undefined results.  Order them, or use sv_verify_chain with separate
 *     workspaces.
 * Arguments, layouts and results are those of sv_verify_chain. */
#define SV_NOALLOC_SCRATCH_BYTES (8u << 20) /* 8 MiB per device */

sv_status sv_verify_chain_noalloc(const sv_chain_args* args, sv_stream_t stream);

/* sv_get_error for the allocation-free scratch of the current device; after
   a device error it also re-zeroes the scratch on `stream`. */
sv_status sv_noalloc_get_error(sv_stream_t stream, int32_t* device_flags);

const char* sv_status_string(sv_status status);

/* Library version, major*10000 + minor*100 + patch. */
int32_t sv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_H */
