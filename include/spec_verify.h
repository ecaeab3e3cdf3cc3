/*
 * spec_verify.h -- C ABI of the MI355X (gfx950) library for the verification
 * step of speculative decoding.
 *
 * The method (p = target, q = draft):
 *   - "投机解码与 EAGLE", section 二 (exactness rule; temperature-0 greedy rule);
 *   - "064 · 投机解码：小模型先起草，大模型怎样并行验收而不改变分布",
 *     section 二 (acceptance a(x) = min(1, p(x)/q(x)); residual
 *     r(x) = max(0, p(x) - q(x)) / sum max(0, p - q); p and q must carry the
 *     temperature / top-k transforms; acceptance rate alpha = sum min(p, q)),
 *     section 三 (the per-position loop: test, stop at the first rejection
 *     and draw from the residual, or draw a bonus token from p_{K+1});
 *   - "EAGLE-2: Faster Inference of Language Models with Dynamic Draft
 *     Trees", section 2.1 (same rule), section 2.2 (tree drafts verified in one
 *     pass; the longest accepted branch wins).
 *
 * Conventions shared by every entry point
 *   - All array arguments except `parents_host` are DEVICE pointers, row-major
 *     and contiguous.  Every buffer is owned by the caller; the library
 *     allocates nothing and keeps no pointer after returning.  Calls on
 *     different streams may run concurrently as long as they use different
 *     workspaces.  The library's own state is: a process-wide atomic counter
 *     that gives every top-k chain call its tag (see the hand-over below),
 *     the per-thread request of spec_profile_events, and the device scratch
 *     of spec_verify_chain_noalloc (one array per GPU, looked up on first use).
 *   - Work is enqueued on `hip_stream` (a hipStream_t; NULL = the null stream)
 *     and the call returns without synchronising.  Inputs must stay valid and
 *     outputs must not be read until the stream has reached the call.
 *   - `workspace` is device scratch of at least the size reported by the
 *     matching *_workspace_bytes function (or spec_workspace_bytes, which
 *     covers every call of a shape), 256-byte aligned.  It must be
 *     zero-filled before its first use (spec_workspace_init, or any zeroing
 *     allocation).  A top-k chain call (temperature > 0, 0 < top_k < V)
 *     needs the part it uses to be zero and leaves it zero (the hand-over
 *     words one call writes are cleared by the same call), so a series of
 *     such calls needs zeroing once.  Every other call leaves scratch data
 *     behind: before a top-k chain call that follows a call of another kind
 *     on the same workspace, zero it again.  A workspace serves one call at a
 *     time: calls that may overlap need separate workspaces.
 *   - Hand-over inside a top-k chain launch: the finisher workgroups of a
 *     batch row wait, with a bounded poll, for the words the selection
 *     workgroups of the same launch store.  Finishers come after every
 *     selection workgroup in the grid, and the GPU dispatches a launch's
 *     workgroups in grid order within each XCD, so a finisher only waits for
 *     workgroups that are running or done; progress relies on that order.
 *     If words still have not arrived after about 0.1 s (another process
 *     holding the GPU's compute units), the row gets accept_len =
 *     SPEC_ROW_TIMED_OUT and -1 tokens, and the launch still ends.  Words
 *     carry the call's tag, so a word a late workgroup stores after its
 *     call gave up is ignored by later calls.  A graph replay reuses the tag
 *     of the captured call: after a replay that reports a timed-out row, zero
 *     the workspace before the next replay.
 *   - Logit rows are bfloat16 (SPEC_BF16, raw bits) or float32 (SPEC_F32).
 *     Draft probabilities are float32.  Uniforms are float32 in [0, 1).
 *   - Host-detectable argument errors return a negative code and launch
 *     nothing.  Bad DATA never aborts a call: the affected batch row gets
 *     accept_len = -1 and all its output tokens (and path entries) = -1,
 *     under these rules:
 *       E1 a target row that is consulted contains NaN, or (sampling mode)
 *          +inf, or only -inf values;
 *       E2 a draft / node token outside [0, V) (every token is checked);
 *       E3 a draft probability that is consulted is NaN, negative or +inf;
 *       E4 a transformed draft row that is consulted keeps zero mass;
 *       E5 a uniform outside [0, 1) (sampling mode; every uniform is checked).
 *     A chain consults position k only when x_0..x_{k-1} were all accepted
 *     (the left-to-right walk of the method): target rows 0..j, and for the
 *     draft, q[x_k] for k <= j (T == 1, no top-k) or whole rows 0..j (any
 *     other transform), plus row j itself for a residual draw; j = first
 *     rejection (K if none).  A greedy tree consults every node row; a
 *     sampled tree the rows of the nodes its walk visits.
 *   - Environment: SPEC_VERIFY_DENSE_BRACKET (a number in [0, 0.5)) sets the
 *     relative width of the bracket the dense final draw (temperature > 0,
 *     top-k off) puts around the normalisers taken from its row statistics.
 *     Results do not depend on it; a normaliser outside its bracket only makes
 *     the draw recompute that row exactly (0 forces that path, for tests).
 *     Read on every call; unset or invalid values leave the built-in width.
 *     SPEC_VERIFY_TREE_ONEPASS = 0 makes spec_verify_tree_sample compute the
 *     residual masses of the node it draws at with one pass each, instead of
 *     one pass for all of them (the same results; for tests).
 *     SPEC_VERIFY_DENSE_PATH = walk | rows picks the route of a chain with
 *     temperature 1 and top-k off: the walk (one workgroup per batch row reads
 *     target rows only up to the first rejection) or every row's statistics
 *     first; by default the walk when B*(K+1) > 1344 or V < 4096.  Results
 *     are the same either way.
 *     SPEC_VERIFY_DENSE_SPLIT sets how many workgroups share each batch row's
 *     draw on the every-row-first route (temperature > 0, top-k off): 0 keeps
 *     one per row, N >= 2 asks for N (at most 16 and the row's 4096-token
 *     chunks) at any batch size; unset, the library splits batches of up to
 *     192 rows (160 with a transformed draft).  Results are the same.
 *     SPEC_VERIFY_SPIN_LIMIT (an integer in [0, 65536]) lowers the number of
 *     polls a top-k chain finisher, or a member of a sampled tree's cluster
 *     (spec_verify_tree_sample_ws), makes before it gives up (tests of the
 *     timed-out path); read on every call.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of logit rows.  A plain integer, so that a value outside the two
 * below is an argument error the library reports (SPEC_EINVAL), not an
 * out-of-range enumeration. */
typedef int32_t spec_dtype_t;
enum { SPEC_F32 = 0, SPEC_BF16 = 1 };

enum {
    SPEC_OK = 0,
    SPEC_EINVAL = -1,        /* bad sizes, pointers, dtype, temperature, parents */
    SPEC_EWORKSPACE = -2,    /* workspace missing, misaligned or too small */
    SPEC_ELAUNCH = -3,       /* a kernel launch failed (hipGetLastError) */
    SPEC_EUNSUPPORTED = -4,  /* valid request outside this build's limits */
    SPEC_ESCRATCH = -5       /* spec_verify_chain_noalloc: more scratch needed than it holds */
};

/* accept_len of a batch row whose top-k chain hand-over timed out (see above). */
#define SPEC_ROW_TIMED_OUT (-2)

/* Limits of this build: K <= SPEC_MAX_K draft positions, N <= SPEC_MAX_NODES
 * tree nodes, top_k <= SPEC_TOPK_MAX when top-k is active, V < 2^24 and V <=
 * SPEC_MAX_V. */
#define SPEC_MAX_K 63
#define SPEC_MAX_NODES 64
#define SPEC_TOPK_MAX 64
#define SPEC_MAX_V (1 << 20)
#define SPEC_EXPAND_MAX 1024     /* children of one expansion layer, E * top_k */
#define SPEC_RERANK_MAX 1024     /* candidate nodes of one reranking */

/* Human-readable text for a return code (static storage). */
const char* spec_error_string(int code);

/* One workspace size (bytes) that serves every spec_verify_chain,
 * spec_verify_chain_topp and spec_accept_rate call with B batch rows and K =
 * K_or_N draft positions, and every spec_verify_tree_greedy(_rows) call with
 * N = K_or_N tree nodes, over V tokens with this top_k, whatever the dtype and
 * temperature; 0 if no such call is valid (B, K_or_N or V below 1, V above
 * SPEC_MAX_V).  It is the largest of the per-call sizes below. */
size_t spec_workspace_bytes(int B, int K_or_N, int V, int top_k);

/* Workspace sizes (bytes) for the calls below with the same arguments; 0 if the
 * arguments are invalid.  Sizes depend only on the arguments. */
size_t spec_chain_workspace_bytes(int B, int K, int V, spec_dtype_t dtype, float temperature, int top_k);
size_t spec_tree_workspace_bytes(int B, int N, int V, spec_dtype_t dtype);
size_t spec_accept_rate_workspace_bytes(int B, int K, int V, spec_dtype_t dtype, float temperature, int top_k);
size_t spec_tree_expand_workspace_bytes(int B, int E, int V, int top_k);

/*
 * spec_verify_chain -- batched verification of B drafted chains of K tokens.
 * "064 · 投机解码", section 二 (the test min(1, p/q), the residual
 * norm(max(0, p - q)), p and q carrying the temperature and top-k) and section
 * 三 (the left-to-right loop, the residual draw at the first rejection, the
 * bonus draw from p_{K+1}); "投机解码与 EAGLE", section 二 (greedy mode);
 * "Việc giải mã giả định và EAGLE-3", step 2 of the residual routine (zero
 * residual mass: draw from the target).
 *
 * For each batch row b (independently):
 *   p'_k = softmax(z_k / T) over the top_k largest logits of row k (all V when
 *          top-k is off), zero elsewhere; k = 0..K.
 *   q'_k = q_k as given when T == 1 and top-k is off; otherwise q_k^(1/T)
 *          renormalised over the top_k largest entries of q_k.
 *   Test k = 0, 1, ...: accept x_k iff u_k < min(1, p'_k(x_k) / q'_k(x_k))
 *   (q'_k(x_k) = 0: accept iff p'_k(x_k) > 0); stop at the first rejection j.
 *   Final draw with u_K: at j < K from r = max(0, p'_j - q'_j) (if r has zero
 *   mass, from p'_j), at j = K from p'_K; the token is the smallest index i
 *   with u_K * S < C_i (C the inclusive prefix sum of r in index order, S its
 *   total).
 *   Top-k sets are exact: k entries, larger value first, lower index on ties.
 * Greedy mode (temperature == 0): accept while x_k equals the argmax of row k
 * (lowest index on ties), then emit the argmax of the first mismatching row
 * (or of row K); draft_probs and uniforms are not read (may be NULL).
 *
 *   target_logits [B][K+1][V]  dtype                   device, read
 *   draft_probs   [B][K][V]    float32                 device, read (rows sum to ~1)
 *   draft_tokens  [B][K]       int32                   device, read
 *   uniforms      [B][K+1]     float32 in [0,1)        device, read
 *   temperature   >= 0, finite (0 = greedy); top_k <= 0 or >= V disables top-k
 *   out_tokens    [B][K+1]     int32                   device, written: x_0..x_{j-1}, y, then -1
 *   out_accept_len[B]          int32                   device, written: j in [0,K], -1 on error,
 *                                                      SPEC_ROW_TIMED_OUT (top-k mode only, see above)
 *   out_diag      [B][2K+2]    float32, may be NULL    device, written:
 *                 [k] = p'_k(x_k), [K+k] = q'_k(x_k) for the tested
 *                 positions k <= j, k < K (NaN for k > j; greedy: [k] = 1 if
 *                 x_k matched, else 0, and [K+k] = NaN),
 *                 [2K] = mass of the final-draw distribution before
 *                 normalisation (residual mass, or 1 for p'), [2K+1] = the
 *                 drawn token's probability under it.
 * Returns SPEC_OK or a negative code.
 */
int spec_verify_chain(const void* target_logits, spec_dtype_t dtype,
                      const float* draft_probs, const int32_t* draft_tokens,
                      const float* uniforms, int B, int K, int V,
                      float temperature, int top_k,
                      int32_t* out_tokens, int32_t* out_accept_len, float* out_diag,
                      void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * spec_verify_chain_topp -- spec_verify_chain with a nucleus (top-p) transform
 * on both distributions ("064 · 投机解码", section 二: the sampling transforms
 * are part of p and q).  After the temperature and top-k, each row keeps the
 * shortest prefix of its kept tokens, in value order (lower index first on
 * ties), whose probability mass reaches top_p, renormalised; a token of zero
 * probability is never kept.  0 < top_p <= 1 (1: spec_verify_chain); top_p < 1
 * needs temperature > 0 (SPEC_EUNSUPPORTED otherwise).  With top-k on, the cut
 * runs over the kept top-k entries; with top-k off, over whole rows (every
 * target and draft row's cut is found first, by a radix select on the values
 * with the masses summed exactly in fixed point, then the tests and the
 * residual draw run in fp64).  The cut is decided on fp64 probabilities.
 * Everything else, workspace included, is as for spec_verify_chain.
 */
int spec_verify_chain_topp(const void* target_logits, spec_dtype_t dtype, const float* draft_probs,
                           const int32_t* draft_tokens, const float* uniforms, int B, int K, int V,
                           float temperature, int top_k, float top_p, int32_t* out_tokens,
                           int32_t* out_accept_len, float* out_diag, void* workspace, size_t workspace_bytes,
                           void* hip_stream);

/*
 * spec_verify_chain_noalloc -- spec_verify_chain for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  Same arguments, results and kernels, no
 * workspace: the call uses a device array of SPEC_NOALLOC_SCRATCH_BYTES that
 * the library holds on each GPU it runs on until the process ends, and calls
 * no hipMalloc, hipFree or other allocating routine.  A call whose workspace
 * (spec_chain_workspace_bytes) would exceed that size returns SPEC_ESCRATCH
 * and launches nothing.  The first call on a device looks the array up (with
 * that device current); the array is zero-filled by a fill kernel on the
 * call's stream before a top-k call whenever another kind of call used it
 * since; that decision is taken when a call is issued, so a graph that
 * captured a top-k call replays without it: between its replays, run no call
 * that leaves scratch behind.  Every call on a GPU shares that GPU's array: calls that may overlap
 * (different streams, or several host threads, without ordering between them)
 * race and give undefined results; order them on one stream.
 */
#define SPEC_NOALLOC_SCRATCH_BYTES (32u << 20)
int spec_verify_chain_noalloc(const void* target_logits, spec_dtype_t dtype, const float* draft_probs,
                              const int32_t* draft_tokens, const float* uniforms, int B, int K, int V,
                              float temperature, int top_k, int32_t* out_tokens, int32_t* out_accept_len,
                              float* out_diag, void* hip_stream);

/*
 * spec_verify_chain_fused -- spec_verify_chain with the target's LM head in
 * front of it, so that the logits never reach memory ("064 · 投机解码", section
 * 三: one target pass yields the K+1 distributions the verification consumes;
 * "Việc giải mã giả định và EAGLE-3": decoding is bound by memory bandwidth).
 * The logits are z[b][k][v] = sum_h hidden[b][k][h] * head_weight[v][h]
 * (bfloat16 operands, fp32 accumulation on the matrix cores); the verification
 * is then exactly spec_verify_chain's on those logits, for the two modes whose
 * selection runs in the GEMM's epilogue: greedy (temperature == 0) and top-k
 * (temperature > 0, 0 < top_k < V, top_k <= SPEC_TOPK_MAX).  Without top-k the
 * residual draw needs whole logit rows: SPEC_EUNSUPPORTED.
 *
 *   hidden        [B][K+1][H]  bfloat16 (raw bits)     device, read; 16-byte aligned
 *   head_weight   [V][H]       bfloat16 (raw bits)     device, read; 16-byte aligned (no bias)
 *   H             hidden size, a multiple of 64 (V*H and B*(K+1)*H below 2^31)
 *   draft_probs, draft_tokens, uniforms, temperature, top_k, out_tokens,
 *   out_accept_len, out_diag: as for spec_verify_chain (the logit rows are the
 *   fp32 logits above; a NaN logit makes its row unusable, E1).
 *   workspace     spec_chain_fused_workspace_bytes(B, K, V, H, temperature, top_k)
 *                 bytes, 256-byte aligned, zero-filled before its first use; a
 *                 top-k call leaves its hand-over words zero, as a top-k chain does,
 *                 and a greedy call leaves scratch behind (zero the workspace before
 *                 a top-k call that follows one on it).
 * Precision: the verification is exact on the fp32 logits the matrix cores
 * produce; they differ from exact logits by the rounding of fp32 accumulation
 * over H/16 steps (a few 1e-6 at |z| ~ 20, H = 4096).
 */
size_t spec_chain_fused_workspace_bytes(int B, int K, int V, int H, float temperature, int top_k);
int spec_verify_chain_fused(const void* hidden, const void* head_weight, const float* draft_probs,
                            const int32_t* draft_tokens, const float* uniforms, int B, int K, int V, int H,
                            float temperature, int top_k, int32_t* out_tokens, int32_t* out_accept_len,
                            float* out_diag, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * spec_verify_tree_greedy -- greedy verification of a static draft tree.
 * "EAGLE-2: Faster Inference of Language Models with Dynamic Draft Trees",
 * section 2.2 (every branch of the draft tree verified in one target pass, the
 * longest accepted branch kept); "投机解码与 EAGLE", section 二 (temperature 0:
 * a draft token is accepted when it is the target's argmax) and its EAGLE part
 * (tree drafts).
 *
 * Node 0 is the root; parents_host[0] = -1 and 0 <= parents_host[n] < n
 * (nodes in topological, e.g. breadth-first, order).  Row n of the logits is
 * the target's next-token distribution after the path to node n.  Node n > 0 is
 * accepted iff its parent is accepted and node_tokens[b][n] equals the argmax
 * of the parent's row (lowest index on ties).  The result is the deepest
 * accepted node n* (lowest node index on ties), its root-to-n* path and the
 * bonus token argmax(row n*).  D = the tree's maximum depth.
 *
 *   target_logits [B][N][V]    dtype                   device, read
 *   node_tokens   [B][N]       int32                   device, read ([b][0] ignored)
 *   parents_host  [N]          int32                   HOST, read during the call only
 *   out_path      [B][D+1]     int32                   device, written: node ids root..n*, then -1
 *   out_tokens    [B][D+1]     int32                   device, written: accepted tokens, bonus, then -1
 *   out_accept_len[B]          int32                   device, written: depth of n*, -1 on error
 */
int spec_verify_tree_greedy(const void* target_logits, spec_dtype_t dtype,
                            const int32_t* node_tokens, const int32_t* parents_host,
                            int B, int N, int V,
                            int32_t* out_path, int32_t* out_tokens, int32_t* out_accept_len,
                            void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * spec_verify_tree_sample -- sampling verification of a static draft tree
 * ("投机解码与 EAGLE", the EAGLE part: a rejected branch makes the verifier try
 * the others; "064 · 投机解码", section 三, and "EAGLE-2: Faster Inference of
 * Language Models with Dynamic Draft Trees", section 2.1, for the single test
 * and the residual).
 *
 * Tree layout as in spec_verify_tree_greedy.  Row n of the logits is the
 * target's distribution after the path to node n; row n of draft_probs is the
 * draft model's distribution at node n, from which node n's children were
 * drawn (independently of one another; rows of leaves are not read).
 * p'_n and q'_n carry the temperature as in spec_verify_chain (T == 1: q as
 * given).  For each batch row, from the root c = 0 with P = p'_c and Q = q'_c:
 * the children of c are tried in increasing node order; child n is accepted
 * iff u[n] < min(1, P(x_n)/Q(x_n)) (Q = 0 accepts iff P > 0), which emits x_n
 * and moves to n; a rejection replaces P by max(0, P - Q)/S, S its mass (P is
 * kept when S = 0), and the next child is tried.  When no child is accepted,
 * or c is a leaf, a token is drawn from P with u[0] (index-ascending inverse
 * CDF: the first y with u[0]*sum P < prefix_y, as in spec_verify_chain).
 * This reading (the pages give no rule for several branches) keeps the
 * emitted tokens distributed as the target's when children are independent
 * draws from q'.  Computed in fp64.  The walk consults the target rows of the
 * nodes it visits and, for a visited node with children, its draft row:
 * q[x_n] of the tested children (T == 1), the whole row when T != 1 or once a
 * residual is formed (E1, E3, E4); E2 and E5 cover every token and uniform.
 *
 *   target_logits [B][N][V]    dtype                   device, read
 *   draft_probs   [B][N][V]    float32                 device, read
 *   node_tokens   [B][N]       int32                   device, read ([b][0] ignored)
 *   uniforms      [B][N]       float32                 device, read (u[n]: node n's test; u[0]: the draw)
 *   parents_host  [N]          int32                   HOST, read during the call only
 *   temperature   > 0 (greedy trees: spec_verify_tree_greedy); top_k must be
 *                 off (<= 0 or >= V) in this build, else SPEC_EUNSUPPORTED
 *   out_path      [B][D+1]     int32                   device, written: node ids root..last accepted, then -1
 *   out_tokens    [B][D+1]     int32                   device, written: accepted tokens, the drawn one, then -1
 *   out_accept_len[B]          int32                   device, written: depth reached, -1 on error
 * Needs no workspace.
 */
int spec_verify_tree_sample(const void* target_logits, spec_dtype_t dtype, const float* draft_probs,
                            const int32_t* node_tokens, const float* uniforms, const int32_t* parents_host,
                            int B, int N, int V, float temperature, int top_k,
                            int32_t* out_path, int32_t* out_tokens, int32_t* out_accept_len,
                            void* hip_stream);

/*
 * Per-row trees (a dynamic draft tree differs from one batch row to the next,
 * e.g. the output of spec_tree_rerank with the root at position 0):
 * spec_verify_tree_greedy_rows and spec_verify_tree_sample_rows are the two
 * calls above with `parents` a DEVICE array [B][N] (row b: parents[b][0] = -1,
 * 0 <= parents[b][n] < n; a row that breaks this is an error row, accept_len
 * -1) instead of parents_host, and out_path / out_tokens of N entries per batch
 * row ([B][N], -1 padded).  Everything else is as above; the greedy call takes
 * the workspace of spec_tree_workspace_bytes(B, N, V, dtype).
 */
int spec_verify_tree_greedy_rows(const void* target_logits, spec_dtype_t dtype, const int32_t* node_tokens,
                                 const int32_t* parents, int B, int N, int V, int32_t* out_path,
                                 int32_t* out_tokens, int32_t* out_accept_len, void* workspace,
                                 size_t workspace_bytes, void* hip_stream);
int spec_verify_tree_sample_rows(const void* target_logits, spec_dtype_t dtype, const float* draft_probs,
                                 const int32_t* node_tokens, const float* uniforms, const int32_t* parents,
                                 int B, int N, int V, float temperature, int top_k, int32_t* out_path,
                                 int32_t* out_tokens, int32_t* out_accept_len, void* hip_stream);

/*
 * spec_verify_tree_sample_ws, spec_verify_tree_sample_rows_ws -- the two
 * sampled-tree calls above (same method, pages and arguments), given a
 * workspace of spec_tree_sample_workspace_bytes(B, N) bytes (256-byte
 * aligned; SPEC_EWORKSPACE if smaller).  With it, a batch of B <= 128 rows
 * shares each row's walk among min(8, 256/B) workgroups, each summing a slice
 * of the vocabulary, which exchange their sums through the workspace; this
 * needs V a multiple of 8, 16-byte aligned rows and V <= 8192 * min(8, 256/B)
 * (4096 * min(8, 256/B) when temperature != 1), else (and for B > 128, where
 * the size is 0) the call runs as without one.
 * Same results as the calls above, up to the rounding order of the sums.
 *
 * The workspace must be zero-filled before its first use; every call leaves
 * it zero, so it can be reused, including by replays of a captured graph.
 * Calls that overlap on one workspace race.  The members of a batch row wait
 * for one another's words.  A row's members are consecutive workgroups, so they
 * sit on different XCDs, and each XCD dispatches its workgroups in grid order:
 * on every XCD the rows already dispatched form a prefix, and every row below
 * the shortest prefix has all its members running and finishes, so progress
 * relies on that order, as the top-k chain's hand-over does.  A wait that
 * exceeds the spin limit (SPEC_VERIFY_SPIN_LIMIT, above) gives up: that batch
 * row's accept_len is SPEC_ROW_TIMED_OUT and its outputs -1.
 */
size_t spec_tree_sample_workspace_bytes(int B, int N);
int spec_verify_tree_sample_ws(const void* target_logits, spec_dtype_t dtype, const float* draft_probs,
                               const int32_t* node_tokens, const float* uniforms, const int32_t* parents_host,
                               int B, int N, int V, float temperature, int top_k, int32_t* out_path,
                               int32_t* out_tokens, int32_t* out_accept_len, void* workspace, size_t workspace_bytes,
                               void* hip_stream);
int spec_verify_tree_sample_rows_ws(const void* target_logits, spec_dtype_t dtype, const float* draft_probs,
                                    const int32_t* node_tokens, const float* uniforms, const int32_t* parents, int B,
                                    int N, int V, float temperature, int top_k, int32_t* out_path,
                                    int32_t* out_tokens, int32_t* out_accept_len, void* workspace,
                                    size_t workspace_bytes, void* hip_stream);

/*
 * EAGLE-2 draft-tree construction ("EAGLE-2: Faster Inference of Language
 * Models with Dynamic Draft Trees", section 4).  A node's value is the product
 * of the draft model's confidences along its path (section 4.1).  Values and
 * their products are float32, and every ordering is decided on those float32
 * numbers, the lower index first among equal keys.
 *
 * spec_tree_expand -- one expansion layer (section 4.1).  For each batch row,
 * each of the E nodes being expanded gets its draft row's top_k most probable
 * tokens as children (larger probability first, lower token index on ties);
 * a child's value is the node's value times the token's probability (one
 * float32 multiply); out_next lists the k_next children of highest value (flat
 * index e*top_k + i), the lower flat index first among equal values -- the
 * nodes to expand next.
 *
 *   draft_probs      [B][E][V]        float32   device, read: the draft distribution at each expanded node
 *   node_values      [B][E]           float32   device, read: the expanded nodes' values
 *   out_child_tokens [B][E][top_k]    int32     device, written
 *   out_child_values [B][E][top_k]    float32   device, written
 *   out_next         [B][k_next]      int32     device, written
 *   1 <= top_k <= min(V, SPEC_TOPK_MAX), 1 <= k_next <= E*top_k <= SPEC_EXPAND_MAX.
 *   workspace: spec_tree_expand_workspace_bytes(B, E, V, top_k) bytes (leaves
 *   scratch behind, like the other non-top-k-chain calls).
 * A batch row whose draft rows hold a NaN, negative or +inf probability, or
 * whose node value is not a finite non-negative number, gets -1 tokens and
 * next indices and NaN values.
 */
int spec_tree_expand(const float* draft_probs, const float* node_values, int B, int E, int V, int top_k,
                     int k_next, int32_t* out_child_tokens, float* out_child_values, int32_t* out_next,
                     void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * spec_tree_rerank -- reranking (section 4.2).  For each batch row, M
 * candidate nodes (the root excluded) with parent indices (-1: a child of the
 * root; otherwise below the node's own index) and values.  The m nodes first
 * in (value descending, depth ascending, index ascending) are kept -- the
 * shallower node wins among equal values, so with values that never grow
 * along a path the kept nodes form a connected tree -- and flattened in that
 * order after the root (position 0).
 *
 *   parents        [B][M]           int32     device, read
 *   values         [B][M]           float32   device, read
 *   out_nodes      [B][m]           int32     device, written: candidate index at position p + 1
 *   out_parent_pos [B][m]           int32     device, written: the parent's position (0 = root)
 *   out_mask       [B][m+1][m+1]    uint8     device, written: 1 where the column is the row's
 *                                             own position or an ancestor's (the attention mask)
 *   1 <= m <= M <= SPEC_RERANK_MAX.  Needs no workspace.
 * A batch row with a parent index out of range, a NaN value, or a kept node
 * whose parent is not kept gets -1 outputs and an all-zero mask.
 */
int spec_tree_rerank(const int32_t* parents, const float* values, int B, int M, int m, int32_t* out_nodes,
                     int32_t* out_parent_pos, uint8_t* out_mask, void* hip_stream);

/*
 * spec_kv_commit -- KV commit of an accepted tree path ("Việc giải mã giả
 * định và EAGLE-3", KV cache rollback: write the draft's entries to scratch,
 * commit on acceptance).  The verifier appended the N tree nodes' KV rows at
 * positions prefix[b] + n; the accepted path path[b][0..d] (d = accept_len[b],
 * the out_path / out_accept_len of a tree verification) moves to positions
 * prefix[b] + 0..d in every plane, in place, and out_len[b] = prefix[b] + d + 1.
 * Rows move in increasing order; as the path increases from node 0, no row is
 * overwritten before it is read.
 *
 *   kv          device, read and written: row (plane, b, s) at byte offset
 *               plane*plane_stride + b*batch_stride + s*pos_stride, row_bytes
 *               long (e.g. planes = layers x {K, V}, a row = heads x head_dim);
 *               16-byte aligned layouts move with 16-byte accesses
 *   capacity    positions s = 0 .. capacity-1 that exist in every (plane, b)
 *               row of the cache (>= 1)
 *   prefix      [B] int32 device; path [B][path_stride] int32 device;
 *   accept_len  [B] int32 device; out_len [B] int32 device, written
 *   N           tree nodes (path entries must be below N)
 * A row with accept_len < 0, a negative prefix, a path that is not node 0
 * followed by increasing node indices below N, or a path whose last (largest)
 * node lies past the cache (prefix[b] + path[b][d] >= capacity) moves nothing
 * and gets out_len -1; the check covers every row the move would touch before
 * any byte of the batch row moves.
 * Rows must not overlap: pos_stride >= row_bytes, and no two (plane, b,
 * position) rows may share bytes (a zero plane_stride with planes > 1, or a
 * zero batch_stride with B > 1, is SPEC_EINVAL; other overlaps are the
 * caller's to avoid and give undefined contents).  B <= 65535 and
 * path_stride <= SPEC_MAX_NODES (a path is at most one tree's nodes), else
 * SPEC_EUNSUPPORTED.
 */
int spec_kv_commit(void* kv, int planes, long long plane_stride, int B, long long batch_stride,
                   long long pos_stride, int row_bytes, int capacity, const int32_t* prefix, const int32_t* path,
                   int path_stride, int N, const int32_t* accept_len, int32_t* out_len, void* hip_stream);

/*
 * ---- A key/value cache held in four bits ----
 *
 * The target's forward pass over a draft reads the whole cache once a step, so
 * at long contexts the cache's bytes are the step's time.  These calls keep it
 * in four bits, around the verification: append the draft's rows, attend to
 * cache and draft, verify, commit the accepted path (spec_kv_commit on the
 * four arrays), score the cached rows, evict.
 *
 * A cached K or V row of head_dim = D elements (D = 64, 128 or 256) is D/2
 * bytes of E2M1 codes (element 2i in the low half of byte i; magnitudes 0, .5,
 * 1, 1.5, 2, 3, 4, 6 for codes 0..7, bit 3 the sign) and D/32 scale bytes, one
 * for each 32 elements: the OCP microscaling layout.  Byte s in 1..252 stands
 * for 2^(s-127), byte 0 comes with an all-zero block, byte 255 means NaN (253
 * and 254, whose values need not be float32 numbers, are not written).
 *
 * Every batch row b has `prefix[b]` committed rows, slots 0 .. prefix[b]-1 of
 * each of its heads, and `counts[b]` new ones (counts NULL: N) in the slots
 * behind them.  A batch row with prefix[b] < 0, counts[b] outside [0, N] or
 * prefix[b] + counts[b] > capacity is an error row: nothing of its cache,
 * scores or positions is read or written, and its outputs are the ones named at
 * each call.  A negative prefix (what spec_kv_commit reports for an error row)
 * so marks a row of the batch as unused.
 */

/* The host knows no lengths, so how attention, score and evict are cut up goes by
 * the cache's capacity and the batch's size: a call on short rows takes longer in
 * a cache of many more slots than they need, and one row far longer than a large
 * batch's others is not spread over the GPU.  Sums differ in their rounding alone. */

/* One layer's cache.  Row (b, h, slot): codes at b*code_batch + h*code_head +
 * slot*code_pos bytes from k_codes / v_codes, scales likewise.  Codes: base and
 * strides multiples of 16 bytes; scales: of D/32 bytes.  No two rows may share
 * bytes (zero strides where B, heads or capacity exceed 1 are SPEC_EINVAL; the
 * stride of a dimension of one element does not count).
 * B and heads at most 65535, capacity at most 2^30, code_pos and scale_pos at
 * most 2^24.  Calls of 2^31 query rows, of 2^32 threads (rows of B, tokens and
 * heads times D/8 in append and read, about 2^27 query rows in attention, 2^22
 * heads of the batch in evict) and more are SPEC_EUNSUPPORTED. */
typedef struct {
    void* k_codes;
    void* k_scales;
    void* v_codes;
    void* v_scales;
    int32_t B, heads, capacity, head_dim;
    int64_t code_batch, code_head, code_pos;
    int64_t scale_batch, scale_head, scale_pos;
} spec_kvq_cache_t;

/* Rows of D elements, (b, n, head) at data + b*batch + n*pos + head*head
 * elements; base and strides multiples of 16 bytes, D contiguous. */
typedef struct {
    const void* data;
    int64_t batch, pos, head;
} spec_kvq_rows_t;

/*
 * spec_kvq_append -- quantise new K and V rows into slots prefix[b] ..
 * prefix[b] + counts[b] - 1.  A block of 32 gets the smallest scale 2^e, e >=
 * -96, with max|x| <= 7 * 2^e (so the largest element is off by at most half a
 * step, as the others are) and its elements round to nearest, ties to the even
 * code.  e ends at 125: larger elements than 7 * 2^125 become 6 * 2^125.  A block holding a NaN or an infinity is stored as NaN (scale 255),
 * and so is the first block of the slot's K row, whichever of the two rows held
 * it: every query that sees the slot answers NaN, and no other.
 *   k, v      rows of (b, n, head), SPEC_F32 or SPEC_BF16, n < N
 *   prefix    [B] int32 device; counts [B] int32 device or NULL
 */
int spec_kvq_append(const spec_kvq_cache_t* cache, const spec_kvq_rows_t* k, const spec_kvq_rows_t* v,
                    spec_dtype_t dtype, int N, const int32_t* prefix, const int32_t* counts, void* hip_stream);

/*
 * spec_kvq_read -- the values that slots prefix[b] .. prefix[b] + counts[b] - 1
 * stand for (exact in either type): out_k, out_v [B][N][heads][D] contiguous,
 * 16-byte aligned.  Rows past counts[b] and error rows are zeros.
 */
int spec_kvq_read(const spec_kvq_cache_t* cache, spec_dtype_t dtype, int N, const int32_t* prefix,
                  const int32_t* counts, void* out_k, void* out_v, void* hip_stream);

/*
 * spec_kvq_attention -- softmax attention of N new tokens' queries.  Query
 * (b, n, hq) reads head hq / (q_heads / heads) of the cache: o = sum_s p_s V_s,
 * p = softmax over its visible slots of scale * (q . K_s).  It sees every
 * committed slot and, of the new ones prefix[b] + m (m < counts[b]), those with
 * m <= n (mask NULL: a chain or a prompt) or with mask[b][n][m] != 0 (a tree's
 * ancestor mask, as spec_tree_rerank writes it).
 *   q        rows of (b, n, hq), SPEC_F32 or SPEC_BF16
 *   mask     [B][N][N] uint8 device, batch rows mask_batch bytes apart (0: one
 *            mask for all), or NULL
 *   scale    above 0, scale * log2(e) a finite float32
 *   out      [B][N][q_heads][D], of q's type, contiguous, 16-byte aligned
 *   out_lse  [B][N][q_heads] float32: log sum_s exp(scale * (q . K_s)); or NULL
 * A query that sees no slot, tokens n >= counts[b] and error rows answer zeros
 * and an out_lse of -inf.  What a query does not see never reaches it, whatever
 * its bytes; a NaN reaches it through a K row alone (spec_kvq_append marks the K
 * row of either).  Queries that are not finite (or, float32, round to an infinite
 * bfloat16) and those with a visible score that, in base two, is no finite float32
 * give unspecified rows.  K and V enter exactly (E2M1 times a power of two is a
 * bfloat16), products and sums are float32 (V of 2^90 and more may overflow in
 * them: they are divided by the probabilities' sum at the end); with bfloat16
 * queries the probabilities round to bfloat16 before they meet V.
 * q_heads a multiple of heads; N <= 65536 (with a mask: N <= SPEC_MAX_NODES).
 * workspace: spec_kvq_attention_workspace_bytes(...) bytes (may be 0), any
 * contents; left as scratch.
 */
size_t spec_kvq_attention_workspace_bytes(int B, int N, int q_heads, int heads, int head_dim, int capacity,
                                          spec_dtype_t dtype);
int spec_kvq_attention(const spec_kvq_rows_t* q, spec_dtype_t dtype, int q_heads, int N,
                       const spec_kvq_cache_t* cache, const int32_t* prefix, const int32_t* counts,
                       const uint8_t* mask, int64_t mask_batch, float scale, void* out, float* out_lse,
                       void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * spec_kvq_score -- accumulated attention weight, after the accepted path was
 * committed.  The accepted queries are tokens path[b][0..d], d = accept_len[b]
 * (path NULL: tokens 0..d), of which the t-th sees slots 0 .. prefix[b] + t.
 * With w_s = sum over them and over the queries hq of a cache head of
 * exp(scale * (q . K_s) - lse), scores[b][h][s] += w_s for committed slots, and
 * the slots the commit added, prefix[b] .. prefix[b] + d, start at w_s; their
 * positions[b][h][s] become seen[b] + (s - prefix[b]).  Sums are float32 in a
 * fixed order.
 *   q, lse       what spec_kvq_attention took and gave ([B][N][q_heads])
 *   prefix       the committed rows before this step; path [B][path_stride]
 *   scores       [B][heads][capacity] float32, positions [B][heads][capacity]
 *                int32, read and written; seen [B] int32: tokens the sequence
 *                had before this step (evicted ones too)
 * A query whose lse is -inf adds nothing (to a slot whose K is a number).
 * Error rows here: accept_len < 0 (or >= path_stride, or >= N), a path that is
 * not token 0 followed by increasing tokens below N, prefix < 0, or prefix + d
 * + 1 > capacity; they are left as they were.  path_stride <= SPEC_MAX_NODES
 * where path is given.
 * workspace: spec_kvq_score_workspace_bytes(...) bytes (path_stride 0: no path;
 * may be 0), any contents; left as scratch.
 */
size_t spec_kvq_score_workspace_bytes(int B, int N, int q_heads, int heads, int head_dim, int capacity,
                                      int path_stride, spec_dtype_t dtype);
int spec_kvq_score(const spec_kvq_rows_t* q, spec_dtype_t dtype, int q_heads, int N, const float* lse,
                   const spec_kvq_cache_t* cache, const int32_t* prefix, const int32_t* path, int path_stride,
                   const int32_t* accept_len, float scale, float* scores, int32_t* positions, const int32_t* seen,
                   void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * spec_kvq_evict -- cut every head of a batch row down to `keep` rows, in
 * place.  Of slots 0 .. lengths[b]-1 the kept ones are first those with
 * positions < sink or >= seen[b] - recent, then the others by score, larger
 * first (NaN after all numbers), the lower slot first among equals.  A kept row
 * below slot keep stays where it is; the i-th kept row at or above it moves
 * into the i-th gap below it (both counted upwards), so only those rows move.
 * Slots past the new length are left as they were.
 *   scores, positions          [B][heads][capacity], read
 *   out_scores, out_positions  the same, written up to the new length: each
 *                              either the array read, or one that overlaps neither
 *   lengths, seen              [B] int32: the rows in the cache, and the tokens the sequence
 *                              has had, this step's among them (spec_kvq_score's seen[b] +
 *                              accept_len[b] + 1)
 *   out_len     [B] int32: min(lengths[b], keep); error rows (lengths[b] < 0 or
 *               above capacity): -1, and nothing of them moves
 *   out_source  [B][heads][keep] int32: the slot each kept row came from, -1
 *               past the new length
 *   1 <= keep <= capacity; sink, recent >= 0
 * workspace: spec_kvq_evict_workspace_bytes(...) bytes, any contents.
 */
size_t spec_kvq_evict_workspace_bytes(int B, int heads, int capacity, int keep);
int spec_kvq_evict(const spec_kvq_cache_t* cache, const float* scores, const int32_t* positions,
                   const int32_t* lengths, const int32_t* seen, int keep, int sink, int recent, float* out_scores,
                   int32_t* out_positions, int32_t* out_len, int32_t* out_source, void* workspace,
                   size_t workspace_bytes, void* hip_stream);

/*
 * spec_accept_rate -- "064 · 投机解码", section 二: the chance that one drafted
 * token is accepted is the overlap of the two distributions,
 * alpha[b][k] = sum_i min(p'_k(i), q'_k(i)) for k < K, with
 * p' and q' transformed as in spec_verify_chain (rows 0..K-1 of the logits are
 * read; row K is not).  Greedy (temperature == 0): 1 if the argmax of target
 * row k equals the argmax of draft row k, else 0.  An invalid row gives NaN.
 *
 *   target_logits [B][K+1][V], draft_probs [B][K][V] (device, read)
 *   out_alpha     [B][K]       float32                 device, written
 */
int spec_accept_rate(const void* target_logits, spec_dtype_t dtype, const float* draft_probs,
                     int B, int K, int V, float temperature, int top_k,
                     float* out_alpha, void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * ---- A paged key/value cache, and attention behind shared prefixes ----
 *
 * A server's sequences grow by unknown amounts and many begin alike.  These
 * calls keep K and V in pages of a pool, hand the pages out on the GPU, and let
 * any number of batch rows attend to one stored prefix:
 *   spec_page_step (pages and slots for the step's new tokens), spec_paged_append
 *   (their rows), spec_paged_plan (once a step), spec_paged_attention (every layer),
 *   LM head, verification; for a tree spec_paged_append again with the accepted
 *   path, which puts its rows in place.
 *
 * A table row t has tables[t][0 .. held[t]-1], the pages of its slots 0 .. in
 * order: slot s is slot s % page_size of page tables[t][s / page_size], and the
 * number tables[t][s / page_size] * page_size + s % page_size names it.  Rows of the
 * batch come first; rows behind them may hold prefixes.
 */

/*
 * spec_page_step -- pages for N new tokens a row.  Row t needs
 * ceil((lengths[t] + counts[t]) / page_size) pages (counts NULL: N), and none
 * where lengths[t] < 0 (a sequence that has ended).  The free pages are a ring:
 * entries head .. head + free - 1 of `ring` (mod pages), state = {head, free}.
 * Rows that need more than they hold take pages from its head, in the order of the
 * rows, as long as they last; the first row that does not get all its own gets
 * none, nor does any after it that needs some.  Rows that need fewer put those
 * they do not need behind its tail (in order, row by row); they are handed out by
 * later calls.  Entries of `tables` from the need on are left as they were.
 *   tables       [T][width] int32, rows table_stride elements apart; held [T]; ring
 *                [pages]; state [2]: read and written
 *   lengths [T], counts [T] or NULL, int32
 *   out_held, out_state   where held and state go: the arrays read (in place), or ones
 *                that overlap nothing
 *   out_granted  [T] int32: counts[t] (0 for a row that has ended), or -1: not enough pages,
 *                counts[t] outside [0, N], more than width pages needed, or held[t] outside
 *                [0, min(width, pages)]; nothing of such a row changes.  It can be the `counts`
 *                of the calls below, which leave rows of -1 out.
 *   out_slots    [T][N] int32: the slot of token n (its place is lengths[t] + n), -1 for
 *                n >= granted[t], and where the page's number is none of the pool's
 * A state outside [0, pages) and [0, pages] serves no row and is left as it is.
 * page_size a power of two from 16 to 1024, T and N at most 65536 and T * N below 2^31,
 * pages * page_size and width * page_size at most 2^30.
 * workspace: 256 bytes, zero-filled before its first use and left zero.
 */
#define SPEC_PAGE_STEP_WORKSPACE_BYTES 256
int spec_page_step(int32_t* tables, int64_t table_stride, int T, int width, int page_size, int pages,
                   const int32_t* held, const int32_t* state, int32_t* ring, const int32_t* lengths,
                   const int32_t* counts, int N, int32_t* out_held, int32_t* out_state, int32_t* out_granted,
                   int32_t* out_slots, void* workspace, size_t workspace_bytes, void* hip_stream);

/* One layer's pages, bfloat16: row (page, slot of it, head) at k (and v) + page*page_stride +
 * slot*slot_stride + head*head_stride elements.  Bases and strides multiples of 16 bytes; no two
 * rows may share memory (the stride of a dimension of one element does not count).  head_dim 64,
 * 128 or 256; heads at most 65535; slot_stride at most 2^20. */
typedef struct {
    void* k;
    void* v;
    int32_t pages, page_size, heads, head_dim;
    int64_t page_stride, slot_stride, head_stride;
} spec_paged_cache_t;

/*
 * spec_paged_append -- K and V rows into slots[b][n], b < B, n < N (rows of `slots`
 * slots_stride elements apart).  Without a path, slot n gets row (b, n).  With one, an
 * accepted path as verification gives it, slot n gets row (b, path[b][n]) for n <=
 * accept_len[b] (none where that is negative or not below N).  A slot of -1, or outside
 * the pool, gets nothing, nor does one whose path entry is outside [0, source_n).
 *   k, v      rows of (b, n, head), SPEC_F32 (rounded to nearest, ties to even) or SPEC_BF16;
 *             source_n of them a batch row (without a path at least N)
 * Two tokens on one slot leave either's row.
 */
int spec_paged_append(const spec_paged_cache_t* cache, const spec_kvq_rows_t* k, const spec_kvq_rows_t* v,
                      spec_dtype_t dtype, int B, int N, int source_n, const int32_t* slots, int64_t slots_stride,
                      const int32_t* path, int path_stride, const int32_t* accept_len, void* hip_stream);

/*
 * spec_paged_plan -- how the attention of a step is cut up, from its lengths: made once,
 * for every layer whose calls have these sizes.
 *   lengths    [T] int32: committed slots of each table row; the new tokens of batch row
 *              b < B <= T lie behind them, counts[b] of them (NULL: N)
 *   prefix_row [B] int32 or NULL: the table row whose committed slots come before
 *              batch row b's own (negative: none).  Neighbouring rows with the same one share
 *              the reading of it.
 *   plan       spec_paged_plan_bytes(...) bytes, 256-byte aligned, any contents; with_prefix:
 *              whether prefix_row is given
 * A batch row with lengths[b] < 0, counts[b] outside [0, N], more slots than width * page_size,
 * or a prefix_row of T or more, or one whose length is outside [0, width * page_size], is an error row.
 */
size_t spec_paged_plan_bytes(int B, int N, int q_heads, int heads, int head_dim, int with_prefix);
int spec_paged_plan(int B, int N, int q_heads, int heads, int head_dim, int T, int width, int page_size,
                    const int32_t* lengths, const int32_t* counts, const int32_t* prefix_row, void* plan,
                    size_t plan_bytes, void* hip_stream);

/*
 * spec_paged_attention -- softmax attention of N new tokens' queries.  Query (b, n, hq)
 * reads head hq / (q_heads / heads).  It sees every slot of its prefix, every
 * committed one of its own, and of the new ones lengths[b] + m (m < counts[b]) those with m <= n
 * (mask NULL) or with mask[b][n][m] != 0.
 *   q          rows of (b, n, hq), SPEC_F32 or SPEC_BF16; mask, scale, out, out_lse: as for
 *              spec_kvq_attention
 *   tables     [T][width], rows table_stride elements apart; B, N, q_heads, heads, head_dim, width and
 *              page_size as the plan was made with.  A call whose sizes are not the plan's writes nothing.
 * A query that sees no slot, tokens n >= counts[b] and error rows answer zeros and an out_lse
 * of -inf.  What a query does not see never reaches it, whatever its bytes.  One that sees a slot
 * whose K or V holds a NaN or an infinity gives unspecified numbers; one that sees a slot whose
 * page is none of the pool's gives NaN.  Products and sums are float32; with bfloat16
 * queries the probabilities round to 16 bits before they meet V, and to bfloat16 where
 * more than 32 query rows of a head meet the same slots (the same queries as SPEC_F32
 * avoid that, and the output is float32).
 * workspace: spec_paged_attention_workspace_bytes(...) bytes (may be 0), any contents;
 * left as scratch.
 */
size_t spec_paged_attention_workspace_bytes(int B, int N, int q_heads, int heads, int head_dim, int with_prefix);
int spec_paged_attention(const spec_kvq_rows_t* q, spec_dtype_t dtype, int B, int N, int q_heads,
                         const spec_paged_cache_t* cache, const int32_t* tables, int64_t table_stride, int width,
                         const void* plan, size_t plan_bytes, int with_prefix, const uint8_t* mask,
                         int64_t mask_batch, float scale, void* out, float* out_lse, void* workspace,
                         size_t workspace_bytes, void* hip_stream);

/*
 * ---- Log probabilities of tokens ----
 *
 * What a server answers beside the tokens that verification emits, and what a
 * draft model is trained on: log p(t) of given tokens under p = softmax(z / T),
 * the rows' entropy, their likeliest tokens; and the gradient for the logits.
 */

/*
 * spec_token_logprobs -- for each of R logit rows z (row r at logits +
 * r*row_stride elements, V of them, any element's alignment), with y = z / T:
 *   out_logprobs[r][m]  = y[t] - log sum_i exp(y_i), t = tokens[r][m]
 *   out_entropy[r]      = -sum_i p_i log p_i
 *   out_top_tokens[r], out_top_logprobs[r]: the top_n largest logits, larger first,
 *                         the lower index first among equals (-1 and -inf where
 *                         fewer than top_n are above -inf)
 *   out_stats[r][3]     = what spec_token_logprobs_grad goes by: the largest logit,
 *                         log2 of sum_i 2^(log2(e)/T * (z_i - it)), the entropy
 * A logit of -inf has probability 0 (a token that has it, log probability -inf).
 * A negative token is none: its log probability is 0.  A row all of whose tokens
 * are negative is not read: log probabilities, entropy and statistics 0, tops -1
 * and -inf; so out_tokens of a verification call can be given as it is.  A row
 * with a NaN, a +inf or only -inf among its logits, or with a token of V or more,
 * answers NaN (and -1).  Sums are float32 over a thread's elements, float64 after.
 *   tokens         [R][M] int32, 0 <= M <= SPEC_TOPK_MAX (M 0: NULL, every row is read)
 *   temperature    above 0; log2(e) / temperature a finite float32
 *   top_n          0 <= top_n <= SPEC_TOPK_MAX
 *   out_logprobs   [R][M] (NULL if M is 0); out_entropy [R], out_stats [R][3] float32, each
 *                  may be NULL; out_top_tokens [R][top_n] int32, out_top_logprobs
 *                  [R][top_n] float32 (NULL if top_n is 0)
 * workspace: spec_token_logprobs_workspace_bytes(...) bytes (may be 0), zero-filled
 * before its first use and left zero by every call, so that calls of any sizes
 * may share one.  Calls that overlap on one workspace race.
 */
size_t spec_token_logprobs_workspace_bytes(int R, int V, int top_n, spec_dtype_t dtype);
int spec_token_logprobs(const void* logits, spec_dtype_t dtype, int64_t row_stride, int R, int V,
                        const int32_t* tokens, int M, float temperature, int top_n, float* out_logprobs,
                        float* out_entropy, float* out_stats, int32_t* out_top_tokens, float* out_top_logprobs,
                        void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * spec_token_logprobs_grad -- the gradient for the logits, of their type:
 *   dz_i = (1/T) (sum_m g_m [i = t_m] - p_i sum_m g_m - h p_i (log p_i + H))
 * where g = grad_logprobs[r], h = grad_entropy[r], H the entropy.  A token given
 * more than once collects each of its gradients; negative tokens' do not count.
 * Rows all of whose tokens are negative get zeros; rows that answered NaN get NaN.
 *   tokens, temperature, stats   as spec_token_logprobs had and gave them (M >= 1)
 *   grad_logprobs  [R][M] float32; grad_entropy [R] float32 or NULL
 *   out_grad       row r at out_grad + r*grad_stride elements; may be the logits
 *                  themselves (the same pointer and stride), else overlaps nothing
 */
int spec_token_logprobs_grad(const void* logits, spec_dtype_t dtype, int64_t row_stride, int R, int V,
                             const int32_t* tokens, int M, const float* stats, const float* grad_logprobs,
                             const float* grad_entropy, float temperature, void* out_grad, int64_t grad_stride,
                             void* hip_stream);

/* Zero-fills `workspace_bytes` (a multiple of 4) of a 256-byte aligned workspace
 * with a fill kernel on hip_stream (no memset node, so it may be captured). */
int spec_workspace_init(void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Instrumentation.
 *
 * spec_profile_events (the library's one per-thread state): the next
 * verification call made BY THIS HOST THREAD
 * launches its dominant (vocabulary-streaming) kernel with `start_event` and
 * `stop_event` attached to the dispatch (hipExtLaunchKernel), so that they hold
 * that kernel's own start and end times; both are hipEvent_t created by the
 * caller.  The request is consumed by that call.
 *
 * spec_copy_probe: plain device-to-device copy of `bytes` (multiple of 16,
 * 16-byte aligned pointers) by a streaming kernel, for calibrating hardware
 * byte counters against a known traffic.
 *
 * spec_read_probe: reads `bytes` (multiple of 16, 16-byte aligned) of device
 * memory once with the same 16-byte non-temporal loads as the verification
 * kernels and writes nothing but, at most, one word to `sink` (4 bytes of device
 * memory, contents meaningless): the achievable streaming-read bandwidth.
 */
int spec_profile_events(void* start_event, void* stop_event);
int spec_copy_probe(const void* src, void* dst, size_t bytes, void* hip_stream);
int spec_read_probe(const void* src, size_t bytes, void* sink, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */
