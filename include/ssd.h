/*
 * ssd.h -- C ABI of the GB300 (sm_103a) speculative-decoding sampling library.
 *
 * The library implements the data-parallel sampling step of speculative
 * decoding and of speculative speculative decoding (SSD / Saguaro) over
 * full-vocabulary logits that already sit in device memory:
 *   - the per-position accept test min(1, p(x)/q(x)) up to the first
 *     rejection and the bonus token drawn from normalize((p - q)^+);
 *   - the top-F bonus-token guesses per draft position;
 *   - Saguaro sampling (cached tokens' draft probability times C, then
 *     renormalised);
 *   - the outcome-cache build and lookup keyed by (row, k accepted, bonus t);
 *   - the geometric fan-out allocation of the cache budget (host helper);
 * and what surrounds a round in a serving loop:
 *   - penalties, biases and grammar masks on the logits before it;
 *   - the pages, slots and positions of the key/value cache after it;
 *   - attention of rows that share a prefix (the branches of a sequence).
 *
 * Sources, cited by page title and section:
 *   [SSD-note] "论文阅读：Speculative Speculative Decoding — 消除推测解码的最后一个顺序瓶颈"
 *   [SD-7.3]   "7.3 Speculative Decoding：投机采样加速"
 *   [SD-blog]  "推测解码：用一个“小模型”骗出 3 倍推理速度"
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers unless the comment says "host".
 *   - The caller owns all memory; the library never allocates.  Scratch
 *     space comes from a caller-provided workspace sized by the matching
 *     *_workspace_size() call.  The first bytes of the workspace (counters)
 *     are cleared on the stream at the start of every call, so a workspace
 *     needs no initialisation and may be reused by any entry point, but two
 *     calls that run concurrently must not share one.  Sizes depend on the
 *     current device's SM count (small batches split rows over more CTAs):
 *     query them with the device current that the call will run on.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is
 *     the legacy default stream).  The library keeps no global state, so
 *     calls are thread-safe.
 *   - The return value reports argument errors (checked on the host before
 *     anything is enqueued) and launch errors.  Errors found on the device
 *     are OR-ed as SSD_DEV_* bits into *dev_status when dev_status is not
 *     NULL; the library never traps and every wait on the device is bounded.
 *   - Logit rows are contiguous over the vocabulary (V elements); successive
 *     rows are `row_stride` elements apart.  Any element-aligned pointer and
 *     stride is accepted; 16-byte aligned rows take the bulk-copy fast path.
 *   - Philox-4x32-10 uniforms: key = (seed lo32, seed hi32), counter =
 *     (c0, c1, stream, round), u = (out0 >> 8) * 2^-24 in [0, 1).
 *     Streams: 0 = accept test, 1 = bonus draw, 2 = draft / Saguaro sample.
 */
#ifndef SSD_H
#define SSD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SSD_OK = 0,
  SSD_ERR_INVALID_ARG = 1,   /* an argument is out of range or inconsistent */
  SSD_ERR_UNSUPPORTED = 2,   /* valid, but beyond the library's compiled limits (e.g. F > 15) */
  SSD_ERR_TABLE_FULL = 3,    /* host-detectable: cache capacity below 2 n */
  SSD_ERR_DUPLICATE_KEY = 4, /* reserved; duplicates are reported via dev_status */
  SSD_ERR_WORKSPACE = 5,     /* workspace NULL, misaligned or too small */
  SSD_ERR_CUDA = 6           /* a CUDA runtime call failed */
} ssd_status;

/* Bits OR-ed into *dev_status by device code. */
#define SSD_DEV_BAD_TOKEN 0x1      /* a draft token outside [0, V); treated as token 0 */
#define SSD_DEV_ZERO_RESIDUAL 0x2  /* residual mass underflowed; bonus drawn from p_k */
#define SSD_DEV_TIMEOUT 0x4        /* a bounded wait gave up; outputs are undefined */
#define SSD_DEV_TABLE_FULL 0x8     /* cache insert found no free slot */
#define SSD_DEV_DUPLICATE_KEY 0x10 /* cache insert met an existing key */
#define SSD_DEV_BAD_TEMPERATURE 0x20 /* a per-sequence temperature negative or not
                                        finite; that sequence is verified greedily */
#define SSD_DEV_BAD_FANOUT 0x40    /* a per-row fan-out outside [0, Fmax]; clamped */
#define SSD_DEV_BAD_PENALTY 0x80   /* a penalty not finite, or a repetition penalty <= 0; left out */
#define SSD_DEV_BAD_LENGTH 0x100   /* a length or count out of range or inconsistent; see the call */
#define SSD_DEV_NO_PAGES 0x200     /* the free pages did not suffice for every request */
#define SSD_DEV_BAD_PAGE 0x400     /* a page id outside [0, num_pages); its tokens read as zeros */

typedef enum { SSD_BF16 = 0, SSD_F32 = 1, SSD_F16 = 2 } ssd_dtype; /* SSD_F16: attention only */

/* A batch of logit rows in device memory. */
typedef struct {
  const void* ptr;    /* device pointer to the first element of row 0 */
  int32_t dtype;      /* ssd_dtype */
  int32_t pad_;       /* must be 0 */
  int64_t row_stride; /* elements between the starts of consecutive rows, >= V */
} ssd_logits;

/* Compiled limits of the library. */
#define SSD_MAX_K 32       /* draft tokens per sequence */
#define SSD_MAX_F 15       /* bonus guesses per position */
#define SSD_MAX_V 16777215 /* vocabulary size (token ids and 24-bit uniforms stay exact) */

/* Static message for a status code. */
const char* ssd_status_string(int status);

/* Library version as 10000*major + 100*minor + patch. */
int ssd_version(void);

/* ---------------------------------------------------------------------------
 * ssd_verify -- rejection-sampling verification of K drafts per sequence.
 * [SD-7.3] §7.3.2 / §7.3.3; [SD-blog] §"三、接受概率为什么是对的";
 * [SSD-note] §"接受-拒绝机制", §"Saguaro 优化二：Saguaro 采样".
 *
 * For sequence b (0 <= b < B) with drafts x_0..x_{K-1}:
 *   p_i = softmax(z_target[b,i,:] / T),  i = 0..K   (position K: all accepted)
 *   q_j = softmax(z_draft[b,j,:] / T),   j = 0..Kq-1
 *   S_j = top-F_j of z_draft[b,j,:] (raw logit desc, ties to the lower index)
 *   q'_j(y) = q_j(y) * (C if y in S_j else 1) / (1 - (1-C) * q_j(S_j))
 *   accept x_i iff u_i < p_i(x_i) / q'_i(x_i),  u_i = U(seeds[b]; b, i, 0, round);
 *   k = the first rejected position, or K when every draft is accepted;
 *   w = (p_k - q'_k)^+ if k < K, else p_K;  Z = sum_y w(y);
 *   bonus t = smallest y with sum_{y'<=y} w(y') > u' * Z,
 *             u' = U(seeds[b]; b, k, 1, round).
 *   guesses[b,j,:] = top-(F_j + 1) of z_draft[b,j,:] minus x_j (j < K),
 *                    truncated to F_j, padded with -1 to Fmax.
 * C = 1 (or all F_j = 0) is plain speculative decoding, bit for bit.
 * T = 0 is the greedy limit T -> 0 (a serving setting the pages do not
 * treat): x_i is accepted iff it is the argmax of z_target[b,i,:] (ties to
 * the lower index), the bonus is the argmax of target row k, resid_mass is
 * 1, and guess_q is 1 for the draft argmax and 0 for other guesses; no
 * uniform is drawn.
 *
 * target      [B, K+1, V] logits: row (b, i) is row b*(K+1)+i.  Target rows
 *             past a known rejection of their sequence are not read: no
 *             output depends on p_i for i > k (the accept tests stop at the
 *             first rejection, [SD-7.3] §7.3.3); a row whose sequence is not
 *             yet decided when its turn comes is read (see
 *             ssd_verify_skipped_bytes).
 * draft       [B, Kq, V] logits, Kq in {K, K+1}: row (b, j) is row b*Kq+j.
 *             Every draft row is read (the guesses of every position).
 *             Verification reads draft rows 0..K-1; row K (when Kq = K+1)
 *             only feeds the guesses for the all-accepted outcome.
 * draft_tokens device [B, K] int32.
 * seeds       device [B] uint64 Philox keys.
 * fanout      HOST [Kq] int32 F_j (F_j in [0, SSD_MAX_F], F_j + 1 <= V),
 *             or NULL for all zero.  With Kq = K, F_K does not exist.
 * C           Saguaro factor in (0, 1].
 * accept_len  device [B] int32 out: k in [0, K].
 * bonus       device [B] int32 out: t in [0, V).
 * resid_mass  device [B] float out (or NULL): Z (1 - alpha_k when k < K;
 *             sum of p_K, i.e. ~1, when k = K).
 * guesses     device [B, Kq, Fmax] int32 out (or NULL).
 * guess_q     device [B, Kq, Fmax] float out (or NULL): q_j of each guess
 *             (plain draft probability), 0 for padding.
 * Fmax        >= max F_j when guesses is given.
 * workspace   device, 256-byte aligned, >= ssd_verify_workspace_size(B,K,Kq,V).
 * dev_status  device int32 (or NULL): SSD_DEV_* bits are OR-ed in.
 * T           temperature, finite and >= 0 (0: greedy).
 * ------------------------------------------------------------------------- */
size_t ssd_verify_workspace_size(int B, int K, int Kq, int V);
ssd_status ssd_verify(const ssd_logits* target, const ssd_logits* draft, int B, int K, int Kq,
                      int V, float T, const int32_t* draft_tokens, const uint64_t* seeds,
                      uint32_t round, const int32_t* fanout, float C, int32_t* accept_len,
                      int32_t* bonus, float* resid_mass, int32_t* guesses, float* guess_q,
                      int Fmax, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                      void* stream);

/* ---------------------------------------------------------------------------
 * ssd_verify_skipped_bytes -- the bytes of target rows that the last call of
 * ssd_verify, ssd_verify_ck, ssd_verify_ex or ssd_verify_round on `workspace`
 * did not read (rows past a rejection already known when their turn came).
 * A measurement aid: the logits streamed by that call are the target and
 * draft bytes minus this count.
 *
 * workspace   the call's workspace (256-byte aligned) and its size; B, K,
 *             Kq, V and dtype (ssd_dtype) those of the call.
 * out         device uint64 out, written in stream order after the call.
 * Errors: SSD_ERR_INVALID_ARG (bad sizes, null pointers), SSD_ERR_WORKSPACE
 * (smaller than ssd_verify_workspace_size).  Enqueues one 8-byte copy.
 * ------------------------------------------------------------------------- */
ssd_status ssd_verify_skipped_bytes(const void* workspace, size_t workspace_bytes, int B, int K,
                                    int Kq, int V, int dtype, uint64_t* out, void* stream);

/* ---------------------------------------------------------------------------
 * ssd_verify_ck -- ssd_verify with one Saguaro factor per draft position.
 * [SSD-note] §"关于逐位置 C 的思考": the pages use one global C and propose a
 * factor per position (positions whose fan-out covers more can bias less).
 *
 * As ssd_verify, with q'_j built from C_pos[j] instead of C:
 *   q'_j(y) = q_j(y) * (C_j if y in S_j else 1) / (1 - (1-C_j) * q_j(S_j)).
 * The drafts x_j must have been drawn from the same q'_j (for example by
 * ssd_saguaro_sample at position j with C = C_pos[j]).
 *
 * C_pos  HOST [K] float, each in (0, 1]; read before the call returns.
 * Every C_pos[j] equal to C gives the results of ssd_verify with C, bit for
 * bit.  Other arguments, errors and outputs: ssd_verify.
 * ------------------------------------------------------------------------- */
ssd_status ssd_verify_ck(const ssd_logits* target, const ssd_logits* draft, int B, int K,
                         int Kq, int V, float T, const int32_t* draft_tokens,
                         const uint64_t* seeds, uint32_t round, const int32_t* fanout,
                         const float* C_pos, int32_t* accept_len, int32_t* bonus,
                         float* resid_mass, int32_t* guesses, float* guess_q, int Fmax,
                         void* workspace, size_t workspace_bytes, int32_t* dev_status,
                         void* stream);

/* ---------------------------------------------------------------------------
 * ssd_verify_ex -- ssd_verify with a temperature per sequence and an
 * optional Saguaro factor per draft position (the pages use one T and one C;
 * a batch of requests with their own sampling settings needs both).
 *
 * As ssd_verify_ck, with sequence b verified at temperature T_rows[b]:
 * T_rows[b] > 0 as ssd_verify at that T; T_rows[b] = 0 greedy (see
 * ssd_verify).  A negative or non-finite T_rows[b] is verified greedily and
 * sets SSD_DEV_BAD_TEMPERATURE.  A call whose T_rows are all equal to T > 0
 * gives the results of ssd_verify_ck with T.
 *
 * T_rows  device [B] float.
 * C_pos   HOST [K] float in (0, 1], or NULL for C = 1 at every position.
 * Other arguments, errors and outputs: ssd_verify.
 * ------------------------------------------------------------------------- */
ssd_status ssd_verify_ex(const ssd_logits* target, const ssd_logits* draft, int B, int K,
                         int Kq, int V, const float* T_rows, const int32_t* draft_tokens,
                         const uint64_t* seeds, uint32_t round, const int32_t* fanout,
                         const float* C_pos, int32_t* accept_len, int32_t* bonus,
                         float* resid_mass, int32_t* guesses, float* guess_q, int Fmax,
                         void* workspace, size_t workspace_bytes, int32_t* dev_status,
                         void* stream);

/* ---------------------------------------------------------------------------
 * ssd_verify_round -- one SSD round in one launch: ssd_verify, the outcome
 * cache of the round's guesses (ssd_cache_build_guesses) and its lookup with
 * every sequence's outcome (ssd_cache_lookup).  [SSD-note] §"SSD 的核心思想":
 * the drafter prepares a continuation per predicted outcome (k, t) and the
 * round goes on at once when the real outcome was predicted; §"Saguaro 优化三":
 * the batch proceeds without waiting only if every sequence hits.
 *
 * Arguments and outputs of ssd_verify (guesses is required), plus:
 * table       device, 16-byte aligned, table_bytes >= ssd_cache_bytes(B*Kq*Fmax);
 *             its previous content is discarded (the launch clears it before
 *             inserting); afterwards it holds the round's guesses in the
 *             format of ssd_cache_build_guesses, so ssd_cache_lookup can read
 *             it.  Too small: SSD_ERR_TABLE_FULL.
 * out_branch  device [B] int32 out: (b*Kq + k)*Fmax + f of the guess that
 *             equals the outcome (k, t) = (accept_len[b], bonus[b]), or -1.
 * all_hit     device int32 out (or NULL): 1 if every sequence hit, else 0.
 * The results equal those of the three calls in sequence; outputs are
 * undefined after SSD_DEV_TIMEOUT.
 * ------------------------------------------------------------------------- */
ssd_status ssd_verify_round(const ssd_logits* target, const ssd_logits* draft, int B, int K,
                            int Kq, int V, float T, const int32_t* draft_tokens,
                            const uint64_t* seeds, uint32_t round, const int32_t* fanout, float C,
                            int32_t* accept_len, int32_t* bonus, float* resid_mass,
                            int32_t* guesses, float* guess_q, int Fmax, void* table,
                            size_t table_bytes, int32_t* out_branch, int32_t* all_hit,
                            void* workspace, size_t workspace_bytes, int32_t* dev_status,
                            void* stream);

/* ---------------------------------------------------------------------------
 * ssd_verify_noalloc -- ssd_verify without a caller workspace.  The pages have
 * no counterpart: this is a deployment convenience.
 *
 * For callers that cannot allocate device memory where they call the library
 * (a plugin of an inference runtime whose enqueue hook may not allocate, a
 * process whose device memory belongs to a pool allocator, a decode loop that
 * cannot pay for cudaMalloc and its implicit synchronisation).  The scratch
 * space is a SSD_NOALLOC_SCRATCH_BYTES array compiled into the library; every
 * GPU that loads the library holds it until the process exits.  Arguments and
 * results are those of ssd_verify.
 *   - Requests whose ssd_verify_workspace_size(B, K, Kq, V) exceeds
 *     SSD_NOALLOC_SCRATCH_BYTES return SSD_ERR_WORKSPACE (use ssd_verify with
 *     your own workspace); nothing is enqueued.  4 MiB covers, for example,
 *     B = 256 sequences with K = 8 at V = 151936.
 *   - The first call on a device looks up the array's address
 *     (cudaGetSymbolAddress, with that device current) and caches it; make
 *     that first call before any stream capture on the device.  The cache is
 *     keyed on the current context: after cudaDeviceReset the next call
 *     looks the address up again (make it, too, outside stream capture).
 *   - All calls on a device share the array; the parts that must start at
 *     zero are cleared at the start of each call.  Calls whose work overlaps
 *     on the GPU (different streams or host threads) race on the array and
 *     must be serialised by the caller.
 *   - Nothing is allocated: no cudaMalloc, cudaFree or allocating library
 *     routine is called.
 * ------------------------------------------------------------------------- */
#define SSD_NOALLOC_SCRATCH_BYTES (4u << 20)
ssd_status ssd_verify_noalloc(const ssd_logits* target, const ssd_logits* draft, int B, int K,
                              int Kq, int V, float T, const int32_t* draft_tokens,
                              const uint64_t* seeds, uint32_t round, const int32_t* fanout,
                              float C, int32_t* accept_len, int32_t* bonus, float* resid_mass,
                              int32_t* guesses, float* guess_q, int Fmax, int32_t* dev_status,
                              void* stream);

/* ---------------------------------------------------------------------------
 * ssd_topf_bonus -- bonus-token guesses alone.  [SSD-note] §"怎么猜奖励 token":
 * the top-F_j draft logits of position j, excluding the token already sampled
 * there.
 *
 * draft        [B, Kq, V] logits.
 * draft_tokens device [B, K] int32 (or NULL = no exclusion); positions
 *              j < K exclude draft_tokens[b, j].
 * fanout       HOST [Kq] int32.
 * guesses      device [B, Kq, Fmax] int32 out, -1 padded.
 * guess_q      device [B, Kq, Fmax] float out (or NULL): q_j(guess) at T.
 * ------------------------------------------------------------------------- */
size_t ssd_topf_workspace_size(int B, int Kq, int V);
ssd_status ssd_topf_bonus(const ssd_logits* draft, int B, int Kq, int V, float T,
                          const int32_t* draft_tokens, int K, const int32_t* fanout, int Fmax,
                          int32_t* guesses, float* guess_q, void* workspace,
                          size_t workspace_bytes, int32_t* dev_status, void* stream);

/* ---------------------------------------------------------------------------
 * ssd_saguaro_sample -- one continuation step of the SSD cache build: every
 * branch row draws its next draft token from the Saguaro distribution.
 * [SSD-note] §"Saguaro 优化二：Saguaro 采样" and §"实现细节：缓存怎么建"; the
 * fan-out of a branch row is that of the outcome position it continues
 * (§"最优扇出度分配"), so it is given per row.
 *
 * For branch row r (0 <= r < R) with F = F_row[r]:
 *   S = top-F of z[r,:];  q' = Saguaro(softmax(z[r,:]/T), S, C);
 *   x = smallest y with sum_{y'<=y} q'(y') > u * sum(q'),
 *       u = U(seeds[r]; r, j, 2, round);
 *   guesses = top-(F+1) of z[r,:] minus x, truncated to F.
 *
 * draft       [R, V] logits.
 * T           temperature, finite and > 0.
 * C           Saguaro factor in (0, 1] (the factor of position j when the
 *             caller uses one per position).
 * F_row       device [R] int32 cached-set size / guesses per row, each in
 *             [0, Fmax] (a value outside is clamped and sets
 *             SSD_DEV_BAD_FANOUT), or NULL: F = Fmax for every row.
 * Fmax        0..SSD_MAX_F, Fmax + 1 <= V: the largest F and the column
 *             count of out_guess.
 * seeds       device [R] uint64.   j: continuation position (counter word).
 * out_token   device [R] int32 out.
 * out_qprime  device [R] float out (or NULL): q'(x).
 * out_guess   device [R, Fmax] int32 out (or NULL), -1 padded.
 * ------------------------------------------------------------------------- */
size_t ssd_saguaro_workspace_size(int R, int V);
ssd_status ssd_saguaro_sample(const ssd_logits* draft, int R, int V, float T, float C,
                              const int32_t* F_row, int Fmax, const uint64_t* seeds, int j,
                              uint32_t round, int32_t* out_token, float* out_qprime,
                              int32_t* out_guess, void* workspace, size_t workspace_bytes,
                              int32_t* dev_status, void* stream);

/* ---------------------------------------------------------------------------
 * ssd_tree_verify -- verification of tree-shaped drafts.  [SD-7.3] §7.3.9
 * item 3 (树形草稿: several candidate continuations per position instead of
 * one chain); the pages give no algorithm, and the per-token rule of §7.3.3
 * is applied to each candidate in turn (multi-candidate rejection sampling):
 *
 * The tree has N nodes, the same for the whole batch: node 0 is the last
 * verified position, node u >= 1 has parent parent[u] < u and holds draft
 * token tokens[b, u], drawn from the draft distribution q_{parent(u)} of its
 * parent.  Target row u of tree b is p_u, the target distribution after node
 * u's path; draft row u is q_u.  For tree b:
 *   u = 0, r = p_0 = softmax(z_target[b,0,:] / T);
 *   for each child v of u in increasing index order:
 *     accept x_v iff U(seeds[b]; b, v-1, 0, round) < r(x_v) / q_u(x_v):
 *       then u = v, r = p_v, and continue with v's children;
 *     else r = (r - q_u)^+ / sum (r - q_u)^+;
 *   when no child of u is accepted (or u is a leaf): bonus t = smallest y
 *   with sum_{y'<=y} r(y') > U(seeds[b]; b, u, 1, round) * sum(r).
 * A chain (parent[u] = u - 1) gives ssd_verify's results with C = 1, F = 0
 * (accept_len, bonus; drafts drawn with counter (b, v-1, 2, round)).
 *
 * target, draft  [B, N, V] logits, same dtype: row (b, u) is row b*N + u.
 * parent      HOST [N] int32: parent[0] = -1, 0 <= parent[u] < u.
 * tokens      device [B, N] int32 (entry 0 of a tree is ignored).
 * accept_len  device [B] int32 out: depth of the last accepted node.
 * path        device [B, Dmax] int32 out (or NULL): the accepted nodes, -1
 *             padded; Dmax >= the tree's depth.
 * bonus       device [B] int32 out.
 * resid_mass  device [B] float out (or NULL): sum (r - q_u)^+ of the last
 *             rejection at the final node, 1 when it rejected nothing.
 * T           temperature, finite and > 0.   N <= 256.
 * workspace   >= ssd_tree_workspace_size(B, N, V), 256-byte aligned.
 * Two launches on `stream`: the streaming pass normalises every row, then
 * one thread-block cluster per tree walks it: its CTAs share the tree's row
 * passes; 8 CTAs, halved while B times the cluster size exceeds the SM
 * count (one CTA per tree when B does).
 * ------------------------------------------------------------------------- */
size_t ssd_tree_workspace_size(int B, int N, int V);
ssd_status ssd_tree_verify(const ssd_logits* target, const ssd_logits* draft, int B, int N, int V,
                           float T, const int32_t* parent, const int32_t* tokens,
                           const uint64_t* seeds, uint32_t round, int32_t* accept_len,
                           int32_t* path, int Dmax, int32_t* bonus, float* resid_mass,
                           void* workspace, size_t workspace_bytes, int32_t* dev_status,
                           void* stream);

/* ---------------------------------------------------------------------------
 * Outcome cache.  [SSD-note] §"SSD 的核心思想": the verification outcome is the
 * pair (k accepted, bonus t); the drafter keeps a continuation per predicted
 * outcome.  Keys are (row, k, t), values are branch ids.
 *
 * The table is an open-addressed hash table of 16-byte slots (64-bit packed
 * key, 32-bit value) with a power-of-two capacity >= 2 n; probing is linear
 * and bounded by the capacity, so a full table can never loop.
 *
 * ssd_cache_bytes(n)  bytes of a table for n keys.
 * ssd_cache_build     clears the table and inserts n keys row[i], k[i], t[i]
 *                     -> branch[i] (all device [n] int32).  Duplicate keys set
 *                     SSD_DEV_DUPLICATE_KEY (the first value is kept).
 * ssd_cache_build_guesses  clears and inserts every non-negative guess
 *                     g = guesses[b, k, f] of a [B, Kq, Fmax] table as key
 *                     (b, k, g) -> branch (b*Kq + k)*Fmax + f.
 * ssd_cache_lookup    out_branch[b] = value of key (b, accept_len[b], bonus[b])
 *                     or -1; *all_hit = 1 if every row hit, else 0 (device
 *                     int32).  [SSD-note] §"Saguaro 优化三": a batch proceeds
 *                     without waiting only if every sequence hits.
 * ------------------------------------------------------------------------- */
size_t ssd_cache_bytes(int n_keys);
ssd_status ssd_cache_build(void* table, size_t table_bytes, const int32_t* row, const int32_t* k,
                           const int32_t* t, const int32_t* branch, int n, int32_t* dev_status,
                           void* stream);
ssd_status ssd_cache_build_guesses(void* table, size_t table_bytes, const int32_t* guesses, int B,
                                   int Kq, int Fmax, int32_t* dev_status, void* stream);
ssd_status ssd_cache_lookup(const void* table, size_t table_bytes, const int32_t* accept_len,
                            const int32_t* bonus, int B, int32_t* out_branch, int32_t* all_hit,
                            void* stream);

/* ---------------------------------------------------------------------------
 * ssd_fanout -- geometric fan-out (host only, no device work).
 * [SSD-note] §"最优扇出度分配": with acceptance P(k) ~ a^k and a per-position
 * miss rate falling as F_k^-r, the Lagrange optimum under sum F_k = budget is
 * F_k ~ a^(k/(1+r)).  Real-valued shares budget * w_k / sum(w) are rounded
 * down, then the remaining units go to the largest fractional parts (ties to
 * the lower k).
 * F_out HOST [K+1] int32 out.  K >= 0, budget >= 0, a > 0, r >= 0.
 * ------------------------------------------------------------------------- */
ssd_status ssd_fanout(int K, int budget, double a, double r, int32_t* F_out);

/* ---------------------------------------------------------------------------
 * ssd_process_logits -- penalties for repeated tokens, biases and grammar
 * masks on the logit rows of a round, before they are verified or sampled.
 * The pages have no counterpart: a serving setting, as T = 0 is.
 *
 * Sequence b has N rows: row 0 follows its last verified token, row u > 0
 * the drafts on the path to node u (a chain of drafts: u - 1, ..., 1).  For
 * token v of row (b, u), with
 *   c    = how often v occurs in history[b, prompt_len[b] .. history_len[b])
 *          and among the drafts on the path to u,
 *   seen = c > 0, or v occurs in history[b, 0 .. prompt_len[b]):
 *   z = in[b, u, v];
 *   if seen:   z = z > 0 ? z / repetition[b] : z * repetition[b];
 *   if c > 0:  z = z - frequency[b] * c - presence[b];
 *   if v is in bias_ids[b, :]:  z = z + its bias;
 *   if the grammar does not allow v:  z = fill;
 *   out[b, u, v] = z, computed in float32 and rounded once to the row type.
 * The grammar overrides every other rule, NaN logits included.
 *
 * in, out      [B, N, V] logits of one dtype, row (b, u) is row b*N + u; out
 *              is in itself (same pointer and row stride) or does not overlap
 *              it.
 * history      device int32, sequence b's tokens start at b * history_stride,
 *              with room for history_max (those past its length are not used;
 *              NULL: no history).  A token outside [0, V) is passed over
 *              and sets SSD_DEV_BAD_TOKEN.
 * history_len  device [B] int32 in [0, history_max] (a value outside is
 *              clamped and sets SSD_DEV_BAD_LENGTH).
 * prompt_len   device [B] int32, or NULL: 0 (every token counts).
 * draft_tokens device int32: the token of node u >= 1 is
 *              draft_tokens[b * draft_stride + u - 1] (or NULL: drafts do not
 *              count).  Tokens outside [0, V): as for history.
 * parent       HOST [N] int32 as in ssd_tree_verify, or NULL for a chain.
 * repetition, frequency, presence   device [B] float, or NULL for none.
 *              A value not finite, or a repetition <= 0, is left out and sets
 *              SSD_DEV_BAD_PENALTY.
 * bias_ids, bias  device [B, n_bias] (or NULL with n_bias = 0), n_bias <=
 *              65535.  A negative id is padding, one >= V is passed over and
 *              sets SSD_DEV_BAD_TOKEN; of a token listed twice the later
 *              entry holds.
 * mask         device int32 words, or NULL: bit v % 32 of word
 *              mask[b * mask_seq_stride + u * mask_row_stride + v / 32] says
 *              whether v is allowed (strides of 0 share a mask).
 * fill         the value of tokens that are not allowed (rounded to the row
 *              type), not NaN.  For
 *              ssd_verify it must be finite: SSD_MASKED_LOGIT is exact in
 *              every type and far below any logit.  A row that allows nothing
 *              is fill throughout.
 * allowed      device [B, N] int32 out (or NULL): how many tokens of the row
 *              the grammar allows; 0 shows a dead end.
 * N <= 256.  One launch, no workspace.
 * ------------------------------------------------------------------------- */
#define SSD_MASKED_LOGIT (-1048576.0f) /* -2^20 */
typedef struct {
  const int32_t* history;
  int64_t history_stride;
  int32_t history_max;
  int32_t n_bias;
  const int32_t* history_len;
  const int32_t* prompt_len;
  const int32_t* draft_tokens;
  int64_t draft_stride;
  const int32_t* parent; /* host */
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_ids;
  const float* bias;
  const int32_t* mask;
  int64_t mask_seq_stride;
  int64_t mask_row_stride;
  float fill;
  int32_t pad_; /* must be 0 */
} ssd_logit_rules;
ssd_status ssd_process_logits(const ssd_logits* in, const ssd_logits* out, int B, int N, int V,
                              const ssd_logit_rules* rules, int32_t* allowed,
                              int32_t* dev_status, void* stream);

/* ---------------------------------------------------------------------------
 * ssd_page_plan -- the pages of a paged key/value cache after a round, and
 * the slots of the tokens that come next.  [SD-blog]'s rollback after a
 * rejection is a matter of lengths here: the pages of rejected drafts are
 * kept for the next drafts, or go back.
 *
 * Request b has lens[b] tokens in the cache, will append new_tokens[b], and
 * holds the pages tables[b, 0 .. held[b]).  need = ceil((lens + new) / page).
 *   1. Every request with held > need gives back tables[b, need .. held): in
 *      the order of b and of columns they are pushed on the stack of free
 *      pages, free_pages[0 .. *free_count), whose top is its end.
 *   2. In the order of b, every request with held < need takes need - held
 *      pages from the top, into tables[b, held .. need).  A request whose
 *      pages are more than are left takes none, and neither does any later
 *      request that needs one (SSD_DEV_NO_PAGES): served[b] = 0.
 *   3. Its tokens stand in rows cu[b] .. cu[b + 1) of the batch's new tokens
 *      (cu: running sums of new_tokens): row cu[b] + i has owner b, position
 *      lens[b] + i and slot tables[b, position / page] * page + position %
 *      page (-1 when b was not served).
 * The inputs are left as they are but for the entries of tables and
 * free_pages named above, so a call repeated on the same inputs gives the
 * same results; the next round passes kv_len (less the tokens rejected),
 * held_out and free_out.
 * A request is not served, and SSD_DEV_BAD_LENGTH set, when lens, new or held
 * are negative, held > cols, lens + new > cols * page, or held pages do not
 * hold lens tokens; it keeps its pages and has no rows.
 *
 * Outputs are not inputs, but arrays of their own (SSD_ERR_INVALID_ARG where
 * an output has an input's address).
 *
 * lens, new_tokens, held  device [B] int32.  B <= 8192; B * cols and max_rows
 *             at most 2^30.
 * tables      device int32, request b's row starts at b * table_stride, cols
 *             columns.
 * free_pages  device [free_cap] int32; free_count device int32 in [0,
 *             free_cap] (clamped otherwise, SSD_DEV_BAD_LENGTH).  Pages given
 *             back may pass the array's end where the same call takes them
 *             again; those that do not fit it after step 2 are lost, and set
 *             SSD_DEV_BAD_LENGTH.
 * slots       device [max_rows] int64 out; positions, owner [max_rows] int32
 *             out (each may be NULL).  Rows past the last token are -1; tokens
 *             past max_rows have no row, and set SSD_DEV_BAD_LENGTH.
 * cu          device [B + 1] int32 out; kv_len (lens + new if served, else
 *             lens), held_out, served device [B] int32 out; free_out device
 *             int32 out.
 * One launch, no workspace.
 * ------------------------------------------------------------------------- */
ssd_status ssd_page_plan(const int32_t* lens, const int32_t* new_tokens, const int32_t* held, int B,
                         int32_t* tables, int64_t table_stride, int cols, int32_t* free_pages,
                         int free_cap, const int32_t* free_count, int page, int max_rows,
                         int64_t* slots, int32_t* positions, int32_t* owner, int32_t* cu,
                         int32_t* kv_len, int32_t* held_out, int32_t* served, int32_t* free_out,
                         int32_t* dev_status, void* stream);

/* ---------------------------------------------------------------------------
 * ssd_prefix_attention -- attention of one query token per row over a paged
 * cache, for rows that share prefixes: every group of rows reads its prefix
 * once, and every row its own tokens after it.  [SSD-note] §"实现细节：缓存怎么建",
 * §"两层 batch": the branches of a sequence (one per predicted outcome) are
 * rows of one drafter batch, over the same prefix.
 *
 * Row r of group g (group_off[g] <= r < group_off[g + 1]) attends to the
 * first prefix_len[g] tokens of pages prefix_tables[g, :] and the first
 * lens[r] tokens of pages tables[r, :].  With s_j = scale * q . k_j over all
 * of them, per query head, query head i reading key/value head i / (Hq/Hkv):
 *   lse = log sum_j exp(s_j);   out = sum_j exp(s_j - lse) v_j.
 * A row with no token at all, or of no group and no own token, gives out = 0
 * and lse = -inf.  Several tokens of one branch are several rows over the
 * same table, each with its own lens.
 *
 * q, out      [R, Hq, D] of dtype (SSD_BF16 or SSD_F16); D elements are
 *             contiguous, strides are in elements and multiples of 8, bases
 *             16-byte aligned.  D: 64, 128 or 256.  Hkv divides Hq.  out is q
 *             itself (same pointer and strides) or does not overlap it, nor k
 *             and v.
 * k, v        [num_pages, page_size, Hkv, D] of dtype, strides and bases as
 *             for q, any order of the first three dimensions.  Bytes of a
 *             page past the last token are not used, whatever they hold.
 * prefix_tables, tables  device int32 page ids, rows of prefix_cols / cols
 *             columns (of none: NULL too).  An id outside [0, num_pages) of a
 *             token that is read sets SSD_DEV_BAD_PAGE; the token reads as
 *             zeros.
 * prefix_len  device [G] int32 in [0, prefix_cols * page_size]; lens device
 *             [R] int32 in [0, cols * page_size] (NULL tables and lens: no
 *             own tokens, whatever cols).  Values outside are clamped and set
 *             SSD_DEV_BAD_LENGTH.  Tables of 2^31 - 2^20 tokens or more, and as
 *             many (row, head) pairs, are SSD_ERR_UNSUPPORTED.
 * group_off   device [G + 1] int32, not falling, within [0, R]; otherwise
 *             SSD_DEV_BAD_LENGTH is set and the rows concerned are undefined.
 * lse         device [R, Hq] float out (or NULL).
 * workspace   256-byte aligned, >= ssd_prefix_attention_workspace_size of the
 *             same descriptor.
 * Scores, their maxima and sums and the outputs' sums are held in float32;
 * the weights exp(s_j - max) are rounded to dtype for the matrix product.
 * ------------------------------------------------------------------------- */
typedef struct {
  const void* ptr;
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
} ssd_paged;
typedef struct {
  int32_t dtype; /* ssd_dtype */
  int32_t R, Hq, Hkv, D;
  int32_t G;
  int32_t num_pages, page_size;
  const void* q;
  int64_t q_row_stride, q_head_stride;
  ssd_paged k, v;
  const int32_t* prefix_tables;
  const int32_t* prefix_len;
  const int32_t* group_off;
  const int32_t* tables;
  const int32_t* lens;
  int64_t prefix_table_stride, table_stride;
  int32_t prefix_cols, cols;
  void* out;
  int64_t out_row_stride, out_head_stride;
  float* lse;
  float scale;
  int32_t pad_; /* must be 0 */
} ssd_attention;
size_t ssd_prefix_attention_workspace_size(const ssd_attention* a);
ssd_status ssd_prefix_attention(const ssd_attention* a, void* workspace, size_t workspace_bytes,
                                int32_t* dev_status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SSD_H */
