/*
 * attn.h -- C-ABI of libattn.so, a GB300 (sm_103a) fused attention forward.
 *
 * The operation.  For every batch b, query head hq and query row i:
 *
 *     O[b,hq,i,:] = sum_j softmax_j( scale * <Q[b,hq,i,:], K[b,hkv,j,:]> + mask(i,j) ) V[b,hkv,j,:]
 *     LSE[b,hq,i] = ln sum_{kept j} exp( scale * <Q[b,hq,i,:], K[b,hkv,j,:]> )
 *
 * with hkv = hq / (Hq / Hkv) (grouped-query attention: contiguous groups of
 * query heads share one key/value head), computed tile by tile with a running
 * max and running sum so the S x S score matrix never reaches memory.  This is
 * the FlashAttention scheme the page "NVIDIA让AI狂肝7天自己写算子"
 * (yetianai.com/news/16520) describes in its FlashAttention-lineage section
 * (block-wise computation that never stores the full attention matrix); the
 * masks and the score scaling follow the page "Opus 4.6 + AutoResearch驱动25轮
 * 迭代..." (yunpan.plus/t/19526-1-1), code excerpt "Apply mask + scale
 * in-register"; causal and non-causal prefill and GQA are the workloads of the
 * benchmark section of the first page named above.
 *
 * mask(i,j) is 0 for a kept entry and -inf for a masked one.  Entry (i,j) is
 * kept when (causal == 0 || j <= i) and (mask_bits == NULL || bit j%32 of word
 * mask_bits[b][i][j/32] is 1).  A row with no kept entry is defined as O = 0
 * and LSE = -inf.
 *
 * Conventions for every entry point:
 *   - q, o:   [B][Hq][S][d] row-major, contiguous, device memory, 16-byte aligned.
 *   - k, v:   [B][Hkv][S][d] row-major, contiguous, device memory, 16-byte aligned.
 *   - lse:    float [B][Hq][S], device memory, natural log; may be NULL (not written).
 *   - mask_bits: uint32 [B][S][ceil(S/32)], device memory, 4-byte aligned, least-
 *             significant bit first, 1 = attend, shared by all heads of a batch
 *             entry; bits past column S-1 are ignored.  NULL = no custom mask.
 *   - d in {64, 128}; Hq % Hkv == 0; B, Hq, Hkv, S >= 1; scale > 0 and finite.
 *   - dtype: ATTN_F16 or ATTN_BF16 (q, k, v and o share it); accumulation is fp32.
 *   - stream: a cudaStream_t (NULL = the legacy default stream).
 *   - Ownership: the caller owns every buffer; the library keeps no pointer to
 *     them after the call returns.  The library's own state is small and cached:
 *     tensor maps (TMA descriptors) keyed by buffer address, shape and tile box,
 *     reused by later calls on the same buffers (a map holds only these, so a
 *     cached one stays valid); a status word per (device, stream); and, per
 *     (device, stream) that has run a custom mask, one workspace.  Without a
 *     custom mask nothing is allocated.  With one, a pre-pass kernel writes the
 *     kept-bit words (mask AND causal AND the key bound, padded to whole
 *     128-column tiles; when no bound applies, the key count is a multiple of
 *     128 and mask_bits is 16-byte aligned those equal mask_bits, which the
 *     attention kernel then reads in place) and an emptiness map per (16-row
 *     block, 128-column tile),
 *     and a compaction kernel lists, per mask row block, the 16-row blocks that
 *     keep anything: the attention kernel computes only those, packed eight to a
 *     128-row tile, and writes O = 0, LSE = -inf for the rows of the others
 *     without computing them.  That output lives in the stream's workspace, of at
 *     least the "custom-mask scratch size": with nm mask row blocks (B, or B*Hq
 *     for per-head masks), R = ceil(Sq/16), T = ceil(Sq/128), U = ceil(Sq/256)
 *     and N = ceil(Sk/128), the sum of nm*Sq*N*16, nm*R*N, nm*R, nm*U*64 and
 *     nm*T*N bytes, each rounded up to a multiple of 256 (Sq = Sk = S for
 *     attn_fwd).  The workspace is a stream-ordered allocation (cudaMallocAsync
 *     on `stream`, whole MiB) made by the first custom-mask call on the stream
 *     and reused by every later one; a call that needs more frees the old block
 *     in stream order (cudaFreeAsync) and allocates a larger one.  Repeated calls
 *     of one shape therefore allocate nothing after the first.  Variable-length
 *     batches (attn_fwd_ex with per-entry lengths or packed offsets) use the same
 *     workspace for their work order, B*ceil(max Sq/256) ints after the mask
 *     scratch (256-byte aligned), and so does attn_fwd_paged without a workspace of the caller's.
 *     The workspace is held until
 *     attn_release_workspace(stream) or process exit: release it before
 *     destroying a stream that has run custom masks, variable-length batches or paged attention.
 *   - Captured calls: attn_fwd and attn_fwd_ex may be captured into a graph.  A captured call goes on using what the
 *     library keeps for the stream it was captured on (its work queue, and its workspace where that was large
 *     enough at the time; otherwise the graph allocates its own): its replays, replays of other graphs captured on
 *     that stream and calls on the stream take their turns, none at the same time as another.  The workspace
 *     a graph works in is not freed when a later call needs more, only by attn_release_workspace:
 *     call that when the graphs are done with.  attn_fwd_paged differs (see there): its replays may run beside anything.
 *   - Errors: arguments are validated before any launch (ATTN_ERR_INVALID /
 *     ATTN_ERR_UNSUPPORTED, nothing launched); a failed launch returns
 *     ATTN_ERR_CUDA.  The work is asynchronous: a kernel that gives up on a
 *     barrier wait (see attn_set_wait_timeout_ns) records ATTN_ERR_TIMEOUT in
 *     the status word of the stream it was launched on, which attn_check(that
 *     stream) reports.  The library never traps and never exits the process.
 *   - Thread safety: calls on different streams may run concurrently, and so may
 *     host threads calling on one stream (the library's caches are guarded by
 *     mutexes), except attn_fwd_noalloc with a custom mask: its calls share one
 *     fixed array and must not overlap on the GPU (see below).
 */
#ifndef ATTN_H
#define ATTN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ATTN_F16 = 0, ATTN_BF16 = 1 } attn_dtype_t;

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID = -1,     /* a null pointer, a non-positive size, misalignment, bad scale */
    ATTN_ERR_UNSUPPORTED = -2, /* a head dim or dtype the library has no kernel for */
    ATTN_ERR_CUDA = -3,        /* a CUDA runtime/driver call failed (launch, tensor map, memory) */
    ATTN_ERR_TIMEOUT = -4,     /* a kernel barrier wait ran out of time; outputs undefined */
    ATTN_ERR_DEVICE = -5,      /* no usable sm_103 device */
    ATTN_ERR_PAGE = -6         /* a kernel met a page id, slot, page count or parent out of range */
} attn_status_t;

/*
 * attn_fwd -- the fused forward pass described above, launched on `stream`.
 * Returns ATTN_OK once the kernel is enqueued.
 */
int attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
             const uint32_t *mask_bits, int B, int Hq, int Hkv, int S, int d, int causal,
             float scale, int dtype, void *stream);

/*
 * attn_fwd_ex -- the same computation with the generalisations a prefill against a
 * key/value cache and local attention need (the pages themselves stop at Sq = Sk and the
 * masks above; these follow the same tile, bit-word and skip path):
 *   - Sq query rows against Sk >= Sq keys, aligned at the bottom right: query i sits at
 *     key position pos(i) = i + Sk - Sq.  q, o: [B][Hq][Sq][d]; k, v: [B][Hkv][Sk][d];
 *     lse: [B][Hq][Sq].
 *   - a band of kept keys: pos(i) - window_left <= j <= pos(i) + window_right
 *     (-1 = unbounded on that side); causal = 1 keeps j <= pos(i) (window_right is then
 *     treated as 0).
 *   - custom masks of [B][Sq][ceil(Sk/32)] words (mask_per_head = 0) or
 *     [B][Hq][Sq][ceil(Sk/32)] (mask_per_head = 1), ANDed with the band.
 *   - visited: as for attn_fwd_visited (nqt = ceil(Sq/bm), nkt = ceil(Sk/bn)), or NULL.
 *   - variable-length batches: seqlens_q / seqlens_k, int32 [B] in device memory (4-byte
 *     aligned) or NULL (= Sq / Sk for every entry), give batch entry b its own lengths
 *     sq_b <= Sq and sk_b <= Sk inside the padded buffers above (values outside [0, Sq] /
 *     [0, Sk] are clamped).  Entry b's query i sits at key position i + sk_b - sq_b, only
 *     keys j < sk_b exist, and rows i >= sq_b of o and lse are not written.  Key rows at or
 *     past sk_b get weight exactly 0, so v must hold finite values there (0 * inf is NaN);
 *     k there may hold anything.  The custom-mask layout keeps the padded shape.
 *   - packed variable-length batches: cu_seqlens_q / cu_seqlens_k, int32 [B+1] in device
 *     memory (4-byte aligned, non-decreasing, cu[0] = 0), or NULL.  When given, entry b is
 *     query rows cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 and key rows cu_seqlens_k[b] ..
 *     cu_seqlens_k[b+1]-1 of head-major packed buffers: q, o: [Hq][Sq][d], k, v:
 *     [Hkv][Sk][d], lse: [Hq][Sq], with Sq / Sk the total row counts; max_seqlen_q /
 *     max_seqlen_k (>= 1) bound every entry's lengths (longer entries are cut to them).
 *     Alignment, causal and window rules are per entry as above; visited is
 *     [B][Hq][ceil(max_seqlen_q/bm)][ceil(max_seqlen_k/bn)].  Custom masks are not supported
 *     with packed layouts (ATTN_ERR_UNSUPPORTED); seqlens_q / seqlens_k must then be NULL.
 * With Sq = Sk = S, windows -1, mask_per_head = 0 and no lengths it is attn_fwd.  Custom masks take
 * stream-ordered scratch of the custom-mask scratch size above.  Errors as for attn_fwd;
 * Sk < Sq is ATTN_ERR_INVALID for padded layouts.
 */
typedef struct {
    const void *q, *k, *v;
    void *o;
    float *lse;
    const uint32_t *mask_bits;
    int mask_per_head;
    int B, Hq, Hkv, Sq, Sk, d;
    int causal, window_left, window_right;
    float scale;
    int dtype;
    void *stream;
    uint8_t *visited;
    const int *seqlens_q, *seqlens_k;
    const int *cu_seqlens_q, *cu_seqlens_k;
    int max_seqlen_q, max_seqlen_k;
} attn_fwd_params_t;

int attn_fwd_ex(const attn_fwd_params_t *params);

/*
 * attn_fwd_visited -- attn_fwd that also records which (query tile, key tile)
 * blocks it computed: visited[((b*Hq + hq)*nqt + qt)*nkt + kt] = 1, uint8,
 * device memory, nqt = ceil(S/bm), nkt = ceil(S/bn) with (bm, bn) from
 * attn_tile_shape.  The caller zeroes `visited`.  Blocks that hold no kept
 * entry -- every mask word over the block is zero, or the block lies above the
 * causal diagonal -- are skipped, following the tile-skip ballot of the page
 * "Opus 4.6 + AutoResearch驱动25轮迭代..." (first code excerpt).  With a custom mask
 * qt numbers the compacted query tiles instead: tile qt holds the 16-row blocks
 * 8*qt .. 8*qt+7 of the ascending list of blocks that keep anything (of batch
 * entry b, or of head (b, hq) for per-head masks).  O and LSE are identical to
 * attn_fwd's.
 */
int attn_fwd_visited(const void *q, const void *k, const void *v, void *o, float *lse,
                     const uint32_t *mask_bits, int B, int Hq, int Hkv, int S, int d,
                     int causal, float scale, int dtype, void *stream, uint8_t *visited);

/*
 * attn_fwd_noalloc -- attn_fwd for callers that must not allocate device memory:
 * code running where cudaMalloc / cudaMallocAsync are unavailable or forbidden,
 * e.g. inside a custom allocator or memory-pool hook (re-entering the allocator
 * would deadlock or recurse), in real-time paths that may not wait on the
 * allocator, or in hosts that hand out a fixed memory budget up front.  It takes
 * the same arguments and computes the same result as attn_fwd.  Without a custom
 * mask the two are the same call.  With one, the mask pre-pass output goes into a
 * fixed device array of ATTN_NOALLOC_SCRATCH_BYTES that this library reserves on
 * every GPU that loads it, held until the process exits, instead of into
 * stream-ordered scratch; calls whose custom-mask scratch size (see the
 * conventions above) exceeds it return ATTN_ERR_INVALID before any launch.
 * Every call looks the array's device address up with the caller's device
 * current (a cheap host call, so a reset or replaced context never sees a stale
 * address); the first call on a device also loads the library's device code
 * there, so make it before any stream capture.  Every call shares the one array
 * and it keeps the last call's contents (each call rewrites every byte it then
 * reads, so nothing needs clearing); calls whose work overlaps on the GPU -- on
 * different streams, say -- race on it, so order them.  It makes no host-side
 * allocation either: on a stream that attn_fwd has not used, its timeout status
 * goes to the status word shared by such streams, which attn_check reports for
 * any of them.  The pages this library follows have no counterpart of this
 * entry point.
 */
#define ATTN_NOALLOC_SCRATCH_BYTES (4u << 20)
int attn_fwd_noalloc(const void *q, const void *k, const void *v, void *o, float *lse,
                     const uint32_t *mask_bits, int B, int Hq, int Hkv, int S, int d, int causal,
                     float scale, int dtype, void *stream);

/*
 * ---------------------------------------------------------------- paged key/value cache
 *
 * A serving step over a cache whose keys and values live in pages: attn_paged_tables turns
 * the requests' lengths into block tables and a slot map, attn_paged_append writes the
 * step's new key / value rows to their slots, and attn_fwd_paged attends from the step's
 * query rows (one token per request, a few, or whole chunks, mixed freely) over the cache.
 *
 * Layout.  k_cache, v_cache: num_pages pages of page_size rows for Hkv heads of d elements.
 * Element (page, h, row, x) is at page*cache_page_stride + h*cache_head_stride +
 * row*cache_row_stride + x (in elements, the same strides for k and v), so pages may hold
 * their heads one after the other ([num_pages][Hkv][page_size][d]) or their rows one after
 * the other ([num_pages][page_size][Hkv][d]), inside larger buffers or not.  New rows, q and
 * o are packed, request after request, with a row and a head stride of their own.  Strides
 * are multiples of 8, not negative (those of a cache's dimensions of more than one entry
 * positive) and at most 2^38, pointers to rows 16-byte aligned; page_size is a multiple of 16.  No output of a
 * call overlaps an input of it, unless said so.
 * Slot s is row s % page_size of page s / page_size.
 * block_table: int32, row b at block_table + b*table_stride, table_width entries: request
 * b's token at position p is in page block_table[b][p / page_size], row p % page_size.
 *
 * All lengths, tables and slots are read on the device, in stream order, so a captured
 * sequence of these calls can be replayed after the arrays' contents changed.  The calls
 * keep no state between them.  Index arrays are int32, 4-byte aligned, device memory.
 * Bad values in them fault nothing: a page id outside [0, num_pages), a slot at or past
 * num_pages*page_size, a free list that runs out or, in attn_paged_tables, a table that is too narrow is
 * left out as described with each call, and recorded as ATTN_ERR_PAGE in the stream's status word,
 * which attn_check(stream) reports.
 */

/*
 * attn_paged_tables -- block tables, slot map, positions and row offsets of a step.
 * Request b has ctx_lens[b] tokens in the cache and brings new_lens[b] more (0: idle;
 * negative lengths count as 0).  Pages that it lacks for ctx + new tokens come from the end
 * of the free list: free_pages[0 .. *free_count - 1] are free, the first page that is handed
 * out is the last of them, requests are served in ascending order, each request's pages
 * likewise, and *free_count_out (which may be free_count itself) is what is left.
 * Writes
 *   block_table[b][i], only for the pages added, i = ceil(ctx/page_size) ..
 *                      ceil((ctx+new)/page_size) - 1 (the others are kept);
 *   cu_seqlens_q[0..B]: offsets of the requests' new rows; seqlens_k[b] = ctx + new;
 *   slots[t], positions[t] (or NULL) for t < max_rows: the slot and the position of new row
 *                      t, -1 behind the last one.
 * When pages run out, when a table row is too narrow, or when a page id (of the free list or
 * of the page that request b's new tokens start in) is out of range, the slots concerned
 * are -1 and so are the table entries that exist; rows past max_rows get no slot.  Each of these
 * sets ATTN_ERR_PAGE.  cu_seqlens_q and seqlens_k are as if all had been well; *free_count_out
 * is never below 0.  With max_free = 0 free_pages may be NULL; with max_rows = 0 (a step without new
 * rows) slots and positions are.  1 <= B <= 16384, max_rows <= 2^30; num_pages*page_size, and the sums of the lengths, fit 31 bits.
 */
typedef struct {
    const int *ctx_lens, *new_lens; /* [B] */
    int *block_table;               /* in / out */
    const int *free_pages;          /* [max_free]; may be NULL if that is 0 */
    const int *free_count;          /* [1], at most max_free (more is cut) */
    int *free_count_out;            /* [1] */
    int *cu_seqlens_q;              /* [B+1] */
    int *seqlens_k;                 /* [B] */
    int *slots, *positions;         /* [max_rows]; positions may be NULL */
    int B, table_width, table_stride, max_free, max_rows, page_size, num_pages;
    void *stream;
} attn_paged_tables_params_t;

int attn_paged_tables(const attn_paged_tables_params_t *params);

/*
 * attn_paged_append -- write new key and value rows into the cache: row t of head h goes to
 * slot slots[t].  A negative slot leaves row t out (rows behind the last request, as
 * attn_paged_tables marks them); one at or past num_pages*page_size too, with ATTN_ERR_PAGE.
 * Slots are distinct (the rows of a slot that is named twice would overwrite each other in
 * no particular order).  k_new, v_new: element (h, t, x) at h*head + t*row + x of their own
 * strides; they do not overlap the cache.  rows <= 2^30; num_pages*page_size fits 31 bits.
 */
typedef struct {
    const void *k_new, *v_new;
    void *k_cache, *v_cache;
    const int *slots; /* [rows] */
    long long k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    long long cache_page_stride, cache_head_stride, cache_row_stride;
    int rows, Hkv, d, num_pages, page_size, dtype;
    void *stream;
} attn_paged_append_params_t;

int attn_paged_append(const attn_paged_append_params_t *params);

/*
 * attn_fwd_paged -- attention of packed query rows over the paged cache.  Request b's query
 * rows are cu_seqlens_q[b] .. cu_seqlens_q[b+1]-1 of q, o and lse (offsets non-decreasing,
 * cu_seqlens_q[0] >= 0; rows past total_q are not touched); its keys are its first
 * seqlens_k[b] cache rows (cut to [0, table_width*page_size]), the query rows' own among them
 * where they have been appended.  Query i of a request with sq rows and sk keys sits at key
 * position i + sk - sq; causal, window_left and window_right as for attn_fwd_ex, with sk < sq
 * allowed (rows without a key give O = 0, LSE = -inf).  Requests longer than max_seqlen_q
 * (>= 1) are cut to their first max_seqlen_q rows.  Neither cut is reported, and positions go by the lengths
 * after it: keep lengths within both bounds, in replays of a captured call as well.  Rows of q, o and lse
 * outside every request are neither read into a result nor written.
 * Roundings: scores, softmax and sums in 32 bits, O rounded once.  The weights go into the product with V in the type
 * of q, as in attn_fwd (each off by half a step at most).  Where max_seqlen_q * Hq / Hkv <= 16 (32 at d = 64) they
 * keep twice the bits, and so they may for requests of few rows in other calls: the last bits of such a
 * request can depend on what it is batched with.
 * The host does not see the lengths: which kernels serve a call goes by the rows of q, B and max_seqlen_q, so a call with
 * much more room than its requests use is slower than one that fits.
 * Element (hq, t, x) of q is at t*q_row_stride + hq*q_head_stride + x, of o likewise with its own
 * strides; lse is [Hq][total_q] or NULL.  Hq / Hkv <= 128, B <= 16384, total_q * Hq < 2^31 - 2^27.  Strides of dimensions of more
 * than one entry are positive, and of the caches' page and head strides one is a multiple of the
 * other (else ATTN_ERR_UNSUPPORTED).
 * Cache rows that no query row of the request may see, behind its last key, ahead of its
 * window, or on pages listed for none of its keys, may hold anything; those that one of its query
 * rows sees hold finite values.  A page id out of range sets ATTN_ERR_PAGE; its keys then count as
 * zeros.
 * workspace: NULL, or device memory, 256-byte aligned, of at least the size that
 * attn_paged_workspace gives for the same parameters; its contents are of no account before and
 * after the call, and calls that may run at the same time (two captured graphs among them) each
 * take their own.  With NULL the call uses the stream's workspace (see the conventions), which
 * later calls on the stream share in stream order; a call that is being captured into a graph
 * brings its own, and so does one on cudaStreamPerThread, one handle for a stream of every thread
 * (NULL is ATTN_ERR_INVALID there).
 */
typedef struct {
    const void *q, *k_cache, *v_cache;
    void *o;
    float *lse;
    const int *block_table, *cu_seqlens_q, *seqlens_k;
    void *workspace;
    unsigned long long workspace_bytes;
    long long q_row_stride, q_head_stride, o_row_stride, o_head_stride;
    long long cache_page_stride, cache_head_stride, cache_row_stride;
    int B, Hq, Hkv, d, total_q, max_seqlen_q;
    int num_pages, page_size, table_width, table_stride;
    int causal, window_left, window_right;
    float scale;
    int dtype;
    void *stream;
} attn_fwd_paged_params_t;

int attn_fwd_paged(const attn_fwd_paged_params_t *params);

/*
 * attn_paged_workspace -- bytes of workspace that attn_fwd_paged wants for these parameters
 * on the current device.  It goes by B, Hq, Hkv, d, total_q and max_seqlen_q alone and reads no pointer.
 */
int attn_paged_workspace(const attn_fwd_paged_params_t *params, unsigned long long *bytes);

/*
 * ---------------------------------------------------------------- drafted trees, norms and rotation
 *
 * A step that checks several continuations of every request at once.  A request's new rows are the nodes of
 * a tree: the last token that is known (node 0; or the last few, a chain) and drafted tokens below it, each with the
 * number of its parent among the request's nodes, below its own.  A step then runs attn_paged_tables (nodes
 * as new tokens), attn_paged_tree (positions, masks), per layer attn_rope (queries, keys and values from the
 * projections into a buffer and into the cache) and attn_fwd_paged_tree, and, once the model's choice behind every node is
 * known, attn_paged_accept and attn_paged_move.  Requests of more nodes than the masks have bits are chunks of a
 * prompt: chains that need no mask, in the same calls.  What holds for the paged cache above (layout, index arrays,
 * bad values, ATTN_ERR_PAGE, replays) holds here.
 */

/*
 * attn_rope -- norms of queries and keys for each head and their rotation by position, in one pass over rows of
 * q [Hq], k [Hkv] and v [Hkv] heads (element (h, t, x) at h*head + t*row + x of their own strides):
 *     y = x * rsqrt(mean(x^2) + eps) * weight      (over the d elements of a head's row; y = x where the weight is NULL)
 *     phi_i = sum over axes a of positions[a][t] * inv_freq[a][i],  0 <= i < rot_dim / 2
 *     (y_a, y_b) -> (y_a cos phi_i - y_b sin phi_i, y_b cos phi_i + y_a sin phi_i)
 * with (a, b) = (i, i + rot_dim/2), or (2i, 2i + 1) where interleaved is not 0; elements from rot_dim on are not turned (without
 * a weight y = x, whatever stands beside them).
 * One axis is the usual rotation; with several (time, height, width) each pair's frequency stands in its axis's row and
 * the other rows hold 0 there.  All in 32 bits, rounded once; angles are exact to 2^-25 of a turn at any position and
 * frequency (positions may be negative).
 * Where slots is NULL, rows go to q_out and k_out (each may be its input with the same strides; nothing else overlaps), and
 * v and the caches are not looked at.  Otherwise q goes to q_out, k and, unturned, v go to slot slots[t] of the caches, and a row
 * of a negative slot is left out, of q_out as well; so is one of a slot at or past num_pages*page_size, with ATTN_ERR_PAGE.
 * Slots are distinct.  A contiguous [B][H][S][d] tensor whose entries share their positions counts as B*H heads of S rows.
 * q_weight, k_weight: [d], of the rows' type, or float where weight_f32 is not 0.  positions: int32, axis a at
 * positions + a*position_stride (at least rows, or 0: all axes share one row); inv_freq: float [axes][rot_dim/2].  With rot_dim = 0 both may be NULL.
 * rot_dim is a multiple of 16, at most d; 1 <= axes <= 4; frequencies are finite, of 2^60 at most; eps >= 0; rows <= 2^30; at most 65536 heads.
 */
typedef struct {
    const void *q, *k, *v;
    void *q_out, *k_out, *k_cache, *v_cache;
    const void *q_weight, *k_weight;
    const int *positions, *slots;
    const float *inv_freq;
    long long q_row_stride, q_head_stride, k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    long long q_out_row_stride, q_out_head_stride, k_out_row_stride, k_out_head_stride;
    long long cache_page_stride, cache_head_stride, cache_row_stride;
    long long position_stride;
    int rows, Hq, Hkv, d, rot_dim, axes, interleaved, weight_f32, num_pages, page_size;
    float eps;
    int dtype;
    void *stream;
} attn_rope_params_t;

int attn_rope(const attn_rope_params_t *params);

/*
 * attn_paged_tree -- positions and masks of the nodes.  Request b's nodes are rows cu_seqlens_q[b] ..
 * cu_seqlens_q[b+1]-1, its context the seqlens_k[b] tokens less these.  Node i's position is context + depth, and bit j of its
 * mask (word j / 32 of tree_mask + t*mask_stride, least significant bit first) is 1 for itself and the nodes above it, with
 * window_left >= 0 those at most window_left positions back.  parents[t]: number of the node above among the request's
 * nodes, -1 for none; one that is not below the node's own number counts as none, with ATTN_ERR_PAGE.  Requests of
 * more than 32*mask_words nodes are chunks: positions context + i, parents not read, masks not written.  Rows of no
 * request are left as they are.  1 <= B <= 16384, 1 <= mask_words <= 32, rows <= 2^30.
 */
typedef struct {
    const int *parents;                  /* [rows] */
    const int *cu_seqlens_q, *seqlens_k; /* [B+1], [B] */
    int *positions;                      /* [rows] */
    uint32_t *tree_mask;                 /* [rows][mask_words] */
    int B, rows, mask_words, mask_stride, window_left;
    void *stream;
} attn_paged_tree_params_t;

int attn_paged_tree(const attn_paged_tree_params_t *params);

/*
 * attn_fwd_paged_tree -- attn_fwd_paged with a mask among each request's new rows.  Row t of a request of sq <= 32*mask_words query
 * rows and sk keys keeps key j
 *     of the context, j < sk - sq:  where window_left < 0 or j >= positions[t] - window_left,
 *     of the new rows, j >= sk - sq:  where bit j - (sk - sq) of its mask is 1, whatever the window
 * (positions below the context's length count as that; positions may be NULL without a window; bits at or past sq are of no
 * account).  Any mask will do, not a tree's alone.  Requests of more rows are chunks, causal with the window, as in
 * attn_fwd_paged.  call.causal is 1 and call.window_right has no effect; all else of `call` is as for attn_fwd_paged, its workspace
 * too (attn_paged_workspace(&call)).  Cache rows of a request from the first context key that a window of its first position
 * leaves on, up to its last key, hold finite values, whether a mask keeps them or not.
 */
typedef struct {
    attn_fwd_paged_params_t call;
    const uint32_t *tree_mask; /* [total_q][mask_words], row t at tree_mask + t*mask_stride */
    const int *positions;      /* [total_q] or NULL */
    int mask_words, mask_stride;
} attn_fwd_paged_tree_params_t;

int attn_fwd_paged_tree(const attn_fwd_paged_tree_params_t *params);

/*
 * attn_paged_accept -- which nodes of every request the model confirms.  The first confirmed[b] nodes (1 at least; NULL: 1 for
 * every request) are known, a chain; a prompt's chunk has all of its rows confirmed.  From the last of them a walk goes to the
 * first child (the lowest number above the node's own whose parent it is) whose token is the model's choice behind the node, targets[node],
 * and on from there, max_path drafted nodes at most.  Writes, for every request,
 *   accepted[b]:     tokens it keeps of this step, confirmed and drafted (0 without rows);
 *   ctx_lens[b]:     its tokens in the cache from now on, seqlens_k - nodes + accepted (what attn_paged_tables takes next);
 *   next_tokens[b]:  the model's choice behind the last node (-1 without rows): the next step's node 0;
 *   path[b][j]:      the j-th drafted node on the walk, -1 behind the last;
 *   src_slots[b][j], dst_slots[b][j]: where that node's row lies in the cache and where a chain would have it, both -1 where
 *                    these are the same place, or (with ATTN_ERR_PAGE) where the table names no such page: attn_paged_move's lists.
 * Pages from ceil(ctx_lens[b] / page_size) on, which hold no token any longer, go back: behind the *free_count ids of the free list, requests and
 * pages in ascending order, *free_count_out (which may be free_count itself) is their number then.  Ids out of range or behind the table's end are
 * left out, and so is what the list (max_free ids) has no room for, each with ATTN_ERR_PAGE.  The table keeps its entries, which
 * attn_paged_tables overwrites.  With free_pages NULL (max_free = 0, free_count and free_count_out not looked at) no page goes back.
 * Pages that go back may still hold rows that src_slots names: every layer's attn_paged_move is ordered ahead of the first write to that
 * layer's caches (attn_rope, attn_paged_append) behind an attn_paged_tables that takes from this free list.  On one stream the calls of a step in
 * their order are; a move on another stream is waited for.
 * No output overlaps an input but for that.  1 <= B <= 16384, 1 <= max_path <= 1024, rows <= 2^30; with rows = 0 (no request has
 * any) tokens, targets and parents may be NULL.
 */
typedef struct {
    const int *tokens, *targets, *parents; /* [rows] */
    const int *confirmed;                  /* [B] or NULL */
    const int *cu_seqlens_q, *seqlens_k;   /* [B+1], [B] */
    const int *block_table;
    int *free_pages;           /* [max_free] in / out, or NULL */
    const int *free_count;     /* [1] */
    int *free_count_out;       /* [1] */
    int *accepted, *ctx_lens, *next_tokens;  /* [B] */
    int *path, *src_slots, *dst_slots;       /* [B][max_path] */
    int B, rows, max_path, table_width, table_stride, max_free, page_size, num_pages;
    void *stream;
} attn_paged_accept_params_t;

int attn_paged_accept(const attn_paged_accept_params_t *params);

/*
 * attn_paged_move -- rows of the caches of `layers` layers (element offset cache_layer_stride from one to the next) go from slot
 * src_slots[list][i] to slot dst_slots[list][i], K and V.  A pair with a negative slot is left out; one with a slot at or past
 * num_pages*page_size too, with ATTN_ERR_PAGE.  Within a list no source is the destination of an earlier pair (it may be that of
 * a later one: it is read before), and destinations are distinct; different lists share no slot that either writes.
 * What attn_paged_accept writes is so, where no two requests share pages that they write, and until the caches are written with slots of a later
 * attn_paged_tables (see there).  layers, Hkv <= 65536, lists and length <= 2^20.
 */
typedef struct {
    void *k_cache, *v_cache;
    const int *src_slots, *dst_slots; /* [lists][length] */
    long long cache_layer_stride, cache_page_stride, cache_head_stride, cache_row_stride;
    int layers, lists, length, Hkv, d, num_pages, page_size, dtype;
    void *stream;
} attn_paged_move_params_t;

int attn_paged_move(const attn_paged_move_params_t *params);

/*
 * attn_check -- read (and clear) the status word of `stream` on the current
 * device, in stream order after the work enqueued on it so far, and synchronise
 * the stream: ATTN_OK, ATTN_ERR_TIMEOUT if a launch on this stream gave up on a
 * barrier wait, ATTN_ERR_PAGE if one met a page id, slot or page count out of range
 * (and none timed out), or ATTN_ERR_CUDA if the stream itself reports an error.  Launches
 * on other streams do not affect it (streams share a word only past the first
 * 1023 distinct streams of a device, and for attn_fwd_noalloc calls on streams
 * attn_fwd has not used).
 */
int attn_check(void *stream);

/*
 * attn_release_workspace -- free (in stream order, cudaFreeAsync on `stream`) the
 * workspace the library holds for `stream` on the current device, if
 * any.  Call it before destroying a stream that ran custom masks; a later call on
 * the stream simply allocates a new one.  ATTN_OK, or ATTN_ERR_CUDA.
 */
int attn_release_workspace(void *stream);

/*
 * attn_debug_counters -- host-side counters since the library was loaded, for
 * tests and tuning: out[0] = workspace allocations, out[1] = tensor maps encoded,
 * out[2] = tensor maps served from the cache; entries past 2 are set to 0.
 * n = the number of entries of `out` (>= 1).
 */
int attn_debug_counters(unsigned long long *out, int n);

/* attn_strerror -- a static, human-readable string for a status code. */
const char *attn_strerror(int status);

/*
 * attn_tile_shape -- rows per query tile (*bm) and key columns per tile (*bn)
 * the kernel uses for head dim d, i.e. the granularity of tile skipping.
 * Returns ATTN_ERR_UNSUPPORTED for a head dim without a kernel.
 */
int attn_tile_shape(int d, int *bm, int *bn);

/*
 * attn_set_wait_timeout_ns -- the longest a kernel thread waits on one
 * barrier before it abandons the launch and records ATTN_ERR_TIMEOUT
 * (default 2e9 ns).  Applies to launches made after the call.  0 restores the
 * default.
 */
int attn_set_wait_timeout_ns(unsigned long long ns);

/*
 * attn_debug_inject -- test hook.  With flag 1 the next launch's load warp
 * never signals its first query tile, so the consumers' waits run out and the
 * launch ends with ATTN_ERR_TIMEOUT (no fault, no hang: every wait is bounded).
 * The flag clears itself after one launch.  0 disarms it.
 */
int attn_debug_inject(int flag);

/* attn_version -- library version, major*10000 + minor*100 + patch. */
int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H */
