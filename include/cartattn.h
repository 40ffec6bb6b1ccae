/*
 * cartattn.h -- C ABI of the GB300 (sm_103a) cartridge-attention library.
 *
 * A cartridge is a trained KV prefix: per layer a [p, kv_head, d] pair of
 * key/value rows living in KV-cache row space.  Cartridge keys are already
 * rotated (RoPE) at positions 0..p-1 and are never rotated again; the real
 * tokens that follow sit at RoPE positions p, p+1, ...  The first
 * `frozen_prefix` rows (1 by default: the attention sink) are frozen
 * constants; the remaining rows are trainable leaves.
 * (Cartridges guide, section "Semantics", parameterization bullet.)
 *
 * Attention runs over concat(sink, trainable rows, real-token K/V) along the
 * sequence with the end-aligned causal mask, source_offset = kv_seq - q_seq:
 * every query sees every cartridge row and is causal over the real tokens.
 * Query head h reads kv head h / (Hq / Hkv).
 * (Cartridges guide, "Semantics", attention bullet.)
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers, row-major, innermost last,
 *     16-byte aligned, owned by the caller.  The library never frees them.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *     validate their arguments synchronously on the host, then enqueue work
 *     asynchronously on `stream`; nothing is written when validation fails.
 *   - RoPE is the rotate-half form: element j pairs with j + d/2 at angle
 *     position * theta^(-2j/d).  Angles are reduced in f32: the frequency
 *     in turns is held as an f32 (hi, lo) pair, position * hi is split
 *     exactly into its rounded value and the fma remainder, and whole turns
 *     are dropped; positions must stay below 2^24.  Training with bf16
 *     inputs evaluates the remaining fraction with sincospif (absolute
 *     error about 2e-7), decode with the hardware sine/cosine (about 5e-7).
 *     Training with f32 inputs forms each angle in fp64 and reduces it
 *     modulo 2*pi in fp64 before an f32 sine/cosine.
 *   - Return value: CART_OK (0) or a negative cart_status.
 *   - The library holds no per-call state.  It caches, per process, the
 *     CUDA driver entry point used to build TMA descriptors and, per device,
 *     one helper stream with two events on which cart_attn_bwd runs its dQ
 *     kernel concurrently with its dK/dV kernel (forked from and joined back
 *     into the caller's stream).  Calls on one device from several host
 *     threads at once must therefore be serialised by the caller.
 */
#ifndef CARTATTN_H_
#define CARTATTN_H_

#include <stddef.h>

#if defined(__GNUC__)
#define CART_API __attribute__((visibility("default")))
#else
#define CART_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum cart_status {
  CART_OK = 0,
  CART_ERR_GEOMETRY = -1,   /* bad sizes: Hq % Hkv, d not 64/128, p < frozen_prefix, n < 1 ... */
  CART_ERR_POINTER = -2,    /* NULL or not 16-byte aligned */
  CART_ERR_DTYPE = -3,      /* dtype not supported for this argument */
  CART_ERR_WORKSPACE = -4,  /* workspace NULL or smaller than the *_workspace_size() answer */
  CART_ERR_CUDA = -5,       /* a CUDA runtime / driver call failed (launch, attribute, TMA map) */
  CART_ERR_DEVICE = -6,     /* current device is not a compute capability 10.3 GPU */
  CART_ERR_TIMEOUT = -7     /* a kernel gave up waiting (see cart_device_status) */
} cart_status;

typedef enum cart_dtype { CART_BF16 = 0, CART_F32 = 1 } cart_dtype;

/* Geometry of one training-shape call.
 *   B      independent sequences sharing ONE cartridge (the packed group)
 *   n      real tokens per sequence (q_seq); kv_seq = p + n < 2^24
 *   Hq     query heads;  Hkv  kv heads;  Hq % Hkv == 0
 *   d      head dimension, 64 or 128
 *   p      cartridge rows INCLUDING the frozen sink rows (p >= 0)
 *   frozen_prefix  leading cartridge rows whose gradient is exactly 0
 *   scale  softmax scale (normally 1/sqrt(d)); finite and > 0
 *   rope_theta     RoPE base (1e6 for the Qwen3 family)
 *   window sliding window in keys, 0 = none: the query at position P sees
 *          the keys at positions P - window + 1 .. P (cartridge row j sits
 *          at position j, so the window may cut through the cartridge and
 *          its sink).  (Cartridges guide, "gemma4 (measured)": on a local-SWA
 *          layer a cartridge is visible exactly as a real prefix, within
 *          the window.)                                                  */
typedef struct cart_geom {
  int B, n, Hq, Hkv, d, p, frozen_prefix;
  float scale;
  double rope_theta;
  int window;
} cart_geom;

/* ------------------------------------------------------------------------
 * cart_write_to_cache -- write the whole cartridge into a cache, converting
 * f32 leaf rows to the cache dtype (round to nearest even for bf16).
 * (Cartridges guide, "Semantics", serving bullet: the prefix is written into
 * an empty KV cache, converted to the cache dtype, and the cache advances to
 * p.  The same conversion produces the bf16 shadow the attention kernels
 * read once per optimizer step.)
 *   kc, vc        [p, Hkv, d] f32 (device)
 *   k_dst, v_dst  destination rows; row r of the cartridge goes to row
 *                 dst_row0 + r, rows are row_stride_elems elements apart
 *                 (row_stride_elems >= Hkv*d, a multiple of 8)
 *   dst_dtype     CART_BF16 or CART_F32
 * Either pair member may be NULL to skip it (not both).                   */
CART_API int cart_write_to_cache(const float* kc, const float* vc, int p, int Hkv, int d, void* k_dst,
                        void* v_dst, long long row_stride_elems, int dst_row0,
                        cart_dtype dst_dtype, void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_fwd -- training forward.
 *   q   [B, n, Hq, d]  in_dtype, NOT rotated (rotated in the library at p+i)
 *   k,v [B, n, Hkv, d] in_dtype, k NOT rotated
 *   kc, vc [p, Hkv, d] cart_dtype (bf16 shadow or f32 leaves), already in
 *          attended space (never rotated)
 *   o   [B, n, Hq, d]  in_dtype (output)
 *   lse [B, Hq, n]     f32 (output): natural-log log-sum-exp of the scaled
 *                      logits of each query row; the backward consumes it.
 * Arithmetic: bf16 tensor-core products with f32 accumulation; f32 inputs
 * are rounded to bf16 on load.  Workspace: cart_attn_fwd_workspace_size().  */
CART_API size_t cart_attn_fwd_workspace_size(const cart_geom* g, cart_dtype in_dtype,
                                    cart_dtype cart_dtype);
CART_API int cart_attn_fwd(const cart_geom* g, cart_dtype in_dtype, cart_dtype cart_dtype,
                  const void* q, const void* k, const void* v, const void* kc, const void* vc,
                  void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_bwd -- training backward through the concat into the cartridge.
 * (Cartridges guide, "Semantics": the backward routes gradients through the
 * concat into the trainable rows; row 0 is the frozen attention sink.)
 *   q,k,v,kc,vc,o,lse  as given to / returned by cart_attn_fwd
 *   dout [B, n, Hq, d] in_dtype: gradient of the loss w.r.t. o
 *   dq [B, n, Hq, d], dk, dv [B, n, Hkv, d]  in_dtype outputs, gradients
 *        w.r.t. the UN-rotated inputs q and k (the transpose rotation at
 *        position p+i is applied) and v
 *   dkc, dvc [p, Hkv, d] f32 outputs: gradient w.r.t. the cartridge rows,
 *        summed over the batch and over the query heads of each group.
 *        accumulate == 0 overwrites, 1 adds to the existing contents.  Rows
 *        < frozen_prefix are set to exactly 0.0 in both modes.
 * Workspace: cart_attn_bwd_workspace_size().                              */
CART_API size_t cart_attn_bwd_workspace_size(const cart_geom* g, cart_dtype in_dtype,
                                    cart_dtype cart_dtype);
CART_API int cart_attn_bwd(const cart_geom* g, cart_dtype in_dtype, cart_dtype cart_dtype,
                  const void* q, const void* k, const void* v, const void* kc, const void* vc,
                  const void* o, const float* lse, const void* dout, void* dq, void* dk,
                  void* dv, float* dkc, float* dvc, int accumulate, void* workspace,
                  size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_bwd_reuse -- cart_attn_bwd that takes the rotated queries and
 * keys, the RoPE table and the bf16 copies from the workspace of the
 * forward call that produced o and lse, instead of recomputing them.
 * (Cartridges guide, "Semantics": the backward of the same attention.)
 *   fwd_workspace [fwd_workspace_bytes]: the workspace passed to that
 *        cart_attn_fwd (same geometry, dtypes and inputs), read only; it
 *        must not have been reused since.  At least
 *        cart_attn_fwd_workspace_size() bytes, 16-byte aligned.
 *   workspace: cart_attn_bwd_reuse_workspace_size() bytes (the backward's
 *        own per-row vectors only).
 *   Everything else, outputs included, is as in cart_attn_bwd; the results
 *   are bit-identical to cart_attn_bwd on the same inputs.  The contents of
 *   fwd_workspace are not checked: a stale one gives wrong gradients.
 *   Returns CART_ERR_WORKSPACE for a missing or short workspace.         */
CART_API size_t cart_attn_bwd_reuse_workspace_size(const cart_geom* g, cart_dtype in_dtype,
                                                   cart_dtype cart_dtype);
CART_API int cart_attn_bwd_reuse(const cart_geom* g, cart_dtype in_dtype, cart_dtype cart_dtype,
                                 const void* q, const void* k, const void* v, const void* kc,
                                 const void* vc, const void* o, const float* lse,
                                 const void* dout, void* dq, void* dk, void* dv, float* dkc,
                                 float* dvc, int accumulate, const void* fwd_workspace,
                                 size_t fwd_workspace_bytes, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_bwd_parts -- cart_attn_bwd for a cartridge composed of several
 * independently trained parts concatenated along the rows, each with its
 * own frozen sink row.  (Cartridges guide, composition: parts are simply
 * concatenated, and every part keeps its sink.)
 *   frozen_rows [n_frozen] host int32: cartridge rows whose gradient is set
 *        to exactly 0.0 in both accumulate modes, in addition to the rows
 *        < frozen_prefix (e.g. each part's first row); any order, repeats
 *        allowed; 0 <= row < p; 0 <= n_frozen <= CART_MAX_FROZEN_ROWS.
 *        The list is copied into the launch: the caller may reuse it after
 *        the call returns.  frozen_rows may be NULL when n_frozen == 0.
 *   Everything else is as in cart_attn_bwd, which equals this call with
 *   n_frozen == 0.  Returns CART_ERR_GEOMETRY for a bad list.            */
#define CART_MAX_FROZEN_ROWS 64
CART_API int cart_attn_bwd_parts(const cart_geom* g, cart_dtype in_dtype, cart_dtype cart_dtype,
                                 const void* q, const void* k, const void* v, const void* kc,
                                 const void* vc, const void* o, const float* lse,
                                 const void* dout, void* dq, void* dk, void* dv, float* dkc,
                                 float* dvc, const int* frozen_rows, int n_frozen,
                                 int accumulate, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_fwd_packed / cart_attn_bwd_packed -- training on packed
 * segments: the group's sequences lie back to back along ONE token axis
 * instead of in a [B, n] batch.  RoPE restarts in every segment (its token i
 * sits at position p + i) and attention runs per segment behind the one
 * shared cartridge, so each segment is exactly one sequence of
 * cart_attn_fwd / cart_attn_bwd.  (Cartridges guide, "Deliberate
 * divergences from the reference", packing bullet; "Batched self-study
 * (measured)", packed training step.)
 *   g->B   number of segments S;  g->n  the longest segment (an upper bound:
 *          it sizes the launch grids and the RoPE table)
 *   total  packed tokens T, 1 <= T <= S * n
 *   cu_seqlens [S + 1] DEVICE int32, 4-byte aligned: 0 = cu[0] <= cu[1] <=
 *          ... <= cu[S] = T, every segment cu[s+1] - cu[s] <= n (empty
 *          segments allowed).  A table that breaks these rules sets device
 *          status bit 6; the kernels clamp it so that every access stays
 *          inside the tensors (the results are then undefined).
 *   q, o, dout, dq [T, Hq, d]; k, v, dk, dv [T, Hkv, d] (dtypes as in the
 *          unpacked calls); lse [Hq, T] f32 (natural log), written by the
 *          forward and read by the backward.
 *   dkc, dvc [p, Hkv, d] f32: summed over every segment; frozen rows as in
 *          cart_attn_bwd_parts (frozen_rows may be NULL when n_frozen == 0).
 * Workspace: the *_packed_workspace_size() answers (0 for bad sizes).     */
CART_API size_t cart_attn_fwd_packed_workspace_size(const cart_geom* g, int total,
                                                    cart_dtype in_dtype, cart_dtype cart_dtype);
CART_API int cart_attn_fwd_packed(const cart_geom* g, int total, const int* cu_seqlens,
                                  cart_dtype in_dtype, cart_dtype cart_dtype, const void* q,
                                  const void* k, const void* v, const void* kc, const void* vc,
                                  void* o, float* lse, void* workspace, size_t workspace_bytes,
                                  void* stream);
CART_API size_t cart_attn_bwd_packed_workspace_size(const cart_geom* g, int total,
                                                    cart_dtype in_dtype, cart_dtype cart_dtype);
CART_API int cart_attn_bwd_packed(const cart_geom* g, int total, const int* cu_seqlens,
                                  cart_dtype in_dtype, cart_dtype cart_dtype, const void* q,
                                  const void* k, const void* v, const void* kc, const void* vc,
                                  const void* o, const float* lse, const void* dout, void* dq,
                                  void* dk, void* dv, float* dkc, float* dvc,
                                  const int* frozen_rows, int n_frozen, int accumulate,
                                  void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_decode -- one q_seq = 1 decode step for B conversations behind
 * ONE shared cartridge.  (Cartridges guide, "Semantics", serving bullet: a
 * normal decode continues at position p with the training-time layout.)
 *   q      [B, Hq, d]  bf16, new token's query, NOT rotated
 *   k_new, v_new [B, Hkv, d] bf16, new token's key (NOT rotated) and value
 *   kc, vc [p, Hkv, d] bf16 shared cartridge (e.g. from cart_write_to_cache)
 *   k_cache, v_cache [B, cache_rows, Hkv, d] bf16 private caches; rows
 *          0..len[b]-1 hold already-rotated keys at positions p..p+len[b]-1
 *   priv_len [B] int32 (device): len[b], 0 <= len[b] < cache_rows (entries
 *          outside that range are clamped into it); cache_rows <= 32768 and
 *          p + cache_rows < 2^24
 *   o      [B, Hq, d] bf16 (output)
 * The new token sits at position p + len[b]: its rotated key and its value
 * are written to private row len[b], then it attends to the p cartridge rows
 * and private rows 0..len[b].  The caller advances len afterwards.
 * Workspace: cart_attn_decode_workspace_size().                           */
CART_API size_t cart_attn_decode_workspace_size(int B, int Hq, int Hkv, int d, int p, int cache_rows);
CART_API int cart_attn_decode(int B, int Hq, int Hkv, int d, int p, float scale, double rope_theta,
                     const void* q, const void* k_new, const void* v_new, const void* kc,
                     const void* vc, void* k_cache, void* v_cache, int cache_rows,
                     const int* priv_len, void* o, void* workspace, size_t workspace_bytes,
                     void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_decode_span -- span verify: `span` consecutive new tokens per
 * conversation in one step (q_seq = span), behind the shared cartridge.
 * (Cartridges guide, "Batched self-study (measured)", the --spec-b bullet:
 * each stream's span of carried and drafted tokens attends to its own cache
 * behind the prefix in one pass; the mask is the end-aligned causal one.)
 *   q      [B, span, Hq, d] bf16, the span's queries, NOT rotated
 *   k_new, v_new [B, span, Hkv, d] bf16, the span's keys (NOT rotated) and
 *          values
 *   o      [B, span, Hq, d] bf16 (output)
 *   priv_len [B]: len[b], clamped into 0 <= len[b] <= cache_rows - span
 *   Token t of conversation b sits at position p + len[b] + t: the span's
 *   rotated keys and values are written to private rows len[b] .. len[b] +
 *   span - 1, and query t attends to the p cartridge rows and private rows
 *   0 .. len[b] + t.  Requires 1 <= span <= cache_rows and
 *   (Hq / Hkv) * span <= 32.  Everything else is as in cart_attn_decode,
 *   which equals this call with span == 1.
 *   window  sliding window in keys (0: none), as in cart_geom: token t
 *   sees the keys at positions p + len[b] + t - window + 1 .. p + len[b] + t.
 * Workspace: cart_attn_decode_span_workspace_size().                      */
CART_API size_t cart_attn_decode_span_workspace_size(int B, int span, int Hq, int Hkv, int d,
                                                     int p, int cache_rows);
CART_API int cart_attn_decode_span(int B, int span, int window, int Hq, int Hkv, int d, int p,
                                   float scale,
                                   double rope_theta, const void* q, const void* k_new,
                                   const void* v_new, const void* kc, const void* vc,
                                   void* k_cache, void* v_cache, int cache_rows,
                                   const int* priv_len, void* o, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_decode_noalloc -- the decode step of cart_attn_decode for
 * callers that cannot allocate device memory: a serving loop running under a
 * fixed device-memory budget planned at start-up (a cudaMalloc on the decode
 * path would synchronize the device and stall the other streams), or a plain
 * C host that links only this library and has no device allocator to carve a
 * workspace from.  The paper has no counterpart; this is a library service.
 *   Arguments, layouts and results are those of cart_attn_decode, without
 *   the workspace: the scratch is a static device array of
 *   CART_DECODE_NOALLOC_SCRATCH_BYTES bytes that every GPU loading the
 *   library holds until the process exits.  (The 64-conversation, p = 4096,
 *   1025-row serving shape needs about 10 MiB.)
 *   Returns CART_ERR_WORKSPACE, without touching the device, when the
 *   problem needs more scratch than that; otherwise as cart_attn_decode.
 *   Calls no cudaMalloc / cudaFree or allocating library routine.
 *   The first call on each device looks up the array's device address (with
 *   that device current) and caches it; make that first call before any
 *   stream capture.  All calls share the one array: calls whose work can
 *   overlap on the GPU (other streams, or other host threads without
 *   ordering) race on it and must be serialised by the caller.  No scratch
 *   word needs to start at zero: each call writes what it reads.          */
#define CART_DECODE_NOALLOC_SCRATCH_BYTES (32u << 20)
CART_API int cart_attn_decode_noalloc(int B, int Hq, int Hkv, int d, int p, float scale,
                                      double rope_theta, const void* q, const void* k_new,
                                      const void* v_new, const void* kc, const void* vc,
                                      void* k_cache, void* v_cache, int cache_rows,
                                      const int* priv_len, void* o, void* stream);

/* ------------------------------------------------------------------------
 * Paged private caches.  A conversation's private rows may lie in pages of a
 * pool instead of in a dense [B, cache_rows] cache, so that conversations
 * hold only the rows they have, and branches of one conversation share their
 * common rows.  One set of tables serves every layer's pool:
 *   k_pages, v_pages [layers, n_pages, page_rows, Hkv, d]: the pools.
 *          page_rows is 16, 32, 64 or 128.  (cart_attn_decode_tree takes one
 *          layer's [n_pages, page_rows, Hkv, d].)
 *   table  [B, max_pages] int32: row r of conversation b is row
 *          r % page_rows of page table[b][r / page_rows].  An entry outside
 *          0 .. n_pages - 1 (-1 by convention) is no page: its rows are not
 *          there, which is never an error (pages that a sliding window has
 *          left behind may be taken out, but for the one that row lens[b]
 *          lies in, if it holds rows below: see cart_pages_reserve).
 *   lens   [B] int32: rows that the conversation holds; < 0 an idle slot.
 *   refs   [n_pages] int32: how many table entries name the page (a caller
 *          may add its own holds); <= 0 is free.
 * All tables are DEVICE memory, 4-byte aligned, max_pages * page_rows < 2^24
 * (with p and CART_MAX_TREE_NODES added, for the tree attention), and a call
 * reads and updates them on the stream: a step of reserve, tree attention,
 * accept and fork never waits for the host and can be captured.
 * Two calls that touch one table or pool must be ordered by the caller.   */

/* ------------------------------------------------------------------------
 * cart_attn_decode_tree -- one step over a tree of drafted tokens per
 * conversation, behind the shared cartridge, with paged private rows: the
 * span verify of cart_attn_decode_span for drafts that branch.
 *   nodes  tokens per conversation, 1 <= nodes <= CART_MAX_TREE_NODES
 *   parents [B, nodes] int32 (device): parents[b][t] = the node that t
 *          follows, an earlier one (< t), or -1: t follows the cached rows.
 *          NULL: a chain (node t follows node t - 1), which with nodes == 1
 *          is the single-token step.
 *   q      [B, nodes, Hq, d], k_new, v_new [B, nodes, Hkv, d] bf16, q and
 *          k_new NOT rotated
 *   kc, vc [p, Hkv, d] bf16 (NULL when p == 0); a non-finite cartridge value
 *          reaches every conversation
 *   o      [B, nodes, Hq, d] bf16 (output)
 * Node t with D ancestors sits at position p + lens[b] + D.  Its rotated key
 * and its value are written to private row lens[b] + t, and it attends to
 * the cartridge, private rows 0 .. lens[b] - 1 (at positions p + row), its
 * ancestors and itself; with window > 0, to those of them at its last
 * `window` positions (as in cart_geom).  Keys and values that it does not
 * attend to, other nodes' and cached rows' that its window has left behind,
 * do not reach it, whatever they hold (but for the cartridge's, above).
 * A query whose every logit is -inf has o = 0.
 * A node is unused when its row has no page, or its parent is neither -1
 * nor an earlier used node (-2 by convention pads a ragged tree): its o is
 * 0, its row is not written, and no node attends to it.  (A conversation
 * that has no used node costs as much as one that has; an idle one, below,
 * costs nothing.)  An unused node
 * that has a valid parent but no page sets device status bit 7.  All nodes
 * of an idle conversation are unused.  lens[b] above max_pages * page_rows
 * counts as that.  The rows lens[b] .. lens[b] + nodes - 1 must lie in pages
 * that no other conversation uses (cart_pages_reserve sees to it).
 * Hq / Hkv must be 1, 2, 4 or 8, d 64 or 128, B * nodes <= 65535.
 * Workspace: cart_attn_decode_tree_workspace_size(); its contents need no
 * initial value and nothing in it outlives the call.  Calls that may overlap
 * (on other streams, or captured into graphs that are replayed at once) need
 * workspaces of their own; so for the page operators below.               */
#define CART_MAX_TREE_NODES 64
CART_API size_t cart_attn_decode_tree_workspace_size(int B, int nodes, int Hq, int Hkv, int d,
                                                     int p, int page_rows, int max_pages);
CART_API int cart_attn_decode_tree(int B, int nodes, int window, int Hq, int Hkv, int d, int p,
                                   float scale, double rope_theta, const void* q,
                                   const void* k_new, const void* v_new, const void* kc,
                                   const void* vc, void* k_pages, void* v_pages, int n_pages,
                                   int page_rows, const int* table, int max_pages,
                                   const int* lens, const int* parents, void* o,
                                   void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cart_pages_fork -- conversation dst[f] becomes the first rows[f] rows of
 * conversation src[f], sharing its pages (no row is copied).
 *   src, dst, rows [forks] int32 (device); rows may be NULL: all rows.
 *          rows[f] above lens[src[f]] counts as that, below 0 as 0 (of an
 *          idle src dst gets no rows: its lens becomes 0).
 *   done   [forks] int32 (output): 1, or 0 for a fork that was left out: src
 *          or dst outside 0 .. B - 1, dst[f] also named by another fork of
 *          the call as its dst, or by any as its src.
 * The pages that dst held before are given back.  lens[dst] is set; rows
 * of dst's table row behind its last page are set to -1.
 * 1 <= forks <= 8192.                                                     */
CART_API int cart_pages_fork(int B, int* table, int max_pages, int* lens, int* refs, int n_pages,
                             int page_rows, const int* src, const int* dst, const int* rows,
                             int forks, int* done, void* stream);

/* ------------------------------------------------------------------------
 * cart_pages_reserve -- gives every conversation room for rows[b] rows in
 * all: what comes before a step that appends.
 *   rows   [B] int32 (device).  < 0, or more than max_pages * page_rows:
 *          the conversation is left as it is.  0 gives all its pages back.
 *   done   [B] int32 (output): 1 where rows[b] rows have room
 * lens[b] becomes min(max(lens[b], 0), rows[b]).  Pages behind the last of
 * rows[b] rows are given back first, of all conversations.  Then the pages
 * from that of row lens[b] to that of row rows[b] - 1 come to be b's alone:
 * missing ones are taken from the pool (lowest free page first, conversations
 * in order), and in the place of one that is shared (refs > 1) a free one is
 * taken, with the rows of b that it holds (below lens[b]) copied in every
 * layer.  When the pool runs out, the conversation that finds too few free
 * pages and all later ones that need any keep what they have, done 0; their
 * next rows may lie in a shared page, so they must not append in that step
 * (lens < 0 for them in its other calls, which then do no work for them, and
 * their real lens kept apart; or parents -2 for all their nodes).
 * Where rows[b] <= lens[b] nothing is to be appended and done is 1.  The page
 * in which rows[b] rows end, if they do not fill it, becomes b's alone even
 * so if a free page is left when it is b's turn.  (A caller that only lowers
 * lens[b] keeps that page shared; a later call gives back those behind.)
 * A missing page is taken as it is.  Where it is the page of row lens[b] and
 * has rows below that, those are there again, with what the page last held,
 * another conversation's rows perhaps: the caller writes them, or does not
 * take that page out.
 * Pages that lose their last holder to such a copy are free from the next
 * call on.
 *   k_pages, v_pages: dtype CART_BF16 or CART_F32, row = Hkv * d elements
 * Workspace: cart_pages_workspace_size().                                 */
CART_API size_t cart_pages_workspace_size(int B, int max_pages, int n_pages);
CART_API int cart_pages_reserve(int B, int layers, int Hkv, int d, cart_dtype dtype, void* k_pages,
                                void* v_pages, int n_pages, int page_rows, int* table,
                                int max_pages, int* lens, int* refs, const int* rows, int* done,
                                void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cart_pages_accept -- keeps the accepted path of each conversation's tree:
 * its rows are moved to follow the cached rows, in every layer.
 *   parents [B, nodes] as in cart_attn_decode_tree (NULL: chains)
 *   node   [B] int32 (device): the last accepted node; its ancestors are
 *          accepted with it.  -1, or an unused node: nothing is.
 *   new_lens [B] int32 (output, not lens itself): lens[b] + accepted nodes
 * Row lens[b] + (i-th node of the path) goes to row lens[b] + i.  The rows
 * behind new_lens[b] are left as they are, and a row whose new place has no
 * page is dropped.                                                        */
CART_API int cart_pages_accept(int B, int nodes, int layers, int Hkv, int d, cart_dtype dtype,
                               void* k_pages, void* v_pages, int n_pages, int page_rows,
                               const int* table, int max_pages, const int* lens,
                               const int* parents, const int* node, int* new_lens, void* stream);

/* ------------------------------------------------------------------------
 * cart_pages_compact -- moves the pool's live pages to its front, so that it
 * can be cut or saved: with n live pages, the live pages numbered n and
 * above go, in order, to the free numbers below n, in every layer.
 *   moved  [n_pages] int32 (output): the page's new number, -1 if it was free
 *   live   [1] int32 (output): n
 * table (entries that name a free page become -1) and refs follow.
 * Workspace: cart_pages_workspace_size().                                 */
CART_API int cart_pages_compact(int B, int layers, int Hkv, int d, cart_dtype dtype, void* k_pages,
                                void* v_pages, int n_pages, int page_rows, int* table,
                                int max_pages, int* refs, int* moved, int* live, void* workspace,
                                size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * A paged cache held to a budget of rows.  The calls below go with the paged
 * private caches above (tables, pools and their rules are the same): a prompt's
 * rows are appended, the attention weight that each row gets is added up, rows
 * of little weight are evicted, and decoding goes on.  Evicting moves rows
 * together, so that a row's place no longer tells its token's position:
 *   place     cartridge row j has place j, private row r place p + r.  What a
 *             query sees goes by places: a query at place x the places up to x,
 *             with window > 0 those above x - window, and always those below
 *             `sinks` (>= 0; cartridge rows, and private ones where it is
 *             above p)
 *   position  of the rotation: pos [B] int32 (device), or NULL for positions
 *             equal to places, which they are until rows are evicted.  Values
 *             outside 0 .. 2^24 - 1 are clamped into it.
 *   weights   [B, Hkv, weight_rows] f32, one layer's: weights[b][g][r] belongs
 *             to private row r of conversation b in kv head g; weight_rows >=
 *             max_pages * page_rows.  Kept by conversation and row, not by
 *             page: fork, reserve and compact leave them as they are (a caller
 *             that forks copies its weights along).
 * Of the calls that take several new tokens of a conversation, none has positions
 * apart from places: cart_attn_decode_tree rotates at p + lens[b], which after an
 * eviction is not the token's position, and nothing tells it so.  A conversation
 * whose rows were evicted goes on by cart_attn_decode_paged, a token at a time.
 * Hq / Hkv is 1 to 8 here, any of them, and d 64 or 128.
 * Workspaces as above: no initial value, nothing outlives the call, calls that
 * may overlap need workspaces of their own.                                */

/* ------------------------------------------------------------------------
 * cart_pages_append -- a run of tokens per conversation goes to its next rows,
 * in one layer: what a prompt's attention leaves to decoding.
 *   cu_seqlens NULL: k, v [B, n, Hkv, d] bf16, n tokens each; total = B * n
 *          [B + 1] int32 (device): k, v [total, Hkv, d], conversation b's tokens
 *          are cu_seqlens[b] .. cu_seqlens[b + 1] - 1 (as in the packed calls;
 *          n is not read).  A token in no conversation's run is left out and
 *          sets device status bit 6.
 *   k      NOT rotated
 *   pos    position of the conversation's first token here (NULL: p + lens[b])
 * Token i of conversation b goes to row lens[b] + i: its key rotated at its
 * position, rounded to bf16, and its value.  The rows must lie in pages that no
 * other conversation uses (cart_pages_reserve sees to it).  A row that has no
 * page is dropped and sets device status bit 7; an idle conversation (lens < 0)
 * has nothing written.  lens is not changed (every layer has its call).      */
CART_API int cart_pages_append(int B, int n, int total, const int* cu_seqlens, int Hkv, int d,
                               int p, double rope_theta, const void* k, const void* v,
                               void* k_pages, void* v_pages, int n_pages, int page_rows,
                               const int* table, int max_pages, const int* lens, const int* pos,
                               void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_weights -- the attention weight that each key gets from the last
 * `queries` tokens of each conversation, whose rows are cached already.
 *   q      [B, queries, Hq, d] bf16, NOT rotated: query i of conversation b has
 *          place p + lens[b] - queries + i (end-aligned); those that would lie
 *          before its first row are not there, and what q and lse hold for them
 *          does not matter
 *   lse    [B, Hq, queries] f32: their natural-log log-sum-exps, as
 *          cart_attn_fwd returns them (-inf: every logit was; the query gives
 *          no weight).  Those of an attention with sinks beside a window are the
 *          caller's to find: cart_attn_fwd has none.
 *   pos    position of query 0 (NULL: its place)
 *   kc     [p, Hkv, d] bf16 (NULL when p == 0)
 *   weights, and cart [B, Hkv, p] f32 for the cartridge's rows (NULL when
 *          p == 0): the sum over the queries that see the key and over the
 *          heads of its group of exp(scale * q . k - lse).
 *          accumulate == 0: rows 0 .. lens[b] - 1 and all of cart are set; 1:
 *          it is added, but for the rows of the queries themselves (from
 *          lens[b] - queries on), which are set.  Rows that have no page count
 *          as seen by no query.  Rows from lens[b] on are left as they are.
 * The rotated queries enter the products as three bf16 terms (all 24 bits of
 * their f32 values), the sums are f32.  A key that a query does not see gets nothing from
 * it, whatever either holds.
 * Workspace: cart_attn_weights_workspace_size().  It has a f32 for each key that
 * the tables can name and each 128 columns (queries * Hq / Hkv) of a kv head: with
 * the queries' terms 1.9 GB for 32768 over as many keys, 8 heads of 4.  A long
 * prompt is weighed in chunks, the rows that are there growing with them and
 * accumulate 1 from the second on.                                        */
CART_API size_t cart_attn_weights_workspace_size(int B, int queries, int Hq, int Hkv, int d, int p,
                                                 int page_rows, int max_pages);
CART_API int cart_attn_weights(int B, int queries, int window, int sinks, int Hq, int Hkv, int d,
                               int p, float scale, double rope_theta, const void* q,
                               const float* lse, const void* kc, const void* k_pages, int n_pages,
                               int page_rows, const int* table, int max_pages, const int* lens,
                               const int* pos, int accumulate, float* weights, int weight_rows,
                               float* cart, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ------------------------------------------------------------------------
 * cart_pages_evict -- conversations that hold more than keep[b] rows come down
 * to keep[b], in every layer and kv head by its own weights.
 *   keep   [B] int32 (device): < 0, or at least lens[b]: left as it is
 *   first, recent  the rows below `first` stay, and the last `recent` ones as
 *          far as there is room beside those; the room that is left goes to the
 *          rows between that have most weight, ties to the lower row, NaN
 *          counting as most
 *   weights [layers, B, Hkv, weight_rows] f32, or NULL: the last rows stay
 *   done   [B] int32 (output; may be keep itself): 1, or 0 where the
 *          conversation holds more than keep[b] rows and was left as it is: a
 *          page of its rows is not there, or there were too few free pages
 * The rows that stay keep their order: the i-th of them becomes row i, and its
 * weight weights[..][i]; rows and weights behind are left as they were.  Pages
 * from that of row `first` to that of row keep[b] - 1 that are shared (refs > 1)
 * are not written, whether or not a row in them changes its place: a free one takes
 * the place of each (lowest first, conversations in order; one that finds too few,
 * and all later ones that need any, are left).  Pages
 * behind the last of keep[b] rows are given back.  What is given back, or loses
 * its last holder, is free from the next call on.  lens[b] becomes keep[b].
 *   k_pages, v_pages: all layers, CART_BF16 or CART_F32; a head's row, d
 *          values, must be a multiple of 16 bytes
 * Workspace: cart_pages_evict_workspace_size().                           */
CART_API size_t cart_pages_evict_workspace_size(int B, int max_pages, int n_pages);
CART_API int cart_pages_evict(int B, int layers, int Hkv, int d, cart_dtype dtype, void* k_pages,
                              void* v_pages, int n_pages, int page_rows, int* table, int max_pages,
                              int* lens, int* refs, float* weights, int weight_rows,
                              const int* keep, int first, int recent, int* done, void* workspace,
                              size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------
 * cart_attn_decode_paged -- one new token per conversation, as
 * cart_attn_decode_tree with one node, with positions apart from rows, a window
 * with sinks, and the weights that the token gives.
 *   q [B, Hq, d], k_new, v_new [B, Hkv, d], o [B, Hq, d] bf16; kc, vc
 *          [p, Hkv, d] bf16 (NULL when p == 0)
 *   pos    position of the new token (NULL: p + lens[b])
 *   weights NULL: not kept.  Else to those of rows below lens[b] is added what
 *          the token's heads give the row, and that of row lens[b] is set.
 * The token's rotated key (rounded to bf16) and its value are written to row
 * lens[b], which must lie in a page of its own; it attends to what it sees of
 * the cartridge and rows 0 .. lens[b] (rows without a page are not there; keys
 * and values that it does not see do not reach it, whatever they hold, but for
 * a cartridge value that is not finite and that some conversation sees).  A
 * query whose every logit is -inf has o = 0 and gives no weight.  A key that is
 * not finite makes the logits of those that see it NaN or infinite.
 * An idle conversation (lens < 0) has o = 0 and nothing written, and so has one
 * whose row lens[b] has no page, which sets device status bit 7.
 * o may be q itself; outputs overlap nothing else that the call is given.
 * The rotated queries enter the products with private rows as three bf16 terms
 * (all 24 bits of their f32 values), those with the cartridge as two (2^-16 of
 * the value): where there is a cartridge, the log-sum-exp that the weights are
 * relative to is as exact as these.  The softmax weights of the values enter as
 * two bf16 terms (2^-15 of the weight); sums are f32.
 * Workspace: cart_attn_decode_paged_workspace_size(), `weights` 1 where they are
 * kept, which takes 4 * Hq bytes for every row that the tables can name; the work
 * is cut for the current device's multiprocessors, so the size is that device's.
 * (Where neither weights, sinks nor positions apart from places are wanted, the tree
 * of one node is the faster call for a few conversations.)                 */
CART_API size_t cart_attn_decode_paged_workspace_size(int B, int Hq, int Hkv, int d, int p,
                                                      int page_rows, int max_pages, int weights);
CART_API int cart_attn_decode_paged(int B, int window, int sinks, int Hq, int Hkv, int d, int p,
                                    float scale, double rope_theta, const void* q,
                                    const void* k_new, const void* v_new, const void* kc,
                                    const void* vc, void* k_pages, void* v_pages, int n_pages,
                                    int page_rows, const int* table, int max_pages,
                                    const int* lens, const int* pos, float* weights,
                                    int weight_rows, void* o, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Human-readable name of a cart_status value (static string). */
CART_API const char* cart_status_string(int status);

/* Reads (and with clear != 0 resets) the device status word that kernels set
 * when a bounded wait gives up (bit 0: a TMA copy, 1: an MMA, 2: the softmax
 * warps, 3: the epilogue), when a work schedule is inconsistent (bit 4), or
 * when the dynamic shared memory does not start 1024-byte aligned (bit 5;
 * the kernel then does nothing), when a packed segment table breaks its
 * rules (bit 6), or when a drafted, appended or decoded token's row has no
 * page (bit 7).  Synchronizes the current device.  Writes the bits to
 * *bits_out (may be NULL); returns CART_OK, CART_ERR_TIMEOUT when any bit is
 * set, or CART_ERR_CUDA. */
CART_API int cart_device_status(unsigned* bits_out, int clear);

/* cart_release -- destroys the current device's helper stream and events
 * (created by the first cart_attn_bwd on that device; see the conventions
 * above) after waiting for the work queued on that stream.  The next
 * backward call creates them again.  Call it with no library call in
 * flight on the device from another host thread.  The library holds no
 * other per-device state besides the static scratch array of
 * cart_attn_decode_noalloc, which lives as long as the loaded library.
 * Returns CART_OK or CART_ERR_CUDA (no usable current device).            */
CART_API int cart_release(void);

/* ------------------------------------------------------------------------
 * Launch tracing (off by default).  cart_trace_enable(1) clears the trace
 * and starts recording: every later kernel launch of the library is
 * bracketed by two CUDA events recorded on the launching stream.
 * cart_trace_enable(0) stops recording and keeps what was recorded.
 * cart_trace_count() returns the number of recorded launches (at most
 * 65536).  cart_trace_get(i, ...) copies the kernel's name (NUL-terminated,
 * truncated to name_len) and, if ms != NULL, waits for launch i to finish
 * and writes its device time in milliseconds.  Not meant for use while a
 * stream is being captured into a CUDA graph. */
CART_API int cart_trace_enable(int on);
CART_API int cart_trace_count(void);
CART_API int cart_trace_get(int i, char* name, int name_len, float* ms);

#ifdef __cplusplus
}
#endif

#endif /* CARTATTN_H_ */
