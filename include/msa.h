/*
 * msa.h — C ABI of libmsa.so, the GB300 (sm_103a) forward path of MiniMax
 * Sparse Attention (MSA).
 *
 * The method (pages: the "MSA" study note, sections 2-1 "Two-branch sparse
 * attention" and 2-3 "Fixed attention budget"; the chipsbuilder.com article,
 * "Funzionamento Delle Due Branch"):
 *   index scores  s[t,g,j] = q^I[t,g] . k^I[j] / sqrt(d_I)      (j <= t)
 *   block scores  S[t,g,b] = max over j in block b, j <= t, of s[t,g,j]
 *   block set     B[t,g]   = {local(t)} + the k-1 best S[t,g,b], b < local(t)
 *   output        O[t,h]   = softmax(scale * q[t,h] K_J^T) V_J,
 *                 J = tokens j <= t of the blocks in B[t, g(h)], g(h) = h / (H_q/H_kv)
 *
 * Conventions for every call:
 *   - Returns a status; work is enqueued asynchronously on `stream`.
 *   - Every tensor pointer is a DEVICE pointer owned by the caller; the
 *     library neither frees nor keeps it after the call returns.
 *   - The library allocates nothing.  Scratch comes from a caller-owned device
 *     workspace whose minimum size the matching *_workspace() call returns.
 *     The workspace must stay alive and untouched until the enqueued work has
 *     finished; two calls in flight at once need two workspaces.
 *   - Tensors are dense, row-major, contiguous; bf16 is stored as 16-bit
 *     words; shapes are given beside each argument.
 *   - Indices are 0-based.  local(t) = t / Bk.  nb = ceil(N / Bk).
 *   - Host-side validation happens before any launch and returns
 *     MSA_ERR_INVALID_ARGUMENT (bad pointer, size or shape),
 *     MSA_ERR_UNSUPPORTED (a valid shape outside the supported set) or
 *     MSA_ERR_WORKSPACE_TOO_SMALL.  A failed launch returns MSA_ERR_CUDA.
 *   - Bad data found on the device (a block id outside [0, nb) other than -1)
 *     does not trap: the entry is skipped and an error word at the start of
 *     the workspace is set.  msa_check_device_error() reads that word; each
 *     call clears it when it starts.
 *
 * Supported shapes: d in {64, 128}; d_I in {32, 64, 128}; Bk in {64, 128};
 * 1 <= k <= 32; H_q / H_kv in {1, 2, 4, 8}; 1 <= H_kv <= 64; N >= 1.
 */
#ifndef MSA_H
#define MSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* msa_stream_t; /* same type as cudaStream_t; NULL = legacy default stream */

typedef enum {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARGUMENT = 1,
  MSA_ERR_UNSUPPORTED = 2,
  MSA_ERR_WORKSPACE_TOO_SMALL = 3,
  MSA_ERR_CUDA = 4,
  MSA_ERR_BAD_INDEX = 5,
  MSA_ERR_TIMEOUT = 6,
  MSA_ERR_NO_PAGES = 7
} msa_status_t;

/* Problem shape.  G = H_kv GQA groups (one index-query head per group);
 * gs = H_q / H_kv query heads per group; k counts the local block. */
typedef struct {
  int64_t N; /* tokens (prefill) or cache capacity per sequence (decode) */
  int H_q;   /* query heads */
  int H_kv;  /* key/value heads = GQA groups = index-query heads */
  int d;     /* head dim of q, k, v */
  int d_I;   /* index head dim of q^I, k^I */
  int Bk;    /* tokens per KV block */
  int k;     /* blocks per (query, group), local block included */
} msa_shape_t;

/* ---------------------------------------------------------------- select
 * Index branch: scoring, block max-pooling and the local-pinned top-k.
 * Pages: "MSA" study note 2-3 (equations for s, S and the block set), 3-2
 * "Index Branch", 3-4 "Forced local block", 3-5 "GPU kernel co-design"
 * (exp-free top-k on raw scores); Flash-MSA "プロキシアテンション" (streaming
 * top-k while sweeping key tiles; local block pinned to +inf).
 *
 *   q_idx     [N, G, d_I] bf16: index queries (one head per group)
 *   k_idx     [N, d_I]    bf16: index keys (one head shared by all groups)
 *   block_idx [G, N, k]   int32 out: slot 0 = local(t); slots 1.. = the
 *             min(k-1, local(t)) blocks b < local(t) of largest S, in
 *             descending S, equal S ordered by ascending b (the lower block
 *             wins a tie at the cut); remaining slots = -1.
 * Ranking uses the fp32 tensor-core dot products q^I . k^I (a positive
 * scale does not change the order).
 */
size_t msa_select_blocks_workspace(int64_t N, int G, int d_I, int Bk, int k);
msa_status_t msa_select_blocks(const void* q_idx, const void* k_idx, int64_t N, int G, int d_I, int Bk,
                               int k, int32_t* block_idx, void* workspace, size_t workspace_bytes,
                               msa_stream_t stream);

/* ---------------------------------------------------------------- invert
 * B -> B*: for every group g and block b, the (t, slot) pairs whose set
 * holds b.  Pages: Flash-MSA "バックワードパス" (B[batch, head, query,
 * slot] -> block inverted to B*[batch, head, block] -> queries) and the
 * "MSA" study note 3-5 (reverse sparse index feeding KV-outer attention).
 *
 *   block_idx [G, N, k] int32 (ids in [0, nb) or -1)
 *   row_ptr   [G, nb+1] int32 out: offsets into the group's entry region
 *   entries   [G, N*k]  int32 out: group g's list of block b is
 *             entries[g*N*k + row_ptr[g][b] .. g*N*k + row_ptr[g][b+1]),
 *             each entry t*k + slot, in ascending t (deterministic).
 *             Entries past n_entries[g] are left untouched.
 *   n_entries [G]       int32 out: entries listed for group g.
 * An id outside [0, nb) other than -1 sets the device error word and is not
 * listed.
 */
size_t msa_invert_blocks_workspace(int64_t N, int G, int Bk, int k);
msa_status_t msa_invert_blocks(const int32_t* block_idx, int64_t N, int G, int Bk, int k, int32_t* row_ptr,
                               int32_t* entries, int32_t* n_entries, void* workspace, size_t workspace_bytes,
                               msa_stream_t stream);

/* ---------------------------------------------------------------- attend
 * Main branch: exact softmax attention over the selected blocks' causally
 * visible tokens, every head of group g reading group g's set, computed
 * KV-outer (each K/V block once per tile of the queries that chose it) with
 * per-(t, h, slot) partial results merged by their log-sum-exp.
 * Pages: "MSA" study note 2-3 (Attn over K_{g,B}, V_{g,B}), 3-3 "Main
 * Branch", 3-5 (KV-outer execution, pre-scheduled tile chunking, two-phase
 * combine, LSE kept); chipsbuilder "Funzionamento Delle Due Branch" (tokens
 * causally visible in the selected blocks); Flash-MSA "フォワードパス" (main
 * LSE saved).
 *
 *   q         [N, H_q, d]  bf16
 *   k, v      [N, H_kv, d] bf16
 *   block_idx [G, N, k]    int32: each row's set (-1 = empty slot; a repeated
 *             id counts once; ids past local(t) hold no visible token and add
 *             nothing)
 *   scale     softmax scale (1/sqrt(d) in the pages)
 *   out       [N, H_q, d]  bf16 out: O[t, h]
 *   lse       [H_q, N]     fp32 out: natural-log log-sum-exp of the scaled
 *             scores over J; -inf (with out = 0) when J is empty.
 */
size_t msa_sparse_attn_fwd_workspace(const msa_shape_t* shape);
msa_status_t msa_sparse_attn_fwd(const void* q, const void* k, const void* v, const int32_t* block_idx,
                                 const msa_shape_t* shape, float scale, void* out, float* lse,
                                 void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* ---------------------------------------------------------------- backward
 * Gradients of msa_sparse_attn_fwd (main branch) and of the index branch's KL
 * alignment loss, over the same block sets.  Pages: "MSA" study note 4-2 (the
 * index branch learns from a KL loss against the mean of the GQA group's
 * main-branch attention probabilities) and 4-3 (the teacher is detached and the
 * index input gets a stop-gradient: the KL reaches only q^I and k^I);
 * Flash-MSA "バックワードパス" (both backward passes over the cached sparse
 * blocks, scheduled through the inverted map B*) and "KLダイバージェンス損失"
 * (the gradient on the index logits is index probability minus teacher).
 *
 * Per row (t, h), group g = h / gs, J = the selected blocks' tokens j <= t:
 *   P_j = exp(scale q.k_j - lse), D = dout.out, dZ_j = P_j (dout.v_j - D),
 *   dq = scale sum_j dZ_j k_j, dk_j += scale dZ_j q, dv_j += P_j dout.
 * Per row (t, g): teacher pbar_j = mean over the group's heads of P_j; index
 * logits z_j = q^I.k^I_j / sqrt(d_I); p_j = softmax over J of z;
 *   kl[g, t] = sum_j pbar_j (log pbar_j - log p_j)
 *   (loss = kl_weight * sum over (t, g) of kl), dL/dz_j = kl_weight (p_j - pbar_j),
 *   dq_idx = sum_j dL/dz_j k^I_j / sqrt(d_I), dk_idx_j += dL/dz_j q^I / sqrt(d_I).
 *
 *   q, k, v, q_idx, k_idx, block_idx, scale: as the forward calls
 *   out, lse  the forward's outputs for the same inputs
 *   dout      [N, H_q, d] bf16: gradient of the loss with respect to out
 *   dq        [N, H_q, d] fp32 out;  dk, dv [N, H_kv, d] fp32 out
 *   dq_idx    [N, G, d_I] fp32 out;  dk_idx [N, d_I] fp32 out
 *   kl        [G, N] fp32 out (nullable): each row's KL
 *   workspace msa_sparse_attn_bwd_workspace(shape) bytes, 256-byte aligned;
 *             it grows with N * G * k (the B* entries and per-slot partials)
 *             plus a teacher buffer bounded by query slabs of at most 131072
 *             positions (G * k * Bk * 2 bytes a position of one slab)
 * The gradient outputs are cleared and then accumulated in place on `stream`.
 */
size_t msa_sparse_attn_bwd_workspace(const msa_shape_t* shape);
msa_status_t msa_sparse_attn_bwd(const void* q, const void* k, const void* v, const void* q_idx, const void* k_idx,
                                 const int32_t* block_idx, const void* out, const float* lse, const void* dout,
                                 const msa_shape_t* shape, float scale, float kl_weight, float* dq, float* dk,
                                 float* dv, float* dq_idx, float* dk_idx, float* kl, void* workspace,
                                 size_t workspace_bytes, msa_stream_t stream);

/* ---------------------------------------------------------------- warmup mode
 * The training-time variant that comes before sparse routing.  Pages: the
 * "MSA" study note, 4-4 "Indexer warmup" (the main branch runs full attention
 * while the index branch learns the KL alignment against the full-context
 * teacher; top-k routing is switched on afterwards), 4-2 and 4-3 (the teacher
 * is the mean of the group's main-branch probabilities, detached, and the KL
 * reaches only q^I and k^I), 1-1 (dense causal GQA attention).  Same
 * definitions as msa_sparse_attn_bwd's index branch, with J(t, g) = every key
 * j <= t.  shape->Bk and shape->k must be valid values but are not used.  No
 * workspace and no device-side error paths.
 *
 * msa_warmup_fwd: dense causal attention and the index branch's normaliser.
 *   q, k, v, q_idx, k_idx: as msa_prefill
 *   out      [N, H_q, d] bf16 out: softmax(scale q.k_j, j <= t) V
 *   lse      [H_q, N] fp32 out: natural-log log-sum-exp of the scaled scores
 *   lse_idx  [G, N] fp32 out: log-sum-exp over j <= t of q^I.k^I_j / sqrt(d_I)
 * msa_warmup_index_grad: the KL loss of every row and its gradients, from the
 *   forward's lse and lse_idx.
 *   kl       [G, N] fp32 out: KL(teacher || index) of each row (not weighted)
 *   dq_idx   [N, G, d_I] fp32 out: kl_weight * d(sum KL)/d q^I
 *   dk_idx   [N, d_I] fp32 out: kl_weight * d(sum KL)/d k^I (overwritten)
 */
msa_status_t msa_warmup_fwd(const void* q, const void* k, const void* v, const void* q_idx, const void* k_idx,
                            const msa_shape_t* shape, float scale, void* out, float* lse, float* lse_idx,
                            msa_stream_t stream);
msa_status_t msa_warmup_index_grad(const void* q, const void* k, const void* q_idx, const void* k_idx,
                                   const float* lse, const float* lse_idx, const msa_shape_t* shape, float scale,
                                   float kl_weight, float* dq_idx, float* dk_idx, float* kl, msa_stream_t stream);

/* ---------------------------------------------------------------- prefill
 * The whole forward pass in one call: msa_select_blocks followed by
 * msa_sparse_attn_fwd on the same shapes and stream, with the same results.
 * Pages: "MSA" study note 3-5 (the index and main branches as separate
 * kernels feeding KV-outer attention and the two-phase combine); the pages
 * give no fused entry point.
 *
 *   q, k, v, q_idx, k_idx, scale, out, lse: as msa_select_blocks and
 *             msa_sparse_attn_fwd
 *   block_idx [G, N, k] int32 out: the sets, as msa_select_blocks
 *   workspace msa_prefill_workspace(shape) bytes, 256-byte aligned (one
 *             workspace serves both stages)
 */
size_t msa_prefill_workspace(const msa_shape_t* shape);
msa_status_t msa_prefill(const void* q, const void* k, const void* v, const void* q_idx, const void* k_idx,
                         const msa_shape_t* shape, float scale, int32_t* block_idx, void* out, float* lse,
                         void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* ---------------------------------------------------------------- varlen prefill
 * Several sequences in one prefill, each in its own run of cells.  Pages:
 * velog llama.cpp analysis, section 4 (with sequences mixed in one shared
 * cache the condition "block of the sequence = run of consecutive cache
 * cells" breaks and the port falls back to dense attention) and section 5
 * (the fix named there: an explicit per-sequence position -> cell -> block
 * map).
 *
 * Layout: sequence s holds cells [cu_seqlens[s], cu_seqlens[s+1]) of the
 * N-cell tensors (q, k, v, q_idx, k_idx, out, lse, block_idx: the msa_prefill
 * layouts with N cells); its position p is cell cu_seqlens[s] + p.  Every
 * cu_seqlens[s] is a multiple of Bk, cu_seqlens[0] = 0, the values do not
 * decrease and cu_seqlens[S] <= N.  A sequence's blocks are therefore whole
 * runs of cells and never shared.  Cells of a sequence past its last token
 * (padding up to the next block boundary) and cells past cu_seqlens[S] are
 * computed like tokens; no real token selects or attends to them (they lie
 * after every token of their block, and blocks of other sequences are never
 * candidates).
 *
 * Per cell t of sequence s the set is msa_select_blocks' rule with the
 * candidates restricted to the sequence: {local(t)} plus the k-1 best blocks b
 * with cu_seqlens[s]/Bk <= b < local(t).  Block ids are cell block ids.  The
 * attention is msa_sparse_attn_fwd on those sets, so out and lse of every
 * real token equal msa_prefill run on that sequence alone (block ids offset
 * by cu_seqlens[s]/Bk).
 *
 *   cu_seqlens [S+1] int32 (device), S >= 1.  A cu_seqlens that breaks the
 *              rules above sets the device error word (MSA_ERR_BAD_INDEX from
 *              msa_check_device_error); every cell then keeps only its local
 *              block.
 *   workspace  msa_select_blocks_varlen_workspace() / msa_prefill_varlen_workspace() bytes
 */
size_t msa_select_blocks_varlen_workspace(int64_t N, int G, int d_I, int Bk, int k);
msa_status_t msa_select_blocks_varlen(const void* q_idx, const void* k_idx, const int32_t* cu_seqlens, int S,
                                      int64_t N, int G, int d_I, int Bk, int k, int32_t* block_idx, void* workspace,
                                      size_t workspace_bytes, msa_stream_t stream);
size_t msa_prefill_varlen_workspace(const msa_shape_t* shape);
msa_status_t msa_prefill_varlen(const void* q, const void* k, const void* v, const void* q_idx, const void* k_idx,
                                const int32_t* cu_seqlens, int S, const msa_shape_t* shape, float scale,
                                int32_t* block_idx, void* out, float* lse, void* workspace, size_t workspace_bytes,
                                msa_stream_t stream);

/* ---------------------------------------------------------------- decode
 * One decode step for B sequences.  The query of sequence s sits at position
 * t = ctx_len[s] - 1 and its k, v and k^I are already in the caches.  The
 * whole index-key cache is scanned (the only part that grows with the
 * context), the block set is chosen as in msa_select_blocks, and only the
 * selected K/V blocks are read.  Pages: velog llama.cpp analysis, section 2
 * (256 B/token index-key scan, fixed K/V read per step) and section 4 (block
 * scores, max-pooling, forced local block, top-k, then attention over the
 * gathered blocks).
 *
 *   q_t          [B, H_q, d] bf16
 *   q_idx_t      [B, G, d_I] bf16
 *   k_idx_cache  [B, shape->N, d_I] bf16  (shape->N = cache capacity)
 *   k_cache      [B, shape->N, H_kv, d] bf16, v_cache likewise
 *   ctx_len      [B] int32 (device): 1 <= ctx_len[s] <= shape->N
 *   out          [B, H_q, d] bf16 out
 *   lse          [B, H_q] fp32 out (nullable)
 *   block_idx    [B, G, k] int32 out (nullable): the sets chosen
 * ctx_len values outside [1, N] set the device error word; that sequence's
 * outputs are zero.  A key whose score is -inf weighs 0; a head that attends to
 * no other key has out 0 and lse -inf.  A NaN score makes out and lse NaN.
 */
size_t msa_decode_workspace(int B, const msa_shape_t* shape);
msa_status_t msa_decode(const void* q_t, const void* q_idx_t, const void* k_idx_cache, const void* k_cache,
                        const void* v_cache, const int32_t* ctx_len, int B, const msa_shape_t* shape, float scale,
                        void* out, float* lse, int32_t* block_idx, void* workspace, size_t workspace_bytes,
                        msa_stream_t stream);

/* ---------------------------------------------------------------- paged decode
 * msa_decode over caches kept in pages: sequence s's token j is row
 * page_table[s][j / page_size] * page_size + j % page_size of the page pools,
 * so sequences of different lengths share one pool without a dense
 * [B, capacity] layout.  Same selection, attention and outputs as msa_decode
 * on the caches the pages spell out.  Pages: velog llama.cpp analysis, section
 * 4 (a per-sequence position -> cache cell -> block map is what lets a decode
 * kernel serve several sequences of different lengths, where the analysed
 * port falls back to one dense unified cache).
 *
 *   k_idx_pool  [n_pages, page_size, d_I] bf16
 *   k_pool      [n_pages, page_size, H_kv, d] bf16, v_pool likewise
 *   page_table  [B, max_pages] int32 (device): physical page of each logical
 *               page; entries past a sequence's ctx_len are not read
 *   page_size   tokens per page, a positive multiple of 16
 *   shape->N    = max_pages * page_size (a sequence's capacity)
 *   workspace   msa_decode_workspace(B, shape) bytes
 *   the rest as msa_decode.
 * A page id read outside [0, n_pages) sets the device error word (reported as
 * MSA_ERR_BAD_INDEX) and page 0 is read in its place.
 */
msa_status_t msa_decode_paged(const void* q_t, const void* q_idx_t, const void* k_idx_pool, const void* k_pool,
                              const void* v_pool, const int32_t* page_table, int64_t max_pages, int64_t n_pages,
                              int page_size, const int32_t* ctx_len, int B, const msa_shape_t* shape, float scale,
                              void* out, float* lse, int32_t* block_idx, void* workspace, size_t workspace_bytes,
                              msa_stream_t stream);

/* ---------------------------------------------------------------- FP8 index inputs
 * The index branch on FP8 inputs.  Pages: the chipsbuilder.com article, "Co-
 * Design Del Kernel" (FP8 is among the precisions of the method's kernel),
 * and the "MSA" study note, 6 "Limitations" item 1 (the index branch scores
 * the whole context, so its inputs carry the cost that grows with it).
 *
 * FP8 here is E4M3 of the OCP 8-bit floating point specification: one byte
 * per element, 1 sign bit, 4 exponent bits (bias 7), 3 mantissa bits, no
 * infinity, largest finite magnitude 448.  The selection rule is exactly that
 * of msa_select_blocks, applied to the decoded values: every product of two
 * E4M3 values is exact and the tensor cores sum them in fp32.  Multiplying all
 * of q^I, or all of k^I, by one positive factor before quantizing changes no
 * ranking, so the selection calls take no scale.  Supported d_I: 64 or 128
 * (MSA_ERR_UNSUPPORTED otherwise).
 *
 * msa_quantize_e4m3: y[i] = the E4M3 code nearest to the fp32 product
 *   (bf16 x[i]) * scale, ties to the even code, magnitudes beyond 448
 *   saturated to 448, NaN kept NaN.  x [n] bf16 (2-byte aligned), y [n] bytes
 *   out; no workspace.
 * msa_select_blocks_fp8: msa_select_blocks with q_idx [N, G, d_I] and
 *   k_idx [N, d_I] as E4M3 codes; workspace msa_select_blocks_workspace().
 * msa_prefill_fp8: msa_prefill with E4M3 q_idx and k_idx (q, k, v stay bf16);
 *   workspace msa_prefill_workspace().
 * msa_decode_fp8: msa_decode with q_idx_t [B, G, d_I] and k_idx_cache
 *   [B, N, d_I] as E4M3 codes, so the scan reads d_I bytes per cached token
 *   instead of 2 d_I; workspace msa_decode_workspace().
 * msa_decode_paged_fp8: msa_decode_paged with E4M3 q_idx_t and k_idx_pool
 *   [n_pages, page_size, d_I].
 */
msa_status_t msa_quantize_e4m3(const void* x, int64_t n, float scale, void* y, msa_stream_t stream);
msa_status_t msa_select_blocks_fp8(const void* q_idx, const void* k_idx, int64_t N, int G, int d_I, int Bk, int k,
                                   int32_t* block_idx, void* workspace, size_t workspace_bytes, msa_stream_t stream);
msa_status_t msa_prefill_fp8(const void* q, const void* k, const void* v, const void* q_idx, const void* k_idx,
                             const msa_shape_t* shape, float scale, int32_t* block_idx, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, msa_stream_t stream);
msa_status_t msa_decode_fp8(const void* q_t, const void* q_idx_t, const void* k_idx_cache, const void* k_cache,
                            const void* v_cache, const int32_t* ctx_len, int B, const msa_shape_t* shape, float scale,
                            void* out, float* lse, int32_t* block_idx, void* workspace, size_t workspace_bytes,
                            msa_stream_t stream);
msa_status_t msa_decode_paged_fp8(const void* q_t, const void* q_idx_t, const void* k_idx_pool, const void* k_pool,
                                  const void* v_pool, const int32_t* page_table, int64_t max_pages, int64_t n_pages,
                                  int page_size, const int32_t* ctx_len, int B, const msa_shape_t* shape, float scale,
                                  void* out, float* lse, int32_t* block_idx, void* workspace, size_t workspace_bytes,
                                  msa_stream_t stream);

/* ---------------------------------------------------------------- decode without allocation
 * The same decode step as msa_decode, for callers that cannot allocate device
 * memory: for instance a plugin whose host application owns every byte of the
 * GPU, or a serving loop that must not call cudaMalloc because it can block
 * and synchronize the device mid-step.  The pages have no counterpart of this
 * call; it exists only for such callers.
 *
 * No workspace argument: the scratch is a fixed 8 MiB array that the library
 * keeps in device memory on every GPU that loads it, until the process exits.
 * The call makes no allocation of any kind (no cudaMalloc/cudaFree, no
 * allocating library routine).  Arguments, layouts and outputs are those of
 * msa_decode.
 *   - The first call on a device looks up the array's device address for that
 *     device (cudaGetSymbolAddress, with the device current); make that first
 *     call before any stream capture.  The address is kept per device and
 *     context: a call made after cudaDeviceReset, or under another context of
 *     the same device, looks it up again, so it is never stale.
 *   - Shapes whose scratch (what msa_decode_workspace() reports for them)
 *     exceeds 8 MiB are rejected with MSA_ERR_WORKSPACE_TOO_SMALL before any
 *     launch.  B = 4, H_q = 64, H_kv = 8, d = 128, k = 16 needs about 2.4 MiB.
 *   - All calls on a device share the one array and it keeps the previous
 *     call's contents; each call clears what must start at zero.  Two calls
 *     that can overlap on the GPU (different streams, or different host
 *     threads) race on it: order them on one stream.
 *   - Device-side bad data (ctx_len outside [1, N]) still zeroes that
 *     sequence's outputs, and a bounded device wait that gives up still ends
 *     its kernel cleanly, but both flags live in the shared array's status
 *     word: this call returns MSA_OK for them and cannot report
 *     MSA_ERR_BAD_INDEX or MSA_ERR_TIMEOUT.  Callers that need those statuses
 *     use msa_decode with a workspace and msa_check_device_error.
 */
msa_status_t msa_decode_noalloc(const void* q_t, const void* q_idx_t, const void* k_idx_cache, const void* k_cache,
                                const void* v_cache, const int32_t* ctx_len, int B, const msa_shape_t* shape,
                                float scale, void* out, float* lse, int32_t* block_idx, msa_stream_t stream);

/* ---------------------------------------------------------------- dense prefill
 * Dense causal GQA attention over a packed batch of whole prompts, without an
 * index branch.  Pages: the "MSA" study note, 1-1 (dense causal GQA
 * attention, the branch that the sparse one replaces), and the velog llama.cpp
 * analysis, section 4 (the path that a serving engine falls back to when
 * several sequences share a batch).
 *
 * Sequence s holds rows [cu_seqlens[s], cu_seqlens[s+1]) of the N-row tensors;
 * cu_seqlens[0] = 0, the values do not decrease and cu_seqlens[S] <= N.  Any
 * lengths are allowed, 0 among them, and starts need no alignment.  For row t
 * of a sequence, over its rows j <= t:
 *   out[t, h] = softmax_j(scale q[t, h].k[j, h / gs]) v[j, h / gs].
 *
 *   q          [N, H_q, d] bf16;  k, v [N, H_kv, d] bf16
 *   cu_seqlens [S+1] int32 (device), S >= 1
 *   out        [N, H_q, d] bf16 out
 *   lse        [H_q, N] fp32 out: natural-log log-sum-exp of the scaled scores
 * Scores, softmax and sums are fp32; probabilities are rounded to bf16 for the
 * product with V.  A key whose score is -inf weighs 0; a row that sees no other
 * key has out 0 and lse -inf.  A NaN score makes the row's out and lse of that
 * head NaN.
 * Rows of no sequence (past cu_seqlens[S]) are neither read into a result nor
 * written: their out and lse stay as they were, whatever q, k and v hold there.
 * A cu_seqlens that breaks the rules sets the device error word
 * (MSA_ERR_BAD_INDEX) and nothing is written.  Supported: d in {64, 128},
 * H_q / H_kv in {1, 2, 4, 8}, H_kv <= 64, 1 <= N <= 2^24, S <= 2^24.
 */
size_t msa_dense_prefill_varlen_workspace(int64_t N, int S, int H_q, int H_kv, int d);
msa_status_t msa_dense_prefill_varlen(const void* q, const void* k, const void* v, const int32_t* cu_seqlens, int S,
                                      int64_t N, int H_q, int H_kv, int d, float scale, void* out, float* lse,
                                      void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* ---------------------------------------------------------------- 4-bit cache
 * A paged K/V cache in 4 bits.  Pages: velog llama.cpp analysis, section 2 (at
 * 1M tokens the K/V cache is what fills the memory: 4096 bytes a token and
 * layer in bf16; the pages name no 4-bit form, this one is the library's own).
 *
 * Format.  A head row of d values has 4 groups of d / 4 channels.  Each group
 * has a scale byte e << 3 | m of value 2^(e - 20) (1 + m / 8), 255 = NaN, and
 * each value a code 0..15 that stands for (code - 8) * scale, which bf16 holds
 * exactly.  Codes fill 32-bit words of 8 channels: nibble n (bits 4n .. 4n + 3)
 * is channel 2n for n < 4 and channel 2 (n - 4) + 1 for n >= 4.
 * Quantization of a group: scale = the smallest one with 7 scale >= max |x|,
 * code = 8 + x / scale rounded to nearest even and clamped to -7 .. 7.
 * Magnitudes beyond 7 * 3584 saturate.  A group that holds a NaN or an infinity
 * gets the NaN scale: all its values read as NaN.
 *
 *   k_codes, v_codes   [n_pages, page_size, H_kv, d / 2] bytes
 *   k_scales, v_scales [n_pages, page_size, H_kv, 4] bytes
 * All four 16-byte aligned; page_size a positive multiple of 16; d in {64, 128};
 * 1 <= H_kv <= 64.  A token takes (d / 2 + 4) * 2 * H_kv bytes (1088 at d = 128,
 * H_kv = 8, against 4096 in bf16).
 *
 * msa_kv4_store: quantizes packed rows into the pages of their sequences.
 *   k, v       [N, H_kv, d] bf16
 *   cu_seqlens [S+1] int32 (device): sequence s's rows are [cu[s], cu[s+1])
 *   pos0       [S] int32 (device): token position of a sequence's first row
 *   page_table [S, max_pages] int32 (device): row i of sequence s becomes token
 *              t = pos0[s] + i - cu[s], in page page_table[s][t / page_size]
 * A whole prompt is stored with pos0 = 0, the new tokens of a decode step with
 * one row a sequence and pos0 = the lengths so far.  Rows of no sequence are
 * passed over.  A row whose position lies outside the table, or whose page id
 * lies outside [0, n_pages), is skipped and sets the device error word
 * (MSA_ERR_BAD_INDEX).  Two rows of a call must not name one place.
 * 1 <= N < 2^31, 1 <= S <= 2^24.
 * msa_kv4_load: the same rows back, k and v [N, H_kv, d] bf16 out (exact
 *   values of the codes); a bad row reads as zeros (and sets the error word),
 *   rows of no sequence stay as they were.
 * workspace: msa_kv4_workspace() bytes (the error word).
 */
typedef struct {
  void* k_codes;
  void* k_scales;
  void* v_codes;
  void* v_scales;
  int64_t n_pages;
  int page_size;
  int H_kv;
  int d;
} msa_kv4_pool_t;
size_t msa_kv4_workspace(void);
msa_status_t msa_kv4_store(const void* k, const void* v, int64_t N, const int32_t* cu_seqlens, int S,
                           const int32_t* pos0, const int32_t* page_table, int64_t max_pages,
                           const msa_kv4_pool_t* pool, void* workspace, size_t workspace_bytes, msa_stream_t stream);
msa_status_t msa_kv4_load(const msa_kv4_pool_t* pool, int64_t N, const int32_t* cu_seqlens, int S,
                          const int32_t* pos0, const int32_t* page_table, int64_t max_pages, void* k, void* v,
                          void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* msa_dense_decode_paged_kv4: one decode token per sequence over its whole
 * 4-bit cache (the single-token form of msa_dense_prefill_varlen).
 *   q_t        [B, H_q, d] bf16
 *   page_table [B, max_pages] int32 (device); entries past a sequence's length
 *              are not read
 *   ctx_len    [B] int32 (device): tokens of each sequence in the cache, its
 *              newest included.  0 is an empty sequence: out 0, lse -inf.
 *   out        [B, H_q, d] bf16 out;  lse [B, H_q] fp32 out (nullable)
 * ctx_len outside [0, max_pages * page_size] counts as 0 and sets the device
 * error word; so does a page id outside [0, n_pages), read as page 0.
 * Scores, softmax and sums are fp32; probabilities are rounded to bf16 for the
 * product with V.  Scores of -inf and NaN count as in msa_dense_prefill_varlen.
 * Supported: H_q / H_kv in {1, 2, 4, 8}.
 *
 * msa_decode_paged_kv4, msa_decode_paged_kv4_fp8: msa_decode_paged and
 * msa_decode_paged_fp8 with K and V in a 4-bit pool (index keys stay in their
 * own pool [n_pages, page_size, d_I] of the same pages).  Same selection, the
 * attention over the chosen blocks on the 4-bit values.  shape->H_kv and d are
 * the pool's, shape->N = max_pages * page_size; workspace
 * msa_decode_workspace(B, shape) bytes.
 */
size_t msa_dense_decode_paged_kv4_workspace(int B, int H_q, int H_kv, int d);
msa_status_t msa_dense_decode_paged_kv4(const void* q_t, const msa_kv4_pool_t* pool, const int32_t* page_table,
                                        int64_t max_pages, const int32_t* ctx_len, int B, int H_q, float scale,
                                        void* out, float* lse, void* workspace, size_t workspace_bytes,
                                        msa_stream_t stream);
msa_status_t msa_decode_paged_kv4(const void* q_t, const void* q_idx_t, const void* k_idx_pool,
                                  const msa_kv4_pool_t* pool, const int32_t* page_table, int64_t max_pages,
                                  const int32_t* ctx_len, int B, const msa_shape_t* shape, float scale, void* out,
                                  float* lse, int32_t* block_idx, void* workspace, size_t workspace_bytes,
                                  msa_stream_t stream);
msa_status_t msa_decode_paged_kv4_fp8(const void* q_t, const void* q_idx_t, const void* k_idx_pool,
                                      const msa_kv4_pool_t* pool, const int32_t* page_table, int64_t max_pages,
                                      const int32_t* ctx_len, int B, const msa_shape_t* shape, float scale, void* out,
                                      float* lse, int32_t* block_idx, void* workspace, size_t workspace_bytes,
                                      msa_stream_t stream);

/* ---------------------------------------------------------------- rotary positions
 * Pages: the "MSA" study note, the model's configuration (d = 128, RoPE
 * dimension 64).  Every other call takes rows that are turned already.
 *
 * A pair (a, b) of a head row's channels at position p turns by p f:
 *   a' = factor (a cos p f - b sin p f),  b' = factor (b cos p f + a sin p f).
 * The first `rot` channels turn, in pairs (i, i + rot / 2) or, interleaved,
 * (2 i, 2 i + 1); the others stay.
 *   turns [rot / 2] uint64 (device): f / (2 pi) in units of 2^-64 turns (the
 *         integer nearest to it, modulo 2^64).  The angle modulo a turn is then
 *         p turns modulo 2^64, with no rounding at any position: scalings for
 *         long contexts are other tables (and, for some, a factor)
 *   rot   a multiple of 16, 16 <= rot <= the row's length, rot <= 128 for the
 *         calls that append
 * cos and sin are fp32 (within 2^-24), a product of each is rounded to fp32, and
 * so is their sum.
 *
 * msa_rope: rows turned (inverse 0) or turned back (inverse 1, the transpose:
 *   the gradient of rows from that of the turned ones).
 *   x, y      [N, H, d], bf16 (f32 = 0) or fp32 (f32 = 1), 16-byte aligned;
 *             d in {32, 64, 128, 256}.  y is x itself or does not overlap it
 *   x_stride, y_stride: elements from row n to row n + 1, at least H d (rows may
 *             lie apart, as slices of a wider projection), multiples of 8 (fp32: 4)
 *   positions [N] int32 (device), any value
 */
typedef struct {
  const uint64_t* turns;
  int rot;
  int interleaved;
  float factor;
} msa_rope_t;
msa_status_t msa_rope(const void* x, int64_t x_stride, void* y, int64_t y_stride, int64_t N, int H, int d, int f32,
                      const int32_t* positions, const msa_rope_t* rope, int inverse, msa_stream_t stream);

/* ---------------------------------------------------------------- rows into a paged cache
 * New tokens on their way into a paged cache, turned as they go: what a step
 * does between its projections and its attention, in one kernel.  Pages: velog
 * llama.cpp analysis, sections 2 and 4 (K, V and index keys in caches of their
 * own; an explicit map from positions to cells).
 *
 * N packed rows as for msa_kv4_store (cu_seqlens, pos0, page_table).  Of each:
 *   k [H_kv, d] is turned, rounded to bf16 and stored; v [H_kv, d] is stored;
 *   k_idx [d_I] (nullable) is turned and stored in k_idx_pool [n_pages,
 *     page_size, d_I];
 *   q [H_q, d] and q_idx [H_kv, d_I] (nullable) are turned into q_out [N, H_q, d]
 *     and q_idx_out [N, H_kv, d_I] (contiguous; q_out may be a contiguous q).
 * All inputs are bf16, 16-byte aligned, with a stride of elements from token to
 * token (multiples of 8).  With idx_f8, k_idx_pool and q_idx_out hold E4M3
 * codes: the turned rows, rounded to bf16, through msa_quantize_e4m3 with
 * idx_scale.
 *   positions [N] int32 (device, nullable): the positions that rows are turned
 *     by, where they are not their tokens' places in the cache (the nodes of a
 *     tree of drafts: ctx_len + depth)
 *   rope (nullable: K and q stay as they are), rope_idx (nullable: the index rows
 *     stay as they are; needs k_idx or q_idx)
 * msa_append_paged stores K and V in bf16 pools [n_pages, page_size, H_kv, d],
 * msa_append_paged_kv4 in a 4-bit pool, with the codes that msa_kv4_store
 * makes of the turned bf16 rows.  Rows of no sequence are passed over, q_out
 * and q_idx_out included; so are rows without a place (position outside the
 * table, page id outside [0, n_pages)), which set the device error word
 * (MSA_ERR_BAD_INDEX).  Two rows of a call must not name one place.
 * Supported: d in {64, 128}, d_I in {32, 64, 128}, 1 <= H_kv <= 64, H_q <= 512,
 * 1 <= N < 2^31, S <= 2^24.  workspace: msa_append_workspace() bytes.
 */
typedef struct {
  void* k;
  void* v;
  int64_t n_pages;
  int page_size;
  int H_kv;
  int d;
} msa_kv_pool_t;
typedef struct {
  const void* q;
  const void* k;
  const void* v;
  const void* q_idx;
  const void* k_idx;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  int64_t q_idx_stride;
  int64_t k_idx_stride;
  void* q_out;
  void* q_idx_out;
  void* k_idx_pool;
  const int32_t* positions;
  int H_q;
  int d_I;
  int idx_f8;
  float idx_scale;
} msa_append_t;
size_t msa_append_workspace(void);
msa_status_t msa_append_paged(const msa_append_t* rows, int64_t N, const int32_t* cu_seqlens, int S,
                              const int32_t* pos0, const int32_t* page_table, int64_t max_pages,
                              const msa_kv_pool_t* pool, const msa_rope_t* rope, const msa_rope_t* rope_idx,
                              void* workspace, size_t workspace_bytes, msa_stream_t stream);
msa_status_t msa_append_paged_kv4(const msa_append_t* rows, int64_t N, const int32_t* cu_seqlens, int S,
                                  const int32_t* pos0, const int32_t* page_table, int64_t max_pages,
                                  const msa_kv4_pool_t* pool, const msa_rope_t* rope, const msa_rope_t* rope_idx,
                                  void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* ---------------------------------------------------------------- drafted trees
 * Speculative decoding on paged caches: a step proposes a tree of tokens a
 * sequence, attends for all of them at once, keeps the branch that the target
 * model accepts.  Pages: velog llama.cpp analysis, sections 2 and 4 (a decode
 * step reads the whole cache for one token; caches of several sequences).
 *
 * A tree has up to T <= 64 nodes.  parents [B, T] int32 (device): the node above
 * node j, below j itself, or -1 (a root).  Node j of sequence b is token
 * ctx_len[b] + j of its cache (msa_append_paged puts it there).  tree_len [B]
 * int32 (device, nullable: T each): nodes of each sequence's tree.
 *
 * msa_tree_decode_paged, msa_tree_decode_paged_kv4: dense attention of the
 * trees' nodes over a bf16 or a 4-bit cache.  Node i sees tokens 0 .. ctx_len - 1,
 * itself and the nodes above it.  (T = 1, parents -1, is a dense decode step; a
 * chain, parents[j] = j - 1, a short prefill after a context.)
 *   q          [B, T, H_q, d] bf16
 *   page_table [B, max_pages] int32 (device); entries past a sequence's last node
 *              are not read
 *   ctx_len    [B] int32 (device): tokens before the tree, 0 allowed
 *   out        [B, T, H_q, d] bf16 out;  lse [B, T, H_q] fp32 out (nullable):
 *              natural-log log-sum-exp of the scaled scores.  Nodes past tree_len
 *              stay as they were.
 * Scores, softmax and sums are fp32; probabilities are rounded to bf16 for the
 * product with V.  Scores of -inf and NaN count as in
 * msa_dense_prefill_varlen; drafts that a node does not see count for nothing,
 * whatever they hold.  The device error word (MSA_ERR_BAD_INDEX) is set by a
 * page id outside [0, n_pages) (page 0 is read), a parent outside [-1, j) (it
 * counts as -1), and lengths below 0, tree_len above T or ctx_len + tree_len
 * above max_pages * page_size (nothing is written for that sequence).
 * Supported: H_q / H_kv in {1, 2, 4, 8}, d in {64, 128}, H_kv <= 64, B <= 2^20,
 * B T < 2^31, bf16 pools of fewer than 2^31 tokens.
 *
 * msa_verify_tree: which branch is accepted, and the token after it, from given
 * random numbers.  Node 0 is the token that the step began with (its parent is
 * not looked at); the drafts are tokens[j], j > 0.  The walk begins at node 0.
 * The children x of its node n are tested in their order with
 *   r = max(0, p - c q),  p = probs[n], q = draft_probs[n], c = 0, W = 1 at first:
 *   accepted where u[j] q(x) W < r(x), and the walk goes on from it;
 *   otherwise c grows by W and W becomes the sum of r.
 * (So a child drawn from q is accepted with probability min(1, p / q), and a
 * rejection leaves max(0, p - q), normalised, for the next one.)  Without
 * draft_probs the drafts were certain: accepted where u[j] W < r(x) with r = p,
 * otherwise r(x) becomes 0 and W falls by it.  Where no child is accepted, the
 * next token is the lowest one whose cumulative sum of r exceeds u_last[b] times
 * the sum of r (of p, where nothing is left of r).
 *   probs, draft_probs (nullable) [B, T, V] fp32, 16-byte aligned, each row a
 *              distribution; a value that is not a positive finite number counts as 0
 *   tokens [B, T] int32 (tokens[b][0] is not looked at);  u [B, T], u_last [B] fp32
 *              in [0, 1) (u_last: below it counts as 0, above as the largest number below 1)
 *   path   [B, T] int32 out: the accepted nodes in order, node 0 first, then -1
 *   n_path [B] int32 out: their number (0 where tree_len is 0)
 *   next   [B] int32 out: the next token (-1 where tree_len is 0 or p holds nothing)
 * Each r is counted in units of 2^-58 (exactly for c = 0 or 1 where p and q are 0 or
 * at least 2^-35, otherwise to 2^-59 and 2^-46 p), and the counts are added as
 * integers: a tree's outcome is the same in any batch.  (In a row that is no
 * distribution a value counts 2 at most, a sum 16.)  A parent outside [-1, j) or a
 * child's token outside [0, V) takes the node out, a tree_len outside [0, T] counts
 * as 0; both set the device error word.  Supported: 1 <= V < 2^31, B <= 2^20.
 * workspace: msa_verify_workspace() bytes.
 */
size_t msa_tree_decode_workspace(int B, int T, int H_q, int H_kv, int d);
msa_status_t msa_tree_decode_paged(const void* q, const msa_kv_pool_t* pool, const int32_t* page_table,
                                   int64_t max_pages, const int32_t* ctx_len, const int32_t* tree_len,
                                   const int32_t* parents, int B, int T, int H_q, float scale, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, msa_stream_t stream);
msa_status_t msa_tree_decode_paged_kv4(const void* q, const msa_kv4_pool_t* pool, const int32_t* page_table,
                                       int64_t max_pages, const int32_t* ctx_len, const int32_t* tree_len,
                                       const int32_t* parents, int B, int T, int H_q, float scale, void* out,
                                       float* lse, void* workspace, size_t workspace_bytes, msa_stream_t stream);
size_t msa_verify_workspace(void);
msa_status_t msa_verify_tree(const float* probs, const float* draft_probs, const int32_t* tokens,
                             const int32_t* parents, const int32_t* tree_len, const float* u, const float* u_last,
                             int B, int T, int64_t V, int32_t* path, int32_t* n_path, int32_t* next, void* workspace,
                             size_t workspace_bytes, msa_stream_t stream);

/* ---------------------------------------------------------------- pages of a cache
 * Page tables with reference counts, for any paged cache of this library (the
 * bf16 pools of msa_decode_paged, the 4-bit pools, the index-key pools).
 * Pages: velog llama.cpp analysis, sections 4 and 5 (an explicit map from a
 * sequence's positions to cache cells is what lets sequences share a cache).
 *
 * State (device, the caller's):
 *   page_table [n_seqs, max_pages] int32: sequence s holds the pages
 *              page_table[s][0 .. ceil(ctx_len[s] / page_size)); entries past
 *              them are not read, and written only where a call says so
 *   ctx_len    [n_seqs] int32
 *   refs       [n_pages] int32: how many sequences hold each page, 0 = free.
 * A new cache has ctx_len and refs 0.  Pages are shared whole: only a page
 * that one sequence holds is ever partly filled.
 *
 * msa_pages_reserve: sequence seqs[i] grows to new_len[i] tokens.  The pages
 *   it lacks are the lowest-numbered free ones, given out in the order of the
 *   entries and of the positions within one.  An entry that names no sequence,
 *   names one twice or would shrink it (or outgrow its table) sets the error
 *   word (MSA_ERR_BAD_INDEX); too few free pages set MSA_ERR_NO_PAGES.  Either
 *   way the call then changes nothing.
 * msa_pages_fork: the empty sequence dst[i] becomes a copy of src[i].  Full
 *   pages are shared; a partly filled last page is copied, in every pool, into
 *   the lowest free page (in the order of the entries).  dst must be distinct
 *   and empty (ctx_len 0) when the call begins; a source may occur often.
 *   Errors as above: the call then changes nothing (an id outside the pools
 *   among a source's full pages is copied as it is and sets the error word).
 * msa_pages_free: sequence seqs[i] becomes empty; its table entries become -1
 *   and its pages' counts fall.  A sequence named twice is freed once; an entry
 *   with a bad sequence or a bad page id is skipped and sets the error word.
 * msa_pages_compact: with L pages held, moves them to pages 0 .. L - 1: the r-th
 *   free page below L takes in the r-th held page from L on.  Contents (every
 *   pool), counts and tables follow.
 *     page_map [n_pages] int32 out (nullable): each page's new id, -1 if free
 *     n_live   [1] int32 out (nullable): L
 *
 * msa_pages_accept: of the tokens of sequence seqs[i] from base[i] on, those at
 *   base[i] + path[i][j], j < n_path[i], stay, as tokens base[i] + j, in every
 *   pool; the sequence then has base[i] + n_path[i] tokens, and the pages past
 *   them are free (their table entries -1).  path [n, T] int32 rises within an
 *   entry and stays below ctx_len - base (what msa_verify_tree returns, for
 *   drafts from base on); n_path 0 cuts the sequence off at base.  Every page
 *   from base on has to be the sequence's own (count 1).  An entry that breaks a
 *   rule, or names a sequence twice, sets the error word and the call changes
 *   nothing.  1 <= T <= 64; the pools' page_bytes are multiples of page_size.
 *   workspace: msa_pages_accept_workspace(pages, n, T) bytes.
 *
 * seqs, new_len, src, dst are int32 device arrays of n entries, n <= 4096 (0 is
 * allowed).  pools: n_pools <= 8 host entries, each a device array of n_pages
 * pages of page_bytes (a multiple of 16) at a 16-byte aligned address; pass every
 * pool that the tables address.  (reserve and free touch no pool, and compact's
 * page_map tells where the pages of further pools go; fork and accept have no such
 * list, so tables that are forked, or of which drafts are accepted, serve at most 8
 * pools: layers beyond these have tables of their own.)  workspace:
 * msa_pages_workspace(pages, n) bytes, n as in the call (0 for compact).
 * Limits: n_pages, max_pages < 2^27; max_pages * page_size < 2^31.
 */
typedef struct {
  int32_t* page_table;
  int32_t* ctx_len;
  int32_t* refs;
  int64_t max_pages;
  int64_t n_pages;
  int n_seqs;
  int page_size;
} msa_pages_t;
typedef struct {
  void* base;
  size_t page_bytes;
} msa_page_pool_t;
size_t msa_pages_workspace(const msa_pages_t* pages, int n);
msa_status_t msa_pages_reserve(const msa_pages_t* pages, const int32_t* seqs, const int32_t* new_len, int n,
                               void* workspace, size_t workspace_bytes, msa_stream_t stream);
msa_status_t msa_pages_fork(const msa_pages_t* pages, const int32_t* src, const int32_t* dst, int n,
                            const msa_page_pool_t* pools, int n_pools, void* workspace, size_t workspace_bytes,
                            msa_stream_t stream);
msa_status_t msa_pages_free(const msa_pages_t* pages, const int32_t* seqs, int n, void* workspace,
                            size_t workspace_bytes, msa_stream_t stream);
size_t msa_pages_accept_workspace(const msa_pages_t* pages, int n, int T);
msa_status_t msa_pages_accept(const msa_pages_t* pages, const int32_t* seqs, const int32_t* base, const int32_t* path,
                              const int32_t* n_path, int n, int T, const msa_page_pool_t* pools, int n_pools,
                              void* workspace, size_t workspace_bytes, msa_stream_t stream);
msa_status_t msa_pages_compact(const msa_pages_t* pages, const msa_page_pool_t* pools, int n_pools, int32_t* page_map,
                               int32_t* n_live, void* workspace, size_t workspace_bytes, msa_stream_t stream);

/* ---------------------------------------------------------------- status
 * msa_check_device_error: waits for `stream`, then returns MSA_ERR_BAD_INDEX
 * if the last call that used `workspace` met bad data on the device,
 * MSA_ERR_TIMEOUT if one of its kernels gave up a bounded wait,
 * MSA_ERR_NO_PAGES if a page call found too few free pages, MSA_OK
 * otherwise (or MSA_ERR_CUDA if the wait itself failed).
 * msa_status_string: a static, readable description of a status.
 */
msa_status_t msa_check_device_error(void* workspace, msa_stream_t stream);
const char* msa_status_string(msa_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H */
