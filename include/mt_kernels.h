/*
 * mt_kernels.h — kernel-level C ABI of the layer templates.
 *
 * These entry points launch one kernel (or one fixed kernel sequence) of the
 * stateless layer templates on caller-provided device buffers. They exist so
 * that each kernel can be checked alone against the oracle; mt_train_step()
 * (mt.h) runs the same launchers. The stateless-template idea itself —
 * kernels that bind a layer's weights by pointer as they stream in, with no
 * persistent autograd graph — is from "MegaTrain: Full Precision Training of
 * 100B+ Parameter Large Language Models on a Single GPU" (chatpaper
 * abstract, optimisation 2) and the chestersoft digest (Methodik, "Stateless
 * Layer Templates").
 *
 * Conventions for every function here:
 *  - all pointer arguments are DEVICE pointers, owned by the caller, 16-byte
 *    aligned; matrices are row-major with a row stride in elements that is a
 *    multiple of 8;
 *  - bf16 means IEEE bfloat16 (uint16 storage), f32 IEEE binary32;
 *  - `stream` is a cudaStream_t (NULL = legacy default stream);
 *  - the call only enqueues work; it returns MT_OK (0), MT_EINVAL for bad
 *    sizes or alignment (nothing enqueued), or MT_ECUDA for a launch error;
 *  - `err_flag` (device int, may be NULL where unused) receives a nonzero
 *    code if a kernel's bounded internal wait gave up (1 to 7) or a position
 *    lay outside a rotation table (8); it is never cleared by the library.
 *    While it holds the code of a wait, the waits of every kernel that is
 *    given it give up early and outputs may stay unwritten. Code 8 stops
 *    nothing, and the code of a wait replaces it.
 */
#ifndef MT_KERNELS_H
#define MT_KERNELS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Epilogues of mtk_gemm_bf16. */
#define MTK_EPI_STORE_BF16 0 /* C (bf16) = A*B                          */
#define MTK_EPI_STORE_F32 1  /* C (f32)  = A*B                          */
#define MTK_EPI_ADD_F32 2    /* C (f32)  = R (f32) + A*B, R may equal C */

/*
 * C[M,N] = A * B on the tcgen05 tensor cores, bf16 operands, f32 accumulation.
 *  a_mn = 0: A is stored [M][K] (row stride lda);  a_mn = 1: A is stored [K][M].
 *  b_mn = 0: B is stored [N][K] (C = A * B^T);     b_mn = 1: B is stored [K][N].
 * With a_mn = b_mn = 0 this is the forward projection y = x W^T; (0, 1) is the
 * data gradient dx = dy W; (1, 1) is the weight gradient dW = dy^T x.
 * M, N, K > 0. Deterministic: fixed K order, no atomics. When a workspace is
 * set (mtk_gemm_use_workspace), the tiles of the last, partial wave are split
 * over K between CTAs and their fp32 partial sums added in a fixed order: the
 * result then differs from the unsplit one in the order of the K sum only, and
 * is the same from run to run.
 */
int mtk_gemm_bf16(const void* A, int64_t lda, int a_mn, const void* B, int64_t ldb, int b_mn, void* C,
                  int64_t ldc, const void* R, int64_t ldr, int M, int N, int K, int epi, int* err_flag,
                  void* stream);

/*
 * Workspace of the mtk_gemm_* calls (this stream-ordered split is a scheduling
 * device of this library; the pages have no counterpart). ws: device memory of
 * mtk_gemm_workspace_bytes() bytes, 16-byte aligned, owned by the caller, whose
 * first mtk_gemm_workspace_clear_bytes() bytes are zero before its first use
 * (the calls leave them in a state later calls accept); NULL (the default)
 * turns the split off. The setting is process-wide and kept until changed.
 * Calls that use the same workspace must not overlap on the GPU (use one
 * stream). Returns MT_EINVAL for a misaligned pointer.
 */
uint64_t mtk_gemm_workspace_bytes(void);
uint64_t mtk_gemm_workspace_clear_bytes(void);
int mtk_gemm_use_workspace(void* ws);

/* RMSNorm forward on x f32 [T,h]: y bf16 = x*rstd*gamma, rstd f32 [T] = 1/sqrt(mean(x^2)+eps).
 * h a multiple of 8; x 16-byte aligned, gamma and y 8-byte aligned (else MT_EINVAL). */
int mtk_rmsnorm_fwd(const void* x, const void* gamma, void* y, void* rstd, int T, int h, float eps, void* stream);

/* Number of rows of the f32 [parts][h] scratch `partial` that mtk_rmsnorm_bwd needs for T rows. */
int mtk_rmsnorm_bwd_parts(int T);

/*
 * RMSNorm backward: dx f32 = dres + rstd*(dy*gamma - xhat*mean(dy*gamma*xhat)), xhat = x*rstd,
 * dy f32 [T,h], dres f32 [T,h] or NULL; dx_bf16 (optional) receives dx rounded to bf16;
 * dgamma bf16 [h] = sum_t dy*xhat, reduced in a fixed order through `partial`.
 * h a multiple of 8. dy, x, dres, dx and partial must be 16-byte aligned, gamma and dx_bf16
 * 8-byte aligned: a row slice at an odd offset is rejected with MT_EINVAL before anything is
 * launched (message in mt_last_error(NULL)).
 */
int mtk_rmsnorm_bwd(const void* dy, const void* x, const void* gamma, const void* rstd, const void* dres, void* dx,
                    void* dx_bf16, void* partial, void* dgamma, int T, int h, void* stream);

/*
 * The same RMSNorm backward with no scratch argument: for callers that cannot allocate
 * device memory where they need this kernel (code under a memory manager that owns the
 * whole device, or paths where the implicit device synchronisation of cudaMalloc/cudaFree
 * is not allowed). The paper has no counterpart of this entry point. It allocates nothing:
 * its scratch is a fixed 9.5 MiB array (304 * 8192 floats) inside the library, held by
 * every GPU that loads it until the process exits. Sizes with min(T, 304) * h above that
 * are rejected with MT_EINVAL (message in mt_last_error(NULL)), and so are pointers that break
 * mtk_rmsnorm_bwd's alignment rule. The first call on a device
 * looks up the array's device address (cudaGetSymbolAddress) with that device current;
 * make that first call before any stream capture. All calls share the array: calls that
 * overlap on the GPU race on it and must be serialised by the caller. Nothing in it needs
 * to start at zero (every element read is written earlier by the same call).
 */
int mtk_rmsnorm_bwd_noalloc(const void* dy, const void* x, const void* gamma, const void* rstd, const void* dres,
                            void* dx, void* dx_bf16, void* dgamma, int T, int h, void* stream);

/*
 * Rotate-half RoPE, in place, on the q and k column ranges of qkv bf16 [T, ld]
 * (columns [0, nh*hd) are q, the next nkv*hd are k). Token t has position t % seq.
 * cos_sin: f32 [seq][hd/2][2]. inverse = 1 applies the transpose (the backward pass).
 */
int mtk_rope(void* qkv, int64_t ld, int T, int seq, int n_heads, int n_kv_heads, int head_dim, const void* cos_sin,
             int inverse, void* stream);

/*
 * Rotary positions in general: scaled frequencies, explicit positions (packed documents), part of
 * the head, both pair layouts. (The pages name no model; mtk_rope is the layer template's form.)
 *
 * mtk_rotary_inv_freq: the frequencies f_i = theta^(-2i/rot_dim), i < rot_dim/2, in radians per
 *   position, scaled for contexts `factor` times longer than the model was trained on. Host only
 *   and pure: inv_freq is a HOST array of rot_dim/2 doubles.
 *     MTK_ROTARY_PLAIN   f_i
 *     MTK_ROTARY_LINEAR  f_i / factor (positions interpolated)
 *     MTK_ROTARY_BASE    the base theta * factor^(rot_dim/(rot_dim-2)) instead of theta (the lowest
 *                        frequency divided by factor, the highest kept); rot_dim > 2
 *     MTK_ROTARY_BANDS   f_i (w + (1-w)/factor), w = (n_i - low)/(high - low) clamped to [0,1],
 *                        n_i = original_positions * f_i / (2 pi) the turns over the trained
 *                        context: high frequencies kept, low ones interpolated, a ramp between
 *                        that is linear in n_i (rules whose ramp is linear in the index i between
 *                        the same ends give other frequencies there; pass those to
 *                        mtk_rotary_table as they are)
 *   MT_EINVAL unless rot_dim is even, 2..256, theta > 0 and, where they are used, factor > 0,
 *   original_positions > 0 and high > low, all finite.
 * mtk_rotary_table: cos_sin f32 [n_pos][rot_dim/2][2] = amplitude * (cos, sin)(p * inv_freq[i]) for
 *   positions p = 0 .. n_pos-1 (amplitude finite). inv_freq is a HOST array, read before the call returns. Angles are
 *   kept modulo whole turns in 64-bit fixed point, so far positions lose nothing.
 * mtk_rotary: y bf16 [T, heads*head_dim] (row stride ldy) = x (row stride ldx) with the first
 *   rot_dim columns of every head rotated: a' = a cos - b sin, b' = b cos + a sin on the pairs
 *   (i, i + rot_dim/2), or (2i, 2i+1) if interleaved; inverse = 1 applies the transpose (the
 *   backward pass). Token t is at positions[t] (int32 [T]), or at t % n_pos if positions is NULL.
 *   y may be x (then ldy = ldx), else they must not overlap. head_dim and rot_dim are multiples
 *   of 16, rot_dim <= head_dim <= 4096, heads <= 65536. A position outside [0, n_pos) sets *err_flag to 8 and
 *   leaves that token unrotated. err_flag: device int, required.
 */
#define MTK_ROTARY_PLAIN 0
#define MTK_ROTARY_LINEAR 1
#define MTK_ROTARY_BASE 2
#define MTK_ROTARY_BANDS 3
int mtk_rotary_inv_freq(int rot_dim, double theta, int scaling, double factor, double original_positions, double low,
                        double high, double* inv_freq);
int mtk_rotary_table(const double* inv_freq, int rot_dim, int n_pos, double amplitude, void* cos_sin, void* stream);
int mtk_rotary(const void* x, int64_t ldx, void* y, int64_t ldy, int T, int heads, int head_dim, int rot_dim,
               int interleaved, const void* positions, const void* cos_sin, int n_pos, int inverse, int* err_flag,
               void* stream);

/*
 * RMSNorm of each query and key head with the rotation in the same pass: for every token and head
 * row x_h (head_dim columns) of the first n_heads + n_kv_heads heads of x,
 *   rstd = 1/sqrt(mean(x_h^2) + eps),  y_h = R(x_h * rstd * g),  g = gq for query heads, gk for keys,
 * with the rotation R of mtk_rotary (rot_dim = 0: no rotation; cos_sin, positions and err_flag may
 * then be NULL). x, y bf16 with row strides ldx, ldy (columns past the key heads, such as v, are
 * neither read nor written); gq, gk bf16 [head_dim]; rstd f32 [T][n_heads + n_kv_heads], or NULL.
 * y may be x (then ldy = ldx), else they must not overlap. head_dim 64 or 128, rot_dim a multiple of
 * 16, at most 65536 heads.
 *
 * mtk_qk_norm_rope_bwd: from dy (row stride lddy), the forward's x and its rstd, with u = R^T dy and
 * n = x_h * rstd: dx_h = rstd (u g - n mean(u g n)), dgq and dgk bf16 [head_dim] = the sums of u n
 * over tokens and query (key) heads, added in a fixed order through `partial`, f32
 * [mtk_qk_norm_rope_bwd_parts(...)][head_dim]. dx may be dy or x (with the same row stride), else it
 * overlaps neither (these are checked; rstd, partial, dgq and dgk have to lie apart from all else).
 * A bad position counts as no rotation, with *err_flag set to 8.
 */
int mtk_qk_norm_rope(const void* x, int64_t ldx, const void* gq, const void* gk, void* y, int64_t ldy, void* rstd,
                     int T, int n_heads, int n_kv_heads, int head_dim, int rot_dim, int interleaved, float eps,
                     const void* positions, const void* cos_sin, int n_pos, int* err_flag, void* stream);
int mtk_qk_norm_rope_bwd_parts(int T, int n_heads, int n_kv_heads, int head_dim);
int mtk_qk_norm_rope_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* gq, const void* gk,
                         const void* rstd, void* dx, int64_t lddx, void* partial, void* dgq, void* dgk, int T,
                         int n_heads, int n_kv_heads, int head_dim, int rot_dim, int interleaved,
                         const void* positions, const void* cos_sin, int n_pos, int* err_flag, void* stream);

/* SwiGLU on gu bf16 [T, 2f] = [g | u]: act bf16 [T,f] = silu(g)*u; backward dgu bf16 [T,2f]. */
int mtk_swiglu_fwd(const void* gu, void* act, int T, int f, void* stream);
int mtk_swiglu_bwd(const void* gu, const void* dact, void* dgu, int T, int f, void* stream);

/*
 * The projections with their pointwise step fused into the GEMM epilogue (what the layer
 * template runs; the unfused kernels above remain for checking each step alone). The fused
 * step works on the f32 accumulator, so results can differ from GEMM-then-kernel by the one
 * bf16 rounding of the intermediate. Deterministic like mtk_gemm_bf16.
 *
 * mtk_gemm_qkv_rope: qkv bf16 [T, (nh+2*nkv)*hd] = a W^T with the q and k heads rotated as
 *   mtk_rope(inverse = 0) does (token t at position t % seq, cos_sin f32 [seq][hd/2][2]);
 *   a bf16 [T,h], w bf16 [(nh+2*nkv)*hd, h]. head_dim 64 or 128.
 * mtk_gemm_swiglu: act bf16 [T,f] = silu(g)*u with g = bf16(b Wg^T), u = bf16(b Wu^T);
 *   b bf16 [T,h], wgu bf16 [2f, h] = [Wg; Wu]; gu (NULL or bf16 [T,2f]) receives [g | u].
 *   f a multiple of 8.
 * mtk_gemm_swiglu_bwd: dact = dy Wd (dy bf16 [T,h], wd bf16 [h,f]) and, from gu bf16 [T,2f] =
 *   [g | u], dgu bf16 [T,2f] = [dact*u*s*(1+g*(1-s)) | dact*g*s], s = sigmoid(g).
 *   f a multiple of 8.
 */
int mtk_gemm_qkv_rope(const void* a, const void* w, void* qkv, const void* cos_sin, int T, int h, int n_heads,
                      int n_kv_heads, int head_dim, int seq, int* err_flag, void* stream);
int mtk_gemm_swiglu(const void* b, const void* wgu, void* act, void* gu, int T, int h, int f, int* err_flag,
                    void* stream);
int mtk_gemm_swiglu_bwd(const void* dy, const void* wd, const void* gu, void* dgu, int T, int h, int f, int* err_flag,
                        void* stream);

/* Embedding gather x f32 [T,h] = E bf16 [V,h] rows tok[t]. */
int mtk_embed_fwd(const void* tok, const void* E, void* x, int T, int h, void* stream);
/* dE bf16 [V,h]: row v = sum of dx f32 rows order[offsets[v]..offsets[v+1]) in that order. */
int mtk_embed_bwd(const void* order, const void* offsets, const void* dx, void* dE, int V, int h, void* stream);

/*
 * Cross-entropy over logits f32 [T,V] with labels int32 [T]:
 * row_loss f32 [T] = logsumexp(z_t) - z_t[label_t]; dlogits bf16 [T,V] = (softmax(z_t) - onehot)/T;
 * loss f32 [1] = mean of row_loss (fixed-order reduction).
 */
int mtk_cross_entropy(const void* logits, const void* labels, void* dlogits, void* row_loss, void* loss, int T, int V,
                      void* stream);

/*
 * Causal grouped-query flash attention on qkv bf16 [B*s, (nh+2*nkv)*hd] (q | k | v), on the
 * tcgen05 tensor cores. o bf16 [B*s, nh*hd]; lse f32 [B, nh, s] = log2 of the softmax
 * denominator of the scores scaled by log2(e)/sqrt(hd), plus the max it was taken against.
 * head_dim is 64 or 128. err_flag: device int, required (bounded internal waits).
 */
int mtk_attn_fwd(const void* qkv, void* o, void* lse, int B, int s, int nh, int nkv, int head_dim, int* err_flag,
                 void* stream);
/* Backward on the tcgen05 tensor cores, deterministic (KV-outer dK/dV, Q-outer dQ, no atomics):
 * dqkv bf16 (layout of qkv) from dout bf16 [B*s, nh*hd]. delta: f32 scratch of
 * B * nh * s128 * 2 floats, s128 = s rounded up to a multiple of 128, 16-byte aligned; it receives
 * (lse2, rowsum(dO * O)) per query row. err_flag: device int, required. */
int mtk_attn_bwd(const void* qkv, const void* o, const void* lse, const void* dout, void* dqkv, void* delta, int B,
                 int s, int nh, int nkv, int head_dim, int* err_flag, void* stream);
/* The same backward with the RoPE backward fused into its output: dq and dk are written with the
 * transpose rotation of mtk_rope(inverse = 1) applied (cos_sin f32 [s][hd/2][2], position = row
 * index within the sequence), which is what the layer template needs when RoPE was applied to q
 * and k after the QKV projection. dv is unchanged. */
int mtk_attn_bwd_rope(const void* qkv, const void* o, const void* lse, const void* dout, void* dqkv, void* delta,
                      const void* cos_sin, int B, int s, int nh, int nkv, int head_dim, int* err_flag, void* stream);

/*
 * Attention over spans: self-attention in which query row i of its sequence sees the keys
 * lo[i] <= j < hi[i], which covers causal, document, prefix and two-sided masks and padding. (An
 * addition to the layer template's causal attention; the pages name no model.)
 *   z_ij = scale q_i.k_j;  cap > 0: z = cap tanh(z / cap);  slopes: z -= slopes[head] |i - j|;
 *   p_i = softmax of z_i over the span, o_i = sum_j p_ij v_j.
 * q bf16 [B*s, nh*hd], k and v bf16 [B*s, nkv*hd] with row strides ldq, ldk, ldv (any column ranges
 * of wider buffers); lo, hi int32 [B*s], positions inside the sequence, or NULL (lo 0, hi i + 1:
 * causal); they are clamped to [0, s]. nkv divides nh, head_dim 64 or 128, s <= 4194304. scale > 0,
 * cap >= 0 (0: none), slopes f32 [nh] or NULL, all finite; capped scores are right to about cap * 2^-22
 * (relative 2^-22 while they stay below the cap before it is applied). Capped up to 50.5 without slopes, v is
 * taken to lie between 2^-40 and 2^40 in size (or 0): beyond, products with the unnormalised
 * probabilities may leave fp32.
 * An empty span (lo >= hi) makes row i padding: o_i = 0, lse_i = -inf, its gradients are 0, and no
 * other row's span may contain it. Padding rows of q, k, v and dout may hold anything, NaN
 * included, where the padding follows the documents of its sequence, precedes them, or lies between
 * documents that are contiguous; all other rows must be finite.
 *
 * mtk_doc_spans: spans and positions of packed documents. HOST arrays, pure: documents d = 0 ..
 *   n_docs-1 are the tokens bounds[d] <= t < bounds[d+1] of the B*s tokens (bounds int32
 *   [n_docs+1], not decreasing; empty documents are allowed; tokens outside are padding). A document
 *   that crosses the end of a sequence is cut there into two. Token t of a document part that starts
 *   at t0 gets lo = t0, hi = max(t + 1, t0 + prefix[d]) up to the part's end, both inside the
 *   sequence, and position t - t0. prefix int32 [n_docs] >= 0 or NULL (0: causal; the document's
 *   length: two-sided). lo, hi int32 [B*s], positions int32 [B*s] or NULL; B*s < 2^31.
 * The row matrices written (o; dq, dk, dv) may be column ranges of one buffer with the ones read or each other
 * but share no element with them: MT_EINVAL, also where they only might, their strides being different and the
 * memory from first to last element the same. lse, lo, hi, slopes, scratch and err_flag lie apart from all that
 * is written, which is not checked.
 * mtk_attn_span_fwd: o bf16 [B*s, nh*hd] (row stride ldo), lse f32 [B, nh, s] in mtk_attn_fwd's
 *   units (log2). err_flag: device int, required, as for all attention entries.
 * mtk_attn_span_bwd: dq bf16 [B*s, nh*hd], dk, dv bf16 [B*s, nkv*hd] (row strides lddq, lddk, lddv;
 *   every row is written) from dout, o and lse, deterministic, no atomics. scratch: device memory of
 *   mtk_attn_span_bwd_scratch_bytes() bytes, 16-byte aligned, not shared by calls that may run at the same
 *   time. (s rounded up to a multiple of 128) * (nh / nkv) <= 2^26. Gradients of slopes are not computed.
 */
int mtk_doc_spans(const int32_t* bounds, int n_docs, const int32_t* prefix, int B, int s, int32_t* lo, int32_t* hi,
                  int32_t* positions);
int mtk_attn_span_fwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                      const void* lo, const void* hi, void* o, int64_t ldo, void* lse, int B, int s, int nh, int nkv,
                      int head_dim, float scale, float cap, const void* slopes, int* err_flag, void* stream);
uint64_t mtk_attn_span_bwd_scratch_bytes(int B, int s, int nh, int nkv, int head_dim);
int mtk_attn_span_bwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                      const void* lo, const void* hi, const void* o, int64_t ldo, const void* lse, const void* dout,
                      int64_t lddo, void* dq, int64_t lddq, void* dk, int64_t lddk, void* dv, int64_t lddv,
                      void* scratch, int B, int s, int nh, int nkv, int head_dim, float scale, float cap,
                      const void* slopes, int* err_flag, void* stream);

/* Block order of the causal attention grids (host-only, pure; no GPU needed). The forward, dQ
 * and dK/dV grids are one-dimensional with n_tiles * n_hb blocks (n_tiles 128-row tiles per
 * sequence; n_hb = heads * batch, KV heads for dK/dV). Block `lin` works on tile rank *rank
 * (0 = the heaviest tile of its head: the last query tile, or the first key tile) of head pair
 * *hb = head + heads * batch. Blocks take ranks heaviest first over groups of 16 head pairs.
 * Returns MT_EINVAL unless 0 <= lin < n_tiles * n_hb and both pointers are set. */
int mtk_attn_block_slot(int lin, int n_tiles, int n_hb, int* rank, int* hb);

/*
 * Self-check of the kernels' bounded waits: one thread waits, through the same wait routine the
 * GEMM and attention pipelines use, on an mbarrier phase that never completes. After limit_ns
 * (0 .. 4e9, the pipelines' own limit) it gives up, stores code 6 in *err_flag (unless a wait's code
 * is already there), writes *gave_up = 1 and returns; no copy or MMA is in flight. This is how a
 * stalled pipeline ends instead of hanging the GPU: the host reads the flag after the step
 * (mt_train_step returns MT_EKERNEL) and the context stays usable. err_flag and gave_up are
 * device ints; the call only enqueues.
 */
int mtk_bounded_wait_check(int* err_flag, int* gave_up, int64_t limit_ns, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MT_KERNELS_H */
