// C ABI of the individual layer-template kernels (declared in include/mt_kernels.h).
// Argument checking happens here; the launchers in kernels.h enqueue the work.
#include <atomic>
#include <string>

#include "kernels.h"
#include "mt.h"
#include "mt_kernels.h"
#include "ptx.cuh"
#include "tile_order.cuh"

using mt::bf16;

namespace {
// One thread waits, through the same bounded wait every pipeline kernel uses, for a phase of an
// mbarrier that nothing ever arrives on. No copy or MMA is in flight, so giving up is all it does.
__global__ void bounded_wait_check_kernel(int* err, unsigned long long limit_ns, int* gave_up) {
  __shared__ uint64_t bar;
  mt::mbar_init(&bar, 1);
  mt::fence_mbar_init();
  const bool ok = mt::mbar_wait_limit(&bar, 0, err, mt::kErrTimeoutProbe, limit_ns);
  *gave_up = ok ? 0 : 1;
}
}  // namespace

namespace {
inline cudaStream_t S(void* s) { return reinterpret_cast<cudaStream_t>(s); }
inline int rc(cudaError_t e) {
  if (e == cudaSuccess) return MT_OK;
  if (e == cudaErrorInvalidValue || e == cudaErrorMisalignedAddress) return MT_EINVAL;
  return MT_ECUDA;
}
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
mt::AttnSpanArgs span_args(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                           const void* lo, const void* hi, int B, int s, int nh, int nkv, int hd, float scale,
                           float cap, const void* slopes) {
  return {static_cast<const bf16*>(q), static_cast<const bf16*>(k), static_cast<const bf16*>(v), ldq, ldk, ldv, B, s,
          nh, nkv, hd, static_cast<const int32_t*>(lo), static_cast<const int32_t*>(hi), scale, cap,
          static_cast<const float*>(slopes)};
}
std::atomic<void*> g_gemm_ws{nullptr};  // workspace of the mtk_gemm_* calls (mtk_gemm_use_workspace)
}  // namespace

void mt_set_global_error(const std::string& m);  // message for mt_last_error(NULL)
extern const char* const kRmsBwdAlignMsg;
const char* const kRmsBwdAlignMsg =
    "rmsnorm backward: dy, x, dres, dx and the scratch must be 16-byte aligned, gamma and dx_bf16 8-byte aligned";

extern "C" {

uint64_t mtk_gemm_workspace_bytes(void) { return mt::gemm_workspace_bytes(); }
uint64_t mtk_gemm_workspace_clear_bytes(void) { return mt::kGemmFlagBytes; }

int mtk_gemm_use_workspace(void* ws) {
  if (ws && !aligned16(ws)) return MT_EINVAL;
  g_gemm_ws.store(ws);
  return MT_OK;
}

int mtk_gemm_bf16(const void* A, int64_t lda, int a_mn, const void* B, int64_t ldb, int b_mn, void* C, int64_t ldc,
                  const void* R, int64_t ldr, int M, int N, int K, int epi, int* err_flag, void* stream) {
  if (!A || !B || !C || !err_flag || M <= 0 || N <= 0 || K <= 0) return MT_EINVAL;
  if (epi < MTK_EPI_STORE_BF16 || epi > MTK_EPI_ADD_F32 || (epi == MTK_EPI_ADD_F32 && !R)) return MT_EINVAL;
  if ((a_mn ? lda < M : lda < K) || (b_mn ? ldb < N : ldb < K) || ldc < N) return MT_EINVAL;
  mt::GemmArgs g;
  g.A = static_cast<const bf16*>(A);
  g.lda = lda;
  g.a_mn = a_mn != 0;
  g.B = static_cast<const bf16*>(B);
  g.ldb = ldb;
  g.b_mn = b_mn != 0;
  g.C = C;
  g.ldc = ldc;
  g.R = static_cast<const float*>(R);
  g.ldr = ldr;
  g.M = M;
  g.N = N;
  g.K = K;
  g.epi = epi;
  g.ws = g_gemm_ws.load();
  return rc(mt::gemm(g, err_flag, S(stream)));
}

int mtk_gemm_qkv_rope(const void* a, const void* w, void* qkv, const void* cos_sin, int T, int h, int n_heads,
                      int n_kv_heads, int head_dim, int seq, int* err_flag, void* stream) {
  if (!a || !w || !qkv || !cos_sin || !err_flag || T <= 0 || h <= 0 || n_heads <= 0 || n_kv_heads <= 0 || seq <= 0 ||
      (head_dim != 64 && head_dim != 128))
    return MT_EINVAL;
  const int n = (n_heads + 2 * n_kv_heads) * head_dim;
  mt::GemmArgs g{static_cast<const bf16*>(a), h, false, static_cast<const bf16*>(w), h, false, qkv, n, nullptr, 0,
                 T, n, h, mt::kEpiRopeBf16};
  g.cs = static_cast<const float*>(cos_sin);
  g.rope_cols = (n_heads + n_kv_heads) * head_dim;
  g.hd = head_dim;
  g.seq = seq;
  g.ws = g_gemm_ws.load();
  return rc(mt::gemm(g, err_flag, S(stream)));
}

int mtk_gemm_swiglu(const void* b, const void* wgu, void* act, void* gu, int T, int h, int f, int* err_flag,
                    void* stream) {
  if (!b || !wgu || !act || !err_flag || T <= 0 || h <= 0 || f <= 0 || f % 8) return MT_EINVAL;
  mt::GemmArgs g{static_cast<const bf16*>(b), h, false, static_cast<const bf16*>(wgu), h, false, act, f, nullptr, 0,
                 T, f, h, mt::kEpiSwigluBf16};
  g.C2 = gu;
  g.ldc2 = 2 * static_cast<int64_t>(f);
  g.ws = g_gemm_ws.load();
  return rc(mt::gemm(g, err_flag, S(stream)));
}

int mtk_gemm_swiglu_bwd(const void* dy, const void* wd, const void* gu, void* dgu, int T, int h, int f, int* err_flag,
                        void* stream) {
  if (!dy || !wd || !gu || !dgu || !err_flag || T <= 0 || h <= 0 || f <= 0 || f % 8) return MT_EINVAL;
  mt::GemmArgs g{static_cast<const bf16*>(dy), h, false, static_cast<const bf16*>(wd), f, true, dgu, 2 * f, nullptr,
                 0, T, f, h, mt::kEpiSwigluBwdBf16};
  g.G = static_cast<const bf16*>(gu);
  g.ldg = 2 * static_cast<int64_t>(f);
  g.ws = g_gemm_ws.load();
  return rc(mt::gemm(g, err_flag, S(stream)));
}

int mtk_rmsnorm_fwd(const void* x, const void* gamma, void* y, void* rstd, int T, int h, float eps, void* stream) {
  if (!x || !gamma || !y || !rstd || T <= 0 || h <= 0 || !aligned16(x) || !aligned16(y)) return MT_EINVAL;
  return rc(mt::rmsnorm_fwd(static_cast<const float*>(x), static_cast<const bf16*>(gamma), static_cast<bf16*>(y),
                            static_cast<float*>(rstd), T, h, eps, S(stream)));
}

int mtk_rmsnorm_bwd_parts(int T) { return T > 0 ? mt::rmsnorm_bwd_parts(T) : 0; }

int mtk_rmsnorm_bwd(const void* dy, const void* x, const void* gamma, const void* rstd, const void* dres, void* dx,
                    void* dx_bf16, void* partial, void* dgamma, int T, int h, void* stream) {
  if (!dy || !x || !gamma || !rstd || !dx || !partial || !dgamma || T <= 0 || h <= 0) return MT_EINVAL;
  if (!mt::rmsnorm_bwd_aligned(static_cast<const float*>(dy), static_cast<const float*>(x),
                               static_cast<const bf16*>(gamma), static_cast<const float*>(dres),
                               static_cast<const float*>(dx), static_cast<const bf16*>(dx_bf16),
                               static_cast<const float*>(partial))) {
    mt_set_global_error(kRmsBwdAlignMsg);
    return MT_EINVAL;
  }
  return rc(mt::rmsnorm_bwd(static_cast<const float*>(dy), static_cast<const float*>(x),
                            static_cast<const bf16*>(gamma), static_cast<const float*>(rstd),
                            static_cast<const float*>(dres), static_cast<float*>(dx), static_cast<bf16*>(dx_bf16),
                            static_cast<float*>(partial), static_cast<bf16*>(dgamma), T, h, S(stream)));
}

int mtk_rope(void* qkv, int64_t ld, int T, int seq, int n_heads, int n_kv_heads, int head_dim, const void* cos_sin,
             int inverse, void* stream) {
  if (!qkv || !cos_sin || T <= 0 || seq <= 0 || n_heads <= 0 || n_kv_heads <= 0) return MT_EINVAL;
  if (ld < static_cast<int64_t>(n_heads + n_kv_heads) * head_dim) return MT_EINVAL;
  return rc(mt::rope(static_cast<bf16*>(qkv), ld, T, seq, n_heads, n_kv_heads, head_dim,
                     static_cast<const float*>(cos_sin), inverse != 0, S(stream)));
}

int mtk_rotary_inv_freq(int rot_dim, double theta, int scaling, double factor, double original_positions, double low,
                        double high, double* inv_freq) {
  return mt::rotary_inv_freq(rot_dim, theta, scaling, factor, original_positions, low, high, inv_freq) ? MT_OK
                                                                                                       : MT_EINVAL;
}

int mtk_rotary_table(const double* inv_freq, int rot_dim, int n_pos, double amplitude, void* cos_sin, void* stream) {
  if (!inv_freq || !cos_sin) return MT_EINVAL;
  return rc(mt::rotary_table(inv_freq, rot_dim, n_pos, amplitude, static_cast<float*>(cos_sin), S(stream)));
}

int mtk_rotary(const void* x, int64_t ldx, void* y, int64_t ldy, int T, int heads, int head_dim, int rot_dim,
               int interleaved, const void* positions, const void* cos_sin, int n_pos, int inverse, int* err_flag,
               void* stream) {
  if (!x || !y) return MT_EINVAL;
  return rc(mt::rotary(static_cast<const bf16*>(x), ldx, static_cast<bf16*>(y), ldy, T, heads, head_dim, rot_dim,
                       interleaved != 0, static_cast<const int32_t*>(positions), static_cast<const float*>(cos_sin),
                       n_pos, inverse != 0, err_flag, S(stream)));
}

int mtk_qk_norm_rope(const void* x, int64_t ldx, const void* gq, const void* gk, void* y, int64_t ldy, void* rstd,
                     int T, int n_heads, int n_kv_heads, int head_dim, int rot_dim, int interleaved, float eps,
                     const void* positions, const void* cos_sin, int n_pos, int* err_flag, void* stream) {
  if (!x || !gq || !gk || !y || !(eps >= 0.f)) return MT_EINVAL;
  return rc(mt::qk_norm_rope(static_cast<const bf16*>(x), ldx, static_cast<const bf16*>(gq),
                             static_cast<const bf16*>(gk), static_cast<bf16*>(y), ldy, static_cast<float*>(rstd), T,
                             n_heads, n_kv_heads, head_dim, rot_dim, interleaved != 0, eps,
                             static_cast<const int32_t*>(positions), static_cast<const float*>(cos_sin), n_pos,
                             err_flag, S(stream)));
}

int mtk_qk_norm_rope_bwd_parts(int T, int n_heads, int n_kv_heads, int head_dim) {
  if (T <= 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads > mt::kRotaryMaxHeads - n_kv_heads ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return mt::qk_norm_rope_bwd_parts(T, n_heads, n_kv_heads, head_dim);
}

int mtk_qk_norm_rope_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* gq, const void* gk,
                         const void* rstd, void* dx, int64_t lddx, void* partial, void* dgq, void* dgk, int T,
                         int n_heads, int n_kv_heads, int head_dim, int rot_dim, int interleaved,
                         const void* positions, const void* cos_sin, int n_pos, int* err_flag, void* stream) {
  if (!dy || !x || !gq || !gk || !rstd || !dx || !partial || !dgq || !dgk) return MT_EINVAL;
  return rc(mt::qk_norm_rope_bwd(static_cast<const bf16*>(dy), lddy, static_cast<const bf16*>(x), ldx,
                                 static_cast<const bf16*>(gq), static_cast<const bf16*>(gk),
                                 static_cast<const float*>(rstd), static_cast<bf16*>(dx), lddx,
                                 static_cast<float*>(partial), static_cast<bf16*>(dgq), static_cast<bf16*>(dgk), T,
                                 n_heads, n_kv_heads, head_dim, rot_dim, interleaved != 0,
                                 static_cast<const int32_t*>(positions), static_cast<const float*>(cos_sin), n_pos,
                                 err_flag, S(stream)));
}

int mtk_swiglu_fwd(const void* gu, void* act, int T, int f, void* stream) {
  if (!gu || !act || T <= 0 || f <= 0) return MT_EINVAL;
  return rc(mt::swiglu_fwd(static_cast<const bf16*>(gu), static_cast<bf16*>(act), T, f, S(stream)));
}

int mtk_swiglu_bwd(const void* gu, const void* dact, void* dgu, int T, int f, void* stream) {
  if (!gu || !dact || !dgu || T <= 0 || f <= 0) return MT_EINVAL;
  return rc(mt::swiglu_bwd(static_cast<const bf16*>(gu), static_cast<const bf16*>(dact), static_cast<bf16*>(dgu), T,
                           f, S(stream)));
}

int mtk_embed_fwd(const void* tok, const void* E, void* x, int T, int h, void* stream) {
  if (!tok || !E || !x || T <= 0 || h <= 0) return MT_EINVAL;
  return rc(mt::embed_fwd(static_cast<const int32_t*>(tok), static_cast<const bf16*>(E), static_cast<float*>(x), T, h,
                          S(stream)));
}

int mtk_embed_bwd(const void* order, const void* offsets, const void* dx, void* dE, int V, int h, void* stream) {
  if (!order || !offsets || !dx || !dE || V <= 0 || h <= 0) return MT_EINVAL;
  return rc(mt::embed_bwd(static_cast<const int32_t*>(order), static_cast<const int32_t*>(offsets),
                          static_cast<const float*>(dx), static_cast<bf16*>(dE), V, h, S(stream)));
}

int mtk_cross_entropy(const void* logits, const void* labels, void* dlogits, void* row_loss, void* loss, int T, int V,
                      void* stream) {
  if (!logits || !labels || !dlogits || !row_loss || !loss || T <= 0 || V <= 0) return MT_EINVAL;
  cudaError_t e = mt::cross_entropy(static_cast<const float*>(logits), static_cast<const int32_t*>(labels),
                                    static_cast<bf16*>(dlogits), static_cast<float*>(row_loss), T, V, S(stream));
  if (e != cudaSuccess) return rc(e);
  return rc(mt::mean_reduce(static_cast<const float*>(row_loss), T, static_cast<float*>(loss), S(stream)));
}

int mtk_token_logprobs(const void* logits, int type, int64_t ld, const void* labels, void* logp, void* lse, int T,
                       int V, float scale, int* err_flag, void* stream) {
  return rc(mt::token_logprobs(logits, type, ld, static_cast<const int32_t*>(labels), static_cast<float*>(logp),
                               static_cast<float*>(lse), T, V, scale, err_flag, S(stream)));
}

int mtk_token_logprobs_bwd(const void* logits, int type, int64_t ld, const void* labels, const void* lse,
                           const void* dlogp, void* dlogits, int64_t ldd, int T, int V, float scale, void* stream) {
  return rc(mt::token_logprobs_bwd(logits, type, ld, static_cast<const int32_t*>(labels),
                                   static_cast<const float*>(lse), static_cast<const float*>(dlogp),
                                   static_cast<bf16*>(dlogits), ldd, T, V, scale, S(stream)));
}

int mtk_policy_loss(const void* logits, int type, int64_t ld, const void* labels, const void* old_logp,
                    const void* advantages, const void* ref_logp, const void* weights, float clip_low, float clip_high,
                    float kl, float scale, void* dlogits, int64_t ldd, void* logp, void* row_loss, void* loss, int T,
                    int V, int* err_flag, void* stream) {
  return rc(mt::policy_loss(logits, type, ld, static_cast<const int32_t*>(labels),
                            static_cast<const float*>(old_logp), static_cast<const float*>(advantages),
                            static_cast<const float*>(ref_logp), static_cast<const float*>(weights), clip_low,
                            clip_high, kl, scale, static_cast<bf16*>(dlogits), ldd, static_cast<float*>(logp),
                            static_cast<float*>(row_loss), static_cast<float*>(loss), T, V, err_flag, S(stream)));
}

int mtk_preference_loss(const void* logp, const void* ref_logp, const void* labels, const void* bounds, int pairs,
                        int T, int kind, float beta, float margin, float smoothing, int average, void* pair_loss,
                        void* loss, void* rewards, void* dlogp, void* stream) {
  return rc(mt::preference_loss(static_cast<const float*>(logp), static_cast<const float*>(ref_logp),
                                static_cast<const int32_t*>(labels), static_cast<const int32_t*>(bounds), pairs, T,
                                kind, beta, margin, smoothing, average != 0, static_cast<float*>(pair_loss),
                                static_cast<float*>(loss), static_cast<float*>(rewards), static_cast<float*>(dlogp),
                                S(stream)));
}

int mtk_layernorm_fwd(const void* x, int type, int64_t ldx, const void* gamma, const void* beta, void* y, int64_t ldy,
                      void* mean, void* rstd, int T, int h, float eps, void* stream) {
  return rc(mt::layernorm_fwd(x, type, ldx, static_cast<const bf16*>(gamma), static_cast<const bf16*>(beta),
                              static_cast<bf16*>(y), ldy, static_cast<float*>(mean), static_cast<float*>(rstd), T, h,
                              eps, S(stream)));
}

int mtk_layernorm_bwd_parts(int T, int h) { return mt::layernorm_bwd_parts(T, h); }

int mtk_layernorm_bwd(const void* dy, int dy_type, int64_t lddy, const void* x, int type, int64_t ldx,
                      const void* gamma, const void* mean, const void* rstd, const void* dres, int64_t lddres,
                      void* dx, void* dx_bf16, void* partial, void* dgamma, void* dbeta, int T, int h, void* stream) {
  return rc(mt::layernorm_bwd(dy, dy_type, lddy, x, type, ldx, static_cast<const bf16*>(gamma),
                              static_cast<const float*>(mean), static_cast<const float*>(rstd), dres, lddres, dx,
                              static_cast<bf16*>(dx_bf16), static_cast<float*>(partial), static_cast<bf16*>(dgamma),
                              static_cast<bf16*>(dbeta), T, h, S(stream)));
}

int mtk_embed_lookup(const void* tok, const void* E, void* x, int type, int T, int h, int V, float scale,
                     int* err_flag, void* stream) {
  return rc(mt::embed_lookup(static_cast<const int32_t*>(tok), static_cast<const bf16*>(E), x, type, T, h, V, scale,
                             err_flag, S(stream)));
}

uint64_t mtk_embed_lookup_bwd_scratch_bytes(int T, int h) {
  if (T <= 0 || T > mt::kEmbedMaxTokens || h <= 0 || h > mt::kEmbedMaxWidth) return 0;
  return mt::embed_lookup_bwd_scratch(T, h);
}

int mtk_embed_lookup_bwd(const void* tok, const void* dx, int type, void* dE, void* scratch, int T, int h, int V,
                         float scale, int accumulate, int* err_flag, void* stream) {
  return rc(mt::embed_lookup_bwd(static_cast<const int32_t*>(tok), dx, type, static_cast<bf16*>(dE), scratch, T, h, V,
                                 scale, accumulate != 0, err_flag, S(stream)));
}

int mtk_attn_fwd(const void* qkv, void* o, void* lse, int B, int s, int nh, int nkv, int head_dim, int* err_flag,
                 void* stream) {
  if (!qkv || !o || !lse || !err_flag || B <= 0 || s <= 0) return MT_EINVAL;
  return rc(mt::attn_fwd(static_cast<const bf16*>(qkv), static_cast<bf16*>(o), static_cast<float*>(lse), B, s, nh, nkv,
                         head_dim, err_flag, S(stream)));
}

int mtk_attn_bwd(const void* qkv, const void* o, const void* lse, const void* dout, void* dqkv, void* delta, int B,
                 int s, int nh, int nkv, int head_dim, int* err_flag, void* stream) {
  if (!qkv || !o || !lse || !dout || !dqkv || !delta || !err_flag || B <= 0 || s <= 0) return MT_EINVAL;
  return rc(mt::attn_bwd(static_cast<const bf16*>(qkv), static_cast<const bf16*>(o), static_cast<const float*>(lse),
                         static_cast<const bf16*>(dout), static_cast<bf16*>(dqkv), static_cast<float*>(delta), nullptr,
                         B, s, nh, nkv, head_dim, err_flag, S(stream)));
}

int mtk_attn_bwd_rope(const void* qkv, const void* o, const void* lse, const void* dout, void* dqkv, void* delta,
                      const void* cos_sin, int B, int s, int nh, int nkv, int head_dim, int* err_flag, void* stream) {
  if (!qkv || !o || !lse || !dout || !dqkv || !delta || !cos_sin || !err_flag || B <= 0 || s <= 0) return MT_EINVAL;
  return rc(mt::attn_bwd(static_cast<const bf16*>(qkv), static_cast<const bf16*>(o), static_cast<const float*>(lse),
                         static_cast<const bf16*>(dout), static_cast<bf16*>(dqkv), static_cast<float*>(delta),
                         static_cast<const float*>(cos_sin), B, s, nh, nkv, head_dim, err_flag, S(stream)));
}

int mtk_doc_spans(const int32_t* bounds, int n_docs, const int32_t* prefix, int B, int s, int32_t* lo, int32_t* hi,
                  int32_t* positions) {
  return mt::doc_spans(bounds, n_docs, prefix, B, s, lo, hi, positions) ? MT_OK : MT_EINVAL;
}

int mtk_attn_span_fwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                      const void* lo, const void* hi, void* o, int64_t ldo, void* lse, int B, int s, int nh, int nkv,
                      int head_dim, float scale, float cap, const void* slopes, int* err_flag, void* stream) {
  return rc(mt::attn_span_fwd(span_args(q, ldq, k, ldk, v, ldv, lo, hi, B, s, nh, nkv, head_dim, scale, cap, slopes),
                              static_cast<bf16*>(o), ldo, static_cast<float*>(lse), err_flag, S(stream)));
}

uint64_t mtk_attn_span_bwd_scratch_bytes(int B, int s, int nh, int nkv, int head_dim) {
  if (B <= 0 || s <= 0 || s > mt::kSpanMaxSeq || nh <= 0 || nkv <= 0 || head_dim <= 0) return 0;
  return mt::attn_span_bwd_scratch(B, s, nh, nkv, head_dim);
}

int mtk_attn_span_bwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                      const void* lo, const void* hi, const void* o, int64_t ldo, const void* lse, const void* dout,
                      int64_t lddo, void* dq, int64_t lddq, void* dk, int64_t lddk, void* dv, int64_t lddv,
                      void* scratch, int B, int s, int nh, int nkv, int head_dim, float scale, float cap,
                      const void* slopes, int* err_flag, void* stream) {
  return rc(mt::attn_span_bwd(span_args(q, ldq, k, ldk, v, ldv, lo, hi, B, s, nh, nkv, head_dim, scale, cap, slopes),
                              static_cast<const bf16*>(o), ldo, static_cast<const float*>(lse),
                              static_cast<const bf16*>(dout), lddo, static_cast<bf16*>(dq), lddq,
                              static_cast<bf16*>(dk), lddk, static_cast<bf16*>(dv), lddv, scratch, err_flag,
                              S(stream)));
}

int mtk_bounded_wait_check(int* err_flag, int* gave_up, int64_t limit_ns, void* stream) {
  if (!err_flag || !gave_up || limit_ns < 0 || limit_ns > static_cast<int64_t>(mt::kWaitLimitNs)) return MT_EINVAL;
  bounded_wait_check_kernel<<<1, 1, 0, S(stream)>>>(err_flag, static_cast<unsigned long long>(limit_ns), gave_up);
  return rc(cudaGetLastError());
}

int mtk_attn_block_slot(int lin, int n_tiles, int n_hb, int* rank, int* hb) {
  if (!rank || !hb || n_tiles <= 0 || n_hb <= 0 || lin < 0 ||
      static_cast<int64_t>(lin) >= static_cast<int64_t>(n_tiles) * n_hb)
    return MT_EINVAL;
  const mt::TileSlot s = mt::heavy_first_slot(lin, n_tiles, n_hb);
  *rank = s.rank;
  *hb = s.hb;
  return MT_OK;
}

}  // extern "C"
