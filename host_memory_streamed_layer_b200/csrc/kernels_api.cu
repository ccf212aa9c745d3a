// C-ABI entry points of the individual kernels (declared in mt_kernels.h).
#include "act_dropout.cuh"
#include "mt_internal.h"
#include "mt_kernels.h"

extern "C" int mt_k_gemm_bf16(const void* A, int64_t lda, int a_mn_major, const void* B, int64_t ldb,
                              int b_mn_major, void* C, int64_t ldc, int out_kind, const float* R, int64_t ldr,
                              int M, int N, int K, void* stream, int32_t* dev_err) {
  if (out_kind < MT_GEMM_OUT_BF16 || out_kind > MT_GEMM_OUT_F32_ADD) return MT_ERR_ARG;
  if (M < 0 || N < 0 || K < 0) return MT_ERR_ARG;
  mt::GemmDesc g{A, lda, a_mn_major != 0, B, ldb, b_mn_major != 0, C, ldc, out_kind, R, ldr, M, N, K, mt::RopeDesc{}};
  return mt::gemm_bf16(g, static_cast<cudaStream_t>(stream), dev_err);
}

extern "C" int64_t mt_k_gemm_wait_limit_ns(int64_t ns) {
  if (ns < 0) {
    const uint64_t cur = mt::gemm_wait_limit_ns(0);
    mt::gemm_wait_limit_ns(cur);
    return (int64_t)cur;
  }
  return (int64_t)mt::gemm_wait_limit_ns((uint64_t)ns);
}

extern "C" int mt_k_gemm_variant(int variant) {
  if (variant < 0 || variant > 2) return MT_ERR_ARG;
  return mt::gemm_variant(variant);
}

extern "C" int mt_k_attn_fwd_variant(int variant) {
  if (variant < 0 || variant > 2) return MT_ERR_ARG;
  return mt::attention_fwd_variant(variant);
}

extern "C" int mt_k_attn_bwd_variant(int variant) {
  if (variant < 0 || variant > 2) return MT_ERR_ARG;
  return mt::attention_bwd_variant(variant);
}

#include <cmath>

namespace {
inline cudaStream_t S(void* p) { return static_cast<cudaStream_t>(p); }
inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
}  // namespace

extern "C" int mt_k_rmsnorm_fwd(const float* x, const void* g, void* y, float* rstd, int T, int d, float eps,
                                void* stream) {
  if (!x || !g || !y || T < 0 || d <= 0 || (d % 4)) return MT_ERR_ARG;
  return mt::launch_rmsnorm_fwd(x, g, y, rstd, T, d, eps, S(stream));
}

extern "C" size_t mt_k_rmsnorm_bwd_partial_floats(int T, int d) {
  return (size_t)mt::rmsnorm_bwd_blocks(T) * (size_t)d;
}

extern "C" int mt_k_rmsnorm_bwd(const float* x, const void* g, const float* rstd, const float* dy, const float* dres,
                                float* dx, void* dx_bf16, float* dg_part, float* dg, int T, int d, void* stream) {
  if (!x || !g || !rstd || !dy || !dx || !dg_part || !dg || T < 0 || d <= 0 || (d % 4) || d > 8192)
    return MT_ERR_ARG;
  return mt::launch_rmsnorm_bwd(x, g, rstd, dy, dres, dx, dx_bf16, dg_part, dg, T, d, S(stream));
}

extern "C" int mt_k_rope(void* buf, int64_t ld, int T, int s, int nheads, int hd, int col0, const float* cos_tab,
                         const float* sin_tab, float sign, void* stream) {
  if (!buf || !cos_tab || !sin_tab || T < 0 || s <= 0 || nheads < 0 || hd <= 0 || (hd % 4) || (col0 % 2) ||
      (ld % 2))
    return MT_ERR_ARG;
  return mt::launch_rope(buf, ld, T, s, nheads, hd, col0, cos_tab, sin_tab, sign, S(stream));
}

extern "C" int mt_k_swiglu_fwd(const void* gu, void* act, int T, int F, void* stream) {
  if (!gu || !act || T < 0 || F <= 0 || (F % 8) || !al16(gu) || !al16(act)) return MT_ERR_ARG;
  return mt::launch_swiglu_fwd(gu, act, T, F, S(stream));
}

extern "C" int mt_k_swiglu_bwd(const void* gu, const void* dact, void* dgu, int T, int F, void* stream) {
  if (!gu || !dact || !dgu || T < 0 || F <= 0 || (F % 8) || !al16(gu) || !al16(dact) || !al16(dgu))
    return MT_ERR_ARG;
  return mt::launch_swiglu_bwd(gu, dact, dgu, T, F, S(stream));
}

extern "C" int mt_k_embed_fwd(const int32_t* tok, const void* E, float* x, int T, int d, void* stream) {
  if (!tok || !E || !x || T < 0 || d <= 0 || (d % 8) || !al16(E) || !al16(x)) return MT_ERR_ARG;
  return mt::launch_embed_fwd(tok, E, x, T, d, S(stream));
}

extern "C" int mt_k_embed_bwd(const int32_t* offs, const int32_t* pos, int n_unique, const float* dx, float* rows,
                              int d, void* stream) {
  if (!offs || !pos || !dx || !rows || n_unique < 0 || d <= 0 || (d % 4)) return MT_ERR_ARG;
  return mt::launch_embed_bwd(offs, pos, n_unique, dx, rows, d, S(stream));
}

extern "C" int mt_k_softmax_ce(const float* z, int64_t ldz, const int32_t* labels, void* dz, int64_t lddz,
                               float* row_loss, int Tc, int V, float scale, void* stream) {
  if (!z || !labels || !dz || !row_loss || Tc < 0 || V <= 0 || (V % 4) || (ldz % 4) || (lddz % 4))
    return MT_ERR_ARG;
  return mt::launch_softmax_ce(z, ldz, labels, dz, lddz, row_loss, Tc, V, scale, S(stream));
}

extern "C" int mt_k_attn_fwd(const void* q, const void* k, const void* v, int64_t ldqkv, void* o, int64_t ldo,
                             float* lse, int b, int s, int H, int Hkv, int hd, void* stream) {
  if (!q || !k || !v || !o || !lse || b < 0 || s < 0 || H <= 0 || Hkv <= 0 || (H % Hkv)) return MT_ERR_ARG;
  if (hd != 64 && hd != 128) return MT_ERR_CONFIG;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(o) || (ldqkv % 8) || (ldo % 8)) return MT_ERR_ARG;
  mt::AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.ldqkv = ldqkv; a.o = o; a.ldo = ldo; a.lse = lse;
  a.b = b; a.s = s; a.H = H; a.Hkv = Hkv; a.hd = hd; a.scale = 1.0f / std::sqrt((float)hd);
  return mt::attention_fwd(a, S(stream));
}

extern "C" int mt_k_attn_bwd(const void* q, const void* k, const void* v, int64_t ldqkv, const void* o,
                             const void* dout, int64_t ldo, const float* lse, float* dvec, float* dq_acc,
                             int64_t ldqa, void* dq, int64_t lddq, void* dk, void* dv, int64_t lddkv, int b, int s,
                             int H, int Hkv, int hd, const float* cos_tab, const float* sin_tab, void* stream) {
  if ((cos_tab == nullptr) != (sin_tab == nullptr)) return MT_ERR_ARG;
  if (!q || !k || !v || !o || !dout || !lse || !dvec || !dq_acc || !dq || !dk || !dv) return MT_ERR_ARG;
  if (b < 0 || s < 0 || H <= 0 || Hkv <= 0 || (H % Hkv)) return MT_ERR_ARG;
  if (hd != 64 && hd != 128) return MT_ERR_CONFIG;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(o) || !al16(dout) || !al16(dq_acc) || (ldqkv % 8) || (ldo % 8) ||
      (ldqa % 4) || (lddq % 4) || (lddkv % 2) || ldqa < (int64_t)H * hd)
    return MT_ERR_ARG;
  mt::AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.ldqkv = ldqkv; a.o = const_cast<void*>(o); a.ldo = ldo; a.lse = const_cast<float*>(lse);
  a.dout = dout; a.dvec = dvec; a.dq_acc = dq_acc; a.ldqa = ldqa; a.dq = dq; a.lddq = lddq; a.dk = dk; a.dv = dv;
  a.lddkv = lddkv; a.b = b; a.s = s; a.H = H; a.Hkv = Hkv; a.hd = hd; a.scale = 1.0f / std::sqrt((float)hd);
  a.rope_cos = cos_tab; a.rope_sin = sin_tab;
  return mt::attention_bwd(a, S(stream));
}

extern "C" int mt_k_attn_fwd_tc(const void* q, const void* k, const void* v, int64_t ldqkv, void* o, int64_t ldo,
                                float* lse, int b, int s, int H, int Hkv, int hd, void* stream, int32_t* dev_err) {
  if (!q || !k || !v || !o || !lse || b < 0 || s < 0 || H <= 0 || Hkv <= 0 || (H % Hkv)) return MT_ERR_ARG;
  if (hd != 64 && hd != 128) return MT_ERR_CONFIG;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(o) || (ldqkv % 8) || (ldo % 8)) return MT_ERR_ARG;
  mt::AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.ldqkv = ldqkv; a.o = o; a.ldo = ldo; a.lse = lse;
  a.b = b; a.s = s; a.H = H; a.Hkv = Hkv; a.hd = hd; a.scale = 1.0f / std::sqrt((float)hd);
  return mt::attention_fwd_tc(a, S(stream), dev_err);
}

extern "C" int mt_k_gemm_bf16_rope(const void* A, int64_t lda, const void* B, int64_t ldb, void* C, int64_t ldc, int M,
                                   int N, int K, int rope_cols, int hd, int s, const float* cos_tab,
                                   const float* sin_tab, void* stream, int32_t* dev_err) {
  if (M < 0 || N < 0 || K < 0 || !cos_tab || !sin_tab) return MT_ERR_ARG;
  mt::GemmDesc g{A, lda, false, B, ldb, false, C, ldc, mt::EPI_BF16_ROPE, nullptr, 0, M, N, K,
                 mt::RopeDesc{cos_tab, sin_tab, rope_cols, hd, s}};
  return mt::gemm_bf16(g, static_cast<cudaStream_t>(stream), dev_err);
}

extern "C" int mt_k_attn_bwd_tc(const void* q, const void* k, const void* v, int64_t ldqkv, const void* o,
                                const void* dout, int64_t ldo, const float* lse, float* dvec, float* dq_acc,
                                int64_t ldqa, void* dq, int64_t lddq, void* dk, void* dv, int64_t lddkv, int b, int s,
                                int H, int Hkv, int hd, const float* cos_tab, const float* sin_tab, void* stream,
                                int32_t* dev_err) {
  if ((cos_tab == nullptr) != (sin_tab == nullptr)) return MT_ERR_ARG;
  if (!q || !k || !v || !o || !dout || !lse || !dvec || !dq_acc || !dq || !dk || !dv) return MT_ERR_ARG;
  if (b < 0 || s < 0 || H <= 0 || Hkv <= 0 || (H % Hkv)) return MT_ERR_ARG;
  if (hd != 128 && hd != 64) return MT_ERR_CONFIG;
  if (!al16(q) || !al16(k) || !al16(v) || !al16(o) || !al16(dout) || !al16(dq_acc) || (ldqkv % 8) || (ldo % 8) ||
      (ldqa % 4) || (lddq % 4) || (lddkv % 8) || ldqa < (int64_t)H * hd)
    return MT_ERR_ARG;
  mt::AttnArgs a{};
  a.q = q; a.k = k; a.v = v; a.ldqkv = ldqkv; a.o = const_cast<void*>(o); a.ldo = ldo; a.lse = const_cast<float*>(lse);
  a.dout = dout; a.dvec = dvec; a.dq_acc = dq_acc; a.ldqa = ldqa; a.dq = dq; a.lddq = lddq; a.dk = dk; a.dv = dv;
  a.lddkv = lddkv; a.b = b; a.s = s; a.H = H; a.Hkv = Hkv; a.hd = hd; a.scale = 1.0f / std::sqrt((float)hd);
  a.rope_cos = cos_tab; a.rope_sin = sin_tab;
  return mt::attention_bwd_tc(a, S(stream), dev_err);
}

// ---------------------------------------------------------------------------
// Layer norm, dropout, linear layers with an epilogue, gated feed-forward.
// ---------------------------------------------------------------------------
namespace {

constexpr int kMostSize = 1 << 30;
// Depth of a product. The tensor cores lose 1e-9 K of a sum that is rounded to
// bf16: 1e-3 here, a quarter of the most that the rounding takes. And a tile's
// main loop, whose end the epilogue awaits for at most a second, takes under 10 ms.
constexpr int kMostDepth = 1 << 20;

bool size_ok(int n) { return n >= 0 && n <= kMostSize; }
bool type_ok(int t) { return t == MT_F32 || t == MT_BF16; }
bool act_ok(int a) { return a >= MT_ACT_NONE && a <= MT_ACT_SILU; }
// A matrix operand: present, aligned, its pitch a multiple of 16 bytes and no shorter than a row.
bool mat_ok(const void* p, int type, int64_t ld, int64_t width) {
  return p && al16(p) && ld >= width && ld % (type == MT_F32 ? 4 : 8) == 0;
}
bool opt_mat_ok(const void* p, int type, int64_t ld, int64_t width) { return !p || mat_ok(p, type, ld, width); }
// Vectors of fp32 and dev_err (each may be NULL here) are read and written by the element.
template <typename... P>
bool al4(const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 3) == 0;
}

// The launchers' dropout; rows: of the call. offset_dev is read as 8 bytes.
int drop_of(const mt_dropout* d, int rows, mt::DropDesc* out) {
  if (d && (reinterpret_cast<uintptr_t>(d->offset_dev) & 7)) return MT_ERR_ARG;
  return mt::make_drop(d, rows, out);
}

}  // namespace

extern "C" int mt_k_layernorm_fwd(const void* x, int x_type, int64_t ldx, const void* g, const void* b, void* y,
                                  int y_type, int64_t ldy, float* mean, float* rstd, int T, int d, float eps,
                                  void* stream) {
  if (!type_ok(x_type) || !type_ok(y_type) || !size_ok(T) || d <= 0 || !(eps >= 0.f)) return MT_ERR_ARG;
  if (d > 8192) return MT_ERR_CONFIG;
  if (T == 0) return MT_OK;
  if (!mat_ok(x, x_type, ldx, d) || !mat_ok(y, y_type, ldy, d) || !g || !al16(g) || !al16(b) ||
      !al4(mean, rstd))
    return MT_ERR_ARG;
  return mt::launch_layernorm_fwd(x, x_type, ldx, g, b, y, y_type, ldy, mean, rstd, T, d, eps, S(stream));
}

extern "C" size_t mt_k_layernorm_bwd_partial_floats(int T, int d) {
  return size_ok(T) && d > 0 && d <= 8192 ? mt::layernorm_bwd_partial_floats(T, d) : 0;
}

extern "C" int mt_k_layernorm_bwd(const void* x, int x_type, int64_t ldx, const void* g, const float* mean,
                                  const float* rstd, const void* dy, int dy_type, int64_t lddy, const void* dres,
                                  int64_t lddres, void* dx, void* dx_bf16, int64_t lddx, float* part, float* dg,
                                  float* db, int T, int d, void* stream) {
  if (!type_ok(x_type) || !type_ok(dy_type) || !size_ok(T) || d <= 0 || !dg) return MT_ERR_ARG;
  if (d > 8192) return MT_ERR_CONFIG;
  if (T > 0) {
    if (!mat_ok(x, x_type, ldx, d) || !mat_ok(dy, dy_type, lddy, d) || !opt_mat_ok(dres, x_type, lddres, d) ||
        !mat_ok(dx, x_type, lddx, d) || !g || !al16(g) || !mean || !rstd || !part || !al4(mean, rstd, part, dg, db))
      return MT_ERR_ARG;
    if (dx_bf16 && (x_type != MT_F32 || !mat_ok(dx_bf16, MT_BF16, lddx, d))) return MT_ERR_ARG;
  }
  const mt::LayerNormBwd a{x,      x_type, ldx, g,       mean, rstd, dy, dy_type, lddy, dres,
                           lddres, dx,     dx_bf16, lddx, part, dg,   db, T,       d};
  return mt::launch_layernorm_bwd(a, S(stream));
}

extern "C" int mt_k_dropout(const void* x, int x_type, int64_t ldx, const mt_dropout* drop, const void* res,
                            int64_t ldr, void* y, int y_type, int64_t ldy, int T, int d, void* stream) {
  mt::DropDesc dd;
  if (!type_ok(x_type) || !type_ok(y_type) || !size_ok(T) || !size_ok(d)) return MT_ERR_ARG;
  if (const int rc = drop_of(drop, T, &dd)) return rc;
  if (T == 0 || d == 0) return MT_OK;
  if (!mat_ok(x, x_type, ldx, d) || !mat_ok(y, y_type, ldy, d) || !opt_mat_ok(res, y_type, ldr, d)) return MT_ERR_ARG;
  return mt::launch_dropout(x, x_type, ldx, dd, res, ldr, y, y_type, ldy, T, d, S(stream));
}

extern "C" int mt_k_linear_fwd(const void* A, int64_t lda, const void* W, int64_t ldw, const void* bias, int act,
                               const mt_dropout* drop, const void* R, int64_t ldr, void* Z, int64_t ldz, void* C,
                               int out_type, int64_t ldc, int M, int N, int K, void* stream, int32_t* dev_err) {
  mt::DropDesc dd;
  if (!type_ok(out_type) || !act_ok(act) || !size_ok(M) || !size_ok(N) || !size_ok(K)) return MT_ERR_ARG;
  if (const int rc = drop_of(drop, M, &dd)) return rc;
  if (M == 0 || N == 0) return MT_OK;
  if (K == 0 || !mat_ok(A, MT_BF16, lda, K) || !mat_ok(W, MT_BF16, ldw, K) || !al16(bias) ||
      !opt_mat_ok(R, out_type, ldr, N) || !opt_mat_ok(Z, MT_BF16, ldz, N) || !mat_ok(C, out_type, ldc, N) ||
      !al4(dev_err))
    return MT_ERR_ARG;
  if (K > kMostDepth) return MT_ERR_CONFIG;
  const mt::LinearFwd a{A, lda, W, ldw, bias, act, R, ldr, Z, ldz, C, out_type, ldc, M, N, K};
  return mt::launch_linear_fwd(a, dd, S(stream), dev_err);
}

extern "C" size_t mt_k_linear_bwd_act_partial_floats(int M, int N) {
  return size_ok(M) && size_ok(N) ? mt::linear_bwd_partial_floats(M, N) : 0;
}

extern "C" int mt_k_linear_bwd_act(const void* dY, int64_t lddy, const void* W, int64_t ldw, const void* Z, int64_t ldz,
                                   int act, const mt_dropout* drop, void* dZ, int64_t lddz, float* part, float* db,
                                   int M, int N, int K, void* stream, int32_t* dev_err) {
  mt::DropDesc dd;
  if (!act_ok(act) || !size_ok(M) || !size_ok(N) || !size_ok(K)) return MT_ERR_ARG;
  if (const int rc = drop_of(drop, M, &dd)) return rc;
  if (N == 0) return MT_OK;
  if (M == 0) return !db || cudaMemsetAsync(db, 0, sizeof(float) * N, S(stream)) == cudaSuccess ? MT_OK : MT_ERR_CUDA;
  if (K == 0 || !mat_ok(dY, MT_BF16, lddy, K) || !mat_ok(W, MT_BF16, ldw, N) || !opt_mat_ok(Z, MT_BF16, ldz, N) ||
      !mat_ok(dZ, MT_BF16, lddz, N) || (act != MT_ACT_NONE && !Z) || (db && !part) || !al16(part) ||
      !al4(db, dev_err))
    return MT_ERR_ARG;
  if (K > kMostDepth) return MT_ERR_CONFIG;
  const mt::LinearBwd a{dY, lddy, W, ldw, Z, ldz, act, dZ, lddz, part, db, M, N, K};
  return mt::launch_linear_bwd_act(a, dd, S(stream), dev_err);
}

extern "C" size_t mt_k_act_bwd_partial_floats(int M, int N) {
  return size_ok(M) && size_ok(N) ? mt::act_bwd_partial_floats(M, N) : 0;
}

extern "C" int mt_k_act_bwd(const void* dC, int dc_type, int64_t lddc, const void* Z, int64_t ldz, int act,
                            const mt_dropout* drop, void* dZ, int64_t lddz, float* part, float* db, int M, int N,
                            void* stream) {
  mt::DropDesc dd;
  if (!type_ok(dc_type) || !act_ok(act) || !size_ok(M) || !size_ok(N)) return MT_ERR_ARG;
  if (const int rc = drop_of(drop, M, &dd)) return rc;
  if (M > 0 && N > 0 &&
      (!mat_ok(dC, dc_type, lddc, N) || !opt_mat_ok(Z, MT_BF16, ldz, N) || !mat_ok(dZ, MT_BF16, lddz, N) ||
       (act != MT_ACT_NONE && !Z) || (db && !part) || !al4(part, db)))
    return MT_ERR_ARG;
  return mt::launch_act_bwd(dC, dc_type, lddc, Z, ldz, act, dd, dZ, lddz, part, db, M, N, S(stream));
}

extern "C" int mt_k_gated_ffn_fwd(const void* x, int64_t ldx, const void* Wgu, int64_t ldw, int act, void* gu,
                                  int64_t ldgu, void* h, int64_t ldh, int M, int F, int K, void* stream,
                                  int32_t* dev_err) {
  if (!act_ok(act) || !size_ok(M) || !size_ok(F) || !size_ok(K) || (F % 8)) return MT_ERR_ARG;
  if (M == 0 || F == 0) return MT_OK;
  if (K == 0 || !mat_ok(x, MT_BF16, ldx, K) || !mat_ok(Wgu, MT_BF16, ldw, K) ||
      !opt_mat_ok(gu, MT_BF16, ldgu, 2 * (int64_t)F) || !mat_ok(h, MT_BF16, ldh, F) || !al4(dev_err))
    return MT_ERR_ARG;
  if (K > kMostDepth) return MT_ERR_CONFIG;
  return mt::launch_gated_ffn_fwd(x, ldx, Wgu, ldw, act, gu, ldgu, h, ldh, M, F, K, S(stream), dev_err);
}

extern "C" int mt_k_gated_ffn_bwd(const void* dy, int64_t lddy, const void* Wd, int64_t ldw, const void* gu,
                                  int64_t ldgu, int act, void* dgu, int64_t lddgu, void* h, int64_t ldh, int M, int F,
                                  int K, void* stream, int32_t* dev_err) {
  if (!act_ok(act) || !size_ok(M) || !size_ok(F) || !size_ok(K) || (F % 8)) return MT_ERR_ARG;
  if (M == 0 || F == 0) return MT_OK;
  if (K == 0 || !mat_ok(dy, MT_BF16, lddy, K) || !mat_ok(Wd, MT_BF16, ldw, F) ||
      !mat_ok(gu, MT_BF16, ldgu, 2 * (int64_t)F) || !mat_ok(dgu, MT_BF16, lddgu, 2 * (int64_t)F) ||
      !opt_mat_ok(h, MT_BF16, ldh, F) || !al4(dev_err))
    return MT_ERR_ARG;
  if (K > kMostDepth) return MT_ERR_CONFIG;
  return mt::launch_gated_ffn_bwd(dy, lddy, Wd, ldw, gu, ldgu, act, dgu, lddgu, h, ldh, M, F, K, S(stream), dev_err);
}
