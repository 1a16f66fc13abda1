// hgemm_block_api.cu — the C ABI of the feed-forward block's operators
// declared in include/hgemm.h: argument checks and dispatch.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <new>

#include "hgemm.h"
#include "internal.h"

namespace {

constexpr int64_t kPitchLimit = int64_t(1) << 40;

// One matrix or vector argument: rows × cols elements of `size` bytes.
struct Span {
  const void* p;
  int64_t rows, cols, ld;
  int size;
  bool empty() const { return rows == 0 || cols == 0; }
  unsigned __int128 bytes() const {
    return empty() ? 0 : (static_cast<unsigned __int128>(rows - 1) * ld + cols) * size;
  }
};

bool dims_ok(int64_t a, int64_t b, int64_t c = 0) {
  return a >= 0 && b >= 0 && c >= 0 && a <= HGEMM_MAX_DIM && b <= HGEMM_MAX_DIM && c <= HGEMM_MAX_DIM;
}

// A pitch that covers a row, a span that cannot overflow, a pointer where
// there are elements, aligned to its element.
bool span_ok(const Span& s) {
  if (s.ld < s.cols || s.ld > kPitchLimit) return false;
  if (s.bytes() >= static_cast<unsigned __int128>(1) << 62) return false;
  if (!s.empty() && !s.p) return false;
  return reinterpret_cast<uintptr_t>(s.p) % s.size == 0;
}

bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.empty() || b.empty()) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + static_cast<uint64_t>(b.bytes()) && b0 < a0 + static_cast<uint64_t>(a.bytes());
}

// The same elements, so that each is read before it is overwritten.
bool same(const Span& a, const Span& b) { return a.p == b.p && a.ld == b.ld; }

const Span kNone{nullptr, 0, 0, 0, 1};

Span half_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) { return Span{p, rows, cols, ld, 2}; }
Span vec(const void* p, int64_t n, int size) { return Span{p, 1, n, n, size}; }
int64_t groups_of(int64_t n) { return (n + HGEMM_CKPT8_GROUP - 1) / HGEMM_CKPT8_GROUP; }

}  // namespace

extern "C" {

int hgemm_linear(const hgemm_half_t* X, int64_t ldx, const hgemm_half_t* W, int64_t ldw, const hgemm_half_t* bias,
                 int act, const hgemm_half_t* R, int64_t ldr, hgemm_half_t* Y, int64_t ldy, int8_t* codes,
                 int64_t ldq, float* scales, int64_t lds, int64_t M, int64_t N, int64_t K, cudaStream_t stream) {
  if (!dims_ok(M, N, K) || act < HGEMM_ACT_NONE || act > HGEMM_ACT_GELU_ERF || !codes != !scales)
    return HGEMM_ERR_INVALID_ARG;
  const Span x = half_matrix(X, M, K, ldx), w = half_matrix(W, N, K, ldw), y = half_matrix(Y, M, N, ldy);
  const Span b = bias ? vec(bias, N, 2) : kNone, r = R ? half_matrix(R, M, N, ldr) : kNone;
  const Span q = codes ? Span{codes, M, N, ldq, 1} : kNone;
  const Span s = codes ? Span{scales, groups_of(N), M, lds, 4} : kNone;
  for (const Span& v : {x, w, y, b, r, q, s})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  for (const Span& o : {y, q, s})
    for (const Span& v : {x, w, b})
      if (overlap(o, v)) return HGEMM_ERR_ALIAS;
  if ((overlap(y, r) && !same(y, r)) || overlap(q, r) || overlap(s, r)) return HGEMM_ERR_ALIAS;
  if (overlap(y, q) || overlap(y, s) || overlap(q, s)) return HGEMM_ERR_ALIAS;
  if (M == 0 || N == 0) return HGEMM_OK;
  const hg::LinearProduct p{X, ldx, false, W, ldw, false, Y, ldy, M, N, K,
                            hg::LinEpi{0, act, bias, R, ldr, codes, ldq, scales, lds, nullptr, 0}};
  return hg::run_linear(p, stream);
}

int hgemm_linear_dgrad(const hgemm_half_t* dY, int64_t lddy, const hgemm_half_t* W, int64_t ldw,
                       const int8_t* codes, int64_t ldq, const float* scales, int64_t lds, int act,
                       hgemm_half_t* dU, int64_t lddu, hgemm_half_t* H, int64_t ldh, int64_t M, int64_t N,
                       int64_t K, cudaStream_t stream) {
  if (!dims_ok(M, N, K) || act < HGEMM_ACT_NONE || act > HGEMM_ACT_GELU_ERF || !codes != !scales)
    return HGEMM_ERR_INVALID_ARG;
  if (!codes && M > 0 && K > 0 && (act != HGEMM_ACT_NONE || H)) return HGEMM_ERR_INVALID_ARG;
  const Span dy = half_matrix(dY, M, N, lddy), w = half_matrix(W, N, K, ldw), du = half_matrix(dU, M, K, lddu);
  const Span h = H ? half_matrix(H, M, K, ldh) : kNone;
  const Span q = codes ? Span{codes, M, K, ldq, 1} : kNone;
  const Span s = codes ? Span{scales, groups_of(K), M, lds, 4} : kNone;
  for (const Span& v : {dy, w, du, h, q, s})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  for (const Span& o : {du, h})
    for (const Span& v : {dy, w, q, s})
      if (overlap(o, v)) return HGEMM_ERR_ALIAS;
  if (overlap(du, h)) return HGEMM_ERR_ALIAS;
  if (M == 0 || K == 0) return HGEMM_OK;
  const hg::LinearProduct p{dY, lddy, false, W, ldw, true, dU, lddu, M, K, N,
                            hg::LinEpi{1, act, nullptr, nullptr, 0, const_cast<int8_t*>(codes), ldq,
                                       const_cast<float*>(scales), lds, H, ldh}};
  return hg::run_linear(p, stream);
}

int hgemm_linear_wgrad(const hgemm_half_t* dY, int64_t lddy, const hgemm_half_t* X, int64_t ldx, hgemm_half_t* dW,
                       int64_t lddw, float* dbias, int accumulate, int64_t M, int64_t N, int64_t K,
                       cudaStream_t stream) {
  if (!dims_ok(M, N, K)) return HGEMM_ERR_INVALID_ARG;
  const Span dy = half_matrix(dY, M, N, lddy), x = half_matrix(X, M, K, ldx), dw = half_matrix(dW, N, K, lddw);
  const Span db = dbias ? vec(dbias, N, 4) : kNone;
  for (const Span& v : {dy, x, dw, db})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  for (const Span& o : {dw, db})
    for (const Span& v : {dy, x})
      if (overlap(o, v)) return HGEMM_ERR_ALIAS;
  if (overlap(dw, db)) return HGEMM_ERR_ALIAS;
  if (N == 0) return HGEMM_OK;
  hg::CallDevice dev;
  int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  if (K > 0) {
    const uint16_t* old = accumulate ? dW : nullptr;
    const hg::LinearProduct p{dY, lddy, true, X, ldx, true, dW, lddw, N, K, M,
                              hg::LinEpi{0, HGEMM_ACT_NONE, nullptr, old, lddw, nullptr, 0, nullptr, 0, nullptr, 0}};
    return hg::run_wgrad(p, dbias, accumulate != 0, stream);
  }
  if (!dbias) return HGEMM_OK;
  return hg::cuda_status(hg::launch_column_sums(dY, lddy, M, N, dbias, accumulate != 0, false, false, stream));
}

int hgemm_layernorm_forward(const hgemm_half_t* X, int64_t ldx, const hgemm_half_t* gamma, const hgemm_half_t* beta,
                            float eps, hgemm_half_t* Y, int64_t ldy, float* mean, float* rstd, int64_t M,
                            int64_t D, cudaStream_t stream) {
  if (!dims_ok(M, D) || !(eps >= 0.f) || std::isinf(eps) || !mean != !rstd) return HGEMM_ERR_INVALID_ARG;
  const Span x = half_matrix(X, M, D, ldx), y = half_matrix(Y, M, D, ldy);
  const Span g = vec(gamma, D, 2), b = vec(beta, D, 2);
  const Span mu = mean ? vec(mean, M, 4) : kNone, rs = rstd ? vec(rstd, M, 4) : kNone;
  for (const Span& v : {x, y, g, b, mu, rs})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  for (const Span& o : {y, mu, rs})
    for (const Span& v : {g, b})
      if (overlap(o, v)) return HGEMM_ERR_ALIAS;
  if ((overlap(y, x) && !same(y, x)) || overlap(mu, x) || overlap(rs, x)) return HGEMM_ERR_ALIAS;
  if (overlap(y, mu) || overlap(y, rs) || overlap(mu, rs)) return HGEMM_ERR_ALIAS;
  if (M == 0 || D == 0) return HGEMM_OK;
  hg::CallDevice dev;
  const int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  hg::NormArgs a{};
  a.x = X, a.ldx = ldx, a.gamma = gamma, a.beta = beta, a.eps = eps, a.y = Y, a.ldy = ldy;
  a.mean = mean, a.rstd = rstd, a.M = M, a.D = D;
  return hg::cuda_status(hg::launch_layernorm_forward(a, dev.num_sms, stream));
}

size_t hgemm_layernorm_backward_workspace_size(int64_t M, int64_t D) {
  if (!dims_ok(M, D) || D == 0) return 0;
  return hg::layernorm_backward_workspace(M, D);
}

int hgemm_layernorm_backward(const hgemm_half_t* dY, int64_t lddy, const hgemm_half_t* X, int64_t ldx,
                             const hgemm_half_t* gamma, const float* mean, const float* rstd, const hgemm_half_t* R,
                             int64_t ldr, hgemm_half_t* dX, int64_t lddx, float* dgamma, float* dbeta,
                             void* workspace, size_t workspace_bytes, int64_t M, int64_t D, cudaStream_t stream) {
  if (!dims_ok(M, D)) return HGEMM_ERR_INVALID_ARG;
  const Span dy = half_matrix(dY, M, D, lddy), x = half_matrix(X, M, D, ldx), dx = half_matrix(dX, M, D, lddx);
  const Span r = R ? half_matrix(R, M, D, ldr) : kNone;
  const Span g = vec(gamma, D, 2), mu = vec(mean, M, 4), rs = vec(rstd, M, 4);
  const Span dg = vec(dgamma, D, 4), db = vec(dbeta, D, 4);
  const size_t need = hgemm_layernorm_backward_workspace_size(M, D);
  for (const Span& v : {dy, x, dx, r, g, mu, rs, dg, db})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  if (D > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u)))
    return HGEMM_ERR_INVALID_ARG;
  const Span ws = vec(workspace, static_cast<int64_t>(need), 1);
  for (const Span& o : {dx, dg, db, ws})
    for (const Span& v : {x, g, mu, rs})
      if (overlap(o, v)) return HGEMM_ERR_ALIAS;
  for (const Span& v : {dy, r}) {
    if (overlap(dx, v) && !same(dx, v)) return HGEMM_ERR_ALIAS;
    if (overlap(dg, v) || overlap(db, v) || overlap(ws, v)) return HGEMM_ERR_ALIAS;
  }
  if (overlap(dx, dg) || overlap(dx, db) || overlap(dx, ws) || overlap(dg, db) || overlap(dg, ws) || overlap(db, ws))
    return HGEMM_ERR_ALIAS;
  if (D == 0) return HGEMM_OK;
  hg::CallDevice dev;
  const int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  hg::NormArgs a{};
  a.x = X, a.ldx = ldx, a.gamma = gamma, a.y = dX, a.ldy = lddx;
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.dy = dY, a.lddy = lddy, a.res = R, a.ldr = ldr, a.dgamma = dgamma, a.dbeta = dbeta;
  a.work = static_cast<float*>(workspace), a.M = M, a.D = D;
  a.status = dev.status, a.timeout_ns = dev.timeout_ns, a.inject = dev.inject;
  return hg::cuda_status(hg::launch_layernorm_backward(a, dev.num_sms, stream));
}

int hgemm_ckpt8_save(const hgemm_half_t* X, int64_t ldx, int8_t* codes, int64_t ldq, float* scales, int64_t lds,
                     int64_t M, int64_t N, cudaStream_t stream) {
  if (!dims_ok(M, N)) return HGEMM_ERR_INVALID_ARG;
  const Span x = half_matrix(X, M, N, ldx), q{codes, M, N, ldq, 1}, s{scales, groups_of(N), M, lds, 4};
  for (const Span& v : {x, q, s})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  if (overlap(q, x) || overlap(s, x) || overlap(q, s)) return HGEMM_ERR_ALIAS;
  if (M == 0 || N == 0) return HGEMM_OK;
  hg::CallDevice dev;
  const int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  return hg::cuda_status(hg::launch_ckpt8_save(X, ldx, codes, ldq, scales, lds, M, N, stream));
}

int hgemm_ckpt8_load(const int8_t* codes, int64_t ldq, const float* scales, int64_t lds, int act, hgemm_half_t* Y,
                     int64_t ldy, int64_t M, int64_t N, cudaStream_t stream) {
  if (!dims_ok(M, N) || act < HGEMM_ACT_NONE || act > HGEMM_ACT_GELU_ERF) return HGEMM_ERR_INVALID_ARG;
  const Span y = half_matrix(Y, M, N, ldy), q{codes, M, N, ldq, 1}, s{scales, groups_of(N), M, lds, 4};
  for (const Span& v : {y, q, s})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  if (overlap(y, q) || overlap(y, s)) return HGEMM_ERR_ALIAS;
  if (M == 0 || N == 0) return HGEMM_OK;
  hg::CallDevice dev;
  const int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  return hg::cuda_status(hg::launch_ckpt8_load(codes, ldq, scales, lds, act, Y, ldy, M, N, stream));
}

namespace {

bool norm_kind_ok(int kind, const void* gamma, const void* beta) {
  if (kind == HGEMM_NORM_NONE) return !gamma && !beta;
  return kind == HGEMM_NORM_LAYER || kind == HGEMM_NORM_RMS;
}

Span vec_or_none(const void* p, int64_t n, int size) { return p ? vec(p, n, size) : kNone; }

}  // namespace

int hgemm_residual_norm_forward(const hgemm_half_t* X, int64_t ldx, float alpha, const hgemm_half_t* Y, int64_t ldy,
                                const hgemm_half_t* gate, int post, const hgemm_half_t* post_gamma,
                                const hgemm_half_t* post_beta, int pre, const hgemm_half_t* pre_gamma,
                                const hgemm_half_t* pre_beta, float eps, hgemm_half_t* Z, int64_t ldz,
                                hgemm_half_t* H, int64_t ldh, float* stats, int64_t M, int64_t D,
                                cudaStream_t stream) {
  if (!dims_ok(M, D) || !(eps >= 0.f) || std::isinf(eps) || !std::isfinite(alpha)) return HGEMM_ERR_INVALID_ARG;
  if (!norm_kind_ok(post, post_gamma, post_beta) || !norm_kind_ok(pre, pre_gamma, pre_beta) ||
      (pre == HGEMM_NORM_NONE && H))
    return HGEMM_ERR_INVALID_ARG;
  const Span x = half_matrix(X, M, D, ldx), y = half_matrix(Y, M, D, ldy), z = half_matrix(Z, M, D, ldz);
  const Span h = pre ? half_matrix(H, M, D, ldh) : kNone;
  const Span g = vec_or_none(gate, D, 2), pg = post ? vec(post_gamma, D, 2) : kNone, pb = vec_or_none(post_beta, D, 2);
  const Span qg = pre ? vec(pre_gamma, D, 2) : kNone, qb = vec_or_none(pre_beta, D, 2);
  const Span st = stats ? Span{stats, 4, M, M, 4} : kNone;
  for (const Span& v : {x, y, z, h, g, pg, pb, qg, qb, st})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  for (const Span& o : {z, h, st})
    for (const Span& v : {g, pg, pb, qg, qb})
      if (overlap(o, v)) return HGEMM_ERR_ALIAS;
  if ((overlap(z, x) && !same(z, x)) || overlap(z, y) || (overlap(h, y) && !same(h, y)) || overlap(h, x))
    return HGEMM_ERR_ALIAS;
  if (overlap(st, x) || overlap(st, y) || overlap(z, h) || overlap(z, st) || overlap(h, st)) return HGEMM_ERR_ALIAS;
  if (M == 0 || D == 0) return HGEMM_OK;
  hg::CallDevice dev;
  const int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  const hg::ResidualNormArgs a{X,   ldx,       alpha,    Y,   ldy, gate, post, post_gamma, post_beta, pre,
                               pre_gamma, pre_beta, eps, Z,   ldz, H,    ldh,  stats,      M,         D};
  return hg::cuda_status(hg::launch_residual_norm_forward(a, dev.num_sms, stream));
}

size_t hgemm_residual_norm_backward_workspace_size(int64_t M, int64_t D) {
  if (!dims_ok(M, D) || D == 0) return 0;
  return hg::residual_norm_backward_workspace(M, D);
}

int hgemm_residual_norm_backward(const hgemm_half_t* dZ, int64_t lddz, const hgemm_half_t* dH, int64_t lddh,
                                 const hgemm_half_t* Z, int64_t ldz, const hgemm_half_t* Y, int64_t ldy, float alpha,
                                 const hgemm_half_t* gate, int post, const hgemm_half_t* post_gamma,
                                 const hgemm_half_t* post_beta, int pre, const hgemm_half_t* pre_gamma,
                                 const float* stats, hgemm_half_t* dX, int64_t lddx, hgemm_half_t* dY, int64_t lddy,
                                 float* dgate, float* dpost_gamma, float* dpost_beta, float* dpre_gamma,
                                 float* dpre_beta, void* workspace, size_t workspace_bytes, int64_t M, int64_t D,
                                 cudaStream_t stream) {
  if (!dims_ok(M, D) || !std::isfinite(alpha)) return HGEMM_ERR_INVALID_ARG;
  if (!norm_kind_ok(post, post_gamma, post_beta) || !norm_kind_ok(pre, pre_gamma, nullptr))
    return HGEMM_ERR_INVALID_ARG;
  if ((!pre && (dH || dpre_gamma || dpre_beta)) || (!post && (dpost_gamma || dpost_beta)) || (!gate && dgate))
    return HGEMM_ERR_INVALID_ARG;
  const Span dz = dZ ? half_matrix(dZ, M, D, lddz) : kNone, dh = pre ? half_matrix(dH, M, D, lddh) : kNone;
  const Span z = half_matrix(Z, M, D, ldz), y = half_matrix(Y, M, D, ldy);
  const Span dx = half_matrix(dX, M, D, lddx), dy = half_matrix(dY, M, D, lddy);
  const Span g = vec_or_none(gate, D, 2), pg = post ? vec(post_gamma, D, 2) : kNone, pb = vec_or_none(post_beta, D, 2);
  const Span qg = pre ? vec(pre_gamma, D, 2) : kNone;
  const Span st = pre || post ? Span{stats, 4, M, M, 4} : kNone;
  const Span sums[5] = {vec_or_none(dgate, D, 4), vec_or_none(dpost_gamma, D, 4), vec_or_none(dpost_beta, D, 4),
                        vec_or_none(dpre_gamma, D, 4), vec_or_none(dpre_beta, D, 4)};
  for (const Span& v : {dz, dh, z, y, dx, dy, g, pg, pb, qg, st})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  for (const Span& v : sums)
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  const size_t need = hgemm_residual_norm_backward_workspace_size(M, D);
  if (D > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u)))
    return HGEMM_ERR_INVALID_ARG;
  const Span ws = vec(workspace, static_cast<int64_t>(need), 1);
  for (const Span& o : {dx, dy, ws, sums[0], sums[1], sums[2], sums[3], sums[4]})
    for (const Span& v : {z, y, g, pg, pb, qg, st})
      if (overlap(o, v)) return HGEMM_ERR_ALIAS;
  if ((overlap(dx, dz) && !same(dx, dz)) || overlap(dx, dh) || (overlap(dy, dh) && !same(dy, dh)) || overlap(dy, dz))
    return HGEMM_ERR_ALIAS;
  if (overlap(dx, dy) || overlap(dx, ws) || overlap(dy, ws) || overlap(dz, ws) || overlap(dh, ws))
    return HGEMM_ERR_ALIAS;
  for (int i = 0; i < 5; ++i) {
    for (const Span& v : {dz, dh, dx, dy, ws})
      if (overlap(sums[i], v)) return HGEMM_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlap(sums[i], sums[j])) return HGEMM_ERR_ALIAS;
  }
  if (D == 0) return HGEMM_OK;
  hg::CallDevice dev;
  const int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  hg::ResidualNormBackArgs a{};
  a.dz = dZ, a.lddz = lddz, a.dh = dH, a.lddh = lddh, a.z = Z, a.ldz = ldz, a.y = Y, a.ldy = ldy, a.alpha = alpha;
  a.gate = gate, a.post = post, a.post_gamma = post_gamma, a.post_beta = post_beta, a.pre = pre;
  a.pre_gamma = pre_gamma, a.stats = stats, a.dx = dX, a.lddx = lddx, a.dy = dY, a.lddy = lddy;
  a.dgate = dgate, a.dpost_gamma = dpost_gamma, a.dpost_beta = dpost_beta;
  a.dpre_gamma = dpre_gamma, a.dpre_beta = dpre_beta;
  a.partials = static_cast<float*>(workspace), a.M = M, a.D = D;
  a.status = dev.status, a.timeout_ns = dev.timeout_ns, a.inject = dev.inject;
  return hg::cuda_status(hg::launch_residual_norm_backward(a, dev.num_sms, stream));
}

namespace {

// The arrays of one tensor, outputs first: weight, master, m, v, their scales,
// then the gradient.
constexpr int kAdamwOutputs = 6;
int adamw_spans(const hgemm_adamw_tensor& t, Span (&s)[kAdamwOutputs + 1]) {
  if (t.n < 0 || t.n > HGEMM_MAX_DIM || (t.grad_type != HGEMM_TYPE_F16 && t.grad_type != HGEMM_TYPE_F32) ||
      !std::isfinite(t.weight_decay) || !t.m_scales != !t.v_scales)
    return HGEMM_ERR_INVALID_ARG;
  if (t.n > 0 && !t.weight && !t.master) return HGEMM_ERR_INVALID_ARG;
  const int state = t.m_scales ? 1 : 4;
  s[0] = vec_or_none(t.weight, t.n, 2);
  s[1] = vec_or_none(t.master, t.n, 4);
  s[2] = vec(t.m, t.n, state);
  s[3] = vec(t.v, t.n, state);
  s[4] = vec_or_none(t.m_scales, groups_of(t.n), 4);
  s[5] = vec_or_none(t.v_scales, groups_of(t.n), 4);
  s[6] = vec(t.grad, t.n, t.grad_type == HGEMM_TYPE_F32 ? 4 : 2);
  for (const Span& v : s)
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  for (int i = 0; i < kAdamwOutputs; ++i)
    for (int j = i + 1; j <= kAdamwOutputs; ++j)
      if (overlap(s[i], s[j])) return HGEMM_ERR_ALIAS;
  return HGEMM_OK;
}

struct Range {
  uintptr_t begin, end;
  bool output;
};

}  // namespace

int hgemm_adamw_check(const hgemm_adamw_tensor* tensors, int64_t count) {
  if (count < 0 || (count > 0 && !tensors)) return HGEMM_ERR_INVALID_ARG;
  if (count > HGEMM_MAX_DIM) return HGEMM_ERR_INVALID_ARG;
  Range* all = new (std::nothrow) Range[static_cast<size_t>(count) * (kAdamwOutputs + 1) + 1];
  if (!all) return HGEMM_ERR_INVALID_ARG;
  size_t n = 0;
  int rc = HGEMM_OK;
  for (int64_t i = 0; i < count && rc == HGEMM_OK; ++i) {
    Span s[kAdamwOutputs + 1];
    rc = adamw_spans(tensors[i], s);
    for (int j = 0; j <= kAdamwOutputs && rc == HGEMM_OK; ++j)
      if (s[j].p && !s[j].empty()) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(s[j].p);
        all[n++] = Range{at, at + static_cast<uintptr_t>(s[j].bytes()), j < kAdamwOutputs};
      }
  }
  if (rc == HGEMM_OK) {
    std::sort(all, all + n, [](const Range& a, const Range& b) { return a.begin < b.begin; });
    // the furthest ends so far, of any array and of outputs
    uintptr_t any = 0, outputs = 0;
    for (size_t i = 0; i < n && rc == HGEMM_OK; ++i) {
      if (all[i].begin < (all[i].output ? any : outputs)) rc = HGEMM_ERR_ALIAS;
      any = std::max(any, all[i].end);
      if (all[i].output) outputs = std::max(outputs, all[i].end);
    }
  }
  delete[] all;
  return rc;
}

int hgemm_adamw(const hgemm_adamw_tensor* tensors, int64_t count, double lr, double beta1, double beta2, double eps,
                int64_t step, double grad_scale, const hgemm_adamw_dynamic* dynamic, cudaStream_t stream) {
  return hgemm_adamw_rounded(tensors, count, lr, beta1, beta2, eps, step, grad_scale, HGEMM_ROUND_NEAREST, dynamic,
                             stream);
}

int hgemm_adamw_rounded(const hgemm_adamw_tensor* tensors, int64_t count, double lr, double beta1, double beta2,
                        double eps, int64_t step, double grad_scale, int rounding, const hgemm_adamw_dynamic* dynamic,
                        cudaStream_t stream) {
  if (rounding != HGEMM_ROUND_NEAREST && rounding != HGEMM_ROUND_RANDOM) return HGEMM_ERR_INVALID_ARG;
  if (count < 0 || count > HGEMM_MAX_DIM || (count > 0 && !tensors)) return HGEMM_ERR_INVALID_ARG;
  if (!std::isfinite(lr) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) ||
      std::isinf(eps) || step < 1 || !std::isfinite(grad_scale) || (reinterpret_cast<uintptr_t>(dynamic) & 3u))
    return HGEMM_ERR_INVALID_ARG;
  bool any = false;
  for (int64_t i = 0; i < count; ++i) {
    Span s[kAdamwOutputs + 1];
    const int rc = adamw_spans(tensors[i], s);
    if (rc != HGEMM_OK) return rc;
    if (dynamic)
      for (const Span& v : s)
        if (overlap(v, Span{dynamic, 1, 1, 1, static_cast<int>(sizeof(*dynamic))})) return HGEMM_ERR_ALIAS;
    any = any || tensors[i].n > 0;
  }
  if (!any) return HGEMM_OK;
  hg::CallDevice dev;
  int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  const double t = static_cast<double>(step);
  hg::AdamwStep s{};
  s.beta1 = static_cast<float>(beta1), s.rest1 = static_cast<float>(1.0 - beta1);
  s.beta2 = static_cast<float>(beta2), s.rest2 = static_cast<float>(1.0 - beta2);
  // (the step's reciprocal takes a denominator below 2^-126 for 0, and a value without a gradient would be 0/0)
  s.eps = eps > 0 ? std::max(static_cast<float>(eps), FLT_MIN) : 0.f;
  s.gscale = static_cast<float>(grad_scale), s.lr = static_cast<float>(lr);
  s.a = static_cast<float>(lr / (1.0 - std::pow(beta1, t)));
  s.b = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, t)));
  s.ln1 = static_cast<float>(std::log(beta1)), s.ln2 = static_cast<float>(std::log(beta2));
  s.minus_zero = -0.f;
  s.dynamic = dynamic;
  s.number = static_cast<uint32_t>(step);
  auto aligned = [](const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; };
  hg::AdamwEntry e[hg::kAdamwTensors];
  int n = 0;
  for (int64_t i = 0; i <= count; ++i) {
    if (n == hg::kAdamwTensors || (i == count && n > 0)) {
      rc = hg::cuda_status(hg::launch_adamw(e, n, s, rounding == HGEMM_ROUND_RANDOM, dev.num_sms, stream));
      if (rc != HGEMM_OK) return rc;
      n = 0;
    }
    if (i == count || tensors[i].n == 0) continue;
    const hgemm_adamw_tensor& x = tensors[i];
    const uintptr_t state = x.m_scales ? 8 : 16;
    const bool vec8 = aligned(x.weight, 16) && aligned(x.master, 16) && aligned(x.grad, 16) &&
                      aligned(x.m, state) && aligned(x.v, state);
    e[n++] = hg::AdamwEntry{x.weight, x.master, x.grad, x.m, x.v, x.m_scales, x.v_scales, x.n, x.weight_decay,
                            static_cast<float>(1.0 - lr * x.weight_decay), 0u,
                            static_cast<int16_t>(x.grad_type), static_cast<int16_t>(vec8)};
  }
  return HGEMM_OK;
}

int hgemm_adamw_load(const int8_t* m, const float* m_scales, const uint8_t* v, const float* v_scales, float* m_out,
                     float* v_out, int64_t n, cudaStream_t stream) {
  if (n < 0 || n > kPitchLimit) return HGEMM_ERR_INVALID_ARG;
  if (!m != !m_scales || !m != !m_out || !v != !v_scales || !v != !v_out || (n > 0 && !m && !v))
    return HGEMM_ERR_INVALID_ARG;
  const Span in[4] = {vec_or_none(m, n, 1), vec_or_none(m_scales, groups_of(n), 4), vec_or_none(v, n, 1),
                      vec_or_none(v_scales, groups_of(n), 4)};
  const Span mo = vec_or_none(m_out, n, 4), vo = vec_or_none(v_out, n, 4);
  for (const Span& x : {in[0], in[1], in[2], in[3], mo, vo})
    if (!span_ok(x)) return HGEMM_ERR_INVALID_ARG;
  for (const Span& x : in)
    if (overlap(mo, x) || overlap(vo, x)) return HGEMM_ERR_ALIAS;
  if (overlap(mo, vo)) return HGEMM_ERR_ALIAS;
  if (n == 0) return HGEMM_OK;
  hg::CallDevice dev;
  const int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  return hg::cuda_status(hg::launch_adamw_load(m, m_scales, v, v_scales, m_out, v_out, n, dev.num_sms, stream));
}

namespace {

bool experts_sizes_ok(int64_t M, int64_t D, int64_t F, int64_t E, int64_t k) {
  return M >= 0 && M <= HGEMM_EXPERTS_MAX_TOKENS && D >= 0 && D <= HGEMM_EXPERTS_MAX_WIDTH && F >= 0 &&
         F <= HGEMM_EXPERTS_MAX_WIDTH && E >= 1 && E <= HGEMM_EXPERTS_MAX && k >= 1 && k <= E &&
         k <= HGEMM_EXPERTS_MAX_CHOICES;
}

}  // namespace

size_t hgemm_experts_workspace_size(int64_t M, int64_t D, int64_t F, int64_t E, int64_t k) {
  if (!experts_sizes_ok(M, D, F, E, k)) return 0;
  // The most that any number of tokens up to M takes: fewer tokens may be cut
  // into more runs of F.
  size_t most = 0;
  for (int64_t m = 0; m <= M; ++m) most = std::max(most, hg::experts_workspace(m, D, F, E, k));
  return most;
}

int hgemm_experts(const hgemm_half_t* X, int64_t ldx, const hgemm_half_t* Wr, int64_t ldwr, const hgemm_half_t* W1,
                  int64_t ldw1, const hgemm_half_t* b1, const hgemm_half_t* W2, int64_t ldw2, const hgemm_half_t* b2,
                  int act, int gated, int64_t k, int normalize, const hgemm_half_t* R, int64_t ldr, hgemm_half_t* Y,
                  int64_t ldy, int32_t* chosen, float* share, void* workspace, size_t workspace_bytes, int64_t M,
                  int64_t D, int64_t F, int64_t E, cudaStream_t stream) {
  if (!experts_sizes_ok(M, D, F, E, k) || act < HGEMM_ACT_NONE || act > HGEMM_ACT_GELU_ERF || (gated & ~1) ||
      (normalize & ~1))
    return HGEMM_ERR_INVALID_ARG;
  const int64_t up = gated ? 2 * F : F;
  const Span x = half_matrix(X, M, D, ldx), wr = half_matrix(Wr, E, D, ldwr), y = half_matrix(Y, M, D, ldy);
  const Span w1 = half_matrix(W1, E * up, D, ldw1), w2 = half_matrix(W2, E * D, F, ldw2);
  const Span v1 = vec_or_none(b1, E * up, 2), v2 = vec_or_none(b2, E * D, 2);
  const Span r = R ? half_matrix(R, M, D, ldr) : kNone;
  const Span c = vec_or_none(chosen, M * k, 4), s = vec_or_none(share, M * k, 4);
  for (const Span& v : {x, wr, w1, w2, v1, v2, r, y, c, s})
    if (!span_ok(v)) return HGEMM_ERR_INVALID_ARG;
  const size_t need = hg::experts_workspace(M, D, F, E, k);
  if (M > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u)))
    return HGEMM_ERR_INVALID_ARG;
  const Span ws = vec(workspace, static_cast<int64_t>(need), 1);
  for (const Span& o : {y, c, s, ws})
    for (const Span& v : {x, wr, w1, w2, v1, v2})
      if (overlap(o, v)) return HGEMM_ERR_ALIAS;
  if ((overlap(y, r) && !same(y, r)) || overlap(c, r) || overlap(s, r) || overlap(ws, r)) return HGEMM_ERR_ALIAS;
  if (overlap(y, c) || overlap(y, s) || overlap(y, ws) || overlap(c, s) || overlap(c, ws) || overlap(s, ws))
    return HGEMM_ERR_ALIAS;
  if (M == 0) return HGEMM_OK;
  hg::CallDevice dev;
  const int rc = hg::call_device(&dev);
  if (rc != HGEMM_OK) return rc;
  hg::ExpertsArgs a{};
  a.X = X, a.ldx = ldx, a.Wr = Wr, a.ldwr = ldwr, a.W1 = W1, a.ldw1 = ldw1, a.b1 = b1, a.W2 = W2, a.ldw2 = ldw2;
  a.b2 = b2, a.act = act, a.gated = gated != 0, a.normalize = normalize != 0, a.R = R, a.ldr = ldr, a.Y = Y;
  a.ldy = ldy, a.chosen = chosen, a.share = share;
  a.M = static_cast<int>(M), a.D = static_cast<int>(D), a.F = static_cast<int>(F), a.E = static_cast<int>(E);
  a.k = static_cast<int>(k);
  a.status = dev.status, a.timeout_ns = dev.timeout_ns, a.inject = dev.inject;
  return hg::cuda_status(hg::launch_experts(a, workspace, dev.num_sms, stream));
}

}  // extern "C"
