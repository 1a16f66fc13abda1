// hgemm_block_api.cu — the C ABI of the feed-forward block's operators
// declared in include/hgemm.h: argument checks and dispatch.
#include <cmath>
#include <cstdint>

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

}  // extern "C"
