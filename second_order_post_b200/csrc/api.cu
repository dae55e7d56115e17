// The C ABI of libkronq.so (declared in include/kronq.h): argument validation
// and dispatch to the kernels. No call allocates device memory.
#include <math.h>

#include <algorithm>
#include <initializer_list>
#include <numeric>
#include <vector>

#include "kernels.cuh"

using namespace kronq;

namespace {

bool is_pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

bool rot_ok(const kronq_rot &r, int64_t d) {
  return is_pow2(r.had) && r.m >= 1 && r.m <= 256 && r.had * r.m == d;
}

bool aligned(const void *p, size_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}

// ---- matrices of the dense operators
constexpr int64_t kMaxRows = int64_t(1) << 30, kMaxWidth = int64_t(1) << 24;

struct View {
  const void *p;
  int64_t ld, rows, cols;
  int es;  // bytes per element
};

// Whether two strided matrices share an element's bytes. With equal strides
// the test is exact (column slices of one wide matrix do not overlap);
// otherwise it compares their address ranges.
bool overlap(const View &a, const View &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.cols <= 0 || b.cols <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  if (pb < pa) return overlap(b, a);
  const uint64_t la = uint64_t(a.ld) * a.es, lb = uint64_t(b.ld) * b.es;
  const uint64_t ca = uint64_t(a.cols) * a.es, cb = uint64_t(b.cols) * b.es;
  const uint64_t off = pb - pa;
  if (off >= (uint64_t(a.rows) - 1) * la + ca) return false;
  if (la != lb) return true;
  const uint64_t r = off / la, c = off % la;  // b starts in a's row r at byte c
  return (c < ca && r < uint64_t(a.rows)) || (c + cb > la && r + 1 < uint64_t(a.rows));
}
bool same(const View &a, const View &b) { return a.p == b.p && a.ld == b.ld && a.es == b.es; }
// a may be exactly b, but may not overlap it in another way
bool bad_alias(const View &a, const View &b) { return !same(a, b) && overlap(a, b); }

View bf16_view(const void *p, int64_t rows, int64_t cols, int64_t ld) {
  return View{p, ld, rows, cols, 2};
}

// The layout rules of a bf16 matrix (absent ones pass).
kronq_status check_views(std::initializer_list<View> vs) {
  for (const View &v : vs)
    if (v.p && v.ld < v.cols) return KRONQ_ERR_INVALID_ARG;
  for (const View &v : vs)
    if (v.p && (v.ld % 8 || !aligned(v.p, 16))) return KRONQ_ERR_UNSUPPORTED;
  return KRONQ_OK;
}

// No output overlaps an input or another output.
bool any_overlap(std::initializer_list<View> outs, std::initializer_list<View> ins) {
  for (const View *o = outs.begin(); o != outs.end(); ++o) {
    for (const View &i : ins)
      if (overlap(*o, i)) return true;
    for (const View *q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return true;
  }
  return false;
}

// Runs f; no C++ exception leaves the library (the launch helpers keep small
// tables whose nodes are allocated on the host).
template <class F>
kronq_status guarded(F f) {
  try {
    return f();
  } catch (...) {
    return KRONQ_ERR_CUDA;
  }
}

bool act_ok(int a) { return a >= KRONQ_ACT_NONE && a <= KRONQ_ACT_GELU_TANH; }

Mat mat(const View &v) { return Mat{const_cast<void *>(v.p), v.ld}; }

kronq_status run_distill(kronq_stream_t stream, const void *Z, kronq_dtype zdtype, int64_t n,
                         int64_t vocab, int64_t ldz, const void *T, kronq_dtype tdtype,
                         const int32_t *idx, int64_t k, int64_t ldt, float tau,
                         const float *weight, float *loss, float *lse, void *dZ, int64_t lddz,
                         int32_t *info_dev) {
  if (n < 0 || vocab <= 0 || k <= 0 || ldz < vocab || ldt < k || !info_dev ||
      (dZ && lddz < vocab))
    return KRONQ_ERR_INVALID_ARG;
  if ((zdtype != KRONQ_F32 && zdtype != KRONQ_BF16) ||
      (tdtype != KRONQ_F32 && tdtype != KRONQ_BF16))
    return KRONQ_ERR_INVALID_ARG;
  if (!(tau >= 1e-4f && tau <= 1e4f)) return KRONQ_ERR_INVALID_ARG;
  if (n > 0 && (!Z || !T || !idx)) return KRONQ_ERR_INVALID_ARG;
  const int ez = zdtype == KRONQ_BF16 ? 2 : 4, et = tdtype == KRONQ_BF16 ? 2 : 4;
  if (!aligned(Z, ez) || !aligned(dZ, ez) || !aligned(T, et) || !aligned(idx, 4) ||
      !aligned(weight, 4) || !aligned(loss, 4) || !aligned(lse, 4) || !aligned(info_dev, 4))
    return KRONQ_ERR_INVALID_ARG;
  if (bad_alias(View{dZ, lddz, n, vocab, ez}, View{Z, ldz, n, vocab, ez}))
    return KRONQ_ERR_INVALID_ARG;
  if (any_overlap({View{dZ, lddz, n, vocab, ez}, View{loss, n, 1, n, 4},
                   View{loss ? lse : nullptr, n, 1, n, 4}},
                  {View{T, ldt, n, k, et}, View{idx, ldt, n, k, 4}, View{weight, n, 1, n, 4},
                   View{loss ? nullptr : lse, n, 1, n, 4}}))
    return KRONQ_ERR_INVALID_ARG;
  if (any_overlap({View{loss, n, 1, n, 4}, View{loss ? lse : nullptr, n, 1, n, 4}},
                  {View{Z, ldz, n, vocab, ez}}))
    return KRONQ_ERR_INVALID_ARG;
  if (vocab > 0x7fffffff || n > 0x7fffffff || k > 1024) return KRONQ_ERR_UNSUPPORTED;
  KQ_TRY(require_sm100());
  DistillArgs a;
  a.Z = Z;
  a.z_bf16 = zdtype == KRONQ_BF16;
  a.n = n;
  a.vocab = vocab;
  a.ldz = ldz;
  a.T = T;
  a.t_bf16 = tdtype == KRONQ_BF16;
  a.idx = idx;
  a.k = static_cast<int>(k);
  a.ldt = ldt;
  a.tau = tau;
  a.weight = weight;
  a.loss = loss;
  a.lse = lse;
  a.dZ = dZ;
  a.lddz = lddz;
  a.info = info_dev;
  return guarded([&] { return distill(as_stream(stream), a); });
}

}  // namespace

extern "C" {

const char *kronq_status_string(kronq_status s) {
  switch (s) {
    case KRONQ_OK: return "ok";
    case KRONQ_ERR_INVALID_ARG: return "invalid argument";
    case KRONQ_ERR_UNSUPPORTED: return "unsupported shape or layout";
    case KRONQ_ERR_NOT_PD: return "matrix not positive definite";
    case KRONQ_ERR_NONFINITE: return "non-finite value";
    case KRONQ_ERR_TIMEOUT: return "device wait timed out";
    case KRONQ_ERR_CUDA: return "CUDA error";
  }
  return "unknown status";
}

kronq_status kronq_accum_cov(kronq_stream_t stream, const void *A,
                             kronq_dtype dtype, int64_t n, int64_t d,
                             int64_t lda, float alpha, float beta, float *H,
                             int32_t *info_dev) {
  if (!H || !info_dev || d <= 0 || n < 0 || lda < d || (n > 0 && !A))
    return KRONQ_ERR_INVALID_ARG;
  if (dtype != KRONQ_F32 && dtype != KRONQ_BF16) return KRONQ_ERR_INVALID_ARG;
  if (d > (int64_t(1) << 20) || n > (int64_t(1) << 31)) return KRONQ_ERR_UNSUPPORTED;
  if (dtype == KRONQ_BF16 && (d % 128 || lda % 8 || !aligned(A, 16)))
    return KRONQ_ERR_UNSUPPORTED;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  if (dtype == KRONQ_BF16)
    return cov_bf16(st, static_cast<const __nv_bfloat16 *>(A), n, d, lda, alpha,
                    beta, H, info_dev);
  return cov_f32(st, static_cast<const float *>(A), n, d, lda, alpha, beta, H);
}

kronq_status kronq_sensitivity(kronq_stream_t stream, const float *H_X,
                               int64_t d_in, const float *H_G, int64_t d_out,
                               double *out_dev) {
  if (!H_X || !H_G || !out_dev || d_in <= 0 || d_out <= 0)
    return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  return launch_sensitivity(as_stream(stream), H_X, d_in, H_G, d_out, out_dev);
}

size_t kronq_workspace_bytes(kronq_ws_kind which, int64_t d_out, int64_t d_in,
                             const kronq_opts *opts) {
  if (d_out <= 0 || d_in <= 0) return 0;
  switch (which) {
    case KRONQ_WS_BIIP:
      if (!opts || opts->rot_in.m < 1 || opts->rot_in.m > 256 ||
          opts->rot_out.m < 1 || opts->rot_out.m > 256)
        return 0;
      return biip_ws_bytes(d_out, d_in, *opts);
    case KRONQ_WS_CHOL:
      if (d_in % 128) return 0;
      return chol_ws_bytes(d_in);
    case KRONQ_WS_QUANT:
      if (!opts) return 0;
      return quant_ws_bytes(d_out, d_in, *opts);
    case KRONQ_WS_LOSS:
      return loss_ws_bytes(d_out, d_in);
    case KRONQ_WS_QUANT_SPLIT:
      if (!opts || d_in % 128 || d_in < 256) return 0;
      return quant_split_ws_bytes(d_out, d_in, chol_split_point(d_in), *opts);
  }
  return 0;
}

kronq_status kronq_biip(kronq_stream_t stream, const kronq_opts *opts,
                        const void *W, kronq_dtype wdtype, int64_t d_out,
                        int64_t d_in, float *W_rot, float *H_X, float *H_G,
                        float *s_x, float *s_g, void *ws, size_t ws_bytes,
                        int32_t *info_dev) {
  if (!opts || !W || !W_rot || !H_X || !H_G || !s_x || !s_g || !ws ||
      !info_dev || d_out <= 0 || d_in <= 0)
    return KRONQ_ERR_INVALID_ARG;
  if (wdtype != KRONQ_F32 && wdtype != KRONQ_BF16) return KRONQ_ERR_INVALID_ARG;
  if (!(opts->scale_exp >= 0.f && opts->scale_exp <= 4.f)) return KRONQ_ERR_INVALID_ARG;
  const bool rot_x = !(opts->flags & KRONQ_FLAG_NO_ROT_IN);
  const bool rot_g = !(opts->flags & KRONQ_FLAG_NO_ROT_OUT);
  if (rot_x && !rot_ok(opts->rot_in, d_in)) return KRONQ_ERR_UNSUPPORTED;
  if (rot_g && !rot_ok(opts->rot_out, d_out)) return KRONQ_ERR_UNSUPPORTED;
  if (d_in % 32 || d_in > 65536 || d_out > 65536)
    return KRONQ_ERR_UNSUPPORTED;
  if (!aligned(ws, 256)) return KRONQ_ERR_INVALID_ARG;
  kronq_opts o = *opts;
  if (!rot_x) o.rot_in = {d_in, 1};
  if (!rot_g) o.rot_out = {d_out, 1};
  if (ws_bytes < biip_ws_bytes(d_out, d_in, o)) return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  return biip(st, o, W, wdtype == KRONQ_BF16, d_out, d_in, W_rot, H_X, H_G, s_x,
              s_g, ws, ws_bytes, info_dev);
}

kronq_status kronq_chol_inv(kronq_stream_t stream, float *H, int64_t d,
                            float damp_rel, void *ws, size_t ws_bytes,
                            int32_t *info_dev) {
  if (!H || !ws || !info_dev || d <= 0 || !(damp_rel >= 0.f) || !isfinite(damp_rel))
    return KRONQ_ERR_INVALID_ARG;
  if (d % 128 || d > 65536) return KRONQ_ERR_UNSUPPORTED;
  if (!aligned(ws, 256) || !aligned(H, 16)) return KRONQ_ERR_INVALID_ARG;
  if (ws_bytes < chol_ws_bytes(d)) return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  return chol_inv(st, H, d, damp_rel, ws, ws_bytes, info_dev);
}

kronq_status kronq_quantize_sublayer(kronq_stream_t stream,
                                     const kronq_opts *opts, float *W_rot,
                                     const float *U, int64_t d_out,
                                     int64_t d_in, uint32_t *codes,
                                     float *scales, uint8_t *zeros, void *ws,
                                     size_t ws_bytes, int32_t *info_dev) {
  if (!opts || !W_rot || !U || !codes || !scales || !zeros || !ws ||
      !info_dev || d_out <= 0 || d_in <= 0)
    return KRONQ_ERR_INVALID_ARG;
  if (opts->bits < 2 || opts->bits > 4) return KRONQ_ERR_INVALID_ARG;
  if (opts->group != 32 && opts->group != 64 && opts->group != 128)
    return KRONQ_ERR_UNSUPPORTED;
  if (opts->block != 128 || d_in % 128) return KRONQ_ERR_UNSUPPORTED;
  if (!aligned(ws, 256) || !aligned(W_rot, 16) || !aligned(U, 16))
    return KRONQ_ERR_INVALID_ARG;
  if (ws_bytes < quant_ws_bytes(d_out, d_in, *opts)) return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  return quantize(st, *opts, W_rot, U, d_out, d_in, codes, scales, zeros, ws,
                  ws_bytes, info_dev);
}

kronq_status kronq_chol_split(kronq_stream_t stream, float *H, int64_t d,
                              float damp_rel, void *ws, size_t ws_bytes,
                              int32_t *info_dev) {
  if (!H || !ws || !info_dev || d <= 0 || !(damp_rel >= 0.f) || !isfinite(damp_rel))
    return KRONQ_ERR_INVALID_ARG;
  if (d % 128 || d < 256 || d > 65536) return KRONQ_ERR_UNSUPPORTED;
  if (!aligned(ws, 256) || !aligned(H, 16)) return KRONQ_ERR_INVALID_ARG;
  if (ws_bytes < chol_ws_bytes(d)) return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  return chol_split(st, H, d, damp_rel, ws, ws_bytes, info_dev);
}

int64_t kronq_chol_split_point(int64_t d) { return d >= 256 ? chol_split_point(d) : 0; }

kronq_status kronq_quantize_split(kronq_stream_t stream, const kronq_opts *opts,
                                  float *W_rot, const float *F, int64_t d_out,
                                  int64_t d_in, uint32_t *codes, float *scales,
                                  uint8_t *zeros, void *ws, size_t ws_bytes,
                                  int32_t *info_dev) {
  if (!opts || !W_rot || !F || !codes || !scales || !zeros || !ws || !info_dev ||
      d_out <= 0 || d_in <= 0)
    return KRONQ_ERR_INVALID_ARG;
  if (opts->bits < 2 || opts->bits > 4) return KRONQ_ERR_INVALID_ARG;
  if (opts->group != 32 && opts->group != 64 && opts->group != 128)
    return KRONQ_ERR_UNSUPPORTED;
  if (opts->block != 128 || d_in % 128 || d_in < 256) return KRONQ_ERR_UNSUPPORTED;
  if (!aligned(ws, 256) || !aligned(W_rot, 16) || !aligned(F, 16))
    return KRONQ_ERR_INVALID_ARG;
  const int64_t h = chol_split_point(d_in);
  if (ws_bytes < quant_split_ws_bytes(d_out, d_in, h, *opts)) return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  return quantize_split(st, *opts, W_rot, F, d_out, d_in, h, codes, scales, zeros, ws,
                        ws_bytes, info_dev);
}

kronq_status kronq_layer_loss(kronq_stream_t stream, const float *W_ref,
                              const float *W_hat, const float *H_X,
                              const float *H_G, int64_t d_out, int64_t d_in,
                              double *loss_dev, void *ws, size_t ws_bytes,
                              int32_t *info_dev) {
  if (!W_ref || !W_hat || !H_X || !H_G || !loss_dev || !ws || !info_dev ||
      d_out <= 0 || d_in <= 0)
    return KRONQ_ERR_INVALID_ARG;
  if (d_in % 128 || d_out % 128) return KRONQ_ERR_UNSUPPORTED;
  if (!aligned(ws, 256) || !aligned(W_ref, 16) || !aligned(W_hat, 16) ||
      !aligned(H_X, 16) || !aligned(H_G, 16))
    return KRONQ_ERR_INVALID_ARG;
  if (ws_bytes < loss_ws_bytes(d_out, d_in)) return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  return layer_loss(st, W_ref, W_hat, H_X, H_G, d_out, d_in, loss_dev, ws,
                    ws_bytes, info_dev);
}

size_t kronq_matvec_desc_bytes(const kronq_opts *opts, int64_t d_out, int64_t d_in) {
  if (!opts || d_out <= 0 || d_in <= 0) return 0;
  return matvec_desc_bytes(d_out, d_in);
}

size_t kronq_matvec_workspace_bytes(int64_t d_out, int64_t d_in, int64_t n_tokens) {
  if (d_out <= 0 || d_in <= 0 || n_tokens <= 0) return 0;
  return matvec_ws_bytes(d_out, d_in, n_tokens);
}

namespace {
kronq_status check_matvec_opts(const kronq_opts *opts, int64_t d_out, int64_t d_in) {
  if (opts->bits < 2 || opts->bits > 4) return KRONQ_ERR_INVALID_ARG;
  if (opts->group != 32 && opts->group != 64 && opts->group != 128)
    return KRONQ_ERR_UNSUPPORTED;
  const bool rot_x = !(opts->flags & KRONQ_FLAG_NO_ROT_IN);
  const bool rot_g = !(opts->flags & KRONQ_FLAG_NO_ROT_OUT);
  if (rot_x && !rot_ok(opts->rot_in, d_in)) return KRONQ_ERR_UNSUPPORTED;
  if (rot_g && !rot_ok(opts->rot_out, d_out)) return KRONQ_ERR_UNSUPPORTED;
  if (d_in % opts->group || d_in % 32 || d_in > 65536 || d_out > 65536)
    return KRONQ_ERR_UNSUPPORTED;
  return KRONQ_OK;
}
}  // namespace

kronq_status kronq_matvec_prepare(kronq_stream_t stream, const kronq_opts *opts,
                                  const float *s_x, const float *s_g, int64_t d_out,
                                  int64_t d_in, void *desc, size_t desc_bytes) {
  if (!opts || !s_x || !s_g || !desc || d_out <= 0 || d_in <= 0) return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(check_matvec_opts(opts, d_out, d_in));
  if (!aligned(desc, 256) || desc_bytes < matvec_desc_bytes(d_out, d_in))
    return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  return matvec_prepare(as_stream(stream), *opts, s_x, s_g, d_out, d_in, desc);
}

kronq_status kronq_dequant_matvec(kronq_stream_t stream, const kronq_opts *opts,
                                  const void *desc, const uint32_t *codes,
                                  const float *scales, const uint8_t *zeros, int64_t d_out,
                                  int64_t d_in, const float *x, int64_t n_tokens, float *y,
                                  void *ws, size_t ws_bytes, int32_t *info_dev) {
  if (!opts || !desc || !codes || !scales || !zeros || !x || !y || !ws || !info_dev ||
      d_out <= 0 || d_in <= 0 || n_tokens <= 0)
    return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(check_matvec_opts(opts, d_out, d_in));
  if (n_tokens > 4096) return KRONQ_ERR_UNSUPPORTED;
  if (!aligned(desc, 256) || !aligned(ws, 256) || !aligned(codes, 16) || !aligned(x, 16) ||
      !aligned(y, 16) || ws_bytes < matvec_ws_bytes(d_out, d_in, n_tokens))
    return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  return dequant_matvec(st, *opts, desc, codes, scales, zeros, d_out, d_in, x, n_tokens, y, ws,
                        info_dev);
}

kronq_status kronq_selftest_timeout(kronq_stream_t stream, uint64_t limit_ns,
                                    int32_t *info_dev) {
  if (!info_dev || limit_ns == 0 || limit_ns > kSelftestMaxNs)
    return KRONQ_ERR_INVALID_ARG;
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  return launch_selftest_timeout(st, limit_ns, info_dev);
}

kronq_status kronq_gemm_f32(kronq_stream_t stream, int64_t M, int64_t N,
                            int64_t K, float alpha, const float *A, int64_t lda,
                            int a_mn, const float *B, int64_t ldb, int b_mn,
                            float beta, float *C, int64_t ldc, void *ws,
                            size_t ws_bytes, int32_t *info_dev) {
  if (M < 0 || N < 0 || K < 0 || !info_dev) return KRONQ_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return KRONQ_OK;
  if (!C || (K > 0 && (!A || !B))) return KRONQ_ERR_INVALID_ARG;
  const int64_t a_rows = a_mn ? K : M, a_cols = a_mn ? M : K;
  const int64_t b_rows = b_mn ? K : N, b_cols = b_mn ? N : K;
  if (ldc < N || (K > 0 && (lda < a_cols || ldb < b_cols))) return KRONQ_ERR_INVALID_ARG;
  if (!aligned(C, 16) || ldc % 4 || (K > 0 && (!aligned(A, 16) || !aligned(B, 16) ||
                                                lda % 4 || ldb % 4)))
    return KRONQ_ERR_UNSUPPORTED;
  if (K > 0) {
    auto overlap = [](const float *p, int64_t rows, int64_t ld, int64_t cols,
                      const float *q, int64_t qrows, int64_t qld, int64_t qcols) {
      const float *pe = p + (rows - 1) * ld + cols, *qe = q + (qrows - 1) * qld + qcols;
      return p < qe && q < pe;
    };
    if (overlap(C, M, ldc, N, A, a_rows, lda, a_cols) ||
        overlap(C, M, ldc, N, B, b_rows, ldb, b_cols))
      return KRONQ_ERR_INVALID_ARG;
  }
  KQ_TRY(require_sm100());
  cudaStream_t st = as_stream(stream);
  KQ_TRY(launch_set_int(st, info_dev, 0));
  GemmArgs g;
  g.M = M; g.N = N; g.K = K;
  g.A = A; g.lda = lda; g.a_mn = a_mn != 0;
  g.B = B; g.ldb = ldb; g.b_mn = b_mn != 0;
  g.C = C; g.ldc = ldc;
  g.alpha = alpha; g.beta = beta;
  if (ws && !aligned(ws, 256)) return KRONQ_ERR_INVALID_ARG;
  return gemm_f32(st, g, ws, ws ? ws_bytes : 0, info_dev);
}

size_t kronq_gemm_f32_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return gemm_scratch_bytes(M, N, K);
}

kronq_status kronq_allocate_bits(const double *score, const int64_t *numel,
                                 int n, double avg_budget, int *bits_out) {
  if (!score || !numel || !bits_out || n <= 0 || !(avg_budget >= 2.0))
    return KRONQ_ERR_INVALID_ARG;
  double total = 0.0;
  for (int i = 0; i < n; ++i) {
    if (numel[i] <= 0 || !isfinite(score[i])) return KRONQ_ERR_INVALID_ARG;
    total += static_cast<double>(numel[i]);
  }
  std::vector<int> order(n);
  std::iota(order.begin(), order.end(), 0);
  std::stable_sort(order.begin(), order.end(),
                   [&](int a, int b) { return score[a] > score[b]; });
  for (int i = 0; i < n; ++i) bits_out[i] = 2;
  double used = 2.0 * total;
  const double cap = avg_budget * total;
  for (int from = 2; from <= 3; ++from) {
    for (int k = 0; k < n; ++k) {
      const int i = order[k];
      if (bits_out[i] == from && used + static_cast<double>(numel[i]) <= cap) {
        bits_out[i] = from + 1;
        used += static_cast<double>(numel[i]);
      }
    }
  }
  return KRONQ_OK;
}

kronq_status kronq_linear(kronq_stream_t stream, const void *X, int64_t n, int64_t d_in,
                          int64_t ldx, const void *W, int64_t d_out, int64_t ldw,
                          const float *bias, kronq_act act, void *Z, int64_t ldz, const void *R,
                          int64_t ldr, void *Y, int64_t ldy, int32_t *info_dev) {
  if (n < 0 || d_in <= 0 || d_out <= 0 || !act_ok(act) || !info_dev || !W ||
      (n > 0 && (!X || !Y)) || !aligned(bias, 4) || !aligned(info_dev, 4))
    return KRONQ_ERR_INVALID_ARG;
  const View x = bf16_view(X, n, d_in, ldx), w = bf16_view(W, d_out, d_in, ldw),
             z = bf16_view(Z, n, d_out, ldz), r = bf16_view(R, n, d_out, ldr),
             y = bf16_view(Y, n, d_out, ldy), b = View{bias, d_out, 1, d_out, 4};
  KQ_TRY(check_views({x, w, z, r, y}));
  if (any_overlap({y, z}, {x, w, b}) || bad_alias(y, r) || overlap(z, r))
    return KRONQ_ERR_INVALID_ARG;
  if (n > kMaxRows || d_in > kMaxWidth || d_out > kMaxWidth) return KRONQ_ERR_UNSUPPORTED;
  if (n == 0) return KRONQ_OK;
  KQ_TRY(require_sm100());
  return guarded([&] {
    return linear_fwd(as_stream(stream), n, d_in, d_out, mat(x), mat(w), bias, act, mat(z), mat(r),
                      mat(y), info_dev);
  });
}

kronq_status kronq_linear_bwd(kronq_stream_t stream, const void *dY, int64_t lddy, const void *Z,
                              int64_t ldz, kronq_act act, const void *X, int64_t ldx,
                              const void *W, int64_t ldw, int64_t n, int64_t d_in, int64_t d_out,
                              void *dZ, int64_t lddz, float *db, const void *dXr, int64_t lddxr,
                              void *dX, int64_t lddx, void *dW, int64_t lddw,
                              int32_t *info_dev) {
  if (n < 0 || d_in <= 0 || d_out <= 0 || !act_ok(act) || !info_dev || !aligned(db, 4) ||
      !aligned(info_dev, 4) || (n > 0 && !dY) ||
      (n > 0 && act != KRONQ_ACT_NONE && (!Z || !dZ)) || (n > 0 && dW && !X) ||
      (n > 0 && dX && !W) || (dXr && !dX))
    return KRONQ_ERR_INVALID_ARG;
  const View dy = bf16_view(dY, n, d_out, lddy),
             z = bf16_view(act == KRONQ_ACT_NONE ? nullptr : Z, n, d_out, ldz),
             x = bf16_view(dW ? X : nullptr, n, d_in, ldx),
             w = bf16_view(dX ? W : nullptr, d_out, d_in, ldw), dz = bf16_view(dZ, n, d_out, lddz),
             dxr = bf16_view(dXr, n, d_in, lddxr), dx = bf16_view(dX, n, d_in, lddx),
             dw = bf16_view(dW, d_out, d_in, lddw), b = View{db, d_out, 1, d_out, 4};
  KQ_TRY(check_views({dy, z, x, w, dz, dxr, dx, dw}));
  if (bad_alias(dz, dy) || bad_alias(dz, z) || bad_alias(dx, dxr) ||
      any_overlap({dz, dx, dw, b}, {x, w}) || any_overlap({dx, dw, b}, {dy, z}) ||
      any_overlap({dz, dw, b}, {dxr}))
    return KRONQ_ERR_INVALID_ARG;
  if (n > kMaxRows || d_in > kMaxWidth || d_out > kMaxWidth) return KRONQ_ERR_UNSUPPORTED;
  KQ_TRY(require_sm100());
  return guarded([&] {
    return linear_bwd(as_stream(stream), n, d_in, d_out, mat(dy), mat(z), act, mat(x), mat(w),
                      mat(dz), db, mat(dxr), mat(dx), mat(dw), info_dev);
  });
}

kronq_status kronq_gated(kronq_stream_t stream, const void *X, int64_t n, int64_t d, int64_t ldx,
                         const void *Wg, const void *Wu, int64_t f, int64_t ldw, kronq_act act,
                         void *A, void *U, int64_t ldau, void *H, int64_t ldh,
                         int32_t *info_dev) {
  if (n < 0 || d <= 0 || f <= 0 || !act_ok(act) || !info_dev || !Wg || !Wu ||
      (n > 0 && (!X || !H)) || (A == nullptr) != (U == nullptr) || !aligned(info_dev, 4))
    return KRONQ_ERR_INVALID_ARG;
  const View x = bf16_view(X, n, d, ldx), wg = bf16_view(Wg, f, d, ldw),
             wu = bf16_view(Wu, f, d, ldw), a = bf16_view(A, n, f, ldau),
             u = bf16_view(U, n, f, ldau), h = bf16_view(H, n, f, ldh);
  KQ_TRY(check_views({x, wg, wu, a, u, h}));
  if (any_overlap({a, u, h}, {x, wg, wu})) return KRONQ_ERR_INVALID_ARG;
  if (n > kMaxRows || d > kMaxWidth || f > kMaxWidth) return KRONQ_ERR_UNSUPPORTED;
  if (n == 0) return KRONQ_OK;
  KQ_TRY(require_sm100());
  return guarded([&] {
    return gated_fwd(as_stream(stream), n, d, f, mat(x), mat(wg), mat(wu), act, mat(a), mat(u),
                     mat(h), info_dev);
  });
}

kronq_status kronq_gated_bwd(kronq_stream_t stream, const void *dH, int64_t lddh, const void *A,
                             const void *U, int64_t ldau, kronq_act act, const void *X,
                             int64_t ldx, const void *Wg, const void *Wu, int64_t ldw, int64_t n,
                             int64_t d, int64_t f, void *Gg, void *Gu, int64_t ldg,
                             const void *dXr, int64_t lddxr, void *dX, int64_t lddx, void *dWg,
                             void *dWu, int64_t lddw, int32_t *info_dev) {
  if (n < 0 || d <= 0 || f <= 0 || !act_ok(act) || !info_dev || !aligned(info_dev, 4) ||
      (n > 0 && (!dH || !A || !U || !Gg || !Gu)) || (dWg == nullptr) != (dWu == nullptr) ||
      (n > 0 && dWg && !X) || (n > 0 && dX && (!Wg || !Wu)) || (dXr && !dX))
    return KRONQ_ERR_INVALID_ARG;
  const View dh = bf16_view(dH, n, f, lddh), a = bf16_view(A, n, f, ldau),
             u = bf16_view(U, n, f, ldau), x = bf16_view(dWg ? X : nullptr, n, d, ldx),
             wg = bf16_view(dX ? Wg : nullptr, f, d, ldw),
             wu = bf16_view(dX ? Wu : nullptr, f, d, ldw), gg = bf16_view(Gg, n, f, ldg),
             gu = bf16_view(Gu, n, f, ldg), dxr = bf16_view(dXr, n, d, lddxr),
             dx = bf16_view(dX, n, d, lddx), dwg = bf16_view(dWg, f, d, lddw),
             dwu = bf16_view(dWu, f, d, lddw);
  KQ_TRY(check_views({dh, a, u, x, wg, wu, gg, gu, dxr, dx, dwg, dwu}));
  for (const View &g : {gg, gu})
    if (bad_alias(g, dh) || bad_alias(g, a) || bad_alias(g, u)) return KRONQ_ERR_INVALID_ARG;
  if (bad_alias(dx, dxr) || any_overlap({gg, gu, dx, dwg, dwu}, {x, wg, wu}) ||
      any_overlap({dx, dwg, dwu}, {dh, a, u}) || any_overlap({gg, gu, dwg, dwu}, {dxr}))
    return KRONQ_ERR_INVALID_ARG;
  if (n > kMaxRows || d > kMaxWidth || f > kMaxWidth) return KRONQ_ERR_UNSUPPORTED;
  KQ_TRY(require_sm100());
  return guarded([&] {
    return gated_bwd(as_stream(stream), n, d, f, mat(dh), mat(a), mat(u), act, mat(x), mat(wg),
                     mat(wu), mat(gg), mat(gu), mat(dxr), mat(dx), mat(dwg), mat(dwu), info_dev);
  });
}

kronq_status kronq_distill_fwd(kronq_stream_t stream, const void *Z, kronq_dtype zdtype,
                               int64_t n, int64_t vocab, int64_t ldz, const void *T,
                               kronq_dtype tdtype, const int32_t *idx, int64_t k, int64_t ldt,
                               float tau, const float *weight, float *loss, float *lse,
                               int32_t *info_dev) {
  if (n > 0 && (!loss || !lse)) return KRONQ_ERR_INVALID_ARG;
  return run_distill(stream, Z, zdtype, n, vocab, ldz, T, tdtype, idx, k, ldt, tau, weight, loss,
                     lse, nullptr, vocab, info_dev);
}

kronq_status kronq_distill_bwd(kronq_stream_t stream, const void *Z, kronq_dtype zdtype,
                               int64_t n, int64_t vocab, int64_t ldz, const void *T,
                               kronq_dtype tdtype, const int32_t *idx, int64_t k, int64_t ldt,
                               float tau, const float *weight, const float *lse, void *dZ,
                               int64_t lddz, int32_t *info_dev) {
  if (n > 0 && (!lse || !dZ)) return KRONQ_ERR_INVALID_ARG;
  return run_distill(stream, Z, zdtype, n, vocab, ldz, T, tdtype, idx, k, ldt, tau, weight,
                     nullptr, const_cast<float *>(lse), dZ, lddz, info_dev);
}

kronq_status kronq_distill_step(kronq_stream_t stream, const void *Z, kronq_dtype zdtype,
                                int64_t n, int64_t vocab, int64_t ldz, const void *T,
                                kronq_dtype tdtype, const int32_t *idx, int64_t k, int64_t ldt,
                                float tau, const float *weight, float *loss, float *lse, void *dZ,
                                int64_t lddz, int32_t *info_dev) {
  if (n > 0 && (!loss || !dZ)) return KRONQ_ERR_INVALID_ARG;
  return run_distill(stream, Z, zdtype, n, vocab, ldz, T, tdtype, idx, k, ldt, tau, weight, loss,
                     lse, dZ, lddz, info_dev);
}

uint64_t kronq_kernel_launches(void) { return launches(); }

const char *kronq_last_cuda_error(void) {
  return cudaGetErrorString(static_cast<cudaError_t>(last_cuda_error()));
}

}  // extern "C"
