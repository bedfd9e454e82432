// C ABI of libqlinear: argument validation, error reporting and dispatch to
// the HIP kernels.  The contract of every entry point is documented in
// include/qlinear.h.  Shape rules follow the pages: K divisible by the group
// size and by whole packed words (the Metal export path filters out layers
// whose weights are not divisible by 8); for the nested superscale formats
// K % 256 == 0 and one step per 256-weight super-block, with detailed
// messages on failure (ExecuTorch PR #20571 review: kernel-side validation).
#include <cmath>
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <mutex>
#include <string>

#include "../../include/qlinear.h"
#include "qp_internal.hpp"

namespace {

thread_local std::string g_err;

qp_status fail(qp_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

qp_status ok() {
  g_err.clear();
  return QP_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Validates the descriptor and copies it into the internal form.
qp_status check_desc(const qp_desc* d, qp::Desc* out) {
  if (!d) return fail(QP_EINVAL, "descriptor is NULL");
  if (d->reserved != 0) return fail(QP_EINVAL, "qp_desc.reserved must be 0");
  if (d->N <= 0 || d->K <= 0)
    return fail(QP_ESHAPE, "N and K must be positive (N=%lld, K=%lld)", (long long)d->N,
                (long long)d->K);
  if (d->N > (int64_t(1) << 31) || d->K > (int64_t(1) << 24))
    return fail(QP_EUNSUPPORTED, "N must be <= 2^31 and K <= 2^24 (N=%lld, K=%lld)",
                (long long)d->N, (long long)d->K);
  const int64_t N = d->N, K = d->K;
  const int gs = d->group_size;
  switch (d->fmt) {
    case QP_FMT_AFFINE: {
      if (d->bits != 2 && d->bits != 4 && d->bits != 8)
        return fail(QP_EUNSUPPORTED, "AFFINE bits must be 2, 4 or 8 (got %d)", d->bits);
      if (gs != 32 && gs != 64 && gs != 128)
        return fail(QP_EUNSUPPORTED, "AFFINE group_size must be 32, 64 or 128 (got %d)", gs);
      if (d->meta_dtype != QP_F16 && d->meta_dtype != QP_BF16)
        return fail(QP_EUNSUPPORTED, "AFFINE meta_dtype must be QP_F16 or QP_BF16 (got %d)",
                    d->meta_dtype);
      if (d->super_block != 0)
        return fail(QP_EINVAL, "AFFINE has no super-block (super_block must be 0, got %d)",
                    d->super_block);
      if (K % gs)
        return fail(QP_ESHAPE, "K=%lld is not a multiple of group_size=%d", (long long)K, gs);
      const int chunk = 128 / d->bits;  // codes per 16-byte chunk
      if (K % chunk)
        return fail(QP_ESHAPE, "K=%lld must be a multiple of %d for %d-bit codes (16-byte chunks)",
                    (long long)K, chunk, d->bits);
      break;
    }
    case QP_FMT_Q4K:
      if (d->bits != 4 || gs != 32 || d->super_block != 256)
        return fail(QP_EUNSUPPORTED,
                    "Q4K needs bits=4, group_size=32, super_block=256 (got %d, %d, %d)", d->bits,
                    gs, d->super_block);
      if (K % 256)
        return fail(QP_ESHAPE, "Q4K needs K %% 256 == 0 (K=%lld, n_super=K/256)", (long long)K);
      break;
    case QP_FMT_Q6K:
      if (d->bits != 6 || gs != 16 || d->super_block != 256)
        return fail(QP_EUNSUPPORTED,
                    "Q6K needs bits=6, group_size=16, super_block=256 (got %d, %d, %d)", d->bits,
                    gs, d->super_block);
      if (K % 256)
        return fail(QP_ESHAPE, "Q6K needs K %% 256 == 0 (K=%lld, n_super=K/256)", (long long)K);
      break;
    case QP_FMT_SYM4:
      if (d->bits != 4 || d->super_block != 0)
        return fail(QP_EUNSUPPORTED, "SYM4 needs bits=4 and super_block=0 (got %d, %d)", d->bits,
                    d->super_block);
      if (K % 32)
        return fail(QP_ESHAPE, "SYM4 needs K %% 32 == 0 (K=%lld)", (long long)K);
      if (!(gs == K || gs == 32 || gs == 64 || gs == 128))
        return fail(QP_EUNSUPPORTED, "SYM4 group_size must be K or 32, 64, 128 (got %d)", gs);
      if (K % gs)
        return fail(QP_ESHAPE, "K=%lld is not a multiple of group_size=%d", (long long)K, gs);
      break;
    case QP_FMT_MXFP4:
      if (d->bits != 4 || gs != 32 || d->super_block != 0)
        return fail(QP_EUNSUPPORTED, "MXFP4 needs bits=4, group_size=32, super_block=0 (got %d, %d, %d)",
                    d->bits, gs, d->super_block);
      if (K % 32)
        return fail(QP_ESHAPE, "MXFP4 needs K %% 32 == 0 (K=%lld)", (long long)K);
      break;
    default:
      return fail(QP_EINVAL, "unknown format %d", d->fmt);
  }
  out->fmt = d->fmt;
  out->bits = d->bits;
  out->gs = gs;
  out->sb = d->super_block;
  out->meta = d->meta_dtype;
  out->N = N;
  out->K = K;
  return QP_OK;
}

void sizes_of(const qp::Desc& d, size_t b[5]) {
  const size_t N = (size_t)d.N, K = (size_t)d.K;
  for (int i = 0; i < 5; ++i) b[i] = 0;
  switch (d.fmt) {
    case QP_FMT_AFFINE:
      b[0] = N * K * d.bits / 8;
      b[2] = N * (K / d.gs) * 2;
      b[3] = N * (K / d.gs) * 2;
      break;
    case QP_FMT_Q4K:
      b[0] = N * K / 2;
      b[2] = N * K / 32;
      b[3] = N * K / 32;
      b[4] = N * (K / 256) * 4;
      break;
    case QP_FMT_Q6K:
      b[0] = N * K / 2;
      b[1] = N * K / 4;
      b[2] = N * K / 16;
      b[4] = N * (K / 256) * 2;
      break;
    case QP_FMT_MXFP4:
      b[0] = N * K / 2;
      b[2] = N * K / 32;
      break;
    default:
      b[0] = N * K / 2;
      b[2] = N * (K / d.gs) * 4;
      break;
  }
}

const char* kBufName[5] = {"qweight", "qweight_hi", "scales", "zeros", "steps"};

// Every buffer the format uses must be a non-NULL, 16-byte aligned pointer.
qp_status check_weights(const qp::Desc& d, const qp_weights* w, bool codes_only) {
  if (!w) return fail(QP_EINVAL, "weights struct is NULL");
  size_t b[5];
  sizes_of(d, b);
  const void* p[5] = {w->qweight, w->qweight_hi, w->scales, w->zeros, w->steps};
  for (int i = 0; i < 5; ++i) {
    if (!b[i] || (codes_only && i >= 2)) continue;
    if (!p[i]) return fail(QP_EINVAL, "%s is NULL but the format needs %zu bytes", kBufName[i], b[i]);
    if (!aligned16(p[i])) return fail(QP_EALIGN, "%s is not 16-byte aligned", kBufName[i]);
  }
  return QP_OK;
}

qp::Bufs bufs_of(const qp_weights* w) {
  return qp::Bufs{w->qweight, w->qweight_hi, w->scales, w->zeros, w->steps};
}

qp_status hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(QP_EHIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

// The qGEMM rounds each dequantized weight once to fp16 (relative error up
// to 2^-11).  That error grows like sqrt(K) against the layer's element
// bound 1e-2 * ||x|| * max|w| / sqrt(K); the kernel is held to the bound up
// to K = 8192 (the largest K of the workloads it is verified on), and longer
// rows take the exact-code MFMA kernel instead.
// fp16-rounded weights hold the output bound up to K = 8192; per-channel
// SYM4 runs on exact codes and MXFP4 weights are fp16 numbers after a power of
// two per row (K up to 2^20: 32-bit tile offsets)
constexpr int64_t kGemmMaxK = 8192;
bool gemm_ok(const qp::Desc& d) {
  const bool exact = (d.fmt == qp::SYM4 && d.gs == d.K) || d.fmt == qp::MXFP4;
  return d.K % 64 == 0 && d.K <= (exact ? (int64_t(1) << 20) : kGemmMaxK);
}

}  // namespace

extern "C" {

int32_t qpack_abi_version(void) { return QP_ABI_VERSION; }

const char* qpack_last_error(void) { return g_err.c_str(); }

qp_status qpack_sizes(const qp_desc* d, size_t bytes_out[5]) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if (!bytes_out) return fail(QP_EINVAL, "bytes_out is NULL");
  sizes_of(dd, bytes_out);
  return ok();
}

qp_status qpack_quantize(const qp_desc* d, const float* W, const qp_weights* out, void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if (!W) return fail(QP_EINVAL, "W is NULL");
  if (!aligned16(W)) return fail(QP_EALIGN, "W is not 16-byte aligned");
  if ((st = check_weights(dd, out, false)) != QP_OK) return st;
  (void)hipGetLastError();
  return hip_status(qp::launch_quantize(dd, W, out->qweight, out->qweight_hi, out->scales,
                                        out->zeros, out->steps, (hipStream_t)stream),
                    "qpack_quantize launch");
}

qp_status qpack_quantize_hqq(const qp_desc* d, const float* W, const qp_weights* out,
                             int32_t iters, float lp_norm, float beta, float kappa,
                             void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if (dd.fmt != qp::AFFINE)
    return fail(QP_EUNSUPPORTED, "qpack_quantize_hqq takes the AFFINE format (got %d)", dd.fmt);
  if (iters < 0 || iters > 10000)
    return fail(QP_EINVAL, "iters must lie in [0, 10000] (got %d)", iters);
  if (!(lp_norm > 0.f && lp_norm <= 1.f))
    return fail(QP_EINVAL, "lp_norm must lie in (0, 1] (got %g)", (double)lp_norm);
  if (!(beta > 0.f && std::isfinite(beta)))
    return fail(QP_EINVAL, "beta must be positive and finite (got %g)", (double)beta);
  if (!(kappa > 0.f && std::isfinite(kappa)))
    return fail(QP_EINVAL, "kappa must be positive and finite (got %g)", (double)kappa);
  if (!W) return fail(QP_EINVAL, "W is NULL");
  if (!aligned16(W)) return fail(QP_EALIGN, "W is not 16-byte aligned");
  if ((st = check_weights(dd, out, false)) != QP_OK) return st;
  (void)hipGetLastError();
  return hip_status(qp::launch_quantize_hqq(dd, W, out->qweight, out->scales, out->zeros, iters,
                                            lp_norm, beta, kappa, (hipStream_t)stream),
                    "qpack_quantize_hqq launch");
}

qp_status qpack_unpack_codes(const qp_desc* d, const qp_weights* w, void* codes, void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if ((st = check_weights(dd, w, true)) != QP_OK) return st;
  if (!codes) return fail(QP_EINVAL, "codes is NULL");
  if (!aligned16(codes)) return fail(QP_EALIGN, "codes is not 16-byte aligned");
  (void)hipGetLastError();
  return hip_status(qp::launch_unpack(dd, bufs_of(w), codes, (hipStream_t)stream),
                    "qpack_unpack_codes launch");
}

qp_status qpack_pack_codes(const qp_desc* d, const void* codes, const qp_weights* out,
                           void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if ((st = check_weights(dd, out, true)) != QP_OK) return st;
  if (!codes) return fail(QP_EINVAL, "codes is NULL");
  if (!aligned16(codes)) return fail(QP_EALIGN, "codes is not 16-byte aligned");
  (void)hipGetLastError();
  return hip_status(
      qp::launch_pack(dd, codes, out->qweight, out->qweight_hi, (hipStream_t)stream),
      "qpack_pack_codes launch");
}

qp_status qpack_encode_nested(const qp_desc* d, const float* s, const float* z,
                              const qp_weights* out, int32_t* bad, void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if (dd.fmt != qp::Q4K && dd.fmt != qp::Q6K)
    return fail(QP_EUNSUPPORTED, "qpack_encode_nested takes the Q4K or Q6K format (got %d)", dd.fmt);
  if (!out) return fail(QP_EINVAL, "out is NULL");
  if (!s) return fail(QP_EINVAL, "s is NULL");
  if (dd.fmt == qp::Q4K && !z) return fail(QP_EINVAL, "Q4K needs the zero points z");
  if (dd.fmt == qp::Q6K && z) return fail(QP_EINVAL, "Q6K has no zero points: z must be NULL");
  if (!aligned16(s) || (z && !aligned16(z)) || (bad && !aligned16(bad)))
    return fail(QP_EALIGN, "s, z and bad must be 16-byte aligned");
  const void* need[3] = {out->scales, dd.fmt == qp::Q4K ? out->zeros : out->scales, out->steps};
  for (int i = 0; i < 3; ++i) {
    if (!need[i]) return fail(QP_EINVAL, "out->scales, out->zeros (Q4K) and out->steps must be set");
    if (!aligned16(need[i])) return fail(QP_EALIGN, "metadata buffers must be 16-byte aligned");
  }
  (void)hipGetLastError();
  return hip_status(qp::launch_encode_nested(dd, s, z, out->scales, out->zeros, out->steps,
                                             reinterpret_cast<int*>(bad), (hipStream_t)stream),
                    "qpack_encode_nested launch");
}

qp_status qpack_concat_n(const qp_desc* d_out, int32_t parts, const qp_desc* d_in,
                         const qp_weights* w_in, const qp_weights* out, void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d_out, &dd);
  if (st != QP_OK) return st;
  if (parts < 1) return fail(QP_EINVAL, "parts must be >= 1 (got %d)", parts);
  if (!d_in || !w_in || !out) return fail(QP_EINVAL, "d_in, w_in and out must not be NULL");
  if ((st = check_weights(dd, out, false)) != QP_OK) return st;
  int64_t rows = 0;
  for (int32_t i = 0; i < parts; ++i) {
    qp::Desc di;
    if ((st = check_desc(&d_in[i], &di)) != QP_OK) return st;
    const qp_desc& a = d_in[i];
    if (a.fmt != d_out->fmt || a.bits != d_out->bits || a.group_size != d_out->group_size ||
        a.super_block != d_out->super_block || a.meta_dtype != d_out->meta_dtype ||
        a.K != d_out->K)
      return fail(QP_EINVAL, "part %d differs from d_out in format, bits, group size, "
                  "super-block, metadata dtype or K", i);
    if ((st = check_weights(di, &w_in[i], false)) != QP_OK) return st;
    rows += a.N;
  }
  if (rows != dd.N)
    return fail(QP_ESHAPE, "the parts' N add up to %lld, d_out has N=%lld", (long long)rows,
                (long long)dd.N);
  // every buffer is N-leading with a fixed byte count per row: each part's
  // buffer lands right after the previous part's
  size_t off[5] = {0, 0, 0, 0, 0};
  void* dst[5] = {out->qweight, out->qweight_hi, out->scales, out->zeros, out->steps};
  (void)hipGetLastError();
  for (int32_t i = 0; i < parts; ++i) {
    qp::Desc di;
    check_desc(&d_in[i], &di);
    size_t b[5];
    sizes_of(di, b);
    const void* src[5] = {w_in[i].qweight, w_in[i].qweight_hi, w_in[i].scales, w_in[i].zeros,
                          w_in[i].steps};
    for (int q = 0; q < 5; ++q) {
      if (!b[q]) continue;
      const hipError_t e = hipMemcpyAsync(static_cast<unsigned char*>(dst[q]) + off[q], src[q],
                                          b[q], hipMemcpyDeviceToDevice, (hipStream_t)stream);
      if (e != hipSuccess) return hip_status(e, "qpack_concat_n copy");
      off[q] += b[q];
    }
  }
  return ok();
}

qp_status qpack_dequantize(const qp_desc* d, const qp_weights* w, void* W_out, int32_t out_dtype,
                           void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if ((st = check_weights(dd, w, false)) != QP_OK) return st;
  if (out_dtype != QP_F16 && out_dtype != QP_BF16 && out_dtype != QP_F32)
    return fail(QP_EINVAL, "out_dtype must be QP_F16, QP_BF16 or QP_F32 (got %d)", out_dtype);
  if (!W_out) return fail(QP_EINVAL, "W_out is NULL");
  if (!aligned16(W_out)) return fail(QP_EALIGN, "W_out is not 16-byte aligned");
  (void)hipGetLastError();
  return hip_status(qp::launch_dequant(dd, bufs_of(w), W_out, out_dtype, (hipStream_t)stream),
                    "qpack_dequantize launch");
}

}  // extern "C"

namespace {

enum Use { USE_GEMV, USE_SKINNY, USE_GEMM, USE_FEW };

// MXFP4 products: up to 8 rows the few-row kernel, whose codes lie four rows to a
// load (8 rows of 4096 x 14336 11.6 us, on 16-row matrix instructions 15.3; 16
// rows 21 and 15, 16 x 8192 x 8192 20 and 16); then those in tiles of 16 to 64
// rows; the qGEMM, 18 us per 1000 columns where its tiles do not fill the chip,
// for more than 16 rows and M N = 2^22 (256 x 4096 x 4096 25 and 80 us, 256 x 8192 x 8192 76 and 144, 256
// x 4096 x 14336 69 and 80, 128 x 5120 x 25600 80 and 97).  Gated pairs: few rows up to 16.
constexpr int64_t kQuadRows = 8, kFewRows = 16, kFewOutputs = int64_t(1) << 22;
constexpr int64_t kMxFewRows = 64, kMxFewTiles = 32;   // both operands MXFP4

// Checks the forward arguments that do not involve a workspace and picks the
// kernel family.
qp_status plan_forward(const qp_desc* d, qp::Desc* dd, int32_t x_dtype, int64_t M,
                       int32_t kernel, Use* use, size_t nbytes[5]) {
  qp_status st = check_desc(d, dd);
  if (st != QP_OK) return st;
  if (M <= 0) return fail(QP_ESHAPE, "M must be positive (got %lld)", (long long)M);
  if (M > (int64_t(1) << 24)) return fail(QP_EUNSUPPORTED, "M must be <= 2^24");
  if (x_dtype != QP_F16 && x_dtype != QP_BF16)
    return fail(QP_EINVAL, "x_dtype must be QP_F16 or QP_BF16 (got %d)", x_dtype);
  if (kernel != QP_KERNEL_AUTO && kernel != QP_KERNEL_GEMV && kernel != QP_KERNEL_GEMM &&
      kernel != QP_KERNEL_GEMV_MFMA)
    return fail(QP_EINVAL, "unknown kernel selector %d", kernel);
  if (kernel == QP_KERNEL_GEMM && !gemm_ok(*dd))
    return fail(QP_EUNSUPPORTED,
                "the qGEMM kernel (fp16-rounded weights) needs K %% 64 == 0 and K <= %lld, "
                "where it meets the output bound (K=%lld; per-channel SYM4 and MXFP4, whose weights "
                "it does not round: K <= 2^20); QP_KERNEL_AUTO and QP_KERNEL_GEMV_MFMA use exact codes at any K",
                (long long)kGemmMaxK, (long long)dd->K);
  sizes_of(*dd, nbytes);
  if (dd->fmt == qp::MXFP4) {
    // One kernel for few rows behind both qGEMV selectors, in tiles of 16
    // rows where K % 64 != 0 keeps more of them from the qGEMM.
    const bool fits = qp::few_fits(*dd);
    const bool many = M > kFewRows && M * dd->N > kFewOutputs;
    *use = kernel == QP_KERNEL_GEMM || (kernel == QP_KERNEL_AUTO && (many || !fits) && gemm_ok(*dd))
               ? USE_GEMM : USE_FEW;
    if (*use == USE_FEW && !fits)
      return fail(QP_EUNSUPPORTED, "MXFP4 rows of K=%lld are too long for the few-row kernel", (long long)dd->K);
    if (*use == USE_FEW && M * ((dd->N + 15) / 16) > (int64_t(1) << 30))
      return fail(QP_EUNSUPPORTED, "MXFP4 in tiles of 16 rows: M * N must be <= 2^34");
    return QP_OK;
  }
  bool small_bufs = (size_t)M * (size_t)dd->K * 2 < (size_t(1) << 31);
  for (int i = 0; i < 5; ++i) small_bufs = small_bufs && nbytes[i] < (size_t(1) << 31);
  const bool gemv_fits = qp::gemv_supported(*dd) && small_bufs;
  const bool skinny_fits = qp::skinny_supported(*dd) && small_bufs;
  if (kernel == QP_KERNEL_GEMV && !gemv_fits)
    return fail(QP_EUNSUPPORTED,
                "the qGEMV kernel needs K <= its register plan (K=%lld) and every buffer < 2 GiB",
                (long long)dd->K);
  if (kernel == QP_KERNEL_GEMV_MFMA && !skinny_fits)
    return fail(QP_EUNSUPPORTED,
                "the MFMA qGEMV kernel needs K %% 128 == 0 and every buffer < 2 GiB (K=%lld)",
                (long long)dd->K);
  if (kernel == QP_KERNEL_AUTO) {
    // The MFMA qGEMV runs one set of MFMAs per 16 activation rows instead of
    // one dot product per row and code pair.  Where it takes over from the
    // streaming qGEMV (timed on the decode layers): 2 rows for per-channel
    // SYM4 and 4-bit affine codes (11.2 vs 12.5 us on 14336 x 4096), 3 for
    // Q6K (20.8 vs 22.3 us on 8192 x 8192), 5 for 8-bit affine codes (at 4
    // rows the qGEMV still wins: 19.1 vs 20.7 us), 3 for the others (Q4K at
    // 2 rows: 24.7 on the qGEMV vs 35.4 us).  Past 16 rows the qGEMM, up to
    // the K where its fp16 weights hold the output bound; beyond that the
    // exact MFMA qGEMV in tiles of 16 activation rows.
    int64_t mfma_from = 3;
    if (dd->fmt == qp::SYM4 && dd->gs == dd->K) mfma_from = 2;
    else if (dd->fmt == qp::AFFINE && dd->bits == 4) mfma_from = 2;
    else if (dd->fmt == qp::AFFINE && dd->bits == 8) mfma_from = 5;
    if (M >= mfma_from && M <= 16 && skinny_fits) *use = USE_SKINNY;
    else if (M <= 8 && gemv_fits) *use = USE_GEMV;
    else if (gemm_ok(*dd)) *use = USE_GEMM;
    else if (skinny_fits) *use = USE_SKINNY;
    else if (gemv_fits) *use = USE_GEMV;
    else return fail(QP_EUNSUPPORTED, "no kernel supports K=%lld for this format", (long long)dd->K);
  } else {
    *use = kernel == QP_KERNEL_GEMM ? USE_GEMM : kernel == QP_KERNEL_GEMV_MFMA ? USE_SKINNY : USE_GEMV;
  }
  return QP_OK;
}

}  // namespace

namespace {

// Memory pool of each device for qlinear_forward's stream-ordered
// workspace, created on first use with that device current; it keeps what
// it has served (release threshold at the maximum), so later calls reuse
// that memory.  Held until the process ends.
constexpr int kPoolDevices = 64;
std::mutex g_pool_mu;
hipMemPool_t g_pool[kPoolDevices];

hipError_t forward_pool(hipMemPool_t* out) {
  *out = nullptr;
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kPoolDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_pool_mu);
  if (!g_pool[dev]) {
    hipMemPoolProps props = {};
    props.allocType = hipMemAllocationTypePinned;
    props.location.type = hipMemLocationTypeDevice;
    props.location.id = dev;
    hipMemPool_t p = nullptr;
    e = hipMemPoolCreate(&p, &props);
    if (e != hipSuccess) return e;
    uint64_t keep = ~uint64_t(0);
    e = hipMemPoolSetAttribute(p, hipMemPoolAttrReleaseThreshold, &keep);
    if (e != hipSuccess) {
      (void)hipMemPoolDestroy(p);
      return e;
    }
    g_pool[dev] = p;
  }
  *out = g_pool[dev];
  return hipSuccess;
}

}  // namespace

extern "C" {

qp_status qlinear_workspace_bytes(const qp_desc* d, int32_t x_dtype, int64_t M, int32_t kernel,
                                  size_t* bytes) {
  if (!bytes) return fail(QP_EINVAL, "bytes is NULL");
  *bytes = 0;
  qp::Desc dd;
  Use use;
  size_t nbytes[5];
  qp_status st = plan_forward(d, &dd, x_dtype, M, kernel, &use, nbytes);
  if (st != QP_OK) return st;
  if (use == USE_GEMM) *bytes = qp::gemm_workspace_bytes(dd, M);
  return ok();
}

qp_status qlinear_forward_ws(const qp_desc* d, const void* x, int32_t x_dtype, int64_t M,
                             const qp_weights* w, const void* bias, void* y, int32_t y_dtype,
                             int32_t kernel, void* workspace, size_t workspace_bytes,
                             void* stream) {
  qp::Desc dd;
  Use use;
  size_t nbytes[5];
  qp_status st = plan_forward(d, &dd, x_dtype, M, kernel, &use, nbytes);
  if (st != QP_OK) return st;
  if ((st = check_weights(dd, w, false)) != QP_OK) return st;
  if (y_dtype != QP_F16 && y_dtype != QP_BF16 && y_dtype != QP_F32)
    return fail(QP_EINVAL, "y_dtype must be QP_F16, QP_BF16 or QP_F32 (got %d)", y_dtype);
  if (!x) return fail(QP_EINVAL, "x is NULL");
  if (!y) return fail(QP_EINVAL, "y is NULL");
  if (!aligned16(x)) return fail(QP_EALIGN, "x is not 16-byte aligned");
  if (!aligned16(y)) return fail(QP_EALIGN, "y is not 16-byte aligned");
  if (bias && !aligned16(bias)) return fail(QP_EALIGN, "bias is not 16-byte aligned");
  if (workspace && !aligned16(workspace))
    return fail(QP_EALIGN, "workspace is not 16-byte aligned");
  void* ws = nullptr;
  if (use == USE_GEMM && workspace) {
    const size_t need = qp::gemm_workspace_bytes(dd, M);
    if (need > 0) {
      if (workspace_bytes < need)
        return fail(QP_EINVAL, "workspace too small: %zu bytes, this call needs %zu",
                    workspace_bytes, need);
      ws = workspace;
    }
  }
  (void)hipGetLastError();
  hipError_t e;
  const char* what;
  if (use == USE_GEMM) {
    e = qp::launch_gemm(dd, x, x_dtype, M, bufs_of(w), bias, y, y_dtype, ws, (hipStream_t)stream);
    what = "qGEMM launch";
  } else if (use == USE_SKINNY) {
    e = qp::launch_skinny(dd, x, x_dtype, M, bufs_of(w), bias, y, y_dtype, nbytes,
                          (hipStream_t)stream);
    what = "MFMA qGEMV launch";
  } else if (use == USE_FEW) {
    e = (M > kQuadRows && qp::mx_rows_fits(dd) ? qp::launch_mx_rows : qp::launch_few)(
        dd, x, x_dtype, M, bufs_of(w), bias, y, y_dtype, (hipStream_t)stream);
    what = "few-row MXFP4 launch";
  } else {
    e = qp::launch_gemv(dd, x, x_dtype, M, bufs_of(w), bias, y, y_dtype, nbytes,
                        (hipStream_t)stream);
    what = "qGEMV launch";
  }
  return hip_status(e, what);
}

qp_status qlinear_forward_static(const qp_desc* d, const void* x, int32_t x_dtype, int64_t M,
                                 const qp_weights* w, const void* bias, void* y, int32_t y_dtype,
                                 int32_t kernel, void* stream) {
  qp::Desc dd;
  Use use;
  size_t nbytes[5];
  qp_status st = plan_forward(d, &dd, x_dtype, M, kernel, &use, nbytes);
  if (st != QP_OK) return st;
  void* ws = nullptr;
  size_t wsb = 0;
  if (use == USE_GEMM && qp::gemm_workspace_bytes(dd, M) > 0) {
    wsb = qp::gemm_workspace_bytes(dd, M);
    if (wsb > qp::static_scratch_bytes())
      return fail(QP_EUNSUPPORTED,
                  "qlinear_forward_static: this call stages %zu bytes of activations, more than "
                  "the library's static scratch (%zu bytes: ceil(M / 16) * 16 * (2 K + 4) "
                  "bytes at most); use qlinear_forward_ws with a workspace",
                  wsb, qp::static_scratch_bytes());
    (void)hipGetLastError();
    const hipError_t e = qp::static_scratch(&ws);
    if (e != hipSuccess) return hip_status(e, "static scratch lookup");
  }
  return qlinear_forward_ws(d, x, x_dtype, M, w, bias, y, y_dtype, kernel, ws, wsb, stream);
}

qp_status qlinear_forward_kernel(const qp_desc* d, const void* x, int32_t x_dtype, int64_t M,
                                 const qp_weights* w, const void* bias, void* y, int32_t y_dtype,
                                 int32_t kernel, void* stream) {
  return qlinear_forward_ws(d, x, x_dtype, M, w, bias, y, y_dtype, kernel, nullptr, 0, stream);
}

qp_status qlinear_forward(const qp_desc* d, const void* x, int32_t x_dtype, int64_t M,
                          const qp_weights* w, const void* bias, void* y, int32_t y_dtype,
                          void* stream) {
  // Where the qGEMM's 224-row tiling wants staged activations, take the
  // workspace stream-ordered from the library's pool and give it back on the
  // same stream after the qGEMM (no other call, on any stream, can see it in
  // between).  Under stream capture, or if the pool cannot serve it, run the
  // workspace-free tiling (same result, slower).
  qp::Desc dd;
  Use use;
  size_t nbytes[5];
  qp_status st = plan_forward(d, &dd, x_dtype, M, QP_KERNEL_AUTO, &use, nbytes);
  if (st != QP_OK) return st;
  const size_t need = use == USE_GEMM ? qp::gemm_workspace_bytes(dd, M) : 0;
  if (need > 0) {
    const hipStream_t s = (hipStream_t)stream;
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    hipMemPool_t pool = nullptr;
    void* ws = nullptr;
    if (hipStreamIsCapturing(s, &cs) == hipSuccess && cs == hipStreamCaptureStatusNone &&
        forward_pool(&pool) == hipSuccess &&
        hipMallocFromPoolAsync(&ws, need, pool, s) == hipSuccess) {
      st = qlinear_forward_ws(d, x, x_dtype, M, w, bias, y, y_dtype, QP_KERNEL_AUTO, ws, need,
                              stream);
      const hipError_t e = hipFreeAsync(ws, s);
      if (st == QP_OK && e != hipSuccess) return hip_status(e, "workspace release");
      return st;
    }
    (void)hipGetLastError();
  }
  return qlinear_forward_kernel(d, x, x_dtype, M, w, bias, y, y_dtype, QP_KERNEL_AUTO, stream);
}

}  // extern "C"

extern "C" {

qp_status qpack_quantize_activations(const void* x, int32_t x_dtype, int64_t M, int64_t K,
                                     void* xq, float* xs, void* stream) {
  if (x_dtype != QP_F16 && x_dtype != QP_BF16)
    return fail(QP_EINVAL, "x_dtype must be QP_F16 or QP_BF16 (got %d)", x_dtype);
  if (M <= 0 || K <= 0)
    return fail(QP_ESHAPE, "M and K must be positive (M=%lld, K=%lld)", (long long)M, (long long)K);
  if (M > (int64_t(1) << 31) - 1 || K > (int64_t(1) << 24))
    return fail(QP_EUNSUPPORTED, "M must be < 2^31 and K <= 2^24 (M=%lld, K=%lld)", (long long)M,
                (long long)K);
  if (!x || !xq || !xs) return fail(QP_EINVAL, "x, xq and xs must not be NULL");
  if (!aligned16(x) || !aligned16(xq) || !aligned16(xs))
    return fail(QP_EALIGN, "x, xq and xs must be 16-byte aligned");
  (void)hipGetLastError();
  return hip_status(qp::launch_quant_act(x, x_dtype, M, K, xq, xs, (hipStream_t)stream),
                    "qpack_quantize_activations launch");
}

qp_status qlinear_forward_a8w4(const qp_desc* d, const void* xq, const float* xs, int64_t M,
                               const qp_weights* w, const float* bias, void* y, int32_t y_dtype,
                               void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if (dd.fmt != qp::SYM4 || dd.gs != dd.K)
    return fail(QP_EUNSUPPORTED,
                "a8w4 takes the SYM4 format with one scale per output channel (group_size = K)");
  if (dd.K % 128)
    return fail(QP_ESHAPE, "a8w4 needs K %% 128 == 0 (K=%lld)", (long long)dd.K);
  if (M <= 0) return fail(QP_ESHAPE, "M must be positive (got %lld)", (long long)M);
  if ((uint64_t)M * (uint64_t)dd.K >= (uint64_t(1) << 31) ||
      (uint64_t)dd.N * (uint64_t)dd.K / 2 >= (uint64_t(1) << 31))
    return fail(QP_EUNSUPPORTED, "a8w4 needs the activations and the codes each < 2 GiB");
  if ((st = check_weights(dd, w, false)) != QP_OK) return st;
  if (y_dtype != QP_F16 && y_dtype != QP_BF16 && y_dtype != QP_F32)
    return fail(QP_EINVAL, "y_dtype must be QP_F16, QP_BF16 or QP_F32 (got %d)", y_dtype);
  if (!xq || !xs || !y) return fail(QP_EINVAL, "xq, xs and y must not be NULL");
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(y))
    return fail(QP_EALIGN, "xq, xs and y must be 16-byte aligned");
  if (bias && !aligned16(bias)) return fail(QP_EALIGN, "bias is not 16-byte aligned");
  (void)hipGetLastError();
  return hip_status(qp::launch_a8w4(dd, xq, xs, M, bufs_of(w), bias, y, y_dtype,
                                    (hipStream_t)stream),
                    "qlinear_forward_a8w4 launch");
}

}  // extern "C"

// ---- the MLP block: norm, checkpoints, gated pair, input gradients

namespace {

// One buffer argument: `need` says whether NULL is an error.
qp_status check_ptr(const void* p, const char* name, bool need) {
  if (!p) return need ? fail(QP_EINVAL, "%s is NULL", name) : QP_OK;
  if (!aligned16(p)) return fail(QP_EALIGN, "%s is not 16-byte aligned", name);
  return QP_OK;
}

struct PtrArg {
  const void* p;
  const char* name;
  bool need;
};
qp_status check_ptrs(std::initializer_list<PtrArg> args) {
  for (const PtrArg& a : args) {
    const qp_status st = check_ptr(a.p, a.name, a.need);
    if (st != QP_OK) return st;
  }
  return QP_OK;
}

// The bytes of one buffer of a call; out: written.  Outputs and workspaces
// must not reach into any other buffer (NULL and empty ones aside).
struct Span {
  const void* p;
  size_t n;
  const char* name;
  bool out;
};
qp_status check_apart(const Span* a, int count) {
  for (int i = 0; i < count; ++i) {
    if (!a[i].out || !a[i].p || !a[i].n) continue;
    const uintptr_t lo = reinterpret_cast<uintptr_t>(a[i].p), hi = lo + a[i].n;
    for (int j = 0; j < count; ++j) {
      if (j == i || !a[j].p || !a[j].n) continue;
      const uintptr_t b = reinterpret_cast<uintptr_t>(a[j].p);
      if (b < hi && lo < b + a[j].n)
        return fail(QP_EINVAL, "%s overlaps %s: they must be buffers of their own", a[i].name, a[j].name);
    }
  }
  return QP_OK;
}
template <int N>
qp_status check_apart(const Span (&a)[N]) {
  return check_apart(a, N);
}
// The five buffers of a layer, as spans.
void weight_spans(const qp::Desc& d, const qp_weights* w, Span* out) {
  const void* p[5] = {w->qweight, w->qweight_hi, w->scales, w->zeros, w->steps};
  size_t n[5];
  sizes_of(d, n);
  for (int i = 0; i < 5; ++i) out[i] = {p[i], n[i], kBufName[i], false};
}
size_t scale_bytes(int64_t M, int64_t n) {
  return (size_t)M * (size_t)((n + qp::kCkptGroup - 1) / qp::kCkptGroup) * 4u;
}

qp_status check_act_dtype(int32_t dt, const char* name) {
  if (dt != QP_F16 && dt != QP_BF16)
    return fail(QP_EINVAL, "%s must be QP_F16 or QP_BF16 (got %d)", name, dt);
  return QP_OK;
}
qp_status check_out_dtype(int32_t dt, const char* name) {
  if (dt != QP_F16 && dt != QP_BF16 && dt != QP_F32)
    return fail(QP_EINVAL, "%s must be QP_F16, QP_BF16 or QP_F32 (got %d)", name, dt);
  return QP_OK;
}

// Row kernels: launches of at most 2^32 threads (one block per row of up to
// 1024 threads; one thread per 8 columns, or per column where K % 8 != 0).
qp_status check_rows(int64_t M, int64_t K) {
  if (M <= 0 || K <= 0)
    return fail(QP_ESHAPE, "M and K must be positive (M=%lld, K=%lld)", (long long)M, (long long)K);
  if (M > (int64_t(1) << 21) || K > (int64_t(1) << 24) ||
      M * K > (int64_t(1) << (K % 8 ? 31 : 34)))
    return fail(QP_EUNSUPPORTED,
                "M must be <= 2^21, K <= 2^24 and M * K <= 2^34 (2^31 where K %% 8 != 0; M=%lld, "
                "K=%lld)",
                (long long)M, (long long)K);
  return QP_OK;
}

// Product kernels' sizes (block counts and 32-bit tile offsets).
qp_status check_block(const qp::Desc& d, int64_t M) {
  if (M <= 0) return fail(QP_ESHAPE, "M must be positive (got %lld)", (long long)M);
  if (M > (int64_t(1) << 20) || d.N > (int64_t(1) << 26) || M * d.N > (int64_t(1) << 36) ||
      M * d.K > (int64_t(1) << 36))
    return fail(QP_EUNSUPPORTED,
                "M must be <= 2^20, N <= 2^26, M * N and M * K <= 2^36 (M=%lld, N=%lld, K=%lld)",
                (long long)M, (long long)d.N, (long long)d.K);
  return QP_OK;
}

qp_status check_workspace(const void* ws, size_t have, size_t need) {
  if (!need) return QP_OK;
  if (!ws) return fail(QP_EINVAL, "workspace is NULL, this call needs %zu bytes", need);
  if (!aligned16(ws)) return fail(QP_EALIGN, "workspace is not 16-byte aligned");
  if (have < need)
    return fail(QP_EINVAL, "workspace too small: %zu bytes, this call needs %zu", have, need);
  return QP_OK;
}

// Which form of the gated pair a call takes.  With checkpoints, or above 16
// rows (one MFMA tile), or with a buffer of 2 GiB, the staged product; one row
// (two in some formats) streams the codes (int4 affine, 4096 -> 2 x 14336:
// 13.8 us in a graph, the MFMA tile with two rows 20.7), up to 16 rows the MFMA
// tile on exact codes.
enum GatedForm { GATED_GEMV, GATED_SKINNY, GATED_STAGED, GATED_FEW };
GatedForm gated_form(const qp::Desc& d, int64_t M, bool save) {
  if (d.fmt == qp::MXFP4)
    return save || M > kFewRows || !qp::few_fits(d) ? GATED_STAGED : GATED_FEW;
  size_t b[5];
  sizes_of(d, b);
  bool small_bufs = (size_t)M * (size_t)d.K * 2 < (size_t(1) << 31);
  for (int i = 0; i < 5; ++i) small_bufs = small_bufs && b[i] < (size_t(1) << 31);
  if (save || !small_bufs || M > 16) return GATED_STAGED;
  if (qp::gated_gemv_supported(d, M)) return GATED_GEMV;
  // Per-channel SYM4 sums (1024 + u) x (fp16) over the whole row before the
  // offset is taken away: about 2^-24 1024 K / 45 scales of rounding, against
  // an element bound of 0.07 scales for rows of unit activations -- a
  // fifteenth of it at K = 8192, more than all of it at 65536.  The staged
  // form sums q x.
  const bool long_row = d.fmt == qp::SYM4 && d.gs == d.K && d.K > 8192;
  return qp::skinny_supported(d) && !long_row ? GATED_SKINNY : GATED_STAGED;
}

}  // namespace

extern "C" {

qp_status qnorm_forward(const void* x, const void* residual, int32_t x_dtype, int64_t M, int64_t K,
                        const void* weight, float eps, void* s, void* y, void* yq, float* ys,
                        float* rstd, void* stream) {
  qp_status st = check_act_dtype(x_dtype, "x_dtype");
  if (st != QP_OK || (st = check_rows(M, K)) != QP_OK) return st;
  if (!(eps > 0.f && std::isfinite(eps)))
    return fail(QP_EINVAL, "eps must be positive and finite (got %g)", (double)eps);
  if (y ? (yq || ys) : (!yq || !ys))
    return fail(QP_EINVAL, "pass y, or yq and ys, and NULL for the other");
  if (s && !residual) return fail(QP_EINVAL, "s is written only with a residual (s = x without)");
  st = check_ptrs({{x, "x", true}, {residual, "residual", false}, {weight, "weight", false},
                   {s, "s", false}, {y, "y", false}, {yq, "yq", false}, {ys, "ys", false},
                   {rstd, "rstd", false}});
  if (st != QP_OK) return st;
  const void* out = y ? y : yq;
  if (out == x || out == residual || out == s || out == weight)
    return fail(QP_EINVAL, "the output must be a buffer of its own");
  const size_t rows = (size_t)M * (size_t)K * 2u;   // s may be x or residual itself
  st = check_apart({{x == s ? nullptr : x, rows, "x", false},
                    {residual == s ? nullptr : residual, rows, "residual", false},
                    {weight, (size_t)K * 2u, "weight", false}, {s, rows, "s", true},
                    {y, rows, "y", true}, {yq, rows / 2u, "yq", true}, {ys, (size_t)M * 4u, "ys", true},
                    {rstd, (size_t)M * 4u, "rstd", true}});
  if (st != QP_OK) return st;
  (void)hipGetLastError();
  return hip_status(qp::launch_norm(x, residual, x_dtype, M, K, weight, eps, s, y, yq, ys, rstd,
                                    (hipStream_t)stream),
                    "qnorm_forward launch");
}

qp_status qnorm_backward_workspace_bytes(int64_t M, int64_t K, size_t* bytes) {
  if (!bytes) return fail(QP_EINVAL, "bytes is NULL");
  *bytes = 0;
  const qp_status st = check_rows(M, K);
  if (st != QP_OK) return st;
  *bytes = (size_t)qp::norm_bwd_parts(M) * (size_t)K * 4u;
  return ok();
}

qp_status qnorm_backward(const void* dy, const void* s, const void* s_codes, const float* s_scales,
                         int32_t x_dtype, int64_t M, int64_t K, const void* weight,
                         const float* rstd, const void* ds_in, void* ds, float* dweight,
                         void* workspace, size_t workspace_bytes, void* stream) {
  qp_status st = check_act_dtype(x_dtype, "x_dtype");
  if (st != QP_OK || (st = check_rows(M, K)) != QP_OK) return st;
  if (s ? (s_codes || s_scales) : (!s_codes || !s_scales))
    return fail(QP_EINVAL, "pass s, or s_codes and s_scales, and NULL for the other");
  if (!ds && !dweight) return fail(QP_EINVAL, "ds and dweight are both NULL");
  st = check_ptrs({{dy, "dy", true}, {s, "s", false}, {s_codes, "s_codes", false},
                   {s_scales, "s_scales", false}, {weight, "weight", false}, {rstd, "rstd", true},
                   {ds_in, "ds_in", false}, {ds, "ds", false}, {dweight, "dweight", false}});
  if (st != QP_OK) return st;
  if (ds && (ds == s || ds == s_codes || ds == weight))
    return fail(QP_EINVAL, "ds must not be s, s_codes or weight");
  if (dweight) {
    st = check_workspace(workspace, workspace_bytes, (size_t)qp::norm_bwd_parts(M) * (size_t)K * 4u);
    if (st != QP_OK) return st;
  }
  const size_t rows = (size_t)M * (size_t)K * 2u;   // ds may be dy or ds_in itself
  st = check_apart({{dy == ds ? nullptr : dy, rows, "dy", false}, {s, rows, "s", false},
                    {s_codes, rows / 2u, "s_codes", false},
                    {s_scales, scale_bytes(M, K), "s_scales", false},
                    {weight, (size_t)K * 2u, "weight", false}, {rstd, (size_t)M * 4u, "rstd", false},
                    {ds_in == ds ? nullptr : ds_in, rows, "ds_in", false}, {ds, rows, "ds", true},
                    {dweight, (size_t)K * 4u, "dweight", true},
                    {dweight ? workspace : nullptr, (size_t)qp::norm_bwd_parts(M) * (size_t)K * 4u,
                     "workspace", true}});
  if (st != QP_OK) return st;
  (void)hipGetLastError();
  return hip_status(qp::launch_norm_bwd(dy, s, s_codes, s_scales, x_dtype, M, K, weight, rstd,
                                        ds_in, ds, dweight, static_cast<float*>(workspace),
                                        (hipStream_t)stream),
                    "qnorm_backward launch");
}

qp_status qpack_checkpoint(const void* x, int32_t x_dtype, int64_t M, int64_t K, void* codes,
                           float* scales, void* stream) {
  qp_status st = check_act_dtype(x_dtype, "x_dtype");
  if (st != QP_OK || (st = check_rows(M, K)) != QP_OK) return st;
  st = check_ptrs({{x, "x", true}, {codes, "codes", true}, {scales, "scales", true}});
  if (st != QP_OK) return st;
  st = check_apart({{x, (size_t)M * (size_t)K * 2u, "x", false},
                    {codes, (size_t)M * (size_t)K, "codes", true},
                    {scales, scale_bytes(M, K), "scales", true}});
  if (st != QP_OK) return st;
  (void)hipGetLastError();
  return hip_status(qp::launch_checkpoint(x, x_dtype, M, K, codes, scales, (hipStream_t)stream),
                    "qpack_checkpoint launch");
}

qp_status qpack_checkpoint_restore(const void* codes, const float* scales, int64_t M, int64_t K,
                                   void* x, int32_t x_dtype, void* stream) {
  qp_status st = check_out_dtype(x_dtype, "x_dtype");
  if (st != QP_OK || (st = check_rows(M, K)) != QP_OK) return st;
  st = check_ptrs({{codes, "codes", true}, {scales, "scales", true}, {x, "x", true}});
  if (st != QP_OK) return st;
  st = check_apart({{codes, (size_t)M * (size_t)K, "codes", false},
                    {scales, scale_bytes(M, K), "scales", false},
                    {x, (size_t)M * (size_t)K * (x_dtype == QP_F32 ? 4u : 2u), "x", true}});
  if (st != QP_OK) return st;
  (void)hipGetLastError();
  return hip_status(qp::launch_checkpoint_restore(codes, scales, M, K, x, x_dtype,
                                                  (hipStream_t)stream),
                    "qpack_checkpoint_restore launch");
}

qp_status qlinear_gated_workspace_bytes(const qp_desc* d, int64_t M, int32_t save, size_t* bytes) {
  if (!bytes) return fail(QP_EINVAL, "bytes is NULL");
  *bytes = 0;
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK || (st = check_block(dd, M)) != QP_OK) return st;
  if (gated_form(dd, M, save != 0) == GATED_STAGED) *bytes = qp::gated_workspace_bytes(dd, M);
  return ok();
}

qp_status qlinear_gated_forward(const qp_desc* d, const void* x, int32_t x_dtype, int64_t M,
                                const qp_weights* gate, const qp_weights* up, const void* bias_gate,
                                const void* bias_up, int32_t act, void* h, int32_t h_dtype,
                                void* gate_codes, float* gate_scales, void* up_codes,
                                float* up_scales, void* workspace, size_t workspace_bytes,
                                void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK || (st = check_act_dtype(x_dtype, "x_dtype")) != QP_OK ||
      (st = check_block(dd, M)) != QP_OK || (st = check_weights(dd, gate, false)) != QP_OK ||
      (st = check_weights(dd, up, false)) != QP_OK ||
      (st = check_out_dtype(h_dtype, "h_dtype")) != QP_OK)
    return st;
  if (act != QP_ACT_SILU && act != QP_ACT_GELU_TANH)
    return fail(QP_EINVAL, "unknown activation %d", act);
  const bool save = gate_codes || gate_scales || up_codes || up_scales;
  st = check_ptrs({{x, "x", true}, {h, "h", true}, {bias_gate, "bias_gate", false},
                   {bias_up, "bias_up", false}, {gate_codes, "gate_codes", save},
                   {gate_scales, "gate_scales", save}, {up_codes, "up_codes", save},
                   {up_scales, "up_scales", save}});
  if (st != QP_OK) return st;
  if (h == x || (save && (gate_codes == up_codes || gate_scales == up_scales)))
    return fail(QP_EINVAL, "h and the checkpoints must be buffers of their own");
  const GatedForm form = gated_form(dd, M, save);
  const size_t need = form == GATED_STAGED ? qp::gated_workspace_bytes(dd, M) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != QP_OK) return st;
  const size_t outs = (size_t)M * (size_t)dd.N;
  Span spans[19] = {{x, (size_t)M * (size_t)dd.K * 2u, "x", false},
                    {bias_gate, (size_t)dd.N * 2u, "bias_gate", false},
                    {bias_up, (size_t)dd.N * 2u, "bias_up", false},
                    {h, outs * (h_dtype == QP_F32 ? 4u : 2u), "h", true},
                    {gate_codes, outs, "gate_codes", true},
                    {gate_scales, scale_bytes(M, dd.N), "gate_scales", true},
                    {up_codes, outs, "up_codes", true},
                    {up_scales, scale_bytes(M, dd.N), "up_scales", true},
                    {workspace, need, "workspace", true}};
  weight_spans(dd, gate, spans + 9);
  weight_spans(dd, up, spans + 14);
  if ((st = check_apart(spans)) != QP_OK) return st;
  qp::GatedArgs a{x, x_dtype, h_dtype, act, M, bufs_of(gate), bufs_of(up), bias_gate, bias_up, h,
                  static_cast<int8_t*>(gate_codes), gate_scales, static_cast<int8_t*>(up_codes),
                  up_scales};
  const hipStream_t s = (hipStream_t)stream;
  (void)hipGetLastError();
  size_t nbytes[5];
  sizes_of(dd, nbytes);
  const hipError_t e = form == GATED_STAGED ? qp::launch_gated(dd, a, workspace, s)
                     : form == GATED_FEW    ? qp::launch_few_gated(dd, a, s)
                     : form == GATED_GEMV   ? qp::launch_gated_gemv(dd, a, nbytes, s)
                                            : qp::launch_gated_skinny(dd, a, nbytes, s);
  return hip_status(e, "qlinear_gated_forward launch");
}

qp_status qlinear_backward_workspace_bytes(const qp_desc* d, int64_t M, int32_t gated,
                                           size_t* bytes) {
  if (!bytes) return fail(QP_EINVAL, "bytes is NULL");
  *bytes = 0;
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK || (st = check_block(dd, M)) != QP_OK) return st;
  *bytes = qp::dx_workspace_bytes(dd, M, gated != 0);
  return ok();
}

qp_status qlinear_backward(const qp_desc* d, const void* dy, int32_t dy_dtype, int64_t M,
                           const qp_weights* w, void* dx, int32_t dx_dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK || (st = check_act_dtype(dy_dtype, "dy_dtype")) != QP_OK ||
      (st = check_block(dd, M)) != QP_OK || (st = check_weights(dd, w, false)) != QP_OK ||
      (st = check_out_dtype(dx_dtype, "dx_dtype")) != QP_OK ||
      (st = check_ptrs({{dy, "dy", true}, {dx, "dx", true}})) != QP_OK ||
      (st = check_workspace(workspace, workspace_bytes, qp::dx_workspace_bytes(dd, M, false))) != QP_OK)
    return st;
  if (dx == dy) return fail(QP_EINVAL, "dx must be a buffer of its own");
  Span spans[8] = {{dy, (size_t)M * (size_t)dd.N * 2u, "dy", false},
                   {dx, (size_t)M * (size_t)dd.K * (dx_dtype == QP_F32 ? 4u : 2u), "dx", true},
                   {workspace, qp::dx_workspace_bytes(dd, M, false), "workspace", true}};
  weight_spans(dd, w, spans + 3);
  if ((st = check_apart(spans)) != QP_OK) return st;
  qp::DxArgs a{};
  a.dy = dy;
  a.dydt = dy_dtype;
  a.dxdt = dx_dtype;
  a.M = M;
  a.w = a.w2 = bufs_of(w);
  a.dx = dx;
  a.ws = workspace;
  (void)hipGetLastError();
  return hip_status(qp::launch_dx(dd, a, (hipStream_t)stream), "qlinear_backward launch");
}

qp_status qlinear_gated_backward(const qp_desc* d, const void* dh, int32_t dh_dtype, int64_t M,
                                 const qp_weights* gate, const qp_weights* up, int32_t act,
                                 const void* gate_codes, const float* gate_scales,
                                 const void* up_codes, const float* up_scales, void* dgate,
                                 void* dup, void* dx, int32_t dx_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK || (st = check_act_dtype(dh_dtype, "dh_dtype")) != QP_OK ||
      (st = check_block(dd, M)) != QP_OK || (st = check_weights(dd, gate, false)) != QP_OK ||
      (st = check_weights(dd, up, false)) != QP_OK ||
      (st = check_out_dtype(dx_dtype, "dx_dtype")) != QP_OK)
    return st;
  if (act != QP_ACT_SILU && act != QP_ACT_GELU_TANH)
    return fail(QP_EINVAL, "unknown activation %d", act);
  st = check_ptrs({{dh, "dh", true}, {gate_codes, "gate_codes", true},
                   {gate_scales, "gate_scales", true}, {up_codes, "up_codes", true},
                   {up_scales, "up_scales", true}, {dgate, "dgate", false}, {dup, "dup", false},
                   {dx, "dx", true}});
  if (st != QP_OK) return st;
  if ((st = check_workspace(workspace, workspace_bytes, qp::dx_workspace_bytes(dd, M, true))) != QP_OK)
    return st;
  if (dx == dh || dgate == dh || dup == dh || (dgate && dgate == dup) || dgate == dx || dup == dx)
    return fail(QP_EINVAL, "dx, dgate and dup must be buffers of their own");
  const size_t ins = (size_t)M * (size_t)dd.N;
  Span spans[19] = {{dh, ins * 2u, "dh", false},
                    {gate_codes, ins, "gate_codes", false},
                    {gate_scales, scale_bytes(M, dd.N), "gate_scales", false},
                    {up_codes, ins, "up_codes", false},
                    {up_scales, scale_bytes(M, dd.N), "up_scales", false},
                    {dgate, ins * 2u, "dgate", true},
                    {dup, ins * 2u, "dup", true},
                    {dx, (size_t)M * (size_t)dd.K * (dx_dtype == QP_F32 ? 4u : 2u), "dx", true},
                    {workspace, qp::dx_workspace_bytes(dd, M, true), "workspace", true}};
  weight_spans(dd, gate, spans + 9);
  weight_spans(dd, up, spans + 14);
  if ((st = check_apart(spans)) != QP_OK) return st;
  qp::DxArgs a{};
  a.dy = dh;
  a.dydt = dh_dtype;
  a.dxdt = dx_dtype;
  a.act = act;
  a.M = M;
  a.w = bufs_of(gate);
  a.w2 = bufs_of(up);
  a.gated = true;
  a.gq = static_cast<const int8_t*>(gate_codes);
  a.gs = gate_scales;
  a.uq = static_cast<const int8_t*>(up_codes);
  a.us = up_scales;
  a.dg = dgate;
  a.du = dup;
  a.dx = dx;
  a.ws = workspace;
  (void)hipGetLastError();
  return hip_status(qp::launch_dx(dd, a, (hipStream_t)stream), "qlinear_gated_backward launch");
}

}  // extern "C"

// ---- MXFP4 activations and mixture-of-experts layers

extern "C" {

qp_status qpack_quantize_activations_mx(const void* x, int32_t x_dtype, int64_t M, int64_t K, void* xq,
                                        void* xs, void* stream) {
  qp_status st = check_out_dtype(x_dtype, "x_dtype");
  if (st != QP_OK) return st;
  if (M <= 0 || K <= 0)
    return fail(QP_ESHAPE, "M and K must be positive (M=%lld, K=%lld)", (long long)M, (long long)K);
  if (K % 32) return fail(QP_ESHAPE, "MXFP4 needs K %% 32 == 0 (K=%lld)", (long long)K);
  if (M > (int64_t(1) << 31) - 1 || K > (int64_t(1) << 24))
    return fail(QP_EUNSUPPORTED, "M must be < 2^31 and K <= 2^24 (M=%lld, K=%lld)", (long long)M,
                (long long)K);
  if ((st = check_ptrs({{x, "x", true}, {xq, "xq", true}, {xs, "xs", true}})) != QP_OK) return st;
  const size_t n = (size_t)M * (size_t)K;
  st = check_apart({{x, n * (x_dtype == QP_F32 ? 4u : 2u), "x", false}, {xq, n / 2, "xq", true},
                    {xs, n / 32, "xs", true}});
  if (st != QP_OK) return st;
  (void)hipGetLastError();
  return hip_status(qp::launch_mx_quant(x, x_dtype, M, K, xq, xs, (hipStream_t)stream),
                    "qpack_quantize_activations_mx launch");
}

qp_status qlinear_forward_mx(const qp_desc* d, const void* xq, const void* xs, int64_t M,
                             const qp_weights* w, const float* bias, void* y, int32_t y_dtype,
                             void* stream) {
  qp::Desc dd;
  qp_status st = check_desc(d, &dd);
  if (st != QP_OK) return st;
  if (dd.fmt != qp::MXFP4)
    return fail(QP_EUNSUPPORTED, "qlinear_forward_mx takes MXFP4 weights (got format %d)", dd.fmt);
  if ((st = check_block(dd, M)) != QP_OK || (st = check_weights(dd, w, false)) != QP_OK ||
      (st = check_out_dtype(y_dtype, "y_dtype")) != QP_OK ||
      (st = check_ptrs({{xq, "xq", true}, {xs, "xs", true}, {bias, "bias", false}, {y, "y", true}})) != QP_OK)
    return st;
  const size_t n = (size_t)M * (size_t)dd.K;
  Span spans[9] = {{xq, n / 2, "xq", false}, {xs, n / 32, "xs", false},
                   {bias, (size_t)dd.N * 4u, "bias", false},
                   {y, (size_t)M * (size_t)dd.N * (y_dtype == QP_F32 ? 4u : 2u), "y", true}};
  weight_spans(dd, w, spans + 4);
  if ((st = check_apart(spans)) != QP_OK) return st;
  (void)hipGetLastError();
  const bool fits = qp::mx_few_fits(dd, M);
  // The tiles' time does not depend on how few of them there are, the few-row
  // kernel's is proportional to M N: 128 x 14336 x 4096 (16 tiles) 52 and 20 us, 256
  // x 8192 x 8192 (32) 44 and 43, 384 x 8192 x 8192 (64) 43 and 62, 128 x 4096 x
  // 14336 (56) 19 and 27; up to 64 rows 64 x 5120 x 25600 (100) 33 and 29.  The tiles
  // need whole dwords of scale bytes per row, and 32-bit offsets inside a tile.
  const bool tiles = ((M > kMxFewRows && qp::mx_tiles(dd, M) > kMxFewTiles) || !fits) && dd.K % 128 == 0 && dd.K <= (int64_t(1) << 20);
  if (!tiles && !fits)
    return fail(QP_EUNSUPPORTED, "qlinear_forward_mx: K=%lld needs K %% 128 == 0 and K <= 2^20", (long long)dd.K);
  const hipStream_t s = (hipStream_t)stream;
  return hip_status(tiles ? qp::launch_mx_mx(dd, xq, xs, M, bufs_of(w), bias, y, y_dtype, s)
                          : qp::launch_mx_few(dd, xq, xs, M, bufs_of(w), bias, y, y_dtype, s),
                    "qlinear_forward_mx launch");
}

}  // extern "C"

namespace {

// The two descriptors of a layer of experts and its sizes.
qp_status check_moe(const qp_desc* d_up, const qp_desc* d_down, int64_t M, int32_t experts, int32_t topk,
                    qp::Desc* up, qp::Desc* down) {
  qp_status st = check_desc(d_up, up);
  if (st != QP_OK || (st = check_desc(d_down, down)) != QP_OK) return st;
  if (M <= 0) return fail(QP_ESHAPE, "M must be positive (got %lld)", (long long)M);
  if (M > qp::moe_max_tokens())
    return fail(QP_EUNSUPPORTED, "qmoe takes at most %d tokens (M=%lld)", qp::moe_max_tokens(), (long long)M);
  if (experts <= 0 || experts > qp::moe_max_experts())
    return fail(QP_EUNSUPPORTED, "experts must lie in [1, %d] (got %d)", qp::moe_max_experts(), experts);
  if (topk <= 0 || topk > experts || topk > qp::moe_max_topk())
    return fail(QP_EUNSUPPORTED, "topk must lie in [1, min(experts, %d)] (got %d)", qp::moe_max_topk(), topk);
  if (!qp::moe_format(*up) || !qp::moe_format(*down))
    return fail(QP_EUNSUPPORTED, "qmoe takes MXFP4, Q4K, SYM4 and 4-bit AFFINE weights");
  if (up->N % experts || down->N % experts)
    return fail(QP_ESHAPE, "the stacked N must be multiples of experts=%d (up N=%lld, down N=%lld)", experts,
                (long long)up->N, (long long)down->N);
  if (down->K != up->N / experts || up->K != down->N / experts)
    return fail(QP_ESHAPE,
                "an expert of %lld x %lld (up) needs a down projection of %lld x %lld, got %lld x %lld",
                (long long)(up->N / experts), (long long)up->K, (long long)up->K,
                (long long)(up->N / experts), (long long)(down->N / experts), (long long)down->K);
  if (M * topk * (up->K > down->K ? up->K : down->K) >= int64_t(1) << 29)
    return fail(QP_EUNSUPPORTED, "M * topk * max(K, inner) must be < 2^29 (M=%lld, topk=%d, K=%lld, inner=%lld)",
                (long long)M, topk, (long long)up->K, (long long)down->K);
  if (!qp::few_fits(*up) || !qp::few_fits(*down))
    return fail(QP_EUNSUPPORTED, "qmoe: rows of K=%lld or inner=%lld are too long (the metadata of 32 rows must "
                "fit LDS)", (long long)up->K, (long long)down->K);
  return QP_OK;
}

}  // namespace

extern "C" {

qp_status qmoe_workspace_bytes(const qp_desc* d_up, const qp_desc* d_down, int64_t M, int32_t experts,
                               int32_t topk, size_t* bytes) {
  if (!bytes) return fail(QP_EINVAL, "bytes is NULL");
  *bytes = 0;
  qp::Desc up, down;
  const qp_status st = check_moe(d_up, d_down, M, experts, topk, &up, &down);
  if (st != QP_OK) return st;
  *bytes = qp::moe_workspace_bytes(M, topk, experts, up.K, down.K);
  return ok();
}

qp_status qmoe_forward(const qp_desc* d_up, const qp_desc* d_down, int32_t experts, int32_t topk,
                       const void* x, int32_t x_dtype, int64_t M, const void* router, int32_t score,
                       int32_t norm, int32_t* ids, float* weights, const qp_weights* gate,
                       const qp_weights* up, const qp_weights* down, int32_t act, void* y,
                       int32_t y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  qp::Desc du, dd;
  qp_status st = check_moe(d_up, d_down, M, experts, topk, &du, &dd);
  if (st != QP_OK || (st = check_act_dtype(x_dtype, "x_dtype")) != QP_OK ||
      (st = check_out_dtype(y_dtype, "y_dtype")) != QP_OK ||
      (st = check_weights(du, gate, false)) != QP_OK || (st = check_weights(du, up, false)) != QP_OK ||
      (st = check_weights(dd, down, false)) != QP_OK)
    return st;
  if (score != QP_SCORE_SOFTMAX && score != QP_SCORE_SIGMOID)
    return fail(QP_EINVAL, "unknown score %d", score);
  if (norm != 0 && norm != 1) return fail(QP_EINVAL, "norm must be 0 or 1 (got %d)", norm);
  if (act != QP_ACT_SILU && act != QP_ACT_GELU_TANH)
    return fail(QP_EINVAL, "unknown activation %d", act);
  st = check_ptrs({{x, "x", true}, {router, "router", false}, {ids, "ids", true},
                   {weights, "weights", true}, {y, "y", true}});
  if (st != QP_OK) return st;
  const size_t need = qp::moe_workspace_bytes(M, topk, experts, du.K, dd.K);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != QP_OK) return st;
  const size_t rows = (size_t)M * (size_t)du.K, slots = (size_t)M * (size_t)topk * 4u;
  Span spans[21] = {{x, rows * 2u, "x", false},
                    {router, (size_t)experts * (size_t)du.K * 2u, "router", false},
                    {ids, slots, "ids", router != nullptr},
                    {weights, slots, "weights", router != nullptr},
                    {y, rows * (y_dtype == QP_F32 ? 4u : 2u), "y", true},
                    {workspace, need, "workspace", true}};
  weight_spans(du, gate, spans + 6);
  weight_spans(du, up, spans + 11);
  weight_spans(dd, down, spans + 16);
  if ((st = check_apart(spans)) != QP_OK) return st;
  const qp::MoeArgs m{x, x_dtype, y_dtype, act, score, norm, experts, topk, M, router, bufs_of(gate),
                      bufs_of(up), bufs_of(down), ids, weights, y, workspace};
  (void)hipGetLastError();
  return hip_status(qp::launch_moe(du, dd, m, (hipStream_t)stream), "qmoe_forward launch");
}

}  // extern "C"
