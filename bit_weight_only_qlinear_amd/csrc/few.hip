// MXFP4 products and gated pairs for few activation rows.
#include "few_kernels.hpp"

namespace qp {
namespace {

// Quads of tokens per pass.  Products of more than eight rows come here only
// where their scales are too long for the 16-row kernel's LDS.
template <int MODE>
int quads(int64_t M) { return M <= 4 ? 1 : M <= 8 || MODE == FM_LINEAR ? 2 : 4; }

template <int MODE, bool XB, bool W>
FewFn mx_fn(int q) {
  if constexpr (MODE != FM_LINEAR)
    if (q == 4) return k_few<F_MX4, XB, W, 4, MODE>;
  return q == 1 ? k_few<F_MX4, XB, W, 1, MODE> : k_few<F_MX4, XB, W, 2, MODE>;
}
template <int MODE>
FewFn mx_fn(bool xb, bool whole, int q) {
  if (whole) return xb ? mx_fn<MODE, true, true>(q) : mx_fn<MODE, false, true>(q);
  return xb ? mx_fn<MODE, true, false>(q) : mx_fn<MODE, false, false>(q);
}

// Sizes and launch of M rows in tiles of 4 q.
template <int MODE>
hipError_t launch(const Desc& d, int xdt, FewArgs& a, hipStream_t s) {
  int q = quads<MODE>(a.M);
  int64_t mt;
  size_t lds;
  for (;; q = 2) {   // a step of 16 rows takes 64 KiB of LDS: long rows in tiles of eight
    mt = (a.M + 4 * q - 1) / (4 * q);
    lds = fill(d, d.N, mt, is_pair(MODE), (int)(a.M < 4 * q ? a.M : 4 * q), 4 * q, a);
    if (q < 4 || a.x_lds || lds <= 80 * 1024) break;
  }
  hipLaunchKernelGGL(mx_fn<MODE>(xdt == BF16, a.x_lds > 0, q), dim3((unsigned)(a.tiles * mt)), dim3(256), lds, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few(const Desc& d, const void* x, int xdt, int64_t M, const Bufs& b,
                      const void* bias, void* y, int ydt, hipStream_t s) {
  FewArgs a{};
  a.w[0] = a.w[1] = b;
  a.x = x;
  a.M = M;
  a.y = y;
  a.ydt = ydt;
  a.bias[0] = bias;
  a.bdt = xdt;
  return launch<FM_LINEAR>(d, xdt, a, s);
}

hipError_t launch_few_gated(const Desc& d, const GatedArgs& g, hipStream_t s) {
  FewArgs a{};
  a.w[0] = g.gate;
  a.w[1] = g.up;
  a.x = g.x;
  a.M = g.M;
  a.y = g.h;
  a.ydt = g.hdt;
  a.bias[0] = g.bias_g;
  a.bias[1] = g.bias_u;
  a.bdt = g.xdt;
  a.act = g.act;
  return launch<FM_GATED>(d, g.xdt, a, s);
}

// The metadata of a gated pass's 32 rows has to fit LDS next to a step of eight rows of
// x (32 KiB), the sums and an expert's lists.
bool few_fits(const Desc& d) {
  FewArgs a{};
  return fill(d, 16, 1, true, 0, 0, a) <= 112 * 1024;
}

}  // namespace qp
