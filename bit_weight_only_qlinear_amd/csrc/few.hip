// MXFP4 products and gated pairs for few activation rows.
#include "few_kernels.hpp"

namespace qp {
namespace {

// Quads of tokens per pass.
int quads(int64_t M) { return M <= 4 ? 1 : M <= 8 ? 2 : 4; }

template <int MODE, bool XB, bool W>
FewFn mx_fn(int64_t M) {
  const int q = quads(M);
  return q == 1 ? k_few<F_MX4, XB, W, 1, MODE> : q == 2 ? k_few<F_MX4, XB, W, 2, MODE> : k_few<F_MX4, XB, W, 4, MODE>;
}
template <int MODE>
FewFn mx_fn(bool xb, bool whole, int64_t M) {
  if (whole) return xb ? mx_fn<MODE, true, true>(M) : mx_fn<MODE, false, true>(M);
  return xb ? mx_fn<MODE, true, false>(M) : mx_fn<MODE, false, false>(M);
}

}  // namespace

hipError_t launch_few(const Desc& d, const void* x, int xdt, int64_t M, const Bufs& b,
                      const void* bias, void* y, int ydt, hipStream_t s) {
  FewArgs a{};
  const size_t lds = fill(d, d.N, (M + 4 * quads(M) - 1) / (4 * quads(M)), false, quads(M), (int)(M < 16 ? M : 16), a);
  a.w[0] = a.w[1] = b;
  a.x = x;
  a.M = M;
  a.y = y;
  a.ydt = ydt;
  a.bias[0] = bias;
  a.bdt = xdt;
  const int64_t per = 4 * quads(M);
  hipLaunchKernelGGL(mx_fn<FM_LINEAR>(xdt == BF16, a.x_lds > 0, M), dim3((unsigned)(a.tiles * ((M + per - 1) / per))),
                     dim3(256), lds, s, a);
  return hipGetLastError();
}

hipError_t launch_few_gated(const Desc& d, const GatedArgs& g, hipStream_t s) {
  FewArgs a{};
  const size_t lds = fill(d, d.N, (g.M + 4 * quads(g.M) - 1) / (4 * quads(g.M)), true, quads(g.M), (int)(g.M < 16 ? g.M : 16), a);
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
  const int64_t per = 4 * quads(g.M);
  hipLaunchKernelGGL(mx_fn<FM_GATED>(g.xdt == BF16, a.x_lds > 0, g.M),
                     dim3((unsigned)(a.tiles * ((g.M + per - 1) / per))), dim3(256), lds, s, a);
  return hipGetLastError();
}

// The metadata of a pass's 32 rows has to fit LDS next to the activations of two
// steps and the sums.
bool few_fits(const Desc& d, bool pair) {
  FewArgs a{};
  return fill(d, 16, 1, pair, 1, 0, a) <= 112 * 1024;
}

}  // namespace qp
