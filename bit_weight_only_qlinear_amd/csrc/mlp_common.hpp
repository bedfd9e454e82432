// Device helpers shared by the MLP-block kernels: the gate's activation
// functions and their derivatives, and the codes of 8-bit checkpoints.
#pragma once

#include "device_common.hpp"
#include "qp_internal.hpp"

namespace qp {

// act(g) and act'(g) in fp32.  silu: g s, s (1 + g (1 - s)) with s the
// logistic function.  gelu (tanh form): with v = a (g + b g^3),
// a = sqrt(2 / pi), b = 0.044715 and t = tanh v = 1 - 2 / (1 + e^(2 v)):
// 1/2 (1 + t) = 1 / (1 + e^(-2 v)) =: s, so act = g s and
// act' = s + 2 g s (1 - s) a (1 + 3 b g^2) -- the logistic form again, with
// no cancellation of 1 + t and no overflow: e^(+inf) gives s = 0.  The
// reciprocal is the hardware's, within one unit in the last place.
template <int ACT>
__device__ __forceinline__ float act_sig(float g, float& slope) {
  if constexpr (ACT == ACT_SILU) {
    slope = 1.f;
    return __builtin_amdgcn_rcpf(1.f + __expf(-g));
  } else {
    constexpr float a2 = 1.5957691216057308f, b = 0.044715f;
    const float g2 = g * g;
    slope = a2 * fmaf(3.f * b, g2, 1.f);
    return __builtin_amdgcn_rcpf(1.f + __expf(-a2 * g * fmaf(b, g2, 1.f)));
  }
}
template <int ACT>
__device__ __forceinline__ float act_f(float g) {
  float sl;
  return g * act_sig<ACT>(g, sl);
}
// act(g) and act'(g) = s + g s (1 - s) slope.  The last product is taken as
// 0 where s is 0 or 1 (a large |g| would make it 0 times infinity).
template <int ACT>
__device__ __forceinline__ void act_fd(float g, float& f, float& d) {
  float sl;
  const float s = act_sig<ACT>(g, sl);
  const float m = s * (1.f - s);
  f = g * s;
  d = s + (m > 0.f ? g * sl * m : 0.f);
}

// Between a wave's LDS writes and its other lanes' reads of them: the LDS
// takes one wave's operations in order, so only the compiler has to keep it.
__device__ __forceinline__ void lds_turn() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace qp
