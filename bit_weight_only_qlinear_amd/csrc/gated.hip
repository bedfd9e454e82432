// Gated pair of projections on packed weights, any K:
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u.
//
// A block owns 64 output features (one checkpoint group) and 4 activation
// rows; each of its 16 waves computes 4 features, its lanes taking every
// 64th chunk of 8 columns, weights dequantized in fp32.  Bounded by the
// dequantization arithmetic; a simple form that is right for every shape.
#include <algorithm>

#include "mlp_common.hpp"

namespace qp {
namespace {

constexpr int kGaRows = 4, kGaFeat = 64;

struct GaArgs {
  GatedArgs a;
  Desc d;
};

__device__ __forceinline__ float val16(uint32_t b, int bf) {
  return bf ? bf16_to_f32(b) : f16_to_f32(b);
}

// Weights k0 .. k0 + 7 of row n in fp32 (k0 % 8 == 0).
__device__ __forceinline__ void weights8(const Desc& d, const Bufs& b, int64_t n, int64_t k0,
                                         float (&w)[8]) {
  const int64_t K = d.K, e0 = n * K + k0;
  const uint32_t* qw = static_cast<const uint32_t*>(b.qweight);
  float S, T;
  if (d.fmt == AFFINE) {
    const int64_t g = n * (K / d.gs) + k0 / d.gs;
    S = meta_to_f32(static_cast<const uint16_t*>(b.scales)[g], d.meta == BF16);
    T = meta_to_f32(static_cast<const uint16_t*>(b.zeros)[g], d.meta == BF16);
  } else if (d.fmt == Q4K) {
    const uint32_t st = static_cast<const uint32_t*>(b.steps)[n * (K / 256) + k0 / 256];
    const int64_t g = n * (K / 32) + k0 / 32;
    S = (float)static_cast<const uint8_t*>(b.scales)[g] * f16_to_f32(st & 0xFFFFu);
    T = -S * ((float)static_cast<const uint8_t*>(b.zeros)[g] * f16_to_f32(st >> 16));
  } else if (d.fmt == Q6K) {
    S = (float)static_cast<const int8_t*>(b.scales)[n * (K / 16) + k0 / 16] *
        f16_to_f32(static_cast<const uint16_t*>(b.steps)[n * (K / 256) + k0 / 256]);
    T = -32.f * S;
  } else {
    S = static_cast<const float*>(b.scales)[n * (K / d.gs) + k0 / d.gs];
    T = -8.f * S;
  }
  if (d.fmt == AFFINE && d.bits == 8) {
    const uint32_t v0 = qw[e0 / 4], v1 = qw[e0 / 4 + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = fmaf((float)((v0 >> (8 * i)) & 255u), S, T);
      w[4 + i] = fmaf((float)((v1 >> (8 * i)) & 255u), S, T);
    }
  } else if (d.fmt == AFFINE && d.bits == 2) {
    const uint32_t v = qw[e0 / 16] >> (2 * (e0 % 16));
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = fmaf((float)((v >> (2 * i)) & 3u), S, T);
  } else {
    const uint32_t v = qw[e0 / 8];
    uint32_t h = 0;
    if (d.fmt == Q6K) h = static_cast<const uint32_t*>(b.qweight_hi)[e0 / 16] >> (2 * (e0 % 16));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = fmaf((float)(((v >> (4 * i)) & 15u) | (((h >> (2 * i)) & 3u) << 4)), S, T);
  }
}

__global__ void __launch_bounds__(1024) k_gated_any(GaArgs ga) {
  __shared__ float sg[kGaRows][kGaFeat], su[kGaRows][kGaFeat];
  const GatedArgs& a = ga.a;
  const Desc& d = ga.d;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * kGaFeat;
  const int xb = a.xdt == BF16;
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  for (int64_t m0 = (int64_t)blockIdx.y * kGaRows; m0 < a.M; m0 += (int64_t)gridDim.y * kGaRows) {
  __syncthreads();   // the rows before are stored
  for (int f = wave; f < kGaFeat; f += 16) {
    const int64_t n = n0 + f;
    float g[kGaRows] = {0.f, 0.f, 0.f, 0.f}, u[kGaRows] = {0.f, 0.f, 0.f, 0.f};
    if (n < d.N) {
      for (int64_t k = 8 * lane; k < d.K; k += 512) {
        float wg[8], wu[8];
        weights8(d, a.gate, n, k, wg);
        weights8(d, a.up, n, k, wu);
#pragma unroll
        for (int r = 0; r < kGaRows; ++r) {
          if (m0 + r >= a.M) break;
          const uint4 v = *reinterpret_cast<const uint4*>(x + (m0 + r) * d.K + k);
          const uint32_t b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float xv = val16((b[e / 2] >> (16 * (e & 1))) & 0xFFFFu, xb);
            g[r] = fmaf(xv, wg[e], g[r]);
            u[r] = fmaf(xv, wu[e], u[r]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kGaRows; ++r) {
      g[r] = wave_sum_all(g[r]);
      u[r] = wave_sum_all(u[r]);
      if (n < d.N) {
        if (a.bias_g) g[r] += val16(static_cast<const uint16_t*>(a.bias_g)[n], xb);
        if (a.bias_u) u[r] += val16(static_cast<const uint16_t*>(a.bias_u)[n], xb);
      }
      if (lane == 0) {
        sg[r][f] = g[r];
        su[r][f] = u[r];
      }
    }
  }
  __syncthreads();
  // wave r: the block's 64 features of row m0 + r
  const int64_t m = m0 + wave, n = n0 + lane;
  if (wave >= kGaRows || m >= a.M) continue;   // whole waves
  const float g = sg[wave][lane], u = su[wave][lane];
  if (n < d.N) {
    const float h = (a.act == ACT_SILU ? act_f<ACT_SILU>(g) : act_f<ACT_GELU_TANH>(g)) * u;
    const int64_t i = m * d.N + n;
    if (a.hdt == F32) static_cast<float*>(a.h)[i] = h;
    else static_cast<uint16_t*>(a.h)[i] =
        (uint16_t)(a.hdt == BF16 ? f32_to_bf16_rne(h) : f32_to_f16_rne(h));
  }
  if (a.gq) {   // features past N hold 0
    const float sc[2] = {div_rn(wave_max_all(fabsf(g)), 127.f), div_rn(wave_max_all(fabsf(u)), 127.f)};
    const int64_t ng = (d.N + kCkptGroup - 1) / kCkptGroup;
    if (n < d.N) {
      a.gq[m * d.N + n] = (int8_t)(sc[0] > 0.f ? rintf(div_rn(g, sc[0])) : 0.f);
      a.uq[m * d.N + n] = (int8_t)(sc[1] > 0.f ? rintf(div_rn(u, sc[1])) : 0.f);
    }
    if (lane == 0) {
      a.gs[m * ng + blockIdx.x] = sc[0];
      a.us[m * ng + blockIdx.x] = sc[1];
    }
  }
  }
}

}  // namespace

hipError_t launch_gated_any(const Desc& d, const GatedArgs& a, hipStream_t s) {
  GaArgs ga{a, d};
  hipLaunchKernelGGL(k_gated_any,
                     dim3((unsigned)((d.N + kGaFeat - 1) / kGaFeat),
                          (unsigned)std::min<int64_t>((a.M + kGaRows - 1) / kGaRows, 4096)),
                     dim3(1024), 0, s, ga);
  return hipGetLastError();
}

}  // namespace qp
