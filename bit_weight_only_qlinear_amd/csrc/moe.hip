// A mixture-of-experts layer for few tokens: the router, the experts' two
// products (one launch each), and the sum over a token's experts.
#include "few_kernels.hpp"

namespace qp {
namespace {

// y [M, N] = sum over slots of weight x partial sum (fixed order).  A slot
// whose expert the token named before adds its weight to that one's sum; one
// outside the layer adds nothing.
__global__ void __launch_bounds__(256) k_combine(const float* __restrict__ part,
                                                 const int* __restrict__ ids,
                                                 const float* __restrict__ weights, int E, int topk,
                                                 int64_t N, void* y, int ydt) {
  const int64_t m = blockIdx.y;
  const int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;   // N % 32 == 0
  if (n >= N) return;
  int e[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    e[s] = s < topk ? ids[m * topk + s] : -1;
    if (e[s] >= E) e[s] = -1;
  }
  // all loads first: a slot's sum lies with the first slot of its expert
  float4 p[kSlots];
  float w[kSlots];
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    int f = s;
#pragma unroll
    for (int k = kSlots - 1; k >= 0; --k)
      if (k < s && e[k] == e[s]) f = k;
    const bool on = e[s] >= 0;   // slots past topk hold -1
    w[s] = on ? weights[m * topk + s] : 0.f;
    p[s] = on ? *reinterpret_cast<const float4*>(part + (m * topk + f) * N + n) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    v[0] = fmaf(w[s], p[s].x, v[0]);
    v[1] = fmaf(w[s], p[s].y, v[1]);
    v[2] = fmaf(w[s], p[s].z, v[2]);
    v[3] = fmaf(w[s], p[s].w, v[3]);
  }
  if (ydt == F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(y) + m * N + n) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = ydt == BF16 ? f32_to_bf16_rne(v[i]) : f32_to_f16_rne(v[i]);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + m * N + n) =
        make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
}

// ---- routing: logits in fp64, so that the choice between two experts next to
// each other does not depend on the order of additions.  A product of two fp16
// values is exact in fp32 (22 bits, 2^-48 .. 2^32); bf16's range is fp32's own, so
// that theirs would overflow or vanish there, and is multiplied in fp64.
template <bool XB>
__device__ __forceinline__ double dot8(const uint4 u, const uint4 v) {
  const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (XB) {
      s = fma((double)__uint_as_float(a[i] << 16), (double)__uint_as_float(b[i] << 16), s);
      s = fma((double)__uint_as_float(a[i] & 0xFFFF0000u), (double)__uint_as_float(b[i] & 0xFFFF0000u), s);
    } else {
      s += (double)(f16_to_f32(a[i] & 0xFFFFu) * f16_to_f32(b[i] & 0xFFFFu));
      s += (double)(f16_to_f32(a[i] >> 16) * f16_to_f32(b[i] >> 16));
    }
  }
  return s;
}
// A lane's part of a logit: columns 8 (lane + 64 (part + parts k)) ..., eight
// loads of each row in flight.
template <bool XB>
__device__ __forceinline__ double logit_part(const uint16_t* x, const uint16_t* r, int64_t K, int lane,
                                             int part, int parts) {
  const uint4* xv = reinterpret_cast<const uint4*>(x);
  const uint4* rv = reinterpret_cast<const uint4*>(r);
  const int n = (int)(K / 8), step = 64 * parts;   // K % 32 == 0
  double s = 0.0;
  for (int c0 = lane + 64 * part; c0 < n; c0 += 8 * step) {
    uint4 u[8], v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int c = c0 + k * step;
      u[k] = c < n ? xv[c] : make_uint4(0, 0, 0, 0);
      v[k] = c < n ? rv[c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s += dot8<XB>(u[k], v[k]);
  }
  return s;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

struct RouteArgs {
  const uint16_t* x;       // [M, K]
  const uint16_t* r;       // [E, K]
  int64_t M, K;
  int E, topk, score, norm;
  double* logits;          // [M, E]
  int* ids;
  float* weights;
};

// Token m's choice from its logits l [E] in LDS, by a block of `threads`.
// An expert's place is the number of those in front of it (a larger logit, or
// the same and a lower index), counted by several threads each; the first topk
// places are the choice.  NaN logits come after all numbers, infinities among
// them, and are never chosen: places that no number takes get expert -1 and weight
// 0.  Where the largest logit is infinite, a softmax's weights are NaN.
struct Choice {
  double l[kExperts];
  double part[16];
  int place[kExperts];
  double top[kSlots], w[kSlots];
  int id[kSlots];
};
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t m, Choice& c, int threads) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E;
  for (int e = tid; e < E; e += threads) c.place[e] = 0;
  if (tid < kSlots) {
    c.id[tid] = -1;
    c.top[tid] = -__builtin_inf();
  }
  __syncthreads();
  // threads per expert: a power of two
  int per = 1;
  while (2 * per * E <= threads) per *= 2;
  for (int i = tid; i < E * per; i += threads) {
    const int e = i / per, s = i % per;
    const double v = c.l[e];
    int n = 0;
    for (int k = s; k < E; k += per) {
      const double o = c.l[k];
      n += o > v || (o == v && k < e) ? 1 : 0;
    }
    if (v != v) n = kExperts;
    if (n) atomicAdd(&c.place[e], n);
  }
  __syncthreads();
  for (int e = tid; e < E; e += threads)
    if (c.place[e] < a.topk) {
      c.id[c.place[e]] = e;
      c.top[c.place[e]] = c.l[e];
    }
  __syncthreads();
  const double hi = c.top[0];
  double sum = 0.0;
  if (a.score == 0) {
    for (int e = tid; e < E; e += threads) sum += c.l[e] == c.l[e] ? exp(c.l[e] - hi) : 0.0;
    sum = wave_sum_f64(sum);
    if (lane == 0) c.part[wave] = sum;
    __syncthreads();
    sum = 0.0;
    for (int w = 0; w < threads / 64; ++w) sum += c.part[w];
  }
  if (tid < a.topk)
    c.w[tid] = c.id[tid] < 0 ? 0.0 : a.score == 0 ? exp(c.top[tid] - hi) / sum : 1.0 / (1.0 + exp(-c.top[tid]));
  __syncthreads();
  if (tid < a.topk) {
    double total = 0.0;
    for (int s = 0; s < a.topk; ++s) total += c.w[s];
    const double w = a.norm && c.id[tid] >= 0 && total != 0.0 ? c.w[tid] / total : c.w[tid];
    a.ids[m * a.topk + tid] = c.id[tid];
    a.weights[m * a.topk + tid] = (float)w;
  }
}

// One block per token: its logits, `parts` waves to each (a power of two, in
// one round of the 16 waves where E <= 8), then the choice.
template <bool XB>
__global__ void __launch_bounds__(1024) k_route(RouteArgs a) {
  __shared__ Choice c;
  __shared__ double s[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m = blockIdx.x;
  int parts = 1;
  while (2 * parts * a.E <= 16) parts *= 2;
  if (parts == 1) {
    for (int e = wave; e < a.E; e += 16) {
      const double v = wave_sum_f64(logit_part<XB>(a.x + m * a.K, a.r + (int64_t)e * a.K, a.K, lane, 0, 1));
      if (lane == 0) c.l[e] = v;
    }
  } else {
    const int e = wave / parts;
    if (e < a.E) {
      const double v = wave_sum_f64(
          logit_part<XB>(a.x + m * a.K, a.r + (int64_t)e * a.K, a.K, lane, wave % parts, parts));
      if (lane == 0) s[wave] = v;
    }
    __syncthreads();
    if ((int)threadIdx.x < a.E) {
      double v = 0.0;
      for (int p = 0; p < parts; ++p) v += s[threadIdx.x * parts + p];
      c.l[threadIdx.x] = v;
    }
  }
  __syncthreads();
  choose(a, m, c, 1024);
}
// A wave per logit, then a block per token.
template <bool XB>
__global__ void __launch_bounds__(256) k_logits(RouteArgs a) {
  const int lane = threadIdx.x & 63, e = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t m = blockIdx.y;
  if (e >= a.E) return;
  const double s = wave_sum_f64(logit_part<XB>(a.x + m * a.K, a.r + (int64_t)e * a.K, a.K, lane, 0, 1));
  if (lane == 0) a.logits[m * a.E + e] = s;
}
__global__ void __launch_bounds__(256) k_choose(RouteArgs a) {
  __shared__ Choice c;
  const int64_t m = blockIdx.x;
  for (int e = threadIdx.x; e < a.E; e += 256) c.l[e] = a.logits[m * a.E + e];
  __syncthreads();
  choose(a, m, c, 256);
}

template <int KIND, bool W, int MODE>
FewFn expert_fn(bool xb, int q) {
  if (q == 1) return xb ? k_few<KIND, true, W, 1, MODE> : k_few<KIND, false, W, 1, MODE>;
  return xb ? k_few<KIND, true, W, 2, MODE> : k_few<KIND, false, W, 2, MODE>;
}
template <int MODE>
FewFn expert_fn(int kind, bool xb, bool whole, int q) {
  switch (kind) {
    case F_MX4: return whole ? expert_fn<F_MX4, true, MODE>(xb, q) : expert_fn<F_MX4, false, MODE>(xb, q);
    case F_AFF4: return whole ? expert_fn<F_AFF4, true, MODE>(xb, q) : expert_fn<F_AFF4, false, MODE>(xb, q);
    case F_AFF4H: return whole ? expert_fn<F_AFF4H, true, MODE>(xb, q) : expert_fn<F_AFF4H, false, MODE>(xb, q);
    case F_Q4K: return whole ? expert_fn<F_Q4K, true, MODE>(xb, q) : expert_fn<F_Q4K, false, MODE>(xb, q);
    default: return whole ? expert_fn<F_SYM4, true, MODE>(xb, q) : expert_fn<F_SYM4, false, MODE>(xb, q);
  }
}

}  // namespace

bool moe_format(const Desc& d) { return few_kind(d) >= 0; }
int moe_max_tokens() { return kTok; }
int moe_max_experts() { return kExperts; }
int moe_max_topk() { return kSlots; }

namespace {
size_t round16(size_t n) { return (n + 15) / 16 * 16; }
}  // namespace

// h (16 bits) and the partial sums, [M topk] rows each, then the logits.
size_t moe_workspace_bytes(int64_t M, int topk, int E, int64_t K, int64_t inner) {
  return round16((size_t)M * topk * (size_t)inner * 2) + round16((size_t)M * topk * (size_t)K * 4) +
         round16((size_t)M * E * 8);
}

hipError_t launch_moe(const Desc& up, const Desc& down, const MoeArgs& m, hipStream_t s) {
  const int64_t inner = down.K, K = up.K;
  unsigned char* ws = static_cast<unsigned char*>(m.ws);
  void* h = ws;
  float* part = reinterpret_cast<float*>(ws + round16((size_t)m.M * m.topk * (size_t)inner * 2));
  double* logits = reinterpret_cast<double*>(reinterpret_cast<unsigned char*>(part) +
                                             round16((size_t)m.M * m.topk * (size_t)K * 4));
  const bool xb = m.xdt == BF16;
  if (m.router) {
    RouteArgs r{static_cast<const uint16_t*>(m.x), static_cast<const uint16_t*>(m.router), m.M, K, m.E,
                m.topk, m.score, m.norm, logits, m.ids, m.weights};
    if (m.E <= 16) {
      hipLaunchKernelGGL((xb ? k_route<true> : k_route<false>), dim3((unsigned)m.M), dim3(1024), 0, s, r);
    } else {
      hipLaunchKernelGGL((xb ? k_logits<true> : k_logits<false>), dim3((unsigned)((m.E + 3) / 4), (unsigned)m.M),
                         dim3(256), 0, s, r);
      hipLaunchKernelGGL(k_choose, dim3((unsigned)m.M), dim3(256), 0, s, r);
    }
  }
  const int64_t most = m.M * m.topk < m.E ? m.M * m.topk : m.E;
  // up to four tokens: the form that holds one quad, in fewer registers
  const int q = m.M <= 4 ? 1 : 2, tokens = (int)(m.M < 4 * q ? m.M : 4 * q);
  // at most so many tiles of 4 q tokens
  const int64_t tiles = (m.M * m.topk + most * (4 * q - 1)) / (4 * q), units = tiles < m.M * m.topk ? tiles : m.M * m.topk;
  // The inner activations are rounded to x's type, as the h of the gated pair is by
  // default: a layer equals its experts' own entry points, and the down projection
  // keeps 16-bit operands for its exact codes.  Next to fp32 ones y's relative L2
  // error grows from 1.65e-3 to 2.35e-3 in bf16, from 2.1e-4 to 2.9e-4 in fp16 (the first of
  // each is y's own rounding); two 16-bit parts would take that back for twice the
  // matrix instructions of the projection and half its tokens per pass.
  FewArgs a{};
  size_t lds = fill(up, inner, most, true, tokens, 4 * q, a);
  a.w[0] = m.gate;
  a.w[1] = m.up;
  a.x = m.x;
  a.M = m.M;
  a.y = h;
  a.ydt = m.xdt;
  a.act = m.act;
  a.ids = m.ids;
  a.E = m.E;
  a.topk = m.topk;
  hipLaunchKernelGGL(expert_fn<FM_UP>(few_kind(up), xb, a.x_lds > 0, q), dim3((unsigned)(a.tiles * units)), dim3(256), lds, s, a);
  lds = fill(down, K, most, false, tokens, 4 * q, a);
  a.w[0] = a.w[1] = m.down;
  a.x = h;
  a.y = part;
  hipLaunchKernelGGL(expert_fn<FM_DOWN>(few_kind(down), xb, a.x_lds > 0, q), dim3((unsigned)(a.tiles * units)), dim3(256), lds, s, a);
  hipLaunchKernelGGL(k_combine, dim3((unsigned)((K + 1023) / 1024), (unsigned)m.M), dim3(256), 0, s, part, m.ids,
                     m.weights, m.E, m.topk, K, m.y, m.ydt);
  return hipGetLastError();
}

}  // namespace qp
