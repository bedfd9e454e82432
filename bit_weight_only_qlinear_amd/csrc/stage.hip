// Staging of a product's 16-bit operand D [M, N] for fp16 MFMA: every row is
// scaled by a power of two that brings its largest magnitude into [2^14,
// 2^15) (bf16's range does not fit fp16, and gradients are small), rounded
// once to fp16, and laid out in the B-fragment order of
// v_mfma_f32_32x32x16_f16: [step of 64 columns][slice of 16][32-row block]
// [chunk 2 r + h] 16-byte chunks, r the row in its block and h the half of the
// slice (lane r + 32 h of the fragment): columns 8 h .. + 7 of the slice, in
// order or (PERM) as (0,4,1,5,2,6,3,7), the order in which packed weights
// dequantize.  Rows past M and columns past N
// are 0, so a product needs no edge cases in its contraction.
//
// D is a given matrix, or for the gated pair's backward [dg | du], computed
// here from dh and the 8-bit checkpoints and also written out in the
// activation type.  (A bound on |dg| and |du| from dh and the scales alone
// would give exponents before any pass, but rows whose gates are all far
// negative would lose their bits to it.)
//
// k_stage_row, N % 8 == 0 and N <= 32768: one block per row, which it keeps in
// registers between the maximum and the fragments; every input is read, and
// dg and du computed, once.  A row's chunks of a fragment are 32 bytes of its
// 1 KiB, so the 32 rows of a block go to blocks of one XCD, whose L2 completes
// the lines.  k_stage_exp and k_stage, any N: row maxima, then one wave per
// 32 x 64 values.  In front of MXFP4 weights the first blocks take the largest scales
// of their columns (mx_tops).  Gated, 2048 x 14336
// (351 MB moved): 82 us, against 34 + 127 us in two passes.
#include "mlp_common.hpp"

namespace qp {
namespace {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  half2_t h;
  h.x = (_Float16)lo;
  h.y = (_Float16)hi;
  return __builtin_bit_cast(uint32_t, h);
}

struct StageK {
  const uint16_t* dy;
  const int8_t* gq;
  const float* gs;
  const int8_t* uq;
  const float* us;
  uint16_t* dg;
  uint16_t* du;
  uint4* xf;
  int* xe;
  int64_t M, N;
  int MB, T1;
  int lead;                  // first blocks: mx_tops (a multiple of 8, as XCDs go)
  const uint8_t* scales[2];
  uint8_t* tops;
  int parts;
  int64_t cols;
};

// Block `part` of a.parts: the largest scale byte below 255 of each 32 columns in
// its run of weight rows, of one layer or two.  A thread takes a column (several
// where there are more than threads) and, where there are fewer, some of the rows.
// The blocks run beside those that stage rows, so the pass over the scales (1/17 of
// the weights) costs no launch.
__device__ __forceinline__ void mx_tops(const StageK& a, int part) {
  if (part >= a.parts) return;
  __shared__ uint32_t top[1024];
  const uint32_t nt = blockDim.x, tid = threadIdx.x;
  const int64_t n0 = a.N * part / a.parts, n1 = a.N * (part + 1) / a.parts;
  const uint32_t width = a.cols < (int64_t)nt ? (uint32_t)a.cols : nt, groups = nt / width;
  const uint32_t g = tid / width, c = tid - g * width;
  for (int64_t c0 = 0; c0 < a.cols; c0 += width) {
    top[tid] = 0;
    __syncthreads();
    if (g < groups && c0 + c < a.cols) {
      uint32_t m = 0;   // bytes plus 1, of which a NaN's is 0
      for (int l = 0; l < 2; ++l) {
        if (!a.scales[l]) break;
        const uint8_t* p = a.scales[l] + c0 + c;
#pragma unroll 8
        for (int64_t n = n0 + g; n < n1; n += groups) m = max(m, (p[n * a.cols] + 1u) & 0xFFu);
      }
      atomicMax(&top[c], m);
    }
    __syncthreads();
    if (tid < width && c0 + tid < a.cols)
      a.tops[tops_at(c0 + tid, part, a.parts)] = (uint8_t)(top[tid] > 0 ? top[tid] - 1u : 0u);
    __syncthreads();
  }
}

template <bool BF>
__device__ __forceinline__ float dval(uint32_t b) {
  return BF ? bf16_to_f32(b) : f16_to_f32(b);
}

// Exponent that brings a largest magnitude of b into [2^14, 2^15).
__device__ __forceinline__ int row_exp(float b) { return b == 0.f ? 0 : 14 - ilogbf(fminf(b, 3.4e38f)); }

// dg and du of one value.
template <int ACT>
__device__ __forceinline__ void pre_grads(float dh, float g, float u, float& dg, float& du) {
  float f, d;
  act_fd<ACT>(g, f, d);
  dg = dh * u * d;
  du = dh * f;
}

// The 8 values n .. n + 7 of a row of dy (and of dg and du where GATED, into
// x and y); 0 past N and where !rok.  sg, su: the group's scales.
template <bool BF, bool GATED, bool V8, int ACT>
__device__ __forceinline__ void load8(const StageK& a, int64_t at, int64_t n, bool rok, float sg,
                                      float su, float (&x)[8], float (&y)[8]) {
  float v[8], gv[8], uv[8];
  if constexpr (V8) {
    const bool ok = rok && n < a.N;
    const uint4 u = ok ? *reinterpret_cast<const uint4*>(a.dy + at) : make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = dval<BF>((w[i / 2] >> (16 * (i & 1))) & 0xFFFFu);
    if constexpr (GATED) {
      const uint2 q = ok ? *reinterpret_cast<const uint2*>(a.gq + at) : make_uint2(0, 0);
      const uint2 p = ok ? *reinterpret_cast<const uint2*>(a.uq + at) : make_uint2(0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        gv[i] = (float)(int8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3))) * sg;
        uv[i] = (float)(int8_t)((i < 4 ? p.x : p.y) >> (8 * (i & 3))) * su;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool ok = rok && n + i < a.N;
      v[i] = ok ? dval<BF>(a.dy[at + i]) : 0.f;
      if constexpr (GATED) {
        gv[i] = ok ? (float)a.gq[at + i] * sg : 0.f;
        uv[i] = ok ? (float)a.uq[at + i] * su : 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (GATED) pre_grads<ACT>(v[i], gv[i], uv[i], x[i], y[i]);
    else x[i] = v[i];
  }
}

// Exponent of each row of D (rows up to MB * 32; 0 past M): e = 14 -
// floor(log2 b) with b the row's largest magnitude in D.
template <bool BF, bool GATED, bool V8, int ACT>
__global__ void __launch_bounds__(256) k_stage_exp(StageK a) {
  __shared__ float red[4];
  if ((int)blockIdx.x < a.lead) {
    mx_tops(a, (int)blockIdx.x);
    return;
  }
  const int64_t row = (int)blockIdx.x - a.lead;
  float b = 0.f;
  if (row < a.M) {
    const int64_t ng = (a.N + kCkptGroup - 1) / kCkptGroup;
    for (int64_t n = 8 * threadIdx.x; n < a.N; n += 8 * 256) {
      const int64_t g = row * ng + n / kCkptGroup;
      float x[8], y[8];
      load8<BF, GATED, V8, ACT>(a, row * a.N + n, n, true, GATED ? a.gs[g] : 0.f,
                                GATED ? a.us[g] : 0.f, x, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b = fmaxf(b, fabsf(x[i]));
        if constexpr (GATED) b = fmaxf(b, fabsf(y[i]));
      }
    }
  }
  b = wave_max_all(b);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = b;
  __syncthreads();
  b = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  if (threadIdx.x == 0) a.xe[row] = row_exp(b);
}

// One wave per 32 rows x 64 columns (one step): D as fp16 B fragments.
template <bool BF, bool GATED, bool V8, int ACT, bool PERM>
__global__ void __launch_bounds__(256) k_stage(StageK a) {
  const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (id >= (int64_t)a.MB * a.T1) return;   // whole waves
  const int lane = threadIdx.x & 63;
  const int t = (int)(id / a.MB), mb = (int)(id - (int64_t)t * a.MB);
  const int64_t row = (int64_t)mb * 32 + (lane & 31);
  const bool rok = row < a.M;
  const int64_t ng = (a.N + kCkptGroup - 1) / kCkptGroup;
  const int e = a.xe[row];
  float sg = 0.f, su = 0.f;
  if (GATED && rok) {
    sg = a.gs[row * ng + t];
    su = a.us[row * ng + t];
  }
  auto rnd = [](float f) { return BF ? f32_to_bf16_rne(f) : f32_to_f16_rne(f); };
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int64_t n = (int64_t)t * 64 + 16 * s + 8 * (lane >> 5);
    const int64_t at = row * a.N + n;
    float dg[8], du[8];
    load8<BF, GATED, V8, ACT>(a, at, n, rok, sg, su, dg, du);
    auto frag = [&](const float (&x)[8], int step) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = PERM ? pack2(ldexpf(x[i], e), ldexpf(x[i + 4], e))
                    : pack2(ldexpf(x[2 * i], e), ldexpf(x[2 * i + 1], e));
      a.xf[(((int64_t)step * 4 + s) * a.MB + mb) * 64 + 2 * (lane & 31) + (lane >> 5)] =
          make_uint4(h[0], h[1], h[2], h[3]);
    };
    frag(dg, t);
    if constexpr (GATED) {
      frag(du, t + a.T1);
      auto out = [&](uint16_t* p, const float (&x)[8]) {
        if (!p || !rok) return;
        if constexpr (V8) {
          if (n < a.N)
            *reinterpret_cast<uint4*>(p + at) =
                make_uint4(rnd(x[0]) | (rnd(x[1]) << 16), rnd(x[2]) | (rnd(x[3]) << 16),
                           rnd(x[4]) | (rnd(x[5]) << 16), rnd(x[6]) | (rnd(x[7]) << 16));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n + i < a.N) p[at + i] = (uint16_t)rnd(x[i]);
        }
      };
      out(a.dg, dg);
      out(a.du, du);
    }
  }
}

// One row per block of NT threads, NC chunks of 8 columns per thread.
template <bool BF, bool GATED, int ACT, bool PERM, int NT, int NC>
__global__ void __launch_bounds__(NT) k_stage_row(StageK a) {
  __shared__ float red[NT / 64];
  if ((int)blockIdx.x < a.lead) {
    mx_tops(a, (int)blockIdx.x);
    return;
  }
  const int bid = (int)blockIdx.x - a.lead;
  // 32 consecutive blocks of an XCD (every 8th block id) share a row block
  const int i0 = bid >> 3;
  const int mb = (i0 >> 5) * 8 + (bid & 7), r = i0 & 31;
  if (mb >= a.MB) return;   // whole blocks
  const int64_t row = (int64_t)mb * 32 + r;
  const bool rok = row < a.M;
  const uint32_t nq = rok ? (uint32_t)(a.N / 8) : 0u, np = (uint32_t)a.T1 * 8u;
  uint4 d[NC];
  uint2 gq[GATED ? NC : 1], uq[GATED ? NC : 1];
  float sg[GATED ? NC : 1], su[GATED ? NC : 1];
  const int64_t rrow = rok ? row : a.M - 1;   // rows past M: any that is there
  const int64_t base = rrow * a.N, gbase = rrow * a.T1;   // 64 columns per scale and step
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const uint32_t c = threadIdx.x + NT * i;
    const bool ok = c < nq;
    // unconditional loads (of the row's first chunk past its end; a zero dy
    // makes everything zero): all of them go out together
    const uint32_t cc = ok ? c : 0u;
    const uint4 v = reinterpret_cast<const uint4*>(a.dy + base)[cc];
    d[i] = make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
    if constexpr (GATED) {
      gq[i] = reinterpret_cast<const uint2*>(a.gq + base)[cc];
      uq[i] = reinterpret_cast<const uint2*>(a.uq + base)[cc];
      sg[i] = a.gs[gbase + cc / 8];
      su[i] = a.us[gbase + cc / 8];
    }
  }
  float x[NC][8], y[GATED ? NC : 1][8], b = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const uint32_t w[4] = {d[i].x, d[i].y, d[i].z, d[i].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = dval<BF>((w[e / 2] >> (16 * (e & 1))) & 0xFFFFu);
      if constexpr (GATED) {
        const float gv = (float)(int8_t)((e < 4 ? gq[i].x : gq[i].y) >> (8 * (e & 3))) * sg[i];
        const float uv = (float)(int8_t)((e < 4 ? uq[i].x : uq[i].y) >> (8 * (e & 3))) * su[i];
        pre_grads<ACT>(v, gv, uv, x[i][e], y[i][e]);
        b = fmaxf(b, fmaxf(fabsf(x[i][e]), fabsf(y[i][e])));
      } else {
        x[i][e] = v;
        b = fmaxf(b, fabsf(v));
      }
    }
  }
  b = wave_max_all(b);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = b;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) b = fmaxf(b, red[i]);
  const int e = row_exp(b);
  if (threadIdx.x == 0) a.xe[row] = e;
  auto rnd = [](float f) { return BF ? f32_to_bf16_rne(f) : f32_to_f16_rne(f); };
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const uint32_t c = threadIdx.x + NT * i;
    if (c < np) {
      auto frag = [&](const float (&v)[8], uint32_t step) {
        uint32_t h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          h[q] = PERM ? pack2(ldexpf(v[q], e), ldexpf(v[q + 4], e))
                      : pack2(ldexpf(v[2 * q], e), ldexpf(v[2 * q + 1], e));
        a.xf[(((int64_t)step * 4 + ((c >> 1) & 3u)) * a.MB + mb) * 64 + 2 * r + (c & 1u)] =
            make_uint4(h[0], h[1], h[2], h[3]);
      };
      frag(x[i], c >> 3);
      if constexpr (GATED) {
        frag(y[i], (c >> 3) + a.T1);
        auto out = [&](uint16_t* p, const float (&v)[8]) {
          if (p && c < nq)
            reinterpret_cast<uint4*>(p + base)[c] =
                make_uint4(rnd(v[0]) | (rnd(v[1]) << 16), rnd(v[2]) | (rnd(v[3]) << 16),
                           rnd(v[4]) | (rnd(v[5]) << 16), rnd(v[6]) | (rnd(v[7]) << 16));
        };
        out(a.dg, x[i]);
        out(a.du, y[i]);
      }
    }
  }
}

typedef void (*StageFn)(StageK);
template <bool BF, bool GATED, int ACT, bool PERM>
StageFn row_pick(uint32_t chunks, int* nt) {
  *nt = chunks <= 256 ? 256 : chunks <= 2048 ? 512 : 1024;
  return chunks <= 256    ? k_stage_row<BF, GATED, ACT, PERM, 256, 1>
         : chunks <= 512  ? k_stage_row<BF, GATED, ACT, PERM, 512, 1>
         : chunks <= 1024 ? k_stage_row<BF, GATED, ACT, PERM, 512, 2>
         : chunks <= 2048 ? k_stage_row<BF, GATED, ACT, PERM, 512, 4>
                          : k_stage_row<BF, GATED, ACT, PERM, 1024, 4>;
}
template <bool BF>
StageFn row_pick(bool gated, int act, bool perm, uint32_t chunks, int* nt) {
  if (!gated) return perm ? row_pick<BF, false, 0, true>(chunks, nt) : row_pick<BF, false, 0, false>(chunks, nt);
  return act == ACT_SILU ? row_pick<BF, true, ACT_SILU, false>(chunks, nt)
                         : row_pick<BF, true, ACT_GELU_TANH, false>(chunks, nt);
}
template <bool BF, bool V8>
void stage_pick(bool gated, int act, bool perm, StageFn* ex, StageFn* st) {
  if (!gated) {
    *ex = k_stage_exp<BF, false, V8, 0>;
    *st = perm ? k_stage<BF, false, V8, 0, true> : k_stage<BF, false, V8, 0, false>;
  } else if (act == ACT_SILU) {
    *ex = k_stage_exp<BF, true, V8, ACT_SILU>;
    *st = k_stage<BF, true, V8, ACT_SILU, false>;
  } else {
    *ex = k_stage_exp<BF, true, V8, ACT_GELU_TANH>;
    *st = k_stage<BF, true, V8, ACT_GELU_TANH, false>;
  }
}

}  // namespace

hipError_t launch_stage(const StageArgs& r, int dt, bool gated, int act, bool perm, hipStream_t s) {
  StageK a{r.d, r.gq, r.gs, r.uq, r.us, r.dg, r.du, static_cast<uint4*>(r.xf), r.xe, r.M, r.N,
           (int)((r.M + 31) / 32), (int)((r.N + 63) / 64), (r.tops_parts + 7) / 8 * 8, {r.scales[0], r.scales[1]}, r.tops,
           r.tops_parts, r.tops_cols};
  const bool bf = dt == BF16;
  if (r.N % 8 == 0 && r.N <= 32768) {
    int nt = 0;
    const uint32_t chunks = (uint32_t)a.T1 * 8u;
    StageFn fn = bf ? row_pick<true>(gated, act, perm, chunks, &nt)
                    : row_pick<false>(gated, act, perm, chunks, &nt);
    hipLaunchKernelGGL(fn, dim3((unsigned)(a.lead + (a.MB + 7) / 8 * 256)), dim3(nt), 0, s, a);
    return hipGetLastError();
  }
  StageFn ex, sf;
  if (r.N % 8 == 0) bf ? stage_pick<true, true>(gated, act, perm, &ex, &sf)
                       : stage_pick<false, true>(gated, act, perm, &ex, &sf);
  else bf ? stage_pick<true, false>(gated, act, perm, &ex, &sf)
          : stage_pick<false, false>(gated, act, perm, &ex, &sf);
  hipLaunchKernelGGL(ex, dim3((unsigned)(a.lead + a.MB * 32)), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sf, dim3((unsigned)(((int64_t)a.MB * a.T1 + 3) / 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qp
