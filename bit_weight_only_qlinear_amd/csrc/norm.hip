// RMS norm with the residual's addition, forward (16-bit rows, or int8 rows
// with one scale each for the a8w4 path) and backward, and 8-bit activation
// checkpoints.
//
// Mathematics, per row of K values:
//   s = x + r (rounded once to the activation type, as it is kept);
//   rstd = (sum s^2 / K + eps)^(-1/2);  y = s w rstd.
//   int8: ys = fl32(max |y| / 127), yq = rint(y / ys).
//   backward: xh = s rstd, c = sum(dy w xh) / K,
//   ds = rstd (dy w - xh c) + ds_in;  dw[k] = sum over rows of dy xh.
// s w of two 16-bit values is exact in fp32 (at most 22 significant bits), so
// the int8 row needs only one reduction: sum s^2 and max |s w| together, and
// max |y| = rstd max |s w|.  (bf16 has fp32's range: a row whose largest |s w|
// is infinite in fp32, or so small that it may have lost bits, is read again and
// takes its products in fp64.)  The sum and the int8 quotient are held in fp64:
// a code then differs from the exact value's only within 1e-14 of a tie, and
// squares of large bf16 do not overflow.  Rows of whole 16-byte chunks are read
// once, kept in registers raw, and written once, bound by memory (2048 x 8192
// with a residual 21 to 24 us, 5.5 to 6.4 TB/s, some of it from the Infinity
// Cache; int8 rows 21 us, 5.5 TB/s, for all their 26 VALU instructions per
// value).  The general forms are bound by 2-byte loads, read twice (2048 x
// 8191: 67 us, int8 65).
//
// A checkpoint is one int8 code per value and an fp32 scale per 64 columns
// of a row: scale = fl32(max |x| / 127), code = rint(x / scale).
#include "device_common.hpp"
#include "qp_internal.hpp"

namespace qp {
namespace {

template <bool BF>
__device__ __forceinline__ float val16(uint32_t bits) {
  return BF ? bf16_to_f32(bits) : f16_to_f32(bits);
}
template <bool BF>
__device__ __forceinline__ uint32_t rnd16(float f) {
  return BF ? f32_to_bf16_rne(f) : f32_to_f16_rne(f);
}
template <bool BF>
__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = val16<BF>(w[i] & 0xFFFFu);
    v[2 * i + 1] = val16<BF>(w[i] >> 16);
  }
}
template <bool BF>
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = rnd16<BF>(v[2 * i]) | (rnd16<BF>(v[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void unpack8i(uint2 u, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (float)(int8_t)(u.x >> (8 * i));
    v[4 + i] = (float)(int8_t)(u.y >> (8 * i));
  }
}
__device__ __forceinline__ uint32_t pack4i(const int (&q)[8], int o) {
  return ((uint32_t)q[o] & 255u) | (((uint32_t)q[o + 1] & 255u) << 8) |
         (((uint32_t)q[o + 2] & 255u) << 16) | ((uint32_t)q[o + 3] << 24);
}

// p[c] where ok, else 0: the load itself is unconditional (p[0] is always
// there), so that a thread's loads go out together, without branches.
__device__ __forceinline__ uint4 ldz(const uint4* p, uint32_t c, bool ok) {
  const uint4 v = p[ok ? c : 0u];
  return make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
}
__device__ __forceinline__ uint2 ldz(const uint2* p, uint32_t c, bool ok) {
  const uint2 v = p[ok ? c : 0u];
  return make_uint2(ok ? v.x : 0u, ok ? v.y : 0u);
}

// v plus its neighbour by a DPP control; lanes without one add 0.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_add(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROW_MASK, 0xF, false);
  const uint32_t hi =
      (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROW_MASK, 0xF, false);
  return v + __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
// Sum over the wave, in lane 63.
__device__ __forceinline__ double wave_sum_d63(double v) {
  v = dpp_add<QP_DPP_QUAD_1032, 0xF>(v);
  v = dpp_add<QP_DPP_QUAD_2301, 0xF>(v);
  v = dpp_add<QP_DPP_ROW_ROR4, 0xF>(v);
  v = dpp_add<QP_DPP_ROW_ROR8, 0xF>(v);
  v = dpp_add<QP_DPP_ROW_BCAST15, 0xA>(v);
  return dpp_add<QP_DPP_ROW_BCAST31, 0xC>(v);
}
// Maximum of values >= 0 over the wave, in lane 63.
__device__ __forceinline__ float wave_max63(float v) {
  v = fmaxf(v, dpp_f<QP_DPP_QUAD_1032>(0.f, v));
  v = fmaxf(v, dpp_f<QP_DPP_QUAD_2301>(0.f, v));
  v = fmaxf(v, dpp_f<QP_DPP_ROW_ROR4>(0.f, v));
  v = fmaxf(v, dpp_f<QP_DPP_ROW_ROR8>(0.f, v));
  v = fmaxf(v, dpp_f<QP_DPP_ROW_BCAST15, 0xA>(0.f, v));
  return fmaxf(v, dpp_f<QP_DPP_ROW_BCAST31, 0xC>(0.f, v));
}

// Sum and maximum over the TPR threads of a row (a multiple of 64); every
// thread gets both.  red: one slot per wave of the block.
template <int TPR, bool MAX = true>
__device__ __forceinline__ void row_reduce(double& sum, float& mx, double* red_s, float* red_m) {
  sum = wave_sum_d63(sum);
  if constexpr (MAX) mx = wave_max63(mx);
  if constexpr (TPR == 64) {
    const uint64_t u = __builtin_bit_cast(uint64_t, sum);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    sum = __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
    mx = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mx), 63));
  } else {
    const int wave = threadIdx.x >> 6, w0 = wave / (TPR / 64) * (TPR / 64);
    __syncthreads();   // a row before may still read the slots
    if ((threadIdx.x & 63) == 63) {
      red_s[wave] = sum;
      if constexpr (MAX) red_m[wave] = mx;
    }
    __syncthreads();
    sum = 0.;
    mx = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) {   // the same order in every thread
      sum += red_s[w0 + i];
      if constexpr (MAX) mx = fmaxf(mx, red_m[w0 + i]);
    }
  }
}

// Whether a row's products s w need more than fp32's range, from the largest
// as fp32 numbers (codes other than 0 come from products of mx / 254 and more).
// A maximum of 0 is one under 2^-150, which rstd <= 2^16 leaves under bf16's
// smallest number: a row of zeros, as zero weights make it, stays ordinary.
// Alike in all threads of a row.
template <bool BF>
__device__ __forceinline__ bool wide_row(float mx, double rstd) {
  if constexpr (!BF) return false;
  const bool wide = !(mx >= 0x1p-100f && mx < __builtin_inff()) && (mx != 0.f || rstd > 0x1p16);
  return __builtin_amdgcn_readfirstlane(wide);
}
// s w rstd of such a row.
template <bool BF>
__device__ __forceinline__ double wide_y(uint32_t s, uint32_t w, double rstd) {
  return (double)val16<BF>(s) * (double)val16<BF>(w) * rstd;
}
__device__ __forceinline__ int wide_code(double y, float ys) {
  return ys > 0.f ? (int)fmin(fmax(rint(y / (double)ys), -127.), 127.) : 0;
}

// The int8 row's scale from max |s w| and rstd, and what s w is multiplied
// with to give the code before rounding (0 for a row of zeros).
__device__ __forceinline__ void q8_scale(float mx, double rstd, float& ys, double& mul) {
  ys = (float)((double)mx * rstd / 127.);
  mul = ys > 0.f ? rstd / (double)ys : 0.;
}
__device__ __forceinline__ int q8_code(float p, double mul) {
  const int q = (int)rint((double)p * mul);
  return q > 127 ? 127 : q < -127 ? -127 : q;
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* r;
  const uint16_t* w;
  uint16_t* s;
  uint16_t* y;
  int8_t* yq;
  float* ys;
  float* rstd;
  int64_t M, K;
  float eps;
};

// The rest of a wide row, its elements one by one: per thread V columns of
// every V * TPR, the ones whose stream it has stored itself (which may be in
// place of x or r).
template <bool BF, int TPR, int V>
__device__ __forceinline__ void wide_rest(const NormArgs& a, int64_t row, int t, double rstd,
                                          double* red_s, float* red_m) {
  const int64_t base = row * a.K;
  asm volatile("" ::: "memory");   // the stream's stores, of another type, come first
  auto each = [&](auto use) __attribute__((always_inline)) {
#pragma unroll 1
    for (int64_t c = (int64_t)t * V; c < a.K; c += TPR * V)
#pragma unroll 1
      for (int64_t k = c; k < c + V; ++k) {
        uint32_t b;
        if (a.r && a.s) b = a.s[base + k];
        else if (a.r) b = rnd16<BF>(val16<BF>(a.x[base + k]) + val16<BF>(a.r[base + k]));
        else b = a.x[base + k];
        use(k, wide_y<BF>(b, a.w ? a.w[k] : BF ? 0x3F80u : 0x3C00u, rstd));
      }
  };
  if (!a.yq) {
    each([&](int64_t k, double y) { a.y[base + k] = (uint16_t)rnd16<BF>((float)y); });
    return;
  }
  float mx = 0.f;
  double none = 0.;
  each([&](int64_t, double y) { mx = max_nan(mx, (float)(fabs(y) / 127.)); });
  none = mx - mx;   // NaN where the row is not finite: the maximum alone would lose it
  row_reduce<TPR>(none, mx, red_s, red_m);
  mx += (float)none;
  if (t == 0) a.ys[row] = mx;
  each([&](int64_t k, double y) { a.yq[base + k] = (int8_t)wide_code(y, mx); });
}

// One row per TPR threads, NU chunks of 8 columns per thread (K % 8 == 0,
// K <= 8 TPR NU).
template <bool BF, int TPR, int NU>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_norm(NormArgs a) {
  constexpr int NT = TPR < 256 ? 256 : TPR;
  __shared__ double red_s[NT / 64];
  __shared__ float red_m[NT / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
  if (TPR < 256 && row >= a.M) return;   // whole waves (TPR == 64 needs no barrier)
  const uint32_t nq = (uint32_t)(a.K / 8);
  const int64_t base = row * a.K;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + base);
  const uint4* rr = reinterpret_cast<const uint4*>(a.r + base);
  const uint4* wr = reinterpret_cast<const uint4*>(a.w);
  uint4 u[NU], w[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const uint32_t c = t + TPR * i;
    u[i] = c < nq ? xr[c] : make_uint4(0, 0, 0, 0);
  }
  if (a.r) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t c = t + TPR * i;
      w[i] = c < nq ? rr[c] : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float v[8], b[8];
      unpack8<BF>(u[i], v);
      unpack8<BF>(w[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += b[e];   // rounds to 24 bits, then to the type: one rounding
      u[i] = pack8<BF>(v);
    }
    if (a.s) {
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        const uint32_t c = t + TPR * i;
        if (c < nq) reinterpret_cast<uint4*>(a.s + base)[c] = u[i];
      }
    }
  }
  const uint32_t one = BF ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const uint32_t c = t + TPR * i;
    w[i] = a.w && c < nq ? wr[c] : make_uint4(one, one, one, one);
  }
  double sum = 0.;
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    float v[8], b[8];
    unpack8<BF>(u[i], v);
    unpack8<BF>(w[i], b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double d = v[e];
      sum = fma(d, d, sum);
      mx = fmaxf(mx, fabsf(v[e] * b[e]));
    }
  }
  row_reduce<TPR>(sum, mx, red_s, red_m);
  const double rstd = 1. / sqrt(sum / (double)a.K + (double)a.eps);
  if (a.rstd && t == 0) a.rstd[row] = (float)rstd;
  if (wide_row<BF>(mx, rstd)) {
    wide_rest<BF, TPR, 8>(a, row, t, rstd, red_s, red_m);
    return;
  }
  if (a.yq) {
    float ys;
    double mul;
    q8_scale(mx, rstd, ys, mul);
    if (t == 0) a.ys[row] = ys;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t c = t + TPR * i;
      float v[8], b[8];
      unpack8<BF>(u[i], v);
      unpack8<BF>(w[i], b);
      int q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = q8_code(v[e] * b[e], mul);
      if (c < nq)
        reinterpret_cast<uint2*>(a.yq + base)[c] = make_uint2(pack4i(q, 0), pack4i(q, 4));
    }
  } else {
    const float rs = (float)rstd;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t c = t + TPR * i;
      float v[8], b[8];
      unpack8<BF>(u[i], v);
      unpack8<BF>(w[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * b[e] * rs;
      if (c < nq) reinterpret_cast<uint4*>(a.y + base)[c] = pack8<BF>(v);
    }
  }
}

// Any K: scalar columns, two passes over the row.  s is written in the
// second pass only, after the thread has read the same element of x and r,
// so it may be either of them.
constexpr int kAny = 1024;   // threads of the general forms: a few columns each, for latency

template <bool BF>
__global__ void __launch_bounds__(kAny) k_norm_any(NormArgs a) {
  __shared__ double red_s[kAny / 64];
  __shared__ float red_m[kAny / 64];
  const int64_t row = blockIdx.x, base = row * a.K;
  auto stream = [&](int64_t k) {
    uint32_t b = a.x[base + k];
    if (a.r) b = rnd16<BF>(val16<BF>(b) + val16<BF>(a.r[base + k]));
    return b;
  };
  auto weight = [&](int64_t k) { return a.w ? val16<BF>(a.w[k]) : 1.f; };
  double sum = 0.;
  float mx = 0.f;
#pragma unroll 4
  for (int64_t k = threadIdx.x; k < a.K; k += kAny) {
    const float v = val16<BF>(stream(k));
    sum = fma((double)v, (double)v, sum);
    mx = fmaxf(mx, fabsf(v * weight(k)));
  }
  row_reduce<kAny>(sum, mx, red_s, red_m);
  const double rstd = 1. / sqrt(sum / (double)a.K + (double)a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = (float)rstd;
  if (wide_row<BF>(mx, rstd)) {
    if (a.r && a.s)
      for (int64_t k = threadIdx.x; k < a.K; k += kAny) a.s[base + k] = (uint16_t)stream(k);
    wide_rest<BF, kAny, 1>(a, row, threadIdx.x, rstd, red_s, red_m);
    return;
  }
  float ys;
  double mul;
  q8_scale(mx, rstd, ys, mul);
  if (a.yq && threadIdx.x == 0) a.ys[row] = ys;
  const float rs = (float)rstd;
#pragma unroll 4
  for (int64_t k = threadIdx.x; k < a.K; k += kAny) {
    const uint32_t b = stream(k);
    const float p = val16<BF>(b) * weight(k);
    if (a.r && a.s) a.s[base + k] = (uint16_t)b;
    if (a.yq) a.yq[base + k] = (int8_t)q8_code(p, mul);
    else a.y[base + k] = (uint16_t)rnd16<BF>(p * rs);
  }
}

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* s;     // the kept stream, or
  const int8_t* sq;      // its checkpoint: codes and scales
  const float* ss;
  const uint16_t* w;
  const float* rstd;
  const uint16_t* ds_in;
  uint16_t* ds;
  float* part;           // [gridDim.x, K] column sums of the block's rows, or null
  int64_t M, K;
};

// One thread's share of a row: dy, the stream (raw, or codes in x, y and the
// scale's bits in z) and ds_in.
template <int NU>
struct BwdRow {
  uint4 d[NU], s[NU], di[NU];
  float rs;
};

template <bool CK, int NT, int NU>
__device__ __forceinline__ void load_row(const NormBwdArgs& a, int64_t row, uint32_t nq, int64_t ng,
                                         BwdRow<NU>& r) {
  const int64_t base = row * a.K;
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const uint32_t c = threadIdx.x + NT * i;
    const bool ok = c < nq;
    r.d[i] = ldz(reinterpret_cast<const uint4*>(a.dy + base), c, ok);
    if constexpr (CK) {
      const uint2 q = ldz(reinterpret_cast<const uint2*>(a.sq + base), c, ok);
      const float sc = a.ss[row * ng + (ok ? c / 8 : 0u)];
      r.s[i] = make_uint4(q.x, q.y, __float_as_uint(sc), 0);
    } else {
      r.s[i] = ldz(reinterpret_cast<const uint4*>(a.s + base), c, ok);
    }
    r.di[i] = make_uint4(0, 0, 0, 0);
    if (a.ds_in) r.di[i] = ldz(reinterpret_cast<const uint4*>(a.ds_in + base), c, ok);
  }
  r.rs = a.rstd[row];
}

// Rows blockIdx.x, + gridDim.x, ...: ds of each, and the rows' share of dw
// in registers (NU * 8 columns per thread).  The next row is on its way
// while one is reduced and written (up to 512 threads: both fit the
// registers).  K % 8 == 0, K <= 8 NT NU.  ds may be ds_in or dy: a row's elements are read
// by the thread that writes them, before it does.
template <bool BF, bool CK, int NT, int NU>
__global__ void __launch_bounds__(NT) k_norm_bwd(NormBwdArgs a) {
  __shared__ double red_s[NT / 64];
  const uint32_t nq = (uint32_t)(a.K / 8);
  const int64_t ng = (a.K + 63) / 64;
  const uint32_t one = BF ? 0x3F803F80u : 0x3C003C00u;
  uint4 w[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const uint32_t c = threadIdx.x + NT * i;
    w[i] = make_uint4(one, one, one, one);
    if (a.w) w[i] = ldz(reinterpret_cast<const uint4*>(a.w), c, c < nq);
  }
  float dw[NU][8];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  constexpr bool AHEAD = NT <= 512;
  BwdRow<NU> r, nx;
  if (AHEAD) load_row<CK, NT, NU>(a, blockIdx.x, nq, ng, nx);
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    if constexpr (AHEAD) {
      r = nx;
      if (row + gridDim.x < a.M) load_row<CK, NT, NU>(a, row + gridDim.x, nq, ng, nx);
    } else {
      load_row<CK, NT, NU>(a, row, nq, ng, r);
    }
    auto stream = [&](int i, float (&v)[8]) __attribute__((always_inline)) {   // xh
      if constexpr (CK) {
        unpack8i(make_uint2(r.s[i].x, r.s[i].y), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * __uint_as_float(r.s[i].z) * r.rs;
      } else {
        unpack8<BF>(r.s[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= r.rs;
      }
    };
    double dot = 0.;
    float none = 0.f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float v[8], g[8], b[8];
      stream(i, v);
      unpack8<BF>(r.d[i], g);
      unpack8<BF>(w[i], b);
      float part = 0.f;   // 8 products in fp32, then fp64
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        part = fmaf(g[e] * b[e], v[e], part);
        dw[i][e] = fmaf(g[e], v[e], dw[i][e]);
      }
      dot += part;
    }
    if (!a.ds) continue;   // uniform
    row_reduce<NT, false>(dot, none, red_s, nullptr);
    const float c1 = (float)(dot / (double)a.K);
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t c = threadIdx.x + NT * i;
      float v[8], g[8], b[8], z[8];
      stream(i, v);
      unpack8<BF>(r.d[i], g);
      unpack8<BF>(w[i], b);
      unpack8<BF>(r.di[i], z);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = fmaf(r.rs, fmaf(-v[e], c1, g[e] * b[e]), z[e]);
      if (c < nq) reinterpret_cast<uint4*>(a.ds + row * a.K)[c] = pack8<BF>(z);
    }
  }
  if (a.part) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      const uint32_t c = threadIdx.x + NT * i;
      if (c < nq) {
        float4* p = reinterpret_cast<float4*>(a.part + (int64_t)blockIdx.x * a.K) + 2 * c;
        p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
        p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
      }
    }
  }
}

template <bool BF, bool CK>
__device__ __forceinline__ float stream_at(const NormBwdArgs& a, int64_t row, int64_t k) {
  if constexpr (CK)
    return (float)a.sq[row * a.K + k] * a.ss[row * ((a.K + 63) / 64) + k / 64];
  else
    return val16<BF>(a.s[row * a.K + k]);
}

// Any K: ds of one row per block, scalar columns.
template <bool BF, bool CK>
__global__ void __launch_bounds__(kAny) k_norm_bwd_any(NormBwdArgs a) {
  __shared__ double red_s[kAny / 64];
  const int64_t row = blockIdx.x, base = row * a.K;
  const float rs = a.rstd[row];
  auto weight = [&](int64_t k) { return a.w ? val16<BF>(a.w[k]) : 1.f; };
  double dot = 0.;
  float none = 0.f;
#pragma unroll 4
  for (int64_t k = threadIdx.x; k < a.K; k += kAny)
    dot += (double)(val16<BF>(a.dy[base + k]) * weight(k) * (stream_at<BF, CK>(a, row, k) * rs));
  row_reduce<kAny, false>(dot, none, red_s, nullptr);
  const float c1 = (float)(dot / (double)a.K);
#pragma unroll 4
  for (int64_t k = threadIdx.x; k < a.K; k += kAny) {
    const float z = a.ds_in ? val16<BF>(a.ds_in[base + k]) : 0.f;
    const float g = val16<BF>(a.dy[base + k]) * weight(k);
    a.ds[base + k] =
        (uint16_t)rnd16<BF>(fmaf(rs, fmaf(-stream_at<BF, CK>(a, row, k) * rs, c1, g), z));
  }
}

// Any K: column sums of dy xh over rows blockIdx.y, + gridDim.y, ...
template <bool BF, bool CK>
__global__ void __launch_bounds__(256) k_norm_dw_any(NormBwdArgs a) {
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (k >= a.K) return;
  float v = 0.f;
  for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y)
    v = fmaf(val16<BF>(a.dy[row * a.K + k]), stream_at<BF, CK>(a, row, k) * a.rstd[row], v);
  a.part[(int64_t)blockIdx.y * a.K + k] = v;
}

// dw[k] = sum of the P partial rows, in fp64 and a fixed order: 32 columns
// per block, 32 half waves taking every 32nd row.
__global__ void __launch_bounds__(1024) k_col_sum(const float* __restrict__ part, int P, int64_t K,
                                                  float* __restrict__ out) {
  __shared__ double red[32][33];
  const int c = threadIdx.x & 31, h = threadIdx.x >> 5;
  const int64_t k = (int64_t)blockIdx.x * 32 + c;
  double v = 0.;
  if (k < K) {
#pragma unroll 8
    for (int p = h; p < P; p += 32) v += (double)part[(int64_t)p * K + k];
  }
  red[h][c] = v;
  __syncthreads();
  if (h == 0 && k < K) {
#pragma unroll
    for (int i = 1; i < 32; ++i) v += red[i][c];
    out[k] = (float)v;
  }
}

// fl32(m / 127): the product with the reciprocal and one correction step,
// correctly rounded away from the subnormals and the infinity.
__device__ __forceinline__ float scale127(float m) {
  if (!(m >= 1e-30f && m < __builtin_inff())) return plain_nan(m / 127.f);
  constexpr float r = 1.f / 127.f;
  const float q = m * r;
  return fmaf(fmaf(-q, 127.f, m), r, q);
}

// Codes of a lane's values under a scale, as bytes: rint of the exact
// quotient.  fma(v, 1 / scale, 1.5 2^23) rounds the product to an integer in
// its low bits; the product is within 4e-5 of the quotient (127 steps, 2^-23
// from the reciprocal and 2^-24 more), so only a value whose product is that
// near to a tie needs the fp64 quotient (about one wave in ten has one): with
// one correction step that is exact at a tie, which then goes to even.  Scales
// that are not finite have 0 for the reciprocal; a NaN's low byte is 0 too.
template <int N>
__device__ __forceinline__ void ckpt_codes(const float (&v)[N], float sc, uint32_t (&c)[N]) {
  constexpr float magic = 12582912.f;
  const float inv = sc > 0.f ? __builtin_amdgcn_rcpf(sc) : 0.f;
  float off = inv > 1e38f ? 1.f : 0.f;   // an infinite or subnormal reciprocal: fp64 too
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float t = fmaf(v[e], inv, magic);
    off = fmaxf(off, fabsf(fmaf(v[e], inv, magic - t)));
    c[e] = __float_as_uint(t);
  }
  if (off > 0.4999f) {
    const double ds = sc, di = 1. / ds;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      double q = (double)v[e] * di;
      q = fma(fma(-q, ds, (double)v[e]), di, q);
      c[e] = (uint32_t)(int)fmin(fmax(rint(q), -127.), 127.);
    }
  }
}
// Low bytes of four words.
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u),
                               __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
}

// 8 lanes per group of 64 columns, 8 columns per lane (K % 8 == 0), NI groups
// per lane, 32 apart, all loads first; rows of ng groups, the last one
// possibly short.
template <bool BF, int NI>
__global__ void __launch_bounds__(256) k_ckpt(const uint16_t* __restrict__ x, int8_t* __restrict__ q,
                                              float* __restrict__ s, uint32_t ng, uint32_t nq,
                                              uint32_t groups) {
  const uint32_t g0 = blockIdx.x * (32u * NI) + threadIdx.x / 8u, l = threadIdx.x & 7u;
  uint4 u[NI];
  uint64_t at[NI];   // chunk of 8 columns
  bool ok[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t grp = g0 + 32u * i;
    at[i] = (uint64_t)grp * 8u + l;
    ok[i] = grp < groups;
    if (nq != 8u * ng) {   // rows of whole groups need no division
      const uint32_t row = grp / ng, c = (grp - row * ng) * 8u + l;
      at[i] = (uint64_t)row * nq + c;
      ok[i] = ok[i] && c < nq;
    }
    const uint4 v = reinterpret_cast<const uint4*>(x)[ok[i] ? at[i] : 0u];   // unconditional
    u[i] = make_uint4(ok[i] ? v.x : 0u, ok[i] ? v.y : 0u, ok[i] ? v.z : 0u, ok[i] ? v.w : 0u);
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float v[8], mx = 0.f;
    unpack8<BF>(u[i], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = max_nan(mx, fabsf(v[e]));
    mx = max_nan(mx, dpp_f<QP_DPP_QUAD_1032>(0.f, mx));
    mx = max_nan(mx, dpp_f<QP_DPP_QUAD_2301>(0.f, mx));
    mx = max_nan(mx, dpp_f<QP_DPP_ROW_HALF_MIRROR>(0.f, mx));   // 8 lanes: the other four
    const float sc = scale127(mx);
    uint32_t cq[8];
    ckpt_codes<8>(v, sc, cq);
    if (ok[i])
      reinterpret_cast<uint2*>(q)[at[i]] =
          make_uint2(bytes4(cq[0], cq[1], cq[2], cq[3]), bytes4(cq[4], cq[5], cq[6], cq[7]));
    if (l == 0 && g0 + 32u * i < groups) s[g0 + 32u * i] = sc;
  }
}

// Any K: one wave per group, one column per lane.
template <bool BF>
__global__ void __launch_bounds__(256) k_ckpt_any(const uint16_t* __restrict__ x,
                                                  int8_t* __restrict__ q, float* __restrict__ s,
                                                  uint32_t ng, int64_t K, uint32_t groups) {
  const uint32_t grp = blockIdx.x * 4u + (threadIdx.x >> 6);
  if (grp >= groups) return;   // whole waves
  const uint32_t lane = threadIdx.x & 63;
  const int64_t row = grp / ng;
  const int64_t k = (int64_t)(grp - (uint32_t)row * ng) * 64 + lane;
  const float v[1] = {k < K ? val16<BF>(x[row * K + k]) : 0.f};
  const float sc = scale127(wave_max_nan(fabsf(v[0])));
  uint32_t c[1];
  ckpt_codes<1>(v, sc, c);
  if (k < K) q[row * K + k] = (int8_t)c[0];
  if (lane == 0) s[grp] = sc;
}

template <int DT>
__device__ __forceinline__ void put(void* x, uint64_t i, float v) {
  if constexpr (DT == F32) static_cast<float*>(x)[i] = v;
  else static_cast<uint16_t*>(x)[i] = (uint16_t)rnd16<DT == BF16>(v);
}

// Codes back to values; V = 8 columns per thread (K % 8 == 0) or 1.
template <int DT, int V>
__global__ void __launch_bounds__(256) k_ckpt_restore(const int8_t* __restrict__ q,
                                                      const float* __restrict__ s, uint32_t ng,
                                                      uint32_t nq, uint32_t n,
                                                      void* __restrict__ x) {
  const uint32_t at = blockIdx.x * 256u + threadIdx.x;
  if (at >= n) return;
  uint32_t gi = at / (64u / V);   // rows of whole groups need no division
  if (nq != (64u / V) * ng) {
    const uint32_t row = at / nq;
    gi = row * ng + (at - row * nq) / (64u / V);
  }
  const float sc = s[gi];
  if constexpr (V == 1) {
    put<DT>(x, at, (float)q[at] * sc);
  } else {
    float v[8];
    unpack8i(reinterpret_cast<const uint2*>(q)[at], v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= sc;
    if constexpr (DT == F32) {
      float4* o = static_cast<float4*>(x) + 2 * at;
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      static_cast<uint4*>(x)[at] = pack8<DT == BF16>(v);
    }
  }
}

typedef void (*NormFn)(NormArgs);
typedef void (*NormBwdFn)(NormBwdArgs);

template <bool BF>
NormFn norm_pick(int tpr, int nu) {
  if (tpr == 64) return nu <= 1 ? k_norm<BF, 64, 1> : nu <= 2 ? k_norm<BF, 64, 2> : k_norm<BF, 64, 4>;
  if (tpr == 256) return nu <= 1 ? k_norm<BF, 256, 1> : nu <= 2 ? k_norm<BF, 256, 2> : k_norm<BF, 256, 4>;
  return nu <= 1 ? k_norm<BF, 1024, 1> : nu <= 2 ? k_norm<BF, 1024, 2> : k_norm<BF, 1024, 4>;
}

template <bool BF, bool CK>
NormBwdFn norm_bwd_pick(int64_t nq) {
  if (nq <= 256) return k_norm_bwd<BF, CK, 256, 1>;
  if (nq <= 512) return k_norm_bwd<BF, CK, 256, 2>;
  if (nq <= 1024) return k_norm_bwd<BF, CK, 512, 2>;
  return k_norm_bwd<BF, CK, 1024, 2>;
}
int norm_bwd_threads(int64_t nq) { return nq <= 512 ? 256 : nq <= 1024 ? 512 : 1024; }

}  // namespace

hipError_t launch_norm(const void* x, const void* r, int dt, int64_t M, int64_t K, const void* w,
                       float eps, void* s, void* y, void* yq, float* ys, float* rstd,
                       hipStream_t st) {
  NormArgs a{static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(r),
             static_cast<const uint16_t*>(w), static_cast<uint16_t*>(s),
             static_cast<uint16_t*>(y), static_cast<int8_t*>(yq), ys, rstd, M, K, eps};
  const int64_t nq = K / 8;
  if (K % 8 || nq > 4096) {
    auto fn = dt == BF16 ? k_norm_any<true> : k_norm_any<false>;
    hipLaunchKernelGGL(fn, dim3((unsigned)M), dim3(kAny), 0, st, a);
    return hipGetLastError();
  }
  int tpr = nq <= 64 ? 64 : nq <= 1024 ? 256 : 1024;
  const int nu = (int)((nq + tpr - 1) / tpr);
  const int rows = tpr == 64 ? 4 : 1;
  auto fn = dt == BF16 ? norm_pick<true>(tpr, nu) : norm_pick<false>(tpr, nu);
  hipLaunchKernelGGL(fn, dim3((unsigned)((M + rows - 1) / rows)), dim3(tpr < 256 ? 256 : tpr), 0,
                     st, a);
  return hipGetLastError();
}

int norm_bwd_parts(int64_t M) { return (int)(M < 512 ? M : 512); }

hipError_t launch_norm_bwd(const void* dy, const void* s, const void* sq, const float* ss, int dt,
                           int64_t M, int64_t K, const void* w, const float* rstd,
                           const void* ds_in, void* ds, float* dw, float* part, hipStream_t st) {
  NormBwdArgs a{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(s),
                static_cast<const int8_t*>(sq), ss, static_cast<const uint16_t*>(w), rstd,
                static_cast<const uint16_t*>(ds_in), static_cast<uint16_t*>(ds),
                dw ? part : nullptr, M, K};
  const bool bf = dt == BF16, ck = sq != nullptr;
  const int64_t nq = K / 8;
  const unsigned P = (unsigned)norm_bwd_parts(M);
  hipError_t e;
  if (K % 8 || nq > 2048) {
    // dw first: ds may be dy itself
    if (dw) {
      auto fn = bf ? (ck ? k_norm_dw_any<true, true> : k_norm_dw_any<true, false>)
                   : (ck ? k_norm_dw_any<false, true> : k_norm_dw_any<false, false>);
      hipLaunchKernelGGL(fn, dim3((unsigned)((K + 255) / 256), P), dim3(256), 0, st, a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (ds) {
      auto fn = bf ? (ck ? k_norm_bwd_any<true, true> : k_norm_bwd_any<true, false>)
                   : (ck ? k_norm_bwd_any<false, true> : k_norm_bwd_any<false, false>);
      hipLaunchKernelGGL(fn, dim3((unsigned)M), dim3(kAny), 0, st, a);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
  } else {
    auto fn = bf ? (ck ? norm_bwd_pick<true, true>(nq) : norm_bwd_pick<true, false>(nq))
                 : (ck ? norm_bwd_pick<false, true>(nq) : norm_bwd_pick<false, false>(nq));
    hipLaunchKernelGGL(fn, dim3(P), dim3(norm_bwd_threads(nq)), 0, st, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (dw) {
    hipLaunchKernelGGL(k_col_sum, dim3((unsigned)((K + 31) / 32)), dim3(1024), 0, st, part, (int)P,
                       K, dw);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_checkpoint(const void* x, int dt, int64_t M, int64_t K, void* q, float* s,
                             hipStream_t st) {
  const uint32_t ng = (uint32_t)((K + 63) / 64);
  const uint32_t groups = (uint32_t)((uint64_t)M * ng);   // < 2^31 (host check)
  if (K % 8) {
    auto fn = dt == BF16 ? k_ckpt_any<true> : k_ckpt_any<false>;
    hipLaunchKernelGGL(fn, dim3((groups + 3u) / 4u), dim3(256), 0, st,
                       static_cast<const uint16_t*>(x), static_cast<int8_t*>(q), s, ng, K, groups);
  } else {
    // four groups per lane where that leaves every CU several blocks
    const bool many = groups >= 32u * 4u * 1024u;
    const uint32_t per = many ? 128u : 32u;
    auto fn = dt == BF16 ? (many ? k_ckpt<true, 4> : k_ckpt<true, 1>)
                         : (many ? k_ckpt<false, 4> : k_ckpt<false, 1>);
    hipLaunchKernelGGL(fn, dim3((groups + per - 1u) / per), dim3(256), 0, st,
                       static_cast<const uint16_t*>(x), static_cast<int8_t*>(q), s, ng,
                       (uint32_t)(K / 8), groups);
  }
  return hipGetLastError();
}

hipError_t launch_checkpoint_restore(const void* q, const float* s, int64_t M, int64_t K, void* x,
                                     int dt, hipStream_t st) {
  const uint32_t ng = (uint32_t)((K + 63) / 64);
  const bool v8 = K % 8 == 0;
  const uint32_t nq = (uint32_t)(v8 ? K / 8 : K);
  const uint32_t n = (uint32_t)((uint64_t)M * nq);   // <= 2^31 (host check)
  auto fn = v8 ? (dt == F32 ? k_ckpt_restore<F32, 8>
                  : dt == BF16 ? k_ckpt_restore<BF16, 8> : k_ckpt_restore<F16, 8>)
               : (dt == F32 ? k_ckpt_restore<F32, 1>
                  : dt == BF16 ? k_ckpt_restore<BF16, 1> : k_ckpt_restore<F16, 1>);
  hipLaunchKernelGGL(fn, dim3((n + 255u) / 256u), dim3(256), 0, st,
                     static_cast<const int8_t*>(q), s, ng, nq, n, x);
  return hipGetLastError();
}

}  // namespace qp
