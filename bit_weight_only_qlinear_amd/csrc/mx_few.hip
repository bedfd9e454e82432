// y [M, N] = X W^T, both MXFP4, for few rows of X.
#include "device_common.hpp"
#include "qp_internal.hpp"

namespace qp {
namespace {

typedef int int4v_t __attribute__((ext_vector_type(4)));
typedef int int8v_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr uint32_t kOff = 0x80000000u;   // at or past every resource: reads 0

struct MxFewArgs {
  const unsigned char *xq, *xs, *wq, *ws;
  const float* bias;
  void* y;
  int64_t M, N, K;
  int ydt, KW, tiles;
  uint32_t x_lds;          // where the scales of x lie in LDS, past those of the weights
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes,
                                           0x00020000);
}
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, unsigned char* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}

// Bound by the codes of W (K/2 bytes a row).  v_mfma_scale_f32_16x16x128_f8f6f4
// takes a lane's 16 bytes as 32 columns of row l % 16 with one scale byte, which
// is the format's own block: codes go from memory into the operands without a
// shuffle, a conversion or LDS.  A step is 512 columns: load i of a row takes
// chunks 4 i + l / 16, 64 bytes of each of 16 rows, and the four loads together
// whole lines.  A wave works on 16 kG rows of W, loaded two steps ahead, and 16 T
// rows of X.  Those come from L2 through the wave's own part of LDS, 256
// bytes of four rows per instruction (as operands, 64 bytes of 16 rows, they
// took as long as the weights): piece p of row t lies at p ^ (t % 16), so that
// 16 lanes of one piece touch every bank once.  KW waves share rows and add up
// through LDS at the end.  The scale bytes of the block's rows, of W and of X,
// are copied to LDS first.  16 x 5120 x 25600: 19 us, 3.7 TB/s.
template <int kG, int T>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) k_mx_few(MxFewArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ __attribute__((aligned(16))) unsigned char xstep[4 * 4096 * T];   // an object of its own: see load_x
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = wave % a.KW, team = wave / a.KW;
  const uint32_t r = lane & 15, g4 = lane >> 4;
  const uint32_t C = (uint32_t)(a.K / 32), rowb = (uint32_t)(a.K / 2);
  const int S = (int)((C + 15) / 16), rows = (4 / a.KW) * 16 * kG;
  const int64_t n0 = (int64_t)(blockIdx.x % (unsigned)a.tiles) * rows;
  const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)a.tiles) * (16 * T);
  const uint32_t nrows = (uint32_t)(a.N - n0 < rows ? a.N - n0 : rows);
  const uint32_t mrows = (uint32_t)(a.M - m0 < 16 * T ? a.M - m0 : 16 * T);
  const __amdgpu_buffer_rsrc_t rw = rsrc_of(a.wq + n0 * rowb, (uint64_t)nrows * rowb);
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(a.xq + m0 * rowb, (uint64_t)mrows * rowb);

  // scale bytes, whole 16-byte units of memory
  auto scales = [&](const unsigned char* p, int64_t row0, uint32_t n, uint32_t at) __attribute__((always_inline)) {
    const uint64_t from = (uint64_t)row0 * C, lo = from & ~uint64_t(15);
    const uint32_t head = (uint32_t)(from - lo), bytes = (head + n * C + 15u) & ~15u;
    const __amdgpu_buffer_rsrc_t rs = rsrc_of(p + lo, bytes);
    for (uint32_t ch = (uint32_t)wave; ch * 1024u < bytes; ch += 4)
      to_lds(rs, smem + at + ch * 1024u, ch * 1024u + 16u * (uint32_t)lane);
    return at + head;
  };
  const uint32_t wsc = scales(a.ws, n0, nrows, 0) + ((uint32_t)team * 16u * kG + r) * C;
  const uint32_t xsc = scales(a.xs, m0, mrows, a.x_lds) + r * C;

  struct Step {
    int4v_t w[kG][4];
  };
  const uint32_t wat = ((uint32_t)team * 16u * kG + r) * rowb + 16u * g4;
  // In this order and issued past the last step too (reading nothing), so that
  // the wait for one step's operands is not one for the next's.
  auto load = [&](int s, Step& st) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = (uint32_t)s * 16u + 4u * i + g4;
      const bool in = c < C;
      const uint32_t at = (uint32_t)s * 256u + 64u * i;
#pragma unroll
      for (int g = 0; g < kG; ++g)
        st.w[g][i] = __builtin_bit_cast(int4v_t, __builtin_amdgcn_raw_buffer_load_b128(
                                                     rw, in ? wat + at + 16u * g * rowb : kOff, 0, 0));
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Step s of X into LDS.  The compiler does not wait for these copies: compute
  // does, by count.  Rows past the last are copied too (as zeros): a branch here
  // would let the products sink behind the next step's wait.
  unsigned char* xl = xstep + wave * 4096 * T;
  auto load_x = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4 * T; ++q) {
      const uint32_t row = 4u * q + g4, c = (uint32_t)s * 16u + (r ^ (row & 15u));
      to_lds(rx, xl + 1024 * q, c < C ? row * rowb + 16u * c : kOff);
    }
  };
  f32x4_t acc[kG][T];
#pragma unroll
  for (int g = 0; g < kG; ++g)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[g][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](int s, int next, const Step& st) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt((4 * kG) | (0x7 << 4) | (0xF << 8));   // all but the next step's codes of W
    __builtin_amdgcn_sched_barrier(0);
    int4v_t x[T][4];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[t][i] = *reinterpret_cast<const int4v_t*>(xl + 4096 * t + 256u * r + 16u * ((4u * i + g4) ^ r));
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
    __builtin_amdgcn_sched_barrier(0);
    load_x(next);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t c = (uint32_t)s * 16u + 4u * i + g4;
      c = c < C ? c : C - 1u;   // codes of 0, with a scale of the same row
      int sw[kG], sx[T];
#pragma unroll
      for (int g = 0; g < kG; ++g) sw[g] = smem[wsc + 16u * g * C + c];
#pragma unroll
      for (int t = 0; t < T; ++t) sx[t] = smem[xsc + 16u * t * C + c];
      auto wide = [](int4v_t v) { return int8v_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; };
#pragma unroll
      for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int t = 0; t < T; ++t)
          acc[g][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(st.w[g][i]), wide(x[t][i]), acc[g][t],
                                                                       4, 4, 0, sw[g], 0, sx[t]);
    }
  };

  // the wave's steps; KW <= S, so there is one
  const int n = (S - kw + a.KW - 1) / a.KW;
  Step s0, s1;
  load_x(kw);
  load(kw, s0);
  load(kw + a.KW, s1);
  {
    // the scales' copies were issued before these loads
    constexpr int w = 2 * 4 * kG;
    static_assert(w < 64, "a wait counts to 63");
    __builtin_amdgcn_s_waitcnt((w & 0xF) | (0x7 << 4) | (0xF << 8) | ((w >> 4) << 14));
    __syncthreads();
  }
  // two by two; past the last step the codes are 0
  for (int i = 0; i < n; i += 2) {
    const int s = kw + i * a.KW;
    compute(s, s + a.KW, s0);
    load(s + 2 * a.KW, s0);
    compute(s + a.KW, s + 2 * a.KW, s1);
    load(s + 3 * a.KW, s1);
  }

  // Lane l holds row 16 t + l % 16 of X and rows 4 (l / 16) .. + 3 of W.
  auto put = [&](int g, int t, f32x4_t v) __attribute__((always_inline)) {
    const int64_t m = m0 + 16 * t + r, nn = n0 + team * 16 * kG + 16 * g + 4 * (int64_t)g4;
    if (m >= a.M || nn >= a.N) return;
    const int cnt = a.N - nn < 4 ? (int)(a.N - nn) : 4;
    if (a.bias)
      for (int i = 0; i < cnt; ++i) v[i] += a.bias[nn + i];
    const int64_t at = m * a.N + nn;
    if (a.ydt == F32) {
      float* y = static_cast<float*>(a.y) + at;
      if (a.N % 4 == 0) *reinterpret_cast<f32x4_t*>(y) = v;
      else
        for (int i = 0; i < cnt; ++i) y[i] = v[i];
    } else {
      uint16_t* y = static_cast<uint16_t*>(a.y) + at;
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = a.ydt == BF16 ? f32_to_bf16_rne(v[i]) : f32_to_f16_rne(v[i]);
      if (a.N % 4 == 0) *reinterpret_cast<uint2*>(y) = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
      else
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < cnt) y[i] = (uint16_t)h[i];
    }
  };
  if (a.KW == 1) {
#pragma unroll
    for (int g = 0; g < kG; ++g)
#pragma unroll
      for (int t = 0; t < T; ++t) put(g, t, acc[g][t]);
    return;
  }
  __syncthreads();   // the scales have been read: their LDS takes the sums
  f32x4_t* red = reinterpret_cast<f32x4_t*>(smem);
#pragma unroll
  for (int p = 0; p < kG * T; ++p) red[(wave * kG * T + p) * 64 + lane] = acc[p / T][p % T];
  __syncthreads();
  for (int p = kw; p < kG * T; p += a.KW) {
    f32x4_t v = red[(team * a.KW * kG * T + p) * 64 + lane];
    for (int w = 1; w < a.KW; ++w) v += red[((team * a.KW + w) * kG * T + p) * 64 + lane];
    put(p / T, p % T, v);
  }
}

size_t scale_lds(int64_t rows, int64_t C) { return ((size_t)rows * C + 15 + 1023) / 1024 * 1024; }
int quads_of(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }   // T

}  // namespace

// The scales of 32 rows of W and of a tile of X have to fit LDS, next to the
// codes of a step of X.
bool mx_few_fits(const Desc& d, int64_t M) {
  const int64_t C = d.K / 32;
  const int T = quads_of(M);
  return scale_lds(32, C) + scale_lds(16 * T, C) + (size_t)T * 16 * 1024 <= 156 * 1024;
}

namespace {
using MxFewFn = void (*)(MxFewArgs);
template <int G>
MxFewFn mx_few_fn(int T) {
  return T == 1 ? k_mx_few<G, 1> : T == 2 ? k_mx_few<G, 2> : k_mx_few<G, 4>;
}
}  // namespace

hipError_t launch_mx_few(const Desc& d, const void* xq, const void* xs, int64_t M, const Bufs& b,
                         const float* bias, void* y, int ydt, hipStream_t s) {
  const int64_t C = d.K / 32, S = (C + 15) / 16;
  const int T = quads_of(M);
  const int64_t mt = (M + 16 * T - 1) / (16 * T);
  // Waves per row: as few as fill the chip (T = 4: LDS holds half as many), and as
  // many as the scales' LDS asks for.  25600 x 5120, four and two of them: 19.0 and
  // 19.5 us for 16 rows, 36.0 and 29.1 for 64.
  const int64_t fill = T == 4 ? 1024 : 2048;
  // Two groups of weight rows per wave, which halve the traffic of X; one where
  // four waves per row would still be fewer than 1024: 16 x 14336 x 4096 11.6 and 9.0 us,
  // 64 x 8192 x 1024 13.7 and 10.0.
  const int G = mt * ((d.N + 31) / 32) * 4 < 1024 ? 1 : 2;
  int KW = 1;
  while (KW < 4 && 2 * KW <= S && (mt * ((d.N + 16 * G - 1) / (16 * G)) * KW < fill ||
                                   scale_lds(4 / KW * 16 * G, C) > 32 * 1024))
    KW *= 2;
  const int rows = 4 / KW * 16 * G;
  const size_t wl = scale_lds(rows, C), xl = scale_lds(16 * T, C), red = KW > 1 ? (size_t)4 * G * T * 1024 : 0;
  MxFewArgs a{static_cast<const unsigned char*>(xq), static_cast<const unsigned char*>(xs),
              static_cast<const unsigned char*>(b.qweight), static_cast<const unsigned char*>(b.scales),
              bias, y, M, d.N, d.K, ydt, KW, (int)((d.N + rows - 1) / rows), (uint32_t)wl};
  hipLaunchKernelGGL(G == 1 ? mx_few_fn<1>(T) : mx_few_fn<2>(T), dim3((unsigned)(a.tiles * mt)), dim3(256), wl + xl > red ? wl + xl : red, s, a);
  return hipGetLastError();
}

}  // namespace qp
