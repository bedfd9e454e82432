// y [M, N] = X W^T for MXFP4 weights and 16-bit X of more than a few rows, on
// exact codes.
#include "device_common.hpp"
#include "qp_internal.hpp"

namespace qp {
namespace {

typedef int int4v_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

constexpr uint32_t kOff = 0x80000000u;   // at or past every resource: reads 0

struct RowsArgs {
  const unsigned char *x, *wq, *ws;
  const void* bias;
  void* y;
  int64_t M, N, K;
  int ydt, KW, tiles;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes,
                                           0x00020000);
}
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, unsigned char* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}
template <bool XB>
__device__ __forceinline__ f32x4_t mfma32(int4v_t a, int4v_t b) {
  const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
  if constexpr (XB)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b),
                                                   zero, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b),
                                                  zero, 0, 0, 0);
}
// The E2M1 values of a word's eight codes (exact).
template <bool XB, int SEL>
__device__ __forceinline__ int e2m1_pair(uint32_t w) {
  if constexpr (XB)
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.f, SEL));
  else
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.f, SEL));
}
template <bool XB>
__device__ __forceinline__ int4v_t e2m1_eight(uint32_t w) {
  return int4v_t{e2m1_pair<XB, 0>(w), e2m1_pair<XB, 1>(w), e2m1_pair<XB, 2>(w), e2m1_pair<XB, 3>(w)};
}
__device__ __forceinline__ float e8m0(uint32_t s) {
  const uint32_t b = s == 0 ? 0x00400000u : s << 23;
  return __uint_as_float(s == 255u ? 0x7FC00000u : b);
}

// v_mfma_f32_16x16x32 with X as A and the codes' values as B, one per 32
// columns: a lane's four outputs then belong to one weight row, so that the
// block's scale is one number of the lane and multiplies the product in fp32
// (in the operand it would leave fp16's range):
//     acc += 2^(s - 127) (x . e2m1).
// A wave takes 16 G rows of W and 16 T rows of X, 128 columns per step.
//  * Codes: a lane loads 16 bytes, block l / 16 of the step in row l % 16.  The
//    product wants 8 codes of one block from each of the four lane groups: a
//    4 x 4 transposition of dwords over the groups, four permlane swaps.
//  * X: 4 T KiB per step through the wave's own part of LDS, 256 bytes of four
//    rows per instruction; piece p of row t lies at p ^ (t % 16), so that 16 lanes
//    of one piece touch every bank once.  NS steps of it, so that two blocks fit a CU.
//  * A sum right behind its product would wait for it (64 x 8192 x 8192 43 us): the
//    products of 32 columns come with the sums of the 32 before.
//  * G = 2 halves the traffic of X, which from L2 is the larger part (32 T bytes
//    per column against 8 G of codes); G = 1 where that leaves too few waves.
//  * KW waves share rows and add up through LDS at the end.  Scale bytes of the
//    block's rows are copied to LDS first.
// 13 x 8192 x 8192: 16.2 us, 2.2 TB/s of codes: 256 blocks of four waves with four
// steps each way from L2 in front; 64 x 4096 x 14336 23 us, 326 TFLOP/s.
template <bool XB, int G, int T, int NS>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) k_mx_rows(RowsArgs a) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ __attribute__((aligned(16))) unsigned char xstep[4 * NS * 4096 * T];   // an object of its own: see load_x
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = wave % a.KW, team = wave / a.KW;
  const uint32_t r = lane & 15, g4 = lane >> 4;
  const uint32_t C = (uint32_t)(a.K / 32), rowb = (uint32_t)(a.K / 2), xrowb = (uint32_t)(a.K * 2);
  const int S = (int)((C + 3) / 4), rows = (4 / a.KW) * 16 * G;
  const int64_t n0 = (int64_t)(blockIdx.x % (unsigned)a.tiles) * rows;
  const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)a.tiles) * (16 * T);
  const uint32_t nrows = (uint32_t)(a.N - n0 < rows ? a.N - n0 : rows);
  const uint32_t mrows = (uint32_t)(a.M - m0 < 16 * T ? a.M - m0 : 16 * T);
  const __amdgpu_buffer_rsrc_t rw = rsrc_of(a.wq + n0 * rowb, (uint64_t)nrows * rowb);
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(a.x + m0 * xrowb, (uint64_t)mrows * xrowb);
  uint32_t wsc;
  {
    const uint64_t from = (uint64_t)n0 * C, lo = from & ~uint64_t(15);
    const uint32_t head = (uint32_t)(from - lo), bytes = (head + nrows * C + 15u) & ~15u;   // whole 16-byte units
    const __amdgpu_buffer_rsrc_t rs = rsrc_of(a.ws + lo, bytes);
    for (uint32_t ch = (uint32_t)wave; ch * 1024u < bytes; ch += 4)
      to_lds(rs, smem + ch * 1024u, ch * 1024u + 16u * (uint32_t)lane);
    wsc = head + ((uint32_t)team * 16u * G + r) * C;
  }

  struct Step {
    int4v_t w[G];
  };
  const uint32_t wat = ((uint32_t)team * 16u * G + r) * rowb + 16u * g4;
  // In this order and issued past the last step too (reading nothing), so that
  // the wait for one step's operands is not one for the next's.
  auto load = [&](int s, Step& st) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    const uint32_t at = (uint32_t)s * 4u + g4 < C ? wat + (uint32_t)s * 64u : kOff;
#pragma unroll
    for (int g = 0; g < G; ++g)
      st.w[g] = __builtin_bit_cast(int4v_t, __builtin_amdgcn_raw_buffer_load_b128(rw, at + 16u * g * rowb, 0, 0));
    __builtin_amdgcn_sched_barrier(0);
  };
  // Step s of X into LDS.  The compiler does not wait for these copies: compute
  // does, by count.  Rows past the last are copied too (as zeros): a branch here
  // would let the products sink behind the next step's wait.
  unsigned char* xl = xstep + wave * (NS * 4096 * T);
  auto load_x = [&](int s, int stage) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < 4 * T; ++q) {
      const uint32_t row = 4u * q + g4, piece = r ^ (row & 15u);
      to_lds(rx, xl + 4096 * T * stage + 1024 * q,
             (uint32_t)s * 4u + piece / 4u < C ? row * xrowb + (uint32_t)s * 256u + 16u * piece : kOff);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4_t acc[G][T];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[g][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  constexpr int kStep = 4 * T + G;    // loads of a step
  constexpr int NW = NS > 1 ? NS : 2;   // steps of codes in registers
  constexpr int kAll = NS * kStep + (NW - NS) * G;
  static_assert(kAll < 64, "a wait counts to 63");
  auto compute = [&](int s, int stage, int next, const Step& st) __attribute__((always_inline)) {
    constexpr int w = (NS - 1) * kStep + (NW - NS) * G;   // all but the later steps' operands
    __builtin_amdgcn_s_waitcnt((w & 0xF) | (0x7 << 4) | (0xF << 8) | ((w >> 4) << 14));
    __builtin_amdgcn_sched_barrier(0);
    int4v_t x[T][4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int t = 0; t < T; ++t)
        x[t][c] = *reinterpret_cast<const int4v_t*>(xl + 4096 * T * stage + (16u * t + r) * 256u + 16u * ((4u * c + g4) ^ r));
    __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
    load_x(next, stage);
    // the products of one block of columns and the sums of the one before, by
    // turns: a sum right behind its product would wait for it
    f32x4_t v[2][T];
    float sc[2];
    uint32_t code[4];
#pragma unroll
    for (int b = 0; b <= 4 * G; ++b) {
      if (b < 4 * G) {
        const int g = b / 4, k = b % 4;
        if (k == 0) {
          const int4v_t d = st.w[g];
          const auto p = __builtin_amdgcn_permlane32_swap((uint32_t)d[0], (uint32_t)d[2], false, false);
          const auto u = __builtin_amdgcn_permlane32_swap((uint32_t)d[1], (uint32_t)d[3], false, false);
          const auto lo = __builtin_amdgcn_permlane16_swap(p[0], u[0], false, false);
          const auto hi = __builtin_amdgcn_permlane16_swap(p[1], u[1], false, false);
          code[0] = lo[0];
          code[1] = lo[1];
          code[2] = hi[0];
          code[3] = hi[1];
        }
        uint32_t c = (uint32_t)s * 4u + k;   // uniform
        c = c < C ? c : C - 1u;              // codes of 0, with a scale of the same row
        sc[b & 1] = e8m0(smem[wsc + 16u * g * C + c]);
        const int4v_t w8 = e2m1_eight<XB>(code[k]);
#pragma unroll
        for (int t = 0; t < T; ++t) v[b & 1][t] = mfma32<XB>(x[t][k], w8);
      }
      __builtin_amdgcn_sched_barrier(0x7FF & ~0x8);   // products stay on their side
      if (b > 0)
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[(b - 1) / 4][t][j] = fmaf(sc[(b - 1) & 1], v[(b - 1) & 1][t][j], acc[(b - 1) / 4][t][j]);
    }
  };

  // the wave's steps; KW <= S, so there is one
  const int n = (S - kw + a.KW - 1) / a.KW;
  Step st[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    if (i < NS) load_x(kw + i * a.KW, i);
    load(kw + i * a.KW, st[i]);
  }
  // the scales' copies were issued before these loads
  __builtin_amdgcn_s_waitcnt((kAll & 0xF) | (0x7 << 4) | (0xF << 8) | ((kAll >> 4) << 14));
  __syncthreads();
  // NW by NW; past the last step the codes are 0
  for (int i = 0; i < n; i += NW) {
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const int s = kw + (i + k) * a.KW;
      compute(s, k % NS, s + NS * a.KW, st[k]);
      load(s + NW * a.KW, st[k]);
    }
  }

  // Lane l holds row l % 16 of W and rows 4 (l / 16) .. + 3 of X.
  auto put = [&](int g, int t, f32x4_t v) __attribute__((always_inline)) {
    const int64_t nn = n0 + team * 16 * G + 16 * g + r;
    if (nn >= a.N) return;
    float b = 0.f;
    if (a.bias) b = meta_to_f32(static_cast<const uint16_t*>(a.bias)[nn], XB);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t m = m0 + 16 * t + 4 * (int64_t)g4 + i;
      if (m >= a.M) continue;
      const float o = v[i] + b;
      if (a.ydt == F32) static_cast<float*>(a.y)[m * a.N + nn] = o;
      else if (a.ydt == BF16) static_cast<uint16_t*>(a.y)[m * a.N + nn] = (uint16_t)f32_to_bf16_rne(o);
      else static_cast<uint16_t*>(a.y)[m * a.N + nn] = (uint16_t)f32_to_f16_rne(o);
    }
  };
  if (a.KW == 1) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int t = 0; t < T; ++t) put(g, t, acc[g][t]);
    return;
  }
  // Every copy into LDS has to be there before the sums take its place: the
  // last steps' copies of X (zeros) are still on their way.
  __builtin_amdgcn_s_waitcnt(0x0F70 & ~(0x3 << 14));   // vmcnt(0)
  __syncthreads();
  f32x4_t* red = reinterpret_cast<f32x4_t*>(xstep);
#pragma unroll
  for (int p = 0; p < G * T; ++p) red[(wave * G * T + p) * 64 + lane] = acc[p / T][p % T];
  __syncthreads();
  for (int p = kw; p < G * T; p += a.KW) {
    f32x4_t v = red[(team * a.KW * G * T + p) * 64 + lane];
    for (int w = 1; w < a.KW; ++w) v += red[((team * a.KW + w) * G * T + p) * 64 + lane];
    put(p / T, p % T, v);
  }
}

size_t scale_lds(int64_t rows, int64_t C) { return ((size_t)rows * C + 15 + 1023) / 1024 * 1024; }
int row_groups(int64_t M) { return M <= 16 ? 1 : M <= 32 ? 2 : 4; }   // T

}  // namespace

// The scales of one wave's rows have to fit LDS next to the steps of X.
bool mx_rows_fits(const Desc& d) { return scale_lds(32, d.K / 32) <= 92 * 1024; }

namespace {
using RowsFn = void (*)(RowsArgs);
template <bool XB, int G>
RowsFn rows_fn(int T) {
  return T == 1 ? k_mx_rows<XB, G, 1, 4> : T == 2 ? k_mx_rows<XB, G, 2, 2> : k_mx_rows<XB, G, 4, 1>;
}
}  // namespace

hipError_t launch_mx_rows(const Desc& d, const void* x, int xdt, int64_t M, const Bufs& b,
                          const void* bias, void* y, int ydt, hipStream_t s) {
  const int T = row_groups(M);
  const int64_t C = d.K / 32, S = (C + 3) / 4, mt = (M + 16 * T - 1) / (16 * T);
  // Waves fill the chip from 1024 on.  G = 2 and 1 where four waves per row are
  // fewer: 16 x 14336 x 4096 20 and 15 us, 64 x 4096 x 4096 15 and 12; where they are not: 32 x
  // 8192 x 8192 17 and 19, 64 x 5120 x 25600 44 and 60.
  const int G = mt * ((d.N + 31) / 32) * 4 < 1024 ? 1 : 2;
  // waves per row: as few as fill the chip, and as many as the scales' LDS asks for
  int KW = 1;
  while (KW < 4 && 2 * KW <= S && (mt * ((d.N + 16 * G - 1) / (16 * G)) * KW < 1024 ||
                                   scale_lds(4 / KW * 16 * G, C) > 15 * 1024))
    KW *= 2;
  const int rows = 4 / KW * 16 * G;
  RowsArgs a{static_cast<const unsigned char*>(x), static_cast<const unsigned char*>(b.qweight),
             static_cast<const unsigned char*>(b.scales), bias, y, M, d.N, d.K, ydt, KW,
             (int)((d.N + rows - 1) / rows)};
  const RowsFn fn = xdt == BF16 ? (G == 1 ? rows_fn<true, 1>(T) : rows_fn<true, 2>(T))
                                : (G == 1 ? rows_fn<false, 1>(T) : rows_fn<false, 2>(T));
  hipLaunchKernelGGL(fn, dim3((unsigned)(a.tiles * mt)), dim3(256), scale_lds(rows, C), s, a);
  return hipGetLastError();
}

}  // namespace qp
