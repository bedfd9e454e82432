// MXFP4 (the microscaling format of E2M1 codes with one E8M0 scale byte per 32
// columns): quantization, dequantization, and the product of two MXFP4
// operands on the scaled matrix cores.
#include <type_traits>

#include "device_common.hpp"
#include "qp_internal.hpp"

namespace qp {
namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef int int8v_t __attribute__((ext_vector_type(8)));
typedef float float16v_t __attribute__((ext_vector_type(16)));

constexpr uint32_t kOff = 0x80000000u;   // at or past every resource: reads 0

__device__ __forceinline__ float e8m0(uint32_t s) {
  const uint32_t b = s == 0u ? 0x00400000u : s << 23;
  return __uint_as_float(s == 255u ? 0x7FC00000u : b);
}

// ---------------------------------------------------------------- quantize
// Memory-bound: a thread takes 8 columns (16 or 32 bytes), four threads a
// block of 32.  With E the exponent field of the block's largest magnitude
// as fp32, floor(log2 max) = E - 127, so the scale byte is E - 2, 0 at least
// (a block of zeros and subnormals too), and 255 where E is 255 (a NaN or an
// infinity; codes of 0).  The codes come from the hardware's conversion,
// which divides by the scale, rounds to the nearest code (ties to even) and
// stops at 6; blocks whose scale is below 2^-64 are taken times 2^64 first
// (exact), so that neither the values nor the scale are subnormal.
// 2048 x 14336 bf16: 14.2 us, 5.2 TB/s (a copy's rate); back: 12.9.
template <int DT>
__global__ void __launch_bounds__(256) k_mx_quant(const void* __restrict__ x, uint32_t* __restrict__ q,
                                                  uint8_t* __restrict__ s, int64_t n8) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n8; t += stride) {
    float v[8];
    if constexpr (DT == F32) {
      const float4 a = static_cast<const float4*>(x)[2 * t], b = static_cast<const float4*>(x)[2 * t + 1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
      const uint4 u = static_cast<const uint4*>(x)[t];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = DT == BF16 ? bf16_to_f32(w[i] & 0xFFFFu) : f16_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = DT == BF16 ? __uint_as_float(w[i] & 0xFFFF0000u) : f16_to_f32(w[i] >> 16);
      }
    }
    // magnitudes compare as their bits (a NaN is larger than all numbers)
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    // n8 and the stride are multiples of 4: a block's threads run together
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, QP_DPP_QUAD_1032, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, QP_DPP_QUAD_2301, 0xF, 0xF, false));
    const uint32_t E = m >> 23, sc = E == 255u ? 255u : E > 2u ? E - 2u : 0u;
    const bool tiny = sc < 64u;
    const float up = tiny ? 0x1p64f : 1.f;
    const float scale = __uint_as_float((tiny ? sc + 64u : sc) << 23);   // 2^(sc - 127) up
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * up, v[1] * up, scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * up, v[3] * up, scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * up, v[5] * up, scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * up, v[7] * up, scale, 3);
    q[t] = sc == 255u ? 0u : w;
    if ((threadIdx.x & 3) == 0) s[t >> 2] = (uint8_t)sc;
  }
}

// ---------------------------------------------------------------- dequantize
// One thread per word; value times scale in fp32 (exact, subnormals kept).
template <int DT>
__global__ void __launch_bounds__(256) k_mx_dequant(const uint32_t* __restrict__ q,
                                                    const uint8_t* __restrict__ s, void* __restrict__ out,
                                                    int64_t n8) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x; t < n8; t += stride) {
    const uint32_t w = q[t];
    const float sc = e8m0(s[t >> 2]);
    const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0);
    const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1);
    const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2);
    const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
    const float v[8] = {a.x * sc, a.y * sc, b.x * sc, b.y * sc, c.x * sc, c.y * sc, d.x * sc, d.y * sc};
    if constexpr (DT == F32) {
      static_cast<float4*>(out)[2 * t] = make_float4(v[0], v[1], v[2], v[3]);
      static_cast<float4*>(out)[2 * t + 1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = DT == BF16 ? f32_to_bf16_rne(v[2 * i]) : f32_to_f16_rne(v[2 * i]);
        const uint32_t hi = DT == BF16 ? f32_to_bf16_rne(v[2 * i + 1]) : f32_to_f16_rne(v[2 * i + 1]);
        p[i] = lo | (hi << 16);
      }
      static_cast<uint4*>(out)[t] = make_uint4(p[0], p[1], p[2], p[3]);
    }
  }
}

unsigned mx_blocks(int64_t n8) {
  const int64_t b = (n8 + 255) / 256;
  return (unsigned)(b < (int64_t(1) << 20) ? b : int64_t(1) << 20);
}

// ---------------------------------------------------------------- product
// y [M, N] = X W^T, both MXFP4, on v_mfma_scale_f32_32x32x64_f8f6f4, which
// multiplies 4-bit codes of 64 columns and applies one scale byte per row and
// 32 columns by itself.  A lane's operand is 32 codes of one row (lane % 32;
// lane / 32 chooses the half), i.e. the 16 bytes as they lie in memory, so
// codes go from HBM to LDS by direct loads and from there to the matrix
// cores untouched; fp32 sums.
//  * Block: 256 weight rows x 64 MW activation rows, 128 columns (64 bytes of
//    codes) a step, 8 waves of 32 MW x 64 outputs.
//  * LDS: four stages, three of them in flight: a step of matrix instructions
//    is shorter than the way from L2 (two stages of 256 columns: 130 us on
//    2048 x 4096 x 14336, waiting most of the time).  Loads return in order, so
//    waiting until two steps' are left is waiting for the oldest step's;
//    one barrier a step, after which the stage of the step before is free.
//  * A row's 16-byte chunk c lies at c ^ (row / 4 % 4) of its 64 bytes: the 16
//    lanes of a read phase, 16 rows of one chunk, then touch every bank once.
//  * Scales: 16 bytes per row for four steps (a dword per step and row touches
//    a line for each four bytes).  A lane's operand is its row's dword, shifted
//    so that its half's bytes are where the instruction's byte select expects
//    them.
// 2048 x 4096 x 14336: 72 us, 3.3 PFLOP/s; of the 72, 32 are the matrix
// instructions alone (18 ns per instruction and SIMD), 11 the stores of 59 MB.
struct MxArgs {
  const unsigned char* xq;
  const unsigned char* xs;
  const unsigned char* wq;
  const unsigned char* ws;
  const float* bias;
  void* y;
  int64_t M, N, K;
  int ydt;
  int tilesM, tilesN;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_rsrc(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)bytes, 0x00020000);
}

constexpr int kMxN = 256;        // weight rows per block
constexpr int kMxK = 128;        // columns per step

template <int MW>
struct MxStage {
  unsigned char w[kMxN * 64];
  unsigned char x[64 * MW * 64];
};
struct MxScales {                // of four steps, 16 bytes per row
  unsigned char w[kMxN * 16];
  unsigned char x[256 * 16];     // 64 MW rows used
};

typedef int int4v_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

// Two values rounded to nearest even, as a pair of dt (bf16: one instruction).
__device__ __forceinline__ uint32_t pack16(float a, float b, int dt) {
  const f32x2_t v = {a, b};
  return dt == BF16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t))
                    : __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
}

template <int MW>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) k_mxmx(MxArgs a) {
  __shared__ __attribute__((aligned(16))) MxStage<MW> st0, st1, st2, st3;
  __shared__ __attribute__((aligned(16))) MxScales sc0, sc1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % MW, wn = wave / MW;   // 64-row block of X; 32 MW rows of W
  const int T = a.tilesM * a.tilesN, bid = blockIdx.x;
  const int tile = T % 8 == 0 ? (bid % 8) * (T / 8) + bid / 8 : bid;   // runs of tiles per XCD
  const int tm = tile % a.tilesM, tn = tile / a.tilesM;
  const int64_t m0 = (int64_t)tm * 64 * MW, n0 = (int64_t)tn * kMxN;
  const uint32_t rowb = (uint32_t)(a.K / 2), srow = (uint32_t)(a.K / 32);
  const uint32_t nr = (uint32_t)(a.N - n0 < kMxN ? a.N - n0 : kMxN);
  const uint32_t mr = (uint32_t)(a.M - m0 < 64 * MW ? a.M - m0 : 64 * MW);
  const __amdgpu_buffer_rsrc_t rw = mx_rsrc(a.wq + n0 * rowb, nr * rowb);
  const __amdgpu_buffer_rsrc_t rx = mx_rsrc(a.xq + m0 * rowb, mr * rowb);
  // waves 0-3 copy the scales of the weight rows, 4-7 those of X, 64 rows each
  const __amdgpu_buffer_rsrc_t rs = wave < 4 ? mx_rsrc(a.ws + n0 * srow, nr * srow)
                                             : mx_rsrc(a.xs + m0 * srow, mr * srow);

  float16v_t acc[MW][2];
#pragma unroll
  for (int i = 0; i < MW; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  // copies of 16 rows: lane's row lane / 4, its chunk (row / 4 % 4 == lane / 16)
  const uint32_t cat = (uint32_t)(16 * wave + (lane >> 2)) * rowb +
                       16u * (((uint32_t)lane & 3u) ^ ((uint32_t)lane >> 4));
  const uint32_t sat = (uint32_t)(64 * (wave & 3) + lane) * srow;
  const int S = (int)(a.K / kMxK);
  using lds_t = __attribute__((address_space(3))) void*;
  // steps at or past the end load zeros, so that every step has as many loads
  auto load = [&](MxStage<MW>& st, int t) __attribute__((always_inline)) {
    const uint32_t at = t < S ? cat + 64u * (uint32_t)t : kOff;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_t)(st.w + 1024 * (wave + 8 * i)), 16,
                                               t < S ? at + 128u * (uint32_t)i * rowb : kOff, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < (MW + 1) / 2; ++i)
      if (MW > 1 || wave < 4)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_t)(st.x + 1024 * (wave + 8 * i)), 16,
                                                 t < S ? at + 128u * (uint32_t)i * rowb : kOff, 0, 0, 0);
  };
  // the scales of steps t .. t + 3 (the row's last ones may reach into the
  // next row's: bytes of steps that are not taken)
  auto load_sc = [&](MxScales& sc, int t) __attribute__((always_inline)) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_t)((wave < 4 ? sc.w : sc.x) + 1024 * (wave & 3)), 16,
                                             t < S ? sat + 4u * (uint32_t)t : kOff, 0, 0, 0);
  };
  constexpr int kLoads = MW == 4 ? 4 : MW == 2 ? 3 : 2;   // per step; MW == 1: 3 in waves 0-3
  // fragment reads: row (lane & 31) + a multiple of 32, chunk 2 s + lane / 32
  const uint32_t frow = (uint32_t)lane & 31u, half = (uint32_t)lane >> 5;
  const uint32_t wbase = (uint32_t)wn * 32u * MW, xbase = (uint32_t)wm * 64u;
  uint32_t fo[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) fo[s] = 64u * frow + 16u * ((2u * s + half) ^ ((frow >> 2) & 3u));
  auto wide = [](int4v_t v) __attribute__((always_inline)) {
    return int8v_t{v[0], v[1], v[2], v[3], 0, 0, 0, 0};   // 4-bit operands: the first four registers
  };
  // Operands of a step's two halves (64 columns each), the second of which is
  // multiplied after the next barrier, while that step's first fragments come
  // from LDS.
  int4v_t A[2][MW], B[2][2];
  uint32_t sw[MW], sx[2];
#pragma unroll
  for (int i = 0; i < MW; ++i) {
    A[1][i] = int4v_t{0, 0, 0, 0};
    sw[i] = 0;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    B[1][j] = int4v_t{0, 0, 0, 0};
    sx[j] = 0;
  }
  // Products of half H, one read of the other half's operands (then of the
  // scales) after each: the reads of eight waves back up in the LDS queue, and
  // what a wave issues behind them would wait.
  auto product = [&](auto H, int k) __attribute__((always_inline)) {
    constexpr int h = decltype(H)::value;
    const int i = k / 2, j = k % 2;
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
        wide(A[h][i]), wide(B[h][j]), acc[i][j], 4, 4, 2 * h, (int)sw[i], 2 * h, (int)sx[j]);
  };
  auto read = [&](const MxStage<MW>& st, auto H, int k) __attribute__((always_inline)) {
    constexpr int h = decltype(H)::value;
    if (k < 2) B[h][k] = *reinterpret_cast<const int4v_t*>(st.x + 64u * xbase + fo[h] + 2048u * k);
    else A[h][k - 2] = *reinterpret_cast<const int4v_t*>(st.w + 64u * wbase + fo[h] + 2048u * (k - 2));
  };
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;
  auto compute = [&](const MxStage<MW>& st, const MxScales& sc, int t, auto U) __attribute__((always_inline)) {
    constexpr uint32_t u = decltype(U)::value;
    // a step past the end multiplies codes of 0, whose scales (the next row's)
    // must not be NaN
    const uint32_t on = t + (int)u < S ? ~0u : 0u;
    uint32_t nw[MW], nx[2];
    constexpr int P = 2 * MW, R = MW + 2;   // products and operands of a half
#pragma unroll
    for (int k = 0; k < (P > R ? P : R); ++k) {
      if (k < P) product(C1{}, k);
      __builtin_amdgcn_sched_barrier(0);
      if (k < R) read(st, C0{}, k);
      if (k < 2) nx[k] = *reinterpret_cast<const uint32_t*>(sc.x + 16u * xbase + 16u * frow + 512u * k + 4u * u);
      else if (k < R) nw[k - 2] = *reinterpret_cast<const uint32_t*>(sc.w + 16u * wbase + 16u * frow + 512u * (k - 2) + 4u * u);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < MW; ++i) sw[i] = (nw[i] & on) >> (8u * half);
#pragma unroll
    for (int j = 0; j < 2; ++j) sx[j] = (nx[j] & on) >> (8u * half);
#pragma unroll
    for (int k = 0; k < (P > R ? P : R); ++k) {
      if (k < P) product(C0{}, k);
      __builtin_amdgcn_sched_barrier(0);
      if (k < R) read(st, C1{}, k);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // This wave's loads of the oldest step have landed; then everyone's have,
  // and everyone is done with the step before.  Younger: two steps' codes, and
  // the next four steps' scales, which go out after a first step's codes.
  auto turn = [](auto U) __attribute__((always_inline)) {
    constexpr int n = 2 * kLoads + (decltype(U)::value ? 1 : 0);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");   // for the compiler alone: no instructions
    __builtin_amdgcn_s_waitcnt((n & 0xF) | (0x7 << 4) | ((n >> 4) << 14));   // and its LDS reads
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_sched_barrier(0);
  };

  load_sc(sc0, 0);
  load(st0, 0);
  load(st1, 1);
  load(st2, 2);
  auto four = [&](int t, const MxScales& sc, MxScales& next) __attribute__((always_inline)) {
    turn(C0{});
    load(st3, t + 3);
    load_sc(next, t + 4);
    compute(st0, sc, t, C0{});
    turn(C1{});
    load(st0, t + 4);
    compute(st1, sc, t, C1{});
    turn(C2{});
    load(st1, t + 5);
    compute(st2, sc, t, C2{});
    turn(C3{});
    load(st2, t + 6);
    compute(st3, sc, t, C3{});
  };
#pragma unroll 1
  for (int t = 0; t < S; t += 8) {
    four(t, sc0, sc1);
    if (t + 4 < S) four(t + 4, sc1, sc0);
  }
#pragma unroll
  for (int k = 0; k < 2 * MW; ++k) product(C1{}, k);
  __builtin_amdgcn_s_waitcnt(0);   // the loads past the end write the stages too
  __syncthreads();

  // Result: lane = activation row l % 32, weight rows 8 g + 4 (l / 32) + 0..3
  // in registers 4 g .. 4 g + 3.  16-bit outputs turn through the wave's own
  // part of the stages, so that every store is a run of 64 MW bytes of a row.
  const int64_t nw = n0 + wbase;
  auto bias4 = [&](int64_t n, float (&v)[4]) {
    if (!a.bias) return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N)
        v[e] += a.bias[n + e];
  };
  constexpr uint32_t RB = 64u * MW;   // bytes of a row in LDS, chunk c at c ^ (row & (4 MW - 1))
  // two waves' parts per stage
  static_assert(32u * RB * 2u <= sizeof(MxStage<MW>), "room for two waves");
  MxStage<MW>& mine = wave < 2 ? st0 : wave < 4 ? st1 : wave < 6 ? st2 : st3;
  unsigned char* own = reinterpret_cast<unsigned char*>(&mine) + (uint32_t)(wave & 1) * 32u * RB;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t mj = m0 + xbase + 32 * j;
    if (j) __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < MW; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e];
        const int64_t n = nw + 32 * i + 8 * g + 4 * half;
        bias4(n, v);
        if (a.ydt == F32) {
          const int64_t m = mj + frow;
          float* y = static_cast<float*>(a.y) + m * a.N + n;
          if (m < a.M) {
            if (a.N % 4 == 0) {
              if (n < a.N) *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n + e < a.N) y[e] = v[e];
            }
          }
        } else {
          const uint2 h = make_uint2(pack16(v[0], v[1], a.ydt), pack16(v[2], v[3], a.ydt));
          *reinterpret_cast<uint2*>(own + frow * RB + 16u * ((4u * i + g) ^ (frow & (4u * MW - 1u))) + 8u * half) = h;
        }
      }
    if (a.ydt == F32) continue;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    constexpr int LR = 4 * MW;   // lanes per row, 8 values each
#pragma unroll
    for (int r = 0; r < 32 * LR / 64; ++r) {
      const int row = r * (64 / LR) + lane / LR, c = lane % LR;
      const uint4 v = *reinterpret_cast<const uint4*>(own + (uint32_t)row * RB +
                                                        16u * ((uint32_t)c ^ ((uint32_t)row & (4u * MW - 1u))));
      const int64_t m = mj + row, n = nw + 8 * c;
      if (m < a.M && n < a.N) {
        uint16_t* y = static_cast<uint16_t*>(a.y) + m * a.N + n;
        if (a.N % 8 == 0) {
          *reinterpret_cast<uint4*>(y) = v;
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < a.N) y[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace

hipError_t launch_mx_quant(const void* x, int xdt, int64_t M, int64_t K, void* q, void* s,
                           hipStream_t st) {
  const int64_t n8 = M * K / 8;
  auto fn = xdt == F32 ? k_mx_quant<F32> : xdt == BF16 ? k_mx_quant<BF16> : k_mx_quant<F16>;
  hipLaunchKernelGGL(fn, dim3(mx_blocks(n8)), dim3(256), 0, st, x, static_cast<uint32_t*>(q),
                     static_cast<uint8_t*>(s), n8);
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const Desc& d, const Bufs& b, void* out, int odt, hipStream_t st) {
  const int64_t n8 = d.N * d.K / 8;
  auto fn = odt == F32 ? k_mx_dequant<F32> : odt == BF16 ? k_mx_dequant<BF16> : k_mx_dequant<F16>;
  hipLaunchKernelGGL(fn, dim3(mx_blocks(n8)), dim3(256), 0, st, static_cast<const uint32_t*>(b.qweight),
                     static_cast<const uint8_t*>(b.scales), out, n8);
  return hipGetLastError();
}

namespace {
int mx_width(int64_t M) { return M <= 64 ? 1 : M <= 128 ? 2 : 4; }   // MW
}  // namespace

int64_t mx_tiles(const Desc& d, int64_t M) {
  const int rows = 64 * mx_width(M);
  return (M + rows - 1) / rows * ((d.N + kMxN - 1) / kMxN);
}

hipError_t launch_mx_mx(const Desc& d, const void* xq, const void* xs, int64_t M, const Bufs& b,
                        const float* bias, void* y, int ydt, hipStream_t s) {
  MxArgs a{static_cast<const unsigned char*>(xq), static_cast<const unsigned char*>(xs),
           static_cast<const unsigned char*>(b.qweight), static_cast<const unsigned char*>(b.scales),
           bias, y, M, d.N, d.K, ydt, 0, 0};
  const int mw = mx_width(M);
  a.tilesM = (int)((M + 64 * mw - 1) / (64 * mw));
  a.tilesN = (int)((d.N + kMxN - 1) / kMxN);
  auto fn = mw == 1 ? k_mxmx<1> : mw == 2 ? k_mxmx<2> : k_mxmx<4>;
  hipLaunchKernelGGL(fn, dim3((unsigned)((int64_t)a.tilesM * a.tilesN)), dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace qp
