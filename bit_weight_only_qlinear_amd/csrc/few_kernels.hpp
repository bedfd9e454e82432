// Packed products for few activation rows: the MXFP4 qGEMV of up to 8 rows, its
// gated pair of up to 16, and the two products of a mixture-of-experts layer, whose
// experts' rows lie one after the other in the packed buffers.
//
// All of them are bound by the codes' way from HBM, so the arithmetic has to
// stay out of the way of 16-byte loads.  v_mfma_f32_4x4x4_16b does that: it
// multiplies 16 independent 4 x 4 x 4 blocks, lane l holding column l % 4 of
// block l / 4 in B and in the result alike.  With the codes as B, a lane owns
// one weight row (of four) and one 32-column chunk (of sixteen), i.e. one
// 16-byte load; its accumulators are four activation rows of exactly that
// chunk, so a format's scale and offset are two numbers of the same lane:
//     y += S sum (MAG + u) x + T sum x,
// with u the code, MAG + u held exactly (128 + u in bf16, 1024 + u in fp16;
// MXFP4: the E2M1 value itself, MAG = T = 0, by one hardware conversion per
// two codes) and sum x from the same instruction against ones.  One wave
// load covers four rows x 256 contiguous bytes.  Four activation rows cost
// the same as one; each further four cost 8 matrix instructions (64 cycles)
// per 1 KiB of codes, still twice what HBM delivers at 16 rows.
//
// Four waves per block.  KW of them split a row's 512-column steps, the
// others take other rows.  A team of KW waves runs over its rows in passes of
// 4 G, as one stream: the codes of the next two steps are always on their way,
// those of the next pass while a pass's sums are taken.  The sums over lanes
// are a transposed reduction (permlane swaps, then DPP), those over waves meet
// in LDS.  The metadata of the block's rows is staged in LDS by direct loads,
// in front of the first codes.
//
// Experts: a block's unit is (an expert that some token chose, 4 Q of its tokens,
// some of its rows or features); every block finds its own from the ids, in LDS.
// Grids cover as many as the tokens could need; blocks past the ones that are end
// at once.  (An expert's tokens one after the other in one block: 22 tokens of
// 2 experts of 736 x 1568 42 us instead of 27, 50 x 4096 x 1536 105 and 100.)
//
// 1 x 4096 x 14336: 9.0 us, 3.5 TB/s, of which 4 us are the launch, the metadata
// and the first codes.  Experts: 2 of 8 of 4096 x 14336 int4 31 + 16 us (4.2 TB/s),
// 64 of 2048 x 1024 MXFP4 with 2 tokens each 33 + 21 (3.9), 32 of 4096 x 1536 with
// 6 each 60 + 33 (3.4; the tokens beyond eight read their expert again).
#pragma once
#include "device_common.hpp"
#include "mlp_common.hpp"
#include "qp_internal.hpp"

namespace qp {
namespace {

enum FKind : int { F_MX4 = 0, F_AFF4 = 1, F_AFF4H = 2, F_Q4K = 3, F_SYM4 = 4 };
enum FMode : int { FM_LINEAR = 0, FM_GATED = 1, FM_UP = 2, FM_DOWN = 3 };
constexpr bool is_pair(int mode) { return mode == FM_GATED || mode == FM_UP; }

constexpr uint32_t kOff = 0x80000000u;   // at or past every resource: reads 0

struct FewArgs {
  Bufs w[2];
  int64_t K, N;            // columns; rows per expert (of the layer)
  int C;                   // 32-column chunks per row
  int gsh;                 // chunk -> group: >> gsh
  int KW, RW;              // waves per row, row teams (KW * RW == 4)
  int feats;               // rows (features of a pair) per team, whole passes
  int tiles;               // blocks per expert (or layer)
  uint32_t mrow[3];        // metadata bytes per row: scales, zeros, steps
  uint32_t mlds[2][3];     // LDS offset of each slice
  uint32_t x_lds;          // and of the tokens' whole rows
  const void* x;           // [rows, K] of 16 bits
  int64_t M;
  void* y;                 // LINEAR, GATED: [M, N] of ydt; UP: h [M topk, N] of
  int ydt;                 //   ydt; DOWN: partial sums [M topk, N] fp32
  const void* bias[2];
  int bdt;                 // type of the biases
  int act;
  const int* ids;          // experts: [M, topk]
  int E, topk;
};

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t few_rsrc(const void* p, uint64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes,
                                           0x00020000);
}

// 16 bytes per lane from `off` into 1 KiB of LDS.
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, unsigned char* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}

template <bool XB>
__device__ __forceinline__ f32x4_t mfma4(uint2 a, uint2 b, f32x4_t c) {
  if constexpr (XB)
    return __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(short4_t, a),
                                                  __builtin_bit_cast(short4_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(half4_t, a),
                                              __builtin_bit_cast(half4_t, b), c, 0, 0, 0);
}

// A barrier for what the block's waves exchange through LDS, which leaves loads in
// flight.  The wait and the barrier do the work; the fences, which are no
// instructions, keep the compiler from moving LDS accesses over them.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// E2M1 codes of byte SEL of w, times a power of two, as a pair (exact).
template <bool XB, int SEL>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w, float scale = 1.f) {
  if constexpr (XB)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, SEL));
}

// The 8 codes of one word as two operands of four; MXFP4 in their order,
// nibbles as (0, 4, 1, 5) and (2, 6, 3, 7).
template <int KIND, bool XB>
__device__ __forceinline__ void code_ops(uint32_t w, uint32_t mask, uint32_t mag, uint2& lo, uint2& hi) {
  if constexpr (KIND == F_MX4) {
    lo = make_uint2(e2m1_pair<XB, 0>(w), e2m1_pair<XB, 1>(w));
    hi = make_uint2(e2m1_pair<XB, 2>(w), e2m1_pair<XB, 3>(w));
  } else {
    lo = make_uint2((w & mask) | mag, ((w >> 4) & mask) | mag);
    hi = make_uint2(((w >> 8) & mask) | mag, ((w >> 12) & mask) | mag);
  }
}

// 8 activations (raw bits) in the order of the code operands.
template <int KIND>
__device__ __forceinline__ void x_ops(uint4 u, uint2& lo, uint2& hi) {
  if constexpr (KIND == F_MX4) {
    lo = make_uint2(u.x, u.y);
    hi = make_uint2(u.z, u.w);
  } else {
    lo = make_uint2(__builtin_amdgcn_perm(u.z, u.x, 0x05040100u),
                    __builtin_amdgcn_perm(u.z, u.x, 0x07060302u));
    hi = make_uint2(__builtin_amdgcn_perm(u.w, u.y, 0x05040100u),
                    __builtin_amdgcn_perm(u.w, u.y, 0x07060302u));
  }
}

// E8M0 byte -> fp32: 2^(s - 127), NaN at 255.
__device__ __forceinline__ float e8m0(uint32_t s) {
  const uint32_t b = s == 0 ? 0x00400000u : s << 23;
  return __uint_as_float(s == 255u ? 0x7FC00000u : b);
}

// Raw metadata of one chunk, and what it stands for.
struct Meta {
  uint32_t s, z, p;
};
template <int KIND, typename LD>
__device__ __forceinline__ Meta load_meta(const FewArgs& a, uint32_t c, LD ld) {
  Meta m{0, 0, 0};
  const uint32_t g = c >> a.gsh;
  if constexpr (KIND == F_MX4) {
    m.s = ld(0, c, (uint8_t)0);
  } else if constexpr (KIND == F_Q4K) {
    m.s = ld(0, c, (uint8_t)0);
    m.z = ld(1, c, (uint8_t)0);
    m.p = ld(2, 4u * (c >> 3), 0u);
  } else if constexpr (KIND == F_SYM4) {
    m.s = ld(0, 4u * g, 0u);
  } else {
    m.s = ld(0, 2u * g, (uint16_t)0);
    m.z = ld(1, 2u * g, (uint16_t)0);
  }
  return m;
}
template <int KIND, bool XB>
__device__ __forceinline__ void scale_of(const Meta& m, float& S, float& T) {
  constexpr float MAG = XB ? 128.f : 1024.f;
  if constexpr (KIND == F_MX4) {
    S = e8m0(m.s);
    T = 0.f;
  } else if constexpr (KIND == F_Q4K) {
    S = (float)m.s * f16_to_f32(m.p & 0xFFFFu);
    T = -S * (MAG + (float)m.z * f16_to_f32(m.p >> 16));
  } else if constexpr (KIND == F_SYM4) {
    S = __uint_as_float(m.s);
    T = -S * (MAG + 8.f);
  } else {
    S = KIND == F_AFF4 ? bf16_to_f32(m.s) : f16_to_f32(m.s);
    T = fmaf(-MAG, S, KIND == F_AFF4 ? bf16_to_f32(m.z) : f16_to_f32(m.z));
  }
}

// What a block works on.
struct Unit {
  int64_t row0;            // first row of its expert in the packed buffers
  int brow0, brows;        // rows (features) of the block inside the expert
  int T;                   // tokens
};

// v[16] summed over the 16 lanes of equal l % 4: afterwards register k of a
// lane of 16-lane row R holds value 4 k + (((R & 1) << 1) | (R >> 1)).
__device__ __forceinline__ void sum16(float (&v)[16], float (&o)[4]) {
  float b[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[2 * k]),
                                                    __float_as_uint(v[2 * k + 1]), false, false);
    b[k] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(b[2 * k]),
                                                    __float_as_uint(b[2 * k + 1]), false, false);
    o[k] = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    o[k] += dpp_f<QP_DPP_ROW_ROR8>(0.f, o[k]);
    o[k] += dpp_f<QP_DPP_ROW_ROR4>(0.f, o[k]);
  }
}

// The tokens of a pass: their rows of x (uniform byte offsets) and how many
// there are.
template <int Q>
struct Tok {
  uint32_t off[4 * Q];
  int n;
};

__device__ __forceinline__ void few_store(void* y, int64_t i, float v, int dt) {
  if (dt == F32) static_cast<float*>(y)[i] = v;
  else if (dt == BF16) static_cast<uint16_t*>(y)[i] = (uint16_t)f32_to_bf16_rne(v);
  else static_cast<uint16_t*>(y)[i] = (uint16_t)f32_to_f16_rne(v);
}

// Tokens t0 .. t0 + 4 Q - 1 of the unit, all rows of the block.  A pass of
// a team takes rows 4 g + l % 4 for g < G from its row f0 on (a pair: g < G / 2
// of layer 0, the others of layer 1).  xrow, orow: rows of x and of the output,
// per token; red: two buffers of the passes' partial sums.
//
// 16-bit activations come through the wave's own part of LDS (xl): a load
// instruction takes 1 KiB of one token's row, where the operands' own layout
// would touch 64 pieces of 64 bytes (16 tokens: 2.4 TB/s of codes at most).
// Token t's 16-byte piece j lies at j ^ (t % 4), so that the 16 lanes of a read
// phase (four tokens, four chunks) touch every bank once.  Tokens that are not
// there read what else is in LDS: they are rows of results of their own.
// WHOLE: the tokens' whole rows are loaded once per block, step by step, and
// serve all of its waves and passes.
template <int KIND, bool XB, bool WHOLE, int Q, int MODE>
__device__ __forceinline__ void few_run(const FewArgs& a, const Unit& u, const unsigned char* smem,
                                        const uint32_t (&mbase)[2][3],
                                        const __amdgpu_buffer_rsrc_t (&rw)[2],
                                        const __amdgpu_buffer_rsrc_t rx, unsigned char* xl,
                                        const int* xrow, const int* orow, int t0, float* red) {
  constexpr bool PAIR = is_pair(MODE);
  constexpr int G = 4;                               // groups of four rows per pass
  constexpr int F = PAIR ? 2 * G : 4 * G;            // features per pass
  constexpr int kRed = 4 * G * 4 * Q;                // sums of a wave and pass
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave % a.KW, team = wave / a.KW;
  const uint32_t j = lane & 3, b = lane >> 2;
  const uint32_t C = (uint32_t)a.C, rowb = (uint32_t)(a.K / 2);
  const int S = (a.C + 15) / 16;
  const int base = team * a.feats;                   // the team's first row
  if constexpr (!WHOLE) xl += wave * 4096 * Q;
  Tok<Q> tok;
  tok.n = u.T - t0 < 4 * Q ? u.T - t0 : 4 * Q;
#pragma unroll
  for (int t = 0; t < (WHOLE ? 0 : 4 * Q); ++t)
    tok.off[t] = t < tok.n ? (uint32_t)__builtin_amdgcn_readfirstlane(xrow[t0 + t]) * (uint32_t)(a.K * 2) : 0u;
  auto layer = [](int g) { return PAIR && g >= G / 2 ? 1 : 0; };
  auto lrow = [&](int f0, int g) { return (uint32_t)f0 + 4u * (PAIR ? g % (G / 2) : g) + j; };

  struct Step {
    uint4 w[G];
  };
  auto load = [&](int f0, int s, bool on, Step& st) __attribute__((always_inline)) {
    const uint32_t at = on && (uint32_t)s * 16u + b < C ? lrow(f0, 0) * rowb + 16u * b + (uint32_t)s * 256u : kOff;
    // in this order, or the wait for one step's first codes is one for all
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      st.w[g] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                              rw[layer(g)], at + 4u * (PAIR ? g % (G / 2) : g) * rowb, 0, 2));
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto load_x = [&](int s) __attribute__((always_inline)) {
    if constexpr (WHOLE) {
    } else {
      const bool ok = (uint32_t)s * 16u + b < C;
#pragma unroll
      for (int t = 0; t < 4 * Q; ++t)
        if (t < tok.n)
          to_lds(rx, xl + 1024 * t,
                 ok ? tok.off[t] + (uint32_t)s * 1024u + 16u * ((uint32_t)lane ^ (t & 3u)) : kOff);
    }
  };
  // nibbles: 128 (bf16) or 1024 (fp16) and the code in its low bits, one
  // v_and_or_b32 from registers (two literals would make it two instructions)
  uint32_t mask = 0x000F000Fu, mag = XB ? 0x43004300u : 0x64006400u;
  asm("" : "+v"(mask), "+s"(mag));
  uint32_t jm[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) jm[i] = j * a.mrow[i];
  const uint32_t xr = j * 1024u + 64u * b + 16u * j;   // piece 0 of the lane's token and chunk

  f32x4_t acc[G][Q];
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int q = 0; q < Q; ++q) acc[g][q] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // Step s of the pass at f0 from st; `more`: another step follows, at sx.
  auto compute = [&](int f0, int s, const Step& st, bool more, int sx) __attribute__((always_inline)) {
    const uint32_t c = (uint32_t)s * 16u + b, cc = c < C ? c : C - 1u;
    if constexpr (!WHOLE) {
      // the compiler does not see these copies: what was issued after them are
      // the next step's G loads (and stores)
      __builtin_amdgcn_s_waitcnt((G & 0xF) | (0x7 << 4) | (0xF << 8));
      __builtin_amdgcn_sched_barrier(0);
    }
    const unsigned char* xs0 = WHOLE ? xl + (uint32_t)(s * tok.n) * 1024u : xl;
    uint2 xo[Q][8];
    f32x4_t xs[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        x_ops<KIND>(*reinterpret_cast<const uint4*>(xs0 + 4096u * q + (xr ^ (16u * v))), xo[q][2 * v], xo[q][2 * v + 1]);
    }
    if (!WHOLE && more) {   // its activations, now that this step's are read
      __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4));   // lgkmcnt(0)
      __builtin_amdgcn_sched_barrier(0);
      load_x(sx);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      xs[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if constexpr (KIND != F_MX4) {
        const uint32_t one = XB ? 0x3F803F80u : 0x3C003C00u;
#pragma unroll
        for (int v = 0; v < 8; ++v) xs[q] = mfma4<XB>(xo[q][v], make_uint2(one, one), xs[q]);
      }
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      // LDS has room for whole passes; rows past the block's last are sums of
      // their own that nothing stores
      const Meta m = load_meta<KIND>(a, cc, [&](int i, uint32_t o, auto t) {
        const uint32_t row = mbase[layer(g)][i] + ((uint32_t)f0 + 4u * (PAIR ? g % (G / 2) : g)) * a.mrow[i];
        return (uint32_t)*reinterpret_cast<const decltype(t)*>(smem + row + (jm[i] + o));
      });
      float Sv, Tv;
      scale_of<KIND, XB>(m, Sv, Tv);
      f32x4_t d[Q];
#pragma unroll
      for (int q = 0; q < Q; ++q) d[q] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      const uint32_t wv[4] = {st.w[g].x, st.w[g].y, st.w[g].z, st.w[g].w};
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint2 lo, hi;
        code_ops<KIND, XB>(wv[v], mask, mag, lo, hi);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          d[q] = mfma4<XB>(xo[q][2 * v], lo, d[q]);
          d[q] = mfma4<XB>(xo[q][2 * v + 1], hi, d[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[g][q][i] = fmaf(Sv, d[q][i], acc[g][q][i]);
          if constexpr (KIND != F_MX4) acc[g][q][i] = fmaf(Tv, xs[q][i], acc[g][q][i]);
        }
    }
  };
  // A pass's sums over lanes; waves that share rows meet in LDS, in two buffers
  // by turns, so that one barrier per pass is enough.
  const int R = lane >> 4, p4 = ((R & 1) << 1) | (R >> 1);
  auto put = [&](int row, int t, float g, float v) __attribute__((always_inline)) {
    if (row >= u.brows || t0 + t >= u.T) return;
    const int64_t n = u.brow0 + row;
    if constexpr (MODE == FM_LINEAR || MODE == FM_GATED) {
      auto bias = [&](const void* p) {
        if (a.bdt == F32) return static_cast<const float*>(p)[n];
        return meta_to_f32(static_cast<const uint16_t*>(p)[n], a.bdt == BF16);
      };
      if (a.bias[0]) g += bias(a.bias[0]);
      if (PAIR && a.bias[1]) v += bias(a.bias[1]);
    }
    if constexpr (PAIR) g = (a.act == ACT_SILU ? act_f<ACT_SILU>(g) : act_f<ACT_GELU_TANH>(g)) * v;
    if constexpr (MODE == FM_DOWN)
      static_cast<float*>(a.y)[(int64_t)orow[t0 + t] * a.N + n] = g;
    else
      few_store(a.y, (int64_t)orow[t0 + t] * a.N + n, g, a.ydt);
  };
  auto finish = [&](int f0, int pass) __attribute__((always_inline)) {
    float* rb = red + (pass & 1) * 4 * kRed;
    float* mine = rb + wave * kRed;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float o[G / 4][4];   // rows 16 h + 4 k + l % 4 of the pass, token 4 q + p4
#pragma unroll
      for (int h = 0; h < G / 4; ++h) {
        float v[16];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[4 * k + i] = acc[4 * h + k][q][i];
            acc[4 * h + k][q][i] = 0.f;
          }
        sum16(v, o[h]);
      }
      if ((lane & 12) == 0) {
        if (a.KW == 1) {
#pragma unroll
          for (int k = 0; k < (PAIR ? G / 2 : G); ++k)
            put(f0 + 4 * k + (int)j, 4 * q + p4, o[k / 4][k % 4], PAIR ? o[(k + G / 2) / 4][(k + G / 2) % 4] : 0.f);
        } else {
#pragma unroll
          for (int k = 0; k < G; ++k) mine[(4 * k + (int)j) * (4 * Q) + 4 * q + p4] = o[k / 4][k % 4];
        }
      }
    }
    if (a.KW == 1) return;
    lds_barrier();
    // the team's threads: (feature, token) with the feature fastest
    for (int i = threadIdx.x - team * a.KW * 64; i < F * 4 * Q; i += a.KW * 64) {
      const int fe = i % F, t = i / F;
      const float* r = rb + team * a.KW * kRed + t;
      float g = 0.f, v = 0.f;
      for (int w = 0; w < a.KW; ++w) {
        g += r[w * kRed + fe * 4 * Q];
        if constexpr (PAIR) v += r[w * kRed + (F + fe) * 4 * Q];
      }
      put(f0 + fe, t, g, v);
    }
  };

  // the wave's steps: n per pass; passes whose rows lie past the block's end
  // are left out, for all teams alike (the first team has the most)
  const int n = (S - kw + a.KW - 1) / a.KW;
  const int passes = ((u.brows < a.feats ? u.brows : a.feats) + F - 1) / F, total = passes * n;
  const int end = base + passes * F;
  int lf = base, lk = 0;   // next load: row and step of its pass
  auto next = [&](Step& st) __attribute__((always_inline)) {
    // Past the last pass it reads nothing, but it is issued: after loads that
    // may not have been, the wait for one step's codes is a wait for all.
    load(lf, kw + lk * a.KW, lf < end, st);
    if (++lk == n) {
      lk = 0;
      lf += F;
    }
  };
  Step s0, s1;
  if constexpr (WHOLE) {
    // 1 KiB of one token and step per load, dealt out to the waves
    for (int i = wave; i < S * tok.n; i += 4) {
      const int s = i / tok.n, t = i - s * tok.n;
      to_lds(rx, xl + 1024 * i,
             (uint32_t)s * 16u + b < C ? (uint32_t)__builtin_amdgcn_readfirstlane(xrow[t0 + t]) * (uint32_t)(a.K * 2) +
                                             (uint32_t)s * 1024u + 16u * ((uint32_t)lane ^ ((uint32_t)t & 3u))
                                       : kOff);
    }
  }
  load_x(kw);
  next(s0);
  next(s1);
  {
    // the metadata's and the rows' copies were issued before these loads
    constexpr int w = 2 * G;
    static_assert(w < 64, "a wait counts to 63");
    __builtin_amdgcn_s_waitcnt((w & 0xF) | (0x7 << 4) | (0xF << 8) | ((w >> 4) << 14));
    __syncthreads();
  }
  int f0 = base, k = 0, pass = 0;
  auto step = [&](int i, Step& st) __attribute__((always_inline)) {
    const bool last = k + 1 == n;
    compute(f0, kw + k * a.KW, st, i + 1 < total, kw + (last ? 0 : (k + 1) * a.KW));
    next(st);
    ++k;
    if (last) {
      if (i < total) finish(f0, pass);
      k = 0;
      f0 += i + 1 < total ? F : 0;
      ++pass;
    }
  };
  // Two by two; an odd last step is followed by one that adds to sums nobody
  // reads.  (Left out by a branch, the compiler's wait for s0's codes is also
  // one for s1's.)
  for (int i = 0; i < total; i += 2) {
    step(i, s0);
    step(i + 1, s1);
  }
}

constexpr int kTok = 64;          // tokens of a call
constexpr int kExperts = 512;
constexpr int kSlots = 16;        // experts per token

// The want-th (expert that some token chose, TQ of its tokens): the expert, its
// tokens (rising) and each one's first slot with it, and the first of the TQ; -1
// where there are fewer.  Every wave ends up with the answer; xrow and orow are
// complete after the last barrier.
template <int MODE, int TQ>
__device__ __forceinline__ int find_unit(const FewArgs& a, int want, int* mask, int* ids, int* xrow,
                                         int* orow, int& T, int& t0) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int n = (int)a.M * a.topk;
  int got[kTok * kSlots / 256];
#pragma unroll
  for (int k = 0; k < kTok * kSlots / 256; ++k) got[k] = tid + 256 * k < n ? a.ids[tid + 256 * k] : -1;
  for (int e = tid; e < 2 * a.E; e += 256) mask[e] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTok * kSlots / 256; ++k) {
    const int i = tid + 256 * k, e = got[k];
    if (i < n) ids[i] = e;
    if (e >= 0 && e < a.E) {
      const int m = i / a.topk;
      atomicOr(&mask[2 * e + (m >> 5)], (int)(1u << (m & 31)));
    }
  }
  __syncthreads();
  // by falling number of tokens, so that the longest blocks start first
  int cnt[kExperts / 64], most = 0;
#pragma unroll
  for (int i = 0; i < kExperts / 64; ++i) {
    const int e = 64 * i + lane;
    cnt[i] = 64 * i < a.E && e < a.E ? __popc((unsigned)mask[2 * e]) + __popc((unsigned)mask[2 * e + 1]) : 0;
    most = cnt[i] > most ? cnt[i] : most;
  }
  for (int off = 32; off > 0; off >>= 1) {
    const int o = __shfl_xor(most, off, 64);
    most = o > most ? o : most;
  }
  int found = -1;
  for (int t = most, left = want; t > 0 && found < 0; --t) {
#pragma unroll
    for (int i = 0; i < kExperts / 64; ++i) {
      if (found >= 0 || 64 * i >= a.E) continue;
      uint64_t bits = __ballot(cnt[i] == t);
      const int p = (t + TQ - 1) / TQ, n = __popcll(bits) * p;
      if (left < n) {
        for (int k = left / p; k > 0; --k) bits &= bits - 1;
        found = 64 * i + __ffsll((unsigned long long)bits) - 1;
        t0 = left % p * TQ;
      }
      left -= n;
    }
  }
  found = __builtin_amdgcn_readfirstlane(found);
  if (found < 0) return -1;
  const uint64_t tok = (uint64_t)(uint32_t)mask[2 * found] | ((uint64_t)(uint32_t)mask[2 * found + 1] << 32);
  T = __popcll(tok);
  if (tid < 64 && ((tok >> lane) & 1)) {
    const int at = __popcll(tok & ((uint64_t(1) << lane) - 1));
    int s = 0;
    while (ids[lane * a.topk + s] != found) ++s;   // ends: the token is in the mask
    const int slot = lane * a.topk + s;
    xrow[at] = MODE == FM_UP ? lane : slot;
    orow[at] = slot;
  }
  __syncthreads();
  return found;
}

template <int KIND, bool XB, bool WHOLE, int Q, int MODE>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2)))
k_few(FewArgs a) {
  constexpr bool EXPERTS = MODE == FM_UP || MODE == FM_DOWN;
  constexpr bool PAIR = is_pair(MODE);
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  // activations by steps, 4 Q KiB per wave: an array of its own, or the compiler
  // takes their loads for writes to the metadata and waits for them before
  // reading it
  __shared__ __attribute__((aligned(16))) unsigned char xstep[WHOLE ? 16 : 4 * 4096 * Q];
  unsigned char* xbuf = WHOLE ? smem + a.x_lds : xstep;
  __shared__ float red[2 * 4 * 64 * Q];
  __shared__ int xrow[kTok], orow[kTok];
  __shared__ int mask[EXPERTS ? 2 * kExperts : 1], ids[EXPERTS ? kTok * kSlots : 1];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  Unit u;
  int expert = 0, t0 = 0;
  const int tile = (int)(blockIdx.x % (unsigned)a.tiles);   // and the expert or the tile of x's rows
  int64_t xbase = 0;
  if constexpr (EXPERTS) {
    expert = find_unit<MODE, 4 * Q>(a, (int)(blockIdx.x / (unsigned)a.tiles), mask, ids, xrow, orow, u.T, t0);
    if (expert < 0) return;
  } else {
    xbase = (int64_t)(blockIdx.x / (unsigned)a.tiles) * (4 * Q);
    u.T = (int)(a.M - xbase < 4 * Q ? a.M - xbase : 4 * Q);
    if (tid < 4 * Q) {
      xrow[tid] = tid;
      orow[tid] = tid;
    }
  }
  const int rows = a.RW * a.feats;
  u.brow0 = tile * rows;
  u.brows = (int)(a.N - u.brow0 < rows ? a.N - u.brow0 : rows);
  u.row0 = (int64_t)expert * a.N + u.brow0;

  // resources of the block's rows; its metadata into LDS (1 KiB per wave and
  // instruction, whole 16-byte units; bytes past the slice read 0)
  __amdgpu_buffer_rsrc_t rw[2];
  uint32_t mbase[2][3];
#pragma unroll
  for (int l = 0; l < (PAIR ? 2 : 1); ++l) {
    rw[l] = few_rsrc(static_cast<const unsigned char*>(a.w[l].qweight) + u.row0 * (a.K / 2),
                     (uint64_t)u.brows * (uint64_t)(a.K / 2));
    const void* arr[3] = {a.w[l].scales, a.w[l].zeros, a.w[l].steps};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint64_t at = (uint64_t)u.row0 * a.mrow[i], lo = at & ~uint64_t(15);
      const uint32_t head = (uint32_t)(at - lo), bytes = head + (uint32_t)u.brows * a.mrow[i];
      mbase[l][i] = a.mlds[l][i] + head;
      if (a.mrow[i]) {
        const __amdgpu_buffer_rsrc_t rm = few_rsrc(static_cast<const unsigned char*>(arr[i]) + lo, (bytes + 15u) & ~15u);
        for (uint32_t ch = (uint32_t)wave; ch * 1024u < bytes; ch += 4)
          to_lds(rm, smem + a.mlds[l][i] + ch * 1024u, ch * 1024u + 16u * (uint32_t)lane);
      }
    }
  }
  if constexpr (!PAIR) rw[1] = rw[0];
  const int64_t xrows = MODE == FM_DOWN ? a.M * a.topk : a.M - xbase;
  const int64_t xr = EXPERTS || xrows < 4 * Q ? xrows : 4 * Q, xrowb = a.K * 2;
  const __amdgpu_buffer_rsrc_t rx =
      few_rsrc(static_cast<const unsigned char*>(a.x) + xbase * xrowb, (uint64_t)(xr * xrowb));
  if constexpr (!EXPERTS) {
    FewArgs b = a;
    if (xbase) b.y = static_cast<unsigned char*>(a.y) + xbase * a.N * (a.ydt == F32 ? 4 : 2);
    __syncthreads();
    few_run<KIND, XB, WHOLE, Q, MODE>(b, u, smem, mbase, rw, rx, xbuf, xrow, orow, 0, red);
  } else {
    if (Q == 1 || u.T - t0 <= 4)
      few_run<KIND, XB, WHOLE, 1, MODE>(a, u, smem, mbase, rw, rx, xbuf, xrow, orow, t0, red);
    else
      few_run<KIND, XB, WHOLE, Q, MODE>(a, u, smem, mbase, rw, rx, xbuf, xrow, orow, t0, red);
  }
}

inline int few_kind(const Desc& d) {
  if (d.fmt == MXFP4) return F_MX4;
  if (d.fmt == AFFINE && d.bits == 4) return d.meta == BF16 ? F_AFF4 : F_AFF4H;
  if (d.fmt == Q4K) return F_Q4K;
  if (d.fmt == SYM4) return F_SYM4;
  return -1;
}

constexpr int64_t kFewWaves = 1536, kFewBlocks = 1024;

// Sizes, LDS layout and launch shape that the modes share; units: experts or row
// tiles of x; tokens: the most a pass can have, of `slots` (4 Q).  a.x_lds: where
// the tokens' whole rows lie, or 0.
inline size_t fill(const Desc& d, int64_t rows, int64_t units, bool pair, int tokens, int slots, FewArgs& a) {
  a.K = d.K;
  a.N = rows;
  a.C = (int)(d.K / 32);
  a.gsh = 0;
  const int kind = few_kind(d);
  if (d.gs == d.K && kind == F_SYM4) a.gsh = 31;
  else while ((32 << a.gsh) < d.gs) ++a.gsh;
  const int S = (a.C + 15) / 16;
  const int F = 16;   // at most so many rows or features in a pass
  // Waves per row: as few as fill the chip, since waves that share rows have to
  // add their sums up and take the activations again: 8 rows of 4096 x 14336 on two
  // and four 11.6 and 15.5 us, 4 of 5120 x 25600 on one and two 16.8 and 20.3.
  // (Passes of 32 rows for up to four tokens: 1 x 14336 x 4096 12.8 instead of 9.3
  // us, 1 x 5120 x 25600 19.8 instead of 15.6.)
  a.KW = 1;
  while (a.KW < 4 && 2 * a.KW <= S && units * ((rows + F - 1) / F) * a.KW < kFewWaves) a.KW *= 2;
  for (int i = 0; i < 3; ++i) a.mrow[i] = 0;
  if (kind == F_MX4) a.mrow[0] = (uint32_t)(d.K / 32);
  else if (kind == F_Q4K) { a.mrow[0] = a.mrow[1] = (uint32_t)(d.K / 32); a.mrow[2] = (uint32_t)(d.K / 256 * 4); }
  else if (kind == F_SYM4) a.mrow[0] = (uint32_t)(d.K / d.gs * 4);
  else a.mrow[0] = a.mrow[1] = (uint32_t)(d.K / d.gs * 2);
  auto meta = [&](int feats) {
    a.RW = 4 / a.KW;
    size_t lds = 0;
    for (int l = 0; l < (pair ? 2 : 1); ++l)
      for (int i = 0; i < 3; ++i) {
        a.mlds[l][i] = (uint32_t)lds;
        if (a.mrow[i]) lds += ((size_t)a.RW * feats * a.mrow[i] + 15 + 1023) / 1024 * 1024;
      }
    return lds;
  };
  while (a.KW < 4 && 2 * a.KW <= S && meta(F) > 32 * 1024) a.KW *= 2;
  a.RW = 4 / a.KW;
  // Rows per team: so many that the blocks of all experts (or row tiles of x)
  // come to a few per CU, while their metadata fits 12 KiB and their codes 1 GiB.
  const int64_t most = units * ((rows + a.RW * F - 1) / (a.RW * F));
  int64_t k = most / kFewBlocks;
  if (k < 1) k = 1;
  while (k > 1 && (meta((int)k * F) > 12 * 1024 || k * F * a.RW * (d.K / 2) > (int64_t(1) << 30))) --k;
  a.feats = (int)k * F;
  a.tiles = (int)((rows + a.RW * a.feats - 1) / (a.RW * a.feats));
  const size_t lds = meta(a.feats), x = (size_t)S * (size_t)tokens * 1024u;
  a.x_lds = 0;
  if (x > 0 && x + lds <= 72 * 1024) a.x_lds = (uint32_t)lds;   // two blocks per CU
  // Slots without a token are read past the last row, a step of n tokens in S n KiB
  // up to KiB (S - 1) n + its slots: 4 with n from 1 (an expert's few), the others with
  // n from slots - 3 or, in one tile of 16, from 9; later tiles with n < slots end
  // inside S slots.
  const int past = slots - tokens > 3 ? slots - tokens : 3;
  return a.x_lds ? lds + x + (size_t)past * 1024u : lds;
}

using FewFn = void (*)(FewArgs);

}  // namespace
}  // namespace qp
