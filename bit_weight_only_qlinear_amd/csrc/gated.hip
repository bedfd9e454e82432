// Gated pair of projections on packed weights, fp16 MFMA:
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u,
// and, for training, 8-bit checkpoints of g and u.
//
//  * A block's 256 weight rows are 128 features of both layers: LDS rows 128
//    wi + 0 .. 63 hold the gate's features 64 wi .. of the tile, rows 128 wi
//    + 64 .. 127 the up's.  A wave (128 rows x 64 or 32 activation rows) so
//    ends with g and u of the same outputs in the same lane, and 64
//    consecutive features of a row, one checkpoint group, in a pair of lanes:
//    the activation, the product and both checkpoints are register work, and
//    neither g nor u goes to memory.
//  * Weights go through LDS dequantized to fp16 as in the qGEMM (same tile
//    layout and column order); activations are staged once per call (stage.hip)
//    and their fragments loaded from L2 straight into registers a step ahead.
//  * Scales and biases come in 16-byte chunks (8 groups, 16 codes or 4 fp32
//    scales) a chunk ahead where the rows are whole chunks, else per step: a
//    wave's 32 rows make two loads of 32 cache lines each per step otherwise.
//  * Bounded by the matrix cores: 4 M N K flop against N K bytes of codes.
//    Where the last round of 256-row tiles would fill at most half of the 256
//    CUs it is cut into tiles of 128 activation rows: 2048 x 4096 x 14336 makes
//    896 tiles, three full rounds and 256 half tiles instead of four rounds.
//    Few tiles are cut along K instead: the blocks' fp32 shares of g and u meet
//    in a fixed order in a second kernel, which then has the activation.
#include "gemm_kernels.hpp"
#include "mlp_common.hpp"

namespace qp {
namespace {

constexpr int kGF = 128;               // features per tile
constexpr uint32_t kOff = 0x80000000u; // past every resource: reads 0

struct GatedK {
  Bufs gate, up;
  const unsigned char* xf;   // staged x: [step][4][MB][64] 16-byte chunks
  const int* xe;             // row exponents
  const uint16_t* bias_g;
  const uint16_t* bias_u;
  void* h;
  int8_t* gq;                // checkpoints of g and u, or null
  float* gs;
  int8_t* uq;
  float* us;
  int64_t M, N, K;
  int lg;                    // log2(group size / 32)
  int mb, xb, hdt, act;
  int MB, T;                 // 32-row blocks of x, steps of 64 columns
  int tilesM, full;          // 256-row tiles; how many of them run whole
  int small, tilesM1;        // all tiles of 128 rows; their number along M
  int split;                 // blocks along K; > 1: sums into part, all tiles alike
  float* part;               // [split, M, 2, Np]
  int64_t Np;                // N rounded up to 4
};

// One k-step of one thread: half a weight row (32 columns), raw.
template <int KIND>
struct GStage {
  uint32_t w[GT<KIND>::W / 2];
  uint32_t h[GT<KIND>::H > 0 ? GT<KIND>::H / 2 : 1];
  uint32_t s0, s1, s2;   // metadata (where it comes per step)
};

// A chunk of a row's metadata: scales, biases or zero codes, step words.
struct GChunk {
  uint4 s, z;
  uint2 p;
};

struct GRes {
  __amdgpu_buffer_rsrc_t w, h, s, z, p;
  uint32_t wo, ho, so, zo, po;   // the thread's half row; starts of its metadata rows
  uint32_t half;
};

__device__ __forceinline__ uint32_t sel4(const uint4& v, int i) {   // uniform i
  const uint32_t a = i & 1 ? v.y : v.x, b = i & 1 ? v.w : v.z;
  return i & 2 ? b : a;
}

// Steps per chunk.
template <int KIND>
__device__ __forceinline__ int chunk_steps(int lg) {
  return KIND == G_Q4K ? 8 : KIND == G_Q6K ? 4 : KIND == G_SYM4 ? 2 << lg : 4 << lg;
}

template <int KIND>
__device__ __forceinline__ void load_chunk(const GRes& r, int c, GChunk& m) {
  m.s = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r.s, r.so + 16u * (uint32_t)c, 0, 0));
  if constexpr (KIND != G_Q6K && KIND != G_SYM4)
    m.z = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r.z, r.zo + 16u * (uint32_t)c, 0, 0));
  if constexpr (KIND == G_Q4K)
    m.p = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r.p, r.po + 8u * (uint32_t)c, 0, 0));
  if constexpr (KIND == G_Q6K)
    m.p.x = __builtin_amdgcn_raw_buffer_load_b16(r.p, r.po + 2u * (uint32_t)c, 0, 0);
}

// The raw metadata of step t (in its chunk) into a stage.
template <int KIND>
__device__ __forceinline__ void chunk_meta(const GChunk& m, int t, int lg, uint32_t half,
                                           GStage<KIND>& st) {
  const int r = t & (chunk_steps<KIND>(lg) - 1);
  if constexpr (KIND == G_Q4K) {
    const uint32_t sh = 16u * (uint32_t)(r & 1) + 8u * half;
    st.s0 = sel4(m.s, r >> 1) >> sh;
    st.s1 = sel4(m.z, r >> 1) >> sh;
    st.s2 = r & 4 ? m.p.y : m.p.x;
  } else if constexpr (KIND == G_Q6K) {
    st.s0 = sel4(m.s, r) >> (16u * half);
    st.s2 = m.p.x;
  } else if constexpr (KIND == G_SYM4) {
    const uint32_t a = sel4(m.s, (2 * r) >> lg), b = sel4(m.s, (2 * r + 1) >> lg);
    st.s0 = half ? b : a;
  } else {
    const uint32_t sh = 16u * (((2u * (uint32_t)r + half) >> lg) & 1u);
    const int w = ((2 * r) >> lg) >> 1;
    st.s0 = sel4(m.s, w) >> sh;
    st.s1 = sel4(m.z, w) >> sh;
  }
}

// Steps at or past the row's end read the next row's data or 0 (every offset
// is range-checked); the staged activations are 0 there.
template <int KIND, bool CH>
__device__ __forceinline__ void load_codes(const GRes& r, int t, int lg, GStage<KIND>& st) {
  constexpr int W = GT<KIND>::W;
  const uint32_t wk = r.wo + (uint32_t)t * (W * 4);
  if constexpr (W == 4) {
    const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r.w, wk, 0, 0));
    st.w[0] = v.x; st.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < W / 8; ++i) {
      const uint4 v = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(r.w, wk + 16u * i, 0, 0));
      st.w[4 * i] = v.x; st.w[4 * i + 1] = v.y; st.w[4 * i + 2] = v.z; st.w[4 * i + 3] = v.w;
    }
  }
  if constexpr (KIND == G_Q6K) {
    const uint2 v = __builtin_bit_cast(
        uint2, __builtin_amdgcn_raw_buffer_load_b64(r.h, r.ho + (uint32_t)t * 16u, 0, 0));
    st.h[0] = v.x; st.h[1] = v.y;
  }
  if constexpr (!CH) {
    const uint32_t g2 = 2u * (uint32_t)t + r.half;
    if constexpr (KIND == G_Q4K) {
      st.s0 = __builtin_amdgcn_raw_buffer_load_b8(r.s, r.so + g2, 0, 0);
      st.s1 = __builtin_amdgcn_raw_buffer_load_b8(r.z, r.zo + g2, 0, 0);
      st.s2 = __builtin_amdgcn_raw_buffer_load_b32(r.p, r.po + (uint32_t)(t / 4) * 4u, 0, 0);
    } else if constexpr (KIND == G_SYM4) {
      st.s0 = __builtin_amdgcn_raw_buffer_load_b32(r.s, r.so + (g2 >> lg) * 4u, 0, 0);
    } else if constexpr (KIND == G_AFF2 || KIND == G_AFF4 || KIND == G_AFF8) {
      st.s0 = __builtin_amdgcn_raw_buffer_load_b16(r.s, r.so + (g2 >> lg) * 2u, 0, 0);
      st.s1 = __builtin_amdgcn_raw_buffer_load_b16(r.z, r.zo + (g2 >> lg) * 2u, 0, 0);
    }
  }
}

// A step's scales and offsets of the half row, for gchunk.
template <int KIND>
struct GScale {
  half2_t S[2], T[2];   // broadcast; Q6K, SYM4: hi and lo parts of the scale (Q6K: per group)
  half2_t s, t;         // Q4K: lo parts
  float Sf, Tf;         // AFF8
};

__device__ __forceinline__ void split2(float v, half2_t& hi, half2_t& lo) {
  hi.x = hi.y = (_Float16)v;
  lo.x = lo.y = (_Float16)(v - (float)hi.x);
}

template <int KIND>
__device__ __forceinline__ void scales_of(const GStage<KIND>& st, int mb, GScale<KIND>& c) {
  if constexpr (KIND == G_Q4K) {
    const float S = (float)(st.s0 & 0xFFu) * f16_to_f32(st.s2 & 0xFFFFu);
    split2(S, c.S[0], c.s);
    split2(-S * ((float)(st.s1 & 0xFFu) * f16_to_f32(st.s2 >> 16)), c.T[0], c.t);
  } else if constexpr (KIND == G_Q6K) {
#pragma unroll
    for (int g = 0; g < 2; ++g)
      split2((float)(int8_t)((st.s0 >> (8 * g)) & 0xFFu) * f16_to_f32(st.s2 & 0xFFFFu), c.S[g], c.T[g]);
  } else if constexpr (KIND == G_SYM4) {
    split2(__uint_as_float(st.s0), c.S[0], c.T[0]);
  } else if constexpr (KIND != G_SYM4C) {
    c.Sf = meta_to_f32(st.s0 & 0xFFFFu, mb);
    c.Tf = meta_to_f32(st.s1 & 0xFFFFu, mb);
    c.S[0].x = c.S[0].y = (_Float16)c.Sf;
    c.T[0].x = c.T[0].y = (_Float16)c.Tf;
  }
}

// Chunk j (8 columns) of the half row as fp16 in the order (0,4,1,5,2,6,3,7).
// Pairs 0 and 2 as 1024 + u; pairs 1 and 3 of nibbles left at mantissa bits 4
// and up of 64, whose unit they are: 64 + u, without a shift.  Then the exact
// u (less the format's zero) and one rounding or two of about 2^-12 each:
// AFF2, AFF4 fma(u, S, T); SYM4, Q6K fma(v, S, v s); Q4K fma(u, S, T) +
// fma(u, s, t), S + s and T + t being the scale and the offset.  8-bit codes
// go through fp32: their scales are the smallest, next to fp16's subnormals.
template <int KIND>
__device__ __forceinline__ uint4 gchunk(const GStage<KIND>& st, int j, const GScale<KIND>& c,
                                        uint32_t magic, uint32_t magic64) {
  uint32_t p[4];
  if constexpr (KIND == G_AFF8) {
    auto f = [&](int e) { return (float)((st.w[2 * j + (e >> 2)] >> (8 * (e & 3))) & 255u); };
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = pack_f16(fmaf(f(i), c.Sf, c.Tf), fmaf(f(i + 4), c.Sf, c.Tf));
    return make_uint4(p[0], p[1], p[2], p[3]);
  }
  constexpr bool NIB = KIND != G_AFF2 && KIND != G_AFF8;
  constexpr float OFF = KIND == G_Q6K ? 32.f : (KIND == G_SYM4 || KIND == G_SYM4C) ? 8.f : 0.f;
  constexpr float M0 = 1024.f + OFF, M1 = (NIB ? 64.f : 1024.f) + OFF;
  const half2_t mag[2] = {{(_Float16)M0, (_Float16)M0}, {(_Float16)M1, (_Float16)M1}};
  uint32_t h = 0;   // Q6K: high bits of columns 0-3 and 4-7 in the halves; AFF2: the codes
  if constexpr (KIND == G_Q6K || KIND == G_AFF2) {
    const uint32_t v = KIND == G_Q6K ? st.h[(j >> 1) % (GT<KIND>::H > 0 ? GT<KIND>::H / 2 : 1)]
                                     : st.w[j >> 1];
    h = __builtin_amdgcn_perm(0u, v, j & 1 ? 0x0C030C02u : 0x0C010C00u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t q;
    if constexpr (KIND == G_AFF2) {
      q = and_or(h >> (2 * i), 0x00030003u, magic);
    } else {
      uint32_t m = i & 1 ? magic64 : magic;
      if constexpr (KIND == G_Q6K) {   // bits 2 i, 2 i + 1 to 4, 5 or (odd i) 8, 9
        const int up = (i & 1 ? 8 : 4) - 2 * i;
        m = and_or(up >= 0 ? h << (up >= 0 ? up : 0) : h >> (up >= 0 ? 0 : -up),
                   i & 1 ? 0x03000300u : 0x00300030u, m);
      }
      q = and_or(i < 2 ? st.w[j] : st.w[j] >> 8, i & 1 ? 0x00F000F0u : 0x000F000Fu, m);
    }
    const half2_t v = __builtin_bit_cast(half2_t, q) - mag[i & 1];   // exact
    half2_t w = v;
    if constexpr (KIND == G_Q4K)
      w = __builtin_elementwise_fma(v, c.S[0], c.T[0]) + __builtin_elementwise_fma(v, c.s, c.t);
    else if constexpr (KIND == G_Q6K)
      w = __builtin_elementwise_fma(v, c.S[j >> 1], v * c.T[j >> 1]);
    else if constexpr (KIND == G_SYM4)
      w = __builtin_elementwise_fma(v, c.S[0], v * c.T[0]);
    else if constexpr (KIND != G_SYM4C)
      w = __builtin_elementwise_fma(v, c.S[0], c.T[0]);
    p[i] = __builtin_bit_cast(uint32_t, w);
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}

// What makes checkpoint codes of a group with the given scale: rint(v up inv)
// & keep.  The quotient is taken in fp32 (the values carry the fp16 weights'
// rounding anyway); up, a power of two, keeps the reciprocal of a subnormal
// scale finite; keep is 0 where the scale is not finite, whose codes are 0.
struct CodeOf {
  float up, inv;
  uint32_t keep;
};
__device__ __forceinline__ CodeOf code_of(float scale) {
  const float up = scale < 0x1p-100f ? 0x1p64f : 1.f;
  return {up, scale > 0.f ? 1.f / (scale * up) : 0.f, scale < __builtin_inff() ? 255u : 0u};
}
__device__ __forceinline__ uint32_t code8(float v, const CodeOf& c) {
  return (uint32_t)(int)rintf(fminf(fmaxf(v * c.up * c.inv, -127.f), 127.f)) & c.keep;
}

// g and u of the lane's four consecutive features f .. f + 3 in block (i, j).
template <int KIND, int J, bool BIAS = true>
__device__ __forceinline__ void pre_act4(const GatedK& a, const float16_t (&acc)[4][J], int i, int j,
                                         int g4, int f, int xe, float (&g)[4], float (&u)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    g[q] = ldexpf(acc[i][j][4 * g4 + q], -xe);
    u[q] = ldexpf(acc[i + 2][j][4 * g4 + q], -xe);
  }
  const int last = (int)a.N - 1;
  asm volatile("" : "+v"(f));   // keeps the loads below from gathering ahead of all their uses
  if constexpr (KIND == G_SYM4C) {   // channel scales: the contraction ran on the codes
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int fc = min(f + q, last);
      g[q] *= static_cast<const float*>(a.gate.scales)[fc];
      u[q] *= static_cast<const float*>(a.up.scales)[fc];
    }
  }
  if constexpr (!BIAS) return;
  if (a.bias_g) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t b = a.bias_g[min(f + q, last)];
      g[q] += a.xb ? bf16_to_f32(b) : f16_to_f32(b);
    }
  }
  if (a.bias_u) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t b = a.bias_u[min(f + q, last)];
      u[q] += a.xb ? bf16_to_f32(b) : f16_to_f32(b);
    }
  }
}

// The wave's 64 features of 32 rows as 16-bit words or bytes in its 8 KiB of
// LDS: h rows of 128 bytes, code rows of 64 behind them, in 16-byte chunks at
// chunk ^ row bits (64 banks: 2 h rows or 4 code rows share a bank line).
__device__ __forceinline__ uint32_t h_at(int r, int chunk) {
  return (uint32_t)(r * 128 + ((chunk ^ (r >> 1)) & 7) * 16);
}
__device__ __forceinline__ uint32_t q_at(int r, int chunk) {
  return (uint32_t)(r * 64 + ((chunk ^ (r >> 2)) & 3) * 16);
}

// Epilogue: lane (el) holds features 8 g + 4 (el >> 5) + q of each 32 of the
// wave's 64, of row el & 31 of each 32-row block.  16-bit outputs whose rows
// keep 16-byte chunks (N % 16 == 0) go through the wave's part of LDS (the
// weight tiles are done with) and leave as whole lines: stored straight from
// the accumulators' layout, 8 bytes of h and 4 of each code row per lane, the
// 2048 x 4096 x 14336 layer with checkpoints took 18 us longer on the L2's
// request rate.
template <int KIND, int J, int ACT>
__device__ __forceinline__ void finish(const GatedK& a, float16_t (&acc)[4][J], int el, int mbw,
                                       int f0, unsigned char* lds) {
  const int N = (int)a.N;
  const bool lines = N % 16 == 0 && a.hdt != F32, vec = N % 4 == 0;
  const int hh = el >> 5;
  static_for<J>([&](auto JJ) {
    constexpr int j = decltype(JJ)::value;
    const int64_t mb = (int64_t)(mbw + j) * 32, m = mb + (el & 31);
    const bool mok = m < a.M;
    const int xe = mok ? a.xe[m] : 0;
    float mg = 0.f, mu = 0.f;
    static_for<8>([&](auto G) {   // g and u in place of the accumulators
      constexpr int i = decltype(G)::value / 4, g4 = decltype(G)::value % 4;
      const int f = f0 + 32 * i + 8 * g4 + 4 * hh;
      float g[4], u[4];
      pre_act4<KIND, J>(a, acc, i, j, g4, f, xe, g, u);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[i][j][4 * g4 + q] = g[q];
        acc[i + 2][j][4 * g4 + q] = u[q];
        mg = max_nan(mg, f + q < N ? fabsf(g[q]) : 0.f);
        mu = max_nan(mu, f + q < N ? fabsf(u[q]) : 0.f);
      }
    });
    CodeOf cg{}, cu{};
    if (a.gq) {   // group scales: 32 values here, 32 in the other half wave
      mg = plain_nan(div_rn(max_nan(mg, __shfl_xor(mg, 32, 64)), 127.f));
      mu = plain_nan(div_rn(max_nan(mu, __shfl_xor(mu, 32, 64)), 127.f));
      cg = code_of(mg);
      cu = code_of(mu);
      if (mok && el < 32) {
        const int64_t at = m * ((a.N + kCkptGroup - 1) / kCkptGroup) + f0 / kCkptGroup;
        a.gs[at] = mg;
        a.us[at] = mu;
      }
    }
    unsigned char* hrow = static_cast<unsigned char*>(a.h) + m * N * (a.hdt == F32 ? 4 : 2);
    int8_t* grow = a.gq + m * N;
    int8_t* urow = a.uq + m * N;
    static_for<8>([&](auto G) {
      constexpr int i = decltype(G)::value / 4, g4 = decltype(G)::value % 4;
      const int f = f0 + 32 * i + 8 * g4 + 4 * hh;
      uint32_t b[4], c[4] = {0, 0, 0, 0}, d[4] = {0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float g = acc[i][j][4 * g4 + q], u = acc[i + 2][j][4 * g4 + q];
        const float v = act_f<ACT>(g) * u;
        b[q] = a.hdt == F32 ? __float_as_uint(v) : a.hdt == BF16 ? f32_to_bf16_rne(v) : f32_to_f16_rne(v);
      }
      if (a.gq) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          c[q] = code8(acc[i][j][4 * g4 + q], cg);
          d[q] = code8(acc[i + 2][j][4 * g4 + q], cu);
        }
      }
      const uint32_t cw = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
      const uint32_t dw = d[0] | d[1] << 8 | d[2] << 16 | d[3] << 24;
      if (lines) {
        *reinterpret_cast<uint2*>(lds + h_at(el & 31, 4 * i + g4) + 8 * hh) =
            make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
        if (a.gq) {
          const uint32_t at = 4096u + q_at(el & 31, 2 * i + g4 / 2) + 8 * (g4 & 1) + 4 * hh;
          *reinterpret_cast<uint32_t*>(lds + at) = cw;
          *reinterpret_cast<uint32_t*>(lds + at + 2048u) = dw;
        }
      } else if (mok && vec && f < N) {
        if (a.hdt == F32)
          *reinterpret_cast<uint4*>(hrow + 4 * f) = make_uint4(b[0], b[1], b[2], b[3]);
        else
          *reinterpret_cast<uint2*>(hrow + 2 * f) = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
        if (a.gq) {
          *reinterpret_cast<uint32_t*>(grow + f) = cw;
          *reinterpret_cast<uint32_t*>(urow + f) = dw;
        }
      } else if (mok && !vec) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (f + q >= N) break;
          if (a.hdt == F32) reinterpret_cast<uint32_t*>(hrow)[f + q] = b[q];
          else reinterpret_cast<uint16_t*>(hrow)[f + q] = (uint16_t)b[q];
          if (a.gq) {
            grow[f + q] = (int8_t)c[q];
            urow[f + q] = (int8_t)d[q];
          }
        }
      }
    });
    if (lines) {
      lds_turn();
      unsigned char* h = static_cast<unsigned char*>(a.h);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 8 * k + (el >> 3), ch = el & 7, f = f0 + 8 * ch;
        const uint4 v = *reinterpret_cast<const uint4*>(lds + h_at(r, ch));
        if (mb + r < a.M && f < N) *reinterpret_cast<uint4*>(h + ((mb + r) * N + f) * 2) = v;
      }
      if (a.gq) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int r = 16 * k + (el >> 2), ch = el & 3, f = f0 + 16 * ch;
          const uint4 v = *reinterpret_cast<const uint4*>(lds + 4096 + q_at(r, ch));
          const uint4 w = *reinterpret_cast<const uint4*>(lds + 6144 + q_at(r, ch));
          if (mb + r < a.M && f < N) {
            *reinterpret_cast<uint4*>(a.gq + (mb + r) * N + f) = v;
            *reinterpret_cast<uint4*>(a.uq + (mb + r) * N + f) = w;
          }
        }
      }
      lds_turn();
    }
  });
}

// The same for one of several blocks along K: its share of g and u.
template <int KIND, int J>
__device__ __forceinline__ void finish_part(const GatedK& a, float16_t (&acc)[4][J], int el, int mbw,
                                            int f0, int sp) {
  static_for<J>([&](auto JJ) {
    constexpr int j = decltype(JJ)::value;
    const int64_t m = (int64_t)(mbw + j) * 32 + (el & 31);
    if (m < a.M) {
      const int xe = a.xe[m];
      float* row = a.part + ((int64_t)sp * a.M + m) * 2 * a.Np;
      static_for<8>([&](auto G) {
        constexpr int i = decltype(G)::value / 4, g4 = decltype(G)::value % 4;
        const int f = f0 + 32 * i + 8 * g4 + 4 * (el >> 5);
        float g[4], u[4];
        pre_act4<KIND, J, false>(a, acc, i, j, g4, f, xe, g, u);
        if (f < a.Np) {
          *reinterpret_cast<float4*>(row + f) = make_float4(g[0], g[1], g[2], g[3]);
          *reinterpret_cast<float4*>(row + a.Np + f) = make_float4(u[0], u[1], u[2], u[3]);
        }
      });
    }
  });
}

// Joins the shares of one row's group of 64 features (one wave each), in
// order: bias, activation, product, checkpoints.
template <int ACT>
__global__ void __launch_bounds__(256) k_gated_join(GatedK a) {
  const uint32_t ng = (uint32_t)((a.N + kCkptGroup - 1) / kCkptGroup);
  const uint32_t id = blockIdx.x * 4u + (threadIdx.x >> 6);
  if (id >= (uint64_t)a.M * ng) return;   // whole waves
  const int64_t m = id / ng, grp = id - (uint32_t)m * ng, f = grp * 64 + (threadIdx.x & 63);
  const bool ok = f < a.N;
  const float* p = a.part + m * 2 * a.Np + (ok ? f : 0);
  const int64_t step = a.M * 2 * a.Np;
  float g = 0.f, u = 0.f;
  for (int s = 0; s < a.split; ++s) {
    g += p[s * step];
    u += p[s * step + a.Np];
  }
  if (ok && a.bias_g) g += a.xb ? bf16_to_f32(a.bias_g[f]) : f16_to_f32(a.bias_g[f]);
  if (ok && a.bias_u) u += a.xb ? bf16_to_f32(a.bias_u[f]) : f16_to_f32(a.bias_u[f]);
  const int64_t at = m * a.N + f;
  if (ok) {
    const float h = act_f<ACT>(g) * u;
    if (a.hdt == F32) static_cast<float*>(a.h)[at] = h;
    else static_cast<uint16_t*>(a.h)[at] =
        (uint16_t)(a.hdt == BF16 ? f32_to_bf16_rne(h) : f32_to_f16_rne(h));
  }
  if (a.gq) {
    const float mg = plain_nan(div_rn(wave_max_nan(ok ? fabsf(g) : 0.f), 127.f));
    const float mu = plain_nan(div_rn(wave_max_nan(ok ? fabsf(u) : 0.f), 127.f));
    if (ok) {
      a.gq[at] = (int8_t)code8(g, code_of(mg));
      a.uq[at] = (int8_t)code8(u, code_of(mu));
    }
    if ((threadIdx.x & 63) == 0) {
      a.gs[m * ng + grp] = mg;
      a.us[m * ng + grp] = mu;
    }
  }
}

// One tile: features n0 .. n0 + 127, 32-row blocks mb0 .. of x (J per wave),
// share sp of the steps along K.
template <int KIND, bool CH, int J>
__device__ __forceinline__ void gated_tile(const GatedK& a, unsigned char* smem, int64_t n0, int mb0,
                                           int sp) {
  const int t0 = (int)((int64_t)a.T * sp / a.split), t1 = (int)((int64_t)a.T * (sp + 1) / a.split);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave >> 2, wj = wave & 3;
  const int64_t K = a.K;
  const int mbw = mb0 + wj * J;   // this wave's first row block

  // the wave stages LDS rows 32 wave .. + 31: one layer, 32 features
  GRes r;
  {
    const bool up = (wave >> 1) & 1;
    const Bufs b = {up ? a.up.qweight : a.gate.qweight, up ? a.up.qweight_hi : a.gate.qweight_hi,
                    up ? a.up.scales : a.gate.scales, up ? a.up.zeros : a.gate.zeros,
                    up ? a.up.steps : a.gate.steps};
    const int64_t nrows = a.N - n0 < kGF ? a.N - n0 : kGF;
    const uint32_t f = (uint32_t)(wrow_of(tid) - 32 * wave + 64 * wi + 32 * (wave & 1));
    auto res = [&](const void* p, int64_t row) {
      return rsrc(static_cast<const unsigned char*>(p) + n0 * row, (uint32_t)(nrows * row));
    };
    r.half = (uint32_t)(tid & 1);
    const int64_t wrow = KIND == G_AFF2 ? K / 4 : KIND == G_AFF8 ? K : K / 2;
    r.w = res(b.qweight, wrow);
    r.wo = f * (uint32_t)wrow + r.half * (uint32_t)(GT<KIND>::W * 2);
    r.h = r.s = r.z = r.p = r.w;
    r.ho = r.so = r.zo = r.po = 0;
    const int64_t ng = (K / 32) >> a.lg;
    if constexpr (KIND == G_Q4K) {
      r.s = res(b.scales, K / 32);
      r.z = res(b.zeros, K / 32);
      r.p = res(b.steps, (K / 256) * 4);
      r.so = r.zo = f * (uint32_t)(K / 32);
      r.po = f * (uint32_t)((K / 256) * 4);
    } else if constexpr (KIND == G_Q6K) {
      r.h = res(b.qweight_hi, K / 4);
      r.ho = f * (uint32_t)(K / 4) + r.half * 8u;
      r.s = res(b.scales, K / 16);
      r.p = res(b.steps, (K / 256) * 2);
      r.so = f * (uint32_t)(K / 16);
      r.po = f * (uint32_t)((K / 256) * 2);
    } else if constexpr (KIND == G_SYM4) {
      r.s = res(b.scales, ng * 4);
      r.so = f * (uint32_t)(ng * 4);
    } else if constexpr (KIND != G_SYM4C) {
      r.s = res(b.scales, ng * 2);
      r.z = res(b.zeros, ng * 2);
      r.so = r.zo = f * (uint32_t)(ng * 2);
    }
  }

  float16_t acc[4][J];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  // weight fragments, as in the qGEMM: lane row lane & 31, chunk 2 s + (lane >> 5)
  uint32_t fa[4];
#pragma unroll
  for (int s = 0; s < 4; ++s)
    fa[s] = (uint32_t)(lane & 31) * 128u + (uint32_t)wi * 128u * 128u +
            (uint32_t)(((2 * s + (lane >> 5)) ^ ((lane >> 1) & 7)) * 16);
  auto rd_a = [&](uint32_t buf, int s, int i) {
    return *reinterpret_cast<const half8_t*>(smem + fa[s] + (buf * kTileBytes + 4096u * i));
  };
  uint32_t xo[J];
#pragma unroll
  for (int j = 0; j < J; ++j)
    xo[j] = mbw + j < a.MB ? (uint32_t)(mbw + j) * 1024u + 16u * (2u * (lane & 31) + (lane >> 5)) : kOff;
  const uint32_t xs = (uint32_t)a.MB * 1024u;   // one k-slice of 16
  auto ld_b = [&](int t, int s, int j) {
    const __amdgpu_buffer_rsrc_t rx = rsrc(a.xf + (int64_t)(t < t1 ? t : t0) * 4 * xs, 4u * xs);
    // the slice as the scalar offset: the range check is on xo[j] alone, and
    // a row block inside a slice is inside all four
    return __builtin_bit_cast(half8_t,
                              __builtin_amdgcn_raw_buffer_load_b128(rx, xo[j], (uint32_t)s * xs, 0));
  };
  const int wn = wrow_of(tid);
  const uint32_t magic = 0x64006400u, magic64 = 0x54005400u;   // 1024, 64
  auto put = [&](uint32_t buf, int p, const GStage<KIND>& st, const GScale<KIND>& sc) {
    const int j = 4 * (tid & 1) + p;
    *reinterpret_cast<uint4*>(smem + (uint32_t)wn * 128u + (uint32_t)((j ^ ((wn >> 1) & 7)) * 16) +
                              buf * kTileBytes) = gchunk<KIND>(st, p, sc, magic, magic64);
  };

  half8_t Bf[4][J];
  GChunk cur, nxt;
  const int MP = chunk_steps<KIND>(a.lg);
  constexpr bool RING = CH && KIND != G_SYM4C;

  // Fragments of the step; A[2] and A[3] of its last slice, with Bf[3], are
  // kept for the products that run after the next barrier.
  half8_t A[4];
  A[2] = A[3] = half8_t{};
#pragma unroll
  for (int j = 0; j < J; ++j) Bf[3][j] = half8_t{};
  auto deferred = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 2; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A[i], Bf[3][j], acc[i][j], 0, 0, 0);
  };

  // One step: MFMAs on LDS buffer buf = (t - t0) & 1 and the fragments of x in Bf (reloaded
  // slice by slice for step t + 1); conversion of step t + 1 (`nx`) into the
  // other buffer; code loads of step t + 2 into `fre`.
  auto kstep = [&](auto BUF, int t, GStage<KIND>& fre, GStage<KIND>& nx) {
    constexpr uint32_t buf = decltype(BUF)::value;
    load_codes<KIND, CH>(r, t + 2, a.lg, fre);
    if constexpr (RING) {
      if (((t + 1) & (MP - 1)) == 0) {   // step t + 1 starts a chunk
        cur = nxt;
        load_chunk<KIND>(r, (t + 1) / MP + 1, nxt);
      }
      chunk_meta<KIND>(cur, t + 1, a.lg, r.half, nx);
    }
    GScale<KIND> sc;
    scales_of<KIND>(nx, a.mb, sc);
    // the matrix cores start on the last step's deferred products while this
    // step's first fragments come from LDS
    A[0] = rd_a(buf, 0, 0);
    A[1] = rd_a(buf, 0, 1);
    __builtin_amdgcn_sched_barrier(0);
    deferred();
    A[2] = rd_a(buf, 0, 2);
    A[3] = rd_a(buf, 0, 3);
#pragma unroll
    for (int j = 0; j < J; ++j) Bf[3][j] = ld_b(t, 3, j);
    static_for<4>([&](auto S) {
      constexpr int s = decltype(S)::value;
      static_for<(s < 3 ? 4 : 2)>([&](auto I) {
        constexpr int i = decltype(I)::value;
#pragma unroll
        for (int j = 0; j < J; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A[i], Bf[s][j], acc[i][j], 0, 0, 0);
        if constexpr (s < 3) A[i] = rd_a(buf, s + 1, i);
      });
      if constexpr (s < 3) {
#pragma unroll
        for (int j = 0; j < J; ++j) Bf[s][j] = ld_b(t + 1, s, j);
      }
      put(buf ^ 1u, s, nx, sc);
    });
    __syncthreads();
  };

  GStage<KIND> st0, st1;
  load_codes<KIND, CH>(r, t0, a.lg, st0);
  load_codes<KIND, CH>(r, t0 + 1, a.lg, st1);
  if constexpr (RING) {
    load_chunk<KIND>(r, t0 / MP, cur);
    load_chunk<KIND>(r, t0 / MP + 1, nxt);
    chunk_meta<KIND>(cur, t0, a.lg, r.half, st0);
  }
#pragma unroll
  for (int s = 0; s < 3; ++s)
#pragma unroll
    for (int j = 0; j < J; ++j) Bf[s][j] = ld_b(t0, s, j);
  {
    GScale<KIND> sc;
    scales_of<KIND>(st0, a.mb, sc);
#pragma unroll
    for (int p = 0; p < 4; ++p) put(0u, p, st0, sc);
  }
  __syncthreads();
  for (int t = t0; t < t1; t += 2) {
    kstep(std::integral_constant<uint32_t, 0>{}, t, st0, st1);
    if (t + 1 < t1) kstep(std::integral_constant<uint32_t, 1>{}, t + 1, st1, st0);
  }
  deferred();

  int el = lane;
  asm volatile("" : "+v"(el));   // keeps the epilogue's addresses after the loop
  const int f0 = (int)n0 + 64 * wi;
  if (f0 >= a.N) return;
  if (a.part) {
    finish_part<KIND, J>(a, acc, el, mbw, f0, sp);
    return;
  }
  unsigned char* lds = smem + 8192 * wave;
  if (a.act == ACT_SILU) finish<KIND, J, ACT_SILU>(a, acc, el, mbw, f0, lds);
  else finish<KIND, J, ACT_GELU_TANH>(a, acc, el, mbw, f0, lds);
}

template <int KIND, bool CH>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
k_gated(GatedK a) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[2 * kTileBytes];
  // contiguous runs of tiles per XCD, m fastest
  const int bid = blockIdx.x;
  auto run = [](int i, int n) { return n % 8 == 0 ? (i % 8) * (n / 8) + i / 8 : i; };
  if (bid < a.full) {
    const int t = run(bid, a.full), sp = t / (a.full / a.split), u = t - sp * (a.full / a.split);
    gated_tile<KIND, CH, 2>(a, smem, (int64_t)(u / a.tilesM) * kGF, (u % a.tilesM) * 8, sp);
  } else {
    const int nh = (int)gridDim.x - a.full, t = run(bid - a.full, nh);
    if (a.small) {
      const int sp = t / (nh / a.split), u = t - sp * (nh / a.split);
      gated_tile<KIND, CH, 1>(a, smem, (int64_t)(u / a.tilesM1) * kGF, (u % a.tilesM1) * 4, sp);
    } else {   // halves of the last round's tiles
      const int u = a.full + t / 2;
      gated_tile<KIND, CH, 1>(a, smem, (int64_t)(u / a.tilesM) * kGF, (u % a.tilesM) * 8 + 4 * (t & 1), 0);
    }
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t frag_bytes(const Desc& d, int64_t M) {
  return (size_t)cdiv(d.K, 64) * 4u * (size_t)cdiv(M, 32) * 1024u;
}

// Tiles and blocks along K.  Time in steps of a 256-row tile (1.85 us on the
// 2048 x 4096 x 14336 layer; 128 rows: 0.7 of that, the weights' share does
// not halve), rounds of 256 blocks, 8 steps of start and end per round, and
// for more than one block along K the shares' traffic and a second kernel.
struct GatedPlan {
  int small, split, full, blocks;
  size_t part;
};
GatedPlan gated_plan(const Desc& d, int64_t M) {
  const int64_t T = cdiv(d.K, 64), nf = cdiv(d.N, kGF), Np = cdiv(d.N, 4) * 4;
  const int64_t t2 = cdiv(M, 256) * nf, t1 = cdiv(M, 128) * nf;
  GatedPlan best{};
  double bt = 0.;
  for (int small = M <= 128 ? 1 : 0; small < 2; ++small) {
    const int64_t tiles = small ? t1 : t2;
    const double c = small ? 0.7 : 1.;
    for (int s = 1; s <= 16 && s * 4 <= T + 3; ++s) {
      if (s > 1 && (tiles * s > 768 || (double)s * M * Np * 8. > 512e6)) break;
      GatedPlan p{small, s, 0, (int)(tiles * s), 0};
      double t;
      if (!small && s == 1) {   // the last round in halves where they fit one
        const int64_t rest = tiles % 256;
        p.full = (int)(rest && rest <= 128 ? tiles - rest : tiles);
        p.blocks = (int)(p.full + 2 * (tiles - p.full));
        t = (double)(T + 8) * ((double)cdiv(p.full, 256) + (p.full < tiles ? 0.7 : 0.));
      } else {
        p.full = small ? 0 : p.blocks;
        t = (double)cdiv(tiles * s, 256) * (double)(cdiv(T, s) + 8) * c;
      }
      if (s > 1) {
        t += 2.2 + (double)s * M * Np * 16. / 4e12 / 1.85e-6;
        p.part = (size_t)s * (size_t)M * 2u * (size_t)Np * 4u;
      }
      if (bt == 0. || t < bt) {
        bt = t;
        best = p;
      }
    }
  }
  return best;
}

template <int KIND>
void (*pick(bool ch))(GatedK) { return ch ? k_gated<KIND, true> : k_gated<KIND, false>; }

}  // namespace

size_t gated_workspace_bytes(const Desc& d, int64_t M) {
  return frag_bytes(d, M) + (size_t)cdiv(M, 32) * 128u + gated_plan(d, M).part;
}

hipError_t launch_gated(const Desc& d, const GatedArgs& g, void* ws, hipStream_t s) {
  GatedK a{};
  a.gate = g.gate;
  a.up = g.up;
  a.xf = static_cast<const unsigned char*>(ws);
  int* xe = reinterpret_cast<int*>(static_cast<unsigned char*>(ws) + frag_bytes(d, g.M));
  a.xe = xe;
  a.bias_g = static_cast<const uint16_t*>(g.bias_g);
  a.bias_u = static_cast<const uint16_t*>(g.bias_u);
  a.h = g.h;
  a.gq = g.gq;
  a.gs = g.gs;
  a.uq = g.uq;
  a.us = g.us;
  a.M = g.M;
  a.N = d.N;
  a.K = d.K;
  a.lg = d.gs == 128 ? 2 : d.gs == 64 ? 1 : 0;
  a.mb = d.meta == BF16;
  a.xb = g.xdt == BF16;
  a.hdt = g.hdt;
  a.act = g.act;
  a.MB = (int)cdiv(g.M, 32);
  a.T = (int)cdiv(d.K, 64);
  const GatedPlan p = gated_plan(d, g.M);
  a.small = p.small;
  a.split = p.split;
  a.full = p.full;
  a.tilesM = (int)cdiv(g.M, 256);
  a.tilesM1 = (int)cdiv(g.M, 128);
  a.Np = cdiv(d.N, 4) * 4;
  if (p.split > 1)
    a.part = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + frag_bytes(d, g.M) +
                                      (size_t)a.MB * 128u);
  StageArgs sa{};
  sa.d = static_cast<const uint16_t*>(g.x);
  sa.xf = ws;
  sa.xe = xe;
  sa.M = g.M;
  sa.N = d.K;
  hipError_t e = launch_stage(sa, g.xdt, false, 0, true, s);
  if (e != hipSuccess) return e;
  // whole 16-byte metadata chunks per row
  const bool ch = d.fmt == Q4K ? d.K % 512 == 0 : d.fmt == SYM4 ? d.K % (4 * d.gs) == 0
                : d.fmt == AFFINE ? d.K % (8 * d.gs) == 0 : true;
  void (*fn)(GatedK) = d.fmt == Q4K ? pick<G_Q4K>(ch)
                     : d.fmt == Q6K ? k_gated<G_Q6K, true>
                     : d.fmt == SYM4 ? (d.gs == d.K ? k_gated<G_SYM4C, true> : pick<G_SYM4>(ch))
                     : d.bits == 2 ? pick<G_AFF2>(ch)
                     : d.bits == 4 ? pick<G_AFF4>(ch) : pick<G_AFF8>(ch);
  hipLaunchKernelGGL(fn, dim3((unsigned)p.blocks), dim3(kThreads), 0, s, a);
  if ((e = hipGetLastError()) != hipSuccess || p.split == 1) return e;
  auto join = g.act == ACT_SILU ? k_gated_join<ACT_SILU> : k_gated_join<ACT_GELU_TANH>;
  hipLaunchKernelGGL(join, dim3((unsigned)cdiv(g.M * cdiv(d.N, kCkptGroup), 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qp
