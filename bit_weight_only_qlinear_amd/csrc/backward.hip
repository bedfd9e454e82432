// Input gradients through packed weights on fp16 MFMA:
//   dx[m, k] = sum_n D[m, n] w[n, k],  D = dy, or for the gated pair
//   D = [dg | du] over the stacked weights [Wg; Wu].
//
// The contraction runs over the weight rows n, while codes are packed along
// k, so a weight tile has to be transposed on its way to the matrix cores.
//  * Each lane loads 32 columns of one weight row (16 bytes of 4-bit codes);
//    the four 16-lane groups of a wave hold four consecutive rows of the same
//    column chunks.  Four v_permlane swaps turn that 4 x 4 (row x word)
//    arrangement around, so that a lane then has 8 columns of four rows: for
//    each column the pairs (n, n+1), (n+2, n+3), cut out of two words at once
//    (v_perm puts the same byte of two rows into the halves of a pair; its low
//    nibbles make 1024 + q, its high ones 64 + q, with no shift), one packed
//    subtract and one packed fma, and one 8-byte LDS write of four
//    consecutive n.  The scales travel the same way: one (S, T) fp16 pair per
//    lane and step, turned by the same swaps.
//  * Weights in fp16, each rounded about once.  AFFINE of 2 and 4 bits: w =
//    fma(q, scale, bias) on fp16 scales and biases, as the qGEMM takes them
//    (bf16 metadata is exact there from 2^-17 up, where the weights themselves
//    reach fp16's subnormals).  8 bits: the fp32 fma, rounded once; their
//    scales are 255ths of a group's range, so ordinary weights (std 3e-4) have
//    bf16 scales that fp16 cannot hold, and 255 codes carry the error (relative
//    L2 of dx 1e-2 there, 2e-4 in fp32; the fp32 form costs 2% at 2048 x 14336
//    x 4096, 252 us, and 7% at 300 rows, 78 us).  Q6K, SYM4: with v =
//    u - 32 or u - 8 exact and the scale split into S + s (two fp16 numbers),
//    w = fma(v, S, v s).  Q4K, scale and offset split: w = fma(q, S, T) +
//    fma(q, s, t).  Rounding the Q4K scale and offset to one fp16 each left
//    weight errors of 2e-4 of the largest weight, past the layer's element
//    bound; a conversion through fp32 would take 2.5 times the instructions.
//  * The LDS tile holds 256 columns of 64 n (128 bytes): column c's 16-byte
//    chunk j at line L = c / 2 (256 bytes, all 64 banks), slot
//    (8 (c & 1) + j) ^ (((L & 7) ^ ((L >> 4) & 7)) + 8 ((L >> 2) & 1)): the 32
//    lanes of an 8-byte write phase (16 columns, both halves of a chunk) and
//    the 16 lanes of a 16-byte read phase (16 neighbouring columns) each touch
//    all 16 slots once.
//  * D is staged once per call as fp16 fragments with one power of two per
//    row (stage.hip), which also computes dg and du from the checkpoints.
//  * Block tile 256 (k) x 256 or 128 (m) x 64 (n), 8 waves as 2 (k) x 4 (m),
//    fragments of D loaded from L2 straight into registers a step ahead.
//  * The output is small and the contraction long, so the steps are split
//    over several blocks where the tiles alone do not fill the 256 CUs; fp32
//    partial sums meet in a fixed order in a second kernel.
#include "gemm_kernels.hpp"
#include "mlp_common.hpp"

namespace qp {
namespace {

constexpr int kDK = 256, kDN = 64;   // tile columns, contraction rows per step
constexpr uint32_t kDTile = kDK * kDN * 2u;
constexpr uint32_t kOff = 0x80000000u;   // past every resource: reads 0

struct DxK {
  Bufs w[2];               // the layer; gate and up
  int64_t N, K, M;
  int gs;
  const unsigned char* xf; // staged D: [step][4][MB][64] 16-byte chunks
  const int* xe;           // row exponents
  float* part;             // [split, M, K] partial sums, or null
  void* dx;
  int dxdt;
  int T1, T;               // steps per part, in all
  int MB;                  // 32-row blocks of D
  int tilesK, tilesM, split;
};

// One step of one lane: 32 columns of weight row 8 wave + 4 ((lane >> 3) & 1)
// + (lane >> 4) of the step.
template <int KIND>
struct DStage {
  uint32_t w[KIND == G_AFF2 ? 2 : KIND == G_AFF8 ? 8 : 4];
  uint32_t h[KIND == G_Q6K ? 2 : 1];
  uint32_t s0, s1, s2;
};

// Per-lane offsets inside a step's 64 rows (kOff for columns past K).
struct DOff {
  uint32_t w, h, s, p;   // s: scales, and zeros alike
};

template <int KIND>
__device__ __forceinline__ constexpr int64_t row_bytes(int64_t K) {
  return KIND == G_AFF2 ? K / 4 : KIND == G_AFF8 ? K : K / 2;
}

template <int KIND>
__device__ __forceinline__ void dload(const DxK& a, const DOff& o, int t, DStage<KIND>& st) {
  // uniform: part and rows of the step; steps past the end get empty resources
  const int second = t >= a.T1 ? 1 : 0;
  const int64_t n0 = (int64_t)(t - (second ? a.T1 : 0)) * kDN;
  const int64_t left = t < a.T ? a.N - n0 : 0;
  const uint32_t rows = (uint32_t)(left < 0 ? 0 : left < kDN ? left : kDN);
  const Bufs& b = a.w[second];
  auto res = [&](const void* p, int64_t row) {
    return rsrc(static_cast<const unsigned char*>(p) + (rows ? n0 * row : 0), rows * (uint32_t)row);
  };
  const int64_t K = a.K;
  const __amdgpu_buffer_rsrc_t rw = res(b.qweight, row_bytes<KIND>(K));
  if constexpr (KIND == G_AFF2) {
    const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rw, o.w, 0, 0));
    st.w[0] = v.x; st.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < (KIND == G_AFF8 ? 2 : 1); ++i) {
      const uint4 v = __builtin_bit_cast(
          uint4, __builtin_amdgcn_raw_buffer_load_b128(rw, o.w + 16u * i, 0, 0));
      st.w[4 * i] = v.x; st.w[4 * i + 1] = v.y; st.w[4 * i + 2] = v.z; st.w[4 * i + 3] = v.w;
    }
  }
  if constexpr (KIND == G_AFF2 || KIND == G_AFF4 || KIND == G_AFF8) {
    const int64_t sr = (K / a.gs) * 2;
    st.s0 = __builtin_amdgcn_raw_buffer_load_b16(res(b.scales, sr), o.s, 0, 0);
    st.s1 = __builtin_amdgcn_raw_buffer_load_b16(res(b.zeros, sr), o.s, 0, 0);
  } else if constexpr (KIND == G_Q4K) {
    st.s0 = __builtin_amdgcn_raw_buffer_load_b8(res(b.scales, K / 32), o.s, 0, 0);
    st.s1 = __builtin_amdgcn_raw_buffer_load_b8(res(b.zeros, K / 32), o.s, 0, 0);
    st.s2 = __builtin_amdgcn_raw_buffer_load_b32(res(b.steps, (K / 256) * 4), o.p, 0, 0);
  } else if constexpr (KIND == G_Q6K) {
    const uint2 v = __builtin_bit_cast(
        uint2, __builtin_amdgcn_raw_buffer_load_b64(res(b.qweight_hi, K / 4), o.h, 0, 0));
    st.h[0] = v.x; st.h[1] = v.y;
    st.s0 = __builtin_amdgcn_raw_buffer_load_b16(res(b.scales, K / 16), o.s, 0, 0);
    st.s2 = __builtin_amdgcn_raw_buffer_load_b16(res(b.steps, (K / 256) * 2), o.p, 0, 0);
  } else {
    st.s0 = __builtin_amdgcn_raw_buffer_load_b32(res(b.scales, (K / a.gs) * 4), o.s, 0, 0);
  }
}

// v_permlane swaps: register t of lane group g <-> register g of lane group t.
__device__ __forceinline__ void turn4(uint32_t (&w)[4]) {
  auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w[0] = c[0]; w[1] = c[1]; w[2] = d[0]; w[3] = d[1];
}

// A stage after the turn: 8 columns of four rows, and the rows' scales and
// offsets as fp16 pairs (S01, S23, T01, T23).
template <int KIND>
struct DTurned {
  uint32_t w[KIND == G_AFF8 ? 8 : 4];   // rows 0..3 (AFF8: columns 0-3, then 4-7)
  uint32_t h[KIND == G_Q6K ? 2 : 1];    // high bits of row pairs
  half2_t S[2], T[2];                   // hi parts (Q6K, SYM4: T is the lo part of S)
  float Sf[KIND == G_AFF8 ? 4 : 1], Tf[KIND == G_AFF8 ? 4 : 1];   // AFF8, instead
  half2_t s[KIND == G_Q4K ? 2 : 1], t[KIND == G_Q4K ? 2 : 1];   // Q4K: lo parts
};

// (hi, lo) fp16 parts of a fp32 number, as the halves of a pair.
__device__ __forceinline__ half2_t split_f16(float v) {
  half2_t r;
  r.x = (_Float16)v;
  r.y = (_Float16)(v - (float)r.x);
  return r;
}

template <int KIND, bool MBF16>
__device__ __forceinline__ void dturn(const DStage<KIND>& st, DTurned<KIND>& d) {
  if constexpr (KIND == G_AFF8) {
    uint32_t p[4] = {st.w[0], st.w[2], st.w[4], st.w[6]}, q[4] = {st.w[1], st.w[3], st.w[5], st.w[7]};
    turn4(p);
    turn4(q);
#pragma unroll
    for (int i = 0; i < 4; ++i) { d.w[i] = p[i]; d.w[4 + i] = q[i]; }
  } else if constexpr (KIND == G_AFF2) {
    uint32_t p[4] = {st.w[0], st.w[0] >> 16, st.w[1], st.w[1] >> 16};
    turn4(p);   // 16-bit pieces: 8 codes in the low half; join the row pairs
    d.w[0] = __builtin_amdgcn_perm(p[1], p[0], 0x05040100u);
    d.w[1] = __builtin_amdgcn_perm(p[3], p[2], 0x05040100u);
  } else {
    uint32_t p[4] = {st.w[0], st.w[1], st.w[2], st.w[3]};
    turn4(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) d.w[i] = p[i];
  }
  if constexpr (KIND == G_Q6K) {
    uint32_t p[4] = {st.h[0], st.h[0] >> 16, st.h[1], st.h[1] >> 16};
    turn4(p);
    d.h[0] = __builtin_amdgcn_perm(p[1], p[0], 0x05040100u);
    d.h[1] = __builtin_amdgcn_perm(p[3], p[2], 0x05040100u);
  }
  uint32_t m[4];
  if constexpr (KIND == G_Q6K) {   // two groups of 16 in the chunk's 32 columns
    const float step = f16_to_f32(st.s2 & 0xFFFFu);
#pragma unroll
    for (int g = 0; g < 2; ++g)
      m[2 * g] = m[2 * g + 1] = __builtin_bit_cast(
          uint32_t, split_f16((float)(int8_t)((st.s0 >> (8 * g)) & 0xFFu) * step));
  } else if constexpr (KIND == G_SYM4) {
    m[0] = m[1] = m[2] = m[3] = __builtin_bit_cast(uint32_t, split_f16(__uint_as_float(st.s0)));
  } else if constexpr (KIND == G_Q4K) {
    const float S = (float)(st.s0 & 0xFFu) * f16_to_f32(st.s2 & 0xFFFFu);
    const float T = -S * ((float)(st.s1 & 0xFFu) * f16_to_f32(st.s2 >> 16));
    const uint32_t hs = __builtin_bit_cast(uint32_t, split_f16(S));
    const uint32_t ht = __builtin_bit_cast(uint32_t, split_f16(T));
    m[0] = m[1] = m[2] = m[3] = __builtin_amdgcn_perm(ht, hs, 0x07060302u);   // lo parts
    turn4(m);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      d.s[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(m[2 * i + 1], m[2 * i], 0x05040100u));
      d.t[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(m[2 * i + 1], m[2 * i], 0x07060302u));
    }
    m[0] = m[1] = m[2] = m[3] = __builtin_amdgcn_perm(ht, hs, 0x05040100u);   // hi parts
  } else if constexpr (KIND == G_AFF8) {
    m[0] = m[1] = m[2] = m[3] = __builtin_amdgcn_perm(st.s1, st.s0, 0x05040100u);   // as stored
    turn4(m);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      d.Sf[i] = meta_to_f32(m[i] & 0xFFFFu, MBF16);
      d.Tf[i] = meta_to_f32(m[i] >> 16, MBF16);
    }
    return;
  } else {
    half2_t v;
    v.x = (_Float16)(MBF16 ? bf16_to_f32(st.s0 & 0xFFFFu) : f16_to_f32(st.s0 & 0xFFFFu));
    v.y = (_Float16)(MBF16 ? bf16_to_f32(st.s1 & 0xFFFFu) : f16_to_f32(st.s1 & 0xFFFFu));
    m[0] = m[1] = m[2] = m[3] = __builtin_bit_cast(uint32_t, v);
  }
  turn4(m);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    d.S[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(m[2 * i + 1], m[2 * i], 0x05040100u));
    d.T[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(m[2 * i + 1], m[2 * i], 0x07060302u));
  }
}

// Columns 2 b and 2 b + 1 of the lane's 8: four consecutive n each.
template <int KIND, int b>
__device__ __forceinline__ void dcols(const DTurned<KIND>& d, uint32_t magic, uint32_t magic64, uint2 (&out)[2]) {
  if constexpr (KIND == G_AFF8) {
    constexpr int o = b < 2 ? 0 : 4, c = (2 * b) & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = fmaf((float)((d.w[o + i] >> (8 * (c + e))) & 255u), d.Sf[i], d.Tf[i]);
      out[e] = make_uint2(pack_f16(w[0], w[1]), pack_f16(w[2], w[3]));
    }
    return;
  }
  // column 2 b: 1024 + u; column 2 b + 1: for nibbles, left where they are in
  // the byte (mantissa bits 4 and up of 64, whose unit they are: 64 + u)
  constexpr bool NIB = KIND != G_AFF2;
  constexpr float OFF = KIND == G_Q6K ? 32.f : KIND == G_SYM4 ? 8.f : 0.f;
  constexpr float M0 = 1024.f + OFF, M1 = (NIB ? 64.f : 1024.f) + OFF;
  const half2_t mag[2] = {{(_Float16)M0, (_Float16)M0}, {(_Float16)M1, (_Float16)M1}};
  uint32_t r[2][2];   // [column][row pair]
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t q[2];
    if constexpr (KIND == G_AFF2) {
      q[0] = and_or(d.w[i] >> (4 * b), 0x00030003u, magic);
      q[1] = and_or(d.w[i] >> (4 * b + 2), 0x00030003u, magic);
    } else {
      constexpr uint32_t sel = 0x0C000C00u | ((4u + b) << 16) | b;
      const uint32_t p = __builtin_amdgcn_perm(d.w[2 * i + 1], d.w[2 * i], sel);
      uint32_t m0 = magic, m1 = magic64;
      if constexpr (KIND == G_Q6K) {   // bits 4 b .. 4 b + 3 of each half: to 4, 5 and 8, 9
        constexpr int e0 = 4 * b - 4, e1 = 4 * b + 2 - 8;
        m0 = and_or(e0 < 0 ? d.h[i] << 4 : d.h[i] >> (e0 < 0 ? 0 : e0), 0x00300030u, magic);
        m1 = and_or(e1 < 0 ? d.h[i] << (e1 < 0 ? -e1 : 0) : d.h[i] >> (e1 < 0 ? 0 : e1), 0x03000300u,
                    magic64);
      }
      q[0] = and_or(p, 0x000F000Fu, m0);
      q[1] = and_or(p, 0x00F000F0u, m1);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const half2_t v = __builtin_bit_cast(half2_t, q[c]) - mag[c];   // exact
      half2_t w;
      if constexpr (KIND == G_Q6K || KIND == G_SYM4)
        w = __builtin_elementwise_fma(v, d.S[i], v * d.T[i]);
      else if constexpr (KIND == G_Q4K)
        w = __builtin_elementwise_fma(v, d.S[i], d.T[i]) + __builtin_elementwise_fma(v, d.s[i], d.t[i]);
      else
        w = __builtin_elementwise_fma(v, d.S[i], d.T[i]);
      r[c][i] = __builtin_bit_cast(uint32_t, w);
    }
  }
  out[0] = make_uint2(r[0][0], r[0][1]);
  out[1] = make_uint2(r[1][0], r[1][1]);
}

// J: 32-row blocks of D per wave (tile rows 128 J).
template <int KIND, bool MBF16, int J>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
k_dx(DxK a) {
  __shared__ __attribute__((aligned(16))) unsigned char smem[2 * kDTile];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave >> 2, wj = wave & 3;

  // contiguous runs of (split, m, k) tiles per XCD, k fastest: the blocks of
  // a run read the same rows of D at the same time
  const int nt = a.tilesK * a.tilesM * a.split, bid = blockIdx.x;
  const int tile = (nt % 8 == 0) ? (bid % 8) * (nt / 8) + bid / 8 : bid;
  const int tk = tile % a.tilesK, tms = tile / a.tilesK;
  const int tm = tms % a.tilesM, sp = tms / a.tilesM;
  const int t0 = (int)((int64_t)a.T * sp / a.split), t1 = (int)((int64_t)a.T * (sp + 1) / a.split);
  const int64_t k0 = (int64_t)tk * kDK, K = a.K;
  const int mb0 = tm * 4 * J + wj * J;   // this wave's first row block

  const int g = lane >> 4, chunk = lane & 7, rsub = (lane >> 3) & 1;
  DOff o;
  {
    const uint32_t row = 8u * wave + 4u * rsub + g;
    const int64_t kc = k0 + 32 * chunk;
    const bool ok = kc < K;
    const uint32_t R = (uint32_t)row_bytes<KIND>(K), kcu = (uint32_t)kc;
    constexpr uint32_t cb = KIND == G_AFF2 ? 4 : KIND == G_AFF8 ? 1 : 2;   // columns per byte
    const uint32_t Ku = (uint32_t)K, gs = (uint32_t)a.gs;
    o.w = ok ? row * R + kcu / cb : kOff;
    o.h = ok ? row * (Ku / 4u) + kcu / 4u : kOff;
    o.p = 0;
    if constexpr (KIND == G_Q4K) {
      o.s = row * (Ku / 32u) + kcu / 32u;
      o.p = ok ? row * (Ku / 256u) * 4u + (kcu / 256u) * 4u : kOff;
    } else if constexpr (KIND == G_Q6K) {
      o.s = row * (Ku / 16u) + kcu / 16u;
      o.p = ok ? row * (Ku / 256u) * 2u + (kcu / 256u) * 2u : kOff;
    } else if constexpr (KIND == G_SYM4) {
      o.s = row * (Ku / gs) * 4u + (kcu / gs) * 4u;
    } else {
      o.s = row * (Ku / gs) * 2u + (kcu / gs) * 2u;
    }
    if (!ok) o.s = kOff;
  }
  // LDS byte of column e = 0 (e adds 256 (e >> 1) and turns slot bits)
  const uint32_t wl = 16u * chunk + 4u * g;
  // fragment base: slot bits of k-slice 0, subtile 0; entry x is slot ^ x
  uint32_t fa[8];
  {
    const uint32_t L = 64u * wi + ((lane & 31) >> 1);
    const uint32_t slot = (((lane & 1u) << 3) | (uint32_t)(lane >> 5)) ^
                          ((((uint32_t)lane >> 1) & 7u) ^ (4u * wi)) ^ ((((uint32_t)lane >> 3) & 1u) << 3);
#pragma unroll
    for (int x = 0; x < 8; ++x) fa[x] = L * 256u + (slot ^ (uint32_t)x) * 16u;
  }
  auto rd_a = [&](uint32_t buf, int s, int i) {
    return *reinterpret_cast<const half8_t*>(smem + fa[(2 * s) ^ i] + (buf * kDTile + 4096u * i));
  };
  uint32_t xo[J];
#pragma unroll
  for (int j = 0; j < J; ++j)
    xo[j] = mb0 + j < a.MB ? (uint32_t)(mb0 + j) * 1024u + 16u * (2u * (lane & 31) + (lane >> 5)) : kOff;
  const uint32_t xs = (uint32_t)a.MB * 1024u;   // one k-slice of 16
  auto ld_b = [&](int t, int s, int j) {
    const __amdgpu_buffer_rsrc_t r = rsrc(a.xf + (int64_t)(t < t1 ? t : t0) * 4 * xs, 4u * xs);
    // the slice as the scalar offset: the range check is on xo[j] alone, and
    // a row block inside a slice is inside all four
    return __builtin_bit_cast(half8_t,
                              __builtin_amdgcn_raw_buffer_load_b128(r, xo[j], (uint32_t)s * xs, 0));
  };
  const uint32_t magic = 0x64006400u, magic64 = 0x54005400u;   // 1024, 64
  // part b of a step's conversion: columns 2 b, 2 b + 1 of the lane's 8, at
  // line wl + b; wl is a multiple of 4, so b only turns slot bits
  uint32_t pa[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const uint32_t L = wl + b, hs = ((L & 7u) ^ ((L >> 4) & 7u)) | (((L >> 2) & 1u) << 3);
    pa[b] = L * 256u + 8u * rsub + (((uint32_t)wave) ^ hs) * 16u;
  }
  auto put = [&](auto B, uint32_t buf, const DTurned<KIND>& d) {
    constexpr int b = decltype(B)::value;
    uint2 v[2];
    dcols<KIND, b>(d, magic, magic64, v);
    *reinterpret_cast<uint2*>(smem + pa[b] + buf * kDTile) = v[0];
    *reinterpret_cast<uint2*>(smem + (pa[b] ^ 128u) + buf * kDTile) = v[1];   // slot ^ 8
  };

  float16_t acc[4][J];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  half8_t Bf[4][J];

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

  // One step: MFMAs on LDS buffer cur = (t - t0) & 1 and the D fragments in Bf
  // (reloaded slice by slice for step t + 1); conversion of step t + 1 into
  // the other buffer; weight loads of step t + 2.  Steps past the end load
  // nothing that is used (empty resources).
  auto kstep = [&](auto CUR, int t, DStage<KIND>& fre, DStage<KIND>& nxt) {
    constexpr uint32_t cur = decltype(CUR)::value;
    dload<KIND>(a, o, t + 2, fre);
    DTurned<KIND> d;
    // the matrix cores start on the last step's deferred products while this
    // step's first fragments come from LDS
    A[0] = rd_a(cur, 0, 0);
    A[1] = rd_a(cur, 0, 1);
    __builtin_amdgcn_sched_barrier(0);
    deferred();
    A[2] = rd_a(cur, 0, 2);
    A[3] = rd_a(cur, 0, 3);
#pragma unroll
    for (int j = 0; j < J; ++j) Bf[3][j] = ld_b(t, 3, j);
    static_for<4>([&](auto S) {
      constexpr int s = decltype(S)::value;
      static_for<(s < 3 ? 4 : 2)>([&](auto I) {
        constexpr int i = decltype(I)::value;
#pragma unroll
        for (int j = 0; j < J; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(A[i], Bf[s][j], acc[i][j], 0, 0, 0);
        if constexpr (s < 3) A[i] = rd_a(cur, s + 1, i);
      });
      if constexpr (s < 3) {
#pragma unroll
        for (int j = 0; j < J; ++j) Bf[s][j] = ld_b(t + 1, s, j);
      }
      // the conversion among the MFMAs of the first three slices
      if constexpr (s == 0) dturn<KIND, MBF16>(nxt, d);
      if constexpr (s == 1 || s == 2) {
        put(std::integral_constant<int, 2 * s - 2>{}, cur ^ 1u, d);
        put(std::integral_constant<int, 2 * s - 1>{}, cur ^ 1u, d);
      }
    });
    __syncthreads();
  };

  DStage<KIND> st0, st1;
  dload<KIND>(a, o, t0, st0);
  dload<KIND>(a, o, t0 + 1, st1);
#pragma unroll
  for (int s = 0; s < 3; ++s)
#pragma unroll
    for (int j = 0; j < J; ++j) Bf[s][j] = ld_b(t0, s, j);
  {
    DTurned<KIND> d;
    dturn<KIND, MBF16>(st0, d);
    static_for<4>([&](auto B) { put(B, 0u, d); });
  }
  __syncthreads();
  for (int t = t0; t < t1; t += 2) {
    kstep(std::integral_constant<uint32_t, 0>{}, t, st0, st1);
    if (t + 1 < t1) kstep(std::integral_constant<uint32_t, 1>{}, t + 1, st1, st0);
  }
  deferred();

  // ---- lane: rows k = 8 g + 4 (lane >> 5) + q of column m = lane & 31.
  // Through the wave's 8 KiB of LDS (the weight tiles are done with), so that
  // the stores are 256-byte pieces of rows of dx: 32 rows of 128 16-bit
  // columns, or of 64 fp32 ones in two passes; 16-byte chunk c of row r at
  // c ^ (r & 15).
  int el = lane;
  asm volatile("" : "+v"(el));   // keeps the epilogue's addresses after the loop
  unsigned char* lds = smem + 8192 * wave;
  const int r0 = el & 31, hh = el >> 5;
  const int64_t kw = k0 + wi * 128;
  static_for<J>([&](auto JJ) {
    constexpr int j = decltype(JJ)::value;
    const int64_t mb = (int64_t)(mb0 + j) * 32;
    if (a.part || a.dxdt == F32) {
      const int xe = !a.part && mb + r0 < a.M ? a.xe[mb + r0] : 0;   // shares stay scaled
      float* out = a.part ? a.part + (int64_t)sp * a.M * K : static_cast<float*>(a.dx);
      static_for<2>([&](auto H) {
        constexpr int h = decltype(H)::value;
        static_for<8>([&](auto G) {
          constexpr int i = 2 * h + decltype(G)::value / 4, gg = decltype(G)::value % 4;
          float4 v;
          v.x = ldexpf(acc[i][j][4 * gg], -xe);
          v.y = ldexpf(acc[i][j][4 * gg + 1], -xe);
          v.z = ldexpf(acc[i][j][4 * gg + 2], -xe);
          v.w = ldexpf(acc[i][j][4 * gg + 3], -xe);
          *reinterpret_cast<float4*>(lds + r0 * 256 + ((8 * (i & 1) + 2 * gg + hh) ^ (r0 & 15)) * 16) = v;
        });
        lds_turn();
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const int r = 4 * t + (el >> 4), c = el & 15;
          const float4 v = *reinterpret_cast<const float4*>(lds + r * 256 + (c ^ (r & 15)) * 16);
          const int64_t k = kw + 64 * h + 4 * c;
          if (mb + r < a.M && k < K) *reinterpret_cast<float4*>(out + (mb + r) * K + k) = v;
        }
        lds_turn();
      });
    } else {
      const int xe = mb + r0 < a.M ? a.xe[mb + r0] : 0;
      static_for<16>([&](auto G) {
        constexpr int i = decltype(G)::value / 4, gg = decltype(G)::value % 4;
        uint32_t h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float v = ldexpf(acc[i][j][4 * gg + q], -xe);
          h[q] = a.dxdt == BF16 ? f32_to_bf16_rne(v) : f32_to_f16_rne(v);
        }
        *reinterpret_cast<uint2*>(lds + r0 * 256 + ((4 * i + gg) ^ (r0 & 15)) * 16 + 8 * hh) =
            make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
      });
      lds_turn();
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int r = 4 * t + (el >> 4), c = el & 15;
        const uint4 v = *reinterpret_cast<const uint4*>(lds + r * 256 + (c ^ (r & 15)) * 16);
        const int64_t k = kw + 8 * c;
        if (mb + r < a.M && k < K)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dx) + (mb + r) * K + k) = v;
      }
      lds_turn();
    }
  });
}

// dx = 2^-e sum of the partial products, in order; 4 columns per thread.
__global__ void __launch_bounds__(256) k_dx_sum(const float4* __restrict__ part, int split,
                                                int64_t n4, uint32_t k4, const int* __restrict__ xe,
                                                void* __restrict__ dx, int dxdt) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  float4 v = part[i];
  for (int s = 1; s < split; ++s) {
    const float4 p = part[(int64_t)s * n4 + i];
    v.x += p.x; v.y += p.y; v.z += p.z; v.w += p.w;
  }
  const int e = -xe[i / k4];
  v = make_float4(ldexpf(v.x, e), ldexpf(v.y, e), ldexpf(v.z, e), ldexpf(v.w, e));
  if (dxdt == F32) {
    static_cast<float4*>(dx)[i] = v;
  } else {
    auto r = [dxdt](float f) { return dxdt == BF16 ? f32_to_bf16_rne(f) : f32_to_f16_rne(f); };
    static_cast<uint2*>(dx)[i] = make_uint2(r(v.x) | (r(v.y) << 16), r(v.z) | (r(v.w) << 16));
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct DxPlan {
  int J, split, tilesK, tilesM, MB, T1, T;
  size_t xf, xe, part;   // workspace bytes of each region (16-byte multiples)
};

DxPlan dx_plan(const Desc& d, int64_t M, bool gated) {
  DxPlan p;
  p.MB = (int)cdiv(M, 32);
  p.T1 = (int)cdiv(d.N, kDN);
  p.T = p.T1 * (gated ? 2 : 1);
  p.tilesK = (int)cdiv(d.K, kDK);
  // Rounds of blocks over 256 CUs, each block its share of the steps (1.6 us
  // with 256 rows of D, 1.1 with 128) and a few steps' worth of start and end;
  // more than one share adds the partial sums' traffic and a second kernel.
  double best = 0.;
  for (int J = M > 128 ? 2 : 1; J >= 1; --J) {
    const int64_t tiles = p.tilesK * cdiv(M, 128 * J);
    for (int s = 1; s <= 32 && s <= p.T; ++s) {
      if (s > 1 && tiles * s > 1024) break;
      double t = (double)cdiv(tiles * s, 256) * (double)(cdiv(p.T, s) + 4) * (J == 2 ? 1.6e-6 : 1.1e-6);
      if (s > 1) t += 3e-6 + (double)s * (double)M * (double)d.K * 8. / 4e12;
      if (best == 0. || t < best) {
        best = t;
        p.J = J;
        p.split = s;
      }
    }
  }
  p.tilesM = (int)cdiv(M, 128 * p.J);
  p.xf = (size_t)p.T * 4u * (size_t)p.MB * 1024u;
  p.xe = (size_t)p.MB * 128u;
  p.part = p.split > 1 ? (size_t)p.split * (size_t)M * (size_t)d.K * 4u : 0;
  return p;
}

typedef void (*DxFn)(DxK);
template <int KIND, bool MB>
DxFn dx_pick(int J) {
  return J == 2 ? k_dx<KIND, MB, 2> : k_dx<KIND, MB, 1>;
}

}  // namespace

size_t dx_workspace_bytes(const Desc& d, int64_t M, bool gated) {
  const DxPlan p = dx_plan(d, M, gated);
  return p.xf + p.xe + p.part;
}

hipError_t launch_dx(const Desc& d, const DxArgs& a, hipStream_t s) {
  const DxPlan p = dx_plan(d, a.M, a.gated);
  unsigned char* ws = static_cast<unsigned char*>(a.ws);
  int* xe = reinterpret_cast<int*>(ws + p.xf);
  StageArgs sa{static_cast<const uint16_t*>(a.dy), a.gq, a.gs, a.uq, a.us,
               static_cast<uint16_t*>(a.dg), static_cast<uint16_t*>(a.du), ws, xe, a.M, d.N};
  hipError_t e = launch_stage(sa, a.dydt, a.gated, a.act, false, s);
  if (e != hipSuccess) return e;
  DxK k{};
  k.w[0] = a.w;
  k.w[1] = a.w2;
  k.N = d.N;
  k.K = d.K;
  k.M = a.M;
  k.gs = d.gs;
  k.xf = ws;
  k.xe = xe;
  k.part = p.split > 1 ? reinterpret_cast<float*>(ws + p.xf + p.xe) : nullptr;
  k.dx = a.dx;
  k.dxdt = a.dxdt;
  k.T1 = p.T1;
  k.T = p.T;
  k.MB = p.MB;
  k.tilesK = p.tilesK;
  k.tilesM = p.tilesM;
  k.split = p.split;
  const bool mb = d.meta == BF16;
  DxFn fn = d.fmt == Q4K ? dx_pick<G_Q4K, false>(p.J)
          : d.fmt == Q6K ? dx_pick<G_Q6K, false>(p.J)
          : d.fmt == SYM4 ? dx_pick<G_SYM4, false>(p.J)
          : d.bits == 2 ? (mb ? dx_pick<G_AFF2, true>(p.J) : dx_pick<G_AFF2, false>(p.J))
          : d.bits == 4 ? (mb ? dx_pick<G_AFF4, true>(p.J) : dx_pick<G_AFF4, false>(p.J))
                        : (mb ? dx_pick<G_AFF8, true>(p.J) : dx_pick<G_AFF8, false>(p.J));
  hipLaunchKernelGGL(fn, dim3((unsigned)(p.tilesK * p.tilesM * p.split)), dim3(kThreads), 0, s, k);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (p.split > 1) {
    const int64_t n4 = a.M * d.K / 4;
    hipLaunchKernelGGL(k_dx_sum, dim3((unsigned)cdiv(n4, 256)), dim3(256), 0, s,
                       reinterpret_cast<const float4*>(k.part), p.split, n4, (uint32_t)(d.K / 4), xe,
                       a.dx, a.dxdt);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace qp
