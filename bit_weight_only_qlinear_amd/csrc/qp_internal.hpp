// Internal declarations shared by the host API and the kernel translation
// units of libqlinear (not part of the public ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qp {

enum Fmt : int { AFFINE = 0, Q4K = 1, Q6K = 2, SYM4 = 3, MXFP4 = 4 };
enum DType : int { F16 = 0, BF16 = 1, F32 = 2 };
enum Act : int { ACT_SILU = 0, ACT_GELU_TANH = 1 };
constexpr int kCkptGroup = 64;   // columns per scale of an 8-bit checkpoint

// Validated, host-side copy of the descriptor.
struct Desc {
  int fmt, bits, gs, sb, meta;
  int64_t N, K;
};

struct Bufs {
  const void* qweight;
  const void* qweight_hi;
  const void* scales;
  const void* zeros;
  const void* steps;
};

// Launchers (each returns the hipError_t of its launch).
hipError_t launch_quantize(const Desc& d, const float* W, void* qweight,
                           void* qweight_hi, void* scales, void* zeros,
                           void* steps, hipStream_t s);
hipError_t launch_quantize_hqq(const Desc& d, const float* W, void* qweight, void* scales,
                               void* zeros, int iters, float p, float beta, float kappa,
                               hipStream_t s);
hipError_t launch_unpack(const Desc& d, const Bufs& b, void* codes,
                         hipStream_t s);
hipError_t launch_pack(const Desc& d, const void* codes, void* qweight,
                       void* qweight_hi, hipStream_t s);
hipError_t launch_dequant(const Desc& d, const Bufs& b, void* out, int out_dt,
                          hipStream_t s);
// True when the qGEMV kernel's register plan covers this K (every lane's
// slice of the activations must fit in registers).
bool gemv_supported(const Desc& d);
// `bytes` are the five buffer sizes of the layout (each < 2 GiB, checked
// by the caller): the kernel addresses them through buffer resources.
hipError_t launch_gemv(const Desc& d, const void* x, int xdt, int64_t M,
                       const Bufs& b, const void* bias, void* y, int ydt,
                       const size_t bytes[5], hipStream_t s);
// Exact-code MFMA qGEMV, activation rows in tiles of 16 (any M): K must be
// a multiple of 128.
bool skinny_supported(const Desc& d);
hipError_t launch_skinny(const Desc& d, const void* x, int xdt, int64_t M,
                         const Bufs& b, const void* bias, void* y, int ydt,
                         const size_t bytes[5], hipStream_t s);
// Workspace bytes of the qGEMM with 224-row tiles and staged activations (M
// rounded up to 16 rows of K fp16); 0 where 256-row tiles are as good or
// the shape is past its 32-bit indexing.
size_t gemm_workspace_bytes(const Desc& d, int64_t M);
// ws: null (256-row tiles), or a device buffer of gemm_workspace_bytes(d, M)
// > 0 bytes (a staging kernel, then the 224-row-tile kernel, same stream).
hipError_t launch_gemm(const Desc& d, const void* x, int xdt, int64_t M,
                       const Bufs& b, const void* bias, void* y, int ydt,
                       void* ws, hipStream_t s);

// Plain per-group metadata (fp32 scales, Q4K zero points) into the nested
// Q4K / Q6K metadata buffers; *bad (optional, device) flags invalid inputs.
hipError_t launch_encode_nested(const Desc& d, const float* sv, const float* zv, void* scales,
                                void* zeros, void* steps, int* bad, hipStream_t st);
// Per-token symmetric int8 activations: q [M, K] int8, s [M] fp32.
hipError_t launch_quant_act(const void* x, int xdt, int64_t M, int64_t K, void* q, float* s,
                            hipStream_t st);
// a8w4 forward (SYM4 per output channel, K % 128 == 0, every buffer < 2 GiB).
hipError_t launch_a8w4(const Desc& d, const void* xq, const float* xs, int64_t M, const Bufs& b,
                       const float* bias, void* y, int ydt, hipStream_t s);

// RMS norm with the residual's addition (norm.hip).  y, or yq and ys.
hipError_t launch_norm(const void* x, const void* r, int dt, int64_t M, int64_t K, const void* w,
                       float eps, void* s, void* y, void* yq, float* ys, float* rstd,
                       hipStream_t st);
// Its backward; s, or its checkpoint (sq, ss).  part: norm_bwd_parts(M) * K
// floats where dw is asked for.
int norm_bwd_parts(int64_t M);
hipError_t launch_norm_bwd(const void* dy, const void* s, const void* sq, const float* ss, int dt,
                           int64_t M, int64_t K, const void* w, const float* rstd,
                           const void* ds_in, void* ds, float* dw, float* part, hipStream_t st);
// 8-bit checkpoints: int8 codes [M, K], fp32 scales [M, ceil(K / 64)].
hipError_t launch_checkpoint(const void* x, int dt, int64_t M, int64_t K, void* q, float* s,
                             hipStream_t st);
hipError_t launch_checkpoint_restore(const void* q, const float* s, int64_t M, int64_t K, void* x,
                                     int dt, hipStream_t st);

// Gated pair of projections: h = act(x Wg^T + bg) * (x Wu^T + bu), both
// layers of descriptor d.  gq .. us: 8-bit checkpoints of the two
// pre-activations, or all null.
struct GatedArgs {
  const void* x;
  int xdt, hdt, act;
  int64_t M;
  Bufs gate, up;
  const void* bias_g;
  const void* bias_u;
  void* h;
  int8_t* gq;
  float* gs;
  int8_t* uq;
  float* us;
};
// The forms of the gated pair: fp16-rounded weights on MFMA with a workspace
// (gated.hip); exact codes on MFMA, K % 128 == 0, 16 rows at most and no
// checkpoints (skinny.hip).
size_t gated_workspace_bytes(const Desc& d, int64_t M);
hipError_t launch_gated(const Desc& d, const GatedArgs& a, void* ws, hipStream_t s);
// Exact codes, streamed: one activation row, or two in some formats, and no
// checkpoints (gemv.hip).
bool gated_gemv_supported(const Desc& d, int64_t M);
hipError_t launch_gated_gemv(const Desc& d, const GatedArgs& a, const size_t bytes[5],
                             hipStream_t s);
hipError_t launch_gated_skinny(const Desc& d, const GatedArgs& a, const size_t bytes[5],
                               hipStream_t s);

// fp16 fragments of a product's 16-bit operand d [M, N] (stage.hip): row
// exponents into xe [ceil(M / 32) * 32], fragments into xf (ceil(N / 64) *
// ceil(M / 32) * 4 KiB, twice that for the gated pair's [dg | du]).
struct StageArgs {
  const uint16_t* d;
  const int8_t* gq;   // gated: checkpoints of the pre-activations
  const float* gs;
  const int8_t* uq;
  const float* us;
  uint16_t* dg;       // gated: the gradients themselves, or null
  uint16_t* du;
  void* xf;
  int* xe;
  int64_t M, N;
  // MXFP4 weights [N, 32 tops_cols] whose rows the product sums over: the largest
  // scale byte below 255 of each 32 columns in `tops_parts` runs of rows, into tops
  // (at tops_at); both layers together for the gated pair.  Or parts 0.
  const uint8_t* scales[2];
  uint8_t* tops;
  int tops_parts;
  int64_t tops_cols;
};
// Eight neighbouring columns' bytes of all runs lie together: a product tile's.
__host__ __device__ inline int64_t tops_at(int64_t col, int part, int parts) {
  return ((col >> 3) * parts + part) * 8 + (col & 7);
}
hipError_t launch_stage(const StageArgs& r, int dt, bool gated, int act, bool perm, hipStream_t s);

// Input gradients.  dx [M, K] = dy [M, N] W, or with `gated` the sum of two
// such products over dg = dh u act'(g) and du = dh act(g).
struct DxArgs {
  const void* dy;         // dy, or dh
  int dydt, dxdt, act;
  int64_t M;
  Bufs w, w2;             // the layer; gate and up layers
  bool gated;
  const int8_t* gq;       // checkpoints of the pre-activations (gated)
  const float* gs;
  const int8_t* uq;
  const float* us;
  void* dg;               // [M, N] of dy's type, or null (gated)
  void* du;
  void* dx;
  void* ws;
};
size_t dx_workspace_bytes(const Desc& d, int64_t M, bool gated);
hipError_t launch_dx(const Desc& d, const DxArgs& a, hipStream_t s);

// Few activation rows (few.hip): MXFP4 layers and gated pairs without
// checkpoints, rows in tiles of up to 16 (any M, any K % 32 == 0).
hipError_t launch_few(const Desc& d, const void* x, int xdt, int64_t M, const Bufs& b,
                      const void* bias, void* y, int ydt, hipStream_t s);
hipError_t launch_few_gated(const Desc& d, const GatedArgs& a, hipStream_t s);

// MXFP4 layers and more than a few rows, on exact codes too (mx_rows.hip).
bool mx_rows_fits(const Desc& d);
hipError_t launch_mx_rows(const Desc& d, const void* x, int xdt, int64_t M, const Bufs& b,
                          const void* bias, void* y, int ydt, hipStream_t s);

// A mixture-of-experts layer for few tokens (moe.hip): experts stacked along
// the rows of `up` (E * inner rows, gate alike) and `down` (E * K rows).
struct MoeArgs {
  const void* x;
  int xdt, ydt, act, score, norm, E, topk;
  int64_t M;
  const void* router;      // [E, K] of xdt, or null: ids and weights are given
  Bufs gate, up, down;
  int* ids;                // [M, topk]
  float* weights;
  void* y;
  void* ws;
};
bool few_fits(const Desc& d);   // rows short enough for the few-row kernels
bool moe_format(const Desc& d);
int moe_max_tokens();
int moe_max_experts();
int moe_max_topk();
size_t moe_workspace_bytes(int64_t M, int topk, int E, int64_t K, int64_t inner);
hipError_t launch_moe(const Desc& up, const Desc& down, const MoeArgs& m, hipStream_t s);

// MXFP4 rows from fp16, bf16 or fp32 ones, and back; products of two MXFP4
// operands on the scaled matrix cores, for few rows of X and any K (mx_few.hip) or
// in tiles and K % 128 == 0 (mx.hip).
hipError_t launch_mx_dequant(const Desc& d, const Bufs& b, void* out, int odt, hipStream_t st);
hipError_t launch_mx_quant(const void* x, int xdt, int64_t M, int64_t K, void* q, void* s,
                           hipStream_t st);
bool mx_few_fits(const Desc& d, int64_t M);   // rows short enough for launch_mx_few
hipError_t launch_mx_few(const Desc& d, const void* xq, const void* xs, int64_t M, const Bufs& b,
                         const float* bias, void* y, int ydt, hipStream_t s);
int64_t mx_tiles(const Desc& d, int64_t M);      // blocks of launch_mx_mx
hipError_t launch_mx_mx(const Desc& d, const void* xq, const void* xs, int64_t M, const Bufs& b,
                        const float* bias, void* y, int ydt, hipStream_t s);

// Static device scratch of the allocation-free forward (noalloc.hip): its
// size, and its address on the current device (looked up once per device).
size_t static_scratch_bytes();
hipError_t static_scratch(void** out);

}  // namespace qp
