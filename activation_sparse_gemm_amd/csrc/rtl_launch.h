// rtl_launch.h -- internal launchers behind the C ABI (host side).  Arguments are
// validated by the ABI layer before any of these is called.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace rtl {

constexpr int kDtF32 = 0;
constexpr int kDtBF16 = 1;

hipError_t launch_sparsify(int dt, int64_t M, int64_t K, const void* X, float eps, void* vals,
                           uint8_t* idx, float* s, hipStream_t stream);

// bf16 path.  Variants of the fused layer: the 2-of-4 selection in the GEMM's A-operand
// prologue, or in the pre-pass over X with the GEMM reading the compressed operand.
constexpr int kVariantAuto = 0, kVariantPrologue = 1, kVariantPrecompressed = 2, kVariantStreamK = 3;
int resolve_variant_bf16(int variant, int64_t M, int64_t N, int64_t K);
size_t fused_bf16_workspace(int64_t M, int64_t N, int64_t K, int64_t R);
// Stream-K GEMM (variant kVariantStreamK): the workspace it needs past the pre-pass
// outputs of the pre-compressed variant (placed at align256(ws_layout(M, K, R,
// true).total)); 0 when the shape runs whole tiles only.
size_t sk_workspace_bytes(int64_t M, int64_t N, int64_t K);
// Stamp for the flags by which one workgroup of a launch tells another that its partial
// results are in the workspace: a per-process random start, then one step per call, never
// 0, so flags left in a workspace by earlier launches do not match.
uint64_t next_launch_epoch();
hipError_t launch_prep_bf16(int variant, int64_t M, int64_t N, int64_t K, int64_t R, const void* X, const void* LB,
                            float eps, void* ws, uint8_t* dbg_idx, float* dbg_s, hipStream_t stream);
hipError_t launch_main_bf16(int variant, int64_t M, int64_t N, int64_t K, int64_t R, const void* X, const void* W,
                            const void* LA, float eps, void* Y, const void* ws, uint8_t* dbg_idx, float* dbg_s,
                            hipStream_t stream);
hipError_t launch_fused_bf16(int variant, int64_t M, int64_t N, int64_t K, int64_t R, const void* X, const void* W,
                             const void* LA, const void* LB, float eps, void* Y, void* ws, uint8_t* dbg_idx,
                             float* dbg_s, hipStream_t stream);
hipError_t launch_dense_bf16(int64_t M, int64_t N, int64_t K, const void* X, const void* W, void* Y,
                             hipStream_t stream);

// FP8 layer (E4M3 sparse product; selection, s and the low-rank branch as in bf16)
size_t fused_fp8_workspace(int64_t M, int64_t N, int64_t K, int64_t R);
hipError_t launch_quant_w_fp8(int64_t N, int64_t K, const void* W, uint8_t* Wq, float* sw, hipStream_t stream);
hipError_t launch_prep_fp8(int64_t M, int64_t K, int64_t R, const void* X, const void* LB, float eps, void* ws,
                           uint8_t* dbg_xq, float* dbg_sx, hipStream_t stream);
hipError_t launch_fused_fp8(int64_t M, int64_t N, int64_t K, int64_t R, const void* X, const uint8_t* Wq,
                            const float* sw, const void* LA, const void* LB, float eps, void* Y, void* ws,
                            uint8_t* dbg_xq, float* dbg_sx, hipStream_t stream);

// MLP pair (bf16): up layer, GELU, down layer.  Producer variant: the down layer's operand
// produced in the up GEMM's epilogue; consumer variant: the up layer stores its bf16 output
// and the down layer's pre-pass applies GELU as it loads it.
constexpr int kMlpAuto = 0, kMlpProducer = 1, kMlpConsumer = 2;
int resolve_mlp_variant(int variant);
size_t mlp_bf16_workspace(int64_t M, int64_t K, int64_t H, int64_t N, int64_t Ru, int64_t Rd);
hipError_t launch_mlp_bf16(int variant, int64_t M, int64_t K, int64_t H, int64_t N, int64_t Ru, int64_t Rd, const void* X,
                           const void* Wu, const void* LAu, const void* LBu, const void* Wd, const void* LAd,
                           const void* LBd, float eps, void* Y, void* ws, uint16_t* dbg_x, uint8_t* dbg_idx,
                           float* dbg_s, hipStream_t stream);
// pieces of launch_mlp_bf16
struct PairDown {
  uint8_t* cvals;
  uint8_t* cidx;
  float* tpart;    // [H / 128, Mp, Rd]
  double* npart;   // [H / 128, Mp, 2]
  const void* LB;  // L_B of the down layer [Rd, H]
  int64_t R;
  uint16_t* dbg_x;
  uint8_t* dbg_idx;
};
hipError_t launch_mlp_up_bf16(int64_t M, int64_t H, int64_t K, int64_t Ru, const void* Wu, const void* LAu,
                              float eps, const void* ws_up, const PairDown& d, hipStream_t stream);
hipError_t launch_prep_gelu_bf16(int64_t M, int64_t N, int64_t K, int64_t R, const void* X, const void* LB, float eps,
                                 void* ws, uint16_t* dbg_x, uint8_t* dbg_idx, float* dbg_s, hipStream_t stream);
hipError_t launch_split_reduce_bf16(int64_t M, int64_t R, int ks, const float* tpart, const double* npart, float eps,
                                    void* T, float* s, float* dbg_s, hipStream_t stream);

// Rotary embedding over several axes and per-head norms of queries and keys (qk_rope.h).
struct StridedHeads {
  const void* p;      // [M, H, D], D contiguous
  int64_t row, head;  // strides in elements
};
struct RopeCall {
  int dt;
  bool norm, halves, inverse;
  int64_t M, H[2], D;      // heads of the two tensors (queries, keys); H[1] may be 0
  StridedHeads x[2], y[2], dx[2];  // gradient: y holds dy, dx the outputs; else y the outputs
  const void* w[2];        // norm weights [D] or null
  float eps;
  const float* pos;        // [M, axes]
  int axes;
  const int32_t* dims;     // host: even widths of the axes
  double theta;
};
hipError_t launch_rope(const RopeCall& c, hipStream_t stream);
size_t qk_back_workspace(int64_t D);
hipError_t launch_qk_back(const RopeCall& c, float* dqw, float* dkw, void* ws, hipStream_t stream);

// Gated feed-forward block (glu_bf16.h): Y = act(X Wg^T) (X Wu^T), and its gradient.
constexpr int kActSilu = 0, kActGelu = 1;
hipError_t launch_glu_bf16(int act, int64_t M, int64_t K, int64_t H, const void* X, const void* Wg, const void* Wu,
                           void* Y, void* G, void* U, hipStream_t stream);
size_t glu_back_workspace(int64_t M, int64_t K, int64_t H);
hipError_t launch_glu_back_bf16(int act, int64_t M, int64_t K, int64_t H, const void* X, const void* Wg,
                                const void* Wu, const void* G, const void* U, const void* dY, void* dX, void* dWg,
                                void* dWu, void* ws, hipStream_t stream);

// Layer norm with weights and per-group scale and shift, and its gradient (layer_norm.h).
struct RowsView {
  const void* p;  // rows of D contiguous elements
  int64_t row;    // stride in elements
};
struct NormCall {
  int dt;
  int64_t M, D, G;          // G: groups, 0 without scale and shift
  RowsView x, y, dy;        // gradient: dy, and y is dx
  RowsView scale, shift;    // [G, D] or null
  const void *w, *b;        // [D] or null
  const int32_t* groups;    // [G + 1] or null
  float eps;
  const float* stats;       // [M, 2]: forward writes them (null: not wanted), the gradient reads them
  bool clear;               // y's rows of no group become zeros, else they stay
};
constexpr int64_t kNormMaxD = 32768;       // bf16 rows in 16-byte pieces (fp32: half)
constexpr int64_t kNormMaxDNarrow = 8192;  // rows taken by the element
bool norm_is_wide(const NormCall& c);
bool norm_fits(int dt, int64_t D, bool wide);
hipError_t launch_norm(const NormCall& c, hipStream_t stream);
size_t norm_back_workspace(int64_t M, int64_t D, int64_t G);
hipError_t launch_norm_back(const NormCall& c, float* dw, float* db, float* dscale, float* dshift, void* ws,
                            hipStream_t stream);

// Low-rank adapters of many requests and their gradient (adapters.h).
struct AdapterCall {
  int64_t M, N, K, R, A;
  const void* x;
  int64_t x_row;
  const void *LA, *LB;  // [A, N, R], [A, R, K]
  const void* plan;
  const float* alpha;   // [A] or null
};
size_t adapters_plan_bytes(int64_t M, int64_t A);
hipError_t launch_adapters_plan(const int32_t* ids, int64_t M, int64_t A, void* plan, hipStream_t stream);
size_t adapters_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A);
hipError_t launch_adapters(const AdapterCall& c, const void* y0, int64_t y0_row, void* y, int64_t y_row, float* t, void* ws,
                           hipStream_t stream);
size_t adapters_back_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A);
hipError_t launch_adapters_back(const AdapterCall& c, const float* t, const void* dy, int64_t dy_row, const void* dx0,
                                int64_t dx0_row, void* dx, int64_t dx_row, float* dla, float* dlb, void* ws,
                                hipStream_t stream);

// AdamW over many tensors (adamw.h).
struct AdamTensor {
  void* p;               // parameters: fp32, or bf16 beside `master`
  const void* g;         // gradients
  float* master;         // fp32 copies of bf16 parameters, else null
  void *m, *v;           // states: fp32, or E4M3 codes of m and of sqrt(v)
  float *m_scale, *v_scale;  // one for 256 codes
  int64_t n;
};
struct AdamRates {
  double beta1, beta2;
  const int64_t* step_at;   // device: the step's number, null: m_up and u_up hold its corrections
  const float* lr_at;       // device: the learning rate, null: lr
  const float* grad_scale;  // device: a factor of the gradients, or null
  float lr, c1, b2, c2;     // c1 = 1 - beta1, b2 = beta2, c2 = 1 - beta2
  float m_up, u_up;         // 1 / (1 - beta1^t), 1 / sqrt(1 - beta2^t)
  float eps, decay;
};
constexpr int64_t kAdamMaxN = (int64_t)1 << 35;
constexpr uint32_t kAdamMaxBlocks = 1u << 23;  // of 256 threads: below 2^32
hipError_t launch_adamw(bool p_bf16, bool g_bf16, bool eight, const AdamTensor* t, int64_t count, const AdamRates& r,
                        hipStream_t stream);

// Allocation-free workspace: the per-device scratch array (noalloc.hip).  `mismatch` is set
// when `stream` does not belong to the current device (no address is resolved then).
size_t noalloc_scratch_bytes();
hipError_t noalloc_scratch(hipStream_t stream, void** out, int* mismatch);

// fp32 path
size_t fused_f32_workspace(int64_t M, int64_t N, int64_t K, int64_t R);
hipError_t launch_fused_f32(int64_t M, int64_t N, int64_t K, int64_t R, const float* X,
                            const float* W, const float* LA, const float* LB, float eps, float* Y,
                            void* ws, uint8_t* dbg_idx, float* dbg_s, hipStream_t stream);
hipError_t launch_dense_f32(int64_t M, int64_t N, int64_t K, const float* X, const float* W,
                            float* Y, hipStream_t stream);

}  // namespace rtl
