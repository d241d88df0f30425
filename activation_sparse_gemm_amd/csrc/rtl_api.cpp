// rtl_api.cpp -- the C ABI declared in include/rtl.h: synchronous validation, then
// dispatch to the gfx950 kernels on the caller's stream.  No exception crosses the ABI,
// and a call that fails validation launches nothing and writes no output.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/rtl.h"
#include "rtl_launch.h"

namespace {

thread_local char g_err[512] = "";

rtl_status fail(rtl_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
rtl_status fail(rtl_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return st;
}

rtl_status ok() {
  g_err[0] = '\0';
  return RTL_OK;
}

size_t elem_size(rtl_dtype dt) { return dt == RTL_BF16 ? 2 : 4; }

bool misaligned(const void* p) { return ((uintptr_t)p & 15u) != 0; }

// [a, a+na) and [b, b+nb) overlap (byte ranges; empty ranges never overlap).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + nb && y < x + na;
}

rtl_status check_dtype(rtl_dtype dt) {
  if (dt != RTL_F32 && dt != RTL_BF16) return fail(RTL_ERR_UNSUPPORTED, "unsupported dtype %d", (int)dt);
  return RTL_OK;
}

// eps guards the division by ||X~||; it is kept in [0, 1] so that s of any nonzero row whose
// output is in the normal floating-point range is itself a normal fp32 number.
rtl_status check_eps(float eps) {
  if (!(eps >= 0.f && eps <= 1.f)) return fail(RTL_ERR_ARG, "eps must lie in [0, 1] (got %g)", (double)eps);
  return RTL_OK;
}

rtl_status hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(RTL_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

}  // namespace

extern "C" {

int rtl_version(void) { return 100; }

const char* rtl_last_error(void) { return g_err; }

const char* rtl_status_string(rtl_status st) {
  switch (st) {
    case RTL_OK: return "RTL_OK";
    case RTL_ERR_NULL: return "RTL_ERR_NULL: a required pointer is NULL";
    case RTL_ERR_SHAPE: return "RTL_ERR_SHAPE: invalid shape";
    case RTL_ERR_ALIGN: return "RTL_ERR_ALIGN: pointer not 16-byte aligned";
    case RTL_ERR_UNSUPPORTED: return "RTL_ERR_UNSUPPORTED: unsupported tie rule, dtype or shape";
    case RTL_ERR_ARG: return "RTL_ERR_ARG: invalid argument";
    case RTL_ERR_WORKSPACE: return "RTL_ERR_WORKSPACE: workspace missing or too small";
    case RTL_ERR_HIP: return "RTL_ERR_HIP: HIP runtime error";
  }
  return "unknown rtl_status";
}

}  // extern "C"

namespace {
// Extents the kernels reach with 32-bit offsets from the start of a tile or row block: K up
// to kMaxK, and fewer than 2^31 output tiles of 256 x 128 (M and N each below 2^31).
constexpr int64_t kMaxK = (int64_t)1 << 22;
rtl_status check_extent(int64_t M, int64_t N, int64_t K) {
  if (K > kMaxK) return fail(RTL_ERR_SHAPE, "K must be at most %lld (K=%lld)", (long long)kMaxK, (long long)K);
  if (M > INT32_MAX || N > INT32_MAX || ((M + 255) / 256) * ((N + 127) / 128) > INT32_MAX)
    return fail(RTL_ERR_SHAPE, "M x N is too large (M=%lld N=%lld)", (long long)M, (long long)N);
  return RTL_OK;
}
}  // namespace

extern "C" {

rtl_status rtl_sparsify(rtl_dtype dt, int64_t M, int64_t K, const void* X, rtl_tie_rule tie, float eps,
                        void* vals, uint8_t* idx, float* s, void* stream) {
  rtl_status st;
  if ((st = check_dtype(dt)) != RTL_OK) return st;
  if (tie != RTL_TIE_LOWER_INDEX) return fail(RTL_ERR_UNSUPPORTED, "unsupported tie rule %d", (int)tie);
  if (M <= 0 || K <= 0 || K % 4 != 0) return fail(RTL_ERR_SHAPE, "need M > 0, K > 0, K %% 4 == 0 (M=%lld K=%lld)",
                                                  (long long)M, (long long)K);
  if ((st = check_extent(M, 1, K)) != RTL_OK) return st;
  if (!X || !vals || !idx || !s) return fail(RTL_ERR_NULL, "X, vals, idx and s are required");
  if (misaligned(X) || misaligned(vals) || misaligned(idx) || misaligned(s))
    return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if ((st = check_eps(eps)) != RTL_OK) return st;
  const size_t es = elem_size(dt);
  const size_t xb = (size_t)M * K * es, vb = (size_t)M * (K / 2) * es, ib = (size_t)M * (K / 4), sb = (size_t)M * 4;
  if (overlap(vals, vb, X, xb) || overlap(idx, ib, X, xb) || overlap(s, sb, X, xb) || overlap(vals, vb, idx, ib) ||
      overlap(vals, vb, s, sb) || overlap(idx, ib, s, sb))
    return fail(RTL_ERR_ARG, "outputs overlap each other or the input");
  return hip_status(rtl::launch_sparsify(dt == RTL_BF16 ? rtl::kDtBF16 : rtl::kDtF32, M, K, X, eps, vals, idx, s,
                                         (hipStream_t)stream),
                    "rtl_sparsify launch");
}

size_t rtl_linear_fused_workspace_bytes(rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R) {
  if (M <= 0 || N <= 0 || K <= 0 || R < 0) return 0;
  if (dt == RTL_BF16) return rtl::fused_bf16_workspace(M, N, K, R);
  if (dt == RTL_F32) return rtl::fused_f32_workspace(M, N, K, R);
  return 0;
}

}  // extern "C"

namespace {

enum Stage { kWhole = 0, kPrep = 1, kMain = 2 };

// Validation shared by rtl_linear_fused{,_ex,_prep,_main,_noalloc}.  Pointers a stage does
// not use are ignored (prep: W, LA, Y; main: LB).  `own_ws`: the library's scratch array
// is the workspace (the caller passes none), checked against its size instead.
rtl_status check_fused(Stage stage, rtl_variant variant, rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R,
                       const void* X, const void* W, const void* LA, const void* LB, rtl_tie_rule tie, float eps,
                       const void* Y, const void* ws, size_t ws_bytes, const void* dbg_idx, const void* dbg_s,
                       bool own_ws = false) {
  rtl_status st;
  if ((st = check_dtype(dt)) != RTL_OK) return st;
  if (variant != RTL_VARIANT_AUTO && variant != RTL_VARIANT_PROLOGUE && variant != RTL_VARIANT_PRECOMPRESSED &&
      variant != RTL_VARIANT_STREAM_K)
    return fail(RTL_ERR_UNSUPPORTED, "unsupported variant %d", (int)variant);
  if (stage != kWhole && dt != RTL_BF16) return fail(RTL_ERR_UNSUPPORTED, "the split launches are bf16 only");
  if (tie != RTL_TIE_LOWER_INDEX) return fail(RTL_ERR_UNSUPPORTED, "unsupported tie rule %d", (int)tie);
  if (M <= 0 || N <= 0 || K <= 0 || K % 4 != 0 || R < 0)
    return fail(RTL_ERR_SHAPE, "need M, N, K > 0, K %% 4 == 0, R >= 0 (M=%lld N=%lld K=%lld R=%lld)", (long long)M,
                (long long)N, (long long)K, (long long)R);
  if ((st = check_extent(M, N, K)) != RTL_OK) return st;
  const bool uses_w = stage != kPrep, uses_lb = stage != kMain;
  if (!X || (uses_w && (!W || !Y)) || (R > 0 && ((uses_w && !LA) || (uses_lb && !LB))))
    return fail(RTL_ERR_NULL, "X, W, Y (and LA, LB when R > 0) are required");
  if (misaligned(X) || (uses_w && (misaligned(W) || misaligned(Y) || misaligned(LA))) || (uses_lb && misaligned(LB)) ||
      misaligned(ws) || misaligned(dbg_idx) || misaligned(dbg_s))
    return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if (dt == RTL_BF16) {
    if (K % 64 != 0) return fail(RTL_ERR_UNSUPPORTED, "bf16 path needs K %% 64 == 0 (K=%lld)", (long long)K);
    if (R % 32 != 0 || R > 128)
      return fail(RTL_ERR_UNSUPPORTED, "bf16 path needs R %% 32 == 0 and R <= 128 (R=%lld)", (long long)R);
  } else if (R > 128) {
    return fail(RTL_ERR_UNSUPPORTED, "fp32 path needs R <= 128 (R=%lld)", (long long)R);
  }
  if ((st = check_eps(eps)) != RTL_OK) return st;
  const size_t es = elem_size(dt);
  const size_t xb = (size_t)M * K * es, wb = (size_t)N * K * es, lab = (size_t)N * R * es, lbb = (size_t)R * K * es;
  const size_t yb = (size_t)M * N * es, ib = (size_t)M * (K / 4), sb = (size_t)M * 4;
  const size_t need = rtl_linear_fused_workspace_bytes(dt, M, N, K, R);
  const void* ins[4] = {X, uses_w ? W : nullptr, (R > 0 && uses_w) ? LA : nullptr, (R > 0 && uses_lb) ? LB : nullptr};
  const size_t inb[4] = {xb, wb, lab, lbb};
  const void* Yc = uses_w ? Y : nullptr;
  for (int i = 0; i < 4; i++) {
    if (overlap(Yc, yb, ins[i], inb[i]) || overlap(dbg_idx, ib, ins[i], inb[i]) || overlap(dbg_s, sb, ins[i], inb[i]) ||
        overlap(ws, need, ins[i], inb[i]))
      return fail(RTL_ERR_ARG, "an output or the workspace overlaps an input");
  }
  if (overlap(Yc, yb, dbg_idx, ib) || overlap(Yc, yb, dbg_s, sb) || overlap(dbg_idx, ib, dbg_s, sb) ||
      overlap(ws, need, Yc, yb) || overlap(ws, need, dbg_idx, ib) || overlap(ws, need, dbg_s, sb))
    return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  if (own_ws) {
    if (need > rtl::noalloc_scratch_bytes())
      return fail(RTL_ERR_WORKSPACE,
                  "this shape needs %zu bytes of workspace; the allocation-free entry point has %zu (use "
                  "rtl_linear_fused with a caller-owned workspace)",
                  need, rtl::noalloc_scratch_bytes());
    return RTL_OK;
  }
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(RTL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, ws ? ws_bytes : (size_t)0);
  return RTL_OK;
}

}  // namespace

extern "C" {

rtl_status rtl_linear_fused_ex(rtl_variant variant, rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R,
                               const void* X, const void* W, const void* LA, const void* LB, rtl_tie_rule tie,
                               float eps, void* Y, void* workspace, size_t ws_bytes, uint8_t* dbg_idx, float* dbg_s,
                               void* stream) {
  rtl_status st = check_fused(kWhole, variant, dt, M, N, K, R, X, W, LA, LB, tie, eps, Y, workspace, ws_bytes,
                              dbg_idx, dbg_s);
  if (st != RTL_OK) return st;
  hipError_t e;
  if (dt == RTL_BF16)
    e = rtl::launch_fused_bf16((int)variant, M, N, K, R, X, W, LA, LB, eps, Y, workspace, dbg_idx, dbg_s,
                               (hipStream_t)stream);
  else
    e = rtl::launch_fused_f32(M, N, K, R, (const float*)X, (const float*)W, (const float*)LA, (const float*)LB, eps,
                              (float*)Y, workspace, dbg_idx, dbg_s, (hipStream_t)stream);
  return hip_status(e, "rtl_linear_fused launch");
}

rtl_status rtl_linear_fused(rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R, const void* X, const void* W,
                            const void* LA, const void* LB, rtl_tie_rule tie, float eps, void* Y, void* workspace,
                            size_t ws_bytes, uint8_t* dbg_idx, float* dbg_s, void* stream) {
  return rtl_linear_fused_ex(RTL_VARIANT_AUTO, dt, M, N, K, R, X, W, LA, LB, tie, eps, Y, workspace, ws_bytes, dbg_idx,
                             dbg_s, stream);
}

rtl_status rtl_linear_fused_noalloc(rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R, const void* X,
                                    const void* W, const void* LA, const void* LB, rtl_tie_rule tie, float eps,
                                    void* Y, uint8_t* dbg_idx, float* dbg_s, void* stream) {
  rtl_status st = check_fused(kWhole, RTL_VARIANT_AUTO, dt, M, N, K, R, X, W, LA, LB, tie, eps, Y, nullptr, 0,
                              dbg_idx, dbg_s, true);
  if (st != RTL_OK) return st;
  void* ws = nullptr;
  int mismatch = 0;
  hipError_t e = rtl::noalloc_scratch((hipStream_t)stream, &ws, &mismatch);
  if (e != hipSuccess) return hip_status(e, "rtl_linear_fused_noalloc scratch address");
  if (mismatch) return fail(RTL_ERR_ARG, "the stream must belong to the current device");
  if (dt == RTL_BF16)
    e = rtl::launch_fused_bf16(RTL_VARIANT_AUTO, M, N, K, R, X, W, LA, LB, eps, Y, ws, dbg_idx, dbg_s,
                               (hipStream_t)stream);
  else
    e = rtl::launch_fused_f32(M, N, K, R, (const float*)X, (const float*)W, (const float*)LA, (const float*)LB, eps,
                              (float*)Y, ws, dbg_idx, dbg_s, (hipStream_t)stream);
  return hip_status(e, "rtl_linear_fused_noalloc launch");
}

rtl_status rtl_linear_fused_prep(rtl_variant variant, rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R,
                                 const void* X, const void* LB, rtl_tie_rule tie, float eps, void* workspace,
                                 size_t ws_bytes, uint8_t* dbg_idx, float* dbg_s, void* stream) {
  rtl_status st = check_fused(kPrep, variant, dt, M, N, K, R, X, nullptr, nullptr, LB, tie, eps, nullptr, workspace,
                              ws_bytes, dbg_idx, dbg_s);
  if (st != RTL_OK) return st;
  return hip_status(rtl::launch_prep_bf16((int)variant, M, N, K, R, X, LB, eps, workspace, dbg_idx, dbg_s,
                                          (hipStream_t)stream),
                    "rtl_linear_fused_prep launch");
}

rtl_status rtl_linear_fused_main(rtl_variant variant, rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R,
                                 const void* X, const void* W, const void* LA, rtl_tie_rule tie, float eps, void* Y,
                                 const void* workspace, size_t ws_bytes, uint8_t* dbg_idx, float* dbg_s,
                                 void* stream) {
  rtl_status st = check_fused(kMain, variant, dt, M, N, K, R, X, W, LA, nullptr, tie, eps, Y, workspace, ws_bytes,
                              dbg_idx, dbg_s);
  if (st != RTL_OK) return st;
  return hip_status(rtl::launch_main_bf16((int)variant, M, N, K, R, X, W, LA, eps, Y, workspace, dbg_idx, dbg_s,
                                          (hipStream_t)stream),
                    "rtl_linear_fused_main launch");
}

size_t rtl_mlp_fused_workspace_bytes(int64_t M, int64_t K, int64_t H, int64_t N, int64_t Ru, int64_t Rd) {
  if (M <= 0 || K <= 0 || H <= 0 || N <= 0 || Ru < 0 || Rd < 0) return 0;
  return rtl::mlp_bf16_workspace(M, K, H, N, Ru, Rd);
}

rtl_status rtl_mlp_fused(rtl_mlp_variant variant, rtl_dtype dt, int64_t M, int64_t K, int64_t H, int64_t N, int64_t Ru, int64_t Rd,
                         const void* X, const void* Wu, const void* LAu, const void* LBu, const void* Wd,
                         const void* LAd, const void* LBd, rtl_tie_rule tie, float eps, void* Y, void* workspace,
                         size_t ws_bytes, void* dbg_xd, uint8_t* dbg_idx, float* dbg_s, void* stream) {
  rtl_status st;
  if ((st = check_dtype(dt)) != RTL_OK) return st;
  if (dt != RTL_BF16) return fail(RTL_ERR_UNSUPPORTED, "the MLP pair is bf16 only");
  if (variant != RTL_MLP_AUTO && variant != RTL_MLP_PRODUCER && variant != RTL_MLP_CONSUMER)
    return fail(RTL_ERR_UNSUPPORTED, "unsupported MLP variant %d", (int)variant);
  if (tie != RTL_TIE_LOWER_INDEX) return fail(RTL_ERR_UNSUPPORTED, "unsupported tie rule %d", (int)tie);
  if (M <= 0 || K <= 0 || H <= 0 || N <= 0 || Ru < 0 || Rd < 0)
    return fail(RTL_ERR_SHAPE, "need M, K, H, N > 0 and ranks >= 0 (M=%lld K=%lld H=%lld N=%lld)", (long long)M,
                (long long)K, (long long)H, (long long)N);
  if ((st = check_extent(M, H, K)) != RTL_OK || (st = check_extent(M, N, H)) != RTL_OK) return st;
  if (K % 64 != 0 || H % 128 != 0 || Ru % 32 != 0 || Ru > 128 || (Rd != 0 && Rd != 32 && Rd != 64))
    return fail(RTL_ERR_UNSUPPORTED,
                "the MLP pair needs K %% 64 == 0, H %% 128 == 0, Ru %% 32 == 0 with Ru <= 128, Rd in {0, 32, 64} "
                "(K=%lld H=%lld Ru=%lld Rd=%lld)",
                (long long)K, (long long)H, (long long)Ru, (long long)Rd);
  if (!X || !Wu || !Wd || !Y || (Ru > 0 && (!LAu || !LBu)) || (Rd > 0 && (!LAd || !LBd)))
    return fail(RTL_ERR_NULL, "X, Wu, Wd, Y (and each layer's LA, LB when its rank > 0) are required");
  const void* ptrs[] = {X, Wu, LAu, LBu, Wd, LAd, LBd, Y, workspace, dbg_xd, dbg_idx, dbg_s};
  for (const void* q : ptrs)
    if (misaligned(q)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if ((st = check_eps(eps)) != RTL_OK) return st;
  const size_t need = rtl::mlp_bf16_workspace(M, K, H, N, Ru, Rd);
  const void* ins[7] = {X, Wu, Ru > 0 ? LAu : nullptr, Ru > 0 ? LBu : nullptr, Wd, Rd > 0 ? LAd : nullptr,
                        Rd > 0 ? LBd : nullptr};
  const size_t inb[7] = {(size_t)(M * K * 2), (size_t)(H * K * 2), (size_t)(H * Ru * 2), (size_t)(Ru * K * 2),
                         (size_t)(N * H * 2), (size_t)(N * Rd * 2), (size_t)(Rd * H * 2)};
  const void* outs[5] = {Y, workspace, dbg_xd, dbg_idx, dbg_s};
  const size_t outb[5] = {(size_t)(M * N * 2), need, (size_t)(M * H * 2), (size_t)(M * (H / 4)), (size_t)(M * 4)};
  for (int o = 0; o < 5; o++) {
    for (int i = 0; i < 7; i++)
      if (overlap(outs[o], outb[o], ins[i], inb[i])) return fail(RTL_ERR_ARG, "an output or the workspace overlaps an input");
    for (int o2 = o + 1; o2 < 5; o2++)
      if (overlap(outs[o], outb[o], outs[o2], outb[o2])) return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  }
  if (!workspace || ws_bytes < need)
    return fail(RTL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : (size_t)0);
  return hip_status(rtl::launch_mlp_bf16((int)variant, M, K, H, N, Ru, Rd, X, Wu, LAu, LBu, Wd, LAd, LBd, eps, Y, workspace,
                                         (uint16_t*)dbg_xd, dbg_idx, dbg_s, (hipStream_t)stream),
                    "rtl_mlp_fused launch");
}

rtl_status rtl_linear_dense_ref(rtl_dtype dt, int64_t M, int64_t N, int64_t K, const void* X, const void* W, void* Y,
                                void* stream) {
  rtl_status st;
  if ((st = check_dtype(dt)) != RTL_OK) return st;
  if (M <= 0 || N <= 0 || K <= 0 || K % 4 != 0)
    return fail(RTL_ERR_SHAPE, "need M, N, K > 0 and K %% 4 == 0 (M=%lld N=%lld K=%lld)", (long long)M, (long long)N,
                (long long)K);
  if ((st = check_extent(M, N, K)) != RTL_OK) return st;
  if (!X || !W || !Y) return fail(RTL_ERR_NULL, "X, W and Y are required");
  if (misaligned(X) || misaligned(W) || misaligned(Y)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if (dt == RTL_BF16 && K % 64 != 0) return fail(RTL_ERR_UNSUPPORTED, "bf16 path needs K %% 64 == 0 (K=%lld)", (long long)K);
  const size_t es = elem_size(dt);
  if (overlap(Y, (size_t)M * N * es, X, (size_t)M * K * es) || overlap(Y, (size_t)M * N * es, W, (size_t)N * K * es))
    return fail(RTL_ERR_ARG, "Y overlaps an input");
  hipError_t e;
  if (dt == RTL_BF16)
    e = rtl::launch_dense_bf16(M, N, K, X, W, Y, (hipStream_t)stream);
  else
    e = rtl::launch_dense_f32(M, N, K, (const float*)X, (const float*)W, (float*)Y, (hipStream_t)stream);
  return hip_status(e, "rtl_linear_dense_ref launch");
}

}  // extern "C"

extern "C" {

rtl_status rtl_quantize_weight_fp8(int64_t N, int64_t K, const void* W, uint8_t* Wq, float* sw, void* stream) {
  if (N <= 0 || K <= 0 || K % 8 != 0)
    return fail(RTL_ERR_SHAPE, "need N > 0, K > 0, K %% 8 == 0 (N=%lld K=%lld)", (long long)N, (long long)K);
  rtl_status st;
  if ((st = check_extent(1, N, K)) != RTL_OK) return st;
  if (!W || !Wq || !sw) return fail(RTL_ERR_NULL, "W, Wq and sw are required");
  if (misaligned(W) || misaligned(Wq) || misaligned(sw)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  const size_t wb = (size_t)N * K * 2, qb = (size_t)N * K, sb = (size_t)N * 4;
  if (overlap(Wq, qb, W, wb) || overlap(sw, sb, W, wb) || overlap(Wq, qb, sw, sb))
    return fail(RTL_ERR_ARG, "outputs overlap each other or the input");
  return hip_status(rtl::launch_quant_w_fp8(N, K, W, Wq, sw, (hipStream_t)stream), "rtl_quantize_weight_fp8 launch");
}

size_t rtl_linear_fused_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 128 != 0 || R < 0) return 0;
  return rtl::fused_fp8_workspace(M, N, K, R);
}

rtl_status rtl_linear_fused_fp8(int64_t M, int64_t N, int64_t K, int64_t R, const void* X, const uint8_t* Wq,
                                const float* sw, const void* LA, const void* LB, rtl_tie_rule tie, float eps, void* Y,
                                void* workspace, size_t ws_bytes, uint8_t* dbg_xq, float* dbg_sx, void* stream) {
  rtl_status st;
  if (tie != RTL_TIE_LOWER_INDEX) return fail(RTL_ERR_UNSUPPORTED, "unsupported tie rule %d", (int)tie);
  if (M <= 0 || N <= 0 || K <= 0 || K % 4 != 0 || R < 0)
    return fail(RTL_ERR_SHAPE, "need M, N, K > 0, K %% 4 == 0, R >= 0 (M=%lld N=%lld K=%lld R=%lld)", (long long)M,
                (long long)N, (long long)K, (long long)R);
  if ((st = check_extent(M, N, K)) != RTL_OK) return st;
  if (!X || !Wq || !sw || !Y || (R > 0 && (!LA || !LB)))
    return fail(RTL_ERR_NULL, "X, Wq, sw, Y (and LA, LB when R > 0) are required");
  if (misaligned(X) || misaligned(Wq) || misaligned(sw) || misaligned(Y) || misaligned(LA) || misaligned(LB) ||
      misaligned(workspace) || misaligned(dbg_xq) || misaligned(dbg_sx))
    return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if (K % 128 != 0) return fail(RTL_ERR_UNSUPPORTED, "fp8 path needs K %% 128 == 0 (K=%lld)", (long long)K);
  if (R % 32 != 0 || R > 128)
    return fail(RTL_ERR_UNSUPPORTED, "fp8 path needs R %% 32 == 0 and R <= 128 (R=%lld)", (long long)R);
  if ((st = check_eps(eps)) != RTL_OK) return st;
  const size_t xb = (size_t)M * K * 2, qb = (size_t)N * K, swb = (size_t)N * 4, lab = (size_t)N * R * 2,
               lbb = (size_t)R * K * 2, yb = (size_t)M * N * 2, xqb = (size_t)M * (K / 2), sxb = (size_t)M * 4;
  const size_t need = rtl_linear_fused_fp8_workspace_bytes(M, N, K, R);
  const void* ins[5] = {X, Wq, sw, R > 0 ? LA : nullptr, R > 0 ? LB : nullptr};
  const size_t inb[5] = {xb, qb, swb, lab, lbb};
  const void* outs[4] = {Y, dbg_xq, dbg_sx, workspace};
  const size_t outb[4] = {yb, xqb, sxb, need};
  for (int o = 0; o < 4; o++) {
    for (int i = 0; i < 5; i++)
      if (overlap(outs[o], outb[o], ins[i], inb[i])) return fail(RTL_ERR_ARG, "an output or the workspace overlaps an input");
    for (int o2 = o + 1; o2 < 4; o2++)
      if (overlap(outs[o], outb[o], outs[o2], outb[o2]))
        return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  }
  if (!workspace || ws_bytes < need)
    return fail(RTL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : (size_t)0);
  return hip_status(rtl::launch_fused_fp8(M, N, K, R, X, Wq, sw, LA, LB, eps, Y, workspace, dbg_xq, dbg_sx,
                                          (hipStream_t)stream),
                    "rtl_linear_fused_fp8 launch");
}

}  // extern "C"

namespace {

// A [M, H, D] tensor with strides, in elements; the stride of an extent of 1 counts as 0.
struct View {
  const void* p;
  int64_t M, H, D, row, head;
  size_t es;
  View(const void* p_, int64_t M_, int64_t H_, int64_t D_, int64_t row_, int64_t head_, size_t es_)
      : p(p_), M(M_), H(H_), D(D_), row(M_ == 1 ? 0 : row_), head(H_ == 1 ? 0 : head_), es(es_) {}
  int64_t span() const { return (M - 1) * row + (H - 1) * head + D; }  // elements
  bool same(const View& o) const { return p == o.p && row == o.row && head == o.head; }
};

rtl_status check_view(const View& v, const char* name, bool output) {
  if (!v.p) return fail(RTL_ERR_NULL, "%s is required", name);
  if (v.row < 0 || v.head < 0 || (__int128)(v.M - 1) * v.row + (__int128)(v.H - 1) * v.head > ((int64_t)1 << 48))
    return fail(RTL_ERR_SHAPE, "strides of %s out of range (row %lld, head %lld)", name, (long long)v.row,
                (long long)v.head);
  if (misaligned(v.p) || (v.row * v.es) % 16 != 0 || (v.head * v.es) % 16 != 0)
    return fail(RTL_ERR_ALIGN, "%s and its strides must be 16-byte aligned", name);
  if (output) {
    const bool rows = (v.H == 1 || v.head >= v.D) && (v.M == 1 || v.row >= (v.H - 1) * v.head + v.D);
    const bool heads = (v.M == 1 || v.row >= v.D) && (v.H == 1 || v.head >= (v.M - 1) * v.row + v.D);
    if (!rows && !heads) return fail(RTL_ERR_ARG, "the elements of %s overlap", name);
  }
  return RTL_OK;
}

// Windows [0, na) and [d, d + nb) that both repeat every `period` elements share none.
bool windows_apart(int64_t d, int64_t na, int64_t nb, int64_t period) {
  const int64_t r = ((d % period) + period) % period;
  return r >= na && r + nb <= period;
}

// Two views that share no element: apart as byte ranges, or interleaved in one buffer with
// the same row stride (each row's heads in a window of its own), the same head stride (each
// head's rows likewise), or the same head stride inside rows of whole heads.
bool apart(const View& a, const View& b) {
  if (!overlap(a.p, (size_t)a.span() * a.es, b.p, (size_t)b.span() * b.es)) return true;
  const int64_t bytes = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
  if (bytes % (int64_t)a.es != 0) return false;
  const int64_t d = bytes / (int64_t)a.es;
  const int64_t ra = (a.H - 1) * a.head + a.D, rb = (b.H - 1) * b.head + b.D;  // a row's window
  const int64_t ha = (a.M - 1) * a.row + a.D, hb = (b.M - 1) * b.row + b.D;    // a head's window
  if (a.row == b.row && a.row > 0 && windows_apart(d, ra, rb, a.row)) return true;
  if (a.head == b.head && a.head > 0 && windows_apart(d, ha, hb, a.head)) return true;
  return a.head == b.head && a.head > 0 && a.row % a.head == 0 && b.row % b.head == 0 &&
         windows_apart(d, a.D, b.D, a.head);
}

bool apart_flat(const View& a, const void* p, size_t bytes) { return !overlap(a.p, (size_t)a.span() * a.es, p, bytes); }

// Checks shared by rtl_rope_axes, rtl_qk_norm_rope and its gradient (everything but the
// tensors); need_axes: a call without axes is refused.
rtl_status check_rope(rtl_dtype dt, int64_t M, int64_t Hq, int64_t Hk, int64_t D, const float* pos, int32_t n_axes,
                      const int32_t* axis_dims, double theta, rtl_rope_pairs pairs, bool need_axes) {
  rtl_status st;
  if ((st = check_dtype(dt)) != RTL_OK) return st;
  if (M <= 0 || Hq <= 0 || Hk < 0 || D <= 0)
    return fail(RTL_ERR_SHAPE, "need M, heads, D > 0 (M=%lld H=%lld,%lld D=%lld)", (long long)M, (long long)Hq,
                (long long)Hk, (long long)D);
  if (Hq > INT32_MAX || Hk > INT32_MAX || M > INT32_MAX || M * (Hq + Hk) > INT32_MAX)
    return fail(RTL_ERR_SHAPE, "M x heads is too large (M=%lld H=%lld,%lld)", (long long)M, (long long)Hq,
                (long long)Hk);
  if (D % 8 != 0 || D > 256) return fail(RTL_ERR_UNSUPPORTED, "need D %% 8 == 0 and D <= 256 (D=%lld)", (long long)D);
  if (pairs != RTL_ROPE_ADJACENT && pairs != RTL_ROPE_HALVES)
    return fail(RTL_ERR_UNSUPPORTED, "unsupported pairing %d", (int)pairs);
  if (n_axes < (need_axes ? 1 : 0) || n_axes > 4) return fail(RTL_ERR_UNSUPPORTED, "unsupported number of axes %d", n_axes);
  if (n_axes == 0) return RTL_OK;
  if (!pos || !axis_dims) return fail(RTL_ERR_NULL, "pos and axis_dims are required");
  if (misaligned(pos)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  int64_t sum = 0;
  for (int a = 0; a < n_axes; a++) {
    if (axis_dims[a] < 2 || axis_dims[a] % 2 != 0 || axis_dims[a] > D)
      return fail(RTL_ERR_SHAPE, "axis %d turns %d channels: need an even number of 2 to D", a, axis_dims[a]);
    sum += axis_dims[a];
  }
  if (sum > D) return fail(RTL_ERR_SHAPE, "the axes turn %lld of %lld channels", (long long)sum, (long long)D);
  if (sum % 8 != 0) return fail(RTL_ERR_UNSUPPORTED, "the axes must turn a multiple of 8 channels (%lld)", (long long)sum);
  if (!(theta >= 1.0 && theta <= 1e30)) return fail(RTL_ERR_ARG, "theta must lie in [1, 1e30] (got %g)", theta);
  return RTL_OK;
}

rtl::RopeCall rope_call(rtl_dtype dt, bool norm, int64_t M, int64_t Hq, int64_t Hk, int64_t D, const float* pos,
                        int32_t n_axes, const int32_t* axis_dims, double theta, rtl_rope_pairs pairs, bool inverse) {
  rtl::RopeCall c{};
  c.dt = dt == RTL_BF16 ? rtl::kDtBF16 : rtl::kDtF32;
  c.norm = norm;
  c.halves = pairs == RTL_ROPE_HALVES;
  c.inverse = inverse;
  c.M = M;
  c.H[0] = Hq;
  c.H[1] = Hk;
  c.D = D;
  c.pos = pos;
  c.axes = n_axes;
  c.dims = axis_dims;
  c.theta = theta;
  return c;
}

rtl::StridedHeads heads(const View& v) { return rtl::StridedHeads{v.p, v.row, v.head}; }

// eps of the head norms: a normal number, so that a head of zeros has a finite r.
rtl_status check_norm_eps(float eps) {
  if (!(eps >= 0x1p-126f && eps <= 1.f)) return fail(RTL_ERR_ARG, "eps must lie in [2^-126, 1] (got %g)", (double)eps);
  return RTL_OK;
}

}  // namespace

extern "C" {

rtl_status rtl_rope_axes(rtl_dtype dt, int64_t M, int64_t H, int64_t D, const void* X, int64_t x_row, int64_t x_head,
                         const float* pos, int32_t n_axes, const int32_t* axis_dims, double theta,
                         rtl_rope_pairs pairs, int32_t inverse, void* Y, int64_t y_row, int64_t y_head, void* stream) {
  rtl_status st;
  if ((st = check_rope(dt, M, H, 0, D, pos, n_axes, axis_dims, theta, pairs, true)) != RTL_OK) return st;
  if (inverse != 0 && inverse != 1) return fail(RTL_ERR_ARG, "inverse must be 0 or 1 (got %d)", inverse);
  const View x(X, M, H, D, x_row, x_head, elem_size(dt)), y(Y, M, H, D, y_row, y_head, elem_size(dt));
  if ((st = check_view(x, "X", false)) != RTL_OK || (st = check_view(y, "Y", true)) != RTL_OK) return st;
  if ((!x.same(y) && !apart(x, y)) || !apart_flat(y, pos, (size_t)M * n_axes * 4))
    return fail(RTL_ERR_ARG, "Y overlaps an input");
  rtl::RopeCall c = rope_call(dt, false, M, H, 0, D, pos, n_axes, axis_dims, theta, pairs, inverse != 0);
  c.x[0] = heads(x);
  c.y[0] = heads(y);
  return hip_status(rtl::launch_rope(c, (hipStream_t)stream), "rtl_rope_axes launch");
}

rtl_status rtl_qk_norm_rope(rtl_dtype dt, int64_t M, int64_t Hq, int64_t Hk, int64_t D, const void* Q, int64_t q_row,
                            int64_t q_head, const void* K, int64_t k_row, int64_t k_head, const void* qw,
                            const void* kw, float eps, const float* pos, int32_t n_axes, const int32_t* axis_dims,
                            double theta, rtl_rope_pairs pairs, void* Qo, int64_t qo_row, int64_t qo_head, void* Ko,
                            int64_t ko_row, int64_t ko_head, void* stream) {
  rtl_status st;
  if ((st = check_rope(dt, M, Hq, Hk, D, pos, n_axes, axis_dims, theta, pairs, false)) != RTL_OK) return st;
  if ((st = check_norm_eps(eps)) != RTL_OK) return st;
  const size_t es = elem_size(dt);
  const int n = Hk > 0 ? 2 : 1;
  const View in[2] = {View(Q, M, Hq, D, q_row, q_head, es), View(K, M, Hk, D, k_row, k_head, es)};
  const View out[2] = {View(Qo, M, Hq, D, qo_row, qo_head, es), View(Ko, M, Hk, D, ko_row, ko_head, es)};
  const void* w[2] = {qw, n == 2 ? kw : nullptr};
  const char* names[2][2] = {{"Q", "K"}, {"Qo", "Ko"}};
  for (int i = 0; i < n; i++) {
    if ((st = check_view(in[i], names[0][i], false)) != RTL_OK || (st = check_view(out[i], names[1][i], true)) != RTL_OK)
      return st;
    if (misaligned(w[i])) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  }
  for (int o = 0; o < n; o++) {
    for (int i = 0; i < n; i++) {
      if (!(i == o && in[i].same(out[o])) && !apart(in[i], out[o])) return fail(RTL_ERR_ARG, "an output overlaps an input");
      if (!apart_flat(out[o], w[i], (size_t)D * es)) return fail(RTL_ERR_ARG, "an output overlaps an input");
    }
    if (n_axes > 0 && !apart_flat(out[o], pos, (size_t)M * n_axes * 4))
      return fail(RTL_ERR_ARG, "an output overlaps an input");
  }
  if (n == 2 && !apart(out[0], out[1])) return fail(RTL_ERR_ARG, "outputs overlap each other");
  rtl::RopeCall c = rope_call(dt, true, M, Hq, Hk, D, pos, n_axes, axis_dims, theta, pairs, false);
  c.eps = eps;
  for (int i = 0; i < n; i++) {
    c.x[i] = heads(in[i]);
    c.y[i] = heads(out[i]);
    c.w[i] = w[i];
  }
  return hip_status(rtl::launch_rope(c, (hipStream_t)stream), "rtl_qk_norm_rope launch");
}

size_t rtl_qk_norm_rope_backward_workspace_bytes(int64_t D) {
  return D <= 0 || D > 256 ? 0 : rtl::qk_back_workspace(D);
}

rtl_status rtl_qk_norm_rope_backward(rtl_dtype dt, int64_t M, int64_t Hq, int64_t Hk, int64_t D, const void* Q,
                                     int64_t q_row, int64_t q_head, const void* K, int64_t k_row, int64_t k_head,
                                     const void* qw, const void* kw, float eps, const float* pos, int32_t n_axes,
                                     const int32_t* axis_dims, double theta, rtl_rope_pairs pairs, const void* dQo,
                                     int64_t dqo_row, int64_t dqo_head, const void* dKo, int64_t dko_row,
                                     int64_t dko_head, void* dQ, int64_t dq_row, int64_t dq_head, void* dK,
                                     int64_t dk_row, int64_t dk_head, float* dqw, float* dkw, void* workspace,
                                     size_t ws_bytes, void* stream) {
  rtl_status st;
  if ((st = check_rope(dt, M, Hq, Hk, D, pos, n_axes, axis_dims, theta, pairs, false)) != RTL_OK) return st;
  if ((st = check_norm_eps(eps)) != RTL_OK) return st;
  const size_t es = elem_size(dt);
  const int n = Hk > 0 ? 2 : 1;
  const View in[2] = {View(Q, M, Hq, D, q_row, q_head, es), View(K, M, Hk, D, k_row, k_head, es)};
  const View dy[2] = {View(dQo, M, Hq, D, dqo_row, dqo_head, es), View(dKo, M, Hk, D, dko_row, dko_head, es)};
  const View dx[2] = {View(dQ, M, Hq, D, dq_row, dq_head, es), View(dK, M, Hk, D, dk_row, dk_head, es)};
  const void* w[2] = {qw, n == 2 ? kw : nullptr};
  float* dw[2] = {dqw, n == 2 ? dkw : nullptr};
  const char* names[3][2] = {{"Q", "K"}, {"dQo", "dKo"}, {"dQ", "dK"}};
  const size_t need = rtl::qk_back_workspace(D), wb = (size_t)D * es, dwb = (size_t)D * 4, pb = (size_t)M * n_axes * 4;
  for (int i = 0; i < n; i++) {
    if ((st = check_view(in[i], names[0][i], false)) != RTL_OK || (st = check_view(dy[i], names[1][i], false)) != RTL_OK ||
        (st = check_view(dx[i], names[2][i], true)) != RTL_OK)
      return st;
    if (misaligned(w[i]) || misaligned(dw[i])) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  }
  if (misaligned(workspace)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  // flat outputs against everything, then the strided ones against what is left
  const void* flat[3] = {dw[0], dw[1], workspace};
  const size_t flatb[3] = {dwb, dwb, need};
  for (int f = 0; f < 3; f++) {
    if (n_axes > 0 && overlap(flat[f], flatb[f], pos, pb)) return fail(RTL_ERR_ARG, "an output or the workspace overlaps an input");
    for (int i = 0; i < n; i++) {
      if (overlap(flat[f], flatb[f], w[i], wb) || !apart_flat(in[i], flat[f], flatb[f]) || !apart_flat(dy[i], flat[f], flatb[f]))
        return fail(RTL_ERR_ARG, "an output or the workspace overlaps an input");
      if (!apart_flat(dx[i], flat[f], flatb[f])) return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
    }
    for (int g = f + 1; g < 3; g++)
      if (overlap(flat[f], flatb[f], flat[g], flatb[g]))
        return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  }
  for (int o = 0; o < n; o++) {
    for (int i = 0; i < n; i++)
      if ((!(i == o && in[i].same(dx[o])) && !apart(in[i], dx[o])) ||
          (!(i == o && dy[i].same(dx[o])) && !apart(dy[i], dx[o])) || !apart_flat(dx[o], w[i], wb))
        return fail(RTL_ERR_ARG, "an output overlaps an input");
    if (n_axes > 0 && !apart_flat(dx[o], pos, pb)) return fail(RTL_ERR_ARG, "an output overlaps an input");
  }
  if (n == 2 && !apart(dx[0], dx[1])) return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  if (!workspace || ws_bytes < need)
    return fail(RTL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : (size_t)0);
  rtl::RopeCall c = rope_call(dt, true, M, Hq, Hk, D, pos, n_axes, axis_dims, theta, pairs, true);
  c.eps = eps;
  for (int i = 0; i < n; i++) {
    c.x[i] = heads(in[i]);
    c.y[i] = heads(dy[i]);
    c.dx[i] = heads(dx[i]);
    c.w[i] = w[i];
  }
  return hip_status(rtl::launch_qk_back(c, dw[0], dw[1], workspace, (hipStream_t)stream),
                    "rtl_qk_norm_rope_backward launch");
}

}  // extern "C"

namespace {

rtl_status check_glu(rtl_act act, rtl_dtype dt, int64_t M, int64_t K, int64_t H) {
  rtl_status st;
  if ((st = check_dtype(dt)) != RTL_OK) return st;
  if (dt != RTL_BF16) return fail(RTL_ERR_UNSUPPORTED, "the gated block is bf16 only");
  if (act != RTL_ACT_SILU && act != RTL_ACT_GELU) return fail(RTL_ERR_UNSUPPORTED, "unsupported activation %d", (int)act);
  if (M <= 0 || K <= 0 || H <= 0)
    return fail(RTL_ERR_SHAPE, "need M, K, H > 0 (M=%lld K=%lld H=%lld)", (long long)M, (long long)K, (long long)H);
  // a tile's rows are reached with 32-bit offsets: 256 rows of K bf16 values stay below 2^31 bytes
  if (K >= kMaxK) return fail(RTL_ERR_SHAPE, "K must be below %lld (K=%lld)", (long long)kMaxK, (long long)K);
  // a launch takes fewer than 2^32 threads: 256 to a 128 x 64 tile, or to 16 outputs of few rows
  if (M > INT32_MAX || H > (1 << 28) - 16 || ((M + 127) / 128) * ((H + 63) / 64) >= 1 << 24)
    return fail(RTL_ERR_SHAPE, "M x H is too large (M=%lld H=%lld)", (long long)M, (long long)H);
  if (K % 64 != 0) return fail(RTL_ERR_UNSUPPORTED, "the gated block needs K %% 64 == 0 (K=%lld)", (long long)K);
  return RTL_OK;
}

// The gradient's limits: its products sum over 2 H padded (dX) and over M padded (dWg, dWu), with the
// same 32-bit offsets, and its first pass has a thread for every eight elements, fewer than 2^32.
bool glu_back_fits(int64_t M, int64_t K, int64_t H) {
  return M <= kMaxK - 64 && H <= kMaxK / 2 - 64 && K < kMaxK && M * ((H + 63) / 64 * 64) < (int64_t)1 << 35;
}

}  // namespace

extern "C" {

rtl_status rtl_glu_fused(rtl_act act, rtl_dtype dt, int64_t M, int64_t K, int64_t H, const void* X, const void* Wg,
                         const void* Wu, void* Y, void* G, void* U, void* stream) {
  rtl_status st;
  if ((st = check_glu(act, dt, M, K, H)) != RTL_OK) return st;
  if (!X || !Wg || !Wu || !Y) return fail(RTL_ERR_NULL, "X, Wg, Wu and Y are required");
  const void* ins[3] = {X, Wg, Wu};
  const size_t inb[3] = {(size_t)M * K * 2, (size_t)H * K * 2, (size_t)H * K * 2};
  const void* outs[3] = {Y, G, U};
  const size_t outb = (size_t)M * H * 2;
  for (int i = 0; i < 3; i++)
    if (misaligned(ins[i]) || misaligned(outs[i])) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  for (int o = 0; o < 3; o++) {
    for (int i = 0; i < 3; i++)
      if (overlap(outs[o], outb, ins[i], inb[i])) return fail(RTL_ERR_ARG, "an output overlaps an input");
    for (int o2 = o + 1; o2 < 3; o2++)
      if (overlap(outs[o], outb, outs[o2], outb)) return fail(RTL_ERR_ARG, "outputs overlap each other");
  }
  return hip_status(rtl::launch_glu_bf16(act == RTL_ACT_SILU ? rtl::kActSilu : rtl::kActGelu, M, K, H, X, Wg, Wu, Y, G, U,
                                         (hipStream_t)stream),
                    "rtl_glu_fused launch");
}

size_t rtl_glu_backward_workspace_bytes(int64_t M, int64_t K, int64_t H) {
  return M <= 0 || K <= 0 || H <= 0 || !glu_back_fits(M, K, H) ? 0 : rtl::glu_back_workspace(M, K, H);
}

rtl_status rtl_glu_backward(rtl_act act, rtl_dtype dt, int64_t M, int64_t K, int64_t H, const void* X, const void* Wg,
                            const void* Wu, const void* G, const void* U, const void* dY, void* dX, void* dWg,
                            void* dWu, void* workspace, size_t ws_bytes, void* stream) {
  rtl_status st;
  if ((st = check_glu(act, dt, M, K, H)) != RTL_OK) return st;
  if (!glu_back_fits(M, K, H))
    return fail(RTL_ERR_SHAPE, "the gradient needs M <= %lld, H <= %lld and M x H below 2^35 (M=%lld H=%lld)",
                (long long)kMaxK - 64, (long long)kMaxK / 2 - 64, (long long)M, (long long)H);
  if (!G || !U || !dY || (!dX && !dWg) || (dWg == nullptr) != (dWu == nullptr) || (dX && (!Wg || !Wu)) || (dWg && !X))
    return fail(RTL_ERR_NULL, "G, U, dY, dX (with Wg, Wu) or dWg and dWu (with X) are required");
  const void* ins[6] = {dWg ? X : nullptr, dX ? Wg : nullptr, dX ? Wu : nullptr, G, U, dY};
  const size_t xb = (size_t)M * K * 2, wb = (size_t)H * K * 2, yb = (size_t)M * H * 2;
  const size_t inb[6] = {xb, wb, wb, yb, yb, yb};
  const size_t need = rtl::glu_back_workspace(M, K, H);
  const void* outs[4] = {dX, dWg, dWu, workspace};
  const size_t outb[4] = {xb, wb, wb, need};
  for (const void* q : ins)
    if (misaligned(q)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  for (const void* q : outs)
    if (misaligned(q)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  for (int o = 0; o < 4; o++) {
    for (int i = 0; i < 6; i++)
      if (overlap(outs[o], outb[o], ins[i], inb[i])) return fail(RTL_ERR_ARG, "an output or the workspace overlaps an input");
    for (int o2 = o + 1; o2 < 4; o2++)
      if (overlap(outs[o], outb[o], outs[o2], outb[o2]))
        return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  }
  if (!workspace || ws_bytes < need)
    return fail(RTL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : (size_t)0);
  return hip_status(rtl::launch_glu_back_bf16(act == RTL_ACT_SILU ? rtl::kActSilu : rtl::kActGelu, M, K, H, X, Wg, Wu, G,
                                              U, dY, dX, dWg, dWu, workspace, (hipStream_t)stream),
                    "rtl_glu_backward launch");
}

}  // extern "C"

namespace {

// A [M, D] tensor with a row stride, aligned to its elements; the stride of one row counts as 0.
View rows_of(const void* p, int64_t M, int64_t D, int64_t row, size_t es) { return View(p, M, 1, D, row, 0, es); }

rtl_status check_rows(const View& v, const char* name, bool output) {
  if (!v.p) return fail(RTL_ERR_NULL, "%s is required", name);
  if (v.row < 0 || (__int128)(v.M - 1) * v.row > ((int64_t)1 << 48))
    return fail(RTL_ERR_SHAPE, "row stride of %s out of range (%lld)", name, (long long)v.row);
  if ((uintptr_t)v.p % v.es != 0) return fail(RTL_ERR_ALIGN, "%s must be aligned to its elements", name);
  if (output && v.M > 1 && v.row < v.D) return fail(RTL_ERR_ARG, "the rows of %s overlap", name);
  return RTL_OK;
}

// What the layer norm and its gradient share; fills the call but for y, dy and stats.
rtl_status check_norm(rtl_dtype dt, int64_t M, int64_t D, const View& x, const void* w, const void* b, int64_t G,
                      const int32_t* groups, const View& scale, rtl::NormCall& c) {
  rtl_status st;
  const size_t es = elem_size(dt);
  if ((st = check_rows(x, "X", false)) != RTL_OK) return st;
  if ((uintptr_t)w % es != 0 || (uintptr_t)b % es != 0 || (uintptr_t)groups % 4 != 0)
    return fail(RTL_ERR_ALIGN, "w, b and groups must be aligned to their elements");
  if (groups == nullptr && G > 1) return fail(RTL_ERR_NULL, "groups is required for G = %lld", (long long)G);
  if (groups != nullptr && G < 1) return fail(RTL_ERR_SHAPE, "groups of G = %lld", (long long)G);
  if (scale.p != nullptr && G < 1) return fail(RTL_ERR_SHAPE, "scale and shift of G = %lld", (long long)G);
  c = rtl::NormCall{};
  c.dt = dt == RTL_BF16 ? rtl::kDtBF16 : rtl::kDtF32;
  c.M = M;
  c.D = D;
  c.G = G;
  c.x = rtl::RowsView{x.p, x.row};
  c.scale = rtl::RowsView{scale.p, scale.row};
  c.w = w;
  c.b = b;
  c.groups = groups;
  return RTL_OK;
}

rtl_status check_norm_sizes(rtl_dtype dt, int64_t M, int64_t D, int64_t G) {
  rtl_status st;
  if ((st = check_dtype(dt)) != RTL_OK) return st;
  if (M <= 0 || D <= 0 || G < 0)
    return fail(RTL_ERR_SHAPE, "need M, D > 0 and G >= 0 (M=%lld D=%lld G=%lld)", (long long)M, (long long)D, (long long)G);
  if (M > INT32_MAX || G >= INT32_MAX) return fail(RTL_ERR_SHAPE, "M or G is too large (M=%lld G=%lld)", (long long)M, (long long)G);
  if (!rtl::norm_fits(dt == RTL_BF16 ? rtl::kDtBF16 : rtl::kDtF32, D, true))
    return fail(RTL_ERR_UNSUPPORTED, "D is too large (D=%lld)", (long long)D);
  return RTL_OK;
}

rtl_status check_rest(rtl_rest rest) {
  if (rest != RTL_REST_KEPT && rest != RTL_REST_ZEROS) return fail(RTL_ERR_ARG, "unsupported rest %d", (int)rest);
  return RTL_OK;
}

rtl_status check_norm_width(const rtl::NormCall& c) {
  if (!rtl::norm_fits(c.dt, c.D, rtl::norm_is_wide(c)))
    return fail(RTL_ERR_UNSUPPORTED, "D above %lld needs 16-byte aligned rows (D=%lld)", (long long)rtl::kNormMaxDNarrow,
                (long long)c.D);
  return RTL_OK;
}

// Flat outputs and a workspace against strided and flat inputs and against each other.
struct Flat {
  const void* p;
  size_t bytes;
};
template <int NO, int NI>
rtl_status check_flat_apart(const Flat (&outs)[NO], const Flat (&ins)[NI]) {
  for (int o = 0; o < NO; o++) {
    for (int i = 0; i < NI; i++)
      if (overlap(outs[o].p, outs[o].bytes, ins[i].p, ins[i].bytes))
        return fail(RTL_ERR_ARG, "an output or the workspace overlaps an input");
    for (int k = o + 1; k < NO; k++)
      if (overlap(outs[o].p, outs[o].bytes, outs[k].p, outs[k].bytes))
        return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  }
  return RTL_OK;
}
Flat range_of(const View& v) { return Flat{v.p, v.p ? (size_t)v.span() * v.es : 0}; }

}  // namespace

extern "C" {

rtl_status rtl_layer_norm(rtl_dtype dt, int64_t M, int64_t D, const void* X, int64_t x_row, const void* w, const void* b,
                          int64_t G, const int32_t* groups, const void* scale, int64_t scale_row, const void* shift,
                          int64_t shift_row, float eps, void* Y, int64_t y_row, float* stats, void* stream) {
  return rtl_layer_norm_ex(RTL_REST_KEPT, dt, M, D, X, x_row, w, b, G, groups, scale, scale_row, shift, shift_row, eps, Y, y_row,
                           stats, stream);
}

rtl_status rtl_layer_norm_ex(rtl_rest rest, rtl_dtype dt, int64_t M, int64_t D, const void* X, int64_t x_row, const void* w,
                             const void* b, int64_t G, const int32_t* groups, const void* scale, int64_t scale_row,
                             const void* shift, int64_t shift_row, float eps, void* Y, int64_t y_row, float* stats,
                             void* stream) {
  rtl_status st;
  if ((st = check_rest(rest)) != RTL_OK) return st;
  if ((st = check_norm_sizes(dt, M, D, G)) != RTL_OK || (st = check_norm_eps(eps)) != RTL_OK) return st;
  const size_t es = elem_size(dt);
  const View x = rows_of(X, M, D, x_row, es), y = rows_of(Y, M, D, y_row, es);
  const View sc = rows_of(scale, G, D, scale_row, es), sh = rows_of(shift, G, D, shift_row, es);
  rtl::NormCall c;
  if ((st = check_norm(dt, M, D, x, w, b, G, groups, sc, c)) != RTL_OK || (st = check_rows(y, "Y", true)) != RTL_OK) return st;
  if ((scale == nullptr) != (shift == nullptr)) return fail(RTL_ERR_NULL, "scale and shift go together");
  if (scale != nullptr &&
      ((st = check_rows(sc, "scale", false)) != RTL_OK || (st = check_rows(sh, "shift", false)) != RTL_OK))
    return st;
  if ((uintptr_t)stats % 8 != 0) return fail(RTL_ERR_ALIGN, "stats must be 8-byte aligned");
  c.y = rtl::RowsView{y.p, y.row};
  c.shift = rtl::RowsView{sh.p, sh.row};
  c.eps = eps;
  c.stats = stats;
  c.clear = rest == RTL_REST_ZEROS;
  if ((st = check_norm_width(c)) != RTL_OK) return st;
  const Flat small[3] = {{w, (size_t)D * es}, {b, (size_t)D * es}, {groups, (size_t)(G + 1) * 4}};
  const Flat wide[2] = {scale ? range_of(sc) : Flat{nullptr, 0}, shift ? range_of(sh) : Flat{nullptr, 0}};
  if (!x.same(y) && !apart(x, y)) return fail(RTL_ERR_ARG, "Y overlaps an input");
  for (const Flat& f : small)
    if (!apart_flat(y, f.p, f.bytes)) return fail(RTL_ERR_ARG, "Y overlaps an input");
  for (const Flat& f : wide)
    if (!apart_flat(y, f.p, f.bytes)) return fail(RTL_ERR_ARG, "Y overlaps an input");
  const Flat outs[1] = {{stats, (size_t)M * 8}};
  const Flat ins[6] = {small[0], small[1], small[2], wide[0], wide[1], range_of(x)};
  if ((st = check_flat_apart(outs, ins)) != RTL_OK) return st;
  if (!apart_flat(y, stats, (size_t)M * 8)) return fail(RTL_ERR_ARG, "outputs overlap each other");
  return hip_status(rtl::launch_norm(c, (hipStream_t)stream), "rtl_layer_norm launch");
}

size_t rtl_layer_norm_backward_workspace_bytes(int64_t M, int64_t D, int64_t G) {
  if (M <= 0 || D <= 0 || G < 0 || M > INT32_MAX || D > rtl::kNormMaxD || G >= INT32_MAX || G * D >= (int64_t)1 << 29) return 0;
  return rtl::norm_back_workspace(M, D, G);
}

rtl_status rtl_layer_norm_backward(rtl_dtype dt, int64_t M, int64_t D, const void* X, int64_t x_row, const float* stats,
                                   const void* dY, int64_t dy_row, const void* w, const void* b, int64_t G,
                                   const int32_t* groups, const void* scale, int64_t scale_row, void* dX, int64_t dx_row,
                                   float* dw, float* db, float* dscale, float* dshift, void* workspace, size_t ws_bytes,
                                   void* stream) {
  return rtl_layer_norm_backward_ex(RTL_REST_KEPT, dt, M, D, X, x_row, stats, dY, dy_row, w, b, G, groups, scale, scale_row, dX,
                                    dx_row, dw, db, dscale, dshift, workspace, ws_bytes, stream);
}

rtl_status rtl_layer_norm_backward_ex(rtl_rest rest, rtl_dtype dt, int64_t M, int64_t D, const void* X, int64_t x_row,
                                      const float* stats, const void* dY, int64_t dy_row, const void* w, const void* b,
                                      int64_t G, const int32_t* groups, const void* scale, int64_t scale_row, void* dX,
                                      int64_t dx_row, float* dw, float* db, float* dscale, float* dshift, void* workspace,
                                      size_t ws_bytes, void* stream) {
  rtl_status st;
  if ((st = check_rest(rest)) != RTL_OK) return st;
  if ((st = check_norm_sizes(dt, M, D, G)) != RTL_OK) return st;
  if (G * D >= (int64_t)1 << 29) return fail(RTL_ERR_SHAPE, "G x D is too large (G=%lld D=%lld)", (long long)G, (long long)D);
  const size_t es = elem_size(dt);
  const View x = rows_of(X, M, D, x_row, es), dy = rows_of(dY, M, D, dy_row, es), dx = rows_of(dX, M, D, dx_row, es);
  const View sc = rows_of(scale, G, D, scale_row, es);
  rtl::NormCall c;
  if ((st = check_norm(dt, M, D, x, w, b, G, groups, sc, c)) != RTL_OK || (st = check_rows(dy, "dY", false)) != RTL_OK ||
      (st = check_rows(dx, "dX", true)) != RTL_OK)
    return st;
  if (scale != nullptr && (st = check_rows(sc, "scale", false)) != RTL_OK) return st;
  if (!stats) return fail(RTL_ERR_NULL, "stats is required");
  if (scale == nullptr && (dscale != nullptr || dshift != nullptr))
    return fail(RTL_ERR_ARG, "dscale and dshift without scale");
  if ((uintptr_t)stats % 8 != 0 || misaligned(dw) || misaligned(db) || misaligned(dscale) || misaligned(dshift) ||
      misaligned(workspace))
    return fail(RTL_ERR_ALIGN, "stats must be 8-byte aligned, the sums and the workspace 16-byte aligned");
  c.y = rtl::RowsView{dx.p, dx.row};
  c.dy = rtl::RowsView{dy.p, dy.row};
  c.stats = stats;
  c.clear = rest == RTL_REST_ZEROS;
  if ((st = check_norm_width(c)) != RTL_OK) return st;
  const size_t need = rtl::norm_back_workspace(M, D, G), wb = (size_t)D * 4, gb = (size_t)(G > 0 ? G : 1) * D * 4;
  const Flat outs[5] = {{dw, wb}, {db, wb}, {dscale, gb}, {dshift, gb}, {workspace, need}};
  const Flat ins[7] = {{w, (size_t)D * es}, {b, (size_t)D * es}, {groups, (size_t)(G + 1) * 4}, {stats, (size_t)M * 8},
                       scale ? range_of(sc) : Flat{nullptr, 0}, range_of(x), range_of(dy)};
  if ((st = check_flat_apart(outs, ins)) != RTL_OK) return st;
  for (const Flat& f : outs)
    if (!apart_flat(dx, f.p, f.bytes)) return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  for (int i = 0; i < 5; i++)
    if (!apart_flat(dx, ins[i].p, ins[i].bytes)) return fail(RTL_ERR_ARG, "an output overlaps an input");
  if ((!x.same(dx) && !apart(x, dx)) || (!dy.same(dx) && !apart(dy, dx)))
    return fail(RTL_ERR_ARG, "an output overlaps an input");
  if (!workspace || ws_bytes < need)
    return fail(RTL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : (size_t)0);
  return hip_status(rtl::launch_norm_back(c, dw, db, dscale, dshift, workspace, (hipStream_t)stream),
                    "rtl_layer_norm_backward launch");
}

}  // extern "C"

namespace {

bool adapters_fit(int64_t M, int64_t A) { return M > 0 && M <= 1 << 24 && A > 0 && A <= 4096; }
bool adapters_fit(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A) {
  return adapters_fit(M, A) && N > 0 && N <= kMaxK && K > 0 && K <= kMaxK && R > 0 && R <= 128 && N % 8 == 0 && K % 8 == 0 &&
         R % 8 == 0 && A * (N > K ? N : K) <= (int64_t)1 << 27;
}

rtl_status check_plan_sizes(int64_t M, int64_t A) {
  if (M <= 0 || A <= 0) return fail(RTL_ERR_SHAPE, "need M, A > 0 (M=%lld A=%lld)", (long long)M, (long long)A);
  if (!adapters_fit(M, A)) return fail(RTL_ERR_SHAPE, "M or A is too large (M=%lld A=%lld)", (long long)M, (long long)A);
  return RTL_OK;
}

rtl_status check_adapters(rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R, int64_t A, const void* LA, const void* LB,
                          const void* plan, size_t plan_bytes, const float* alpha) {
  rtl_status st;
  if ((st = check_dtype(dt)) != RTL_OK) return st;
  if (dt != RTL_BF16) return fail(RTL_ERR_UNSUPPORTED, "adapters are bf16 only");
  if ((st = check_plan_sizes(M, A)) != RTL_OK) return st;
  if (N <= 0 || K <= 0 || R <= 0 || N > kMaxK || K > kMaxK)
    return fail(RTL_ERR_SHAPE, "need N, K in 1 .. 2^22 and R > 0 (N=%lld K=%lld R=%lld)", (long long)N, (long long)K, (long long)R);
  if (N % 8 != 0 || K % 8 != 0 || R % 8 != 0 || R > 128)
    return fail(RTL_ERR_UNSUPPORTED, "adapters need N, K, R multiples of 8 and R <= 128 (N=%lld K=%lld R=%lld)", (long long)N,
                (long long)K, (long long)R);
  if (!adapters_fit(M, N, K, R, A)) return fail(RTL_ERR_SHAPE, "the factors are too large (A=%lld R=%lld)", (long long)A, (long long)R);
  if (!LA || !LB || !plan) return fail(RTL_ERR_NULL, "LA, LB and the plan are required");
  if (misaligned(LA) || misaligned(LB) || misaligned(plan)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  if ((uintptr_t)alpha % 4 != 0) return fail(RTL_ERR_ALIGN, "alpha must be aligned to its elements");
  if (plan_bytes != rtl::adapters_plan_bytes(M, A))
    return fail(RTL_ERR_ARG, "the plan has %zu bytes, one for M=%lld and A=%lld has %zu", plan_bytes, (long long)M, (long long)A,
                rtl::adapters_plan_bytes(M, A));
  return RTL_OK;
}

// A [M, C] tensor of bf16 rows that 16-byte accesses reach.
rtl_status check_bf16_rows(const View& v, const char* name, bool output) {
  rtl_status st = check_rows(v, name, output);
  if (st != RTL_OK) return st;
  if (misaligned(v.p) || v.row % 8 != 0) return fail(RTL_ERR_ALIGN, "%s and its rows must be 16-byte aligned", name);
  return RTL_OK;
}

}  // namespace

extern "C" {

size_t rtl_adapters_plan_bytes(int64_t M, int64_t A) { return adapters_fit(M, A) ? rtl::adapters_plan_bytes(M, A) : 0; }

rtl_status rtl_adapters_plan(int64_t M, int64_t A, const int32_t* ids, void* plan, size_t plan_bytes, void* stream) {
  rtl_status st;
  if ((st = check_plan_sizes(M, A)) != RTL_OK) return st;
  if (!ids || !plan) return fail(RTL_ERR_NULL, "ids and the plan are required");
  if ((uintptr_t)ids % 4 != 0 || misaligned(plan)) return fail(RTL_ERR_ALIGN, "the plan must be 16-byte aligned, ids to its elements");
  const size_t need = rtl::adapters_plan_bytes(M, A);
  if (plan_bytes != need) return fail(RTL_ERR_ARG, "the plan needs %zu bytes, got %zu", need, plan_bytes);
  if (overlap(plan, need, ids, (size_t)M * 4)) return fail(RTL_ERR_ARG, "the plan overlaps ids");
  return hip_status(rtl::launch_adapters_plan(ids, M, A, plan, (hipStream_t)stream), "rtl_adapters_plan launch");
}

size_t rtl_adapters_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A) {
  return adapters_fit(M, N, K, R, A) ? rtl::adapters_workspace(M, N, K, R, A) : 0;
}

rtl_status rtl_adapters(rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R, int64_t A, const void* X, int64_t x_row,
                        const void* LA, const void* LB, const float* alpha, const void* plan, size_t plan_bytes,
                        const void* Y0, int64_t y0_row, void* Y, int64_t y_row, float* T, void* workspace, size_t ws_bytes,
                        void* stream) {
  rtl_status st;
  if ((st = check_adapters(dt, M, N, K, R, A, LA, LB, plan, plan_bytes, alpha)) != RTL_OK) return st;
  const View x = rows_of(X, M, K, x_row, 2), y0 = rows_of(Y0, M, N, y0_row, 2), y = rows_of(Y, M, N, y_row, 2);
  if ((st = check_bf16_rows(x, "X", false)) != RTL_OK || (st = check_bf16_rows(y, "Y", true)) != RTL_OK) return st;
  if (Y0 != nullptr && (st = check_bf16_rows(y0, "Y0", false)) != RTL_OK) return st;
  if (misaligned(T) || misaligned(workspace)) return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  const size_t need = rtl::adapters_workspace(M, N, K, R, A), tb = (size_t)M * R * 4;
  const Flat ins[6] = {{LA, (size_t)A * N * R * 2}, {LB, (size_t)A * K * R * 2}, {plan, plan_bytes}, {alpha, (size_t)A * 4},
                       range_of(x), Y0 ? range_of(y0) : Flat{nullptr, 0}};
  const Flat outs[2] = {{T, tb}, {workspace, need}};
  if ((st = check_flat_apart(outs, ins)) != RTL_OK) return st;
  for (const Flat& f : outs)
    if (!apart_flat(y, f.p, f.bytes)) return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
  for (int i = 0; i < 4; i++)
    if (!apart_flat(y, ins[i].p, ins[i].bytes)) return fail(RTL_ERR_ARG, "Y overlaps an input");
  if (!apart(x, y) || (Y0 != nullptr && !y0.same(y) && !apart(y0, y))) return fail(RTL_ERR_ARG, "Y overlaps an input");
  if (!workspace || ws_bytes < need)
    return fail(RTL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : (size_t)0);
  const rtl::AdapterCall c{M, N, K, R, A, X, x.row, LA, LB, plan, alpha};
  return hip_status(rtl::launch_adapters(c, Y0, y0.row, Y, y.row, T, workspace, (hipStream_t)stream), "rtl_adapters launch");
}

size_t rtl_adapters_backward_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A) {
  return adapters_fit(M, N, K, R, A) ? rtl::adapters_back_workspace(M, N, K, R, A) : 0;
}

rtl_status rtl_adapters_backward(rtl_dtype dt, int64_t M, int64_t N, int64_t K, int64_t R, int64_t A, const void* X,
                                 int64_t x_row, const void* LA, const void* LB, const float* alpha, const void* plan,
                                 size_t plan_bytes, const float* T, const void* dY, int64_t dy_row, const void* dX0,
                                 int64_t dx0_row, void* dX, int64_t dx_row, float* dLA, float* dLB, void* workspace,
                                 size_t ws_bytes, void* stream) {
  rtl_status st;
  if ((st = check_adapters(dt, M, N, K, R, A, LA, LB, plan, plan_bytes, alpha)) != RTL_OK) return st;
  if (!dX && !dLA && !dLB) return fail(RTL_ERR_NULL, "one of dX, dLA and dLB is required");
  if (!dX) dX0 = nullptr;
  if (!dLB) X = nullptr;
  if (!dLA) T = nullptr;
  const View x = rows_of(X, M, K, x_row, 2), dy = rows_of(dY, M, N, dy_row, 2), dx0 = rows_of(dX0, M, K, dx0_row, 2),
             dx = rows_of(dX, M, K, dx_row, 2);
  if ((st = check_bf16_rows(dy, "dY", false)) != RTL_OK || (dLB && (st = check_bf16_rows(x, "X", false)) != RTL_OK) ||
      (dX && (st = check_bf16_rows(dx, "dX", true)) != RTL_OK) || (dX0 && (st = check_bf16_rows(dx0, "dX0", false)) != RTL_OK))
    return st;
  if (dLA && !T) return fail(RTL_ERR_NULL, "T is required");
  if (misaligned(T) || misaligned(dLA) || misaligned(dLB) || misaligned(workspace))
    return fail(RTL_ERR_ALIGN, "tensor pointers must be 16-byte aligned");
  const size_t need = rtl::adapters_back_workspace(M, N, K, R, A);
  const Flat none{nullptr, 0};
  const Flat ins[8] = {{LA, (size_t)A * N * R * 2}, {LB, (size_t)A * K * R * 2}, {plan, plan_bytes}, {alpha, (size_t)A * 4},
                       {T, (size_t)M * R * 4}, range_of(dy), X ? range_of(x) : none, dX0 ? range_of(dx0) : none};
  const Flat outs[3] = {{dLA, (size_t)A * N * R * 4}, {dLB, (size_t)A * K * R * 4}, {workspace, need}};
  if ((st = check_flat_apart(outs, ins)) != RTL_OK) return st;
  if (dX != nullptr) {
    for (const Flat& f : outs)
      if (!apart_flat(dx, f.p, f.bytes)) return fail(RTL_ERR_ARG, "outputs overlap each other or the workspace");
    for (int i = 0; i < 5; i++)
      if (!apart_flat(dx, ins[i].p, ins[i].bytes)) return fail(RTL_ERR_ARG, "dX overlaps an input");
    if (!apart(dy, dx) || (X && !apart(x, dx)) || (dX0 && !dx0.same(dx) && !apart(dx0, dx)))
      return fail(RTL_ERR_ARG, "dX overlaps an input");
  }
  if (!workspace || ws_bytes < need)
    return fail(RTL_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace ? ws_bytes : (size_t)0);
  const rtl::AdapterCall c{M, N, K, R, A, X, x.row, LA, LB, plan, alpha};
  return hip_status(rtl::launch_adapters_back(c, T, dY, dy.row, dX0, dx0.row, dX, dx.row, dLA, dLB, workspace, (hipStream_t)stream),
                    "rtl_adapters_backward launch");
}

}  // extern "C"

namespace {

// Memory ranges of a list of tensors, sorted, so that one pass finds those that overlap.
struct Range {
  uintptr_t from, to;
  bool output;
  bool operator<(const Range& o) const { return from < o.from; }
};

}  // namespace

extern "C" {

rtl_status rtl_adamw(rtl_dtype p_dt, rtl_dtype g_dt, rtl_states states, int64_t count, const rtl_adamw_tensor* tensors,
                     int64_t step, const int64_t* step_at, double lr, const float* lr_at, double beta1, double beta2,
                     double eps, double weight_decay, const float* grad_scale, void* stream) {
  rtl_status st;
  if ((st = check_dtype(p_dt)) != RTL_OK || (st = check_dtype(g_dt)) != RTL_OK) return st;
  if (states != RTL_STATES_8 && states != RTL_STATES_32) return fail(RTL_ERR_UNSUPPORTED, "unsupported states %d", (int)states);
  if (count <= 0 || count > 1 << 20) return fail(RTL_ERR_SHAPE, "need 1 to 2^20 tensors (%lld)", (long long)count);
  if (!tensors) return fail(RTL_ERR_NULL, "tensors is required");
  if (!step_at && step < 1) return fail(RTL_ERR_ARG, "step counts from 1 (got %lld)", (long long)step);
  if ((!lr_at && !std::isfinite((float)lr)) || !std::isfinite((float)weight_decay) || !(beta1 >= 0 && (float)beta1 < 1) || !(beta2 >= 0 && (float)beta2 < 1) ||
      !(eps >= 0 && eps <= 1))
    return fail(RTL_ERR_ARG, "need finite lr and weight_decay, betas in [0, 1), eps in [0, 1] (lr=%g betas=%g,%g eps=%g decay=%g)", lr,
                beta1, beta2, eps, weight_decay);
  if ((uintptr_t)step_at % 8 != 0 || (uintptr_t)lr_at % 4 != 0 || (uintptr_t)grad_scale % 4 != 0)
    return fail(RTL_ERR_ALIGN, "step_at, lr_at and grad_scale must be aligned to their elements");
  const bool eight = states == RTL_STATES_8, bf16 = p_dt == RTL_BF16;
  const size_t ps = elem_size(p_dt), gs = elem_size(g_dt), ss = eight ? 1 : 4;
  for (int64_t i = 0; i < count; i++) {
    const rtl_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.n > rtl::kAdamMaxN) return fail(RTL_ERR_SHAPE, "tensor %lld has %lld elements", (long long)i, (long long)t.n);
    if (t.n == 0) continue;
    if (!t.p || !t.g || !t.m || !t.v || bf16 != (t.master != nullptr) || eight != (t.m_scale != nullptr) ||
        eight != (t.v_scale != nullptr))
      return fail(RTL_ERR_NULL, "tensor %lld needs p, g, m, v, a master beside bf16 parameters alone and scales beside 8-bit states alone",
                  (long long)i);
    if (misaligned(t.p) || misaligned(t.g) || misaligned(t.master) || misaligned(t.m) || misaligned(t.v) ||
        (uintptr_t)t.m_scale % 4 != 0 || (uintptr_t)t.v_scale % 4 != 0)
      return fail(RTL_ERR_ALIGN, "tensor %lld must be 16-byte aligned", (long long)i);
  }
  Range* all = (Range*)malloc(sizeof(Range) * (size_t)(7 * count + 3));
  if (all == nullptr) return fail(RTL_ERR_HIP, "no host memory for %lld tensors", (long long)count);
  size_t k = 0;
  auto add = [&](const void* p, size_t bytes, bool output) {
    if (p != nullptr && bytes > 0) all[k++] = Range{(uintptr_t)p, (uintptr_t)p + bytes, output};
  };
  for (int64_t i = 0; i < count; i++) {
    const rtl_adamw_tensor& t = tensors[i];
    const size_t n = (size_t)t.n, blocks = (n + 255) / 256 * 4;
    add(t.p, n * ps, true);
    add(t.g, n * gs, false);
    add(t.master, bf16 ? n * 4 : 0, true);
    add(t.m, n * ss, true);
    add(t.v, n * ss, true);
    add(t.m_scale, eight ? blocks : 0, true);
    add(t.v_scale, eight ? blocks : 0, true);
  }
  add(step_at, 8, false);
  add(lr_at, 4, false);
  add(grad_scale, 4, false);
  std::sort(all, all + k);
  uintptr_t end = 0, out_end = 0;
  bool clash = false;
  for (size_t i = 0; i < k; i++) {
    clash |= all[i].from < (all[i].output ? end : out_end);
    end = std::max(end, all[i].to);
    if (all[i].output) out_end = std::max(out_end, all[i].to);
  }
  free(all);
  if (clash) return fail(RTL_ERR_ARG, "tensors overlap each other");
  rtl::AdamRates r{};
  r.beta1 = beta1;
  r.beta2 = beta2;
  r.step_at = step_at;
  r.lr_at = lr_at;
  r.grad_scale = grad_scale;
  r.lr = (float)lr;
  r.c1 = (float)(1.0 - beta1);
  r.b2 = (float)beta2;
  r.c2 = (float)(1.0 - beta2);
  if (!step_at) {
    r.m_up = (float)(1.0 / (1.0 - std::pow(beta1, (double)step)));
    r.u_up = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  }
  r.eps = (float)eps;
  r.decay = (float)weight_decay;
  static_assert(sizeof(rtl::AdamTensor) == sizeof(rtl_adamw_tensor), "one layout");
  return hip_status(rtl::launch_adamw(bf16, g_dt == RTL_BF16, eight, reinterpret_cast<const rtl::AdamTensor*>(tensors), count, r,
                                      (hipStream_t)stream),
                    "rtl_adamw launch");
}

}  // extern "C"
