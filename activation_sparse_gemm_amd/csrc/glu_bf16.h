// glu_bf16.h -- the gated feed-forward block's projections, activation and product in one
// kernel, and their gradient (bf16, compiled into mlp_bf16.hip's unit):
//
//   G = X Wg^T,  U = X Wu^T,  Y = act(G) U           act: SiLU g / (1 + exp(-g)), or exact GELU
//   dG = dY U act'(G),  dU = dY act(G),  dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X
//
// Forward, many rows: one matrix product over both weights.  A workgroup's tile holds the gate
// and the up columns of the same outputs, placed so that each lane's accumulators hold G and U
// of the same four consecutive columns; the activation and the product are formed from the
// fp32 accumulators and G and U reach memory only where the caller keeps them.
// Forward, few rows: both weights are streamed once, the K range split over a workgroup's
// waves and added in LDS.
#pragma once
#include "gemm_common.h"

namespace rtl {

struct GluArgs {
  int64_t M, K, H;
  const uint16_t *X, *Wg, *Wu;
  uint16_t *Y, *G, *U;  // G, U: null unless kept
  int tiles_m, tiles_n;
};

template <int ACT>
__device__ __forceinline__ float glu_act(float g) {
  return ACT == kActSilu ? g / (1.f + __expf(-g)) : gelu_erf(g);
}
// act(g) and act'(g).
template <int ACT>
__device__ __forceinline__ void glu_act_slope(float g, float& v, float& d) {
  if (ACT == kActSilu) {
    const float p = 1.f / (1.f + __expf(-g));
    v = g * p;
    d = p * (1.f + g * (1.f - p));
  } else {
    const float p = 0.5f * (1.f + erff(g * 0.70710678118654752f));
    v = g * p;
    d = p + g * (0.39894228040143268f * __expf(-0.5f * g * g));
  }
}

// Four consecutive values of row `row` from column `col` on, rounded to bf16 (nearest even).
__device__ __forceinline__ void store4(uint16_t* Y, int64_t M, int64_t N, int64_t row, int64_t col, const float (&v)[4]) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const uint32_t w0 = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[0], (__bf16)v[1]});
  const uint32_t w1 = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[2], (__bf16)v[3]});
  if (row >= M) return;
  uint16_t* y = Y + row * N + col;
  if ((N & 3) == 0 && col + 4 <= N) {
    __builtin_nontemporal_store(u32x2{w0, w1}, reinterpret_cast<u32x2*>(y));
  } else {
    const uint32_t w[2] = {w0, w1};
#pragma unroll
    for (int e = 0; e < 4; e++)
      if (col + e < N) y[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// The tiled product: WM x WN waves, each on 16 RB rows and 64 gate + 64 up columns, K in steps
// of 64.  X and weight tiles go straight to LDS (two buffers): step kt's loads are waited for
// before its barrier, step kt + 1's are issued right after it, into the buffer that every wave
// has finished with.
//
// LDS row n of a wave column's 128 weight rows: gate for n < 64, up for the rest; row 16 nb +
// r16 of either half is output column 4 r16 + nb, so that lane r16 holds four consecutive
// columns over the blocks nb = 0..3.
template <int ACT, int WM, int WN, int RB>
__global__ __launch_bounds__(64 * WM * WN) void glu_kernel(const GluArgs a) {
  constexpr int NW = WM * WN, BM = 16 * RB * WM, BN = 128 * WN, NB = 8;
  constexpr int ABLK = BM / 8, LD = (BM + BN) / 8 / NW;  // 8-row blocks of the X tile; loads per wave and step
  constexpr int STAGE = (BM + BN) * 128;
  static_assert(ABLK % NW == 0 && 8 % NW == 0 && LD * NW * 8 == BM + BN, "whole blocks per wave");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * STAGE];

  int tm, tn;
  tile_coords(a.tiles_m, a.tiles_n, tm, tn);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int q = lane >> 4, r16 = lane & 15;
  const int64_t M = a.M, K = a.K, H = a.H;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * (BN / 2);
  const int KT = (int)(K / kBK);

  // Rows past M or H lie outside the buffers and read as zeros.
  const __amdgpu_buffer_rsrc_t xres = make_rsrc(a.X + m0 * K, (M - m0) * K * 2);
  const __amdgpu_buffer_rsrc_t gres = make_rsrc(a.Wg + n0 * K, (H - n0) * K * 2);
  const __amdgpu_buffer_rsrc_t ures = make_rsrc(a.Wu + n0 * K, (H - n0) * K * 2);
  // Lane l of a load writes 16-byte position l % 8 of row l / 8 of its 8-row block, where
  // sw_off keeps chunk (l % 8) ^ (l / 8).
  const int row8 = lane >> 3;
  const uint32_t chunk = 16 * ((lane & 7) ^ row8);
  const uint32_t a_voff = (uint32_t)(row8 * K * 2) + chunk, b_voff = (uint32_t)(4 * row8 * K * 2) + chunk;
  auto load = [&](int kt, int buf) {
#pragma unroll
    for (int i = 0; i < LD; i++) {
      auto* dst = (__attribute__((address_space(3))) void*)(lds + buf * STAGE + (i * NW + wave) * 1024);
      if (i * NW < ABLK) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(xres, dst, 16, a_voff,
                                                 (int)((int64_t)(i * NW + wave) * 8 * K * 2 + (int64_t)kt * 128), 0, 0);
      } else {
        const int n8 = i * NW + wave - ABLK, at = n8 & 7;  // 8-row block among the weight rows, within its half
        const int64_t col = 64 * (n8 >> 4) + 32 * (at & 1) + (at >> 1);
        const bool up = ((i * NW - ABLK) >> 3) & 1;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(up ? ures : gres, dst, 16, b_voff,
                                                 (int)(col * K * 2 + (int64_t)kt * 128), 0, 0);
      }
    }
  };

  f32x4 acc[RB][NB];
#pragma unroll
  for (int rb = 0; rb < RB; rb++)
#pragma unroll
    for (int nb = 0; nb < NB; nb++) acc[rb][nb] = f32x4{0.f, 0.f, 0.f, 0.f};

  load(0, 0);
  for (int kt = 0; kt < KT; kt++) {
    const int buf = kt & 1;
    wait_vmcnt<0>();
    barrier_nofence();
    if (kt + 1 < KT) load(kt + 1, buf ^ 1);
    const uint8_t* al = lds + buf * STAGE;
    const uint8_t* bl = al + BM * 128;
#pragma unroll
    for (int kk = 0; kk < 2; kk++) {
      u32x4 av[RB];
#pragma unroll
      for (int rb = 0; rb < RB; rb++)
        av[rb] = *reinterpret_cast<const u32x4*>(al + sw_off(16 * RB * wm + 16 * rb + r16, 4 * kk + q));
#pragma unroll
      for (int nb = 0; nb < NB; nb++) {
        const u32x4 bv = *reinterpret_cast<const u32x4*>(bl + sw_off(128 * wn + 16 * nb + r16, 4 * kk + q));
#pragma unroll
        for (int rb = 0; rb < RB; rb++)
          acc[rb][nb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, av[rb]), __builtin_bit_cast(bf16x8, bv), acc[rb][nb], 0, 0, 0);
      }
    }
  }

  const int64_t col = n0 + 64 * wn + 4 * r16;
#pragma unroll
  for (int rb = 0; rb < RB; rb++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t row = m0 + 16 * RB * wm + 16 * rb + 4 * q + j;
      float g[4], u[4], y[4];
#pragma unroll
      for (int e = 0; e < 4; e++) {
        g[e] = acc[rb][e][j];
        u[e] = acc[rb][4 + e][j];
        y[e] = glu_act<ACT>(g[e]) * u[e];
      }
      store4(a.Y, M, H, row, col, y);
      if (a.G != nullptr) store4(a.G, M, H, row, col, g);
      if (a.U != nullptr) store4(a.U, M, H, row, col, u);
    }
}

// Few rows (M <= 16 MB): a workgroup of NW waves forms 16 output columns; wave w takes the K
// steps w, w + NW, ..., each lane loading 16-byte chunks of its weight row straight into the
// MFMA's operand order, and the waves' partial sums are added in LDS in wave order.  Bound by
// the weights' bytes.
template <int ACT, int MB, int NW>
__global__ __launch_bounds__(64 * NW) void glu_rows_kernel(const GluArgs a) {
  __shared__ f32x4 red[NW][2 * MB][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int64_t M = a.M, K = a.K, H = a.H, n0 = (int64_t)blockIdx.x * 16;
  const int KT = (int)(K / kBK);
  const __amdgpu_buffer_rsrc_t xres = make_rsrc(a.X, M * K * 2);
  const __amdgpu_buffer_rsrc_t gres = make_rsrc(a.Wg + n0 * K, (H - n0) * K * 2);
  const __amdgpu_buffer_rsrc_t ures = make_rsrc(a.Wu + n0 * K, (H - n0) * K * 2);
  const uint32_t voff = (uint32_t)(r16 * K * 2 + 16 * q);
  f32x4 acc[2][MB];
#pragma unroll
  for (int p = 0; p < 2; p++)
#pragma unroll
    for (int mb = 0; mb < MB; mb++) acc[p][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
  // UN K steps at a time: every load of the batch is issued before the first product.
  auto batch = [&](int s0, auto un) {
    constexpr int UN = decltype(un)::value;
    u32x4 w[UN][2][2], x[UN][MB][2];
#pragma unroll
    for (int i = 0; i < UN; i++)
#pragma unroll
      for (int kk = 0; kk < 2; kk++) {
        const int at = (s0 + i * NW) * 128 + 64 * kk;
        w[i][0][kk] = __builtin_amdgcn_raw_buffer_load_b128(gres, voff, at, 0);
        w[i][1][kk] = __builtin_amdgcn_raw_buffer_load_b128(ures, voff, at, 0);
#pragma unroll
        for (int mb = 0; mb < MB; mb++)
          x[i][mb][kk] = __builtin_amdgcn_raw_buffer_load_b128(xres, voff, (int)(16 * mb * K * 2) + at, 0);
      }
#pragma unroll
    for (int i = 0; i < UN; i++)
#pragma unroll
      for (int kk = 0; kk < 2; kk++)
#pragma unroll
        for (int p = 0; p < 2; p++)
#pragma unroll
          for (int mb = 0; mb < MB; mb++)
            acc[p][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[i][mb][kk]),
                                                                 __builtin_bit_cast(bf16x8, w[i][p][kk]), acc[p][mb],
                                                                 0, 0, 0);
  };
  constexpr int UN = MB == 1 ? 4 : 2;
  int s = wave;
  for (; s + (UN - 1) * NW < KT; s += UN * NW) batch(s, std::integral_constant<int, UN>());
  for (; s < KT; s += NW) batch(s, std::integral_constant<int, 1>());
#pragma unroll
  for (int p = 0; p < 2; p++)
#pragma unroll
    for (int mb = 0; mb < MB; mb++) red[wave][p * MB + mb][lane] = acc[p][mb];
  __syncthreads();
  for (int mb = wave; mb < MB; mb += NW) {
    f32x4 g = red[0][mb][lane], u = red[0][MB + mb][lane];
    for (int w = 1; w < NW; w++) {
      g += red[w][mb][lane];
      u += red[w][MB + mb][lane];
    }
    const int64_t col = n0 + r16;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t row = 16 * mb + 4 * q + j;
      if (row >= M || col >= H) continue;
      a.Y[row * H + col] = (uint16_t)f32_to_bf16_bits(glu_act<ACT>(g[j]) * u[j]);
      if (a.G != nullptr) a.G[row * H + col] = (uint16_t)f32_to_bf16_bits(g[j]);
      if (a.U != nullptr) a.U[row * H + col] = (uint16_t)f32_to_bf16_bits(u[j]);
    }
  }
}

namespace {

template <int ACT, int WM, int WN, int RB>
void glu_tiles(GluArgs a, hipStream_t stream) {
  constexpr int BM = 16 * RB * WM, BH = 64 * WN;
  a.tiles_m = (int)((a.M + BM - 1) / BM);
  a.tiles_n = (int)((a.H + BH - 1) / BH);
  hipLaunchKernelGGL((glu_kernel<ACT, WM, WN, RB>), dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(64 * WM * WN), 0,
                     stream, a);
}

template <int ACT>
void glu_launch(const GluArgs& a, hipStream_t stream) {
  const dim3 cols((unsigned)((a.H + 15) / 16)), block(512);
  if (a.M <= 16) hipLaunchKernelGGL((glu_rows_kernel<ACT, 1, 8>), cols, block, 0, stream, a);
  else if (a.M <= 32) hipLaunchKernelGGL((glu_rows_kernel<ACT, 2, 8>), cols, block, 0, stream, a);
  else if (((a.M + 255) / 256) * ((a.H + 127) / 128) >= 256) glu_tiles<ACT, 4, 2, 4>(a, stream);
  else if (((a.M + 127) / 128) * ((a.H + 127) / 128) >= 256) glu_tiles<ACT, 2, 2, 4>(a, stream);
  else glu_tiles<ACT, 2, 1, 4>(a, stream);
}

}  // namespace

hipError_t launch_glu_bf16(int act, int64_t M, int64_t K, int64_t H, const void* X, const void* Wg, const void* Wu,
                           void* Y, void* G, void* U, hipStream_t stream) {
  GluArgs a{};
  a.M = M; a.K = K; a.H = H;
  a.X = (const uint16_t*)X; a.Wg = (const uint16_t*)Wg; a.Wu = (const uint16_t*)Wu;
  a.Y = (uint16_t*)Y; a.G = (uint16_t*)G; a.U = (uint16_t*)U;
  if (act == kActSilu) glu_launch<kActSilu>(a, stream);
  else glu_launch<kActGelu>(a, stream);
  return hipGetLastError();
}

// ------------------------------------------------------------------ gradient

// Transpose of a 64 x 64 tile: src [rows, cols] -> dst [cols, ld] at column at0 on; rows of
// src past `rows` (up to the tile's end) are written as zeros.
__global__ __launch_bounds__(256) void glu_transpose_kernel(const uint16_t* src, int64_t rows, int64_t cols,
                                                            uint16_t* dst, int64_t ld, int64_t at0) {
  __shared__ uint16_t tile[64][66];
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  for (int i = y; i < 64; i += 4)
    tile[i][x] = r0 + i < rows && c0 + x < cols ? src[(r0 + i) * cols + c0 + x] : (uint16_t)0;
  __syncthreads();
  for (int i = y; i < 64; i += 4)
    if (c0 + i < cols) dst[(c0 + i) * ld + at0 + r0 + x] = tile[x][i];
}

// dG and dU of a 64 x 64 tile, rounded to bf16 (they are the matrix cores' operands), as rows
// P [M, 2 Hp] (dU from column Hp on) and transposed, [H, Mp] each; zeros in the padding.
template <int ACT>
__global__ __launch_bounds__(256) void glu_back_kernel(int64_t M, int64_t H, const uint16_t* G, const uint16_t* U,
                                                       const uint16_t* dY, uint16_t* P, int64_t Hp, uint16_t* dGt,
                                                       uint16_t* dUt, int64_t Mp) {
  __shared__ uint16_t tg[64][66], tu[64][66];
  const int64_t r0 = (int64_t)blockIdx.x * 64, c0 = (int64_t)blockIdx.y * 64;
  const int x = threadIdx.x & 63, y = threadIdx.x >> 6;
  for (int i = y; i < 64; i += 4) {
    uint16_t dg = 0, du = 0;
    if (r0 + i < M && c0 + x < H) {
      const int64_t at = (r0 + i) * H + c0 + x;
      const float g = __uint_as_float((uint32_t)G[at] << 16), u = __uint_as_float((uint32_t)U[at] << 16);
      const float d = __uint_as_float((uint32_t)dY[at] << 16);
      float v, s;
      glu_act_slope<ACT>(g, v, s);
      dg = (uint16_t)f32_to_bf16_bits(d * u * s);
      du = (uint16_t)f32_to_bf16_bits(d * v);
    }
    tg[i][x] = dg;
    tu[i][x] = du;
    if (P != nullptr && r0 + i < M) {
      P[(r0 + i) * 2 * Hp + c0 + x] = dg;
      P[(r0 + i) * 2 * Hp + Hp + c0 + x] = du;
    }
  }
  if (dGt == nullptr) return;
  __syncthreads();
  for (int i = y; i < 64; i += 4)
    if (c0 + i < H) {
      dGt[(c0 + i) * Mp + r0 + x] = tg[x][i];
      dUt[(c0 + i) * Mp + r0 + x] = tu[x][i];
    }
}

namespace {
inline int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }
struct GluBackLayout {
  size_t p, wt, dgt, dut, xt, total;
};
GluBackLayout glu_back_layout(int64_t M, int64_t K, int64_t H) {
  GluBackLayout L;
  const int64_t Hp = pad64(H), Mp = pad64(M);
  L.p = 0;
  L.wt = L.p + align256((size_t)(M * 2 * Hp * 2));
  L.dgt = L.wt + align256((size_t)(K * 2 * Hp * 2));
  L.dut = L.dgt + align256((size_t)(H * Mp * 2));
  L.xt = L.dut + align256((size_t)(H * Mp * 2));
  L.total = L.xt + align256((size_t)(K * Mp * 2));
  return L;
}
}  // namespace

size_t glu_back_workspace(int64_t M, int64_t K, int64_t H) { return glu_back_layout(M, K, H).total; }

hipError_t launch_glu_back_bf16(int act, int64_t M, int64_t K, int64_t H, const void* X, const void* Wg,
                                const void* Wu, const void* G, const void* U, const void* dY, void* dX, void* dWg,
                                void* dWu, void* ws, hipStream_t stream) {
  const bool want_dx = dX != nullptr, want_dw = dWg != nullptr;
  const GluBackLayout L = glu_back_layout(M, K, H);
  const int64_t Hp = pad64(H), Mp = pad64(M);
  uint8_t* b = (uint8_t*)ws;
  uint16_t *P = want_dx ? (uint16_t*)(b + L.p) : nullptr, *wt = (uint16_t*)(b + L.wt);
  uint16_t *dgt = want_dw ? (uint16_t*)(b + L.dgt) : nullptr, *dut = (uint16_t*)(b + L.dut);
  uint16_t* xt = (uint16_t*)(b + L.xt);
  const dim3 block(256), tiles((unsigned)(Mp / 64), (unsigned)(Hp / 64));
  if (act == kActSilu)
    hipLaunchKernelGGL((glu_back_kernel<kActSilu>), tiles, block, 0, stream, M, H, (const uint16_t*)G,
                       (const uint16_t*)U, (const uint16_t*)dY, P, Hp, dgt, dut, Mp);
  else
    hipLaunchKernelGGL((glu_back_kernel<kActGelu>), tiles, block, 0, stream, M, H, (const uint16_t*)G,
                       (const uint16_t*)U, (const uint16_t*)dY, P, Hp, dgt, dut, Mp);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (want_dx) {
    const dim3 wtiles((unsigned)(Hp / 64), (unsigned)(K / 64));
    hipLaunchKernelGGL(glu_transpose_kernel, wtiles, block, 0, stream, (const uint16_t*)Wg, H, K, wt, 2 * Hp,
                       (int64_t)0);
    hipLaunchKernelGGL(glu_transpose_kernel, wtiles, block, 0, stream, (const uint16_t*)Wu, H, K, wt, 2 * Hp, Hp);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = launch_dense_bf16(M, K, 2 * Hp, P, wt, dX, stream)) != hipSuccess) return e;
  }
  if (want_dw) {
    hipLaunchKernelGGL(glu_transpose_kernel, dim3((unsigned)(Mp / 64), (unsigned)(K / 64)), block, 0, stream,
                       (const uint16_t*)X, M, K, xt, Mp, (int64_t)0);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if ((e = launch_dense_bf16(H, K, Mp, dgt, xt, dWg, stream)) != hipSuccess) return e;
    if ((e = launch_dense_bf16(H, K, Mp, dut, xt, dWu, stream)) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rtl
