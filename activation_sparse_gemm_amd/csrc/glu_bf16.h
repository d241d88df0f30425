// glu_bf16.h -- the gated feed-forward block's projections, activation and product in one
// kernel, and their gradient (bf16, compiled into mlp_bf16.hip's unit):
//
//   G = X Wg^T,  U = X Wu^T,  Y = act(G) U           act: SiLU g / (1 + exp(-g)), or exact GELU
//   dG = dY U act'(G),  dU = dY act(G),  dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X
//
// Forward, many rows: one matrix product over both weights (ring_gemm.h).  A workgroup's tile
// holds the gate and the up columns of the same outputs, placed so that each lane's
// accumulators hold G and U of the same consecutive columns; the activation and the product are
// formed from the fp32 accumulators and G and U reach memory only where the caller keeps them.
// Forward, few rows: both weights are streamed once, the K range split over a workgroup's
// waves and added in LDS.
// Gradient: one pass forms P = [dG | dU], then dX = P [Wg; Wu] and [dWg; dWu] = P^T X read P, X
// and the weights as they lie (ring_gemm.h's transposing reads).
#pragma once
#include "ring_gemm.h"

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

// N (2 or 4) consecutive values of row `row` from column `col` on, rounded to bf16 (nearest even).
template <int N>
__device__ __forceinline__ void store_cols(uint16_t* Y, int64_t M, int64_t H, int64_t row, int64_t col,
                                           const float (&v)[N]) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; i++)
    w[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
  if (row >= M) return;
  uint16_t* y = Y + row * H + col;
  if (H % N == 0 && col + N <= H) {
    if constexpr (N == 4) __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2*>(y));
    else *reinterpret_cast<uint32_t*>(y) = w[0];
  } else {
#pragma unroll
    for (int e = 0; e < N; e++)
      if (col + e < H) y[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  }
}

// Buffer resource of `bytes` (as make_rsrc clamps them), or of none: loads then read zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_if(bool live, const void* p, int64_t bytes) {
  return make_rsrc(p, live ? bytes : 0);
}

// The tiled product: 2 x 2 waves of RB x NB blocks, 32 RB rows and 32 NB weight rows (16 NB
// outputs) a tile.  Of a wave column's 16 NB weight rows the first half are gate rows, the
// second up; row 16 nb + r16 of either half is output column NB / 2 r16 + nb, so that lane r16
// holds NB / 2 consecutive columns over its blocks.
template <int ACT, int RB, int NB>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(RB == 8 ? 1 : 2, RB == 8 ? 1 : 2)))
void glu_kernel(const GluArgs a) {
  constexpr int BM = 32 * RB, BN = 32 * NB, NC = NB / 2;
  typedef KRows<BM> OpA;
  typedef KRows<BN> OpB;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kSlots * OpA::kBytes];
  int tm, tn;
  tile_coords(a.tiles_m, a.tiles_n, tm, tn);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int q = lane >> 4, r16 = lane & 15;
  const int64_t M = a.M, K = a.K, H = a.H;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * (BN / 2);
  const int steps = (int)(K / kRK);
  // Rows past M or H lie outside the buffers and read as zeros.
  const uint16_t *X = a.X + m0 * K, *Wg = a.Wg + n0 * K, *Wu = a.Wu + n0 * K;
  const int64_t xb = (M - m0) * K * 2, wb = (H - n0) * K * 2;
  const OpA oa(K, 1, wave, lane);
  const OpB ob(K, NC, wave, lane);
  auto load_a = [&](int kt, uint8_t* dst, int i) {
    oa.load(rsrc_if(kt >= 0, X, xb), dst, i, 8 * (i * kRingWaves + wave), kt < 0 ? 0 : kt);
  };
  auto load_b = [&](int kt, uint8_t* dst, int i) {
    const int blk = i * kRingWaves + wave, at = blk % (2 * NB);  // 8-row block, and within its wave column
    const bool up = at >= NB;
    const int of = up ? at - NB : at;  // half `of & 1` of block nb = of / 2
    ob.load(rsrc_if(kt >= 0, up ? Wu : Wg, wb), dst, i, blk / (2 * NB) * (16 * NC) + (of & 1) * (8 * NC) + (of >> 1),
            kt < 0 ? 0 : kt);
  };
  f32x4 acc[RB][NB];
  ring_product(acc, lds, oa, ob, load_a, load_b, steps, (tm + tn) % 8 % steps, wm, wn);

  const int64_t col = n0 + 16 * NC * wn + NC * r16;
#pragma unroll
  for (int rb = 0; rb < RB; rb++)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t row = m0 + 16 * (RB * wm + rb) + 4 * q + j;
      float g[NC], u[NC], y[NC];
#pragma unroll
      for (int e = 0; e < NC; e++) {
        g[e] = acc[rb][e][j];
        u[e] = acc[rb][NC + e][j];
        y[e] = glu_act<ACT>(g[e]) * u[e];
      }
      store_cols<NC>(a.Y, M, H, row, col, y);
      if (a.G != nullptr) store_cols<NC>(a.G, M, H, row, col, g);
      if (a.U != nullptr) store_cols<NC>(a.U, M, H, row, col, u);
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

// Tiles of 32 R rows by 16 R outputs.
template <int ACT, int R>
void glu_tiles(GluArgs a, hipStream_t stream) {
  a.tiles_m = (int)((a.M + 32 * R - 1) / (32 * R));
  a.tiles_n = (int)((a.H + 16 * R - 1) / (16 * R));
  hipLaunchKernelGGL((glu_kernel<ACT, R, R>), dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(256), 0, stream, a);
}

template <int ACT>
void glu_launch(const GluArgs& a, hipStream_t stream) {
  const dim3 cols((unsigned)((a.H + 15) / 16)), block(512);
  if (a.M <= 16) hipLaunchKernelGGL((glu_rows_kernel<ACT, 1, 8>), cols, block, 0, stream, a);
  else if (a.M <= 32) hipLaunchKernelGGL((glu_rows_kernel<ACT, 2, 8>), cols, block, 0, stream, a);
  else if (((a.M + 255) / 256) * ((a.H + 127) / 128) >= 192) glu_tiles<ACT, 8>(a, stream);
  else glu_tiles<ACT, 4>(a, stream);
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

// P [M, 2 Hp] = [dG | dU], each padded to Hp columns with zeros, rounded to bf16: the matrix
// cores' operand.  (Formed inside the products instead, it would be formed again for every
// tile that reads it, 2 H / 256 + K / 256 times.)  One 16-byte chunk of each half per thread.
template <int ACT>
__global__ __launch_bounds__(256) void glu_back_kernel(int64_t M, int64_t H, int64_t Hp, const uint16_t* G,
                                                       const uint16_t* U, const uint16_t* dY, uint16_t* P) {
  const int64_t c8 = Hp / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= M * c8) return;
  const int64_t m = id / c8, h = (id - m * c8) * 8, at = m * H + h;
  u32x4 g{}, u{}, d{};
  if (H % 8 == 0 && h + 8 <= H) {
    g = *reinterpret_cast<const u32x4*>(G + at);
    u = *reinterpret_cast<const u32x4*>(U + at);
    d = *reinterpret_cast<const u32x4*>(dY + at);
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (h + e < H) {
        g[e >> 1] |= (uint32_t)G[at + e] << (16 * (e & 1));
        u[e >> 1] |= (uint32_t)U[at + e] << (16 * (e & 1));
        d[e >> 1] |= (uint32_t)dY[at + e] << (16 * (e & 1));
      }
  }
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  u32x4 dg, du;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    float v0, s0, v1, s1;
    glu_act_slope<ACT>(bf16lo(g[i]), v0, s0);
    glu_act_slope<ACT>(bf16hi(g[i]), v1, s1);
    const float d0 = bf16lo(d[i]), d1 = bf16hi(d[i]);
    dg[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)(d0 * bf16lo(u[i]) * s0), (__bf16)(d1 * bf16hi(u[i]) * s1)});
    du[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)(d0 * v0), (__bf16)(d1 * v1)});
  }
  *reinterpret_cast<u32x4*>(P + m * 2 * Hp + h) = dg;
  *reinterpret_cast<u32x4*>(P + m * 2 * Hp + Hp + h) = du;
}

// A wave's RB x NB blocks to bf16 rows through its LDS block of 16 * (32 NB + 16) bytes, as
// 16-byte chunks; row(i) gives the address of the wave's row i at its first column or null,
// `cols` (a multiple of 8) the columns from there on.
template <int RB, int NB, typename Row>
__device__ __forceinline__ void store_rows(const f32x4 (&acc)[RB][NB], uint8_t* blk, int lane, int64_t cols, Row row) {
  constexpr int CW = NB * 16, PITCH = 2 * CW + 16, CPR = CW / 8;
  const int q = lane >> 4, r16 = lane & 15;
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int rb = 0; rb < RB; rb++) {
#pragma unroll
    for (int nb = 0; nb < NB; nb++)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const uint32_t w = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)acc[rb][nb][j], (__bf16)acc[rb][nb][j + 1]});
        uint8_t* at = blk + (4 * q + j) * PITCH + (nb * 16 + r16) * 2;
        *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
        *reinterpret_cast<uint16_t*>(at + PITCH) = (uint16_t)(w >> 16);
      }
#pragma unroll
    for (int c = 0; c < 16 * CPR / 64; c++) {
      const int id = lane + 64 * c, rr = id / CPR, cc = id % CPR;
      const u32x4 v = *reinterpret_cast<const u32x4*>(blk + rr * PITCH + cc * 16);
      uint16_t* y = row(16 * rb + rr);
      if (y != nullptr && 8 * cc < cols) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y + 8 * cc));
    }
  }
}

struct GluBackArgs {
  int64_t M, K, H, Hp;
  const uint16_t *P, *X, *Wg, *Wu;
  uint16_t *dX, *dWg, *dWu;
  float* part;       // split sum of dX: [splits][M][K]
  int per;           // K steps per split
  int tiles_m, tiles_n;
};

// dX = P [Wg; Wu]: k runs over P's 2 Hp columns, along P's rows and down the weights' columns.
// With SPLIT, blockIdx.y takes `per` of the steps and leaves its fp32 sums in its part.
template <int R, bool SPLIT>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(R == 8 ? 1 : 2, R == 8 ? 1 : 2)))
void glu_dx_kernel(const GluBackArgs a) {
  constexpr int T = 32 * R;
  typedef KRows<T> OpA;
  typedef KCols<T> OpB;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kSlots * OpA::kBytes];
  int tm, tn;
  tile_coords(a.tiles_m, a.tiles_n, tm, tn);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int64_t M = a.M, K = a.K, H = a.H, ld = 2 * a.Hp;
  const int64_t m0 = (int64_t)tm * T, c0 = (int64_t)tn * T;
  const int half = (int)(a.Hp / kRK), all = 2 * half;
  const int first = SPLIT ? blockIdx.y * a.per : 0, steps = SPLIT ? min(a.per, all - first) : all;
  const uint16_t* P = a.P + m0 * ld;
  const OpA oa(ld, 1, wave, lane);
  const OpB ob(K, wave, lane);
  auto load_a = [&](int kt, uint8_t* dst, int i) {
    oa.load(rsrc_if(kt >= 0, P, (M - m0) * ld * 2), dst, i, 8 * (i * kRingWaves + wave), kt < 0 ? 0 : first + kt);
  };
  auto load_b = [&](int kt, uint8_t* dst, int i) {
    // rows of Wg, then of Wu; past H (P's padding) they read as zeros
    const int s = first + (kt < 0 ? 0 : kt);
    const int64_t h = (int64_t)(s < half ? s : s - half) * kRK;
    ob.load(rsrc_if(kt >= 0, (s < half ? a.Wg : a.Wu) + h * K + c0, ((H - h) * K - c0) * 2), dst, i);
  };
  f32x4 acc[R][R];
  ring_product(acc, lds, oa, ob, load_a, load_b, steps, (tm + tn) % 8 % steps, wm, wn);

  const int64_t row0 = m0 + 16 * R * wm, col0 = c0 + 16 * R * wn;
  if constexpr (SPLIT) {
    float* out = a.part + (int64_t)blockIdx.y * M * K;
    const int q = lane >> 4, r16 = lane & 15;
#pragma unroll
    for (int rb = 0; rb < R; rb++)
#pragma unroll
      for (int nb = 0; nb < R; nb++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const int64_t row = row0 + 16 * rb + 4 * q + j, col = col0 + 16 * nb + r16;
          if (row < M && col < K) out[row * K + col] = acc[rb][nb][j];
        }
  } else {
    __syncthreads();  // the ring is free
    store_rows<R, R>(acc, lds + wave * 16 * (32 * R + 16), lane, K - col0, [&](int i) {
      return row0 + i < M ? a.dX + (row0 + i) * K + col0 : (uint16_t*)nullptr;
    });
  }
}

// dX = the splits' sum in order, four values per thread (K % 64 == 0).
__global__ __launch_bounds__(256) void glu_sum_kernel(const float* part, int splits, int64_t n, uint16_t* dX) {
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= n) return;
  f32x4 s = *reinterpret_cast<const f32x4*>(part + at);
  for (int k = 1; k < splits; k++) s += *reinterpret_cast<const f32x4*>(part + (int64_t)k * n + at);
  *reinterpret_cast<u32x2*>(dX + at) = u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
}

// [dWg; dWu] = P^T X: k runs over the tokens, down the columns of both.
template <int R>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(R == 8 ? 1 : 2, R == 8 ? 1 : 2)))
void glu_dw_kernel(const GluBackArgs a) {
  constexpr int T = 32 * R;
  typedef KCols<T> Op;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kSlots * Op::kBytes];
  int tm, tn;
  tile_coords(a.tiles_m, a.tiles_n, tm, tn);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int64_t M = a.M, K = a.K, H = a.H, Hp = a.Hp, ld = 2 * Hp;
  const int64_t r0 = (int64_t)tm * T, c0 = (int64_t)tn * T;
  const int steps = (int)((M + kRK - 1) / kRK);
  const Op oa(ld, wave, lane), ob(K, wave, lane);
  // tokens past M lie outside the buffers and read as zeros
  auto load_a = [&](int kt, uint8_t* dst, int i) {
    const int64_t m = (int64_t)(kt < 0 ? 0 : kt) * kRK;
    oa.load(rsrc_if(kt >= 0, a.P + m * ld + r0, ((M - m) * ld - r0) * 2), dst, i);
  };
  auto load_b = [&](int kt, uint8_t* dst, int i) {
    const int64_t m = (int64_t)(kt < 0 ? 0 : kt) * kRK;
    ob.load(rsrc_if(kt >= 0, a.X + m * K + c0, ((M - m) * K - c0) * 2), dst, i);
  };
  f32x4 acc[R][R];
  ring_product(acc, lds, oa, ob, load_a, load_b, steps, (tm + tn) % 8 % steps, wm, wn);

  __syncthreads();  // the ring is free
  const int64_t row0 = r0 + 16 * R * wm, col0 = c0 + 16 * R * wn;
  store_rows<R, R>(acc, lds + wave * 16 * (32 * R + 16), lane, K - col0, [&](int i) {
    const int64_t r = row0 + i;  // 0 .. H - 1: a row of dWg; Hp .. Hp + H - 1: of dWu
    return r < H ? a.dWg + r * K + col0 : r >= Hp && r < Hp + H ? a.dWu + (r - Hp) * K + col0 : (uint16_t*)nullptr;
  });
}

namespace {
inline int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// dX: 256 x 256 tiles where they occupy three quarters of the CUs; else 128 x 128 tiles, and
// where those do not give every CU its two workgroups, the sum over the 2 Hp columns is split,
// in parts of at least 16 steps.
struct GluDxPlan {
  int splits, per;
  bool big;
};
GluDxPlan glu_dx_plan(int64_t M, int64_t K, int64_t H) {
  const int64_t steps = 2 * pad64(H) / kRK;
  if (((M + 255) / 256) * ((K + 255) / 256) >= 192) return {1, (int)steps, true};
  const int64_t tiles = ((M + 127) / 128) * ((K + 127) / 128);
  const int64_t splits = std::max<int64_t>(1, std::min(512 / tiles, steps / 16));
  const int64_t per = (steps + splits - 1) / splits;
  return {(int)((steps + per - 1) / per), (int)per, false};
}

struct GluBackLayout {
  size_t p, part, total;
};
GluBackLayout glu_back_layout(int64_t M, int64_t K, int64_t H) {
  GluBackLayout L;
  const GluDxPlan d = glu_dx_plan(M, K, H);
  L.p = 0;
  L.part = align256((size_t)(M * 2 * pad64(H) * 2));
  L.total = L.part + (d.splits > 1 ? align256((size_t)d.splits * M * K * 4) : 0);
  return L;
}

template <int R>
void glu_dw_launch(GluBackArgs a, hipStream_t stream) {
  a.tiles_m = (int)((2 * a.Hp + 32 * R - 1) / (32 * R));
  a.tiles_n = (int)((a.K + 32 * R - 1) / (32 * R));
  hipLaunchKernelGGL((glu_dw_kernel<R>), dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(256), 0, stream, a);
}
}  // namespace

size_t glu_back_workspace(int64_t M, int64_t K, int64_t H) { return glu_back_layout(M, K, H).total; }

hipError_t launch_glu_back_bf16(int act, int64_t M, int64_t K, int64_t H, const void* X, const void* Wg,
                                const void* Wu, const void* G, const void* U, const void* dY, void* dX, void* dWg,
                                void* dWu, void* ws, hipStream_t stream) {
  const GluBackLayout L = glu_back_layout(M, K, H);
  GluBackArgs a{};
  a.M = M; a.K = K; a.H = H; a.Hp = pad64(H);
  uint16_t* P = (uint16_t*)((uint8_t*)ws + L.p);
  a.P = P; a.X = (const uint16_t*)X; a.Wg = (const uint16_t*)Wg; a.Wu = (const uint16_t*)Wu;
  a.dX = (uint16_t*)dX; a.dWg = (uint16_t*)dWg; a.dWu = (uint16_t*)dWu;
  a.part = (float*)((uint8_t*)ws + L.part);
  const dim3 block(256), chunks((unsigned)((M * (a.Hp / 8) + 255) / 256));
  if (act == kActSilu)
    hipLaunchKernelGGL((glu_back_kernel<kActSilu>), chunks, block, 0, stream, M, H, a.Hp, (const uint16_t*)G,
                       (const uint16_t*)U, (const uint16_t*)dY, P);
  else
    hipLaunchKernelGGL((glu_back_kernel<kActGelu>), chunks, block, 0, stream, M, H, a.Hp, (const uint16_t*)G,
                       (const uint16_t*)U, (const uint16_t*)dY, P);
  if (dX != nullptr) {
    const GluDxPlan d = glu_dx_plan(M, K, H);
    const int64_t T = d.big ? 256 : 128;
    a.per = d.per;
    a.tiles_m = (int)((M + T - 1) / T);
    a.tiles_n = (int)((K + T - 1) / T);
    const dim3 grid((unsigned)(a.tiles_m * a.tiles_n), (unsigned)d.splits);
    if (d.big) hipLaunchKernelGGL((glu_dx_kernel<8, false>), grid, block, 0, stream, a);
    else if (d.splits == 1) hipLaunchKernelGGL((glu_dx_kernel<4, false>), grid, block, 0, stream, a);
    else {
      hipLaunchKernelGGL((glu_dx_kernel<4, true>), grid, block, 0, stream, a);
      hipLaunchKernelGGL(glu_sum_kernel, dim3((unsigned)((M * K / 4 + 255) / 256)), block, 0, stream, a.part, d.splits,
                         M * K, a.dX);
    }
  }
  if (dWg != nullptr) {
    if (((2 * a.Hp + 255) / 256) * ((K + 255) / 256) >= 192) glu_dw_launch<8>(a, stream);
    else glu_dw_launch<4>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace rtl
