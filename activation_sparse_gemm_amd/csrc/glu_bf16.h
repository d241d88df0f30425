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
// Forward, few rows or few outputs: the K range split over a workgroup's waves and added in LDS.
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

// act(g) and act'(g).  SiLU: g p, p (1 + g (1 - p)) with p = 1 / (1 + exp(-g)).  GELU: g Phi(g),
// Phi(g) + g phi(g), with Phi from Abramowitz and Stegun 7.1.26 (erf within 1.5e-7): for x = |g| /
// sqrt 2, t = 1 / (1 + 0.3275911 x), Phi(-|g|) = (a1 t + .. + a5 t^5) exp(-x^2) / 2, whose exp(-x^2)
// is also that of phi(g).  A fifth of the instructions of the library's erf, which took a sixth
// of a tile's time at K = 2560.  Relative to Phi(g) itself it is within 6e-5 to g = -3, 5e-4 to -4 and
// 1.1% to -8, where 1 + erf in fp32 has nothing left.
struct ActValue {
  float v, slope;
};
template <int ACT>
__device__ __forceinline__ ActValue glu_act(float g) {
  if (ACT == kActSilu) {
    const float p = __builtin_amdgcn_rcpf(1.f + __expf(-g));
    return {g * p, p * (1.f + g * (1.f - p))};
  }
  const float x = fabsf(g) * 0.70710678118654752f, e = __expf(-x * x);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.f));
  const float poly = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f),
                              0.254829592f);
  const float tail = 0.5f * poly * e;  // Phi(-|g|)
  const float p = g < 0.f ? tail : 1.f - tail;
  return {g * p, fmaf(g, 0.39894228040143268f * e, p)};
}

// Values at any even address, where rows of an odd H start: the hardware takes whole loads and
// stores there (8190 x 512 x 9809's gradient in 444 us, against 713 element by element).
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// N (2 or 4) consecutive values of row `row` from column `col` on, rounded to bf16 (nearest even);
// PAST: fours by stores that bypass the caches.
template <int N, bool PAST>
__device__ __forceinline__ void store_cols(uint16_t* Y, int64_t M, int64_t H, int64_t row, int64_t col,
                                           const float (&v)[N]) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; i++)
    w[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
  if (row >= M) return;
  uint16_t* y = Y + row * H + col;
  if (col + N <= H) {
    if constexpr (N == 4 && PAST) __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2_any*>(y));
    else if constexpr (N == 4) *reinterpret_cast<u32x2_any*>(y) = u32x2{w[0], w[1]};
    else *reinterpret_cast<u32_any*>(y) = w[0];
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

// The tiled product: WM x WN waves of RB x NB blocks, 16 RB WM rows and 16 NB WN weight rows (8 NB
// WN outputs) a tile.  Of a wave column's 16 NB weight rows the first half are gate rows, the
// second up; row 16 nb + r16 of either half is output column NB / 2 r16 + nb, so that lane r16
// holds NB / 2 consecutive columns over its blocks.  Measured: 32760 x 5120 x 13824 6.0-6.5 ms
// (1.43-1.54 PFLOP/s; the matrix cores 78% busy at the 1.8 GHz that the power limit leaves), 4173 x
// 2560 x 6916 with GELU, G and U kept 255-290 us (1.02-1.16): 935 tiles take four rounds of 256, and of a
// tile's 67 us the first loads and the stores of three outputs 17.  PAST: outputs bypass the caches,
// which pays (4173 x 2560 x 6912 with G and U 257 us against 265, 24830 x 192 x 4672 223 against
// 235) unless rows end inside a 64-byte piece, whose parts then go out one by one (24830 x 192 x
// 4666 179 against 152, 4096 x 640 x 8196 with G and U 164 against 153).  The large tiles' Y goes past
// them at every width: 14 shapes with such rows, odd ones among them, from 4096 x 640 x 8193 to 8192 x
// 5120 x 13828, gain up to 4% alone (113 against 118, 20000 x 256 x 6000 223 against 231) and 5% with G
// and U kept (8000 x 1024 x 7000 248 against 261), and lose 1% at most (16000 x 640 x 6913 with G and U).
template <int ACT, int RB, int NB, int WM, int WN, int DEPTH, bool PAST>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256),
                          amdgpu_waves_per_eu(RB == 8 || DEPTH == 4 ? 1 : 2, RB == 8 || DEPTH == 4 ? 1 : 2)))
void glu_kernel(const GluArgs a) {
  static_assert(WM * WN == kRingWaves, "four waves");
  constexpr int BM = 16 * RB * WM, BN = 16 * NB * WN, NC = NB / 2;
  typedef KRows<BM> OpA;
  typedef KRows<BN> OpB;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ring_slots(DEPTH) * OpA::kBytes];
  int tm, tn;
  tile_coords(a.tiles_m, a.tiles_n, tm, tn);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;
  const int q = lane >> 4, r16 = lane & 15;
  const int64_t M = a.M, K = a.K, H = a.H;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * (BN / 2);
  const int steps = (int)(K / kRK);
  // Rows past M or H lie outside the buffers and read as zeros.
  const uint16_t *X = a.X + m0 * K, *Wg = a.Wg + n0 * K, *Wu = a.Wu + n0 * K;
  const int64_t xb = (M - m0) * K * 2, wb = (H - n0) * K * 2;
  const OpA oa(K, 1, wave, lane);
  const OpB ob(K, NC, wave, lane);
  auto at_a = [&](int kt) { return typename OpA::Tile{oa, rsrc_if(kt >= 0, X, xb), max(kt, 0) * (kRK * 2)}; };
  struct Weights {
    const OpB& op;
    __amdgpu_buffer_rsrc_t gate, up;
    int koff;
    __device__ __forceinline__ void load(uint8_t* dst, int i) const {
      const int blk = i * kRingWaves + op.wave, at = blk % (2 * NB);  // 8-row block, and within its wave column
      const int of = at % NB;  // half `of & 1` of block nb = of / 2
      op.load(at >= NB ? up : gate, dst, i, blk / (2 * NB) * (16 * NC) + (of & 1) * (8 * NC) + (of >> 1), koff);
    }
  };
  auto at_b = [&](int kt) {
    return Weights{ob, rsrc_if(kt >= 0, Wg, wb), rsrc_if(kt >= 0, Wu, wb), max(kt, 0) * (kRK * 2)};
  };
  f32x4 acc[RB][NB];
  ring_product<DEPTH>(acc, lds, oa, ob, at_a, at_b, steps, wm, wn);

  const int64_t col = n0 + 16 * NC * wn + NC * r16;
#pragma unroll
  for (int rb = 0; rb < RB; rb++) {
    settle(acc[rb]);
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t row = m0 + 16 * (RB * wm + rb) + 4 * q + j;
      float g[NC], u[NC], y[NC];
#pragma unroll
      for (int e = 0; e < NC; e++) {
        g[e] = acc[rb][e][j];
        u[e] = acc[rb][NC + e][j];
        y[e] = glu_act<ACT>(g[e]).v * u[e];
      }
      store_cols<NC, PAST || RB == 8>(a.Y, M, H, row, col, y);
      if (a.G != nullptr) store_cols<NC, PAST>(a.G, M, H, row, col, g);
      if (a.U != nullptr) store_cols<NC, PAST>(a.U, M, H, row, col, u);
    }
  }
}

// Few rows, or few outputs: a workgroup forms 16 MB rows of 16 output columns; wave w takes the K
// steps w, w + 4, ... of 64, each with a ring of D LDS slots of its own (16 gate rows, 16 up rows and the rows of X,
// in whole 128-byte lines that go straight to LDS) and no barrier, and the waves' sums are added
// in wave order.  Bound by the weights' bytes: 1 x 5120 x 13824 reads 283 MB in 44-47 us (6.0-6.4
// TB/s), 32 x 5120 x 13824 in 56.  (Loading fragments
// straight into registers, 64 pieces of 16 bytes an instruction, is held by the address path
// instead: 16 rows of X then cost 25% of the time.)
template <int ACT, int MB>
__global__ __launch_bounds__(64 * kRingWaves) void glu_rows_kernel(const GluArgs a) {
  constexpr int D = 2;  // 48 KB a workgroup at MB = 1, three to a CU; D = 4 measured 5-15% slower
  constexpr int LOADS = 4 + 2 * MB, SLOT = LOADS * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kRingWaves * D * SLOT];
  static_assert(kRingWaves * D * SLOT >= kRingWaves * 2 * MB * 1024, "the sums fit the rings");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int q = lane >> 4, r16 = lane & 15;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MB), M = min(a.M - m0, (int64_t)(16 * MB));
  const int64_t K = a.K, H = a.H, n0 = (int64_t)blockIdx.x * 16;
  const uint16_t* X = a.X + m0 * K;
  const int KT = (int)(K / kBK);
  uint8_t* const ring = lds + wave * (D * SLOT);
  const KRows<256> op(K, 1, 0, lane);  // eight rows a load, block by block
  auto load = [&](int s, uint8_t* slot) {
    const bool live = s < KT;  // past the end: zeros
    const int koff = live ? s * (kBK * 2) : 0;
    const __amdgpu_buffer_rsrc_t gr = rsrc_if(live, a.Wg + n0 * K, (H - n0) * K * 2),
                                 ur = rsrc_if(live, a.Wu + n0 * K, (H - n0) * K * 2), xr = rsrc_if(live, X, M * K * 2);
    auto one = [&](__amdgpu_buffer_rsrc_t res, int at, int row) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(res, (__attribute__((address_space(3))) void*)(slot + at * 1024), 16, op.voff,
                                               (int)(row * K * 2) + koff, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < 2; i++) {
      one(gr, i, 8 * i);
      one(ur, 2 + i, 8 * i);
    }
#pragma unroll
    for (int i = 0; i < 2 * MB; i++) one(xr, 4 + i, 8 * i);
  };
  f32x4 acc[2][MB];
#pragma unroll
  for (int p = 0; p < 2; p++)
#pragma unroll
    for (int mb = 0; mb < MB; mb++) acc[p][mb] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < D; i++) load(wave + i * kRingWaves, ring + i * SLOT);
  for (int s = wave; s < KT; s += D * kRingWaves)
#pragma unroll
    for (int i = 0; i < D; i++) {
      uint8_t* slot = ring + i * SLOT;
      wait_vmcnt<(D - 1) * LOADS>();  // this slot's loads have arrived
      asm volatile("" ::: "memory");
      u32x4 w[2][2], x[MB][2];
#pragma unroll
      for (int kk = 0; kk < 2; kk++) {
#pragma unroll
        for (int p = 0; p < 2; p++) w[p][kk] = op.read(slot, p, kk);
#pragma unroll
        for (int mb = 0; mb < MB; mb++) x[mb][kk] = op.read(slot, 2 + mb, kk);
      }
      wait_ring<63>();  // the reads: the slot is free
      asm volatile("" ::: "memory");
      load(s + (D + i) * kRingWaves, slot);
#pragma unroll
      for (int kk = 0; kk < 2; kk++)
#pragma unroll
        for (int p = 0; p < 2; p++)
#pragma unroll
          for (int mb = 0; mb < MB; mb++)
            acc[p][mb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[mb][kk]),
                                                                 __builtin_bit_cast(bf16x8, w[p][kk]), acc[p][mb], 0, 0, 0);
    }
  wait_vmcnt<0>();
  __syncthreads();  // every wave's ring is free
  f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int p = 0; p < 2; p++)
#pragma unroll
    for (int mb = 0; mb < MB; mb++) red[(wave * 2 * MB + p * MB + mb) * 64 + lane] = acc[p][mb];
  __syncthreads();
  for (int mb = wave; mb < MB; mb += kRingWaves) {
    f32x4 g = red[mb * 64 + lane], u = red[(MB + mb) * 64 + lane];
    for (int w = 1; w < kRingWaves; w++) {
      g += red[(w * 2 * MB + mb) * 64 + lane];
      u += red[(w * 2 * MB + MB + mb) * 64 + lane];
    }
    const int64_t col = n0 + r16;
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int64_t row = 16 * mb + 4 * q + j;
      if (row >= M || col >= H) continue;
      const int64_t at = (m0 + row) * H + col;
      a.Y[at] = __builtin_bit_cast(uint16_t, (__bf16)(glu_act<ACT>(g[j]).v * u[j]));
      if (a.G != nullptr) a.G[at] = __builtin_bit_cast(uint16_t, (__bf16)g[j]);
      if (a.U != nullptr) a.U[at] = __builtin_bit_cast(uint16_t, (__bf16)u[j]);
    }
  }
}

namespace {

template <int ACT, int RB, int NB, int WM, int WN, int DEPTH>
void glu_tiles(GluArgs a, hipStream_t stream) {
  constexpr int BM = 16 * RB * WM, BH = 8 * NB * WN;
  a.tiles_m = (int)((a.M + BM - 1) / BM);
  a.tiles_n = (int)((a.H + BH - 1) / BH);
  const dim3 grid((unsigned)(a.tiles_m * a.tiles_n)), block(256);
  if (NB == 4 || a.H % 32 == 0) hipLaunchKernelGGL((glu_kernel<ACT, RB, NB, WM, WN, DEPTH, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((glu_kernel<ACT, RB, NB, WM, WN, DEPTH, NB == 4>), grid, block, 0, stream, a);
}

template <int ACT, int MB>
void glu_rows(const GluArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.H + 15) / 16), (unsigned)((a.M + 16 * MB - 1) / (16 * MB)));
  hipLaunchKernelGGL((glu_rows_kernel<ACT, MB>), grid, dim3(64 * kRingWaves), 0, stream, a);
}

// Whether more than two 128 x 64 tiles a CU take less time than 256 x 128 tiles: costs in
// microseconds fitted to measured calls.  A large tile costs 1.15 a K step and 9 for its first
// loads and its stores, which nothing covers, and a round of 256 lasts as long as its tiles; two
// small ones a CU cost 0.8 a step and 4.2, a last round of one to a CU about two thirds.  (Small
// against large: 3324 x 64 x 10672 72 and 94, 2048 x 2560 x 5120 98 and 110, 564 x 128 x 12712 24
// and 39; 4173 x 2560 x 6916 266 and 227, 1024 x 5120 x 13824 277 and 221.)
inline bool glu_small(int64_t M, int64_t K, int64_t H) {
  const int64_t large = ((M + 255) / 256) * ((H + 127) / 128), small = ((M + 127) / 128) * ((H + 63) / 64);
  const double steps = (double)(K / kRK), rest = (double)(small % 512);
  const double rounds = (double)(small / 512) + (rest > 256 ? 1. : rest > 0 ? 0.65 : 0.);
  return rounds * (0.8 * steps + 4.2) < (double)((large + 255) / 256) * (1.15 * steps + 9.);
}

// By rows, then by the number of 128 x 64 tiles (microseconds at K = 2560 where none is given):
//  - up to 32 rows, and up to 64 where such tiles would leave a third of the CUs without one: the
//    weights streamed (64 x 6912, 108 tiles: 21 against 25; 64 x 13824, K = 5120, 216: 75 against 53);
//  - few outputs: the same kernel, whose waves share K, by 16 rows where that makes at most one
//    workgroup to two CUs, else by 32 or 64 where one to a CU (80 x 121, K = 5120: 9.5 against 25; 437 x
//    400: 13 against 16.4; with 441 workgroups of 64 rows, 437 x 1000, 21.8 against 17.6);
//  - at most half as many tiles as CUs: half as wide ones (100 x 6912: 20 against 25);
//  - at most one to a CU: four steps ahead, since nothing else hides a load (200 x 6912: 27
//    against 33; 100 x 10000, K = 5120: 41 against 53);
//  - at most two to a CU, or more where glu_small says so; else 256 x 128 tiles (900 x 5000, 640
//    tiles: 52 against 65).
// Waves of 32 x 128 store whole 128-byte lines, waves of 64 x 64 read a fifth less from LDS, which
// tells the more steps there are.  One tile to a CU, means over three to nine shapes of 100 to 1000
// rows, 64 x 64 against 32 x 128: K = 640 9.4 and 8.9, 1280 13.7 and 13.4, 1920 17.9 and 17.7, 2560 22.1
// and 22.2, 4096 31.3 and 32.1, 5120 39.4 and 41.5.  More than one to a CU: 32 x 128 (128 x 13824 at K =
// 640 with G and U 15 against 17, 564 x 12712 at K = 128 22 against 26, 500 x 6912 43 against 42.5).
template <int ACT>
void glu_launch(const GluArgs& a, hipStream_t stream) {
  const int64_t tiles = ((a.M + 127) / 128) * ((a.H + 63) / 64);
  auto groups = [&](int64_t rows) { return (a.M + rows - 1) / rows * ((a.H + 15) / 16); };
  if (a.M <= 16 || groups(16) <= 128) glu_rows<ACT, 1>(a, stream);
  else if (a.M <= 32 || groups(32) <= 256) glu_rows<ACT, 2>(a, stream);
  else if ((a.M <= 64 && tiles < 171) || groups(64) <= 256) glu_rows<ACT, 4>(a, stream);
  else if (tiles <= 128) glu_tiles<ACT, 2, 4, 4, 1, 4>(a, stream);
  else if (tiles <= 256 && a.K > 1920) glu_tiles<ACT, 4, 4, 2, 2, 4>(a, stream);
  else if (tiles <= 256) glu_tiles<ACT, 2, 8, 4, 1, 4>(a, stream);
  else if (tiles <= 512 || glu_small(a.M, a.K, a.H)) glu_tiles<ACT, 2, 8, 4, 1, 2>(a, stream);
  else glu_tiles<ACT, 8, 8, 2, 2, 2>(a, stream);
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
// Bound by memory: 8190 x 13824 reads three and writes two times 226 MB in 181 us (6.2 TB/s).
//
// The rounding, 2^-8 of an element at most, adds to a gradient what the gradient's own rounding
// to bf16 does, as long as many elements share the sum of squares; in a product of few of them
// one large element's error shows in full.  Up to kGluFewElements of them (where the products
// are held by the weights' bytes) an element goes into two bf16 values, its leading digits in the
// first P and what they leave, rounded, in a second one, and the products run over both: dG and dU
// then hold to 2^-16.  (Twice the products' steps: 1 x 5120 x 13824 takes 192 us instead of 149, 2 x
// 2560 x 6912 56 instead of 42.)
constexpr int64_t kGluFewElements = 1 << 14;
inline int glu_passes(int64_t M, int64_t H) { return M * H <= kGluFewElements ? 2 : 1; }
// The two parts of v: the next bf16 value towards zero (below v, also where v is one) and the rest (a
// bf16 value is exact in its two parts).  Each has v's sign and is 0 only where v is (down to
// 2^-102), so that with an infinite weight or token both give the same infinity, where opposite
// ones, or a part of 0, would give NaN.  An infinity or NaN is its own second part.
struct GluParts {
  __bf16 hi, lo;
};
__device__ __forceinline__ GluParts glu_parts(float v) {
  if (!__builtin_isfinite(v) || v == 0.f) return {(__bf16)v, (__bf16)v};
  const float hi = __uint_as_float((__float_as_uint(v) - 1) & 0xFFFF0000u);
  return {(__bf16)hi, (__bf16)(v - hi)};
}
template <int ACT>
__global__ __launch_bounds__(256) void glu_back_kernel(int64_t M, int64_t H, int64_t Hp, const uint16_t* G,
                                                       const uint16_t* U, const uint16_t* dY, uint16_t* P, int passes) {
  const int64_t c8 = Hp / 8, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= M * c8) return;
  const int64_t m = id / c8, h = (id - m * c8) * 8, at = m * H + h;
  u32x4 g{}, u{}, d{};
  if (h + 8 <= H) {
    g = *reinterpret_cast<const u32x4_any*>(G + at);
    u = *reinterpret_cast<const u32x4_any*>(U + at);
    d = *reinterpret_cast<const u32x4_any*>(dY + at);
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
  u32x4 p[2][2];  // pass; dG, dU
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const ActValue a0 = glu_act<ACT>(bf16lo(g[i])), a1 = glu_act<ACT>(bf16hi(g[i]));
    const float d0 = bf16lo(d[i]), d1 = bf16hi(d[i]);
    const float v[2][2] = {{d0 * bf16lo(u[i]) * a0.slope, d1 * bf16hi(u[i]) * a1.slope}, {d0 * a0.v, d1 * a1.v}};
#pragma unroll
    for (int k = 0; k < 2; k++) {
      if (passes == 1) {
        p[0][k][i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[k][0], (__bf16)v[k][1]});
      } else {
        const GluParts a = glu_parts(v[k][0]), b = glu_parts(v[k][1]);
        p[0][k][i] = __builtin_bit_cast(uint32_t, bf16x2_t{a.hi, b.hi});
        p[1][k][i] = __builtin_bit_cast(uint32_t, bf16x2_t{a.lo, b.lo});
      }
    }
  }
  for (int pass = 0; pass < passes; pass++) {
    uint16_t* row = P + ((int64_t)pass * M + m) * 2 * Hp + h;
    *reinterpret_cast<u32x4*>(row) = pass ? p[1][0] : p[0][0];
    *reinterpret_cast<u32x4*>(row + Hp) = pass ? p[1][1] : p[0][1];
  }
}

// A wave's row of NB blocks to 16 bf16 rows through its LDS block of 16 * (32 NB + 16) bytes, as
// 16-byte chunks; row(i) gives the address of row i at its first column or null, `cols` (a
// multiple of 8) the columns from there on.
template <int NB, typename Row>
__device__ __forceinline__ void store_rows(const f32x4 (&acc)[NB], uint8_t* blk, int lane, int64_t cols, Row row) {
  constexpr int CW = NB * 16, PITCH = 2 * CW + 16, CPR = CW / 8;
  const int q = lane >> 4, r16 = lane & 15;
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int nb = 0; nb < NB; nb++)
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const uint32_t w = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)acc[nb][j], (__bf16)acc[nb][j + 1]});
      uint8_t* at = blk + (4 * q + j) * PITCH + (nb * 16 + r16) * 2;
      *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
      *reinterpret_cast<uint16_t*>(at + PITCH) = (uint16_t)(w >> 16);
    }
#pragma unroll
  for (int c = 0; c < 16 * CPR / 64; c++) {
    const int id = lane + 64 * c, rr = id / CPR, cc = id % CPR;
    const u32x4 v = *reinterpret_cast<const u32x4*>(blk + rr * PITCH + cc * 16);
    uint16_t* y = row(rr);
    if (y != nullptr && 8 * cc < cols) __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(y + 8 * cc));
  }
}

// The gradient's two products, dX = P [Wg; Wu] (0) and [dWg; dWu] = P^T X (1), run as one launch,
// the one with the longer jobs first, so that the other's tiles fill the CUs that its last round
// would leave idle.  A job is a tile over all of k, or, where a product has few tiles, a part of a
// tile's k: the parts' fp32 sums go to `part` in accumulator order and are added in split order by
// glu_join_kernel.  Bound by the matrix cores and the power they draw (71% busy at 1.75 GHz) where
// both sides are large: 8190 x 5120 x 13824 3.5-3.8 ms (1.22-1.33 PFLOP/s); by the tiles' first
// loads and stores where few tokens meet whole weights: 333 x 2560 x 6912 79-80 us.
struct GluJobs {
  int tiles_m, tiles_n, splits;
  int steps, per;  // K steps of a tile, of a part
  int count;       // workgroups, tiles * splits; 0 if the product is not wanted
  float* part;     // [splits][tiles][T * T]
};
struct GluBackArgs {
  int64_t M, K, H, Hp;
  const uint16_t *P, *X, *Wg, *Wu;
  uint16_t *dX, *dWg, *dWu;
  GluJobs jobs[2];
  int passes;            // step s is K step s / passes of P's s % passes
  int join[2];           // tiles of each that are split
  int first, second_at;  // the product that goes first; workgroup from which the second runs (a multiple of 8)
};

// What workgroup i of a product does: a tile, its K steps, and its part (-1: the whole tile).
struct GluJob {
  int tm, tn, first, steps, part;
};
__device__ __forceinline__ GluJob glu_job(const GluJobs& g, int w) {
  // Workgroups go round the XCDs: each gets a contiguous run of the jobs, split by split.
  const int n = g.count, tiles = g.tiles_m * g.tiles_n;
  const int at = (w & 7) * (n >> 3) + min(w & 7, n & 7) + (w >> 3);
  GluJob j;
  j.part = g.splits > 1 ? at : -1;
  j.first = at / tiles * g.per;
  j.steps = min(g.per, g.steps - j.first);
  tile_from_index(at % tiles, g.tiles_m, g.tiles_n, j.tm, j.tn);
  return j;
}

// Output row r: of dX, or of [dWg; padding; dWu; padding] (Hp rows each).
template <bool DW>
__device__ __forceinline__ uint16_t* glu_row(const GluBackArgs& a, int64_t r) {
  if (!DW) return r < a.M ? a.dX + r * a.K : nullptr;
  return r < a.H ? a.dWg + r * a.K : r >= a.Hp && r < a.Hp + a.H ? a.dWu + (r - a.Hp) * a.K : nullptr;
}

// Stores a wave's blocks to the output's rows or to its part (decided row of blocks by row of
// blocks: as two loops the accumulators move about on the way to them).
template <int R, bool DW>
__device__ __forceinline__ void glu_finish(const GluBackArgs& a, const GluJob& j, f32x4 (&acc)[R][R], uint8_t* lds,
                                           int wave, int lane) {
  __syncthreads();  // the ring is free
  f32x4* part = reinterpret_cast<f32x4*>(a.jobs[DW].part) + ((int64_t)j.part * kRingWaves + wave) * (R * R * 64) + lane;
  const int64_t row0 = (int64_t)j.tm * (32 * R) + 16 * R * (wave & 1), col0 = (int64_t)j.tn * (32 * R) + 16 * R * (wave >> 1);
#pragma unroll
  for (int rb = 0; rb < R; rb++) {
    settle(acc[rb]);
    if (j.part >= 0) {
#pragma unroll
      for (int nb = 0; nb < R; nb++) part[(rb * R + nb) * 64] = acc[rb][nb];
    } else {
      store_rows<R>(acc[rb], lds + wave * 16 * (32 * R + 16), lane, a.K - col0, [&](int i) {
        uint16_t* y = glu_row<DW>(a, row0 + 16 * rb + i);
        return y == nullptr ? y : y + col0;
      });
    }
  }
}

// dX = P [Wg; Wu]: k runs over P's 2 Hp columns, along P's rows and down the weights' columns.
template <int R>
__device__ __forceinline__ void glu_dx_tile(const GluBackArgs& a, int w, uint8_t* lds, int wave, int lane) {
  constexpr int T = 32 * R;
  typedef KRows<T> OpA;
  typedef KCols<T> OpB;
  const GluJob j = glu_job(a.jobs[0], w);
  const int64_t M = a.M, K = a.K, H = a.H, ld = 2 * a.Hp;
  const int half = (int)(a.Hp / kRK);
  const int64_t m0 = (int64_t)j.tm * T, c0 = (int64_t)j.tn * T;
  const uint16_t* P = a.P + m0 * ld;
  const int two = a.passes - 1;
  const OpA oa(ld, 1, wave, lane);
  const OpB ob(K, wave, lane);
  auto at_a = [&](int kt) {
    const int s = j.first + max(kt, 0);
    return typename OpA::Tile{oa, rsrc_if(kt >= 0, P + (s & two) * M * ld, (M - m0) * ld * 2), (s >> two) * (kRK * 2)};
  };
  auto at_b = [&](int kt) {
    // rows of Wg, then of Wu; past H (P's padding) they read as zeros
    const int s = (j.first + max(kt, 0)) >> two;
    const int64_t h = (int64_t)(s < half ? s : s - half) * kRK;
    return typename OpB::Tile{ob, rsrc_if(kt >= 0, (s < half ? a.Wg : a.Wu) + h * K + c0, ((H - h) * K - c0) * 2)};
  };
  f32x4 acc[R][R];
  ring_product<2>(acc, lds, oa, ob, at_a, at_b, j.steps, wave & 1, wave >> 1);
  glu_finish<R, false>(a, j, acc, lds, wave, lane);
}

// [dWg; dWu] = P^T X: k runs over the tokens, down the columns of both.
template <int R>
__device__ __forceinline__ void glu_dw_tile(const GluBackArgs& a, int w, uint8_t* lds, int wave, int lane) {
  constexpr int T = 32 * R;
  typedef KCols<T> Op;
  const GluJob j = glu_job(a.jobs[1], w);
  const int64_t M = a.M, K = a.K, ld = 2 * a.Hp;
  const int64_t r0 = (int64_t)j.tm * T, c0 = (int64_t)j.tn * T;
  const Op oa(ld, wave, lane), ob(K, wave, lane);
  const int two = a.passes - 1;
  // tokens past M lie outside the buffers and read as zeros
  auto at_a = [&](int kt) {
    const int s = j.first + max(kt, 0);
    const int64_t m = (int64_t)(s >> two) * kRK;
    return typename Op::Tile{oa, rsrc_if(kt >= 0, a.P + ((s & two) * M + m) * ld + r0, ((M - m) * ld - r0) * 2)};
  };
  auto at_b = [&](int kt) {
    const int64_t m = (int64_t)((j.first + max(kt, 0)) >> two) * kRK;
    return typename Op::Tile{ob, rsrc_if(kt >= 0, a.X + m * K + c0, ((M - m) * K - c0) * 2)};
  };
  f32x4 acc[R][R];
  ring_product<2>(acc, lds, oa, ob, at_a, at_b, j.steps, wave & 1, wave >> 1);
  glu_finish<R, true>(a, j, acc, lds, wave, lane);
}

template <int R>
__global__ __attribute__((amdgpu_flat_work_group_size(256, 256), amdgpu_waves_per_eu(R == 8 ? 1 : 2, R == 8 ? 1 : 2)))
void glu_grad_kernel(const GluBackArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ring_slots(2) * KCols<32 * R>::kBytes];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool second = (int)blockIdx.x >= a.second_at;
  const int which = second ? 1 - a.first : a.first, w = second ? blockIdx.x - a.second_at : blockIdx.x;
  if (w >= a.jobs[which].count) return;  // between the products, up to the multiple of 8
  if (which == 0) glu_dx_tile<R>(a, w, lds, wave, lane);
  else glu_dw_tile<R>(a, w, lds, wave, lane);
}

// One wave per 16-row strip of a split tile's wave: the parts' sum in split order, stored.
template <int R, bool DW>
__device__ __forceinline__ void glu_join(const GluBackArgs& a, int at, uint8_t* lds, int lane) {
  const GluJobs& g = a.jobs[DW];
  const int rb = at % R, wave = at / R % kRingWaves, i = at / R / kRingWaves;
  const int tiles = g.tiles_m * g.tiles_n;
  int tm, tn;
  tile_from_index(i, g.tiles_m, g.tiles_n, tm, tn);
  const f32x4* in =
      reinterpret_cast<const f32x4*>(g.part) + ((int64_t)i * kRingWaves + wave) * (R * R * 64) + rb * R * 64 + lane;
  const int64_t part = (int64_t)tiles * kRingWaves * (R * R * 64);
  f32x4 acc[R];
#pragma unroll
  for (int nb = 0; nb < R; nb++) acc[nb] = in[nb * 64];
#pragma unroll 4  // four parts' loads in flight (16 parts: 2 us less)
  for (int s = 1; s < g.splits; s++) {
    in += part;
#pragma unroll
    for (int nb = 0; nb < R; nb++) acc[nb] += in[nb * 64];
  }
  const int64_t row0 = (int64_t)tm * (32 * R) + 16 * (R * (wave & 1) + rb), col0 = (int64_t)tn * (32 * R) + 16 * R * (wave >> 1);
  store_rows<R>(acc, lds, lane, a.K - col0, [&](int r) {
    uint16_t* y = glu_row<DW>(a, row0 + r);
    return y == nullptr ? y : y + col0;
  });
}
template <int R>
__global__ __launch_bounds__(64) void glu_join_kernel(const GluBackArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[16 * (32 * R + 16)];
  const int dx = a.join[0] * kRingWaves * R;
  if ((int)blockIdx.x < dx) glu_join<R, false>(a, blockIdx.x, lds, threadIdx.x);
  else glu_join<R, true>(a, blockIdx.x - dx, lds, threadIdx.x);
}

namespace {
inline int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

// Ways to run the jobs, with costs in microseconds fitted to measured calls: tiles of 32 R, P
// workgroups at once, each `step` per K step and `tile` for its first loads and its stores, a part
// `way` through memory and back.  (Small tiles four steps ahead, one to a CU, as in the forward
// product: 25% faster where one such round holds all jobs, up to 20% slower elsewhere; not kept.)
struct GluWay {
  int R;
  int64_t P;
  double step, tile, way;
};
// What a split more adds, in the join's wave that adds them one after another and since jobs alone on
// a CU take less than `step` (100 x 1280 x 3456 in 16 splits 28.8 us, in 8 25.3).
constexpr double kGluSplit = 1.;
constexpr GluWay kGluWays[2] = {{8, 256, 1.55, 12., 0.1}, {4, 512, 1.02, 3.5, 0.026}};

struct GluPlan {
  int R;
  GluJobs jobs[2];
  double cost;
  size_t part_bytes(int k) const { return jobs[k].splits > 1 ? (size_t)jobs[k].count * (32 * R) * (32 * R) * 4 : 0; }
};

// The jobs of one product of `rows` x `cols` outputs: its tiles, each in `splits` parts.
GluJobs glu_jobs(int R, int64_t rows, int64_t cols, int64_t steps, int64_t splits) {
  const int64_t T = 32 * R, tm = (rows + T - 1) / T, tn = (cols + T - 1) / T;
  const int64_t per = (steps + splits - 1) / splits;
  GluJobs g{};
  g.tiles_m = (int)tm;
  g.tiles_n = (int)tn;
  g.splits = (int)((steps + per - 1) / per);
  g.steps = (int)steps;
  g.per = (int)per;
  g.count = (int)std::min<int64_t>(tm * tn * g.splits, INT32_MAX);
  return g;
}

// When n1 jobs of length l1, then n2 of length l2 <= l1 are done on P workgroups: the first leave r1
// of them one l1 behind the others, which meanwhile take late = ceil(l1 / l2) of the second each.
double glu_makespan(int64_t P, int64_t n1, double l1, int64_t n2, double l2) {
  const int64_t q1 = n1 / P, r1 = n1 % P, late = r1 > 0 ? (int64_t)std::ceil(l1 / l2) : 0;
  int64_t i = (n2 + r1 * late + P - 1) / P;
  if (i < late) i = (n2 + P - r1 - 1) / (P - r1);
  return std::max(q1 * l1 + i * l2, (r1 > 0 ? q1 + 1 : q1) * l1);
}

// Tile size and splits with the least makespan.  (The plan does not depend on whether both products
// are wanted: each has the same bits with the other and without.)
GluPlan glu_plan(int64_t M, int64_t K, int64_t H) {
  const int64_t rows[2] = {M, 2 * pad64(H)}, passes = glu_passes(M, H);
  const int64_t steps[2] = {passes * 2 * pad64(H) / kRK, passes * ((M + kRK - 1) / kRK)};
  GluPlan best{};
  for (const GluWay& c : kGluWays) {
    GluJobs options[2][6];
    int n[2] = {0, 0};
    for (int k = 0; k < 2; k++)
      for (int64_t s : {1, 2, 3, 5, 8, 16}) {
        const GluJobs g = glu_jobs(c.R, rows[k], K, steps[k], s);
        if (s > 1 && (s > steps[k] / 4 || (int64_t)g.tiles_m * g.tiles_n * g.splits > 2 * c.P)) break;
        options[k][n[k]++] = g;
      }
    for (int x = 0; x < n[0]; x++)
      for (int w = 0; w < n[1]; w++) {
        const GluJobs &dx = options[0][x], &dw = options[1][w];
        const bool dx_first = dx.per >= dw.per;
        const GluJobs &one = dx_first ? dx : dw, &two = dx_first ? dw : dx;
        const double cost = glu_makespan(c.P, one.count, one.per * c.step + c.tile, two.count, two.per * c.step + c.tile) +
                            c.way * ((dx.splits > 1 ? dx.count : 0) + (dw.splits > 1 ? dw.count : 0)) +
                            kGluSplit * std::max(dx.splits, dw.splits);
        if (best.R == 0 || cost < best.cost) best = GluPlan{c.R, {dx, dw}, cost};
      }
  }
  return best;
}

template <int R>
void glu_products(const GluBackArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(a.second_at + a.jobs[1 - a.first].count));
  hipLaunchKernelGGL((glu_grad_kernel<R>), grid, dim3(256), 0, stream, a);
  const int split = a.join[0] + a.join[1];
  if (split > 0)
    hipLaunchKernelGGL((glu_join_kernel<R>), dim3((unsigned)(split * kRingWaves * R)), dim3(64), 0, stream, a);
}
}  // namespace

// Workspace: P [passes, M, 2 Hp] bf16 | parts of dX | parts of [dWg; dWu].
size_t glu_back_workspace(int64_t M, int64_t K, int64_t H) {
  const GluPlan p = glu_plan(M, K, H);
  return align256((size_t)(glu_passes(M, H) * M * 2 * pad64(H) * 2)) + align256(p.part_bytes(0)) + align256(p.part_bytes(1));
}

hipError_t launch_glu_back_bf16(int act, int64_t M, int64_t K, int64_t H, const void* X, const void* Wg,
                                const void* Wu, const void* G, const void* U, const void* dY, void* dX, void* dWg,
                                void* dWu, void* ws, hipStream_t stream) {
  const GluPlan p = glu_plan(M, K, H);
  GluBackArgs a{};
  a.M = M; a.K = K; a.H = H; a.Hp = pad64(H);
  uint16_t* P = (uint16_t*)ws;
  a.P = P; a.X = (const uint16_t*)X; a.Wg = (const uint16_t*)Wg; a.Wu = (const uint16_t*)Wu;
  a.dX = (uint16_t*)dX; a.dWg = (uint16_t*)dWg; a.dWu = (uint16_t*)dWu;
  a.passes = glu_passes(M, H);
  uint8_t* parts = (uint8_t*)ws + align256((size_t)(a.passes * M * 2 * a.Hp * 2));
  const bool want[2] = {dX != nullptr, dWg != nullptr};
  for (int k = 0; k < 2; k++) {
    a.jobs[k] = p.jobs[k];
    if (!want[k]) a.jobs[k].count = 0;
    a.join[k] = want[k] && p.jobs[k].splits > 1 ? p.jobs[k].tiles_m * p.jobs[k].tiles_n : 0;
  }
  a.jobs[0].part = (float*)parts;
  a.jobs[1].part = (float*)(parts + align256(p.part_bytes(0)));
  a.first = p.jobs[1].per > p.jobs[0].per ? 1 : 0;
  a.second_at = (a.jobs[a.first].count + 7) / 8 * 8;
  const dim3 block(256), chunks((unsigned)((M * (a.Hp / 8) + 255) / 256));
  if (act == kActSilu)
    hipLaunchKernelGGL((glu_back_kernel<kActSilu>), chunks, block, 0, stream, M, H, a.Hp, (const uint16_t*)G,
                       (const uint16_t*)U, (const uint16_t*)dY, P, a.passes);
  else
    hipLaunchKernelGGL((glu_back_kernel<kActGelu>), chunks, block, 0, stream, M, H, a.Hp, (const uint16_t*)G,
                       (const uint16_t*)U, (const uint16_t*)dY, P, a.passes);
  if (p.R == 8) glu_products<8>(a, stream);
  else glu_products<4>(a, stream);
  return hipGetLastError();
}

}  // namespace rtl
