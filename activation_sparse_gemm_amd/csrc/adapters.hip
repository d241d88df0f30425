// adapters.hip -- low-rank adapters of many requests beside a shared projection, and their gradient.
// Row m of a batch belongs to a request whose adapter a (or none) has factors L_B[a] [R, K] and L_A[a]
// [N, R] and a factor alpha[a]:
//
//   T = X L_B[a]^T,  Y = Y0 + alpha T L_A[a]^T
//   back: dT = alpha dY L_A[a],  dX = dX0 + dT L_B[a],
//         dL_B[a] = sum over a's rows of dT^T X,  dL_A[a] = alpha times that of dY^T T
//
// A plan sorts the batch's rows by adapter, in their order, and cuts each adapter's rows into tiles of
// 64: every kernel takes its rows through it, so that a tile meets one pair of factors whatever the
// order of the requests.  What the plan holds is bounded where it is read: no access leaves the arrays.
//
// Bound: memory (X, Y0 and Y pass once, 2 R flops a byte of them).  T and dT are held in fp32 and enter
// the next product in two bf16 parts (two_parts), 16 digits: its rounding to one, 2^-9, would be
// the largest error of an adapter's share, and the products are too small to hold the kernels.
// The gradients' sums of few rows take three (kFewRows).
//
//   down:   T's parts over K, one tile and split of K a workgroup, the waves taking K in turn
//   join:   the parts' sum; T as operand fragments (and transposed ones for the gradients)
//   up:     Y0 + T L_A^T, a tile's 64 rows by strips of 32 columns a wave
//   turn:   factors transposed, which makes dT a `down` and dX an `up`
//   grad:   dL_B and dL_A, 128 (64) columns by R a workgroup, over a share of an adapter's rows
#include <algorithm>
#include <type_traits>

#include "bf16_common.h"

namespace rtl {

namespace {

constexpr int kTile = 64;     // rows of a tile
constexpr int kThreads = 256;
constexpr int kWaves = 4;

struct Plan {
  const int32_t *start, *tbase;  // [A + 2]: first position, first tile of each adapter; A: the rows without one
  const int4* tiles;             // {adapter, first position, rows, 0}
  const int32_t* order;          // [M]: row at each position
  const int32_t* count;          // tiles
  int A;
  int64_t M, most;               // most: tiles there can be
};

int64_t max_tiles(int64_t M, int64_t A) { return std::min(M, M / kTile + A + 1); }
size_t plan_words(int64_t M, int64_t A, size_t* tiles, size_t* order) {
  size_t at = 4 + 2 * (size_t)(A + 2);
  at = (at + 3) & ~(size_t)3;
  *tiles = at;
  at += 4 * (size_t)max_tiles(M, A);
  *order = at;
  return at + (size_t)M;
}
Plan plan_of(const void* p, int64_t M, int64_t A) {
  size_t tiles, order;
  plan_words(M, A, &tiles, &order);
  const int32_t* w = (const int32_t*)p;
  return Plan{w + 4, w + 4 + A + 2, (const int4*)(w + tiles), w + order, w, (int)A, M, max_tiles(M, A)};
}

// ---------------------------------------------------------------- the plan

// Every workgroup counts all rows (in LDS, whole numbers: no order) and then places the rows of its
// own adapters in their order.
__global__ __launch_bounds__(kThreads) void plan_kernel(const int32_t* ids, int64_t M, int A, int32_t* head, int4* tiles,
                                                        int32_t* order) {
  extern __shared__ int32_t lds[];
  int32_t* count = lds;           // [A + 1], then the first positions
  int32_t* first = lds + A + 1;   // [A + 2] first tiles
  __shared__ int32_t wave_sum[kWaves][2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int a = threadIdx.x; a <= A; a += kThreads) count[a] = 0;
  __syncthreads();
  auto key = [&](int64_t m) {
    const int a = ids[m];
    return a < 0 || a >= A ? A : a;
  };
  for (int64_t m0 = 0; m0 < M; m0 += kThreads) {
    const int64_t m = m0 + threadIdx.x;
    const int k = m < M ? key(m) : -1;
    // one count for a wave of one adapter
    const int k0 = __builtin_amdgcn_readfirstlane(k);
    const uint64_t same = __ballot(k == k0);
    if (k0 >= 0 && lane == 0) atomicAdd(&count[k0], __popcll(same));
    if (k >= 0 && k != k0) atomicAdd(&count[k], 1);
  }
  __syncthreads();
  // first positions and tiles: sums over the adapters before, kThreads at a time
  int32_t rows_before = 0, tiles_before = 0;
  for (int a0 = 0; a0 <= A; a0 += kThreads) {
    const int a = a0 + threadIdx.x;
    const int n = a <= A ? count[a] : 0, t = (n + kTile - 1) / kTile;
    int sn = n, st = t;  // inclusive sums over the wave
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int un = __shfl_up(sn, o, 64), ut = __shfl_up(st, o, 64);
      if (lane >= o) {
        sn += un;
        st += ut;
      }
    }
    if (lane == 63) {
      wave_sum[wave][0] = sn;
      wave_sum[wave][1] = st;
    }
    __syncthreads();
    for (int w = 0; w < wave; w++) {
      sn += wave_sum[w][0];
      st += wave_sum[w][1];
    }
    if (a <= A) {
      count[a] = rows_before + sn - n;
      first[a] = tiles_before + st - t;
    }
    for (int w = 0; w < kWaves; w++) {
      rows_before += wave_sum[w][0];
      tiles_before += wave_sum[w][1];
    }
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    for (int a = threadIdx.x; a <= A; a += kThreads) {
      head[4 + a] = count[a];
      head[4 + A + 2 + a] = first[a];
    }
    if (threadIdx.x == 0) {
      head[0] = tiles_before;
      head[1] = head[2] = head[3] = 0;
      head[4 + A + 1] = (int32_t)M;
      head[4 + A + 2 + A + 1] = tiles_before;
    }
  }
  for (int a = blockIdx.x; a <= A; a += gridDim.x) {
    const int from = count[a], n = (a < A ? count[a + 1] : (int32_t)M) - from;
    if (n <= 0) continue;
    for (int t = threadIdx.x; t * kTile < n; t += kThreads) tiles[first[a] + t] = make_int4(a, from + t * kTile, min(kTile, n - t * kTile), 0);
    int32_t at = from;
    for (int64_t m0 = 0; m0 < M && at < from + n; m0 += kThreads) {  // at: the same in all threads
      const int64_t m = m0 + threadIdx.x;
      const bool mine = m < M && key(m) == a;
      const uint64_t which = __ballot(mine);
      if (lane == 0) wave_sum[wave][0] = __popcll(which);
      __syncthreads();
      int before = 0, all = 0;
      for (int w = 0; w < kWaves; w++) {
        if (w < wave) before += wave_sum[w][0];
        all += wave_sum[w][0];
      }
      const int to = at + before + __popcll(which & ((1ull << lane) - 1));
      if (mine && to < from + n) order[to] = (int32_t)m;
      at += all;
      __syncthreads();
    }
  }
}

// ---------------------------------------------------------------- products

// A tile as the plan gives it, within the arrays whatever it holds; rows 0: nothing to do.
struct Tile {
  int adapter, rows;
  int64_t pos;
};
__device__ __forceinline__ Tile tile_of(const Plan& p, int64_t index) {
  Tile t{0, 0, 0};
  if (index >= *p.count) return t;
  const int4 v = p.tiles[index];
  t.adapter = __builtin_amdgcn_readfirstlane(min(max(v.x, 0), p.A));
  t.pos = min(max(__builtin_amdgcn_readfirstlane(v.y), 0), (int)p.M - 1);
  t.rows = (int)min((int64_t)min(max(__builtin_amdgcn_readfirstlane(v.z), 0), kTile), p.M - t.pos);
  return t;
}
__device__ __forceinline__ int64_t row_at(const Plan& p, int64_t pos) {
  return min(max(p.order[pos], 0), (int)p.M - 1);
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// down: part[split][position][r] = sum over the split's K of X[row][k] W[adapter][r][k].  A workgroup
// takes one tile and one split; its waves take 64 of K in turn, each with all 64 rows and all R, so that
// nothing is loaded twice, and their sums are added in LDS in one order.  Blocks of 16 r by 16 rows: lane
// (r16, q) of a block holds row r16 and r = 4q .. 4q + 3.
struct DownArgs {
  Plan plan;
  const uint16_t *x, *w;  // [M, K] with a row stride, [A, R, K]
  int64_t x_row, K, part_stride;
  int R, steps;           // steps of 64 a split
  float* part;
};
template <int RB>
__global__ __launch_bounds__(kThreads) void down_kernel(const DownArgs a) {
  constexpr int BLOCKS = 4 * RB, ROUND = BLOCKS < 16 ? BLOCKS : 16;
  __shared__ f32x4 sums[kWaves][ROUND][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
  const Tile t = tile_of(a.plan, blockIdx.x);
  if (t.rows == 0 || t.adapter >= a.plan.A) return;
  const int blocks = (t.rows + 15) / 16;
  const uint16_t *xp[4], *wp[RB];
#pragma unroll
  for (int b = 0; b < 4; b++)  // rows past the last repeat it: their sums are dropped
    xp[b] = a.x + row_at(a.plan, t.pos + min(16 * b + r16, t.rows - 1)) * a.x_row + 8 * q;
#pragma unroll
  for (int b = 0; b < RB; b++) wp[b] = a.w + ((int64_t)t.adapter * a.R + min(16 * b + r16, a.R - 1)) * a.K + 8 * q;
  f32x4 acc[4][RB];
#pragma unroll
  for (int b = 0; b < 4; b++)
#pragma unroll
    for (int c = 0; c < RB; c++) acc[b][c] = f32x4{};
  struct Step {
    u32x4 x[2][4], w[2][RB];
  };
  const int64_t first = (int64_t)blockIdx.y * a.steps, last = min(first + a.steps, (a.K + 63) / 64);
  auto fetch = [&](int64_t s, Step& it) {
    if (s >= last) return;
    const int64_t k = s * 64;
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const bool in = k + 32 * h + 8 * q < a.K;
#pragma unroll
      for (int b = 0; b < 4; b++) {
        it.x[h][b] = u32x4{};
        if (b < blocks && in) it.x[h][b] = *reinterpret_cast<const u32x4*>(xp[b] + k + 32 * h);
      }
#pragma unroll
      for (int b = 0; b < RB; b++) {
        it.w[h][b] = u32x4{};
        if (in) it.w[h][b] = *reinterpret_cast<const u32x4*>(wp[b] + k + 32 * h);
      }
    }
  };
  auto form = [&](const Step& it) {
#pragma unroll
    for (int h = 0; h < 2; h++)
#pragma unroll
      for (int b = 0; b < 4; b++)
        if (b < blocks)
#pragma unroll
          for (int c = 0; c < RB; c++) acc[b][c] = mfma16(it.w[h][c], it.x[h][b], acc[b][c]);
  };
  Step one, two;
  fetch(first + wave, one);
  for (int64_t s = first + wave; s < last; s += 2 * kWaves) {
    fetch(s + kWaves, two);
    form(one);
    if (s + kWaves >= last) break;
    fetch(s + 2 * kWaves, one);
    form(two);
  }
  float* part = a.part + blockIdx.y * a.part_stride;
#pragma unroll
  for (int round = 0; round < BLOCKS; round += ROUND) {
    if (round > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < ROUND; i++) sums[wave][i][lane] = acc[(round + i) / RB][(round + i) % RB];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROUND / kWaves; i++) {
      const int at = i * kWaves + wave, b = (round + at) / RB, c = (round + at) % RB;
      f32x4 v = sums[0][at][lane];
#pragma unroll
      for (int w = 1; w < kWaves; w++) v += sums[w][at][lane];
      const int m = 16 * b + r16, r = 16 * c + 4 * q;
      if (m < t.rows && r < a.R) *reinterpret_cast<f32x4*>(part + (t.pos + m) * a.R + r) = v;
    }
  }
}

// join: a tile's sum over the splits (or a kept T's rows), scaled by alpha, in two bf16 parts, as
// operands: `rows` for up (lane (r16, q): row r16 of a block, r = 8q .. 8q + 7 of 32) and `cols` for
// grad (lane (r16, q): r = r16 of a block, rows 8q .. 8q + 7 of 32); T itself to `t`.
struct JoinArgs {
  Plan plan;
  const float* part;  // [splits][M][R] by position
  const float* kept;  // [M, R] by row, in its place
  int64_t part_stride;
  int splits, R, RK, RB, width;  // RK: R in 32s, RB: in 16s as grad takes them; width: the wider of the two
  const float* alpha;
  float* t;           // [M, R] by row, or null
  u32x4 *rows, *cols; // or null
  int parts;          // of cols
};
__device__ __forceinline__ void parts_of(const float (&v)[8], u32x4& hi, u32x4& lo) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const Bf16Parts x = two_parts(v[2 * i]), y = two_parts(v[2 * i + 1]);
    hi[i] = __builtin_bit_cast(uint32_t, bf16x2_t{x.hi, y.hi});
    lo[i] = __builtin_bit_cast(uint32_t, bf16x2_t{x.lo, y.lo});
  }
}
__global__ __launch_bounds__(kThreads) void join_kernel(const JoinArgs a) {
  extern __shared__ float tile[];  // [64][pitch]
  const int pitch = a.width + 4, quads = a.width / 4;
  const Tile t = tile_of(a.plan, blockIdx.x);
  if (t.rows == 0) return;
  const bool bare = t.adapter >= a.plan.A;
  if (bare && a.t == nullptr) return;
  const float alpha = bare || a.alpha == nullptr ? 1.f : a.alpha[t.adapter];
  for (int id = threadIdx.x; id < kTile * quads; id += kThreads) {
    const int m = id / quads, r = id % quads * 4;
    f32x4 v{};
    if (m < t.rows && r < a.R) {
      const int64_t row = row_at(a.plan, t.pos + m);
      if (a.kept != nullptr) {
        v = *reinterpret_cast<const f32x4*>(a.kept + row * a.R + r);
      } else if (!bare) {
        const float* p = a.part + (t.pos + m) * a.R + r;
#pragma unroll 4
        for (int s = 0; s < a.splits; s++) v += *reinterpret_cast<const f32x4*>(p + s * a.part_stride);
      }
      if (a.t != nullptr) *reinterpret_cast<f32x4*>(a.t + row * a.R + r) = v;
    }
    *reinterpret_cast<f32x4*>(tile + m * pitch + r) = v * alpha;
  }
  if (bare) return;
  __syncthreads();
  if (a.rows != nullptr) {
    const int n = 4 * a.RK * 64;
    u32x4* to = a.rows + (int64_t)blockIdx.x * 2 * n;
    for (int id = threadIdx.x; id < n; id += kThreads) {
      const int lane = id & 63, kk = (id >> 6) % a.RK, mb = (id >> 6) / a.RK;
      const float* p = tile + (16 * mb + (lane & 15)) * pitch + 32 * kk + 8 * (lane >> 4);
      float v[8];
      u32x4 hi, lo;
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = p[i];
      parts_of(v, hi, lo);
      to[id] = hi;
      to[n + id] = lo;
    }
  }
  if (a.cols != nullptr) {
    const int n = 2 * a.RB * 64;
    u32x4* to = a.cols + (int64_t)blockIdx.x * a.parts * n;
    for (int id = threadIdx.x; id < n; id += kThreads) {
      const int lane = id & 63, rb = (id >> 6) % a.RB, half = (id >> 6) / a.RB;
      const float* p = tile + (32 * half + 8 * (lane >> 4)) * pitch + 16 * rb + (lane & 15);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = p[i * pitch];
      if (a.parts == 3) {
        u32x4 w[3];
#pragma unroll
        for (int i = 0; i < 4; i++) {
          typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
          __bf16 x[3], y[3];
          three_parts(v[2 * i], x);
          three_parts(v[2 * i + 1], y);
#pragma unroll
          for (int k = 0; k < 3; k++) w[k][i] = __builtin_bit_cast(uint32_t, bf16x2_t{x[k], y[k]});
        }
#pragma unroll
        for (int k = 0; k < 3; k++) to[k * n + id] = w[k];
      } else {
        u32x4 hi, lo;
        parts_of(v, hi, lo);
        to[id] = hi;
        to[n + id] = lo;
      }
    }
  }
}

// up: Y[row][n] = Y0[row][n] + sum over r of T[row][r] W[adapter][n][r].  The waves of a workgroup take
// strips of 32 columns in turn, with the tile's T in registers.  The two blocks of a strip take the
// columns 8 (i / 4) + 4 b + i % 4, so that lane (r16, q) ends with columns 8q .. 8q + 7 of row r16: one
// 16-byte access to Y0 and Y.
struct UpArgs {
  Plan plan;
  const u32x4* t;          // join's rows
  const uint16_t *w, *y0;  // [A, N, R]; [M, N] with a row stride, or null
  uint16_t* y;
  int64_t y0_row, y_row, N;
  int R, strips;           // strips of a workgroup
};
template <int RK>
__global__ __launch_bounds__(kThreads) void up_kernel(const UpArgs a) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
  const Tile t = tile_of(a.plan, blockIdx.x);
  if (t.rows == 0) return;
  const bool bare = t.adapter >= a.plan.A;
  if (bare && a.y0 == a.y) return;
  const int blocks = (t.rows + 15) / 16;
  u32x4 tv[2][4][RK];
  int64_t row[4];
#pragma unroll
  for (int b = 0; b < 4; b++) {
    row[b] = 16 * b + r16 < t.rows ? row_at(a.plan, t.pos + 16 * b + r16) : -1;
#pragma unroll
    for (int k = 0; k < RK; k++)
#pragma unroll
      for (int h = 0; h < 2; h++) {
        tv[h][b][k] = u32x4{};
        if (!bare && b < blocks) tv[h][b][k] = a.t[(((int64_t)blockIdx.x * 2 + h) * 4 + b) * RK * 64 + k * 64 + lane];
      }
  }
  const uint16_t* w = a.w + (int64_t)(bare ? 0 : t.adapter) * a.N * a.R;
  struct Strip {
    u32x4 y[4], w[2][RK];
  };
  const int64_t all = (a.N + 31) / 32, first = (int64_t)blockIdx.y * a.strips, last = min(first + a.strips, all);
  auto fetch = [&](int64_t s, Strip& it) {
    if (s >= last) return;
    const int64_t n = s * 32 + 8 * q;
#pragma unroll
    for (int b = 0; b < 4; b++) {
      it.y[b] = u32x4{};
      if (a.y0 != nullptr && row[b] >= 0 && n < a.N) it.y[b] = *reinterpret_cast<const u32x4*>(a.y0 + row[b] * a.y0_row + n);
    }
#pragma unroll
    for (int b = 0; b < 2; b++) {
      const int64_t col = s * 32 + 8 * (r16 >> 2) + 4 * b + (r16 & 3);
#pragma unroll
      for (int k = 0; k < RK; k++) {
        it.w[b][k] = u32x4{};
        if (!bare && col < a.N && 32 * k + 8 * q < a.R) it.w[b][k] = *reinterpret_cast<const u32x4*>(w + col * a.R + 32 * k + 8 * q);
      }
    }
  };
  auto form = [&](int64_t s, const Strip& it) {
    const int64_t n = s * 32 + 8 * q;
#pragma unroll
    for (int b = 0; b < 4; b++) {
      if (b >= blocks) break;
      f32x4 c[2];
#pragma unroll
      for (int i = 0; i < 2; i++) {
        c[i] = f32x4{};
#pragma unroll
        for (int k = 0; k < RK; k++) {
          c[i] = mfma16(it.w[i][k], tv[0][b][k], c[i]);
          c[i] = mfma16(it.w[i][k], tv[1][b][k], c[i]);
        }
      }
      if (row[b] < 0 || n >= a.N) continue;
      u32x4 out;
#pragma unroll
      for (int i = 0; i < 4; i++)
        out[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)(bf16lo(it.y[b][i]) + c[i >> 1][2 * (i & 1)]),
                                                      (__bf16)(bf16hi(it.y[b][i]) + c[i >> 1][2 * (i & 1) + 1])});
      *reinterpret_cast<u32x4*>(a.y + row[b] * a.y_row + n) = out;
    }
  };
  Strip one, two;
  fetch(first + wave, one);
  for (int64_t s = first + wave; s < last; s += 2 * kWaves) {
    fetch(s + kWaves, two);
    form(s, one);
    if (s + kWaves >= last) break;
    fetch(s + 2 * kWaves, one);
    form(s + kWaves, two);
  }
}

// turn: in [A][rows][cols] to out [A][cols][rows], 64 x 64 elements a workgroup, for the adapters that
// have rows.
struct TurnArgs {
  Plan plan;
  const uint16_t* in[2];
  uint16_t* out[2];
  int64_t rows[2], cols[2];
  uint32_t tiles[2];  // workgroups of each
};
__global__ __launch_bounds__(kThreads) void turn_kernel(const TurnArgs a) {
  __shared__ uint16_t block[64][72];
  const int64_t adapter = blockIdx.y;
  if (a.plan.start[adapter] >= a.plan.start[adapter + 1]) return;
  const int k = blockIdx.x >= a.tiles[0];
  const int64_t rows = a.rows[k], cols = a.cols[k], wide = (cols + 63) / 64;
  const int64_t at = blockIdx.x - (k ? a.tiles[0] : 0), r0 = at / wide * 64, c0 = at % wide * 64;
  const uint16_t* in = a.in[k] + adapter * rows * cols;
  uint16_t* out = a.out[k] + adapter * rows * cols;
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int id = threadIdx.x + i * kThreads, r = id >> 3, c = id % 8 * 8;
    if (r0 + r < rows && c0 + c < cols)
      *reinterpret_cast<u32x4*>(&block[r][c]) = *reinterpret_cast<const u32x4*>(in + (r0 + r) * cols + c0 + c);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; i++) {
    const int id = threadIdx.x + i * kThreads, c = id & 63, r = (id >> 6) * 8;
    if (c0 + c < cols && r0 + r < rows) {
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; e++) v[e] = (uint32_t)block[r + 2 * e][c] | (uint32_t)block[r + 2 * e + 1][c] << 16;
      *reinterpret_cast<u32x4*>(out + (c0 + c) * rows + r0 + r) = v;
    }
  }
}

// grad: for C columns of Z (X for dL_B, dY for dL_A) and all R, the sum over a share of an adapter's rows
// of Z[row][c] S[row][r], S = dT or alpha T in parts (join's cols).  Share j of the launch is rows
// [i share, (i + 1) share) of adapter a where j = start[a] / share + a + i: every adapter, one
// without rows among them, has its own.  A share that is all of an adapter's rows goes to the
// output, the others to `part`, which grad_join adds.  The waves take 32 rows in turn: Z's rows go
// through the wave's own LDS, to be read with the rows along a lane (the transposing read), their
// 32-byte blocks swizzled so that the eight rows that half a wave reads lie in different banks.
struct GradArgs {
  Plan plan;
  const uint16_t* z[2];  // X, dY
  int64_t z_row[2], cols[2];
  uint32_t tiles[2];     // column tiles of each; 0 if its gradient is not wanted
  const u32x4* s[2];
  float* out[2];         // dL_B [A, R, K], dL_A [A, N, R]
  float* part[2];        // the same for each share
  int R, share;
};
template <int RB>
struct GradSize {
  static constexpr int CB = RB == 8 ? 4 : 8, C = 16 * CB;  // 32 blocks of 16 x 16 at the most
};

// Adapter of share j, and which of its shares.
__device__ __forceinline__ int share_of(const Plan& p, int64_t j, int share, int64_t& i) {
  int lo = 0, n = p.A;  // the last adapter whose first share is at or below j
  while (n > 1) {
    const int half = n / 2;
    if ((int64_t)p.start[lo + half] / share + lo + half <= j) {
      lo += half;
      n -= half;
    } else {
      n = half;
    }
  }
  i = j - ((int64_t)p.start[lo] / share + lo);
  return lo;
}

template <int RB, int PARTS, bool LA>
__device__ __forceinline__ void grad_tile(const GradArgs& a, uint8_t* lds, int64_t c0, int64_t j, int adapter, int64_t i,
                                          int64_t from, int64_t rows) {
  constexpr int CB = GradSize<RB>::CB, C = GradSize<RB>::C, PER = C / 8, LOADS = 32 * PER / 64, BLOCKS = CB * RB;
  constexpr int ROUND = BLOCKS < 16 ? BLOCKS : 16, STEP = 32 * kWaves;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
  const int64_t n = a.plan.start[adapter + 1] - a.plan.start[adapter];
  f32x4 acc[CB][RB];
#pragma unroll
  for (int c = 0; c < CB; c++)
#pragma unroll
    for (int b = 0; b < RB; b++) acc[c][b] = f32x4{};
  uint8_t* mine = lds + wave * 32 * C * 2;
  const int sub = lane / PER, p = lane % PER;
  const bool in = c0 + 8 * p < a.cols[LA];
  const uint16_t* z = a.z[LA] + c0 + 8 * p;
  // the share's first tile
  const int64_t tile = min(max(a.plan.tbase[adapter] + i * (a.share / kTile), (int64_t)0), a.plan.most - (rows + kTile - 1) / kTile);
  const u32x4* s = a.s[LA] + tile * PARTS * 2 * RB * 64 + lane;
  u32x4 zv[LOADS], sv[PARTS][RB];
  auto index = [&](int64_t r0) {  // lane l: row r0 + l % 32 of the share
    return r0 + (lane & 31) < rows ? (int)row_at(a.plan, from + r0 + (lane & 31)) : -1;
  };
  auto fetch_z = [&](int rows32) {
#pragma unroll
    for (int l = 0; l < LOADS; l++) {
      const int m = __shfl(rows32, l * (64 / PER) + sub, 64);
      zv[l] = u32x4{};
      if (m >= 0 && in) zv[l] = *reinterpret_cast<const u32x4*>(z + m * a.z_row[LA]);
    }
  };
  auto fetch_s = [&](int64_t r0) {
    const u32x4* t = s + (r0 / kTile * PARTS * 2 + r0 / 32 % 2) * RB * 64;
#pragma unroll
    for (int h = 0; h < PARTS; h++)
#pragma unroll
      for (int b = 0; b < RB; b++) sv[h][b] = t[(h * 2 * RB + b) * 64];
  };
  int64_t r0 = 32 * wave;
  int ahead = index(r0);
  if (r0 < rows) {
    fetch_z(ahead);
    fetch_s(r0);
  }
  ahead = index(r0 + STEP);
  for (; r0 < rows; r0 += STEP) {
#pragma unroll
    for (int l = 0; l < LOADS; l++) {
      const int r = l * (64 / PER) + sub, f = C == 128 ? (r & 3) | (r >> 3 & 1) << 2 : (r >> 1 & 1) | (r >> 3 & 1) << 1;
      *reinterpret_cast<u32x4*>(mine + r * C * 2 + ((((p >> 1) ^ f) << 1) | (p & 1)) * 16) = zv[l];
    }
    // the next rows' loads go out ahead of this step's products, those of S behind them, into the
    // registers that the products have read
    const bool more = r0 + STEP < rows;
    if (more) fetch_z(ahead);
    ahead = index(r0 + 2 * STEP);
    const int jr = (lane & 15) >> 2, f = C == 128 ? jr | (q & 1) << 2 : jr >> 1 | (q & 1) << 1;
    const uint8_t* at = mine + (8 * q + jr) * C * 2 + (lane & 3) * 8;
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int c = 0; c < CB; c++) {
      const uint8_t* block = at + ((c ^ f) << 5);
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
          (__attribute__((address_space(3))) bf16x4*)block));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
          (__attribute__((address_space(3))) bf16x4*)(block + 4 * C * 2)));
      const u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
      for (int h = 0; h < PARTS; h++)
#pragma unroll
        for (int b = 0; b < RB; b++) acc[c][b] = LA ? mfma16(sv[h][b], v, acc[c][b]) : mfma16(v, sv[h][b], acc[c][b]);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (more) fetch_s(r0 + STEP);
  }
  // the waves' sums, in one order; block (c, b): lane (r16, q) holds r = 16 b + r16 and columns 16 c +
  // 4q .. + 3 (dL_B), or column 16 c + r16 and r = 16 b + 4q .. + 3 (dL_A)
  f32x4(*sums)[ROUND][64] = reinterpret_cast<f32x4(*)[ROUND][64]>(lds);
  const int64_t cols = a.cols[LA];
  float* out = n <= a.share ? a.out[LA] + (int64_t)adapter * a.R * cols : a.part[LA] + j * a.R * cols;
#pragma unroll
  for (int round = 0; round < BLOCKS; round += ROUND) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROUND; k++) sums[wave][k][lane] = acc[(round + k) / RB][(round + k) % RB];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROUND / kWaves; k++) {
      const int at = k * kWaves + wave, c = (round + at) / RB, b = (round + at) % RB;
      f32x4 v = sums[0][at][lane];
#pragma unroll
      for (int w = 1; w < kWaves; w++) v += sums[w][at][lane];
      const int64_t col = c0 + 16 * c + (LA ? r16 : 4 * q);
      const int r = 16 * b + (LA ? 4 * q : r16);
      if (col < cols && r < a.R) *reinterpret_cast<f32x4*>(out + (LA ? col * a.R + r : r * cols + col)) = v;
    }
  }
}
template <int RB, int PARTS>
__global__ __launch_bounds__(kThreads, 2) void grad_kernel(const GradArgs a) {
  constexpr int C = GradSize<RB>::C, ROUND = GradSize<RB>::CB * RB < 16 ? GradSize<RB>::CB * RB : 16;
  __shared__ __align__(16) uint8_t lds[kWaves * (ROUND * 1024 > 64 * C ? ROUND * 1024 : 64 * C)];
  int64_t i;
  const int64_t j = blockIdx.y;
  const int adapter = __builtin_amdgcn_readfirstlane(share_of(a.plan, j, a.share, i));
  const int64_t first = a.plan.start[adapter], n = a.plan.start[adapter + 1] - first;
  if (i < 0 || i * a.share >= max(n, (int64_t)1)) return;
  const int64_t from = first + i * a.share, rows = max(min(n - i * a.share, (int64_t)a.share), (int64_t)0);
  if (first < 0 || from + rows > a.plan.M) return;
  if (blockIdx.x >= a.tiles[0]) grad_tile<RB, PARTS, true>(a, lds, (int64_t)(blockIdx.x - a.tiles[0]) * C, j, adapter, i, from, rows);
  else grad_tile<RB, PARTS, false>(a, lds, (int64_t)blockIdx.x * C, j, adapter, i, from, rows);
}

// The shares of the adapters that have several, added in their order.
__global__ __launch_bounds__(kThreads) void grad_join_kernel(const GradArgs a) {
  const int adapter = blockIdx.y, k = blockIdx.z;
  const int64_t first = a.plan.start[adapter], n = a.plan.start[adapter + 1] - first, size = a.R * a.cols[k];
  if (a.out[k] == nullptr || n <= a.share || first < 0 || first + n > a.plan.M) return;
  const int64_t at = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
  if (at >= size) return;
  const float* p = a.part[k] + (first / a.share + adapter) * size + at;
  f32x4 v{};
  const int64_t shares = (n + a.share - 1) / a.share;
#pragma unroll 4
  for (int64_t i = 0; i < shares; i++) v += *reinterpret_cast<const f32x4*>(p + i * size);
  *reinterpret_cast<f32x4*>(a.out[k] + adapter * size + at) = v;
}

// ---------------------------------------------------------------- launches

// Splits of a `down` over C channels: about two workgroups a CU, each with eight steps of 64 at least.
struct Splits {
  int count, steps;
};
Splits down_splits(int64_t tiles, int64_t C) {
  const int64_t steps = (C + 63) / 64;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(512 / tiles, steps / 8));
  const int64_t per = (steps + want - 1) / want;
  return Splits{(int)((steps + per - 1) / per), (int)per};
}

int rank_blocks(int64_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }
int rank_steps(int64_t R) { return (int)((R + 31) / 32); }
size_t rows_bytes(int64_t M, int64_t A, int64_t R) { return (size_t)max_tiles(M, A) * 2 * 4 * rank_steps(R) * 1024; }
// Parts of S in the gradients' sums.  Two hold it to 2^-16 of each element, 5e-6 of a sum of many rows; where
// rows are few and one may be most of a sum, three hold all of it, at half as many products again.
constexpr int64_t kFewRows = 1024;
int sum_parts(int64_t M) { return M <= kFewRows ? 3 : 2; }
size_t cols_bytes(int64_t M, int64_t A, int64_t R) { return (size_t)max_tiles(M, A) * sum_parts(M) * 2 * rank_blocks(R) * 1024; }

void down(const Plan& plan, const void* x, int64_t x_row, const void* w, int64_t C, int64_t R, float* part, hipStream_t stream) {
  const int64_t tiles = max_tiles(plan.M, plan.A);
  const Splits sp = down_splits(tiles, C);
  DownArgs a{plan, (const uint16_t*)x, (const uint16_t*)w, x_row, C, plan.M * R, (int)R, sp.steps, part};
  const dim3 grid((unsigned)tiles, (unsigned)sp.count);
  switch (rank_blocks(R)) {
    case 1: hipLaunchKernelGGL(down_kernel<1>, grid, dim3(kThreads), 0, stream, a); break;
    case 2: hipLaunchKernelGGL(down_kernel<2>, grid, dim3(kThreads), 0, stream, a); break;
    case 4: hipLaunchKernelGGL(down_kernel<4>, grid, dim3(kThreads), 0, stream, a); break;
    default: hipLaunchKernelGGL(down_kernel<8>, grid, dim3(kThreads), 0, stream, a); break;
  }
}

void join(const Plan& plan, const float* part, const float* kept, int splits, int64_t R, const float* alpha, float* t,
          void* rows, void* cols, hipStream_t stream) {
  const int width = std::max(32 * rank_steps(R), 16 * rank_blocks(R));
  JoinArgs a{plan, part, kept, plan.M * R, splits, (int)R, rank_steps(R), rank_blocks(R), width, alpha, t, (u32x4*)rows, (u32x4*)cols,
             sum_parts(plan.M)};
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)max_tiles(plan.M, plan.A)), dim3(kThreads),
                     (size_t)kTile * (width + 4) * 4, stream, a);
}

void up(const Plan& plan, const void* t, const void* w, const void* y0, int64_t y0_row, void* y, int64_t y_row, int64_t N,
        int64_t R, hipStream_t stream) {
  const int64_t tiles = max_tiles(plan.M, plan.A), all = (N + 31) / 32;
  // about four workgroups a CU, each wave with two strips at least
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>((1024 + tiles - 1) / tiles, all / 8));
  const int64_t strips = (all + want - 1) / want;
  UpArgs a{plan, (const u32x4*)t, (const uint16_t*)w, (const uint16_t*)y0, (uint16_t*)y, y0_row, y_row, N, (int)R, (int)strips};
  const dim3 grid((unsigned)tiles, (unsigned)((all + strips - 1) / strips));
  switch (rank_steps(R)) {
    case 1: hipLaunchKernelGGL(up_kernel<1>, grid, dim3(kThreads), 0, stream, a); break;
    case 2: hipLaunchKernelGGL(up_kernel<2>, grid, dim3(kThreads), 0, stream, a); break;
    case 3: hipLaunchKernelGGL(up_kernel<3>, grid, dim3(kThreads), 0, stream, a); break;
    default: hipLaunchKernelGGL(up_kernel<4>, grid, dim3(kThreads), 0, stream, a); break;
  }
}

size_t align(size_t n) { return (n + 255) & ~(size_t)255; }

size_t part_bytes(int64_t M, int64_t A, int64_t R, int64_t C) {
  return align((size_t)down_splits(max_tiles(M, A), C).count * M * R * 4);
}

// Rows of a share: enough shares to fill the chip with column tiles, each of 256 rows at least.
int64_t grad_share(int64_t M, int64_t A, int64_t R, int64_t K, int64_t N) {
  const int64_t C = rank_blocks(R) == 8 ? 64 : 128, tiles = (K + C - 1) / C + (N + C - 1) / C;
  const int64_t want = std::max<int64_t>(1, 768 / tiles);
  return std::max<int64_t>(256, ((M + want - 1) / want + 63) / 64 * 64);
}
int64_t grad_shares(int64_t M, int64_t A, int64_t share) { return M / share + A; }
bool grad_splits(int64_t M, int64_t share) { return M > share; }

}  // namespace

size_t adapters_plan_bytes(int64_t M, int64_t A) {
  size_t tiles, order;
  return plan_words(M, A, &tiles, &order) * 4;
}

hipError_t launch_adapters_plan(const int32_t* ids, int64_t M, int64_t A, void* plan, hipStream_t stream) {
  size_t tiles, order;
  plan_words(M, A, &tiles, &order);
  int32_t* w = (int32_t*)plan;
  hipLaunchKernelGGL(plan_kernel, dim3((unsigned)(A + 1)), dim3(kThreads), (size_t)(2 * A + 3) * 4, stream, ids, M, (int)A, w,
                     (int4*)(w + tiles), w + order);
  return hipGetLastError();
}

size_t adapters_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A) {
  return part_bytes(M, A, R, K) + align(rows_bytes(M, A, R));
}

hipError_t launch_adapters(const AdapterCall& c, const void* y0, int64_t y0_row, void* y, int64_t y_row, float* t, void* ws,
                           hipStream_t stream) {
  const Plan plan = plan_of(c.plan, c.M, c.A);
  float* part = (float*)ws;
  void* rows = (uint8_t*)ws + part_bytes(c.M, c.A, c.R, c.K);
  down(plan, c.x, c.x_row, c.LB, c.K, c.R, part, stream);
  join(plan, part, nullptr, down_splits(max_tiles(c.M, c.A), c.K).count, c.R, c.alpha, t, rows, nullptr, stream);
  up(plan, rows, c.LA, y0, y0_row, y, y_row, c.N, c.R, stream);
  return hipGetLastError();
}

// Workspace of the gradient: L_A^T, L_B^T | parts of dT | operands of dT, of dT and T transposed | shares.
size_t adapters_back_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A) {
  const int64_t share = grad_share(M, A, R, K, N);
  return align((size_t)A * N * R * 2) + align((size_t)A * K * R * 2) + part_bytes(M, A, R, N) + align(rows_bytes(M, A, R)) +
         2 * align(cols_bytes(M, A, R)) + (grad_splits(M, share) ? align((size_t)grad_shares(M, A, share) * R * (K + N) * 4) : 0);
}

hipError_t launch_adapters_back(const AdapterCall& c, const float* t, const void* dy, int64_t dy_row, const void* dx0,
                                int64_t dx0_row, void* dx, int64_t dx_row, float* dla, float* dlb, void* ws,
                                hipStream_t stream) {
  const Plan plan = plan_of(c.plan, c.M, c.A);
  const int64_t share = grad_share(c.M, c.A, c.R, c.K, c.N);
  uint8_t* at = (uint8_t*)ws;
  auto take = [&](size_t bytes) {
    void* p = at;
    at += align(bytes);
    return p;
  };
  void* lat = take((size_t)c.A * c.N * c.R * 2);
  void* lbt = take((size_t)c.A * c.K * c.R * 2);
  float* part = (float*)take(part_bytes(c.M, c.A, c.R, c.N));
  void* rows = take(rows_bytes(c.M, c.A, c.R));
  void* dcols = take(cols_bytes(c.M, c.A, c.R));
  void* tcols = take(cols_bytes(c.M, c.A, c.R));
  float* shares = (float*)at;
  const bool dt = dx != nullptr || dlb != nullptr;
  if (dt) {
    TurnArgs a{};
    a.plan = plan;
    a.in[0] = (const uint16_t*)c.LA;
    a.out[0] = (uint16_t*)lat;
    a.rows[0] = c.N;
    a.cols[0] = c.R;
    a.in[1] = (const uint16_t*)c.LB;
    a.out[1] = (uint16_t*)lbt;
    a.rows[1] = c.R;
    a.cols[1] = c.K;
    a.tiles[0] = (uint32_t)(((c.N + 63) / 64) * ((c.R + 63) / 64));
    a.tiles[1] = dx != nullptr ? (uint32_t)(((c.K + 63) / 64) * ((c.R + 63) / 64)) : 0;
    hipLaunchKernelGGL(turn_kernel, dim3(a.tiles[0] + a.tiles[1], (unsigned)c.A), dim3(kThreads), 0, stream, a);
    down(plan, dy, dy_row, lat, c.N, c.R, part, stream);
    join(plan, part, nullptr, down_splits(max_tiles(c.M, c.A), c.N).count, c.R, c.alpha, nullptr, dx != nullptr ? rows : nullptr,
         dlb != nullptr ? dcols : nullptr, stream);
  }
  if (dla != nullptr) join(plan, nullptr, t, 0, c.R, c.alpha, nullptr, nullptr, tcols, stream);
  if (dx != nullptr) up(plan, rows, lbt, dx0, dx0_row, dx, dx_row, c.K, c.R, stream);
  if (dla != nullptr || dlb != nullptr) {
    const int64_t C = rank_blocks(c.R) == 8 ? 64 : 128;
    GradArgs a{};
    a.plan = plan;
    a.z[0] = (const uint16_t*)c.x;
    a.z_row[0] = c.x_row;
    a.cols[0] = c.K;
    a.z[1] = (const uint16_t*)dy;
    a.z_row[1] = dy_row;
    a.cols[1] = c.N;
    a.s[0] = (const u32x4*)dcols;
    a.s[1] = (const u32x4*)tcols;
    a.out[0] = dlb;
    a.out[1] = dla;
    a.tiles[0] = dlb != nullptr ? (uint32_t)((c.K + C - 1) / C) : 0;
    a.tiles[1] = dla != nullptr ? (uint32_t)((c.N + C - 1) / C) : 0;
    a.part[0] = shares;
    a.part[1] = shares + grad_shares(c.M, c.A, share) * c.R * c.K;
    a.R = (int)c.R;
    a.share = (int)share;
    const dim3 grid(a.tiles[0] + a.tiles[1], (unsigned)grad_shares(c.M, c.A, share));
    auto go = [&](auto parts) {
      constexpr int P = decltype(parts)::value;
      switch (rank_blocks(c.R)) {
        case 1: hipLaunchKernelGGL((grad_kernel<1, P>), grid, dim3(kThreads), 0, stream, a); break;
        case 2: hipLaunchKernelGGL((grad_kernel<2, P>), grid, dim3(kThreads), 0, stream, a); break;
        case 4: hipLaunchKernelGGL((grad_kernel<4, P>), grid, dim3(kThreads), 0, stream, a); break;
        default: hipLaunchKernelGGL((grad_kernel<8, P>), grid, dim3(kThreads), 0, stream, a); break;
      }
    };
    if (sum_parts(c.M) == 3) go(std::integral_constant<int, 3>());
    else go(std::integral_constant<int, 2>());
    if (grad_splits(c.M, share)) {
      const int64_t most = c.R * std::max(c.K, c.N) / 4;
      hipLaunchKernelGGL(grad_join_kernel, dim3((unsigned)((most + kThreads - 1) / kThreads), (unsigned)c.A, 2), dim3(kThreads), 0,
                         stream, a);
    }
  }
  return hipGetLastError();
}

}  // namespace rtl
