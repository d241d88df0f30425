// adapters.h -- low-rank adapters of many requests beside a shared projection, and their gradient.
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
// the next products in three bf16 parts (three_parts), all 24 digits.  One would leave 2^-9 of an adapter's
// share, two 2^-16; the products are too small to hold the kernels (up with three parts and with two: 24 rows of 5120 -> 13824,
// R = 32 8.0 and 7.6 us; 4608 of 2560 -> 7680, R = 64 39 and 37; 32760 of 5120 -> 5120, R = 64 145 and 141, join 11 and 10).
// 32760 rows of 5120 -> 5120, R = 64: down 102 us, join 11, up 145; a read of X takes 60, a copy of Y0 to Y 120.
// (The gradients' sums, which leave in fp32, were 5e-6 off with two.)
//
//   down:   T in pieces over K, the waves taking 64 of K in turn
//   join:   T's pieces summed, T in the layouts of the products that it enters
//   up:     Y0 + T L_A^T, strips of 64 columns a wave
//   turn:   factors transposed, which makes dT a `down` and dX an `up`
//   grad:   dL_B and dL_A, tiles of 256 (128) columns by R over runs of an adapter's rows
#pragma once
#include <algorithm>
#include <type_traits>

#include "bf16_common.h"

namespace rtl {

namespace lora {

constexpr int kTile = 64;     // rows of a tile
constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kParts = 3;     // of T and dT in the next products

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
// own adapters in their order, a thread four rows at a time.  Bound: the two passes' latency (32760 rows: 97 us
// with 256 threads of a row each, 34 so).
constexpr int kPlanThreads = 1024, kPlanWaves = kPlanThreads / 64, kPlanRows = 4;
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int32_t* ids, int64_t M, int A, int32_t* head, int4* tiles,
                                                        int32_t* order) {
  extern __shared__ int32_t lds[];
  int32_t* count = lds;           // [A + 1], then the first positions
  int32_t* first = lds + A + 1;   // [A + 2] first tiles
  __shared__ int32_t wave_sum[2][kPlanWaves][2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int a = threadIdx.x; a <= A; a += kPlanThreads) count[a] = 0;
  __syncthreads();
  auto key = [&](int64_t m) {
    const int a = ids[m];
    return a < 0 || a >= A ? A : a;
  };
  for (int64_t m0 = 0; m0 < M; m0 += kPlanThreads * kPlanRows) {
    int of[kPlanRows];
#pragma unroll
    for (int i = 0; i < kPlanRows; i++) {
      const int64_t m = m0 + i * kPlanThreads + threadIdx.x;
      of[i] = m < M ? key(m) : -1;
    }
#pragma unroll
    for (int i = 0; i < kPlanRows; i++) {
      // one count for a wave of one adapter
      const int k0 = __builtin_amdgcn_readfirstlane(of[i]);
      const uint64_t same = __ballot(of[i] == k0);
      if (k0 >= 0 && lane == 0) atomicAdd(&count[k0], __popcll(same));
      if (of[i] >= 0 && of[i] != k0) atomicAdd(&count[of[i]], 1);
    }
  }
  __syncthreads();
  // first positions and tiles: sums over the adapters before, kPlanThreads at a time
  int32_t rows_before = 0, tiles_before = 0;
  for (int a0 = 0; a0 <= A; a0 += kPlanThreads) {
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
      wave_sum[0][wave][0] = sn;
      wave_sum[0][wave][1] = st;
    }
    __syncthreads();
    for (int w = 0; w < wave; w++) {
      sn += wave_sum[0][w][0];
      st += wave_sum[0][w][1];
    }
    if (a <= A) {
      count[a] = rows_before + sn - n;
      first[a] = tiles_before + st - t;
    }
    for (int w = 0; w < kPlanWaves; w++) {
      rows_before += wave_sum[0][w][0];
      tiles_before += wave_sum[0][w][1];
    }
    __syncthreads();
  }
  if (blockIdx.x == 0) {
    for (int a = threadIdx.x; a <= A; a += kPlanThreads) {
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
    for (int t = threadIdx.x; t * kTile < n; t += kPlanThreads) tiles[first[a] + t] = make_int4(a, from + t * kTile, min(kTile, n - t * kTile), 0);
    int32_t at = from;
    int turn = 0;
    for (int64_t m0 = 0; m0 < M && at < from + n; m0 += kPlanThreads * kPlanRows) {  // at: the same in all threads
      const int64_t m = m0 + threadIdx.x * kPlanRows;
      bool mine[kPlanRows];
      int sum = 0;
#pragma unroll
      for (int i = 0; i < kPlanRows; i++) {
        mine[i] = m + i < M && key(m + i) == a;
        sum += mine[i];
      }
      int to = sum;  // inclusive sum over the wave
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(to, o, 64);
        if (lane >= o) to += up;
      }
      if (lane == 63) wave_sum[turn][wave][0] = to;
      __syncthreads();
      to += at - sum;
      for (int w = 0; w < kPlanWaves; w++) {
        const int of_wave = wave_sum[turn][w][0];
        if (w < wave) to += of_wave;
        at += of_wave;
      }
      turn ^= 1;  // two sets: the next sums are written while a wave may still read these
#pragma unroll
      for (int i = 0; i < kPlanRows; i++) {
        if (mine[i] && to < from + n) order[to] = (int32_t)(m + i);
        to += mine[i];
      }
    }
    __syncthreads();
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
// Work in equal shares: `tiles` tiles of `steps` steps each, one after another, are dealt out to `groups`
// workgroups, `least` steps each at the least; a workgroup goes through its pieces of tiles.  All workgroups
// run at once and end together, where whole tiles, one a workgroup, left half the chip idle in the last
// round (down at 32760 x 5120, 514 tiles on 512 places: 141 us).  The piece of a tile that workgroup w
// has is number w + tile (pieces in order raise one or the other).
struct Stream {
  int64_t steps;
  int groups, least;
  __device__ __forceinline__ int64_t len(int64_t tiles) const {
    return max((tiles * steps + groups - 1) / groups, (int64_t)least);
  }
  // First and last workgroup of a tile.
  __device__ __forceinline__ void of(int64_t tile, int64_t len, int64_t& first, int64_t& last) const {
    first = min(tile * steps / len, (int64_t)groups - 1);
    last = min((tile * steps + steps - 1) / len, (int64_t)groups - 1);
  }
};
// Tiles of rows with an adapter (they come first), and all of them.
__device__ __forceinline__ int64_t used_tiles(const Plan& p) { return min(max((int64_t)p.tbase[p.A], (int64_t)0), p.most); }
__device__ __forceinline__ int64_t all_tiles(const Plan& p) { return min(max((int64_t)*p.count, (int64_t)0), p.most); }

__device__ __forceinline__ int64_t row_at(const Plan& p, int64_t pos) {
  return min(max(p.order[pos], 0), (int)p.M - 1);
}

// Keeps the loads of the next step ahead of this step's products: the compiler would move them to
// where they are used, to save registers (down at 32760 x 5120: 150 us without).
__device__ __forceinline__ void hold() { __builtin_amdgcn_sched_barrier(0); }

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ void parts_of(const float (&v)[8], u32x4 (&w)[kParts]) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int i = 0; i < 4; i++) {
    __bf16 x[3], y[3];
    three_parts(v[2 * i], x);
    three_parts(v[2 * i + 1], y);
#pragma unroll
    for (int k = 0; k < kParts; k++) w[k][i] = __builtin_bit_cast(uint32_t, bf16x2_t{x[k], y[k]});
  }
}

// join: T of half a tile, 32 rows, the sum of down's pieces or (kept) its rows as they are; unscaled to `t`, and scaled
// by alpha in bf16 parts as the products take it: `rows`, up's operand, [tile][part][block of 16 rows][RK][lane]
// (lane (r16, q): row r16, r = 8q .. 8q + 7 of 32), and `cols`, grad's, [tile][part][half][RB][lane] (r =
// r16 of a block, rows 8q .. 8q + 7 of the half).  Rows past the tile's are zeros, and r past R up to 32 RK; `cols` past
// that (R of 72 to 96 in blocks for 128) hold what lies there, in sums that grad does not store.
// A launch of its own: summed by each workgroup of up that needed it, T cost 8 to 19 us of up's time
// (4608 rows, 2560 -> 7680, R = 64, 72 tiles of up to 8 pieces on 512 workgroups: 53 us for 35; this takes 6), but
// for the few rows of join_here.
struct JoinArgs {
  Plan plan;
  const float *part, *kept;  // one of them
  Stream down;
  const float* alpha;        // [A] or null
  float* t;                  // [M, R] by row, or null
  u32x4 *rows, *cols;        // or null
  int R, RB, RK;             // R in 16s as grad takes them, in 32s as up does
};
constexpr int kJoinThreads = 512;
constexpr int kJoinHere = 16;  // rows of a batch up to which up joins (join_here)
constexpr int join_pitch(int RK) { return 32 * RK + 4; }
// T of ROWS rows of a tile from row m0 on, scaled to `lds`, unscaled to a.t (put).
template <int THREADS, int ROWS>
__device__ __forceinline__ void sum_rows(const JoinArgs& a, const Tile& t, int64_t index, int m0, int64_t down_len, bool put, float* lds) {
  const int left = t.rows - m0, R = a.R, wide = 8 * a.RK, pitch = join_pitch(a.RK);
  const bool bare = t.adapter >= a.plan.A;
  const float alpha = bare || a.alpha == nullptr ? 1.f : a.alpha[t.adapter];
  int64_t first = 0, last = -1;
  if (a.kept != nullptr) last = 0;
  else if (!bare) a.down.of(index, down_len, first, last);
  for (int id = threadIdx.x; id < ROWS * wide; id += THREADS) {
    const int m = id / wide, r = id % wide * 4;
    f32x4 v{};
    if (m < left && r < R) {
      const int64_t row = row_at(a.plan, t.pos + m0 + m);
      if (a.kept != nullptr) {
        v = *reinterpret_cast<const f32x4*>(a.kept + row * R + r);
      } else {
        const float* p = a.part + ((first + index) * kTile + m0 + m) * R + r;
#pragma unroll 8
        for (int64_t w = first; w <= last; w++, p += kTile * R) v += *reinterpret_cast<const f32x4*>(p);
      }
      if (put) *reinterpret_cast<f32x4*>(a.t + row * R + r) = v;
    }
    *reinterpret_cast<f32x4*>(lds + m * pitch + r) = v * alpha;
  }
}
// up's operand of BLOCKS blocks of 16 rows; its parts lie 4 RK 64 apart.
template <int THREADS, int BLOCKS>
__device__ __forceinline__ void form_rows(int RK, const float* lds, u32x4* to) {
  const int pitch = join_pitch(RK);
  for (int id = threadIdx.x; id < BLOCKS * RK * 64; id += THREADS) {
    const int lane = id & 63, k = (id >> 6) % RK, block = (id >> 6) / RK;
    const float* p = lds + (16 * block + (lane & 15)) * pitch + 32 * k + 8 * (lane >> 4);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = p[i];
    u32x4 w[kParts];
    parts_of(v, w);
#pragma unroll
    for (int h = 0; h < kParts; h++) to[id + h * 4 * RK * 64] = w[h];
  }
}
template <int THREADS>
__device__ __forceinline__ void join_half(const JoinArgs& a, int64_t index, int half, float* lds) {
  const Tile t = tile_of(a.plan, index);
  const bool bare = t.adapter >= a.plan.A;
  if (t.rows == 0 || (bare && (a.t == nullptr || t.rows <= 32 * half))) return;
  sum_rows<THREADS, 32>(a, t, index, 32 * half, a.kept != nullptr ? 1 : a.down.len(used_tiles(a.plan)), a.t != nullptr, lds);
  if (bare) return;
  __syncthreads();
  if (a.rows != nullptr) form_rows<THREADS, 2>(a.RK, lds, a.rows + (index * 4 * kParts + 2 * half) * a.RK * 64);
  if (a.cols != nullptr) {
    const int n = 2 * a.RB * 64;
    const int pitch = join_pitch(a.RK);
    u32x4* to = a.cols + index * kParts * n + half * a.RB * 64;
    for (int id = threadIdx.x; id < a.RB * 64; id += THREADS) {
      const int lane = id & 63;
      const float* p = lds + 8 * (lane >> 4) * pitch + 16 * (id >> 6) + (lane & 15);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = p[i * pitch];
      u32x4 w[kParts];
      parts_of(v, w);
#pragma unroll
      for (int k = 0; k < kParts; k++) to[k * n + id] = w[k];
    }
  }
}
__global__ __launch_bounds__(kJoinThreads) void join_kernel(const JoinArgs a) {
  __shared__ __align__(16) float lds[32 * join_pitch(4)];
  join_half<kJoinThreads>(a, blockIdx.x >> 1, blockIdx.x & 1, lds);
}

// Memory is met in whole lines, eight rows of 128 bytes an access with a row's eight chunks in neighbouring lanes, and
// passes through the wave's own LDS to and from the matrix instructions' layout (lane (r16, q): chunks q and 4 + q
// of row r16; line_at is free of bank conflicts both ways).  Read as the instructions have it, neighbouring lanes on
// different rows, every lane is an access of its own: 63 of them an instruction instead of 16, the address and data
// units 85% busy, and down and up at 32760 x 5120, R = 64, took 105 and 170 us instead of 99 and 142 (T in
// two parts).  The LDS
// is the wave's own and its instructions run in order: no barrier, only an order that the compiler keeps between
// what one lane writes and another reads (in_order, which leaves no instruction).
__device__ __forceinline__ void in_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local"); }
__device__ __forceinline__ int line_at(int row, int chunk) { return row * 128 + ((chunk ^ (row & 7)) << 4); }

// down: piece[row][r] of a tile = sum over the piece's K of X[row][k] W[adapter][r][k].  The waves take 64 of
// K in turn, each with all the rows and all R, so that nothing is loaded twice, and their sums are added in LDS in one
// order.  Blocks of 16 r by 16 rows: lane (r16, q) of a block holds row r16 and r = 4q .. 4q + 3.
// The loop has no condition but its count: the last loads repeat.
struct DownArgs {
  Plan plan;
  const uint16_t *x, *w;  // [M, K] with a row stride, [A, R, K]
  int64_t x_row, K;
  int R;
  Stream stream;
  float* part;            // [pieces][64][R]
};
// Workgroups a CU, by their registers.
constexpr int down_per_cu(int RB) { return RB == 8 ? 1 : RB == 4 ? 2 : 3; }  // and LDS
template <int RB, int MB>  // MB: blocks of rows
__device__ __forceinline__ void down_piece(const DownArgs& a, const Tile& t, int64_t first, int64_t last, float* part, uint8_t* lds) {
  constexpr int BLOCKS = MB * RB, ROUND = BLOCKS < 8 ? BLOCKS : 8;
  static_assert(BLOCKS % ROUND == 0, "whole rounds");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
  const int64_t whole = a.K / 64, end = min(last, whole);
  const int row = lane >> 3, chunk = lane & 7;  // of an access
  const uint16_t* xp[MB][2];
#pragma unroll
  for (int b = 0; b < MB; b++)
#pragma unroll
    for (int i = 0; i < 2; i++)  // rows past the last repeat it: their sums are dropped
      xp[b][i] = a.x + row_at(a.plan, t.pos + min(16 * b + 8 * i + row, t.rows - 1)) * a.x_row + (first + wave) * 64 + 8 * chunk;
  // eight r past R repeat R's last eight
  const uint16_t* w0 = a.w + (int64_t)t.adapter * a.R * a.K + (first + wave) * 64;
  const uint32_t w_lane = (uint32_t)(row * a.K + 8 * chunk);
  auto wp = [&](int b, int i) { return w0 + (int64_t)min(16 * b + 8 * i, a.R - 8) * a.K; };
  uint8_t* mine = lds + wave * ((4 + RB) * 2048);  // blocks of X, then of W
  f32x4 acc[MB][RB];
#pragma unroll
  for (int b = 0; b < MB; b++)
#pragma unroll
    for (int c = 0; c < RB; c++) acc[b][c] = f32x4{};
  u32x4 x[MB][2], w[RB][2];
  const int64_t count = max((end - first - wave + kWaves - 1) / kWaves, (int64_t)0);
  auto fetch = [&](int64_t i) {
    const int64_t k = min(i, count - 1) * (64 * kWaves);
#pragma unroll
    for (int b = 0; b < RB; b++)
#pragma unroll
      for (int i = 0; i < 2; i++) w[b][i] = *reinterpret_cast<const u32x4*>(wp(b, i) + k + w_lane);
#pragma unroll
    for (int b = 0; b < MB; b++)
#pragma unroll
      for (int i = 0; i < 2; i++) x[b][i] = *reinterpret_cast<const u32x4*>(xp[b][i] + k);
  };
  auto put = [&]() {
    in_order();
#pragma unroll
    for (int i = 0; i < 2; i++) {
#pragma unroll
      for (int b = 0; b < RB; b++) *reinterpret_cast<u32x4*>(mine + (4 + b) * 2048 + line_at(8 * i + row, chunk)) = w[b][i];
#pragma unroll
      for (int b = 0; b < MB; b++) *reinterpret_cast<u32x4*>(mine + b * 2048 + line_at(8 * i + row, chunk)) = x[b][i];
    }
    in_order();
  };
  auto form = [&]() {
#pragma unroll
    for (int h = 0; h < 2; h++) {
      u32x4 f[RB];
#pragma unroll
      for (int c = 0; c < RB; c++) f[c] = *reinterpret_cast<const u32x4*>(mine + (4 + c) * 2048 + line_at(r16, 4 * h + q));
#pragma unroll
      for (int b = 0; b < MB; b++) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(mine + b * 2048 + line_at(r16, 4 * h + q));
#pragma unroll
        for (int c = 0; c < RB; c++) acc[b][c] = mfma16(f[c], v, acc[b][c]);
      }
    }
  };
  __syncthreads();  // the sums that lie there are read
  if (count > 0) {
    fetch(0);
    for (int64_t i = 0; i < count; i++) {
      put();
      hold();
      fetch(i + 1);
      hold();
      form();
      hold();
    }
  }
  // what K leaves past its whole steps, by the wave whose turn it is
  if (last > whole && (whole - first) % kWaves == wave) {
    const int64_t k = (whole - first - wave) * 64;
    const bool in = whole * 64 + 8 * chunk < a.K;
#pragma unroll
    for (int i = 0; i < 2; i++) {
#pragma unroll
      for (int b = 0; b < MB; b++) x[b][i] = in ? *reinterpret_cast<const u32x4*>(xp[b][i] + k) : u32x4{};
#pragma unroll
      for (int b = 0; b < RB; b++) w[b][i] = in ? *reinterpret_cast<const u32x4*>(wp(b, i) + k + w_lane) : u32x4{};
    }
    put();
    form();
  }
  f32x4(*sums)[ROUND][64] = reinterpret_cast<f32x4(*)[ROUND][64]>(lds);
#pragma unroll
  for (int round = 0; round < BLOCKS; round += ROUND) {
    __syncthreads();  // what lay there is read
#pragma unroll
    for (int i = 0; i < ROUND; i++) sums[wave][i][lane] = acc[(round + i) / RB][(round + i) % RB];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < (ROUND + kWaves - 1) / kWaves; i++) {
      const int at = i * kWaves + wave, b = (round + at) / RB, c = (round + at) % RB;
      const int m = 16 * b + r16, r = 16 * c + 4 * q;
      if (at >= ROUND) continue;
      f32x4 v = sums[0][at][lane];
#pragma unroll
      for (int w = 1; w < kWaves; w++) v += sums[w][at][lane];
      if (m < t.rows && r < a.R) *reinterpret_cast<f32x4*>(part + m * a.R + r) = v;
    }
  }
}
template <int RB>
__global__ __launch_bounds__(kThreads, down_per_cu(RB)) void down_kernel(const DownArgs a) {
  __shared__ __align__(16) uint8_t lds[kWaves * (4 + RB) * 2048];  // the waves' lines, then their sums
  const int64_t tiles = used_tiles(a.plan), len = a.stream.len(tiles);
  int64_t at = blockIdx.x * len;
  const int64_t end = min(at + len, tiles * a.stream.steps);
  while (at < end) {
    const int64_t index = at / a.stream.steps, first = at - index * a.stream.steps, last = min(a.stream.steps, first + end - at);
    at += last - first;
    const Tile t = tile_of(a.plan, index);
    if (t.rows == 0 || t.adapter >= a.plan.A) continue;
    float* part = a.part + (blockIdx.x + index) * (int64_t)(kTile * a.R);
    if (t.rows <= 16) down_piece<RB, 1>(a, t, first, last, part, lds);
    else down_piece<RB, 4>(a, t, first, last, part, lds);
  }
}

// up: Y[row][n] = Y0[row][n] + sum over r of T[row][r] W[adapter][n][r].  The waves of a workgroup take the
// strips of 64 columns of its piece of a tile in turn, with the tile's T (join's rows) in LDS.  A strip is four blocks of columns: half s takes columns 32 s + 8 (i / 4) + 4 b + i % 4 into its
// blocks b = 0, 1, so that lane (r16, q) ends with columns 32 s + 8q .. + 7 of row r16.  Y0, Y and the factors pass in whole
// lines.
struct UpArgs {
  Plan plan;
  const uint16_t *w, *y0;  // [A, N, R]; [M, N] with a row stride, or null
  uint16_t* y;
  int64_t y0_row, y_row, N;
  int R;
  Stream stream;
  const u32x4* t;
  JoinArgs join;  // JOIN
};
// Workgroups a CU, by their registers.
constexpr int up_per_cu(int RK) { return RK <= 2 ? 2 : 1; }  // and LDS
// A wave's LDS: two blocks of rows and a strip's factors.
constexpr int up_lines(int RK) { return 2 * 2048 + RK * 4096; }
// MB: blocks of rows.  JOIN: T is summed here, in place of join's launch.
template <int RK, bool ADD, bool JOIN, int MB>
__device__ __forceinline__ void up_piece(const UpArgs& a, const Tile& t, int64_t index, int64_t first, int64_t last,
                                         int64_t down_len, u32x4* operands, uint8_t* lines) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  constexpr int PER = 4 * RK, WL = 64 * PER / 64;  // chunks of a factor's row, accesses of a strip's factors
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
  const int R = a.R, l8 = lane >> 3, chunk = lane & 7;
  const u32x4* tv = operands + lane;
  uint8_t *mine = lines + wave * up_lines(RK), *mine_w = mine + 2 * 2048;
  const int64_t whole = a.N / 64, end = min(last, whole), n0 = (first + wave) * 64;
  // Factors: access j takes chunks 64 j + lane of the strip's 64 columns, PER each; r past R as zeros.  In LDS column n's
  // chunk c lies so that the columns of 8 neighbouring lanes of a block fall in different banks.
  auto w_at = [](int n, int c) {
    const int g = RK % 2 ? n >> 3 & 1 : (n & 3) | (n >> 3 & 1) << 2;
    return n * (PER * 16) + ((c ^ g) << 4);
  };
  const uint16_t* w0 = a.w + ((int64_t)t.adapter * a.N + n0) * R;
  int w_off[WL];  // -1: past R
  int w_to[WL];
#pragma unroll
  for (int j = 0; j < WL; j++) {
    const int n = (64 * j + lane) / PER, c = (64 * j + lane) % PER;
    w_off[j] = 8 * c < R ? n * R + 8 * c : -1;
    w_to[j] = w_at(n, c);
  }
  const uint16_t* yp[MB][2];
  int row[MB][2];  // -1: past the last, which is repeated and not stored
#pragma unroll
  for (int b = 0; b < MB; b++)
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int m = 16 * b + 8 * i + l8, at = (int)row_at(a.plan, t.pos + min(m, t.rows - 1));
      yp[b][i] = ADD ? a.y0 + at * a.y0_row + n0 + 8 * chunk : nullptr;
      row[b][i] = m < t.rows ? at : -1;
    }
  uint16_t* op = a.y + n0 + 8 * chunk;
  u32x4 y[MB][2], w[WL];
  const int64_t count = max((end - first - wave + kWaves - 1) / kWaves, (int64_t)0);
  auto place = [&](int64_t i) { return min(i, count - 1) * (64 * kWaves); };
  auto fetch_y = [&](int64_t n, int b) {
#pragma unroll
    for (int k = 0; k < 2; k++) y[b][k] = ADD ? *reinterpret_cast<const u32x4*>(yp[b][k] + n) : u32x4{};
  };
  auto fetch_w = [&](int64_t n) {
#pragma unroll
    for (int j = 0; j < WL; j++) w[j] = w_off[j] >= 0 ? *reinterpret_cast<const u32x4*>(w0 + n * R + w_off[j]) : u32x4{};
  };
  u32x4 f[4][RK];
  auto ready = [&]() {
    in_order();
#pragma unroll
    for (int j = 0; j < WL; j++) *reinterpret_cast<u32x4*>(mine_w + w_to[j]) = w[j];
    in_order();
#pragma unroll
    for (int c = 0; c < 4; c++)
#pragma unroll
      for (int k = 0; k < RK; k++)
        f[c][k] = *reinterpret_cast<const u32x4*>(mine_w + w_at(32 * (c >> 1) + 8 * (r16 >> 2) + 4 * (c & 1) + (r16 & 3), 4 * k + q));
  };
  auto form = [&](int64_t n, int b, bool in) {
    uint8_t* block = mine + (b & 1) * 2048;
    u32x4 v[2], tb[kParts][RK];
    in_order();
    if (ADD) {
#pragma unroll
      for (int i = 0; i < 2; i++) *reinterpret_cast<u32x4*>(block + line_at(8 * i + l8, chunk)) = y[b][i];
      in_order();
#pragma unroll
      for (int s = 0; s < 2; s++) v[s] = *reinterpret_cast<const u32x4*>(block + line_at(r16, 4 * s + q));
    } else {
      v[0] = v[1] = u32x4{};
    }
#pragma unroll
    for (int k = 0; k < RK; k++)
#pragma unroll
      for (int h = 0; h < kParts; h++) tb[h][k] = tv[((h * 4 + b) * RK + k) * 64];
    in_order();
#pragma unroll
    for (int s = 0; s < 2; s++) {
      u32x4 out;
#pragma unroll
      for (int c = 0; c < 2; c++) {
        f32x4 z = {bf16lo(v[s][2 * c]), bf16hi(v[s][2 * c]), bf16lo(v[s][2 * c + 1]), bf16hi(v[s][2 * c + 1])};
#pragma unroll
        for (int k = 0; k < RK; k++)
#pragma unroll
          for (int h = 0; h < kParts; h++) z = mfma16(f[2 * s + c][k], tb[h][k], z);
        out[2 * c] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)z[0], (__bf16)z[1]});
        out[2 * c + 1] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)z[2], (__bf16)z[3]});
      }
      *reinterpret_cast<u32x4*>(block + line_at(r16, 4 * s + q)) = out;
    }
    in_order();
#pragma unroll
    for (int k = 0; k < 2; k++) {
      const u32x4 out = *reinterpret_cast<const u32x4*>(block + line_at(8 * k + l8, chunk));
      if (row[b][k] >= 0 && in) *reinterpret_cast<u32x4*>(op + (int64_t)row[b][k] * a.y_row + n) = out;
    }
  };
  if (count > 0) {
    fetch_w(0);
#pragma unroll
    for (int b = 0; b < MB; b++) fetch_y(0, b);
  }
  if constexpr (JOIN) {
    float* tile = reinterpret_cast<float*>(lines);
    __syncthreads();  // the tile before is read
    sum_rows<kThreads, 16 * MB>(a.join, t, index, 0, down_len, a.join.t != nullptr && first == 0, tile);
    __syncthreads();
    form_rows<kThreads, MB>(RK, tile, operands);
    __syncthreads();
  } else {  // T, behind the first loads
    const u32x4* t_from = a.t + index * (4 * kParts * RK * 64);
    u32x4 v[kParts * RK];
    static_assert(kThreads == 4 * 64, "a part's blocks of RK in RK accesses");
#pragma unroll
    for (int j = 0; j < kParts * RK; j++) v[j] = t_from[threadIdx.x + j * kThreads];
    __syncthreads();  // the tile before is read
#pragma unroll
    for (int j = 0; j < kParts * RK; j++) operands[threadIdx.x + j * kThreads] = v[j];
    __syncthreads();
  }
  // The next strip's factors go out first, each block of rows when this strip's is done with: every load has a
  // whole strip's time, and none waits for one that is not needed yet (they return in order).
  for (int64_t i = 0; i < count; i++) {
    const int64_t n = place(i + 1);
    ready();
    hold();
    fetch_w(n);
    hold();
#pragma unroll
    for (int b = 0; b < MB; b++) {
      form(i * (64 * kWaves), b, true);
      hold();
      fetch_y(n, b);
      hold();
    }
  }
  // the columns past the whole strips, by the wave whose turn it is
  if (last > whole && (whole - first) % kWaves == wave) {
    const int64_t n = (whole - first - wave) * 64;
    const bool in = whole * 64 + 8 * chunk < a.N;
#pragma unroll
    for (int b = 0; b < MB; b++)
#pragma unroll
      for (int k = 0; k < 2; k++) y[b][k] = ADD && in ? *reinterpret_cast<const u32x4*>(yp[b][k] + n) : u32x4{};
#pragma unroll
    for (int j = 0; j < WL; j++)
      w[j] = w_off[j] >= 0 && whole * 64 + (64 * j + lane) / PER < a.N ? *reinterpret_cast<const u32x4*>(w0 + n * R + w_off[j]) : u32x4{};
    ready();
#pragma unroll
    for (int b = 0; b < MB; b++) form(n, b, in);
  }
}
// Y0, or zeros, to the columns c0 .. c1 - 1 of a tile's rows: 512 bytes of eight rows an access, eight accesses in flight
// (one at a time, a tenth of the rows of 4608 x 7680 without an adapter took up from 36 to 54 us).
template <bool ADD>
__device__ __forceinline__ void copy_piece(const UpArgs& a, const Tile& t, int64_t c0, int64_t c1) {
  constexpr int Q = kTile / 8;
  const int r = threadIdx.x >> 5;
  int64_t row[Q];
#pragma unroll
  for (int i = 0; i < Q; i++) row[i] = row_at(a.plan, t.pos + min(r + 8 * i, t.rows - 1));
  for (int64_t n = c0 + (threadIdx.x & 31) * 8; n < c1; n += 256) {
    u32x4 v[Q];
#pragma unroll
    for (int i = 0; i < Q; i++) v[i] = ADD ? *reinterpret_cast<const u32x4*>(a.y0 + row[i] * a.y0_row + n) : u32x4{};
    hold();
#pragma unroll
    for (int i = 0; i < Q; i++)
      if (r + 8 * i < t.rows) *reinterpret_cast<u32x4*>(a.y + row[i] * a.y_row + n) = v[i];
  }
}
template <int RK, bool ADD, bool JOIN>
__global__ __launch_bounds__(kThreads, up_per_cu(RK)) void up_kernel(const UpArgs a) {
  extern __shared__ __align__(16) uint8_t dynamic[];
  u32x4* operands = reinterpret_cast<u32x4*>(dynamic);  // [kParts][4][RK][64]
  uint8_t* lines = dynamic + 4 * kParts * RK * 1024;    // the waves' lines
  const bool zeros = JOIN && a.join.t != nullptr;  // T of rows without an adapter
  const int64_t used = used_tiles(a.plan), tiles = a.y0 == a.y && !zeros ? used : all_tiles(a.plan), len = a.stream.len(tiles);
  const int64_t down_len = JOIN ? a.join.down.len(used) : 0;
  int64_t at = blockIdx.x * len;
  const int64_t end = min(at + len, tiles * a.stream.steps);
  while (at < end) {
    const int64_t index = at / a.stream.steps, first = at - index * a.stream.steps, last = min(a.stream.steps, first + end - at);
    at += last - first;
    const Tile t = tile_of(a.plan, index);
    if (t.rows == 0) continue;
    if (t.adapter >= a.plan.A) {  // Y0 as it is
      if (zeros && first == 0) {
        __syncthreads();  // the tile before is read
        sum_rows<kThreads, kJoinHere>(a.join, t, index, 0, down_len, true, reinterpret_cast<float*>(lines));
      }
      if (a.y0 != a.y) copy_piece<ADD>(a, t, first * 64, min(last * 64, a.N));
      continue;
    }
    if (JOIN || t.rows <= 16) up_piece<RK, ADD, JOIN, 1>(a, t, index, first, last, down_len, operands, lines);
    else if constexpr (!JOIN) up_piece<RK, ADD, JOIN, 4>(a, t, index, first, last, down_len, operands, lines);
  }
}

// turn: in [A][rows][cols] to out [A][cols][rows], 64 x 64 elements a workgroup, for the adapters that
// have rows; and, in the same launch, a kept T's operands.
struct TurnArgs {
  Plan plan;
  const uint16_t* in[2];
  uint16_t* out[2];
  int64_t rows[2], cols[2];
  uint32_t tiles[2];  // workgroups of each, for an adapter
  uint32_t turns;     // all of them; the others take half a tile each of the kept T
  JoinArgs kept;
};
__global__ __launch_bounds__(kThreads) void turn_kernel(const TurnArgs a) {
  __shared__ __align__(16) float lds[32 * join_pitch(4)];
  if (blockIdx.x >= a.turns) {
    const uint32_t at = blockIdx.x - a.turns;
    join_half<kThreads>(a.kept, at >> 1, at & 1, lds);
    return;
  }
  uint16_t(*block)[72] = reinterpret_cast<uint16_t(*)[72]>(lds);
  static_assert(sizeof(lds) >= 64 * sizeof(*block), "a block's LDS");
  const uint32_t per = a.tiles[0] + a.tiles[1], place = blockIdx.x % per;
  const int64_t adapter = blockIdx.x / per;
  if (a.plan.start[adapter] >= a.plan.start[adapter + 1]) return;
  const int k = place >= a.tiles[0];
  const int64_t rows = a.rows[k], cols = a.cols[k], wide = (cols + 63) / 64;
  const int64_t at = place - (k ? a.tiles[0] : 0), r0 = at / wide * 64, c0 = at % wide * 64;
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

// grad: for C columns of Z (X for dL_B, dY for dL_A) and all R, the sum over an adapter's rows of Z[row][c]
// S[row][r], S = dT or alpha T in parts (join's cols).  Column tiles, each with all tiles of rows, are dealt out as
// Stream says; a workgroup goes through its runs of tiles of one adapter and one column tile.  A run
// that is all of the adapter's goes to the output, else to `part`: the first run of a workgroup, begun by the
// one before, to 2 w, the last to 2 w + 1; grad_join adds them.  Of eight waves, four take 32
// rows in turn and two take half the columns each: the two read the same lines of S, which L1 then holds once
// (16380 rows of 5120 and 5120, R = 64: 107 us with the waves along the rows alone, 90 with two across, 74 with S not read
// again; four across gain 1 us here and lose 3 in grad_join).  Z's rows go through the wave's own LDS, to be
// read with the rows along a lane (the transposing read), their 32-byte blocks swizzled so that the
// eight rows that half a wave reads lie in different banks.
struct GradArgs {
  Plan plan;
  const uint16_t* z[2];  // X, dY
  int64_t z_row[2], cols[2];
  uint32_t tiles[2];     // column tiles of each; 0 if its gradient is not wanted
  const u32x4* s[2];
  float* out[2];         // dL_B [A, R, K], dL_A [A, N, R]
  float* part;           // [2 workgroups][C R]: [R][C] of dL_B, [C][R] of dL_A
  int R, groups;
};
constexpr int kGradWaves = 8, kAcross = 2, kAlong = kGradWaves / kAcross, kGradThreads = 64 * kGradWaves;
// RB: R in 16s of a wave.  SPLIT: the waves across take half of R each (R > 64), not half of the columns.
template <int RB, bool SPLIT>
struct GradSize {
  static constexpr int CB = 8, C = 16 * CB, COLUMNS = SPLIT ? C : kAcross * C;  // a wave's, the workgroup's
  static constexpr int BLOCKS = CB * RB, ROUND = 8;
};
__device__ __forceinline__ int64_t grad_len(const GradArgs& a, int64_t tiles) {
  return max(((int64_t)(a.tiles[0] + a.tiles[1]) * tiles + a.groups - 1) / a.groups, (int64_t)2);
}

template <int RB, bool SPLIT, bool LA>
__device__ __forceinline__ void grad_run(const GradArgs& a, uint8_t* lds, int64_t c0, int64_t tile, int64_t from, int64_t rows,
                                         float* out, int64_t out_row) {
  typedef GradSize<RB, SPLIT> Size;
  constexpr int CB = Size::CB, C = Size::C, PER = C / 8, LOADS = 32 * PER / 64, BLOCKS = Size::BLOCKS, ROUND = Size::ROUND;
  constexpr int STEP = 32 * kAlong, ALL = SPLIT ? kAcross * RB : RB;  // blocks of r of S
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, q = lane >> 4;
  const int along = wave / kAcross, across = wave % kAcross;
  const int at0 = across * (SPLIT ? 16 * RB : C), r_end = a.R - (SPLIT ? at0 : 0);  // first r or column of the wave
  if (!SPLIT) c0 += at0;
  out += at0 * (LA != SPLIT ? out_row : 1);
  f32x4 acc[CB][RB];
#pragma unroll
  for (int c = 0; c < CB; c++)
#pragma unroll
    for (int b = 0; b < RB; b++) acc[c][b] = f32x4{};
  uint8_t* mine = lds + wave * 32 * C * 2;
  const int sub = lane / PER, p = lane % PER;
  const uint16_t* z = a.z[LA] + (c0 + 8 * p < a.cols[LA] ? c0 + 8 * p : 0);  // columns past the last: dropped
  const u32x4* s = a.s[LA] + (tile * kParts * 2 * ALL + (SPLIT ? across * RB : 0)) * 64 + lane;
  u32x4 zv[LOADS], sv[kParts][RB];
  auto index = [&](int64_t r0) {  // lane l: row r0 + l % 32 of the run, or its last
    return (int)row_at(a.plan, from + min(r0 + (lane & 31), rows - 1));
  };
  auto fetch_z = [&](int rows32) {
#pragma unroll
    for (int l = 0; l < LOADS; l++) {
      zv[l] = *reinterpret_cast<const u32x4*>(z + __shfl(rows32, l * (64 / PER) + sub, 64) * a.z_row[LA]);
    }
  };
  auto fetch_s = [&](int64_t r0) {
    const u32x4* t = s + (r0 / kTile * kParts * 2 + r0 / 32 % 2) * ALL * 64;
#pragma unroll
    for (int h = 0; h < kParts; h++)
#pragma unroll
      for (int b = 0; b < RB; b++) sv[h][b] = t[(h * 2 * ALL + b) * 64];
  };
  int64_t r0 = 32 * along;
  int ahead = index(r0);
  if (r0 < rows) {
    fetch_z(ahead);
    fetch_s(r0);
  }
  ahead = index(r0 + STEP);
  // A lane's place in the wave's rows as it writes and as it reads them, made anew each step: kept, the sixteen
  // addresses that come of them are more registers than there are, and what spills waits for the loads.
  const int jr = (lane & 15) >> 2;
  int put_at = (sub * C + ((p >> 1) ^ (sub & 3)) * 16 + (p & 1) * 8) * 2;
  int get_at = (8 * q + jr) * C * 2 + ((jr | (q & 1) << 2) << 5) + (lane & 3) * 8;
  for (; r0 < rows; r0 += STEP) {
    asm volatile("" : "+v"(put_at), "+v"(get_at));
    if (r0 + 32 > rows) {  // nothing of the last row again, which may hold what no zero of S takes away
#pragma unroll
      for (int l = 0; l < LOADS; l++)
        if (r0 + l * (64 / PER) + sub >= rows) zv[l] = u32x4{};
    }
    in_order();
#pragma unroll
    for (int l = 0; l < LOADS; l++) {
      *reinterpret_cast<u32x4*>(mine + ((put_at ^ (l >> 1 & 1) << 7) + l * (64 / PER) * C * 2)) = zv[l];
    }
    in_order();
    // the next rows' loads go out ahead of this step's products, those of S behind them, into the
    // registers that the products have read
    const bool more = r0 + STEP < rows;
    hold();
    if (more) fetch_z(ahead);
    ahead = index(r0 + 2 * STEP);
    hold();
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int c = 0; c < CB; c++) {
      const uint8_t* block = mine + (get_at ^ c << 5);
      const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
          (__attribute__((address_space(3))) bf16x4*)block));
      const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
          (__attribute__((address_space(3))) bf16x4*)(block + 4 * C * 2)));
      const u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
      for (int h = 0; h < kParts; h++)
#pragma unroll
        for (int b = 0; b < RB; b++) acc[c][b] = LA ? mfma16(sv[h][b], v, acc[c][b]) : mfma16(v, sv[h][b], acc[c][b]);
    }
    hold();
    if (more) fetch_s(r0 + STEP);
  }
  // the waves' sums, in one order; block (c, b): lane (r16, q) holds r = 16 b + r16 and columns 16 c +
  // 4q .. + 3 (dL_B), or column 16 c + r16 and r = 16 b + 4q .. + 3 (dL_A)
  f32x4(*sums)[ROUND][64] = reinterpret_cast<f32x4(*)[ROUND][64]>(lds);
#pragma unroll
  for (int round = 0; round < BLOCKS; round += ROUND) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROUND; k++) sums[wave][k][lane] = acc[(round + k) / RB][(round + k) % RB];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROUND / kAlong; k++) {
      const int at = k * kAlong + along, c = (round + at) / RB, b = (round + at) % RB;
      f32x4 v = sums[across][at][lane];
#pragma unroll
      for (int w = 1; w < kAlong; w++) v += sums[w * kAcross + across][at][lane];
      const int col = 16 * c + (LA ? r16 : 4 * q), r = 16 * b + (LA ? 4 * q : r16);
      if (c0 + col < a.cols[LA] && r < r_end) *reinterpret_cast<f32x4*>(out + (LA ? col * out_row + r : r * out_row + col)) = v;
    }
  }
  __syncthreads();  // before the next run's rows
}
template <int RB, bool SPLIT>
__global__ __launch_bounds__(kGradThreads, 1) void grad_kernel(const GradArgs a) {
  constexpr int C = GradSize<RB, SPLIT>::COLUMNS, LINES = 64 * GradSize<RB, SPLIT>::C, SUMS = 1024 * GradSize<RB, SPLIT>::ROUND;
  __shared__ __align__(16) uint8_t lds[kGradWaves * (LINES > SUMS ? LINES : SUMS)];
  const int64_t tiles = used_tiles(a.plan), len = grad_len(a, tiles);
  int64_t at = blockIdx.x * len;
  const int64_t end = min(at + len, (a.tiles[0] + a.tiles[1]) * tiles);
  while (at < end) {
    const int64_t column = at / tiles, tile = at - column * tiles;
    const int adapter = min(max(__builtin_amdgcn_readfirstlane(a.plan.tiles[tile].x), 0), a.plan.A - 1);
    const int64_t t0 = a.plan.tbase[adapter], t1 = a.plan.tbase[adapter + 1], p0 = a.plan.start[adapter], p1 = a.plan.start[adapter + 1];
    const int64_t stop = min(tile + end - at, min(max(t1, tile + 1), tiles));  // first tile past the run
    at += stop - tile;
    // positions of the run; a plan that was not made leaves none
    const int64_t from = p0 + (tile - t0) * kTile, rows = min(p1, p0 + (stop - t0) * kTile) - from;
    if (from < 0 || rows <= 0 || rows > (stop - tile) * kTile || from + rows > a.plan.M) continue;
    const bool la = column >= a.tiles[0], whole = tile <= t0 && stop >= t1;
    const int64_t c0 = (la ? column - a.tiles[0] : column) * C;
    float* part = a.part + (2 * (int64_t)blockIdx.x + (tile > t0 ? 0 : 1)) * C * a.R;
    if (la) grad_run<RB, SPLIT, true>(a, lds, c0, tile, from, rows, whole ? a.out[1] + (adapter * a.cols[1] + c0) * a.R : part, a.R);
    else grad_run<RB, SPLIT, false>(a, lds, c0, tile, from, rows, whole ? a.out[0] + adapter * a.R * a.cols[0] + c0 : part, whole ? a.cols[0] : C);
  }
}

// The runs of each adapter and column tile that has several, added in their order; zeros for an adapter without
// rows.
template <int C>
__global__ __launch_bounds__(kThreads) void grad_join_kernel(const GradArgs a) {
  const int64_t column = blockIdx.x, adapter = blockIdx.y;
  const bool la = column >= a.tiles[0];
  const int64_t c0 = (la ? column - a.tiles[0] : column) * C, cols = a.cols[la];
  const int64_t tiles = used_tiles(a.plan), len = grad_len(a, tiles), t0 = a.plan.tbase[adapter], t1 = a.plan.tbase[adapter + 1];
  int64_t first = 0, last = -1;
  if (t0 >= 0 && t1 > t0 && t1 <= tiles) {
    first = (column * tiles + t0) / len;
    last = (column * tiles + t1 - 1) / len;
    if (first == last || last >= a.groups) return;
  }
  for (int id = blockIdx.z * kThreads + threadIdx.x; id < C * a.R / 4; id += gridDim.z * kThreads) {
    // four of a row of the run's sums
    const int wide = (la ? a.R : C) / 4, row = id / wide, x = id % wide * 4, col = la ? row : x;
    if (c0 + col >= cols) continue;
    f32x4 v{};
#pragma unroll 4
    for (int64_t w = first; w <= last; w++)
      v += *reinterpret_cast<const f32x4*>(a.part + (2 * w + (w == first)) * C * a.R + (int64_t)id * 4);
    float* out = a.out[la] + adapter * a.R * cols + (la ? (c0 + row) * a.R + x : row * cols + c0 + x);
    *reinterpret_cast<f32x4*>(out) = v;
  }
}

// ---------------------------------------------------------------- launches

int rank_blocks(int64_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : 8; }
int rank_steps(int64_t R) { return (int)((R + 31) / 32); }
size_t cols_bytes(int64_t M, int64_t A, int64_t R) { return (size_t)max_tiles(M, A) * kParts * 2 * rank_blocks(R) * 1024; }

// The workgroups that the chip's 256 CUs hold at once, by their registers and LDS.
constexpr int kCus = 256;
Stream stream_of(int64_t most, int64_t steps, int per_cu, int least) {
  return Stream{steps, (int)std::min<int64_t>(per_cu * kCus, (most * steps + least - 1) / least), least};
}
Stream down_stream(int64_t most, int64_t C, int64_t R) {
  return stream_of(most, (C + 63) / 64, down_per_cu(rank_blocks(R)), kWaves);
}
size_t align(size_t n) { return (n + 255) & ~(size_t)255; }
size_t part_bytes(int64_t M, int64_t A, int64_t R, int64_t C) {
  const int64_t most = max_tiles(M, A);
  return align((size_t)(most + down_stream(most, C, R).groups) * kTile * R * 4);
}

size_t rows_bytes(int64_t M, int64_t A, int64_t R) { return (size_t)max_tiles(M, A) * 4 * kParts * rank_steps(R) * 1024; }

JoinArgs join_of(const Plan& plan, int64_t R, const float* alpha) {
  JoinArgs a{};
  a.plan = plan;
  a.alpha = alpha;
  a.R = (int)R;
  a.RB = rank_blocks(R);
  a.RK = rank_steps(R);
  return a;
}
// One block of rows at the most: up sums T itself, each workgroup what it needs, a launch less (5120 -> 5120, R = 128: one
// row 15.5 us and 14.4 so, 8 rows of 8 adapters 17.0 and 15.4, 64 rows of one 26 and, with T in two parts, 58).
bool join_here(int64_t M) { return M <= kJoinHere; }
void join(const JoinArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)(2 * a.plan.most)), dim3(kJoinThreads), 0, stream, a);
}

void down(const Plan& plan, const void* x, int64_t x_row, const void* w, int64_t C, int64_t R, float* part, hipStream_t stream) {
  const DownArgs a{plan, (const uint16_t*)x, (const uint16_t*)w, x_row, C, (int)R, down_stream(plan.most, C, R), part};
  const dim3 grid((unsigned)a.stream.groups);
  switch (rank_blocks(R)) {
    case 1: hipLaunchKernelGGL(down_kernel<1>, grid, dim3(kThreads), 0, stream, a); break;
    case 2: hipLaunchKernelGGL(down_kernel<2>, grid, dim3(kThreads), 0, stream, a); break;
    case 4: hipLaunchKernelGGL(down_kernel<4>, grid, dim3(kThreads), 0, stream, a); break;
    default: hipLaunchKernelGGL(down_kernel<8>, grid, dim3(kThreads), 0, stream, a); break;
  }
}

// t: join's rows, or null: summed as `j` says.
void up(const Plan& plan, const void* w, const void* y0, int64_t y0_row, void* y, int64_t y_row, int64_t N, int64_t R, const void* t,
        const JoinArgs& j, hipStream_t stream) {
  const int rk = rank_steps(R);
  const UpArgs a{plan, (const uint16_t*)w, (const uint16_t*)y0, (uint16_t*)y, y0_row, y_row, N, (int)R,
                 stream_of(plan.most, (N + 63) / 64, up_per_cu(rk), kWaves), (const u32x4*)t, j};
  const dim3 grid((unsigned)a.stream.groups);
  auto go = [&](auto k) {
    constexpr int RK = decltype(k)::value;
    constexpr size_t lds = 4 * kParts * RK * 1024 + kWaves * up_lines(RK);
    static_assert(kWaves * up_lines(RK) >= kJoinHere * join_pitch(RK) * 4, "a tile's T in the lines' place");
    auto run = [&](auto add, auto here) {
      hipLaunchKernelGGL((up_kernel<RK, decltype(add)::value, decltype(here)::value>), grid, dim3(kThreads), lds, stream, a);
    };
    if (y0 != nullptr) t == nullptr ? run(std::true_type(), std::true_type()) : run(std::true_type(), std::false_type());
    else t == nullptr ? run(std::false_type(), std::true_type()) : run(std::false_type(), std::false_type());
  };
  switch (rk) {
    case 1: go(std::integral_constant<int, 1>()); break;
    case 2: go(std::integral_constant<int, 2>()); break;
    case 3: go(std::integral_constant<int, 3>()); break;
    default: go(std::integral_constant<int, 4>()); break;
  }
}

constexpr int kGradGroups = kCus;
int64_t grad_columns(int64_t R) { return rank_blocks(R) == 8 ? 128 : 256; }

}  // namespace lora

size_t adapters_plan_bytes(int64_t M, int64_t A) {
  using namespace lora;
  size_t tiles, order;
  return plan_words(M, A, &tiles, &order) * 4;
}

hipError_t launch_adapters_plan(const int32_t* ids, int64_t M, int64_t A, void* plan, hipStream_t stream) {
  using namespace lora;
  size_t tiles, order;
  plan_words(M, A, &tiles, &order);
  int32_t* w = (int32_t*)plan;
  hipLaunchKernelGGL(plan_kernel, dim3((unsigned)(A + 1)), dim3(kPlanThreads), (size_t)(2 * A + 3) * 4, stream, ids, M, (int)A, w,
                     (int4*)(w + tiles), w + order);
  return hipGetLastError();
}

// Workspace: down's pieces | up's operands.
size_t adapters_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A) {
  using namespace lora;
  return part_bytes(M, A, R, K) + align(rows_bytes(M, A, R));
}

hipError_t launch_adapters(const AdapterCall& c, const void* y0, int64_t y0_row, void* y, int64_t y_row, float* t, void* ws,
                           hipStream_t stream) {
  using namespace lora;
  const Plan plan = plan_of(c.plan, c.M, c.A);
  float* part = (float*)ws;
  down(plan, c.x, c.x_row, c.LB, c.K, c.R, part, stream);
  JoinArgs j = join_of(plan, c.R, c.alpha);
  j.part = part;
  j.down = down_stream(plan.most, c.K, c.R);
  j.t = t;
  j.rows = (u32x4*)((uint8_t*)ws + part_bytes(c.M, c.A, c.R, c.K));
  const bool here = join_here(c.M);
  if (here) j.rows = nullptr;
  else join(j, stream);
  up(plan, c.LA, y0, y0_row, y, y_row, c.N, c.R, j.rows, j, stream);
  return hipGetLastError();
}

// Workspace of the gradient: L_A^T, L_B^T | down's pieces | dT as up's operand | dT and T as grad's | grad's runs.
size_t adapters_back_workspace(int64_t M, int64_t N, int64_t K, int64_t R, int64_t A) {
  using namespace lora;
  return align((size_t)A * N * R * 2) + align((size_t)A * K * R * 2) + part_bytes(M, A, R, N) + align(rows_bytes(M, A, R)) + 2 * align(cols_bytes(M, A, R)) +
         align((size_t)2 * kGradGroups * grad_columns(R) * R * 4);
}

hipError_t launch_adapters_back(const AdapterCall& c, const float* t, const void* dy, int64_t dy_row, const void* dx0,
                                int64_t dx0_row, void* dx, int64_t dx_row, float* dla, float* dlb, void* ws,
                                hipStream_t stream) {
  using namespace lora;
  const Plan plan = plan_of(c.plan, c.M, c.A);
  uint8_t* at = (uint8_t*)ws;
  auto take = [&](size_t bytes) {
    void* p = at;
    at += align(bytes);
    return p;
  };
  void* lat = take((size_t)c.A * c.N * c.R * 2);
  void* lbt = take((size_t)c.A * c.K * c.R * 2);
  float* part = (float*)take(part_bytes(c.M, c.A, c.R, c.N));
  void* drows = take(rows_bytes(c.M, c.A, c.R));
  void* dcols = take(cols_bytes(c.M, c.A, c.R));
  void* tcols = take(cols_bytes(c.M, c.A, c.R));
  float* runs = (float*)at;
  const bool dt = dx != nullptr || dlb != nullptr;
  {
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
    a.tiles[0] = dt ? (uint32_t)(((c.N + 63) / 64) * ((c.R + 63) / 64)) : 0;
    a.tiles[1] = dx != nullptr ? (uint32_t)(((c.K + 63) / 64) * ((c.R + 63) / 64)) : 0;
    a.turns = (uint32_t)(c.A * (a.tiles[0] + a.tiles[1]));
    a.kept = join_of(plan, c.R, c.alpha);
    a.kept.kept = t;
    a.kept.cols = (u32x4*)tcols;
    hipLaunchKernelGGL(turn_kernel, dim3(a.turns + (dla != nullptr ? 2 * (unsigned)plan.most : 0)), dim3(kThreads), 0, stream, a);
  }
  if (dt) {
    down(plan, dy, dy_row, lat, c.N, c.R, part, stream);
    JoinArgs j = join_of(plan, c.R, c.alpha);
    j.part = part;
    j.down = down_stream(plan.most, c.N, c.R);
    j.rows = dx != nullptr ? (u32x4*)drows : nullptr;
    j.cols = dlb != nullptr ? (u32x4*)dcols : nullptr;
    join(j, stream);
    if (dx != nullptr) up(plan, lbt, dx0, dx0_row, dx, dx_row, c.K, c.R, drows, j, stream);
  }
  if (dla != nullptr || dlb != nullptr) {
    const int64_t C = grad_columns(c.R);
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
    a.part = runs;
    a.R = (int)c.R;
    a.groups = kGradGroups;
    const dim3 grid((unsigned)kGradGroups);
    const int64_t joins = (int64_t)(a.tiles[0] + a.tiles[1]) * c.A, most = C * c.R / 4 / kThreads;
    const dim3 columns(a.tiles[0] + a.tiles[1], (unsigned)c.A, (unsigned)std::max<int64_t>(1, std::min(most, 4 * kCus / joins)));
    switch (rank_blocks(c.R)) {
      case 1: hipLaunchKernelGGL((grad_kernel<1, false>), grid, dim3(kGradThreads), 0, stream, a); break;
      case 2: hipLaunchKernelGGL((grad_kernel<2, false>), grid, dim3(kGradThreads), 0, stream, a); break;
      case 4: hipLaunchKernelGGL((grad_kernel<4, false>), grid, dim3(kGradThreads), 0, stream, a); break;
      default: hipLaunchKernelGGL((grad_kernel<4, true>), grid, dim3(kGradThreads), 0, stream, a); break;
    }
    if (C == 128) hipLaunchKernelGGL(grad_join_kernel<128>, columns, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL(grad_join_kernel<256>, columns, dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace rtl
