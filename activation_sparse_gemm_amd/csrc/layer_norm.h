// layer_norm.h -- layer norm of every row with the weights of the layer and the scale and shift of
// the row's request, and its gradient with the sums over rows that the weights', the scales' and
// the shifts' gradients are.
//
//   n = (x - mean) r,  r = 1 / sqrt(mean((x - mean)^2) + eps)
//   y = (n w + b) (1 + scale_g) + shift_g          g: the row's group, a run of rows
//   back, from the kept mean and r, with c = dy (1 + scale_g) and t = c w:
//     dx = r (t - mean(t) - n mean(t n))
//     S0_g = sum of dy, S1_g = sum of dy n over the group's rows, and from these alone
//     dshift_g = S0_g,  dscale_g = w S1_g + b S0_g,
//     dw = sum_g (1 + scale_g) S1_g,  db = sum_g (1 + scale_g) S0_g
//
// Bound: memory (each element read once and written once; the gradient reads two and writes one).  32760 x 5120 in
// bf16: forward 122 us, 5.5 TB/s; the gradient's pass 210, 5.0 with its chunks' sums, and 26 to join them.
// A row is held in the registers of W waves, so that it is read once for mean, squares and result.
// Groups are ascending offsets in device memory: a row finds its group there, and rows outside
// every group are left as they were or become zeros.  Whatever the offsets hold, no access leaves the arrays.
#pragma once
#include <algorithm>
#include <type_traits>

#include "rtl_device.h"
#include "rtl_launch.h"

namespace rtl {

namespace norm {

// V elements of a row: 16 bytes, or one element where rows are not 16-byte aligned.
template <bool BF16, int V>
struct Piece {
  static_assert(V == 1 || V == (BF16 ? 8 : 4), "16 bytes, or one element");
  typedef typename std::conditional<V == 1, uint32_t, u32x4>::type Raw;
  __device__ __forceinline__ static Raw load(const void* p, int64_t at) {
    if constexpr (V > 1) {
      return *reinterpret_cast<const u32x4*>((const uint8_t*)p + at * (BF16 ? 2 : 4));
    } else if constexpr (BF16) {
      return (uint32_t)((const uint16_t*)p)[at] << 16;
    } else {
      return ((const uint32_t*)p)[at];
    }
  }
  __device__ __forceinline__ static void unpack(const Raw& r, float (&v)[V]) {
    if constexpr (V == 1) {
      v[0] = __uint_as_float(r);
    } else if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[2 * i] = bf16lo(r[i]);
        v[2 * i + 1] = bf16hi(r[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) v[i] = __uint_as_float(r[i]);
    }
  }
  // Plain stores: hinted to leave the caches first they make the norm faster (32760 x 2560: 65 -> 55 us) and
  // the product that reads its result slower (norm and a copy of 32760 x 5120: 241 -> 252 us).
  __device__ __forceinline__ static void store(void* p, int64_t at, const float (&v)[V]) {
    if constexpr (V == 1) {
      if constexpr (BF16) ((__bf16*)p)[at] = (__bf16)v[0];
      else ((float*)p)[at] = v[0];
    } else {
      u32x4 w;
      if constexpr (BF16) {
        typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
      } else {
#pragma unroll
        for (int i = 0; i < 4; i++) w[i] = __float_as_uint(v[i]);
      }
      *reinterpret_cast<u32x4*>((uint8_t*)p + at * (BF16 ? 2 : 4)) = w;
    }
  }
};

// Sum over the wave's 64 lanes, the same in each: row exchanges as operands of the sums for lanes
// 1, 2, 4 and 8 apart, shuffles for 16 and 32.
template <int CTRL>
__device__ __forceinline__ float add_lanes(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lanes_sum(float v) {
  v = add_lanes<0xB1>(v);   // quad_perm 1,0,3,2
  v = add_lanes<0x4E>(v);   // quad_perm 2,3,0,1
  v = add_lanes<0x141>(v);  // row_half_mirror
  v = add_lanes<0x140>(v);  // row_mirror
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Index of the row's group: the last offset at or below `row` of groups[0 .. G], -1 or G where none
// holds the row.  64 offsets at a time (one for the whole wave to read where G < 64).
__device__ __forceinline__ int find_group(const int32_t* groups, int G, int64_t row, int lane) {
  if (groups == nullptr) return 0;
  int lo = 0, n = G + 1;  // the count of offsets at or below the row lies in [lo, lo + n]
  while (n > 64) {
    const int step = (n + 63) / 64, i = lo + lane * step;
    const int c = __popcll(__ballot(i < lo + n && groups[min(i, G)] <= row));
    if (c == 0) return lo - 1;
    const int end = lo + n;
    lo += (c - 1) * step;
    n = min(step, end - lo);
  }
  const int i = lo + lane;
  return lo + __popcll(__ballot(lane < n && groups[min(i, G)] <= row)) - 1;
}

struct NormArgs {
  int64_t M, x_row, y_row, d_row, scale_row, shift_row;  // strides in elements
  int D, G;
  float eps, inv_d;
  const void *x, *dy, *w, *b, *scale, *shift;
  void* y;                // dx in the gradient
  const int32_t* groups;  // [G + 1], null: one group of all rows
  float* stats;           // [M, 2]
  float* part;            // gradient: [slots][2][D]
  int rows;               // gradient: rows of a chunk
  bool clear;             // zeros to y's rows of no group
};

constexpr int kNormThreads = 256;
// Workgroups come in rows of 2^20: a launch takes fewer than 2^32 threads in one dimension.
dim3 norm_grid(int64_t blocks) {
  const int64_t row = std::min<int64_t>(blocks, 1 << 20);
  return dim3((unsigned)row, (unsigned)((blocks + row - 1) / row));
}
__device__ __forceinline__ int64_t norm_block() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Zeros to a row of y, a lane its pieces.
template <bool BF16, int V, int W, int J>
__device__ __forceinline__ void clear_row(const NormArgs& a, int64_t row, int at0) {
  const float zeros[V] = {};
#pragma unroll
  for (int j = 0; j < J; j++) {
    const int at = at0 + j * W * 64 * V;
    if (at < a.D) Piece<BF16, V>::store(a.y, row * a.y_row + at, zeros);
  }
}

// Forward: W waves a row, J pieces a lane.
template <bool BF16, int V, int W, int J>
__global__ __launch_bounds__(W == 1 ? kNormThreads : W * 64) void norm_kernel(const NormArgs a) {
  typedef Piece<BF16, V> P;
  __shared__ float sums[W > 1 ? 3 : 1][W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = W > 1 ? wave : 0;
  const int64_t row = W > 1 ? norm_block() : norm_block() * (kNormThreads / 64) + wave;
  if (row >= a.M) return;  // whole waves, or whole workgroups
  const int at0 = (part * 64 + lane) * V;
  typename P::Raw raw[J];
#pragma unroll
  for (int j = 0; j < J; j++) {
    raw[j] = typename P::Raw{};
    const int at = at0 + j * W * 64 * V;
    if (at < a.D) raw[j] = P::load(a.x, row * a.x_row + at);
  }
  const int g = find_group(a.groups, a.G, row, lane);
  if (g < 0 || g >= max(a.G, 1)) {  // the same for all waves of the row
    if (a.clear) clear_row<BF16, V, W, J>(a, row, at0);
    return;
  }

  auto across = [&](float v, int k) {
    v = lanes_sum(v);
    if constexpr (W > 1) {
      if (lane == 0) sums[k][part] = v;
      __syncthreads();
      v = 0.f;
#pragma unroll
      for (int i = 0; i < W; i++) v += sums[k][i];
    }
    return v;
  };
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < J; j++) {
    float v[V];
    P::unpack(raw[j], v);
#pragma unroll
    for (int i = 0; i < V; i++) s += v[i];
  }
  // The squares of the distances from this mean, and the distances' own sum, which is what the
  // mean's rounding left: a row far from 0 keeps its digits.
  const float mean0 = across(s, 0) * a.inv_d;
  float q = 0.f, e = 0.f;
#pragma unroll
  for (int j = 0; j < J; j++) {
    float v[V];
    P::unpack(raw[j], v);
#pragma unroll
    for (int i = 0; i < V; i++) {
      const float d = at0 + j * W * 64 * V < a.D ? v[i] - mean0 : 0.f;
      e += d;
      q = fmaf(d, d, q);
    }
  }
  if constexpr (W > 1) {
    e = lanes_sum(e);
    q = lanes_sum(q);
    if (lane == 0) {
      sums[1][part] = e;
      sums[2][part] = q;
    }
    __syncthreads();
    e = q = 0.f;
#pragma unroll
    for (int i = 0; i < W; i++) {
      e += sums[1][i];
      q += sums[2][i];
    }
  } else {
    e = lanes_sum(e);
    q = lanes_sum(q);
  }
  e *= a.inv_d;
  const float var = fmaf(q, a.inv_d, -e * e);
  const float r = 1.f / sqrtf((var < 0.f ? 0.f : var) + a.eps);  // a NaN stays one
  if (a.stats != nullptr && lane == 0 && part == 0) {
    a.stats[2 * row] = mean0 + e;
    a.stats[2 * row + 1] = r;
  }
#pragma unroll
  for (int j = 0; j < J; j++) {
    const int at = at0 + j * W * 64 * V;
    if (at >= a.D) continue;
    float v[V], u[V];
    P::unpack(raw[j], v);
#pragma unroll
    for (int i = 0; i < V; i++) v[i] = ((v[i] - mean0) - e) * r;
    if (a.w != nullptr) {
      P::unpack(P::load(a.w, at), u);
#pragma unroll
      for (int i = 0; i < V; i++) v[i] *= u[i];
    }
    if (a.b != nullptr) {
      P::unpack(P::load(a.b, at), u);
#pragma unroll
      for (int i = 0; i < V; i++) v[i] += u[i];
    }
    if (a.scale != nullptr) {
      float h[V];
      P::unpack(P::load(a.scale, g * a.scale_row + at), u);
      P::unpack(P::load(a.shift, g * a.shift_row + at), h);
#pragma unroll
      for (int i = 0; i < V; i++) v[i] = fmaf(v[i], 1.f + u[i], h[i]);
    }
    P::store(a.y, row * a.y_row + at, v);
  }
}

// Gradient: W waves (W == 1: each wave for itself) walk over a chunk of consecutive rows, the next
// row's loads in flight while one is formed, and hold the sums of their columns; at the end of a
// group in the chunk, and of the chunk, the sums go to slot chunk + group (rows in order raise one or the
// other, so each pair has a slot of its own).  A sum in fp32 runs over at most kNormChunk rows; what follows is
// in double.  Longer chunks halve the sums' bytes and end unevenly: 32760 x 5120 in chunks of 32 rows 209 + 21 us
// (sums), of 64 301 + 11, of 16 216 + 39.
constexpr int kNormChunk = 32;
template <bool BF16, int V, int W, int J>
__global__ __launch_bounds__(W == 1 ? kNormThreads : W * 64) void norm_back_kernel(const NormArgs a) {
  typedef Piece<BF16, V> P;
  __shared__ float sums[2][W][2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), part = W > 1 ? wave : 0;
  const int64_t chunk = W > 1 ? norm_block() : norm_block() * (kNormThreads / 64) + wave;
  const int64_t first = chunk * a.rows, last = min(first + a.rows, a.M);
  if (first >= a.M) return;
  const int at0 = (part * 64 + lane) * V;
  float s0[J][V], s1[J][V], up[J][V];  // up: w (1 + scale)
#pragma unroll
  for (int j = 0; j < J; j++)
#pragma unroll
    for (int i = 0; i < V; i++) s0[j][i] = s1[j][i] = up[j][i] = 0.f;
  auto flush = [&](int g) {
    float* to = a.part + (chunk + g) * 2 * a.D;
#pragma unroll
    for (int j = 0; j < J; j++) {
      const int at = at0 + j * W * 64 * V;
      if (at < a.D) {
        if constexpr (V == 1) {
          to[at] = s0[j][0];
          to[a.D + at] = s1[j][0];
        } else {
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            *reinterpret_cast<f32x4*>(to + at + i) = f32x4{s0[j][i], s0[j][i + 1], s0[j][i + 2], s0[j][i + 3]};
            *reinterpret_cast<f32x4*>(to + a.D + at + i) = f32x4{s1[j][i], s1[j][i + 1], s1[j][i + 2], s1[j][i + 3]};
          }
        }
      }
#pragma unroll
      for (int i = 0; i < V; i++) s0[j][i] = s1[j][i] = 0.f;
    }
  };
  struct Row {
    typename P::Raw x[J], d[J];
    float mean, r;
  };
  auto fetch = [&](int64_t row, Row& it) {
    if (row >= last) return;
    it.mean = a.stats[2 * row];
    it.r = a.stats[2 * row + 1];
#pragma unroll
    for (int j = 0; j < J; j++) {
      const int at = at0 + j * W * 64 * V;
      it.x[j] = it.d[j] = typename P::Raw{};
      if (at < a.D) {
        it.x[j] = P::load(a.x, row * a.x_row + at);
        it.d[j] = P::load(a.dy, row * a.d_row + at);
      }
    }
  };
  int g = 0, open = -1;                             // the row's group; the one whose sums are held
  int64_t end = a.groups != nullptr ? -1 : a.M;  // first row past group g
  int turn = 0;
  auto form = [&](int64_t row, const Row& it) {
    if (row >= end) {
      g = find_group(a.groups, a.G, row, lane);
      end = g < a.G ? a.groups[g + 1] : a.M;
    }
    if (g < 0 || g >= max(a.G, 1)) {
      if (a.clear) clear_row<BF16, V, W, J>(a, row, at0);
      return;
    }
    if (g != open) {
      if (open >= 0 && a.part != nullptr) flush(open);
      open = g;
#pragma unroll
      for (int j = 0; j < J; j++) {
        const int at = at0 + j * W * 64 * V;
        float u[V];
#pragma unroll
        for (int i = 0; i < V; i++) up[j][i] = 1.f;
        if (at >= a.D) continue;
        if (a.w != nullptr) P::unpack(P::load(a.w, at), up[j]);
        if (a.scale != nullptr) {
          P::unpack(P::load(a.scale, g * a.scale_row + at), u);
#pragma unroll
          for (int i = 0; i < V; i++) up[j][i] *= 1.f + u[i];
        }
      }
    }
    float c0 = 0.f, c1 = 0.f;
#pragma unroll
    for (int j = 0; j < J; j++) {
      const bool in = at0 + j * W * 64 * V < a.D;
      float v[V], d[V];
      P::unpack(it.x[j], v);
      P::unpack(it.d[j], d);
#pragma unroll
      for (int i = 0; i < V; i++) {
        const float n = in ? (v[i] - it.mean) * it.r : 0.f, t = d[i] * up[j][i];
        s0[j][i] += d[i];
        s1[j][i] = fmaf(d[i], n, s1[j][i]);
        c0 += t;
        c1 = fmaf(t, n, c1);
      }
    }
    c0 = lanes_sum(c0);
    c1 = lanes_sum(c1);
    if constexpr (W > 1) {
      if (lane == 0) {
        sums[turn][part][0] = c0;
        sums[turn][part][1] = c1;
      }
      __syncthreads();
      c0 = c1 = 0.f;
#pragma unroll
      for (int i = 0; i < W; i++) {
        c0 += sums[turn][i][0];
        c1 += sums[turn][i][1];
      }
      turn ^= 1;  // two sets: the next row's are written while a wave may still read these
    }
    c0 *= a.inv_d;
    c1 *= a.inv_d;
#pragma unroll
    for (int j = 0; j < J; j++) {
      const int at = at0 + j * W * 64 * V;
      if (at >= a.D) continue;
      float v[V], d[V];
      P::unpack(it.x[j], v);
      P::unpack(it.d[j], d);
#pragma unroll
      for (int i = 0; i < V; i++) {
        const float n = (v[i] - it.mean) * it.r;
        v[i] = it.r * fmaf(-n, c1, fmaf(d[i], up[j][i], -c0));
      }
      P::store(a.y, row * a.y_row + at, v);
    }
  };
  Row one, two;
  fetch(first, one);
  for (int64_t row = first; row < last; row += 2) {
    fetch(row + 1, two);
    form(row, one);
    if (row + 1 >= last) break;
    fetch(row + 2, one);
    form(row + 1, two);
  }
  if (open >= 0 && a.part != nullptr) flush(open);
}

struct SumArgs {
  int64_t M, scale_row;
  int D, G, rows;
  const float* part;
  const int32_t* groups;
  const void *w, *b, *scale;
  float *dw, *db, *dscale, *dshift;  // null: not wanted
  double* group;                     // [G][2][D]: the groups' sums, for dw and db of several groups
};

// Rows [lo, hi) of group g, within M; none where hi <= lo.
__device__ __forceinline__ void rows_of_group(const SumArgs& a, int64_t g, int64_t& lo, int64_t& hi) {
  lo = 0;
  hi = a.M;
  if (a.groups != nullptr) {
    lo = max((int64_t)a.groups[g], (int64_t)0);
    hi = min((int64_t)a.groups[g + 1], a.M);
  }
}

__device__ __forceinline__ float value_at(bool bf16, const void* p, int64_t at) {
  return bf16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[at] << 16) : ((const float*)p)[at];
}

// Column sums of a workgroup's 32 columns: lane c of 32 / CV holds CV of them, row lane l of LR every
// LR-th of the terms; the row lanes' sums are added in one order.  For 32 threads, column `col` of each.
template <int CV, int THREADS>
struct NormColumns {
  static constexpr int LC = 32 / CV, LR = THREADS / LC, K = THREADS / 32;
  double s[2][CV];
  __device__ __forceinline__ static int lane() { return threadIdx.x % LC * CV; }
  __device__ __forceinline__ static int row() { return threadIdx.x / LC; }
  __device__ __forceinline__ NormColumns() {
#pragma unroll
    for (int i = 0; i < CV; i++) s[0][i] = s[1][i] = 0.0;
  }
  // Both sums of column threadIdx.x in the first 32 threads.
  __device__ __forceinline__ void join(double& s0, double& s1) {
    __shared__ double red[2][LR][33];
#pragma unroll
    for (int i = 0; i < CV; i++) {
      red[0][row()][lane() + i] = s[0][i];
      red[1][row()][lane() + i] = s[1][i];
    }
    __syncthreads();
    const int c = threadIdx.x % 32, k = threadIdx.x / 32;
    auto add = [&](int from, int step, int n) {
      s0 = s1 = 0.0;
#pragma unroll
      for (int r = 0; r < n; r++) {
        s0 += red[0][from + r * step][c];
        s1 += red[1][from + r * step][c];
      }
    };
    if constexpr (LR > K) {  // every K-th, then the K sums
      add(k, K, LR / K);
      red[0][k][c] = s0;
      red[1][k][c] = s1;
      __syncthreads();
    }
    if (k == 0) add(0, 1, K);
  }
};

// The sums of a group over its chunks, 32 columns a workgroup, in double.  Groups come in rows of kNormSumGroups (norm_grid's
// reason).
constexpr int64_t kNormSumGroups = 1 << 20;
template <bool BF16, int CV, int THREADS>
__global__ __launch_bounds__(THREADS) void norm_sum_kernel(const SumArgs a) {
  typedef NormColumns<CV, THREADS> Columns;
  Columns t;
  const int64_t g = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  if (g >= a.G) return;
  const int col0 = blockIdx.y * 32, at = col0 + t.lane();
  int64_t lo, hi;
  rows_of_group(a, g, lo, hi);
  if (hi > lo && at < a.D) {
    const int64_t from = lo / a.rows + g, to = (hi - 1) / a.rows + g;
#pragma unroll 4
    for (int64_t s = from + t.row(); s <= to; s += Columns::LR) {
      const float* p = a.part + s * 2 * a.D + at;
      if constexpr (CV == 1) {
        t.s[0][0] += (double)p[0];
        t.s[1][0] += (double)p[a.D];
      } else {
        const f32x4 v0 = *reinterpret_cast<const f32x4*>(p), v1 = *reinterpret_cast<const f32x4*>(p + a.D);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          t.s[0][i] += (double)v0[i];
          t.s[1][i] += (double)v1[i];
        }
      }
    }
  }
  double s0, s1;
  t.join(s0, s1);
  const int col = col0 + threadIdx.x;
  if (threadIdx.x >= 32 || col >= a.D) return;
  if (a.dscale != nullptr) {
    const double w = a.w != nullptr ? (double)value_at(BF16, a.w, col) : 1.0, b = a.b != nullptr ? (double)value_at(BF16, a.b, col) : 0.0;
    a.dscale[g * a.D + col] = hi > lo ? (float)(w * s1 + b * s0) : 0.f;  // 0 too where w or b is infinite
  }
  if (a.dshift != nullptr) a.dshift[g * a.D + col] = (float)s0;
  if (a.group != nullptr) {
    a.group[2 * g * a.D + col] = s0;
    a.group[(2 * g + 1) * a.D + col] = s1;
  } else {
    if (a.dw != nullptr) a.dw[col] = (float)s1;
    if (a.db != nullptr) a.db[col] = (float)s0;
  }
}

// dw and db over the groups: sum_g (1 + scale_g) S_g.  An empty group's scale, which may hold anything, does
// not enter.
template <bool BF16>
__global__ __launch_bounds__(256) void norm_weight_kernel(const SumArgs a) {
  typedef NormColumns<1, 256> Columns;
  Columns t;
  const int col0 = blockIdx.x * 32, at = col0 + t.lane();
  if (at < a.D) {
#pragma unroll 4
    for (int64_t g = t.row(); g < a.G; g += Columns::LR) {
      int64_t lo, hi;
      rows_of_group(a, g, lo, hi);
      const double k = a.scale != nullptr && hi > lo ? 1.0 + (double)value_at(BF16, a.scale, g * a.scale_row + at) : 1.0;
      t.s[0][0] += k * a.group[2 * g * a.D + at];
      t.s[1][0] += k * a.group[(2 * g + 1) * a.D + at];
    }
  }
  double s0, s1;
  t.join(s0, s1);
  const int col = col0 + threadIdx.x;
  if (threadIdx.x >= 32 || col >= a.D) return;
  if (a.dw != nullptr) a.dw[col] = (float)s1;
  if (a.db != nullptr) a.db[col] = (float)s0;
}

template <int N>
using Int = std::integral_constant<int, N>;

// Calls f(Int<J>) for the least of Js that is at least `need`; false if none is.
template <int... Js, typename F>
bool pick(int64_t need, F f) {
  bool done = false;
  auto one = [&](auto j) {
    if (!done && need <= decltype(j)::value) {
      done = true;
      f(j);
    }
  };
  (one(Int<Js>()), ...);
  return done;
}

// Whether rows can be taken in 16-byte pieces.
bool norm_wide(const NormCall& c) {
  const int64_t es = c.dt == kDtBF16 ? 2 : 4;
  uint64_t bits = (uint64_t)(c.D * es);
  for (const RowsView& v : {c.x, c.y, c.dy, c.scale, c.shift})
    if (v.p != nullptr) bits |= (uint64_t)(uintptr_t)v.p | (uint64_t)(v.row * es);
  for (const void* p : {c.w, c.b}) bits |= (uint64_t)(uintptr_t)p;
  return bits % 16 == 0;
}

NormArgs norm_args(const NormCall& c) {
  NormArgs a{};
  a.M = c.M;
  a.D = (int)c.D;
  a.G = (int)c.G;
  a.x = c.x.p;
  a.x_row = c.x.row;
  a.y = const_cast<void*>(c.y.p);
  a.y_row = c.y.row;
  a.dy = c.dy.p;
  a.d_row = c.dy.row;
  a.scale = c.scale.p;
  a.scale_row = c.scale.row;
  a.shift = c.shift.p;
  a.shift_row = c.shift.row;
  a.w = c.w;
  a.b = c.b;
  a.eps = c.eps;
  a.inv_d = 1.f / (float)c.D;
  a.groups = c.groups;
  a.stats = const_cast<float*>(c.stats);
  a.clear = c.clear;
  return a;
}

// A row takes a wave of its own where there are many (from kNormWaveRows on) and it is no wider than kNormWavePieces
// pieces a lane: no wait for other waves.  Few rows take four waves each for their latency, wide ones for
// the rows in flight.  bf16, us with one wave and with four: 512 rows of 5120 7.0 and 4.8; 4096 of 512 4.0 and
// 6.7, of 5120 21.7 and 17.7; 32760 of 1024 24 and 40, of 2560 65 and 76, of 4096 102 and 98, of 5120 134 and 122.
constexpr int64_t kNormWaveRows = 1024, kNormWavePieces = 6;

template <bool BF16>
void norm_forward(const NormCall& c, hipStream_t stream) {
  constexpr int V = BF16 ? 8 : 4;
  const NormArgs a = norm_args(c);
  auto go = [&](auto v, auto w, auto j) {
    constexpr int VV = decltype(v)::value, W = decltype(w)::value, J = decltype(j)::value;
    hipLaunchKernelGGL((norm_kernel<BF16, VV, W, J>), norm_grid(W > 1 ? c.M : (c.M + 3) / 4), dim3(W == 1 ? kNormThreads : W * 64), 0, stream, a);
  };
  if (!norm_wide(c)) {
    if (c.D <= 2048) pick<1, 2, 4, 8>((c.D + 255) / 256, [&](auto j) { go(Int<1>(), Int<4>(), j); });
    else pick<4, 8>((c.D + 1023) / 1024, [&](auto j) { go(Int<1>(), Int<16>(), j); });
    return;
  }
  const int64_t pieces = c.D / V, one = (pieces + 63) / 64;
  if (c.M >= kNormWaveRows && one <= kNormWavePieces) pick<1, 2, 3, 4, 6>(one, [&](auto j) { go(Int<V>(), Int<1>(), j); });
  else pick<1, 2, 3, 4, 6, 8, 12, 16>((pieces + 255) / 256, [&](auto j) { go(Int<V>(), Int<4>(), j); });
}

// Waves a row of the gradient: up to four pieces a lane.
int norm_back_waves(int64_t pieces) { return pieces <= 64 * 2 ? 1 : pieces <= 256 * 4 ? 4 : pieces <= 512 * 4 ? 8 : 16; }

// Workgroups of 32 columns' sums below which each takes 1024 threads, not 256: fewer leave the chip's places free (the gradient of 7284 x
// 200 20.8 us and 17.8 so, of 32760 x 1024 55.7 and 49.5, of 64 x 5120 12.9 and 13.2; with 640 workgroups no gain).
constexpr int64_t kNormSumBlocks = 256;

int norm_chunk(int64_t M) {
  // enough chunks to fill the chip, few enough that their sums stay small against the rows
  return (int)std::max<int64_t>(2, std::min<int64_t>(kNormChunk, M / 512));
}

template <bool BF16>
void norm_backward(const NormCall& c, NormArgs a, hipStream_t stream) {
  constexpr int V = BF16 ? 8 : 4;
  const int64_t chunks = (c.M + a.rows - 1) / a.rows;
  auto go = [&](auto v, auto w, auto j) {
    constexpr int VV = decltype(v)::value, W = decltype(w)::value, J = decltype(j)::value;
    hipLaunchKernelGGL((norm_back_kernel<BF16, VV, W, J>), norm_grid(W > 1 ? chunks : (chunks + 3) / 4), dim3(W == 1 ? kNormThreads : W * 64), 0, stream, a);
  };
  if (!norm_wide(c)) {
    const int64_t D = c.D;
    if (D <= 256) pick<1, 2, 4>((D + 63) / 64, [&](auto j) { go(Int<1>(), Int<1>(), j); });
    else if (D <= 2048) pick<2, 4, 8>((D + 255) / 256, [&](auto j) { go(Int<1>(), Int<4>(), j); });
    else pick<4, 8>((D + 1023) / 1024, [&](auto j) { go(Int<1>(), Int<16>(), j); });
    return;
  }
  const int64_t pieces = c.D / V;
  switch (norm_back_waves(pieces)) {
    case 1: pick<1, 2>((pieces + 63) / 64, [&](auto j) { go(Int<V>(), Int<1>(), j); }); break;
    case 4: pick<1, 2, 3, 4>((pieces + 255) / 256, [&](auto j) { go(Int<V>(), Int<4>(), j); }); break;
    case 8: pick<3, 4>((pieces + 511) / 512, [&](auto j) { go(Int<V>(), Int<8>(), j); }); break;
    default: pick<3, 4>((pieces + 1023) / 1024, [&](auto j) { go(Int<V>(), Int<16>(), j); }); break;
  }
}

size_t norm_part_bytes(int64_t M, int64_t D, int64_t G) {
  const int64_t rows = norm_chunk(M);
  return (((size_t)((M + rows - 1) / rows + std::max<int64_t>(G, 1)) * 2 * D * 4) + 255) & ~(size_t)255;
}

}  // namespace norm

bool norm_fits(int dt, int64_t D, bool wide) {
  using namespace norm;
  return wide ? D <= (dt == kDtBF16 ? kNormMaxD : kNormMaxD / 2) : D <= kNormMaxDNarrow;
}
bool norm_is_wide(const NormCall& c) {
  using namespace norm;
  return norm_wide(c);
}

hipError_t launch_norm(const NormCall& c, hipStream_t stream) {
  using namespace norm;
  if (c.dt == kDtBF16) norm_forward<true>(c, stream);
  else norm_forward<false>(c, stream);
  return hipGetLastError();
}

// Workspace: the chunks' sums, then the groups'.
size_t norm_back_workspace(int64_t M, int64_t D, int64_t G) {
  using namespace norm;
  return norm_part_bytes(M, D, G) + (size_t)std::max<int64_t>(G, 1) * 2 * D * 8;
}

hipError_t launch_norm_back(const NormCall& c, float* dw, float* db, float* dscale, float* dshift, void* ws,
                            hipStream_t stream) {
  using namespace norm;
  NormArgs a = norm_args(c);
  a.rows = norm_chunk(c.M);
  const bool sums = dw != nullptr || db != nullptr || dscale != nullptr || dshift != nullptr;
  a.part = sums ? (float*)ws : nullptr;
  if (c.dt == kDtBF16) norm_backward<true>(c, a, stream);
  else norm_backward<false>(c, a, stream);
  if (!sums) return hipGetLastError();
  SumArgs s{};
  s.M = c.M;
  s.D = (int)c.D;
  s.G = (int)std::max<int64_t>(c.G, 1);
  s.rows = a.rows;
  s.part = a.part;
  s.groups = c.groups;
  s.w = c.w;
  s.b = c.b;
  s.scale = c.scale.p;
  s.scale_row = c.scale.row;
  s.dw = dw;
  s.db = db;
  s.dscale = dscale;
  s.dshift = dshift;
  const bool several = (dw != nullptr || db != nullptr) && (s.G > 1 || s.scale != nullptr);
  s.group = several ? (double*)((uint8_t*)ws + norm_part_bytes(c.M, c.D, c.G)) : nullptr;
  const unsigned cols = (unsigned)((c.D + 31) / 32);
  auto go = [&](auto bf16) {
    constexpr bool B = decltype(bf16)::value;
    const int64_t wide = std::min<int64_t>(s.G, kNormSumGroups);
    const dim3 grid((unsigned)wide, cols, (unsigned)((s.G + wide - 1) / wide));
    auto sum = [&](auto threads) {
      constexpr int T = decltype(threads)::value;
      if (c.D % 4 == 0) hipLaunchKernelGGL((norm_sum_kernel<B, 4, T>), grid, dim3(T), 0, stream, s);
      else hipLaunchKernelGGL((norm_sum_kernel<B, 1, T>), grid, dim3(T), 0, stream, s);
    };
    if ((int64_t)cols * s.G < kNormSumBlocks) sum(Int<1024>());
    else sum(Int<256>());
    if (several) hipLaunchKernelGGL(norm_weight_kernel<B>, dim3(cols), dim3(256), 0, stream, s);
  };
  if (c.dt == kDtBF16) go(std::true_type());
  else go(std::false_type());
  return hipGetLastError();
}

}  // namespace rtl
