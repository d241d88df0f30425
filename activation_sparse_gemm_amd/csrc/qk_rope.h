// qk_rope.h -- the rotary embedding over several position axes, alone or after the RMS norm
// of each query and key head, and the gradient of the two together.  Row-wise passes over
// [M, heads, D] with a row and a head stride, compiled into sparsify.hip's unit.
//
//   phi_p = pos[m, axis(p)] f_p          one angle per token and channel pair p
//   (x0, x1) -> (x0 cos - x1 sin, x1 cos + x0 sin)
//   norm:  n = x r w,  r = 1 / sqrt(mean(x^2) + eps)
//   back:  t = R^T dy,  dw = sum t n0,  dx = r (w t - n0 / D sum(w t n0)),  n0 = x r
//
// Bound: memory (each element read once and written once; the gradient reads two and writes
// one).  A group of GL lanes owns one head of one token, a lane eight channels (four pairs):
// one 16-byte access (bf16, pairs side by side) or two, the norm's sum inside the group's lanes.
// A group takes HC heads of its token, so that a lane's four angles are formed once for HC
// heads and HC loads are in flight before the first is used.
//
// Angles are formed in revolutions (pos f / 2 pi), from frequencies in two fp32 words and reduced
// by their nearest whole number before the product is rounded, so a position as far as 2^24 loses
// nothing: the reduced angle is within 2^-25 revolutions.
#pragma once
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "rtl_device.h"
#include "rtl_launch.h"

namespace rtl {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;

// Frequencies in revolutions per unit of position (the sum of two fp32 words), and the position
// axis, of each pair.
struct RopeTable {
  float hi[kRopeMaxPairs], lo[kRopeMaxPairs];
  uint8_t axis[kRopeMaxPairs];
};

struct RopeTensor {
  void* p;
  int64_t row, head;  // strides in elements
};

struct RopeArgs {
  int H[2];                // heads of the two tensors (queries, keys); the second may be 0
  uint32_t items, nq, nc;  // items: (token, chunk of HC heads) pairs; chunks of the first tensor, of both
  uint32_t blocks[2];      // backward: workgroups on the first tensor, on the second
  int D, pairs, axes;
  float eps, sign, inv_d;
  const float* pos;
  RopeTensor x[2], y[2];   // backward: y is dy, dx the output
  RopeTensor dx[2];
  const void* w[2];
  float* part;             // backward: [workgroups][D]
};

// Eight values of a head as fp32, channels lo .. lo + 3 and hi .. hi + 3: one piece of 16 bytes in bf16,
// or two pieces where a pair's channels lie half the rotated width apart, and in fp32, whose pieces
// then follow on from lane to lane (side by side they are 32 bytes apart: 16000 x 32 x 64 in 53
// us against 41).  Units at or past the rotated channels hold eight consecutive channels.
template <bool BF16, bool HALVES>
struct RopeUnit {
  int lo, hi;  // channel of the first four values and of the last four
  __device__ __forceinline__ RopeUnit(int u, int pairs) {
    const bool split = (HALVES || !BF16) && 4 * u < pairs;
    lo = split ? 4 * u : 8 * u;
    hi = split ? 4 * u + pairs : 8 * u + 4;
  }
  struct Raw {
    u32x4 a, b;  // bf16: a only
  };
  __device__ __forceinline__ Raw load(const void* base, int64_t at) const {
    Raw r;
    if (BF16) {
      const uint16_t* p = (const uint16_t*)base + at;
      if (HALVES) {
        const u32x2 v0 = *reinterpret_cast<const u32x2*>(p + lo), v1 = *reinterpret_cast<const u32x2*>(p + hi);
        r.a = u32x4{v0[0], v0[1], v1[0], v1[1]};
      } else {
        r.a = *reinterpret_cast<const u32x4*>(p + lo);
      }
    } else {
      const float* p = (const float*)base + at;
      r.a = *reinterpret_cast<const u32x4*>(p + lo);
      r.b = *reinterpret_cast<const u32x4*>(p + hi);
    }
    return r;
  }
  // Values in memory order: v[0..3] from lo, v[4..7] from hi.
  __device__ __forceinline__ static void unpack(const Raw& r, float (&v)[8]) {
    if (BF16) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[2 * i] = bf16lo(r.a[i]);
        v[2 * i + 1] = bf16hi(r.a[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        v[i] = __uint_as_float(r.a[i]);
        v[4 + i] = __uint_as_float(r.b[i]);
      }
    }
  }
  template <bool PAST, typename V>
  __device__ __forceinline__ static void put(V v, void* p) {
    if constexpr (PAST) __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
    else *reinterpret_cast<V*>(p) = v;
  }
  // PAST: by stores that bypass the caches.
  template <bool PAST>
  __device__ __forceinline__ void store(void* base, int64_t at, const float (&v)[8]) const {
    if (BF16) {
      typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; i++)
        w[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
      uint16_t* p = (uint16_t*)base + at;
      if (HALVES) {
        put<PAST>(u32x2{w[0], w[1]}, p + lo);
        put<PAST>(u32x2{w[2], w[3]}, p + hi);
      } else {
        put<PAST>(u32x4{w[0], w[1], w[2], w[3]}, p + lo);
      }
    } else {
      float* p = (float*)base + at;
      put<PAST>(f32x4{v[0], v[1], v[2], v[3]}, p + lo);
      put<PAST>(f32x4{v[4], v[5], v[6], v[7]}, p + hi);
    }
  }
  // Rotates the unit's four pairs: (2i, 2i + 1) in place, or (i, 4 + i).
  __device__ __forceinline__ void rotate(float (&v)[8], const float (&c)[4], const float (&s)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int a = HALVES ? i : 2 * i, b = HALVES ? 4 + i : 2 * i + 1;
      const float x0 = v[a], x1 = v[b];
      v[a] = x0 * c[i] - x1 * s[i];
      v[b] = x1 * c[i] + x0 * s[i];
    }
  }
};

// A unit's four frequencies and axes.
template <bool BF16, bool HALVES>
struct RopeFreq {
  f32x4 hi, lo;
  int axis[4];
  bool turned;  // false past the rotated channels
  __device__ __forceinline__ RopeFreq(const RopeArgs& a, const RopeTable& t, int u) : turned(4 * u < a.pairs) {
    if (!turned) return;
    // the pairs of the unit's first four values and of its last (the same four in RTL_ROPE_HALVES)
    const int p0 = BF16 || HALVES ? 4 * u : 2 * u, p1 = BF16 || HALVES ? 4 * u + 2 : 2 * u + a.pairs / 2;
    const float2 h0 = *reinterpret_cast<const float2*>(t.hi + p0), h1 = *reinterpret_cast<const float2*>(t.hi + p1);
    const float2 l0 = *reinterpret_cast<const float2*>(t.lo + p0), l1 = *reinterpret_cast<const float2*>(t.lo + p1);
    hi = f32x4{h0.x, h0.y, h1.x, h1.y};
    lo = f32x4{l0.x, l0.y, l1.x, l1.y};
    const uint32_t four = *reinterpret_cast<const uint16_t*>(t.axis + p0) | (uint32_t)*reinterpret_cast<const uint16_t*>(t.axis + p1) << 16;
#pragma unroll
    for (int i = 0; i < 4; i++) axis[i] = (four >> (8 * i)) & 255;
  }
};
// cos and sin (times `sign`) of the unit's four angles for token m; 1 and 0 past the rotated
// channels.  By the hardware's instructions, which take revolutions: within 2.2 * 2^-24 of the exact
// values at every multiple of 2^-24 in [-1/2, 1/2] (measured), as near as the library's functions.
template <typename Freq>
__device__ __forceinline__ void rope_angles(const RopeArgs& a, const Freq& f, int64_t m, float (&c)[4],
                                            float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (!f.turned) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const float p = a.pos[m * a.axes + f.axis[i]];
    // p hi - (its nearest whole number) in one rounding, then p lo
    const float r = fmaf(p, f.lo[i], fmaf(p, f.hi[i], -rintf(p * f.hi[i])));
    s[i] = a.sign * __builtin_amdgcn_sinf(r);
    c[i] = __builtin_amdgcn_cosf(r);
  }
}

// v + v of the lane that the row pattern CTRL names (no LDS: the exchange is an operand of the sum).
template <int CTRL>
__device__ __forceinline__ float add_row(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
// Sum over the GL lanes of a group, the same in each of them: over lanes 1, 2, 4 and 8 apart (by
// swaps in a quad, then mirrors, whose halves are uniform by then), 16 apart through a shuffle.
template <int GL>
__device__ __forceinline__ float group_sum(float v) {
  v = add_row<0xB1>(v);   // quad_perm 1,0,3,2
  v = add_row<0x4E>(v);   // quad_perm 2,3,0,1
  if (GL >= 8) v = add_row<0x141>(v);   // row_half_mirror
  if (GL >= 16) v = add_row<0x140>(v);  // row_mirror
  if (GL >= 32) v += __shfl_xor(v, 16, 64);
  return v;
}

// The unit's eight weights in the order of RopeUnit::unpack (1 without weights).
template <bool BF16, bool HALVES>
__device__ __forceinline__ void rope_weights(const RopeUnit<BF16, HALVES>& un, const void* w, float (&v)[8]) {
  if (w != nullptr) {
    RopeUnit<BF16, HALVES>::unpack(un.load(w, 0), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = 1.f;
  }
}

// The rotation, after the norm (NORM) or alone.  Measured in bf16: alone 32760 x 40 x 128 in 112-120
// us (5.6-6.0 TB/s, where a copy of its size runs at 5.5); with the norm 32760 x 80 x 128 in 222-237
// us (5.7-6.0) and 4608 x 48 x 128 in 20 us (5.8).  PAST: stores that bypass the caches (rope_past).
// Loads that do lost up to 20% where the input still lay in the last-level cache.
template <bool BF16, bool HALVES, bool NORM, bool PAST, int GL, int HC>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(const RopeArgs a, const RopeTable t) {
  const int u = threadIdx.x % GL;
  const uint32_t item = (blockIdx.y * gridDim.x + blockIdx.x) * (kRopeThreads / GL) + threadIdx.x / GL;
  const bool live = item < a.items && 8 * u < a.D;
  if (!NORM && !live) return;
  const uint32_t token = live ? item / a.nc : 0, chunk = live ? item - token * a.nc : 0;
  const int64_t m = token;
  const int which = chunk >= a.nq;
  const int h0 = (int)(which ? chunk - a.nq : chunk) * HC;
  const int nh = live ? min(HC, a.H[which] - h0) : 0;
  const RopeUnit<BF16, HALVES> un(u, a.pairs);
  const RopeTensor x = a.x[which], y = a.y[which];

  typename RopeUnit<BF16, HALVES>::Raw raw[HC];
#pragma unroll
  for (int j = 0; j < HC; j++)
    if (j < nh) raw[j] = un.load(x.p, m * x.row + (int64_t)(h0 + j) * x.head);
  float c[4], s[4], w[8];
  if (nh > 0) {
    rope_angles(a, RopeFreq<BF16, HALVES>(a, t, u), m, c, s);
    if (NORM) rope_weights<BF16, HALVES>(un, a.w[which], w);
  }
#pragma unroll
  for (int j = 0; j < HC; j++) {
    float v[8];
    if (j < nh) {
      RopeUnit<BF16, HALVES>::unpack(raw[j], v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = 0.f;
    }
    if (NORM) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) q += v[i] * v[i];
      const float r = __builtin_amdgcn_rsqf(fmaf(group_sum<GL>(q), a.inv_d, a.eps));
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = v[i] * r * w[i];
    }
    if (j < nh) {
      un.rotate(v, c, s);
      un.template store<PAST>(y.p, m * y.row + (int64_t)(h0 + j) * y.head, v);
    }
  }
}

// Gradient of norm and rotation.  A fixed number of workgroups walks over the items, each on one
// of the two tensors (shared out by their heads), the next item's loads in flight while one is
// formed; each lane sums its channels' dw in fp32 over kQkBackFlush items at a time and these in
// double, in LDS (it can meet 2^18 heads, where a tensor's share is one workgroup; as one fp32 sum
// 1700 alike terms were 400 half steps off), the workgroup adds its groups, and qk_dw_kernel adds the
// workgroups: one order, the same result on every run.
// Bound by memory and, nearly as much, by its vector instructions (the norm, two sums and the
// rotation for every element of two inputs).  Measured: 4608 x 32 x 128 in bf16 22 us (5.2 TB/s).
constexpr uint32_t kQkBackFlush = 16;  // even
template <bool BF16, bool HALVES, int GL, int HC>
__global__ __launch_bounds__(kRopeThreads) void qk_back_kernel(const RopeArgs a, const RopeTable t) {
  constexpr int NG = kRopeThreads / GL;
  typedef RopeUnit<BF16, HALVES> Unit;
  __shared__ double sums[8][kRopeThreads + 8];  // 64 columns of the last sum fall in different banks
  const int u = threadIdx.x % GL, g = threadIdx.x / GL;
  const Unit un(u, a.pairs);
  const bool lane = 8 * u < a.D;
  const int which = blockIdx.x >= a.blocks[0];
  const uint32_t block = which ? blockIdx.x - a.blocks[0] : blockIdx.x;
  const int H = a.H[which];
  const uint32_t nc = (uint32_t)(H + HC - 1) / HC, items = a.items * nc, stride = a.blocks[which] * NG;  // a.items: tokens
  const RopeTensor x = a.x[which], y = a.y[which], dx = a.dx[which];
  float w[8], dw[8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    w[i] = dw[i] = 0.f;
    sums[i][threadIdx.x] = 0.0;
  }
  if (lane) rope_weights<BF16, HALVES>(un, a.w[which], w);

  const RopeFreq<BF16, HALVES> freq(a, t, u);
  struct Item {
    typename Unit::Raw x[HC], y[HC];
    uint32_t m;
    int h0, nh;  // the same for all lanes of a group; lanes past D hold zeros
  };
  auto fetch = [&](uint32_t item, Item& it) {
    const bool live = item < items;
    it.m = live ? item / nc : 0;
    it.h0 = (int)((live ? item : 0) - it.m * nc) * HC;
    it.nh = live ? min(HC, H - it.h0) : 0;
    const int64_t xat = (int64_t)it.m * x.row + (int64_t)it.h0 * x.head, yat = (int64_t)it.m * y.row + (int64_t)it.h0 * y.head;
#pragma unroll
    for (int j = 0; j < HC; j++) {
      it.x[j] = it.y[j] = typename Unit::Raw{};
      if (j < it.nh && lane) {
        it.x[j] = un.load(x.p, xat + j * x.head);
        it.y[j] = un.load(y.p, yat + j * y.head);
      }
    }
  };
  auto form = [&](const Item& it) {
    if (it.nh == 0) return;
    float c[4], s[4];
    rope_angles(a, freq, it.m, c, s);
    const int64_t at = (int64_t)it.m * dx.row + (int64_t)it.h0 * dx.head;
#pragma unroll
    for (int j = 0; j < HC; j++) {
      if (j >= it.nh) break;
      float v[8], d[8];
      Unit::unpack(it.x[j], v);
      Unit::unpack(it.y[j], d);
      un.rotate(d, c, s);
      float q = 0.f, p = 0.f, wd[8];
#pragma unroll
      for (int i = 0; i < 8; i++) q = fmaf(v[i], v[i], q);
      const float r = __builtin_amdgcn_rsqf(fmaf(group_sum<GL>(q), a.inv_d, a.eps));
      // with n = x r: dw = t n, dx = r (w t - n sum(w t n) / D), no factor larger than the result
#pragma unroll
      for (int i = 0; i < 8; i++) {
        v[i] *= r;
        dw[i] = fmaf(d[i], v[i], dw[i]);
        wd[i] = d[i] * w[i];
        p = fmaf(wd[i], v[i], p);
      }
      const float k = group_sum<GL>(p) * a.inv_d;
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = r * fmaf(-v[i], k, wd[i]);
      if (lane) un.template store<true>(dx.p, at + j * dx.head, v);
    }
  };
  auto flush = [&]() {  // the lane's own sums: nothing to wait for
#pragma unroll
    for (int i = 0; i < 8; i++) {
      sums[i][threadIdx.x] += (double)dw[i];
      dw[i] = 0.f;
    }
  };
  Item one, two;
  uint32_t item = block * NG + g;
  const uint32_t rounds = (items + stride - 1) / stride;  // the same for every lane: the sums are exchanged
  fetch(item, one);
  for (uint32_t r = 0; r < rounds; r += 2) {
    fetch(item + stride, two);
    form(one);
    if (r + 1 == rounds) break;
    fetch(item + 2 * stride, one);
    form(two);
    item += 2 * stride;
    if (r % kQkBackFlush == kQkBackFlush - 2) flush();
  }
  flush();
  __syncthreads();
  for (int at = threadIdx.x; at < a.D; at += kRopeThreads) {
    double sum = 0.0;
    for (int j = 0; j < NG; j++) sum += sums[at % 8][j * GL + at / 8];
    const Unit ue(at / 8, a.pairs);
    a.part[(int64_t)blockIdx.x * a.D + (at % 8 < 4 ? ue.lo + at % 8 : ue.hi + at % 8 - 4)] = (float)sum;
  }
}

// dw[k][ch] = sum over tensor k's workgroups of part[.][ch], in double precision: 16 columns a
// workgroup, 64 bytes of a row to four lanes, 64 rows at a time (D = 128: 4 us, a launch's latency).
__global__ __launch_bounds__(256) void qk_dw_kernel(const float* part, int blocks_q, int blocks_k, int D, float* dqw,
                                                    float* dkw) {
  __shared__ double red[64][16];
  const int c4 = (threadIdx.x & 3) * 4, lane = threadIdx.x >> 2, col0 = blockIdx.x * 16, k = blockIdx.y;
  const float* rows = part + (k ? (int64_t)blocks_q * D : 0);
  const int blocks = k ? blocks_k : blocks_q;
  float* out = k ? dkw : dqw;
  if (out == nullptr) return;
  double sum[4] = {0.0, 0.0, 0.0, 0.0};
  if (col0 + c4 < D) {
#pragma unroll 4
    for (int b = lane; b < blocks; b += 64) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(rows + (int64_t)b * D + col0 + c4);
#pragma unroll
      for (int i = 0; i < 4; i++) sum[i] += (double)v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++) red[lane][c4 + i] = sum[i];
  __syncthreads();
  const int col = col0 + threadIdx.x;
  if (threadIdx.x < 16 && col < D) {
    double all = 0.0;
    for (int j = 0; j < 64; j++) all += red[j][threadIdx.x];
    out[col] = (float)all;
  }
}

namespace {

// Workgroups of the gradient kernel: enough to fill the chip, few enough that the sum over
// them stays small against the pass itself.
constexpr int64_t kQkBackBlocks = 1024;
// Heads per group there (with the next item's in flight; measured at 32760 x 80 x 128: one 519 us,
// two 458, four 573, whose registers leave two waves a SIMD).
constexpr int kQkBackHeads = 2;

int rope_heads(int64_t M, int64_t H, int gl) {
  // Heads per group: eight where the lanes still fill the chip (256 CUs of 2048), else fewer, so
  // that a short call spreads over more CUs.
  for (int hc : {8, 4, 2})
    if (M * ((H + hc - 1) / hc) * gl >= (int64_t)256 * 2048) return hc;
  return 1;
}

void rope_fill(const RopeCall& c, int hc, RopeArgs& a, RopeTable& t) {
  a = RopeArgs{};
  a.H[0] = (int)c.H[0];
  a.H[1] = (int)c.H[1];
  a.nq = (uint32_t)((c.H[0] + hc - 1) / hc);
  a.nc = a.nq + (uint32_t)((c.H[1] + hc - 1) / hc);
  a.items = (uint32_t)c.M * a.nc;
  a.D = (int)c.D;
  a.axes = c.axes;
  a.eps = c.eps;
  a.inv_d = 1.f / (float)c.D;
  a.pos = c.pos;
  for (int k = 0; k < 2; k++) {
    a.x[k] = RopeTensor{const_cast<void*>(c.x[k].p), c.x[k].row, c.x[k].head};
    a.y[k] = RopeTensor{const_cast<void*>(c.y[k].p), c.y[k].row, c.y[k].head};
    a.dx[k] = RopeTensor{const_cast<void*>(c.dx[k].p), c.dx[k].row, c.dx[k].head};
    a.w[k] = c.w[k];
  }
  int p = 0;
  for (int ax = 0; ax < c.axes; ax++) {
    // theta^(-2 i / d) / (2 pi), each from the last by one product: i products of 2^-53 each
    const double ratio = pow(c.theta, -2.0 / (double)c.dims[ax]);
    double f = 0.15915494309189533577;
    for (int i = 0; i < c.dims[ax] / 2; i++, p++, f *= ratio) {
      t.hi[p] = (float)f;
      t.lo[p] = (float)(f - (double)t.hi[p]);
      t.axis[p] = (uint8_t)ax;
    }
  }
  a.pairs = p;
  a.sign = c.inverse ? -1.f : 1.f;
}

// Whether the outputs are stored past the caches.  That pays where a head fills whole 128-byte lines
// (rotation of 16000 x 32 heads: 128 wide in bf16 41 us against 48, 64 in fp32 41 against 45), or
// whole halves of them and two lines at least (112 in fp32 79 against 98; 90000 tokens 508 against
// 488); a line that is stored in parts goes out in parts (80 in bf16 41 against 28, 120 at 90000
// tokens 411 against 275, 48 in fp32 39 against 33).  The gradient always stores so: it gains up to 17%
// where a head fills lines (16000 x 32 x 128 in bf16 73 us against 85) and elsewhere loses at
// most as much at many tokens (60000 x 32 x 56: 158 against 131) and gains it at fewer (16000 x
// 32 x 56 in fp32 67 against 77, 4000 tokens 3-8%).
bool rope_past(const RopeCall& c) {
  const int64_t es = c.dt == kDtBF16 ? 2 : 4, width = c.D * es;
  uint64_t bits = (uint64_t)width;
  for (int k = 0; k < (c.H[1] > 0 ? 2 : 1); k++)
    bits |= (uint64_t)(uintptr_t)c.y[k].p | (uint64_t)(c.y[k].row * es) | (uint64_t)(c.y[k].head * es);
  return bits % 128 == 0 || (bits % 64 == 0 && width >= 256);
}

template <bool BF16, bool HALVES, bool NORM, int GL>
void rope_launch(const RopeCall& c, hipStream_t stream) {
  RopeArgs a;
  RopeTable t;
  const int hc = rope_heads(c.M, c.H[0] + c.H[1], GL);
  rope_fill(c, hc, a, t);
  // rows of 2^20 workgroups: a launch takes fewer than 2^32 threads in one dimension
  const uint32_t blocks = (a.items + kRopeThreads / GL - 1) / (kRopeThreads / GL), row = std::min(blocks, 1u << 20);
  const dim3 grid(row, (blocks + row - 1) / row), block(kRopeThreads);
  auto go = [&](auto p) {
    constexpr bool P = decltype(p)::value;
    if (hc == 8) hipLaunchKernelGGL((rope_kernel<BF16, HALVES, NORM, P, GL, 8>), grid, block, 0, stream, a, t);
    else if (hc == 4) hipLaunchKernelGGL((rope_kernel<BF16, HALVES, NORM, P, GL, 4>), grid, block, 0, stream, a, t);
    else if (hc == 2) hipLaunchKernelGGL((rope_kernel<BF16, HALVES, NORM, P, GL, 2>), grid, block, 0, stream, a, t);
    else hipLaunchKernelGGL((rope_kernel<BF16, HALVES, NORM, P, GL, 1>), grid, block, 0, stream, a, t);
  };
  if (rope_past(c)) go(std::true_type());
  else go(std::false_type());
}

template <bool BF16, bool HALVES, int GL>
void qk_back_launch(const RopeCall& c, float* part, RopeArgs& a, hipStream_t stream) {
  RopeTable t;
  const int hc = rope_heads(c.M, c.H[0] + c.H[1], GL) >= kQkBackHeads ? kQkBackHeads : 1;
  rope_fill(c, hc, a, t);
  a.items = (uint32_t)c.M;  // tokens; the kernel counts its own tensor's chunks
  a.part = part;
  // Workgroups: up to kQkBackBlocks, shared out by heads, no more than a tensor has items for.
  const int64_t ng = kRopeThreads / GL;
  for (int k = 0; k < 2; k++) {
    const int64_t want = (c.M * ((c.H[k] + hc - 1) / hc) + ng - 1) / ng;
    const int64_t share = std::max<int64_t>(1, kQkBackBlocks * c.H[k] / (c.H[0] + c.H[1]) - 1);
    a.blocks[k] = (uint32_t)std::min(want, share);
  }
  const dim3 grid(a.blocks[0] + a.blocks[1]), block(kRopeThreads);
  if (hc == kQkBackHeads) hipLaunchKernelGGL((qk_back_kernel<BF16, HALVES, GL, kQkBackHeads>), grid, block, 0, stream, a, t);
  else hipLaunchKernelGGL((qk_back_kernel<BF16, HALVES, GL, 1>), grid, block, 0, stream, a, t);
}

// Calls f(std::integral_constant<int, GL>) for the lanes of a group, the power of two (four or
// more) that holds D / 8 units.
template <typename F>
void rope_lanes(int64_t D, F f) {
  if (D <= 32) f(std::integral_constant<int, 4>());
  else if (D <= 64) f(std::integral_constant<int, 8>());
  else if (D <= 128) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 32>());
}

}  // namespace

size_t qk_back_workspace(int64_t D) { return (size_t)kQkBackBlocks * D * 4; }

hipError_t launch_rope(const RopeCall& c, hipStream_t stream) {
  const bool norm = c.norm, halves = c.halves, bf16 = c.dt == kDtBF16;
  rope_lanes(c.D, [&](auto gl) {
    constexpr int GL = decltype(gl)::value;
    auto go = [&](auto b, auto h) {
      constexpr bool B = decltype(b)::value, H = decltype(h)::value;
      if (norm) rope_launch<B, H, true, GL>(c, stream);
      else rope_launch<B, H, false, GL>(c, stream);
    };
    if (bf16 && halves) go(std::true_type(), std::true_type());
    else if (bf16) go(std::true_type(), std::false_type());
    else if (halves) go(std::false_type(), std::true_type());
    else go(std::false_type(), std::false_type());
  });
  return hipGetLastError();
}

hipError_t launch_qk_back(const RopeCall& c, float* dqw, float* dkw, void* ws, hipStream_t stream) {
  RopeArgs a{};
  float* part = (float*)ws;
  const bool halves = c.halves, bf16 = c.dt == kDtBF16;
  rope_lanes(c.D, [&](auto gl) {
    constexpr int GL = decltype(gl)::value;
    if (bf16 && halves) qk_back_launch<true, true, GL>(c, part, a, stream);
    else if (bf16) qk_back_launch<true, false, GL>(c, part, a, stream);
    else if (halves) qk_back_launch<false, true, GL>(c, part, a, stream);
    else qk_back_launch<false, false, GL>(c, part, a, stream);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (dqw == nullptr && dkw == nullptr)) return e;
  hipLaunchKernelGGL(qk_dw_kernel, dim3((unsigned)((c.D + 15) / 16), 2), dim3(256), 0, stream, part, (int)a.blocks[0],
                     (int)a.blocks[1], (int)c.D, dqw, dkw);
  return hipGetLastError();
}

}  // namespace rtl
