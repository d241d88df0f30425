// qk_rope.h -- the rotary embedding over several position axes, alone or after the RMS norm
// of each query and key head, and the gradient of the two together.  Row-wise passes over
// [M, heads, D] with a row and a head stride, compiled into sparsify.hip's unit.
//
//   phi_p = pos[m, axis(p)] f_p          one angle per token and channel pair p
//   (x0, x1) -> (x0 cos - x1 sin, x1 cos + x0 sin)
//   norm:  n = x r w,  r = 1 / sqrt(mean(x^2) + eps)
//   back:  t = R^T dy,  dw = sum t x r,  dx = r w t - x r^3 / D sum(w t x)
//
// Bound: memory (each element read once and written once; the gradient reads two and writes
// one).  A group of GL lanes owns one head of one token, a lane eight channels (four pairs):
// one 16-byte access (two of 8 where a pair's channels lie D/2 apart), the norm's sum inside
// the group's lanes.  A group takes HC heads of its token, so that a lane's four angles are
// formed once for HC heads and HC loads are in flight before the first is used.
//
// Angles are formed in double precision and in revolutions (pos f / 2 pi, reduced by its
// nearest whole number), so a far position loses nothing; the reduced angle is rounded to
// fp32 (2^-25 revolutions = 1.9e-7 radians at most).
#pragma once
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "rtl_device.h"
#include "rtl_launch.h"

namespace rtl {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;

// Frequencies in revolutions per unit of position, and the position axis, of each pair.
struct RopeTable {
  double f[kRopeMaxPairs];
  uint8_t axis[kRopeMaxPairs];
};

struct RopeTensor {
  void* p;
  int64_t row, head;  // strides in elements
};

struct RopeArgs {
  int64_t M, items;        // items: (token, chunk of HC heads) pairs
  int H[2];                // heads of the two tensors (queries, keys); the second may be 0
  int nq, nc;              // chunks of the first tensor, of both
  int D, pairs, axes;
  float eps, sign;
  const float* pos;
  RopeTensor x[2], y[2];   // backward: y is dy, dx the output
  RopeTensor dx[2];
  const void* w[2];
  float* part;             // backward: [workgroups][2][D]
};

// Eight values of a head as fp32: values 2i and 2i + 1 are pair 4 u + i of unit u.  Units at
// or past the rotated channels hold eight consecutive channels.
template <bool BF16, bool HALVES>
struct RopeUnit {
  int lo, hi;  // channel of the first four values and of the last four
  __device__ __forceinline__ RopeUnit(int u, int pairs) {
    const bool split = HALVES && 4 * u < pairs;
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
  __device__ __forceinline__ void store(void* base, int64_t at, const float (&v)[8]) const {
    if (BF16) {
      typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; i++)
        w[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[2 * i], (__bf16)v[2 * i + 1]});
      uint16_t* p = (uint16_t*)base + at;
      if (HALVES) {
        *reinterpret_cast<u32x2*>(p + lo) = u32x2{w[0], w[1]};
        *reinterpret_cast<u32x2*>(p + hi) = u32x2{w[2], w[3]};
      } else {
        *reinterpret_cast<u32x4*>(p + lo) = u32x4{w[0], w[1], w[2], w[3]};
      }
    } else {
      float* p = (float*)base + at;
      *reinterpret_cast<f32x4*>(p + lo) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(p + hi) = f32x4{v[4], v[5], v[6], v[7]};
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

// cos and sin (times `sign`) of the unit's four angles; 1 and 0 past the rotated channels.
__device__ __forceinline__ void rope_angles(const RopeArgs& a, const RopeTable& t, int64_t m, int u, float (&c)[4],
                                            float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i++) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  if (4 * u >= a.pairs) return;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int p = 4 * u + i;
    const double rev = (double)a.pos[m * a.axes + t.axis[p]] * t.f[p];
    const float r = (float)(rev - rint(rev));
    sincospif(2.f * r, &s[i], &c[i]);
    s[i] *= a.sign;
  }
}

// Sum over the GL lanes of a group, the same in each of them.
template <int GL>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = GL / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
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

template <bool BF16, bool HALVES, bool NORM, int GL, int HC>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(const RopeArgs a, const RopeTable t) {
  const int u = threadIdx.x % GL;
  const int64_t item = (int64_t)blockIdx.x * (kRopeThreads / GL) + threadIdx.x / GL;
  const bool live = item < a.items && 8 * u < a.D;
  if (!NORM && !live) return;
  const int64_t m = live ? item / a.nc : 0;
  const int chunk = live ? (int)(item % a.nc) : 0;
  const int which = chunk >= a.nq;
  const int h0 = (which ? chunk - a.nq : chunk) * HC;
  const int nh = live ? min(HC, a.H[which] - h0) : 0;
  const RopeUnit<BF16, HALVES> un(u, a.pairs);
  const RopeTensor x = a.x[which], y = a.y[which];

  typename RopeUnit<BF16, HALVES>::Raw raw[HC];
#pragma unroll
  for (int j = 0; j < HC; j++)
    if (j < nh) raw[j] = un.load(x.p, m * x.row + (int64_t)(h0 + j) * x.head);
  float c[4], s[4], w[8];
  if (nh > 0) {
    rope_angles(a, t, m, u, c, s);
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
      const float r = 1.f / sqrtf(group_sum<GL>(q) / (float)a.D + a.eps);
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = v[i] * r * w[i];
    }
    if (j < nh) {
      un.rotate(v, c, s);
      un.store(y.p, m * y.row + (int64_t)(h0 + j) * y.head, v);
    }
  }
}

// Gradient of norm and rotation.  A fixed number of workgroups walks over the items; each
// lane sums its channels' dw in fp32 over the items it meets, the workgroup adds its groups in
// LDS, and qk_dw_kernel adds the workgroups: one order, the same result on every run.
template <bool BF16, bool HALVES, int GL, int HC>
__global__ __launch_bounds__(kRopeThreads) void qk_back_kernel(const RopeArgs a, const RopeTable t) {
  constexpr int NG = kRopeThreads / GL;
  __shared__ float red[2][NG * GL * 8];
  const int u = threadIdx.x % GL, g = threadIdx.x / GL;
  const RopeUnit<BF16, HALVES> un(u, a.pairs);
  const bool lane = 8 * u < a.D;
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; i++) dw[0][i] = dw[1][i] = 0.f;
  for (int64_t first = (int64_t)blockIdx.x * NG; first < a.items; first += (int64_t)gridDim.x * NG) {
    const int64_t item = first + g;
    const bool live = item < a.items && lane;
    const int64_t m = live ? item / a.nc : 0;
    const int chunk = live ? (int)(item % a.nc) : 0;
    const int which = chunk >= a.nq;
    const int h0 = (which ? chunk - a.nq : chunk) * HC;
    const int nh = live ? min(HC, a.H[which] - h0) : 0;
    const RopeTensor x = a.x[which], y = a.y[which], dx = a.dx[which];
    typename RopeUnit<BF16, HALVES>::Raw rx[HC], ry[HC];
#pragma unroll
    for (int j = 0; j < HC; j++)
      if (j < nh) {
        rx[j] = un.load(x.p, m * x.row + (int64_t)(h0 + j) * x.head);
        ry[j] = un.load(y.p, m * y.row + (int64_t)(h0 + j) * y.head);
      }
    float c[4], s[4], w[8], acc[8];
#pragma unroll
    for (int i = 0; i < 8; i++) w[i] = acc[i] = 0.f;
    if (nh > 0) {
      rope_angles(a, t, m, u, c, s);
      rope_weights<BF16, HALVES>(un, a.w[which], w);
    }
#pragma unroll
    for (int j = 0; j < HC; j++) {
      float v[8], d[8];
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = d[i] = 0.f;
      if (j < nh) {
        RopeUnit<BF16, HALVES>::unpack(rx[j], v);
        RopeUnit<BF16, HALVES>::unpack(ry[j], d);
        un.rotate(d, c, s);
      }
      float q = 0.f, p = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        q += v[i] * v[i];
        p += d[i] * w[i] * v[i];
      }
      const float r = 1.f / sqrtf(group_sum<GL>(q) / (float)a.D + a.eps);
      // x r^3 / D sum(w t x) as (x r) (r (sum(w t x) r / D))
      const float k = r * (group_sum<GL>(p) * r / (float)a.D);
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const float n = v[i] * r;
        acc[i] += d[i] * n;
        v[i] = r * (d[i] * w[i]) - n * k;
      }
      if (j < nh) un.store(dx.p, m * dx.row + (int64_t)(h0 + j) * dx.head, v);
    }
#pragma unroll
    for (int i = 0; i < 8; i++) dw[which][i] += acc[i];
  }
#pragma unroll
  for (int k = 0; k < 2; k++)
#pragma unroll
    for (int i = 0; i < 8; i++) red[k][(g * GL + u) * 8 + i] = dw[k][i];
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * GL * 8; e += kRopeThreads) {
    const int k = e / (GL * 8), at = e % (GL * 8);
    float sum = 0.f;
    for (int j = 0; j < NG; j++) sum += red[k][j * GL * 8 + at];
    const RopeUnit<BF16, HALVES> ue(at / 8, a.pairs);
    const int i = at % 8, ch = i < 4 ? ue.lo + i : ue.hi + i - 4;
    if (at < a.D) a.part[((int64_t)blockIdx.x * 2 + k) * a.D + ch] = sum;
  }
}

// dw[k][ch] = sum over workgroups of part[.][k][ch], in double precision.
__global__ __launch_bounds__(256) void qk_dw_kernel(const float* part, int blocks, int D, float* dqw, float* dkw) {
  __shared__ double red[256];
  const int col = blockIdx.x * 16 + threadIdx.x % 16, lane = threadIdx.x / 16;
  double sum = 0.0;
  if (col < 2 * D)
    for (int b = lane; b < blocks; b += 16) sum += (double)part[(int64_t)b * 2 * D + col];
  red[threadIdx.x] = sum;
  __syncthreads();
  if (lane == 0 && col < 2 * D) {
    for (int j = 1; j < 16; j++) sum += red[j * 16 + threadIdx.x];
    float* out = col < D ? dqw : dkw;
    if (out != nullptr) out[col < D ? col : col - D] = (float)sum;
  }
}

namespace {

// Workgroups of the gradient kernel: enough to fill the chip, few enough that the sum over
// them stays small against the pass itself.
constexpr int64_t kQkBackBlocks = 1024;

int rope_heads(int64_t M, int64_t H, int gl) {
  // Heads per group: eight where the lanes still fill the chip (256 CUs of 2048), else fewer, so
  // that a short call spreads over more CUs.
  for (int hc : {8, 4, 2})
    if (M * ((H + hc - 1) / hc) * gl >= (int64_t)256 * 2048) return hc;
  return 1;
}

void rope_fill(const RopeCall& c, int hc, RopeArgs& a, RopeTable& t) {
  a = RopeArgs{};
  a.M = c.M;
  a.H[0] = (int)c.H[0];
  a.H[1] = (int)c.H[1];
  a.nq = (a.H[0] + hc - 1) / hc;
  a.nc = a.nq + (a.H[1] + hc - 1) / hc;
  a.items = c.M * a.nc;
  a.D = (int)c.D;
  a.axes = c.axes;
  a.eps = c.eps;
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
      t.f[p] = f;
      t.axis[p] = (uint8_t)ax;
    }
  }
  a.pairs = p;
  a.sign = c.inverse ? -1.f : 1.f;
}

template <bool BF16, bool HALVES, bool NORM, int GL>
void rope_launch(const RopeCall& c, hipStream_t stream) {
  RopeArgs a;
  RopeTable t;
  const int hc = rope_heads(c.M, c.H[0] + c.H[1], GL);
  rope_fill(c, hc, a, t);
  const dim3 grid((unsigned)((a.items + kRopeThreads / GL - 1) / (kRopeThreads / GL))), block(kRopeThreads);
  if (hc == 8) hipLaunchKernelGGL((rope_kernel<BF16, HALVES, NORM, GL, 8>), grid, block, 0, stream, a, t);
  else if (hc == 4) hipLaunchKernelGGL((rope_kernel<BF16, HALVES, NORM, GL, 4>), grid, block, 0, stream, a, t);
  else if (hc == 2) hipLaunchKernelGGL((rope_kernel<BF16, HALVES, NORM, GL, 2>), grid, block, 0, stream, a, t);
  else hipLaunchKernelGGL((rope_kernel<BF16, HALVES, NORM, GL, 1>), grid, block, 0, stream, a, t);
}

template <bool BF16, bool HALVES, int GL>
void qk_back_launch(const RopeCall& c, float* part, int64_t blocks, hipStream_t stream) {
  RopeArgs a;
  RopeTable t;
  const int hc = rope_heads(c.M, c.H[0] + c.H[1], GL) >= 4 ? 4 : 1;
  rope_fill(c, hc, a, t);
  a.part = part;
  const dim3 grid((unsigned)blocks), block(kRopeThreads);
  if (hc == 4) hipLaunchKernelGGL((qk_back_kernel<BF16, HALVES, GL, 4>), grid, block, 0, stream, a, t);
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

int64_t qk_back_blocks(const RopeCall& c) {
  int64_t gl = 4;
  while (8 * gl < c.D) gl *= 2;
  const int64_t groups = c.M * (c.H[0] + c.H[1]), per = kRopeThreads / gl;
  return std::min(kQkBackBlocks, (groups + per - 1) / per);
}

}  // namespace

size_t qk_back_workspace(int64_t D) { return (size_t)kQkBackBlocks * 2 * D * 4; }

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
  const int64_t blocks = qk_back_blocks(c);
  float* part = (float*)ws;
  const bool halves = c.halves, bf16 = c.dt == kDtBF16;
  rope_lanes(c.D, [&](auto gl) {
    constexpr int GL = decltype(gl)::value;
    if (bf16 && halves) qk_back_launch<true, true, GL>(c, part, blocks, stream);
    else if (bf16) qk_back_launch<true, false, GL>(c, part, blocks, stream);
    else if (halves) qk_back_launch<false, true, GL>(c, part, blocks, stream);
    else qk_back_launch<false, false, GL>(c, part, blocks, stream);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || (dqw == nullptr && dkw == nullptr)) return e;
  hipLaunchKernelGGL(qk_dw_kernel, dim3((unsigned)((2 * c.D + 15) / 16)), dim3(256), 0, stream, part, (int)blocks,
                     (int)c.D, dqw, dkw);
  return hipGetLastError();
}

}  // namespace rtl
