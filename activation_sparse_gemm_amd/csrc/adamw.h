// adamw.h -- the AdamW step over many tensors in few launches, states in 32 or in 8 bits.
//
//   g' = g gs,  m += (1 - b1) (g' - m),  v = b2 v + (1 - b2) g'^2
//   p -= lr ((m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps) + decay p)
//
// In 8 bits a run of kAdamBlock elements shares a scale: m is held as E4M3 codes of m 448 / max|m|, v
// through its root, as codes of sqrt(v) 448 / max sqrt(v), where a root that is not 0 takes the smallest
// code at least: rounded to 0 it would leave the next step to divide m by eps alone.  E4M3 spans 2^17.8,
// the root's square twice that.  The states are formed by single fp32 operations in the order written
// (no contraction), so that a value next to the border of two codes is coded the same wherever it
// is computed so.
//
// Bound: memory (28 bytes an element with 32-bit states, 16 with 8-bit ones; 2 more where bf16 parameters are
// written beside their masters, 2 less where gradients are bf16).  A launch takes up to kAdamTensors tensors, their addresses in
// its arguments, so that nothing is copied to the device first and a captured call holds them.  Measured, bf16 beside
// masters: 320 factors, 176 M elements, 32-bit states, 970 us, 5.1 TB/s (fp32 gradients 1008, 5.2); 212 M elements, 8-bit
// states, 634, 5.4 TB/s.
#pragma once
#include <algorithm>

#include "fp8_common.h"
#include "rtl_launch.h"

namespace rtl {

namespace adam {

constexpr int kAdamThreads = 256;
constexpr int kAdamTensors = 56;  // of 64 bytes: the arguments stay below 4 KB
constexpr int kAdamBlock = 256;   // a wave's four elements a lane
constexpr int kAdamTurns = 4;     // pieces of four elements in flight a thread
constexpr int kAdamChunk = kAdamThreads * 4 * kAdamTurns;

struct AdamArgs {
  AdamTensor t[kAdamTensors];
  uint32_t first[kAdamTensors + 1];  // first workgroup of each tensor
  int count;
  AdamRates r;
};
static_assert(sizeof(AdamArgs) <= 4096, "a launch's arguments");

// Four elements as fp32, or fewer at a tensor's end (`n` of them, the rest 0).
template <bool BF16>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t at, int n) {
  f32x4 v{};
  if (n >= 4) {
    if constexpr (BF16) {
      const u32x2 w = *reinterpret_cast<const u32x2*>((const uint16_t*)p + at);
      v = f32x4{bf16lo(w[0]), bf16hi(w[0]), bf16lo(w[1]), bf16hi(w[1])};
    } else {
      v = *reinterpret_cast<const f32x4*>((const float*)p + at);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 3; i++)
      if (i < n) v[i] = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)p)[at + i] << 16) : ((const float*)p)[at + i];
  }
  return v;
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t at, int n, const f32x4& v) {
  if (n >= 4) {
    if constexpr (BF16) {
      typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
      const u32x2 w = {__builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[0], (__bf16)v[1]}),
                       __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)v[2], (__bf16)v[3]})};
      *reinterpret_cast<u32x2*>((uint16_t*)p + at) = w;
    } else {
      *reinterpret_cast<f32x4*>((float*)p + at) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 3; i++)
      if (i < n) {
        if constexpr (BF16) ((__bf16*)p)[at + i] = (__bf16)v[i];
        else ((float*)p)[at + i] = v[i];
      }
  }
}
__device__ __forceinline__ uint32_t load_codes(const uint8_t* p, int64_t at, int n) {
  if (n >= 4) return *reinterpret_cast<const uint32_t*>(p + at);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 3; i++)
    if (i < n) w |= (uint32_t)p[at + i] << (8 * i);
  return w;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t at, int n, uint32_t w) {
  if (n >= 4) {
    *reinterpret_cast<uint32_t*>(p + at) = w;
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; i++)
    if (i < n) p[at + i] = (uint8_t)(w >> (8 * i));
}
__device__ __forceinline__ f32x4 decode(uint32_t w) {
  return f32x4{__builtin_amdgcn_cvt_f32_fp8((int)w, 0), __builtin_amdgcn_cvt_f32_fp8((int)w, 1),
               __builtin_amdgcn_cvt_f32_fp8((int)w, 2), __builtin_amdgcn_cvt_f32_fp8((int)w, 3)};
}

// Largest of non-negative values over the wave, the same in each lane; a NaN counts as the largest.
template <int CTRL>
__device__ __forceinline__ uint32_t most_lanes(uint32_t v) {
  return umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_most(const f32x4& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) m = umax(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = most_lanes<0xB1>(m);
  m = most_lanes<0x4E>(m);
  m = most_lanes<0x141>(m);
  m = most_lanes<0x140>(m);
  m = umax(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  return __uint_as_float(umax(m, (uint32_t)__shfl_xor((int)m, 32, 64)));
}

// Codes of four values whose block's largest magnitude is `most`.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode(const f32x4& v, float most) {
  const float inverse = fp8_inv_scale(most);
  f32x4 s;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    s[i] = v[i] * inverse;
    if (ROOT) s[i] = v[i] > 0.f ? fmaxf(s[i], 0x1p-9f) : s[i];
  }
  return fp8x4(s[0], s[1], s[2], s[3]);
}

template <bool PBF16, bool GBF16, bool EIGHT>
__global__ __launch_bounds__(kAdamThreads) void adamw_kernel(const AdamArgs a) {
#pragma clang fp contract(off)
  __shared__ float corrections[2];
  int i = 0;
  for (int n = a.count; n > 1;) {  // the tensor of this workgroup
    const int half = n / 2;
    if (a.first[i + half] <= blockIdx.x) {
      i += half;
      n -= half;
    } else {
      n = half;
    }
  }
  const AdamTensor t = a.t[i];
  AdamRates r = a.r;
  if (r.step_at != nullptr) {  // the step's number is on the device: its corrections are formed here
    if (threadIdx.x == 0) {
      const double step = (double)*r.step_at;
      corrections[0] = (float)(1.0 / (1.0 - pow(r.beta1, step)));
      corrections[1] = (float)(1.0 / sqrt(1.0 - pow(r.beta2, step)));
    }
    __syncthreads();
    r.m_up = corrections[0];
    r.u_up = corrections[1];
  }
  const float rate = r.lr_at != nullptr ? *r.lr_at : r.lr;
  const float clip = r.grad_scale != nullptr ? *r.grad_scale : 1.f;
  const int64_t at0 = (int64_t)(blockIdx.x - a.first[i]) * kAdamChunk + threadIdx.x * 4;

  f32x4 p[kAdamTurns], g[kAdamTurns], m[kAdamTurns], v[kAdamTurns];
  uint32_t mc[kAdamTurns], vc[kAdamTurns];
  float ms[kAdamTurns], vs[kAdamTurns];
  int left[kAdamTurns];
#pragma unroll
  for (int k = 0; k < kAdamTurns; k++) {
    const int64_t at = at0 + k * kAdamThreads * 4;
    left[k] = (int)min(max(t.n - at, (int64_t)0), (int64_t)4);
    p[k] = PBF16 ? load4<false>(t.master, at, left[k]) : load4<false>(t.p, at, left[k]);
    g[k] = load4<GBF16>(t.g, at, left[k]);
    if constexpr (EIGHT) {
      const int64_t block = min(at, t.n - 1) / kAdamBlock;  // the wave's
      mc[k] = load_codes((const uint8_t*)t.m, at, left[k]);
      vc[k] = load_codes((const uint8_t*)t.v, at, left[k]);
      ms[k] = t.m_scale[block];
      vs[k] = t.v_scale[block];
    } else {
      m[k] = load4<false>(t.m, at, left[k]);
      v[k] = load4<false>(t.v, at, left[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kAdamTurns; k++) {
    const int64_t at = at0 + k * kAdamThreads * 4;
    f32x4 u;
    if constexpr (EIGHT) {
      m[k] = decode(mc[k]);
      u = decode(vc[k]);
    }
#pragma unroll
    for (int e = 0; e < 4; e++) {
      if constexpr (EIGHT) {
        m[k][e] = m[k][e] * ms[k];
        u[e] = u[e] * vs[k];
        v[k][e] = u[e] * u[e];
      }
      const float gr = r.grad_scale != nullptr ? g[k][e] * clip : g[k][e];
      const float dm = gr - m[k][e], up = dm * r.c1;
      m[k][e] = m[k][e] + up;
      const float gg = gr * gr, keep = v[k][e] * r.b2, add = gg * r.c2;
      v[k][e] = keep + add;
      u[e] = sqrtf(v[k][e]);
      const float den = u[e] * r.u_up + r.eps;
      const float step = m[k][e] * r.m_up / den;
      p[k][e] = p[k][e] - (step + p[k][e] * r.decay) * rate;
    }
    if constexpr (EIGHT) {
      // whole waves: past the end the elements are 0 (a gradient of 0 on states of 0) and store nothing
      const float mm = wave_most(m[k]), mu = wave_most(u);
      if (left[k] > 0) {
        store_codes((uint8_t*)t.m, at, left[k], encode<false>(m[k], mm));
        store_codes((uint8_t*)t.v, at, left[k], encode<true>(u, mu));
        if ((threadIdx.x & 63) == 0) {
          t.m_scale[at / kAdamBlock] = mm / 448.f;
          t.v_scale[at / kAdamBlock] = mu / 448.f;
        }
      }
    } else {
      store4<false>(t.m, at, left[k], m[k]);
      store4<false>(t.v, at, left[k], v[k]);
    }
    if constexpr (PBF16) {
      store4<false>(t.master, at, left[k], p[k]);
      store4<true>(t.p, at, left[k], p[k]);
    } else {
      store4<false>(t.p, at, left[k], p[k]);
    }
  }
}

template <bool PBF16, bool GBF16, bool EIGHT>
hipError_t adamw_launch(const AdamTensor* t, int64_t count, const AdamRates& r, hipStream_t stream) {
  AdamArgs a;
  a.r = r;
  a.count = 0;
  uint32_t blocks = 0;
  auto go = [&]() {
    if (a.count == 0) return hipSuccess;
    a.first[a.count] = blocks;
    hipLaunchKernelGGL((adamw_kernel<PBF16, GBF16, EIGHT>), dim3(blocks), dim3(kAdamThreads), 0, stream, a);
    a.count = 0;
    blocks = 0;
    return hipGetLastError();
  };
  for (int64_t i = 0; i < count; i++) {
    if (t[i].n == 0) continue;
    const uint32_t need = (uint32_t)((t[i].n + kAdamChunk - 1) / kAdamChunk);
    if (a.count == kAdamTensors || blocks + need > kAdamMaxBlocks) {
      const hipError_t e = go();
      if (e != hipSuccess) return e;
    }
    a.t[a.count] = t[i];
    a.first[a.count++] = blocks;
    blocks += need;
  }
  return go();
}

}  // namespace adam

hipError_t launch_adamw(bool p_bf16, bool g_bf16, bool eight, const AdamTensor* t, int64_t count, const AdamRates& r,
                        hipStream_t stream) {
  using namespace adam;
  static_assert(kAdamMaxN <= (int64_t)kAdamMaxBlocks * kAdamChunk, "a tensor fits one launch");
  if (p_bf16)
    return g_bf16 ? (eight ? adamw_launch<true, true, true>(t, count, r, stream) : adamw_launch<true, true, false>(t, count, r, stream))
                  : (eight ? adamw_launch<true, false, true>(t, count, r, stream) : adamw_launch<true, false, false>(t, count, r, stream));
  return g_bf16 ? (eight ? adamw_launch<false, true, true>(t, count, r, stream) : adamw_launch<false, true, false>(t, count, r, stream))
                : (eight ? adamw_launch<false, false, true>(t, count, r, stream) : adamw_launch<false, false, false>(t, count, r, stream));
}

}  // namespace rtl
