// ring_gemm.h -- the bf16 matrix product of the gated block: C[r, c] = sum_k A[r, k] B[c, k],
// with either operand stored with k along its rows or along its columns (so that the
// gradients' products need no transposed copies), on output tiles of four waves.
//
// K runs in steps of 64.  A step's A tile and its B tile are items of a ring of 2 d + 1 LDS slots
// (d = 2, or 4 where a CU has one small tile only), filled with 16-byte loads that go straight to
// LDS.  All through step s a wave reads the fragments it needs next, B_s two blocks ahead and all
// of A_{s+1} into the other set of registers, and issues the loads of A_{s+d} (into B_{s-1}'s slot)
// and B_{s+d} (into A_s's, read in step s - 1).  Behind the next to last column block, when its
// last read of the step has returned, it waits for its loads of A_{s+2} and B_{s+1} and meets the
// others at the step's one barrier; the last block's products then cover the first reads of
// B_{s+1}.
//
// Bound: the vector-memory path.  Rows are loaded in whole 128-byte lines: half lines double
// the requests to L2, which then take longer than the products (7.4 against 5.4 ms without
// loads, 32760 x 27648 x 5120).  A 256 x 256 tile of four 128 x 128 waves moves 64 KB in and 128
// KB of fragments out of LDS a step, against 2048 cycles of matrix instructions.
#pragma once
#include "gemm_common.h"

namespace rtl {

constexpr int kRK = 64;      // K per ring step
// LDS slots at d steps ahead.  Five slots of 256 x 256 tiles take all 160 KB, two 128 x 128 tiles'
// likewise; nine of a 128 x 128 tile 144 KB.
constexpr int ring_slots(int d) { return 2 * d + 1; }
constexpr int kRingWaves = 4;

// Operand with k along its rows: element (r, k) at p[r * ld + k].  A tile holds ROWS rows of 128
// bytes, chunks swizzled by the row (sw_off).
template <int ROWS>
struct KRows {
  static constexpr int kBytes = ROWS * 128, kLoads = ROWS / 8 / kRingWaves;
  uint32_t voff, rd[2];
  int wave;
  int64_t ld;
  // The eight rows of a load lie `step` rows apart.
  __device__ __forceinline__ KRows(int64_t ld_, int step, int wave_, int lane) : wave(wave_), ld(ld_) {
    const int row = lane >> 3, r16 = lane & 15, q = lane >> 4;
    voff = (uint32_t)(row * step * ld * 2 + (((lane & 7) ^ row) << 4));
    rd[0] = sw_off(r16, q);
    rd[1] = sw_off(r16, 4 + q);
  }
  // Load i of a step from `res`, whose first row is `row` and first k `koff` / 2, into the tile at `dst`.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t res, uint8_t* dst, int i, int64_t row, int koff) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        res, (__attribute__((address_space(3))) void*)(dst + (i * kRingWaves + wave) * 1024), 16, voff,
        (int)(row * ld * 2) + koff, 0, 0);
  }
  // A step's tile of consecutive rows.
  struct Tile {
    const KRows& op;
    __amdgpu_buffer_rsrc_t res;
    int koff;
    __device__ __forceinline__ void load(uint8_t* dst, int i) const {
      op.load(res, dst, i, 8 * (i * kRingWaves + op.wave), koff);
    }
  };
  // Fragment of 16-row block `blk`, K half kk: lane (r16, q) holds row r16, k = 32 kk + 8q .. + 7.
  __device__ __forceinline__ u32x4 read(const uint8_t* tile, int blk, int kk) const {
    return *reinterpret_cast<const u32x4*>(tile + blk * 2048 + rd[kk]);
  }
};

// Operand with k along its columns: element (c, k) at p[k * ld + c].  A tile holds two halves of
// 32 rows (k) of COLS columns; a fragment read takes, per 16 lanes, four rows of one 32-byte
// block of 16 columns and hands lane i column i of the four (the transposing LDS read).  Rows
// k = j + 4c + 8b + 16d (bits j: 2, c, b, d) that one half-wave reads together differ in w = j +
// 4b; the row's 32-byte blocks are swizzled by w, so those eight rows fall in different banks,
// and the rows of one w lie together, so that a load's lanes all share one swizzle.
template <int COLS>
struct KCols {
  static_assert(COLS == 256 || COLS == 128, "a load covers two rows, or four");
  static constexpr int kBytes = COLS * 128, kLoads = COLS / 8 / kRingWaves;
  uint32_t voff[2], rd;
  int wave;
  int64_t ld;
  __device__ __forceinline__ KCols(int64_t ld_, int wave_, int lane) : wave(wave_), ld(ld_) {
    constexpr int CPR = COLS / 8;  // 16-byte chunks of a row
    const int sub = lane / CPR, p = lane % CPR, c = sub & 1, d = sub >> 1;
#pragma unroll
    for (int b = 0; b < 2; b++)
      voff[b] = (uint32_t)((wave + 4 * c + 8 * b + 16 * d) * ld * 2 + ((((p >> 1) ^ (wave + 4 * b)) << 1) | (p & 1)) * 16);
    const int j = (lane & 15) >> 2, q = lane >> 4, w = j + 4 * (q & 1), dq = q >> 1;
    rd = (uint32_t)((COLS == 256 ? (dq * 8 + w) * 1024 : w * 1024 + dq * 512) + (w << 5) + (lane & 3) * 8);
  }
  // Load i of a step: the buffer starts at the step's first row; two (COLS == 256) or four rows
  // of 16 (32), pairs of loads by b.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t res, uint8_t* dst, int i) const {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        res, (__attribute__((address_space(3))) void*)(dst + (i * kRingWaves + wave) * 1024), 16, voff[i & 1],
        (int)((i >> 1) * (COLS == 256 ? 16 : 32) * ld * 2), 0, 0);
  }
  struct Tile {
    const KCols& op;
    __amdgpu_buffer_rsrc_t res;
    __device__ __forceinline__ void load(uint8_t* dst, int i) const { op.load(res, dst, i); }
  };
  __device__ __forceinline__ u32x4 read(const uint8_t* tile, int blk, int kk) const {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    // blocks 0..7 of a row by the swizzle, 8..15 256 bytes on; the second four k (c = 1) one row on
    const uint8_t* at = tile + kk * (kBytes / 2) + (rd ^ (uint32_t)((blk & 7) << 5)) + (blk >> 3) * 256;
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
        (__attribute__((address_space(3))) bf16x4*)at));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
        (__attribute__((address_space(3))) bf16x4*)(at + COLS * 2)));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
};

// acc += A B^T on one 16 x 16 block, K = 32.  The sum stays in its accumulation registers: in
// the compiler's form of the instruction it may land in others, and with 64 blocks, which fill
// all 256, two register moves then go with every product.  Before settle() nothing but the next
// product on the same block touches an accumulator, RB products further on (two at least).  That
// one needs no distance: the hardware holds it back until exactly these registers are written (the
// compiler, too, puts its own products on one accumulator next to each other).  The compiler sees no
// matrix instruction here and keeps no wait states for it: tests/test_matrix_operands.py holds the
// compiled kernels to them.
__device__ __forceinline__ void mfma_acc(f32x4& acc, u32x4 a, u32x4 b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// acc = 0, as a product of zeros: of plain zeros the compiler makes one register and copies it.
__device__ __forceinline__ void mfma_zero(f32x4& acc) {
  const u32x4 z{};
  asm volatile("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %1, 0" : "=a"(acc) : "v"(z));
}
// Waits until the products of mfma_acc on a row of blocks are written (the compiler does not see
// them): the accumulators pass through a statement that idles longer than the instruction takes.
// Called where the row is used: as one statement for all rows it has the compiler copy all of
// them to general registers at once.
template <int NB>
__device__ __forceinline__ void settle(f32x4 (&acc)[NB]) {
#pragma unroll
  for (int nb = 0; nb < NB; nb += 4)
    asm volatile("s_nop 15\n\ts_nop 15" : "+a"(acc[nb]), "+a"(acc[nb + 1]), "+a"(acc[nb + 2]), "+a"(acc[nb + 3]));
}

// Waits until at most N of the wave's loads are in flight and all its LDS reads have returned.
template <int N>
__device__ __forceinline__ void wait_ring() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (0 << 8) | ((N >> 4) << 14));
}

template <int RB>
struct ARegs {
  u32x4 v[2][RB];
};

// One ring step of a wave's RB x NB blocks of 16 x 16.  tb, ta1, tb1: the tiles of B_s, A_{s+1},
// B_{s+1}; da, db: where sa.load(da, i) puts load i of A_{s+d} and sb.load(db, i) of B_{s+d}.  The five slots are distinct (__restrict__ says so: without it the compiler has every
// transposing read wait for every load in flight).
template <int DEPTH, int RB, int NB, typename OpA, typename OpB, typename SrcA, typename SrcB>
__device__ __forceinline__ void ring_step(f32x4 (&acc)[RB][NB], const uint8_t* __restrict__ tb,
                                          const uint8_t* __restrict__ ta1, const uint8_t* __restrict__ tb1,
                                          uint8_t* __restrict__ da, uint8_t* __restrict__ db, const OpA& oa,
                                          const OpB& ob, const SrcA& sa, const SrcB& sb, const ARegs<RB>& cur, ARegs<RB>& next,
                                          u32x4 (&bv)[4][2], int wm, int wn) {
  constexpr int LA = OpA::kLoads, LD = LA + OpB::kLoads;
  static_assert(NB % 4 == 0 && 3 * (NB - 1) >= LD && 3 * (NB - 1) >= 2 * RB, "three reads and loads a block suffice");
#pragma unroll
  for (int nb = 0; nb < NB; nb++) {
    if (nb == NB - 1) {
      wait_ring<OpB::kLoads + (DEPTH - 2) * LD>();  // in flight: B_{s+2}, and A and B of s + 3 .. s + d
      barrier_nofence();
    }
#pragma unroll
    for (int p = 0; p < 2 * RB; p++) {
      mfma_acc(acc[p % RB][nb], cur.v[p / RB][p % RB], bv[nb % 4][p / RB]);
      // what else the block does, a little behind each product: a lone wave's pipe runs empty
      // where several other instructions follow one another (the last product takes what is left)
      constexpr int A0 = 2, L0 = 2 + RB / 4, D = RB >= 4 ? RB / 2 : 1;
      if (nb + 2 < NB && p < 2) bv[(nb + 2) % 4][p] = ob.read(tb, NB * wn + nb + 2, p);
      if (nb == NB - 1 && p < 4) bv[p / 2][p % 2] = ob.read(tb1, NB * wn + p / 2, p % 2);
#pragma unroll
      for (int t = 0; t < 3; t++) {
        const int i = 3 * nb + t;
        if (nb < NB - 1 && p == min(A0 + t * D, 2 * RB - 1) && i < 2 * RB) next.v[i / RB][i % RB] = oa.read(ta1, RB * wm + i % RB, i / RB);
        if (nb < NB - 1 && p == min(L0 + t * D, 2 * RB - 1) && i < LD) {
          if (i < LA) sa.load(da, i);
          else sb.load(db, i - LA);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The product over `steps` K steps.  at_a(kt) and at_b(kt) give the source of step kt's tile, whose
// load(dst, i) issues its load i; past the end (kt = -1) the loads read zeros.  The caller settles
// each row of blocks before it reads it.  (Tiles that start at different steps and go round, so
// that one of those that share an operand takes each L2 miss, measured 2% slower.)
template <int DEPTH, int RB, int NB, typename OpA, typename OpB, typename AtA, typename AtB>
__device__ __forceinline__ void ring_product(f32x4 (&acc)[RB][NB], uint8_t* lds, const OpA& oa, const OpB& ob,
                                             AtA at_a, AtB at_b, int steps, int wm, int wn) {
  static_assert(OpB::kBytes <= OpA::kBytes, "either operand's tile fits every slot");
  constexpr int SLOT = OpA::kBytes, LA = OpA::kLoads, LB = OpB::kLoads, RING = ring_slots(DEPTH) * SLOT;
  auto step_or_none = [&](int s) { return s < steps ? s : -1; };
#pragma unroll
  for (int rb = 0; rb < RB; rb++)
#pragma unroll
    for (int nb = 0; nb < NB; nb++) mfma_zero(acc[rb][nb]);
  // A_0, B_0, A_1, B_1, .. into slots 0, 1, 2, 3, ..
#pragma unroll
  for (int s = 0; s < DEPTH; s++) {
    const auto sa = at_a(step_or_none(s));
    const auto sb = at_b(step_or_none(s));
#pragma unroll
    for (int i = 0; i < LA; i++) sa.load(lds + 2 * s * SLOT, i);
#pragma unroll
    for (int i = 0; i < LB; i++) sb.load(lds + (2 * s + 1) * SLOT, i);
  }
  wait_vmcnt<LB + (DEPTH - 2) * (LA + LB)>();  // A_0, B_0, A_1 have arrived
  barrier_nofence();
  ARegs<RB> av[2];
  u32x4 bv[4][2];
#pragma unroll
  for (int kk = 0; kk < 2; kk++) {
#pragma unroll
    for (int rb = 0; rb < RB; rb++) av[0].v[kk][rb] = oa.read(lds, RB * wm + rb, kk);
#pragma unroll
    for (int nb = 0; nb < 2; nb++) bv[nb][kk] = ob.read(lds + SLOT, NB * wn + nb, kk);
  }
  wait_ring<63>();  // the reads: A_0's slot is free
  barrier_nofence();
  // Slots of B_{s+d} (A_s's), B_s, A_{s+1}, B_{s+1}, A_{s+d} (B_{s-1}'s); two on with every step.
  int o0 = 0, o1 = SLOT, o2 = 2 * SLOT, o3 = 3 * SLOT, o4 = 2 * DEPTH * SLOT;
  auto on = [&](int o) { return o + 2 * SLOT >= RING ? o + 2 * SLOT - RING : o + 2 * SLOT; };
  auto step = [&](int s, const ARegs<RB>& cur, ARegs<RB>& next) {
    const int kt = step_or_none(s + DEPTH);
    ring_step<DEPTH, RB, NB>(acc, lds + o1, lds + o2, lds + o3, lds + o4, lds + o0, oa, ob, at_a(kt), at_b(kt), cur, next,
                             bv, wm, wn);
    if (DEPTH == 2) {  // the five are the whole ring
      const int t0 = o0, t1 = o1;
      o0 = o2; o1 = o3; o2 = o4; o3 = t0; o4 = t1;
    } else {
      o0 = o2; o1 = o3; o2 = on(o2); o3 = on(o3); o4 = on(o4);
    }
  };
  int s = 0;
  for (; s + 2 <= steps; s += 2) {  // the two sets of A fragments
    step(s, av[0], av[1]);
    step(s + 1, av[1], av[0]);
  }
  if (s < steps) step(s, av[0], av[1]);
  wait_vmcnt<0>();  // no load into the ring is left in flight
}

}  // namespace rtl
