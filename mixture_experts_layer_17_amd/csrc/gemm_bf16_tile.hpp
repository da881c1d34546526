// Tiles of the bf16 matrix products (internal): configurations, and the moves of
// an operand from global memory through LDS into MFMA fragments, for operands
// contiguous along the contraction or along their rows or columns.
#pragma once

#include "gemm_common.hpp"

namespace moe {
namespace gemm {

// Tile configuration: BM x BN outputs, WM x WN waves, K-step BK, LDS ring of
// NA stages for the A tile and NB stages for the B tile (equal, or 3 and 2).
template <int BM_, int BN_, int WM_, int WN_, int BK_, int NA_, int NB_, int SPREAD_, bool REGEPI_>
struct Cfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, BK = BK_, NA = NA_, NB = NB_;
  // equal rings: 0 issues a K-step's loads right after the barrier; 1 spreads
  // them over the step's first two 16-deep MFMA slices (A, then B); 2 over all four
  static constexpr int kSpread = SPREAD_;
  // epilogue: straight from registers (tiles computed transposed, the next
  // tile's first steps in flight meanwhile), or staged through LDS as bf16 for
  // 16-byte streaming stores of whole rows (the two-workgroup-per-CU tiles,
  // where the other workgroup's main loop overlaps it)
  static constexpr bool kRegEpi = REGEPI_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int WTM = BM / WM, WTN = BN / WN;
  static constexpr int TM = WTM / 32, TN = WTN / 32;
  static constexpr int kA = BM * BK, kB = BN * BK;  // elements per stage
  static constexpr int kBOff = NA * kA;              // the B ring follows the A ring
  // resident waves per SIMD the register allocation must allow: two
  // workgroups per compute unit for the 128-row tiles, one for 256 x 256
  static constexpr int kWavesPerSimd = (BM == 128 ? 2 : 1) * kWaves / 4;
  // LDS-staged epilogue tiles: G1 two BM x (BN/2 + 8), the others BM x (BN + 8)
  static constexpr int kEpi = REGEPI_ ? 0 : cmax(2 * BM * (BN / 2 + 8), BM * (BN + 8));
  static constexpr int kLds = cmax(NA * kA + NB * kB, kEpi);  // elements (bf16)
  static_assert(BK == 32 || BK == 64, "K step");
  static_assert(NA >= 2 && NB >= 2 && (NA == NB ? NA <= 5 : NA + NB == 5), "LDS ring depths: equal, or 3 and 2");
  static_assert(kLds * 2 <= 160 * 1024, "LDS budget");
  static_assert(SPREAD_ == 0 || (NA == NB && BK / 16 >= 2 * SPREAD_), "spread loads need equal rings and the slices");
};
// 256 x 256, 8 waves of 128 x 64, K step 64, two stages per operand, each
// step's loads issued over the first two MFMA slices
using Big = Cfg<256, 256, 2, 4, 64, 2, 2, 1, true>;
// 128 x 128, 4 waves of 64 x 64, K step 64, three A stages (two workgroups per CU)
using Small = Cfg<128, 128, 2, 2, 64, 3, 2, 0, false>;
// 128 x 256, 8 waves of 64 x 64, K step 32: two workgroups per CU (short segments, forward GEMMs)
using Mid = Cfg<128, 256, 2, 4, 32, 3, 2, 0, false>;

// K-contiguous operand: element (mn, k) at m0[mn*ld + k] for k < ksplit, else
// m1[mn*ld + k - ksplit]; rows mn >= mn_valid read as zero.
struct KcOp {
  const uint16_t* m0;
  const uint16_t* m1;
  int64_t ld;
  int ksplit;
  int mn_valid;
};

// M/N-contiguous operand: element (mn, k) at m0[k*ld + c0 + mn]; k >= k_valid
// reads as zero.  Dual: tile columns [0, W/2) come from m0 and [W/2, W) from
// m1, both at column c0 + (mn mod W/2).
struct McOp {
  const uint16_t* m0;
  const uint16_t* m1;
  int64_t ld;
  int c0;
  int k_valid;
};

// 16-byte chunk swizzles.  K-contiguous tile rows hold BK elements; a fragment
// read has 16 lanes on 16 consecutive rows at one chunk.  M/N-contiguous tile
// rows (one k each) hold RS elements; a transposing read has 32 lanes on 4
// consecutive k-rows x 4 consecutive chunks.
template <int BK>
__device__ __forceinline__ int kc_swz(int row) {
  return BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3;
}
template <int RS>
__device__ __forceinline__ int mc_swz(int k) {
  static_assert(RS >= 64, "M/N-contiguous tile rows of at least 64 elements");
  return RS >= 128 ? 4 * (k & 3) : 4 * ((k >> 1) & 1);
}

// Issue the LDS-DMA loads of a ROWS x BK K-contiguous tile (K-step at k0).
// Loads u in [U0, U1) of this wave's share (U1 < 0: all).
template <class C, int ROWS, int U0 = 0, int U1 = -1>
__device__ __forceinline__ void dma_kc(const KcOp& op, int k0, uint16_t* dst, int wave, int lane) {
  constexpr int CPR = C::BK / 8;          // chunks per row
  constexpr int RPI = 64 / CPR;           // rows per instruction (1 KB)
  constexpr int NI = ROWS / RPI;
  static_assert(NI % C::kWaves == 0, "K-contiguous tile does not split over the waves");
  const bool hi = k0 >= op.ksplit;
  const uint16_t* m = hi ? op.m1 : op.m0;
  const int kk = hi ? k0 - op.ksplit : k0;
  const int rows = op.mn_valid < ROWS ? op.mn_valid : ROWS;
  const __amdgpu_buffer_rsrc_t r = rsrc(m, static_cast<int64_t>(rows) * op.ld * 2);
  const int rl = lane / CPR, ph = lane % CPR;
  constexpr int UE = U1 < 0 ? NI / C::kWaves : U1;
#pragma unroll
  for (int u = U0; u < UE; ++u) {
    const int i = wave + u * C::kWaves;
    const int row = i * RPI + rl;
    const int lc = ph ^ kc_swz<C::BK>(row);
    dma16(r, dst + i * 512, static_cast<int>((row * op.ld + kk + lc * 8) * 2));
  }
}

// Issue the LDS-DMA loads of a BK x ROWS M/N-contiguous tile, as NSUB
// sub-tiles of BK x ROWS/NSUB (dual: one per matrix).
template <class C, int ROWS, int NSUB, int U0 = 0, int U1 = -1>
__device__ __forceinline__ void dma_mc(const McOp& op, int k0, uint16_t* dst, int wave, int lane) {
  constexpr int RS = ROWS / NSUB;
  constexpr int CPR = RS / 8;             // chunks per k-row
  constexpr int KPI = 64 / CPR;           // k-rows per instruction (1 KB)
  constexpr int NIS = C::BK / KPI;        // instructions per sub-tile
  constexpr int NI = NIS * NSUB;
  static_assert(KPI >= 1 && C::BK % KPI == 0 && NI % C::kWaves == 0, "M/N-contiguous tile split");
  int kv = op.k_valid - k0;
  kv = kv < 0 ? 0 : (kv > C::BK ? C::BK : kv);
  const int kl = lane / CPR, ph = lane % CPR;
  constexpr int UE = U1 < 0 ? NI / C::kWaves : U1;
#pragma unroll
  for (int u = U0; u < UE; ++u) {
    const int i = wave + u * C::kWaves;
    const int sub = i / NIS, ii = i % NIS;
    const uint16_t* m = (NSUB == 2 && sub == 1 ? op.m1 : op.m0) + k0 * op.ld;
    const __amdgpu_buffer_rsrc_t r = rsrc(m, static_cast<int64_t>(kv) * op.ld * 2);
    const int kr = ii * KPI + kl;
    const int lc = ph ^ mc_swz<RS>(kr);
    dma16(r, dst + sub * (C::BK * RS) + ii * 512, static_cast<int>((kr * op.ld + op.c0 + lc * 8) * 2));
  }
}

// MFMA fragment from a K-contiguous tile: rows base .. base+31, k-slice ks.
template <class C>
__device__ __forceinline__ bf16x8 frag_kc(const uint16_t* t, int base, int ks, int lane) {
  const int row = base + (lane & 31);
  const int ph = (ks * 2 + (lane >> 5)) ^ kc_swz<C::BK>(row);
  return *reinterpret_cast<const bf16x8*>(t + row * C::BK + ph * 8);
}

// MFMA fragment from an M/N-contiguous (sub-)tile of RS columns: columns
// col .. col+31, k-slice ks.  Two transposing reads: within each 16-lane
// group G, lane i gets slot s from element i%4 of the address of lane 4s + i/4;
// lane L points at k-row 16 ks + 8(G/2) + 4 half + L/4, columns col + 16(G%2) + 4(L%4).
template <class C, int RS>
__device__ __forceinline__ bf16x8 frag_mc(const uint16_t* t, int col, int ks, int lane) {
  const int G = lane >> 4, L = lane & 15;
  const int k = ks * 16 + 8 * (G >> 1) + (L >> 2);
  const int c = col + 16 * (G & 1) + 4 * (L & 3);
  const int ph = (c >> 3) ^ mc_swz<RS>(k);  // same swizzle for k + 4
  const uint16_t* p = t + k * RS + ph * 8 + (c & 7);
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * RS));
  bf16x8 r;
  short tmp[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  __builtin_memcpy(&r, tmp, 16);
  return r;
}

}  // namespace gemm
}  // namespace moe
