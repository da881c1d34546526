// Orthogonalising a stack of matrices by Newton-Schulz products, and the Muon
// step around it (momentum before, weight write after).
//
//   X_0 = U / (|U|_F + eps);   per step:  A = X X^T (the shorter side),
//   B = b A + c A A,  X <- a X + B X          (X <- a X + X B for tall X)
//
// Matrix products on fp16 MFMA (v_mfma_f32_32x32x16_f16, fp32 accumulate):
// three launches per step (Gram, polynomial, apply), each over the tiles of all
// matrices.  A and B are symmetric: only tiles on and below the diagonal are
// computed, the others are written as their mirror images.
//
// Why fp16 and not bf16: the iterates are bounded (singular values stay near or
// below 1), so a power-of-two scale keeps them inside fp16's range and its three
// extra mantissa bits cost nothing.  Rounding X itself would still hurt: small
// singular values grow by a factor of a (3.44) per step, and with them the
// rounding noise outside the matrix's own range (a gradient's rank is at most
// its token count).  So X is held as an fp16 pair hi + lo.  bf16 gradients: the
// products use hi only (their error stays inside X's range, where it does not
// grow), the a X term uses both, but in the last step.  The diagonals of A and B,
// which outweigh the other entries, are kept apart in fp32 and applied in the
// epilogues.  Against fp64 the result is off by 0.08-0.15% (rms, before its
// rounding; rank 1 to full rank, 64 to 8200 rows), less than its rounding to bf16
// (0.17%).  fp32 gradients
// need the products too at fp32 accuracy: X, A and B are pairs and every
// product is hi hi + hi lo + lo hi (22 bits; lo lo is below fp32's last bit).
//
// Scaling: X, A and B are stored times kS = 2^12.  A matrix's own scale is kept
// apart: X = c_i Xs with c_0 = 2^-q / (|U|_F + eps) and Xs_0 = 2^q U (a bf16
// gradient then enters exactly), c_i growing towards 1 (and 1 from then on), so
// that a matrix whose norm is far below eps keeps its accuracy too.
#include <math.h>

#include <type_traits>

#include "gemm_common.hpp"

namespace moe {
namespace {
using gemm::dma16;
using gemm::f32x16;
using gemm::i16x4;
using gemm::lds_get16;
using gemm::lds_put16;
using gemm::lds_void;
using gemm::rsrc;
using gemm::to_chunks;
using gemm::wait_vm;

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float kS = 4096.0f;
constexpr int kPad = 64;         // rows and columns of the fp16 buffers are padded with zeros to this
constexpr int kMaxSteps = 16;
constexpr int kMaxDim = 32768;
constexpr int kNormThreads = 256;
constexpr int kMaxChunks = 256;  // norm partials per matrix

enum { kGram = 0, kPoly = 1, kApply = 2 };
enum { kOutX = 0, kOutO = 1, kOutW = 2 };  // apply: next X, the result, or the updated weight

// ---------------------------------------------------------------------------
// fp16 pairs
// ---------------------------------------------------------------------------
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
  f16x8 h, l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = static_cast<_Float16>(v[i]);
    l[i] = static_cast<_Float16>(v[i] - static_cast<float>(h[i]));
  }
  hi = __builtin_bit_cast(uint4, h);
  lo = __builtin_bit_cast(uint4, l);
}

// The same with lo in 8 bits: E4M3, times a power of two `scale` that takes the
// largest possible lo (2^-11 of a value, see make_plan) to at most 448.
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ void split8_fp8(const float* v, float scale, uint4& hi, uint2& lo) {
  f16x8 h;
  float l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = static_cast<_Float16>(v[i]);
    l[i] = (v[i] - static_cast<float>(h[i])) * scale;
  }
  hi = __builtin_bit_cast(uint4, h);
  int a = 0, b = 0;
  a = __builtin_amdgcn_cvt_pk_fp8_f32(l[0], l[1], a, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(l[2], l[3], a, true);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(l[4], l[5], b, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(l[6], l[7], b, true);
  lo = make_uint2(static_cast<uint32_t>(a), static_cast<uint32_t>(b));
}
__device__ __forceinline__ void lo_fp8(const uint2& u, float* l) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int w = static_cast<int>(i ? u.y : u.x);
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    l[4 * i] = a[0];
    l[4 * i + 1] = a[1];
    l[4 * i + 2] = b[0];
    l[4 * i + 3] = b[1];
  }
}

// Up to 8 elements at p (element alignment) as floats, and back.
template <class T>
__device__ __forceinline__ void ld8(const T* p, int n, float* o) {
  constexpr int V = Elem<T>::kVec;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < 8; i += V) {
      uint4 v;
      __builtin_memcpy(&v, p + i, 16);
      Elem<T>::unpack(v, o + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = i < n ? Elem<T>::load1(p, i) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void st8(T* p, int n, const float* v) {
  constexpr int V = Elem<T>::kVec;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < 8; i += V) {
      const uint4 u = Elem<T>::pack(v + i);
      __builtin_memcpy(p + i, &u, 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) Elem<T>::store1(p, i, v[i]);
  }
}

// ---------------------------------------------------------------------------
// Update before the products: U = G, or momentum M' = beta M + G and
// U = G + beta M' (nesterov) or M'.  fp32.
// ---------------------------------------------------------------------------
struct PreArgs {
  const void* g;
  const float* mom;   // nullptr: U = G
  float* mom_out;
  float beta;
  int nesterov;
  double* part;       // [E][chunks] sums of squares
  float* cs;          // [E][2][steps]: c_i, then c_i / c_{i+1}
  uint16_t* xh;       // [E][rp][cp]
  void* xl;           // lo: fp16 for fp32 gradients, else 8 bits; nullptr: not needed
  int32_t* ticket;    // zeroed here
  int tickets;        // per matrix
  int rows, cols, rp, cp, chunks, steps;
  float eps, lo_scale, growth[kMaxSteps];
};

template <class T, bool MOM>
__device__ __forceinline__ void update8(const PreArgs& a, int64_t o, int n, bool store, float* u) {
  ld8(static_cast<const T*>(a.g) + o, n, u);
  if constexpr (MOM) {
    float m[8];
    if (store) {
      ld8(a.mom + o, n, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = a.beta * m[i] + u[i];
      st8(a.mom_out + o, n, m);
    } else {
      ld8(a.mom_out + o, n, m);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = a.nesterov ? u[i] + a.beta * m[i] : m[i];
  }
}

// Sum of squares of one chunk of a matrix (its elements as one run), in double:
// squares of fp32 values neither overflow nor vanish there.
template <class T, bool MOM>
__global__ __launch_bounds__(kNormThreads) void orth_norm_kernel(PreArgs a) {
  __shared__ double red[kNormThreads / 64];
  const int64_t n = static_cast<int64_t>(a.rows) * a.cols, e = blockIdx.y;
  double s = 0.0;
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x) * 8; i < n;
       i += static_cast<int64_t>(a.chunks) * kNormThreads * 8) {
    float u[8];
    const int k = n - i < 8 ? static_cast<int>(n - i) : 8;
    update8<T, MOM>(a, e * n + i, k, true, u);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < k) s += static_cast<double>(u[j]) * static_cast<double>(u[j]);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kNormThreads / 64; ++w) s += red[w];
    a.part[e * a.chunks + blockIdx.x] = s;
  }
}

// The scaled fp16 pair of U with zero padding, and the scales c_i.
template <class T, bool MOM>
__global__ __launch_bounds__(kNormThreads) void orth_scale_kernel(PreArgs a) {
  __shared__ double red[kNormThreads / 64];
  const int64_t e = blockIdx.y;
  double s = static_cast<int>(threadIdx.x) < a.chunks ? a.part[e * a.chunks + threadIdx.x] : 0.0;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < kNormThreads / 64; ++w) s += red[w];
  const double norm = sqrt(s);
  const bool ok = norm - norm == 0.0;  // a non-finite element makes the whole matrix NaN
  int q = 0;
  if (ok && norm > 0.0) {
    frexp(norm, &q);  // norm = f 2^q, f in [1/2, 1)
    q = -q;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    double c = ok && norm > 0.0 ? ldexp(1.0, -q) / (norm + static_cast<double>(a.eps)) : 1.0;
    float* cs = a.cs + e * 2 * a.steps;
    for (int i = 0; i < a.steps; ++i) {  // X may grow by growth[i]; c >= 1 becomes 1
      const double next = fmin(1.0, c * static_cast<double>(a.growth[i]));
      cs[i] = static_cast<float>(c);
      cs[a.steps + i] = static_cast<float>(c / next);  // also where c itself is below fp32's range
      c = next;
    }
  }
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.tickets; i += kNormThreads) a.ticket[e * a.tickets + i] = 0;
  const int64_t n = static_cast<int64_t>(a.rows) * a.cols;
  const int64_t np = static_cast<int64_t>(a.rp) * a.cp;
  const int cv = a.cp / 8;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kNormThreads + threadIdx.x; i < np / 8;
       i += static_cast<int64_t>(gridDim.x) * kNormThreads) {
    const int r = static_cast<int>(i / cv), c = static_cast<int>(i % cv) * 8;
    float u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = 0.f;
    if (r < a.rows && c < a.cols) {
      const int k = a.cols - c < 8 ? a.cols - c : 8;
      update8<T, MOM>(a, e * n + static_cast<int64_t>(r) * a.cols + c, k, false, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = ldexpf(u[j], q) * kS;
        if (!ok) u[j] = NAN;
        if (j >= k) u[j] = 0.f;
      }
    }
    const int64_t o = e * np + i * 8;
    uint4 hi;
    if constexpr (sizeof(T) == 4) {
      uint4 lo;
      split8(u, hi, lo);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.xl) + o) = lo;
    } else {
      uint2 lo;
      split8_fp8(u, a.lo_scale, hi, lo);
      if (a.xl) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.xl) + o) = lo;
    }
    *reinterpret_cast<uint4*>(a.xh + o) = hi;
  }
}

// ---------------------------------------------------------------------------
// The products.
// ---------------------------------------------------------------------------
struct MmArgs {
  const uint16_t *ah, *al, *bh, *bl;  // operands (lo parts: fp32 gradients only)
  int64_t sa, sb;                     // elements per matrix
  int lda, ldb, K;
  int M, N;                           // padded output rows and columns
  int tm, tn;                         // output tiles (symmetric kinds: tn = 1, tm = all lower tiles)
  unsigned tiles;                     // tm * tn * E
  // epilogue
  const uint16_t* eh;                 // A (poly) or X (apply) at the output's place
  const void* el;                     // and its lo part; apply without split operands: 8 bits, or none (zero)
  const float* din;                   // diagonal of A (poly) or of B (apply)
  float* dout;                        // of A (gram) or of B (poly)
  int64_t sd;
  uint16_t* oh;                       // outputs; ol as el, nullptr: not wanted
  void* ol;
  int64_t so;
  int ldo;
  const float* cs;
  int steps, step, out;
  float ca, cb, cc;                   // the step's coefficients
  float lo_scale;
  // result / weight
  void* o;
  const void* w;
  int rows, cols;
  float keep, gain;                   // w' = keep w - gain O
  // K split over `ks` workgroups per tile (symmetric kinds on the smallest tiles)
  int ks;
  float* part;                        // [tile][ks] accumulators
  int32_t* ticket;                    // [tile], zero before and after a launch
};

// BM x BN outputs per workgroup by 2 x NW waves of WM x WN; K step BK; a ring of
// kRing K steps of both operands in LDS; fragments of KG 16-deep slices (a phase)
// in registers at a time, twice.  PAIRS: operands with lo parts, which come into
// the same step, so that the four tiles of a step serve its three products.
template <int BM_, int BN_, int BK_, int RING_, int KG_, bool PAIRS_, int NW_ = 2>
struct Tile {
  static constexpr int kNW = NW_, kWaves = 2 * NW_, kThreads = 64 * kWaves;
  static constexpr int BM = BM_, BN = BN_, BK = BK_, kRing = RING_, KG = KG_;
  static constexpr bool kPairs = PAIRS_;
  static constexpr int kPhases = BK / 16 / KG;  // per step
  static constexpr int WM = BM / 2, WN = BN / NW_, TM = WM / 32, TN = WN / 32;
  static constexpr int kA = BM * BK, kHi = (BM + BN) * BK;  // elements: the A tile, then the B tile (then lo likewise)
  static constexpr int kSlot = kHi * (PAIRS_ ? 2 : 1);
  static constexpr int kLoads = kSlot / 512 / kWaves;       // LDS-DMA instructions per wave and step
  static constexpr int kLds = kRing * kSlot;
  // symmetric outputs go by squares of this size, each within whole waves' outputs
  static constexpr int kSq = WM >= 128 ? 128 : BN;
  static constexpr int kWavesPerSimd = kLds * 2 > 80 * 1024 ? kWaves / 4 : 2;  // workgroups per compute unit the LDS allows, at most 2
  static_assert(BM == BN, "square tiles: symmetric outputs go by their lower triangle");
  static_assert(kA % (512 * kWaves) == 0 && kHi % (512 * kWaves) == 0, "whole LDS-DMA instructions per wave");
};

// 16-byte chunk swizzles against bank conflicts.  K-contiguous tiles (BK
// elements per row): a fragment read takes one chunk column of 16 consecutive
// rows at a time.  M/N-contiguous tiles (W elements per k-row): a transposing
// read takes 4 consecutive k-rows times 4 chunks.
template <int BK>
__device__ __forceinline__ int kc_swz(int row) {
  return BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3;
}
template <int W>
__device__ __forceinline__ int mc_swz(int k) {
  return W >= 128 ? 4 * (k & 3) : 4 * ((k >> 1) & 1);
}

// MFMA fragment from a tile whose rows (RS elements, one k each) run along M/N,
// with 16-byte chunks swizzled by swz(k): two transposing reads.  In each group
// G of 16 lanes, lane L points at k-row 16 ks + 8 (G/2) + L/4 (then 4 further)
// and columns base + 16 (G%2) + 4 (L%4), and receives the four k values of
// column base + 16 (G%2) + L.
template <int RS, class F>
__device__ __forceinline__ f16x8 frag_tr(const uint16_t* t, int base, int ks, int lane, F&& swz) {
  const int G = lane >> 4, L = lane & 15;
  const int k = ks * 16 + 8 * (G >> 1) + (L >> 2);
  const int c = base + 16 * (G & 1) + 4 * (L & 3);
  const uint16_t* p = t + k * RS + ((c >> 3) ^ swz(k)) * 8 + (c & 7);
  const uint16_t* q = t + (k + 4) * RS + ((c >> 3) ^ swz(k + 4)) * 8 + (c & 7);
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
  const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(q));
  const short v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  f16x8 r;
  __builtin_memcpy(&r, v, 16);
  return r;
}

// One operand of a tile: W rows (KC: stored with K contiguous) or columns.
template <int W, int BK, bool KC, int WAVES>
struct Operand {
  static constexpr int kLoads = W * BK / 512 / WAVES;  // LDS-DMA instructions per wave and step
  __amdgpu_buffer_rsrc_t hi, lo;
  int voff, vstep, kstep;  // this lane's byte offset, per load, and per K step

  // mn0: first row or column of the tile, of mn
  __device__ __forceinline__ void init(const uint16_t* h, const uint16_t* l, int ld, int mn0, int mn, int K, int wave,
                                       int lane) {
    if constexpr (KC) {
      const int rows = mn - mn0 < W ? mn - mn0 : W;
      const int64_t o = static_cast<int64_t>(mn0) * ld, bytes = static_cast<int64_t>(rows) * ld * 2;
      hi = rsrc(h + o, bytes);
      lo = rsrc(l ? l + o : h + o, bytes);
      constexpr int CPR = BK / 8, RPI = 64 / CPR;
      const int row = wave * RPI + lane / CPR;
      // rows advance by WAVES RPI per load: a multiple of the swizzle's period
      voff = (row * ld + ((lane % CPR) ^ kc_swz<BK>(row)) * 8) * 2;
      vstep = WAVES * RPI * ld * 2;
      kstep = BK * 2;
    } else {
      const int64_t bytes = (static_cast<int64_t>(K) * ld - mn0) * 2;
      hi = rsrc(h + mn0, bytes);
      lo = rsrc(l ? l + mn0 : h + mn0, bytes);
      constexpr int CPR = W / 8, KPI = 64 / CPR;
      const int k = wave * KPI + lane / CPR;
      voff = (k * ld + ((lane % CPR) ^ mc_swz<W>(k)) * 8) * 2;
      vstep = WAVES * KPI * ld * 2;
      kstep = BK * ld * 2;
    }
  }
  // Loads of the K step at byte offset soff into dst (this operand's part of a ring slot).
  __device__ __forceinline__ void issue(bool low, int soff, uint16_t* dst, int wave) const {
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(low ? lo : hi, (lds_void*)(dst + (wave + WAVES * u) * 512), 16,
                                               voff + u * vstep, soff, 0, 0);
  }
  // MFMA fragment: 32 rows (or columns) from `base`, k-slice ks of 16.
  __device__ static __forceinline__ f16x8 frag(const uint16_t* t, int base, int ks, int lane) {
    if constexpr (KC) {
      const int row = base + (lane & 31);
      const int ph = (ks * 2 + (lane >> 5)) ^ kc_swz<BK>(row);
      return *reinterpret_cast<const f16x8*>(t + row * BK + ph * 8);
    } else {
      return frag_tr<W>(t, base, ks, lane, [](int k) { return mc_swz<W>(k); });
    }
  }
};

// Fragments of slice ks from one ring slot.  The restrict-qualified tile
// pointers are what tells the compiler that these reads do not touch the slots
// that LDS-DMA loads in flight write; without them every read waits for all loads.
template <class C, bool AKC, bool BKC>
__device__ __forceinline__ void read_frags(const uint16_t* __restrict__ as, const uint16_t* __restrict__ bs, int wm,
                                           int wn, int ks, int lane, f16x8 (&fa)[C::TM], f16x8 (&fb)[C::TN]) {
#pragma unroll
  for (int i = 0; i < C::TM; ++i) fa[i] = Operand<C::BM, C::BK, AKC, C::kWaves>::frag(as, wm * C::WM + i * 32, ks, lane);
#pragma unroll
  for (int j = 0; j < C::TN; ++j) fb[j] = Operand<C::BN, C::BK, BKC, C::kWaves>::frag(bs, wn * C::WN + j * 32, ks, lane);
}

// Tile i of those of the lower triangle, in row order.
__device__ __forceinline__ void tri_tile(int i, int& r, int& c) {
  r = static_cast<int>((__builtin_sqrtf(8.0f * static_cast<float>(i) + 1.0f) - 1.0f) * 0.5f);
  while (r * (r + 1) / 2 > i) --r;
  while ((r + 1) * (r + 2) / 2 <= i) ++r;
  c = i - r * (r + 1) / 2;
}

// ---------------------------------------------------------------------------
// Epilogue.  Each wave handles its WM x WN outputs in blocks of 32 rows, alone
// (no barriers), through two buffers of its own in the ring's LDS.  A buffer
// holds the block's hi and lo parts (32 rows of WN fp16 values each).  What the
// epilogue reads of X or A comes by LDS-DMA, a block ahead, as whole row
// pieces; the results go back into the same places and leave as whole row
// pieces too, and for the symmetric outputs once more transposed.  (Straight
// from registers, where a lane holds 16 bytes of its row at a time, the apply
// launch of 128 matrices of 4096 x 1536 took 4.07 ms and not 3.08, with 256 x 128 tiles.)
// ---------------------------------------------------------------------------

// Chunk swizzle of a block's rows: free of conflicts for 16 consecutive rows at
// one chunk (the accumulators' order) and for the transposing reads' 4 rows
// times 2 chunks.
template <int WT>
__device__ __forceinline__ int ep_swz(int r) {
  if constexpr (WT == 128) return ((r & 3) << 2) | ((r >> 2) & 3);
  else if constexpr (WT == 64) return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  else return (r >> 2) & 3;
}

// A block's 8-bit lo part: rows of WT bytes, in 16-byte chunks (what LDS-DMA
// moves) swizzled likewise.  lo8_at: the 8 bytes of columns 8 q .. 8 q + 7.
template <int WT>
__device__ __forceinline__ int lo8_swz(int r) {
  return WT == 64 ? (r >> 2) & 3 : (r >> 3) & 1;
}
template <int WT>
__device__ __forceinline__ uint2* lo8_at(uint16_t* lo, int r, int q) {
  return reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(lo) + r * WT + (((q >> 1) ^ lo8_swz<WT>(r)) * 16) +
                                  (q & 1) * 8);
}

// Transposed pieces of a block (restrict-qualified as in read_frags).
template <int WN, bool SPLIT>
__device__ __forceinline__ void mirror_frags(const uint16_t* __restrict__ hi, const uint16_t* __restrict__ lo, int cb,
                                             int ks, int lane, f16x8& vh, f16x8& vl) {
  auto swz = [](int r) { return ep_swz<WN>(r); };
  vh = frag_tr<WN>(hi, cb, ks, lane, swz);
  if constexpr (SPLIT) vl = frag_tr<WN>(lo, cb, ks, lane, swz);
}

// Barrier of the K loop: LDS accesses are ordered across it, the LDS-DMA loads in
// flight are left alone (a full fence may wait for all of them).
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// LDS accesses of one wave are in order; this keeps the compiler's order too.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Linear combination that makes a stored value (times kS) from hi x, lo y of
// the staged input and the accumulator v, per row or per column:
//   gram   v' = kv v
//   poly   o = (b + c (D_r + D_c)) (x + y) + kv v            (A A = O O + (D_r + D_c) O off the diagonal)
//   apply  o = f ((a + D) x + (a + theta D) y + kv v)
// (D: the diagonal in fp32; O: A without it.)  In apply the diagonal acts on
// what the product saw of X: on x + y for pairs (theta 1), on x for hi-only
// products (theta 0).  With the diagonal on y too and O not, hi-only products
// would treat a rounding in B's range and outside it alike, far off for both where
// the rank is low: theta 1/2 is off by 0.06-0.08% (rms, without the output's
// rounding) for full rank but 0.18% for rank 42 of 128; 0 by 0.08-0.12% for all.
template <class C, int KIND, bool SPLIT, bool BYROW>
struct Coef {
  static constexpr float kTheta = SPLIT ? 1.0f : 0.0f;
  static constexpr bool kCols = KIND == kPoly || (KIND == kApply && !BYROW);
  float dr[C::TM];                                // at this lane's rows
  float dc[kCols ? C::TN : 1][2][8];              // at its columns
  float a, b, c, v, f, lo_scale, lo_inv;

  // cs: c_i, ratio: c_i / c_{i+1}
  __device__ __forceinline__ void init(const MmArgs& p, int64_t e, float cs, float ratio, int mw, int nw, int lane) {
    const int rl = lane & 31, g = lane >> 5;
    a = p.ca;
    b = p.cb;
    c = p.cc;
    lo_scale = p.lo_scale;
    lo_inv = SPLIT ? 1.0f : 1.0f / p.lo_scale;
    f = KIND != kApply ? 1.0f : p.out == kOutX ? ratio : cs / kS;
    v = KIND == kGram ? cs * cs / kS : (KIND == kPoly ? p.cc : f) / kS;
    if constexpr (KIND != kGram) {
      const float* d = p.din + e * p.sd;
#pragma unroll
      for (int i = 0; i < C::TM; ++i) {
        const int row = mw + 32 * i + rl;
        dr[i] = (KIND == kPoly || BYROW) && row < p.M ? d[row] : 0.f;
      }
      if constexpr (kCols)
#pragma unroll
        for (int i = 0; i < C::TN; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = nw + 32 * i + 16 * h + 8 * g;
#pragma unroll
            for (int q = 0; q < 8; q += 4) {
              const float4 t = col < p.N ? *reinterpret_cast<const float4*>(d + col + q) : make_float4(0.f, 0.f, 0.f, 0.f);
              dc[i][h][q] = t.x;
              dc[i][h][q + 1] = t.y;
              dc[i][h][q + 2] = t.z;
              dc[i][h][q + 3] = t.w;
            }
          }
    }
  }
};

// Block i: accumulators -> stored values, in place of the staged hi / lo.
template <class C, int KIND, bool SPLIT, bool BYROW, bool FINAL, bool HASLO>
__device__ __forceinline__ void epi_block(const f32x16 (&acc)[C::TN], uint16_t* __restrict__ hi,
                                          uint16_t* __restrict__ lo, const Coef<C, KIND, SPLIT, BYROW>& k, int i,
                                          int lane) {
  using K = Coef<C, KIND, SPLIT, BYROW>;
  const int rl = lane & 31, g = lane >> 5;
  float ax = 0.f, ay = 0.f;  // coefficients of x and y where they go by rows
  if constexpr (KIND == kPoly) ax = k.b + k.c * k.dr[i];
  if constexpr (KIND == kApply && BYROW) {
    ax = k.f * (k.a + k.dr[i]);
    ay = k.f * (k.a + K::kTheta * k.dr[i]) * k.lo_inv;
  }
#pragma unroll
  for (int j = 0; j < C::TN; ++j) {
    float v[2][8];
    to_chunks(acc[j], v);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = rl * C::WN + ((4 * j + 2 * h + g) ^ ep_swz<C::WN>(rl)) * 8;
      f16x8 x, ys;
      float y[8];
      uint2* const at8 = lo8_at<C::WN>(lo, rl, 4 * j + 2 * h + g);
      if constexpr (KIND != kGram) x = *reinterpret_cast<const f16x8*>(hi + at);
      if constexpr (HASLO && SPLIT) ys = *reinterpret_cast<const f16x8*>(lo + at);
      if constexpr (HASLO && !SPLIT) {
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 t = *reinterpret_cast<const u32x2*>(at8);
        lo_fp8(make_uint2(t[0], t[1]), y);
      } else if constexpr (HASLO) {
#pragma unroll
        for (int q = 0; q < 8; ++q) y[q] = static_cast<float>(ys[q]);
      }
      float o[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        o[q] = k.v * v[h][q];
        if constexpr (KIND == kPoly) {
          const float t = ax + k.c * k.dc[j][h][q];
          o[q] += t * static_cast<float>(x[q]);
          if constexpr (HASLO) o[q] += t * y[q];
        } else if constexpr (KIND == kApply) {
          if constexpr (!BYROW) {
            ax = k.f * (k.a + k.dc[j][h][q]);
            ay = k.f * (k.a + K::kTheta * k.dc[j][h][q]) * k.lo_inv;
          }
          o[q] += ax * static_cast<float>(x[q]);
          if constexpr (HASLO) o[q] += ay * y[q];
        }
      }
      if constexpr (FINAL) {  // fp32: the chunk's first half in hi's place, the second in lo's
        lds_put16(hi + at, Elem<float>::pack(o));
        lds_put16(lo + at, Elem<float>::pack(o + 4));
      } else if constexpr (SPLIT) {
        uint4 uh, ul;
        split8(o, uh, ul);
        lds_put16(hi + at, uh);
        lds_put16(lo + at, ul);
      } else if constexpr (KIND == kApply) {
        uint4 uh;
        uint2 ul;
        split8_fp8(o, k.lo_scale, uh, ul);
        lds_put16(hi + at, uh);
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 t = {ul.x, ul.y};
        *reinterpret_cast<u32x2*>(at8) = t;
      } else {
        f16x8 r;
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = static_cast<_Float16>(o[q]);
        *reinterpret_cast<f16x8*>(hi + at) = r;
      }
    }
  }
}

// The diagonal of a symmetric output within block i and its 32 columns j:
// written in fp32, and zero in the matrix.
template <class C, int KIND, bool SPLIT>
__device__ __forceinline__ void epi_diagonal(const f32x16& acc, uint16_t* hi, uint16_t* lo,
                                             const Coef<C, KIND, SPLIT, true>& k, int i, int j, float* dout,
                                             bool in, int lane) {
  const int rl = lane & 31, g = lane >> 5;
  float v[2][8];
  to_chunks(acc, v);
  float t = 0.f;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 8; ++q) t = 16 * h + 8 * g + q == rl ? v[h][q] : t;
  if (((rl >> 3) & 1) == g) {
    float d = k.v * t / kS;  // poly: O's diagonal is zero
    if constexpr (KIND == kPoly) d += k.dr[i] * (k.b + k.c * k.dr[i]);
    if (in) *dout = d;
    const int at = rl * C::WN + ((4 * j + (rl >> 3)) ^ ep_swz<C::WN>(rl)) * 8 + (rl & 7);
    hi[at] = 0;
    if constexpr (SPLIT) lo[at] = 0;
  }
}

// NT: streaming stores.
template <bool NT>
__device__ __forceinline__ void st16(void* p, const uint4& v) {
  if constexpr (NT) {
    typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 t = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(t, static_cast<u32x4*>(p));
  } else {
    *static_cast<uint4*>(p) = v;
  }
}

// stage() brings a block's inputs, run() does the rest; coefs() loads the
// coefficients.  The kernel stages the first block (and where a tile is one block,
// WM = 32, calls coefs() too) before the K loop ends, so that the latency passes
// behind it.
template <class C, int KIND, bool SPLIT, bool BYROW, bool FINAL, bool HASLO>
struct Epilogue {
  static constexpr int WN = C::WN, kPart = 32 * WN, CPR = WN / 8, RPI = 64 / CPR, kPieces = 32 / RPI;
  static constexpr bool kLo8 = KIND == kApply && !SPLIT;
  static constexpr int CPR8 = WN / 16, RPI8 = 64 / CPR8, kPieces8 = 32 / RPI8;  // the same for an 8-bit lo part
  static constexpr int kStage = kPieces + (HASLO ? (kLo8 ? kPieces8 : kPieces) : 0);
  // 256 x 256 tiles are used where the outputs are far larger than the L2s: by
  // streaming stores 128 of 2048 x 1024 took 6.62 ms, not 6.74
  static constexpr bool NT = C::BM == 256;
  static_assert(WN == 64 || WN == 32, "row piece layouts");
  static_assert(C::kWaves * 2 * kPart <= C::kSlot && (C::TM == 1 || C::kRing == 2), "a buffer per wave in each ring slot");

  const MmArgs& p;
  const int64_t e;
  const int mw, nw, lane;  // this wave's outputs begin at row mw, column nw
  const int64_t ob, eo;
  Coef<C, KIND, SPLIT, BYROW> k;
  __amdgpu_buffer_rsrc_t rh, rlo;
  uint16_t* buf[2];        // this wave's buffers, of even and odd blocks

  __device__ __forceinline__ Epilogue(const MmArgs& p_, int64_t e_, int mw_, int nw_, int lane_)
      : p(p_), e(e_), mw(mw_), nw(nw_), lane(lane_), ob(e_ * p_.so),
        eo(e_ * p_.so + static_cast<int64_t>(mw_) * p_.ldo + nw_) {
    const int64_t left = mw < p.M && nw < p.N ? (static_cast<int64_t>(p.M - mw) * p.ldo - nw) * 2 : 0;
    if constexpr (KIND != kGram) rh = rsrc(p.eh + eo, left);
    if constexpr (HASLO)
      rlo = kLo8 ? rsrc(static_cast<const uint8_t*>(p.el) + eo, left / 2)
                 : rsrc(static_cast<const uint16_t*>(p.el) + eo, left);
  }
  __device__ __forceinline__ void coefs(float cs, float ratio) { k.init(p, e, cs, ratio, mw, nw, lane); }
  __device__ __forceinline__ void place(uint16_t* even, uint16_t* odd, int wave) {
    buf[0] = even + wave * 2 * kPart;
    buf[1] = odd + wave * 2 * kPart;
  }
  // row pieces: piece u of a block is rows [u RPI, (u + 1) RPI), 16 bytes per lane
  __device__ __forceinline__ int piece_col(int u) const {
    return ((lane % CPR) ^ ep_swz<WN>(u * RPI + lane / CPR)) * 8;
  }
  __device__ __forceinline__ void stage(int i) const {
    if constexpr (KIND == kGram) return;
    uint16_t* b = buf[i & 1];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int voff = ((32 * i + u * RPI + lane / CPR) * p.ldo + piece_col(u)) * 2;
      dma16(rh, b + u * 512, voff);
      if constexpr (HASLO && !kLo8) dma16(rlo, b + kPart + u * 512, voff);
    }
    if constexpr (HASLO && kLo8)
#pragma unroll
      for (int u = 0; u < kPieces8; ++u) {
        const int r = u * RPI8 + lane / CPR8;
        dma16(rlo, b + kPart + u * 512, (32 * i + r) * p.ldo + ((lane % CPR8) ^ lo8_swz<WN>(r)) * 16);
      }
  }

  // Waits until block i's inputs have landed, but neither for those of block i + 1
  // nor for the outputs of block i - 1, which were issued after them (vector memory
  // operations complete in order).  On the matrix's edge some of those stores may
  // not have been issued: there the wait covers them.
  static constexpr int kStores = kPieces * (SPLIT && !FINAL ? 2 : 1);                    // per block, at least
  static constexpr int kMirror = KIND == kApply ? 0 : WN / 32 * 2 * (SPLIT ? 2 : 1);  // and below the diagonal
  __device__ __forceinline__ void wait_block(int i, bool full, bool below) const {
    const bool more = i + 1 < C::TM;
    if (i == 0 || !full) {
      if (more) wait_vm<kStage>();
      else wait_vm<0>();
    } else if (kLo8 && !FINAL && p.ol) {
      if (more) wait_vm<kStage + kStores + kPieces8>();
      else wait_vm<kStores + kPieces8>();
    } else if (below) {
      if (more) wait_vm<kStage + kStores + kMirror>();
      else wait_vm<kStores + kMirror>();
    } else {
      if (more) wait_vm<kStage + kStores>();
      else wait_vm<kStores>();
    }
  }

  // staged: the first block is on its way (and the second, if there is one)
  __device__ __forceinline__ void run(const f32x16 (&acc)[C::TM][C::TN], bool staged) const {
    const int rl = lane & 31, g = lane >> 5, pr = lane / CPR, pr8 = lane / CPR8;
    // symmetric outputs, by squares: above the diagonal there is nothing to do,
    // squares on it are computed whole, those below are written twice
    const bool below = KIND != kApply && mw / C::kSq > nw / C::kSq;
    if (KIND != kApply && mw / C::kSq < nw / C::kSq) {
      wait_vm<0>();  // no load into LDS outlives its wave
      return;
    }
    const bool full = FINAL ? mw + C::WM <= p.rows && nw + WN <= p.cols : mw + C::WM <= p.M && nw + WN <= p.N;
    if (!staged) stage(0);
#pragma unroll
    for (int i = 0; i < C::TM; ++i) {
      uint16_t* hi = buf[i & 1];
      uint16_t* lo = hi + kPart;
      if constexpr (KIND != kGram) wait_block(i, full, below);
      epi_block<C, KIND, SPLIT, BYROW, FINAL, HASLO>(acc[i], hi, lo, k, i, lane);
      if constexpr (KIND != kApply) {
        const int row = mw + 32 * i + rl;
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
          if (mw + 32 * i == nw + 32 * j) {
            wave_lds_fence();
            epi_diagonal<C, KIND, SPLIT>(acc[i][j], hi, lo, k, i, j, p.dout + e * p.sd + row, row < p.M, lane);
          }
      }
      wave_lds_fence();
      if constexpr (FINAL) {
        using T = typename std::conditional<SPLIT, float, uint16_t>::type;
#pragma unroll 1
        for (int u = 0; u < kPieces; ++u) {
          float o[8];
          Elem<float>::unpack(lds_get16(hi + u * 512 + lane * 8), o);
          Elem<float>::unpack(lds_get16(lo + u * 512 + lane * 8), o + 4);
          const int orow = mw + 32 * i + u * RPI + pr, col = nw + piece_col(u);
          if (orow < p.rows && col < p.cols) {
            const int64_t off = (e * p.rows + orow) * p.cols + col;
            const int n = p.cols - col;
            if (p.out == kOutW) {
              float w[8];
              ld8(static_cast<const T*>(p.w) + off, n, w);
#pragma unroll
              for (int q = 0; q < 8; ++q) o[q] = p.keep * w[q] - p.gain * o[q];
            }
            st8(static_cast<T*>(p.o) + off, n, o);
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
          const int orow = 32 * i + u * RPI + pr, col = piece_col(u);
          const uint4 vh = lds_get16(hi + u * 512 + lane * 8);
          uint4 vl;
          if constexpr (SPLIT) vl = lds_get16(lo + u * 512 + lane * 8);
          if (mw + orow < p.M && nw + col < p.N) {
            const int64_t off = eo + orow * p.ldo + col;
            st16<NT>(p.oh + off, vh);
            if constexpr (SPLIT) st16<NT>(static_cast<uint16_t*>(p.ol) + off, vl);
          }
        }
        if (kLo8 && p.ol)
#pragma unroll
          for (int u = 0; u < kPieces8; ++u) {
            const int r = u * RPI8 + pr8, orow = 32 * i + r, col = ((lane % CPR8) ^ lo8_swz<WN>(r)) * 16;
            const uint4 vl = lds_get16(lo + u * 512 + lane * 8);
            if (mw + orow < p.M && nw + col < p.N)
              st16<NT>(static_cast<uint8_t*>(p.ol) + eo + orow * p.ldo + col, vl);
          }
      }
      if constexpr (KIND != kApply) {
        if (below) {  // the mirror image: 8 of the block's rows at one column per lane
          const int64_t mo = ob + static_cast<int64_t>(nw + rl) * p.ldo + mw + 8 * g;
#pragma unroll
          for (int t = 0; t < WN / 32 * 2; ++t) {
            const int cb = (t >> 1) * 32, ks = t & 1;
            f16x8 vh, vl;
            mirror_frags<WN, SPLIT>(hi, lo, cb, ks, lane, vh, vl);
            if (nw + cb + rl < p.N && mw + 32 * i + ks * 16 + 8 * g < p.M) {
              const int64_t off = mo + cb * p.ldo + 32 * i + ks * 16;
              *reinterpret_cast<uint4*>(p.oh + off) = __builtin_bit_cast(uint4, vh);
              if constexpr (SPLIT)
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.ol) + off) = __builtin_bit_cast(uint4, vl);
            }
          }
        }
      }
      wave_lds_fence();
      if constexpr (KIND != kGram)
        if (i + 2 < C::TM) {
          __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer has been read out
          stage(i + 2);
        }
    }
  }
};

// Joins the workgroups that share a tile's K: each writes its accumulators to
// the workspace, and the last to arrive adds them all, in order, whichever it
// is.  True in that one.  Accumulators and tickets are device-scope atomics
// (they meet behind the XCDs' caches) ordered by waiting for the stores, not by
// fences: a device-scope fence writes back a whole L2, which with some hundred
// workgroups took 60 us.
template <class C>
__device__ __forceinline__ bool join_k(f32x16 (&acc)[C::TM][C::TN], const MmArgs& p, int64_t lid, int ks_i,
                                       uint16_t* lds, int tid) {
  constexpr int kVec = C::TM * C::TN * 8;  // pairs of floats per thread
  uint64_t* part = reinterpret_cast<uint64_t*>(p.part) + lid * p.ks * kVec * 256 + tid;
  uint64_t* mine = part + static_cast<int64_t>(ks_i) * kVec * 256;
#pragma unroll
  for (int v = 0; v < kVec; ++v) {
    const f32x16& t = acc[v / 8 / C::TN][v / 8 % C::TN];
    const uint64_t lo = __float_as_uint(t[2 * (v % 8)]), hi = __float_as_uint(t[2 * (v % 8) + 1]);
    __hip_atomic_store(mine + v * 256, lo | hi << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  int* last = reinterpret_cast<int*>(lds);
  wait_vm<0>();
  __syncthreads();  // all partials are out; the ring is no longer read
  if (tid == 0) {
    const int n = __hip_atomic_fetch_add(p.ticket + lid, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *last = n == p.ks - 1;
    if (n == p.ks - 1) __hip_atomic_store(p.ticket + lid, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  const bool is_last = *last != 0;
  __syncthreads();  // before the epilogue uses this LDS
  if (!is_last) return false;
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
#pragma unroll 2
  for (int k = 0; k < p.ks; ++k) {
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const uint64_t u = __hip_atomic_load(part + (static_cast<int64_t>(k) * kVec + v) * 256, __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT);
      f32x16& t = acc[v / 8 / C::TN][v / 8 % C::TN];
      t[2 * (v % 8)] += __uint_as_float(static_cast<uint32_t>(u));
      t[2 * (v % 8) + 1] += __uint_as_float(static_cast<uint32_t>(u >> 32));
    }
  }
  return true;
}

// MODE of apply: the next X from one without a lo part, from one with it, or the
// last step's result.
enum { kX0 = 0, kX = 1, kLast = 2 };

template <class C, int KIND, bool AKC, bool BKC, int MODE>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::kWavesPerSimd)))
void orth_mm_kernel(MmArgs p) {
  constexpr bool SPLIT = C::kPairs;
  __shared__ __attribute__((aligned(16))) uint16_t lds[C::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::kNW, wn = wave % C::kNW;
  // consecutive tiles of a matrix on one XCD (workgroups go to the 8 XCDs in
  // turn); 32-bit arithmetic, as 64-bit divisions took half a microsecond of each launch
  constexpr bool kKSplit = C::BM == 64 && KIND != kApply;
  const unsigned ks_n = kKSplit ? p.ks : 1, total = p.tiles * ks_n;
  const unsigned wid = blockIdx.x % kNumXcd * ((total + kNumXcd - 1) / kNumXcd) + blockIdx.x / kNumXcd;
  if (blockIdx.x / kNumXcd >= (total + kNumXcd - 1) / kNumXcd || wid >= total) return;
  const unsigned lid = kKSplit ? wid / ks_n : wid;
  const int ks_i = kKSplit ? static_cast<int>(wid - lid * ks_n) : 0;
  const unsigned per = p.tm * p.tn, el = lid / per;
  const int64_t e = el;
  const int t = static_cast<int>(lid - el * per);
  int r, c;
  if constexpr (KIND == kApply) {  // the shorter side inside
    if (p.tm <= p.tn) { c = t / p.tm; r = t - c * p.tm; }
    else { r = t / p.tn; c = t - r * p.tn; }
  } else {
    tri_tile(t, r, c);
  }
  const int m0 = __builtin_amdgcn_readfirstlane(r * C::BM), n0 = __builtin_amdgcn_readfirstlane(c * C::BN);

  Operand<C::BM, C::BK, AKC, C::kWaves> A;
  Operand<C::BN, C::BK, BKC, C::kWaves> B;
  A.init(p.ah + e * p.sa, SPLIT ? p.al + e * p.sa : nullptr, p.lda, m0, p.M, p.K, wave, lane);
  B.init(p.bh + e * p.sb, SPLIT ? p.bl + e * p.sb : nullptr, p.ldb, n0, p.N, p.K, wave, lane);
  constexpr bool kHasLo = KIND == kGram ? false : SPLIT || (KIND == kApply && MODE == kX);
  Epilogue<C, KIND, SPLIT, KIND != kApply || !BKC, MODE == kLast, kHasLo> epi(p, e, m0 + wm * C::WM, n0 + wn * C::WN,
                                                                              lane);
  const float cs = p.cs[e * 2 * p.steps + p.step], ratio = p.cs[e * 2 * p.steps + p.steps + p.step];
  const bool early = ks_n == 1;
  if (C::TM == 1 && early) epi.coefs(cs, ratio);
  const int nk1 = (p.K + C::BK - 1) / C::BK;
  const int k_lo = kKSplit ? static_cast<int>(static_cast<unsigned>(nk1 * ks_i) / ks_n) : 0;
  const int nk = (kKSplit ? static_cast<int>(static_cast<unsigned>(nk1 * (ks_i + 1)) / ks_n) : nk1) - k_lo;
  int head = 0;  // K step (from k_lo) to load next, and its ring slot
  int head_slot = 0;
  auto issue = [&]() {
    uint16_t* dst = lds + head_slot * C::kSlot;
    const int k = k_lo + head;
    A.issue(false, k * A.kstep, dst, wave);
    B.issue(false, k * B.kstep, dst + C::kA, wave);
    if constexpr (SPLIT) {
      A.issue(true, k * A.kstep, dst + C::kHi, wave);
      B.issue(true, k * B.kstep, dst + C::kHi + C::kA, wave);
    }
    ++head;
    head_slot = head_slot + 1 == C::kRing ? 0 : head_slot + 1;
  };

  f32x16 acc[C::TM][C::TN];
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  // K loop.  The fragments of a phase are read while the MFMAs of the one before
  // it run.  Before a step's last phase all its fragments are in registers:
  // there the waves meet, the next step's loads are known to have landed, and the
  // step's own ring slot is free for the loads of step kt + kRing.
  constexpr int kLoG = SPLIT ? C::KG : 1;
  f16x8 fa[2][C::KG][C::TM], fb[2][C::KG][C::TN];
  f16x8 la[2][kLoG][C::TM], lb[2][kLoG][C::TN];
  auto read = [&](int slot, int ph, int buf) {
    const uint16_t* as = lds + slot * C::kSlot;
#pragma unroll
    for (int g = 0; g < C::KG; ++g) {
      read_frags<C, AKC, BKC>(as, as + C::kA, wm, wn, ph * C::KG + g, lane, fa[buf][g], fb[buf][g]);
      if constexpr (SPLIT)
        read_frags<C, AKC, BKC>(as + C::kHi, as + C::kHi + C::kA, wm, wn, ph * C::KG + g, lane, la[buf][g],
                                lb[buf][g]);
    }
  };
  // a wave whose outputs lie above the diagonal only helps with the loads
  const bool idle = KIND != kApply && (m0 + wm * C::WM) / C::kSq < (n0 + wn * C::WN) / C::kSq;
  auto mma = [&](int buf) {
    if (KIND != kApply && idle) return;
    auto product = [&](const f16x8 (&x)[C::TM], const f16x8 (&y)[C::TN]) {
#pragma unroll
      for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(y[j], x[i], acc[i][j], 0, 0, 0);
    };
#pragma unroll
    for (int g = 0; g < C::KG; ++g) {
      product(fa[buf][g], fb[buf][g]);
      if constexpr (SPLIT) {
        product(fa[buf][g], lb[buf][g]);
        product(la[buf][g], fb[buf][g]);
      }
    }
  };
  for (int s = 0; s < C::kRing && s < nk; ++s) issue();
  if (nk >= C::kRing) wait_vm<(C::kRing - 1) * C::kLoads>();
  else wait_vm<0>();
  lds_barrier();
  read(0, 0, 0);
  int slot = 0;
  static_assert(C::kRing == 2 || C::kRing == 3, "ring waits");
  static_assert(C::kPhases % 2 == 0, "phase buffers alternate");
  for (int kt = 0; kt + 1 < nk; ++kt) {
#pragma unroll
    for (int ph = 0; ph + 1 < C::kPhases; ++ph) {
      read(slot, ph + 1, (ph + 1) & 1);
      mma(ph & 1);
    }
    // the loads of one more step may stay outstanding, if there are any
    if (C::kRing == 3 && kt + 2 < nk) wait_vm<C::kLoads>();
    else wait_vm<0>();
    lds_barrier();
    if (head < nk) issue();
    slot = slot + 1 == C::kRing ? 0 : slot + 1;
    read(slot, 0, 0);
    mma((C::kPhases - 1) & 1);
  }
  // the last step; no other slot is read any more, so the epilogue's first inputs
  // can go into the next one
  if (early) {
    epi.place(lds + (slot + 1 == C::kRing ? 0 : slot + 1) * C::kSlot, lds + slot * C::kSlot, wave);
    epi.stage(0);
  }
#pragma unroll
  for (int ph = 0; ph < C::kPhases; ++ph) {
    if (ph + 1 < C::kPhases) read(slot, ph + 1, (ph + 1) & 1);
    mma(ph & 1);
  }
  if constexpr (kKSplit) {
    if (ks_n > 1 && !join_k<C>(acc, p, lid, ks_i, lds, tid)) return;
  }
  if constexpr (C::TM > 1) {
    epi.coefs(cs, ratio);
    lds_barrier();  // the last step's slot is no longer read
    epi.stage(1);
  } else if (!early) {  // after join_k, whose barriers came after the last reads of the ring
    epi.coefs(cs, ratio);
    epi.place(lds, lds, wave);
  }
  epi.run(acc, early);
}

// ---------------------------------------------------------------------------
// Small matrices: all steps of a matrix in one workgroup, X and A in LDS.  The
// same arithmetic as above with 32 x 32 outputs per wave and task; a chain of
// short launches would cost more than the work (8 matrices of 64 x 128: 17
// launches).
// ---------------------------------------------------------------------------
constexpr int kSmallThreads = 512, kSmallWaves = kSmallThreads / 64;
constexpr int kSmallA = 2, kSmallX = 5;        // 32 x 32 outputs of A and of X per wave at most
constexpr int kSmallLds = 160 * 1024;

// LDS rows of any multiple of 64 elements, 16-byte chunks swizzled: free of
// conflicts for 8 consecutive rows at one chunk and for the transposing reads.
__device__ __forceinline__ int sm_swz(int r) { return ((r & 3) << 1) | ((r >> 2) & 1); }
__device__ __forceinline__ int sm_at(int r, int ld, int chunk) { return r * ld + (chunk ^ sm_swz(r)) * 8; }

template <bool KC>
__device__ __forceinline__ f16x8 sm_frag(const uint16_t* t, int ld, int base, int ks, int lane) {
  if constexpr (KC) {
    return *reinterpret_cast<const f16x8*>(t + sm_at(base + (lane & 31), ld, ks * 2 + (lane >> 5)));
  } else {  // as frag_tr
    const int G = lane >> 4, L = lane & 15;
    const int k = ks * 16 + 8 * (G >> 1) + (L >> 2);
    const int c = base + 16 * (G & 1) + 4 * (L & 3);
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(t + sm_at(k, ld, c >> 3) + (c & 7)));
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(t + sm_at(k + 4, ld, c >> 3) + (c & 7)));
    const short v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    f16x8 r;
    __builtin_memcpy(&r, v, 16);
    return r;
  }
}

struct SmMat {
  uint16_t *h, *l;
  int ld;
};

// This wave's tasks of an M x N output: 32 x 32 outputs at (r, c) each.
template <int TASKS>
struct SmTasks {
  int r[TASKS], c[TASKS], n;
  __device__ __forceinline__ void init(int M, int N, int wave) {
    const int nc = N / 32, all = M / 32 * nc;
    n = 0;
#pragma unroll
    for (int u = 0; u < TASKS; ++u) {
      const int t = u * kSmallWaves + wave;
      r[u] = __builtin_amdgcn_readfirstlane(t / nc * 32);
      c[u] = __builtin_amdgcn_readfirstlane(t % nc * 32);
      n += t < all;
    }
  }
};

template <bool AKC, bool BKC, bool SPLIT, int TASKS>
__device__ __forceinline__ void sm_product(f32x16 (&acc)[TASKS], const SmMat& A, const SmMat& B,
                                           const SmTasks<TASKS>& t, int K, int lane) {
#pragma unroll
  for (int u = 0; u < TASKS; ++u) {
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[u][q] = 0.f;
    if (u >= t.n) continue;
    const int r = t.r[u], c = t.c[u];
    for (int k4 = 0; k4 < K / 16; k4 += 4) {  // K is a multiple of 64
      f16x8 a[4], b[4], al[SPLIT ? 4 : 1], bl[SPLIT ? 4 : 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = sm_frag<AKC>(A.h, A.ld, r, k4 + i, lane);
        b[i] = sm_frag<BKC>(B.h, B.ld, c, k4 + i, lane);
        if constexpr (SPLIT) {
          al[i] = sm_frag<AKC>(A.l, A.ld, r, k4 + i, lane);
          bl[i] = sm_frag<BKC>(B.l, B.ld, c, k4 + i, lane);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b[i], a[i], acc[u], 0, 0, 0);
        if constexpr (SPLIT) {
          acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bl[i], a[i], acc[u], 0, 0, 0);
          acc[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b[i], al[i], acc[u], 0, 0, 0);
        }
      }
    }
  }
}

// The 8-column chunks of a wave's task as (row, column, values).
template <class F>
__device__ __forceinline__ void sm_chunks(const f32x16& acc, int r, int c, int lane, F&& f) {
  float v[2][8];
  to_chunks(acc, v);
#pragma unroll
  for (int h = 0; h < 2; ++h) f(r + (lane & 31), c + 16 * h + 8 * (lane >> 5), v[h]);
}

__device__ __forceinline__ void sm_get(const SmMat& m, int r, int c, float* x) {  // the hi part
  const int at = sm_at(r, m.ld, c >> 3);
  const f16x8 h = *reinterpret_cast<const f16x8*>(m.h + at);
#pragma unroll
  for (int q = 0; q < 8; ++q) x[q] = static_cast<float>(h[q]);
}

__device__ __forceinline__ void sm_row8(const float* d, int c, float* o) {  // c a multiple of 8
  Elem<float>::unpack(lds_get16(d + c), o);
  Elem<float>::unpack(lds_get16(d + c + 4), o + 4);
}

struct SmArgs {
  PreArgs pre;
  float coef[kMaxSteps][3];
  void* o;
  const void* w;   // nullptr: write the result, else the updated weight
  float keep, gain;
};

// AT, XT: outputs of A and of X per wave.  With one of each (X up to 8192 elements)
// the kernel is short and spills nothing: 8 of 64 x 128 fp32 31.5 -> 26 us.
template <class T, bool MOM, bool TALL, int AT, int XT>
__global__ __launch_bounds__(kSmallThreads) void orth_small_kernel(SmArgs p) {
  constexpr bool SPLIT = sizeof(T) == 4;
  constexpr float kTheta = SPLIT ? 1.0f : 0.0f;  // as in Coef
  __shared__ __attribute__((aligned(16))) uint8_t lds[kSmallLds];
  const PreArgs& a = p.pre;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t e = blockIdx.x;
  const int rp = a.rp, cp = a.cp, mp = TALL ? cp : rp, n = rp * cp;
  uint16_t* base = reinterpret_cast<uint16_t*>(lds);
  const SmMat X{base, base + n, cp};
  const SmMat A{base + 2 * n, base + 2 * n + mp * mp, mp};
  float* da = reinterpret_cast<float*>(base + 2 * n + (SPLIT ? 2 : 1) * mp * mp);
  float* db = da + mp;
  double* red = reinterpret_cast<double*>(db + mp);

  // norm, then the scaled pair (both passes give an element to the same thread)
  const int64_t g0 = e * a.rows * a.cols;
  const int cv = cp / 8;
  double s = 0.0;
  auto each = [&](auto&& f) {
    for (int i = tid; i < n / 8; i += kSmallThreads) {
      const int r = i / cv, c = i - r * cv;
      const int k = r < a.rows ? a.cols - 8 * c : 0;
      f(r, c, k < 0 ? 0 : (k < 8 ? k : 8), g0 + static_cast<int64_t>(r) * a.cols + 8 * c);
    }
  };
  each([&](int, int, int k, int64_t o) {
    float u[8];
    if (k > 0) update8<T, MOM>(a, o, k, true, u);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < k) s += static_cast<double>(u[j]) * static_cast<double>(u[j]);
  });
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o, 64);
  if (lane == 0) red[wave] = s;
  __syncthreads();
  s = 0.0;
  for (int w = 0; w < kSmallWaves; ++w) s += red[w];
  const double norm = sqrt(s);
  const bool ok = norm - norm == 0.0;
  int q2 = 0;
  if (ok && norm > 0.0) {
    frexp(norm, &q2);
    q2 = -q2;
  }
  double cd = ok && norm > 0.0 ? ldexp(1.0, -q2) / (norm + static_cast<double>(a.eps)) : 1.0;
  each([&](int r, int c, int k, int64_t o) {
    float u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (k > 0) update8<T, MOM>(a, o, k, false, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] = j < k ? (ok ? ldexpf(u[j], q2) * kS : NAN) : 0.f;
    uint4 hi, lo;
    split8(u, hi, lo);
    lds_put16(X.h + sm_at(r, cp, c), hi);
    lds_put16(X.l + sm_at(r, cp, c), lo);
  });
  __syncthreads();

  SmTasks<AT> ta;  // tasks of A, and of X
  SmTasks<XT> tx;
  ta.init(mp, mp, wave);
  tx.init(rp, cp, wave);
  for (int st = 0; st < a.steps; ++st) {
    const float ci = static_cast<float>(cd);
    const double next = fmin(1.0, cd * static_cast<double>(a.growth[st]));
    const float ratio = static_cast<float>(cd / next);
    cd = next;
    const float ca = p.coef[st][0], cb = p.coef[st][1], cc = p.coef[st][2];
    const bool last = st + 1 == a.steps;
    // Gram
    {
      f32x16 acc[AT];
      sm_product<!TALL, !TALL, SPLIT, AT>(acc, X, X, ta, TALL ? rp : cp, lane);
#pragma unroll
      for (int u = 0; u < AT; ++u) {
        if (u >= ta.n) continue;
        sm_chunks(acc[u], ta.r[u], ta.c[u], lane, [&](int r, int c, float* v) {
          float t = 0.f;
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const bool dg = c + q == r;
            v[q] *= ci * ci / kS;
            t = dg ? v[q] : t;
            v[q] = dg ? 0.f : v[q];
          }
          if (r >= c && r < c + 8) da[r] = t / kS;
          uint4 hi, lo;
          split8(v, hi, lo);
          lds_put16(A.h + sm_at(r, mp, c >> 3), hi);
          if constexpr (SPLIT) lds_put16(A.l + sm_at(r, mp, c >> 3), lo);
        });
      }
    }
    __syncthreads();
    // polynomial, in A's place
    {
      f32x16 acc[AT];
      sm_product<true, true, SPLIT, AT>(acc, A, A, ta, mp, lane);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < AT; ++u) {
        if (u >= ta.n) continue;
        sm_chunks(acc[u], ta.r[u], ta.c[u], lane, [&](int r, int c, float* v) {
          float x[8];
          const int at = sm_at(r, mp, c >> 3);
          sm_get(A, r, c, x);
          if constexpr (SPLIT) {
            const f16x8 l = *reinterpret_cast<const f16x8*>(A.l + at);
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] += static_cast<float>(l[q]);
          }
          const float d = da[r];
          float dc[8], t = 0.f;
          sm_row8(da, c, dc);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const bool dg = c + q == r;
            v[q] *= cc / kS;
            t = dg ? v[q] : t;
            v[q] = dg ? 0.f : v[q] + x[q] * (cb + cc * (d + dc[q]));
          }
          if (r >= c && r < c + 8) db[r] = t / kS + d * (cb + cc * d);
          uint4 hi, lo;
          split8(v, hi, lo);
          lds_put16(A.h + at, hi);
          if constexpr (SPLIT) lds_put16(A.l + at, lo);
        });
      }
    }
    __syncthreads();
    // apply, in X's place or to the result
    f32x16 acc[XT];
    if constexpr (TALL) sm_product<true, true, SPLIT, XT>(acc, X, A, tx, mp, lane);
    else sm_product<true, false, SPLIT, XT>(acc, A, X, tx, mp, lane);
    __syncthreads();
    const float f = last ? ci / kS : ratio;
#pragma unroll
    for (int u = 0; u < XT; ++u) {
      if (u >= tx.n) continue;
      sm_chunks(acc[u], tx.r[u], tx.c[u], lane, [&](int r, int c, float* v) {
        float x[8];
        const int at = sm_at(r, cp, c >> 3);
        sm_get(X, r, c, x);
        const f16x8 l = *reinterpret_cast<const f16x8*>(X.l + at);
        float dc[8];
        if constexpr (TALL) sm_row8(db, c, dc);
        const float dr = TALL ? 0.f : db[r];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float d = TALL ? dc[q] : dr, y = static_cast<float>(l[q]);
          v[q] = f * ((ca + d) * x[q] + (SPLIT || !last ? ca + kTheta * d : 0.f) * y + v[q] / kS);
        }
        if (!last) {
          uint4 hi, lo;
          split8(v, hi, lo);
          lds_put16(X.h + at, hi);
          lds_put16(X.l + at, lo);
        } else if (r < a.rows && c < a.cols) {
          const int64_t o = g0 + static_cast<int64_t>(r) * a.cols + c;
          const int k = a.cols - c;
          if (p.w) {
            float w[8];
            ld8(static_cast<const T*>(p.w) + o, k, w);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] = p.keep * w[q] - p.gain * v[q];
          }
          st8(static_cast<T*>(p.o) + o, k, v);
        }
      });
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
struct Sizes {
  int64_t E, x, a;  // matrices; fp16 elements of X and of A per matrix
  int rp, cp, mp, chunks;
  bool tall, split;
};

Sizes sizes_of(int E, int rows, int cols, bool split) {
  Sizes z;
  z.E = E;
  z.split = split;
  z.rp = static_cast<int>(align_up(rows, kPad));
  z.cp = static_cast<int>(align_up(cols, kPad));
  z.tall = z.rp > z.cp;
  z.mp = z.tall ? z.cp : z.rp;
  z.x = static_cast<int64_t>(z.rp) * z.cp;
  z.a = static_cast<int64_t>(z.mp) * z.mp;
  const int64_t c = cdiv(static_cast<int64_t>(rows) * cols, 8 * kNormThreads * 4);
  z.chunks = static_cast<int>(c < kMaxChunks ? c : kMaxChunks);
  return z;
}

// Tile sizes, chosen per product by how many tiles there are for the 256 compute
// units.  64 x 64 up to 768 of them, three to a unit by their LDS (one matrix of 2048
// x 1024: Gram 14 us against 26 us with 128 x 128; past that, one of 2048 x 2048,
// apply 41 us against 32 us).  Else 256 x 256 (eight waves, one workgroup per unit)
// or 128 x 128 (two per unit), see use_big.
using Big = Tile<256, 256, 64, 2, 2, false, 4>;
using Mid = Tile<128, 128, 64, 2, 2, false>;
using Small = Tile<64, 64, 64, 3, 2, false>;
using BigPairs = Tile<256, 256, 32, 2, 1, true, 4>;
using MidPairs = Tile<128, 128, 32, 2, 1, true>;
using SmallPairs = Tile<64, 64, 32, 3, 1, true>;
// where both operands are stored with K contiguous: K steps of 64 read whole
// 128-byte lines (one of 2900 x 2000: polynomial 62.5 -> 53.6 us; 4 of 1000 x 500:
// apply 16.6 -> 14.3 us; the others lost, 8 of 1001 x 777: Gram 30 -> 33 us).  Two
// of these fit a unit, so that past 512 tiles a second round begins, and they are
// the fastest there too: over 14 sizes of 528 to 756 tiles the whole call took 0.86
// to 1.02 of the time with SmallPairs and 0.93 to 1.02 of that with MidPairs (8 of
// 777 x 1001, 728 tiles: Gram 29.2 us against 31.8 and 30.7, polynomial 25.5
// against 28.2 and 29.2).
using SmallPairsK = Tile<64, 64, 64, 2, 2, true>;

// 256 x 256 tiles do the work of four 128 x 128 ones from half the LDS and L2
// traffic, in rounds of 256 against 512.  A round takes 1.7 times as long, its last
// partial one about as long as a full one, so the shorter sum of rounds is taken.
// Over 49 products of 19 sizes it was off by 3% at most in bf16 and 11% in fp32 (two
// of 1.1 rounds).  Measured, 256 x 256 against 128 x 128: apply of 128 of 4096 x
// 1536 (48 rounds against 96) 2.71 ms against 3.23; one of 4096 x 4096 (1 against 2)
// 134 us against 160, fp32 332 against 407; 8 of 1024 x 2048 (1 against 2) 46.5
// against 49; two of 2048 x 2048 (1 against 1) 59 against 45; 40 of 512 x 1024 (2
// against 3) 54 against 42.
bool use_big(int64_t big, int64_t mid) { return 17 * cdiv(big, 256) <= 10 * cdiv(mid, 512); }

// Tiles of a symmetric m x m output, and of an r x c one, in E matrices.
template <class C>
int64_t sym_tiles(int64_t m, int64_t E) {
  const int64_t n = cdiv(m, C::BM);
  return n * (n + 1) / 2 * E;
}
template <class C>
int64_t rect_tiles(int64_t r, int64_t c, int64_t E) {
  return cdiv(r, C::BM) * cdiv(c, C::BN) * E;
}

// Workgroups that share the K steps of a symmetric product's tile (Small tiles):
// enough to occupy the chip, each with at least eight of the steps of 64, and
// only where it shortens the longest chain by 16 steps or more, about 5 us, which
// is what joining costs (4096 x 128: Gram 25 -> 12 us; at 8 steps saved 12 -> 13 us).
int k_split(int64_t tiles, int64_t steps) {
  if (tiles < 1) return 1;
  int64_t n = 512 / tiles;
  if (n > steps / 8) n = steps / 8;
  if (n > 16) n = 16;
  return n > 1 && steps - cdiv(steps, n) >= 16 ? static_cast<int>(n) : 1;
}
// of the Gram (K = the longer side) or the polynomial (the shorter side); 1 where other tiles are used
int k_split(const Sizes& z, int64_t K) {
  const int64_t tiles = sym_tiles<Small>(z.mp, z.E);
  return tiles > 256 ? 1 : k_split(tiles, cdiv(K, 64) * (z.split ? 2 : 1));
}

struct Ws {
  double* part;
  float *cs, *da, *db;  // scales; diagonals of A and B
  float* kpart;         // split-K accumulators
  int32_t* ticket;      // and their tickets: `tickets` per matrix
  int tickets;
  uint16_t *xh[2], *ah, *al, *bh, *bl;
  void* xl[2];
};

// X as two buffers (a product reads one and writes the other), with its lo parts
// (without split operands in 8 bits, and read only where it is written: one
// buffer serves); A and B (pairs when split).
size_t ws_layout(const Sizes& z, char* base, Ws* w) {
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* p = base + o;
    o += align_up(bytes, 256);
    return reinterpret_cast<uint16_t*>(p);
  };
  Ws t;
  t.part = reinterpret_cast<double*>(take(static_cast<size_t>(z.E) * z.chunks * 8));
  t.cs = reinterpret_cast<float*>(take(static_cast<size_t>(z.E) * 2 * kMaxSteps * 4));
  t.da = reinterpret_cast<float*>(take(static_cast<size_t>(z.E) * z.mp * 4));
  t.db = reinterpret_cast<float*>(take(static_cast<size_t>(z.E) * z.mp * 4));
  const int64_t tiles = sym_tiles<Small>(z.mp, z.E);
  const int kg = k_split(z, z.rp > z.cp ? z.rp : z.cp), kp = k_split(z, z.mp), ks = kg > kp ? kg : kp;
  t.kpart = reinterpret_cast<float*>(take(ks > 1 ? static_cast<size_t>(tiles) * ks * Small::BM * Small::BN * 4 : 0));
  t.ticket = reinterpret_cast<int32_t*>(take(ks > 1 ? static_cast<size_t>(tiles) * 4 : 0));
  t.tickets = ks > 1 ? static_cast<int>(tiles / z.E) : 0;
  const size_t xb = static_cast<size_t>(z.E) * z.x * 2, ab = static_cast<size_t>(z.E) * z.a * 2;
  t.xh[0] = take(xb);
  t.xh[1] = take(xb);
  t.xl[0] = take(z.split ? xb : xb / 2);
  t.xl[1] = z.split ? take(xb) : t.xl[0];
  t.ah = take(ab);
  t.bh = take(ab);
  t.al = z.split ? take(ab) : t.ah;
  t.bl = z.split ? take(ab) : t.bh;
  if (w) *w = t;
  return o;
}

template <class C, int KIND, bool AKC, bool BKC>
void launch_mm(const char* name, const MmArgs& a, hipStream_t s) {
  const dim3 grid(xcd_grid(static_cast<int64_t>(a.tiles) * a.ks));
  auto go = [&](auto mode) {
    MOE_LAUNCH(name, (orth_mm_kernel<C, KIND, AKC, BKC, decltype(mode)::value>), grid, dim3(C::kThreads), 0, s, a);
  };
  if constexpr (KIND == kApply) {
    if (a.out != kOutX) return go(std::integral_constant<int, kLast>{});
    if constexpr (!C::kPairs)
      if (!a.el) return go(std::integral_constant<int, kX0>{});
  }
  go(std::integral_constant<int, kX>{});
}

template <int KIND, bool AKC, bool BKC>
void launch_any(const char* name, MmArgs& a, const Sizes& z, hipStream_t s) {
  auto go = [&](auto tile) {
    using C = decltype(tile);
    if constexpr (KIND == kApply) {
      a.tm = static_cast<int>(cdiv(a.M, C::BM));
      a.tn = static_cast<int>(cdiv(a.N, C::BN));
    } else {
      a.tm = static_cast<int>(sym_tiles<C>(a.M, 1));
      a.tn = 1;
    }
    a.tiles = static_cast<unsigned>(static_cast<int64_t>(a.tm) * a.tn * z.E);
    a.ks = C::BM == 64 && !(KIND == kApply) ? k_split(z, a.K) : 1;
    launch_mm<C, KIND, AKC, BKC>(name, a, s);
  };
  const bool ap = KIND == kApply;
  if ((ap ? rect_tiles<Small>(a.M, a.N, z.E) : sym_tiles<Small>(a.M, z.E)) <= 768)
    z.split ? go(typename std::conditional<AKC && BKC, SmallPairsK, SmallPairs>::type{}) : go(Small{});
  else if (ap ? use_big(rect_tiles<Big>(a.M, a.N, z.E), rect_tiles<Mid>(a.M, a.N, z.E))
              : use_big(sym_tiles<Big>(a.M, z.E), sym_tiles<Mid>(a.M, z.E)))
    z.split ? go(BigPairs{}) : go(Big{});
  else
    z.split ? go(MidPairs{}) : go(Mid{});
}

void run_products(const Sizes& z, const Ws& w, MmArgs a, const float (*coef)[3], int out, bool exact0,
                  hipStream_t s) {
  a.cs = w.cs;
  a.sd = z.mp;
  a.part = w.kpart;
  a.ticket = w.ticket;
  for (int i = 0; i < a.steps; ++i) {
    const int cur = i & 1, nxt = cur ^ 1;
    const uint16_t* xl = static_cast<const uint16_t*>(w.xl[cur]);  // as an operand: with split operands only
    a.step = i;
    a.ca = coef[i][0];
    a.cb = coef[i][1];
    a.cc = coef[i][2];
    a.out = kOutX;
    // Gram: the shorter side's inner products
    a.ah = a.bh = w.xh[cur];
    a.al = a.bl = xl;
    a.sa = a.sb = z.x;
    a.lda = a.ldb = z.cp;
    a.K = z.tall ? z.rp : z.cp;
    a.M = a.N = z.mp;
    a.oh = w.ah;
    a.ol = w.al;
    a.dout = w.da;
    a.so = z.a;
    a.ldo = z.mp;
    if (z.tall) launch_any<kGram, false, false>("orth_gram", a, z, s);
    else launch_any<kGram, true, true>("orth_gram", a, z, s);
    // polynomial
    a.ah = a.bh = a.eh = w.ah;
    a.al = a.bl = w.al;
    a.el = w.al;
    a.sa = a.sb = z.a;
    a.lda = a.ldb = a.K = z.mp;
    a.oh = w.bh;
    a.ol = w.bl;
    a.din = w.da;
    a.dout = w.db;
    launch_any<kPoly, true, true>("orth_poly", a, z, s);
    // apply
    a.M = z.rp;
    a.N = z.cp;
    a.eh = w.xh[cur];
    // without split operands the last step does without X's lo part, and the first
    // of a bf16 gradient has none.  Singular values are near 1 by then, where the
    // polynomial makes of a small change c between -1.6 c and 1.7 c, which is nearer to
    // none than to the a c of the other steps (64 x 128 of full rank 0.13% off, with it
    // 0.15%; but rank 1, whose noise is elsewhere, 0.09% against 0.04%)
    a.el = !z.split && (i + 1 == a.steps || (i == 0 && exact0)) ? nullptr : w.xl[cur];
    a.din = w.db;
    a.oh = w.xh[nxt];
    a.ol = !z.split && i + 2 >= a.steps ? nullptr : w.xl[nxt];
    a.so = z.x;
    a.ldo = z.cp;
    a.out = i + 1 < a.steps ? static_cast<int>(kOutX) : out;
    if (z.tall) {  // X B, B symmetric
      a.ah = w.xh[cur];
      a.al = xl;
      a.sa = z.x;
      a.lda = z.cp;
      a.bh = w.bh;
      a.bl = w.bl;
      a.sb = z.a;
      a.ldb = z.mp;
      launch_any<kApply, true, true>("orth_apply", a, z, s);
    } else {  // B X
      a.ah = w.bh;
      a.al = w.bl;
      a.sa = z.a;
      a.lda = z.mp;
      a.bh = w.xh[cur];
      a.bl = xl;
      a.sb = z.x;
      a.ldb = z.cp;
      launch_any<kApply, true, false>("orth_apply", a, z, s);
    }
  }
}

template <class T, bool MOM>
void run_pre(const Sizes& z, const PreArgs& a, hipStream_t s) {
  const unsigned E = static_cast<unsigned>(z.E);
  MOE_LAUNCH("orth_norm", (orth_norm_kernel<T, MOM>), dim3(z.chunks, E), dim3(kNormThreads), 0, s, a);
  const int64_t blocks = cdiv(z.x / 8, kNormThreads * 4);
  MOE_LAUNCH("orth_scale", (orth_scale_kernel<T, MOM>), dim3(static_cast<unsigned>(blocks < 1024 ? blocks : 1024), E),
             dim3(kNormThreads), 0, s, a);
}

// Coefficients of every step with the ranges they lead to: singular values
// start in [0, 1] and |a x + b x^3 + c x^5| over [0, s] bounds the next ones.
// The fp16 buffers hold values up to 15 (kS 15 < 65504); steps that could leave
// that range are refused.  growth: the largest factor by which a step multiplies
// a singular value.  lo_scale: what 8-bit lo parts are multiplied by; a value x kS
// has |lo| <= 2^-11 |x| kS = 2 |x|, and |x| is at most the largest singular value.
struct Plan {
  float coef[kMaxSteps][3];
  float growth[kMaxSteps];
  float lo_scale;
};
constexpr double kRange = 15.0;

int make_plan(const float* coef, int steps, Plan& p) {
  static const float kQuintic[3] = {3.4445f, -4.7750f, 2.0315f};
  double s = 1.0 + 1e-3, most = s;
  for (int i = 0; i < steps; ++i) {
    const float* c = coef ? coef + 3 * i : kQuintic;
    for (int j = 0; j < 3; ++j) {
      if (!(c[j] - c[j] == 0.f)) return MOE_EINVAL;
      p.coef[i][j] = c[j];
    }
    const double a = c[0], b = c[1], q = c[2];
    // extrema over [0, s]: of x (a + b x^2 + q x^4), of a + b y + q y^2 and of b y + q y^2 (y = x^2)
    double top = 0.0, gain = std::fabs(a), poly = 0.0;
    auto at = [&](double x) {
      if (!(x >= 0.0) || x > s) return;
      const double y = x * x, b2 = b * y + q * y * y;
      top = std::fmax(top, std::fabs(x * (a + b2)));
      gain = std::fmax(gain, std::fabs(a + b2));
      poly = std::fmax(poly, std::fabs(b2));
    };
    at(s);
    if (q != 0.0) {
      if (-b / (2.0 * q) > 0.0) at(std::sqrt(-b / (2.0 * q)));
      const double disc = 9.0 * b * b - 20.0 * a * q;
      if (disc >= 0.0)
        for (double r : {(-3.0 * b + std::sqrt(disc)) / (10.0 * q), (-3.0 * b - std::sqrt(disc)) / (10.0 * q)})
          if (r > 0.0) at(std::sqrt(r));
    } else if (b != 0.0 && -a / (3.0 * b) > 0.0) {
      at(std::sqrt(-a / (3.0 * b)));
    }
    if (!(s * s <= kRange) || !(top <= kRange) || !(poly <= kRange)) return MOE_EUNSUPPORTED;
    p.growth[i] = static_cast<float>(gain > 1.0 ? gain : 1.0);
    s = top * (1.0 + 1e-2);  // rounding in the products
    most = std::fmax(most, s);
  }
  p.lo_scale = 256.0f;
  while (p.lo_scale * 2.0 * most > 440.0) p.lo_scale *= 0.5f;
  return MOE_OK;
}

int check_shape(int64_t E, int rows, int cols, int dtype) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL;
  if (E < 0 || rows < 1 || cols < 1) return MOE_EINVAL;
  if (E > 65535 || rows > kMaxDim || cols > kMaxDim) return MOE_EUNSUPPORTED;
  // a matrix is addressed with 31-bit byte offsets
  if (static_cast<int64_t>(align_up(rows, kPad)) * static_cast<int64_t>(align_up(cols, kPad)) * 2 > 0x7FFFFF00ll)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// Matrices that fit one workgroup: X (pairs) and A in its LDS, their 32 x 32
// outputs within its waves' tasks.  Whatever their number: 1 to 4096 of 32 x 64 to 128
// x 192 took 0.21 to 0.86 of the time of the tiled launches (one of 128 x 128 fp32 63
// us against 76, 1024 of 64 x 192 fp32 143 against 418), also in fp32 past 8192
// elements, where the kernel spills 28 registers.
bool small_fits(const Sizes& z) {
  const int64_t bytes = 4 * z.x + (z.split ? 4 : 2) * z.a + 8 * z.mp + 8 * kSmallWaves;
  return bytes <= kSmallLds && z.x <= 1024 * kSmallWaves * kSmallX && z.a <= 1024 * kSmallWaves * kSmallA;
}

template <class T, bool MOM>
void run_small(const Sizes& z, const SmArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(z.E)), block(kSmallThreads);
  auto go = [&](auto at, auto xt) {
    constexpr int AT = decltype(at)::value, XT = decltype(xt)::value;
    if (z.tall) MOE_LAUNCH("orth_small", (orth_small_kernel<T, MOM, true, AT, XT>), grid, block, 0, s, a);
    else MOE_LAUNCH("orth_small", (orth_small_kernel<T, MOM, false, AT, XT>), grid, block, 0, s, a);
  };
  using One = std::integral_constant<int, 1>;
  if (z.x <= 1024 * kSmallWaves && z.a <= 1024 * kSmallWaves) go(One{}, One{});
  else go(std::integral_constant<int, kSmallA>{}, std::integral_constant<int, kSmallX>{});
}

struct Step {  // the Muon step's part; mom nullptr: orthogonalise only
  const float* mom;
  float* mom_out;
  float beta;
  int nesterov;
  const void* w;
  float keep, gain;
};

int run(const void* g, int dtype, int E, int rows, int cols, int steps, const float* coef, float eps, const Step& st,
        void* out, void* ws, size_t ws_bytes, hipStream_t s) {
  const int bad = check_shape(E, rows, cols, dtype);
  if (bad != MOE_OK) return bad;
  if (steps < 1 || !(eps >= 0.f) || !(eps < 3.0e38f)) return MOE_EINVAL;
  if (steps > kMaxSteps) return MOE_EUNSUPPORTED;
  Plan plan;
  const int pst = make_plan(coef, steps, plan);
  if (pst != MOE_OK) return pst;
  if (E == 0) return MOE_OK;
  if (!g || !out || !ws) return MOE_EINVAL;
  for (const void* p : {g, static_cast<const void*>(out), static_cast<const void*>(ws),
                        static_cast<const void*>(st.mom), static_cast<const void*>(st.mom_out), st.w})
    if (!aligned16(p)) return MOE_EINVAL;
  const Sizes z = sizes_of(E, rows, cols, dtype == MOE_F32);
  if (ws_bytes < ws_layout(z, nullptr, nullptr)) return MOE_EWORKSPACE;
  Ws w;
  ws_layout(z, static_cast<char*>(ws), &w);
  PreArgs pre{};
  pre.g = g;
  pre.mom = st.mom;
  pre.mom_out = st.mom_out;
  pre.beta = st.beta;
  pre.nesterov = st.nesterov;
  pre.part = w.part;
  pre.cs = w.cs;
  pre.ticket = w.ticket;
  pre.tickets = w.tickets;
  pre.xh = w.xh[0];
  // a bf16 gradient has its 8 mantissa bits in hi (its smallest elements, below
  // 2^-26 of the norm, lose bits far below the result's accuracy)
  const bool exact0 = !z.split && (!st.mom || steps == 1);
  pre.xl = exact0 ? nullptr : w.xl[0];
  pre.rows = rows;
  pre.cols = cols;
  pre.rp = z.rp;
  pre.cp = z.cp;
  pre.chunks = z.chunks;
  pre.steps = steps;
  pre.eps = eps;
  pre.lo_scale = plan.lo_scale;
  for (int i = 0; i < steps; ++i) pre.growth[i] = plan.growth[i];
  if (small_fits(z)) {
    SmArgs sm{};
    sm.pre = pre;
    for (int i = 0; i < steps; ++i)
      for (int j = 0; j < 3; ++j) sm.coef[i][j] = plan.coef[i][j];
    sm.o = out;
    sm.w = st.w;
    sm.keep = st.keep;
    sm.gain = st.gain;
    if (z.split) st.mom ? run_small<float, true>(z, sm, s) : run_small<float, false>(z, sm, s);
    else st.mom ? run_small<uint16_t, true>(z, sm, s) : run_small<uint16_t, false>(z, sm, s);
    return launch_status();
  }
  if (z.split) {
    if (st.mom) run_pre<float, true>(z, pre, s);
    else run_pre<float, false>(z, pre, s);
  } else {
    if (st.mom) run_pre<uint16_t, true>(z, pre, s);
    else run_pre<uint16_t, false>(z, pre, s);
  }
  MmArgs a{};
  a.steps = steps;
  a.o = out;
  a.w = st.w;
  a.rows = rows;
  a.cols = cols;
  a.keep = st.keep;
  a.gain = st.gain;
  a.lo_scale = plan.lo_scale;
  const int kind = st.w ? kOutW : kOutO;
  run_products(z, w, a, plan.coef, kind, exact0, s);
  return launch_status();
}

bool finite(float v) { return v - v == 0.f; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_orthogonalize_workspace(int32_t E, int32_t rows, int32_t cols, int dtype) {
  if (check_shape(E, rows, cols, dtype) != MOE_OK) return 0;
  return ws_layout(sizes_of(E, rows, cols, dtype == MOE_F32), nullptr, nullptr);
}

extern "C" int moe_orthogonalize(const void* g, int dtype, int32_t E, int32_t rows, int32_t cols, int32_t steps,
                                 const float* coef, float eps, void* out, void* ws, size_t ws_bytes, void* stream) {
  return run(g, dtype, E, rows, cols, steps, coef, eps, Step{}, out, ws, ws_bytes, static_cast<hipStream_t>(stream));
}

extern "C" int moe_muon_step(const void* g, int dtype, int32_t E, int32_t rows, int32_t cols, const float* mom,
                             float momentum, int nesterov, int32_t steps, const float* coef, float eps, const void* w,
                             float lr, float weight_decay, float scale, float* mom_out, void* w_out, void* ws,
                             size_t ws_bytes, void* stream) {
  if (!finite(momentum) || !finite(lr) || !finite(weight_decay) || !finite(scale)) return MOE_EINVAL;
  if (E != 0 && (!mom || !mom_out || !w)) return MOE_EINVAL;
  const Step st{mom, mom_out, momentum, nesterov != 0, w, 1.0f - lr * weight_decay, lr * scale};
  if (!finite(st.keep) || !finite(st.gain)) return MOE_EINVAL;
  return run(g, dtype, E, rows, cols, steps, coef, eps, st, w_out, ws, ws_bytes, static_cast<hipStream_t>(stream));
}
