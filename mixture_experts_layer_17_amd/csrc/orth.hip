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
// grow), the a X term uses both; measured against fp64, the result is off by
// 0.07-0.16% (rms), less than its rounding to bf16 (0.17%).  fp32 gradients
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
__device__ __forceinline__ void add8(const uint4& u, float* o) {
  const f16x8 h = __builtin_bit_cast(f16x8, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] += static_cast<float>(h[i]);
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
  float* cs;          // [E][steps + 1]
  uint16_t *xh, *xl;  // [E][rp][cp]
  int rows, cols, rp, cp, chunks, steps;
  float eps, growth[kMaxSteps];
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
    float* cs = a.cs + e * (a.steps + 1);
    cs[0] = static_cast<float>(c);
    for (int i = 0; i < a.steps; ++i) {  // X may grow by growth[i]; c >= 1 becomes 1
      c = fmin(1.0, c * static_cast<double>(a.growth[i]));
      cs[i + 1] = static_cast<float>(c);
    }
  }
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
    uint4 hi, lo;
    split8(u, hi, lo);
    const int64_t o = e * np + i * 8;
    *reinterpret_cast<uint4*>(a.xh + o) = hi;
    *reinterpret_cast<uint4*>(a.xl + o) = lo;
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
  int64_t tiles;                      // tm * tn * E
  // epilogue
  const uint16_t *eh, *el;            // A (poly) or X (apply) at the output's place
  uint16_t *oh, *ol;                  // fp16 pair output
  int64_t so;
  int ldo;
  const float* cs;
  int steps, step, out;
  float ca, cb, cc;                   // the step's coefficients
  // result / weight
  void* o;
  const void* w;
  int rows, cols;
  float keep, gain;                   // w' = keep w - gain O
};

// BT x BT outputs per workgroup by four waves of WT x WT; K step BK; a ring of
// kRing K steps of both operands in LDS.
template <int BT_, int BK_>
struct Tile {
  static constexpr int BT = BT_, BK = BK_, WT = BT / 2, TM = WT / 32;
  static constexpr int kRing = 4;
  static constexpr int kOp = BT * BK;          // elements of one operand's K step
  static constexpr int kLoads = kOp / 512 / 4; // LDS-DMA instructions per wave, operand and step
  static constexpr int kLds = kRing * 2 * kOp;
  static_assert(kOp % 2048 == 0 && BT * BT <= kLds, "the output tile is mirrored through the ring's LDS");
};

// 16-byte chunk swizzles against bank conflicts.  K-contiguous tiles (BK
// elements per row): a fragment read takes one chunk column of 16 consecutive
// rows at a time.  M/N-contiguous tiles (BT elements per k-row): a transposing
// read takes 4 consecutive k-rows times 4 chunks.
template <int BK>
__device__ __forceinline__ int kc_swz(int row) {
  return BK == 64 ? (row >> 1) & 7 : (row >> 2) & 3;
}
template <int BT>
__device__ __forceinline__ int mc_swz(int k) {
  return BT >= 128 ? 4 * (k & 3) : 4 * ((k >> 1) & 1);
}

template <class C, bool KC>
struct Operand {
  __amdgpu_buffer_rsrc_t hi, lo;
  int voff, vstep, kstep;  // this lane's byte offset, per load, and per K step

  // rows0: first row (KC) or column of the tile; valid: rows (KC) of the operand
  __device__ __forceinline__ void init(const uint16_t* h, const uint16_t* l, int ld, int mn0, int mn, int K, int wave,
                                       int lane) {
    if constexpr (KC) {
      const int rows = mn - mn0 < C::BT ? mn - mn0 : C::BT;
      const int64_t o = static_cast<int64_t>(mn0) * ld, bytes = static_cast<int64_t>(rows) * ld * 2;
      hi = rsrc(h + o, bytes);
      lo = rsrc(l ? l + o : h + o, bytes);
      constexpr int CPR = C::BK / 8, RPI = 64 / CPR;
      const int row = wave * RPI + lane / CPR;
      // rows advance by 4 RPI per load: a multiple of the swizzle's period
      voff = (row * ld + ((lane % CPR) ^ kc_swz<C::BK>(row)) * 8) * 2;
      vstep = 4 * RPI * ld * 2;
      kstep = C::BK * 2;
    } else {
      const int64_t bytes = (static_cast<int64_t>(K) * ld - mn0) * 2;
      hi = rsrc(h + mn0, bytes);
      lo = rsrc(l ? l + mn0 : h + mn0, bytes);
      constexpr int CPR = C::BT / 8, KPI = 64 / CPR;
      const int k = wave * KPI + lane / CPR;
      voff = (k * ld + ((lane % CPR) ^ mc_swz<C::BT>(k)) * 8) * 2;
      vstep = 4 * KPI * ld * 2;
      kstep = C::BK * ld * 2;
    }
  }
  // Loads of the K step at byte offset soff into dst (this operand's ring slot).
  __device__ __forceinline__ void issue(bool low, int soff, uint16_t* dst, int wave) const {
#pragma unroll
    for (int u = 0; u < C::kLoads; ++u)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(low ? lo : hi, (lds_void*)(dst + (wave + 4 * u) * 512), 16,
                                               voff + u * vstep, soff, 0, 0);
  }
  // MFMA fragment: 32 rows (or columns) from `base`, k-slice ks of 16.
  __device__ static __forceinline__ f16x8 frag(const uint16_t* t, int base, int ks, int lane) {
    if constexpr (KC) {
      const int row = base + (lane & 31);
      const int ph = (ks * 2 + (lane >> 5)) ^ kc_swz<C::BK>(row);
      return *reinterpret_cast<const f16x8*>(t + row * C::BK + ph * 8);
    } else {
      return frag_tr<C::BT>(t, base, ks, lane);
    }
  }
  // The same from a tile whose rows (RS elements) run along M/N: two transposing
  // reads.  In each group G of 16 lanes, lane L points at k-row 16 ks + 8 (G/2) +
  // L/4 (then 4 further) and columns base + 16 (G%2) + 4 (L%4), and receives
  // the four k values of column base + 16 (G%2) + L.
  template <int RS>
  __device__ static __forceinline__ f16x8 frag_tr(const uint16_t* t, int base, int ks, int lane) {
    const int G = lane >> 4, L = lane & 15;
    const int k = ks * 16 + 8 * (G >> 1) + (L >> 2);
    const int c = base + 16 * (G & 1) + 4 * (L & 3);
    const uint16_t* p = t + k * RS + ((c >> 3) ^ mc_swz<RS>(k)) * 8 + (c & 7);  // k + 4 swizzles alike
    typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
    const i16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p));
    const i16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 4 * RS));
    const short v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    f16x8 r;
    __builtin_memcpy(&r, v, 16);
    return r;
  }
};

// Fragments of slice ks from one ring slot.  The restrict-qualified tile
// pointers are what tells the compiler that these reads do not touch the slots
// that LDS-DMA loads in flight write; without them every read waits for all loads.
template <class C, bool AKC, bool BKC>
__device__ __forceinline__ void read_frags(const uint16_t* __restrict__ as, const uint16_t* __restrict__ bs, int wm,
                                           int wn, int ks, int lane, f16x8 (&fa)[C::TM], f16x8 (&fb)[C::TM]) {
#pragma unroll
  for (int i = 0; i < C::TM; ++i) fa[i] = Operand<C, AKC>::frag(as, wm * C::WT + i * 32, ks, lane);
#pragma unroll
  for (int j = 0; j < C::TM; ++j) fb[j] = Operand<C, BKC>::frag(bs, wn * C::WT + j * 32, ks, lane);
}

// Lower-triangle tile of index i in row order: (r, c) with c <= r.
__device__ __forceinline__ void tri_tile(int i, int& r, int& c) {
  r = static_cast<int>((__builtin_sqrtf(8.0f * static_cast<float>(i) + 1.0f) - 1.0f) * 0.5f);
  while (r * (r + 1) / 2 > i) --r;
  while ((r + 1) * (r + 2) / 2 <= i) ++r;
  c = i - r * (r + 1) / 2;
}

template <class C, int KIND, bool AKC, bool BKC, bool SPLIT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(C::BT == 256 ? 1 : 2)))
void orth_mm_kernel(MmArgs p) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[C::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  // consecutive tiles of a matrix on one XCD (workgroups go to the 8 XCDs in turn)
  const int64_t lid = xcd_tile(blockIdx.x, p.tiles);
  if (lid < 0) return;
  const int per = p.tm * p.tn;
  const int64_t e = lid / per;
  const int t = static_cast<int>(lid - e * per);
  int r, c;
  if constexpr (KIND == kApply) {  // the shorter side inside
    if (p.tm <= p.tn) { c = t / p.tm; r = t - c * p.tm; }
    else { r = t / p.tn; c = t - r * p.tn; }
  } else {
    tri_tile(t, r, c);
  }
  const int m0 = __builtin_amdgcn_readfirstlane(r * C::BT), n0 = __builtin_amdgcn_readfirstlane(c * C::BT);

  Operand<C, AKC> A;
  Operand<C, BKC> B;
  A.init(p.ah + e * p.sa, SPLIT ? p.al + e * p.sa : nullptr, p.lda, m0, p.M, p.K, wave, lane);
  B.init(p.bh + e * p.sb, SPLIT ? p.bl + e * p.sb : nullptr, p.ldb, n0, p.N, p.K, wave, lane);
  const int nk1 = (p.K + C::BK - 1) / C::BK;
  const int nk = SPLIT ? 3 * nk1 : nk1;  // hi hi, hi lo, lo hi
  auto issue = [&](int kt) {
    uint16_t* dst = lds + (kt % C::kRing) * 2 * C::kOp;
    const int part = SPLIT ? (kt >= nk1) + (kt >= 2 * nk1) : 0;
    const int k = kt - part * nk1;
    A.issue(SPLIT && part == 2, k * A.kstep, dst, wave);
    B.issue(SPLIT && part == 1, k * B.kstep, dst + C::kOp, wave);
  };

  f32x16 acc[C::TM][C::TM];
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TM; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;

  // K loop.  The fragments of a slice are read while the MFMAs of the one before
  // it run.  Before a step's last slice all its fragments are in registers:
  // there the waves meet, the next step's loads are known to have landed, and the
  // step's own ring slot is free for the loads of step kt + kRing.
  constexpr int NS = C::BK / 16;
  constexpr int kLoads2 = 2 * C::kLoads;
  f16x8 fa[2][C::TM], fb[2][C::TM];
  auto read = [&](int kt, int ks, int buf) {
    const uint16_t* as = lds + (kt % C::kRing) * 2 * C::kOp;
    read_frags<C, AKC, BKC>(as, as + C::kOp, wm, wn, ks, lane, fa[buf], fb[buf]);
  };
  auto mma = [&](int buf) {
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[buf][j], fa[buf][i], acc[i][j], 0, 0, 0);
  };
  // at most `ahead` steps' loads outstanding
  auto wait_ahead = [&](int ahead) {
    if (ahead >= 2) wait_vm<2 * kLoads2>();
    else if (ahead == 1) wait_vm<kLoads2>();
    else wait_vm<0>();
  };
  for (int s = 0; s < C::kRing && s < nk; ++s) issue(s);
  if (nk >= C::kRing) wait_vm<3 * kLoads2>();
  else wait_vm<0>();
  __syncthreads();
  read(0, 0, 0);
  for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
    for (int ks = 0; ks < NS; ++ks) {
      if (ks + 1 < NS) {
        read(kt, ks + 1, (ks + 1) & 1);
      } else if (kt + 1 < nk) {
        wait_ahead(nk - 2 - kt);
        __syncthreads();
        if (kt + C::kRing < nk) issue(kt + C::kRing);
        read(kt + 1, 0, 0);
      }
      mma(ks & 1);
    }
  }
  static_assert(NS % 2 == 0, "slice buffers alternate");

  // ---- epilogue: 8-column chunks of one row per lane
  const float* cs = p.cs + e * (p.steps + 1) + p.step;
  const float ci = cs[0], cn = cs[1];
  const int64_t ob = e * p.so;
  const bool mirror = KIND != kApply && m0 != n0;
  if (mirror) __syncthreads();  // the ring's LDS becomes the mirror tile
  const int rl = lane & 31, hc = 8 * (lane >> 5);
  auto finish = [&](int i, int j, int cch, const float* v, float* o) {  // the stored (scaled) values of a chunk
    const int row = m0 + wm * C::WT + i * 32 + rl, col = n0 + wn * C::WT + j * 32 + 16 * cch + hc;
    if constexpr (KIND == kGram) {
      const float f = ci * ci / kS;
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = v[q] * f;
    } else {
      float x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = 0.f;
      if (row < p.M && col < p.N) {
        const int64_t off = ob + static_cast<int64_t>(row) * p.ldo + col;
        add8(*reinterpret_cast<const uint4*>(p.eh + off), x);
        if (SPLIT || KIND == kApply) add8(*reinterpret_cast<const uint4*>(p.el + off), x);
      }
      const float fx = KIND == kPoly ? p.cb : p.ca, fv = (KIND == kPoly ? p.cc : 1.0f) / kS;
#pragma unroll
      for (int q = 0; q < 8; ++q) o[q] = fx * x[q] + fv * v[q];
    }
  };
  if constexpr (KIND == kApply) {
    const float f = p.out == kOutX ? ci / cn : ci / kS;
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TM; ++j) {
        float v[2][8];
        to_chunks(acc[i][j], v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = m0 + wm * C::WT + i * 32 + rl, col = n0 + wn * C::WT + j * 32 + 16 * h + hc;
          float o[8];
          finish(i, j, h, v[h], o);
#pragma unroll
          for (int q = 0; q < 8; ++q) o[q] *= f;
          if (p.out == kOutX) {
            if (row < p.M && col < p.N) {
              uint4 hi, lo;
              split8(o, hi, lo);
              const int64_t off = ob + static_cast<int64_t>(row) * p.ldo + col;
              *reinterpret_cast<uint4*>(p.oh + off) = hi;
              *reinterpret_cast<uint4*>(p.ol + off) = lo;
            }
          } else if (row < p.rows && col < p.cols) {
            using T = typename std::conditional<SPLIT, float, uint16_t>::type;
            const int64_t off = (e * p.rows + row) * p.cols + col;
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
      }
  } else {
    // symmetric outputs: the tile, and its mirror image through LDS (row-major
    // there, read back with the transposing reads)
    uint4 keep_lo[SPLIT ? C::TM : 1][SPLIT ? C::TM : 1][2];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TM; ++j) {
        float v[2][8];
        to_chunks(acc[i][j], v);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int rr = wm * C::WT + i * 32 + rl, cc = wn * C::WT + j * 32 + 16 * h + hc;
          float o[8];
          finish(i, j, h, v[h], o);
          uint4 hi, lo;
          split8(o, hi, lo);
          if (m0 + rr < p.M && n0 + cc < p.N) {
            const int64_t off = ob + static_cast<int64_t>(m0 + rr) * p.ldo + n0 + cc;
            *reinterpret_cast<uint4*>(p.oh + off) = hi;
            if constexpr (SPLIT) *reinterpret_cast<uint4*>(p.ol + off) = lo;
          }
          if (mirror) lds_put16(lds + rr * C::BT + ((cc >> 3) ^ mc_swz<C::BT>(rr)) * 8, hi);
          if constexpr (SPLIT) keep_lo[i][j][h] = lo;
        }
      }
    if (mirror) {
      auto flush = [&](uint16_t* out) {
        __syncthreads();
        for (int i = wave; i < (C::BT / 32) * (C::BT / 16); i += 4) {
          const int cb = (i % (C::BT / 32)) * 32, ks = i / (C::BT / 32);
          const f16x8 v = Operand<C, false>::template frag_tr<C::BT>(lds, cb, ks, lane);
          const int row = n0 + cb + rl, col = m0 + ks * 16 + hc;
          if (row < p.N && col < p.M)
            *reinterpret_cast<uint4*>(out + ob + static_cast<int64_t>(row) * p.ldo + col) =
                __builtin_bit_cast(uint4, v);
        }
      };
      flush(p.oh);
      if constexpr (SPLIT) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < C::TM; ++i)
#pragma unroll
          for (int j = 0; j < C::TM; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int rr = wm * C::WT + i * 32 + rl, cc = wn * C::WT + j * 32 + 16 * h + hc;
              lds_put16(lds + rr * C::BT + ((cc >> 3) ^ mc_swz<C::BT>(rr)) * 8, keep_lo[i][j][h]);
            }
        flush(p.ol);
      }
    }
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

struct Ws {
  double* part;
  float* cs;
  uint16_t *xh[2], *xl[2], *ah, *al, *bh, *bl;
};

// X as two buffers of pairs (a product reads one and writes the other; without
// split operands lo is only read where it is written, so one buffer serves), A
// and B (pairs when split).
size_t ws_layout(const Sizes& z, char* base, Ws* w) {
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* p = base + o;
    o += align_up(bytes, 256);
    return reinterpret_cast<uint16_t*>(p);
  };
  Ws t;
  t.part = reinterpret_cast<double*>(take(static_cast<size_t>(z.E) * z.chunks * 8));
  t.cs = reinterpret_cast<float*>(take(static_cast<size_t>(z.E) * (kMaxSteps + 1) * 4));
  const size_t xb = static_cast<size_t>(z.E) * z.x * 2, ab = static_cast<size_t>(z.E) * z.a * 2;
  t.xh[0] = take(xb);
  t.xh[1] = take(xb);
  t.xl[0] = take(xb);
  t.xl[1] = z.split ? take(xb) : t.xl[0];
  t.ah = take(ab);
  t.bh = take(ab);
  t.al = z.split ? take(ab) : t.ah;
  t.bl = z.split ? take(ab) : t.bh;
  if (w) *w = t;
  return o;
}

template <class C, int KIND, bool AKC, bool BKC>
void launch_mm(const char* name, const MmArgs& a, bool split, hipStream_t s) {
  const dim3 grid(xcd_grid(a.tiles));
  if (split) MOE_LAUNCH(name, (orth_mm_kernel<C, KIND, AKC, BKC, true>), grid, dim3(256), 0, s, a);
  else MOE_LAUNCH(name, (orth_mm_kernel<C, KIND, AKC, BKC, false>), grid, dim3(256), 0, s, a);
}

template <class C>
void run_products(const Sizes& z, const Ws& w, MmArgs a, const float (*coef)[3], int out, hipStream_t s) {
  const int64_t nm = cdiv(z.mp, C::BT), sym = nm * (nm + 1) / 2;
  const int64_t nr = cdiv(z.rp, C::BT), nc = cdiv(z.cp, C::BT);
  a.cs = w.cs;
  for (int i = 0; i < a.steps; ++i) {
    const int cur = i & 1, nxt = cur ^ 1;
    a.step = i;
    a.ca = coef[i][0];
    a.cb = coef[i][1];
    a.cc = coef[i][2];
    a.out = kOutX;
    // Gram: the shorter side's inner products
    a.ah = a.bh = w.xh[cur];
    a.al = a.bl = w.xl[cur];
    a.sa = a.sb = z.x;
    a.lda = a.ldb = z.cp;
    a.K = z.tall ? z.rp : z.cp;
    a.M = a.N = z.mp;
    a.tm = static_cast<int>(sym);
    a.tn = 1;
    a.tiles = sym * z.E;
    a.oh = w.ah;
    a.ol = w.al;
    a.so = z.a;
    a.ldo = z.mp;
    if (z.tall) launch_mm<C, kGram, false, false>("orth_gram", a, z.split, s);
    else launch_mm<C, kGram, true, true>("orth_gram", a, z.split, s);
    // polynomial
    a.ah = a.bh = a.eh = w.ah;
    a.al = a.bl = a.el = w.al;
    a.sa = a.sb = z.a;
    a.lda = a.ldb = a.K = z.mp;
    a.oh = w.bh;
    a.ol = w.bl;
    launch_mm<C, kPoly, true, true>("orth_poly", a, z.split, s);
    // apply
    a.M = z.rp;
    a.N = z.cp;
    a.tm = static_cast<int>(nr);
    a.tn = static_cast<int>(nc);
    a.tiles = nr * nc * z.E;
    a.eh = w.xh[cur];
    a.el = w.xl[cur];
    a.oh = w.xh[nxt];
    a.ol = w.xl[nxt];
    a.so = z.x;
    a.ldo = z.cp;
    a.out = i + 1 < a.steps ? static_cast<int>(kOutX) : out;
    if (z.tall) {  // X B, B symmetric
      a.ah = w.xh[cur];
      a.al = w.xl[cur];
      a.sa = z.x;
      a.lda = z.cp;
      a.bh = w.bh;
      a.bl = w.bl;
      a.sb = z.a;
      a.ldb = z.mp;
      launch_mm<C, kApply, true, true>("orth_apply", a, z.split, s);
    } else {  // B X
      a.ah = w.bh;
      a.al = w.bl;
      a.sa = z.a;
      a.lda = z.mp;
      a.bh = w.xh[cur];
      a.bl = w.xl[cur];
      a.sb = z.x;
      a.ldb = z.cp;
      launch_mm<C, kApply, true, false>("orth_apply", a, z.split, s);
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
// a singular value.
struct Plan {
  float coef[kMaxSteps][3];
  float growth[kMaxSteps];
};
constexpr double kRange = 15.0;

int make_plan(const float* coef, int steps, Plan& p) {
  static const float kQuintic[3] = {3.4445f, -4.7750f, 2.0315f};
  double s = 1.0 + 1e-3;
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
  }
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
  pre.xh = w.xh[0];
  pre.xl = w.xl[0];
  pre.rows = rows;
  pre.cols = cols;
  pre.rp = z.rp;
  pre.cp = z.cp;
  pre.chunks = z.chunks;
  pre.steps = steps;
  pre.eps = eps;
  for (int i = 0; i < steps; ++i) pre.growth[i] = plan.growth[i];
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
  const int kind = st.w ? kOutW : kOutO;
  const int64_t big = cdiv(z.rp, 256) * cdiv(z.cp, 256) * E;
  if (big >= 256) run_products<Tile<256, 32>>(z, w, a, plan.coef, kind, s);
  else run_products<Tile<128, 32>>(z, w, a, plan.coef, kind, s);
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
  return run(g, dtype, E, rows, cols, steps, coef, eps, st, w_out, ws, ws_bytes, static_cast<hipStream_t>(stream));
}
