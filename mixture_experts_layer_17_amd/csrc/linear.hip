// Dense product with bias, activation and residual in its epilogue, and its
// backward: the shared expert beside the routed ones.
//
//   forward   z = x W + bias,  y = act(z) + residual
//   backward  dz = dy act'(z)  (one pass, which also sums db by row chunks),
//             dx = (dz W^T) in_act'(in_z) + dres,  dw = x^T dz
//
// bf16 runs on v_mfma_f32_32x32x16_bf16 with the tiles of the grouped expert
// products: operands go from global memory straight into LDS rings and are read
// from there as they lie, contiguous along the contraction or along their rows or
// columns, so that no operand is transposed.  fp32 runs on v_mfma_f32_32x32x2_f32
// with tiles staged through registers, for any size and alignment.
//
// dz goes into the bf16 products rounded to bf16, which is what the instruction takes:
// its rounding and the result's come to 1.4 times the result's own (8192 x 2048 x 1024,
// silu: 2.35e-3 of dw in the root of mean squares, 1.66e-3 without); as two bf16 parts
// it would double both products (47 and 43 of 118 us).  db is summed before it.
//
// 16-byte loads need rows of whole 16 bytes: a bf16 operand with an odd row
// length is first copied into the workspace with padded rows (zeros behind).
//
// Few output tiles leave compute units idle; then the contraction is split over
// workgroups, which write fp32 sums, and a second launch adds them in order and
// applies the epilogue.
#include "gemm_bf16_tile.hpp"

namespace moe {
namespace {
using namespace gemm;

constexpr int kCUs = 256;
constexpr int64_t kMaxWidth = 1 << 20;

enum { kActNone = MOE_ACT_NONE, kActRelu = MOE_ACT_RELU, kActSilu = MOE_ACT_SILU, kActGelu = MOE_ACT_GELU };

// v[i] = act(v[i]), and v[i] *= act'(z[i]); one choice for all eight.
__device__ __forceinline__ void act8(float (&v)[8], int act) {
  if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = silu_f(v[i]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.5f * v[i] * erfcf(-0.70710678f * v[i]);
  } else if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] > 0.f || v[i] != v[i] ? v[i] : 0.f;
  }
}
__device__ __forceinline__ void times_dact8(float (&v)[8], const float (&z)[8], int act) {
  if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = sigmoid_f(z[i]);
      v[i] *= s * (1.0f + z[i] * (1.0f - s));
    }
  } else if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= 0.5f * erfcf(-0.70710678f * z[i]) + z[i] * 0.39894228f * __expf(-0.5f * z[i] * z[i]);
  } else if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= z[i] > 0.f ? 1.f : 0.f;
  }
}

// ---------------------------------------------------------------------------
// Eight consecutive columns of a row: the whole epilogue.
// ---------------------------------------------------------------------------
struct Epilogue {
  const void* bias;  // [cols]
  void* z;           // the pre-activation, kept for the backward
  const void* in_z;  // times in_act'(in_z)
  const void* add;   // residual or dres
  void* out;
  int act, in_act;
  int64_t ld;        // of all of them: the number of columns
};

template <class T>
__device__ __forceinline__ void read8(const void* p, int64_t i, int valid, bool vec, float (&x)[8]) {
  const T* q = static_cast<const T*>(p) + i;
  if (vec) {
#pragma unroll
    for (int u = 0; u < 8; u += Elem<T>::kVec) Elem<T>::unpack(*reinterpret_cast<const uint4*>(q + u), x + u);
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = u < valid ? Elem<T>::load1(q, u) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void write8(void* p, int64_t i, int valid, bool vec, const float (&x)[8]) {
  T* q = static_cast<T*>(p) + i;
  if (vec) {
#pragma unroll
    for (int u = 0; u < 8; u += Elem<T>::kVec) *reinterpret_cast<uint4*>(q + u) = Elem<T>::pack(x + u);
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (u < valid) Elem<T>::store1(q, u, x[u]);
  }
}

template <class T>
__device__ __forceinline__ void apply8(const Epilogue& e, int64_t row, int col, float (&v)[8]) {
  const int valid = e.ld - col < 8 ? static_cast<int>(e.ld - col) : 8;
  const bool vec = valid == 8 && e.ld % Elem<T>::kVec == 0;
  const int64_t o = row * e.ld + col;
  float u[8];
  if (e.bias) {
    read8<T>(e.bias, col, valid, valid == 8, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += u[i];
  }
  if (e.z) write8<T>(e.z, o, valid, vec, v);
  act8(v, e.act);
  if (e.in_act != kActNone) {
    read8<T>(e.in_z, o, valid, vec, u);
    times_dact8(v, u, e.in_act);
  }
  if (e.add) {
    read8<T>(e.add, o, valid, vec, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += u[i];
  }
  write8<T>(e.out, o, valid, vec, v);
}

// One product: out [rows, cols] = A B over `depth`, A(row, k), B(k, col).
struct Product {
  const void* a;
  const void* b;
  int64_t lda, ldb;
  int64_t rows;
  int cols;
  int64_t depth;
  int gm, gn;        // tiles
  int splits;        // workgroups that share a tile's contraction
  int64_t per_split; // contraction of one of them, whole K steps
  float* part;       // [splits][rows][part_ld] where splits > 1
  int64_t part_ld;
  Epilogue epi;
};

constexpr int kGroupRows = 4;  // row tiles taken together, column tile by column tile

// Tile of workgroup id: XCDs take contiguous ranges, and inside a range
// neighbours share row or column operands in one L2.
__device__ __forceinline__ bool product_tile(const Product& p, int64_t id, int& mt, int& nt, int& split) {
  const int64_t lid = xcd_tile(id, static_cast<int64_t>(p.gm) * p.gn * p.splits);
  if (lid < 0) return false;
  const int64_t tiles = static_cast<int64_t>(p.gm) * p.gn;
  split = static_cast<int>(lid / tiles);
  const int64_t t = lid - split * tiles;
  const int64_t band = t / (static_cast<int64_t>(kGroupRows) * p.gn);
  const int m0 = static_cast<int>(band) * kGroupRows;
  const int h = p.gm - m0 < kGroupRows ? p.gm - m0 : kGroupRows;
  const int64_t r = t - band * kGroupRows * p.gn;
  nt = static_cast<int>(r / h);
  mt = m0 + static_cast<int>(r - static_cast<int64_t>(nt) * h);
  return true;
}

// What the epilogue reads of 32 rows of a wave's columns: all of it asked for before any of it is used, and before
// anything is stored (outputs may lie where inputs do, so the compiler would wait for one after the other).
template <class T, class C>
struct EpilogueInputs {
  static constexpr int kQuads = 8 / Elem<T>::kVec;
  uint4 add[C::TN][2][kQuads], in_z[C::TN][2][kQuads];
  __device__ __forceinline__ void load(const Epilogue& e, int64_t rows, int64_t row, int col) {
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int at = col + j * 32 + 16 * c;
        const bool ok = row < rows && at < e.ld;
        const int64_t o = row * e.ld + at;
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          add[j][c][q] = ok && e.add ? *reinterpret_cast<const uint4*>(static_cast<const T*>(e.add) + o + q * Elem<T>::kVec)
                                     : make_uint4(0, 0, 0, 0);
          in_z[j][c][q] = ok && e.in_act != kActNone
                              ? *reinterpret_cast<const uint4*>(static_cast<const T*>(e.in_z) + o + q * Elem<T>::kVec)
                              : make_uint4(0, 0, 0, 0);
        }
      }
  }
};

// The accumulators of a wave (tiles computed transposed): runs of eight columns
// through the epilogue, or as fp32 sums where the contraction is split.
template <class T, class C>
__device__ __forceinline__ void finish(const Acc<C>& acc, const Product& p, int64_t row0, int col0, int split, int lane,
                                       int wm, int wn) {
  const int rl = lane & 31, hc = 8 * (lane >> 5);
  const int64_t first = row0 + wm * C::WTM + rl;
  const int col1 = col0 + wn * C::WTN + hc;
  const Epilogue& e = p.epi;
  if (p.splits == 1 && e.ld % 8 == 0) {
    constexpr int Q = 8 / Elem<T>::kVec;
    uint4 bias[C::TN][2][Q];
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int at = col1 + j * 32 + 16 * c;
          bias[j][c][q] = e.bias && at < e.ld ? *reinterpret_cast<const uint4*>(static_cast<const T*>(e.bias) + at + q * Elem<T>::kVec)
                                              : make_uint4(0, 0, 0, 0);
        }
    constexpr int kAhead = sizeof(T) == 2 ? 2 : 1;  // the next 32 rows' inputs are on their way, where registers allow
    EpilogueInputs<T, C> in[kAhead];
    if (kAhead == 2) in[0].load(e, p.rows, first, col1);
#pragma unroll
    for (int i = 0; i < C::TM; ++i) {
      const int64_t row = first + i * 32;
      if (kAhead == 1) in[0].load(e, p.rows, row, col1);
      else if (i + 1 < C::TM) in[(i + 1) % kAhead].load(e, p.rows, row + 32, col1);
#pragma unroll
      for (int j = 0; j < C::TN; ++j) {
        float v[2][8];
        to_chunks(acc[i][j], v);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int at = col1 + j * 32 + 16 * c;
          if (row < p.rows && at < e.ld) {
            const int64_t o = row * e.ld + at;
            float u[8];
#pragma unroll
            for (int q = 0; q < Q; ++q) Elem<T>::unpack(bias[j][c][q], u + q * Elem<T>::kVec);
#pragma unroll
            for (int t = 0; t < 8; ++t) v[c][t] += u[t];
            if (e.z) write8<T>(e.z, o, 8, true, v[c]);
            act8(v[c], e.act);
            if (e.in_act != kActNone) {
#pragma unroll
              for (int q = 0; q < Q; ++q) Elem<T>::unpack(in[i % kAhead].in_z[j][c][q], u + q * Elem<T>::kVec);
              times_dact8(v[c], u, e.in_act);
            }
            if (e.add) {
#pragma unroll
              for (int q = 0; q < Q; ++q) Elem<T>::unpack(in[i % kAhead].add[j][c][q], u + q * Elem<T>::kVec);
#pragma unroll
              for (int t = 0; t < 8; ++t) v[c][t] += u[t];
            }
            write8<T>(e.out, o, 8, true, v[c]);
          }
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < C::TM; ++i) {
    const int64_t row = first + i * 32;
#pragma unroll
    for (int j = 0; j < C::TN; ++j) {
      float v[2][8];
      to_chunks(acc[i][j], v);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = col1 + j * 32 + 16 * c;
        if (row < p.rows && col < p.cols) {
          if (p.splits > 1) {
            float* q = p.part + (split * p.rows + row) * p.part_ld + col;
            *reinterpret_cast<float4*>(q) = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
            *reinterpret_cast<float4*>(q + 4) = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
          } else {
            apply8<T>(e, row, col, v[c]);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// bf16
// ---------------------------------------------------------------------------
// A K step of the wide tile takes 1.6 us on a full chip at all three layouts (8192 x 4096 x 2048: 1130 to 1160 TFLOP/s,
// a large library product's rate), behind 15 us of launch, first loads and epilogue; 128 x 128 tiles take 1.0 us for two.
using Wide = Cfg<256, 256, 2, 4, 64, 2, 2, 1, true>;   // one workgroup per CU
using Narrow = Cfg<128, 128, 2, 2, 64, 2, 2, 1, true>; // two

// One K step of an operand contiguous along the contraction; rows past the
// last one and chunks past the contraction's end read as zero.
template <class C, int ROWS>
__device__ __forceinline__ void load_kc(const uint16_t* base, int64_t ld, int rows, int k0, int k_end, uint16_t* dst,
                                        int wave, int lane) {
  constexpr int CPR = C::BK / 8, RPI = 64 / CPR, NI = ROWS / RPI;
  static_assert(NI % C::kWaves == 0, "tile rows over the waves");
  const __amdgpu_buffer_rsrc_t r = rsrc(base, static_cast<int64_t>(rows < ROWS ? rows : ROWS) * ld * 2);
  const int rl = lane / CPR, ph = lane % CPR;
#pragma unroll
  for (int u = 0; u < NI / C::kWaves; ++u) {
    const int i = wave + u * C::kWaves;
    const int row = i * RPI + rl;
    const int k = k0 + (ph ^ kc_swz<C::BK>(row)) * 8;
    dma16(r, dst + i * 512, k < k_end ? static_cast<int>((row * ld + k) * 2) : 0x7FFFFFF0);
  }
}

// One K step: slice by slice fragments and products, with issue(slice) first (the next step's loads).  The stages come as
// restricted pointers: only then does the compiler know that the loads on their way into the other stages do not touch
// them, and does not wait for all of those before each transposing read.
template <class C, bool AKC, bool BKC, class F>
__device__ __forceinline__ void multiply_step(const uint16_t* __restrict__ As, const uint16_t* __restrict__ Bs, int wm, int wn,
                                              int lane, Acc<C>& acc, F&& issue) {
#pragma unroll
  for (int ks = 0; ks < C::BK / 16; ++ks) {
    issue(ks);
    bf16x8 a[C::TM], b[C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
      a[i] = AKC ? frag_kc<C>(As, wm * C::WTM + i * 32, ks, lane) : frag_mc<C, C::BM>(As, wm * C::WTM + i * 32, ks, lane);
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
      b[j] = BKC ? frag_kc<C>(Bs, wn * C::WTN + j * 32, ks, lane) : frag_mc<C, C::BN>(Bs, wn * C::WTN + j * 32, ks, lane);
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
  }
}

template <class C, bool AKC, bool BKC>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(C::kWavesPerSimd)))
void linear_bf16_kernel(Product p) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[C::kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  int mt, nt, split;
  if (!product_tile(p, blockIdx.x, mt, nt, split)) return;
  mt = __builtin_amdgcn_readfirstlane(mt);
  nt = __builtin_amdgcn_readfirstlane(nt);
  split = __builtin_amdgcn_readfirstlane(split);
  const int64_t row0 = static_cast<int64_t>(mt) * C::BM;
  const int col0 = nt * C::BN;
  const int64_t k0 = split * p.per_split;
  const int64_t len = p.depth - k0 < p.per_split ? p.depth - k0 : p.per_split;
  const int nk = static_cast<int>((len + C::BK - 1) / C::BK);
  const uint16_t* A = static_cast<const uint16_t*>(p.a);
  const uint16_t* B = static_cast<const uint16_t*>(p.b);
  const int rows = static_cast<int>(p.rows - row0 < C::BM ? p.rows - row0 : C::BM);
  const int cols = p.cols - col0 < C::BN ? p.cols - col0 : C::BN;

  auto load_a = [&](int kt) {
    uint16_t* st = lds + (kt & 1) * C::kA;
    if constexpr (AKC)
      load_kc<C, C::BM>(A + row0 * p.lda, p.lda, rows, static_cast<int>(k0) + kt * C::BK, static_cast<int>(p.depth), st, wave, lane);
    else
      dma_mc<C, C::BM, 1>(McOp{A + k0 * p.lda, nullptr, p.lda, static_cast<int>(row0), static_cast<int>(len)}, kt * C::BK,
                          st, wave, lane);
  };
  auto load_b = [&](int kt) {
    uint16_t* st = lds + C::kBOff + (kt & 1) * C::kB;
    if constexpr (BKC)
      load_kc<C, C::BN>(B + col0 * p.ldb, p.ldb, cols, static_cast<int>(k0) + kt * C::BK, static_cast<int>(p.depth), st, wave, lane);
    else
      dma_mc<C, C::BN, 1>(McOp{B + k0 * p.ldb, nullptr, p.ldb, col0, static_cast<int>(len)}, kt * C::BK, st, wave, lane);
  };

  Acc<C> acc;
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  load_a(0);
  load_b(0);
  for (int kt = 0; kt < nk; ++kt) {
    wait_vm<0>();
    __syncthreads();
    const bool more = kt + 1 < nk;
    multiply_step<C, AKC, BKC>(lds + (kt & 1) * C::kA, lds + C::kBOff + (kt & 1) * C::kB, wm, wn, lane, acc, [&](int ks) {
      if (more && ks == 0) load_a(kt + 1);
      if (more && ks == 1) load_b(kt + 1);
    });
  }
  finish<uint16_t, C>(acc, p, row0, col0, split, lane, wm, wn);
}

// ---------------------------------------------------------------------------
// fp32: square tiles on four waves, both operands in LDS with the contraction
// along the rows.  The next steps' values are on their way into registers while a
// step is multiplied: two of the 128 x 128 tiles' (4096^3: 1177 -> 1073 us), one
// of the 64 x 64 tiles', which spread a small product over the chip and take 64 of
// the contraction a step, so that a step outlasts its loads (1001 x 333 x 777:
// 17 us, 19 with two ahead).
// ---------------------------------------------------------------------------
template <int BT, int BK_, int AHEAD>
struct Tile32 {
  static constexpr int kAhead = AHEAD;
  static constexpr int BM = BT, BN = BT, BK = BK_, WN = 2, kThreads = 256;
  static constexpr int WTM = BT / 2, WTN = BT / 2, TM = WTM / 32, TN = WTN / 32;
  static constexpr int kN = BT * BK / 4 / kThreads;  // 16-byte vectors a thread brings per operand and step
  // row length in LDS: rows written across (KC) start in banks of their own, whole rows on 16 bytes
  static constexpr int ld(bool kc) { return kc ? BT + 1 : BT + 4; }
};
using Large32 = Tile32<128, 32, 2>;
using Small32 = Tile32<64, 64, 1>;

// This thread's values of a BK x BT tile.  KC: element (i, k) at p[i ld + k], p at the tile's first row, n rows; else at
// p[k ld + col0 + i].  The step starts at k0 of the contraction, of which `left` are there.  Buffer loads need no more
// than 4-byte alignment and give zero past the last row; a KC row's end is masked, and what lies past the columns of
// the others goes into outputs that nobody stores.
template <class C, bool KC>
__device__ __forceinline__ void fetch32(const float* p, int64_t ld, int n, int col0, int64_t k0, int64_t left, int tid,
                                        float (&v)[C::kN][4]) {
  typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
  const __amdgpu_buffer_rsrc_t r =
      KC ? rsrc(p, (n < C::BM ? n : C::BM) * ld * 4) : rsrc(p + k0 * ld, (left < C::BK ? left : C::BK) * ld * 4);
#pragma unroll
  for (int u = 0; u < C::kN; ++u) {
    const int id = tid + u * C::kThreads;
    const int i = KC ? id / (C::BK / 4) : id % (C::BM / 4) * 4;
    const int k = KC ? id % (C::BK / 4) * 4 : id / (C::BM / 4);
    const int64_t at = KC ? i * ld + k0 + k : k * ld + col0 + i;
    const u32x4 f = __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(at * 4), 0, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s) v[u][s] = KC && k + s >= left ? 0.f : __uint_as_float(f[s]);
  }
}
template <class C, bool KC>
__device__ __forceinline__ void place32(float* t, int tid, const float (&v)[C::kN][4]) {
#pragma unroll
  for (int u = 0; u < C::kN; ++u) {
    const int id = tid + u * C::kThreads;
    if constexpr (KC) {
#pragma unroll
      for (int s = 0; s < 4; ++s) t[(id % (C::BK / 4) * 4 + s) * C::ld(true) + id / (C::BK / 4)] = v[u][s];
    } else {
      *reinterpret_cast<float4*>(t + id / (C::BM / 4) * C::ld(false) + id % (C::BM / 4) * 4) = make_float4(v[u][0], v[u][1], v[u][2], v[u][3]);
    }
  }
}

template <class C, bool AKC, bool BKC>
__global__ __launch_bounds__(C::kThreads) __attribute__((amdgpu_waves_per_eu(2))) void linear_f32_kernel(Product p) {
  constexpr int lda = C::ld(AKC), ldb = C::ld(BKC);
  __shared__ __attribute__((aligned(16))) float as[2][C::BK * lda], bs[2][C::BK * ldb];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  int mt, nt, split;
  if (!product_tile(p, blockIdx.x, mt, nt, split)) return;
  const int64_t row0 = static_cast<int64_t>(mt) * C::BM;
  const int col0 = nt * C::BN;
  const int64_t k0 = split * p.per_split;
  const int64_t len = p.depth - k0 < p.per_split ? p.depth - k0 : p.per_split;
  const int nk = static_cast<int>((len + C::BK - 1) / C::BK);
  const float* A = static_cast<const float*>(p.a) + (AKC ? row0 * p.lda : 0);
  const float* B = static_cast<const float*>(p.b) + (BKC ? col0 * p.ldb : 0);
  const int rows = static_cast<int>(p.rows - row0 < C::BM ? p.rows - row0 : C::BM);
  const int cols = p.cols - col0 < C::BN ? p.cols - col0 : C::BN;

  Acc<C> acc;
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  struct Values {
    float a[C::kN][4], b[C::kN][4];
  };
  // (past the last step: zeros, by the buffers' ends and the mask)
  auto fetch = [&](int kt, Values& v) {
    const int64_t k = static_cast<int64_t>(kt) * C::BK;
    fetch32<C, AKC>(A, p.lda, rows, static_cast<int>(row0), k0 + k, len - k, tid, v.a);
    fetch32<C, BKC>(B, p.ldb, cols, col0, k0 + k, len - k, tid, v.b);
  };
  auto step = [&](int kt, Values& v) {
    const int st = kt & 1;
    place32<C, AKC>(as[st], tid, v.a);
    place32<C, BKC>(bs[st], tid, v.b);
    __syncthreads();  // also: every wave is past the step before last, whose stage this was
    fetch(kt + C::kAhead, v);
#pragma unroll 8
    for (int k = 0; k < C::BK; k += 2) {
      const int kr = k + (lane >> 5);
      float a[C::TM], b[C::TN];
#pragma unroll
      for (int i = 0; i < C::TM; ++i) a[i] = as[st][kr * lda + wm * C::WTM + i * 32 + (lane & 31)];
#pragma unroll
      for (int j = 0; j < C::TN; ++j) b[j] = bs[st][kr * ldb + wn * C::WTN + j * 32 + (lane & 31)];
#pragma unroll
      for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(b[j], a[i], acc[i][j], 0, 0, 0);
    }
  };
  Values even, odd;
  fetch(0, even);
  if constexpr (C::kAhead == 2) {
    fetch(1, odd);
    for (int kt = 0; kt < nk; kt += 2) {
      step(kt, even);
      if (kt + 1 < nk) step(kt + 1, odd);
    }
  } else {
    for (int kt = 0; kt < nk; ++kt) step(kt, even);
  }
  finish<float, C>(acc, p, row0, col0, split, lane, wm, wn);
}

// ---------------------------------------------------------------------------
// Up to four rows: bound by reading w, so no tiles.  A workgroup takes 32 columns
// (16 where that leaves half the chip idle) and the whole contraction: lanes of
// 16 bytes of a row of w, eight such loads in flight a lane; x comes through LDS
// in fp32.  One launch: no split, whose second launch costs more than it gains
// here (one row, 2048 x 1024 bf16: 13.8 us with it, 10.4 with 32 columns a workgroup).
// ---------------------------------------------------------------------------
constexpr int kFewRows = 4;
constexpr int kFewChunk = 4096;           // of the contraction at a time in LDS
constexpr int64_t kFewDepth = 8192;       // past it a workgroup would read too long alone

template <class T, int R, int kFewCols>
__global__ __launch_bounds__(256) void linear_few_kernel(Product p) {
  constexpr int V = Elem<T>::kVec, L = kFewCols / V, KL = 256 / L;
  __shared__ float xs[R][kFewChunk];
  __shared__ float sums[4][R][kFewCols];
  const int tid = threadIdx.x, cl = tid % L, kl = tid / L;
  const int col = blockIdx.x * kFewCols + cl * V;
  const bool in = col < p.cols;           // whole vectors: cols is a multiple of V
  const T* w = static_cast<const T*>(p.b) + col;
  float acc[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) acc[r][v] = 0.f;
  for (int64_t k0 = 0; k0 < p.depth; k0 += kFewChunk) {
    const int n = static_cast<int>(p.depth - k0 < kFewChunk ? p.depth - k0 : kFewChunk);
    if (k0 > 0) __syncthreads();
    for (int r = 0; r < R; ++r)
      for (int k = tid; k < n; k += 256) xs[r][k] = r < p.rows ? Elem<T>::load1(p.a, r * p.lda + k0 + k) : 0.f;
    __syncthreads();
    if (in) {
      for (int k = kl; k < n; k += 8 * KL) {
        uint4 q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int kk = k + u * KL;
          q[u] = *reinterpret_cast<const uint4*>(w + (k0 + (kk < n ? kk : k)) * p.ldb);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int kk = k + u * KL;
          float f[V];
          Elem<T>::unpack(q[u], f);
          if (kk < n) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const float xv = xs[r][kk];
#pragma unroll
              for (int v = 0; v < V; ++v) acc[r][v] = fmaf(xv, f[v], acc[r][v]);
            }
          }
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int o = 32; o >= L; o >>= 1) acc[r][v] += __shfl_xor(acc[r][v], o, 64);
      if ((tid & 63) < L) sums[tid >> 6][r][cl * V + v] = acc[r][v];
    }
  __syncthreads();
  if (tid < R * (kFewCols / 8)) {
    const int r = tid / (kFewCols / 8), c = tid % (kFewCols / 8) * 8;
    const int at = blockIdx.x * kFewCols + c;
    if (r < p.rows && at < p.cols) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = (sums[0][r][c + i] + sums[1][r][c + i]) + (sums[2][r][c + i] + sums[3][r][c + i]);
      apply8<T>(p.epi, r, at, v);
    }
  }
}

// ---------------------------------------------------------------------------
// The sums of a split contraction, added in order, through the epilogue.
// ---------------------------------------------------------------------------
template <class T>
__global__ __launch_bounds__(256) void linear_join_kernel(Product p) {
  const uint32_t per = static_cast<uint32_t>(p.part_ld / 8), i = blockIdx.x * 256u + threadIdx.x;  // fewer than 2^32
  if (i >= p.rows * per) return;
  const int64_t row = i / per;
  const int col = static_cast<int>(i % per) * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) {
    const float* q = p.part + (s * p.rows + row) * p.part_ld + col;
    const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
    v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
    v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
  }
  apply8<T>(p.epi, row, col, v);
}

// dst [rows, ld] = src [rows, cols], zeros behind (bf16, ld a multiple of 8).  A
// thread's eight values start anywhere on 2 bytes: they come as the five words
// that hold them, shifted by half a word where the first is a word's upper half;
// only at the very end, where those would pass it, one by one.
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ src, int64_t rows, int cols, int ld,
                                                       uint16_t* __restrict__ dst) {
  typedef uint32_t words __attribute__((ext_vector_type(4), aligned(4)));
  const uint32_t per = ld / 8, i = blockIdx.x * 256u + threadIdx.x;  // fewer than 2^32
  if (i >= rows * per) return;
  const int64_t row = i / per;
  const int c = static_cast<int>(i % per) * 8;
  const int64_t o = row * cols + c;
  uint32_t w[4];
  if (o + 10 <= rows * cols) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(src) + (o >> 1);
    const words v = *reinterpret_cast<const words*>(q);
    const uint32_t f[5] = {v[0], v[1], v[2], v[3], q[4]};
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = o & 1 ? f[u] >> 16 | f[u + 1] << 16 : f[u];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (c + 2 * u >= cols) w[u] = 0;
      else if (c + 2 * u + 1 >= cols) w[u] &= 0xFFFFu;
    }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      w[u] = c + 2 * u < cols ? src[o + 2 * u] : 0;
      if (c + 2 * u + 1 < cols) w[u] |= static_cast<uint32_t>(src[o + 2 * u + 1]) << 16;
    }
  }
  *reinterpret_cast<uint4*>(dst + row * ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
}

// ---------------------------------------------------------------------------
// dz = dy act'(z) and its column sums over chunks of rows.  A workgroup takes a
// chunk and 512 columns: 64 lanes of eight columns, four rows at a time.  8192 x
// 1024 bf16: 11 us, 4.6 TB/s.
// ---------------------------------------------------------------------------
struct DzArgs {
  const void* dy;
  const void* z;     // null: no activation
  int64_t rows, chunk;
  int cols, ld_dz;
  int act;
  void* dz;          // null: not written
  float* part;       // [chunks][part_ld], null: no sums
  int64_t part_ld;
};

template <class T>
__global__ __launch_bounds__(256) void linear_dz_kernel(DzArgs p) {
  __shared__ float sums[4][512];
  const int lane = threadIdx.x & 63, phase = threadIdx.x >> 6;
  const int col = (blockIdx.x * 64 + lane) * 8;
  const int64_t r0 = blockIdx.y * p.chunk, r1 = r0 + p.chunk < p.rows ? r0 + p.chunk : p.rows;
  const int valid = p.cols - col < 8 ? p.cols - col : 8;
  const bool vec = valid == 8 && p.cols % Elem<T>::kVec == 0;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (valid > 0) {
#pragma unroll 2
    for (int64_t r = r0 + phase; r < r1; r += 4) {
      float g[8], z[8];
      read8<T>(p.dy, r * p.cols + col, valid, vec, g);
      if (p.z) {
        read8<T>(p.z, r * p.cols + col, valid, vec, z);
        times_dact8(g, z, p.act);
      }
      // behind the last column: zeros, as the products need them (ld_dz is a multiple of 8 for bf16)
      if (p.dz) write8<T>(p.dz, r * p.ld_dz + col, p.ld_dz - col < 8 ? p.ld_dz - col : 8, p.ld_dz % Elem<T>::kVec == 0 && p.ld_dz - col >= 8, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += g[i];
    }
  }
  if (!p.part) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[phase][lane * 8 + i] = acc[i];
  __syncthreads();
  for (int c = threadIdx.x; c < 512; c += 256) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 512 + c;
    if (at < p.cols) p.part[blockIdx.y * p.part_ld + at] = (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
  }
}

// db = the chunks' sums in order: 16 columns by 16 parts of the chunks, each part's loads eight at a time.
template <class T>
__global__ __launch_bounds__(256) void linear_db_kernel(const float* __restrict__ part, int64_t part_ld, int64_t chunks,
                                                        int cols, T* __restrict__ db) {
  __shared__ float sums[16][16];
  const int c = threadIdx.x & 15, ph = threadIdx.x >> 4;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 16 + c;
  float acc = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int64_t k = ph; k < chunks; k += 16) acc += part[k * part_ld + col];
  }
  sums[ph][c] = acc;
  __syncthreads();
  if (ph == 0 && col < cols) {
    acc = 0.f;
#pragma unroll
    for (int q = 0; q < 16; ++q) acc += sums[q][c];
    Elem<T>::store1(db, col, acc);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
int64_t up8(int64_t n) { return (n + 7) & ~int64_t{7}; }

struct Plan {
  bool wide;
  int splits;
  int64_t per_split, part_ld;
  size_t part_bytes;
};

// The two tile sizes of a type: BT x BT outputs, K steps of bk, workgroups that a compute unit holds at once, and what
// was measured (us): a K step with one workgroup on a unit and with all that fit, first loads and epilogue likewise.
struct TileCost {
  int bt, bk, per_cu;
  double step1, step, fixed1, fixed;
};
constexpr TileCost kTiles[2][2] = {
    {{64, 64, 2, 1.6, 2.9, 4.0, 5.0}, {128, 32, 2, 2.3, 4.1, 7.0, 8.0}},        // fp32
    {{128, 64, 2, 0.67, 1.0, 5.0, 5.0}, {256, 64, 1, 1.2, 1.6, 5.0, 11.0}},     // bf16
};

// Tile size and split of a product by the estimated time: whole rounds of workgroups over the chip and what is left
// behind them, plus the second launch of a split.
Plan plan_product(int dtype, int64_t rows, int64_t cols, int64_t depth) {
  Plan best{};
  double least = 1e300;
  for (int wide = 0; wide < 2; ++wide) {
    const TileCost& c = kTiles[dtype == MOE_BF16][wide];
    const int64_t steps = cdiv(depth, c.bk), tiles = cdiv(rows, c.bt) * cdiv(cols, c.bt), slots = c.per_cu * kCUs;
    for (int s = 1; s <= 64; s *= 2) {
      const int64_t per = cdiv(steps, s);
      if (s > 1 && (per < 2 || cdiv(steps, per) <= s / 2)) break;
      const int n = static_cast<int>(cdiv(steps, per));
      const double bytes = n > 1 ? (n + 1.0) * rows * cols * 4 : 0;
      if (bytes > 1.0e9) break;
      const int64_t groups = tiles * n, left = groups % slots;
      double t = groups / slots * (per * c.step + c.fixed);
      if (left > 0) {
        const double full = c.per_cu == 1 ? static_cast<double>(left) / kCUs : left > kCUs ? 1.0 : 0.0;
        t += per * (c.step1 + full * (c.step - c.step1)) + c.fixed1 + full * (c.fixed - c.fixed1);
      }
      if (n > 1) t += 5.0 + bytes / 3.0e6;
      if (t < least) {
        least = t;
        best = Plan{wide != 0, n, per * c.bk, up8(cols), n > 1 ? align_up(static_cast<size_t>(n) * rows * up8(cols) * 4, 256) : 0};
      }
    }
  }
  return best;
}

template <class T, bool AKC, bool BKC>
int launch_product(const void* a, int64_t lda, const void* b, int64_t ldb, int64_t rows, int64_t cols, int64_t depth,
                   const Epilogue& epi, void* part, const char* name, hipStream_t s) {
  constexpr bool bf = sizeof(T) == 2;
  const Plan pl = plan_product(bf ? MOE_BF16 : MOE_F32, rows, cols, depth);
  const int bt = kTiles[bf][pl.wide].bt;
  Product p{a, b, lda, ldb, rows, static_cast<int>(cols), depth, static_cast<int>(cdiv(rows, bt)),
            static_cast<int>(cdiv(cols, bt)), pl.splits, pl.per_split, static_cast<float*>(part), pl.part_ld, epi};
  const dim3 grid(xcd_grid(static_cast<int64_t>(p.gm) * p.gn * p.splits));
  if constexpr (bf) {
    if (pl.wide) MOE_LAUNCH(name, (linear_bf16_kernel<Wide, AKC, BKC>), grid, dim3(Wide::kThreads), 0, s, p);
    else MOE_LAUNCH(name, (linear_bf16_kernel<Narrow, AKC, BKC>), grid, dim3(Narrow::kThreads), 0, s, p);
  } else {
    if (pl.wide) MOE_LAUNCH(name, (linear_f32_kernel<Large32, AKC, BKC>), grid, dim3(Large32::kThreads), 0, s, p);
    else MOE_LAUNCH(name, (linear_f32_kernel<Small32, AKC, BKC>), grid, dim3(Small32::kThreads), 0, s, p);
  }
  if (p.splits > 1)
    MOE_LAUNCH("linear_join", linear_join_kernel<T>, dim3(static_cast<unsigned>(cdiv(rows * (pl.part_ld / 8), 256))),
               dim3(256), 0, s, p);
  return launch_status();
}

void launch_pad(const void* src, int64_t rows, int64_t cols, void* dst, hipStream_t s) {
  const int64_t ld = up8(cols);
  MOE_LAUNCH("linear_pad", pad_rows_kernel, dim3(static_cast<unsigned>(cdiv(rows * (ld / 8), 256))), dim3(256), 0, s,
             static_cast<const uint16_t*>(src), rows, static_cast<int>(cols), static_cast<int>(ld), static_cast<uint16_t*>(dst));
}

// Rows per workgroup of the dz pass: about four workgroups per compute unit.
int64_t dz_chunk(int64_t M, int64_t N) {
  const int64_t c = cdiv(M * cdiv(N, 512), 4 * kCUs);
  return (c < 16 ? 16 : c + 3) & ~int64_t{3};
}

struct Buffers {
  size_t x, w, dz, sums, part, total;
};
Buffers buffers(int dtype, int64_t M, int64_t K, int64_t N, bool bwd) {
  Buffers b{};
  b.total = 256;
  if (M == 0) return b;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t o = at;
    at += align_up(n, 256);
    return o;
  };
  if (dtype == MOE_BF16) {
    b.x = take(K % 8 ? static_cast<size_t>(M) * up8(K) * 2 : 0);
    b.w = take(N % 8 ? static_cast<size_t>(K) * up8(N) * 2 : 0);
  }
  if (bwd) {
    b.dz = take(dtype == MOE_BF16 ? static_cast<size_t>(M) * up8(N) * 2 : static_cast<size_t>(M) * N * 4);
    b.sums = take(static_cast<size_t>(cdiv(M, dz_chunk(M, N))) * up8(N) * 4);
    const size_t dx = plan_product(dtype, M, K, N).part_bytes, dw = plan_product(dtype, K, N, M).part_bytes;
    b.part = take(dx > dw ? dx : dw);
  } else {
    b.part = take(plan_product(dtype, M, N, K).part_bytes);
  }
  if (at > b.total) b.total = at;
  return b;
}

// Whether a product's launch stays below 2^32 threads (its tiles have two to four a row, so many rows of few columns do
// not).
bool product_fits(int dtype, int64_t rows, int64_t cols, int64_t depth) {
  const Plan pl = plan_product(dtype, rows, cols, depth);
  const int bt = kTiles[dtype == MOE_BF16][pl.wide].bt;
  const int64_t threads = dtype == MOE_BF16 && pl.wide ? Wide::kThreads : 256;
  return xcd_grid(cdiv(rows, bt) * cdiv(cols, bt) * pl.splits) * threads < (1ll << 32);
}

// 2^32 threads in one launch are too many: those beside the products have a thread per eight elements at most.
int linear_sizes(int dtype, int64_t M, int64_t K, int64_t N, bool bwd) {
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || M < 0 || K < 1 || N < 1) return MOE_EINVAL;
  if (M >= (1ll << 31) || K > kMaxWidth || N > kMaxWidth) return MOE_EUNSUPPORTED;
  const int64_t big = M > K ? M : K, side = K > N ? K : N;
  if (big * up8(side) / 8 >= (1ll << 32) - 256) return MOE_EUNSUPPORTED;
  if (M >= (1ll << 28) && !product_fits(dtype, M, bwd ? K : N, bwd ? N : K)) return MOE_EUNSUPPORTED;  // (dw's is far below)
  return MOE_OK;
}
bool act_ok(int act) { return act >= kActNone && act <= kActGelu; }

// Whether linear_few_kernel takes the product.
template <class T>
bool few_rows(int64_t M, int64_t K, int64_t N) {
  return M <= kFewRows && K <= kFewDepth && N % Elem<T>::kVec == 0;
}

template <class T, int R>
int launch_few(const Product& p, hipStream_t s) {
  if (cdiv(p.cols, 32) >= kCUs / 2)
    MOE_LAUNCH("linear_few", (linear_few_kernel<T, R, 32>), dim3(static_cast<unsigned>(cdiv(p.cols, 32))), dim3(256), 0, s, p);
  else
    MOE_LAUNCH("linear_few", (linear_few_kernel<T, R, 16>), dim3(static_cast<unsigned>(cdiv(p.cols, 16))), dim3(256), 0, s, p);
  return launch_status();
}

template <class T>
int linear_fwd(const void* x, const void* w, const void* bias, const void* residual, int64_t M, int64_t K, int64_t N,
               int act, void* y, void* z, char* ws, hipStream_t s) {
  constexpr bool bf = sizeof(T) == 2;
  const Buffers b = buffers(bf ? MOE_BF16 : MOE_F32, M, K, N, false);
  int64_t lda = K, ldb = N, depth = K;
  const Epilogue e{bias, z, nullptr, residual, y, act, kActNone, N};
  if (few_rows<T>(M, K, N)) {
    const Product p{x, w, K, N, M, static_cast<int>(N), K, 1, 1, 1, K, nullptr, 0, e};
    return M == 1 ? launch_few<T, 1>(p, s) : M == 2 ? launch_few<T, 2>(p, s) : launch_few<T, 4>(p, s);
  }
  if (bf && K % 8) {
    launch_pad(x, M, K, ws + b.x, s);
    x = ws + b.x;
    lda = up8(K);
  }
  if (bf && N % 8) {
    launch_pad(w, K, N, ws + b.w, s);
    w = ws + b.w;
    ldb = up8(N);
  }
  return launch_product<T, true, false>(x, lda, w, ldb, M, N, depth, e, ws + b.part, "linear_fwd", s);
}

template <class T>
int linear_bwd(const void* dy, const void* x, const void* w, const void* z, int64_t M, int64_t K, int64_t N, int act,
               const void* in_z, int in_act, const void* dres, void* dx, void* dw, void* db, char* ws, hipStream_t s) {
  constexpr bool bf = sizeof(T) == 2;
  const Buffers b = buffers(bf ? MOE_BF16 : MOE_F32, M, K, N, true);
  const int64_t ldn = bf ? up8(N) : N;
  const void* dz = dy;
  const bool write = (dx || dw) && (act != kActNone || ldn != N);
  if (write || db) {
    const int64_t chunk = dz_chunk(M, N), chunks = cdiv(M, chunk);
    float* sums = reinterpret_cast<float*>(ws + b.sums);
    const DzArgs a{dy, act != kActNone ? z : nullptr, M, chunk, static_cast<int>(N), static_cast<int>(ldn), act,
                   write ? ws + b.dz : nullptr, db ? sums : nullptr, up8(N)};
    MOE_LAUNCH("linear_dz", linear_dz_kernel<T>, dim3(static_cast<unsigned>(cdiv(N, 512)), static_cast<unsigned>(chunks)),
               dim3(256), 0, s, a);
    if (db)
      MOE_LAUNCH("linear_db", linear_db_kernel<T>, dim3(static_cast<unsigned>(cdiv(N, 16))), dim3(256), 0, s, sums, up8(N),
                 chunks, static_cast<int>(N), static_cast<T*>(db));
    if (write) dz = ws + b.dz;
  }
  if (dx) {
    if (bf && N % 8) {
      launch_pad(w, K, N, ws + b.w, s);
      w = ws + b.w;
    }
    const Epilogue e{nullptr, nullptr, in_z, dres, dx, kActNone, in_act, K};
    const int st = launch_product<T, true, true>(dz, ldn, w, ldn, M, K, N, e, ws + b.part, "linear_dx", s);
    if (st != MOE_OK) return st;
  }
  if (dw) {
    int64_t ldx = K;
    if (bf && K % 8) {
      launch_pad(x, M, K, ws + b.x, s);
      x = ws + b.x;
      ldx = up8(K);
    }
    const Epilogue e{nullptr, nullptr, nullptr, nullptr, dw, kActNone, kActNone, N};
    return launch_product<T, false, false>(x, ldx, dz, ldn, K, N, M, e, ws + b.part, "linear_dw", s);
  }
  return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_linear_workspace(int dtype, int64_t M, int32_t K, int32_t N, int is_bwd) {
  if (linear_sizes(dtype, M, K, N, is_bwd != 0) != MOE_OK) return 0;
  return buffers(dtype, M, K, N, is_bwd != 0).total;
}

extern "C" int moe_linear(const void* x, const void* w, const void* bias, const void* residual, int dtype, int64_t M,
                          int32_t K, int32_t N, int act, void* y, void* z, void* ws, size_t ws_bytes, void* stream) {
  const int st = linear_sizes(dtype, M, K, N, false);
  if (st != MOE_OK) return st;
  if (!act_ok(act)) return MOE_EINVAL;
  if (M == 0) return MOE_OK;
  if (!x || !w || !y || !ws) return MOE_EINVAL;
  for (const void* q : {x, w, bias, residual, static_cast<const void*>(y), static_cast<const void*>(z), static_cast<const void*>(ws)})
    if (!aligned16(q)) return MOE_EINVAL;
  if (ws_bytes < buffers(dtype, M, K, N, false).total) return MOE_EWORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* b = static_cast<char*>(ws);
  return dtype == MOE_BF16 ? linear_fwd<uint16_t>(x, w, bias, residual, M, K, N, act, y, z, b, s)
                           : linear_fwd<float>(x, w, bias, residual, M, K, N, act, y, z, b, s);
}

extern "C" int moe_linear_bwd(const void* dy, const void* x, const void* w, const void* z, int dtype, int64_t M,
                              int32_t K, int32_t N, int act, const void* in_z, int in_act, const void* dres, void* dx,
                              void* dw, void* db, void* ws, size_t ws_bytes, void* stream) {
  const int st = linear_sizes(dtype, M, K, N, true);
  if (st != MOE_OK) return st;
  if (!act_ok(act) || !act_ok(in_act)) return MOE_EINVAL;
  if (!dx && (dres || in_act != kActNone)) return MOE_EINVAL;
  if (M > 0 && ((!dy && (dx || dw || db)) || (dx && !w) || (dw && !x) || (act != kActNone && !z) ||
                (in_act != kActNone && !in_z) || !ws))
    return MOE_EINVAL;
  for (const void* q : {dy, x, w, z, in_z, dres, static_cast<const void*>(dx), static_cast<const void*>(dw),
                        static_cast<const void*>(db), static_cast<const void*>(ws)})
    if (!aligned16(q)) return MOE_EINVAL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const size_t es = dtype == MOE_BF16 ? 2 : 4;
  if (M == 0) {
    if (dw) launch_zero(dw, static_cast<size_t>(K) * N * es, s);
    if (db) launch_zero(db, static_cast<size_t>(N) * es, s);
    return launch_status();
  }
  if (ws_bytes < buffers(dtype, M, K, N, true).total) return MOE_EWORKSPACE;
  char* b = static_cast<char*>(ws);
  return dtype == MOE_BF16 ? linear_bwd<uint16_t>(dy, x, w, z, M, K, N, act, in_z, in_act, dres, dx, dw, db, b, s)
                           : linear_bwd<float>(dy, x, w, z, M, K, N, act, in_z, in_act, dres, dx, dw, db, b, s);
}
