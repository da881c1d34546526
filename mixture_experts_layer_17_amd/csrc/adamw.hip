// AdamW step of a list of tensors in few launches, and the values of 8-bit states.
//
// Per element, in fp32:  m' = b1 m + (1 - b1) g,  v' = b2 v + (1 - b2) g^2,
//   w' = w - (lr decay w + lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps))
// One pass: every operand read once and written once, which is what bounds it:
// 50 M bf16 values with fp32 weights and states, 28 bytes each, take 268 us, 5.3 TB/s
// (a large copy reaches 5.2; in place 5.1).  268 M bf16 values with 8-bit states take
// 565 to 625 us, 4.4 to 4.8 TB/s: there the hash, two codes and the root, some 70
// vector operations a value, take about as long as the bytes.
//
// The tensors' addresses and sizes travel in the kernel's arguments (kMaxList a
// launch), so nothing is copied to the device and a captured graph keeps them.
// A workgroup takes a unit of one tensor, found by a search over the
// tensors' first units in scalar registers: four turns of its 256 lanes where there
// is work for every compute unit several times over, else one.
//
// States in 8 bits: m and the root of v as E4M3 codes with one power of two per
// 32 values (a lane holds 8, four lanes a block).  The root has half the range
// of v.  A state moves by a fraction of a step of such a code (v by 1 - b2, a
// thousandth), so rounding to nearest would leave it where it is; it is rounded
// up with the chance that the part cut off gives, from a hash of the seed, the
// step, the tensor and the element, which keeps its expectation and makes the
// step repeatable.  A root above zero is not stored as zero: the next step
// would divide by little more than eps.
#include <cmath>

#include "common.hpp"

namespace moe {
namespace {

constexpr int kMaxList = 56;    // tensors per launch: the arguments stay below 4 KB
constexpr int kThreads = 256;
constexpr int kPer = 8;         // elements per lane and turn: 16 bytes of bf16
constexpr int kTurn = kThreads * kPer;  // elements of a workgroup's turn
constexpr int64_t kMaxUnits = int64_t{1} << 24;  // a launch holds fewer than 2^32 threads

struct ListEntry {
  const void* w;
  const void* g;
  void* w_out;
  int64_t n;
  int64_t offset;  // of its states, in elements
  double lr;
  float rate;      // lr / (1 - beta1^step), for a step counted on the host
  float decay;     // lr weight_decay
  uint32_t seed;
};

struct AdamArgs {
  ListEntry list[kMaxList];
  int32_t first[kMaxList + 1];  // the first unit of each tensor
  int32_t count;
  int32_t turns;                // of a unit
  const void* m;
  const void* v;
  const uint8_t* m_scale;
  const uint8_t* v_scale;
  const float* master;
  void* m_out;
  void* v_out;
  uint8_t* m_scale_out;
  uint8_t* v_scale_out;
  float* master_out;
  double beta1, beta2;
  float b1, b1_low, a1, a1_low; // beta1 and 1 - beta1, each in two parts
  float b2, b2_low, a2;
  float least_root;             // roots and gradients from here on have a v' of 2^-100 or more
  float eps, root2;             // root2: 1 / sqrt(1 - beta2^step)
  int64_t step;
  const int64_t* step_dev;
  const float* gscale;
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

// A hash of 32 bits: two rounds of xor-shift and odd multiplication and a last shift.
// Shifts and factors are those that C. Wellons published (2018) as the least biased
// found in a search over such hashes.
__host__ __device__ __forceinline__ uint32_t mix(uint32_t h) {
  h ^= h >> 16;
  h *= 0x7FEB352Du;
  h ^= h >> 15;
  h *= 0x846CA68Bu;
  return h ^ (h >> 16);
}
constexpr uint32_t kGolden = 0x9E3779B9u;

// b^t by squaring, t >= 0.
__host__ __device__ __forceinline__ double int_pow(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : (byte == 0 ? 0x00400000u : byte << 23));
}

// Eight E4M3 codes times their block's power of two.
__device__ __forceinline__ void decode8(uint2 q, uint32_t byte, float (&x)[kPer]) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  const float s = scale_of(byte);
  const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q.x), false), b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q.x), true);
  const f2 c = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q.y), false), d = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q.y), true);
  x[0] = a[0] * s; x[1] = a[1] * s; x[2] = b[0] * s; x[3] = b[1] * s;
  x[4] = c[0] * s; x[5] = c[1] * s; x[6] = d[0] * s; x[7] = d[1] * s;
}

// The E4M3 code of y in [0, 448] with the random number (r + 1/2) / 2^16, by 64 bits.
__device__ __forceinline__ uint32_t code64(double y, uint32_t r) {
  uint32_t c;
  if (y < 0x1p-6) {
    c = static_cast<uint32_t>(y * 512.0 + (r + 0.5) * 0x1p-16);
  } else {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(y)) + (static_cast<uint64_t>(16 * r + 8) << 29);
    c = static_cast<uint32_t>(b >> 49) - (1016u << 3);
  }
  return c < 126u ? c : 126u;
}

// The codes of a lane's eight values under their block's scale, which comes out
// as its byte: the power of two that puts the block's largest value into
// (224, 448], so that it is never cut.  Scaled by a further 2^-120 a value has
// its code in the float's bits 20 to 26, subnormal codes as subnormal floats, and
// the random number is added below them; four places to the left the code stands
// in the word's last byte, m's sign bit before it.  Blocks with an infinity or a
// NaN get the byte 255, which reads as NaN.  ROOT: values above zero get a code
// above zero.
//
// Values within kNear units of fp32 of where the code or the scale changes are
// decided by exact(j), the j-th value in 64 bits: 16 in 2^20 are, and the codes
// are those of the formula, whatever the order of its operations.  The window's
// half is in the sum already, so the test is of its low bits alone.
constexpr uint32_t kNear = 8;
template <bool ROOT, class F>
__device__ __forceinline__ uint2 encode8(const float (&x)[kPer], const uint32_t (&h)[kPer], uint32_t& byte, F&& exact) {
  auto quad_max = [](uint32_t v) {
    v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true)));  // lane ^ 1
    return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true)));  // lane ^ 2
  };
  auto size = [&](int i) { return ROOT ? __float_as_uint(x[i]) : __float_as_uint(x[i]) & 0x7FFFFFFFu; };
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) top = max(top, size(i));
  top = quad_max(top);
  const bool finite = top < 0x7F800000u;
  uint32_t above = (top & 0x7FFFFFu) > 0x600000u ? 1u : 0u;  // 1.75 times a power of two
  if (finite && ((top + kNear - 0x600000u) & 0x7FFFFFu) < 2 * kNear) {
    const double edge = static_cast<double>(__uint_as_float((top & 0x7F800000u) | 0x600000u));
    above = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (size(i) + 2 * kNear > top && fabs(exact(i)) > edge) above = 1;
    above = quad_max(above);
  }
  const int e = static_cast<int>(top >> 23) - 8 + static_cast<int>(above);
  byte = finite ? (e > 0 ? e : 0) : 255;
  const float inv = __uint_as_float((254u - (finite ? byte : 0u)) << 23);
  uint32_t t[kPer], low = 0xFFFFFFFFu, least = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float y = fabsf(x[i]) * inv * 0x1p-120f;
    t[i] = __float_as_uint(y) + (ROOT ? (h[i] & 0xFFFFu) << 4 : h[i] >> 16 << 4) + (8u + kNear);
    low = min(low, t[i] & 0xFFFFFu);
    if (ROOT) least = min(least, t[i]);
  }
  if (low < 2 * kNear && finite) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if ((t[i] & 0xFFFFFu) < 2 * kNear)
        t[i] = code64(fabs(exact(i)) * static_cast<double>(inv), ROOT ? h[i] & 0xFFFFu : h[i] >> 16) << 20;
    if (ROOT) least = 0;
  }
  if (ROOT && least < 1u << 20) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) t[i] = max(t[i], x[i] > 0.f ? 1u << 20 : 0u);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    t[i] <<= 4;
    if (!ROOT) t[i] = (t[i] & 0x7FFFFFFFu) | (__float_as_uint(x[i]) & 0x80000000u);
  }
  auto last_bytes = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0C0C0703u), cd = __builtin_amdgcn_perm(d, c, 0x07030C0Cu);
    return ab | cd;
  };
  const uint2 q = make_uint2(last_bytes(t[0], t[1], t[2], t[3]), last_bytes(t[4], t[5], t[6], t[7]));
  return make_uint2(finite ? q.x : 0u, finite ? q.y : 0u);
}

__device__ __forceinline__ float decode1(const void* q, const uint8_t* scale, int64_t i) {
  return __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(q)[i], 0) * scale_of(scale[i >> 5]);
}

// Roots of eight values >= 0 by the hardware's instruction, within a unit; it
// takes subnormal values for zero, so small ones go through the library's.  (The
// reciprocal beside it is the hardware's too, within a unit: both stay below what
// rounding the weight costs.)
__device__ __forceinline__ void square_roots(const float (&v)[kPer], float (&r)[kPer]) {
  uint32_t least = 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    r[j] = __builtin_amdgcn_sqrtf(v[j]);
    least = min(least, __float_as_uint(v[j]) - 1u);  // zeros pass
  }
  if (least < 0x0D800000u) {  // 2^-100
#pragma unroll
    for (int j = 0; j < kPer; ++j) r[j] = sqrtf(v[j]);
  }
}

// The roots of 8-bit states have fp32's range, their squares have not: where v left it
// (or is zero) the root is again(j), formed in 64 bits, and zero only if that is.  True
// where a denominator root root2 + eps is not one that the hardware's reciprocal takes.
// For lanes with a root or gradient that small or large; zeros do not count as small,
// so that what has not been trained yet costs no more.  Looking for them takes 2% of a
// step (268 M bf16 values: 584 us, 572 without).
template <class F>
__device__ __forceinline__ bool wide_roots(const float (&v)[kPer], float (&r)[kPer], float root2, float eps, F&& again) {
  bool far = false;
#pragma unroll 1
  for (int j = 0; j < kPer; ++j) {  // a loop: side by side the eight would take registers and code from the whole kernel
    float vj = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) vj = i == j ? v[i] : vj;
    if (vj >= 0x1p-100f && vj < INFINITY) continue;
    const double u = again(j);
    const float x = u > 0.0 && u < 0x1p-149 ? 0x1p-149f : static_cast<float>(u), den = x * root2 + eps;
#pragma unroll
    for (int i = 0; i < kPer; ++i) r[i] = i == j ? x : r[i];
    far = far || (x > 0.f && !(den >= 0x1p-126f && den <= 0x1p126f));
  }
  return far;
}

template <class T>
__device__ __forceinline__ void load8(const T* p, int64_t i, int valid, float (&x)[kPer]) {
  if (valid == kPer) {
#pragma unroll
    for (int u = 0; u < kPer; u += Elem<T>::kVec) Elem<T>::unpack(*reinterpret_cast<const uint4*>(p + i + u), x + u);
  } else {
#pragma unroll
    for (int u = 0; u < kPer; ++u) x[u] = u < valid ? Elem<T>::load1(p, i + u) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store8(T* p, int64_t i, int valid, const float (&x)[kPer]) {
  if (valid == kPer) {
#pragma unroll
    for (int u = 0; u < kPer; u += Elem<T>::kVec) *reinterpret_cast<uint4*>(p + i + u) = Elem<T>::pack(x + u);
  } else {
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      if (u < valid) Elem<T>::store1(p, i + u, x[u]);
  }
}

// T: weights and gradients (float, or uint16_t for bf16).  States are whole
// blocks of 32: what lies behind a tensor's end in its last block is zero.
template <class T, bool EIGHT, bool MASTER>
__global__ __launch_bounds__(kThreads) void adamw_kernel(AdamArgs p) {
  const int b = blockIdx.x;
  int lo = 0, hi = p.count;  // first[lo] <= b < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.first[mid] <= b) lo = mid;
    else hi = mid;
  }
  const ListEntry& t = p.list[lo];
  const int64_t n = t.n, base = static_cast<int64_t>(b - p.first[lo]) * p.turns * kTurn;
  const int64_t step = p.step_dev ? *p.step_dev : p.step;
  const float b1 = p.b1, b1_low = p.b1_low, a1 = p.a1, a1_low = p.a1_low, b2 = p.b2, b2_low = p.b2_low, a2 = p.a2;
  float rate = t.rate, root2 = p.root2;
  if (p.step_dev) {
    rate = static_cast<float>(t.lr / (1.0 - int_pow(p.beta1, step)));
    root2 = static_cast<float>(1.0 / sqrt(1.0 - int_pow(p.beta2, step)));
  }
  const float gs = p.gscale ? *p.gscale : 1.0f;
  const uint32_t key = mix(mix(t.seed) + kGolden * static_cast<uint32_t>(step));

  for (int u = 0; u < p.turns; ++u) {
    const int64_t i = base + (u * kThreads + static_cast<int>(threadIdx.x)) * kPer;
    if (i >= ((n + 31) & ~int64_t{31})) break;
    const int valid = n - i >= kPer ? kPer : (n > i ? static_cast<int>(n - i) : 0);
    const int64_t o = t.offset + i;
    float w[kPer], g[kPer], m[kPer], v[kPer];
    if constexpr (MASTER) load8(p.master, o, kPer, w);
    else load8(static_cast<const T*>(t.w), i, valid, w);
    load8(static_cast<const T*>(t.g), i, valid, g);
    if constexpr (EIGHT) {
      decode8(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.m) + o), p.m_scale[o >> 5], m);
      decode8(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.v) + o), p.v_scale[o >> 5], v);
    } else {
      load8(static_cast<const float*>(p.m), o, kPer, m);
      load8(static_cast<const float*>(p.v), o, kPer, v);
    }
    uint32_t least = 0xFFFFFFFFu, most = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float gg = g[j] * gs;
      if constexpr (EIGHT) {
        // m's terms can cancel; their roundings (and those of the constants) are added up beside them, so that the sum
        // is within a unit of the formula's and the code that it gets can be told
        const float t = a1 * gg;
        float low = fmaf(a1, gg, -t);
        low = fmaf(a1, fmaf(g[j], gs, -gg), low);
        low = fmaf(a1_low, gg, low);
        low = fmaf(b1_low, m[j], low);
        m[j] = fmaf(b1, m[j], t) + low;
        const uint32_t size = max(__float_as_uint(v[j]), __float_as_uint(gg) & 0x7FFFFFFFu);  // of the larger of the two
        least = min(least, size - 1u);  // zeros pass
        most = max(most, size);
        v[j] *= v[j];
      } else {
        m[j] = fmaf(b1, m[j], fmaf(b1_low, fminf(fmaxf(m[j], -3.402823466e38f), 3.402823466e38f), a1 * gg));
      }
      // a beta in 32 bits is off by up to 2^-25, a large part of 1 - beta near 1 (at 0.99999 a thousandth, in the end all of
      // it): the rest of it joins what is added (of the largest finite value at most, so that an infinite state of 32 bits
      // stays one)
      v[j] = fmaf(b2, v[j], fmaf(b2_low, EIGHT ? v[j] : fminf(v[j], 3.402823466e38f), a2 * gg * gg));
    }
    float root[kPer];
    bool far = false;
    if constexpr (EIGHT) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) root[j] = __builtin_amdgcn_sqrtf(v[j]);
      if (least < __float_as_uint(p.least_root) || most > 0x5D800000u) {  // 2^60
        far = wide_roots(v, root, root2, p.eps, [&](int j) {
          const double r = decode1(p.v, p.v_scale, o + j);
          const double gg = j < valid ? static_cast<double>(Elem<T>::load1(t.g, i + j)) * gs : 0.0;
          return sqrt(p.beta2 * r * r + (1.0 - p.beta2) * gg * gg);
        });
      }
    } else {
      square_roots(v, root);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (EIGHT) v[j] = root[j];
      // the decay is part of what is subtracted: 1 - lr weight_decay in 32 bits would be a multiple of 2^-24
      w[j] -= fmaf(t.decay, w[j], rate * (m[j] * __builtin_amdgcn_rcpf(root[j] * root2 + p.eps)));
    }
    // again from what is in memory, by a division (as a case of the loop above it cost 45 us of 573)
    if (EIGHT && far) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        float x = 0.f;
        if constexpr (MASTER) x = p.master[o + j];
        else x = j < valid ? Elem<T>::load1(t.w, i + j) : 0.f;
        w[j] = x - fmaf(t.decay, x, rate * (m[j] / (root[j] * root2 + p.eps)));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // behind the tensor's end (its gradient reads as zero) states and master stay what they are made of: zero
    if (valid < kPer) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j >= valid) m[j] = v[j] = w[j] = 0.f;
    }
    store8(static_cast<T*>(t.w_out), i, valid, w);
    if constexpr (MASTER) store8(p.master_out, o, kPer, w);
    if constexpr (EIGHT) {
      uint32_t h[kPer], bm, bv;
#pragma unroll
      for (int j = 0; j < kPer; ++j) h[j] = mix((static_cast<uint32_t>(i) + j) * kGolden + key);
      // one value again in 64 bits, from what is still in memory (outputs may be in its place, stored below)
      auto grad = [&](int j) { return j < valid ? static_cast<double>(Elem<T>::load1(t.g, i + j)) * gs : 0.0; };
      const uint2 qm = encode8<false>(m, h, bm, [&](int j) {
        return p.beta1 * decode1(p.m, p.m_scale, o + j) + (1.0 - p.beta1) * grad(j);
      });
      const uint2 qv = encode8<true>(v, h, bv, [&](int j) {
        const double root = decode1(p.v, p.v_scale, o + j), gg = grad(j);
        return sqrt(p.beta2 * root * root + (1.0 - p.beta2) * gg * gg);
      });
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.m_out) + o) = qm;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.v_out) + o) = qv;
      if ((threadIdx.x & 3) == 0) {
        p.m_scale_out[o >> 5] = static_cast<uint8_t>(bm);
        p.v_scale_out[o >> 5] = static_cast<uint8_t>(bv);
      }
    } else {
      store8(static_cast<float*>(p.m_out), o, kPer, m);
      store8(static_cast<float*>(p.v_out), o, kPer, v);
    }
  }
}

// The values of 8-bit states (m, and the root of v) in bf16, which holds them exactly: four bits times a power of two.
__global__ __launch_bounds__(kThreads) void state_values_kernel(const uint8_t* __restrict__ m,
                                                                const uint8_t* __restrict__ m_scale,
                                                                const uint8_t* __restrict__ v,
                                                                const uint8_t* __restrict__ v_scale, int64_t n,
                                                                uint16_t* __restrict__ m_out,
                                                                uint16_t* __restrict__ v_out) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * kPer;
  if (i >= n) return;
  float x[kPer];
  if (blockIdx.y == 0) {
    decode8(*reinterpret_cast<const uint2*>(m + i), m_scale[i >> 5], x);
    *reinterpret_cast<uint4*>(m_out + i) = Elem<uint16_t>::pack(x);
  } else {
    decode8(*reinterpret_cast<const uint2*>(v + i), v_scale[i >> 5], x);
    *reinterpret_cast<uint4*>(v_out + i) = Elem<uint16_t>::pack(x);
  }
}

int64_t pad32(int64_t n) { return (n + 31) & ~int64_t{31}; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t count, int dtype, int bits, int64_t state_len,
                              const void* m, const void* v, const uint8_t* m_scale, const uint8_t* v_scale,
                              const float* master, double lr, double beta1, double beta2, double eps, int64_t step,
                              const int64_t* step_dev, const float* grad_scale, uint32_t seed, void* m_out, void* v_out,
                              uint8_t* m_scale_out, uint8_t* v_scale_out, float* master_out, void* stream) {
  if (count < 0 || (dtype != MOE_F32 && dtype != MOE_BF16) || (bits != 32 && bits != 8) || state_len < 0) return MOE_EINVAL;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !std::isfinite(eps) ||
      !std::isfinite(lr) || (!step_dev && step < 1))
    return MOE_EINVAL;
  if (!std::isfinite(static_cast<float>(lr))) return MOE_EINVAL;
  // what the hardware's reciprocal takes: below, a value without gradient would become 0 times infinity, far above (from
  // 2^126 on, with the root) it is zero
  if (eps > 0.0 && !(eps >= 0x1p-126 && eps <= 0x1p100)) return MOE_EINVAL;
  if (dtype == MOE_F32 && (master || master_out)) return MOE_EINVAL;
  if (!master != !master_out) return MOE_EINVAL;
  if (count == 0) return MOE_OK;
  if (!tensors || !m || !v || !m_out || !v_out) return MOE_EINVAL;
  if (bits == 8 && (!m_scale || !v_scale || !m_scale_out || !v_scale_out)) return MOE_EINVAL;
  for (const void* q : {m, v, static_cast<const void*>(m_scale), static_cast<const void*>(v_scale),
                        static_cast<const void*>(master), static_cast<const void*>(step_dev),
                        static_cast<const void*>(grad_scale), static_cast<const void*>(m_out),
                        static_cast<const void*>(v_out), static_cast<const void*>(m_scale_out),
                        static_cast<const void*>(v_scale_out), static_cast<const void*>(master_out)})
    if (!aligned16(q)) return MOE_EINVAL;
  int64_t end = 0;
  for (int32_t i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.n < 0 || t.offset < end || t.offset % 32 || t.offset > state_len ||
        t.n > ((state_len - t.offset) & ~int64_t{31}))  // a tensor takes whole blocks (no sum that could pass 64 bits)
      return MOE_EINVAL;
    if (t.n > 0 && (!t.w || !t.g || !t.w_out)) return MOE_EINVAL;
    if (!aligned16(t.w) || !aligned16(t.g) || !aligned16(t.w_out)) return MOE_EINVAL;
    if (!std::isfinite(t.weight_decay) || !std::isfinite(t.lr_scale) || !std::isfinite(static_cast<float>(lr * t.lr_scale)) ||
        !std::isfinite(static_cast<float>(lr * t.lr_scale * t.weight_decay)))
      return MOE_EINVAL;
    if (t.n > (kMaxUnits - 1) * 4 * kTurn) return MOE_EUNSUPPORTED;
    end = t.offset + pad32(t.n);
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  AdamArgs a;
  a.m = m; a.v = v; a.m_scale = m_scale; a.v_scale = v_scale; a.master = master;
  a.m_out = m_out; a.v_out = v_out; a.m_scale_out = m_scale_out; a.v_scale_out = v_scale_out; a.master_out = master_out;
  a.beta1 = beta1; a.beta2 = beta2; a.eps = static_cast<float>(eps);
  a.b1 = static_cast<float>(beta1); a.b1_low = static_cast<float>(beta1 - a.b1);
  a.a1 = static_cast<float>(1.0 - beta1); a.a1_low = static_cast<float>(1.0 - beta1 - a.a1);
  a.b2 = static_cast<float>(beta2); a.b2_low = static_cast<float>(beta2 - a.b2); a.a2 = static_cast<float>(1.0 - beta2);
  a.least_root = 0x1p-50f / std::sqrt(a.b2 > 0.f && a.b2 < a.a2 ? a.b2 : a.a2);
  const double c1 = step_dev ? 1.0 : 1.0 - int_pow(beta1, step);
  a.root2 = step_dev ? 1.0f : static_cast<float>(1.0 / std::sqrt(1.0 - int_pow(beta2, step)));
  // one turn a unit until four would still leave eight workgroups to a compute unit
  int64_t all = 0;
  for (int32_t i = 0; i < count; ++i) all += cdiv(tensors[i].n, 4 * kTurn);
  a.turns = all >= 8 * 256 ? 4 : 1;
  const int64_t unit = a.turns * kTurn;
  a.step = step; a.step_dev = step_dev; a.gscale = grad_scale;
  for (int32_t i = 0; i < count;) {
    a.count = 0;
    int64_t units = 0;
    for (; i < count && a.count < kMaxList; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      const int64_t more = cdiv(t.n, unit);
      if (more == 0) continue;
      if (units + more >= kMaxUnits) break;
      const double rate = lr * t.lr_scale;
      a.list[a.count] = ListEntry{t.w, t.g, t.w_out, t.n, t.offset, rate, static_cast<float>(rate / c1),
                                  static_cast<float>(rate * t.weight_decay), seed + kGolden * static_cast<uint32_t>(i)};
      a.first[a.count++] = static_cast<int32_t>(units);
      units += more;
    }
    if (a.count == 0) break;
    a.first[a.count] = static_cast<int32_t>(units);
    const dim3 grid(static_cast<unsigned>(units)), block(kThreads);
    if (dtype == MOE_F32) {
      if (bits == 8) MOE_LAUNCH("adamw", (adamw_kernel<float, true, false>), grid, block, 0, s, a);
      else MOE_LAUNCH("adamw", (adamw_kernel<float, false, false>), grid, block, 0, s, a);
    } else if (master) {
      if (bits == 8) MOE_LAUNCH("adamw", (adamw_kernel<uint16_t, true, true>), grid, block, 0, s, a);
      else MOE_LAUNCH("adamw", (adamw_kernel<uint16_t, false, true>), grid, block, 0, s, a);
    } else {
      if (bits == 8) MOE_LAUNCH("adamw", (adamw_kernel<uint16_t, true, false>), grid, block, 0, s, a);
      else MOE_LAUNCH("adamw", (adamw_kernel<uint16_t, false, false>), grid, block, 0, s, a);
    }
    const int st = launch_status();
    if (st != MOE_OK) return st;
  }
  return MOE_OK;
}

extern "C" int moe_adamw_state_values(const uint8_t* m, const uint8_t* m_scale, const uint8_t* v, const uint8_t* v_scale,
                                      int64_t state_len, void* m_values, void* root_values, void* stream) {
  if (state_len < 0 || state_len % 32) return MOE_EINVAL;
  if (state_len == 0) return MOE_OK;
  if (!m || !m_scale || !v || !v_scale || !m_values || !root_values) return MOE_EINVAL;
  for (const void* q : {static_cast<const void*>(m), static_cast<const void*>(m_scale), static_cast<const void*>(v),
                        static_cast<const void*>(v_scale), static_cast<const void*>(m_values),
                        static_cast<const void*>(root_values)})
    if (!aligned16(q)) return MOE_EINVAL;
  if (state_len > (kMaxUnits / 2 - 1) * kTurn) return MOE_EUNSUPPORTED;
  MOE_LAUNCH("adamw_state_values", state_values_kernel, dim3(static_cast<unsigned>(cdiv(state_len, kTurn)), 2), dim3(kThreads),
             0, static_cast<hipStream_t>(stream), m, m_scale, v, v_scale, state_len, static_cast<uint16_t*>(m_values),
             static_cast<uint16_t*>(root_values));
  return launch_status();
}
