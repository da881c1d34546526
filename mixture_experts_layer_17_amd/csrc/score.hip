// Routing by scores, its backward, and the update of the balancing bias.
//
// A token's scores are s = softmax(l) over all experts or s = sigmoid(l); it
// chooses by c = s + b (b: a bias per expert that only moves the choice).  With
// groups, the groups whose best one or two choices sum highest stay in; then
// the k best c inside them are taken and their s, renormalised or not, times a
// factor, are the gates.
//
// Which expert is chosen must not hang on rounding, so the order is that of c in
// 64 bits: near ties in 32 bits are common (16384 tokens of 256 experts have some
// ten pairs within 2^-24 of each other at the border of the choice).
//
// Sixteen lanes take a token (one DPP row: its maxima and sums are rotations
// inside the row), four tokens a wave, 64 tokens a workgroup, so that a 64-bit
// mask per expert in LDS gives each chosen slot its rank among the workgroup's
// tokens.  The counts go out as [expert][workgroup]; one wave per expert turns
// its row into exclusive sums, and the workgroups of the last launch make the
// experts' offsets from the totals themselves.  No step runs on one workgroup.
#include <cmath>
#include <type_traits>

#include "common.hpp"

namespace moe {
namespace {

constexpr int kRow = 16;          // lanes per token
constexpr int kTok = 64;          // tokens per workgroup (bits of a mask)
constexpr int kSelThreads = kRow * kTok;

// ---------------------------------------------------------------------------
// Reductions over the 16 lanes of a DPP row (every lane must be active): the
// rotations by 8, 4, 2 and 1 leave the result in all lanes.
// ---------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ uint32_t ror(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x120 | N, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ float ror(float v) {
  return __uint_as_float(ror<N>(__float_as_uint(v)));
}
template <int N>
__device__ __forceinline__ uint64_t ror(uint64_t v) {
  return static_cast<uint64_t>(ror<N>(static_cast<uint32_t>(v >> 32))) << 32 | ror<N>(static_cast<uint32_t>(v));
}
template <int N>
__device__ __forceinline__ double ror(double v) {
  return __longlong_as_double(static_cast<long long>(ror<N>(static_cast<uint64_t>(__double_as_longlong(v)))));
}
template <class T, class F>
__device__ __forceinline__ T row_reduce(T v, F f) {
  v = f(v, ror<8>(v));
  v = f(v, ror<4>(v));
  v = f(v, ror<2>(v));
  return f(v, ror<1>(v));
}
template <class T>
__device__ __forceinline__ T row_max(T v) {
  return row_reduce(v, [](T a, T b) { return a > b ? a : b; });
}
__device__ __forceinline__ float row_fmax(float v) {
  return row_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  return row_reduce(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}
template <class T>
__device__ __forceinline__ T row_sum(T v) {
  return row_reduce(v, [](T a, T b) { return a + b; });
}

// Choices as whole numbers of the same order: 0 is out of the race, 1 a NaN (it
// ranks below every number), and -0 is +0.
__device__ __forceinline__ uint64_t order_key(double c) {
  if (c != c) return 1;
  const int64_t b = __double_as_longlong(c + 0.0);
  return static_cast<uint64_t>(b) ^ (static_cast<uint64_t>(b >> 63) | 0x8000000000000000ull);
}

// The score of logit x under a row maximum m before it is divided by the sum: a
// row of -inf has none, and a NaN spoils its row.
__device__ __forceinline__ double softmax_part(float x, float m) {
  if (m == -INFINITY) return x == x ? 0.0 : NAN;
  return exp(static_cast<double>(x) - static_cast<double>(m));
}
__device__ __forceinline__ float softmax_part32(float x, float m) {
  if (m == -INFINITY) return x == x ? 0.f : NAN;
  return expf(x - m);
}

// LDS written by some lanes of a wave and read by others of the same wave.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct ScoreArgs {
  const float* logits;
  const float* bias;  // may be null
  int64_t T;
  int E, k, sigmoid, groups, top_groups, group_best, renorm;
  float scale;
  int32_t* topk_idx;
  float* gates;
  int32_t* rank;        // [T, k] rank of the slot among its workgroup's tokens
  int32_t* blk_counts;  // [E, workgroups]
  int64_t nblk;
  // for a single workgroup, which writes them itself
  int32_t *counts, *offsets, *perm_src, *perm_dst, *mx_blk_offsets;
};

// The expert of a lane's c-th value: runs of four where rows are 16-byte aligned
// and whole (VEC), else single ones.
template <bool VEC>
__device__ __forceinline__ int expert_of(int c, int lane) {
  return VEC ? ((c >> 2) * kRow + lane) * 4 + (c & 3) : c * kRow + lane;
}

// e / size for e below 256 without a division: (e + 1/2) / size is at least 1/512 away from a whole number.
__device__ __forceinline__ int group_of(int e, float per) { return static_cast<int>((static_cast<float>(e) + 0.5f) * per); }

// A lane's values of a row; `none` past its end.
template <int C, bool VEC>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float none, float (&x)[C]) {
  if constexpr (VEC) {
#pragma unroll
    for (int c = 0; c < C; c += 4) {
      const int e = expert_of<VEC>(c, lane);
      const float4 v = e < E ? *reinterpret_cast<const float4*>(row + e) : make_float4(none, none, none, none);
      x[c] = v.x; x[c + 1] = v.y; x[c + 2] = v.z; x[c + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = expert_of<VEC>(c, lane);
      x[c] = e < E ? row[e] : none;
    }
  }
}

// Offsets of the experts, for thread tid = expert with its count: exclusive sums
// in `first` (LDS, every thread past the call's barrier may read it); where the
// pointers are given, counts, offsets and 32-row block offsets go out too.  By
// the first 256 threads of a workgroup, all of whose threads call it.
__device__ __forceinline__ void offsets_of(int own, int E, int32_t* first, int32_t* counts, int32_t* offsets,
                                           int32_t* mx_blk_offsets) {
  __shared__ int32_t part[2][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int ownb = (own + 31) / 32;
  int incl = own, inclb = ownb;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o, 64), upb = __shfl_up(inclb, o, 64);
    if (lane >= o) {
      incl += up;
      inclb += upb;
    }
  }
  if (wave < 4 && lane == 63) {
    part[0][wave] = incl;
    part[1][wave] = inclb;
  }
  __syncthreads();
  if (tid < kMaxE) {
    for (int w = 0; w < wave; ++w) {
      incl += part[0][w];
      inclb += part[1][w];
    }
    first[tid] = incl - own;
    if (offsets && tid < E) {
      if (tid == 0) offsets[0] = 0;
      offsets[tid + 1] = incl;
      if (mx_blk_offsets) {
        if (tid == 0) mx_blk_offsets[0] = 0;
        mx_blk_offsets[tid + 1] = inclb;
      }
      if (counts) counts[tid] = own;
    }
  }
  __syncthreads();
}

// Leaves in `on` (one bit per c) the values whose group stays.  `key` is the
// token's row in LDS, the bits of its choices; their place then takes the groups'.
template <int C, bool VEC>
__device__ __forceinline__ void keep_groups(const ScoreArgs& p, uint64_t* key, int lane, int tok, uint32_t& on) {
  const int size = p.E / p.groups;
  // lanes 0, 1, .. take groups: the sums of their best, kept in registers until every lane has read the row
  double sum[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int g = u * kRow + lane;
    double b0 = -INFINITY, b1 = -INFINITY;
    bool nan = false;
    if (g < p.groups) {
      int i = (g + tok) % size;  // lanes start apart, else they would meet on one LDS bank
      for (int n = 0; n < size; ++n) {
        const double v = __longlong_as_double(static_cast<long long>(key[g * size + i]));
        if (++i == size) i = 0;
        nan |= v != v;
        b1 = v > b0 ? b0 : (v > b1 ? v : b1);
        b0 = v > b0 ? v : b0;
      }
    }
    sum[u] = nan ? NAN : (p.group_best == 1 ? b0 : b0 + b1);
  }
  wave_sync();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u * kRow + lane < p.groups) key[u * kRow + lane] = order_key(sum[u]);
  wave_sync();
  // a group stays when fewer than top_groups come before it
  uint32_t stay = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int g = u * kRow + lane;
    if (g < p.groups) {
      const uint64_t mine = key[g];
      int before = 0;
      for (int h = 0; h < p.groups; ++h) before += key[h] > mine || (key[h] == mine && h < g);
      stay |= static_cast<uint32_t>(before < p.top_groups) << u;
    }
  }
  wave_sync();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u * kRow + lane < p.groups) key[u * kRow + lane] = (stay >> u) & 1;
  wave_sync();
  const float per = 1.0f / static_cast<float>(size);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = expert_of<VEC>(c, lane);
    if (e < p.E && !key[group_of(e, per)]) on &= ~(1u << c);
  }
}

// The choice of a token by 64 bits: lane j gets its j-th expert.
template <int C, bool VEC>
__device__ __forceinline__ int choose_exact(const ScoreArgs& p, const float (&l)[C], float m, uint32_t on, uint64_t* mine,
                                            int lane, int tok) {
  double s[C];
  if (p.sigmoid) {
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = 1.0 / (1.0 + exp(-static_cast<double>(l[c])));
  } else {
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s[c] = (on >> c) & 1 ? softmax_part(l[c], m) : 0.0;
      sum += s[c];
    }
    sum = row_sum(sum);
    const double inv = sum == 0.0 ? 0.0 : 1.0 / sum;
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] *= inv;
  }
  if (p.bias) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if ((on >> c) & 1) s[c] += static_cast<double>(p.bias[expert_of<VEC>(c, lane)]);
  }
  if (p.groups > 1) {
    wave_sync();
#pragma unroll
    for (int c = 0; c < C; ++c)
      if ((on >> c) & 1) mine[expert_of<VEC>(c, lane)] = static_cast<uint64_t>(__double_as_longlong(s[c]));
    wave_sync();
    keep_groups<C, VEC>(p, mine, lane, tok, on);
  }
  uint64_t key[C];
#pragma unroll
  for (int c = 0; c < C; ++c) key[c] = (on >> c) & 1 ? order_key(s[c]) : 0;
  int my_e = 0;
  for (int j = 0; j < p.k; ++j) {
    uint64_t best = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) best = key[c] > best ? key[c] : best;
    best = row_max(best);
    uint32_t e_best = 0xFFFFFFFFu;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t e = expert_of<VEC>(c, lane);
      if (key[c] == best && e < e_best) e_best = e;
    }
    e_best = row_min(e_best);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (static_cast<uint32_t>(expert_of<VEC>(c, lane)) == e_best) key[c] = 0;
    if (lane == j) my_e = static_cast<int>(e_best);
  }
  return my_e;
}

// ---------------------------------------------------------------------------
// The choice in 32 bits, which finds the candidates, and that of 64 among them.
// A value may be off by tol + rel |c|, so where two that follow each other are
// nearer than both may be off, the candidates (with those that may come before the
// k-th) are ordered by their choices in 64 bits, one a lane.  A lane's values carry
// their place c in the key's last four bits, so that a maximum brings it along,
// which cuts the value by up to 2^-19 of itself.  Where that does not tell (NaN,
// infinities, more than 16 candidates, groups too near at their border) the wave
// chooses by choose_exact.  16384 x 256 sigmoid scores, bias, 8 groups: 17 us
// without a near pair, 23 like this, 28 with choose_exact for every wave that has one (some
// wave of every compute unit's 16 does, and the others wait for it), 34 all in
// 64 bits, one after the other.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t order_key32(float c) {
  const uint32_t b = __float_as_uint(c);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value32(uint32_t k) {
  k &= ~15u;
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// keep_groups in 32 bits; false where two groups at the border are within `edge`.
template <int C, bool VEC>
__device__ __forceinline__ bool keep_groups32(const ScoreArgs& p, float* val, float edge, int lane, int tok,
                                              uint32_t& on) {
  const int size = p.E / p.groups;
  float sum[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int g = u * kRow + lane;
    float b0 = -INFINITY, b1 = -INFINITY;
    if (g < p.groups) {
      auto take = [&](float v) {
        b1 = fmaxf(b1, fminf(b0, v));
        b0 = fmaxf(b0, v);
      };
      if (VEC && size % 4 == 0) {
        const float4* q = reinterpret_cast<const float4*>(val + g * size);
        int i = (g + tok) % (size / 4);  // lanes start apart, else they would meet on one LDS bank
        for (int n = 0; n < size / 4; ++n) {
          const float4 v = q[i];
          if (++i == size / 4) i = 0;
          take(v.x); take(v.y); take(v.z); take(v.w);
        }
      } else {
        int i = (g + tok) % size;
        for (int n = 0; n < size; ++n) {
          take(val[g * size + i]);
          if (++i == size) i = 0;
        }
      }
    }
    sum[u] = p.group_best == 1 ? b0 : b0 + b1;
  }
  wave_sync();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u * kRow + lane < p.groups) val[u * kRow + lane] = sum[u];
  wave_sync();
  uint32_t stay = 0;
  bool sure = true;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u * kRow + lane < p.groups) {
      int over = 0, near = 0;  // groups that come first for sure, and that may
      for (int h = 0; h < p.groups; ++h) {
        over += val[h] > sum[u] + edge;
        near += val[h] >= sum[u] - edge;
      }
      stay |= static_cast<uint32_t>(over < p.top_groups) << u;
      sure = sure && (over >= p.top_groups || near <= p.top_groups);  // near counts the group itself
    }
  }
  wave_sync();
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u * kRow + lane < p.groups) val[u * kRow + lane] = (stay >> u) & 1 ? 1.f : 0.f;
  wave_sync();
  const float per = 1.0f / static_cast<float>(size);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = expert_of<VEC>(c, lane);
    if (e < p.E && val[group_of(e, per)] == 0.f) on &= ~(1u << c);
  }
  return sure;
}

// The candidates of a row's lanes (experts, -1: none) in the order of their choices in 64 bits, as choose_exact forms
// them: each lane counts those before its own.
template <int C, bool VEC>
__device__ __forceinline__ int by_choice(const ScoreArgs& p, const float (&l)[C], float m, uint32_t on, int e, int lane,
                                         const float* logits) {
  double c = 0.0;
  if (p.sigmoid) {
    if (e >= 0) c = 1.0 / (1.0 + exp(-static_cast<double>(logits[e])));
  } else {
    double inv = 1.0;
    if (p.bias) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < C; ++i) sum += (on >> i) & 1 ? softmax_part(l[i], m) : 0.0;
      sum = row_sum(sum);
      inv = sum == 0.0 ? 0.0 : 1.0 / sum;
    }
    if (e >= 0) c = softmax_part(logits[e], m) * inv;
  }
  if (p.bias && e >= 0) c += static_cast<double>(p.bias[e]);
  const uint64_t key = e >= 0 ? order_key(c) : 0;
  const uint32_t at = e >= 0 ? static_cast<uint32_t>(e) : 0x10000u + lane;
  int before = 0;
  auto count = [&](uint64_t k, uint32_t a) { before += k > key || (k == key && a < at); };
  count(ror<1>(key), ror<1>(at)); count(ror<2>(key), ror<2>(at)); count(ror<3>(key), ror<3>(at));
  count(ror<4>(key), ror<4>(at)); count(ror<5>(key), ror<5>(at)); count(ror<6>(key), ror<6>(at));
  count(ror<7>(key), ror<7>(at)); count(ror<8>(key), ror<8>(at)); count(ror<9>(key), ror<9>(at));
  count(ror<10>(key), ror<10>(at)); count(ror<11>(key), ror<11>(at)); count(ror<12>(key), ror<12>(at));
  count(ror<13>(key), ror<13>(at)); count(ror<14>(key), ror<14>(at)); count(ror<15>(key), ror<15>(at));
  return __builtin_amdgcn_ds_permute((((threadIdx.x & 63) & ~(kRow - 1)) + before) * 4, e);
}

// False where the 32 bits do not tell (all lanes of the wave agree).
template <int C, bool VEC>
__device__ __forceinline__ bool choose_fast(const ScoreArgs& p, const float (&l)[C], const float (&s)[C], float m, float most,
                                            uint32_t on, float* mine, int lane, int tok, const float* logits, int& my_e) {
  const uint32_t on_all = on;
  float c[C], check = 0.f;
#pragma unroll
  for (int i = 0; i < C; ++i) c[i] = s[i];
  if (p.bias) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < C; i += 4) {
        const int e = expert_of<VEC>(i, lane);
        const float4 b = e < p.E ? *reinterpret_cast<const float4*>(p.bias + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        c[i] += b.x; c[i + 1] += b.y; c[i + 2] += b.z; c[i + 3] += b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int e = expert_of<VEC>(i, lane);
        c[i] += e < p.E ? p.bias[e] : 0.f;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) check = fmaf(c[i], 0.f, check);
  bool sure = check == 0.f;  // a NaN or an infinity makes it NaN
  // a choice is off by tol + rel |c| at most.  Without a bias it is off relative to itself: by 2^-24 of the exponent
  // (up to 44: smaller ones are below tol), a few units, and the key's 2^-19
  const float tol = p.bias ? (p.sigmoid ? 0x1p-22f : 0x1p-19f * most) : 0x1p-62f * most;
  const float rel = p.bias ? 0x1p-18f : 0x1p-17f;
  if (p.groups > 1) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < C; i += 4)
        if ((on >> i) & 1)
          *reinterpret_cast<float4*>(mine + expert_of<VEC>(i, lane)) = make_float4(c[i], c[i + 1], c[i + 2], c[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if ((on >> i) & 1) mine[expert_of<VEC>(i, lane)] = c[i];
    }
    wave_sync();
    float mag = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) mag = (on >> i) & 1 ? fmaxf(mag, fabsf(c[i])) : mag;
    // two sums of two choices each, not cut yet, whose terms may cancel: each term by its score and half a unit, each
    // sum by a unit of at most twice the largest
    const float edge = 4.0f * tol + (p.bias ? 0x1p-21f : 0x1p-16f) * row_fmax(mag);
    sure = keep_groups32<C, VEC>(p, mine, edge, lane, tok, on) && sure;
  }
  uint32_t key[C];
#pragma unroll
  for (int i = 0; i < C; ++i) key[i] = (on >> i) & 1 ? (order_key32(c[i]) & ~15u) | i : 0u;
  // lane j takes the j-th candidate: k of them, and those that 64 bits may put before the k-th
  const int row = (threadIdx.x & 63) / kRow;
  float last = 0.f, kth = 0.f;
  bool more = true, near = false;
  int e_mine = -1;
  for (int j = 0; __any(more); ++j) {
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < C; ++i) own = max(own, key[i]);
    const uint32_t best = row_max(own);
    const uint32_t owners = static_cast<uint32_t>(__ballot(own == best) >> (row * kRow)) & 0xFFFFu;
    const float v = key_value32(best);
    const bool apart = best == 0 || last - v > 2.0f * (tol + rel * fabsf(last));
    more = more && (j < p.k || !(best == 0 || kth - v > 2.0f * (tol + rel * fabsf(kth))));
    sure = sure && !(more && j == kRow);  // too many of them
    more = more && j < kRow;
    near = near || (more && j > 0 && !apart);
    last = v;
    if (j == p.k - 1) kth = v;
    const int i = best & 15, ln = __ffs(owners) - 1;
    const int e = VEC ? ((i >> 2) * kRow + ln) * 4 + (i & 3) : i * kRow + ln;
    if (more && lane == j) e_mine = e;
    if (lane == ln) {
#pragma unroll
      for (int q = 0; q < C; ++q) key[q] = key[q] == best ? 0u : key[q];
    }
  }
  if (!__all(sure)) return false;
  if (__any(near)) e_mine = by_choice<C, VEC>(p, l, m, on_all, e_mine, lane, logits);
  my_e = e_mine < 0 ? 0 : e_mine;
  return true;
}

template <int C, bool VEC>
__global__ __launch_bounds__(kSelThreads) void score_select_kernel(ScoreArgs p) {
  extern __shared__ __align__(16) unsigned char smem[];
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(smem);                // [E]
  // with groups, the choices of the tokens: [kTok][E] of 8 bytes (of which the first way uses 4)
  const int E = p.E;
  uint64_t* rows = reinterpret_cast<uint64_t*>(smem + ((E * 8 + 15) & ~15));
  const int tid = threadIdx.x, lane = tid & (kRow - 1), tok = tid / kRow;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTok + tok;
  const bool live = t < p.T;
  const float* row = p.logits + (live ? t : p.T - 1) * E;  // lanes without a token follow the last one

  float l[C];
  load_row<C, VEC>(row, E, lane, 0.f, l);
  for (int e = tid; e < E; e += kSelThreads) mask[e] = 0ull;
  uint32_t on = 0;
#pragma unroll
  for (int c = 0; c < C; ++c) on |= static_cast<uint32_t>(expert_of<VEC>(c, lane) < E) << c;

  // scores in 32 bits; softmax's maximum serves the gates too
  float s[C], m = 0.f, sum = 1.f, inv = 1.f;
  if (p.sigmoid) {
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] = sigmoid_f(l[c]);
  } else {
    m = -INFINITY;
#pragma unroll
    for (int c = 0; c < C; ++c) m = (on >> c) & 1 ? fmaxf(m, l[c]) : m;
    m = row_fmax(m);
    sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s[c] = (on >> c) & 1 ? (m == -INFINITY ? softmax_part32(l[c], m) : __expf(l[c] - m)) : 0.f;
      sum += s[c];
    }
    sum = row_sum(sum);
    inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
    for (int c = 0; c < C; ++c) s[c] *= inv;
  }
  uint64_t* mine = rows + static_cast<size_t>(tok) * E;
  int my_e = 0;
  if (!choose_fast<C, VEC>(p, l, s, m, inv, on, reinterpret_cast<float*>(mine), lane, tok, row, my_e))
    my_e = choose_exact<C, VEC>(p, l, m, on, mine, lane, tok);

  // the gate of lane j's expert, in 64 bits; where the scores are gates as they are, so is softmax's sum (a sum of 32 bits
  // would put several roundings into a gate)
  double total = 0.0;
  if (!p.sigmoid && !p.renorm) {
#pragma unroll
    for (int c = 0; c < C; ++c) total += (on >> c) & 1 ? softmax_part(l[c], m) : 0.0;
    total = row_sum(total);
  }
  const float lj = lane < p.k ? row[my_e] : -INFINITY;
  const float mj = p.renorm ? row_fmax(lj) : m;
  double gate = 0.0;
  if (lane < p.k) {
    if (p.sigmoid) gate = 1.0 / (1.0 + exp(-static_cast<double>(lj)));
    else if (!p.renorm) gate = total == 0.0 ? 0.0 : softmax_part(lj, m) / total;
    else gate = sum != sum ? NAN : softmax_part(lj, mj);  // from the chosen logits alone: the sum divides out
  }
  if (p.renorm) {
    const double tot = row_sum(gate);
    gate = tot == 0.0 ? 0.0 : gate / tot;
  }
  const bool chosen = live && lane < p.k;
  __syncthreads();
  if (chosen) {
    p.topk_idx[t * p.k + lane] = my_e;
    p.gates[t * p.k + lane] = static_cast<float>(gate * static_cast<double>(p.scale));
    atomicOr(&mask[my_e], 1ull << tok);
  }
  __syncthreads();
  const int below = chosen ? __popcll(mask[my_e] & ((1ull << tok) - 1ull)) : 0;
  if (p.nblk > 1) {
    if (chosen) p.rank[t * p.k + lane] = below;
    for (int e = tid; e < E; e += kSelThreads) p.blk_counts[e * p.nblk + blockIdx.x] = __popcll(mask[e]);
    return;
  }
  // a single workgroup: the metadata at once
  __shared__ int32_t first[kMaxE];
  offsets_of(tid < E ? __popcll(mask[tid]) : 0, E, first, p.counts, p.offsets, p.mx_blk_offsets);
  if (chosen) {
    const int at = first[my_e] + below;
    p.perm_dst[t * p.k + lane] = at;
    p.perm_src[at] = static_cast<int32_t>(t * p.k + lane);
  }
}

// One wave per expert: its counts over the workgroups become exclusive sums in
// place, their total its count.
__global__ __launch_bounds__(64) void score_scan_kernel(int32_t* __restrict__ blk, int64_t nblk,
                                                        int32_t* __restrict__ counts) {
  const int e = blockIdx.x, lane = threadIdx.x;
  int32_t* row = blk + static_cast<int64_t>(e) * nblk;
  int base = 0;
  for (int64_t b0 = 0; b0 < nblk; b0 += 64) {
    const int64_t b = b0 + lane;
    const int own = b < nblk ? row[b] : 0;
    int incl = own;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    if (b < nblk) row[b] = base + incl - own;
    base += __shfl(incl, 63, 64);
  }
  if (lane == 0) counts[e] = base;
}

// Scan and scatter at once, for few counts: a workgroup takes the 64 tokens of its routing block and sums the counts of
// all blocks for itself, those before its own apart.
__global__ __launch_bounds__(256) void score_place_kernel(const int32_t* __restrict__ topk_idx,
                                                          const int32_t* __restrict__ rank,
                                                          const int32_t* __restrict__ blk, int64_t nblk, int64_t R, int k,
                                                          int E, int32_t* __restrict__ counts,
                                                          int32_t* __restrict__ offsets,
                                                          int32_t* __restrict__ mx_blk_offsets,
                                                          int32_t* __restrict__ perm_src, int32_t* __restrict__ perm_dst) {
  __shared__ int32_t first[kMaxE];
  const int tid = threadIdx.x, mine = blockIdx.x;
  int own = 0, before = 0;
  if (tid < E) {
    const int32_t* row = blk + tid * nblk;
#pragma unroll 8
    for (int b = 0; b < nblk; ++b) {
      const int c = row[b];
      own += c;
      before += b < mine ? c : 0;
    }
  }
  offsets_of(own, E, first, mine == 0 ? counts : nullptr, mine == 0 ? offsets : nullptr, mx_blk_offsets);
  first[tid] += before;  // its own entry, which the others read after the barrier
  __syncthreads();
  const int64_t i0 = static_cast<int64_t>(mine) * kTok * k;
  for (int u = tid; u < kTok * k && i0 + u < R; u += 256) {
    const int64_t i = i0 + u;
    const int row = first[topk_idx[i]] + rank[i];
    perm_dst[i] = row;
    perm_src[row] = static_cast<int32_t>(i);
  }
}

// Every workgroup makes the experts' offsets (exclusive sums of the counts) for
// itself; the first one writes them out.
__global__ __launch_bounds__(256) void score_scatter_kernel(const int32_t* __restrict__ topk_idx,
                                                            const int32_t* __restrict__ rank,
                                                            const int32_t* __restrict__ blk_base, int64_t nblk,
                                                            int64_t R, int k, int E,
                                                            const int32_t* __restrict__ counts,
                                                            int32_t* __restrict__ offsets,
                                                            int32_t* __restrict__ mx_blk_offsets,
                                                            int32_t* __restrict__ perm_src,
                                                            int32_t* __restrict__ perm_dst) {
  __shared__ int32_t first[kMaxE];
  const int tid = threadIdx.x;
  const bool out = blockIdx.x == 0;
  offsets_of(tid < E ? counts[tid] : 0, E, first, nullptr, out ? offsets : nullptr, mx_blk_offsets);
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + tid;
  if (i >= R) return;
  const int64_t b = i / (k * kTok);
  const int e = topk_idx[i];
  const int row = first[e] + blk_base[e * nblk + b] + rank[i];
  perm_dst[i] = row;
  perm_src[row] = static_cast<int32_t>(i);
}

// ---------------------------------------------------------------------------
// Backward.  With a = scale, S the sum of the chosen scores:
//   renormalised    ds_j = (a dg_j - sum_i a dg_i s_i / S) / S
//   not             ds_j = a dg_j
//   sigmoid         dl_j = ds_j s_j (1 - s_j), zero elsewhere
//   softmax         dl_e = s_e (ds_e - sum_j ds_j s_j), where the sum is zero
//                   for renormalised gates: then dl is zero elsewhere too, and
//                   s / S is the softmax over the chosen logits alone
// Softmax without renormalising needs whole rows; with it they are read all the
// same: a NaN or +inf in them, also of an expert not chosen, makes the gates NaN,
// and the gradient must not hide that.  Sixteen lanes take a token, lane j its
// slot j, the row in registers; what the slots add meets it in LDS.  16384 x 128
// without renormalising: 6.5 us, 2.6 TB/s of rows read and written: too short for
// the rate of a large copy.
// ---------------------------------------------------------------------------
struct ScoreBwdArgs {
  const float* logits;
  const int32_t* topk_idx;
  const float* dgates;
  int64_t T;
  int E, k, sigmoid, renorm, accumulate;
  float scale;
  float* dlogits;
};

template <int C, bool VEC>
__global__ __launch_bounds__(256) void score_bwd_kernel(ScoreBwdArgs p) {
  extern __shared__ __align__(16) float brow[];
  const int tid = threadIdx.x, lane = tid & (kRow - 1), tok = tid / kRow;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / kRow) + tok;
  const bool live = t < p.T;
  const int64_t tt = live ? t : p.T - 1;
  const int E = p.E;
  const float* row = p.logits + tt * E;
  float* add = brow + tok * E;  // what the slots add to their experts' gradients
  const int e = lane < p.k ? p.topk_idx[tt * p.k + lane] : -1;
  const bool slot = static_cast<unsigned>(e) < static_cast<unsigned>(E);  // e addresses the row: a slot outside it counts as absent
  const float dg = slot ? p.scale * p.dgates[tt * p.k + lane] : 0.f;
  const float l = slot ? row[e] : -INFINITY;
  const bool full = !p.sigmoid && !p.renorm;

  float x[C], m = -INFINITY, inv = 0.f, whole = 1.f;
  if (full) {
    load_row<C, VEC>(row, E, lane, -INFINITY, x);
#pragma unroll
    for (int c = 0; c < C; ++c) m = fmaxf(m, x[c]);
    m = row_fmax(m);
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x[c] = expert_of<VEC>(c, lane) < E ? softmax_part32(x[c], m) : 0.f;
      sum += x[c];
    }
    sum = row_sum(sum);
    inv = sum == 0.f ? 0.f : 1.0f / sum;
  } else if (!p.sigmoid) {
    m = row_fmax(l);
    load_row<C, VEC>(row, E, lane, -INFINITY, x);
    float bad = 0.f;  // a NaN or +inf anywhere leaves the row without scores: `whole` becomes NaN
#pragma unroll
    for (int c = 0; c < C; ++c) bad = x[c] < INFINITY ? bad : NAN;
    whole = 1.f + row_sum(bad);
  }
  // the slot's score (of all experts, or of the chosen ones alone) and gradient, in 64 bits: a lane has one
  double s = 0.0, ds = dg * whole;
  if (slot) s = p.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l))) : softmax_part(l, m) * (full ? inv : 1.0);
  if (p.renorm) {
    const double tot = row_sum(s), w = tot == 0.0 ? 0.0 : 1.0 / tot;
    ds = (ds - row_sum(ds * s) * w) * w;
  }
  const double dl = p.sigmoid ? ds * s / (1.0 + exp(static_cast<double>(l))) : s * ds;
  const float inner = full ? static_cast<float>(row_sum(dl)) : 0.f;

#pragma unroll
  for (int c = 0; c < C; ++c)
    if (expert_of<VEC>(c, lane) < E) add[expert_of<VEC>(c, lane)] = 0.f;
  wave_sync();
  if (slot) add[e] = static_cast<float>(dl);
  wave_sync();
  if (!live) return;
  float* dst = p.dlogits + t * E;
#pragma unroll
  for (int c = 0; c < C; c += VEC ? 4 : 1) {
    const int at = expert_of<VEC>(c, lane);
    if (at >= E) continue;
    if constexpr (VEC) {
      float4 v = *reinterpret_cast<const float4*>(add + at);
      if (full) {
        v.x -= x[c] * inv * inner; v.y -= x[c + 1] * inv * inner; v.z -= x[c + 2] * inv * inner; v.w -= x[c + 3] * inv * inner;
      }
      if (p.accumulate) {
        const float4 a = *reinterpret_cast<const float4*>(dst + at);
        v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
      }
      *reinterpret_cast<float4*>(dst + at) = v;
    } else {
      float v = add[at];
      if (full) v -= x[c] * inv * inner;
      dst[at] = p.accumulate ? dst[at] + v : v;
    }
  }
}

// bias_out[e] = bias[e] + rate sign(sum of the counts - E counts[e]): up for an
// expert below the mean load, down for one above.  Whole numbers of 64 bits, so
// the sign is exact.
__global__ __launch_bounds__(1024) void bias_update_kernel(const int32_t* __restrict__ counts, int64_t S, int E, float rate,
                                                           const float* __restrict__ bias, float* __restrict__ bias_out) {
  __shared__ unsigned long long n[kMaxE];
  __shared__ long long part_sum[4];
  const int tid = threadIdx.x, parts = 1024 / E, e = tid % E, part = tid / E;
  if (tid < kMaxE) n[tid] = 0;
  __syncthreads();
  if (part < parts && part < S) {
    long long own = 0;
#pragma unroll 4
    for (int64_t s = part; s < S; s += parts) own += counts[s * E + e];
    atomicAdd(&n[e], static_cast<unsigned long long>(own));  // whole numbers: in any order
  }
  __syncthreads();
  if (tid < kMaxE) {
    long long sum = static_cast<long long>(n[tid]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) sum += __shfl_xor(sum, o, 64);
    if ((tid & 63) == 0) part_sum[tid >> 6] = sum;
  }
  __syncthreads();
  if (tid < E) {
    const long long diff = part_sum[0] + part_sum[1] + part_sum[2] + part_sum[3] - static_cast<long long>(n[tid]) * E;
    bias_out[tid] = diff == 0 ? bias[tid] : bias[tid] + (diff > 0 ? rate : -rate);
  }
}

// Sixteen lanes a token: more would be 2^32 threads in a launch.
constexpr int64_t kMaxTokens = (int64_t{1} << 28) - kTok;
int score_sizes(int64_t T, int E, int k) {
  if (E > kMaxE || k > kMaxK || T > kMaxTokens) return MOE_EUNSUPPORTED;
  return T >= 0 && E >= 1 && k >= 1 && k <= E && T * k < (1ll << 31) ? MOE_OK : MOE_EINVAL;
}
size_t score_ws_bytes(int64_t T, int E, int k) {
  return align_up(static_cast<size_t>(T * k) * 4, 256) + align_up(static_cast<size_t>(cdiv(T, kTok) * E) * 4, 256);
}

template <int C>
void launch_score_select(const ScoreArgs& a, hipStream_t s) {
  const size_t lds = align_up(static_cast<size_t>(a.E) * 8, 16) + (a.groups > 1 ? static_cast<size_t>(kTok) * a.E * 8 : 0);
  const dim3 grid(static_cast<unsigned>(a.nblk)), block(kSelThreads);
  if (a.E % 4 == 0) MOE_LAUNCH("score_select", (score_select_kernel<C, true>), grid, block, lds, s, a);
  else MOE_LAUNCH("score_select", (score_select_kernel<C, false>), grid, block, lds, s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_route_scored_workspace(int64_t T, int32_t E, int32_t k) {
  return score_sizes(T, E, k) == MOE_OK ? score_ws_bytes(T, E, k) : 0;
}

extern "C" int moe_route_scored(const float* logits, const float* bias, int64_t T, int32_t E, int32_t k, int score,
                                int32_t groups, int32_t top_groups, int32_t group_best, int renorm, float scale,
                                int32_t* topk_idx, float* gates, int32_t* counts, int32_t* offsets, int32_t* perm_src,
                                int32_t* perm_dst, int32_t* mx_blk_offsets, void* ws, size_t ws_bytes, void* stream) {
  const int sizes = score_sizes(T, E, k);
  if (sizes != MOE_OK) return sizes;
  if ((score != MOE_SOFTMAX && score != MOE_SIGMOID) || !std::isfinite(scale)) return MOE_EINVAL;
  if (groups < 1 || groups > E || E % groups || top_groups < 1 || top_groups > groups || group_best < 1 ||
      group_best > 2 || group_best > E / groups || static_cast<int64_t>(top_groups) * (E / groups) < k)
    return MOE_EINVAL;
  if (groups > 64) return MOE_EUNSUPPORTED;
  if (!counts || !offsets || !ws) return MOE_EINVAL;
  if (T > 0 && (!logits || !topk_idx || !gates || !perm_src || !perm_dst)) return MOE_EINVAL;
  for (const void* q : {static_cast<const void*>(logits), static_cast<const void*>(bias),
                        static_cast<const void*>(topk_idx), static_cast<const void*>(gates),
                        static_cast<const void*>(counts), static_cast<const void*>(offsets),
                        static_cast<const void*>(perm_src), static_cast<const void*>(perm_dst),
                        static_cast<const void*>(mx_blk_offsets), static_cast<const void*>(ws)})
    if (!aligned16(q)) return MOE_EINVAL;
  if (ws_bytes < score_ws_bytes(T, E, k)) return MOE_EWORKSPACE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t nblk = cdiv(T, kTok), R = T * k;
  int32_t* rank = static_cast<int32_t*>(ws);
  int32_t* blk = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + align_up(static_cast<size_t>(R) * 4, 256));
  if (T > 0) {
    const ScoreArgs a{logits, bias, T, E, k, score == MOE_SIGMOID, top_groups == groups ? 1 : groups,  // all stay
                      top_groups, group_best, renorm, scale, topk_idx, gates, rank, blk, nblk, counts, offsets, perm_src, perm_dst,
                      mx_blk_offsets};
    if (E <= 64) launch_score_select<4>(a, s);
    else if (E <= 128) launch_score_select<8>(a, s);
    else launch_score_select<16>(a, s);
  }
  if (nblk == 1) return launch_status();
  // few counts: every workgroup can sum them for itself, which is a launch less.  A thread walks its expert's counts one
  // after the other, so the number of workgroups decides, and for many experts what they all read.  Calls in a row, two
  // launches against three: 128 workgroups and 1, 8, 32 or 60 experts 9.6, 10.1, 10.7, 11.5 against 9.9, 10.5, 11.2, 11.5
  // us, 192 of them 11.0, 12.1, 12.5, 13.5 against 10.5, 11.1, 11.7, 12.0, 1024 with 8 experts 41 against 29; 128 experts
  // 11.4 against 12.3 (96 workgroups) and 12.6 against 12.3 (128), 256 experts 11.5 against 12.6 (48) and 14.7 against 13.4 (96)
  if (nblk > 0 && nblk <= 128 && nblk * E <= 12288) {
    MOE_LAUNCH("score_place", score_place_kernel, dim3(static_cast<unsigned>(nblk)), dim3(256), 0, s, topk_idx, rank, blk,
               nblk, R, k, E, counts, offsets, mx_blk_offsets, perm_src, perm_dst);
    return launch_status();
  }
  MOE_LAUNCH("score_scan", score_scan_kernel, dim3(static_cast<unsigned>(E)), dim3(64), 0, s, blk, nblk, counts);
  MOE_LAUNCH("score_scatter", score_scatter_kernel, dim3(static_cast<unsigned>(R > 0 ? cdiv(R, 256) : 1)), dim3(256), 0,
             s, topk_idx, rank, blk, nblk, R, k, E, counts, offsets, mx_blk_offsets, perm_src, perm_dst);
  return launch_status();
}

extern "C" int moe_route_scored_bwd(const float* logits, const int32_t* topk_idx, const float* dgates, int64_t T,
                                    int32_t E, int32_t k, int score, int renorm, float scale, int accumulate,
                                    float* dlogits, void* stream) {
  const int sizes = score_sizes(T, E, k);
  if (sizes != MOE_OK) return sizes;
  if ((score != MOE_SOFTMAX && score != MOE_SIGMOID) || !std::isfinite(scale)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_idx || !dgates || !dlogits) return MOE_EINVAL;
  if (!aligned16(logits) || !aligned16(topk_idx) || !aligned16(dgates) || !aligned16(dlogits)) return MOE_EINVAL;
  const ScoreBwdArgs a{logits, topk_idx, dgates, T, E, k, score == MOE_SIGMOID, renorm, accumulate, scale, dlogits};
  hipStream_t s = static_cast<hipStream_t>(stream);
  constexpr int kTokens = 256 / kRow;
  const dim3 grid(static_cast<unsigned>(cdiv(T, kTokens))), block(256);
  const size_t lds = static_cast<size_t>(kTokens) * E * 4;
  auto launch = [&](auto c) {
    constexpr int C = decltype(c)::value;
    if (E % 4 == 0) MOE_LAUNCH("score_bwd", (score_bwd_kernel<C, true>), grid, block, lds, s, a);
    else MOE_LAUNCH("score_bwd", (score_bwd_kernel<C, false>), grid, block, lds, s, a);
  };
  if (E <= 64) launch(std::integral_constant<int, 4>{});
  else if (E <= 128) launch(std::integral_constant<int, 8>{});
  else launch(std::integral_constant<int, 16>{});
  return launch_status();
}

extern "C" int moe_route_bias_update(const int32_t* counts, int64_t S, int32_t E, float rate, const float* bias,
                                     float* bias_out, void* stream) {
  if (E < 1 || E > kMaxE || S < 1 || !counts || !bias || !bias_out || !std::isfinite(rate)) return MOE_EINVAL;
  if (!aligned16(counts) || !aligned16(bias) || !aligned16(bias_out)) return MOE_EINVAL;
  MOE_LAUNCH("route_bias_update", bias_update_kernel, dim3(1), dim3(1024), 0, static_cast<hipStream_t>(stream), counts,
             S, E, rate, bias, bias_out);
  return launch_status();
}
