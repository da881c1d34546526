// The router's balance loss and z loss, with the per-expert counts, forward
// and backward.
//
//   p = softmax of a token's E logits, lse = their log-sum-exp.  Over the
//   tokens of sequence s that count (not masked, at least one logit above
//   -inf): n_s tokens, c[s,e] = chosen slots of expert e, P[s,e] = mean of p.
//   S' sequences have n_s > 0, N = sum n_s.
//     L_bal = alpha / S' sum_s E sum_e c[s,e] / (k n_s) P[s,e]
//     L_z   = zeta / N sum_t lse_t^2
//   gradient of L_bal and L_z for upstream (g0, g1):
//     dl[t,e] = p_e (a_e - sum_j a_j p_j) + g1 2 zeta / N lse p_e,
//     a_e = g0 alpha E c[s,e] / (k n_s^2 S')        (c has no gradient)
//
// The logits are at most a few tens of MB: the passes over them are short and
// latency counts.  A group of lanes owns a token (four experts per lane), so a
// wave works on 64 / lanes tokens at once.  Sums over tokens are built in
// a fixed order without float atomics: each workgroup walks the pieces that
// sequence borders cut out of its kTok consecutive tokens and writes one
// partial record per piece at slot (block + sequence).  Going from one piece to
// the next either the block or the sequence grows by one, so slots never
// collide, ceil(T / kTok) + S of them suffice, and those of a sequence are
// consecutive.  A second launch adds each sequence's records and its last
// workgroup to finish forms the two losses (partials in a fixed order again).
#include <algorithm>
#include <type_traits>

#include "common.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTok = 32;      // tokens per workgroup of the forward
constexpr int64_t kGridX = 1 << 16;  // workgroups of the backward beyond these go along y
constexpr int kCols = 16;     // experts per workgroup of the second launch
constexpr int kSumThreads = 512;

struct Ws {  // workspace regions
  float* p;       // [slots][E] sums of p
  int32_t* c;     // [slots][E] chosen counts
  float* z;       // [slots] sums of lse^2
  int32_t* n;     // [slots] tokens that count
  float* bal;     // [S][expert groups] sum_e c P / n of each sequence
  float* zs;      // [S] sums of lse^2 of each sequence
  int32_t* ticket;
};

int64_t slots_of(int64_t T, int64_t S) { return cdiv(T, kTok) + S; }

size_t ws_layout(int64_t T, int E, int64_t S, char* base, Ws* w) {
  const size_t slots = static_cast<size_t>(slots_of(T, S));
  size_t o = 0;
  auto take = [&](size_t bytes) {
    char* p = base + o;
    o += align_up(bytes, 256);
    return p;
  };
  char* p = take(slots * E * 4);
  char* c = take(slots * E * 4);
  char* z = take(slots * 4);
  char* n = take(slots * 4);
  char* b = take(static_cast<size_t>(S) * cdiv(E, kCols) * 4);
  char* q = take(static_cast<size_t>(S) * 4);
  char* t = take(4);
  if (w) *w = Ws{reinterpret_cast<float*>(p), reinterpret_cast<int32_t*>(c), reinterpret_cast<float*>(z),
                 reinterpret_cast<int32_t*>(n), reinterpret_cast<float*>(b), reinterpret_cast<float*>(q),
                 reinterpret_cast<int32_t*>(t)};
  return o;
}

// First token at or after which sequence s begins, within [0, T].
__device__ __forceinline__ int64_t seq_at(const int32_t* seq, int64_t s, int64_t S, int64_t T) {
  if (!seq) return s == 0 ? 0 : T;
  const int64_t v = seq[s];
  return v < 0 ? 0 : (v > T ? T : v);
}

// The sequence that holds token t (or begins next after it): the number of
// sequences that end at or before t, found 256 probes at a time.  All threads of
// the workgroup call it.
__device__ __forceinline__ int64_t first_seq(const int32_t* seq, int64_t S, int64_t T, int64_t t, int* cnt) {
  if (!seq) return 0;
  int64_t lo = 0, n = S;  // the answer is in [lo, lo + n]
  while (n > 0) {
    const int64_t step = (n + kThreads - 1) / kThreads, last = (threadIdx.x + 1) * step;  // thread's piece ends there
    if (threadIdx.x == 0) *cnt = 0;
    __syncthreads();
    if (last <= n && seq_at(seq, lo + last, S, T) <= t) atomicAdd(cnt, 1);
    __syncthreads();
    const int64_t whole = *cnt * step;
    __syncthreads();
    lo += whole;
    if (step == 1) break;
    n = n - whole < step ? n - whole : step;
  }
  return lo;
}

// Walk over the sequences' pieces within tokens [t0, t1): f(s, lo, hi) for each
// that is not empty.  Runs of empty sequences are skipped by another search.
template <class F>
__device__ __forceinline__ void each_piece(const int32_t* seq, int64_t S, int64_t T, int64_t t0, int64_t t1, int* cnt,
                                           F&& f) {
  for (int64_t s = first_seq(seq, S, T, t0, cnt); s < S;) {
    const int64_t from = seq_at(seq, s, S, T), to = seq_at(seq, s + 1, S, T);
    if (from >= t1) break;
    const int64_t lo = from < t0 ? t0 : from, hi = to > t1 ? t1 : to;
    if (lo < hi) {
      f(s, lo, hi);
      ++s;
    } else {
      const int64_t next = first_seq(seq, S, T, lo, cnt);
      s = next > s ? next : s + 1;
    }
  }
}

__device__ __forceinline__ double wave_sum_d(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ int wave_sum_i(int v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Lanes per token LPT; a lane holds experts 4 l .. 4 l + 3 of its token.
template <int LPT>
struct Row {
  static constexpr int kRows = 64 / LPT;  // tokens per wave and pass
  __device__ static __forceinline__ float max(float v) {
#pragma unroll
    for (int o = LPT / 2; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
  }
  __device__ static __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = LPT / 2; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
  }
  // sum over the wave's tokens (lanes of equal place in their group)
  __device__ static __forceinline__ float over_tokens(float v) {
#pragma unroll
    for (int o = 32; o >= LPT; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
  }
};

__device__ __forceinline__ void ld_logits(const float* l, int64_t t, int E, int e0, bool on, float (&v)[4]) {
  const float* p = l + t * E + e0;
  if (on && (E & 3) == 0 && e0 < E) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = on && e0 + i < E ? p[i] : -INFINITY;
  }
}

// v becomes exp(v - max); returns their sum over the token, and lse.  A token of
// -inf only gives zeros and the sum 0; NaN and +inf logits give the sum NaN
// (fmaxf passes over a NaN, its exponential does not).
template <int LPT>
__device__ __forceinline__ float softmax4(float (&v)[4], float& lse) {
  float m = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
  m = Row<LPT>::max(m);
  float s = 0.f;
  const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = expf(v[i] - mm);
    s += v[i];
  }
  s = Row<LPT>::sum(s);
  lse = mm + logf(s);
  return s;
}

struct FwdArgs {
  const float* logits;
  const int32_t* idx;
  const int32_t* seq;
  const uint8_t* mask;
  float* lse;
  int32_t* counts;
  float* probs;
  float* loss;
  float* norm;
  int64_t T, S;
  int E, k;
  float alpha, zeta;
  Ws ws;
};

template <int LPT>
__global__ __launch_bounds__(kThreads) void balance_partial_kernel(FwdArgs a) {
  constexpr int RW = Row<LPT>::kRows, kPass = kWaves * RW;
  __shared__ int s_cnt, s_hist[kMaxE], s_n[kWaves];
  __shared__ float s_p[kWaves][kMaxE], s_z[kWaves];
  __shared__ uint8_t s_on[kTok];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane % LPT, e0 = 4 * l, E = a.E;
  const int64_t b = blockIdx.x, t0 = b * kTok, t1 = t0 + kTok < a.T ? t0 + kTok : a.T;
  if (b == 0 && tid == 0) *a.ws.ticket = 0;
  // every token of the block: lse, and whether it counts by its mask and logits
  // (the pieces below take the sequences into account)
  constexpr int NP = (kTok + kPass - 1) / kPass;
  float p[NP][4], lse[NP];
#pragma unroll
  for (int q = 0; q < NP; ++q) {
    const int r = q * kPass + wave * RW + lane / LPT;
    const bool in = r < kTok && t0 + r < t1;
    ld_logits(a.logits, t0 + r, E, e0, in, p[q]);
  }
#pragma unroll
  for (int q = 0; q < NP; ++q) {
    const int r = q * kPass + wave * RW + lane / LPT;
    const bool in = r < kTok && t0 + r < t1;
    const float s = softmax4<LPT>(p[q], lse[q]);
    const bool on = in && s != 0.f && (!a.mask || a.mask[t0 + r]);  // NaN counts
#pragma unroll
    for (int i = 0; i < 4; ++i) p[q][i] = on ? p[q][i] / s : 0.f;
    if (!on) lse[q] = 0.f;
    if (l == 0 && r < kTok) s_on[r] = on;
    if (l == 0 && in) a.lse[t0 + r] = 0.f;
  }
  each_piece(a.seq, a.S, a.T, t0, t1, &s_cnt, [&](int64_t s, int64_t lo, int64_t hi) {
    for (int e = tid; e < E; e += kThreads) s_hist[e] = 0;
    __syncthreads();
    float ps[4] = {0.f, 0.f, 0.f, 0.f}, z = 0.f;
    int n = 0;
#pragma unroll
    for (int q = 0; q < NP; ++q) {
      const int r = q * kPass + wave * RW + lane / LPT;
      const bool here = r < kTok && t0 + r >= lo && t0 + r < hi;
      if (here && s_on[r]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) ps[i] += p[q][i];
        if (l == 0) {
          z += lse[q] * lse[q];
          n += 1;
          a.lse[t0 + r] = lse[q];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) ps[i] = Row<LPT>::over_tokens(ps[i]);
    z = wave_sum(z);
    n = wave_sum_i(n);
    if (lane < LPT)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e0 + i < E) s_p[wave][e0 + i] = ps[i];
    if (lane == 0) {
      s_z[wave] = z;
      s_n[wave] = n;
    }
    const int base = static_cast<int>(lo - t0);
    for (int i = tid; i < static_cast<int>(hi - lo) * a.k; i += kThreads) {
      const int e = a.idx[lo * a.k + i];
      if (s_on[base + i / a.k] && e >= 0 && e < E) atomicAdd(&s_hist[e], 1);
    }
    __syncthreads();
    const int64_t slot = b + s;
    for (int e = tid; e < E; e += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += s_p[w][e];
      a.ws.p[slot * E + e] = v;
      a.ws.c[slot * E + e] = s_hist[e];
    }
    if (tid == 0) {
      float zz = 0.f;
      int nn = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        zz += s_z[w];
        nn += s_n[w];
      }
      a.ws.z[slot] = zz;
      a.ws.n[slot] = nn;
    }
    __syncthreads();
  });
}

// Workgroup (x, y): experts [16 x, 16 x + 16) of sequences y, y + gridDim.y, ...
// The last workgroup of the launch to finish forms the losses; which one that
// is does not matter to the result.
__global__ __launch_bounds__(kSumThreads) void balance_sum_kernel(FwdArgs a) {
  constexpr int G = kSumThreads / kCols, W = kSumThreads / 64;
  __shared__ double s_p[G][kCols + 1], s_f[W];
  __shared__ int s_c[G][kCols + 1], s_i[W], s_last;
  const int tid = threadIdx.x, cl = tid % kCols, g = tid / kCols, E = a.E;
  const int e = blockIdx.x * kCols + cl;
  // partials cross workgroups as device-scope atomics, ordered by waiting for the
  // stores: a device-scope fence would write back a whole L2 per workgroup
  auto st = [](float* p, float v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  for (int64_t s = blockIdx.y; s < a.S; s += gridDim.y) {
    const int64_t lo = seq_at(a.seq, s, a.S, a.T), hi = seq_at(a.seq, s + 1, a.S, a.T);
    const int64_t f = lo < hi ? lo / kTok + s : 0, end = lo < hi ? (hi - 1) / kTok + s + 1 : 0;
    double p = 0.0, z = 0.0;
    int c = 0, n = 0;
    if (e < E)
#pragma unroll 4
      for (int64_t i = f + g; i < end; i += G) {
        p += static_cast<double>(a.ws.p[i * E + e]);
        c += a.ws.c[i * E + e];
      }
    for (int64_t i = f + tid; i < end; i += kSumThreads) {
      n += a.ws.n[i];
      z += static_cast<double>(a.ws.z[i]);
    }
    n = wave_sum_i(n);
    z = wave_sum_d(z);
    s_p[g][cl] = p;
    s_c[g][cl] = c;
    if ((tid & 63) == 0) {
      s_i[tid >> 6] = n;
      s_f[tid >> 6] = z;
    }
    __syncthreads();
    n = 0;
    z = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      n += s_i[w];
      z += s_f[w];
    }
    if (g == 0) {
#pragma unroll
      for (int k = 1; k < G; ++k) {
        p += s_p[k][cl];
        c += s_c[k][cl];
      }
      const double inv = n > 0 ? 1.0 / n : 0.0;
      float term = 0.f;
      if (e < E) {
        p *= inv;
        a.probs[s * E + e] = static_cast<float>(p);
        a.counts[s * E + e] = c;
        term = static_cast<float>(c * p * inv);
      }
#pragma unroll
      for (int o = kCols / 2; o >= 1; o >>= 1) term += __shfl_xor(term, o, 64);
      if (cl == 0) st(a.ws.bal + s * gridDim.x + blockIdx.x, term);
      if (cl == 0 && blockIdx.x == 0) {
        st(a.norm + 2 + s, static_cast<float>(n));
        st(a.ws.zs + s, static_cast<float>(z));
      }
    }
    __syncthreads();
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): thread 0 wrote this workgroup's partials
  if (tid == 0) {
    const int total = static_cast<int>(gridDim.x * gridDim.y);
    s_last = __hip_atomic_fetch_add(a.ws.ticket, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == total - 1;
  }
  __syncthreads();
  if (!s_last) return;
  auto ld = [](const float* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); };
  double v[4] = {0.0, 0.0, 0.0, 0.0};  // sum of terms, of lse^2, live sequences, tokens
  const int64_t terms = a.S * gridDim.x;
  for (int64_t i = tid; i < terms; i += kSumThreads) v[0] += ld(a.ws.bal + i);
  for (int64_t s = tid; s < a.S; s += kSumThreads) {
    const float n = ld(a.norm + 2 + s);
    v[1] += ld(a.ws.zs + s);
    v[2] += n > 0.f ? 1.0 : 0.0;
    v[3] += n;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = wave_sum_d(v[i]);
    __syncthreads();
    if ((tid & 63) == 0) s_f[tid >> 6] = v[i];
    __syncthreads();
    v[i] = 0.0;
    for (int w = 0; w < W; ++w) v[i] += s_f[w];
  }
  if (tid == 0) {
    a.loss[0] = v[2] > 0.0 ? static_cast<float>(a.alpha * E / (a.k * v[2]) * v[0]) : 0.f;
    a.loss[1] = v[3] > 0.0 && a.zeta != 0.f ? static_cast<float>(a.zeta / v[3] * v[1]) : 0.f;
    a.norm[0] = static_cast<float>(v[2]);
    a.norm[1] = static_cast<float>(v[3]);
  }
}

struct BwdArgs {
  const float *logits, *lse;
  const int32_t* counts;
  const float* norm;
  const int32_t* seq;
  const uint8_t* mask;
  const float* dloss;
  const int32_t* idx;
  const float *gates, *dgates;
  float* dlogits;
  int64_t T, S;
  int E, k;
  float alpha, zeta;
};

// The same walk over pieces as the forward; the softmax comes back as
// exp(l - lse) from the saved lse, divided by its sum: for logits far from zero
// the rounding of lse (half an ulp, all of log E at the type's lowest value)
// would be the relative error of every p.  A token of -inf only has lse 0 saved
// and gets zeros from the exponentials.  A workgroup
// takes the tokens that its lanes hold at once: with more, one after the other,
// their loads waited for each other (16384 x 128: 13.1 us at 32 tokens, 10.5 at
// the 8 of this kernel; 12.8 with a loop over the grid around it).
template <int LPT>
__global__ __launch_bounds__(kThreads) void balance_bwd_kernel(BwdArgs a) {
  constexpr int kPass = kThreads / LPT;
  __shared__ int s_cnt;
  const int l = threadIdx.x % LPT, e0 = 4 * l, E = a.E;
  const int64_t t0 = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * kPass;
  if (t0 >= a.T) return;
  const int64_t t1 = t0 + kPass < a.T ? t0 + kPass : a.T;
  const int64_t t = t0 + threadIdx.x / LPT;
  const bool on = t < t1;
  float p[4], dl[4] = {0.f, 0.f, 0.f, 0.f}, zc = 0.f;
  ld_logits(a.logits, t, E, e0, on, p);
  const float live = a.norm[0], ntot = a.norm[1];
  const float g0 = a.dloss ? a.dloss[0] : 1.f, g1 = a.dloss ? a.dloss[1] : 1.f;
  const float zs = ntot > 0.f ? g1 * 2.0f * a.zeta / ntot : 0.f;
  if (on) {
    const float lse = a.lse[t];
    const bool use = !a.mask || a.mask[t];
    zc = use ? zs * lse : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = use && e0 + i < E ? expf(p[i] - lse) : 0.f;
    if (a.gates) {
      const int64_t o = t * a.k;
      float dot = 0.f;
      for (int j = 0; j < a.k; ++j) dot += a.gates[o + j] * a.dgates[o + j];
      for (int j = 0; j < a.k; ++j) {
        const int c = a.idx[o + j] - e0;
        const float v = a.gates[o + j] * (a.dgates[o + j] - dot);
#pragma unroll
        for (int i = 0; i < 4; ++i) dl[i] += c == i ? v : 0.f;
      }
    }
  }
  each_piece(a.seq, a.S, a.T, t0, t1, &s_cnt, [&](int64_t s, int64_t lo, int64_t hi) {
    const float n = a.norm[2 + s];
    if (!(n > 0.f)) return;
    const float f = g0 * a.alpha * static_cast<float>(E) / (static_cast<float>(a.k) * n * n * live);
    const int even = static_cast<int>(static_cast<float>(a.k) * n / static_cast<float>(E));  // at most n: k <= E
    float c[4], dot = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // less about the average count, as a_e - sum_j a_j p_j does not see a common
      // number: the difference of the large terms would lose what near-even counts
      // differ by, and so would a count past 2^24 itself in fp32
      c[i] = e0 + i < E ? f * static_cast<float>(a.counts[s * E + e0 + i] - even) : 0.f;
      dot += c[i] * p[i];
      sum += p[i];
    }
    dot = Row<LPT>::sum(dot);
    sum = Row<LPT>::sum(sum);
    const float inv = 1.0f / sum;
    // a token that does not count has the sum 0 (one that does over E^-2, however coarse its lse);
    // 0 times an infinite upstream gradient would not be 0
    if (on && t >= lo && t < hi && sum != 0.f)
#pragma unroll
      for (int i = 0; i < 4; ++i) dl[i] += p[i] * inv * (c[i] - dot * inv + zc);
  });
  if (!on) return;
  float* o = a.dlogits + t * E + e0;
  if ((E & 3) == 0) {
    if (e0 < E) *reinterpret_cast<float4*>(o) = make_float4(dl[0], dl[1], dl[2], dl[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e0 + i < E) o[i] = dl[i];
  }
}

// Lanes per token: the smallest power of two that covers E with four experts each.
template <class F>
void by_lanes(int E, F&& f) {
  if (E <= 8) f(std::integral_constant<int, 2>{});
  else if (E <= 16) f(std::integral_constant<int, 4>{});
  else if (E <= 32) f(std::integral_constant<int, 8>{});
  else if (E <= 64) f(std::integral_constant<int, 16>{});
  else if (E <= 128) f(std::integral_constant<int, 32>{});
  else f(std::integral_constant<int, 64>{});
}

int check_sizes(int64_t T, int E, int k, int64_t S) {
  // a launch has fewer than 2^32 threads along x: the forward's, of kThreads for every kTok tokens begun
  constexpr int64_t kMaxT = ((int64_t{1} << 32) / kThreads - 1) * kTok;
  if (E > kMaxE || k > kMaxK || T > kMaxT) return MOE_EUNSUPPORTED;
  if (T < 0 || E < 1 || k < 1 || k > E || T * k >= (int64_t{1} << 31)) return MOE_EINVAL;
  if (S < 1 || S >= (int64_t{1} << 31)) return MOE_EINVAL;
  return MOE_OK;
}

bool finite(float v) { return v - v == 0.f; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t moe_balance_loss_workspace(int64_t T, int32_t E, int64_t S) {
  return check_sizes(T, E, 1, S) == MOE_OK ? ws_layout(T, E, S, nullptr, nullptr) : 0;
}

extern "C" int moe_balance_loss(const float* logits, const int32_t* topk_idx, int64_t T, int32_t E, int32_t k,
                                const int32_t* seq_offsets, int64_t S, const uint8_t* token_mask, float alpha,
                                float zeta, float* loss, int32_t* counts, float* probs, float* lse, float* norm,
                                void* ws, size_t ws_bytes, void* stream) {
  const int st = check_sizes(T, E, k, S);
  if (st != MOE_OK) return st;
  if ((!seq_offsets && S != 1) || !finite(alpha) || !finite(zeta)) return MOE_EINVAL;
  if (!loss || !counts || !probs || !norm || !ws) return MOE_EINVAL;
  if (T > 0 && (!logits || !topk_idx || !lse)) return MOE_EINVAL;
  for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(topk_idx),
                        static_cast<const void*>(seq_offsets), static_cast<const void*>(token_mask),
                        static_cast<const void*>(loss), static_cast<const void*>(counts),
                        static_cast<const void*>(probs), static_cast<const void*>(lse),
                        static_cast<const void*>(norm), static_cast<const void*>(ws)})
    if (!aligned16(p)) return MOE_EINVAL;
  if (ws_bytes < ws_layout(T, E, S, nullptr, nullptr)) return MOE_EWORKSPACE;
  FwdArgs a{logits, topk_idx, seq_offsets, token_mask, lse, counts, probs, loss, norm, T, S, E, k, alpha, zeta, {}};
  ws_layout(T, E, S, static_cast<char*>(ws), &a.ws);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t blocks = T > 0 ? cdiv(T, kTok) : 1;  // without tokens, one workgroup to clear the ticket
  by_lanes(E, [&](auto lpt) {
    MOE_LAUNCH("balance_partial", (balance_partial_kernel<decltype(lpt)::value>), dim3(static_cast<unsigned>(blocks)),
               dim3(kThreads), 0, s, a);
  });
  const dim3 grid(static_cast<unsigned>(cdiv(E, kCols)), static_cast<unsigned>(S < 4096 ? S : 4096));
  MOE_LAUNCH("balance_sum", balance_sum_kernel, grid, dim3(kSumThreads), 0, s, a);
  return launch_status();
}

extern "C" int moe_balance_loss_bwd(const float* logits, const float* lse, const int32_t* counts, const float* norm,
                                    int64_t T, int32_t E, int32_t k, const int32_t* seq_offsets, int64_t S,
                                    const uint8_t* token_mask, float alpha, float zeta, const float* dloss,
                                    const int32_t* topk_idx, const float* gates, const float* dgates, float* dlogits,
                                    void* stream) {
  const int st = check_sizes(T, E, k, S);
  if (st != MOE_OK) return st;
  if ((!seq_offsets && S != 1) || !finite(alpha) || !finite(zeta)) return MOE_EINVAL;
  if ((gates == nullptr) != (dgates == nullptr) || (gates && !topk_idx)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!logits || !lse || !counts || !norm || !dlogits) return MOE_EINVAL;
  for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(lse),
                        static_cast<const void*>(counts), static_cast<const void*>(norm),
                        static_cast<const void*>(seq_offsets), static_cast<const void*>(token_mask),
                        static_cast<const void*>(dloss), static_cast<const void*>(topk_idx),
                        static_cast<const void*>(gates), static_cast<const void*>(dgates),
                        static_cast<const void*>(dlogits)})
    if (!aligned16(p)) return MOE_EINVAL;
  const BwdArgs a{logits, lse, counts, norm, seq_offsets, token_mask, dloss, topk_idx, gates, dgates, dlogits,
                  T, S, E, k, alpha, zeta};
  by_lanes(E, [&](auto lpt) {
    const int64_t groups = cdiv(T * decltype(lpt)::value, kThreads), x = std::min(groups, kGridX);
    MOE_LAUNCH("balance_bwd", (balance_bwd_kernel<decltype(lpt)::value>),
               dim3(static_cast<unsigned>(x), static_cast<unsigned>(cdiv(groups, x))), dim3(kThreads), 0,
               static_cast<hipStream_t>(stream), a);
  });
  return launch_status();
}
