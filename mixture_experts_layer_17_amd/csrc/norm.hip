// Layer norm of token rows (forward and backward): the norm before the router
// and the experts.
//
//   forward   s = x (+ residual, rounded to the storage type), mu = mean(s),
//             rstd = 1 / sqrt(mean((s - mu)^2) + eps), y = (s - mu) rstd w + b
//   backward  h = (s - mu) rstd, v = dy w,
//             dx = rstd (v - mean(v) - h mean(v h)) (+ dres),
//             dw = sum_t dy h, db = sum_t dy
//
// Both directions are bound by HBM: every row is read once, kept in registers
// as stored (16-byte vectors), and written once.  All statistics and sums are
// fp32; each output is rounded once.  A row belongs to a wave, or to a
// workgroup of four waves when its vectors would not fit a wave's registers.
// The mean and the centred second moment of a row come from two passes over
// the registers inside a wave; waves are joined by the parallel-variance
// formula, so four waves cost one barrier.
//
// Rows need not be 16-byte aligned (any d): vectors are loaded and stored at
// element alignment, which the global memory instructions accept, and only the
// row's last partial vector goes element by element.
//
// The weight gradients are sums over the rows: each workgroup keeps its rows'
// partial sums in registers, writes them to the workspace once, and a second
// launch adds the workgroups' partials in a fixed order (no float atomics).
#include "common.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;

// The `n` (clamped to [0, kVec]) elements at p as one 16-byte vector, zeros beyond.
template <class T>
__device__ __forceinline__ uint4 ld_vec(const T* p, int n) {
  constexpr int V = Elem<T>::kVec;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (n >= V) {
    __builtin_memcpy(&v, p, 16);
  } else if (n > 0) {
    T t[V] = {};
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) t[i] = p[i];
    __builtin_memcpy(&v, t, 16);
  }
  return v;
}

// NT: streaming stores, for outputs larger than the caches (see stream_out).
template <bool NT, class T>
__device__ __forceinline__ void st_vec(T* p, int n, const uint4& v) {
  constexpr int V = Elem<T>::kVec;
  if (n >= V) {
    if constexpr (NT) {
      typedef unsigned int u32x4 __attribute__((ext_vector_type(4), aligned(2)));
      const u32x4 w = {v.x, v.y, v.z, v.w};
      __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
    } else {
      __builtin_memcpy(p, &v, 16);
    }
  } else if (n > 0) {
    T t[V];
    __builtin_memcpy(t, &v, 16);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = t[i];
  }
}

struct FwdArgs {
  const void *x, *res, *w, *b;
  void *y, *sum;
  float *mean, *rstd;
  int64_t T;
  int d;
  float eps;
};

struct BwdArgs {
  const void *dy, *x, *w, *dres;
  const float *mean, *rstd;
  void* dx;
  float* part;  // [2][gridDim.x][d]: dw then db partials; nullptr when neither is wanted
  int64_t T;
  int d;
};

// ---------------------------------------------------------------------------
// Forward, row in registers: TPR threads per row (64, or the workgroup's 256),
// NV vectors per thread.
// ---------------------------------------------------------------------------
template <class T, int NV, int TPR, bool RES, bool NT>
__global__ __launch_bounds__(kThreads) void layernorm_fwd_kernel(FwdArgs a) {
  constexpr int V = Elem<T>::kVec, RPB = kThreads / TPR;
  __shared__ float red[2][kThreads / 64][2];
  const int d = a.d, tl = threadIdx.x % TPR;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  uint4 w[NV], b[NV];
  int nv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + tl) * V;
    nv[i] = d - c;
    if (a.w) w[i] = ld_vec(static_cast<const T*>(a.w) + c, nv[i]);
    if (a.b) b[i] = ld_vec(static_cast<const T*>(a.b) + c, nv[i]);
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * RPB;
  int64_t t = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  uint4 xv[NV], rv[NV];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t o = row * d + (i * TPR + tl) * V;
      xv[i] = ld_vec(x + o, nv[i]);
      if constexpr (RES) rv[i] = ld_vec(res + o, nv[i]);
    }
  };
  if (t < a.T) load(t);
  for (int par = 0; t < a.T; t += step, par ^= 1) {
    float s[NV][V];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Elem<T>::unpack(xv[i], s[i]);
      if constexpr (RES) {
        float r[V];
        Elem<T>::unpack(rv[i], r);
#pragma unroll
        for (int j = 0; j < V; ++j) s[i][j] += r[j];
        const uint4 sv = Elem<T>::pack(s[i]);
        if (a.sum) st_vec<NT>(static_cast<T*>(a.sum) + t * d + (i * TPR + tl) * V, nv[i], sv);
        Elem<T>::unpack(sv, s[i]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) m += s[i][j];  // elements past the row are zero
    }
    if (t + step < a.T) load(t + step);  // in flight during this row's arithmetic
    // this wave's count, mean and centred second moment
    int cnt = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int first = (i * TPR + (tl & ~63)) * V;
      cnt += d - first < 0 ? 0 : (d - first > 64 * V ? 64 * V : d - first);
    }
    m = wave_sum(m) / static_cast<float>(cnt > 0 ? cnt : 1);
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float c = j < nv[i] ? s[i][j] - m : 0.f;
        q += c * c;
      }
    q = wave_sum(q);
    if constexpr (TPR > 64) {  // join the waves: total = sum of counts, M2 += n_w (m_w - mean)^2
      if ((threadIdx.x & 63) == 0) {
        red[par][threadIdx.x >> 6][0] = m * static_cast<float>(cnt);
        red[par][threadIdx.x >> 6][1] = q;
      }
      __syncthreads();
      float tot = 0.f, q2 = 0.f;
#pragma unroll
      for (int k = 0; k < TPR / 64; ++k) tot += red[par][k][0];
      const float mean = tot / static_cast<float>(d);
#pragma unroll
      for (int k = 0; k < TPR / 64; ++k) {
        int ck = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int first = (i * TPR + k * 64) * V;
          ck += d - first < 0 ? 0 : (d - first > 64 * V ? 64 * V : d - first);
        }
        const float dm = ck > 0 ? red[par][k][0] / static_cast<float>(ck) - mean : 0.f;
        q2 += red[par][k][1] + static_cast<float>(ck) * dm * dm;
      }
      m = mean;
      q = q2;
    }
    const float rs = 1.0f / sqrtf(q / static_cast<float>(d) + a.eps);
    if (tl == 0) {
      if (a.mean) a.mean[t] = m;
      if (a.rstd) a.rstd[t] = rs;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V], f[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = (s[i][j] - m) * rs;
      if (a.w) {
        Elem<T>::unpack(w[i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] *= f[j];
      }
      if (a.b) {
        Elem<T>::unpack(b[i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] += f[j];
      }
      st_vec<NT>(static_cast<T*>(a.y) + t * d + (i * TPR + tl) * V, nv[i], Elem<T>::pack(o));
    }
  }
}

// Sum over a workgroup of 256; `red` holds one float per wave and value.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[threadIdx.x >> 6][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 64; ++k) v[i] += red[k][i];
  }
  __syncthreads();
}

// Forward for rows too long for a workgroup's registers: three passes over the
// row, the later two from the caches.
template <class T, bool NT>
__global__ __launch_bounds__(kThreads) void layernorm_fwd_long_kernel(FwdArgs a) {
  constexpr int V = Elem<T>::kVec;
  __shared__ float red[kThreads / 64][1];
  const int d = a.d;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t o0 = t * d;
    auto row = [&](int c, float* s) {
      Elem<T>::unpack(ld_vec(static_cast<const T*>(a.x) + o0 + c, d - c), s);
      if (a.res) {
        float r[V];
        Elem<T>::unpack(ld_vec(static_cast<const T*>(a.res) + o0 + c, d - c), r);
  #pragma unroll
        for (int j = 0; j < V; ++j) s[j] += r[j];
        Elem<T>::unpack(Elem<T>::pack(s), s);
      }
    };
    float acc[1] = {0.f};
    for (int c = threadIdx.x * V; c < d; c += kThreads * V) {
      float s[V];
      row(c, s);
  #pragma unroll
      for (int j = 0; j < V; ++j) acc[0] += s[j];
    }
    block_sum(acc, red);
    const float m = acc[0] / static_cast<float>(d);
    acc[0] = 0.f;
    for (int c = threadIdx.x * V; c < d; c += kThreads * V) {
      float s[V];
      row(c, s);
  #pragma unroll
      for (int j = 0; j < V; ++j) {
        const float e = c + j < d ? s[j] - m : 0.f;
        acc[0] += e * e;
      }
    }
    block_sum(acc, red);
    const float rs = 1.0f / sqrtf(acc[0] / static_cast<float>(d) + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[t] = m;
      if (a.rstd) a.rstd[t] = rs;
    }
    for (int c = threadIdx.x * V; c < d; c += kThreads * V) {
      float s[V], f[V];
      row(c, s);
      if (a.sum) st_vec<NT>(static_cast<T*>(a.sum) + o0 + c, d - c, Elem<T>::pack(s));
  #pragma unroll
      for (int j = 0; j < V; ++j) s[j] = (s[j] - m) * rs;
      if (a.w) {
        Elem<T>::unpack(ld_vec(static_cast<const T*>(a.w) + c, d - c), f);
  #pragma unroll
        for (int j = 0; j < V; ++j) s[j] *= f[j];
      }
      if (a.b) {
        Elem<T>::unpack(ld_vec(static_cast<const T*>(a.b) + c, d - c), f);
  #pragma unroll
        for (int j = 0; j < V; ++j) s[j] += f[j];
      }
      st_vec<NT>(static_cast<T*>(a.y) + o0 + c, d - c, Elem<T>::pack(s));
    }
  }
}

// ---------------------------------------------------------------------------
// Backward, row in registers; the workgroup's dw, db partials too.
// ---------------------------------------------------------------------------
template <class T, int NV, int TPR, bool WGRAD, bool NT>
__global__ __launch_bounds__(kThreads) void layernorm_bwd_kernel(BwdArgs a) {
  constexpr int V = Elem<T>::kVec, RPB = kThreads / TPR;
  __shared__ float red[2][kThreads / 64][2];
  __shared__ float comb[RPB][RPB > 1 && WGRAD ? TPR * NV * V : 1];
  const int d = a.d, tl = threadIdx.x % TPR;
  const T* dy = static_cast<const T*>(a.dy);
  const T* x = static_cast<const T*>(a.x);
  const T* dres = static_cast<const T*>(a.dres);
  uint4 w[NV];
  int nv[NV];
  float gw[WGRAD ? NV : 1][V], gb[WGRAD ? NV : 1][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * TPR + tl) * V;
    nv[i] = d - c;
    if (a.w) w[i] = ld_vec(static_cast<const T*>(a.w) + c, nv[i]);
    if constexpr (WGRAD)
#pragma unroll
      for (int j = 0; j < V; ++j) gw[i][j] = gb[i][j] = 0.f;
  }
  const float inv_d = 1.0f / static_cast<float>(d);
  const int64_t step = static_cast<int64_t>(gridDim.x) * RPB;
  int64_t t = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / TPR;
  uint4 gv[NV], xv[NV], rv[NV];
  float mu = 0.f, rs = 0.f;
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t o = row * d + (i * TPR + tl) * V;
      gv[i] = ld_vec(dy + o, nv[i]);
      xv[i] = ld_vec(x + o, nv[i]);
      if (dres) rv[i] = ld_vec(dres + o, nv[i]);
    }
    mu = a.mean[row];
    rs = a.rstd[row];
  };
  if (t < a.T) load(t);
  for (int par = 0; t < a.T; t += step, par ^= 1) {
    float h[NV][V], v[NV][V];
    uint4 rcur[NV];
    float s[2] = {0.f, 0.f};
    const float m = mu, r = rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Elem<T>::unpack(gv[i], v[i]);
      Elem<T>::unpack(xv[i], h[i]);
      rcur[i] = rv[i];
      float f[V];
      if (a.w) Elem<T>::unpack(w[i], f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        // past the row dy is zero, so v and both partials stay zero there
        h[i][j] = (h[i][j] - m) * r;
        if constexpr (WGRAD) {
          gw[i][j] += v[i][j] * h[i][j];
          gb[i][j] += v[i][j];
        }
        if (a.w) v[i][j] *= f[j];
        s[0] += v[i][j];
        s[1] += v[i][j] * h[i][j];
      }
    }
    if (t + step < a.T) load(t + step);
    s[0] = wave_sum(s[0]);
    s[1] = wave_sum(s[1]);
    if constexpr (TPR > 64) {
      if ((threadIdx.x & 63) == 0) {
        red[par][threadIdx.x >> 6][0] = s[0];
        red[par][threadIdx.x >> 6][1] = s[1];
      }
      __syncthreads();
      s[0] = s[1] = 0.f;
#pragma unroll
      for (int k = 0; k < TPR / 64; ++k) {
        s[0] += red[par][k][0];
        s[1] += red[par][k][1];
      }
    }
    const float c0 = s[0] * inv_d, c1 = s[1] * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float o[V], f[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = r * (v[i][j] - c0 - h[i][j] * c1);
      if (dres) {
        Elem<T>::unpack(rcur[i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] += f[j];
      }
      st_vec<NT>(static_cast<T*>(a.dx) + t * d + (i * TPR + tl) * V, nv[i], Elem<T>::pack(o));
    }
  }
  if constexpr (WGRAD) {
    float* pw = a.part + static_cast<int64_t>(blockIdx.x) * d;
    float* pb = a.part + (static_cast<int64_t>(gridDim.x) + blockIdx.x) * d;
    const int grp = threadIdx.x / TPR;
    auto flush = [&](float (&g)[NV][V], float* dst) {
      if constexpr (RPB > 1) {  // the row groups meet in LDS and are added in order
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) comb[grp][(i * V + j) * TPR + tl] = g[i][j];
        __syncthreads();
        for (int k = threadIdx.x; k < TPR * NV * V; k += kThreads) {
          const int c = (k / TPR / V * TPR + k % TPR) * V + k / TPR % V;  // entry (i V + j) TPR + tl
          float s = comb[0][k];
#pragma unroll
          for (int r = 1; r < RPB; ++r) s += comb[r][k];
          if (c < d) dst[c] = s;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j < nv[i]) dst[(i * TPR + tl) * V + j] = g[i][j];
      }
    };
    flush(gw, pw);
    flush(gb, pb);
  }
}

// Backward of long rows: dx in two passes per row; dw, db by columns below.
template <class T, bool NT>
__global__ __launch_bounds__(kThreads) void layernorm_bwd_long_kernel(BwdArgs a) {
  constexpr int V = Elem<T>::kVec;
  __shared__ float red[kThreads / 64][2];
  const int d = a.d;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t o0 = t * d;
    const float m = a.mean[t], r = a.rstd[t];
    auto row = [&](int c, float* v, float* h) {
      Elem<T>::unpack(ld_vec(static_cast<const T*>(a.dy) + o0 + c, d - c), v);
      Elem<T>::unpack(ld_vec(static_cast<const T*>(a.x) + o0 + c, d - c), h);
      if (a.w) {
        float f[V];
        Elem<T>::unpack(ld_vec(static_cast<const T*>(a.w) + c, d - c), f);
  #pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= f[j];
      }
  #pragma unroll
      for (int j = 0; j < V; ++j) h[j] = (h[j] - m) * r;
    };
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x * V; c < d; c += kThreads * V) {
      float v[V], h[V];
      row(c, v, h);
  #pragma unroll
      for (int j = 0; j < V; ++j) {
        s[0] += v[j];
        s[1] += v[j] * h[j];
      }
    }
    block_sum(s, red);
    const float c0 = s[0] / static_cast<float>(d), c1 = s[1] / static_cast<float>(d);
    for (int c = threadIdx.x * V; c < d; c += kThreads * V) {
      float v[V], h[V], o[V];
      row(c, v, h);
  #pragma unroll
      for (int j = 0; j < V; ++j) o[j] = r * (v[j] - c0 - h[j] * c1);
      if (a.dres) {
        Elem<T>::unpack(ld_vec(static_cast<const T*>(a.dres) + o0 + c, d - c), v);
  #pragma unroll
        for (int j = 0; j < V; ++j) o[j] += v[j];
      }
      st_vec<NT>(static_cast<T*>(a.dx) + o0 + c, d - c, Elem<T>::pack(o));
    }
  }
}

// dw, db partials of long rows: workgroup (x, y) sums the rows y, y + gridDim.y,
// ... of 256 columns.
template <class T>
__global__ __launch_bounds__(kThreads) void layernorm_wgrad_long_kernel(BwdArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.d) return;
  float gw = 0.f, gb = 0.f;
  for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
    const float g = Elem<T>::load1(a.dy, t * a.d + c);
    gw += g * ((Elem<T>::load1(a.x, t * a.d + c) - a.mean[t]) * a.rstd[t]);
    gb += g;
  }
  a.part[static_cast<int64_t>(blockIdx.y) * a.d + c] = gw;
  a.part[(static_cast<int64_t>(gridDim.y) + blockIdx.y) * a.d + c] = gb;
}

// Sums the G partial rows of dw (blockIdx.y = 0) or db (1): 16 columns per
// workgroup, 16 row groups joined in order through LDS.
template <class T>
__global__ __launch_bounds__(kThreads) void layernorm_wgrad_sum_kernel(const float* __restrict__ part, int G, int d,
                                                                       T* dw, T* db) {
  __shared__ float red[16][17];
  T* out = blockIdx.y ? db : dw;
  if (!out) return;
  const int cl = threadIdx.x % 16, g = threadIdx.x / 16;
  const int c = blockIdx.x * 16 + cl;
  const float* p = part + static_cast<int64_t>(blockIdx.y) * G * d;
  float s = 0.f;
  if (c < d)
#pragma unroll 8
    for (int r = g; r < G; r += 16) s += p[static_cast<int64_t>(r) * d + c];
  red[g][cl] = s;
  __syncthreads();
  if (g == 0 && c < d) {
#pragma unroll
    for (int k = 1; k < 16; ++k) s += red[k][cl];
    Elem<T>::store1(out, c, s);
  }
}

// Threads per row and vectors per thread that hold a row of d elements in
// registers (vec elements per vector): a wave with up to 4 vectors per lane,
// else the workgroup with up to kMaxNv.  nv = 0: the long-row kernels.
constexpr int kWaveNv = 4, kMaxNv = 4;
struct Shape {
  int tpr, nv;
};
Shape shape_for(int d, int vec) {
  for (int tpr = 64; tpr <= kThreads; tpr *= 4)
    for (int nv = 1; nv <= (tpr == 64 ? kWaveNv : kMaxNv); nv *= 2)
      if (static_cast<int64_t>(tpr) * nv * vec >= d) return {tpr, nv};
  return {kThreads, 0};
}

// Outputs that fill the L2s (8 x 4 MB) leave by streaming stores; smaller ones stay
// cached for the router and the dispatch that read them.  For the kernel alone the
// streaming stores are the faster ones from 8 MB on (rows of 2048 bf16 with a
// residual: 8 MB 11.9 -> 9.3 us, 24 MB 21.9 -> 19.6, 32 MB 26.4 -> 24.5, 128 MB
// 104 -> 86, 6.2 TB/s; their backward at 32 MB 30.6 -> 29.8), but a reader that
// follows loses by them: norm and a 32-expert router together 308 -> 311 us at 16 MB,
// 355 -> 368 at 31, 357 -> 373 at 32, 1010 -> 1031 at 128.  A training step of eight
// experts is the same with either at 32 and at 64 MB (1563 and 1565, 2921 and 2920 us).
bool stream_out(int64_t T, int d, int bytes) { return T * d * bytes >= int64_t{32} << 20; }

constexpr int kMaxBlocks = 2048;  // forward: up to eight workgroups per compute unit, looping over rows
unsigned long_grid(int64_t T) { return static_cast<unsigned>(T < kMaxBlocks ? T : kMaxBlocks); }

// Workgroups of the backward, each writing 2 d partial sums: one per compute unit
// where a workgroup has four rows in flight (8192 rows of 2048: 35 us against 44
// us with two), two where it has one (16384 rows of 4096: 115 us against 120 us).
constexpr int kMaxGroups = 512;
int bwd_groups(int64_t T, int tpr = kThreads) {
  const int64_t most = tpr == 64 ? kMaxGroups / 2 : kMaxGroups, n = cdiv(T > 0 ? T : 1, kThreads / tpr);
  return static_cast<int>(n < most ? n : most);
}

size_t bwd_ws_bytes(int64_t T, int d) { return static_cast<size_t>(2) * bwd_groups(T) * d * sizeof(float); }

template <class T, int NV, int TPR, bool NT>
void launch_fwd(const FwdArgs& a, hipStream_t s) {
  const int64_t blocks = cdiv(a.T, kThreads / TPR);
  const dim3 grid(static_cast<unsigned>(blocks < kMaxBlocks ? blocks : kMaxBlocks));
  if (a.res) MOE_LAUNCH("layernorm", (layernorm_fwd_kernel<T, NV, TPR, true, NT>), grid, dim3(kThreads), 0, s, a);
  else MOE_LAUNCH("layernorm", (layernorm_fwd_kernel<T, NV, TPR, false, NT>), grid, dim3(kThreads), 0, s, a);
}

template <class T, bool NT>
int run_fwd(const FwdArgs& a, hipStream_t s) {
  const Shape sh = shape_for(a.d, Elem<T>::kVec);
  if (sh.nv == 0) {
    MOE_LAUNCH("layernorm", (layernorm_fwd_long_kernel<T, NT>), dim3(long_grid(a.T)), dim3(kThreads), 0, s, a);
  } else if (sh.tpr == 64) {
    if (sh.nv == 1) launch_fwd<T, 1, 64, NT>(a, s);
    else if (sh.nv == 2) launch_fwd<T, 2, 64, NT>(a, s);
    else launch_fwd<T, 4, 64, NT>(a, s);
  } else {
    if (sh.nv == 2) launch_fwd<T, 2, 256, NT>(a, s);
    else launch_fwd<T, 4, 256, NT>(a, s);
  }
  return launch_status();
}

template <class T, int NV, int TPR, bool NT>
void launch_bwd(const BwdArgs& a, int G, hipStream_t s) {
  if (a.part)
    MOE_LAUNCH("layernorm_bwd", (layernorm_bwd_kernel<T, NV, TPR, true, NT>), dim3(G), dim3(kThreads), 0, s, a);
  else
    MOE_LAUNCH("layernorm_bwd", (layernorm_bwd_kernel<T, NV, TPR, false, NT>), dim3(G), dim3(kThreads), 0, s, a);
}

template <class T, bool NT>
int run_bwd(const BwdArgs& a, void* dw, void* db, hipStream_t s) {
  const Shape sh = shape_for(a.d, Elem<T>::kVec);
  int G = bwd_groups(a.T, sh.tpr);
  if (a.T == 0) {
    G = 0;  // no rows: the sums are zero
  } else if (sh.nv == 0) {
    if (a.part) {  // first: dx may take the place of dy or x
      G = G < 64 ? G : 64;
      MOE_LAUNCH("layernorm_wgrad", (layernorm_wgrad_long_kernel<T>),
                 dim3(static_cast<unsigned>(cdiv(a.d, kThreads)), G), dim3(kThreads), 0, s, a);
    }
    MOE_LAUNCH("layernorm_bwd", (layernorm_bwd_long_kernel<T, NT>), dim3(long_grid(a.T)), dim3(kThreads), 0, s, a);
  } else if (sh.tpr == 64) {
    if (sh.nv == 1) launch_bwd<T, 1, 64, NT>(a, G, s);
    else if (sh.nv == 2) launch_bwd<T, 2, 64, NT>(a, G, s);
    else launch_bwd<T, 4, 64, NT>(a, G, s);
  } else {
    if (sh.nv == 2) launch_bwd<T, 2, 256, NT>(a, G, s);
    else launch_bwd<T, 4, 256, NT>(a, G, s);
  }
  if (a.part)
    MOE_LAUNCH("layernorm_wgrad_sum", (layernorm_wgrad_sum_kernel<T>), dim3(static_cast<unsigned>(cdiv(a.d, 16)), 2),
               dim3(kThreads), 0, s, a.part, G, a.d, static_cast<T*>(dw), static_cast<T*>(db));
  return launch_status();
}

constexpr int kMaxD = 1 << 20;

bool norm_size_ok(int64_t T, int32_t d) { return T >= 0 && T < (int64_t{1} << 31) && d >= 1 && d <= kMaxD; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_layernorm(const void* x, const void* residual, const void* weight, const void* bias, int dtype,
                             int64_t T, int32_t d, float eps, void* y, void* sum, float* mean, float* rstd,
                             void* stream) {
  if (!norm_size_ok(T, d)) return d > kMaxD ? MOE_EUNSUPPORTED : MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL;
  if (!(eps >= 0.f) || !(eps < 3.0e38f)) return MOE_EINVAL;
  if (sum && !residual) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!x || !y) return MOE_EINVAL;
  for (const void* p : {x, residual, weight, bias, static_cast<const void*>(y), static_cast<const void*>(sum),
                        static_cast<const void*>(mean), static_cast<const void*>(rstd)})
    if (!aligned16(p)) return MOE_EINVAL;
  const FwdArgs a{x, residual, weight, bias, y, sum, mean, rstd, T, d, eps};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool nt = stream_out(T, d, dtype == MOE_F32 ? 4 : 2);
  if (dtype == MOE_F32) return nt ? run_fwd<float, true>(a, s) : run_fwd<float, false>(a, s);
  return nt ? run_fwd<uint16_t, true>(a, s) : run_fwd<uint16_t, false>(a, s);
}

extern "C" size_t moe_layernorm_bwd_workspace(int64_t T, int32_t d) {
  return norm_size_ok(T, d) ? bwd_ws_bytes(T, d) : 0;
}

extern "C" int moe_layernorm_bwd(const void* dy, const void* x, const void* weight, const float* mean,
                                 const float* rstd, const void* dres, int dtype, int64_t T, int32_t d, void* dx,
                                 void* dw, void* db, void* ws, size_t ws_bytes, void* stream) {
  if (!norm_size_ok(T, d)) return d > kMaxD ? MOE_EUNSUPPORTED : MOE_EINVAL;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_EINVAL;
  if (T > 0 && (!dy || !x || !mean || !rstd || !dx)) return MOE_EINVAL;
  for (const void* p : {dy, x, weight, static_cast<const void*>(mean), static_cast<const void*>(rstd), dres,
                        static_cast<const void*>(dx), static_cast<const void*>(dw), static_cast<const void*>(db),
                        static_cast<const void*>(ws)})
    if (!aligned16(p)) return MOE_EINVAL;
  if (dw || db) {
    if (!ws) return MOE_EINVAL;
    if (ws_bytes < bwd_ws_bytes(T, d)) return MOE_EWORKSPACE;
  }
  const BwdArgs a{dy, x, weight, dres, mean, rstd, dx, dw || db ? static_cast<float*>(ws) : nullptr, T, d};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool nt = stream_out(T, d, dtype == MOE_F32 ? 4 : 2);
  if (dtype == MOE_F32) return nt ? run_bwd<float, true>(a, dw, db, s) : run_bwd<float, false>(a, dw, db, s);
  return nt ? run_bwd<uint16_t, true>(a, dw, db, s) : run_bwd<uint16_t, false>(a, dw, db, s);
}
