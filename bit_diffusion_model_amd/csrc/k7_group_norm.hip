// Kernel 7: group norm with an activation, channels last, and the same norm leaving as
// 8-bit codes with one scale per position (the input of the W8A8 product).
//
// Mathematics: X [B][S][C], C = G cpg.  For image b and group g, over the S positions and the
// group's cpg channels: mean, var (biased); y = act((x - mean) / sqrt(var + eps) gamma_c +
// beta_c), x - mean formed first so that a mean far from zero costs no digits.
//
// Bound by HBM: x read, y written, once each at best.  Three kernels:
//  * k7_one: a block holds one image's group in registers: x read once, mean and variance by
//    two exact passes over the registers, one launch.  Where the group fits (32 values per
//    thread of 1024);
//  * k7_stats, then k7_apply (or k7_apply_quant): statistics per block of positions, and the
//    output pass, which first joins the blocks' statistics (by itself where there are few,
//    after k7_join where there are many).  A thread keeps the same V consecutive channels over
//    all its positions, so group boundaries may fall anywhere: sums are kept per channel and
//    meet per group in LDS.
// Statistics in fp32 without cancellation: a block's pivot p is the mean of the first rows that
// it holds in registers; it sums d = x - p and d^2, so (mean, M2) = (p + sum d / n, sum d^2 -
// (sum d)^2 / n); blocks are joined in fp64 around the first block's mean m_0: mean = m_0 +
// sum n_i (m_i - m_0) / n, M2 = sum (M2_i + n_i (m_i - m_0)^2) - n (mean - m_0)^2 (the pairwise
// formula of Chan, Golub and LeVeque, summed).
#include <type_traits>

#include "../../include/svdq.h"
#include "int8.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

constexpr int GN_NT = 256;

// ---- vectors of V channels; rows are 4-byte aligned for V > 1

typedef uint32_t u32x4a __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2a __attribute__((ext_vector_type(2), aligned(4)));

template <typename T, int V>
struct Vec {  // V values as loaded
  static constexpr int W = V * (int)sizeof(T) / 4;
  uint32_t w[W < 1 ? 1 : W];
};

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> loadv(const T* p) {
  Vec<T, V> r;
  constexpr int W = Vec<T, V>::W;
  if constexpr (W >= 4) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const u32x4a q = reinterpret_cast<const u32x4a*>(p)[i];
      r.w[4 * i] = q.x, r.w[4 * i + 1] = q.y, r.w[4 * i + 2] = q.z, r.w[4 * i + 3] = q.w;
    }
  } else if constexpr (W == 2) {
    const u32x2a q = *reinterpret_cast<const u32x2a*>(p);
    r.w[0] = q.x, r.w[1] = q.y;
  } else if constexpr (W == 1) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    r.w[0] = *p;
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void valuev(const Vec<T, V>& r, float v[V]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = __uint_as_float(r.w[e]);
  } else if constexpr (V == 1) {
    v[0] = __uint_as_float(r.w[0] << 16);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = e & 1 ? bf16_hi_to_f32(r.w[e / 2]) : bf16_lo_to_f32(r.w[e / 2]);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

template <typename TY, int V>
__device__ __forceinline__ void storev(TY* p, const float v[V]) {
  constexpr int W = V * (int)sizeof(TY) / 4;
  uint32_t w[W < 1 ? 1 : W];
  if constexpr (sizeof(TY) == 4) {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = __float_as_uint(v[e]);
  } else if constexpr (V > 1) {
#pragma unroll
    for (int e = 0; e < V; e += 2) w[e / 2] = pack_bf16(v[e], v[e + 1]);
  }
  if constexpr (W >= 4) {
#pragma unroll
    for (int i = 0; i < W / 4; ++i)
      reinterpret_cast<u32x4a*>(p)[i] = u32x4a{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
  } else if constexpr (W == 2) {
    *reinterpret_cast<u32x2a*>(p) = u32x2a{w[0], w[1]};
  } else if constexpr (W == 1) {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  } else {
    *reinterpret_cast<__bf16*>(p) = (__bf16)v[0];
  }
}

// SiLU y / (1 + exp(-y)): a large negative y gives y times 1 / inf = -0.  GELU in its exact form.
__device__ __forceinline__ float norm_act(float y, int act) {
  if (act == SVDQ_GN_SILU) return y * __builtin_amdgcn_rcpf(1.0f + __expf(-y));
  if (act == SVDQ_GN_GELU) return gelu_erf(y);
  return y;
}

// ---- one launch: a block per (group, image)

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// Sum over the block (at most 16 waves), in the same order on every call
__device__ __forceinline__ float block_sum(float v, float* scratch) {
  const int waves = (int)((blockDim.x + 63) >> 6);
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < waves; ++i) s += scratch[i];
  return s;
}

// NV vectors of V channels per thread.  stat != NULL: the statistics alone, (mean, rstd) to stat[b][g].
template <typename T, typename TY, int V, int NV>
__global__ __launch_bounds__(1024) void k7_one(const T* __restrict__ X, int64_t bsx, int64_t ldx, int S, int C, int G,
                                               float eps, const float* __restrict__ gamma,
                                               const float* __restrict__ beta, int act, TY* __restrict__ Y, int64_t bsy,
                                               int64_t ldy, float2* __restrict__ stat) {
  extern __shared__ float lds[];  // gamma, beta of the group
  __shared__ float scratch[16];
  const int cpg = C / G, c0 = (int)blockIdx.x * cpg, vpr = cpg / V, total = S * vpr;
  const T* x = X + blockIdx.y * bsx + c0;
  // the thread's vectors t, t + threads, ..: (row, col) advance by the quotient and the rest
  const int nt = (int)blockDim.x, dr = nt / vpr, dc = nt - dr * vpr;
  const int r0 = (int)threadIdx.x / vpr, q0 = (int)threadIdx.x - r0 * vpr;
  Vec<T, V> raw[NV];
  int r = r0, q = q0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = r < S;  // past the end: the first vector again, not used
    raw[j] = loadv<T, V>(x + (in ? r * ldx + q * V : 0));
    q += dc, r += dr;
    if (q >= vpr) q -= vpr, ++r;
  }
  if (!stat)
    for (int c = threadIdx.x; c < cpg; c += nt) {
      lds[c] = gamma ? gamma[c0 + c] : 1.0f;
      lds[cpg + c] = beta ? beta[c0 + c] : 0.0f;
    }
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[V], t = 0.0f;
    valuev<T, V>(raw[j], v);
#pragma unroll
    for (int e = 0; e < V; ++e) t += v[e];
    s += (int)threadIdx.x + j * nt < total ? t : 0.0f;
  }
  const float n = (float)S * (float)cpg;
  const float mean = block_sum(s, scratch) / n;
  s = 0.0f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[V], t = 0.0f;
    valuev<T, V>(raw[j], v);
#pragma unroll
    for (int e = 0; e < V; ++e) t += (v[e] - mean) * (v[e] - mean);
    s += (int)threadIdx.x + j * nt < total ? t : 0.0f;
  }
  const float rstd = 1.0f / sqrtf(block_sum(s, scratch) / n + eps);
  if (stat) {
    if (threadIdx.x == 0) stat[(int64_t)blockIdx.y * G + blockIdx.x] = make_float2(mean, rstd);
    return;
  }
  TY* y = Y + blockIdx.y * bsy + c0;
  r = r0, q = q0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (r < S) {
      float v[V];
      valuev<T, V>(raw[j], v);
#pragma unroll
      for (int e = 0; e < V; ++e)
        v[e] = norm_act((v[e] - mean) * (rstd * lds[q * V + e]) + lds[cpg + q * V + e], act);
      storev<TY, V>(y + r * ldy + q * V, v);
    }
    q += dc, r += dr;
    if (q >= vpr) q -= vpr, ++r;
  }
}

// ---- statistics per block of positions

// The threads' places: ct columns of V channels side by side, rp positions below each other.
struct Place {
  int ct, rp, col, row;
  bool on;
};
__host__ __device__ __forceinline__ int place_ct(int cv) { return cv < GN_NT ? cv : GN_NT; }
__device__ __forceinline__ Place place(int cv) {
  Place p;
  p.ct = place_ct(cv);
  p.rp = GN_NT / p.ct;
  p.col = threadIdx.x % p.ct;
  p.row = threadIdx.x / p.ct;
  p.on = p.row < p.rp;
  return p;
}

// Sums per group of the block's per-channel values red[r][c] (r < rp, C channels): out[g].
// 2^k threads per group (as many as there are), joined by shuffles inside a wave.
__device__ __forceinline__ void group_sums(const float2* red, int rp, int C, int G, float2* out) {
  const int cpg = C / G;
  int tpg = 1;
  while (tpg < 64 && tpg * 2 * G <= GN_NT) tpg *= 2;
  const int per = GN_NT / tpg, dr = tpg / cpg, dc = tpg - dr * cpg;
  for (int g0 = 0; g0 < G; g0 += per) {
    const int g = g0 + threadIdx.x / tpg, t = threadIdx.x % tpg;
    float2 s = make_float2(0.0f, 0.0f);
    if (g < G) {
      int r = t / cpg, c = t - r * cpg;
      while (r < rp) {
        const float2 v = red[r * C + g * cpg + c];
        s.x += v.x, s.y += v.y;
        c += dc, r += dr;
        if (c >= cpg) c -= cpg, ++r;
      }
    }
    for (int m = tpg / 2; m >= 1; m >>= 1) s.x += __shfl_xor(s.x, m, 64), s.y += __shfl_xor(s.y, m, 64);
    if (g < G && t == 0) out[g] = s;
  }
}

// Statistics of positions [blockIdx.x * chunk, + chunk) of image blockIdx.y: part[b][i][g] =
// (mean, M2).  LDS: red [rp C], gsum [G] (float2), piv [G].  HELD rows per thread stay in
// registers while the pivot is found; with more than GN_NT columns they are read again.
template <typename T, int V>
__global__ __launch_bounds__(GN_NT) void k7_stats(const T* __restrict__ X, int64_t bsx, int64_t ldx, int64_t S, int C,
                                                  int G, int64_t chunk, float2* __restrict__ part) {
  extern __shared__ float lds[];
  constexpr int HELD = 8;
  const int cv = C / V, cpg = C / G;
  const Place pl = place(cv);
  float2* red = reinterpret_cast<float2*>(lds);
  float2* gsum = red + pl.rp * C;
  float* piv = reinterpret_cast<float*>(gsum + G);
  const int64_t r0 = (int64_t)blockIdx.x * chunk;
  const int rows = (int)(r0 + chunk < S ? chunk : S - r0);
  const T* x = X + blockIdx.y * bsx + r0 * ldx;
  const int first = rows < HELD * pl.rp ? rows : HELD * pl.rp;

  Vec<T, V> raw[HELD];
  for (int c = pl.col; c < cv && pl.on; c += pl.ct) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      const int r = pl.row + i * pl.rp;
      raw[i] = loadv<T, V>(x + (r < rows ? r : 0) * ldx + c * V);
    }
    float s[V] = {};
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
      float v[V];
      valuev<T, V>(raw[i], v);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += pl.row + i * pl.rp < rows ? v[e] : 0.0f;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[pl.row * C + c * V + e] = make_float2(s[e], 0.0f);
  }
  __syncthreads();
  group_sums(red, pl.rp, C, G, gsum);
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += GN_NT) piv[g] = gsum[g].x / (float)(first * cpg);
  __syncthreads();

  for (int c = pl.col; c < cv && pl.on; c += pl.ct) {
    float p[V], s[V] = {}, q[V] = {};
    {
      int g = c * V / cpg, in = c * V - g * cpg;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        p[e] = piv[g];
        if (++in == cpg) in = 0, ++g;
      }
    }
    auto add = [&](const Vec<T, V>& w, bool on) {
      float v[V];
      valuev<T, V>(w, v);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = on ? v[e] - p[e] : 0.0f;
        s[e] += d;
        q[e] += d * d;
      }
    };
    if (cv > GN_NT) {  // several columns per thread: the registers hold the last one's rows
#pragma unroll
      for (int i = 0; i < HELD; ++i) {
        const int r = pl.row + i * pl.rp;
        raw[i] = loadv<T, V>(x + (r < rows ? r : 0) * ldx + c * V);
      }
    }
#pragma unroll
    for (int i = 0; i < HELD; ++i) add(raw[i], pl.row + i * pl.rp < rows);
    // the rest, HELD rows' loads in flight at once
    for (int i = pl.row + HELD * pl.rp; i < rows; i += HELD * pl.rp) {
#pragma unroll
      for (int j = 0; j < HELD; ++j) {
        const int r = i + j * pl.rp;
        raw[j] = loadv<T, V>(x + (r < rows ? r : 0) * ldx + c * V);
      }
#pragma unroll
      for (int j = 0; j < HELD; ++j) add(raw[j], i + j * pl.rp < rows);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[pl.row * C + c * V + e] = make_float2(s[e], q[e]);
  }
  __syncthreads();
  group_sums(red, pl.rp, C, G, gsum);
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += GN_NT) {
    const double n = (double)rows * cpg, d = gsum[g].x;
    part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * G + g] =
        make_float2((float)(piv[g] + d / n), (float)fmax(gsum[g].y - d * d / n, 0.0));
  }
}

// ---- joining the blocks' statistics

struct Stats {
  const float2* at;  // parts == 0: (mean, rstd) [B][G]; otherwise (mean, M2) [B][parts][G]
  int parts;
  int64_t S, chunk;
  int C, G;
  float eps;
};

struct Join {
  double n, d, q;
};
// One block's (mean, M2) around m0
__device__ __forceinline__ void join_add(Join& j, const Stats& st, int i, float2 v, float m0) {
  const double n = (double)((i + 1) * st.chunk < st.S ? st.chunk : st.S - i * st.chunk) * (st.C / st.G);
  const double d = (double)v.x - (double)m0;
  j.n += n;
  j.d += n * d;
  j.q += (double)v.y + n * d * d;
}
// A NaN or an infinity leaves NaN statistics, as the formula does (the maximum would drop it)
__device__ __forceinline__ float2 join_end(const Join& j, float m0, float eps) {
  const double d = j.d / j.n;
  double var = j.q / j.n - d * d;
  if (var < 0.0) var = 0.0;
  return make_float2((float)((double)m0 + d), 1.0f / sqrtf((float)var + eps));
}

// (mean, rstd) of all groups of image b into out[G] (LDS); 256 threads, scratch [256]
__device__ __forceinline__ void join_groups(const Stats& st, int64_t b, float2* out, Join* scratch) {
  if (st.parts == 0) {
    for (int g = threadIdx.x; g < st.G; g += GN_NT) out[g] = st.at[b * st.G + g];
    __syncthreads();
    return;
  }
  const float2* p = st.at + b * st.parts * (int64_t)st.G;
  const int width = st.G < GN_NT ? st.G : GN_NT, rows = GN_NT / width;
  for (int g0 = 0; g0 < st.G; g0 += width) {
    const int g = g0 + (int)threadIdx.x % width, r = (int)threadIdx.x / width;
    Join j = {0.0, 0.0, 0.0};
    const bool on = r < rows && g < st.G;
    const float m0 = on ? p[g].x : 0.0f;
    if (on)
      for (int i = r; i < st.parts; i += rows) join_add(j, st, i, p[(int64_t)i * st.G + g], m0);
    scratch[threadIdx.x] = j;
    __syncthreads();
    if (on && r == 0) {
      for (int i = 1; i < rows; ++i) {
        const Join o = scratch[i * width + (int)threadIdx.x];
        j.n += o.n, j.d += o.d, j.q += o.q;
      }
      out[g] = join_end(j, m0, st.eps);
    }
    __syncthreads();
  }
}

// Many blocks: group blockIdx.x of image blockIdx.y by a block of its own
__global__ __launch_bounds__(GN_NT) void k7_join(Stats st, float2* __restrict__ out) {
  __shared__ Join scratch[GN_NT];
  const float2* p = st.at + (int64_t)blockIdx.y * st.parts * st.G + blockIdx.x;
  const float m0 = p[0].x;
  Join j = {0.0, 0.0, 0.0};
  for (int i = threadIdx.x; i < st.parts; i += GN_NT) join_add(j, st, i, p[(int64_t)i * st.G], m0);
  scratch[threadIdx.x] = j;
  for (int m = GN_NT / 2; m >= 1; m >>= 1) {
    __syncthreads();
    if ((int)threadIdx.x < m) {
      const Join o = scratch[threadIdx.x + m];
      j.n += o.n, j.d += o.d, j.q += o.q;
      scratch[threadIdx.x] = j;
    }
  }
  if (threadIdx.x == 0) out[(int64_t)blockIdx.y * st.G + blockIdx.x] = join_end(j, m0, st.eps);
}

// ---- the output pass

// Positions [i * chunk, + chunk) of image blockIdx.y, i counted from the end: the statistics pass
// ended there, so that part of x is the likeliest to be in cache still.
template <typename T, typename TY, int V>
__global__ __launch_bounds__(GN_NT) void k7_apply(const T* __restrict__ X, int64_t bsx, int64_t ldx, int64_t chunk,
                                                  Stats st, const float* __restrict__ gamma,
                                                  const float* __restrict__ beta, int act, TY* __restrict__ Y,
                                                  int64_t bsy, int64_t ldy) {
  extern __shared__ float lds[];
  __shared__ Join scratch[GN_NT];
  float2* stat = reinterpret_cast<float2*>(lds);
  constexpr int U = 4;
  const int C = st.C, cv = C / V, cpg = C / st.G;
  const Place pl = place(cv);
  const int64_t r0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * chunk;
  const int rows = (int)(r0 + chunk < st.S ? chunk : st.S - r0);
  const T* x = X + blockIdx.y * bsx + r0 * ldx;
  TY* y = Y + blockIdx.y * bsy + r0 * ldy;
  Vec<T, V> raw[U];
  auto load = [&](int c, int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = i + u * pl.rp;
      raw[u] = loadv<T, V>(x + (r < rows ? r : 0) * ldx + c * V);
    }
  };
  if (pl.on) load(pl.col, pl.row);  // under way while the statistics are joined
  join_groups(st, blockIdx.y, stat, scratch);
  if (!pl.on) return;
  for (int c = pl.col; c < cv; c += pl.ct) {
    float mean[V], a[V], b[V];
    int g = c * V / cpg, in = c * V - g * cpg;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      mean[e] = stat[g].x;
      a[e] = stat[g].y * (gamma ? gamma[c * V + e] : 1.0f);
      b[e] = beta ? beta[c * V + e] : 0.0f;
      if (++in == cpg) in = 0, ++g;
    }
    if (c != pl.col) load(c, pl.row);
    for (int i = pl.row; i < rows; i += U * pl.rp) {
      if (i != pl.row) load(c, i);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = i + u * pl.rp;
        if (r >= rows) break;
        float v[V];
        valuev<T, V>(raw[u], v);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = norm_act((v[e] - mean[e]) * a[e] + b[e], act);
        storev<TY, V>(y + r * ldy + c * V, v);
      }
    }
  }
}

// The output pass into codes: a wave takes whole positions (rows of C channels), NC chunks of
// 512 channels in registers.  Per channel (mean, rstd gamma, beta, inv_s) wait in LDS, eight planes
// of C / 8 so that neighbouring lanes read neighbouring 16 bytes.
template <typename T, bool VEC, int NC>
__global__ __launch_bounds__(GN_NT) void k7_apply_quant(const T* __restrict__ X, int64_t bsx, int64_t ldx,
                                                        int64_t chunk, Stats st, const float* __restrict__ gamma,
                                                        const float* __restrict__ beta, int act,
                                                        const float* __restrict__ inv_s, int8_t* __restrict__ qX,
                                                        int64_t ldq, float* __restrict__ sX) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ Join scratch[GN_NT];
  const int C = st.C, cpg = C / st.G, c8 = (C + 7) / 8;
  float4* coef = reinterpret_cast<float4*>(lds);
  float2* stat = reinterpret_cast<float2*>(coef + 8 * c8);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t r0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * chunk;
  const int rows = (int)(r0 + chunk < st.S ? chunk : st.S - r0);
  typedef Row<T, VEC> RowX;
  auto row_at = [&](int i) { return RowX(X + blockIdx.y * bsx + (r0 + (i < rows ? i : 0)) * ldx, C); };
  typename RowX::Raw raw[NC];
  {
    const RowX x = row_at(wave);
#pragma unroll
    for (int j = 0; j < NC; ++j) raw[j] = x.load(8 * lane + 512 * j);
  }
  join_groups(st, blockIdx.y, stat, scratch);
  for (int c = threadIdx.x; c < 8 * c8; c += GN_NT) {
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // channels past C: value act(0) * 0
    if (c < C) {
      const float2 s = stat[c / cpg];
      f = make_float4(s.x, s.y * (gamma ? gamma[c] : 1.0f), beta ? beta[c] : 0.0f, inv_s ? inv_s[c] : 1.0f);
    }
    coef[(c & 7) * c8 + (c >> 3)] = f;
  }
  __syncthreads();
  for (int i = wave; i < rows; i += 4) {
    const RowX x = row_at(i);
    float v[NC][8];
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k8 = lane + 64 * j;
      x.value(raw[j], 8 * k8, v[j]);
      const bool in = k8 < c8;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 f = coef[e * c8 + (in ? k8 : 0)];
        v[j][e] = in ? norm_act((v[j][e] - f.x) * f.y + f.z, act) * f.w : 0.0f;
        a = umax(a, abs_bits(v[j][e]));
      }
    }
    const RowX next = row_at(i + 4);  // the next row's loads under this row's reduction
#pragma unroll
    for (int j = 0; j < NC; ++j) raw[j] = next.load(8 * lane + 512 * j);
    float s, r;
    row_scale(wave_umax(a), s, r);
    const int64_t row = blockIdx.y * st.S + r0 + i;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int64_t k = 8 * (lane + 64 * j);
      if (k < ldq)
        *reinterpret_cast<uint2*>(qX + row * ldq + k) = make_uint2(codes4(v[j][0], v[j][1], v[j][2], v[j][3], r),
                                                                   codes4(v[j][4], v[j][5], v[j][6], v[j][7], r));
    }
    if (lane == 0) sX[row] = s;
  }
}

// ---- launches

bool vec_ok(const void* p, int64_t bs, int64_t ld, int dtype) {
  return rows_aligned4(p, ld, dtype) && (dtype == 0 || bs % 2 == 0);
}

// Vector width of k7_one: the widest of 8, 4, 2 that divides a group and keeps 4-byte alignment
int one_width(int cpg, bool vec, int dtype) {
  for (int v = 8; v > 1; v /= 2)
    if (cpg % v == 0 && (vec || dtype == 0)) return v;
  return 1;
}

template <typename T, typename TY, int V, int NV>
void launch_one_nv(const NormArgs& a, void* Y, int64_t bsy, int64_t ldy, float2* stat, hipStream_t st) {
  const int cpg = a.C / a.G;
  const int64_t vectors = a.S * (cpg / V);
  int64_t nt = ((vectors + NV - 1) / NV + 63) / 64 * 64;
  if (nt > 1024) nt = 1024;
  hipLaunchKernelGGL((k7_one<T, TY, V, NV>), dim3((uint32_t)a.G, (uint32_t)a.B), dim3((uint32_t)nt), (size_t)cpg * 8, st,
                     static_cast<const T*>(a.X), a.bsx, a.ldx, (int)a.S, a.C, a.G, a.eps, a.gamma, a.beta, a.act,
                     static_cast<TY*>(Y), bsy, ldy, stat);
}
template <typename T, typename TY, int V>
void launch_one_v(const NormArgs& a, void* Y, int64_t bsy, int64_t ldy, float2* stat, hipStream_t st) {
  // 8 values per thread where 1024 threads then hold the group, otherwise 32
  if (a.S * (a.C / a.G) <= 8 * 1024) launch_one_nv<T, TY, V, 8 / V>(a, Y, bsy, ldy, stat, st);
  else launch_one_nv<T, TY, V, 32 / V>(a, Y, bsy, ldy, stat, st);
}
template <typename T, typename TY>
void launch_one(const NormArgs& a, int width, void* Y, int64_t bsy, int64_t ldy, float2* stat, hipStream_t st) {
  if (width == 8) launch_one_v<T, TY, 8>(a, Y, bsy, ldy, stat, st);
  else if (width == 4) launch_one_v<T, TY, 4>(a, Y, bsy, ldy, stat, st);
  else if (width == 2) launch_one_v<T, TY, 2>(a, Y, bsy, ldy, stat, st);
  else launch_one_v<T, TY, 1>(a, Y, bsy, ldy, stat, st);
}

template <typename T, int V>
void launch_stats(const NormArgs& a, const NormPlan& p, float2* part, hipStream_t st) {
  const int rp = GN_NT / place_ct(a.C / V);
  const size_t bytes = (size_t)rp * a.C * 8 + (size_t)a.G * 12;
  hipLaunchKernelGGL((k7_stats<T, V>), dim3(p.parts, (uint32_t)a.B), dim3(GN_NT), bytes, st,
                     static_cast<const T*>(a.X), a.bsx, a.ldx, a.S, a.C, a.G, p.chunk, part);
}

template <typename T, typename TY, int V>
void launch_apply(const NormArgs& a, const NormPlan& p, const Stats& s, void* Y, int64_t bsy, int64_t ldy,
                  hipStream_t st) {
  hipLaunchKernelGGL((k7_apply<T, TY, V>), dim3(p.blocks, (uint32_t)a.B), dim3(GN_NT), (size_t)a.G * 8, st,
                     static_cast<const T*>(a.X), a.bsx, a.ldx, p.rows, s, a.gamma, a.beta, a.act,
                     static_cast<TY*>(Y), bsy, ldy);
}

// Statistics for an output pass: by k7_one where a group fits a block, else by blocks of positions
Stats run_stats(const NormArgs& a, const NormPlan& p, void* ws, hipStream_t st) {
  float2* part = static_cast<float2*>(ws);
  Stats s{part, 0, a.S, p.chunk, a.C, a.G, a.eps};
  const bool vec = vec_ok(a.X, a.bsx, a.ldx, a.xdtype);
  if (p.one) {
    const int w = one_width(a.C / a.G, vec, a.xdtype);
    a.xdtype == 0 ? launch_one<float, float>(a, w, nullptr, 0, 0, part, st)
                  : launch_one<uint16_t, uint16_t>(a, w, nullptr, 0, 0, part, st);
    return s;
  }
  const bool v8 = a.C % 8 == 0 && vec;
  if (a.xdtype == 0) v8 ? launch_stats<float, 8>(a, p, part, st) : launch_stats<float, 1>(a, p, part, st);
  else v8 ? launch_stats<uint16_t, 8>(a, p, part, st) : launch_stats<uint16_t, 1>(a, p, part, st);
  s.parts = (int)p.parts;
  if (p.join) {
    float2* out = part + (size_t)a.B * p.parts * a.G;
    hipLaunchKernelGGL(k7_join, dim3((uint32_t)a.G, (uint32_t)a.B), dim3(GN_NT), 0, st, s, out);
    s.at = out;
    s.parts = 0;
  }
  return s;
}

}  // namespace

NormPlan plan_norm(int64_t B, int64_t S, int C, int G) {
  NormPlan p{};
  const int64_t cpg = C / G;
  p.one = S * cpg <= 32 * 1024;
  // statistics: blocks of at least 8 rows per thread; up to 256 blocks joined by every output
  // block itself, more (up to 1024) by a launch of their own
  const int ct = place_ct(C % 8 == 0 ? C / 8 : C), rp = GN_NT / ct;
  const int64_t least = 8 * rp;
  auto split = [&](int64_t blocks) {
    int64_t chunk = (S * B + blocks - 1) / blocks;
    return chunk < least ? least : chunk;
  };
  p.chunk = split(256);
  p.join = p.chunk * C > 131072;
  if (p.join) p.chunk = split(1024);
  p.parts = (uint32_t)((S + p.chunk - 1) / p.chunk);
  p.bytes = ((size_t)B * p.parts * G + (size_t)B * G) * sizeof(float2);
  // the output pass: about 2048 blocks of at least 4 rows per thread
  p.rows = (S * B + 2047) / 2048;
  if (p.rows < 4 * rp) p.rows = 4 * rp;
  p.blocks = (uint32_t)((S + p.rows - 1) / p.rows);
  return p;
}

hipError_t launch_norm(const NormArgs& a, void* Y, int ydtype, int64_t bsy, int64_t ldy, void* ws, hipStream_t st) {
  const NormPlan p = plan_norm(a.B, a.S, a.C, a.G);
  const bool vec = vec_ok(a.X, a.bsx, a.ldx, a.xdtype) && vec_ok(Y, bsy, ldy, ydtype);
  if (p.one) {
    const int w = one_width(a.C / a.G, vec, a.xdtype == 0 && ydtype == 0 ? 0 : 1);
    if (a.xdtype == 0 && ydtype == 0) launch_one<float, float>(a, w, Y, bsy, ldy, nullptr, st);
    else if (a.xdtype == 0) launch_one<float, uint16_t>(a, w, Y, bsy, ldy, nullptr, st);
    else if (ydtype == 0) launch_one<uint16_t, float>(a, w, Y, bsy, ldy, nullptr, st);
    else launch_one<uint16_t, uint16_t>(a, w, Y, bsy, ldy, nullptr, st);
    return hipGetLastError();
  }
  const Stats s = run_stats(a, p, ws, st);
  const bool v8 = a.C % 8 == 0 && vec;
  if (a.xdtype == 0 && ydtype == 0)
    v8 ? launch_apply<float, float, 8>(a, p, s, Y, bsy, ldy, st) : launch_apply<float, float, 1>(a, p, s, Y, bsy, ldy, st);
  else if (a.xdtype == 0)
    v8 ? launch_apply<float, uint16_t, 8>(a, p, s, Y, bsy, ldy, st) : launch_apply<float, uint16_t, 1>(a, p, s, Y, bsy, ldy, st);
  else if (ydtype == 0)
    v8 ? launch_apply<uint16_t, float, 8>(a, p, s, Y, bsy, ldy, st) : launch_apply<uint16_t, float, 1>(a, p, s, Y, bsy, ldy, st);
  else
    v8 ? launch_apply<uint16_t, uint16_t, 8>(a, p, s, Y, bsy, ldy, st) : launch_apply<uint16_t, uint16_t, 1>(a, p, s, Y, bsy, ldy, st);
  return hipGetLastError();
}

hipError_t launch_norm_quant(const NormArgs& a, const float* inv_s, int8_t* qX, float* sX, void* ws, hipStream_t st) {
  const NormPlan p = plan_norm(a.B, a.S, a.C, a.G);
  const Stats s = run_stats(a, p, ws, st);
  const bool vec = vec_ok(a.X, a.bsx, a.ldx, a.xdtype);
  const size_t bytes = (size_t)((a.C + 7) / 8) * 8 * 16 + (size_t)a.G * 8;
  const int64_t ldq = i8_ld(a.C);
  // about 2048 blocks of at least 8 rows (two per wave)
  int64_t rows = (a.S * a.B + 2047) / 2048;
  if (rows < 8) rows = 8;
  const dim3 g((uint32_t)((a.S + rows - 1) / rows), (uint32_t)a.B), b(GN_NT);
  auto go = [&](auto kernel, auto x) {
    hipLaunchKernelGGL(kernel, g, b, bytes, st, x, a.bsx, a.ldx, rows, s, a.gamma, a.beta, a.act, inv_s, qX, ldq, sX);
  };
  const float* x32 = static_cast<const float*>(a.X);
  const uint16_t* x16 = static_cast<const uint16_t*>(a.X);
  auto by_type = [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    if (a.xdtype == 0) go(k7_apply_quant<float, true, NC>, x32);
    else vec ? go(k7_apply_quant<uint16_t, true, NC>, x16) : go(k7_apply_quant<uint16_t, false, NC>, x16);
  };
  if (ldq <= 512) by_type(std::integral_constant<int, 1>{});
  else if (ldq <= 1024) by_type(std::integral_constant<int, 2>{});
  else if (ldq <= 2048) by_type(std::integral_constant<int, 4>{});
  else by_type(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

}  // namespace svdq
