// Kernel 7: group norm with an activation, channels last, and the same norm leaving as
// 8-bit codes with one scale per position (the input of the W8A8 product).
//
// Mathematics: X [B][S][C], C = G cpg.  For image b and group g, over the S positions and the
// group's cpg channels: mean, var (biased); y = act((x - mean) / sqrt(var + eps) gamma_c +
// beta_c), x - mean formed first so that a mean far from zero costs no digits.
//
// Bound by HBM where x and y pass the 256 MB cache (262144x256 fp32, x read twice and y written: 157 us a
// call with inputs in turn, 5.1 TB/s; 151 on one input over and over), by the cache below that (65536x256
// bf16 26 us), by launches and the blocks' meeting in the smallest.  Three kernels:
//  * k7_one: a block holds one image's group in registers: x read once, mean and variance by
//    two passes over the registers, one launch.  Taken where a group's values fit the
//    registers of 1024 threads in few loads (the plan below holds the figures: 2x64x1280 in
//    groups of 40 3.4 us against the two launches' 9.7);
//  * k7_stats, then k7_apply (or k7_apply_quant): statistics per block of positions, and the
//    output pass, which first joins the blocks' statistics (by itself where there are few,
//    after k7_join where there are many: an output block would read them all).  A thread keeps
//    the same V consecutive channels over all its positions, so group boundaries may fall
//    anywhere: sums are kept per channel and meet per group in LDS.
// Statistics in fp32: a thread sums d = x - p and d^2 per channel, so that (mean, M2) = (p + sum d / n,
// sum d^2 - (sum d)^2 / n).  p is its first value for eight positions, then these eight's mean: M2 >= 8 (p - mean)^2,
// so that the subtraction loses at most a factor n / 8.  n, the thread's positions, is at most 512 (16 at
// 65536x256, 64 at 262144x256); with the first value for all of 4096 positions a first value 30 standard
// deviations off cost 5e-4 of M2.
// Threads, then blocks, are joined by mean = sum n_i mean_i / n, M2 = sum (M2_i + n_i (mean_i -
// mean)^2) (the pairwise formula of Chan, Golub and LeVeque, summed).
#include <type_traits>

#include "../../include/svdq.h"
#include "int8.hpp"
#include "kernels.hpp"
#include "vec.hpp"

namespace svdq {
namespace {

constexpr int ST_NT = 256, AP_NT = 256;  // threads of the statistics and output passes (1024: 16-27 us for 10)

// The activation of N values (one branch for all): SiLU y / (1 + exp(-y)), exp as a power of 2 (a large
// negative y gives y times 1 / inf = -0); GELU in its exact form, for FINE outputs by the longer fit: fp32, and codes,
// where the shorter one's 8.5e-6 would move one rounding in a thousand.
template <bool FINE, int N>
__device__ __forceinline__ void norm_act(float (&y)[N], int act) {
  if (act == SVDQ_GN_SILU) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      y[e] *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(y[e] * -1.44269504088896341f));
  } else if (act == SVDQ_GN_GELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = FINE ? gelu_erf(y[e]) : gelu5(y[e]);
  }
}

// ---- one launch: a block per (group, image)

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
__device__ __forceinline__ float2 block_sum(float2 v, float2* scratch) {
  const int waves = (int)((blockDim.x + 63) >> 6);
  v = make_float2(wave_sum(v.x), wave_sum(v.y));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
  for (int i = 0; i < waves; ++i) s.x += scratch[i].x, s.y += scratch[i].y;
  return s;
}

// The sum of the values over n is a first mean p only, off by the roundings of a sum (a constant group: two bits of
// 3000.7, which eps = 1e-5 would show as 0.15); the second pass takes d = x - p, which is small or exact, and gives
// mean = p + sum d / n, M2 = sum d^2 - (sum d)^2 / n.
//
// Y may be X: a thread loads all that it needs before it stores, so neither is __restrict__.
// NV vectors of V channels per thread.  stat != NULL: the statistics alone, (mean, rstd) to stat[b][g].
template <typename T, typename TY, int V, int NV>
__global__ __launch_bounds__(1024) void k7_one(const T* X, int64_t bsx, int64_t ldx, int S, int C, int G, float eps,
                                               const float* __restrict__ gamma, const float* __restrict__ beta,
                                               int act, TY* Y, int64_t bsy,
                                               int64_t ldy, float2* __restrict__ stat) {
  extern __shared__ float lds[];  // gamma, beta of the group
  __shared__ float2 scratch[16];
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
  const float p = block_sum(s, &scratch[0].x) / n;
  float2 sums = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float v[V];
    float2 t = make_float2(0.0f, 0.0f);
    valuev<T, V>(raw[j], v);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = v[e] - p;
      t.x += d;
      t.y = fmaf(d, d, t.y);
    }
    if ((int)threadIdx.x + j * nt < total) sums.x += t.x, sums.y += t.y;
  }
  sums = block_sum(sums, scratch);
  const float mean = p + sums.x / n, m2 = sums.y - sums.x * (sums.x / n);
  const float rstd = 1.0f / sqrtf((m2 < 0.0f ? 0.0f : m2) / n + eps);  // (a NaN passes)
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
      for (int e = 0; e < V; ++e) v[e] = fmaf(v[e] - mean, rstd * lds[q * V + e], lds[cpg + q * V + e]);
      norm_act<sizeof(TY) == 4>(v, act);
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
__host__ __device__ __forceinline__ int place_ct(int cv, int nt) { return cv < nt ? cv : nt; }
template <int NT>
__device__ __forceinline__ Place place(int cv) {
  Place p;
  p.ct = place_ct(cv, NT);
  p.rp = NT / p.ct;
  p.row = threadIdx.x / p.ct;
  p.col = threadIdx.x - p.row * p.ct;
  p.on = p.row < p.rp;
  return p;
}

// Joins the threads' statistics red[r][c] = (mean, M2) (r < rp: positions r, r + rp, .. of `rows`)
// per group: out[g] = (mean, M2).  2^k threads per group (as many as there are), shuffles in a wave.
__device__ __forceinline__ void group_stats(const float2* red, int rp, int rows, int C, int G, float2* __restrict__ out) {
  const int cpg = C / G;
  int tpg = 1;
  while (tpg < 64 && tpg * 2 * G <= ST_NT) tpg *= 2;
  const int per = ST_NT / tpg, dr = tpg / cpg, dc = tpg - dr * cpg, t = threadIdx.x % tpg;
  const int full = rows / rp, more = rows - full * rp;  // rows of threads r < more have one position more
  const int top = rows < rp ? rows : rp;
  for (int g0 = 0; g0 < G; g0 += per) {
    const int g = g0 + threadIdx.x / tpg;
    const float2* at = red + (g < G ? g : 0) * cpg;
    const float m0 = at[0].x;
    auto each = [&](auto f) {
      float s = 0.0f;
      int r = t / cpg, c = t - r * cpg;
      while (r < top) {
        s += f((float)(full + (r < more)), at[r * C + c]);
        c += dc, r += dr;
        if (c >= cpg) c -= cpg, ++r;
      }
      for (int m = tpg / 2; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
      return s;
    };
    const float mean = m0 + each([&](float n, float2 v) { return n * (v.x - m0); }) / ((float)rows * (float)cpg);
    const float m2 = each([&](float n, float2 v) { return v.y + n * (v.x - mean) * (v.x - mean); });
    if (g < G && t == 0) out[g] = make_float2(mean, m2);
  }
}

// Statistics of positions [blockIdx.x * chunk, + chunk) of image blockIdx.y: part[b][i][g] =
// (mean, M2).  LDS: red [rp C].
template <typename T, int V>
__global__ __launch_bounds__(ST_NT) void k7_stats(const T* __restrict__ X, int64_t bsx, int64_t ldx, int64_t S, int C,
                                                  int G, int64_t chunk, float2* __restrict__ part) {
  extern __shared__ float lds[];
  constexpr int U = 8;  // loads in flight
  const int cv = C / V;
  const Place pl = place<ST_NT>(cv);
  float2* red = reinterpret_cast<float2*>(lds);
  const int64_t r0 = (int64_t)blockIdx.x * chunk;
  const int rows = (int)(r0 + chunk < S ? chunk : S - r0);
  const T* x = X + blockIdx.y * bsx + r0 * ldx;
  const int64_t step = pl.rp * ldx;
  if (pl.on && pl.row < rows)
    for (int c = pl.col; c < cv; c += pl.ct) {
      float p[V], s[V] = {}, q[V] = {};
      const T* at = x + pl.row * ldx + c * V;
      valuev<T, V>(loadv<T, V>(at), p);
      auto add = [&](const Vec<T, V>& w) {
        float v[V];
        valuev<T, V>(w, v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = v[e] - p[e];
          s[e] += d;
          q[e] = fmaf(d, d, q[e]);
        }
      };
      Vec<T, V> raw[U];
      int i = pl.row;
      auto whole = [&] { return i + (U - 1) * pl.rp < rows; };
      auto eight = [&] {
#pragma unroll
        for (int j = 0; j < U; ++j, at += step) raw[j] = loadv<T, V>(at);
#pragma unroll
        for (int j = 0; j < U; ++j) add(raw[j]);
        i += U * pl.rp;
      };
      if (whole()) {
        eight();
#pragma unroll
        for (int e = 0; e < V; ++e) {  // the same sums about the eight's mean
          const float to = p[e] + s[e] * (1.0f / U), d = to - p[e];
          q[e] = fmaf(-d, fmaf(-(float)U, d, 2.0f * s[e]), q[e]);
          s[e] = fmaf(-(float)U, d, s[e]);
          p[e] = to;
        }
        while (whole()) eight();
      }
      const T* end = at;  // at most U - 1 more positions
#pragma unroll
      for (int j = 0; j < U - 1; ++j) {
        raw[j] = loadv<T, V>(i + j * pl.rp < rows ? end : x + c * V);
        end += step;
      }
#pragma unroll
      for (int j = 0; j < U - 1; ++j)
        if (i + j * pl.rp < rows) add(raw[j]);
      const float n = (float)((rows - pl.row + pl.rp - 1) / pl.rp);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        // (a NaN passes: only a negative remainder of rounding is cut off)
        const float m2 = q[e] - s[e] * (s[e] / n);
        red[pl.row * C + c * V + e] = make_float2(p[e] + s[e] / n, m2 < 0.0f ? 0.0f : m2);
      }
    }
  __syncthreads();
  group_stats(red, pl.rp, rows, C, G, part + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * G);
}

// ---- joining the blocks' statistics

struct Stats {
  const float2* at;  // parts == 0: (mean, rstd) [B][G]; otherwise (mean, M2) [B][parts][G]
  int parts;
  int64_t S, chunk;
  int C, G;
  float eps;
};

// Positions that block i covered, times channels of a group
__device__ __forceinline__ float part_count(const Stats& st, int i) {
  const int64_t rows = i + 1 < st.parts ? st.chunk : st.S - (st.parts - 1) * st.chunk;
  return (float)rows * (float)(st.C / st.G);
}

// (mean, rstd) of all groups of image b into out[G] (LDS); AP_NT threads, scratch [AP_NT].  Threads
// side by side take groups side by side; rows of threads share a group's parts.  One round
// of loads where a thread has at most 16 parts (the usual case), two for the rest.
__device__ __forceinline__ void join_groups(const Stats& st, int64_t b, float2* out, double* scratch) {
  if (st.parts == 0) {
    for (int g = threadIdx.x; g < st.G; g += AP_NT) out[g] = st.at[b * st.G + g];
    __syncthreads();
    return;
  }
  constexpr int U = 16;
  const float2* p = st.at + b * st.parts * (int64_t)st.G;
  const int width = st.G < AP_NT ? st.G : AP_NT, rows = AP_NT / width;
  const int col = (int)threadIdx.x % width, r = (int)threadIdx.x / width;
  const float full = part_count(st, 0), last = part_count(st, st.parts - 1), n = (float)st.S * (float)(st.C / st.G);
  auto across = [&](double v) {  // over the rows of threads, in their order
    scratch[threadIdx.x] = v;
    __syncthreads();
    double s = 0.0;
    for (int i = 0; i < rows; ++i) s += scratch[i * width + col];
    __syncthreads();
    return s;
  };
  for (int g0 = 0; g0 < st.G; g0 += width) {
    const int g = g0 + col;
    const bool on = r < rows && g < st.G;
    const float2* q = p + (on ? g : 0);
    const int parts = on ? st.parts : 0;
    float2 v[U];
    auto load = [&](int i) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = q[(i + u * rows < parts ? i + u * rows : 0) * st.G];
    };
    auto count = [&](int i) { return i < parts ? (i + 1 < parts ? full : last) : 0.0f; };
    load(r);
    double s = 0.0;
    for (int i = r; i < parts; i += U * rows) {
      if (i != r) load(i);
#pragma unroll
      for (int u = 0; u < U; ++u) s += (double)count(i + u * rows) * (double)v[u].x;
    }
    const float mean = (float)(across(s) / (double)n);
    float m2 = 0.0f;
    for (int i = r; i < parts; i += U * rows) {
      if (parts > r + U * rows) load(i);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float d = v[u].x - mean;
        m2 += i + u * rows < parts ? v[u].y + count(i + u * rows) * d * d : 0.0f;
      }
    }
    const float var = (float)across(m2) / n;
    if (on && r == 0) out[g] = make_float2(mean, 1.0f / sqrtf(var + st.eps));
  }
  __syncthreads();
}

// Many blocks: group blockIdx.x of image blockIdx.y by a block of its own
constexpr int JN_NT = 256;
__global__ __launch_bounds__(JN_NT) void k7_join(Stats st, float2* __restrict__ out) {
  __shared__ float scratch[16];
  constexpr int U = 4;
  const float2* p = st.at + (int64_t)blockIdx.y * st.parts * st.G + blockIdx.x;
  const float full = part_count(st, 0), last = part_count(st, st.parts - 1), n = (float)st.S * (float)(st.C / st.G);
  auto count = [&](int i) { return i < st.parts ? (i + 1 < st.parts ? full : last) : 0.0f; };
  float2 v[U];
  auto load = [&](int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = p[(int64_t)(i + u * JN_NT < st.parts ? i + u * JN_NT : 0) * st.G];
  };
  load(threadIdx.x);
  const float m0 = p[0].x;
  float s = 0.0f;
  for (int i = threadIdx.x; i < st.parts; i += U * JN_NT) {
    if (i != (int)threadIdx.x) load(i);
#pragma unroll
    for (int u = 0; u < U; ++u) s += count(i + u * JN_NT) * (v[u].x - m0);
  }
  const float mean = m0 + block_sum(s, scratch) / n;
  float m2 = 0.0f;
  for (int i = threadIdx.x; i < st.parts; i += U * JN_NT) {
    if (st.parts > U * JN_NT) load(i);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float d = v[u].x - mean;
      m2 += i + u * JN_NT < st.parts ? v[u].y + count(i + u * JN_NT) * d * d : 0.0f;
    }
  }
  m2 = block_sum(m2, scratch);
  if (threadIdx.x == 0) out[(int64_t)blockIdx.y * st.G + blockIdx.x] = make_float2(mean, 1.0f / sqrtf(m2 / n + st.eps));
}

// ---- the output pass

// Positions [i * chunk, + chunk) of image blockIdx.y, i counted from the end: the statistics pass
// ended there, so that part of x is the likeliest to be in cache still.  Y may be X: a value is stored by the thread that
// loaded it, after it did, so neither is __restrict__; a load past the end takes a value that another thread may have
// written by then, and does not use it.
template <typename T, typename TY, int V, bool NT>
__global__ __launch_bounds__(AP_NT) void k7_apply(const T* X, int64_t bsx, int64_t ldx, int64_t chunk, Stats st,
                                                  const float* __restrict__ gamma, const float* __restrict__ beta,
                                                  int act, TY* Y, int64_t bsy, int64_t ldy) {
  extern __shared__ float lds[];
  __shared__ double scratch[AP_NT];
  float2* stat = reinterpret_cast<float2*>(lds);
  constexpr int U = 8;
  const int C = st.C, cv = C / V, cpg = C / st.G;
  const Place pl = place<AP_NT>(cv);
  const int64_t r0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * chunk;
  const int rows = (int)(r0 + chunk < st.S ? chunk : st.S - r0);
  const T* x = X + blockIdx.y * bsx + r0 * ldx;
  TY* y = Y + blockIdx.y * bsy + r0 * ldy;
  const int64_t step = pl.rp * ldx, ystep = pl.rp * ldy;
  Vec<T, V> raw[U];
  auto load = [&](int c, int i) {
    const T* at = x + i * ldx + c * V;
#pragma unroll
    for (int u = 0; u < U; ++u, at += step) raw[u] = loadv<T, V>(i + u * pl.rp < rows ? at : x + c * V);
  };
  float a[V], b[V];
  auto affine = [&](int c) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      a[e] = gamma ? gamma[c * V + e] : 1.0f;
      b[e] = beta ? beta[c * V + e] : 0.0f;
    }
  };
  if (pl.on) {  // under way while the statistics are joined
    load(pl.col, pl.row);
    affine(pl.col);
  }
  join_groups(st, blockIdx.y, stat, scratch);
  if (!pl.on) return;
  for (int c = pl.col; c < cv; c += pl.ct) {
    if (c != pl.col) load(c, pl.row), affine(c);
    float mean[V];
    int g = c * V / cpg, in = c * V - g * cpg;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      mean[e] = stat[g].x;
      a[e] *= stat[g].y;
      if (++in == cpg) in = 0, ++g;
    }
    for (int i = pl.row; i < rows; i += U * pl.rp) {
      if (i != pl.row) load(c, i);
      TY* to = y + i * ldy + c * V;
#pragma unroll
      for (int u = 0; u < U; ++u, to += ystep) {
        if (i + u * pl.rp >= rows) break;
        float v[V];
        valuev<T, V>(raw[u], v);
#pragma unroll
        for (int e = 0; e < V; ++e) v[e] = fmaf(v[e] - mean[e], a[e], b[e]);
        norm_act<sizeof(TY) == 4>(v, act);
        storev<TY, V, NT>(to, v);
      }
    }
  }
}

// The output pass into codes: a wave takes U whole positions (rows of C channels) at once, NC chunks
// of 512 channels each in registers.  Per channel (mean, rstd gamma, beta, inv_s) wait in LDS, eight
// planes of C / 8 so that neighbouring lanes read neighbouring 16 bytes, read once for U rows.
// The next rows' loads are under way while these are computed (4x4096x320 with its statistics 21.4 -> 18.7
// us back to back).  Bound by vector instructions, 31 to a lane's value; a row of 320, 640 or 1280
// channels fills 62% of the lanes that it takes, so that is 50 to a value (4x4096x320: 14 us of this pass).
template <typename T, bool VEC, int NC, int U>
__global__ __launch_bounds__(AP_NT) void k7_apply_quant(const T* __restrict__ X, int64_t bsx, int64_t ldx,
                                                        int64_t chunk, Stats st, const float* __restrict__ gamma,
                                                        const float* __restrict__ beta, int act,
                                                        const float* __restrict__ inv_s, int8_t* __restrict__ qX,
                                                        int64_t ldq, float* __restrict__ sX) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ double scratch[AP_NT];
  constexpr int NW = AP_NT / 64;
  const int C = st.C, cpg = C / st.G, c8 = (C + 7) / 8;
  float4* coef = reinterpret_cast<float4*>(lds);
  float2* stat = reinterpret_cast<float2*>(coef + 8 * c8);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t r0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * chunk;
  const int rows = (int)(r0 + chunk < st.S ? chunk : st.S - r0);
  typedef Row<T, VEC> RowX;
  auto row_at = [&](int i) { return RowX(X + blockIdx.y * bsx + (r0 + (i < rows ? i : 0)) * ldx, C); };
  typename RowX::Raw raw[U][NC], next[U][NC];
  auto load = [&](int i, typename RowX::Raw (&to)[U][NC]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const RowX x = row_at(i + u);
#pragma unroll
      for (int j = 0; j < NC; ++j) to[u][j] = x.load(8 * lane + 512 * j);
    }
  };
  load(wave * U, raw);
  // gamma, beta and inv_s while the statistics are joined; channels past C: value act(0) * 0
  for (int c = threadIdx.x; c < 8 * c8; c += AP_NT)
    coef[(c & 7) * c8 + (c >> 3)] = c < C ? make_float4(0.0f, gamma ? gamma[c] : 1.0f, beta ? beta[c] : 0.0f,
                                                        inv_s ? inv_s[c] : 1.0f)
                                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  join_groups(st, blockIdx.y, stat, scratch);
  for (int c = threadIdx.x; c < C; c += AP_NT) {
    const float2 s = stat[c / cpg];
    float4& f = coef[(c & 7) * c8 + (c >> 3)];
    f.x = s.x, f.y *= s.y;
  }
  __syncthreads();
  for (int i = wave * U; i < rows; i += NW * U) {
    load(i + NW * U, next);  // under way while these rows are computed
    float v[U][NC][8];
    uint32_t a[U] = {};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k8 = lane + 64 * j;
      const bool in = k8 < c8;
#pragma unroll
      for (int u = 0; u < U; ++u) row_at(i + u).value(raw[u][j], 8 * k8, v[u][j]);
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 k = coef[e * c8 + (in ? k8 : 0)];
        f[e] = in ? k.w : 0.0f;  // lanes past the row: 0 whatever the value
#pragma unroll
        for (int u = 0; u < U; ++u) v[u][j][e] = fmaf(in ? v[u][j][e] - k.x : 0.0f, k.y, k.z);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        norm_act<true>(v[u][j], act);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[u][j][e] *= f[e];
          a[u] = umax(a[u], abs_bits(v[u][j][e]));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < NC; ++j) raw[u][j] = next[u][j];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i + u >= rows) break;
      float s, r;
      row_scale(wave_umax(a[u]), s, r);
      const int64_t row = blockIdx.y * st.S + r0 + i + u;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int64_t k = 8 * (lane + 64 * j);
        if (k < ldq)
          *reinterpret_cast<uint2*>(qX + row * ldq + k) =
              make_uint2(codes4(v[u][j][0], v[u][j][1], v[u][j][2], v[u][j][3], r),
                         codes4(v[u][j][4], v[u][j][5], v[u][j][6], v[u][j][7], r));
      }
      if (lane == 0) sX[row] = s;
    }
  }
}

// The same for narrow rows (C <= 8 LPR, a multiple of 8): LPR lanes per row, 64 / LPR rows per
// wave at once; a lane keeps its 8 channels' coefficients in registers.  us, all launches, against
// a wave per row: 65536x256 35.2 (40.6), x128 27.0 (38.7), x64 19.3 (36.8; 16 lanes a row 21.9), x32 16.7
// (36.1; 16 lanes 19.9); a few thousand rows cost the same either way (2x4096x128 15.8, 14.3).
template <typename T, int LPR>
__global__ __launch_bounds__(AP_NT) void k7_apply_quant_narrow(const T* __restrict__ X, int64_t bsx, int64_t ldx,
                                                               int64_t chunk, Stats st, const float* __restrict__ gamma,
                                                               const float* __restrict__ beta, int act,
                                                               const float* __restrict__ inv_s,
                                                               int8_t* __restrict__ qX, int64_t ldq,
                                                               float* __restrict__ sX) {
  extern __shared__ __attribute__((aligned(16))) float lds[];
  __shared__ double scratch[AP_NT];
  float2* stat = reinterpret_cast<float2*>(lds);
  constexpr int U = 4, STEP = AP_NT / LPR;
  const int C = st.C, cpg = C / st.G;
  const int li = threadIdx.x % LPR, first = threadIdx.x / LPR, c = 8 * li;
  const bool on = c < C;
  const int64_t r0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * chunk;
  const int rows = (int)(r0 + chunk < st.S ? chunk : st.S - r0);
  const T* x = X + blockIdx.y * bsx + r0 * ldx + (on ? c : 0);
  Vec<T, 8> raw[U];
  auto load = [&](int i) {
#pragma unroll
    for (int u = 0; u < U; ++u) raw[u] = loadv<T, 8>(x + (i + u * STEP < rows ? i + u * STEP : 0) * ldx);
  };
  load(first);
  float a[8], b[8], f[8], mean[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = on ? (gamma ? gamma[c + e] : 1.0f) : 0.0f;
    b[e] = on && beta ? beta[c + e] : 0.0f;
    f[e] = on ? (inv_s ? inv_s[c + e] : 1.0f) : 0.0f;
  }
  join_groups(st, blockIdx.y, stat, scratch);
  int g = (on ? c : 0) / cpg, in = (on ? c : 0) - g * cpg;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    mean[e] = stat[g].x;
    a[e] *= stat[g].y;
    if (++in == cpg) in = 0, g = g + 1 < st.G ? g + 1 : g;
  }
  for (int i = first; i < rows + first; i += U * STEP) {  // whole rows of lanes stay together
    if (i != first) load(i);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = i + u * STEP;
      if (r - first >= rows) break;  // the same for the whole block
      float v[8];
      valuev<T, 8>(raw[u], v);
      uint32_t top = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf(on ? v[e] - mean[e] : 0.0f, a[e], b[e]);  // off: a = b = f = 0
      norm_act<true>(v, act);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] *= f[e];
        top = umax(top, abs_bits(v[e]));
      }
      float s, q;
      row_scale(wave_umax<LPR>(top), s, q);
      if (r >= rows) continue;
      const int64_t row = blockIdx.y * st.S + r0 + r;
      int8_t* to = qX + row * ldq + c;
      *reinterpret_cast<uint2*>(to) = make_uint2(codes4(v[0], v[1], v[2], v[3], q), codes4(v[4], v[5], v[6], v[7], q));
#pragma unroll
      for (int z = 8 * LPR; z < 128; z += 8 * LPR) *reinterpret_cast<uint2*>(to + z) = make_uint2(0, 0);  // to the end of the row
      if (li == 0) sX[row] = s;
    }
  }
}

// ---- launches

// Vector width of k7_one: the widest of 8, 4, 2 that divides a group
int one_width(int cpg) {
  for (int v = 8; v > 1; v /= 2)
    if (cpg % v == 0) return v;
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
  if constexpr (V > 1) {  // one value per load: never more than 8 loads
    if (a.S * (a.C / a.G) > 8 * 1024) return launch_one_nv<T, TY, V, 32 / V>(a, Y, bsy, ldy, stat, st);
  }
  launch_one_nv<T, TY, V, 8 / V>(a, Y, bsy, ldy, stat, st);
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
  const int rp = ST_NT / place_ct(a.C / V, ST_NT);
  const size_t bytes = (size_t)rp * a.C * 8;
  hipLaunchKernelGGL((k7_stats<T, V>), dim3(p.parts, (uint32_t)a.B), dim3(ST_NT), bytes, st,
                     static_cast<const T*>(a.X), a.bsx, a.ldx, a.S, a.C, a.G, p.chunk, part);
}

template <typename T, typename TY, int V>
void launch_apply(const NormArgs& a, const NormPlan& p, const Stats& s, void* Y, int64_t bsy, int64_t ldy,
                  hipStream_t st) {
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(p.blocks, (uint32_t)a.B), dim3(AP_NT), (size_t)a.G * 8, st,
                       static_cast<const T*>(a.X), a.bsx, a.ldx, p.rows, s, a.gamma, a.beta, a.act,
                       static_cast<TY*>(Y), bsy, ldy);
  };
  if constexpr (V == 8) {  // x and y past the 256 MB cache: y would only push x out
    if ((double)a.B * (double)a.S * a.C * (sizeof(T) + sizeof(TY)) > 268435456.0) return go(k7_apply<T, TY, V, true>);
  }
  go(k7_apply<T, TY, V, false>);
}

// Statistics for an output pass: by k7_one where a group fits a block, else by blocks of positions
Stats run_stats(const NormArgs& a, const NormPlan& p, void* ws, hipStream_t st) {
  float2* part = static_cast<float2*>(ws);
  Stats s{part, 0, a.S, p.chunk, a.C, a.G, a.eps};
  if (p.one) {
    const int w = one_width(a.C / a.G);
    a.xdtype == 0 ? launch_one<float, float>(a, w, nullptr, 0, 0, part, st)
                  : launch_one<uint16_t, uint16_t>(a, w, nullptr, 0, 0, part, st);
    return s;
  }
  const bool v8 = a.C % 8 == 0;
  if (a.xdtype == 0) v8 ? launch_stats<float, 8>(a, p, part, st) : launch_stats<float, 1>(a, p, part, st);
  else v8 ? launch_stats<uint16_t, 8>(a, p, part, st) : launch_stats<uint16_t, 1>(a, p, part, st);
  s.parts = (int)p.parts;
  if (p.join) {
    float2* out = part + (size_t)a.B * p.parts * a.G;
    hipLaunchKernelGGL(k7_join, dim3((uint32_t)a.G, (uint32_t)a.B), dim3(JN_NT), 0, st, s, out);
    s.at = out;
    s.parts = 0;
  }
  return s;
}

}  // namespace

NormPlan plan_norm(int64_t B, int64_t S, int C, int G) {
  NormPlan p{};
  const int64_t cpg = C / G;
  // What counts are the loads, at most 8 per thread of 1024, and the rows that they touch.  Measured (us, bf16, SiLU, back to
  // back; one launch / two): 2x64x1280 in groups of 40 3.4 / 9.7, 2x256x1280 5.3 / 10.0, 2x1024x640 of 20 8.0 / 11.3,
  // 2x2048x512 of 16 9.0 / 12.3, 2x1024x320 of 10 7.8 / 10.8, 2x2000x320 11.8 / 11.7, 2x2700x96 of 3 9.2 / 10.7, 2x700x77
  // of 11 5.8 / 9.9, 2x8000x32 of 1 12.1 / 10.7, 2x8000x128 of 4 22.1 / 12.4.  Statistics alone, in front of the codes (either way
  // two launches): 2x64x1280 9.1 / 12.5, 2x1024x640 9.2 / 11.8, 2x2048x512 10.0 / 12.4, 2x4096x256 of 8 11.9 / 12.3, 2x2700x96
  // 8.6 / 11.0, 2x8000x128 13.8 / 12.4.  Not in the rule, and against it: many images (8x1024x640 14.0 / 15.7, 16x1024x640
  // 26.4 / 22.0, codes 26.5 / 22.1) and short pieces of long rows, whose lines are read by several blocks (2x4096x256 in
  // groups of 8, 16 bytes to a row, 15.6 / 12.4; one image 10.3).
  p.one = S * cpg <= 32 * 1024 && S * (cpg / one_width((int)cpg)) <= 8 * 1024 && S <= 4096;
  // Measured (us, both launches or all three; statistics blocks / output blocks):
  //   2x4096x320 bf16 256 / 256 13.4, 256 / 512 15.0, 256 joined apart / 256 14.9, 256 / 1024 17.2
  //   1x16384x128 bf16 128 / 256 13.2, 256 / 256 15.3, 256 joined apart / 256 14.7
  //   1x65536x256 bf16 512 joined apart / 768 28.6, 512 / 2048 35.7, 256 / 512 joined inside 30.9
  //   1x262144x128 bf16 512 joined apart / 768 42.8, 256 / 512 joined inside 44.4
  // so up to 2^23 values one block of each kind per CU, the output blocks joining at most 128 parts
  // per image; above, a join of its own.
  const int64_t n = B * S * C;
  p.join = n > (int64_t(1) << 23);
  int64_t parts = p.join ? (512 + B - 1) / B : (256 + B - 1) / B;
  if (!p.join && parts > 128) parts = 128;
  const int cv = C % 8 == 0 ? C / 8 : C, rp = 256 / place_ct(cv, 256);
  p.chunk = (S + parts - 1) / parts;
  if (p.chunk < 2 * rp) p.chunk = 2 * rp;
  if (p.chunk > 512 * rp) p.chunk = 512 * rp;  // positions that a thread sums
  p.parts = (uint32_t)((S + p.chunk - 1) / p.chunk);
  p.bytes = ((size_t)B * p.parts * G + (size_t)B * G) * sizeof(float2);
  const int64_t blocks = !p.join ? 256 : n <= (int64_t(1) << 25) ? 768 : 2048;
  p.rows = (S * B + blocks - 1) / blocks;
  if (p.rows < 2 * rp) p.rows = 2 * rp;
  p.blocks = (uint32_t)((S + p.rows - 1) / p.rows);
  return p;
}

hipError_t launch_norm(const NormArgs& a, void* Y, int ydtype, int64_t bsy, int64_t ldy, void* ws, hipStream_t st) {
  const NormPlan p = plan_norm(a.B, a.S, a.C, a.G);
  if (p.one) {
    const int w = one_width(a.C / a.G);
    if (a.xdtype == 0 && ydtype == 0) launch_one<float, float>(a, w, Y, bsy, ldy, nullptr, st);
    else if (a.xdtype == 0) launch_one<float, uint16_t>(a, w, Y, bsy, ldy, nullptr, st);
    else if (ydtype == 0) launch_one<uint16_t, float>(a, w, Y, bsy, ldy, nullptr, st);
    else launch_one<uint16_t, uint16_t>(a, w, Y, bsy, ldy, nullptr, st);
    return hipGetLastError();
  }
  const Stats s = run_stats(a, p, ws, st);
  const bool v8 = a.C % 8 == 0;
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
  const bool vec = rows_aligned4(a.X, a.ldx, a.xdtype) && (a.xdtype == 0 || a.bsx % 2 == 0);
  const size_t bytes = (size_t)((a.C + 7) / 8) * 8 * 16 + (size_t)a.G * 8;
  const int64_t ldq = i8_ld(a.C);
  // about 768 blocks; whole turns of the four waves where a wave takes several rows at once
  const int turn = ldq <= 512 ? 16 : 8;
  const int64_t rows = ((a.S * a.B + 767) / 768 + turn - 1) / turn * turn;
  const dim3 g((uint32_t)((a.S + rows - 1) / rows), (uint32_t)a.B), b(AP_NT);
  auto go = [&](auto kernel, auto x, size_t lds) {
    hipLaunchKernelGGL(kernel, g, b, lds, st, x, a.bsx, a.ldx, rows, s, a.gamma, a.beta, a.act, inv_s, qX, ldq, sX);
  };
  const float* x32 = static_cast<const float*>(a.X);
  const uint16_t* x16 = static_cast<const uint16_t*>(a.X);
  auto by_type = [&](auto nc) {
    constexpr int NC = decltype(nc)::value, U = NC == 1 ? 4 : NC == 2 ? 2 : 1;
    if (a.xdtype == 0) go(k7_apply_quant<float, true, NC, U>, x32, bytes);
    else vec ? go(k7_apply_quant<uint16_t, true, NC, U>, x16, bytes) : go(k7_apply_quant<uint16_t, false, NC, U>, x16, bytes);
  };
  const bool even = a.C % 8 == 0;
  auto narrow = [&](auto lpr) {
    constexpr int LPR = decltype(lpr)::value;
    a.xdtype == 0 ? go(k7_apply_quant_narrow<float, LPR>, x32, (size_t)a.G * 8)
                  : go(k7_apply_quant_narrow<uint16_t, LPR>, x16, (size_t)a.G * 8);
  };
  if (even && a.C <= 256) {
    if (a.C <= 32) narrow(std::integral_constant<int, 4>{});
    else if (a.C <= 64) narrow(std::integral_constant<int, 8>{});
    else if (a.C <= 128) narrow(std::integral_constant<int, 16>{});
    else narrow(std::integral_constant<int, 32>{});
  } else if (ldq <= 512) by_type(std::integral_constant<int, 1>{});
  else if (ldq <= 1024) by_type(std::integral_constant<int, 2>{});
  else if (ldq <= 2048) by_type(std::integral_constant<int, 4>{});
  else by_type(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

}  // namespace svdq
