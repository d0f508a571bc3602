// Kernel 7: group norm with an activation, channels last, and the same norm leaving as
// 8-bit codes with one scale per position (the input of the W8A8 product).
//
// Mathematics: X [B][S][C], C = G cpg.  For image b and group g, over the S positions and the
// group's cpg channels: mean, var (biased); y = act((x - mean) / sqrt(var + eps) gamma_c +
// beta_c).  Statistics in fp32 without cancellation: a block first takes the mean of the
// rows it holds in registers as its pivot p and sums d = x - p and d^2 over its rows; the
// blocks' (count, mean, M2) are then joined by mean = sum n_i mean_i / n and
// M2 = sum M2_i + n_i (mean_i - mean)^2 (Chan, Golub and LeVeque's pairwise formula).
//
// Design (gfx950): bound by HBM (x read for the statistics and again for the output, mostly
// from cache, y written once).  Three launches: statistics per block of positions,
// their join per (image, group), the output pass.  A thread keeps the same V consecutive
// channels over all its positions, so the group's boundaries may fall anywhere: sums are
// kept per channel and meet per group in LDS.
#include "../../include/svdq.h"
#include "int8.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

constexpr int GN_NT = 256;
constexpr int GN_ROWS = 8;  // positions a thread holds at once

__device__ __forceinline__ void load8_vec(const uint16_t* p, float v[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16_lo_to_f32(w.x), v[1] = bf16_hi_to_f32(w.x), v[2] = bf16_lo_to_f32(w.y), v[3] = bf16_hi_to_f32(w.y);
  v[4] = bf16_lo_to_f32(w.z), v[5] = bf16_hi_to_f32(w.z), v[6] = bf16_lo_to_f32(w.w), v[7] = bf16_hi_to_f32(w.w);
}
__device__ __forceinline__ void load8_vec(const float* p, float v[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// V consecutive channels (V = 8: 16-byte aligned; V = 1: any alignment)
template <typename T, int V>
__device__ __forceinline__ void loadv(const T* p, float v[V]) {
  if constexpr (V == 8) load8_vec(p, v);
  else v[0] = load1(p);
}

template <int V>
__device__ __forceinline__ void storev(float* p, const float v[V]) {
  if constexpr (V == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    p[0] = v[0];
  }
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}
template <int V>
__device__ __forceinline__ void storev(uint16_t* p, const float v[V]) {
  if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                              pack_bf16(v[6], v[7]));
  } else {
    *p = __builtin_bit_cast(uint16_t, (__bf16)v[0]);
  }
}

// SiLU y / (1 + exp(-y)); GELU in its exact form.  A large negative y gives exp(-y) = inf
// and the quotient -0.
__device__ __forceinline__ float norm_act(float y, int act) {
  if (act == SVDQ_GN_SILU) return y / (1.0f + __expf(-y));
  if (act == SVDQ_GN_GELU) return gelu_erf(y);
  return y;
}

// The threads' places: CT columns of V channels side by side, RP positions below each other.
struct Place {
  int ct, rp, col, row;
  bool on;
};
__device__ __forceinline__ Place place(int cv) {
  Place p;
  p.ct = cv < GN_NT ? cv : GN_NT;
  p.rp = GN_NT / p.ct;
  p.col = threadIdx.x % p.ct;
  p.row = threadIdx.x / p.ct;
  p.on = p.row < p.rp;
  return p;
}

// Sum per group of the block's per-channel values red[r][c] (r < rp, C channels): out[g].
// 2^k threads per group (as many as there are), joined by shuffles inside a wave.
__device__ __forceinline__ void group_sums(const float* red, int rp, int C, int G, float* out) {
  const int cpg = C / G;
  int tpg = 1;
  while (tpg < 64 && tpg * 2 * G <= GN_NT) tpg *= 2;
  const int per = GN_NT / tpg;
  for (int g0 = 0; g0 < G; g0 += per) {
    const int g = g0 + threadIdx.x / tpg, t = threadIdx.x % tpg;
    float s = 0.0f;
    if (g < G)
      for (int i = t; i < rp * cpg; i += tpg) s += red[(i / cpg) * C + g * cpg + i % cpg];
    for (int m = tpg / 2; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
    if (g < G && t == 0) out[g] = s;
  }
}

// Statistics of positions [blockIdx.x * chunk, + chunk) of image blockIdx.y: part[b][i][g] =
// (mean, M2).  LDS: red [max(rp C, C)] floats, gsum [G], gpiv [G].
template <typename T, int V>
__global__ __launch_bounds__(GN_NT) void k7_stats(const T* __restrict__ X, int64_t bsx, int64_t ldx, int64_t S, int C,
                                                  int G, int64_t chunk, float2* __restrict__ part) {
  extern __shared__ float lds[];
  const int cv = C / V, cpg = C / G;
  const Place pl = place(cv);
  float* red = lds;
  float* gsum = lds + pl.rp * C;
  float* gpiv = gsum + G;
  const int64_t r0 = (int64_t)blockIdx.x * chunk, r1 = r0 + chunk < S ? r0 + chunk : S;
  const T* x = X + blockIdx.y * bsx;
  const int first = (int)(r1 - r0 < (int64_t)GN_ROWS * pl.rp ? r1 - r0 : (int64_t)GN_ROWS * pl.rp);

  // the mean of the first rows is the pivot of all of them
  for (int c = pl.col; c < cv && pl.on; c += pl.ct) {
    float s[V] = {};
    for (int i = pl.row; i < first; i += pl.rp) {
      float v[V];
      loadv<T, V>(x + (r0 + i) * ldx + (int64_t)c * V, v);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += v[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[pl.row * C + c * V + e] = s[e];
  }
  __syncthreads();
  group_sums(red, pl.rp, C, G, gsum);
  __syncthreads();
  for (int g = threadIdx.x; g < G; g += GN_NT) gpiv[g] = gsum[g] / (float)(first * cpg);
  __syncthreads();

  for (int pass = 0; pass < 2; ++pass) {  // sums of d, then of d^2
    for (int c = pl.col; c < cv && pl.on; c += pl.ct) {
      float p[V], s[V] = {};
#pragma unroll
      for (int e = 0; e < V; ++e) p[e] = gpiv[(c * V + e) / cpg];
      for (int64_t i = r0 + pl.row; i < r1; i += pl.rp) {
        float v[V];
        loadv<T, V>(x + i * ldx + (int64_t)c * V, v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float d = v[e] - p[e];
          s[e] += pass ? d * d : d;
        }
      }
#pragma unroll
      for (int e = 0; e < V; ++e) red[pl.row * C + c * V + e] = s[e];
    }
    __syncthreads();
    group_sums(red, pl.rp, C, G, gsum);
    __syncthreads();
    if (pass == 0) {  // the pivot becomes the block's mean
      for (int g = threadIdx.x; g < G; g += GN_NT) gpiv[g] += gsum[g] / ((float)(r1 - r0) * (float)cpg);
      __syncthreads();
    }
  }
  for (int g = threadIdx.x; g < G; g += GN_NT)
    part[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * G + g] = make_float2(gpiv[g], gsum[g]);
}

__device__ __forceinline__ float block_sum(float v, float* scratch) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
  __syncthreads();
  return (scratch[0] + scratch[1]) + (scratch[2] + scratch[3]);
}

// Joins the n blocks' statistics of group blockIdx.x of image blockIdx.y: stat[b][g] = (mean, rstd)
__global__ __launch_bounds__(GN_NT) void k7_join(const float2* __restrict__ part, int n, int64_t S, int64_t chunk,
                                                 int C, int G, float eps, float2* __restrict__ stat) {
  __shared__ float scratch[4];
  const int g = blockIdx.x, cpg = C / G;
  const float2* p = part + (int64_t)blockIdx.y * n * G + g;
  const float m0 = p[0].x, total = (float)S * (float)cpg;
  auto count = [&](int i) { return (float)((i + 1) * chunk < S ? chunk : S - i * chunk) * (float)cpg; };
  float s = 0.0f;
  for (int i = threadIdx.x; i < n; i += GN_NT) s += count(i) * (p[(int64_t)i * G].x - m0);
  const float mean = m0 + block_sum(s, scratch) / total;
  float q = 0.0f;
  for (int i = threadIdx.x; i < n; i += GN_NT) {
    const float2 v = p[(int64_t)i * G];
    const float d = v.x - mean;
    q += v.y + count(i) * d * d;
  }
  const float var = block_sum(q, scratch) / total;
  if (threadIdx.x == 0) stat[(int64_t)blockIdx.y * G + g] = make_float2(mean, 1.0f / sqrtf(var + eps));
}

// The output pass: positions [blockIdx.x * chunk, + chunk) of image blockIdx.y
template <typename T, typename TY, int V>
__global__ __launch_bounds__(GN_NT) void k7_apply(const T* __restrict__ X, int64_t bsx, int64_t ldx, int64_t S, int C,
                                                  int G, int64_t chunk, const float2* __restrict__ stat,
                                                  const float* __restrict__ gamma, const float* __restrict__ beta,
                                                  int act, TY* __restrict__ Y, int64_t bsy, int64_t ldy) {
  const int cv = C / V, cpg = C / G;
  const Place pl = place(cv);
  if (!pl.on) return;
  const int64_t r0 = (int64_t)blockIdx.x * chunk, r1 = r0 + chunk < S ? r0 + chunk : S;
  const T* x = X + blockIdx.y * bsx;
  TY* y = Y + blockIdx.y * bsy;
  for (int c = pl.col; c < cv; c += pl.ct) {
    float mean[V], a[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float2 st = stat[(int64_t)blockIdx.y * G + (c * V + e) / cpg];
      mean[e] = st.x;
      a[e] = st.y * (gamma ? gamma[c * V + e] : 1.0f);
      b[e] = beta ? beta[c * V + e] : 0.0f;
    }
    for (int64_t i = r0 + pl.row; i < r1; i += pl.rp) {
      float v[V];
      loadv<T, V>(x + i * ldx + (int64_t)c * V, v);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = norm_act((v[e] - mean[e]) * a[e] + b[e], act);
      storev<V>(y + i * ldy + (int64_t)c * V, v);
    }
  }
}

// The output pass into codes: a wave takes whole positions (rows of C channels) of image
// blockIdx.y.  Per channel (mean, a, beta, inv_s) wait in LDS, eight planes of C / 8 so that
// neighbouring lanes read neighbouring 16 bytes.  The row is walked twice (the second time
// from cache).
template <typename T, bool VEC>
__global__ __launch_bounds__(GN_NT) void k7_apply_quant(const T* __restrict__ X, int64_t bsx, int64_t ldx, int64_t S,
                                                        int C, int G, int64_t chunk, const float2* __restrict__ stat,
                                                        const float* __restrict__ gamma,
                                                        const float* __restrict__ beta, int act,
                                                        const float* __restrict__ inv_s, int8_t* __restrict__ qX,
                                                        int64_t ldq, float* __restrict__ sX) {
  extern __shared__ float lds[];
  float4* coef = reinterpret_cast<float4*>(lds);
  const int cpg = C / G, c8 = (C + 7) / 8;
  for (int c = threadIdx.x; c < 8 * c8; c += GN_NT) {
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // channels past C: value 0
    if (c < C) {
      const float2 st = stat[(int64_t)blockIdx.y * G + c / cpg];
      f = make_float4(st.x, st.y * (gamma ? gamma[c] : 1.0f), beta ? beta[c] : 0.0f, inv_s ? inv_s[c] : 1.0f);
    }
    coef[(c & 7) * c8 + (c >> 3)] = f;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * chunk, r1 = r0 + chunk < S ? r0 + chunk : S;
  for (int64_t i = r0 + wave; i < r1; i += 4) {
    const Row<T, VEC> x(X + blockIdx.y * bsx + i * ldx, C);
    const int64_t row = blockIdx.y * S + i;
    auto value8 = [&](int k8, float v[8]) {
      x.value(x.load(8 * k8), 8 * k8, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 f = coef[e * c8 + k8];
        v[e] = norm_act((v[e] - f.x) * f.y + f.z, act) * f.w;
      }
    };
    uint32_t a = 0;
    for (int k8 = lane; k8 < c8; k8 += 64) {
      float v[8];
      value8(k8, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) a = umax(a, abs_bits(v[e]));
    }
    float s, r;
    row_scale(wave_umax(a), s, r);
    for (int k8 = lane; k8 < ldq / 8; k8 += 64) {
      float v[8] = {};
      if (k8 < c8) value8(k8, v);
      *reinterpret_cast<uint2*>(qX + row * ldq + 8 * (int64_t)k8) =
          make_uint2(codes4(v[0], v[1], v[2], v[3], r), codes4(v[4], v[5], v[6], v[7], r));
    }
    if (lane == 0) sX[row] = s;
  }
}

bool vec_ok(const void* p, int64_t bs, int64_t ld, int dtype) {
  const int64_t per = dtype == 0 ? 4 : 8;  // values in 16 bytes
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % per == 0 && bs % per == 0;
}

template <typename T, int V>
void launch_stats(const NormArgs& a, const NormPlan& p, float2* part, hipStream_t st) {
  const int cv = a.C / V, ct = cv < GN_NT ? cv : GN_NT, rp = GN_NT / ct;
  const size_t bytes = ((size_t)rp * a.C + 2 * (size_t)a.G) * 4;
  hipLaunchKernelGGL((k7_stats<T, V>), dim3(p.parts, (uint32_t)a.B), dim3(GN_NT), bytes, st,
                     static_cast<const T*>(a.X), a.bsx, a.ldx, a.S, a.C, a.G, p.chunk, part);
}

template <typename T, typename TY, int V>
void launch_apply(const NormArgs& a, const NormPlan& p, const float2* stat, void* Y, int64_t bsy, int64_t ldy,
                  hipStream_t st) {
  hipLaunchKernelGGL((k7_apply<T, TY, V>), dim3(p.parts, (uint32_t)a.B), dim3(GN_NT), 0, st,
                     static_cast<const T*>(a.X), a.bsx, a.ldx, a.S, a.C, a.G, p.chunk, stat, a.gamma, a.beta, a.act,
                     static_cast<TY*>(Y), bsy, ldy);
}

hipError_t run_stats(const NormArgs& a, const NormPlan& p, void* ws, float2** stat, hipStream_t st) {
  float2* part = static_cast<float2*>(ws);
  *stat = part + (size_t)a.B * p.parts * a.G;
  const bool v8 = a.C % 8 == 0 && vec_ok(a.X, a.bsx, a.ldx, a.xdtype);
  if (a.xdtype == 0) v8 ? launch_stats<float, 8>(a, p, part, st) : launch_stats<float, 1>(a, p, part, st);
  else v8 ? launch_stats<uint16_t, 8>(a, p, part, st) : launch_stats<uint16_t, 1>(a, p, part, st);
  hipLaunchKernelGGL(k7_join, dim3((uint32_t)a.G, (uint32_t)a.B), dim3(GN_NT), 0, st, part, p.parts, a.S, p.chunk, a.C,
                     a.G, a.eps, *stat);
  return hipGetLastError();
}

}  // namespace

NormPlan plan_norm(int64_t B, int64_t S, int C, int G) {
  NormPlan p;
  int64_t chunk = (S * B + 1023) / 1024;  // about 1024 blocks
  const int64_t least = 16384 / C > 8 ? 16384 / C : 8;
  if (chunk < least) chunk = least;
  p.chunk = chunk;
  p.parts = (uint32_t)((S + chunk - 1) / chunk);
  p.bytes = ((size_t)B * p.parts * G + (size_t)B * G) * sizeof(float2);
  return p;
}

hipError_t launch_norm(const NormArgs& a, void* Y, int ydtype, int64_t bsy, int64_t ldy, void* ws, hipStream_t st) {
  const NormPlan p = plan_norm(a.B, a.S, a.C, a.G);
  float2* stat;
  hipError_t e = run_stats(a, p, ws, &stat, st);
  if (e != hipSuccess) return e;
  const bool v8 = a.C % 8 == 0 && vec_ok(a.X, a.bsx, a.ldx, a.xdtype) && vec_ok(Y, bsy, ldy, ydtype);
  if (a.xdtype == 0 && ydtype == 0)
    v8 ? launch_apply<float, float, 8>(a, p, stat, Y, bsy, ldy, st) : launch_apply<float, float, 1>(a, p, stat, Y, bsy, ldy, st);
  else if (a.xdtype == 0)
    v8 ? launch_apply<float, uint16_t, 8>(a, p, stat, Y, bsy, ldy, st) : launch_apply<float, uint16_t, 1>(a, p, stat, Y, bsy, ldy, st);
  else if (ydtype == 0)
    v8 ? launch_apply<uint16_t, float, 8>(a, p, stat, Y, bsy, ldy, st) : launch_apply<uint16_t, float, 1>(a, p, stat, Y, bsy, ldy, st);
  else
    v8 ? launch_apply<uint16_t, uint16_t, 8>(a, p, stat, Y, bsy, ldy, st) : launch_apply<uint16_t, uint16_t, 1>(a, p, stat, Y, bsy, ldy, st);
  return hipGetLastError();
}

hipError_t launch_norm_quant(const NormArgs& a, const float* inv_s, int8_t* qX, float* sX, void* ws, hipStream_t st) {
  const NormPlan p = plan_norm(a.B, a.S, a.C, a.G);
  float2* stat;
  hipError_t e = run_stats(a, p, ws, &stat, st);
  if (e != hipSuccess) return e;
  const bool vec = vec_ok(a.X, a.bsx, a.ldx, a.xdtype);
  const size_t bytes = (size_t)((a.C + 7) / 8) * 8 * 16;
  const dim3 g(p.parts, (uint32_t)a.B), b(GN_NT);
  const int64_t ldq = i8_ld(a.C);
  auto go = [&](auto kernel, auto x) {
    hipLaunchKernelGGL(kernel, g, b, bytes, st, x, a.bsx, a.ldx, a.S, a.C, a.G, p.chunk, stat, a.gamma, a.beta, a.act,
                       inv_s, qX, ldq, sX);
  };
  if (a.xdtype == 0) {
    const float* x = static_cast<const float*>(a.X);
    vec ? go(k7_apply_quant<float, true>, x) : go(k7_apply_quant<float, false>, x);
  } else {
    const uint16_t* x = static_cast<const uint16_t*>(a.X);
    vec ? go(k7_apply_quant<uint16_t, true>, x) : go(k7_apply_quant<uint16_t, false>, x);
  }
  return hipGetLastError();
}

}  // namespace svdq
