// Kernel 10: layer norm, its gradient, and the same norm leaving as E4M3 codes with a scale for each block of 128.
//
// Mathematics (per row of C values): mean, biased variance; z = (x - mean) rstd, rstd = 1 / sqrt(var + eps);
// y = z (o + gamma) + beta, o 0 or 1, gamma and beta of all rows or of the row's image.  Backwards, from the forward's
// mean and rstd: g = dy (o + gamma); dx = rstd (g - sum(g) / C - z sum(g z) / C); dgamma = sum over rows dy z,
// dbeta = sum over rows dy.
//
// Design (gfx950): bound by HBM, x (and dy) read once: a row stays in registers, 8 values a lane and chunk, NC chunks.  A
// row takes L = 8 (gradient), 16, 32 or 64 lanes, or a team of several waves: few waves of up to 4 chunks where there are
// rows enough to fill the card, more waves of fewer chunks where there are not.
// Statistics: a first mean p of the lanes' own group, then d = x - p, sum d and sum d^2: mean = p + c, c = sum d / n,
// M2 = sum d^2 - (sum d) c, so that neither a mean far from zero nor the rounding of p costs digits (a constant row gives
// beta).  Waves join by the pairwise formula (Chan, Golub and LeVeque) about the first one's mean, at one barrier, from p and
// c apart: the first means' differences are exact, and a mean rounded to fp32 before it is subtracted cost rstd 2.4e-5 at a
// mean of 1e4 standard deviations.  What a mean near zero keeps is the rounding of x - p, which is alike for all values of a
// binade: 1e-8 of a standard deviation, which y and rstd do not show, but 3e-7 to 4e-7 of means that are sigma / sqrt(C), where
// an fp32 sum of the values is off by 1e-7 (adding d by pairs changes nothing, 3.9e-7 to 3.8e-7, and costs 6 us of 26 at
// 2 x 4608 x 3072).
// The columns' sums of the gradient stay in registers over a block's rows, the next row on its way while one is
// computed; a block joins its teams in LDS and leaves one partial sum; a second launch adds the blocks'; for few rows
// blocks of their own sum the columns in the same launch.  Every order is fixed: no atomics.
// Measured: 65536 x 4096 fp32 427 us (5.0 TB/s, as a large copy); 2 x 4608 x 3072 bf16, modulated, 25 (4.6 TB/s; the vector
// units are busy 62%, 383 instructions a wave of 24 values a lane); 4608 x 3072 to codes 12.9 (553, busy 81%; 16 behind a
// product that has lowered the clock; kernel 8 on a written y 8.6); gradient 2 x 4608 x 3072 bf16 39 (35 and the second
// launch's 4; 4.3 TB/s), 3 x 333 x 1111 fp32 9.2 in one launch.
#include <algorithm>
#include <type_traits>

#include "fp8.hpp"
#include "gemm8.hpp"
#include "kernels.hpp"
#include "vec.hpp"

namespace svdq {
namespace {

// The sum over groups of L lanes, the same bits in every lane: every step adds the two halves of what is joined, to
// which both sides come symmetrically (mirrors, not rotations).
template <int L>
__device__ __forceinline__ float lane_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});   // quad [1 0 3 2]
  v += dpp(v, std::integral_constant<int, 0x4E>{});   // quad [2 3 0 1]
  v += dpp(v, std::integral_constant<int, 0x141>{});  // halves of a row of 16 mirrored
  if constexpr (L >= 16) v += dpp(v, std::integral_constant<int, 0x140>{});  // rows mirrored
  if constexpr (L >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (L >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

// f(e, in) for the 8 values from k, in: whether e lies within the row; whole: all of the chunk's do (the same for all lanes)
template <typename F>
__device__ __forceinline__ void within(bool whole, int k, int C, F&& f) {
  if (whole) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f(e, true);
  } else {
    asm("" : "+v"(k));  // compared here, not kept from one use to the next (8 masks each)
#pragma unroll
    for (int e = 0; e < 8; ++e) f(e, k + e < C);
  }
}

template <typename TY>
__device__ __forceinline__ void store_row8(TY* p, int k, int C, const float v[8]) {
  if (k + 8 <= C) {
    storev<TY, 8>(p + k, v);
  } else if (k < C) {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (k + e < C) storev<TY, 1>(p + k + e, v + e);
  }
}

// Where a thread stands: lane `li` of its row's lanes, row `sub` of the `rpb` that the block has at a time.
template <int L>
struct Seat {
  int li, sub, rpb, wave, team;
  __device__ __forceinline__ Seat(int w) {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (L == 64) {
      team = wave / w, li = (wave - team * w) * 64 + lane, sub = team, rpb = (int)(blockDim.x >> 6) / w;
    } else {
      team = wave, li = lane % L, sub = wave * (64 / L) + lane / L, rpb = (int)(blockDim.x >> 6) * (64 / L);
    }
  }
};

constexpr int MAX_WAVES = 16;

// Row r of image b: r = b S + s by the launch's reciprocal of S (see divisor())
__device__ __forceinline__ void locate(const LayerNormArgs& a, int64_t r, int64_t& b, int64_t& s) {
  b = (int64_t)(((uint64_t)r * a.div_m) >> a.div_p);
  s = r - b * a.S;
}

// 1 / sqrt(v), v >= 2^-126: the hardware's and one Newton step (within a step of fp32); 0 of an infinite v
__device__ __forceinline__ float inv_sqrt(float v) {
  const float y = __builtin_amdgcn_rsqf(v);
  return v < INFINITY ? fmaf(y, fmaf(-0.5f * v * y, y, 0.5f), y) : y;
}

// Reads of a row's chunks.  Where a wave has one row, by the row's buffer (what lies past it reads as 0, no branch); VEC:
// bf16 rows begin at words.
template <typename T, int L, bool VEC>
struct Chunks {
  typedef Row<T, VEC> R;
  typedef typename R::Raw Raw;
  R r;
  __device__ __forceinline__ Chunks(const T* p, int C) : r(p, C) {}
  __device__ __forceinline__ Raw load(int k) const { return r.load(k); }
  __device__ __forceinline__ void value(const Raw& w, int k, float v[8]) const { r.value(w, k, v); }
  __device__ __forceinline__ void inner(const Raw& w, float v[8]) const { r.inner(w, v); }
};
template <typename T, bool VEC>
struct Chunks<T, 32, VEC> {
  typedef Vec<T, 8> Raw;
  const T* p;
  int C;
  __device__ __forceinline__ Chunks(const T* p, int C) : p(p), C(C) {}
  __device__ __forceinline__ Raw load(int k) const { return load8(p, k, C); }
  __device__ __forceinline__ void value(const Raw& w, int, float v[8]) const { valuev<T, 8>(w, v); }
  __device__ __forceinline__ void inner(const Raw& w, float v[8]) const { valuev<T, 8>(w, v); }
};
template <typename T, bool VEC>
struct Chunks<T, 16, VEC> : Chunks<T, 32, VEC> {
  using Chunks<T, 32, VEC>::Chunks;
};
template <typename T, bool VEC>
struct Chunks<T, 8, VEC> : Chunks<T, 32, VEC> {
  using Chunks<T, 32, VEC>::Chunks;
};

// Most waves of a block whose rows are held in NC chunks (hold_norm)
constexpr int norm_waves(int NC) { return NC == 1 ? 4 : NC == 2 ? 13 : NC == 3 ? 10 : 8; }

// OUT: 0 fp32, 1 bf16, 2 codes.  w waves to a row.
// Y may be X: a row is loaded whole, by the team that stores it, before it is stored.
// (6 waves to a SIMD where 3 chunks a lane still fit: 4608 x 3072 to codes 13.2 us, 13.8 with 5)
template <typename T, int OUT, int L, int NC, bool VEC>
__global__ __launch_bounds__(64 * norm_waves(NC), L == 64 && NC == 3 ? 6 : 1) void k10_norm(
    LayerNormArgs a, int w, int64_t r0, void* Y, int64_t bsy, int64_t ldy, float* __restrict__ sX, int64_t Mp,
    float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  typedef typename std::conditional<OUT == 0, float, uint16_t>::type TY;
  __shared__ float4 meet[MAX_WAVES];
  const Seat<L> at(w);
  const int C = a.C, step = (L == 64 ? 64 * w : L) * 8;
  const int64_t M = a.B * a.S;
  // the values that this wave (or group of lanes) holds of a row
  auto count = [&](int i) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = i * 512 + j * step;
      n += C - k < 0 ? 0 : C - k < 512 ? C - k : 512;
    }
    return (float)n;
  };
  const float n = L < 64 ? (float)C : count(at.wave - at.team * w), rn = 1.0f / n, rc = 1.0f / (float)C;
  auto whole = [&](int j) { return j + (L == 64 ? 2 : 1) < NC || (j + 1) * step <= C; };  // (the launch sees to the first)
  const int64_t r = r0 + (int64_t)blockIdx.x * at.rpb + at.sub;
  const bool on = r < M;
  int64_t b, s;
  locate(a, on ? r : 0, b, s);
  const Chunks<T, L, VEC> x(static_cast<const T*>(a.X) + b * a.bsx + s * a.ldx, on ? C : 0);
  const Chunks<float, L, true> gamma(a.gamma ? a.gamma + b * a.gs : nullptr, a.gamma ? C : 0);
  const Chunks<float, L, true> beta(a.beta ? a.beta + b * a.gs : nullptr, a.beta ? C : 0);
  const float one = !a.gamma || a.one_plus ? 1.0f : 0.0f;  // without gamma: 1 + 0
  typedef typename Chunks<float, L, true>::Raw RawF;
  float v[NC][8];
  typename Chunks<T, L, VEC>::Raw raw[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) raw[j] = x.load(8 * at.li + j * step);
  // gamma and beta come from cache, a chunk ahead of their use (two: fewer waves to a SIMD, 29.6 us against 26.8 for 9216 x
  // 3072 to codes; at 4 chunks that streams better, 427 against 437 for 65536 x 4096 fp32)
  constexpr int AHEAD = NC == 4 ? 2 : 1;
  RawF gw[AHEAD], bw[AHEAD];
#pragma unroll
  for (int j = 0; j < AHEAD; ++j) gw[j] = gamma.load(8 * at.li + j * step), bw[j] = beta.load(8 * at.li + j * step);
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    if (whole(j)) x.inner(raw[j], v[j]);
    else x.value(raw[j], 8 * at.li + j * step, v[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += v[j][e];  // what lies past C is 0
  }
  const float p = lane_sum<L>(sum) * rn;
  float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
  for (int j = 0; j < NC; ++j)
    within(whole(j), 8 * at.li + j * step, C, [&](int e, bool in) {
      const float d = in ? v[j][e] - p : 0.0f;
      s1 += d;
      s2 = fmaf(d, d, s2);
    });
  s1 = lane_sum<L>(s1), s2 = lane_sum<L>(s2);
  const float c = s1 * rn;  // the mean is p + c
  float mean = p + c, m2 = s2 - s1 * c;
  m2 = m2 < 0.0f ? 0.0f : m2;  // (a NaN passes)
  if (L == 64 && w > 1) {
    if ((threadIdx.x & 63) == 0) meet[at.wave] = make_float4(p, c, m2, n);
    __syncthreads();
    const float4* t = meet + at.team * w;
    // how far a wave's mean lies from the first one's: two small differences, not that of two rounded means
    auto apart = [&](int i) { return (t[i].x - t[0].x) + (t[i].y - t[0].y); };
    float d = 0.0f, q = t[0].z;
    for (int i = 1; i < w; ++i) d = fmaf(t[i].w, apart(i), d);
    d *= rc;
    mean = t[0].x + (t[0].y + d);
    q = fmaf(t[0].w * d, d, q);
    for (int i = 1; i < w; ++i) {
      const float e = apart(i) - d;
      q += fmaf(t[i].w * e, e, t[i].z);
    }
    m2 = q;
  }
  const float rstd = inv_sqrt(m2 * rc + a.eps);
  if (on && at.li == 0) {
    if (mean_out) mean_out[r] = mean;
    if (rstd_out) rstd_out[r] = rstd;
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int k = 8 * at.li + j * step;
    float g[8], t[8];
    gamma.value(gw[j % AHEAD], k, g);
    beta.value(bw[j % AHEAD], k, t);
    if (j + AHEAD < NC) gw[j % AHEAD] = gamma.load(k + AHEAD * step), bw[j % AHEAD] = beta.load(k + AHEAD * step);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = (v[j][e] - mean) * rstd * (one + g[e]) + t[e];  // one rounding an operation
    if constexpr (OUT < 2) {
      TY* y = static_cast<TY*>(Y) + b * bsy + s * ldy;
      if (whole(j)) {
        if (on) storev<TY, 8>(y + k, v[j]);
      } else {
        store_row8(y, k, on ? C : 0, v[j]);
      }
    } else {
      uint32_t top = 0;
      within(whole(j), k, C, [&](int e, bool in) {
        v[j][e] = in ? v[j][e] : 0.0f;  // past the row: zeros
        top = umax(top, abs_bits(v[j][e]));
      });
      top = wave_umax<16>(top);
      float sc, f;
      block_scale(top, sc, f);
      if (on && k < (int)ldy)  // ldy: a row of codes, C rounded up to 128
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(Y) + r * ldy + k) =
            make_uint2(e4m3x4(v[j][0], v[j][1], v[j][2], v[j][3], f), e4m3x4(v[j][4], v[j][5], v[j][6], v[j][7], f));
      if (on && (at.li & 15) == 0 && k < C) sX[(int64_t)(k >> 7) * Mp + r] = sc;
    }
    if constexpr (NC > 2) __builtin_amdgcn_sched_barrier(0);
  }
}

// The gradient.  Rows are in `images` runs of `len` (the images, or all rows as one run); block `block` of `blocks` takes
// rows [block * per, + per) of run blockIdx.y and leaves its columns' sums in part[run][block][2][C], or with one block to a
// run in dgamma and dbeta [run][C] themselves.  SUMS: whether it does.
// dX may be X or dY: a row is loaded whole, by the block that stores it, before it is stored.
template <typename T, typename TD>
struct GradArgs {
  const TD* dY;
  int64_t bsd, ldd;
  const float *mean, *rstd;
  T* dX;
  int64_t bso, ldo;
  float *part, *dgamma, *dbeta;
};

template <typename T, typename TD, int L, int NC, bool SUMS, bool VEC>
__device__ __forceinline__ void grad_rows(const LayerNormArgs& a, int w, int64_t len, int64_t per, const GradArgs<T, TD>& g,
                                          uint32_t block, uint32_t blocks) {
  const TD* dY = g.dY;
  T* dX = g.dX;
  const int64_t bsd = g.bsd, ldd = g.ldd, bso = g.bso, ldo = g.ldo;
  const float *__restrict__ mean_in = g.mean, *__restrict__ rstd_in = g.rstd;
  float *__restrict__ part = g.part, *__restrict__ dgamma = g.dgamma, *__restrict__ dbeta = g.dbeta;
  extern __shared__ float cols[];  // [teams][2][step * NC], where several meet
  __shared__ float2 meet[2][MAX_WAVES];
  const Seat<L> at(w);
  const int C = a.C, step = (L == 64 ? 64 * w : L) * 8;
  const int64_t base = (int64_t)blockIdx.y * len, r0 = base + (int64_t)block * per;
  const int64_t r1 = r0 + per < base + len ? r0 + per : base + len;
  auto whole = [&](int j) { return L == 64 && (j + 1) * step <= C; };
  struct Row1 {
    typename Chunks<T, L, VEC>::Raw x[NC];
    typename Chunks<TD, L, VEC>::Raw d[NC];
    float mean, rstd;
  };
  auto x_of = [&](int64_t r) {
    int64_t b, s;
    locate(a, r < r1 ? r : r0, b, s);
    return Chunks<T, L, VEC>(static_cast<const T*>(a.X) + b * a.bsx + s * a.ldx, r < r1 ? C : 0);
  };
  auto d_of = [&](int64_t r) {
    int64_t b, s;
    locate(a, r < r1 ? r : r0, b, s);
    return Chunks<TD, L, VEC>(dY + b * bsd + s * ldd, r < r1 ? C : 0);
  };
  auto fetch = [&](int64_t r, Row1& w1) {
    const auto x = x_of(r);
    const auto d = d_of(r);
    w1.mean = mean_in[r < r1 ? r : r0], w1.rstd = rstd_in[r < r1 ? r : r0];
#pragma unroll
    for (int j = 0; j < NC; ++j) w1.x[j] = x.load(8 * at.li + j * step), w1.d[j] = d.load(8 * at.li + j * step);
  };
  constexpr bool FETCH_AHEAD = NC == 1;  // (two chunks of two rows do not fit the registers of 16 waves)
  Row1 cur, next;
  fetch(r0 + at.sub, cur);
  float gm[NC][8], ag[NC][8], ab[NC][8];
  const float rc = 1.0f / (float)C, one = !a.gamma || a.one_plus ? 1.0f : 0.0f;  // without gamma: 1 + 0
  // a block's rows share their gamma: a run is an image where images have their own
  const Chunks<float, L, true> gamma(a.gamma ? a.gamma + blockIdx.y * a.gs : nullptr, a.gamma ? C : 0);
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    gamma.value(gamma.load(8 * at.li + j * step), 8 * at.li + j * step, gm[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) gm[j][e] += one, ag[j][e] = ab[j][e] = 0.0f;
  }
  int turn = 0;
  for (int64_t rb = r0; rb < r1; rb += at.rpb, turn ^= 1) {
    const int64_t r = rb + at.sub;
    const bool on = r < r1;
    if constexpr (FETCH_AHEAD) fetch(r + at.rpb, next);
    int64_t b, s;
    locate(a, on ? r : r0, b, s);
    float z[NC][8], d[NC][8], s1 = 0.0f, s2 = 0.0f;
    const auto x = x_of(r);
    const auto dy = d_of(r);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = 8 * at.li + j * step;
      // (zeros past the row and past the last row: nothing of theirs is added)
      if (whole(j)) x.inner(cur.x[j], z[j]), dy.inner(cur.d[j], d[j]);
      else x.value(cur.x[j], k, z[j]), dy.value(cur.d[j], k, d[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[j][e] = (z[j][e] - cur.mean) * cur.rstd;
      within(whole(j) && (L < 64 || on), k, on ? C : 0, [&](int e, bool in) {
        z[j][e] = in ? z[j][e] : 0.0f;
        if constexpr (SUMS) {
          ag[j][e] = fmaf(d[j][e], z[j][e], ag[j][e]);
          ab[j][e] += d[j][e];
        }
        d[j][e] *= gm[j][e];
        s1 += d[j][e];
        s2 = fmaf(d[j][e], z[j][e], s2);
      });
    }
    s1 = lane_sum<L>(s1), s2 = lane_sum<L>(s2);
    if (L == 64 && w > 1) {
      if ((threadIdx.x & 63) == 0) meet[turn][at.wave] = make_float2(s1, s2);
      __syncthreads();
      const float2* t = meet[turn] + at.team * w;
      s1 = s2 = 0.0f;
      for (int i = 0; i < w; ++i) s1 += t[i].x, s2 += t[i].y;
    }
    s1 *= rc, s2 *= rc;
    T* o = dX + b * bso + s * ldo;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = 8 * at.li + j * step;
#pragma unroll
      for (int e = 0; e < 8; ++e) d[j][e] = (d[j][e] - s1 - z[j][e] * s2) * cur.rstd;
      if (whole(j)) {
        if (on) storev<T, 8>(o + k, d[j]);
      } else {
        store_row8(o, k, on ? C : 0, d[j]);
      }
    }
    if constexpr (FETCH_AHEAD) cur = next;
    else if (rb + at.rpb < r1) fetch(r + at.rpb, cur);
  }
  if constexpr (SUMS) {
    // the rows that a wave has side by side, then the block's teams in turn
    if constexpr (L < 64) {
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          auto add = [](float v) {
            if constexpr (L == 8)  // rows rotated by 8
              v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, true));
            if constexpr (L <= 16) {
              const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
              v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
            }
            const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
            return __uint_as_float(h[0]) + __uint_as_float(h[1]);
          };
          ag[j][e] = add(ag[j][e]), ab[j][e] = add(ab[j][e]);
        }
    }
    const int teams = L == 64 ? at.rpb : (int)(blockDim.x >> 6), wide = step * NC;
    const int64_t run = (int64_t)blockIdx.y * blocks + block;
    float* pg = blocks > 1 ? part + run * 2 * C : dgamma ? dgamma + run * C : nullptr;
    float* pb = blocks > 1 ? part + run * 2 * C + C : dbeta ? dbeta + run * C : nullptr;
    const bool mine = L == 64 || (int)(threadIdx.x & 63) < L;  // one group of a wave's lanes has its sums
    if (teams == 1) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int k = 8 * at.li + j * step;
        if (pg) store_row8(pg, k, mine ? C : 0, ag[j]);
        if (pb) store_row8(pb, k, mine ? C : 0, ab[j]);
      }
      return;
    }
    if (mine) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float4* g = reinterpret_cast<float4*>(cols + at.team * 2 * wide + 8 * at.li + j * step);
        float4* b = reinterpret_cast<float4*>(cols + (at.team * 2 + 1) * wide + 8 * at.li + j * step);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          g[h] = make_float4(ag[j][4 * h], ag[j][4 * h + 1], ag[j][4 * h + 2], ag[j][4 * h + 3]);
          b[h] = make_float4(ab[j][4 * h], ab[j][4 * h + 1], ab[j][4 * h + 2], ab[j][4 * h + 3]);
        }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      float g = cols[c], b = cols[wide + c];
      for (int t = 1; t < teams; ++t) g += cols[t * 2 * wide + c], b += cols[(t * 2 + 1) * wide + c];
      if (pg) pg[c] = g;
      if (pb) pb[c] = b;
    }
  }
}

template <typename T, typename TD, int L, int NC, bool SUMS, bool VEC>
__global__ __launch_bounds__(1024) void k10_grad(LayerNormArgs a, int w, int64_t len, int64_t per, GradArgs<T, TD> g) {
  grad_rows<T, TD, L, NC, SUMS, VEC>(a, w, len, per, g, blockIdx.x, gridDim.x);
}

// The columns' sums of a run, cw = 16, 32 or 64 columns to a block and 64 / cw rows to a wave: the forward's mean and
// rstd are known, so nothing of a row has to meet first.
__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(uint16_t bf16) { return __uint_as_float((uint32_t)bf16 << 16); }
template <typename T, typename TD>
__device__ __forceinline__ void grad_cols(const LayerNormArgs& a, int64_t len, const GradArgs<T, TD>& g, uint32_t block,
                                          int cw) {
  constexpr int U = 8;  // rows on their way
  __shared__ float2 sums[MAX_WAVES][64];
  const int C = a.C, lane = threadIdx.x & 63, c = (int)block * cw + (lane & (cw - 1)), slots = (int)blockDim.x / cw;
  // the run's first row; within a run 32 bits of bytes reach (the launch sees to it)
  const int64_t base = (int64_t)blockIdx.y * len;
  const char* X = (const char*)(static_cast<const T*>(a.X) + (int64_t)blockIdx.y * a.bsx);
  const char* D = (const char*)(g.dY + (int64_t)blockIdx.y * g.bsd);
  const float *mean_in = g.mean + base, *rstd_in = g.rstd + base;
  const uint32_t ldx = (uint32_t)a.ldx * sizeof(T), ldd = (uint32_t)g.ldd * sizeof(TD), rows = (uint32_t)len;
  const uint32_t at = c < C ? c : 0;
  float sg = 0.0f, sb = 0.0f;
  for (uint32_t r = threadIdx.x / cw; r < rows; r += slots * U) {
    T x[U];
    TD d[U];
    float mean[U], rstd[U];
    const uint32_t ox = r * ldx + at * sizeof(T), od = r * ldd + at * sizeof(TD);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = r + u * slots < rows;  // else row r once more
      x[u] = *reinterpret_cast<const T*>(X + (in ? ox + u * (slots * ldx) : ox));
      d[u] = *reinterpret_cast<const TD*>(D + (in ? od + u * (slots * ldd) : od));
      mean[u] = mean_in[in ? r + u * slots : r], rstd[u] = rstd_in[in ? r + u * slots : r];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float dv = r + u * slots < rows ? as_f32(d[u]) : 0.0f, z = (as_f32(x[u]) - mean[u]) * rstd[u];
      if (r + u * slots < rows) sg = fmaf(dv, z, sg);
      sb += dv;
    }
  }
  auto add = [&](float v) {  // a wave's rows
    if (cw == 16) {
      const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    }
    if (cw <= 32) {
      const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      v = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    }
    return v;
  };
  sums[threadIdx.x >> 6][lane] = make_float2(add(sg), add(sb));
  __syncthreads();
  if ((int)threadIdx.x < cw && c < C) {
    float2 s = sums[0][lane];
    for (int i = 1; i < (int)(blockDim.x >> 6); ++i) s.x += sums[i][lane].x, s.y += sums[i][lane].y;
    if (g.dgamma) g.dgamma[(int64_t)blockIdx.y * C + c] = s.x;
    if (g.dbeta) g.dbeta[(int64_t)blockIdx.y * C + c] = s.y;
  }
}

// Up to 1024 rows: dX and the columns' sums in one launch, by blocks of their own, which read x and dy once more (fp32
// 16 x 1111 4.6 us, with a second launch 10.5; 400 x 1111 5.5, 9.0; 999 x 1111 9.6, 11.2; 999 x 3072 13.4, 15.8; 1400 x 3072
// 17.6, 17.0)
template <typename T, typename TD, int L, int NC, bool VEC>
__global__ __launch_bounds__(1024) void k10_grad_apart(LayerNormArgs a, int w, int64_t len, int64_t per, GradArgs<T, TD> g,
                                                      int cw, uint32_t col_blocks) {
  if (blockIdx.x < col_blocks) grad_cols<T, TD>(a, len, g, blockIdx.x, cw);
  else grad_rows<T, TD, L, NC, false, VEC>(a, w, len, per, g, blockIdx.x - col_blocks, gridDim.x - col_blocks);
}

// The blocks' partial sums of a run, added in a fixed order: 32 columns, 32 threads each.
constexpr int JOIN = 32;
__global__ __launch_bounds__(32 * JOIN) void k10_join(const float* __restrict__ part, int parts, int C,
                                                     float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float2 sums[JOIN][33];
  const int c = (int)blockIdx.x * 32 + (threadIdx.x & 31), q = threadIdx.x >> 5;
  const float* p = part + (int64_t)blockIdx.y * parts * 2 * C + c;
  float2 s = make_float2(0.0f, 0.0f);
  if (c < C) {
#pragma unroll 4
    for (int i = q; i < parts; i += JOIN) s.x += p[(int64_t)i * 2 * C], s.y += p[(int64_t)i * 2 * C + C];
  }
  sums[q][threadIdx.x & 31] = s;
  __syncthreads();
  if (q == 0 && c < C) {
    s = sums[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < JOIN; ++i) s.x += sums[i][threadIdx.x].x, s.y += sums[i][threadIdx.x].y;
    if (dgamma) dgamma[(int64_t)blockIdx.y * C + c] = s.x;
    if (dbeta) dbeta[(int64_t)blockIdx.y * C + c] = s.y;
  }
}

// How a row is held: L lanes, NC chunks, w waves
struct Hold {
  int L, NC, w;
};
Hold hold(int C, int NC) {
  if (C <= 128) return Hold{16, 1, 1};
  if (C <= 256) return Hold{32, 1, 1};
  return Hold{64, NC, (C + 512 * NC - 1) / (512 * NC)};
}

// The gradient's: 8 lanes up to 64 values (100000 x 64 bf16 15.0 us, by 16 lanes 21.2; 130869 x 33 19.2, 28.6)
Hold hold_grad(int C) { return C <= 64 ? Hold{8, 1, 1} : hold(C, C <= 8192 ? 1 : 2); }

// f(L, NC) as constants.  The norm: 16 lanes of 1 to 4 chunks, 32 of 1, 3 or 4, 64 of 1 to 4; the gradient: one chunk, or
// 64 lanes of 2 (past 8192 values).
template <int L, int... NCs, typename F>
void by_chunks(int NC, F&& f) {
  (void)((NC == NCs ? (f(std::integral_constant<int, L>{}, std::integral_constant<int, NCs>{}), true) : false) || ...);
}

// Few rows: one chunk a lane, so long as that is at most 4 waves; then two, and past 8192 values four, since a join of many
// waves costs more than their loads save (bf16: 8 x 8192 in 16, 8, 4 waves 5.1, 4.1, 4.1 us; 300 x 3072 in 6, 3, 2: 4.65,
// 3.97, 3.92; 400 x 1500 in 3, 2, 1: 3.66, 3.84, 3.69).
// Else what leaves the fewest lanes idle in the fewest waves: 100000 x 320 by 16 lanes 34 us (64: 48), 100000 x 768 by 32
// lanes 60 (64 lanes: 88), 4608 x 3072 by 64 lanes of 3 chunks 12.8 (before gamma came one chunk ahead 13.4; 1: 23.0, 2:
// 14.8, 4: 14.0), 16384 x 2048 of 4 30 (1: 38, 2: 34).
Hold hold_norm(int64_t M, int C) {
  const int one = (C + 511) / 512;  // waves of one chunk
  if (M * one < (C <= 1024 ? 16 : 8) * (int64_t)device_cus()) return hold(C, one <= 4 ? 1 : one <= MAX_WAVES ? 2 : 4);
  if (C <= 512) return Hold{16, (C + 127) / 128, 1};
  if (C <= 1024) return Hold{32, (C + 255) / 256, 1};
  Hold best = hold(C, 2);
  for (int NC : {3, 4}) {
    const Hold h = hold(C, NC);
    if (h.w * NC <= best.w * best.NC && (NC - 2) * 512 * h.w <= C) best = h;  // all chunks but the last two are whole
  }
  return best;
}

// a with the reciprocal of S that locate() uses: for r < 2^31, r m >> p = floor(r / S) with p = 31 + ceil(log2 S) and m =
// ceil(2^p / S), since m S - 2^p < S <= 2^(p - 31), so that r (m S - 2^p) < 2^p
LayerNormArgs divisor(LayerNormArgs a) {
  a.div_p = 31;
  while ((int64_t(1) << (a.div_p - 31)) < a.S) ++a.div_p;
  a.div_m = ((uint64_t(1) << a.div_p) + (uint64_t)a.S - 1) / (uint64_t)a.S;
  return a;
}

template <int OUT>
hipError_t launch(const LayerNormArgs& args, void* Y, int64_t bsy, int64_t ldy, float* sX, float* mean, float* rstd,
                  hipStream_t st) {
  const LayerNormArgs a = divisor(args);
  const int64_t M = a.B * a.S;
  const Hold h = hold_norm(M, a.C);
  const int waves = h.w >= 3 ? h.w : 4;
  const int64_t rpb = h.L == 64 ? waves / h.w : 4 * (64 / h.L);
  const dim3 block(64 * waves);
  const int64_t slab = (int64_t)1 << 21;  // blocks to a launch (it takes fewer than 2^32 threads)
  auto run = [&](auto l, auto c) {
    constexpr int L = decltype(l)::value, NC = decltype(c)::value;
    auto go = [&](auto kernel) {
      for (int64_t r = 0; r < M; r += slab * rpb) {
        const int64_t blocks = std::min((M - r + rpb - 1) / rpb, slab);
        hipLaunchKernelGGL(kernel, dim3((uint32_t)blocks), block, 0, st, a, h.w, r, Y, bsy, ldy, sX, fp8_pad(M), mean, rstd);
      }
    };
    if (a.xdtype == 0) go(k10_norm<float, OUT, L, NC, true>);
    else if (L < 64 || (rows_aligned4(a.X, a.ldx, 1) && a.bsx % 2 == 0)) go(k10_norm<uint16_t, OUT, L, NC, true>);
    else if constexpr (L == 64) go(k10_norm<uint16_t, OUT, L, NC, false>);
  };
  if (h.L == 16) by_chunks<16, 1, 2, 3, 4>(h.NC, run);
  else if (h.L == 32) by_chunks<32, 1, 3, 4>(h.NC, run);
  else by_chunks<64, 1, 2, 3, 4>(h.NC, run);
  return hipGetLastError();
}

hipError_t launch_join(const float* part, uint32_t parts, int64_t runs, int C, float* dgamma, float* dbeta, hipStream_t st) {
  const dim3 grid((uint32_t)((C + 31) / 32), (uint32_t)runs);
  hipLaunchKernelGGL(k10_join, grid, dim3(32 * JOIN), 0, st, part, (int)parts, C, dgamma, dbeta);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, void* Y, int ydtype, int64_t bsy, int64_t ldy, float* mean,
                             float* rstd, hipStream_t st) {
  return ydtype == 0 ? launch<0>(a, Y, bsy, ldy, nullptr, mean, rstd, st) : launch<1>(a, Y, bsy, ldy, nullptr, mean, rstd, st);
}

hipError_t launch_layer_norm_fp8(const LayerNormArgs& a, uint8_t* qX, float* sX, float* mean, float* rstd, hipStream_t st) {
  return launch<2>(a, qX, 0, i8_ld(a.C), sX, mean, rstd, st);
}

LayerNormPlan plan_layer_norm(int64_t M, int C) {
  const Hold h = hold_norm(M, C);
  return LayerNormPlan{h.L, h.NC, h.w};
}

// 16 columns to a block, or more where the card would have to take more than half of its units for them
int columns_apart(int64_t len, int64_t runs, int C) {
  const int64_t cus = device_cus();
  if (len > 1024) return 0;
  for (int cw : {16, 32, 64}) {
    const int64_t blocks = runs * ((C + cw - 1) / cw);
    if (blocks <= (cw == 64 ? cus * 3 / 4 : cus / 2)) return cw;
  }
  return 0;
}

LayerNormGradPlan plan_layer_norm_grad(int64_t B, int64_t S, int C, bool each, bool sums, bool apart) {
  const Hold h = hold_grad(C);
  LayerNormGradPlan p;
  p.runs = each ? B : 1;
  p.len = each ? S : B * S;
  // as many teams to a block as 16 waves hold, and one such block to a unit: half the partial sums of two blocks of 8
  // waves (2x4608x3072 bf16 41.7 us against 48.8, 1024x4096 16.2 against 19.8, 39787x176 36.0 against 36.3)
  p.w = h.w;
  p.waves = MAX_WAVES / h.w * h.w;
  const int64_t rpb = h.L == 64 ? p.waves / h.w : p.waves * (64 / h.L);
  p.cw = sums && apart ? columns_apart(p.len, p.runs, C) : 0;
  p.cols = p.cw ? (uint32_t)((C + p.cw - 1) / p.cw) : 0;
  // blocks of rows to a run: what the columns' blocks leave of the card; else the card, but one where that does it in 4
  // turns and there are sums, whose second launch takes more than that (without sums one block 6.5 us at 512 x 64 fp32, 7.5 at
  // 64 x 400, the card's 3.2 and 3.8)
  const int64_t cus = device_cus(), left = cus / p.runs - p.cols;
  const int64_t most = p.cw ? (left > 1 ? left : 1) : sums && p.len <= 4 * rpb ? 1 : (cus + p.runs - 1) / p.runs;
  const int64_t turns = (p.len + rpb * most - 1) / (rpb * most);
  p.per = turns * rpb;
  p.parts = (uint32_t)((p.len + p.per - 1) / p.per);
  p.bytes = sums && !p.cw && p.parts > 1 ? (size_t)p.runs * p.parts * 2 * (size_t)C * 4 : 0;
  return p;
}

hipError_t launch_layer_norm_grad(const LayerNormArgs& args, const void* dY, int ddtype, int64_t bsd, int64_t ldd,
                                  const float* mean, const float* rstd, void* dX, int64_t bso, int64_t ldo,
                                  float* dgamma, float* dbeta, void* ws, hipStream_t st) {
  const LayerNormArgs a = divisor(args);
  const bool sums = dgamma || dbeta;
  // the columns' blocks read x and dy beside those that write dX, at 32-bit offsets from a run's first row
  const bool one_run = a.gs != 0 || a.B == 1 || (a.bsx == a.S * a.ldx && bsd == a.S * ldd);
  const int64_t run_rows = a.gs != 0 ? a.S : a.B * a.S, most_ld = a.ldx > ldd ? a.ldx : ldd;
  const bool apart = dX != a.X && dX != dY && one_run && run_rows * most_ld < ((int64_t)1 << 29);
  const LayerNormGradPlan p = plan_layer_norm_grad(a.B, a.S, a.C, a.gs != 0, sums, apart);
  const Hold h = hold_grad(a.C);
  float* part = p.bytes ? static_cast<float*>(ws) : nullptr;
  const dim3 grid(p.cols + p.parts, (uint32_t)p.runs), block(64 * p.waves);
  const int teams = p.waves / h.w;
  const int lanes = h.L == 64 ? 64 * h.w : h.L;
  const size_t lds = sums && !p.cw && teams > 1 ? (size_t)teams * 2 * lanes * 8 * 4 : 0;  // at most 64 KB
  const bool words = rows_aligned4(a.X, a.ldx, a.xdtype) && (a.xdtype == 0 || a.bsx % 2 == 0) &&
                     rows_aligned4(dY, ldd, ddtype) && (ddtype == 0 || bsd % 2 == 0);  // bf16 rows begin at words
  auto run = [&](auto l, auto c) {
    constexpr int L = decltype(l)::value, NC = decltype(c)::value;
    auto typed = [&](auto tx, auto td) {
      typedef decltype(tx) T;
      typedef decltype(td) TD;
      const GradArgs<T, TD> g{static_cast<const TD*>(dY), bsd, ldd, mean, rstd, static_cast<T*>(dX), bso, ldo,
                              part, dgamma, dbeta};
      auto go = [&](auto kernel, auto... more) {
        hipLaunchKernelGGL(kernel, grid, block, lds, st, a, p.w, p.len, p.per, g, more...);
      };
      auto kind = [&](auto vec) {
        if (p.cw) go(k10_grad_apart<T, TD, L, NC, decltype(vec)::value>, p.cw, p.cols);
        else if (sums) go(k10_grad<T, TD, L, NC, true, decltype(vec)::value>);
        else go(k10_grad<T, TD, L, NC, false, decltype(vec)::value>);
      };
      if constexpr (L == 64 && (sizeof(T) == 2 || sizeof(TD) == 2)) {
        if (!words) return kind(std::false_type{});
      }
      kind(std::true_type{});
    };
    if (a.xdtype == 0) ddtype == 0 ? typed(float{}, float{}) : typed(float{}, uint16_t{});
    else ddtype == 0 ? typed(uint16_t{}, float{}) : typed(uint16_t{}, uint16_t{});
  };
  if (h.L == 8) by_chunks<8, 1>(h.NC, run);
  else if (h.L == 16) by_chunks<16, 1>(h.NC, run);
  else if (h.L == 32) by_chunks<32, 1>(h.NC, run);
  else by_chunks<64, 1, 2>(h.NC, run);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part || !sums) return e;
  return launch_join(part, p.parts, p.runs, a.C, dgamma, dbeta, st);
}

hipError_t launch_layer_norm_no_rows(int64_t runs, int C, float* dgamma, float* dbeta, hipStream_t st) {
  return launch_join(nullptr, 0, runs, C, dgamma, dbeta, st);
}

}  // namespace svdq
