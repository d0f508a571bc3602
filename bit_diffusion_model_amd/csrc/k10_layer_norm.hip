// Kernel 10: layer norm, its gradient, and the same norm leaving as E4M3 codes with a scale for each block of 128.
//
// Mathematics (per row of C values): mean, biased variance; z = (x - mean) rstd, rstd = 1 / sqrt(var + eps);
// y = z (o + gamma) + beta, o 0 or 1, gamma and beta of all rows or of the row's image.  Backwards, from the forward's
// mean and rstd: g = dy (o + gamma); dx = rstd (g - sum(g) / C - z sum(g z) / C); dgamma = sum over rows dy z,
// dbeta = sum over rows dy.
//
// Design (gfx950): bound by HBM, x (and dy) read once: a row stays in registers, 8 values a lane and chunk.  A row takes
// L = 16, 32 or 64 lanes (up to 512 values, or 1024 in two chunks), or a team of several waves (two chunks: 1024 values
// a wave); a block has several rows or teams at a time and walks over a range of rows, the next row on its way while one is
// computed, with gamma and beta in registers as long as the image stays the same.
// Statistics: a first mean p of the lanes' own group, then d = x - p, sum d and sum d^2: mean = p + sum d / n,
// M2 = sum d^2 - (sum d)^2 / n, so that neither a mean far from zero nor the rounding of p costs digits (a constant row
// gives beta).  Waves join by the pairwise formula (Chan, Golub and LeVeque) about the first one's mean.  One barrier a row.
// The columns' sums of the gradient stay in registers over a block's rows; a block adds its rows' in LDS in turn and leaves
// one partial sum; a second launch adds the blocks'.  Every order is fixed: no atomics.
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
  v += dpp(v, std::integral_constant<int, 0x140>{});  // rows mirrored
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

// f(e) for the values e of a vector at k that lie within the row
template <typename F>
__device__ __forceinline__ void within(int k, int C, F&& f) {
  if (k + 8 <= C) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f(e);
  } else if (k < C) {
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (k + e < C) f(e);
  }
}

template <typename TY, bool NT = false>
__device__ __forceinline__ void store_row8(TY* p, int k, int C, const float v[8]) {
  if (k + 8 <= C) {
    storev<TY, 8, NT>(p + k, v);
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

// OUT: 0 fp32, 1 bf16, 2 codes.  A block takes rows [blockIdx.x * per, + per) of the B * S; w waves to a row.
// Y may be X: a row is loaded whole, by the block that stores it, before it is stored.
template <typename T, int OUT, int L, int NC>
__global__ __launch_bounds__(1024) void k10_norm(LayerNormArgs a, int w, int64_t per, void* Y, int64_t bsy, int64_t ldy,
                                                float* __restrict__ sX, int64_t Mp, float* __restrict__ mean_out,
                                                float* __restrict__ rstd_out) {
  typedef typename std::conditional<OUT == 0, float, uint16_t>::type TY;
  __shared__ float2 meet[2][MAX_WAVES];
  const Seat<L> at(w);
  const int C = a.C, step = (L == 64 ? 64 * w : L) * 8;
  const int64_t M = a.B * a.S, r0 = (int64_t)blockIdx.x * per, r1 = r0 + per < M ? r0 + per : M;
  const T* X = static_cast<const T*>(a.X);
  auto locate = [&](int64_t r, int64_t& b, int64_t& s) {
    b = (uint32_t)r / (uint32_t)a.S;
    s = r - b * a.S;
  };
  Vec<T, 8> raw[NC];
  auto fetch = [&](int64_t r, Vec<T, 8>* v) {
    int64_t b, s;
    locate(r < r1 ? r : r0, b, s);
    const T* x = X + b * a.bsx + s * a.ldx;
#pragma unroll
    for (int j = 0; j < NC; ++j) v[j] = load8(x, 8 * at.li + j * step, r < r1 ? C : 0);
  };
  fetch(r0 + at.sub, raw);
  float gm[NC][8], bt[NC][8];
  int64_t image = -1;
  // the values that this wave (or group of lanes) holds of a row
  const int mine = L < 64 ? C : [&] {
    int n = 0;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = (at.li & ~63) * 8 + j * step;
      n += C - k < 0 ? 0 : C - k < 512 ? C - k : 512;
    }
    return n;
  }();
  const float n = (float)mine, rn = mine ? 1.0f / n : 0.0f;
  int turn = 0;
  for (int64_t rb = r0; rb < r1; rb += at.rpb, turn ^= 1) {
    const int64_t r = rb + at.sub;
    const bool on = r < r1;
    float v[NC][8];
#pragma unroll
    for (int j = 0; j < NC; ++j) valuev<T, 8>(raw[j], v[j]);
    Vec<T, 8> next[NC];
    fetch(r + at.rpb, next);
    int64_t b, s;
    locate(on ? r : r0, b, s);
    if (a.gs ? b != image : image < 0) {
      image = b;
      const float *g = a.gamma + (a.gs ? b * a.gs : 0), *t = a.beta + (a.gs ? b * a.gs : 0);
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int k = 8 * at.li + j * step;
        if (a.gamma) valuev<float, 8>(load8(g, k, C), gm[j]);
        if (a.beta) valuev<float, 8>(load8(t, k, C), bt[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          gm[j][e] = a.gamma ? a.one_plus ? 1.0f + gm[j][e] : gm[j][e] : 1.0f;
          bt[j][e] = a.beta ? bt[j][e] : 0.0f;
        }
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += v[j][e];  // what lies past C is 0
    const float p = lane_sum<L>(sum) * rn;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      within(8 * at.li + j * step, C, [&](int e) {
        const float d = v[j][e] - p;
        s1 += d;
        s2 = fmaf(d, d, s2);
      });
    s1 = lane_sum<L>(s1), s2 = lane_sum<L>(s2);
    float mean = p + s1 * rn, m2 = s2 - s1 * (s1 * rn);
    m2 = m2 < 0.0f ? 0.0f : m2;  // (a NaN passes)
    if (L == 64 && w > 1) {
      if ((threadIdx.x & 63) == 0) meet[turn][at.wave] = make_float2(mean, m2);
      __syncthreads();
      const float2* t = meet[turn] + at.team * w;
      const float m0 = t[0].x;
      auto count = [&](int i) {
        int c = 0;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const int k = i * 512 + j * step;
          c += C - k < 0 ? 0 : C - k < 512 ? C - k : 512;
        }
        return (float)c;
      };
      float d = 0.0f, q = 0.0f;
      for (int i = 1; i < w; ++i) d += count(i) * (t[i].x - m0);
      mean = m0 + d / (float)C;
      for (int i = 0; i < w; ++i) q += t[i].y + count(i) * (t[i].x - mean) * (t[i].x - mean);
      m2 = q;
    }
    const float rstd = 1.0f / sqrtf(m2 / (float)C + a.eps);
    if (on && at.li == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int k = 8 * at.li + j * step;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = fmaf((v[j][e] - mean) * rstd, gm[j][e], bt[j][e]);
      if constexpr (OUT < 2) {
        store_row8(static_cast<TY*>(Y) + b * bsy + s * ldy, k, on ? C : 0, v[j]);
      } else {
        uint32_t top = 0;
        if (k + 8 > C) {  // past the row: zeros
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = k + e < C ? v[j][e] : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) top = umax(top, abs_bits(v[j][e]));
        top = wave_umax<16>(top);
        float sc, f;
        block_scale(top, sc, f);
        if (on && k < (int)ldy)  // ldy: a row of codes, C rounded up to 128
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(Y) + r * ldy + k) =
              make_uint2(e4m3x4(v[j][0], v[j][1], v[j][2], v[j][3], f), e4m3x4(v[j][4], v[j][5], v[j][6], v[j][7], f));
        if (on && (at.li & 15) == 0 && k < C) sX[(int64_t)(k >> 7) * Mp + r] = sc;
      }
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) raw[j] = next[j];
  }
}

// The gradient.  Rows are in `images` runs of `len` (the images, or all rows as one run); a block takes rows
// [blockIdx.x * per, + per) of run blockIdx.y and leaves its columns' sums in part[run][blockIdx.x][2][C], or with one
// block to a run in dgamma and dbeta [run][C] themselves.  SUMS: whether they are wanted.
// dX may be X or dY: a row is loaded whole, by the block that stores it, before it is stored.
template <typename T, typename TD, int L, int NC, bool SUMS>
__global__ __launch_bounds__(1024) void k10_grad(LayerNormArgs a, int w, int64_t len, int64_t per, const TD* dY,
                                                int64_t bsd, int64_t ldd, const float* __restrict__ mean_in,
                                                const float* __restrict__ rstd_in, T* dX, int64_t bso, int64_t ldo,
                                                float* __restrict__ part, float* __restrict__ dgamma,
                                                float* __restrict__ dbeta) {
  extern __shared__ float cols[];  // [2][step * NC], where several teams meet
  __shared__ float2 meet[2][MAX_WAVES];
  const Seat<L> at(w);
  const int C = a.C, step = (L == 64 ? 64 * w : L) * 8;
  const int64_t base = (int64_t)blockIdx.y * len, r0 = base + (int64_t)blockIdx.x * per;
  const int64_t r1 = r0 + per < base + len ? r0 + per : base + len;
  const T* X = static_cast<const T*>(a.X);
  struct Row1 {
    Vec<T, 8> x[NC];
    Vec<TD, 8> d[NC];
    float mean, rstd;
  };
  auto locate = [&](int64_t r, int64_t& b, int64_t& s) {
    b = (uint32_t)r / (uint32_t)a.S;
    s = r - b * a.S;
  };
  auto fetch = [&](int64_t r, Row1& w1) {
    const bool on = r < r1;
    int64_t b, s;
    if (!on) r = r0;
    locate(r, b, s);
    const T* x = X + b * a.bsx + s * a.ldx;
    const TD* d = dY + b * bsd + s * ldd;
    w1.mean = mean_in[r], w1.rstd = rstd_in[r];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      w1.x[j] = load8(x, 8 * at.li + j * step, on ? C : 0);
      w1.d[j] = load8(d, 8 * at.li + j * step, on ? C : 0);
    }
  };
  Row1 cur, next;
  if (r0 < r1) fetch(r0 + at.sub, cur);
  float gm[NC][8], ag[NC][8], ab[NC][8];
#pragma unroll
  for (int j = 0; j < NC; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) ag[j][e] = ab[j][e] = 0.0f;
  int64_t image = -1;
  const float rc = 1.0f / (float)C;
  int turn = 0;
  for (int64_t rb = r0; rb < r1; rb += at.rpb, turn ^= 1) {
    const int64_t r = rb + at.sub;
    const bool on = r < r1;
    fetch(r + at.rpb, next);
    int64_t b, s;
    locate(on ? r : r0, b, s);
    if (a.gs ? b != image : image < 0) {
      image = b;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        if (a.gamma) valuev<float, 8>(load8(a.gamma + (a.gs ? b * a.gs : 0), 8 * at.li + j * step, C), gm[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) gm[j][e] = a.gamma ? a.one_plus ? 1.0f + gm[j][e] : gm[j][e] : 1.0f;
      }
    }
    float z[NC][8], d[NC][8], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      valuev<T, 8>(cur.x[j], z[j]);
      valuev<TD, 8>(cur.d[j], d[j]);  // zeros past the row and past the last row: nothing of theirs is added
#pragma unroll
      for (int e = 0; e < 8; ++e) z[j][e] = (z[j][e] - cur.mean) * cur.rstd;
      if (!on || 8 * at.li + j * step + 8 > C) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[j][e] = on && 8 * at.li + j * step + e < C ? z[j][e] : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (SUMS) {
          ag[j][e] = fmaf(d[j][e], z[j][e], ag[j][e]);
          ab[j][e] += d[j][e];
        }
        d[j][e] *= gm[j][e];
        s1 += d[j][e];
        s2 = fmaf(d[j][e], z[j][e], s2);
      }
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
#pragma unroll
      for (int e = 0; e < 8; ++e) d[j][e] = (d[j][e] - s1 - z[j][e] * s2) * cur.rstd;
      store_row8(o, 8 * at.li + j * step, on ? C : 0, d[j]);
    }
    cur = next;
  }
  if constexpr (SUMS) {
    // the rows that a wave has side by side, then the block's teams in turn
    if constexpr (L < 64) {
#pragma unroll
      for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          auto add = [](float v) {
            if constexpr (L == 16) {
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
    const int64_t run = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    float* pg = gridDim.x > 1 ? part + run * 2 * C : dgamma ? dgamma + run * C : nullptr;
    float* pb = gridDim.x > 1 ? part + run * 2 * C + C : dbeta ? dbeta + run * C : nullptr;
    if (teams == 1) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int k = 8 * at.li + j * step, end = L == 64 || (int)(threadIdx.x & 63) < L ? C : 0;
        if (pg) store_row8(pg, k, end, ag[j]);
        if (pb) store_row8(pb, k, end, ab[j]);
      }
      return;
    }
    for (int t = 0; t < teams; ++t) {
      if (at.team == t && (L == 64 || (int)(threadIdx.x & 63) < L)) {
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          float4* g = reinterpret_cast<float4*>(cols + 8 * at.li + j * step);
          float4* b = reinterpret_cast<float4*>(cols + wide + 8 * at.li + j * step);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float4 u = make_float4(0, 0, 0, 0), v = u;
            if (t) u = g[h], v = b[h];
            g[h] = make_float4(u.x + ag[j][4 * h], u.y + ag[j][4 * h + 1], u.z + ag[j][4 * h + 2], u.w + ag[j][4 * h + 3]);
            b[h] = make_float4(v.x + ab[j][4 * h], v.y + ab[j][4 * h + 1], v.z + ab[j][4 * h + 2], v.w + ab[j][4 * h + 3]);
          }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < C; c += blockDim.x) {
      if (pg) pg[c] = cols[c];
      if (pb) pb[c] = cols[wide + c];
    }
  }
}

// The blocks' partial sums of a run, added in a fixed order: 32 columns, 8 threads each.
__global__ __launch_bounds__(256) void k10_join(const float* __restrict__ part, int parts, int C,
                                                float* __restrict__ dgamma, float* __restrict__ dbeta) {
  __shared__ float2 sums[8][32];
  const int c = (int)blockIdx.x * 32 + (threadIdx.x & 31), q = threadIdx.x >> 5;
  const float* p = part + (int64_t)blockIdx.y * parts * 2 * C + c;
  float2 s = make_float2(0.0f, 0.0f);
  if (c < C) {
#pragma unroll 8
    for (int i = q; i < parts; i += 8) s.x += p[(int64_t)i * 2 * C], s.y += p[(int64_t)i * 2 * C + C];
  }
  sums[q][threadIdx.x & 31] = s;
  __syncthreads();
  if (q == 0 && c < C) {
    s = sums[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 8; ++i) s.x += sums[i][threadIdx.x].x, s.y += sums[i][threadIdx.x].y;
    if (dgamma) dgamma[(int64_t)blockIdx.y * C + c] = s.x;
    if (dbeta) dbeta[(int64_t)blockIdx.y * C + c] = s.y;
  }
}

// How a row is held: L lanes, NC chunks, w waves
struct Hold {
  int L, NC, w;
};
Hold hold(int C) {
  if (C <= 128) return Hold{16, 1, 1};
  if (C <= 256) return Hold{32, 1, 1};
  if (C <= 512) return Hold{64, 1, 1};
  return Hold{64, 2, (C + 1023) / 1024};
}

template <typename F>
void by_hold(const Hold& h, F&& f) {
  if (h.L == 16) f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  else if (h.L == 32) f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  else if (h.NC == 1) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
}

template <int OUT>
hipError_t launch(const LayerNormArgs& a, void* Y, int64_t bsy, int64_t ldy, float* sX, float* mean, float* rstd,
                  hipStream_t st) {
  const Hold h = hold(a.C);
  const int64_t M = a.B * a.S;
  const int waves = h.w > 1 ? h.w : 4;
  const int rpb = h.w > 1 ? 1 : 4 * (64 / h.L);
  // enough blocks to fill the card, then rows to a block
  const int64_t most = (int64_t)device_cus() * (32 / waves);
  int64_t turns = (M + rpb * most - 1) / (rpb * most);
  const int64_t per = turns * rpb;
  const dim3 grid((uint32_t)((M + per - 1) / per)), block(64 * waves);
  by_hold(h, [&](auto l, auto c) {
    constexpr int L = decltype(l)::value, NC = decltype(c)::value;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, a, h.w, per, Y, bsy, ldy, sX, fp8_pad(M), mean, rstd); };
    if (a.xdtype == 0) go(k10_norm<float, OUT, L, NC>);
    else go(k10_norm<uint16_t, OUT, L, NC>);
  });
  return hipGetLastError();
}

hipError_t launch_join(const float* part, uint32_t parts, int64_t runs, int C, float* dgamma, float* dbeta, hipStream_t st) {
  hipLaunchKernelGGL(k10_join, dim3((uint32_t)((C + 31) / 32), (uint32_t)runs), dim3(256), 0, st, part, (int)parts, C, dgamma, dbeta);
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

LayerNormGradPlan plan_layer_norm_grad(int64_t B, int64_t S, int C, bool each, bool sums) {
  const Hold h = hold(C);
  LayerNormGradPlan p;
  p.runs = each ? B : 1;
  p.len = each ? S : B * S;
  // teams to a block: up to 12 waves
  p.w = h.w;
  p.waves = h.w > 1 ? (h.w > 12 ? h.w : 12 / h.w * h.w) : 8;
  const int64_t rpb = h.w > 1 ? p.waves / h.w : p.waves * (64 / h.L);
  const int64_t most = (device_cus() * 2 + p.runs - 1) / p.runs;  // blocks to a run
  const int64_t turns = (p.len + rpb * most - 1) / (rpb * most);
  p.per = turns * rpb;
  p.parts = (uint32_t)((p.len + p.per - 1) / p.per);
  p.bytes = sums && p.parts > 1 ? (size_t)p.runs * p.parts * 2 * (size_t)C * 4 : 0;
  return p;
}

hipError_t launch_layer_norm_grad(const LayerNormArgs& a, const void* dY, int ddtype, int64_t bsd, int64_t ldd,
                                  const float* mean, const float* rstd, void* dX, int64_t bso, int64_t ldo,
                                  float* dgamma, float* dbeta, void* ws, hipStream_t st) {
  const bool sums = dgamma || dbeta;
  const LayerNormGradPlan p = plan_layer_norm_grad(a.B, a.S, a.C, a.gs != 0, sums);
  const Hold h = hold(a.C);
  float* part = p.parts > 1 ? static_cast<float*>(ws) : nullptr;
  const dim3 grid(p.parts, (uint32_t)p.runs), block(64 * p.waves);
  const size_t lds = sums && p.waves > h.w ? (size_t)2 * (h.L == 64 ? 64 * h.w : h.L) * 8 * h.NC * 4 : 0;  // at most 48 KB
  by_hold(h, [&](auto l, auto c) {
    constexpr int L = decltype(l)::value, NC = decltype(c)::value;
    auto typed = [&](auto tx, auto td) {
      typedef decltype(tx) T;
      typedef decltype(td) TD;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, block, lds, st, a, p.w, p.len, p.per, static_cast<const TD*>(dY), bsd, ldd, mean,
                           rstd, static_cast<T*>(dX), bso, ldo, part, dgamma, dbeta);
      };
      if (sums) go(k10_grad<T, TD, L, NC, true>);
      else go(k10_grad<T, TD, L, NC, false>);
    };
    if (a.xdtype == 0) ddtype == 0 ? typed(float{}, float{}) : typed(float{}, uint16_t{});
    else ddtype == 0 ? typed(uint16_t{}, float{}) : typed(uint16_t{}, uint16_t{});
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part || !sums) return e;
  return launch_join(part, p.parts, p.runs, a.C, dgamma, dbeta, st);
}

hipError_t launch_layer_norm_no_rows(int64_t runs, int C, float* dgamma, float* dbeta, hipStream_t st) {
  return launch_join(nullptr, 0, runs, C, dgamma, dbeta, st);
}

}  // namespace svdq
