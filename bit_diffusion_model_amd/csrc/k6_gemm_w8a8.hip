// Kernel 6: the W8A8 product, 8-bit codes with one scale per token and one per channel.
//
// Mathematics: I[m][n] = sum_k qX[m][k] qW[n][k], exact in 32-bit integers (K <= 131072:
// 127^2 K < 2^31); y = ((float)I s_X[m]) s_W[n] + bias[n], in fp32, then optionally GELU,
// rounded once to the output type.  qX comes as rows of ld bytes; qW in the fragment order of
// svdq_prepare_weights_int8: [N / 16][ld / 64] fragments of 1 KB, lane l of a fragment holding
// channel l & 15 and the 16 codes k = 16 (l >> 4) .., N padded to 16 with zeros.  Integer sums
// do not depend on their order, so tiles, K ranges and kernels may be chosen freely: every
// choice gives the same bits.
#include <type_traits>

#include "gemm8.hpp"
#include "int8.hpp"
#include "kernels.hpp"

namespace svdq {
namespace {

typedef int v16i __attribute__((ext_vector_type(16)));

// ---- tiles: v_mfma_i32_32x32x32_i8, both operands through LDS
//
// A block owns BM x BN outputs, WM x WN waves with TI x TJ accumulators of 32 x 32 each, and
// walks K in stages of 128 bytes.  KG K groups of such waves (where there are fewer tiles than
// compute units) take the stages in turn, each with its own buffers, and meet in the epilogue.
// Both operands go global -> LDS by LDS-destination buffer loads into two buffers: the weights
// in their fragment order, whose reads are contiguous; a token row's eight 16-byte slots
// XOR-swizzled by the row so that the operand reads of 16 consecutive rows fall in distinct
// bank groups (no bank conflicts counted).  A stage has four steps of 32 bytes of K; a step's
// operands are read into registers during the step before it.  The one barrier of a stage
// lies before its last step: by then every wave has read the whole buffer (its last step
// waits in registers), so the loads of stage k+2 can go into it, a whole stage ahead of their
// use, and the next stage's first operands are read under the last step's MFMAs.
// The weights are the MFMA's A operand: a lane then holds one token, its registers channels,
// and the channels stand in the A operand's rows in such an order that eight registers are
// eight consecutive channels.  They go from registers to memory in 16-byte pieces, two lanes'
// pieces adjacent: 128 us for 4608x3072x9216, against 136 by whole 128-byte rows put together
// in LDS; 64 bytes put together by lane swaps gained nothing over the 32.
// Rows past M and channel blocks past N lie beyond the buffers' ranges: they read as zeros
// and are not stored.  Blocks are numbered so that each XCD (own L2; blocks go to the eight
// XCDs in turn) gets a contiguous run of tiles in strips of 8 tile rows, whose operand panels
// it then shares.
// P > 1 parts: blockIdx.y takes a range of the stages and stores raw sums to part[y].
//
// What bounds it: tiles of 256 with the operands in cache the card's power (4608x12288x3072 in
// 140 us, 2.5 POP/s; MFMAs alone 97); out of cache the operands' way: 173 us, the MFMA units of a
// busy CU occupied 53% of the time, a stage being fetched one stage, about 1 us, ahead (LDS has
// no room for a third buffer).  Products with few stages: fetch, epilogue and stores in turn
// (16384x320x1280: 20.7 us, of which 42 MB of stores 5).  Blocks that stay and take tile after
// tile, with loads running ahead over the tiles' ends, were no faster there (23.5 us against
// 23.3) and slower in long products (144 against 128): the registers they need crowd the loop.
//
// The LDS arrays come from the kernel (ROOM bytes at least each), so that two tile shapes can
// share them; separate arrays, addressed statically: the compiler then knows that
// operand reads do not touch the buffer whose loads are in flight, and does not wait for them.

template <int WM, int WN, int TI, int TJ, int KG, int ROOM, int OUT>
__device__ __forceinline__ void tile(const int8_t* __restrict__ qX, int64_t ld, const int8_t* __restrict__ qW,
                                     const Out& o, int64_t m0, int64_t n0, int* __restrict__ part, int64_t ldp,
                                     uint8_t* la0, uint8_t* la1, uint8_t* lb0, uint8_t* lb1, float* scales) {
  constexpr int BM = 32 * TI * WM, BN = 32 * TJ * WN, NW = WM * WN;  // NW waves per K group
  constexpr int AB = BM * 128, BB = BN * 128, NA = AB / 1024 / NW, NB = BB / 1024 / NW, NL = NA + NB;
  static_assert(AB % (1024 * NW) == 0 && BB % (1024 * NW) == 0, "whole 1 KB loads per wave");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), wave = wid % NW, g = wid / NW;
  const int l32 = lane & 31, kh = lane >> 5;
  const int ch = (l32 & 19) | (l32 & 4) << 1 | (l32 & 8) >> 1;  // the channel that is row l32 of the A operand
  const int wr = (wave / WN) * 32 * TI, wc = (wave % WN) * 32 * TJ;

  const uint32_t rows = (uint32_t)(o.M - m0 < BM ? o.M - m0 : BM), cols = (uint32_t)(o.N - n0 < BN ? o.N - n0 : BN);
  const uint32_t blocks = (cols + 15) / 16;  // channel blocks of 16 (the last one zero past N)
  const int all = (int)(ld / 128), per = (all + (int)gridDim.y - 1) / (int)gridDim.y;
  const int s0 = (int)blockIdx.y * per, nst = all - s0 < per ? all - s0 : per;  // this part's stages (>= 1)
  const int turns = (nst + KG - 1) / KG;  // stages per K group: group g takes g, g + KG, ..
  uint32_t va[NA], vb[NB];
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    const uint32_t f = wave + NW * q;  // fragment f & 1 of the stage of channel block f >> 1
    vb[q] = (uint32_t)lane * 16 + (f >> 1) * 16 * (uint32_t)ld + (f & 1) * 1024;
  }
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int row = (wave + NW * q) * 8 + (lane >> 3);
    va[q] = (uint32_t)row * (uint32_t)ld + (uint32_t)(((lane & 7) ^ swz8(row)) * 16);
  }
  // the tile's scales and biases (a global load in the epilogue would be waited for there)
  if (!part) {
    for (int i = tid; i < BM; i += 64 * NW * KG) scales[i] = i < (int)rows ? o.sX[m0 + i] : 0.0f;
    for (int i = tid; i < BN; i += 64 * NW * KG) {
      scales[BM + i] = i < (int)cols ? o.sW[n0 + i] : 0.0f;
      scales[BM + BN + i] = o.bias && i < (int)cols ? o.bias[n0 + i] : kNoBias;
    }
  }
  // past the end the buffers have no range: nothing is read and the LDS gets zeros
  auto issue = [&](int k, uint8_t* a, uint8_t* b) {
    const int s = k * KG + g;
    const uint32_t on = s < nst ? 0xFFFFFFFFu : 0u;
    const __amdgpu_buffer_rsrc_t rA = make_rsrc(qX + m0 * ld, (rows * (uint32_t)ld) & on);
    const __amdgpu_buffer_rsrc_t rB = make_rsrc(qW + n0 * ld, (blocks * 16 * (uint32_t)ld) & on);
#pragma unroll
    for (int q = 0; q < NA; ++q) dma16(rA, a + g * AB + (wave + NW * q) * 1024, va[q], (uint32_t)(s0 + s) * 128);
    // channel block c of the tile: 16 ld bytes from the one before it, 2 KB (two fragments) per stage
#pragma unroll
    for (int q = 0; q < NB; ++q)
      dma16(rB, b + g * BB + (wave + NW * q) * 1024, vb[q], (uint32_t)(s0 + s) * 2048);
  };

  v16i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v16i{};
  v4i A[2][TI], B[2][TJ];
  auto read = [&](const uint8_t* a, const uint8_t* b, int s, v4i* fa, v4i* fb) {
    a += g * AB, b += g * BB;
    auto ra = [&](int i) {
      const int r = wr + 32 * i + l32;
      fa[i] = *reinterpret_cast<const v4i*>(a + r * 128 + (((2 * s + kh) ^ swz8(r)) * 16));
    };
    ra(0);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int c = wc + 32 * j + ch, k16 = 2 * s + kh;  // lane (c % 16) + 16 (k16 % 4) of a fragment
      fb[j] = *reinterpret_cast<const v4i*>(b + (c >> 4) * 2048 + (k16 >> 2) * 1024 + (k16 & 3) * 256 + (c & 15) * 16);
    }
#pragma unroll
    for (int i = 1; i < TI; ++i) ra(i);
  };
  auto multiply = [&](const v4i* fa, const v4i* fb) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
  };
  // a step's order: one MFMA, the next step's reads, the other MFMAs (each ahead of one load)
  auto order = [&](bool loads) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, TI + TJ, 0);
    if (loads) {
#pragma unroll
      for (int x = 1; x < TI * TJ; ++x) {
        __builtin_amdgcn_sched_group_barrier(0x020, (NL + TI * TJ - 2) / (TI * TJ > 1 ? TI * TJ - 1 : 1), 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
    } else {
      __builtin_amdgcn_sched_group_barrier(0x008, TI * TJ, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto stage = [&](int k, uint8_t* ca, uint8_t* cb, const uint8_t* na, const uint8_t* nb) {
    read(ca, cb, 1, A[1], B[1]);
    multiply(A[0], B[0]);
    order(false);
    read(ca, cb, 2, A[0], B[0]);
    multiply(A[1], B[1]);
    order(false);
    read(ca, cb, 3, A[1], B[1]);
    multiply(A[0], B[0]);
    order(false);
    wait_vm_lgkm0<0>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue(k + 2, ca, cb);
    read(na, nb, 0, A[0], B[0]);
    multiply(A[1], B[1]);
    order(true);
  };
  issue(0, la0, lb0);
  issue(1, la1, lb1);
  wait_vm_lgkm0<NL>();
  __builtin_amdgcn_s_barrier();
  read(la0, lb0, 0, A[0], B[0]);
  int k = 0;
  for (; k + 2 <= turns; k += 2) {
    stage(k, la0, lb0, la1, lb1);
    stage(k + 1, la1, lb1, la0, lb0);
  }
  if (k < turns) stage(k, la0, lb0, la1, lb1);
  auto owner = [&](int u) { return KG > 1 ? u % KG : g; };  // the K group that finishes unit u of 8 registers
  if constexpr (KG > 1) {
    // the K groups' sums meet in LDS: each unit of 8 registers is finished by one group
    wait_vm_lgkm0<0>();
    __builtin_amdgcn_s_barrier();  // the buffers are free
    constexpr int UNITS = TI * TJ * 2;
    static_assert(KG * NW * UNITS * 2048 <= 4 * ROOM && ROOM % 2048 == 0, "room for the sums");
    auto slot = [&](int grp, int u, int q) {
      const int at = ((grp * NW + wave) * UNITS + u) * 2048 + q * 1024;
      return reinterpret_cast<v4i*>(one_of(at / ROOM, la0, la1, lb0, lb1) + at % ROOM + lane * 16);
    };
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int u = (i * TJ + j) * 2 + q / 2;
          const v16i c = acc[i][j];
          if (owner(u) != g) *slot(g, u, q & 1) = v4i{c[4 * q], c[4 * q + 1], c[4 * q + 2], c[4 * q + 3]};
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        v16i c = acc[i][j];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int u = (i * TJ + j) * 2 + q / 2;
          if (owner(u) != g) continue;
#pragma unroll
          for (int h = 1; h < KG; ++h) {
            const v4i d = *slot((g + h) % KG, u, q & 1);
            c[4 * q] += d[0], c[4 * q + 1] += d[1], c[4 * q + 2] += d[2], c[4 * q + 3] += d[3];
          }
        }
        acc[i][j] = c;
      }
  }
  const int64_t m1 = m0 + wr + l32, n1 = n0 + wc + 8 * kh;
  if (KG == 4 && part) {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int u = 0; u < 2 * TJ; ++u) {
        if (owner(i * 2 * TJ + u) != g) continue;
        const int64_t m = m1 + 32 * i, n = n1 + 16 * u;
        const v16i& c = acc[i][u / 2];
        const int r = 8 * (u & 1);
        if (m < o.M && n < ldp) {
          int4* q = reinterpret_cast<int4*>(part + ((int64_t)blockIdx.y * o.M + m) * ldp + n);
          q[0] = make_int4(c[r], c[r + 1], c[r + 2], c[r + 3]);
          q[1] = make_int4(c[r + 4], c[r + 5], c[r + 6], c[r + 7]);
        }
      }
    return;
  }
  float sw[2 * TJ][8], bb[2 * TJ][8];
  const float* sc = scales + BM + wc + 8 * kh;  // this lane's channels' scales; BN further their biases
#pragma unroll
  for (int u = 0; u < 2 * TJ; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) sw[u][e] = sc[16 * u + e], bb[u][e] = sc[BN + 16 * u + e];
  auto finish = [&](auto whole) {  // whole: no bounds to check
    constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const float sx = scales[wr + 32 * i + l32];
#pragma unroll
      for (int u = 0; u < 2 * TJ; ++u)
        if (owner(i * 2 * TJ + u) == g) {
          const int64_t m = m1 + 32 * i, n = n1 + 16 * u;
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = (float)acc[i][u / 2][8 * (u & 1) + e] * sx * sw[u][e] + bb[u][e];
          if (WHOLE || m < o.M) store8<OUT, WHOLE>(o, m, n, y);
        }
    }
  };
  if (rows == BM && cols == BN) finish(std::true_type{});
  else finish(std::false_type{});
  wait_vm_lgkm0<0>();  // no load into LDS outlives the block, not the last ones without a range either
}

// HALVES: the tiles from `whole` on are cut into two of half as many rows, one block each
template <int WM, int WN, int TI, int TJ, int KG, bool HALVES, int OUT>
__global__ __launch_bounds__(64 * WM * WN * KG, TI * TJ == 1 ? 4 : 2) void k6_tiles(const int8_t* __restrict__ qX, int64_t ld,
                                                              const int8_t* __restrict__ qW, Out o, uint32_t tiles_m,
                                                              uint32_t tiles_n, uint32_t whole, int* __restrict__ part,
                                                              int64_t ldp) {
  constexpr int BM = 32 * TI * WM, BN = 32 * TJ * WN, ROOM = KG * (BM < BN ? BM : BN) * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t la0[KG * BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t la1[KG * BM * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t lb0[KG * BN * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t lb1[KG * BN * 128];
  __shared__ __attribute__((aligned(16))) float scales[BM + 2 * BN];  // the rows', the channels', the biases
  uint32_t m, n;
  if (!HALVES || blockIdx.x < whole) {
    const uint32_t xcd = blockIdx.x & 7, t8 = whole >> 3, r8 = whole & 7;
    tile_at(xcd * t8 + (xcd < r8 ? xcd : r8) + (blockIdx.x >> 3), tiles_m, tiles_n, m, n);
    tile<WM, WN, TI, TJ, KG, ROOM, OUT>(qX, ld, qW, o, (int64_t)m * BM, (int64_t)n * BN, part, ldp, la0, la1, lb0, lb1, scales);
  } else if constexpr (HALVES) {
    const uint32_t h = blockIdx.x - whole;
    tile_at(whole + (h >> 1), tiles_m, tiles_n, m, n);
    const int64_t m0 = (int64_t)m * BM + (h & 1) * (BM / 2);
    if (m0 < o.M)
      tile<WM, WN, TI / 2, TJ, KG, ROOM, OUT>(qX, ld, qW, o, m0, (int64_t)n * BN, part, ldp, la0, la1, lb0, lb1, scales);
  }
}

// The second step of a K split: the parts' sums, then the scales.  A thread owns 8 columns.
__global__ __launch_bounds__(256) void k6_join(const int* __restrict__ part, int parts, int64_t ldp, Out o) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = ldp / 8;
  if (i >= o.M * per) return;
  const int64_t m = i / per, n = i % per * 8;
  int I[8] = {};
  for (int p = 0; p < parts; ++p) {
    const int4* q = reinterpret_cast<const int4*>(part + ((int64_t)p * o.M + m) * ldp + n);
    const int4 u = q[0], v = q[1];
    I[0] += u.x, I[1] += u.y, I[2] += u.z, I[3] += u.w, I[4] += v.x, I[5] += v.y, I[6] += v.z, I[7] += v.w;
  }
  float sw[8], bb[8];
  load_channels(o, n, sw, bb);
  const float sx = o.sX[m];
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = (float)I[e] * sx * sw[e] + bb[e];
  if (o.ydtype == 0) store8<0, false>(o, m, n, y);
  else if (o.ydtype == 1) store8<1, false>(o, m, n, y);
  else store8<2, false>(o, m, n, y);
}

// ---- few tokens: v_mfma_i32_16x16x64_i8, weights straight from memory
//
// Bound by the weights' read (1x3072x9216 4.5 us with the launch: 28 MB at 6.3 TB/s; more rows cost
// their own reads: 16 7.2).  A block of 8 waves owns 16 channels (one channel block of the
// weights' fragment order) and up to 16 NT tokens; its waves take the fragments of 64 along K in
// turn, U loads of 1 KB in flight each, and add their integer sums in LDS.  The weights are
// the A operand, the tokens the B operand: lane l holds token l & 15 and k = 16 (l >> 4) .. + 15.
constexpr int FEW_NW = 8, FEW_U = 6;
constexpr uint32_t kNoLoad = 0x7FFFFF00u;  // past the token rows' range (32 rows of at most 128 KB)

template <int NT>
struct FewSums {
  int v[FEW_NW][NT][64][4];
};

template <int NT>
__device__ __forceinline__ void few_finish(const v4i acc[NT], FewSums<NT>& sums, int wave, int lane, const Out& o,
                                           const float* sx, int64_t n0) {
#pragma unroll
  for (int t = 0; t < NT; ++t) *reinterpret_cast<v4i*>(&sums.v[wave][t][lane][0]) = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * NT; i += 64 * FEW_NW) {
    const int c = i & 15, m = i >> 4;  // consecutive threads: consecutive channels
    const int64_t n = n0 + c;
    if (m >= o.M || n >= o.N) continue;
    int I = 0;
#pragma unroll
    for (int w = 0; w < FEW_NW; ++w) I += sums.v[w][m >> 4][(m & 15) + 16 * (c >> 2)][c & 3];
    float y = (float)I * sx[m] * o.sW[n];
    if (o.bias) y += o.bias[n];
    store1(o, m, n, y);
  }
}

template <int NT>
__global__ __launch_bounds__(64 * FEW_NW) void k6_few(const int8_t* __restrict__ qX, int64_t ld,
                                                      const int8_t* __restrict__ qW, Out o) {
  __shared__ FewSums<NT> sums;
  constexpr int U = FEW_U;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int8_t* wl = qW + n0 * ld + lane * 16;
  const __amdgpu_buffer_rsrc_t rX = make_rsrc(qX, (uint32_t)o.M * (uint32_t)ld);  // tokens past M read zeros
  const uint32_t xoff = (uint32_t)(lane & 15) * (uint32_t)ld + (uint32_t)(lane >> 4) * 16;
  const int frags = (int)(ld / 64);
  v4i acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = v4i{};
  for (int f = wave; f < frags; f += FEW_NW * U) {
    uint4 w[U], x[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = f + u * FEW_NW;  // past the end: any weights, zero tokens
      w[u] = *reinterpret_cast<const uint4*>(wl + (at < frags ? at : frags - 1) * 1024);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        x[u][t] = buf_load16(rX, at < frags ? (uint32_t)at * 64 + (uint32_t)(16 * t) * (uint32_t)ld + xoff : kNoLoad);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, w[u]), __builtin_bit_cast(v4i, x[u][t]),
                                                       acc[t], 0, 0, 0);
  }
  few_finish<NT>(acc, sums, wave, lane, o, o.sX, n0);
}

// The whole layer for few tokens in one launch: every block quantizes the tokens' rows for
// itself (X is small and in L2; the first weights are already on their way).  All 512 threads
// share each row, 8 values each (ld <= 4096), so the smoothing factors are read once for all
// rows and the rows' maxima meet in one barrier.  Codes stand in LDS, rows 16 bytes longer
// than ld so that a fragment's 16 rows fall in distinct bank groups.  RM: most rows.  80
// registers let three blocks share a CU: all blocks of 12288 channels run at once.
template <typename T, bool VEC, bool SMOOTH, int RM>
__global__ __launch_bounds__(64 * FEW_NW) __attribute__((amdgpu_waves_per_eu(6, 6))) void k6_few_layer(
    const T* __restrict__ X, int64_t ldx, int K, const float* __restrict__ inv_s, int64_t ld,
    const int8_t* __restrict__ qW, Out o) {
  extern __shared__ __attribute__((aligned(16))) uint8_t codes[];
  __shared__ FewSums<1> sums;
  __shared__ uint32_t tops[RM][FEW_NW];
  __shared__ float sx[RM], rx[RM];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int8_t* wl = qW + n0 * ld + lane * 16;
  const int frags = (int)(ld / 64), M = (int)o.M;
  const uint32_t row_bytes = (uint32_t)ld + 16;
  const int k0 = 8 * (int)threadIdx.x;
  float v[RM][8];
  uint32_t top[RM];
  uint4 w[FEW_U];
  auto load_w = [&](int g) {
#pragma unroll
    for (int u = 0; u < FEW_U; ++u) {
      const int at = g + u * FEW_NW;
      w[u] = *reinterpret_cast<const uint4*>(wl + (at < frags ? at : frags - 1) * 1024);
    }
  };
  {
    typedef Row<T, VEC> RowX;
    typedef Row<float, true> RowS;
    auto row = [&](int m) { return RowX(X + (m < M ? m : 0) * ldx, m < M ? K : 0); };  // past M: no range, zeros
    const RowS f(inv_s, SMOOTH ? K : 0);
    typename RowX::Raw raw[RM];
#pragma unroll
    for (int m = 0; m < RM; ++m) raw[m] = row(m).load(k0);
    typename RowS::Raw u0 = {};
    if (SMOOTH) u0 = f.load(k0);
    load_w(wave);
    float s[8];
    if (SMOOTH) f.value(u0, k0, s);
#pragma unroll
    for (int m = 0; m < RM; ++m) {
      row(m).value(raw[m], k0, v[m]);
      top[m] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (SMOOTH) v[m][e] *= s[e];
        top[m] = umax(top[m], abs_bits(v[m][e]));
      }
    }
  }
#pragma unroll
  for (int m = 0; m < RM; ++m) top[m] = wave_umax(top[m]);
  if (lane == 0) {
#pragma unroll
    for (int m = 0; m < RM; ++m) tops[m][wave] = top[m];
  }
  __syncthreads();
  if ((int)threadIdx.x < RM) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < FEW_NW; ++i) a = umax(a, tops[threadIdx.x][i]);
    row_scale(a, sx[threadIdx.x], rx[threadIdx.x]);
  }
  __syncthreads();
  if (k0 < ld) {
#pragma unroll
    for (int m = 0; m < RM; ++m)
      if (m < M) {
        const float r = rx[m];
        *reinterpret_cast<uint2*>(codes + (uint32_t)m * row_bytes + k0) =
            make_uint2(codes4(v[m][0], v[m][1], v[m][2], v[m][3], r), codes4(v[m][4], v[m][5], v[m][6], v[m][7], r));
      }
  }
  __syncthreads();
  v4i acc[1] = {};
  const bool on = (lane & 15) < M;
  const uint8_t* xl = codes + (uint32_t)(on ? lane & 15 : 0) * row_bytes + (uint32_t)(lane >> 4) * 16;
  for (int g = wave; g < frags; g += FEW_NW * FEW_U) {
    if (g != wave) load_w(g);
#pragma unroll
    for (int u = 0; u < FEW_U; ++u) {
      const int at = g + u * FEW_NW;
      if (at >= frags) break;
      v4i x = *reinterpret_cast<const v4i*>(xl + at * 64);
      if (!on) x = v4i{};  // tokens past M
      acc[0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, w[u]), x, acc[0], 0, 0, 0);
    }
  }
  few_finish<1>(acc, sums, wave, lane, o, sx, n0);
}

template <int WM, int WN, int TI, int TJ, int KG, bool HALVES = false>
void launch_tiles(const W8A8Plan& p, int64_t ld, const int8_t* qX, const int8_t* qW, const Out& o, int* part,
                  hipStream_t st) {
  constexpr int BM = 32 * TI * WM, BN = 32 * TJ * WN;
  const uint32_t tm = (uint32_t)((o.M + BM - 1) / BM), tn = (uint32_t)((o.N + BN - 1) / BN);
  const uint32_t whole = HALVES ? tm * tn - (uint32_t)p.halved : tm * tn;
  const uint32_t blocks = whole + 2 * (tm * tn - whole);
  const dim3 grid(blocks, (uint32_t)p.parts), block(64 * WM * WN * KG);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, qX, ld, qW, o, tm, tn, whole, part, p.ldp); };
  if (o.ydtype == 0) go(k6_tiles<WM, WN, TI, TJ, KG, HALVES, 0>);
  else if (o.ydtype == 1) go(k6_tiles<WM, WN, TI, TJ, KG, HALVES, 1>);
  else go(k6_tiles<WM, WN, TI, TJ, KG, HALVES, 2>);
}

// ---- the choice of kernel
//
// Every choice gives the same bits, so it is made by estimated time alone (us; S = stages of
// 128 along K, c = blocks that share a compute unit; a round of c blocks takes a[c] S + b[c]).
// The estimates are fitted to 550 measured times (256 CUs, 20 launches back to back; M x K x N;
// over those the choice costs 2% more than the best of the six):
//   few     2.3 + weight bytes x (0.075 + 0.006 M) / MB: 1x3072x9216 4.5 (64 x 2: 8.2), 16x3072x9216 7.2 (8.1),
//           32x3072x9216 11.2 (8.2), 32x1280x1280 4.2 (5.4), 16x12288x3072 9.7 (64 x 4 in 4 parts: 15)
//   64      one K group, up to four blocks to a CU: 2048x640x640 5.3 (128: 6.1), 1024x3072x3072 14.8 (128 x 2: 18.2),
//           512x320x1280 3.7 (128: 5.1); 16384x320x1280 27 (128: 20.7)
//   64 x 2  two K groups (blocks of 8 waves, two to a CU): 512x3072x3072 10.9 (64 x 4: 15.6), 512x12288x3072 36 (64: 50)
//   64 x 4  four K groups (tiles <= CUs): 256x12288x3072 26.9 (one group 48.5, two 32.5)
//   128     two blocks to a CU: 512x3072x9216 22.5 (64 x 2: 29), 2048x12288x3072 74.7 (64 x 2: 110), 8192x640x640 9.8 (64: 10.5)
//   128 x 2 two K groups (tiles <= CUs): 1024x12288x3072 55.3 (one group 69.5), 256x3072x9216 17.5 (one group 19.6)
//   256     1024x3072x9216 35.3 (128: 42), 4608x12288x3072 121-140 (128: 151), 8192x3072x9216 181 (210); 2048x3072x9216 70.6
//           (63.2); a last round for at most half of the CUs runs as tiles of 128 x 256: 9216x3072x9216 275 (whole
//           tiles 285), 2304x3072x9216 77 (82), with GELU 81 (90), 8192x4096x8448 280 (302), 16384x320x2560 35 (39),
//           4608x3072x12288 with GELU 201 (203)
// K parts (tiles of 64 with four groups, S / parts >= 8, all parts on the CUs at once) add the
// partial sums' traffic and a launch, 6 + 12 bytes x M N parts / 6 TB/s: 64x12288x3072 15.6 in 4 parts, 26.3 in one.

// Tiles of 256 that a last round leaves for at most half of the CUs, after at least one whole round
int64_t halved_tiles(int64_t M, int64_t N, int cus) {
  const int64_t T = ((M + 255) / 256) * ((N + 255) / 256), rest = T % cus;
  return T > cus && 2 * rest <= cus ? rest : 0;
}

struct Cost {
  double us;
  int tile, groups, parts;
};

Cost tiles_cost(int64_t M, int64_t N, int S, int cus, int tile, int groups) {
  const double T = (double)((M + tile - 1) / tile) * (double)((N + tile - 1) / tile);
  const double rounds = T / cus;
  double us = 0.0;
  auto by_line = [&](const double* a, const double* b, int most) {  // a[c - 1], b[c - 1]: c blocks on a CU
    const double full = (double)(int64_t)(rounds / most), rest = rounds - full * most;
    us = full * (a[most - 1] * S + b[most - 1]);
    if (rest > 0) us += a[(int)(rest + 0.999999) - 1] * S + b[(int)(rest + 0.999999) - 1];
  };
  static const double a64[] = {0.315, 0.42, 0.42, 0.64}, b64[] = {0.0, 0.8, 0.8, 2.9}, a642[] = {0.26, 0.335},
                      b642[] = {2.5, 3.6}, a644[] = {0.19}, b644[] = {3.6}, a128[] = {0.575, 0.725}, b128[] = {2.6, 5.6},
                      a1282[] = {0.46}, b1282[] = {5.7};
  if (tile == 64 && groups == 1) by_line(a64, b64, 4), us += 2.6;
  else if (tile == 64 && groups == 2) by_line(a642, b642, 2), us += 1.0;
  else if (tile == 64) by_line(a644, b644, 1), us += 0.9;
  else if (tile == 128 && groups == 1) by_line(a128, b128, 2), us += 1.1;
  else if (tile == 128) by_line(a1282, b1282, 1), us += 0.2;
  else {
    const double full = (double)(int64_t)rounds, rest = rounds - full;
    const bool halved = full > 0 && rest <= 0.5;
    us = full * (1.245 * S + 8.3) + (rest == 0 ? 0.0 : (halved ? 0.9 : rest <= 0.625 ? 1.08 : 1.245) * S + 8.3);
  }
  return Cost{us, tile, groups, 1};
}

}  // namespace

W8A8Plan plan_w8a8(int64_t M, int64_t K, int64_t N) {
  const int cus = device_cus();
  const int64_t ld = i8_ld(K), ldp = (N + 7) / 8 * 8;
  const int S = (int)(ld / 128);
  Cost best{1e30, 64, 1, 1};
  auto take = [&](const Cost& c) {
    if (c.us < best.us) best = c;
  };
  take(tiles_cost(M, N, S, cus, 64, 1));
  take(tiles_cost(M, N, S, cus, 128, 1));
  take(tiles_cost(M, N, S, cus, 256, 1));
  const int64_t T64 = ((M + 63) / 64) * ((N + 63) / 64), T128 = ((M + 127) / 128) * ((N + 127) / 128);
  if (T128 <= cus) take(tiles_cost(M, N, S, cus, 128, 2));
  if (T64 <= 2 * cus) take(tiles_cost(M, N, S, cus, 64, 2));
  if (T64 <= cus) {
    for (int parts = 1; parts <= 8 && parts * T64 <= cus && (parts == 1 || S / parts >= 8); parts *= 2) {
      const int per = (S + parts - 1) / parts;
      Cost c = tiles_cost(M, N, per, cus, 64, 4);
      c.parts = (S + per - 1) / per;  // no empty part
      if (c.parts > 1) c.us += 6.0 + 12.0 * (double)(M * ldp) * c.parts / 6e6;
      take(c);
    }
  }
  if (M <= 32) take(Cost{2.3 + (double)(N * ld) * 1e-6 * (0.075 + 0.006 * (double)M), 0, 1, 1});
  W8A8Plan p{best.tile, best.groups, best.parts, ldp, 0, 0};
  if (p.tile == 256) p.halved = halved_tiles(M, N, cus);
  if (p.parts > 1) p.bytes = (size_t)p.parts * (size_t)M * (size_t)ldp * 4;
  return p;
}

// Measured against the quantizer's launch and k6_few (us): 4x3072x9216 6.3 against 2.6 + 5.0, 4x3072x12288
// 7.6 against 3.2 + 6.0, 2x1280x1280 3.4 against 2.8 + 2.7; at 6 and 8 rows the values no longer fit 80
// registers (8x3072x3072 10.7 against 2.9 + 3.2).
bool few_layer(int64_t M, int64_t K) {
  return M <= 4 && i8_ld(K) <= 4096;
}

hipError_t launch_few_layer(int64_t M, int64_t K, int64_t N, const void* X, int xdtype, int64_t ldx, const float* inv_s,
                            const int8_t* qW, const float* sW, const float* bias, void* Y, int64_t ldy, int ydtype,
                            hipStream_t st) {
  const Out o{nullptr, sW, bias, Y, ldy, M, N, ydtype};
  const int64_t ld = i8_ld(K);
  const dim3 g((uint32_t)((N + 15) / 16)), b(64 * FEW_NW);
  const size_t lds = (size_t)M * (size_t)(ld + 16);
  auto go = [&](auto kernel, auto x) { hipLaunchKernelGGL(kernel, g, b, lds, st, x, ldx, (int)K, inv_s, ld, qW, o); };
  const uint16_t* x16 = static_cast<const uint16_t*>(X);
  const float* x32 = static_cast<const float*>(X);
  auto rows = [&](auto rm) {
    constexpr int RM = decltype(rm)::value;
    if (xdtype == 0) inv_s ? go(k6_few_layer<float, true, true, RM>, x32) : go(k6_few_layer<float, true, false, RM>, x32);
    else if (rows_aligned4(X, ldx, xdtype))
      inv_s ? go(k6_few_layer<uint16_t, true, true, RM>, x16) : go(k6_few_layer<uint16_t, true, false, RM>, x16);
    else inv_s ? go(k6_few_layer<uint16_t, false, true, RM>, x16) : go(k6_few_layer<uint16_t, false, false, RM>, x16);
  };
  if (M <= 1) rows(std::integral_constant<int, 1>{});
  else if (M <= 2) rows(std::integral_constant<int, 2>{});
  else rows(std::integral_constant<int, 4>{});
  return hipGetLastError();
}

hipError_t launch_w8a8(int64_t M, int64_t K, int64_t N, const int8_t* qX, const float* sX, const int8_t* qW,
                       const float* sW, const float* bias, void* Y, int64_t ldy, int ydtype, void* ws, hipStream_t st) {
  const int64_t ld = i8_ld(K);
  const Out o{sX, sW, bias, Y, ldy, M, N, ydtype};
  const W8A8Plan p = plan_w8a8(M, K, N);
  if (p.tile == 0) {
    const dim3 g((uint32_t)((N + 15) / 16)), b(64 * FEW_NW);
    if (M <= 16) hipLaunchKernelGGL(k6_few<1>, g, b, 0, st, qX, ld, qW, o);
    else hipLaunchKernelGGL(k6_few<2>, g, b, 0, st, qX, ld, qW, o);
    return hipGetLastError();
  }
  int* part = p.parts > 1 ? static_cast<int*>(ws) : nullptr;
  if (p.tile == 256 && p.halved) launch_tiles<2, 4, 4, 2, 1, true>(p, ld, qX, qW, o, part, st);
  else if (p.tile == 256) launch_tiles<2, 4, 4, 2, 1>(p, ld, qX, qW, o, part, st);
  else if (p.tile == 128 && p.groups == 1) launch_tiles<2, 2, 2, 2, 1>(p, ld, qX, qW, o, part, st);
  else if (p.tile == 128) launch_tiles<2, 2, 2, 2, 2>(p, ld, qX, qW, o, part, st);
  else if (p.groups == 1) launch_tiles<2, 2, 1, 1, 1>(p, ld, qX, qW, o, part, st);
  else if (p.groups == 2) launch_tiles<2, 2, 1, 1, 2>(p, ld, qX, qW, o, part, st);
  else launch_tiles<2, 2, 1, 1, 4>(p, ld, qX, qW, o, part, st);
  if (p.parts > 1)
    hipLaunchKernelGGL(k6_join, dim3((uint32_t)((M * (p.ldp / 8) + 255) / 256)), dim3(256), 0, st, part, p.parts, p.ldp, o);
  return hipGetLastError();
}

}  // namespace svdq
