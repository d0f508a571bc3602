// Kernel 9: the matrix product on E4M3 codes with a scale for each block of 128.
//
// Mathematics: y[m][n] = sum over blocks b of 128 along K of (sX[b][m] sW[n / 128][b]) D_b[m][n] + bias[n], D_b[m][n]
// the sum of the block's 128 products of codes as the matrix core adds them (see Accuracy); blocks added in
// fp32, then optionally GELU, rounded once to the output type.  qX comes as rows of ld bytes, sX as rows of Mp = M
// rounded up to 4 along the tokens; qW in the fragment order of svdq_prepare_weights_int8: [N / 16][ld / 64] fragments
// of 1 KB, lane l of a fragment holding channel l & 15 and the 16 codes k = 16 (l >> 4) .., N padded to 16 with zeros.
// The matrix core takes 128 codes of K (a block) of 16 x 16 outputs at once, 32 to a lane; a lane's 32 are two 16-byte
// pieces of a fragment, the same pieces for both operands: a sum does not ask in which order k comes.
//
// Accuracy: on E4M3 operands the matrix core takes the products of 8 successive codes together: with E the largest sum of
// two codes' exponents (-6 of a subnormal code; zeros do not count), it drops from each product, toward zero, what lies
// below 2^(E - 13): bit for bit so, and in the older 16x16x32 form, at a third of the rate, too.  Products of normal codes
// within 7 binades of the largest lose nothing; so with terms of random signs the loss is 1.3e-5 of the outputs' root mean
// square for codes of normals, 2.1e-5 with channels 30 times as large, 5e-5 to 6e-5 for codes of all binades alike, the
// same for one block and for 96; with terms of one sign 2.4e-6 of the sum.  Rounding to bf16 costs 1.7e-3 in the root mean
// square, so bf16 outputs of tiles take that loss: 1.1% of them round the other way (1.7% with those channels, 3.3% of all
// binades alike, 0.05% of one sign), and what cancels to below a hundredth of the others is off by more than its rounding.
// fp32 outputs, and the few-token kernels of either type (bound by the weights' read), widen the codes to f16, exactly,
// whose products are kept whole in the fp32 sum (1e-8 to 9e-8 of the root mean square): twice the MFMA time and the
// conversions (4608 x 3072 x 9216 252 us for 124).
#include <type_traits>

#include "fp8.hpp"
#include "gemm8.hpp"
#include "kernels.hpp"
#include "vec.hpp"

namespace svdq {
namespace {

__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t r, float* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4, voff, soff, 0, 0);
}

__device__ __forceinline__ v8i join8(v4i a, v4i b) { return v8i{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}; }

// unscaled E4M3 x E4M3 (both scale operands the constant 0 choose the form without scales)
__device__ __forceinline__ v4f mfma16(v8i a, v8i b, v4f c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Codes as f16 (exact: E4M3 has 4 significant bits and binary exponents from -9 to 8)
typedef _Float16 v8hf __attribute__((ext_vector_type(8)));
struct Half32 { v8hf v[4]; };
__device__ __forceinline__ v8hf widen8(int a, int b) {
  const h2 p = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
  const h2 q = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
  const h2 r = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
  const h2 t = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  return v8hf{p.x, p.y, q.x, q.y, r.x, r.y, t.x, t.y};
}
__device__ __forceinline__ Half32 widen(v8i c) {
  Half32 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h.v[i] = widen8(c[2 * i], c[2 * i + 1]);
  return h;
}

// 8 codes a lane of a 16 x 16 tile, 32 of K
__device__ __forceinline__ v4f dot32(uint32_t a0, uint32_t a1, uint32_t b0, uint32_t b1, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8((int)a0, (int)a1), widen8((int)b0, (int)b1), c, 0, 0, 0);
}

// The swizzle of a token row's eight 16-byte slots.  An operand's 16 lanes of one slot and 16 of the next are read 4 by 4
// in turn ({0-3, 12-15} of one with {4-11} of the other): so the 8 even rows (and the 8 odd ones) of each such 16
// fall in 8 different slots.  (Kernel 6's, made for 32 rows of one slot, costs 2 accesses in each here.)
__device__ __forceinline__ int swz16(int row) { return (row & 6) | (row >> 2 & 1); }

// Token rows of a stage in LDS: whole loads of 8 rows for each wave
constexpr int tile_rows(int WM, int WN, int IA) { return (2 * IA * WM + WM * WN - 1) / (WM * WN) * WM * WN * 8; }

struct Scales {
  const float *sX, *sW;
  int64_t Mp, blocks;  // length of a row of sX; blocks of 128 along K (a row of sW)
};

// ---- tiles: v_mfma_f32_16x16x128_f8f6f4 (fp32 outputs: 4 v_mfma_f32_16x16x32_f16), both operands through LDS
//
// A block owns BM x BN outputs, WM x WN waves with IA groups of 16 tokens by TJ of 32 channels each, and walks K in stages
// of 128 bytes, which are the scales' blocks.  Loads into LDS, barrier and the order of tiles are the integer product's
// (kernel 6); what differs is the sum: an MFMA starts from zero, and its 4 results a lane go to the tile's sums by 4 FMAs
// with the one factor sX[token] sW[channel block], for the weights are the A operand, so that a lane is one token, and a
// wave's channels lie in one block of 128.  The FMAs of a group of 16 tokens run under the next group's MFMAs, the last
// group's under the next stage's first (MFMAs of 32 x 32 x 64 want two of them and 16 FMAs a tile, and registers for two
// sets of results: 186 us against 178 at 4608 x 12288 x 3072).  Operands are read 2 or 3 groups before their use (165 for
// 178), a stage's loads spread over its groups (159 for 163), the tokens' scales come with the operands, by 4-byte loads
// into LDS (a wave's 64 lanes fetch the scales that are its share); the weights' stand in a register, lane s for stage s of
// 64, and are read out by lane.
// Bound.  4608 x 12288 x 3072 bf16, 150 to 160 us, 2.2 POP/s: power.  The matrix cores are busy 64% of the cycles on 252
// units in tiles of 224 rows (77% on 216 units in tiles of 256) and the clock falls to 1.95 GHz (1.81); without the FMAs it
// takes as long.  At K = 3072 the share of a round that nothing overlaps, a tile's first loads and its stores, 7.2 us for
// 34.6 of work: 4608 x 3072 x 9216 124 to 128 us, 2.1 POP/s, the matrix cores busy 58%; 4608 x 3072 x 12288 with GELU 180 to
// 200, 52%.  fp32 outputs (512 x 9216 x 3072 46 us): the conversions, at half the vector rate, twice for each operand in
// tiles of 64 (vector units busy 58%, matrix cores 35%).
template <int WM, int WN, int IA, int TJ, int KG, int ROOM, int OUT>
__device__ __forceinline__ void tile(const uint8_t* __restrict__ qX, int64_t ld, const uint8_t* __restrict__ qW,
                                     const Scales& sc, const Out& o, int64_t m0, int64_t n0, float* __restrict__ part,
                                     int64_t ldp, uint8_t* la0, uint8_t* la1, uint8_t* lb0, uint8_t* lb1, float* lx0,
                                     float* lx1) {
  constexpr int BM = 16 * IA * WM, BN = 32 * TJ * WN, NW = WM * WN;  // NW waves per K group
  // Whole 1 KB loads per wave and stage: the token rows in LDS are BM rounded up to that (the rest is not read)
  constexpr int AB = tile_rows(WM, WN, IA) * 128, BB = BN * 128, NA = AB / 1024 / NW, NB = BB / 1024 / NW, NL = NA + NB + 1;
  constexpr int XW = BM / NW > 16 ? 32 : 16;  // token scales that a wave fetches, into a slot of 64
  constexpr int JB = 2 * TJ;  // a wave's operands: IA groups of 16 tokens, JB of 16 channels
  static_assert(BB % (1024 * NW) == 0, "whole 1 KB loads per wave");
  static_assert(XW * NW >= BM, "a share of the scales is one load, and holds whole groups of 16");
  static_assert(32 * TJ <= 128, "one block of channels to a wave");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wid = __builtin_amdgcn_readfirstlane(tid >> 6), wave = wid % NW, g = wid / NW;
  const int l16 = lane & 15, l4 = lane >> 4;
  const int ch = (l16 >> 2) * 8 + (l16 & 3);  // the channel of 32 that is row l16 of an even operand; 4 on: of the odd one
  const int wr = (wave / WN) * 16 * IA, wc = (wave % WN) * 32 * TJ;

  const uint32_t rows = (uint32_t)(o.M - m0 < BM ? o.M - m0 : BM), cols = (uint32_t)(o.N - n0 < BN ? o.N - n0 : BN);
  const uint32_t blocks = (cols + 15) / 16;  // channel blocks of 16 (the last one zero past N)
  const int all = (int)sc.blocks, per = (all + (int)gridDim.y - 1) / (int)gridDim.y;
  const int s0 = (int)blockIdx.y * per, nst = all - s0 < per ? all - s0 : per;  // this part's stages (>= 1)
  const int turns = (nst + KG - 1) / KG;  // stages per K group: group g takes g, g + KG, ..
  uint32_t va[NA], vb[NB];
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    // fragment f & 1 of the stage of channel block f >> 1; odd blocks with their channels' fours exchanged (see get_b)
    const uint32_t f = wave + NW * q;
    vb[q] = (uint32_t)(lane ^ (f >> 1 & 1) * 4) * 16 + (f >> 1) * 16 * (uint32_t)ld + (f & 1) * 1024;
  }
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int row = (wave + NW * q) * 8 + (lane >> 3);
    va[q] = (uint32_t)row * (uint32_t)ld + (uint32_t)(((lane & 7) ^ swz16(row)) * 16);
  }
  // the wave's share of the stage's token scales: one each for its first XW lanes, nothing for the others
  const uint32_t vx = lane < XW && wave * XW + lane < (int)rows ? (uint32_t)(wave * XW + lane) * 4 : kNoStore;
  // the weights' scales of this wave's channels (channels past N: the last block's; they are not stored)
  const int64_t cb = (n0 + wc) / 128, cbs = (o.N + 127) / 128;
  const float* sw_row = sc.sW + (cb < cbs ? cb : cbs - 1) * sc.blocks;
  auto load_sw = [&](int k) {  // lane l: turn k + l
    const int s = s0 + (k + lane) * KG + g;
    return s < all ? sw_row[s] : 0.0f;
  };
  // load n of stage k; past the end the buffers have no range: nothing is read and the LDS gets zeros
  auto issue = [&](int n, int k, uint8_t* a, uint8_t* b, float* x) {
    const int s = k * KG + g;
    const uint32_t on = s < nst ? 0xFFFFFFFFu : 0u;
    if (n < NA) {
      dma16(make_rsrc(qX + m0 * ld, (rows * (uint32_t)ld) & on), a + g * AB + (wave + NW * n) * 1024, va[n],
            (uint32_t)(s0 + s) * 128);
    } else if (n < NA + NB) {  // channel block c: 16 ld bytes from the one before it, 2 KB (two fragments) per stage
      dma16(make_rsrc(qW + n0 * ld, (blocks * 16 * (uint32_t)ld) & on), b + g * BB + (wave + NW * (n - NA)) * 1024, vb[n - NA],
            (uint32_t)(s0 + s) * 2048);
    } else {
      dma4(make_rsrc(sc.sX + (int64_t)(s0 + (s < nst ? s : 0)) * sc.Mp + m0, (rows * 4) & on), x + (g * NW + wave) * 64, vx, 0);
    }
  };

  constexpr bool FINE = OUT == 0;
  // Token operands in registers; how many groups ahead they are read; a stage's loads go out over STEPS groups, PER in each,
  // the first AHEAD of them behind the barrier, the others in the next stage
  // (7 groups a stage: with 4 sets of registers, group i in set i & 3, only two groups are ahead without meeting)
  constexpr int RING = IA == 6 ? 3 : IA > 2 ? 4 : 2, AHEAD = IA % 8 == 0 ? 3 : IA > 2 ? 2 : 1;
  constexpr int STEPS = IA > 4 ? 5 : IA > 2 ? 3 : 1;
  static_assert(IA % RING == 0 || (IA % RING == 3 && AHEAD == 2), "the groups in flight lie in different sets");
  constexpr int PER = (NL + STEPS - 1) / STEPS, FIRST = PER * AHEAD < NL ? PER * AHEAD : NL;
  v4f acc[IA][JB], T[JB];
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    T[j] = v4f{};
#pragma unroll
    for (int i = 0; i < IA; ++i) acc[i][j] = v4f{};
  }
  v8i fa[RING], fb[JB];  // a lane's 32 codes of a stage
  float fx[RING];
#pragma unroll
  for (int i = 0; i < RING; ++i) fx[i] = 0.0f;
  const int r0 = wr + l16;
  const uint32_t at_a = (uint32_t)(g * AB + r0 * 128 + ((l4 ^ swz16(r0)) * 16));  // and the slot 4 on: bit 6
  auto get_a = [&](const uint8_t* a, int i) {
    return join8(*reinterpret_cast<const v4i*>(a + at_a + 2048 * i), *reinterpret_cast<const v4i*>(a + (at_a ^ 64) + 2048 * i));
  };
  // An operand's 16 rows are channels of two blocks of 16: with the fours of the odd one exchanged they lie in 16 different
  // slots (without: two in each, 16 M cycles of bank conflicts in 70 M)
  const uint32_t at_b = (uint32_t)(g * BB + ((wc + ch) >> 4) * 2048 + l4 * 256 + ((ch & 15) ^ (ch >> 2 & 4)) * 16);
  auto get_b = [&](const uint8_t* b, int j) {
    const uint8_t* q = b + (at_b ^ 64 * (j & 1)) + 4096 * (j >> 1);
    return join8(*reinterpret_cast<const v4i*>(q), *reinterpret_cast<const v4i*>(q + 1024));
  };
  auto get_x = [&](const float* x, int i) {
    const int r = r0 + 16 * i;
    return x[(g * NW + r / XW) * 64 + r % XW];
  };
  auto add = [&](int i, int j, float w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(T[j][e], w, acc[i][j][e]);
  };
  auto stage = [&](int k, float sw, uint8_t* ca, uint8_t* cb_, float* cx, uint8_t* na, uint8_t* nb, float* nx) {
    Half32 hb[FINE ? JB : 1];
    if constexpr (FINE) {
#pragma unroll
      for (int j = 0; j < JB; ++j) hb[j] = widen(fb[j]);
    }
#pragma unroll
    for (int i = 0; i < IA; ++i) {
      const float held = fx[(i + IA - 1) % IA % RING];  // the factor of the group before this one
      if (i == IA - AHEAD) {
        // every read of this stage's buffers is done or in registers: they may be filled again
        wait_vm_lgkm0<0>();
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
      }
      const int part = (i + AHEAD) % IA;  // this group's share of the loads
      const int from = part * PER, to = part < STEPS ? (from + PER < NL ? from + PER : NL) : from;
      const int ahead = (i + AHEAD) % IA;
      fa[ahead % RING] = get_a(i + AHEAD < IA ? ca : na, ahead);
      fx[ahead % RING] = get_x(i + AHEAD < IA ? cx : nx, ahead);
      fx[i % RING] *= sw;
      Half32 ha;
      if constexpr (FINE) ha = widen(fa[i % RING]);
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        add((i + IA - 1) % IA, j, held);
        v4f t = {};
        if constexpr (FINE) {
#pragma unroll
          for (int s = 0; s < 4; ++s) t = __builtin_amdgcn_mfma_f32_16x16x32_f16(hb[j].v[s], ha.v[s], t, 0, 0, 0);
        } else {
          t = mfma16(fb[j], fa[i % RING], t);
        }
        T[j] = t;
        if (i + 1 == IA) fb[j] = get_b(nb, j);
#pragma unroll
        for (int n = from + j; n < to; n += JB)
          i < IA - AHEAD ? issue(n, k + 1, na, nb, nx) : issue(n, k + 2, ca, cb_, cx);
      }
      if constexpr (!FINE) {
        __builtin_amdgcn_sched_group_barrier(0x100, 3, 0);
#pragma unroll
        for (int j = 0; j < JB; ++j) {
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          if (i + 1 == IA) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
          if (from + j < to) __builtin_amdgcn_sched_group_barrier(0x020, (PER + JB - 1) / JB, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int n = 0; n < NL; ++n) issue(n, 0, la0, lb0, lx0);
#pragma unroll
  for (int n = 0; n < FIRST; ++n) issue(n, 1, la1, lb1, lx1);
  wait_vm_lgkm0<FIRST>();
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) fa[i] = get_a(la0, i), fx[i] = get_x(lx0, i);
#pragma unroll
  for (int j = 0; j < JB; ++j) fb[j] = get_b(lb0, j);
  for (int kc = 0; kc < turns; kc += 64) {
    const int swv = __float_as_int(load_sw(kc));
    const int end = turns - kc < 64 ? turns : kc + 64;
    auto sw_at = [&](int k) { return __int_as_float(__builtin_amdgcn_readlane(swv, k - kc)); };
    int k = kc;
    for (; k + 2 <= end; k += 2) {
      stage(k, sw_at(k), la0, lb0, lx0, la1, lb1, lx1);
      stage(k + 1, sw_at(k + 1), la1, lb1, lx1, la0, lb0, lx0);
    }
    if (k < end) stage(k, sw_at(k), la0, lb0, lx0, la1, lb1, lx1);
  }
#pragma unroll
  for (int j = 0; j < JB; ++j) add(IA - 1, j, fx[(IA - 1) % RING]);  // the last group's results still wait
  auto owner = [&](int u) { return KG > 1 ? u % KG : g; };  // the K group that finishes unit u of 8 registers
  if constexpr (KG > 1) {
    // the K groups' sums meet in LDS, in a fixed order: each unit of 8 registers is finished by one group
    wait_vm_lgkm0<0>();
    __builtin_amdgcn_s_barrier();  // the buffers are free
    constexpr int REGS8 = IA * JB / 2;
    static_assert(KG * NW * REGS8 * 2048 <= 4 * ROOM && ROOM % 2048 == 0, "room for the sums");
    auto slot_of = [&](int grp, int u, int q) {
      const int at = ((grp * NW + wave) * REGS8 + u) * 2048 + q * 1024;
      return reinterpret_cast<v4f*>(one_of(at / ROOM, la0, la1, lb0, lb1) + at % ROOM + lane * 16);
    };
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const int u = (i * JB + j) / 2;
        if (owner(u) != g) *slot_of(g, u, j & 1) = acc[i][j];
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const int u = (i * JB + j) / 2;
        if (owner(u) != g) continue;
#pragma unroll
        for (int h = 1; h < KG; ++h) acc[i][j] += *slot_of((g + h) % KG, u, j & 1);
      }
  }
  // lane: token l16 of each group; of each pair of channel groups 8 consecutive channels
  const int64_t m1 = m0 + wr + l16, n1 = n0 + wc + 8 * l4;
  if (KG == 4 && part) {
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
      for (int u = 0; u < TJ; ++u) {
        if (owner(i * TJ + u) != g) continue;
        const int64_t m = m1 + 16 * i, n = n1 + 32 * u;
        if (m < o.M && n < ldp) {
          v4f* q = reinterpret_cast<v4f*>(part + ((int64_t)blockIdx.y * o.M + m) * ldp + n);
          q[0] = acc[i][2 * u], q[1] = acc[i][2 * u + 1];
        }
      }
    wait_vm_lgkm0<0>();
    return;
  }
  float bb[TJ][8];
#pragma unroll
  for (int u = 0; u < TJ; ++u)
#pragma unroll
    for (int e = 0; e < 8; ++e) bb[u][e] = o.bias && n1 + 32 * u + e < o.N ? o.bias[n1 + 32 * u + e] : kNoBias;
  auto finish = [&](auto whole) {  // whole: no bounds to check
    constexpr bool WHOLE = decltype(whole)::value;
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
      for (int u = 0; u < TJ; ++u)
        if (owner(i * TJ + u) == g) {
          const int64_t m = m1 + 16 * i, n = n1 + 32 * u;
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] = acc[i][2 * u + e / 4][e % 4] + bb[u][e];
          if (WHOLE || m < o.M) store8<OUT, WHOLE>(o, m, n, y);
        }
  };
  if (rows == BM && cols == BN) finish(std::true_type{});
  else finish(std::false_type{});
  wait_vm_lgkm0<0>();  // no load into LDS outlives the block, not the last ones without a range either
}

template <int WM, int WN, int IA, int TJ, int KG, int OUT>
__global__ __launch_bounds__(64 * WM * WN * KG, IA * TJ == 2 ? 4 : 2) void k9_tiles(
    const uint8_t* __restrict__ qX, int64_t ld, const uint8_t* __restrict__ qW, Scales sc, Out o, uint32_t tiles_m,
    uint32_t tiles_n, float* __restrict__ part, int64_t ldp) {
  constexpr int BM = 16 * IA * WM, BN = 32 * TJ * WN, ROWS = tile_rows(WM, WN, IA), ROOM = KG * (ROWS < BN ? ROWS : BN) * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t la0[KG * ROWS * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t la1[KG * ROWS * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t lb0[KG * BN * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t lb1[KG * BN * 128];
  __shared__ __attribute__((aligned(16))) float lx0[KG * WM * WN * 64], lx1[KG * WM * WN * 64];
  uint32_t m, n;
  const uint32_t xcd = blockIdx.x & 7, t8 = gridDim.x >> 3, r8 = gridDim.x & 7;
  tile_at(xcd * t8 + (xcd < r8 ? xcd : r8) + (blockIdx.x >> 3), tiles_m, tiles_n, m, n);
  tile<WM, WN, IA, TJ, KG, ROOM, OUT>(qX, ld, qW, sc, o, (int64_t)m * BM, (int64_t)n * BN, part, ldp, la0, la1, lb0, lb1,
                                      lx0, lx1);
}

// The second step of a K split: the parts' sums in order, then the bias.  A thread owns 8 columns.
__global__ __launch_bounds__(256) void k9_join(const float* __restrict__ part, int parts, int64_t ldp, Out o) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = ldp / 8;
  if (i >= o.M * per) return;
  const int64_t m = i / per, n = i % per * 8;
  float y[8] = {};
  for (int p = 0; p < parts; ++p) {
    const float4* q = reinterpret_cast<const float4*>(part + ((int64_t)p * o.M + m) * ldp + n);
    const float4 u = q[0], v = q[1];
    y[0] += u.x, y[1] += u.y, y[2] += u.z, y[3] += u.w, y[4] += v.x, y[5] += v.y, y[6] += v.z, y[7] += v.w;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] += o.bias && n + e < o.N ? o.bias[n + e] : kNoBias;
  if (o.ydtype == 0) store8<0, false>(o, m, n, y);
  else if (o.ydtype == 1) store8<1, false>(o, m, n, y);
  else store8<2, false>(o, m, n, y);
}

// ---- few tokens: v_mfma_f32_16x16x128_f8f6f4, weights straight from memory
//
// Bound by the weights' read.  A block of 8 waves owns 16 channels (one channel block of the weights' fragment order)
// and up to 16 NT tokens; its waves take the blocks of 128 along K in turn, U of them (2 KB each) in flight, and add
// their sums in LDS, in the waves' order.  The weights are the A operand, the tokens the B operand: lane l holds token
// l & 15 and 16 codes from k = 16 (l >> 4) of each half of the block.
constexpr int FEW_NW = 8, FEW_U = 3;
constexpr uint32_t kNoLoad = 0x7FFFFF00u;  // past the token rows' range (32 rows of at most 128 KB)

template <int NT>
struct FewSums {
  float v[FEW_NW][NT][64][4];
};

template <int NT>
__device__ __forceinline__ void few_finish(const v4f acc[NT], FewSums<NT>& sums, int wave, int lane, const Out& o,
                                           int64_t n0) {
#pragma unroll
  for (int t = 0; t < NT; ++t) *reinterpret_cast<v4f*>(&sums.v[wave][t][lane][0]) = acc[t];
  __syncthreads();
  for (int i = threadIdx.x; i < 256 * NT; i += 64 * FEW_NW) {
    const int c = i & 15, m = i >> 4;  // consecutive threads: consecutive channels
    const int64_t n = n0 + c;
    if (m >= o.M || n >= o.N) continue;
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < FEW_NW; ++w) y += sums.v[w][m >> 4][(m & 15) + 16 * (c >> 2)][c & 3];
    if (o.bias) y += o.bias[n];
    store1(o, m, n, y);
  }
}

template <int NT>
__global__ __launch_bounds__(64 * FEW_NW) void k9_few(const uint8_t* __restrict__ qX, int64_t ld,
                                                      const uint8_t* __restrict__ qW, Scales sc, Out o) {
  __shared__ FewSums<NT> sums;
  constexpr int U = FEW_U;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const uint8_t* wl = qW + n0 * ld + lane * 16;
  const __amdgpu_buffer_rsrc_t rX = make_rsrc(qX, (uint32_t)o.M * (uint32_t)ld);  // tokens past M read zeros
  const uint32_t xoff = (uint32_t)(lane & 15) * (uint32_t)ld + (uint32_t)(lane >> 4) * 16;
  const int nb = (int)sc.blocks;
  const float* sw = sc.sW + n0 / 128 * nb;
  const float* sx[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) sx[t] = sc.sX + ((lane & 15) + 16 * t < o.M ? (lane & 15) + 16 * t : 0);
  v4f acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = v4f{};
  for (int b0 = wave; b0 < nb; b0 += FEW_NW * U) {
    uint4 w[U][2], x[U][NT][2];
    float s[U][NT], c[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = b0 + u * FEW_NW, in = at < nb ? at : nb - 1;  // past the end: any weights, zero tokens, factor 0
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[u][h] = *reinterpret_cast<const uint4*>(wl + in * 2048 + h * 1024);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t off = (uint32_t)at * 128 + h * 64 + (uint32_t)(16 * t) * (uint32_t)ld + xoff;
          x[u][t][h] = buf_load16(rX, at < nb ? off : kNoLoad);
        }
      }
      c[u] = at < nb ? sw[in] : 0.0f;
#pragma unroll
      for (int t = 0; t < NT; ++t) s[u][t] = sx[t][in * sc.Mp];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        v4f d = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          d = dot32(w[u][h].x, w[u][h].y, x[u][t][h].x, x[u][t][h].y, d);
          d = dot32(w[u][h].z, w[u][h].w, x[u][t][h].z, x[u][t][h].w, d);
        }
        const float k = b0 + u * FEW_NW < nb ? s[u][t] * c[u] : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = fmaf(d[e], k, acc[t][e]);
      }
  }
  few_finish<NT>(acc, sums, wave, lane, o, n0);
}

// The whole layer for few tokens in one launch.  Blocks of 128 are quantized independently: four lanes take one, 32
// values each, so a workgroup does 128 of the M x nb at a time (one step up to 5 tokens of 3072 values), its first weights
// on their way; codes and scales go to LDS, and each wave takes the NU blocks that are its share of K (b = wave, wave +
// 8, ..) from there to registers.  Every workgroup repeats this (X is small and in L2), so it stays and takes `turns`
// channel blocks, the next one's weights on their way while one's sums meet in LDS (a workgroup to each channel block, every
// one of which quantizes: 24 us for 12 at 1x3072x18432; 57 MB at 4.7 TB/s).
template <typename T, int NU>
__global__ __launch_bounds__(64 * FEW_NW) void k9_few_layer(const T* __restrict__ X, int64_t ldx, int K, int64_t ld,
                                                            const uint8_t* __restrict__ qW, Scales sc, Out o, int turns) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // codes [M][nb][128], scales [M][nb]
  __shared__ FewSums<1> sums[2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t cbs = (o.N + 15) / 16, cb0 = (int64_t)blockIdx.x * turns, cb1 = cb0 + turns < cbs ? cb0 + turns : cbs;
  const int nb = (int)sc.blocks, l4 = lane >> 4, m = lane & 15, jobs = (int)o.M * nb;
  float* lds_s = reinterpret_cast<float*>(lds + jobs * 128);
  uint4 w[NU][2];
  float c[NU];
  auto load_w = [&](int64_t cb) {
    const uint8_t* wl = qW + cb * 16 * ld + lane * 16;
    const float* sw = sc.sW + (cb >> 3) * nb;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const int at = wave + u * FEW_NW, in = at < nb ? at : nb - 1;  // past the end: any weights, zero tokens
#pragma unroll
      for (int h = 0; h < 2; ++h) w[u][h] = *reinterpret_cast<const uint4*>(wl + in * 2048 + h * 1024);
      c[u] = sw[in];
    }
  };
  for (int j0 = wave * 16; j0 == wave * 16 || j0 < jobs; j0 += FEW_NW * 16) {
    const int j = j0 + m, row = j / nb, k0 = (j - row * nb) * 128 + 16 * l4;
    const T* x = X + (j < jobs ? row : 0) * ldx;
    Vec<T, 8> raw[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) raw[q] = load8(x, k0 + (q >> 1) * 64 + (q & 1) * 8, j < jobs ? K : 0);
    if (j0 == wave * 16) load_w(cb0);
    if (j0 >= jobs) break;
    float v[32], s, r;
    uint32_t a = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) valuev<T, 8>(raw[q], v + 8 * q);
#pragma unroll
    for (int e = 0; e < 32; ++e) a = umax(a, abs_bits(v[e]));
    const auto p = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    a = umax(p[0], p[1]);
    const auto t = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    a = umax(t[0], t[1]);
    block_scale(a, s, r);
    if (j < jobs) {
      if (l4 == 0) lds_s[j] = s;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 q;
        q.x = e4m3x4(v[16 * h], v[16 * h + 1], v[16 * h + 2], v[16 * h + 3], r);
        q.y = e4m3x4(v[16 * h + 4], v[16 * h + 5], v[16 * h + 6], v[16 * h + 7], r);
        q.z = e4m3x4(v[16 * h + 8], v[16 * h + 9], v[16 * h + 10], v[16 * h + 11], r);
        q.w = e4m3x4(v[16 * h + 12], v[16 * h + 13], v[16 * h + 14], v[16 * h + 15], r);
        *reinterpret_cast<uint4*>(lds + j * 128 + h * 64 + l4 * 16) = q;
      }
    }
  }
  __syncthreads();
  uint4 codes[NU][2];
  float s[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u) {
    const bool in = m < o.M && wave + u * FEW_NW < nb;
    const int j = in ? m * nb + wave + u * FEW_NW : 0;
    s[u] = in ? lds_s[j] : 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      codes[u][h] = in ? *reinterpret_cast<const uint4*>(lds + j * 128 + h * 64 + l4 * 16) : make_uint4(0, 0, 0, 0);
  }
  for (int64_t cb = cb0; cb < cb1; ++cb) {
    v4f acc[1] = {};
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      v4f d = {};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        d = dot32(w[u][h].x, w[u][h].y, codes[u][h].x, codes[u][h].y, d);
        d = dot32(w[u][h].z, w[u][h].w, codes[u][h].z, codes[u][h].w, d);
      }
      const float k = s[u] * c[u];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[0][e] = fmaf(d[e], k, acc[0][e]);
    }
    if (cb + 1 < cb1) load_w(cb + 1);
    few_finish<1>(acc, sums[(cb - cb0) & 1], wave, lane, o, cb * 16);
  }
}

template <int WM, int WN, int IA, int TJ, int KG>
void launch_tiles(const Fp8Plan& p, int64_t ld, const uint8_t* qX, const uint8_t* qW, const Scales& sc, const Out& o,
                  float* part, hipStream_t st) {
  constexpr int BM = 16 * IA * WM, BN = 32 * TJ * WN;
  const uint32_t tm = (uint32_t)((o.M + BM - 1) / BM), tn = (uint32_t)((o.N + BN - 1) / BN);
  const dim3 grid(tm * tn, (uint32_t)p.parts), block(64 * WM * WN * KG);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, st, qX, ld, qW, sc, o, tm, tn, part, p.ldp); };
  if constexpr (IA * TJ <= 8)  // (tiles of 256 columns have no registers for f16 operands)
    if (o.ydtype == 0) return go(k9_tiles<WM, WN, IA, TJ, KG, 0>);
  if (o.ydtype == 1) go(k9_tiles<WM, WN, IA, TJ, KG, 1>);
  else go(k9_tiles<WM, WN, IA, TJ, KG, 2>);
}

// ---- the choice of kernel
//
// By estimated time alone (us; S = blocks of 128 along K, c = workgroups that share a compute unit; a round of c takes
// a[c] S + b[c], a launch once more const).  The lines are least squares over 650 drawn sizes (256 CUs, launches back to
// back, inputs in turn; M x K x N); over 500 others the choice costs 1.0% (bf16) and 0.4% (fp32) more than the best.
// bf16 outputs, then fp32 ones (whose products in f16 take twice the MFMA time and the conversions besides):
//   few     up to 32 tokens, the weights' read: 1x3072x18432 11.2, 32x3072x18432 15.0 (240 sizes: 1.0% over the best)
//   64      one K group: 333x1000x1111 5.8 (64 x 2: 6.1, 128: 8.9) / 6.8; 154x768x2304 5.1 (5.4, 7.0) / 6.1
//   64 x 2  two K groups: 512x9216x3072 30.3 (64: 39.9, 128 x 2: 39.9) / 45.3 (53.2, 65.7)
//   64 x 4  four K groups, and K in parts of at least 8 blocks: 64x12288x3072 16.4 in 4 parts, 28.3 in one, 64 x 2 33.8 /
//           17.2, 30.8, 34.6
//   128     4608x3072x9216 150 (64: 200) / 252 (325)
//   128 x 2 two K groups: 1024x4096x4096 24.6 (128: 27.8, 64: 29.4) / 40.4 (44.7, 46.3)
//   256     4096x4096x4096 59 (128: 73); bf16 outputs only
//   224, 192  rows by 256 columns: where they leave a last round emptier or save one.  192: 3000x5000x3500 53 (256: 62, 224:
//           57), 6670x9062x2561 181 (214, 198), 2048x1280x5120 20 (22.8, 22), but 4608x12288x3072 222; 224: that 150 (159),
//           4608x3072x9216 124 (126, 192: 135), 4609x2196x5826 65 (69, 81).  Over 59 drawn sizes 256 alone costs 4.7% more.
//           (Cutting the last round's tiles of 256 into halves gained 4% on those alone and lost 4% to 192 and 224.)
struct Cost {
  double us;
  int rows, cols, groups, parts;
};

Cost tiles_cost(int64_t M, int64_t N, int S, int cus, int tile, int groups, bool fine) {
  const int cols = tile > 128 ? 256 : tile;
  const double T = (double)((M + tile - 1) / tile) * (double)((N + cols - 1) / cols);
  const double rounds = T / cus;
  double us = 0.0;
  auto by_line = [&](const double* a, const double* b, int most) {  // a[c - 1], b[c - 1]: c blocks on a CU
    const double full = (double)(int64_t)(rounds / most), rest = rounds - full * most;
    us = full * (a[most - 1] * S + b[most - 1]);
    if (rest > 0) us += a[(int)(rest + 0.999999) - 1] * S + b[(int)(rest + 0.999999) - 1];
  };
  // [0] bf16 outputs, [1] fp32
  static const double a64[2][4] = {{0.334, 0.504, 0.546, 0.719}, {0.414, 0.603, 0.834, 1.062}},
                      b64[2][4] = {{0.0, 0.88, 1.95, 2.86}, {0.0, 1.4, 2.9, 3.34}},
                      a642[2][2] = {{0.296, 0.342}, {0.324, 0.515}}, b642[2][2] = {{0.0, 2.44}, {0.0, 2.17}},
                      a644[2][1] = {{0.2}, {0.258}}, b644[2][1] = {{5.53}, {5.94}},
                      a128[2][2] = {{0.629, 0.939}, {0.914, 1.58}}, b128[2][2] = {{2.31, 4.45}, {2.89, 6.71}},
                      a1282[2][1] = {{0.485}, {0.781}}, b1282[2][1] = {{6.83}, {9.38}};
  // tiles of 256, 224 and 192 rows, one to a CU: a step of a round of up to 30% of the CUs, of all, and between the two
  // along a line (the more of them work, the lower their clock)
  static const double few256[3] = {1.049, 0.945, 0.752}, all256[3] = {1.555, 1.44, 1.3}, b256[3] = {8.15, 7.19, 6.53},
                      once[3] = {1.53, 2.32, 1.97};
  if (tile == 64 && groups == 1) by_line(a64[fine], b64[fine], 4), us += fine ? 3.2 : 2.84;
  else if (tile == 64 && groups == 2) by_line(a642[fine], b642[fine], 2), us += fine ? 4.1 : 3.23;
  else if (tile == 64) by_line(a644[fine], b644[fine], 1);
  else if (tile == 128 && groups == 1) by_line(a128[fine], b128[fine], 2), us += fine ? 3.77 : 2.1;
  else if (tile == 128) by_line(a1282[fine], b1282[fine], 1);
  else {
    const int h = (256 - tile) / 32;  // 256, 224, 192 rows
    const double full = (double)(int64_t)rounds, rest = rounds - full;
    const double u = rest <= 0.3 ? 0.0 : (rest - 0.3) / 0.7;
    us = full * (all256[h] * S + b256[h]) + once[h];
    if (rest > 0) us += ((1 - u) * few256[h] + u * all256[h]) * S + b256[h];
  }
  return Cost{us, tile, cols, groups, 1};
}

}  // namespace

Fp8Plan plan_fp8(int64_t M, int64_t K, int64_t N, bool fine) {
  const int cus = device_cus();
  const int64_t ld = i8_ld(K), ldp = (N + 7) / 8 * 8;
  const int S = (int)(ld / 128);
  Cost best{1e30, 64, 64, 1, 1};
  auto take = [&](const Cost& c) {
    if (c.us < best.us) best = c;
  };
  take(tiles_cost(M, N, S, cus, 64, 1, fine));
  take(tiles_cost(M, N, S, cus, 128, 1, fine));
  if (!fine)
    for (int rows : {256, 224, 192}) take(tiles_cost(M, N, S, cus, rows, 1, fine));
  const int64_t T64 = ((M + 63) / 64) * ((N + 63) / 64), T128 = ((M + 127) / 128) * ((N + 127) / 128);
  if (T128 <= cus) take(tiles_cost(M, N, S, cus, 128, 2, fine));
  if (T64 <= 2 * cus) take(tiles_cost(M, N, S, cus, 64, 2, fine));
  if (T64 <= cus) {
    for (int parts = 1; parts <= 8 && parts * T64 <= cus && (parts == 1 || S / parts >= 8); parts *= 2) {
      const int per = (S + parts - 1) / parts;
      Cost c = tiles_cost(M, N, per, cus, 64, 4, fine);
      c.parts = (S + per - 1) / per;  // no empty part
      if (c.parts > 1) c.us += 2.4 + 5.2e-6 * (double)(M * ldp) * c.parts;
      take(c);
    }
  }
  if (M <= 32) {  // the weights' bytes, the workgroups' starts and a wave's steps along K; a second set of 16 tokens
    const double more = M > 16, n = (double)N, k = (double)ld;
    take(Cost{2.62 + n * k * 1e-6 * (0.132 + 0.11 * more) + n * 1e-3 * (0.053 + 0.111 * more) + k * 3.5e-4, 0, 16, 1, 1});
  }
  Fp8Plan p{best.rows, best.cols, best.groups, best.parts, ldp, 0};
  if (p.parts > 1) p.bytes = (size_t)p.parts * (size_t)M * (size_t)ldp * 4;
  return p;
}

// Up to 256 blocks of X: with a bf16 output 1x3072x18432 takes 11.7 us in one launch and 13.0 in two, 10x3072x18432 13.0 and
// 17.2, 1x768x768 3.6 and 5.2, 8x3072x9216 10.5 and 10.0; 12x4096x4096 (384 blocks) 9.0 and 8.8, 16x4096x16384 19.5 and 19.3.
// A launch more is 3 us of the caller's time besides.
bool few_layer_fp8(int64_t M, int64_t K) { return M <= 16 && K <= 4 * FEW_NW * 128 && M * fp8_blocks(K) <= 256; }

hipError_t launch_few_layer_fp8(int64_t M, int64_t K, int64_t N, const void* X, int xdtype, int64_t ldx,
                                const uint8_t* qW, const float* sW, const float* bias, void* Y, int64_t ldy, int ydtype,
                                hipStream_t st) {
  const Out o{nullptr, nullptr, bias, Y, ldy, M, N, ydtype};
  const Scales sc{nullptr, sW, 0, fp8_blocks(K)};
  // as many workgroups as the card holds (two to a unit), and no more turns than that takes
  const int64_t ld = i8_ld(K), cbs = (N + 15) / 16, most = 2 * (int64_t)device_cus(), turns = (cbs + most - 1) / most;
  const dim3 g((uint32_t)((cbs + turns - 1) / turns)), b(64 * FEW_NW);
  const size_t lds = (size_t)(M * sc.blocks) * 132;  // at most 33 KB: up to 256 blocks run here
  auto typed = [&](auto x) {
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, g, b, lds, st, x, ldx, (int)K, ld, qW, sc, o, (int)turns); };
    typedef typename std::remove_const<typename std::remove_pointer<decltype(x)>::type>::type T;
    const int64_t nu = (sc.blocks + FEW_NW - 1) / FEW_NW;
    if (nu <= 1) go(k9_few_layer<T, 1>);
    else if (nu <= 2) go(k9_few_layer<T, 2>);
    else if (nu <= 3) go(k9_few_layer<T, 3>);
    else go(k9_few_layer<T, 4>);
  };
  if (xdtype == 0) typed(static_cast<const float*>(X));
  else typed(static_cast<const uint16_t*>(X));
  return hipGetLastError();
}

hipError_t launch_gemm_fp8(int64_t M, int64_t K, int64_t N, const uint8_t* qX, const float* sX, const uint8_t* qW,
                           const float* sW, const float* bias, void* Y, int64_t ldy, int ydtype, void* ws,
                           hipStream_t st) {
  const int64_t ld = i8_ld(K);
  const Out o{nullptr, nullptr, bias, Y, ldy, M, N, ydtype};
  const Scales sc{sX, sW, fp8_pad(M), fp8_blocks(K)};
  const Fp8Plan p = plan_fp8(M, K, N, ydtype == 0);
  if (p.rows == 0) {
    const dim3 g((uint32_t)((N + 15) / 16)), b(64 * FEW_NW);
    if (M <= 16) hipLaunchKernelGGL(k9_few<1>, g, b, 0, st, qX, ld, qW, sc, o);
    else hipLaunchKernelGGL(k9_few<2>, g, b, 0, st, qX, ld, qW, sc, o);
    return hipGetLastError();
  }
  float* part = p.parts > 1 ? static_cast<float*>(ws) : nullptr;
  if (p.rows == 256) launch_tiles<2, 4, 8, 2, 1>(p, ld, qX, qW, sc, o, part, st);
  else if (p.rows == 224) launch_tiles<2, 4, 7, 2, 1>(p, ld, qX, qW, sc, o, part, st);
  else if (p.rows == 192) launch_tiles<2, 4, 6, 2, 1>(p, ld, qX, qW, sc, o, part, st);
  else if (p.rows == 128 && p.groups == 1) launch_tiles<2, 2, 4, 2, 1>(p, ld, qX, qW, sc, o, part, st);
  else if (p.rows == 128) launch_tiles<2, 2, 4, 2, 2>(p, ld, qX, qW, sc, o, part, st);
  else if (p.groups == 1) launch_tiles<2, 2, 2, 1, 1>(p, ld, qX, qW, sc, o, part, st);
  else if (p.groups == 2) launch_tiles<2, 2, 2, 1, 2>(p, ld, qX, qW, sc, o, part, st);
  else launch_tiles<2, 2, 2, 1, 4>(p, ld, qX, qW, sc, o, part, st);
  if (p.parts > 1)
    hipLaunchKernelGGL(k9_join, dim3((uint32_t)((M * (p.ldp / 8) + 255) / 256)), dim3(256), 0, st, part, p.parts, p.ldp, o);
  return hipGetLastError();
}

}  // namespace svdq
